// The chunk kernels of linear attention for binary16 storage.
#include "pn_linattn_chunk.hpp"

namespace pn {
template hipError_t launch_chunks<f16>(const LaChunkArgs&, bool, hipStream_t);
}  // namespace pn
