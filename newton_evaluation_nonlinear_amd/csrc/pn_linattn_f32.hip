// The chunk kernels of linear attention for float32 storage.
#include "pn_linattn_chunk.hpp"

namespace pn {
template hipError_t launch_chunks<float>(const LaChunkArgs&, bool, hipStream_t);
}  // namespace pn
