// The chunk kernels of linear attention for bfloat16 storage.
#include "pn_linattn_chunk.hpp"

namespace pn {
template hipError_t launch_chunks<bf16>(const LaChunkArgs&, bool, hipStream_t);
}  // namespace pn
