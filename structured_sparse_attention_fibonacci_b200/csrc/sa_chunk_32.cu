// The chunk attention's kernels for head dim 32.
#define SA_CHUNK_KERNELS
#include "sa_chunk.cuh"

namespace sa {
template cudaError_t launch_chunk_of<32>(const ChunkArgs&, bool, bool, cudaStream_t);
template cudaError_t chunk_error_of<32>(unsigned*, bool);
}  // namespace sa
