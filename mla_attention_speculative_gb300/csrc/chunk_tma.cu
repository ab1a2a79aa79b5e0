// The chunk attention's tensor-core kernels: bf16 caches whose pages are whole runs of 8 rows.

#include "chunk_sm103.cuh"

namespace mla {
namespace chunk {

Kernel kernel_tma(int dim) { return pick<kTma>(dim); }
int tma_status(bool clear) { return read_status(clear); }

}  // namespace chunk
}  // namespace mla
