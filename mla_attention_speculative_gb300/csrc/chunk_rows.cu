// The chunk attention's tensor-core kernels: bf16 caches of any other page size.

#include "chunk_sm103.cuh"

namespace mla {
namespace chunk {

Kernel kernel_rows(int dim) { return pick<kRows>(dim); }
int rows_status(bool clear) { return read_status(clear); }

}  // namespace chunk
}  // namespace mla
