// The chunk attention's tensor-core kernels: e4m3 caches.

#include "chunk_sm103.cuh"

namespace mla {
namespace chunk {

Kernel kernel_convert(int dim) { return pick<kConvert>(dim); }
int convert_status(bool clear) { return read_status(clear); }

}  // namespace chunk
}  // namespace mla
