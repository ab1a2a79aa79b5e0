// Decode attention kernels: bf16 caches.
#include "decode_kernel.cuh"

namespace mla {
namespace decode {

Kernel kernel_bf16(int dp, int nt) { return kernel_for<kBf16>(dp, nt); }
int bf16_status(bool clear) { return read_status(clear); }

}  // namespace decode
}  // namespace mla
