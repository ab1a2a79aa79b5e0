// Decode attention kernels: fp32 caches.
#include "decode_kernel.cuh"

namespace mla {
namespace decode {

Kernel kernel_fp32(int dp, int nt) { return kernel_for<kFp32>(dp, nt); }
int fp32_status(bool clear) { return read_status(clear); }

}  // namespace decode
}  // namespace mla
