// Decode attention kernels: e4m3 caches.
#include "decode_kernel.cuh"

namespace mla {
namespace decode {

Kernel kernel_e4m3(int dp, int nt) { return kernel_for<kE4m3>(dp, nt); }
int e4m3_status(bool clear) { return read_status(clear); }

}  // namespace decode
}  // namespace mla
