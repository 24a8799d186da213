// hold_tmem.cu -- in the bounded-wait tests' copy of the library only: a kernel that
// holds the tensor memory of every SM for a while, for kernels that have to wait for
// their columns.
#include "sm100.cuh"

namespace {

constexpr uint64_t kMaxHoldNs = 100000000ull;
constexpr int kSms = 148;
constexpr int kSmemBytes = 117000;       // one CTA per SM, and a CTA of half an SM beside it

__global__ void hold_tmem_kernel(uint64_t ns) {
    extern __shared__ uint8_t dyn[];
    __shared__ uint32_t slot;
    gdr::tmem_alloc(&slot, 512);
    __syncwarp();
    const uint32_t tmem = *(volatile uint32_t*)&slot;
    const uint64_t t0 = gdr::global_timer_ns();
    while (gdr::global_timer_ns() - t0 < (ns < kMaxHoldNs ? ns : kMaxHoldNs)) __nanosleep(1000);
    __syncwarp();
    gdr::tmem_dealloc(tmem, 512);
}

}  // namespace

extern "C" int gdr_test_hold_tmem(uint64_t ns, void* stream) {
    const cudaError_t e = cudaFuncSetAttribute(hold_tmem_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return (int)e;
    hold_tmem_kernel<<<kSms, 32, kSmemBytes, static_cast<cudaStream_t>(stream)>>>(ns);
    return (int)cudaGetLastError();
}
