// The sticky status words of all units, read and cleared by one warp (sm_103a).
//
// Each unit has a word of its own (common.cuh).  One launch, one copy of 4 bytes and one wait read
// them all, however many units there are (22 us a call; a copy and a wait a word, there and
// back, took 222 with 12 of them).  The exchange is atomic, so that a bit that another stream raises
// meanwhile is in this answer or the next.  No memory is allocated: callers may forbid it.
#include "status.h"

#include <atomic>

namespace attn {
namespace status {

constexpr int kSlots = 256;  // calls in flight at once have a slot each
static __device__ int g_slots[kSlots];

__global__ void __launch_bounds__(kMaxWords) exchange_kernel(const Words words, int slot) {
    int* const word = words.at[threadIdx.x];
    const int bits = (int)__reduce_or_sync(0xffffffffu, word ? (unsigned)atomicExch(word, 0) : 0u);
    if (threadIdx.x == 0) g_slots[slot] = bits;
}

cudaError_t exchange(const Words& words, cudaStream_t s, int* bits) {
    static std::atomic<unsigned> calls{0};
    const int slot = (int)(calls.fetch_add(1, std::memory_order_relaxed) % kSlots);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kMaxWords);
    cfg.stream = s;
    cudaError_t e = cudaLaunchKernelEx(&cfg, exchange_kernel, words, slot);
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbolAsync(bits, g_slots, sizeof(int), slot * sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e;
}

}  // namespace status
}  // namespace attn
