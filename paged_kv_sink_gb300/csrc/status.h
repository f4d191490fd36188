// Reading the units' status words (status.cu).
#pragma once

#include <cuda_runtime.h>

namespace attn {
namespace status {

constexpr int kMaxWords = 32;

struct Words {
    int* at[kMaxWords];  // on the current device; NULL: none
};

// Takes the bits of all words, leaves 0 in them, and returns their OR; synchronises `s`.
cudaError_t exchange(const Words& words, cudaStream_t s, int* bits);

}  // namespace status
}  // namespace attn
