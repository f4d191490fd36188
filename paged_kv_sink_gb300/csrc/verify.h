// Host/device interface of the verification of drafted tokens (verify.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace attn {
namespace verify {

enum { kF32 = 0, kBF16 = 1, kF16 = 2 };
constexpr int kMaxNodes = 256;  // of a request

struct Args {
    const void* target;        // (total, vocab) probabilities after each node
    const void* draft;         // (total, vocab), or NULL
    long long target_rs, draft_rs;  // row strides, elements
    const int32_t* tokens;     // (total,)
    const int32_t* parents;    // (total,), or NULL: each node hangs on the one before it
    const int32_t* cu;         // (batch+1,)
    const float* u;            // (total,) for the tests
    const float* u_next;       // (batch,) for the next token
    const int32_t* base;       // (batch,), or NULL: 0
    int32_t* src;              // (batch, max_nodes)
    int32_t* counts;           // (batch,)
    int32_t* next;             // (batch,)
    int batch, total, max_nodes, vocab, dtype;
};

cudaError_t launch(const Args& a, cudaStream_t s);
cudaError_t status_word(int** word);

}  // namespace verify
}  // namespace attn
