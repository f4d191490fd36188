// Host interface of the bounded-wait self-test (selftest.cu).
#pragma once

#include <cuda_runtime.h>

namespace attn {
namespace selftest {

cudaError_t launch_wait(int complete, cudaStream_t s);
cudaError_t status_word(int** word);

}  // namespace selftest
}  // namespace attn
