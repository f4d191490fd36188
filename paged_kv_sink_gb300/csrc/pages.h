// Host/device interface of the pages' bookkeeping (pages.cu).
//
// refs[p] is the number of page-table entries that hold page p (0: free).  A request of
// L tokens holds its row's first ceil(L / page_size) entries.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace attn {
namespace pages {

constexpr int kMaxPools = 8;

// The tensors whose pages move together: (num_pages, bytes).
struct Pools {
    void* base[kMaxPools];
    long long bytes[kMaxPools];  // of a page
    int pieces[kMaxPools];       // (set by the launches) work items of a page
    int count;
};

struct Table {
    int32_t* table;  // (batch, max_pages)
    int32_t* refs;   // (num_pages,)
    int batch, max_pages, page_size, num_pages;
};

size_t reserve_scratch(const Table& t);
size_t compact_scratch(const Table& t);
// A copy from page src[i] to dst[i] for i < *count (count NULL: n); either one outside
// the pool: none.
cudaError_t launch_copy(const Pools& p, const int32_t* src, const int32_t* dst, const int32_t* count, int n, int num_pages,
                        bool report, cudaStream_t s);
cudaError_t launch_fork(const Table& t, const int32_t* seqlens, const int32_t* src, int out_batch, int32_t* out_table,
                        int32_t* out_seqlens, cudaStream_t s);
cudaError_t launch_release(const Table& t, const int32_t* seqlens, const int32_t* new_seqlens, cudaStream_t s);
cudaError_t launch_reserve(const Pools& p, const Table& t, const int32_t* seqlens, const int32_t* new_seqlens,
                           int32_t* missing, void* scratch, cudaStream_t s);
cudaError_t launch_compact(const Pools& p, const Table& t, const int32_t* seqlens, int32_t* held, void* scratch,
                           cudaStream_t s);
cudaError_t status_word(int** word);

}  // namespace pages
}  // namespace attn
