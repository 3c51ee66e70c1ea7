// Launch interface of the page kernels (pages.cu) for the C-ABI layer. Which pages a sequence holds is
// in table (slots, max_pages) int32, -1: none; lens (slots) counts its tokens; refs (pages) counts the
// table entries that name a page: a page with none is free.
#pragma once

#include <cuda_runtime.h>

namespace attn {

struct PageState {
    int* table;
    int* lens;
    int* refs;
    int pages, slots, max_pages, page_size;
};

constexpr int kPagesMaxSeqs = 8192;           // sequences per reserve / fork call
constexpr int kPagesMaxSlots = 1 << 18;       // table rows (a bitmap of them lies in shared memory)
constexpr int kPagesMaxPages = 0x7fffffff - 8192;   // the scans' 32-bit indices pass the last page by up to
                                                    // a tile (4096 pages)

cudaError_t launch_pages_reserve(const PageState& s, const int* seqs, const int* counts, int* start,
                                 int n, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageState& s, const int* src, const int* dst, int* from, int* to,
                              int n, cudaStream_t stream);
cudaError_t launch_pages_free(const PageState& s, const int* seqs, int n, int whole, int wl, int ns,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const PageState& s, int* from, int* to, int* count, int* ws,
                                 cudaStream_t stream);
cudaError_t launch_pages_copy(void* pool, const int* from, const int* to, const int* count, int layers,
                              int pages, long long page_bytes, int n, cudaStream_t stream);

}  // namespace attn
