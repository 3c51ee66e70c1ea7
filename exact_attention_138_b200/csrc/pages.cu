// Pages of a K/V cache: reserving them for new tokens, forking and freeing sequences, compacting the
// pool, and moving page contents (state: pages.h). All of it runs on the device, so that a decode step
// that admits, forks and ends sequences needs no read-back and can be captured into a graph.
//
// Results depend on the state alone, not on timing: free pages are handed out from the lowest number up
// in the order of the requests, and reference counts change by integer atomics. A reserve or fork that
// cannot be served (too few free pages, an index out of range or given twice, no room in the table)
// changes nothing, marks its results with -1 and sets the device status; free passes over rows out of
// range, serves the others and sets it too.
//
// What bounds them: the page copies by HBM; the others are a chain of a few dependent reads (sequence
// -> length -> table entry -> count), so they are launched once, as one cluster of up to 8 CTAs that
// scans the counts in parallel and agrees through distributed shared memory.
#include <cooperative_groups.h>

#include "kernels.h"
#include "pages.h"
#include "sm100_ptx.cuh"

namespace attn {

namespace {

constexpr int kPgThreads = 1024, kPgWarps = kPgThreads / 32;
constexpr int kPgTile = 4 * kPgThreads;       // pages one CTA looks at per step, 4 per thread
static_assert(kPagesMaxPages <= 0x7fffffff - 2 * kPgTile, "scan indices");
constexpr int kPgCluster = 8;
constexpr int kErrPages = 6;                  // ATTN_ERR_PAGES

// Inclusive prefix sums over the CTA's threads, with one barrier each: every warp scans the warps' sums
// for itself, and two buffers take turns, so that one is rewritten only a barrier after it was read.
struct BlockScan {
    long long* sums;      // 2 x kPgWarps
    int turn = 0;
    __device__ __forceinline__ long long operator()(long long v, long long* total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        long long* buf = sums + turn * kPgWarps;
        turn ^= 1;
        if (lane == 31) buf[warp] = v;
        __syncthreads();
        long long s = buf[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        *total = __shfl_sync(0xffffffffu, s, kPgWarps - 1);
        const long long before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
        return warp > 0 ? v + before : v;
    }
};
static_assert(kPgWarps == 32, "one lane per warp's sum");

// refs of pages p .. p+3 (p a multiple of 4); pages past the end read as in use.
__device__ __forceinline__ int4 refs4(const int* refs, int p, int pages) {
    if (p + 4 <= pages) return *reinterpret_cast<const int4*>(refs + p);
    int4 r = make_int4(1, 1, 1, 1);
    if (p < pages) r.x = refs[p];
    if (p + 1 < pages) r.y = refs[p + 1];
    if (p + 2 < pages) r.z = refs[p + 2];
    return r;
}

// Pages of one CTA of a cluster of `ctas`: whole tiles, [begin, end).
__device__ __forceinline__ void slice_of(int pages, int rank, int ctas, int& begin, int& end) {
    const long long each = (static_cast<long long>(pages) + static_cast<long long>(ctas) * kPgTile - 1) /
                           (static_cast<long long>(ctas) * kPgTile) * kPgTile;
    begin = static_cast<int>(min(each * rank, static_cast<long long>(pages)));
    end = static_cast<int>(min(each * (rank + 1), static_cast<long long>(pages)));
}

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Reserve (FORK false): sequence seqs[i] grows by counts[i] tokens; start[i] gets its length before.
// Fork (FORK true): dst[i] becomes a copy of src[i] that shares its full pages; a partly filled last
// page gets a page of its own, and from[i] -> to[i] is the copy the caller has to make.
template <bool FORK>
__global__ void __launch_bounds__(kPgThreads) pages_take_kernel(const PageState s, const int* __restrict__ seqs,
                                                                const int* __restrict__ arg, int* out0,
                                                                int* out1, int n, int ctas) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t* marks = reinterpret_cast<uint32_t*>(smem);                 // table rows of this call
    const int words = (s.slots + 31) / 32;
    int* pre = reinterpret_cast<int*>(marks + words);                    // pages needed before entry i
    int* len = pre + n + 1;                                              // tokens before the call
    __shared__ long long sums[2 * kPgWarps];
    __shared__ int isums[kPgWarps];
    __shared__ int free_here;
    BlockScan scan{sums};
    const int rank = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
    const int cap = s.max_pages * s.page_size;
    // ---- free pages of this CTA's slice (their counts arrive while the entries are read)
    int begin, end;
    slice_of(s.pages, rank, ctas, begin, end);
    int mine = 0;
    int4 r4 = make_int4(1, 1, 1, 1);
    for (int p = begin + 4 * tid; p < end; p += kPgTile) {
        r4 = refs4(s.refs, p, s.pages);
        mine += (r4.x == 0) + (r4.y == 0) + (r4.z == 0) + (r4.w == 0);
    }
    // ---- the call's entries: in range, each row once, room in the table (every CTA for itself)
    for (int i = tid; i < words; i += kPgThreads) marks[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < n; i += kPgThreads) {
        const int q = seqs[i];
        if (q < 0 || q >= s.slots) {
            bad = true;
            continue;
        }
        bad |= (atomicOr(&marks[q >> 5], 1u << (q & 31)) >> (q & 31) & 1u) != 0;
    }
    __syncthreads();
    long long need_all = 0;
    for (int base = 0; base < n; base += kPgThreads) {
        const int i = base + tid;
        long long need = 0;
        if (i < n) {
            const int q = FORK ? arg[i] : seqs[i];
            int have = 0;
            if (q < 0 || q >= s.slots) {
                bad = true;
            } else {
                have = s.lens[q];
                bad |= have < 0 || have > cap;
                if (FORK) {
                    bad |= (marks[q >> 5] >> (q & 31) & 1u) != 0;        // copied and replaced at once
                    const int d = seqs[i];
                    bad |= d >= 0 && d < s.slots && s.lens[d] != 0;      // only onto an empty sequence
                    need = have % s.page_size != 0;
                } else {
                    const int c = arg[i];
                    bad |= c < 0 || (!bad && c > cap - have);
                    if (!bad) need = ceil_div(have + c, s.page_size) - ceil_div(have, s.page_size);
                }
            }
            len[i] = have;
        }
        long long part;
        const long long incl = scan(need, &part);
        if (i < n) pre[i] = static_cast<int>(min(need_all + incl - need, 0x7fffffffLL));
        need_all += part;
    }
    if (tid == 0) pre[n] = static_cast<int>(min(need_all, 0x7fffffffLL));
    long long total;
    const long long mine_incl = scan(mine, &total);
    if (tid == 0) free_here = static_cast<int>(total);
    bad = __syncthreads_or(bad);
    cluster.sync();                                    // all have read lens, all counts are there
    int before = 0, free_all = 0;
    for (int x = 0; x < ctas; ++x) {
        const int f = *cluster.map_shared_rank(&free_here, x);
        if (x < rank) before += f;
        free_all += f;
    }
    const bool refused = bad || need_all > free_all;
    const int want = refused ? 0 : static_cast<int>(need_all);
    // ---- the r-th free page goes to the r-th request
    for (int p0 = begin; p0 < end && before < want; p0 += kPgTile) {
        const int p = p0 + 4 * tid;
        if (end - begin > kPgTile) r4 = p < end ? refs4(s.refs, p, s.pages) : make_int4(1, 1, 1, 1);
        const int zero[4] = {r4.x == 0, r4.y == 0, r4.z == 0, r4.w == 0};
        const int here = zero[0] + zero[1] + zero[2] + zero[3];
        long long tile = total, incl = mine_incl;          // a slice of one tile has been scanned
        if (end - begin > kPgTile) incl = scan(here, &tile);
        int r = before + static_cast<int>(incl) - here;
        before += static_cast<int>(tile);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!zero[e]) continue;
            if (r < want) {
                int a = 0, b = n - 1;                  // the last entry with pre[i] <= r
                while (a < b) {
                    const int m = (a + b + 1) / 2;
                    if (pre[m] <= r) a = m;
                    else b = m - 1;
                }
                const int slot = (FORK ? len[a] / s.page_size : ceil_div(len[a], s.page_size)) + r - pre[a];
                s.table[static_cast<size_t>(seqs[a]) * s.max_pages + slot] = p + e;
                s.refs[p + e] = 1;
                if (FORK) {
                    const int old = s.table[static_cast<size_t>(arg[a]) * s.max_pages + slot];
                    const bool held = old >= 0 && old < s.pages;
                    out0[a] = held ? old : -1;
                    out1[a] = held ? p + e : -1;
                }
            }
            ++r;
        }
    }
    if (FORK && !refused) {
        // shared pages: (entry, 128 pages) per warp
        int longest = 0;
        for (int i = tid; i < n; i += kPgThreads) longest = max(longest, len[i] / s.page_size);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
        if ((tid & 31) == 0) isums[tid >> 5] = longest;
        __syncthreads();
        for (int w = 0; w < kPgWarps; ++w) longest = max(longest, isums[w]);
        const int chunks = (longest + 127) / 128;
        const long long jobs = static_cast<long long>(n) * chunks;
        for (long long j = rank * kPgWarps + (tid >> 5); j < jobs; j += ctas * kPgWarps) {
            const int i = static_cast<int>(j / chunks), m0 = static_cast<int>(j % chunks) * 128 + (tid & 31);
            const int full = len[i] / s.page_size;
            const int* from = s.table + static_cast<size_t>(arg[i]) * s.max_pages;
            int* to = s.table + static_cast<size_t>(seqs[i]) * s.max_pages;
            int pg[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pg[e] = m0 + 32 * e < full ? from[m0 + 32 * e] : -1;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m0 + 32 * e < full) {
                    to[m0 + 32 * e] = pg[e];
                    if (pg[e] >= 0 && pg[e] < s.pages) atomicAdd(&s.refs[pg[e]], 1);
                }
        }
    }
    if (rank == 0) {
        for (int i = tid; i < n; i += kPgThreads) {
            if (FORK) {
                if (refused || pre[i + 1] == pre[i]) out0[i] = out1[i] = -1;
                if (!refused) s.lens[seqs[i]] = len[i];
            } else {
                out0[i] = refused ? -1 : len[i];
                if (!refused) s.lens[seqs[i]] = len[i] + arg[i];
            }
        }
        if (refused && tid == 0) report_refusal(kErrPages);
    }
    cluster.sync();                                    // free_here may still be read by a neighbour
}

// One CTA per sequence: its pages (whole), or those that no query from its next token on can see
// under a window of wl keys and ns sinks, lose a reference. Entries are taken with an exchange, so a
// row given twice gives its pages back once.
__global__ void __launch_bounds__(256) pages_free_kernel(const PageState s, const int* __restrict__ seqs,
                                                         int whole, int wl, int ns) {
    const int q = seqs[blockIdx.x];
    if (q < 0 || q >= s.slots) {
        if (threadIdx.x == 0) report_refusal(kErrPages);
        return;
    }
    const long long cap = static_cast<long long>(s.max_pages) * s.page_size;
    const long long len = min(max(static_cast<long long>(s.lens[q]), 0LL), cap);
    __syncthreads();
    long long m0 = 0, m1 = (len + s.page_size - 1) / s.page_size;
    if (!whole) {
        m0 = (static_cast<long long>(ns) + s.page_size - 1) / s.page_size;
        m1 = len > wl ? (len - wl) / s.page_size : 0;
    }
    int* row = s.table + static_cast<size_t>(q) * s.max_pages;
#pragma unroll 4
    for (long long m = m0 + threadIdx.x; m < m1; m += blockDim.x) {
        if (row[m] < 0) continue;
        const int pg = atomicExch(&row[m], -1);
        if (pg >= 0 && pg < s.pages) atomicSub(&s.refs[pg], 1);
    }
    if (whole && threadIdx.x == 0) s.lens[q] = 0;
}

// Compaction, second part: the table's entries and the counts follow the pages (all threads of the
// grid). A rank is read for entries that name a page in use, which is in the plan; others are left.
__device__ __forceinline__ void pages_follow(int* table, long long entries, int* refs, int pages, const int* from,
                                             const int* to, const int* rank_of, int low, int all) {
    if (all == 0) return;
    const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long nt = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long r = t0; r < all; r += nt) {
        const int a = from[r];
        refs[to[r]] = refs[a];
        refs[a] = 0;
    }
#pragma unroll 4
    for (long long i = t0; i < entries; i += nt) {
        const int p = table[i];
        if (p < low || p >= pages) continue;
        const int r = rank_of[p];
        if (r >= 0 && r < all && from[r] == p) table[i] = to[r];
    }
}

// Compaction, first part: with L pages in use, those numbered L and above (movers) go to the free
// pages below L (holes), both in ascending order. from[r] -> to[r], rank[p] = r of mover p,
// meta = {L, movers}.
__global__ void __launch_bounds__(kPgThreads) pages_plan_kernel(const int* refs, int pages,
                                                                int* from, int* to, int* count, int* rank_of,
                                                                int* meta, int cap, int ctas, int* table,
                                                                long long entries, int* refs_out) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ long long sums[2 * kPgWarps];
    __shared__ int here[3];                            // used pages, movers, holes of this slice
    BlockScan scan{sums};
    const int rank = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
    int begin, end;
    slice_of(pages, rank, ctas, begin, end);
    const bool one = end - begin <= kPgTile;
    int4 r4 = make_int4(0, 0, 0, 0);
    int used = 0;
    long long total;
    for (int p = begin + 4 * tid; p < end; p += kPgTile) {
        r4 = refs4(refs, p, pages);
        for (int e = 0; e < 4; ++e) used += p + e < pages && (&r4.x)[e] != 0;
    }
    scan(used, &total);
    if (tid == 0) here[0] = static_cast<int>(total);
    cluster.sync();
    int low = 0;
    for (int x = 0; x < ctas; ++x) low += cluster.map_shared_rank(here, x)[0];
    // movers and holes before this slice
    int mv = 0, ho = 0;
    for (int p = begin + 4 * tid; p < end; p += kPgTile) {
        if (!one) r4 = refs4(refs, p, pages);
        for (int e = 0; e < 4; ++e) {
            mv += p + e < pages && p + e >= low && (&r4.x)[e] != 0;
            ho += p + e < low && (&r4.x)[e] == 0;
        }
    }
    // (movers, holes) are scanned in one word
    const long long both = scan(static_cast<long long>(mv) << 32 | static_cast<unsigned>(ho), &total);
    if (tid == 0) {
        here[1] = static_cast<int>(total >> 32);
        here[2] = static_cast<int>(total);
    }
    cluster.sync();
    int mb = 0, hb = 0, all = 0;
    for (int x = 0; x < ctas; ++x) {
        const int* h = cluster.map_shared_rank(here, x);
        if (x < rank) {
            mb += h[1];
            hb += h[2];
        }
        all += h[1];
    }
    for (int p0 = begin; p0 < end; p0 += kPgTile) {
        const int p = p0 + 4 * tid;
        if (!one) r4 = p < end ? refs4(refs, p, pages) : make_int4(1, 1, 1, 1);
        int m[4], h[4], ms = 0, hs = 0;
        for (int e = 0; e < 4; ++e) {
            const bool in = p + e < end;
            m[e] = in && p + e >= low && (&r4.x)[e] != 0;
            h[e] = in && p + e < low && (&r4.x)[e] == 0;
            ms += m[e];
            hs += h[e];
        }
        long long incl = both, tile = total;               // a slice of one tile has been scanned
        if (!one) incl = scan(static_cast<long long>(ms) << 32 | static_cast<unsigned>(hs), &tile);
        int mr = mb + static_cast<int>(incl >> 32) - ms, hr = hb + static_cast<int>(incl) - hs;
        mb += static_cast<int>(tile >> 32);
        hb += static_cast<int>(tile);
        for (int e = 0; e < 4; ++e) {
            if (m[e]) {
                from[mr] = p + e;
                rank_of[p + e] = mr++;
            }
            if (h[e]) to[hr++] = p + e;
        }
    }
    for (int i = all + rank * kPgThreads + tid; i < cap; i += ctas * kPgThreads) from[i] = to[i] = -1;
    if (rank == 0 && tid == 0) {
        *count = all;
        meta[0] = low;
        meta[1] = all;
    }
    cluster.sync();                                    // the plan is written (and here[] read)
    if (table) pages_follow(table, entries, refs_out, pages, from, to, rank_of, low, all);
}

// Second part as a launch of its own, for tables that a cluster would take long to walk.
__global__ void __launch_bounds__(256) pages_follow_kernel(int* table, long long entries, int* refs, int pages,
                                                           const int* from, const int* to, const int* rank_of,
                                                           const int* meta) {
    pages_follow(table, entries, refs, pages, from, to, rank_of, meta[0], meta[1]);
}

// Page contents from[i] -> to[i] in every layer: pieces of up to 32 KB, one CTA at a time, eight
// 16-byte loads in flight per thread.
constexpr int kCopyThreads = 256, kCopyUnroll = 8;
constexpr int kCopyPiece = kCopyThreads * kCopyUnroll;       // 16-byte words

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(uint4* pool, const int* __restrict__ from,
                                                                  const int* __restrict__ to,
                                                                  const int* __restrict__ count, int layers,
                                                                  int pages, long long page_words, int n) {
    const int live = count ? min(*count, n) : n;
    const long long pieces = (page_words + kCopyPiece - 1) / kCopyPiece;
    const long long jobs = pieces * layers * max(live, 0);
    for (long long j = blockIdx.x; j < jobs; j += gridDim.x) {
        const long long i = j / (pieces * layers);
        const int layer = static_cast<int>(j / pieces % layers);
        const long long w0 = j % pieces * kCopyPiece + threadIdx.x;
        const int a = from[i], b = to[i];
        if (a < 0 || a >= pages || b < 0 || b >= pages) continue;
        const uint4* src = pool + (static_cast<size_t>(layer) * pages + a) * page_words;
        uint4* dst = pool + (static_cast<size_t>(layer) * pages + b) * page_words;
        uint4 v[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (w0 + u * kCopyThreads < page_words) v[u] = src[w0 + u * kCopyThreads];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (w0 + u * kCopyThreads < page_words) dst[w0 + u * kCopyThreads] = v[u];
    }
}

// CTAs that scan the counts: one tile each at least, one CTA alone up to 4 tiles (no cluster to wait
// for).
int scan_ctas(int pages) { return pages <= 4 * kPgTile ? 1 : kPgCluster; }

template <typename... Args>
cudaError_t launch_cluster(void (*kern)(Args...), int ctas, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool FORK>
cudaError_t launch_take(const PageState& s, const int* seqs, const int* arg, int* out0, int* out1, int n,
                        cudaStream_t stream) {
    const size_t smem = static_cast<size_t>((s.slots + 31) / 32 + 2 * n + 1) * sizeof(int);
    // the bound of every call, so that two host threads never set it against each other
    constexpr int kMost = (kPagesMaxSlots / 32 + 2 * kPagesMaxSeqs + 1) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(pages_take_kernel<FORK>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    const int ctas = scan_ctas(s.pages);
    return launch_cluster(pages_take_kernel<FORK>, ctas, smem, stream, s, seqs, arg, out0, out1, n, ctas);
}

}  // namespace

cudaError_t launch_pages_reserve(const PageState& s, const int* seqs, const int* counts, int* start,
                                 int n, cudaStream_t stream) {
    return launch_take<false>(s, seqs, counts, start, nullptr, n, stream);
}

cudaError_t launch_pages_fork(const PageState& s, const int* src, const int* dst, int* from, int* to,
                              int n, cudaStream_t stream) {
    return launch_take<true>(s, dst, src, from, to, n, stream);
}

cudaError_t launch_pages_free(const PageState& s, const int* seqs, int n, int whole, int wl, int ns,
                              cudaStream_t stream) {
    pages_free_kernel<<<n, 256, 0, stream>>>(s, seqs, whole, wl, ns);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PageState& s, int* from, int* to, int* count, int* ws,
                                 cudaStream_t stream) {
    const int cap = s.pages / 2 > 0 ? s.pages / 2 : 1;
    const int ctas = scan_ctas(s.pages);
    int* rank_of = ws + 4;
    const long long entries = static_cast<long long>(s.slots) * s.max_pages;
    const bool together = entries <= 16LL * ctas * kPgThreads;       // 16 entries per thread at most
    cudaError_t e = launch_cluster(pages_plan_kernel, ctas, 0, stream, static_cast<const int*>(s.refs), s.pages,
                                   from, to, count, rank_of, ws, cap, ctas, together ? s.table : nullptr, entries,
                                   s.refs);
    if (e != cudaSuccess || together) return e;
    long long blocks = (entries + 1023) / 1024;
    blocks = blocks < 1 ? 1 : (blocks > 148 * 8 ? 148 * 8 : blocks);
    pages_follow_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        s.table, entries, s.refs, s.pages, static_cast<const int*>(from), static_cast<const int*>(to),
        static_cast<const int*>(rank_of), static_cast<const int*>(ws));
    return cudaGetLastError();
}

cudaError_t launch_pages_copy(void* pool, const int* from, const int* to, const int* count, int layers,
                              int pages, long long page_bytes, int n, cudaStream_t stream) {
    const long long words = page_bytes / 16;
    const long long jobs = (words + kCopyPiece - 1) / kCopyPiece * layers * n;
    const long long blocks = jobs < 148 * 8 ? jobs : 148 * 8;
    pages_copy_kernel<<<static_cast<unsigned>(blocks), kCopyThreads, 0, stream>>>(
        static_cast<uint4*>(pool), from, to, count, layers, pages, words, n);
    return cudaGetLastError();
}

}  // namespace attn
