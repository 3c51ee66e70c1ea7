// Kernels of the 4-bit paged K/V cache (layout and formulas: kv4.h): quantising new rows into their
// pages, reading rows back, and attention of a few new tokens per sequence over the cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv4.h"
#include "sm100_ptx.cuh"

namespace attn {

namespace {

// Page that holds token `pos` of table row `slot`, or -1 (outside the table, or not a page).
__device__ __forceinline__ int kv4_page(const Kv4Pool& p, int slot, long long pos) {
    const long long m = pos / p.page_size;
    if (slot < 0 || slot >= p.slots || pos < 0 || m >= p.max_pages) return -1;
    const int pg = p.table[static_cast<size_t>(slot) * p.max_pages + m];
    return pg < p.pages ? pg : -1;
}

// Block of page `pg` and head h that holds token `pos`.
__device__ __forceinline__ uint8_t* kv4_block(const Kv4Pool& p, int pg, int h, long long pos) {
    const int bpp = p.page_size / kKv4Block;
    const size_t blk = (static_cast<size_t>(pg) * p.Hkv + h) * bpp + (pos / kKv4Block) % bpp;
    return p.data + blk * kv4_block_bytes(p.d);
}

// ------------------------------------------------------------------------------------------
// Append and gather. One CTA of 128 threads per (block of 16 tokens, head, batch entry); a team of 8
// lanes holds a group of one token, 4 channels per lane, so minimum and maximum take three
// shuffles, a lane's nibbles of V are one 16-bit unit and those of K half a word. Blocks that the
// rows fill are put together in shared memory and copied out in 16-byte pieces; at the ragged
// ends each token's own 2- and 4-byte units are stored (neighbours' tokens are never touched).
// Bound by HBM for long chunks, by latency (table entry, then store) for single tokens.
// ------------------------------------------------------------------------------------------
constexpr int kRowThreads = 128;

// q of x in a group with lo, s, from t = x - lo: the whole number nearest (x - lo)/s, ties to even.
// t·(1/s) is within a few 2^-22 of the quotient, so it decides unless it lies next to a border; there
// the exact border (n + 1/2)·s (s has 8 bits) is compared with t and what t lost of x - lo.
__device__ __forceinline__ int kv4_quantise(float x, float lo, float s, float inv) {
    const float t = x - lo;
    const float f = t * inv;
    float n = rintf(f);
    if (fabsf(fabsf(f - n) - 0.5f) < 1e-4f) {
        n = floorf(f);
        const float border = (n + 0.5f) * s;              // exact: at most 5 + 8 bits
        const float bb = t - x, lost = (x - (t - bb)) + (-lo - bb);   // x - lo = t + lost exactly
        const bool up = t > border || (t == border && (lost > 0.f || (lost == 0.f && (static_cast<int>(n) & 1))));
        n = up ? n + 1.f : n;
    }
    return static_cast<int>(fminf(fmaxf(n, 0.f), 15.f));
}

// One lane's 4 channels (bf16 in w) of a group shared by 8 lanes: nibbles (channel i in bits 4·i) and
// the group's parameter word.
__device__ __forceinline__ uint32_t kv4_group(uint2 w, uint32_t& param) {
    float x[4];
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
    float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
    float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    bool nan = !(x[0] == x[0] && x[1] == x[1] && x[2] == x[2] && x[3] == x[3]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        nan |= __shfl_xor_sync(0xffffffffu, nan, o);
    }
    uint32_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f)));
    float s = __uint_as_float(sb << 16);
    if (s < 0x1p-100f) { s = 0.f; sb = 0; }
    // a NaN or an infinity makes its whole group NaN
    if (nan || !(s < INFINITY)) { sb = 0x7fc0u; s = 0.f; }
    param = sb | (__float_as_uint(lo) & 0xffff0000u);
    if (s == 0.f) return 0;
    const float inv = 1.f / s;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n |= static_cast<uint32_t>(kv4_quantise(x[i], lo, s, inv)) << (4 * i);
    return n;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4RowsArgs a) {
    constexpr int G = D / 32, BB = kv4_block_bytes(D);
    constexpr int TASKS = 16 * G;                        // (token, group), by teams of 8 lanes
    __shared__ __align__(16) uint8_t stage[BB];
    const int i = blockIdx.z, h = blockIdx.y;
    const int first = a.start[i];
    const int count = min(a.counts ? a.counts[i] : a.n, a.n);
    if (first < 0 || count < 1) return;
    const long long blk = first / kKv4Block + static_cast<long long>(blockIdx.x);
    const long long t0 = blk * kKv4Block - first;        // row of the block's first token
    if (t0 >= count) return;
    const int slot = a.pool.seqs ? a.pool.seqs[i] : i;
    const int pg = kv4_page(a.pool, slot, blk * kKv4Block);
    if (pg < 0) return;
    uint8_t* block = kv4_block(a.pool, pg, h, blk * kKv4Block);
    const bool whole = t0 >= 0 && t0 + kKv4Block <= count;
    uint8_t* out = whole ? stage : block;
    const int team = threadIdx.x >> 3, row = threadIdx.x & 7;
    const size_t base = (static_cast<size_t>(i) * a.pool.Hkv + h) * a.n * D;
    const __nv_bfloat16* src[2] = {static_cast<const __nv_bfloat16*>(a.k) + base,
                                   static_cast<const __nv_bfloat16*>(a.v) + base};
    uint2 w[2][G];
#pragma unroll
    for (int x = 0; x < G; ++x) {                        // all loads before the first use
        const int task = x * (kRowThreads / 8) + team;
        const long long t = t0 + task / G;
        const bool live = t >= 0 && t < count;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
            w[kv][x] = live ? *reinterpret_cast<const uint2*>(src[kv] + t * D + task % G * 32 + row * 4)
                            : make_uint2(0u, 0u);
    }
    static_assert(TASKS == G * (kRowThreads / 8), "one task per team and round");
#pragma unroll
    for (int x = 0; x < G; ++x) {
        const int task = x * (kRowThreads / 8) + team;
        const int tok = task / G, g = task % G;
        const bool live = t0 + tok >= 0 && t0 + tok < count;
        uint32_t kp, vp;
        uint32_t kn = kv4_group(w[0][x], kp), vn = kv4_group(w[1][x], vp);
        // K: channels 4·row .. 4·row+3 are j = 2·(row & 1) + {0, 0, 1, 1}, h = {0, 1, 0, 1} of word
        // c = row / 2: nibbles to bits 4·(j + 4·h)
        kn = (kn & 0xfu) | (kn & 0xf0u) << 12 | (kn & 0xf00u) >> 4 | (kn & 0xf000u) << 8;
        kn <<= 8 * (row & 1);
        kn |= __shfl_xor_sync(0xffffffffu, kn, 1);
        if (!live) continue;
        if (!(row & 1)) {
            const int word = ((tok >> 3) * 32 + (tok & 7) * 4 + (row >> 1)) * G + g;
            *reinterpret_cast<uint32_t*>(out + word * 4) = kn;
        }
        const int unit = (((tok >> 3) * 32 + row * 4 + ((tok & 7) >> 1)) * G + g) * 2 + (tok & 1);
        *reinterpret_cast<uint16_t*>(out + 8 * D + unit * 2) = static_cast<uint16_t>(vn);
        if (row < 2)
            *reinterpret_cast<uint32_t*>(out + 16 * D + row * 2 * D + (tok * G + g) * 4) = row ? vp : kp;
    }
    if (whole) {
        __syncthreads();
        for (int x = threadIdx.x; x < BB / 16; x += kRowThreads)
            reinterpret_cast<uint4*>(block)[x] = reinterpret_cast<const uint4*>(stage)[x];
    }
}

// Rows beyond counts, of entries left out and on pages that the table does not hold are zeros.
template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const Kv4RowsArgs a) {
    constexpr int G = D / 32, BB = kv4_block_bytes(D);
    __shared__ __align__(16) uint8_t stage[BB];
    const int i = blockIdx.z, h = blockIdx.y;
    const int start = a.start[i];
    const int first = max(start, 0);
    const int count = start < 0 ? 0 : min(a.counts ? a.counts[i] : a.n, a.n);
    const long long blk = first / kKv4Block + static_cast<long long>(blockIdx.x);
    const long long t0 = blk * kKv4Block - first;
    if (t0 >= a.n) return;
    int pg = -1;
    if (t0 < count) pg = kv4_page(a.pool, a.pool.seqs ? a.pool.seqs[i] : i, blk * kKv4Block);
    if (pg >= 0) {
        const uint8_t* block = kv4_block(a.pool, pg, h, blk * kKv4Block);
        for (int x = threadIdx.x; x < BB / 16; x += kRowThreads)
            reinterpret_cast<uint4*>(stage)[x] = reinterpret_cast<const uint4*>(block)[x];
    }
    __syncthreads();
    const int team = threadIdx.x >> 3, row = threadIdx.x & 7;
    const size_t base = (static_cast<size_t>(i) * a.pool.Hkv + h) * a.n * D;
#pragma unroll
    for (int x = 0; x < G; ++x) {
        const int task = x * (kRowThreads / 8) + team;
        const int tok = task / G, g = task % G;
        const long long t = t0 + tok;
        if (t < 0 || t >= a.n) continue;
        uint2 w[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
        if (pg >= 0 && t < count) {
            const uint32_t kw = *reinterpret_cast<const uint32_t*>(
                stage + (((tok >> 3) * 32 + (tok & 7) * 4 + (row >> 1)) * G + g) * 4) >> (8 * (row & 1));
            const uint32_t vw = *reinterpret_cast<const uint16_t*>(
                stage + 8 * D + ((((tok >> 3) * 32 + row * 4 + ((tok & 7) >> 1)) * G + g) * 2 + (tok & 1)) * 2);
            const uint32_t nib[2] = {(kw & 0xfu) | (kw >> 12 & 0xf0u) | (kw << 4 & 0xf00u) | (kw >> 8 & 0xf000u),
                                     vw};
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t p = *reinterpret_cast<const uint32_t*>(stage + (16 + 2 * kv) * D + (tok * G + g) * 4);
                const float s = __uint_as_float(p << 16), lo = __uint_as_float(p & 0xffff0000u);
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = fmaf(s, static_cast<float>(nib[kv] >> (4 * e) & 15u), lo);
                w[kv] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            }
        }
        const size_t at = base + t * D + g * 32 + row * 4;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.k) + at) = w[0];
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.v) + at) = w[1];
    }
}

// ------------------------------------------------------------------------------------------
// Attention over the cache.
//
// All query rows of one K/V head (its query heads times nq tokens) share every byte that is read,
// so a (batch entry, K/V head, block of 8·NT rows) is one segment of work, its keys the blocks of
// 16 tokens that any row sees: those of the sinks, then those of the window. The segments' tiles
// (4 blocks) laid end to end are cut into equal runs, one per CTA, whatever the lengths of the
// sequences; a CTA writes the segments it holds whole and leaves the parts of the others in
// the workspace, where a second launch joins them with the rule that joins two softmax blocks.
//
// Each of a CTA's 4 warps takes every fourth block through a ring of its own (bulk copies
// of a whole block, contiguous in memory, one mbarrier per stage): no barrier among the warps until a
// segment ends. The two products run as mma.m16n8k16 (fp16 in, fp32 sums); tcgen05's smallest tile
// of 128 rows would be filled to 1/16 to 1/128 by the 1 to 8 rows there are, and its operands would
// first have to be unpacked into shared memory.
//   S (16 keys x 8 rows) = K · Q^T. A nibble masked out of its word IS the fp16 number q·2^-24 (or,
//   from the next position, 16·q·2^-24): both are subnormals, which the tensor cores take exactly, so
//   unpacking a word of 8 costs 4 ANDs and a shift. Q is scaled by a power of two that brings the row's
//   largest value to 2^14 .. 2^15 (its bf16 values are then exact in fp16 down to 2^-29 of the largest;
//   channels that meet 16·q carry Q/16). Per group g: S += s_g·acc_g + lo_g·sum_g(Q), in fp32.
//   O^T (channels x 8 rows) += V^T · P^T with P·s_g in fp16, scaled by a power of two (2^4 at the
//   largest s of the cache so far: 11 bits down to weights of 2^-18, 2^-28 absolute) and transposed
//   between the fragment layouts by movmatrix; lo's share, sum of P·lo_g, stays in fp32.
// Running maximum, sum and O are per warp; the maximum moves only when a score exceeds it by more than
// 8 (P up to 2^8; the result does not depend on it).
// ------------------------------------------------------------------------------------------
constexpr int kAttWarps = 4, kAttThreads = 32 * kAttWarps;
constexpr int kAttMaxCtas = 592;           // runs at most (4 per SM); sizes the workspace
constexpr float kAttLog2e = 1.44269504088896340736f;
constexpr float kAttLn2 = 0.69314718055994530942f;

template <int D, int NT>
struct AttCfg {
    static constexpr int G = D / 32;
    static constexpr int BB = kv4_block_bytes(D);
    static constexpr int ROWS = 8 * NT;
    static constexpr int STAGES = D == 128 ? 3 : (D == 64 ? 5 : 8);
    static constexpr int CTAS = NT == 1 ? 4 : 2;                        // per SM
    static constexpr int RING = kAttWarps * STAGES * BB;
    static constexpr int OPAD = D + 4;
    static constexpr int MERGE = kAttWarps * ROWS * (OPAD + 2) * 4;     // O rows, then (m, l)
    static constexpr int SMEM = RING + MERGE + kAttWarps * STAGES * 8 + 128;
    static constexpr int PART = ROWS * (D + 2);                         // floats of a part
};

struct AttParams {
    Kv4AttendArgs a;
    float scale_log2;
    int R, RB;            // query rows per K/V head, row blocks of 8·NT
};

// Keys of batch entry b that some of its rows see, as blocks of 16: sink blocks [0, sb), then nb - sb
// blocks from wb0 on.
struct AttSeq {
    int slot, sb, wb0, nb;
    long long off;        // key position of query 0
    int last;             // last visible key
};

__device__ __forceinline__ AttSeq att_seq(const Kv4AttendArgs& a, int b) {
    AttSeq s;
    s.slot = a.pool.seqs ? a.pool.seqs[b] : b;
    const bool ok = s.slot >= 0 && s.slot < a.pool.slots;
    const long long cap = static_cast<long long>(a.pool.max_pages) * a.pool.page_size;
    long long len = ok ? a.lens[s.slot] : 0;
    len = len < 0 ? 0 : (len > cap ? cap : len);
    s.off = len - a.nq;
    long long lo = a.wl < 0 ? 0 : s.off - a.wl;
    lo = lo < 0 ? 0 : lo;
    long long hi = a.wr < 0 ? len - 1 : s.off + a.nq - 1 + a.wr;
    hi = hi > len - 1 ? len - 1 : hi;
    s.last = static_cast<int>(hi);
    s.sb = s.wb0 = s.nb = 0;
    if (hi >= 0 && hi >= lo) {
        const long long ns = a.ns < hi + 1 ? a.ns : hi + 1;
        const int sb = static_cast<int>((ns + kKv4Block - 1) / kKv4Block);
        const int w0 = static_cast<int>(lo / kKv4Block), w1 = static_cast<int>(hi / kKv4Block);
        s.wb0 = sb >= w0 ? 0 : w0;
        s.sb = sb >= w0 ? 0 : sb;
        s.nb = s.sb + w1 - s.wb0 + 1;
    }
    return s;
}

__device__ __forceinline__ int att_tiles(const Kv4AttendArgs& a, int b) {
    return (att_seq(a, b).nb + kAttWarps - 1) / kAttWarps;
}

// Sum of att_tiles over [0, n) (all threads of the CTA get it; `scratch` of kAttWarps long longs).
__device__ __forceinline__ long long att_prefix(const Kv4AttendArgs& a, int n, int threads,
                                                long long* scratch) {
    long long t = 0;
    for (int b = threadIdx.x; b < n; b += threads) t += att_tiles(a, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = t;
    __syncthreads();
    t = 0;
    for (int w = 0; w < threads / 32; ++w) t += scratch[w];
    __syncthreads();
    return t;
}

// Runs that `total` tiles are cut into: one per CTA, none shorter than 2 tiles.
__host__ __device__ inline long long att_runs(long long total, int ctas) {
    const long long r = (total + 1) / 2;
    return r < ctas ? r : ctas;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// G words at p (16-, 8- or 4-byte aligned by G).
template <int G>
__device__ __forceinline__ void lds_words(uint32_t (&w)[G], const uint8_t* p) {
    if constexpr (G == 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(p);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    } else if constexpr (G == 2) {
        const uint2 t = *reinterpret_cast<const uint2*>(p);
        w[0] = t.x; w[1] = t.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kAttThreads, AttCfg<D, NT>::CTAS) kv4_attend_kernel(const AttParams p) {
    using C = AttCfg<D, NT>;
    constexpr int G = C::G, ST = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* merge = reinterpret_cast<float*>(smem + C::RING);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING + C::MERGE);
    long long* scratch = reinterpret_cast<long long*>(bars + kAttWarps * ST);
    int* abort_s = reinterpret_cast<int*>(scratch + kAttWarps);
    volatile int* abort = abort_s;
    const Kv4AttendArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * ST * C::BB;
    uint64_t* full = bars + warp * ST;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kAttWarps * ST; ++s) mbar_init(&bars[s], 1);
        *abort_s = 0;
        fence_barrier_init();
    }
    // ---- this CTA's run of tiles, and the segment it begins in (att_prefix synchronises the CTA)
    const int HR = a.pool.Hkv * p.RB;
    const long long per_head = att_prefix(a, a.B, kAttThreads, scratch);
    const long long total = per_head * HR;
    const long long runs = att_runs(total, gridDim.x);
    if (blockIdx.x >= runs) return;
    const long long x0 = total * blockIdx.x / runs, x1 = total * (blockIdx.x + 1) / runs;
    int b = 0, hr;
    long long tile;       // in the segment
    {
        // batch entry of tile x0: entries hold HR segments of att_tiles(b) tiles each
        long long before = 0;
        while (true) {    // b advances by whole chunks of threads, then by the prefix within one
            const int bb = b + static_cast<int>(threadIdx.x);
            long long t = bb < a.B ? static_cast<long long>(att_tiles(a, bb)) * HR : 0, incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) scratch[warp] = incl;
            __syncthreads();
            long long chunk = 0, mine = before;
            for (int w = 0; w < kAttWarps; ++w) {
                if (w < warp) mine += scratch[w];
                chunk += scratch[w];
            }
            __syncthreads();
            if (x0 >= before + chunk) {
                before += chunk;
                b += kAttThreads;
                if (b >= a.B) return;      // only if lens changed under the call
                continue;
            }
            mine += incl - t;                              // tiles before entry bb
            if (x0 >= mine && x0 < mine + t) {
                scratch[0] = bb;
                scratch[1] = x0 - mine;
            }
            __syncthreads();
            b = static_cast<int>(scratch[0]);
            tile = scratch[1];
            __syncthreads();
            break;
        }
    }
    AttSeq seq = att_seq(a, b);
    if (seq.nb == 0) return;               // (as above: the loops below count on what they read)
    {
        const int nt = (seq.nb + kAttWarps - 1) / kAttWarps;
        hr = static_cast<int>(tile / nt);
        tile -= static_cast<long long>(hr) * nt;
    }
    const int bpp = a.pool.page_size / kKv4Block;
    const uint64_t lim = a.timeout_ns;

    // ---- fetching: a cursor over the run's tiles, ST blocks ahead of the one over the computation
    AttSeq fs = seq;
    int fb = b, fhr = hr, ft = static_cast<int>(tile);
    long long fx = x0;
    int pid = -1, fblk = 0, fhead = 0;      // page of the next block to fetch (loaded ahead of its use)
    bool more = true;
    // moves the cursor to this warp's next block and starts loading its page number
    auto seek = [&]() {
        while (fx < x1) {
            const int li = ft * kAttWarps + warp;
            const bool have = li < fs.nb;
            if (have) {
                const int tb = li < fs.sb ? li : fs.wb0 + li - fs.sb;
                fblk = tb % bpp;
                fhead = fhr / p.RB;
                pid = a.pool.table[static_cast<size_t>(fs.slot) * a.pool.max_pages + tb / bpp];
            }
            ++fx;
            if (++ft * kAttWarps >= fs.nb) {
                ft = 0;
                if (++fhr == HR) {
                    fhr = 0;
                    if (fx < x1)
                        do fs = att_seq(a, ++fb);
                        while (fs.nb == 0 && fb + 1 < a.B);
                }
            }
            if (have) return;
        }
        more = false;
    };
    uint32_t valid = 0;                     // stages that hold a block (not a page that is missing)
    int issued = 0, taken = 0;              // blocks
    auto fetch = [&]() {
        if (!more) return;
        const int s = issued % ST;
        const bool ok = pid >= 0 && pid < a.pool.pages;
        valid = ok ? valid | (1u << s) : valid & ~(1u << s);
        if (lane == 0) {
            if (ok) {
                const uint8_t* src =
                    a.pool.data + ((static_cast<size_t>(pid) * a.pool.Hkv + fhead) * bpp + fblk) * C::BB;
                mbar_arrive_expect_tx(&full[s], C::BB);
                bulk_load(ring + s * C::BB, src, C::BB, &full[s]);
            } else {
                mbar_arrive(&full[s]);
            }
        }
        ++issued;
        seek();
    };
    seek();
    for (int s = 0; s < ST; ++s) fetch();

    long long x = x0;
    bool ok = true;
    while (x < x1) {
        // ---- one segment's part of the run
        const int nt_all = (seq.nb + kAttWarps - 1) / kAttWarps;
        const int t0 = static_cast<int>(tile);
        const int t1 = static_cast<int>(min(static_cast<long long>(nt_all), tile + (x1 - x)));
        const int head = hr / p.RB, row0 = hr % p.RB * C::ROWS;
        const size_t qbase = (static_cast<size_t>(b) * a.pool.Hkv + head) * p.R;
        // Q as the B operand of S: lane (gid, c) holds row gid, channels 32·g + 8·c .. + 7
        uint32_t qf[NT][G][4];
        float qsum[NT][G][2];       // scale·log2(e)·sum over the group, of rows 2c, 2c + 1
        float cq[NT][2];            // scale·log2(e)·2^24 / (Q's power of two), of rows 2c, 2c + 1
        int pos[NT][2];             // key position of those rows, relative to off
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + n * 8 + gid;
            uint4 w[G];
            float amax = 0.f, sum[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                w[g] = r < p.R ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                                (qbase + r) * D + g * 32 + c * 8)
                               : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
                sum[g] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
                    amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
                    sum[g] += lo + hi;
                }
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax in 2^(e-127) .. 2^(e-126): times 2^(141-e) it lies in 2^14 .. 2^15
            const int up = min(141 - static_cast<int>(__float_as_uint(amax) >> 23), 127);
            const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float m = (e & 1) ? f * 0.0625f : f;
                    qf[n][g][e] = pack_f16x2(__uint_as_float(u[e] << 16) * m,
                                             __uint_as_float(u[e] & 0xffff0000u) * m);
                }
            }
            const float back = ldexpf(p.scale_log2, 24 - up);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int src = (2 * c + e) * 4;
                cq[n][e] = __shfl_sync(0xffffffffu, back, src);
#pragma unroll
                for (int g = 0; g < G; ++g)
                    qsum[n][g][e] = __shfl_sync(0xffffffffu, sum[g], src) * p.scale_log2;
                pos[n][e] = (row0 + n * 8 + 2 * c + e) % a.nq;
            }
        }
        // blocks [full_lo, full_hi] (by first key) are seen whole by every row
        const long long full_lo = a.wl < 0 ? 0 : seq.off + a.nq - 1 - a.wl;
        const long long full_hi = (a.wr < 0 ? seq.last : min(seq.off + a.wr, static_cast<long long>(seq.last))) -
                                  (kKv4Block - 1);
        float m[NT][2], l[NT][2], ol[NT][G][2], acc[NT][2 * G][4];
        float fv = 0x1p127f;        // power of two on P·s
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
#pragma unroll
                for (int g = 0; g < G; ++g) ol[n][g][e] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < 2 * G; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][t][e] = 0.f;
        }
        for (int t = t0; ok && t < t1; ++t) {
            const int li = t * kAttWarps + warp;
            if (li >= seq.nb) break;
            const int st = taken % ST;
            const bool held = valid >> st & 1u;
            ok = bounded_wait_warp(&full[st], (taken / ST) & 1, abort, lim);
            ++taken;
            if (!ok) break;
            if (held) {
                const int tb = li < seq.sb ? li : seq.wb0 + li - seq.sb;
                const long long k0 = static_cast<long long>(tb) * kKv4Block;
                const bool edge = (k0 < full_lo && k0 + kKv4Block > a.ns) || k0 > full_hi;
                const uint8_t* blk = ring + st * C::BB;
                // parameters of keys gid and gid + 8
                float ks[2][G], kl[2][G], vs[2][G], vl[2][G];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[G];
                    lds_words<G>(w, blk + 16 * D + (h * 8 + gid) * G * 4);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        ks[h][g] = __uint_as_float(w[g] << 16);
                        kl[h][g] = __uint_as_float(w[g] & 0xffff0000u);
                    }
                    lds_words<G>(w, blk + 18 * D + (h * 8 + gid) * G * 4);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        vs[h][g] = __uint_as_float(w[g] << 16);
                        vl[h][g] = __uint_as_float(w[g] & 0xffff0000u);
                    }
                }
                // ---- S
                float z[NT][4];     // (key gid, rows 2c, 2c + 1), (key gid + 8, ...)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[n][e] = 0.f;
                {
                    uint32_t k0w[G], k1w[G];
                    lds_words<G>(k0w, blk + lane * G * 4);
                    lds_words<G>(k1w, blk + (32 + lane) * G * 4);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint32_t y0 = k0w[g] >> 8, y1 = k1w[g] >> 8;
                        const uint32_t a00 = k0w[g] & 0x000f000fu, a01 = k1w[g] & 0x000f000fu;
                        const uint32_t a02 = k0w[g] & 0x00f000f0u, a03 = k1w[g] & 0x00f000f0u;
                        const uint32_t a10 = y0 & 0x000f000fu, a11 = y1 & 0x000f000fu;
                        const uint32_t a12 = y0 & 0x00f000f0u, a13 = y1 & 0x00f000f0u;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float s[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(s, a00, a01, a02, a03, qf[n][g][0], qf[n][g][1]);
                            mma_f16(s, a10, a11, a12, a13, qf[n][g][2], qf[n][g][3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                z[n][e] = fmaf(s[e] * cq[n][e & 1], ks[e >> 1][g],
                                               fmaf(kl[e >> 1][g], qsum[n][g][e & 1], z[n][e]));
                        }
                    }
                }
                uint32_t hidden[NT];
                if (edge) {
                    // keys a row does not see; the parameters of keys that no row sees may be anything
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        hidden[n] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const long long key = k0 + gid + 8 * (e >> 1);
                            const long long at = seq.off + pos[n][e & 1];
                            const bool seen = key <= seq.last && (a.wr < 0 || key <= at + a.wr) &&
                                              (a.wl < 0 || key >= at - a.wl || key < a.ns);
                            if (!seen) {
                                z[n][e] = -INFINITY;
                                hidden[n] |= 1u << e;
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const long long key = k0 + gid + 8 * h;
                        if (key > seq.last || (a.wl >= 0 && key < seq.off - a.wl && key >= a.ns)) {
#pragma unroll
                            for (int g = 0; g < G; ++g) vs[h][g] = vl[h][g] = 0.f;
                        }
                    }
                }
                // ---- the running maximum, and the power of two on P·s, move rarely
                bool grow = false;
                float smax = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) grow |= fmaxf(z[n][e], z[n][2 + e]) > m[n][e] + 8.f;
#pragma unroll
                for (int g = 0; g < G; ++g) smax = fmaxf(smax, fmaxf(vs[0][g], vs[1][g]));
                if (__any_sync(0xffffffffu, grow || smax * fv > 128.f)) {
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1)
                        smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, o));
                    float ratio = 1.f;
                    if (smax * fv > 128.f) {
                        // smax < 2^(e-126): times 2^(131-e) below 2^5
                        const int e = min(131 - static_cast<int>(__float_as_uint(smax) >> 23), 127);
                        const float now = e < -126 ? 0x1p-126f : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                        ratio = now / fv;
                        fv = now;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = fmaxf(z[n][e], z[n][2 + e]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                            t = fmaxf(t, m[n][e]);
                            const float al = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - t);
                            m[n][e] = t;
                            l[n][e] *= al;
#pragma unroll
                            for (int g = 0; g < G; ++g) ol[n][g][e] *= al;
                            const float ar = al * ratio;
#pragma unroll
                            for (int q = 0; q < 2 * G; ++q) {
                                acc[n][q][e] *= ar;
                                acc[n][q][2 + e] *= ar;
                            }
                        }
                }
                // ---- P, and P·s in fp16 as the B operand of O^T
                uint32_t v0w[G], v1w[G];
                lds_words<G>(v0w, blk + 8 * D + lane * G * 4);
                lds_words<G>(v1w, blk + 8 * D + (32 + lane) * G * 4);
                float pr[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
                    const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
                    pr[n][0] = ex2_approx(z[n][0] - m0);
                    pr[n][1] = ex2_approx(z[n][1] - m1);
                    pr[n][2] = ex2_approx(z[n][2] - m0);
                    pr[n][3] = ex2_approx(z[n][3] - m1);
                    l[n][0] += pr[n][0] + pr[n][2];
                    l[n][1] += pr[n][1] + pr[n][3];
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float f0 = vs[0][g] * fv, f1 = vs[1][g] * fv;
                    const uint32_t y0 = v0w[g] >> 8, y1 = v1w[g] >> 8;
                    const uint32_t a00 = v0w[g] & 0x000f000fu, a01 = v0w[g] & 0x00f000f0u;
                    const uint32_t a02 = v1w[g] & 0x000f000fu, a03 = v1w[g] & 0x00f000f0u;
                    const uint32_t a10 = y0 & 0x000f000fu, a11 = y0 & 0x00f000f0u;
                    const uint32_t a12 = y1 & 0x000f000fu, a13 = y1 & 0x00f000f0u;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float w0 = pr[n][0] * f0, w1 = pr[n][1] * f0, w2 = pr[n][2] * f1, w3 = pr[n][3] * f1;
                        float u0 = pr[n][0] * vl[0][g], u1 = pr[n][1] * vl[0][g];
                        float u2 = pr[n][2] * vl[1][g], u3 = pr[n][3] * vl[1][g];
                        if (edge) {     // 0 times a NaN or an infinity that the row does not see
                            if (hidden[n] & 1u) w0 = u0 = 0.f;
                            if (hidden[n] & 2u) w1 = u1 = 0.f;
                            if (hidden[n] & 4u) w2 = u2 = 0.f;
                            if (hidden[n] & 8u) w3 = u3 = 0.f;
                        }
                        ol[n][g][0] += u0 + u2;
                        ol[n][g][1] += u1 + u3;
                        const uint32_t b0 = movmatrix_trans(pack_f16x2(w0, w1));
                        const uint32_t b1 = movmatrix_trans(pack_f16x2(w2, w3));
                        mma_f16(acc[n][2 * g], a00, a01, a02, a03, b0, b1);
                        mma_f16(acc[n][2 * g + 1], a10, a11, a12, a13, b0, b1);
                    }
                }
            }
            __syncwarp();           // every lane has read the stage
            fetch();
        }
        // ---- this warp's part: O unnormalised in units of 2^m, m and l
        float* orow = merge + warp * C::ROWS * C::OPAD;
        float* ml = merge + kAttWarps * C::ROWS * C::OPAD + warp * C::ROWS * 2;
        const float back = 1.f / fv;                       // exact: a power of two
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float lt = l[n][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
                const int r = n * 8 + 2 * c + e;
                if (gid == 0) {
                    ml[2 * r] = m[n][e];
                    ml[2 * r + 1] = lt;
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float t = ol[n][g][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                    // channels 32·g + 4·gid + j; odd j were multiplied by 16
                    *reinterpret_cast<float4*>(orow + r * C::OPAD + g * 32 + gid * 4) =
                        make_float4(fmaf(acc[n][2 * g][e] * 0x1p24f, back, t),
                                    fmaf(acc[n][2 * g][2 + e] * 0x1p20f, back, t),
                                    fmaf(acc[n][2 * g + 1][e] * 0x1p24f, back, t),
                                    fmaf(acc[n][2 * g + 1][2 + e] * 0x1p20f, back, t));
                }
            }
        __syncthreads();
        // ---- join the warps; whole segments are finished here, parts go to the workspace
        const bool whole = t0 == 0 && t1 == nt_all;
        float* part = a.ws + (2 * static_cast<size_t>(blockIdx.x) + (x == x0 ? 0 : 1)) * C::PART;
        constexpr int C4 = D / 4;
        for (int idx = threadIdx.x; idx < C::ROWS * C4; idx += kAttThreads) {
            const int r = idx / C4, c4 = idx % C4;
            if (row0 + r >= p.R) continue;
            const float* mls = merge + kAttWarps * C::ROWS * C::OPAD + r * 2;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, mls[w * C::ROWS * 2]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float mw = mls[w * C::ROWS * 2];
                if (mw == -INFINITY) {
                    L += mls[w * C::ROWS * 2 + 1];         // 0, or NaN when every score was
                    continue;
                }
                const float f = ex2_approx(mw - M);
                L = fmaf(f, mls[w * C::ROWS * 2 + 1], L);
                const float4 t = *reinterpret_cast<const float4*>(merge + (w * C::ROWS + r) * C::OPAD + c4 * 4);
                o.x = fmaf(f, t.x, o.x); o.y = fmaf(f, t.y, o.y);
                o.z = fmaf(f, t.z, o.z); o.w = fmaf(f, t.w, o.w);
            }
            if (whole) {
                const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);    // NaN stays
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (qbase + row0 + r) * D + c4 * 4;
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (c4 == 0) a.lse[qbase + row0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttLn2;
            } else {
                *reinterpret_cast<float4*>(part + r * D + c4 * 4) = o;
                if (c4 == 0) {
                    part[C::ROWS * D + 2 * r] = M;
                    part[C::ROWS * D + 2 * r + 1] = L;
                }
            }
        }
        __syncthreads();
        // ---- next segment
        x += t1 - t0;
        tile = 0;
        if (++hr == HR) {
            hr = 0;
            if (x < x1)
                do seq = att_seq(a, ++b);
                while (seq.nb == 0 && b + 1 < a.B);
            if (seq.nb == 0) break;
        }
    }
    if (!ok || *abort) {          // let the copies in flight land
        const uint64_t t0 = globaltimer_ns();
        for (int i = taken > 0 ? taken - 1 : 0; i < issued; ++i)
            while (!mbar_try_wait(&full[i % ST], (i / ST) & 1))
                if (globaltimer_ns() - t0 > 100000000ull) break;
    }
}

// Joins the parts of segments that several runs share, and clears the rows of batch entries that see
// no key. One CTA per (row, segment), a thread per channel.
template <int D, int NT>
__global__ void __launch_bounds__(D) kv4_join_kernel(const AttParams p, int ctas) {
    using C = AttCfg<D, NT>;
    __shared__ long long scratch[kAttWarps];
    const Kv4AttendArgs& a = p.a;
    const int HR = a.pool.Hkv * p.RB;
    const int b = static_cast<int>(blockIdx.x / HR), hr = static_cast<int>(blockIdx.x % HR);
    const int row = hr % p.RB * C::ROWS + static_cast<int>(blockIdx.y);
    if (row >= p.R) return;
    const size_t out = (static_cast<size_t>(b) * a.pool.Hkv + hr / p.RB) * p.R + row;
    const int nt = att_tiles(a, b);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + out * D + threadIdx.x;
    if (nt == 0) {
        *o = __float2bfloat16_rn(0.f);
        if (threadIdx.x == 0) a.lse[out] = -INFINITY;
        return;
    }
    const long long before = att_prefix(a, b, D, scratch);
    const long long total = att_prefix(a, a.B, D, scratch) * HR;
    const long long runs = att_runs(total, ctas);
    const long long xs = before * HR + static_cast<long long>(hr) * nt, xe = xs + nt;
    // run of tile x: the last r with total·r / runs <= x
    const auto run_of = [&](long long x) {
        long long r = x * runs / total;
        while (r + 1 < runs && total * (r + 1) / runs <= x) ++r;
        return r;
    };
    const long long r0 = run_of(xs), r1 = run_of(xe - 1);
    if (r0 == r1) return;                                  // one run held the whole segment
    const int r = static_cast<int>(blockIdx.y);
    const auto part_of = [&](long long run) {
        const bool first = run > r0 || total * run / runs == xs;
        return a.ws + (2 * static_cast<size_t>(run) + (first ? 0 : 1)) * C::PART;
    };
    float M = -INFINITY;
    for (long long q = r0; q <= r1; ++q) M = fmaxf(M, part_of(q)[C::ROWS * D + 2 * r]);
    float L = 0.f, v = 0.f;
    for (long long q = r0; q <= r1; ++q) {
        const float* part = part_of(q);
        const float mq = part[C::ROWS * D + 2 * r];
        if (mq == -INFINITY) {
            L += part[C::ROWS * D + 2 * r + 1];
            continue;
        }
        const float f = ex2_approx(mq - M);
        L = fmaf(f, part[C::ROWS * D + 2 * r + 1], L);
        v = fmaf(f, part[r * D + threadIdx.x], v);
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    *o = __float2bfloat16_rn(v * inv);
    if (threadIdx.x == 0) a.lse[out] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttLn2;
}

template <int D, int NT>
cudaError_t launch_attend(const Kv4AttendArgs& a, cudaStream_t stream) {
    using C = AttCfg<D, NT>;
    AttParams p;
    p.a = a;
    p.scale_log2 = a.scale * kAttLog2e;
    p.R = a.H / a.pool.Hkv * a.nq;
    p.RB = (p.R + C::ROWS - 1) / C::ROWS;
    cudaError_t e = cudaFuncSetAttribute(kv4_attend_kernel<D, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const long long segs = static_cast<long long>(a.B) * a.pool.Hkv * p.RB;
    if (segs > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    int ctas = 148 * C::CTAS;
    if (ctas > kAttMaxCtas) ctas = kAttMaxCtas;
    kv4_attend_kernel<D, NT><<<ctas, kAttThreads, C::SMEM, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int rows = p.R < C::ROWS ? p.R : C::ROWS;
    kv4_join_kernel<D, NT><<<dim3(static_cast<unsigned>(segs), rows), D, 0, stream>>>(p, ctas);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_attend_d(const Kv4AttendArgs& a, cudaStream_t stream) {
    // 8 rows at a time, or 16 where a K/V head has more: the second 8 reuse what was unpacked
    return a.H / a.pool.Hkv * a.nq <= 8 ? launch_attend<D, 1>(a, stream) : launch_attend<D, 2>(a, stream);
}

template <int D>
cudaError_t launch_rows(const Kv4RowsArgs& a, bool append, cudaStream_t stream) {
    const long long blocks = (static_cast<long long>(a.n) + 15 + kKv4Block - 1) / kKv4Block;
    const dim3 grid(static_cast<unsigned>(blocks), a.pool.Hkv, a.B);
    if (append) kv4_append_kernel<D><<<grid, kRowThreads, 0, stream>>>(a);
    else kv4_gather_kernel<D><<<grid, kRowThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_rows_d(const Kv4RowsArgs& a, bool append, cudaStream_t stream) {
    switch (a.pool.d) {
        case 32: return launch_rows<32>(a, append, stream);
        case 64: return launch_rows<64>(a, append, stream);
        case 128: return launch_rows<128>(a, append, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t stream) {
    return launch_rows_d(a, true, stream);
}

cudaError_t launch_kv4_gather(const Kv4RowsArgs& a, cudaStream_t stream) {
    return launch_rows_d(a, false, stream);
}

size_t kv4_attend_ws_bytes(int H, int Hkv, int nq, int d) {
    const int rows = static_cast<long long>(H / Hkv) * nq <= 8 ? 8 : 16;
    return 2 * static_cast<size_t>(kAttMaxCtas) * rows * (d + 2) * sizeof(float);
}

cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, cudaStream_t stream) {
    switch (a.pool.d) {
        case 32: return launch_attend_d<32>(a, stream);
        case 64: return launch_attend_d<64>(a, stream);
        case 128: return launch_attend_d<128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
