// Kernels of the 4-bit paged K/V cache (layout and formulas: kv4.h): quantising new rows into their
// pages, reading rows back, and attention of a few new tokens per sequence over the cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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
// Append and gather. One CTA of 128 threads per (block of 16 tokens, head, batch entry); a team of 4
// lanes holds a group of one token, 8 channels per lane: extrema take two shuffles, a lane's nibbles
// of K are one word and those of V two 16-bit units, so nothing is exchanged to pack them. Blocks
// that the rows fill are put together in shared memory and copied out in 16-byte pieces; at the ragged
// ends each token's own 2- and 4-byte units are stored (neighbours' tokens are never touched).
// Bound by instruction issue for long chunks (about 12 per value), by latency (length, table entry,
// then store) for single tokens.
// ------------------------------------------------------------------------------------------
constexpr int kRowThreads = 128;

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {       // NaN if either is
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// One lane's 8 channels (bf16 in w) of a group shared by 4 lanes: whole numbers, each in the low bits
// of a word, and the group's parameter word. Least and greatest travel as one word (lo, -hi), both by
// minima. (x - lo)/s is taken as t·(1/s), t = x - lo, within a few 2^-22 of it, which decides unless it
// lies next to a border; there what is left of t, t - n·s (exact: n·s has 12 bits), is compared with
// s/2. Exact ties are common among bf16 values (1 in 500, 40% of the warps), so that path is short.
// Likewise s = (hi - lo)/15 before its rounding to bf16. No quotient exceeds 15.1: s is at least
// (1 - 2^-8) of a 15th of the range.
__device__ __forceinline__ void kv4_group(uint4 w, uint32_t (&n)[8], uint32_t& param) {
    constexpr uint32_t kNeg = 0x80008000u;
    const uint32_t least = bmin2(bmin2(w.x, w.y), bmin2(w.z, w.w));
    const uint32_t most = bmin2(bmin2(w.x ^ kNeg, w.y ^ kNeg), bmin2(w.z ^ kNeg, w.w ^ kNeg));
    uint32_t e = bmin2(__byte_perm(least, most, 0x5410), __byte_perm(least, most, 0x7632));
    e = bmin2(e, __shfl_xor_sync(0xffffffffu, e, 1));
    e = bmin2(e, __shfl_xor_sync(0xffffffffu, e, 2));
    const float lo = __uint_as_float(e << 16), range = -__uint_as_float(e & 0xffff0000u) - lo;
    float s = range * (1.f / 15.f);
    if ((__float_as_uint(s) & 0xffffu) - 0x7ffeu <= 4u) s = __fdiv_rn(range, 15.f);
    uint32_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    s = __uint_as_float(sb << 16);
    float inv = __fdividef(1.f, s);                       // s < 2^125
    if (!(s >= 0x1p-100f && s < INFINITY)) {
        // nothing to tell apart, or a NaN or an infinity, which make the whole group NaN
        sb = s < 0x1p-100f ? 0u : 0x7fc0u;
        s = inv = 0.f;
    }
    param = sb | e << 16;
    constexpr float kWhole = 12582912.f;                  // 1.5·2^23: adding it rounds to a whole number
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16) - lo;
        const float r = fmaf(t, inv, kWhole);
        far = fmaxf(far, fabsf(fmaf(t, inv, kWhole - r)));
        n[i] = __float_as_uint(r);
    }
    if (far > 0.4999f) {
        const float half = 0.5f * s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16), t = x - lo;
            const float rest = fmaf(kWhole - __uint_as_float(n[i]), s, t);
            if (fabsf(rest) >= half) {
                // t may have lost some of x - lo; at a tie that decides, or else the even number
                const float b = t - x, lost = copysignf(1.f, rest) * ((x - (t - b)) + (-lo - b));
                const bool out = fabsf(rest) > half || lost > 0.f || (lost == 0.f && (n[i] & 1u));
                if (out) n[i] += rest > 0.f ? 1u : 0xffffffffu;
            }
        }
    }
    if (s == 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = 0;
    }
}

// A team's task of round x: K or V, token of the block, group. kRowThreads / 4 = 32 teams take the
// 2·16·G tasks in G rounds; a warp's tasks of one round are all K or all V.
struct RowTask {
    int kv, tok, g;
};
template <int G>
__device__ __forceinline__ RowTask row_task(int x) {
    const int id = x * (kRowThreads / 4) + (threadIdx.x >> 2);
    return RowTask{id / (16 * G), id % (16 * G) / G, id % G};
}

// Bytes of a token's group in its block: K word of lane c, first V unit of lane c (the second lies 16·G
// bytes on: the next row), parameters.
template <int D>
__device__ __forceinline__ int kv4_k_at(int tok, int g, int c) {
    return (((tok >> 3) * 32 + (tok & 7) * 4 + c) * (D / 32) + g) * 4;
}
template <int D>
__device__ __forceinline__ int kv4_v_at(int tok, int g, int c) {
    return 8 * D + (((tok >> 3) * 32 + 8 * c + ((tok & 7) >> 1)) * (D / 32) + g) * 4 + (tok & 1) * 2;
}
template <int D>
__device__ __forceinline__ int kv4_p_at(int kv, int tok, int g) {
    return (16 + 2 * kv) * D + (tok * (D / 32) + g) * 4;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4RowsArgs a) {
    constexpr int G = D / 32, BB = kv4_block_bytes(D);
    __shared__ __align__(16) uint8_t stage[BB];
    const int i = blockIdx.z, h = blockIdx.y;
    const int first = a.start[i];
    const int count = min(a.counts ? a.counts[i] : a.n, a.n);
    if (first < 0 || count < 1) return;
    const long long blk = first / kKv4Block + static_cast<long long>(blockIdx.x);
    const long long t0 = blk * kKv4Block - first;        // row of the block's first token
    if (t0 >= count) return;
    const bool whole = t0 >= 0 && t0 + kKv4Block <= count;
    const int lo = t0 < 0 ? static_cast<int>(-t0) : 0;   // tokens [lo, hi) of the block are rows
    const int hi = static_cast<int>(min(count - t0, static_cast<long long>(kKv4Block)));
    const int slot = a.pool.seqs ? a.pool.seqs[i] : i;
    const int c = threadIdx.x & 3;
    const long long base = (static_cast<long long>(i) * a.pool.Hkv + h) * a.n + t0;
    uint4 w[G];
#pragma unroll
    for (int x = 0; x < G; ++x) {        // all loads before the first use, and before the page's number
        const RowTask t = row_task<G>(x);
        w[x] = make_uint4(0u, 0u, 0u, 0u);
        if (t.tok >= lo && t.tok < hi)
            w[x] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(t.kv ? a.v : a.k) +
                                                   (base + t.tok) * D + t.g * 32 + c * 8);
    }
    const int pg = kv4_page(a.pool, slot, blk * kKv4Block);
    if (pg < 0) return;
    uint8_t* block = kv4_block(a.pool, pg, h, blk * kKv4Block);
    uint8_t* out = whole ? stage : block;
#pragma unroll
    for (int x = 0; x < G; ++x) {
        const RowTask t = row_task<G>(x);
        uint32_t n[8], param;
        kv4_group(w[x], n, param);
        if (t.tok < lo || t.tok >= hi) continue;
        if (t.kv == 0) {
            const uint32_t even = n[0] + (n[2] << 4) + (n[4] << 8) + (n[6] << 12);
            const uint32_t odd = n[1] + (n[3] << 4) + (n[5] << 8) + (n[7] << 12);
            *reinterpret_cast<uint32_t*>(out + kv4_k_at<D>(t.tok, t.g, c)) = __byte_perm(even, odd, 0x5410);
        } else {
            uint8_t* v = out + kv4_v_at<D>(t.tok, t.g, c);
            *reinterpret_cast<uint16_t*>(v) =
                static_cast<uint16_t>(n[0] + (n[1] << 4) + (n[2] << 8) + (n[3] << 12));
            *reinterpret_cast<uint16_t*>(v + 16 * G) =
                static_cast<uint16_t>(n[4] + (n[5] << 4) + (n[6] << 8) + (n[7] << 12));
        }
        if (c == 0) *reinterpret_cast<uint32_t*>(out + kv4_p_at<D>(t.kv, t.tok, t.g)) = param;
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
    const int c = threadIdx.x & 3;
    const int lo = t0 < 0 ? static_cast<int>(-t0) : 0;   // tokens [lo, hi) are rows, [lo, held) in use
    const int hi = static_cast<int>(min(a.n - t0, static_cast<long long>(kKv4Block)));
    const int held = pg < 0 ? 0 : static_cast<int>(min(count - t0, static_cast<long long>(kKv4Block)));
    const long long base = (static_cast<long long>(i) * a.pool.Hkv + h) * a.n + t0;
#pragma unroll
    for (int x = 0; x < G; ++x) {
        const RowTask t = row_task<G>(x);
        if (t.tok < lo || t.tok >= hi) continue;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (t.tok < held) {
            uint32_t n[2];               // 4 nibbles each: channels 0 .. 3 and 4 .. 7
            if (t.kv == 0) {             // channels (0, 1), (2, 3) .. in bits 4·j and 4·j + 16
                const uint32_t k = *reinterpret_cast<const uint32_t*>(stage + kv4_k_at<D>(t.tok, t.g, c));
                n[0] = (k & 0xfu) | (k >> 12 & 0xf0u) | (k << 4 & 0xf00u) | (k >> 8 & 0xf000u);
                const uint32_t k2 = k >> 8;
                n[1] = (k2 & 0xfu) | (k2 >> 12 & 0xf0u) | (k2 << 4 & 0xf00u) | (k2 >> 8 & 0xf000u);
            } else {
                const uint8_t* v = stage + kv4_v_at<D>(t.tok, t.g, c);
                n[0] = *reinterpret_cast<const uint16_t*>(v);
                n[1] = *reinterpret_cast<const uint16_t*>(v + 16 * G);
            }
            const uint32_t p = *reinterpret_cast<const uint32_t*>(stage + kv4_p_at<D>(t.kv, t.tok, t.g));
            const float s = __uint_as_float(p << 16), least = __uint_as_float(p & 0xffff0000u);
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // 2^23 + q, less 2^23: cheaper than a conversion
                const float q0 = __uint_as_float((n[e / 2] >> (8 * (e % 2)) & 15u) | 0x4b000000u) - 8388608.f;
                const float q1 = __uint_as_float((n[e / 2] >> (8 * (e % 2) + 4) & 15u) | 0x4b000000u) - 8388608.f;
                y[e] = pack_bf16x2(fmaf(s, q0, least), fmaf(s, q1, least));
            }
            w = make_uint4(y[0], y[1], y[2], y[3]);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(t.kv ? a.v : a.k) + (base + t.tok) * D + t.g * 32 +
                                  c * 8) = w;
    }
}

// ------------------------------------------------------------------------------------------
// Attention over the cache.
//
// All query rows of one K/V head (its query heads times nq tokens) share every byte that is read,
// so a (batch entry, K/V head, block of 8·NT rows) is one segment of work, its keys the blocks of
// 16 tokens that any row sees: those of the sinks, then those of the window. The segments' tiles
// (8 blocks, or 4) laid end to end are cut into equal runs, one per CTA, whatever the lengths of the
// sequences; a CTA writes the segments it holds whole and leaves the parts of the others in
// the workspace, where a second launch joins them with the rule that joins two softmax blocks.
//
// Each of a CTA's 4 warps takes its blocks of a tile through a ring of its own (bulk copies
// of whole blocks, contiguous in memory, one mbarrier per stage): no barrier among the warps until a
// segment ends. The two products run as mma.m16n8k16 (fp16 in, fp32 sums); tcgen05's smallest tile
// of 128 rows would be filled to 1/16 to 1/128 by the 1 to 8 rows there are, and its operands would
// first have to be unpacked into shared memory.
//   S (16 keys x 8 rows) = K · Q^T. A nibble masked out of its word IS the fp16 number q·2^-24 (or,
//   from the next position, 16·q·2^-24): both are subnormals, which the tensor cores take exactly, so
//   unpacking a word of 8 costs 4 ANDs and a shift. Q is scaled by a power of two that brings the row's
//   largest value to 2^14 .. 2^15 (its bf16 values are then exact in fp16 down to 2^-27 of the largest;
//   channels that meet 16·q carry Q/16). Per group g: S += s_g·acc_g + lo_g·sum_g(Q), in fp32.
//   O^T (channels x 8 rows) += V^T · P^T with P·s_g in fp16, scaled by a power of two of the row's own
//   that brings the largest P·s it has seen to 2^2 .. 2^3 or above (11 bits down to 2^-16 of that, errors
//   of 2^-27 of it below), and transposed between the fragment layouts by movmatrix; lo's share, sum of
//   P·lo_g, stays in fp32. (The largest s of the cache would not do: a row may give all its weight to
//   tokens whose values are far below another's.)
// Running maximum, sum, O and the power of two are per warp and row; they move only when a score exceeds
// the maximum by more than 8 (P up to 2^8) or a P·s reaches 2^15 (the result does not depend on it). The
// row's own power of two and its test cost 2% (64 sequences up to 8192, 32 heads on 8, d 128: 87.9 us
// against 85.9 with one for all rows that follows s; a cheaper, looser test of a lane's largest P times its
// largest s: 88.4).
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
    // blocks a warp takes per step: two where they hide each other's latency and registers allow (d =
    // 128: 50 against 58 us on one sequence of 131072); with smaller d one (16 sequences, 4 rows, d 64,
    // window 1024: 17.2 against 18.6 us)
    static constexpr int BL = NT == 1 && D == 128 ? 2 : 1;
    static constexpr int TILE = kAttWarps * BL;                         // blocks per tile
    static constexpr int SB = BL * BB;                                  // bytes per stage
    static constexpr int STAGES = D == 128 ? (NT == 1 ? 3 : 4) : 8;
    static constexpr int CTAS = NT == 1 ? (D == 128 ? 3 : 4) : 2;       // per SM
    static constexpr int RING = kAttWarps * STAGES * SB;
    static constexpr int OPAD = D + 4;
    static constexpr int SLOT = ROWS * (OPAD + 2);                      // floats: O rows, then (m, l)
    static constexpr int MERGE = 2 * SLOT * 4;
    static constexpr int QFRAG = NT * G * 32 * 16;                      // Q's fragments
    static constexpr int SMEM = RING + MERGE + QFRAG + kAttWarps * STAGES * 8 + 512;   // and AttShared
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

__device__ __forceinline__ int att_tiles(const AttSeq& s, int tile) { return (s.nb + tile - 1) / tile; }

// Sum of v over the CTA's threads below this one, and over all of them (`scratch`: one per warp).
__device__ __forceinline__ long long att_scan(long long v, long long* all, long long* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
        if (w < warp) before += scratch[w];
        sum += scratch[w];
    }
    __syncthreads();
    *all = sum;
    return before + incl - v;
}

// The line that is cut into runs: segment after segment, each kAttSwitch places for beginning it (a
// CTA that holds many short segments would finish last otherwise: 64 sequences of 1 to 8192 tokens
// took 112 us without, 103, 89, 87 and 89 us with 1, 3, 4 and 6 places) and one place per tile. Where
// runs are short anyway, the switches are not counted. (tiles, segments) of the entries below one are
// summed in one word.
constexpr int kAttSwitch = 4;
__device__ __forceinline__ long long att_pair(const AttSeq& s, int tile) {
    return s.nb > 0 ? static_cast<long long>(att_tiles(s, tile)) << 16 | 1 : 0;
}
__device__ __forceinline__ int att_switch(long long pairs, int HR, int ctas) {
    return (pairs >> 16) * HR >= 4LL * ctas ? kAttSwitch : 0;
}
__device__ __forceinline__ long long att_line(long long pairs, int HR, int sw) {
    return ((pairs >> 16) + (pairs & 0xffff) * sw) * HR;
}

// Runs that a line of `total` places is cut into (one per CTA), and the first place of run k. Almost
// always 32 bits do: a 64-bit division takes ten times as long, and every CTA waits for it.
__host__ __device__ inline long long att_runs(long long total, int ctas) {
    return total < ctas ? total : ctas;
}
__device__ __forceinline__ long long att_run_start(long long total, int k, long long runs) {
    if (total < (1LL << 22)) return static_cast<unsigned>(total) * static_cast<unsigned>(k) / static_cast<unsigned>(runs);
    return total * k / runs;
}
// Run that holds place x: the last k with total·k / runs <= x.
__device__ __forceinline__ int att_run_of(long long x, long long total, long long runs) {
    long long k = total < (1LL << 22) ? static_cast<unsigned>(x) * static_cast<unsigned>(runs) / static_cast<unsigned>(total)
                                      : x * runs / total;
    while (k + 1 < runs && att_run_start(total, static_cast<int>(k) + 1, runs) <= x) ++k;
    return static_cast<int>(k);
}

// D = A·B + C, fp16 operands.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

// D = A·B + C, bf16 operands, 8 or 16 along the sum.
template <bool K16>
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
    if constexpr (K16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%4,%5}, {%6,%7}, "
            "{%8,%9,%10,%11};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    else
        asm(
            "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
            "{%7,%8,%9,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(b0), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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

// A run's part of a segment: batch entry, (K/V head, row block), the tiles [t0, t1) that the run holds,
// the place of t0 on the line, and which of the run's parts it is.
struct AttPart {
    AttSeq seq;
    int b, hr, t0, t1;
    long long x;
    int number;
};

struct AttShared {
    long long scratch[kAttWarps];
    AttPart part, fetch[kAttWarps];     // the computation's place, and each warp's fetching
    int abort, more;
};
static_assert(sizeof(AttShared) <= 512, "shared block");

// Clips the part to the run's end, or moves on to the next segment (false: the run is over).
template <int TILE>
__device__ __forceinline__ void att_clip(AttPart& q, long long x1) {
    q.t1 = static_cast<int>(min(static_cast<long long>(att_tiles(q.seq, TILE)), q.t0 + (x1 - q.x)));
}
template <int TILE>
__device__ __forceinline__ bool att_next(const Kv4AttendArgs& a, AttPart& q, int HR, int sw, long long x1) {
    if (q.t1 < att_tiles(q.seq, TILE)) return false;
    q.x += q.t1 - q.t0 + sw;
    if (q.x >= x1) return false;
    q.t0 = 0;
    ++q.number;
    if (++q.hr == HR) {
        q.hr = 0;
        do {
            if (++q.b >= a.B) return false;            // only if lens changed under the call
            q.seq = att_seq(a, q.b);
        } while (q.seq.nb == 0);
    }
    att_clip<TILE>(q, x1);
    return true;
}

// Steps of warp w in the part: its blocks begin at list positions TILE·t + BL·w below nb.
template <int TILE, int BL>
__device__ __forceinline__ int att_steps(const AttPart& q, int w) {
    const int rest = q.seq.nb - 1 - BL * w;
    const int last = rest >= 0 ? rest / TILE : -1;             // its last tile
    return max(min(q.t1, last + 1) - q.t0, 0);
}

template <int D, int NT>
__global__ void __launch_bounds__(kAttThreads, AttCfg<D, NT>::CTAS) kv4_attend_kernel(const AttParams p) {
    using C = AttCfg<D, NT>;
    constexpr int G = C::G, ST = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* merge = reinterpret_cast<float*>(smem + C::RING);
    uint4* qfrag = reinterpret_cast<uint4*>(smem + C::RING + C::MERGE);   // [NT][G][lane]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING + C::MERGE + C::QFRAG);
    AttShared* sh = reinterpret_cast<AttShared*>(bars + kAttWarps * ST);
    volatile int* abort = &sh->abort;
    const Kv4AttendArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * ST * C::SB;
    uint64_t* full = bars + warp * ST;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kAttWarps * ST; ++s) mbar_init(&bars[s], 1);
        sh->abort = 0;
        sh->part.b = -1;
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");    // the joining launch may be set up
    // ---- this CTA's run of tiles, and the segment it begins in
    const int HR = a.pool.Hkv * p.RB;
    long long x1;
    int sw;
    {
        // a thread per batch entry; the one that holds the run's first tile writes down the place.
        // More entries than threads: chunks of them, once for the total and once for the place
        long long total = 0, before = 0;
        AttSeq mine{};
        for (int b0 = 0; b0 < a.B; b0 += kAttThreads) {
            const int b = b0 + static_cast<int>(threadIdx.x);
            mine.nb = 0;
            if (b < a.B) mine = att_seq(a, b);
            long long all;
            before = total + att_scan(att_pair(mine, C::TILE), &all, sh->scratch);
            total += all;
        }
        sw = att_switch(total, HR, gridDim.x);
        total = att_line(total, HR, sw);
        const long long runs = att_runs(total, gridDim.x);
        if (blockIdx.x >= runs) return;
        const long long x0 = att_run_start(total, blockIdx.x, runs);
        x1 = att_run_start(total, blockIdx.x + 1, runs);
        long long chunk = 0;
        for (int b0 = 0; b0 < a.B; b0 += kAttThreads) {
            const int b = b0 + static_cast<int>(threadIdx.x);
            if (a.B > kAttThreads) {
                mine.nb = 0;
                if (b < a.B) mine = att_seq(a, b);
                long long all;
                before = chunk + att_scan(att_pair(mine, C::TILE), &all, sh->scratch);
                chunk += all;
            }
            const int nt = att_tiles(mine, C::TILE);
            const long long at = x0 - att_line(before, HR, sw), each = nt + sw;
            if (nt > 0 && at >= 0 && at < each * HR) {
                AttPart q;
                q.seq = mine;
                q.b = b;
                q.number = 0;
                q.hr = static_cast<int>(at < (1LL << 31) ? static_cast<unsigned>(at) / static_cast<unsigned>(each)
                                                         : at / each);
                q.t0 = max(static_cast<int>(at - q.hr * each) - sw, 0);
                q.x = x0 - at + q.hr * each + sw + q.t0;
                if (q.x >= x1) continue;               // the run has places but no tile
                att_clip<C::TILE>(q, x1);
                sh->part = q;
                for (int w = 0; w < kAttWarps; ++w) sh->fetch[w] = q;
            }
        }
        __syncthreads();
        if (sh->part.b < 0) return;        // no tile
    }
    const AttPart& q = sh->part;
    const int bpp = a.pool.page_size / kKv4Block;
    const int step_pages = C::TILE / bpp, step_blocks = C::TILE % bpp;    // one tile on
    const uint64_t lim = a.timeout_ns;

    // ---- fetching: its own place in the run, ST steps ahead of the computation's. Lane i < BL holds
    // block i of the warp's next step: block f_blk of page column f_col, the page's number loaded one
    // step ahead of its use; `left` steps remain in the place's part.
    AttPart& f = sh->fetch[warp];
    int left = 0, f_li = 0, f_sb = 0, f_nb = 0, f_col = 0, f_blk = 0, n_blk = 0, pid = -1;
    const int* row = nullptr;              // the sequence's row of the table
    const uint8_t* heads = nullptr;        // page 0's blocks of the part's head
    bool more = true;
    const size_t page_bytes = static_cast<size_t>(a.pool.Hkv) * bpp * C::BB;
    auto place = [&]() {                   // column and block of list position f_li
        const int tb = f_li < f_sb ? f_li : f.seq.wb0 + f_li - f_sb;
        f_col = tb / bpp;
        f_blk = tb - f_col * bpp;
    };
    auto open = [&]() {
        left = att_steps<C::TILE, C::BL>(f, warp);
        f_li = f.t0 * C::TILE + warp * C::BL + lane;
        f_sb = f.seq.sb;
        f_nb = lane < C::BL ? f.seq.nb : 0;
        place();
        row = a.pool.table + static_cast<size_t>(f.seq.slot) * a.pool.max_pages;
        heads = a.pool.data + static_cast<size_t>(f.hr / p.RB) * bpp * C::BB;
    };
    auto look = [&]() {                    // starts loading the page numbers of the next step
        while (left == 0) {
            __syncwarp();
            int go = 0;
            if (lane == 0) go = att_next<C::TILE>(a, f, HR, sw, x1);
            go = __shfl_sync(0xffffffffu, go, 0);
            __syncwarp();
            if (!go) {
                more = false;
                return;
            }
            open();
        }
        pid = f_li < f_nb ? row[f_col] : -1;
        n_blk = f_blk;
        --left;
        const bool in_sinks = f_li < f_sb;
        f_li += C::TILE;
        f_col += step_pages;
        f_blk += step_blocks;
        if (f_blk >= bpp) {
            f_blk -= bpp;
            ++f_col;
        }
        if (in_sinks && f_li >= f_sb) place();
    };
    uint32_t valid = 0;                    // BL bits per stage: blocks on a page
    Kv4Ring<ST> steps;
    auto fetch = [&]() {
        if (!more) return;
        const int fs = steps.fill;
        const bool held = static_cast<unsigned>(pid) < static_cast<unsigned>(a.pool.pages);
        const uint32_t bits = __ballot_sync(0xffffffffu, held);
        valid = (valid & ~(((1u << C::BL) - 1u) << (fs * C::BL))) | bits << (fs * C::BL);
        if (lane == 0) mbar_arrive_expect_tx(&full[fs], __popc(bits) * C::BB);
        __syncwarp();
        if (held)
            bulk_load(ring + fs * C::SB + lane * C::BB,
                      heads + static_cast<size_t>(pid) * page_bytes + static_cast<size_t>(n_blk) * C::BB, C::BB,
                      &full[fs]);
        steps.start();
        look();
    };
    open();
    look();
    for (int s = 0; s < ST; ++s) fetch();

    while (true) {
        // ---- one segment's part of the run
        const int head = q.hr / p.RB, row0 = q.hr % p.RB * C::ROWS;
        const size_t qbase = (static_cast<size_t>(q.b) * a.pool.Hkv + head) * p.R;
        // Q as the B operand of S: lane (gid, c) holds row gid, channels 32·g + 8·c .. + 7. qs is the
        // B operand that meets the keys' lo: scale·log2(e)·(sum over each group) in three bf16 parts
        // (Q lies in shared memory: the 4 warps read the same fragments, and 16 registers fewer let four
        // CTAs stay on an SM)
        uint32_t qs[NT][2];
        float cq[NT][2];            // scale·log2(e)·2^24 / (Q's power of two), of rows 2c, 2c + 1
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
                sum[g] *= p.scale_log2;
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax in 2^(e-127) .. 2^(e-126): times 2^(141-e) it lies in 2^14 .. 2^15
            const int up = min(141 - static_cast<int>(__float_as_uint(amax) >> 23), 127);
            const float fq = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
                uint32_t qf[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float m = (e & 1) ? fq * 0.0625f : fq;
                    qf[e] = pack_f16x2(__uint_as_float(u[e] << 16) * m,
                                       __uint_as_float(u[e] & 0xffff0000u) * m);
                }
                if (warp == 0) qfrag[(n * G + g) * 32 + lane] = make_uint4(qf[0], qf[1], qf[2], qf[3]);
            }
            const float back = ldexpf(p.scale_log2, 24 - up);
            cq[n][0] = __shfl_sync(0xffffffffu, back, 8 * c);
            cq[n][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
            // sums x = hi + mid + low. Along the sum, lane c holds: d = 128 the groups 2·(c & 1) and the
            // next, hi in c < 2, mid in c >= 2, low in c < 2 of the second half; d = 64 both groups,
            // part c; d = 32 (hi, mid) in c = 0, low in c = 1
            uint32_t part[3];
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                const float s0 = G == 4 ? ((c & 1) ? sum[G / 2] : sum[0]) : sum[0];
                const float s1 = G == 4 ? ((c & 1) ? sum[G - 1] : sum[G / 4]) : sum[G - 1];
                float h0 = s0, h1 = s1, b0 = 0.f, b1 = 0.f;
#pragma unroll
                for (int k = 0; k <= t; ++k) {
                    b0 = __bfloat162float(__float2bfloat16_rn(h0));
                    b1 = __bfloat162float(__float2bfloat16_rn(h1));
                    h0 -= b0;
                    h1 -= b1;
                }
                part[t] = pack_bf16x2(b0, b1);
            }
            if constexpr (G == 4) {
                qs[n][0] = c < 2 ? part[0] : part[1];
                qs[n][1] = c < 2 ? part[2] : 0u;
            } else if constexpr (G == 2) {
                qs[n][0] = c == 0 ? part[0] : c == 1 ? part[1] : c == 2 ? part[2] : 0u;
                qs[n][1] = 0u;
            } else {
                qs[n][0] = c == 0 ? (part[0] & 0xffffu) | (part[1] << 16) : c == 1 ? part[2] & 0xffffu : 0u;
                qs[n][1] = 0u;
            }
        }
        __syncthreads();
        // blocks [full_lo, full_hi], and those below full_ns, are seen whole by every row
        const long long lo_key = a.wl < 0 ? 0 : q.seq.off + a.nq - 1 - a.wl;
        const long long hi_key = a.wr < 0 ? q.seq.last : min(q.seq.off + a.wr, static_cast<long long>(q.seq.last));
        const int full_lo = static_cast<int>(max(lo_key + kKv4Block - 1, 0LL) / kKv4Block);
        const int full_hi = hi_key < kKv4Block - 1 ? -1 : static_cast<int>((hi_key + 1) / kKv4Block) - 1;
        const int full_ns = a.ns / kKv4Block;
        // nm = minus the running maximum (0 until a row has seen a key); a score moves it when its
        // excess is above thr.
        float nm[NT][2], thr[NT][2], acc[NT][2 * G][4];
        float l[NT][2], ol[NT][G][2];
        float fv[NT][2];            // power of two on P·s (s is 0 or at least 2^-100)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                nm[n][e] = 0.f;
                thr[n][e] = -INFINITY;
                fv[n][e] = 0x1p118f;
                l[n][e] = 0.f;
#pragma unroll
                for (int g = 0; g < G; ++g) ol[n][g][e] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < 2 * G; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][t][e] = 0.f;
        }
        // One step: BL blocks of 16 keys at blk, token blocks tb[], those that are there in `on`. EDGE:
        // some row does not see some key. Everything is done for all blocks before the next thing, so
        // that their chains of dependent instructions overlap.
        auto step = [&](const uint8_t* blk, const int (&tb)[C::BL], uint32_t on, auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
            constexpr int BL = C::BL;
            // ---- scores relative to the running maximum: t = S - m
            float t[BL][NT][4];     // (key gid, rows 2c, 2c + 1), (key gid + 8, ...)
            float zs[BL][NT][4];
#pragma unroll
            for (int x = 0; x < BL; ++x) {
                const uint8_t* par = blk + x * C::BB + 16 * D;
                uint32_t a0, a1;                 // the keys' lo as the A operand
                if constexpr (G == 4) {
                    const uint2 w0 = *reinterpret_cast<const uint2*>(par + gid * 16 + (c & 1) * 8);
                    const uint2 w1 = *reinterpret_cast<const uint2*>(par + (8 + gid) * 16 + (c & 1) * 8);
                    a0 = __byte_perm(w0.x, w0.y, 0x7632);
                    a1 = __byte_perm(w1.x, w1.y, 0x7632);
                } else {
                    uint32_t w0[G], w1[G];
                    lds_words<G>(w0, par + gid * G * 4);
                    lds_words<G>(w1, par + (8 + gid) * G * 4);
                    a0 = __byte_perm(w0[0], w0[G - 1], 0x7632);
                    a1 = __byte_perm(w1[0], w1[G - 1], 0x7632);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float ref[4] = {nm[n][0], nm[n][1], nm[n][0], nm[n][1]};
                    mma_bf16<G == 4>(t[x][n], a0, a1, qs[n][0], qs[n][1], ref);
                }
                uint32_t k0w[G], k1w[G], p0[G], p1[G];
                lds_words<G>(k0w, blk + x * C::BB + lane * G * 4);
                lds_words<G>(k1w, blk + x * C::BB + (32 + lane) * G * 4);
                lds_words<G>(p0, par + gid * G * 4);
                lds_words<G>(p1, par + (8 + gid) * G * 4);
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t y0 = k0w[g] >> 8, y1 = k1w[g] >> 8;
                    const uint32_t a00 = k0w[g] & 0x000f000fu, a01 = k1w[g] & 0x000f000fu;
                    const uint32_t a02 = k0w[g] & 0x00f000f0u, a03 = k1w[g] & 0x00f000f0u;
                    const uint32_t a10 = y0 & 0x000f000fu, a11 = y1 & 0x000f000fu;
                    const uint32_t a12 = y0 & 0x00f000f0u, a13 = y1 & 0x00f000f0u;
                    const float s0 = __uint_as_float(p0[g] << 16), s1 = __uint_as_float(p1[g] << 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 qf = qfrag[(n * G + g) * 32 + lane];
                        float s[4];
                        mma_f16(s, a00, a01, a02, a03, qf.x, qf.y, zero);
                        mma_f16(s, a10, a11, a12, a13, qf.z, qf.w, s);
                        float(&z)[4] = zs[x][n];
                        z[0] = g == 0 ? s[0] * s0 : fmaf(s[0], s0, z[0]);
                        z[1] = g == 0 ? s[1] * s0 : fmaf(s[1], s0, z[1]);
                        z[2] = g == 0 ? s[2] * s1 : fmaf(s[2], s1, z[2]);
                        z[3] = g == 0 ? s[3] * s1 : fmaf(s[3], s1, z[3]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[x][n][e] = fmaf(zs[x][n][e], cq[n][e & 1], t[x][n][e]);
            }
            // V's parameters of keys gid and gid + 8
            float vs[BL][2][G], vl[BL][2][G], sk[BL][2];       // sk: the largest s of a key's groups
            uint32_t hidden[BL][NT];
#pragma unroll
            for (int x = 0; x < BL; ++x) {
                uint32_t w0[G], w1[G];
                lds_words<G>(w0, blk + x * C::BB + 18 * D + gid * G * 4);
                lds_words<G>(w1, blk + x * C::BB + 18 * D + (8 + gid) * G * 4);
                if constexpr (EDGE) {
                    // keys a row does not see; the parameters of keys that no row sees may be anything
                    const long long k0 = static_cast<long long>(tb[x]) * kKv4Block + gid;
                    const bool there = on >> x & 1u;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        hidden[x][n] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const long long key = k0 + 8 * (e >> 1);
                            const long long at = q.seq.off + (row0 + n * 8 + 2 * c + (e & 1)) % a.nq;
                            const bool seen = there && key <= q.seq.last && (a.wr < 0 || key <= at + a.wr) &&
                                              (a.wl < 0 || key >= at - a.wl || key < a.ns);
                            if (!seen) {
                                t[x][n][e] = -INFINITY;
                                hidden[x][n] |= 1u << e;
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const long long key = k0 + 8 * h;
                        if (!there || key > q.seq.last || (a.wl >= 0 && key < q.seq.off - a.wl && key >= a.ns)) {
#pragma unroll
                            for (int g = 0; g < G; ++g) (h == 0 ? w0 : w1)[g] = 0;
                        }
                    }
                }
                sk[x][0] = sk[x][1] = 0.f;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    vs[x][0][g] = __uint_as_float(w0[g] << 16);
                    vs[x][1][g] = __uint_as_float(w1[g] << 16);
                    vl[x][0][g] = __uint_as_float(w0[g] & 0xffff0000u);
                    vl[x][1][g] = __uint_as_float(w1[g] & 0xffff0000u);
                    sk[x][0] = fmaxf(sk[x][0], vs[x][0][g]);
                    sk[x][1] = fmaxf(sk[x][1], vs[x][1][g]);
                }
            }
            // ---- P, and P times the row's power of two
            float pr[BL][NT][4], pf[BL][NT][4];         // (key gid, rows 2c, 2c + 1), (key gid + 8, ...)
            auto weigh = [&]() {
#pragma unroll
                for (int x = 0; x < BL; ++x)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pr[x][n][e] = ex2_approx(t[x][n][e]);
                            pf[x][n][e] = pr[x][n][e] * fv[n][e & 1];
                        }
            };
            weigh();
            // ---- the running maximum and the power of two move rarely
            float tmax[NT][2], wmax = 0.f;
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    tmax[n][e] = fmaxf(t[0][n][e], t[0][n][2 + e]);
#pragma unroll
                    for (int x = 1; x < BL; ++x) tmax[n][e] = fmax3(tmax[n][e], t[x][n][e], t[x][n][2 + e]);
                    grow |= tmax[n][e] > thr[n][e];
#pragma unroll
                    for (int x = 0; x < BL; ++x)
                        wmax = fmax3(wmax, pf[x][n][e] * sk[x][0], pf[x][n][2 + e] * sk[x][1]);
                }
            if (__any_sync(0xffffffffu, grow || wmax > 32768.f)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float d = tmax[n][e];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, o));
                        const bool up = d > fminf(thr[n][e], 0.f);     // so that P <= 1 below
                        const float al = !up ? 1.f : thr[n][e] == -INFINITY ? 0.f : ex2_approx(-d);
                        if (up) {
                            nm[n][e] -= d;
                            thr[n][e] = 8.f;
#pragma unroll
                            for (int x = 0; x < BL; ++x) {
                                t[x][n][e] -= d;
                                t[x][n][2 + e] -= d;
                            }
                        }
                        l[n][e] *= al;
#pragma unroll
                        for (int g = 0; g < G; ++g) ol[n][g][e] *= al;
                        // the row's largest P·s: of these keys, and 2^2 over the power of two before
                        float w = 0.f;
#pragma unroll
                        for (int x = 0; x < BL; ++x)
                            w = fmax3(w, ex2_approx(t[x][n][e]) * sk[x][0], ex2_approx(t[x][n][2 + e]) * sk[x][1]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
                        const int was = static_cast<int>(__float_as_uint(fv[n][e]) >> 23) - 127;
                        w = fmaxf(w, al * __uint_as_float(static_cast<uint32_t>(129 - was) << 23));
                        // w in 2^(k-127) .. 2^(k-126), times 2^(129-k) in 2^2 .. 2^3; k < 253 (w < 2^126)
                        const int now = min(129 - static_cast<int>(__float_as_uint(w) >> 23), 118);
                        fv[n][e] = __uint_as_float(static_cast<uint32_t>(127 + now) << 23);
                        const float ar = al == 0.f ? 0.f : ex2_approx(static_cast<float>(now - was) + (up ? -d : 0.f));
#pragma unroll
                        for (int k = 0; k < 2 * G; ++k) {
                            acc[n][k][e] *= ar;
                            acc[n][k][2 + e] *= ar;
                        }
                    }
                weigh();
            }
            // ---- P·s in fp16 as the B operand of O^T
#pragma unroll
            for (int x = 0; x < BL; ++x)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    l[n][0] += pr[x][n][0] + pr[x][n][2];
                    l[n][1] += pr[x][n][1] + pr[x][n][3];
                }
#pragma unroll
            for (int x = 0; x < BL; ++x) {
                uint32_t v0w[G], v1w[G];
                lds_words<G>(v0w, blk + x * C::BB + 8 * D + lane * G * 4);
                lds_words<G>(v1w, blk + x * C::BB + 8 * D + (32 + lane) * G * 4);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t y0 = v0w[g] >> 8, y1 = v1w[g] >> 8;
                    const uint32_t a00 = v0w[g] & 0x000f000fu, a01 = v0w[g] & 0x00f000f0u;
                    const uint32_t a02 = v1w[g] & 0x000f000fu, a03 = v1w[g] & 0x00f000f0u;
                    const uint32_t a10 = y0 & 0x000f000fu, a11 = y0 & 0x00f000f0u;
                    const uint32_t a12 = y1 & 0x000f000fu, a13 = y1 & 0x00f000f0u;
                    const float f0 = vs[x][0][g], f1 = vs[x][1][g], u0 = vl[x][0][g], u1 = vl[x][1][g];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float(&P)[4] = pr[x][n];
                        const float(&F)[4] = pf[x][n];
                        float w0 = F[0] * f0, w1 = F[1] * f0, w2 = F[2] * f1, w3 = F[3] * f1;
                        float(&o)[2] = ol[n][g];
                        if constexpr (EDGE) {       // 0 times a NaN or an infinity that the row does not see
                            const uint32_t no = hidden[x][n];
                            if (no & 1u) w0 = 0.f; else o[0] = fmaf(P[0], u0, o[0]);
                            if (no & 2u) w1 = 0.f; else o[1] = fmaf(P[1], u0, o[1]);
                            if (no & 4u) w2 = 0.f; else o[0] = fmaf(P[2], u1, o[0]);
                            if (no & 8u) w3 = 0.f; else o[1] = fmaf(P[3], u1, o[1]);
                        } else {
                            o[0] = fmaf(P[2], u1, fmaf(P[0], u0, o[0]));
                            o[1] = fmaf(P[3], u1, fmaf(P[1], u0, o[1]));
                        }
                        const uint32_t b0 = movmatrix_trans(pack_f16x2(w0, w1));
                        const uint32_t b1 = movmatrix_trans(pack_f16x2(w2, w3));
                        mma_f16(acc[n][2 * g], a00, a01, a02, a03, b0, b1, acc[n][2 * g]);
                        mma_f16(acc[n][2 * g + 1], a10, a11, a12, a13, b0, b1, acc[n][2 * g + 1]);
                    }
                }
            }
        };
        const int mine = att_steps<C::TILE, C::BL>(q, warp);
        const int sb = q.seq.sb, wb0 = q.seq.wb0 - sb;
        int li = q.t0 * C::TILE + warp * C::BL;
        for (int i = 0; i < mine; ++i, li += C::TILE) {
            const int cs = steps.use;
            if (!bounded_wait_warp(&full[cs], steps.phase, abort, lim)) break;
            const uint32_t on = valid >> (cs * C::BL) & ((1u << C::BL) - 1u);
            if (on) {
                int tb[C::BL];
                bool inner = on == (1u << C::BL) - 1u;
#pragma unroll
                for (int x = 0; x < C::BL; ++x) {
                    tb[x] = li + x < sb ? li + x : wb0 + li + x;
                    inner = inner && tb[x] <= full_hi && (tb[x] >= full_lo || tb[x] < full_ns);
                }
                const uint8_t* blk = ring + cs * C::SB;
                if (inner) step(blk, tb, on, std::false_type{});
                else step(blk, tb, on, std::true_type{});
            }
            steps.take();
            __syncwarp();           // every lane has read the stage
            fetch();
        }
        // ---- this warp's part: O unnormalised in units of 2^m, m and l (of rows 2c, 2c + 1)
        float4 o[NT][2][G];         // channels 32·g + 4·gid ..
        float m[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = thr[n][e] == -INFINITY ? -INFINITY : -nm[n][e];
                const float back = 1.f / fv[n][e];         // exact: a power of two
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float t = ol[n][g][e];
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
                    // channels 32·g + 4·gid + j; odd j were multiplied by 16
                    o[n][e][g] = make_float4(fmaf(acc[n][2 * g][e] * 0x1p24f, back, t),
                                             fmaf(acc[n][2 * g][2 + e] * 0x1p20f, back, t),
                                             fmaf(acc[n][2 * g + 1][e] * 0x1p24f, back, t),
                                             fmaf(acc[n][2 * g + 1][2 + e] * 0x1p20f, back, t));
                }
            }
        // ---- the warps' parts are joined in two rounds: 2 and 3 into 0 and 1, then 1 into 0
        auto put = [&](float* slot) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * c + e;
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        *reinterpret_cast<float4*>(slot + r * C::OPAD + g * 32 + gid * 4) = o[n][e][g];
                    if (gid == 0)
                        *reinterpret_cast<float2*>(slot + C::ROWS * C::OPAD + 2 * r) = make_float2(m[n][e], l[n][e]);
                }
        };
        auto take = [&](const float* slot) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * c + e;
                    const float2 ml = *reinterpret_cast<const float2*>(slot + C::ROWS * C::OPAD + 2 * r);
                    const float M = fmaxf(m[n][e], ml.x);
                    // a part that saw no key has O = 0, and l = 0 or NaN when every score was
                    const float fa = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - M);
                    const float fb = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                    l[n][e] = (m[n][e] == -INFINITY ? l[n][e] : fa * l[n][e]) + (ml.x == -INFINITY ? ml.y : fb * ml.y);
                    m[n][e] = M;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const float4 t = *reinterpret_cast<const float4*>(slot + r * C::OPAD + g * 32 + gid * 4);
                        float4& w = o[n][e][g];
                        w.x = fmaf(fb, t.x, fa * w.x); w.y = fmaf(fb, t.y, fa * w.y);
                        w.z = fmaf(fb, t.z, fa * w.z); w.w = fmaf(fb, t.w, fa * w.w);
                    }
                }
        };
        const bool whole = q.t0 == 0 && q.t1 == att_tiles(q.seq, C::TILE);
        float* part = a.ws + (2 * static_cast<size_t>(blockIdx.x) + (q.number == 0 ? 0 : 1)) * C::PART;
        if (warp >= 2) put(merge + (warp - 2) * C::SLOT);
        __syncthreads();
        if (threadIdx.x == kAttThreads - 1) sh->more = att_next<C::TILE>(a, sh->part, HR, sw, x1);   // nobody reads it
        if (warp < 2) take(merge + warp * C::SLOT);
        if (warp == 1) put(merge + C::SLOT);
        __syncthreads();
        const bool more_parts = sh->more;
        // ---- whole segments are finished here, parts go to the workspace
        if (warp == 0) {
            take(merge + C::SLOT);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * c + e;
                    if (row0 + r >= p.R) continue;
                    const float L = l[n][e];
                    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);    // NaN stays
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const float4 w = o[n][e][g];
                        if (whole)
                            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + (qbase + row0 + r) * D +
                                                      g * 32 + gid * 4) =
                                make_uint2(pack_bf16x2(w.x * inv, w.y * inv), pack_bf16x2(w.z * inv, w.w * inv));
                        else
                            *reinterpret_cast<float4*>(part + r * D + g * 32 + gid * 4) = w;
                    }
                    if (gid == 0) {
                        if (whole)
                            a.lse[qbase + row0 + r] = L == 0.f ? -INFINITY : (m[n][e] + log2f(L)) * kAttLn2;
                        else
                            *reinterpret_cast<float2*>(part + C::ROWS * D + 2 * r) = make_float2(m[n][e], L);
                    }
                }
        }
        if (!more_parts) break;
    }
    if (*abort) {                 // let the copies in flight land
        const uint64_t t0 = globaltimer_ns();
        for (; steps.taken < steps.issued; steps.take())
            while (!mbar_try_wait(&full[steps.use], steps.phase))
                if (globaltimer_ns() - t0 > 100000000ull) break;
    }
}

// Joins the parts of segments that several runs share, and clears the rows of batch entries that see
// no key. One CTA per (segment, row): teams of D / 4 lanes take every so many parts, so a long
// sequence's parts (up to the number of runs) are read side by side.
constexpr int kJoinThreads = 128;

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const AttParams p, int ctas) {
    using C = AttCfg<D, NT>;
    constexpr int LPP = D / 4, TEAMS = kJoinThreads / LPP;
    __shared__ long long scratch[2][kJoinThreads / 32];
    __shared__ float4 osum[TEAMS][LPP];
    __shared__ float2 msum[TEAMS];
    const Kv4AttendArgs& a = p.a;
    const int HR = a.pool.Hkv * p.RB;
    const int b = static_cast<int>(blockIdx.x / HR), hr = static_cast<int>(blockIdx.x % HR);
    const int r = static_cast<int>(blockIdx.y), row = hr % p.RB * C::ROWS + r;
    if (row >= p.R) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int team = threadIdx.x / LPP, lane4 = threadIdx.x % LPP;
    const size_t out = (static_cast<size_t>(b) * a.pool.Hkv + hr / p.RB) * p.R + row;
    uint2* o = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + out * D) + lane4;
    // (tiles, segments) of the entries before b and of all
    long long before = 0, total = 0;
    for (int x = threadIdx.x; x < a.B; x += kJoinThreads) {
        const long long t = att_pair(att_seq(a, x), C::TILE);
        total += t;
        if (x < b) before += t;
    }
    const int nt = att_tiles(att_seq(a, b), C::TILE);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, x);
        before += __shfl_xor_sync(0xffffffffu, before, x);
    }
    if ((threadIdx.x & 31) == 0) {
        scratch[0][threadIdx.x >> 5] = total;
        scratch[1][threadIdx.x >> 5] = before;
    }
    __syncthreads();
    total = before = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        total += scratch[0][w];
        before += scratch[1][w];
    }
    const int sw = att_switch(total, HR, ctas);
    total = att_line(total, HR, sw);
    const long long runs = att_runs(total, ctas);
    const long long seg = att_line(before, HR, sw) + static_cast<long long>(hr) * (nt + sw), xs = seg + sw;
    int r0 = 0, r1 = 0, slot0 = 0;
    if (nt > 0) {
        r0 = att_run_of(xs, total, runs);
        r1 = att_run_of(xs + nt - 1, total, runs);
        // the segment is the first of every run's but perhaps the first run's
        slot0 = att_run_start(total, r0, runs) >= seg ? 0 : 1;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the runs' parts are there
    if (nt == 0) {
        if (team == 0) *o = make_uint2(0u, 0u);
        if (threadIdx.x == 0) a.lse[out] = -INFINITY;
        return;
    }
    if (r0 == r1) return;                                  // one run held the whole segment
    const auto part_of = [&](int k) {
        return a.ws + (2 * static_cast<size_t>(k) + (k == r0 ? slot0 : 0)) * C::PART;
    };
    // each team keeps a running maximum over its parts, four of them loaded at a time; a part that saw no
    // key has m = -inf, O = 0, and l = 0 or NaN when every score was
    constexpr int U = 4;
    float M = -INFINITY, L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = r0 + team; k0 <= r1; k0 += U * TEAMS) {
        float2 ml[U];
        float4 t[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const int k = k0 + x * TEAMS;
            const float* part = part_of(min(k, r1));
            ml[x] = *reinterpret_cast<const float2*>(part + C::ROWS * D + 2 * r);
            t[x] = *reinterpret_cast<const float4*>(part + r * D + lane4 * 4);
            if (k > r1) ml[x] = make_float2(-INFINITY, 0.f);
        }
        float top = M;
#pragma unroll
        for (int x = 0; x < U; ++x) top = fmaxf(top, ml[x].x);
        const float old = M == -INFINITY ? 0.f : ex2_approx(M - top);
        M = top;
        L *= M == -INFINITY ? 1.f : old;
        v.x *= old; v.y *= old; v.z *= old; v.w *= old;
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const float f = ml[x].x == -INFINITY ? 0.f : ex2_approx(ml[x].x - M);
            L += ml[x].x == -INFINITY ? ml[x].y : f * ml[x].y;
            if (ml[x].x == -INFINITY) continue;
            v.x = fmaf(f, t[x].x, v.x); v.y = fmaf(f, t[x].y, v.y);
            v.z = fmaf(f, t[x].z, v.z); v.w = fmaf(f, t[x].w, v.w);
        }
    }
    osum[team][lane4] = v;
    if (lane4 == 0) msum[team] = make_float2(M, L);
    __syncthreads();
    if (team != 0) return;
#pragma unroll
    for (int w = 1; w < TEAMS; ++w) M = fmaxf(M, msum[w].x);
    L = 0.f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < TEAMS; ++w) {
        const float2 ml = msum[w];
        const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
        L += ml.x == -INFINITY ? ml.y : f * ml.y;
        const float4 t = osum[w][lane4];
        v.x = fmaf(f, t.x, v.x); v.y = fmaf(f, t.y, v.y);
        v.z = fmaf(f, t.z, v.z); v.w = fmaf(f, t.w, v.w);
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    *o = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    if (lane4 == 0) a.lse[out] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttLn2;
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
    // launched while the runs are still going, up to its wait for them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(segs), static_cast<unsigned>(rows));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT>, p, ctas);
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
