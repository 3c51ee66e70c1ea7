// The 4-bit paged K/V cache: its layout, and the launch interface of its kernels (kv4.cu, pages.cu)
// for the C-ABI layer.
//
// A group is 32 channels of one token and K/V head. It is held as whole numbers q in 0..15 and two
// bf16 parameters, lo = the group's least value (itself a bf16 input, so exact) and
// s = bf16((greatest - lo) / 15), and stands for lo + s·q. 16 consecutive tokens of one head make a
// block of 20·d bytes; a page holds page_size / 16 blocks of each head, one head after the other.
//   [0, 8d)     K: words (half, row, c, group); token = 8·half + row; nibble j + 4·h of the word is
//               channel 32·group + 8·c + 2·j + h
//   [8d, 16d)   V: words (half, row, c, group); the low 16 bits are token 8·half + 2·c, the high ones
//               the next; nibble j of 16 bits is channel 32·group + 4·row + j
//   [16d, 18d)  K parameters (token, group): s in the low 16 bits of a word, lo in the high ones
//   [18d, 20d)  V parameters
// (half < 2, row < 8, c < 4, j < 4, h < 2). Lane 4·row + c of a warp so finds its words of an mma
// fragment of 16 tokens side by side: two (d = 128: 16-byte) conflict-free reads for K and two for V,
// with no exchange between lanes; masks of 4 bits are the only unpacking.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

constexpr int kKv4Block = 16;                                   // tokens per block
__host__ __device__ constexpr int kv4_block_bytes(int d) { return 20 * d; }

struct Kv4Pool {
    uint8_t* data;         // (pages, Hkv, page_size / 16, 20·d) bytes
    const int* table;      // (slots, max_pages) page of each page_size tokens, -1: none
    const int* seqs;       // table row of each batch entry, nullptr: its own index
    int pages, slots, max_pages, page_size, Hkv, d;
};

struct Kv4RowsArgs {       // append and gather: rows [0, n) of each batch entry at start[i] + row
    Kv4Pool pool;
    const int* start;      // first token, negative: the entry is left out
    const int* counts;     // rows in use, nullptr: n
    void* k;               // (B, Hkv, n, d) bf16
    void* v;
    int B, n;
};

struct Kv4AttendArgs {
    Kv4Pool pool;
    const int* lens;       // tokens of each table row
    const void* q;         // (B, H, nq, d) bf16
    void* o;
    float* lse;            // (B, H, nq)
    int B, H, nq;
    float scale;
    int wl, wr, ns;        // visible window and sinks (see MaskSpec), off = len - nq
    float* ws;
    uint64_t timeout_ns;
};

// One warp's ring of `ST` stages in the cache's attention: steps [0, issued) were started, [0, taken) waited
// for and used. A wait that runs out changes nothing here, so that the steps [taken, issued) are always the
// copies that may still be on their way.
template <int ST>
struct Kv4Ring {
    int issued = 0, taken = 0;
    int fill = 0, use = 0;         // stages of steps `issued` and `taken`
    uint32_t phase = 0;            // of step `taken`
    __host__ __device__ void start() {
        ++issued;
        fill = fill + 1 == ST ? 0 : fill + 1;
    }
    __host__ __device__ void take() {
        ++taken;
        if (++use == ST) {
            use = 0;
            phase ^= 1u;
        }
    }
};

cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t stream);
cudaError_t launch_kv4_gather(const Kv4RowsArgs& a, cudaStream_t stream);
cudaError_t launch_kv4_attend(const Kv4AttendArgs& a, cudaStream_t stream);
size_t kv4_attend_ws_bytes(int H, int Hkv, int nq, int d);

}  // namespace attn
