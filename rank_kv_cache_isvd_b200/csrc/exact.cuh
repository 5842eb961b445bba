// Attention over exact KV rows (no factorisation): arguments of its kernels, the partition of the
// work that the split kernel and the merge kernel share, and their launchers.
//
// A sequence b holds n_b = lens[b] rows. The last ql_b = q_lens[b] of them are the call's query
// tokens: token i sits at position p = n_b - ql_b + i and sees the rows j <= p with j < sinks or
// j > p - window. With a shared prefix every token also sees all P prefix rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "iskv.h"

namespace iskv {

constexpr int EX_D = 128;
constexpr int EX_QROWS = 8;            // query rows of a split-kernel tile (tokens x GQA group)
constexpr int EX_REC = EX_QROWS * (2 + EX_D);   // floats of a record: m[8], l[8], O[8][128]
constexpr int EX_MAXREC = 1024;        // records that one merge block can combine
constexpr int EX_PRE_MAX = 256;        // of them at most from the tile kernel

struct ExactArgs {
    const char *k, *v;                 // rows of the sequences
    long long seq_st, head_st, row_st; // bytes
    int B, H, rows;
    const int *lens;                   // NULL: every sequence holds `rows` rows
    const char *q;
    char *out;
    long long q_seq, q_head, q_tok;    // bytes
    long long o_seq, o_head, o_tok;
    int G, m;
    const int *q_lens;                 // NULL: m tokens each
    int window, sinks;
    const char *pk, *pv;               // shared prefix
    long long p_head, p_row;           // bytes
    int P;
    int shared_here;                   // 1: the split kernel computes the shared prefix too
    float *rec;                        // records of the split kernel
    float *scores;                     // mass: scaled scores [B][H][G][score_st], log2 units
    long long score_st;
    const float *mass;
    float *mass_out;
    const float *pre_ml;               // prefix records of the tile kernel: (m, l) [H][nsp][B*G][2]
    const float *pre_o;                //                                   O [H][nsp][B*G][128]
    int nsp;                           // their number of splits (0: none)
    int direct;                        // 1: an item that one block covers writes its outputs itself
    float scale_log2;                  // log2(e) / sqrt(128)
    int grid;                          // blocks of the split kernel
    int after;                         // 1: launched next to the kernel before it, whose end it awaits
};

// Tokens per tile of query rows.
__host__ __device__ inline int ex_tpt(int G) { return EX_QROWS / G; }

__device__ __forceinline__ int ex_len(const ExactArgs &a, int b) {
    const int n = a.lens ? a.lens[b] : a.rows;
    return min(max(n, 0), a.rows);
}
__device__ __forceinline__ int ex_qlen(const ExactArgs &a, int b) {
    const int n = a.q_lens ? a.q_lens[b] : a.m;
    return min(max(n, 0), a.m);
}

// The flat space of steps. Items in order: the shared prefix's (kv-head, tile of 8 (sequence,
// q-head) rows), then every sequence's (kv-head, tile of 8 (token, q-head) rows). An item takes
// S steps of `rs` rows; each block of the split kernel takes `per` consecutive steps.
struct ExactSpan {
    int S;            // steps per item
    int RT;           // tiles per kv-head
};

__device__ __forceinline__ ExactSpan ex_shared_span(const ExactArgs &a, int rs) {
    ExactSpan s;
    const int tpt = ex_tpt(a.G);
    s.S = a.shared_here ? (a.P + rs - 1) / rs : 0;
    s.RT = (a.B + tpt - 1) / tpt;
    return s;
}
// Sequence of n rows and ql tokens. No tile sees more rows than the bound here, and an item has
// a step even where nothing is visible: it writes zeros.
__device__ __forceinline__ ExactSpan ex_seq_span(const ExactArgs &a, int n, int ql, int rs) {
    ExactSpan s;
    const int tpt = ex_tpt(a.G);
    const long long most = (long long)a.sinks + a.window + tpt - 1;
    const int c = most < n ? (int)most : n;
    s.RT = (ql + tpt - 1) / tpt;
    s.S = s.RT ? max(1, (c + rs - 1) / rs) : 0;
    return s;
}

// Steps of all items, by one warp (every lane returns the sum).
__device__ __forceinline__ long long ex_total(const ExactArgs &a, int rs) {
    const int lane = threadIdx.x & 31;
    const ExactSpan p = ex_shared_span(a, rs);
    long long t = 0;
    if (!a.lens && !a.q_lens) {
        const ExactSpan s = ex_seq_span(a, a.rows, a.m, rs);
        t = (long long)a.B * a.H * s.RT * s.S;
    } else {
        for (int b = lane; b < a.B; b += 32) {
            const ExactSpan s = ex_seq_span(a, ex_len(a, b), ex_qlen(a, b), rs);
            t += (long long)a.H * s.RT * s.S;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return t + (long long)a.H * p.RT * p.S;
}

// First flat step of sequence b's items, by one warp.
__device__ __forceinline__ long long ex_first(const ExactArgs &a, int b, int rs) {
    const int lane = threadIdx.x & 31;
    const ExactSpan p = ex_shared_span(a, rs);
    long long t = 0;
    if (!a.lens && !a.q_lens) {
        const ExactSpan s = ex_seq_span(a, a.rows, a.m, rs);
        t = (long long)b * a.H * s.RT * s.S;
    } else {
        for (int i = lane; i < b; i += 32) {
            const ExactSpan s = ex_seq_span(a, ex_len(a, i), ex_qlen(a, i), rs);
            t += (long long)a.H * s.RT * s.S;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return t + (long long)a.H * p.RT * p.S;
}

// Rows per step and threads per block of the split kernel.
constexpr int ex_warps(bool f32_rows) { return f32_rows ? 4 : 8; }
constexpr int ex_step_rows(bool f32_rows) { return 16 * ex_warps(f32_rows); }

cudaError_t launch_exact_split(const ExactArgs &a, bool f32_rows, bool f32_io, cudaStream_t s);
cudaError_t launch_exact_merge(const ExactArgs &a, bool f32_rows, bool f32_io, cudaStream_t s);

}  // namespace iskv
