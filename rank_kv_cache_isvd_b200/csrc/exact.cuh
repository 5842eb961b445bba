// Attention over exact KV rows (no factorisation): arguments of its kernels, the partition of the
// work that the split kernel and the merge kernel share, and their launchers.
//
// A sequence b holds n_b = lens[b] rows. The last ql_b = q_lens[b] of them are the call's query
// tokens: token i sits at position p = n_b - ql_b + i and sees the rows j <= p with j < sinks or
// j > p - window. With a shared prefix every token also sees all P prefix rows.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "exact_order.cuh"
#include "iskv.h"

namespace iskv {

constexpr int EX_D = 128;
constexpr int EX_QROWS = 8;            // query rows of a split-kernel tile (tokens x GQA group)
constexpr int EX_REC = EX_QROWS * (2 + EX_D);   // floats of a record: m[8], l[8], O[8][128]
constexpr int EX_PRE_MAX = 32;         // splits of a shared prefix at most
// A device-side wait polls this often at most, each time suspended for up to so long (5 s in all).
constexpr uint32_t EX_POLLS = ISKV_EXACT_POLLS, EX_SUSPEND_NS = 20000;

struct ExactArgs {
    int B, H, rows;
    const int *lens;                   // NULL: every sequence holds `rows` rows
    const char *q;
    char *out;
    long long q_seq, q_head, q_tok;    // bytes
    long long o_seq, o_head, o_tok;
    int G, m;
    const int *q_lens;                 // NULL: m tokens each
    int window, sinks;
    int P;                             // shared prefix rows
    int shared_here;                   // 1: the split kernel computes the shared prefix too
    int seq_mul, head_mul, p_head_mul; // 0 where all sequences, or kv-heads, share one stream
    float *rec;                        // records of the split kernel
    float *scores;                     // mass: scaled scores [B][H][G][score_st], log2 units
    long long score_st;
    const float *mass;
    float *mass_out;
    const float *pre_ml;               // prefix records of the tile kernel: (m, l) [H][nsp][B*G][2]
    const float *pre_o;                //                                   O [H][nsp][B*G][128]
    int nsp;                           // their number of splits (0: none)
    float scale_log2;                  // log2(e) / sqrt(128)
    int grid;                          // blocks of the split kernel
    int by_items;                      // 1: a team of warps takes whole items; 0: it takes steps
    int team, teams;                   // warps of a team (1, 2, 4, 8), teams of the grid
    int cluster;                       // by items, team 8: blocks that share an item's steps
    int rt_max;                        // tiles per (sequence, kv-head) at most
    unsigned items, share, extra;      // by items: their number, and per team; `extra` teams take 1 more
    uint32_t polls;                    // of a wait, before it gives up
    int after;                         // 1: launched next to the kernel before it, whose end it awaits
};

// Maps of the rows (see exact_api.cu): own keys and values, prefix keys and values.
struct ExactMaps {
    CUtensorMap k, v, pk, pv;
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

// Items in order: the shared prefix's (kv-head, tile of 8 (sequence, q-head) rows), then every
// sequence's (kv-head, tile of 8 (token, q-head) rows). An item takes S steps of `rs` rows.
// By steps: the flat space of (item, step) is cut into equal ranges, one per team of warps. By items:
// the list of (sequence, kv-head, tile) is, one range per team or cluster of blocks.
struct ExactSpan {
    int S;            // steps per item (0: there are no items)
    int RT;           // tiles per kv-head
};

__device__ __forceinline__ ExactSpan ex_shared_span(const ExactArgs &a, int rs) {
    ExactSpan s;
    const int tpt = ex_tpt(a.G);
    s.S = a.shared_here ? (a.P + rs - 1) / rs : 0;
    s.RT = a.shared_here ? (a.B + tpt - 1) / tpt : 0;
    return s;
}
// Sequence of n rows and ql tokens. An item has a step even where nothing is visible: it writes
// zeros.
__device__ __forceinline__ ExactSpan ex_seq_span(const ExactArgs &a, int n, int ql, int rs, int wr) {
    ExactSpan s;
    const int tpt = ex_tpt(a.G);
    s.RT = (ql + tpt - 1) / tpt;
    s.S = s.RT ? max(1, (ex_most_rows(a.window, a.sinks, tpt, n, wr) + rs - 1) / rs) : 0;
    return s;
}

// By steps: length of the shared part of the space and of the first `seqs` sequences' part, by one
// warp (every lane returns the sum).
__device__ __forceinline__ unsigned ex_length(const ExactArgs &a, int seqs, int rs, int wr) {
    const int lane = threadIdx.x & 31;
    const ExactSpan p = ex_shared_span(a, rs);
    unsigned t = 0;
    if (!a.lens && !a.q_lens) {
        const ExactSpan s = ex_seq_span(a, a.rows, a.m, rs, wr);
        t = (unsigned)seqs * a.H * s.RT * s.S;
    } else {
        for (int b = lane; b < seqs; b += 32) {
            const ExactSpan s = ex_seq_span(a, ex_len(a, b), ex_qlen(a, b), rs, wr);
            t += (unsigned)a.H * s.RT * s.S;
        }
        t = __reduce_add_sync(0xffffffffu, t);
    }
    return t + (unsigned)a.H * p.RT * p.S;
}

constexpr int EX_WARPS = 8;            // warps per block of the split kernel

cudaError_t launch_exact_split(const ExactArgs &a, const ExactMaps &maps, bool f32_rows, bool f32_io,
                               cudaStream_t s);
cudaError_t launch_exact_merge(const ExactArgs &a, bool f32_rows, bool f32_io, cudaStream_t s);

// Clusters of 2, 4 or 8 blocks of the split kernel that the current device runs at once (0: error).
int exact_split_clusters(int cluster);

// Sticky status of the split kernel's bounded waits on the current device: 0 or 1. Clears it.
cudaError_t exact_split_status(int *timed_out, cudaStream_t s);

}  // namespace iskv
