// Arguments of the tile kernel (exact_tile.cu): attention of many query rows over exact rows on the
// tensor cores.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace iskv {

constexpr int TILE_ROWS = 128;         // query rows per tile, and key rows per block

struct TileArgs {
    int B, H, G;
    int rows;                          // capacity of a sequence (prefix: its rows)
    const int *lens, *q_lens;
    int m;                             // tokens per sequence (prefix: sequences)
    int window, sinks;
    int seq_mul, head_mul;             // 0 where all sequences, or kv-heads, share one stream
    int tq;                            // tokens per tile: 128 / G
    int pairs;                         // pairs of tiles per (sequence, kv-head)
    int nsp;                           // splits of the rows' blocks
    char *out;                         // whole results (nsp 1) ...
    long long o_seq, o_head, o_tok;    // bytes
    float *pre_ml, *pre_o;             // ... or records [B H][nsp][m G][2] and [..][128]
                                       // (prefix: [H][nsp][sequences G])
    float scale_log2;
};

// Maps of q (channels, q-heads, tokens, sequences) in boxes of 64 channels, and of the rows (64
// channels, rows, halves, kv-heads, sequences) in boxes of 128 whole rows.
cudaError_t launch_exact_tile(const TileArgs &a, const CUtensorMap &q, const CUtensorMap &k,
                              const CUtensorMap &v, bool prefix, bool alternate, cudaStream_t s);

// Joins the records of launch_exact_tile (not prefix) with nsp > 1.
cudaError_t launch_exact_tile_merge(const TileArgs &a, cudaStream_t s);

// Sticky status of the tile kernel's bounded waits on the current device: 0 or 1. Clears it.
cudaError_t exact_tile_status(int *timed_out, cudaStream_t s);

}  // namespace iskv
