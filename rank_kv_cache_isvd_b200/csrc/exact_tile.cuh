// Arguments of the kernels for many query rows: the tile kernel (exact_tile.cu: bf16, tcgen05) and
// the rows kernel (exact_rows.cu: float32 operands).
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
    int tq;                            // tokens per tile (rows kernel: per group of 8 tiles)
    int pairs;                         // pairs of tiles (groups) per (sequence, kv-head)
    int nsp;                           // splits of the rows' blocks
    const char *q;                     // rows kernel
    long long q_seq, q_head, q_tok;    // bytes
    char *out;                         // whole results (nsp 1) ...
    long long o_seq, o_head, o_tok;    // bytes
    float *pre_ml, *pre_o;             // ... or records [B H][nsp][m G][2] and [..][128]
                                       // (prefix: [H][nsp][sequences G])
    float scale_log2;
    unsigned polls;                    // of a wait, before it gives up
};

// Maps of q (channels, q-heads, tokens, sequences) in boxes of 64 channels; of the rows (64 channels,
// rows, halves, kv-heads, sequences) in boxes of 128 whole rows, and (channels, rows, kv-heads,
// sequences) in boxes of 64 channels of 16 rows (not prefix).
struct TileMaps {
    CUtensorMap q, k, v, k16, v16;
};
cudaError_t launch_exact_tile(const TileArgs &a, const TileMaps &maps, bool prefix, bool alternate,
                              cudaStream_t s);

// Maps of the rows in boxes of ex_warp_rows() whole rows.
cudaError_t launch_exact_rows(const TileArgs &a, const CUtensorMap &k, const CUtensorMap &v,
                              bool f32_rows, bool f32_io, bool prefix, cudaStream_t s);

// Joins the records of either (not prefix) with nsp > 1.
cudaError_t launch_exact_tile_merge(const TileArgs &a, bool f32_io, cudaStream_t s);

// Sticky status of the kernels' bounded waits on the current device: 0 or 1. Clears it.
cudaError_t exact_tile_status(int *timed_out, cudaStream_t s);
cudaError_t exact_rows_status(int *timed_out, cudaStream_t s);

}  // namespace iskv
