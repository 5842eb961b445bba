// Arguments of the eviction kernels.
#pragma once

#include <cuda_runtime.h>

namespace iskv {

struct EvictArgs {
    char *k, *v;                       // rows, moved in place
    long long seq_st, head_st, row_st; // bytes
    int B, H, rows, esz;
    const int *lens;                   // NULL: every sequence holds `rows` rows
    int *lens_out;
    const float *mass;                 // [B][H][rows]
    float *mass_out;
    const int *pos;
    int *pos_out;
    int budget, recent, sinks;
    int *moves;                        // [B*H][2][max_moves]: sources, targets
    int *n_moves, *keep;               // [B*H]
    int max_moves;
};

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t s);

}  // namespace iskv
