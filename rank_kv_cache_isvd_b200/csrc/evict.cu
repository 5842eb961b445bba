// Eviction from an exact cache by accumulated attention weight.
//
// Per (sequence, kv-head) of n > R rows the kept set is the R rows of the largest (key, lowest
// slot), where key orders the weights as numbers and puts the fixed rows (position < sinks, or
// among the `recent` latest positions) above all. Kept rows of slots >= R move into the freed
// slots below R, both in ascending order: sources and targets are disjoint, so the rows move in
// place without an order between them, and only what has to move is touched.
//
// evict_select_kernel: one block per unit, keys in registers up to 32768 rows. T, the R-th largest
// key, comes from three digits of 11, 11 and 10 bits: a histogram of the keys that share the digits
// found so far, and the digit where the count from above reaches R. 11 bits are sign, exponent and
// two bits of the fraction, so that weights of a few octaves spread over enough bins for the
// shared-memory atomics (they took 32 counting passes' place, 20 us of 85 us at 32768 rows). The
// number of kept rows before a slot then gives every freed slot and every moved row its index.
//
// evict_move_kernel copies the rows, which is what the operator is bound by (HBM: 4 x 256 bytes per
// moved bf16 row).
#include "evict.cuh"
#include "exact.cuh"

namespace iskv {
namespace {

constexpr int SEL_T = 1024;
constexpr int SEL_W = SEL_T / 32;
constexpr int BINS = 2048;
constexpr int MOVE_T = 256;
constexpr int MOVE_ROWS = 4;               // 16-byte pieces in flight per thread

// Order-preserving key of a weight (-0 equals 0; a NaN, of either sign, is above all weights);
// fixed rows get the largest.
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int sinks, int latest) {
    if (pos < sinks || pos > latest) return 0xffffffffu;
    if (isnan(w)) return 0xfffffffeu;
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// E keys per thread and turn: a turn is SEL_T * E slots, of which each warp has a run, in order:
// slot = turn + warp 32 E + 32 e + lane. With one turn the keys stay in registers.
template <int E>
__global__ void __launch_bounds__(SEL_T, 1) evict_select_kernel(EvictArgs a) {
    __shared__ unsigned hist[BINS];
    __shared__ int sh[SEL_W], sh2[SEL_W];
    __shared__ unsigned found[2];                    // digit, keys above it
    __shared__ int kept_low;                         // kept rows of slots < R
    constexpr int TURN = SEL_T * E;
    const int unit = blockIdx.x, b = unit / a.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = min(max(a.lens ? a.lens[b] : a.rows, 0), a.rows);
    const float *mass = a.mass + (long long)unit * a.rows;
    const int *pos = a.pos + (long long)unit * a.rows;
    float *mass_out = a.mass_out + (long long)unit * a.rows;
    int *pos_out = a.pos_out + (long long)unit * a.rows;
    int *src = a.moves + (long long)unit * 2 * a.max_moves, *dst = src + a.max_moves;
    const int R = min(n, a.budget);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // what the slots below R have; moved rows replace theirs in the kernel after this one
    if (mass_out != mass) {
#pragma unroll 8
        for (int i = tid; i < R; i += SEL_T) mass_out[i] = mass[i];
    }
    if (pos_out != pos) {
#pragma unroll 8
        for (int i = tid; i < R; i += SEL_T) pos_out[i] = pos[i];
    }
    if (tid == 0) {
        a.keep[unit] = R;
        if (n <= a.budget) a.n_moves[unit] = 0;
    }
    if (n <= a.budget) return;

    int latest = -0x7fffffff - 1;
#pragma unroll 8
    for (int i = tid; i < n; i += SEL_T) latest = max(latest, pos[i]);
    latest = __reduce_max_sync(0xffffffffu, latest);
    if (lane == 0) sh[warp] = latest;
    __syncthreads();
    latest = __reduce_max_sync(0xffffffffu, sh[lane]);
    latest = latest < a.recent - 0x7fffffff ? -0x7fffffff - 1 : latest - a.recent;

    uint32_t key[E];
    auto fetch = [&](int turn) {                     // slots past n: key 0, and j < n is asked
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = turn + (warp * E + e) * 32 + lane;
            key[e] = j < n ? evict_key(mass[j], pos[j], a.sinks, latest) : 0u;
        }
    };
    const bool one = n <= TURN;
    if (one) fetch(0);

    // T by digits; `above` keys exceed the digits found so far
    uint32_t T = 0, mask = 0;
    int above = 0;
#pragma unroll 1
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
        for (int i = tid; i < BINS; i += SEL_T) hist[i] = 0;
        __syncthreads();
        for (int turn = 0; turn < n; turn += TURN) {
            if (!one) fetch(turn);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = turn + (warp * E + e) * 32 + lane;
                if (turn + (warp * E + e) * 32 >= n) break;
                const bool in = j < n && (key[e] & mask) == T;
                const unsigned d = (key[e] >> shift) & ((1u << bits) - 1u);
                // equal digits in a whole warp (many equal weights): one atomic
                int same;
                __match_all_sync(0xffffffffu, in ? d : 0xffffffffu, &same);
                if (same) {
                    if (in && lane == 0) atomicAdd(&hist[d], 32u);
                } else if (in) {
                    atomicAdd(&hist[d], 1u);
                }
            }
        }
        __syncthreads();
        // bins from the top: thread i has bins 2047 - 2 i and 2046 - 2 i
        const int b0 = BINS - 1 - 2 * tid;
        const unsigned h0 = hist[b0], h1 = hist[b0 - 1];
        unsigned sum = h0 + h1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) sh[warp] = (int)sum;
        __syncthreads();
        unsigned before = lane < warp ? (unsigned)sh[lane] : 0u;
        before = __reduce_add_sync(0xffffffffu, before);
        const unsigned upto = above + before + sum, from = upto - h0 - h1;
        if (from < (unsigned)R && upto >= (unsigned)R) {
            const bool first = from + h0 >= (unsigned)R;
            found[0] = (unsigned)(first ? b0 : b0 - 1);
            found[1] = first ? from : from + h0;
        }
        __syncthreads();
        T |= found[0] << shift;
        above = (int)found[1];
        mask |= ((1u << bits) - 1u) << shift;
    }
    const int ties = R - above;                      // keys equal to T that stay: the lowest slots

    // kept rows before each warp's runs, turn by turn
    const unsigned below = (1u << lane) - 1u;
    int gt_before = 0, eq_before = 0;                // of the turns before
    if (tid == 0) kept_low = 0;
    for (int pass = 0; pass < 2; ++pass) {           // 0: kept_low; 1: the lists
        gt_before = eq_before = 0;
        for (int turn = 0; turn < n; turn += TURN) {
            if (!one) fetch(turn);
            int gt = 0, eq = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = turn + (warp * E + e) * 32 + lane;
                gt += j < n && key[e] > T;
                eq += j < n && key[e] == T;
            }
            gt = __reduce_add_sync(0xffffffffu, gt);
            eq = __reduce_add_sync(0xffffffffu, eq);
            __syncthreads();
            if (lane == 0) {
                sh[warp] = gt;
                sh2[warp] = eq;
            }
            __syncthreads();
            int g0 = gt_before + __reduce_add_sync(0xffffffffu, lane < warp ? sh[lane] : 0);
            int e0 = eq_before + __reduce_add_sync(0xffffffffu, lane < warp ? sh2[lane] : 0);
            gt_before += __reduce_add_sync(0xffffffffu, sh[lane]);
            eq_before += __reduce_add_sync(0xffffffffu, sh2[lane]);
            const int run = turn + warp * E * 32;    // the warp's first slot
            if (pass == 0) {
                // the warp with slot R counts the kept rows before it
                if (run <= R && R < run + E * 32) {
                    int low_gt = 0, low_eq = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int j = run + e * 32 + lane;
                        low_gt += j < R && key[e] > T;
                        low_eq += j < R && key[e] == T;
                    }
                    low_gt = g0 + __reduce_add_sync(0xffffffffu, low_gt);
                    low_eq = e0 + __reduce_add_sync(0xffffffffu, low_eq);
                    if (lane == 0) kept_low = low_gt + min(low_eq, ties);
                }
                continue;
            }
            const int low = kept_low;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = run + e * 32 + lane;
                if (run + e * 32 >= n) break;
                const bool is_gt = j < n && key[e] > T, is_eq = j < n && key[e] == T;
                const unsigned mg = __ballot_sync(0xffffffffu, is_gt);
                const unsigned me = __ballot_sync(0xffffffffu, is_eq);
                const int eq_at = e0 + __popc(me & below);
                const int kept_at = g0 + __popc(mg & below) + min(eq_at, ties);   // before slot j
                const bool kept = is_gt || (is_eq && eq_at < ties);
                if (j < R && !kept) dst[j - kept_at] = j;
                if (j >= R && kept) src[kept_at - low] = j;
                g0 += __popc(mg);
                e0 += __popc(me);
            }
        }
        __syncthreads();
    }
    if (tid == 0) a.n_moves[unit] = R - kept_low;
}

// Block (x, unit): the unit's moves, 16 bytes of a key or value row per thread, MOVE_ROWS in flight.
__global__ void __launch_bounds__(MOVE_T) evict_move_kernel(EvictArgs a, int vecs) {
    const int unit = blockIdx.y, b = unit / a.H, h = unit - b * a.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.lens_out[b] = a.keep[unit];
    const int n = a.n_moves[unit];
    const int *src = a.moves + (long long)unit * 2 * a.max_moves, *dst = src + a.max_moves;
    const long long at = (long long)unit * a.rows;
    // a row has `vecs` 16-byte pieces (16 or 32); keys and values are its two halves
    const int per_row = 2 * vecs, total = n * per_row;
    char *kb = a.k + b * a.seq_st + h * a.head_st, *vb = a.v + b * a.seq_st + h * a.head_st;
    const int stride = gridDim.x * MOVE_T;
    for (int base = blockIdx.x * MOVE_T + threadIdx.x; base < total; base += stride * MOVE_ROWS) {
        uint4 x[MOVE_ROWS];
        char *to[MOVE_ROWS];
#pragma unroll
        for (int i = 0; i < MOVE_ROWS; ++i) {
            const int e = base + i * stride;
            to[i] = nullptr;
            if (e < total) {
                const int r = e / per_row, w = e - r * per_row;
                char *rows = w < vecs ? kb : vb;
                const int off = (w < vecs ? w : w - vecs) * 16;
                const int s = src[r], d = dst[r];
                x[i] = *reinterpret_cast<const uint4 *>(rows + s * a.row_st + off);
                to[i] = rows + d * a.row_st + off;
                if (w == 0) a.mass_out[at + d] = a.mass[at + s];
                if (w == vecs) a.pos_out[at + d] = a.pos[at + s];
            }
        }
#pragma unroll
        for (int i = 0; i < MOVE_ROWS; ++i)
            if (to[i]) *reinterpret_cast<uint4 *>(to[i]) = x[i];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t s) {
    const int units = a.B * a.H;
    if (a.rows <= 8 * SEL_T) evict_select_kernel<8><<<units, SEL_T, 0, s>>>(a);
    else evict_select_kernel<32><<<units, SEL_T, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int vecs = a.esz == 2 ? 16 : 32;
    const long long want = ((long long)a.max_moves * 2 * vecs + MOVE_T * MOVE_ROWS - 1) /
                           (MOVE_T * MOVE_ROWS);
    long long x = (8LL * sms + units - 1) / units;
    if (x > want) x = want;
    if (x < 1) x = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x, (unsigned)units);
    cfg.blockDim = dim3(MOVE_T);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, a, vecs);
}

}  // namespace iskv
