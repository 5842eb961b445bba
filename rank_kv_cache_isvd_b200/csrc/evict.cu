// Eviction from an exact cache by accumulated attention weight.
//
// Per (sequence, kv-head) of n > R rows the kept set is the R rows of the largest (key, lowest
// slot), where key orders the weights as numbers and puts the fixed rows (position < sinks, or
// among the `recent` latest positions) above all. Kept rows of slots >= R move into the freed
// slots below R, both in ascending order: sources and targets are disjoint, so the rows move in
// place without an order between them, and only what has to move is touched.
//
// evict_select_kernel: one block per unit. The R-th largest key is found bit by bit: the largest T
// with #{key >= T} >= R, one count over the unit's keys per bit. A block scan then gives every
// freed slot and every moved row its index. evict_move_kernel copies the rows, which is what the
// operator is bound by (HBM: 4 x 256 bytes per moved bf16 row).
#include "exact.cuh"
#include "evict.cuh"

namespace iskv {
namespace {

constexpr int SEL_T = 1024;
constexpr int SEL_W = SEL_T / 32;
constexpr int MOVE_T = 256;
constexpr int MOVE_ROWS = 4;               // rows in flight per warp

// Order-preserving key of a weight (-0 equals 0; a NaN, of either sign, is above all weights);
// fixed rows get the largest.
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int sinks, int latest) {
    if (pos < sinks || pos > latest) return 0xffffffffu;
    if (isnan(w)) return 0xfffffffeu;
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of x over the block's threads before this one's warp (exclusive), and over all.
__device__ __forceinline__ int warp_offsets(int x, int *sh, int &all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sh[warp] = x;
    __syncthreads();
    const int v = sh[lane];
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    all = __shfl_sync(0xffffffffu, sum, 31);
    return __shfl_sync(0xffffffffu, sum - v, warp);
}

template <bool IN_SMEM>
__global__ void __launch_bounds__(SEL_T, 1) evict_select_kernel(EvictArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ int sh[32];
    __shared__ int cnt[2];
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
    if (tid == 0) {
        a.keep[unit] = R;
        if (n <= a.budget) a.n_moves[unit] = 0;
    }
    if (n <= a.budget) {
        if (mass_out != mass)
            for (int i = tid; i < n; i += SEL_T) mass_out[i] = mass[i];
        if (pos_out != pos)
            for (int i = tid; i < n; i += SEL_T) pos_out[i] = pos[i];
        return;
    }
    // the latest position, then the keys
    int latest = -0x7fffffff - 1;
    for (int i = tid; i < n; i += SEL_T) latest = max(latest, pos[i]);
    latest = __reduce_max_sync(0xffffffffu, latest);
    if (lane == 0) sh[warp] = latest;
    if (tid < 2) cnt[tid] = 0;
    __syncthreads();
    latest = __reduce_max_sync(0xffffffffu, sh[lane]);
    latest = latest < a.recent - 0x7fffffff ? -0x7fffffff - 1 : latest - a.recent;
    auto key = [&](int i) {
        return IN_SMEM ? keys[i] : evict_key(mass[i], pos[i], a.sinks, latest);
    };
    if (IN_SMEM) {
        for (int i = tid; i < n; i += SEL_T) keys[i] = evict_key(mass[i], pos[i], a.sinks, latest);
        // each thread counts the keys it wrote: no barrier needed before the counts
    }
    // T: bit by bit from the top, kept where at least R keys reach it
    uint32_t T = 0;
    int above = 0;                                   // #{key >= T + 2^bit ...} of the last refusal
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = T | (1u << bit);
        int x = 0;
        for (int i = tid; i < n; i += SEL_T) x += key(i) >= c;
        x = __reduce_add_sync(0xffffffffu, x);
        if (lane == 0) atomicAdd(&cnt[bit & 1], x);
        __syncthreads();
        const int all = cnt[bit & 1];
        if (tid == 0) cnt[(bit & 1) ^ 1] = 0;
        __syncthreads();
        if (all >= R) T = c;
        else above = all;
    }
    // above = #{key > T} once every higher candidate has been refused: the last refusal was the
    // candidate just above T (or none, and then no key exceeds T)
    const int ties = R - above;                      // keys equal to T that stay: the lowest slots
    // warps own runs of slots in order
    const int run = ((n + SEL_W - 1) / SEL_W + 31) / 32 * 32;
    const int lo = warp * run, hi = min(n, lo + run);
    if (IN_SMEM) __syncthreads();
    int eq = 0;
    for (int i = lo; i < hi; i += 32) {
        const int j = i + lane;
        eq += __popc(__ballot_sync(0xffffffffu, j < hi && key(j) == T));
    }
    int all;
    int eq0 = warp_offsets(eq, sh, all);
    const unsigned below = (1u << lane) - 1u;
    int freed = 0, moved = 0;
    for (int i = lo, e = eq0; i < hi; i += 32) {
        const int j = i + lane;
        const uint32_t k = j < hi ? key(j) : 0u;
        const unsigned te = __ballot_sync(0xffffffffu, j < hi && k == T);
        const bool kept = j < hi && (k > T || (k == T && e + __popc(te & below) < ties));
        e += __popc(te);
        freed += __popc(__ballot_sync(0xffffffffu, j < hi && !kept && j < R));
        moved += __popc(__ballot_sync(0xffffffffu, kept && j >= R));
    }
    int all_freed, all_moved;
    int f0 = warp_offsets(freed, sh, all_freed);
    int m0 = warp_offsets(moved, sh, all_moved);
    for (int i = lo, e = eq0; i < hi; i += 32) {
        const int j = i + lane;
        const uint32_t k = j < hi ? key(j) : 0u;
        const unsigned te = __ballot_sync(0xffffffffu, j < hi && k == T);
        const bool kept = j < hi && (k > T || (k == T && e + __popc(te & below) < ties));
        e += __popc(te);
        const unsigned fr = __ballot_sync(0xffffffffu, j < hi && !kept && j < R);
        const unsigned mv = __ballot_sync(0xffffffffu, kept && j >= R);
        if (fr >> lane & 1) dst[f0 + __popc(fr & below)] = j;
        if (mv >> lane & 1) src[m0 + __popc(mv & below)] = j;
        if (kept && j < R) {
            if (mass_out != mass) mass_out[j] = mass[j];
            if (pos_out != pos) pos_out[j] = pos[j];
        }
        f0 += __popc(fr);
        m0 += __popc(mv);
    }
    __syncthreads();                                 // the lists are complete
    if (tid == 0) a.n_moves[unit] = all_moved;
    for (int i = tid; i < all_moved; i += SEL_T) {
        const int s = src[i], d = dst[i];
        mass_out[d] = mass[s];
        pos_out[d] = pos[s];
    }
}

// Block (x, unit): moves of the unit from x * rows per block on; a warp has MOVE_ROWS rows of one
// of K and V in flight per step.
__global__ void __launch_bounds__(MOVE_T) evict_move_kernel(EvictArgs a, int vecs) {
    const int unit = blockIdx.y, b = unit / a.H, h = unit - b * a.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.lens_out[b] = a.keep[unit];
    const int n = a.n_moves[unit];
    const int *src = a.moves + (long long)unit * 2 * a.max_moves, *dst = src + a.max_moves;
    // a row has `vecs` 16-byte pieces (16 or 32); keys and values are its two halves
    const int per_row = 2 * vecs, total = n * per_row;
    char *kb = a.k + b * a.seq_st + h * a.head_st, *vb = a.v + b * a.seq_st + h * a.head_st;
    const int stride = gridDim.x * MOVE_T;
    for (int base = blockIdx.x * MOVE_T + threadIdx.x; base < total; base += stride * MOVE_ROWS) {
        uint4 x[MOVE_ROWS];
        char *to[MOVE_ROWS];
#pragma unroll
        for (int i = 0; i < MOVE_ROWS; ++i) {
            const long long e = (long long)base + (long long)i * stride;
            to[i] = nullptr;
            if (e < total) {
                const int r = (int)(e / per_row), w = (int)(e - (long long)r * per_row);
                char *rows = w < vecs ? kb : vb;
                const int off = (w < vecs ? w : w - vecs) * 16;
                x[i] = *reinterpret_cast<const uint4 *>(rows + src[r] * a.row_st + off);
                to[i] = rows + dst[r] * a.row_st + off;
            }
        }
#pragma unroll
        for (int i = 0; i < MOVE_ROWS; ++i)
            if (to[i]) *reinterpret_cast<uint4 *>(to[i]) = x[i];
    }
}

constexpr int SEL_SMEM_KEYS = 50 * 1024;             // 200 KB of keys

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t s) {
    const int units = a.B * a.H;
    cudaError_t e;
    if (a.rows <= SEL_SMEM_KEYS) {
        const int bytes = a.rows * 4;
        e = cudaFuncSetAttribute(evict_select_kernel<true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        evict_select_kernel<true><<<units, SEL_T, bytes, s>>>(a);
    } else {
        evict_select_kernel<false><<<units, SEL_T, 0, s>>>(a);
    }
    e = cudaGetLastError();
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
