// Eviction from an exact cache by accumulated attention weight.
//
// Per (sequence, kv-head) of n > R rows the kept set is the R rows of the largest (key, lowest
// slot), where key orders the weights as numbers and puts the fixed rows (position < sinks, or
// among the `recent` latest positions) above all. Kept rows of slots >= R move into the freed
// slots below R, both in ascending order: sources and targets are disjoint, so the rows move in
// place without an order between them, and only what has to move is touched.
//
// evict_select_kernel: a block, or a cluster of them, per unit, keys in registers. T, the R-th largest
// key, comes from three digits of 11, 11 and 10 bits: a histogram of the keys that share the digits
// found so far, and the digit where the count from above reaches R. 11 bits are sign, exponent and
// two bits of the fraction, so that weights of a few octaves spread over enough bins for the
// shared-memory atomics. (32 counting passes, one per bit, took twice the time at 32768 rows.) The
// number of kept rows before a slot then gives every freed slot and every moved row its index.
// Blocks behind the units' copy what the slots below R have into the output arrays meanwhile.
//
// evict_move_kernel copies the rows, which is what the operator is bound by (HBM: 4 x 256 bytes per
// moved bf16 row).
//
// Short caches that lose few rows are bound by latency: there one launch does it all, a block per unit,
// the kv-heads of a sequence in one cluster (4160 rows of 8 kv-heads, 64 out: 13.7 -> 12.9 us).
#include "evict.cuh"
#include "exact.cuh"

namespace iskv {
namespace {

constexpr int SEL_T = 1024;
constexpr int SEL_W = SEL_T / 32;
constexpr int BINS = 2048;
constexpr int MOVE_T = 256;
constexpr int MOVE_ROWS = 4;               // 16-byte pieces in flight per thread
constexpr int FUSED_MOVES = 512;           // moves per unit that one block does by itself

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// The value at this block's shared address of `p`, in the cluster's block `rank`.
__device__ __forceinline__ unsigned of_rank(const void *p, int rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    unsigned v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
    return v;
}

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
// FUSED: the block of a unit moves its rows as well; the cluster is a sequence's kv-heads.
template <int E, bool FUSED>
__global__ void __launch_bounds__(SEL_T, 1) evict_select_kernel(EvictArgs a, int cluster) {
    __shared__ unsigned hist[2][BINS];
    __shared__ unsigned sh[SEL_W];
    __shared__ uint4 of_warp[SEL_W];
    __shared__ unsigned found[2];                    // digit, keys above it
    __shared__ unsigned counts[4];                   // of this block: > T, = T, the same below R
    __shared__ int sh_latest;
    constexpr int TURN = SEL_T * E;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = a.B * a.H;
    if (!FUSED) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!FUSED && (int)blockIdx.x >= units * cluster) {
        // what the slots below R have; moved rows replace theirs in the kernel after this one
        const int copies = gridDim.x - units * cluster, at = blockIdx.x - units * cluster;
        for (int unit = at; unit < units; unit += copies) {
            const int b = unit / a.H;
            const int n = min(max(a.lens ? a.lens[b] : a.rows, 0), a.rows), R = min(n, a.budget);
            const long long base = (long long)unit * a.rows;
            for (int i0 = 0; i0 < R; i0 += 8 * SEL_T) {
                float m[8];
                int p[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int i = i0 + x * SEL_T + tid;
                    m[x] = i < R ? a.mass[base + i] : 0.f;
                    p[x] = i < R ? a.pos[base + i] : 0;
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int i = i0 + x * SEL_T + tid;
                    if (i < R) {
                        a.mass_out[base + i] = m[x];
                        a.pos_out[base + i] = p[x];
                    }
                }
            }
        }
        return;
    }
    if (FUSED) cluster = 1;                          // blocks per unit
    const int rank = cluster > 1 ? (int)(blockIdx.x & (unsigned)(cluster - 1)) : 0;
    const int unit = blockIdx.x / cluster, b = unit / a.H, h = unit - b * a.H;
    const int n = min(max(a.lens ? a.lens[b] : a.rows, 0), a.rows);
    const float *mass = a.mass + (long long)unit * a.rows;
    const int *pos = a.pos + (long long)unit * a.rows;
    int *src = a.moves + (long long)unit * 2 * a.max_moves, *dst = src + a.max_moves;
    const int R = min(n, a.budget);
    if (FUSED) {
        // all threads of the sequence's blocks have read its length, which lens_out may replace
        __syncthreads();
        if (a.H > 1) cluster_sync();
        if (tid == 0 && h == 0) a.lens_out[b] = R;
    } else if (tid == 0 && rank == 0) {
        a.keep[unit] = R;
        if (n <= a.budget) a.n_moves[unit] = 0;
    }
    if (n <= a.budget) {                             // all blocks of the cluster
        if (FUSED)
            for (int i = tid; i < n; i += SEL_T) {
                a.mass_out[(long long)unit * a.rows + i] = mass[i];
                a.pos_out[(long long)unit * a.rows + i] = pos[i];
            }
        return;
    }
    // the block's slots: [lo, hi)
    const int span = ((n + cluster - 1) / cluster + 31) & ~31;
    const int lo = min(n, rank * span), hi = min(n, lo + span);
    const bool one = hi - lo <= TURN;

    // the latest position, and with one turn the weights
    float wt[E];
    int ps[E], latest = -0x7fffffff - 1;
    if (one) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = lo + (warp * E + e) * 32 + lane;
            ps[e] = j < hi ? pos[j] : -0x7fffffff - 1;
            wt[e] = j < hi ? mass[j] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) latest = max(latest, ps[e]);
    } else {
#pragma unroll 8
        for (int i = lo + tid; i < hi; i += SEL_T) latest = max(latest, pos[i]);
    }
    for (int i = tid; i < 2 * BINS; i += SEL_T) (&hist[0][0])[i] = 0;
    latest = __reduce_max_sync(0xffffffffu, latest);
    if (lane == 0) sh[warp] = (unsigned)latest;
    __syncthreads();
    latest = __reduce_max_sync(0xffffffffu, (int)sh[lane]);
    if (cluster > 1) {
        if (tid == 0) sh_latest = latest;
        __syncthreads();
        cluster_sync();
        for (int x = 0; x < cluster; ++x) latest = max(latest, (int)of_rank(&sh_latest, x));
    }
    latest = latest < a.recent - 0x7fffffff ? -0x7fffffff - 1 : latest - a.recent;

    uint32_t key[E];
    auto fetch = [&](int turn) {                     // slots past hi: key 0, and j < hi is asked
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = turn + (warp * E + e) * 32 + lane;
            key[e] = j < hi ? evict_key(mass[j], pos[j], a.sinks, latest) : 0u;
        }
    };
    if (one) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = lo + (warp * E + e) * 32 + lane;
            key[e] = j < hi ? evict_key(wt[e], ps[e], a.sinks, latest) : 0u;
        }
    }

    // T by digits; `above` keys exceed the digits found so far
    uint32_t T = 0, mask = 0;
    unsigned above = 0;
#pragma unroll 1
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
        unsigned *h = hist[digit & 1];
        for (int turn = lo; turn < hi; turn += TURN) {
            if (!one) fetch(turn);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j0 = turn + (warp * E + e) * 32;
                if (j0 >= hi) break;
                const bool in = j0 + lane < hi && (key[e] & mask) == T;
                if (!__any_sync(0xffffffffu, in)) continue;      // most, from the second digit on
                const unsigned d = (key[e] >> shift) & ((1u << bits) - 1u);
                // one digit in the whole warp (many equal weights): one atomic
                const unsigned d0 = __shfl_sync(0xffffffffu, d, 0);
                if (__all_sync(0xffffffffu, in && d == d0)) {
                    if (lane == 0) atomicAdd(&h[d], 32u);
                } else if (in) {
                    atomicAdd(&h[d], 1u);
                }
            }
        }
        __syncthreads();
        if (cluster > 1) cluster_sync();
        // bins from the top: thread i has bins 2047 - 2 i and 2046 - 2 i
        const int b0 = BINS - 1 - 2 * tid;
        unsigned h0 = 0, h1 = 0;
        if (cluster > 1) {
            for (int x = 0; x < cluster; ++x) {
                h0 += of_rank(&h[b0], x);
                h1 += of_rank(&h[b0 - 1], x);
            }
        } else {
            h0 = h[b0];
            h1 = h[b0 - 1];
        }
        unsigned sum = h0 + h1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) sh[warp] = sum;
        __syncthreads();
        const unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? sh[lane] : 0u);
        const unsigned upto = above + before + sum, from = upto - h0 - h1;
        if (from < (unsigned)R && upto >= (unsigned)R) {
            const bool first = from + h0 >= (unsigned)R;
            found[0] = (unsigned)(first ? b0 : b0 - 1);
            found[1] = first ? from : from + h0;
        }
        // this buffer is used again by the third digit, which all blocks begin after the second's
        // cluster barrier: no block then reads the first's counts
        __syncthreads();
        T |= found[0] << shift;
        above = found[1];
        mask |= ((1u << bits) - 1u) << shift;
        if (digit == 1) {
            for (int i = tid; i < BINS; i += SEL_T) hist[0][i] = 0;
            __syncthreads();
        }
    }
    const int ties = R - (int)above;                 // keys equal to T that stay: the lowest slots

    // keys > T, = T, the same below R: of each warp, of the block, of the blocks before it and of all
    unsigned c[4] = {0, 0, 0, 0};
    for (int turn = lo; turn < hi; turn += TURN) {
        if (!one) fetch(turn);
        unsigned all = 0, under = 0;                 // two counts each, of at most 32 E
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = turn + (warp * E + e) * 32 + lane;
            const unsigned x = j >= hi ? 0u : key[e] > T ? 1u : key[e] == T ? 1u << 16 : 0u;
            all += x;
            under += j < R ? x : 0u;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        under = __reduce_add_sync(0xffffffffu, under);
        c[0] += all & 0xffffu;
        c[1] += all >> 16;
        c[2] += under & 0xffffu;
        c[3] += under >> 16;
    }
    if (lane == 0) of_warp[warp] = make_uint4(c[0], c[1], c[2], c[3]);
    __syncthreads();
    const uint4 cw = of_warp[lane];
    int gt_before = 0, eq_before = 0;
    int low_gt = (int)__reduce_add_sync(0xffffffffu, cw.z);
    int low_eq = (int)__reduce_add_sync(0xffffffffu, cw.w);
    if (cluster > 1) {
        const unsigned gt_here = __reduce_add_sync(0xffffffffu, cw.x);
        const unsigned eq_here = __reduce_add_sync(0xffffffffu, cw.y);
        if (tid == 0) {
            counts[0] = gt_here;
            counts[1] = eq_here;
            counts[2] = (unsigned)low_gt;
            counts[3] = (unsigned)low_eq;
        }
        __syncwarp();
        cluster_sync();
        low_gt = low_eq = 0;
        for (int x = 0; x < cluster; ++x) {
            if (x < rank) {
                gt_before += (int)of_rank(&counts[0], x);
                eq_before += (int)of_rank(&counts[1], x);
            }
            low_gt += (int)of_rank(&counts[2], x);
            low_eq += (int)of_rank(&counts[3], x);
        }
        // no block ends while others read its counts: the wait is at the end
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const int low = low_gt + min(low_eq, ties);      // kept rows of slots < R
    const unsigned below = (1u << lane) - 1u;
    for (int turn = lo; turn < hi; turn += TURN) {
        if (!one) fetch(turn);
        uint4 x = cw;                                // the warps' counts of this turn
        if (!one) {
            unsigned all = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = turn + (warp * E + e) * 32 + lane;
                all += j >= hi ? 0u : key[e] > T ? 1u : key[e] == T ? 1u << 16 : 0u;
            }
            all = __reduce_add_sync(0xffffffffu, all);
            __syncthreads();
            if (lane == 0) sh[warp] = all;
            __syncthreads();
            x.x = sh[lane] & 0xffffu;
            x.y = sh[lane] >> 16;
        }
        int g0 = gt_before + (int)__reduce_add_sync(0xffffffffu, lane < warp ? x.x : 0u);
        int e0 = eq_before + (int)__reduce_add_sync(0xffffffffu, lane < warp ? x.y : 0u);
        if (!one) {
            gt_before += (int)__reduce_add_sync(0xffffffffu, x.x);
            eq_before += (int)__reduce_add_sync(0xffffffffu, x.y);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j0 = turn + (warp * E + e) * 32, j = j0 + lane;
            if (j0 >= hi) break;
            const bool is_gt = j < hi && key[e] > T, is_eq = j < hi && key[e] == T;
            const unsigned mg = __ballot_sync(0xffffffffu, is_gt);
            const unsigned me = __ballot_sync(0xffffffffu, is_eq);
            const int eq_at = e0 + __popc(me & below);
            const int kept_at = g0 + __popc(mg & below) + min(eq_at, ties);   // before slot j
            const bool kept = is_gt || (is_eq && eq_at < ties);
            if (j < min(R, hi) && !kept) dst[j - kept_at] = j;
            if (j >= R && kept) src[kept_at - low] = j;
            if (FUSED && j < R && kept) {            // (one turn: they are at hand)
                a.mass_out[(long long)unit * a.rows + j] = wt[e];
                a.pos_out[(long long)unit * a.rows + j] = ps[e];
            }
            g0 += __popc(mg);
            e0 += __popc(me);
        }
    }
    if (!FUSED) {
        if (tid == 0 && rank == 0) a.n_moves[unit] = R - low;
        if (cluster > 1) {
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
        return;
    }
    __syncthreads();                                 // the lists are complete
    const int moves = R - low, vecs = a.esz == 2 ? 16 : 32, per_row = 2 * vecs;
    char *kb = a.k + b * a.seq_st + h * a.head_st, *vb = a.v + b * a.seq_st + h * a.head_st;
    const long long at = (long long)unit * a.rows;
    for (int e0 = tid; e0 < moves * per_row; e0 += MOVE_ROWS * SEL_T) {
        uint4 x[MOVE_ROWS];
        char *to[MOVE_ROWS];
#pragma unroll
        for (int i = 0; i < MOVE_ROWS; ++i) {
            const int e = e0 + i * SEL_T;
            to[i] = nullptr;
            if (e < moves * per_row) {
                const int r = e / per_row, w = e - r * per_row;
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
    for (int i = tid; i < moves; i += SEL_T) {
        const int s = src[i], d = dst[i];
        a.mass_out[at + d] = mass[s];
        a.pos_out[at + d] = pos[s];
    }
}

// Block (x, unit): the unit's moves, 16 bytes of a key or value row per thread, MOVE_ROWS in flight.
// Both ends of a move are used once, so they pass through L2 first out (8 x 32768 rows: 77.6 -> 72.8 us;
// loads alone 79.0, stores alone 78.1).
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
            const int e = base + i * stride;
            to[i] = nullptr;
            if (e < total) {
                const int r = e / per_row, w = e - r * per_row;
                char *rows = w < vecs ? kb : vb;
                const int off = (w < vecs ? w : w - vecs) * 16;
                x[i] = __ldcs(reinterpret_cast<const uint4 *>(rows + src[r] * a.row_st + off));
                to[i] = rows + dst[r] * a.row_st + off;
            }
        }
#pragma unroll
        for (int i = 0; i < MOVE_ROWS; ++i)
            if (to[i]) __stcs(reinterpret_cast<uint4 *>(to[i]), x[i]);
    }
    const long long at = (long long)unit * a.rows;
    for (int i = blockIdx.x * MOVE_T + threadIdx.x; i < n; i += stride) {
        const int s = src[i], d = dst[i];
        const float m = a.mass[at + s];
        const int p = a.pos[at + s];
        a.mass_out[at + d] = m;
        a.pos_out[at + d] = p;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t s) {
    const int units = a.B * a.H;
    if (a.rows <= 8 * SEL_T && a.H <= 8 && a.max_moves <= FUSED_MOVES) {
        cudaLaunchConfig_t one = {};
        one.gridDim = dim3(units);
        one.blockDim = dim3(SEL_T);
        one.stream = s;
        cudaLaunchAttribute cl;
        cl.id = cudaLaunchAttributeClusterDimension;
        cl.val.clusterDim.x = a.H;
        cl.val.clusterDim.y = cl.val.clusterDim.z = 1;
        one.attrs = &cl;
        one.numAttrs = a.H > 1 ? 1 : 0;
        return cudaLaunchKernelEx(&one, evict_select_kernel<8, true>, a, a.H);
    }
    // long rows and few units: up to four blocks share a unit. Clusters fill a whole number of
    // blocks, so the copying blocks come in clusters as well.
    int cluster = 1;
    while (cluster < 4 && a.rows > 8 * SEL_T * cluster && units * 2 * cluster <= sms) cluster *= 2;
    int copies = 0;
    if (a.mass_out != a.mass || a.pos_out != a.pos) {
        copies = sms - units * cluster;
        if (copies < 16) copies = 16;
        if (copies > units) copies = units;
        copies = (copies + cluster - 1) / cluster * cluster;
    }
    cudaLaunchConfig_t sel = {};
    sel.gridDim = dim3(units * cluster + copies);
    sel.blockDim = dim3(SEL_T);
    sel.stream = s;
    cudaLaunchAttribute cl;
    cl.id = cudaLaunchAttributeClusterDimension;
    cl.val.clusterDim.x = cluster;
    cl.val.clusterDim.y = cl.val.clusterDim.z = 1;
    sel.attrs = &cl;
    sel.numAttrs = cluster > 1 ? 1 : 0;
    const cudaError_t e = a.rows <= 8 * SEL_T * cluster
                              ? cudaLaunchKernelEx(&sel, evict_select_kernel<8, false>, a, cluster)
                              : cudaLaunchKernelEx(&sel, evict_select_kernel<16, false>, a, cluster);
    if (e != cudaSuccess) return e;
    const int vecs = a.esz == 2 ? 16 : 32;
    const long long want = ((long long)a.max_moves * 2 * vecs + MOVE_T * MOVE_ROWS - 1) /
                           (MOVE_T * MOVE_ROWS);
    // two rounds of blocks (8 x 32768 rows, a tenth moved: 69.0 us; one round 72.9, four 70.0)
    long long x = (16LL * sms + units - 1) / units;
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
