// Attention of many query rows over exact rows where operands are float32 (or queries cannot be
// mapped for the tile kernel): prompts, chunks of them, and a prefix that a batch shares.
//
// Float32 results need products of 22 to 24 bits, which the tensor cores give as sums of bf16 or
// tf32 products (exact_warp.cuh): 64 mma.sync per 32 keys and 8 rows, the bound of this kernel at
// 145 TFLOP/s of float32 work. A CTA takes 64 query rows, 8 per warp, and all warps share one ring
// of key and value units in shared memory. (The split kernel, which gives each tile of 8 rows its own
// copy of the rows, was bound by L2 here: 950 us against 435 us at 94 x 4 queries of 8 kv-heads over
// 7264 shared float32 rows.) They reach 73 TFLOP/s over bf16 rows (130 x 8 queries over 16384 shared
// rows: 964 us) and 27 over float32 rows (a causal prompt of 4096: 5070 us, over bf16 rows 1785); fetching
// and decoding instructions, then the splitting, take the rest. As in the tile kernel a CTA does a split
// of the rows' steps where CTAs are few.
#include <atomic>

#include "exact_tile.cuh"
#include "exact_warp.cuh"

namespace iskv {
namespace {

constexpr int W = EX_WARPS;
constexpr int RING = 24;               // units
constexpr int LAG = 6;                 // a unit is refilled this many units after warp 0 read it
constexpr size_t ROWS_SMEM = RING * (UNIT + 16) + 1024;

__device__ int g_rows_status;

template <bool F32ROWS, bool F32IO, bool PREFIX>
__global__ void __launch_bounds__(32 * W, 1)
exact_rows_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    using Rows = WarpRows<F32ROWS, F32IO>;
    constexpr int WR = Rows::WR, NT = Rows::NT;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + RING * UNIT);
    const uint32_t ring = smem_u32(smem), full = smem_u32(bars), empty = full + RING * 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // groups in descending order, units within: the longest start first
    const int units = PREFIX ? a.H : a.B * a.H;
    int id = blockIdx.x;
    const int unit = id % units;
    id /= units;
    const int sp = id % a.nsp, group = a.pairs - 1 - id / a.nsp;
    const int b = PREFIX ? 0 : unit / a.H, h = PREFIX ? unit : unit - b * a.H;
    const int n = PREFIX ? a.rows : min(max(a.lens ? a.lens[b] : a.rows, 0), a.rows);
    const int ql = PREFIX ? a.m : min(max(a.q_lens ? a.q_lens[b] : a.m, 0), a.m);
    const int t0 = group * a.tq, t1 = min(t0 + a.tq, ql);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (t0 >= ql) return;
    ExactOrder o = {n, 0, 0, 0};       // of the rows that the group sees
    if (!PREFIX) o = ex_order(n, ql, t0, t1, a.window, a.sinks, WR);
    const int steps = (o.C + WR - 1) / WR;
    const int s0 = (int)((long long)steps * sp / a.nsp), s1 = (int)((long long)steps * (sp + 1) / a.nsp);
    const int loads = 2 * (s1 - s0);

    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(bars + i, 1);
            mbar_init(bars + RING + i, W);
        }
        fence_mbar_init();
    }
    __syncthreads();
    int issued = 0;
    // Once a wait of this lane has given up: how many loads were issued then (-1 before). It waits no more (no
    // polls: a branch around each wait took up to 12 % of a call) and issues no more copies; what is left of
    // the steps says nothing then.
    int late = -1;
    uint32_t polls = a.polls;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool ok = wait_for(bar, parity, polls);
        late = !ok && late < 0 ? issued : late;
        polls = ok ? polls : 0u;
    };
    // Unit u (keys and values of a step in turn), by warp 0 once all warps are done with its place.
    auto load = [&]() {
        if (issued >= loads) return;
        const int at = issued % RING;
        if (issued >= RING) wait(empty + at * 8, (issued / RING + 1) & 1);
        if (lane == 0 && late < 0) {
            const int row = ex_row(o, (s0 + issued / 2) * WR);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + at * 8),
                         "r"(UNIT)
                         : "memory");
            tma_load_5d(ring + at * UNIT, issued & 1 ? &vmap : &kmap, row, h * a.head_mul,
                        b * a.seq_mul, full + at * 8);
        }
        ++issued;
    };
    if (warp == 0)
        for (int i = 0; i < RING; ++i) load();

    // this warp's tile of 8 rows
    const int tpt = ex_tpt(a.G);
    Rows x8;
    x8.init();
    const int tok_in = x8.g / a.G, head = x8.g - tok_in * a.G;
    const int tile0 = t0 + warp * tpt, ti = tile0 + tok_in;
    const bool any = tile0 < t1, live = tok_in < tpt && ti < t1;
    const int pos = PREFIX ? n - 1 : n - ql + ti;
    const int tp0 = PREFIX ? n - 1 : n - ql + tile0;
    const int tp1 = PREFIX ? n - 1 : n - ql + min(tile0 + tpt, t1) - 1;
    const char *qp = a.q;
    if (live)
        qp += (PREFIX ? ti : b) * a.q_seq + (h * a.G + head) * a.q_head + (PREFIX ? 0 : ti) * a.q_tok;
    x8.begin(qp, live);

    for (int u = 0; u < loads; u += 2) {
        const int c0 = (s0 + u / 2) * WR;
        const int seen = ex_seen(o, c0, WR), row0 = ex_row(o, c0);
        const int ka = u % RING, va = (u + 1) % RING;
        wait(full + ka * 8, (u / RING) & 1);
        wait(full + va * 8, ((u + 1) / RING) & 1);
        if (!PREFIX && seen < WR) {
            // values that no token of the group sees may be anything (the same steps in all warps)
            if (warp == 0) Rows::clear(ring + va * UNIT, seen);
            __syncthreads();
        }
        // rows of this step that the warp's tokens see: all, some, or none
        const bool all = seen == WR && (PREFIX || (row0 + WR - 1 <= tp0 &&
                                                   (row0 + WR <= a.sinks || row0 > tp1 - a.window)));
        const bool none = !any || (!PREFIX && (row0 > tp1 || (row0 + WR - 1 <= tp0 - a.window &&
                                                              row0 >= a.sinks)));
        if (!none) {
            float s[NT][2];
            x8.scores(ring + ka * UNIT, s);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) s[nt][x] *= a.scale_log2;
            if (!all) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = 8 * nt + 2 * x8.t + x, j = row0 + r;
                        const bool see = r < seen && (PREFIX || (j <= pos && (j < a.sinks ||
                                                                 j > pos - a.window)));
                        if (!see) s[nt][x] = -CUDART_INF_F;
                    }
            }
            x8.weights(s);
            x8.values(ring + va * UNIT);
        }
        __syncwarp();
        if (lane == 0) {
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(empty + ka * 8) : "memory");
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(empty + va * 8) : "memory");
        }
        if (warp == 0 && u >= LAG) {
            load();
            load();
        }
    }

    const float l = x8.sum();
    if (live) {
        const bool record = PREFIX || a.nsp > 1;
        const long long at = ((long long)unit * a.nsp + sp) * a.m * a.G + (long long)ti * a.G + head;
        if (record) {
            if (x8.t == 0) *reinterpret_cast<float2 *>(a.pre_ml + 2 * at) = make_float2(x8.m, l);
            float *to = a.pre_o + at * EX_D + 2 * x8.t;
#pragma unroll
            for (int i = 0; i < 16; ++i) *reinterpret_cast<float2 *>(to + 8 * i) = x8.o[i];
        } else {
            const float inv = inverse(l);
            char *to = a.out + b * a.o_seq + (long long)(h * a.G + head) * a.o_head + ti * a.o_tok;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = 8 * i + 2 * x8.t;
                if constexpr (F32IO)
                    *reinterpret_cast<float2 *>(to + d * 4) =
                        make_float2(x8.o[i].x * inv, x8.o[i].y * inv);
                else
                    *reinterpret_cast<uint32_t *>(to + d * 2) = pack(x8.o[i].x * inv, x8.o[i].y * inv);
            }
        }
    }
    if (late >= 0) {
        // copies still in flight end before the block does (bounded); the first lane has issued them
        atomicExch(&g_rows_status, 1);
        if (warp == 0 && lane == 0)
            for (int i = max(0, late - RING); i < late; ++i)
                wait_for(full + (i % RING) * 8, (i / RING) & 1, EX_POLLS);
    }
}

template <bool F32ROWS, bool F32IO, bool PREFIX>
cudaError_t launch(const TileArgs &a, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s) {
    auto kern = exact_rows_kernel<F32ROWS, F32IO, PREFIX>;
    static std::atomic<unsigned long long> set{0};   // devices whose attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ROWS_SMEM);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    const long long blocks = (long long)(PREFIX ? a.H : a.B * a.H) * a.pairs * a.nsp;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    kern<<<(unsigned)blocks, 32 * W, ROWS_SMEM, s>>>(a, k, v);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_exact_rows(const TileArgs &a, const CUtensorMap &k, const CUtensorMap &v,
                              bool f32_rows, bool f32_io, bool prefix, cudaStream_t s) {
    if (f32_rows)
        return prefix ? launch<true, true, true>(a, k, v, s) : launch<true, true, false>(a, k, v, s);
    if (f32_io)
        return prefix ? launch<false, true, true>(a, k, v, s) : launch<false, true, false>(a, k, v, s);
    return prefix ? launch<false, false, true>(a, k, v, s) : launch<false, false, false>(a, k, v, s);
}

cudaError_t exact_rows_status(int *timed_out, cudaStream_t s) {
    int x = 0;
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&x, g_rows_status, sizeof(int), 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && x)
        e = cudaMemcpyToSymbolAsync(g_rows_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    *timed_out = x;
    return e;
}

}  // namespace iskv
