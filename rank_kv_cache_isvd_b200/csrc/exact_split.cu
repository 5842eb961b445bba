// Attention of few query rows over many exact KV rows, and the merge of its splits.
//
//   o_q = sum_j p_qj v_j / sum_j p_qj,   p_qj = 2^(s_qj - m_q),   s_qj = q . k_j log2(e)/sqrt(128)
//
// Decode reads every visible key and value once and does 4 G flops per pair of their bytes: it is
// bound by HBM. So the layout serves the loads. A warp owns 32 bf16 (16 float32) rows of a step and a
// ring of three units of 8 KB in shared memory, which it fills by TMA (keys and values in turn) and
// waits for by itself: no barrier joins the warps until the end of an item, and up to 192 KB per SM are
// in flight (6.8 TB/s while they stream). (Loads by cp.async, one per 16 bytes, cost 750 instructions
// per warp and step, two thirds of them for addresses: 220 us at 8 x 32768 rows of 8 kv-heads.)
//
// The products of a warp's 8 query rows are in exact_warp.cuh.
//
// Behind a kernel that does a shared prefix (it starts on the SMs that the other leaves) the records of
// that one join where an item ends. (Two kernels side by side on parts of the SMs, with all records
// joined by the merge kernel, took 77 to 94 us at 130 sequences where this took 73, the merge 12 of them.)
//
// Teams of 1, 2, 4 or 8 warps work by themselves. By items: a team takes whole items; long ones go to
// a block or a cluster of up to 8 blocks that share out the item's steps and join their results
// through distributed shared memory: o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. One launch, no
// workspace. By steps: the flat space of (item, step) is cut into equal ranges, one per team, so that
// items of any number and lengths fill the GPU evenly; an item that several teams share leaves one
// record per team in global memory, which the merge kernel joins in the same way.
#include <math_constants.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "exact.cuh"
#include "exact_warp.cuh"

namespace iskv {
namespace {

constexpr int UNITS = 3;               // of a warp's ring: keys, values, keys, ... of its steps
constexpr int RED = EX_D + 8;          // stride of joined rows: the warps' stores meet no conflicts

__device__ int g_split_status;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// Address of this block's shared address `a` in the cluster's block `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t a, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float ldc1(uint32_t a) {
    float f;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
    return f;
}
__device__ __forceinline__ float4 ldc4(uint32_t a) {
    float4 f;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                 : "r"(a)
                 : "memory");
    return f;
}

// Where an item's rows and queries are, and the order of its rows.
struct Item {
    int b, h, rt;         // b < 0: shared prefix
    int n, ql;            // of sequence b
    ExactOrder o;
    int i0, i1;           // its tokens (sequences, for the shared prefix)
};

template <int WR>
__device__ __forceinline__ void geometry(const ExactArgs &a, Item &it) {
    const int tpt = ex_tpt(a.G);
    it.i0 = it.rt * tpt;
    if (it.b < 0) {
        it.i1 = min(it.i0 + tpt, a.B);
        it.o = {a.P, 0, 0, 0};
    } else {
        it.i1 = min(it.i0 + tpt, it.ql);
        it.o = ex_order(it.n, it.ql, it.i0, it.i1, a.window, a.sinks, WR);
    }
}

// A way through a share of the work: the item, and the steps [s0, s1) of it to do.
template <int WR>
struct Walk {
    Item it;
    int s0, s1;
    unsigned g, end;      // by steps: place in the flat space; by items: number of the item
    unsigned first;       // by steps: where the item begins
    int S;                // by steps: its length there

    // -- by items: `rank` of `parts` blocks does its part of every item
    __device__ __forceinline__ void settle(const ExactArgs &a, int rs, int rank, int parts) {
        geometry<WR>(a, it);
        const unsigned n = (unsigned)max(1, (it.o.C + rs - 1) / rs);
        s0 = (int)(n * rank / parts);
        s1 = (int)(n * (rank + 1) / parts);
    }
    __device__ __forceinline__ void seq(const ExactArgs &a) {
        it.n = ex_len(a, it.b);
        it.ql = ex_qlen(a, it.b);
    }
    // Items that have no tokens are passed over. False: the share is done.
    __device__ __forceinline__ bool begin(const ExactArgs &a, unsigned from, unsigned to, int rs,
                                          int rank, int parts) {
        g = from;
        end = to;
        if (g >= end) return false;
        const unsigned unit = g / (unsigned)a.rt_max;
        it.rt = (int)(g - unit * a.rt_max);
        it.b = (int)(unit / (unsigned)a.H);
        it.h = (int)(unit - (unsigned)it.b * a.H);
        seq(a);
        while (it.rt * ex_tpt(a.G) >= it.ql)
            if (!step(a)) return false;
        settle(a, rs, rank, parts);
        return true;
    }
    __device__ __forceinline__ bool step(const ExactArgs &a) {
        if (++g >= end) return false;
        if (++it.rt == a.rt_max) {
            it.rt = 0;
            if (++it.h == a.H) {
                it.h = 0;
                ++it.b;
                seq(a);
            }
        }
        return true;
    }

    // -- by steps
    __device__ __forceinline__ void cut() {
        s0 = (int)(g - first);
        s1 = (int)min((unsigned)S, s0 + (end - g));
    }
    // From the item that place g < length of the space belongs to. By a whole warp.
    __device__ __forceinline__ void begin_steps(const ExactArgs &a, unsigned from, unsigned to, int rs) {
        g = from;
        end = to;
        const int lane = threadIdx.x & 31;
        const ExactSpan p = ex_shared_span(a, rs);
        unsigned at = (unsigned)a.H * p.RT * p.S;
        ExactSpan s = p;
        if (g < at) {
            it.b = -1;
            it.n = it.ql = 0;
            at = 0;
        } else if (!a.lens && !a.q_lens) {
            s = ex_seq_span(a, a.rows, a.m, rs, WR);
            const unsigned each = (unsigned)a.H * s.RT * s.S;
            it.b = (int)((g - at) / each);
            at += it.b * each;
            it.n = a.rows;
            it.ql = a.m;
        } else {
            it.b = 0;
            for (int b0 = 0; b0 < a.B; b0 += 32) {
                const int b = b0 + lane;
                unsigned len = 0;
                if (b < a.B) {
                    const ExactSpan x = ex_seq_span(a, ex_len(a, b), ex_qlen(a, b), rs, WR);
                    len = (unsigned)a.H * x.RT * x.S;
                }
                unsigned sum = len;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned x = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += x;
                }
                const unsigned past = __ballot_sync(0xffffffffu, at + sum > g);
                if (past) {
                    const int l = __ffs(past) - 1;
                    it.b = b0 + l;
                    at += __shfl_sync(0xffffffffu, sum - len, l);
                    break;
                }
                at += __shfl_sync(0xffffffffu, sum, 31);
            }
            seq(a);
            s = ex_seq_span(a, it.n, it.ql, rs, WR);
        }
        S = s.S;
        const unsigned i = (g - at) / (unsigned)S;
        it.h = (int)(i / (unsigned)s.RT);
        it.rt = (int)(i - (unsigned)it.h * s.RT);
        first = at + i * S;
        geometry<WR>(a, it);
        cut();
    }

    // To the next item of the share; false: there is none.
    __device__ __forceinline__ bool next(const ExactArgs &a, int rs, int rank, int parts) {
        if (a.by_items) {
            do {
                if (!step(a)) return false;
            } while (it.rt * ex_tpt(a.G) >= it.ql);
            settle(a, rs, rank, parts);
            return true;
        }
        g += (unsigned)(s1 - s0);
        if (g >= end) return false;
        first += S;
        const int RT = it.b < 0 ? ex_shared_span(a, rs).RT
                                : (it.ql + ex_tpt(a.G) - 1) / ex_tpt(a.G);
        if (++it.rt == RT) {
            it.rt = 0;
            if (++it.h == a.H) {
                it.h = 0;
                ExactSpan s;
                do {
                    ++it.b;
                    seq(a);
                    s = ex_seq_span(a, it.n, it.ql, rs, WR);
                } while (s.S == 0 && it.b + 1 < a.B);
                S = s.S;
            }
        }
        geometry<WR>(a, it);
        cut();
        return true;
    }
};

template <bool F32ROWS, bool F32IO, bool MASS>
__global__ void __launch_bounds__(32 * EX_WARPS, 1)
exact_split_kernel(const __grid_constant__ ExactArgs a, const __grid_constant__ ExactMaps maps) {
    using Rows = WarpRows<F32ROWS, F32IO>;
    constexpr int WR = Rows::WR, NT = Rows::NT;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    float *red = reinterpret_cast<float *>(smem + EX_WARPS * UNITS * UNIT);   // [8][8][RED]
    float *red_m = red + EX_WARPS * EX_QROWS * RED, *red_l = red_m + EX_WARPS * EX_QROWS;  // [8][8]
    float *sum_m = red_l + EX_WARPS * EX_QROWS, *sum_l = sum_m + EX_QROWS;    // [8], of a block
    uint64_t *bars = reinterpret_cast<uint64_t *>(sum_l + EX_QROWS);          // [8][UNITS]
    const uint32_t ring = smem_u32(smem) + warp * UNITS * UNIT;
    const uint32_t bar = smem_u32(bars) + warp * UNITS * 8;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
        if (a.rows > 0) {                            // the first copies then find the maps at hand
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k))
                         : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v))
                         : "memory");
        }
#pragma unroll
        for (int i = 0; i < UNITS; ++i) mbar_init(bars + warp * UNITS + i, 1);
        fence_mbar_init();
    }
    __syncwarp();
    // teams of T warps, tw of which this one is; `parts` blocks of a cluster share an item
    const int T = a.team, tw = warp & (T - 1), team0 = warp - tw;
    const int rs = WR * T;
    const int parts = a.by_items ? a.cluster : 1;
    const int rank = parts > 1 ? (int)(blockIdx.x & (unsigned)(parts - 1)) : 0;
    auto team_sync = [&]() {
        if (T == EX_WARPS) __syncthreads();
        else if (T == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / T), "r"(32 * T) : "memory");
    };
    Walk<WR> w;
    unsigned from, to;
    bool have;
    const unsigned my_team = (blockIdx.x / (unsigned)parts) * (EX_WARPS / T) + warp / T;
    if (a.by_items) {
        from = my_team * a.share + min(my_team, a.extra);
        to = min(a.items, from + a.share + (my_team < a.extra ? 1u : 0u));
        have = w.begin(a, from, to, rs, rank, parts);
    } else {
        const unsigned length = ex_length(a, a.B, rs, WR);
        const unsigned per = (length + a.teams - 1) / a.teams;
        from = my_team * per;
        to = min(length, from + per);
        have = from < length;
        if (have) w.begin_steps(a, from, to, rs);
    }
    // Once a wait of this lane has given up: how many loads were issued then (-1 before). It waits no more
    // and, if it is the first lane, issues no more copies. The lanes do not agree on it (a vote behind every
    // wait took 6 % of a call over float32 rows); they go through what is left of the steps, whose results
    // say nothing then.
    int late = -1;
    if (have) {
        Walk<WR> nw = w;                             // what is loaded next: nw's step `ns`, keys
        int ns = nw.s0, loads = 0;                   // first (`loads` even), then values
        uint32_t ld_at = 0;
        bool more = true;
        // Queries into L2, ahead of the rows' copies: they are read when the item begins.
        auto bring_queries = [&](const Item &it) {
            const int row = lane >> 2, line = lane & 3, i = it.i0 + row / a.G;
            if (i < it.i1 && (F32IO || line < 2))
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    a.q + (it.b < 0 ? i : it.b) * a.q_seq + (it.h * a.G + row % a.G) * a.q_head +
                    (it.b < 0 ? 0 : i) * a.q_tok + line * 128));
        };
        bring_queries(nw.it);
        uint64_t policy = l2_policy(nw.it.b >= 0);
        // Fills one unit of the ring with this warp's rows of the next step that has any.
        auto load = [&]() {
            while (more) {
                while (ns >= nw.s1) {
                    more = nw.next(a, rs, rank, parts);
                    if (!more) return;
                    ns = nw.s0;
                    bring_queries(nw.it);
                    policy = l2_policy(nw.it.b >= 0);
                }
                const Item &it = nw.it;
                const int c0 = ns * rs + tw * WR;
                if (c0 >= it.o.C) {
                    ++ns;
                    continue;
                }
                if (lane == 0 && late < 0) {
                    const int row = ex_row(it.o, c0);
                    const uint32_t b = bar + ld_at * 8;
                    const CUtensorMap *map = it.b < 0 ? (loads & 1 ? &maps.pv : &maps.pk)
                                                      : (loads & 1 ? &maps.v : &maps.k);
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b),
                                 "r"(UNIT)
                                 : "memory");
                    const int hd = it.h * (it.b < 0 ? a.p_head_mul : a.head_mul);
                    const int sq = it.b < 0 ? 0 : it.b * a.seq_mul;
                    tma_load_5d(ring + ld_at * UNIT, map, row, hd, sq, b, policy);
                }
                ns += loads & 1;
                ++loads;
                ld_at = ld_at + 1 == UNITS ? 0 : ld_at + 1;
                return;
            }
        };
        // (not unrolled: a first pass waits for its instructions, 0.5 to 2 us of a call)
#pragma unroll 1
        for (int i = 0; i < UNITS; ++i) load();

        Rows x8;
        x8.init();
        uint32_t unit = 0, parity = 0;
        auto full = [&]() {                          // the unit in use has arrived
            if (late < 0 && !wait_for(bar + unit * 8, parity, a.polls)) late = loads;
        };
        auto taken = [&]() {                         // the unit in use is free: refill it
            __syncwarp();
            load();
            if (++unit == UNITS) {
                unit = 0;
                parity ^= 1;
            }
        };
        const int tok = g / a.G, head = g - tok * a.G;

        // a warp per query row, four channels per lane
        auto write = [&](const Item &it, int r, const float4 &y, float L) {
            const int tk = it.i0 + r / a.G, hd = r % a.G;
            if (r / a.G >= ex_tpt(a.G) || tk >= it.i1) return;
            const float inv = inverse(L);
            char *op = a.out + it.b * a.o_seq + (it.h * a.G + hd) * a.o_head + tk * a.o_tok;
            if constexpr (F32IO)
                *reinterpret_cast<float4 *>(op + lane * 16) =
                    make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
            else
                *reinterpret_cast<uint2 *>(op + lane * 8) =
                    make_uint2(pack(y.x * inv, y.y * inv), pack(y.z * inv, y.w * inv));
        };
        auto put = [&](int slot, int r, float M, float L, const float4 &y) {
            float *rec = a.rec + (long long)slot * EX_REC;
            if (lane == 0) {
                rec[r] = M;
                rec[EX_QROWS + r] = L;
            }
            *reinterpret_cast<float4 *>(rec + 2 * EX_QROWS + r * EX_D + lane * 4) = y;
        };
        while (have) {
            const Item it = w.it;
            const int ti = it.i0 + tok;
            const bool live = ti < it.i1;
            const int pos = it.n - it.ql + ti;       // position of this lane's query row
            const char *qp = a.q;
            if (live)
                qp += (it.b < 0 ? ti : it.b) * a.q_seq + (it.h * a.G + head) * a.q_head +
                      (it.b < 0 ? 0 : ti) * a.q_tok;
            x8.begin(qp, live);
            // one token: every row of the order is visible to it, up to C and outside the filling
            const bool plain = it.b < 0 || it.i1 - it.i0 == 1;

            for (int st = w.s0; st < w.s1; ++st) {
                const int c0 = st * rs + tw * WR;
                if (c0 >= it.o.C) continue;
                const int seen = ex_seen(it.o, c0, WR);
                full();
                float s[NT][2];                      // scores of row g at 8 nt + 2 t + x
                x8.scores(ring + unit * UNIT, s);
                taken();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) s[nt][x] *= a.scale_log2;
                if (seen < WR || !plain) {
                    const int row0 = ex_row(it.o, c0);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int r = 8 * nt + 2 * t + x, j = row0 + r;
                            const bool see = r < seen && (plain || (j <= pos && (j < a.sinks ||
                                                                    j > pos - a.window)));
                            if (!see) s[nt][x] = -CUDART_INF_F;
                        }
                }
                if constexpr (MASS) {
                    if (g < a.G) {
                        float *sc = a.scores +
                                    (((long long)it.b * a.H + it.h) * a.G + g) * a.score_st + c0 + 2 * t;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            *reinterpret_cast<float2 *>(sc + 8 * nt) = make_float2(s[nt][0], s[nt][1]);
                    }
                }
                x8.weights(s);
                full();
                if (seen < WR) Rows::clear(ring + unit * UNIT, seen);
                x8.values(ring + unit * UNIT);
                taken();
            }

            // ---- the team's part of the item is complete: join its warps ------------------------
            const float l = x8.sum();
            const bool whole = a.by_items || (w.s0 == 0 && w.s1 == w.S);
            const bool finish = a.by_items || (whole && !MASS && !a.shared_here && !a.nsp);
            // A part of an item leaves a record: the team's, 0 where the item began before it and 1
            // where it goes on behind it; or the item's, where other records join it.
            int slot = 2 * (int)my_team + (w.s0 == 0 ? 1 : 0);
            if (whole) {
                const int RT = ex_shared_span(a, rs).RT;
                slot = 2 * a.teams + (it.b < 0 ? it.h * RT + it.rt : a.H * RT + it.b * a.H + it.h);
            }
            if (!MASS && T == 1 && !(finish && a.nsp)) {
                // one warp: straight from its registers
                if (live && g < a.G * ex_tpt(a.G)) {
                    if (finish) {
                        const float inv = inverse(l);
                        char *op = a.out + it.b * a.o_seq + (it.h * a.G + head) * a.o_head + ti * a.o_tok;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int d = 8 * i + 2 * t;
                            if constexpr (F32IO)
                                *reinterpret_cast<float2 *>(op + d * 4) =
                                    make_float2(x8.o[i].x * inv, x8.o[i].y * inv);
                            else
                                *reinterpret_cast<uint32_t *>(op + d * 2) =
                                    pack(x8.o[i].x * inv, x8.o[i].y * inv);
                        }
                    } else {
                        float *rec = a.rec + (long long)slot * EX_REC;
                        if (t == 0) {
                            rec[g] = x8.m;
                            rec[EX_QROWS + g] = l;
                        }
                        rec += 2 * EX_QROWS + g * EX_D + 2 * t;
#pragma unroll
                        for (int i = 0; i < 16; ++i) *reinterpret_cast<float2 *>(rec + 8 * i) = x8.o[i];
                    }
                }
                have = w.next(a, rs, rank, parts);
                continue;
            }
            float *mine = red + (warp * EX_QROWS + g) * RED + 2 * t;
#pragma unroll
            for (int i = 0; i < 16; ++i) *reinterpret_cast<float2 *>(mine + 8 * i) = x8.o[i];
            if (t == 0) {
                red_m[warp * EX_QROWS + g] = x8.m;
                red_l[warp * EX_QROWS + g] = l;
            }
            team_sync();
            const int used = (it.i1 - it.i0) * a.G;
            const int nsp = !MASS && finish && rank == 0 ? a.nsp : 0;   // (one block of a cluster)
            if (nsp) asm volatile("griddepcontrol.wait;" ::: "memory");
            // Joins the team's parts of row r, and (p_m, p_l, p_y) where there is a prefix.
            auto join = [&](int r, float p_m, float p_l, const float4 &p_y) {
                float M = p_m, mx[EX_WARPS];
#pragma unroll
                for (int x = 0; x < EX_WARPS; ++x) {
                    mx[x] = x < T ? red_m[(team0 + x) * EX_QROWS + r] : -CUDART_INF_F;
                    M = fmaxf(M, mx[x]);
                }
                const float ref = M == -CUDART_INF_F ? 0.f : M;
                const float f0 = ex2(p_m - ref);
                float L = f0 * p_l;
                float4 y = make_float4(f0 * p_y.x, f0 * p_y.y, f0 * p_y.z, f0 * p_y.w);
#pragma unroll
                for (int x = 0; x < EX_WARPS; ++x) {
                    if (x >= T) break;
                    const float f = ex2(mx[x] - ref);
                    const float4 v = *reinterpret_cast<const float4 *>(
                        red + ((team0 + x) * EX_QROWS + r) * RED + lane * 4);
                    L += f * red_l[(team0 + x) * EX_QROWS + r];
                    y.x += f * v.x;
                    y.y += f * v.y;
                    y.z += f * v.z;
                    y.w += f * v.w;
                }
                if (finish && parts == 1) {
                    write(it, r, y, L);
                    if (MASS) __syncwarp();          // every lane has read the row's references and sums
                    if (MASS && lane == 0) {
                        // (reference, sum) of the row for the weights below
                        red_m[team0 * EX_QROWS + r] = ref;
                        red_l[team0 * EX_QROWS + r] = L;
                    }
                } else if (finish) {
                    // the sum replaces the first warp's part, which this warp alone reads
                    *reinterpret_cast<float4 *>(red + r * RED + lane * 4) = y;
                    if (lane == 0) {
                        sum_m[r] = M;
                        sum_l[r] = L;
                    }
                } else {
                    put(slot, r, M, L, y);
                }
            };
            if (!MASS && nsp) {
                // the prefix's records of K of the warp's rows, all loads of a turn in flight together
                auto with_prefix = [&](auto k_, auto u_) {
                    constexpr int K = decltype(k_)::value, U = decltype(u_)::value;
                    for (int r0 = tw; r0 < used; r0 += K * T) {
                        const long long pre = ((long long)it.h * a.nsp * a.B + it.b) * a.G + r0;
                        const long long pre_st = (long long)a.B * a.G;
                        float pm_[K], pl_[K], f[K];
                        float4 y[K];
#pragma unroll
                        for (int k = 0; k < K; ++k) {        // lane x: record x
                            pm_[k] = -CUDART_INF_F;
                            pl_[k] = 0.f;
                            if (lane < nsp && r0 + k * T < used) {
                                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(
                                    a.pre_ml + 2 * (pre + k * T + lane * pre_st)));
                                pm_[k] = ml.x;
                                pl_[k] = ml.y;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < K; ++k) {
                            float top = pm_[k];
#pragma unroll
                            for (int x = 16; x > 0; x >>= 1)
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                            f[k] = ex2(pm_[k] - (top == -CUDART_INF_F ? 0.f : top));
                            float add = f[k] * pl_[k];
#pragma unroll
                            for (int x = 16; x > 0; x >>= 1)
                                add += __shfl_xor_sync(0xffffffffu, add, x);
                            pm_[k] = top;
                            pl_[k] = add;
                            y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        for (int x0 = 0; x0 < nsp; x0 += U) {
                            float4 v[U][K];
#pragma unroll
                            for (int u = 0; u < U; ++u)
#pragma unroll
                                for (int k = 0; k < K; ++k)
                                    v[u][k] = x0 + u < nsp && r0 + k * T < used
                                                  ? __ldcg(reinterpret_cast<const float4 *>(
                                                        a.pre_o + (pre + k * T + (x0 + u) * pre_st) * EX_D +
                                                        lane * 4))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int u = 0; u < U; ++u)
#pragma unroll
                                for (int k = 0; k < K; ++k) {
                                    const float fx = __shfl_sync(0xffffffffu, f[k], (x0 + u) & 31);
                                    y[k].x += fx * v[u][k].x;
                                    y[k].y += fx * v[u][k].y;
                                    y[k].z += fx * v[u][k].z;
                                    y[k].w += fx * v[u][k].w;
                                }
                        }
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            if (r0 + k * T < used) join(r0 + k * T, pm_[k], pl_[k], y[k]);
                    }
                };
                if (used <= T) with_prefix(std::integral_constant<int, 1>{}, std::integral_constant<int, 9>{});
                else with_prefix(std::integral_constant<int, 4>{}, std::integral_constant<int, 3>{});
            } else {
                for (int r = tw; r < used; r += T)
                    join(r, -CUDART_INF_F, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
            }
            if (parts > 1) {
                // row r of the item is finished by block r mod parts; all loads are issued at once
                __syncthreads();
                cluster_sync();
                const int r = rank + warp * parts;
                if (r < used || MASS) {
                    const uint32_t ra = smem_u32(red) + (r & 7) * RED * 4 + lane * 16;
                    const uint32_t ma = smem_u32(sum_m), la = smem_u32(sum_l);
                    float mx[8], lx[8];
                    float4 v[8];
                    if (r < used) {
                        float M = -CUDART_INF_F;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            if (x >= parts) break;
                            mx[x] = ldc1(map_rank(ma + r * 4, x));
                            lx[x] = ldc1(map_rank(la + r * 4, x));
                            v[x] = ldc4(map_rank(ra, x));
                        }
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            if (x >= parts) break;
                            M = fmaxf(M, mx[x]);
                        }
                        const float ref = M == -CUDART_INF_F ? 0.f : M;
                        float L = 0.f;
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            if (x >= parts) break;
                            const float f = ex2(mx[x] - ref);
                            L += f * lx[x];
                            y.x += f * v[x].x;
                            y.y += f * v[x].y;
                            y.z += f * v[x].z;
                            y.w += f * v[x].w;
                        }
                        write(it, r, y, L);
                    }
                    if (MASS && warp < used) {
                        // every block: (reference, sum) of all rows; warp = row, lane x = block x
                        const float mr = lane < parts ? ldc1(map_rank(ma + warp * 4, lane))
                                                      : -CUDART_INF_F;
                        const float lr = lane < parts ? ldc1(map_rank(la + warp * 4, lane)) : 0.f;
                        float M = mr;
#pragma unroll
                        for (int x = 4; x > 0; x >>= 1)
                            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
                        const float ref = M == -CUDART_INF_F ? 0.f : M;
                        float L = ex2(mr - ref) * lr;
#pragma unroll
                        for (int x = 4; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
                        if (lane == 0) {
                            red_m[warp] = ref;
                            red_l[warp] = L;
                        }
                    }
                }
            }
            if (MASS && a.by_items) {
                // the weights of the rows whose scores this team has
                team_sync();
                const int hi = min(it.o.C, w.s1 * rs);
                const float *sc = a.scores + ((long long)it.b * a.H + it.h) * a.G * a.score_st;
                const long long base = ((long long)it.b * a.H + it.h) * a.rows;
                // U groups of four rows per thread and turn, whose loads are in flight together;
                // scores are padded to whole groups of rows
                auto add = [&](auto rows_, auto u_) {
                    constexpr int RN = decltype(rows_)::value, U = decltype(u_)::value;
                    float ref[RN], inv[RN];
#pragma unroll
                    for (int r = 0; r < RN; ++r) {
                        ref[r] = r < a.G ? red_m[team0 * EX_QROWS + r] : 0.f;
                        inv[r] = r < a.G ? inverse(red_l[team0 * EX_QROWS + r]) : 0.f;
                    }
                    const int j0 = w.s0 * rs + 4 * (tw * 32 + lane), step = 128 * T;
                    for (int j = j0; j < hi; j += U * step) {
                        float4 f[U][RN];
                        float old[U][4];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int at = j + u * step;
#pragma unroll
                            for (int r = 0; r < RN; ++r)
                                f[u][r] = at < hi && r < a.G
                                              ? *reinterpret_cast<const float4 *>(sc + r * a.score_st + at)
                                              : make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F,
                                                            -CUDART_INF_F);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                old[u][y] = at + y < hi ? a.mass[base + at + y] : 0.f;
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int at = j + u * step;
#pragma unroll
                            for (int r = 0; r < RN; ++r) {
                                old[u][0] += ex2(f[u][r].x - ref[r]) * inv[r];
                                old[u][1] += ex2(f[u][r].y - ref[r]) * inv[r];
                                old[u][2] += ex2(f[u][r].z - ref[r]) * inv[r];
                                old[u][3] += ex2(f[u][r].w - ref[r]) * inv[r];
                            }
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if (at + y < hi) a.mass_out[base + at + y] = old[u][y];
                        }
                    }
                };
                if (a.G <= 4) add(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
                else add(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
            }
            team_sync();                             // what joined may be overwritten
            if (parts > 1) cluster_sync();
            have = w.next(a, rs, rank, parts);
        }
        if (late >= 0) {
            // copies still in flight end before the block does (bounded); the first lane has issued them
            atomicExch(&g_split_status, 1);
            for (int i = max(0, late - UNITS); lane == 0 && i < late; ++i)
                wait_for(bar + (i % UNITS) * 8, (i / UNITS) & 1, EX_POLLS);
        }
    }
    // the merge waits for this kernel alone: it must not end before the one that ran beside it
    if (a.after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- merge --------------------------------------------------------------------------------------
// Blocks 0 .. B*H*RTmax - 1 each join the records of one item (for the shared prefix: a sequence's
// own records with its rows of the prefix's). The blocks after them add the weights to `mass`.
constexpr int MERGE_T = 256;
constexpr int MASS_ROWS = 4 * MERGE_T;      // rows per mass block
constexpr int MERGE_CHUNK = 256;            // records whose weights are at hand

template <bool F32ROWS, bool F32IO, bool MASS>
__global__ void __launch_bounds__(MERGE_T)
exact_merge_kernel(const __grid_constant__ ExactArgs a, int rt_max, int mass_blocks) {
    constexpr int WR = ex_warp_rows(F32ROWS);
    const int RS = WR * a.team;
    __shared__ float wgt[EX_QROWS][MERGE_CHUNK];
    __shared__ float row_m[EX_QROWS], row_l[EX_QROWS];
    __shared__ __align__(16) float part[MERGE_T * 4];
    const int n_items = a.B * a.H * rt_max;
    const bool mass_block = (int)blockIdx.x >= n_items;
    int b, h, rt = 0, chunk = 0;
    if (!mass_block) {
        const int unit = blockIdx.x / rt_max;
        rt = blockIdx.x - unit * rt_max;
        b = unit / a.H;
        h = unit - b * a.H;
    } else {
        const int x = blockIdx.x - n_items;
        const int unit = x / mass_blocks;
        chunk = x - unit * mass_blocks;
        b = unit / a.H;
        h = unit - b * a.H;
    }
    const int n = ex_len(a, b), ql = ex_qlen(a, b), tpt = ex_tpt(a.G);
    const ExactSpan sp = ex_seq_span(a, n, ql, RS, WR), sh = ex_shared_span(a, RS);
    if (rt >= sp.RT || (mass_block && chunk * MASS_ROWS >= n)) return;
    const unsigned length = ex_length(a, a.B, RS, WR);
    const unsigned per = (length + a.teams - 1) / a.teams;
    const unsigned first = ex_length(a, b, RS, WR) + ((unsigned)h * sp.RT + rt) * sp.S;
    const int own_c0 = (int)(first / per), own_c1 = (int)((first + sp.S - 1) / per);
    const int n_own = own_c1 - own_c0 + 1;
    if (!MASS && !a.shared_here && !a.nsp && n_own == 1) return;   // the split kernel wrote it
    // shared prefix: tile and row of this sequence
    int n_sh = 0, sh_c0 = 0;
    const int sh_rt = b / tpt, sh_row = (b - sh_rt * tpt) * a.G;
    if (a.shared_here && sh.S) {
        const unsigned f = ((unsigned)h * sh.RT + sh_rt) * sh.S;
        sh_c0 = (int)(f / per);
        n_sh = (int)((f + sh.S - 1) / per) - sh_c0 + 1;
    }
    const int nrec = n_own + n_sh + a.nsp;
    const int whole0 = 2 * a.teams;
    auto slot_of = [&](int i) {
        if (i < n_own)
            return n_own == 1 ? whole0 + a.H * sh.RT + b * a.H + h
                              : 2 * (own_c0 + i) + (i == 0 ? 1 : 0);
        return n_sh == 1 ? whole0 + h * sh.RT + sh_rt
                         : 2 * (sh_c0 + i - n_own) + (i == n_own ? 1 : 0);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rows = min(tpt, ql - rt * tpt) * a.G;              // live rows of the tile
    auto ml = [&](int i, int r, float &m_, float &l_) {
        if (i < n_own + n_sh) {
            const float *rec = a.rec + (long long)slot_of(i) * EX_REC;
            const int rr = i < n_own ? r : sh_row + r;
            m_ = rec[rr];
            l_ = rec[EX_QROWS + rr];
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(
                a.pre_ml + 2 * (((long long)h * a.nsp + (i - n_own - n_sh)) * a.B * a.G +
                                (long long)b * a.G + r));
            m_ = x.x;
            l_ = x.y;
        }
    };
    // a warp per row: M = max m_i, L = sum of 2^(m_i - M) l_i
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < rows) {
        float M = -CUDART_INF_F, L = 0.f;
        for (int i = lane; i < nrec; i += 32) {
            float m_, l_;
            ml(i, warp, m_, l_);
            const float top = fmaxf(M, m_);
            if (top > -CUDART_INF_F) L = L * ex2(M - top) + l_ * ex2(m_ - top);
            M = top;
        }
        float top = M;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        L *= ex2(M - ref);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) {
            row_m[warp] = ref;
            row_l[warp] = L;
        }
    }
    __syncthreads();
    if (MASS && mass_block) {
        float inv[EX_QROWS], ref[EX_QROWS];
        const float *sc[EX_QROWS];
#pragma unroll
        for (int r = 0; r < EX_QROWS; ++r) {
            if (r >= a.G) break;
            inv[r] = inverse(row_l[r]);
            ref[r] = row_m[r];
            sc[r] = a.scores + (((long long)b * a.H + h) * a.G + r) * a.score_st;
        }
        const long long base = ((long long)b * a.H + h) * a.rows;
#pragma unroll
        for (int x = 0; x < MASS_ROWS / MERGE_T; ++x) {
            const int j = chunk * MASS_ROWS + x * MERGE_T + threadIdx.x;
            if (j >= n) break;
            float w = 0.f;
#pragma unroll
            for (int r = 0; r < EX_QROWS; ++r) {
                if (r >= a.G) break;
                w += ex2(sc[r][j] - ref[r]) * inv[r];
            }
            a.mass_out[base + j] = a.mass[base + j] + w;
        }
        return;
    }
    // thread = (replica, row, 4 channels); replica y takes the records y, y + reps, ...
    const int lanes = rows * (EX_D / 4), reps = MERGE_T / lanes;
    const int y = threadIdx.x / lanes, e = threadIdx.x - y * lanes;
    const int r = e / (EX_D / 4), d = (e % (EX_D / 4)) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < nrec; i0 += MERGE_CHUNK) {
        const int i1 = min(nrec, i0 + MERGE_CHUNK);
        if (i0 > 0) __syncthreads();
        if (warp < rows)
            for (int i = i0 + lane; i < i1; i += 32) {
                float m_, l_;
                ml(i, warp, m_, l_);
                wgt[warp][i - i0] = ex2(m_ - row_m[warp]);
            }
        __syncthreads();
        if (y < reps) {
#pragma unroll 4
            for (int i = i0 + y; i < i1; i += reps) {
                const float *src;
                if (i < n_own + n_sh)
                    src = a.rec + (long long)slot_of(i) * EX_REC + 2 * EX_QROWS +
                          (i < n_own ? r : sh_row + r) * EX_D + d;
                else
                    src = a.pre_o + (((long long)h * a.nsp + (i - n_own - n_sh)) * a.B * a.G +
                                     (long long)b * a.G + r) * EX_D + d;
                const float4 v = *reinterpret_cast<const float4 *>(src);
                const float f = wgt[r][i - i0];
                acc.x += f * v.x;
                acc.y += f * v.y;
                acc.z += f * v.z;
                acc.w += f * v.w;
            }
        }
    }
    *reinterpret_cast<float4 *>(part + threadIdx.x * 4) = acc;
    __syncthreads();
    if (y == 0) {
        for (int z = 1; z < reps; ++z) {
            const float4 v = *reinterpret_cast<const float4 *>(part + (z * lanes + e) * 4);
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        const float inv = inverse(row_l[r]);
        const int tk = rt * tpt + r / a.G, hd = r % a.G;
        char *op = a.out + b * a.o_seq + (h * a.G + hd) * a.o_head + tk * a.o_tok;
        if constexpr (F32IO)
            *reinterpret_cast<float4 *>(op + d * 4) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        else
            *reinterpret_cast<uint2 *>(op + d * 2) =
                make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
    }
}

// The kernel's shared-memory limit, set on the first launch on each device.
cudaError_t once_per_device(std::atomic<unsigned long long> &set, const void *kern, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (set.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_release);
    return e;
}

constexpr size_t SPLIT_SMEM = EX_WARPS * UNITS * (UNIT + 8) + EX_WARPS * EX_QROWS * (RED + 2) * 4 +
                              2 * EX_QROWS * 4;
static_assert(SPLIT_SMEM <= 227 * 1024, "shared memory");

void config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *at, int grid, int cluster, bool after) {
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * EX_WARPS);
    cfg.dynamicSmemBytes = SPLIT_SMEM;
    int n = 0;
    if (after) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = at;
    cfg.numAttrs = n;
}

template <bool F32ROWS, bool F32IO, bool MASS>
cudaError_t split(const ExactArgs &a, const ExactMaps &maps, cudaStream_t s) {
    auto kern = exact_split_kernel<F32ROWS, F32IO, MASS>;
    static std::atomic<unsigned long long> set{0};   // devices whose attribute is set
    const cudaError_t e = once_per_device(set, reinterpret_cast<const void *>(kern), (int)SPLIT_SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    config(cfg, at, a.grid, a.cluster, a.after);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

template <bool F32ROWS, bool F32IO, bool MASS>
cudaError_t merge(const ExactArgs &a, cudaStream_t s) {
    const int tpt = ex_tpt(a.G);
    const int rt_max = (a.m + tpt - 1) / tpt;
    const int mass_blocks = MASS ? (a.rows + MASS_ROWS - 1) / MASS_ROWS : 0;
    const long long blocks = (long long)a.B * a.H * (rt_max + mass_blocks);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(MERGE_T);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, exact_merge_kernel<F32ROWS, F32IO, MASS>, a, rt_max, mass_blocks);
}

}  // namespace

cudaError_t launch_exact_split(const ExactArgs &a, const ExactMaps &maps, bool f32_rows, bool f32_io,
                               cudaStream_t s) {
    if (a.mass) {
        if (f32_rows) return split<true, true, true>(a, maps, s);
        return f32_io ? split<false, true, true>(a, maps, s) : split<false, false, true>(a, maps, s);
    }
    if (f32_rows) return split<true, true, false>(a, maps, s);
    return f32_io ? split<false, true, false>(a, maps, s) : split<false, false, false>(a, maps, s);
}

cudaError_t launch_exact_merge(const ExactArgs &a, bool f32_rows, bool f32_io, cudaStream_t s) {
    if (a.by_items) return cudaSuccess;              // nothing is left to join
    if (a.mass) {
        if (f32_rows) return merge<true, true, true>(a, s);
        return f32_io ? merge<false, true, true>(a, s) : merge<false, false, true>(a, s);
    }
    if (f32_rows) return merge<true, true, false>(a, s);
    return f32_io ? merge<false, true, false>(a, s) : merge<false, false, false>(a, s);
}

int exact_split_clusters(int cluster) {
    // the same shared memory, to a few KB, and one block per SM for all variants
    static std::atomic<int> known[64][4];            // per device and log2 of the cluster; 0: unknown
    static std::atomic<unsigned long long> set{0};
    int dev = 0, lg = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    while ((1 << lg) < cluster) ++lg;
    std::atomic<int> &slot = known[dev & 63][lg];
    int n = slot.load(std::memory_order_acquire);
    if (n) return n;
    auto kern = exact_split_kernel<false, true, false>;
    if (once_per_device(set, reinterpret_cast<const void *>(kern), (int)SPLIT_SMEM) !=
        cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    config(cfg, at, cluster, cluster, false);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) return 0;
    slot.store(n, std::memory_order_release);
    return n;
}

cudaError_t exact_split_status(int *timed_out, cudaStream_t s) {
    int x = 0;
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&x, g_split_status, sizeof(int), 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && x)
        e = cudaMemcpyToSymbolAsync(g_split_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    *timed_out = x;
    return e;
}

}  // namespace iskv
