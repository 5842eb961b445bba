// Attention of few query rows over many exact KV rows, and the merge of its splits.
//
//   o_q = sum_j p_qj v_j / sum_j p_qj,   p_qj = 2^(s_qj - m_q),   s_qj = q . k_j log2(e)/sqrt(128)
//
// Decode reads every visible key and value once and does 4 G flops per pair of their bytes: it is
// bound by HBM. So the layout serves the loads. A warp owns 16 rows of a step at a time and a ring
// of three such stages in shared memory, which it fills by TMA (one box of keys, one of values) and
// waits for by itself: no barrier joins the warps until the end of an item, and 128 KB per SM are in
// flight. (Loads by cp.async, one per 16 bytes, cost 750 instructions per warp and step, two thirds
// of them for addresses: 220 us at 8 x 32768 rows of 8 kv-heads.)
//
// Products run on mma.sync m16n8k16 (bf16): a tile of 8 query rows fills half of its 16 rows, and
// tcgen05 would want 64 or 128. Float32 operands are split in three bf16 terms (24 bits), x = hi +
// mid + lo: hi sits in rows 0-7 of the A operand and mid in rows 8-15, so one instruction does both
// terms and both sums land in one thread; lo takes a second one. The same for the weights p, so
// that float32 outputs keep float32 accuracy (a weight rounded to bf16 would cost 2^-9).
//
// Tensor cores truncate where they add, always toward zero: over the hundred steps of a long cache
// the outputs lost 4e-6. So each step's products start from zero and are added to the outputs in
// float32 arithmetic (round to nearest), smallest terms first: 8e-7 at 8 x 32768 rows.
//
// By items: a cluster of 1 to 8 blocks shares out an item's steps and joins their results through
// distributed shared memory: o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. One launch, no
// workspace. By steps: the flat space of (item, step) is cut into equal ranges, one per block, so
// that items of any number and lengths fill the GPU evenly; an item that several blocks share
// leaves one record per block in global memory, which the merge kernel joins in the same way.
#include <math_constants.h>
#include <string.h>

#include <atomic>

#include "exact.cuh"
#include "tc_util.cuh"

namespace iskv {
namespace {

constexpr int STAGES = 3;
constexpr uint32_t POLLS = 1u << 18, SUSPEND_NS = 20000;

__device__ int g_split_status;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float2 lds2(uint32_t addr) {
    float2 f;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "r"(addr) : "memory");
    return f;
}
__device__ __forceinline__ float lds1(uint32_t addr) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(addr) : "memory");
    return f;
}
// c += A B with A = 16 x 16, B = 16 x 8, bf16. This thread's A registers: row lane/4 (a0, a2) and
// row lane/4 + 8 (a1, a3), columns 2 (lane%4) + {0, 1} (a0, a1) and + 8 (a2, a3).
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c = A B
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float lo_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
// (x, y) = sum of three pairs of bf16, each the rounding of what the ones before leave.
__device__ __forceinline__ void split3(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack(x, y);
    const float rx = x - lo_of(h), ry = y - hi_of(h);
    m = pack(rx, ry);
    l = pack(rx - lo_of(m), ry - hi_of(m));
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int row, int head,
                                            int seq, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(head), "r"(seq), "r"(bar)
        : "memory");
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < POLLS; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(SUSPEND_NS)
            : "memory");
        if (done) return true;
    }
    return false;
}
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
__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); }

// Where an item's rows and queries are. Its visible rows in an order without the gap between sinks
// and window: c < skp (sk of them, filled up to a multiple of 16) are the sinks, then the rows from
// lo on, up to C.
struct Item {
    int b, h, rt;         // b < 0: shared prefix
    int weight;
    int n, ql;            // of sequence b
    int C, sk, skp, lo;
    int S;
    int i0, i1;           // its tokens (sequences, for the shared prefix)
};

template <int RS>
__device__ __forceinline__ void geometry(const ExactArgs &a, Item &it) {
    const int tpt = ex_tpt(a.G);
    it.i0 = it.rt * tpt;
    it.sk = it.skp = it.lo = 0;
    if (it.b < 0) {
        it.i1 = min(it.i0 + tpt, a.B);
        it.C = a.P;
    } else {
        it.i1 = min(it.i0 + tpt, it.ql);
        const int p0 = it.n - it.ql + it.i0;
        const int hi = max(0, it.n - it.ql + it.i1);
        const int sk = min(a.sinks, hi), lo = max(0, p0 - a.window + 1);
        it.C = hi;
        if (lo > sk) {
            it.sk = sk;
            it.skp = (sk + 15) & ~15;
            it.lo = lo;
            it.C = it.skp + hi - lo;
        }
    }
    it.S = max(1, (it.C + RS - 1) / RS);
}

// A position in the list of items: the item, and where the space that is cut begins with it.
struct Cursor {
    Item it;
    unsigned first;
};

// The item after it: next tile, next kv-head, next sequence with tokens. It must exist.
template <int RS>
__device__ __forceinline__ void next_item(const ExactArgs &a, Cursor &c) {
    Item &it = c.it;
    c.first += it.weight;
    const int RT = it.b < 0 ? ex_shared_span(a, RS).RT
                            : (it.ql + ex_tpt(a.G) - 1) / ex_tpt(a.G);
    if (++it.rt == RT) {
        it.rt = 0;
        if (++it.h == a.H) {
            it.h = 0;
            ExactSpan s;
            do {
                ++it.b;
                it.n = ex_len(a, it.b);
                it.ql = ex_qlen(a, it.b);
                s = ex_seq_span(a, it.n, it.ql, RS);
            } while (s.S == 0 && it.b + 1 < a.B);
            it.weight = s.weight;
        }
    }
    geometry<RS>(a, it);
}

// The item that place g of the space belongs to (g < its length). By a whole warp.
template <int RS>
__device__ __forceinline__ Cursor find_item(const ExactArgs &a, unsigned g) {
    Cursor c;
    Item &it = c.it;
    const int lane = threadIdx.x & 31;
    const ExactSpan p = ex_shared_span(a, RS);
    unsigned at = (unsigned)a.H * p.RT * p.weight;
    int RT = p.RT;
    if (g < at) {
        it.b = -1;
        it.weight = p.weight;
        it.n = it.ql = 0;
        at = 0;
    } else if (!a.lens && !a.q_lens) {
        const ExactSpan s = ex_seq_span(a, a.rows, a.m, RS);
        const unsigned each = (unsigned)a.H * s.RT * s.weight;
        it.b = (int)((g - at) / each);
        at += it.b * each;
        it.n = a.rows;
        it.ql = a.m;
        it.weight = s.weight;
        RT = s.RT;
    } else {
        it.b = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            unsigned len = 0;
            if (b < a.B) {
                const ExactSpan s = ex_seq_span(a, ex_len(a, b), ex_qlen(a, b), RS);
                len = (unsigned)a.H * s.RT * s.weight;
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
        it.n = ex_len(a, it.b);
        it.ql = ex_qlen(a, it.b);
        const ExactSpan s = ex_seq_span(a, it.n, it.ql, RS);
        it.weight = s.weight;
        RT = s.RT;
    }
    const unsigned i = (g - at) / (unsigned)it.weight;
    it.h = (int)(i / (unsigned)RT);
    it.rt = (int)(i - (unsigned)it.h * RT);
    c.first = at + i * it.weight;
    geometry<RS>(a, it);
    return c;
}

// A block's way through its share: the item, and the steps [s0, s1) of it that are the block's.
template <int RS>
struct Walk {
    Cursor c;
    unsigned g, end;      // place in the space, end of the share
    int s0, s1;

    __device__ __forceinline__ void span(const ExactArgs &a, int rank) {
        if (a.by_items) {
            s0 = (int)((unsigned)c.it.S * rank / a.cluster);
            s1 = (int)((unsigned)c.it.S * (rank + 1) / a.cluster);
        } else {
            s0 = (int)(g - c.first);
            s1 = (int)min((unsigned)c.it.weight, s0 + (end - g));
        }
    }
    // To the next item of the share; false: there is none.
    __device__ __forceinline__ bool next(const ExactArgs &a, int rank) {
        g += a.by_items ? 1u : (unsigned)(s1 - s0);
        if (g >= end) return false;
        next_item<RS>(a, c);
        span(a, rank);
        return true;
    }
};

template <bool F32ROWS, bool F32IO, bool MASS>
__global__ void __launch_bounds__(32 * ex_warps(F32ROWS), 1)
exact_split_kernel(const __grid_constant__ ExactArgs a, const __grid_constant__ ExactMaps maps) {
    constexpr int W = ex_warps(F32ROWS);
    constexpr int RS = ex_step_rows(F32ROWS);
    constexpr int HALF = 16 * (F32ROWS ? 512 : 256); // keys of a stage, then as much of values
    constexpr int STAGE = 2 * HALF;
    constexpr int PARTS = F32ROWS ? 4 : 2;           // 128-byte parts of a row
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    float *red = reinterpret_cast<float *>(smem + W * STAGES * STAGE);   // [W][8][128]
    float *red_m = red + W * EX_QROWS * EX_D, *red_l = red_m + W * EX_QROWS;
    float *sum_m = red_l + W * EX_QROWS, *sum_l = sum_m + EX_QROWS;      // [8] each
    uint64_t *bars = reinterpret_cast<uint64_t *>(sum_l + EX_QROWS);     // [W][STAGES]
    const uint32_t ring = smem_u32(smem) + warp * STAGES * STAGE;
    const uint32_t bar = smem_u32(bars) + warp * STAGES * 8;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) mbar_init(bars + warp * STAGES + i, 1);
        fence_mbar_init();
    }
    __syncwarp();
    const int rank = a.cluster > 1 ? (int)(blockIdx.x % (unsigned)a.cluster) : 0;
    const unsigned length = ex_length(a, a.B, RS);
    const unsigned shares = (unsigned)a.grid / a.cluster, share = blockIdx.x / a.cluster;
    Walk<RS> w;
    if (a.by_items) {
        w.g = (unsigned)((unsigned long long)length * share / shares);
        w.end = (unsigned)((unsigned long long)length * (share + 1) / shares);
    } else {
        const unsigned per = (length + shares - 1) / shares;
        w.g = min(length, share * per);
        w.end = min(length, w.g + per);
    }
    bool late = false;                               // a wait hit its bound
    if (w.g < w.end) {
        w.c = find_item<RS>(a, w.g);
        w.span(a, rank);
        Walk<RS> nw = w;                             // what is loaded next: nw's step `ns`
        int ns = nw.s0, ld_stage = 0, ld_count = 0;
        bool more = true;
        // Fills one stage, with this warp's rows of the next step that has any.
        auto load = [&]() {
            while (more) {
                while (ns >= nw.s1) {
                    more = nw.next(a, rank);
                    if (!more) return;
                    ns = nw.s0;
                }
                const Item &it = nw.c.it;
                const int c0 = ns * RS + warp * 16;
                ++ns;
                if (c0 >= it.C) continue;
                if (lane == 0) {
                    const int row = c0 < it.skp ? c0 : c0 - it.skp + it.lo;
                    const uint32_t dst = ring + ld_stage * STAGE, b = bar + ld_stage * 8;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b),
                                 "r"(STAGE)
                                 : "memory");
                    if (it.b < 0) {
                        tma_load_5d(dst, &maps.pk, row, it.h * a.p_head_mul, 0, b);
                        tma_load_5d(dst + HALF, &maps.pv, row, it.h * a.p_head_mul, 0, b);
                    } else {
                        tma_load_5d(dst, &maps.k, row, it.h * a.head_mul, it.b * a.seq_mul, b);
                        tma_load_5d(dst + HALF, &maps.v, row, it.h * a.head_mul, it.b * a.seq_mul, b);
                    }
                }
                ++ld_count;
                ld_stage = ld_stage + 1 == STAGES ? 0 : ld_stage + 1;
                return;
            }
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) load();

        // fragment addresses: 128-byte rows of a part, whose 16-byte chunks are permuted by row
        const int kr = (lane & 7) + ((lane >> 4) << 3), vr = lane & 15;
        const uint32_t k_at = kr * 128 + ((((lane >> 3) & 1) ^ (kr & 7)) << 4);
        const uint32_t v_at = vr * 128 + (((lane >> 4) ^ (vr & 7)) << 4);
        int stage = 0;
        uint32_t parity = 0;
        const int tok = g / a.G, head = g - tok * a.G;

        bool have = true;
        while (have) {
            const Item it = w.c.it;
            uint32_t qh[8][2], qm[F32IO ? 8 : 1][2], ql[F32IO ? 8 : 1][2];
            float2 o[16];
            float m = -CUDART_INF_F, l = 0.f;
            const int ti = it.i0 + tok;
            const bool live = ti < it.i1;
            const int pos = it.n - it.ql + ti;       // position of this lane's query row
            const char *qp = a.q;
            if (live)
                qp += (it.b < 0 ? ti : it.b) * a.q_seq + (it.h * a.G + head) * a.q_head +
                      (it.b < 0 ? 0 : ti) * a.q_tok;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int d = ks * 16 + x * 8 + 2 * t;
                    if constexpr (F32IO) {
                        float2 f = make_float2(0.f, 0.f);
                        if (live) f = *reinterpret_cast<const float2 *>(qp + d * 4);
                        split3(f.x, f.y, qh[ks][x], qm[ks][x], ql[ks][x]);
                    } else {
                        qh[ks][x] = live ? *reinterpret_cast<const uint32_t *>(qp + d * 2) : 0u;
                    }
                }
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = make_float2(0.f, 0.f);
            // one token: every row of the order is visible to it, up to C and outside the filling
            const bool plain = it.b < 0 || it.i1 - it.i0 == 1;

            for (int st = w.s0; st < w.s1; ++st) {
                const int c0 = st * RS + warp * 16;
                if (c0 >= it.C) continue;
                load();
                late |= !wait_for(bar + stage * 8, parity);
                const uint32_t kb_ = ring + stage * STAGE, vb_ = kb_ + HALF;
                const bool sinks = c0 < it.skp;
                const int seen = min(16, (sinks ? it.sk : it.C) - c0);   // rows with a row behind
                if (seen < 16) {
                    // values of rows that nobody sees may be anything: 0 x NaN would reach o
                    for (int r = seen; r < 16; ++r)
                        if (lane < 8 * PARTS)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             vb_ + (lane >> 3) * 2048 + r * 128 + (lane & 7) * 16),
                                         "r"(0)
                                         : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                float s[2][4];
                if constexpr (!F32ROWS) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        uint32_t kb[4];
                        ldsm4(kb_ + (ks >> 2) * 2048 + (k_at ^ ((ks & 3) << 5)), kb);
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const uint32_t b0 = kb[2 * nt], b1 = kb[2 * nt + 1];
                            if constexpr (F32IO) {
                                if (ks == 0) mma0(s[nt], ql[ks][0], 0u, ql[ks][1], 0u, b0, b1);
                                else mma(s[nt], ql[ks][0], 0u, ql[ks][1], 0u, b0, b1);
                                mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], b0, b1);
                            } else {
                                if (ks == 0) mma0(s[nt], qh[ks][0], 0u, qh[ks][1], 0u, b0, b1);
                                else mma(s[nt], qh[ks][0], 0u, qh[ks][1], 0u, b0, b1);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            uint32_t kh[2], km[2], kl[2];
                            const int r = nt * 8 + g;
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int ch = ((ks & 1) * 4 + 2 * x + (t >> 1)) ^ (r & 7);
                                const float2 f = lds2(kb_ + (ks >> 1) * 2048 + r * 128 + ch * 16 +
                                                      (t & 1) * 8);
                                split3(f.x, f.y, kh[x], km[x], kl[x]);
                            }
                            if (ks == 0)
                                mma0(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], kl[0], kl[1]);
                            else
                                mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], kl[0], kl[1]);
                            mma(s[nt], ql[ks][0], 0u, ql[ks][1], 0u, kh[0], kh[1]);
                            mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], km[0], km[1]);
                            mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], kh[0], kh[1]);
                        }
                }
                // scores of row g at 8 nt + 2 t + x of the 16 (rows 8-15 hold the mid terms' sums)
                float p[2][2];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        p[nt][x] = (s[nt][x] + s[nt][2 + x]) * a.scale_log2;
                if (seen < 16 || !plain) {
                    const int row0 = sinks ? c0 : c0 - it.skp + it.lo;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int r = 8 * nt + 2 * t + x, j = row0 + r;
                            const bool see = r < seen && (plain || (j <= pos && (j < a.sinks ||
                                                                    j > pos - a.window)));
                            if (!see) p[nt][x] = -CUDART_INF_F;
                        }
                }
                float top = fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[1][0], p[1][1]));
                if constexpr (MASS) {
                    if (g < a.G) {
                        float *sc = a.scores +
                                    (((long long)it.b * a.H + it.h) * a.G + g) * a.score_st + c0 + 2 * t;
                        *reinterpret_cast<float2 *>(sc) = make_float2(p[0][0], p[0][1]);
                        *reinterpret_cast<float2 *>(sc + 8) = make_float2(p[1][0], p[1][1]);
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // The reference m moves only when a score passes it by 2^8: p stays below 256, and
                // the sums keep their float32 accuracy.
                const bool raise = top > m + 8.f || (m == -CUDART_INF_F && top > m);
                if (__any_sync(0xffffffffu, raise)) {
                    const float nm = raise ? top : m;
                    const float f = m == -CUDART_INF_F ? 0.f : ex2(m - nm);
                    m = nm;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        o[i].x *= f;
                        o[i].y *= f;
                    }
                }
                const float ref = m == -CUDART_INF_F ? 0.f : m;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) p[nt][x] = ex2(p[nt][x] - ref);
                l += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
                uint32_t ph[2], pm[2], pl[2];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
                    split3(p[nt][0], p[nt][1], ph[nt], pm[nt], pl[nt]);
                if constexpr (!F32ROWS) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t vb[4];
                        ldsm4t(vb_ + (i >> 2) * 2048 + (v_at ^ ((i & 3) << 5)), vb);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t b0 = vb[2 * x], b1 = vb[2 * x + 1];
                            float c[4];
                            if constexpr (F32IO) {
                                mma0(c, pl[0], 0u, pl[1], 0u, b0, b1);
                                mma(c, ph[0], pm[0], ph[1], pm[1], b0, b1);
                            } else {
                                mma0(c, ph[0], pm[0], ph[1], pm[1], b0, b1);
                            }
                            o[2 * i + x] = add2(o[2 * i + x],
                                                add2(make_float2(c[0], c[1]), make_float2(c[2], c[3])));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        uint32_t vh[2], vm[2], vl[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float f[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int r = 8 * x + 2 * t + y;
                                const int ch = ((i & 3) * 2 + (g >> 2)) ^ (r & 7);
                                f[y] = lds1(vb_ + (i >> 2) * 2048 + r * 128 + ch * 16 + (g & 3) * 4);
                            }
                            split3(f[0], f[1], vh[x], vm[x], vl[x]);
                        }
                        float c[4];
                        mma0(c, ph[0], pm[0], ph[1], pm[1], vl[0], vl[1]);
                        mma(c, pl[0], 0u, pl[1], 0u, vh[0], vh[1]);
                        mma(c, ph[0], pm[0], ph[1], pm[1], vm[0], vm[1]);
                        mma(c, ph[0], pm[0], ph[1], pm[1], vh[0], vh[1]);
                        o[i] = add2(o[i], add2(make_float2(c[0], c[1]), make_float2(c[2], c[3])));
                    }
                }
                __syncwarp();                        // the stage may be refilled by the next load
                if (++stage == STAGES) {
                    stage = 0;
                    parity ^= 1;
                }
            }

            // ---- this block's part of the item is complete: join the warps ----------------------
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            float *mine = red + (warp * EX_QROWS + g) * EX_D + 2 * t;
#pragma unroll
            for (int i = 0; i < 16; ++i) *reinterpret_cast<float2 *>(mine + 8 * i) = o[i];
            if (t == 0) {
                red_m[warp * EX_QROWS + g] = m;
                red_l[warp * EX_QROWS + g] = l;
            }
            __syncthreads();
            // Whole items end here; parts leave a record. A record's place: the block's, 0 where
            // the item began before it and 1 where it goes on behind it, or (whole, but joined with
            // other records or weights) the item's.
            const bool whole = a.by_items || (w.s0 == 0 && w.s1 == it.weight);
            const bool finish = a.by_items || (whole && !MASS && !a.shared_here && !a.nsp);
            long long slot = 2LL * blockIdx.x + (w.s0 == 0 ? 1 : 0);
            if (whole) {
                const int RT = ex_shared_span(a, RS).RT;
                slot = 2LL * a.grid + (it.b < 0 ? it.h * RT + it.rt : a.H * RT + it.b * a.H + it.h);
            }
            for (int e = threadIdx.x; e < EX_QROWS * EX_D / 4; e += 32 * W) {
                const int r = e / (EX_D / 4), d = (e % (EX_D / 4)) * 4;
                float M = -CUDART_INF_F;
#pragma unroll
                for (int x = 0; x < W; ++x) M = fmaxf(M, red_m[x * EX_QROWS + r]);
                const float ref = M == -CUDART_INF_F ? 0.f : M;
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < W; ++x) {
                    const float f = ex2(red_m[x * EX_QROWS + r] - ref);
                    const float4 y = *reinterpret_cast<const float4 *>(
                        red + (x * EX_QROWS + r) * EX_D + d);
                    L += f * red_l[x * EX_QROWS + r];
                    acc.x += f * y.x;
                    acc.y += f * y.y;
                    acc.z += f * y.z;
                    acc.w += f * y.w;
                }
                if (finish) {
                    // the sum replaces warp 0's part, which this thread alone reads
                    *reinterpret_cast<float4 *>(red + r * EX_D + d) = acc;
                    if (d == 0) {
                        sum_m[r] = M;
                        sum_l[r] = L;
                    }
                } else {
                    float *rec = a.rec + slot * EX_REC;
                    if (d == 0) {
                        rec[r] = M;
                        rec[EX_QROWS + r] = L;
                    }
                    *reinterpret_cast<float4 *>(rec + 2 * EX_QROWS + r * EX_D + d) = acc;
                }
            }
            __syncthreads();
            if (finish) {
                if (a.cluster > 1) cluster_sync();
                if (a.nsp) asm volatile("griddepcontrol.wait;" ::: "memory");
                const int c = a.by_items ? a.cluster : 1;
                const uint32_t red_a = smem_u32(red), m_a = smem_u32(sum_m), l_a = smem_u32(sum_l);
                constexpr int E = EX_QROWS * EX_D / 4;
                // the cluster's blocks share out the outputs
                for (int e = E * rank / c + threadIdx.x; e < E * (rank + 1) / c; e += 32 * W) {
                    const int r = e / (EX_D / 4), d = (e % (EX_D / 4)) * 4;
                    const int tk = it.i0 + r / a.G, hd = r % a.G;
                    if (r / a.G >= ex_tpt(a.G) || tk >= it.i1) continue;
                    float M = -CUDART_INF_F;
                    for (int x = 0; x < c; ++x) M = fmaxf(M, ldc1(map_rank(m_a + r * 4, c > 1 ? x : rank)));
                    const long long pre = (long long)it.h * a.nsp * a.B * a.G + (long long)it.b * a.G + r;
                    const long long pre_st = (long long)a.B * a.G;
                    for (int x = 0; x < a.nsp; ++x)
                        M = fmaxf(M, __ldcg(a.pre_ml + 2 * (pre + x * pre_st)));
                    const float ref = M == -CUDART_INF_F ? 0.f : M;
                    float L = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    auto add = [&](float m_, float l_, const float4 &y) {
                        const float f = ex2(m_ - ref);
                        L += f * l_;
                        acc.x += f * y.x;
                        acc.y += f * y.y;
                        acc.z += f * y.z;
                        acc.w += f * y.w;
                    };
                    for (int x = 0; x < c; ++x) {
                        const int rk = c > 1 ? x : rank;
                        add(ldc1(map_rank(m_a + r * 4, rk)), ldc1(map_rank(l_a + r * 4, rk)),
                            ldc4(map_rank(red_a + (r * EX_D + d) * 4, rk)));
                    }
#pragma unroll 4
                    for (int x = 0; x < a.nsp; ++x) {
                        const long long at = pre + x * pre_st;
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.pre_ml + 2 * at));
                        add(ml.x, ml.y,
                            __ldcg(reinterpret_cast<const float4 *>(a.pre_o + at * EX_D + d)));
                    }
                    const float inv = inverse(L);
                    char *op = a.out + it.b * a.o_seq + (it.h * a.G + hd) * a.o_head + tk * a.o_tok;
                    if constexpr (F32IO)
                        *reinterpret_cast<float4 *>(op + d * 4) =
                            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                    else
                        *reinterpret_cast<uint2 *>(op + d * 2) =
                            make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
                }
                if constexpr (MASS) {
                    // every block of the cluster adds the weights of the rows whose scores it has
                    float ref[EX_QROWS], inv[EX_QROWS];
                    const float *sc[EX_QROWS];
#pragma unroll
                    for (int r = 0; r < EX_QROWS; ++r) {
                        if (r >= a.G) break;
                        float M = -CUDART_INF_F, L = 0.f;
                        for (int x = 0; x < c; ++x)
                            M = fmaxf(M, ldc1(map_rank(m_a + r * 4, c > 1 ? x : rank)));
                        ref[r] = M == -CUDART_INF_F ? 0.f : M;
                        for (int x = 0; x < c; ++x)
                            L += ex2(ldc1(map_rank(m_a + r * 4, c > 1 ? x : rank)) - ref[r]) *
                                 ldc1(map_rank(l_a + r * 4, c > 1 ? x : rank));
                        inv[r] = inverse(L);
                        sc[r] = a.scores + (((long long)it.b * a.H + it.h) * a.G + r) * a.score_st;
                    }
                    const long long base = ((long long)it.b * a.H + it.h) * a.rows;
                    const int hi = min(it.C, w.s1 * RS);
                    for (int j = w.s0 * RS + threadIdx.x; j < hi; j += 32 * W) {
                        float x = 0.f;
#pragma unroll
                        for (int r = 0; r < EX_QROWS; ++r) {
                            if (r >= a.G) break;
                            x += ex2(sc[r][j] - ref[r]) * inv[r];
                        }
                        a.mass_out[base + j] = a.mass[base + j] + x;
                    }
                }
                __syncthreads();
                if (a.cluster > 1) cluster_sync();   // its records have been read
            }
            have = w.next(a, rank);
        }
        if (late) {
            // copies still in flight end before the block does (bounded)
            atomicExch(&g_split_status, 1);
            for (int i = max(0, ld_count - STAGES); i < ld_count; ++i)
                wait_for(bar + (i % STAGES) * 8, (i / STAGES) & 1);
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

template <bool F32ROWS, bool F32IO, bool MASS>
__global__ void __launch_bounds__(MERGE_T)
exact_merge_kernel(const __grid_constant__ ExactArgs a, int rt_max, int mass_blocks) {
    constexpr int RS = ex_step_rows(F32ROWS);
    __shared__ float wgt[EX_QROWS][EX_MAXREC];
    __shared__ int slot_of[EX_MAXREC];
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
    const ExactSpan sp = ex_seq_span(a, n, ql, RS), sh = ex_shared_span(a, RS);
    if (rt >= sp.RT || (mass_block && chunk * MASS_ROWS >= n)) return;
    const unsigned length = ex_length(a, a.B, RS);
    const unsigned per = (length + a.grid - 1) / a.grid;
    const unsigned first = ex_length(a, b, RS) + ((unsigned)h * sp.RT + rt) * sp.S;
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
    const int whole0 = 2 * a.grid;
    for (int i = threadIdx.x; i < n_own + n_sh; i += MERGE_T) {
        if (i < n_own)
            slot_of[i] = n_own == 1 ? whole0 + a.H * sh.RT + b * a.H + h
                                    : 2 * (own_c0 + i) + (i == 0 ? 1 : 0);
        else
            slot_of[i] = n_sh == 1 ? whole0 + h * sh.RT + sh_rt
                                   : 2 * (sh_c0 + i - n_own) + (i == n_own ? 1 : 0);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    const int rows = min(tpt, ql - rt * tpt) * a.G;              // live rows of the tile
    auto ml = [&](int i, int r, float &m_, float &l_) {
        if (i < n_own + n_sh) {
            const float *rec = a.rec + (long long)slot_of[i] * EX_REC;
            const int rr = i < n_own ? r : sh_row + r;
            m_ = rec[rr];
            l_ = rec[EX_QROWS + rr];
        } else {
            const float *x = a.pre_ml + 2 * (((long long)h * a.nsp + (i - n_own - n_sh)) * a.B * a.G +
                                             (long long)b * a.G + r);
            m_ = x[0];
            l_ = x[1];
        }
    };
    // a warp per row: M = max m_i, weights 2^(m_i - M), L = sum of weight x l_i
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < rows) {
        float M = -CUDART_INF_F;
        for (int i = lane; i < nrec; i += 32) {
            float m_, l_;
            ml(i, warp, m_, l_);
            wgt[warp][i] = m_;
            M = fmaxf(M, m_);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float ref = M == -CUDART_INF_F ? 0.f : M;
        float L = 0.f;
        for (int i = lane; i < nrec; i += 32) {
            float m_, l_;
            ml(i, warp, m_, l_);
            const float f = ex2(wgt[warp][i] - ref);
            wgt[warp][i] = f;
            L += f * l_;
        }
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
    if (y < reps) {
#pragma unroll 4
        for (int i = y; i < nrec; i += reps) {
            const float *src;
            if (i < n_own + n_sh)
                src = a.rec + (long long)slot_of[i] * EX_REC + 2 * EX_QROWS +
                      (i < n_own ? r : sh_row + r) * EX_D + d;
            else
                src = a.pre_o + (((long long)h * a.nsp + (i - n_own - n_sh)) * a.B * a.G +
                                 (long long)b * a.G + r) * EX_D + d;
            const float4 v = *reinterpret_cast<const float4 *>(src);
            const float f = wgt[r][i];
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
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

template <bool F32ROWS>
constexpr size_t split_smem() {
    constexpr int W = ex_warps(F32ROWS);
    return W * STAGES * 2 * 16 * (F32ROWS ? 512 : 256) + W * EX_QROWS * (EX_D + 2) * 4 +
           2 * EX_QROWS * 4 + W * STAGES * 8;
}
static_assert(split_smem<false>() <= 227 * 1024 && split_smem<true>() <= 227 * 1024, "shared memory");

template <bool F32ROWS, bool F32IO, bool MASS>
void config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *at, int grid, int cluster, bool after) {
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * ex_warps(F32ROWS));
    cfg.dynamicSmemBytes = split_smem<F32ROWS>();
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
    const size_t bytes = split_smem<F32ROWS>();
    static std::atomic<unsigned long long> set{0};   // devices whose attribute is set
    const cudaError_t e = once_per_device(set, reinterpret_cast<const void *>(kern), (int)bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    config<F32ROWS, F32IO, MASS>(cfg, at, a.grid, a.cluster, a.after);
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
    if (once_per_device(set, reinterpret_cast<const void *>(kern), (int)split_smem<false>()) !=
        cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    config<false, true, false>(cfg, at, cluster, cluster, false);
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
