// Attention of few query rows over many exact KV rows, and the merge of its splits.
//
//   o_q = sum_j p_qj v_j / sum_j p_qj,   p_qj = 2^(s_qj - m_q),   s_qj = q . k_j log2(e)/sqrt(128)
//
// Decode reads every visible key and value once and does 4 G flops per byte pair: it is bound by
// HBM. So the layout serves the loads. A warp owns 16 rows of a step at a time and a ring of
// three such stages in shared memory, filled by its own cp.async: no barrier joins the warps until
// the end of an item, and about 128 KB per SM are in flight. Rows that no query of the tile sees
// are never read (zero-filled), whatever they hold.
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
// The flat space of (item, step) is cut into equal ranges, one per block, so that sequences of any
// lengths fill the GPU evenly. An item that several blocks share leaves one record per block,
// which the merge kernel joins: o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
#include <math_constants.h>

#include <atomic>

#include "exact.cuh"

namespace iskv {
namespace {

constexpr int STAGES = 3;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes global -> shared, or 16 zero bytes where `bytes` is 0 (src is not read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
// c += A B with A = 16 x 16, B = 16 x 8, bf16. This thread's A registers: row lane/4 (a0, a2) and
// row lane/4 + 8 (a1, a3), columns 2 (lane%4) + {0, 1} (a0, a1) and + 8 (a2, a3).
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float lo_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
// (x, y) = sum of three pairs of bf16, each the rounding of what the ones before leave. A value
// that is not finite stays in the first term alone (inf - inf would make it NaN).
__device__ __forceinline__ void split3(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack(x, y);
    float rx = x - lo_of(h), ry = y - hi_of(h);
    rx = fabsf(x) <= 3.3895313e38f ? rx : 0.f;
    ry = fabsf(y) <= 3.3895313e38f ? ry : 0.f;
    m = pack(rx, ry);
    l = pack(rx - lo_of(m), ry - hi_of(m));
}

// Where an item's rows and queries are. Row c of its C visible rows: c < sk ? c : c - sk + lo.
struct Item {
    long long first;      // flat step of its step 0
    int b, h, rt;         // b < 0: shared prefix
    int S;
    int n, ql;            // of sequence b
    int C, sk, lo;
    int i0, i1;           // its tokens (sequences, for the shared prefix)
    const char *k, *v;
    long long row_st;
};

__device__ __forceinline__ void geometry(const ExactArgs &a, Item &it) {
    const int tpt = ex_tpt(a.G);
    it.i0 = it.rt * tpt;
    if (it.b < 0) {
        it.i1 = min(it.i0 + tpt, a.B);
        it.C = it.sk = a.P;
        it.lo = 0;
        it.k = a.pk + it.h * a.p_head;
        it.v = a.pv + it.h * a.p_head;
        it.row_st = a.p_row;
        return;
    }
    it.i1 = min(it.i0 + tpt, it.ql);
    const int p0 = it.n - it.ql + it.i0;
    const int hi = max(0, it.n - it.ql + it.i1);
    it.sk = min(a.sinks, hi);
    it.lo = max(it.sk, p0 - a.window + 1);
    it.C = it.sk + max(0, hi - it.lo);
    it.k = a.k + it.b * a.seq_st + it.h * a.head_st;
    it.v = a.v + it.b * a.seq_st + it.h * a.head_st;
    it.row_st = a.row_st;
}

// The item after `it`: next tile, next kv-head, next sequence with tokens. It must exist.
template <int RS>
__device__ __forceinline__ void next_item(const ExactArgs &a, Item &it) {
    it.first += it.S;
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
            it.S = s.S;
        }
    }
    geometry(a, it);
}

// The item that flat step g belongs to (g < total).
template <int RS>
__device__ __forceinline__ Item find_item(const ExactArgs &a, long long g) {
    Item it;
    const int lane = threadIdx.x & 31;
    const ExactSpan p = ex_shared_span(a, RS);
    const long long shared = (long long)a.H * p.RT * p.S;
    long long at = shared;
    int RT = p.RT;
    if (g < shared) {
        it.b = -1;
        it.S = p.S;
        it.n = it.ql = 0;
        at = 0;
    } else if (!a.lens && !a.q_lens) {
        const ExactSpan s = ex_seq_span(a, a.rows, a.m, RS);
        const long long each = (long long)a.H * s.RT * s.S;
        it.b = (int)((g - at) / each);
        at += it.b * each;
        it.n = a.rows;
        it.ql = a.m;
        it.S = s.S;
        RT = s.RT;
    } else {
        it.b = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            long long steps = 0;
            if (b < a.B) {
                const ExactSpan s = ex_seq_span(a, ex_len(a, b), ex_qlen(a, b), RS);
                steps = (long long)a.H * s.RT * s.S;
            }
            long long sum = steps;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, at + sum > g);
            if (past) {
                const int l = __ffs(past) - 1;
                it.b = b0 + l;
                at += __shfl_sync(0xffffffffu, sum - steps, l);
                break;
            }
            at += __shfl_sync(0xffffffffu, sum, 31);
        }
        it.n = ex_len(a, it.b);
        it.ql = ex_qlen(a, it.b);
        const ExactSpan s = ex_seq_span(a, it.n, it.ql, RS);
        it.S = s.S;
        RT = s.RT;
    }
    const long long i = (g - at) / it.S;
    it.h = (int)(i / RT);
    it.rt = (int)(i - (long long)it.h * RT);
    it.first = at + i * it.S;
    geometry(a, it);
    return it;
}

template <bool F32ROWS, bool F32IO, bool MASS>
__global__ void __launch_bounds__(32 * ex_warps(F32ROWS), 1) exact_split_kernel(ExactArgs a) {
    constexpr int W = ex_warps(F32ROWS);
    constexpr int RS = ex_step_rows(F32ROWS);
    constexpr int RB = F32ROWS ? 512 : 256;          // bytes of a row
    constexpr int CH = RB / 16;                      // its 16-byte chunks
    constexpr int STAGE = 2 * 16 * RB;               // K rows, then V rows
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * STAGES * STAGE;
    float *red = reinterpret_cast<float *>(smem + W * STAGES * STAGE);   // [W][8][128]
    float *red_m = red + W * EX_QROWS * EX_D, *red_l = red_m + W * EX_QROWS;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long total = ex_total(a, RS);
    const long long per = (total + a.grid - 1) / a.grid;
    const long long g0 = blockIdx.x * per, g1 = min(total, g0 + per);
    if (g0 >= g1) {
        if (a.after) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }

    Item it = find_item<RS>(a, g0), nx = it;
    long long at = g0, ahead = g0;                   // flat steps: computed, loaded
    int ahead_stage = 0;

    auto load = [&]() {
        if (ahead < g1) {
            if (ahead >= nx.first + nx.S) next_item<RS>(a, nx);
            const int c0 = (int)(ahead - nx.first) * RS + warp * 16;
            if (c0 < nx.C) {
                uint8_t *st = ring + ahead_stage * STAGE;
                constexpr int STEPS = 16 * CH / 32;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int r = F32ROWS ? i : 2 * i + (lane >> 4);
                    const int ch = lane & (CH - 1);
                    const int c = c0 + r;
                    const int row = c < nx.sk ? c : c - nx.sk + nx.lo;
                    const bool in = c < nx.C;
                    const long long off = in ? row * nx.row_st + ch * 16 : 0;
                    // chunks permuted by row, so that the fragment reads below meet no conflicts
                    const int kc = F32ROWS ? ch ^ ((r & 7) << 1) : ch ^ (r & 7);
                    const int vc = F32ROWS ? ch ^ ((((r >> 1) & 3) | ((r & 1) << 2)) << 1)
                                           : ch ^ (r & 7);
                    cp_async16(smem_addr(st + r * RB + kc * 16), nx.k + off, in ? 16u : 0u);
                    cp_async16(smem_addr(st + (16 + r) * RB + vc * 16), nx.v + off, in ? 16u : 0u);
                }
            }
            ++ahead;
            ahead_stage = ahead_stage + 1 == STAGES ? 0 : ahead_stage + 1;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load();

    int stage = 0;
    bool fresh = true;                               // a new item begins: its queries are read
    long long seg0 = at;
    uint32_t qh[8][2], qm[F32IO ? 8 : 1][2], ql[F32IO ? 8 : 1][2];
    float o[16][2];
    float m = -CUDART_INF_F, l = 0.f;
    int pos = 0;                                     // position of this lane's query row
    const int tok = g / a.G, head = g - tok * a.G;
    while (at < g1) {
        load();
        if (fresh) {
            fresh = false;
            seg0 = at;
            const int i = it.i0 + tok;
            const bool live = i < it.i1;
            pos = it.n - it.ql + i;
            const char *qp = a.q;
            if (live)
                qp += (it.b < 0 ? i : it.b) * a.q_seq + (it.h * a.G + head) * a.q_head +
                      (it.b < 0 ? 0 : i) * a.q_tok;
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
            for (int i2 = 0; i2 < 16; ++i2) o[i2][0] = o[i2][1] = 0.f;
            m = -CUDART_INF_F;
            l = 0.f;
        }
        cp_wait<STAGES - 1>();
        __syncwarp();
        const int c0 = (int)(at - it.first) * RS + warp * 16;
        if (c0 < it.C) {
            const uint8_t *ks_ = ring + stage * STAGE, *vs_ = ks_ + 16 * RB;
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            if constexpr (!F32ROWS) {
                const int r = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t kb[4];
                    ldsm4(smem_addr(ks_ + r * RB + (((2 * ks + cc) ^ (r & 7)) * 16)), kb);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        if constexpr (F32IO) {
                            mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], kb[2 * nt],
                                kb[2 * nt + 1]);
                            mma(s[nt], ql[ks][0], 0u, ql[ks][1], 0u, kb[2 * nt], kb[2 * nt + 1]);
                        } else {
                            mma(s[nt], qh[ks][0], 0u, qh[ks][1], 0u, kb[2 * nt], kb[2 * nt + 1]);
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
                            const int ch = (4 * ks + 2 * x + (t >> 1)) ^ ((r & 7) << 1);
                            const float2 f = *reinterpret_cast<const float2 *>(
                                ks_ + r * RB + ch * 16 + (t & 1) * 8);
                            split3(f.x, f.y, kh[x], km[x], kl[x]);
                        }
                        mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], kh[0], kh[1]);
                        mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], km[0], km[1]);
                        mma(s[nt], qh[ks][0], qm[ks][0], qh[ks][1], qm[ks][1], kl[0], kl[1]);
                        mma(s[nt], ql[ks][0], 0u, ql[ks][1], 0u, kh[0], kh[1]);
                    }
            }
            // scores of row g at columns c0 + 8 nt + 2 t + x (rows 8-15 hold the mid terms' sums)
            float p[2][2];
            float top = -CUDART_INF_F;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int c = c0 + 8 * nt + 2 * t + x;
                    const int row = c < it.sk ? c : c - it.sk + it.lo;
                    const bool see = c < it.C && (it.b < 0 || (row <= pos && (row < a.sinks ||
                                                                  row > pos - a.window)));
                    p[nt][x] = see ? (s[nt][x] + s[nt][2 + x]) * a.scale_log2 : -CUDART_INF_F;
                    top = fmaxf(top, p[nt][x]);
                }
            if constexpr (MASS) {
                if (g < a.G) {
                    float *sc = a.scores + (((long long)it.b * a.H + it.h) * a.G + g) * a.score_st +
                                c0 + 2 * t;
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
                for (int i = 0; i < 16; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) o[i][x] *= f;
            }
            const float ref = m == -CUDART_INF_F ? 0.f : m;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    p[nt][x] = ex2(p[nt][x] - ref);
                    l += p[nt][x];
                }
            uint32_t ph[2], pm[2], pl[2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) split3(p[nt][0], p[nt][1], ph[nt], pm[nt], pl[nt]);
            if constexpr (!F32ROWS) {
                const int r = lane & 15, cc = lane >> 4;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t vb[4];
                    ldsm4t(smem_addr(vs_ + r * RB + (((2 * i + cc) ^ (r & 7)) * 16)), vb);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
                        if constexpr (F32IO)
                            mma(c, pl[0], 0u, pl[1], 0u, vb[2 * x], vb[2 * x + 1]);
                        mma(c, ph[0], pm[0], ph[1], pm[1], vb[2 * x], vb[2 * x + 1]);
                        o[2 * i + x][0] += c[0] + c[2];
                        o[2 * i + x][1] += c[1] + c[3];
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
                            const int ch = (2 * i + (g >> 2)) ^
                                           ((((r >> 1) & 3) | ((r & 1) << 2)) << 1);
                            f[y] = *reinterpret_cast<const float *>(vs_ + r * RB + ch * 16 +
                                                                    (g & 3) * 4);
                        }
                        split3(f[0], f[1], vh[x], vm[x], vl[x]);
                    }
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma(c, ph[0], pm[0], ph[1], pm[1], vl[0], vl[1]);
                    mma(c, pl[0], 0u, pl[1], 0u, vh[0], vh[1]);
                    mma(c, ph[0], pm[0], ph[1], pm[1], vm[0], vm[1]);
                    mma(c, ph[0], pm[0], ph[1], pm[1], vh[0], vh[1]);
                    o[i][0] += c[0] + c[2];
                    o[i][1] += c[1] + c[3];
                }
            }
        }
        __syncwarp();                                // the stage may be refilled by the next load
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        ++at;
        if (at < it.first + it.S && at < g1) continue;

        // ---- the item, or this block's part of it, ends: join the warps -------------------------
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        __syncthreads();                             // the last item's reads of `red` are done
        float *mine = red + (warp * EX_QROWS + g) * EX_D + 2 * t;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            *reinterpret_cast<float2 *>(mine + 8 * i) = make_float2(o[i][0], o[i][1]);
        if (t == 0) {
            red_m[warp * EX_QROWS + g] = m;
            red_l[warp * EX_QROWS + g] = l;
        }
        __syncthreads();
        const bool whole = seg0 == it.first && at == it.first + it.S;
        const long long slot = whole ? 2LL * a.grid + (it.b < 0 ? (long long)it.h * ex_shared_span(a, RS).RT + it.rt
                                                   : (a.shared_here ? (long long)a.H * ex_shared_span(a, RS).RT : 0LL) +
                                                         (long long)it.b * a.H + it.h)
                                     : 2LL * blockIdx.x + (seg0 == it.first ? 1 : 0);
        for (int e = threadIdx.x; e < EX_QROWS * EX_D / 4; e += 32 * W) {
            const int r = e / (EX_D / 4), d = (e % (EX_D / 4)) * 4;
            float M = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, red_m[w * EX_QROWS + r]);
            const float ref = M == -CUDART_INF_F ? 0.f : M;
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = ex2(red_m[w * EX_QROWS + r] - ref);
                const float4 x = *reinterpret_cast<const float4 *>(
                    red + (w * EX_QROWS + r) * EX_D + d);
                L += f * red_l[w * EX_QROWS + r];
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
            }
            if (whole && a.direct) {
                const int tk = it.i0 + r / a.G, hd = r % a.G;
                if (r / a.G < ex_tpt(a.G) && tk < it.i1) {
                    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
                    char *op = a.out + it.b * a.o_seq + (it.h * a.G + hd) * a.o_head + tk * a.o_tok;
                    if constexpr (F32IO)
                        *reinterpret_cast<float4 *>(op + d * 4) =
                            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                    else
                        *reinterpret_cast<uint2 *>(op + d * 2) =
                            make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
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
        fresh = true;
        if (at < g1) next_item<RS>(a, it);
    }
    cp_wait<0>();
    // the merge waits for this kernel alone: it must not end before the one that ran beside it
    if (a.after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- merge --------------------------------------------------------------------------------------
// Blocks 0 .. B*H*RTmax - 1 each join the records of one item (for the shared prefix: a sequence's
// own records with its rows of the prefix's). The blocks after them add the weights to `mass`.
constexpr int MERGE_T = 256;
constexpr int MASS_ROWS = 4 * MERGE_T;      // rows per mass block

struct RecList {
    long long first;      // flat step of the item
    int S;
};

template <bool F32ROWS, bool F32IO, bool MASS>
__global__ void __launch_bounds__(MERGE_T) exact_merge_kernel(ExactArgs a, int rt_max, int mass_blocks) {
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
    const long long total = ex_total(a, RS);
    const long long per = (total + a.grid - 1) / a.grid;
    const long long first = ex_first(a, b, RS) + ((long long)h * sp.RT + rt) * sp.S;
    const int own_c0 = (int)(first / per), own_c1 = (int)((first + sp.S - 1) / per);
    const int n_own = own_c1 - own_c0 + 1;
    if (a.direct && n_own == 1) return;              // the split kernel wrote it
    // shared prefix: tile and row of this sequence
    int n_sh = 0, sh_c0 = 0;
    const int sh_rt = b / tpt, sh_row = (b - sh_rt * tpt) * a.G;
    if (a.shared_here && sh.S) {
        const long long f = ((long long)h * sh.RT + sh_rt) * sh.S;
        sh_c0 = (int)(f / per);
        n_sh = (int)((f + sh.S - 1) / per) - sh_c0 + 1;
    }
    const int nrec = n_own + n_sh + a.nsp;
    const long long whole0 = 2LL * a.grid, shared_items = a.shared_here ? (long long)a.H * sh.RT : 0;
    for (int i = threadIdx.x; i < n_own + n_sh; i += MERGE_T) {
        long long s;
        if (i < n_own)
            s = n_own == 1 ? whole0 + shared_items + (long long)b * a.H + h
                           : 2LL * (own_c0 + i) + (i == 0 ? 1 : 0);
        else
            s = n_sh == 1 ? whole0 + (long long)h * sh.RT + sh_rt
                          : 2LL * (sh_c0 + i - n_own) + (i == n_own ? 1 : 0);
        slot_of[i] = (int)s;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    const int rows = (a.direct ? min(tpt, ql - rt * tpt) : 1) * a.G;     // live rows of the tile
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
        float inv[EX_QROWS];
        const float *sc[EX_QROWS];
        for (int gq = 0; gq < a.G; ++gq) {
            inv[gq] = row_l[gq] > 0.f ? 1.f / row_l[gq] : (row_l[gq] == 0.f ? 0.f : row_l[gq]);
            sc[gq] = a.scores + (((long long)b * a.H + h) * a.G + gq) * a.score_st;
        }
        const long long base = ((long long)b * a.H + h) * a.rows;
        for (int x = 0; x < MASS_ROWS / MERGE_T; ++x) {
            const int j = chunk * MASS_ROWS + x * MERGE_T + threadIdx.x;
            if (j >= n) break;
            float w = 0.f;
            for (int gq = 0; gq < a.G; ++gq) w += ex2(sc[gq][j] - row_m[gq]) * inv[gq];
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
        const float L = row_l[r];
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
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
    return W * STAGES * 2 * 16 * (F32ROWS ? 512 : 256) + W * EX_QROWS * (EX_D + 2) * 4;
}

template <bool F32ROWS, bool F32IO, bool MASS>
cudaError_t split(const ExactArgs &a, cudaStream_t s) {
    auto kern = exact_split_kernel<F32ROWS, F32IO, MASS>;
    const size_t bytes = split_smem<F32ROWS>();
    static std::atomic<unsigned long long> set{0};   // devices whose attribute is set
    const cudaError_t e = once_per_device(set, reinterpret_cast<const void *>(kern), (int)bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(32 * ex_warps(F32ROWS));
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = a.after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
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

cudaError_t launch_exact_split(const ExactArgs &a, bool f32_rows, bool f32_io, cudaStream_t s) {
    if (a.mass) {
        if (f32_rows) return split<true, true, true>(a, s);
        return f32_io ? split<false, true, true>(a, s) : split<false, false, true>(a, s);
    }
    if (f32_rows) return split<true, true, false>(a, s);
    return f32_io ? split<false, true, false>(a, s) : split<false, false, false>(a, s);
}

cudaError_t launch_exact_merge(const ExactArgs &a, bool f32_rows, bool f32_io, cudaStream_t s) {
    if (a.mass) {
        if (f32_rows) return merge<true, true, true>(a, s);
        return f32_io ? merge<false, true, true>(a, s) : merge<false, false, true>(a, s);
    }
    if (f32_rows) return merge<true, true, false>(a, s);
    return f32_io ? merge<false, true, false>(a, s) : merge<false, false, false>(a, s);
}

}  // namespace iskv
