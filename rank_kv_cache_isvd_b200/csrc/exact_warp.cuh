// Eight query rows of one warp against 8 KB of key rows and of value rows in shared memory: 32 bf16
// or 16 float32 rows, as [128-byte part][row][128 bytes], 16-byte chunks permuted by row (TMA's
// 128-byte swizzle). Used by the split kernel and the rows kernel.
//
// Products run on mma.sync: 8 query rows fill half of its 16 rows, and tcgen05 would want 64 or 128.
// - bf16 rows (m16n8k16, bf16): float32 queries are split in three bf16 terms (24 bits), x = hi + mid
//   + lo: hi sits in rows 0-7 of the A operand and mid in rows 8-15, so one instruction does both terms
//   and both sums land in one thread; lo takes a second one. The weights p likewise, so that float32
//   outputs keep float32 accuracy (a weight rounded to bf16 would cost up to 2^-8); for bf16 outputs their
//   first two terms are used, which cost no more than one.
// - float32 rows (m16n8k8, tf32): every operand is split in two tf32 terms (22 bits), the queries' and
//   weights' in rows 0-7 and 8-15: (hi | lo) x hi and (hi | 0) x lo. Three bf16 terms took half as many
//   instructions again, most of them for the splitting.
//
// Tensor cores truncate where they add, always toward zero: over the hundred steps of a long cache
// outputs lost 4e-6. So products start from zero every step (keys of float32 rows: every 32 channels)
// and are added in float32 arithmetic (round to nearest), smallest terms first: 8e-7 at 8 x 32768 rows.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "exact.cuh"
#include "tc_util.cuh"

namespace iskv {

constexpr int UNIT = 8192;             // bytes of keys or values per warp and step

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
// c += A B, bf16: A 16 x 16, B 16 x 8. This thread's A registers: row lane/4 (a0, a2) and row
// lane/4 + 8 (a1, a3), columns 2 (lane%4) + {0, 1} (a0, a1) and + 8 (a2, a3).
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
// The same in tf32: A 16 x 8, B 8 x 8; columns lane%4 (a0, a1) and + 4 (a2, a3).
__device__ __forceinline__ void mma_tf(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0_tf(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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
// x = sum of two tf32: the first rounded by integer arithmetic (the conversion instruction runs at a
// quarter of its rate), the second the exact rest, of which the product reads the upper 11 bits.
__device__ __forceinline__ void split_tf(float x, uint32_t &h, uint32_t &l) {
    h = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    l = __float_as_uint(x - __uint_as_float(h));
}
__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); }

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int row, int head,
                                            int seq, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(head), "r"(seq), "r"(bar)
        : "memory");
}
// L2's policy for rows. A decode reads a sequence's own rows once: they leave L2 first, before scores and
// records, which are read twice (weights of 8 x 32768 rows: 187 -> 183 us, window of 4 x 65536: 19.1 -> 18.8),
// and before a shared prefix, which the next call reads again (130 sequences behind a prefix of 4001:
// 67.5 -> 61.2 us). The prefix itself stays as long as it can: with its rows first out as well, two sequences of
// 8192 rows behind a prefix of 16384 took 40.7 us instead of 35.1.
__device__ __forceinline__ uint64_t l2_policy(bool once) {
    uint64_t p;
    if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int row, int head, int seq,
                                            uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(head), "r"(seq), "r"(bar),
        "l"(policy)
        : "memory");
}
// False: the wait gave up.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, uint32_t polls) {
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(EX_SUSPEND_NS)
            : "memory");
        if (done) return true;
    }
    return false;
}

template <bool F32ROWS, bool F32IO>
struct WarpRows {
    static constexpr int WR = ex_warp_rows(F32ROWS);
    static constexpr int NT = WR / 8;                // groups of 8 rows: columns of a product S
    static constexpr int PARTS = F32ROWS ? 4 : 2;    // 128-byte parts of a row
    static constexpr int PART = UNIT / PARTS;
    static constexpr int QT = F32ROWS ? 16 : 8;      // steps of a product over the channels

    // query terms (float32 rows: the queries, split at each use: their terms would not fit)
    uint32_t qa[QT][2], qb[F32IO && !F32ROWS ? QT : 1][2], qc[F32IO && !F32ROWS ? QT : 1][2];
    float2 o[16];                                    // this lane: channels 8 i + 2 t + {0, 1} of row g
    float m, l;                                      // reference and this lane's part of the sum
    uint32_t pa[NT][2], pb[NT][2], pc[F32IO && !F32ROWS ? NT : 1];   // weight terms
    int g, t;
    uint32_t k_at, v_at;                             // fragment offsets in a part (bf16)

    __device__ __forceinline__ void init() {
        const int lane = threadIdx.x & 31, kr = (lane & 7) + ((lane >> 4) << 3), vr = lane & 15;
        g = lane >> 2;
        t = lane & 3;
        k_at = kr * 128 + ((((lane >> 3) & 1) ^ (kr & 7)) << 4);
        v_at = vr * 128 + (((lane >> 4) ^ (vr & 7)) << 4);
    }
    // Row g's query (zeros where it is not live), empty sums.
    __device__ __forceinline__ void begin(const char *q, bool live) {
#pragma unroll
        for (int ks = 0; ks < QT; ++ks) {
            if constexpr (F32ROWS) {
                // channels 8 ks + 2 t and + 1 take the places t and t + 4 of the 8
                float2 f = make_float2(0.f, 0.f);
                if (live) f = *reinterpret_cast<const float2 *>(q + (ks * 8 + 2 * t) * 4);
                qa[ks][0] = __float_as_uint(f.x);
                qa[ks][1] = __float_as_uint(f.y);
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int d = ks * 16 + x * 8 + 2 * t;
                    if constexpr (F32IO) {
                        float2 f = make_float2(0.f, 0.f);
                        if (live) f = *reinterpret_cast<const float2 *>(q + d * 4);
                        split3(f.x, f.y, qa[ks][x], qb[ks][x], qc[ks][x]);
                    } else {
                        qa[ks][x] = live ? *reinterpret_cast<const uint32_t *>(q + d * 2) : 0u;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = make_float2(0.f, 0.f);
        m = -CUDART_INF_F;
        l = 0.f;
    }
    // Unscaled scores of row g at rows 8 nt + 2 t + x of the keys at `k`.
    __device__ __forceinline__ void scores(uint32_t k, float (&s)[NT][2]) {
        if constexpr (!F32ROWS) {
            // two chains of products per 8 rows, so that few wait on one another
            float c[NT][4], e[F32IO ? NT : 1][4];
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int np = 0; np < NT / 2; ++np) {
                    uint32_t kb[4];
                    ldsm4(k + (ks >> 2) * PART + np * 2048 + (k_at ^ ((ks & 3) << 5)), kb);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int nt = 2 * np + y;
                        const uint32_t b0 = kb[2 * y], b1 = kb[2 * y + 1];
                        if constexpr (F32IO) {
                            if (ks == 0) {
                                mma0(e[nt], qc[ks][0], 0u, qc[ks][1], 0u, b0, b1);
                                mma0(c[nt], qa[ks][0], qb[ks][0], qa[ks][1], qb[ks][1], b0, b1);
                            } else {
                                mma(e[nt], qc[ks][0], 0u, qc[ks][1], 0u, b0, b1);
                                mma(c[nt], qa[ks][0], qb[ks][0], qa[ks][1], qb[ks][1], b0, b1);
                            }
                        } else {
                            if (ks == 0) mma0(c[nt], qa[ks][0], 0u, qa[ks][1], 0u, b0, b1);
                            else mma(c[nt], qa[ks][0], 0u, qa[ks][1], 0u, b0, b1);
                        }
                    }
                }
            // rows 8-15 hold the mid terms' sums
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    s[nt][x] = F32IO ? (e[nt][x] + c[nt][2 + x]) + c[nt][x] : c[nt][x];
        } else {
            float e[NT][4];                          // hi x lo
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = 0.f;
#pragma unroll
            for (int kp = 0; kp < 4; ++kp) {
                float c[NT][4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int ks = 4 * kp + y;
                    uint32_t q0, q1, r0, r1;
                    split_tf(__uint_as_float(qa[ks][0]), q0, r0);
                    split_tf(__uint_as_float(qa[ks][1]), q1, r1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int r = nt * 8 + g;
                        const float2 f = lds2(k + kp * PART + r * 128 +
                                              (((2 * y + (t >> 1)) ^ (r & 7)) << 4) + (t & 1) * 8);
                        uint32_t h0, l0, h1, l1;
                        split_tf(f.x, h0, l0);
                        split_tf(f.y, h1, l1);
                        if (ks == 0) mma0_tf(e[nt], q0, 0u, q1, 0u, l0, l1);
                        else mma_tf(e[nt], q0, 0u, q1, 0u, l0, l1);
                        if (y == 0) mma0_tf(c[nt], q0, r0, q1, r1, h0, h1);
                        else mma_tf(c[nt], q0, r0, q1, r1, h0, h1);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) s[nt][x] += c[nt][2 + x] + c[nt][x];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) s[nt][x] += e[nt][x];
        }
    }
    // Weights of scores in log2 units (-inf where not seen), and the sums so far brought to the same
    // reference. It moves only when a score passes it by 2^8: weights stay below 256, and the sums
    // keep their float32 accuracy.
    __device__ __forceinline__ void weights(const float (&s)[NT][2]) {
        float top = -CUDART_INF_F;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top = fmaxf(top, fmaxf(s[nt][0], s[nt][1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
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
        float add = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float x = ex2(s[nt][0] - ref), y = ex2(s[nt][1] - ref);
            add += x + y;
            if constexpr (F32ROWS) {
                split_tf(x, pa[nt][0], pb[nt][0]);
                split_tf(y, pa[nt][1], pb[nt][1]);
            } else {
                uint32_t c;
                split3(x, y, pa[nt][0], pb[nt][0], c);
                if constexpr (F32IO) pc[nt] = c;
            }
        }
        l += add;
    }
    // o += weights x the values at `v`.
    __device__ __forceinline__ void values(uint32_t v) {
        if constexpr (!F32ROWS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t vb[NT / 2][4];
#pragma unroll
                for (int kp = 0; kp < NT / 2; ++kp)
                    ldsm4t(v + (i >> 2) * PART + kp * 2048 + (v_at ^ ((i & 3) << 5)), vb[kp]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float c[4];
                    if constexpr (F32IO) {
#pragma unroll
                        for (int kp = 0; kp < NT / 2; ++kp) {
                            const uint32_t b0 = vb[kp][2 * x], b1 = vb[kp][2 * x + 1];
                            if (kp == 0) mma0(c, pc[0], 0u, pc[1], 0u, b0, b1);
                            else mma(c, pc[2 * kp], 0u, pc[2 * kp + 1], 0u, b0, b1);
                        }
                    }
#pragma unroll
                    for (int kp = 0; kp < NT / 2; ++kp) {
                        const uint32_t b0 = vb[kp][2 * x], b1 = vb[kp][2 * x + 1];
                        const int y = 2 * kp;
                        if (kp == 0 && !F32IO) mma0(c, pa[0][0], pb[0][0], pa[1][0], pb[1][0], b0, b1);
                        else mma(c, pa[y][0], pb[y][0], pa[y + 1][0], pb[y + 1][0], b0, b1);
                    }
                    o[2 * i + x] =
                        add2(o[2 * i + x], add2(make_float2(c[2], c[3]), make_float2(c[0], c[1])));
                }
            }
        } else {
            // rows 8 nt + 2 t and + 1 take the places t and t + 4 of the 8
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint32_t h[NT][2], w[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int r = 8 * nt + 2 * t + y;
                        const float f = lds1(v + (i >> 2) * PART + r * 128 +
                                             ((((i & 3) * 2 + (g >> 2)) ^ (r & 7)) << 4) + (g & 3) * 4);
                        split_tf(f, h[nt][y], w[nt][y]);
                    }
                float c[4];
                mma0_tf(c, pa[0][0], 0u, pa[0][1], 0u, w[0][0], w[0][1]);
#pragma unroll
                for (int nt = 1; nt < NT; ++nt)
                    mma_tf(c, pa[nt][0], 0u, pa[nt][1], 0u, w[nt][0], w[nt][1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_tf(c, pa[nt][0], pb[nt][0], pa[nt][1], pb[nt][1], h[nt][0], h[nt][1]);
                o[i] = add2(o[i], add2(make_float2(c[2], c[3]), make_float2(c[0], c[1])));
            }
        }
    }
    // Sum of the four lanes of a row.
    __device__ __forceinline__ float sum() const {
        float x = l + __shfl_xor_sync(0xffffffffu, l, 1);
        return x + __shfl_xor_sync(0xffffffffu, x, 2);
    }
    // Values of rows from `seen` (0 .. WR) on become zeros: rows that nobody sees may be anything, and
    // 0 x NaN would reach o. By the whole warp.
    static __device__ __forceinline__ void clear(uint32_t v, int seen) {
        const int lane = threadIdx.x & 31;
        for (int r = max(seen, 0); r < WR; ++r)
            if (lane < 8 * PARTS)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 v + (lane >> 3) * PART + r * 128 + (lane & 7) * 16),
                             "r"(0)
                             : "memory");
        fence_proxy_async_smem();
        __syncwarp();
    }
};

}  // namespace iskv
