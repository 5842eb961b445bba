// Attention of many query rows over exact rows on the tensor cores (tcgen05), for prompts, chunks of
// them, and a prefix that a batch shares.
//
//   S = Q K^T (128 query rows x 128 key rows),  P = 2^(S c - m),  O = O 2^(m_old - m) + P V
//
// with c = log2(e)/sqrt(128), one pass over the key blocks, m and the sum l of P per query row in
// registers. A tile's 128 query rows are tokens x the q-heads of one kv-head, so that the group
// shares every key block, and a window covers few blocks: 32 tokens per tile at a group of 4.
//
// One CTA of 384 threads per SM works on two tiles at once:
// - warp 0 loads Q once and then K and V blocks by TMA into a ring of five 32 KB stages;
// - warp 1 issues the products. S of tile i sits in tensor memory columns 128 i .. , its P (bf16)
//   overwrites the first half of them and is the A operand of P V; O sits in columns 256 + 128 i;
// - warps 4-7 and 8-11 are the softmax of tile 0 and of tile 1: a thread owns a query row, so
//   maxima and sums need no shuffles. While one group computes, the tensor cores work for the other;
//   P V of the first 64 keys of a block runs while the weights of the others are computed.
// (S in two buffers of 64 keys, so that the next S is complete when a softmax ends, was slower: with
// 64 columns the products read Q from shared memory at its full rate and take 50 cycles for the work
// of 32, and the tensor cores become the bound.)
//
// A prefix with no more rows than one tile is bound by HBM instead. There the two groups share the
// tile and take alternate blocks; their results join in shared memory at the end.
//
// m moves only when a row's maximum passes it by 2^8 (a power of two that P, O and l carry along
// exactly enough: P is at most 256). Moving it rescales O in tensor memory, which the softmax warp
// does itself: S of this block being complete says that the P V before it is too.
//
// P is rounded to bf16 (half a step, up to 2^-8 of a weight, at random over the keys): the product's
// operands are of one type, and a second term of P would be half as many products again for an error of the size
// that rounding the outputs makes anyway (2.1e-3 to 2.3e-3 against 64 bits, of which 1.6e-3 to 1.7e-3 are the
// outputs' own; the two errors are independent and of one size, so 1.41 times at most). The sum l takes the
// unrounded values, and all sums are float32.
//
// Every wait is bounded (iskv_exact_wait_limit). A wait that gives up sets the CTA's abort flag and the device's status
// word; all roles then leave their loops, copies in flight are waited for, and tensor memory is
// freed.
#include <math_constants.h>

#include <atomic>

#include "exact.cuh"
#include "exact_tile.cuh"
#include "tc_util.cuh"

namespace iskv {
namespace {

constexpr int TT = 384;
constexpr int NSTAGE = 5;
constexpr int BLOCK_BYTES = 128 * 256;       // 128 rows of 128 bf16: two halves of 64 channels
constexpr int HALF_BYTES = 128 * 128;

// setmaxnreg: 128 control threads and 256 softmax threads share what the launch was given
constexpr int REG_LO = 72, REG_HI = 216, REG_LAUNCH = 168;
static_assert(128 * REG_LO + 256 * REG_HI <= TT * REG_LAUNCH, "register split");

__device__ int g_tile_status;

struct Bars {
    uint64_t q_full, kv_full[NSTAGE], kv_empty[NSTAGE], s_full[2], p_full[2][2], o_full;
    uint32_t tmem;
    int abort, issued;
};
constexpr size_t TILE_SMEM = 2 * BLOCK_BYTES + NSTAGE * BLOCK_BYTES + sizeof(Bars) + 1024;

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, uint32_t polls,
                                         volatile int *abort) {
    const uint32_t a = smem_u32(bar);
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(a), "r"(parity), "r"(EX_SUSPEND_NS)
            : "memory");
        if (done) return true;
        if (*abort) return false;
    }
    *abort = 1;
    return false;
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int row, int head,
                                            int seq, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(head), "r"(seq),
        "r"(smem_u32(bar))
        : "memory");
}
// The instructions of the issuing warp run with all its lanes in step, and `lead` (1 in one lane, 0 in
// the others) is their predicate: operands then stay in uniform registers. Issued under a branch on
// the lane, each product took about 100 cycles to issue, against the 50 to 65 that it runs.
//
// D[tmem] (+)= A[smem] B[smem]^T and D[tmem] (+)= A[tmem] B[smem]^T, bf16 operands. Shared-memory
// descriptors are given by their low words and the high one.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
// Arrives on the barrier when every product issued before is complete.
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
// High words: 8 rows of 128 bytes per 1024, 128-byte swizzle. K-major (Q, K: channels contiguous),
// and operands whose N index is contiguous (V: channels), where the low word's upper half is the
// distance of the next 64 channels.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) {
    return ((addr & 0x3FFFFu) >> 4) | (uint32_t)(HALF_BYTES >> 4) << 16;
}
// D fp32, A and B bf16, 128 x 128; b_mn: B's N index is contiguous.
__host__ __device__ constexpr uint32_t idesc_tile(bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((128u >> 3) << 17) |
           ((128u >> 4) << 24);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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
// (a0, a1) * b + (c, c) in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The lowest n bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// What a CTA works on. PREFIX: "tokens" are the batch's sequences, the rows have no sequence, and
// every row is visible. Rows are taken in an order without the gap between sinks and window: c < skp
// (sk of them, filled up to a multiple of 16) are the sinks, then the rows from lo on, up to C. A
// window then begins with a block, and a few sinks cost 16 keys and no block: 9 blocks instead of
// 10.5 at a window of 1024 with 4 sinks.
struct Work {
    int b, h, t0;              // sequence, kv-head, first token of the pair of tiles
    int sp;                    // split
    int n, ql;
    int C, sk, skp, lo;
    int first, count;          // this CTA's blocks: first .. first + count - 1
    __device__ int base(int i) const { return (first + i) * TILE_ROWS; }   // in the order
    __device__ int row(int c) const { return c < skp ? c : c - skp + lo; }
};

template <bool PREFIX>
__device__ __forceinline__ Work work_of(const TileArgs &a, bool alternate) {
    Work w;
    // pairs in descending order, kv-heads and sequences within: the longest rows start first
    int id = blockIdx.x;
    const int bh = PREFIX ? a.H : a.B * a.H;
    const int unit = id % bh;
    id /= bh;
    w.sp = id % a.nsp;
    const int pair = a.pairs - 1 - id / a.nsp;
    w.b = PREFIX ? 0 : unit / a.H;
    w.h = PREFIX ? unit : unit - w.b * a.H;
    w.t0 = pair * (alternate ? 1 : 2) * a.tq;
    w.sk = w.skp = w.lo = 0;
    if (PREFIX) {
        w.n = w.C = a.rows;
        w.ql = a.m;
    } else {
        w.n = min(max(a.lens ? a.lens[w.b] : a.rows, 0), a.rows);
        w.ql = min(max(a.q_lens ? a.q_lens[w.b] : a.m, 0), a.m);
        const int t1 = min(w.t0 + (alternate ? 1 : 2) * a.tq, w.ql);
        const int hi = max(0, w.n - w.ql + t1), sk = min(a.sinks, hi);
        const int lo = max(0, w.n - w.ql + w.t0 - a.window + 1);
        w.C = hi;
        if (lo > sk) {
            w.sk = sk;
            w.skp = (sk + 15) & ~15;
            w.lo = lo;
            w.C = w.skp + hi - lo;
        }
    }
    w.count = (w.C + TILE_ROWS - 1) / TILE_ROWS;
    const long long all = w.count;
    w.first = (int)(all * w.sp / a.nsp);
    w.count = (int)(all * (w.sp + 1) / a.nsp) - w.first;
    return w;
}

template <bool PREFIX, bool ALT>
__global__ void __launch_bounds__(TT, 1)
exact_tile_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ TileMaps maps) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *qs = smem, *ring = smem + 2 * BLOCK_BYTES;
    Bars *bars = reinterpret_cast<Bars *>(ring + NSTAGE * BLOCK_BYTES);
    volatile int *abort_flag = &bars->abort;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // the same in all lanes
    const Work w = work_of<PREFIX>(a, ALT);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (w.t0 >= w.ql) return;
    const int N = w.count;

    if (tid == 0) {
        mbar_init(&bars->q_full, 1);
        for (int i = 0; i < NSTAGE; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        mbar_init(&bars->o_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i][0], 4);
            mbar_init(&bars->p_full[i][1], 4);
        }
        bars->abort = bars->issued = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc(&bars->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;

    // The order in which blocks' keys and values enter the ring is the order in which the products
    // take them: both tiles on every block: K0 V0 K1 V1 ...; the two groups on alternate blocks of
    // one tile: K0 K1 V0 K2 V1 K3 ...
    constexpr int AHEAD = ALT ? 2 : 1;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LO));
      if (warp == 0) {
        if (lane == 0 && N > 0) {
            constexpr int QT = ALT ? 1 : 2;
            const uint32_t q_bytes = (uint32_t)QT * a.tq * a.G * 256;
            mbar_arrive_expect_tx(&bars->q_full, q_bytes);
            for (int i = 0; i < QT; ++i)
                for (int x = 0; x < 2; ++x) {
                    uint8_t *dst = qs + i * BLOCK_BYTES + x * HALF_BYTES;
                    const int t = w.t0 + i * a.tq;
                    if (PREFIX) tma_load_4d(dst, &maps.q, x * 64, w.h * a.G, 0, t, &bars->q_full);
                    else tma_load_4d(dst, &maps.q, x * 64, w.h * a.G, t, w.b, &bars->q_full);
                }
            int issued = 0;
            auto load = [&](const CUtensorMap *map, const CUtensorMap *map16, int blk) {
                const int st = issued % NSTAGE;
                if (issued >= NSTAGE &&
                    !wait_bar(&bars->kv_empty[st], (issued / NSTAGE + 1) & 1, a.polls, abort_flag))
                    return false;
                const int c = w.base(blk), hd = w.h * a.head_mul, sq = w.b * a.seq_mul;
                uint8_t *dst = ring + st * BLOCK_BYTES;
                mbar_arrive_expect_tx(&bars->kv_full[st], BLOCK_BYTES);
                if (!PREFIX && c < w.skp && c + TILE_ROWS > w.skp) {
                    // sinks and window meet in this block: 16 rows at a time, one half after the other
                    for (int x = 0; x < TILE_ROWS; x += 16)
                        for (int y = 0; y < 2; ++y)
                            tma_load_4d(dst + y * HALF_BYTES + x * 128, map16, y * 64, w.row(c + x), hd,
                                        sq, &bars->kv_full[st]);
                } else {
                    tma_load_5d(dst, map, w.row(c), hd, sq, &bars->kv_full[st]);
                }
                ++issued;
                return true;
            };
            bool ok = true;
            for (int j = 0; ok && j < AHEAD && j < N; ++j) ok = load(&maps.k, &maps.k16, j);
            for (int j = 0; ok && j < N; ++j) {
                ok = load(&maps.v, &maps.v16, j);
                if (ok && j + AHEAD < N) ok = load(&maps.k, &maps.k16, j + AHEAD);
            }
            bars->issued = issued;
        }
      } else if (warp == 1) {
        const uint32_t lead = elect_one();
        const uint32_t ring_a = smem_u32(ring), empty_a = smem_u32(bars->kv_empty);
        const uint32_t q_desc = desc_k(smem_u32(qs));
        int st = 0;                                    // stage of the ring to take next
        uint32_t phase = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {   // the same answer in every lane
            return __all_sync(0xffffffffu, wait_bar(bar, parity, a.polls, abort_flag)) != 0;
        };
        auto full = [&]() { return wait(&bars->kv_full[st], phase); };
        auto qk = [&](int i, uint32_t k) {              // S_i = Q_i K^T
            const uint32_t q = q_desc + ((ALT ? 0 : i) * BLOCK_BYTES >> 4), kd = desc_k(k);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint32_t off = ((s >> 2) * HALF_BYTES + (s & 3) * 32) >> 4;
                mma_ss(lead, tmem + i * 128, q + off, kd + off, DESC_HI, idesc_tile(false), s > 0);
            }
            commit(lead, smem_u32(&bars->s_full[i]));
        };
        // O_i (+)= P_i V, 64 keys at a time: the first while the second's weights are computed
        auto pv = [&](int i, uint32_t v, uint32_t parity, bool acc) {
            const uint32_t vd = desc_mn(v);
            bool ok = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (ok) ok = wait(&bars->p_full[i][h], parity);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int s = 4 * h; s < 4 * h + 4; ++s)
                    mma_ts(lead, tmem + 256 + i * 128, tmem + i * 128 + s * 8, vd + (s * 2048 >> 4),
                           DESC_HI, idesc_tile(true), acc || s > 0);
            }
            return ok;
        };
        // Values of rows that no token of the pair sees may be anything: 0 x NaN would reach O.
        auto scrub = [&](int blk) {
            if (PREFIX) return;
            const int base = w.base(blk);
            const bool tail = base + TILE_ROWS > w.C, fill = base < w.skp && base + TILE_ROWS > w.sk;
            if (!tail && !fill) return;
            uint8_t *v = ring + st * BLOCK_BYTES;
            // rows from r0 to r1 lie together in each half
            auto zero = [&](int r0, int r1) {
                for (int x = 0; x < 2; ++x)
                    for (int e = r0 * 128 + lane * 16; e < r1 * 128; e += 512)
                        *reinterpret_cast<uint4 *>(v + x * HALF_BYTES + e) = make_uint4(0, 0, 0, 0);
            };
            if (tail) zero(w.C - base, TILE_ROWS);
            if (fill) zero(max(0, w.sk - base), min(TILE_ROWS, w.skp - base));
            fence_proxy_async_smem();
            __syncwarp();
        };
        auto release = [&]() {
            commit(lead, empty_a + st * 8);
            if (++st == NSTAGE) {
                st = 0;
                phase ^= 1;
            }
        };
        auto addr = [&]() { return ring_a + st * BLOCK_BYTES; };
        bool ok = N > 0 && wait(&bars->q_full, 0);
        if (!ALT) {
            if (ok) ok = full();
            if (ok) {
                qk(0, addr());
                qk(1, addr());
                release();
            }
            for (int j = 0; ok && j < N; ++j) {
                ok = full();                            // V_j; K_j+1 is behind it
                if (!ok) break;
                scrub(j);
                const bool more = j + 1 < N;
                const uint32_t v = addr(), k = ring_a + (st + 1 < NSTAGE ? st + 1 : 0) * BLOCK_BYTES;
                ok = pv(0, v, j & 1, j > 0);
                if (ok && more) {
                    ok = st + 1 < NSTAGE ? wait(&bars->kv_full[st + 1], phase)
                                         : wait(&bars->kv_full[0], phase ^ 1);
                    if (ok) qk(0, k);
                }
                if (ok) ok = pv(1, v, j & 1, j > 0);
                if (!ok) break;
                release();
                if (more) {
                    qk(1, k);
                    release();
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (ok && i < N) {
                    ok = full();
                    if (ok) {
                        qk(i, addr());
                        release();
                    }
                }
            }
            for (int j0 = 0; ok && j0 < N; j0 += 2) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = j0 + i;
                    if (!ok || j >= N) continue;
                    ok = full();
                    if (ok) scrub(j);
                    if (ok) ok = pv(i, addr(), (j >> 1) & 1, j > 1);
                    if (!ok) continue;
                    release();
                    if (j + 2 < N) {
                        ok = full();
                        if (ok) {
                            qk(i, addr());
                            release();
                        }
                    }
                }
            }
        }
        // commits follow all products before them, so these come when both tiles are complete;
        // after an abort they bound what is in flight
        if (N > 0) commit(lead, smem_u32(&bars->o_full));
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HI));
        const int i = (warp - 4) >> 2;                  // tile (ALT: share of the blocks)
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_bits = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_t = tmem + i * 128 + lane_bits, o_t = tmem + 256 + i * 128 + lane_bits;
        const int tl = row / a.G, gq = row - tl * a.G;
        const int tok = w.t0 + (ALT ? 0 : i * a.tq) + tl;
        const bool live = tl < a.tq && tok < w.ql;
        const int pos = PREFIX ? w.n - 1 : w.n - w.ql + tok;
        // the tile's own range of positions
        const int tile0 = w.t0 + (ALT ? 0 : i * a.tq);
        const int tp0 = PREFIX ? w.n - 1 : w.n - w.ql + tile0;
        const int tp1 = PREFIX ? w.n - 1 : w.n - w.ql + min(tile0 + a.tq, w.ql) - 1;
        const int mine = ALT ? (N - i + 1) / 2 : N;
        float m = -CUDART_INF_F;
        float2 l2 = make_float2(0.f, 0.f);
        bool ok = true;
        for (int x = 0; x < mine; ++x) {
            ok = wait_bar(&bars->s_full[i], x & 1, a.polls, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            float s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_t + c * 32, s[c]);
            tmem_wait_ld();
            const int base = w.base(ALT ? 2 * x + i : x);
            // (blocks inside every token's view need no mask)
            const int r0 = w.row(base);
            const bool inside =
                PREFIX ? base + TILE_ROWS <= w.n
                       : base >= w.skp ? r0 + TILE_ROWS - 1 <= tp0 && r0 > tp1 - a.window
                                       : base + TILE_ROWS <= w.sk;
            if (!inside) {
                // keys of this block that the row sees: below hi + 1 and not below lo, or below sk
                const int hi = pos - w.lo + w.skp - base;
                const int lo = PREFIX ? 0 : max(w.skp - base, hi - a.window + 1);
                const int sk = PREFIX ? 0 : (w.skp ? w.sk : a.sinks) - base;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // bit e: key 32 c + e is seen
                    const uint32_t see = bits_below(hi + 1 - 32 * c) &
                                         (~bits_below(lo - 32 * c) | bits_below(sk - 32 * c));
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[c][e] = see & (1u << e) ? s[c][e] : -CUDART_INF_F;
                }
            }
            float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int e = 0; e < 32; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) tops[c] = fmaxf(tops[c], s[c][e]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a.scale_log2;
            const bool raise = top > m + 8.f || (m == -CUDART_INF_F && top > m);
            if (__any_sync(0xffffffffu, raise)) {
                const float nm = raise ? top : m;
                const float f = m == -CUDART_INF_F ? 0.f : ex2(m - nm);
                m = nm;
                l2.x *= f;
                l2.y *= f;
                if (x > 0) {
                    // S of this block was issued behind the P V before it: O has that
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        uint32_t u[32];
                        tmem_ld32(o_t + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
                        tmem_st32(o_t + c * 32, u);
                    }
                }
            }
            const float ref = m == -CUDART_INF_F ? 0.f : m;
            const float2 sc = make_float2(a.scale_log2, a.scale_log2), nr = make_float2(-ref, -ref);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t p[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int q = c * 64 + 2 * e;
                    float2 y = fma2(make_float2(s[q >> 5][q & 31], s[q >> 5][(q & 31) + 1]), sc, nr);
                    y.x = ex2(y.x);
                    y.y = ex2(y.y);
                    l2 = add2(l2, y);
                    p[e] = pack(y.x, y.y);
                }
                tmem_st32(s_t + c * 32, p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&bars->p_full[i][c]);
            }
        }
        // ---- the tile is complete: out = O / l, or a record of this split -----------------------
        const float l = l2.x + l2.y;
        if (N > 0 && ok) {
            ok = wait_bar(&bars->o_full, 0, a.polls, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        }
        float *half = reinterpret_cast<float *>(ring);  // free by now; see `give`
        constexpr int CG = ALT ? 2 : 4;                 // quarters of the channels that a group puts out
        const int c0 = ALT && i == 1 ? 2 : 0;
        if (ALT) {
            // The groups' shares of the blocks join, each group for half of the channels: it gives
            // the other half, [channel][row], and both m and l to the other.
            float *give = half + (1 - i) * 64 * TILE_ROWS;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float o[32];
                if (mine > 0) {
                    tmem_ld32(o_t + (2 - c0 + c) * 32, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) give[(c * 32 + e) * TILE_ROWS + row] = mine > 0 ? o[e] : 0.f;
            }
            half[(128 + 2 * i) * TILE_ROWS + row] = m;
            half[(129 + 2 * i) * TILE_ROWS + row] = l;
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (ok) {
            const bool record = PREFIX || a.nsp > 1;
            float f0 = 1.f, f1 = 0.f, all_m = m, all_l = l;
            if (ALT) {
                const float m1 = half[(130 - 2 * i) * TILE_ROWS + row];
                const float l1 = half[(131 - 2 * i) * TILE_ROWS + row];
                all_m = fmaxf(m, m1);
                const float ref = all_m == -CUDART_INF_F ? 0.f : all_m;
                f0 = ex2(m - ref);
                f1 = ex2(m1 - ref);
                all_l = f0 * l + f1 * l1;
            }
            const float inv = all_l > 0.f ? 1.f / all_l : (all_l == 0.f ? 0.f : all_l);
            // Rows leave through shared memory (free by now), so that a warp's stores are contiguous:
            // a lane owns a row here and writes 16-byte pieces of two (bf16) or one (record) there.
            const long long at = ((long long)(w.b * a.H + w.h) * a.nsp + w.sp) * a.m * a.G +
                                 (long long)tok * a.G + gq;
            char *to = record ? reinterpret_cast<char *>(a.pre_o + at * EX_D)
                              : a.out + w.b * a.o_seq + (long long)(w.h * a.G + gq) * a.o_head +
                                    tok * a.o_tok;
            if (!live) to = nullptr;
            else if (record && c0 == 0)
                *reinterpret_cast<float2 *>(a.pre_ml + 2 * at) = make_float2(all_m, all_l);
            uint8_t *stage = ring + (ALT ? 3 * BLOCK_BYTES : 0) + (warp - 4) * 4096;
            // two halves of 64 channels (record: four of 32), 128 bytes of a row each
#pragma unroll
            for (int x = 0; x < CG; ++x) {
                const int c = c0 + x;
                float o[32];
                if (mine > 0) {
                    tmem_ld32(o_t + c * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (ALT) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = f0 * o[e] + f1 * half[(i * 64 + x * 32 + e) * TILE_ROWS + row];
                }
                if (record) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4 *>(stage + lane * 128 + ((e ^ (lane & 7)) * 16)) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4 *>(stage + lane * 128 +
                                                   (((4 * (x & 1) + e) ^ (lane & 7)) * 16)) =
                            make_uint4(pack(o[8 * e] * inv, o[8 * e + 1] * inv),
                                       pack(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                       pack(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                       pack(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
                    if (!(x & 1)) continue;
                }
                __syncwarp();
                const int part = record ? c : c >> 1;
#pragma unroll
                for (int k = 0; k < 8; ++k) {        // four rows at a time, 128 bytes each
                    const int r = 4 * k + (lane >> 3), e = lane & 7;
                    char *dst = reinterpret_cast<char *>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), r));
                    const uint4 v =
                        *reinterpret_cast<const uint4 *>(stage + r * 128 + ((e ^ (r & 7)) * 16));
                    if (dst) *reinterpret_cast<uint4 *>(dst + part * 128 + e * 16) = v;
                }
                __syncwarp();
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) {
        // products and copies in flight end before the block does (bounded waits)
        atomicExch(&g_tile_status, 1);
        if (N > 0) {
            int unset;
            auto drain = [&](uint64_t *bar, uint32_t parity) {
                unset = 0;
                wait_bar(bar, parity, EX_POLLS, &unset);
            };
            drain(&bars->o_full, 0);
            drain(&bars->q_full, 0);
            for (int i = max(0, bars->issued - NSTAGE); i < bars->issued; ++i)
                drain(&bars->kv_full[i % NSTAGE], (i / NSTAGE) & 1);
        }
    }
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the records of split rows: a warp per query row, four channels per lane.
template <bool F32IO>
__global__ void __launch_bounds__(256) exact_tile_merge_kernel(const __grid_constant__ TileArgs a) {
    const int lane = threadIdx.x & 31;
    const long long per_unit = (long long)a.m * a.G;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= per_unit * a.B * a.H) return;
    const int unit = (int)(row / per_unit), b = unit / a.H, h = unit - b * a.H;
    const long long x = row - unit * per_unit;
    const int tok = (int)(x / a.G), g = (int)(x - (long long)tok * a.G);
    if (tok >= min(max(a.q_lens ? a.q_lens[b] : a.m, 0), a.m)) return;
    const long long at = unit * per_unit * a.nsp + x;
    float M = -CUDART_INF_F;
    for (int r = 0; r < a.nsp; ++r) M = fmaxf(M, a.pre_ml[2 * (at + r * per_unit)]);
    const float ref = M == -CUDART_INF_F ? 0.f : M;
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < a.nsp; ++r) {
        const float2 ml = *reinterpret_cast<const float2 *>(a.pre_ml + 2 * (at + r * per_unit));
        const float f = ex2(ml.x - ref);
        const float4 v =
            *reinterpret_cast<const float4 *>(a.pre_o + (at + r * per_unit) * EX_D + lane * 4);
        L += f * ml.y;
        o.x += f * v.x;
        o.y += f * v.y;
        o.z += f * v.z;
        o.w += f * v.w;
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    char *op = a.out + b * a.o_seq + (long long)(h * a.G + g) * a.o_head + tok * a.o_tok;
    if constexpr (F32IO)
        *reinterpret_cast<float4 *>(op + lane * 16) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    else
        *reinterpret_cast<uint2 *>(op + lane * 8) =
            make_uint2(pack(o.x * inv, o.y * inv), pack(o.z * inv, o.w * inv));
}

template <bool PREFIX, bool ALT>
cudaError_t launch(const TileArgs &a, const TileMaps &maps, cudaStream_t s) {
    auto kern = exact_tile_kernel<PREFIX, ALT>;
    static std::atomic<unsigned long long> set{0};   // devices where the kernel may be launched
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(set.load(std::memory_order_acquire) & bit)) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        // setmaxnreg.inc draws on what the launch was given: less would wait for good
        if (((fa.numRegs + 7) & ~7) < REG_LAUNCH) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TILE_SMEM);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    const long long blocks = (long long)(PREFIX ? a.H : a.B * a.H) * a.pairs * a.nsp;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    kern<<<(unsigned)blocks, TT, TILE_SMEM, s>>>(a, maps);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_exact_tile(const TileArgs &a, const TileMaps &maps, bool prefix, bool alternate,
                              cudaStream_t s) {
    if (prefix) return alternate ? launch<true, true>(a, maps, s) : launch<true, false>(a, maps, s);
    return alternate ? launch<false, true>(a, maps, s) : launch<false, false>(a, maps, s);
}

cudaError_t launch_exact_tile_merge(const TileArgs &a, bool f32_io, cudaStream_t s) {
    const long long blocks = ((long long)a.B * a.H * a.m * a.G + 7) / 8;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return f32_io ? cudaLaunchKernelEx(&cfg, exact_tile_merge_kernel<true>, a)
                  : cudaLaunchKernelEx(&cfg, exact_tile_merge_kernel<false>, a);
}

cudaError_t exact_tile_status(int *timed_out, cudaStream_t s) {
    int x = 0;
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&x, g_tile_status, sizeof(int), 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && x)
        e = cudaMemcpyToSymbolAsync(g_tile_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    *timed_out = x;
    return e;
}

}  // namespace iskv
