// C entry points of attention over exact caches and of their eviction: checks of arguments,
// workspace sizes, launches. See include/iskv.h.
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "evict.cuh"
#include "exact.cuh"
#include "exact_tile.cuh"
#include "iskv_internal.cuh"

using namespace iskv;

namespace {

constexpr long long kMaxRows = 1LL << 24;
constexpr int kMaxUnits = 65535;
constexpr int kMaxDevices = 64;

int sm_count() {
    static int known[kMaxDevices];
    static std::mutex mu;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        known[dev] = n;
    }
    return known[dev];
}

std::atomic<int> g_polls{(int)EX_POLLS};   // of a device-side wait, before it gives up

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int esz_of(int dtype) { return dtype == ISKV_BF16 ? 2 : 4; }

// A stride of `count` items that step over at least `least` elements: 16-byte multiples.
bool stride_ok(long long st, int count, int esz) {
    if (count <= 1) return true;
    return st >= 0 && st < (1LL << 40) && (st * esz) % 16 == 0;
}

int check_rows(const iskv_exact_rows *r) {
    if (!r || r->batch < 1 || r->n_kv_heads < 1 || r->rows < 0 || r->rows > kMaxRows ||
        (r->dtype != ISKV_BF16 && r->dtype != ISKV_F32))
        return ISKV_ERR_INVALID_ARG;
    if (r->rows > 0 && (!r->k || !r->v)) return ISKV_ERR_INVALID_ARG;
    if (!aligned16(r->k) || !aligned16(r->v)) return ISKV_ERR_INVALID_ARG;
    const int e = esz_of(r->dtype);
    if (!stride_ok(r->seq_stride, r->batch, e) || !stride_ok(r->head_stride, r->n_kv_heads, e) ||
        !stride_ok(r->row_stride, r->rows, e))
        return ISKV_ERR_INVALID_ARG;
    // rows of one sequence in one place, or overlapping
    if (r->rows > 1 && r->row_stride < EX_D) return ISKV_ERR_INVALID_ARG;
    if ((long long)r->batch * r->n_kv_heads > kMaxUnits) return ISKV_ERR_UNSUPPORTED;
    return ISKV_OK;
}

int check_queries(const iskv_exact_rows *r, const iskv_exact_queries *q) {
    if (!q || !q->q || !q->out || q->m < 1 || q->m > kMaxRows || q->n_q_heads < r->n_kv_heads ||
        q->n_q_heads % r->n_kv_heads != 0 || q->n_q_heads / r->n_kv_heads > GMAX ||
        (q->dtype != ISKV_BF16 && q->dtype != ISKV_F32) || !aligned16(q->q) || !aligned16(q->out))
        return ISKV_ERR_INVALID_ARG;
    const int e = esz_of(q->dtype);
    if (!stride_ok(q->q_seq_stride, r->batch, e) || !stride_ok(q->q_head_stride, q->n_q_heads, e) ||
        !stride_ok(q->q_tok_stride, q->m, e) || !stride_ok(q->o_seq_stride, r->batch, e) ||
        !stride_ok(q->o_head_stride, q->n_q_heads, e) || !stride_ok(q->o_tok_stride, q->m, e))
        return ISKV_ERR_INVALID_ARG;
    // two outputs in one place
    if ((r->batch > 1 && q->o_seq_stride < EX_D) || (q->n_q_heads > 1 && q->o_head_stride < EX_D) ||
        (q->m > 1 && q->o_tok_stride < EX_D))
        return ISKV_ERR_INVALID_ARG;
    // float32 rows go with float32 queries and outputs
    if (r->dtype == ISKV_F32 && q->dtype != ISKV_F32) return ISKV_ERR_UNSUPPORTED;
    return ISKV_OK;
}

// The split kernel counts (tile, step) pairs in 32 bits.
int check_split(const iskv_exact_rows *r, const iskv_exact_queries *q) {
    const int tpt = ex_tpt(q->n_q_heads / r->n_kv_heads);
    const long long tiles = (q->m + tpt - 1) / tpt;
    return (long long)r->batch * r->n_kv_heads * tiles * (r->rows / 16 + 3) > 0x7fffffffLL
               ? ISKV_ERR_UNSUPPORTED
               : ISKV_OK;
}

// 0 where the items of a dimension all sit in one place: maps then have an extent of 1 there.
int multiplier(long long stride, int count) { return count > 1 && stride == 0 ? 0 : 1; }

void fill(ExactArgs &a, const iskv_exact_rows *r, const iskv_exact_queries *q, int sms) {
    memset(&a, 0, sizeof(a));
    const long long f = esz_of(q->dtype);
    a.B = r->batch;
    a.H = r->n_kv_heads;
    a.rows = r->rows;
    a.lens = r->lens;
    a.q = static_cast<const char *>(q->q);
    a.out = static_cast<char *>(q->out);
    a.q_seq = q->q_seq_stride * f;
    a.q_head = q->q_head_stride * f;
    a.q_tok = q->q_tok_stride * f;
    a.o_seq = q->o_seq_stride * f;
    a.o_head = q->o_head_stride * f;
    a.o_tok = q->o_tok_stride * f;
    a.G = q->n_q_heads / r->n_kv_heads;
    a.m = q->m;
    a.q_lens = q->q_lens;
    a.window = (int)kMaxRows;
    a.seq_mul = multiplier(r->seq_stride, r->batch);
    a.head_mul = multiplier(r->head_stride, r->n_kv_heads);
    a.p_head_mul = 1;
    a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)EX_D));
    a.grid = sms;
    a.cluster = 1;
    a.polls = (uint32_t)g_polls.load(std::memory_order_relaxed);
}

// Workspace of the split kernel: its teams' records, and with `items` one per item as well.
size_t record_bytes(int sms, long long items) {
    return align256((size_t)(2LL * EX_WARPS * sms + items) * EX_REC * sizeof(float));
}
long long score_stride(int rows) { return (rows + 31) / 32 * 32; }
size_t score_bytes(const iskv_exact_rows *r, int n_q_heads) {
    return align256((size_t)r->batch * n_q_heads * score_stride(r->rows) * sizeof(float));
}

int launched(cudaError_t e) {
    if (e == cudaSuccess) return ISKV_OK;
    cudaGetLastError();
    return ISKV_ERR_CUDA;
}

// ---- the tile kernel: which calls take it, and how their work is cut ------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        cudaGetLastError();
        return static_cast<EncodeTiledFn>(nullptr);
    }();
    return fn;
}

// Map of `n` dimensions: extents, byte strides of all but the first, boxes. The first dimension is
// 128 bytes of a row; shared memory gets rows of 128 bytes, swizzled.
bool encode(CUtensorMap *map, int dtype, int n, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box) {
    const EncodeTiledFn enc = encode_tiled();
    const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
    return enc && enc(map, dtype == ISKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                      n, const_cast<void *>(base), dims, strides, box, steps,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows as (channels of a 128-byte part, row, part, kv-head, sequence), boxes of `box_rows` whole
// rows: [part][row][128 bytes] in shared memory. An extent whose items share one place becomes 1.
bool rows_map(CUtensorMap *map, const void *base, int dtype, int rows, int heads, int seqs,
              long long row_st, long long head_st, long long seq_st, int box_rows) {
    const cuuint64_t e = (cuuint64_t)esz_of(dtype), parts = EX_D * e / 128;
    auto ext = [](long long st, int n) { return (cuuint64_t)(n > 1 && st == 0 ? 1 : n); };
    auto str = [](long long st, int n) { return (cuuint64_t)(n > 1 && st ? st : 512); };
    const cuuint64_t dims[5] = {128 / e, (cuuint64_t)rows, parts, ext(head_st, heads),
                                ext(seq_st, seqs)};
    const cuuint64_t strides[4] = {str(row_st * e, rows), 128, str(head_st * e, heads),
                                   str(seq_st * e, seqs)};
    const cuuint32_t box[5] = {(cuuint32_t)(128 / e), (cuuint32_t)box_rows, (cuuint32_t)parts, 1, 1};
    return encode(map, dtype, 5, base, dims, strides, box);
}

// The same rows as (channels, row, kv-head, sequence), boxes of 64 channels of 16 bf16 rows.
bool rows16_map(CUtensorMap *map, const iskv_exact_rows *r, const void *base) {
    auto ext = [](long long st, int n) { return (cuuint64_t)(n > 1 && st == 0 ? 1 : n); };
    auto str = [](long long st, int n) { return (cuuint64_t)(n > 1 && st ? st * 2 : 256); };
    const cuuint64_t dims[4] = {EX_D, (cuuint64_t)r->rows, ext(r->head_stride, r->n_kv_heads),
                                ext(r->seq_stride, r->batch)};
    const cuuint64_t strides[3] = {str(r->row_stride, r->rows), str(r->head_stride, r->n_kv_heads),
                                   str(r->seq_stride, r->batch)};
    const cuuint32_t box[4] = {64, 16, 1, 1};
    return encode(map, ISKV_BF16, 4, base, dims, strides, box);
}

bool own_maps(CUtensorMap *k, CUtensorMap *v, const iskv_exact_rows *r, int box_rows) {
    if (r->rows == 0) return true;                   // never read
    return rows_map(k, r->k, r->dtype, r->rows, r->n_kv_heads, r->batch, r->row_stride,
                    r->head_stride, r->seq_stride, box_rows) &&
           rows_map(v, r->v, r->dtype, r->rows, r->n_kv_heads, r->batch, r->row_stride,
                    r->head_stride, r->seq_stride, box_rows);
}
bool prefix_maps(CUtensorMap *k, CUtensorMap *v, const iskv_exact_rows *r,
                 const iskv_exact_prefix *p, int box_rows) {
    if (p->rows == 0) return true;
    return rows_map(k, p->k, r->dtype, p->rows, r->n_kv_heads, 1, p->row_stride, p->head_stride, 0,
                    box_rows) &&
           rows_map(v, p->v, r->dtype, p->rows, r->n_kv_heads, 1, p->row_stride, p->head_stride, 0,
                    box_rows);
}

struct TilePlan {
    bool use, tile, alternate;         // tile: by the tile kernel, else by the rows kernel
    int tq, pairs, nsp;
};

// Whether a call takes the kernels for many query rows. One tile of 8 reads the rows once in the split kernel
// as well.
bool many_rows(int tokens, int G, long long seen) {
    return tokens * (long long)G > EX_QROWS && seen > 0;
}

// `tokens` query tokens (prefix: sequences) per unit, over at most `seen` rows each.
TilePlan tile_plan(int units, int tokens, int G, long long seen, bool tile, int sms) {
    TilePlan p;
    memset(&p, 0, sizeof(p));
    p.use = many_rows(tokens, G, seen);
    if (!p.use) return p;
    p.tile = tile;
    p.tq = tile ? TILE_ROWS / G : EX_WARPS * ex_tpt(G);
    const long long tiles = (tokens + p.tq - 1) / p.tq;
    p.alternate = tile && tiles == 1;         // one tile: the CTA's halves share out its blocks
    p.pairs = (int)(!tile || p.alternate ? tiles : (tiles + 1) / 2);
    const long long ctas = (long long)units * p.pairs;
    const long long blocks = (seen + TILE_ROWS - 1) / TILE_ROWS;
    // fewer CTAs than SMs: split the rows, in parts of a few blocks at least (a CTA's beginning and
    // end take the time of about four blocks of the tile kernel, of one of the rows kernel)
    long long nsp = ctas >= sms ? 1 : sms / ctas;
    const long long most = blocks / (tile ? 4 : 1) > 1 ? blocks / (tile ? 4 : 1) : 1;
    if (nsp > most) nsp = most;
    if (nsp > EX_PRE_MAX) nsp = EX_PRE_MAX;
    p.nsp = (int)nsp;
    return p;
}
size_t tile_record_bytes(const TilePlan &p, long long units, long long tokens, int G) {
    if (!p.use) return 0;
    return align256((size_t)(units * p.nsp * tokens * G) * 2 * sizeof(float)) +
           align256((size_t)(units * p.nsp * tokens * G) * EX_D * sizeof(float));
}

bool all_bf16(const iskv_exact_rows *r, const iskv_exact_queries *q) {
    return r->dtype == ISKV_BF16 && q->dtype == ISKV_BF16;
}

TilePlan window_plan(const iskv_exact_rows *r, const iskv_exact_queries *q, int window, int sinks,
                     bool tile, int sms) {
    const int G = q->n_q_heads / r->n_kv_heads;
    // rows that a pair of tiles sees at most
    const long long near = (long long)window + sinks + 15 + 2 * (TILE_ROWS / G);
    return tile_plan(r->batch * r->n_kv_heads, q->m, G, near < r->rows ? near : r->rows, tile, sms);
}

TilePlan prefix_plan(const iskv_exact_rows *r, const iskv_exact_queries *q,
                     const iskv_exact_prefix *p, bool tile, int sms) {
    return tile_plan(r->n_kv_heads, r->batch, q->n_q_heads / r->n_kv_heads, p->rows, tile, sms);
}

// Arguments of the kernels for many rows.
void tile_args(TileArgs &t, const TilePlan &p, const ExactArgs &a, bool prefix, float *records) {
    memset(&t, 0, sizeof(t));
    t.B = a.B;
    t.H = a.H;
    t.G = a.G;
    t.rows = prefix ? a.P : a.rows;
    t.lens = a.lens;
    t.q_lens = a.q_lens;
    t.m = prefix ? a.B : a.m;
    t.window = a.window;
    t.sinks = a.sinks;
    t.seq_mul = prefix ? 0 : a.seq_mul;
    t.head_mul = prefix ? a.p_head_mul : a.head_mul;
    t.tq = p.tq;
    t.pairs = p.pairs;
    t.nsp = p.nsp;
    t.q = a.q;
    t.q_seq = a.q_seq;
    t.q_head = a.q_head;
    t.q_tok = a.q_tok;
    t.out = a.out;
    t.o_seq = a.o_seq;
    t.o_head = a.o_head;
    t.o_tok = a.o_tok;
    t.scale_log2 = a.scale_log2;
    t.polls = a.polls;
    t.pre_ml = records;
    if (records)
        t.pre_o = reinterpret_cast<float *>(
            reinterpret_cast<char *>(records) +
            align256((size_t)(prefix ? a.H : a.B * a.H) * p.nsp * t.m * a.G * 2 * sizeof(float)));
}
// Queries as (64 channels of a half, q-head, token, sequence), boxes of one group's heads and one
// tile's tokens (prefix: sequences). False where items share a place: the tile kernel cannot take
// such queries, and the rows kernel does.
bool query_map(CUtensorMap *map, const ExactArgs &a, bool prefix, int tq) {
    const long long ext[3] = {(long long)a.H * a.G, a.m, a.B}, st[3] = {a.q_head, a.q_tok, a.q_seq};
    cuuint64_t dims[4] = {EX_D, 0, 0, 0}, strides[3];
    for (int i = 0; i < 3; ++i) {
        if (ext[i] > 1 && st[i] == 0) return false;
        dims[i + 1] = (cuuint64_t)ext[i];
        strides[i] = (cuuint64_t)(ext[i] > 1 ? st[i] : 256);
    }
    const cuuint32_t box[4] = {64, (cuuint32_t)a.G, (cuuint32_t)(prefix ? 1 : tq),
                               (cuuint32_t)(prefix ? tq : 1)};
    return encode(map, ISKV_BF16, 4, a.q, dims, strides, box);
}

// How the split kernel's work is cut: by items where they fill the GPU well enough (one launch, no
// records), else by steps.
void split_plan(ExactArgs &a, bool f32_rows, int sms) {
    const int tpt = ex_tpt(a.G), wr = ex_warp_rows(f32_rows);
    const int tiles = (a.m + tpt - 1) / tpt;
    const long long items = (long long)a.B * a.H * tiles;
    const int most = ex_most_rows(a.window, a.sinks, tpt, a.rows, wr);
    a.cluster = 1;
    a.by_items = 0;
    a.rt_max = tiles;
    // bf16 rows saturate HBM from fewer SMs than there are, and with more copies in flight it gives less
    // (10 x 32768 rows of 8 kv-heads: 214 us on 148 SMs, 203 on 100; 150 x 2048, ragged: 174 and 162; with
    // weights, 10 x 8192 ragged: 67 on 148, 63 on 120). Float32 rows are bound by instructions.
    auto by_steps = [&](int team) {
        a.grid = f32_rows || a.shared_here ? sms : a.mass ? sms - sms / 5 : sms - sms / 3;
        a.team = team;
        a.teams = a.grid * (EX_WARPS / team);
    };
    // a shared prefix's tiles and the sequences' own rows join by records
    if (a.shared_here) return by_steps(EX_WARPS);
    // teams as large as there are warps for every item, and no larger than the item has rows for
    int team = EX_WARPS, c = 1;
    while (team > 1 && (items * team > (long long)sms * EX_WARPS || most <= wr * team / 2)) team /= 2;
    const int steps = (most + wr * team - 1) / (wr * team);
    if (team == EX_WARPS)
        while (c < 8 && items * 2 * c <= sms && steps > c) c *= 2;
    long long slots = (long long)sms * (EX_WARPS / team);    // teams that run at once
    for (; c > 1; c /= 2) {
        slots = exact_split_clusters(c);
        if (slots >= items) break;
    }
    if (c == 1) slots = (long long)sms * (EX_WARPS / team);
    const long long rounds = (items + slots - 1) / slots;
    // Long items that leave teams idle go by steps, which are shared out evenly but cost records and a
    // merge. By items 10 x 8192 rows of 8 kv-heads take 53 us on 80 SMs, by steps 64: one round on half of
    // the SMs saturates HBM. But where lengths may differ (a list, read on the device) short items leave
    // more idle: 19 x 8192, ragged, 98 and 81 us, in several rounds 150 x 2048 258 and 205, of float32 rows
    // 75 x 2 x 4096 196 and 121. Of 16 steps, 40 x 1000 ragged, items take 30 us and steps 34.
    const bool idle = 4 * items < (f32_rows || a.lens || rounds > 1 ? 3 : 2) * rounds * slots;
    if (idle && steps > (f32_rows ? 8 : 16) * c) return by_steps(items >= 2 * sms ? 1 : EX_WARPS);
    const long long teams = items < slots ? items : slots;
    a.by_items = 1;
    a.team = team;
    a.cluster = c;
    // few items: their teams spread over the SMs
    const int per_block = EX_WARPS / team;
    a.grid = (int)((teams + per_block - 1) / per_block) * c;
    a.teams = a.grid / c * per_block;
    a.items = (unsigned)items;
    a.share = (unsigned)(items / a.teams);
    a.extra = (unsigned)(items % a.teams);
}

int run_split(ExactArgs &a, ExactMaps &maps, const iskv_exact_rows *r, const iskv_exact_queries *q,
              cudaStream_t s) {
    const bool fr = r->dtype == ISKV_F32, fi = q->dtype == ISKV_F32;
    if (!own_maps(&maps.k, &maps.v, r, ex_warp_rows(fr))) return ISKV_ERR_CUDA;
    split_plan(a, fr, a.grid);
    const int rc = launched(launch_exact_split(a, maps, fr, fi, s));
    return rc == ISKV_OK ? launched(launch_exact_merge(a, fr, fi, s)) : rc;
}

}  // namespace

extern "C" int iskv_window_attn_workspace(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                          int window, int sinks, size_t *bytes) {
    if (!bytes || window < 1 || sinks < 0) return ISKV_ERR_INVALID_ARG;
    int rc = check_rows(r);
    if (rc == ISKV_OK) rc = check_queries(r, q);
    if (rc != ISKV_OK) return rc;
    const long long units = (long long)r->batch * r->n_kv_heads;
    const int G = q->n_q_heads / r->n_kv_heads;
    if (!many_rows(q->m, G, r->rows)) rc = check_split(r, q);
    if (rc != ISKV_OK) return rc;
    // a grid's blocks (the rows are split only where they are fewer than the SMs)
    for (int tile = 0; tile <= (all_bf16(r, q) ? 1 : 0); ++tile) {
        const TilePlan p = window_plan(r, q, window, sinks, tile != 0, 1);
        if (p.use && units * p.pairs > 0x7fffffffLL) return ISKV_ERR_UNSUPPORTED;
    }
    const int sms = sm_count();
    if (!sms) return ISKV_ERR_CUDA;
    *bytes = record_bytes(sms, 0);
    // what the call takes: queries that cannot be mapped go to the rows kernel
    for (int tile = 0; tile <= (all_bf16(r, q) ? 1 : 0); ++tile) {
        const TilePlan p = window_plan(r, q, window, sinks, tile != 0, sms);
        const size_t b = p.nsp > 1 ? tile_record_bytes(p, units, q->m, G) : 0;
        if (b > *bytes) *bytes = b;
    }
    return ISKV_OK;
}

extern "C" int iskv_window_attn(const iskv_exact_rows *r, const iskv_exact_queries *q, int window,
                                int sinks, void *ws, size_t ws_bytes, iskv_stream_t stream) {
    if (!ws || !aligned16(ws)) return ISKV_ERR_INVALID_ARG;
    size_t need = 0;
    const int rc = iskv_window_attn_workspace(r, q, window, sinks, &need);
    if (rc != ISKV_OK) return rc;
    if (ws_bytes < need) return ISKV_ERR_CAPACITY;
    ExactArgs a;
    fill(a, r, q, sm_count());
    a.window = window < kMaxRows ? window : (int)kMaxRows;
    a.sinks = sinks < r->rows ? sinks : r->rows;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fr = r->dtype == ISKV_F32, fi = q->dtype == ISKV_F32;
    TileMaps tm;
    TilePlan p = window_plan(r, q, window, sinks, all_bf16(r, q), a.grid);
    if (p.tile && !query_map(&tm.q, a, false, p.tq))
        p = window_plan(r, q, window, sinks, false, a.grid);
    if (p.use) {
        if (!own_maps(&tm.k, &tm.v, r, p.tile ? TILE_ROWS : ex_warp_rows(fr)) ||
            (p.tile && !(rows16_map(&tm.k16, r, r->k) && rows16_map(&tm.v16, r, r->v))))
            return ISKV_ERR_CUDA;
        TileArgs t;
        tile_args(t, p, a, false, p.nsp > 1 ? static_cast<float *>(ws) : nullptr);
        const int e = launched(p.tile ? launch_exact_tile(t, tm, false, p.alternate, s)
                                      : launch_exact_rows(t, tm.k, tm.v, fr, fi, false, s));
        if (e != ISKV_OK || p.nsp == 1) return e;
        return launched(launch_exact_tile_merge(t, fi, s));
    }
    a.rec = static_cast<float *>(ws);
    ExactMaps maps;
    return run_split(a, maps, r, q, s);
}

extern "C" int iskv_mass_decode_workspace(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                          size_t *bytes) {
    if (!bytes) return ISKV_ERR_INVALID_ARG;
    int rc = check_rows(r);
    if (rc == ISKV_OK) rc = check_queries(r, q);
    if (rc == ISKV_OK) rc = check_split(r, q);
    if (rc != ISKV_OK) return rc;
    if (q->m != 1 || q->q_lens) return ISKV_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (!sms) return ISKV_ERR_CUDA;
    *bytes = record_bytes(sms, (long long)r->batch * r->n_kv_heads) + score_bytes(r, q->n_q_heads);
    return ISKV_OK;
}

extern "C" int iskv_mass_decode(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                const float *mass, float *mass_out, void *ws, size_t ws_bytes,
                                iskv_stream_t stream) {
    if (!ws || !aligned16(ws)) return ISKV_ERR_INVALID_ARG;
    size_t need = 0;
    const int rc = iskv_mass_decode_workspace(r, q, &need);
    if (rc != ISKV_OK) return rc;
    if (r->rows > 0 && (!mass || !mass_out)) return ISKV_ERR_INVALID_ARG;
    if (ws_bytes < need) return ISKV_ERR_CAPACITY;
    ExactArgs a;
    fill(a, r, q, sm_count());
    a.rec = static_cast<float *>(ws);
    a.scores = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                         record_bytes(a.grid, (long long)a.B * a.H));
    a.score_st = score_stride(r->rows);
    // an empty cache has no weights to add
    a.mass = mass;
    a.mass_out = mass_out;
    ExactMaps maps;
    return run_split(a, maps, r, q, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int iskv_prefix_decode_workspace(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                            const iskv_exact_prefix *p, size_t *bytes) {
    if (!bytes || !p) return ISKV_ERR_INVALID_ARG;
    int rc = check_rows(r);
    if (rc == ISKV_OK) rc = check_queries(r, q);
    if (rc == ISKV_OK) rc = check_split(r, q);
    if (rc != ISKV_OK) return rc;
    const int e = esz_of(r->dtype);
    if (q->m != 1 || q->q_lens || p->rows < 0 || p->rows > kMaxRows ||
        (p->rows > 0 && (!p->k || !p->v)) || !aligned16(p->k) || !aligned16(p->v) ||
        !stride_ok(p->head_stride, r->n_kv_heads, e) || !stride_ok(p->row_stride, p->rows, e) ||
        (p->rows > 1 && p->row_stride < EX_D))
        return ISKV_ERR_INVALID_ARG;
    const int tpt = ex_tpt(q->n_q_heads / r->n_kv_heads);
    const long long tiles = (r->batch + tpt - 1) / tpt;
    // one tile: the split kernel takes the prefix, and counts its steps in 32 bits with the others
    if (tiles == 1 && (long long)r->n_kv_heads * (p->rows / 16 + 3) > 0x7fffffffLL)
        return ISKV_ERR_UNSUPPORTED;
    const int sms = sm_count();
    if (!sms) return ISKV_ERR_CUDA;
    size_t records = 0;
    for (int tile = 0; tile <= (all_bf16(r, q) ? 1 : 0); ++tile) {
        const size_t b = tile_record_bytes(prefix_plan(r, q, p, tile != 0, sms), r->n_kv_heads,
                                           r->batch, q->n_q_heads / r->n_kv_heads);
        if (b > records) records = b;
    }
    *bytes = record_bytes(sms, (long long)r->n_kv_heads * (r->batch + tiles)) + records;
    return ISKV_OK;
}

extern "C" int iskv_prefix_decode(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                  const iskv_exact_prefix *p, void *ws, size_t ws_bytes,
                                  iskv_stream_t stream) {
    if (!ws || !aligned16(ws)) return ISKV_ERR_INVALID_ARG;
    size_t need = 0;
    const int rc = iskv_prefix_decode_workspace(r, q, p, &need);
    if (rc != ISKV_OK) return rc;
    if (ws_bytes < need) return ISKV_ERR_CAPACITY;
    ExactArgs a;
    fill(a, r, q, sm_count());
    a.P = p->rows;
    a.p_head_mul = multiplier(p->head_stride, r->n_kv_heads);
    a.rec = static_cast<float *>(ws);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fr = r->dtype == ISKV_F32, fi = q->dtype == ISKV_F32;
    ExactMaps maps;
    TileMaps tm;
    TilePlan plan = prefix_plan(r, q, p, all_bf16(r, q), a.grid);
    if (plan.tile && !query_map(&tm.q, a, true, plan.tq)) plan = prefix_plan(r, q, p, false, a.grid);
    if (plan.use) {
        if (!prefix_maps(&tm.k, &tm.v, r, p, plan.tile ? TILE_ROWS : ex_warp_rows(fr)))
            return ISKV_ERR_CUDA;
        const int tpt = ex_tpt(a.G);
        const size_t at = record_bytes(a.grid, (long long)a.H * (a.B + (a.B + tpt - 1) / tpt));
        TileArgs t;
        tile_args(t, plan, a, true, reinterpret_cast<float *>(static_cast<char *>(ws) + at));
        const int e = launched(plan.tile ? launch_exact_tile(t, tm, true, plan.alternate, s)
                                         : launch_exact_rows(t, tm.k, tm.v, fr, fi, true, s));
        if (e != ISKV_OK) return e;
        a.pre_ml = t.pre_ml;
        a.pre_o = t.pre_o;
        a.nsp = plan.nsp;
        a.after = 1;
        return run_split(a, maps, r, q, s);
    }
    a.shared_here = p->rows > 0;
    if (!prefix_maps(&maps.pk, &maps.pv, r, p, ex_warp_rows(r->dtype == ISKV_F32))) return ISKV_ERR_CUDA;
    return run_split(a, maps, r, q, s);
}

extern "C" int iskv_evict_workspace(const iskv_exact_rows *r, int budget, size_t *bytes) {
    if (!bytes || budget < 1) return ISKV_ERR_INVALID_ARG;
    const int rc = check_rows(r);
    if (rc != ISKV_OK) return rc;
    const long long units = (long long)r->batch * r->n_kv_heads;
    const long long over = r->rows > budget ? r->rows - budget : 0;
    const long long moves = over < budget ? over : budget;
    *bytes = align256((size_t)units * 2 * sizeof(int)) +
             align256((size_t)units * 2 * (moves > 0 ? moves : 1) * sizeof(int));
    return ISKV_OK;
}

extern "C" int iskv_evict(const iskv_exact_rows *r, const float *mass, float *mass_out,
                          const int *pos, int *pos_out, int *lens_out, int budget, int recent,
                          int sinks, void *ws, size_t ws_bytes, iskv_stream_t stream) {
    if (!ws || !aligned16(ws)) return ISKV_ERR_INVALID_ARG;
    size_t need = 0;
    const int rc = iskv_evict_workspace(r, budget, &need);
    if (rc != ISKV_OK) return rc;
    if (recent < 0 || sinks < 0 || (long long)recent + sinks > budget || !lens_out)
        return ISKV_ERR_INVALID_ARG;
    if (r->rows > 0 && (!mass || !mass_out || !pos || !pos_out)) return ISKV_ERR_INVALID_ARG;
    // rows that two units, or two slots, share cannot be moved in place
    if ((r->batch > 1 && r->seq_stride < EX_D) || (r->n_kv_heads > 1 && r->head_stride < EX_D))
        return ISKV_ERR_INVALID_ARG;
    if (ws_bytes < need) return ISKV_ERR_CAPACITY;
    const int sms = sm_count();
    if (!sms) return ISKV_ERR_CUDA;
    EvictArgs a;
    memset(&a, 0, sizeof(a));
    a.esz = esz_of(r->dtype);
    a.k = const_cast<char *>(static_cast<const char *>(r->k));
    a.v = const_cast<char *>(static_cast<const char *>(r->v));
    a.seq_st = r->seq_stride * a.esz;
    a.head_st = r->head_stride * a.esz;
    a.row_st = r->row_stride * a.esz;
    a.B = r->batch;
    a.H = r->n_kv_heads;
    a.rows = r->rows;
    a.lens = r->lens;
    a.lens_out = lens_out;
    a.mass = mass;
    a.mass_out = mass_out;
    a.pos = pos;
    a.pos_out = pos_out;
    a.budget = budget;
    a.recent = recent;
    a.sinks = sinks;
    const int over = r->rows > budget ? r->rows - budget : 0;
    a.max_moves = over < budget ? over : budget;
    const long long units = (long long)a.B * a.H;
    a.n_moves = static_cast<int *>(ws);
    a.keep = a.n_moves + units;
    a.moves = reinterpret_cast<int *>(static_cast<char *>(ws) + align256((size_t)units * 8));
    return launched(launch_evict(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int iskv_exact_wait_limit(int polls) {
    if (polls < 0) return ISKV_ERR_INVALID_ARG;
    g_polls.store(polls, std::memory_order_relaxed);
    return ISKV_OK;
}

extern "C" int iskv_exact_status(iskv_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int tile = 0, rows = 0, split = 0;
    int rc = launched(exact_tile_status(&tile, s));
    if (rc == ISKV_OK) rc = launched(exact_rows_status(&rows, s));
    if (rc == ISKV_OK) rc = launched(exact_split_status(&split, s));
    return rc != ISKV_OK ? rc : tile || rows || split ? ISKV_ERR_TIMEOUT : ISKV_OK;
}
