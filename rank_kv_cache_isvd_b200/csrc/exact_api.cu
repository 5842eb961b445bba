// C entry points of attention over exact caches and of their eviction: checks of arguments,
// workspace sizes, launches. See include/iskv.h.
#include <math.h>
#include <string.h>

#include <mutex>

#include "evict.cuh"
#include "exact.cuh"
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

void fill(ExactArgs &a, const iskv_exact_rows *r, const iskv_exact_queries *q, int sms) {
    memset(&a, 0, sizeof(a));
    const long long e = esz_of(r->dtype), f = esz_of(q->dtype);
    a.k = static_cast<const char *>(r->k);
    a.v = static_cast<const char *>(r->v);
    a.seq_st = r->seq_stride * e;
    a.head_st = r->head_stride * e;
    a.row_st = r->row_stride * e;
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
    a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)EX_D));
    a.grid = sms;
}

// Workspace of the split kernel: its blocks' records, and with `items` one per item as well.
size_t record_bytes(int grid, long long items) {
    return align256((size_t)(2LL * grid + items) * EX_REC * sizeof(float));
}
long long score_stride(int rows) { return (rows + 15) / 16 * 16; }
size_t score_bytes(const iskv_exact_rows *r, int n_q_heads) {
    return align256((size_t)r->batch * n_q_heads * score_stride(r->rows) * sizeof(float));
}

int launched(cudaError_t e) {
    if (e == cudaSuccess) return ISKV_OK;
    cudaGetLastError();
    return ISKV_ERR_CUDA;
}

int run_split(const ExactArgs &a, const iskv_exact_rows *r, const iskv_exact_queries *q,
              cudaStream_t s) {
    const bool fr = r->dtype == ISKV_F32, fi = q->dtype == ISKV_F32;
    const int rc = launched(launch_exact_split(a, fr, fi, s));
    return rc == ISKV_OK ? launched(launch_exact_merge(a, fr, fi, s)) : rc;
}

}  // namespace

extern "C" int iskv_window_attn_workspace(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                          int window, int sinks, size_t *bytes) {
    if (!bytes || window < 1 || sinks < 0) return ISKV_ERR_INVALID_ARG;
    int rc = check_rows(r);
    if (rc == ISKV_OK) rc = check_queries(r, q);
    if (rc != ISKV_OK) return rc;
    const int sms = sm_count();
    if (!sms) return ISKV_ERR_CUDA;
    *bytes = record_bytes(sms, 0);
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
    a.direct = 1;
    a.rec = static_cast<float *>(ws);
    return run_split(a, r, q, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int iskv_mass_decode_workspace(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                          size_t *bytes) {
    if (!bytes) return ISKV_ERR_INVALID_ARG;
    int rc = check_rows(r);
    if (rc == ISKV_OK) rc = check_queries(r, q);
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
    return run_split(a, r, q, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int iskv_prefix_decode_workspace(const iskv_exact_rows *r, const iskv_exact_queries *q,
                                            const iskv_exact_prefix *p, size_t *bytes) {
    if (!bytes || !p) return ISKV_ERR_INVALID_ARG;
    int rc = check_rows(r);
    if (rc == ISKV_OK) rc = check_queries(r, q);
    if (rc != ISKV_OK) return rc;
    const int e = esz_of(r->dtype);
    if (q->m != 1 || q->q_lens || p->rows < 0 || p->rows > kMaxRows ||
        (p->rows > 0 && (!p->k || !p->v)) || !aligned16(p->k) || !aligned16(p->v) ||
        !stride_ok(p->head_stride, r->n_kv_heads, e) || !stride_ok(p->row_stride, p->rows, e))
        return ISKV_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (!sms) return ISKV_ERR_CUDA;
    const int tpt = ex_tpt(q->n_q_heads / r->n_kv_heads);
    const long long tiles = (r->batch + tpt - 1) / tpt;
    *bytes = record_bytes(sms, (long long)r->n_kv_heads * (r->batch + tiles));
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
    const long long e = esz_of(r->dtype);
    a.pk = static_cast<const char *>(p->k);
    a.pv = static_cast<const char *>(p->v);
    a.p_head = p->head_stride * e;
    a.p_row = p->row_stride * e;
    a.P = p->rows;
    a.rec = static_cast<float *>(ws);
    a.shared_here = p->rows > 0;
    return run_split(a, r, q, reinterpret_cast<cudaStream_t>(stream));
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
    if ((r->batch > 1 && r->seq_stride < EX_D) || (r->n_kv_heads > 1 && r->head_stride < EX_D) ||
        (r->rows > 1 && r->row_stride < EX_D))
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
