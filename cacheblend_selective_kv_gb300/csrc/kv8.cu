// C ABI of the 8-bit paged K/V cache (cb_kv8_*): the handle and the checks of its calls' arguments.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "cb_kv8.cuh"

using namespace cb;

namespace {

cb_status fail(cb_status code, const char* fmt, ...) {
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_last_error(msg);
    return code;
}

constexpr int64_t kMaxRows = (int64_t)1 << 30;

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const char *x = (const char*)a, *y = (const char*)b;
    return a_bytes > 0 && b_bytes > 0 && x < y + b_bytes && y < x + a_bytes;
}

// Two arrays of n_layers x n_rows rows of w bytes at the same strides, the second `apart` bytes behind the first: does a row
// of one overlap a row of the other?  Rows l2 - l1 layers and r2 - r1 rows apart do when those strides bring `apart` to
// less than w; for each distance in layers the two nearest in rows are looked at.
bool rows_overlap(int64_t apart, int64_t w, int64_t row_stride, int32_t n_rows, int64_t layer_stride, int32_t n_layers) {
    for (int64_t l = 1 - n_layers; l < n_layers; ++l) {
        const int64_t d = apart + l * layer_stride, below = d >= 0 ? d / row_stride : -((-d + row_stride - 1) / row_stride);
        for (int64_t r = below; r <= below + 1; ++r)             // d - r rows: the nearest to 0 from both sides
            if (r > -(int64_t)n_rows && r < n_rows && std::llabs(d - r * row_stride) < w) return true;
    }
    return false;
}

cb_status check_handle(const cb_kv8* c, const char* who) {
    set_last_error("");
    return c ? CB_OK : fail(CB_ERR_INVALID_ARG, "%s: null cache", who);
}

// The handle's device is made current for a call and the caller's put back (the last step before a launch).
struct OnDevice {
    int was = -1;
    bool moved = false;
    cb_status to(const cb_kv8* c, const char* who) {
        if (cudaGetDevice(&was) != cudaSuccess || (was != c->device && cudaSetDevice(c->device) != cudaSuccess)) {
            cudaGetLastError();
            return fail(CB_ERR_CUDA, "%s: the cache's CUDA device %d is not available", who, c->device);
        }
        moved = was != c->device;
        return CB_OK;
    }
    ~OnDevice() {
        if (moved) cudaSetDevice(was);
    }
};

cb_status check_layers(const cb_kv8& c, int32_t layer, int32_t n_layers, const char* who) {
    if (layer < 0 || n_layers < 0 || layer > c.cfg.n_layers - n_layers)
        return fail(CB_ERR_INVALID_ARG, "%s: layers [%d, %d + %d) outside the cache's %d", who, layer, layer, n_layers,
                    c.cfg.n_layers);
    return CB_OK;
}

cb_status check_seqs(const cb_kv8& c, const cb_kv8_seqs* q, const char* who, Kv8Seqs& out) {
    if (!q) return fail(CB_ERR_INVALID_ARG, "%s: null seqs", who);
    if (q->n_seqs < 0 || q->n_seqs > 65535) return fail(CB_ERR_INVALID_ARG, "%s: n_seqs %d outside [0, 65535]", who, q->n_seqs);
    if (q->max_len < 0 || q->max_len > kMaxRows) return fail(CB_ERR_INVALID_ARG, "%s: max_len %d outside [0, 2^30]", who, q->max_len);
    if (q->table_ld < 0 || (int64_t)q->table_ld * c.cfg.page_size < q->max_len)
        return fail(CB_ERR_INVALID_ARG, "%s: max_len %d needs more than the block tables' %d pages of %d rows", who, q->max_len,
                    q->table_ld, c.cfg.page_size);
    if (q->n_seqs > 0 && q->max_len > 0 && !q->table) return fail(CB_ERR_INVALID_ARG, "%s: null block table", who);
    out = Kv8Seqs{q->n_seqs, q->table, q->table_ld, q->lens, q->max_len, c.cfg.n_pages, c.shift, c.status};
    return CB_OK;
}

// rows of the batch: ragged through `start`, or shared evenly
cb_status check_rows(const Kv8Seqs& q, const int32_t* start, int32_t n_rows, const char* who, Kv8Rows& out) {
    if (n_rows < 0 || n_rows > kMaxRows) return fail(CB_ERR_INVALID_ARG, "%s: %d rows outside [0, 2^30]", who, n_rows);
    if (q.n == 0 && n_rows > 0 && !start) return fail(CB_ERR_INVALID_ARG, "%s: %d rows but no sequence", who, n_rows);
    if (!start && q.n > 0 && n_rows % q.n != 0)
        return fail(CB_ERR_INVALID_ARG, "%s: %d rows cannot be shared evenly by %d sequences (give their offsets)", who, n_rows, q.n);
    out = Kv8Rows{start, start || q.n == 0 ? 0 : n_rows / q.n, n_rows};
    return CB_OK;
}

// blocks that a write or a read looks at, counted in 32 bits
cb_status check_blocks(const cb_kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const char* who) {
    if (((int64_t)(r.n_rows >> q.shift) + 2 * (int64_t)q.n) * c.cfg.n_kv_heads > 0x7fffffff - 256)
        return fail(CB_ERR_UNSUPPORTED, "%s: %d rows are too many for one call", who, r.n_rows);
    return CB_OK;
}

cb_status cuda_result(cudaError_t e, const char* who) {
    if (e == cudaSuccess) return CB_OK;
    cudaGetLastError();                                // a refused launch is reported here, not by the caller's next call
    return fail(CB_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

// K and V rows beside the cache: [n_layers][rows][Hkv][hd], 16-byte vectors
cb_status check_io(const cb_kv8& c, const void* k, const void* v, int64_t layer_stride, int64_t row_stride, int32_t n_layers,
                   int32_t n_rows, bool output, const char* who, Kv8Io& io) {
    const int64_t w = (int64_t)c.cfg.n_kv_heads * c.cfg.head_dim, es = c.cfg.dtype == CB_BF16 ? 2 : 4;
    if (!k || !v) return fail(CB_ERR_INVALID_ARG, "%s: null k or v", who);
    if ((uintptr_t)k % 16 || (uintptr_t)v % 16 || row_stride * es % 16 || layer_stride * es % 16)
        return fail(CB_ERR_INVALID_ARG, "%s: k, v and their strides must be multiples of 16 bytes", who);
    if (row_stride < w || (n_layers > 1 && layer_stride < 0) || row_stride > ((int64_t)1 << 40) ||
        layer_stride > ((int64_t)1 << 50))
        return fail(CB_ERR_INVALID_ARG, "%s: row stride %lld below a row's %lld elements, or a stride out of range", who,
                    (long long)row_stride, (long long)w);
    // layers behind each other, or interleaved row by row (what is only read may also be one layer for all)
    const bool apart = layer_stride >= (n_rows - 1) * row_stride + w || (layer_stride >= w && row_stride >= (n_layers - 1) * layer_stride + w);
    if (n_layers > 1 && !apart && (output || layer_stride != 0))
        return fail(CB_ERR_INVALID_ARG, "%s: the layers' rows overlap (layer stride %lld)", who, (long long)layer_stride);
    // (rows that span 2^40 bytes are on no device: of those only the first are compared)
    const int32_t looked = row_stride * es < ((int64_t)1 << 40) / n_rows ? n_rows : 1;
    if (output && rows_overlap((const char*)v - (const char*)k, w * es, row_stride * es, looked, layer_stride * es, n_layers))
        return fail(CB_ERR_INVALID_ARG, "%s: k and v overlap", who);
    io = Kv8Io{const_cast<void*>(k), const_cast<void*>(v), layer_stride, row_stride, c.cfg.dtype == CB_BF16};
    return CB_OK;
}

}  // namespace

extern "C" {

cb_status cb_kv8_create(const cb_kv8_config* cfg, void* codes, float* scales, cb_kv8** out) {
    set_last_error("");
    if (!cfg || !out) return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: null argument");
    *out = nullptr;
    const cb_kv8_config& c = *cfg;
    if (!codes || !scales) return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: null codes or scales");
    if ((uintptr_t)codes % 128 || (uintptr_t)scales % 4)
        return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: codes must be 128-byte aligned, scales 4-byte aligned");
    if (c.n_layers <= 0 || c.n_layers > 1024 || c.n_heads <= 0 || c.n_kv_heads <= 0 || c.head_dim <= 0)
        return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: non-positive dimension, or more than 1024 layers");
    if (c.n_heads % c.n_kv_heads != 0) return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: n_heads must be a multiple of n_kv_heads");
    if (c.head_dim != 64 && c.head_dim != 128) return fail(CB_ERR_UNSUPPORTED, "cb_kv8_create: head_dim must be 64 or 128");
    if (c.n_heads / c.n_kv_heads > 8) return fail(CB_ERR_UNSUPPORTED, "cb_kv8_create: at most 8 query heads per KV head");
    if (c.n_kv_heads > 1024 || 2 * c.n_layers * (int64_t)c.n_kv_heads > 65535)
        return fail(CB_ERR_UNSUPPORTED, "cb_kv8_create: more than 65535 K and V heads over all layers");
    if (c.dtype != CB_F32 && c.dtype != CB_BF16) return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: dtype must be CB_F32 or CB_BF16");
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)))
        return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: page_size %d is not 16, 32, 64, 128 or 256", c.page_size);
    if (c.n_pages <= 0 || c.n_pages * (int64_t)c.page_size * c.n_kv_heads > (int64_t)0x7fffffff || c.n_pages > 0x7fffffff)
        return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: n_pages * page_size * n_kv_heads must be in [1, 2^31)");
    if (c.weight_cells < 0 || c.weight_cells > ((int64_t)1 << 36))
        return fail(CB_ERR_INVALID_ARG, "cb_kv8_create: weight_cells outside [0, 2^36]");
    cb_kv8* h = new (std::nothrow) cb_kv8();
    if (!h) return fail(CB_ERR_OOM, "cb_kv8_create: host allocation failed");
    h->cfg = c;
    h->codes = (uint8_t*)codes;
    h->scales = scales;
    h->shift = 0;
    while ((1 << h->shift) < c.page_size) ++h->shift;
    const char* pdl = getenv("CB_PDL");
    h->pdl = !(pdl && pdl[0] == '0');
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return fail(CB_ERR_CUDA, "cb_kv8_create: no CUDA device");
    }
    // one allocation: status, voided, arrival counts (zero between calls), pieces, statistics, what is to be joined, scores
    const size_t head = 256 + ((size_t)kv8_most_ctas(h->num_sms) * 4 + 255) / 256 * 256;
    const size_t part = (kv8_part_floats(h->num_sms) * 4 + 255) / 256 * 256;
    // a row of a call that returns weights takes at least 129 cells
    const size_t stats = c.weight_cells > 0 ? (((size_t)c.weight_cells / 129 + 1) * sizeof(float2) + 255) / 256 * 256 : 0;
    const size_t todo = ((size_t)h->num_sms * 4 * 4 + 255) / 256 * 256;
    if (cudaMalloc(&h->scratch, head + part + stats + todo + (size_t)c.weight_cells * 4) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return fail(CB_ERR_OOM, "cb_kv8_create: workspace allocation failed");
    }
    char* at = (char*)h->scratch;
    h->status = (unsigned*)at;
    h->voided = (unsigned*)(at + 128);
    h->arrived = (unsigned*)(at + 256);
    h->part = (float*)(at + head);
    h->stats = (float2*)(at + head + part);
    h->todo = (int*)(at + head + part + stats);
    h->scores = (float*)(at + head + part + stats + todo);
    // cleared before the handle is given out, whatever stream its first call uses
    if (!kv8_make_map(*h, h->map) || cudaMemset(h->scratch, 0, head) != cudaSuccess ||
        cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(h->scratch);
        delete h;
        return fail(CB_ERR_CUDA, "cb_kv8_create: no tensor map of the codes, or a device error");
    }
    *out = h;
    return CB_OK;
}

cb_status cb_kv8_destroy(cb_kv8* c) {
    set_last_error("");
    if (!c) return CB_OK;
    OnDevice on;
    if (on.to(c, "cb_kv8_destroy") != CB_OK) return CB_ERR_CUDA;
    cudaDeviceSynchronize();
    cudaFree(c->scratch);
    delete c;
    return CB_OK;
}

cb_status cb_kv8_status(cb_kv8* c, uint32_t* bits, int32_t clear) {
    cb_status st = check_handle(c, "cb_kv8_status");
    if (st != CB_OK) return st;
    if (!bits) return fail(CB_ERR_INVALID_ARG, "cb_kv8_status: null bits");
    OnDevice on;
    st = on.to(c, "cb_kv8_status");
    if (st != CB_OK) return st;
    // (a memset may still run when it returns, and a call's stream need not wait for it)
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(bits, c->status, 4, cudaMemcpyDeviceToHost) != cudaSuccess ||
        (clear && (cudaMemset(c->status, 0, 64) != cudaSuccess || cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess))) {
        cudaGetLastError();
        return fail(CB_ERR_CUDA, "cb_kv8_status: device error");
    }
    return CB_OK;
}

cb_status cb_kv8_write(cb_kv8* c, const cb_kv8_seqs* seqs, int32_t layer, int32_t n_layers, const void* k, const void* v,
                       int64_t layer_stride, int64_t row_stride, const int32_t* row_start, int32_t n_rows, void* stream) {
    const char* who = "cb_kv8_write";
    Kv8Seqs q;
    Kv8Rows r;
    Kv8Io io;
    cb_status st = check_handle(c, who);
    if (st == CB_OK) st = check_layers(*c, layer, n_layers, who);
    if (st == CB_OK) st = check_seqs(*c, seqs, who, q);
    if (st == CB_OK) st = check_rows(q, row_start, n_rows, who, r);
    if (st != CB_OK) return st;
    if (n_rows == 0 || n_layers == 0 || q.n == 0) return CB_OK;
    st = check_blocks(*c, q, r, who);
    if (st == CB_OK) st = check_io(*c, k, v, layer_stride, row_stride, n_layers, n_rows, false, who, io);
    OnDevice on;
    if (st == CB_OK) st = on.to(c, who);
    if (st != CB_OK) return st;
    return cuda_result(launch_kv8_write(*c, q, r, io, layer, n_layers, (cudaStream_t)stream), who);
}

cb_status cb_kv8_read(cb_kv8* c, const cb_kv8_seqs* seqs, int32_t layer, int32_t n_layers, void* k, void* v,
                      int64_t layer_stride, int64_t row_stride, const int32_t* row_start, int32_t n_rows, void* stream) {
    const char* who = "cb_kv8_read";
    Kv8Seqs q;
    Kv8Rows r;
    Kv8Io io;
    cb_status st = check_handle(c, who);
    if (st == CB_OK) st = check_layers(*c, layer, n_layers, who);
    if (st == CB_OK) st = check_seqs(*c, seqs, who, q);
    if (st == CB_OK) st = check_rows(q, row_start, n_rows, who, r);
    if (st != CB_OK) return st;
    if (n_rows == 0 || n_layers == 0 || q.n == 0) return CB_OK;
    st = check_blocks(*c, q, r, who);
    if (st == CB_OK) st = check_io(*c, k, v, layer_stride, row_stride, n_layers, n_rows, true, who, io);
    OnDevice on;
    if (st == CB_OK) st = on.to(c, who);
    if (st != CB_OK) return st;
    return cuda_result(launch_kv8_read(*c, q, r, io, layer, n_layers, (cudaStream_t)stream), who);
}

cb_status cb_kv8_attention(cb_kv8* c, const cb_kv8_seqs* seqs, int32_t layer, const void* q, int64_t q_stride,
                           const int32_t* q_start, int32_t n_q, float scale, void* out, int64_t out_stride, float* weights,
                           int32_t weights_ld, int32_t add, void* stream) {
    const char* who = "cb_kv8_attention";
    Kv8Seqs sq;
    Kv8Rows r;
    cb_status st = check_handle(c, who);
    if (st == CB_OK) st = check_layers(*c, layer, 1, who);
    if (st == CB_OK) st = check_seqs(*c, seqs, who, sq);
    if (st == CB_OK) st = check_rows(sq, q_start, n_q, who, r);
    if (st != CB_OK) return st;
    const int64_t w = (int64_t)c->cfg.n_heads * c->cfg.head_dim, es = c->cfg.dtype == CB_BF16 ? 2 : 4;
    if (!std::isfinite(scale)) return fail(CB_ERR_INVALID_ARG, "%s: scale is not finite", who);
    if (n_q > 0) {
        if (!q || !out) return fail(CB_ERR_INVALID_ARG, "%s: null q or out", who);
        if ((uintptr_t)q % 16 || (uintptr_t)out % 16 || q_stride * es % 16 || out_stride * es % 16)
            return fail(CB_ERR_INVALID_ARG, "%s: q, out and their strides must be multiples of 16 bytes", who);
        if (q_stride < w || out_stride < w || q_stride > ((int64_t)1 << 40) || out_stride > ((int64_t)1 << 40))
            return fail(CB_ERR_INVALID_ARG, "%s: a row stride below a row's %lld elements, or out of range", who, (long long)w);
        if (overlap(q, ((n_q - 1) * q_stride + w) * es, out, ((n_q - 1) * out_stride + w) * es))
            return fail(CB_ERR_INVALID_ARG, "%s: q and out overlap", who);
    }
    if (weights) {
        if (weights_ld < sq.max_len) return fail(CB_ERR_INVALID_ARG, "%s: weights_ld %d below max_len %d", who, weights_ld, sq.max_len);
        const int64_t row = (((int64_t)sq.max_len + 127) / 128) * 128 + 1, rows = (int64_t)n_q * c->cfg.n_heads;
        if (sq.max_len > 0 && rows > c->cfg.weight_cells / row)          // (rows * row may pass 64 bits)
            return fail(CB_ERR_INVALID_ARG, "%s: returning weights needs %.0f cells, the cache was created with %lld", who,
                        (double)rows * (double)row, (long long)c->cfg.weight_cells);
    }
    // tiles of 128 keys and at least one query row, of every KV head, and what an item counts besides
    if (((int64_t)n_q + sq.n) * c->cfg.n_kv_heads > 0x7fffffff / ((int64_t)sq.max_len / 128 + 8))
        return fail(CB_ERR_UNSUPPORTED, "%s: %d query rows over %d keys are too many for one call", who, n_q, sq.max_len);
    if (sq.n == 0 || (n_q == 0 && !weights)) return CB_OK;
    OnDevice on;
    st = on.to(c, who);
    if (st != CB_OK) return st;
    const Kv8Attn a{q, q_stride, out, out_stride, scale, weights, weights_ld, add != 0};
    return cuda_result(launch_kv8_attention(*c, sq, r, a, layer, (cudaStream_t)stream), who);
}

cb_status cb_kv8_evict(cb_kv8* c, const cb_kv8_seqs* seqs, const int32_t* dst_table, int32_t dst_ld, int32_t layer,
                       int32_t n_layers, const float* weights, int32_t weights_ld, int32_t n_keep, int32_t n_sink,
                       int32_t n_recent, float* out_weights, int32_t* out_rows, int32_t* out_lens, void* stream) {
    const char* who = "cb_kv8_evict";
    Kv8Seqs q;
    cb_status st = check_handle(c, who);
    if (st == CB_OK) st = check_layers(*c, layer, n_layers, who);
    if (st == CB_OK) st = check_seqs(*c, seqs, who, q);
    if (st != CB_OK) return st;
    if (n_keep <= 0 || n_sink < 0 || n_recent < 0 || n_sink > n_keep - n_recent)
        return fail(CB_ERR_INVALID_ARG, "%s: need n_keep > 0 and n_sink + n_recent <= n_keep (%d, %d, %d)", who, n_keep, n_sink,
                    n_recent);
    if (q.n == 0 || n_layers == 0) return CB_OK;
    if (!dst_table || !weights || !out_weights || !out_rows || !out_lens)
        return fail(CB_ERR_INVALID_ARG, "%s: null destination table, weights or output", who);
    const int most = n_keep < q.max_len ? n_keep : q.max_len;
    if ((int64_t)dst_ld * c->cfg.page_size < most)
        return fail(CB_ERR_INVALID_ARG, "%s: the destination tables' %d pages hold fewer than %d rows", who, dst_ld, most);
    // one table at two widths would be evicted in place by CTAs that take it for two tables
    const int64_t src_end = ((int64_t)(q.n - 1) * q.table_ld + (q.max_len + c->cfg.page_size - 1) / c->cfg.page_size) * 4;
    const int64_t dst_end = ((int64_t)(q.n - 1) * dst_ld + (most + c->cfg.page_size - 1) / c->cfg.page_size) * 4;
    const bool same = dst_table == q.table && (dst_ld == q.table_ld || q.n == 1);
    if (!same && overlap(dst_table, dst_end, q.table, src_end))
        return fail(CB_ERR_INVALID_ARG, "%s: dst_table overlaps the sequences' table without being the same", who);
    if (weights_ld < q.max_len) return fail(CB_ERR_INVALID_ARG, "%s: weights_ld %d below max_len %d", who, weights_ld, q.max_len);
    const int64_t cells = (int64_t)n_layers * q.n * c->cfg.n_kv_heads * weights_ld * 4;
    if (weights != out_weights && overlap(weights, cells, out_weights, cells))
        return fail(CB_ERR_INVALID_ARG, "%s: weights and out_weights overlap without being the same", who);
    OnDevice on;
    st = on.to(c, who);
    if (st != CB_OK) return st;
    const Kv8Evict e{dst_table, same ? q.table_ld : dst_ld, weights, out_weights, weights_ld, n_keep, n_sink, n_recent, out_rows, out_lens};
    return cuda_result(launch_kv8_evict(*c, q, e, layer, n_layers, (cudaStream_t)stream), who);
}

}  // extern "C"
