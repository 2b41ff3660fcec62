// Host side of the paged 8-bit cache's C ABI (kv8_*): handles, argument checks,
// launches. Every call runs on the handle's device, whichever is current.
#include <atomic>
#include <cmath>
#include <cstdio>
#include <new>

#include "kv8_internal.cuh"

using namespace srh;
using kv8::Cache;

namespace {

thread_local char g_create_error[256] = {0};

int fail(kv8_cache* c, int code, const char* msg) {
    std::snprintf(c ? c->last_error : g_create_error, 256, "%s", msg);
    return code;
}
int cuda_fail(kv8_cache* c, cudaError_t e, const char* where) {
    std::snprintf(c ? c->last_error : g_create_error, 256, "%s: %s", where, cudaGetErrorString(e));
    return SRH_ERR_CUDA;
}

// The handle's device for the time of a call.
struct OnDevice {
    int before = -1;
    cudaError_t err = cudaSuccess;
    explicit OnDevice(int device) {
        int now = -1;
        err = cudaGetDevice(&now);
        if (err == cudaSuccess && now != device) {
            err = cudaSetDevice(device);
            if (err == cudaSuccess) before = now;
        }
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};
#define KV8_DEVICE(c)                                                          \
    OnDevice on_device_((c)->device);                                          \
    if (on_device_.err != cudaSuccess) return cuda_fail((c), on_device_.err, "cudaSetDevice")

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Row stride of an input (0 repeats one row) or of an output (rows apart).
bool row_ok(long long stride, long long width, long long rows, bool out) {
    if (stride < 0 || stride % 8) return false;
    return !out || rows <= 1 || stride >= width;
}

// Rows of bf16 values in memory.
struct Rows {
    const uint16_t* p;
    long long stride, n, width;      // elements, rows, elements
};
// Whether any row of a shares memory with a row of b. Rows of one stride may lie between
// each other's; of different strides, ranges that cross count as shared.
bool meet(const Rows& a, const Rows& b) {
    using Wide = unsigned __int128;
    if (a.n < 1 || b.n < 1) return false;
    if (reinterpret_cast<uintptr_t>(a.p) > reinterpret_cast<uintptr_t>(b.p)) return meet(b, a);
    const uint64_t apart = (reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) / sizeof(uint16_t);
    if (apart >= (Wide)(a.n - 1) * (Wide)a.stride + (Wide)a.width) return false;
    if (a.n == 1) return true;
    if (b.n > 1 && b.stride != a.stride) return true;
    if (a.stride == 0) return true;
    // b's first row begins `d` behind a row of a; a's next one may reach into it
    const uint64_t d = apart % (uint64_t)a.stride, before = apart / (uint64_t)a.stride;
    if (d < (uint64_t)a.width) return true;
    return d + (uint64_t)b.width > (uint64_t)a.stride && before + 1 < (uint64_t)a.n;
}

const char* config_error(const kv8_config* k) {
    if (!k) return "config is NULL";
    if (k->batch < 1 || k->batch > kv8::kMaxBatch) return "batch must be in [1, 4096]";
    if (k->n_kv_heads < 1 || k->n_kv_heads > 256) return "n_kv_heads must be in [1, 256]";
    if (k->head_dim != 128 && k->head_dim != 256 && k->head_dim != 512) return "head_dim must be 128, 256 or 512";
    if (k->block_tokens != 16 && k->block_tokens != 32 && k->block_tokens != 64 && k->block_tokens != 128)
        return "block_tokens must be 16, 32, 64 or 128";
    if (k->n_blocks < 1) return "n_blocks must be >= 1";
    if (k->max_blocks < 1 || (long long)k->max_blocks * k->block_tokens > (1ll << 30))
        return "max_blocks must be >= 1 and max_blocks * block_tokens <= 2^30";
    if (k->shared_kv != 0 && k->shared_kv != 1) return "shared_kv must be 0 or 1";
    const long long dense = (long long)k->n_kv_heads * k->block_tokens * k->head_dim;
    if (k->block_stride != 0 && (k->block_stride < dense || k->block_stride % 16 || k->block_stride >= (1ll << 39)))
        return "block_stride must be 0 or a multiple of 16 that holds a block";
    return nullptr;
}

const char* pool_error(const kv8_cache* c, const kv8_pool* p) {
    if (!p || !p->k_codes || !p->k_scale) return "pool pointers must not be NULL";
    if (!aligned(p->k_codes, 16) || !aligned(p->k_scale, 4)) return "codes must be 16-byte aligned, scales 4-byte";
    if (c->cfg.shared_kv) return nullptr;
    if (!p->v_codes || !p->v_scale) return "pool pointers must not be NULL";
    if (!aligned(p->v_codes, 16) || !aligned(p->v_scale, 4)) return "codes must be 16-byte aligned, scales 4-byte";
    return nullptr;
}

bool takes_4_bits(const kv8_config& k) { return !k.shared_kv && k.head_dim <= 256; }

// A 4-bit pool of this handle; null where it is sound.
const char* pool4_error(const kv8_cache* c, const kv4_pool* p) {
    if (!takes_4_bits(c->cfg)) return "4 bits are for 128- and 256-dim heads with K and V apart";
    if (!p || !p->k_codes || !p->k_scale || !p->v_codes || !p->v_scale) return "pool pointers must not be NULL";
    if (!aligned(p->k_codes, 16) || !aligned(p->v_codes, 16) || !aligned(p->k_scale, 16) || !aligned(p->v_scale, 16))
        return "codes and scales must be 16-byte aligned";
    const long long dense = (long long)c->cfg.n_kv_heads * c->cfg.block_tokens * c->cfg.head_dim / 2;
    if (p->block_stride != 0 && (p->block_stride < dense || p->block_stride % 16 || p->block_stride >= (1ll << 39)))
        return "block_stride must be 0 or a multiple of 16 that holds a block";
    return nullptr;
}
long long stride4(const kv8_cache* c, const kv4_pool* p) {
    return p->block_stride ? p->block_stride : (long long)c->cfg.n_kv_heads * c->cfg.block_tokens * c->cfg.head_dim / 2;
}

const char* heads_error(const kv8_heads& h, int n_tok, int head_dim) {
    if (h.n_heads < 0 || h.n_heads > 1024) return "n_heads must be in [0, 1024]";
    if (h.n_heads == 0) return nullptr;
    if (!h.x || !h.out) return "NULL pointer";
    if (!aligned(h.x, 16) || !aligned(h.out, 16) || !aligned(h.weight, 16)) return "x, out and weight must be 16-byte aligned";
    const long long width = (long long)h.n_heads * head_dim;
    if (!row_ok(h.x_row, width, n_tok, false) || !row_ok(h.out_row, width, h.slot ? h.n_slots : n_tok, true))
        return "row strides must be multiples of 8 (outputs' at least a row)";
    if (h.slot && (h.n_slots < 0 || !aligned(h.slot, 8))) return "n_slots must be >= 0, slots 8-byte aligned";
    if (h.out == h.x && (h.slot || h.x_row != h.out_row)) return "in place needs the same row stride and no slots";
    return nullptr;
}
// Outputs of `h` on rows that anything else of the call reads or writes.
const char* overlap_error(const kv8_heads& h, const kv8_heads& other, int n_tok, int head_dim) {
    if (h.n_heads == 0) return nullptr;
    const long long n_out = h.slot ? h.n_slots : n_tok;
    const Rows out{h.out, h.out_row, n_out, (long long)h.n_heads * head_dim};
    if (h.out != h.x && meet(out, {h.x, h.x_row, n_tok, out.width})) return "out overlaps x without being x";
    if (other.n_heads == 0) return nullptr;
    const long long width = (long long)other.n_heads * head_dim;
    if (meet(out, {other.x, other.x_row, n_tok, width}) ||
        meet(out, {other.out, other.out_row, other.slot ? other.n_slots : n_tok, width}))
        return "the outputs of one kind of heads overlap the other's rows";
    return nullptr;
}

}  // namespace

extern "C" {

int kv8_create(const kv8_config* cfg, kv8_cache** out) {
    if (!out) return fail(nullptr, SRH_ERR_INVALID, "out is NULL");
    *out = nullptr;
    if (const char* why = config_error(cfg)) return fail(nullptr, SRH_ERR_INVALID, why);
    kv8_cache* c = new (std::nothrow) kv8_cache();
    if (!c) return fail(nullptr, SRH_ERR_NOMEM, "host allocation failed");
    c->cfg = *cfg;
    while ((1 << c->bs_log2) < cfg->block_tokens) ++c->bs_log2;
    c->d_blocks = cfg->head_dim / 128;
    c->block_stride = cfg->block_stride ? cfg->block_stride
                                        : (long long)cfg->n_kv_heads * cfg->block_tokens * cfg->head_dim;
    const char* where = "cudaGetDevice";
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device);
    if (e == cudaSuccess) {
        // once per device: 18 calls of a few microseconds
        static std::atomic<uint64_t> set{0};
        const uint64_t bit = c->device < 64 ? 1ull << c->device : 0;
        where = "kernel attributes";
        if (!bit || !(set.load() & bit)) {
            e = kv8::set_attend_attrs();
            if (e == cudaSuccess) e = kv8::set_resize_attrs();
            if (e == cudaSuccess) e = kv8::set_attend4_attrs();
            if (e == cudaSuccess) set.fetch_or(bit);
        }
    }
    if (e == cudaSuccess) {
        where = "device scratch";
        kv8::attend_scratch(c->sm_count, cfg->head_dim, &c->part_o_floats, &c->part_ml_floats, &c->meta_n);
        if (takes_4_bits(*cfg)) {
            size_t o = 0, ml = 0, meta = 0;
            kv8::attend4_scratch(c->sm_count, &o, &ml, &meta, &c->arrived_n);
            if (o > c->part_o_floats) c->part_o_floats = o;
            if (ml > c->part_ml_floats) c->part_ml_floats = ml;
            if (meta > c->meta_n) c->meta_n = meta;
        }
        e = cudaMalloc(&c->d_err, sizeof(uint32_t));
        if (e == cudaSuccess) e = cudaMemset(c->d_err, 0, sizeof(uint32_t));
        if (e == cudaSuccess) e = cudaMalloc(&c->d_part_o, c->part_o_floats * sizeof(float));
        if (e == cudaSuccess) e = cudaMalloc(&c->d_part_ml, c->part_ml_floats * sizeof(float));
        if (e == cudaSuccess) e = cudaMalloc(&c->d_meta, c->meta_n * sizeof(int4));
        if (e == cudaSuccess) e = cudaMalloc(&c->d_ctrl, 2 * sizeof(int));
        if (e == cudaSuccess) e = cudaMemset(c->d_ctrl, 0, 2 * sizeof(int));
        if (c->arrived_n) {
            if (e == cudaSuccess) e = cudaMalloc(&c->d_arrived, c->arrived_n * sizeof(int));
            if (e == cudaSuccess) e = cudaMemset(c->d_arrived, 0, c->arrived_n * sizeof(int));
        }
        // the clears run on the legacy stream, which streams that do not block do not wait for
        if (e == cudaSuccess) e = cudaStreamSynchronize(0);
    }
    if (e != cudaSuccess) {
        const int rc = e == cudaErrorMemoryAllocation ? SRH_ERR_NOMEM : SRH_ERR_CUDA;
        cuda_fail(nullptr, e, where);
        kv8_destroy(c);
        return rc;
    }
    *out = c;
    return SRH_OK;
}

void kv8_destroy(kv8_cache* c) {
    if (!c) return;
    {
        OnDevice on(c->device);
        if (c->d_err) cudaDeviceSynchronize();
        cudaFree(c->d_err);
        cudaFree(c->d_part_o);
        cudaFree(c->d_part_ml);
        cudaFree(c->d_meta);
        cudaFree(c->d_ctrl);
        cudaFree(c->d_arrived);
    }
    delete c;
}

int kv8_resize(kv8_cache* c, const int32_t* d_new_len, int n_req, int32_t* d_len, int32_t* d_table, int32_t* d_free,
               int32_t* d_n_free, int32_t* d_cu, int32_t* d_pos, int64_t* d_slot, int cap, srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (!d_new_len || !d_len || !d_table || !d_free || !d_n_free || !d_cu) return fail(c, SRH_ERR_INVALID, "NULL pointer");
    if (n_req < 1 || n_req > c->cfg.batch) return fail(c, SRH_ERR_INVALID, "n_req must be in [1, batch]");
    if (cap < 0 || !d_pos != !d_slot || (!d_pos && cap))
        return fail(c, SRH_ERR_INVALID, "d_pos and d_slot come together, with cap >= 0 (0 without them)");
    if (!aligned(d_slot, 8)) return fail(c, SRH_ERR_INVALID, "slots must be 8-byte aligned");
    KV8_DEVICE(c);
    const cudaError_t e = kv8::launch_resize(*c, d_new_len, n_req, d_len, d_table, d_free, d_n_free, d_cu, d_pos, d_slot,
                                             cap, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, "kv8_resize launch");
}

static int norm_rope(kv8_cache* c, const kv8_heads* q, const kv8_heads* k, int n_tok, int head_dim, const int32_t* d_pos,
                     long long pos_row, int n_axes, const uint8_t* d_axis, const double* d_inv_freq, int rot_dim, int rot_off,
                     int style, float eps, srh_stream_t stream) {
    if (!q && !k) return fail(c, SRH_ERR_INVALID, "no heads");
    const kv8_heads none{};
    const kv8_heads a = q ? *q : none, b = k ? *k : none;
    if (n_tok < 0) return fail(c, SRH_ERR_INVALID, "n_tok must be >= 0");
    if (head_dim < 8 || head_dim > 512 || head_dim % 8)
        return fail(c, SRH_ERR_INVALID, "head_dim must be a multiple of 8 in [8, 512]");
    if (rot_dim < 0 || rot_off < 0 || rot_dim % 16 || rot_off % 8 || rot_dim > head_dim - rot_off)
        return fail(c, SRH_ERR_INVALID, "rot_dim must be a multiple of 16, rot_off of 8, both within head_dim");
    if (style != KV8_ROPE_PAIRS && style != KV8_ROPE_HALVES) return fail(c, SRH_ERR_INVALID, "unknown rotation style");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(c, SRH_ERR_INVALID, "eps must be finite and >= 0");
    for (const kv8_heads* h : {&a, &b})
        if (const char* why = heads_error(*h, n_tok, head_dim)) return fail(c, SRH_ERR_INVALID, why);
    if (a.n_heads + b.n_heads < 1) return fail(c, SRH_ERR_INVALID, "no heads");
    if (rot_dim && (!d_pos || !d_inv_freq || !aligned(d_pos, 4) || !aligned(d_inv_freq, 8)))
        return fail(c, SRH_ERR_INVALID, "d_pos and d_inv_freq must not be NULL, and aligned");
    if (n_tok == 0) return SRH_OK;
    if (const char* why = overlap_error(a, b, n_tok, head_dim)) return fail(c, SRH_ERR_INVALID, why);
    if (const char* why = overlap_error(b, a, n_tok, head_dim)) return fail(c, SRH_ERR_INVALID, why);
    KV8_DEVICE(c);
    const cudaError_t e = kv8::launch_norm_rope(*c, a, b, n_tok, head_dim, d_pos, pos_row, n_axes, d_axis, d_inv_freq,
                                                rot_dim, rot_off, style, eps, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, "kv8_norm_rope launch");
}

int kv8_norm_rope(kv8_cache* c, const kv8_heads* q, const kv8_heads* k, int n_tok, int head_dim, const int32_t* d_pos,
                  const double* d_inv_freq, int rot_dim, int rot_off, int style, float eps, srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    return norm_rope(c, q, k, n_tok, head_dim, d_pos, 0, 1, nullptr, d_inv_freq, rot_dim, rot_off, style, eps, stream);
}

int kv8_norm_rope_axes(kv8_cache* c, const kv8_heads* q, const kv8_heads* k, int n_tok, int head_dim, const int32_t* d_pos,
                       long long pos_row, int n_axes, const uint8_t* d_axis, const double* d_inv_freq, int rot_dim,
                       int rot_off, int style, float eps, srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (n_axes < 1 || n_axes > 8) return fail(c, SRH_ERR_INVALID, "n_axes must be in [1, 8]");
    if (pos_row != 0 && pos_row < n_tok) return fail(c, SRH_ERR_INVALID, "pos_row must be 0 or at least n_tok");
    if (rot_dim && !d_axis) return fail(c, SRH_ERR_INVALID, "d_axis must not be NULL");
    return norm_rope(c, q, k, n_tok, head_dim, d_pos, pos_row, n_axes, d_axis, d_inv_freq, rot_dim, rot_off, style, eps, stream);
}

int kv8_append(kv8_cache* c, const kv8_pool* pool, const int32_t* d_table, const int32_t* d_len, const int32_t* d_cu,
               int n_req, const uint16_t* d_k, long long k_row, const uint16_t* d_v, long long v_row, int n_rows,
               srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (const char* why = pool_error(c, pool)) return fail(c, SRH_ERR_INVALID, why);
    if (n_req < 1 || n_req > c->cfg.batch) return fail(c, SRH_ERR_INVALID, "n_req must be in [1, batch]");
    if (n_rows < 0) return fail(c, SRH_ERR_INVALID, "n_rows must be >= 0");
    if (n_rows == 0) return SRH_OK;
    const bool sep = !c->cfg.shared_kv;
    if (!d_table || !d_len || !d_cu || !d_k || (sep && !d_v)) return fail(c, SRH_ERR_INVALID, "NULL pointer");
    if (!aligned(d_k, 16) || (sep && !aligned(d_v, 16))) return fail(c, SRH_ERR_INVALID, "rows must be 16-byte aligned");
    if (!row_ok(k_row, 0, n_rows, false) || (sep && !row_ok(v_row, 0, n_rows, false)))
        return fail(c, SRH_ERR_INVALID, "row strides must be multiples of 8, >= 0");
    KV8_DEVICE(c);
    const cudaError_t e = kv8::launch_append(*c, *pool, d_table, d_len, d_cu, n_req, d_k, k_row, sep ? d_v : d_k,
                                             sep ? v_row : k_row, n_rows, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, "kv8_append launch");
}

// What kv8_attend and kv4_attend are given, but for the pool; *none: there are no rows.
static int attend_args(kv8_cache* c, const int32_t* d_table, const int32_t* d_len, const int32_t* d_cu, int n_req,
                       const uint16_t* d_q, long long q_row, int n_rows, int n_heads, float scale, int window,
                       uint16_t* d_out, long long out_row, bool* none) {
    if (n_req < 1 || n_req > c->cfg.batch) return fail(c, SRH_ERR_INVALID, "n_req must be in [1, batch]");
    if (n_rows < 0) return fail(c, SRH_ERR_INVALID, "n_rows must be >= 0");
    if (n_heads < 1 || n_heads % c->cfg.n_kv_heads) return fail(c, SRH_ERR_INVALID, "n_heads must be a multiple of n_kv_heads");
    if ((long long)n_rows * n_heads > (1ll << 30)) return fail(c, SRH_ERR_INVALID, "n_rows * n_heads must be <= 2^30");
    if (!std::isfinite(scale)) return fail(c, SRH_ERR_INVALID, "scale must be finite");
    if (window < 0) return fail(c, SRH_ERR_INVALID, "window must be >= 0");
    if (n_rows == 0) {
        *none = true;
        return SRH_OK;
    }
    if (!d_table || !d_len || !d_cu || !d_q || !d_out) return fail(c, SRH_ERR_INVALID, "NULL pointer");
    if (!aligned(d_q, 16) || !aligned(d_out, 16)) return fail(c, SRH_ERR_INVALID, "q and out must be 16-byte aligned");
    const long long width = (long long)n_heads * c->cfg.head_dim;
    if (!row_ok(q_row, width, n_rows, false) || !row_ok(out_row, width, n_rows, true))
        return fail(c, SRH_ERR_INVALID, "row strides must be multiples of 8 (the output's at least a row)");
    if (meet({d_q, q_row, n_rows, width}, {d_out, out_row, n_rows, width}))
        return fail(c, SRH_ERR_INVALID, "out must not overlap q");
    return SRH_OK;
}

int kv8_attend(kv8_cache* c, const kv8_pool* pool, const int32_t* d_table, const int32_t* d_len, const int32_t* d_cu,
               int n_req, const uint16_t* d_q, long long q_row, int n_rows, int n_heads, float scale, int window,
               uint16_t* d_out, long long out_row, srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (const char* why = pool_error(c, pool)) return fail(c, SRH_ERR_INVALID, why);
    bool none = false;
    if (const int rc = attend_args(c, d_table, d_len, d_cu, n_req, d_q, q_row, n_rows, n_heads, scale, window, d_out, out_row,
                                   &none))
        return rc;
    if (none) return SRH_OK;
    KV8_DEVICE(c);
    const cudaError_t e = kv8::launch_attend(*c, *pool, d_table, d_len, d_cu, n_req, d_q, q_row, n_rows, n_heads, scale,
                                             window, d_out, out_row, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, "kv8_attend launch");
}

int kv4_attend(kv8_cache* c, const kv4_pool* pool, const int32_t* d_table, const int32_t* d_len, const int32_t* d_cu,
               int n_req, const uint16_t* d_q, long long q_row, int n_rows, int n_heads, float scale, int window,
               uint16_t* d_out, long long out_row, srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (const char* why = pool4_error(c, pool)) return fail(c, SRH_ERR_INVALID, why);
    bool none = false;
    if (const int rc = attend_args(c, d_table, d_len, d_cu, n_req, d_q, q_row, n_rows, n_heads, scale, window, d_out, out_row,
                                   &none))
        return rc;
    if (none) return SRH_OK;
    KV8_DEVICE(c);
    kv4_pool p = *pool;
    p.block_stride = stride4(c, pool);
    const cudaError_t e = kv8::launch_attend4(*c, p, d_table, d_len, d_cu, n_req, d_q, q_row, n_rows, n_heads, scale, window,
                                              d_out, out_row, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, "kv4_attend launch");
}

int kv4_append(kv8_cache* c, const kv4_pool* pool, const int32_t* d_table, const int32_t* d_len, const int32_t* d_cu,
               int n_req, const uint16_t* d_k, long long k_row, const uint16_t* d_v, long long v_row, int n_rows,
               srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (const char* why = pool4_error(c, pool)) return fail(c, SRH_ERR_INVALID, why);
    if (n_req < 1 || n_req > c->cfg.batch) return fail(c, SRH_ERR_INVALID, "n_req must be in [1, batch]");
    if (n_rows < 0) return fail(c, SRH_ERR_INVALID, "n_rows must be >= 0");
    if (n_rows == 0) return SRH_OK;
    if (!d_table || !d_len || !d_cu || !d_k || !d_v) return fail(c, SRH_ERR_INVALID, "NULL pointer");
    if (!aligned(d_k, 16) || !aligned(d_v, 16)) return fail(c, SRH_ERR_INVALID, "rows must be 16-byte aligned");
    if (!row_ok(k_row, 0, n_rows, false) || !row_ok(v_row, 0, n_rows, false))
        return fail(c, SRH_ERR_INVALID, "row strides must be multiples of 8, >= 0");
    KV8_DEVICE(c);
    const kv8::Layer l{{{pool->k_codes, pool->k_scale, const_cast<uint16_t*>(d_k), k_row},
                        {pool->v_codes, pool->v_scale, const_cast<uint16_t*>(d_v), v_row}},
                       2, 4, stride4(c, pool)};
    const cudaError_t e = kv8::launch_append4(*c, l, d_table, d_len, d_cu, n_req, n_rows, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, "kv4_append launch");
}

// kv8_read and kv4_read, their pools checked.
static int read_rows(kv8_cache* c, kv8::Layer l, const int32_t* d_table, const int32_t* d_len, const int32_t* d_start,
                     const int32_t* d_cu, int n_req, int n_rows, srh_stream_t stream, const char* where) {
    if (n_req < 1 || n_req > c->cfg.batch) return fail(c, SRH_ERR_INVALID, "n_req must be in [1, batch]");
    if (n_rows < 0) return fail(c, SRH_ERR_INVALID, "n_rows must be >= 0");
    if (n_rows == 0) return SRH_OK;
    if (!d_table || !d_len || !d_start || !d_cu) return fail(c, SRH_ERR_INVALID, "NULL pointer");
    const long long width = (long long)c->cfg.n_kv_heads * c->cfg.head_dim;
    for (int i = 0; i < l.parts; ++i) {
        if (!l.part[i].x) return fail(c, SRH_ERR_INVALID, "NULL pointer");
        if (!aligned(l.part[i].x, 16)) return fail(c, SRH_ERR_INVALID, "rows must be 16-byte aligned");
        if (!row_ok(l.part[i].x_row, width, n_rows, true))
            return fail(c, SRH_ERR_INVALID, "row strides must be multiples of 8, at least a row");
    }
    if (l.parts == 2 && meet({l.part[0].x, l.part[0].x_row, n_rows, width}, {l.part[1].x, l.part[1].x_row, n_rows, width}))
        return fail(c, SRH_ERR_INVALID, "rows of K and V must not overlap");
    KV8_DEVICE(c);
    const cudaError_t e = kv8::launch_read(*c, l, d_table, d_len, d_start, d_cu, n_req, n_rows, (cudaStream_t)stream);
    return e == cudaSuccess ? SRH_OK : cuda_fail(c, e, where);
}

int kv8_read(kv8_cache* c, const kv8_pool* pool, const int32_t* d_table, const int32_t* d_len, const int32_t* d_start,
             const int32_t* d_cu, int n_req, uint16_t* d_k, long long k_row, uint16_t* d_v, long long v_row, int n_rows,
             srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (const char* why = pool_error(c, pool)) return fail(c, SRH_ERR_INVALID, why);
    return read_rows(c, {{{pool->k_codes, pool->k_scale, d_k, k_row}, {pool->v_codes, pool->v_scale, d_v, v_row}},
                         c->cfg.shared_kv ? 1 : 2, 8, c->block_stride},
                     d_table, d_len, d_start, d_cu, n_req, n_rows, stream, "kv8_read launch");
}

int kv4_read(kv8_cache* c, const kv4_pool* pool, const int32_t* d_table, const int32_t* d_len, const int32_t* d_start,
             const int32_t* d_cu, int n_req, uint16_t* d_k, long long k_row, uint16_t* d_v, long long v_row, int n_rows,
             srh_stream_t stream) {
    if (!c) return SRH_ERR_INVALID;
    if (const char* why = pool4_error(c, pool)) return fail(c, SRH_ERR_INVALID, why);
    return read_rows(c, {{{pool->k_codes, pool->k_scale, d_k, k_row}, {pool->v_codes, pool->v_scale, d_v, v_row}}, 2, 4,
                         stride4(c, pool)},
                     d_table, d_len, d_start, d_cu, n_req, n_rows, stream, "kv4_read launch");
}

int kv8_check_error(kv8_cache* c) {
    if (!c) return SRH_ERR_INVALID;
    KV8_DEVICE(c);
    uint32_t w = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&w, c->d_err, sizeof w, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(c->d_err, 0, sizeof w);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(c, e, "kv8_check_error");
    if (w & kv8::kErrNoBlocks) return fail(c, SRH_ERR_NOMEM, "too few free blocks; the call changed nothing");
    if (w & kErrBounds) return fail(c, SRH_ERR_BOUNDS, "a length, table entry, cu value or slot was out of bounds");
    if (w & kErrTimeout) return fail(c, SRH_ERR_TIMEOUT, "a device wait timed out");
    if (w & kErrRange) return fail(c, SRH_ERR_RANGE, "an appended value is not finite or too large (448 * 2^64 in 8 bits, 2^120 in 4)");
    return SRH_OK;
}

const char* kv8_last_error(kv8_cache* c) { return c ? c->last_error : g_create_error; }

}  // extern "C"
