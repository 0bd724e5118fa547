// C-ABI entry points of the decoder block's operators (declarations and
// contracts in include/igemm_decoder.h): the host gates, the launch plans and
// the workspaces.  Every step of the computation runs in the kernels of
// layer_norm.hpp, rows_i8.hpp, linear_i8.hpp, kv_cache.hpp and cache_attn.hpp.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "decoder_host.hpp"
#include "host_checks.hpp"
#include "igemm_decoder.h"

namespace {

using namespace igc;

// Rows [n0, n1, n2] of d elements of `eb` bytes behind a view whose strides
// and pointer are multiples of `align` bytes.
struct Rows {
    const void* p;
    int64_t s[3];   // bytes; 0 for axes of one entry
    size_t bytes;   // first to last element
};

int32_t check_rows(const igc_attn_view& v, const int64_t n[3], int64_t d, int64_t eb,
                   int64_t align, bool write, Rows* out) {
    Rows x{v.data, {v.batch, v.token, v.head}, 0};
    if (n[0] == 0 || n[1] == 0 || n[2] == 0 || d == 0) {
        *out = x;
        return IGC_OK;
    }
    if (!v.data) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(v.data, (uintptr_t)align)) return IGC_DECLINE_ALIGNMENT;
    double extent = 0;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) x.s[i] = 0;
        if (x.s[i] < 0) return IGC_DECLINE_STRIDE;
        if (x.s[i] * eb % align) return IGC_DECLINE_ALIGNMENT;
        if (x.s[i] >= kBatchStrideLim) return IGC_DECLINE_SIZE_LIMIT;
        extent += (double)n[i] * (double)x.s[i];
    }
    if (extent > kExtentLim) return IGC_DECLINE_SIZE_LIMIT;
    if (write) {
        // axes from the smallest stride up: each has to step over all before
        int ord[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (x.s[ord[j]] < x.s[ord[i]]) {
                    const int t = ord[i];
                    ord[i] = ord[j];
                    ord[j] = t;
                }
        int64_t ext = d;
        for (int i = 0; i < 3; ++i) {
            const int k = ord[i];
            if (n[k] == 1) continue;
            if (x.s[k] < ext) return IGC_DECLINE_OVERLAP;
            ext += (n[k] - 1) * x.s[k];
        }
    }
    int64_t last = d;
    for (int i = 0; i < 3; ++i) {
        last += (n[i] - 1) * x.s[i];
        x.s[i] *= eb;
    }
    x.bytes = (size_t)(last * eb);
    *out = x;
    return IGC_OK;
}

bool same_rows(const Rows& a, const Rows& b) {
    return a.p == b.p && a.s[0] == b.s[0] && a.s[1] == b.s[1] && a.s[2] == b.s[2];
}

// Axis sizes with a single stride over the rows of each of the tensors, where
// they have one.
bool one_stride(const int64_t n[3], const Rows* const* t, int count) {
    for (int i = 0; i < count; ++i) {
        const int64_t s2 = t[i]->s[2], s1 = n[2] == 1 ? t[i]->s[1] : s2 * n[2];
        if (n[2] == 1 && n[1] == 1) continue;   // stride s[0], if any
        if (n[1] > 1 && t[i]->s[1] != s1) return false;
        if (n[0] > 1 && t[i]->s[0] != s1 * n[1]) return false;
    }
    return true;
}
int64_t flat_stride(const int64_t n[3], const Rows& t) {
    return n[2] > 1 ? t.s[2] : n[1] > 1 ? t.s[1] : t.s[0];
}

// A workspace of `need` bytes: the caller's, or one of the stream's.
struct Workspace {
    void* p = nullptr;
    void* own = nullptr;
    hipError_t take(void* given, size_t need, hipStream_t st) {
        p = given;
        if (p || !need) return hipSuccess;
        const hipError_t e = hipMallocAsync(&own, need, st);
        p = own;
        return e;
    }
    hipError_t release(hipStream_t st) { return own ? hipFreeAsync(own, st) : hipSuccess; }
};

int32_t check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws || !need) return IGC_OK;
    if (!aligned(ws, 16)) return IGC_DECLINE_ALIGNMENT;
    return have < need ? IGC_DECLINE_WORKSPACE : IGC_OK;
}

int32_t finish(hipError_t e, Workspace& w, hipStream_t st) {
    const hipError_t f = w.release(st);
    if (e == hipSuccess) e = f;
    return e == hipSuccess ? 1 : -(int32_t)e;
}

// ------------------------------------------------------------ layer norm
int64_t ln_rows(const igc_layer_norm* p) { return p->n[0] * p->n[1] * p->n[2]; }

int32_t check_ln_shape(const igc_layer_norm* p) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    for (int64_t n : p->n) {
        if (n < 0) return IGC_DECLINE_SHAPE;
        if (n >= kLim31) return IGC_DECLINE_SIZE_LIMIT;
    }
    if (p->channels < 1) return IGC_DECLINE_SHAPE;
    if (p->channels > kLnMaxChannels) return IGC_DECLINE_SIZE_LIMIT;
    if (p->n[2] && (p->n[0] * p->n[1] >= kLim31 || ln_rows(p) >= kLim31))
        return IGC_DECLINE_SIZE_LIMIT;
    const LnForm f = ln_form((int)p->channels);
    if (!launchable(ceil_div(ln_rows(p), f.threads / f.lanes), f.threads))
        return IGC_DECLINE_SIZE_LIMIT;
    if (!(p->eps >= 0.0) || !isfinite((float)p->eps)) return IGC_DECLINE_SCALE;
    return IGC_OK;
}

// Workgroups of the backward pass, which walk the rows: as many as run at
// once, with the same number of rounds each.
int64_t ln_blocks(const igc_layer_norm* p) {
    const LnForm f = ln_form((int)p->channels);
    const int64_t tiles = ceil_div(ln_rows(p), f.threads / f.lanes);
    const int64_t rounds = ceil_div(tiles, ln_bwd_fill(f) * kNumCUs);
    return rounds ? ceil_div(tiles, rounds) : 0;
}

size_t ln_ws(const igc_layer_norm* p) {
    if (!p->dweight && !p->dbias) return 0;
    return (size_t)(ln_blocks(p) * 2 * p->channels) * sizeof(float);
}

struct LnTensors {
    Rows x, g, o;
};

int32_t check_ln(const igc_layer_norm* p, bool backward, LnTensors* t) {
    int32_t r;
    if ((r = check_ln_shape(p))) return r;
    const int64_t c = p->channels;
    if ((r = check_rows(p->x, p->n, c, 2, 2, false, &t->x))) return r;
    if ((r = check_rows(p->out, p->n, c, 2, 2, true, &t->o))) return r;
    t->g = t->x;
    if (backward && (r = check_rows(p->grad, p->n, c, 2, 2, false, &t->g))) return r;
    float* const grads[2] = {backward ? p->dweight : nullptr, backward ? p->dbias : nullptr};
    const float* const small[2] = {p->weight, backward ? nullptr : p->bias};
    const size_t cb = (size_t)c * 4, ws = backward ? ln_ws(p) : 0;
    for (int i = 0; i < 2; ++i)
        if (!aligned(small[i], 4) || !aligned(grads[i], 4)) return IGC_DECLINE_ALIGNMENT;
    // out may be the tensor it takes the place of, and nothing else
    const Rows& same = backward ? t->g : t->x;
    if (!same_rows(t->o, same) && meet(t->o.p, t->o.bytes, same.p, same.bytes))
        return IGC_DECLINE_OVERLAP;
    if (backward && meet(t->o.p, t->o.bytes, t->x.p, t->x.bytes)) return IGC_DECLINE_OVERLAP;
    if (meet(grads[0], cb, grads[1], cb)) return IGC_DECLINE_OVERLAP;
    const struct { const void* p; size_t n; } in[4] = {
        {t->x.p, t->x.bytes}, {t->g.p, t->g.bytes}, {small[0], cb}, {small[1], cb}};
    for (const auto& i : in) {
        for (const float* d : grads)
            if (meet(d, cb, i.p, i.n)) return IGC_DECLINE_OVERLAP;
        if (ws && meet(p->workspace, ws, i.p, i.n)) return IGC_DECLINE_OVERLAP;
    }
    for (const float* s : small)
        if (meet(t->o.p, t->o.bytes, s, cb)) return IGC_DECLINE_OVERLAP;
    for (const float* d : grads)
        if (meet(d, cb, t->o.p, t->o.bytes) || (ws && meet(p->workspace, ws, d, cb)))
            return IGC_DECLINE_OVERLAP;
    if (ws && meet(p->workspace, ws, t->o.p, t->o.bytes)) return IGC_DECLINE_OVERLAP;
    return check_workspace(p->workspace, p->workspace_bytes, ws);
}

int32_t run_ln(const igc_layer_norm* p, bool backward, void* stream) {
    LnTensors t;
    if (check_ln(p, backward, &t) != IGC_OK) return 0;
    LnArgs a{};
    a.rows = (int)ln_rows(p);
    if (a.rows == 0 && !(backward && (p->dweight || p->dbias))) return 1;
    const Rows* all[3] = {&t.x, &t.o, &t.g};
    a.flat = one_stride(p->n, all, 3);
    const Rows* in[3] = {&t.x, &t.g, &t.o};
    int64_t* to[3] = {a.x_s, a.g_s, a.o_s};
    for (int i = 0; i < 3; ++i) {
        for (int k = 0; k < 3; ++k) to[i][k] = in[i]->s[k];
        if (a.flat) to[i][2] = flat_stride(p->n, *in[i]);
    }
    a.x = (const uint8_t*)t.x.p;
    a.dy = (const uint8_t*)t.g.p;
    a.out = (uint8_t*)const_cast<void*>(t.o.p);
    a.w = p->weight;
    a.b = p->bias;
    a.n1 = (int)p->n[1];
    a.n2 = (int)p->n[2];
    a.C = (int)p->channels;
    a.eps = (float)p->eps;
    a.inv_c = 1.0f / (float)a.C;
    const hipStream_t st = (hipStream_t)stream;
    Workspace w;
    if (backward) {
        a.dw = p->dweight;
        a.db = p->dbias;
        a.blocks = (int)ln_blocks(p);
        const hipError_t e = w.take(p->workspace, ln_ws(p), st);
        if (e != hipSuccess) return -(int32_t)e;
        a.partial = a.dw || a.db ? (float*)w.p : nullptr;
    }
    const hipError_t e = p->dtype == IGC_DTYPE_BF16 ? launch_layer_norm<DT_BF16>(a, backward, st)
                                                    : launch_layer_norm<DT_FP16>(a, backward, st);
    return finish(e, w, st);
}

// ------------------------------------------------------------ rows in 8 bits
int32_t check_quant(const igc_quantize_rows* p, Rows* x, Rows* q) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    for (int64_t n : p->n) {
        if (n < 0) return IGC_DECLINE_SHAPE;
        if (n >= kLim31) return IGC_DECLINE_SIZE_LIMIT;
    }
    if (p->channels < 1) return IGC_DECLINE_SHAPE;
    if (p->channels > kQuantMaxChannels) return IGC_DECLINE_SIZE_LIMIT;
    const int64_t n01 = p->n[0] * p->n[1];
    if (p->n[2] && (n01 >= kLim31 || n01 * p->n[2] >= kLim31)) return IGC_DECLINE_SIZE_LIMIT;
    const int64_t rows = n01 * p->n[2];
    const LnForm f = ln_form((int)p->channels);
    if (!launchable(ceil_div(rows, f.threads / f.lanes), f.threads)) return IGC_DECLINE_SIZE_LIMIT;
    int32_t r;
    if ((r = check_rows(p->x, p->n, p->channels, 2, 2, false, x))) return r;
    if ((r = check_rows(p->q, p->n, p->channels, 1, 16, true, q))) return r;
    if (rows == 0) return IGC_OK;
    if (!p->scale) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(p->scale, 4)) return IGC_DECLINE_ALIGNMENT;
    const size_t sb = (size_t)rows * 4;
    if (meet(q->p, q->bytes, x->p, x->bytes) || meet(p->scale, sb, x->p, x->bytes) ||
        meet(p->scale, sb, q->p, q->bytes))
        return IGC_DECLINE_OVERLAP;
    return IGC_OK;
}

// ------------------------------------------------------------ their product
// Few rows, whose workgroups each read x again (32 rows x 4096 x 4096: 8.4 us,
// tiles 10.5; x 8192 x 8192: 25 and 20), or the largest tiles that still give
// every CU one (4096 x 4096 x 4096: 72 us in tiles of 256, 90 in tiles of 128; 2048
// x 4096 x 4096: 55 and 44; 2048 x 2048 x 4096: 23 us in tiles of 128, 34 in tiles
// of 64; 1024 x 1024 x 4096: 19 and 11).  What the rule does not see: few columns
// of a long k (32 rows x 300 x 131056: 115 us as few rows, 186 in tiles) and a
// last round of few tiles (4352 x 4096 x 4096: 111 us in tiles of 256, 101 of 128).
LinForm lin_form(const igc_linear_i8* p) {
    if (p->m <= 16 || (p->m <= kFewRows && p->n * p->k <= (int64_t)1 << 25))
        return {0, 1, ceil_div(p->n, 16), kFewWaves * 64};
    for (int tile : {256, 128}) {
        const LinForm f{tile, ceil_div(p->m, tile), ceil_div(p->n, tile), 256};
        if (f.tiles_m * f.tiles_n >= kNumCUs) return f;
    }
    return {64, ceil_div(p->m, 64), ceil_div(p->n, 64), 256};
}

int32_t check_linear(const igc_linear_i8* p) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    if (p->m < 0 || p->n < 0 || p->k < 0) return IGC_DECLINE_SHAPE;
    if (p->m >= kLim31 || p->n >= kLim31 || p->k > kQuantMaxChannels)
        return IGC_DECLINE_SIZE_LIMIT;
    if (p->m == 0 || p->n == 0) return IGC_OK;
    const int64_t k16 = ceil_div(p->k, 16) * 16;
    if (!p->y || !p->x_scale || !p->w_scale || (p->k && (!p->x || !p->w)))
        return IGC_DECLINE_NULL_POINTER;
    if ((p->k && (!aligned(p->x, 16) || !aligned(p->w, 16) || p->x_pitch % 16 ||
                  p->w_pitch % 16)) ||
        !aligned(p->y, 2) || !aligned(p->x_scale, 4) || !aligned(p->w_scale, 4) ||
        !aligned(p->bias, 4))
        return IGC_DECLINE_ALIGNMENT;
    // rows of one may follow each other at any pitch, and x may repeat a row
    if ((p->k && (p->x_pitch < 0 || p->w_pitch < 0)) || (p->m > 1 && p->y_pitch < p->n))
        return IGC_DECLINE_STRIDE;
    const int64_t lim = (int64_t)1 << 22;
    if (p->x_pitch >= lim || p->w_pitch >= lim || p->y_pitch >= kBatchStrideLim ||
        (double)p->m * (double)p->y_pitch > kExtentLim)
        return IGC_DECLINE_SIZE_LIMIT;
    const LinForm f = lin_form(p);
    if (!launchable(f.tiles_m * f.tiles_n, f.threads)) return IGC_DECLINE_SIZE_LIMIT;
    const size_t yb = (size_t)((p->m - 1) * p->y_pitch + p->n) * 2;
    const size_t xb = p->k ? (size_t)((p->m - 1) * p->x_pitch + k16) : 0;
    const size_t wb = p->k ? (size_t)((p->n - 1) * p->w_pitch + k16) : 0;
    if (meet(p->y, yb, p->x, xb) || meet(p->y, yb, p->w, wb) ||
        meet(p->y, yb, p->x_scale, (size_t)p->m * 4) ||
        meet(p->y, yb, p->w_scale, (size_t)p->n * 4) || meet(p->y, yb, p->bias, (size_t)p->n * 4))
        return IGC_DECLINE_OVERLAP;
    return IGC_OK;
}

// ------------------------------------------------------------ the cache
int64_t cache_pitch(const igc_kv_cache& c) { return ceil_div(c.head_dim, 16) * 16; }
int64_t cache_rows(const igc_kv_cache& c) { return c.pages * c.kv_heads * c.page_tokens; }

int32_t check_cache(const igc_kv_cache& c) {
    if (c.pages < 0 || c.kv_heads < 0) return IGC_DECLINE_SHAPE;
    if (c.page_tokens < 16 || c.page_tokens > 1024 || log2_exact(c.page_tokens) < 0)
        return IGC_DECLINE_SHAPE;
    if (c.head_dim < 8 || c.head_dim > 128 || c.head_dim % 8) return IGC_DECLINE_HEAD_DIM;
    if (c.pages >= kLim31 || c.kv_heads >= kLim31 ||
        (c.kv_heads && c.pages > ((int64_t)1 << 40) / (c.kv_heads * c.page_tokens)))
        return IGC_DECLINE_SIZE_LIMIT;
    if (cache_rows(c) == 0) return IGC_OK;
    if (!c.k || !c.v || !c.k_scale || !c.v_scale) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 16) ||
        !aligned(c.v_scale, 16))
        return IGC_DECLINE_ALIGNMENT;
    const size_t kb = (size_t)(cache_rows(c) * cache_pitch(c)), sb = (size_t)cache_rows(c) * 4;
    const struct { const void* p; size_t n; } part[4] = {
        {c.k, kb}, {c.v, kb}, {c.k_scale, sb}, {c.v_scale, sb}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (meet(part[i].p, part[i].n, part[j].p, part[j].n)) return IGC_DECLINE_OVERLAP;
    return IGC_OK;
}

bool meets_cache(const igc_kv_cache& c, const void* w, size_t n) {
    const size_t kb = (size_t)(cache_rows(c) * cache_pitch(c)), sb = (size_t)cache_rows(c) * 4;
    return meet(w, n, c.k, kb) || meet(w, n, c.v, kb) || meet(w, n, c.k_scale, sb) ||
           meet(w, n, c.v_scale, sb);
}

// Gate of a table of `batch` rows; its bytes.
int32_t check_table(const int32_t* table, int64_t batch, int64_t stride, int64_t entries,
                    size_t* bytes) {
    *bytes = 0;
    if (entries < 0) return IGC_DECLINE_SHAPE;
    if (entries >= kLim31) return IGC_DECLINE_SIZE_LIMIT;
    if (batch == 0 || entries == 0) return IGC_OK;
    if (!table) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(table, 4)) return IGC_DECLINE_ALIGNMENT;
    if (stride < 0 || stride >= kBatchStrideLim) return IGC_DECLINE_STRIDE;
    if ((double)(batch - 1) * (double)stride > kExtentLim) return IGC_DECLINE_SIZE_LIMIT;
    *bytes = (size_t)((batch - 1) * stride + entries) * 4;
    return IGC_OK;
}

// Whether two outputs of one shape [n0, n1, n2, d] share no element: they lie
// apart, or have the same strides and the blocks of some inner axes of the one
// lie between those of the other (the halves of one buffer's rows, say).
bool outputs_apart(const Tensor& x, const Tensor& y, const int64_t n[3], int64_t d) {
    if (!meet(x.p, x.bytes, y.p, y.bytes)) return true;
    if (x.b != y.b || x.t != y.t || x.h != y.h) return false;
    const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
    const int64_t delta = (int64_t)(a < b ? b - a : a - b);
    struct Axis { int64_t n, s; } ax[3] = {{n[0], x.b}, {n[1], x.t}, {n[2], x.h}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (ax[j].s < ax[i].s) {
                const Axis t = ax[i];
                ax[i] = ax[j];
                ax[j] = t;
            }
    int64_t block = 2 * d;   // bytes of the inner `i` axes
    for (int i = 0; i < 3; ++i) {
        if (delta >= block) {
            int64_t both = block + delta;
            int j = i;
            for (; j < 3 && (ax[j].n == 1 || ax[j].s >= both); ++j)
                both += (ax[j].n - 1) * ax[j].s;
            if (j == 3) return true;
        }
        block += (ax[i].n - 1) * ax[i].s;
    }
    return false;
}

// Runs of tokens that a workgroup of kv_cache_write / read takes, a sequence;
// workgroups of a launch.
int64_t io_runs(const igc_kv_io* p) {
    return ceil_div(p->tokens, cache_run(qk_lanes((int)p->cache.head_dim)));
}
int64_t io_groups(const igc_kv_io* p) {
    return p->batch * io_runs(p) * 2 * ceil_div(p->cache.kv_heads, kCacheHeads);
}

int32_t check_io(const igc_kv_io* p, bool write, Tensor t[2]) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    if (p->batch < 0 || p->tokens < 0) return IGC_DECLINE_SHAPE;
    int32_t r;
    if ((r = check_cache(p->cache))) return r;
    if (p->batch >= kLim31 || p->tokens >= kLim31) return IGC_DECLINE_SIZE_LIMIT;
    const igc_kv_cache& c = p->cache;
    const int64_t hc = ceil_div(c.kv_heads, kCacheHeads);
    if (hc && p->batch * p->tokens > ((int64_t)1 << 40) / hc) return IGC_DECLINE_SIZE_LIMIT;
    if (!launchable(io_groups(p), kCacheThreads)) return IGC_DECLINE_SIZE_LIMIT;
    const igc_attn_view* v[2] = {&p->k, &p->v};
    for (int i = 0; i < 2; ++i)
        if ((r = check_view(*v[i], p->batch, p->tokens, c.kv_heads, c.head_dim, !write,
                            kBatchStrideLim, &t[i])))
            return r;
    size_t tb;
    if ((r = check_table(p->table, p->batch, p->table_stride, p->table_entries, &tb))) return r;
    if (io_groups(p) == 0) return IGC_OK;
    if (!p->start) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(p->start, 4) || !aligned(p->lens, 4)) return IGC_DECLINE_ALIGNMENT;
    const size_t bb = (size_t)p->batch * 4;
    const struct { const void* p; size_t n; } small[3] = {
        {p->table, tb}, {p->start, bb}, {p->lens, bb}};
    for (int i = 0; i < 2; ++i)
        if (meets_cache(c, t[i].p, t[i].bytes)) return IGC_DECLINE_OVERLAP;
    for (const auto& s : small) {
        if (write && meets_cache(c, s.p, s.n)) return IGC_DECLINE_OVERLAP;
        if (!write)
            for (int i = 0; i < 2; ++i)
                if (meet(s.p, s.n, t[i].p, t[i].bytes)) return IGC_DECLINE_OVERLAP;
    }
    const int64_t n[3] = {p->batch, p->tokens, c.kv_heads};
    if (!write && !outputs_apart(t[0], t[1], n, c.head_dim)) return IGC_DECLINE_OVERLAP;
    return IGC_OK;
}

int32_t run_io(const igc_kv_io* p, bool write, void* stream) {
    Tensor t[2];
    if (check_io(p, write, t) != IGC_OK) return 0;
    if (io_groups(p) == 0) return 1;
    const igc_kv_cache& c = p->cache;
    CacheArgs a{};
    a.pool[0] = c.k;
    a.pool[1] = c.v;
    a.scale[0] = c.k_scale;
    a.scale[1] = c.v_scale;
    for (int i = 0; i < 2; ++i) {
        a.t[i] = (uint8_t*)const_cast<void*>(t[i].p);
        a.t_b[i] = t[i].b;
        a.t_t[i] = t[i].t;
        a.t_h[i] = t[i].h;
    }
    a.table = p->table;
    a.start = p->start;
    a.lens = p->lens;
    a.table_stride = p->table_stride;
    a.B = (int)p->batch;
    a.T = (int)p->tokens;
    a.H = (int)c.kv_heads;
    a.D = (int)c.head_dim;
    a.Dp = (int)cache_pitch(c);
    a.hc = (int)ceil_div(c.kv_heads, kCacheHeads);
    a.runs = (int)io_runs(p);
    a.entries = (int)p->table_entries;
    a.pages = (int)c.pages;
    a.shift = log2_exact(c.page_tokens);
    const hipStream_t st = (hipStream_t)stream;
    const hipError_t e = p->dtype == IGC_DTYPE_BF16 ? launch_kv_cache<DT_BF16>(a, write, st)
                                                    : launch_kv_cache<DT_FP16>(a, write, st);
    return e == hipSuccess ? 1 : -(int32_t)e;
}

// ------------------------------------------------------------ attention over it
struct CacheAttnPlan {
    int64_t tile, row_tiles;            // rows a workgroup
    int64_t slots, groups;              // slots of cache_plan.hpp; workgroups
    int64_t capacity;
    bool split;
    int64_t part_floats, stat_floats;
};

// The attention arguments whose gates are cross attention's.
int32_t check_cache_attn_shape(const igc_cache_attn* p) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    if (p->batch < 0 || p->q_len < 0 || p->q_heads < 0 || p->table_entries < 0)
        return IGC_DECLINE_SHAPE;
    const igc_kv_cache& c = p->cache;
    if (c.kv_heads < 0 || c.page_tokens < 16 || c.page_tokens > 1024) return IGC_DECLINE_SHAPE;
    if (p->q_heads > 0 && (c.kv_heads == 0 || p->q_heads % c.kv_heads)) return IGC_DECLINE_GROUPS;
    if (c.head_dim < 8 || c.head_dim > 128 || c.head_dim % 8) return IGC_DECLINE_HEAD_DIM;
    const float c2 = (float)(p->scale * 1.4426950408889634);
    if (!(p->scale > 0.0) || (float)p->scale < 1e-30f || !isfinite(c2)) return IGC_DECLINE_SCALE;
    if (p->batch >= kLim31 || p->q_len >= kLim31 || p->q_heads >= kLim31 ||
        c.kv_heads >= kLim31 || p->table_entries >= kLim31)
        return IGC_DECLINE_SIZE_LIMIT;
    const int64_t g = c.kv_heads ? p->q_heads / c.kv_heads : 1;
    if ((g && p->q_len >= kLim31 / 4 / g) || p->batch * p->q_heads >= kLim31 ||
        p->table_entries * c.page_tokens >= kLim31 - 4096)
        return IGC_DECLINE_SIZE_LIMIT;
    return IGC_OK;
}

// Rows of a workgroup: 16 where that holds them all (4 x 65537 tokens, 4 rows a
// key head: 78 us, 32 rows 86; 8 x 784: 9.5 and 10.8).  A sequence is split
// between workgroups from 641 tokens of its table on (8 sequences, 16 heads of
// 128 over 4 key heads, 640 tokens: 8.2 us whole and 9.2 split; 704: 9.6 and 9.2;
// 1024: 12.1 and 9.6; 1 sequence, 32 heads over 8, 704: 9.4 and 9.0; 4 with 5
// drafts, 8 heads of 64, 704: 7.8 and 8.1, 1024: 9.2 and 8.1), where the card has
// a workgroup a CU for three of each, or for two of 32 rows, which fill a CU
// alone (16 x 4096 with 32 rows: 28 us, two a CU 36); else two a CU that even out
// ragged lengths (16 x 4099 with 5 drafts, 8 heads of 80: 21.8 us, one a CU 24.5),
// if those are 2.5 a sequence (24 of them: 27.7 us split and 32.2 whole; 28, which
// stay whole: 30.8 and 32.6) or long ones 2 (32 x 16000, 8 heads of 128: 141 and
// 153).  Short sequences in a wide table pay for it (8 x 300 in a table of 640
// tokens: 6.2 us, of 4096: 10.0).
CacheAttnPlan cache_attn_plan(const igc_cache_attn* p) {
    CacheAttnPlan x{};
    const igc_kv_cache& c = p->cache;
    const int64_t rows = c.kv_heads ? p->q_len * (p->q_heads / c.kv_heads) : 0;
    x.tile = rows <= 16 ? 16 : 32;
    x.row_tiles = ceil_div(rows, x.tile);
    x.capacity = p->table_entries * c.page_tokens;
    const int64_t hr = c.kv_heads * x.row_tiles;
    x.slots = hr ? kNumCUs / hr : 0;
    if (x.tile == 16 && x.slots < 3 * p->batch) x.slots = hr ? 2 * kNumCUs / hr : 0;
    const bool fair = x.tile != 16 || x.slots * 2 >= 5 * p->batch || x.capacity > 8192;
    x.split = p->batch > 0 && cache_splits(x.slots, p->batch) && fair && x.capacity > 640;
    if (!x.split) x.slots = p->batch;
    x.groups = hr * (x.split ? cache_slots_bound(x.slots, p->batch, x.capacity) : p->batch);
    if (x.split) {
        const int64_t n = x.groups * (rows < x.tile ? rows : x.tile);
        x.part_floats = n * c.head_dim;
        x.stat_floats = n * 2;
    }
    return x;
}

size_t cache_attn_ws(const CacheAttnPlan& x) {
    return (size_t)(x.part_floats + x.stat_floats) * sizeof(float);
}

int32_t check_cache_attn(const igc_cache_attn* p, Tensor* q, Tensor* o, CacheAttnPlan* plan) {
    int32_t r;
    if ((r = check_cache_attn_shape(p))) return r;
    if ((r = check_cache(p->cache))) return r;
    const igc_kv_cache& c = p->cache;
    if ((r = check_view(p->q, p->batch, p->q_len, p->q_heads, c.head_dim, false, kStrideLim, q)))
        return r;
    if ((r = check_view(p->out, p->batch, p->q_len, p->q_heads, c.head_dim, true, kStrideLim, o)))
        return r;
    const int64_t g = c.kv_heads ? p->q_heads / c.kv_heads : 1;
    for (const Tensor* x : {q, o})
        if (33 * x->t + g * x->h >= kLim31) return IGC_DECLINE_SIZE_LIMIT;
    size_t tb;
    if ((r = check_table(p->table, p->batch, p->table_stride, p->table_entries, &tb))) return r;
    if (p->batch && p->q_len && p->q_heads && !p->lens) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(p->lens, 4) || !aligned(p->lse, 4)) return IGC_DECLINE_ALIGNMENT;
    *plan = cache_attn_plan(p);
    // (a split leaves at most kCacheMostSlots groups, and so few rows to join)
    if (!launchable(plan->groups, kCacheWaves * 64)) return IGC_DECLINE_SIZE_LIMIT;
    const size_t lb = (size_t)(p->batch * p->q_heads * p->q_len) * 4, bb = (size_t)p->batch * 4;
    const size_t ws = cache_attn_ws(*plan);
    const struct { const void* p; size_t n; } outs[3] = {
        {o->p, o->bytes}, {p->lse, lb}, {p->workspace, p->workspace ? ws : 0}};
    for (int i = 0; i < 3; ++i) {
        if (meet(outs[i].p, outs[i].n, q->p, q->bytes) || meet(outs[i].p, outs[i].n, p->table, tb) ||
            meet(outs[i].p, outs[i].n, p->lens, bb) || meets_cache(c, outs[i].p, outs[i].n))
            return IGC_DECLINE_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return IGC_DECLINE_OVERLAP;
    }
    return check_workspace(p->workspace, p->workspace_bytes, ws);
}

}  // namespace

extern "C" {

int32_t quantize_rows_check(const igc_quantize_rows* args) {
    Rows x, q;
    return check_quant(args, &x, &q);
}

int32_t quantize_rows(const igc_quantize_rows* args, void* stream) {
    Rows x, q;
    if (check_quant(args, &x, &q) != IGC_OK) return 0;
    QuantArgs a{};
    a.rows = (int)(args->n[0] * args->n[1] * args->n[2]);
    if (a.rows == 0) return 1;
    const Rows* both[2] = {&x, &q};
    a.flat = one_stride(args->n, both, 2);
    for (int k = 0; k < 3; ++k) {
        a.x_s[k] = x.s[k];
        a.q_s[k] = q.s[k];
    }
    if (a.flat) {
        a.x_s[2] = flat_stride(args->n, x);
        a.q_s[2] = flat_stride(args->n, q);
    }
    a.x = (const uint8_t*)x.p;
    a.q = (uint8_t*)const_cast<void*>(q.p);
    a.scale = args->scale;
    a.n1 = (int)args->n[1];
    a.n2 = (int)args->n[2];
    a.C = (int)args->channels;
    const hipStream_t st = (hipStream_t)stream;
    const hipError_t e = args->dtype == IGC_DTYPE_BF16 ? launch_quantize_rows<DT_BF16>(a, st)
                                                       : launch_quantize_rows<DT_FP16>(a, st);
    return e == hipSuccess ? 1 : -(int32_t)e;
}

int32_t linear_i8_check(const igc_linear_i8* args) { return check_linear(args); }

int32_t linear_i8(const igc_linear_i8* args, void* stream) {
    if (check_linear(args) != IGC_OK) return 0;
    if (args->m == 0 || args->n == 0) return 1;
    const LinForm f = lin_form(args);
    LinArgs a{};
    a.x = (const uint8_t*)args->x;
    a.w = (const uint8_t*)args->w;
    a.xs = args->x_scale;
    a.ws = args->w_scale;
    a.bias = args->bias;
    a.y = (uint8_t*)args->y;
    a.x_p = args->x_pitch;
    a.w_p = args->w_pitch;
    a.y_p = args->y_pitch * 2;
    a.M = (int)args->m;
    a.N = (int)args->n;
    a.K = (int)args->k;
    a.K16 = (int)(ceil_div(args->k, 16) * 16);
    a.tiles_m = (int)f.tiles_m;
    a.tiles_n = (int)f.tiles_n;
    const hipStream_t st = (hipStream_t)stream;
    const hipError_t e = args->dtype == IGC_DTYPE_BF16 ? launch_linear_i8<DT_BF16>(a, f.tile, st)
                                                       : launch_linear_i8<DT_FP16>(a, f.tile, st);
    return e == hipSuccess ? 1 : -(int32_t)e;
}

int32_t kv_cache_write_check(const igc_kv_io* args) {
    Tensor t[2];
    return check_io(args, true, t);
}

int32_t kv_cache_read_check(const igc_kv_io* args) {
    Tensor t[2];
    return check_io(args, false, t);
}

int32_t kv_cache_write(const igc_kv_io* args, void* stream) { return run_io(args, true, stream); }

int32_t kv_cache_read(const igc_kv_io* args, void* stream) { return run_io(args, false, stream); }

int32_t cache_attn_fwd_check(const igc_cache_attn* args) {
    Tensor q, o;
    CacheAttnPlan plan;
    return check_cache_attn(args, &q, &o, &plan);
}

size_t cache_attn_fwd_workspace_bytes(const igc_cache_attn* args) {
    if (check_cache_attn_shape(args) != IGC_OK) return 0;
    return cache_attn_ws(cache_attn_plan(args));
}

int32_t cache_attn_fwd(const igc_cache_attn* args, void* stream) {
    Tensor q, o;
    CacheAttnPlan plan;
    if (check_cache_attn(args, &q, &o, &plan) != IGC_OK) return 0;
    if (args->batch == 0 || args->q_len == 0 || args->q_heads == 0) return 1;
    const igc_kv_cache& c = args->cache;
    CacheAttnArgs x{};
    AttnArgs& a = x.a;
    a.q = (const uint8_t*)q.p;
    a.out = (uint8_t*)const_cast<void*>(o.p);
    a.q_b = q.b; a.q_t = q.t; a.q_h = q.h;
    a.o_b = o.b; a.o_t = o.t; a.o_h = o.h;
    a.lse = args->lse;
    a.B = (int)args->batch;
    a.Tq = (int)args->q_len;
    a.Hq = (int)args->q_heads;
    a.Hk = (int)c.kv_heads;
    a.G = a.Hq / a.Hk;
    a.D = (int)c.head_dim;
    a.rows = a.Tq * a.G;
    a.row_tiles = (int)plan.row_tiles;
    a.scale = (float)args->scale;
    a.c = (float)(args->scale * 1.4426950408889634);
    set_group_divisor(&a);
    x.pool[0] = c.k;
    x.pool[1] = c.v;
    x.scales[0] = c.k_scale;
    x.scales[1] = c.v_scale;
    x.table = args->table;
    x.lens = args->lens;
    x.table_stride = args->table_stride;
    x.capacity = plan.capacity;
    x.slots = plan.slots;
    x.entries = (int)args->table_entries;
    x.pages = (int)c.pages;
    x.shift = log2_exact(c.page_tokens);
    x.Dp = (int)cache_pitch(c);
    x.causal = args->causal != 0;
    x.tile = (int)plan.tile;
    x.split = plan.split;
    x.fixed = plan.split && cache_fixed(plan.slots, args->batch, plan.capacity)
                  ? (int)cache_most(plan.capacity) : 0;
    const hipStream_t st = (hipStream_t)stream;
    Workspace w;
    hipError_t e = w.take(args->workspace, cache_attn_ws(plan), st);
    if (e != hipSuccess) return -(int32_t)e;
    a.part = (float*)w.p;
    a.stat = a.part + plan.part_floats;
    e = args->dtype == IGC_DTYPE_BF16
            ? launch_cache_attn<DT_BF16>(x, (unsigned)plan.groups, st)
            : launch_cache_attn<DT_FP16>(x, (unsigned)plan.groups, st);
    return finish(e, w, st);
}

int32_t layer_norm_fwd_check(const igc_layer_norm* args) {
    LnTensors t;
    return check_ln(args, false, &t);
}

int32_t layer_norm_bwd_check(const igc_layer_norm* args) {
    LnTensors t;
    return check_ln(args, true, &t);
}

size_t layer_norm_bwd_workspace_bytes(const igc_layer_norm* args) {
    return check_ln_shape(args) == IGC_OK ? ln_ws(args) : 0;
}

int32_t layer_norm_fwd(const igc_layer_norm* args, void* stream) {
    return run_ln(args, false, stream);
}

int32_t layer_norm_bwd(const igc_layer_norm* args, void* stream) {
    return run_ln(args, true, stream);
}

}  // extern "C"
