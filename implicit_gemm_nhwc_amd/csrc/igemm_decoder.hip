// C-ABI entry points of the decoder block's operators (declarations and
// contracts in include/igemm_decoder.h): the host gates, the launch plans and
// the workspaces.  Every step of the computation runs in the kernels of
// layer_norm.hpp.
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
    const int64_t rounds = ceil_div(tiles, 3 * kNumCUs);
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

}  // namespace

extern "C" {

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
