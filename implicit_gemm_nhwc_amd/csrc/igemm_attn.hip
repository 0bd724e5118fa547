// C-ABI entry points of the attention operators (declarations and contracts
// in include/igemm_attn.h): the host gates, the launch plans and the
// workspaces.  Every step of the computation runs in the kernels of
// attn_fwd.hpp, attn_short.hpp, attn_bwd.hpp and
// qk_norm.hpp.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "attn_host.hpp"
#include "igemm_attn.h"

namespace {

using namespace igc;

constexpr int64_t kLim31 = (int64_t)1 << 31;
constexpr int64_t kStrideLim = (int64_t)1 << 23;        // strides within a tile, elements
constexpr int64_t kBatchStrideLim = (int64_t)1 << 40;   // strides between 64-bit bases, elements
constexpr double kExtentLim = 0x1p56;                   // no address space holds more
constexpr int64_t kQkBwdBlocks = 3 * kNumCUs;           // three a CU: what the registers hold

// Whether a launch of so many workgroups holds fewer than 2^32 threads; HIP
// takes the count modulo 2^32 (2^24 - 16 workgroups of 512 threads ran half of
// themselves and reported success).
bool launchable(int64_t groups, int64_t threads) {
    return groups <= (((int64_t)1 << 32) - 1) / threads;
}

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool meet(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

// A tensor [batch, token, head, d] behind a view: its byte range, with the
// strides of axes of one entry (which say nothing) taken as 0.
struct Tensor {
    const void* p;
    int64_t b, t, h;   // strides, bytes
    size_t bytes;      // first to last element
};

// Gate of one view; `write` for outputs.  Empty tensors may be NULL.
int32_t check_view(const igc_attn_view& v, int64_t nb, int64_t nt, int64_t nh, int64_t d,
                   bool write, int64_t head_lim, Tensor* out) {
    Tensor x{v.data, 0, 0, 0, 0};
    const int64_t n[3] = {nb, nt, nh};
    int64_t s[3] = {v.batch, v.token, v.head};
    if (nb == 0 || nt == 0 || nh == 0) {
        *out = x;
        return IGC_OK;
    }
    if (!v.data) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(v.data, 16)) return IGC_DECLINE_ALIGNMENT;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) s[i] = 0;
        if (s[i] < 0) return IGC_DECLINE_STRIDE;
        if (s[i] % 8) return IGC_DECLINE_ALIGNMENT;
        if (s[i] >= (i == 0 ? kBatchStrideLim : i == 1 ? kStrideLim : head_lim))
            return IGC_DECLINE_SIZE_LIMIT;
    }
    if ((double)nb * (double)s[0] + (double)nt * (double)s[1] + (double)nh * (double)s[2] >
        kExtentLim)
        return IGC_DECLINE_SIZE_LIMIT;
    if (write) {
        // axes from the smallest stride up: each has to step over all before
        int ord[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (s[ord[j]] < s[ord[i]]) { const int t = ord[i]; ord[i] = ord[j]; ord[j] = t; }
        int64_t ext = d;
        for (int i = 0; i < 3; ++i) {
            const int k = ord[i];
            if (n[k] == 1) continue;
            if (s[k] < ext) return IGC_DECLINE_OVERLAP;
            ext += (n[k] - 1) * s[k];
        }
    }
    x.b = s[0] * 2;
    x.t = s[1] * 2;
    x.h = s[2] * 2;
    x.bytes = (size_t)((n[0] - 1) * x.b + (n[1] - 1) * x.t + (n[2] - 1) * x.h + d * 2);
    *out = x;
    return IGC_OK;
}

// scale * log2(e), as the kernels hold it.
float scale_log2(const igc_cross_attn* p) { return (float)(p->scale * 1.4426950408889634); }

// Shapes and parameters of cross attention.
int32_t check_attn_shape(const igc_cross_attn* p) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    if (p->batch < 0 || p->q_len < 0 || p->kv_len < 0 || p->q_heads < 0 || p->kv_heads < 0)
        return IGC_DECLINE_SHAPE;
    if (p->q_heads > 0 && (p->kv_heads == 0 || p->q_heads % p->kv_heads)) return IGC_DECLINE_GROUPS;
    if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8) return IGC_DECLINE_HEAD_DIM;
    if (!(p->scale > 0.0) || (float)p->scale < 1e-30f || !isfinite(scale_log2(p)))
        return IGC_DECLINE_SCALE;
    if (p->batch >= kLim31 || p->q_len >= kLim31 || p->kv_len >= kLim31 || p->q_heads >= kLim31 ||
        p->kv_heads >= kLim31)
        return IGC_DECLINE_SIZE_LIMIT;
    const int64_t g = p->kv_heads ? p->q_heads / p->kv_heads : 1;
    if (g * p->q_len >= kLim31 / 4 || p->kv_len >= kLim31 - 4096 ||
        p->batch * p->q_heads >= kLim31)
        return IGC_DECLINE_SIZE_LIMIT;
    return IGC_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups a key head of the few-keys kernels, whose waves walk blocks of 32
// rows: as many rounds as the card's `slots` workgroups need, spread evenly.
int64_t short_tiles(int64_t bh, int64_t rows, int64_t slots) {
    const int64_t blocks = ceil_div(rows, 32);
    int64_t per = bh > 0 ? slots / bh : 1;   // workgroups a head that run at once
    if (per < 1) per = 1;
    const int64_t rounds = ceil_div(blocks, per * kAttnWaves);
    const int64_t n = ceil_div(blocks, (rounds > 0 ? rounds : 1) * kAttnWaves);
    return n < 1 ? 1 : n;
}

// Plan of a forward launch from the shapes alone (checked before).
AttnPlan fwd_plan(const igc_cross_attn* p) {
    AttnPlan x{};
    const int64_t bh = p->batch * p->kv_heads;
    const int64_t rows = p->kv_heads ? p->q_len * (p->q_heads / p->kv_heads) : 0;
    x.token = rows <= 32;
    x.nsplit = 1;
    x.split = kLim31 - 1;
    x.few_keys = !x.token && p->kv_len <= kShortKeys;
    if (x.few_keys) {
        x.row_tiles = (int)short_tiles(bh, rows, (p->head_dim <= 64 ? 3 : 2) * kNumCUs);
        return x;
    }
    int64_t groups, step;
    if (x.token) {
        x.row_tiles = 1;
        groups = bh;
        step = kTokenStep;
    } else {
        x.row_tiles = (int)ceil_div(rows, kAttnWaves * 32);
        groups = bh * x.row_tiles;
        step = kKeyTile;
    }
    const int64_t steps = ceil_div(p->kv_len, step);
    int64_t n = 1;
    if (!x.token) {
        // two workgroups a CU, three tiles a split at least (four: a training
        // call of 46.4 us, masked fp16, takes 43.6 with three; one workgroup or
        // four a CU are slower on the other middle-sized calls)
        n = groups > 0 ? 2 * kNumCUs / groups : 1;
        if (n > steps / 3) n = steps / 3;
    } else if (steps > 4) {
        // The join is another launch: four rounds of the waves (1024 keys of
        // 128, 32 key heads) take 10.9 us in one workgroup a head and 10.7
        // split, two 7.8 and 10.7.  Splits fill the card once (2048 keys of
        // 64, 64 key heads: 13.2 us, in twice as many 14.8); from 16 rounds a
        // split on, four times over, so that ragged lengths even out (4 x
        // 30000 .. 65537 keys: 145 us, filled once 170, equal lengths 194 and
        // 197).
        n = groups > 0 ? kNumCUs / groups : 1;
        if (ceil_div(steps, n < 1 ? 1 : n) > 16) n = groups > 0 ? 4 * kNumCUs / groups : 1;
    }
    if (n < 1) n = 1;
    const int64_t per = ceil_div(steps > 0 ? steps : 1, n);
    x.nsplit = (int)ceil_div(steps > 0 ? steps : 1, per);
    x.split = (int)(per * step < kLim31 ? per * step : kLim31 - 1);
    if (x.nsplit > 1) {
        x.part_floats = x.nsplit * bh * rows * p->head_dim;
        x.stat_floats = x.nsplit * bh * rows * 2;
    }
    return x;
}

size_t fwd_ws(const AttnPlan& x) {
    return (size_t)((x.part_floats + x.stat_floats) * (int64_t)sizeof(float));
}

struct AttnTensors {
    Tensor q, k, v, o;
};

// The kernels address a tile of packed rows (at most 65 tokens, all heads of
// a group) in 32 bits.
bool packed_fits(const igc_cross_attn* p, const Tensor& x) {
    const int64_t g = p->kv_heads ? p->q_heads / p->kv_heads : 1;
    return (kRowTile + 1) * x.t + g * x.h < kLim31;
}

int32_t check_attn_views(const igc_cross_attn* p, AttnTensors* t, bool write_out) {
    int32_t r;
    const int64_t d = p->head_dim;
    const bool any = p->batch && p->q_len && p->q_heads;
    if ((r = check_view(p->q, p->batch, p->q_len, p->q_heads, d, false, kStrideLim, &t->q)))
        return r;
    // a head of the keys is a 64-bit base: a long head-major cache has large
    // head strides
    const int64_t nb = any ? p->batch : 0;
    if ((r = check_view(p->k, nb, p->kv_len, p->kv_heads, d, false, kBatchStrideLim, &t->k)))
        return r;
    if ((r = check_view(p->v, nb, p->kv_len, p->kv_heads, d, false, kBatchStrideLim, &t->v)))
        return r;
    if ((r = check_view(p->out, p->batch, p->q_len, p->q_heads, d, write_out, kStrideLim, &t->o)))
        return r;
    if (!packed_fits(p, t->q) || !packed_fits(p, t->o)) return IGC_DECLINE_SIZE_LIMIT;
    if (p->kv_lens && !aligned(p->kv_lens, 4)) return IGC_DECLINE_ALIGNMENT;
    if (p->lse && !aligned(p->lse, 4)) return IGC_DECLINE_ALIGNMENT;
    if (p->key_mask && (p->key_mask_stride < 0 || p->key_mask_stride >= kBatchStrideLim))
        return IGC_DECLINE_STRIDE;
    if (p->key_mask && (double)(p->batch - 1) * (double)p->key_mask_stride > kExtentLim)
        return IGC_DECLINE_SIZE_LIMIT;
    return IGC_OK;
}

size_t lse_bytes(const igc_cross_attn* p) {
    return (size_t)(p->batch * p->q_heads * p->q_len) * sizeof(float);
}

// Whether [w, w + n) meets an input of the call.
bool meets_inputs(const igc_cross_attn* p, const AttnTensors& t, const void* w, size_t n) {
    const size_t mask = p->batch && p->kv_len
                            ? (size_t)((p->batch - 1) * p->key_mask_stride + p->kv_len) : 0;
    return meet(w, n, t.q.p, t.q.bytes) || meet(w, n, t.k.p, t.k.bytes) ||
           meet(w, n, t.v.p, t.v.bytes) || meet(w, n, p->kv_lens, (size_t)p->batch * 4) ||
           meet(w, n, p->key_mask, mask);
}

int32_t check_fwd(const igc_cross_attn* p, AttnTensors* t, AttnPlan* plan) {
    int32_t r;
    if ((r = check_attn_shape(p))) return r;
    if ((r = check_attn_views(p, t, true))) return r;
    *plan = fwd_plan(p);
    if (!launchable(p->batch * p->kv_heads * plan->row_tiles * plan->nsplit,
                    (plan->token ? kTokenWaves : kAttnWaves) * 64))
        return IGC_DECLINE_SIZE_LIMIT;
    const size_t ws = fwd_ws(*plan);
    if (meets_inputs(p, *t, t->o.p, t->o.bytes) || meets_inputs(p, *t, p->lse, lse_bytes(p)) ||
        meet(p->lse, lse_bytes(p), t->o.p, t->o.bytes))
        return IGC_DECLINE_OVERLAP;
    if (p->workspace && ws) {
        if (!aligned(p->workspace, 16)) return IGC_DECLINE_ALIGNMENT;
        if (p->workspace_bytes < ws) return IGC_DECLINE_WORKSPACE;
        if (meets_inputs(p, *t, p->workspace, ws) || meet(p->workspace, ws, t->o.p, t->o.bytes) ||
            meet(p->workspace, ws, p->lse, lse_bytes(p)))
            return IGC_DECLINE_OVERLAP;
    }
    return IGC_OK;
}

// Kernel arguments common to the passes.
AttnArgs attn_args(const igc_cross_attn* p, const AttnTensors& t) {
    AttnArgs a{};
    a.q = (const uint8_t*)t.q.p;
    a.k = (const uint8_t*)t.k.p;
    a.v = (const uint8_t*)t.v.p;
    a.q_b = t.q.b; a.q_t = t.q.t; a.q_h = t.q.h;
    a.k_b = t.k.b; a.k_t = t.k.t; a.k_h = t.k.h;
    a.v_b = t.v.b; a.v_t = t.v.t; a.v_h = t.v.h;
    a.o_b = t.o.b; a.o_t = t.o.t; a.o_h = t.o.h;
    a.lens = p->kv_lens;
    a.mask = p->key_mask;
    a.mask_b = p->key_mask_stride;
    a.lse = p->lse;
    a.B = (int)p->batch;
    a.Tq = (int)p->q_len;
    a.Tk = (int)p->kv_len;
    a.Hq = (int)p->q_heads;
    a.Hk = (int)p->kv_heads;
    a.G = a.Hq && a.Hk ? a.Hq / a.Hk : 1;   // a divisor also without query heads
    a.D = (int)p->head_dim;
    a.rows = a.Hq ? a.Tq * a.G : 0;
    a.scale = (float)p->scale;
    a.c = scale_log2(p);
    if (a.G > 1) {
        // row / G = mulhi(row, ceil(2^(31 + L) / G)) >> (L - 1), L = ceil(log2 G)
        int L = 0;
        while (((int64_t)1 << L) < a.G) ++L;
        a.g_mul = (uint32_t)((((uint64_t)1 << (31 + L)) + a.G - 1) / a.G);
        a.g_shift = L - 1;
    }
    return a;
}

// Plan of a backward pass from the shapes alone (checked before).
AttnGradPlan bwd_plan(const igc_cross_attn* p) {
    AttnGradPlan x{};
    const int64_t bh = p->batch * p->kv_heads;
    const int64_t rows = p->kv_heads ? p->q_len * (p->q_heads / p->kv_heads) : 0;
    const int64_t row64 = ceil_div(rows, kRowTile), key64 = ceil_div(p->kv_len, kKeyTile);
    if (bh == 0) return x;
    x.rows_pad = (int)(row64 * kRowTile);
    // row pass: four workgroups a CU, of 16 rows at least
    int64_t n = ceil_div(4 * kNumCUs, bh);
    if (n > x.rows_pad / 16) n = x.rows_pad / 16;
    if (n > 256) n = 256;
    x.bound_n = (int)(n < 1 ? 1 : n);
    // splits of `least` tiles at least, for `want` workgroups
    auto split = [](int64_t want, int64_t least, int64_t groups, int64_t tiles, int64_t unit,
                    int* nsplit, int* len) {
        int64_t n = groups > 0 ? want / groups : 1;
        if (n > tiles / least) n = tiles / least;
        if (n < 1) n = 1;
        const int64_t per = ceil_div(tiles > 0 ? tiles : 1, n);
        *nsplit = (int)ceil_div(tiles > 0 ? tiles : 1, per);
        *len = (int)(per * unit < kLim31 ? per * unit : kLim31 - 1);
    };
    const int64_t key32 = ceil_div(p->kv_len, 32);
    x.kv_waves = (int)(key32 < 1 ? 1 : key32 < kAttnWaves ? key32 : kAttnWaves);
    x.key_tiles = (int)ceil_div(key32, x.kv_waves);
    // dk dv: one workgroup a CU (eight waves of many registers)
    split(kNumCUs, 2, bh * x.key_tiles, row64, kRowTile, &x.kv_nsplit, &x.kv_split);
    // Two waves a key block halve a workgroup's walk, but add up at its end,
    // and then leave room for one workgroup a CU instead of two: up to eight
    // row tiles one wave is as fast or faster (3 tiles of 3882 keys of 64:
    // 21 us, two waves 30; 8 tiles 16 both; 13 tiles of 77 keys 24 and 21).
    const int64_t walk = ceil_div(x.kv_split < rows ? x.kv_split : rows, kRowTile);
    x.kv_groups = p->head_dim <= 96 && walk <= 8 ? 1 : 2;
    x.row_tiles = (int)ceil_div(rows, kAttnWaves * 32);
    // dq: two a CU (four waves)
    split(2 * kNumCUs, 3, bh * x.row_tiles, key64, kKeyTile, &x.q_nsplit, &x.q_split);
    x.few_keys = p->kv_len <= kShortKeys;
    if (x.few_keys) {
        x.row_tiles = (int)short_tiles(bh, x.rows_pad, (p->head_dim <= 64 ? 2 : 1) * kNumCUs);
        x.q_nsplit = 1;
        x.bound_n = x.row_tiles * kAttnWaves;   // one a wave
    }
    x.stat_floats = 2 * bh * x.rows_pad;
    x.bound_words = p->dtype == IGC_DTYPE_FP16 ? 2 * bh * x.bound_n : 0;
    int64_t f = x.kv_nsplit > 1 ? 2 * x.kv_nsplit * bh * p->kv_len * p->head_dim : 0;
    const int64_t g = x.q_nsplit > 1 ? x.q_nsplit * bh * rows * p->head_dim : 0;
    x.part_floats = f > g ? f : g;
    return x;
}

size_t bwd_ws(const AttnGradPlan& x) {
    return (size_t)(x.part_floats + x.stat_floats + x.bound_words) * sizeof(float);
}

struct GradTensors {
    AttnTensors f;
    Tensor g, dq, dk, dv;
};

int32_t check_bwd(const igc_cross_attn_grad* p, GradTensors* t, AttnGradPlan* plan) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    const igc_cross_attn* f = &p->fwd;
    int32_t r;
    if ((r = check_attn_shape(f))) return r;
    if ((r = check_attn_views(f, &t->f, false))) return r;
    const int64_t d = f->head_dim;
    const bool rows = f->batch && f->q_len && f->q_heads;
    if (rows && !f->lse) return IGC_DECLINE_NULL_POINTER;
    if ((r = check_view(p->dout, f->batch, f->q_len, f->q_heads, d, false, kStrideLim, &t->g)))
        return r;
    t->dq = t->dk = t->dv = Tensor{nullptr, 0, 0, 0, 0};
    if (p->dq.data &&
        (r = check_view(p->dq, f->batch, f->q_len, f->q_heads, d, true, kStrideLim, &t->dq)))
        return r;
    if (f->batch && f->kv_len && f->kv_heads && !p->dk.data != !p->dv.data)
        return IGC_DECLINE_NULL_POINTER;
    if (p->dk.data) {
        if ((r = check_view(p->dk, f->batch, f->kv_len, f->kv_heads, d, true, kBatchStrideLim,
                            &t->dk)))
            return r;
        if ((r = check_view(p->dv, f->batch, f->kv_len, f->kv_heads, d, true, kBatchStrideLim,
                            &t->dv)))
            return r;
    }
    for (const Tensor* x : {&t->g, &t->dq})
        if (!packed_fits(f, *x)) return IGC_DECLINE_SIZE_LIMIT;
    *plan = bwd_plan(f);
    const int64_t bh = f->batch * f->kv_heads;
    if (bh > 0 &&
        (!launchable(bh * plan->key_tiles * plan->kv_nsplit,
                     plan->kv_waves * plan->kv_groups * 64) ||
         !launchable(bh * plan->row_tiles * plan->q_nsplit, kAttnWaves * 64) ||
         (!plan->few_keys && !launchable(bh * plan->bound_n, kAttnWaves * 64))))
        return IGC_DECLINE_SIZE_LIMIT;
    const size_t ws = bwd_ws(*plan);
    auto meets = [&](const void* w, size_t n) {
        return meets_inputs(f, t->f, w, n) || meet(w, n, t->f.o.p, t->f.o.bytes) ||
               meet(w, n, t->g.p, t->g.bytes) || meet(w, n, f->lse, lse_bytes(f));
    };
    for (const Tensor* x : {&t->dq, &t->dk, &t->dv})
        if (meets(x->p, x->bytes) || (f->workspace && meet(f->workspace, ws, x->p, x->bytes)))
            return IGC_DECLINE_OVERLAP;
    if (f->workspace && ws) {
        if (!aligned(f->workspace, 16)) return IGC_DECLINE_ALIGNMENT;
        if (f->workspace_bytes < ws) return IGC_DECLINE_WORKSPACE;
        if (meets(f->workspace, ws)) return IGC_DECLINE_OVERLAP;
    }
    return IGC_OK;
}

// ------------------------------------------------- norm and rotation
int32_t check_qk_shape(const igc_qk_norm* p) {
    if (!p) return IGC_DECLINE_NULL_POINTER;
    if (p->dtype != IGC_DTYPE_BF16 && p->dtype != IGC_DTYPE_FP16) return IGC_DECLINE_DTYPE;
    for (const igc_qk_part* x : {&p->q, &p->k}) {
        if (x->batch < 0 || x->tokens < 0 || x->heads < 0 || x->table_rows < 0)
            return IGC_DECLINE_SHAPE;
        if (x->batch >= kLim31 || x->tokens >= kLim31 || x->heads >= kLim31 ||
            x->table_rows >= kLim31)
            return IGC_DECLINE_SIZE_LIMIT;
        if (x->batch && x->tokens && x->heads &&
            (x->batch * x->tokens >= ((int64_t)1 << 40) / x->heads))
            return IGC_DECLINE_SIZE_LIMIT;
    }
    if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8) return IGC_DECLINE_HEAD_DIM;
    if (p->rot_dim < 0 || p->rot_dim > p->head_dim || p->rot_dim % 2) return IGC_DECLINE_HEAD_DIM;
    if (!(p->eps >= 0.0) || !isfinite((float)p->eps)) return IGC_DECLINE_SCALE;
    return IGC_OK;
}

struct QkTensors {
    Tensor x, g, o;
};

bool qk_empty(const igc_qk_part& x) { return !x.batch || !x.tokens || !x.heads; }

bool same_view(const Tensor& a, const Tensor& b) {
    return a.p == b.p && a.b == b.b && a.t == b.t && a.h == b.h;
}

// Rounds of 256 threads that one part needs.
int64_t qk_tiles(const igc_qk_part& x, int64_t d) {
    if (qk_empty(x)) return 0;
    const int64_t items = x.batch * x.tokens * ceil_div(x.heads, kQkHeads);
    return ceil_div(items, kQkThreads / qk_lanes((int)d));
}

// Workgroups of one part.  Backward they loop, so that the partial weight
// gradients stay few: as many as run at once, both parts together (one more
// would run alone at the end: 16 x 4096 queries and 1024 keys of 128, 242 us
// with 769 workgroups), with the same number of rounds each (32 x 3136 queries
// and 333 keys, 8 heads of 64: 74 us; with up to 1024 a part 83).  Registers
// for a fourth workgroup a CU would spill (82 us).
int64_t qk_blocks(const igc_qk_norm* p, const igc_qk_part& x, bool backward) {
    const int64_t n = qk_tiles(x, p->head_dim);
    if (!backward || n == 0) return n;
    const int64_t q = qk_tiles(p->q, p->head_dim), k = qk_tiles(p->k, p->head_dim);
    int64_t rounds = ceil_div(q + k, kQkBwdBlocks);
    // two parts round up
    if (ceil_div(q, rounds) + ceil_div(k, rounds) > kQkBwdBlocks)
        rounds = ceil_div(q + k, kQkBwdBlocks - 1);
    return ceil_div(n, rounds);
}

size_t qk_ws(const igc_qk_norm* p) {
    if (!p->q.dweight && !p->k.dweight) return 0;
    return (size_t)((qk_blocks(p, p->q, true) + qk_blocks(p, p->k, true)) *
                    qk_lanes((int)p->head_dim) * 8) * sizeof(float);
}

int32_t check_qk(const igc_qk_norm* p, bool backward, QkTensors t[2]) {
    int32_t r;
    if ((r = check_qk_shape(p))) return r;
    const igc_qk_part* parts[2] = {&p->q, &p->k};
    const int64_t d = p->head_dim;
    const size_t ws = backward ? qk_ws(p) : 0;
    bool in_place = true;
    for (int i = 0; i < 2; ++i) {
        const igc_qk_part& x = *parts[i];
        const int64_t nb = qk_empty(x) ? 0 : x.batch;
        const int64_t lim = kBatchStrideLim;   // every row has a 64-bit address
        if ((r = check_view(x.x, nb, x.tokens, x.heads, d, false, lim, &t[i].x))) return r;
        if ((r = check_view(x.out, nb, x.tokens, x.heads, d, true, lim, &t[i].o))) return r;
        t[i].g = t[i].x;
        if (backward && (r = check_view(x.grad, nb, x.tokens, x.heads, d, false, lim, &t[i].g)))
            return r;
        if (!aligned(x.weight, 4) || !aligned(x.dweight, 4) || !aligned(x.table, 4) ||
            !aligned(x.positions, 4))
            return IGC_DECLINE_ALIGNMENT;
        if (!nb) continue;
        if (p->rot_dim && !x.table) return IGC_DECLINE_NULL_POINTER;
        if (p->rot_dim && !x.positions && x.table_rows < x.tokens) return IGC_DECLINE_SHAPE;
        if (p->rot_dim && x.positions && x.table_rows == 0) return IGC_DECLINE_SHAPE;
        if (x.positions && (x.positions_stride < 0 || x.positions_stride >= kBatchStrideLim))
            return IGC_DECLINE_STRIDE;
        if (x.positions && (double)(x.batch - 1) * (double)x.positions_stride > kExtentLim)
            return IGC_DECLINE_SIZE_LIMIT;
        if (backward) {
            if (meet(t[i].o.p, t[i].o.bytes, t[i].x.p, t[i].x.bytes)) return IGC_DECLINE_OVERLAP;
            if (!same_view(t[i].o, t[i].g)) {
                in_place = false;
                if (meet(t[i].o.p, t[i].o.bytes, t[i].g.p, t[i].g.bytes))
                    return IGC_DECLINE_OVERLAP;
            }
        } else if (!same_view(t[i].o, t[i].x)) {
            in_place = false;
            if (meet(t[i].o.p, t[i].o.bytes, t[i].x.p, t[i].x.bytes)) return IGC_DECLINE_OVERLAP;
        }
    }
    // both parts are of checked sizes here
    const int64_t blocks = qk_blocks(p, p->q, backward) + qk_blocks(p, p->k, backward);
    if (!launchable(blocks, kQkThreads)) return IGC_DECLINE_SIZE_LIMIT;
    for (int i = 0; i < 2; ++i) {
        const Tensor &o = t[i].o, &ox = t[1 - i].x, &og = t[1 - i].g;
        if ((!in_place || backward) && meet(o.p, o.bytes, ox.p, ox.bytes))
            return IGC_DECLINE_OVERLAP;
        if (!in_place && meet(o.p, o.bytes, og.p, og.bytes)) return IGC_DECLINE_OVERLAP;
        for (int j = 0; j < 2; ++j) {
            // small inputs against everything written
            const igc_qk_part& y = *parts[j];
            const struct { const void* p; size_t n; } in[3] = {
                {y.weight, (size_t)d * 4},
                {y.table, (size_t)(y.table_rows * p->rot_dim) * 4},
                {y.positions, qk_empty(y) ? 0
                                          : (size_t)((y.batch - 1) * y.positions_stride +
                                                     y.tokens) * 4}};
            const void* dw = backward ? parts[i]->dweight : nullptr;
            for (const auto& s : in)
                if (meet(s.p, s.n, o.p, o.bytes) || meet(s.p, s.n, dw, (size_t)d * 4) ||
                    (ws && meet(s.p, s.n, p->workspace, ws)))
                    return IGC_DECLINE_OVERLAP;
            if (meet(dw, (size_t)d * 4, t[j].x.p, t[j].x.bytes) ||
                meet(dw, (size_t)d * 4, t[j].g.p, t[j].g.bytes) ||
                meet(dw, (size_t)d * 4, t[j].o.p, t[j].o.bytes))
                return IGC_DECLINE_OVERLAP;
        }
        if (ws && p->workspace &&
            (meet(p->workspace, ws, o.p, o.bytes) || meet(p->workspace, ws, t[i].x.p, t[i].x.bytes) ||
             meet(p->workspace, ws, t[i].g.p, t[i].g.bytes) ||
             meet(p->workspace, ws, parts[i]->dweight, (size_t)d * 4)))
            return IGC_DECLINE_OVERLAP;
    }
    if (backward && p->q.dweight &&
        meet(p->q.dweight, (size_t)d * 4, p->k.dweight, (size_t)d * 4))
        return IGC_DECLINE_OVERLAP;
    if (ws && p->workspace) {
        if (!aligned(p->workspace, 16)) return IGC_DECLINE_ALIGNMENT;
        if (p->workspace_bytes < ws) return IGC_DECLINE_WORKSPACE;
    }
    return IGC_OK;
}

int32_t run_qk(const igc_qk_norm* p, bool backward, void* stream) {
    QkTensors t[2];
    if (check_qk(p, backward, t) != IGC_OK) return 0;
    const igc_qk_part* parts[2] = {&p->q, &p->k};
    QkArgs a{};
    a.D = (int)p->head_dim;
    a.R = (int)p->rot_dim;
    a.eps = (float)p->eps;
    a.inv_d = 1.0f / (float)a.D;
    for (int i = 0; i < 2; ++i) {
        const igc_qk_part& x = *parts[i];
        QkPart& o = a.part[i];
        o.x = (const uint8_t*)t[i].x.p;
        o.dy = (const uint8_t*)t[i].g.p;
        o.out = (uint8_t*)const_cast<void*>(t[i].o.p);
        o.w = x.weight;
        o.dw = backward ? x.dweight : nullptr;
        o.table = a.R ? x.table : nullptr;
        o.table_rows = (int)x.table_rows;
        o.pos = x.positions;
        o.pos_b = x.positions_stride;
        o.x_b = t[i].x.b; o.x_t = t[i].x.t; o.x_h = t[i].x.h;
        o.dy_b = t[i].g.b; o.dy_t = t[i].g.t; o.dy_h = t[i].g.h;
        o.o_b = t[i].o.b; o.o_t = t[i].o.t; o.o_h = t[i].o.h;
        o.B = (int)x.batch;
        o.T = (int)x.tokens;
        o.H = (int)x.heads;
        o.hc = (int)ceil_div(x.heads, kQkHeads);
        o.items = qk_empty(x) ? 0 : x.batch * x.tokens * o.hc;
        o.blocks = (int)qk_blocks(p, x, backward);
    }
    const int mode = p->interleaved ? ROT_PAIRS : a.R % 16 == 0 ? ROT_HALVES : ROT_HALVES_ANY;
    const hipStream_t st = (hipStream_t)stream;
    void* own = nullptr;
    const size_t ws = backward ? qk_ws(p) : 0;
    if (ws) {
        void* w = p->workspace;
        if (!w) {
            const hipError_t e = hipMallocAsync(&own, ws, st);
            if (e != hipSuccess) return -(int32_t)e;
            w = own;
        }
        a.partial = (float*)w;
    }
    hipError_t e = p->dtype == IGC_DTYPE_BF16 ? launch_qk_norm<DT_BF16>(a, mode, backward, st)
                                              : launch_qk_norm<DT_FP16>(a, mode, backward, st);
    if (own) {
        const hipError_t f = hipFreeAsync(own, st);
        if (e == hipSuccess) e = f;
    }
    return e == hipSuccess ? 1 : -(int32_t)e;
}

}  // namespace

extern "C" {

int32_t cross_attn_bwd_check(const igc_cross_attn_grad* args) {
    GradTensors t;
    AttnGradPlan plan;
    return check_bwd(args, &t, &plan);
}

size_t cross_attn_bwd_workspace_bytes(const igc_cross_attn_grad* args) {
    if (!args || check_attn_shape(&args->fwd) != IGC_OK) return 0;
    return bwd_ws(bwd_plan(&args->fwd));
}

int32_t cross_attn_bwd(const igc_cross_attn_grad* args, void* stream) {
    GradTensors t;
    AttnGradPlan plan;
    if (check_bwd(args, &t, &plan) != IGC_OK) return 0;
    const igc_cross_attn* f = &args->fwd;
    if (f->batch == 0 || f->kv_heads == 0) return 1;
    const hipStream_t st = (hipStream_t)stream;
    AttnArgs a = attn_args(f, t.f);
    a.o = (const uint8_t*)t.f.o.p;
    a.dout = (const uint8_t*)t.g.p;
    a.do_b = t.g.b; a.do_t = t.g.t; a.do_h = t.g.h;
    a.dq = (uint8_t*)const_cast<void*>(t.dq.p);
    a.dq_b = t.dq.b; a.dq_t = t.dq.t; a.dq_h = t.dq.h;
    a.dk = (uint8_t*)const_cast<void*>(t.dk.p);
    a.dk_b = t.dk.b; a.dk_t = t.dk.t; a.dk_h = t.dk.h;
    a.dv = (uint8_t*)const_cast<void*>(t.dv.p);
    a.dv_b = t.dv.b; a.dv_t = t.dv.t; a.dv_h = t.dv.h;
    a.rows_pad = plan.rows_pad;
    a.bound_n = plan.bound_n;
    void* own = nullptr;
    if (const size_t ws = bwd_ws(plan)) {
        void* w = f->workspace;
        if (!w) {
            const hipError_t e = hipMallocAsync(&own, ws, st);
            if (e != hipSuccess) return -(int32_t)e;
            w = own;
        }
        a.part = (float*)w;
        a.stat = a.part + plan.part_floats;
        a.bound = (uint32_t*)(a.stat + plan.stat_floats);
    }
    hipError_t e = f->dtype == IGC_DTYPE_BF16 ? launch_attn_bwd<DT_BF16>(a, plan, st)
                                              : launch_attn_bwd<DT_FP16>(a, plan, st);
    if (own) {
        const hipError_t x = hipFreeAsync(own, st);
        if (e == hipSuccess) e = x;
    }
    return e == hipSuccess ? 1 : -(int32_t)e;
}

int32_t qk_norm_rope_fwd_check(const igc_qk_norm* args) {
    QkTensors t[2];
    return check_qk(args, false, t);
}

int32_t qk_norm_rope_bwd_check(const igc_qk_norm* args) {
    QkTensors t[2];
    return check_qk(args, true, t);
}

size_t qk_norm_rope_bwd_workspace_bytes(const igc_qk_norm* args) {
    return check_qk_shape(args) == IGC_OK ? qk_ws(args) : 0;
}

int32_t qk_norm_rope_fwd(const igc_qk_norm* args, void* stream) {
    return run_qk(args, false, stream);
}

int32_t qk_norm_rope_bwd(const igc_qk_norm* args, void* stream) {
    return run_qk(args, true, stream);
}

int32_t cross_attn_fwd_check(const igc_cross_attn* args) {
    AttnTensors t;
    AttnPlan plan;
    return check_fwd(args, &t, &plan);
}

size_t cross_attn_fwd_workspace_bytes(const igc_cross_attn* args) {
    if (check_attn_shape(args) != IGC_OK) return 0;
    return fwd_ws(fwd_plan(args));
}

int32_t cross_attn_fwd(const igc_cross_attn* args, void* stream) {
    AttnTensors t;
    AttnPlan plan;
    if (check_fwd(args, &t, &plan) != IGC_OK) return 0;
    if (args->batch == 0 || args->q_len == 0 || args->q_heads == 0) return 1;
    const hipStream_t st = (hipStream_t)stream;
    AttnArgs a = attn_args(args, t);
    a.out = (uint8_t*)t.o.p;
    a.row_tiles = plan.row_tiles;
    a.nsplit = plan.nsplit;
    a.split = plan.split;
    void* own = nullptr;
    if (const size_t ws = fwd_ws(plan)) {
        void* w = args->workspace;
        if (!w) {
            const hipError_t e = hipMallocAsync(&own, ws, st);
            if (e != hipSuccess) return -(int32_t)e;
            w = own;
        }
        a.part = (float*)w;
        a.stat = a.part + plan.part_floats;
    }
    hipError_t e = args->dtype == IGC_DTYPE_BF16 ? launch_attn_fwd<DT_BF16>(a, plan, st)
                                                 : launch_attn_fwd<DT_FP16>(a, plan, st);
    if (own) {
        const hipError_t f = hipFreeAsync(own, st);
        if (e == hipSuccess) e = f;
    }
    return e == hipSuccess ? 1 : -(int32_t)e;
}

}  // extern "C"
