// ssd_mixer_ops.cpp -- the C ABI of sliding-window attention with sinks and of
// the RMS norm with the residual's addition (declared in include/ssd.h):
// argument checks, workspace layout, launch plans.  Validation touches no HIP
// API, so every error path runs without a device.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "../../include/ssd.h"
#include "ssd_ops_host.h"
#include "ssd_ops_internal.h"

namespace ssd {

AttnBwdPlan attn_bwd_plan(const AttnArgs &a) {
    AttnBwdPlan p{};
    const int far = a.seqlen - a.window;  // queries that see token 0 as a sink only
    if (a.sinks == 0 || far <= 0) return p;
    const int keys = std::min(a.sinks, far);
    p.sink_tiles = (keys + kSinkKeys - 1) / kSinkKeys;
    // One tile of the kernel's, or as many as leave 64 partial sums to add.  The backward pass by chunks of 128, 256 and
    // 512: 2 x 2048 tokens, 40 heads of 64 over 8, 4 sinks 130, 136 and 149 us; one of 4096, 16 heads over 4 80, 78 and 80;
    // 3 x 257 fp32, heads of 32 32, 44 and 44.  By 16, 32, 64 and 128 sums: 16 384 tokens, 8 heads of 64 over 2 154, 131, 123
    // and 119; 32 768, heads of 128, 679, 626, 606 and 598, where the sums take twice the workspace.
    p.chunk = std::max(128, (far + 64 * 128 - 1) / (64 * 128) * 128);
    p.nchunks = (far + p.chunk - 1) / p.chunk;
    p.parts = 1 + p.nchunks;
    p.rows = (int64_t)p.sink_tiles * kSinkKeys;
    return p;
}

// One block walks all slots of a sequence and head of keys, or several blocks do
// and a second kernel joins them.  Times of one block and of several, us on the
// device (many calls in a captured graph) and, from Python, a call:
//   bf16 heads of 64, 8 walks:    6 turns  8.0, 8.7 and 11.3, 15.7
//     (a turn is 256 slots)       9       10.0, 7.8     11.6, 15.4
//                                12       12.0, 8.6     12.6, 15.1
//                                24       20.2, 8.7     20.8, 15.2
//     64 walks                   32       27.3, 26.9    27.4, 26.8
//     128 walks                  24       31.0, 34.5    31.0, 34.4
//   bf16 heads of 128, 8 walks:   8       11.8, 7.7     12.4, 15.4
//     (128 slots)                12       15.4, 9.0     16.0, 15.4
//   bf16 heads of 32, 8 walks:   14       10.8, 8.8     11.4, 15.4
//   fp32 heads of 128, 8 walks:   2       13.8, 11.5    14.4, 15.3
//     (64 slots)                  4       22.9, 11.8    23.4, 15.3
//     128 walks                   4       24.1, 18.9    24.2, 19.1
//   fp32 heads of 64, 8 walks:    4       14.0, 9.3     14.5, 15.5
// So a turn takes kTurnUs, a walk is not faster than memory (kBytesPerUs, caches
// that the last-level cache holds), and several blocks cost 3 us of the device's
// time and 4 more of the host's: kSplitUs lies where what a captured graph loses by
// one block and what a call from Python loses by several are alike.
constexpr float kTurnUs[2][3] = {{0.52f, 0.67f, 0.88f}, {2.2f, 2.4f, 4.45f}};  // bf16, fp32: heads of 32, 64, 128
constexpr float kSplitUs = 6.7f, kBytesPerUs = 8e6f;
// A block takes a compute unit's LDS, so that blocks run in rounds of 256 (128 walks, fp32 heads of 64, 12 turns: 256
// blocks 26.8 us, 512 32.5, 1024 36.3; 384 walks, fp32 heads of 128, 128 turns: 384 blocks, two rounds, 1167 us, 768 of
// half the turns, three rounds, 895).
constexpr int64_t kStepBlocks = 256, kStepRounds = 4;

AttnStepPlan attn_step_plan(const AttnArgs &a) {
    const int64_t esz = a.bf16 ? 2 : 4, slots = (int64_t)a.window + a.sinks, turn = 32 * attn_step_waves(a.headdim, (int)esz);
    const int64_t turns = (slots + turn - 1) / turn;
    // sequences, heads of keys, and blocks of 32 heads that share one
    const int64_t walks = std::max<int64_t>(1, a.batch * a.kvheads * ((a.heads / a.kvheads + 31) / 32));
    const float us = kTurnUs[a.bf16 ? 0 : 1][a.headdim / 64];
    const float least = (float)walks * (float)turns * (float)(turn * 2 * a.headdim * esz) / kBytesPerUs;
    const auto walk = [&](int64_t n) {
        const int64_t rounds = (walks * n + kStepBlocks - 1) / kStepBlocks, each = (turns + n - 1) / n;
        return std::max((float)rounds * (float)each * us, least);
    };
    int64_t splits = 1;
    float best = walk(1) - kSplitUs;
    for (int64_t rounds = 1; rounds <= kStepRounds; ++rounds) {
        const int64_t n = std::min(turns, rounds * kStepBlocks / walks);
        if (n > 1 && walk(n) < best) {
            best = walk(n);
            splits = n;
        }
    }
    const int64_t run = (turns + splits - 1) / splits * turn;
    return AttnStepPlan{(int)((slots + run - 1) / run), (int)run};
}

// 512 blocks: two for each compute unit (a wave's registers leave one to a SIMD).
NormBwdPlan norm_bwd_plan(const NormArgs &a) {
    const int64_t rows = a.batch * a.seqlen;
    const int64_t beside = a.channels <= kNormWaveRow ? 4 : 1;  // rows of a block at a time
    const int64_t parts = std::min<int64_t>((rows + beside - 1) / beside, 512);
    // sums over rows take 256 in 32 bits at most
    return NormBwdPlan{(int)std::max<int64_t>({1, parts, (rows + 256 * beside - 1) / (256 * beside)})};
}

namespace {

// ---------------------------------------------------------------------------
// Sliding-window attention with sinks
// ---------------------------------------------------------------------------

constexpr int64_t kMaxAttnRow = (int64_t)1 << 22;  // a tile's rows within 32-bit byte offsets

// Heads of d elements for (batch, seqlen, heads): as rows_of, and the alignment of the strides that count.
ssd_status heads_of(const ssd_head_stride &in, int64_t batch, int64_t seqlen, int64_t heads, int64_t d, size_t esz,
                    HeadStrides *out, size_t *bytes, bool *whole) {
    HeadStrides s{in.batch, in.row, in.head};
    int64_t dense;
    if (!product({batch, seqlen, heads, d}, &dense)) return SSD_ERROR_UNSUPPORTED;
    if (s.batch == 0 && s.row == 0 && s.head == 0) s = HeadStrides{seqlen * heads * d, heads * d, d};
    if (s.batch < 0 || s.row < 0 || s.head < 0 || (seqlen > 1 && s.row < d)) return SSD_ERROR_INVALID_VALUE;
    if (seqlen <= 1) s.row = d;  // these play no part
    if (heads <= 1) s.head = d;
    if (batch <= 1) s.batch = 0;
    *out = s;
    *bytes = 0;
    if (s.row >= kMaxAttnRow) return SSD_ERROR_UNSUPPORTED;
    if ((s.row * esz) % 16 != 0 || (s.head * esz) % 16 != 0 || (s.batch * esz) % 16 != 0) *whole = false;
    if (batch == 0 || seqlen == 0) return SSD_OK;
    const int64_t most = std::numeric_limits<int64_t>::max() / 64;
    int64_t b, r, h;
    if (!product({batch - 1, s.batch}, &b) || !product({seqlen - 1, s.row}, &r) || !product({heads - 1, s.head}, &h) ||
        b > most || r > most || h > most)
        return SSD_ERROR_UNSUPPORTED;
    *bytes = (size_t)(b + r + h + d) * esz;
    return SSD_OK;
}

struct AttnBytes {
    size_t q, k, v, y, dy;  // strided inputs
    size_t heads, kvheads, lse, cache, lens;
};

ssd_status check_attn(const ssd_attn_shape *s, bool cached, AttnArgs *a, AttnBytes *n) {
    if (s == nullptr) return SSD_ERROR_INVALID_VALUE;
    if (s->batch < 0 || s->seqlen < 0 || s->nheads < 1 || s->nkvheads < 1 || s->headdim < 1 || s->window < 1 ||
        s->sinks < 0 || s->reserved[0] != 0 || s->reserved[1] != 0)
        return SSD_ERROR_INVALID_VALUE;
    if (s->nheads % s->nkvheads != 0 || !dtype_ok(s->dtype)) return SSD_ERROR_INVALID_VALUE;
    // (the kernels multiply scores by scale log2(e))
    if (!(s->scale > 0.f) || !std::isfinite(s->scale * 1.4426950408889634f)) return SSD_ERROR_INVALID_VALUE;
    if (s->headdim != 32 && s->headdim != 64 && s->headdim != 128) return SSD_ERROR_UNSUPPORTED;
    if (s->batch > 65535 || s->seqlen > kMaxLen || s->nheads > 65535) return SSD_ERROR_UNSUPPORTED;
    if (cached && (s->window > kMaxLen || s->sinks > kMaxLen || s->window + s->sinks > kMaxLen))
        return SSD_ERROR_UNSUPPORTED;
    *a = AttnArgs{};
    *n = AttnBytes{};
    const size_t e = size_of(s->dtype);
    const int64_t qw = s->nheads * s->headdim, kw = s->nkvheads * s->headdim;
    const struct {
        const ssd_head_stride &in;
        int64_t heads;
        HeadStrides *out;
        size_t *bytes;
    } rows[] = {{s->q, s->nheads, &a->qs, &n->q},
                {s->k, s->nkvheads, &a->ks, &n->k},
                {s->v, s->nkvheads, &a->vs, &n->v},
                {s->y, s->nheads, &a->ys, &n->y},
                {s->dy, s->nheads, &a->dys, &n->dy}};
    bool whole = true;
    for (const auto &r : rows) {
        const ssd_status st = heads_of(r.in, s->batch, s->seqlen, r.heads, s->headdim, e, r.out, r.bytes, &whole);
        if (st != SSD_OK) return st;
    }
    if (!whole) return SSD_ERROR_MISALIGNED;
    int64_t t;
    // every buffer within int64, and fewer than 2^23 blocks of 128 queries or keys (and 512 threads at most: 32 bits)
    const int64_t slots = cached ? s->window + s->sinks : 0;
    if (!product({s->batch, s->nkvheads, slots, s->headdim, 4}, &t) ||
        !product({s->batch, s->seqlen, qw, 4}, &t) || !product({s->batch, s->nheads, s->seqlen / 32 + 4}, &t) ||
        t >= (int64_t)1 << 25)
        return SSD_ERROR_UNSUPPORTED;
    a->batch = s->batch;
    a->seqlen = (int)s->seqlen;
    a->heads = (int)s->nheads;
    a->kvheads = (int)s->nkvheads;
    a->headdim = (int)s->headdim;
    a->window = (int)std::min<int64_t>(s->window, kAttnFar);
    a->sinks = (int)std::min<int64_t>(s->sinks, kAttnFar);
    a->scale = s->scale;
    a->bf16 = s->dtype == SSD_DTYPE_BF16;
    const size_t tok = (size_t)(s->batch * s->seqlen);
    n->heads = tok * qw * e;
    n->kvheads = tok * kw * e;
    n->lse = tok * s->nheads * 4;
    n->cache = (size_t)(s->batch * s->nkvheads * slots * s->headdim) * e;
    n->lens = (size_t)s->batch * 4;
    return SSD_OK;
}

size_t attn_bwd_carve(AttnArgs *a, const AttnBwdPlan &p, void *ws) {
    Carver w{static_cast<unsigned char *>(ws), 0};
    a->stats = w.take((size_t)a->batch * a->heads * a->seqlen * 2);
    a->partials = w.take((size_t)a->batch * a->kvheads * p.parts * 2 * p.rows * a->headdim);
    return w.off;
}

size_t attn_step_carve(AttnArgs *a, const AttnStepPlan &p, void *ws) {
    if (p.splits == 1) return 0;
    Carver w{static_cast<unsigned char *>(ws), 0};
    const size_t n = (size_t)a->batch * a->heads * p.splits;
    a->part_y = w.take(n * a->headdim);
    a->part_ml = w.take(n * 2);
    return w.off;
}

// The backward pass's partial sums within int64, its sinks' blocks below 2^23.
ssd_status check_attn_bwd(const ssd_attn_shape *s, AttnArgs *a, AttnBytes *n) {
    const ssd_status st = check_attn(s, false, a, n);
    if (st != SSD_OK) return st;
    const AttnBwdPlan p = attn_bwd_plan(*a);
    int64_t t;
    if (!product({a->batch, a->kvheads, p.parts, 2 * p.rows, a->headdim, 4}, &t)) return SSD_ERROR_UNSUPPORTED;
    if (!product({a->batch * a->kvheads, (int64_t)p.sink_tiles * p.nchunks}, &t) ||
        t >= (int64_t)1 << 23)
        return SSD_ERROR_UNSUPPORTED;
    return SSD_OK;
}

ssd_status check_attn_step(const ssd_attn_shape *s, AttnArgs *a, AttnBytes *n) {
    const ssd_status st = check_attn(s, true, a, n);
    if (st != SSD_OK) return st;
    return s->seqlen == 1 ? SSD_OK : SSD_ERROR_INVALID_VALUE;
}

// ---------------------------------------------------------------------------
// RMS norm
// ---------------------------------------------------------------------------

struct NormBytes {
    size_t x, residual, dy, dres;  // strided inputs
    size_t row, tok_x, tok_res, tok_y, scales, lens;
};

Stored stored(int32_t t) { return t == SSD_DTYPE_F32 ? Stored::f32 : t == SSD_DTYPE_BF16 ? Stored::bf16 : Stored::e4m3; }

ssd_status check_norm(const ssd_norm_shape *s, bool backward, NormArgs *a, NormBytes *n) {
    if (s == nullptr) return SSD_ERROR_INVALID_VALUE;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->reserved != 0) return SSD_ERROR_INVALID_VALUE;
    const bool codes = s->y_dtype == SSD_DTYPE_E4M3;
    if (!dtype_ok(s->dtype) || !dtype_ok(s->res_dtype) || !(dtype_ok(s->y_dtype) || (codes && !backward)))
        return SSD_ERROR_INVALID_VALUE;
    if (!(s->eps >= 0.f) || !std::isfinite(s->eps)) return SSD_ERROR_INVALID_VALUE;
    if (codes ? s->scale_block != 0 && s->scale_block != 32 && s->scale_block != 64 && s->scale_block != 128
              : s->scale_block != 0)
        return SSD_ERROR_INVALID_VALUE;
    if (s->batch > 65535 || s->seqlen > kMaxLen || s->channels >= kMaxRow) return SSD_ERROR_UNSUPPORTED;
    *a = NormArgs{};
    *n = NormBytes{};
    const size_t i = size_of(s->dtype), r = size_of(s->res_dtype), o = codes ? 1 : size_of(s->y_dtype);
    const struct {
        const ssd_stride &in;
        size_t esz;
        Strides *out;
        size_t *bytes;
    } rows[] = {{s->x, i, &a->xs, &n->x}, {s->residual, r, &a->rs, &n->residual}, {s->dy, o, &a->dys, &n->dy}, {s->dres, r, &a->drs, &n->dres}};
    for (const auto &q : rows) {
        const ssd_status st = rows_of(q.in, s->batch, s->seqlen, s->channels, q.esz, q.out, q.bytes);
        if (st != SSD_OK) return st;
        if (q.out->row >= kMaxRow) return SSD_ERROR_UNSUPPORTED;
    }
    int64_t t;
    if (!product({s->batch, s->seqlen}, &t) || t >= (int64_t)1 << 31) return SSD_ERROR_UNSUPPORTED;
    a->batch = s->batch;
    a->seqlen = (int)s->seqlen;
    a->channels = (int)s->channels;
    a->scale_block = s->scale_block;
    a->eps = s->eps;
    a->x = stored(s->dtype);
    a->res = stored(s->res_dtype);
    a->y = stored(s->y_dtype);
    const size_t tok = (size_t)t;
    n->row = (size_t)s->channels * 4;
    n->tok_x = tok * s->channels * i;
    n->tok_res = tok * s->channels * r;
    n->tok_y = tok * s->channels * o;
    n->scales = tok * (s->scale_block == 0 ? 1 : (s->channels + s->scale_block - 1) / s->scale_block) * 4;
    n->lens = (size_t)s->batch * 4;
    return SSD_OK;
}

size_t norm_workspace(const NormArgs &a) {
    return align_up((size_t)norm_bwd_plan(a).parts * a.channels * sizeof(float));
}

// The very buffer of an input may be an output only where both are dense.
const void *in_place(const void *in, const Strides &s, const NormArgs &a) {
    const bool dense = (a.seqlen <= 1 || s.row == a.channels) && (a.batch <= 1 || s.batch == (int64_t)a.seqlen * a.channels);
    return dense ? in : nullptr;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_window_attn_fwd(const ssd_attn_shape *shape, const void *q, const void *k, const void *v,
                               const int32_t *positions, const int32_t *lengths, void *k_cache, void *v_cache,
                               void *y, float *lse, void *stream) {
    AttnArgs a;
    AttnBytes n;
    const bool cached = k_cache != nullptr || v_cache != nullptr;
    ssd_status st = check_attn(shape, cached, &a, &n);
    if (st != SSD_OK) return st;
    if ((k_cache == nullptr) != (v_cache == nullptr) || (positions != nullptr && !cached)) return SSD_ERROR_INVALID_VALUE;
    st = check_buffers({{q, n.q, 16, true},
                        {k, n.k, 16, true},
                        {v, n.v, 16, true},
                        {positions, n.lens, 4, false},
                        {lengths, n.lens, 4, false}},
                       {{k_cache, n.cache, 16, false}, {v_cache, n.cache, 16, false}, {y, n.heads, 16, true}, {lse, n.lse, 4, false}});
    if (st != SSD_OK) return st;
    if (a.batch == 0 || a.seqlen == 0) return SSD_OK;
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.lengths = lengths;
    a.kc = k_cache;
    a.vc = v_cache;
    a.y = y;
    a.lse = lse;
    return launch_attn_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

size_t ssd_window_attn_bwd_workspace_size(const ssd_attn_shape *shape) {
    AttnArgs a;
    AttnBytes n;
    return check_attn_bwd(shape, &a, &n) == SSD_OK ? attn_bwd_carve(&a, attn_bwd_plan(a), nullptr) : 0;
}

ssd_status ssd_window_attn_bwd(const ssd_attn_shape *shape, const void *q, const void *k, const void *v,
                               const void *y, const float *lse, const void *dy, const int32_t *lengths, void *dq,
                               void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream) {
    AttnArgs a;
    AttnBytes n;
    ssd_status st = check_attn_bwd(shape, &a, &n);
    if (st != SSD_OK) return st;
    const AttnBwdPlan plan = attn_bwd_plan(a);
    const size_t need = attn_bwd_carve(&a, plan, workspace);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SSD_ERROR_WORKSPACE;
    st = check_buffers({{q, n.q, 16, true},
                        {k, n.k, 16, true},
                        {v, n.v, 16, true},
                        {y, n.y, 16, true},
                        {lse, n.lse, 4, true},
                        {dy, n.dy, 16, true},
                        {lengths, n.lens, 4, false}},
                       {{dq, n.heads, 16, true}, {dk, n.kvheads, 16, true}, {dv, n.kvheads, 16, true}, {workspace, need, kAlign, false}});
    if (st != SSD_OK) return st;
    if (a.batch == 0 || a.seqlen == 0) return SSD_OK;
    a.q = q;
    a.k = k;
    a.v = v;
    a.y = const_cast<void *>(y);
    a.lse = const_cast<float *>(lse);
    a.dy = dy;
    a.lengths = lengths;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    return launch_attn_bwd(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

size_t ssd_window_attn_step_workspace_size(const ssd_attn_shape *shape) {
    AttnArgs a;
    AttnBytes n;
    return check_attn_step(shape, &a, &n) == SSD_OK ? attn_step_carve(&a, attn_step_plan(a), nullptr) : 0;
}

ssd_status ssd_window_attn_step(const ssd_attn_shape *shape, const void *q, const void *k, const void *v,
                                const int32_t *positions, void *k_cache, void *v_cache, void *y, void *workspace,
                                size_t workspace_bytes, void *stream) {
    AttnArgs a;
    AttnBytes n;
    ssd_status st = check_attn_step(shape, &a, &n);
    if (st != SSD_OK) return st;
    const AttnStepPlan plan = attn_step_plan(a);
    const size_t need = attn_step_carve(&a, plan, workspace);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SSD_ERROR_WORKSPACE;
    st = check_buffers({{q, n.q, 16, true}, {k, n.k, 16, true}, {v, n.v, 16, true}, {positions, n.lens, 4, true}},
                       {{k_cache, n.cache, 16, true}, {v_cache, n.cache, 16, true}, {y, n.heads, 16, true}, {workspace, need, kAlign, false}});
    if (st != SSD_OK) return st;
    if (a.batch == 0) return SSD_OK;
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.kc = k_cache;
    a.vc = v_cache;
    a.y = y;
    return launch_attn_step(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

ssd_status ssd_rms_norm_fwd(const ssd_norm_shape *shape, const void *x, const void *residual, const float *weight,
                            const int32_t *lengths, void *y, float *scales, void *residual_out, void *stream) {
    NormArgs a;
    NormBytes n;
    ssd_status st = check_norm(shape, false, &a, &n);
    if (st != SSD_OK) return st;
    const bool codes = a.y == Stored::e4m3;
    if (!codes && scales != nullptr) return SSD_ERROR_INVALID_VALUE;
    const size_t i = size_of(shape->dtype), r = size_of(shape->res_dtype);
    st = check_buffers({{x, n.x, i, true},
                        {residual, n.residual, r, false},
                        {weight, n.row, 4, false},
                        {lengths, n.lens, 4, false}},
                       {{y, n.tok_y, codes ? 1 : size_of(shape->y_dtype), true},
                        {scales, n.scales, 4, codes},
                        {residual_out, n.tok_res, r, false, in_place(residual, a.rs, a)}});
    if (st != SSD_OK) return st;
    if (a.batch == 0 || a.seqlen == 0) return SSD_OK;
    a.in = x;
    a.residual = residual;
    if (residual == nullptr && residual_out == nullptr) a.res = Stored::none;
    a.weight = weight;
    a.lengths = lengths;
    a.out = y;
    a.scales = scales;
    a.residual_out = residual_out;
    return launch_norm_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

size_t ssd_rms_norm_bwd_workspace_size(const ssd_norm_shape *shape) {
    NormArgs a;
    NormBytes n;
    return check_norm(shape, true, &a, &n) == SSD_OK ? norm_workspace(a) : 0;
}

ssd_status ssd_rms_norm_bwd(const ssd_norm_shape *shape, const void *dy, const void *u, const float *weight,
                            const void *d_residual_out, const int32_t *lengths, void *dx, void *d_residual,
                            float *dweight, void *workspace, size_t workspace_bytes, void *stream) {
    NormArgs a;
    NormBytes n;
    ssd_status st = check_norm(shape, true, &a, &n);
    if (st != SSD_OK) return st;
    const size_t need = norm_workspace(a);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SSD_ERROR_WORKSPACE;
    const size_t i = size_of(shape->dtype), r = size_of(shape->res_dtype), o = size_of(shape->y_dtype);
    st = check_buffers({{dy, n.dy, o, true},
                        {u, n.residual, r, true},
                        {weight, n.row, 4, false},
                        {d_residual_out, n.dres, r, false},
                        {lengths, n.lens, 4, false}},
                       {{dx, n.tok_x, i, true},
                        {d_residual, n.tok_res, r, false, in_place(d_residual_out, a.drs, a)},
                        {dweight, n.row, 4, false},
                        {workspace, need, kAlign, false}});
    if (st != SSD_OK) return st;
    // without tokens the sums are 0
    if (a.batch * a.seqlen == 0 && dweight == nullptr) return SSD_OK;
    a.in = dy;
    a.residual = u;
    a.weight = weight;
    a.dres = d_residual_out;
    a.lengths = lengths;
    a.out = dx;
    a.residual_out = d_residual;
    a.dweight = dweight;
    a.partials = static_cast<float *>(workspace);
    return launch_norm_bwd(a, norm_bwd_plan(a), static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

}  // extern "C"
