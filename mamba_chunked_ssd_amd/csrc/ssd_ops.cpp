// ssd_ops.cpp -- the C ABI of the short causal convolution and the selective
// scan (declared in include/ssd.h): argument checks, workspace layout, launch
// plans.  Validation touches no HIP API, so every error path runs without a
// device.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <limits>

#include "../../include/ssd.h"
#include "ssd_host.h"
#include "ssd_ops_internal.h"

namespace ssd {

// Strips long enough that the group formed twice and the partial sums stay
// small, short enough that every SIMD gets two waves (2 x 2048 tokens of 5376
// channels: 46 us with the 32 tokens this gives, 50 with 16, 47 with 64, 54 with
// 128; 3 x 1021 tokens of 264: 17 us with its 16, 27 with 128).
ConvBwdPlan conv_bwd_plan(int64_t batch, int64_t seqlen, int64_t channels) {
    ConvBwdPlan p;
    // of four channels a lane; with one there are up to four times as many
    const int64_t waves = (channels + 255) / 256;
    p.strip = 128;
    while (p.strip > 16 && batch * waves * ((seqlen + p.strip - 1) / p.strip) < 2 * 1024) p.strip /= 2;
    p.nstrips = (int)std::max<int64_t>(1, (seqlen + p.strip - 1) / p.strip);
    p.parts = batch * ((p.nstrips + 3) / 4);
    return p;
}

// Segments of the time axis.  They cost the summary pass (two thirds of the
// output pass's work; the backward sweep is there anyway) and a carry whose
// time grows with their number, and pay by filling the SIMDs: one wave alone
// runs at 45 % of a SIMD's rate, six at 80 %.
//
// Whole or cut, forward: whole, the time goes in steps with the waves on the
// fullest of the 1024 SIMDs, cut, with the waves.  Measured per 2048 tokens of
// 16 states (5120 channels are 320 waves a sequence), whole and cut:
//   1280 waves 387 and 284 us, 1600 388 and 355, 1920 390 and 424,
//   2240 512 and 483, 2560 513 and 544, 3200 607 and 670,
// which 180 + 105 steps and 25 + 0.203 waves follow within 4 %.  Backward: 2560
// waves 1691 and 1602 us, 3840 2366 and 2327, 5120 2812 and 3050.
//
// How many, when cut: enough for 16 384 waves (4 x 2048 tokens 281 us, with
// 8192 waves 306), but no more than the square root of the length, or the carry
// weighs.  With half the root, the root, 1.5, 2 and 4 times it: 65 536 tokens of
// 64 channels forward 132, 94, 102, 103 and 148 us, backward 288, 180, 186, 174
// and 234; 8191 of 771 forward 92, 84, 85, 87 and 95, backward 204, 181, 183,
// 181 and 192.
constexpr int64_t kBwdWhole = 4096, kScanWaves = 16384;
bool scan_whole(int64_t waves, bool backward) {
    if (backward) return waves >= kBwdWhole;
    return 180 + 105 * ((waves + 1023) / 1024) <= 25 + waves * 203 / 1000;
}
ScanPlan scan_plan(int64_t batch, int64_t seqlen, int64_t channels, int64_t dstate, int64_t ngroups, bool backward) {
    ScanPlan p;
    // the backward pass has no layout of two lanes a channel (its registers do not hold 8 tokens a lane)
    p.np = backward ? std::max(16, padded_states(dstate)) : padded_states(dstate);
    const int64_t cpg = channels / ngroups, cb = 1024 / p.np;
    p.gblocks = (int)((cpg + cb - 1) / cb);
    p.nblk = (int)(ngroups * p.gblocks);
    p.tiles = (seqlen + kScanSegment - 1) / kScanSegment * (kScanSegment / kScanTile);
    const int64_t waves = std::max<int64_t>(1, batch * p.nblk * 4);
    const int64_t root = (int64_t)std::ceil(std::sqrt((double)seqlen));
    int64_t nseg = scan_whole(waves, backward) ? 1 : (kScanWaves + waves - 1) / waves;
    nseg = std::max<int64_t>(1, std::min<int64_t>({nseg, seqlen / 16, root}));
    int64_t len = (seqlen + nseg - 1) / nseg;
    len = std::max<int64_t>(kScanSegment, (len + kScanSegment - 1) / kScanSegment * kScanSegment);
    p.seglen = (int)len;
    p.nseg = (int)std::max<int64_t>(1, (seqlen + len - 1) / len);
    p.runs = (int)((len + kScanRun - 1) / kScanRun);
    return p;
}

namespace {

constexpr int64_t kMaxLen = (int64_t)1 << 30;
constexpr int64_t kMaxRow = (int64_t)1 << 24;

bool product(std::initializer_list<int64_t> v, int64_t *out) {
    int64_t r = 1;
    for (int64_t x : v) {
        if (x < 0 || (x != 0 && r > std::numeric_limits<int64_t>::max() / 16 / x)) return false;
        r *= x;
    }
    *out = r;
    return true;
}

// Rows of `width` elements for (batch, seqlen): fills in the dense strides for
// {0, 0}; *bytes is what lies between the first and the last element.
ssd_status rows_of(const ssd_stride &in, int64_t batch, int64_t seqlen, int64_t width, size_t esz, Strides *out,
                   size_t *bytes) {
    Strides s{in.batch, in.row};
    int64_t dense;
    if (!product({batch, seqlen, width}, &dense)) return SSD_ERROR_UNSUPPORTED;
    if (s.batch == 0 && s.row == 0) s = Strides{seqlen * width, width};
    if (s.batch < 0 || s.row < 0 || (seqlen > 1 && s.row < width)) return SSD_ERROR_INVALID_VALUE;
    if (seqlen <= 1) s.row = width;  // plays no part
    *out = s;
    *bytes = 0;
    if (batch == 0 || seqlen == 0) return SSD_OK;
    int64_t span_b, span_r;
    if (!product({batch - 1, s.batch}, &span_b) || !product({seqlen - 1, s.row}, &span_r))
        return SSD_ERROR_UNSUPPORTED;
    const int64_t most = std::numeric_limits<int64_t>::max() / 16;
    if (span_b > most - span_r || span_b + span_r > most - width) return SSD_ERROR_UNSUPPORTED;
    *bytes = (size_t)(span_b + span_r + width) * esz;
    return SSD_OK;
}

// One buffer of a call: what the checks need to know of it.
struct Buffer {
    const void *ptr;
    size_t bytes;
    size_t align;
    bool required;
    const void *may_be = nullptr;  // an output: the one input it may be (initial and final state)
};

// Required pointers, alignment, and that no output meets another buffer.
ssd_status check_buffers(std::initializer_list<Buffer> ins, std::initializer_list<Buffer> outs) {
    for (const auto *list : {&ins, &outs})
        for (const Buffer &x : *list)
            if (x.required && x.bytes > 0 && x.ptr == nullptr) return SSD_ERROR_INVALID_VALUE;
    for (const auto *list : {&ins, &outs})
        for (const Buffer &x : *list)
            if (!aligned(x.ptr, x.align)) return SSD_ERROR_MISALIGNED;
    for (const Buffer &o : outs) {
        if (o.ptr == nullptr) continue;
        const Range r = range_of(o.ptr, o.bytes);
        for (const Buffer &i : ins)
            if (i.ptr != nullptr && !(i.ptr == o.ptr && i.ptr == o.may_be) && overlap(r, range_of(i.ptr, i.bytes)))
                return SSD_ERROR_INVALID_VALUE;
        for (const Buffer &q : outs)
            if (&q != &o && q.ptr != nullptr && overlap(r, range_of(q.ptr, q.bytes))) return SSD_ERROR_INVALID_VALUE;
    }
    return SSD_OK;
}

bool dtype_ok(int32_t t) { return t == SSD_DTYPE_F32 || t == SSD_DTYPE_BF16; }
size_t size_of(int32_t t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }

// ---------------------------------------------------------------------------
// Short causal convolution
// ---------------------------------------------------------------------------

struct ConvBytes {
    size_t x, dy;           // strided inputs
    size_t row, filter, y, dx, state, state32;
};

ssd_status check_conv(const ssd_conv_shape *s, ConvArgs *a, ConvBytes *n) {
    if (s == nullptr) return SSD_ERROR_INVALID_VALUE;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->reserved != 0) return SSD_ERROR_INVALID_VALUE;
    if (!dtype_ok(s->dtype) || (s->y_dtype != SSD_DTYPE_F32 && s->y_dtype != s->dtype) ||
        (s->dx_dtype != SSD_DTYPE_F32 && s->dx_dtype != s->dtype))
        return SSD_ERROR_INVALID_VALUE;
    if (s->activation != SSD_ACT_NONE && s->activation != SSD_ACT_SILU) return SSD_ERROR_INVALID_VALUE;
    if (s->width < 1) return SSD_ERROR_INVALID_VALUE;
    if (s->width < 2 || s->width > 4) return SSD_ERROR_UNSUPPORTED;
    if (s->batch > 65535 || s->seqlen > kMaxLen || s->channels > kMaxLen) return SSD_ERROR_UNSUPPORTED;
    *a = ConvArgs{};
    *n = ConvBytes{};
    ssd_status st = rows_of(s->x, s->batch, s->seqlen, s->channels, size_of(s->dtype), &a->xs, &n->x);
    if (st == SSD_OK) st = rows_of(s->dy, s->batch, s->seqlen, s->channels, size_of(s->y_dtype), &a->dys, &n->dy);
    if (st != SSD_OK) return st;
    if (a->xs.row >= kMaxRow || a->dys.row >= kMaxRow) return SSD_ERROR_UNSUPPORTED;  // 32-bit offsets in a group
    // launch geometry: fewer than 2^24 blocks, of 64 channels and 64 tokens at the least
    int64_t work;
    if (!product({(s->channels + 63) / 64, s->seqlen / 64 + 2}, &work) || work >= (int64_t)1 << 24)
        return SSD_ERROR_UNSUPPORTED;
    const size_t tok = (size_t)(s->batch * s->seqlen * s->channels);
    const size_t held = (size_t)(s->batch * (s->width - 1) * s->channels);
    a->batch = s->batch;
    a->seqlen = (int)s->seqlen;
    a->channels = (int)s->channels;
    a->width = s->width;
    a->silu = s->activation == SSD_ACT_SILU;
    a->in_bf16 = s->dtype == SSD_DTYPE_BF16;
    a->y_bf16 = s->y_dtype == SSD_DTYPE_BF16;
    a->dx_bf16 = s->dx_dtype == SSD_DTYPE_BF16;
    n->row = (size_t)s->channels * 4;
    n->filter = n->row * s->width;
    n->y = tok * size_of(s->y_dtype);
    n->dx = tok * size_of(s->dx_dtype);
    n->state = held * size_of(s->dtype);
    n->state32 = held * 4;
    return SSD_OK;
}

size_t conv_workspace(const ConvArgs &a) {
    const ConvBwdPlan p = conv_bwd_plan(a.batch, a.seqlen, a.channels);
    return align_up((size_t)p.parts * (a.width + 1) * a.channels * sizeof(float));
}

// ---------------------------------------------------------------------------
// Selective scan
// ---------------------------------------------------------------------------

struct ScanBytes {
    size_t x, dt, B, C, z, dy;  // strided inputs
    size_t row, A, y, tok32, bc32, state;
};

ssd_status check_scan(const ssd_selective_shape *s, ScanArgs *a, ScanBytes *n) {
    if (s == nullptr) return SSD_ERROR_INVALID_VALUE;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->dstate < 1 || s->ngroups < 1 || s->reserved != 0)
        return SSD_ERROR_INVALID_VALUE;
    if (s->channels % s->ngroups != 0) return SSD_ERROR_INVALID_VALUE;
    if (!dtype_ok(s->dtype) || (s->y_dtype != SSD_DTYPE_F32 && s->y_dtype != s->dtype)) return SSD_ERROR_INVALID_VALUE;
    if ((s->flags & ~(uint32_t)SSD_SCAN_DT_SOFTPLUS) != 0) return SSD_ERROR_INVALID_VALUE;
    if (s->dstate > 64) return SSD_ERROR_UNSUPPORTED;
    if (s->batch > 65535 || s->seqlen > kMaxLen || s->channels >= kMaxRow) return SSD_ERROR_UNSUPPORTED;
    *a = ScanArgs{};
    *n = ScanBytes{};
    const size_t i = size_of(s->dtype), o = size_of(s->y_dtype);
    const int64_t gn = s->ngroups * s->dstate;
    const struct {
        const ssd_stride &in;
        int64_t width;
        size_t esz;
        Strides *out;
        size_t *bytes;
    } rows[] = {{s->x, s->channels, i, &a->xs, &n->x},   {s->dt, s->channels, i, &a->dts, &n->dt},
                {s->B, gn, i, &a->Bs, &n->B},            {s->C, gn, i, &a->Cs, &n->C},
                {s->z, s->channels, i, &a->zs, &n->z},   {s->dy, s->channels, o, &a->dys, &n->dy}};
    for (const auto &r : rows) {
        const ssd_status st = rows_of(r.in, s->batch, s->seqlen, r.width, r.esz, r.out, r.bytes);
        if (st != SSD_OK) return st;
        if (r.out->row >= kMaxRow) return SSD_ERROR_UNSUPPORTED;  // a tile's rows within 32-bit byte offsets
    }
    const ScanPlan p = scan_plan(s->batch, s->seqlen, s->channels, s->dstate, s->ngroups, true);
    int64_t t;
    // launch geometry, and every buffer of the backward pass within int64
    if ((int64_t)p.nblk * p.nseg >= (int64_t)1 << 24) return SSD_ERROR_UNSUPPORTED;
    if (!product({s->batch, p.tiles + 1, s->channels, 64, 4}, &t) ||
        !product({p.nblk, s->batch, s->seqlen, 64, 4}, &t) || !product({s->batch, s->seqlen, gn, 4}, &t))
        return SSD_ERROR_UNSUPPORTED;
    const size_t tok = (size_t)(s->batch * s->seqlen * s->channels);
    a->batch = s->batch;
    a->seqlen = (int)s->seqlen;
    a->channels = (int)s->channels;
    a->dstate = (int)s->dstate;
    a->ngroups = (int)s->ngroups;
    a->in_bf16 = s->dtype == SSD_DTYPE_BF16;
    a->y_bf16 = s->y_dtype == SSD_DTYPE_BF16;
    a->softplus = (s->flags & SSD_SCAN_DT_SOFTPLUS) != 0;
    n->row = (size_t)s->channels * 4;
    n->A = n->row * s->dstate;
    n->y = tok * o;
    n->tok32 = tok * 4;
    n->bc32 = (size_t)(s->batch * s->seqlen * gn) * 4;
    n->state = (size_t)(s->batch * s->channels * s->dstate) * 4;
    return SSD_OK;
}

ScanPlan plan_of(const ScanArgs &a, bool backward) {
    return scan_plan(a.batch, a.seqlen, a.channels, a.dstate, a.ngroups, backward);
}

// Hands out the workspace's regions, each 256-byte aligned.
struct Carver {
    unsigned char *base;
    size_t off;
    float *take(size_t floats) {
        float *p = base != nullptr ? reinterpret_cast<float *>(base + off) : nullptr;
        off = align_up(off + floats * sizeof(float));
        return p;
    }
};

size_t scan_fwd_carve(ScanArgs *a, const ScanPlan &p, void *ws) {
    Carver w{static_cast<unsigned char *>(ws), 0};
    const size_t segs = (size_t)a->batch * p.nseg * a->channels;
    if (p.nseg > 1) {
        a->seg_state = w.take(segs * p.np);
        a->seg_steps = w.take(segs);
    }
    return w.off;
}

size_t scan_bwd_carve(ScanArgs *a, const ScanPlan &p, void *ws) {
    Carver w{static_cast<unsigned char *>(ws), 0};
    const size_t segs = (size_t)a->batch * p.nseg * a->channels;
    if (p.nseg > 1) {
        a->seg_state = w.take(segs * p.np);
        a->seg_adj = w.take(segs * p.np);
        a->seg_steps = w.take(segs);
        a->tile_steps = w.take((size_t)a->batch * p.tiles * a->channels);
    }
    a->tile_state = w.take((size_t)a->batch * p.tiles * a->channels * p.np);
    const size_t bc = (size_t)p.nblk * a->batch * a->seqlen * a->dstate;
    a->dbp = w.take(bc);
    a->dcp = w.take(bc);
    a->dap = w.take(segs * p.runs * p.np);
    a->ddp = w.take(segs * p.runs);
    a->dbiasp = w.take(segs * p.runs);
    return w.off;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_causal_conv_fwd(const ssd_conv_shape *shape, const void *x, const float *weight, const float *bias,
                               const void *initial_states, const int32_t *lengths, void *y, void *final_states,
                               void *stream) {
    ConvArgs a;
    ConvBytes n;
    ssd_status st = check_conv(shape, &a, &n);
    if (st != SSD_OK) return st;
    const size_t i = size_of(shape->dtype);
    st = check_buffers({{x, n.x, i, true},
                        {weight, n.filter, 4, n.y > 0},
                        {bias, n.row, 4, false},
                        {initial_states, n.state, i, false},
                        {lengths, (size_t)a.batch * 4, 4, false}},
                       {{y, n.y, size_of(shape->y_dtype), true}, {final_states, n.state, i, false, initial_states}});
    if (st != SSD_OK) return st;
    // without tokens only the final state is written, and that through no filter
    if (a.batch == 0 || (a.seqlen == 0 && final_states == nullptr)) return SSD_OK;
    if (weight == nullptr) return SSD_ERROR_INVALID_VALUE;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.init = initial_states;
    a.lengths = lengths;
    a.y = y;
    a.final_state = final_states;
    return launch_conv_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

size_t ssd_causal_conv_bwd_workspace_size(const ssd_conv_shape *shape) {
    ConvArgs a;
    ConvBytes n;
    return check_conv(shape, &a, &n) == SSD_OK ? conv_workspace(a) : 0;
}

ssd_status ssd_causal_conv_bwd(const ssd_conv_shape *shape, const void *x, const float *weight, const float *bias,
                               const void *initial_states, const int32_t *lengths, const void *dy,
                               const float *d_final_states, void *dx, float *dweight, float *dbias,
                               float *d_initial_states, void *workspace, size_t workspace_bytes, void *stream) {
    ConvArgs a;
    ConvBytes n;
    ssd_status st = check_conv(shape, &a, &n);
    if (st != SSD_OK) return st;
    const size_t need = conv_workspace(a), i = size_of(shape->dtype);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SSD_ERROR_WORKSPACE;
    st = check_buffers({{x, n.x, i, true},
                        {weight, n.filter, 4, true},
                        {bias, n.row, 4, false},
                        {initial_states, n.state, i, false},
                        {lengths, (size_t)a.batch * 4, 4, false},
                        {dy, n.dy, size_of(shape->y_dtype), true},
                        {d_final_states, n.state32, 4, false}},
                       {{dx, n.dx, size_of(shape->dx_dtype), true},
                        {dweight, n.filter, 4, true},
                        {dbias, n.row, 4, false},
                        {d_initial_states, n.state32, 4, false},
                        {workspace, need, kAlign, false}});
    if (st != SSD_OK) return st;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.init = initial_states;
    a.lengths = lengths;
    a.dy = dy;
    a.dfinal = d_final_states;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dinit = d_initial_states;
    a.partials = static_cast<float *>(workspace);
    const ConvBwdPlan plan = conv_bwd_plan(a.batch, a.seqlen, a.channels);
    return launch_conv_bwd(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

ssd_status ssd_causal_conv_step(const ssd_conv_shape *shape, const void *x, const float *weight, const float *bias,
                                void *state, void *y, void *stream) {
    ConvArgs a;
    ConvBytes n;
    ssd_status st = check_conv(shape, &a, &n);
    if (st != SSD_OK) return st;
    if (shape->seqlen != 1) return SSD_ERROR_INVALID_VALUE;
    const size_t i = size_of(shape->dtype);
    st = check_buffers({{x, n.x, i, true}, {weight, n.filter, 4, a.batch > 0}, {bias, n.row, 4, false}},
                       {{state, n.state, i, true}, {y, n.y, size_of(shape->y_dtype), true}});
    if (st != SSD_OK) return st;
    if (a.batch == 0) return SSD_OK;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.init = state;
    a.y = y;
    return launch_conv_step(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

size_t ssd_selective_scan_fwd_workspace_size(const ssd_selective_shape *shape) {
    ScanArgs a;
    ScanBytes n;
    return check_scan(shape, &a, &n) == SSD_OK ? scan_fwd_carve(&a, plan_of(a, false), nullptr) : 0;
}

size_t ssd_selective_scan_bwd_workspace_size(const ssd_selective_shape *shape) {
    ScanArgs a;
    ScanBytes n;
    return check_scan(shape, &a, &n) == SSD_OK ? scan_bwd_carve(&a, plan_of(a, true), nullptr) : 0;
}

ssd_status ssd_selective_scan_fwd(const ssd_selective_shape *shape, const void *x, const void *dt, const float *A,
                                  const void *B, const void *C, const float *D, const void *z, const float *dt_bias,
                                  const float *initial_states, const int32_t *lengths, void *y, float *final_states,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    ScanArgs a;
    ScanBytes n;
    ssd_status st = check_scan(shape, &a, &n);
    if (st != SSD_OK) return st;
    const ScanPlan plan = plan_of(a, false);
    const size_t need = scan_fwd_carve(&a, plan, workspace), i = size_of(shape->dtype);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SSD_ERROR_WORKSPACE;
    st = check_buffers({{x, n.x, i, true},
                        {dt, n.dt, i, true},
                        {A, n.A, 4, a.batch > 0},
                        {B, n.B, i, true},
                        {C, n.C, i, true},
                        {D, n.row, 4, false},
                        {z, n.z, i, false},
                        {dt_bias, n.row, 4, false},
                        {initial_states, n.state, 4, false},
                        {lengths, (size_t)a.batch * 4, 4, false}},
                       {{y, n.y, size_of(shape->y_dtype), true},
                        {final_states, n.state, 4, false, initial_states},
                        {workspace, need, kAlign, false}});
    if (st != SSD_OK) return st;
    if (a.batch == 0 || (a.seqlen == 0 && final_states == nullptr)) return SSD_OK;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.init = initial_states;
    a.lengths = lengths;
    a.y = y;
    a.final_state = final_states;
    return launch_scan_fwd(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

ssd_status ssd_selective_scan_bwd(const ssd_selective_shape *shape, const void *x, const void *dt, const float *A,
                                  const void *B, const void *C, const float *D, const void *z, const float *dt_bias,
                                  const float *initial_states, const int32_t *lengths, const void *dy,
                                  const float *d_final_states, float *dx, float *ddt, float *dA, float *dB, float *dC,
                                  float *dD, float *dz, float *ddt_bias, float *d_initial_states, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    ScanArgs a;
    ScanBytes n;
    ssd_status st = check_scan(shape, &a, &n);
    if (st != SSD_OK) return st;
    const ScanPlan plan = plan_of(a, true);
    const size_t need = scan_bwd_carve(&a, plan, workspace), i = size_of(shape->dtype);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr)) return SSD_ERROR_WORKSPACE;
    if (n.tok32 > 0 && (z == nullptr) != (dz == nullptr)) return SSD_ERROR_INVALID_VALUE;
    st = check_buffers({{x, n.x, i, true},
                        {dt, n.dt, i, true},
                        {A, n.A, 4, true},
                        {B, n.B, i, true},
                        {C, n.C, i, true},
                        {D, n.row, 4, false},
                        {z, n.z, i, false},
                        {dt_bias, n.row, 4, false},
                        {initial_states, n.state, 4, false},
                        {lengths, (size_t)a.batch * 4, 4, false},
                        {dy, n.dy, size_of(shape->y_dtype), true},
                        {d_final_states, n.state, 4, false}},
                       {{dx, n.tok32, 4, true},
                        {ddt, n.tok32, 4, true},
                        {dA, n.A, 4, true},
                        {dB, n.bc32, 4, true},
                        {dC, n.bc32, 4, true},
                        {dD, n.row, 4, false},
                        {dz, n.tok32, 4, false},
                        {ddt_bias, n.row, 4, false},
                        {d_initial_states, n.state, 4, false},
                        {workspace, need, kAlign, false}});
    if (st != SSD_OK) return st;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.init = initial_states;
    a.lengths = lengths;
    a.dy = dy;
    a.dfinal = d_final_states;
    a.dx = dx;
    a.ddt = ddt;
    a.dA = dA;
    a.dB = dB;
    a.dC = dC;
    a.dD = dD;
    a.dz = dz;
    a.ddt_bias = ddt_bias;
    a.dinit = d_initial_states;
    return launch_scan_bwd(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

ssd_status ssd_selective_scan_step(const ssd_selective_shape *shape, const void *x, const void *dt, const float *A,
                                   const void *B, const void *C, const float *D, const void *z, const float *dt_bias,
                                   float *state, void *y, void *stream) {
    ScanArgs a;
    ScanBytes n;
    ssd_status st = check_scan(shape, &a, &n);
    if (st != SSD_OK) return st;
    if (shape->seqlen != 1) return SSD_ERROR_INVALID_VALUE;
    const size_t i = size_of(shape->dtype);
    st = check_buffers({{x, n.x, i, true},
                        {dt, n.dt, i, true},
                        {A, n.A, 4, a.batch > 0},
                        {B, n.B, i, true},
                        {C, n.C, i, true},
                        {D, n.row, 4, false},
                        {z, n.z, i, false},
                        {dt_bias, n.row, 4, false}},
                       {{state, n.state, 4, true}, {y, n.y, size_of(shape->y_dtype), true}});
    if (st != SSD_OK) return st;
    if (a.batch == 0) return SSD_OK;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.init = state;
    a.y = y;
    return launch_scan_step(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERROR_LAUNCH;
}

}  // extern "C"
