// ssd_ops_host.h -- host helpers shared by the layer operators' C-ABI
// translation units (ssd_ops.cpp, ssd_mixer_ops.cpp): sizes without overflow,
// strided rows, buffer checks, workspace regions.  Host code only.
#pragma once

#include <cstdint>
#include <initializer_list>
#include <limits>

#include "ssd_host.h"
#include "ssd_ops_internal.h"

namespace ssd {

constexpr int64_t kMaxLen = (int64_t)1 << 30;
constexpr int64_t kMaxRow = (int64_t)1 << 24;

inline bool product(std::initializer_list<int64_t> v, int64_t *out) {
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
inline ssd_status rows_of(const ssd_stride &in, int64_t batch, int64_t seqlen, int64_t width, size_t esz, Strides *out,
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
inline ssd_status check_buffers(std::initializer_list<Buffer> ins, std::initializer_list<Buffer> outs) {
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

inline bool dtype_ok(int32_t t) { return t == SSD_DTYPE_F32 || t == SSD_DTYPE_BF16; }
inline size_t size_of(int32_t t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }

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

}  // namespace ssd
