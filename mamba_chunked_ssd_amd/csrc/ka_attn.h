// ka_attn.h -- what the kernels of sliding-window attention share: fragments of
// the 32 x 32 matrix instructions, tiles of rows in LDS, and the mask.
//
// One instruction covers 32 x 32 outputs and 16 values of the contraction, in
// bf16 one v_mfma_f32_32x32x16_bf16, in fp32 eight v_mfma_f32_32x32x2_f32 fed
// from the same registers: lane l holds eight consecutive values k = 8 (l / 32)
// .. + 7 of row (A) or column (B) l % 32, and the fp32 instruction number j
// contracts the two k = j and 8 + j.  Results: lane l, register r holds row
// 8 (r / 4) + 4 (l / 32) + r % 4 of column l % 32.
//
// A contraction takes its terms in any order, as long as both operands do.  So
// results go back in as a B operand without moving between lanes: registers 8 s
// .. 8 s + 7 of a lane are the rows 16 s + 4 h + {0..3} and 16 s + 8 + 4 h +
// {0..3}, h = l / 32, and the A operand beside them is read from LDS in that
// order (Tile::across).
#pragma once

#include "ssd_launch.h"
#include "ssd_ops_device.h"
#include "ssd_ops_internal.h"

namespace ssd {

typedef float floatx16 __attribute__((ext_vector_type(16)));

template <typename T>
struct Frag;
template <>
struct Frag<uint16_t> {
    u32x4 v;
};
template <>
struct Frag<float> {
    float v[8];
};

__device__ __forceinline__ floatx16 mma(const Frag<uint16_t> &a, const Frag<uint16_t> &b, const floatx16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mma(const Frag<float> &a, const Frag<float> &b, floatx16 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ floatx16 zero16() {
    return floatx16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// Registers 8 s .. 8 s + 7 of a result as the next product's B operand (bf16:
// rounded to nearest even, relative 2^-9; the sums they enter are fp32).
__device__ __forceinline__ void to_frag(const float (&p)[16], int s, Frag<uint16_t> &f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = pack_bf16(p[8 * s + 2 * i], p[8 * s + 2 * i + 1]);
}
__device__ __forceinline__ void to_frag(const float (&p)[16], int s, Frag<float> &f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = p[8 * s + i];
}

// Eight consecutive elements from memory (16-byte aligned), or 0.
__device__ __forceinline__ void load_frag(Frag<uint16_t> &f, const uint16_t *p, bool on) {
    f.v = on ? *reinterpret_cast<const u32x4 *>(p) : u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ void load_frag(Frag<float> &f, const float *p, bool on) {
    const floatx4 a = on ? *reinterpret_cast<const floatx4 *>(p) : zero4();
    const floatx4 b = on ? *reinterpret_cast<const floatx4 *>(p + 4) : zero4();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.v[i] = a[i];
        f.v[4 + i] = b[i];
    }
}
__device__ __forceinline__ float dot_frag(const Frag<uint16_t> &a, const Frag<uint16_t> &b, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(bf16lo(a.v[i]), bf16lo(b.v[i]), s);
        s = fmaf(bf16hi(a.v[i]), bf16hi(b.v[i]), s);
    }
    return s;
}
__device__ __forceinline__ float dot_frag(const Frag<float> &a, const Frag<float> &b, float s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(a.v[i], b.v[i], s);
    return s;
}

// x of the other half of the wave's lanes.
__device__ __forceinline__ float other_half(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float((threadIdx.x & 32) != 0 ? r[0] : r[1]);
}
__device__ __forceinline__ float both_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float wave_sum(float v) {
    v = lane_total<16>(v);
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return both_halves(__uint_as_float(s[0]) + __uint_as_float(s[1]));
}

// ROWS rows of D elements in LDS, in pieces of 16 bytes.  A row's pieces are
// permuted by an exclusive or with bits of the row's number, so that the reads
// below meet each of the 64 banks once (per 256 bytes): 16 rows of one column
// of pieces (down), and four rows by four pieces (across).  The permutation is
// in the copies' source addresses; LDS itself is filled in order.
template <typename T, int D, int ROWS>
struct Tile {
    static constexpr int kRow = D * (int)sizeof(T);  // bytes
    static constexpr int kPieces = kRow / 16;
    static constexpr int kBytes = ROWS * kRow;
    static constexpr int kPer = 16 / (int)sizeof(T);  // elements of a piece

    __device__ static constexpr int turn(int r) {
        if constexpr (kPieces >= 16) return (r & 3) << 2 | (r >> 2 & 3);
        else if constexpr (kPieces == 8) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
        else return r >> 2 & 3;
    }
    __device__ static int at(int r, int piece) { return r * kRow + ((piece ^ turn(r)) << 4); }

    // A operand: row r0 + l % 32, elements 16 s + 8 (l / 32) .. + 7.
    __device__ static void down(const unsigned char *lds, int r0, int s, int lane, Frag<uint16_t> &f) {
        f.v = *reinterpret_cast<const u32x4 *>(lds + at(r0 + (lane & 31), 2 * s + (lane >> 5)));
    }
    __device__ static void down(const unsigned char *lds, int r0, int s, int lane, Frag<float> &f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const floatx4 v = *reinterpret_cast<const floatx4 *>(lds + at(r0 + (lane & 31), 4 * s + 2 * (lane >> 5) + i));
#pragma unroll
            for (int e = 0; e < 4; ++e) f.v[4 * i + e] = v[e];
        }
    }
    // A operand of the transpose: element c0 + l % 32 of the rows r0 + 4 h + {0..3} and r0 + 8 + 4 h + {0..3}.
    __device__ static void across(const unsigned char *lds, int r0, int c0, int lane, Frag<uint16_t> &f) {
        const int i = lane & 15, h = lane >> 5;
        const int piece = c0 / 8 + 2 * (lane >> 4 & 1) + (i >> 1 & 1), r = r0 + 4 * h + (i >> 2);
        const u32x2 lo = tr_read(lds + at(r, piece) + 8 * (i & 1));
        const u32x2 hi = tr_read(lds + at(r + 8, piece) + 8 * (i & 1));
        f.v = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
    __device__ static void across(const unsigned char *lds, int r0, int c0, int lane, Frag<float> &f) {
        const int c = c0 + (lane & 31), h = lane >> 5;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f.v[j] = *reinterpret_cast<const float *>(lds + at(r0 + 4 * h + (j & 3) + 8 * (j >> 2), c / 4) + 4 * (c & 3));
    }

    // Rows 0 .. rows - 1 of a matrix copied in by THREADS threads without passing through registers; those behind
    // them become 0.  stride: bytes between rows.
    template <int THREADS>
    __device__ static void copy(uint32_t lds, const unsigned char *base, int64_t stride, int rows) {
        const i32x4 desc = buffer_desc(base, rows > 0 ? (uint32_t)((rows - 1) * stride + kRow) : 0u);
        constexpr int kWavePieces = 64;
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
#pragma unroll
        for (int k = 0; k < (kBytes / 16 + THREADS - 1) / THREADS; ++k) {
            const int first = (k * (THREADS / 64) + wave) * kWavePieces;
            if (kBytes / 16 % THREADS != 0 && first >= kBytes / 16) break;  // (a tile of fewer pieces than threads)
            const int n = first + (threadIdx.x & 63), r = n / kPieces, piece = (n % kPieces) ^ turn(r);
            lds_dma_x4(desc, lds + first * 16, r * (int)stride + piece * 16);
        }
    }
    // By one wave, rows that follow one another without a gap.
    __device__ static void copy_wave(uint32_t lds, const unsigned char *base, int rows, int lane) {
        const i32x4 desc = buffer_desc(base, rows > 0 ? (uint32_t)(rows * kRow) : 0u);
#pragma unroll
        for (int k = 0; k < kBytes / 1024; ++k) {
            const int n = k * 64 + lane, r = n / kPieces, piece = (n % kPieces) ^ turn(r);
            lds_dma_x4(desc, lds + k * 1024, r * kRow + piece * 16);
        }
    }
    // The same through registers, row r from row(r), null: 0.
    template <int THREADS, typename F>
    __device__ static void gather(unsigned char *lds, F &&row) {
        static_assert(kBytes / 16 % THREADS == 0, "every thread takes as many pieces");
#pragma unroll 2
        for (int k = 0; k < kBytes / 16 / THREADS; ++k) {
            const int n = k * THREADS + threadIdx.x, r = n / kPieces, piece = n % kPieces;
            const T *p = row(r);
            u32x4 v = {0, 0, 0, 0};
            if (p != nullptr) v = *reinterpret_cast<const u32x4 *>(p + piece * kPer);
            *reinterpret_cast<u32x4 *>(lds + at(r, piece)) = v;
        }
    }
};

// Waits for all copies but the newest N of this wave.
template <int N>
__device__ __forceinline__ void lds_dma_wait_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Does token t see token j?
__device__ __forceinline__ bool sees(int t, int j, int window, int sinks) {
    return j <= t && (t - j < window || j < sinks);
}

// A result whose columns are rows of memory: lane l's column is row l % 32, its
// values the elements 32 b + 8 (r / 4) + 4 (l / 32) + r % 4 of it.  Lanes l and l
// + 32 exchange halves, so that each stores whole pieces of eight.
__device__ __forceinline__ void store_column(uint16_t *row, int b, int h, const float (&v)[16], bool on) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        u32x4 out;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = pack_bf16(v[8 * g + 2 * i], v[8 * g + 2 * i + 1]);
            const uint32_t hi = pack_bf16(v[8 * g + 4 + 2 * i], v[8 * g + 4 + 2 * i + 1]);
            const auto s = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
            out[i] = s[0];
            out[2 + i] = s[1];
        }
        if (on) *reinterpret_cast<u32x4 *>(row + 32 * b + 16 * g + 8 * h) = out;
    }
}
__device__ __forceinline__ void store_column(float *row, int b, int h, const float (&v)[16], bool on) {
    if (!on) return;
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *reinterpret_cast<floatx4 *>(row + 32 * b + 8 * g + 4 * h) = floatx4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
}

__device__ __forceinline__ float widen(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void narrow(uint16_t *p, float v) { *p = (uint16_t)(pack_bf16(v, 0.f) & 0xffffu); }
__device__ __forceinline__ void narrow(float *p, float v) { *p = v; }

}  // namespace ssd
