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

// Eight registers of a result (8 s .. 8 s + 7) as the next product's B operand
// (bf16: rounded to nearest even, by 2^-8 at most; the sums they enter are fp32).
// So results are 2.1e-3 from 64 bits forward and 2.4e-3 backward, where bf16
// results alone would be 1.6e-3; what is rounded off as a second operand gives
// 1.6e-3 and 1.7e-3 for a fifth to a quarter more time (2 x 2048 tokens, 40 heads of
// 64: 10 us forward, 27 backward; 16 384 tokens, heads of 128: 41 forward), and
// makes NaN of the infinite values that a row sees.
__device__ __forceinline__ void to_frag(const float (&p)[8], Frag<uint16_t> &f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
}
__device__ __forceinline__ void to_frag(const float (&p)[8], Frag<float> &f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = p[i];
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
// The loads of f have arrived.  Said before a loop that uses f beside copies
// (lds_dma_x4) in flight: the compiler, which does not count those, would wait
// in every turn for the loads, and so for the copies.
__device__ __forceinline__ void arrived(Frag<uint16_t> &f) { asm volatile("" : "+v"(f.v)); }
__device__ __forceinline__ void arrived(Frag<float> &f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(f.v[i]));
}
// Nothing is scheduled across.  Between groups of LDS reads and products: left
// alone, the compiler reuses one operand's registers and waits for each read
// right before its product.
__device__ __forceinline__ void group_end() { __builtin_amdgcn_sched_barrier(0); }

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

    // Filled through registers, row r from row(r), null: 0.
    template <int THREADS, typename F>
    __device__ static void gather(unsigned char *lds, F &&row) {
#pragma unroll 2
        for (int k = 0; k < (kBytes / 16 + THREADS - 1) / THREADS; ++k) {
            const int n = k * THREADS + (int)threadIdx.x % THREADS;
            if (kBytes / 16 % THREADS != 0 && n >= kBytes / 16) break;
            const int r = n / kPieces, piece = n % kPieces;
            const T *p = row(r);
            u32x4 v = {0, 0, 0, 0};
            if (p != nullptr) v = *reinterpret_cast<const u32x4 *>(p + piece * kPer);
            *reinterpret_cast<u32x4 *>(lds + at(r, piece)) = v;
        }
    }
};

// Copies into a Tile by WAVES waves, asynchronous and not through registers.
// The offsets of a lane's pieces are the same for every tile of a matrix.
template <typename Tl, int WAVES>
struct Copier {
    static constexpr int kAll = Tl::kBytes / 1024;  // pieces of a wave's instruction
    static constexpr int kEach = (kAll + WAVES - 1) / WAVES;
    int off[kEach];
    uint32_t stride, to;
    // stride: bytes between rows; wave: this one's number among the WAVES
    __device__ void init(int64_t bytes, int wave, int lane) {
        stride = (uint32_t)bytes;
        to = (uint32_t)wave * 1024;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int n = (k * WAVES + wave) * 64 + lane, r = n / Tl::kPieces;
            off[k] = r * (int)stride + ((n % Tl::kPieces) ^ Tl::turn(r)) * 16;
        }
    }
    // Rows 0 .. rows - 1 from base on; those behind them become 0.
    __device__ void copy(uint32_t lds, const void *base, int rows) const {
        const i32x4 desc = buffer_desc(base, rows > 0 ? (uint32_t)(rows - 1) * stride + Tl::kRow : 0u);
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (kAll % WAVES == 0 || to + k * WAVES * 1024 < Tl::kBytes) lds_dma_x4(desc, lds + to + k * WAVES * 1024, off[k]);
    }
};

// Waits for all copies but the newest N of this wave.
template <int N>
__device__ __forceinline__ void lds_dma_wait_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The mask of a block of keys whose first is token j0, for the lane's query t:
// register r of block kb is key j0 + 4 h + place(kb, r), which t sees if it is
// none of those behind `last` and, but for the sinks, after `before`.
__device__ constexpr int place(int kb, int r) { return 32 * kb + 8 * (r / 4) + r % 4; }
struct Mask {
    int last, before, sunk;
    __device__ Mask(int t, int j0, int h, int window, int sinks)
        : last(t - j0 - 4 * h), before(last - window), sunk(sinks - j0 - 4 * h) {}
    // without branches: comparisons, and the rest on scalar registers
    __device__ bool seen(int at) const { return (at <= last) & ((at > before) | (at < sunk)); }
};
// Masks of 32 KB keys for the queries w0 .. w0 + 31 of a wave: which comparisons they need.
struct Needs {
    bool last, before;
    __device__ Needs(int j0, int keys, int w0, int window, int sinks)
        : last(j0 + keys - 1 > w0), before(w0 + 31 - j0 >= window && j0 + keys > sinks) {}
};

// Which tiles of KT keys a run of queries from token t0 to t1 takes: those of
// the window from token `from`, on a grid that `first` lies on, and before them
// the sinks below `from`.
template <int KT>
struct Walk {
    int from, lo, sunk, nsink, ntiles;
    __device__ Walk(int t0, int t1, int first, int window, int sinks) {
        lo = max(t0 - window + 1, 0);
        from = lo >= first ? first + (lo - first) / KT * KT : first - (first - lo + KT - 1) / KT * KT;
        sunk = min(sinks, max(from, 0));
        nsink = (sunk + KT - 1) / KT;
        ntiles = nsink + (t1 - from) / KT + 1;
    }
    __device__ int start(int n) const { return n < nsink ? n * KT : from + (n - nsink) * KT; }
    // Does a query of this run see a token of tile n that the cache may hold?  (No older one is there.)
    __device__ bool held(int n, int j, int sinks, int end) const {
        return n < nsink ? j < sunk : j >= 0 && j < end && (j >= lo || j < sinks);
    }
};

constexpr float kInf = __builtin_inff();

// The running softmax of a lane's query (column) and its sum of values, o^T =
// V^T P^T: m the reference of the exponentials and l this lane's half of their
// sum, in units of log(2).
template <typename T, int D>
struct Running {
    static constexpr int DB = D / 32;
    float m = -kInf, l = 0.f;
    floatx16 o[DB];
    __device__ void init() {
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = zero16();
    }
    __device__ float ref() const { return m == -kInf ? 0.f : m; }
    // Scores of 32 KB keys (-infinity: not seen), whose values are the rows of the tile at v.
    template <typename Tl, int KB>
    __device__ void take(const floatx16 (&s)[KB], float c, const unsigned char *v, int lane) {
        float top = s[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
        top = fmaxf(top, other_half(top)) * c;
        // The reference follows the maximum only where it has fallen 2^8 behind: p stays below 2^8, which costs no
        // precision, and most tiles rescale nothing.
        if (__any(top > m + 8.f)) {
            const float next = fmaxf(m, top);
            const float by = next == -kInf ? 1.f : fast_exp2(m - next);
            l *= by;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] *= by;
            m = next;
        }
        const float from = ref();
        // 16 keys at a time: their values are read while the weights of those before them are formed
        constexpr int kSteps = 2 * KB;
        Frag<T> vf[2][DB];
        const auto read = [&](int step) {
#pragma unroll
            for (int db = 0; db < DB; ++db) Tl::across(v, 16 * step, 32 * db, lane, vf[step & 1][db]);
        };
        read(0);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            if (step + 1 < kSteps) read(step + 1);
            float p[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                p[r] = fast_exp2(fmaf(s[step / 2][8 * (step % 2) + r], c, -from));
            }
            // The running sum takes eight weights as one term (one by one, 65 536 like weights left it 2.6e-4 off; a whole
            // tile's as one takes 11 registers more, which cost heads of 64 4 %).
            l += ((((((p[0] + p[1]) + p[2]) + p[3]) + p[4]) + p[5]) + p[6]) + p[7];
            Frag<T> pf;
            to_frag(p, pf);
            group_end();
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] = mma(vf[step & 1][db], pf, o[db]);
        }
    }
};

// S^T = K Q^T of 32 KB keys, the rows of the tile at k.
template <typename Tl, typename T, int NS, int KB>
__device__ __forceinline__ void scores(const unsigned char *k, const Frag<T> (&q)[NS], int lane, floatx16 (&s)[KB]) {
    Frag<T> kf[KB > 1 ? 2 : 1][NS];
#pragma unroll
    for (int ks = 0; ks < NS; ++ks) Tl::down(k, 0, ks, lane, kf[0][ks]);
    group_end();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        if (kb + 1 < KB) {
#pragma unroll
            for (int ks = 0; ks < NS; ++ks) Tl::down(k, 32 * (kb + 1), ks, lane, kf[(kb + 1) & 1][ks]);
        }
        s[kb] = zero16();
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) s[kb] = mma(kf[kb & 1][ks], q[ks], s[kb]);
        group_end();
    }
}

// s = X A^T and g = Y B^T of 32 rows of the tiles at x and y, side by side: neither chain of products waits for itself,
// and where registers hold them all, both operands are read at once.
template <typename Tl, typename T, int NS>
__device__ __forceinline__ void both_scores(const unsigned char *x, const unsigned char *y, const Frag<T> (&a)[NS],
                                            const Frag<T> (&b)[NS], int lane, floatx16 &s, floatx16 &g) {
    constexpr int kAtOnce = NS * sizeof(T) <= 8 ? NS : NS / 2;
    s = zero16();
    g = zero16();
#pragma unroll
    for (int k0 = 0; k0 < NS; k0 += kAtOnce) {
        Frag<T> xf[kAtOnce], yf[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            Tl::down(x, 0, k0 + k, lane, xf[k]);
            Tl::down(y, 0, k0 + k, lane, yf[k]);
        }
        group_end();
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            s = mma(xf[k], a[k0 + k], s);
            g = mma(yf[k], b[k0 + k], g);
        }
    }
}

// Results of NW waves over the same 32 columns joined through LDS: (wave,
// column, m and l), then (wave, column, D values).  write(column, element,
// value, m, l) gets the joined sums, not yet divided, of the first `columns`.
template <typename T, int D, int NW>
struct Join {
    static constexpr int kPad = D + 4, kBytes = NW * 32 * (2 + kPad) * (int)sizeof(float);
    template <typename F>
    __device__ static void run(unsigned char *lds, const Running<T, D> &a, int wave, int lane, int columns, F &&write) {
        float *ml = reinterpret_cast<float *>(lds), *os = ml + NW * 32 * 2;
        const int col = lane & 31, h = lane >> 5;
        const float l = both_halves(a.l);
        __syncthreads();
        if (col < columns) {
            if (h == 0) {
                ml[(wave * 32 + col) * 2] = a.m;
                ml[(wave * 32 + col) * 2 + 1] = l;
            }
            float *row = os + (wave * 32 + col) * kPad;
#pragma unroll
            for (int db = 0; db < D / 32; ++db)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<floatx4 *>(row + 32 * db + 8 * g + 4 * h) =
                        floatx4{a.o[db][4 * g], a.o[db][4 * g + 1], a.o[db][4 * g + 2], a.o[db][4 * g + 3]};
        }
        __syncthreads();
        for (int e = threadIdx.x; e < columns * D; e += 64 * NW) {
            const int c = e / D, d = e % D;
            float most = -kInf, sum = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) most = fmaxf(most, ml[(k * 32 + c) * 2]);
            const float from = most == -kInf ? 0.f : most;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float w = fast_exp2(ml[(k * 32 + c) * 2] - from);
                sum = fmaf(ml[(k * 32 + c) * 2 + 1], w, sum);
                y = fmaf(os[(k * 32 + c) * kPad + d], w, y);
            }
            write(c, d, y, most, sum);
        }
    }
};

// A wave's two stages of 32 keys and values; four waves to a block where they
// fit its 128 KB (fp32 rows of 128 elements: two).
template <typename T, int D>
struct WaveLds {
    static constexpr int kStage = 2 * Tile<T, D, 32>::kBytes, kWaves = 8 * kStage <= 131072 ? 4 : 2;
    static constexpr int kResults = Join<T, D, kWaves>::kBytes, kCopies = kWaves * 2 * kStage;
    static constexpr int kBytes = kCopies > kResults ? kCopies : kResults;
};

// Blocks of 128 queries up to which the waves of a block share 32 of them instead:
// about what the compute units hold at once of those blocks (four for one of 128),
// and twice as many where the window covers the sequence, whose blocks of 128 are
// unlike one another.  One sequence, 8 heads over 2, 4 sinks, us of the forward
// pass by 128 and by 32, and what 32 change in the backward pass:
//   bf16 heads of 32, window 128: 192 blocks 10, 9, 0; 384 blocks 12, 14, +4
//     of 64:  128 blocks 11, 10, 0; 160 blocks 11, 16, +6; all tokens: 256 blocks 71, 66, -3; 320 blocks 95, 96, +9
//     of 128: 64 blocks 14, 13, -5; 96 blocks 14, 23, +5; all tokens: 128 blocks 54, 50, -9; 160 blocks 66, 82, +6
//   fp32 heads of 32, window 128: 192 blocks 20, 18, 0; 224 blocks 20, 21, +4
//     of 64:  128 blocks 29, 24, -8; 160 blocks 29, 35, +7; all tokens: 192 blocks 244, 190, -56; 256 blocks 326, 324, +19
//     of 128: 64 blocks 52, 28, -42; 96 blocks 52, 53, -15; all tokens: 128 blocks 321, 298, -21; 160 blocks 402, 533, +187
// (windows of 16 and 512 cross where 128 does, within a step of 32 blocks.)
// Tokens with a past all have a window behind them, so that its length plays no
// part.  512 tokens a sequence behind a window of 2048, the forward pass:
//   bf16 heads of 32: 256 blocks 61, 53; 320 blocks 70, 74
//     of 64:  128 blocks 85, 66; 160 blocks 88, 114     of 128: 64 blocks 133, 106; 96 blocks 139, 197
//   fp32 heads of 32: 128 blocks 144, 94; 160 blocks 148, 167
//     of 64:  96 blocks 256, 250 (256 behind 4096: 64 blocks 478, 256; 96 blocks 549, 604)
//     of 128: 64 blocks 490, 469; 96 blocks 555, 1018
template <typename T, int D>
inline bool few_queries(int64_t blocks, int seqlen, int window, bool past) {
    constexpr bool bf16 = sizeof(T) == 2;
    constexpr int64_t most = D == 128 ? 64 : D == 64 ? 128 : bf16 ? 320 : 192;
    constexpr int64_t most_past = D == 128 ? 64 : D == 64 ? (bf16 ? 128 : 64) : bf16 ? 256 : 128;
    return blocks <= (past ? most_past : window >= seqlen ? 2 * most : most);
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

// ---------------------------------------------------------------------------
// Results of columns that may not see all rows which a product takes: a row's
// value that is not finite makes 0 times it NaN where it is not seen.  A wave
// with a result that is not finite forms it again from memory, 32 rows at a
// time as before, but with such values taken out of the product, and beside it a
// product of their kinds with 1 where a column sees the row, else 0, which tells
// what of them each result has seen.  So a diverged step costs some times a sound
// one, however many of its values are not finite.
// ---------------------------------------------------------------------------

// Kinds, which sums over 32 rows keep apart: infinity 1, -infinity 2^7, NaN 2^14.
// A weight of kOddNan makes a NaN of each (0 times infinity).
constexpr float kOddMinus = 128.f, kOddNan = 16384.f;

// Element c of eight rows in the order of Tile::across (row(i) for the lane's rows i = 0 .. 3, 8 .. 11; null: 0).
template <typename T, typename F>
__device__ __forceinline__ void load_apart(Frag<T> &finite, Frag<T> &kind, int c, F &&row) {
    float x[8], k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const T *p = row((j & 3) + 8 * (j >> 2));
        const float v = p != nullptr ? widen(p[c]) : 0.f;
        const bool sound = v - v == 0.f;
        x[j] = sound ? v : 0.f;
        k[j] = sound ? 0.f : v != v ? kOddNan : v > 0.f ? 1.f : kOddMinus;
    }
    to_frag(x, finite);
    to_frag(k, kind);
}
// What a product of kinds says of each register: bit r infinity, bit 16 + r -infinity, both NaN.
__device__ __forceinline__ uint32_t odd_of(const floatx16 &n) {
    uint32_t bits = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const uint32_t sum = n[r] >= kOddNan ? (uint32_t)kOddMinus + 1u : (uint32_t)n[r];
        bits |= ((sum & 127u) != 0 ? 1u << r : 0u) | (sum >> 7 != 0 ? 1u << (16 + r) : 0u);
    }
    return bits;
}
__device__ __forceinline__ float with_odd(float v, uint32_t odd, int r) {
    if ((odd >> r & 1) != 0) v += kInf;
    if ((odd >> (16 + r) & 1) != 0) v -= kInf;
    return v;
}

}  // namespace ssd
