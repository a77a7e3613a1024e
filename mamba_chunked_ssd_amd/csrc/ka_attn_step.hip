// ka_attn_step.hip -- sliding-window attention with sinks for one token of each
// sequence.
//
//   slot(t) <- k, v ;  y = sum_s exp(scale q . k_s - lse) v_s over the slots
//   0 .. min(t + 1, sinks + window) - 1 of the cache, all of which t sees
//
// Bound by memory: the cache is read once.  A block takes a run of slots of one
// sequence and head of keys for all heads that share it (32 columns of the
// matrix instructions; a product's time hides behind the loads).  Each wave
// walks 32 slots at a time on its own, the next 32 on their way into its part of
// LDS, with its own running maximum and sum; the waves' results are joined in
// LDS, and where few sequences leave compute units idle, so that a sequence's
// slots are split over blocks, those of the blocks by a second kernel.
//
// bf16 weights are rounded to 8 bits for their product, as over prompts.  In two
// operands, 16 bits together (and once more in one where a value is infinite, of
// which the second operand makes NaN), one sequence's 2052 slots took 11.4 us for
// 9.4, 128 walks over 1024 slots of heads of 128 16.2 for 13.9.
//
// Measured: 128 sequences, 40 heads of 64 over 8, 2052 slots 77.6 us, 5.8 TB/s (a
// large copy: 5.1); one sequence 10.5 us.
#include "ka_attn.h"

namespace ssd {
namespace {

template <typename T>
struct AttnStepIn {
    const T *q, *k, *v;
    T *kc, *vc;
    const int32_t *positions;
    T *y;
    float *part_y, *part_ml;
    HeadStrides qs, ks, vs;
    int64_t slots;
    int heads, kvheads, splits, run;
    int window, sinks;
    float c;
};

__device__ __forceinline__ int slot_of(int j, int window, int sinks) { return j < sinks ? j : sinks + (j - sinks) % window; }

template <typename T, int D>
struct StepLds {
    static constexpr int kWaves = attn_step_waves(D, sizeof(T)), kStage = WaveLds<T, D>::kStage;
    static constexpr int kResults = Join<T, D, kWaves>::kBytes, kCopies = kWaves * 2 * kStage;
    static constexpr int kBytes = kCopies > kResults ? kCopies : kResults;
};

template <typename T, int D>
__global__ __launch_bounds__((64 * StepLds<T, D>::kWaves), 1) void attn_step_kernel(const AttnStepIn<T> a) {
    constexpr int NS = D / 16, NW = StepLds<T, D>::kWaves;
    typedef Tile<T, D, 32> Tl;
    constexpr int kStage = StepLds<T, D>::kStage, kCopies = 2 * Copier<Tl, 1>::kEach;
    extern __shared__ __align__(16) unsigned char lds[];  // (waves, 2 stages, keys and values); then the waves' results

    const int group = a.heads / a.kvheads, hblocks = (group + 31) / 32;
    int n = blockIdx.x;
    const int split = n % a.splits;
    n /= a.splits;
    const int hb = n % hblocks;
    n /= hblocks;
    const int kvh = n % a.kvheads, b = n / a.kvheads;
    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int head0 = kvh * group + 32 * hb, nh = min(32, group - 32 * hb);
    const int t = min(a.positions[b], kAttnFar);
    if (t < 0) {
        if (split == 0)
            for (int e = threadIdx.x; e < nh * D; e += 64 * NW) narrow(a.y + ((int64_t)b * a.heads + head0) * D + e, 0.f);
        return;
    }
    const int count = (int)min((int64_t)t + 1, a.slots), fresh = slot_of(t, a.window, a.sinks);
    const int s0 = split * a.run, s1 = min(s0 + a.run, count);

    Frag<T> qf[NS];
    const T *qrow = a.q + (int64_t)b * a.qs.batch + (head0 + col) * a.qs.head;
#pragma unroll
    for (int s = 0; s < NS; ++s) load_frag(qf[s], qrow + 16 * s + 8 * h, col < nh);

    const int64_t cache = ((int64_t)b * a.kvheads + kvh) * a.slots * D;
    unsigned char *own = lds + wave * 2 * kStage;
    Copier<Tl, 1> copier;
    copier.init(Tl::kRow, 0, lane);
    const auto stage = [&](int at, int buf) {
        const uint32_t kl = lds_addr(own + buf * kStage);
        copier.copy(kl, a.kc + cache + (int64_t)at * D, min(s1 - at, 32));
        copier.copy(kl + Tl::kBytes, a.vc + cache + (int64_t)at * D, min(s1 - at, 32));
    };

    int at = s0 + 32 * wave, buf = 0;
    if (at < s1) stage(at, 0);
#pragma unroll
    for (int s = 0; s < NS; ++s) arrived(qf[s]);
    Running<T, D> run;
    run.init();
    for (; at < s1; at += 32 * NW, buf ^= 1) {
        if (at + 32 * NW < s1) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // what was read of the other stage has arrived
            stage(at + 32 * NW, buf ^ 1);
            lds_dma_wait_but<kCopies>();
        } else {
            lds_dma_wait();
        }
        unsigned char *kl = own + buf * kStage, *vl = kl + Tl::kBytes;
        if (fresh >= at && fresh < at + 32) {
            // the new token: its slot's old one is replaced here and in the cache (by the one wave that reads it)
            const T *kn = a.k + (int64_t)b * a.ks.batch + kvh * a.ks.head, *vn = a.v + (int64_t)b * a.vs.batch + kvh * a.vs.head;
            for (int p = lane; p < 2 * Tl::kPieces; p += 64) {
                const bool second = p >= Tl::kPieces;
                const int piece = second ? p - Tl::kPieces : p;
                const u32x4 x = *reinterpret_cast<const u32x4 *>((second ? vn : kn) + piece * Tl::kPer);
                *reinterpret_cast<u32x4 *>((second ? vl : kl) + Tl::at(fresh - at, piece)) = x;
                if (hb == 0) *reinterpret_cast<u32x4 *>((second ? a.vc : a.kc) + cache + (int64_t)fresh * D + piece * Tl::kPer) = x;
            }
            lds_dma_wait();
        }
        floatx16 s[1];
        scores<Tl>(kl, qf, lane, s);
        if (at + 32 > s1) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[0][r] = place(0, r) < s1 - at - 4 * h ? s[0][r] : -kInf;
        }
        run.template take<Tl, 1>(s, a.c, vl, lane);
    }
    Join<T, D, NW>::run(lds, run, wave, lane, nh, [&](int c, int d, float y, float m, float l) {
        const int64_t head = (int64_t)b * a.heads + head0 + c;
        if (a.splits == 1) {
            narrow(a.y + head * D + d, y / l);
        } else {
            a.part_y[(head * a.splits + split) * D + d] = y;
            if (d == 0) *reinterpret_cast<float2 *>(a.part_ml + (head * a.splits + split) * 2) = float2{m, l};
        }
    });
}

// Joins the blocks' results, a block of D threads to a head of a sequence.
template <typename T>
__global__ __launch_bounds__(128) void attn_join_kernel(const AttnStepIn<T> a, int D) {
    const int64_t head = blockIdx.x;
    const int d = threadIdx.x;
    if (a.positions[head / a.heads] < 0) return;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + head * a.splits;
    const float *py = a.part_y + head * a.splits * D + d;
    float most = -kInf, sum = 0.f, y = 0.f;
    for (int k = 0; k < a.splits; ++k) most = fmaxf(most, ml[k].x);
    const float from = most == -kInf ? 0.f : most;
#pragma unroll 8
    for (int k = 0; k < a.splits; ++k) {
        const float w = fast_exp2(ml[k].x - from);
        sum = fmaf(ml[k].y, w, sum);
        y = fmaf(py[(int64_t)k * D], w, y);
    }
    narrow(a.y + head * D + d, y / sum);
}

template <typename T, int D>
hipError_t attn_step_sized(const AttnStepIn<T> &in, int64_t batch, hipStream_t stream) {
    constexpr int kLds = StepLds<T, D>::kBytes;
    const hipError_t e = allow_lds<attn_step_kernel<T, D>>(kLds);
    if (e != hipSuccess) return e;
    const int64_t hblocks = (in.heads / in.kvheads + 31) / 32;
    attn_step_kernel<T, D><<<dim3((uint32_t)(batch * in.kvheads * hblocks * in.splits)), dim3(64 * StepLds<T, D>::kWaves), kLds, stream>>>(in);
    return hipGetLastError();
}

template <typename T>
hipError_t attn_step_typed(const AttnArgs &a, const AttnStepPlan &p, hipStream_t stream) {
    const AttnStepIn<T> in{static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.v),
                           static_cast<T *>(a.kc), static_cast<T *>(a.vc), a.positions, static_cast<T *>(a.y), a.part_y, a.part_ml,
                           a.qs, a.ks, a.vs, (int64_t)a.window + a.sinks, a.heads, a.kvheads, p.splits, p.run,
                           a.window, a.sinks, a.scale * kLog2e};
    const hipError_t e = a.headdim == 32   ? attn_step_sized<T, 32>(in, a.batch, stream)
                         : a.headdim == 64 ? attn_step_sized<T, 64>(in, a.batch, stream)
                                           : attn_step_sized<T, 128>(in, a.batch, stream);
    if (e != hipSuccess || p.splits == 1) return e;
    attn_join_kernel<T><<<dim3((uint32_t)(a.batch * a.heads)), dim3(a.headdim), 0, stream>>>(in, a.headdim);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_step(const AttnArgs &a, const AttnStepPlan &plan, hipStream_t stream) {
    return a.bf16 ? attn_step_typed<uint16_t>(a, plan, stream) : attn_step_typed<float>(a, plan, stream);
}

}  // namespace ssd
