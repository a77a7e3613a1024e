// Host-only driver of sliding-window attention's and the RMS norm's entry
// points for the sanitizer builds (see stub_mixer_launch.cpp): plans and
// workspaces over a range of sizes, with real host memory of exactly the
// reported size as workspace, sizes near the limits, and calls from many threads
// at once.  Prints "ok" and exits 0 when every check holds.
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <thread>
#include <vector>

#include "../../include/ssd.h"
#include "../../mamba_chunked_ssd_amd/csrc/ssd_ops_internal.h"

extern std::atomic<long> g_mixer_launches[5];

static std::atomic<int> g_fail;
#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            std::fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
            ++g_fail;                                                         \
        }                                                                     \
    } while (0)

// Disjoint, never dereferenced device addresses.
struct Fake {
    uintptr_t base = (uintptr_t)1 << 44;
    template <typename T = void>
    T *next() {
        base += (uintptr_t)1 << 36;
        return (T *)base;
    }
};

static ssd_attn_shape attn(int64_t b, int64_t L, int64_t h, int64_t kv, int64_t d, int64_t w, int64_t n) {
    ssd_attn_shape s{};
    s.batch = b; s.seqlen = L; s.nheads = h; s.nkvheads = kv; s.headdim = d; s.window = w; s.sinks = n;
    s.scale = 0.125f; s.dtype = SSD_DTYPE_BF16;
    return s;
}
static ssd_norm_shape norm(int64_t b, int64_t L, int64_t c) {
    ssd_norm_shape s{};
    s.batch = b; s.seqlen = L; s.channels = c; s.eps = 1e-5f;
    s.dtype = SSD_DTYPE_BF16; s.res_dtype = SSD_DTYPE_F32; s.y_dtype = SSD_DTYPE_BF16;
    return s;
}

static void *memory(size_t n) { return n > 0 ? std::aligned_alloc(256, n) : nullptr; }

static void attn_bwd(const ssd_attn_shape &s) {
    const size_t n = ssd_window_attn_bwd_workspace_size(&s);
    void *ws = memory(n);
    auto call = [&](size_t bytes) {
        Fake q;
        return ssd_window_attn_bwd(&s, q.next(), q.next(), q.next(), q.next(), q.next<float>(), q.next(), nullptr, q.next(),
                                   q.next(), q.next(), ws, bytes, nullptr);
    };
    CHECK(call(n) == SSD_OK);
    if (n > 0) CHECK(call(n - 1) == SSD_ERROR_WORKSPACE);
    std::free(ws);
}
static void attn_step(ssd_attn_shape s) {
    s.seqlen = 1;
    const size_t n = ssd_window_attn_step_workspace_size(&s);
    void *ws = memory(n);
    auto call = [&](size_t bytes) {
        Fake q;
        return ssd_window_attn_step(&s, q.next(), q.next(), q.next(), q.next<int32_t>(), q.next(), q.next(), q.next(), ws, bytes, nullptr);
    };
    CHECK(call(n) == SSD_OK);
    if (n > 0) CHECK(call(n - 1) == SSD_ERROR_WORKSPACE);
    std::free(ws);
}
static void norm_bwd(const ssd_norm_shape &s) {
    const size_t n = ssd_rms_norm_bwd_workspace_size(&s);
    void *ws = memory(n);
    auto call = [&](size_t bytes) {
        Fake q;
        return ssd_rms_norm_bwd(&s, q.next(), q.next(), q.next<float>(), q.next(), nullptr, q.next(), q.next(), q.next<float>(), ws, bytes, nullptr);
    };
    CHECK(call(n) == SSD_OK);
    if (n > 0) CHECK(call(n - 1) == SSD_ERROR_WORKSPACE);
    std::free(ws);
}

// Plans at sizes that no buffer need exist for.
static void plans() {
    for (int64_t L : {1, 2, 100, 128, 129, 4096, 65536, 1 << 24, 1 << 30})
        for (int64_t w : {1, 64, 512, 4096, 1 << 20})
            for (int64_t n : {0, 1, 32, 33, 1000, 1 << 20}) {
                ssd::AttnArgs a{};
                a.batch = 1; a.seqlen = (int)L; a.window = (int)w; a.sinks = (int)n; a.heads = a.kvheads = 1;
                const ssd::AttnBwdPlan p = ssd::attn_bwd_plan(a);
                const int64_t far = L - w;
                if (n == 0 || far <= 0) {
                    CHECK(p.sink_tiles == 0 && p.rows == 0 && p.nchunks == 0);
                    continue;
                }
                // every sink that some query sees from farther than the window lies in a tile, every such query in a chunk
                CHECK(p.rows == (int64_t)p.sink_tiles * ssd::kSinkKeys && p.rows >= (n < far ? n : far));
                CHECK((int64_t)p.chunk * p.nchunks >= far && (int64_t)p.chunk * (p.nchunks - 1) < far);
                CHECK(p.nchunks <= 64 && p.chunk % 128 == 0 && p.parts == 1 + p.nchunks);
            }
    for (int64_t b : {1, 3, 128, 65535})
        for (int64_t slots : {1, 31, 128, 129, 2052, 65536, 1 << 29}) {
            ssd::AttnArgs a{};
            a.batch = b; a.window = (int)slots; a.heads = a.kvheads = 8; a.headdim = 128; a.bf16 = b == 1;
            const ssd::AttnStepPlan p = ssd::attn_step_plan(a);
            CHECK(p.splits >= 1 && p.run % (32 * ssd::attn_step_waves(128, a.bf16 ? 2 : 4)) == 0 && (int64_t)p.splits * p.run >= slots && (int64_t)(p.splits - 1) * p.run < slots);
            CHECK(p.splits == 1 || b * 8 * p.splits <= 1024 + b * 8);
        }
    for (int64_t rows : {0, 1, 5, 4096, 1 << 20, (1 << 30) - 1})
        for (int c : {1, 4096, 4097, 100000}) {
            ssd::NormArgs a{};
            a.batch = 2; a.seqlen = (int)rows; a.channels = c;
            const int64_t beside = c <= ssd::kNormWaveRow ? 4 : 1, parts = ssd::norm_bwd_plan(a).parts;
            CHECK(parts >= 1 && parts < (1 << 24) && parts * beside * 256 >= 2 * rows);  // 256 rows to a sum in 32 bits
        }
}

static void limits() {
    const int64_t huge[] = {-1, (int64_t)1 << 31, (int64_t)1 << 40, (int64_t)1 << 62, std::numeric_limits<int64_t>::max()};
    for (int64_t v : huge) {
        ssd_attn_shape s = attn(2, 2, 2, 2, 64, 8, 1);
        for (int64_t *f : {&s.batch, &s.seqlen, &s.nheads, &s.nkvheads, &s.headdim, &s.q.row, &s.dy.row}) {
            const int64_t keep = *f;
            *f = v;
            CHECK(ssd_window_attn_bwd_workspace_size(&s) == 0);
            *f = keep;
        }
        s.seqlen = 1;
        for (int64_t *f : {&s.batch, &s.nheads, &s.nkvheads, &s.window, &s.sinks}) {
            const int64_t keep = *f;
            *f = v;
            CHECK(ssd_window_attn_step_workspace_size(&s) == 0);
            *f = keep;
        }
        ssd_norm_shape m = norm(2, 2, 16);
        for (int64_t *f : {&m.batch, &m.seqlen, &m.channels, &m.dy.row, &m.residual.row}) {
            const int64_t keep = *f;
            *f = v;
            CHECK(ssd_rms_norm_bwd_workspace_size(&m) == 0);
            *f = keep;
        }
    }
    // an attention without a cache may have any window
    ssd_attn_shape s = attn(1, 300, 2, 2, 64, std::numeric_limits<int64_t>::max(), std::numeric_limits<int64_t>::max());
    CHECK(ssd_window_attn_bwd_workspace_size(&s) > 0);
}

int main() {
    plans();
    limits();
    std::vector<std::thread> threads;
    for (int k = 0; k < 8; ++k)
        threads.emplace_back([k] {
            for (int64_t L : {0, 1, 33, 128, 1000})
                for (int64_t w : {1, 60, 5000})
                    for (int64_t n : {0, 3, 200}) {
                        attn_bwd(attn(1 + k % 3, L, 6, 2, 64, w, n));
                        attn_step(attn(1 + k, 1, 6, 2, 128, w, n));
                    }
            for (int64_t c : {1, 100, 4096, 5000, 20000}) {
                norm_bwd(norm(2, 17 + k, c));
                norm_bwd(norm(1, 0, c));
            }
        });
    for (auto &t : threads) t.join();
    CHECK(g_mixer_launches[1] > 0 && g_mixer_launches[2] > 0 && g_mixer_launches[4] > 0);
    if (g_fail == 0) std::puts("ok");
    return g_fail == 0 ? 0 : 1;
}
