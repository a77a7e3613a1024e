// Host-only driver of the convolution's and the selective scan's entry points
// for the sanitizer builds (see stub_ops_launch.cpp): plans and workspaces over
// a range of sizes, with real host memory of exactly the reported size as
// workspace, and calls from many threads at once.  Prints "ok" and exits 0
// when every check holds.
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#include "../../include/ssd.h"
#include "../../mamba_chunked_ssd_amd/csrc/ssd_ops_internal.h"

extern std::atomic<long> g_ops_launches[6];

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
        base += (uintptr_t)64 << 30;
        return (T *)base;
    }
};

static ssd_conv_shape conv(int64_t b, int64_t L, int64_t c, int w) {
    ssd_conv_shape s{};
    s.batch = b; s.seqlen = L; s.channels = c; s.width = w; s.activation = SSD_ACT_SILU;
    s.dtype = SSD_DTYPE_BF16; s.y_dtype = SSD_DTYPE_F32; s.dx_dtype = SSD_DTYPE_BF16;
    return s;
}
static ssd_selective_shape scan(int64_t b, int64_t L, int64_t c, int64_t n, int64_t g) {
    ssd_selective_shape s{};
    s.batch = b; s.seqlen = L; s.channels = c; s.dstate = n; s.ngroups = g;
    s.dtype = SSD_DTYPE_F32; s.y_dtype = SSD_DTYPE_F32; s.flags = SSD_SCAN_DT_SOFTPLUS;
    return s;
}

static void conv_bwd(const ssd_conv_shape &s) {
    Fake f;
    const size_t n = ssd_causal_conv_bwd_workspace_size(&s);
    void *ws = n > 0 ? std::aligned_alloc(256, n) : nullptr;
    auto call = [&](size_t bytes) {
        Fake q;
        return ssd_causal_conv_bwd(&s, q.next(), q.next<float>(), q.next<float>(), q.next(), q.next<int32_t>(), q.next(),
                                   q.next<float>(), q.next(), q.next<float>(), q.next<float>(), q.next<float>(), ws,
                                   bytes, nullptr);
    };
    CHECK(call(n) == SSD_OK);
    if (n > 0) CHECK(call(n - 1) == SSD_ERROR_WORKSPACE);
    std::free(ws);
}

static void scan_calls(const ssd_selective_shape &s) {
    const size_t nf = ssd_selective_scan_fwd_workspace_size(&s), nb = ssd_selective_scan_bwd_workspace_size(&s);
    void *wf = nf > 0 ? std::aligned_alloc(256, nf) : nullptr, *wb = nb > 0 ? std::aligned_alloc(256, nb) : nullptr;
    Fake q;
    CHECK(ssd_selective_scan_fwd(&s, q.next(), q.next(), q.next<float>(), q.next(), q.next(), q.next<float>(), q.next(),
                                 q.next<float>(), q.next<float>(), q.next<int32_t>(), q.next(), q.next<float>(), wf, nf,
                                 nullptr) == SSD_OK);
    Fake r;
    CHECK(ssd_selective_scan_bwd(&s, r.next(), r.next(), r.next<float>(), r.next(), r.next(), r.next<float>(), r.next(),
                                 r.next<float>(), r.next<float>(), r.next<int32_t>(), r.next(), r.next<float>(),
                                 r.next<float>(), r.next<float>(), r.next<float>(), r.next<float>(), r.next<float>(),
                                 r.next<float>(), r.next<float>(), r.next<float>(), r.next<float>(), wb, nb,
                                 nullptr) == SSD_OK);
    std::free(wf);
    std::free(wb);
}

static void plans() {
    for (int64_t b : {1, 2, 7})
        for (int64_t L : {0, 1, 15, 16, 17, 63, 333, 2048, 70000})
            for (int64_t c : {1, 63, 64, 65, 771, 5120})
                for (int64_t n : {1, 8, 9, 16, 33, 64})
                    for (bool bwd : {false, true}) {
                        const ssd::ScanPlan p = ssd::scan_plan(b, L, c, n, 1, bwd);
                        CHECK(p.np >= n && p.np <= 64 && p.nseg >= 1);
                        CHECK(p.seglen % ssd::kScanSegment == 0 && (int64_t)p.nseg * p.seglen >= L);
                        CHECK(p.nseg == 1 || (int64_t)(p.nseg - 1) * p.seglen < L);
                        CHECK((int64_t)p.gblocks * (1024 / p.np) >= c);
                        CHECK(p.tiles * ssd::kScanTile >= L && p.tiles * ssd::kScanTile % ssd::kScanSegment == 0);
                    }
}

static void everything() {
    for (int64_t b : {0, 1, 3})
        for (int64_t L : {0, 1, 100, 1000})
            for (int64_t c : {1, 264}) {
                conv_bwd(conv(b, L, c, 4));
                scan_calls(scan(b, L, c, 16, 1));
                if (c == 264) scan_calls(scan(b, L, c, 23, 4));
            }
}

int main() {
    plans();
    everything();
    std::vector<std::thread> ts;
    for (int i = 0; i < 8; ++i) ts.emplace_back(everything);
    for (auto &t : ts) t.join();
    // shapes past the limits: no overflow on the way to the refusal
    const int64_t big = INT64_MAX;
    for (int64_t v : {big, big / 2, (int64_t)1 << 40}) {
        ssd_conv_shape c = conv(1, 1, 1, 4);
        ssd_selective_shape s = scan(1, 1, 1, 16, 1);
        for (int64_t *f : {&c.batch, &c.seqlen, &c.channels, &c.x.row, &c.dy.batch}) {
            const int64_t keep = *f;
            *f = v;
            if (f == &c.x.row || f == &c.dy.batch) c.batch = c.seqlen = 2;
            CHECK(ssd_causal_conv_bwd_workspace_size(&c) == 0);
            *f = keep;
            c.batch = c.seqlen = 1;
        }
        for (int64_t *f : {&s.batch, &s.seqlen, &s.channels, &s.dstate, &s.ngroups, &s.B.row}) {
            const int64_t keep = *f;
            *f = v;
            if (f == &s.B.row) s.seqlen = 2;
            CHECK(ssd_selective_scan_bwd_workspace_size(&s) == 0);
            *f = keep;
            s.seqlen = 1;
        }
    }
    CHECK(g_ops_launches[1] > 0 && g_ops_launches[3] > 0 && g_ops_launches[4] > 0);
    if (g_fail == 0) std::puts("ok");
    return g_fail == 0 ? 0 : 1;
}
