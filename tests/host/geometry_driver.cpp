// Host-only checks of the launch geometry of the convolution and the selective
// scan at sizes that no buffer need exist for.  Prints "ok" and exits 0 when
// every check holds.
#include <cstdio>

#include "../../include/ssd.h"
#include "../../mamba_chunked_ssd_amd/csrc/ssd_ops_internal.h"

static int g_fail;
#define CHECK(c)                                                              \
    do {                                                                      \
        if (!(c)) {                                                           \
            std::fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
            ++g_fail;                                                         \
        }                                                                     \
    } while (0)

// The backward pass's last sums: a launch of fewer than 2^32 threads over
// every output, whatever the entry points accept.
static void sums(int64_t b, int64_t L, int64_t c, int64_t n, int64_t g) {
    ssd_selective_shape s{};
    s.batch = b; s.seqlen = L; s.channels = c; s.dstate = n; s.ngroups = g;
    s.dtype = SSD_DTYPE_BF16; s.y_dtype = SSD_DTYPE_BF16;
    CHECK(ssd_selective_scan_bwd_workspace_size(&s) > 0);  // accepted
    const ssd::ScanPlan p = ssd::scan_plan(b, L, c, n, g, true);
    const ssd::ScanSums q = ssd::scan_sums(b, L, c, n, g, p.gblocks);
    CHECK(q.blocks >= 1 && (int64_t)q.blocks <= q.groups && (int64_t)q.blocks * 256 < (int64_t)1 << 32);
    CHECK(q.rates == c * n && q.rows == (p.gblocks == 1 ? 0 : b * L * g * n));
    const int64_t outputs = q.rates + 2 * c + 2 * q.rows;
    CHECK(q.groups * ssd::kSumOutputs >= outputs && (q.groups - 1) * ssd::kSumOutputs < outputs);
}

// Segments that the carry walks one after the other: the square root of the
// length at most.
static void segments(int64_t b, int64_t L, int64_t c, int64_t n) {
    for (bool bwd : {false, true}) {
        const ssd::ScanPlan p = ssd::scan_plan(b, L, c, n, 1, bwd);
        CHECK((int64_t)(p.nseg - 1) * (p.nseg - 1) < L && (int64_t)p.nseg * p.seglen >= L);
    }
}

int main() {
    for (int64_t L : {1, 15, 16, 300, 2048, 8191, 65536, 1 << 20})
        for (int64_t c : {1, 64, 771, 5120}) segments(1, L, c, 16), segments(2, L, c, 64);
    sums(1, 1, 1, 1, 1);
    sums(2, 2048, 5120, 16, 1);
    sums(16, 4096, 1088, 64, 64);      // 2^29 outputs and some
    sums(1, (int64_t)1 << 24, 128, 16, 1);
    sums(64, 65536, 17, 64, 1);
    sums(256, 65536, 128, 16, 1);
    sums(65535, 65536, 17, 64, 1);     // 5e11
    if (g_fail == 0) std::puts("ok");
    return g_fail == 0 ? 0 : 1;
}
