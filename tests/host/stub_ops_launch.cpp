// Stub launchers of the convolution and the selective scan for the host-only
// sanitizer builds of ssd_ops.cpp (see stub_launch.cpp).  Each touches the
// first and the last element of every workspace region that its kernels write,
// so that a layout larger than the size the queries report is a fault there.
#include <hip/hip_runtime_api.h>

#include <atomic>

#include "../../mamba_chunked_ssd_amd/csrc/ssd_ops_internal.h"

std::atomic<long> g_ops_launches[6];

namespace ssd {
namespace {
void touch(float *p, size_t n) {
    if (n > 0) p[0] = p[n - 1] = 1.f;
}
}  // namespace

hipError_t launch_conv_fwd(const ConvArgs &, hipStream_t) {
    g_ops_launches[0]++;
    return hipSuccess;
}
hipError_t launch_conv_bwd(const ConvArgs &a, const ConvBwdPlan &p, hipStream_t) {
    g_ops_launches[1]++;
    touch(a.partials, (size_t)p.parts * (a.width + 1) * a.channels);
    return hipSuccess;
}
hipError_t launch_conv_step(const ConvArgs &, hipStream_t) {
    g_ops_launches[2]++;
    return hipSuccess;
}
hipError_t launch_scan_fwd(const ScanArgs &a, const ScanPlan &p, hipStream_t) {
    g_ops_launches[3]++;
    const size_t segs = (size_t)a.batch * p.nseg * a.channels;
    if (p.nseg > 1) {
        touch(a.seg_state, segs * p.np);
        touch(a.seg_steps, segs);
    }
    return hipSuccess;
}
hipError_t launch_scan_bwd(const ScanArgs &a, const ScanPlan &p, hipStream_t) {
    g_ops_launches[4]++;
    const size_t segs = (size_t)a.batch * p.nseg * a.channels;
    const size_t rows = (size_t)p.nblk * a.batch * a.seqlen * a.dstate;
    if (p.nseg > 1) {
        touch(a.seg_state, segs * p.np);
        touch(a.seg_adj, segs * p.np);
        touch(a.seg_steps, segs);
        touch(a.tile_steps, (size_t)a.batch * p.tiles * a.channels);
    }
    touch(a.tile_state, (size_t)a.batch * p.tiles * a.channels * p.np);
    touch(a.dbp, rows);
    touch(a.dcp, rows);
    touch(a.dap, segs * p.np);
    touch(a.ddp, segs);
    touch(a.dbiasp, segs);
    return hipSuccess;
}
hipError_t launch_scan_step(const ScanArgs &, hipStream_t) {
    g_ops_launches[5]++;
    return hipSuccess;
}

}  // namespace ssd
