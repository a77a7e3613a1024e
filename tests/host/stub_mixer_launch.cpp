// Stub launchers of sliding-window attention and the RMS norm for the host-only
// sanitizer builds of ssd_mixer_ops.cpp (see stub_launch.cpp).  Each touches the
// first and the last element of every workspace region that its kernels write.
#include <hip/hip_runtime_api.h>

#include <atomic>

#include "../../mamba_chunked_ssd_amd/csrc/ssd_ops_internal.h"

std::atomic<long> g_mixer_launches[5];

namespace ssd {
namespace {
void touch(float *p, size_t n) {
    if (n > 0) p[0] = p[n - 1] = 1.f;
}
}  // namespace

hipError_t launch_attn_fwd(const AttnArgs &, hipStream_t) {
    g_mixer_launches[0]++;
    return hipSuccess;
}
hipError_t launch_attn_bwd(const AttnArgs &a, const AttnBwdPlan &p, hipStream_t) {
    g_mixer_launches[1]++;
    touch(a.stats, (size_t)a.batch * a.heads * a.seqlen * 2);
    touch(a.partials, (size_t)a.batch * a.kvheads * p.parts * 2 * p.rows * a.headdim);
    return hipSuccess;
}
hipError_t launch_attn_step(const AttnArgs &a, const AttnStepPlan &p, hipStream_t) {
    g_mixer_launches[2]++;
    if (p.splits > 1) {
        touch(a.part_y, (size_t)a.batch * a.heads * p.splits * a.headdim);
        touch(a.part_ml, (size_t)a.batch * a.heads * p.splits * 2);
    }
    return hipSuccess;
}
hipError_t launch_norm_fwd(const NormArgs &, hipStream_t) {
    g_mixer_launches[3]++;
    return hipSuccess;
}
hipError_t launch_norm_bwd(const NormArgs &a, const NormBwdPlan &p, hipStream_t) {
    g_mixer_launches[4]++;
    if (a.partials != nullptr) touch(a.partials, (size_t)p.parts * a.channels);
    return hipSuccess;
}

}  // namespace ssd
