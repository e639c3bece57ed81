// Host-only stand-ins for the clipping's launchers that note what they are called with and succeed; the other
// operators' are host_stubs_ops.cpp's.
#include <vector>

#define launch_grad_sumsq stub_grad_sumsq
#define launch_grad_scale stub_grad_scale
#include "host_stubs_ops.cpp"
#undef launch_grad_sumsq
#undef launch_grad_scale

struct Launch {
    int64_t pass, first_count, tensors, chunks, slots, past, norm;
};
static std::vector<Launch> launches;

namespace tefp8 {
hipError_t launch_grad_sumsq(const ClipBatch& b, double*, int64_t have, bool past, hipStream_t)
{
    launches.push_back({0, b.n ? b.t[0].n : 0, b.n, b.chunks, have, past, 0});
    return hipSuccess;
}
hipError_t launch_grad_scale(const ClipBatch& b, const double*, int64_t slots, float, float* norm, bool past, hipStream_t)
{
    launches.push_back({1, b.n ? b.t[0].n : 0, b.n, b.chunks, slots, past, norm != nullptr});
    return hipSuccess;
}
}  // namespace tefp8

extern "C" int64_t recorded(Launch* out, int64_t most)
{
    const int64_t n = (int64_t)launches.size();
    for (int64_t i = 0; i < n && i < most; ++i) out[i] = launches[(size_t)i];
    launches.clear();
    return n;
}
