// Tables of rotary angles whose frequencies are scaled for long contexts: the
// frequencies on the host, amplitude * (cos, sin) of position * frequency in
// binary64 on the device.  A model's table is laid out once.
#include <cmath>

#include "paged.h"

namespace hd {
namespace {

constexpr int kFillThreads = 256;

__global__ void __launch_bounds__(kFillThreads)
    rope_fill_kernel(const __grid_constant__ RopeFrequencies f, double amplitude, int pairs, long long entries, float2 *table) {
    const long long i = (long long)blockIdx.x * kFillThreads + threadIdx.x;
    if (i >= entries) return;
    double sn, cs;
    sincos((double)(i / pairs) * f.f[i % pairs], &sn, &cs);
    table[i] = make_float2((float)(amplitude * cs), (float)(amplitude * sn));
}

bool positive(double x) { return x > 0.0 && std::isfinite(x); }

}  // namespace

cudaError_t launch_rope_fill(const RopeFrequencies &f, double amplitude, int pairs, int positions, float2 *table, cudaStream_t s) {
    const long long entries = (long long)pairs * positions, grid = (entries + kFillThreads - 1) / kFillThreads;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    rope_fill_kernel<<<(unsigned)grid, kFillThreads, 0, s>>>(f, amplitude, pairs, entries, table);
    return cudaGetLastError();
}

}  // namespace hd

extern "C" {

hd_status hd_rope_frequencies(const hd_rope_params *p, double *frequencies, double *amplitude) {
    if (!p || !frequencies || !amplitude) return HD_ERR_INVALID_ARG;
    const int rot = p->rotary_dim;
    if (rot < 8 || rot > hd::kHeadDim || rot % 8 || !(p->theta > 1.0) || !std::isfinite(p->theta) ||
        p->scaling < HD_ROPE_PLAIN || p->scaling > HD_ROPE_BANDS)
        return HD_ERR_INVALID_ARG;
    if (p->amplitude != 0.0 && !hd::positive(p->amplitude)) return HD_ERR_INVALID_ARG;
    const bool ramp = p->scaling == HD_ROPE_RAMP, ranged = ramp || p->scaling == HD_ROPE_BANDS;
    if (p->scaling != HD_ROPE_PLAIN && !hd::positive(p->factor)) return HD_ERR_INVALID_ARG;
    if (ranged && (!hd::positive(p->original_context) || !hd::positive(p->slow) || !hd::positive(p->fast) || p->slow >= p->fast))
        return HD_ERR_INVALID_ARG;
    if (ramp && p->amplitude == 0.0 && p->factor < 1.0) return HD_ERR_INVALID_ARG;
    constexpr double kTau = 6.283185307179586476925;
    double lo = 0.0, hi = 0.0;
    if (ramp) {
        const auto number = [&](double turns) { return rot * std::log(p->original_context / (turns * kTau)) / (2.0 * std::log(p->theta)); };
        lo = std::fmax(std::floor(number(p->fast)), 0.0);
        hi = std::fmin(std::ceil(number(p->slow)), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(p->theta, -2.0 * i / rot);
        double slowed = 0.0;   // the part of the pair that the factor slows
        if (p->scaling == HD_ROPE_LINEAR) slowed = 1.0;
        if (ramp) slowed = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
        if (p->scaling == HD_ROPE_BANDS)
            slowed = 1.0 - std::fmin(std::fmax((p->original_context * f / kTau - p->slow) / (p->fast - p->slow), 0.0), 1.0);
        frequencies[i] = slowed == 0.0 ? f : f * (1.0 - slowed) + f / p->factor * slowed;
    }
    *amplitude = p->amplitude != 0.0 ? p->amplitude : ramp ? 0.1 * std::log(p->factor) + 1.0 : 1.0;
    return HD_OK;
}

hd_status hd_rope_fill(const hd_rope_params *p, int32_t positions, float *table, void *stream) {
    hd::RopeFrequencies f{};
    double amplitude = 1.0;
    const hd_status st = hd_rope_frequencies(p, f.f, &amplitude);
    if (st != HD_OK) return st;
    if (positions < 1 || !table || (reinterpret_cast<uintptr_t>(table) & 15)) return HD_ERR_INVALID_ARG;
    return hd::launch_rope_fill(f, amplitude, p->rotary_dim / 2, positions, reinterpret_cast<float2 *>(table),
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? HD_OK
               : HD_ERR_CUDA;
}

}  // extern "C"
