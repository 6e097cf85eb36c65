// pa_rotary.cpp -- host side of the rotary positions: angular frequencies and
// their scalings, as 64-bit fractions of a turn.
//
// A turn count w / (2 pi) is taken modulo 1 and held with 64 fractional bits (the
// rest, below 2^-64, is dropped).  In units of 2^-53 of the value the quotient is off
// by two (its own rounding and that of 2 pi), and w by some 14 + 2 ln(base) more: the
// power with its rounded exponent, the base's own change and the division by the
// factor.  So position t is off by t * w * (16 + 2 ln(base)) 2^-53 radians: 2^-28 at
// t = 2^20 for the fastest pair of base 10,000.  The by-parts mixes add the error of
// their share g, which is that of L w times high / (high - low), and matters up to s
// times as much where w / s remains.
#include <cmath>
#include <cstdint>

#include "pa.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

uint64_t turns_of(double w) {
    const double t = w / kTwoPi;
    const double frac = t - std::floor(t);            // in [0, 1]; 1 only by rounding of a tiny negative
    if (!(frac < 1.0)) return 0;
    return (uint64_t)std::ldexp(frac, 64);            // frac <= 1 - 2^-53: fits
}

}  // namespace

extern "C" {

pa_status pa_rotary_turns(const double *angular, int64_t n, uint64_t *turns_out) {
    if (n < 0 || (n > 0 && (!angular || !turns_out))) return PA_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i)
        if (!std::isfinite(angular[i])) return PA_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i) turns_out[i] = turns_of(angular[i]);
    return PA_OK;
}

pa_status pa_rotary_sections(const int32_t *sections, int32_t num_axes, int32_t order, int32_t num_pairs,
                             uint8_t *axis_out) {
    if (!sections || !axis_out || num_axes < 1 || num_axes > 4 || num_pairs < 1) return PA_ERR_INVALID_ARG;
    if (order != PA_AXES_BLOCKS && order != PA_AXES_CYCLED) return PA_ERR_INVALID_ARG;
    int64_t sum = 0;
    for (int32_t a = 0; a < num_axes; ++a) {
        if (sections[a] < 0) return PA_ERR_INVALID_ARG;
        sum += sections[a];
    }
    if (sum != num_pairs) return PA_ERR_INVALID_ARG;
    int32_t axis = 0, left = sections[0];
    for (int32_t i = 0; i < num_pairs; ++i) {
        if (order == PA_AXES_CYCLED) {
            axis = i % num_axes;
            if (i >= (int64_t)num_axes * sections[axis]) axis = 0;
        } else {
            while (left == 0) left = sections[++axis];
            --left;
        }
        axis_out[i] = (uint8_t)axis;
    }
    return PA_OK;
}

pa_status pa_rotary_frequencies(const pa_rotary_params *params, uint64_t *turns_out) {
    if (!params || !turns_out) return PA_ERR_INVALID_ARG;
    const pa_rotary_params p = *params;
    if (p.rot_dim < 2 || p.rot_dim % 2 != 0) return PA_ERR_INVALID_ARG;
    if (p.scaling < PA_ROTARY_PLAIN || p.scaling > PA_ROTARY_PARTS_INDEX) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(p.base) || !(p.base > 1.0)) return PA_ERR_INVALID_ARG;
    if (p.scaling != PA_ROTARY_PLAIN && (!std::isfinite(p.factor) || !(p.factor >= 1.0))) return PA_ERR_INVALID_ARG;
    const bool parts = p.scaling == PA_ROTARY_PARTS || p.scaling == PA_ROTARY_PARTS_INDEX;
    if (parts) {
        if (!std::isfinite(p.original_len) || !(p.original_len > 0.0)) return PA_ERR_INVALID_ARG;
        if (!std::isfinite(p.low) || !std::isfinite(p.high) || !(p.low > 0.0) || !(p.high > p.low))
            return PA_ERR_INVALID_ARG;
    }
    double base = p.base;
    if (p.scaling == PA_ROTARY_BASE && p.rot_dim > 2)
        base *= std::pow(p.factor, (double)p.rot_dim / (p.rot_dim - 2));
    if (!std::isfinite(base)) return PA_ERR_INVALID_ARG;
    double first = 0.0, last = 0.0;
    if (p.scaling == PA_ROTARY_PARTS_INDEX) {
        // w_i = 2 pi turns / L  <=>  i = rot_dim ln(L / (2 pi turns)) / (2 ln base)
        auto at = [&](double turns) {
            return p.rot_dim * std::log(p.original_len / (kTwoPi * turns)) / (2.0 * std::log(base));
        };
        first = std::fmax(std::floor(at(p.high)), 0.0);
        last = std::fmin(std::ceil(at(p.low)), (double)(p.rot_dim - 1));
    }
    for (int32_t i = 0; i < p.rot_dim / 2; ++i) {
        double w = std::pow(base, -2.0 * i / p.rot_dim);
        if (p.scaling == PA_ROTARY_LINEAR) {
            w /= p.factor;
        } else if (parts) {
            double g;                                  // share of the unscaled frequency
            if (p.scaling == PA_ROTARY_PARTS)
                g = (p.original_len * w / kTwoPi - p.low) / (p.high - p.low);
            else
                g = 1.0 - (i - first) / std::fmax(last - first, 1e-3);
            g = std::fmin(std::fmax(g, 0.0), 1.0);
            w = (1.0 - g) * w / p.factor + g * w;
        }
        turns_out[i] = turns_of(w);
    }
    return PA_OK;
}

}  // extern "C"
