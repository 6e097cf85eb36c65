// pa_rotary.cuh -- rotary angles on the device: exact reduction of the phase in
// integers, and the rotation of one chunk of pairs.
#pragma once

#include <cstdint>

#include "pa_device.cuh"

namespace pa {

// (cos, sin) of `offset` positions at `turns` (64-bit fraction of a turn per
// position), times m.  offset * turns mod 2^64 is the phase modulo one turn,
// exactly; its top 32 bits as a signed number are the phase in
// [-1/2, 1/2) turns to 2^-32, and the angle in [-pi, pi] carries the fp32
// rounding of that (2^-23).  There sin.approx and cos.approx are within 2^-20.5
// of the true values (PTX's bound), 2^-11 of a bf16 rounding step of the result's
// length, which the one rounding to bf16 hides; the library's accurate functions
// would cost some twenty instructions more a pair.
__device__ __forceinline__ float2 phase_cos_sin(uint32_t phase) {
    const float angle = (float)(int32_t)phase * 1.46291807926715968105e-9f;   // 2 pi / 2^32
    float s, c;
    asm("sin.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(angle));
    asm("cos.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(angle));
    return make_float2(c, s);
}
__device__ __forceinline__ float2 rotary_cos_sin(int64_t offset, uint64_t turns, float m) {
    const float2 cs = phase_cos_sin((uint32_t)(((uint64_t)offset * turns) >> 32));
    return make_float2(cs.x * m, cs.y * m);
}
// The same phase of a 32-bit offset in three instructions: its upper word is
// offset * upper + the upper word of offset * lower, less lower for a negative offset
// (whose unsigned form is 2^32 too large).
__device__ __forceinline__ float2 rotary_cos_sin(int32_t offset, uint64_t turns) {
    const uint32_t lower = (uint32_t)turns;
    return phase_cos_sin((uint32_t)offset * (uint32_t)(turns >> 32) + __umulhi((uint32_t)offset, lower) -
                         (offset < 0 ? lower : 0u));
}

// V bf16 values (V = 8, 4, 2 or 1) moved as one access.
template <int V> struct BfVec;
template <> struct BfVec<8> { using type = uint4; };
template <> struct BfVec<4> { using type = uint2; };
template <> struct BfVec<2> { using type = uint32_t; };
template <> struct BfVec<1> { using type = uint16_t; };

template <int V>
__device__ __forceinline__ void bf_unpack(const typename BfVec<V>::type &v, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = __uint_as_float((uint32_t)v << 16);
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <int V>
__device__ __forceinline__ typename BfVec<V>::type bf_pack(const float (&x)[V]) {
    typename BfVec<V>::type v;
    if constexpr (V == 1) {
        v = (uint16_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    } else {
        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
    return v;
}

// Rotates V pairs held in two vectors: lo[i], hi[i] are pair i in the half
// layout; in the interleaved layout lo holds pairs 0 .. V/2 - 1 and hi the rest,
// each as neighbours (one pair, lo and hi, when V = 1).  fp32, one rounding.
template <int V, bool INTERLEAVED>
__device__ __forceinline__ void rotate_pairs(typename BfVec<V>::type &lo, typename BfVec<V>::type &hi,
                                             const float2 (&cs)[V]) {
    float a[V], b[V], oa[V], ob[V];
    bf_unpack<V>(lo, a);
    bf_unpack<V>(hi, b);
    if constexpr (INTERLEAVED && V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 p = cs[i], q = cs[V / 2 + i];
            oa[2 * i] = a[2 * i] * p.x - a[2 * i + 1] * p.y;
            oa[2 * i + 1] = a[2 * i + 1] * p.x + a[2 * i] * p.y;
            ob[2 * i] = b[2 * i] * q.x - b[2 * i + 1] * q.y;
            ob[2 * i + 1] = b[2 * i + 1] * q.x + b[2 * i] * q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            oa[i] = a[i] * cs[i].x - b[i] * cs[i].y;
            ob[i] = b[i] * cs[i].x + a[i] * cs[i].y;
        }
    }
    lo = bf_pack<V>(oa);
    hi = bf_pack<V>(ob);
}

// The largest vector width that divides a head's pairs (and so, head_dim being
// a multiple of 8, the components that pass as well).
inline int rotary_vec(int rot_dim) {
    const int half = rot_dim / 2;
    return half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : half % 2 == 0 ? 2 : 1;
}

}  // namespace pa
