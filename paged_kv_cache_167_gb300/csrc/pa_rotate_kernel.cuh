// pa_rotate_kernel.cuh -- rotary positions of queries and keys, and the slot
// writer fed with the rotated keys: the kernel and its launch, for positions of one
// axis (pa_rotary.cu) and of several (pa_rotary_axes.cu).
//
// A head of d components is cut into chunks: V pairs (two V-wide vectors) for
// its rotated part, V components for the part that passes; V = 8 (16-byte
// accesses) wherever the number of pairs is a multiple of 8.  One CTA takes one
// token: thread (x, y) owns chunk x of heads y, y + Y, ..., so the V angles of a
// thread are computed once and kept in registers for all of its heads, and all
// of its loads are issued before the angles they wait for.
//
// With positions of several axes (time, height, width: pair i is turned by the
// position on axis(i)) a thread loads the token's position on every axis beside its
// components and picks one a pair by a two-bit code from the parameters.  It takes as
// many registers as leave an SM the CTAs it has with one axis (8,192 tokens of 64/8 heads of
// 128, three axes: 53.9 us, 58.3 with one CTA fewer), and where a token's heads are
// few a CTA takes several tokens, so that a thread still has several heads to one set of
// angles (5,001 tokens of 16 heads of 80: 5.9 us, 8.1 with a head a thread).
//
// What bounds it: every component is read and written once (two operations a
// byte), so DRAM, and the host's call where tokens are few.  GB300, of the measured
// copy bandwidth: 8,192 tokens of 64 query and 8 key heads of 128 components 52 us
// (0.96), 32,000 tokens of a fused projection 191 us (1.01); 64 tokens 2.3 us.
#pragma once

#include <type_traits>

#include "pa_internal.h"
#include "pa_rotary.cuh"

namespace pa {
namespace {

struct RotateParams {
    const uint16_t *q;           // [N] rows of num_q_heads heads
    const uint16_t *k;           // cache form only: [N] rows of num_kv_heads heads
    const uint16_t *v;
    int64_t q_stride, k_stride, v_stride;   // elements from token to token
    uint16_t *q_out;             // [N][num_q_heads][d]
    uint16_t *pool;
    int64_t num_blocks;
    int64_t block_stride, kv_stride;        // elements
    const int64_t *positions;
    const int64_t *slots;
    const uint64_t *turns;
    int32_t num_q_heads, num_kv_heads, block_size, d;
    int32_t rot_chunks;          // rot_dim / 2 / V
    int32_t chunks;              // rot_chunks + (d - rot_dim) / V
    float mscale;
    int32_t inverse;
    int64_t num_tokens;
    unsigned int *err;
};

struct OneAxis {};   // in AxesView's place where every pair is turned by the same position

constexpr int kRotateThreads = 128;

// The CTAs an SM that a thread of U heads leaves room for (0: no bound).
template <int V, int U, class Axes>
constexpr int kRotateCtas =
    V != 8 || std::is_same<Axes, OneAxis>::value ? 0 : U == 5 ? 5 : U == 4 ? 6 : U == 3 ? 8 : U == 2 ? 9 : 0;

// grid (tokens / Z, head groups of Y * U, chunk groups), block (X, Y, Z); Z is 1 with one axis.
template <int V, bool INTERLEAVED, int U, bool CACHE, class Axes>
__global__ void __launch_bounds__(kRotateThreads, kRotateCtas<V, U, Axes>)
    rotate_kernel(const RotateParams p, const __grid_constant__ Axes axes) {
    using Vec = typename BfVec<V>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    int64_t n = blockIdx.x;
    const int c = blockIdx.z * blockDim.x + threadIdx.x;
    if (c >= p.chunks) return;
    if constexpr (!std::is_same<Axes, OneAxis>::value) {
        n = n * blockDim.z + threadIdx.z;
        if (n >= p.num_tokens) return;
    }
    const bool turning = c < p.rot_chunks;
    const int half = p.rot_chunks * V;
    // where the chunk's first vector lies in a head, and its second one
    const int at0 = !turning ? 2 * half + (c - p.rot_chunks) * V : INTERLEAVED ? 2 * c * V : c * V;
    const int at1 = INTERLEAVED ? at0 + V : half + at0;

    int64_t slot = -1, row = 0;
    if (CACHE) {
        slot = __ldg(p.slots + n);
        if (slot >= p.num_blocks * p.block_size) {
            if (blockIdx.y == 0 && c == 0 && threadIdx.y == 0) raise_error(p.err, PA_DEVERR_SLOT);
            slot = -1;
        }
        if (slot >= 0) {
            const int64_t blk = (slot >> 32) == 0 ? (int64_t)((uint32_t)slot / (uint32_t)p.block_size)
                                                  : slot / p.block_size;
            row = blk * p.block_stride + (slot - blk * p.block_size) * p.d;
        }
    }
    const int heads = p.num_q_heads + (CACHE ? 2 * p.num_kv_heads : 0);
    const int h0 = blockIdx.y * (blockDim.y * U) + threadIdx.y;
    Vec lo[U], hi[U];
    uint16_t *dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * blockDim.y;
        dst[u] = nullptr;
        if (h >= heads) continue;
        const uint16_t *src;
        if (!CACHE || h < p.num_q_heads) {
            src = p.q + n * p.q_stride + h * p.d;
            dst[u] = p.q_out + (n * p.num_q_heads + h) * p.d;
        } else {
            if (slot < 0) continue;                       // padding: keys and values are skipped
            int g = h - p.num_q_heads;
            const bool value = g >= p.num_kv_heads;
            if (value) g -= p.num_kv_heads;
            src = (value ? p.v + n * p.v_stride : p.k + n * p.k_stride) + g * p.d;
            dst[u] = p.pool + row + (value ? p.kv_stride : 0) + (int64_t)g * p.block_size * p.d;
        }
        lo[u] = *reinterpret_cast<const Vec *>(src + at0);
        if (turning) hi[u] = *reinterpret_cast<const Vec *>(src + at1);
    }
    float2 cs[V];
    if constexpr (std::is_same<Axes, OneAxis>::value) {
        if (turning) {
            const int64_t pos = p.inverse ? -__ldg(p.positions + n) : __ldg(p.positions + n);
#pragma unroll
            for (int i = 0; i < V; ++i) cs[i] = rotary_cos_sin(pos, __ldg(p.turns + c * V + i), p.mscale);
        }
    } else if (turning) {
        int64_t pos[kMaxAxes];
#pragma unroll
        for (int x = 0; x < kMaxAxes; ++x) {
            pos[x] = x < axes.num_axes ? __ldg(p.positions + x * axes.stride + n) : 0;
            if (p.inverse) pos[x] = -pos[x];
        }
        // V divides 16: a chunk's codes lie in one word
        const uint32_t code = axes.code[c * V / 16] >> (2 * (c * V % 16));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t x = (code >> (2 * i)) & 3u;
            const int64_t low = x & 1u ? pos[1] : pos[0], high = x & 1u ? pos[3] : pos[2];
            cs[i] = rotary_cos_sin(x & 2u ? high : low, __ldg(p.turns + c * V + i), p.mscale);
        }
    }
    const int first_value = p.num_q_heads + p.num_kv_heads;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!dst[u]) continue;
        if (turning) {
            if (!CACHE || h0 + u * (int)blockDim.y < first_value) rotate_pairs<V, INTERLEAVED>(lo[u], hi[u], cs);
            *reinterpret_cast<Vec *>(dst[u] + at1) = hi[u];
        }
        *reinterpret_cast<Vec *>(dst[u] + at0) = lo[u];
    }
}

template <int V, bool INTERLEAVED, bool CACHE, class Axes>
cudaError_t launch_rotate_v(RotateParams &p, const Axes &axes, int64_t tokens, cudaStream_t stream) {
    const int heads = p.num_q_heads + (CACHE ? 2 * p.num_kv_heads : 0);
    const int x = p.chunks < kRotateThreads ? p.chunks : kRotateThreads;
    int y = kRotateThreads / x;
    if (y > heads) y = heads;
    const unsigned gz = (unsigned)((p.chunks + x - 1) / x);
    // Several heads a thread (up to six, the number that wastes least) once that
    // still fills every SM: 8,192 tokens 52 us, with one head a thread 61, with four
    // and a rest of one 60.  One otherwise, for a short call's latency: 64 tokens 2.3
    // us, with several 2.8.
    const int rows = (heads + y - 1) / y, groups = (rows + 5) / 6, most = (rows + groups - 1) / groups;
    const bool wide = tokens * groups * gz >= 4ll * device_sm_count();
    int u = wide ? (V == 8 ? most : most > 2 ? 4 : most) : 1;
    if constexpr (!std::is_same<Axes, OneAxis>::value) {
        // few heads: up to four a thread, and the CTA's other threads on further tokens
        // (64: a block's largest z)
        const int few = heads < 4 ? heads : 4, fy = (heads + few - 1) / few;
        const int z = kRotateThreads / (x * fy) < 64 ? kRotateThreads / (x * fy) : 64;
        if (V == 8 && u == 1 && few > 1 && z > 1 && (tokens + z - 1) / z * gz >= 4ll * device_sm_count()) {
            const dim3 fgrid((unsigned)((tokens + z - 1) / z), 1, gz), fblock(x, fy, z);
            switch (few) {
                case 2:
                    return launch_pdl(rotate_kernel<V, INTERLEAVED, 2, CACHE, Axes>, fgrid, fblock, stream, 0, p, axes);
                case 3:
                    return launch_pdl(rotate_kernel<V, INTERLEAVED, 3, CACHE, Axes>, fgrid, fblock, stream, 0, p, axes);
                default:
                    return launch_pdl(rotate_kernel<V, INTERLEAVED, 4, CACHE, Axes>, fgrid, fblock, stream, 0, p, axes);
            }
        }
    }
    const dim3 grid((unsigned)tokens, (unsigned)((heads + y * u - 1) / (y * u)), gz), block(x, y);
    if constexpr (V == 8) {
        switch (u) {
            case 2: return launch_pdl(rotate_kernel<V, INTERLEAVED, 2, CACHE, Axes>, grid, block, stream, 0, p, axes);
            case 3: return launch_pdl(rotate_kernel<V, INTERLEAVED, 3, CACHE, Axes>, grid, block, stream, 0, p, axes);
            case 4: return launch_pdl(rotate_kernel<V, INTERLEAVED, 4, CACHE, Axes>, grid, block, stream, 0, p, axes);
            case 5: return launch_pdl(rotate_kernel<V, INTERLEAVED, 5, CACHE, Axes>, grid, block, stream, 0, p, axes);
            case 6: return launch_pdl(rotate_kernel<V, INTERLEAVED, 6, CACHE, Axes>, grid, block, stream, 0, p, axes);
            default: return launch_pdl(rotate_kernel<V, INTERLEAVED, 1, CACHE, Axes>, grid, block, stream, 0, p, axes);
        }
    }
    return u == 4   ? launch_pdl(rotate_kernel<V, INTERLEAVED, 4, CACHE, Axes>, grid, block, stream, 0, p, axes)
           : u == 2 ? launch_pdl(rotate_kernel<V, INTERLEAVED, 2, CACHE, Axes>, grid, block, stream, 0, p, axes)
                    : launch_pdl(rotate_kernel<V, INTERLEAVED, 1, CACHE, Axes>, grid, block, stream, 0, p, axes);
}

template <bool CACHE, class Axes>
cudaError_t launch_rotate_any(RotateParams &p, const Axes &axes, int32_t rot_dim, bool interleaved, int64_t tokens,
                              cudaStream_t stream) {
    const int v = rotary_vec(rot_dim);
    p.num_tokens = tokens;
    p.rot_chunks = rot_dim / 2 / v;
    p.chunks = p.rot_chunks + (p.d - rot_dim) / v;
    switch (v) {
        case 8:
            return interleaved ? launch_rotate_v<8, true, CACHE>(p, axes, tokens, stream)
                               : launch_rotate_v<8, false, CACHE>(p, axes, tokens, stream);
        case 4:
            return interleaved ? launch_rotate_v<4, true, CACHE>(p, axes, tokens, stream)
                               : launch_rotate_v<4, false, CACHE>(p, axes, tokens, stream);
        case 2:
            return interleaved ? launch_rotate_v<2, true, CACHE>(p, axes, tokens, stream)
                               : launch_rotate_v<2, false, CACHE>(p, axes, tokens, stream);
        default:
            return interleaved ? launch_rotate_v<1, true, CACHE>(p, axes, tokens, stream)
                               : launch_rotate_v<1, false, CACHE>(p, axes, tokens, stream);
    }
}

inline RotateParams rotate_params(void *out, const void *x, int64_t x_stride, const int64_t *positions,
                                  int32_t num_heads, int32_t head_dim, const pa_rotary &rotary) {
    RotateParams p = {};
    p.q = static_cast<const uint16_t *>(x);
    p.q_stride = x_stride;
    p.q_out = static_cast<uint16_t *>(out);
    p.positions = positions;
    p.turns = rotary.turns;
    p.num_q_heads = num_heads;
    p.d = head_dim;
    p.mscale = rotary.mscale;
    p.inverse = (rotary.flags & PA_ROTARY_INVERSE) != 0;
    return p;
}

template <class Axes>
cudaError_t launch_rotate_cache(const PoolView &pool, void *q_out, const void *q, int64_t q_stride, const void *k,
                                int64_t k_stride, const void *v, int64_t v_stride, const int64_t *positions,
                                const int64_t *slots, int64_t num_tokens, int32_t num_q_heads,
                                const pa_rotary &rotary, const Axes &axes, cudaStream_t stream) {
    RotateParams p = rotate_params(q_out, q, q_stride, positions, num_q_heads, pool.head_dim, rotary);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.pool = static_cast<uint16_t *>(const_cast<void *>(pool.base));
    p.num_blocks = pool.num_blocks;
    p.block_stride = pool.block_stride;
    p.kv_stride = pool.kv_stride;
    p.slots = slots;
    p.num_kv_heads = pool.num_kv_heads;
    p.block_size = pool.block_size;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    return launch_rotate_any<true>(p, axes, rotary.rot_dim, (rotary.flags & PA_ROTARY_INTERLEAVED) != 0, num_tokens,
                                   stream);
}

}  // namespace
}  // namespace pa
