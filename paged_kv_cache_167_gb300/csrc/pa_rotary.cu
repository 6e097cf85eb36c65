// pa_rotary.cu -- rotary positions of queries and keys, and the slot writer
// fed with the rotated keys.
//
// A head of d components is cut into chunks: V pairs (two V-wide vectors) for
// its rotated part, V components for the part that passes; V = 8 (16-byte
// accesses) wherever the number of pairs is a multiple of 8.  One CTA takes one
// token: thread (x, y) owns chunk x of heads y, y + Y, ..., so the V angles of a
// thread are computed once and kept in registers for all of its heads, and all
// of its loads are issued before the angles they wait for.
//
// What bounds it: every component is read and written once (two operations a
// byte), so DRAM, and the host's call where tokens are few.  GB300, of the measured
// copy bandwidth: 8,192 tokens of 64 query and 8 key heads of 128 components 52 us
// (0.96), 32,000 tokens of a fused projection 191 us (1.01); 64 tokens 2.3 us.
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
    unsigned int *err;
};

constexpr int kRotateThreads = 128;

// grid (tokens, head groups of Y * U, chunk groups), block (X, Y).
template <int V, bool INTERLEAVED, int U, bool CACHE>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(const RotateParams p) {
    using Vec = typename BfVec<V>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t n = blockIdx.x;
    const int c = blockIdx.z * blockDim.x + threadIdx.x;
    if (c >= p.chunks) return;
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
    if (turning) {
        const int64_t pos = p.inverse ? -__ldg(p.positions + n) : __ldg(p.positions + n);
#pragma unroll
        for (int i = 0; i < V; ++i) cs[i] = rotary_cos_sin(pos, __ldg(p.turns + c * V + i), p.mscale);
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

template <int V, bool INTERLEAVED, bool CACHE>
cudaError_t launch_rotate_v(RotateParams &p, int64_t tokens, cudaStream_t stream) {
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
    const int u = wide ? (V == 8 ? most : most > 2 ? 4 : most) : 1;
    const dim3 grid((unsigned)tokens, (unsigned)((heads + y * u - 1) / (y * u)), gz), block(x, y);
    if constexpr (V == 8) {
        switch (u) {
            case 2: return launch_pdl(rotate_kernel<V, INTERLEAVED, 2, CACHE>, grid, block, stream, 0, p);
            case 3: return launch_pdl(rotate_kernel<V, INTERLEAVED, 3, CACHE>, grid, block, stream, 0, p);
            case 4: return launch_pdl(rotate_kernel<V, INTERLEAVED, 4, CACHE>, grid, block, stream, 0, p);
            case 5: return launch_pdl(rotate_kernel<V, INTERLEAVED, 5, CACHE>, grid, block, stream, 0, p);
            case 6: return launch_pdl(rotate_kernel<V, INTERLEAVED, 6, CACHE>, grid, block, stream, 0, p);
            default: return launch_pdl(rotate_kernel<V, INTERLEAVED, 1, CACHE>, grid, block, stream, 0, p);
        }
    }
    return u == 4   ? launch_pdl(rotate_kernel<V, INTERLEAVED, 4, CACHE>, grid, block, stream, 0, p)
           : u == 2 ? launch_pdl(rotate_kernel<V, INTERLEAVED, 2, CACHE>, grid, block, stream, 0, p)
                    : launch_pdl(rotate_kernel<V, INTERLEAVED, 1, CACHE>, grid, block, stream, 0, p);
}

template <bool CACHE>
cudaError_t launch_rotate_any(RotateParams &p, int32_t rot_dim, bool interleaved, int64_t tokens,
                              cudaStream_t stream) {
    const int v = rotary_vec(rot_dim);
    p.rot_chunks = rot_dim / 2 / v;
    p.chunks = p.rot_chunks + (p.d - rot_dim) / v;
    switch (v) {
        case 8:
            return interleaved ? launch_rotate_v<8, true, CACHE>(p, tokens, stream)
                               : launch_rotate_v<8, false, CACHE>(p, tokens, stream);
        case 4:
            return interleaved ? launch_rotate_v<4, true, CACHE>(p, tokens, stream)
                               : launch_rotate_v<4, false, CACHE>(p, tokens, stream);
        case 2:
            return interleaved ? launch_rotate_v<2, true, CACHE>(p, tokens, stream)
                               : launch_rotate_v<2, false, CACHE>(p, tokens, stream);
        default:
            return interleaved ? launch_rotate_v<1, true, CACHE>(p, tokens, stream)
                               : launch_rotate_v<1, false, CACHE>(p, tokens, stream);
    }
}

}  // namespace

cudaError_t launch_rotate(void *out, const void *x, int64_t x_stride, const int64_t *positions, int64_t num_tokens,
                          int32_t num_heads, int32_t head_dim, const pa_rotary &rotary, cudaStream_t stream) {
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
    return launch_rotate_any<false>(p, rotary.rot_dim, (rotary.flags & PA_ROTARY_INTERLEAVED) != 0, num_tokens,
                                    stream);
}

cudaError_t launch_rotate_and_cache(const PoolView &pool, void *q_out, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                    const int64_t *positions, const int64_t *slots, int64_t num_tokens,
                                    int32_t num_q_heads, const pa_rotary &rotary, cudaStream_t stream) {
    RotateParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.pool = static_cast<uint16_t *>(const_cast<void *>(pool.base));
    p.num_blocks = pool.num_blocks;
    p.block_stride = pool.block_stride;
    p.kv_stride = pool.kv_stride;
    p.positions = positions;
    p.slots = slots;
    p.turns = rotary.turns;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = pool.num_kv_heads;
    p.block_size = pool.block_size;
    p.d = pool.head_dim;
    p.mscale = rotary.mscale;
    p.inverse = (rotary.flags & PA_ROTARY_INVERSE) != 0;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    return launch_rotate_any<true>(p, rotary.rot_dim, (rotary.flags & PA_ROTARY_INTERLEAVED) != 0, num_tokens,
                                   stream);
}

}  // namespace pa
