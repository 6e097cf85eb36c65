// pa_compact.cu -- compaction of a sequence's kept tokens to consecutive
// positions, in place or into other blocks, keys re-rotated on the way.
//
// One CTA walks the rows of one (sequence, K or V, kv-head) in tiles of
// kTileRows: the tile's rows are gathered into shared memory, and only then
// written.  In place that order is enough: row i is written at position
// start + i <= keep[i] < keep[i + 1], so no later tile reads what an earlier
// one has written, and within a tile every row is read before any is written.
#include "pa_internal.h"
#include "pa_rotary.cuh"

namespace pa {
namespace {

constexpr int kTileRows = 64;
constexpr int kCompactThreads = 256;

struct CompactParams {
    uint16_t *pool;
    int64_t num_blocks;
    int64_t block_stride, kv_stride;   // elements
    int32_t block_size, d;
    const int32_t *src_tables, *dst_tables;
    int32_t max_blocks;
    const int32_t *seq_lens;
    const int32_t *keep;
    int32_t max_keep;
    const int32_t *keep_lens;
    const int32_t *starts;             // may be null
    const uint64_t *turns;             // null: keys move as they are
    int32_t rot_chunks, chunks;        // of a key row, V pairs or V components each
    unsigned int *err;
};

// grid (kv-head, 2, sequence)
template <int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
    using Vec = typename BfVec<V>::type;
    extern __shared__ __align__(16) uint16_t tile[];         // [kTileRows][d]
    __shared__ int64_t src_row[kTileRows], dst_row[kTileRows];   // element offsets; -1: the row stays
    __shared__ int32_t shift[kTileRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int h = blockIdx.x, kv = blockIdx.y, s = blockIdx.z;
    const int tid = threadIdx.x;
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    const int64_t len = __ldg(p.seq_lens + s), n = __ldg(p.keep_lens + s);
    const int64_t start = p.starts ? __ldg(p.starts + s) : 0;
    if (len < 0 || len > cap || n < 0 || n > p.max_keep || start < 0) {
        if (tid == 0 && h == 0 && kv == 0) raise_error(p.err, PA_DEVERR_SEQ_LEN);
        return;
    }
    const int32_t *keep = p.keep + (int64_t)s * p.max_keep;
    const int32_t *src_table = p.src_tables + (int64_t)s * p.max_blocks;
    const int32_t *dst_table = p.dst_tables + (int64_t)s * p.max_blocks;
    const int64_t base = kv * p.kv_stride + (int64_t)h * p.block_size * p.d;
    const bool turn = p.turns != nullptr && kv == 0;
    const int row_vecs = p.d / 8;
    for (int64_t i0 = 0; i0 < n; i0 += kTileRows) {
        const int rows = (int)(n - i0 < kTileRows ? n - i0 : kTileRows);
        if (tid < rows) {
            const int64_t i = i0 + tid, to = start + i;
            const int64_t from = __ldg(keep + i);
            const int64_t before = i > 0 ? __ldg(keep + i - 1) : -1;
            int64_t src = -1, dst = -1;
            if (from <= before || from < to || from >= len) {
                if (h == 0 && kv == 0) raise_error(p.err, PA_DEVERR_KEEP);
            } else {
                const int sb = __ldg(src_table + from / p.block_size), db = __ldg(dst_table + to / p.block_size);
                if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
                    if (h == 0 && kv == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
                } else if (from != to || sb != db) {
                    src = sb * p.block_stride + base + (from % p.block_size) * p.d;
                    dst = db * p.block_stride + base + (to % p.block_size) * p.d;
                }
            }
            src_row[tid] = src;
            dst_row[tid] = dst;
            shift[tid] = (int32_t)(to - from);
        }
        __syncthreads();
        for (int e = tid; e < rows * row_vecs; e += kCompactThreads) {
            const int r = e / row_vecs, c = e - r * row_vecs;
            if (src_row[r] >= 0)
                reinterpret_cast<uint4 *>(tile)[e] = *reinterpret_cast<const uint4 *>(p.pool + src_row[r] + c * 8);
        }
        __syncthreads();
        if (!turn) {
            for (int e = tid; e < rows * row_vecs; e += kCompactThreads) {
                const int r = e / row_vecs, c = e - r * row_vecs;
                if (src_row[r] >= 0)
                    *reinterpret_cast<uint4 *>(p.pool + dst_row[r] + c * 8) = reinterpret_cast<const uint4 *>(tile)[e];
            }
        } else {
            const int half = p.rot_chunks * V;
            for (int e = tid; e < rows * p.chunks; e += kCompactThreads) {
                const int r = e / p.chunks, c = e - r * p.chunks;
                if (src_row[r] < 0) continue;
                const uint16_t *from = tile + r * p.d;
                uint16_t *to = p.pool + dst_row[r];
                if (c >= p.rot_chunks) {
                    const int at = 2 * half + (c - p.rot_chunks) * V;
                    *reinterpret_cast<Vec *>(to + at) = *reinterpret_cast<const Vec *>(from + at);
                    continue;
                }
                const int at0 = INTERLEAVED ? 2 * c * V : c * V, at1 = INTERLEAVED ? at0 + V : half + at0;
                Vec lo = *reinterpret_cast<const Vec *>(from + at0), hi = *reinterpret_cast<const Vec *>(from + at1);
                float2 cs[V];
#pragma unroll
                for (int i = 0; i < V; ++i) cs[i] = rotary_cos_sin(shift[r], __ldg(p.turns + c * V + i), 1.f);
                rotate_pairs<V, INTERLEAVED>(lo, hi, cs);
                *reinterpret_cast<Vec *>(to + at0) = lo;
                *reinterpret_cast<Vec *>(to + at1) = hi;
            }
        }
        __syncthreads();
    }
}

template <int V, bool INTERLEAVED>
cudaError_t launch_compact_v(CompactParams &p, int32_t num_kv_heads, int32_t num_seqs, cudaStream_t stream) {
    const size_t smem = (size_t)kTileRows * p.d * 2;       // 32 KB at the widest head
    return launch_pdl(compact_kernel<V, INTERLEAVED>, dim3(num_kv_heads, 2, num_seqs), dim3(kCompactThreads), stream,
                      smem, p);
}

}  // namespace

cudaError_t launch_compact(const PoolView &pool, const int32_t *src_tables, const int32_t *dst_tables,
                           int32_t max_blocks, const int32_t *seq_lens, const int32_t *keep, int32_t max_keep,
                           const int32_t *keep_lens, const int32_t *starts, int32_t num_seqs,
                           const pa_rotary *rotary, cudaStream_t stream) {
    CompactParams p = {};
    p.pool = static_cast<uint16_t *>(const_cast<void *>(pool.base));
    p.num_blocks = pool.num_blocks;
    p.block_stride = pool.block_stride;
    p.kv_stride = pool.kv_stride;
    p.block_size = pool.block_size;
    p.d = pool.head_dim;
    p.src_tables = src_tables;
    p.dst_tables = dst_tables;
    p.max_blocks = max_blocks;
    p.seq_lens = seq_lens;
    p.keep = keep;
    p.max_keep = max_keep;
    p.keep_lens = keep_lens;
    p.starts = starts;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    if (!rotary) return launch_compact_v<8, false>(p, pool.num_kv_heads, num_seqs, stream);
    const int v = rotary_vec(rotary->rot_dim);
    const bool interleaved = (rotary->flags & PA_ROTARY_INTERLEAVED) != 0;
    p.turns = rotary->turns;
    p.rot_chunks = rotary->rot_dim / 2 / v;
    p.chunks = p.rot_chunks + (p.d - rotary->rot_dim) / v;
    const int hkv = pool.num_kv_heads;
    switch (v) {
        case 8:
            return interleaved ? launch_compact_v<8, true>(p, hkv, num_seqs, stream)
                               : launch_compact_v<8, false>(p, hkv, num_seqs, stream);
        case 4:
            return interleaved ? launch_compact_v<4, true>(p, hkv, num_seqs, stream)
                               : launch_compact_v<4, false>(p, hkv, num_seqs, stream);
        case 2:
            return interleaved ? launch_compact_v<2, true>(p, hkv, num_seqs, stream)
                               : launch_compact_v<2, false>(p, hkv, num_seqs, stream);
        default:
            return interleaved ? launch_compact_v<1, true>(p, hkv, num_seqs, stream)
                               : launch_compact_v<1, false>(p, hkv, num_seqs, stream);
    }
}

}  // namespace pa
