// pa_compact.cu -- compaction of a sequence's kept tokens to consecutive
// positions, in place or into other blocks, keys re-rotated on the way.
//
// A unit is one sequence's K or V rows of one or several kv-heads (several share
// the rows' places and, for keys, their angles); it is taken in tiles of up to 32 KB.
// A tile is gathered into shared memory by asynchronous 16-byte copies, two tiles
// (in a cluster three) ahead of the one being written; the positions and table
// entries that say where its rows lie are fetched further ahead still, so that no
// step waits for that chain of loads.
//
// In place, row i is written at start + i <= keep[i] < keep[i + 1]: what a tile
// writes lies before everything that later tiles read, so it is enough that a
// tile is written only when it and all earlier ones have been read.  One CTA has
// that from a barrier per tile.  Where there are too few units for the SMs, a
// cluster of up to 16 CTAs takes a unit's tiles in turn: each CTA writes into
// the shared memory of all others how many of its tiles have landed, and writes
// its own tile of a step to the pool when all have landed theirs.  That is said
// one step ahead, so the way from SM to SM is not waited for (the cluster's own
// barrier cost 1.6 us a step).  The counts are relaxed stores, one word for each
// sender: what they order are reads that have ended (their bytes are in shared
// memory) before writes that have not begun; nobody reads what was written, so no
// store has to be waited for.  That is an argument about the hardware, outside the PTX
// memory model, which orders one CTA's reads before another's writes by release and
// acquire alone: a copy whose bytes have arrived, been waited for and counted cannot
// return what a store issued after that count writes.  Release stores would make it
// one of the model too, but wait for the CTA's own stores to the pool: 131,072 tokens of
// one sequence 124 us instead of 105, a window 56 instead of 49.  Out of place the tiles
// are free of one another and any number of CTAs share them.
//
// What bounds it: every moved row is read and written once, so DRAM where there are
// enough units.  GB300, of the measured copy bandwidth: 64 x 3,000 tokens, half of
// them kept, 89 us (0.86), the keys turned, each by its own distance, 113 us (0.68:
// 64 registers a thread for four CTAs an SM, and the angles); a window over 8 x 8,192
// tokens, all keys turned by one distance, 49 us (0.81); 131,072 tokens of one
// sequence in place 104 us (0.76: 256 CTAs, a step of all of them takes 1.6 us), out
// of place 91 us (0.87); 64 sequences with one to six accepted rows each 2.9 us, a
// chain of three dependent loads behind a launch.
#include <algorithm>

#include "pa_internal.h"
#include "pa_rotary.cuh"

namespace pa {
namespace {

constexpr int kLoads = 4;                                  // 16-byte copies a thread has in a tile
constexpr int kMaxHead = 256;                              // components
// Rows of a tile at most.
constexpr int max_rows(int threads) { return threads == 32 ? 32 : threads == 512 ? 256 : 96; }

// What is done to the components of a key: nothing, all of them turned, or some of
// them.  A kernel each, since registers decide how many CTAs an SM holds: 131,072
// tokens that do not turn went from 112 to 105 us, and a window from 52 to 50.
enum { kAsTheyAre = 0, kWhole = 1, kParts = 2 };

struct CompactParams {
    uint16_t *pool;
    int64_t num_blocks;
    int64_t block_stride, kv_stride;   // elements
    int32_t block_size, d;
    int32_t block_log;                 // of a block_size that is a power of two, else -1
    const int32_t *src_tables, *dst_tables;
    int32_t max_blocks;
    const int32_t *seq_lens;
    const int32_t *keep;
    int32_t max_keep;
    const int32_t *keep_lens;
    const int32_t *starts;             // may be null
    const uint64_t *turns;             // null: keys move as they are
    int32_t rot_chunks, chunks;        // of a key row, V pairs or V components each
    int32_t rows;                      // of a tile
    int32_t heads;                     // of a unit
    unsigned int *err;
};

__device__ __forceinline__ void copy_async(uint4 *to, const uint16_t *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Stores value at this address in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_there(int32_t *at, uint32_t rank, int32_t value) {
    asm volatile(
        "{\n\t.reg .b32 there;\n\t"
        "mapa.shared::cluster.u32 there, %0, %1;\n\t"
        "st.relaxed.cluster.shared::cluster.s32 [there], %2;\n\t}" ::"r"(smem_addr(at)),
        "r"(rank), "r"(value)
        : "memory");
}
__device__ __forceinline__ int32_t load_here(const int32_t *at) {
    int32_t v;
    asm volatile("ld.relaxed.cluster.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(smem_addr(at)) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What is being found out about one row, one step of the chain after another.
struct RowLookup {
    int32_t from = 0, before = 0;      // keep[i] and keep[i - 1]
    int32_t to = 0;                    // i, then start + i
    int32_t src_block = 0, dst_block = 0;
    int32_t own_block = -1;            // out of place: what src_tables has where dst_block is
    bool row = false;                  // false: no such row, or a bad one
};

// grid (CTAs of one unit, 2 x head groups, sequence); CLUSTER: they are a cluster
// and write in order, else each goes its own way (one CTA, or out of place).
// STAGES tiles are in shared memory or on their way there.
template <int V, bool INTERLEAVED, int TURNS, int THREADS, int STAGES, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, THREADS == 32 ? 8 : THREADS == 512 ? 1 : THREADS == 256 && CLUSTER ? 3 : 4)
    compact_kernel(const CompactParams p) {
    using Vec = typename BfVec<V>::type;
    constexpr int kRings = STAGES + 2;                     // tiles whose rows' places are known
    extern __shared__ __align__(16) uint4 ring[];          // [STAGES][rows][heads][d / 8], then the rows' places
    const int row_vecs = p.heads * (p.d / 8), tile_vecs = p.rows * row_vecs;
    int64_t *src_rows = reinterpret_cast<int64_t *>(ring + STAGES * tile_vecs);   // [kRings][rows]; -1: stays
    int64_t *dst_rows = src_rows + kRings * p.rows;
    uint64_t *turns = reinterpret_cast<uint64_t *>(dst_rows + kRings * p.rows);    // [V][rot_chunks]
    int32_t *shifts = reinterpret_cast<int32_t *>(turns + p.rot_chunks * V);
    __shared__ int32_t landed[16];                         // CLUSTER: tiles that have landed in each of its CTAs
    if (CLUSTER) {
        if (threadIdx.x < 16) landed[threadIdx.x] = 0;
        cluster_sync();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kv = blockIdx.y & 1, h = (blockIdx.y >> 1) * p.heads, s = blockIdx.z, tid = threadIdx.x;
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    const int32_t *keep = p.keep + (int64_t)s * p.max_keep;
    const bool looks = tid < p.rows;

    // The chain behind a row's place: keep -> table entries -> offsets, one call
    // (and one step of the loop below) each, so that no call uses what it has just
    // asked for.  Threads 0 .. rows - 1 take a row.  The first tiles' positions are
    // asked for together with the lengths (any of max_keep may be read), each kind of
    // load for all of them at once: 1.0 to 1.8 us less a call than one tile after the
    // other behind the lengths.
    uint32_t next_row = blockIdx.x * p.rows + tid;         // of the next look_keep (past 2^31 by a few tiles at most)
    auto look_keep = [&]() {
        RowLookup r;
        const uint32_t i = next_row;
        next_row += gridDim.x * p.rows;
        r.row = looks && i < (uint32_t)p.max_keep;
        if (!r.row) return r;
        r.before = i > 0 ? __ldg(keep + i - 1) : -1;
        r.from = __ldg(keep + i);
        r.to = (int32_t)i;
        return r;
    };
    RowLookup first[STAGES + 2];
#pragma unroll
    for (int k = 0; k < STAGES + 2; ++k) first[k] = look_keep();
    const int32_t len = __ldg(p.seq_lens + s), n = __ldg(p.keep_lens + s);
    const int32_t start = p.starts ? __ldg(p.starts + s) : 0;
    const bool reports = h == 0 && kv == 0;
    if (len < 0 || len > cap || n < 0 || n > p.max_keep || start < 0) {
        if (tid == 0 && reports && blockIdx.x == 0) raise_error(p.err, PA_DEVERR_SEQ_LEN);
        return;                                            // (a whole cluster does, before any count)
    }
    const int32_t *src_table = p.src_tables + (int64_t)s * p.max_blocks;
    const int32_t *dst_table = p.dst_tables + (int64_t)s * p.max_blocks;
    const int64_t base = kv * p.kv_stride + (int64_t)h * p.block_size * p.d;
    const bool turn = TURNS != kAsTheyAre && kv == 0;
    const int32_t tiles = (int32_t)(((uint32_t)n + p.rows - 1) / p.rows);
    const int32_t steps = (tiles - (CLUSTER ? 0 : (int)blockIdx.x) + (int)gridDim.x - 1) / (int)gridDim.x;
    auto block_of = [&](int32_t t) {
        return p.block_log >= 0 ? (uint32_t)t >> p.block_log : (uint32_t)t / (uint32_t)p.block_size;
    };
    auto look_blocks = [&](RowLookup r) {
        r.row = r.row && r.to < n;
        r.to = (int32_t)min((uint32_t)start + (uint32_t)r.to, (uint32_t)INT32_MAX);   // (beyond every length: refused)
        if (r.row && (r.from <= r.before || r.from < r.to || r.from >= len)) {
            if (reports) raise_error(p.err, PA_DEVERR_KEEP);
            r.row = false;
        }
        if (r.row) {
            r.src_block = __ldg(src_table + block_of(r.from));
            r.dst_block = __ldg(dst_table + block_of(r.to));
            if (src_table != dst_table) r.own_block = __ldg(src_table + block_of(r.to));
        }
        return r;
    };
    auto put_row = [&](int slot, const RowLookup &r) {
        if (!looks) return;
        int64_t src = -1, dst = -1;
        if (r.row) {
            if (r.src_block < 0 || r.src_block >= p.num_blocks || r.dst_block < 0 || r.dst_block >= p.num_blocks) {
                if (reports) raise_error(p.err, PA_DEVERR_BLOCK_ID);
            } else if (r.from != r.to || r.src_block != r.dst_block) {
                // out of place nothing orders the tiles: a block that the sequence
                // still reads is not written
                if (r.dst_block == r.own_block) {
                    if (reports) raise_error(p.err, PA_DEVERR_BLOCK_ID);
                    src_rows[slot * p.rows + tid] = -1;
                    return;
                }
                src = r.src_block * p.block_stride + base + (int64_t)(r.from - (int)block_of(r.from) * p.block_size) * p.d;
                dst = r.dst_block * p.block_stride + base + (int64_t)(r.to - (int)block_of(r.to) * p.block_size) * p.d;
            }
        }
        const int at = slot * p.rows + tid;
        src_rows[at] = src;
        dst_rows[at] = dst;
        shifts[at] = r.to - r.from;
    };

    // A tile's vectors are taken `at_once` whole rows at a time; this thread's are one
    // vector of rows my_row, my_row + at_once, ..., my_off elements from the row's place.
    const int head_stride = p.heads > 1 ? p.block_size * p.d : 0;   // (two heads share a unit only where it fits)
    const int at_once = THREADS / row_vecs;
    int my_row = tid / row_vecs, my_off = tid - my_row * row_vecs;
    my_off = my_off / (p.d / 8) * head_stride + my_off % (p.d / 8) * 8;
    if (my_row >= at_once) my_row = p.rows;                // (no whole row is left for it)
    auto begin_copies = [&](int32_t k, int stage, int slot) {
        if (k < steps) {
            const int64_t *src = src_rows + slot * p.rows;
            uint4 *tile = ring + stage * tile_vecs + tid;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int r = my_row + u * at_once;
                if (r < p.rows && src[r] >= 0) copy_async(tile + u * at_once * row_vecs, p.pool + src[r] + my_off);
            }
        }
        copy_commit();                                     // (an empty group where nothing is left)
    };
    auto next = [](int i, int count) { return i + 1 == count ? 0 : i + 1; };

    // This thread's chunk of the rows it turns, every `apart`-th row from `row0` on,
    // and its chunk of the components that pass, in a loop of their own: neighbouring
    // threads do the same, where a row's chunks side by side would have each warp go
    // both ways (33 x 3,000 tokens of 64 components, 32 of them turned: 26 us, now 22).
    const int half = TURNS == kWhole ? p.d / 2 : p.rot_chunks * V;
    const int pass_chunks = TURNS == kParts ? p.chunks - p.rot_chunks : 0;
    const int apart = turn ? THREADS / p.rot_chunks : 1;
    int row0 = turn ? tid / p.rot_chunks : 0;
    const int c = turn ? tid - row0 * p.rot_chunks : 0;
    if (row0 >= apart) row0 = p.rows;                      // (no whole row is left for it)
    float2 cs[V];
    int32_t turned = 0;                                    // the shift that cs belongs to
    const int at0 = INTERLEAVED ? 2 * c * V : c * V;
    const int at1 = INTERLEAVED ? at0 + V : half + at0;

#pragma unroll
    for (int k = 0; k <= STAGES; ++k) first[k] = look_blocks(first[k]);
    if (turn)
        for (int i = tid; i < half; i += THREADS) turns[i % V * p.rot_chunks + i / V] = __ldg(p.turns + i);
#pragma unroll
    for (int k = 0; k < STAGES; ++k) put_row(k, first[k]);
    RowLookup blocks = first[STAGES], kept = first[STAGES + 1];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) begin_copies(k, k, k);
    auto say_landed = [&](int32_t count) {
        if (CLUSTER && tid < (int)gridDim.x) store_there(&landed[blockIdx.x], tid, count);
    };
    // Whether the first `count` tiles have landed in all CTAs of the cluster; gives
    // up, as every wait of the library does, after kWaitLimitNs.
    auto all_landed = [&](int32_t count) {
        const int lane = tid & 31;
        uint64_t since = 0;
        for (int tries = 0;; ++tries) {
            const bool there = lane >= (int)gridDim.x || load_here(&landed[lane]) >= count;
            if (__all_sync(0xffffffffu, there)) return true;
            if ((tries & 255) == 255) {
                const uint64_t now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
                if (since == 0) since = now;
                if (now - since > kWaitLimitNs) {
                    if (lane == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
                    return false;
                }
            }
        }
    };
    constexpr int kPending = CLUSTER ? (STAGES > 2 ? STAGES - 3 : 0) : STAGES - 2;
    if (CLUSTER && steps > 0) {
        copy_wait<STAGES - 2>();                           // tile 0
        __syncthreads();
        say_landed(1);
    }
    int stage = 0, ahead = STAGES - 1;                     // tile k's place, and tile k + STAGES - 1's
    int slot = 0, slot_ahead = STAGES - 1, slot_put = STAGES;
    bool writing = true;
    for (int32_t k = 0; k < steps; ++k) {
        copy_wait<kPending>();                             // tile k has landed; in a cluster, tile k + 1
        __syncthreads();                                   // in all threads, and tile k - 1 is written
        say_landed(k + 2);
        begin_copies(k + STAGES - 1, ahead, slot_ahead);   // into the place of tile k - 1, written before the barrier
        put_row(slot_put, blocks);                         // of tile k + STAGES
        blocks = look_blocks(kept);
        kept = look_keep();
        // (a wait that gives up leaves the warp's remaining rows unwritten; the CTA
        // goes on counting, so that the others end)
        if (CLUSTER && writing) writing = all_landed(k + 1);
        const int64_t *src = src_rows + slot * p.rows, *dst = dst_rows + slot * p.rows;
        const int32_t *shift_of = shifts + slot * p.rows;
        const uint4 *tile = ring + stage * tile_vecs;
        stage = next(stage, STAGES);
        ahead = next(ahead, STAGES);
        slot = next(slot, kRings);
        slot_ahead = next(slot_ahead, kRings);
        slot_put = next(slot_put, kRings);
        if (!writing) continue;
        if (!turn) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int r = my_row + u * at_once;
                if (r < p.rows && src[r] >= 0)
                    *reinterpret_cast<uint4 *>(p.pool + dst[r] + my_off) = tile[tid + u * at_once * row_vecs];
            }
            continue;
        }
        const uint16_t *rows = reinterpret_cast<const uint16_t *>(tile);
        for (int r = row0; r < p.rows; r += apart) {
            if (src[r] < 0) continue;
            const uint16_t *from = rows + r * p.heads * p.d;
            uint16_t *to = p.pool + dst[r];
            const int32_t shift = shift_of[r];
            if (shift != turned && shift != 0) {           // a window slides by one distance: once for all its rows
#pragma unroll
                for (int i = 0; i < V; ++i) cs[i] = rotary_cos_sin(shift, turns[i * p.rot_chunks + c]);
                turned = shift;
            }
            for (int i = 0; i < p.heads; ++i, from += p.d, to += head_stride) {
                Vec lo = *reinterpret_cast<const Vec *>(from + at0), hi = *reinterpret_cast<const Vec *>(from + at1);
                // (shift 0: into another block at its old position)
                if (shift != 0) rotate_pairs<V, INTERLEAVED>(lo, hi, cs);
                *reinterpret_cast<Vec *>(to + at0) = lo;
                *reinterpret_cast<Vec *>(to + at1) = hi;
            }
        }
        for (int j = tid; j < p.rows * pass_chunks; j += THREADS) {
            const int r = (uint32_t)j / (uint32_t)pass_chunks, at = 2 * half + (j - r * pass_chunks) * V;
            if (src[r] < 0) continue;
            const uint16_t *from = rows + r * p.heads * p.d + at;
            uint16_t *to = p.pool + dst[r] + at;
            for (int i = 0; i < p.heads; ++i, from += p.d, to += head_stride)
                *reinterpret_cast<Vec *>(to) = *reinterpret_cast<const Vec *>(from);
        }
    }
    copy_wait<0>();
    if (CLUSTER) cluster_sync();                           // nobody leaves while others may still store here
}

// Dynamic shared memory of a launch: the tiles, their rows' places, the frequencies.
constexpr size_t compact_smem(int stages, size_t tile_vecs, size_t rows, size_t turns) {
    return stages * tile_vecs * sizeof(uint4) + (stages + 2) * rows * (2 * sizeof(int64_t) + sizeof(int32_t)) +
           turns * sizeof(uint64_t);
}

template <int V, bool INTERLEAVED, int TURNS, int THREADS, int STAGES, bool CLUSTER>
cudaError_t launch_compact_as(const CompactParams &p, int x, int32_t num_kv_heads, int32_t num_seqs,
                              cudaStream_t stream) {
    const auto kernel = compact_kernel<V, INTERLEAVED, TURNS, THREADS, STAGES, CLUSTER>;
    const size_t smem = compact_smem(STAGES, (size_t)p.rows * p.heads * (p.d / 8), p.rows, p.rot_chunks * V);
    // The limit belongs to the kernel, and other host threads may be about to launch
    // it: it is the most that any call asks for, so that no call lowers it for another.
    // (A tile has at most kLoads vectors a thread.)
    constexpr size_t kLimit = compact_smem(STAGES, kLoads * THREADS, max_rows(THREADS), kMaxHead / 2);
    static_assert(kLimit <= 227 * 1024, "what a CTA may have");
    if (smem > kLimit) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLimit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(x, 2 * (num_kv_heads / p.heads), num_seqs);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    if (CLUSTER && x > 8) {                                // 16 CTAs a cluster is an opt-in
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int V, bool INTERLEAVED, int TURNS>
cudaError_t launch_compact_v(CompactParams &p, int32_t num_kv_heads, int32_t num_seqs, cudaStream_t stream) {
    // threads of a CTA that is not in a cluster: two loops need more registers than
    // four CTAs of 256 have (330 x 3,000 tokens, half turned: 160 us, now 143)
    constexpr int kAlone = TURNS == kParts ? 192 : 256;
    const int row_vecs = p.d / 8;
    p.heads = 1;
    if (p.max_keep <= 32 && p.max_keep <= kLoads * (32 / row_vecs) && p.rot_chunks <= 32) {
        // a few rows a sequence (accepted drafts): one warp has them in one tile,
        // and all units are on the SMs at once (64 sequences: 2.9 us, 6.7 with 256
        // threads)
        p.rows = p.max_keep;
        return launch_compact_as<V, INTERLEAVED, TURNS, 32, 2, false>(p, 1, num_kv_heads, num_seqs, stream);
    }
    // Two heads share a unit, and the angles, where keys turn and units are many
    // (in place a cluster of 16 has to be enough to give every SM two CTAs): of
    // 64 x 3,000 tokens 127 us became 120, of a window 53 became 50.  (Not where a
    // head's slab of a block is so large that the way to the next needs 64 bits: that
    // would cost every kernel registers, and some of them spills.)
    const bool ordered = p.src_tables == p.dst_tables;
    const int sms = device_sm_count();
    const int64_t pairs = (int64_t)num_kv_heads * num_seqs;
    const bool near = (int64_t)p.block_size * p.d <= 1 << 30;
    if (TURNS != kAsTheyAre && near && num_kv_heads % 2 == 0 && (!ordered || pairs * 16 >= 2 * sms)) p.heads = 2;
    p.rows = std::min({kLoads * (kAlone / (row_vecs * p.heads)), max_rows(kAlone), p.max_keep});
    const int64_t units = 2ll * (num_kv_heads / p.heads) * num_seqs;
    const int64_t tiles = ((int64_t)p.max_keep + p.rows - 1) / p.rows;
    // Then CTAs share a unit, no more than there are tiles: out of place enough to
    // give every SM four (33 x 3,000 tokens of 128 components: 28.7 us, with six 30.9;
    // half turned of 64: 22.2, with two 35), in place the smallest cluster that gives
    // it two.
    if (!ordered) {
        const int x = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, 4 * sms / units));
        return launch_compact_as<V, INTERLEAVED, TURNS, kAlone, 3, false>(p, x, num_kv_heads, num_seqs, stream);
    }
    int x = 1;
    while (x < 16 && x < tiles && units * x < 2 * sms) x *= 2;
    if (x == 1) return launch_compact_as<V, INTERLEAVED, TURNS, kAlone, 3, false>(p, x, num_kv_heads, num_seqs, stream);
    // Four stages.  Of 32 KB for up to six clusters of 16, one CTA on an SM (65,536
    // tokens of one sequence and two heads, half of them kept: 26 us, with 16 KB 41;
    // eight such clusters do not always fit at once: 52 against 44).  Of 16 KB for more
    // clusters of 16 (131,072 tokens, eight heads: 104 us; 112 against 133 when tiles
    // of 12 KB were tried; a fifth stage: 183, since no longer all clusters are on the
    // SMs at once).  Of 12 KB otherwise, so that four CTAs fit an SM (a window over
    // 8 x 8,192 tokens: 49 us, with 16 KB 72).
    if (x == 16 && units <= 6) {
        p.rows = std::min({kLoads * (512 / (row_vecs * p.heads)), max_rows(512), p.max_keep});
        return launch_compact_as<V, INTERLEAVED, TURNS, 512, 4, true>(p, x, num_kv_heads, num_seqs, stream);
    }
    if (x == 16) {
        p.rows = std::min({kLoads * (256 / (row_vecs * p.heads)), max_rows(256), p.max_keep});
        return launch_compact_as<V, INTERLEAVED, TURNS, 256, 4, true>(p, x, num_kv_heads, num_seqs, stream);
    }
    p.rows = std::min({kLoads * (192 / (row_vecs * p.heads)), max_rows(192), p.max_keep});
    return launch_compact_as<V, INTERLEAVED, TURNS, 192, 4, true>(p, x, num_kv_heads, num_seqs, stream);
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
    p.block_log = -1;
    for (int i = 0; i < 31; ++i)
        if (pool.block_size == 1 << i) p.block_log = i;
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
    if (!rotary) return launch_compact_v<8, false, kAsTheyAre>(p, pool.num_kv_heads, num_seqs, stream);
    const int v = rotary_vec(rotary->rot_dim);
    const bool interleaved = (rotary->flags & PA_ROTARY_INTERLEAVED) != 0;
    p.turns = rotary->turns;
    p.rot_chunks = rotary->rot_dim / 2 / v;
    p.chunks = p.rot_chunks + (p.d - rotary->rot_dim) / v;
    const int hkv = pool.num_kv_heads;
    if (v == 8 && rotary->rot_dim == p.d)
        return interleaved ? launch_compact_v<8, true, kWhole>(p, hkv, num_seqs, stream)
                           : launch_compact_v<8, false, kWhole>(p, hkv, num_seqs, stream);
    switch (v) {
        case 8:
            return interleaved ? launch_compact_v<8, true, kParts>(p, hkv, num_seqs, stream)
                               : launch_compact_v<8, false, kParts>(p, hkv, num_seqs, stream);
        case 4:
            return interleaved ? launch_compact_v<4, true, kParts>(p, hkv, num_seqs, stream)
                               : launch_compact_v<4, false, kParts>(p, hkv, num_seqs, stream);
        case 2:
            return interleaved ? launch_compact_v<2, true, kParts>(p, hkv, num_seqs, stream)
                               : launch_compact_v<2, false, kParts>(p, hkv, num_seqs, stream);
        default:
            return interleaved ? launch_compact_v<1, true, kParts>(p, hkv, num_seqs, stream)
                               : launch_compact_v<1, false, kParts>(p, hkv, num_seqs, stream);
    }
}

}  // namespace pa
