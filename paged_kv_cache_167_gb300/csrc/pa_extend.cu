// pa_extend.cu -- a step's block tables, positions and slots, built on the GPU
// from the requests' lengths and a list of free blocks.
//
// Sequence s has c_s cached tokens and n_s new ones.  It needs
//     need_s = ceil((c_s + n_s) / b) - ceil(c_s / b)
// more blocks, which are entries cursor + sum_{r < s} need_r ... of the free list,
// and its tokens stand at sum_{r < s} n_r ... of the step's flat arrays: two
// exclusive sums over the sequences, then one token a thread.  A new block's first
// slot always belongs to a new token, so the thread of that token writes the table
// entry and nobody else needs it: every thread reads ids from the free list.
//
// One launch.  A CTA owns a range of tokens (and the sequences that begin in it).
// With up to kThreads sequences one block-wide scan gives both sums.  With more, the
// CTAs of a cluster first add up all sequences between them, in pieces of 128 or more
// (512 pieces at most, a warp a piece), and each scans the pieces' sums, which tells it
// where its range begins to within a piece; it then scans on from there, kThreads
// sequences at a time, to the range's end.  So no cluster waits for another and no
// workspace is needed.
//
// What bounds it: latency (16 bytes a token are written, some 12 a sequence read).  GB300:
// 64 sequences of a token 2.8 us, one of 131,071 tokens 3.5, 4,096 mixed 6.0 us, 16,384 of a
// token 8.8 us, 65,536 24 (8.0, 17.6 and 49 with every CTA adding up all of them).
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr unsigned kCluster = 8;     // CTAs that add up the sequences together, where they are many

struct ExtendParams {
    ExtendArgs a;
    int32_t per;              // tokens a CTA
    uint32_t ctas;            // that have tokens (the grid is whole clusters)
    uint32_t div_mul;         // division by the block size: see divided
    int32_t div_shift;
    unsigned int *err;
};

struct Sums {
    int64_t tok, blk;
};

__device__ __forceinline__ Sums operator+(Sums x, Sums y) { return {x.tok + y.tok, x.blk + y.blk}; }

__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
    return {__shfl_up_sync(0xffffffffu, v.tok, d), __shfl_up_sync(0xffffffffu, v.blk, d)};
}

__device__ __forceinline__ Sums warp_sum(Sums v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v.tok += __shfl_xor_sync(0xffffffffu, v.tok, d);
        v.blk += __shfl_xor_sync(0xffffffffu, v.blk, d);
    }
    return v;
}

// Block-wide: `inclusive` of each thread's v, and the sum of all.  Synchronises first.
__device__ __forceinline__ Sums block_scan(Sums v, Sums *part, Sums &inclusive) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums u = shfl_up(v, d);
        if (lane >= d) v = v + u;
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    Sums all = {0, 0};
#pragma unroll
    for (int w = 0; w < kWarpsPerCta; ++w) {
        if (w == warp) v = v + all;
        all = all + part[w];
    }
    inclusive = v;
    return all;
}

// One sequence's lengths as they count: a sequence whose lengths are negative or
// leave its table has no new tokens.
struct Request {
    int32_t ctx, n, have, need;
    bool bad;
};

// n / b for 0 <= n < 2^31, as (n * m) >> (31 + s) with 2^s >= b and m = floor(2^(31 + s) / b) + 1:
// m b = 2^(31 + s) + e with 0 < e <= b <= 2^s, so n m / 2^(31 + s) is above n / b by less than 1 / b.
// (The division itself was most of what a CTA did with 16,384 sequences.)
__device__ __forceinline__ uint32_t divided(const ExtendParams &p, uint32_t n) {
    return (uint32_t)(((uint64_t)n * p.div_mul) >> p.div_shift);
}
__device__ __forceinline__ int32_t blocks_of(const ExtendParams &p, uint32_t tokens) {   // rounded up
    return tokens == 0 ? 0 : (int32_t)divided(p, tokens - 1) + 1;
}

__device__ __forceinline__ Request request(const ExtendParams &p, int32_t ctx, int32_t n) {
    const ExtendArgs &a = p.a;
    Request r;
    const int64_t end = (int64_t)ctx + n;
    const int64_t cap = min((int64_t)a.max_blocks * a.block_size, (int64_t)INT32_MAX);
    r.bad = ctx < 0 || n < 0 || end > cap;
    r.ctx = ctx;
    r.n = r.bad ? 0 : n;
    r.have = r.bad ? 0 : blocks_of(p, (uint32_t)ctx);
    r.need = r.bad ? 0 : blocks_of(p, (uint32_t)end) - r.have;
    return r;
}

__device__ __forceinline__ Request load_request(const ExtendParams &p, int s) {
    return s < p.a.num_seqs ? request(p, __ldg(p.a.ctx_lens + s), __ldg(p.a.new_lens + s))
                            : Request{0, 0, 0, 0, false};
}

__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const __grid_constant__ ExtendParams p) {
    const ExtendArgs &a = p.a;
    // (in a cluster: every CTA has begun before another writes to its shared memory, below)
    if (a.num_seqs > kThreads) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ Sums part[kWarpsPerCta];      // of a scan's warps
    __shared__ Sums piece_[kThreads];        // of the pieces
    __shared__ int32_t end_[kThreads];       // of a scanned sequence: its tokens' end in the flat arrays
    __shared__ int32_t start_[kThreads];     // and their start
    __shared__ int32_t blk_[kThreads];       // its new blocks' place in the free list; -1: not served
    __shared__ int32_t ctx_[kThreads];
    __shared__ int32_t off_[kThreads];       // what is added to its positions
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = a.num_seqs;
    const bool last = blockIdx.x + 1 == p.ctas;
    const int64_t lo = (int64_t)blockIdx.x * p.per;
    const int64_t hi = min(lo + p.per, (int64_t)a.max_tokens);
    const int32_t cursor = __ldg(a.cursor);
    const bool cursor_ok = cursor >= 0 && cursor <= a.num_free;
    const int64_t left = cursor_ok ? a.num_free - cursor : 0;

    // ---- where to begin: the sums before sequence `first`
    Sums before = {0, 0}, total = {0, 0};
    int first = 0;
    if (B > kThreads) {
        const int piece = (B + 128 * kThreads - 1) / (128 * kThreads) * 128;
        const int pieces = (B + piece - 1) / piece;
        // the cluster's CTAs take turns at the pieces, and each leaves its sums with all of them
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        uint32_t rank, ctas;
        asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
        for (int i = warp * ctas + rank; i < pieces; i += kWarpsPerCta * ctas) {
            Sums mine = {0, 0};
            for (int s = i * piece + lane; s < (i + 1) * piece; s += 128) {
                Request r[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) r[q] = load_request(p, s + 32 * q);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mine.tok += r[q].n;
                    mine.blk += r[q].need;
                }
            }
            mine = warp_sum(mine);
            if (lane < ctas) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(piece_ + i)), "r"(lane));
                asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(at), "l"(mine.tok), "l"(mine.blk)
                             : "memory");
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        // thread t holds piece t's sums; the first piece that reaches the range
        const Sums own = tid < pieces ? piece_[tid] : Sums{0, 0};
        Sums at;
        total = block_scan(own, part, at);     // at: inclusive
        const bool reaches = tid < pieces && at.tok >= lo;
        const int n = __syncthreads_count(reaches);   // sums only grow: the last n pieces reach it
        if (n == 0) {
            first = B;
        } else {
            if (tid == pieces - n) {
                piece_[0] = {at.tok - own.tok, at.blk - own.blk};
            }
            __syncthreads();
            first = (pieces - n) * piece;
            before = piece_[0];
        }
    }

    if (blockIdx.x >= p.ctas) return;      // there to fill a cluster

    // ---- kThreads sequences at a time: scan, the sequences' own outputs, their tokens
    for (int base = first; base < B; base += kThreads) {
        const int s = base + tid;
        const Request r = load_request(p, s);
        const int32_t off = s < B && a.position_offsets ? __ldg(a.position_offsets + s) : 0;
        Sums v;
        const Sums all = block_scan(Sums{r.n, r.need}, part, v);   // (the last round's sequences have been read)
        const Sums at = {before.tok + v.tok - r.n, before.blk + v.blk - r.need};
        const int64_t tok_end = at.tok + r.n;
        const bool served = tok_end <= a.max_tokens && (r.need == 0 || at.blk + r.need <= left);
        if (s < B && at.tok >= lo && (at.tok < hi || last)) {   // this CTA's sequence
            a.seq_lens_out[s] = served ? r.ctx + r.n : r.ctx;
            a.cu_seqlens[s] = (int32_t)min(at.tok, (int64_t)a.max_tokens);
            if (r.bad) raise_error(p.err, PA_DEVERR_SEQ_LEN);
            if (!served) {
                raise_error(p.err, PA_DEVERR_NO_ROOM);
                // the first sequence that is not served ends what the step takes from the list
                if (at.blk <= left && at.tok <= a.max_tokens) *a.cursor_out = cursor + (int32_t)at.blk;
            }
        }
        const int64_t chunk_lo = before.tok;
        before = before + all;
        if (B <= kThreads) total = before;
        start_[tid] = (int32_t)min(at.tok, (int64_t)a.max_tokens);
        end_[tid] = (int32_t)min(tok_end, (int64_t)a.max_tokens);
        blk_[tid] = served ? (int32_t)at.blk : -1;
        ctx_[tid] = r.ctx;
        off_[tid] = off;
        __syncthreads();
        const int64_t t1 = min(hi, before.tok);
        for (int64_t i = max(lo, chunk_lo) + tid; i < t1; i += kThreads) {
            int at0 = 0, n = kThreads;     // the sequence of token i: the first whose end is beyond it
#pragma unroll
            for (int step = 0; step < 9; ++step) {
                const int half = n >> 1;
                const bool right = end_[at0 + half - 1] <= (int32_t)i;
                at0 += right ? half : 0;
                n -= half;
            }
            const int32_t pos = ctx_[at0] + (int32_t)(i - start_[at0]);
            const uint32_t b = (uint32_t)a.block_size;
            const uint32_t column = divided(p, (uint32_t)pos), slot = (uint32_t)pos - column * b;
            const int32_t have = blocks_of(p, (uint32_t)ctx_[at0]);
            int64_t out = -1;
            if (blk_[at0] >= 0) {
                int32_t *entry = a.tables + (int64_t)(base + at0) * a.max_blocks + column;
                const bool fresh = (int32_t)column >= have;
                int32_t id = fresh ? __ldg(a.free_blocks + cursor + blk_[at0] + ((int32_t)column - have)) : *entry;
                if (id < 0 || id >= a.num_blocks) {
                    raise_error(p.err, PA_DEVERR_BLOCK_ID);
                    id = -1;
                }
                if (fresh && slot == 0) *entry = id;
                if (id >= 0) out = (int64_t)id * b + slot;
            }
            a.positions[i] = (int64_t)pos + off_[at0];
            a.slots[i] = out;
        }
        if (before.tok >= hi && !last) break;      // later sequences begin behind the range
    }
    // ---- what is the step's as a whole, and the places behind its tokens
    if (blockIdx.x == 0 && tid == 0) {
        a.cu_seqlens[B] = (int32_t)min(total.tok, (int64_t)a.max_tokens);
        if (!cursor_ok) raise_error(p.err, PA_DEVERR_NO_ROOM);
        if (total.blk <= left && total.tok <= a.max_tokens) *a.cursor_out = cursor + (int32_t)total.blk;
    }
    for (int64_t i = max(lo, total.tok) + tid; i < hi; i += kThreads) {
        a.positions[i] = 0;
        a.slots[i] = -1;
    }
}

}  // namespace

cudaError_t launch_extend_tables(const ExtendArgs &a, cudaStream_t stream) {
    ExtendParams p;
    p.a = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    int64_t ctas = ((int64_t)a.max_tokens + kThreads - 1) / kThreads;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    if (ctas > sms) ctas = sms;
    if (ctas < 1) ctas = 1;
    int s = 0;
    while ((1ll << s) < a.block_size) ++s;
    p.div_mul = (uint32_t)((1ull << (31 + s)) / (uint64_t)a.block_size + 1);
    p.div_shift = 31 + s;
    p.per = (int32_t)(((int64_t)a.max_tokens + ctas - 1) / ctas);
    ctas = p.per > 0 ? ((int64_t)a.max_tokens + p.per - 1) / p.per : 1;
    p.ctas = (uint32_t)ctas;
    const unsigned cluster = a.num_seqs > kThreads ? kCluster : 1u;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(((unsigned)ctas + cluster - 1) / cluster * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, extend_tables_kernel, p);
}

}  // namespace pa
