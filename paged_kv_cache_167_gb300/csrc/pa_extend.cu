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
// With up to kThreads sequences one block-wide scan gives both sums.  With more,
// each CTA first adds up all sequences, a contiguous sixteenth a warp, which tells
// it the sums at sixteen places; it then scans on, kThreads sequences at a time,
// from the last place before its range to the range's end.  So no CTA waits for
// another and no workspace is needed; the lengths are read by every CTA, from L2.
//
// What bounds it: latency (16 bytes a token are written, some 12 a sequence read).
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarpsPerCta = kThreads / 32;

struct ExtendParams {
    ExtendArgs a;
    int32_t per;              // tokens a CTA
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

// One sequence's lengths as they count: a sequence whose lengths are negative or
// leave its table has no new tokens.
struct Request {
    int32_t ctx, n, have, need;
    bool bad;
};

__device__ __forceinline__ Request request(const ExtendArgs &a, int32_t ctx, int32_t n) {
    Request r;
    const int64_t end = (int64_t)ctx + n;
    const int64_t cap = min((int64_t)a.max_blocks * a.block_size, (int64_t)INT32_MAX);
    r.bad = ctx < 0 || n < 0 || end > cap;
    r.ctx = ctx;
    r.n = r.bad ? 0 : n;
    const uint32_t b = (uint32_t)a.block_size;
    r.have = r.bad ? 0 : (int32_t)(((uint32_t)ctx + b - 1u) / b);
    r.need = r.bad ? 0 : (int32_t)(((uint32_t)end + b - 1u) / b) - r.have;
    return r;
}

__device__ __forceinline__ Request load_request(const ExtendArgs &a, int s) {
    return s < a.num_seqs ? request(a, __ldg(a.ctx_lens + s), __ldg(a.new_lens + s)) : Request{0, 0, 0, 0, false};
}

__global__ void __launch_bounds__(kThreads) extend_tables_kernel(const __grid_constant__ ExtendParams p) {
    const ExtendArgs &a = p.a;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ Sums part[kWarpsPerCta];      // totals: of the warps' sixteenths, then of a scan's warps
    __shared__ int32_t end_[kThreads];       // of a scanned sequence: its tokens' end in the flat arrays
    __shared__ int32_t start_[kThreads];     // and their start
    __shared__ int32_t blk_[kThreads];       // its new blocks' place in the free list; -1: not served
    __shared__ int32_t ctx_[kThreads];
    __shared__ int32_t off_[kThreads];       // what is added to its positions
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = a.num_seqs;
    const bool last = blockIdx.x + 1 == gridDim.x;
    const int64_t lo = (int64_t)blockIdx.x * p.per;
    const int64_t hi = min(lo + p.per, (int64_t)a.max_tokens);
    const int32_t cursor = __ldg(a.cursor);
    const bool cursor_ok = cursor >= 0 && cursor <= a.num_free;
    const int64_t left = cursor_ok ? a.num_free - cursor : 0;

    // ---- where to begin: the sums before sequence `first`
    Sums before = {0, 0}, total = {0, 0};
    int first = 0;
    if (B > kThreads) {
        const int seg = (B + kWarpsPerCta - 1) / kWarpsPerCta;
        const int s1 = min(B, (warp + 1) * seg);
        Sums mine = {0, 0};
#pragma unroll 8
        for (int s = warp * seg + lane; s < s1; s += 32) {
            const Request r = load_request(a, s);
            mine.tok += r.n;
            mine.blk += r.need;
        }
        mine = warp_sum(mine);
        if (lane == 0) part[warp] = mine;
        __syncthreads();
        bool found = false;
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w) {
            const Sums v = part[w];
            if (!found && total.tok + v.tok >= lo) {   // the first sixteenth that reaches the range
                found = true;
                first = w * seg;
                before = total;
            }
            total = total + v;
        }
        if (!found) first = B;
    }

    // ---- kThreads sequences at a time: scan, the sequences' own outputs, their tokens
    for (int base = first; base < B; base += kThreads) {
        const int s = base + tid;
        const Request r = load_request(a, s);
        const int32_t off = s < B && a.position_offsets ? __ldg(a.position_offsets + s) : 0;
        Sums v = {r.n, r.need};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums u = shfl_up(v, d);
            if (lane >= d) v = v + u;
        }
        __syncthreads();      // the totals and the last round's sequences have been read
        if (lane == 31) part[warp] = v;
        __syncthreads();
        Sums all = {0, 0}, mine = before;
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w) {
            if (w == warp) mine = mine + all;
            all = all + part[w];
        }
        const Sums at = {mine.tok + v.tok - r.n, mine.blk + v.blk - r.need};
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
            const uint32_t column = (uint32_t)pos / b, slot = (uint32_t)pos - column * b;
            const int32_t have = (int32_t)(((uint32_t)ctx_[at0] + b - 1u) / b);
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
    p.per = (int32_t)(((int64_t)a.max_tokens + ctas - 1) / ctas);
    ctas = p.per > 0 ? ((int64_t)a.max_tokens + p.per - 1) / p.per : 1;
    return launch_pdl(extend_tables_kernel, dim3((unsigned)ctas), dim3(kThreads), stream, 0, p);
}

}  // namespace pa
