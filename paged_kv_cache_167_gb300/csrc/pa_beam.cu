// pa_beam.cu -- beam search's selection: the best continuations of a group's
// beams over the whole vocabulary.
//
// score(j, v) = beam_scores[j] + x - log sum exp x.  Two kernels, one pass over
// the logits:
//
// 1. scan: CTA (slice, row) reads its slice of one row once.  Each thread keeps
//    the running maximum and the sum of exponentials relative to it (rescaled
//    when the maximum rises), and which vector its maximum came from.  The n-th
//    largest of the threads' maxima is a lower bound of the slice's n-th largest
//    element, so only the few threads whose maximum reaches it can hold a
//    candidate: their elements (and no others) are read again, from L2, and
//    those at or above the bound are ranked.  Keys are (value, lower index
//    first), so they are unique, ties need no further rule, and a row of equal
//    values collects no more than one vector per bounding thread.
// 2. merge: one CTA per group joins the slices' sums in fp64, turns the lists
//    (each sorted) into fp64 scores and picks the n best by the same bound, taken
//    over the lists' heads.
#include <algorithm>
#include <cfloat>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;            // candidates ranked at once
constexpr float kLog2eHi = 1.44269502162933349609375f;     // log2(e) rounded to fp32
constexpr float kLog2eLo = 1.92596299112661746887e-8f;     // and the rest

// fp32 bits in increasing order; both zeros and the subnormals (which the
// fp32 maximum flushes, and whose scores fp64 cannot tell apart) are one value.
__device__ __forceinline__ uint32_t order_of(float x) {
    uint32_t b = __float_as_uint(x);
    if ((b & 0x7f800000u) == 0) b = 0;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) {
    return ((uint64_t)order << 32) | (0xffffffffu - index);
}
constexpr uint64_t kLeastKey = (uint64_t)(0x007fffffu + 1) << 32;   // above every key of -inf (order 0x007fffff)

// exp(t) for t <= 0: 2^(t log2 e), the product carried to more than fp32
__device__ __forceinline__ float exp_neg(float t) { return fast_exp2(__fmaf_rn(t, kLog2eHi, t * kLog2eLo)); }

struct BeamParams {
    const void *logits;
    int64_t row_stride;              // elements
    const float *beam_scores;
    const uint8_t *finished;
    int32_t end_token;
    int32_t num_beams, vocab, num_out, slices;
    // workspace, one entry per (row, slice)
    double *sums;
    float *maxima;
    int32_t *counts;
    float *values;                   // [..][num_out], descending
    int32_t *indices;
    float *scores_out;
    int32_t *parents_out, *tokens_out;
    unsigned int *err;
};

// Sixteen bytes of a row as fp32.
template <typename T> struct Elements;
template <> struct Elements<uint16_t> {                        // bf16
    static constexpr int kVec = 8;
    static constexpr uint32_t kMinusInf = 0xff80u;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <> struct Elements<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kMinusInf = 0xff800000u;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};

// A row read in vectors j of elements [j * kVec, (j + 1) * kVec), -inf behind the
// last one.  Which thread sums which elements, and so every rounding, goes by the
// element's index alone: equal rows have equal sums, wherever they begin.  A row
// that does not begin on 16 bytes (an odd vocabulary) takes each vector out of
// the two aligned ones around it; the second of them is the next lane's first.
// (Before a row that is not aligned lies another row, so the first aligned
// vector is inside the tensor.)
template <typename T>
struct Row {
    static constexpr int kVec = Elements<T>::kVec;
    const T *x;
    int32_t vocab;
    uint32_t skew;                   // elements between the aligned address below x and x

    __device__ __forceinline__ Row(const T *row, int32_t n)
        : x(row), vocab(n), skew((uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)) {}

    __device__ __forceinline__ uint4 load(int32_t j) const {
        const int32_t e0 = j * kVec;
        const uint4 *at = reinterpret_cast<const uint4 *>(x + (e0 - (int32_t)skew));
        if (skew == 0) {
            if (vocab - e0 >= kVec) return __ldg(at);
        } else if ((int64_t)e0 + 2 * kVec - skew <= vocab) {
            const uint4 a = __ldg(at), b = __ldg(at + 1);
            uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const uint32_t bytes = skew * sizeof(T);
            if (bytes & 8u) {
#pragma unroll
                for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
            }
            if (bytes & 4u) {
#pragma unroll
                for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
            }
            if (sizeof(T) == 2) {
                const uint32_t shift = (bytes & 2u) * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], shift);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
        uint32_t e[kVec], w[4];      // the row's last elements, one by one
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            e[i] = Elements<T>::kMinusInf;
            if (i < vocab - e0) {
                if constexpr (sizeof(T) == 2)
                    e[i] = __ldg(reinterpret_cast<const unsigned short *>(x) + e0 + i);
                else
                    e[i] = __float_as_uint(__ldg(reinterpret_cast<const float *>(x) + e0 + i));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2)
                w[i] = e[2 * i] | (e[2 * i + 1] << 16);
            else
                w[i] = e[i];
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Whether a beam's logits matter: in use and not ended.
__device__ __forceinline__ bool beam_runs(const BeamParams &p, int row) {
    if (p.finished && __ldg(p.finished + row)) return false;
    const float score = __ldg(p.beam_scores + row);
    return score > -INFINITY && score < INFINITY;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const BeamParams p) {
    using E = Elements<T>;
    constexpr int VN = E::kVec;
    constexpr int kUnroll = 4;
    __shared__ uint64_t keys[kCap];          // the threads' bounds first, then the candidates
    __shared__ int32_t holders[kThreads];
    __shared__ int num_holders, num_found;
    __shared__ uint64_t bound;
    __shared__ float warp_max[kWarps];
    __shared__ double warp_sum[kWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = blockIdx.x, row = blockIdx.y;
    const int64_t entry = (int64_t)row * p.slices + slice;
    const int n = p.num_out;
    if (!beam_runs(p, row)) {
        if (tid == 0) {
            p.counts[entry] = 0;
            p.maxima[entry] = -INFINITY;
            p.sums[entry] = 0.0;
        }
        return;
    }
    const Row<T> x(static_cast<const T *>(p.logits) + (int64_t)row * p.row_stride, p.vocab);
    const int32_t vectors = (p.vocab + VN - 1) / VN;
    const int32_t lo = (int32_t)((int64_t)vectors * slice / p.slices);
    const int32_t hi = (int32_t)((int64_t)vectors * (slice + 1) / p.slices);

    float m = -INFINITY, sum = 0.f;
    int32_t best = lo;
    for (int32_t j0 = lo + tid; j0 < hi; j0 += kThreads * kUnroll) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (j0 + u * kThreads < hi) v[u] = x.load(j0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t j = j0 + u * kThreads;
            if (j >= hi) break;
            float e[VN];
            E::unpack(v[u], e);
            float top = e[0];
#pragma unroll
            for (int i = 1; i < VN; ++i) top = fmaxf(top, e[i]);
            if (top > m) {
                sum *= exp_neg(m - top);
                m = top;
                best = j;
            }
            const float ref = m == -INFINITY ? 0.f : m;      // NaN and +inf end up in the sum as NaN
#pragma unroll
            for (int i = 0; i < VN; ++i) sum += exp_neg(e[i] - ref);
        }
    }

    // slice maximum and sum
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) warp_max[warp] = top;
    // the thread's best key lies between those of its vector's last and first element
    const uint64_t least = m > -INFINITY ? key_of(order_of(m), (uint32_t)best * VN + (VN - 1)) : 0;
    const uint64_t most = m > -INFINITY ? key_of(order_of(m), (uint32_t)best * VN) : 0;
    keys[tid] = least;
    if (tid == 0) bound = kLeastKey;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_max[w]);
    double part = top == -INFINITY ? (double)sum : (double)sum * (double)exp_neg(m - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) warp_sum[warp] = part;
    // the n-th largest of the threads' bounds
    int above = 0;
    for (int t = 0; t < kThreads; ++t) above += keys[t] > least;
    if (least != 0 && above == n - 1 && least > kLeastKey) bound = least;
    __syncthreads();
    if (tid == 0) {
        double total = 0.0;
        for (int w = 0; w < kWarps; ++w) total += warp_sum[w];
        p.sums[entry] = total;
        p.maxima[entry] = top;
    }
    int found;
    while (true) {
        const uint64_t limit = bound;
        if (tid == 0) num_holders = num_found = 0;
        __syncthreads();
        if (most >= limit) holders[atomicAdd(&num_holders, 1)] = tid;
        __syncthreads();
        for (int w = warp; w < num_holders; w += kWarps)
            for (int32_t j = lo + holders[w] + lane * kThreads; j < hi; j += 32 * kThreads) {
                float e[VN];
                E::unpack(x.load(j), e);
#pragma unroll
                for (int i = 0; i < VN; ++i) {
                    const uint64_t key = key_of(order_of(e[i]), (uint32_t)j * VN + i);
                    if (e[i] > -INFINITY && key >= limit) {
                        const int at = atomicAdd(&num_found, 1);
                        if (at < kCap) keys[at] = key;
                    }
                }
            }
        __syncthreads();
        found = num_found;
        if (found <= kCap) break;
        // More than are ranked at once (many large values in few threads): the
        // n-th largest of those held is a higher bound; kCap - n elements drop out.
        for (int c = tid; c < kCap; c += kThreads) {
            const uint64_t mine = keys[c];
            int rank = 0;
            for (int t = 0; t < kCap; ++t) rank += keys[t] > mine;
            if (rank == n - 1) bound = mine;
        }
        __syncthreads();
    }
    for (int c = tid; c < found; c += kThreads) {
        const uint64_t mine = keys[c];
        int rank = 0;
        for (int t = 0; t < found; ++t) rank += keys[t] > mine;
        if (rank < n) {
            p.values[entry * n + rank] = value_of((uint32_t)(mine >> 32));
            p.indices[entry * n + rank] = (int32_t)(0xffffffffu - (uint32_t)mine);
        }
    }
    if (tid == 0) p.counts[entry] = found < n ? found : n;
}

// A candidate of a group: fp64 score in increasing integer order, then the flat
// index, lower first.
struct Candidate {
    int64_t score;
    int32_t index;
};
__device__ __forceinline__ int64_t order_of(double s) {
    const int64_t b = __double_as_longlong(s + 0.0);
    return b ^ (int64_t)((uint64_t)(b >> 63) >> 1);
}
__device__ __forceinline__ double score_of(int64_t o) {
    return __longlong_as_double(o ^ (int64_t)((uint64_t)(o >> 63) >> 1));
}
__device__ __forceinline__ bool better(const Candidate &a, const Candidate &b) {
    return a.score > b.score || (a.score == b.score && a.index < b.index);
}

struct Beam {
    double score, lse;
    int32_t kind;                    // 0: nothing but -inf, 1: runs, 2: ended
};

__device__ __forceinline__ int list_count(const BeamParams &p, const Beam &b, int64_t entry, int slice) {
    return b.kind == 1 ? __ldcg(p.counts + entry) : b.kind == 2 && slice == 0 ? 1 : 0;
}
__device__ __forceinline__ Candidate list_item(const BeamParams &p, const Beam &b, int j, int64_t entry, int i) {
    Candidate c;
    if (b.kind == 2) {
        c.score = order_of(b.score);
        c.index = j * p.vocab + p.end_token;
    } else {
        c.score = order_of(b.score + ((double)__ldcg(p.values + entry * p.num_out + i) - b.lse));
        c.index = j * p.vocab + __ldcg(p.indices + entry * p.num_out + i);
    }
    return c;
}

// Dynamic shared memory: beams [num_beams], list heads [num_beams * slices],
// candidates [num_out * min(num_out, lists)], chosen indices [num_out].
__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamParams p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ int num_found;
    __shared__ Candidate bound;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, g = blockIdx.x, n = p.num_out, lists = p.num_beams * p.slices;
    Beam *beams = reinterpret_cast<Beam *>(dyn);
    Candidate *heads = reinterpret_cast<Candidate *>(beams + p.num_beams);
    Candidate *found = heads + lists;
    int32_t *chosen = reinterpret_cast<int32_t *>(found + n * min(n, lists));
    if (tid == 0) {
        num_found = 0;
        bound.score = INT64_MIN;
        bound.index = INT32_MAX;
    }
    for (int j = tid; j < p.num_beams; j += kThreads) {
        const int row = g * p.num_beams + j;
        const float score = __ldg(p.beam_scores + row);
        Beam b = {(double)score, 0.0, 0};
        bool bad = !(score < INFINITY);
        if (!bad && score > -INFINITY) {
            if (p.finished && __ldg(p.finished + row)) {
                b.kind = 2;
            } else {
                float top = -INFINITY;
                double total = 0.0;
                for (int s = 0; s < p.slices; ++s) top = fmaxf(top, __ldcg(p.maxima + (int64_t)row * p.slices + s));
                for (int s = 0; s < p.slices; ++s) {
                    const int64_t e = (int64_t)row * p.slices + s;
                    const double part = __ldcg(p.sums + e);
                    const float m = __ldcg(p.maxima + e);
                    total += m == top || part != part ? part : part * exp((double)m - (double)top);
                }
                bad = !(top < INFINITY) || total != total;
                if (!bad && top > -INFINITY) {
                    b.kind = 1;
                    b.lse = (double)top + log(total);
                }
            }
        }
        if (bad) raise_error(p.err, PA_DEVERR_VALUE);
        beams[j] = b;
    }
    __syncthreads();
    for (int l = tid; l < lists; l += kThreads) {
        const int j = l / p.slices, s = l - j * p.slices;
        const int64_t entry = ((int64_t)g * p.num_beams + j) * p.slices + s;
        Candidate c = {INT64_MIN, INT32_MAX};
        if (list_count(p, beams[j], entry, s) > 0) c = list_item(p, beams[j], j, entry, 0);
        heads[l] = c;
    }
    __syncthreads();
    for (int l = tid; l < lists; l += kThreads) {
        const Candidate mine = heads[l];
        int rank = 0;
        for (int t = 0; t < lists; ++t) rank += better(heads[t], mine);
        if (rank == n - 1 && mine.score != INT64_MIN) bound = mine;
    }
    __syncthreads();
    for (int l = tid; l < lists; l += kThreads) {
        if (heads[l].score == INT64_MIN || better(bound, heads[l])) continue;
        const int j = l / p.slices, s = l - j * p.slices;
        const int64_t entry = ((int64_t)g * p.num_beams + j) * p.slices + s;
        const int count = list_count(p, beams[j], entry, s);
        for (int i = 0; i < count; ++i) {
            const Candidate c = list_item(p, beams[j], j, entry, i);
            if (better(bound, c)) break;
            found[atomicAdd(&num_found, 1)] = c;
        }
    }
    __syncthreads();
    const int total = num_found, listed = total < n ? total : n;
    for (int c = tid; c < total; c += kThreads) {
        const Candidate mine = found[c];
        int rank = 0;
        for (int t = 0; t < total; ++t) rank += better(found[t], mine);
        if (rank >= n) continue;
        chosen[rank] = mine.index;
        const int64_t o = (int64_t)g * n + rank;
        p.scores_out[o] = (float)score_of(mine.score);
        p.parents_out[o] = mine.index / p.vocab;
        p.tokens_out[o] = mine.index % p.vocab;
    }
    __syncthreads();
    if (tid == 0 && listed < n) {
        // every candidate above -inf is listed: the lowest other indices fill up
        int at = listed;
        for (int f = 0; at < n; ++f) {
            bool taken = false;
            for (int c = 0; c < listed; ++c) taken |= chosen[c] == f;
            if (taken) continue;
            const int64_t o = (int64_t)g * n + at++;
            p.scores_out[o] = -INFINITY;
            p.parents_out[o] = f / p.vocab;
            p.tokens_out[o] = f % p.vocab;
        }
    }
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Slices per row: enough CTAs to fill the SMs several times over, none shorter
// than 4096 elements.
int beam_slices(int64_t rows, int64_t vocab) {
    const int64_t want = (4 * 152 + rows - 1) / rows, most = (vocab + 4095) / 4096;
    return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 32}));
}

size_t merge_smem(int beams, int slices, int n) {
    const int lists = beams * slices;
    return beams * sizeof(Beam) + (size_t)lists * sizeof(Candidate) + (size_t)n * std::min(n, lists) * sizeof(Candidate) +
           n * sizeof(int32_t);
}

}  // namespace

size_t beam_workspace(int64_t rows, int32_t vocab, int32_t num_out) {
    const size_t entries = (size_t)rows * beam_slices(rows, vocab);
    return round_up(entries * 8) + 2 * round_up(entries * 4) + 2 * round_up(entries * num_out * 4);
}

cudaError_t launch_beam_select(const BeamArgs &a, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.num_groups * a.num_beams;
    BeamParams p = {};
    p.logits = a.logits;
    p.row_stride = a.row_stride;
    p.beam_scores = a.beam_scores;
    p.finished = a.finished;
    p.end_token = a.end_token;
    p.num_beams = a.num_beams;
    p.vocab = a.vocab;
    p.num_out = a.num_out;
    p.slices = beam_slices(rows, a.vocab);
    const size_t entries = (size_t)rows * p.slices;
    char *w = static_cast<char *>(a.workspace);
    p.sums = reinterpret_cast<double *>(w);
    w += round_up(entries * 8);
    p.maxima = reinterpret_cast<float *>(w);
    w += round_up(entries * 4);
    p.counts = reinterpret_cast<int32_t *>(w);
    w += round_up(entries * 4);
    p.values = reinterpret_cast<float *>(w);
    w += round_up(entries * a.num_out * 4);
    p.indices = reinterpret_cast<int32_t *>(w);
    p.scores_out = a.scores_out;
    p.parents_out = a.parents_out;
    p.tokens_out = a.tokens_out;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    const dim3 grid(p.slices, (unsigned)rows);
    cudaError_t e = a.bf16 ? launch_pdl(beam_scan_kernel<uint16_t>, grid, dim3(kThreads), stream, p)
                           : launch_pdl(beam_scan_kernel<float>, grid, dim3(kThreads), stream, p);
    if (e != cudaSuccess) return e;
    const size_t smem = merge_smem(a.num_beams, p.slices, a.num_out);
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(beam_merge_kernel, dim3(a.num_groups), dim3(kThreads), stream, p, smem);
}

}  // namespace pa
