// pa_beam.cu -- beam search's selection: the best continuations of a group's
// beams over the whole vocabulary.
//
// score(j, v) = beam_scores[j] + x - log sum exp x.  Two steps, one pass over the
// logits; two kernels, or one where a group's CTAs are a cluster:
//
// 1. scan: CTA (slice, row) reads an equal share of the row's chunks (1024
//    vectors of 16 bytes, four for each thread) once, three chunks on their way
//    into shared memory at a time.  Each thread keeps the maximum, the chunk it
//    came from and the sum of exponentials; which elements a thread has goes by
//    their index in the row.  The n-th largest of the maxima of 4 n groups of
//    threads is a lower bound of the slice's n-th largest element (and close to
//    it: some 9 elements reach it at n = 8), so only the few threads whose maximum
//    reaches it can hold a candidate: their four vectors of that chunk (and the
//    others only if the second best chunk reaches it too) are read again, from
//    cache, and the elements at or above the bound are ranked.  Keys are (value,
//    lower index first), so they are unique and ties need no further rule.
// 2. merge: one CTA per group (of a cluster, the first) adds up each row's slices,
//    turns the slices' lists (each sorted) into fp64 scores and picks the n best by
//    the same bound, taken over the lists' fronts.
//
// The exponentials: 2^(x L - c) with L = log2(e) rounded to fp32 and c the running
// maximum's m L rounded to an integer: one fused multiply-add (x L is not rounded
// by itself) and one hardware 2^x.  The sum is then relative to c / L, which fp64
// holds, so c's rounding biases nothing; L's own (2^-26) acts on the distance to
// the maximum only; and a rising c scales the sum by a power of two, exactly, with
// no branch.  A thread adds the elements of a chunk by halves and the chunks in a
// compensated sum, so its error does not grow with the row (one running sum a thread
// was up to 1.9e-6 off in rows of one value, whose roundings all go the same way; this
// costs 64 x 8 rows 0.5 of 56 us); above the thread sums are integers, in units of
// 2^-40 in a slice and of 2^-32 between slices.  So equal rows have equal sums
// wherever they begin.  A slice whose maximum is beyond 2^22 in
// size, where c would have no fraction left to lose (a row of the type's lowest
// value, say), is summed again from its differences to that maximum.
//
// What bounds it: the logits are read once (plus the candidates' vectors from
// cache).  GB300, of the measured copy bandwidth: 64 x 8 rows of 128,256 fp32 logits
// 55.6 us (0.70; the merge takes 5 us, and the SMs' last slices end at different times).
// Below that a chain of latencies: 32 x 4 rows of 128,256 bf16 logits 15.3 us (about 5
// to stream, 3 for the slice's end, 4 to merge), 4 rows of 32,000 in one cluster 9.7.
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;            // vectors a thread loads at once
constexpr int kChunk = kThreads * kUnroll;
constexpr int kStages = 3;            // chunks in flight or at work
constexpr int kPart = 33;             // a warp's 32 neighbouring vectors and the one behind them
constexpr size_t kScanSmem = (size_t)kStages * kWarps * kUnroll * kPart * sizeof(uint4);
constexpr int kCtasPerSm = 4;
constexpr int kMaxCluster = 16;
constexpr int kHalfTheSms = 76;       // of a GB300
constexpr int kFewLists = 64, kMaxLists = 640;   // of a group
constexpr int kCap = 1024;            // candidates ranked at once
constexpr float kLog2e = 1.44269502162933349609375f;   // log2(e) rounded to fp32
constexpr float kFar = 4194304.f;                      // 2^22
constexpr float kUnit = 1099511627776.f;               // 2^40 (a slice has less than 2^22 elements, each below 2^0.5)
constexpr unsigned long long kStrange = ~0ull;         // a warp's sum with a NaN or +inf

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

// Sixteen bytes from global to shared memory, past the registers.
__device__ __forceinline__ void copy_async(uint4 *to, const uint4 *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Two fp32 in one 64-bit register, for the paired multiply-add and add.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_sub(uint64_t a, uint64_t b) {
    return pair_fma(b, pair(-1.f, -1.f), a);
}

// The reference c of a maximum, an integer below 2^24; finite for -inf, so that
// 0 * 2^(c - c') is 0.
__device__ __forceinline__ float reference_of(float m) {
    return rintf(__fmul_rn(fminf(fmaxf(m, -kFar), kFar), kLog2e));
}
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar && fabsf(m) < INFINITY; }

struct BeamParams {
    const void *logits;
    int64_t row_stride;              // elements
    const float *beam_scores;
    const uint8_t *finished;
    int32_t end_token;
    int32_t num_beams, vocab, num_out;
    int32_t row_vectors;             // ceil(vocab / elements of a vector)
    int32_t row_chunks;              // ceil(row_vectors / kChunk)
    int32_t slices;                  // of a row
    int32_t depth;                   // of the lists' fronts in the merge
    // workspace, one entry for each (row, slice)
    unsigned long long *sums;        // of 2^(x L - reference_of(maximum)), or of e^(x - maximum) if that is far; 2^-32
    float *maxima;                   // +inf: a NaN or +inf was met
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
    // of several vectors; NaN is passed over, as fmaxf does
    static __device__ __forceinline__ float maximum(const uint4 (&v)[kUnroll]) {
        auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); };
        __nv_bfloat162 t[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            t[u] = __hmax2(__hmax2(h(v[u].x), h(v[u].y)), __hmax2(h(v[u].z), h(v[u].w)));
        const __nv_bfloat162 m = __hmax2(__hmax2(t[0], t[1]), __hmax2(t[2], t[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ uint32_t minus_inf_word() { return 0xff80ff80u; }
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
    static __device__ __forceinline__ float maximum(const uint4 (&v)[kUnroll]) {
        float t[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            t[u] = fmaxf(fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                         fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
        return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    }
    static __device__ __forceinline__ uint32_t minus_inf_word() { return 0xff800000u; }
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

    // Vectors [0, whole()) lie inside the row together with the aligned ones
    // they are taken from, aligned() and the one after each.
    __device__ __forceinline__ int32_t whole() const {
        return skew == 0 ? vocab / kVec : (int32_t)(((int64_t)vocab + skew) / kVec) - 1;
    }
    __device__ __forceinline__ const uint4 *aligned() const { return reinterpret_cast<const uint4 *>(x - skew); }
    // The vector that begins skew elements into a.
    __device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b) const {
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
    __device__ __forceinline__ uint4 load(int32_t j) const {
        if (j < whole()) {
            const uint4 a = __ldg(aligned() + j);
            return skew == 0 ? a : shifted(a, __ldg(aligned() + j + 1));
        }
        const int32_t e0 = j * kVec;
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

struct ScanShared {
    __align__(16) uint64_t keys[kCap];              // the groups' bounds first, then the candidates
    int32_t holders[kThreads];                      // of candidates in one chunk: chunk * kThreads + thread
    int32_t rich[kThreads];                         // in more than one: the thread
    int num_holders, num_rich, num_found;
    uint64_t bound;
    unsigned long long warp_sum[kWarps];            // 2^-40, or kStrange
    float warp_max[kWarps];
};
static_assert(sizeof(ScanShared) <= kScanSmem, "the selection reuses the copies' shared memory");

// One slice of a row: its sum, maximum and list.
template <typename T>
__device__ __forceinline__ void scan_slice(const BeamParams &p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    using E = Elements<T>;
    constexpr int VN = E::kVec;
    uint4 *parts = reinterpret_cast<uint4 *>(dyn);  // [stage][warp][load][kPart] while the slice streams by
    ScanShared &sh = *reinterpret_cast<ScanShared *>(dyn);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.y, n = p.num_out;
    const int64_t entry = (int64_t)row * p.slices + blockIdx.x;
    if (!beam_runs(p, row)) {
        if (tid == 0) p.counts[entry] = 0;
        return;
    }
    // (at most 2^19 chunks and 640 slices: the products fit)
    const int32_t first = (int32_t)((uint32_t)p.row_chunks * blockIdx.x / (uint32_t)p.slices);
    const int32_t last = (int32_t)((uint32_t)p.row_chunks * (blockIdx.x + 1) / (uint32_t)p.slices);
    const Row<T> x(static_cast<const T *>(p.logits) + (int64_t)row * p.row_stride, p.vocab);
    const int32_t whole = x.whole(), vectors = p.row_vectors;
    const uint32_t none = E::minus_inf_word();
    float m = -INFINITY, second = -INFINITY;        // the largest of the chunks' maxima, and of the others'
    int32_t best = first;
    float c = reference_of(m);
    uint64_t sum = 0, lost = 0;                     // pairs: the sum, and what it has too much (Kahan's method)
    auto take = [&](const uint4 (&v)[kUnroll], int32_t k) {
        const float top = E::maximum(v);
        second = fmaxf(second, fminf(m, top));
        if (top > m) {
            m = top;
            best = k;
        }
        const float next = fmaxf(c, reference_of(top)), down = fast_exp2(c - next);
        c = next;
        sum = pair_mul(sum, pair(down, down));
        lost = pair_mul(lost, pair(down, down));
        const uint64_t minus_c = pair(-c, -c), scale = pair(kLog2e, kLog2e);
        uint64_t of[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float e[VN];
            uint64_t t[VN / 2];
            E::unpack(v[u], e);
#pragma unroll
            for (int i = 0; i < VN / 2; ++i) {      // NaN and +inf end up in the sum as NaN or inf
                const float2 s = unpair(pair_fma(pair(e[2 * i], e[2 * i + 1]), scale, minus_c));
                t[i] = pair(fast_exp2(s.x), fast_exp2(s.y));
            }
#pragma unroll
            for (int i = VN / 4; i > 0; i /= 2)     // by halves: equal elements double exactly
#pragma unroll
                for (int k = 0; k < i; ++k) t[k] = pair_add(t[k], t[k + i]);
            of[u] = t[0];
        }
        const uint64_t chunk = pair_add(pair_add(of[0], of[1]), pair_add(of[2], of[3]));
        const uint64_t more = pair_sub(chunk, lost), next_sum = pair_add(sum, more);
        lost = pair_sub(pair_sub(next_sum, sum), more);
        sum = next_sum;
    };
    // A thread copies its own vectors and reads its own copies; those of a warp are
    // neighbours, and a row that does not begin on 16 bytes (SKEW) needs the one
    // behind them too.
    auto stream = [&](auto skewed) {
        constexpr bool SKEW = decltype(skewed)::value;
        const int32_t available = SKEW ? whole + 1 : whole;
        const uint4 *from = x.aligned() + (int64_t)first * kChunk + tid;   // of the next chunk to start
        uint4 *const mine = parts + warp * (kUnroll * kPart) + lane;
        constexpr int kStage = kWarps * kUnroll * kPart;
        auto start = [&](int32_t chunk, uint4 *to) {
            if (chunk < last) {
                if ((chunk + 1) * kChunk < available) {    // (all of it, and one more)
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) copy_async(to + u * kPart, from + u * kThreads);
                    if (SKEW && lane == 31) {
#pragma unroll
                        for (int u = 0; u < kUnroll; ++u) copy_async(to + u * kPart + 1, from + u * kThreads + 1);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        const int32_t j = chunk * kChunk + u * kThreads + tid;
                        if (j < available) copy_async(to + u * kPart, from + u * kThreads);
                        if (SKEW && lane == 31 && j + 1 < available)
                            copy_async(to + u * kPart + 1, from + u * kThreads + 1);
                    }
                }
            }
            from += kChunk;
            copy_commit();                          // (an empty group where nothing is left)
        };
#pragma unroll
        for (int s = 0; s < kStages; ++s) start(first + s, mine + s * kStage);
        uint4 *at = mine;
        for (int32_t k = first; k < last; ++k) {
            copy_wait<kStages - 1>();               // chunk k has landed; the later ones may be under way
            if (SKEW) __syncwarp();
            uint4 v[kUnroll];
            if ((k + 1) * kChunk <= whole) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    v[u] = SKEW ? x.shifted(at[u * kPart], at[u * kPart + 1]) : at[u * kPart];
            } else {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int32_t j = k * kChunk + u * kThreads + tid;
                    v[u] = make_uint4(none, none, none, none);
                    if (j < whole)
                        v[u] = SKEW ? x.shifted(at[u * kPart], at[u * kPart + 1]) : at[u * kPart];
                    else if (j < vectors)
                        v[u] = x.load(j);           // the row's last one or two
                }
            }
            if (SKEW) __syncwarp();                 // every lane has read what its neighbours copied
            start(k + kStages, at);
            at = at == mine + (kStages - 1) * kStage ? mine : at + kStage;
            take(v, k);
        }
    };
    if (x.skew == 0)
        stream(std::false_type());
    else
        stream(std::true_type());
    float2 held = unpair(sum), over = unpair(lost);
    copy_wait<0>();
    __syncthreads();                                // the copies' shared memory is free

    // the slice's maximum, and the bounds of the groups (2^k neighbouring threads)
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.warp_max[warp] = top;
    // the thread's best key lies between those of its best chunk's last and first element
    const uint32_t begin = ((uint32_t)best * kChunk + tid) * VN;
    const uint64_t least = m > -INFINITY ? key_of(order_of(m), begin + (kUnroll - 1) * kThreads * VN + (VN - 1)) : 0;
    const uint64_t most = m > -INFINITY ? key_of(order_of(m), begin) : 0;
    const int group_log = n <= 8 ? 3 : n <= 16 ? 2 : n <= 32 ? 1 : 0, groups = kThreads >> group_log;
    uint64_t group = least;
    for (int o = 1; o < (1 << group_log); o <<= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, group, o);
        group = other > group ? other : group;
    }
    if ((tid & ((1 << group_log) - 1)) == 0) sh.keys[tid >> group_log] = group;
    if (tid == 0) {
        sh.bound = kLeastKey;
        sh.num_holders = sh.num_rich = sh.num_found = 0;
    }
    __syncthreads();
    const int32_t end = min(last * kChunk, vectors);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sh.warp_max[i]);
    float unit = kUnit;
    if (is_far(top)) {
        held = over = make_float2(0.f, 0.f);
        for (int32_t j = first * kChunk + tid; j < end; j += kThreads) {
            float e[VN];
            E::unpack(x.load(j), e);
#pragma unroll
            for (int i = 0; i < VN; ++i) e[i] = fast_exp2((e[i] - top) * kLog2e);
#pragma unroll
            for (int i = VN / 2; i > 0; i /= 2)
#pragma unroll
                for (int k = 0; k < i; ++k) e[k] += e[k + i];
            const float more = e[0] - over.x, next = held.x + more;
            over.x = (next - held.x) - more;
            held.x = next;
        }
    } else {
        unit *= fast_exp2(c - reference_of(top));
    }
    // both halves and what they have too much, exactly: whole and rest, and then integers
    const float whole_sum = held.x + held.y, second_half = whole_sum - held.x;
    const float rest = ((held.x - (whole_sum - second_half)) + (held.y - second_half)) - (over.x + over.y);
    const unsigned long long part = __float2ull_rn(whole_sum * unit) + (unsigned long long)__float2ll_rn(rest * unit);
    // (32 numbers of 24 bits fit a word)
    const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)part & 0xffffffu);
    const uint32_t mid = __reduce_add_sync(0xffffffffu, (uint32_t)(part >> 24) & 0xffffffu);
    const uint32_t high = __reduce_add_sync(0xffffffffu, (uint32_t)(part >> 48));
    const bool strange = __any_sync(0xffffffffu, !(fabsf(whole_sum) < INFINITY));
    if (lane == 0) sh.warp_sum[warp] = strange ? kStrange : low + ((uint64_t)mid << 24) + ((uint64_t)high << 48);
    if (tid < groups) {                             // the n-th largest of the groups' bounds
        const uint64_t mine = sh.keys[tid];
        int above = 0;
        for (int t = 0; t < groups; t += 2) {
            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(sh.keys + t);
            above += (k.x > mine) + (k.y > mine);
        }
        if (mine != 0 && above == n - 1) sh.bound = mine;
    }
    __syncthreads();
    if (tid == 0) {
        unsigned long long total = 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            bad |= sh.warp_sum[i] == kStrange;
            total += sh.warp_sum[i];
        }
        p.sums[entry] = (total + 128) >> 8;
        p.maxima[entry] = bad ? INFINITY : top;
    }
    int found;
    while (true) {
        const uint64_t limit = sh.bound;
        if (most >= limit) {
            if (second > -INFINITY && order_of(second) >= (uint32_t)(limit >> 32))
                sh.rich[atomicAdd(&sh.num_rich, 1)] = tid;
            else
                sh.holders[atomicAdd(&sh.num_holders, 1)] = best * kThreads + tid;
        }
        __syncthreads();
        auto collect = [&](int32_t j) {
            float e[VN];
            E::unpack(x.load(j), e);
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const uint64_t key = key_of(order_of(e[i]), (uint32_t)j * VN + i);
                if (e[i] > -INFINITY && key >= limit) {
                    const int to = atomicAdd(&sh.num_found, 1);
                    if (to < kCap) sh.keys[to] = key;
                }
            }
        };
        for (int i = tid; i < sh.num_holders * kUnroll; i += kThreads) {
            const int32_t h = sh.holders[i / kUnroll];
            const int32_t j = h / kThreads * kChunk + i % kUnroll * kThreads + h % kThreads;
            if (j < end) collect(j);
        }
        for (int h = warp; h < sh.num_rich; h += kWarps)
            for (int32_t j = first * kChunk + sh.rich[h] + lane * kThreads; j < end; j += 32 * kThreads) collect(j);
        __syncthreads();
        found = sh.num_found;
        if (found <= kCap) break;
        // More than are ranked at once (many large or equal values in few threads):
        // the n-th largest of those held is a higher bound; kCap - n elements drop out.
        for (int k = tid; k < kCap; k += kThreads) {
            const uint64_t mine = sh.keys[k];
            int rank = 0;
            for (int t = 0; t < kCap; ++t) rank += sh.keys[t] > mine;
            if (rank == n - 1) sh.bound = mine;
        }
        __syncthreads();
        if (tid == 0) sh.num_holders = sh.num_rich = sh.num_found = 0;
        __syncthreads();
    }
    for (int k = tid; k < found; k += kThreads) {
        const uint64_t mine = sh.keys[k];
        int rank = 0;
        for (int t = 0; t < found; ++t) rank += sh.keys[t] > mine;
        if (rank < n) {
            p.values[entry * n + rank] = value_of((uint32_t)(mine >> 32));
            p.indices[entry * n + rank] = (int32_t)(0xffffffffu - (uint32_t)mine);
        }
    }
    if (tid == 0) p.counts[entry] = found < n ? found : n;
}

// A candidate of a group: fp64 score in increasing integer order; equal scores by the
// row, then by the logit (which a score of its size may not hold: 0 and 2^-80), then by
// the index, as the row's lists are.
struct Candidate {
    int64_t score;
    int32_t index;                   // flat: row * vocab + token
    uint32_t logit;                  // order_of the logit
};
__device__ __forceinline__ int64_t order_of(double s) {
    const int64_t b = __double_as_longlong(s);
    return b == INT64_MIN ? 0 : b ^ (int64_t)((uint64_t)(b >> 63) >> 1);   // -0 is 0
}
__device__ __forceinline__ double score_of(int64_t o) {
    return __longlong_as_double(o ^ (int64_t)((uint64_t)(o >> 63) >> 1));
}
// (Without a branch but for the rare case: 9.7 us at 1 x 4 rows of 32,000, 10.0 with one
// for each step, and 9.45 without the logit.)
__device__ __forceinline__ bool better(const Candidate &a, const Candidate &b, int32_t vocab) {
    const bool equal = a.score == b.score;
    bool r = a.score > b.score || (equal && a.index < b.index);
    if (equal && a.logit != b.logit) {
        const int32_t row_a = a.index / vocab, row_b = b.index / vocab;
        r = row_a != row_b ? row_a < row_b : a.logit > b.logit;
    }
    return r;
}

// log(t 2^-32) for t > 0.  t = m 2^e with m in [0.707, 1.414]; log m = 2 artanh(z)
// with z = (m - 1) / (m + 1), |z| < 0.1716, artanh(z) = z (1 + z^2 / 3 + z^4 / 5 + ...).
// The bracket less 1 is below 0.01, so fp32 holds it to 2^-30; the rest is
// fp64, of which this part has two lanes an SM.  Within 2^-29 of the value.
__device__ __forceinline__ double log_units(unsigned long long t) {
    const double d = (double)t;
    const int64_t b = __double_as_longlong(d);
    int e = (int)(b >> 52) - 1023;
    double m = __longlong_as_double((b & 0x000fffffffffffffll) | 0x3ff0000000000000ll);   // [1, 2)
    if (m > 1.4142135623730951) {
        m *= 0.5;
        ++e;
    }
    const double up = m + 1.0;
    double r = (double)(1.0f / (float)up);
    r += r * (1.0 - up * r);
    const double z = (m - 1.0) * r;
    const float q = (float)z * (float)z;
    const float series = q * (1.f / 3 + q * (1.f / 5 + q * (1.f / 7 + q * (1.f / 9 + q * (1.f / 11 + q * (1.f / 13))))));
    return (e - 32) * 0.693147180559945309417232 + 2.0 * (z + z * (double)series);
}

constexpr Candidate kNoCandidate = {INT64_MIN, INT32_MAX, 0};

struct Beam {
    double base, offset;             // score(v) = (x - base) + offset
    unsigned long long total;        // the row's sum, 2^-32 units
    float top;
    int32_t kind;                    // 0: nothing but -inf, 1: runs, 2: ended
    int32_t flat;                    // j * vocab
};

// The number of items in [0, count) better than `mine`, which is item `of`, by
// the `per` neighbouring threads that share it (a power of two; all get it).
__device__ __forceinline__ int rank_of(const Candidate *items, int count, const Candidate &mine, int per,
                                       int32_t vocab) {
    int rank = 0;
#pragma unroll 4
    for (int t = threadIdx.x & (per - 1); t < count; t += per) rank += better(items[t], mine, vocab);
    for (int o = 1; o < per; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    return rank;
}
// Threads an item can have so that one round takes all of them.
__device__ __forceinline__ int share_of(int count) { return count <= 32 ? 8 : count <= 64 ? 4 : count <= 128 ? 2 : 1; }

// One group's selection out of its rows' lists.  Dynamic shared memory: the lists'
// fronts (their first `depth` candidates) [lists * depth], the candidates to rank
// [kCap], beams [num_beams], counts and the lists to look further into [lists] each.
__device__ __forceinline__ void merge_group(const BeamParams &p, int g) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Candidate best[kThreads];
    __shared__ Candidate bound;
    __shared__ int num_found, num_deep;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.num_out;
    const int lists = p.num_beams * p.slices, row0 = g * p.num_beams, depth = p.depth, fronts = lists * depth;
    const int64_t entry0 = (int64_t)row0 * p.slices;
    Candidate *front = reinterpret_cast<Candidate *>(dyn);
    Candidate *found = front + fronts;
    Beam *beams = reinterpret_cast<Beam *>(found + kCap);
    int32_t *counts = reinterpret_cast<int32_t *>(beams + p.num_beams), *deep = counts + lists;
    if (tid == 0) {
        num_found = num_deep = 0;
        bound = kNoCandidate;
    }
    // the fronts, raw, and every list's count: loads that depend on nothing
    for (int e = tid; e < fronts; e += kThreads) {
        const int l = e / depth, i = e - l * depth;
        const int64_t at = (entry0 + l) * n + i;
        front[e].score = (int64_t)__float_as_uint(__ldcg(p.values + at));
        front[e].index = __ldcg(p.indices + at);
    }
    for (int l = tid; l < lists; l += kThreads) counts[l] = __ldcg(p.counts + entry0 + l);
    // a warp per row: its maximum, and its sum relative to that.  (A row that
    // does not run has left its records as they were: read, and not used.)
    for (int j = warp; j < p.num_beams; j += kWarps) {
        const int64_t e0 = entry0 + j * p.slices;
        const float first = lane < p.slices ? __ldcg(p.maxima + e0 + lane) : -INFINITY;
        const unsigned long long first_sum = lane < p.slices ? __ldcg(p.sums + e0 + lane) : 0;
        const float score = __ldg(p.beam_scores + row0 + j);
        const bool done = p.finished && __ldg(p.finished + row0 + j);
        int kind = score > -INFINITY && score < INFINITY ? (done ? 2 : 1) : 0;
        float top = first;
        for (int i = lane + 32; i < p.slices; i += 32) top = fmaxf(top, __ldcg(p.maxima + e0 + i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool bad = !(score < INFINITY) || (kind == 1 && top == INFINITY);
        const bool far = is_far(top);
        const float reference = reference_of(top);
        unsigned long long total = 0;
        auto add = [&](float maximum, unsigned long long sum) {
            if (maximum == -INFINITY) return;
            if (!far && !is_far(maximum)) {
                const float down = reference - reference_of(maximum);
                if (down < 64.f) total += (sum + (1ull << (int)down >> 1)) >> (int)down;
            } else {                                // the slice's reference above the row's, in powers of two
                const float up = !far            ? __fmaf_rn(maximum, kLog2e, -reference)
                                 : is_far(maximum) ? (maximum - top) * kLog2e
                                                   : __fmaf_rn(-top, kLog2e, reference_of(maximum));
                total += up == 0.f ? sum : __float2ull_rn((float)sum * fast_exp2(up));
            }
        };
        if (kind == 1 && !bad) {
            add(first, first_sum);
            for (int i = lane + 32; i < p.slices; i += 32) add(__ldcg(p.maxima + e0 + i), __ldcg(p.sums + e0 + i));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (bad || (kind == 1 && top == -INFINITY)) kind = 0;
        if (lane == 0) {
            if (bad) raise_error(p.err, PA_DEVERR_VALUE);
            beams[j].offset = score;
            beams[j].total = total;
            beams[j].top = top;
            beams[j].kind = kind;
            beams[j].flat = j * p.vocab;
        }
    }
    __syncthreads();
    for (int j = tid; j < p.num_beams; j += kThreads) {    // fp64 once for all rows, side by side
        if (beams[j].kind != 1) continue;
        const float top = beams[j].top;
        beams[j].base = is_far(top) ? (double)top : (double)reference_of(top) * (1.0 / (double)kLog2e);
        beams[j].offset -= log_units(beams[j].total);
    }
    __syncthreads();
    auto candidate = [&](const Beam &b, float v, int32_t token) {
        Candidate c;
        c.score = order_of(b.kind == 2 ? b.offset : ((double)v - b.base) + b.offset);
        c.index = b.flat + (b.kind == 2 ? p.end_token : token);
        c.logit = order_of(v);
        return c;
    };
    for (int e = tid; e < fronts; e += kThreads) {
        const int l = e / depth, i = e - l * depth, j = l / p.slices;
        const Beam &b = beams[j];
        // an ended beam's one candidate is in its first list
        const int count = b.kind == 1 ? counts[l] : b.kind == 2 && l == j * p.slices ? 1 : 0;
        Candidate c = kNoCandidate;
        if (i < count) c = candidate(b, __uint_as_float((uint32_t)front[e].score), front[e].index);
        front[e] = c;
    }
    __syncthreads();
    // The n-th largest of the fronts (or, where they are many, of the maxima of
    // 256 groups of them) is a lower bound of the n-th largest candidate.
    const Candidate *items = front;
    int num_items = fronts;
    if (fronts > kThreads) {
        Candidate c = kNoCandidate;
        for (int e = tid; e < fronts; e += kThreads)
            if (better(front[e], c, p.vocab)) c = front[e];
        best[tid] = c;
        items = best;
        num_items = kThreads;
        __syncthreads();
    }
    {
        const int per = share_of(num_items), of = tid / per;
        const Candidate mine = items[min(of, num_items - 1)];
        const int rank = rank_of(items, num_items, mine, per, p.vocab);
        if (of < num_items && rank == n - 1 && mine.score != INT64_MIN) bound = mine;
    }
    __syncthreads();
    int total;
    while (true) {
        // The candidates at or above the bound, hardly more than n: those in the
        // fronts, then what lies behind a front that is all above it.
        const Candidate limit = bound;
        auto take = [&](const Candidate &c) {
            if (c.score == INT64_MIN || better(limit, c, p.vocab)) return;
            const int at = atomicAdd(&num_found, 1);
            if (at < kCap) found[at] = c;
        };
        for (int e = tid; e < fronts; e += kThreads) {
            const Candidate c = front[e];
            take(c);
            const int l = e / depth;
            if (e - l * depth == depth - 1 && c.score != INT64_MIN && !better(limit, c, p.vocab) &&
                beams[l / p.slices].kind == 1 && counts[l] > depth)
                deep[atomicAdd(&num_deep, 1)] = l;
        }
        __syncthreads();
        for (int d = tid; d < num_deep * (n - depth); d += kThreads) {
            const int l = deep[d / (n - depth)], i = depth + d % (n - depth);
            if (i >= counts[l]) continue;
            const int64_t at = (entry0 + l) * n + i;
            take(candidate(beams[l / p.slices], __ldcg(p.values + at), __ldcg(p.indices + at)));
        }
        __syncthreads();
        total = num_found;
        if (total <= kCap) break;
        for (int k = tid; k < kCap; k += kThreads) {       // as in the scan: a higher bound, again
            const Candidate mine = found[k];
            int rank = 0;
            for (int t = 0; t < kCap; ++t) rank += better(found[t], mine, p.vocab);
            if (rank == n - 1) bound = mine;
        }
        __syncthreads();
        if (tid == 0) num_found = num_deep = 0;
        __syncthreads();
    }
    const int listed = total < n ? total : n;
    const int per = share_of(total);
    for (int k0 = 0; k0 < total; k0 += kThreads / per) {
        const int k = k0 + tid / per;
        const Candidate mine = found[min(k, total - 1)];
        const int rank = rank_of(found, total, mine, per, p.vocab);
        if (k >= total || rank >= n || (tid & (per - 1)) != 0) continue;
        const int64_t o = (int64_t)g * n + rank;
        p.scores_out[o] = (float)score_of(mine.score);
        p.parents_out[o] = mine.index / p.vocab;
        p.tokens_out[o] = mine.index % p.vocab;
    }
    if (listed == n || tid != 0) return;
    // every candidate above -inf is listed: the lowest other indices fill up
    int at = listed;
    for (int f = 0; at < n; ++f) {
        bool taken = false;
        for (int k = 0; k < listed; ++k) taken |= found[k].index == f;
        if (taken) continue;
        const int64_t o = (int64_t)g * n + at++;
        p.scores_out[o] = -INFINITY;
        p.parents_out[o] = f / p.vocab;
        p.tokens_out[o] = f % p.vocab;
    }
}

// grid (slices, rows).  CLUSTER: a group's CTAs are a cluster, and its first one
// merges when all have written their records.
template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) beam_scan_kernel(const BeamParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    scan_slice<T>(p);
    if (!CLUSTER) return;
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    const int g = blockIdx.y / p.num_beams;
    if (blockIdx.x == 0 && (int)blockIdx.y == g * p.num_beams) merge_group(p, g);
}

// grid (groups): where a group has more CTAs than a cluster.
__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    merge_group(p, blockIdx.x);
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

int32_t chunks_of(int32_t vocab, int32_t vec) {
    return (int32_t)(((int64_t)vocab + (int64_t)vec * kChunk - 1) / ((int64_t)vec * kChunk));
}

// Slices of a row (the workspace is sized by it, without a device at hand).  Each is
// a list to merge, and its end costs some 3 us, so where rows give half the SMs a CTA
// each a slice has up to 16 chunks (64 x 8 rows of 128,256 fp32 logits in 2 slices a row
// 55.6 us, in one 56.8, in 8 67.6); below that 4, or a group at least 16 slices (1 x 1
// row of 32,000 bf16 in 4 slices 9.0 us, in one 10.6), but no more than 64 (1 x 64 rows
// of 128,256 fp32 in 2 slices each 21.3 us, in 8 29.3).  Either side of the border,
// 128,256 bf16 logits, 4 chunks against 16, us: 8 x 4 rows 11.6 and 14.5, 18 x 4 13.5
// and 14.9, 72 x 1 16.7 and 14.7, 9 x 8 15.7 and 16.2; 20 x 4 14.7 and 15.0, 10 x 8 17.1
// and 16.1, 24 x 4 15.0 and 15.1, 100 x 1 20.6 and 15.3, 127 x 1 25.1 and 15.9, 32 x 4
// 16.6 and 15.5, 64 x 4 25.8 and 21.7.
int32_t slices_of(int64_t rows, int32_t beams, int32_t row_chunks) {
    int32_t slices = (row_chunks + 15) / 16;
    if (rows < kHalfTheSms)
        slices = std::max({slices, kMaxCluster / beams, std::min((row_chunks + 3) / 4, kFewLists / beams)});
    return std::min({slices, std::max(kMaxLists / beams, 1), row_chunks});
}

// Front entries of each list: together 4 n or more, or the whole lists.
int32_t depth_of(int32_t lists, int32_t n) { return std::min(n, (4 * n + lists - 1) / lists); }

size_t merge_smem(int32_t beams, int32_t slices, int32_t n) {
    const int lists = beams * slices;
    return ((size_t)lists * depth_of(lists, n) + kCap) * sizeof(Candidate) +
           beams * sizeof(Beam) + 2 * (size_t)lists * sizeof(int32_t);
}

}  // namespace

// For either type: fp32's vectors, the shorter ones, make the more chunks.
size_t beam_workspace(int32_t groups, int32_t beams, int32_t vocab, int32_t num_out) {
    const int64_t rows = (int64_t)groups * beams;
    const size_t entries = (size_t)rows * slices_of(rows, beams, chunks_of(vocab, 4));
    return round_up(entries * 8) + 2 * round_up(entries * 4) + 2 * round_up(entries * num_out * 4);
}

cudaError_t launch_beam_select(const BeamArgs &a, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.num_groups * a.num_beams;
    const int32_t vec = a.bf16 ? 8 : 4;
    BeamParams p = {};
    p.logits = a.logits;
    p.row_stride = a.row_stride;
    p.beam_scores = a.beam_scores;
    p.finished = a.finished;
    p.end_token = a.end_token;
    p.num_beams = a.num_beams;
    p.vocab = a.vocab;
    p.num_out = a.num_out;
    p.row_vectors = (int32_t)(((int64_t)a.vocab + vec - 1) / vec);
    p.row_chunks = chunks_of(a.vocab, vec);
    p.slices = slices_of(rows, a.num_beams, p.row_chunks);
    // Where few CTAs have all the work, a group's are one cluster and need no second
    // launch (1 x 4 rows of 32,000 bf16 logits 9.7 us, in two kernels 10.1, and 2 us
    // less on the host).  Where they are many, clusters pack the SMs worse than single
    // CTAs do: with several slices a row much (31 x 4 rows of 128,256 bf16 logits in 4
    // slices 19.6 us, in two kernels 16.2), with one it depends (as clusters and in two
    // kernels: 32 x 4 rows 15.6 and 15.5 us, 36 x 4 17.1 and 16.5, 64 x 4 21.3 and 21.8,
    // 16 x 8 19.9 and 16.8).
    const bool cluster = a.num_beams * p.slices <= kMaxCluster && rows * p.slices <= kHalfTheSms;
    const size_t entries = (size_t)rows * p.slices;
    char *w = static_cast<char *>(a.workspace);
    p.sums = reinterpret_cast<unsigned long long *>(w);
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
    p.depth = depth_of(a.num_beams * p.slices, a.num_out);
    const auto scan = a.bf16 ? (cluster ? beam_scan_kernel<uint16_t, true> : beam_scan_kernel<uint16_t, false>)
                             : (cluster ? beam_scan_kernel<float, true> : beam_scan_kernel<float, false>);
    const size_t smem = merge_smem(a.num_beams, p.slices, a.num_out);   // (at most 34 KB: 640 lists)
    // more than the 48 KB a kernel may take unasked: a setting of the loaded kernel
    cudaError_t e = cudaFuncSetAttribute(scan, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScanSmem);
    if (e != cudaSuccess) return e;
    if (!cluster) {
        e = launch_pdl(scan, dim3(p.slices, (unsigned)rows), dim3(kThreads), stream, kScanSmem, p);
        if (e != cudaSuccess) return e;
        return launch_pdl(beam_merge_kernel, dim3(a.num_groups), dim3(kThreads), stream, smem, p);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.slices, (unsigned)rows);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kScanSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.slices;
    attr[1].val.clusterDim.y = a.num_beams;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (a.num_beams * p.slices > 8) {                      // an opt-in
        e = cudaFuncSetAttribute(scan, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, scan, p);
}

}  // namespace pa
