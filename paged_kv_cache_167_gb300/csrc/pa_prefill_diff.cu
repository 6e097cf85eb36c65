// pa_prefill_diff.cu -- differential attention of a chunk of prompt tokens against
// the paged context, on the tcgen05 tensor cores (sm_103a).
//
// The mathematics (pa_decode_diff.cuh): pair g of KV heads has keys K1, K2 and one
// value row V = [V_2g | V_2g+1] of 2d components; query pair h computes
//     x_h = softmax(s q_2h K1^T) V - lambda_h softmax(s q_2h+1 K2^T) V
// for each query j over keys 0 .. ctx + j, then (optionally) the norm of the row.
//
// Why a cluster of two CTAs: one map of a 128-row tile holds 128 x 2d fp32 sums, half
// of an SM's tensor memory at d = 128; with two score tiles beside it the other half
// is gone as well, so the two maps cannot share an SM.  CTA r of a cluster runs map r
// as an attention of its own (scores 128 x 128 x d, products 128 x 2d x 128 for each
// term of the probabilities: with values twice as wide and two terms the tensor cores
// have two and a half times the work a score that plain attention has, against one
// exponential).  The maps meet once a unit: each CTA finishes one half of the 2d
// columns, so it sends the other half of its own map, divided by the row's sum and
// weighted, to the other CTA: 64 KB of fp32 (the difference and the norm lose nothing
// before the one rounding to bf16), stored asynchronously into the unit's last two value
// slots there, which nothing reads any more; the bytes themselves complete the receiver's
// barrier.  That takes some 4,500 cycles (15 bytes a cycle; nothing but such stores
// reaches 19, bulk copies 15), the norm's sums and the output another 5,000, against 2,000
// for each of the unit's tiles with one term.  (With one term, the halves staged and sent
// as bulk copies: 61.3 us instead of 58.7 for 2,048 tokens; cut to 24 bits a value: 57.5,
// too little for a rounding more.)
//
// A probability enters P.V as two bf16 terms, its rounding and what that left, as in decode
// and for its reason: what the difference takes out of two maps that are alike leaves the
// roundings of both, and the norm scales them up.  Off from the definition on average, maps
// correlated by 0, 0.99 or 0.999, lambda 0.8 or 1, 40 to 2,048 keys: 0.0017 of the output,
// what rounding the output costs.  With PA_DIFF_ONE_TERM a probability is rounded once, by up
// to 2^-8 of it: 0.0020 to 0.0022, 0.0045 to 0.0104 and 0.0052 to 0.0315, for two thirds of
// the time.
//
// What bounds it: the tensor pipe.  GB300, by graph replay: 16 x (4,096 + 512) tokens of 64/8
// heads, d = 128: 1.64 to 1.71 ms, 1.02 to 1.07 PFLOP/s of the definition's 6d a key and query
// head (with the second term's 4d: 1.71 to 1.78, 0.91 to 0.95 of the measured bf16 rate in a
// burst, all of the sustained one); with one term 1.08 to 1.11 ms (1.58 to 1.63 PFLOP/s).  2,048
// tokens from the start (32/8 heads) 74 to 77 us, 57 to 63 with one term: a cluster has three
// or four units, and their ends weigh more.  5 x 333 tokens at up to 3,000 (16/8 heads, d = 64)
// 44 to 68 us by their lengths, 39 to 59 with one term: 120 units dealt to 76 clusters by
// number, so the busiest has 1.6 times the mean's tiles.
//
// Design, as far as it is not pa_prefill.cu's:
//  * A unit is an M-tile of 128 rows (query j0 + r / G, pair r % G of the G query
//    pairs that share their keys), one KV pair and one sequence; the grid is
//    persistent, clusters walking units in rounds of alternating direction.
//  * Rows' keys belong to two threads of different warps (32 of each half of the tile
//    each), which share one accumulator, so they agree on the reference maximum.  A
//    tile's first probabilities are made with the reference as it is, while each finds its
//    maximum; a barrier of the two warps then says whether any row exceeds it by more than
//    8 (log2), and only then do the maxima meet and the tile start over, from its scores in
//    tensor memory (the probabilities have taken their registers).  P.V of a half of
//    the keys starts when that half's probabilities are there.
//  * Shared memory (d = 128): one query tile 32 KB, two key tiles 64 KB, four half value
//    tiles of 64 keys 128 KB.  The query tile is free once a unit's last scores are there,
//    so the next unit's is copied under the last products; the warp that copies values
//    stores a unit's output from its value slots before it fills them again.
//  * Both maps multiply the same values, and each CTA copies all of them for itself (96 KB a
//    tile and CTA from L2; neighbouring clusters' tiles share them there).
//  * The copying and issuing warps run few instructions a tile, all lanes together: with
//    every descriptor put together anew by one lane, two copies a block of keys and waits
//    that acquired at cluster scope, those warps, not the tensor pipe, made the tile
//    (2,400 cycles, 1.40 ms a call).
//  * All waits are bounded, and both CTAs meet at the end before either's shared memory
//    goes.
#include <algorithm>
#include <type_traits>

#include "pa_prefill_common.cuh"

namespace pa {
namespace prefill {
namespace {

struct DiffParams {
    __nv_bfloat16 *out;          // [B][C][pairs][2 DH]
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *ctx_lens;
    int32_t max_ctx_len;
    int32_t chunk;
    int32_t num_pairs;           // query pairs of a token
    int64_t num_blocks;
    float scale_log2;
    unsigned int *err;
    int32_t num_mt;              // M-tiles per sequence
    int32_t num_kv;              // groups of G query pairs
    int32_t num_seqs;
    int32_t by_length;           // units in the order of their tiles, not of their keys
    int32_t by_head;             // group u reads key head u for both maps, values of pair u / 2
    const float *lambda;         // [pairs]
    const float *norm_weight;    // [2 DH] or nullptr
    float eps, out_scale;
};

template <int DH>
struct DiffSmem {
    static constexpr int kHalves = DH / 64;                      // 64-wide halves of a head
    static constexpr uint32_t kQTile = kHalves * kHalf;          // [half][128 rows][128 B]
    static constexpr uint32_t kKTile = kHalves * kHalf;          // [8 keys][half][8 keys][128 B]: see the map
    static constexpr uint32_t kVHalf = 64u * 2u * DH * 2u;       // 64 keys: [block][head][half][BS][128 B]
    static constexpr int kVSlots = 4;
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffK = kOffQ + kQTile;
    static constexpr uint32_t kOffV = kOffK + 2 * kKTile;
    static constexpr uint32_t kOffX = kOffV + kVSlots * kVHalf;  // float [2][2][128]: see mx
    static constexpr uint32_t kOffBar = kOffX + 2048;
    static constexpr uint32_t kOffW = kOffBar + 384;             // float [DH]: this CTA's half of the norm's weights
    static constexpr uint32_t kBytes = kOffW + DH * 4;
    static_assert(kBytes <= 232448, "shared memory");
};

// ---- cluster ------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The other CTA's address of this CTA's shared-memory address.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
// Stores to the other CTA's shared memory that complete their bytes on its barrier.
__device__ __forceinline__ void store_async(uint32_t addr, float4 v, uint32_t bar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
        "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
        : "memory");
}
// Arrives, once this thread's MMAs so far have completed, on the barrier at this offset
// in the other CTA as well.
__device__ __forceinline__ void umma_commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}
// A matrix descriptor that lies `bytes` behind another.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (uint64_t)(bytes >> 4); }

// Waits for a barrier that the other CTA's threads, stores or MMAs complete: its acquire is
// at cluster scope, which orders what that CTA did before (its reads of slots that are
// stored to or filled next, the data it stored here) before what this thread does now.  The
// waits within a CTA, several a tile, acquire at its own scope.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, unsigned int *err) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            raise_error(err, PA_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Named barriers whose threads all learn whether any of them saw `mine`: the two warps
// of the same rows, and all softmax warps.  A warp that gives up alone would leave the
// others waiting for it, and these barriers have no limit; so giving up is decided
// here, by everyone alike.
__device__ __forceinline__ bool barrier_or(int id, int threads, bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)mine), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ bool part_or(int warp, bool mine) { return barrier_or(1 + (warp & 3), kParts * 32, mine); }
__device__ __forceinline__ bool soft_or(bool mine) { return barrier_or(5, kSoftWarps * 32, mine); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : PA_R8(0), PA_R8(8)
        : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 32) tmem_ld32(taddr, r);
    else tmem_ld16(taddr, r);
}

__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// ---- the kernel -----------------------------------------------------------------

// Barriers, as in pa_prefill.cu unless noted: Q landed, K landed[2], V half landed[4],
// S ready[2] (a K slot is free with it), P ready[2][half of the keys], P.V done[2] (a S
// buffer is free with it), V half free[4], Q free, unit's P.V done (in both CTAs: two
// arrivals), O read, the two MMA lanes' drains; then full[8] (the other CTA's data for a warp
// has landed), norm[4] (its partial sums of squares of a lane quadrant's rows), out[2] (a
// unit's output is staged in its last value slots, or written: by unit parity).
// The tiles of the CTA's units are numbered T = 0, 1, ...; its value halves H = 2T, 2T + 1.
template <int DH, int G, int BS, int TERMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefill_diff_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o,
                        const DiffParams p) {
    using SM = DiffSmem<DH>;
    constexpr int QPT = kRows / G;                 // queries per M-tile
    constexpr int DV = 2 * DH;                     // value components
    constexpr int NBK = kKeys / BS;                // blocks of a key tile
    constexpr int NBV = 64 / BS;                   // blocks of half a value tile
    constexpr int kVS = SM::kVSlots;
    constexpr uint32_t kVBlock = (uint32_t)(DV / 64) * BS * 128u;   // one block's V box
    constexpr uint32_t kTmem = 512;                // S0, S1, O
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t base = smem_addr(smem_raw);
    const uint32_t sQ = base + SM::kOffQ, sK = base + SM::kOffK, sV = base + SM::kOffV;
    const uint32_t barQ = base + SM::kOffBar, barK = barQ + 8, barV = barK + 16, barS = barV + 8 * kVS,
                   barP = barS + 16, barOP = barP + 32, barVfree = barOP + 16, barQfree = barVfree + 8 * kVS,
                   barUnit = barQfree + 8, barOfree = barUnit + 8, barEnd = barOfree + 8, barEndQk = barEnd + 8,
                   barFull = barEndQk + 8, barNorm = barFull + 64, barOut = barNorm + 32;
    constexpr int kNumBars = 1 + 2 + kVS + 2 + 4 + 2 + kVS + 1 + 1 + 1 + 1 + 1 + 8 + 4 + 2;
    static_assert(8 * kNumBars + 8 <= 384, "barrier area");
    static_assert(kVS == 4, "two tiles of value halves");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + SM::kOffBar + 8 * kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem_raw + SM::kOffBar + 8 * kNumBars + 4);
    // The halves' maxima of a tile ([tile parity][half][row]), in the epilogue their
    // sums, then the four partial sums of squares of a row ([2 * CTA + half][row]).
    float *mx = reinterpret_cast<float *>(smem_raw + SM::kOffX);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the same in every lane, and known to be
    const uint32_t rank = cluster_rank();

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const uint32_t b = barQ + 8 * i;
            uint32_t count = 1;
            if ((b >= barP && b < barOP) || b == barOfree || b >= barOut) count = kSoftWarps * 32;
            if (b == barUnit) count = 2;                     // both CTAs' P.V lanes
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(count) : "memory");
        }
        // the tiles' swizzle wants 1,024-byte alignment, which dynamic shared memory
        // has where nothing static lies before it; checked, not assumed
        *abort_flag = (base & 1023u) != 0 ? 1 : 0;
        if ((base & 1023u) != 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();        // both CTAs' barriers are set up before either arrives on the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tO = tmem + 256;
    const bool usable = *abort_flag == 0;
    float *weights = reinterpret_cast<float *>(smem_raw + SM::kOffW);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid < DH) weights[tid] = p.norm_weight ? __ldg(p.norm_weight + rank * DH + tid) : 1.f;
    __syncthreads();

    // ---- this cluster's units
    const int C = (int)gridDim.x / 2, cl = (int)blockIdx.x / 2;
    const int per_mt = p.num_kv * p.num_seqs;
    const int n_units = usable ? p.num_mt * per_mt : 0;
    auto unit_index = [&](int k) { return k * C + ((k & 1) ? C - 1 - cl : cl); };
    const int rounds = (n_units + C - 1) / C;
    const int my_units = rounds > 0 ? rounds - 1 + (unit_index(rounds - 1) < n_units ? 1 : 0) : 0;
    struct Unit {
        int s, g, j0, ctx, seq_end, nblk, n_tiles;
    };
    auto unit = [&](int k) {
        Unit U;
        const int u = unit_index(k);
        const int mt = p.by_length ? u / per_mt : u % p.num_mt, gs = p.by_length ? u % per_mt : u / p.num_mt;
        U.g = gs % p.num_kv;
        U.s = gs / p.num_kv;
        U.j0 = (p.num_mt - 1 - mt) * QPT;     // the longest rows first
        int ctx = __ldg(p.ctx_lens + U.s);
        if (ctx < 0 || ctx > p.max_ctx_len) {
            raise_error(p.err, PA_DEVERR_SEQ_LEN);
            ctx = ctx < 0 ? 0 : p.max_ctx_len;
        }
        U.ctx = ctx;
        U.seq_end = ctx + p.chunk;
        U.nblk = (U.seq_end + BS - 1) / BS;
        const int last_q = min(U.j0 + QPT, p.chunk) - 1;
        U.n_tiles = (ctx + last_q + 1 + kKeys - 1) / kKeys;    // at least one
        return U;
    };
    constexpr uint32_t idesc_qk = idesc_bf16(kRows, kKeys, false);
    constexpr uint32_t idesc_pv = idesc_bf16(kRows, DV, true);

    if (warp == kKWarp || warp == kVWarp) {
        // ---- copy warps: a lane per box, block ids in registers a load of 32 ahead.  The
        // K warp copies tiles of NBK blocks, the V warp halves of NBV.
        auto copy = [&](auto which) {
            constexpr bool is_k = decltype(which)::value;
            constexpr int nb = is_k ? NBK : NBV, per_tile = is_k ? 1 : 2, spl = 32 / nb, slots = is_k ? 2 : kVS;
            const uint32_t bar0 = is_k ? barK : barV, free0 = is_k ? barS : barVfree;
            auto ids_load = [&](const Unit &U, int c) -> int {
                const int bi = c * 32 + lane;
                return bi < U.nblk && bi < U.n_tiles * NBK ? __ldg(p.tables + (size_t)U.s * p.max_blocks + bi) : 0;
            };
            auto ids_check = [&](int v, const Unit &U, int c) -> int {   // out-of-bounds coordinate: zero fill
                const int bi = c * 32 + lane;
                if (!(bi < U.nblk && bi < U.n_tiles * NBK)) return (int)p.num_blocks;
                if (v < 0 || v >= p.num_blocks) {
                    raise_error(p.err, PA_DEVERR_BLOCK_ID);
                    return (int)p.num_blocks;
                }
                return v;
            };
            // Unit x's output, from its value slot to memory; then the unit's value slots are free
            // for copies again: what the other CTA stored in them has been read before the output
            // was staged (V warp; every unit once, in order: two barriers by parity, so that none is
            // lapped).
            int out_slot[2] = {0, 0};
            auto store_out = [&](int x) -> bool {
                const uint32_t parity = (uint32_t)((x >> 1) & 1);
                const bool done = __all_sync(0xffffffffu, mbar_wait(barOut + 8 * (x & 1), parity, p.err));
                const Unit Y = unit(x);
                if (done && Y.j0 + min(QPT, p.chunk) <= p.chunk) {
                    if (lane == 0) {
                        const uint32_t src = sV + (uint32_t)(x & 1 ? out_slot[1] : out_slot[0]) * SM::kVHalf;
#pragma unroll
                        for (int h = 0; h < SM::kHalves; ++h)
                            tma_store_4d(&tmap_o, (int)rank * DH + h * 64, 0, Y.g, Y.s * p.chunk + Y.j0,
                                         src + h * kHalf);
                        bulk_commit();
                        bulk_wait_read();
                    }
                    __syncwarp();
                }
                return done;
            };
            bool ok = true;
            int N = 0;      // tiles or halves issued so far
            int nq = 0;     // query tiles issued (K warp)
            int prev_steps = 0;
            Unit U;
            int raw_cur = 0, raw_next = 0;
            if (my_units > 0) {
                U = unit(0);
                raw_cur = ids_load(U, 0);
                raw_next = ids_load(U, 1);
            }
            for (int k = 0; k < my_units && ok; ++k) {
                Unit X = U;            // the next unit, and its first ids
                int nraw_cur = 0, nraw_next = 0;
                if (k + 1 < my_units) {
                    X = unit(k + 1);
                    nraw_cur = ids_load(X, 0);
                    nraw_next = ids_load(X, 1);
                }
                if (is_k) {
                    if (k > 0)     // the previous unit's Q.K have all read the query tile
                        ok = __all_sync(0xffffffffu, mbar_wait(barQfree, (uint32_t)((k - 1) & 1), p.err));
                    if (!ok) {
                        *abort_flag = 1;
                        break;
                    }
                    nq = k + 1;
                    if (lane == 0) mbar_expect(barQ, SM::kQTile);
                    __syncwarp();
                    if (lane < SM::kHalves)
                        tma_load_5d(sQ + lane * kHalf, &tmap_q, lane * 64, (int)rank, 0, U.g, U.s * p.chunk + U.j0,
                                    barQ);
                }
                const int key_head = p.by_head ? U.g : 2 * U.g + (int)rank;
                const int value_head = p.by_head ? (U.g >> 1) * 2 : 2 * U.g;
                int ids_cur = ids_check(raw_cur, U, 0);
                const int steps = U.n_tiles * per_tile;
                for (int t = 0; t < steps; ++t, ++N) {
                    if (t > 0 && t % spl == 0) {
                        ids_cur = ids_check(raw_next, U, t / spl);
                        raw_next = ids_load(U, t / spl + 1);
                    }
                    const int tb = (t % spl) * nb, st = N % slots;
                    const int blk = __shfl_sync(0xffffffffu, ids_cur, (tb + lane) & 31);
                    if (N >= slots) {   // the slot's previous tile has been consumed by its MMAs
                        const int np = N - slots;
                        const uint32_t bar = free0 + 8 * (np % slots), parity = (uint32_t)((np / slots) & 1);
                        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err));
                        if (!ok) {
                            *abort_flag = 1;
                            break;
                        }
                    }
                    // A unit's last two value slots also hold its exchange and its output, and are
                    // next filled four halves on: from this unit's third half on, or, behind a unit
                    // of two halves, from the first of the unit after.
                    if (!is_k) {
                        const int x = t == 2 ? k - 1 : t == 0 && prev_steps == 2 ? k - 2 : -1;
                        if (x >= 0 && !store_out(x)) {
                            ok = false;
                            *abort_flag = 1;
                            break;
                        }
                    }
                    if (lane == 0) mbar_expect(bar0 + 8 * st, is_k ? SM::kKTile : SM::kVHalf);
                    __syncwarp();
                    if (is_k) {
                        if (lane < NBK)
                            tma_load_5d(sK + st * SM::kKTile + lane * (uint32_t)(BS * DH * 2), &tmap_k, 0, 0, 0,
                                        key_head * (BS / 8), blk, bar0 + 8 * st);
                    } else if (lane < NBV) {
                        tma_load_5d(sV + st * SM::kVHalf + lane * kVBlock, &tmap_v, 0, 0, 0, value_head, blk,
                                    bar0 + 8 * st);
                    }
                }
                prev_steps = steps;
                if (k & 1) out_slot[1] = (N + kVS - 2) % kVS;     // where this unit's output will be staged
                else out_slot[0] = (N + kVS - 2) % kVS;
                U = X;
                raw_cur = nraw_cur;
                raw_next = nraw_next;
            }
            if (!is_k) {    // the outputs no later half waited for
                for (int x = max(0, my_units - (prev_steps == 2 ? 2 : 1)); x < my_units && ok && !*abort_flag; ++x)
                    ok = store_out(x);
                if (lane == 0) bulk_wait_all();   // no store in flight when the CTA ends
            }
            if (!ok || *abort_flag) {
                // wait (bounded) for this warp's copies still in flight before the memory is released
                for (int t = max(0, N - slots); t < N; ++t)
                    mbar_wait(bar0 + 8 * (t % slots), (uint32_t)((t / slots) & 1), p.err);
                if (nq > 0) mbar_wait(barQ, (uint32_t)((nq - 1) & 1), p.err);
            }
            __syncwarp();
        };
        if (warp == kKWarp) copy(std::true_type());
        else copy(std::false_type());
    } else if (warp == kMmaWarp || warp == kQkWarp) {
        // ---- two issuing warps, as in pa_prefill.cu.  The whole warp walks the tiles and one
        // lane issues, from descriptors that differ by an addition: issued by one lane on its
        // own, with every descriptor put together anew, a tile's sixteen products and their
        // waits took as long as the products themselves.
        const bool is_qk = warp == kQkWarp;
        const bool leader = elect_one();
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err));
            return ok;
        };
        const uint64_t dQ = smem_desc(sQ, 16, 1024), dK = smem_desc(sK, 16, SM::kHalves * 1024);
        const uint64_t dV = smem_desc(sV, BS * 128, BS >= 16 ? 1024 : kVBlock);
        int T = 0;
        for (int k = 0; k < my_units && ok && !*abort_flag; ++k) {
            const int n_tiles = unit(k).n_tiles;
            if (is_qk) {
                if (!wait(barQ, (uint32_t)(k & 1))) break;
                for (int t = 0; t < n_tiles; ++t, ++T) {
                    const int st = T & 1;      // K slot and S buffer
                    const uint32_t ph = (uint32_t)((T >> 1) & 1);
                    if (!wait(barK + 8 * st, ph)) break;
                    // S buffer st held P(T - 2): its P.V must have completed
                    if (T >= 2 && !wait(barOP + 8 * st, ph ^ 1u)) break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t dk = desc_at(dK, st * SM::kKTile);
                        const uint32_t dst = tmem + st * 128;
#pragma unroll
                        for (int kk = 0; kk < DH / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                            const uint32_t k_off = (kk >> 2) * 1024 + (kk & 3) * 32;
                            umma(dst, desc_at(dQ, off), desc_at(dk, k_off), idesc_qk, kk > 0);
                        }
                        umma_commit(barS + 8 * st);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (leader) umma_commit(barQfree);
            } else {
                // O is overwritten by this unit's first P.V: the previous unit's epilogue has read it
                if (k > 0 && !wait(barOfree, (uint32_t)((k - 1) & 1))) break;
                for (int t = 0; t < n_tiles && ok; ++t, ++T) {
                    const int sb = T & 1;
                    const uint32_t ph = (uint32_t)((T >> 1) & 1);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int st = (2 * T + hf) & (kVS - 1);
                        if (!wait(barV + 8 * st, ph)) break;     // half 2T + hf, four slots: (2T + hf) / 4 = T / 2
                        if (!wait(barP + 16 * sb + 8 * hf, ph)) break;
                        tc_fence_after();
                        if (leader) {
                            const uint64_t dv = desc_at(dV, st * SM::kVHalf);
                            const uint32_t tP = tmem + sb * 128 + hf * 64;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                // 16 keys: within one block for b >= 16 (8-key groups 1024 B apart), or
                                // two whole blocks for b = 8 (groups one block apart).  P of 32 keys
                                // lies in 16 columns, the first half of those its scores had.
                                const uint32_t v_off =
                                    (uint32_t)(kk * 16 / BS) * kVBlock + (uint32_t)((kk * 16) % BS) * 128u;
                                const uint32_t a = tP + (kk >> 1) * 32 + (kk & 1) * 8;
                                umma_ts(tO, a, desc_at(dv, v_off), idesc_pv, (t > 0 || hf > 0 || kk > 0) ? 1u : 0u);
                                if (TERMS == 2) umma_ts(tO, a + 16, desc_at(dv, v_off), idesc_pv, 1u);
                            }
                            umma_commit(barVfree + 8 * st);
                            if (hf == 1) umma_commit(barOP + 8 * sb);
                        }
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if (leader) umma_commit_both(barUnit);   // every P.V of the unit has completed, in this CTA
            }
        }
        // one more commit, on a barrier used once, tracks every MMA this warp issued
        if (!ok) *abort_flag = 1;   // give up: drain what was issued
        const uint32_t end = is_qk ? barEndQk : barEnd;
        if (leader) umma_commit(end);
        __syncwarp();
        mbar_wait(end, 0, p.err);
        __syncwarp();
    } else {
        // ---- softmax warps: row r, key half pt (scale_log2 > 0: maxima of raw scores)
        const int r = (warp & 3) * 32 + lane, pt = warp >> 2;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const float c = p.scale_log2;
        const uint32_t other = rank ^ 1u;
        int T = 0;
        for (int k = 0; k < my_units; ++k) {
            const Unit U = unit(k);
            const int jr = U.j0 + r / G;
            const int pos = min(U.ctx + jr, U.seq_end - 1);   // last key this row may attend
            const int pair = U.g * G + r % G;
            const float lam = rank == 0 ? 1.f : -__ldg(p.lambda + pair);
            float m_ref = -INFINITY;                          // reference maximum, log2 domain
            float l = 0.f;                                    // of this thread's keys
            int done = 0;
            for (int t = 0; t < U.n_tiles; ++t, ++T) {
                const int sb = T & 1;
                bool ok = mbar_wait(barS + 8 * sb, (uint32_t)((T >> 1) & 1), p.err);
                // this thread's keys: 32 of the tile's first half, 32 of its second
                uint32_t sr[2][32];
                const uint32_t tS = tmem + sb * 128 + lane_off + pt * 32;
                if (__all_sync(0xffffffffu, ok)) {
                    tc_fence_after();
                    tmem_ld32(tS, sr[0]);
                    tmem_ld32(tS + 64, sr[1]);
                    tmem_ld_wait();
                } else {
                    ok = false;
                }
                const int key0 = t * kKeys + pt * 32;
                const bool edge = !__all_sync(0xffffffffu, key0 + 64 + 31 <= pos);   // some row's causal edge
                auto hide = [&](int cc) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (key0 + cc * 64 + i > pos) sr[cc][i] = __float_as_uint(-INFINITY);
                };
                if (edge) {
                    hide(0);
                    hide(1);
                }
                const float2 c2 = make_float2(c, c);
                float2 ps2 = make_float2(0.f, 0.f), ps2b = make_float2(0.f, 0.f);
                auto probabilities = [&](int cc) {   // of half cc, in its scores' place, and their sums
                    const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
                    const float2 nm2 = make_float2(nm, nm);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = __ffma2_rn(
                            make_float2(__uint_as_float(sr[cc][2 * e]), __uint_as_float(sr[cc][2 * e + 1])), c2, nm2);
                        const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        if (e & 1) ps2b = __fadd2_rn(ps2b, pe);
                        else ps2 = __fadd2_rn(ps2, pe);
                        sr[cc][2 * e] = __float_as_uint(pe.x);
                        sr[cc][2 * e + 1] = __float_as_uint(pe.y);
                    }
                };
                // The first half's probabilities by the reference as it is, while the maximum is
                // found; a barrier of the row's two warps then says whether any of their rows
                // exceeds it by more than the threshold.  Rarely (and with the first tile): both
                // threads of a row take the larger of their maxima and start over.
                const float mine = max_tree64(sr[0], sr[1]);
                const float mine_l = mine * c;
                const bool trouble = !ok || *abort_flag;
                bool give_up = false;
                float alpha = 1.f;
#pragma unroll 1
                for (bool first = true;; first = false) {
                    ps2 = ps2b = make_float2(0.f, 0.f);
                    if (!first) {      // the scores once more
                        tmem_ld32(tS, sr[0]);
                        tmem_ld_wait();
                        if (edge) hide(0);
                    }
                    probabilities(0);
                    if (!first || !part_or(warp, trouble || mine_l > m_ref + kRescaleThreshold ||
                                                     (m_ref == -INFINITY && mine_l != -INFINITY)))
                        break;
                    mx[(sb * 2 + pt) * 128 + r] = mine_l;
                    if (part_or(warp, trouble)) {
                        give_up = true;
                        break;
                    }
                    const float mt_ = fmaxf(mine_l, mx[(sb * 2 + (pt ^ 1)) * 128 + r]);
                    if (mt_ > m_ref + kRescaleThreshold || (m_ref == -INFINITY && mt_ != -INFINITY)) {
                        alpha = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - mt_);
                        m_ref = mt_;
                    }
                    // rescale this thread's half of the accumulator's columns once P.V(T - 1) has
                    // completed (its barrier's previous phase, P.V(T - 3), completed before
                    // Q.K(T - 1) was issued, which S(T - 1), read before this tile, needed)
                    if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        const int tp = T - 1;
                        mbar_wait(barOP + 8 * (tp & 1), (uint32_t)((tp >> 1) & 1), p.err);
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < DH / 32; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(tO + pt * DH + lane_off + cc * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(tO + pt * DH + lane_off + cc * 32, o);
                        }
                        tmem_st_wait();
                    }
                }
                if (give_up) {
                    *abort_flag = 1;
                    mbar_arrive_u32(barP + 16 * sb);   // keep the arrival counts balanced
                    mbar_arrive_u32(barP + 16 * sb + 8);
                    break;
                }
                const int tail_lo = U.seq_end - t * kKeys;
                const bool zero_tail = tail_lo > 0 && tail_lo < kKeys && (U.seq_end % BS) != 0;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    // P into the columns its scores were read from: hi = bf16(p) into the first
                    // half of them, lo = bf16(p - hi) into the second
                    if (hf == 1) probabilities(1);
                    uint32_t pw[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pw[e] = pack_bf16x2(__uint_as_float(sr[hf][2 * e]), __uint_as_float(sr[hf][2 * e + 1]));
                    tmem_st16(tS + hf * 64, pw);
                    if (TERMS == 2) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float lo0 = __uint_as_float(sr[hf][2 * e]) - __uint_as_float(pw[e] << 16);
                            const float lo1 = __uint_as_float(sr[hf][2 * e + 1]) - __uint_as_float(pw[e] & 0xffff0000u);
                            pw[e] = pack_bf16x2(lo0, lo1);
                        }
                        tmem_st16(tS + hf * 64 + 16, pw);
                    }
                    tmem_st_wait();
                    // Keys past the sequence end inside its last block: zero their V rows (their p
                    // is 0, but the slots may hold non-finite junk).  P.V(T - 1) is waited for
                    // first, so that the wait for the half's copy is exact: every half before tile
                    // T has then landed, and P.V of this one waits for the arrival below.
                    if (zero_tail && tail_lo / 64 == hf) {
                        if (T > 0) {
                            const int tp = T - 1;
                            mbar_wait(barOP + 8 * (tp & 1), (uint32_t)((tp >> 1) & 1), p.err);
                        }
                        const int H = 2 * T + hf, sv = H % kVS;
                        mbar_wait(barV + 8 * sv, (uint32_t)((H / kVS) & 1), p.err);
                        const int lo = tail_lo % 64, nrows = BS - U.seq_end % BS;   // to the block's end
                        constexpr int kChunks = DV / 8;                             // 16-byte chunks of a row
                        for (int idx = tid; idx < nrows * kChunks; idx += kSoftWarps * 32) {
                            const int rr = lo + idx / kChunks, c16 = idx % kChunks;
                            const uint32_t addr = sV + sv * SM::kVHalf + (uint32_t)(rr / BS) * kVBlock +
                                                  (uint32_t)(c16 / 8) * (BS * 128u) + (uint32_t)(rr % BS) * 128u +
                                                  (uint32_t)(c16 % 8) * 16u;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    tc_fence_before();
                    mbar_arrive_u32(barP + 16 * sb + 8 * hf);
                }
                ps2 = __fadd2_rn(ps2, ps2b);
                l = l * alpha + (ps2.x + ps2.y);
                done = t + 1;
            }
            // ---- epilogue.  The row's sum over both halves (the reference is one); -1: gave up
            const bool fin = done == U.n_tiles && !*abort_flag && mbar_wait_cluster(barUnit, (uint32_t)(k & 1), p.err);
            float *lx = mx + (T & 1) * 256;           // the parity that the last tile did not use
            lx[pt * 128 + r] = fin ? l : -1.f;
            part_sync(warp);
            const float lo = lx[(pt ^ 1) * 128 + r];
            part_sync(warp);                          // read, before squares are written there
            bool ok = __all_sync(0xffffffffu, fin && lo != -1.f);   // the partner warp finds the same
            const float lt = l + lo;
            const float f = lt > 0.f ? lam / lt : 0.f;
            tc_fence_after();
            // ---- the maps meet: x = this CTA's half of the columns (its product rounded as the
            // other's is: contracted with the sum, equal maps would not cancel).  Both CTAs' P.V of the unit
            // have completed, so its last two value slots are free in both (a quarter of 2d each).
            const uint32_t out_off = SM::kOffV + (uint32_t)((2 * T - 2) % kVS) * SM::kVHalf;
            const uint32_t sX = base + out_off;
            const uint32_t sY = sV + (uint32_t)((2 * T - 1) % kVS) * SM::kVHalf;
            const uint32_t my_off = (uint32_t)(pt * (DH / 16) * 128 + r) * 16u;   // chunk i: + i * 2048
            constexpr int W = DH / 4;                 // columns of a thread and quarter
            const uint32_t my_full = barFull + 8 * warp, my_norm = barNorm + 8 * (warp & 3);
            float x[2][W], ss = 0.f;
            if (ok) {
                if (lane == 0) mbar_expect(my_full, 2 * 32 * W * 4);
                if (lane == 0 && pt == 0 && p.norm_weight != nullptr) mbar_expect(my_norm, 2 * 32 * 4);
                __syncwarp();
                const uint32_t peer_full = peer_addr(my_full, other);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t dst = peer_addr((q == 0 ? sX : sY) + my_off, other);
                    uint32_t o[W];
                    tmem_ld<W>(tO + lane_off + other * DH + q * (DH / 2) + pt * W, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < W / 4; ++i)
                        store_async(dst + i * 2048u,
                                    make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                                __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f),
                                    peer_full);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t o[W];
                    tmem_ld<W>(tO + lane_off + rank * DH + q * (DH / 2) + pt * W, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < W; ++i) x[q][i] = __fmul_rn(__uint_as_float(o[i]), f);
                }
            }
            // O has been read: the next unit's first P.V may overwrite it
            tc_fence_before();
            mbar_arrive_u32(barOfree);
            if (ok) ok = mbar_wait_cluster(my_full, (uint32_t)(k & 1), p.err);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < W / 4; ++i) {
                        const float4 v = lds_f4((q == 0 ? sX : sY) + my_off + i * 2048u);
                        x[q][4 * i] += v.x;
                        x[q][4 * i + 1] += v.y;
                        x[q][4 * i + 2] += v.z;
                        x[q][4 * i + 3] += v.w;
                    }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};   // four chains, not one as long as the row
#pragma unroll
                    for (int i = 0; i < W; ++i) s4[i & 3] += x[q][i] * x[q][i];
                    ss += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                }
            }
            float scale = p.out_scale;
            if (p.norm_weight != nullptr) {
                const int at = (int)(2 * rank) + pt;
                mx[at * 128 + r] = ss;
                float4 four;      // lane i < 8 sends those of the warp's rows 4 i .. 4 i + 3
                four.x = __shfl_sync(0xffffffffu, ss, (lane & 7) * 4);
                four.y = __shfl_sync(0xffffffffu, ss, (lane & 7) * 4 + 1);
                four.z = __shfl_sync(0xffffffffu, ss, (lane & 7) * 4 + 2);
                four.w = __shfl_sync(0xffffffffu, ss, (lane & 7) * 4 + 3);
                if (ok && lane < 8)
                    store_async(peer_addr(smem_addr(mx + at * 128 + (warp & 3) * 32 + lane * 4), other), four,
                                peer_addr(my_norm, other));
                ok = !part_or(warp, !ok) && mbar_wait_cluster(my_norm, (uint32_t)(k & 1), p.err);
                ss = (mx[r] + mx[128 + r]) + (mx[256 + r] + mx[384 + r]);
                scale *= rsqrtf(ss * (1.f / DV) + p.eps);
            }
            // every softmax thread has read the exchanged halves, sums and squares
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (soft_or(!ok)) {
                *abort_flag = 1;
                break;
            }
            // ---- this CTA's half of the row: staged for a tensor store, or written straight
            const bool tma_out = U.j0 + min(QPT, p.chunk) <= p.chunk;
            const bool row_ok = jr < p.chunk;
            __nv_bfloat16 *dst =
                p.out + (((size_t)U.s * p.chunk + jr) * p.num_pairs + pair) * DV + rank * DH;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c0 = q * (DH / 2) + pt * W;     // first column within the CTA's half
#pragma unroll
                for (int i8 = 0; i8 < W / 8; ++i8) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = x[q][i8 * 8 + e] * scale;
                    const float4 *w4 = reinterpret_cast<const float4 *>(weights + c0 + i8 * 8);
                    const float4 wa = w4[0], wb = w4[1];
                    y[0] *= wa.x;
                    y[1] *= wa.y;
                    y[2] *= wa.z;
                    y[3] *= wa.w;
                    y[4] *= wb.x;
                    y[5] *= wb.y;
                    y[6] *= wb.z;
                    y[7] *= wb.w;
                    uint4 v;
                    v.x = pack_bf16x2(y[0], y[1]);
                    v.y = pack_bf16x2(y[2], y[3]);
                    v.z = pack_bf16x2(y[4], y[5]);
                    v.w = pack_bf16x2(y[6], y[7]);
                    const int col = c0 + i8 * 8;
                    if (tma_out) {
                        // 16-byte chunk j of a 128-byte line goes to chunk j ^ (r % 8): the swizzle
                        // that the tensor store undoes
                        const uint32_t line = out_off + (uint32_t)(col / 64) * kHalf + (uint32_t)r * 128u;
                        const uint32_t c16 = (uint32_t)(col % 64) / 8;
                        *reinterpret_cast<uint4 *>(smem_raw + line + ((c16 ^ ((uint32_t)r & 7u)) << 4)) = v;
                    } else if (row_ok) {
                        *reinterpret_cast<uint4 *>(dst + col) = v;
                    }
                }
            }
            // staged (or written): the V warp may store it, and fill the slots again
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive_u32(barOut + 8 * (k & 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();        // the other CTA may still write to this one's shared memory until here
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

// ---- host side --------------------------------------------------------------------

template <int DH, int G, int BS, int TERMS>
cudaError_t launch_kernel(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const CUtensorMap &mo,
                          const DiffParams &prm, cudaStream_t stream) {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !configured[dev]) {
        cudaError_t e = cudaFuncSetAttribute(prefill_diff_kernel<DH, G, BS, TERMS>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DiffSmem<DH>::kBytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const int64_t n_units = (int64_t)prm.num_mt * prm.num_kv * prm.num_seqs;
    if (n_units == 0) return cudaSuccess;
    if (n_units > INT32_MAX / 2) return cudaErrorInvalidValue;
    int64_t clusters = prefill_ctas() / 2;
    if (prefill_ctas() == 1) clusters = 1;
    if (clusters <= 0) clusters = device_sm_count() / 2;
    if (clusters <= 0) return cudaErrorUnknown;
    clusters = std::min(clusters, n_units);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = DiffSmem<DH>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_diff_kernel<DH, G, BS, TERMS>, mq, mk, mv, mo, prm);
}

template <int DH, int G, int BS>
cudaError_t launch_terms(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const CUtensorMap &mo,
                         const DiffParams &prm, bool one, cudaStream_t stream) {
    return one ? launch_kernel<DH, G, BS, 1>(mq, mk, mv, mo, prm, stream)
               : launch_kernel<DH, G, BS, 2>(mq, mk, mv, mo, prm, stream);
}

bool encode_bf16(CUtensorMap *map, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
                 const cuuint32_t *box) {
    auto encode = tensor_map_encoder();
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH, int G>
cudaError_t launch_pairs(const PrefillArgs &a, const pa_diff &diff, bool by_head, cudaStream_t stream) {
    const int BS = a.pool.block_size, Hkv = a.pool.num_kv_heads, groups = by_head ? Hkv : Hkv / 2;
    const cuuint64_t row = (cuuint64_t)a.num_q_heads * DH * 2, rows = (cuuint64_t)a.num_seqs * a.chunk_len;
    CUtensorMap mq, mk, mv, mo;
    {   // q as (d, map, pair in group, group, token); box one map of 128 / G tokens' pairs
        const cuuint64_t dims[5] = {DH, 2, G, (cuuint64_t)groups, rows};
        const cuuint64_t strides[4] = {DH * 2, 2 * DH * 2, (cuuint64_t)G * 2 * DH * 2, row};
        const cuuint32_t box[5] = {64, 1, G, 1, kRows / G};
        if (!encode_bf16(&mq, 5, a.q, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {   // the output as (2d, pair in group, group, token); box a whole M-tile's queries, or all of them when fewer
        const cuuint64_t dims[4] = {2 * DH, G, (cuuint64_t)groups, rows};
        const cuuint64_t strides[3] = {2 * DH * 2, (cuuint64_t)G * 2 * DH * 2, row};
        const cuuint32_t box[4] = {64, G, 1, (cuuint32_t)std::max(1, std::min(kRows / G, a.chunk_len))};
        if (!encode_bf16(&mo, 4, a.out, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {   // keys as (64 of d, slot in eight, half of d, eight of slots in a head, block): one box a
        // block, laid out [eight slots][half][8][128 B], so that eights of keys lie evenly
        // apart over the whole tile (boxes of one half each took twice as many copies)
        const cuuint64_t dims[5] = {64, 8, DH / 64, (cuuint64_t)Hkv * (BS / 8), (cuuint64_t)a.pool.num_blocks};
        const cuuint64_t strides[4] = {DH * 2, 128, 8 * DH * 2, (cuuint64_t)a.pool.block_stride * 2};
        const cuuint32_t box[5] = {64, 8, DH / 64, (cuuint32_t)(BS / 8), 1};
        if (!encode_bf16(&mk, 5, a.pool.base, dims, strides, box)) return cudaErrorInvalidValue;
    }
    // values: one box per block, of both heads
    if (encode_pool_block_map(&mv, a.pool, 1, BS, 2) != cudaSuccess) return cudaErrorInvalidValue;
    DiffParams prm;
    prm.out = static_cast<__nv_bfloat16 *>(a.out);
    prm.tables = a.tables;
    prm.max_blocks = a.max_blocks;
    prm.ctx_lens = a.ctx_lens;
    prm.max_ctx_len = a.max_ctx_len;
    prm.chunk = a.chunk_len;
    prm.num_pairs = a.num_q_heads / 2;
    prm.num_blocks = a.pool.num_blocks;
    prm.scale_log2 = a.scale * kLog2e;
    prm.err = device_error_word();
    if (!prm.err) return cudaErrorUnknown;
    prm.num_mt = (a.chunk_len + kRows / G - 1) / (kRows / G);
    prm.num_kv = groups;
    prm.num_seqs = a.num_seqs;
    // The order of the units.  By tile, longest first over all groups and sequences, balances
    // the clusters best (2,048 tokens from the start, 32/8 heads, 8 MB: 94 us in the other order,
    // 74 in this), but neighbours then read different keys; where all keys and values are more
    // than L2 keeps (16 x (4,096 + 512), 300 MB: 1,680 us, 1,940 by tile), or where the
    // contexts, not the tiles, make the lengths (5 x 333 at up to 3,000: 44.4 us, 47.1 by
    // tile), the tiles of one group and sequence follow each other and read them together.
    // 48 MB lies between the sizes measured, well within L2.  The host knows bounds, not
    // lengths: short prompts called with a large max_ctx_len take the second order.
    prm.by_length = a.max_ctx_len < a.chunk_len &&
                    (int64_t)a.num_seqs * ((int64_t)a.max_ctx_len + a.chunk_len) * Hkv * DH * 4 <= (48ll << 20);
    prm.by_head = by_head ? 1 : 0;
    prm.lambda = diff.lambda;
    prm.norm_weight = diff.norm_weight;
    prm.eps = diff.eps;
    prm.out_scale = diff.out_scale;
    const bool one = (diff.flags & PA_DIFF_ONE_TERM) != 0;
    switch (BS) {
        case 8: return launch_terms<DH, G, 8>(mq, mk, mv, mo, prm, one, stream);
        case 16: return launch_terms<DH, G, 16>(mq, mk, mv, mo, prm, one, stream);
        case 32: return launch_terms<DH, G, 32>(mq, mk, mv, mo, prm, one, stream);
        case 64: return launch_terms<DH, G, 64>(mq, mk, mv, mo, prm, one, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int DH>
cudaError_t launch_dim(const PrefillArgs &a, const pa_diff &diff, cudaStream_t stream) {
    const int R = a.num_q_heads / a.pool.num_kv_heads;
    // Keys by head: the R query heads of a key head are R / 2 whole pairs, both maps on
    // the one key head.  With R = 1 it is what keys by map are.
    const bool by_head = (diff.flags & PA_DIFF_KEYS_BY_HEAD) != 0 && R > 1;
    switch (by_head ? R / 2 : R) {
        case 1: return launch_pairs<DH, 1>(a, diff, by_head, stream);
        case 2: return launch_pairs<DH, 2>(a, diff, by_head, stream);
        case 4: return launch_pairs<DH, 4>(a, diff, by_head, stream);
        case 8: return launch_pairs<DH, 8>(a, diff, by_head, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace prefill

bool prefill_diff_supported(int head_dim, int pairs, int block_size) {
    return (head_dim == 64 || head_dim == 128) && (pairs == 1 || pairs == 2 || pairs == 4 || pairs == 8) &&
           (block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64);
}

cudaError_t launch_prefill_diff(const PrefillArgs &a, const pa_diff &diff, cudaStream_t stream) {
    return a.pool.head_dim == 64 ? prefill::launch_dim<64>(a, diff, stream)
                                 : prefill::launch_dim<128>(a, diff, stream);
}

}  // namespace pa
