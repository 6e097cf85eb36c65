// pa_decode_diff.cuh -- the parts of differential decode attention that differ from
// the plain one's; the schedule, the copies and the kernels around them are those of
// pa_decode_kernel.cuh.
//
// The mathematics.  KV heads come in pairs: pair g has the key heads 2g and 2g + 1
// (K1, K2) and one value row V = [V_2g | V_2g+1] of 2d components.  Query heads come
// in pairs too, h = (2h, 2h + 1), R of them a KV pair, and
//     x_h = softmax(s q_2h K1^T) V - lambda_h softmax(s q_2h+1 K2^T) V,
// then, with a norm weight, x_h / sqrt(mean x_h^2 + eps) * weight, and the scale of
// the output.  (With keys by head, query head i of the group's 2R reads key head
// 2g + i / R instead.)
//
// How it runs on the plain kernel's frame: K rows [K1 | K2] and V rows [V1 | V2] of
// 2d components are one row each (a copy box takes both heads of a slot, so a
// pipeline stage is 16 tokens of twice the width), and the 2R maps are columns of the
// score MMA: the first R of them read K1, the others K2.  Up to R = 4 all 2R columns fit
// one n8 tile, which meets both key heads, and each column keeps the product with its own
// (a product with zeros instead would carry another head's infinities over).  R = 8 has
// a tile for each key head, at d = 128 in a warp of its own.  The values are staged once
// and serve every column, so every byte of the cache is read once; what the difference
// needs of two maps meets only where a unit's rows are finished: one warp a query pair
// holds both maps' sums of a whole row, so the norm is one warp reduction.
//
// The probabilities enter P.V as two bf16 terms, as in the plain kernel: the
// difference of two maps is smaller than either, and the norm scales it up again, so
// a rounding of p (up to 2^-8) would weigh more here than there.
//
// What bounds it: DRAM, as the plain kernel.  GB300, of the measured copy bandwidth: 4 x
// 32,768 tokens of 32/8 heads, d = 128, 87 us (0.91); 64 x 600-850 of 64/8 40.2 us (0.71: the
// start, a unit's end to every 46 stages, the merge behind); 33 x 1-3,000, d = 64, 37 us (0.81).
#pragma once

namespace pa {
namespace decode {

// Warps that share a ring and its stages: two, one for each key head and its maps, where
// rows of 256 components have sixteen maps (R = 8): a warp with all of them would run 800
// instructions a stage, one warp to a scheduler, and that takes longer than the stage's 16
// KB take to arrive (64 sequences of 600-850 tokens, 64/8 heads: 45.2 us, 42.4 with two).
// (Two rings a CTA instead of four, so that two CTAs fit an SM: 43.0 us, and 90.4 instead
// of 86.5 for 4 x 32,768 tokens.)
template <int D, int G>
constexpr int kDiffParts = D == 256 && G == 16 ? 2 : 1;

template <int D, int G>
struct DiffState {
    static constexpr int R = G / 2;           // query pairs of a unit
    static constexpr int NB = G > 8 && kDiffParts<D, G> == 1 ? 2 : 1;  // n8 tiles of map columns a warp has
    float m[NB][2];           // running max (log2 domain) of columns 2t, 2t + 1 of each tile
    float l[NB][2];           // this lane's share of their denominators
    float o[D / 16][NB][4];   // O^T tiles
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i][nb][0] = o[i][nb][1] = o[i][nb][2] = o[i][nb][3] = 0.f;
        }
    }
};

// Query head (within the unit's G) of map column c: the first R columns read key
// head 2g, the others 2g + 1.
template <int G>
__device__ __forceinline__ int diff_head_of(int c, bool by_head) {
    constexpr int R = G / 2;
    return by_head ? c : (c < R ? 2 * c : 2 * (c - R) + 1);
}
// The column of map j (0, 1) of query pair r.
template <int G>
__device__ __forceinline__ int diff_column_of(int r, int j, bool by_head) {
    return by_head ? 2 * r + j : r + j * (G / 2);
}

template <int D, int G, int BS>
struct DiffOp {
    using S = Shape<D, BS>;
    using State = DiffState<D, G>;
    static constexpr int R = State::R, NB = State::NB;
    static constexpr bool kSplit = kDiffParts<D, G> == 2;   // this warp has the maps of key head `part` alone
    static constexpr int kCols = kSplit ? R : G;         // its columns: part * kCols + 0 .. kCols - 1
    static constexpr int d = D / 2;        // one head's components
    static constexpr int kCh = d / 32;     // 16-byte chunks of one key row that a lane reads
    struct Q {
        uint32_t w[NB][4 * kCh];           // this lane's column's q, in its K chunk order
    };

    static __device__ __forceinline__ void load_q(Q &q, const __nv_bfloat16 *rows, int lane, bool by_head, int part) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int own = nb * 8 + g;      // among this warp's columns
            const __nv_bfloat16 *row = rows + diff_head_of<G>(own < kCols ? part * kCols + own : 0, by_head) * d;
#pragma unroll
            for (int idx = 0; idx < kCh; ++idx) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (own < kCols) v = *reinterpret_cast<const uint4 *>(row + (idx >> 1) * 64 + (2 * t + (idx & 1)) * 8);
                q.w[nb][4 * idx + 0] = v.x;
                q.w[nb][4 * idx + 1] = v.y;
                q.w[nb][4 * idx + 2] = v.z;
                q.w[nb][4 * idx + 3] = v.w;
            }
        }
    }

    // One pipeline stage, as stage_compute: 16 tokens, token tok0 + j valid while < tok_end.
    static __device__ __forceinline__ void compute(uint32_t kslot, uint32_t vslot, const Q &q, int tok0, int tok_end,
                                                   float scale_log2, int lane, int part, State &st) {
        const int g = lane >> 2, t = lane & 3;
        const int nvalid = tok_end - tok0;
        const bool tail = nvalid < S::TPS;
        float c[2][4];   // by key head
#pragma unroll
        for (int kh = 0; kh < (kSplit ? 1 : 2); ++kh) {
            c[kh][0] = c[kh][1] = c[kh][2] = c[kh][3] = 0.f;
#pragma unroll
            for (int idx = 0; idx < kCh; ++idx) {
                const int hh = (kh + part) * (d / 64) + (idx >> 1), ch = 2 * t + (idx & 1);
                const uint4 a = lds128(kslot + chunk_at(row_off<D, BS>(g, hh), ch));
                const uint4 b = lds128(kslot + chunk_at(row_off<D, BS>(g + 8, hh), ch));
                const uint32_t *w = &q.w[NB == 2 ? kh : 0][4 * idx];
                mma_bf16(c[kh], a.x, b.x, a.y, b.y, w[0], w[1]);
                mma_bf16(c[kh], a.z, b.z, a.w, b.w, w[2], w[3]);
            }
        }
        float x[NB][4];
        if constexpr (kSplit) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[0][i] = c[0][i];
        } else if constexpr (NB == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[0][i] = c[0][i];
                x[1][i] = c[1][i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[0][i] = 2 * t + (i & 1) < R ? c[0][i] : c[1][i];
        }
        const bool v0 = !tail || g < nvalid, v1 = !tail || g + 8 < nvalid;
        uint32_t pb[NB][2][2];   // [tile][token row g | g + 8][hi | lo]: bf16 pairs of columns (2t, 2t + 1)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float (&y)[4] = x[nb];
            y[0] = v0 ? y[0] * scale_log2 : -INFINITY;
            y[1] = v0 ? y[1] * scale_log2 : -INFINITY;
            y[2] = v1 ? y[2] * scale_log2 : -INFINITY;
            y[3] = v1 ? y[3] * scale_log2 : -INFINITY;
            float mh0 = fmaxf(y[0], y[2]), mh1 = fmaxf(y[1], y[3]);
#pragma unroll
            for (int dist = 4; dist < 32; dist <<= 1) {
                mh0 = fmaxf(mh0, __shfl_xor_sync(0xffffffffu, mh0, dist));
                mh1 = fmaxf(mh1, __shfl_xor_sync(0xffffffffu, mh1, dist));
            }
            const float mn0 = fmaxf(st.m[nb][0], mh0), mn1 = fmaxf(st.m[nb][1], mh1);
            const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
            const float al0 = fast_exp2(st.m[nb][0] - mu0), al1 = fast_exp2(st.m[nb][1] - mu1);
            const bool moved = mn0 != st.m[nb][0] || mn1 != st.m[nb][1];
            float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float pa = fast_exp2(y[2 * r] - mu0), pc = fast_exp2(y[2 * r + 1] - mu1);
                const __nv_bfloat162 hi = __floats2bfloat162_rn(pa, pc);
                const __nv_bfloat162 lo = __floats2bfloat162_rn(pa - __low2float(hi), pc - __high2float(hi));
                ps0 += pa;
                ps1 += pc;
                pb[nb][r][0] = *reinterpret_cast<const uint32_t *>(&hi);
                pb[nb][r][1] = *reinterpret_cast<const uint32_t *>(&lo);
            }
            st.l[nb][0] = st.l[nb][0] * al0 + ps0;
            st.l[nb][1] = st.l[nb][1] * al1 + ps1;
            st.m[nb][0] = mn0;
            st.m[nb][1] = mn1;
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    st.o[mt][nb][0] *= al0;
                    st.o[mt][nb][1] *= al1;
                    st.o[mt][nb][2] *= al0;
                    st.o[mt][nb][3] *= al1;
                }
            }
        }
        uint32_t bt[NB][4];   // P^T operands: hi of tokens 0-7, 8-15, then lo
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            bt[nb][0] = transpose8x8(pb[nb][0][0]);
            bt[nb][1] = transpose8x8(pb[nb][1][0]);
            bt[nb][2] = transpose8x8(pb[nb][0][1]);
            bt[nb][3] = transpose8x8(pb[nb][1][1]);
        }
        // ---- O^T += V^T . P^T, 128 components (two 64-wide halves) at a time: tile mt of them
        // has rows of element mt of each half's chunk g
#pragma unroll
        for (int hp = 0; hp < D / 128; ++hp) {
            uint32_t vw[4][2][4];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int j = 2 * t + (kk & 1) + 8 * (kk >> 1);
                const bool valid = !tail || j < nvalid;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint4 w = lds128(vslot + chunk_at(row_off<D, BS>(j, 2 * hp + hh), g));
                    if (!valid) w = make_uint4(0u, 0u, 0u, 0u);
                    vw[kk][hh][0] = w.x;
                    vw[kk][hh][1] = w.y;
                    vw[kk][hh][2] = w.z;
                    vw[kk][hh][3] = w.w;
                }
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const uint32_t sel = (mt & 1) ? 0x7632u : 0x5410u;
                const uint32_t a0 = __byte_perm(vw[0][0][mt >> 1], vw[1][0][mt >> 1], sel);
                const uint32_t a1 = __byte_perm(vw[0][1][mt >> 1], vw[1][1][mt >> 1], sel);
                const uint32_t a2 = __byte_perm(vw[2][0][mt >> 1], vw[3][0][mt >> 1], sel);
                const uint32_t a3 = __byte_perm(vw[2][1][mt >> 1], vw[3][1][mt >> 1], sel);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    mma_bf16(st.o[hp * 8 + mt][nb], a0, a1, a2, a3, bt[nb][0], bt[nb][1]);
                    mma_bf16(st.o[hp * 8 + mt][nb], a0, a1, a2, a3, bt[nb][2], bt[nb][3]);
                }
            }
        }
    }

    // As warp_publish, by map column.
    static __device__ __forceinline__ void publish(State &st, bool has_work, int lane, int warp, int part, float *cm,
                                                   float *cl, float *co) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float l[2] = {st.l[nb][0], st.l[nb][1]};
#pragma unroll
            for (int dist = 4; dist < 32; dist <<= 1) {
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], dist);
                l[1] += __shfl_xor_sync(0xffffffffu, l[1], dist);
            }
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int own = nb * 8 + 2 * t + hi, c = part * kCols + own;
                if (own >= kCols) continue;
                float *dst = co + (warp * G + c) * D;
#pragma unroll
                for (int hp = 0; hp < D / 128; ++hp)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr) {
                        float4 *d4 = reinterpret_cast<float4 *>(dst + (2 * hp + rr) * 64 + g * 8);
                        const int i = 2 * rr + hi, m0 = hp * 8;
                        d4[0] = make_float4(st.o[m0][nb][i], st.o[m0 + 1][nb][i], st.o[m0 + 2][nb][i],
                                            st.o[m0 + 3][nb][i]);
                        d4[1] = make_float4(st.o[m0 + 4][nb][i], st.o[m0 + 5][nb][i], st.o[m0 + 6][nb][i],
                                            st.o[m0 + 7][nb][i]);
                    }
                if (g == 0) {
                    cm[warp * G + c] = has_work ? st.m[nb][hi] : -INFINITY;
                    cl[warp * G + c] = has_work ? l[hi] : 0.f;
                }
            }
        }
    }

    // (What is summed for each map is written as the operations that are meant: contracted
    // differently for the two, equal maps would not cancel.)

    // A finished row of query pair h (of the whole batch's row `row`): the lane's four
    // components of every 128, already divided by their maps' sums.
    static __device__ __forceinline__ void finish_row(const Params &p, size_t row, int h, int lane,
                                                      const float (&a)[D / 128][4], const float (&b)[D / 128][4]) {
        const float lam = __ldg(p.lambda + h);
        float x[D / 128][4], ss = 0.f;
#pragma unroll
        for (int k = 0; k < D / 128; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[k][e] = __fmaf_rn(-lam, b[k][e], a[k][e]);
                ss += x[k][e] * x[k][e];
            }
        float f = p.out_scale;
        if (p.norm_weight != nullptr) {
#pragma unroll
            for (int dist = 1; dist < 32; dist <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, dist);
            f *= rsqrtf(ss * (1.f / D) + p.eps);
        }
#pragma unroll
        for (int k = 0; k < D / 128; ++k) {
            const int i = k * 128 + lane * 4;
            float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
            if (p.norm_weight != nullptr) w = __ldg(reinterpret_cast<const float4 *>(p.norm_weight + i));
            *reinterpret_cast<uint2 *>(p.out + row * D + i) =
                make_uint2(pack_bf16x2(x[k][0] * f * w.x, x[k][1] * f * w.y),
                           pack_bf16x2(x[k][2] * f * w.z, x[k][3] * f * w.w));
        }
    }

    // The warps' (m, l, o) of one unit combined: finished rows (a warp a query pair), or
    // fp32 partials by column, as cta_combine_store's.
    static __device__ __forceinline__ void combine_store(const Params &p, const float *cm, const float *cl,
                                                         const float *co, bool final, size_t row0, int pair0,
                                                         float *o_base, float *ml_base) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const bool by_head = p.by_head != 0;
        for (int r = warp; r < R; r += kWarps * kDiffParts<D, G>) {
            float acc[2][D / 128][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = final ? diff_column_of<G>(r, j, by_head) : 2 * r + j;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, cm[w * G + c]);
                float f[kWarps], lsum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    f[w] = M == -INFINITY ? 0.f : fast_exp2(cm[w * G + c] - M);
                    lsum = __fmaf_rn(cl[w * G + c], f[w], lsum);
                }
                const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
#pragma unroll
                for (int k = 0; k < D / 128; ++k) {
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float4 v =
                            *reinterpret_cast<const float4 *>(co + (w * G + c) * D + k * 128 + lane * 4);
                        s.x = __fmaf_rn(v.x, f[w], s.x);
                        s.y = __fmaf_rn(v.y, f[w], s.y);
                        s.z = __fmaf_rn(v.z, f[w], s.z);
                        s.w = __fmaf_rn(v.w, f[w], s.w);
                    }
                    acc[j][k][0] = __fmul_rn(s.x, inv);
                    acc[j][k][1] = __fmul_rn(s.y, inv);
                    acc[j][k][2] = __fmul_rn(s.z, inv);
                    acc[j][k][3] = __fmul_rn(s.w, inv);
                    if (!final)
                        *reinterpret_cast<float4 *>(o_base + (size_t)c * D + k * 128 + lane * 4) =
                            make_float4(acc[j][k][0], acc[j][k][1], acc[j][k][2], acc[j][k][3]);
                }
                if (!final && lane == 0) *reinterpret_cast<float2 *>(ml_base + c * 2) = make_float2(M, lsum);
            }
            if (final) finish_row(p, row0 + r, pair0 + r, lane, acc[0], acc[1]);
        }
    }

    // Merge of a unit cut between CTAs, from the records of CTAs ca .. cb (the first
    // one's is record 2 ca + first_rec, the others' 2 cc): a warp a query pair.
    static __device__ __forceinline__ void merge(const Params &p, int ca, int cb, int first_rec, size_t row0,
                                                 int pair0, int warp, int nwarps, int lane) {
        constexpr int kR = 2;   // records of both maps loaded together
        for (int r = warp; r < R; r += nwarps) {
            float M[2] = {-INFINITY, -INFINITY}, wsum[2] = {0.f, 0.f}, out[2][D / 128][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < D / 128; ++k) out[j][k][0] = out[j][k][1] = out[j][k][2] = out[j][k][3] = 0.f;
            const int c0 = diff_column_of<G>(r, 0, p.by_head != 0), c1 = diff_column_of<G>(r, 1, p.by_head != 0);
            for (int first = ca; first <= cb; first += kR) {
                float2 ml[2][kR];
                float4 ov[2][kR][D / 128];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < kR; ++q) {
                        const int cc = first + q;
                        ml[j][q] = make_float2(-INFINITY, 0.f);
                        if (cc <= cb) {
                            const size_t rec = (2 * (size_t)cc + (cc == ca ? first_rec : 0)) * G + (j == 0 ? c0 : c1);
                            ml[j][q] = *reinterpret_cast<const float2 *>(p.ws_ml + rec * 2);
#pragma unroll
                            for (int k = 0; k < D / 128; ++k)
                                ov[j][q][k] =
                                    *reinterpret_cast<const float4 *>(p.ws_o + rec * D + k * 128 + lane * 4);
                        }
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float Mn = M[j];
#pragma unroll
                    for (int q = 0; q < kR; ++q) Mn = fmaxf(Mn, ml[j][q].x);
                    if (Mn == -INFINITY) continue;
                    const float f = M[j] == -INFINITY ? 0.f : fast_exp2(M[j] - Mn);
                    wsum[j] = __fmul_rn(wsum[j], f);
#pragma unroll
                    for (int k = 0; k < D / 128; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) out[j][k][e] = __fmul_rn(out[j][k][e], f);
#pragma unroll
                    for (int q = 0; q < kR; ++q) {
                        if (ml[j][q].x == -INFINITY) continue;
                        const float w = __fmul_rn(ml[j][q].y, fast_exp2(ml[j][q].x - Mn));
                        wsum[j] = __fadd_rn(wsum[j], w);
#pragma unroll
                        for (int k = 0; k < D / 128; ++k) {
                            out[j][k][0] = __fmaf_rn(w, ov[j][q][k].x, out[j][k][0]);
                            out[j][k][1] = __fmaf_rn(w, ov[j][q][k].y, out[j][k][1]);
                            out[j][k][2] = __fmaf_rn(w, ov[j][q][k].z, out[j][k][2]);
                            out[j][k][3] = __fmaf_rn(w, ov[j][q][k].w, out[j][k][3]);
                        }
                    }
                    M[j] = Mn;
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float inv = wsum[j] > 0.f ? 1.f / wsum[j] : 0.f;
#pragma unroll
                for (int k = 0; k < D / 128; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) out[j][k][e] = __fmul_rn(out[j][k][e], inv);
            }
            finish_row(p, row0 + r, pair0 + r, lane, out[0], out[1]);
        }
    }
};

}  // namespace decode
}  // namespace pa
