// pa_internal.h -- host-side interface between the C ABI layer (pa_api.cpp)
// and the kernel translation units.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>

#include "pa.h"

namespace pa {

// A validated, stride-resolved view of one layer of the block pool.
struct PoolView {
    const void *base;
    int64_t num_blocks;
    int32_t num_kv_heads;
    int32_t block_size;
    int32_t head_dim;
    int64_t block_stride;  // elements
    int64_t kv_stride;     // elements
};

// Device address of the current device's error word (set up once per device);
// nullptr if the CUDA runtime failed.
unsigned int *device_error_word();
cudaError_t launch_wait_timeout(uint64_t limit_ns, cudaStream_t stream);

// Number of SMs of the current device (cached per device); 0 on failure.
int device_sm_count();

// The driver's cuTensorMapEncodeTiled, resolved once through the runtime;
// nullptr if the driver does not provide it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Tensor map of the K (kv = 0) or V (kv = 1) half of a pool layer as (d within
// a 64-wide half, slot, half of d, kv-head, block): one box is `box_rows`
// slots (the whole block when box_rows = block_size) of one (block, K|V,
// kv-head) slab, laid out [half][slot][64] with 128-byte swizzle (head_dim 64
// or 128), or of box_heads such slabs one behind the other.  A block coordinate of
// num_blocks reads as zeros.
cudaError_t encode_pool_block_map(CUtensorMap *map, const PoolView &pool, int kv, int box_rows, int box_heads = 1);

// ---- slot writer and block copies (pa_cache.cu) ---------------------------
cudaError_t launch_reshape_and_cache(const PoolView &pool, const void *k, const void *v,
                                     const int64_t *slots, int64_t num_tokens, cudaStream_t stream);
cudaError_t launch_append_last(const PoolView &pool, const int32_t *tables, int32_t max_blocks,
                               const int32_t *seq_lens, int32_t num_seqs, int32_t max_len, const void *k,
                               const void *v, cudaStream_t stream);
cudaError_t launch_copy_blocks(const PoolView &pool, const int32_t *pairs, int32_t num_pairs,
                               cudaStream_t stream);
// host_dev: the device address of the pinned host buffer
cudaError_t launch_swap_blocks(const PoolView &pool, void *host_dev, int64_t host_blocks, const int32_t *pairs,
                               int32_t num_pairs, int32_t direction, cudaStream_t stream);

// ---- a step's tables, positions and slots (pa_extend.cu) --------------------
struct ExtendArgs {
    int32_t *tables;
    int32_t max_blocks;
    int32_t *seq_lens_out;
    int32_t *cu_seqlens;
    int64_t *positions;
    int64_t *slots;
    int32_t max_tokens;
    const int32_t *ctx_lens;
    const int32_t *new_lens;
    const int32_t *position_offsets;   // may be null
    int32_t num_seqs;
    const int32_t *free_blocks;
    int32_t num_free;
    const int32_t *cursor;
    int32_t *cursor_out;
    int32_t block_size;
    int64_t num_blocks;
};
cudaError_t launch_extend_tables(const ExtendArgs &a, cudaStream_t stream);

// ---- rotary positions (pa_rotary.cu); arguments validated, strides resolved --
// Positions of several axes: two bits a pair name the axis that turns it.
constexpr int kMaxAxes = 4;
constexpr int kMaxAxisPairs = 512;     // head_dim up to 1024
struct AxesView {
    int64_t stride;                    // elements between two axes' positions
    int32_t num_axes;
    uint32_t code[kMaxAxisPairs / 16];
};
cudaError_t launch_rotate(void *out, const void *x, int64_t x_stride, const int64_t *positions, int64_t num_tokens,
                          int32_t num_heads, int32_t head_dim, const pa_rotary &rotary, cudaStream_t stream);
cudaError_t launch_rotate_and_cache(const PoolView &pool, void *q_out, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                    const int64_t *positions, const int64_t *slots, int64_t num_tokens,
                                    int32_t num_q_heads, const pa_rotary &rotary, cudaStream_t stream);
// the same with positions of several axes (pa_rotary_axes.cu)
cudaError_t launch_rotate_axes(void *out, const void *x, int64_t x_stride, const int64_t *positions,
                               int64_t num_tokens, int32_t num_heads, int32_t head_dim, const pa_rotary &rotary,
                               const AxesView &axes, cudaStream_t stream);
cudaError_t launch_rotate_and_cache_axes(const PoolView &pool, void *q_out, const void *q, int64_t q_stride,
                                         const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                         const int64_t *positions, const int64_t *slots, int64_t num_tokens,
                                         int32_t num_q_heads, const pa_rotary &rotary, const AxesView &axes,
                                         cudaStream_t stream);

// ---- compaction of cached tokens (pa_compact.cu) ----------------------------
cudaError_t launch_compact(const PoolView &pool, const int32_t *src_tables, const int32_t *dst_tables,
                           int32_t max_blocks, const int32_t *seq_lens, const int32_t *keep, int32_t max_keep,
                           const int32_t *keep_lens, const int32_t *starts, int32_t num_seqs,
                           const pa_rotary *rotary, cudaStream_t stream);

// ---- beam selection (pa_beam.cu) --------------------------------------------
struct BeamArgs {
    float *scores_out;
    int32_t *parents_out, *tokens_out;
    const void *logits;
    bool bf16;                 // else fp32
    int64_t row_stride;        // elements
    const float *beam_scores;
    const uint8_t *finished;   // may be null
    int32_t end_token;
    int32_t num_groups, num_beams, vocab, num_out;
    void *workspace;           // beam_workspace bytes, 256-byte aligned
};
size_t beam_workspace(int32_t groups, int32_t beams, int32_t vocab, int32_t num_out);
cudaError_t launch_beam_select(const BeamArgs &a, cudaStream_t stream);

// ---- decode (pa_decode_*.cu) -----------------------------------------------
struct DecodeArgs {
    void *out;
    const void *q;
    PoolView pool;
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *seq_lens;
    int32_t num_seqs;
    int32_t num_q_heads;
    int32_t max_seq_len;
    float scale;
    int32_t partition_tokens;  // resolved (> 0, multiple of block_size)
    int32_t num_partitions;    // ceil(max_seq_len / partition_tokens), >= 1
    float *ws_o;               // split: [B][Hq][P][d] when num_partitions > 1; stream-K: [2C][G][d]
    float *ws_ml;              // split: [B][Hq][P][2]; stream-K: [2C][G][2]
    bool stream_k;             // persistent balanced schedule (automatic plan)
    int32_t num_ctas;          // stream-K grid size C
    bool early_meta = false;   // stream-K: read lengths and tables before the previous kernel completes
    const void *new_k = nullptr;   // stream-K: last token's K/V per sequence, stored before attending
    const void *new_v = nullptr;
    const float *pre_o = nullptr;      // cascade: prefix partial [B][Hq][d] fp32 (normalised)
    const float *pre_lse = nullptr;    // and its log-sum-exp [B][Hq]
    const pa_diff *diff = nullptr;     // differential attention (stream-K only)
};

// Tokens per pipeline stage of the decode kernel for a block size (the
// granularity a partition length is rounded to).
int decode_stage_tokens(int block_size);
bool decode_supported(int head_dim, int group, int block_size);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t stream);
cudaError_t launch_decode_diff(const DecodeArgs &a, cudaStream_t stream);   // pa_decode_diff_*.cu

// ---- prefill (pa_prefill.cu) -----------------------------------------------
struct PrefillArgs {
    void *out;
    const void *q;
    PoolView pool;
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *ctx_lens;
    int32_t num_seqs;
    int32_t chunk_len;
    int32_t num_q_heads;
    int32_t max_ctx_len;
    float scale;
    bool causal = true;        // false: every query sees keys 0 .. ctx_lens[s] - 1
    float *o_part = nullptr;   // non-null: fp32 normalised output + lse instead of out
    float *lse = nullptr;
    const int32_t *order = nullptr;   // non-null: sequences in this order (a permutation)
    // grouped decode: members' suffix tables and lengths (nullptr: none)
    const int32_t *sfx_tables = nullptr;
    int32_t sfx_max_blocks = 0;
    const int32_t *sfx_lens = nullptr;
    int32_t sfx_nb = 0;        // suffix-tile blocks per member
    int32_t max_sfx_len = 0;
    const void *new_k = nullptr;
    const void *new_v = nullptr;
    bool early_meta = false;   // order, ctx_lens and tables are not written by the kernel before
};
bool prefill_supported(int head_dim, int group, int block_size);
cudaError_t launch_prefill(const PrefillArgs &a, cudaStream_t stream);
void set_prefill_ctas(int32_t ctas);   // 0: one CTA per SM
int32_t prefill_ctas();

// ---- differential prefill (pa_prefill_diff.cu) -------------------------------
bool prefill_diff_supported(int head_dim, int pairs, int block_size);
cudaError_t launch_prefill_diff(const PrefillArgs &a, const pa_diff &diff, cudaStream_t stream);

}  // namespace pa
