// Internal interfaces between the C ABI (abi.cu) and the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace fw {

// Launches `kernel` so that it may start while the previous kernel in the
// stream still runs (programmatic stream serialization); the kernel calls
// pdl_wait() before it reads anything that kernel wrote.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_after_previous(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                         cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kKvTile = 128;          // keys per KV tile (MMA M extent in decode, N in prefill)

// Device event counters (the FW_COUNTER_* indices of the C ABI).
constexpr int kCounterPrefillReplays = 0;   // (query row, KV tile) steps the static-anchor check replayed
constexpr int kCounterLatentRescales = 1;   // (query row, key step) steps whose latent anchor moved
constexpr int kNumCounters = 4;
constexpr int kSoftmaxStartWarp = 2;  // decode: warps 2..5 run the softmax / epilogue

constexpr int kDecodeMinSpan = 8;     // decode: fewest KV tiles one CTA range holds (auto mode)
constexpr int kLatentMinSpan = 32;    // latent-head decode: the same, for its heavier tiles
// What starting a piece costs a decode CTA, in KV tiles of streaming (the
// next unit's Q, the pipeline refill, the previous piece's epilogue): a
// clock64 trace of the FP8 kernel puts a piece boundary at ~8,400 cycles
// against ~1,425 per tile inside a piece.  The planned tile sequence gives
// every unit this many empty slots before its tiles, so equal ranges of it
// carry equal work, piece starts included.
constexpr int kDecodePieceCostBf16 = 4;
constexpr int kDecodePieceCostFp8 = 5;
constexpr int kTreeMinSpan = 2;       // tree decode: fewest KV tiles (and empty slots) one CTA range holds (4: a
                                      // 700-key request takes 17.0 us instead of 14.1)
// Tree decode: empty slots before a unit's tiles.  One row tile over a BF16
// cache streams a tile in 1.4 us, and starting a unit costs about as much (16
// ragged requests, hd 128: 56.6 us at 1 slot, 57.9 at 3, 58.5 at 5); an FP8 tile
// takes half of that (144 us at 1, 139 at 5), and two row tiles share a unit's
// longer start and end (121-draft trees: 146 at 1, 141 at 5; since pieces end
// faster 3 .. 7 are within 1 us, FP8 136 at 3, 133 at 5, 132.6 at 7).
constexpr int kTreePieceCostOne = 1;
constexpr int kTreePieceCost = 5;
// Chunk attention: the same, in keys; every unit weighs a tile more than its keys, for
// the tiles that its first and last key share.  Two row tiles: 16 prompts of 300 .. 5,000
// tokens 861 us at 0, 828 at 256, 832 at 384, 866 at 640; a mixed batch 349, 329, 330, 326;
// over FP8 caches 766 at 256, 755 at 384, 760 at 640, and prompts there 980, 959, 995 (one row
// tile: 174 us at 128, 170 at 384, 172 at 640); pairs of CTAs 163 at 0, 158, 154, 154.
constexpr int kChunkMinSpan = 256;
constexpr int kChunkPieceCostOne = 128;
constexpr int kChunkPieceCost = 384;
constexpr int kChunkPieceCostPair = 640;
constexpr int kMaxTableRows = 8192;   // page tables: requests whose sums fit a block's shared memory
constexpr int kLatentRows = 64;       // latent-head decode: query heads per CTA (MMA N of one CTA)
constexpr int kLatentPairRows = 128;  // latent-head decode on CTA pairs: query heads per pair

// One decode launch, fully resolved on the host.
//
// Scheduling: the (batch row, KV head, row group) units are laid end to end
// in that order, each contributing ceil(n_b / 128) KV tiles; the plan kernel
// writes the exclusive prefix PB[b] of these tile counts per batch row, the
// total T and the range span.  CTA c then processes the global tile ranges
// [r * span, (r + 1) * span) for r = c, c + grid, ...; the part of a unit
// inside one range is a "piece" and writes a split-KV partial unless the unit
// fits in a single range.  With head_ride the KV head leaves the unit: the
// units are (batch row, row group), and CTA c takes KV head c % Hkv over the
// ranges c / Hkv, c / Hkv + grid / Hkv, ...; the Hkv CTAs of one range then
// read the heads of the same token rows at the same time (one DRAM row and,
// for 128-byte FP8 rows, one 256-byte L2 fetch serve two of them).
// KV-cache append ("Writing Page Attention with PyPTO", section 4.3): row
// (b, t, kv head) of the new keys/values goes to cache token row
// layer_base + max(slot_mapping[b * q_len + t], 0).  rows = 0: nothing.
struct AppendParams {
    int64_t rows;                              // B * q_len * Hkv
    int q_len, Hkv, Dk, Dv, ps;
    int kv8;                                   // 1: E4M3 caches, code of x / scale
    float k_scale, v_scale;
    const uint16_t *k_new, *v_new;             // [B, q_len, Hkv, D] bf16; v_new may be null
    int64_t kn_stride[3], vn_stride[3];        // elements (b, t, head); last dim contiguous
    const int32_t *slot_mapping;               // [B * q_len]
    int64_t layer_base, cache_rows;            // token rows; cache_rows = pages * ps
    void *k_cache, *v_cache;                   // [pages, ps, Hkv, D]
    int64_t kc_stride[3], vc_stride[3];        // elements (page, slot, head)
};

struct DecodeParams {
    int B, q_len, Hq, Hkv, G, ps, max_pages, num_pages;
    int head_mode;        // 0: a unit holds whole head groups for tokens_per_unit tokens;
                          // 1: a unit holds `rows` consecutive heads of one token
    int rows;             // NQ: padded MMA N extent
    int tokens_per_unit, heads_per_unit, head_chunks, row_groups, units_per_row;
    int forced_span;      // KV tiles per range, 0 = auto
    int min_span;         // lower bound of the auto span
    int max_pieces;       // workspace slots per query row
    int grid;             // CTAs of the attention kernel
    int range_groups;     // 1: CTA c takes ranges c, c + grid, ...; R > 1: the R row groups of
                          // a unit ride on the CTA index (CTA c runs row group c % R over ranges
                          // c / R, c / R + grid / R, ...), so they read the same keys together
    int Dv;
    int packed;           // latent heads: 1 when q rows are read through the flattened (token, head)
                          // axis (one KV head, q contiguous over it): a row group is `rows` consecutive
                          // packed rows t * Hq + h and may straddle tokens ("TokenSpeed-MLA 2.0.1",
                          // packed-query paragraph); 0: one token's heads per row group
    int window_left;      // < 0: none; else token t sees keys max(0, n - q_len + t - W) .. n - q_len + t
    int causal;           // 1: token t sees keys up to its own position n - q_len + t; 0: all n keys
    AppendParams app;     // appended by the plan launch's extra blocks before the attention reads
    int32_t *plan;        // [0] = T, [1] = span, [2 .. 2 + B] = PB
    const int32_t *block_table; int64_t bt_stride;
    const int32_t *seq_lens;
    void *out; int64_t out_stride[4];          // [B, q_len, Hq, Dv] bf16
    float *lse; int64_t lse_stride[3];         // [B, q_len, Hq] or nullptr
    float *ws_o;                               // [B*q_len*Hq, max_pieces, Dv]
    float *ws_lse;                             // [B*q_len*Hq, max_pieces] (log2 units)
    float scale_log2;                          // scale * log2(e) (times k_scale for an FP8 cache)
    float out_scale;                           // v_scale for an FP8 cache, else 1
    uint64_t timeout_ns;
    int *status;                               // device status word
    unsigned long long *counters;              // device event counters (FW_COUNTER_*)
    int test_stall;                            // test hook: the producer first waits on a barrier nothing completes
    int piece_cost;                            // empty slots before each unit's tiles in the planned sequence
    int head_ride;        // 1: the KV heads ride on the CTA index (CTA c runs KV head c % Hkv over
                          // ranges c / Hkv, c / Hkv + grid / Hkv, ... of the (batch row, row group)
                          // units), so the Hkv CTAs reading one token row's heads run side by side
};

// One varlen prefill launch.  The plan kernel lists the units (sequence,
// query head, pair of consecutive 128-row query tiles) longest first; the
// CTAs (CTA pairs at head dim 256) take list entries in that order as they
// free up, from a counter in the plan.
struct PrefillParams {
    int B, Hq, Hkv, G, causal, Dv;
    int online;           // 0: static anchor with check and replay; 1: online softmax, conditional rescale
    int64_t total_q, total_k;
    const int32_t *cu_q, *cu_k;
    void *out; int64_t out_stride[3];          // [total_q, Hq, Dv] bf16
    float *lse; int64_t lse_stride[2];         // [total_q, Hq] or nullptr
    float scale_log2;
    uint64_t timeout_ns;
    int *status;
    unsigned long long *counters;              // device event counters (FW_COUNTER_*)
    int32_t *plan;        // [0] = entries, [1] = pairs, [2 .. 2 + B] = pair prefix PP, [3 + B] = next entry
                          // to hand out (CTAs take entries in list order as they free up)
    int32_t *list;        // entries pair_index * Hq + head, sorted by cost, longest first
    int64_t list_capacity;
    int grid;
};

// One tree decode call (fw_paged_decode_tree), fully resolved on the host.
struct TreeCut {                               // a unit whose first piece ended a CTA's range
    int count;                                 // its pieces, 0: none
    int b, g, rt0, nrt, d;                     // request, KV head, row tiles, drafts
    int pad_[2];
};
struct TreeParams {
    int B, T, Hq, Hkv, G, D, ps, max_pages, num_pages;
    int ps_shift;                              // log2 of ps, -1: not a power of two
    int kv8;                                   // 1: E4M3 caches
    const uint16_t *q; int64_t q_stride[3];    // [B, T, Hq, D] bf16
    const void *k_cache, *v_cache;
    int64_t kc_stride[3], vc_stride[3];        // elements (page, slot, head)
    const int32_t *block_table; int64_t bt_stride;
    const int32_t *seq_lens;
    const int32_t *draft_lens;                 // null: T drafts each
    const int32_t *mask; int64_t mask_stride[2];   // (b, t); words contiguous
    void *out; int64_t out_stride[3];          // [B, T, Hq, D] bf16
    float *lse; int64_t lse_stride[3];         // [B, T, Hq] or null
    float scale_log2;                          // scale * k_scale * log2(e)
    float out_scale;                           // v_scale
    int tile_tokens;                           // whole drafts of a 128-row tile (G <= 128)
    int head_chunks;                           // > 1: 128-head row tiles of one draft (G > 128)
    int row_tiles;                             // row tiles of T drafts
    int grid;                                  // CTAs
    int ride;                                  // 1: the KV heads ride on the CTA index
    int min_span, piece_cost;                  // least key tiles of a range; empty slots before a unit's tiles
    float *part_o;                             // [2 * grid][row tiles of a unit * 128][D] unnormalised pieces
    float2 *part_ml;                           // base (log2) and row sum of each of their rows
    TreeCut *cuts;                             // [grid]
    int test_stall;                            // test hook: the producer first waits on a barrier nothing completes
    uint64_t timeout_ns;
    int *status;
};

// One fw_tree_mask launch.
struct TreeMaskParams {
    int B, T, W;                               // W: words a mask row holds
    const int32_t *parents; int64_t parent_stride;
    const int32_t *draft_lens;                 // null: T
    int32_t *mask; int64_t mask_stride[2];
    int32_t *depths; int64_t depth_stride;     // null: not wanted
    int *status;
};

// One fw_build_page_tables call.
struct PageTableParams {
    int B, max_pages, F, ps;
    int ps_shift;                              // log2 of ps, -1: not a power of two
    int padded, L;                             // 1: L places per request; 0: packed
    int N;                                     // places in all
    const int32_t *seq_lens, *new_lens, *held;
    int32_t *queue;
    const int32_t *range;
    int32_t *table; int64_t table_stride;
    int32_t *slots, *cu_new, *held_out, *range_out;
    int in_place;                              // held_out is held, or range_out free_range
    int num_sms;
    int *status;
};

// One fw_kv_commit launch.
struct CommitParams {
    int B, A, Hkv, ps, layers, max_pages;
    int64_t layer_pages;
    int k_units, v_units;                      // 16-byte units of one head row (v_units 0: no values)
    const int32_t *path; int64_t path_stride;
    const int32_t *path_lens, *base_lens;
    const int32_t *table; int64_t table_stride;
    void *k_cache, *v_cache;
    int64_t kc_stride[3], vc_stride[3];        // bytes (page, slot, head)
    int32_t *new_lens;
    int num_sms;
    int *status;
};

// One chunk attention call (fw_paged_prefill), fully resolved on the host.
struct ChunkCut {                              // a unit whose first piece ended a CTA's range
    int count;                                 // its pieces, 0: none
    int g, rt0, nrt, d, q0;                    // KV head, row tiles, the request's tokens and first packed row
    int pad_[2];
};
struct ChunkParams {
    int B, Hq, Hkv, G, D, ps, max_pages, num_pages;
    int ps_shift;                              // log2 of ps, -1: not a power of two
    int kv8;                                   // 1: E4M3 caches
    int causal, window;                        // window < 0: none
    int64_t total_q;
    const int32_t *cu;                         // [B + 1] first packed rows
    const int32_t *seq_lens;
    const int32_t *block_table; int64_t bt_stride;
    void *out; int64_t out_stride[2];          // [total_q, Hq, D] bf16
    float *lse; int64_t lse_stride[2];         // [total_q, Hq] or null
    float scale_log2;                          // scale * k_scale * log2(e)
    float out_scale;                           // v_scale
    int tile_tokens;                           // whole tokens of a 128-row tile (G <= 128)
    int head_chunks;                           // > 1: 128-head row tiles of one token (G > 128)
    int row_tiles;                             // row tiles of a unit, 1 or 2
    int grid;                                  // CTAs
    int workers;                               // CTAs, or pairs of them, that take a range each
    int ride;                                  // 1: the KV heads ride on the worker's number
    int min_span, piece_cost;                  // in keys: least a range holds; what a unit's start weighs
    float *part_o;                             // [2 * workers][row tiles of a unit * 128][D] unnormalised pieces
    float2 *part_ml;                           // base (log2) and row sum of each of their rows
    ChunkCut *cuts;                            // [workers]
    int test_stall;                            // test hook: the producer first waits on a barrier nothing completes
    uint64_t timeout_ns;
    int *status;
};

// One fw_verify_drafts launch.
struct VerifyParams {
    int B, T, V, A;
    int context;                               // 1: the rows begin with the committed context's
    const int32_t *tokens; int64_t token_stride;
    const int32_t *parents; int64_t parent_stride;
    const int32_t *draft_lens;                 // null: T
    const float *target; int64_t target_stride[2];     // (b, row)
    const float *draft; int64_t draft_stride[2];       // null: drafts proposed with certainty
    const float *uniforms; int64_t uniform_stride;
    int32_t *path; int64_t path_stride;
    int32_t *path_lens, *next_tokens;
    int num_sms;
    int *status;
};

// One fw_qk_norm_rope or fw_qk_norm_rope_append launch.
struct NormRopeParams {
    int64_t N;                                 // tokens
    int Hq, Hkv, D, rot, axes, interleaved;
    const uint16_t *q, *k, *v;                 // v null: keys go to k_out, or values are not appended
    int64_t q_stride[2], k_stride[2], v_stride[2];     // elements (token, head)
    uint16_t *q_out, *k_out;                   // k_out null: keys go to the cache
    int64_t qo_stride[2], ko_stride[2];
    const void *weight[2];                     // of queries and keys; null: not normed
    int weight_f32[2];
    float eps;
    const float *inv_freq;                     // [rot / 2]
    const int32_t *positions; int64_t pos_stride;      // (axis); tokens contiguous
    const int32_t *axis_map;                   // [rot / 2] or null
    const int32_t *slots;                      // [N], null: no append
    int64_t layer_base, cache_rows;
    int ps, ps_shift, kv8;                     // ps_shift: log2 of ps, -1: not a power of two
    void *k_cache, *v_cache;
    int64_t kc_stride[3], vc_stride[3];        // elements (page, slot, head)
    float k_scale, v_scale;
    float k_inv, v_inv;                        // their reciprocals; 0: the kernel divides
    int num_sms;
    int *status;
};

// plan kernel + attention kernel + combine kernel, in stream order
cudaError_t launch_decode(const DecodeParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                          const CUtensorMap &tm_v, int head_dim, cudaStream_t stream,
                          cudaEvent_t timing_start, cudaEvent_t timing_stop, int *launches);
size_t decode_smem_bytes(int head_dim, int rows);
cudaError_t launch_decode_plan(const DecodeParams &p, cudaStream_t stream);
cudaError_t launch_decode_combine(const DecodeParams &p, int head_dim_v, cudaStream_t stream);
// Standalone KV-cache append (the fused form runs inside launch_decode_plan).
cudaError_t launch_kv_append(const AppendParams &a, int *status, cudaStream_t stream);

// Latent-head decode (Dk = 576, Dv = 512, row groups of 64 query heads):
// plan kernel + attention kernel + combine kernel, in stream order
cudaError_t launch_latent_decode(const DecodeParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                 const CUtensorMap &tm_v, cudaStream_t stream, cudaEvent_t timing_start,
                                 cudaEvent_t timing_stop, int *launches);
size_t latent_decode_smem_bytes();

// The same on CTA pairs (row groups of 128 query heads, cta_group::2 MMAs)
cudaError_t launch_latent_pair_decode(const DecodeParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                      const CUtensorMap &tm_v, cudaStream_t stream, cudaEvent_t timing_start,
                                      cudaEvent_t timing_stop, int *launches);
size_t latent_pair_decode_smem_bytes();

// Decode over an FP8 E4M3 KV cache (Dk = Dv = 128): plan + attention + combine
cudaError_t launch_decode_fp8(const DecodeParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                              const CUtensorMap &tm_v, cudaStream_t stream, cudaEvent_t timing_start,
                              cudaEvent_t timing_stop, int *launches);

// Speculative decoding: the drafts' attention, their masks, the step's page
// tables, the move of the accepted path
cudaError_t launch_tree_decode(const TreeParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                               const CUtensorMap &tm_v, cudaStream_t stream, int *launches);
cudaError_t launch_tree_decode_fp8(const TreeParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                   const CUtensorMap &tm_v, cudaStream_t stream, int *launches);
cudaError_t launch_tree_merge(const TreeParams &p, int row_tiles, cudaStream_t stream);
size_t tree_workspace_bytes(int head_dim, int grid);
void tree_place_workspace(TreeParams *p, void *ws);
cudaError_t launch_tree_mask(const TreeMaskParams &p, cudaStream_t stream);
cudaError_t launch_page_tables(const PageTableParams &p, cudaStream_t stream, int *launches);
cudaError_t launch_kv_commit(const CommitParams &p, cudaStream_t stream);
cudaError_t launch_chunk(const ChunkParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                         cudaStream_t stream, int *launches);
cudaError_t launch_chunk_pair(const ChunkParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                              const CUtensorMap &tm_v, cudaStream_t stream, int *launches);
cudaError_t launch_chunk_merge(const ChunkParams &p, cudaStream_t stream);
size_t chunk_workspace_bytes(int head_dim, int grid);
void chunk_place_workspace(ChunkParams *p, void *ws);
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream);
cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream);

// plan kernel + attention kernel, in stream order
cudaError_t launch_prefill(const PrefillParams &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                           const CUtensorMap &tm_v, int head_dim, cudaStream_t stream,
                           cudaEvent_t timing_start, cudaEvent_t timing_stop, int *launches);

}  // namespace fw
