// Declarations shared by the library's translation units (not part of the ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "chunk_plan.h"

namespace tpl {

constexpr int kStatusCapacity = -5;

// A launch that may be scheduled before the grid in front of it has completed (programmatic
// serialisation). Its kernel executes griddepcontrol.wait in every thread that goes on, before
// it reads or writes anything in global memory, so that results are those of stream order, and
// reads what other kernels wrote with coherent loads: one through a const __restrict__ pointer
// or __ldg counts as invariant and may be moved above the wait.
inline cudaLaunchConfig_t programmatic(dim3 grid, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// ---------------------------------------------------------------- capture
constexpr int kCaptureMaxTensors = 8;
struct CaptureMeta {
  const __nv_bfloat16* tensors[kCaptureMaxTensors];
  int32_t types[kCaptureMaxTensors];
  int32_t n_tensors;
  int32_t layer;
  int32_t* hdr;        // [capacity][6]
  void* rows_out;      // [capacity][H] bf16
};

cudaError_t launch_capture(int T, int H, const int32_t* row_req, const int32_t* row_pos,
                           const int64_t* sel, int n_sel, uint64_t* gtable, int cap_log2,
                           size_t table_smem, const CaptureMeta& meta, int64_t capacity,
                           int64_t* n_out_dev, int32_t* match_rows, int32_t* n_match_ws, int* status,
                           int copy_grid, cudaStream_t st);

// ---------------------------------------------------------------- RMSNorm
cudaError_t launch_add_rms_norm(int T, int H, const void* a, const void* res, const void* gamma,
                                float eps, void* res_out, void* x_out, cudaStream_t st);
int max_norm_hidden();

// ---------------------------------------------------------------- packing
// Weights are packed as blocks of 256 rows x 64 K elements (32 KB) in the
// 128-byte-swizzled K-major image the MMA reads; block (w_tile, kb) sits at
// (w_tile * nkb + kb) * 32 KB. Rows or K past the end are zero.
enum PackMode : int { PACK_GATE_UP = 0, PACK_ROW = 1, PACK_QKV = 2 };
struct PackSpec {
  int mode;
  const __nv_bfloat16* src[3];
  int64_t H;       // hidden: K of the column kinds, output rows of PACK_ROW
  int64_t Is;      // PACK_GATE_UP: rows per shard; PACK_ROW: K per shard
  int64_t t;
  int64_t nb;      // PACK_GATE_UP: 128-row blocks per shard
  int64_t nkb;     // k-blocks per weight tile
  int64_t kbs;     // PACK_ROW: k-blocks per shard
  int64_t n_col;   // PACK_QKV: packed rows in total
  int64_t ws;      // PACK_QKV: packed rows per shard
  int q_per, kv_per, rep, hd;
};
cudaError_t launch_pack(const PackSpec& s, int64_t n_blocks, void* dst, cudaStream_t st);

// ---------------------------------------------------------------- attention core
struct AttnParams {
  const int4* pairs;       // [n_pairs] {sequence start, length, q tile, 0}, heaviest first
  const int* n_pairs;      // written by the preparation kernel
  int* next_unit;          // units handed out so far (CTAs take the next one when free); zeroed by the preparation kernel
  __nv_bfloat16* out;      // shard r, token m at out + r * out_sstride + m * out_rstride
  long long out_sstride;   // [t][T][q_per * 128]: T * q_per * 128; gathered [T][t * q_per * 128]: q_per * 128
  int out_rstride;         // q_per * 128, or t * q_per * 128 gathered
  int* status;
  unsigned long long timeout_ns;
  int T, q_per, kv_per, rep, group, heads;  // group = nq / nkv, heads = t * q_per
  float scale_log2;        // log2(e) / sqrt(hd)
  int out_align32;         // out is 32-byte aligned (rows are then written with 32-byte stores)
};
// Builds the (sequence, q tile) table from cu_seqlens (device) into `pairs` and
// runs the attention kernel on `grid` CTAs; map_qkv covers qkv as
// (w_s, T, t, 1) with 64 x 128 boxes.
cudaError_t launch_attention(const CUtensorMap& map_qkv, const AttnParams& p, const int* cu, int n_seqs,
                             int max_tiles, int4* pairs, int* n_pairs, int grid, cudaStream_t st);

// ---------------------------------------------------------------- GEMM
struct GemmParams;
// Launch the GEMM instantiation for (swap, kind, bn); cudaErrorInvalidValue
// when no such instantiation exists.
cudaError_t launch_gemm(bool swap, int kind, int bn, const CUtensorMap& map_act, const GemmParams& p,
                        int grid, cudaStream_t st);
int gemm_stages(bool swap, int kind, int bn);
struct MlpDecodeParams;
// The fused decode-shaped MLP block (T <= 128): one launch.
cudaError_t launch_mlp_decode(int bn, const CUtensorMap& map_x, const CUtensorMap& map_h,
                              const MlpDecodeParams& P, int grid, cudaStream_t st);
// CTAs of the fused kernel that fit on one SM (0 when it cannot run on this device).
int mlp_decode_ctas_per_sm(int bn);

// Paged KV cache (kv_cache.cu).
struct PagedAttnParams {
  const __nv_bfloat16* qkv;          // new tokens: shard r, token i at qkv + r * sstride_in + i * rstride_in
  long long sstride_in;
  int rstride_in;
  const int* qsl;                    // [n_reqs + 1] new-token offsets
  const int* seq_lens;               // [n_reqs] tokens of each request, new ones included
  const int* block_tables;           // [n_reqs][max_blocks]
  const int* slots;                  // [T] cache slot of each new token, written before it is read (null: none)
  long long n_slots;                 // num_blocks * block_size
  __nv_bfloat16* cache_k;            // [t][num_blocks][block_size][kv_per][128]
  __nv_bfloat16* cache_v;
  __nv_bfloat16* out;                // shard r, token i at out + r * sstride_out + i * rstride_out
  long long sstride_out;
  int rstride_out;
  float* partials;                   // [item][q_stride][128 + 2]: o, max, sum of each split
  int* status;
  int t, q_per, kv_per, rep, max_blocks, num_blocks, block_size, max_query_len, max_seq_len;
  int split_len, n_splits;           // keys per split, splits per (request, shard, kv head)
  int q_stride;                      // query slots of one item: max_query_len * (q heads per kv head)
  float scale_log2;
};
cudaError_t launch_kv_write(const void* qkv, int T, int t, long long sstride, int rstride, int q_per, int kv_per,
                            const int* slots, long long n_slots, void* ck, void* cv, int* status, int nsm,
                            cudaStream_t st);
cudaError_t launch_paged_attention(const PagedAttnParams& p, int n_reqs, cudaStream_t st);

// Rotary positions (rope.cu).
constexpr int kRopeMaxDim = 256;
struct RopeFreqs {
  double inv_freq[kRopeMaxDim / 2];
  double scale;                      // multiplies cos and sin
};
struct RopeParams {
  const __nv_bfloat16* in;           // shard r, token i at in + r * sstride + i * rstride (out likewise)
  __nv_bfloat16* out;
  long long sstride;
  int rstride;
  const int* pos;                    // [T]
  const float* table;                // [n_pos][rd]: cos, then sin, of each pair
  long long n_pos;
  const __nv_bfloat16* q_gamma;      // [hd] or null
  const __nv_bfloat16* k_gamma;
  float eps;
  const int* slots;                  // [T] or null: no cache write
  long long n_slots;
  __nv_bfloat16* cache_k;
  __nv_bfloat16* cache_v;
  int* status;
  int T, t, q_per, kv_per, hd, rd, interleaved;
};
cudaError_t launch_rope_table(const RopeFreqs& f, long long n_pos, int rotary_dim, float* table, int nsm, cudaStream_t st);
cudaError_t launch_qk_norm_rope(const RopeParams& p, int nsm, cudaStream_t st);

// Pages moved inside the cache (kv_pages.cu), the caches of all layers in one launch.
constexpr int kMaxKvLayers = 128;
struct KvLayers {
  void* k[kMaxKvLayers];
  void* v[kMaxKvLayers];
};
struct CompactParams {
  const int* qsl;                    // [n_reqs + 1]
  const int* seq_lens;               // [n_reqs], drafted tokens included
  const int* accepted;               // [n_reqs][max_accepted] rising draft indices, ended by a negative one
  const int* src_tables;             // [n_reqs][max_blocks]
  const int* dst_tables;
  int* new_lens;                     // [n_reqs]
  int* status;
  long long n_slots;                 // num_blocks * block_size
  int t, kv_per, max_blocks, num_blocks, block_size, max_accepted;
};
cudaError_t launch_kv_copy_blocks(const KvLayers& layers, int n_layers, const int* pairs, int n_pairs,
                                  long long num_blocks, int block_size, int kv_per, int t, int* status, cudaStream_t st);
cudaError_t launch_kv_compact(const KvLayers& layers, int n_layers, const CompactParams& p, int n_reqs, int nsm,
                              cudaStream_t st);

// Attention of drafted token trees over the cache (tree_attention.cu).
struct TreeItem {
  int r, g, row0, rows, q0, last, pad0, pad1;   // rows 0: none; last: the last CTA that holds a part
};
struct TreeAttnParams {
  const __nv_bfloat16* qkv;          // drafted tokens: shard r, token i at qkv + r * sstride_in + i * rstride_in
  long long sstride_in;
  int rstride_in;
  const int* qsl;                    // [n_reqs + 1]
  const int* seq_lens;               // [n_reqs], drafted tokens included
  const int* block_tables;           // [n_reqs][max_blocks]
  const int* mask;                   // [T][mask_words]
  const __nv_bfloat16* cache_k;      // [t][num_blocks][block_size][kv_per][128]
  const __nv_bfloat16* cache_v;
  __nv_bfloat16* out;                // shard r, token i at out + r * sstride_out + i * rstride_out
  long long sstride_out;
  int rstride_out;
  int* status;
  int T, n_reqs, t, q_per, kv_per, max_blocks, num_blocks, block_size, max_query_len, max_seq_len, mask_words;
  float scale_log2;                  // log2(e) / sqrt(hd)
  TreeItem* items;                   // [grid] the item each CTA begins and others go on with, for the merge
  float* partials;                   // [2 * grid] slots of part_rows x (128 + 2)
  int part_rows;
  int out_align32;                   // out is 32-byte aligned (rows are then written with 32-byte stores)
  unsigned long long timeout_ns;
};
int tree_group_rows(int max_rows);   // query rows of one item: 128 or 256
cudaError_t launch_tree_mask(int T, int n_reqs, int max_query_len, int words, const int* parents, const int* qsl,
                             const int* seq_lens, int* mask, int* positions, int* status, cudaStream_t st);
cudaError_t launch_tree_attention(const TreeAttnParams& p, int grid, cudaStream_t st);

// Attention of chunks of new tokens over the cache (chunk_attention.cu).
struct ChunkAttnParams {
  ChunkCall call;                    // bounds, groups, window and sinks
  const __nv_bfloat16* qkv;          // new tokens: shard r, token i at qkv + r * sstride_in + i * rstride_in
  long long sstride_in;
  int rstride_in;
  const int* qsl;                    // [n_reqs + 1]
  const int* seq_lens;               // [n_reqs], new tokens included
  const int* block_tables;           // [n_reqs][max_blocks]
  const void* cache_k;               // [t][num_blocks][block_size][kv_per][128] bf16, or e4m3 codes
  const void* cache_v;
  const uint8_t* scales_k;           // [t][num_blocks][block_size][kv_per] of codes; null: the caches are bf16
  const uint8_t* scales_v;
  __nv_bfloat16* out;                // shard r, token i at out + r * sstride_out + i * rstride_out
  long long sstride_out;
  int rstride_out;
  int* status;
  int n_reqs, t, kv_per, max_blocks, num_blocks, block_size;
  unsigned block_magic;              // 2^32 / block_size rounded up (not used for 1)
  float scale_log2;                  // log2(e) / sqrt(hd)
  unsigned* counters;                // [SMs][8] parts that are there, of the item that a CTA begins; 0 between calls. Null: a kernel joins them
  TreeItem* items;                   // [grid] the item each CTA begins and others go on with, for that kernel
  float* partials;                   // [2 * grid] slots of part_rows x (128 + 2)
  int group_rows;                    // query rows of a group: up to 8, 128 or 256
  int part_rows;
  int q_box_rows;                    // rows of a box of the map of the queries
  int out_align32;                   // out is 32-byte aligned (rows are then written with 32-byte stores)
  unsigned long long timeout_ns;
};
// Query rows of a group of a call; many: it has an item for every SM; max_keys: the most that a token sees.
int chunk_group_rows(int max_rows, bool q8, bool many, int max_keys);
int chunk_decode_ctas(bool q8);      // CTAs per SM of the kernel for up to 8 rows (chunk_decode.cu)
cudaError_t launch_chunk_decode(const ChunkAttnParams& p, int grid, cudaStream_t st);
cudaError_t launch_chunk_attention(const CUtensorMap& map_q, const ChunkAttnParams& p, int grid, cudaStream_t st);

// A cache in 8 bits (kv_quant.cu).
struct KvQuantParams {
  const __nv_bfloat16* qkv;          // write: shard r, token i at qkv + r * sstride + i * rstride
  long long sstride;
  int rstride;
  const int* slots;                  // [n]
  long long n_slots;                 // num_blocks * block_size
  uint8_t* codes[2];                 // k, v: [t][n_slots][kv_per][128] e4m3
  uint8_t* scales[2];                // [t][n_slots][kv_per]
  __nv_bfloat16* out[2];             // read: [t][n][kv_per][128]
  int* status;
  int n, t, q_per, kv_per;
};
cudaError_t launch_kv_quant_write(const KvQuantParams& p, cudaStream_t st);
cudaError_t launch_kv_quant_read(const KvQuantParams& p, int nsm, cudaStream_t st);

// Mixture of experts (moe.cu): routing sort, row gather, weighted combine.
cudaError_t launch_moe_route(const int* ids, int n_entries, int k, int E, int max_rows, int* rank, int* perm_row,
                             int* row_src, int* tile_expert, int* m_valid, int* pair_tiles, int* pair_count,
                             int* status, cudaStream_t st);
cudaError_t launch_moe_gather(const void* x, int H, const int* row_src, const int* m_valid, int max_rows,
                              void* x_perm, int nsm, cudaStream_t st);
cudaError_t launch_moe_combine(const void* y_perm, int H, int T, int k, const int* perm_row, const float* gates,
                               void* y, int nsm, cudaStream_t st);

}  // namespace tpl
