// Internal interface of the operators that read or keep part of the paged cache: tree and sparse
// attention (attention.cu), page bounds, page scores and attention weights (key_scores.cu), page
// selection and eviction (select.cu).
#pragma once

#include "kernels.h"

namespace bdlm {

// What block attention takes beyond launch_attention's arguments.
struct AttnExt {
  bool tree = false;                     // the kernels that take a tree mask and write lse
  const uint64_t* tree_mask = nullptr;   // [B, L] visibility words, or null: every query sees all L
  float* lse = nullptr;                  // [B, L, Hq], or null
  bool head_tables = false;              // page_table holds a row per (sequence, KV head)
};

// Adapts a plan to lists that fill their tables (page selections).
void plan_even_lists(AttnPlan& pl, int B, int Hkv, int max_pages, int num_sms);
cudaError_t launch_attention_ext(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                 const CUtensorMap& tm_v, const int32_t* page_table,
                                 const int32_t* prefix_lens, uint16_t* out, int B, int L, int Hq,
                                 int Hkv, int max_pages, int num_pages, float sm_scale,
                                 const AttnPlan& plan, float* part, int* cnt, int* err,
                                 int num_sms, cudaStream_t stream, int table_div, int mask_block,
                                 const BlockKvWrite* kv_write, const AttnExt* ext);

// ------------------------------------------------------------------ key_scores.cu
constexpr int kKeyTile = 128;    // keys (tokens, or pages) per tile
constexpr int kAmaxPerTile = 8;  // page scores: largest |bound| of a tile, one value per warp

struct KeyParams {
  const int32_t* page_table;
  const int32_t* prefix_lens;
  int B, L, Hq, Hkv, G, max_pages, num_pages;
  int l0, rows;                // query rows l0 * G .. + rows of each (sequence, KV head)
  int max_tiles;               // tiles of the longest list the page table allows
  int* err;
  // attention weights
  const float* lse;            // [B, L, Hq]
  float* weights;              // [B, Hkv, max_pages * 16]
  float decay, scale_log2;
  // page scores
  const uint16_t* q;
  const uint16_t* bounds;      // [num_pages, Hkv, 2, 128]
  float* scores;               // [B, groups, Hkv, max_pages]
  float* amax;                 // [B, Hkv, max_tiles, kAmaxPerTile]
  int group, groups, width;    // positions per group, groups per sequence, query rows per group
};

int key_rows_max();   // query rows of one launch
cudaError_t launch_attention_weights(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                     const KeyParams& p, int num_sms, cudaStream_t stream);
// The maps are used for more than kDirectRows rows: tm_q as for attention weights, tm_bounds rows of
// 128 values, boxes of one row of 64.
constexpr int kDirectRows = 64;
cudaError_t launch_page_scores(const CUtensorMap& tm_q, const CUtensorMap& tm_bounds,
                               const KeyParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_page_bounds(const uint16_t* k_pages, const int32_t* page_table,
                               const int32_t* from, const int32_t* to, int B, int Hkv,
                               int max_pages, int num_pages, int num_sms, uint16_t* bounds,
                               int* err, cudaStream_t stream);

// ------------------------------------------------------------------ select.cu
struct SelectParams {
  const uint16_t* q;
  const uint16_t* bounds;
  const int32_t* page_table;
  const int32_t* prefix_lens;
  const float* scores;
  const float* amax;
  unsigned long long* exact;   // [B, groups, Hkv, max_pages]: near ties' scores, where they are many
  int B, L, Hq, Hkv, G, max_pages, num_pages, group, groups;
  int max_tiles;
  int n_select, sel_cols;
  int32_t* sel_table;
  int32_t* sel_lens;
  int* err;
};
constexpr int kSelectMaxPages = 262144;   // a list's page bitmap fits shared memory
// Whether launch_select_pages needs no scores (short lists that fill the GPU once at most): scores, amax
// and exact are not used then.
bool select_scores_itself(int lists, int max_pages, int rows, int num_sms);
cudaError_t launch_select_pages(const SelectParams& p, int num_sms, cudaStream_t stream);

struct EvictParams {
  const int32_t* lens;
  const float* weights;
  float* to_weights;
  int32_t* kept;       // [B, Hkv, keep]
  int32_t* new_lens;
  int B, Hkv, max_pages, keep, recent;
  int* err;
};
struct CompactParams {
  uint16_t* k_pages;
  uint16_t* v_pages;
  const int32_t* page_table;
  const int32_t* to_table;    // page_table itself: in place
  const int32_t* base;        // [B] first position, or null: 0
  const int32_t* idx;         // [B, heads, n_max]
  const int32_t* counts;      // [B]
  int B, Hkv, heads, max_pages, num_pages, n_max;
  int* err;
};
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);
// The choice and the move of what it keeps (m: base null, idx kept, counts new_lens, n_max keep).
cudaError_t launch_evict(const EvictParams& p, const CompactParams& m, int num_sms,
                         cudaStream_t stream);

}  // namespace bdlm
