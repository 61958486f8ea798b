// Internal interface of the operators on the cache's side of a step: page tables and slot maps, rotary
// positions (positions.cu), the 8-bit cache's writes (kv8.cu) and the attention over it (kv8_attention.cu).
#pragma once

#include "kernels.h"

namespace bdlm {

// ------------------------------------------------------------------ positions.cu
struct TableParams {
  const int32_t* old_lens;
  const int32_t* new_lens;
  const int32_t* free_pages;
  const int32_t* free_from;   // or null: 0
  int32_t* page_table;
  int32_t* lens_out;
  int32_t* first;             // [B + 1]
  int32_t* positions;         // [max_tokens], or null
  int32_t* slots;             // [max_tokens], or null
  int32_t* free_next;         // or null
  int2* plan;                 // [B]: tokens before the call, first page taken from the list
  int B, max_pages, num_pages, n_free, max_tokens;
  int* err;
};
cudaError_t launch_build_tables(const TableParams& p, cudaStream_t stream);

struct RotaryParams {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  long long q_stride, k_stride;   // elements from a token to the next
  const int32_t* start;           // [B]
  const int32_t* positions;       // [B, n], or null: start[b] + i
  int n, Hq, Hkv;
  long long rows;
  int inverse;
};
cudaError_t launch_rotary(const RotaryParams& p, const bdlm_rotary_desc& r, cudaStream_t stream);

// ------------------------------------------------------------------ kv8.cu
struct WriteKv8Params {
  const uint16_t* x[2];        // k_new, v_new
  uint8_t* pages[2];
  float* scales;
  const int32_t* first;        // [B + 1], or null: rows b * n
  const int32_t* page_table;
  const int32_t* prefix_lens;
  int B, n, n_rows, Hkv, max_pages, num_pages;
  int* err;
};
cudaError_t launch_write_kv8(const WriteKv8Params& p, cudaStream_t stream);

// ------------------------------------------------------------------ kv8_attention.cu
struct Kv8AttnParams {
  const uint16_t* q;
  const float* scales;
  const int32_t* page_table;
  const int32_t* prefix_lens;
  uint16_t* out;
  int B, L, Hq, Hkv, max_pages, num_pages;
  float scale_log2;
  int* err;
};
struct Kv8AttnPlan {
  int lsub, row_groups, rows;   // block positions and query rows of a row group
  int n_rows;                   // rows padded
  int grid;
  bool many_parts, join_here;   // join_here: by the attention kernel itself
  long long parts;
  size_t part_bytes, cum_offset, q_offset, q_scale_offset, bytes, work_bytes;   // of the workspace
};
Kv8AttnPlan plan_attention_kv8(int B, int L, int Hq, int Hkv, int max_pages, int num_sms);
// tm_k, tm_v: units of 16 x 128 bytes, boxes of one.  tm_q (n_rows >= 128): the parts of the queries at q_offset,
// [B * L][Hq][256] bytes, boxes of 128 bytes x G heads x lsub positions.  data: plan.bytes; work: plan.work_bytes,
// zero between calls.
cudaError_t launch_attention_kv8(const Kv8AttnParams& p, const Kv8AttnPlan& plan, const CUtensorMap& tm_q,
                                 const CUtensorMap& tm_k, const CUtensorMap& tm_v, void* data, int* work,
                                 cudaStream_t stream);

}  // namespace bdlm
