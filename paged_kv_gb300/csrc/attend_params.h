// Host-side declarations of pkv_paged_attention's launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/pkv.h"

namespace pkv {

struct AttendParams {
  pkv_kv_cache c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;                  // or nullptr
  int64_t q_ts, q_hs, o_ts, o_hs;
  const int32_t* cached_len;   // [B]
  const int32_t* device_len;   // [B]
  const int32_t* table_idx;    // [B]
  const int32_t* kv_begin;     // [B] or nullptr
  const int32_t* page_table;   // [pt_rows, pt_cols]
  int32_t* status;             // or nullptr
  int64_t n_tokens;
  int64_t pt_rows, pt_cols;
  int B, max_q_len;
  int q_heads, group;          // group: query heads per cache head
  int window;                  // 0: none
  float scale_log2;            // sm_scale * log2(e)
  bool bf16;
  // Workspace: one counter per CTA, then two partial results per CTA.
  uint32_t* counters;
  float* partials;
};

// Rows (query token, query head of one cache head) per block of the row
// kernel, and its CTAs.
struct RowShape {
  int rows;      // 8 or 16
  int max_ctas;
};
RowShape row_shape(int max_q_len, int group, int num_sms);
// Workspace bytes of the row kernel.
size_t row_workspace_bytes(const RowShape& s, int head_dim);
cudaError_t launch_attend_rows(const AttendParams& P, const RowShape& s, cudaStream_t stream);

}  // namespace pkv
