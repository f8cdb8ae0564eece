// pkv_paged_attention: argument checks and the choice of kernel.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "attend_params.h"
#include "kv_cache.cuh"
#include "page_kernels.h"

namespace {

size_t workspace_need(int max_q_len, int group, int head_dim) {
  const int sms = pkv::num_sms();
  size_t partials = pkv::row_partial_bytes(pkv::row_ctas(sms), head_dim);
  if (pkv::has_tiles(max_q_len, group))
    partials += pkv::tile_partial_bytes(pkv::tile_ctas(sms), head_dim);
  return pkv::kCounterBytes + partials;
}

}  // namespace

extern "C" {

size_t pkv_paged_attention_workspace_bytes(int B, int64_t n_tokens, int max_q_len, int q_heads,
                                           int kv_heads, int head_dim) {
  if (B < 0 || B > pkv::kMaxFillBatch || n_tokens < 0 || n_tokens > INT32_MAX || max_q_len < 1 ||
      kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || head_dim < 16 ||
      head_dim > PKV_MAX_HEAD_DIM)
    return 0;
  max_q_len = static_cast<int>(std::min<int64_t>(max_q_len, std::max<int64_t>(n_tokens, 1)));
  return workspace_need(max_q_len, q_heads / kv_heads, head_dim);
}

int pkv_paged_attention(const pkv_kv_cache* cache, const void* q, int64_t q_token_stride,
                        int64_t q_head_stride, int q_heads, pkv_dtype dt, int64_t n_tokens,
                        void* out, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                        const int32_t* cached_len, const int32_t* device_len,
                        const int32_t* table_idx, const int32_t* kv_begin, int B, int max_q_len,
                        const int32_t* page_table, int64_t pt_rows, int64_t pt_cols,
                        float sm_scale, int window, int32_t* status, void* workspace,
                        size_t workspace_bytes, pkv_stream_t stream) {
  using namespace pkv;
  int bad = cache_error(cache);
  if (bad != PKV_OK) return bad;
  if (dt != PKV_BF16 && dt != PKV_FP16)
    return fail(PKV_EINVAL, "dtype %d is not bf16 or fp16", static_cast<int>(dt));
  if (B < 0 || B > PKV_MAX_FILL_BATCH)
    return fail(PKV_EINVAL, "B=%d outside [0, %d]", B, PKV_MAX_FILL_BATCH);
  if (q_heads < 1 || q_heads > 65535 || q_heads % cache->kv_heads != 0)
    return fail(PKV_EINVAL, "q_heads=%d is not a multiple of kv_heads=%d in [1, 65535]", q_heads,
                cache->kv_heads);
  if (n_tokens < 0 || n_tokens > INT32_MAX / q_heads)
    return fail(PKV_EINVAL, "n_tokens=%lld: need 0 <= n_tokens * q_heads < 2^31",
                (long long)n_tokens);
  if (max_q_len < 1) return fail(PKV_EINVAL, "max_q_len=%d < 1", max_q_len);
  if (!std::isfinite(sm_scale)) return fail(PKV_EINVAL, "sm_scale is not finite");
  if (B == 0 || n_tokens == 0) return ok();
  if ((bad = rows_error("q", q, q_token_stride, q_head_stride)) != PKV_OK) return bad;
  if ((bad = rows_error("out", out, o_token_stride, o_head_stride)) != PKV_OK) return bad;
  if (cached_len == nullptr || device_len == nullptr || table_idx == nullptr ||
      page_table == nullptr)
    return fail(PKV_EINVAL, "NULL pointer argument");
  if (pt_rows < 1 || pt_cols < 1 || pt_cols > (int64_t{1} << 30))
    return fail(PKV_EINVAL, "page table shape [%lld, %lld]: need rows >= 1, columns in [1, 2^30]",
                (long long)pt_rows, (long long)pt_cols);
  max_q_len = static_cast<int>(std::min<int64_t>(max_q_len, n_tokens));
  const int group = q_heads / cache->kv_heads;
  const size_t need = workspace_need(max_q_len, group, cache->head_dim);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PKV_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned16(workspace)) return fail(PKV_EINVAL, "workspace is not 16-byte aligned");
  AttendParams P;
  P.c = *cache;
  P.page_div = Divider::by(static_cast<uint32_t>(cache->page_size));
  P.page_step = static_cast<uint32_t>(cache->page_stride / 16);
  P.token_step = static_cast<uint32_t>(cache->token_stride / 16);
  P.head_step = static_cast<uint32_t>(cache->head_stride / 16);
  P.q = static_cast<const uint16_t*>(q);
  P.out = static_cast<uint16_t*>(out);
  P.lse = lse;
  P.q_ts = q_token_stride, P.q_hs = q_head_stride;
  P.o_ts = o_token_stride, P.o_hs = o_head_stride;
  P.cached_len = cached_len;
  P.device_len = device_len;
  P.table_idx = table_idx;
  P.kv_begin = kv_begin;
  P.page_table = page_table;
  P.status = status;
  P.n_tokens = n_tokens;
  P.pt_rows = pt_rows, P.pt_cols = pt_cols;
  P.B = B;
  P.max_q_len = max_q_len;
  P.q_heads = q_heads;
  P.group = group;
  P.group_div = Divider::by(static_cast<uint32_t>(group));
  P.window = std::max(window, 0);
  P.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  P.bf16 = dt == PKV_BF16;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int sms = num_sms();
  uint32_t* counters = static_cast<uint32_t*>(workspace);
  if (!counters_fit(sms)) return fail(PKV_EUNSUPPORTED, "%d SMs", sms);
  float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  const bool tiles = has_tiles(max_q_len, group);
  // Alone, the row kernel takes the longer requests too: all of them are past
  // max_q_len, and get zeros.
  P.row_most = tiles ? kRowLimit : INT32_MAX;
  cudaError_t e = cudaSuccess;
  if (tiles) {
    P.counters = counters + row_counters(sms);
    P.partials = partials + row_partial_bytes(row_ctas(sms), cache->head_dim) / 4;
    e = launch_attend_tiles(P, tile_ctas(sms), st);
  }
  P.counters = counters;
  P.partials = partials;
  if (e == cudaSuccess)
    e = launch_attend_rows(P, row_ctas(sms), tiles, st);
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return ok();
}

}  // extern "C"
