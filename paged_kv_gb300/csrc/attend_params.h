// Host-side declarations of pkv_paged_attention's launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/pkv.h"

namespace pkv {

// Division of 31-bit numbers by a constant: floor(x / d) = (x * mul) >> (31 + shift)
// with shift = ceil(log2 d), mul = ceil(2^(31 + shift) / d) < 2^32.  (Write
// mul d = 2^(31 + shift) + e with 0 <= e < d <= 2^shift: x e < 2^(31 + shift),
// so x mul / 2^(31 + shift) exceeds x / d by less than 1 / d.)
struct Divider {
  uint32_t mul, shift;
  static Divider by(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t{1} << s) < d) ++s;
    return {static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + d - 1) / d), 31 + s};
  }
#ifdef __CUDACC__
  __device__
#endif
  uint32_t divide(uint32_t x) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(x) * mul) >> shift);
  }
};

struct AttendParams {
  pkv_kv_cache c;
  Divider page_div;            // by c.page_size
  Divider group_div;           // by group
  uint32_t page_step, token_step, head_step;  // c's strides in 16 bytes
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
  int row_most;                // rows of a request that the row kernel still takes
  int window;                  // 0: none
  float scale_log2;            // sm_scale * log2(e)
  bool bf16;
  uint32_t* counters;          // the kernel's workspace: one counter per CTA,
  float* partials;             // then two partial results per CTA
};

// Requests of up to kRowLimit query rows a cache head go to the row kernel,
// longer ones to the tile kernel, whose units cost the same for 1 as for 128
// rows.  Row and tile kernel: 256 requests of 16 rows 258 and 496 us, of 32 479
// and 502; 16 long ones of 16 rows 113 and 192, of 32 194 and 196.
constexpr int kRowLimit = 32;
inline bool has_tiles(int max_q_len, int group) {
  return static_cast<int64_t>(max_q_len) * group > kRowLimit;
}

// The workspace begins with both kernels' counters, at places that depend on
// the device alone, so that calls of any shape can follow one another on it.
// The partial results come after, the row kernel's first: the kernels run side
// by side.
constexpr int kRowCtasPerSm = 3, kRowWarps = 4;
inline int row_ctas(int num_sms) { return num_sms * kRowCtasPerSm; }
inline int row_counters(int num_sms) { return 3 * kRowWarps * row_ctas(num_sms); }
inline int tile_ctas(int num_sms) { return num_sms; }
constexpr size_t kCounterBytes = PKV_ATTENTION_ZERO_BYTES;  // enough for 431 SMs
inline bool counters_fit(int num_sms) {
  return static_cast<size_t>(row_counters(num_sms) + 2 * tile_ctas(num_sms)) * 4 <= kCounterBytes;
}

// Bytes of the kernels' partial results.
size_t row_partial_bytes(int ctas, int head_dim);
size_t tile_partial_bytes(int ctas, int head_dim);

// beside: the launch before it on the stream is the same call's tile kernel, and
// the two may run side by side.
cudaError_t launch_attend_rows(const AttendParams& P, int ctas, bool beside, cudaStream_t stream);
cudaError_t launch_attend_tiles(const AttendParams& P, int ctas, cudaStream_t stream);

}  // namespace pkv
