// pkv_update_bounds: channelwise bounds of the keys of the pages that a step
// appended to.
//
// A run is the call's tokens of one page; its first token leads it, and the slots
// 0 .. the run's last are in use.  A warp takes a run of one head: a slot's row is
// read by LPR lanes of 16 codes each, 32 / LPR slots at a time, kept as fp16 pairs
// (which hold every code exactly and whose minimum and maximum are one instruction
// for two), and joined over the slots by shuffles.
//
// Bound: the keys' bytes, and with few tokens the chain of loads from a token's
// place to its page.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "attend_params.h"
#include "device_common.cuh"
#include "kv_cache.cuh"
#include "launch_early.h"

namespace pkv {

namespace {

constexpr int kWarps = 8;

struct BoundsParams {
  pkv_kv_cache c;
  Divider page_div;
  uint8_t* bounds;
  const int32_t* out_loc;
  const int64_t* total;
  int32_t* status;
  int64_t n_tokens;
  int window;  // tokens a warp looks at
};

__device__ __forceinline__ uint32_t min_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two fp16 values that are e4m3 values to their codes.
__device__ __forceinline__ uint32_t codes_of(uint32_t f16x2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(f16x2));
  return r;
}

template <int LPR>
__device__ __forceinline__ void bound_page(const BoundsParams& P, int page, int head, int slots) {
  const int lane = threadIdx.x & 31, sub = lane / LPR, ch = lane % LPR;
  const bool live = ch * 16 < P.c.head_dim;
  const uint8_t* src = static_cast<const uint8_t*>(P.c.k) + page * P.c.page_stride +
                       head * P.c.head_stride + ch * 16;
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = 0x7c007c00u, hi[i] = 0xfc00fc00u;  // +inf, -inf
  constexpr int kRows = 32 / LPR, kAhead = 4;
#pragma unroll 1
  for (int t = sub; t < slots; t += kRows * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      // (A slot that is not there: the first of these again.)
      const int at = t + a * kRows < slots ? t + a * kRows : t;
      if (live) v[a] = *reinterpret_cast<const uint4*>(src + at * P.c.token_stride);
    }
    if (live) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = e4m3x2_to_f16x2(w[i]), y = e4m3x2_to_f16x2(w[i] >> 16);
          lo[2 * i] = min_nan(lo[2 * i], x), hi[2 * i] = max_nan(hi[2 * i], x);
          lo[2 * i + 1] = min_nan(lo[2 * i + 1], y), hi[2 * i + 1] = max_nan(hi[2 * i + 1], y);
        }
      }
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(kFull, lo[i], o));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(kFull, hi[i], o));
    }
  }
  if (live && sub < 2) {
    uint4 out;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = sub == 0 ? lo[2 * i] : hi[2 * i], b = sub == 0 ? lo[2 * i + 1] : hi[2 * i + 1];
      w[i] = codes_of(a) | codes_of(b) << 16;
    }
    out = make_uint4(w[0], w[1], w[2], w[3]);
    uint8_t* dst = P.bounds + (static_cast<int64_t>(page) * P.c.kv_heads + head) * 2 * P.c.head_dim;
    *reinterpret_cast<uint4*>(dst + sub * P.c.head_dim + ch * 16) = out;
  }
}

template <int LPR>
__global__ void __launch_bounds__(kWarps * 32) bounds_kernel(const __grid_constant__ BoundsParams P) {
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t n = P.total != nullptr ? max(int64_t{0}, min(P.n_tokens, *P.total)) : P.n_tokens;
  const int64_t j0 = item / P.c.kv_heads * P.window;
  const int head = static_cast<int>(item % P.c.kv_heads);
  if (j0 >= n) return;
  const int slots = static_cast<int>(P.c.num_pages * P.c.page_size);
  auto page_of = [&](int loc) {
    return loc >= 0 && loc < slots
               ? static_cast<int>(P.page_div.divide(static_cast<uint32_t>(loc))) : -1;
  };
  const int64_t j = j0 + lane;
  const int loc = j < n ? P.out_loc[j] : -1;
  const int prior = j < n && j > 0 ? P.out_loc[j - 1] : -1;
  const int page = page_of(loc);
  const bool mine = lane < P.window && j < n;
  if (mine && page < 0 && head == 0 && P.status != nullptr) atomicOr(P.status, PKV_ST_ROW_OOB);
  // The page before a token's; a token that is skipped parts no run, so behind some the warp
  // looks for it 32 at a time (behind 70000: 0.5 ms, a lane for itself 3.9).
  int before = page_of(prior);
  unsigned behind = __ballot_sync(kFull, mine && page >= 0 && before < 0 && j > 1);
#pragma unroll 1
  while (behind != 0u) {
    const int l = __ffs(behind) - 1;
    behind &= behind - 1u;
    int found = -1;
#pragma unroll 1
    for (int64_t k = j0 + l - 2; k >= 0 && found < 0; k -= 32) {
      const int p = k >= lane ? page_of(P.out_loc[k - lane]) : -1;
      const unsigned held = __ballot_sync(kFull, p >= 0);
      if (held != 0u) found = __shfl_sync(kFull, p, __ffs(held) - 1);
    }
    if (lane == l) before = found;
  }
  unsigned leads = __ballot_sync(kFull, mine && page >= 0 && before != page);
#pragma unroll 1
  while (leads != 0u) {
    const int l = __ffs(leads) - 1;
    leads &= leads - 1u;
    const int p = __shfl_sync(kFull, page, l);
    // The run's last token: among the lanes from l on, or further on.
    int last = 0, now = page, at = loc;
    unsigned from = kFull << l;
#pragma unroll 1
    for (int64_t k = j0;;) {
      const unsigned ends = __ballot_sync(kFull, k + lane >= n || (now >= 0 && now != p)) & from;
      const unsigned here = ends != 0u ? (ends & (0u - ends)) - 1u : kFull;  // below the first end
      const unsigned held = __ballot_sync(kFull, now == p) & here & from;
      if (held != 0u) last = __shfl_sync(kFull, at, 31 - __clz(held));
      if (ends != 0u) break;
      k += 32;
      from = kFull;
      at = k + lane < n ? P.out_loc[k + lane] : -1;
      now = page_of(at);
    }
    bound_page<LPR>(P, p, head, last - p * P.c.page_size + 1);
  }
}

}  // namespace

}  // namespace pkv

extern "C" int pkv_update_bounds(const pkv_kv_cache* cache, void* bounds, const int32_t* out_loc,
                                 int64_t n_tokens, const int64_t* total_tokens, int32_t* status,
                                 pkv_stream_t stream) {
  using namespace pkv;
  const int bad = cache_error(cache);
  if (bad != PKV_OK) return bad;
  if (n_tokens < 0 || n_tokens > INT32_MAX)
    return fail(PKV_EINVAL, "n_tokens=%lld outside [0, 2^31)", (long long)n_tokens);
  if (n_tokens == 0) return ok();
  if (bounds == nullptr || out_loc == nullptr) return fail(PKV_EINVAL, "NULL pointer argument");
  if (!aligned16(bounds)) return fail(PKV_EINVAL, "bounds are not 16-byte aligned");
  BoundsParams P;
  P.c = *cache;
  P.page_div = Divider::by(static_cast<uint32_t>(cache->page_size));
  P.bounds = static_cast<uint8_t*>(bounds);
  P.out_loc = out_loc;
  P.total = total_tokens;
  P.status = status;
  P.n_tokens = n_tokens;
  // Windows of 16 tokens hold about a run each of a long prompt's pages; with few
  // tokens each may be a run, and a warp takes one.
  const int64_t warps = static_cast<int64_t>(num_sms()) * 64;
  P.window = 1;
  while (P.window < 16 && div_ceil(n_tokens, 2 * P.window) * cache->kv_heads >= warps) P.window *= 2;
  const int64_t items = div_ceil(n_tokens, P.window) * cache->kv_heads;
  if (div_ceil(items, kWarps) > INT32_MAX)
    return fail(PKV_EINVAL, "%lld tokens of %d heads are too many", (long long)n_tokens,
                cache->kv_heads);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_early(cache->head_dim > 64 ? bounds_kernel<8> : bounds_kernel<4>,
                                     dim3(static_cast<unsigned>(div_ceil(items, kWarps))),
                                     kWarps * 32, 0, s, P);
  if (e != cudaSuccess) return cuda_fail(e, "bounds launch");
  return ok();
}
