// pkv_append_kv: a step's keys and values, rotated and rounded to e4m3, into
// the paged cache.
//
//   k' = R(p) k,  a = max |k'| over the call's tokens of a (page, head),
//   s = 2^e least with a <= 448 s,  code = rn_e4m3(k' / s)
//
// A run is the call's tokens of one page; its first token leads it.  One warp
// owns one (run, head, k or v): it alone reads and writes that page's scale
// and codes of that head, so nothing is shared between warps and a run's
// result does not depend on the launch.  A head's row is spread over the lanes
// in quads (4 elements, 8 bytes in, 4 bytes out); the rotate-half partner of
// a quad lies a fixed number of lanes away and comes by one shuffle.  A run of
// up to kHold tokens is loaded at once and stays in registers, unrotated,
// between the maximum and the rounding: turning it twice costs less than the
// registers of turned values, which would halve the warps that keep loads in
// flight.  A longer run is read a second time, from L2.
//
// Bound: bytes, and with few tokens the two dependent loads (a token's place,
// then what the place needs).
//
// e4m3 keeps its relative precision over 2^-6 .. 448, so a power-of-two scale
// costs nothing against a tight one and lets a page's scale grow later
// without a second rounding error (but for subnormals).

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "device_common.cuh"
#include "kv_cache.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kHold = 16;    // tokens of a run held in registers
constexpr int kQHeads = 8;   // query heads a warp rotates together
constexpr int kMaxWindow = 16;
constexpr int kMinExp = -64, kMaxExp = 119;

struct AppendParams {
  pkv_kv_cache c;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  uint16_t* q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, o_ts, o_hs;
  const int32_t* positions;
  const int32_t* out_loc;
  const float* cos_sin;
  const int64_t* total;
  int32_t* status;
  int64_t n_tokens;
  int64_t max_pos;
  int64_t kv_blocks;
  int rot, q_heads, window;
};

// The angle's cosines and sines for this lane's quad.
struct Turn {
  float c[4], s[4];
};

template <bool INTER>
__device__ __forceinline__ Turn load_turn(const AppendParams& P, int64_t pos, int lane) {
  Turn t;
  const int half = P.rot >> 1;
  const float* row = P.cos_sin + pos * P.rot;
  if (INTER) {
    if (lane * 4 < P.rot) {
      const float2 c = *reinterpret_cast<const float2*>(row + 2 * lane);
      const float2 s = *reinterpret_cast<const float2*>(row + half + 2 * lane);
      t.c[0] = t.c[1] = c.x;
      t.c[2] = t.c[3] = c.y;
      t.s[0] = -s.x, t.s[1] = s.x, t.s[2] = -s.y, t.s[3] = s.y;
      return t;
    }
  } else if (lane * 4 < P.rot) {
    const bool second = lane * 4 >= half;
    const int i = lane * 4 - (second ? half : 0);
    const float4 c = *reinterpret_cast<const float4*>(row + i);
    const float4 s = *reinterpret_cast<const float4*>(row + half + i);
    t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
    t.s[0] = second ? s.x : -s.x;
    t.s[1] = second ? s.y : -s.y;
    t.s[2] = second ? s.z : -s.z;
    t.s[3] = second ? s.w : -s.w;
    return t;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t.c[i] = 1.0f, t.s[i] = 0.0f;
  return t;
}

// Rotates this lane's quad; every lane of the warp takes part.
template <bool INTER>
__device__ __forceinline__ float4 rotate(const AppendParams& P, float4 x, const Turn& t, int lane) {
  float4 y;
  if (INTER) {
    y = make_float4(x.y, x.x, x.w, x.z);
  } else {
    const int quads = P.rot >> 3;  // quads in each half
    int from = lane;
    if (lane < quads) from = lane + quads;
    else if (lane < 2 * quads) from = lane - quads;
    y.x = __shfl_sync(kFull, x.x, from);
    y.y = __shfl_sync(kFull, x.y, from);
    y.z = __shfl_sync(kFull, x.z, from);
    y.w = __shfl_sync(kFull, x.w, from);
  }
  // Elements past rot_dim have t.s = 0 and must not pick up 0 * inf.
  if (lane * 4 < P.rot) {
    x.x = fmaf(x.x, t.c[0], y.x * t.s[0]);
    x.y = fmaf(x.y, t.c[1], y.y * t.s[1]);
    x.z = fmaf(x.z, t.c[2], y.z * t.s[2]);
    x.w = fmaf(x.w, t.c[3], y.w * t.s[3]);
  }
  return x;
}

template <typename T>
__device__ __forceinline__ float4 unpack4(uint2 raw) {
  const float2 a = Pair<T>::unpack(raw.x), b = Pair<T>::unpack(raw.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

// Least 2^e with a <= 448 * 2^e.  448 = 1.75 * 2^8, so e is the exponent of a
// minus 8, and one more where a's significand is above 1.75.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(kMinExp, min(kMaxExp, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float finite_mag(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;  // NaN and infinities do not count
}

__device__ __forceinline__ float max4(float4 x) {
  return fmaxf(fmaxf(finite_mag(x.x), finite_mag(x.y)), fmaxf(finite_mag(x.z), finite_mag(x.w)));
}

__device__ __forceinline__ bool finite4(float4 x) {
  return isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w);
}

// A divisor that multiplies where it can: powers of two (every scale this
// kernel makes) by their exact reciprocal, other scales by division.
struct Divide {
  float s, inv;
  bool power;
  __device__ explicit Divide(float scale) {
    s = scale;
    inv = 1.0f / scale;
    power = (__float_as_uint(scale) & 0x7fffffu) == 0u;
  }
  __device__ __forceinline__ uint32_t codes(float4 x) const {
    if (power) {
      x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
    } else {
      x.x /= s, x.y /= s, x.z /= s, x.w /= s;
    }
    return e4m3x2(x.x, x.y) | (e4m3x2(x.z, x.w) << 16);
  }
};

// Rounds the page's codes before slot `first` from one scale to a larger one.
__device__ __forceinline__ void regrow(uint8_t* dst, int64_t token_stride, int first, float before,
                                       float now, bool live) {
  const float ratio = before / now;
  for (int t = 0; t < first; ++t) {
    if (live) {
      uint32_t* at = reinterpret_cast<uint32_t*>(dst + t * token_stride);
      const uint32_t old = *at;
      const float2 x = Pair<__half>::unpack(e4m3x2_to_f16x2(old));
      const float2 y = Pair<__half>::unpack(e4m3x2_to_f16x2(old >> 16));
      *at = e4m3x2(x.x * ratio, x.y * ratio) | (e4m3x2(y.x * ratio, y.y * ratio) << 16);
    }
  }
}

// What one warp needs of its (page, head, k or v).
struct Target {
  const uint16_t* src;
  int64_t ts;
  uint8_t* dst;
  float* scale;
  bool turning, live;
};

__device__ __forceinline__ Target target(const AppendParams& P, int page, int head, bool is_v,
                                         int lane) {
  const pkv_kv_cache& C = P.c;
  Target t;
  t.src = (is_v ? P.v + head * P.v_hs : P.k + head * P.k_hs) + lane * 4;
  t.ts = is_v ? P.v_ts : P.k_ts;
  t.dst = static_cast<uint8_t*>(is_v ? C.v : C.k) + page * C.page_stride + head * C.head_stride +
          lane * 4;
  t.scale = (is_v ? C.v_scale : C.k_scale) + static_cast<int64_t>(page) * C.kv_heads + head;
  t.turning = !is_v && P.rot > 0;
  t.live = lane * 4 < C.head_dim;
  return t;
}

// A run of at most kHold tokens.  Lane l holds token w0 + l's slot in the page
// (-1: not written) and position; the run's tokens are j0 .. j0 + cnt - 1,
// j0 = w0 + at.
template <typename T, bool INTER>
__device__ __forceinline__ void append_held(const AppendParams& P, const Target& D, int64_t j0,
                                            int at, unsigned valid, int slot, int pos, int lane) {
  if (valid == 0u) return;
  const float before = *D.scale;
  uint2 raw[kHold];
#pragma unroll
  for (int t = 0; t < kHold; ++t) {
    raw[t] = make_uint2(0u, 0u);
    if (((valid >> t) & 1u) != 0u && D.live)
      raw[t] = *reinterpret_cast<const uint2*>(D.src + (j0 + t) * D.ts);
  }
  auto value = [&](int t) -> float4 {
    float4 x = unpack4<T>(raw[t]);
    if (D.turning) {
      const Turn turn = load_turn<INTER>(P, __shfl_sync(kFull, pos, at + t), lane);
      x = rotate<INTER>(P, x, turn, lane);
    }
    return x;
  };
  float amax = 0.0f;
  bool fine = true;
#pragma unroll
  for (int t = 0; t < kHold; ++t) {
    if ((valid >> t) & 1u) {
      const float4 x = value(t);
      amax = fmaxf(amax, max4(x));
      fine = fine && finite4(x);
    }
  }
  amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
  const float want = scale_for(amax);
  const int first = __shfl_sync(kFull, slot, at + __ffs(valid) - 1);
  const float now = first == 0 ? want : fmaxf(before, want);
  if (first > 0 && now != before) regrow(D.dst, P.c.token_stride, first, before, now, D.live);
  const Divide div(now);
#pragma unroll
  for (int t = 0; t < kHold; ++t) {
    if ((valid >> t) & 1u) {
      const float4 x = value(t);
      const int o = __shfl_sync(kFull, slot, at + t);
      if (D.live) *reinterpret_cast<uint32_t*>(D.dst + o * P.c.token_stride) = div.codes(x);
    }
  }
  if (lane == 0) *D.scale = now;
  if (!__all_sync(kFull, fine) && lane == 0 && P.status != nullptr)
    atomicOr(P.status, PKV_ST_NONFINITE);
}

// A run of any length that begins at token j0, read twice.
template <typename T, bool INTER>
__device__ __noinline__ void append_long(const AppendParams& P, const Target& D, int64_t n,
                                         int64_t j0, int page, int lane) {
  const int ps = P.c.page_size;
  const int64_t slots = P.c.num_pages * ps;
  const float before = *D.scale;
  // The run's tokens from `base` on, 32 at a time: lane l holds base + l's
  // slot (-1: not written) and position.  Returns how many are in the run.
  int slot = -1, pos = 0;
  auto scan = [&](int64_t base) -> int {
    const int64_t j = base + lane;
    bool in_run = false;
    slot = -1;
    if (j < n) {
      const int loc = P.out_loc[j];
      const bool inside = loc >= 0 && loc < slots;
      in_run = !inside || loc / ps == page;
      if (in_run && inside) {
        if (P.rot > 0) pos = P.positions[j];
        if (P.rot == 0 || (pos >= 0 && pos < P.max_pos)) slot = loc - page * ps;
      }
    }
    const unsigned out = ~__ballot_sync(kFull, in_run);
    const int cnt = out == 0u ? 32 : __ffs(out) - 1;
    if (lane >= cnt) slot = -1;
    return cnt;
  };
  auto load = [&](int64_t j, int t) -> float4 {
    uint2 raw = make_uint2(0u, 0u);
    if (D.live) raw = *reinterpret_cast<const uint2*>(D.src + j * D.ts);
    float4 x = unpack4<T>(raw);
    if (D.turning) {
      const Turn turn = load_turn<INTER>(P, __shfl_sync(kFull, pos, t), lane);
      x = rotate<INTER>(P, x, turn, lane);
    }
    return x;
  };
  float amax = 0.0f;
  bool fine = true;
  int first = -1;  // the first written slot of the run
  for (int64_t base = j0;; base += 32) {
    const int cnt = scan(base);
    const unsigned valid = __ballot_sync(kFull, slot >= 0);
    if (first < 0 && valid != 0u) first = __shfl_sync(kFull, slot, __ffs(valid) - 1);
#pragma unroll 8
    for (int t = 0; t < cnt; ++t) {
      if ((valid >> t) & 1u) {
        const float4 x = load(base + t, t);
        amax = fmaxf(amax, max4(x));
        fine = fine && finite4(x);
      }
    }
    if (cnt < 32) break;
  }
  if (first < 0) return;
  amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
  const float want = scale_for(amax);
  const float now = first == 0 ? want : fmaxf(before, want);
  if (first > 0 && now != before) regrow(D.dst, P.c.token_stride, first, before, now, D.live);
  const Divide div(now);
  for (int64_t base = j0;; base += 32) {
    const int cnt = scan(base);
    const unsigned valid = __ballot_sync(kFull, slot >= 0);
#pragma unroll 8
    for (int t = 0; t < cnt; ++t) {
      if ((valid >> t) & 1u) {
        const float4 x = load(base + t, t);
        const int o = __shfl_sync(kFull, slot, t);
        if (D.live) *reinterpret_cast<uint32_t*>(D.dst + o * P.c.token_stride) = div.codes(x);
      }
    }
    if (cnt < 32) break;
  }
  if (lane == 0) *D.scale = now;
  if (!__all_sync(kFull, fine) && lane == 0 && P.status != nullptr)
    atomicOr(P.status, PKV_ST_NONFINITE);
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, 3) append_kernel(const AppendParams P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t n = P.n_tokens;
  if (P.total != nullptr) n = max(int64_t{0}, min(n, *P.total));
  const int ps = P.c.page_size;
  const int64_t slots = P.c.num_pages * ps;
  if (blockIdx.x < P.kv_blocks) {
    // ---- this block's window of tokens: the runs that begin in it.  Lane l
    // looks at token w0 + l; a run of at most kHold tokens ends within them.
    const int64_t w0 = static_cast<int64_t>(blockIdx.x) * P.window;
    const int64_t j = w0 + lane;
    int loc = -1, pos = 0, prev = -1;
    if (j < n) {
      loc = P.out_loc[j];
      if (P.rot > 0) pos = P.positions[j];
    }
    if (lane == 0 && w0 > 0 && w0 <= n) prev = P.out_loc[w0 - 1];
    const bool inside = loc >= 0 && loc < slots;
    const int page = inside ? loc / ps : -1;
    const bool placed = P.rot == 0 || (pos >= 0 && pos < P.max_pos);
    const int before = __shfl_up_sync(kFull, loc, 1);
    if (lane > 0) prev = before;
    bool lead = lane < P.window && inside;
    if (lead && j > 0) {
      for (int64_t p = j - 1;;) {  // past skipped tokens, if any
        if (prev >= 0 && prev < slots) {
          lead = prev / ps != page;
          break;
        }
        if (--p < 0) break;
        prev = P.out_loc[p];
      }
    }
    if (warp == 0 && lane < P.window && j < n && P.status != nullptr) {
      const int bad = !inside ? PKV_ST_ROW_OOB : !placed ? PKV_ST_COL_OOB : 0;
      if (bad != 0) atomicOr(P.status, bad);
    }
    const unsigned leads = __ballot_sync(kFull, lead);
    const int per = 2 * P.c.kv_heads;
    const int items = __popc(leads) * per;
    for (int it = warp; it < items; it += kWarps) {
      unsigned m = leads;
      for (int r = it / per; r > 0; --r) m &= m - 1;
      const int at = __ffs(m) - 1;
      const int run_page = __shfl_sync(kFull, page, at);
      const unsigned in_run = __ballot_sync(kFull, j < n && (!inside || page == run_page));
      const unsigned valid = __ballot_sync(kFull, inside && page == run_page && placed) >> at;
      const int cnt = __ffs(~(in_run >> at)) - 1;  // at <= 15: bit 31 - at and up are clear or past
      const int rest = it % per;
      const bool is_v = rest >= P.c.kv_heads;
      const Target D = target(P, run_page, is_v ? rest - P.c.kv_heads : rest, is_v, lane);
      if (cnt >= 0 && cnt <= kHold) {
        append_held<T, INTER>(P, D, w0 + at, at, valid & ((1u << cnt) - 1u), loc - run_page * ps,
                              pos, lane);
      } else {
        append_long<T, INTER>(P, D, n, w0 + at, run_page, lane);
      }
    }
    return;
  }
  // ---- queries: kQHeads heads of one token a warp
  const int groups = (P.q_heads + kQHeads - 1) / kQHeads;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) - P.kv_blocks) * kWarps + warp;
  const int64_t j = unit / groups;
  const int h0 = static_cast<int>(unit - j * groups) * kQHeads;
  if (j >= n) return;
  const int loc = P.out_loc[j];
  const int pos = P.rot > 0 ? P.positions[j] : 0;
  const bool live = lane * 4 < P.c.head_dim;
  uint2 raw[kQHeads];
#pragma unroll
  for (int i = 0; i < kQHeads; ++i) {
    raw[i] = make_uint2(0u, 0u);
    if (live && h0 + i < P.q_heads)
      raw[i] = *reinterpret_cast<const uint2*>(P.q + j * P.q_ts + (h0 + i) * P.q_hs + lane * 4);
  }
  if (loc < 0 || loc >= slots) return;
  Turn turn;
  if (P.rot > 0) {
    if (pos < 0 || pos >= P.max_pos) return;
    turn = load_turn<INTER>(P, pos, lane);
  }
#pragma unroll
  for (int i = 0; i < kQHeads; ++i) {
    uint2 y = raw[i];
    if (P.rot > 0) {
      const float4 x = rotate<INTER>(P, unpack4<T>(raw[i]), turn, lane);
      if (lane * 4 < P.rot) y = make_uint2(Pair<T>::pack(x.x, x.y), Pair<T>::pack(x.z, x.w));
    }
    if (live && h0 + i < P.q_heads)
      *reinterpret_cast<uint2*>(P.q_out + j * P.o_ts + (h0 + i) * P.o_hs + lane * 4) = y;
  }
}

template <typename T>
void launch(const AppendParams& P, bool inter, int64_t blocks, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(blocks);
  if (inter) append_kernel<T, true><<<grid, kWarps * 32, 0, s>>>(P);
  else append_kernel<T, false><<<grid, kWarps * 32, 0, s>>>(P);
}

}  // namespace

}  // namespace pkv

extern "C" int pkv_append_kv(const pkv_kv_cache* cache, const void* k, int64_t k_token_stride,
                             int64_t k_head_stride, const void* v, int64_t v_token_stride,
                             int64_t v_head_stride, pkv_dtype dt, int64_t n_tokens,
                             const int64_t* total_tokens, const int32_t* positions,
                             const int32_t* out_loc, const float* cos_sin, int64_t max_pos,
                             int rot_dim, int interleaved, const void* q, int64_t q_token_stride,
                             int64_t q_head_stride, int q_heads, void* q_out,
                             int64_t o_token_stride, int64_t o_head_stride, int32_t* status,
                             pkv_stream_t stream) {
  using namespace pkv;
  int bad = cache_error(cache);
  if (bad != PKV_OK) return bad;
  if (dt != PKV_BF16 && dt != PKV_FP16)
    return fail(PKV_EINVAL, "dtype %d is not bf16 or fp16", static_cast<int>(dt));
  if (n_tokens < 0 || n_tokens > INT32_MAX)
    return fail(PKV_EINVAL, "n_tokens=%lld outside [0, 2^31)", (long long)n_tokens);
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 8 != 0)
    return fail(PKV_EINVAL, "rot_dim=%d is not a multiple of 8 in [0, head_dim=%d]", rot_dim,
                cache->head_dim);
  if (rot_dim > 0 && (cos_sin == nullptr || max_pos < 1 || !aligned16(cos_sin)))
    return fail(PKV_EINVAL, "rot_dim=%d needs a 16-byte aligned cos_sin with max_pos >= 1", rot_dim);
  if (n_tokens == 0) return ok();
  if (positions == nullptr && rot_dim > 0) return fail(PKV_EINVAL, "positions is NULL");
  if (out_loc == nullptr) return fail(PKV_EINVAL, "out_loc is NULL");
  if ((bad = rows_error("k", k, k_token_stride, k_head_stride)) != PKV_OK) return bad;
  if ((bad = rows_error("v", v, v_token_stride, v_head_stride)) != PKV_OK) return bad;
  if (q != nullptr) {
    if (q_heads < 1 || q_heads > 65535)
      return fail(PKV_EINVAL, "q_heads=%d outside [1, 65535]", q_heads);
    if ((bad = rows_error("q", q, q_token_stride, q_head_stride)) != PKV_OK) return bad;
    if ((bad = rows_error("q_out", q_out, o_token_stride, o_head_stride)) != PKV_OK) return bad;
  } else if (q_heads != 0) {
    return fail(PKV_EINVAL, "q_heads=%d without q", q_heads);
  }
  AppendParams P;
  P.c = *cache;
  P.k = static_cast<const uint16_t*>(k);
  P.v = static_cast<const uint16_t*>(v);
  P.q = static_cast<const uint16_t*>(q);
  P.q_out = static_cast<uint16_t*>(q_out);
  P.k_ts = k_token_stride, P.k_hs = k_head_stride;
  P.v_ts = v_token_stride, P.v_hs = v_head_stride;
  P.q_ts = q_token_stride, P.q_hs = q_head_stride;
  P.o_ts = o_token_stride, P.o_hs = o_head_stride;
  P.positions = positions;
  P.out_loc = out_loc;
  P.cos_sin = cos_sin;
  P.total = total_tokens;
  P.status = status;
  P.n_tokens = n_tokens;
  P.max_pos = max_pos;
  P.rot = rot_dim;
  P.q_heads = q_heads;
  // Tokens a block looks at: enough blocks to fill the SMs first, then up to
  // kMaxWindow, so that most blocks of a long step lead a whole page.
  P.window = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(kMaxWindow, n_tokens / (4 * num_sms()))));
  P.kv_blocks = div_ceil(n_tokens, P.window);
  const int64_t q_units = n_tokens * ((q_heads + kQHeads - 1) / kQHeads);
  const int64_t blocks = P.kv_blocks + div_ceil(q_units, kWarps);
  if (blocks > INT32_MAX)
    return fail(PKV_EINVAL, "n_tokens * q_heads = %lld * %d is too large", (long long)n_tokens,
                q_heads);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == PKV_BF16) launch<__nv_bfloat16>(P, interleaved != 0, blocks, s);
  else launch<__half>(P, interleaved != 0, blocks, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "append launch");
  return ok();
}
