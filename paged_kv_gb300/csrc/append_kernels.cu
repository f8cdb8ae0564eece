// pkv_append_kv: a step's keys and values, rotated and rounded to e4m3, into
// the paged cache.
//
//   k' = R(p) k,  a = max |k'| over the call's tokens of a (page, head),
//   s = 2^e least with a <= 448 s,  code = rn_e4m3(k' / s)
//
// A run is the call's tokens of one page; its first token leads it.  One warp
// owns one (run, head, k or v): it alone reads and writes that page's scale
// and codes of that head, so nothing is shared between warps and a run's
// result does not depend on the launch.
//
// A row (one token of one head) takes LPR lanes, each with two quads of 4
// elements whose rotation stays inside the lane: with rotate-half, quad i and
// the quad half the rotated width further on; a warp has 32 / LPR rows in
// hand.  A run of up to kHold tokens is loaded at once and stays in registers,
// unrotated, between the maximum and the rounding: turning it twice costs
// fewer cycles than the registers of turned values, which would halve the
// warps that keep loads in flight.  A longer run is read twice, from L2.
//
// e4m3 keeps its relative precision over 2^-6 .. 448, so a power-of-two scale
// costs nothing against a tight one and lets a page's scale grow later
// without a second rounding error (but for subnormals).
//
// Bound: bytes, and with few tokens the two dependent loads (a token's place,
// then what the place needs).  About 65 thousand tokens in 256 chunks, 16 query
// and 8 cache heads of 128, bf16: 202 us, 4.8 TB/s of the 6.8 that a copy
// reaches (the queries alone 96 us, 5.6 TB/s; keys and values alone 130 us,
// 3.1 TB/s: 24 warps an SM, each waiting for its run's rows, then its turns).
// 256 single tokens: 6.5 us.  Windows of 16 tokens a block: 202 us, of 8 211, of
// 4 233; but the single tokens take 61 us with 16, so short steps have windows of
// one.  Heads of at most 64 take 8 lanes a row, which 16 would leave half idle:
// 131 us against 178 for the chunks with heads of 64.

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
constexpr int kQHeads = 16;  // query heads a warp rotates together (8: 217 us, 32: 234)
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

// Which quads of a row a lane holds, and the angles they turn by.
struct Lane {
  int sub;        // row of the warp's 32 / LPR
  int a, b;       // first elements of its two quads
  int angle;      // cosines of cos_sin[p, angle ..]; < 0: not rotated
  bool live;
};

template <int LPR, bool INTER>
__device__ __forceinline__ Lane lane_of(const AppendParams& P, int lane) {
  Lane L;
  L.sub = lane / LPR;
  const int l = lane % LPR, pairs = P.rot >> 3;
  L.live = l * 8 < P.c.head_dim;
  const bool turned = l < pairs;
  L.a = turned && !INTER ? l * 4 : l * 8;
  L.b = turned && !INTER ? l * 4 + (P.rot >> 1) : l * 8 + 4;
  L.angle = turned ? l * 4 : -1;
  return L;
}

struct Octet {
  float a[4], b[4];
};

template <typename T>
__device__ __forceinline__ Octet unpack8(uint2 x, uint2 y) {
  const float2 p = Pair<T>::unpack(x.x), q = Pair<T>::unpack(x.y);
  const float2 r = Pair<T>::unpack(y.x), s = Pair<T>::unpack(y.y);
  return {{p.x, p.y, q.x, q.y}, {r.x, r.y, s.x, s.y}};
}

struct Turn {
  float4 c, s;
};

__device__ __forceinline__ Turn load_turn(const AppendParams& P, const Lane& L, int pos) {
  Turn t;
  t.c = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  t.s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (L.angle >= 0) {
    const float* row = P.cos_sin + static_cast<int64_t>(pos) * P.rot + L.angle;
    t.c = *reinterpret_cast<const float4*>(row);
    t.s = *reinterpret_cast<const float4*>(row + (P.rot >> 1));
  }
  return t;
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = fmaf(x, c, -(y * s));
  b = fmaf(y, c, x * s);
}

template <bool INTER>
__device__ __forceinline__ void rotate(Octet& x, const Turn& t, const Lane& L) {
  if (L.angle < 0) return;  // 0 * inf must not get in
  if (INTER) {
    turn_pair(x.a[0], x.a[1], t.c.x, t.s.x);
    turn_pair(x.a[2], x.a[3], t.c.y, t.s.y);
    turn_pair(x.b[0], x.b[1], t.c.z, t.s.z);
    turn_pair(x.b[2], x.b[3], t.c.w, t.s.w);
  } else {
    turn_pair(x.a[0], x.b[0], t.c.x, t.s.x);
    turn_pair(x.a[1], x.b[1], t.c.y, t.s.y);
    turn_pair(x.a[2], x.b[2], t.c.z, t.s.z);
    turn_pair(x.a[3], x.b[3], t.c.w, t.s.w);
  }
}

// Least 2^e with a <= 448 * 2^e.  448 = 1.75 * 2^8, so e is the exponent of a
// minus 8, and one more where a's significand is above 1.75.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(kMinExp, min(kMaxExp, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Running maximum of magnitudes; a NaN or an infinity stays visible in it.
__device__ __forceinline__ float max_all(float m, const Octet& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmax_nan(m, fmax_nan(fabsf(x.a[i]), fabsf(x.b[i])));
  return m;
}
// The same over finite values only.
__device__ __forceinline__ float max_finite(float m, const Octet& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (isfinite(x.a[i])) m = fmaxf(m, fabsf(x.a[i]));
    if (isfinite(x.b[i])) m = fmaxf(m, fabsf(x.b[i]));
  }
  return m;
}

__device__ __forceinline__ void store_codes(uint8_t* row, const Lane& L, const Octet& x, float inv) {
  if (!L.live) return;
  *reinterpret_cast<uint32_t*>(row + L.a) =
      e4m3x2(x.a[0] * inv, x.a[1] * inv) | (e4m3x2(x.a[2] * inv, x.a[3] * inv) << 16);
  *reinterpret_cast<uint32_t*>(row + L.b) =
      e4m3x2(x.b[0] * inv, x.b[1] * inv) | (e4m3x2(x.b[2] * inv, x.b[3] * inv) << 16);
}

// Rounds the page's codes before slot `first` from one scale to a larger one.
__device__ __forceinline__ void regrow(uint8_t* dst, int64_t token_stride, int head_dim, int first,
                                       float before, float now, int lane) {
  const float ratio = before / now;
  for (int t = 0; t < first; ++t) {
    if (lane * 4 < head_dim) {
      uint32_t* at = reinterpret_cast<uint32_t*>(dst + t * token_stride + lane * 4);
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
};

__device__ __forceinline__ Target target(const AppendParams& P, int page, int head, bool is_v) {
  const pkv_kv_cache& C = P.c;
  Target t;
  t.src = is_v ? P.v + head * P.v_hs : P.k + head * P.k_hs;
  t.ts = is_v ? P.v_ts : P.k_ts;
  t.dst = static_cast<uint8_t*>(is_v ? C.v : C.k) + page * C.page_stride + head * C.head_stride;
  t.scale = (is_v ? C.v_scale : C.k_scale) + static_cast<int64_t>(page) * C.kv_heads + head;
  return t;
}

// A run of at most kHold tokens.  Lane l holds token w0 + l's slot in the page
// and position; the run's tokens are j0 .. , j0 = w0 + at, those with a bit in
// `valid` are written.
template <typename T, int LPR, bool INTER, bool TURN>
__device__ __forceinline__ void append_held(const AppendParams& P, const Target& D, const Lane& L,
                                            int64_t j0, int at, unsigned valid, int slot, int pos,
                                            int lane) {
  constexpr int kRows = 32 / LPR, kIters = kHold / kRows;
  if (valid == 0u) return;
  const float before = *D.scale;
  uint2 ra[kIters], rb[kIters];
  const uint16_t* src = D.src + (j0 + L.sub) * D.ts;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    ra[i] = rb[i] = make_uint2(0u, 0u);
    if (((valid >> (i * kRows + L.sub)) & 1u) != 0u && L.live) {
      ra[i] = *reinterpret_cast<const uint2*>(src + L.a);
      rb[i] = *reinterpret_cast<const uint2*>(src + L.b);
    }
    src += kRows * D.ts;
  }
  constexpr unsigned kGroup = (1u << kRows) - 1u;
  auto value = [&](int i) -> Octet {
    Octet x = unpack8<T>(ra[i], rb[i]);
    if (TURN) {
      const int t = i * kRows + L.sub;
      const int p = __shfl_sync(kFull, pos, (at + t) & 31);
      if ((valid >> t) & 1u) {
        const Turn turn = load_turn(P, L, p);
        rotate<INTER>(x, turn, L);
      }
    }
    return x;
  };
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    if ((valid >> (i * kRows)) & kGroup) amax = max_all(amax, value(i));
  }
  const bool fine = __all_sync(kFull, isfinite(amax));
  if (!fine) {
    amax = 0.0f;
#pragma unroll 1
    for (int i = 0; i < kIters; ++i) {
      // (The registers are indexed by a loop that is not unrolled: rare.)
      Octet x = {};
#pragma unroll
      for (int k = 0; k < kIters; ++k)
        if (k == i) x = unpack8<T>(ra[k], rb[k]);
      if (TURN) {
        const int t = i * kRows + L.sub;
        const int p = __shfl_sync(kFull, pos, (at + t) & 31);
        if ((valid >> t) & 1u) rotate<INTER>(x, load_turn(P, L, p), L);
      }
      amax = max_finite(amax, x);
    }
  }
  amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
  const float want = scale_for(amax);
  const int first = __shfl_sync(kFull, slot, at + __ffs(valid) - 1);
  const float now = first == 0 ? want : fmaxf(before, want);
  if (first > 0 && now != before)
    regrow(D.dst, P.c.token_stride, P.c.head_dim, first, before, now, lane);
  const float inv = 1.0f / now;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    if ((valid >> (i * kRows)) & kGroup) {
      const int t = i * kRows + L.sub;
      const Octet x = value(i);
      const int o = __shfl_sync(kFull, slot, (at + t) & 31);
      if ((valid >> t) & 1u) store_codes(D.dst + o * P.c.token_stride, L, x, inv);
    }
  }
  if (lane == 0) *D.scale = now;
  if (!fine && lane == 0 && P.status != nullptr) atomicOr(P.status, PKV_ST_NONFINITE);
}

// A run of any length that begins at token j0, read twice.
template <typename T, int LPR, bool INTER>
__device__ __noinline__ void append_long(const AppendParams& P, const Target D, int64_t n,
                                         int64_t j0, int page, bool is_v, int lane) {
  constexpr int kRows = 32 / LPR;
  const Lane L = lane_of<LPR, INTER>(P, lane);
  const int ps = P.c.page_size;
  const int64_t slots = P.c.num_pages * ps;
  const float before = *D.scale;
  const bool turning = !is_v && P.rot > 0;
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
  // Calls f(slot, values) for every row group of the run; slot < 0: not written.
  auto each = [&](auto&& f) {
    for (int64_t base = j0;; base += 32) {
      const int cnt = scan(base);
#pragma unroll 4
      for (int t0 = 0; t0 < cnt; t0 += kRows) {
        const int t = t0 + L.sub;
        const int o = __shfl_sync(kFull, slot, t), p = __shfl_sync(kFull, pos, t);
        uint2 a = make_uint2(0u, 0u), b = make_uint2(0u, 0u);
        if (o >= 0 && L.live) {
          const uint16_t* src = D.src + (base + t) * D.ts;
          a = *reinterpret_cast<const uint2*>(src + L.a);
          b = *reinterpret_cast<const uint2*>(src + L.b);
        }
        Octet x = unpack8<T>(a, b);
        if (turning && o >= 0) rotate<INTER>(x, load_turn(P, L, p), L);
        f(o, x);
      }
      if (cnt < 32) break;
    }
  };
  float amax = 0.0f;
  int first = ps;  // the first written slot of the run
  each([&](int o, const Octet& x) {
    amax = max_all(amax, x);
    if (o >= 0) first = min(first, o);
  });
  first = __reduce_min_sync(kFull, first);
  if (first == ps) return;
  const bool fine = __all_sync(kFull, isfinite(amax));
  if (!fine) {
    amax = 0.0f;
    each([&](int, const Octet& x) { amax = max_finite(amax, x); });
  }
  amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
  const float want = scale_for(amax);
  const float now = first == 0 ? want : fmaxf(before, want);
  if (first > 0 && now != before)
    regrow(D.dst, P.c.token_stride, P.c.head_dim, first, before, now, lane);
  const float inv = 1.0f / now;
  each([&](int o, const Octet& x) {
    if (o >= 0) store_codes(D.dst + o * P.c.token_stride, L, x, inv);
  });
  if (lane == 0) *D.scale = now;
  if (!fine && lane == 0 && P.status != nullptr) atomicOr(P.status, PKV_ST_NONFINITE);
}

template <typename T, int LPR, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, 3) append_kernel(
    const __grid_constant__ AppendParams P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t n = P.n_tokens;
  if (P.total != nullptr) n = max(int64_t{0}, min(n, *P.total));
  const int ps = P.c.page_size;
  const int64_t slots = P.c.num_pages * ps;
  const Lane L = lane_of<LPR, INTER>(P, lane);
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
      const int cnt = __ffs(~(in_run >> at)) - 1;  // -1: all 32
      const int rest = it % per;
      const bool is_v = rest >= P.c.kv_heads;
      const Target D = target(P, run_page, is_v ? rest - P.c.kv_heads : rest, is_v);
      if (cnt < 0 || cnt > kHold) {
        append_long<T, LPR, INTER>(P, D, n, w0 + at, run_page, is_v, lane);
      } else {
        const unsigned mine = valid & ((1u << cnt) - 1u);
        const int slot = loc - run_page * ps;
        if (!is_v && P.rot > 0)
          append_held<T, LPR, INTER, true>(P, D, L, w0 + at, at, mine, slot, pos, lane);
        else
          append_held<T, LPR, INTER, false>(P, D, L, w0 + at, at, mine, slot, pos, lane);
      }
    }
    return;
  }
  // ---- queries: kQHeads heads of one token a warp
  constexpr int kRows = 32 / LPR, kIters = kQHeads / kRows;
  const int groups = (P.q_heads + kQHeads - 1) / kQHeads;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) - P.kv_blocks) * kWarps + warp;
  const int64_t j = unit / groups;
  const int h0 = static_cast<int>(unit - j * groups) * kQHeads + L.sub;
  if (j >= n) return;
  const int loc = P.out_loc[j];
  const int pos = P.rot > 0 ? P.positions[j] : 0;
  uint2 ra[kIters], rb[kIters];
  const uint16_t* src = P.q + j * P.q_ts + h0 * P.q_hs;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    ra[i] = rb[i] = make_uint2(0u, 0u);
    if (L.live && h0 + i * kRows < P.q_heads) {
      ra[i] = *reinterpret_cast<const uint2*>(src + L.a);
      rb[i] = *reinterpret_cast<const uint2*>(src + L.b);
    }
    src += kRows * P.q_hs;
  }
  if (loc < 0 || loc >= slots) return;
  Turn turn;
  if (P.rot > 0) {
    if (pos < 0 || pos >= P.max_pos) return;
    turn = load_turn(P, L, pos);
  }
  uint16_t* dst = P.q_out + j * P.o_ts + h0 * P.o_hs;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    uint2 ya = ra[i], yb = rb[i];
    if (L.angle >= 0) {
      Octet x = unpack8<T>(ra[i], rb[i]);
      rotate<INTER>(x, turn, L);
      ya = make_uint2(Pair<T>::pack(x.a[0], x.a[1]), Pair<T>::pack(x.a[2], x.a[3]));
      yb = make_uint2(Pair<T>::pack(x.b[0], x.b[1]), Pair<T>::pack(x.b[2], x.b[3]));
    }
    if (L.live && h0 + i * kRows < P.q_heads) {
      *reinterpret_cast<uint2*>(dst + L.a) = ya;
      *reinterpret_cast<uint2*>(dst + L.b) = yb;
    }
    dst += kRows * P.o_hs;
  }
}

template <typename T>
void launch(const AppendParams& P, bool inter, int64_t blocks, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(blocks);
  if (P.c.head_dim > 64) {
    if (inter) append_kernel<T, 16, true><<<grid, kWarps * 32, 0, s>>>(P);
    else append_kernel<T, 16, false><<<grid, kWarps * 32, 0, s>>>(P);
  } else {
    if (inter) append_kernel<T, 8, true><<<grid, kWarps * 32, 0, s>>>(P);
    else append_kernel<T, 8, false><<<grid, kWarps * 32, 0, s>>>(P);
  }
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
