// pkv_beam_select: the best continuations of each request's beams.
//
//   t(w, v) = scores[w] + x[w, v] - ln sum_u exp x[w, u]
//
// Two kernels.  The first reads the logits once: a warp takes a slice of a row (256
// vectors of 16 bytes) in two batches, the next one under way, and leaves the slice's
// maximum `ref`, sum exp(x - ref), and largest logit apart from the ending.  The second
// has a CTA a request: it joins the slices' sums, takes as threshold a bound of the
// n-th largest of the slices' maxima (so many candidates are at least as large), reads
// the slices above it again and ranks what they hold, some n entries.
//
// Exact order.  A lane sums exp(x - m) under its running maximum m, which then passes
// to the slice's and to the row's.  With d a difference rounded once, exp's argument
// d log2(e) is off by at most |d log2 e| (2^-24 + 2^-24 + 2^-26); the differences on the
// way from a logit to the slice's maximum add up to theirs, whose mean under the
// slice's weights is at most log2 of its elements, 11: 1.0e-6.  Three exponentials on
// that way are off by 2^-22 each, the sum by some 11 + 5 + 4 roundings of 2^-24.  A row's
// log-sum-exp is therefore off by less than 3e-6 (1.02 + 0.72 + 1.19), the difference of
// two by less than kNear; joining the slices (sums of two fp32 values) adds nothing to
// speak of.  Candidates of different rows that lie nearer than kNear and could change the
// result make the CTA sum their rows again (exp_below), to some 2^-36, and compare them by
// all bits of t (make_words): equal rows, and rows that differ by a constant, tie where the
// numbers are equal, and a score far from zero hides nothing.  Candidates of one row
// go by their logits and need no sums.  No fp64: this part has a 64th of its rate.
//
// Bound: the logits' bytes; with few rows the chain of loads and barriers.  Equal or flat
// rows are a request's CTA's alone: 4 equal ones of 32000 take 34 us more than others, 8 of
// 151936 in each of 32 requests 0.8 ms, 64 of 256000 5 ms; with more than kCand equal
// candidates, so all of their rows are read some five times, 0.3, 4.7 and 40 ms.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "device_attr.h"
#include "device_common.cuh"
#include "double_float.cuh"
#include "launch_early.h"
#include "radix_nth.cuh"

namespace pkv {

namespace {

constexpr int kBatch = 4;            // vectors a lane holds at once
constexpr int kVecs = 2 * kBatch;    // vectors of a slice, a lane
constexpr int kSlice = 32 * kVecs;   // vectors of a slice
constexpr int kStreamWarps = 8;
constexpr int kThreads = 512;        // of the second kernel
constexpr int kWarps = kThreads / 32;
constexpr int kMostSlices = 288;     // of a row; 9 a lane
constexpr int kCand = 1024;          // candidates it can rank at once, endings apart
constexpr int kWords = 9;            // of a number in units of 2^-149: 2^129 is bit 278
constexpr int kBins = 1024;
constexpr float kBinsPerNat = 16.0f;
constexpr float kNear = 6e-6f;
// Scores within +-kFar and logits at most kFar below their beam's largest: sums and
// differences of them stay in fp32's range.
constexpr float kFar = 0x1p126f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kEnd = 1u << 31;  // a candidate that ends its beam

struct BeamParams {
  const void* logits;
  int64_t row_stride;
  const float* scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  float* out_scores;
  float* ended;   // or nullptr
  int32_t* status;
  float4* parts;  // [rows, slices]: ref, sum, the largest but for the ending
  int B, W, V, n_out, eos, slices;
};

template <typename T> struct Elements;  // of a 16-byte vector
template <> struct Elements<float> {
  static constexpr int kPer = 4;
  static constexpr uint32_t kMinusInf = 0xff800000u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <> struct Elements<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kMinusInf = 0xff80ff80u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// A row in vectors: the first begins at the 16-byte boundary at or below the row,
// `lead` elements before it.
template <typename T>
struct Row {
  const uint4* base;
  int lead, vectors;
};
template <typename T>
__device__ __forceinline__ Row<T> row_of(const BeamParams& P, int row) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(
      static_cast<const T*>(P.logits) + static_cast<int64_t>(row) * P.row_stride);
  Row<T> r;
  r.base = reinterpret_cast<const uint4*>(a & ~uintptr_t{15});
  r.lead = static_cast<int>(a & 15u) / static_cast<int>(sizeof(T));
  r.vectors = (r.lead + P.V + Elements<T>::kPer - 1) / Elements<T>::kPer;
  return r;
}
// (Not by the read-only path: the kernel may start before the logits are written.)
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Vector k of the row, -inf in the places outside it.
template <typename T>
__device__ __forceinline__ uint4 load_vector(const Row<T>& r, int k) {
  constexpr uint32_t kNo = Elements<T>::kMinusInf;
  return k < r.vectors ? load_once(r.base + k) : make_uint4(kNo, kNo, kNo, kNo);
}
// The same with the ending's place (element `end` from the first vector's begin, or
// -1) masked, too.
template <typename T>
__device__ __forceinline__ void unpack_row(const Row<T>& r, int V, int k, const uint4& v, int end,
                                           float (&x)[Elements<T>::kPer]) {
  constexpr int kPer = Elements<T>::kPer;
  Elements<T>::unpack(v, x);
  if (k == 0 || k >= r.vectors - 1 || (end >= 0 && end / kPer == k)) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int at = k * kPer + e;
      if (at < r.lead || at >= r.lead + V || at == end) x[e] = -INFINITY;
    }
  }
}

// Two fp32 values at a time.
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float batch_max(const uint4 (&v)[kBatch], float) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    m = fmax_nan(m, fmax_nan(fmax_nan(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                             fmax_nan(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
  return m;
}
__device__ __forceinline__ float batch_max(const uint4 (&v)[kBatch], __nv_bfloat16) {
  uint32_t m = 0xff80ff80u;
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    m = bf16x2_max_nan(m, bf16x2_max_nan(bf16x2_max_nan(v[i].x, v[i].y), bf16x2_max_nan(v[i].z, v[i].w)));
  return fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

struct LaneState {
  float m, s;    // largest logit, sum of exp(x - m)
  float other;   // the largest but for the ending
};

// Takes a batch of vectors k0 + 32 i of the row into the lane's state.  rare: the batch
// may hold the row's edges or the ending.
template <typename T>
__device__ __forceinline__ void take_batch(const BeamParams& P, const Row<T>& r, int k0, bool rare,
                                           int end, uint4 (&v)[kBatch], LaneState& S) {
  constexpr int kPer = Elements<T>::kPer;
  float other = -INFINITY;
  if (rare) {
    // Places outside the row become -inf in the vectors themselves.
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * 32;
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int at = k * kPer + e;
        if (at < r.lead || at >= r.lead + P.V) {
          if (kPer == 4) w[e] = 0xff800000u;
          else w[e / 2] = (e & 1) ? (w[e / 2] & 0xffffu) | 0xff800000u : (w[e / 2] & 0xffff0000u) | 0xff80u;
        }
      }
      v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      float x[kPer];
      unpack_row<T>(r, P.V, k, v[i], end, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) other = fmax_nan(other, x[e]);
    }
  }
  const float most = batch_max(v, T{});
  S.other = fmax_nan(S.other, rare ? other : most);
  const float m = fmax_nan(S.m, most), base = m == -INFINITY ? 0.0f : m;
  S.s *= ex2((S.m - base) * kLog2e);
  S.m = m;
  const unsigned long long minus = pack2(-base, -base), unit = pack2(kLog2e, kLog2e);
  unsigned long long sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    float x[kPer];
    Elements<T>::unpack(v[i], x);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const float2 y = unpack2(mul2(add2(pack2(x[e], x[e + 1]), minus), unit));
      sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(ex2(y.x), ex2(y.y)));
    }
  }
  const float2 a = unpack2(add2(sum[0], sum[1]));
  S.s += a.x + a.y;
}

template <typename T>
__global__ void __launch_bounds__(kStreamWarps * 32, 4) beam_stream_kernel(
    const __grid_constant__ BeamParams P) {
  constexpr int kPer = Elements<T>::kPer;
  const int lane = threadIdx.x & 31;
  const int warps = static_cast<int>(gridDim.x) * kStreamWarps;
  const int items = P.B * P.W * P.slices;  // (the host bounds it)
  launch_dependents();
  grid_dependency_wait();
  // The next item from `i` on whose beam is not dead.
  auto live_from = [&](int i) {
    while (i < items && __ldcg(P.scores + i / P.slices) == -INFINITY) i += warps;
    return i;
  };
  auto load = [&](const Row<T>& r, int k, uint4 (&v)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v[i] = load_vector(r, k + i * 32);
  };
  int item = live_from(static_cast<int>(blockIdx.x) * kStreamWarps + (threadIdx.x >> 5));
  if (item >= items) return;
  uint4 a[kBatch], b[kBatch];
  Row<T> r = row_of<T>(P, item / P.slices);
  load(r, item % P.slices * kSlice + lane, a);
  for (;;) {
    const int k0 = item % P.slices * kSlice;
    load(r, k0 + 32 * kBatch + lane, b);
    const int end = P.eos >= 0 && P.eos < P.V ? P.eos + r.lead : -1;
    const bool rare = k0 == 0 || k0 + kSlice >= r.vectors ||
                      (end >= 0 && end / kPer >= k0 && end / kPer < k0 + kSlice);
    LaneState S = {-INFINITY, 0.0f, -INFINITY};
    take_batch<T>(P, r, k0 + lane, rare, end, a, S);
    const Row<T> mine = r;
    const int next = live_from(item + warps);
    if (next < items) {
      r = row_of<T>(P, next / P.slices);
      load(r, next % P.slices * kSlice + lane, a);
    }
    take_batch<T>(P, mine, k0 + 32 * kBatch + lane, rare, end, b, S);
    // (max.NaN gives the positive NaN, whose key is above all others.)
    const float ref = key_float(__reduce_max_sync(kFull, float_key(S.m)));
    const float top = key_float(__reduce_max_sync(kFull, float_key(S.other)));
    const float base = ref == -INFINITY ? 0.0f : ref;
    const float total = warp_sum(S.s * ex2((S.m - base) * kLog2e));
    if (lane == 0) P.parts[item] = make_float4(ref, total, top, 0.0f);
    if (next >= items) break;
    item = next;
  }
}

struct Shared {
  FF log[PKV_MAX_BEAMS];         // ln sum_u exp(x_u - m)
  FF off[PKV_MAX_BEAMS];         // score less that: t is this plus x - m
  float score[PKV_MAX_BEAMS];
  float xmin[PKV_MAX_BEAMS];     // logits from here on are candidates
  float m[PKV_MAX_BEAMS];        // largest logit, the ending's among them
  float x_end[PKV_MAX_BEAMS];    // the ending's
  int live[PKV_MAX_BEAMS];
  unsigned long long key[kCand + PKV_MAX_BEAMS];   // falls as t does
  unsigned long long rest[kCand + PKV_MAX_BEAMS];  // order of equal ones and in a beam, ascending
  float x[kCand + PKV_MAX_BEAMS];
  uint32_t id[kCand + PKV_MAX_BEAMS];              // kEnd | w << 20 | v
  uint32_t words[kWords][kCand + PKV_MAX_BEAMS];   // t by all its bits, rises as t does
  int rank[kCand + PKV_MAX_BEAMS];
  float lanes[PKV_MAX_BEAMS * 32];                 // largest of the lanes of few slices
  NthScratch<kThreads> nth;
  FF part[kWarps];
  uint32_t count, hits, flag;
  unsigned long long near;
};
// After it in shared memory: each slice's largest t, bounded from below, then the list of
// those that may reach the threshold.
size_t finish_bytes(int pairs) {
  return sizeof(Shared) + static_cast<size_t>(pairs) * 4 + (pairs + 1) / 2 * 4;
}

__device__ __forceinline__ int beam_of(uint32_t id) { return (id >> 20) & (PKV_MAX_BEAMS - 1); }
__device__ __forceinline__ int token_of(uint32_t id) { return id & 0xfffffu; }

__device__ __forceinline__ FF total(const Shared& S, int w, float x) {
  return add(S.off[w], two_sum(x, -S.m[w]));
}

// t as fp32 computes it is off.h + (x - m).  It is off by the sums' error, off's lower half
// and three roundings, together at most kNear + 2^-23 (|off| + |t|): where a score cancels a
// gap of the logits, t is small and its error is not.  This is at least that, with room for
// the roundings of a bound that is formed with it.
__device__ __forceinline__ float slack(float off, float t) {
  return kNear + 0x1p-22f * (fabsf(off) + fabsf(t));
}
// Lower bound of a candidate's t, -inf for none.
__device__ __forceinline__ float at_least(float off, float above) {
  const float t = off + above;
  return t - slack(off, t);
}

// A lower bound of the n-th largest of t[0 .. count), -inf if fewer are above that;
// *have is how many are.  All threads call it; best is at least the largest.
__device__ float nth_bound(Shared& S, const float* t, int count, uint32_t n, float best,
                           uint32_t* have) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* bins = S.nth.bins;
  for (int i = tid; i < kBins; i += kThreads) bins[i] = 0u;
  __syncthreads();
  for (int i = tid; i < count; i += kThreads)
    if (t[i] > -INFINITY)
      atomicAdd(&bins[static_cast<int>(fminf((best - t[i]) * kBinsPerNat, kBins - 1.0f))], 1u);
  __syncthreads();
  constexpr int kOwn = kBins / kThreads;
  uint32_t own = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) own += bins[tid * kOwn + i];
  uint32_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) S.nth.scan[warp] = incl;
  __syncthreads();
  uint32_t before = incl - own, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += S.nth.scan[w];
    all += S.nth.scan[w];
  }
  *have = all;
  if (all < n) {  // (uniform)
    __syncthreads();
    return -INFINITY;
  }
  if (before < n && before + own >= n) {
    int bin = tid * kOwn;
    for (uint32_t c = before + bins[bin]; c < n; c += bins[bin]) ++bin;
    S.nth.prefix = static_cast<uint32_t>(bin);
  }
  __syncthreads();
  const int bin = static_cast<int>(S.nth.prefix);
  __syncthreads();
  if (bin < kBins - 1) {
    // (best - t, below 64, and this difference are rounded.)
    const float low = best - (bin + 1) * (1.0f / kBinsPerNat);
    return low - fabsf(low) * 0x1p-22f - 0x1p-18f;
  }
  // Further away than the bins reach.
  uint32_t ignore;
  return key_float(nth_key<kThreads, 2>(S.nth, n, &ignore, [&](auto&& f) {
    for (int i = tid; i < count; i += kThreads) f(t[i] > -INFINITY ? float_key(t[i]) : 0u);
  }));
}

// Sum of exp(x - m) over a row to some 2^-36: all threads, each of which gets it.  An
// element's place in the row alone says when it is added: rows of equal logits have equal
// sums wherever they begin.
template <typename T>
__device__ FF exact_sum(const BeamParams& P, Shared& S, int row, float m) {
  constexpr int kAhead = 8;  // elements of a thread whose loads are on their way together
  const int tid = threadIdx.x;
  const T* logits = static_cast<const T*>(P.logits) + static_cast<int64_t>(row) * P.row_stride;
  FF s = {0.0f, 0.0f};
#pragma unroll 1
  for (int v0 = tid; v0 < P.V; v0 += kThreads * kAhead) {
    float x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = v0 + i * kThreads;
      x[i] = v < P.V ? static_cast<float>(logits[v]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) s = add(s, exp_below(x[i], m));
  }
  s = warp_sum(s);
  __syncthreads();
  if ((tid & 31) == 0) S.part[tid >> 5] = s;
  __syncthreads();
  s = S.part[0];
#pragma unroll 1
  for (int w = 1; w < kWarps; ++w) s = add(s, S.part[w]);
  return s;
}

// Keys of candidate i: with best at least every t, t - best - 64 (at most -64) as a sum
// of two fp32 values, whose order is that of the pairs.
__device__ __forceinline__ void make_keys(Shared& S, int i, float best) {
  const uint32_t id = S.id[i];
  const int w = beam_of(id);
  const FF t = add(add(total(S, w, S.x[i]), -best), -64.0f);
  S.key[i] = static_cast<unsigned long long>(float_key(t.h)) << 32 | float_key(t.l);
  S.rest[i] = static_cast<unsigned long long>(w) << 52 |
              static_cast<unsigned long long>(~float_key(S.x[i])) << 20 | token_of(id);
}

// w += x, in two's complement and units of 2^-149.
__device__ __forceinline__ void add_bits(uint32_t (&w)[kWords], float x) {
  const uint32_t u = __float_as_uint(x), e = (u >> 23) & 255u;
  const unsigned long long m = (u & 0x7fffffu) | (e != 0u ? 0x800000u : 0u);
  const int shift = static_cast<int>(max(e, 1u)) - 1, at = shift >> 5;
  const unsigned long long part = m << (shift & 31);
  const bool minus = (u >> 31) != 0u;
  uint32_t carry = minus ? 1u : 0u;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    uint32_t a = k == at ? static_cast<uint32_t>(part)
                 : k == at + 1 ? static_cast<uint32_t>(part >> 32) : 0u;
    if (minus) a = ~a;
    const unsigned long long sum = static_cast<unsigned long long>(w[k]) + a + carry;
    w[k] = static_cast<uint32_t>(sum);
    carry = static_cast<uint32_t>(sum >> 32);
  }
}

// Candidate i's t = score + x - m - log by all its bits: exact but for log itself.
__device__ __forceinline__ void make_words(Shared& S, int i) {
  const int b = beam_of(S.id[i]);
  uint32_t w[kWords] = {};
  add_bits(w, S.score[b]);
  add_bits(w, S.x[i]);
  add_bits(w, -S.m[b]);
  add_bits(w, -S.log[b].h);
  add_bits(w, -S.log[b].l);
  w[kWords - 1] ^= 0x80000000u;
#pragma unroll
  for (int k = 0; k < kWords; ++k) S.words[k][i] = w[k];
}

// Whether candidate i comes before j of another beam, by their words and then by beam.
__device__ __forceinline__ bool before(const Shared& S, int i, int j) {
#pragma unroll 1
  for (int k = kWords - 1; k >= 0; --k) {
    const uint32_t a = S.words[k][i], b = S.words[k][j];
    if (a != b) return a > b;
  }
  return S.rest[i] < S.rest[j];
}

// The places of c candidates: among those that go on, of an ending among all.  A warp a
// candidate.  Those of one beam go by their logits, those of two by their keys, but where
// these are nearer than their errors (the sums', and the pairs' roundings at the size of
// score, t and best): then, EXACT, by their words; else the rows of those that it may
// matter for are left in S.near.
template <bool EXACT>
__device__ void rank_all(Shared& S, int c, int n_out, float best) {
  const int lane = threadIdx.x & 31;
  auto rounding = [&](uint32_t id, unsigned long long key) {
    return 0x1p-43f * (fabsf(S.off[beam_of(id)].h) + fabsf(best)) +
           0x1p-43f * fabsf(key_float(static_cast<uint32_t>(key >> 32)));
  };
#pragma unroll 1
  for (int i = threadIdx.x >> 5; i < c; i += kWarps) {
    const unsigned long long key = S.key[i], rest = S.rest[i];
    const uint32_t id = S.id[i];
    const bool ending = (id & kEnd) != 0u;
    const float near_i = kNear + rounding(id, key);
    int better = 0, close = 0;
    unsigned long long rows = 0ull;
#pragma unroll 1
    for (int j0 = 0; j0 < c; j0 += 32) {
      const int j = j0 + lane;
      bool is_better = false, is_near = false;
      if (j < c) {
        const unsigned long long other = S.key[j];
        const uint32_t jd = S.id[j];
        const bool counts = ending || (jd & kEnd) == 0u;
        if (beam_of(jd) == beam_of(id)) {
          is_better = S.rest[j] < rest;
        } else {
          const float d = (key_float(static_cast<uint32_t>(other >> 32)) -
                           key_float(static_cast<uint32_t>(key >> 32))) +
                          (key_float(static_cast<uint32_t>(other)) -
                           key_float(static_cast<uint32_t>(key)));
          is_near = fabsf(d) <= near_i + rounding(jd, other);
          if (!EXACT && is_near) rows |= 1ull << beam_of(jd) | 1ull << beam_of(id);
          is_better = EXACT && is_near ? before(S, j, i) : other > key;
        }
        is_better = is_better && counts;
        is_near = is_near && counts;
      }
      better += __popc(__ballot_sync(kFull, is_better));
      if (!EXACT) close += __popc(__ballot_sync(kFull, is_near));
    }
    if (lane == 0) S.rank[i] = better;
    // (A candidate that no exchange brings among the best matters to nobody.)
    if (!EXACT && rows != 0ull && better - close < n_out) atomicOr(&S.near, rows);
  }
}

// The n_out best of a row but for the ending, by logit and then by place, appended to
// the candidates.  All threads; reads the row some four times.
template <typename T>
__device__ void row_best(const BeamParams& P, Shared& S, int w, int row) {
  constexpr int kPer = Elements<T>::kPer;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<T> r = row_of<T>(P, row);
  const int end = P.eos >= 0 && P.eos < P.V ? P.eos + r.lead : -1;
  const float least = S.m[w] - kFar;
  uint32_t count;
  const uint32_t nth = nth_key<kThreads, 3>(S.nth, P.n_out, &count, [&](auto&& f) {
#pragma unroll 1
    for (int k = tid; k < r.vectors; k += kThreads) {
      float x[kPer];
      unpack_row<T>(r, P.V, k, load_vector(r, k), end, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f(x[e] > -INFINITY && x[e] >= least ? float_key(x[e]) : 0u);
    }
  });
  // Larger ones in any order, equal ones in theirs.
  uint32_t ties = 0;  // seen so far
  const uint32_t want = nth == 0u ? 0u : S.nth.left;
#pragma unroll 1
  for (int v0 = 0; v0 < P.V; v0 += kThreads) {
    const int v = v0 + tid;
    uint32_t key = 0u;
    float x = 0.0f;
    if (v < P.V && v != P.eos) {
      x = static_cast<float>(static_cast<const T*>(P.logits)[static_cast<int64_t>(row) * P.row_stride + v]);
      if (x > -INFINITY && x >= least) key = float_key(x);
    }
    const bool tie = nth != 0u && key == nth;
    bool take = key > nth;
    if (nth != 0u) {
      const unsigned t = __ballot_sync(kFull, tie);
      if (lane == 0) S.nth.scan[warp] = __popc(t);
      __syncthreads();
      uint32_t before = ties;
#pragma unroll 1
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += S.nth.scan[i];
        ties += S.nth.scan[i];
      }
      before += __popc(t & ((1u << lane) - 1u));
      if (tie && before < want) take = true;
      __syncthreads();
    }
    if (take) {
      const uint32_t at = atomicAdd(&S.count, 1u);
      S.x[at] = x;
      S.id[at] = static_cast<uint32_t>(w) << 20 | static_cast<uint32_t>(v);
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_finish_kernel(const __grid_constant__ BeamParams P) {
  extern __shared__ __align__(16) uint8_t raw_smem[];
  Shared& S = *reinterpret_cast<Shared*>(raw_smem);
  constexpr int kPer = Elements<T>::kPer;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, W = P.W, C = P.slices, n_out = P.n_out, pairs = W * C;
  float* tops = reinterpret_cast<float*>(raw_smem + sizeof(Shared));
  uint16_t* hits = reinterpret_cast<uint16_t*>(tops + pairs);
  const int64_t row0 = static_cast<int64_t>(b) * W;
  const bool endings = P.eos >= 0 && P.eos < P.V;
  if (tid == 0) {
    S.count = S.hits = S.flag = 0u;
    S.near = 0ull;
  }
  __syncthreads();
  grid_dependency_wait();

  // ---- the rows' sums
#pragma unroll 1
  for (int w = warp; w < W; w += kWarps) {
    constexpr int kOwn = kMostSlices / 32;
    const int64_t row = row0 + w;
    const float score = P.scores[row];
    float m = -INFINITY, x_end = -INFINITY;
    float4 part[kOwn];
    if (score != -INFINITY) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (i * 32 + lane < C) part[i] = __ldcg(P.parts + row * C + i * 32 + lane);
      if (endings)
        x_end = static_cast<float>(static_cast<const T*>(P.logits)[row * P.row_stride + P.eos]);
      uint32_t key = 0u;
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (i * 32 + lane < C) key = max(key, float_key(part[i].x));
      m = key_float(__reduce_max_sync(kFull, key));
    }
    const bool bad = score != -INFINITY && (!(fabsf(score) <= kFar) || !(m < INFINITY));
    const bool live = score != -INFINITY && !bad && m > -INFINITY;
    FF off = {0.0f, 0.0f}, log = off;
    if (live) {
      FF sum = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (i * 32 < C && i * 32 + lane < C) sum = add(sum, mul(exp_below(part[i].x, m), part[i].y));
      log = log_of(warp_sum(sum));
      off = add(FF{-log.h, -log.l}, score);
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (i * 32 + lane < C)
        tops[w * C + i * 32 + lane] =
            live && part[i].z >= m - kFar ? at_least(off.h, part[i].z - m) : -INFINITY;
    if (lane == 0) {
      S.m[w] = m;
      S.x_end[w] = x_end;
      S.live[w] = live;
      S.log[w] = log;
      S.off[w] = off;
      S.score[w] = score;
      if (bad) atomicOr(&S.flag, PKV_ST_NONFINITE);
      else if (score != -INFINITY && !live) atomicOr(&S.flag, PKV_ST_ALL_NEG_INF);
    }
  }
  __syncthreads();
  if (tid == 0 && S.flag != 0u && P.status != nullptr)
    atomicOr(P.status, static_cast<int>(S.flag));
  // At least every t (for good: offsets that are refined move by less).
  float best = -INFINITY;
#pragma unroll
  for (int i = 0; i < PKV_MAX_BEAMS; i += 32)
    if (i + lane < W && S.live[i + lane] != 0) best = fmaxf(best, S.off[i + lane].h);
  best = key_float(__reduce_max_sync(kFull, float_key(best))) + 1e-4f;

  // ---- a threshold that n_out candidates reach, the endings apart
  uint32_t have;
  float least = nth_bound(S, tops, pairs, n_out, best, &have);
  auto add_hits = [&](float t) {
    if (tid < W) {
      const float off = S.off[tid].h, x = t - off;
      S.xmin[tid] = fmaxf(S.m[tid] - kFar, __fadd_rd(__fsub_rd(x, slack(off, x)), S.m[tid]));
    }
    // (From a slice's lower bound up to its upper one: twice its slack.)
    for (int i = tid; i < pairs; i += kThreads)
      if (tops[i] > -INFINITY && tops[i] + 3.0f * slack(S.off[i / C].h, tops[i]) >= t)
        hits[atomicAdd(&S.hits, 1u)] = static_cast<uint16_t>(i);
    __syncthreads();
  };
  // The vectors of hit slice i.
  auto load_slice = [&](int i, int* w, int* k0, uint4 (&v)[kVecs]) {
    *w = hits[i] / C;
    *k0 = (hits[i] - *w * C) * kSlice + lane;
    const Row<T> r = row_of<T>(P, static_cast<int>(row0) + *w);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) v[k] = load_vector(r, *k0 + k * 32);
    return r;
  };
  add_hits(least);
  if (least == -INFINITY && have > 0u && static_cast<int>(have) * 32 >= n_out) {
    // Few slices hold any: the same by their lanes.
    const int few = static_cast<int>(S.hits);  // < n_out
#pragma unroll 1
    for (int i = warp; i < few; i += kWarps) {
      int w, k0;
      uint4 v[kVecs];
      const Row<T> r = load_slice(i, &w, &k0, v);
      const int end = endings ? P.eos + r.lead : -1;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        float x[kPer];
        unpack_row<T>(r, P.V, k0 + k * 32, v[k], end, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) top = fmaxf(top, x[e]);
      }
      S.lanes[i * 32 + lane] = top > -INFINITY && top >= S.m[w] - kFar
                                   ? at_least(S.off[w].h, top - S.m[w]) : -INFINITY;
    }
    __syncthreads();
    least = nth_bound(S, S.lanes, few * 32, n_out, best, &have);
    if (tid == 0) S.hits = 0u;
    __syncthreads();
    add_hits(least);
  }

  // ---- what reaches it
  const int n_hits = static_cast<int>(S.hits);
#pragma unroll 1
  for (int i = warp; i < n_hits; i += kWarps) {
    int w, k0;
    uint4 v[kVecs];
    const Row<T> r = load_slice(i, &w, &k0, v);
    const int end = endings ? P.eos + r.lead : -1;
    const float xmin = S.xmin[w];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      float x[kPer];
      unpack_row<T>(r, P.V, k0 + k * 32, v[k], end, x);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < kPer; ++e) top = fmaxf(top, x[e]);
      if (!(top > -INFINITY && top >= xmin)) continue;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (x[e] > -INFINITY && x[e] >= xmin) {
          const uint32_t at = atomicAdd(&S.count, 1u);
          if (at < kCand) {
            S.x[at] = x[e];
            S.id[at] = static_cast<uint32_t>(w) << 20 |
                       static_cast<uint32_t>((k0 + k * 32) * kPer + e - r.lead);
          }
        }
      }
    }
  }
  __syncthreads();
  const bool many = S.count > kCand;
  __syncthreads();
  auto refine = [&](int w) {
    const FF log = log_of(exact_sum<T>(P, S, static_cast<int>(row0) + w, S.m[w]));
    if (tid == 0) {
      S.log[w] = log;
      S.off[w] = add(FF{-log.h, -log.l}, S.score[w]);
    }
    __syncthreads();
  };
  if (many) {
    // Too many equal or nearly equal ones for the list (flat rows): all sums again, and
    // each row's best, of which the best so far stay.
    if (tid == 0) S.count = 0u;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < W; ++w) {
      if (S.live[w] == 0) continue;
      refine(w);
      row_best<T>(P, S, w, static_cast<int>(row0) + w);
      const int c = static_cast<int>(S.count);  // at most 2 n_out
      if (tid < c) {
        make_keys(S, tid, best);
        make_words(S, tid);
      }
      __syncthreads();
      rank_all<true>(S, c, n_out, best);
      __syncthreads();
      int to = n_out;
      float x = 0.0f;
      uint32_t id = 0u;
      if (tid < c) {
        to = S.rank[tid];
        x = S.x[tid];
        id = S.id[tid];
      }
      __syncthreads();
      if (to < n_out) {
        S.x[to] = x;
        S.id[to] = id;
      }
      if (tid == 0) S.count = min(c, n_out);
      __syncthreads();
    }
  }
  const int going = static_cast<int>(S.count);
  __syncthreads();
  if (endings && tid < W && S.live[tid] != 0 && S.x_end[tid] > -INFINITY &&
      S.x_end[tid] >= S.m[tid] - kFar) {
    const uint32_t at = atomicAdd(&S.count, 1u);
    S.x[at] = S.x_end[tid];
    S.id[at] = kEnd | static_cast<uint32_t>(tid) << 20 | static_cast<uint32_t>(P.eos);
  }
  if (tid < W && P.ended != nullptr) P.ended[row0 + tid] = -INFINITY;
  __syncthreads();
  const int c = static_cast<int>(S.count);

  // ---- ranks, again where the sums' errors leave them open
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const bool exact = pass > 0 || many;
    for (int i = tid; i < c; i += kThreads) {
      make_keys(S, i, best);
      if (exact) make_words(S, i);
    }
    __syncthreads();
    if (exact) rank_all<true>(S, c, n_out, best);
    else rank_all<false>(S, c, n_out, best);
    __syncthreads();
    const unsigned long long again = pass == 0 ? S.near : 0ull;
    if (again == 0ull) break;
#pragma unroll 1
    for (int w = 0; w < W; ++w)
      if ((again >> w) & 1ull) refine(w);
  }

  // ---- results
  for (int i = tid; i < c; i += kThreads) {
    const uint32_t id = S.id[i];
    if (S.rank[i] >= n_out) continue;
    const int w = beam_of(id);
    const float t = total(S, w, S.x[i]).h;
    if ((id & kEnd) != 0u) {
      if (P.ended != nullptr) P.ended[row0 + w] = t;
      continue;
    }
    const int64_t at = static_cast<int64_t>(b) * n_out + S.rank[i];
    P.out_parents[at] = w;
    P.out_tokens[at] = token_of(id);
    P.out_scores[at] = t;
  }
  for (int i = going + tid; i < n_out; i += kThreads) {
    const int64_t at = static_cast<int64_t>(b) * n_out + i;
    P.out_parents[at] = -1;
    P.out_tokens[at] = -1;
    P.out_scores[at] = -INFINITY;
  }
}

template <typename T>
int64_t slice_count(int V) {
  constexpr int kPer = Elements<T>::kPer;
  // (A row may begin anywhere in its first vector.)
  return div_ceil(div_ceil(static_cast<int64_t>(V) + kPer - 1, kPer), kSlice);
}

int64_t slice_count(int V, pkv_dtype dt) {
  return dt == PKV_BF16 ? slice_count<__nv_bfloat16>(V) : slice_count<float>(V);
}

template <typename T>
cudaError_t launch(const BeamParams& P, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0ull};
  const auto finish = beam_finish_kernel<T>;
  cudaError_t e = set_smem_limit_once(done, finish,
                                      static_cast<int>(finish_bytes(PKV_MAX_BEAMS * kMostSlices)));
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(P.B) * P.W * P.slices;
  const int64_t ctas = std::min<int64_t>(div_ceil(items, kStreamWarps), 4 * num_sms());
  e = launch_early(beam_stream_kernel<T>, dim3(static_cast<unsigned>(ctas)), kStreamWarps * 32, 0, s, P);
  if (e != cudaSuccess) return e;
  return launch_early(finish, dim3(static_cast<unsigned>(P.B)), kThreads, finish_bytes(P.W * P.slices),
                      s, P);
}

int beam_sizes_error(int B, int W, int V, pkv_dtype dt) {
  if (dt != PKV_FP32 && dt != PKV_BF16)
    return fail(PKV_EINVAL, "dtype %d is not fp32 or bf16", static_cast<int>(dt));
  if (B < 0 || B > 65535) return fail(PKV_EINVAL, "B=%d outside [0, 65535]", B);
  if (W < 1 || W > PKV_MAX_BEAMS) return fail(PKV_EINVAL, "W=%d outside [1, %d]", W, PKV_MAX_BEAMS);
  if (static_cast<int64_t>(B) * W > 65535) return fail(PKV_EINVAL, "B * W=%lld above 65535",
                                                       (long long)B * W);
  if (V < 1) return fail(PKV_EINVAL, "V=%d < 1", V);
  const int max_v = dt == PKV_BF16 ? PKV_MAX_VOCAB_BF16 : PKV_MAX_VOCAB_FP32;
  if (V > max_v) return fail(PKV_EUNSUPPORTED, "V=%d above the maximum %d", V, max_v);
  return PKV_OK;
}

}  // namespace

}  // namespace pkv

extern "C" size_t pkv_beam_select_workspace_bytes(int B, int W, int V, pkv_dtype dt) {
  using namespace pkv;
  if (beam_sizes_error(B, W, V, dt) != PKV_OK) return 0;
  return static_cast<size_t>(static_cast<int64_t>(B) * W * slice_count(V, dt)) * sizeof(float4);
}

extern "C" int pkv_beam_select(const void* logits, pkv_dtype dt, int B, int W, int V,
                               int64_t row_stride, const float* scores, int n_out, int eos,
                               int32_t* out_parents, int32_t* out_tokens, float* out_scores,
                               float* ended, int32_t* status, void* workspace,
                               size_t workspace_bytes, pkv_stream_t stream) {
  using namespace pkv;
  const int bad = beam_sizes_error(B, W, V, dt);
  if (bad != PKV_OK) return bad;
  if (row_stride < V)
    return fail(PKV_EINVAL, "row_stride=%lld < V=%d", (long long)row_stride, V);
  if (n_out < 1 || n_out > PKV_MAX_BEAMS)
    return fail(PKV_EINVAL, "n_out=%d outside [1, %d]", n_out, PKV_MAX_BEAMS);
  if (B == 0) return ok();
  if (logits == nullptr || scores == nullptr || out_parents == nullptr || out_tokens == nullptr ||
      out_scores == nullptr)
    return fail(PKV_EINVAL, "NULL pointer argument");
  if (reinterpret_cast<uintptr_t>(logits) % (dt == PKV_BF16 ? 2 : 4) != 0)
    return fail(PKV_EINVAL, "logits are not aligned to their type");
  const size_t rows = static_cast<size_t>(B) * W, picks = static_cast<size_t>(B) * n_out;
  if ((overlap(scores, rows * 4, out_scores, picks * 4) && !(scores == out_scores && n_out == W)) ||
      overlap(scores, rows * 4, ended, ended != nullptr ? rows * 4 : 0))
    return fail(PKV_EINVAL, "an output overlaps the scores");
  const size_t need = pkv_beam_select_workspace_bytes(B, W, V, dt);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PKV_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned16(workspace)) return fail(PKV_EINVAL, "workspace is not 16-byte aligned");
  BeamParams P;
  P.logits = logits;
  P.row_stride = row_stride;
  P.scores = scores;
  P.out_parents = out_parents, P.out_tokens = out_tokens, P.out_scores = out_scores;
  P.ended = ended;
  P.status = status;
  P.B = B, P.W = W, P.V = V, P.n_out = n_out, P.eos = eos;
  P.slices = static_cast<int>(slice_count(V, dt));
  P.parts = static_cast<float4*>(workspace);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == PKV_BF16 ? launch<__nv_bfloat16>(P, s) : launch<float>(P, s);
  if (e != cudaSuccess) return cuda_fail(e, "beam launch");
  return ok();
}
