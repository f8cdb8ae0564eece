// pkv_select_pages: for each query token and cache head, the pages that its
// attention is to read.
//
//   score(page) = max over g of k_scale sum_d max(q_gd lo_d, q_gd hi_d)
//               = max over g of k_scale (q+_g . hi + q-_g . lo)
//
// with q+ and q- the parts of q above and below zero: a product of the page's
// bounds, one row of 2 D codes, with a column [q-; q+] for each query head.
//
// Two kernels.  (1) Every CTA sums up the requests' work; its warps take equal shares of
// all (token, head)s' pages, 16 at a time as the rows of mma.m16n8k16 (codes are exact in
// fp16, and queries scaled by a power of two, but for elements below 2^-31 of the
// largest), up to 8 query heads as its columns.  Bounds come through a warp's ring of
// shared memory, two products ahead.  (2) A CTA a (token, head) finds the k-th largest
// score (a histogram, then the ranks within its bin) and lists the pages in order.
//
// Exact choice.  The product's 16 steps are each off by at most 2^-22 of the sum of
// the terms' magnitudes, which is at most 448 k_scale sum_d |q_d|: e = 2^-17 of that
// bounds a score's error, so the k-th largest true score lies within e_max of the
// k-th largest score T, and only pages whose score is within e + e_max of T can be
// taken or left wrongly.  Where there are more of those than places, their sums
// are taken again as sums of two fp32 values (products of a query's 11 bits, scaled as
// above, with a code's 4 are exact in fp32), and their places in the order stand where the
// scores were.
//
// Bound: for many long requests the bounds' bytes, after 10 us of dependent loads (place,
// page, bounds); for few tokens those chains.  64 requests of up to 32768, 8 heads of 128,
// pages of 16: 59 us, of which the scores 40 (150 MB) and the choice the rest; one of
// 36863: 18 us.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "attend_params.h"
#include "attend_units.cuh"
#include "device_attr.h"
#include "device_common.cuh"
#include "double_float.cuh"
#include "kv_cache.cuh"
#include "launch_early.h"
#include "page_kernels.h"
#include "radix_nth.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;       // of the first kernel
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;           // pages of a product
constexpr int kStages = 3;          // products of a warp whose bounds are under way
constexpr int kLead = 2;            // cost of a (token, head)'s start, in products
constexpr int kBins = 1024;
constexpr int kFew = 256;           // pages that are ranked all against all
constexpr int kHeld = 4096;         // scores kept in shared memory; more are read again
constexpr int kAhead = 4;           // loads of a thread that are on their way at once
constexpr float kDown = 0x1p-32f;   // keeps scores under scales of up to 2^119 finite
constexpr uint32_t kNoRow = ~0u, kNoScale = 0x7fc0dead;  // of no page: none, and a NaN of its own
constexpr float kNoPage = -3.0e38f; // below all scores

struct SelectParams {
  AttendParams a;         // q, lengths, table, cache
  const uint8_t* bounds;
  int32_t* pages;         // [n_tokens, kv_heads, budget]
  int32_t* lengths;       // [n_tokens]
  int2* where;            // workspace: [n_tokens] table row, position or -1
  float2* sums;           // workspace: [n_tokens, kv_heads] Cell::sums and unit
  float2* score;          // workspace: [n_tokens, kv_heads, most]: score and scale, then, where
                          // sums are in doubt, a page's place in the order
  int most;               // pages of a table row
  int budget, sink, recent;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^e that puts x (the largest magnitude of the head's queries) in [2^14, 2^15).
__device__ __forceinline__ float unit_for(float x) {
  const int e = static_cast<int>(__float_as_uint(x) >> 23);
  return __uint_as_float(static_cast<uint32_t>(max(1, min(268 - e, 253))) << 23);
}

// The page of a location, or -1.
__device__ __forceinline__ int page_of(const AttendParams& A, int loc) {
  const int slots = static_cast<int>(A.c.num_pages * A.c.page_size);
  return loc >= 0 && loc < slots ? static_cast<int>(A.page_div.divide(static_cast<uint32_t>(loc)))
                                 : -1;
}

// The page that logical page b of a table row is, or -1.
__device__ __forceinline__ int page_at(const AttendParams& A, int row, int b) {
  return page_of(A, __ldcg(A.page_table + static_cast<int64_t>(row) * A.pt_cols +
                          static_cast<int64_t>(b) * A.c.page_size));
}

// A page's score times `unit` (measure_queries), to some 2^-46 of its terms: one warp, all
// lanes get it.  The power of two keeps products of queries at the ends of their range
// within fp32's.  Lanes share a query head's dimensions, as few as the heads allow: the
// sums' chains are what it waits for.
template <typename T>
__device__ double exact_score(const SelectParams& P, const uint16_t* q, float unit, int row, int h,
                              int b) {
  const AttendParams& A = P.a;
  const int lane = threadIdx.x & 31;
  const int page = page_at(A, row, b);
  if (page < 0) return -1.0e308;
  const int64_t at = static_cast<int64_t>(page) * A.c.kv_heads + h;
  const uint8_t* bounds = P.bounds + at * 2 * A.c.head_dim;
  const int each = A.group > 4 ? 4 : A.group > 2 ? 8 : A.group > 1 ? 16 : 32;  // lanes of a head
  float best_h = -INFINITY, best_l = 0.0f;
  for (int g0 = 0; g0 < A.group; g0 += 32 / each) {
    const int g = g0 + lane / each;
    FF s = {0.0f, 0.0f};
    if (g < A.group) {
      for (int d = (lane % each) * 4; d < A.c.head_dim; d += each * 4) {
        const uint32_t lo = *reinterpret_cast<const uint32_t*>(bounds + d);
        const uint32_t hi = *reinterpret_cast<const uint32_t*>(bounds + A.c.head_dim + d);
        const uint2 x = *reinterpret_cast<const uint2*>(q + g * A.q_hs + d);
        const float2 l0 = Pair<__half>::unpack(e4m3x2_to_f16x2(lo));
        const float2 l1 = Pair<__half>::unpack(e4m3x2_to_f16x2(lo >> 16));
        const float2 h0 = Pair<__half>::unpack(e4m3x2_to_f16x2(hi));
        const float2 h1 = Pair<__half>::unpack(e4m3x2_to_f16x2(hi >> 16));
        float2 a = Pair<T>::unpack(x.x), z = Pair<T>::unpack(x.y);
        a.x *= unit, a.y *= unit, z.x *= unit, z.y *= unit;
        const FF u = two_sum(fmaxf(a.x * l0.x, a.x * h0.x), fmaxf(a.y * l0.y, a.y * h0.y));
        const FF v = two_sum(fmaxf(z.x * l1.x, z.x * h1.x), fmaxf(z.y * l1.y, z.y * h1.y));
        s = add(s, add(u, v));
      }
    }
#pragma unroll 1
    for (int o = each / 2; o > 0; o >>= 1)
      s = add(s, {__shfl_xor_sync(kFull, s.h, o), __shfl_xor_sync(kFull, s.l, o)});
    if (g < A.group && (s.h > best_h || (s.h == best_h && s.l > best_l))) best_h = s.h, best_l = s.l;
  }
  double best = static_cast<double>(best_h) + static_cast<double>(best_l);
#pragma unroll 1
  for (int o = 16; o >= each; o >>= 1) best = fmax(best, __shfl_xor_sync(kFull, best, o));
  return best * static_cast<double>(A.c.k_scale[at]);
}

// An order of doubles as whole numbers; never 0 or kSure.
__device__ __forceinline__ unsigned long long double_key(double x) {
  const long long b = __double_as_longlong(x + 0.0);
  return static_cast<unsigned long long>(b) ^
         (static_cast<unsigned long long>(b >> 63) | 0x8000000000000000ull);
}

constexpr unsigned long long kSure = ~0ull;  // above all of those

// What a warp of the CTA knows of its (token, head).
struct Cell {
  const uint16_t* q;  // the head's queries
  int row, count;     // table row, pages
  int h;
  float unit;         // scale of the queries
  float sums;         // largest sum of magnitudes of a query, scaled
};

// Queries' largest element and sum, by one warp: c's unit and sums.
template <typename T>
__device__ __forceinline__ void measure_queries(const SelectParams& P, Cell& c) {
  const AttendParams& A = P.a;
  const int lane = threadIdx.x & 31, each = A.c.head_dim >> 3;  // vectors of a row
  float amax = 0.0f, sums = 0.0f;
  for (int g0 = 0; g0 < A.group; g0 += 2) {  // half a warp a row (of at most 16 vectors)
    const int g = g0 + (lane >> 4), d = lane & 15;
    float sum = 0.0f;
    if (g < A.group && d < each) {
      const uint4 x = *reinterpret_cast<const uint4*>(c.q + g * A.q_hs + d * 8);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = Pair<T>::unpack(xs[k]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        sum += fabsf(f.x) + fabsf(f.y);
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    sums = fmaxf(sums, sum);
  }
  sums = fmaxf(sums, __shfl_xor_sync(kFull, sums, 16));
  amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
  c.unit = unit_for(amax);
  c.sums = sums * c.unit;
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// Scores of the pages [b0, end) of a cell, by one warp through its ring of kStages *
// kTile * KW * 64 bytes of shared memory.  KW: 16-byte pieces of a page's bounds that a
// lane holds.
template <typename T, int KW>
__device__ __forceinline__ void score_pages(const SelectParams& P, Cell& c, int b0, int end,
                                            float2* score, uint32_t ring) {
  constexpr int kPieces = 4 * KW, kRow = kPieces * 16;  // of a page in the ring
  const AttendParams& A = P.a;
  const int lane = threadIdx.x & 31, r = lane >> 2, col = lane & 3;
  const int dim = A.c.head_dim, halves = dim >> 4, heads = A.c.kv_heads;
  const int tiles = (end - b0 + kTile - 1) / kTile;
  // Bounds' places and scales of two products, one a lane: of those computed (scales
  // alone), of the next two and, as yet their locations, of the two after.
  const int32_t* table = A.page_table + static_cast<int64_t>(c.row) * A.pt_cols;
  auto look = [&](int pair) {
    const int b = b0 + 32 * pair + lane;
    return b < end ? __ldcg(table + static_cast<int64_t>(b) * A.c.page_size) : -1;
  };
  // (In units of 32 bytes, which a row of 2 dim is a multiple of: 32 bits reach 128 GiB.)
  const uint32_t step = static_cast<uint32_t>(dim >> 4);
  auto row_of = [&](int page) {
    return page >= 0 ? (static_cast<uint32_t>(page) * heads + c.h) * step : kNoRow;
  };
  auto scale_of = [&](int page) {
    return page >= 0 ? __ldcg(A.c.k_scale + static_cast<int64_t>(page) * heads + c.h)
                     : __uint_as_float(kNoScale);
  };
  int page = page_of(A, look(0));
  int loc = look(1);
  uint32_t from = row_of(page);
  float ks = 0.0f, ks_next = scale_of(page);
  // (8 lanes read four pieces of two neighbouring rows: into different banks.)
  auto place = [](int row, int piece) { return row * kRow + ((piece ^ ((row & 1) << 2)) << 4); };
  constexpr int kAt = 32 / kPieces;  // rows of a round
  const int piece = lane % kPieces;
  const uint8_t* base = P.bounds + piece * 16;
  auto issue = [&](int t) {
    if (t < tiles) {
      const uint32_t slot = ring + (t % kStages) * (kTile * kRow);
#pragma unroll
      for (int i = 0; i < kTile / kAt; ++i) {
        const int row = i * kAt + lane / kPieces;
        const uint32_t at = __shfl_sync(kFull, from, ((t & 1) << 4) + row);
        const bool valid = at != kNoRow && piece < 2 * halves;
        cp_async16_zfill(slot + place(row, piece),
                         valid ? base + static_cast<uint64_t>(at) * 32 : P.bounds, valid);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  static_assert(kStages == 3, "two products ahead: the next pair's");
  issue(0);
  issue(1);
  measure_queries<T>(P, c);
  uint32_t qf[KW * 8];
  auto load_queries = [&](int g0) {
    const int g = g0 + r;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int piece = col + 4 * k;
      const bool upper = piece >= halves;
      const int d = (upper ? piece - halves : piece) * 16;
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      if (g < A.group && piece < 2 * halves) {
        x = *reinterpret_cast<const uint4*>(c.q + g * A.q_hs + d);
        y = *reinterpret_cast<const uint4*>(c.q + g * A.q_hs + d + 8);
      }
      const uint32_t xs[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f = Pair<T>::unpack(xs[i]);
        f.x *= c.unit, f.y *= c.unit;
        f.x = upper ? fmaxf(f.x, 0.0f) : fminf(f.x, 0.0f);
        f.y = upper ? fmaxf(f.y, 0.0f) : fminf(f.y, 0.0f);
        qf[8 * k + i] = Pair<__half>::pack(f.x, f.y);
      }
    }
  };
  load_queries(0);
#pragma unroll 1
  for (int t = 0; t < tiles; ++t) {
    if ((t & 1) == 0) {
      ks = ks_next;
      page = page_of(A, loc);
      loc = look(t / 2 + 2);
      from = row_of(page);
      ks_next = scale_of(page);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    const uint32_t slot = ring + (t % kStages) * (kTile * kRow);
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int g0 = 0; g0 < A.group; g0 += 8) {
      if (A.group > 8) load_queries(g0);
      float s[2][4] = {};  // two sums, so that products wait less for one another
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const uint4 u = lds128(slot + place(r, col + 4 * k));
        const uint4 v = lds128(slot + place(r + 8, col + 4 * k));
        const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma16816(s[i & 1], e4m3x2_to_f16x2(x[i]), e4m3x2_to_f16x2(y[i]),
                   e4m3x2_to_f16x2(x[i] >> 16), e4m3x2_to_f16x2(y[i] >> 16), qf[8 * k + 2 * i],
                   qf[8 * k + 2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (g0 + 2 * col + (i & 1) < A.group) {
          best[i >> 1] = fmax_nan(best[i >> 1], s[0][i] + s[1][i]);
        }
      }
    }
    __syncwarp();  // the slot may be refilled
    issue(t + kStages - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      best[i] = fmax_nan(best[i], __shfl_xor_sync(kFull, best[i], 1));
      best[i] = fmax_nan(best[i], __shfl_xor_sync(kFull, best[i], 2));
      const int row = r + 8 * i, at = b0 + t * kTile + row;
      const float scale = __shfl_sync(kFull, ks, ((t & 1) << 4) + row);
      if (col == 0 && at < end) {
        // (A NaN: above all, and no error to reckon with.)
        const float x = best[i] * (scale * kDown);
        const float2 out = __float_as_uint(scale) == kNoScale ? make_float2(kNoPage, 0.0f)
                           : isfinite(x)                      ? make_float2(x, scale)
                                                              : make_float2(INFINITY, 0.0f);
        __stcg(score + at, out);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Products for the pages of one of a request's (token, head), its last token's: 0 where
// all pages are taken, or the request is refused.
__device__ __forceinline__ int request_tiles(const SelectParams& P, const Request& r) {
  if (r.bad != 0 || r.q_len == 0) return 0;
  const int count = (r.end - 1) / P.a.c.page_size + 1;
  return count > P.budget ? (count + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ int64_t request_cost(const SelectParams& P, const Request& r) {
  const int tiles = request_tiles(P, r);
  return tiles > 0 ? static_cast<int64_t>(tiles + kLead) * r.q_len * P.a.c.kv_heads : 0;
}

// The last of the ascending x[0 .. kThreads) that is at most v; x[0] is.
__device__ __forceinline__ int last_within(const int64_t* x, int64_t v) {
  int lo = 0, hi = kThreads;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (x[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int KW>
__host__ __device__ constexpr int ring_bytes() { return kWarps * kStages * kTile * KW * 64; }

template <typename T, int KW>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const __grid_constant__ SelectParams P) {
  extern __shared__ __align__(128) uint8_t smem[];  // the warps' rings
  // Cost and tokens before each thread's requests.
  __shared__ int64_t s_cost[kThreads], s_tok[kThreads], s_sum[2][kWarps];
  const AttendParams& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = A.c.kv_heads, ps = A.c.page_size;
  launch_dependents();
  grid_dependency_wait();
  const int per = (A.B + kThreads - 1) / kThreads;
  const int i0 = min(A.B, tid * per), i1 = min(A.B, i0 + per);
  int64_t cost = 0, toks = 0;
  int bad = 0;
  for (int i = i0; i < i1; ++i) {
    const Request r = load_request(A, i);
    bad |= r.bad;
    toks += r.q_len;
    cost += request_cost(P, r);
  }
  int64_t ci = cost, ti = toks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(kFull, ci, o), y = __shfl_up_sync(kFull, ti, o);
    if (lane >= o) ci += x, ti += y;
  }
  if (lane == 31) s_sum[0][warp] = ci, s_sum[1][warp] = ti;
  __syncthreads();
  ci -= cost, ti -= toks;
  int64_t total = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) ci += s_sum[0][w], ti += s_sum[1][w];
    total += s_sum[0][w], all += s_sum[1][w];
  }
  s_cost[tid] = ci;
  s_tok[tid] = ti;
  if (blockIdx.x == 0 && A.status != nullptr) {
    if (tid == 0 && all > A.n_tokens) bad |= PKV_ST_TOKEN_CAP;
    if (bad != 0) atomicOr(A.status, bad);
  }
  __syncthreads();
  // ---- where the tokens are
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + tid; j < A.n_tokens;
       j += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int k = last_within(s_tok, j);
    int64_t t = j - s_tok[k];
    int2 w = make_int2(-1, -1);
    int length = 0;
    for (int i = k * per; i < A.B; ++i) {
      const Request r = load_request(A, i);
      if (t >= r.q_len) {
        t -= r.q_len;
        continue;
      }
      if (r.bad == 0) {
        const int p = r.cached + static_cast<int>(t);
        w = make_int2(r.table_row, p);
        length = (min(p / ps + 1, P.budget) - 1) * ps + p % ps + 1;
      }
      break;
    }
    P.where[j] = w;
    P.lengths[j] = length;
  }
  // ---- this warp's share of the products
  const int64_t workers = min(static_cast<int64_t>(gridDim.x) * kWarps, total);
  const int64_t me = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  if (me >= workers) return;
  const int64_t first = me * total / workers;
  int64_t left = (me + 1) * total / workers - first;
  const int k = last_within(s_cost, first);
  int64_t at = first - s_cost[k], q_off = s_tok[k];
  int req = k * per;
  Request r = load_request(A, req);
  for (int64_t n = request_cost(P, r); at >= n; n = request_cost(P, r)) {
    at -= n;
    q_off += r.q_len;
    r = load_request(A, ++req);
  }
  int whole = request_tiles(P, r) + kLead;
  const int64_t cell = at / whole;
  at -= cell * whole;
  Cell c;
  c.h = static_cast<int>(cell / r.q_len);
  int tok = static_cast<int>(cell - static_cast<int64_t>(c.h) * r.q_len);
  const uint32_t ring = smem_addr(smem) + warp * (ring_bytes<KW>() / kWarps);
  for (;;) {
    const int64_t j = q_off + tok;
    const int take = static_cast<int>(min(left, whole - at));
    const int t0 = max(0, static_cast<int>(at) - kLead);
    const int t1 = max(0, static_cast<int>(at) + take - kLead);
    c.row = r.table_row;
    c.count = (r.cached + tok) / ps + 1;
    const int b0 = t0 * kTile, end = min(c.count, t1 * kTile);
    if (j < A.n_tokens && c.count > P.budget && b0 < end) {
      c.q = A.q + j * A.q_ts + static_cast<int64_t>(c.h) * A.group * A.q_hs;
      score_pages<T, KW>(P, c, b0, end, P.score + (j * heads + c.h) * P.most, ring);
      if (t0 == 0 && lane == 0) __stcg(P.sums + j * heads + c.h, make_float2(c.sums, c.unit));
    }
    left -= take;
    if (left <= 0) break;
    at = 0;
    if (++tok == r.q_len) {
      tok = 0;
      if (++c.h == heads) {
        c.h = 0;
        do {
          q_off += r.q_len;
          r = load_request(A, ++req);
        } while (request_tiles(P, r) == 0);
        whole = request_tiles(P, r) + kLead;
      }
    }
  }
}

template <int THREADS>
struct PickShared {
  NthScratch<THREADS> nth;
  float score[kHeld];
  unsigned long long key[kFew];
  float red[3][THREADS / 32];
  int sum[2][THREADS / 32];
  int few;
};

// Lists a cell's pages, by one CTA, whose warps have neighbouring pages each.
template <typename T, int THREADS>
__device__ void pick_pages(const SelectParams& P, PickShared<THREADS>& S, const Cell& c,
                           float2* score, int32_t* out) {
  constexpr int kWarps = THREADS / 32;
  const AttendParams& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m0 = P.sink, m1 = c.count - P.recent;     // pages that compete
  const int k = P.budget - P.sink - P.recent;         // for so many places
  const bool held = m1 - m0 <= kHeld;
  const int chunk = (c.count + THREADS - 1) / THREADS * 32;
  const int w0 = min(c.count, warp * chunk), w1 = min(c.count, w0 + chunk);
  const int b0 = max(w0, m0) + lane, b1 = min(w1, m1);  // this lane's that compete: every 32nd
  auto at = [&](int b) { return held ? S.score[b - m0] : __ldcg(&score[b].x); };
  // Sums of x and y over the warps before, and over all.
  auto scan = [&](int x, int y, int2* all) {
    if (lane == 0) S.sum[0][warp] = x, S.sum[1][warp] = y;
    __syncthreads();
    x = lane < kWarps ? S.sum[0][lane] : 0, y = lane < kWarps ? S.sum[1][lane] : 0;
    *all = make_int2(__reduce_add_sync(kFull, x), __reduce_add_sync(kFull, y));
    const int2 before = make_int2(__reduce_add_sync(kFull, lane < warp ? x : 0),
                                  __reduce_add_sync(kFull, lane < warp ? y : 0));
    __syncthreads();
    return before;
  };
  float t = 0.0f, e = 0.0f;    // the k-th largest score; those within e of it are in doubt
  auto in_doubt = [&](float s) { return s == t || fabsf(s - t) <= e; };
  if (k > 0) {
    // The scores' range and the largest scale.
    float hi = kNoPage, lo = INFINITY, scale = 0.0f;
    for (int first = b0; first < b1; first += 32 * kAhead) {
      float2 s[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        s[i] = make_float2(INFINITY, 0.0f);
        if (first + 32 * i < b1) s[i] = __ldcg(score + first + 32 * i);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (held && first + 32 * i < b1) S.score[first + 32 * i - m0] = s[i].x;
        scale = fmaxf(scale, s[i].y);
        if (s[i].x < INFINITY && s[i].x != kNoPage) hi = fmaxf(hi, s[i].x), lo = fminf(lo, s[i].x);
      }
    }
    auto widest = [&]() {
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        scale = fmaxf(scale, __shfl_xor_sync(kFull, scale, o));
      }
    };
    widest();
    for (int i = tid; i < kBins; i += THREADS) S.nth.bins[i] = 0u;
    if (lane == 0) S.red[0][warp] = hi, S.red[1][warp] = lo, S.red[2][warp] = scale;
    if (tid == 0) S.few = 0;
    __syncthreads();
    const int other = lane < kWarps ? lane : 0;
    hi = S.red[0][other], lo = S.red[1][other], scale = S.red[2][other];
    widest();
    // Bins of equal width from the largest score down; a NaN page's in the first, one
    // that is no page's in the last.
    const float inv = hi > lo ? (kBins - 0.5f) / (hi - lo) : 0.0f;
    auto bin_of = [&](float s) {
      return s == kNoPage ? kBins - 1
                          : static_cast<int>(fminf(fmaxf((hi - s) * inv, 0.0f), kBins - 1.0f));
    };
#pragma unroll 2
    for (int b = b0; b < b1; b += 32) atomicAdd(&S.nth.bins[bin_of(at(b))], 1u);
    __syncthreads();
    // The bin of the k-th largest: a thread has kOwn of them.
    constexpr int kOwn = kBins / THREADS;
    int own = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own += static_cast<int>(S.nth.bins[tid * kOwn + i]);
    const int incl = warp_inclusive_scan(own, lane);
    int2 all;
    const int n = scan(__shfl_sync(kFull, incl, 31), 0, &all).x + incl - own;
    if (n < k && n + own >= k) {
      int bin = tid * kOwn, m = n;
      while (m + static_cast<int>(S.nth.bins[bin]) < k) m += static_cast<int>(S.nth.bins[bin++]);
      S.nth.prefix = static_cast<uint32_t>(bin);
      S.nth.left = static_cast<uint32_t>(k - m);
      S.nth.scan[0] = S.nth.bins[bin];
    }
    __syncthreads();
    const int bin = static_cast<int>(S.nth.prefix), left = static_cast<int>(S.nth.left);
    const int inside = static_cast<int>(S.nth.scan[0]);
    if (inside <= kFew) {
#pragma unroll 2
      for (int b = b0; b < b1; b += 32) {
        const float s = at(b);
        if (bin_of(s) == bin) S.key[atomicAdd(&S.few, 1)] = float_key(s);
      }
      __syncthreads();
      if (tid < inside) {
        const unsigned long long mine = S.key[tid];
        int better = 0, same = 0;
        for (int i = 0; i < inside; ++i) {
          better += S.key[i] > mine ? 1 : 0;
          same += S.key[i] == mine ? 1 : 0;
        }
        if (better < left && better + same >= left) S.red[0][0] = key_float(static_cast<uint32_t>(mine));
      }
      __syncthreads();
      t = S.red[0][0];
    } else {
      __syncthreads();
      uint32_t m;
      t = key_float(nth_key<THREADS, 3>(S.nth, k, &m, [&](auto&& f) {
        for (int b = b0; b < b1; b += 32) f(float_key(at(b)));
      }));
    }
    // Each score, and so the k-th largest, is off by at most half of this.
    e = 2.0f * (0x1p-17f * 448.0f * kDown) * c.sums * scale;
  }
  // With sums taken again, their order by whole numbers in the scores' places: 0 for a page
  // that is not taken and kSure for one that is, but where scores are held those in doubt
  // alone have one.
  unsigned long long* const keys = reinterpret_cast<unsigned long long*>(score);
  auto key_of = [&](int b) { return held && !in_doubt(at(b)) ? 0ull : __ldcg(keys + b); };
  // 0: not taken, 1: taken, 2: in doubt; with `again`: equal to the last one taken
  unsigned long long nth = 0;
  auto kind = [&](int b, bool again) {
    if (b >= c.count) return 0;
    if (b < m0 || b >= m1) return 1;
    if (k == 0) return 0;
    if (!again || held) {
      const float s = at(b);
      if (!in_doubt(s)) return s > t ? 1 : 0;
      if (!again) return 2;
    }
    const unsigned long long y = __ldcg(keys + b);
    return y > nth ? 1 : y == nth ? 2 : 0;
  };
  int2 before, all;  // sure ones, and those in doubt (or equal)
  auto number = [&](bool again) {
    int sure = 0, open = 0;
#pragma unroll 2
    for (int b = w0; b < w1; b += 32) {
      const int x = kind(b + lane, again);
      sure += __popc(__ballot_sync(kFull, x == 1));
      open += __popc(__ballot_sync(kFull, x == 2));
    }
    before = scan(sure, open, &all);
  };
  number(false);
  const int places = P.budget - all.x;  // for those in doubt
  int ties = all.y;                     // of those equal to the last one taken, so many are
  const bool decided = all.y <= places; // none in doubt, or all of them taken
  if (!decided) {
    // Their sums again.
    const int open = all.y;
    if (tid == 0) S.few = 0;
    __syncthreads();
#pragma unroll 1
    for (int w = w0; w < w1; w += 32) {
      const int b = w + lane;
      const bool competes = b >= m0 && b < m1;
      const float s = competes ? at(b) : 0.0f;
      const bool doubt = competes && in_doubt(s);
      unsigned todo = __ballot_sync(kFull, doubt);  // (all have read their scores)
      if (!held && competes && !doubt) keys[b] = s > t ? kSure : 0ull;
      while (todo != 0u) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1u;
        const float x = __shfl_sync(kFull, s, l);
        const double y = x == INFINITY ? INFINITY : exact_score<T>(P, c.q, c.unit, c.row, c.h, w + l);
        if (lane == 0) {
          const unsigned long long key = double_key(y);
          keys[w + l] = key;
          const int i = atomicAdd(&S.few, 1);
          if (i < kFew) S.key[i] = key;
        }
      }
    }
    __syncthreads();
    if (open <= kFew) {
      // The last one taken, by rank.
      if (tid < open) {
        const unsigned long long mine = S.key[tid];
        int better = 0, same = 0;
        for (int i = 0; i < open; ++i) {
          better += S.key[i] > mine ? 1 : 0;
          same += S.key[i] == mine ? 1 : 0;
        }
        if (better < places && better + same >= places) {
          S.nth.prefix = static_cast<uint32_t>(tid);
          S.nth.left = static_cast<uint32_t>(places - better);
        }
      }
      __syncthreads();
      nth = S.key[S.nth.prefix];
      ties = static_cast<int>(S.nth.left);
    } else {
      // The upper halves' n-th largest, then that of the lower halves beside it.
      uint32_t n;
      const uint32_t up = nth_key<THREADS, 3>(S.nth, places, &n, [&](auto&& f) {
        for (int b = b0; b < b1; b += 32) {
          const unsigned long long y = key_of(b);
          f(y == kSure ? 0u : static_cast<uint32_t>(y >> 32));
        }
      });
      const int rest = static_cast<int>(S.nth.left);
      __syncthreads();
      const uint32_t low = nth_key<THREADS, 3>(S.nth, rest, &n, [&](auto&& f) {
        for (int b = b0; b < b1; b += 32) {
          const unsigned long long y = key_of(b);
          f(y != kSure && static_cast<uint32_t>(y >> 32) == up ? static_cast<uint32_t>(y) : 0u);
        }
      });
      // (0 where fewer than `rest` are above 0: it is one of those that are 0.)
      nth = static_cast<unsigned long long>(up) << 32 | low;
      ties = low != 0u ? static_cast<int>(S.nth.left) : rest - static_cast<int>(n);
    }
    number(true);
  }
  // ---- the list, in order
  const unsigned below = (1u << lane) - 1u;
  bool bad = false;
  for (int w = w0; w < w1; w += 32 * kAhead) {
    int place[kAhead], loc[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int b = w + 32 * i + lane, x = b < w1 ? kind(b, !decided) : 0;
      const unsigned sure = __ballot_sync(kFull, x == 1), equal = __ballot_sync(kFull, x == 2);
      const int q = before.y + __popc(equal & below);
      place[i] = before.x + __popc(sure & below) + min(q, ties);
      if (!(x == 1 || (x == 2 && q < ties))) place[i] = P.budget;
      if (place[i] < P.budget)
        loc[i] = A.page_table[static_cast<int64_t>(c.row) * A.pt_cols +
                              static_cast<int64_t>(b) * A.c.page_size];
      before.x += __popc(sure), before.y += __popc(equal);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (place[i] < P.budget) {
        const int page = page_of(A, loc[i]);
        out[place[i]] = page;
        bad = bad || page < 0;
      }
    }
  }
  if (bad && A.status != nullptr) atomicOr(A.status, PKV_ST_ROW_OOB);
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) pick_kernel(const __grid_constant__ SelectParams P) {
  static_assert(THREADS >= kFew, "a thread ranks a page");
  __shared__ PickShared<THREADS> S;
  const AttendParams& A = P.a;
  const int tid = threadIdx.x;
  const int64_t cell = blockIdx.x;
  const int j = static_cast<int>(cell / A.c.kv_heads);
  launch_dependents();
  grid_dependency_wait();
  const int2 w = __ldcg(P.where + j);
  const float2 sums = __ldcg(P.sums + cell);  // (not written where nothing was scored)
  Cell c;
  c.h = static_cast<int>(cell - static_cast<int64_t>(j) * A.c.kv_heads);
  c.row = w.x;
  c.count = w.y < 0 ? 0 : w.y / A.c.page_size + 1;
  int32_t* out = P.pages + cell * P.budget;
  if (c.count <= P.budget) {  // all of them
    for (int i = tid; i < P.budget; i += THREADS) {
      const int page = i < c.count ? page_at(A, c.row, i) : -1;
      out[i] = page;
      if (i < c.count && page < 0 && A.status != nullptr) atomicOr(A.status, PKV_ST_ROW_OOB);
    }
    return;
  }
  c.q = A.q + j * A.q_ts + static_cast<int64_t>(c.h) * A.group * A.q_hs;
  c.sums = sums.x;
  c.unit = sums.y;
  pick_pages<T, THREADS>(P, S, c, P.score + cell * P.most, out);
}

template <typename T, int KW>
cudaError_t launch(const SelectParams& P, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0ull};
  const auto kernel = score_kernel<T, KW>;
  cudaError_t e = set_smem_limit_once(done, kernel, ring_bytes<KW>());
  if (e != cudaSuccess) return e;
  const int64_t cells = P.a.n_tokens * P.a.c.kv_heads;
  const int64_t most = cells * div_ceil(div_ceil(P.most, kTile) + kLead, kWarps);
  const int sms = num_sms();
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(most, int64_t{2} * sms)));
  e = launch_early(kernel, grid, kThreads, ring_bytes<KW>(), s, P);
  if (e != cudaSuccess) return e;
  // Few cells: as many threads for each as there are (one request over 2304 pages: 19 us,
  // with 256 21); else all cells at once.
  const dim3 picks(static_cast<unsigned>(cells));
  return cells <= sms ? launch_early(pick_kernel<T, 1024>, picks, 1024, 0, s, P)
                      : launch_early(pick_kernel<T, 256>, picks, 256, 0, s, P);
}

template <typename T>
cudaError_t launch(const SelectParams& P, cudaStream_t s) {
  return P.a.c.head_dim > 64 ? launch<T, 4>(P, s) : launch<T, 2>(P, s);
}

int64_t round16(int64_t bytes) { return div_ceil(bytes, 16) * 16; }

}  // namespace

}  // namespace pkv

extern "C" size_t pkv_select_pages_workspace_bytes(int64_t n_tokens, int kv_heads, int64_t pt_cols,
                                                   int page_size) {
  using namespace pkv;
  if (n_tokens < 0 || n_tokens > PKV_MAX_SPARSE_TOKENS || kv_heads < 1 || kv_heads > 65535 ||
      pt_cols < 1 || pt_cols > (int64_t{1} << 30) || page_size < 1)
    return 0;
  const int64_t cells = n_tokens * kv_heads * div_ceil(pt_cols, page_size);
  return static_cast<size_t>(round16(n_tokens * 8) + round16(n_tokens * kv_heads * 8) + 8 * cells);
}

extern "C" int pkv_select_pages(const pkv_kv_cache* cache, const void* bounds, const void* q,
                                int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                                pkv_dtype dt, int64_t n_tokens, const int32_t* cached_len,
                                const int32_t* device_len, const int32_t* table_idx, int B,
                                int max_q_len, const int32_t* page_table, int64_t pt_rows,
                                int64_t pt_cols, int budget, int sink, int recent, int32_t* pages,
                                int32_t* out_lengths, int32_t* status, void* workspace,
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
  if (n_tokens < 0 || n_tokens > PKV_MAX_SPARSE_TOKENS)
    return fail(PKV_EINVAL, "n_tokens=%lld outside [0, %d]", (long long)n_tokens,
                PKV_MAX_SPARSE_TOKENS);
  if (max_q_len < 1) return fail(PKV_EINVAL, "max_q_len=%d < 1", max_q_len);
  if (budget < 1 || budget > 65536) return fail(PKV_EINVAL, "budget=%d outside [1, 65536]", budget);
  if (sink < 0 || recent < 1 || sink > budget - recent)
    return fail(PKV_EINVAL, "sink=%d and recent=%d: need sink >= 0, recent >= 1 and at most "
                "budget=%d in all", sink, recent, budget);
  if (B == 0 || n_tokens == 0) return ok();
  if ((bad = rows_error("q", q, q_token_stride, q_head_stride)) != PKV_OK) return bad;
  if (bounds == nullptr || cached_len == nullptr || device_len == nullptr || table_idx == nullptr ||
      page_table == nullptr || pages == nullptr || out_lengths == nullptr)
    return fail(PKV_EINVAL, "NULL pointer argument");
  if (!aligned16(bounds)) return fail(PKV_EINVAL, "bounds are not 16-byte aligned");
  if (cache->num_pages * cache->kv_heads > int64_t{kNoRow} / (cache->head_dim / 16))
    return fail(PKV_EINVAL, "bounds of %lld pages of %d heads are too large",
                (long long)cache->num_pages, cache->kv_heads);
  if (pt_rows < 1 || pt_cols < 1 || pt_rows > INT32_MAX || pt_cols > (int64_t{1} << 30))
    return fail(PKV_EINVAL, "page table shape [%lld, %lld]: need rows in [1, 2^31), columns in "
                "[1, 2^30]", (long long)pt_rows, (long long)pt_cols);
  const size_t need = pkv_select_pages_workspace_bytes(n_tokens, cache->kv_heads, pt_cols,
                                                       cache->page_size);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PKV_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned16(workspace)) return fail(PKV_EINVAL, "workspace is not 16-byte aligned");
  SelectParams P = {};
  AttendParams& A = P.a;
  A.c = *cache;
  A.page_div = Divider::by(static_cast<uint32_t>(cache->page_size));
  A.q = static_cast<const uint16_t*>(q);
  A.q_ts = q_token_stride, A.q_hs = q_head_stride;
  A.cached_len = cached_len;
  A.device_len = device_len;
  A.table_idx = table_idx;
  A.page_table = page_table;
  A.status = status;
  A.n_tokens = n_tokens;
  A.pt_rows = pt_rows, A.pt_cols = pt_cols;
  A.B = B;
  A.max_q_len = static_cast<int>(std::min<int64_t>(max_q_len, n_tokens));
  A.q_heads = q_heads;
  A.group = q_heads / cache->kv_heads;
  P.bounds = static_cast<const uint8_t*>(bounds);
  P.pages = pages;
  P.lengths = out_lengths;
  P.most = static_cast<int>(div_ceil(pt_cols, cache->page_size));
  uint8_t* at = static_cast<uint8_t*>(workspace);
  P.where = reinterpret_cast<int2*>(at);
  at += round16(n_tokens * 8);
  P.sums = reinterpret_cast<float2*>(at);
  at += round16(n_tokens * cache->kv_heads * 8);
  P.score = reinterpret_cast<float2*>(at);
  P.budget = budget, P.sink = sink, P.recent = recent;
  if (n_tokens * cache->kv_heads > INT32_MAX)
    return fail(PKV_EINVAL, "%lld tokens of %d heads are too many", (long long)n_tokens,
                cache->kv_heads);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == PKV_BF16 ? launch<__nv_bfloat16>(P, s) : launch<__half>(P, s);
  if (e != cudaSuccess) return cuda_fail(e, "page selection launch");
  return ok();
}
