// pkv_adjust_logits: penalties for repeated tokens, biases and grammar masks.
//
// A CTA owns one slice of one row's vocabulary and a shared-memory cell for
// every token of it.  It scans the row's whole history (a few KB to some tens
// of KB, from L2 after the row's first slice) and counts the tokens that fall
// in its slice: a prompt token sets the cell's "seen" bit, a made one adds 1.
// Integer sums, so the order of the atomics leaves no trace.  Then:
//   * out of place: the slice streams through once, kUnroll 16-byte loads a
//     thread in flight; an element whose cell is zero and whose mask bit is
//     set is copied, and logits under a zero mask are not even read.  The few
//     biased tokens are computed again from the logits and overwritten;
//   * in place: only tokens with a cell or a bias are read and written (the
//     thread that takes a cell's content applies it), then masked places are
//     filled with -inf.
// The row's biases that fall in the slice are gathered in list order; the
// thread of a token's first bias adds all of them, so the sum has one order.
//
// Cells are 16 bits where the row's made tokens number at most 16383 (a
// 14-bit count), else 32 bits, in two passes of half a slice.  (32 bits for all:
// the two sizes below take 55 and 517 us, 4 x 32000 fp32 6.2 against 4.6.)
//
// Bound: bytes (out of place: one read and one write of the logits).  For 256 x
// 151936 bf16 (histories to 2512 tokens, 64 biases a row, a third of the rows
// masked) 44 us, 3.7 TB/s; for 1024 x 256000 bf16 (histories to 36863 tokens,
// 300 biases a row) 428 us, 2.7 TB/s, of which the histories take half: every
// slice of a row reads them all (150 us, the latency of those reads more than
// their count), atomics on the frequent tokens 40, penalties in the stream 60.
// Measured against this for the second size: two CTAs an SM with 96 KB of cells
// 478; the slices of a row as a cluster that counts each token once, in the
// owner's cells, 748; the history in a hash table by a kernel of its own and
// the named tokens written one by one 977 (they touch most of the row's
// sectors again).

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "device_attr.h"
#include "device_common.cuh"
#include "kv_cache.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 512;
constexpr int kUnroll = 4;
constexpr int kCellBytes = 64 * 1024;  // shared memory of the cells: three CTAs an SM
constexpr int kPadBytes = 32;          // and what aligns them
constexpr int kMaxCount16 = 16383;
constexpr int kBiasCap = kThreads;     // gathered biases of a slice

struct AdjustParams {
  const void* logits;
  void* out;
  int64_t in_stride, out_stride;
  const int32_t* token_pool;
  const int32_t* table_idx;
  const int32_t* prompt_len;
  const int32_t* device_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_ptr;
  const int32_t* bias_ids;
  const float* bias_values;
  const uint32_t* mask;
  int32_t* status;
  int64_t pool_rows, pool_cols, n_bias, mask_stride;
  int B, V, slice, slices;
};

template <int BITS> struct CellOf;
template <> struct CellOf<16> {
  static constexpr uint32_t kSeen = 0x8000u, kCount = 0x3fffu;
};
template <> struct CellOf<32> {
  static constexpr uint32_t kSeen = 0x80000000u, kCount = 0x3fffffffu;
};

template <int BITS>
__device__ __forceinline__ void cell_add(uint32_t* cells, int i, uint32_t x) {
  if (BITS == 32) atomicAdd(cells + i, x);
  else atomicAdd(cells + (i >> 1), x << ((i & 1) * 16));
}
template <int BITS>
__device__ __forceinline__ void cell_or(uint32_t* cells, int i, uint32_t x) {
  if (BITS == 32) atomicOr(cells + i, x);
  else atomicOr(cells + (i >> 1), x << ((i & 1) * 16));
}
template <int BITS>
__device__ __forceinline__ uint32_t cell_get(const uint32_t* cells, int i) {
  return BITS == 32 ? cells[i] : reinterpret_cast<const uint16_t*>(cells)[i];
}
// Takes the cell's content: one caller gets it, the others zero.
template <int BITS>
__device__ __forceinline__ uint32_t cell_take(uint32_t* cells, int i) {
  if (BITS == 32) return atomicExch(cells + i, 0u);
  const int sh = (i & 1) * 16;
  return (atomicAnd(cells + (i >> 1), ~(0xffffu << sh)) >> sh) & 0xffffu;
}

// One row as its CTAs see it.
struct Row {
  float rep, inv, pres, freq;  // inv = 1 / rep
  int len, prompt;
  const int32_t* hist;
  int bias_begin, bias_end;
  const uint32_t* mask;
};

template <int BITS>
__device__ __forceinline__ float penalise(const Row& r, float x, uint32_t cell) {
  // A product with the reciprocal: both are rounded to 32 bits, so it is within
  // 1.5 units in the last place of the quotient for repetitions of 2^-126 to
  // 2^126 (a division for each element of
  // the stream costs 20 times the instructions).  Without branches: the choice
  // at the end leaves an unnamed token as it is, whatever the penalties hold.
  const float count = static_cast<float>(cell & CellOf<BITS>::kCount);
  float y = x * (x > 0.0f ? r.inv : r.rep);
  y = count > 0.0f ? y - r.freq * count - r.pres : y;
  return cell != 0u ? y : x;
}

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ bool allowed(const Row& r, int v) {
  return r.mask == nullptr || ((r.mask[v >> 5] >> (v & 31)) & 1u) != 0u;
}

// -inf in every element of a 16-byte vector.
template <typename T> __device__ __forceinline__ uint32_t minus_inf_word();
template <> __device__ __forceinline__ uint32_t minus_inf_word<float>() { return 0xff800000u; }
template <> __device__ __forceinline__ uint32_t minus_inf_word<__nv_bfloat16>() { return 0xff80ff80u; }

// How the logits are gone over: in place; out of place with every row on a
// 16-byte boundary; or anywhere.  (With rows anywhere the second's code would do,
// but 256 x 151936 take 44 us with it instead of 42, 1024 x 256000 446 instead of
// 420; 404 x 115753 fp32 take 71 us, and 146 element by element.)
enum class Way { kInPlace, kAligned, kAnywhere };

// The tokens [v0, v1) of one row.
template <typename T, int BITS, Way WAY>
__device__ void adjust_range(const AdjustParams& P, const Row& r, const T* in, T* out, int v0,
                             int v1, uint32_t* cells, int* s_id, float* s_val, int* s_count, int bad) {
  using C = CellOf<BITS>;
  const int tid = threadIdx.x, lane = tid & 31;
  const int nv = v1 - v0;
  // Vectors begin `head` tokens in, where the row reaches a 16-byte boundary (on
  // both sides, or there are none).  Cells lie `pad` further on, so
  // that a vector's cells are aligned too.
  constexpr int kVec = 16 / sizeof(T);
  constexpr bool INPLACE = WAY == Way::kInPlace;
  int head = 0, pad = 0, vecs = nv / kVec;
  if (WAY == Way::kAnywhere) {
    vecs = 0;
    const uintptr_t a = reinterpret_cast<uintptr_t>(in + v0);
    if (((a ^ reinterpret_cast<uintptr_t>(out + v0)) & 15) == 0) {
      head = static_cast<int>((16 - (a & 15)) & 15) / static_cast<int>(sizeof(T));
      pad = head == 0 ? 0 : kVec - head;
      head = min(head, nv);
      vecs = (nv - head) / kVec;
    }
  }
  const bool counted = r.len > 0;
  const bool biased = r.bias_end > r.bias_begin;
  int listed = 0;  // biases of the slice

  // ---- cells and the slice's biases
  // The first round of the row's biases sets out too.
  int id = -1;
  float val = 0.0f;
  if (r.bias_begin + tid < r.bias_end)
    id = P.bias_ids[r.bias_begin + tid], val = P.bias_values[r.bias_begin + tid];
  if (counted) {
    const int words = ((nv + pad) * (BITS / 8) + 15) / 16;
    for (int i = tid; i < words; i += kThreads)
      reinterpret_cast<uint4*>(cells)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    auto one = [&](int tok, bool made) {
      const uint32_t i = static_cast<uint32_t>(tok - v0);
      if (i >= static_cast<uint32_t>(nv)) return;
      if (made) cell_add<BITS>(cells, i + pad, 1u);
      else cell_or<BITS>(cells, i + pad, C::kSeen);
    };
    auto note = [&](int tok, int at) { one(tok, at >= r.prompt); };
    // 16-byte loads from the first aligned entry on; nearly every four lie on
    // one side of the prompt's end.
    const int head = min(
        r.len, static_cast<int>((4 - ((reinterpret_cast<uintptr_t>(r.hist) >> 2) & 3)) & 3));
    const int quads = (r.len - head) >> 2;
    if (tid < head) note(r.hist[tid], tid);
    const int4* h4 = reinterpret_cast<const int4*>(r.hist + head);
#pragma unroll 2
    for (int i = tid; i < quads; i += kThreads) {
      const int4 t = h4[i];
      const int at = head + 4 * i;
      if (at >= r.prompt) {
        one(t.x, true), one(t.y, true), one(t.z, true), one(t.w, true);
      } else if (at + 3 < r.prompt) {
        one(t.x, false), one(t.y, false), one(t.z, false), one(t.w, false);
      } else {
        note(t.x, at), note(t.y, at + 1), note(t.z, at + 2), note(t.w, at + 3);
      }
    }
    const int rest = head + 4 * quads + tid;
    if (rest < r.len) note(r.hist[rest], rest);
  }
  if (biased) {
    // The slice's biases in list order, a thread an entry and round.
    int n = 0;
    for (int e0 = r.bias_begin; e0 < r.bias_end; e0 += kThreads) {
      const int e = e0 + tid;
      if (e0 != r.bias_begin) {
        id = -1;
        if (e < r.bias_end) id = P.bias_ids[e], val = P.bias_values[e];
      }
      if (e < r.bias_end && (id < 0 || id >= P.V)) bad |= PKV_ST_COL_OOB;
      const bool mine = id >= v0 && id < v1;
      const unsigned m = __ballot_sync(kFull, mine);
      if (e0 != r.bias_begin) __syncthreads();  // the counts have been read
      if (lane == 0) s_count[tid >> 5] = __popc(m);
      __syncthreads();
      int at = n + __popc(m & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        const int c = s_count[w];
        if (w < (tid >> 5)) at += c;
        n += c;
      }
      if (mine && at < kBiasCap) s_id[at] = id, s_val[at] = val;
    }
    listed = n;
    if (tid < 4 && n + tid < kBiasCap) s_id[n + tid] = -1;  // the last four's rest
  }
  __syncthreads();

  if (v0 == 0 && bad != 0 && P.status != nullptr) atomicOr(P.status, bad);

  // The thread of a biased token's first bias has the token, and its logit with
  // all its biases: `mine` is the token or -1.  A slice's gathered list has at
  // most an entry a thread; a longer one is not gathered, and searched in place.
  auto penalty = [&](int v, float x) {
    if (!counted) return x;
    return penalise<BITS>(
        r, x, INPLACE ? cell_take<BITS>(cells, v - v0) : cell_get<BITS>(cells, v - v0 + pad));
  };
  const T* src = INPLACE ? out : in;
  int mine = -1;
  float mine_x = 0.0f;
  if (listed <= kBiasCap && tid < listed) {
    mine = s_id[tid];
    mine_x = load_one(src + mine);
    int before = 0, same = 0;
    for (int k = 0; k < listed; k += 4) {
      const int4 o = *reinterpret_cast<const int4*>(s_id + k);
      const int m = (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
      same += m;
      if (k + 3 < tid) before += m;
    }
    for (int k = tid & ~3; k < tid; ++k) before += s_id[k] == mine;
    if (before != 0) {
      mine = -1;
    } else {
      mine_x = penalty(mine, mine_x);
      if (same == 1) mine_x += s_val[tid];
      else
        for (int k = tid; k < listed; ++k)
          if (s_id[k] == mine) mine_x += s_val[k];
      if (!allowed(r, mine)) mine = -1;
    }
  }
  auto store_biased = [&] {
    if (mine >= 0) store_one(out + mine, mine_x);
    if (listed <= kBiasCap) return;
    for (int e = r.bias_begin + tid; e < r.bias_end; e += kThreads) {
      const int v = P.bias_ids[e];
      if (v < v0 || v >= v1) continue;
      bool first = true;
      for (int k = r.bias_begin; k < e && first; ++k) first = P.bias_ids[k] != v;
      if (!first) continue;
      float x = penalty(v, load_one(src + v));
      for (int k = e; k < r.bias_end; ++k)
        if (P.bias_ids[k] == v) x += P.bias_values[k];
      if (allowed(r, v)) store_one(out + v, x);
    }
  };

  if (INPLACE) {
    if (biased) {
      store_biased();
      __syncthreads();
    }
    for (int i = tid; i < r.len; i += kThreads) {
      const int tok = r.hist[i];
      const uint32_t k = static_cast<uint32_t>(tok - v0);
      if (k >= static_cast<uint32_t>(nv) || cell_get<BITS>(cells, k) == 0u) continue;
      const uint32_t c = cell_take<BITS>(cells, k);
      if (c != 0u) store_one(out + tok, penalise<BITS>(r, load_one(out + tok), c));
    }
    if (r.mask != nullptr) {
      __syncthreads();  // a masked place is -inf whatever was written there
      const int w0 = v0 >> 5, w1 = (v1 + 31) >> 5;
      for (int w = w0 + (tid >> 5); w < w1; w += kThreads / 32) {
        const uint32_t bits = r.mask[w];
        const int v = w * 32 + lane;
        if (v < v1 && ((bits >> lane) & 1u) == 0u) store_one(out + v, -INFINITY);
      }
    }
    return;
  }

  // ---- out of place: the slice once through
  constexpr uint32_t kAll = (1u << kVec) - 1u;
  const int first = v0 + head;
  const bool split = WAY == Way::kAnywhere && r.mask != nullptr;  // vectors may span two mask words
  const uint32_t* own = cells + (head + pad) * BITS / 32;  // the first vector's cells
  for (int i0 = tid; i0 < vecs; i0 += kThreads * kUnroll) {
    uint4 raw[kUnroll];
    uint32_t bits[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads, v = first + i * kVec;
      bits[u] = kAll;
      if (i < vecs && r.mask != nullptr) bits[u] = r.mask[v >> 5] >> (v & 31);
    }
    if (split) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kThreads, v = first + i * kVec;
        if (i < vecs && (v & 31) > 32 - kVec) bits[u] |= r.mask[(v >> 5) + 1] << (32 - (v & 31));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      bits[u] &= kAll;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < vecs && bits[u] != 0u) raw[u] = ld_stream_v4(in + first + i * kVec);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= vecs) break;
      constexpr int kWords = kVec * BITS / 32;  // of cells
      uint32_t cw[kWords];
      uint32_t any = 0u;
#pragma unroll
      for (int k = 0; k < kWords; k += kWords < 4 ? 2 : 4) {
        if (kWords < 4) {
          uint2 c = make_uint2(0u, 0u);
          if (counted) c = *reinterpret_cast<const uint2*>(own + i * kWords);
          cw[k] = c.x, cw[k + 1] = c.y;
        } else {
          uint4 c = make_uint4(0u, 0u, 0u, 0u);
          if (counted) c = *reinterpret_cast<const uint4*>(own + i * kWords + k);
          cw[k] = c.x, cw[k + 1] = c.y, cw[k + 2] = c.z, cw[k + 3] = c.w;
        }
      }
#pragma unroll
      for (int k = 0; k < kWords; ++k) any |= cw[k];
      uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      if (any != 0u) {
        auto cell = [&](int k) {
          return BITS == 32 ? cw[k] : (cw[k >> 1] >> ((k & 1) * 16)) & 0xffffu;
        };
        if (sizeof(T) == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = __float_as_uint(penalise<BITS>(r, __uint_as_float(w[k]), cell(k)));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = cell(2 * k & (kVec - 1)), hi = cell((2 * k + 1) & (kVec - 1));
            if ((lo | hi) == 0u) continue;
            const float x = penalise<BITS>(r, __uint_as_float(w[k] << 16), lo);
            const float y = penalise<BITS>(r, __uint_as_float(w[k] & 0xffff0000u), hi);
            const uint32_t z = __bfloat16_as_ushort(__float2bfloat16_rn(x)) |
                               static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(y))) << 16;
            // (Rounding would change a NaN's bits, and the other one may be no one's.)
            const uint32_t keep = (lo != 0u ? 0u : 0xffffu) | (hi != 0u ? 0u : 0xffff0000u);
            w[k] = (z & ~keep) | (w[k] & keep);
          }
        }
      }
      if (bits[u] != kAll) {
        const uint32_t inf = minus_inf_word<T>();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t hide;
          if (sizeof(T) == 4) {
            hide = (bits[u] >> k) & 1u ? 0u : 0xffffffffu;
          } else {
            hide = ((bits[u] >> (2 * k)) & 1u ? 0u : 0xffffu) |
                   ((bits[u] >> (2 * k + 1)) & 1u ? 0u : 0xffff0000u);
          }
          w[k] = (w[k] & ~hide) | (inf & hide);
        }
      }
      *reinterpret_cast<uint4*>(out + first + i * kVec) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  for (int e = tid; e < nv - vecs * kVec; e += kThreads) {
    const int i = e < head ? e : e + vecs * kVec, v = v0 + i;
    T x = in[v];
    const uint32_t c = counted ? cell_get<BITS>(cells, i + pad) : 0u;
    if (!allowed(r, v)) store_one(&x, -INFINITY);
    else if (c != 0u) store_one(&x, penalise<BITS>(r, load_one(&x), c));
    out[v] = x;
  }
  if (biased) {
    __syncthreads();  // biased tokens are written over
    store_biased();
  }
}

template <typename T, Way WAY>
__global__ void __launch_bounds__(kThreads, 3) adjust_kernel(const AdjustParams P) {
  extern __shared__ __align__(16) uint32_t cells[];
  __shared__ __align__(16) int s_id[kBiasCap];
  __shared__ float s_val[kBiasCap];
  __shared__ int s_count[kThreads / 32];
  const int b = blockIdx.x / P.slices, sl = blockIdx.x - b * P.slices;
  const int v0 = sl * P.slice, v1 = min(P.V, v0 + P.slice);
  const T* in = static_cast<const T*>(P.logits) + b * P.in_stride;
  T* out = static_cast<T*>(P.out) + b * P.out_stride;

  Row r;
  r.mask = P.mask != nullptr ? P.mask + b * P.mask_stride : nullptr;
  r.rep = P.repetition != nullptr ? P.repetition[b] : 1.0f;
  r.inv = 1.0f / r.rep;
  r.pres = P.presence != nullptr ? P.presence[b] : 0.0f;
  r.freq = P.frequency != nullptr ? P.frequency[b] : 0.0f;
  r.len = r.prompt = 0;
  r.hist = nullptr;
  int bad = 0;
  if (P.token_pool != nullptr) {
    const int64_t t = P.table_idx[b];
    const int len = P.device_len[b];
    if (t < 0 || t >= P.pool_rows) {
      bad |= PKV_ST_ROW_OOB;
    } else if (len < 0 || len > P.pool_cols) {
      bad |= PKV_ST_COL_OOB;
    } else {
      r.len = len;
      r.hist = P.token_pool + t * P.pool_cols;
      r.prompt = max(0, min(len, P.prompt_len[b]));
    }
  }
  r.bias_begin = r.bias_end = 0;
  if (P.bias_ptr != nullptr) {
    const int e0 = P.bias_ptr[b], e1 = P.bias_ptr[b + 1];
    if (e0 < 0 || e1 < e0 || e1 > P.n_bias) bad |= PKV_ST_COL_OOB;
    else r.bias_begin = e0, r.bias_end = e1;
  }
  if (r.len - r.prompt <= kMaxCount16) {
    adjust_range<T, 16, WAY>(P, r, in, out, v0, v1, cells, s_id, s_val, s_count, bad);
  } else {
    const int mid = min(v1, v0 + P.slice / 2);
    adjust_range<T, 32, WAY>(P, r, in, out, v0, mid, cells, s_id, s_val, s_count, bad);
    __syncthreads();
    if (mid < v1)
      adjust_range<T, 32, WAY>(P, r, in, out, mid, v1, cells, s_id, s_val, s_count, bad);
  }
}

template <typename T, Way WAY>
cudaError_t launch(const AdjustParams& P, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0ull};
  const auto kernel = adjust_kernel<T, WAY>;
  const cudaError_t e = set_smem_limit_once(done, kernel, kCellBytes + kPadBytes);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(P.B) * P.slices, kThreads, P.slice * 2 + kPadBytes, s>>>(P);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AdjustParams& P, cudaStream_t s) {
  if (P.logits == P.out) return launch<T, Way::kInPlace>(P, s);
  constexpr int kVec = 16 / sizeof(T);
  const bool aligned = aligned16(P.logits) && aligned16(P.out) && P.in_stride % kVec == 0 &&
                       P.out_stride % kVec == 0;
  return aligned ? launch<T, Way::kAligned>(P, s) : launch<T, Way::kAnywhere>(P, s);
}

// Whether a row of x shares bytes with a row of y (rows of one buffer may take
// turns).  Each side's rows ascend without overlapping one another.
bool rows_overlap(const void* x, int64_t x_stride, const void* y, int64_t y_stride, int B, int V,
                  int elt) {
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  const uintptr_t size = static_cast<uintptr_t>(V) * elt;
  const uintptr_t xs = x_stride * elt, ys = y_stride * elt;
  if (x0 + (B - 1) * xs + size <= y0 || y0 + (B - 1) * ys + size <= x0) return false;
  for (int i = 0, j = 0; i < B && j < B;) {
    const uintptr_t a = x0 + i * xs, b = y0 + j * ys;
    if (a + size <= b) ++i;
    else if (b + size <= a) ++j;
    else return true;
  }
  return false;
}

}  // namespace

}  // namespace pkv

extern "C" int pkv_adjust_logits(const void* logits, int64_t row_stride, pkv_dtype dt, int B, int V,
                                 void* out, int64_t out_stride, const int32_t* token_pool,
                                 int64_t pool_rows, int64_t pool_cols, const int32_t* table_idx,
                                 const int32_t* prompt_len, const int32_t* device_len,
                                 const float* repetition, const float* presence,
                                 const float* frequency, const int32_t* bias_ptr,
                                 const int32_t* bias_ids, const float* bias_values, int64_t n_bias,
                                 const int32_t* mask, int64_t mask_stride, int32_t* status,
                                 pkv_stream_t stream) {
  using namespace pkv;
  if (dt != PKV_FP32 && dt != PKV_BF16)
    return fail(PKV_EINVAL, "dtype %d is not fp32 or bf16", static_cast<int>(dt));
  if (B < 0 || B > 65535) return fail(PKV_EINVAL, "B=%d outside [0, 65535]", B);
  if (V < 1) return fail(PKV_EINVAL, "V=%d < 1", V);
  if (row_stride < V || out_stride < V)
    return fail(PKV_EINVAL, "row strides %lld and %lld: need at least V=%d", (long long)row_stride,
                (long long)out_stride, V);
  const int max_v = dt == PKV_BF16 ? PKV_MAX_VOCAB_BF16 : PKV_MAX_VOCAB_FP32;
  if (V > max_v) return fail(PKV_EUNSUPPORTED, "V=%d above the maximum %d", V, max_v);
  if (B == 0) return ok();
  if (logits == nullptr) return fail(PKV_EINVAL, "logits is NULL");
  if (out == nullptr) return fail(PKV_EINVAL, "out is NULL");
  if (logits == out && row_stride != out_stride)
    return fail(PKV_EINVAL, "in place the row strides have to be the same");
  if (logits != out && rows_overlap(logits, row_stride, out, out_stride, B, V, dt == PKV_BF16 ? 2 : 4))
    return fail(PKV_EINVAL, "logits and out overlap without being the same");
  if (token_pool != nullptr || table_idx != nullptr || prompt_len != nullptr || device_len != nullptr) {
    if (token_pool == nullptr || table_idx == nullptr || prompt_len == nullptr || device_len == nullptr)
      return fail(PKV_EINVAL, "token_pool, table_idx, prompt_len and device_len go together");
    if (pool_rows < 1 || pool_cols < 1 || pool_cols >= (int64_t{1} << 30))
      return fail(PKV_EINVAL, "token pool shape [%lld, %lld]", (long long)pool_rows,
                  (long long)pool_cols);
  }
  if (bias_ptr != nullptr || bias_ids != nullptr || bias_values != nullptr) {
    if (bias_ptr == nullptr || (n_bias > 0 && (bias_ids == nullptr || bias_values == nullptr)))
      return fail(PKV_EINVAL, "bias_ptr, bias_ids and bias_values go together");
    // (The kernel's 32-bit indexes go up to kThreads past a list's end.)
    if (n_bias < 0 || n_bias > (int64_t{1} << 30))
      return fail(PKV_EINVAL, "n_bias=%lld outside [0, 2^30]", (long long)n_bias);
  }
  if (mask != nullptr && mask_stride < (V + 31) / 32)
    return fail(PKV_EINVAL, "mask_stride=%lld below ceil(V / 32)=%d", (long long)mask_stride,
                (V + 31) / 32);
  AdjustParams P;
  P.logits = logits;
  P.out = out;
  P.in_stride = row_stride, P.out_stride = out_stride;
  P.token_pool = token_pool;
  P.table_idx = table_idx;
  P.prompt_len = prompt_len;
  P.device_len = device_len;
  P.repetition = repetition;
  P.presence = presence;
  P.frequency = frequency;
  P.bias_ptr = bias_ptr;
  P.bias_ids = bias_ids;
  P.bias_values = bias_values;
  P.mask = reinterpret_cast<const uint32_t*>(mask);
  P.status = status;
  P.pool_rows = pool_rows, P.pool_cols = pool_cols;
  P.n_bias = n_bias;
  P.mask_stride = mask_stride;
  P.B = B, P.V = V;
  // Slices: as few as the cells allow, but enough for two CTAs an SM (otherwise
  // 4 x 32000 fp32 takes 7.9 us instead of 4.6, 16 x 151936 bf16 8.7 of 6.9); a
  // multiple of 2048 tokens, so that no mask word or vector straddles two
  // (or two halves of one).
  const int cap = kCellBytes / 2;
  const int64_t want = std::max<int64_t>(div_ceil(V, cap), div_ceil(2 * num_sms(), B));
  P.slice = static_cast<int>(
      std::min<int64_t>(cap / 2048 * 2048, div_ceil(div_ceil(V, want), 2048) * 2048));
  P.slices = static_cast<int>(div_ceil(V, P.slice));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dt == PKV_BF16 ? launch_type<__nv_bfloat16>(P, s) : launch_type<float>(P, s);
  if (e != cudaSuccess) return cuda_fail(e, "adjust launch");
  return ok();
}
