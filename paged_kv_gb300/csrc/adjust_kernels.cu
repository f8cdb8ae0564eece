// pkv_adjust_logits: penalties for repeated tokens, biases and grammar masks.
//
// A CTA owns one slice of one row's vocabulary and a shared-memory cell for
// every token of it.  It scans the row's whole history (a few KB to some tens
// of KB, from L2 after the first slice) and counts the tokens that fall in
// its slice: a prompt token sets the cell's "seen" bit, a made one adds 1; a
// bias sets its bit.  Integer sums, so the order of the atomics leaves no
// trace.  Then:
//   * out of place: the slice streams through once, 16 bytes a thread; an
//     element whose cell is zero and whose mask bit is set is copied;
//   * in place: only tokens with a cell are read and written (the first
//     thread to take a cell's content applies it), then masked places are
//     filled with -inf.
// Biases are added by searching the row's list for the element's token, in
// list order: only elements with a bias do, and the sum has one order.
//
// Bound: bytes (out of place: one read and one write of the logits).  Cells
// are 16 bits where a count fits 14 bits (token pools of up to 16383
// columns), 32 bits otherwise.

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
constexpr int kCellBytes = 96 * 1024;  // shared memory of the cells: two CTAs an SM
constexpr int kMaxCount16 = 16383;

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
  bool vec;       // 16-byte accesses are aligned on both sides
};

template <int BITS> struct CellOf;
template <> struct CellOf<16> {
  static constexpr uint32_t kSeen = 0x8000u, kBias = 0x4000u, kCount = 0x3fffu;
};
template <> struct CellOf<32> {
  static constexpr uint32_t kSeen = 0x80000000u, kBias = 0x40000000u, kCount = 0x3fffffffu;
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

struct Row {
  float rep, pres, freq;
  int bias_begin, bias_end;
};

template <int BITS>
__device__ __forceinline__ float adjust(const AdjustParams& P, const Row& r, float x, uint32_t cell,
                                        int v) {
  using C = CellOf<BITS>;
  const uint32_t count = cell & C::kCount;
  if ((cell & ~C::kBias) != 0u) x = x > 0.0f ? x / r.rep : x * r.rep;
  if (count != 0u) x = x - r.freq * static_cast<float>(count) - r.pres;
  if ((cell & C::kBias) != 0u) {
    for (int e = r.bias_begin; e < r.bias_end; ++e)
      if (P.bias_ids[e] == v) x += P.bias_values[e];
  }
  return x;
}

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, int BITS, bool INPLACE>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const AdjustParams P) {
  using C = CellOf<BITS>;
  extern __shared__ __align__(16) uint32_t cells[];
  const int tid = threadIdx.x;
  const int b = blockIdx.x / P.slices, sl = blockIdx.x - b * P.slices;
  const int v0 = sl * P.slice, v1 = min(P.V, v0 + P.slice), nv = v1 - v0;
  const T* in = static_cast<const T*>(P.logits) + b * P.in_stride;
  T* out = static_cast<T*>(P.out) + b * P.out_stride;
  const uint32_t* mask = P.mask != nullptr ? P.mask + b * P.mask_stride : nullptr;

  Row r;
  r.rep = P.repetition != nullptr ? P.repetition[b] : 1.0f;
  r.pres = P.presence != nullptr ? P.presence[b] : 0.0f;
  r.freq = P.frequency != nullptr ? P.frequency[b] : 0.0f;
  int bad = 0;
  int len = 0, prompt = 0;
  const int32_t* hist = nullptr;
  if (P.token_pool != nullptr) {
    const int64_t t = P.table_idx[b];
    len = P.device_len[b];
    if (t < 0 || t >= P.pool_rows) {
      bad |= PKV_ST_ROW_OOB;
      len = 0;
    } else if (len < 0 || len > P.pool_cols) {
      bad |= PKV_ST_COL_OOB;
      len = 0;
    } else {
      hist = P.token_pool + t * P.pool_cols;
      prompt = max(0, min(len, P.prompt_len[b]));
    }
  }
  r.bias_begin = r.bias_end = 0;
  if (P.bias_ptr != nullptr) {
    const int e0 = P.bias_ptr[b], e1 = P.bias_ptr[b + 1];
    if (e0 < 0 || e1 < e0 || e1 > P.n_bias) bad |= PKV_ST_COL_OOB;
    else r.bias_begin = e0, r.bias_end = e1;
  }
  const bool touched = len > 0 || r.bias_end > r.bias_begin;

  // ---- cells
  if (touched) {
    const int words = (nv * (BITS / 8) + 15) / 16;
    for (int i = tid; i < words; i += kThreads)
      reinterpret_cast<uint4*>(cells)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    auto note = [&](int tok, int at) {
      const int i = tok - v0;
      if (i < 0 || i >= nv) return;
      if (at >= prompt) cell_add<BITS>(cells, i, 1u);
      else cell_or<BITS>(cells, i, C::kSeen);
    };
    int head = 0;
    if (len > 0) {
      // 16-byte loads from the first aligned entry on.
      head = min(len, static_cast<int>((4 - ((reinterpret_cast<uintptr_t>(hist) >> 2) & 3)) & 3));
      const int quads = (len - head) >> 2;
      if (tid < head) note(hist[tid], tid);
      const int4* h4 = reinterpret_cast<const int4*>(hist + head);
#pragma unroll 4
      for (int i = tid; i < quads; i += kThreads) {
        const int4 t = h4[i];
        const int at = head + 4 * i;
        note(t.x, at), note(t.y, at + 1), note(t.z, at + 2), note(t.w, at + 3);
      }
      const int rest = head + 4 * quads + tid;
      if (rest < len) note(hist[rest], rest);
    }
    for (int e = r.bias_begin + tid; e < r.bias_end; e += kThreads) {
      const int v = P.bias_ids[e];
      if (v < 0 || v >= P.V) bad |= PKV_ST_COL_OOB;
      else if (v >= v0 && v < v1) cell_or<BITS>(cells, v - v0, C::kBias);
    }
    __syncthreads();
  }
  if (sl == 0 && bad != 0 && P.status != nullptr) atomicOr(P.status, bad);

  if (INPLACE) {
    auto apply = [&](int tok) {
      const int i = tok - v0;
      if (i < 0 || i >= nv || cell_get<BITS>(cells, i) == 0u) return;
      const uint32_t c = cell_take<BITS>(cells, i);
      if (c != 0u) store_one(out + tok, adjust<BITS>(P, r, load_one(out + tok), c, tok));
    };
    for (int i = tid; i < len; i += kThreads) apply(hist[i]);
    for (int e = r.bias_begin + tid; e < r.bias_end; e += kThreads) apply(P.bias_ids[e]);
    if (mask != nullptr) {
      __syncthreads();  // a masked place is -inf whatever was written there
      const int w0 = v0 >> 5, w1 = (v1 + 31) >> 5;
      for (int w = w0 + (tid >> 5); w < w1; w += kThreads / 32) {
        const uint32_t bits = mask[w];
        const int v = w * 32 + (tid & 31);
        if (v < v1 && ((bits >> (tid & 31)) & 1u) == 0u) store_one(out + v, -INFINITY);
      }
    }
    return;
  }

  // ---- out of place: the slice once through
  constexpr int kVec = 16 / sizeof(T);
  if (P.vec) {
    const int vecs = (nv + kVec - 1) / kVec;
    for (int i = tid; i < vecs; i += kThreads) {
      const int at = i * kVec, v = v0 + at;
      const uint32_t bits = mask != nullptr ? mask[v >> 5] >> (v & 31) : 0xffffffffu;
      const bool full = at + kVec <= nv;
      uint32_t any = 0u;
      if (touched) {
        constexpr int kWords = kVec * BITS / 32;
#pragma unroll
        for (int k = 0; k < kWords; ++k) any |= cells[at * BITS / 32 + k];
      }
      constexpr uint32_t kAll = (1u << kVec) - 1u;
      if (full && any == 0u && (bits & kAll) == kAll) {
        *reinterpret_cast<uint4*>(out + v) = ld_stream_v4(in + v);
        continue;
      }
      __align__(16) T x[kVec];
      if (full) {
        *reinterpret_cast<uint4*>(x) = ld_stream_v4(in + v);
      } else {
        for (int k = 0; k < nv - at; ++k) x[k] = in[v + k];
      }
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const uint32_t c = touched ? cell_get<BITS>(cells, at + k) : 0u;
        if (((bits >> k) & 1u) == 0u) store_one(x + k, -INFINITY);
        else if (c != 0u) store_one(x + k, adjust<BITS>(P, r, load_one(x + k), c, v + k));
      }
      if (full) {
        *reinterpret_cast<uint4*>(out + v) = *reinterpret_cast<const uint4*>(x);
      } else {
        for (int k = 0; k < nv - at; ++k) out[v + k] = x[k];
      }
    }
  } else {
    for (int i = tid; i < nv; i += kThreads) {
      const int v = v0 + i;
      T x = in[v];
      const uint32_t c = touched ? cell_get<BITS>(cells, i) : 0u;
      if (mask != nullptr && ((mask[v >> 5] >> (v & 31)) & 1u) == 0u) store_one(&x, -INFINITY);
      else if (c != 0u) store_one(&x, adjust<BITS>(P, r, load_one(&x), c, v));
      out[v] = x;
    }
  }
}

template <typename T, int BITS, bool INPLACE>
cudaError_t launch(const AdjustParams& P, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0ull};
  const auto kernel = adjust_kernel<T, BITS, INPLACE>;
  const cudaError_t e = set_smem_limit_once(done, kernel, kCellBytes);
  if (e != cudaSuccess) return e;
  const int bytes = (P.slice * (BITS / 8) + 15) / 16 * 16;
  kernel<<<static_cast<unsigned>(P.B) * P.slices, kThreads, bytes, s>>>(P);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AdjustParams& P, int bits, cudaStream_t s) {
  const bool inplace = P.logits == P.out;
  if (bits == 16) return inplace ? launch<T, 16, true>(P, s) : launch<T, 16, false>(P, s);
  return inplace ? launch<T, 32, true>(P, s) : launch<T, 32, false>(P, s);
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
  const int elt = dt == PKV_BF16 ? 2 : 4;
  if (logits != out) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits), o = reinterpret_cast<uintptr_t>(out);
    const uintptr_t an = a + ((B - 1) * row_stride + V) * elt, on = o + ((B - 1) * out_stride + V) * elt;
    if (a < on && o < an) return fail(PKV_EINVAL, "logits and out overlap without being the same");
  }
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
    if (n_bias < 0 || n_bias > INT32_MAX)
      return fail(PKV_EINVAL, "n_bias=%lld outside [0, 2^31)", (long long)n_bias);
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
  P.vec = aligned16(logits) && aligned16(out) && (row_stride * elt) % 16 == 0 &&
          (out_stride * elt) % 16 == 0;
  const int bits = token_pool == nullptr || pool_cols <= kMaxCount16 ? 16 : 32;
  // Slices: as few as the cells allow, but enough for two CTAs an SM; a
  // multiple of 1024 tokens, so that mask words and vectors never straddle.
  const int cap = kCellBytes / (bits / 8);
  const int64_t want = std::max<int64_t>(div_ceil(V, cap), div_ceil(2 * num_sms(), B));
  P.slice = static_cast<int>(
      std::min<int64_t>(cap / 1024 * 1024, div_ceil(div_ceil(V, want), 1024) * 1024));
  P.slices = static_cast<int>(div_ceil(V, P.slice));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dt == PKV_BF16 ? launch_type<__nv_bfloat16>(P, bits, s) : launch_type<float>(P, bits, s);
  if (e != cudaSuccess) return cuda_fail(e, "adjust launch");
  return ok();
}
