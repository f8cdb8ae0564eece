// Attention of few query rows a request over the paged e4m3 cache: decoding
// (one token a request), verification of a few draft tokens.
//
// A row is one (query token, query head); the rows of one cache head share its
// keys and values.  A work unit is kStep positions for one block of up to kRows
// rows of one (request, cache head).  All units of the call, in batch order,
// are cut into contiguous ranges of equal cost, one per warp, so ragged lengths balance
// and one long request fills the machine.  A warp that holds only part of a
// block leaves its partial (m, l, O) in the workspace; partials are joined in
// warp order, first within groups of kGroup warps, then over the groups, each
// time by the last to arrive, so that no join is long and every sum has one
// order.  Warps share nothing: there is no barrier after the start.
//
// A warp streams its units through its own ring of shared memory (cp.async).
// Per unit, with keys and values as the A operand so that the few rows are the
// narrow side of the product:
//   S^T[32 x 8] = K[32 x D] Q^T,   O^T[D x 8] += V^T[D x 32] P^T
// on mma.m16n8k16 with fp16 inputs: e4m3 codes are exact in fp16, and a bf16
// query row, scaled below 2^15 by a power of two, is too, but for elements below
// 2^-31 of its largest (which keep an absolute 2^-39 of it).  Scores take the
// page's key scale in fp32.  Weights carry the page's value scale:
// p = 2^-22 2^(s - m) vs goes to fp16 (11 bits), l sums 2^(s - m) in fp32.  m is
// such that the largest p of the positions that it was taken from is 1: p keeps
// 11 bits down to 2^-14 of that and some down to 2^-24.  With that 2^-22, scales
// of 2^-64 to 2^119 put l's largest terms between 2^-97 and 2^101: neither sums
// nor terms of 2^-29 of the largest are lost.  The reference m is not the running
// maximum: it is taken from a row's first positions and moves only where the
// weights under it sum to more than 2^15.  So a unit needs no maximum over its
// lanes, and few units rescale.
//
// Bound: for up to 8 rows a cache head each cached byte is read once (2 D per
// position and head), for more once for every 8 rows.  A warp copies its next
// unit only when the present one is done (the ring's other slot is free by then,
// not before): memory waits on its 716 instructions a unit (half of them
// conversions of codes and their addresses) and they on memory, with 12 warps an
// SM to hide it.  256 requests of up to 2513 positions, 16 query and 8 cache heads
// of 128, pages of 16, bf16: 133 us, 5.2 TB/s; 16 of up to 36864, 32 and 4 heads,
// pages of 64, fp16: 74 us, 4.0 TB/s; 61 of up to 2006 under a window of 777 with
// 1 to 5 new tokens, 12 heads of 64, pages of 1: 34 us (scattered rows of 64
// bytes); one of 701: 16.4 us, of which the joins 5 and the rest the start's chain
// of loads (lengths, places, rows).
// Blocks of 16 rows, which read the cache half as often but spill and leave one
// row in two idle where there are 8: 256 requests of 16 rows 292 us against 258
// (of 32: 538 against 479), 16 long ones of 16 rows 143 against 113.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "api_common.h"
#include "attend_params.h"
#include "attend_units.cuh"
#include "device_attr.h"
#include "device_common.cuh"
#include "kv_cache.cuh"

namespace pkv {

namespace {

constexpr int kWarps = kRowWarps;
constexpr int kRows = 8;                 // of a block: the narrow side of the products
constexpr int kStep = 32;                // positions a warp takes at a time: one a lane
constexpr int kStages = 2;               // ring slots of a warp: kStages - 1 units under way
constexpr int kLook = 4;                 // units whose places are read at once (1: 149 us for the
                                         // 256 requests against 145, 8: 154)
// Cost of a block's start in units, and the least cost of a warp's range.  256
// requests decoding: 149 us without the first, 135, 132 and 133 with 1, 2 and 3;
// draft verification 35, 34, 32 and 32.  A few short requests beside a prompt
// batch: 272 us from 1 on, 257 from 2 on (fewer partials to join).
constexpr int kLead = 3, kLeast = 2;
// Warps whose partials are joined first.  With 8, 16 and 32: one request 13.3,
// 14.5 and 14.3 us, long contexts 72, 72 and 78.
constexpr int kGroup = 16;
static_assert(kStep == 32, "a lane looks up one position");
constexpr float kUnit = 0x1p-22f;        // a weight in fp16 is this times 2^(s - m) vs
constexpr float kLimit = 32768.0f;       // sum of such weights that moves m
constexpr float kLn2 = 0.693147180559945309f;

template <int DP>
struct Layout {
  static constexpr int kSlot = 2 * kStep * DP;             // K then V codes
  static constexpr int kScales = 2 * kStep * 4;            // key then value scales
  static constexpr int kRing = kStages * (kSlot + kScales);
  static constexpr int kBytes = kWarps * kRing;
  static_assert(kBytes >= kWarps * 32 * 16 + 16, "room for find_range");
};

// Floats of one partial result: O [rows, DP], then (m, l) [rows].
__host__ __device__ constexpr int partial_floats(int rows, int dp) { return rows * dp + 2 * rows; }

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// Four 8x8 matrices of 16-bit elements, each transposed.
__device__ __forceinline__ uint4 ldsm_trans(uint32_t a) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Any e4m3 NaN (0x7f or 0xff) among four codes.
__device__ __forceinline__ bool has_nan(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
}

// Joins the partials of slots slot_of(0) .. slot_of(n - 1), in this order, and
// hands each row's m, l and 4 channels of O to put(row, d, m, l, o).  One warp;
// a lane has 4 channels of kJoin rows, and 4 partials of them on their way:
// the join is at the end of everything and waits for memory alone.
template <int DP, int ROWS, typename Slot, typename Put>
__device__ __forceinline__ void join(const AttendParams& P, int rows, int n, Slot&& slot_of, Put&& put) {
  constexpr int kFloats = partial_floats(ROWS, DP), kJoin = 4;
  const int lane = threadIdx.x & 31, d = lane * 4;
  const bool live = d < P.c.head_dim;
  for (int r0 = 0; r0 < rows; r0 += kJoin) {
    float m[kJoin], l[kJoin];
    float4 o[kJoin];
#pragma unroll
    for (int r = 0; r < kJoin; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
      o[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int c0 = 0; c0 < n; c0 += 32) {
      // Lane i has partial c0 + i's statistics.
      const int cnt = min(32, n - c0);
      float f[kJoin], ls[kJoin];
#pragma unroll
      for (int r = 0; r < kJoin; ++r) {
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < cnt && r0 + r < rows)
          ml = __ldcg(reinterpret_cast<const float2*>(P.partials + slot_of(c0 + lane) * kFloats +
                                                      ROWS * DP) + r0 + r);
        f[r] = ml.x;
        ls[r] = ml.y;
      }
#pragma unroll
      for (int r = 0; r < kJoin; ++r) {
        float top = f[r];
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
        const float now = fmaxf(m[r], top);
        const float ref = now == -INFINITY ? 0.0f : now;
        const float keep = ex2(m[r] - ref);
        f[r] = ex2(f[r] - ref);
        m[r] = now;
        l[r] *= keep;
        o[r].x *= keep, o[r].y *= keep, o[r].z *= keep, o[r].w *= keep;
      }
#pragma unroll 4
      for (int i = 0; i < cnt; ++i) {
        const float* p = P.partials + slot_of(c0 + i) * kFloats + r0 * DP + d;
        float4 x[kJoin];
#pragma unroll
        for (int r = 0; r < kJoin; ++r) {
          x[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (live && r0 + r < rows) x[r] = __ldcg(reinterpret_cast<const float4*>(p + r * DP));
        }
#pragma unroll
        for (int r = 0; r < kJoin; ++r) {
          const float fi = __shfl_sync(kFull, f[r], i), li = __shfl_sync(kFull, ls[r], i);
          if (li != 0.0f) {  // otherwise that part saw nothing
            l[r] = fmaf(li, fi, l[r]);
            o[r].x = fmaf(x[r].x, fi, o[r].x);
            o[r].y = fmaf(x[r].y, fi, o[r].y);
            o[r].z = fmaf(x[r].z, fi, o[r].z);
            o[r].w = fmaf(x[r].w, fi, o[r].w);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kJoin; ++r)
      if (live && r0 + r < rows) put(r0 + r, d, m[r], l[r], o[r]);
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kWarps * 32, kRowCtasPerSm) attend_rows_kernel(
    const __grid_constant__ AttendParams P) {
  using L = Layout<DP>;
  constexpr int kChunks = DP / 16;
  const UnitShape kShape{kRows, kStep, 1, P.row_most, kLeast, kLead};
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row_lane = lane >> 2, col_lane = lane & 3;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * kWarps + warp;

  Cursor ld;  // where this warp loads
  const Range range = find_range<kWarps * 32, kWarps>(P, kShape, smem, &ld);
  if (ld.left == 0) {
    grid_dependency_wait();
    return;
  }
  Cursor cu = ld;  // where it computes

  // Ring: columns past head_dim stay zero throughout.
  const uint32_t ring = smem_addr(smem) + warp * L::kRing;
  if (P.c.head_dim < DP) {
    for (int i = lane; i < L::kRing / 16; i += 32)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring + i * 16), "r"(0) : "memory");
    __syncwarp();
  }
  auto chunk_at = [](int tok, int ch) {  // swizzled byte offset of a 16-byte chunk
    const int x = DP == 128 ? (tok & 7) : ((tok >> 1) & 3);
    return tok * DP + ((ch ^ x) << 4);
  };
  const int ps = P.c.page_size;
  const int slots = static_cast<int>(P.c.num_pages * ps);
  const int chunks = P.c.head_dim >> 4;
  int issued = 0;

  // The locations of this lane's position in the next units of the block, up to
  // kLook of them read at once, a unit ahead.
  int next[kLook], known = 0;
  auto look = [&]() {
    const int32_t* row = P.page_table + ld.r.table_row * P.pt_cols;
    known = static_cast<int>(min(ld.left, static_cast<int64_t>(min(ld.k.tiles - ld.tile, kLook))));
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      const int tok = ld.k.start + (ld.tile + i) * kStep + lane;
      next[i] = -1;
      if (i < known && tok >= ld.k.lo && tok < ld.k.end) next[i] = row[tok];
    }
  };
  look();
  constexpr int kPer = 32 / kChunks;  // positions a round of the warp's copies covers
  const int ch = lane % kChunks;
  // Copies the next unit, or commits an empty group.
  auto issue = [&]() {
    if (ld.left > 0) {
      const uint32_t slot = ring + (issued % kStages) * (L::kSlot + L::kScales);
      ++issued;
      int loc = next[0];
      const bool valid = loc >= 0 && loc < slots;
      if (!valid) {
        const int tok = ld.k.start + ld.tile * kStep + lane;
        if (tok >= ld.k.lo && tok < ld.k.end && P.status != nullptr)
          atomicOr(P.status, PKV_ST_ROW_OOB);
        loc = 0;
      }
      const int page = static_cast<int>(P.page_div.divide(static_cast<uint32_t>(loc)));
      // In units of 16 bytes: 32 bits reach 64 GiB.
      const uint32_t at = static_cast<uint32_t>(page) * P.page_step +
                          static_cast<uint32_t>(loc - page * ps) * P.token_step +
                          static_cast<uint32_t>(ld.head) * P.head_step;
      const int64_t sc = static_cast<int64_t>(page) * P.c.kv_heads + ld.head;
      cp_async4_zfill(slot + L::kSlot + lane * 4, P.c.k_scale + sc, valid);
      cp_async4_zfill(slot + L::kSlot + kStep * 4 + lane * 4, P.c.v_scale + sc, valid);
      const unsigned ok = __ballot_sync(kFull, valid) >> (lane / kChunks);
      const uint32_t dst = slot + chunk_at(lane / kChunks, ch);
#pragma unroll
      for (int i = 0; i < kStep / kPer; ++i) {
        const uint32_t from = __shfl_sync(kFull, at, i * kPer + lane / kChunks);
        if (ch < chunks) {
          const bool v = (ok >> (i * kPer)) & 1u;
          const uint64_t off = static_cast<uint64_t>(from) * 16 + ch * 16;
          // (The swizzle repeats every 8 positions.)
          const uint32_t to = kPer == 8 ? dst + i * 8 * DP
                              : (i & 1) ? slot + chunk_at(kPer + lane / kChunks, ch) + (i >> 1) * 8 * DP
                                        : dst + (i >> 1) * 8 * DP;
          cp_async16_zfill(to, static_cast<const uint8_t*>(P.c.k) + off, v);
          cp_async16_zfill(to + kStep * DP, static_cast<const uint8_t*>(P.c.v) + off, v);
        }
      }
      --ld.left;
      if (++ld.tile >= ld.k.tiles && ld.left > 0) next_block(P, ld, kShape);
      if (--known == 0) {
        look();
      } else {
#pragma unroll
        for (int i = 1; i < kLook; ++i) next[i - 1] = next[i];
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t qf[DP / 8];          // Q^T fragments
  float cf[2];                  // per row: score scale in log2 units
  int hi[2], lo[2];             // per row: positions seen
  float m[2], l[2];
  float o[DP / 16][4];
  int used = 0;

  while (cu.left > 0) {
    // ---- this block's units in the CTA's range
    const int t_begin = cu.tile;
    const int t_end = static_cast<int>(min(static_cast<int64_t>(cu.k.tiles), cu.tile + cu.left));
    const bool whole = t_begin == 0 && t_end == cu.k.tiles;
    int all_hi = INT32_MAX, all_lo = 0;  // seen by every row: [all_lo, all_hi]
    // Queries: this thread's fragment holds row row_lane,
    // elements [col_lane * DP / 4, + DP / 4).
    const bool live = row_lane < cu.k.rows && cu.r.end != 0;
    const int row = cu.k.row0 + row_lane, tok = row / P.group, g = row - tok * P.group;
    const uint16_t* src = P.q + (cu.q_off + tok) * P.q_ts +
                          static_cast<int64_t>(cu.head * P.group + g) * P.q_hs;
    const bool there = live && cu.q_off + tok < P.n_tokens;
    float amax = 0.0f;
    uint32_t raw[DP / 8];
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      const int d = col_lane * (DP / 4) + i * 8;
      if (there && d < P.c.head_dim) x = *reinterpret_cast<const uint4*>(src + d);
      raw[4 * i] = x.x, raw[4 * i + 1] = x.y, raw[4 * i + 2] = x.z, raw[4 * i + 3] = x.w;
    }
    float unit = 1.0f;
    if (P.bf16) {
      // To fp16 by way of a power of two that puts the row's largest in [2^14,
      // 2^15): bf16's 8 bits then fit down to 2^-31 of it.
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        const float2 x = Pair<T>::unpack(raw[i]);
        amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
      const int e = static_cast<int>(__float_as_uint(amax) >> 23);
      unit = __uint_as_float(static_cast<uint32_t>(min(268 - e, 253)) << 23);
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        const float2 x = Pair<T>::unpack(raw[i]);
        raw[i] = Pair<__half>::pack(x.x * unit, x.y * unit);
      }
    }
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) qf[i] = raw[i];
    // The products' columns of this thread: rows 2 col_lane and the next.
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 2 * col_lane + c;
      // (1 / unit by its exponent: a division takes its slow way for the large
      // units of rows that are not there.)
      cf[c] = P.scale_log2 * __uint_as_float(
          0x7f000000u - __float_as_uint(__shfl_sync(kFull, unit, (2 * col_lane + c) * 4)));
      const int p = cu.r.cached + (cu.k.row0 + r) / P.group;
      // (A row that is not there sees everything: it must not keep m waiting.)
      hi[c] = r < cu.k.rows ? min(p, cu.k.end - 1) : INT32_MAX;
      lo[c] = r < cu.k.rows ? cu.r.begin : 0;
      if (P.window > 0 && r < cu.k.rows) lo[c] = max(lo[c], p - P.window + 1);
      if (r < cu.k.rows) {
        all_hi = min(all_hi, hi[c]);
        all_lo = max(all_lo, lo[c]);
      }
      m[c] = -INFINITY;
      l[c] = 0.0f;
    }
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[d][i] = 0.0f;
    all_hi = __reduce_min_sync(kFull, all_hi);
    all_lo = __reduce_max_sync(kFull, all_lo);

    for (int tile = t_begin; tile < t_end; ++tile) {
      const int base = cu.k.start + tile * kStep;
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint32_t slot = ring + (used % kStages) * (L::kSlot + L::kScales);
      ++used;
      // ---- S^T = K Q^T, two tiles of 16 positions
      constexpr int kM = kStep / 16;
      float s[kM][4];
#pragma unroll
      for (int mt = 0; mt < kM; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][i] = 0.0f;
#pragma unroll
      for (int w = 0; w < DP / 64; ++w) {
        const int ch = col_lane * (DP / 64) + w;
#pragma unroll
        for (int mt = 0; mt < kM; ++mt) {
          const uint4 a = lds128(slot + chunk_at(16 * mt + row_lane, ch));
          const uint4 b = lds128(slot + chunk_at(16 * mt + row_lane + 8, ch));
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = e4m3x2_to_f16x2(aw[j]), a2 = e4m3x2_to_f16x2(aw[j] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(bw[j]), a3 = e4m3x2_to_f16x2(bw[j] >> 16);
            mma16816(s[mt], a0, a1, a2, a3, qf[8 * w + 2 * j], qf[8 * w + 2 * j + 1]);
          }
        }
      }
      // ---- softmax.  Position i of this thread: base + 8 i + row_lane.
      const uint32_t sc = slot + L::kSlot + row_lane * 4;
      float ks[2 * kM], vs[2 * kM];  // vs times kUnit
#pragma unroll
      for (int i = 0; i < 2 * kM; ++i) {
        ks[i] = lds32(sc + 32 * i);
        vs[i] = lds32(sc + kStep * 4 + 32 * i) * kUnit;
      }
      const bool partial = base < all_lo || base + kStep - 1 > all_hi;  // uniform
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 2 * kM; ++i) {
          float& x = s[i >> 1][2 * (i & 1) + c];
          x *= ks[i] * cf[c];
          if (partial) {
            const int p = base + 8 * i + row_lane;
            if (p < lo[c] || p > hi[c]) x = -INFINITY;
          }
        }
      }
      // Weights under the references as they are; where their sum passes the
      // limit, or a row has no reference yet, m moves and they are done again.
      float pw[kM][4], part[2];
      for (bool moved = false;; moved = true) {
        bool past = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float ref = m[c] == -INFINITY ? 0.0f : m[c];
          float held = 0.0f;
          part[c] = 0.0f;
#pragma unroll
          for (int i = 0; i < 2 * kM; ++i) {
            const float w = ex2(s[i >> 1][2 * (i & 1) + c] - ref);
            part[c] += w;
            const float x = w * vs[i];
            held += x;
            pw[i >> 1][2 * (i & 1) + c] = x;
          }
          past = past || !(held <= kLimit) || m[c] == -INFINITY;
        }
        if (moved || !__any_sync(kFull, past)) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float t = -INFINITY;
#pragma unroll
          for (int i = 0; i < 2 * kM; ++i)
            t = fmaxf(t, s[i >> 1][2 * (i & 1) + c] + lg2(fmaxf(vs[i], 0x1p-64f * kUnit)));
          t = fmaxf(t, __shfl_xor_sync(kFull, t, 4));
          t = fmaxf(t, __shfl_xor_sync(kFull, t, 8));
          t = fmaxf(t, __shfl_xor_sync(kFull, t, 16));
          // (The same in all lanes that hold the row's columns.)
          const float now = fmaxf(m[c], t);
          const float f = now == -INFINITY ? 1.0f : ex2(m[c] - now);
          m[c] = now;
          l[c] *= f;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            o[d][c] *= f;
            o[d][2 + c] *= f;
          }
        }
      }
      uint32_t pf[kM][2];
      l[0] += part[0];
      l[1] += part[1];
#pragma unroll
      for (int i = 0; i < 2 * kM; ++i)
        pf[i >> 1][i & 1] = transpose8x8(Pair<__half>::pack(pw[i >> 1][2 * (i & 1)],
                                                                pw[i >> 1][2 * (i & 1) + 1]));
      // ---- O^T += V^T P^T.  A transposed 8x8 of byte pairs holds, for one
      // pair of channels, two positions; the two channels go to rows r and
      // r + 8 of the product.
      const uint32_t vbase = slot + kStep * DP;
#pragma unroll
      for (int d2 = 0; d2 < DP / 32; ++d2) {
        if (2 * d2 * 16 >= P.c.head_dim) break;
#pragma unroll
        for (int mt = 0; mt < kM; ++mt) {
          // x4: positions 0-7, 8-15 of two chunks
          const uint4 v = ldsm_trans(vbase + chunk_at(16 * mt + (lane & 15), 2 * d2 + (lane >> 4)));
          uint32_t vw[4] = {v.x, v.y, v.z, v.w};
          // A NaN code in a position that some row does not see must reach only
          // the rows that do.
          if (partial) {
            const bool nan = has_nan(v.x) || has_nan(v.y) || has_nan(v.z) || has_nan(v.w);
            if (__any_sync(kFull, nan)) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t na[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  // 1 where the code is a NaN, and 0 in the code's place.
                  uint32_t x = vw[2 * k + j], ones = 0u, keep = 0xffffffffu;
#pragma unroll
                  for (int b = 0; b < 4; ++b) {
                    if (((x >> (8 * b)) & 0x7fu) == 0x7fu) {
                      ones |= 0x38u << (8 * b);  // e4m3 1.0
                      keep &= ~(0xffu << (8 * b));
                    }
                  }
                  vw[2 * k + j] = x & keep;
                  na[2 * j] = e4m3x2_to_f16x2(__byte_perm(ones, 0u, 0x0020));
                  na[2 * j + 1] = e4m3x2_to_f16x2(__byte_perm(ones, 0u, 0x0031));
                }
                float seen[4];
                const int p0 = base + 16 * mt + row_lane, p1 = p0 + 8;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  seen[c] = (p0 >= lo[c] && p0 <= hi[c]) ? 1.0f : 0.0f;
                  seen[2 + c] = (p1 >= lo[c] && p1 <= hi[c]) ? 1.0f : 0.0f;
                }
                const uint32_t b0 = transpose8x8(Pair<__half>::pack(seen[0], seen[1]));
                const uint32_t b1 = transpose8x8(Pair<__half>::pack(seen[2], seen[3]));
                float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16816(hit, na[0], na[1], na[2], na[3], b0, b1);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (hit[i] > 0.0f) o[2 * d2 + k][i] = __uint_as_float(0x7fffffffu);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x = __byte_perm(vw[2 * k], 0u, 0x3120);
            const uint32_t y = __byte_perm(vw[2 * k + 1], 0u, 0x3120);
            const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2_to_f16x2(x >> 16);
            const uint32_t a2 = e4m3x2_to_f16x2(y), a3 = e4m3x2_to_f16x2(y >> 16);
            mma16816(o[2 * d2 + k], a0, a1, a2, a3, pf[mt][0], pf[mt][1]);
          }
        }
      }
      __syncwarp();  // the slot may be refilled
      issue();
    }

    // ---- the block's end, or the range's
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float t = l[c];
      t += __shfl_xor_sync(kFull, t, 4);
      t += __shfl_xor_sync(kFull, t, 8);
      t += __shfl_xor_sync(kFull, t, 16);
      l[c] = t;
    }
    auto lse_of = [](float mm, float ll) {
      return ll != 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    };
    // Where row r of the block goes (token j; false: not written).
    auto place = [&](int r, int64_t* j, int* h) {
      const int tok = (cu.k.row0 + r) / P.group;
      *j = cu.q_off + tok;
      *h = cu.head * P.group + cu.k.row0 + r - tok * P.group;
      return r < cu.k.rows && *j < P.n_tokens;
    };
    if (whole) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        int64_t j;
        int h;
        if (!place(2 * col_lane + c, &j, &h)) continue;
        const float inv = l[c] != 0.0f ? (1.0f / kUnit) / l[c] : 0.0f;  // NaN stays NaN
        uint16_t* dst = P.out + j * P.o_ts + static_cast<int64_t>(h) * P.o_hs + 2 * row_lane;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
          if (d * 16 < P.c.head_dim)
            *reinterpret_cast<uint32_t*>(dst + d * 16) =
                Pair<T>::pack(o[d][c] * inv, o[d][2 + c] * inv);
        if (row_lane == 0 && P.lse != nullptr)
          P.lse[j * P.q_heads + h] = lse_of(m[c], l[c]);
      }
    } else {
      // Partial slots: 0 for a block that began in an earlier warp, 1 for one
      // that begins here and goes on.
      constexpr int kFloats = partial_floats(kRows, DP);
      float* mine = P.partials + (2 * worker + (t_begin == 0 ? 1 : 0)) * kFloats;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 2 * col_lane + c;
        if (r >= cu.k.rows) continue;
        float* dst = mine + r * DP + 2 * row_lane;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
          __stcg(reinterpret_cast<float2*>(dst + d * 16), make_float2(o[d][c], o[d][2 + c]));
        if (row_lane == 0)
          __stcg(reinterpret_cast<float2*>(mine + kRows * DP) + r, make_float2(m[c], l[c]));
      }
      int64_t c0, c1;
      block_workers(range, cu, &c0, &c1);
      // This warp's group of the block: workers [g0, g1].
      const int64_t first_group = c0 / kGroup, group = worker / kGroup;
      const int groups = static_cast<int>(c1 / kGroup - first_group) + 1;
      const int64_t g0 = max(c0, group * kGroup), g1 = min(c1, group * kGroup + kGroup - 1);
      auto slot_of = [&](int64_t w) { return 2 * w + (w == c0 ? 1 : 0); };
      // True in the last of n arrivals at a counter, which it resets.
      auto last_of = [&](uint32_t* counter, int64_t n) {
        __threadfence();
        __syncwarp();
        uint32_t is_last = 0u;
        if (lane == 0) {
          is_last = atomicAdd(counter, 1u) == static_cast<uint32_t>(n - 1) ? 1u : 0u;
          if (is_last != 0u) *counter = 0u;  // ready for the next call
        }
        is_last = __shfl_sync(kFull, is_last, 0);
        __threadfence();
        return is_last != 0u;
      };
      auto put_out = [&](int r, int d, float mm, float ll, const float4& x) {
        int64_t j;
        int h;
        if (!place(r, &j, &h)) return;
        const float inv = ll != 0.0f ? (1.0f / kUnit) / ll : 0.0f;
        *reinterpret_cast<uint2*>(P.out + j * P.o_ts + static_cast<int64_t>(h) * P.o_hs + d) =
            make_uint2(Pair<T>::pack(x.x * inv, x.y * inv), Pair<T>::pack(x.z * inv, x.w * inv));
        if (d == 0 && P.lse != nullptr) P.lse[j * P.q_heads + h] = lse_of(mm, ll);
      };
      auto in_group = [&](int i) { return slot_of(g0 + i); };
      const int members = static_cast<int>(g1 - g0) + 1;
      if (last_of(P.counters + slot_of(g0), members)) {
        if (groups == 1) {
          join<DP, kRows>(P, cu.k.rows, members, in_group, put_out);
        } else {
          // The group's sum takes the place of its first partial (which this
          // warp alone still reads, row by row ahead of the writes).
          float* sum = P.partials + slot_of(g0) * kFloats;
          join<DP, kRows>(P, cu.k.rows, members, in_group,
                          [&](int r, int d, float mm, float ll, const float4& x) {
                            __stcg(reinterpret_cast<float4*>(sum + r * DP + d), x);
                            if (d == 0)
                              __stcg(reinterpret_cast<float2*>(sum + kRows * DP) + r,
                                     make_float2(mm, ll));
                          });
          if (last_of(P.counters + 2 * range.workers + c0, groups)) {
            join<DP, kRows>(P, cu.k.rows, groups,
                            [&](int i) { return slot_of(max(c0, (first_group + i) * kGroup)); },
                            put_out);
          }
        }
      }
    }
    cu.left -= t_end - t_begin;
    if (cu.left > 0) next_block(P, cu, kShape);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  grid_dependency_wait();  // this grid ends no sooner than the tile kernel's
}

template <typename T, int DP>
cudaError_t launch(const AttendParams& P, int ctas, bool beside, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0ull};
  const auto kernel = attend_rows_kernel<T, DP>;
  constexpr int bytes = Layout<DP>::kBytes;
  const cudaError_t e = set_smem_limit_once(done, kernel, bytes);
  if (e != cudaSuccess) return e;
  // After the tile kernel it need not wait for that, whose results are other
  // rows': it starts wherever that leaves room.
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(ctas);
  config.blockDim = dim3(kWarps * 32);
  config.dynamicSmemBytes = bytes;
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&config, kernel, P);
}

template <typename T>
cudaError_t launch_type(const AttendParams& P, int ctas, bool beside, cudaStream_t stream) {
  return P.c.head_dim > 64 ? launch<T, 128>(P, ctas, beside, stream)
                           : launch<T, 64>(P, ctas, beside, stream);
}

}  // namespace

size_t row_partial_bytes(int ctas, int head_dim) {
  return static_cast<size_t>(ctas) * kWarps * 2 * partial_floats(kRows, head_dim > 64 ? 128 : 64) * 4;
}

cudaError_t launch_attend_rows(const AttendParams& P, int ctas, bool beside, cudaStream_t stream) {
  return P.bf16 ? launch_type<__nv_bfloat16>(P, ctas, beside, stream)
                : launch_type<__half>(P, ctas, beside, stream);
}

}  // namespace pkv
