// Attention of few query rows a request over the paged e4m3 cache: decoding
// (one token a request), verification of a few draft tokens.
//
// A row is one (query token, query head); the rows of one cache head share its
// keys and values.  A work unit is a tile of kTile positions for one block of
// up to 8 * NT rows of one (request, cache head).  All units of the call, in
// batch order, are cut into equal contiguous ranges, one per CTA, so ragged
// lengths balance and one long request fills the machine.  A CTA that holds
// only part of a block's units leaves its partial (m, l, O) in the workspace;
// the last of the block's CTAs to finish joins the partials in CTA order.
//
// Inside a CTA each warp streams its own 16-position steps through its own
// ring of shared memory (cp.async) and keeps its own running softmax; the
// warps meet once at the end of a block.  Per step, with keys and values as
// the A operand so that the few rows are the narrow side of the product:
//   S^T[16 x 8] = K[16 x D] Q^T,   O^T[D x 8] += V^T[D x 16] P^T
// on mma.m16n8k16 with fp16 inputs: e4m3 codes are exact in fp16, and a query
// is scaled to at most 2 by a power of two, so the products are exact.  Scores
// take the page's key scale in fp32.  Weights carry the page's value scale:
// with m the running maximum of s + log2(vs), p = 2^(s - m) vs <= 2^8 goes to
// fp16 (11 bits), and l sums 2^(s - m) in fp32, so neither over- nor
// underflows for any scales.  m moves only when it would rise by more than 8:
// sums stay far below fp16's and fp32's limits and most steps rescale nothing.
//
// Bound: bytes.  Each cached byte is read once (2 D per position and head).

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

constexpr int kWarps = 4;
constexpr int kStep = 16;                // positions a warp takes at a time
constexpr int kTile = kWarps * kStep;    // positions of a work unit
constexpr int kStages = 4;               // ring slots of a warp
constexpr float kLazy = 8.0f;            // log2 of how far sums may outgrow their reference
constexpr float kLn2 = 0.693147180559945309f;

template <int DP>
struct Layout {
  static constexpr int kPitch = DP + 8;                    // floats a row of the joining buffer
  static constexpr int kSlot = 2 * kStep * DP;             // K then V codes
  static constexpr int kScales = 2 * kStep * 4;            // key then value scales
  static constexpr int kRing = kWarps * kStages * (kSlot + kScales);
};

template <int DP, int NT>
constexpr int smem_bytes() {
  return Layout<DP>::kRing + kWarps * 8 * NT * Layout<DP>::kPitch * 4 + kWarps * 8 * NT * 8 + 64;
}

// Floats of one partial result: O [rows, DP], then m and l [rows].
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

template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kWarps * 32, kRowCtasPerSm) attend_rows_kernel(const AttendParams P) {
  using L = Layout<DP>;
  constexpr int kRows = 8 * NT;
  constexpr int kChunks = DP / 16;
  constexpr UnitShape kShape{kRows, kTile, 1, kRowLimit};
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_o = reinterpret_cast<float*>(smem + L::kRing);
  float2* s_ml = reinterpret_cast<float2*>(s_o + kWarps * kRows * L::kPitch);
  int* s_last = reinterpret_cast<int*>(s_ml + kWarps * kRows);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row_lane = lane >> 2, col_lane = lane & 3;

  Cursor ld;  // where this warp loads
  const Range range = find_range<kWarps * 32>(P, kShape, smem, &ld);
  if (ld.left == 0) return;
  Cursor cu = ld;  // where it computes

  // Ring: columns past head_dim stay zero throughout.
  const uint32_t ring = smem_addr(smem) + warp * kStages * (L::kSlot + L::kScales);
  if (P.c.head_dim < DP) {
    for (int i = lane; i < kStages * (L::kSlot + L::kScales) / 16; i += 32)
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

  // Copies the next step of this warp's share, or commits an empty group.
  auto issue = [&]() {
    while (ld.left > 0) {
      const int base = ld.k.start + ld.tile * kTile + warp * kStep;
      const bool some = base < ld.k.end;
      if (some) {
        const uint32_t slot = ring + (issued % kStages) * (L::kSlot + L::kScales);
        ++issued;
        const int tok = base + (lane & 15);
        bool valid = tok >= ld.k.lo && tok < ld.k.end;
        int loc = 0;
        if (valid) loc = P.page_table[ld.r.table_row * P.pt_cols + tok];
        if (loc < 0 || loc >= slots) {
          if (P.status != nullptr) atomicOr(P.status, PKV_ST_ROW_OOB);
          loc = 0;
          valid = false;
        }
        const int page = static_cast<int>(P.page_div.divide(static_cast<uint32_t>(loc)));
        const int64_t at = page * P.c.page_stride + (loc - page * ps) * P.c.token_stride +
                           ld.head * P.c.head_stride;
        const unsigned ok = __ballot_sync(kFull, valid);
        constexpr int kPer = 32 / kChunks;  // positions a round of the warp covers
        const int ch = lane % kChunks;
#pragma unroll
        for (int i = 0; i < kStep / kPer; ++i) {
          const int t = i * kPer + lane / kChunks;
          const int64_t off = __shfl_sync(kFull, at, t);
          if (ch < chunks) {
            const bool v = (ok >> t) & 1u;
            const uint32_t dst = slot + chunk_at(t, ch);
            cp_async16_zfill(dst, static_cast<const uint8_t*>(P.c.k) + off + ch * 16, v);
            cp_async16_zfill(dst + kStep * DP, static_cast<const uint8_t*>(P.c.v) + off + ch * 16, v);
          }
        }
        const float* sc = lane < 16 ? P.c.k_scale : P.c.v_scale;
        cp_async4_zfill(slot + L::kSlot + lane * 4,
                        sc + static_cast<int64_t>(page) * P.c.kv_heads + ld.head, valid);
      }
      --ld.left;
      if (++ld.tile >= ld.k.tiles && ld.left > 0) next_block(P, ld, kShape);
      if (some) break;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t qf[NT][DP / 8];      // Q^T fragments
  float cf[NT][2];              // per row: score scale in log2 units
  int hi[NT][2], lo[NT][2];     // per row: positions seen
  float m[NT][2], l[NT][2];
  float o[DP / 16][NT][4];
  int used = 0;

  while (cu.left > 0) {
    // ---- this block's units in the CTA's range
    const int t_begin = cu.tile;
    const int t_end = static_cast<int>(min(static_cast<int64_t>(cu.k.tiles), cu.tile + cu.left));
    const bool whole = t_begin == 0 && t_end == cu.k.tiles;
    int all_hi = INT32_MAX, all_lo = 0;  // seen by every row: [all_lo, all_hi]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // Queries: this thread's fragment holds row nt * 8 + row_lane,
      // elements [col_lane * DP / 4, + DP / 4).
      const int row = nt * 8 + row_lane;
      const bool live = row < cu.k.rows && cu.r.end != 0;
      const int tok = (cu.k.row0 + row) / P.group, g = (cu.k.row0 + row) - tok * P.group;
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
        // To fp16 by way of a power of two that puts the row's largest in [1, 2).
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          const float2 x = Pair<T>::unpack(raw[i]);
          amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int e = static_cast<int>(__float_as_uint(amax) >> 23);
        if (e > 0 && e < 254) unit = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          const float2 x = Pair<T>::unpack(raw[i]);
          raw[i] = Pair<__half>::pack(x.x * unit, x.y * unit);
        }
      }
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) qf[nt][i] = raw[i];
      // The products' columns of this thread: rows 2 col_lane and the next.
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * col_lane + c;
        cf[nt][c] = P.scale_log2 / __shfl_sync(kFull, unit, (2 * col_lane + c) * 4);
        const int p = cu.r.cached + (cu.k.row0 + r) / P.group;
        hi[nt][c] = r < cu.k.rows ? p : -1;
        lo[nt][c] = cu.r.begin;
        if (P.window > 0) lo[nt][c] = max(lo[nt][c], p - P.window + 1);
        if (r < cu.k.rows) {
          all_hi = min(all_hi, hi[nt][c]);
          all_lo = max(all_lo, lo[nt][c]);
        }
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
      }
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][nt][i] = 0.0f;
    }
    all_hi = __reduce_min_sync(kFull, all_hi);
    all_lo = __reduce_max_sync(kFull, all_lo);

    for (int tile = t_begin; tile < t_end; ++tile) {
      const int base = cu.k.start + tile * kTile + warp * kStep;
      if (base >= cu.k.end) continue;
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint32_t slot = ring + (used % kStages) * (L::kSlot + L::kScales);
      ++used;
      // ---- S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.0f;
#pragma unroll
      for (int w = 0; w < DP / 64; ++w) {
        const int ch = col_lane * (DP / 64) + w;
        const uint4 a = lds128(slot + chunk_at(row_lane, ch));
        const uint4 b = lds128(slot + chunk_at(row_lane + 8, ch));
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = e4m3x2_to_f16x2(aw[j]), a2 = e4m3x2_to_f16x2(aw[j] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(bw[j]), a3 = e4m3x2_to_f16x2(bw[j] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(s[nt], a0, a1, a2, a3, qf[nt][8 * w + 2 * j], qf[nt][8 * w + 2 * j + 1]);
        }
      }
      // ---- softmax
      const uint32_t sc = slot + L::kSlot + row_lane * 4;
      const float ks0 = lds32(sc), ks1 = lds32(sc + 32);
      const float vs0 = lds32(sc + 64), vs1 = lds32(sc + 96);
      const float lv0 = lg2(fmaxf(vs0, 5.42101086e-20f)), lv1 = lg2(fmaxf(vs1, 5.42101086e-20f));
      const int p0 = base + row_lane, p1 = p0 + 8;
      const bool partial = base < all_lo || base + kStep - 1 > all_hi;  // uniform
      float top[NT][2];
      bool rise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s[nt][c] *= ks0 * cf[nt][c];
          s[nt][2 + c] *= ks1 * cf[nt][c];
          if (partial) {
            if (p0 < lo[nt][c] || p0 > hi[nt][c]) s[nt][c] = -INFINITY;
            if (p1 < lo[nt][c] || p1 > hi[nt][c]) s[nt][2 + c] = -INFINITY;
          }
          float t = fmaxf(s[nt][c] + lv0, s[nt][2 + c] + lv1);
          t = fmaxf(t, __shfl_xor_sync(kFull, t, 4));
          t = fmaxf(t, __shfl_xor_sync(kFull, t, 8));
          t = fmaxf(t, __shfl_xor_sync(kFull, t, 16));
          top[nt][c] = t;
          rise = rise || t > m[nt][c] + kLazy;
        }
      }
      if (__any_sync(kFull, rise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float now = fmaxf(m[nt][c], top[nt][c]);
            const float f = now == -INFINITY ? 1.0f : ex2(m[nt][c] - now);
            m[nt][c] = now;
            l[nt][c] *= f;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
              o[d][nt][c] *= f;
              o[d][nt][2 + c] *= f;
            }
          }
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float ref = m[nt][c] == -INFINITY ? 0.0f : m[nt][c];
          w[c] = ex2(s[nt][c] - ref);
          w[2 + c] = ex2(s[nt][2 + c] - ref);
          l[nt][c] += w[c] + w[2 + c];
        }
        pf[nt][0] = transpose8x8(Pair<__half>::pack(w[0] * vs0, w[1] * vs0));
        pf[nt][1] = transpose8x8(Pair<__half>::pack(w[2] * vs1, w[3] * vs1));
      }
      // ---- O^T += V^T P^T.  A transposed 8x8 of byte pairs holds, for one
      // pair of channels, two positions; the two channels go to rows r and
      // r + 8 of the product.
      const uint32_t vbase = slot + kStep * DP;
      const int tok = (lane & 7) + (lane & 8);  // x4: positions 0-7, 8-15 of two chunks
#pragma unroll
      for (int d2 = 0; d2 < DP / 32; ++d2) {
        if (2 * d2 * 16 >= P.c.head_dim) break;
        uint4 v = ldsm_trans(vbase + chunk_at(tok, 2 * d2 + (lane >> 4)));
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
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float seen[4];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  seen[c] = (p0 >= lo[nt][c] && p0 <= hi[nt][c]) ? 1.0f : 0.0f;
                  seen[2 + c] = (p1 >= lo[nt][c] && p1 <= hi[nt][c]) ? 1.0f : 0.0f;
                }
                const uint32_t b0 = transpose8x8(Pair<__half>::pack(seen[0], seen[1]));
                const uint32_t b1 = transpose8x8(Pair<__half>::pack(seen[2], seen[3]));
                float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16816(hit, na[0], na[1], na[2], na[3], b0, b1);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (hit[i] > 0.0f) o[2 * d2 + k][nt][i] = __uint_as_float(0x7fffffffu);
              }
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = vw[2 * k], y = vw[2 * k + 1];
          const uint32_t a0 = e4m3x2_to_f16x2(__byte_perm(x, 0u, 0x0020));
          const uint32_t a1 = e4m3x2_to_f16x2(__byte_perm(x, 0u, 0x0031));
          const uint32_t a2 = e4m3x2_to_f16x2(__byte_perm(y, 0u, 0x0020));
          const uint32_t a3 = e4m3x2_to_f16x2(__byte_perm(y, 0u, 0x0031));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[2 * d2 + k][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
      }
      __syncwarp();  // the slot may be refilled
      issue();
    }

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float t = l[nt][c];
        t += __shfl_xor_sync(kFull, t, 4);
        t += __shfl_xor_sync(kFull, t, 8);
        t += __shfl_xor_sync(kFull, t, 16);
        const int r = nt * 8 + 2 * col_lane + c;
        if (row_lane == 0) s_ml[warp * kRows + r] = make_float2(m[nt][c], t);
        if (r < cu.k.rows) {
          float* dst = s_o + (warp * kRows + r) * L::kPitch + 2 * row_lane;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d)
            *reinterpret_cast<float2*>(dst + d * 16) = make_float2(o[d][nt][c], o[d][nt][2 + c]);
        }
      }
    }
    __syncthreads();
    // Joins `count` partials (m, l, O) of one row and four channels.
    struct Sum { float m, l; float4 o; };
    auto store = [&](int row, int d, const Sum& a) {
      const int tok = (cu.k.row0 + row) / P.group, g = cu.k.row0 + row - tok * P.group;
      const int64_t j = cu.q_off + tok;
      if (j >= P.n_tokens) return;
      const int h = cu.head * P.group + g;
      const float inv = a.l != 0.0f ? 1.0f / a.l : 0.0f;  // NaN stays NaN
      *reinterpret_cast<uint2*>(P.out + j * P.o_ts + static_cast<int64_t>(h) * P.o_hs + d) =
          make_uint2(Pair<T>::pack(a.o.x * inv, a.o.y * inv), Pair<T>::pack(a.o.z * inv, a.o.w * inv));
      if (d == 0 && P.lse != nullptr)
        P.lse[j * P.q_heads + h] = a.l != 0.0f ? (a.m + log2f(a.l)) * kLn2 : -INFINITY;
    };
    auto add = [](Sum& a, float bm, float bl, const float4& bo) {
      const float now = fmaxf(a.m, bm);
      if (now == -INFINITY && bl == 0.0f) return;  // nothing seen there
      const float ref = now == -INFINITY ? 0.0f : now;
      const float fa = ex2(a.m - ref), fb = ex2(bm - ref);
      a.m = now;
      a.l = a.l * fa + bl * fb;
      a.o.x = a.o.x * fa + bo.x * fb;
      a.o.y = a.o.y * fa + bo.y * fb;
      a.o.z = a.o.z * fa + bo.z * fb;
      a.o.w = a.o.w * fa + bo.w * fb;
    };
    // Partial slots: 0 for a block that began in an earlier CTA, 1 for one
    // that begins here and goes on.
    const int64_t seg_first = range.last - cu.left;              // this segment's first unit
    const int64_t block_first = seg_first - t_begin;       // the block's first unit
    int64_t c0, c1;
    block_ctas(range, block_first, cu.k.tiles, &c0, &c1);
    const int quads = P.c.head_dim >> 2;
    const int pf_floats = partial_floats(kRows, DP);
    float* mine = P.partials + (2 * blockIdx.x + (t_begin == 0 ? 1 : 0)) * static_cast<int64_t>(pf_floats);
    for (int i = tid; i < cu.k.rows * quads; i += kWarps * 32) {
      const int row = i / quads, d = (i - row * quads) * 4;
      Sum a{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * kRows + row];
        add(a, ml.x, ml.y, *reinterpret_cast<const float4*>(s_o + (w * kRows + row) * L::kPitch + d));
      }
      if (whole) {
        store(row, d, a);
      } else {
        __stcg(reinterpret_cast<float4*>(mine + row * DP + d), a.o);
        if (d == 0) __stcg(reinterpret_cast<float2*>(mine + kRows * DP + 2 * row), make_float2(a.m, a.l));
      }
    }
    if (!whole) {
      // The last of the block's CTAs to get here joins its partials.
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = atomicAdd(P.counters + c0, 1u);
        const bool mine_last = before == static_cast<uint32_t>(c1 - c0);
        if (mine_last) P.counters[c0] = 0u;  // ready for the next call
        __threadfence();
        *s_last = mine_last ? 1 : 0;
      }
      __syncthreads();
      if (*s_last != 0) {
        for (int i = tid; i < cu.k.rows * quads; i += kWarps * 32) {
          const int row = i / quads, d = (i - row * quads) * 4;
          Sum a{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
          for (int64_t c = c0; c <= c1; ++c) {
            const float* p = P.partials + (2 * c + (c == c0 ? 1 : 0)) * static_cast<int64_t>(pf_floats);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + kRows * DP + 2 * row));
            add(a, ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(p + row * DP + d)));
          }
          store(row, d, a);
        }
      }
    }
    __syncthreads();  // the joining buffer is free again
    cu.left -= t_end - t_begin;
    if (cu.left > 0) next_block(P, cu, kShape);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int DP, int NT>
cudaError_t launch(const AttendParams& P, int ctas, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0ull};
  const auto kernel = attend_rows_kernel<T, DP, NT>;
  const int bytes = smem_bytes<DP, NT>();
  const cudaError_t e = set_smem_limit_once(done, kernel, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kWarps * 32, bytes, stream>>>(P);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AttendParams& P, int rows, int ctas, cudaStream_t stream) {
  const bool wide = P.c.head_dim > 64;
  if (rows == 8)
    return wide ? launch<T, 128, 1>(P, ctas, stream) : launch<T, 64, 1>(P, ctas, stream);
  return wide ? launch<T, 128, 2>(P, ctas, stream) : launch<T, 64, 2>(P, ctas, stream);
}

}  // namespace

int row_block(int max_q_len, int group) {
  return static_cast<int64_t>(max_q_len) * group <= 8 ? 8 : 16;
}

size_t row_partial_bytes(int rows, int ctas, int head_dim) {
  return static_cast<size_t>(ctas) * 2 * partial_floats(rows, head_dim > 64 ? 128 : 64) * 4;
}

cudaError_t launch_attend_rows(const AttendParams& P, int rows, int ctas, cudaStream_t stream) {
  return P.bf16 ? launch_type<__nv_bfloat16>(P, rows, ctas, stream)
                : launch_type<__half>(P, rows, ctas, stream);
}

}  // namespace pkv
