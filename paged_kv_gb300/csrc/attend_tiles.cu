// Attention of many query rows a request over the paged e4m3 cache: prompt
// chunks on the tensor cores.
//
// A unit (attend_units.cuh) is 128 positions for a block of up to 256 rows of
// one (request, cache head), held as two tiles of 128 rows.  Per unit and tile
//   S[128 x 128] = Q K^T   on kind::f8f6f4: K's codes go to the tensor core as
//     they are; a query row, scaled by a power of two, is the sum of NS e4m3
//     rows, exactly: 4 significant bits each, so 2 for bf16 and 3 for fp16
//     (elements below 2^-9 of a row's largest keep an absolute 2^-17 of it);
//   S times the page's key scale and the row's factor, softmax in fp32;
//   O[128 x D] += P V      on kind::f16: P is bf16 in tensor memory, in S's
//     place; V is made bf16 (code times page scale) on its way to shared
//     memory.  bf16 on both sides because weights and scales need its range: a
//     long context's weights may lie 2^-20 below an early large one and still
//     add up to as much.
// The running maximum m moves only when it would rise by more than 8 (in
// log2): then O is rescaled in tensor memory by the row's own thread.
//
// Roles (16 warps): warps 0-3 and 4-7 are the softmax of tile 0 and 1, a
// thread a row; warps 8-11 load: K by cp.async, V through registers (converted
// there), page places and scales a unit ahead; one thread of warp 12 issues
// the products.  While one tile is in its softmax the other's products run.
//   k_full/k_empty, v_full/v_empty: rings of units in shared memory;
//   sc_full: the units' key scales;  q_full[t]: the block's queries;
//   s_full[t]: S is there, and O and P of the unit before are done with;
//   p_full[t]: P is there (and O rescaled), S may be overwritten.
// Products of one thread run in issue order, so P V and the next Q K^T of a
// tile, which writes over P, need no barrier between them.
//
// Every wait ends: after kWaitNs a thread sets `dead`, with which all waits
// return at once, the loops (whose lengths do not depend on data) run out,
// tensor memory is freed and PKV_ST_TIMEOUT is set.
//
// Bound: instruction issue of the softmax and conversion warps (about 1500
// issue cycles per SM quarter a unit against 1024 tensor cycles).

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
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 512;
constexpr int kTileRows = 128;
constexpr int kBlockRows = 2 * kTileRows;
constexpr int kTile = 128;               // positions of a unit
constexpr int kPitch = 128;              // bytes of an 8-bit row in shared memory
constexpr int kQBytes = kTileRows * kPitch;
constexpr int kKBytes = kTile * kPitch;
constexpr int kVHalf = kTile * 128;      // 64 channels of bf16
constexpr int kVBytes = 2 * kVHalf;
constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr long long kWaitNs = 2000000000ll;
__host__ __device__ constexpr UnitShape unit_shape() {
  return UnitShape{kBlockRows, kTile, kRowLimit + 1, int64_t{1} << 40};
}

template <int NS>
struct Plan {
  static constexpr int kK = 3;                       // ring slots
  static constexpr int kV = NS == 2 ? 3 : 2;
  static constexpr int kSc = kK + 1;
  static constexpr int q = 0;
  static constexpr int k = q + 2 * NS * kQBytes;
  static constexpr int v = k + kK * kKBytes;
  static constexpr int sc = v + kV * kVBytes;        // key scales, kSc slots
  static constexpr int vs = sc + kSc * kTile * 4;    // value scales, 3 slots
  static constexpr int off = vs + 3 * kTile * 4;     // byte offsets, 3 slots
  static constexpr int bar = off + 3 * kTile * 8;
  static constexpr int bytes = bar + 512 + 1024;     // and room to align
};

struct Bars {
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3], sc_full[4];
  uint64_t q_full[2], s_full[2], p_full[2];
  uint32_t tmem;
  int dead;
  int last[2];
  int nan;
};

// Phase bookkeeping of a ring.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) slot = 0, phase ^= 1u;
  }
};

__device__ __forceinline__ void wait(Bars* B, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&B->dead) != 0) return;
    if (globaltimer_ns() - t0 > kWaitNs) {
      *reinterpret_cast<volatile int*>(&B->dead) = 1;
      return;
    }
  }
}

template <int ID>
__device__ __forceinline__ void bar_sync(int id_add = 0) {
  asm volatile("bar.sync %0, 128;" ::"r"(ID + id_add) : "memory");
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// Floats of one tile's partial result: O as [D / 4][128 rows] float4, m and l,
// [128 rows] float2, and whether a NaN was left out.
__host__ __device__ constexpr int64_t partial_floats(int head_dim) {
  return static_cast<int64_t>(kTileRows) * (head_dim + 2) + 4;
}

// ------------------------------------------------------------------ loading

template <int NS>
__device__ void load_role(const AttendParams& P, Cursor c, uint8_t* smem, Bars* B) {
  using L = Plan<NS>;
  const int tid = threadIdx.x & 127;
  const int ps = P.c.page_size;
  const int slots = static_cast<int>(P.c.num_pages * ps);
  const int chunks = P.c.head_dim >> 4;
  const int ch = tid & 7, t0 = tid >> 3;
  const bool mine = ch < chunks;
  float* s_sc = reinterpret_cast<float*>(smem + L::sc);
  float* s_vs = reinterpret_cast<float*>(smem + L::vs);
  int64_t* s_off = reinterpret_cast<int64_t*>(smem + L::off);

  // Places run two units ahead of the loads: unit u's table entry is read at
  // u - 2, its scales at u - 1.
  Cursor a = c;               // the unit whose table entry is read next
  auto step = [&](Cursor& x) {
    --x.left;
    if (++x.tile >= x.k.tiles && x.left > 0) next_block(P, x, unit_shape());
  };
  struct Place { int loc, head; };  // loc -1: nothing there
  auto read_place = [&]() -> Place {
    Place p{-1, 0};
    if (a.left > 0) {
      const int tok = a.k.start + a.tile * kTile + tid;
      if (tok < a.k.end) {
        p.loc = P.page_table[a.r.table_row * P.pt_cols + tok];
        if (p.loc < 0 || p.loc >= slots) {
          if (P.status != nullptr) atomicOr(P.status, PKV_ST_ROW_OOB);
          p.loc = -1;
        }
      }
      p.head = a.head;
      step(a);
    }
    return p;
  };
  float ks = 0.0f, vs = 0.0f;
  auto resolve = [&](const Place& p, int slot) {  // byte offsets, and the scales' loads
    int64_t off = -1;
    ks = vs = 0.0f;
    if (p.loc >= 0) {
      const int page = p.loc / ps;
      off = page * P.c.page_stride + (p.loc - page * ps) * P.c.token_stride +
            p.head * P.c.head_stride;
      const int64_t s = static_cast<int64_t>(page) * P.c.kv_heads + p.head;
      ks = P.c.k_scale[s];
      vs = P.c.v_scale[s];
    }
    s_off[slot * kTile + tid] = off;
  };

  Ring kr, vr, sr;
  int three = 0;              // slot of unit i's places
  uint4 raw[8];
  bool pending = false;       // V of the unit before is in `raw`
  bool pending_partial = false;
  int pending_three = 0;
  auto convert = [&]() {
    wait(B, &B->v_empty[vr.slot], vr.phase ^ 1u);
    uint8_t* dst = smem + L::v + vr.slot * kVBytes + (ch >> 2) * kVHalf;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = t0 + 16 * i;
      const float scale = s_vs[pending_three * kTile + t];
      uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      if (pending_partial) {
        // A NaN that some row does not see: zero here, put back at the end.
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t hit = (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
          if (hit != 0u) nan = true;
          w[k] &= ~(hit * 255u);
        }
      }
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = Pair<__half>::unpack(e4m3x2_to_f16x2(w[k]));
        const float2 y = Pair<__half>::unpack(e4m3x2_to_f16x2(w[k] >> 16));
        o[2 * k] = Pair<__nv_bfloat16>::pack(x.x * scale, x.y * scale);
        o[2 * k + 1] = Pair<__nv_bfloat16>::pack(y.x * scale, y.y * scale);
      }
      if (mine) {
        // 32 bytes: chunks 2 (ch % 4) and the next; the halves' lanes store
        // them in opposite order, so that a quarter warp covers all banks.
        const int c0 = (ch & 3) * 2, swap = ch >> 2;
        uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
        *reinterpret_cast<uint4*>(dst + chunk_at(t, c0 + swap)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(dst + chunk_at(t, c0 + 1 - swap)) = swap ? lo : hi;
      }
    }
    if (nan) *reinterpret_cast<volatile int*>(&B->nan) = 1;
    tc::fence_smem();
    mbar_arrive(&B->v_full[vr.slot]);
    vr.next(L::kV);
  };

  Place ahead = read_place();
  resolve(ahead, 0);
  ahead = read_place();
  while (c.left > 0) {
    // ---- this unit's scales; the next one's offsets; the one after's entry
    s_sc[sr.slot * kTile + tid] = ks;
    s_vs[three * kTile + tid] = vs;
    const int next_three = three == 2 ? 0 : three + 1;
    resolve(ahead, next_three);
    ahead = read_place();
    bar_sync<1>();
    mbar_arrive(&B->sc_full[sr.slot]);
    sr.next(L::kSc);
    // ---- K
    wait(B, &B->k_empty[kr.slot], kr.phase ^ 1u);
    const int64_t* offs = s_off + three * kTile + t0;
    const uint32_t kdst = smem_addr(smem + L::k + kr.slot * kKBytes);
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t off = offs[16 * i];
        const uint8_t* src = static_cast<const uint8_t*>(P.c.k) + (off < 0 ? 0 : off) + ch * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(kdst + chunk_at(t0 + 16 * i, ch)), "l"(src), "r"(off < 0 ? 0 : 16)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // ---- V of the unit before, then this unit's loads
    if (pending) convert();
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t off = offs[16 * i];
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (off >= 0)
          raw[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(P.c.v) + off + ch * 16));
      }
    }
    {
      // Whether every row of the block sees every position of this unit.
      const int base = c.k.start + c.tile * kTile;
      const int t_first = c.k.row0 / P.group, t_last = (c.k.row0 + c.k.rows - 1) / P.group;
      int all_lo = c.r.begin;
      if (P.window > 0) all_lo = max(all_lo, c.r.cached + t_last - P.window + 1);
      pending_partial = base < all_lo || base + kTile - 1 > min(c.r.cached + t_first, c.k.end - 1);
    }
    pending = true;
    pending_three = three;
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc::fence_smem();
    mbar_arrive(&B->k_full[kr.slot]);
    kr.next(L::kK);
    three = next_three;
    step(c);
  }
  if (pending) convert();
}

// ------------------------------------------------------------------ products

template <int NS>
__device__ void mma_role(const AttendParams& P, Cursor c, uint8_t* smem, Bars* B) {
  using L = Plan<NS>;
  const uint32_t tmem = B->tmem;
  const int ksteps = (P.c.head_dim + 31) >> 5;
  const uint32_t qk_instr = tc::instruction(0, kTile, false);
  const uint32_t pv_instr = tc::instruction(1, P.c.head_dim, true);
  const uint32_t q0 = smem_addr(smem + L::q), k0 = smem_addr(smem + L::k), v0 = smem_addr(smem + L::v);
  Ring kr, vr;
  uint32_t q_phase[2] = {0u, 0u}, p_phase[2] = {0u, 0u};
  auto qk = [&](int t) {
    const uint64_t kd = tc::operand(k0 + kr.slot * kKBytes, 1024, 16);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint64_t qd = tc::operand(q0 + (t * NS + s) * kQBytes, 1024, 16);
      for (int k = 0; k < ksteps; ++k)
        tc::mma8_ss(tmem + t * kTile, qd + 2 * k, kd + 2 * k, qk_instr, s + k > 0);
    }
  };
  while (c.left > 0) {
    const int n = static_cast<int>(min(static_cast<int64_t>(c.k.tiles - c.tile), c.left));
    const int tiles = c.k.rows > kTileRows ? 2 : 1;
    wait(B, &B->k_full[kr.slot], kr.phase);
    for (int t = 0; t < tiles; ++t) {
      wait(B, &B->q_full[t], q_phase[t]);
      q_phase[t] ^= 1u;
      tc::fence_after();
      qk(t);
      tc::commit(&B->s_full[t]);
    }
    tc::commit(&B->k_empty[kr.slot]);
    kr.next(L::kK);
    for (int j = 0; j < n; ++j) {
      const uint64_t vd = tc::operand(v0 + vr.slot * kVBytes, 1024, kVHalf);
      for (int t = 0; t < tiles; ++t) {
        wait(B, &B->p_full[t], p_phase[t]);
        p_phase[t] ^= 1u;
        if (t == 0) wait(B, &B->v_full[vr.slot], vr.phase);
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tc::mma16_ts(tmem + 256 + t * 128, tmem + t * kTile + 8 * k, vd + 128 * k, pv_instr,
                       j + k > 0);
        if (j + 1 < n) {
          if (t == 0) wait(B, &B->k_full[kr.slot], kr.phase);
          tc::fence_after();
          qk(t);
        }
        tc::commit(&B->s_full[t]);
      }
      tc::commit(&B->v_empty[vr.slot]);
      vr.next(L::kV);
      if (j + 1 < n) {
        tc::commit(&B->k_empty[kr.slot]);
        kr.next(L::kK);
      }
    }
    c.left -= n;
    if (c.left > 0) next_block(P, c, unit_shape());
  }
}

// ------------------------------------------------------------------ softmax

template <typename T, int NS>
__device__ void softmax_role(const AttendParams& P, Cursor c, const Range& range, uint8_t* smem,
                             Bars* B, int t) {
  using L = Plan<NS>;
  const int tid = threadIdx.x & 127, warp = tid >> 5;
  const uint32_t s_tmem = B->tmem + (static_cast<uint32_t>(warp * 32) << 16) + t * kTile;
  const uint32_t o_tmem = s_tmem + 256;
  const int d = P.c.head_dim;
  const float* s_sc = reinterpret_cast<const float*>(smem + L::sc);
  uint32_t s_phase = 0u;
  Ring sr;
  while (c.left > 0) {
    const int t_begin = c.tile;
    const int n = static_cast<int>(min(static_cast<int64_t>(c.k.tiles - c.tile), c.left));
    const bool whole = n == c.k.tiles;
    if (t == 1 && c.k.rows <= kTileRows) {  // nothing for this tile
      for (int j = 0; j < n; ++j) sr.next(L::kSc);
      c.left -= n;
      if (c.left > 0) next_block(P, c, unit_shape());
      continue;
    }
    const int row = t * kTileRows + tid;  // of the block
    const int tok = (c.k.row0 + row) / P.group, g = c.k.row0 + row - tok * P.group;
    const int64_t j_row = c.q_off + tok;
    const int h = c.head * P.group + g;
    const bool live = row < c.k.rows;
    const bool there = live && j_row < P.n_tokens;
    // ---- the row's query as NS e4m3 rows
    float factor;  // score (log2) of a product of codes
    {
      const uint16_t* src = P.q + j_row * P.q_ts + static_cast<int64_t>(h) * P.q_hs;
      float amax = 0.0f;
      if (there) {
        for (int i = 0; i < d; i += 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + i);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 y = Pair<T>::unpack(w[k]);
            amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
          }
        }
      }
      // To [128, 256) by a power of two.  A row that is not finite is a NaN
      // below whatever its unit.
      const int e = static_cast<int>(__float_as_uint(amax) >> 23);
      const float unit =
          e > 8 && e < 255 ? __uint_as_float(static_cast<uint32_t>(261 - e) << 23) : 1.0f;
      factor = fmaxf(fabsf(P.scale_log2) / unit, 1.17549435e-38f);  // -inf stays -inf
      const float sign = P.scale_log2 < 0.0f ? -unit : unit;
      uint8_t* q = smem + L::q + t * NS * kQBytes;
      for (int i = 0; i < d; i += 16) {
        uint32_t w[8];
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        if (there) {
          x = *reinterpret_cast<const uint4*>(src + i);
          y = *reinterpret_cast<const uint4*>(src + i + 8);
        }
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
        float v[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 z = Pair<T>::unpack(w[k]);
          v[2 * k] = z.x * sign;
          v[2 * k + 1] = z.y * sign;
          // The codes have no infinity.
          if (!isfinite(v[2 * k])) v[2 * k] = __uint_as_float(0x7fffffffu);
          if (!isfinite(v[2 * k + 1])) v[2 * k + 1] = __uint_as_float(0x7fffffffu);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a = e4m3x2(v[4 * k], v[4 * k + 1]), b = e4m3x2(v[4 * k + 2], v[4 * k + 3]);
            o[k] = a | (b << 16);
            const float2 ra = Pair<__half>::unpack(e4m3x2_to_f16x2(a));
            const float2 rb = Pair<__half>::unpack(e4m3x2_to_f16x2(b));
            v[4 * k] -= ra.x, v[4 * k + 1] -= ra.y, v[4 * k + 2] -= rb.x, v[4 * k + 3] -= rb.y;
          }
          *reinterpret_cast<uint4*>(q + s * kQBytes + chunk_at(tid, i >> 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc::fence_smem();
      tc::fence_before();
      mbar_arrive(&B->q_full[t]);
    }
    // Positions that this row sees, and those that all rows of the tile see.
    const int pos = c.r.cached + tok;
    int lo = c.r.begin;
    if (P.window > 0) lo = max(lo, pos - P.window + 1);
    const int hi = min(pos, c.k.end - 1);
    const int first_row = c.k.row0 + t * kTileRows;
    const int last_row = c.k.row0 + min(c.k.rows, (t + 1) * kTileRows) - 1;
    const int all_hi = min(c.r.cached + first_row / P.group, c.k.end - 1);
    int all_lo = c.r.begin;
    if (P.window > 0) all_lo = max(all_lo, c.r.cached + last_row / P.group - P.window + 1);

    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < n; ++j) {
      const int base = c.k.start + (t_begin + j) * kTile;
      wait(B, &B->s_full[t], s_phase);
      s_phase ^= 1u;
      tc::fence_after();
      // (After s_full, by when the scales are long there: a tile that skipped
      // blocks must not look at an earlier phase of this ring.)
      wait(B, &B->sc_full[sr.slot], sr.phase);
      const float4* sc = reinterpret_cast<const float4*>(s_sc + sr.slot * kTile);
      uint32_t u[kTile];
#pragma unroll
      for (int k = 0; k < 4; ++k) tc::ld32(s_tmem + 32 * k, u + 32 * k);
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < kTile / 4; ++k) {
        const float4 s4 = sc[k];
        const float2 x = unpack2(mul2(pack2(__uint_as_float(u[4 * k]), __uint_as_float(u[4 * k + 1])),
                                      pack2(s4.x, s4.y)));
        const float2 y = unpack2(mul2(pack2(__uint_as_float(u[4 * k + 2]), __uint_as_float(u[4 * k + 3])),
                                      pack2(s4.z, s4.w)));
        u[4 * k] = __float_as_uint(x.x), u[4 * k + 1] = __float_as_uint(x.y);
        u[4 * k + 2] = __float_as_uint(y.x), u[4 * k + 3] = __float_as_uint(y.y);
      }
      sr.next(L::kSc);
      if (base < all_lo || base + kTile - 1 > all_hi) {
        const int from = lo - base, to = hi - base;  // columns seen: [from, to]
#pragma unroll
        for (int k = 0; k < kTile; ++k)
          if (k < from || k > to) u[k] = 0xff800000u;
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < kTile; k += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top[i] = fmaxf(fmaxf(top[i], __uint_as_float(u[k + 2 * i])), __uint_as_float(u[k + 2 * i + 1]));
      }
      const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * factor;
      const bool rise = most > m + kLazy;
      if (__any_sync(kFull, rise)) {
        const float now = rise ? most : m;
        const float f = m == -INFINITY ? 0.0f : ex2(m - now);
        m = now;
        l *= f;
        if (j > 0) {
          for (int k = 0; k < d; k += 16) {
            uint32_t o[16];
            tc::ld16(o_tmem + k, o);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc::st16(o_tmem + k, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t f2 = pack2(factor, factor), r2 = pack2(-ref, -ref);
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = 32 * q + 2 * i;
          const float2 x = unpack2(
              fma2(pack2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), f2, r2));
          const float a = ex2(x.x), b = ex2(x.y);
          sum[i & 1] = add2(sum[i & 1], pack2(a, b));
          p[i] = Pair<__nv_bfloat16>::pack(a, b);
        }
        tc::st16(s_tmem + 16 * q, p);
      }
      const float2 s = unpack2(add2(sum[0], sum[1]));
      l += s.x + s.y;
      tc::wait_st();
      tc::fence_before();
      mbar_arrive(&B->p_full[t]);
    }
    // ---- the block's end: O is complete
    wait(B, &B->s_full[t], s_phase);
    s_phase ^= 1u;
    tc::fence_after();
    bool nan = *reinterpret_cast<volatile int*>(&B->nan) != 0;
    const int64_t out_at = j_row * P.o_ts + static_cast<int64_t>(h) * P.o_hs;
    // NaN codes of partly seen units were left out of the products.
    auto put_nans = [&](int k, float (&o)[16]) {
      for (int p = lo; p <= hi && p < c.k.end; ++p) {
        const int loc = P.page_table[c.r.table_row * P.pt_cols + p];
        if (loc < 0 || loc >= P.c.num_pages * P.c.page_size) continue;
        const int page = loc / P.c.page_size;
        const uint8_t* v = static_cast<const uint8_t*>(P.c.v) + page * P.c.page_stride +
                           (loc - page * P.c.page_size) * P.c.token_stride +
                           c.head * P.c.head_stride + k;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((v[i] & 0x7f) == 0x7f) o[i] = __uint_as_float(0x7fffffffu);
      }
    };
    auto store16 = [&](int k, const float (&o)[16], float inv) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = Pair<T>::pack(o[2 * i] * inv, o[2 * i + 1] * inv);
      uint4* dst = reinterpret_cast<uint4*>(P.out + out_at + k);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    };
    auto store_lse = [&](float mm, float ll) {
      if (P.lse != nullptr)
        P.lse[j_row * P.q_heads + h] = ll != 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    };
    if (whole) {
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      for (int k = 0; k < d; k += 16) {
        uint32_t r[16];
        tc::ld16(o_tmem + k, r);
        tc::wait_ld();
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = l != 0.0f ? __uint_as_float(r[i]) : 0.0f;
        if (there) {
          if (nan) put_nans(k, o);
          store16(k, o, inv);
        }
      }
      if (there) store_lse(m, l);
    } else {
      int64_t c0, c1;
      block_ctas(range, range.last - c.left - t_begin, c.k.tiles, &c0, &c1);
      const int64_t size = partial_floats(d);
      auto partial = [&](int64_t cta) {
        const int64_t at = (2 * cta + (cta == c0 ? 1 : 0)) * 2 + t;
        return P.partials + at * size;
      };
      float4* mine = reinterpret_cast<float4*>(partial(blockIdx.x));
      for (int k = 0; k < d; k += 16) {
        uint32_t r[16];
        tc::ld16(o_tmem + k, r);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __stcg(mine + (k / 4 + i) * kTileRows + tid,
                 make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                             __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])));
      }
      float2* stats = reinterpret_cast<float2*>(mine + (d / 4) * kTileRows);
      __stcg(stats + tid, make_float2(m, l));
      if (tid == 0) __stcg(stats + kTileRows, make_float2(nan ? 1.0f : 0.0f, 0.0f));
      __threadfence();
      bar_sync<2>(t);
      if (tid == 0) {
        uint32_t* counter = P.counters + 2 * c0 + t;
        const bool is_last = atomicAdd(counter, 1u) == static_cast<uint32_t>(c1 - c0);
        if (is_last) *counter = 0u;  // ready for the next call
        __threadfence();
        *reinterpret_cast<volatile int*>(&B->last[t]) = is_last ? 1 : 0;
      }
      bar_sync<2>(t);
      if (*reinterpret_cast<volatile int*>(&B->last[t]) != 0 && there) {
        // Joined in CTA order.
        auto stat_of = [&](int64_t cta, int i) {
          return __ldcg(
              reinterpret_cast<const float2*>(partial(cta) + static_cast<int64_t>(kTileRows) * d) + i);
        };
        auto stat = [&](int64_t cta) { return stat_of(cta, tid); };
        float mm = -INFINITY, ll = 0.0f;
        for (int64_t cta = c0; cta <= c1; ++cta) {
          mm = fmaxf(mm, stat(cta).x);
          nan = nan || stat_of(cta, kTileRows).x != 0.0f;
        }
        const float ref = mm == -INFINITY ? 0.0f : mm;
        for (int64_t cta = c0; cta <= c1; ++cta) {
          const float2 s = stat(cta);
          ll += s.y * ex2(s.x - ref);
        }
        const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
        for (int k = 0; k < d; k += 16) {
          float o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.0f;
          for (int64_t cta = c0; cta <= c1; ++cta) {
            const float2 s = stat(cta);
            if (s.y == 0.0f) continue;  // that part saw nothing
            const float f = ex2(s.x - ref);
            const float4* p = reinterpret_cast<const float4*>(partial(cta));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 x = __ldcg(p + (k / 4 + i) * kTileRows + tid);
              o[4 * i] = fmaf(x.x, f, o[4 * i]);
              o[4 * i + 1] = fmaf(x.y, f, o[4 * i + 1]);
              o[4 * i + 2] = fmaf(x.z, f, o[4 * i + 2]);
              o[4 * i + 3] = fmaf(x.w, f, o[4 * i + 3]);
            }
          }
          if (nan) put_nans(k, o);
          store16(k, o, inv);
        }
        store_lse(mm, ll);
      }
    }
    tc::fence_before();  // O is read; the next block's products may overwrite it
    c.left -= n;
    if (c.left > 0) next_block(P, c, unit_shape());
  }
}

// ------------------------------------------------------------------ kernel

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

template <typename T, int NS>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(
    const __grid_constant__ AttendParams P) {
  using L = Plan<NS>;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  Bars* B = reinterpret_cast<Bars*>(smem + L::bar);
  const int tid = threadIdx.x, warp = tid >> 5;
  Cursor c;
  const Range range = find_range<kThreads>(P, unit_shape(), smem, &c);
  if (c.left == 0) return;
  if (P.c.head_dim % 32 != 0) {
    // The last step of Q K^T sums over 32 elements: zeros past head_dim.
    for (int i = tid; i < (L::v - L::q) / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + L::q)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_smem();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kK; ++i) mbar_init(&B->k_full[i], 128), mbar_init(&B->k_empty[i], 1);
    for (int i = 0; i < L::kV; ++i) mbar_init(&B->v_full[i], 128), mbar_init(&B->v_empty[i], 1);
    for (int i = 0; i < L::kSc; ++i) mbar_init(&B->sc_full[i], 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->q_full[i], 128);
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->p_full[i], 128);
    }
    B->dead = 0;
    B->nan = 0;
    fence_mbar_init();
  }
  if (warp == 12) tc::alloc(&B->tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  // 512 threads of 128 registers: 2 * 176 + 104 + 56 = 4 * 128.
  if (warp < 8) {
    regs_up<176>();
    softmax_role<T, NS>(P, c, range, smem, B, warp >> 2);
  } else if (warp < 12) {
    regs_down<104>();
    load_role<NS>(P, c, smem, B);
  } else {
    regs_down<56>();
    if (tid == 12 * 32) mma_role<NS>(P, c, smem, B);
  }
  // Every product has been waited for (by the last block's softmax).
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 12) tc::dealloc(B->tmem, 512);
  if (tid == 0 && B->dead != 0 && P.status != nullptr) atomicOr(P.status, PKV_ST_TIMEOUT);
}

template <typename T, int NS>
cudaError_t launch(const AttendParams& P, int ctas, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0ull};
  const auto kernel = attend_tiles_kernel<T, NS>;
  const cudaError_t e = set_smem_limit_once(done, kernel, Plan<NS>::bytes);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kThreads, Plan<NS>::bytes, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

size_t tile_partial_bytes(int ctas, int head_dim) {
  return static_cast<size_t>(ctas) * 4 * partial_floats(head_dim) * 4;
}

cudaError_t launch_attend_tiles(const AttendParams& P, int ctas, cudaStream_t stream) {
  return P.bf16 ? launch<__nv_bfloat16, 2>(P, ctas, stream) : launch<__half, 3>(P, ctas, stream);
}

}  // namespace pkv
