// Attention of many query rows a request over the paged e4m3 cache: prompt
// chunks on the tensor cores.
//
// A unit (attend_units.cuh) is 128 positions for a block of up to 256 rows of
// one (request, cache head), held as two tiles of 128 rows.  Per unit and tile
//   S[128 x 128] = Q K^T   on kind::f8f6f4: K's codes go to the tensor core as
//     they are; a query row, scaled by a power of two, is the sum of NS rows of
//     8-bit codes: e4m3 (4 significant bits, which leave a signed rest of 4 bits
//     less), the last one e5m2, whose 3 bits hold what is left and reach down to
//     2^-16.  So 2 rows for bf16 and 3 for fp16 are the query exactly, but for
//     elements below 2^-13 (bf16) or 2^-10 (fp16) of a row's largest, which keep
//     an absolute 2^-21 of it;
//   S times the page's key scale and the row's factor, softmax in fp32;
//   O[128 x D] += P V      on kind::f16: V's codes made 16 bits wide (exactly) on
//     their way to shared memory, P = 2^(s - m) vs in tensor memory, in S's
//     place, with the page's value scale in it.  l sums 2^(s - m) in fp32.
// P and V take the queries' type.  bf16 (8 bits) has fp32's range: m is taken
// from a row's first columns, its weight 2^22, and moves only when weights pass
// 2^60.  fp16 (11 bits) is held below 2^15 with m's weight at 2^3, which keeps 11
// bits down to 2^-17 of that and some down to 2^-27.  m lies so (by 2^22) that
// l's terms of up to 2^22 / vs keep 2^-29 of the largest for a vs of 2^119; terms
// of small scales may pass 2^100 long before P's do, and move m too.  When m
// moves, O is rescaled in tensor memory by the row's own thread.  bf16 calls with
// weights in fp16 move m often: 2 x 4096 tokens take 546 us with them instead of
// 433, 48 short chunks 285 instead of 249.  (With bf16 weights the error against
// 64 bits is 0.0023; rounding the results to bf16 alone makes 0.0017.)
//
// Roles (16 warps): warps 0-3 and 4-7 are the softmax of tile 0 and 1, a
// thread a row; warps 8-11 bring V, converting it in registers; warp 12 issues
// the products; warps 13-15 look up the positions' places and scales and bring
// K by cp.async.  While one tile is in its softmax the other's products run.
//   k_full/k_empty, v_full/v_empty: rings of units in shared memory;
//   sc_full/sc_empty: places and scales;  q_full[t]: the block's queries;
//   s_full[t]: S is there, and O and P of the unit before are done with;
//   p_full[t]: P is there (and O rescaled), S may be overwritten.
// Products of one thread run in issue order, so P V and the next Q K^T of a
// tile, which writes over P, need no barrier between them.
//
// A block's start and end (queries to codes, results out) are rolled loops over
// whole rows, a half warp each: this code runs once in 10 to 50 units, and its
// fetch is what it costs (unrolled it is slower).
//
// Bound: neither the tensor pipe (2048 clocks a unit, 41 % busy) nor the
// exponentials (1024), but the chain S -> softmax -> P V of each tile, whose links
// wait for one another: a unit takes 3800 to 4200 clocks with both tiles in turn,
// and a block's change about 20000.  2 x 4096 tokens over 4096 cached, 16 query
// and 8 cache heads of 128, bf16: 433 us, 951 TFLOP/s, half of what a library
// product of that size reaches; 48 chunks of 1 to 512 tokens over up to 2000: 249
// us, 410 TFLOP/s.
//
// Every wait ends: after kWaitTries a thread sets `dead`, with which all waits
// return at once, the loops (whose lengths do not depend on data) run out, the
// products in flight are waited for (with a limit), tensor memory is freed and
// PKV_ST_TIMEOUT is set.

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
constexpr int kPlaceThreads = 96;
constexpr int kTileRows = 128;
constexpr int kBlockRows = 2 * kTileRows;
constexpr int kTile = 128;               // positions of a unit
constexpr int kPitch = 128;              // bytes of an 8-bit row in shared memory
constexpr int kQBytes = kTileRows * kPitch;
constexpr int kKBytes = kTile * kPitch;
constexpr int kVHalf = kTile * 128;      // 64 channels of bf16
constexpr int kVBytes = 2 * kVHalf;
// Cost of a block's start, in units: 48 prompt chunks of 1 to 512 tokens take
// 310 us with 0, 261 with 3, 257 with 6.
constexpr int kLead = 6;
constexpr int kPart = 32;                // columns a softmax thread has in registers
constexpr float kLn2 = 0.693147180559945309f;
// Least factor of a score whose product with a key scale (2^-64 and more) is
// normal, and fp32's least normal number, at which smaller products are held.
constexpr float kLeastFactor = 0x1p-62f, kTiny = 0x1p-126f;
constexpr int kWaitTries = 1 << 20;
__host__ __device__ constexpr UnitShape unit_shape() {
  return UnitShape{kBlockRows, kTile, kRowLimit + 1, INT32_MAX, 1, kLead};
}

// P and V are of the queries' type.  An entry of P is `unit` 2^(s - m) vs, and
// the sum of kPart of them may reach `limit` before m has to move.  m is the
// largest s + log2 vs - kRaise.  A unit adds up to 2^126 to l in bf16 (fp16's
// limit keeps it below 2^100): where l passes kSumLimit, m goes up by kStep.
constexpr float kRaise = 22.0f, kSumLimit = 0x1p100f, kStep = 64.0f;
template <typename W> struct Weight;
template <> struct Weight<__nv_bfloat16> {
  static constexpr float unit = 1.0f, limit = 0x1p60f;
  static constexpr int type = 1;
};
template <> struct Weight<__half> {
  static constexpr float unit = 0x1p-19f, limit = 0x1p15f;
  static constexpr int type = 0;
};

template <int NS>
struct Plan {
  static constexpr int kK = 3;                       // ring slots
  static constexpr int kV = NS == 2 ? 3 : 2;
  static constexpr int kSc = kK + 1;
  static constexpr int q = 0;
  static constexpr int k = q + 2 * NS * kQBytes;
  static constexpr int v = k + kK * kKBytes;
  static constexpr int sc = v + kV * kVBytes;        // scales, kSc slots: ks, lv, vs (above)
  static constexpr int gr = sc + kSc * 3 * kTile * 4;   // the same of each group of 16
  static constexpr int off = gr + kSc * 8 * 16;         // byte offsets
  static constexpr int bar = off + kSc * kTile * 8;
  static constexpr int bytes = bar + 512 + 1024;     // and room to align
};

struct Bars {
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3], sc_full[4], sc_empty[4];
  uint64_t q_full[2], s_full[2], p_full[2];
  uint32_t tmem;
  int dead;
  int last[2];
  int partial[4];
  int mixed[4][3];   // a group of 16 positions spans pages
  int nan;
  uint64_t drained;
};

static_assert(sizeof(Bars) <= 512, "its place in Plan");

// Phase bookkeeping of a ring.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) slot = 0, phase ^= 1u;
  }
};

// The rest of a wait: the hardware suspends the thread between tries.
__device__ __noinline__ void wait_more(Bars* B, uint64_t* bar, uint32_t parity) {
  for (int i = 0; !mbar_try_wait(bar, parity); ++i) {
    if (i == kWaitTries) *reinterpret_cast<volatile int*>(&B->dead) = 1;
    if (*reinterpret_cast<volatile int*>(&B->dead) != 0) break;
  }
}

// By whole warps, which leave it converged: what follows may be an instruction
// that all lanes have to issue together.
__device__ __forceinline__ void wait(Bars* B, uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  if (!__all_sync(kFull, ok != 0u)) wait_more(B, bar, parity);
  __syncwarp();
}

// As wait(), for up to three barriers at once: lane 0 looks at the first, lane
// 1 at the second, the others at the third.
__device__ __forceinline__ void wait3(Bars* B, uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                      uint64_t* c, uint32_t pc) {
  const int lane = threadIdx.x & 31;
  wait(B, lane == 0 ? a : lane == 1 ? b : c, lane == 0 ? pa : lane == 1 ? pb : pc);
}

// One arrival a warp (32 arrivals on one word would take their turns).
__device__ __forceinline__ void arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The 128 softmax threads of tile t.
__device__ __forceinline__ void tile_sync(int t) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(2 + t) : "memory");
}

__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// Three warps: finds the places of a unit's positions in the cache, two units
// ahead (unit J's table entries are read at J - 2, its scales at J - 1), and
// copies K.  A thread has positions tid and tid + 96 (below 128).
template <typename T, int NS>
__device__ __noinline__ void place_role(const AttendParams& P, Cursor a, uint8_t* smem, Bars* B) {
  using L = Plan<NS>;
  const int tid = threadIdx.x - 13 * 32;
  const int units = static_cast<int>(a.left);
  const int slots = static_cast<int>(P.c.num_pages * P.c.page_size);
  const int chunks = P.c.head_dim >> 4;
  float* s_sc = reinterpret_cast<float*>(smem + L::sc);
  float4* s_gr = reinterpret_cast<float4*>(smem + L::gr);
  int64_t* s_off = reinterpret_cast<int64_t*>(smem + L::off);
  constexpr int kPer = 2;
  const bool second = tid + kPlaceThreads < kTile;

  // A place outside the block's positions takes the nearest one's location, for
  // its scales alone; loc -1: outside the cache, or no position at all.
  struct Places { int loc[kPer]; bool in[kPer]; bool some, partial; int head; };
  int all_lo = 0, all_hi = 0;
  auto block_bounds = [&]() {  // positions that every row of the block sees
    const int t_first = a.k.row0 / P.group, t_last = (a.k.row0 + a.k.rows - 1) / P.group;
    all_lo = a.r.begin;
    if (P.window > 0) all_lo = max(all_lo, a.r.cached + t_last - P.window + 1);
    all_hi = min(a.r.cached + t_first, a.k.end - 1);
  };
  block_bounds();
  auto read_places = [&]() -> Places {
    Places p;
    p.loc[0] = p.loc[1] = -1;
    p.in[0] = p.in[1] = p.some = false;
    p.head = 0;
    p.partial = false;
    if (a.left > 0) {
      const int base = a.k.start + a.tile * kTile;
      const int32_t* row = P.page_table + a.r.table_row * P.pt_cols;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int tok = base + tid + i * kPlaceThreads;
        if (a.k.lo < a.k.end && (i == 0 || second)) {
          const int near = max(a.k.lo, min(tok, a.k.end - 1));
          p.in[i] = near == tok;
          p.some = true;
          p.loc[i] = row[near];  // not looked at before resolve()
        }
      }
      p.head = a.head;
      p.partial = base < all_lo || base + kTile - 1 > all_hi;
      --a.left;
      if (++a.tile >= a.k.tiles && a.left > 0) {
        next_block(P, a, unit_shape());
        block_bounds();
      }
    }
    return p;
  };
  float ks[kPer], vs[kPer];
  bool mixed = false;  // a group of this warp's positions spans pages
  auto resolve = [&](const Places& p, int slot) {  // byte offsets, and the scales' loads
    mixed = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      int64_t off = -1;
      int page = -1;
      ks[i] = 1.0f;  // (of a zero key; it must not turn a masked -inf into NaN)
      vs[i] = 0.0f;
      const bool mine = p.some && (i == 0 || second);
      if (mine && (p.loc[i] < 0 || p.loc[i] >= slots)) {
        if (P.status != nullptr) atomicOr(P.status, PKV_ST_ROW_OOB);
      } else if (mine) {
        page = static_cast<int>(P.page_div.divide(static_cast<uint32_t>(p.loc[i])));
        if (p.in[i])
          off = page * P.c.page_stride + (p.loc[i] - page * P.c.page_size) * P.c.token_stride +
                p.head * P.c.head_stride;
        const int64_t s = static_cast<int64_t>(page) * P.c.kv_heads + p.head;
        ks[i] = P.c.k_scale[s];
        vs[i] = P.c.v_scale[s];
      }
      if (i == 0 || second) {
        s_off[slot * kTile + tid + i * kPlaceThreads] = off;
        const int first = __shfl_sync(kFull, page, threadIdx.x & 16);  // whole warps
        mixed |= page != first;
      }
    }
    mixed = __any_sync(kFull, mixed);
    if (tid == 0) B->partial[slot] = p.partial ? 1 : 0;
  };
  Ring kr, er;                 // K slots; the place slots being reused
  er.slot = 1;
  Places ahead = read_places();
  resolve(ahead, 0);
  ahead = read_places();
  for (int u = 0; u < units; ++u) {
    const int slot = u % L::kSc, next = (u + 1) % L::kSc;
    float k0[kPer], v0[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) k0[i] = ks[i], v0[i] = vs[i];
    const bool m0 = mixed;
    if (u + 1 < units) {
      // The values' warps are done with it.  They alone: the softmax may still be
      // units behind, so what it reads (scales, mixed) is written further below.
      wait(B, &B->sc_empty[er.slot], er.phase ^ 1u);
      er.next(L::kSc);
      resolve(ahead, next);
      ahead = read_places();
    }
    // A unit kSc earlier is through its softmax once K's slot is free again.
    wait(B, &B->k_empty[kr.slot], kr.phase ^ 1u);
    if ((tid & 31) == 0) B->mixed[slot][tid >> 5] = m0 ? 1 : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i == 0 || second) {
        const int tok = tid + i * kPlaceThreads;
        float* at = s_sc + slot * 3 * kTile + tok;
        const float lv = lg2(fmaxf(v0[i], 0x1p-64f)) - kRaise;
        const float vw = v0[i] * Weight<T>::unit;
        at[0] = k0[i];
        at[kTile] = lv;
        at[2 * kTile] = vw;
        if ((tok & 15) == 0) s_gr[slot * 8 + (tok >> 4)] = make_float4(k0[i], lv, vw, 0.0f);
      }
    }
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kPlaceThreads) : "memory");
    arrive(&B->sc_full[slot]);
    const int64_t* offs = s_off + slot * kTile;
    const uint32_t kdst = smem_addr(smem + L::k + kr.slot * kKBytes);
    const int ch = tid & 7;
    if (ch < chunks) {
      const uint8_t* base = static_cast<const uint8_t*>(P.c.k) + ch * 16;
#pragma unroll
      for (int i = 0; i < (kTile + kPlaceThreads / 8 - 1) / (kPlaceThreads / 8); ++i) {
        const int t = (tid >> 3) + i * (kPlaceThreads / 8);
        if (t < kTile) {
          const int64_t off = offs[t];
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                       ::"r"(kdst + chunk_at(t, ch)), "l"(base + (off < 0 ? 0 : off)),
                       "r"(off < 0 ? 0 : 16) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (u > 0) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      tc::fence_smem();
      arrive(&B->k_full[kr.slot == 0 ? L::kK - 1 : kr.slot - 1]);
    }
    kr.next(L::kK);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  tc::fence_smem();
  arrive(&B->k_full[kr.slot == 0 ? L::kK - 1 : kr.slot - 1]);
}

// 16 codes to 16 values of 16 bits; exact.
template <typename T>
__device__ __forceinline__ void widen(const uint4& c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[2 * k] = e4m3x2_to_f16x2(w[k]);
    o[2 * k + 1] = e4m3x2_to_f16x2(w[k] >> 16);
  }
  if (Weight<T>::type == 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 x = Pair<__half>::unpack(o[k]);
      o[k] = Pair<T>::pack(x.x, x.y);
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Two fp16 values as 8-bit codes, to nearest.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Zeroes the NaN codes of a word; true if there were any.
__device__ __forceinline__ bool drop_nans(uint32_t& w) {
  const uint32_t hit = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
  w &= ~(hit * 255u);
  return hit != 0u;
}

// Four warps: V, a unit ahead in registers, made 16 bits wide on its way to
// shared memory.  A thread has 16 channels (one 16-byte chunk) of 8 positions.
template <typename T, int NS>
__device__ __noinline__ void value_role(const AttendParams& P, int units, uint8_t* smem, Bars* B) {
  using L = Plan<NS>;
  const int tid = threadIdx.x & 127;
  const int ch = tid & 7, t0 = tid >> 3;
  const bool mine = ch < (P.c.head_dim >> 4);
  const int64_t* s_off = reinterpret_cast<const int64_t*>(smem + L::off);
  const uint8_t* src = static_cast<const uint8_t*>(P.c.v) + ch * 16;
  // 32 bytes a position: chunks 2 (ch % 4) and the next of its half; the
  // halves' lanes store them in opposite order, so that a quarter warp covers
  // all banks.
  const int swap = ch >> 2;
  const uint32_t first = chunk_at(t0, (ch & 3) * 2 + swap) + (ch >> 2) * kVHalf;
  const uint32_t other = chunk_at(t0, (ch & 3) * 2 + 1 - swap) + (ch >> 2) * kVHalf;
  Ring vr, sr;
  auto load = [&](int u, uint4 (&raw)[8]) {
    wait(B, &B->sc_full[sr.slot], sr.phase);
    sr.next(L::kSc);
    const int64_t* offs = s_off + (u % L::kSc) * kTile + t0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t off = offs[16 * i];
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (off >= 0 && mine) raw[i] = __ldg(reinterpret_cast<const uint4*>(src + off));
    }
  };
  auto convert = [&](int u, uint4 (&raw)[8]) {
    const int slot = u % L::kSc;
    wait(B, &B->v_empty[vr.slot], vr.phase ^ 1u);
    if (B->partial[slot] != 0) {
      // A NaN that some row does not see: zero here, put back at the end.
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        nan |= drop_nans(raw[i].x);
        nan |= drop_nans(raw[i].y);
        nan |= drop_nans(raw[i].z);
        nan |= drop_nans(raw[i].w);
      }
      if (nan) *reinterpret_cast<volatile int*>(&B->nan) = 1;
    }
    uint8_t* dst = smem + L::v + vr.slot * kVBytes;
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 lo, hi;
        widen<T>(raw[i], lo, hi);
        // (16 positions on, the swizzle is the same.)
        *reinterpret_cast<uint4*>(dst + first + i * 16 * 128) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(dst + other + i * 16 * 128) = swap ? lo : hi;
      }
    }
    tc::fence_smem();
    arrive(&B->v_full[vr.slot]);
    arrive(&B->sc_empty[slot]);
    vr.next(L::kV);
  };
  uint4 r0[8], r1[8];
  load(0, r0);
  for (int u = 0; u < units; u += 2) {
    if (u + 1 < units) load(u + 1, r1);
    convert(u, r0);
    if (u + 1 < units) {
      if (u + 2 < units) load(u + 2, r0);
      convert(u + 1, r1);
    }
  }
}

// ------------------------------------------------------------------ products

// One whole warp, so that its operands stay in uniform registers; one elected
// lane issues.
template <typename T, int NS>
__device__ __noinline__ void mma_role(const AttendParams& P, Cursor c, uint8_t* smem, Bars* B) {
  using L = Plan<NS>;
  const uint32_t tmem = __shfl_sync(kFull, B->tmem, 0);
  const int ksteps = (P.c.head_dim + 31) >> 5;
  const uint32_t qk_instr = tc::instruction(0, 0, kTile, false);
  const uint32_t qk_last = tc::instruction(1, 0, kTile, false);  // e5m2 codes
  const uint32_t pv_instr =
      tc::instruction(Weight<T>::type, Weight<T>::type, P.c.head_dim, true);
  constexpr uint32_t kHi = tc::operand_hi(1024);
  const uint32_t q0 = tc::operand_lo(smem_addr(smem + L::q), 16);
  const uint32_t k0 = tc::operand_lo(smem_addr(smem + L::k), 16);
  const uint32_t v0 = tc::operand_lo(smem_addr(smem + L::v), kVHalf);
  Ring kr, vr;
  uint32_t q_phase = 0u, p_phase = 0u;  // bit t: tile t's
  auto qk = [&](int t) {
    const uint32_t kd = k0 + kr.slot * (kKBytes / 16), qd = q0 + t * (NS * kQBytes / 16);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < ksteps)
          tc::mma8_ss(tmem + t * kTile, qd + s * (kQBytes / 16) + 2 * k, kd + 2 * k, kHi,
                      s + 1 < NS ? qk_instr : qk_last, s + k > 0);
      }
    }
  };
  while (c.left > 0) {
    const int n = __shfl_sync(
        kFull, static_cast<int>(min(static_cast<int64_t>(c.k.tiles - c.tile), c.left)), 0);
    const int tiles = __shfl_sync(kFull, c.k.rows > kTileRows ? 2 : 1, 0);
    c.left -= n;
    if (c.left > 0) next_block(P, c, unit_shape());
    wait(B, &B->k_full[kr.slot], kr.phase);
    for (int t = 0; t < tiles; ++t) {
      wait(B, &B->q_full[t], (q_phase >> t) & 1u);
      q_phase ^= 1u << t;
      tc::fence_after();
      if (tc::elect()) {
        qk(t);
        tc::commit(&B->s_full[t]);
        mbar_arrive(&B->s_full[t]);
        if (t == tiles - 1) tc::commit(&B->k_empty[kr.slot]);
      }
      __syncwarp();
    }
    kr.next(L::kK);
    for (int j = 0; j < n; ++j) {
      const uint32_t vd = v0 + vr.slot * (kVBytes / 16);
      const bool more = j + 1 < n;
      for (int t = 0; t < tiles; ++t) {
        uint64_t* p = &B->p_full[t];
        const uint32_t phase = (p_phase >> t) & 1u;
        // (V, and K of the next unit where there is one.)
        wait3(B, p, phase, &B->v_full[vr.slot], vr.phase, more ? &B->k_full[kr.slot] : p,
              more ? kr.phase : phase);
        p_phase ^= 1u << t;
        tc::fence_after();
        if (tc::elect()) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            tc::mma16_ts(tmem + 256 + t * 128, tmem + t * kTile + 8 * k, vd + 128 * k, kHi, pv_instr,
                         j + k > 0);
          if (more) qk(t);
          tc::commit(&B->s_full[t]);
          mbar_arrive(&B->s_full[t]);
          if (t == tiles - 1) {
            tc::commit(&B->v_empty[vr.slot]);
            if (more) tc::commit(&B->k_empty[kr.slot]);
          }
        }
        __syncwarp();
      }
      vr.next(L::kV);
      if (more) kr.next(L::kK);
    }
  }
}

// Waits until all products that the warp has issued are done: before tensor
// memory is freed, after waits that ran out too.
__device__ __noinline__ void drain(Bars* B) {
  if (tc::elect()) tc::commit(&B->drained);
  __syncwarp();
  for (int i = 0; i < kWaitTries && !mbar_try_wait(&B->drained, 0u); ++i) {
  }
}

// ------------------------------------------------------------------ softmax

// Multiplies what a row has summed by f, when its reference moves: O (not yet
// there in a block's first unit) and the `done` columns of P that this unit has
// written.  (A function of its own, as are the rarer forms of the softmax
// below: the loop that runs for every unit stays small enough for the
// instruction caches.)
template <typename W>
__device__ __noinline__ void rescale(uint32_t o_tmem, int d, uint32_t p_tmem, int done, float f) {
  tc::wait_st();  // an earlier quarter of the unit has stored P, and perhaps O
#pragma unroll 1
  for (int k = 0; k < d; k += 32) {
    uint32_t o[32];
    tc::ld32(o_tmem + k, o);  // (past d: columns that nothing reads)
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tc::st32(o_tmem + k, o);
  }
#pragma unroll 1
  for (int k = 0; k < done; k += 16) {
    uint32_t p[16];
    tc::ld16(p_tmem + k, p);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = Pair<W>::unpack(p[i]);
      p[i] = Pair<W>::pack(x.x * f, x.y * f);
    }
    tc::st16(p_tmem + k, p);
  }
}

// The largest s + lv of kPart columns of a row, of those in [from, to].
template <bool GROUPS>
__device__ __noinline__ float highest(uint32_t s_tmem, const float* sc, const float4* gr, int from,
                                      int to, float factor) {
  uint32_t x[kPart];
  tc::ld32(s_tmem, x);
  float most = -INFINITY;
#pragma unroll
  for (int k = 0; k < kPart; ++k) {
    const float ks = GROUPS ? gr[k / 16].x : sc[k], lv = GROUPS ? gr[k / 16].y : sc[kTile + k];
    const float t = fmaf(__uint_as_float(x[k]), ks * factor, lv);
    if (k >= from && k <= to) most = fmaxf(most, t);
  }
  return most;
}

// One row's softmax of one unit: reads S, adds to l, leaves P in S's place.
// Columns outside [from, to] are not seen.  GROUPS: scales are the same over 16
// columns.  W: P's type.  TINY: ks * factor may leave fp32's range below.
//
// S goes through the registers kPart columns at a time (all 128 would not fit).
// The reference m is not the running maximum but one from the row's first
// columns, for as long as the weights under it stay below W's limit; their sum
// shows that, so no maximum is taken.  Where it is passed, m and what was
// summed under it move, and the columns are done again.
template <bool GROUPS, typename W, bool TINY = false>
__device__ __forceinline__ float2 softmax_unit(uint32_t s_tmem, uint32_t o_tmem, const float* sc,
                                               const float4* gr, int from, int to, float factor,
                                               int o_cols, float m, float l) {
#pragma unroll 1
  for (int q = 0; q < kTile / kPart; ++q) {
    uint32_t p[kPart / 2];
    uint64_t sum = 0ull;  // of the weights
    bool moved = false;
    for (;;) {
      uint32_t x[kPart];
      tc::ld32(s_tmem + kPart * q, x);
      if (__any_sync(kFull, from > 0 || to < kPart - 1)) {
#pragma unroll
        for (int k = 0; k < kPart; ++k)
          if (k < from || k > to) x[k] = 0xff800000u;
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t r2 = pack2(-ref, -ref);
      sum = 0ull;
      uint64_t held = 0ull;  // what P's entries sum to
#pragma unroll
      for (int g = 0; g < kPart / 16; ++g) {
        float4 scale;
        if (GROUPS) scale = gr[g];
        const float fg = scale.x * factor;
        const uint64_t fg2 = pack2(fg, fg), vg2 = pack2(scale.z, scale.z);
        uint64_t gsum = 0ull;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          uint64_t f = fg2, v = vg2;
          const int col = 16 * g + i;
          if (!GROUPS) {
            const float2 ks = *reinterpret_cast<const float2*>(sc + col);
            const float2 vs = *reinterpret_cast<const float2*>(sc + 2 * kTile + col);
            f = mul2(pack2(ks.x, ks.y), pack2(factor, factor));
            if (TINY) {  // (a column that is not seen stays at -inf)
              const float2 x = unpack2(f);
              f = pack2(fmaxf(x.x, kTiny), fmaxf(x.y, kTiny));
            }
            v = pack2(vs.x, vs.y);
          }
          const float2 a = unpack2(
              fma2(pack2(__uint_as_float(x[col]), __uint_as_float(x[col + 1])), f, r2));
          const uint64_t w = pack2(ex2(a.x), ex2(a.y));
          gsum = i == 0 ? w : add2(gsum, w);
          const uint64_t pw = mul2(w, v);
          if (!GROUPS) held = add2(held, pw);
          const float2 pa = unpack2(pw);
          p[col / 2] = Pair<W>::pack(pa.x, pa.y);
        }
        sum = g == 0 ? gsum : add2(sum, gsum);
        if (GROUPS) held = fma2(gsum, vg2, held);
      }
      const float2 h = unpack2(held);
      const bool past = !(h.x + h.y <= Weight<W>::limit) || m == -INFINITY;
      if (moved || !__any_sync(kFull, past)) break;
      const float most = highest<GROUPS>(s_tmem + kPart * q, sc, gr, from, to, factor);
      const float now = past ? fmaxf(m, most) : m;
      const float f = m == -INFINITY ? 0.0f : ex2(m - now);
      m = now;
      l *= f;
      rescale<W>(o_tmem, o_cols, s_tmem, kPart / 2 * q, f);
      moved = true;
    }
    tc::st16(s_tmem + kPart / 2 * q, p);  // over columns that have been read
    const float2 s = unpack2(sum);
    l += s.x + s.y;
    gr += kPart / 16;
    sc += kPart;
    from -= kPart, to -= kPart;
  }
  if (Weight<W>::type == 1) {
    const bool past = l > kSumLimit;
    if (__any_sync(kFull, past)) {
      const float f = past ? 0x1p-64f : 1.0f;
      if (past) m += kStep;
      l *= f;
      rescale<W>(o_tmem, o_cols, s_tmem, kTile / 2, f);
    }
  }
  return make_float2(m, l);
}

template <typename W>
__device__ __noinline__ float2 softmax_mixed(uint32_t s_tmem, uint32_t o_tmem, const float* sc,
                                             const float4* gr, int from, int to, float factor,
                                             int o_cols, float m, float l) {
  if (__any_sync(kFull, factor < kLeastFactor))
    return softmax_unit<false, W, true>(s_tmem, o_tmem, sc, gr, from, to, factor, o_cols, m, l);
  return softmax_unit<false, W>(s_tmem, o_tmem, sc, gr, from, to, factor, o_cols, m, l);
}

// What a block's units need of one softmax thread.
struct RowState {
  float m, l;
  uint32_t unit;      // units before this one in the CTA's range
  uint32_t s_phase;
};

// The softmax of one row over `n` units.
//   from, to: columns of the first unit that the row sees, going down by kTile
//   a unit;  tile: bit 0 the tile, bit 1 scales by groups may be used.
template <typename W>
__device__ __noinline__ RowState softmax_units(RowState r, Bars* B, const float* s_sc,
                                               const float4* s_gr, uint32_t s_tmem, uint32_t o_tmem,
                                               float factor, int d, int n, int from, int to,
                                               int tile) {
  const int t = tile & 1;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint32_t slot = r.unit % Plan<2>::kSc;
    wait(B, &B->s_full[t], r.s_phase);  // (and the unit's scales with it)
    r.s_phase ^= 1u;
    tc::fence_after();
    const float4* gr = s_gr + slot * 8;
    const int cols = j > 0 ? d : 0;
    const int* mixed = B->mixed[slot];
    const bool groups = (tile & 2) != 0 && (mixed[0] | mixed[1] | mixed[2]) == 0;
    const float2 ml =
        groups ? softmax_unit<true, W>(s_tmem, o_tmem, s_sc, gr, from, to, factor, cols, r.m, r.l)
               : softmax_mixed<W>(s_tmem, o_tmem, s_sc + slot * 3 * kTile, gr, from, to, factor, cols,
                                  r.m, r.l);
    r.m = ml.x;
    r.l = ml.y;
    tc::wait_st();
    tc::fence_before();
    arrive(&B->p_full[t]);
    ++r.unit;
    from -= kTile, to -= kTile;
  }
  return r;
}

template <typename T, int NS>
__device__ __noinline__ void softmax_role(const AttendParams& P, Cursor c, const Range& range,
                                          uint8_t* smem, Bars* B, int t) {
  using L = Plan<NS>;
  static_assert(L::kSc == Plan<2>::kSc, "one ring size");
  const int tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;  // tid: the row of the tile
  const int d = P.c.head_dim;
  const uint32_t lanes = B->tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const uint32_t s_tmem = lanes + t * kTile, o_tmem = s_tmem + 256;
  const float* s_sc = reinterpret_cast<const float*>(smem + L::sc);
  const float4* s_gr = reinterpret_cast<const float4*>(smem + L::gr);
  const int by_groups = P.c.page_size % 16 == 0 ? 2 : 0;
  RowState st{0.0f, 0.0f, 0u, 0u};
  while (c.left > 0) {
    const int t_begin = c.tile;
    const int n = static_cast<int>(min(static_cast<int64_t>(c.k.tiles - c.tile), c.left));
    const bool whole = n == c.k.tiles;
    if (t == 1 && c.k.rows <= kTileRows) {  // nothing for this tile
      st.unit += n;
      c.left -= n;
      if (c.left > 0) next_block(P, c, unit_shape());
      continue;
    }
    // This thread's row: its token and head.
    const uint32_t at = static_cast<uint32_t>(c.k.row0 + t * kTileRows + tid);
    const uint32_t tok = P.group_div.divide(at);
    const int64_t j_row = c.q_off + tok;
    const int head = c.head * P.group + static_cast<int>(at - tok * P.group);
    const bool live = t * kTileRows + tid < c.k.rows;
    const bool there = live && j_row < P.n_tokens;
    const uint32_t rows_there = __ballot_sync(kFull, there);
    uint8_t* q = smem + L::q + t * NS * kQBytes;
    // ---- the warp's queries, each as NS rows of codes.  They come as they are to
    // the place of their first two codes (32 rows of 128 bytes in each: a row's
    // first and second half) and are converted there.  A half warp has a row and
    // a lane 8 channels of it.  The loops are rolled: this code runs once a
    // block, and its fetch costs more than its instructions.
    float factor = 0.0f;  // of this thread's row: score (log2) of a product of codes
    const int half = lane >> 4, ch = lane & 15;
    uint8_t* const half_row = q + (ch >> 3) * kQBytes;
    {
      const uint32_t dst = smem_addr(half_row);
      const int64_t from = j_row * P.q_ts + static_cast<int64_t>(head) * P.q_hs;
#pragma unroll 4
      for (int i = half; i < 32; i += 2) {
        const int64_t off = __shfl_sync(kFull, from, i) + ch * 8;
        const bool mine = ((rows_there >> i) & 1u) != 0u && ch * 8 < d;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(dst + chunk_at(warp * 32 + i, ch & 7)), "l"(P.q + (mine ? off : 0)),
                     "r"(mine ? 16 : 0) : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      const bool store = ch * 8 < ((d + 31) & ~31);  // (zeros past d: Q K^T sums over 32s)
      const float sign = P.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int row = warp * 32 + 2 * i + half;
        const uint4 raw = *reinterpret_cast<const uint4*>(half_row + chunk_at(row, ch & 7));
        uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
        // The row's largest, as bits, so that a NaN is larger than all.
        uint32_t top = 0u;
#pragma unroll
        for (int n = 0; n < 4; ++n) top = __vmaxu2(top, x[n] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        // To [128, 256) by a power of two (2^126 at most).
        const int e = static_cast<int>(__float_as_uint(Pair<T>::unpack(top).x) >> 23);
        const float unit = top != 0u && e < 255  // (zeros: a row that is not there)
                               ? __uint_as_float(static_cast<uint32_t>(261 - max(e, 8)) << 23)
                               : 1.0f;
        const float f = __shfl_sync(kFull, unit, (lane & 1) * 16);  // (and all have read)
        if ((lane >> 1) == i) factor = f;
        // Not all codes have an infinity: a row that is not finite is NaNs (0x7f in
        // e4m3 and in e5m2).
        const uint32_t nans = e == 255 ? 0x7f7f7f7fu : 0u;
        // In fp16, whose 11 bits hold an element of either type and what is
        // left of it after each code exactly (down to 2^-24; e4m3 codes end at
        // 2^-9, e5m2 codes at 2^-16).
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float2 z = Pair<T>::unpack(x[n]);
          x[n] = Pair<__half>::pack(z.x * (unit * sign), z.y * (unit * sign));
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint32_t o[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            o[n] = s + 1 < NS ? e4m3x2_of_f16x2(x[n]) : e5m2x2_of_f16x2(x[n]);
            if (s + 1 < NS) x[n] = sub_f16x2(x[n], e4m3x2_to_f16x2(o[n]));
          }
          if (store)
            *reinterpret_cast<uint2*>(q + s * kQBytes + chunk_at(row, ch >> 1) + (ch & 1) * 8) =
                make_uint2((o[0] | (o[1] << 16)) | nans, (o[2] | (o[3] << 16)) | nans);
        }
      }
      factor = fabsf(P.scale_log2) / factor;
      tc::fence_smem();
      tc::fence_before();
      arrive(&B->q_full[t]);
    }
    // The positions that this thread's row sees.
    const int pos = c.r.cached + static_cast<int>(tok);
    int lo = c.r.begin, hi = min(pos, c.k.end - 1);
    if (P.window > 0) lo = max(lo, pos - P.window + 1);
    if (!live) lo = 0, hi = INT32_MAX;  // (never without an m)
    {
      const int base = c.k.start + t_begin * kTile;
      st.m = -INFINITY;
      st.l = 0.0f;
      const int how = __any_sync(kFull, factor < kLeastFactor) ? 0 : by_groups;
      st = softmax_units<T>(st, B, s_sc, s_gr, s_tmem, o_tmem, factor, d, n, lo - base, hi - base,
                            t + how);
    }
    // ---- the block's end: O is complete
    wait(B, &B->s_full[t], st.s_phase);
    st.s_phase ^= 1u;
    tc::fence_after();
    const float m = st.m, l = st.l;
    bool nan = *reinterpret_cast<volatile int*>(&B->nan) != 0;
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
    // Results go out by way of the queries' place, which is free: rows of 2 D
    // bytes, their first half in the first codes' rows of this warp and the
    // second in the second's.
    auto stage16 = [&](int k, const float (&o)[16], float inv) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = Pair<T>::pack(o[2 * i] * inv, o[2 * i + 1] * inv);
      uint8_t* dst = q + (k >> 6) * kQBytes;
      const int chunk = (k >> 3) & 7;
      *reinterpret_cast<uint4*>(dst + chunk_at(tid, chunk)) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + chunk_at(tid, chunk + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
    };
    auto store_rows = [&] {
      __syncwarp();
      const int64_t to = j_row * P.o_ts + static_cast<int64_t>(head) * P.o_hs;
#pragma unroll 4
      for (int i = half; i < 32; i += 2) {
        const int64_t off = __shfl_sync(kFull, to, i) + ch * 8;
        if (((rows_there >> i) & 1u) != 0u && ch * 8 < d)
          *reinterpret_cast<uint4*>(P.out + off) =
              *reinterpret_cast<const uint4*>(half_row + chunk_at(warp * 32 + i, ch & 7));
      }
    };
    auto store_lse = [&](float mm, float ll) {
      if (P.lse != nullptr)
        P.lse[j_row * P.q_heads + head] = ll != 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    };
    if (whole) {
      const float inv = l != 0.0f ? (1.0f / Weight<T>::unit) / l : 0.0f;
#pragma unroll 1
      for (int k = 0; k < d; k += 16) {
        uint32_t r[16];
        __syncwarp();
        tc::ld16(o_tmem + k, r);
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = l != 0.0f ? __uint_as_float(r[i]) : 0.0f;
        if (there && nan) put_nans(k, o);
        stage16(k, o, inv);
      }
      store_rows();
      if (there) store_lse(m, l);
    } else {
      int64_t c0, c1;
      block_workers(range, c, &c0, &c1);
      const int64_t size = partial_floats(d);
      auto partial = [&](int64_t cta) {
        const int64_t at = (2 * cta + (cta == c0 ? 1 : 0)) * 2 + t;
        return P.partials + at * size;
      };
      float4* mine = reinterpret_cast<float4*>(partial(blockIdx.x));
#pragma unroll 1
      for (int k = 0; k < d; k += 16) {
        uint32_t r[16];
        tc::ld16(o_tmem + k, r);
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
      tile_sync(t);
      if (tid == 0) {
        uint32_t* counter = P.counters + 2 * c0 + t;
        const bool is_last = atomicAdd(counter, 1u) == static_cast<uint32_t>(c1 - c0);
        if (is_last) *counter = 0u;  // ready for the next call
        __threadfence();
        *reinterpret_cast<volatile int*>(&B->last[t]) = is_last ? 1 : 0;
      }
      tile_sync(t);
      if (*reinterpret_cast<volatile int*>(&B->last[t]) != 0) {
        // Joined in CTA order.
        auto stat_of = [&](int64_t cta, int i) {
          return __ldcg(
              reinterpret_cast<const float2*>(partial(cta) + static_cast<int64_t>(kTileRows) * d) + i);
        };
        float mm = -INFINITY, ll = 0.0f;
#pragma unroll 2
        for (int64_t cta = c0; cta <= c1; ++cta) {
          mm = fmaxf(mm, stat_of(cta, tid).x);
          nan = nan || stat_of(cta, kTileRows).x != 0.0f;
        }
        const float ref = mm == -INFINITY ? 0.0f : mm;
#pragma unroll 2
        for (int64_t cta = c0; cta <= c1; ++cta) {
          const float2 s = stat_of(cta, tid);
          ll += s.y * ex2(s.x - ref);
        }
        const float inv = ll != 0.0f ? (1.0f / Weight<T>::unit) / ll : 0.0f;
#pragma unroll 1
        for (int k = 0; k < d; k += 32) {
          float o[2][16];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i >> 4][i & 15] = 0.0f;
#pragma unroll 2
          for (int64_t cta = c0; cta <= c1; ++cta) {
            const float2 s = stat_of(cta, tid);
            const float f = ex2(s.x - ref);
            const float4* p = reinterpret_cast<const float4*>(partial(cta)) + (k / 4) * kTileRows + tid;
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[i] = k + 4 * i < d ? __ldcg(p + i * kTileRows) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s.y == 0.0f) continue;  // that part saw nothing
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* to = &o[i >> 2][4 * (i & 3)];
              to[0] = fmaf(x[i].x, f, to[0]);
              to[1] = fmaf(x[i].y, f, to[1]);
              to[2] = fmaf(x[i].z, f, to[2]);
              to[3] = fmaf(x[i].w, f, to[3]);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (k + 16 * i >= d) break;
            if (nan && there) put_nans(k + 16 * i, o[i]);
            stage16(k + 16 * i, o[i], inv);
          }
        }
        store_rows();
        if (there) store_lse(mm, ll);
      }
    }
    __syncwarp();
    tc::fence_before();  // O is read; the next block's products may overwrite it
    c.left -= n;
    if (c.left > 0) next_block(P, c, unit_shape());
  }
}

// ------------------------------------------------------------------ kernel

template <typename T, int NS>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(
    const __grid_constant__ AttendParams P) {
  using L = Plan<NS>;
  launch_dependents();  // the row kernel's blocks may start beside these
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  Bars* B = reinterpret_cast<Bars*>(smem + L::bar);
  const int tid = threadIdx.x, warp = tid >> 5;
  Cursor c;
  const Range range = find_range<kThreads, 1>(P, unit_shape(), smem, &c);
  if (c.left == 0) return;
  if (P.c.head_dim % 32 != 0) {
    // The last step of Q K^T sums over 32 elements: zeros past head_dim.
    for (int i = tid; i < (L::v - L::q) / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + L::q)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_smem();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kK; ++i) mbar_init(&B->k_full[i], 3), mbar_init(&B->k_empty[i], 1);
    for (int i = 0; i < L::kV; ++i) mbar_init(&B->v_full[i], 4), mbar_init(&B->v_empty[i], 1);
    for (int i = 0; i < L::kSc; ++i) mbar_init(&B->sc_full[i], 3), mbar_init(&B->sc_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->q_full[i], 4);
      mbar_init(&B->s_full[i], 2);
      mbar_init(&B->p_full[i], 4);
    }
    mbar_init(&B->drained, 1);
    B->dead = 0;
    B->nan = 0;
    fence_mbar_init();
  }
  if (warp == 12) tc::alloc(&B->tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp < 8) {
    softmax_role<T, NS>(P, c, range, smem, B, warp >> 2);
  } else if (warp < 12) {
    value_role<T, NS>(P, static_cast<int>(c.left), smem, B);
  } else if (warp == 12) {
    mma_role<T, NS>(P, c, smem, B);
    drain(B);
  } else {
    place_role<T, NS>(P, c, smem, B);
  }
  __syncwarp();
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
