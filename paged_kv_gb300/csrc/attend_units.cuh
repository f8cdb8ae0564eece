// How the attention kernels cut a call into work units.
//
// The query rows of one (request, cache head) -- row = query token * group +
// query head in the group -- are cut into blocks of `rows`, the positions that
// a block sees into tiles of `tile`.  A unit is one tile of one block; a call's
// units are ordered by request, head, block, tile, and every worker (a CTA, or a
// warp) takes a contiguous range of them.  The ranges cost the same, where a
// unit costs one and the start of a block `lead` (its queries come, its results
// leave): many short blocks are as much work as one long one of more units.  A
// kernel takes only the requests whose row count lies in [min_rows, max_rows];
// others are another kernel's.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attend_params.h"
#include "device_common.cuh"

namespace pkv {

// The row kernel runs beside the tile kernel of its call: the first's blocks
// start when all of the second's have, wherever those leave room, and it ends
// only when the second has.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct UnitShape {
  int rows, tile;
  int min_rows, max_rows;
  int least;  // cost of a worker's range, where there is so much
  int lead;
};

// What the call asks of one request.
struct Request {
  int cached, table_row, begin;
  int q_len;       // query tokens, at most n_tokens
  int end;         // device_len where it can be read, 0 otherwise
  int bad;
};

__device__ __forceinline__ Request load_request(const AttendParams& P, int i) {
  Request r;
  const int c = P.cached_len[i], d = P.device_len[i];
  r.table_row = P.table_idx[i];
  r.begin = P.kv_begin != nullptr ? max(0, P.kv_begin[i]) : 0;
  const int64_t n = static_cast<int64_t>(d) - c;
  r.cached = c;
  r.q_len = static_cast<int>(max(int64_t{0}, min(n, P.n_tokens)));
  r.end = d;
  r.bad = 0;
  if (r.q_len > 0) {
    if (n > min(int64_t{P.max_q_len}, P.n_tokens)) r.bad |= PKV_ST_TOKEN_CAP;
    if (r.table_row < 0 || r.table_row >= P.pt_rows) r.bad |= PKV_ST_ROW_OOB;
    if (c < 0 || d > P.pt_cols) r.bad |= PKV_ST_COL_OOB;
    if (r.bad != 0) r.end = 0;
  }
  return r;
}

// One block of rows: rows [row0, row0 + rows) of one request and cache head,
// and the positions [lo, end) that any of them sees.  Tiles begin at `start`,
// the multiple of 16 at or below lo, so that groups of 16 positions lie within
// pages of a multiple of 16 tokens.
struct Block {
  int row0, rows, start, lo, end, tiles;
};

__device__ __forceinline__ Block make_block(const AttendParams& P, const Request& r, int b,
                                            const UnitShape& u) {
  Block k;
  k.row0 = b * u.rows;
  k.rows = min(u.rows, r.q_len * P.group - k.row0);
  const int t0 = k.row0 / P.group, t1 = (k.row0 + k.rows - 1) / P.group;
  int lo = r.begin;
  if (P.window > 0) lo = max(lo, r.cached + t0 - P.window + 1);
  k.lo = lo;
  k.start = lo & ~15;
  k.end = r.end == 0 ? lo : r.cached + t1 + 1;
  if (k.end < k.lo) k.end = k.lo;
  k.tiles = max(1, (k.end - k.start + u.tile - 1) / u.tile);
  return k;
}

// Blocks of one (request, cache head) that this kernel takes.
__device__ __forceinline__ int block_count(const AttendParams& P, const Request& r,
                                           const UnitShape& u) {
  const int n = r.q_len * P.group;  // (the host bounds n_tokens * q_heads by 2^31)
  if (n < u.min_rows || n > u.max_rows) return 0;
  return (n - 1) / u.rows + 1;
}

__device__ __forceinline__ int64_t request_cost(const AttendParams& P, const Request& r,
                                                 const UnitShape& u) {
  const int nb = block_count(P, r, u);
  int64_t cost = static_cast<int64_t>(nb) * u.lead;
  if (r.bad != 0) return (cost + nb) * P.c.kv_heads;  // (one empty tile a block)
  for (int b = 0; b < nb; ++b) cost += make_block(P, r, b, u).tiles;
  return cost * P.c.kv_heads;
}

// A place in the call's units: what a warp loads from or computes on.
struct Cursor {
  Request r;
  Block k;
  int64_t q_off;   // the request's first packed token
  int64_t left;    // units left in this worker's range
  int64_t cost;    // of everything before the block's first unit
  int req, head, block, tile;
};

// Goes to the next block.  Only called while units are left.
__device__ __forceinline__ void next_block(const AttendParams& P, Cursor& c, const UnitShape& u) {
  c.tile = 0;
  c.cost += c.k.tiles + u.lead;
  if (++c.block >= block_count(P, c.r, u)) {
    c.block = 0;
    if (++c.head >= P.c.kv_heads) {
      c.head = 0;
      do {
        c.q_off += c.r.q_len;
        ++c.req;
        if (c.req >= P.B) return;
        c.r = load_request(P, c.req);
      } while (block_count(P, c.r, u) == 0);
    }
  }
  c.k = make_block(P, c.r, c.block, u);
}

// A worker's (CTA's or warp's) range of the call's units.
struct Range {
  int64_t total;    // the call's cost
  int64_t workers;  // workers that it is cut for
};

// Finds this worker's range and sets *c to its first unit (c->left 0: none).
// A CTA has WORKERS of them (1, or one a warp).  All THREADS of the CTA take
// part; `scratch` is THREADS * 16 + 16 bytes of shared memory, free again on
// return.  Block 0 reports the requests' errors.
template <int THREADS, int WORKERS>
__device__ Range find_range(const AttendParams& P, const UnitShape& u, void* scratch, Cursor* c) {
  constexpr int kW = THREADS / 32;
  static_assert(WORKERS == 1 || WORKERS == kW, "a CTA's workers");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Cost and tokens before each thread's requests.
  long long* s_u = static_cast<long long*>(scratch);
  long long* s_t = s_u + THREADS;
  const int per = (P.B + THREADS - 1) / THREADS;
  const int i0 = min(P.B, tid * per), i1 = min(P.B, i0 + per);
  long long units = 0, toks = 0;
  int bad = 0;
  for (int i = i0; i < i1; ++i) {
    const Request r = load_request(P, i);
    bad |= r.bad;
    units += request_cost(P, r, u);
    toks += r.q_len;
  }
  long long ui = units, ti = toks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(kFull, ui, o), b = __shfl_up_sync(kFull, ti, o);
    if (lane >= o) ui += a, ti += b;
  }
  if (lane == 31) s_u[warp] = ui, s_t[warp] = ti;
  __syncthreads();
  long long ubase = ui - units, tbase = ti - toks, total = 0, ntok = 0;
#pragma unroll 1
  for (int w = 0; w < kW; ++w) {
    if (w < warp) ubase += s_u[w], tbase += s_t[w];
    total += s_u[w], ntok += s_t[w];
  }
  __syncthreads();
  s_u[tid] = ubase;
  s_t[tid] = tbase;
  if (blockIdx.x == 0 && P.status != nullptr) {
    if (tid == 0 && ntok > P.n_tokens) bad |= PKV_ST_TOKEN_CAP;
    if (bad != 0) atomicOr(P.status, bad);
  }
  __syncthreads();
  Range g;
  g.total = total;
  g.workers = min(static_cast<long long>(gridDim.x) * WORKERS, (total + u.least - 1) / u.least);
  c->left = 0;
  const long long me = static_cast<long long>(blockIdx.x) * WORKERS + (WORKERS == 1 ? 0 : warp);
  if (me < g.workers) {
    const long long first = me * total / g.workers;
    const long long last = (me + 1) * total / g.workers;
    // The last thread whose requests begin at or before `first` (threads
    // without units begin where the next one does, and are passed over).
    int k = 0;
#pragma unroll 1
    for (int t = lane; t < THREADS; t += 32) {
      if (s_u[t] <= first) k = t;
    }
    k = __reduce_max_sync(kFull, k);
    long long at = first - s_u[k];
    c->q_off = s_t[k];
    c->req = k * per;
    for (;;) {
      c->r = load_request(P, c->req);
      const long long n = request_cost(P, c->r, u);
      if (at < n) {
        const long long per_head = n / P.c.kv_heads;
        c->head = static_cast<int>(at / per_head);
        at -= c->head * per_head;
        break;
      }
      at -= n;
      c->q_off += c->r.q_len;
      ++c->req;
    }
    c->block = 0;
    if (c->r.bad != 0) {
      c->block = static_cast<int>(at / (1 + u.lead));
      at -= static_cast<long long>(c->block) * (1 + u.lead);
    }
    for (;;) {
      c->k = make_block(P, c->r, c->block, u);
      if (at < c->k.tiles + u.lead) break;
      at -= c->k.tiles + u.lead;
      ++c->block;
    }
    c->cost = first - at + u.lead;
    c->tile = max(0, static_cast<int>(at) - u.lead);
    // The range's units.
    Cursor n = *c;
    long long rest = last - c->cost;
    while (n.tile < rest) {
      const long long here = min(static_cast<long long>(n.k.tiles), rest);
      c->left += here - n.tile;
      rest -= n.k.tiles + u.lead;
      if (rest <= 0) break;
      next_block(P, n, u);
    }
  }
  __syncthreads();
  return g;
}

// The workers that hold the first and the last unit of the cursor's block.
__device__ __forceinline__ void block_workers(const Range& g, const Cursor& c, int64_t* c0,
                                              int64_t* c1) {
  *c0 = ((c.cost + 1) * g.workers - 1) / g.total;
  *c1 = ((c.cost + c.k.tiles) * g.workers - 1) / g.total;
}

}  // namespace pkv
