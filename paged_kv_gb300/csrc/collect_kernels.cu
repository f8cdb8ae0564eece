// pkv_collect_pages and pkv_compact_pages: the free list of a pool whose pages rows
// may share, found by marking what live rows hold; and the same after the live pages
// have moved to the front.
//
// A page may be held by many rows, and nothing counts them: the table rows alone say
// what is held, so no count can be off after an aborted request.
//
// Kernels: (1) mark sets a bit for each held page; (2) list gives every page its rank
// among the held and the free ones by a popcount over the words before it (each
// CTA counts them all: a pool of 200 thousand pages has 25 KB of bits), and writes
// the free list, and for the moves the k-th page above and the k-th hole below the
// live count; (3) with moves, all SMs copy pages and rewrite table rows.
//
// Bound: collecting, its launches and one load after another; compacting, the moved
// pages' bytes.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pkv.h"
#include "api_common.h"
#include "device_common.cuh"
#include "launch_early.h"
#include "layer_pages.cuh"

namespace pkv {

namespace {

constexpr int kMarkThreads = 256;
constexpr int kListThreads = 512;
constexpr int kMoveWarps = 8;
constexpr int kCols = 256;  // columns of a piece of a table row

struct CollectParams {
  const int32_t* table_idx;
  const int32_t* lengths;
  const int32_t* page_table;
  int32_t* out_table;      // nullptr: nothing moves
  int32_t* free_slots;
  int64_t* count_out;      // or nullptr
  int32_t* status;         // or nullptr
  int32_t* head;           // workspace: [0] errors, [1] live pages, [2] moves; zeroed
  uint32_t* bits;          // workspace: [words], zeroed
  int32_t* turn;           // workspace: [num_pages], the number of a moving page, else -1
  int32_t* src;            // workspace: [num_pages]
  int32_t* dst;            // workspace: [num_pages]
  int64_t pt_rows, pt_cols, num_pages;
  Divider page_div;
  int B, page_size, words;
};

// One CTA row (blockIdx.y strides over them) and up to kMarkThreads of its pages.
__global__ void __launch_bounds__(kMarkThreads) mark_kernel(const __grid_constant__ CollectParams P) {
  const int ps = P.page_size;
  int bad = 0;
  for (int i = blockIdx.y; i < P.B; i += gridDim.y) {
    const int64_t row = P.table_idx[i];
    const int len = P.lengths[i];
    if (row < 0 || row >= P.pt_rows) {
      bad |= PKV_ST_ROW_OOB;
      continue;
    }
    if (len < 0 || len > P.pt_cols) {
      bad |= PKV_ST_COL_OOB;
      continue;
    }
    const int pages = static_cast<int>(div_ceil(len, ps));
    const bool inside = static_cast<int64_t>(pages) * ps <= P.pt_cols;
    if (P.out_table != nullptr && !inside) {
      bad |= PKV_ST_COL_OOB;
      continue;
    }
    const int32_t* at = P.page_table + row * P.pt_cols;
    for (int j = blockIdx.x * kMarkThreads + threadIdx.x; j < pages; j += gridDim.x * kMarkThreads) {
      const int loc = at[static_cast<int64_t>(j) * ps];
      const int page = loc < 0 ? -1 : static_cast<int>(P.page_div.divide(static_cast<uint32_t>(loc)));
      if (page < 0 || page >= P.num_pages || page * ps != loc) {
        bad |= PKV_ST_ROW_OOB;
        continue;
      }
      const uint32_t bit = 1u << (page & 31);
      if ((__ldcg(P.bits + (page >> 5)) & bit) == 0u) atomicOr(P.bits + (page >> 5), bit);
    }
  }
  if (bad != 0) atomicOr(P.head, bad);
}

template <bool MOVE>
__global__ void __launch_bounds__(kListThreads) list_kernel(const __grid_constant__ CollectParams P) {
  constexpr int kWarps = kListThreads / 32;
  __shared__ int s_warp[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  const int bad = *P.head;
  if (bad != 0) {
    if (blockIdx.x == 0 && tid == 0) {
      if (P.count_out != nullptr) *P.count_out = 0;
      if (P.status != nullptr) atomicOr(P.status, bad);
    }
    return;
  }
  auto block_sum = [&](int x) {
    x = __reduce_add_sync(kFull, x);
    __syncthreads();
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < kWarps; ++w) x += s_warp[w];
    return x;
  };
  // This CTA's words, and the held pages before them and in all.
  const int64_t each = div_ceil(P.words, gridDim.x);
  const int w0 = static_cast<int>(min(each * blockIdx.x, static_cast<int64_t>(P.words)));
  const int w1 = static_cast<int>(min(each * (blockIdx.x + 1), static_cast<int64_t>(P.words)));
  int before = 0, all = 0;
  for (int w = tid; w < P.words; w += kListThreads) {
    const int c = __popc(__ldcg(P.bits + w));
    all += c;
    if (w < w0) before += c;
  }
  before = block_sum(before);
  const int live = block_sum(all);
  // Held pages below `live`, where the moves' holes and pages part.
  int below = 0;
  if (MOVE) {
    for (int w = tid; w <= live >> 5 && w < P.words; w += kListThreads) {
      uint32_t x = __ldcg(P.bits + w);
      if (w == live >> 5) x &= (1u << (live & 31)) - 1u;
      below += __popc(x);
    }
    below = block_sum(below);
  }
  if (blockIdx.x == 0 && tid == 0) {
    P.head[1] = live;
    P.head[2] = live - below;
    if (P.count_out != nullptr) *P.count_out = P.num_pages - live;
  }
  const int64_t ps = P.page_size;
  if (MOVE) {
    const int64_t n = P.num_pages - live;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kListThreads + tid; i < n;
         i += static_cast<int64_t>(gridDim.x) * kListThreads)
      P.free_slots[i] = static_cast<int32_t>((live + i) * ps);
  }
  // A warp takes 32 words, then a page a lane, word by word.
  for (int v0 = w0; v0 < w1; v0 += kListThreads) {
    const int v = v0 + tid;
    const uint32_t word = v < w1 ? __ldcg(P.bits + v) : 0u;
    const int mine = __popc(word);
    const int incl = warp_inclusive_scan(mine, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int base = before;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += s_warp[w];
      before += s_warp[w];
    }
    const int first = base + incl - mine;  // held pages before word v
    for (int l = 0; l < 32; ++l) {
      const int at = v0 + warp * 32 + l;
      if (at >= w1) break;
      const uint32_t x = __shfl_sync(kFull, word, l);
      const int held = __shfl_sync(kFull, first, l) + __popc(x & ((1u << lane) - 1u));
      const int64_t page = static_cast<int64_t>(at) * 32 + lane;
      const bool is_held = (x >> lane) & 1u;
      if (page >= P.num_pages) continue;
      if (!MOVE) {
        if (!is_held) P.free_slots[page - held] = static_cast<int32_t>(page * ps);
      } else {
        const bool moves = is_held && page >= live;
        P.turn[page] = moves ? held - below : -1;
        if (moves) P.src[held - below] = static_cast<int32_t>(page);
        else if (!is_held && page < live) P.dst[page - held] = static_cast<int32_t>(page);
      }
    }
  }
}

__global__ void __launch_bounds__(kMoveWarps * 32, 3) move_kernel(
    const __grid_constant__ CollectParams P, const __grid_constant__ Layers L, const int pieces) {
  grid_dependency_wait();
  if (P.head[0] != 0) return;
  const int lane = threadIdx.x & 31, ps = P.page_size;
  const int live = P.head[1], moves = P.head[2];
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kMoveWarps;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  // Table rows first: they are short.
  const int parts = static_cast<int>(div_ceil(P.pt_cols, kCols));
  const bool same = P.out_table == P.page_table;
  for (int64_t i = me; i < static_cast<int64_t>(P.B) * parts; i += warps) {
    const int r = static_cast<int>(i / parts);
    const int c0 = static_cast<int>(i - static_cast<int64_t>(r) * parts) * kCols;
    const int held = static_cast<int>(div_ceil(P.lengths[r], ps)) * ps;
    if (c0 >= held) continue;
    const int64_t row = static_cast<int64_t>(P.table_idx[r]) * P.pt_cols + c0;
    constexpr int kEach = kCols / 32;
    // An entry's page, its turn to move and its new place: loads of all entries together.
    int loc[kEach], page[kEach], turn[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (j * 32 + lane < held - c0) loc[j] = P.page_table[row + j * 32 + lane];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      turn[j] = -1;
      if (j * 32 + lane < held - c0 && loc[j] >= 0) {
        // (An entry inside a page may be anything: only held pages have a turn.)
        page[j] = static_cast<int>(P.page_div.divide(static_cast<uint32_t>(loc[j])));
        if (page[j] >= live && page[j] < P.num_pages) turn[j] = P.turn[page[j]];
      }
    }
    int to[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (turn[j] >= 0) to[j] = P.dst[turn[j]];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (j * 32 + lane >= held - c0) continue;
      const int now = turn[j] >= 0 ? to[j] * ps + (loc[j] - page[j] * ps) : loc[j];
      if (!same || now != loc[j]) P.out_table[row + j * 32 + lane] = now;
    }
  }
  if (L.n == 0) return;
  // Whole pages where there are enough for all warps (a pool of 256 rows in 4 layers: 248 us,
  // by pieces 260), else pieces of them (4 conversations in 28 layers: 26 us, whole 33).
  const bool whole = static_cast<int64_t>(moves) * 2 * L.n >= warps;
  const int split = whole ? 1 : pieces, turns = whole ? pieces : 1;
  const int sides = 2 * L.n * split;
  // Part `at` of move k; the pages of the next one come while this one is copied.
  const int step_k = static_cast<int>(warps / sides), step_at = static_cast<int>(warps % sides);
  int64_t k = me / sides;
  int at = static_cast<int>(me % sides);
  int src = k < moves ? P.src[k] : 0, dst = k < moves ? P.dst[k] : 0;
  while (k < moves) {
    const int side = at / split, piece = at - side * split;
    const int from = src, to = dst;
    k += step_k, at += step_at;
    if (at >= sides) at -= sides, ++k;
    if (k < moves) src = P.src[k], dst = P.dst[k];
    for (int t = 0; t < turns; ++t)
      copy_page(L, side >> 1, side & 1, from, to, ps, piece + t);
  }
}

int64_t words_of(int64_t num_pages) { return div_ceil(num_pages, 32); }
// Workspace: 16 bytes of head, the bits, then turn, src and dst, each rounded to 16.
int64_t bits_bytes(int64_t num_pages) { return div_ceil(words_of(num_pages) * 4, 16) * 16; }
int64_t list_bytes(int64_t num_pages) { return div_ceil(num_pages * 4, 16) * 16; }

int collect(CollectParams P, const Layers& L, void* workspace, size_t workspace_bytes,
            pkv_stream_t stream) {
  if (P.B < 0 || P.B > PKV_MAX_FILL_BATCH)
    return fail(PKV_EINVAL, "B=%d outside [0, %d]", P.B, PKV_MAX_FILL_BATCH);
  if (P.page_size < 1) return fail(PKV_EINVAL, "page_size=%d < 1", P.page_size);
  if (P.num_pages < 1 || P.num_pages > INT32_MAX / P.page_size)
    return fail(PKV_EINVAL, "num_pages=%lld with page_size=%d: need 1 <= tokens < 2^31",
                (long long)P.num_pages, P.page_size);
  if (L.n > 0 && L.num_pages < P.num_pages)
    return fail(PKV_EINVAL, "num_pages=%lld, the caches have %lld", (long long)P.num_pages,
                (long long)L.num_pages);
  if (P.free_slots == nullptr ||
      (P.B > 0 && (P.table_idx == nullptr || P.lengths == nullptr || P.page_table == nullptr)))
    return fail(PKV_EINVAL, "NULL pointer argument");
  if (P.B > 0 && (P.pt_rows < 1 || P.pt_cols < 1 || P.pt_rows > INT32_MAX ||
                  P.pt_cols > (int64_t{1} << 30)))
    return fail(PKV_EINVAL, "page table shape [%lld, %lld]: need rows in [1, 2^31), columns in "
                "[1, 2^30]", (long long)P.pt_rows, (long long)P.pt_cols);
  const size_t table = static_cast<size_t>(P.pt_rows) * P.pt_cols * 4;
  if (P.B > 0 && P.out_table != P.page_table && P.out_table != nullptr &&
      overlap(P.page_table, table, P.out_table, table))
    return fail(PKV_EINVAL, "page_table and out_table overlap without being the same");
  const size_t need = pkv_collect_pages_workspace_bytes(P.num_pages);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PKV_EINVAL, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned16(workspace)) return fail(PKV_EINVAL, "workspace is not 16-byte aligned");
  uint8_t* at = static_cast<uint8_t*>(workspace);
  P.head = reinterpret_cast<int32_t*>(at);
  P.bits = reinterpret_cast<uint32_t*>(at + 16);
  at += 16 + bits_bytes(P.num_pages);
  P.turn = reinterpret_cast<int32_t*>(at);
  P.src = reinterpret_cast<int32_t*>(at + list_bytes(P.num_pages));
  P.dst = reinterpret_cast<int32_t*>(at + 2 * list_bytes(P.num_pages));
  P.words = static_cast<int>(words_of(P.num_pages));
  P.page_div = Divider::by(static_cast<uint32_t>(P.page_size));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(workspace, 0, 16 + bits_bytes(P.num_pages), s);
  if (e != cudaSuccess) return cuda_fail(e, "workspace reset");
  const int sms = num_sms();
  if (P.B > 0) {
    // Enough CTAs a row for two an SM, each with pages of its own.
    const int64_t most = std::max<int64_t>(1, div_ceil(div_ceil(P.pt_cols, P.page_size), kMarkThreads));
    const int64_t x = std::min<int64_t>(most, std::max<int64_t>(1, 2 * sms / P.B));
    mark_kernel<<<dim3(static_cast<unsigned>(x), static_cast<unsigned>(P.B)), kMarkThreads, 0, s>>>(P);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "mark launch");
  }
  const int64_t ctas = std::min<int64_t>(sms, div_ceil(P.words, 32));
  const bool move = P.out_table != nullptr && P.B > 0;
  e = launch_early(move ? list_kernel<true> : list_kernel<false>, dim3(static_cast<unsigned>(ctas)),
                   kListThreads, 0, s, P);
  if (e != cudaSuccess) return cuda_fail(e, "list launch");
  if (move) {
    e = launch_early(move_kernel, dim3(static_cast<unsigned>(sms) * 6), kMoveWarps * 32, 0, s, P, L,
                     page_pieces(L));
    if (e != cudaSuccess) return cuda_fail(e, "move launch");
  }
  return ok();
}

}  // namespace

}  // namespace pkv

extern "C" size_t pkv_collect_pages_workspace_bytes(int64_t num_pages) {
  using namespace pkv;
  if (num_pages < 1 || num_pages > INT32_MAX) return 0;
  return static_cast<size_t>(16 + bits_bytes(num_pages) + 3 * list_bytes(num_pages));
}

extern "C" int pkv_collect_pages(const int32_t* table_idx, const int32_t* lengths, int B,
                                 int page_size, int64_t num_pages, const int32_t* page_table,
                                 int64_t pt_rows, int64_t pt_cols, int32_t* free_slots,
                                 int64_t* count_out, int32_t* status, void* workspace,
                                 size_t workspace_bytes, pkv_stream_t stream) {
  using namespace pkv;
  CollectParams P = {};
  P.table_idx = table_idx, P.lengths = lengths, P.page_table = page_table;
  P.free_slots = free_slots;
  P.count_out = count_out;
  P.status = status;
  P.pt_rows = pt_rows, P.pt_cols = pt_cols, P.num_pages = num_pages;
  P.B = B, P.page_size = page_size;
  Layers L;
  L.n = 0, L.num_pages = 0;
  return collect(P, L, workspace, workspace_bytes, stream);
}

extern "C" int pkv_compact_pages(const int32_t* table_idx, const int32_t* lengths, int B,
                                 int page_size, int64_t num_pages, const int32_t* page_table,
                                 int64_t pt_rows, int64_t pt_cols, int32_t* out_table,
                                 int32_t* free_slots, int64_t* count_out,
                                 const pkv_kv_cache* layers, void* const* bounds, int n_layers,
                                 int32_t* status, void* workspace, size_t workspace_bytes,
                                 pkv_stream_t stream) {
  using namespace pkv;
  CollectParams P = {};
  P.table_idx = table_idx, P.lengths = lengths, P.page_table = page_table;
  P.out_table = out_table;
  P.free_slots = free_slots;
  P.count_out = count_out;
  P.status = status;
  P.pt_rows = pt_rows, P.pt_cols = pt_cols, P.num_pages = num_pages;
  P.B = B, P.page_size = page_size;
  if (out_table == nullptr && B > 0) return fail(PKV_EINVAL, "out_table is NULL");
  Layers L;
  const int bad = make_layers(layers, bounds, n_layers, page_size, &L);
  if (bad != PKV_OK) return bad;
  return collect(P, L, workspace, workspace_bytes, stream);
}
