// The n-th largest of many keys, by a CTA.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"

namespace pkv {

template <int THREADS>
struct NthScratch {
  uint32_t bins[2048];
  uint32_t scan[THREADS / 32];
  uint32_t prefix, left;
};

// The n-th largest (n >= 1) of the keys that each(f) hands to f in all threads, 0
// standing for none, by counting their upper 11 bits, the next 11 of those that
// share the first, and so on; with fewer than 3 rounds a lower bound of it, whose
// other bits are 0.  0 if there are fewer than n keys; *count is their number.
// Afterwards S.left is how many of the n have the same upper bits (after 3 rounds:
// are equal to it).  All threads of the CTA call it and get the result.
template <int THREADS, int ROUNDS, typename Each>
__device__ uint32_t nth_key(NthScratch<THREADS>& S, uint32_t n, uint32_t* count, Each&& each) {
  constexpr int kBins = 2048;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0, left = n;
  *count = 0;
#pragma unroll 1
  for (int round = 0; round < ROUNDS; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const uint32_t mask = round == 2 ? 1023u : 2047u;
    const uint32_t above = round == 0 ? 0u : round == 1 ? ~0u << 21 : ~0u << 10;
    for (int i = tid; i < kBins; i += THREADS) S.bins[i] = 0u;
    __syncthreads();
    each([&](uint32_t key) {
      if (key != 0u && (key & above) == prefix) atomicAdd(&S.bins[(key >> shift) & mask], 1u);
    });
    __syncthreads();
    // Thread t's bins, from the top: kBins - 1 - t kOwn and the kOwn - 1 below.
    constexpr int kOwn = kBins / THREADS;
    static_assert(kOwn * THREADS == kBins, "every bin is a thread's");
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own += S.bins[kBins - 1 - tid * kOwn - i];
    uint32_t incl = warp_inclusive_scan(own, lane);
    if (lane == 31) S.scan[warp] = incl;
    __syncthreads();
    uint32_t before = incl - own, total = 0;
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += S.scan[w];
      total += S.scan[w];
    }
    if (round == 0) {
      *count = total;
      if (total < n) {
        __syncthreads();
        return 0u;
      }
    }
    if (before < left && before + own >= left) {
      uint32_t c = before;
#pragma unroll 1
      for (int i = 0; i < kOwn; ++i) {
        const int bin = kBins - 1 - tid * kOwn - i;
        if (c + S.bins[bin] >= left) {
          S.prefix = prefix | static_cast<uint32_t>(bin) << shift;
          S.left = left - c;
          break;
        }
        c += S.bins[bin];
      }
    }
    __syncthreads();
    prefix = S.prefix;
    left = S.left;
    __syncthreads();
  }
  return prefix;
}

}  // namespace pkv
