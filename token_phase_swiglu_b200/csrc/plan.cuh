// Splitting the work of a packed batch, whose lengths only the device knows,
// evenly over the CTAs: every CTA adds up the units of all sequences, takes its
// share [u0, u1) of them, and finds the sequence that holds its first unit.
#pragma once

#include "common.cuh"

namespace fmlp {

// Unit ranges [unit_begin(c), unit_begin(c + 1)) of `ctas` CTAs, and the CTA whose
// range holds unit u (ctas <= units, so that no range is empty).
__device__ __forceinline__ int64_t share_begin(int64_t c, int64_t ctas, int64_t units) {
  return c * units / ctas;
}
__device__ __forceinline__ int share_of(int64_t u, int64_t ctas, int64_t units) {
  return (int)(((u + 1) * ctas - 1) / units);
}

template <int kThreads>
struct UnitPlan {
  int64_t total;    // units of all sequences
  int64_t first_b;  // the sequence of this CTA's first unit,
  int64_t first_prefix;  // and the units before that sequence
  int64_t scan[kThreads / 32];
};

// Called by all kThreads threads of a CTA with sh.total zero (and visible).
// units_of(b, first): the units of sequence b; `first` is true once per sequence.
// Returns the number of CTAs that share the work; leaves u0 = u1 for the others.
template <int kThreads, typename F>
__device__ __forceinline__ int64_t plan_units(UnitPlan<kThreads>& sh, int64_t B, F units_of,
                                              int64_t& u0, int64_t& u1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t mine = 0, chunk0 = 0;
  for (int64_t b = threadIdx.x; b < B; b += kThreads) {
    const int64_t n = units_of(b, true);
    if (b == threadIdx.x) chunk0 = n;
    mine += n;
  }
  if (mine) atomicAdd((unsigned long long*)&sh.total, (unsigned long long)mine);
  __syncthreads();
  const int64_t total = sh.total, ctas = min((int64_t)gridDim.x, total);
  u0 = u1 = 0;
  if (blockIdx.x >= ctas) return ctas;
  u0 = share_begin(blockIdx.x, ctas, total);
  u1 = share_begin(blockIdx.x + 1, ctas, total);
  int64_t carry = 0;  // units of the blocks of sequences before
  for (int64_t b0 = 0; b0 < B && carry <= u0; b0 += kThreads) {
    const int64_t b = b0 + threadIdx.x;
    const int64_t n = b0 == 0 ? chunk0 : b < B ? units_of(b, false) : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    int64_t before = carry, all = carry;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh.scan[w];
      all += sh.scan[w];
    }
    const int64_t lo = before + incl - n;
    if (n && lo <= u0 && u0 < lo + n) {
      sh.first_b = b;
      sh.first_prefix = lo;
    }
    carry = all;
  }
  __syncthreads();
  return ctas;
}

}  // namespace fmlp
