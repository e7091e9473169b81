// Selection by rank or by mass, shared by the threshold, filtered sampling and top-logit kernels:
// order-preserving keys of float32 logits, histograms of counts or of fixed-point masses in shared
// memory, and the search for the bin a running sum from the top ends in.
#pragma once

#include "common.cuh"

namespace specv {

constexpr int kBins = 2048;  // histogram bins: an 11-bit digit of a key, or distance bins

// Order-preserving key: a < b as floats iff key(a) < key(b); -0 is folded onto +0.
__device__ __forceinline__ uint32_t fkey(float f) {
  uint32_t u = __float_as_uint(f);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ unsigned long long warp_incl_u64(unsigned long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  return v;
}

struct Pick {
  int bin;                  // the bin holding the need-th unit from the top
  unsigned long long above; // units in the bins above it
  unsigned long long total; // units in every bin
};

// A histogram of 64-bit sums kept as three arrays of 32-bit words, bits 0-13, 14-27 and 28 up of every
// added value, so that every update is a 32-bit shared-memory atomic whose result is not waited for (a
// returned old value, needed to carry between two words, would stall each thread on every update).  With
// at most 2^18 adds of values below 2^60 per bin, none of the words can wrap: 2^18 (2^14 - 1) < 2^32, and
// the high words sum the values' bits 28 up.  mid and hi null: plain 32-bit counts.
struct Hist {
  unsigned int* lo;
  unsigned int* mid;
  unsigned int* hi;
  __device__ __forceinline__ unsigned long long get(int b) const {
    if (!mid) return lo[b];
    return (static_cast<unsigned long long>(hi[b]) << 28) + (static_cast<unsigned long long>(mid[b]) << 14) + lo[b];
  }
  __device__ __forceinline__ void add(int b, unsigned long long v) const {
    if (!mid) {
      atomicAdd(lo + b, static_cast<unsigned int>(v));
      return;
    }
    const unsigned int l = static_cast<unsigned int>(v) & 0x3fffu;
    const unsigned int m = static_cast<unsigned int>(v >> 14) & 0x3fffu;
    const unsigned int h = static_cast<unsigned int>(v >> 28);
    if (l) atomicAdd(lo + b, l);
    if (m) atomicAdd(mid + b, m);
    if (h) atomicAdd(hi + b, h);
  }
  template <int kThreads>
  __device__ __forceinline__ void zero(int nb) const {
    for (int k = threadIdx.x; k < nb; k += kThreads) {
      lo[k] = 0u;
      if (mid) {
        mid[k] = 0u;
        hi[k] = 0u;
      }
    }
    __syncthreads();
  }
};

// Over the nb bins of h read from the highest bin down: the bin where the running sum first reaches
// need (1 <= need <= total), the sum above that bin, and the total.  Every thread gets the result.
template <int kThreads, typename H>
__device__ Pick pick_from_top(const H& h, int nb, unsigned long long need, unsigned long long* wsum, Pick* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = nb / kThreads;  // bins per thread, thread 0 holding the highest
  unsigned long long local = 0;
  for (int j = 0; j < per; ++j) local += h.get(nb - 1 - (tid * per + j));
  const unsigned long long incl_w = warp_incl_u64(local, lane);
  if (lane == 31) wsum[warp] = incl_w;
  __syncthreads();
  unsigned long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const unsigned long long incl = before + incl_w;
  const unsigned long long excl = incl - local;
  if (excl < need && need <= incl) {
    unsigned long long run = excl;
    for (int j = 0; j < per; ++j) {
      const int bin = nb - 1 - (tid * per + j);
      const unsigned long long v = h.get(bin);
      if (run + v >= need) {
        out->bin = bin;
        out->above = run;
        break;
      }
      run += v;
    }
  }
  if (tid == 0) out->total = total;
  __syncthreads();
  const Pick p = *out;
  __syncthreads();
  return p;
}

}  // namespace specv
