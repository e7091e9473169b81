// Unevaluated pairs of float32 (T. J. Dekker, "A floating-point technique for extending the available
// precision", 1971; D. E. Knuth's two-sum): some 45 bits for the scalars of a row.  float64 units are 64 times
// scarcer than float32 on this chip, so that a block-wide float64 sum costs as much as streaming a short row.
#pragma once

#include "common.cuh"
#include "weight.cuh"

#ifdef __CUDACC__
namespace specv {

struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

// |a| >= |b| or a = 0
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}

__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const Pair s = two_sum(a.hi, b.hi);
  return fast_two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

__device__ __forceinline__ Pair operator-(const Pair& a) { return Pair{-a.hi, -a.lo}; }
__device__ __forceinline__ Pair operator-(const Pair& a, const Pair& b) { return a + -b; }

__device__ __forceinline__ Pair operator*(const Pair& a, const Pair& b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return fast_two_sum(p, __fadd_rn(__fmaf_rn(a.hi, b.hi, -p), __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}

__device__ __forceinline__ Pair operator*(const Pair& a, float b) { return a * Pair{b, 0.f}; }

__device__ __forceinline__ float value(const Pair& a) { return __fadd_rn(a.hi, a.lo); }

// Not unrolled: code that runs once per row waits for its instructions, some 16 cycles each where it is laid out
// in a line (four unrolled sums of a warp took 13000 cycles in the distillation kernel).
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    v = v + Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
  return v;
}

// 2^y for |y| <= 0.51 to 2^-40, by the table (entry(j), j < 64) and polynomial of weight.cuh.
template <typename F>
__device__ __forceinline__ Pair exp2_near(float y, F&& entry) {
  const float k = __fmaf_rn(y, 64.f, 12582912.f);
  const int m = __float_as_int(k) - 0x4b400000;
  const float s = __fmaf_rn(__fsub_rn(k, 12582912.f), -0.015625f, y);
  const float scale = m < 0 ? 0.5f : 1.f;  // m in [-33, 33]
  const float2 t64 = entry(m & 63);
  const Pair T{t64.x * scale, t64.y * scale};
  const float t = __fmul_rn(s, kLn2Hi);
  const float tl = __fmaf_rn(s, kLn2Hi, -t) + __fmul_rn(s, kLn2Lo);
  const float q = __fmul_rn(__fmul_rn(t, t), __fmaf_rn(t, __fmaf_rn(t, 1.f / 24.f, 1.f / 6.f), 0.5f));
  return T + T * Pair{t, __fadd_rn(tl, q)};
}

// ln(s) of a positive normal s, by one thread of a warp (the table in constant memory, which serves one address at a
// time): s = 2^n f with f in [0.707, 1.414); y = log2(f) in float32, and what it misses,
// ln(f 2^-y) = d - d^2 / 2 with d = f 2^-y - 1 below 2^-21.
__device__ __forceinline__ Pair log_pair(const Pair& s) {
  const int n = ((__float_as_int(s.hi) - 0x3f3504f3) >> 23);
  // in two steps: 2^-n itself may be out of range
  const float down1 = __int_as_float((127 - n / 2) << 23), down2 = __int_as_float((127 - (n - n / 2)) << 23);
  const Pair f{s.hi * down1 * down2, s.lo * down1 * down2};
  const float y = log2f(f.hi);
  const Pair d = f * exp2_near(-y, [](int j) { return make_float2(kExp2Table.hi[j], kExp2Table.lo[j]); }) - Pair{1.f, 0.f};
  const float miss = __fadd_rn(d.hi, __fadd_rn(d.lo, -0.5f * d.hi * d.hi));
  return Pair{kLn2Hi, kLn2Lo} * static_cast<float>(n) + (Pair{kLn2Hi, kLn2Lo} * y + Pair{miss, 0.f});
}

}  // namespace specv
#endif  // __CUDACC__
