// Softmax weights in fixed point: exp((l - M) / T) * 2^45 for a logit l <= M, rounded, within 2^-38 (of
// the largest weight, 1) and within 2^-34 of itself.  Sums of these are exact and independent of their
// order, and two of them compare as the real sums do unless those agree to some ten digits, so a token
// drawn or a nucleus cut next to a border is the one the definition gives.
//
// 2^y with y = (l - M) log2(e) / T is split as 2^n 2^(j/64) 2^s, |s| <= 1/128 (a table and a short
// polynomial, as P. T. P. Tang, "Table-driven implementation of the exponential function in IEEE
// floating-point arithmetic", ACM TOMS 15, 1989).  Every product whose rounding would show is carried as
// an unevaluated pair of float32 (T. J. Dekker, "A floating-point technique for extending the available
// precision", 1971): float64 units are 64 times scarcer than float32 on this chip.
#pragma once

#include "common.cuh"

namespace specv {

constexpr int kFixBits = 45;  // 2^18 weights of at most 1 sum to at most 2^63
// ln(2) as the float32 nearest to it and the rest
constexpr float kLn2Hi = 0.693147182464599609375f;
constexpr float kLn2Lo = -1.904654299957767e-09f;
// -87 log2(e), and the roundings of its product with a scale below that: weights below e^-87 are 0, and one of e^-87 itself
// (bfloat16 logits 21.75 apart at T = 1/4) is not
constexpr float kLowestLog2 = -125.51449f;

struct Exp2Table {
  float hi[64], lo[64];
};

// 2^(j/64) = sum_k (j ln2 / 64)^k / k! in double, as a float32 and the rest.
constexpr Exp2Table make_exp2_table() {
  Exp2Table t = {};
  for (int j = 0; j < 64; ++j) {
    const double x = j * (0.693147180559945309417232121458 / 64.0);
    double term = 1.0, sum = 1.0;
    for (int k = 1; k < 30; ++k) {
      term *= x / k;
      sum += term;
    }
    t.hi[j] = static_cast<float>(sum);
    t.lo[j] = static_cast<float>(sum - static_cast<double>(t.hi[j]));
  }
  return t;
}

#ifdef __CUDACC__
static __constant__ Exp2Table kExp2Table = make_exp2_table();

// The same in global memory, for loads of one entry per thread (constant memory serves one address at a time).
static __device__ const Exp2Table kExp2TableGlobal = make_exp2_table();

// Entry threadIdx.x of the table, for the first 64 threads to store into 64 float2 of shared memory.
__device__ __forceinline__ float2 exp2_table_entry() {
  return threadIdx.x < 64 ? make_float2(kExp2TableGlobal.hi[threadIdx.x], kExp2TableGlobal.lo[threadIdx.x])
                          : make_float2(0.f, 0.f);
}

struct Weight {
  float M;            // the row's largest logit
  float c_hi, c_lo;   // log2(e) / T
  const float2* tab;  // the table in shared memory

  __device__ __forceinline__ unsigned long long operator()(float l) const {
    // d + dl = l - M exactly
    const float d = __fsub_rn(l, M);
    const float bb = __fsub_rn(d, l);
    const float dl = __fadd_rn(__fsub_rn(l, __fsub_rn(d, bb)), __fsub_rn(-M, bb));
    const float y = __fmul_rn(d, c_hi);
    if (!(y >= kLowestLog2)) return 0ull;  // also l = -inf
    const float yl = __fmaf_rn(d, c_hi, -y) + __fmaf_rn(d, c_lo, __fmul_rn(dl, c_hi));
    // y = (64 n + j) / 64 + s; the add of 1.5 2^23 rounds to an integer in the low bits
    const float k = __fmaf_rn(y, 64.f, 12582912.f);
    const int m = __float_as_int(k) - 0x4b400000;
    const float s = __fmaf_rn(__fsub_rn(k, 12582912.f), -0.015625f, y);  // exact
    const float2 T = tab[m & 63];
    const int sh = -(m >> 6);
    if (sh > kFixBits + 1) return 0ull;
    // t + tl = (s + yl) ln 2, |t| < 0.0055; 2^(s + yl) = 1 + t + p
    const float t = __fmul_rn(s, kLn2Hi);
    const float tl = __fmaf_rn(s, kLn2Hi, -t) + __fmaf_rn(s, kLn2Lo, __fmul_rn(yl, kLn2Hi));
    const float q = __fmul_rn(__fmul_rn(t, t), __fmaf_rn(t, __fmaf_rn(t, 1.f / 24.f, 1.f / 6.f), 0.5f));
    const float p = __fadd_rn(tl, __fmaf_rn(t, tl, q));
    // a1 + lo = (T.x + T.y) (1 + t + p)
    const float a = __fmul_rn(T.x, t);
    const float al = __fmaf_rn(T.x, t, -a);
    const float b = __fadd_rn(al, __fmaf_rn(T.x, p, __fmaf_rn(T.y, t, T.y)));
    const float a1 = __fadd_rn(T.x, a);
    const float lo = __fadd_rn(__fsub_rn(a, __fsub_rn(a1, T.x)), b);
    // to 2^-45: the high part as a multiple of 2^-21 (exact), the rest rounded
    const float h = __fmaf_rn(a1, 2097152.f, 12582912.f);
    const float rest = __fadd_rn(__fmaf_rn(__fsub_rn(h, 12582912.f), -4.76837158203125e-07f, a1), lo);
    const long long fix = (static_cast<long long>(__float_as_int(h) - 0x4b400000) << (kFixBits - 21)) +
                          __float2int_rn(__fmul_rn(rest, 35184372088832.f));
    return sh == 0 ? static_cast<unsigned long long>(fix)
                   : (static_cast<unsigned long long>(fix) + (1ull << (sh - 1))) >> sh;
  }
};

// log2(e) / T as a pair of float32, T in [2^-64, 2^64]: an approximate quotient, and what its remainder and
// log2(e)'s own rest add.
__device__ __forceinline__ void weight_scale(float temperature, float& c_hi, float& c_lo) {
  const float inv = __fdividef(1.f, temperature);
  const float near = __fmul_rn(1.44269502162933349609375f, inv);
  const float rest =
      __fmul_rn(__fadd_rn(__fmaf_rn(-near, temperature, 1.44269502162933349609375f), 1.925963033500e-08f), inv);
  c_hi = __fadd_rn(near, rest);
  c_lo = __fsub_rn(rest, __fsub_rn(c_hi, near));
}

// ln(total / 2^45) of a sum of weights that holds a weight of 1, to float32 precision near 0 too.
__device__ __forceinline__ float log_weight(unsigned long long total) {
  return log1pf(__fmul_rn(__ull2float_rn(total - (1ull << kFixBits)), 2.842170943040401e-14f));
}

// floor(f * total) for f in [0, 1) (or -0), exactly; `rem` tells whether something was cut off.
__device__ __forceinline__ unsigned long long share_floor(float f, unsigned long long total, bool& rem) {
  const uint32_t bits = __float_as_uint(fabsf(f));
  const int e = static_cast<int>(bits >> 23);
  const unsigned long long m = e ? ((bits & 0x7fffffu) | 0x800000u) : (bits & 0x7fffffu);
  const int s = e ? 150 - e : 149;  // f = m 2^-s, s >= 24
  const unsigned long long hi = __umul64hi(total, m), lo = total * m;
  unsigned long long r;
  if (s < 64) {
    r = (hi << (64 - s)) | (lo >> s);
    rem = (lo & ((1ull << s) - 1)) != 0;
  } else if (s < 128) {
    r = s > 64 ? hi >> (s - 64) : hi;
    rem = lo != 0 || (s > 64 && (hi & ((1ull << (s - 64)) - 1)) != 0);
  } else {
    r = 0;
    rem = (hi | lo) != 0;
  }
  return r;
}
#endif  // __CUDACC__

}  // namespace specv
