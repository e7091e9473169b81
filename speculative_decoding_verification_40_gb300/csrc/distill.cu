// Distillation of a draft model from a teacher's top logits on sm_103a: loss, gradient, and both at once.
// The operations are specified in include/spec_verify.h.
//
// With z = s / T, lse = logsumexp(z) over the vocabulary and lse_rest the same over the tokens outside the
// row's record, p_i the record's probabilities, m their sum and r the teacher's mass outside it,
//   L       = sum_i p_i (ln p_i - z_i + lse) + r (ln r - lse_rest + lse)
//   dL/dz_j = (m + r) q_j - p_j            for a token of the record,
//             (m + r - r / Q_rest) q_j     for any other, Q_rest = exp(lse_rest - lse), q_j = exp(z_j - lse).
//
// A cluster of CTAs takes a row, each its slice, and reads it once.  Weights are 2^((s - R) log2(e) / T) with R the
// largest of the slice's first loads, so that nothing is rescaled on the way.  Where such references are far off
// (logits sorted upwards, masked runs, a student that gives the record all but 2^-60 of its mass), the sums are taken
// again, over the record and over the rest relative to the largest logit of each, so that neither leaves float32's
// range however far the two lie apart.  The tail is summed by itself, a bitmap of the record's tokens keeping them out (the whole sum less the record's would cancel
// for a student that agrees with its teacher).  For loss and gradient at once the slice stays in shared memory
// between the sums and the gradient: one read and one write of the row.
#include <atomic>
#include <cstddef>

#include "../../include/spec_verify.h"
#include "common.cuh"
#include "pair.cuh"
#include "row_bounds.cuh"
#include "row_kernels.h"
#include "softmax.cuh"

namespace specv {

namespace {

constexpr int kDT = 256;              // threads per CTA (of the most)
constexpr int kDW = kDT / 32;
constexpr int kDU = 4;                // vectors in flight per thread where the slice is not kept
constexpr int kDSplit = 8;            // CTAs per row (the portable cluster size)
constexpr int kMaxTop = SPEC_MAX_TOP;
// Bytes of a row that a CTA keeps at most while another doubling of the cluster helps: three CTAs per SM (2048 x 128256
// bf16: 254 us when four CTAs per SM, of half as much each, took 313).
constexpr int kKeepBytes = 70 * 1024;

// ---------------------------------------------------------------- gradients' types

template <typename T>
__device__ __forceinline__ T to_grad(float g);
template <>
__device__ __forceinline__ float to_grad<float>(float g) {
  return g;
}
template <>
__device__ __forceinline__ __nv_bfloat16 to_grad<__nv_bfloat16>(float g) {
  return __float2bfloat16_rn(g);
}

template <typename T>
__device__ __forceinline__ uint4 pack_grad(const float* g);
template <>
__device__ __forceinline__ uint4 pack_grad<float>(const float* g) {
  return make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
}
template <>
__device__ __forceinline__ uint4 pack_grad<__nv_bfloat16>(const float* g) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(g[2 * j], g[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- the record

// ln p of an entry is (v - base) / T - off: base 0 and off the teacher's log-sum-exp, or base the record's
// largest value and off the logarithm of its own sum.
struct Record {
  Pair inv_t, off;
  float base;
};

__device__ __forceinline__ Pair entry_log(const Record& rec, float v) {
  // past float32's range a pair is void (an infinity less itself); a float32 product says so
  const float far = __fmul_rn(v - rec.base, rec.inv_t.hi);
  return fabsf(far) < 1e38f ? two_sum(v, -rec.base) * rec.inv_t - rec.off : Pair{far, 0.f};
}

// exp(x) of a pair, to float32 precision of the result.
__device__ __forceinline__ float exp_pair(const Pair& x) {
  const float e = expf(x.hi);
  return fabsf(x.hi) < INFINITY ? __fmaf_rn(e, x.lo, e) : e;
}

// exp(x) of a pair to some 2^-38 of itself, by the table and polynomial of weight.cuh: the teacher's mass beyond the
// record is what these leave of 1.  In as few instructions as it takes, and only where there is a tail: short rows feel
// every instruction that runs once (captured calls of 640 x 1307 float32, record of 8, the gradient: 7.5 us, 7.0 with
// exp_pair; of 1614 x 1784 bf16, record of 44, the loss: 15.7, 15.5).
__device__ __forceinline__ Pair tail_probability(Pair x, const float2* tab) {
  const float y = __fmul_rn(x.hi, 1.44269502162933349609375f);
  if (!(fabsf(y) < 120.f)) return Pair{exp_pair(x), 0.f};
  const float yl = __fmaf_rn(x.hi, 1.44269502162933349609375f, -y) +
                   __fmaf_rn(x.hi, 1.925963033500e-08f, __fmul_rn(x.lo, 1.44269502162933349609375f));
  const float k = __fmaf_rn(y, 64.f, 12582912.f);  // y = (64 n + j) / 64 + s
  const int m = __float_as_int(k) - 0x4b400000;
  const float s = __fmaf_rn(__fsub_rn(k, 12582912.f), -0.015625f, y);
  const float2 T = tab[m & 63];
  const float t = __fmul_rn(s, kLn2Hi);  // 2^(s + yl) = 1 + t + p
  const float tl = __fmaf_rn(s, kLn2Hi, -t) + __fmaf_rn(s, kLn2Lo, __fmul_rn(yl, kLn2Hi));
  const float q = __fmul_rn(__fmul_rn(t, t), __fmaf_rn(t, __fmaf_rn(t, 1.f / 24.f, 1.f / 6.f), 0.5f));
  const float p = __fadd_rn(__fmaf_rn(t, tl, tl), q);
  const float a = __fmul_rn(T.x, t);  // (T.x + T.y) (1 + t + p)
  const float rest = __fmaf_rn(T.x, t, -a) + __fmaf_rn(T.x, p, __fmaf_rn(T.y, t, T.y));
  const Pair e = fast_two_sum(T.x, a);
  const float scale = __int_as_float((127 + (m >> 6)) << 23);
  return Pair{e.hi * scale, (e.lo + rest) * scale};
}

__device__ __forceinline__ Pair probability(const Pair& x, bool tail, const float2* tab) {
  return tail ? tail_probability(x, tab) : Pair{exp_pair(x), 0.f};
}

// The teacher's mass beyond the record, given the record's, its log-sum-exp and how far the student's own mass there lies
// below its whole (in the logarithm): what the rounding of a float32 log-sum-exp leaves (eight steps of 2^-24 of
// 1 + |lse|: its own, its logits', and those of a float32 sum) is none where the student has next to nothing there.
__device__ __forceinline__ float beyond(const Pair& mass, float lse, float gap) {
  const float tail = fmaxf(0.f, value(Pair{1.f, 0.f} - mass));
  return gap > 60.f && tail <= __fmul_rn(4.76837158e-7f, 1.f + fabsf(lse)) ? 0.f : tail;
}

template <int kT>
__device__ __forceinline__ Pair block_sum(Pair v, Pair* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  Pair t = part[0];
#pragma unroll 1
  for (int w = 1; w < kT / 32; ++w) t = t + part[w];
  __syncthreads();
  return t;
}

template <int kT>
__device__ __forceinline__ float block_max(float m, float* red) {
  m = warp_max_nan(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int w = 1; w < kT / 32; ++w) m = max_nan(m, red[w]);
  __syncthreads();
  return m;
}

// The shift of the record's logarithms; *bad is set where the record has none.
template <int kT>
__device__ Record read_record(const DistillParams& p, int r, float teacher_lse, float* red, Pair* part, int* bad) {
  Record rec;
  rec.inv_t = Pair{p.inv_t, p.inv_t_rest};
  rec.base = 0.f;
  rec.off = Pair{0.f, 0.f};
  if (p.teacher_lse) {
    rec.off.hi = teacher_lse;
    *bad |= !(fabsf(rec.off.hi) < INFINITY);
    return rec;
  }
  const int32_t* ids = p.ids + static_cast<size_t>(r) * p.K;
  const float* values = p.values + static_cast<size_t>(r) * p.K;
  float top = -INFINITY;
  for (int k = threadIdx.x; k < p.K; k += kT)
    if (ids[k] != -1) top = max_nan(top, values[k]);
  rec.base = block_max<kT>(top, red);
  *bad |= !(fabsf(rec.base) < INFINITY);  // nothing to renormalise, or nothing to go by
  Pair s{0.f, 0.f};
  for (int k = threadIdx.x; k < p.K; k += kT)
    if (ids[k] >= 0 && values[k] > -INFINITY) s = s + Pair{exp_pair(entry_log(rec, values[k])), 0.f};
  rec.off = log_pair(block_sum<kT>(s, part));
  return rec;
}

// ---------------------------------------------------------------- slices

// What a CTA takes of a row: vectors [v0, v1) of the nv in its 16-byte aligned body; the first CTA also the
// elements before the body, the last one those after it.
template <typename T>
struct Slice {
  static constexpr int kV = Elems<T>::kVec;
  int head, nv, per, v0, v1;
  bool first, last;

  // split is a power of two
  __device__ __forceinline__ Slice(const T* row, int V, int rank, int split) {
    const int past = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T));
    head = past ? min(V, kV - past) : 0;
    nv = (V - head) / kV;
    per = (nv + split - 1) >> (__ffs(split) - 1);
    v0 = min(nv, rank * per);
    v1 = min(nv, v0 + per);
    first = rank == 0;
    last = rank == split - 1;
  }
  // bit of a token in the slice's bitmap (its vectors' elements, then up to 8 before and 8 after the body); -1
  // for a token of another slice
  __device__ __forceinline__ int bit(int id) const {
    const int b = id - head;
    if (b < 0) return first ? per * kV + id : -1;
    if (b >= nv * kV) return last ? per * kV + 8 + b - nv * kV : -1;
    return b >= v0 * kV && b < v1 * kV ? b - v0 * kV : -1;
  }
};

// Threads per CTA.  The code that runs once per warp and row is half of the loss's instructions at 32000 logits a row,
// so fewer warps with more logits each gain (2304 x 128256 bf16: 105 us with 128 threads and eight CTAs per SM, 113
// with 256 and four; 2048 x 32128: 37, 44; 8 x 128256: 9.5, 8.5).  With the slice kept, shared memory leaves room
// for three CTAs only, and their warps have to hide the loads (2048 x 128256: 254 us with 256, 282 with 128).
__host__ __device__ constexpr int threads_of(bool grad) { return grad ? kDT : kDT / 2; }

// What a CTA tells the others of its cluster (pairs are stored as 8-byte vectors).
struct __align__(8) Part {
  Pair rest, top;       // weights of its tokens outside and inside the record, relative to its first loads' largest
                        // logit; in the second pass to the row's largest outside, and inside
  Pair mass, against;   // over its tokens of the record: sum of p, of p (ln p - (s - ref) / T)
  float ref;            // its first loads' largest logit; in the second pass the row's largest
  int flags;            // 1: a token twice, 2: a token with p > 0 has the student's logit -inf
  float out, in;        // its largest logits outside and inside (second pass only)
};

struct Shared {
  float red[kDW];
  float2 tab[64];                    // for the record's probabilities
  Pair part[4][kDW];
  int count[kMaxTop / 32];
  Part parts[kDSplit];
  float ref, ref_out, ref_in;        // the references of Part::against, rest and top
  float most, k_in, k_out;           // the largest of the references; what a weight is worth in the gradient
  int flags, again;
  int any;                           // the flags of the CTA's threads
};

// A token of the record that lies in this CTA's slice: its teacher's logit and probability, its student logit.
struct __align__(16) Entry {
  float v, p, l;
  int id;
};

static_assert(sizeof(Part) % 8 == 0 && offsetof(Shared, parts) % 8 == 0, "pairs of every CTA's part lie on 8 bytes");

__host__ __device__ constexpr int shared_bytes() { return (static_cast<int>(sizeof(Shared)) + 15) / 16 * 16; }

// Groups of kDU vectors of a thread of kT that a slice of n vectors has, in words of one bit each, and their bytes for
// the kT threads: which groups hold a token of the record.
__host__ __device__ inline int hit_words(int n, int threads) { return (n + 32 * kDU * threads - 1) / (32 * kDU * threads); }
__host__ __device__ inline int hit_bytes(int n, int threads) { return hit_words(n, threads) * threads * 4; }

// Bytes of the bitmap of a slice of `per` vectors of kV elements.
__host__ __device__ inline int bitmap_bytes(int per, int kV) { return (per * kV + 16 + 127) / 128 * 16; }

__host__ __device__ inline int entry_bytes(int K) { return (K * static_cast<int>(sizeof(Entry)) + 15) / 16 * 16; }

// exp(-x) of what the roundings of a scale miss: next to nothing but for logits of 10^4 T and more.
__device__ __forceinline__ Pair make_up(float x) {
  const bool little = fabsf(x) < 0.00195f;
  return Pair{little ? 1.f : fast_exp2(-1.44269502f * x), little ? __fmaf_rn(0.5f * x, x, -x) : 0.f};
}

// Weights 2^(s c + shift), shift the float32 nearest to -ref c: one FFMA and one exponential a logit.  They stand
// for 2^((s - ref) c) times e^miss, the product's own rounding, which is taken out of their sums.  Where the product is
// 2^31 and more (a small T, a mask by the type's lowest value), two logits next to ref are 2^64 apart in weight or one
// value, so that a power of two in the place of c that keeps the product exact, and any two apart by 2^512, says the
// same.
struct Scale {
  float c, shift, miss;
  __device__ __forceinline__ Scale(float c_, float ref) {
    c = c_;
    if (!(fabsf(__fmul_rn(ref, c)) < 2147483648.f))
      c = __uint_as_float((288u << 23) - (__float_as_uint(ref) & 0x7f800000u));  // 2^34 by ref's own power of two
    shift = -__fmul_rn(ref, c);
    miss = __fmul_rn(__fmaf_rn(ref, c, shift), kLn2Hi);
  }
  __device__ __forceinline__ float operator()(float s) const { return fast_exp2(__fmaf_rn(s, c, shift)); }
  __device__ __forceinline__ Pair clean(const Pair& sum) const { return sum * make_up(miss); }
};

// Adds the weights of a vector's elements outside the record (bits: which are in it) to acc, two at a time.
template <typename T>
__device__ __forceinline__ void vector_sum(const uint4& r, unsigned int bits, const Scale& w, unsigned long long& acc) {
  constexpr int kV = Elems<T>::kVec;
  float f[kV];
  Elems<T>::widen(r, f);
  if (bits == 0) {
    const unsigned long long c2 = pack2(w.c, w.c), shift2 = pack2(w.shift, w.shift);
#pragma unroll
    for (int j = 0; j < kV; j += 2) {
      float a, b;
      unpack2(fma2(pack2(f[j], f[j + 1]), c2, shift2), a, b);
      acc = add2(acc, pack2(fast_exp2(a), fast_exp2(b)));
    }
  } else {
    float some = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j) some += (bits >> j) & 1u ? 0.f : w(f[j]);
    acc = add2(acc, pack2(some, 0.f));
  }
}

// Starts the copy of a slice into shared memory: every thread the vectors that it will read itself, so that only
// its own copies have to be waited for.  The first kDU of each thread are a group of their own.
template <typename T, int kT>
__device__ __forceinline__ void keep_slice(const T* row, const Slice<T>& s, uint4* kept) {
  const uint4* r4 = reinterpret_cast<const uint4*>(row + s.head) + s.v0;
  const int n = s.v1 - s.v0;
  int v = threadIdx.x;
  auto copy = [&]() {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(kept + v)), "l"(r4 + v) : "memory");
  };
  for (int u = 0; u < kDU && v < n; ++u, v += kT) copy();
  asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 4
  for (; v < n; v += kT) copy();
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int kLeft>
__device__ __forceinline__ void kept_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Sums a slice: the weights outside the record.  kKept: from the slice in shared memory; else from global memory,
// r holding the thread's first loads.  hits: the groups of vectors (a bit each, this thread's words kT apart) that
// hold a token of the record; only those look into the bitmap (2304 x 128256 bf16: 98 us, 104 where every vector did).
template <typename T, int kT, bool kKept>
__device__ Pair sum_slice(const T* row, int V, const Slice<T>& s, const uint32_t* bits, const uint32_t* hits,
                          uint4 (&r)[kDU], const Scale& w, const uint4* kept) {
  constexpr int kV = Elems<T>::kVec;
  const uint4* r4 = reinterpret_cast<const uint4*>(row + s.head) + s.v0;
  const int tid = threadIdx.x, n = s.v1 - s.v0;
  Pair sum{0.f, 0.f};
  auto in_record = [&](int at) { return (bits[at * kV / 32] >> (at * kV % 32)) & ((1u << kV) - 1u); };
  uint32_t hit = 0;
#pragma unroll 1
  for (int g = 0, v = tid; (v & ~31) < n; ++g, v += kDU * kT) {  // (a warp's lanes stay together)
    if (g % 32 == 0) hit = hits[g / 32 * kT + tid];
    unsigned long long acc = 0ull;
    if ((v | 31) + (kDU - 1) * kT < n && !__any_sync(0xffffffffu, hit & 1u)) {
#pragma unroll
      for (int u = 0; u < kDU; ++u) vector_sum<T>(kKept ? kept[v + u * kT] : r[u], 0u, w, acc);
    } else {
#pragma unroll
      for (int u = 0; u < kDU; ++u) {
        const int at = v + u * kT;
        if (at < n) vector_sum<T>(kKept ? kept[at] : r[u], in_record(at), w, acc);
      }
    }
    hit >>= 1;
    float a, b;
    unpack2(acc, a, b);
    const Pair t = two_sum(sum.hi, a + b);
    sum = Pair{t.hi, sum.lo + t.lo};
    if (!kKept) {
      const int next = v + kDU * kT;
      if ((next | 31) + (kDU - 1) * kT < n) {
#pragma unroll
        for (int u = 0; u < kDU; ++u) r[u] = ldg_stream(r4 + next + u * kT);
      } else {
#pragma unroll
        for (int u = 0; u < kDU; ++u)
          if (next + u * kT < n) r[u] = ldg_stream(r4 + next + u * kT);
      }
    }
  }
  auto one = [&](int id, int bit) {
    if ((bits[bit >> 5] >> (bit & 31)) & 1u) return;
    const Pair t = two_sum(sum.hi, w(Elems<T>::one(row, id)));
    sum = Pair{t.hi, sum.lo + t.lo};
  };
  if (s.first && tid < s.head) one(tid, s.per * kV + tid);
  if (s.last && tid < V - s.head - s.nv * kV) one(s.head + s.nv * kV + tid, s.per * kV + 8 + tid);
  return sum;
}

template <typename T, int kT>
__device__ __forceinline__ void first_loads(const T* row, const Slice<T>& s, uint4 (&r)[kDU]) {
  const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
  const uint4* r4 = reinterpret_cast<const uint4*>(row + s.head) + s.v0;
#pragma unroll
  for (int u = 0; u < kDU; ++u) {
    const int at = threadIdx.x + u * kT;
    r[u] = at < s.v1 - s.v0 ? ldg_stream(r4 + at) : make_uint4(none, none, none, none);
  }
}

// out = 0 for a slice.
template <typename T, int kT>
__device__ void zero_slice(T* out, int V, const Slice<T>& s, bool vec) {
  constexpr int kV = Elems<T>::kVec;
  for (int v = s.v0 + threadIdx.x; v < s.v1; v += kT) {
    if (vec)
      reinterpret_cast<uint4*>(out + s.head)[v] = make_uint4(0u, 0u, 0u, 0u);
    else
      for (int j = 0; j < kV; ++j) out[s.head + v * kV + j] = to_grad<T>(0.f);
  }
  if (s.first && threadIdx.x < s.head) out[threadIdx.x] = to_grad<T>(0.f);
  const int after = s.head + s.nv * kV + threadIdx.x;
  if (s.last && after < V) out[after] = to_grad<T>(0.f);
}

// The gradients 2^(s c + shift) k of a vector, two at a time (f32x2).
template <typename T>
__device__ __forceinline__ void grad_vector(const uint4& r, T* body, int v, bool vec, float c, float shift, float k) {
  constexpr int kV = Elems<T>::kVec;
  const unsigned long long c2 = pack2(c, c), shift2 = pack2(shift, shift), k2 = pack2(k, k);
  float f[kV];
  Elems<T>::widen(r, f);
#pragma unroll
  for (int j = 0; j < kV; j += 2) {
    float a, b;
    unpack2(fma2(pack2(f[j], f[j + 1]), c2, shift2), a, b);
    unpack2(mul2(pack2(fast_exp2(a), fast_exp2(b)), k2), f[j], f[j + 1]);
  }
  if (vec) {
    reinterpret_cast<uint4*>(body)[v] = pack_grad<T>(f);
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) body[v * kV + j] = to_grad<T>(f[j]);
  }
}

// The elements of a slice outside the body.
template <typename T, typename F>
__device__ __forceinline__ void map_ends(const T* row, T* out, int V, const Slice<T>& s, F&& fn) {
  const int tid = threadIdx.x;
  if (s.first && tid < s.head) out[tid] = to_grad<T>(fn(Elems<T>::one(row, tid)));
  const int after = s.head + s.nv * Elems<T>::kVec + tid;
  if (s.last && after < V) out[after] = to_grad<T>(fn(Elems<T>::one(row, after)));
}

// ---------------------------------------------------------------- loss, and loss with gradient

// Where the first references are kept: the tail's sum at least kLeastRest, so that the weights that are 0 (below 2^-126)
// are nothing to it and its quotients stay in range; a slice's sums below kFarSum, so that its weights lose nothing to the step to
// the common reference, and a slice with mass of the record within kFarRef T of that, so that the loss's terms (some 45
// bits) lose no more than 2^-30 to the change of reference.
constexpr float kFarSum = 1073741824.f;  // 2^30
constexpr float kFarRef = 16384.f;
constexpr float kLeastRest = 8.6736174e-19f;  // 2^-60

__device__ __forceinline__ void dsmem_st_pair(uint32_t addr, const Pair& v) { dsmem_st_v2(addr, v.hi, v.lo); }
__device__ __forceinline__ void dsmem_st_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 2^((from - to) c): what a sum relative to `from` is worth relative to `to`.  (Nothing below float32's range: a pair
// of so large a difference is void.)
__device__ __forceinline__ float step(float from, float to, float c) {
  if ((from - to) * c < -150.f) return 0.f;
  const Pair y = two_sum(from, -to) * Pair{c, 0.f};
  const float e = exp2f(y.hi);
  return __fmaf_rn(e, y.lo * kLn2Hi, e);
}

// a + b, a = m x for the float32 factors m and x: a pair past float32's range is void, and the product stands for it.
__device__ __forceinline__ float shifted(float m, const Pair& x, const Pair& b) {
  const float far = __fmul_rn(m, x.hi);
  return fabsf(far) < INFINITY ? value(x * m + b) : far;
}

// The largest logits of a slice outside its record's tokens and of those tokens (NaN and +inf stand out), and from them,
// over the cluster, the row's; they become the references (sh.ref, sh.ref_out, sh.ref_in).  0: the row is invalid, 1:
// it has nothing but -inf outside the record, 2: the rest.  (A function of its own for its registers' sake.)
template <typename T, int kT>
__device__ __noinline__ int own_references(const T* row, int V, const uint32_t* bits, const Entry* entries, int n,
                                           int rank, int split, Shared& sh) {
  constexpr int kV = Elems<T>::kVec;
  const Slice<T> s(row, V, rank, split);
  const int tid = threadIdx.x;
  const uint4* r4 = reinterpret_cast<const uint4*>(row + s.head) + s.v0;
  float out = -INFINITY, in = -INFINITY;
  for (int v = tid; v < s.v1 - s.v0; v += kT) {
    const uint32_t listed = bits[v * kV / 32] >> (v * kV % 32);
    float f[kV];
    Elems<T>::widen(ldg_stream(r4 + v), f);
#pragma unroll
    for (int j = 0; j < kV; ++j) out = (listed >> j) & 1u ? out : max_nan(out, f[j]);
  }
  auto one = [&](int id, int bit) {
    if (!((bits[bit >> 5] >> (bit & 31)) & 1u)) out = max_nan(out, Elems<T>::one(row, id));
  };
  if (s.first && tid < s.head) one(tid, s.per * kV + tid);
  if (s.last && tid < V - s.head - s.nv * kV) one(s.head + s.nv * kV + tid, s.per * kV + 8 + tid);
  for (int i = tid; i < n; i += kT) in = max_nan(in, entries[i].l);
  out = block_max<kT>(out, sh.red);
  in = block_max<kT>(in, sh.red);
  if (tid < split) {
    const uint32_t mine = smem_addr(&sh), there = dsmem_map(mine, tid) - mine;
    dsmem_st_f32(there + smem_addr(&sh.parts[rank].out), out);
    dsmem_st_f32(there + smem_addr(&sh.parts[rank].in), in);
  }
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  for (int i = 0; i < split; ++i) {
    out = max_nan(out, sh.parts[i].out);
    in = max_nan(in, sh.parts[i].in);
  }
  const float most = max_nan(out, in);
  if (tid == 0) {
    sh.any = 0;
    sh.ref = most;
    sh.ref_out = out > -INFINITY ? out : most;  // (nothing is there to be summed)
    sh.ref_in = in > -INFINITY ? in : most;
  }
  __syncthreads();
  return !(fabsf(most) < INFINITY) ? 0 : out > -INFINITY ? 2 : 1;
}

// Of a first pass without any weight outside the record (less than V 2^-126 to the record's 2^-20: e^-60 and less):
// whether the teacher has no mass there either, so that nothing more has to be known (both models' vocabularies
// constrained alike: 2304 x 128256 bf16 108 us, 238 with a second pass).
__device__ __noinline__ bool nothing_beyond(const DistillParams& p, int r, const Shared& sh, int split, float most,
                                            float c) {
  Pair mass{0.f, 0.f};
  float top = 0.f;
#pragma unroll 1
  for (int i = 0; i < split; ++i) {
    mass = mass + sh.parts[i].mass;
    top += value(sh.parts[i].top) * step(sh.parts[i].ref, most, c);
  }
  return top >= 9.5367432e-7f && !(p.teacher_lse && beyond(mass, p.teacher_lse[r], INFINITY) > 0.f);
}

// The row's loss and statistics from its CTAs' parts, by one thread while the others go on to the gradient.  again: of
// the second pass.
__device__ __noinline__ void write_loss(const DistillParams& p, int r, const Shared& sh, int split, Pair inv_t, float c,
                                        int flags, int again) {
  const Part* parts = sh.parts;
  const float most = sh.most, ref_out = again ? sh.ref_out : most;
  Pair rest{0.f, 0.f}, inside{0.f, 0.f}, mass{0.f, 0.f}, loss{0.f, 0.f};
#pragma unroll 1
  for (int i = 0; i < split; ++i) {
    const float f = again ? 1.f : step(parts[i].ref, most, c);
    rest = rest + parts[i].rest * f;
    inside = inside + parts[i].top * f;
    if (!(value(parts[i].mass) > 0.f)) continue;  // (its reference may be anything)
    mass = mass + parts[i].mass;
    loss = loss + (parts[i].against + parts[i].mass * (two_sum(most, -parts[i].ref) * inv_t));
  }
  const bool some_rest = value(rest) > 0.f;
  const Pair ln = log_pair(again ? rest * step(ref_out, most, c) + inside * step(sh.ref_in, most, c) : rest + inside);
  const Pair ln_rest = some_rest ? log_pair(rest) : Pair{-INFINITY, 0.f};
  const float gap = ln.hi - ln_rest.hi + (most - ref_out) * inv_t.hi;
  const float tail = p.teacher_lse ? beyond(mass, p.teacher_lse[r], gap) : 0.f;
  loss = loss + mass * ln;
  if (tail > 0.f && some_rest)
    loss = loss + ((log_pair(Pair{tail, 0.f}) - ln_rest + ln) * tail + two_sum(most, -ref_out) * tail * inv_t);
  const bool infinite = (flags & 2) || (tail > 0.f && !some_rest), invalid = flags & 1;
  // (a term past float32's range, of a masked token with p > 0, leaves a pair void: +inf)
  p.loss[r] = invalid ? NAN : infinite || !(fabsf(value(loss)) < INFINITY) ? INFINITY : value(loss);
  p.stats[2 * r] = invalid ? NAN : shifted(most, inv_t, ln);
  p.stats[2 * r + 1] = invalid ? NAN : some_rest ? shifted(ref_out, inv_t, ln_rest) : -INFINITY;
}

// Loss and statistics of a row, and its gradient (kGrad).  Bound: without the gradient the loads (eight CTAs per SM,
// 64 registers; half of the issue slots are used); with it the phases of a row (copy, sum, exchange,
// gradient), which two other CTAs on the SM cover in part, and 17.6 instructions a logit, the row's fixed part among
// them.  Measured: the loss of 2304 x 128256 bf16, record of 64, 99.6 us (5.95 TB/s), 515 x 50001 bf16 21.8 us with the
// host's call; loss and gradient of 2048 x 128256 bf16, record of 128, 236 us (4.5 TB/s read and written), 37 x 32001
// float32 18 to 22 us with the host's call.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(threads_of(kGrad), kGrad ? 3 : 8) distill_kernel(const __grid_constant__ DistillParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  constexpr int kV = Elems<T>::kVec, kT = threads_of(kGrad), kW = kT / 32;
  const int split = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int r = blockIdx.x >> (__ffs(split) - 1), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (split > 1) cluster_arrive_relaxed();
  const T* row = static_cast<const T*>(p.student) + static_cast<size_t>(r) * p.V;
  T* out = kGrad ? static_cast<T*>(p.grad) + static_cast<size_t>(r) * p.V : nullptr;
  const int32_t* ids = p.ids + static_cast<size_t>(r) * p.K;
  const float* values = p.values + static_cast<size_t>(r) * p.K;
  const Slice<T> s(row, p.V, rank, split);
  if (!index_ok(r < p.N && split <= kDSplit && s.per * split >= s.nv && s.head + s.nv * kV <= p.V)) return;
  Entry* entries = reinterpret_cast<Entry*>(raw + shared_bytes());
  uint32_t* bits = reinterpret_cast<uint32_t*>(raw + shared_bytes() + entry_bytes(p.K));
  uint32_t* hits = bits + bitmap_bytes(s.per, kV) / 4;
  uint4* kept = reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(hits) + hit_bytes(s.per, kT));

  // the record's tokens of this slice; whether the record holds any at all
  uint4 first[kDU];
  if (!kGrad) first_loads<T, kT>(row, s, first);
  const int id0 = tid < p.K ? __ldg(ids + tid) : -1;
  const float v0 = tid < p.K ? __ldg(values + tid) : 0.f;
  const float teacher_lse = p.teacher_lse ? __ldg(p.teacher_lse + r) : 0.f;
  const float g = kGrad && p.grad_loss ? __ldg(p.grad_loss + r) : 1.f;
  const float2 entry = p.teacher_lse ? exp2_table_entry() : make_float2(0.f, 0.f);
  if (kGrad) keep_slice<T, kT>(row, s, kept);  // behind the loads above, which the row waits for first
  for (int i = tid; i < (bitmap_bytes(s.per, kV) + hit_bytes(s.per, kT)) / 16; i += kT)
    reinterpret_cast<uint4*>(bits)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < 64) sh.tab[tid] = entry;
  int some = id0 != -1;
  for (int k = tid + kT; k < p.K; k += kT) some |= ids[k] != -1;
  some = __syncthreads_or(some);
  if (!some) {  // the position is left out
    if (rank == 0 && tid == 0) {
      p.loss[r] = 0.f;
      p.stats[2 * r] = 0.f;
      p.stats[2 * r + 1] = 0.f;
    }
    if (kGrad) {
      zero_slice<T, kT>(out, p.V, s, p.vec != 0);
      kept_wait<0>();
    }
    __syncwarp();
    if (split > 1) cluster_wait();
    return;
  }
  // this slice's tokens of the record, marked and listed in the record's order
  int bad = 0, twice = 0;
  unsigned int own = 0;  // bit i: entry tid + i kT is one
#pragma unroll
  for (int i = 0; i < kMaxTop / kT; ++i) {
    bool mine = false;
    if (i * kT < p.K) {
      const int k = i * kT + tid, id = i == 0 ? id0 : k < p.K ? ids[k] : -1;
      const float v = i == 0 ? v0 : k < p.K ? values[k] : 0.f;
      if (id != -1) {
        bad |= id < 0 || id >= p.V || !(v < INFINITY);
        const int b = id >= 0 && id < p.V ? s.bit(id) : -1;
        mine = b >= 0 && index_ok(b < s.per * kV + 16);
        if (mine) {
          twice |= (atomicOr(bits + (b >> 5), 1u << (b & 31)) >> (b & 31)) & 1u;
          const int v = b / kV, group = v / (kT * kDU);
          if (v < s.per && index_ok(group / 32 < hit_words(s.per, kT))) atomicOr(hits + group / 32 * kT + v % kT, 1u << (group % 32));
        }
      }
    }
    const unsigned int all = __ballot_sync(0xffffffffu, mine);
    own |= mine ? 1u << i : 0u;
    if (lane == 0) sh.count[i * kW + warp] = __popc(all);
  }
  const Record rec = read_record<kT>(p, r, teacher_lse, sh.red, sh.part[0], &bad);
  {
    float m;
    if (kGrad) {
      kept_wait<1>();
      m = -INFINITY;
      for (int u = 0, v = tid; u < kDU && v < s.v1 - s.v0; ++u, v += kT) {
        const uint4 one[1] = {kept[v]};
        m = max_nan(m, GroupMax<T, 1>::get(one));
      }
    } else {
      m = GroupMax<T, kDU>::get(first);
    }
    m = warp_max_nan(m);
    if (lane == 0) sh.red[warp] = m;
  }
  if (tid == 0) sh.any = 0;
  bad = __syncthreads_or(bad);
  float ref = sh.red[0];
#pragma unroll
  for (int w = 1; w < kW; ++w) ref = fmaxf(ref, sh.red[w]);
  if (!(fabsf(ref) < INFINITY)) ref = 0.f;
  if (tid == 0) sh.ref = sh.ref_out = sh.ref_in = ref;
  const float c = p.c;
  int n;  // entries of this slice
  {
    const int mine = sh.count[lane];  // kMaxTop / 32 = 32 runs of 32 entries
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    n = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int i = 0; i < kMaxTop / kT; ++i) {
      if (i * kT >= p.K) break;
      const bool is = (own >> i) & 1u;
      const unsigned int all = __ballot_sync(0xffffffffu, is);
      const int base = __shfl_sync(0xffffffffu, incl - mine, i * kW + warp);
      if (is) {
        const int k = i * kT + tid;
        const int at = base + __popc(all & ((1u << lane) - 1u));
        if (index_ok(at < n && at < p.K))
          entries[at] = i == 0 ? Entry{v0, 0.f, 0.f, id0} : Entry{values[k], 0.f, 0.f, ids[k]};
      }
    }
  }
  __syncthreads();

  int flags = bad ? 1 : 0, again = 0, some_rest = 1;
  // the sums relative to the slice's reference; again with the row's own where those were far off
  for (;; again = 1) {
    const Scale w(c, ref);
    flags |= twice;
    // the first entry's logit is on its way while the slice is streamed
    const float logit = again == 0 && tid < n && index_ok(entries[tid].id >= 0 && entries[tid].id < p.V)
                            ? Elems<T>::one(row, entries[tid].id)
                            : 0.f;
    if (kGrad && again == 0) kept_wait<0>();
    Pair sum{0.f, 0.f};
    if (some_rest) sum = warp_sum(w.clean(sum_slice<T, kT, kGrad>(row, p.V, s, bits, hits, first, w, kept)));
    if (warp * 32 < n) {
      const float ref = sh.ref;
      const Scale w(c, sh.ref_in);
      Pair mass{0.f, 0.f}, against{0.f, 0.f}, top{0.f, 0.f};
      for (int i = tid; i < n; i += kT) {
        Entry e = entries[i];
        if (!index_ok(e.id >= 0 && e.id < p.V && i < p.K)) continue;
        if (again == 0) e.l = i < kT ? logit : Elems<T>::one(row, e.id);
        const Pair x = entry_log(rec, e.v);
        const Pair pr = probability(x, p.teacher_lse != nullptr, sh.tab);
        e.p = value(pr);
        if (again == 0) entries[i] = e;
        mass = mass + pr;
        if (e.p > 0.f) {  // (p before 1 / T: a masked logit times 1 / T may leave float32's range)
          if (e.l > -INFINITY)
            against = against + (x * pr - two_sum(e.l, -ref) * pr * rec.inv_t);
          else
            flags |= 2;
        }
        top = top + Pair{w(e.l), 0.f};
      }
      top = w.clean(top);
      mass = warp_sum(mass);
      against = warp_sum(against);
      top = warp_sum(top);
      if (lane == 0) {
        sh.part[1][warp] = top;
        sh.part[2][warp] = mass;
        sh.part[3][warp] = against;
      }
    } else if (lane < 3) {
      sh.part[1 + lane][warp] = Pair{0.f, 0.f};
    }
    if (lane == 0) sh.part[0][warp] = sum;
    if (flags) atomicOr(&sh.any, flags);
    __syncthreads();
    if (again == 0 && split > 1) cluster_wait();  // every CTA of the cluster has started
    if (warp == 0) {
      // eight lanes add up each of the four sums
      Pair t = lane % 8 < kW ? sh.part[lane / 8][lane % 8] : Pair{0.f, 0.f};
#pragma unroll 1
      for (int o = 4; o > 0; o >>= 1)
        t = t + Pair{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)};
      // to every CTA of the cluster, lane 8 i + c sum i to CTA c
      const uint32_t mine = smem_addr(&sh), cta = lane % 8, which = lane / 8;
      if (cta < static_cast<uint32_t>(split)) {
        const uint32_t there = dsmem_map(mine, cta) - mine;
        Part* to = &sh.parts[rank];
        Pair* place = which == 0 ? &to->rest : which == 1 ? &to->top : which == 2 ? &to->mass : &to->against;
        dsmem_st_pair(there + smem_addr(place), t);
        if (which == 0) dsmem_st_f32(there + smem_addr(&to->ref), sh.ref);
        if (which == 2) dsmem_st_u32(there + smem_addr(&to->flags), static_cast<uint32_t>(sh.any));
      }
      __syncwarp();
    }
    if (split > 1)
      cluster_sync();
    else
      __syncthreads();
    if (warp == 0) {
      // lane i takes CTA i's part, relative to the largest of the references; float32 will do for the gradient, but for
      // what the record's mass leaves of 1
      const Part& part = sh.parts[lane < split ? lane : 0];
      float most = part.ref;
      int any = part.flags;
#pragma unroll 1
      for (int o = 1; o < split; o <<= 1) {
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        any |= __shfl_xor_sync(0xffffffffu, any, o);
      }
      // a slice whose sums left its first loads far below, or whose record is far from them
      const bool far = !(value(part.rest + part.top) < kFarSum) ||
                       (value(part.mass) > 0.f && !((most - part.ref) * p.inv_t < kFarRef));
      const float f_out = step(again ? sh.ref_out : part.ref, most, c);
      float rest = value(part.rest) * (again ? 1.f : f_out);
#pragma unroll 1
      for (int o = 1; o < split; o <<= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
      if (kGrad) {
        const float f_in = again ? step(sh.ref_in, most, c) : f_out;
        float total = again ? value(part.rest) * f_out + value(part.top) * f_in : value(part.rest + part.top) * f_out;
        Pair mass = part.mass;
#pragma unroll 1
        for (int o = 1; o < split; o <<= 1) {
          total += __shfl_xor_sync(0xffffffffu, total, o);
          mass = mass + Pair{__shfl_xor_sync(0xffffffffu, mass.hi, o), __shfl_xor_sync(0xffffffffu, mass.lo, o)};
        }
        // a token of the record has q = weight f_in / total, f_in the step from its reference to the common one; any
        // other weighs f_out / total in the row and f / rest in the tail
        const float gap = again ? (most - sh.ref_out) * p.inv_t - logf(__fdividef(rest, total))
                          : rest > 0.f ? 0.f : INFINITY;
        const float tail = p.teacher_lse ? beyond(mass, p.teacher_lse[r], gap) : 0.f, both = value(mass) + tail;
        // (approximate quotients, two steps of 2^-23: their operands' weights carry the exponential's 2^-22 each)
        const float scale = __fmul_rn(g, p.inv_t), f = again ? 1.f : f_out;
        const float share = tail > 0.f && rest > 0.f ? __fdividef(__fmul_rn(tail, f), rest) : 0.f;
        if (lane == rank) {
          sh.k_in = __fdividef(__fmul_rn(both, f_in), total) * __fmul_rn(scale, value(make_up(Scale(c, sh.ref_in).miss)));
          sh.k_out = (any & 1) ? NAN : (__fdividef(__fmul_rn(both, f_out), total) - share) * __fmul_rn(scale, value(make_up(w.miss)));
        }
      }
      bool redo = __any_sync(0xffffffffu, far);
      if (!(rest >= kLeastRest)) redo |= rest != 0.f || !nothing_beyond(p, r, sh, split, most, c);
      if (lane == 0) {
        sh.most = most;
        sh.flags = any;
        sh.again = !again && !(any & 1) && redo;
      }
    }
    __syncthreads();
    flags = sh.flags;
    if (!sh.again) break;
    flags &= 1;
    const int found = own_references<T, kT>(row, p.V, bits, entries, n, rank, split, sh);
    if (found == 0) {  // NaN or +inf in the row, or nothing but -inf
      flags |= 1;
      if (tid == 0) sh.k_out = NAN;
      __syncthreads();
      break;
    }
    ref = sh.ref_out;
    some_rest = found == 2;
    if (!kGrad && some_rest) first_loads<T, kT>(row, s, first);
  }

  const bool invalid = flags & 1;
  if (rank == 0 && tid == kT - 1) write_loss(p, r, sh, split, rec.inv_t, c, flags, again);
  if (!kGrad) return;
  if (g == 0.f) {
    zero_slice<T, kT>(out, p.V, s, p.vec != 0);
    return;
  }
  const float k_in = sh.k_in, k_out = sh.k_out, scale = __fmul_rn(g, p.inv_t);
  const Scale w(c, ref);
  T* body = out + s.head;
  const bool vec = p.vec != 0;
  for (int v = tid; v < s.v1 - s.v0; v += kT) grad_vector<T>(kept[v], body, s.v0 + v, vec, w.c, w.shift, k_out);
  map_ends(row, out, p.V, s, [&](float l) { return w(l) * k_out; });
  if (invalid) return;
  __syncthreads();
  // the slice's tokens of the record, over what was written there
  const Scale w_in(c, sh.ref_in);
  for (int i = tid; i < n; i += kT) {
    const Entry e = entries[i];
    if (index_ok(e.id >= 0 && e.id < p.V)) out[e.id] = to_grad<T>(__fmaf_rn(w_in(e.l), k_in, -__fmul_rn(e.p, scale)));
  }
}

// ---------------------------------------------------------------- gradient from the forward pass's stats

// A float32 log-sum-exp tells the weights relative to it to 2^-24 of itself, nothing from here up.
constexpr float kTelling = 4194304.f;  // 2^22

// One read and one write of the row: q_j needs the two statistics and nothing of the row's other logits, so a row's CTAs
// know nothing of each other.  Bound by DRAM: 1536 x 152064 float32, record of 64, 292 us (6.4 TB/s read and
// written, 94 % of the copy peak); 64 x 32128 float32 7.5 us.
template <typename T>
__global__ void __launch_bounds__(kDT, 4) distill_backward_kernel(DistillParams p, int split) {
  __shared__ float red[kDW];
  __shared__ Pair part[kDW];
  __shared__ float2 tab[64];
  const int r = blockIdx.x >> (__ffs(split) - 1), rank = blockIdx.x & (split - 1), tid = threadIdx.x;
  const T* row = static_cast<const T*>(p.student) + static_cast<size_t>(r) * p.V;
  T* out = static_cast<T*>(p.grad) + static_cast<size_t>(r) * p.V;
  const Slice<T> s(row, p.V, rank, split);
  if (!index_ok(r < p.N && s.per * split >= s.nv)) return;
  const float g = p.grad_loss ? p.grad_loss[r] : 1.f;
  const int32_t* ids = p.ids + static_cast<size_t>(r) * p.K;
  const float* values = p.values + static_cast<size_t>(r) * p.K;
  const uint4* r4 = reinterpret_cast<const uint4*>(row + s.head);
  int v = s.v0 + tid;
  uint4 q[kDU];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < kDU; ++u)
      if (v + u * kDT < s.v1) q[u] = ldg_stream(r4 + v + u * kDT);
  };
  const float teacher_lse = p.teacher_lse ? p.teacher_lse[r] : 0.f;
  const float lse = p.stats[2 * r], lse_rest = p.stats[2 * r + 1];
  if (p.teacher_lse && tid < 64) tab[tid] = exp2_table_entry();
  int some = 0, bad = 0;
  if (g != 0.f)
    for (int k = tid; k < p.K; k += kDT) {
      const int id = ids[k];
      some |= id != -1;
      bad |= id != -1 && (id < 0 || id >= p.V || !(values[k] < INFINITY));
    }
  some = __syncthreads_or(some);
  if (!some) {  // no gradient reaches this row: zeros, its logits unread
    zero_slice<T, kDT>(out, p.V, s, p.vec != 0);
    return;
  }
  load();  // in flight while the record is read
  const Record rec = read_record<kDT>(p, r, teacher_lse, red, part, &bad);
  Pair mass{0.f, 0.f};
  for (int k = tid; k < p.K; k += kDT)
    if (ids[k] >= 0 && values[k] > -INFINITY) mass = mass + probability(entry_log(rec, values[k]), p.teacher_lse != nullptr, tab);
  mass = block_sum<kDT>(mass, part);
  bad |= !(fabsf(lse) < kTelling);  // the forward pass found the row invalid, or its statistics tell nothing
  bad = __syncthreads_or(bad);
  const float gap = lse - lse_rest;
  const float tail = p.teacher_lse ? beyond(mass, teacher_lse, gap) : 0.f;
  const float both = value(mass + Pair{tail, 0.f}), scale = __fmul_rn(g, rec.inv_t.hi);
  // weights 2^(s c + shift), shift the float32 nearest to -T lse c; what the roundings of it and of T lse miss goes
  // into the factors
  auto scale_of = [&](float lse, float& k) {
    const float ref = __fmul_rn(lse, p.temperature);
    const Scale w(p.c, ref);
    k = scale * value(make_up(w.miss + __fmul_rn(__fmaf_rn(lse, p.temperature, -ref), p.inv_t)));  // (lse - ref / T)
    return w;
  };
  // tokens outside the record: q less their share of the tail, relative to lse, or to lse_rest where that is so far
  // below that q is nothing and the quotient of the two would leave float32's range
  float k_in;
  const Scale w_in = scale_of(lse, k_in);
  Scale w = w_in;
  float k_out;
  if (__builtin_expect(gap > 40.f && fabsf(lse_rest) < kTelling, 0)) {
    float k;
    w = scale_of(lse_rest, k);
    k_out = (both * exp_pair(two_sum(lse_rest, -lse)) - tail) * k;
  } else {
    const float share =
        tail > 0.f && fabsf(lse_rest) < kTelling ? tail * exp_pair(two_sum(lse, -lse_rest)) : 0.f;
    k_out = (both - share) * k_in;
  }
  k_in *= both;
  if (bad) k_out = NAN;
  T* body = out + s.head;
  const bool vec = p.vec != 0;
  while (v < s.v1) {
#pragma unroll
    for (int u = 0; u < kDU; ++u)
      if (v + u * kDT < s.v1) grad_vector<T>(q[u], body, v + u * kDT, vec, w.c, w.shift, k_out);
    v += kDU * kDT;
    load();
  }
  map_ends(row, out, p.V, s, [&](float l) { return w(l) * k_out; });
  if (bad) return;
  __syncthreads();
  for (int k = tid; k < p.K; k += kDT) {  // the slice's tokens of the record, over what was written there
    const int id = ids[k];
    if (id < 0 || s.bit(id) < 0 || !index_ok(id < p.V)) continue;
    const float pk = values[k] > -INFINITY ? exp_pair(entry_log(rec, values[k])) : 0.f;
    out[id] = to_grad<T>(__fmaf_rn(w_in(Elems<T>::one(row, id)), k_in, -__fmul_rn(pk, scale)));
  }
}

// ---------------------------------------------------------------- launches

// CTAs per row: doubled while the batch gives at most `most` CTAs and a CTA is left 2048 logits.  Most: two per SM of
// 256 threads, four of 128 (the loss of 512 x 128256 float32: 49 us with four or six, 69 with two or three; 200 x
// 128256 bf16: 19 with four, 24 with two or six).
int split_for(int N, int V, int most) {
  int split = 1;
  while (split < kDSplit && static_cast<long long>(N) * split <= most && V / (2 * split) >= 2048) split *= 2;
  return split;
}

template <typename K>
cudaError_t allow_smem(K kernel, std::atomic<unsigned long long>& prepared) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (prepared.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           shared_bytes() + entry_bytes(SPEC_MAX_TOP) + bitmap_bytes(kMaxVocab / 4 / kDSplit, 4) +
                               hit_bytes(kMaxVocab / 4 / kDSplit, kDT) + kMaxVocab / 4 / kDSplit * 16);
  if (e == cudaSuccess) prepared.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <typename T, bool kGrad>
cudaError_t launch_loss(const DistillParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> prepared{0};
  const cudaError_t e = allow_smem(distill_kernel<T, kGrad>, prepared);
  if (e != cudaSuccess) return e;
  constexpr int kV = Elems<T>::kVec;
  int split = split_for(p.N, p.V, (kGrad ? 2 : 4) * (p.sms > 0 ? p.sms : 152));
  auto bytes = [&](int n) { return (p.V / kV + n - 1) / n * 16; };  // of the row a CTA keeps
  if (kGrad)
    while (split < kDSplit && bytes(split) > kKeepBytes) split *= 2;
  const int per = (p.V / kV + split - 1) / split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.N) * split);
  cfg.blockDim = dim3(threads_of(kGrad));
  cfg.dynamicSmemBytes = shared_bytes() + entry_bytes(p.K) + bitmap_bytes(per, kV) +
                         hit_bytes(per, threads_of(kGrad)) + (kGrad ? per * 16 : 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, distill_kernel<T, kGrad>, p);
}

template <typename T>
cudaError_t launch_backward(const DistillParams& p, cudaStream_t stream) {
  const int split = split_for(p.N, p.V, 2 * (p.sms > 0 ? p.sms : 152));
  distill_backward_kernel<T><<<static_cast<unsigned>(p.N) * split, kDT, 0, stream>>>(p, split);
  return cudaGetLastError();
}

}  // namespace

#ifdef SPEC_DEBUG_BOUNDS
cudaError_t distill_bounds(uint32_t* word) { return take_row_bounds(word); }
#endif

cudaError_t distill_forward_launch(const DistillParams& p, int dtype, cudaStream_t stream) {
  return dtype == 0 ? launch_loss<float, false>(p, stream) : launch_loss<__nv_bfloat16, false>(p, stream);
}

cudaError_t distill_backward_launch(const DistillParams& p, int dtype, cudaStream_t stream) {
  return dtype == 0 ? launch_backward<float>(p, stream) : launch_backward<__nv_bfloat16>(p, stream);
}

cudaError_t distill_loss_grad_launch(const DistillParams& p, int dtype, cudaStream_t stream) {
  return dtype == 0 ? launch_loss<float, true>(p, stream) : launch_loss<__nv_bfloat16, true>(p, stream);
}

}  // namespace specv
