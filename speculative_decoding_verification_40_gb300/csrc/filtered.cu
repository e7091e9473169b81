// Filtered sampling (temperature, top-k, top-p, min-p per row, one given uniform per row) and top logits
// on sm_103a.  The operations are specified in include/spec_verify.h.
//
// Every filter keeps the logits at or above some value, so a row's kept set is {l >= tau}, and it is nearly
// always a few thousand logits at most.  A cluster of CTAs streams a row once, each its slice: the first
// loads of every warp give an estimate of the value that some 1000 logits of the row lie above; logits at
// or above it go to a list in the first CTA's shared memory, the others only into a float32 sum of weights
// (and only where a nucleus needs the row's total).  The first CTA then finds tau on the list (by rank for
// top-k, by the exact fixed-point masses of weight.cuh for top-p) and draws from it.
//
// The list decides a row only where it provably holds all that matters: at least k logits, a mass past the
// nucleus at both ends of the float sum's error bound, the min-p cut above the estimate.  A nucleus that ends
// below the list takes a second pass of the whole cluster: a sample of the row says between which two
// values the nucleus must end, the pass sums the exact weights above them (per group of 512 tokens) and lists
// the logits between them.  A row whose cut is known (no filter, min-p alone with more logits than
// the list holds) takes the second pass for the group sums alone.  A list that ran over or came out shorter than
// k is made once more, with an estimate that its length corrects.  What is left (more ties than the list
// holds) is decided by exact selection over the whole row by the first CTA.
#include <atomic>
#include <cstring>
#include <type_traits>

#include "../../include/spec_verify.h"
#include "common.cuh"
#include "row_bounds.cuh"
#include "row_kernels.h"
#include "select.cuh"
#include "softmax.cuh"
#include "weight.cuh"

namespace specv {

namespace {

constexpr int kFT = 256;            // threads per CTA: four CTAs per SM, one row's finish overlaps others' loads
constexpr int kFW = kFT / 32;
constexpr int kGroup = 512;         // tokens per group of the draw
constexpr int kGroups = kMaxVocab / kGroup;
static_assert(kGroup == 2 * kFT && kGroups == 2 * kFT, "the draw's scans take two values per thread");
constexpr int kMaxSplit = 8;        // CTAs per row (the portable cluster size)
constexpr int kLeastSlice = 2048;   // logits that a CTA of several takes at least
constexpr int kListCap = 2400;      // logits a row's list holds
static_assert(kListCap < 2 * kLeastSlice, "a row that its list holds is one CTA's: a cluster's CTAs meet in estimate()");
constexpr int kListAim = 1000;      // logits the estimate aims at; vocabularies sorted by frequency give half to twice
constexpr int kSample = 1024;       // sampled maxima behind the estimate
constexpr int kSampleBins = 512;    // and the bins that rank them
constexpr int kBinMaxima = 48;      // maxima in the bin of the wanted rank that are ranked no further
constexpr int kListBins = 512;      // bins of a histogram over the list
constexpr int kBracketAim = 1100;   // logits the second pass's list aims at
constexpr int kProbe = 16;          // vectors per thread of the sample that places it
constexpr int kFew = 32;            // candidates one warp ranks directly
constexpr int kFewKept = 128;       // kept tokens a draw adds up pair by pair
constexpr float kMinTemp = 5.42101086e-20f, kMaxTemp = 1.84467441e19f;  // 2^-64, 2^64
constexpr float kRestOne = 1073741824.f;                                 // 2^30
constexpr uint32_t kKeyNegInf = 0x007fffffu;                             // fkey(-inf)

struct CutResult {
  uint32_t key;               // the cut
  unsigned long long above;   // units of the keys above it
  unsigned long long at;      // units of the keys equal to it
};

struct Words {
  unsigned int lo[kBins], mid[kBins], hi[kBins], top[kBins];
};

// A histogram as Hist (select.cuh) of masses up to 2^45, bits 42 up of every value in a fourth word: with three, 2^18 of
// the largest weight in one bin would wrap the third.
struct WideHist : Hist {
  unsigned int* top;
  __device__ __forceinline__ unsigned long long get(int b) const {
    return (static_cast<unsigned long long>(top[b]) << 42) + Hist::get(b);
  }
  __device__ __forceinline__ void add(int b, unsigned long long v) const {
    Hist::add(b, v & ((1ull << 42) - 1));
    const unsigned int t = static_cast<unsigned int>(v >> 42);
    if (t) atomicAdd(top + b, t);
  }
  template <int kThreads>
  __device__ __forceinline__ void zero(int nb) const {
    for (int k = threadIdx.x; k < nb; k += kThreads) top[k] = 0u;
    Hist::zero<kThreads>(nb);
  }
};

static_assert(kFW * kGroup * sizeof(float) <= kListCap * sizeof(unsigned long long), "the second pass gathers there");

struct Shared {
  union {
    struct {
      float val[kListCap];               // the list: logits and their tokens
      int id[kListCap];
      union {
        unsigned long long w[kListCap];  // their weights
        unsigned long long pairs[kBins];  // top logits: (key, token) pairs to sort
      };
    };
    Words row_hist;                      // selection over the whole row
  };
  union {
    struct {
      unsigned int lo[kListBins], mid[kListBins], hi[kListBins];  // selection over the list
    } hist;
    struct {
      unsigned long long w[kFewKept];    // a draw from few tokens: their weights and ids
      int id[kFewKept];
    } kept;
    struct {
      uint4 key[kSample / 4];            // keys of sampled maxima, from every CTA of the cluster
      unsigned int count[kSampleBins];   // and their histogram
    } sample;
  };
  struct {
    unsigned long long group[kGroups];   // draw: weight per group, then per token of a group
    unsigned long long token[kGroup];
  } draw;
  unsigned long long wsum[kFW];
  float2 tab[64];
  float red[kFW];
  uint32_t low[kFW];
  float bottom[kFW];
  Pick pick;
  CutResult cut;
  unsigned long long few_units[kFew];
  uint32_t few_key[kFew];
  unsigned long long rest[kMaxSplit];  // per CTA of the cluster: the weights below the estimate (2^30 for its own),
  float most[kMaxSplit];               // the largest logit (of the list, where there is one) and the smallest key
  uint32_t lowest[kMaxSplit];
  float below;                       // the estimate
  unsigned long long at_below;
  int at, n, few;
  unsigned int least;
  // the first CTA's decision on a second pass
  int next, aim;                       // Next; for another list, its aim
  uint32_t key_lo, key_hi;             // for a second pass: list [key_lo, key_hi), sum from key_hi up
  float M;
};

// Starts the copy of n bytes from p on (both multiples of 16) into the L2; n <= 0: nothing.
__device__ __forceinline__ void prefetch_l2(const void* p, int n) {
  if (n > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Block-wide inclusive scan of one value per thread; *total gets the sum of all.
// A function of its own: code that runs once per row waits for its instructions.
__device__ __noinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* wsum,
                                                      unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = warp_incl_u64(v, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  unsigned long long t = 0;
#pragma unroll
  for (int w = 0; w < kFW; ++w) {
    if (w < warp) incl += wsum[w];
    t += wsum[w];
  }
  __syncthreads();
  *total = t;
  return incl;
}

__device__ __forceinline__ uint32_t dsmem_add_u32(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void dsmem_st_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void dsmem_st_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- sources of (logit, token)

// A whole row, each thread a strided share: fn(logit, token, 0).
template <typename T>
struct RowSource {
  const T* row;
  int V;
  template <typename F>
  __device__ __forceinline__ void each(F&& fn) const {
    constexpr int kV = Elems<T>::kVec;
    const int head = head_of(row, V);
    const int nv = (V - head) / kV;
    const uint4* r4 = reinterpret_cast<const uint4*>(row + head);
    for (int v = threadIdx.x; v < nv; v += kFT) {
      float f[kV];
      Elems<T>::widen(__ldg(r4 + v), f);
#pragma unroll
      for (int j = 0; j < kV; ++j) fn(f[j], head + v * kV + j, 0);
    }
    for (int k = threadIdx.x; k < head; k += kFT) fn(Elems<T>::one(row, k), k, 0);
    for (int k = head + nv * kV + threadIdx.x; k < V; k += kFT) fn(Elems<T>::one(row, k), k, 0);
  }
  // elements before the row's first 16-byte boundary (rows of an odd vocabulary start anywhere)
  __device__ static __forceinline__ int head_of(const T* row, int V) {
    const int past = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T));
    return past ? min(V, Elems<T>::kVec - past) : 0;
  }
};

// The list in shared memory: fn(logit, token, entry).
struct ListSource {
  const float* val;
  const int* id;
  int n;
  template <typename F>
  __device__ __forceinline__ void each(F&& fn) const {
    for (int i = threadIdx.x; i < n; i += kFT) fn(val[i], id[i], i);
  }
};

// ---------------------------------------------------------------- selection

// Of the `few` candidates of sh.few_key[] and sh.few_units[], above units lying above them all, the key at which
// the running units reach need.
__device__ __noinline__ CutResult rank_few(int few, unsigned long long above, unsigned long long need, Shared& sh) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const uint32_t key = lane < few ? sh.few_key[lane] : 0u;
    unsigned long long over = above, at = 0;
#pragma unroll 4
    for (int j = 0; j < few; ++j) {
      const uint32_t kj = sh.few_key[j];
      const unsigned long long uj = sh.few_units[j];
      over += kj > key ? uj : 0ull;
      at += kj == key ? uj : 0ull;
    }
    if (lane < few && over < need && need <= over + at) sh.cut = CutResult{key, over, at};
  }
  __syncthreads();
  const CutResult c = sh.cut;
  __syncthreads();
  return c;
}

// The key at which the running units of the source's logits with lo <= key <= hi, largest first, reach need
// (1 <= need <= their sum); units(l, entry) is a mass (kMass), or every logit counts one.  One histogram of
// kNB linear digits of key - lo per level (the range is narrow, so one or two levels do); once at most 32
// logits are left in the bin, one warp ranks them.
template <bool kMass, int kNB, typename S, typename U>
__device__ CutResult select_key(const S& src, uint32_t lo, uint32_t hi, unsigned long long need, U&& units,
                                Shared& sh) {
  const int tid = threadIdx.x;
  constexpr bool kRow = kNB == kBins;
  const Hist narrow{kRow ? sh.row_hist.lo : sh.hist.lo, !kMass ? nullptr : kRow ? sh.row_hist.mid : sh.hist.mid,
                    !kMass ? nullptr : kRow ? sh.row_hist.hi : sh.hist.hi};
  using H = std::conditional_t<kRow && kMass, WideHist, Hist>;
  H h;
  if constexpr (kRow && kMass)
    h = H{narrow, sh.row_hist.top};
  else
    h = narrow;
  unsigned long long above = 0;
  constexpr int kDigit = kNB == 2048 ? 11 : 9;
  static_assert(kNB == 1 << kDigit, "a digit fills the bins");
  int shift = max(0, 32 - __clz(hi - lo) - kDigit);
  for (;;) {
    __syncthreads();  // the last level's histogram and candidates have been read
    if (tid == 0) sh.few = 0;
    h.template zero<kFT>(kNB);
    src.each([&](float l, int, int i) {
      const uint32_t key = fkey(l);
      if (key < lo || key > hi) return;
      const unsigned long long u = kMass ? units(l, i) : 1ull;
      h.add(static_cast<int>((key - lo) >> shift), u);
    });
    __syncthreads();
    const Pick p = pick_from_top<kFT>(h, kNB, need - above, sh.wsum, &sh.pick);
    if (!index_ok(p.bin >= 0 && p.bin < kNB)) return CutResult{hi, above, 0ull};
    above += p.above;
    lo += static_cast<uint32_t>(p.bin) << shift;
    if (shift == 0) {
      const unsigned long long at = h.get(p.bin);
      __syncthreads();
      return CutResult{lo, above, at};
    }
    hi = lo + ((1u << shift) - 1u);
    src.each([&](float l, int, int i) {
      const uint32_t key = fkey(l);
      if (key < lo || key > hi) return;
      const int at = atomicAdd(&sh.few, 1);
      if (at < kFew) {
        sh.few_key[at] = key;
        sh.few_units[at] = kMass ? units(l, i) : 1ull;
      }
    });
    __syncthreads();
    const int few = sh.few;
    if (few <= kFew) return rank_few(few, above, need, sh);
    shift = max(0, shift - kDigit);
  }
}

// Bins of a list's logits by their distance from the row's largest, bin kListBins - 1 the nearest: 512 over the
// list's range.  (Bins of keys would not do: keys are as dense between 2^-20 and 2^-19 as between 4 and 8.)
struct ValueBins {
  float M, scale;
  __device__ __forceinline__ ValueBins(float M_, float low) {
    const float range = M_ - low;
    M = M_;
    scale = range > 0.f && range < 1e30f ? __fdividef(kListBins - 0.5f, range) : 0.f;
  }
  __device__ __forceinline__ int operator()(float l) const {
    return kListBins - 1 - min(kListBins - 1, static_cast<int>((M - l) * scale));
  }
};

// The part of a list in one bin, from a key up.
struct BinSource {
  const ListSource& src;
  const ValueBins& bins;
  int bin;
  uint32_t floor;
  template <typename F>
  __device__ __forceinline__ void each(F&& fn) const {
    src.each([&](float l, int id, int i) {
      if (bins(l) == bin && fkey(l) >= floor) fn(l, id, i);
    });
  }
};

// The key at which the running units of the list's logits with key >= floor, largest first, reach need; sh.hist
// holds their units per bin.
template <bool kMass, typename U>
__device__ CutResult cut_list(const ListSource& src, const ValueBins& bins, uint32_t floor, uint32_t hi,
                              unsigned long long need, U&& units, Shared& sh) {
  const Hist h{sh.hist.lo, kMass ? sh.hist.mid : nullptr, kMass ? sh.hist.hi : nullptr};
  if (threadIdx.x == 0) sh.few = 0;
  const Pick p = pick_from_top<kFT>(h, kListBins, need, sh.wsum, &sh.pick);
  const BinSource part{src, bins, p.bin, floor};
  part.each([&](float l, int, int i) {
    const int at = atomicAdd(&sh.few, 1);
    if (at < kFew) {
      sh.few_key[at] = fkey(l);
      sh.few_units[at] = kMass ? units(l, i) : 1ull;
    }
  });
  __syncthreads();
  if (sh.few <= kFew) return rank_few(sh.few, p.above, need, sh);
  CutResult c = select_key<kMass, kListBins>(part, floor, hi, need - p.above, units, sh);
  c.above += p.above;
  return c;
}

// ---------------------------------------------------------------- the draw

// The index among 2 kFT values (thread t holds 2t and 2t + 1, incl their running sum) that the running sum passes
// target in, and the sum below it: the thread that holds it gets the index, the others -1.
__device__ __forceinline__ int locate(unsigned long long a, unsigned long long b, unsigned long long incl,
                                      unsigned long long target, unsigned long long* below) {
  const unsigned long long at = incl - a - b, mid = incl - b;
  if (!(at <= target && target < incl)) return -1;
  *below = target < mid ? at : mid;
  return 2 * threadIdx.x + (target < mid ? 0 : 1);
}

// Finds the token the running sum of weights passes u * total in, sh.draw.group[] holding the weight of every
// group of 512 tokens; fill(g) puts the weights of group g's tokens into sh.draw.token[] (zeroed before).  The
// thread that owns the token gets it, the others -1; *total is the sum.
template <typename F>
__device__ int draw_from_groups(float u, Shared& sh, unsigned long long* total, F&& fill) {
  const int tid = threadIdx.x;
  unsigned long long a = sh.draw.group[2 * tid], b = sh.draw.group[2 * tid + 1];
  unsigned long long incl = block_scan(a + b, sh.wsum, total), below = 0;
  bool rem;
  const unsigned long long target = share_floor(u, *total, rem);
  const int mine = locate(a, b, incl, target, &below);
  if (mine >= 0) {
    sh.at = mine;
    sh.at_below = below;
  }
  sh.draw.token[tid] = 0ull;
  sh.draw.token[tid + kFT] = 0ull;
  __syncthreads();
  const int g = sh.at;
  if (!index_ok(g >= 0 && g < kGroups)) return -1;
  fill(g);
  __syncthreads();
  a = sh.draw.token[2 * tid];
  b = sh.draw.token[2 * tid + 1];
  unsigned long long group_total;
  incl = block_scan(a + b, sh.wsum, &group_total);
  const int token = locate(a, b, incl, target - sh.at_below, &below);
  return token >= 0 ? g * kGroup + token : -1;
}

struct RowFilter {
  float t, p, m, u;
  int k;
};

struct RowOut {
  int32_t* token;
  float* thr;
  float* logp;
};

// The drawn token's outputs.
__device__ __forceinline__ void write_drawn(const RowOut& out, const RowFilter& f, int token, float l, float M,
                                            float least, unsigned long long total) {
  *out.token = token;
  if (out.thr) *out.thr = least;
  // both terms have the same sign, so float32 keeps the difference to a few roundings
  if (out.logp) *out.logp = f.t == 0.f ? 0.f : __fdiv_rn(l - M, f.t) - log_weight(total);
}

// A weight as the draw counts it: at u = 0 a weight below the fixed point is one unit, so that the first token
// with any weight is drawn.
__device__ __forceinline__ unsigned long long draw_unit(unsigned long long w, float l, const Weight& weight, float u) {
  return w == 0 && u == 0.f && __fmul_rn(__fsub_rn(l, weight.M), weight.c_hi) >= kLowestLog2 ? 1ull : w;
}

// Draws from the list's logits with key >= tau: the smallest token whose running weight exceeds u * total.
template <typename T>
__device__ void draw_from_list(const ListSource& src, uint32_t tau, const Weight& weight, const RowFilter& f,
                               Shared& sh, const T* row, int V, const RowOut& out) {
  const int tid = threadIdx.x;
  unsigned int least = 0xffffffffu;
  __syncthreads();
  if (tid == 0) {
    sh.least = 0xffffffffu;
    sh.few = 0;
  }
  __syncthreads();
  src.each([&](float l, int id, int i) {
    const uint32_t key = fkey(l);
    if (key < tau) return;
    const int at = atomicAdd(&sh.few, 1);
    atomicMin(&sh.least, key);
    if (at < kFewKept) {
      sh.kept.id[at] = id;
      sh.kept.w[at] = draw_unit(sh.w[i], l, weight, f.u);
    }
  });
  __syncthreads();
  const int few = sh.few;
  if (few <= kFewKept) {  // every token adds up the weights before its own
    if ((tid & ~31) >= few) return;
    const int id = tid < few ? sh.kept.id[tid] : -1;
    unsigned long long total = 0, below = 0;
#pragma unroll 4
    for (int j = 0; j < few; ++j) {
      const unsigned long long w = sh.kept.w[j];
      total += w;
      below += sh.kept.id[j] < id ? w : 0ull;
    }
    bool rem;
    const unsigned long long target = share_floor(f.u, total, rem);
    if (tid < few && below <= target && target - below < sh.kept.w[tid])
      write_drawn(out, f, id, Elems<T>::one(row, id), weight.M, key_float(sh.least), total);
    return;
  }
  const Hist groups{sh.hist.lo, sh.hist.mid, sh.hist.hi};
  __syncthreads();
  if (tid == 0) sh.least = 0xffffffffu;
  groups.zero<kFT>(kGroups);
  src.each([&](float l, int id, int i) {
    const uint32_t key = fkey(l);
    if (key < tau) return;
    least = min(least, key);
    if (index_ok(id >= 0 && id < kMaxVocab)) groups.add(id / kGroup, draw_unit(sh.w[i], l, weight, f.u));
  });
  least = __reduce_min_sync(0xffffffffu, least);
  if ((tid & 31) == 0) atomicMin(&sh.least, least);
  __syncthreads();
  sh.draw.group[2 * tid] = groups.get(2 * tid);
  sh.draw.group[2 * tid + 1] = groups.get(2 * tid + 1);
  unsigned long long total;
  const int token = draw_from_groups(f.u, sh, &total, [&](int g) {
    src.each([&](float l, int id, int i) {
      if (id / kGroup == g && fkey(l) >= tau) sh.draw.token[id % kGroup] = draw_unit(sh.w[i], l, weight, f.u);
    });
  });
  if (token >= 0 && index_ok(token < V))
    write_drawn(out, f, token, Elems<T>::one(row, token), weight.M, key_float(sh.least), total);
}

// The eight logits a lane holds of half a group of 512 tokens, as they lie in memory (-inf beyond the row).
template <typename T>
struct Half {
  static constexpr int kV = Elems<T>::kVec;
  uint4 r[8 / kV];

  // h: the half; aligned: 16-byte loads may be used
  __device__ __forceinline__ void load(const T* row, int V, int h, int lane, bool aligned) {
    const int base = h * (kGroup / 2) + lane * kV;
    if (aligned && (h + 1) * (kGroup / 2) <= V) {
#pragma unroll
      for (int u = 0; u < 8 / kV; ++u) r[u] = __ldg(reinterpret_cast<const uint4*>(row + base + u * 32 * kV));
    } else {
      T part[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = base + j / kV * 32 * kV + j % kV;
        part[j] = k < V ? row[k] : static_cast<T>(-INFINITY);
      }
      memcpy(r, part, sizeof(r));
    }
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
#pragma unroll
    for (int u = 0; u < 8 / kV; ++u) Elems<T>::widen(r[u], f + u * kV);
  }
  __device__ static __forceinline__ int token(int h, int j, int lane) {
    return h * (kGroup / 2) + (j / kV * 32 + lane) * kV + j % kV;
  }
};

// Runs half(h, the half's logits) over both halves of groups [g0, g1), one warp per group, the next half's loads in
// flight meanwhile, and end(g) after each group.
template <typename T, typename F, typename E>
__device__ __forceinline__ void each_group(const T* row, int V, int g0, int g1, F&& half, E&& end) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool aligned = reinterpret_cast<uintptr_t>(row) % 16 == 0;
  Half<T> first, second;
  if (g0 + warp < g1) first.load(row, V, 2 * (g0 + warp), lane, aligned);
#pragma unroll 1
  for (int g = g0 + warp; g < g1; g += kFW) {
    float v[8];
    second.load(row, V, 2 * g + 1, lane, aligned);
    first.widen(v);
    half(2 * g, v);
    if (g + kFW < g1) first.load(row, V, 2 * (g + kFW), lane, aligned);
    second.widen(v);
    half(2 * g + 1, v);
    end(g);
  }
}

// The second pass over groups [g0, g1): the exact weights of the groups' tokens with key >= key_hi to sums + 8 g (an
// address in the cluster's shared memory); returns the smallest such key of this thread's logits.  (This and
// bracket_groups are functions of their own for their registers' sake: inlined, their loops spill.)
template <typename T>
__device__ __noinline__ unsigned int sum_groups(const T* row, int V, int g0, int g1, uint32_t key_hi, Weight weight,
                                                float u, uint32_t sums) {
  unsigned int least = 0xffffffffu;
  unsigned long long sum = 0;
  each_group(row, V, g0, g1,
             [&](int, const float (&v)[8]) {
#pragma unroll
               for (int j = 0; j < 8; ++j) {
                 const uint32_t key = fkey(v[j]);
                 if (key < key_hi) continue;
                 least = min(least, key);
                 sum += draw_unit(weight(v[j]), v[j], weight, u);
               }
             },
             [&](int g) {
               sum = warp_sum_u64(sum);
               if ((threadIdx.x & 31) == 0 && index_ok(g < kGroups)) dsmem_st_u64(sums + 8 * g, sum);
               sum = 0;
             });
  return least;
}

// The same for a nucleus's bracket: the tokens of logits from lo up to hi go to this CTA's list, and the float32
// weights of the logits below are summed relative to lo (this thread's sum, in 2^-30, is returned).  The logits kept
// (from hi up) are few, and a warp gathers those of a group (in the room of the list's weights) before it weighs
// them, 32 at a time: a weight is 45 instructions, which one lane in 32 would otherwise make the others wait for.
template <typename T>
__device__ __noinline__ unsigned long long bracket_groups(const T* row, int V, int g0, int g1, float lo, float hi,
                                                          Weight weight, Shared& sh, uint32_t sums) {
  const int lane = threadIdx.x & 31;
  float* gathered = reinterpret_cast<float*>(sh.w) + (threadIdx.x >> 5) * kGroup;
  const unsigned int before = (1u << lane) - 1u;
  const float from_lo = __fsub_rn(0.f, lo), from_hi = __fsub_rn(0.f, hi);
  const unsigned long long lo2 = pack2(from_lo, from_lo), hi2 = pack2(from_hi, from_hi),
                           c2 = pack2(weight.c_hi, weight.c_hi);
  float tail = 0.f, comp = 0.f;
  int kept = 0;
  each_group(row, V, g0, g1,
             [&](int h, const float (&v)[8]) {
               float a0 = 0.f, a1 = 0.f;
               unsigned int under_lo = 0, under_hi = 0;  // a bit each, the first logit's highest
#pragma unroll
               for (int j = 0; j < 8; j += 2) {
                 const unsigned long long v2 = pack2(v[j], v[j + 1]), d2 = add2(v2, lo2);
                 float d0, d1, y0, y1;
                 unpack2(d2, d0, d1);
                 under_lo = __funnelshift_l(__float_as_uint(d0), under_lo, 1);
                 under_lo = __funnelshift_l(__float_as_uint(d1), under_lo, 1);
                 unpack2(mul2(d2, c2), y0, y1);
                 const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
                 if (d0 < 0.f) a0 += e0;
                 if (d1 < 0.f) a1 += e1;
                 unpack2(add2(v2, hi2), d0, d1);
                 under_hi = __funnelshift_l(__float_as_uint(d0), under_hi, 1);
                 under_hi = __funnelshift_l(__float_as_uint(d1), under_hi, 1);
               }
               const unsigned int keep = ~under_hi & 0xffu, n_keep = __popc(keep);
               unsigned int list = under_hi & ~under_lo & 0xffu;
               if (__any_sync(0xffffffffu, keep != 0)) {
                 int at = kept;  // and the logits that the lanes before this one keep, bit by bit of their numbers
#pragma unroll
                 for (int b = 0; b < 4; ++b) {
                   const unsigned int all = __ballot_sync(0xffffffffu, (n_keep >> b) & 1u);
                   at += __popc(all & before) << b;
                   kept += __popc(all) << b;
                 }
#pragma unroll
                 for (int j = 0; j < 8; ++j) {
                   const unsigned int is = (keep >> (7 - j)) & 1u;
                   if (is && index_ok(at < kGroup)) gathered[at] = v[j];
                   at += is;
                 }
               }
               if (list) {
                 const int n = __popc(list);
                 int at = atomicAdd(&sh.n, n);
                 if (at + n <= kListCap) {
#pragma unroll 1
                   do {
                     const int j = __clz(list) - 24;
                     list &= ~(128u >> j);
                     if (index_ok(at < kListCap && Half<T>::token(h, j, lane) < V)) sh.id[at++] = Half<T>::token(h, j, lane);
                   } while (list);
                 }
               }
               const float acc = a0 + a1;
               const float t = __fadd_rn(tail, acc);
               const float b = __fsub_rn(t, tail);
               comp += __fadd_rn(__fsub_rn(tail, __fsub_rn(t, b)), __fsub_rn(acc, b));
               tail = t;
             },
             [&](int g) {
               unsigned long long sum = 0;
               if (kept > 0) {
                 __syncwarp();
#pragma unroll 1
                 for (int i = lane; i < kept; i += 32) sum += weight(gathered[i]);  // (all of them count: a nucleus's)
                 __syncwarp();
                 sum = warp_sum_u64(sum);
                 kept = 0;
               }
               if (lane == 0 && index_ok(g < kGroups)) dsmem_st_u64(sums + 8 * g, sum);
             });
  return __float2ull_rn(__fmul_rn(tail, kRestOne)) + __float2ll_rn(__fmul_rn(comp, kRestOne));
}

// The draw itself once sh.draw.group[] holds the weights of the whole row's groups.
template <typename T>
__device__ void draw_from_row(const T* row, int V, uint32_t tau, const Weight& weight, const RowFilter& f, Shared& sh,
                              unsigned int least, const RowOut& out) {
  unsigned long long total;
  const int token = draw_from_groups(f.u, sh, &total, [&](int g) {
#pragma unroll 1
    for (int i = threadIdx.x; i < kGroup; i += kFT) {
      const int k = g * kGroup + i;
      if (k >= V) break;
      const float l = Elems<T>::one(row, k);
      if (fkey(l) >= tau) sh.draw.token[i] = draw_unit(weight(l), l, weight, f.u);
    }
  });
  if (token >= 0 && index_ok(token < V))
    write_drawn(out, f, token, Elems<T>::one(row, token), weight.M, key_float(least), total);
}

// ---------------------------------------------------------------- one pass over a row

// What a CTA of the row's cluster streams: vectors [v0, v1) of the nv in the row's aligned body.
struct Slice {
  int head, nv, v0, v1;
  int rank, split;  // the first CTA takes the elements before the body too, the last one those after it
};

template <typename T>
__device__ __forceinline__ Slice slice_of(const T* row, int V, int rank, int split) {
  Slice s;
  s.head = RowSource<T>::head_of(row, V);
  s.nv = (V - s.head) / Elems<T>::kVec;
  const int per = (s.nv + split - 1) >> (__ffs(split) - 1);  // split is a power of two
  s.v0 = min(s.nv, rank * per);
  s.v1 = min(s.nv, s.v0 + per);
  s.rank = rank;
  s.split = split;
  return s;
}

constexpr int kU = 4;  // vectors in flight per thread
constexpr int kAhead = 128;  // vectors per run that the L2 gets ahead of the stream

// The bins per logit of a histogram of maxima between lo and hi.  (Maxima more than 1e30 below hi, masked by their type's
// lowest value, share the last bin; 0: they are one value.)
__device__ __forceinline__ float sample_scale(float hi, float lo) {
  const float range = fminf(hi - lo, 1e30f);
  return range > 0.f ? __fdividef(static_cast<float>(kSampleBins) - 0.5f, range) : 0.f;
}

__device__ __forceinline__ int sample_bin(uint32_t key, float hi, float scale) {
  return min(kSampleBins - 1, static_cast<int>((hi - key_float(key)) * scale));
}

struct SampleRank {
  int bin, above, in;  // the bin the want-th maximum from the top is in (-1: there are fewer), those above it, in it
};

// Every warp by itself, over sh.sample.count: lane i holds 16 bins.
__device__ __forceinline__ SampleRank sample_rank(const Shared& sh, int want) {
  const int lane = threadIdx.x & 31;
  constexpr int kPer = kSampleBins / 32;
  int mine = 0;
#pragma unroll 4
  for (int j = 0; j < kPer; ++j) mine += sh.sample.count[lane * kPer + j];
  int incl = mine;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  const unsigned int reached = __ballot_sync(0xffffffffu, incl >= want);
  if (reached == 0) return SampleRank{-1, 0, 0};
  const int who = __ffs(reached) - 1;
  int run = __shfl_sync(0xffffffffu, incl - mine, who), bin = who * kPer;
#pragma unroll 1
  for (;; ++bin) {
    if (!index_ok(bin < kSampleBins)) return SampleRank{-1, 0, 0};
    const int in = sh.sample.count[bin];
    if (run + in >= want) return SampleRank{bin, run, in};
    run += in;
  }
}

// The value some `aim` logits of the row lie at or above.  Every thread knows four maxima of the `sampled` logits
// each that it loaded first, at 32 places of the CTA's slice; an aim of a share a of the row's logits corresponds
// to the share 1 - exp(-a sampled) of those maxima, and the value of that rank among 1024 of them, the same
// ones in every CTA of the cluster, is read off their histogram over their range.  -inf, so that the list takes
// every logit, for a row that the list can hold.  floor_of(estimate, largest sampled maximum) is the value used.
template <typename F>
__device__ float estimate(const Slice& s, int V, int aim, const float (&top)[4], float sampled, Shared& sh,
                          F&& floor_of) {
  if (V <= kListCap) return -INFINITY;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t key[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) key[u] = top[u] == top[u] ? fkey(top[u]) : kKeyNegInf;
  if (s.split > 1) {
    // 1024 / split of this CTA's maxima to every CTA of the cluster, once all of them have started
    cluster_wait_acquire();
    if ((tid & (s.split - 1)) == 0) {
      const uint32_t at = smem_addr(&sh.sample.key[(s.rank * kFT + tid) >> (__ffs(s.split) - 1)]);
#pragma unroll 1
      for (int c = 0; c < s.split; ++c)
        asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dsmem_map(at, c)), "r"(key[0]),
                     "r"(key[1]), "r"(key[2]), "r"(key[3]) : "memory");
    }
    __syncwarp();
    cluster_sync();
    const uint4 all = sh.sample.key[tid];
    key[0] = all.x;
    key[1] = all.y;
    key[2] = all.z;
    key[3] = all.w;
  } else {
    sh.sample.key[tid] = make_uint4(key[0], key[1], key[2], key[3]);
  }
  uint32_t lo_key = 0xffffffffu, hi_key = 0u;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    lo_key = min(lo_key, key[u] > kKeyNegInf ? key[u] : 0xffffffffu);
    hi_key = max(hi_key, key[u]);
  }
  // over the block, with the bins cleared
  auto extremes = [&](uint32_t& low, uint32_t& high) {
    sh.sample.count[tid] = 0u;
    sh.sample.count[tid + kFT] = 0u;
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) sh.wsum[warp] = (static_cast<unsigned long long>(high) << 32) | low;
    __syncthreads();
    const unsigned long long both = sh.wsum[lane % kFW];
    low = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(both));
    high = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(both >> 32));
  };
  extremes(lo_key, hi_key);
  if (hi_key <= kKeyNegInf || !(key_float(hi_key) < INFINITY)) return -INFINITY;  // nothing finite, or +inf
  const float share = __fdividef(static_cast<float>(aim), static_cast<float>(V)), most = key_float(hi_key);
  int want =
      max(1, min(kSample, __float2int_rn(kSample * (1.f - fast_exp2(-1.442695f * share * sampled)))));
  float hi = most, scale = sample_scale(hi, key_float(lo_key));
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (key[u] > kKeyNegInf) atomicAdd(&sh.sample.count[sample_bin(key[u], hi, scale)], 1u);
  __syncthreads();
  SampleRank rank = sample_rank(sh, want);
  if (rank.bin < 0) return -INFINITY;  // fewer finite maxima than that
  // Where the bin of the wanted rank holds many maxima (a stretch of logits masked by a finite value, -1e4 or the type's
  // lowest, makes the bins as wide as its distance), once more with bins between the smallest and the largest maximum of
  // that bin; a single value, the mask itself, is left out where others lie above it (a list cannot hold its ties).
  // 512 rows of 152064, a third of them masked by -1e4, top 64: 90 us (741 where the list ran over and one CTA selected
  // from the row).
  if (__builtin_expect(rank.in > kBinMaxima && scale > 0.f, 0)) {
    int others = 0;
#pragma unroll 1
    for (int round = 0; rank.in > kBinMaxima && round < 4; ++round) {
      const uint4 all = sh.sample.key[tid];
      want -= rank.above;
      others |= rank.above;
      uint32_t low = 0xffffffffu, high = 0u;
      auto narrow = [&](uint32_t k) {
        if (k < lo_key || k > hi_key || sample_bin(k, hi, scale) != rank.bin) return;
        low = min(low, k);
        high = max(high, k);
      };
      narrow(all.x);
      narrow(all.y);
      narrow(all.z);
      narrow(all.w);
      __syncthreads();  // the bins have been read
      extremes(low, high);
      lo_key = low;
      hi_key = high;
      hi = key_float(hi_key);
      scale = sample_scale(hi, key_float(lo_key));
      if (scale == 0.f) return floor_of(others ? key_float(lo_key + 1) : hi, most);
      auto count = [&](uint32_t k) {
        if (k >= lo_key && k <= hi_key) atomicAdd(&sh.sample.count[sample_bin(k, hi, scale)], 1u);
      };
      count(all.x);
      count(all.y);
      count(all.z);
      count(all.w);
      __syncthreads();
      rank = sample_rank(sh, want);
    }
  }
  const float value = scale > 0.f ? hi - __fdividef(static_cast<float>(rank.bin + 1), scale) : hi;
  return floor_of(value, most);
}

// A warp streams four runs of its share of the slice at once, a vector of each per step, so that its first loads
// come from four places.
template <typename T>
struct Stream {
  uint4 r[kU], next[kU];  // the thread's vectors of this step and of the next one
  const uint4* run;       // the first run
  int p, q;               // the thread's place in the runs: of the next load, and of `r`
  int sub, least, all;    // vectors per run, of the last (shortest) run, of the warp's share

  // The vectors at place p of the runs, -inf past their ends.
  __device__ __forceinline__ void load(uint4 (&to)[kU]) {
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
    if ((p | 31) < least) {
#pragma unroll
      for (int u = 0; u < kU; ++u) to[u] = ldg_stream(run + p + u * sub);
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        to[u] = p < sub && p + u * sub < all ? ldg_stream(run + p + u * sub) : make_uint4(none, none, none, none);
    }
    p += 32;
  }
  __device__ __forceinline__ Stream(const T* row, const Slice& s) {
    const int warp = threadIdx.x >> 5;
    const int per = (s.v1 - s.v0 + kFW - 1) / kFW;
    const int w0 = min(s.v1, s.v0 + warp * per);
    all = min(s.v1, w0 + per) - w0;
    sub = (all + kU - 1) / kU;
    least = max(0, all - (kU - 1) * sub);
    run = reinterpret_cast<const uint4*>(row + s.head) + w0;
    q = p = threadIdx.x & 31;
    load(r);
    load(next);
    // DRAM would idle while the estimate is made: the next vectors of run `lane` to the L2 (top 64 of
    // 1536 x 152064: 206 us, 212 without; 256 or 64 vectors: 205 and 208)
    const int lane = threadIdx.x & 31;
    if (lane < kU) prefetch_l2(run + lane * sub + 64, min(kAhead, min(sub, all - lane * sub) - 64) * 16);
  }
};

// One step of a stream: the tokens of the vectors' logits at or above `cut` (and NaN) go to the list; kSum: the
// weights of the others are added to sum + comp.  The sign of l - cut says whether a logit is below it: one
// bit each, the first logit's highest.
template <typename T, bool kSum>
__device__ __forceinline__ void stream_step(const uint4 (&r)[kU], int token, int apart, unsigned long long cut2,
                                            unsigned long long c2, Shared& sh, float& sum, float& comp) {
  constexpr int kV = Elems<T>::kVec, kN = kU * kV;
  uint32_t under = 0;
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    float f[kV];
    Elems<T>::widen(r[u], f);
#pragma unroll
    for (int j = 0; j < kV; j += 2) {
      const unsigned long long d2 = add2(pack2(f[j], f[j + 1]), cut2);
      float d0, d1;
      unpack2(d2, d0, d1);
      under = __funnelshift_l(__float_as_uint(d0), under, 1);
      under = __funnelshift_l(__float_as_uint(d1), under, 1);
      if (kSum) {
        float y0, y1;
        unpack2(mul2(d2, c2), y0, y1);
        const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
        if (d0 < 0.f) a0 += e0;
        if (d1 < 0.f) a1 += e1;
      }
    }
  }
  uint32_t push = ~under & (kN == 32 ? 0xffffffffu : (1u << (kN % 32)) - 1u);
  if (push) {
    const int n = __popc(push);
    int at = atomicAdd(&sh.n, n);
    if (at + n <= kListCap) {
#pragma unroll 1
      do {
        const int e = __clz(push) - (32 - kN);  // element of the step
        push &= ~(1u << (kN - 1 - e));
        if (index_ok(at < kListCap)) sh.id[at++] = token + e / kV * apart + e % kV;
      } while (push);
    }
  }
  if (kSum) {  // sum + comp += a0 + a1 exactly but for comp's own rounding (Knuth's two-sum)
    const float acc = a0 + a1;
    const float t = __fadd_rn(sum, acc);
    const float b = __fsub_rn(t, sum);
    comp += __fadd_rn(__fsub_rn(sum, __fsub_rn(t, b)), __fsub_rn(acc, b));
    sum = t;
  }
}

// Streams the slice.  Tokens whose logits are at or above `below` (the estimate, returned) go to this CTA's list
// (sh.n counts them all and may pass kListCap); kSum: the weights 2^((l - below) c) of the others are summed
// (*rest, this thread's, in 2^-30).  aim: logits of the whole row the list should get.  Two steps at a time, so
// that the vectors of the next step stay in the registers that they were loaded into.
template <typename T, bool kSum, typename F>
__device__ float stream(const T* row, int V, const Slice& s, Stream<T>& q, int aim, float c, Shared& sh, F&& floor_of,
                        unsigned long long* rest) {
  constexpr int kV = Elems<T>::kVec;
  static_assert(kU == 4, "four runs, four maxima");
  const int tid = threadIdx.x;
  float tops[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint4 pair[2] = {q.r[u], q.next[u]};
    tops[u] = GroupMax<T, 2>::get(pair);
  }
  // logits behind each maximum: a number that every warp of the cluster must agree on, so of the longest runs
  const float steps = static_cast<float>(s.nv) * (1.f / (32 * kU * kFW)) / static_cast<float>(s.split);
  const float sampled = kV * fminf(2.f, steps);
  const float below = estimate(s, V, aim, tops, sampled, sh, floor_of);
  // -inf - -inf has no sign: a list of every finite logit compares with the lowest of them
  const float cut = fmaxf(below, -3.402823466e38f);
  const float minus = __fsub_rn(0.f, cut);  // (+0 for a cut of 0: -0 - 0 is -0, and would count as below it)
  const unsigned long long cut2 = pack2(minus, minus), c2 = pack2(c, c);
  float sum = 0.f, comp = 0.f;  // compensated: a thread adds hundreds of groups
  const int first = s.head + static_cast<int>(q.run - reinterpret_cast<const uint4*>(row + s.head)) * kV;
  const int apart = q.sub * kV;
#pragma unroll 1
  for (;;) {
    stream_step<T, kSum>(q.r, first + q.q * kV, apart, cut2, c2, sh, sum, comp);
    if ((q.q & ~31) + 32 >= q.sub) break;
    q.load(q.r);
    stream_step<T, kSum>(q.next, first + (q.q + 32) * kV, apart, cut2, c2, sh, sum, comp);
    q.q += 64;
    if ((q.q & ~31) >= q.sub) break;
    q.load(q.next);
  }
  // the row's ends outside its aligned body
  auto one = [&](int id) {
    const float l = Elems<T>::one(row, id);
    if (l < cut) {
      if (kSum) comp += fast_exp2((l - cut) * c);
    } else if (l >= cut || l != l) {
      const int at = atomicAdd(&sh.n, 1);
      if (at < kListCap) sh.id[at] = id;
    }
  };
  if (s.rank == 0 && tid < s.head) one(tid);
  if (s.rank == s.split - 1 && s.head + s.nv * kV + tid < V) one(s.head + s.nv * kV + tid);
  if (kSum) *rest = __float2ull_rn(__fmul_rn(sum, kRestOne)) + __float2ll_rn(__fmul_rn(comp, kRestOne));
  return below;
}

// The list's logits from its tokens, and the largest of them: NaN or +inf if the row holds one.  The smallest
// goes to sh.bottom.
template <typename T>
__device__ float gather_list(const T* row, int V, Shared& sh) {
  const int n = sh.n;
  float m = -INFINITY, least = INFINITY;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kFT) {
    if (!index_ok(i < kListCap && sh.id[i] >= 0 && sh.id[i] < V)) continue;
    const float l = Elems<T>::one(row, sh.id[i]);
    sh.val[i] = l;
    m = max_nan(m, l);
    least = fminf(least, l);
  }
  m = warp_max_nan(m);
  least = -warp_max_nan(-least);
  if ((threadIdx.x & 31) == 0) {
    sh.red[threadIdx.x >> 5] = m;
    sh.bottom[threadIdx.x >> 5] = least;
  }
  __syncthreads();
  m = sh.red[0];
#pragma unroll 1
  for (int w = 1; w < kFW; ++w) m = max_nan(m, sh.red[w]);
  return m;
}

// The row's largest logit where the list ran over; -inf logits aside, NaN or +inf as above.
template <typename T>
__device__ __noinline__ float row_max(const T* row, int V, Shared& sh) {
  float m = -INFINITY;
  RowSource<T>{row, V}.each([&](float l, int, int) { m = max_nan(m, l); });
  m = warp_max_nan(m);
  if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = sh.red[0];
  for (int w = 1; w < kFW; ++w) m = max_nan(m, sh.red[w]);
  return m;
}

// Leaves in the first CTA of the cluster, for which it returns true, the CTAs' lists as one, its size (sh.n, which
// may pass kListCap), and the CTAs' sums, largest logits and smallest keys (sh.rest, sh.most, sh.lowest).
__device__ bool join(const Slice& s, Shared& sh, unsigned long long rest, float most, uint32_t lowest) {
  const int rank = s.rank, split = s.split, tid = threadIdx.x;
  rest = warp_sum_u64(rest);
  most = warp_max_nan(most);
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  __syncthreads();  // sh.wsum and sh.red may still be read; the list is complete
  if ((tid & 31) == 0) {
    sh.wsum[tid >> 5] = rest;
    sh.red[tid >> 5] = most;
    sh.low[tid >> 5] = lowest;
  }
  __syncthreads();
  const uint32_t mine = smem_addr(&sh), first = dsmem_map(mine, 0);
  auto there = [&](const void* p) { return first + (smem_addr(p) - mine); };
  if (tid == 0) {
#pragma unroll 1
    for (int w = 1; w < kFW; ++w) {
      rest += sh.wsum[w];
      most = max_nan(most, sh.red[w]);
      lowest = min(lowest, sh.low[w]);
    }
    dsmem_st_u64(there(&sh.rest[rank]), rest);
    dsmem_st_f32(there(&sh.most[rank]), most);
    dsmem_st_u32(there(&sh.lowest[rank]), lowest);
  }
  if (rank != 0) {  // the first CTA's list may go on growing meanwhile
    const int n = sh.n;
    if (tid == 0) sh.at = static_cast<int>(dsmem_add_u32(there(&sh.n), static_cast<uint32_t>(n)));
    __syncthreads();
    const int at = sh.at;
#pragma unroll 1
    for (int i = tid; i < min(n, kListCap) && at + i < kListCap; i += kFT)
      dsmem_st_u32(there(&sh.id[at + i]), static_cast<uint32_t>(sh.id[i]));
  }
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  return rank == 0;
}

// Streams the row by its cluster: join() has the results, and the estimate is in sh.below of every CTA.
template <typename T, typename F>
__device__ bool stream_cluster(const T* row, int V, const Slice& s, Stream<T>& q, bool sum, int aim, float c,
                               Shared& sh, F&& floor_of) {
  unsigned long long rest = 0;
  const float below = sum ? stream<T, true>(row, V, s, q, aim, c, sh, floor_of, &rest)
                          : stream<T, false>(row, V, s, q, aim, c, sh, floor_of, &rest);
  if (threadIdx.x == 0) sh.below = below;
  return join(s, sh, rest, 0.f, 0xffffffffu);
}

// ---------------------------------------------------------------- filtered sampling

__device__ __forceinline__ bool load_filter(const FilterParams& q, int r, RowFilter& f) {
  f.t = q.temperature ? q.temperature[r] : q.temperature0;
  f.k = q.top_k ? q.top_k[r] : q.top_k0;
  f.p = q.top_p ? q.top_p[r] : q.top_p0;
  f.m = q.min_p ? q.min_p[r] : q.min_p0;
  f.u = q.uniforms[r];
  return (f.t == 0.f || (f.t >= kMinTemp && f.t <= kMaxTemp)) && f.k >= 0 && f.p > 0.f && f.p <= 1.f && f.m >= 0.f &&
         f.m <= 1.f && f.u >= 0.f && f.u < 1.f;
}

__device__ __forceinline__ void invalid_row(const FilterParams& q, int r, uint32_t err) {
  if (threadIdx.x != 0) return;
  q.tokens[r] = -1;
  if (q.thr) q.thr[r] = NAN;
  if (q.logp) q.logp[r] = NAN;
  atomicOr(q.err, err);
}

// ceil(p * total), at least 1: the units a nucleus has to reach.
__device__ __forceinline__ unsigned long long nucleus_units(float p, unsigned long long total) {
  bool rem;
  const unsigned long long n = share_floor(p, total, rem);
  return n + (rem || n == 0 ? 1ull : 0ull);
}

// The key of the smallest float32 at or above M + T ln(min_p), M itself for min_p = 1.  close(x, margin) says
// whether a logit of the row lies within margin of x: only then does it take more than float32 to tell (float64
// operations are few and slow on this chip).
template <typename C>
__device__ uint32_t min_p_key(float M, const RowFilter& f, C&& close) {
  if (f.m == 1.f) return fkey(M);
  const float down = __fmul_rn(f.t, logf(f.m)), x = M + down;
  if (!close(x, 1e-6f * (fabsf(M) - 2.f * down))) return fkey(x);
  return fkey(__double2float_ru(static_cast<double>(M) + static_cast<double>(f.t) * log(static_cast<double>(f.m))));
}

// What the rests of sh.rest[] (weights relative to the logit `low`, in 2^-30) are worth, and by how much that may
// be off, in units u = 2^-24 of it.  A weight 2^-y carries three roundings of y (y ln2 u each), and the mean of y
// under weights that sum to S is at most log2(V / S) (w log2(1 / w) is concave in w); the exponential's 2^-22;
// up to 16 additions before a compensated one, and two of those.  The scaling here adds 5 u, its own logarithm
// less than that, weights too small for the threads' roundings to 2^-30 less than V 2^-45 + 2^-20 of the
// weight of `low`.
__device__ __forceinline__ void rest_bounds(const Shared& sh, int split, float low, const Weight& weight, int V,
                                            unsigned long long* least, unsigned long long* most) {
  unsigned long long rest = 0;
#pragma unroll 1
  for (int i = 0; i < split; ++i) rest += sh.rest[i];
  const unsigned long long one = weight(low);
  const float sum = __fmul_rn(__ull2float_rn(rest), 1.f / kRestOne);
  const float scaled = __fmul_rn(sum, __ull2float_rn(one));
  const unsigned long long mid = __float2ull_rn(scaled);
  const float mean = fmaxf(0.f, __log2f(static_cast<float>(V)) - __log2f(fmaxf(sum, 1e-9f)));
  const float units = 2.1f * mean + 34.f;
  const unsigned long long err =
      __float2ull_ru(__fmul_ru(scaled, __fmul_ru(units, 5.9604645e-8f))) + V + (one >> 20) + 1;
  *least = mid > err ? mid - err : 0ull;
  *most = mid + err;
}

// drawn; selection over the whole row; a second pass; one for the exact total alone; another list
enum Next { kDone, kWhole, kSecond, kTotal, kAgain };

// Starts the copy of a row into the L2, 16 KB a thread.
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* row, int V) {
  constexpr int kBytes = 16384;
  const int head = RowSource<T>::head_of(row, V), bytes = (V - head) / Elems<T>::kVec * 16;
  const char* body = reinterpret_cast<const char*>(row + head);
  for (int at = threadIdx.x * kBytes; at < bytes; at += kFT * kBytes) prefetch_l2(body + at, min(kBytes, bytes - at));
}

// Places the second pass of a nucleus that ends below the list: a sample of the row's logits below `low` says
// between which values the share phi of their weight is reached.  The bracket takes about kBracketAim logits of
// the row around that point.  False if the sample cannot say.
template <typename T>
__device__ bool place_bracket(const T* row, int V, float low, float phi, const Weight& weight, float t, Shared& sh) {
  constexpr int kV = Elems<T>::kVec;
  const int tid = threadIdx.x;
  const int head = RowSource<T>::head_of(row, V), nv = (V - head) / kV, step = max(1, nv / (kProbe * kFT));
  const uint4* r4 = reinterpret_cast<const uint4*>(row + head);
  unsigned int* mass = sh.hist.lo;
  unsigned int* count = sh.hist.mid;
  __syncthreads();
  for (int i = tid; i < kListBins; i += kFT) mass[i] = count[i] = 0u;
  __syncthreads();
  // bins of the distance from `low`, 24 T in all (below that a weight is 2^-34 of its own)
  const float bins = __fdividef(static_cast<float>(kListBins), 24.f * t);
  int seen = 0;
#pragma unroll 1
  for (int i = 0; i < kProbe; i += 4) {
    uint4 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int v = ((i + u) * kFT + tid) * step;
      const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
      r[u] = v < nv ? __ldg(r4 + v) : make_uint4(none, none, none, none);
      seen += v < nv;
    }
    if (i == 0) prefetch_row(row, V);  // for the pass itself
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[kV];
      Elems<T>::widen(r[u], f);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const float d = low - f[j];
        const int bin = d > 0.f ? static_cast<int>(fminf(d * bins, 1e6f)) : kListBins;
        if (bin < kListBins) {
          atomicAdd(mass + bin, __float2uint_rn(fast_exp2(-d * weight.c_hi) * 16384.f));  // 2^18 of them fit a word
          atomicAdd(count + bin, 1u);
        }
      }
    }
  }
  unsigned long long n = seen, total;
  block_scan(n, sh.wsum, &n);
  const unsigned int m0 = mass[2 * tid], m1 = mass[2 * tid + 1];
  const unsigned long long incl = block_scan(m0 + m1, sh.wsum, &total);
  const unsigned long long target = __float2ull_rn(phi * __ull2float_rn(total));
  unsigned long long below;
  if (tid == 0) sh.at = -1;
  __syncthreads();
  const int mine = locate(m0, m1, incl, target, &below);
  if (mine >= 0) sh.at = mine;
  __syncthreads();
  const int centre = sh.at;
  if (centre < 0 || n == 0) return false;
  // one thread widens it, bin by bin, to the sample's share of kBracketAim
  if (tid == 0) {
    const float share = __fdividef(static_cast<float>(n * kV), static_cast<float>(V));
    const int want = max(1, static_cast<int>(kBracketAim * share));
    int a = centre, b = centre, got = static_cast<int>(count[centre]);
    bool up = true;
    while (got < want && (a > 0 || b < kListBins - 1)) {
      if ((up && a > 0) || b == kListBins - 1)
        got += static_cast<int>(count[--a]);
      else
        got += static_cast<int>(count[++b]);
      up = !up;
    }
    sh.key_hi = fkey(low - __fdividef(static_cast<float>(a), bins));
    sh.key_lo = fkey(low - __fdividef(static_cast<float>(b + 1), bins));
  }
  __syncthreads();
  return sh.key_lo < sh.key_hi;
}

// Cuts and draws a row from its list, or says what will where the list does not hold all that decides the row: a
// second pass (sh.key_lo, sh.key_hi; kTotal where the bounds of the total leave two candidates), another list
// (sh.aim, if this one was the first), or the whole row.  total: the row's exact weight, 0 where it is not known.
template <typename T>
__device__ Next sample_from_list(const T* row, int V, const Weight& weight, const RowFilter& f, Shared& sh,
                                 const RowOut& out, int split, int aim, bool again, unsigned long long total) {
  const int tid = threadIdx.x;
  const float M = weight.M;
  const bool k = f.k > 0 && f.k < V;
  if (sh.n > kListCap) {  // only min-p alone tells its cut all the same
    if (f.t == 0.f || k || f.p < 1.f) {
      if (tid == 0) sh.aim = max(1, static_cast<int>(static_cast<float>(aim) * kListAim / sh.n));
      return again ? kWhole : kAgain;
    }
    const uint32_t key = min_p_key(M, f, [](float, float) { return true; });
    if (tid == 0) sh.key_lo = sh.key_hi = key;
    __syncthreads();
    return kSecond;
  }
  const ListSource src{sh.val, sh.id, sh.n};
  const uint32_t hi = fkey(M);
  const bool complete = sh.below == -INFINITY;                     // the list holds every finite logit of the row
  const uint32_t lo = complete ? kKeyNegInf + 1 : fkey(sh.below);  // and all logits from here up anyway
  auto units = [&](float, int i) { return sh.w[i]; };
  float bottom = sh.bottom[0];
#pragma unroll 1
  for (int w = 1; w < kFW; ++w) bottom = fminf(bottom, sh.bottom[w]);
  const ValueBins bins(M, bottom);
  uint32_t tau = lo;
  bool cut = complete;  // every logit of the row at or above tau is on the list
  if (f.t == 0.f) {
    tau = hi;
    cut = true;
  } else if (k) {
    if (f.k < src.n) {
      const Hist counts{sh.hist.lo, nullptr, nullptr};
      counts.zero<kFT>(kListBins);
      src.each([&](float l, int, int) { counts.add(bins(l), 1ull); });
      __syncthreads();
      tau = cut_list<false>(src, bins, lo, hi, f.k, units, sh).key;
    }
    if (f.k > src.n && !complete) {
      if (f.k > kListCap - 600) return kWhole;
      if (tid == 0) sh.aim = min(V, static_cast<int>(static_cast<float>(aim) * (f.k + 300) / max(src.n, 1)));
      return again ? kWhole : kAgain;
    }
    cut = true;
  }
  // the weights, and a nucleus's masses
  const bool nucleus = f.t != 0.f && f.p < 1.f;
  const Hist masses{sh.hist.lo, sh.hist.mid, sh.hist.hi};
  if (nucleus) masses.zero<kFT>(kListBins);
  unsigned long long mass = 0;
#pragma unroll 1
  for (int i = tid; i < src.n; i += kFT) {
    const float l = sh.val[i];
    const unsigned long long w = weight(l);
    sh.w[i] = w;
    if (nucleus && fkey(l) >= tau) {
      mass += w;
      masses.add(bins(l), w);
    }
  }
  bool beyond = false;  // the nucleus ends below the list
  float phi = 0.f;
  if (nucleus) {
    block_scan(mass, sh.wsum, &mass);
    unsigned long long least = 0, most = 0;  // of what the list leaves out of the total
    if (!cut && total != 0)
      least = most = total - mass;
    else if (!cut)
      rest_bounds(sh, split, sh.below, weight, V, &least, &most);
    const unsigned long long need = nucleus_units(f.p, mass + least), need_most = nucleus_units(f.p, mass + most);
    if (need_most <= mass) {
      const CutResult c = cut_list<true>(src, bins, tau, hi, need, units, sh);
      if (need_most > c.above + c.at) return kTotal;
      tau = c.key;
      cut = true;
    } else {
      if (need <= mass) return kTotal;
      beyond = true;  // unless min-p cuts higher
      phi = __fdividef(__ull2float_rn(need - mass), __ull2float_rn(most + 1));
    }
  }
  if (f.t != 0.f && f.m > 0.f) {
    const uint32_t key = min_p_key(M, f, [&](float x, float margin) {
      int near = 0;
      src.each([&](float l, int, int) { near |= fabsf(l - x) <= margin; });
      return __syncthreads_or(near || fabsf(sh.below - x) <= margin) != 0;
    });
    cut = cut || key >= lo;
    if (beyond && !cut && key > kKeyNegInf + 1) return kWhole;  // two cuts below the list
    tau = max(tau, key);
  }
  if (!cut && beyond) return place_bracket(row, V, sh.below, phi, weight, f.t, sh) ? kSecond : kWhole;
  if (!cut) return kWhole;
  draw_from_list(src, tau, weight, f, sh, row, V, out);
  return kDone;
}

// The same over the whole row: exact selection, several passes over it by one CTA.
template <typename T>
__device__ __noinline__ void sample_from_row(const T* row, int V, const Weight& weight, const RowFilter& f, Shared& sh,
                                             const RowOut& out) {
  const RowSource<T> src{row, V};
  const float M = weight.M;
  const uint32_t hi = fkey(M);
  uint32_t tau = kKeyNegInf + 1;
  auto units = [&](float l, int) { return weight(l); };
  if (f.t == 0.f) {
    tau = hi;
  } else {
    if (f.k > 0 && f.k < V) {
      unsigned long long n = 0;
      src.each([&](float l, int, int) { n += fkey(l) >= tau; });
      block_scan(n, sh.wsum, &n);
      if (static_cast<unsigned long long>(f.k) < n) tau = select_key<false, kBins>(src, tau, hi, f.k, units, sh).key;
    }
    if (f.p < 1.f) {
      unsigned long long total = 0;
      src.each([&](float l, int, int) { total += fkey(l) >= tau ? units(l, 0) : 0ull; });
      block_scan(total, sh.wsum, &total);
      // 33 T below the largest logit a weight is below 2^-47, no unit
      const uint32_t lo = fkey(__fsub_rd(M, __fmul_ru(33.f, f.t)));
      tau = max(tau, select_key<true, kBins>(src, max(tau, lo), hi, nucleus_units(f.p, total), units, sh).key);
    }
    if (f.m > 0.f) tau = max(tau, min_p_key(M, f, [](float, float) { return true; }));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kGroups; i += kFT) sh.draw.group[i] = 0ull;
  if (threadIdx.x == 0) sh.least = 0xffffffffu;
  __syncthreads();
  unsigned int least =
      sum_groups(row, V, 0, (V + kGroup - 1) / kGroup, tau, weight, f.u, dsmem_map(smem_addr(sh.draw.group), 0));
  least = __reduce_min_sync(0xffffffffu, least);
  if ((threadIdx.x & 31) == 0) atomicMin(&sh.least, least);
  __syncthreads();
  draw_from_row(row, V, tau, weight, f, sh, sh.least, out);
}

// The cluster's second pass: exact weights of the logits from key_hi up into the first CTA's groups, and, for a
// nucleus (key_lo < key_hi), those between into its list.  The first CTA cuts and draws; false where the bracket
// does not hold the nucleus's end or the bounds of the total leave two candidates (sh.next, sh.key_lo, sh.key_hi: what
// to do about it).  total: the row's exact weight, 0 where it is not known.  sums: the group sums alone are wanted, by
// the first CTA (true there).
template <typename T>
__device__ bool second_pass(const T* row, int V, const Slice& s, uint32_t key_lo, uint32_t key_hi,
                            const Weight& weight, const RowFilter& f, Shared& sh, const RowOut& out,
                            unsigned long long total = 0, bool sums = false) {
  const int tid = threadIdx.x;
  const int groups = (V + kGroup - 1) / kGroup, per = (groups + s.split - 1) >> (__ffs(s.split) - 1);
  const int g0 = min(groups, s.rank * per), g1 = min(groups, g0 + per);
  const uint32_t to = dsmem_map(smem_addr(sh.draw.group), 0);
  const bool nucleus = key_lo < key_hi;
  unsigned long long rest = 0;
  unsigned int least = 0xffffffffu;
  if (nucleus)
    rest = bracket_groups(row, V, g0, g1, key_float(key_lo), key_float(key_hi), weight, sh, to);
  else
    least = sum_groups(row, V, g0, g1, key_hi, weight, sums ? 1.f : f.u, to);  // (a total has no units for u = 0)
  if (!join(s, sh, rest, 0.f, least)) return !sums;
  if (sums) return true;
  uint32_t lowest = sh.lowest[0], tau = key_hi;
#pragma unroll 1
  for (int i = 1; i < s.split; ++i) lowest = min(lowest, sh.lowest[i]);
  if (nucleus) {
    if (sh.n > kListCap) return false;
    const ListSource src{sh.val, sh.id, sh.n};
    gather_list(row, V, sh);
    unsigned long long mass = 0, above = 0, left, most;
    const ValueBins bins(key_float(key_hi), key_float(key_lo));
    const Hist masses{sh.hist.lo, sh.hist.mid, sh.hist.hi};
    masses.zero<kFT>(kListBins);
#pragma unroll 1
    for (int i = tid; i < src.n; i += kFT) {
      const unsigned long long w = weight(sh.val[i]);
      sh.w[i] = w;
      mass += w;
      masses.add(bins(sh.val[i]), w);
    }
    block_scan(mass, sh.wsum, &mass);
    above = sh.draw.group[2 * tid] + sh.draw.group[2 * tid + 1];
    block_scan(above, sh.wsum, &above);
    rest_bounds(sh, s.split, key_float(key_lo), weight, V, &left, &most);
    if (total != 0) left = most = total - above - mass;
    const unsigned long long need = nucleus_units(f.p, above + mass + left);
    const unsigned long long need_most = nucleus_units(f.p, above + mass + most);
    if (need_most <= above || need > above + mass) {  // the sample was off: the window above, or below
      const float lo = key_float(key_lo), hi = key_float(key_hi), width = fmaxf(hi - lo, 1e-6f * fabsf(hi));
      if (tid == 0) {
        sh.key_lo = need_most <= above ? key_hi : fkey(lo - width);
        sh.key_hi = need_most <= above ? fkey(hi + width) : key_lo;
        sh.next = kSecond;
      }
      return false;
    }
    const bool unsure = need <= above || need_most > above + mass;
    CutResult c{0u, 0ull, 0ull};
    auto units = [&](float, int i) { return sh.w[i]; };
    if (!unsure) c = cut_list<true>(src, bins, key_lo, key_hi - 1, need - above, units, sh);
    if (unsure || need_most > above + c.above + c.at) {
      if (tid == 0) sh.next = kTotal;
      return false;
    }
    tau = lowest = c.key;
    // the kept part of the list into the groups
    const Hist more{sh.hist.lo, sh.hist.mid, sh.hist.hi};
    __syncthreads();
    more.zero<kFT>(kGroups);
    src.each([&](float l, int id, int i) {
      if (fkey(l) >= tau) more.add(id / kGroup, draw_unit(sh.w[i], l, weight, f.u));
    });
    __syncthreads();
    sh.draw.group[2 * tid] += more.get(2 * tid);
    sh.draw.group[2 * tid + 1] += more.get(2 * tid + 1);
    __syncthreads();
  }
  draw_from_row(row, V, tau, weight, f, sh, lowest, out);
  return true;
}

// A row without filters: the largest logit and the smallest finite one, by its cluster.  The second pass finds the
// row in the L2.
template <typename T>
__device__ void scan_row(const T* row, int V, const Slice& s, Shared& sh) {
  float m = -INFINITY;
  unsigned int least = 0xffffffffu;
  auto one = [&](float l) {
    m = max_nan(m, l);
    if (l > -INFINITY) least = min(least, fkey(l));
  };
  const uint4* r4 = reinterpret_cast<const uint4*>(row + s.head);
  constexpr int kV = Elems<T>::kVec;
#pragma unroll 4
  for (int v = s.v0 + threadIdx.x; v < s.v1; v += kFT) {
    float f[kV];
    Elems<T>::widen(__ldg(r4 + v), f);
#pragma unroll
    for (int j = 0; j < kV; ++j) one(f[j]);
  }
  if (s.rank == 0 && threadIdx.x < s.head) one(Elems<T>::one(row, threadIdx.x));
  const int k = s.head + s.nv * kV + threadIdx.x;
  if (s.rank == s.split - 1 && k < V) one(Elems<T>::one(row, k));
  if (s.split > 1) cluster_wait_acquire();
  join(s, sh, 0, m, least);
}

// The batch, a cluster of CTAs per row.  Bound: for many rows DRAM while they stream (four CTAs
// per SM with 64 KB of loads in flight together), then the chain of barriers of a row's list (some 25000 cycles: gather, weights, cut, draw), which
// the SM's other rows cover, and the second pass of the last rows, which nothing covers (130000 to 200000 cycles).
// Measured: 1280 x 152064 float32, top-p 0.9 to 0.95, 303 to 360 us (2.2 to 2.6 TB/s; one row in twenty takes a second
// pass; 196 us, 4.0 TB/s, where none does); the same rows with top-k and top-p 196 us; 64 x 128256 bf16 with mixed
// filters 43 to 59 us; 333 x 50001 float32, min-p, 33.4 us; 8 x 32128 bf16 16 us.
template <typename T>
__global__ void __launch_bounds__(kFT, 4) sample_filtered_kernel(FilterParams q) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int split = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int r = blockIdx.x >> (__ffs(split) - 1), V = q.V, tid = threadIdx.x;
  const T* row = static_cast<const T*>(q.logits) + static_cast<size_t>(r) * V;
  RowFilter f;
  const bool valid = load_filter(q, r, f);
  const Slice s = slice_of(row, V, rank, split);
  if (!index_ok(r < q.R && split <= kMaxSplit && (V + kGroup - 1) / kGroup <= kGroups)) return;
  Stream<T> first(row, s);
  const float2 entry = exp2_table_entry();
  if (tid == 0) sh.n = 0;
  if (tid < 64) sh.tab[tid] = entry;
  for (int i = tid; i < kGroups; i += kFT) sh.draw.group[i] = 0ull;
  if (!valid) {
    if (rank == 0) invalid_row(q, r, kErrArg);
    return;
  }
  if (split > 1) cluster_arrive_release();  // the first CTA's counters are set before another CTA adds to them
  if (V <= kListCap) __syncthreads();       // (longer rows: the estimate has barriers)
  const RowOut out{q.tokens + r, q.thr ? q.thr + r : nullptr, q.logp ? q.logp + r : nullptr};
  Weight weight{0.f, 0.f, 0.f, sh.tab};
  if (f.t == 0.f)
    f.u = 0.f;  // the first of the largest logits
  else
    weight_scale(f.t, weight.c_hi, weight.c_lo);
  const bool k = f.k > 0 && f.k < V, only_min_p = f.t != 0.f && !k && f.p == 1.f;
  const bool unfiltered = only_min_p && f.m == 0.f && V > kListCap;
  // min-p alone: no logit below the sampled maximum's cut can be kept, whatever the row's maximum is
  auto floor_of = [&](float estimate, float sampled_max) {
    if (!only_min_p) return estimate;
    const float down = __fmul_rn(f.t, logf(f.m));  // two roundings and the logarithm's two
    return sampled_max + down - 1e-6f * (fabsf(sampled_max) - down);
  };
  int aim = f.t == 0.f ? 64 : k ? min(max(800, min(f.k, kListCap) + 256), 1300) : kListAim;
  for (bool again = false;; again = true) {
    if (unfiltered)
      scan_row(row, V, s, sh);
    else
      stream_cluster(row, V, s, first, f.t != 0.f && !k && f.p < 1.f, aim, weight.c_hi, sh, floor_of);
    Next next = kDone;
    if (rank == 0) {
      float M;
      if (unfiltered) {
        M = sh.most[0];
        for (int i = 1; i < split; ++i) M = max_nan(M, sh.most[i]);
      } else {
        M = sh.n <= kListCap ? gather_list(row, V, sh) : row_max(row, V, sh);
      }
      weight.M = M;
      if (!(M > -INFINITY && M < INFINITY)) {
        invalid_row(q, r, kErrNonfinite);
      } else if (unfiltered) {
        next = kSecond;
        if (tid == 0) sh.key_lo = sh.key_hi = kKeyNegInf + 1;
      } else {
        next = sample_from_list(row, V, weight, f, sh, out, split, aim, again, 0ull);
        if (next == kWhole) {
          sample_from_row(row, V, weight, f, sh, out);
          next = kDone;
        }
      }
    }
    __syncthreads();
    if (tid == 0) {
      if (rank == 0) {  // (the others get theirs from the first CTA)
        sh.next = next;
        sh.M = weight.M;
      }
      if (next != kTotal) sh.n = 0;  // (the first CTA's list stays)
    }
    __syncthreads();
    uint32_t key_lo, key_hi;
    int then;
    // the first CTA's decision to every CTA, into its own shared memory
    auto share_decision = [&]() {
      if (split > 1) {
        if (rank == 0 && tid < split) {
          const uint32_t mine = smem_addr(&sh), there = dsmem_map(mine, tid) - mine;
          dsmem_st_u32(there + smem_addr(&sh.next), static_cast<uint32_t>(sh.next));
          dsmem_st_u32(there + smem_addr(&sh.aim), static_cast<uint32_t>(sh.aim));
          dsmem_st_u32(there + smem_addr(&sh.key_lo), sh.key_lo);
          dsmem_st_u32(there + smem_addr(&sh.key_hi), sh.key_hi);
          dsmem_st_f32(there + smem_addr(&sh.M), sh.M);
        }
        __syncwarp();
        cluster_sync();
      }
      then = sh.next;
      aim = sh.aim;
      key_lo = sh.key_lo;
      key_hi = sh.key_hi;
      weight.M = sh.M;
    };
    share_decision();
    if (then == kDone) return;
    if (then == kTotal) {
      if (tid == 0 && rank != 0) sh.n = 0;
      __syncthreads();
      if (!second_pass(row, V, s, kKeyNegInf + 1, kKeyNegInf + 1, weight, f, sh, out, 0ull, true)) return;
      unsigned long long total = sh.draw.group[2 * tid] + sh.draw.group[2 * tid + 1];
      block_scan(total, sh.wsum, &total);
      if (sample_from_list(row, V, weight, f, sh, out, split, aim, true, total) != kDone)
        sample_from_row(row, V, weight, f, sh, out);
      return;
    }
    if (then == kSecond) {
      constexpr int kTries = 6;
      unsigned long long total = 0;
#pragma unroll 1
      for (int tries = 1;; ++tries) {
        if (then == kTotal) {
          second_pass(row, V, s, kKeyNegInf + 1, kKeyNegInf + 1, weight, f, sh, out, 0ull, true);
          if (rank == 0) {
            total = sh.draw.group[2 * tid] + sh.draw.group[2 * tid + 1];
            block_scan(total, sh.wsum, &total);
          }
          if (split > 1) cluster_sync();  // the sums are read
        }
        __syncthreads();
        if (tid == 0) sh.next = kDone;  // unless the pass says what else to do
        const bool done = second_pass(row, V, s, key_lo, key_hi, weight, f, sh, out, total);
        __syncthreads();
        then = sh.next;
        if (rank == 0 && !done && (then == kDone || sh.key_lo >= sh.key_hi || tries == kTries)) {
          sample_from_row(row, V, weight, f, sh, out);
          then = kDone;
        }
        __syncthreads();
        if (tid == 0) {
          sh.n = 0;
          if (rank == 0) sh.next = then;
        }
        __syncthreads();
        share_decision();
        if (then == kDone) return;
      }
    }
    if (split > 1) cluster_arrive_release();
    first = Stream<T>(row, s);
  }
}

// ---------------------------------------------------------------- top logits

// Descending bitonic sort of s[0, n2), n2 a power of two.
__device__ void sort_desc_u64(unsigned long long* s, int n2) {
  for (int size = 2; size <= n2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < n2 / 2; i += kFT) {
        const int lo = 2 * i - (i & (stride - 1));
        const int hi = lo + stride;
        const unsigned long long a = s[lo], b = s[hi];
        if (((lo & size) == 0) ? a < b : a > b) {
          s[lo] = b;
          s[hi] = a;
        }
      }
      __syncthreads();
    }
  }
}

// Sorts the logits above tau, and those equal to it up to token `last`, by value and then token, and writes
// the first K (m of them at most, m <= kBins); padding beyond.
template <typename S>
__device__ void write_top(const S& src, uint32_t tau, unsigned int last, int m, int K, Shared& sh, float* values,
                          int32_t* ids) {
  const int tid = threadIdx.x, warp_first = tid & ~31;
  int n2 = 1;
  while (n2 < m) n2 <<= 1;
  if (tid == 0) sh.at = 0;
  for (int i = tid; i < n2; i += kFT) sh.pairs[i] = 0ull;
  __syncthreads();
  src.each([&](float l, int id, int) {
    const uint32_t key = fkey(l);
    if (key > tau || (key == tau && static_cast<unsigned int>(id) <= last)) {
      const int at = atomicAdd(&sh.at, 1);
      if (at < m && index_ok(at < kBins)) sh.pairs[at] = (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - id);
    }
  });
  __syncthreads();
  if (m <= kFT) {  // every pair's place is the number of pairs above it
    const unsigned long long p = tid < m ? sh.pairs[tid] : 0ull;
    int place = 0;
    if (warp_first < m) {
#pragma unroll 4
      for (int j = 0; j < m; ++j) place += sh.pairs[j] > p;
    }
    if (tid < m && place < K) {
      values[place] = key_float(static_cast<uint32_t>(p >> 32));
      ids[place] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(p));
    }
    for (int i = m + tid; i < K; i += kFT) {
      values[i] = -INFINITY;
      ids[i] = -1;
    }
    return;
  }
  sort_desc_u64(sh.pairs, n2);
  for (int i = tid; i < K; i += kFT) {
    const unsigned long long p = i < n2 ? sh.pairs[i] : 0ull;
    values[i] = p ? key_float(static_cast<uint32_t>(p >> 32)) : -INFINITY;
    ids[i] = p ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(p)) : -1;
  }
}

// The K largest of the whole row by exact selection, several passes over it by one CTA.
template <typename T>
__device__ void top_from_row(const T* row, int V, float M, int K, Shared& sh, float* values, int32_t* ids) {
  const RowSource<T> src{row, V};
  uint32_t tau = kKeyNegInf + 1;
  unsigned int last = 0xffffffffu;  // of the logits equal to tau, tokens up to this one
  unsigned long long n = 0;
  src.each([&](float l, int, int) { n += l > -INFINITY; });
  block_scan(n, sh.wsum, &n);
  if (static_cast<unsigned long long>(K) < n) {
    auto one = [](float, int) { return 1ull; };
    const CutResult c = select_key<false, kBins>(src, tau, fkey(M), K, one, sh);
    tau = c.key;
    // the tokens at tau in ascending order: two digits of nine bits
    const Hist counts{sh.row_hist.lo, nullptr, nullptr};
    unsigned long long left = K - c.above;
    counts.zero<kFT>(512);
    src.each([&](float l, int id, int) {
      if (fkey(l) == tau) counts.add(511 - (id >> 9), 1ull);
    });
    __syncthreads();
    const Pick a = pick_from_top<kFT>(counts, 512, left, sh.wsum, &sh.pick);
    const int hi = 511 - a.bin;
    left -= a.above;
    counts.zero<kFT>(512);
    src.each([&](float l, int id, int) {
      if (fkey(l) == tau && (id >> 9) == hi) counts.add(511 - (id & 511), 1ull);
    });
    __syncthreads();
    const Pick b = pick_from_top<kFT>(counts, 512, left, sh.wsum, &sh.pick);
    last = hi * 512 + (511 - b.bin);
  }
  write_top(src, tau, last, static_cast<int>(min(n, static_cast<unsigned long long>(K))), K, sh, values, ids);
}

// The K largest logits from the list (ranked by counting for up to kFT of them, sorted beyond) and the log-sum-exp from
// the list's exact weights and the stream's float32 sum of the rest.  Bound as above.  Measured: top 64 of 1536 x
// 152064 float32 209 us (4.5 TB/s; 6 TB/s while the rows stream); top 20 of 5 x 32000 12.9 us.
template <typename T>
__global__ void __launch_bounds__(kFT, 4) top_logits_kernel(TopParams q) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int split = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int r = blockIdx.x >> (__ffs(split) - 1), tid = threadIdx.x;
  const int K = q.K, V = q.V;
  const T* row = static_cast<const T*>(q.logits) + static_cast<size_t>(r) * V;
  const Slice s = slice_of(row, V, rank, split);
  if (!index_ok(r < q.R && split <= kMaxSplit && (V + kGroup - 1) / kGroup <= kGroups)) return;
  Stream<T> first(row, s);
  const float2 entry = exp2_table_entry();
  if (tid == 0) sh.n = 0;
  if (split > 1) cluster_arrive_release();  // the first CTA's counters are set before another CTA adds to them
  if (V <= kListCap) __syncthreads();       // (longer rows: the estimate has barriers)
  float* values = q.values + static_cast<size_t>(r) * K;
  int32_t* ids = q.ids + static_cast<size_t>(r) * K;
  Weight weight{0.f, 0.f, 0.f, sh.tab};
  weight_scale(q.temperature, weight.c_hi, weight.c_lo);
  if (tid < 64) sh.tab[tid] = entry;
  int aim = min(max(800, K + 256), 1300);
  for (bool again = false;; again = true) {
    stream_cluster(row, V, s, first, q.lse != nullptr, aim, weight.c_hi, sh,
                   [](float estimate, float) { return estimate; });
    // a list that ran over or is too short is made once more
    const bool bad = sh.n > kListCap || (sh.n < K && sh.below > -INFINITY);
    int then = bad && !again;
    const int wanted = sh.n < K ? K + 300 : max(kListAim, K + 300);
    aim = max(1, static_cast<int>(static_cast<float>(aim) * wanted / max(sh.n, 1)));
    if (split > 1) {
      if (rank == 0 && tid == 0) {
        sh.next = then;
        sh.aim = aim;
      }
      __syncthreads();
      cluster_sync();
      const uint32_t mine = smem_addr(&sh), there = dsmem_map(mine, 0) - mine;
      then = static_cast<int>(dsmem_ld_u32(there + smem_addr(&sh.next)));
      aim = static_cast<int>(dsmem_ld_u32(there + smem_addr(&sh.aim)));
      __syncwarp();
      cluster_sync();
    }
    if (!then) break;
    __syncthreads();
    if (tid == 0) sh.n = 0;
    __syncthreads();
    if (split > 1) cluster_arrive_release();
    first = Stream<T>(row, s);
  }
  if (rank != 0) return;
  const int n = sh.n;
  const bool all = n <= kListCap;  // the list holds every logit from the estimate up
  const ListSource src{sh.val, sh.id, n};
  const float below = sh.below;
  const float M = all ? gather_list(row, V, sh) : row_max(row, V, sh);
  if (!(M > -INFINITY && M < INFINITY)) {
    for (int i = tid; i < K; i += kFT) {
      values[i] = NAN;
      ids[i] = -1;
    }
    if (tid == 0 && q.lse) q.lse[r] = NAN;
    return;
  }
  weight.M = M;
  if (q.lse) {
    unsigned long long total = 0;
    if (all)
      src.each([&](float l, int, int) { total += weight(l); });
    else
      RowSource<T>{row, V}.each([&](float l, int, int) { total += weight(l); });
    block_scan(total, sh.wsum, &total);
    if (tid == 0) {
      if (all && below > -INFINITY) {
        unsigned long long rest = 0;
        for (int i = 0; i < split; ++i) rest += sh.rest[i];
        const float sum = __fmul_rn(__ull2float_rn(rest), 1.f / kRestOne);
        total += __float2ull_rn(__fmul_rn(sum, __ull2float_rn(weight(below))));
      }
      // M / T and its remainder, and ln of the sum relative to the largest weight
      const float s = __fdiv_rn(M, q.temperature);
      const float rest = log_weight(total) + __fdiv_rn(__fmaf_rn(-s, q.temperature, M), q.temperature);
      q.lse[r] = fabsf(s) < INFINITY ? s + rest : s;
    }
  }
  if (all && (n >= K || below == -INFINITY)) {
    uint32_t tau = kKeyNegInf + 1;
    unsigned long long m = n;
    if (K < n) {
      float bottom = sh.bottom[0];
#pragma unroll 1
      for (int w = 1; w < kFW; ++w) bottom = fminf(bottom, sh.bottom[w]);
      const ValueBins bins(M, bottom);
      const Hist counts{sh.hist.lo, nullptr, nullptr};
      __syncthreads();
      counts.zero<kFT>(kListBins);
      src.each([&](float l, int, int) { counts.add(bins(l), 1ull); });
      __syncthreads();
      const CutResult c = cut_list<false>(src, bins, tau, fkey(M), K, [](float, int) { return 1ull; }, sh);
      tau = c.key;
      m = c.above + c.at;
    }
    if (m <= kBins) {
      write_top(src, tau, 0xffffffffu, static_cast<int>(m), K, sh, values, ids);
      return;
    }
  }
  top_from_row(row, V, M, K, sh, values, ids);
}

}  // namespace

// CTAs per row: doubled while the batch gives at most `most` CTAs and a CTA is left kLeastSlice logits.
static int row_split(int R, int V, int most) {
  int split = 1;
  while (split < kMaxSplit && 2LL * R * split <= most && V / (2 * split) >= kLeastSlice) split *= 2;
  return split;
}

template <typename P>
static cudaError_t launch_rows(void (*kernel)(P), std::atomic<unsigned long long>& prepared, const P& p, int split,
                               cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(prepared.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)));
    if (e != cudaSuccess) return e;
    prepared.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.R) * split);
  cfg.blockDim = dim3(kFT);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

#ifdef SPEC_DEBUG_BOUNDS
cudaError_t filtered_bounds(uint32_t* word) { return take_row_bounds(word); }
#endif

// Sampling: up to 27 CTAs per eight SMs (513 on 152), since a row's second pass is the faster the more CTAs share it
// (rows of 128256 with mixed filters: 64 of them 63 us with eight CTAs per row, 81 with two, 134 with one; 150 75 us
// with four, 132 with one), while the others wait as the first one finishes its list (top-k and top-p: 100 rows 26 us
// with one or two, 28 with four, 44 with eight; 250 rows 33 with one, 42 with two).
cudaError_t sample_filtered_launch(const FilterParams& p, int dtype, cudaStream_t stream) {
  static std::atomic<unsigned long long> f32{0}, bf16{0};
  const int split = row_split(p.R, p.V, 27 * (p.sms > 0 ? p.sms : 152) / 8);
  return dtype == 0 ? launch_rows(sample_filtered_kernel<float>, f32, p, split, stream)
                    : launch_rows(sample_filtered_kernel<__nv_bfloat16>, bf16, p, split, stream);
}

// Top logits: up to two CTAs per SM (150 rows of 128256, top 64: 24.5 us with two CTAs per row, 31.8 with four; 250
// rows: 30.4 with one, 35.7 with two; one row: 13.9 with eight, 20.8 with one).
cudaError_t top_logits_launch(const TopParams& p, int dtype, cudaStream_t stream) {
  static std::atomic<unsigned long long> f32{0}, bf16{0};
  const int split = row_split(p.R, p.V, 2 * (p.sms > 0 ? p.sms : 152));
  return dtype == 0 ? launch_rows(top_logits_kernel<float>, f32, p, split, stream)
                    : launch_rows(top_logits_kernel<__nv_bfloat16>, bf16, p, split, stream);
}

}  // namespace specv
