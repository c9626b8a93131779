// Sampling: one token of each row of logits, drawn with a given number u from
// the softmax at temperature T, cut to the top k, to the nucleus of mass p and to
// the tokens that have min_p of the best one's probability.
//
// Weights are integers, w(x) = 2^39 exp((x - max) / T) rounded: off by half a unit, 2^-40
// of the best token's weight, and by 2^-29 of themselves before that rounding (2^-31 near the
// best token, 2^-30 down to 2^-10 of its weight).  Sums of them are exact whatever their order, so that
// the cut and the token are those of the definition unless a weight is that near to
// min_p, or a sum over n tokens within 2^-29 of itself and n 2^-40 of its border with u or p,
// and results do not depend on how a row is split.
// (With sums of 32-bit exponentials, 1e-6 off, one row in ten of a large
// vocabulary would draw a neighbour.)
//
// One cluster per row: its CTAs hold the row in shared memory, brought once by
// bulk copies, and every later pass reads it there.
//   maximum     as the copies arrive; T = 0 ends with its lowest place.
//   top k       a histogram of counts over kBins steps of x below the maximum, the
//               bin that the k-th token falls into; k of a few hundred at most:
//               the tokens down to that bin are listed and the first CTA does the
//               rest on the list.  Otherwise the bin is refined until it holds a
//               list of tokens or a single value.
//   nucleus     the same with sums of weights.
//   draw        the CTA that u falls into by the CTAs' sums, then sums of the kept
//               tokens' weights by groups of 32 vectors, the group and the token.
// Equal values are taken by their index where the cut passes among them.
//
// Measured on GB300: 192 rows of 128001 bf16 logits, nucleus of 0.95, 160 us (0.31 TB/s of the
// logits read; 24 us to the maximum, 40 for every token's weight and bin, the rest
// in cluster barriers, the refined bin and the draw); 8 rows of 50257 fp32 without
// filters 9.5 us, one of 32000 f16 with all 12.1: latency of the barriers.

#include <cfloat>
#include <climits>

#include "dv_kernels.h"
#include "tc_common.cuh"

namespace dv {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 256;                 // tokens ranked against each other: one a thread
constexpr int kChunks = 8;                 // bulk copies of a CTA's part of the row
constexpr int kMaxCluster = 16;
constexpr int kMaxGroups = kSampleMaxV * 4 / 16 / kMaxCluster / 32 + 2;   // groups of 32 vectors, at most
constexpr int kUnit = 39;                  // a weight of 1 is 2^39
constexpr float kReach = 28.5f;            // exp(-28.5) 2^39 < 1/4: nothing below weighs anything
constexpr float kCold = 1e-30f, kHot = 1e30f;
constexpr long long kUnwindNs = 2000000000LL;
static_assert(kList <= kThreads && kBins % kThreads == 0, "a thread to a listed token, whole bins to a thread");

// 2^(31 + j / 512), rounded, from square roots of 2.
constexpr int kPowerCount = 512;
struct Powers {
  uint32_t v[kPowerCount];
};
constexpr double root_of(double a) {
  double x = 1.0 + (a - 1.0) / 2;
  for (int i = 0; i < 40; ++i) x = (x + a / x) / 2;
  return x;
}
constexpr Powers make_powers() {
  Powers p{};
  double root[9] = {};                     // 2^(1/2), 2^(1/4), ...
  double a = 2.0;
  for (int i = 0; i < 9; ++i) root[i] = a = root_of(a);
  for (int j = 0; j < kPowerCount; ++j) {
    double x = 2147483648.0;               // 2^31
    for (int i = 0; i < 9; ++i)
      if (j >> (8 - i) & 1) x *= root[i];
    p.v[j] = (uint32_t)(x + 0.5);
  }
  return p;
}
__device__ constexpr Powers kPowers = make_powers();

__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);   // (-0 as 0)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// The weight of x below the maximum m: y = (x - m) log2(e) / T as the sum of two
// floats (exact difference, product with log2(e) / T in two floats), 2^y as a 32-bit
// table entry times 1 + z, |z| < 2^-10.5, and a shift.
struct Scale {
  float m, hi, lo;   // hi + lo = log2(e) / T
  const uint32_t* table;
  // 2^31 times the mantissa of the weight, in [1, 2) but for rounding, and its shift
  __device__ __forceinline__ uint32_t mantissa(float x, int* shift, float* at) const {
    const float d = __fsub_rn(x, m), b = __fsub_rn(d, x);
    const float e = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));   // x - m = d + e
    const float y = __fmul_rn(d, hi);
    const float below = __fmaf_rn(d, lo, __fmaf_rn(e, hi, __fmaf_rn(d, hi, -y)));
    constexpr float kMagic = 24576.f;               // 1.5 2^14: sums are multiples of 2^-9
    const float t = __fadd_rn(fmaxf(y, -41.f), kMagic);
    const int k = __float_as_int(t) - __float_as_int(kMagic);   // y = k / 512 + r, |r| <= 2^-10
    const float r = __fsub_rn(y, __fsub_rn(t, kMagic));
    const float q = __fmul_rn(r, 0.69314718056f);
    const float s = __fmul_rn(__fmul_rn(q, q), __fmaf_rn(q, __fmaf_rn(q, 1.f / 24, 1.f / 6), 0.5f));
    // r ln 2 in one product and the rest of it with the small terms: 2^-24 of 2^-10.5
    const float z = __fmaf_rn(r, 0.69314718056f, __fmaf_rn(below, 0.69314718056f, __fmaf_rn(r, -1.9046542e-9f, s)));
    const uint32_t base = table[k & (kPowerCount - 1)];
    const float near = __uint_as_float(0x3f800000u | ((base >> 8) & 0x007fffffu));   // 2^(j/512)
    // base (1 + z) as a whole number below 2^32 (the product, below 2^22, becomes one by 1.5 2^23)
    constexpr float kWhole = 12582912.f;
    const float zi = __fmaf_rn(__fmul_rn(z, 2147483648.f), near, kWhole);
    const uint32_t w = base + (uint32_t)(__float_as_int(zi) - __float_as_int(kWhole));
    *shift = -(k >> 9);
    *at = y;
    return w;
  }
  __device__ __forceinline__ u64 operator()(float x) const {
    int shift;
    float y;
    const uint32_t w = mantissa(x, &shift, &y);
    // w 2^8 >> shift, rounded
    const u64 out = shift > 8 ? (u64)(((w >> min(shift - 9, 31)) + 1) >> 1) : (u64)w << (8 - shift);
    return y >= -40.f ? out : 0;                    // (NaN: x is -inf, or so far below that y is)
  }
  // Nothing below this weighs `least` or more: what is rounded to it weighs least - 1/2 at
  // least (1e-4 to the safe side).
  __device__ __forceinline__ float floor_of(u64 least) const {
    if (least == 0) return -INFINITY;
    const float y = log2f(__ull2float_rn(2 * least - 1)) - (kUnit + 1 + 1e-3f);   // < 0
    return m + (y * 1.0001f / hi - fabsf(m) * 1e-6f);
  }
};

// v f in whole numbers, f in [0, 1), rounded up or down: exact (double precision is slow
// on this GPU: with targets, log2(e) / T and floors in it, by every thread, 192 rows
// of 128001 took 310 us).
__device__ __forceinline__ u64 times(u64 v, float f, bool up) {
  if (!(f > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(f);
  const int e = bits >> 23;
  const uint32_t mant = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;   // f = mant 2^-shift
  const int shift = 150 - (e ? e : 1);                                            // 24 to 149
  const u64 lo = v * mant, hi = __umul64hi(v, mant);                              // hi below 2^24
  u64 out, rest;
  if (shift < 64) {
    out = (hi << (64 - shift)) | (lo >> shift);
    rest = lo << (64 - shift);
  } else {
    out = shift < 128 ? hi >> (shift - 64) : 0;
    rest = lo | (shift < 128 ? hi & ((1ull << (shift - 64)) - 1) : hi);
  }
  return out + (up && rest ? 1 : 0);
}

// Where the order (x descending, then index) is cut: kept are tokens before and
// at (key, index).
struct Cut {
  uint32_t key;
  int index;   // in the row's vectors; a CTA's own where the cut is among equal values
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

struct Shared {
  uint32_t table[kPowerCount];
  u64 group[kMaxGroups];       // sums of 32 vectors
  u64 box[2][kMaxCluster][2];  // what the cluster's CTAs tell each other
  u64 answer[3];               // what a thread tells all
  u64 list[kList];             // (key, lower index first)
  u64 weight[kList], sorted[kList];
  uint32_t count[kBins], carry[kBins];   // a histogram: counts, or weights as count + 2^32 carry
  uint32_t kmin[kBins], kmax[kBins];     // the keys in a bin
  float dense[kWarps][256];    // a group's tokens that a pass looks at, and their places in it
  uint8_t place[kWarps][256];
  u64 scan[kWarps];
  float redm[kWarps];
  int redi[kWarps];
  uint64_t full[kChunks];
  u64 rest;
  uint32_t listed[2];
  int found, late;
};

__device__ __forceinline__ uint32_t remote(const void* local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::saddr(local)), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_remote(u64* local, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(local, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_remote(const uint32_t* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add_remote(uint32_t* local, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote(local, rank)), "r"(v) : "memory");
  return old;
}

// All threads of the cluster meet, with what they have written to each other.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}

// Sum over a warp of values of 2^42 at most.
__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x1fffffu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 21));
  return ((u64)hi << 21) + lo;
}
// Inclusive sum over the block's threads; *total: all of it.  Two barriers.
__device__ __forceinline__ u64 block_scan(u64 v, u64* tmp, u64* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  __syncthreads();
  if (lane == 31) tmp[wid] = v;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < wid) before += tmp[w];
    all += tmp[w];
  }
  *total = all;
  return v + before;
}

template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);   // tokens of a vector
  Shared& sh;
  const uint8_t* part;     // the CTA's vectors
  int v0, vecs;            // its first one, and how many
  uint32_t rank, size;     // in the cluster
  int turn = 0;            // exchanges so far

  __device__ __forceinline__ void open(int v, float* f) const {
    unpack<T>(*reinterpret_cast<const uint4*>(part + (size_t)v * 16), f);
  }
  // Every CTA's two values, in box[turn of this call].
  __device__ __forceinline__ int exchange(u64 a, u64 b) {
    const int t = turn++ & 1;
    if (threadIdx.x < size) {
      st_remote(&sh.box[t][rank][0], threadIdx.x, a);
      st_remote(&sh.box[t][rank][1], threadIdx.x, b);
    }
    cluster_sync();
    return t;
  }
  // Tokens of group g (of 32 vectors) above -inf, from `floor` to `top`, side by side in the
  // warp's buffer; returns their number.  What is done with a token costs 40 instructions,
  // and a nucleus holds few of a group's: done where they are, every warp would run
  // them for all.
  __device__ __forceinline__ int pack(int g, float floor, float top) const {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, v = g * 32 + lane;
    float x[E];
    uint32_t takes = 0;
    if (v < vecs) {
      open(v, x);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (x[e] >= floor && x[e] <= top && x[e] > -INFINITY) takes |= 1u << e;
    }
    const uint32_t any = __reduce_or_sync(0xffffffffu, takes);
    if (!any) return 0;
    int n = 0;
    __syncwarp();   // (the buffer's last readers)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (!(any >> e & 1)) continue;
      const bool take = takes >> e & 1;
      const uint32_t hit = __ballot_sync(0xffffffffu, take);
      if (take) {
        const int at = n + __popc(hit & ((1u << lane) - 1));
        sh.dense[wid][at] = x[e];
        sh.place[wid][at] = (uint8_t)(lane * E + e);
      }
      n += __popc(hit);
    }
    __syncwarp();
    return n;
  }
  // f(x, index) of every token of the CTA above -inf, from `floor` to `top`
  template <typename F>
  __device__ __forceinline__ void each(float floor, float top, F f) const {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    for (int g = wid; g * 32 < vecs; g += kWarps) {
      const int n = pack(g, floor, top);
      for (int i = lane; i < n; i += 32) f(sh.dense[wid][i], (v0 + g * 32) * E + sh.place[wid][i]);
    }
  }
  // The same where nearly all tokens count and little is done with them.
  template <typename F>
  __device__ __forceinline__ void each_of_all(F f) const {
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
      float x[E];
      open(v, x);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (x[e] > -INFINITY) f(x[e]);
    }
  }
  // The bin that holds the `target`-th unit (of count or weight) of the
  // histogram that all CTAs have filled, what is before it and in it, and its keys (kKeys);
  // kBins if there is less in all.  Every CTA adds the cluster's bins for itself: one barrier.  No
  // CTA may clear its bins before the cluster's next one.
  struct Found {
    int bin;
    u64 before, inside;
    uint32_t klo, khi;
    u64 target;   // less what is before the bin
    u64 mine;     // this CTA's share of what is before
  };
  // target_of: the target, of the sum of all bins
  template <bool kMass, bool kKeys, typename F>
  __device__ __forceinline__ Found crossing(F target_of) {
    constexpr int kPer = kBins / kThreads;
    cluster_sync();   // the histograms are complete
    u64 sum = 0, bin[kPer], total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) bin[k] = 0;
#pragma unroll 4
    for (uint32_t r = 0; r < size; ++r)
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        bin[k] += ld_remote(&sh.count[threadIdx.x * kPer + k], r);
        if (kMass) bin[k] += (u64)ld_remote(&sh.carry[threadIdx.x * kPer + k], r) << 32;
      }
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += bin[k];
    u64 at = block_scan(sum, sh.scan, &total) - sum;
    const u64 target = target_of(total);
    if (total < target) return Found{kBins, 0, 0, 0, 0, 0, 0};   // (the same in every thread of the cluster)
    if (at < target && target <= at + sum) {   // one thread
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (at < target && target <= at + bin[k]) {
          sh.answer[0] = threadIdx.x * kPer + k;
          sh.answer[1] = at;
          sh.answer[2] = bin[k];
        }
        at += bin[k];
      }
    }
    __syncthreads();
    Found f{(int)sh.answer[0], sh.answer[1], sh.answer[2], 0, 0, target - sh.answer[1], 0};
    if (kKeys) {
      const uint32_t r = threadIdx.x & 31;
      f.klo = __reduce_min_sync(0xffffffffu, r < size ? ld_remote(&sh.kmin[f.bin], r) : 0xffffffffu);
      f.khi = __reduce_max_sync(0xffffffffu, r < size ? ld_remote(&sh.kmax[f.bin], r) : 0u);
    }
    sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = threadIdx.x * kPer + k;
      if (i < f.bin) sum += kMass ? ((u64)sh.carry[i] << 32) + sh.count[i] : sh.count[i];
    }
    (void)block_scan(sum, sh.scan, &f.mine);
    return f;
  }
  __device__ __forceinline__ void clear_bins() {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      sh.count[i] = sh.carry[i] = sh.kmax[i] = 0;
      sh.kmin[i] = 0xffffffffu;
    }
    __syncthreads();
  }
  template <bool kMass>
  __device__ __forceinline__ void add_bin(int b, u64 w) {
    if (!kMass) {
      atomicAdd(&sh.count[b], 1u);
    } else {
      const uint32_t lo = (uint32_t)w, old = atomicAdd(&sh.count[b], lo);
      const uint32_t up = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
      if (up) atomicAdd(&sh.carry[b], up);
    }
  }
  __device__ __forceinline__ void add_key(int b, uint32_t key) {
    atomicMin(&sh.kmin[b], key);
    atomicMax(&sh.kmax[b], key);
  }
  // Tokens that `take` into every CTA's list, their number into the first CTA's
  // listed[which], 0 before.
  template <typename F>
  __device__ __forceinline__ void gather(int which, float floor, float top, F take) {
    each(floor, top, [&](float x, int i) {
      if (!take(x, i)) return;
      const uint32_t at = add_remote(&sh.listed[which], 0, 1);
      if (at < (uint32_t)kList)
        for (uint32_t r = 0; r < size; ++r) st_remote(&sh.list[at], r, ((u64)ord32(x) << 32) | (uint32_t)~i);
    });
    cluster_sync();
  }
  // The group of 32 vectors, in order, that the sum `left` falls into: the first
  // whose sum up to and with it is above `left`; *left becomes what is left in it.
  // Some group's is.  Two barriers or more.
  __device__ __forceinline__ int locate(u64* left) {
    constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
    const int groups = (vecs + 31) / 32;
    u64 sum = 0, unused;
    if (threadIdx.x == 0) sh.found = groups;   // (behind the last)
#pragma unroll
    for (int q = 0; q < kPer; ++q) sum += (int)threadIdx.x * kPer + q < groups ? sh.group[threadIdx.x * kPer + q] : 0;
    const u64 upto = block_scan(sum, sh.scan, &unused);
    if (upto > *left && upto - sum <= *left) {
      u64 at = upto - sum;
      int g = threadIdx.x * kPer;
      while (at + sh.group[g] <= *left) at += sh.group[g++];
      sh.found = g;
      sh.rest = *left - at;
    }
    __syncthreads();
    *left = sh.rest;
    return sh.found;
  }
};

// Bins of x below the maximum, `step` to a unit.
struct Bins {
  float m, step;
  __device__ __forceinline__ uint32_t of(float x) const { return __float2uint_rz((m - x) * step); }
  // Bounds of bin b's x: difference, product and quotient are rounded (2^-23 together, and the
  // differences here outwards).
  __device__ __forceinline__ float low(int b) const { return __fsub_rd(m, (float)(b + 1) / step * 1.000001f); }
  __device__ __forceinline__ float high(int b) const { return b ? __fsub_ru(m, (float)b / step * 0.999999f) : m; }
};

__device__ __forceinline__ float listed_x(u64 entry) { return unord32((uint32_t)(entry >> 32)); }

// The cut of the order at the unit of count or weight that `target_of` names, of the sum
// of those that `have` keeps; `have` itself if they hold less.  `first`: the answer of the
// histogram over `bins`, if it is known.  (Its bins have no keys: with two more atomic
// operations a token 192 rows of 128001 took 160.6 us instead of 158.5.)
// *mine: the weight of this CTA's tokens that the cut keeps (kMass).
template <bool kMass, typename T, typename F>
__device__ __forceinline__ Cut find_cut(Row<T>& row, const Scale& weigh, Cut have, const Bins& bins, F target_of,
                                        const typename Row<T>::Found* first, u64* mine) {
  Shared& sh = row.sh;
  typename Row<T>::Found f;
  if (first) {
    f = *first;
  } else {
    row.clear_bins();
    const auto count = [&](float x) {
      const uint32_t b = bins.of(x);
      const u64 w = kMass ? weigh(x) : 1;
      if (b < (uint32_t)kBins && w) row.template add_bin<kMass>((int)b, w);
    };
    if (have.key == 0) {
      row.each_of_all(count);
    } else {
      row.each(unord32(have.key), weigh.m, [&](float x, int i) {
        if (have.keeps(ord32(x), i)) count(x);
      });
    }
    f = row.template crossing<kMass, false>(target_of);
    if (f.bin == kBins) {   // (a weight's target is never above the sum)
      *mine = 0;
      return have;
    }
  }
  u64 before = 0;             // of what is left
  const u64 target = f.target;
  *mine = f.mine;
  // the tokens that are left: those `have` keeps in the bin, with keys in [f.klo, f.khi]
  const uint32_t bin = f.bin;
  f.klo = ord32(bins.low(bin));
  f.khi = ord32(bins.high(bin));
  for (bool exact = false;; exact = true) {
    if (exact && f.klo == f.khi) break;   // one value
    const float low_x = unord32(f.klo), high_x = unord32(f.khi);
    // how many there are, at most: their weight over the least of them
    const u64 least = kMass ? weigh(low_x) : 1;
    if (least > 0 && f.inside <= (u64)kList * least) {
      row.gather(kMass, low_x, high_x, [&](float x, int i) {
        return bins.of(x) == bin && have.keeps(ord32(x), i) && (!kMass || weigh(x) != 0);
      });
      // (no CTA ends before the cluster's next barrier: the draw has one)
      const int n = min((int)ld_remote(&sh.listed[kMass], 0), kList), i = threadIdx.x;
      if (i < n) sh.weight[i] = kMass ? weigh(listed_x(sh.list[i])) : 1;
      __syncthreads();
      if (i < n) {
        u64 at = before;
        for (int j = 0; j < n; ++j)
          if (sh.list[j] > sh.list[i]) at += sh.weight[j];
        if (at < target && target <= at + sh.weight[i]) sh.sorted[0] = sh.list[i];
      }
      __syncthreads();
      const u64 last = sh.sorted[0];
      const Cut cut{(uint32_t)(last >> 32), (int)~(uint32_t)last};
      if (kMass) {   // the CTA's own of them
        u64 kept = 0, all;
        const int index = i < n ? (int)~(uint32_t)sh.list[i] : -1;
        if (i < n && sh.list[i] >= last && index >= row.v0 * Row<T>::E && index < (row.v0 + row.vecs) * Row<T>::E)
          kept = sh.weight[i];
        (void)block_scan(kept, sh.scan, &all);
        *mine += all;
      }
      __syncthreads();
      return cut;
    }
    int shift = 0;
    while ((f.khi - f.klo) >> shift >= (uint32_t)kBins) ++shift;
    cluster_sync();   // the last histogram has been read
    row.clear_bins();
    row.each(low_x, high_x, [&](float x, int i) {
      const uint32_t k = ord32(x);
      if (bins.of(x) != bin || !have.keeps(k, i)) return;
      const u64 w = kMass ? weigh(x) : 1;
      if (!w) return;
      row.template add_bin<kMass>((int)((f.khi - k) >> shift), w);
      row.add_key((int)((f.khi - k) >> shift), k);
    });
    const u64 left = target - before;
    f = row.template crossing<kMass, true>([&](u64) { return left; });
    if (f.bin == kBins) return have;
    before += f.before;
    *mine += f.mine;
  }
  const uint32_t klo = f.klo;
  // equal values: the first r of them, by index
  const u64 one = kMass ? weigh(unord32(klo)) : 1;
  const u64 r = (target - before + one - 1) / one;
  const float value = unord32(klo);
  u64 here = 0, total;
  // (index order: a warp to a group of 32 vectors, as in the draw)
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, groups = (row.vecs + 31) / 32;
  for (int g = wid; g < groups; g += kWarps) {
    uint32_t n = 0;
    const int v = g * 32 + lane;
    if (v < row.vecs) {
      float x[Row<T>::E];
      row.open(v, x);
#pragma unroll
      for (int e = 0; e < Row<T>::E; ++e)
        n += x[e] == value && have.keeps(klo, (row.v0 + v) * Row<T>::E + e);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sh.group[g] = n;
    here += n;
  }
  (void)block_scan(lane == 0 ? here : 0, sh.scan, &total);
  const int t = row.exchange(total, 0);
  u64 ahead = 0;
  for (uint32_t q = 0; q < row.rank; ++q) ahead += sh.box[t][q][0];
  Cut cut{klo, -1};
  *mine += (ahead >= r ? 0 : min(total, r - ahead)) * one;
  if (ahead + total <= r) {
    cut.index = INT_MAX;
  } else if (ahead < r) {
    // the CTA's own (r - ahead)-th of them
    u64 left = r - ahead - 1;
    const int v = row.locate(&left) * 32 + lane;
    uint32_t n = 0, bits = 0;
    if (v < row.vecs) {
      float x[Row<T>::E];
      row.open(v, x);
#pragma unroll
      for (int e = 0; e < Row<T>::E; ++e)
        if (x[e] == value && have.keeps(klo, (row.v0 + v) * Row<T>::E + e)) bits |= 1u << e;
    }
    n = __popc(bits);
    uint32_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t m = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += m;
    }
    int index = -1;
    if (upto - n <= left && left < upto) {
      for (uint32_t skip = (uint32_t)left - (upto - n); skip; --skip) bits &= bits - 1;
      index = (row.v0 + v) * Row<T>::E + __ffs(bits) - 1;
    }
    cut.index = __reduce_max_sync(0xffffffffu, index);
  }
  // (a value equal to the cut's that `have` left out stays out: have's index is smaller there)
  if (have.key == cut.key) cut.index = min(cut.index, have.index);
  __syncthreads();
  return cut;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleLaunch a) {
  extern __shared__ __align__(128) uint8_t part[];
  __shared__ Shared sh;
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = blockIdx.x % a.split;
  const int b = blockIdx.x / a.split;
  for (int i = tid; i < kPowerCount; i += kThreads) sh.table[i] = kPowers.v[i];
  if (tid == 0) {
    for (int q = 0; q < kChunks; ++q) tc::mbar_init(&sh.full[q], 1);
    tc::fence_mbar_init();
    sh.listed[0] = sh.listed[1] = 0;
    sh.late = 0;
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  cluster_arrive();   // the others may write here from now on (waited for before the first exchange)
  // The row as 16-byte vectors from the boundary at or below its first token on;
  // the tokens of its first and last vector that are not the row's are -inf.
  const T* x0 = static_cast<const T*>(a.logits) + (size_t)b * a.ld;
  const int off = (int)((reinterpret_cast<uintptr_t>(x0) & 15u) / sizeof(T));
  const int all = (off + a.V + E - 1) / E;
  const char* base = reinterpret_cast<const char*>(x0 - off);
  const int v0 = min((int)rank * a.part_vecs, all), v1 = min(v0 + a.part_vecs, all), vecs = v1 - v0;
  const int whole0 = max(v0, off > 0 ? 1 : 0), whole1 = max(whole0, min(v1, (off + a.V) / E));  // copied
  const int chunk = (a.part_vecs + kChunks - 1) / kChunks;
  if (tid == 0)
    for (int q = 0; q < kChunks; ++q) {
      const int c0 = max(whole0, v0 + q * chunk), c1 = min(whole1, v0 + (q + 1) * chunk);
      const uint32_t bytes = c1 > c0 ? (uint32_t)(c1 - c0) * 16 : 0;
      tc::mbar_arrive_expect_tx(&sh.full[q], bytes);
      if (bytes) tc::bulk_g2s(part + (size_t)(c0 - v0) * 16, base + (size_t)c0 * 16, bytes, &sh.full[q]);
    }
  for (int i = tid; i < 2 * E; i += kThreads) {   // the ends
    const int v = i < E ? 0 : all - 1, t = v * E + i % E;   // token t - off
    const bool edge = v < whole0 || v >= whole1;
    if (v >= v0 && v < v1 && edge)
      reinterpret_cast<T*>(part)[(size_t)(v - v0) * E + i % E] =
          t >= off && t < off + a.V ? x0[t - off] : Elem<T>::from_f(-INFINITY);
  }
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const float u = a.u[b];
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f;
  const float min_p = a.min_p ? a.min_p[b] : 0.f;
  __syncthreads();
  Row<T> row{sh, part, v0, vecs, rank, (uint32_t)a.split};

  // ---- maximum
  float m = -INFINITY;
  bool bad = false;
  for (int q = 0; q < kChunks; ++q) {
    if (lane == 0 && !tc::mbar_wait_soon(&sh.full[q], 0, a.wait_ns)) {
      sh.late = 1;
      set_error(a.hdr, DV_ERR_TIMEOUT, 61);
    }
    __syncwarp();   // the other lanes read behind the first one's wait (a shuffle orders no memory)
    // (the first lane's look at it, the warp's: lanes that saw different values would part)
    if (__shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&sh.late), 0)) break;
    const int c1 = min(vecs, (q + 1) * chunk);
    for (int v = q * chunk + tid; v < c1; v += kThreads) {
      float f[E];
      row.open(v, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        bad |= !(f[e] <= FLT_MAX);   // a NaN or +inf
        m = fmaxf(m, f[e]);
      }
    }
  }
  m = warp_max(m);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.redm[wid] = m;
    sh.redi[wid] = bad;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    m = fmaxf(m, sh.redm[w]);
    bad |= sh.redi[w] != 0;
  }
  bad |= sh.late != 0;
  if (sh.late && tid == 0)   // no copy may be in flight when the CTA ends
    for (int q = 0; q < kChunks; ++q)
      if (!tc::mbar_wait(&sh.full[q], 0, kUnwindNs > a.wait_ns ? kUnwindNs : a.wait_ns)) break;
  __syncwarp();
  cluster_wait();   // every CTA of the cluster has begun
  {
    const int t = row.exchange(__float_as_uint(m), bad ? 1 : 0);
    for (uint32_t r = 0; r < row.size; ++r) {
      m = fmaxf(m, __uint_as_float((uint32_t)sh.box[t][r][0]));
      bad |= sh.box[t][r][1] != 0;
    }
  }
  // (temperatures beyond kCold and kHot: log2(e) / T or a difference of logits leaves the range of fp32)
  bad |= !(m > -INFINITY) || !(temp == 0.f || (temp >= kCold && temp <= kHot)) || u != u || p != p || min_p != min_p;
  if (bad) {   // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      a.token[b] = -1;
      if (a.prob) a.prob[b] = 0.f;
      set_error(a.hdr, DV_ERR_INVALID_ARG, b);
    }
    cluster_sync();
    return;
  }

  if (temp == 0.f) {   // the best token, the first of equal ones
    int first = INT_MAX;
    row.each(m, m, [&](float x, int i) {
      if (x == m) first = min(first, i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.redi[wid] = first;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) first = min(first, sh.redi[w]);
    const int t = row.exchange((u64)(uint32_t)first, 0);
    for (uint32_t r = 0; r < row.size; ++r) first = min(first, (int)(uint32_t)sh.box[t][r][0]);
    if (rank == 0 && tid == 0) {
      a.token[b] = first - off;
      if (a.prob) a.prob[b] = 1.f;
    }
    cluster_sync();
    return;
  }

  Scale weigh;
  weigh.m = m;
  // log2(e) = 1.44269502 + 1.92596303e-8
  weigh.hi = __fdiv_rn(1.44269502f, temp);
  weigh.lo = __fdiv_rn(__fmaf_rn(-weigh.hi, temp, 1.44269502f) + 1.92596303e-8f, temp);
  weigh.table = sh.table;
  const Bins bins{m, (float)kBins / (kReach * temp)};
  const u64 least = min_p > 0.f ? __float2ull_ru(fminf(min_p, 1.f) * (float)(1ull << kUnit)) : 0;
  const auto mass_target = [&](u64 mass) {   // tokens are kept while what is before them is below
    return max(times(mass, p, true), (u64)1);
  };
  const auto draw_target = [&](u64 mass) {   // the token whose sum is the first above
    return u < 1.f ? times(mass, u, false) : mass - 1;
  };
  const auto put = [&](float x, int i, u64 mass) {
    a.token[b] = i - off;
    if (a.prob) {
      int shift;
      float y;
      const double w = (double)weigh.mantissa(x, &shift, &y) * __hiloint2double((1023 + kUnit - 31 - shift) << 20, 0);
      a.prob[b] = (float)(w / (double)mass);
    }
  };
  Cut cut{0, INT_MAX};
  const bool has_k = k > 0 && k < a.V, has_p = p < 1.f;

  // ---- top k
  if (has_k) {
    row.clear_bins();
    row.each_of_all([&](float x) {
      const uint32_t bin = bins.of(x);
      if (bin < (uint32_t)kBins) row.template add_bin<false>((int)bin, 0);
    });
    const auto found = row.template crossing<false, false>([&](u64) { return (u64)k; });
    if (found.bin < kBins && found.before + found.inside <= (u64)kList) {
      // the few best tokens: one CTA does the rest
      row.gather(0, bins.low(found.bin), m, [&](float x, int) { return bins.of(x) <= (uint32_t)found.bin; });
      if (rank != 0) return;
      const int n = min((int)sh.listed[0], kList);
      u64 mine = 0, w = 0;
      int at = 0;
      if (tid < n) {
        mine = sh.list[tid];
        for (int j = 0; j < n; ++j) at += sh.list[j] > mine;
        w = weigh(listed_x(mine));
      }
      __syncthreads();
      if (tid < n) {
        sh.sorted[at] = mine;
        sh.weight[at] = at < k ? w : 0;
      }
      __syncthreads();
      u64 mass, v = tid < n ? sh.weight[tid] : 0;
      const u64 upto = block_scan(v, sh.scan, &mass);
      const bool keep = tid < n && tid < k && (!has_p || upto - v < mass_target(mass)) && v >= least;
      __syncthreads();
      if (tid < n) sh.weight[tid] = keep ? v : 0;
      (void)block_scan(keep ? v : 0, sh.scan, &mass);
      if (keep && v) {
        mine = sh.sorted[tid];
        u64 sum = 0;   // of the kept tokens up to this one by index
        for (int j = 0; j < n; ++j) sum += (uint32_t)~sh.sorted[j] <= (uint32_t)~mine ? sh.weight[j] : 0;
        const u64 t = draw_target(mass);
        if (sum > t && sum - v <= t) put(listed_x(mine), (int)~(uint32_t)mine, mass);
      }
      return;
    }
    u64 unused;
    if (found.bin == kBins)
      cluster_sync();   // fewer than k within reach: the bins have been read by all, and the nucleus may clear them
    else
      cut = find_cut<false>(row, weigh, cut, bins, [](u64 all) { return all; }, &found, &unused);
  }

  // ---- sums of groups of 32 vectors: kept tokens that weigh `low` at least
  const int groups = (vecs + 31) / 32;
  const auto sums = [&](u64 low, u64* total) {
    u64 mine = 0;
    const float floor_x = fmaxf(weigh.floor_of(low), cut.key ? unord32(cut.key) : -INFINITY);
    const bool every = floor_x == -INFINITY;
    for (int g = wid; g < groups; g += kWarps) {
      u64 w = 0;
      if (every) {
        const int v = g * 32 + lane;
        if (v < vecs) {
          float x[E];
          row.open(v, x);
#pragma unroll
          for (int e = 0; e < E; ++e) w += weigh(x[e]);
        }
      } else {
        const int n = row.pack(g, floor_x, m);
        for (int i = lane; i < n; i += 32) {
          const float x = sh.dense[wid][i];
          const u64 we = weigh(x);
          if (we >= low && cut.keeps(ord32(x), (v0 + g * 32) * E + sh.place[wid][i])) w += we;
        }
      }
      w = warp_sum_u64(w);
      if (lane == 0) sh.group[g] = w;
      mine += w;
    }
    (void)block_scan(lane == 0 ? mine : 0, sh.scan, total);
    __syncthreads();
  };

  // ---- nucleus
  u64 total, mass = 0, ahead = 0;
  if (has_p)
    cut = find_cut<true>(row, weigh, cut, bins, mass_target, (const typename Row<T>::Found*)nullptr, &total);

  // ---- draw
  const bool summed = !has_p || least > 0;   // (the nucleus knows every CTA's weight already)
  if (summed) sums(least, &total);
  const int t = row.exchange(total, 0);
  mass = 0;
  for (uint32_t r = 0; r < row.size; ++r) {
    if (r < rank) ahead += sh.box[t][r][0];
    mass += sh.box[t][r][0];
  }
  const u64 aim = draw_target(mass);
  if (aim < ahead || aim >= ahead + total) return;   // (nothing of this CTA is read by others any more)
  if (!summed) sums(0, &total);
  u64 left = aim - ahead;
  const int v = row.locate(&left) * 32 + lane;
  if (wid != 0) return;
  float x[E];
  u64 we[E], w = 0;
  if (v < vecs) row.open(v, x);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    we[e] = 0;
    if (v < vecs) {
      const u64 full = weigh(x[e]);
      if (full >= least && cut.keeps(ord32(x[e]), (v0 + v) * E + e)) we[e] = full;
    }
    w += we[e];
  }
  u64 run = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 n = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += n;
  }
  if (run > left && run - w <= left) {
    u64 at = run - w;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (at <= left && left < at + we[e]) put(x[e], (v0 + v) * E + e, mass);
      at += we[e];
    }
  }
}

template <typename T>
cudaError_t run_sample(const SampleLaunch& a, cudaStream_t stream) {
  static PerDevice attr;   // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return (int)e;
    return (int)cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(kSampleMaxV * sizeof(T) / kMaxCluster + 1024));
  });
  if (ea != cudaSuccess) return ea;
  return launch_k(sample_kernel<T>, dim3((unsigned)a.B * a.split), dim3(kThreads), (size_t)a.part_vecs * 16, stream, true,
                  a.split, a);
}

}  // namespace

cudaError_t launch_sample(const SampleLaunch& L, dv_dtype dt, WsHeader* hdr, int num_sms, cudaStream_t stream) {
  SampleLaunch a = L;
  a.hdr = hdr;
  a.wait_ns = wait_limit_ns();
  const long long es = dt == DV_F32 ? 4 : 2, bytes = a.V * es;
  // CTAs of a row: 64 KB of it each (two CTAs an SM; 192 rows of 128001 bf16: 160 us, with 32
  // KB 310, with 128 KB 178), and as long as that leaves half of the GPU idle, 8192
  // tokens (one row of 32000: 12.1 us; 4096: 12.9, 2048: 18.5; 8 of 50257: 9.2, 10.9, 10.7)
  int c = 1;
  while (c < kMaxCluster && bytes > (long long)c * 65536) c *= 2;
  while (c < kMaxCluster && (long long)a.B * c * 2 <= num_sms && a.V > c * 8192) c *= 2;
  a.split = c;
  const int E = (int)(16 / es), vecs = (a.V + 2 * E - 2) / E;
  a.part_vecs = ((vecs + c - 1) / c + 31) / 32 * 32;
  switch (dt) {
    case DV_F32: return run_sample<float>(a, stream);
    case DV_F16: return run_sample<__half>(a, stream);
    case DV_BF16: return run_sample<__nv_bfloat16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dv
