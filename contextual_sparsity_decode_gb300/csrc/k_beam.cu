// Beam selection: the K best continuations of a sequence over its W beams and
// the vocabulary,
//     score(w, v) = cum[w] + x[w][v] - logsumexp(x[w][:]),
// by score descending, ties to the lower w V + v.
//
// Within a beam the order is that of the logits themselves (the log-sum-exp is
// one number per row), so the selection inside a row is exact and needs no
// arithmetic; only the candidates of different beams are compared by score, in
// double precision (and those of a beam whose scores round to the same double by
// their logits).
//
// One pass over the logits of the beams that are not done (the floor: each is
// read once; 48 x 10 rows of 128001 bf16 logits with a fifth of the beams done
// are 98 MB, 14.4 us).
//   scan  a CTA walks a part of a row in tiles of kBeamTile tokens, which bulk
//         copies bring into a ring of shared memory: a running maximum and
//         compensated sum of exponentials per thread, and the groups of 8 tokens
//         (kThreads apart) whose maximum may be among the K largest: the K best
//         groups, by maximum and then its lowest token, hold the K best tokens
//         (each group left out is preceded by K tokens of others).  The threads'
//         running maxima give a value tau that K groups reach, sharper with
//         every tile; a group is listed if
//         its maximum is above the tau before its tile (an equal one comes
//         after K others) and reaches the one with it: about K / k groups of
//         tile k.  A list that grows long all the same is cut back.  At the
//         part's end the K best groups' tokens are read again and ranked.  No
//         sort, and one barrier a tile.
//   join  one CTA per sequence, launched while the scan runs: log-sum-exp of
//         the parts in double, then the K best of the parts' lists.
// -inf tokens are never listed: a part with fewer than K others adds its
// lowest ones, which lie among its first 2 K tokens.
// The tokens of a thread and the order of every sum depend on the token index
// alone, not on the row's address, so rows with equal logits get equal sums.

// Measured on GB300, both kernels: 48 x 10 rows of 128001 bf16 logits, a fifth of
// the beams done, 51.5 us (1.9 TB/s of the logits read; bound by instructions,
// 19.5 a token, and by uneven SMs); 8 x 8 of 50257 fp32 15.5 us, 4 of 32000 f16
// 7.5 us.

#include "dv_kernels.h"
#include "tc_common.cuh"

namespace dv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 2;                    // groups of 8 tokens per thread and tile
static_assert(kThreads * kGroups * 8 == kBeamTile, "tokens per tile");
constexpr int kLong = 64;                      // a warp's list longer than this: all are cut back
constexpr int kMine = kLong + 32 * kGroups;    // a warp's list: a tile's groups always fit behind
constexpr int kListed = kWarps * kMine;
static_assert(kListed >= kBeamMaxK * 8, "the best groups' tokens fit too");
static_assert(kBeamMaxK * kListed / kThreads <= 32 * kWarps, "what is left of a list is dealt out 32 to a warp");
constexpr int kFew = 256;                     // entries ranked against each other directly
constexpr int kJoinListed = 1024;
typedef unsigned long long u64;

// Order-preserving map of a float to unsigned (-0 as 0).
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ u64 key_of(float f, int v) { return ((u64)ord32(f) << 32) | (uint32_t)~v; }

// The r-th largest of a warp's values, equal ones counted singly; 0 where
// fewer are not 0.
__device__ __forceinline__ uint32_t warp_rth(uint32_t v, int r) {
  for (;;) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, v);
    r -= __popc(__ballot_sync(0xffffffffu, v == top));
    if (r <= 0 || top == 0) return top;
    if (v == top) v = 0;
  }
}
// A value that at least K of the block's values reach, not far below the K-th
// largest, in two steps: each warp's r-th largest, and the j-th largest of
// those, r j >= K (for K = 4 the fourth of the warps' maxima; the least of all
// warps' would let ten times as many values through).
struct Reach {
  int r, j;
  __device__ __forceinline__ explicit Reach(int K) {
    constexpr int kMost = kWarps - 1;
    r = (K + kMost - 1) / kMost;
    j = (K + r - 1) / r;
  }
  // a warp's share, to be stored in red[] by lane 0 ...
  __device__ __forceinline__ uint32_t share(uint32_t v) const { return warp_rth(v, r); }
  // ... and the answer, after a barrier; 0 where fewer values are not 0
  __device__ __forceinline__ uint32_t value(const uint32_t* red) const {
    const uint32_t mine = red[threadIdx.x % kWarps];
    int above = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) above += red[q] > mine;
    return __reduce_min_sync(0xffffffffu, above < j ? mine : ~0u);
  }
};
__device__ __forceinline__ uint32_t block_reached(uint32_t v, int K, uint32_t* red) {
  const Reach reach(K);
  const uint32_t t = reach.share(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
  __syncthreads();
  return reach.value(red);
}
// The r-th largest of the block's values; 0 where fewer are not 0.  Starts and
// ends with a barrier.
template <typename U>
__device__ __forceinline__ U block_rth(U v, int r, U* all, U* result) {
  __syncthreads();
  all[threadIdx.x] = v;
  if (threadIdx.x == 0) *result = ~U(0);
  __syncthreads();
  int above = 0;
#pragma unroll 8
  for (int q = 0; q < kThreads; ++q) above += all[q] > v;
  if (above < r) atomicMin(result, v);
  __syncthreads();
  return *result;
}

// A candidate of the join: its score as an order-preserving integer, and where
// it is.  Comparing integers keeps double-precision work, slow on this GPU, to
// the few that are listed.
// The tie orders equal scores: by beam, then by logit, larger first (scores that
// are equal in double precision may differ), then by token.
struct __align__(16) Cand {
  u64 key, tie;
};
static_assert(kBeamMaxWidth <= 1 << 10 && kBeamMaxV <= 1 << 22, "a tie: 10 bits of beam, 32 of logit, 22 of token");
__device__ __forceinline__ u64 tie_of(int w, float x, int v) {
  return ((u64)w << 54) | ((u64)~ord32(x) << 22) | (uint32_t)v;
}
__device__ __forceinline__ u64 ord64(double d) {
  const u64 u = (u64)__double_as_longlong(d + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double unord64(u64 o) {
  return __longlong_as_double((long long)((o >> 63) ? (o & 0x7fffffffffffffffull) : ~o));
}
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  return a.key != b.key ? a.key > b.key : a.tie < b.tie;
}

struct JoinRow {
  double base;  // log-sum-exp; an ended beam's score
  float cum;
  int kind;     // 0: the listed tokens, 1: every token at -inf, 2: ended
};

// Bounds of an entry's score in fp32: the score lies in [lo, hi] (three
// roundings of at most 2^-24 of the summed magnitudes).
__device__ __forceinline__ void join_bounds(const JoinRow& r, float x, bool ends, float* lo, float* hi) {
  if (ends) {
    *lo = *hi = (float)r.base;
  } else if (r.kind != 0 || x == -INFINITY) {
    *lo = *hi = -INFINITY;
  } else {
    const float lse = (float)r.base, f = r.cum + (x - lse);
    const float e = 0x1p-21f * (fabsf(r.cum) + fabsf(x) + fabsf(lse));
    *lo = f - e;
    *hi = f + e;
  }
}

__device__ __forceinline__ void put(const BeamLaunch& a, int s, int k, const Cand& c) {
  a.score[(size_t)s * a.K + k] = (float)unord64(c.key);
  a.token[(size_t)s * a.K + k] = (int)(c.tie & ((1u << 22) - 1));
  a.beam[(size_t)s * a.K + k] = (int)(c.tie >> 54);
}

// Cuts a list of n entries (0: none) back to those that reach the K-th largest
// of the thread maxima over it (the K-th largest entry where n <= kThreads);
// returns the new length, at most K ceil(n / kThreads).
__device__ __noinline__ int cut_back(u64* list, u64* kept, int n, int K, u64* all, u64* result, int* listed) {
  u64 best = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) best = list[i] > best ? list[i] : best;
  const u64 t = block_rth<u64>(best, K, all, result);
  if (threadIdx.x == 0) *listed = 0;
  __syncthreads();
  if (best && best >= t)
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (list[i] && list[i] >= t) kept[atomicAdd(listed, 1)] = list[i];
  __syncthreads();
  n = *listed;
  for (int i = threadIdx.x; i < n; i += kThreads) list[i] = kept[i];
  __syncthreads();
  return n;
}

// Token e of the group that token v (counted from the part's first) is in.
__device__ __forceinline__ int group_token(int v, int e) {
  constexpr int kSpan = 8 * kThreads;
  return v / kSpan * kSpan + v % kThreads + e * kThreads;
}

template <typename T>
struct Ring {
  static constexpr int kStages = sizeof(T) == 4 ? 3 : 4;
  static constexpr uint32_t kBytes = kBeamTile * sizeof(T) + 32;   // a tile, from and to 16-byte boundaries
};
constexpr long long kUnwindNs = 2000000000LL;
constexpr float kSlack = 1.f;   // exponents up to 1.44: their rounding stays within 2^-24

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) beam_scan_kernel(const BeamLaunch a) {
  constexpr int ST = Ring<T>::kStages;
  extern __shared__ __align__(16) uint8_t ring[];
  // keys (value, lower token first): of groups, by their maximum; of tokens
  __shared__ u64 list[kListed], kept[kListed];
  __shared__ u64 all[kThreads];
  __shared__ u64 rth;
  __shared__ uint64_t full[ST];
  __shared__ uint32_t red[2][kWarps];
  __shared__ float redm[kWarps], reds[kWarps];
  __shared__ int listed, found, stop[2];   // stop: by the tile's parity (a thread may be one barrier ahead)
  const int part = blockIdx.x, row = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    for (int q = 0; q < ST; ++q) tc::mbar_init(&full[q], 1);
    tc::fence_mbar_init();
    listed = stop[0] = stop[1] = 0;
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  if (a.done && a.done[row]) return;  // an ended beam's logits are not read
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.ld;
  const char* first = static_cast<const char*>(a.logits);
  const char* last = first + ((size_t)(a.S * a.W - 1) * a.ld + a.V) * sizeof(T);
  const uint32_t off = reinterpret_cast<uintptr_t>(x) & 15u;
  const int lo = part * a.part_tiles * kBeamTile, hi = min(a.V, lo + a.part_tiles * kBeamTile);
  const int tiles = (hi - lo + kBeamTile - 1) / kBeamTile;
  // Rows begin at any address.  Copies begin and end on 16-byte boundaries and
  // stay within the logits' memory [first, last); the few tokens at its very
  // ends that they cannot bring are stored one by one.
  const char* begin = reinterpret_cast<const char*>(x) - off;
  const int skip = begin < first ? 16 : 0;        // the first vector begins before the logits
  const long long room = (last - begin) & ~15LL;  // bytes of whole vectors from `begin` on
  const auto issue = [&](int k) {                 // tile k, by one thread
    const int t0 = lo + k * kBeamTile, n = min(kBeamTile, hi - t0);
    const long long b0 = (long long)t0 * sizeof(T);  // from `begin`: a multiple of 16
    const long long b1 = min((b0 + off + (long long)n * sizeof(T) + 15) & ~15LL, room);
    const int cut = b0 == 0 ? skip : 0;
    const uint32_t bytes = (uint32_t)max(0LL, b1 - b0 - cut);
    uint8_t* stage = ring + (k % ST) * Ring<T>::kBytes;
    T* tokens = reinterpret_cast<T*>(stage + off);
    if (cut)
      for (int e = 0; e < n && off + (e + 1) * sizeof(T) <= 16; ++e) tokens[e] = x[e];
    for (int e = n - 1; e >= 0 && b0 + off + (long long)(e + 1) * sizeof(T) > b1; --e) tokens[e] = x[t0 + e];
    // a stage that held tokens stored one by one, and was read by every thread
    // before the last barrier, is written by a copy: order the two kinds of access
    tc::fence_proxy_async();
    tc::mbar_arrive_expect_tx(&full[k % ST], bytes);
    if (bytes) tc::bulk_g2s(stage + cut, begin + b0 + cut, bytes, &full[k % ST]);
  };
  int issued = 0;
  if (tid == 0)
    while (issued < min(ST, tiles)) issue(issued++);
  __syncthreads();  // (tokens stored one by one)
  // the thread's maximum, and its sum of exponentials, sum - lost, relative to ref
  // (as long as there is none, to from = 0)
  float m = -INFINITY, ref = -INFINITY, from = 0.f, sum = 0.f, lost = 0.f, tau = -INFINITY;
  bool over = false;
  int mine = 0;   // entries of the warp's list
  const Reach reach(a.K);
  for (int k = 0; k < tiles; ++k) {
    const int v0 = lo + k * kBeamTile;
    if (lane == 0 && !tc::mbar_wait_soon(&full[k % ST], (k / ST) & 1, a.wait_ns)) {  // one lane polls
      stop[k & 1] = 1;
      set_error(a.hdr, DV_ERR_TIMEOUT, 51);
    }
    __syncwarp();
    const T* tile = reinterpret_cast<const T*>(ring + (k % ST) * Ring<T>::kBytes + off) + tid;
    float f[8 * kGroups];   // tokens v0 + tid + i kThreads
#pragma unroll
    for (int i = 0; i < 8 * kGroups; ++i) f[i] = Elem<T>::to_f(tile[i * kThreads]);
    if (v0 + kBeamTile > hi) {
#pragma unroll
      for (int i = 0; i < 8 * kGroups; ++i) f[i] = v0 + tid + i * kThreads < hi ? f[i] : -INFINITY;
    }
    float g8[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float* x8 = f + 8 * g;
      g8[g] = max3(max3(max3(x8[0], x8[1], x8[2]), x8[3], x8[4]), max3(x8[5], x8[6], x8[7]), -INFINITY);
    }
    const float top = fmaxf(g8[0], g8[1]);
    // The sum is kept relative to a reference that follows the thread's maximum
    // once it is kSlack above: scaled at every rise, the sum of a row that rises
    // slowly would gather an error with every tile.  The difference is taken
    // first: a logit may be the type's lowest value.  A NaN or +inf among the
    // tokens makes the sum a NaN.
    const float mn = fmaxf(m, top);
    const bool moved = mn > ref + kSlack;
    const float keep = moved ? ex2((ref - mn) * kLog2e) : 1.f;   // (0 from -inf: the sum was 0, or a NaN)
    ref = moved ? mn : ref;
    from = moved ? mn : from;
    u64 s2[2] = {0, 0};   // (two tokens an instruction: 52.5 us instead of 54.4 at 48 x 10 rows)
    const u64 minus_ref = pack2(-from, -from), log2e = pack2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < 8 * kGroups; i += 2) {
      float y0, y1;
      open2(mul2(add2(pack2(f[i], f[i + 1]), minus_ref), log2e), &y0, &y1);
      s2[(i >> 1) & 1] = add2(s2[(i >> 1) & 1], pack2(ex2(y0), ex2(y1)));
    }
    float s4[4];
    open2(s2[0], &s4[0], &s4[1]);
    open2(s2[1], &s4[2], &s4[3]);
    // Compensated: a part may have 1024 tiles, and a plain fp32 sum of a flat row
    // rounds the same way at each (1.2e-5 off in all); beams are compared by it.
    const float add = __fmaf_rn(-lost, keep, (s4[0] + s4[1]) + (s4[2] + s4[3]));
    const float old = sum * keep, next = __fadd_rn(old, add);
    lost = __fsub_rn(__fsub_rn(next, old), add);
    sum = next;
    m = mn;
    const bool sharpen = k < 4 || (k & 3) == 0;   // (the maxima change ever more slowly)
    if (sharpen) {
      const uint32_t wt = reach.share(m > -INFINITY ? ord32(m) : 0u);
      if (lane == 0) red[k & 1][wid] = wt;
    }
    const bool full_list = __syncthreads_or(over);
    // every thread has the tile in registers: its stage takes the next
    if (stop[k & 1]) break;
    if (tid == 0 && k + ST < tiles) issue(issued++);
    if (full_list) {
      for (int i = mine + lane; i < kMine; i += 32) list[wid * kMine + i] = 0;
      __syncthreads();
      const int n = cut_back(list, kept, kListed, a.K, all, &rth, &listed);
      tau = fmaxf(tau, unord32((uint32_t)(rth >> 32)));
      // dealt out again, 32 to a warp (n <= K kListed / kThreads)
      __syncthreads();
      mine = min(max(n - wid * 32, 0), 32);
      if (lane < mine) list[wid * kMine + lane] = kept[wid * 32 + lane];
      __syncwarp();
    }
    float now = tau;
    if (sharpen) {
      const uint32_t reached = reach.value(red[k & 1]);   // 0: fewer than K threads hold tokens
      if (reached) now = fmaxf(tau, unord32(reached));
    }
    static_assert(kGroups == 2, "two ballots");
    if (__any_sync(0xffffffffu, top > tau && top >= now)) {
      const uint32_t hit0 = __ballot_sync(0xffffffffu, g8[0] > tau && g8[0] >= now);
      const uint32_t hit1 = __ballot_sync(0xffffffffu, g8[1] > tau && g8[1] >= now);
      u64* at = list + wid * kMine + mine;
      const uint32_t below = (1u << lane) - 1;
      int i0 = 7, i1 = 15;   // the lowest tokens that hold the maxima
#pragma unroll
      for (int i = 6; i >= 0; --i) {
        if (f[i] == g8[0]) i0 = i;
        if (f[8 + i] == g8[1]) i1 = 8 + i;
      }
      if ((hit0 >> lane) & 1) at[__popc(hit0 & below)] = key_of(g8[0], v0 + tid + i0 * kThreads);
      if ((hit1 >> lane) & 1) at[__popc(hit0) + __popc(hit1 & below)] = key_of(g8[1], v0 + tid + i1 * kThreads);
      mine += __popc(hit0) + __popc(hit1);
    }
    over = mine > kLong;
    tau = now;
  }
  // No copy may be in flight when the CTA exits.  (Unless a wait gave up, all
  // have been waited for.)
  if (stop[0] | stop[1])
    for (int k = max(0, issued - ST); k < issued; ++k)
      if (!tc::mbar_wait(&full[k % ST], (k / ST) & 1, kUnwindNs > a.wait_ns ? kUnwindNs : a.wait_ns)) break;
  // the part's maximum and sum
  const float wm = warp_max(m);
  sum -= lost;
  const float ws = warp_sum(m > -INFINITY ? sum * ex2((ref - wm) * kLog2e) : sum != sum ? sum : 0.f);
  if (lane == 0) {
    redm[wid] = wm;
    reds[wid] = ws;
  }
  if (tid == 0) found = 0;
  __syncthreads();
  const size_t slot = (size_t)row * a.parts + part;
  if (wid == 0) {
    const float pm = lane < kWarps ? redm[lane] : -INFINITY, ps = lane < kWarps ? reds[lane] : 0.f;
    const float top = warp_max(pm);
    float t = pm > -INFINITY ? ps * ex2((pm - top) * kLog2e) : ps != ps ? ps : 0.f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) a.stat[slot] = make_float2(top, t);
  }
  // K groups reach tau, so the K best tokens do: those of the listed groups,
  // read again, each warp its own
  __syncwarp();
  for (int i = lane; i < 8 * mine; i += 32) {
    const u64 group = list[wid * kMine + (i >> 3)];
    if (unord32((uint32_t)(group >> 32)) < tau) continue;
    const int v = group_token(~(uint32_t)group - lo, i & 7) + lo;
    const float y = v < hi ? Elem<T>::to_f(x[v]) : -INFINITY;
    if (y > -INFINITY && y >= tau) {
      const int at = atomicAdd(&found, 1);
      if (at < kListed) kept[at] = key_of(y, v);
    }
  }
  __syncthreads();
  int n = found;
  if (n > kFew) {
    // many equal values: the K best groups by value and then the lower token,
    // then their tokens
    for (int i = mine + lane; i < kMine; i += 32) list[wid * kMine + i] = 0;
    __syncthreads();
    n = cut_back(list, kept, kListed, a.K, all, &rth, &listed);
    for (int i = tid; i < n; i += kThreads) {
      const u64 key = list[i];
      int rank = 0;
#pragma unroll 8
      for (int q = 0; q < n; ++q) rank += list[q] > key;
      if (rank < a.K) kept[rank] = key;
    }
    __syncthreads();
    n = min(n, a.K);
    for (int i = tid; i < n; i += kThreads) list[i] = kept[i];
    if (tid == 0) listed = 0;
    __syncthreads();
    for (int i = tid; i < 8 * n; i += kThreads) {
      const int v = group_token(~(uint32_t)list[i >> 3] - lo, i & 7) + lo;
      const float y = v < hi ? Elem<T>::to_f(x[v]) : -INFINITY;
      if (y > -INFINITY) kept[atomicAdd(&listed, 1)] = key_of(y, v);
    }
    __syncthreads();
    n = listed;
    if (n > kFew) n = cut_back(kept, list, n, a.K, all, &rth, &listed);
  }
  int2* out = a.cand + slot * a.K;
  for (int i = tid; i < n; i += kThreads) {
    const u64 key = kept[i];
    int rank = 0;
#pragma unroll 8
    for (int q = 0; q < n; ++q) rank += kept[q] > key;
    if (rank < a.K) out[rank] = make_int2(__float_as_int(unord32(key >> 32)), (int)~(uint32_t)key);
  }
  if (n < a.K && wid == 0) {  // the lowest tokens at -inf
    int k = n;
    for (int c = lo; c < min(hi, lo + 2 * a.K) && k < a.K; c += 32) {
      const int v = c + lane;
      const bool is = v < hi && Elem<T>::to_f(x[v]) == -INFINITY;
      const uint32_t ball = __ballot_sync(0xffffffffu, is);
      const int at = k + __popc(ball & ((1u << lane) - 1));
      if (is && at < a.K) out[at] = make_int2(__float_as_int(-INFINITY), v);
      k += __popc(ball);
    }
    for (k += lane; k < a.K; k += 32) out[k] = make_int2(0, -1);
  }
}

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamLaunch a) {
  __shared__ Cand list[kJoinListed];
  __shared__ JoinRow rows[kBeamMaxWidth];
  __shared__ float2 stat[kBeamMaxWidth];   // a row's maximum, and whether it holds a NaN or +inf
  __shared__ double sums[kBeamMaxWidth];
  __shared__ uint32_t red[kWarps];
  __shared__ Cand redc[kWarps];
  __shared__ int listed;
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int per_row = a.parts * a.K, total = a.W * per_row;
  constexpr int kHeld = 4;  // entries that a thread reads at once, and keeps if there are no more
  // entries are dealt out so that every warp gets its share of a short list
  const int first = lane * kWarps + wid;
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) listed = 0;
  // one round of reads: the rows' sums, their scores so far, and the lists
  float cum = 0.f;
  int ended = 0;
  if (tid < a.W) {
    cum = a.cum[s * a.W + tid];
    ended = a.done ? a.done[s * a.W + tid] : 0;
  }
  int2 held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = first + k * kThreads;
    held[k] = make_int2(0, -1);
    if (i < total) held[k] = __ldcg(&a.cand[(size_t)s * total + i]);
  }
  for (int q = wid; q < a.W; q += kWarps) {  // a warp to a row, a lane to a part
    const float2* st = a.stat + (size_t)(s * a.W + q) * a.parts;
    const float2 p0 = lane < a.parts ? __ldcg(&st[lane]) : make_float2(-INFINITY, 0.f);
    float M = p0.x;
    bool nan = p0.y != p0.y;
    for (int c = lane + 32; c < a.parts; c += 32) {
      const float2 p = __ldcg(&st[c]);
      nan |= p.y != p.y;
      M = fmaxf(M, p.x);
    }
    M = warp_max(M);
    nan = __any_sync(0xffffffffu, nan);
    double t = p0.y > 0.f ? (double)p0.y * (double)ex2((p0.x - M) * kLog2e) : 0.0;
    for (int c = lane + 32; c < a.parts; c += 32) {
      const float2 p = __ldcg(&st[c]);
      if (p.y > 0.f) t += (double)p.y * (double)ex2((p.x - M) * kLog2e);
    }
    int span = 32;
    while (span > 1 && span / 2 >= a.parts) span >>= 1;  // lanes that hold a part
    for (int o = span >> 1; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) {
      stat[q] = make_float2(M, nan ? 1.f : 0.f);
      sums[q] = t;
    }
  }
  __syncthreads();
  if (tid < a.W) {
    const bool open = cum > -INFINITY && cum < INFINITY;   // NaN and +inf count as -inf
    const float2 st = stat[tid];
    JoinRow j{0.0, cum, 1};
    if (ended) {
      // (at -inf its end token has no place before lower ones: kind 1)
      if (open) {
        j.kind = 2;
        j.base = (double)cum;
      }
    } else if (st.y == 0.f && st.x > -INFINITY && open) {
      j.kind = 0;
      j.base = (double)st.x + log(sums[tid]);
    }
    rows[tid] = j;
  }
  __syncthreads();
  // Entry i, with what was read of it: its beam, its token (-1: none) and its
  // logit.  A beam that lists nothing offers its K lowest tokens at -inf; an
  // ended beam's end token, at its score, takes its own place among them or
  // that of the last (*ends).
  const auto entry = [&](int i, const int2& p, int* w, float* x, bool* ends) {
    *w = i / per_row;
    const int e = i - *w * per_row, kind = rows[*w].kind;
    *x = -INFINITY;
    *ends = false;
    if (kind == 0) {
      *x = __int_as_float(p.x);
      return p.y;
    }
    if (e >= a.K) return -1;
    if (kind == 2 && (e == a.end || (e == a.K - 1 && a.end >= a.K))) {
      *ends = true;
      return a.end;
    }
    return e < a.V ? e : -1;
  };
  const auto read = [&](int i, int k) {
    return k < kHeld ? held[k < kHeld ? k : 0] : __ldcg(&a.cand[(size_t)s * total + i]);
  };
  // K scores reach t, so none of the K best has an upper bound below it
  uint32_t best = 0;
  const auto bound = [&](int i, const int2& p) {
    int w;
    float x, lo, hi;
    bool ends;
    if (entry(i, p, &w, &x, &ends) < 0) return;
    join_bounds(rows[w], x, ends, &lo, &hi);
    best = max(best, ord32(lo));
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (first + k * kThreads < total) bound(first + k * kThreads, held[k]);
  for (int i = first + kHeld * kThreads; i < total; i += kThreads) bound(i, read(i, kHeld));
  const uint32_t t = block_reached(best, a.K, red);
  // the candidate of an entry whose upper bound reaches t
  const auto candidate = [&](int i, const int2& p, Cand* c) {
    int w;
    float x, lo, hi;
    bool ends;
    const int v = entry(i, p, &w, &x, &ends);
    if (v < 0) return false;
    const JoinRow& r = rows[w];
    join_bounds(r, x, ends, &lo, &hi);
    if (ord32(hi) < t) return false;
    c->key = ord64(ends ? r.base : r.kind != 0 ? -INFINITY : (double)r.cum + ((double)x - r.base));
    c->tie = tie_of(w, x, v);
    return true;
  };
  const auto add = [&](int i, const int2& p) {
    Cand c;
    if (!candidate(i, p, &c)) return;
    const int at = atomicAdd(&listed, 1);
    if (at < kJoinListed) list[at] = c;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (first + k * kThreads < total) add(first + k * kThreads, held[k]);
  for (int i = first + kHeld * kThreads; i < total; i += kThreads) add(i, read(i, kHeld));
  __syncthreads();
  const int n = listed;
  if (n <= kJoinListed) {
    for (int i = tid; i < n; i += kThreads) {
      const Cand c = list[i];
      int rank = 0;
#pragma unroll 4
      for (int q = 0; q < n; ++q) rank += before(list[q], c);
      if (rank < a.K) put(a, s, rank, c);
    }
    return;
  }
  // more equal scores than the list holds: one more of the best each round
  Cand prev{~0ull, 0};
  for (int k = 0; k < a.K; ++k) {
    Cand top{0, ~0ull};
    for (int i = tid; i < total; i += kThreads) {
      Cand c;
      if (candidate(i, read(i, kHeld), &c) && before(prev, c) && before(c, top)) top = c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Cand d;
      d.key = __shfl_xor_sync(0xffffffffu, top.key, o);
      d.tie = __shfl_xor_sync(0xffffffffu, top.tie, o);
      if (before(d, top)) top = d;
    }
    if (lane == 0) redc[wid] = top;
    __syncthreads();
    top = redc[0];
#pragma unroll
    for (int q = 1; q < kWarps; ++q)
      if (before(redc[q], top)) top = redc[q];
    __syncthreads();
    if (tid == 0) put(a, s, k, top);
    prev = top;
  }
}

}  // namespace

namespace {

// Tiles of a part.  Time is taken to be that of the tiles on the busiest SM, a
// part's start and end costing about two more, and of a round's latency (about
// eight tiles) for every time the GPU is filled (`per_sm` CTAs an SM); the least
// is taken, fewer parts where equal.  The constants fit 480 rows of 128001 bf16
// logits (parts of 8, 11 and 32 tiles: 57, 53 and 58 us; of 16: 51.6).  CTAs
// that share an SM are counted as if they ran one after another, which is too
// much below about four: 64 rows of 50257 get two parts each, and latency, not
// the tiles, is what they take.
int part_tiles(int rows, int V, int num_sms, int per_sm) {
  const int tiles = (V + kBeamTile - 1) / kBeamTile;
  const long long slots = (long long)per_sm * num_sms;
  int best = tiles;
  long long least = -1;
  for (int parts = 1; parts <= tiles; parts += 1 + parts / 16) {  // long rows: coarser steps
    const int t = (tiles + parts - 1) / parts;
    const long long ctas = (long long)rows * ((tiles + t - 1) / t);
    const long long cost = (ctas + num_sms - 1) / num_sms * (t + 2) + 8 * ((ctas + slots - 1) / slots);
    if (least < 0 || cost < least) {
      least = cost;
      best = t;
    }
  }
  return best;
}

template <typename T>
cudaError_t run_beam(const BeamLaunch& a, cudaStream_t stream) {
  constexpr size_t smem = Ring<T>::kStages * Ring<T>::kBytes;
  static PerDevice attr;  // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(beam_scan_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (ea != cudaSuccess) return ea;
  const cudaError_t e = launch_k(beam_scan_kernel<T>, dim3(a.parts, a.S * a.W), dim3(kThreads), smem, stream, true, 1, a);
  if (e != cudaSuccess) return e;
  return launch_k(beam_join_kernel, dim3(a.S), dim3(kThreads), 0, stream, true, 1, a);
}

}  // namespace

cudaError_t launch_beam_select(const BeamLaunch& L, dv_dtype dt, WsHeader* hdr, int num_sms, cudaStream_t stream) {
  BeamLaunch a = L;
  a.hdr = hdr;
  a.wait_ns = wait_limit_ns();
  a.part_tiles = part_tiles(a.S * a.W, a.V, num_sms, dt == DV_F32 ? 3 : 4);
  a.parts = ((a.V + kBeamTile - 1) / kBeamTile + a.part_tiles - 1) / a.part_tiles;
  switch (dt) {
    case DV_F32: return run_beam<float>(a, stream);
    case DV_F16: return run_beam<__half>(a, stream);
    case DV_BF16: return run_beam<__nv_bfloat16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dv
