// Matrices in 4 bits (layout: k_q4.cu) with one or two vectors: products with
// rows of the matrix, and sums of listed rows, on the integer dot product of four
// bytes (dp4a).
//
// A word of eight codes is two registers of four bytes by a mask, and a shift and
// a mask.  Vectors and coefficients enter in fixed point below the largest of their group
// (of the CTA's share): four signed digits of base 256, 30 bits.  So every sum of
// products of codes and digits is a whole number that 32 bits hold, the offset of
// 8 comes off exactly, and what is rounded is the fixed point (2^-31 of the
// largest) and the sums over groups, in fp32.
//
// The first product reads every selected byte once, for both vectors.  The second runs once a
// vector, over the whole list: the union of two lists is read twice, also the rows that only the
// other one names (2 x 14336 of 28672 neurons of 7168 bf16: both products 130 us; one list of
// them 46).  Integer products run at 64
// lanes a cycle and SM: four digits of one vector take 1 a weight where 47 weights
// a cycle and SM come from memory; logic and permutations (64 a cycle too, on
// another pipe) take 0.4 and 0.7.  (With m16n8k16 products of opened codes the 50257 x
// 5120 product took 68 us, however its loads were arranged: 3.5 cycles an SM each.  Now 35.4: 3.7
// TB/s of codes and scales.)

#include <climits>

#include "dv_kernels.h"

namespace dv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDigits = 4;
constexpr uint32_t kMagic = 0x4b400000u;   // 1.5 2^23 as a float: a whole number below 2^22 added to it is one in float
constexpr float kMagicF = 12582912.f;

// Elements (0, 4, 1, 5) and (2, 6, 3, 7) of a word as bytes.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) { return w & 0x0f0f0f0fu; }
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return (w >> 4) & 0x0f0f0f0fu; }
__device__ __forceinline__ int high_of(int e) { return (e >> 1) & 1; }
__device__ __forceinline__ int byte_of(int e) { return (e & 1) * 2 + (e >> 2); }

template <typename S>
__device__ __forceinline__ uint32_t ld_raw(const void* p) {
  if constexpr (sizeof(S) == 4) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  } else {
    uint16_t h;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(h) : "l"(p));
    return h;
  }
}
template <typename S> __device__ __forceinline__ float of_raw(uint32_t r);
template <> __device__ __forceinline__ float of_raw<float>(uint32_t r) { return __uint_as_float(r); }
template <> __device__ __forceinline__ float of_raw<__half>(uint32_t r) {
  return __half2float(__ushort_as_half((unsigned short)r));
}
template <> __device__ __forceinline__ float of_raw<__nv_bfloat16>(uint32_t r) { return __uint_as_float(r << 16); }

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The exponent that brings values of at most `top` into [-2^30, 2^30] (2^-150 is finer than
// the least of fp32).
__device__ __forceinline__ int fixed_shift(uint32_t top) { return min(30 - ((int)(top >> 23) - 126), 150); }
__device__ __forceinline__ int fixed(float v, int shift) {   // (two steps: 2^shift alone may be out of range)
  return __float2int_rn(v * pow2(shift / 2) * pow2(shift - shift / 2));
}
// Digits of base 256, the highest first, each in [-128, 127].
__device__ __forceinline__ void digits_of(int v, int* d) {
#pragma unroll
  for (int p = kDigits - 1; p > 0; --p) {
    d[p] = (int)(signed char)(v & 255);
    v = (v - d[p]) >> 8;
  }
  d[0] = v;
}

// ---- products with rows -----------------------------------------------------------------

// Vectors in shared memory: digits of the 32 elements of chunk (16 bytes of a row)
// k in the order of the chunk's codes, [vector][digit][half of it][chunk] of 16 bytes; -8
// times their sums, of either half of the block, [vector][chunk][half][digit]; and a
// the unit of a group's highest digit, [vector][group]: about its largest times 2^-6, so that
// neither its product with a scale nor that with a sum of digits leaves the range of fp32
// where products of weights and elements do not.
struct VecLayout {
  int chunks;   // a multiple of 32
  int groups;
  __host__ __device__ VecLayout(int blocks, int group) : chunks((blocks * 4 + 31) & ~31), groups(chunks * 32 / group) {}
  __host__ __device__ size_t digit_bytes() const { return (size_t)chunks * (kDigits * 32); }
  __host__ __device__ size_t offset_bytes() const { return (size_t)chunks * (kDigits * 8); }
  __host__ __device__ size_t bytes(int B) const { return B * (digit_bytes() + offset_bytes() + groups * 4); }
};

template <typename S>
__device__ __forceinline__ void stage_group(const S* y, int d, int group, int gi, const VecLayout& v, uint8_t* xs,
                                            float* unit) {
  const int lane = threadIdx.x & 31;
  float x[4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = gi * group + i * 32 + lane;
    x[i] = i * 32 < group && t < d ? Elem<S>::to_f(y[t]) : 0.f;
    top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const int shift = fixed_shift(top);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i * 32 >= group) break;
    const int t = gi * group + i * 32 + lane;
    int dig[kDigits];
    digits_of(top < 0x7f800000u ? fixed(x[i], shift) : 0, dig);
    const int r = t & 63, chunk = (t >> 7) * 4 + (r >> 4), half = (r >> 3) & 1, e = t & 7;
    uint8_t* at = xs + ((size_t)half * v.chunks + chunk) * 16 + ((t >> 6) & 1) * 8 + high_of(e) * 4 + byte_of(e);
#pragma unroll
    for (int p = 0; p < kDigits; ++p) at[(size_t)p * 2 * v.chunks * 16] = (uint8_t)dig[p];
  }
  // (an infinity or a NaN: every product a NaN)
  if (lane == 0) *unit = top < 0x7f800000u ? pow2(24 - shift) : __int_as_float(0x7fc00000);
}

// A warp takes kRows rows at a time, a lane one chunk of every 32 of a row; the next
// kAhead steps (of 32 chunks) of the rows are on their way while one is multiplied.
template <typename S, int B, int kRows, int kAhead, bool kList, bool two>
__global__ void __launch_bounds__(kThreads, 2) q4_vec_rows_kernel(const Q4Rows a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const VecLayout v(a.blocks, a.group);
  const uint8_t* offsets = smem + B * v.digit_bytes();
  float* units = reinterpret_cast<float*>(smem + B * (v.digit_bytes() + v.offset_bytes()));
  // at level 1 of the launch policy the list, its count and the weights are read
  // before the wait
  if (!a.early) grid_dep_wait();
  if (!a.early) grid_dep_launch();
  const int n = kList ? max(0, min(*a.count, a.cap)) : a.N;
  if (kList && blockIdx.x == 0 && tid == 0 && *a.count > a.cap) set_error(a.hdr, DV_ERR_CAPACITY, *a.count);
  const int tiles = (n + kRows - 1) / kRows, stride = gridDim.x * kWarps;
  const int steps = v.chunks >> 5, last = a.blocks * 4 - 1;

  constexpr int kNone = INT_MIN;
  int row[kRows];
  const uint8_t* q[kRows];
  const uint8_t* sp[kRows];
  const auto rows_of = [&](int t) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int u = t * kRows + k;
      row[k] = u < n ? u : kNone;
      if (kList && u < n) {
        const int r = max(a.list[u], kNone + 1);
        row[k] = u > 0 && a.list[u - 1] == r ? kNone : r;   // (an entry listed twice counts once)
        if (row[k] != kNone && (row[k] < 0 || row[k] >= a.N)) {
          if (lane == 0) set_error(a.hdr, DV_ERR_INDEX_RANGE, row[k]);
          row[k] = kNone;
        }
      }
      const size_t r = max(row[k], 0);
      q[k] = a.q + r * a.pitch;
      sp[k] = static_cast<const uint8_t*>(a.scale) + r * a.groups * sizeof(S);
    }
  };
  uint4 w[kAhead][kRows];
  uint32_t sc[kAhead][kRows][two ? 2 : 1];
  // (where there is no row or no chunk another is read and not used: a load under a condition
  // is waited for at once)
  const auto fetch = [&](int j, int s) {
    const int chunk = min(s * 32 + lane, last), gi = two ? chunk >> 2 << 1 : chunk >> 2;
    const int g1 = min(gi + 1, a.groups - 1);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      w[j][k] = ld_stream(q[k] + chunk * 16);
      sc[j][k][0] = ld_raw<S>(sp[k] + gi * (int)sizeof(S));
      if (two) sc[j][k][two] = ld_raw<S>(sp[k] + g1 * (int)sizeof(S));
    }
  };
  int t = blockIdx.x * kWarps + wid;
  if (t < tiles) {
    rows_of(t);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j < steps) fetch(j, j);
  }
  if (a.early) {
    grid_dep_wait();
    grid_dep_launch();
  }
  for (int i = wid; i < v.groups * B; i += kWarps) {
    const int b = i / v.groups, gi = i - b * v.groups;
    stage_group<S>(static_cast<const S*>(a.y) + (size_t)b * a.d, a.d, a.group, gi, v, smem + b * v.digit_bytes(), units + i);
  }
  __syncthreads();
  for (int i = tid; i < B * v.chunks * 2 * kDigits; i += kThreads) {
    // -8 times the sum of one digit over one half of a chunk, with kMagic
    const int p = i % kDigits, h = i / kDigits & 1, c = i / (2 * kDigits), b = c / v.chunks;
    const uint8_t* from = smem + b * v.digit_bytes() + ((size_t)p * 2 * v.chunks + (c - b * v.chunks)) * 16 + h * 8;
    int sum = (int)kMagic;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint2 x = *reinterpret_cast<const uint2*>(from + (size_t)k * v.chunks * 16);
      sum = __dp4a((int)x.x, (int)0xf8f8f8f8u, __dp4a((int)x.y, (int)0xf8f8f8f8u, sum));
    }
    reinterpret_cast<int*>(smem + B * v.digit_bytes())[i] = sum;
  }
  __syncthreads();
  while (t < tiles) {
    float acc[kRows][B];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int b = 0; b < B; ++b) acc[k][b] = 0.f;
    int mine[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) mine[k] = row[k];
    const int u0 = t * kRows;
    t += stride;
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = s0 + j;
        if (s >= steps) break;
        const int chunk = s * 32 + lane, gi = two ? chunk >> 2 << 1 : chunk >> 2;
        uint32_t code[kRows][8];   // [word][low, high]
        float scale[kRows][two ? 2 : 1];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const uint32_t ww[4] = {w[j][k].x, w[j][k].y, w[j][k].z, w[j][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            code[k][2 * i] = low_codes(ww[i]);
            code[k][2 * i + 1] = high_codes(ww[i]);
          }
#pragma unroll
          for (int h = 0; h < (two ? 2 : 1); ++h) scale[k][h] = of_raw<S>(sc[j][k][h]);
        }
        // the slot takes the step after the ones ahead, of these rows or the warp's next
        if (s + kAhead < steps) fetch(j, s + kAhead);
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint4* off = reinterpret_cast<const uint4*>(offsets) + ((size_t)b * v.chunks + chunk) * 2;
          const uint4 o0 = off[0], o1 = off[1];
          const int of0[kDigits] = {(int)o0.x, (int)o0.y, (int)o0.z, (int)o0.w};
          const int of1[kDigits] = {(int)o1.x, (int)o1.y, (int)o1.z, (int)o1.w};
          float f[kRows][two ? 2 : 1];
#pragma unroll
          for (int p = 0; p < kDigits; ++p) {
            const uint4* from = reinterpret_cast<const uint4*>(smem) + (size_t)b * (v.chunks * kDigits * 2) +
                                (size_t)p * 2 * v.chunks + chunk;
            const uint4 lo = from[0], hi = from[v.chunks];
            const int x[8] = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
              int sum[2] = {two ? of0[p] : of0[p] + (of1[p] - (int)kMagic), of1[p]};
#pragma unroll
              for (int i = 0; i < 8; ++i) {   // registers 2 and 3 of every four are of the block's second half
                int& at = sum[two ? (i >> 1) & 1 : 0];
                at = __dp4a((int)code[k][i], x[i], at);
              }
#pragma unroll
              for (int h = 0; h < (two ? 2 : 1); ++h) {
                const float part = __int_as_float(sum[h]) - kMagicF;   // exact
                f[k][h] = p == 0 ? part : fmaf(part, 1.f / (1 << (8 * p)), f[k][h]);
              }
            }
          }
#pragma unroll
          for (int h = 0; h < (two ? 2 : 1); ++h) {
            const float unit = units[b * v.groups + gi + h];
#pragma unroll
            for (int k = 0; k < kRows; ++k) acc[k][b] = fmaf(f[k][h], scale[k][h] * unit, acc[k][b]);
          }
        }
      }
    }
    if (t < tiles) {
      rows_of(t);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (j < steps) fetch(j, j);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float sum = warp_sum(acc[k][b]);
        if (lane != 0 || u0 + k >= n) continue;
        if (kList) {
          bool live = mine[k] != kNone;
          if (live && a.member) live = bit_test(a.member + (size_t)b * a.words, mine[k]);
          a.act[(size_t)b * a.ld_act + u0 + k] = live ? (sum > 0.f || sum != sum ? sum : 0.f) : 0.f;
        } else {
          float* o = a.out + (size_t)b * a.N + u0 + k;
          *o = a.accumulate ? *o + sum : sum;
        }
      }
  }
}

// ---- sums of listed rows ------------------------------------------------------------------

// out[b][t] (+)= sum_u act[b][u] s[j_u][group of t] (code[j_u][t] - 8).  A CTA owns a
// share of the list and whole rows of it (128 bytes of every row to a CTA instead took 39
// us for 53 MB: a row's memory page is opened once a CTA); a thread owns two words,
// 8 g .. 8 g + 7 of either half of a block; a step is four rows, whose codes of an element a
// 4 x 4 transpose of bytes puts side by side.  The CTAs' sums go to the workspace and
// a second kernel adds them in order.
//
// The coefficients act s of as many steps as fit are staged together; the largest of a
// group gives the unit of its digits, and a part's whole numbers become floats at its end.
constexpr int kColThreads = 512;           // at most
constexpr int kColAhead = 3;               // steps loaded ahead
constexpr int kStaged = 4096;              // (step, group) pairs staged at a time
constexpr int kMaxGroups = 512;            // rows of 32768, groups of 64

__device__ __forceinline__ float ld_scale_dt(const void* s, size_t i, int dt) {
  return dt == DV_F32 ? __ldg(static_cast<const float*>(s) + i)
         : dt == DV_F16 ? __half2float(__ldg(static_cast<const __half*>(s) + i))
                        : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(s) + i));
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

template <bool two>
__global__ void __launch_bounds__(kColThreads, 1) q4_vec_cols_kernel(const Q4Cols a) {
  extern __shared__ __align__(128) uint8_t smem[];   // coefficients of (step, group), four rows; then their digits
  __shared__ uint32_t top[kMaxGroups];
  __shared__ int id[kStaged / 2 * 4];
  float4* coef = reinterpret_cast<float4*>(smem);
  const int tid = threadIdx.x, threads = blockDim.x;
  const int words = a.blocks * 16, pair = blockIdx.y * threads + tid;   // the thread's two words
  const bool mine = 2 * pair < words;
  const int block = min(pair >> 3, a.blocks - 1);
  // groups of the CTA's words
  const int first_block = (blockIdx.y * threads) >> 3;
  const int per = two ? 2 : 1, g_first = first_block * per;
  const int groups = min((threads + 7) / 8 * per, a.blocks * per - g_first);
  const int set = (block - first_block) * per;
  const int n = max(0, min(*a.count, a.cap));
  const int quads_all = (n + 3) >> 2, share = (quads_all + gridDim.x - 1) / gridDim.x;
  const int lo = min(quads_all, (int)blockIdx.x * share), hi = min(quads_all, lo + share);
  const int at_once = min(kStaged / groups, kStaged / 2);
  const uint8_t* q = a.q + (size_t)min(pair, words / 2 - 1) * 8;

  uint2 w[kColAhead][4];
  const auto fetch = [&](int k, int s) {   // rows of step s
    const int4 j = reinterpret_cast<const int4*>(id)[s];
    w[k][0] = ld_stream8(q + (size_t)j.x * a.pitch);
    w[k][1] = ld_stream8(q + (size_t)j.y * a.pitch);
    w[k][2] = ld_stream8(q + (size_t)j.z * a.pitch);
    w[k][3] = ld_stream8(q + (size_t)j.w * a.pitch);
  };
  float out[2][8];   // elements (0, 2), (4, 6), (1, 3), (5, 7) of either word
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) out[h][i] = 0.f;
  bool waited = false;
  for (int q0 = lo; q0 < hi; q0 += at_once) {
    const int steps = min(at_once, hi - q0), m = min(4 * steps, n - 4 * q0);
    __syncthreads();
    for (int e = tid; e < 4 * steps; e += threads) {
      const int j = e < m ? a.list[4 * q0 + e] : 0;
      // (an entry outside is reported, and has activation 0, from the first product on: row 0 is read)
      id[e] = j >= 0 && j < a.N ? j : 0;
    }
    for (int g = tid; g < groups; g += threads) top[g] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kColAhead; ++k)
      if (k < steps) fetch(k, k);
    if (!waited) {
      grid_dep_wait();   // the activations
      grid_dep_launch();
      waited = true;
    }
    // coefficients, a row's groups by neighbouring threads, four entries of a thread at a time
    const int items = 4 * steps * groups;
    for (int i0 = tid; i0 < items; i0 += 4 * threads) {
      float x[4], s[4];
      int e[4], g[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = min(i0 + k * threads, items - 1);
        e[k] = i / groups;
        g[k] = i - e[k] * groups;
        x[k] = __ldcg(a.act + 4 * q0 + min(e[k], m - 1));
        s[k] = ld_scale_dt(a.scale, (size_t)id[e[k]] * a.groups + min(g_first + g[k], a.groups - 1), a.dt);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i0 + k * threads >= items) break;
        const float c = x[k] == 0.f || e[k] >= m ? 0.f : x[k] * s[k];   // (0 adds nothing, whatever the row holds)
        reinterpret_cast<float*>(coef + (size_t)(e[k] >> 2) * groups + g[k])[e[k] & 3] = c;
        const uint32_t bits = __float_as_uint(fabsf(c));
        if (bits) atomicMax(&top[g[k]], bits);
      }
    }
    __syncthreads();
    for (int i = tid; i < steps * groups; i += threads) {
      const uint32_t most = top[i % groups];
      const int shift = fixed_shift(most);
      const float4 c = coef[i];
      const float cc[4] = {c.x, c.y, c.z, c.w};
      uint32_t packed[kDigits] = {};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int dig[kDigits];
        digits_of(most < 0x7f800000u ? fixed(cc[r], shift) : 0, dig);
#pragma unroll
        for (int p = 0; p < kDigits; ++p) packed[p] |= (uint32_t)(dig[p] & 255) << (8 * r);
      }
      reinterpret_cast<uint4*>(coef)[i] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    }
    __syncthreads();
    int acc[2][8][kDigits], offset[two ? 2 : 1][kDigits];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int p = 0; p < kDigits; ++p) {
        offset[two && h][p] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[h][i][p] = 0;
      }
    for (int s0 = 0; s0 < steps; s0 += kColAhead) {
#pragma unroll
      for (int k = 0; k < kColAhead; ++k) {
        if (s0 + k >= steps) break;
        uint32_t r[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = h ? w[k][0].y : w[k][0].x, w1 = h ? w[k][1].y : w[k][1].x;
          const uint32_t w2 = h ? w[k][2].y : w[k][2].x, w3 = h ? w[k][3].y : w[k][3].x;
          const uint32_t t0 = __byte_perm(w0, w1, 0x5140), t1 = __byte_perm(w2, w3, 0x5140);
          const uint32_t t2 = __byte_perm(w0, w1, 0x7362), t3 = __byte_perm(w2, w3, 0x7362);
          r[h][0] = __byte_perm(t0, t1, 0x5410);
          r[h][1] = __byte_perm(t0, t1, 0x7632);
          r[h][2] = __byte_perm(t2, t3, 0x5410);
          r[h][3] = __byte_perm(t2, t3, 0x7632);
        }
        if (s0 + k + kColAhead < steps) fetch(k, s0 + k + kColAhead);
        const uint4* dig = reinterpret_cast<const uint4*>(coef) + (size_t)(s0 + k) * groups + set;
        uint4 x[two ? 2 : 1];
        x[0] = dig[0];
        if (two) x[two] = dig[1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 xh = x[two && h];
          const int xx[kDigits] = {(int)xh.x, (int)xh.y, (int)xh.z, (int)xh.w};
          if (h == 0 || two) {
#pragma unroll
            for (int p = 0; p < kDigits; ++p) offset[two && h][p] = __dp4a(xx[p], (int)0xf8f8f8f8u, offset[two && h][p]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c0 = (int)low_codes(r[h][i]), c1 = (int)high_codes(r[h][i]);
#pragma unroll
            for (int p = 0; p < kDigits; ++p) {
              acc[h][2 * i][p] = __dp4a(c0, xx[p], acc[h][2 * i][p]);
              acc[h][2 * i + 1][p] = __dp4a(c1, xx[p], acc[h][2 * i + 1][p]);
            }
          }
        }
      }
    }
    // the part's sums: whole numbers, times the unit
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t most = top[set + (two && h)];
      const int shift = fixed_shift(most);
      const float u0 = pow2(-(shift / 2)), u1 = pow2(-(shift - shift / 2));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        long long whole = 0;
#pragma unroll
        for (int p = 0; p < kDigits; ++p) whole = whole * 256 + (acc[h][i][p] + offset[two && h][p]);
        // (an infinity or a NaN among the coefficients)
        out[h][i] = most < 0x7f800000u ? out[h][i] + __ll2float_rn(whole) * u0 * u1 : __int_as_float(0x7fc00000);
      }
    }
  }
  if (!waited) {
    grid_dep_wait();
    grid_dep_launch();
  }
  if (!mine) return;
  // register i holds element 0 2 4 6 1 3 5 7
  float* part = a.part + (size_t)blockIdx.x * a.blocks * 128 + (size_t)(pair >> 3) * 128 + 8 * (pair & 7);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float4* to = reinterpret_cast<float4*>(part + 64 * h);
    to[0] = make_float4(out[h][0], out[h][4], out[h][1], out[h][5]);
    to[1] = make_float4(out[h][2], out[h][6], out[h][3], out[h][7]);
  }
}

// ---- launches ------------------------------------------------------------------------------

template <typename S, int B, int kRows, int kAhead, bool kList, bool two>
cudaError_t run_rows(const Q4Rows& a, bool pdl, int num_sms, cudaStream_t stream) {
  const size_t smem = VecLayout(a.blocks, a.group).bytes(B);
  static PerDevice attr;   // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(q4_vec_rows_kernel<S, B, kRows, kAhead, kList, two>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  });
  if (ea != cudaSuccess) return ea;
  const long long tiles = ((kList ? a.cap : a.N) + kRows - 1) / kRows, ctas = (tiles + kWarps - 1) / kWarps;
  const long long most = 2LL * num_sms;
  return launch_k(q4_vec_rows_kernel<S, B, kRows, kAhead, kList, two>, dim3((unsigned)(ctas < most ? ctas : most)),
                  dim3(kThreads), smem, stream, pdl, 1, a);
}
// Rows at a time: two (one: 55 us for 50257 x 5120, 30 for 14336 listed rows of 7168; two:
// 35.8 and 21.6; four: 35.0 and 24.7); one where two would leave half of the GPU's
// warps (16 an SM) without rows (1024 of 5120: 6.9 us, two: 7.2).
template <typename S, int B, bool kList, bool two>
cudaError_t run_rows_shape(const Q4Rows& a, bool pdl, int num_sms, cudaStream_t stream) {
  const int rows = kList ? a.cap : a.N;
  return rows < 8 * num_sms ? run_rows<S, B, 1, 5, kList, two>(a, pdl, num_sms, stream)
                            : run_rows<S, B, 2, 4, kList, two>(a, pdl, num_sms, stream);
}
template <typename S>
cudaError_t run_rows_of(const Q4Rows& a, bool pdl, int num_sms, cudaStream_t stream) {
  const bool two = a.group == 64;
  if (a.B == 1) {
    if (a.list) return two ? run_rows_shape<S, 1, true, true>(a, pdl, num_sms, stream) : run_rows_shape<S, 1, true, false>(a, pdl, num_sms, stream);
    return two ? run_rows_shape<S, 1, false, true>(a, pdl, num_sms, stream) : run_rows_shape<S, 1, false, false>(a, pdl, num_sms, stream);
  }
  if (a.list) return two ? run_rows_shape<S, 2, true, true>(a, pdl, num_sms, stream) : run_rows_shape<S, 2, true, false>(a, pdl, num_sms, stream);
  return two ? run_rows_shape<S, 2, false, true>(a, pdl, num_sms, stream) : run_rows_shape<S, 2, false, false>(a, pdl, num_sms, stream);
}

template <bool two>
cudaError_t run_cols(const Q4Cols& all, int num_sms, cudaStream_t stream) {
  static PerDevice attr;   // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(q4_vec_cols_kernel<two>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStaged * 16);
  });
  if (ea != cudaSuccess) return ea;
  Q4Cols a = all;
  // a thread to two words; rows of more than 8192 elements in equal slabs of whole blocks
  const int slabs = (a.blocks * 8 + kColThreads - 1) / kColThreads;
  const int threads = ((a.blocks + slabs - 1) / slabs * 8 + 31) / 32 * 32;
  // shares: a CTA for every SM, of four steps each at least (1024 rows: the second kernel
  // then has 64 sums to add)
  const int most = (a.cap + 15) / 16;
  int shares = (num_sms < kQ4Splits ? num_sms : kQ4Splits) / slabs;
  shares = shares < 1 ? 1 : shares > most ? most : shares;
  a.B = 1;
  for (int b = 0; b < all.B; ++b) {
    cudaError_t e = launch_k(q4_vec_cols_kernel<two>, dim3(shares, slabs), dim3(threads), kStaged * 16, stream, true, 1, a);
    if (e == cudaSuccess) e = launch_q4_join(a, shares, stream);
    if (e != cudaSuccess) return e;
    a.act += a.ld_act;
    a.out += a.d;
  }
  return cudaSuccess;
}

}  // namespace

bool q4_vec_supported(int B, int d) {
  return B <= 2 && VecLayout((d + 127) / 128, 64).bytes(B) <= 227 * 1024;
}

cudaError_t launch_q4_vec_rows(const Q4Rows& a, dv_dtype dt, bool pdl, cudaStream_t stream) {
  const int num_sms = num_sms_current();
  switch (dt) {
    case DV_F32: return run_rows_of<float>(a, pdl, num_sms, stream);
    case DV_F16: return run_rows_of<__half>(a, pdl, num_sms, stream);
    case DV_BF16: return run_rows_of<__nv_bfloat16>(a, pdl, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_q4_vec_cols(const Q4Cols& a, cudaStream_t stream) {
  const int num_sms = num_sms_current();
  return a.group == 64 ? run_cols<true>(a, num_sms, stream) : run_cols<false>(a, num_sms, stream);
}

}  // namespace dv
