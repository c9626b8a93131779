// Matrices in 4 bits with group scales, w[n][t] = (code[n][t] - 8) s[n][t / G]:
// quantisation, the choice among the kernels of both kinds of product, and the
// m16n8k16 form of the first.
//   with rows (all, or a list's)   one and two vectors: k_q4_vec.cu; three to 32 by many
//                                  rows: k_q4_tc.cu; the rest here
//   sums of listed rows            one and two vectors: k_q4_vec.cu; more: k_q4_tc_cols.cu
//
// Layout.  A row is blocks of 128 elements in 64 bytes.  Word w of a block
// (g = w / 2, s = w % 2) holds elements 64 s + 8 g + e, e < 8, at bit
// 4 (e / 2) + 16 (e % 2), so that
//   - (word >> 4 i) & 0x000f000f are elements 2 i and 2 i + 1 side by side: one
//     logic operation makes a pair of 16-bit floats of them;
//   - the 16 bytes of chunk c (of 4) are elements 16 c .. 16 c + 15 of either
//     half of the block: as the A operand of an m16n8k16 product, whose lane
//     (g, c) holds four k of row g and of row g + 8, a 16-byte load is four
//     k-steps, two of each half, and the vector's elements that go with it are
//     contiguous;
//   - a word opened is eight neighbouring elements in order: 16 bytes of a tile
//     in which elements are contiguous (the second product).
//
// The codes less 8 are exact in both 16-bit types and a product of one of
// them with a 16-bit factor is exact in fp32; sums are fp32 and the scale is
// applied to the sum over a group (to the coefficient in the second product).
// 32-bit factors (a DV_F32 vector, the coefficients) enter as three bf16 pieces
// that add up to them, as further columns of the product.
//
// Measured on GB300: 5 fp32 vectors with 5001 rows of 5000 14.3 us (0.98 TB/s of codes and
// scales: latency of two launches and of blocks loaded four ahead); quantisation of 20480 x
// 5120 f16 with values 110 us (4.3 TB/s, 0.63 of a copy's rate: instructions).

#include "dv_kernels.h"

namespace dv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlockBytes = kQ4BlockBytes;

// ---- pairs of codes -------------------------------------------------------------

template <typename P> struct Pairs;
template <> struct Pairs<__half> {
  // element pairs i = 0..3 of a word, less 8
  static __device__ __forceinline__ void open(uint32_t w, uint32_t* p) {
    const __half2 m1032 = __half2half2(__ushort_as_half(0xe408));           // -1032
    const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));             // 1/16
    const __half2 m72 = __half2half2(__ushort_as_half(0xd480));             // -72
    const uint32_t v = w >> 8;
    const uint32_t a[4] = {(w & 0x000f000fu) | 0x64006400u, (w & 0x00f000f0u) | 0x64006400u,
                           (v & 0x000f000fu) | 0x64006400u, (v & 0x00f000f0u) | 0x64006400u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = *reinterpret_cast<const __half2*>(&a[i]);
      const __half2 r = (i & 1) ? __hfma2(h, r16, m72) : __hadd2(h, m1032);  // 1024 + 16 q, 1024 + q
      p[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};
template <> struct Pairs<__nv_bfloat16> {
  static __device__ __forceinline__ void open(uint32_t w, uint32_t* p) {
    const __nv_bfloat162 m136 = __bfloat162bfloat162(__ushort_as_bfloat16(0xc308));  // -136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;       // 128 + q
      const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), m136);
      p[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};

// D += A B, m16n8k16: A 16 x 16 in four registers, B 16 x 8 in two.
template <typename P>
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An fp32 value as three bf16 pieces whose sum it is (24 bits of mantissa in
// three of 8; a value that is not finite is its own first piece).
__device__ __forceinline__ void pieces3(float v, __nv_bfloat16* p) {
  p[0] = __float2bfloat16_rz(v);       // (towards zero: the largest values do not become infinite)
  float r = v - __bfloat162float(p[0]);
  r = fabsf(r) < INFINITY ? r : 0.f;   // (what is left of an infinity or a NaN is a NaN)
  p[1] = __float2bfloat16_rn(r);
  p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}

template <typename S>
__device__ __forceinline__ float ld_scale(const void* s, size_t i) {
  return Elem<S>::to_f(__ldg(static_cast<const S*>(s) + i));
}

// ---- quantisation ------------------------------------------------------------------

// round-to-even(f / s), 0 where s is 0: a quotient that was rounded onto a border between two
// whole numbers is put on its side of it by the exact sign of f - ratio s.
__device__ __noinline__ float nearest(float f, float s) {
  if (!(s > 0.f)) return 0.f;
  const float ratio = __fdiv_rn(f, s);
  if (fabsf(ratio - truncf(ratio)) == 0.5f) {
    const double rem = (double)f - (double)ratio * (double)s;
    if (rem > 0.) return ceilf(ratio);
    if (rem < 0.) return floorf(ratio);
  }
  return rintf(ratio);
}

// The largest magnitude among 8 elements as an integer (a NaN's is above infinity's), and 8
// elements r s of the storage type (r whole, 4 bits: one rounding).
__device__ __forceinline__ uint32_t top_of(const uint4* w, const float* f, float) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
  return top;
}
__device__ __forceinline__ void values_of(const float* r, float s, uint4* o) {
  float* h = reinterpret_cast<float*>(o);
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = r[e] * s;
}
template <typename P>
__device__ __forceinline__ uint32_t top_of_pairs(const P* p) {
  const P m = __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
  return max(__float_as_uint(__low2float(m)), __float_as_uint(__high2float(m))) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t top_of(const uint4* w, const float*, __half) {
  return top_of_pairs(reinterpret_cast<const __half2*>(w));
}
__device__ __forceinline__ uint32_t top_of(const uint4* w, const float*, __nv_bfloat16) {
  return top_of_pairs(reinterpret_cast<const __nv_bfloat162*>(w));
}
__device__ __forceinline__ void values_of(const float* r, __half s, uint4* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<__half2*>(o)[i] = __hmul2(__floats2half2_rn(r[2 * i], r[2 * i + 1]), __half2half2(s));
}
__device__ __forceinline__ void values_of(const float* r, __nv_bfloat16 s, uint4* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<__nv_bfloat162*>(o)[i] = __hmul2(__floats2bfloat162_rn(r[2 * i], r[2 * i + 1]), __bfloat162bfloat162(s));
}

// One half-warp per block of 128 elements, a lane to a word: 8 elements in, one
// word out; kItems blocks at a time, whose loads are issued together.  The matrix is read
// once and codes, scales and values are written once.
constexpr int kItems = 2;

template <typename T>
__global__ void __launch_bounds__(kThreads) q4_quantize_kernel(const T* __restrict__ W, int d, uint32_t blocks,
                                                              uint32_t total, int group, uint32_t* __restrict__ q,
                                                              T* __restrict__ scale, T* __restrict__ values) {
  constexpr int kVecs = 8 / Elem<T>::kVec;   // 16-byte vectors of 8 elements
  const int lane = threadIdx.x & 31, word = lane & 15;
  const int s = word & 1, at = 64 * s + 8 * (word >> 1);
  const int groups = (d + group - 1) / group;
  // (whole warps take part in the exchanges below, also behind the last block; fewer than
  // 2^32 blocks: more would not fit the GPU, and 64-bit divisions took most of the time)
  const uint32_t first = blockIdx.x * (kThreads / 16) + threadIdx.x / 16, stride = gridDim.x * (kThreads / 16);
  uint4 w[kItems][kVecs];
  uint32_t n_of[kItems];
  int t_of[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = min(first + k * stride, total - 1), n = i / blocks;
    const int t = (int)(i - n * blocks) * 128 + at;
    n_of[k] = n;
    t_of[k] = t;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)   // (behind the row's end its first vector: not used)
      w[k][v] = ld_stream(W + (size_t)n * d + (t + v * Elem<T>::kVec < d ? t + v * Elem<T>::kVec : 0));
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = first + k * stride;
    const bool in = i < total;
    const size_t n = n_of[k];
    const int t = t_of[k];
    float f[8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (t + v * Elem<T>::kVec >= d) w[k][v] = make_uint4(0, 0, 0, 0);
      unpack<T>(w[k][v], f + v * Elem<T>::kVec);
    }
    uint32_t top = top_of(w[k], f, T());
#pragma unroll
    for (int o = 2; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t other = __shfl_xor_sync(0xffffffffu, top, 1);
    if (group == 128) top = max(top, other);
    const bool fine = top < 0x7f800000u;
    // (a / 7 in fp32 and then in 16 bits is a / 7 rounded once: with at most 11 bits of a it is at least
    // 2^-15 relative from a border of the 16-bit type)
    const T sc = Elem<T>::from_f(fine ? __fdiv_rn(__uint_as_float(top), 7.f) : __int_as_float(0x7fc00000));
    const float sf = Elem<T>::to_f(sc);
    // round-to-even(f / s): the product with 1 / s, and a step where what it leaves, which is
    // exact, is more than half of s, or half of it and the code odd.  Codes are added up as floats, eight of them to two
    // whole numbers of 16 bits.  (With a division and a correction for every element 20480 x 5120 took 182 us, with the
    // correction asked for by every element 135.)
    const bool quick = fine && sf > 0x1p-100f;
    const float inv = quick ? __frcp_rn(sf) : 0.f, half = 0.5f * sf;
    constexpr float kWhole = 12582912.f;   // 1.5 2^23
    float r[8], most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r[e] = __fsub_rn(__fmaf_rn(f[e], inv, kWhole), kWhole);
      most = fmaxf(most, fabsf(__fmaf_rn(-r[e], sf, f[e])));
    }
    if (most >= half) {   // (seldom: asked once for a lane's eight elements)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float left = __fmaf_rn(-r[e], sf, f[e]);
        const bool odd = __float_as_int(__fadd_rn(r[e], kWhole)) & 1;
        if (fabsf(left) > half || (fabsf(left) == half && odd)) r[e] += copysignf(1.f, left);
      }
    }
    if (!quick) {   // (1 / s or s / 2 would leave the range of fp32, or the scale is 0 or a NaN)
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const float x = nearest(e < 4 ? (e < 2 ? (e ? f[1] : f[0]) : (e & 1 ? f[3] : f[2]))
                                      : (e < 6 ? (e & 1 ? f[5] : f[4]) : (e & 1 ? f[7] : f[6])), fine ? sf : 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = k == e ? x : r[k];
      }
    }
    if (!(sf > 0x1p-14f)) {   // (a scale of fewer bits may be far below max / 7: elsewhere |r| <= 7)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = fminf(fmaxf(r[e], -8.f), 7.f);
    }
    float even = kWhole + 34952.f, odd = kWhole + 34952.f;   // 0x8888: 8 more for each
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float& sum = e & 1 ? odd : even;
      sum = __fmaf_rn(r[e], (float)(1 << (4 * (e >> 1))), sum);
    }
    const uint32_t code = __byte_perm(__float_as_uint(even), __float_as_uint(odd), 0x5410);
    if (!in) continue;
    q[(size_t)i * (kBlockBytes / 4) + word] = code;
    if (t < d && (t % group) == 0) scale[n * groups + t / group] = sc;
    if (values) {
      uint4 o[kVecs];
      values_of(r, sc, o);   // (a NaN as the scale: NaNs)
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (t + v * Elem<T>::kVec < d) *reinterpret_cast<uint4*>(values + n * d + t + v * Elem<T>::kVec) = o[v];
    }
  }
}

// ---- products with rows of a matrix ----------------------------------------------------

// Pieces of 32-bit vectors, rows of whole blocks, zero behind d: for every
// kPieceRows vectors their first pieces, then their second, then their third.
constexpr int kPieceRows = 10;   // 30 columns of a product

__global__ void __launch_bounds__(kThreads) q4_pieces_kernel(const float* __restrict__ y, int B, int d, int ld,
                                                            __nv_bfloat16* __restrict__ x) {
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
  if (t >= ld) return;
  const int b0 = b / kPieceRows * kPieceRows, rows = min(kPieceRows, B - b0);
  __nv_bfloat16 p[3];
  pieces3(t < d ? y[(size_t)b * d + t] : 0.f, p);
#pragma unroll
  for (int k = 0; k < 3; ++k) x[((size_t)3 * b0 + k * rows + b - b0) * ld + t] = p[k];
}

// A CTA takes 16 rows, its warp p the rows' blocks p, p + 8, ...  For what neither k_q4_vec.cu
// nor k_q4_tc.cu takes: three and more vectors with few rows or of less than 64 elements, and
// two vectors of more than its shared memory holds with few rows.
constexpr int kAhead = 4;   // blocks whose loads are issued before the first is used

template <typename S, typename P, int NT, bool kList>
__global__ void __launch_bounds__(kThreads) q4_rows_kernel(const Q4Rows a) {
  __shared__ float red[kWarps][16][8 * NT + 1];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int u0 = blockIdx.x * 16;
  grid_dep_wait();
  grid_dep_launch();
  int row[2];
  const int n = kList ? max(0, min(*a.count, a.cap)) : a.N;
#pragma unroll
  for (int k = 0; k < 2; ++k) {   // (a list is a union: each of its rows once, and in range)
    const int u = u0 + g + 8 * k;
    row[k] = u >= n ? -1 : kList ? a.list[u] : u;
  }
  const uint8_t* q0 = a.q + (size_t)max(row[0], 0) * a.pitch + 16 * c;
  const uint8_t* q1 = a.q + (size_t)max(row[1], 0) * a.pitch + 16 * c;
  const size_t s0 = (size_t)max(row[0], 0) * a.groups, s1 = (size_t)max(row[1], 0) * a.groups;
  const int halves = a.group == 64 ? 2 : 1;   // scales of a block
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  const P* x = static_cast<const P*>(a.x);
  for (int k0 = wid; k0 < a.blocks; k0 += kWarps * kAhead) {
    uint4 w[kAhead][2];
    float sc[kAhead][2][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int kb = k0 + i * kWarps;
      w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
      if (kb < a.blocks) {
        if (row[0] >= 0) w[i][0] = ld_stream(q0 + (size_t)kb * kBlockBytes);
        if (row[1] >= 0) w[i][1] = ld_stream(q1 + (size_t)kb * kBlockBytes);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int kb = k0 + i * kWarps;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int gi = halves == 2 ? 2 * kb + h : kb;
        const bool in = kb < a.blocks && gi < a.groups;
        sc[i][h][0] = in && row[0] >= 0 ? ld_scale<S>(a.scale, s0 + gi) : 0.f;
        sc[i][h][1] = in && row[1] >= 0 ? ld_scale<S>(a.scale, s1 + gi) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int kb = k0 + i * kWarps;
      if (kb >= a.blocks) break;
      const uint32_t w0[4] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w};
      const uint32_t w1[4] = {w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
      float d[NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 0 || halves == 2) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) d[t][r] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t p0[4], p1[4];
          Pairs<P>::open(w0[2 * j + h], p0);
          Pairs<P>::open(w1[2 * j + h], p1);
          const int e = kb * 128 + 64 * h + 16 * c + 8 * j;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint4 v = make_uint4(0, 0, 0, 0);
            // (plain loads: with a 32-bit vector the pieces are another kernel's output)
            if (8 * t + g < a.cols && e < a.x_len) v = *reinterpret_cast<const uint4*>(x + (size_t)(8 * t + g) * a.ldx + e);
            mma16816<P>(d[t], p0[0], p1[0], p0[1], p1[1], v.x, v.y);
            mma16816<P>(d[t], p0[2], p1[2], p0[3], p1[3], v.z, v.w);
          }
        }
        if (h == 1 || halves == 2) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(sc[i][h][r >> 1], d[t][r], acc[t][r]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wid][g + 8 * (r >> 1)][8 * t + 2 * c + (r & 1)] = acc[t][r];
  __syncthreads();
  // sums over the parts (and a 32-bit vector's pieces), in a fixed order
  for (int i = tid; i < 16 * a.B; i += kThreads) {
    const int r = i % 16, b = i / 16, u = u0 + r;
    if (u >= n) continue;
    float sum = 0.f;
    for (int p = 0; p < kWarps; ++p)
      for (int col = b; col < a.cols; col += a.B) sum += red[p][r][col];
    if (kList) {
      const bool live = bit_test(a.member + (size_t)b * a.words, a.list[u]);
      a.act[(size_t)b * a.ld_act + u] = live ? (sum > 0.f || sum != sum ? sum : 0.f) : 0.f;
    } else {
      float* o = a.out + (size_t)b * a.N + u;
      *o = a.accumulate ? *o + sum : sum;
    }
  }
}

// ---- sums of the second product's shares ----------------------------------------------------

// out[b][t] (+)= the sum over the shares, [share][vector][ld]: 32 elements a CTA, eight warps
// that take every eighth share, in a fixed order.
__global__ void __launch_bounds__(256) q4_join_kernel(const float* __restrict__ part, int parts, int ld, int d,
                                                     float* __restrict__ out, int accumulate) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, b = blockIdx.y, t = blockIdx.x * 32 + lane;
  grid_dep_wait();
  grid_dep_launch();
  float sum = 0.f;
#pragma unroll 10
  for (int r = wid; r < parts; r += 8) sum += __ldcg(part + ((size_t)r * gridDim.y + b) * ld + t);   // (ld: whole blocks)
  red[wid][lane] = sum;
  __syncthreads();
  if (wid != 0 || t >= d) return;
  sum = red[0][lane];
#pragma unroll
  for (int k = 1; k < 8; ++k) sum += red[k][lane];
  float* o = out + (size_t)b * d + t;
  *o = accumulate ? *o + sum : sum;
}

template <typename S, typename P, int NT>
cudaError_t run_rows(const Q4Rows& a, bool pdl, cudaStream_t stream) {
  const dim3 grid(((a.list ? a.cap : a.N) + 15) / 16);
  return a.list ? launch_k(q4_rows_kernel<S, P, NT, true>, grid, dim3(kThreads), 0, stream, pdl, 1, a)
                : launch_k(q4_rows_kernel<S, P, NT, false>, grid, dim3(kThreads), 0, stream, pdl, 1, a);
}
template <typename S, typename P>
cudaError_t run_rows_nt(const Q4Rows& a, bool pdl, cudaStream_t stream) {
  const int nt = (a.cols + 7) / 8;
  if (nt <= 1) return run_rows<S, P, 1>(a, pdl, stream);
  if (nt <= 2) return run_rows<S, P, 2>(a, pdl, stream);
  return run_rows<S, P, 4>(a, pdl, stream);
}

// The first product: y in its storage type, or as pieces made by a kernel before it.
cudaError_t launch_rows(Q4Rows a, const void* y, void* pieces, dv_dtype dt, bool pdl, cudaStream_t stream) {
  a.y = y;
  a.blocks = (a.d + 127) / 128;
  a.pitch = (size_t)a.blocks * kBlockBytes;
  a.groups = (a.d + a.group - 1) / a.group;
  if (q4_vec_supported(a.B, a.d)) return launch_q4_vec_rows(a, dt, pdl, stream);
  if (dt == DV_F32) {
    const int ld = a.blocks * 128;
    const cudaError_t e = launch_k(q4_pieces_kernel, dim3((ld + kThreads - 1) / kThreads, a.B), dim3(kThreads), 0, stream,
                                   true, 1, static_cast<const float*>(y), a.B, a.d, ld, static_cast<__nv_bfloat16*>(pieces));
    if (e != cudaSuccess) return e;
    a.ldx = ld; a.x_len = ld;
    const int B = a.B;
    for (int b0 = 0; b0 < B; b0 += kPieceRows) {
      Q4Rows r = a;
      r.B = B - b0 < kPieceRows ? B - b0 : kPieceRows;
      r.cols = 3 * r.B;
      r.x = static_cast<const __nv_bfloat16*>(pieces) + (size_t)3 * b0 * ld;
      if (r.out) r.out += (size_t)b0 * r.N;
      if (r.act) r.act += (size_t)b0 * r.ld_act;
      if (r.member) r.member += (size_t)b0 * r.words;
      const cudaError_t er = q4_tc_takes(r) ? launch_q4_tc_rows(r, dt, r.hdr, true, stream)
                                            : run_rows_nt<float, __nv_bfloat16>(r, true, stream);
      if (er != cudaSuccess) return er;
    }
    return cudaSuccess;
  }
  a.x = y; a.cols = a.B; a.ldx = a.d; a.x_len = a.d;
  if (q4_tc_takes(a)) return launch_q4_tc_rows(a, dt, a.hdr, pdl, stream);
  return dt == DV_F16 ? run_rows_nt<__half, __half>(a, pdl, stream)
                      : run_rows_nt<__nv_bfloat16, __nv_bfloat16>(a, pdl, stream);
}

}  // namespace

cudaError_t launch_q4_join(const Q4Cols& a, int shares, cudaStream_t stream) {
  return launch_k(q4_join_kernel, dim3((a.d + 31) / 32, a.B), dim3(256), 0, stream, true, 1, (const float*)a.part, shares,
                  a.blocks * 128, a.d, a.out, a.accumulate);
}

size_t q4_part_floats(int B, int d) {
  // shares of one vector's lists (k_q4_vec.cu), or B vectors' shares times slabs of at most
  // eight blocks (k_q4_tc_cols.cu)
  const size_t blocks = (size_t)(d + 127) / 128;
  const size_t one = kQ4Splits * blocks * 128, many = (kQ4Splits * 8 + blocks) * 128 * (size_t)B;
  return many > one ? many : one;
}

cudaError_t launch_q4_quantize(const void* W, int N, int d, dv_dtype dt, int group, void* q, void* scale, void* values,
                               int num_sms, cudaStream_t stream) {
  const int blocks = (d + 127) / 128;
  const long long total = (long long)N * blocks, per = kThreads / 16;
  if (total + 4 * per * num_sms >= 1LL << 32) return cudaErrorInvalidValue;   // (more than a GPU holds)
  const long long ctas = (total + per * kItems - 1) / (per * kItems);   // kItems blocks a half-warp
  const dim3 grid((unsigned)ctas);
  const auto run = [&](auto* w) {
    using T = std::remove_cv_t<std::remove_pointer_t<decltype(w)>>;
    return launch_k(q4_quantize_kernel<T>, grid, dim3(kThreads), 0, stream, false, 1, static_cast<const T*>(w), d,
                    (uint32_t)blocks, (uint32_t)total, group, static_cast<uint32_t*>(q), static_cast<T*>(scale), static_cast<T*>(values));
  };
  switch (dt) {
    case DV_F32: return run(static_cast<const float*>(W));
    case DV_F16: return run(static_cast<const __half*>(W));
    case DV_BF16: return run(static_cast<const __nv_bfloat16*>(W));
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_q4_matvec(const Q4MatvecLaunch& L, dv_dtype dt, cudaStream_t stream) {
  Q4Rows a{};
  a.q = L.q; a.scale = L.scale; a.group = L.group; a.B = L.B; a.d = L.d; a.N = L.N;
  a.out = L.out; a.accumulate = L.accumulate; a.part = L.part; a.hdr = L.hdr;
  return launch_rows(a, L.y, L.pieces, dt, true, stream);
}

cudaError_t launch_q4_sparse_mlp(const Q4MlpLaunch& L, dv_dtype dt, WsHeader* hdr, cudaStream_t stream) {
  Q4Rows a{};
  a.q = L.q1; a.scale = L.s1; a.group = L.group1; a.B = L.B; a.d = L.d; a.N = L.N;
  a.list = L.idx; a.count = L.count; a.cap = L.cap; a.act = L.act; a.hdr = hdr;
  if (L.B > 1) {
    const cudaError_t e =
        launch_union(L.idx, L.cap, L.count, L.B, L.N, L.U, L.U_count, L.member, nullptr, hdr, stream);
    if (e != cudaSuccess) return e;
    a.list = L.U; a.count = L.U_count; a.cap = mlp_union_cap(L.B, L.N, L.cap);
    a.member = L.member; a.words = (L.N + 31) / 32;
  }
  a.ld_act = (a.cap + 3) & ~3;
  // batch 1 under the overlap policy: everything but y is read before the wait
  a.early = launch_overlap() > 0 && L.B == 1 ? 1 : 0;
  cudaError_t e = launch_rows(a, L.y, L.pieces, dt, a.early != 0, stream);
  if (e != cudaSuccess) return e;
  Q4Cols c{};
  c.q = L.q2; c.scale = L.s2; c.group = L.group2; c.B = L.B; c.d = L.d; c.N = L.N;
  c.list = a.list; c.count = a.count; c.cap = a.cap; c.act = L.act; c.ld_act = a.ld_act;
  c.out = L.out; c.accumulate = L.accumulate; c.dt = dt; c.part = L.part;
  const int blocks = (L.d + 127) / 128;
  c.pitch = (size_t)blocks * kBlockBytes;
  c.groups = (L.d + L.group2 - 1) / L.group2;
  c.blocks = blocks;
  c.hdr = hdr;
  return L.B <= 2 ? launch_q4_vec_cols(c, stream) : launch_q4_tc_cols(c, stream);
}

}  // namespace dv
