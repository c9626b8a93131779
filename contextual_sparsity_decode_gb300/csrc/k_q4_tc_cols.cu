// Matrices in 4 bits (layout: k_q4.cu), the second product of the sparse MLP for three
// and more vectors, on the 5th-generation tensor cores:
//     out[b][t] (+)= sum_u act[b][u] s[j_u][group of t] (code[j_u][t] - 8).
//
// A CTA owns a share of the list and a slab of the rows' blocks, whose sums stay in tensor
// memory.  A step is 64 listed rows of one block: M = 128 elements, K = 64 rows, N = the
// vectors' coefficients act s in three bf16 pieces that add up to them, side by side
// (with groups of 64 once for either half of the block: a row of the accumulator reads its
// half's columns).  The codes are exact in bf16.  A word of a row holds eight
// neighbouring elements, so that the opened codes are stored as they are to a tile
// in which elements are contiguous (MN-major).
//   warps 0-7    open the codes of a step, a 16-byte chunk a thread; at the end take the
//                sums out
//   warps 8-15   make the coefficients of a step, a pair of rows by every eighth vector
//                a thread
//   warps 16-19  the listed rows' slabs and their activations into a ring of stages
//                (cp.async), their scales as floats
//   warp 20      the products
// The shares' sums go to the workspace and q4_join_kernel adds them in order.
//
// On m16n8k16 products (3.5 cycles an SM each, three for 16 rows by 16 elements by 8 vectors)
// 16 vectors by 16050 of 28672 rows of 7168 took 68 us, here 59 (alone under a profiler; groups
// of 64, which make the coefficients twice; 32 vectors with both products 245 and 187).  Bound
// by the chain of a step (codes opened, coefficients made, products, their end): 1800 cycles,
// of which the two are 900.  A list of 600 rows is 2 us slower than it was there: fewer and longer shares.

#include <climits>

#include "dv_kernels.h"
#include "q4_tc.cuh"

namespace dv {
namespace {

constexpr int kThreads = 672;
constexpr int kChunk = 64;       // rows of a step
constexpr int kPair = 2;         // blocks of a step
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kABytes = kChunk * 256;   // of a block

// Bp: vectors, rounded up; two: groups of 64.
template <int Bp, bool two>
struct Cols {
  static constexpr int kOne = (3 * Bp + 15) / 16 * 16;     // columns of a block's (half's) pieces
  static constexpr int kN = two ? 2 * kOne : kOne;
  static constexpr int kSlab = kN <= 64 ? 8 : kN <= 128 ? 4 : 2;   // blocks whose sums fit tensor memory
  static constexpr int kScales = two ? 2 * kSlab : kSlab;
  static constexpr int kStages = 3, kBufs = 2;             // of rows; steps under way
  static constexpr uint32_t kPitch = kSlab * kQ4BlockBytes;
  static constexpr uint32_t kWBytes = kChunk * kPitch;
  static constexpr uint32_t kActBytes = Bp * kChunk * 4;
  static constexpr uint32_t kScaleBytes = kScales * kChunk * 4;
  static constexpr uint32_t kBBytes = kN * 128;            // K = 64: a swizzled line a column
  static constexpr size_t kSmem = 1024 + kBufs * kPair * (kABytes + kBBytes) + (size_t)kStages * (kWBytes + kActBytes + kScaleBytes);
  static_assert(kN * kSlab <= (int)kTmemCols && kN <= 256, "fits tensor memory and one product");
  static_assert(kBBytes % 1024 == 0 && kSmem + 1024 <= 227 * 1024, "fits an SM");
};

// A scale as it is stored (a load under a condition would be waited for at once), and its value.
template <bool wide>
__device__ __forceinline__ uint32_t ld_raw(const void* s, size_t i) {
  return wide ? __ldg(static_cast<const uint32_t*>(s) + i) : __ldg(static_cast<const uint16_t*>(s) + i);
}
__device__ __forceinline__ float of_raw(uint32_t r, int dt) {
  return dt == DV_F32 ? __uint_as_float(r) : dt == DV_F16 ? __half2float(__ushort_as_half((unsigned short)r)) : __uint_as_float(r << 16);
}
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }
// Two fp32 values as three pairs of bf16 pieces whose sums they are (24 bits of mantissa in three of
// 8; of an infinity or a NaN the pieces' sum is a NaN).
__device__ __forceinline__ void pieces3(float a, float b, uint32_t* p) {
  // (cut off: the largest values do not become infinite; a product's NaN keeps its upper bits)
  const uint32_t hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  const float ra = a - __uint_as_float(__float_as_uint(a) & 0xffff0000u);
  const float rb = b - __uint_as_float(__float_as_uint(b) & 0xffff0000u);
  const uint32_t mid = bits_of(__floats2bfloat162_rn(ra, rb));
  p[0] = hi;
  p[1] = mid;
  p[2] = bits_of(__floats2bfloat162_rn(ra - __uint_as_float(mid << 16), rb - __uint_as_float(mid & 0xffff0000u)));
}

template <int Bp, bool two, bool wide>
__global__ void __launch_bounds__(kThreads, 1) q4_tc_cols_kernel(const Q4Cols a) {
  using Z = Cols<Bp, two>;
  constexpr int S = Z::kStages, kBufs = Z::kBufs, kPer = two ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_w[S], full_s[S], empty[S], ready[kBufs], done[kBufs], fin;
  __shared__ uint32_t tmem_base;
  __shared__ int stop_s, odd_s;   // odd: a scale that is not finite has been met
  volatile int* stop = &stop_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;                        // [buffer][block][half of it][row][128 bytes]
  uint8_t* sB = sA + kBufs * kPair * kABytes;   // [buffer][block][column][128 bytes]
  uint8_t* sW = sB + kBufs * kPair * Z::kBBytes;         // [stage][row][slab]
  uint8_t* sAct = sW + S * Z::kWBytes;       // [stage][vector][row]
  uint8_t* sScale = sAct + S * Z::kActBytes; // [stage][group][row]
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full_w[s], 128);
      tc::mbar_init(&full_s[s], 128);
      tc::mbar_init(&empty[s], 16);
    }
    for (int q = 0; q < kBufs; ++q) {
      tc::mbar_init(&ready[q], 16);
      tc::mbar_init(&done[q], 1);
    }
    tc::mbar_init(&fin, 1);
    tc::fence_mbar_init();
    stop_s = odd_s = 0;
  }
  if (warp == 20) tc::tmem_alloc(&tmem_base, kTmemCols);
  grid_dep_wait();   // no global memory is touched before
  grid_dep_launch();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base;
  const long long unwind_ns = a.wait_ns > kUnwindNs ? a.wait_ns : kUnwindNs;
  const int kb0 = blockIdx.x * Z::kSlab, here = min(Z::kSlab, a.blocks - kb0);
  const int n = max(0, min(*a.count, a.cap));
  const int all = (n + kChunk - 1) / kChunk, share = (all + gridDim.y - 1) / gridDim.y;
  const int lo = min(all, (int)blockIdx.y * share), chunks = min(all, lo + share) - lo;

  if (warp < 16) {
    const bool opens = warp < 8;
    const int w8 = warp & 7;
    // codes: this thread's row and chunk of a block
    const int r = w8 * 8 + (lane & 7), c = lane >> 3;
    int step = 0;
    bool ok = true;
    for (int k = 0; ok && k < chunks; ++k) {
      const int slot = k % S;
      if (!wait_warp(&full_w[slot], (k / S) & 1, stop, a, 81) ||
          (!opens && !wait_warp(&full_s[slot], (k / S) & 1, stop, a, 82))) {
        ok = false;
        break;
      }
      const uint8_t* packed = sW + slot * Z::kWBytes + r * Z::kPitch;
      float2 v[Bp / 8];
      if (!opens) {   // (behind the list nothing counts)
        const int u = (lo + k) * kChunk + 2 * lane;
#pragma unroll
        for (int i = 0; i < Bp / 8; ++i) {
          v[i] = *reinterpret_cast<const float2*>(sAct + slot * Z::kActBytes + ((w8 + 8 * i) * kChunk + 2 * lane) * 4);
          if (u >= n) v[i].x = 0.f;
          if (u + 1 >= n) v[i].y = 0.f;
        }
      }
      const bool odd = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&odd_s), 0) != 0;
      for (int j0 = 0; j0 < here; j0 += kPair, ++step) {
        const int q = step % kBufs;
        if (step >= kBufs && !wait_warp(&done[q], (step / kBufs - 1) & 1, stop, a, 83)) {
          ok = false;
          break;
        }
        if (opens) {
          uint4 w[kPair];   // (behind the row's last block: the stage's bytes, which no product reads)
#pragma unroll
          for (int x = 0; x < kPair; ++x)
            w[x] = *reinterpret_cast<const uint4*>(packed + (((4 * (j0 + x) + c) ^ (r & 7)) << 4));
#pragma unroll
          for (int x = 0; x < kPair; ++x) {
            const uint32_t ww[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
            uint8_t* to = sA + (q * kPair + x) * kABytes + r * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // word 4 c + i: elements 8 g .. 8 g + 7 of half i % 2, g = 2 c + i / 2
              uint32_t p[4];
              Open<__nv_bfloat16>::word(ww[i], p);
              *reinterpret_cast<uint4*>(to + (i & 1) * (kChunk * 128) + (((2 * c + (i >> 1)) ^ (r & 7)) << 4)) =
                  make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
        } else {
          uint8_t* to = sB + q * kPair * Z::kBBytes + (((lane >> 2) ^ w8) << 4) + (lane & 3) * 4;   // (a column n: n % 8 = w8)
          float2 s[kPair][kPer];   // (all read before the first store)
#pragma unroll
          for (int x = 0; x < kPair; ++x)
#pragma unroll
            for (int h = 0; h < kPer; ++h)
              s[x][h] = *reinterpret_cast<const float2*>(sScale + slot * Z::kScaleBytes +
                                                         (((j0 + x) * kPer + h) * kChunk + 2 * lane) * 4);
#pragma unroll
          for (int i = 0; i < Bp / 8; ++i) {
            if (w8 + 8 * i >= a.B) break;
            uint32_t p[kPair][kPer][3];
#pragma unroll
            for (int x = 0; x < kPair; ++x)
#pragma unroll
              for (int h = 0; h < kPer; ++h) {
                float cx = v[i].x * s[x][h].x, cy = v[i].y * s[x][h].y;
                if (odd) {   // (an activation of 0 adds nothing, whatever the row holds)
                  if (v[i].x == 0.f) cx = 0.f;
                  if (v[i].y == 0.f) cy = 0.f;
                }
                pieces3(cx, cy, p[x][h]);
              }
#pragma unroll
            for (int x = 0; x < kPair; ++x)
#pragma unroll
              for (int h = 0; h < kPer; ++h)
#pragma unroll
                for (int z = 0; z < 3; ++z)
                  *reinterpret_cast<uint32_t*>(to + x * Z::kBBytes + (h * Z::kOne + z * Bp + w8 + 8 * i) * 128) = p[x][h][z];
          }
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ready[q]);
      }
      if (!ok) break;
      if (lane == 0) tc::mbar_arrive(&empty[slot]);
    }
    if (opens) {
      // ---- sums: a row of the accumulator is an element
      if (chunks > 0) ok = wait_warp(&fin, 0, stop, a, 84) && ok;
      tc::fence_after_sync();
      const int e = (warp & 3) * 32 + lane;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const bool skip = __any_sync(0xffffffffu, *stop != 0) || !ok;
      for (int j = warp >> 2; !skip && j < here; j += 2) {
        float* part = a.part + ((size_t)blockIdx.y * a.B * a.blocks + kb0 + j) * 128 + e;
#pragma unroll
        for (int i = 0; i < Bp / 8; ++i) {
          float p[3][8];
          const uint32_t at = tmem + lanes + j * Z::kN + (two && (warp & 2) ? Z::kOne : 0) + 8 * i;
          if (chunks > 0) {
#pragma unroll
            for (int z = 0; z < 3; ++z) tc::tmem_ld8(at + z * Bp, p[z]);
            tc::tmem_ld_wait();
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int b = 8 * i + k;
            if (b < a.B) part[(size_t)b * a.blocks * 128] = chunks > 0 ? p[2][k] + p[1][k] + p[0][k] : 0.f;
          }
        }
      }
      tc::fence_before_sync();
    }
  } else if (warp < 20) {
    // ---- rows, activations, scales
    constexpr int kLanes = Z::kSlab * 4, kRows = 128 / kLanes, kTurns = kChunk / kRows;   // lanes to a row's slab
    const int t = tid - 512, c = t % kLanes, r0 = t / kLanes;
    constexpr int kMine = (Z::kScales + 1) / 2;   // scales: two threads to a row
    const int sr = t & 63;
    // The list is read two chunks ahead and the scales one: what a chunk waits for was asked
    // for during the chunk before.  (Asked for by the chunk itself, 2 us each: 68 us
    // for 16 vectors by 16050 rows of 7168.)
    int rows[kTurns], mine = 0;
    uint32_t sc[kMine], sc_next[kMine];
    const auto list_of = [&](int k) {   // (an entry outside has activation 0 from the first product on: row 0 is read)
      const int u0 = (lo + k) * kChunk;
#pragma unroll
      for (int i = 0; i < kTurns; ++i) rows[i] = a.list[min(u0 + r0 + i * kRows, n - 1)];
    };
    const auto scales_of = [&](int row, uint32_t* to) {
      const size_t at = (size_t)(row >= 0 && row < a.N ? row : 0) * a.groups;
#pragma unroll
      for (int i = 0; i < kMine; ++i) to[i] = ld_raw<wide>(a.scale, at + min(kb0 * kPer + 2 * i + (t >> 6), a.groups - 1));
    };
    const auto entry = [&](int k) { return a.list[min((lo + k) * kChunk + sr, n - 1)]; };
    if (chunks > 0) {
      list_of(0);
      scales_of(entry(0), sc_next);
      mine = entry(1);
    }
    bool ok = true;
    for (int k = 0; ok && k < chunks; ++k) {
      const int slot = k % S, u0 = (lo + k) * kChunk;
      if (k >= S && !wait_bar(&empty[slot], ((k / S) - 1) & 1, stop, a, 85)) {
        ok = false;
        break;
      }
      uint8_t* to = sW + slot * Z::kWBytes;
      if (c < 4 * here) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          const int r = r0 + i * kRows;
          const size_t j = rows[i] >= 0 && rows[i] < a.N ? rows[i] : 0;
          cp_async16(to + r * Z::kPitch + ((c ^ (r & 7)) << 4), a.q + j * a.pitch + (size_t)kb0 * kQ4BlockBytes + c * 16);
        }
      }
      for (int i = t; i < a.B * (kChunk / 4); i += 128) {   // four activations at a time, up to the list's end
        const int b = i / (kChunk / 4), x = i % (kChunk / 4) * 4;
        if (u0 + x < n)
          cp_async16(sAct + slot * Z::kActBytes + (b * kChunk + x) * 4, a.act + (size_t)b * a.ld_act + u0 + x);
      }
      cp_async_arrive(&full_w[slot]);
#pragma unroll
      for (int i = 0; i < kMine; ++i) sc[i] = sc_next[i];
      scales_of(mine, sc_next);
      list_of(k + 1);
      mine = entry(k + 2);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const float f = of_raw(sc[i], a.dt);
        if (!(fabsf(f) < INFINITY)) *reinterpret_cast<volatile int*>(&odd_s) = 1;
        *reinterpret_cast<float*>(sScale + slot * Z::kScaleBytes + ((2 * i + (t >> 6)) * kChunk + sr) * 4) = f;
      }
      tc::mbar_arrive(&full_s[slot]);
    }
    cp_async_commit();
    cp_async_wait<0>();   // no copy is in flight when the CTA ends
  } else {
    // ---- products
    constexpr uint32_t idesc = tc::idesc_f16(128, Z::kN, true, true, false);
    int step = 0;
    bool ok = true;
    for (int k = 0; ok && k < chunks; ++k)
      for (int j0 = 0; j0 < here; j0 += kPair, ++step) {
        const int q = step % kBufs;
        if (!wait_warp(&ready[q], (step / kBufs) & 1, stop, a, 86)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int x = 0; x < kPair; ++x) {
            if (j0 + x >= here) break;
            const uint32_t at = tc::saddr(sA + (q * kPair + x) * kABytes), y = tc::saddr(sB + (q * kPair + x) * Z::kBBytes);
#pragma unroll
            for (int kk = 0; kk < kChunk / 16; ++kk)
              tc::mma_f16(tmem + (j0 + x) * Z::kN, tc::smem_desc(at + kk * 2048, kChunk * 128, 1024, 2),
                          tc::smem_desc(y + kk * 32, 16, 1024, 2), idesc, (k | kk) != 0);
          }
          tc::mma_commit(&done[q]);
        }
        __syncwarp();
      }
    // every product has ended before tensor memory is given back
    if (tc::elect_one()) tc::mma_commit(&fin);
    __syncwarp();
    (void)tc::mbar_wait(&fin, 0, unwind_ns);
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 20) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int Bp, bool two, bool wide>
cudaError_t run(const Q4Cols& a, int num_sms, cudaStream_t stream) {
  using Z = Cols<Bp, two>;
  static PerDevice attr;   // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(q4_tc_cols_kernel<Bp, two, wide>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Z::kSmem);
  });
  if (ea != cudaSuccess) return ea;
  // a CTA for every SM, of one step's rows each at least; the slabs of a share side by side
  const int slabs = (a.blocks + Z::kSlab - 1) / Z::kSlab, most = (a.cap + kChunk - 1) / kChunk;
  int shares = (num_sms < kQ4Splits ? num_sms : kQ4Splits) / slabs;
  shares = shares < 1 ? 1 : shares > most ? most : shares;
  const cudaError_t e = launch_k(q4_tc_cols_kernel<Bp, two, wide>, dim3(slabs, shares), dim3(kThreads), Z::kSmem, stream, true, 1, a);
  return e == cudaSuccess ? launch_q4_join(a, shares, stream) : e;
}
template <int Bp>
cudaError_t run_group(const Q4Cols& a, int num_sms, cudaStream_t stream) {
  if (a.dt == DV_F32) return a.group == 64 ? run<Bp, true, true>(a, num_sms, stream) : run<Bp, false, true>(a, num_sms, stream);
  return a.group == 64 ? run<Bp, true, false>(a, num_sms, stream) : run<Bp, false, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_q4_tc_cols(const Q4Cols& L, cudaStream_t stream) {
  Q4Cols a = L;
  a.wait_ns = wait_limit_ns();
  const int num_sms = num_sms_current();
  return a.B <= 8 ? run_group<8>(a, num_sms, stream) : a.B <= 16 ? run_group<16>(a, num_sms, stream) : run_group<32>(a, num_sms, stream);
}

}  // namespace dv
