// Matrices in 4 bits (layout: k_q4.cu), several vectors (32-bit ones as three bf16 pieces): products
// with many rows of the matrix on the 5th-generation tensor cores.
//
// A tile is 128 rows; a product is a block of 128 elements of them (M = 128, K = 128)
// with the vectors (N = 16 or 32).  The codes of a block go from registers to tensor
// memory as 16-bit floats, a thread to a row (the A operand: shared memory would have
// to take and give back four times the packed bytes); the vectors come by TMA; the
// accumulator holds one group's sums, which the row's thread takes out, scales and
// adds to its own in fp32 (a group's scale cannot be in the codes, which are
// exact).
//   warps 0-3, 4-7   two groups of 128 threads, a row each: every other block.  Open the
//                    codes, store them to tensor memory, two blocks ahead of the sums
//                    they take out.
//   warps 8-11       packed rows into a ring of shared-memory stages (four blocks, 256
//                    bytes of a row), cp.async, 16 lanes to a row
//   warp 12          the vectors' tiles (TMA), warp 13 the products
// Measured on GB300: 32 bf16 vectors with 28672 rows of 7168 53.3 us (2.1 TB/s of codes and
// scales; m16n8k16 products, which read them from registers, took 152).  A block costs a group
// 1800 cycles, half of them the opening.

#include <climits>

#include "dv_kernels.h"
#include "q4_tc.cuh"
#include "tma_map.h"

namespace dv {
namespace {

constexpr int kThreads = 448;
constexpr int kRowsTile = 128;
constexpr int kStageBlocks = 4;
constexpr uint32_t kRowBytes = kStageBlocks * kQ4BlockBytes;   // of a stage
constexpr uint32_t kWBytes = kRowsTile * kRowBytes;
constexpr uint32_t kTmemCols = 512;

template <int NB>
struct Sizes {
  static constexpr uint32_t kXBlock = 2 * NB * 128;             // the vectors' 128 elements
  static constexpr uint32_t kXBytes = kStageBlocks * kXBlock;
  static constexpr int kStages = NB == 32 ? 3 : 4;
  static constexpr uint32_t kRedBytes = kRowsTile * (NB + 1) * 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * (kWBytes + kXBytes) + kRedBytes;
  static_assert(kSmem + 1024 <= 227 * 1024, "fits an SM");
};

__device__ __forceinline__ void row_groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// A scale as it is stored (asked for here and not where it is used), and its value.
template <typename T> struct Raw {
  unsigned short h;
  __device__ __forceinline__ void ask(const void* s, size_t i) {
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(h) : "l"(static_cast<const uint16_t*>(s) + i));
  }
  __device__ __forceinline__ float value() const { return Elem<T>::to_f(*reinterpret_cast<const T*>(&h)); }
};
template <> struct Raw<float> {
  float f;
  __device__ __forceinline__ void ask(const void* s, size_t i) {
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(f) : "l"(static_cast<const float*>(s) + i));
  }
  __device__ __forceinline__ float value() const { return f; }
};

// CTA c's part of the work: stages [c.lo, c.hi) of all tiles' stages in order, or whole tiles.
// With `split`, tiles that parts meet inside are written to the workspace, at most
// two a CTA, [CTA][its first or its last][vector][row], and q4_tc_join_kernel adds them in order.
struct Part {
  int lo, hi;   // (2^17 tiles of 64 stages at most, times 152: 32 bits)
  __device__ Part(int c, int ctas, int tiles, int stages, int split) {
    const int all = split ? tiles * stages : tiles, unit = split ? 1 : stages;
    lo = all * c / ctas * unit;
    hi = all * (c + 1) / ctas * unit;
  }
};
// The next tile of a part: stages [k0, k1) of it.
struct Walk {
  int at, hi, stages, tile = 0, k0 = 0, k1 = 0;
  __device__ Walk(const Part& p, int s) : at(p.lo), hi(p.hi), stages(s) {}
  __device__ __forceinline__ bool next() {
    if (at >= hi) return false;
    tile = at / stages;
    k0 = at - tile * stages;
    k1 = min(stages, k0 + (hi - at));
    at += k1 - k0;
    return true;
  }
};

// two: groups of 64, an accumulator to each half of a block.  S: the scales' type; float: T is
// bf16 and the columns are the B vectors' first pieces, their second and their third.
template <typename T, typename S_, int NB, bool kList, bool two>
__global__ void __launch_bounds__(kThreads, 1)
    q4_tc_rows_kernel(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ Q4Rows a) {
  using Z = Sizes<NB>;
  constexpr int S = Z::kStages;
  constexpr bool kPieces = sizeof(S_) == 4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_w[S], empty_w[S], full_x[S], empty_x[S], ready[2][2], done[2][2], fin;
  __shared__ uint32_t tmem_base;
  __shared__ int stop_s;
  volatile int* stop = &stop_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sX = smem;
  uint8_t* sW = smem + S * Z::kXBytes;
  float* red = reinterpret_cast<float*>(sW + S * kWBytes);   // [row][NB + 1]
  const long long unwind_ns = a.wait_ns > kUnwindNs ? a.wait_ns : kUnwindNs;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full_w[s], 128);
      tc::mbar_init(&empty_w[s], 8);
      tc::mbar_init(&full_x[s], 1);
      tc::mbar_init(&empty_x[s], 1);
    }
    for (int g = 0; g < 2; ++g)
      for (int q = 0; q < 2; ++q) {
        tc::mbar_init(&ready[g][q], 128);
        tc::mbar_init(&done[g][q], 1);
      }
    tc::mbar_init(&fin, 1);
    tc::fence_mbar_init();
    stop_s = 0;
  }
  if (warp == 13) tc::tmem_alloc(&tmem_base, kTmemCols);
  grid_dep_wait();   // no global memory is touched before
  grid_dep_launch();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base;
  const int n = kList ? max(0, min(*a.count, a.cap)) : a.N;
  const int tiles = (n + kRowsTile - 1) / kRowsTile;
  const int stages = (a.blocks + kStageBlocks - 1) / kStageBlocks;   // of a tile

  const Part own(blockIdx.x, gridDim.x, tiles, stages, a.split);
  Walk walk(own, stages);

  if (warp < 8) {
    // ---- codes to tensor memory, sums out of it
    const int grp = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tA = tmem + grp * 256 + lanes, tD = tA + 128;
    float acc[NB];
    uint32_t made = 0, taken = 0;   // this group's blocks so far, and those whose sums are out
    float s0[2] = {0.f, 0.f}, s1[2] = {0.f, 0.f};   // scales of the blocks under way
    bool ok = true;
    const auto take = [&] {   // the oldest block's sums
      const int q = taken & 1;
      if (!wait_warp(&done[grp][q], (taken >> 1) & 1, stop, a, 71)) return false;
      tc::fence_after_sync();
#pragma unroll
      for (int h = 0; h < (two ? 2 : 1); ++h) {
        const float f = h ? (q ? s1[1] : s0[1]) : (q ? s1[0] : s0[0]);
        float v[NB];
        if constexpr (NB == 32) {
          tc::tmem_ld32(tD + q * (two ? 2 * NB : NB) + h * NB, v);
        } else {
          tc::tmem_ld8(tD + q * (two ? 2 * NB : NB) + h * NB, v);
          tc::tmem_ld8(tD + q * (two ? 2 * NB : NB) + h * NB + 8, v + 8);
        }
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] = fmaf(f, v[i], acc[i]);
      }
      ++taken;
      return true;
    };
    int st = 0;
    // (all eight warps go through all tiles, also once a wait has given up: they meet at their end)
    while (walk.next()) {
      const int u = walk.tile * kRowsTile + r;
      int row = u < n ? u : -1;
      if (kList && u < n) {
        row = a.list[u];
        if (row < 0 || row >= a.N) {
          if (grp == 0) set_error(a.hdr, DV_ERR_INDEX_RANGE, row);
          row = -1;
        }
      }
      const size_t scales = (size_t)max(row, 0) * a.groups;
      // scales of the group's two blocks of a stage, asked for a stage ahead (at their block they
      // were waited for, since a select takes them to their slot's register: 61.5 us for 32 x
      // 28672 x 7168)
      Raw<S_> sc[2][two ? 2 : 1];
      const auto ask = [&](int k) {
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
          const int kb = min(k * kStageBlocks + 2 * j2 + grp, a.blocks - 1), gi = two ? 2 * kb : kb;
          sc[j2][0].ask(a.scale, scales + gi);
          if (two) sc[j2][two].ask(a.scale, scales + min(gi + 1, a.groups - 1));
        }
      };
      ask(walk.k0);
#pragma unroll
      for (int i = 0; i < NB; ++i) acc[i] = 0.f;
      for (int k = walk.k0; ok && k < walk.k1; ++k, ++st) {
        const int slot = st % S;
        if (!wait_warp(&full_w[slot], (st / S) & 1, stop, a, 72)) {
          ok = false;
          break;
        }
        const uint8_t* packed = sW + slot * kWBytes + r * kRowBytes;
        float f[2][two ? 2 : 1];
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2)
#pragma unroll
          for (int h = 0; h < (two ? 2 : 1); ++h) f[j2][h] = sc[j2][h].value();
        ask(k + 1);
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
          const int j = 2 * j2 + grp, kb = k * kStageBlocks + j;
          if (kb >= a.blocks) continue;
          if (made - taken == 2 && !take()) {
            ok = false;
            break;
          }
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(w + 4 * c) =
                *reinterpret_cast<const uint4*>(packed + (((4 * j + c) ^ (r & 7)) << 4));
          const int q = made & 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // words h, h + 2, ... are the half's 32 pairs in order
            uint32_t p[32];
#pragma unroll
            for (int g = 0; g < 8; ++g) Open<T>::word(w[2 * g + h], p + 4 * g);
            tc::tmem_st32(tA + q * 64 + h * 32, p);
          }
          (q ? s1[0] : s0[0]) = f[j2][0];
          if (two) (q ? s1[1] : s0[1]) = f[j2][two];
          tc::tmem_st_wait();
          tc::fence_before_sync();
          tc::mbar_arrive(&ready[grp][q]);
          ++made;
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty_w[slot]);
      }
      while (ok && taken != made) ok = take();
      if (grp == 1) {
#pragma unroll
        for (int i = 0; i < NB; ++i) red[r * (NB + 1) + i] = acc[i];
      }
      row_groups_sync();
      const bool whole = walk.k1 - walk.k0 == stages;
      if (grp == 0 && (u < n || !whole) && !*stop) {
        float* part = a.part + (size_t)(2 * blockIdx.x + (walk.at - (walk.k1 - walk.k0) != own.lo)) * a.B * kRowsTile + r;
        const auto put = [&](int b, float sum) {
          if (kList) {
            bool live = row >= 0;
            if (live && a.member) live = bit_test(a.member + (size_t)b * a.words, row);
            a.act[(size_t)b * a.ld_act + u] = live ? (sum > 0.f || sum != sum ? sum : 0.f) : 0.f;
          } else if (!whole) {
            part[b * kRowsTile] = sum;
          } else {
            float* o = a.out + (size_t)b * a.N + u;
            *o = a.accumulate ? *o + sum : sum;
          }
        };
#pragma unroll
        for (int b = 0; b < NB; ++b) {   // (registers cannot be indexed: unrolled)
          if (b >= (kPieces ? 3 * a.B : a.B)) break;
          float sum = acc[b] + red[r * (NB + 1) + b];
          if (kPieces) {   // (a thread's own row: the least pieces' columns come last)
            red[r * (NB + 1) + b] = sum;
            continue;
          }
          put(b, sum);
        }
        if (kPieces)
          for (int b = 0; b < a.B; ++b) {
            const float* p = red + r * (NB + 1) + b;
            put(b, p[2 * a.B] + p[a.B] + p[0]);
          }
      }
      row_groups_sync();
    }
    tc::fence_before_sync();
  } else if (warp < 12) {
    // ---- packed rows: 16 lanes to a row's 256 bytes, chunk c of row r at c ^ (r % 8)
    const int t = tid - 256, c = t & 15, r0 = t >> 4;
    int st = 0;
    bool ok = true;
    while (ok && walk.next()) {
      int rows[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int u = min(walk.tile * kRowsTile + r0 + 8 * q, n - 1);
        const int l = kList ? a.list[u] : u;
        rows[q] = l >= 0 && l < a.N ? l : 0;
      }
      for (int k = walk.k0; k < walk.k1; ++k, ++st) {
        const int slot = st % S;
        if (st >= S && !wait_bar(&empty_w[slot], ((st / S) - 1) & 1, stop, a, 73)) {
          ok = false;
          break;
        }
        uint8_t* base = sW + slot * kWBytes + r0 * kRowBytes + ((c ^ (r0 & 7)) << 4);
        const uint32_t at = k * kRowBytes + c * 16;
        if (at < a.pitch) {
#pragma unroll
          for (int q = 0; q < 16; ++q)   // (rows 8 apart: the same place in their 256 bytes)
            cp_async16(base + q * 8 * kRowBytes, a.q + (size_t)rows[q] * a.pitch + at);
        }
        cp_async_arrive(&full_w[slot]);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();   // no copy is in flight when the CTA ends
  } else if (warp == 12) {
    // ---- the vectors' tiles
    if (lane == 0) {
      int st = 0;
      bool ok = true;
      while (ok && walk.next())
        for (int k = walk.k0; k < walk.k1; ++k, ++st) {
          const int slot = st % S;
          if (st >= S && !wait_bar(&empty_x[slot], ((st / S) - 1) & 1, stop, a, 74)) {
            ok = false;
            break;
          }
          const int here = min(kStageBlocks, a.blocks - k * kStageBlocks);
          tc::mbar_arrive_expect_tx(&full_x[slot], here * Z::kXBlock);
          for (int j = 0; j < 2 * here; ++j)
            tc::tma_load_2d(sX + slot * Z::kXBytes + j * (Z::kXBlock / 2), &mapX, (k * kStageBlocks * 2 + j) * 64, 0,
                            &full_x[slot]);
        }
      // no copy is in flight when the CTA ends
      for (int s = max(0, st - S); s < st; ++s)
        if (!tc::mbar_wait(&full_x[s % S], (s / S) & 1, unwind_ns)) break;
    }
    __syncwarp();
  } else {
    // ---- products
    constexpr bool kBf16 = !std::is_same<T, __half>::value;
    constexpr uint32_t idesc = tc::idesc_f16(kRowsTile, NB, kBf16, false, false);
    uint32_t made[2] = {0, 0};
    int st = 0;
    bool ok = true;
    while (ok && walk.next())
      for (int k = walk.k0; ok && k < walk.k1; ++k, ++st) {
        const int slot = st % S;
        if (!wait_warp(&full_x[slot], (st / S) & 1, stop, a, 75)) {
          ok = false;
          break;
        }
        const uint32_t x = tc::saddr(sX + slot * Z::kXBytes);
        const int here = min(kStageBlocks, a.blocks - k * kStageBlocks);
        for (int j = 0; j < here; ++j) {
          const int grp = j & 1;
          const uint32_t m = grp ? made[1] : made[0];
          if (!wait_warp(&ready[grp][m & 1], (m >> 1) & 1, stop, a, 76)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint32_t tA = tmem + grp * 256 + (m & 1) * 64, tD = tmem + grp * 256 + 128 + (m & 1) * (two ? 2 * NB : NB);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16_ts(tD + (two ? h * NB : 0), tA + h * 32 + kk * 8,
                               tc::smem_desc(x + j * Z::kXBlock + h * (NB * 128) + kk * 32, 16, 1024, 2), idesc,
                               kk != 0 || (h != 0 && !two));
            tc::mma_commit(&done[grp][m & 1]);
          }
          __syncwarp();
          if (grp) ++made[1]; else ++made[0];
        }
        if (!ok) break;
        if (tc::elect_one()) tc::mma_commit(&empty_x[slot]);
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
  if (warp == 13) tc::tmem_dealloc(tmem, kTmemCols);
}

// Tiles that parts meet inside: the sums of all their parts, in order.  A CTA to every border
// between parts and every vector; the first border inside a tile does it.
__global__ void __launch_bounds__(kRowsTile) q4_tc_join_kernel(const Q4Rows a, int ctas) {
  const int tiles = (a.N + kRowsTile - 1) / kRowsTile, stages = (a.blocks + kStageBlocks - 1) / kStageBlocks;
  const int c = blockIdx.x + 1, b = blockIdx.y, all = tiles * stages;
  const int at = all * c / ctas, t = at / stages, begin = t * stages, before = all * (c - 1) / ctas;
  const int row = t * kRowsTile + threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  if (at == begin || before > begin || row >= a.N) return;
  // (every CTA has a stage at least, and the tile's last is the last that begins in it)
  const int end = min(ctas, ((begin + stages) * ctas + all - 1) / all);
  const size_t pitch = (size_t)a.B * kRowsTile;
  const float* part = a.part + (size_t)b * kRowsTile + threadIdx.x;
  float sum = __ldcg(part + (2 * (c - 1) + (before != begin)) * pitch);
#pragma unroll 4
  for (int k = c; k < end; ++k) sum += __ldcg(part + 2 * k * pitch);
  float* o = a.out + (size_t)b * a.N + row;
  *o = a.accumulate ? *o + sum : sum;
}

template <typename T, typename S, int NB, bool kList, bool two>
cudaError_t run(const Q4Rows& a, bool pdl, int num_sms, cudaStream_t stream) {
  static PerDevice attr;   // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(q4_tc_rows_kernel<T, S, NB, kList, two>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)Sizes<NB>::kSmem);
  });
  if (ea != cudaSuccess) return ea;
  CUtensorMap map;
  if (!make_map(&map, a.x, (uint64_t)a.ldx, (uint64_t)a.cols, NB, !std::is_same<T, __half>::value)) return cudaErrorInvalidValue;
  const int tiles = ((kList ? a.cap : a.N) + kRowsTile - 1) / kRowsTile;
  const int units = a.split ? tiles * ((a.blocks + kStageBlocks - 1) / kStageBlocks) : tiles;
  const int ctas = units < num_sms ? units : num_sms;
  const cudaError_t e = launch_k(q4_tc_rows_kernel<T, S, NB, kList, two>, dim3(ctas), dim3(kThreads), Sizes<NB>::kSmem, stream,
                                 pdl, 1, map, a);
  if (e != cudaSuccess || !a.split || ctas == 1) return e;
  return launch_k(q4_tc_join_kernel, dim3(ctas - 1, a.B), dim3(kRowsTile), 0, stream, true, 1, a, ctas);
}
template <typename T, typename S, int NB>
cudaError_t run_nb(const Q4Rows& a, bool pdl, int num_sms, cudaStream_t stream) {
  if (a.list) return a.group == 64 ? run<T, S, NB, true, true>(a, pdl, num_sms, stream) : run<T, S, NB, true, false>(a, pdl, num_sms, stream);
  return a.group == 64 ? run<T, S, NB, false, true>(a, pdl, num_sms, stream) : run<T, S, NB, false, false>(a, pdl, num_sms, stream);
}

}  // namespace

size_t q4_tc_part_floats(int B) { return B < 2 ? 0 : (size_t)2 * kQ4Splits * B * kRowsTile; }

// A step of a tile costs the same for 3 and for 16 vectors and takes a launch's setting up; m16n8k16
// products cost by the vectors, 16 rows a CTA.  Rows of 5120 in groups of 128, bf16, us, here and there:
//   vectors    2048 rows     5120          10240         40000
//         8     9.0   5.6   12.5  11.9   17.8  17.7    43    51
//        16     9.9   6.0   13.7  13.4   19.2  20.8    45    63
//        32    13.2   7.8   18.0  22.1   23.3  37.1    51   123
// The rule looks at rows and vectors alone, and the border moves with the rows' length: for 8, 16 and
// 32 vectors it lies at 20000, 20000 and 5000 rows of 1024, and at 6000, 4000 and 3000 of 12288.  In
// between the slower form is taken, by a fourth at most (8 vectors by 10240 rows of 1024: 8.9 here and 7.0
// there; 32 by 3584 of 12288: 20.0 and 25.1).  Tiles of a list are
// not cut, and a list is mostly shorter than its bound.
// 32-bit vectors count three times.
bool q4_tc_takes(const Q4Rows& a) {
  if (a.d < 64) return false;
  const int rows = a.list ? a.cap : a.N, some = a.cols <= 8 ? 54 : a.cols <= 16 ? 34 : 24;   // rows for an SM
  return rows >= num_sms_current() * (a.list ? some + some / 2 : some);
}

cudaError_t launch_q4_tc_rows(const Q4Rows& L, dv_dtype dt, WsHeader* hdr, bool pdl, cudaStream_t stream) {
  Q4Rows a = L;
  a.hdr = hdr;
  a.wait_ns = wait_limit_ns();
  const int sms = num_sms_current(), num_sms = sms < kQ4Splits ? sms : kQ4Splits;
  // Tiles are cut where whole ones would leave the SMs idle for a sixth of the time or more (32 x 28672
  // x 7168, 224 tiles: 59.5 us whole, 53.4 cut; 8 x 40000 x 5120, 313: 52 and 43)
  const int tiles = (a.N + kRowsTile - 1) / kRowsTile, turns = (tiles + num_sms - 1) / num_sms;
  a.split = !a.list && tiles * 20 < turns * num_sms * 17 ? 1 : 0;
  const bool few = a.cols <= 16;
  if (dt == DV_F32)
    return few ? run_nb<__nv_bfloat16, float, 16>(a, pdl, num_sms, stream) : run_nb<__nv_bfloat16, float, 32>(a, pdl, num_sms, stream);
  if (dt == DV_F16)
    return few ? run_nb<__half, __half, 16>(a, pdl, num_sms, stream) : run_nb<__half, __half, 32>(a, pdl, num_sms, stream);
  return few ? run_nb<__nv_bfloat16, __nv_bfloat16, 16>(a, pdl, num_sms, stream)
             : run_nb<__nv_bfloat16, __nv_bfloat16, 32>(a, pdl, num_sms, stream);
}

}  // namespace dv
