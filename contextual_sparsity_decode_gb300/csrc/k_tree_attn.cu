// Attention of a drafted token tree over the KV cache.
//
// The T nodes of a sequence's tree sit in the cache slots pos .. pos + T - 1
// behind the committed positions; node t sees every committed position and the
// nodes u with mask[t][u] != 0:
//     out[t] = sum_j p_j V[j] / sum_j p_j,   p_j = exp(scale q_t . K[j] - m)
// with the running maximum m and sum kept in 32 bits, one pass over K and V.
//
// A unit is one (sequence, K/V head, block of query rows): all T g query rows
// of a K/V head share its K and V, so K and V are read once for the whole tree
// (rows r = t g + e, e < g the query heads of the K/V head).  Units are cut
// into tiles of 64 keys.  The grid is persistent, and every CTA takes an equal
// share of all units' tiles, in order, whatever the sequences' lengths (read on
// the device); a unit that crosses CTAs leaves a partial result (maximum, sum,
// numerator) per CTA, and a second small kernel joins them in tile order, so
// results do not depend on timing.  (Joined by the last of its CTAs to finish,
// behind a fence and an atomic counter, one sequence of 8 nodes over 512
// positions took 17.6 us instead of 13.2, and three of 125 rows over 32768
// positions 98 instead of 83.)

// Bound by the reads of K and V for trees of up to 128 rows a K/V head.  Measured
// on GB300: 8 sequences of 64 nodes over 2047 positions of 96 heads of 128 (f16,
// 855 MB): 160 us, 5.3 TB/s, 0.79 of a plain copy's rate; 3 of 25 x 5 rows over
// up to 32768 positions of 8 heads (bf16, 398 MB): 82 us, 4.8 TB/s; one of 8
// nodes over 512 positions of 32 heads of 64: 12 us, all latency.

#include <cuda.h>

#include <type_traits>

#include "dv_kernels.h"
#include "tc_common.cuh"
#include "tma_map.h"

namespace dv {
namespace {

typedef unsigned long long u64;

constexpr int kKeys = 64;      // keys per tile

struct TreeArgs {
  TreeLaunch L;
  float scale_log2;            // scale log2(e): exponentials are taken to base 2
  WsHeader* hdr;
  long long wait_ns;
};

// What every role of a CTA needs to walk its share of the tiles.  Tile numbers
// fit 32 bits: the host refuses shapes whose tiles might not.
struct TreePlan {
  uint32_t pre[kTreeMaxB + 1];   // tiles of the sequences before b
  int pos[kTreeMaxB], nodes[kTreeMaxB];
};

struct Seg {
  int b, head, row0, rows;       // rows row0 .. row0 + rows - 1 of the sequence's T g
  int pos, nodes, n;             // committed positions, tree nodes, their sum
  int k0, k1, tiles;             // tiles [k0, k1) of the unit's `tiles`
  bool ok;                       // the head index is in range
};

// Checks and lengths of sequence b; returns its tiles.
__device__ __forceinline__ uint32_t plan_one(const TreeArgs& a, TreePlan* p, int b, int rows_per_unit) {
  const TreeLaunch& L = a.L;
  const bool report = blockIdx.x == 0;
  const int n = L.pos[b];
  int nd = L.nodes ? L.nodes[b] : L.T;
  int cnt = L.head_idx ? L.head_count[b] : L.h;
  if (nd > L.T) {
    if (report) set_error(a.hdr, DV_ERR_CAPACITY, nd);
    nd = L.T;
  }
  if (L.head_idx && cnt > L.cap) {
    if (report) set_error(a.hdr, DV_ERR_CAPACITY, cnt);
    cnt = L.cap;
  }
  if (nd > 0 && (n < 0 || n > L.n_max - nd)) {
    if (report) set_error(a.hdr, DV_ERR_POSITION, n);
    nd = 0;
  }
  nd = max(nd, 0);
  p->pos[b] = n;
  p->nodes[b] = nd;
  if (nd == 0 || cnt <= 0) return 0;
  uint32_t work = (uint32_t)cnt * (uint32_t)((n + nd + kKeys - 1) / kKeys);
  if (nd * L.g > rows_per_unit) work *= (uint32_t)((nd * L.g + rows_per_unit - 1) / rows_per_unit);
  return work;
}

// Lengths of all sequences and the prefix sums of their tiles.  NT threads;
// ends with a barrier (the only one up to 32 sequences, which one warp plans).
template <int NT>
__device__ __forceinline__ void tree_plan(const TreeArgs& a, TreePlan* p, int rows_per_unit) {
  const int tid = threadIdx.x, B = a.L.B;
  if (B > 32) {
    for (int b = tid; b < B; b += NT) p->pre[b + 1] = plan_one(a, p, b, rows_per_unit);
    __syncthreads();
  }
  if (tid < 32) {
    uint32_t carry = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + tid;
      uint32_t v = b >= B ? 0 : B > 32 ? p->pre[b + 1] : plan_one(a, p, b, rows_per_unit);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (tid >= o) v += u;
      }
      v += carry;
      if (b < B) p->pre[b + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (tid == 0) p->pre[0] = 0;
  }
  __syncthreads();
}

// A unit that several CTAs share, as the join reads it: written by the CTA whose
// share holds the unit's first tile (a share has at most one such unit, its
// last); count 0: none.
struct __align__(16) Shared {
  int b, head, row0, rows;
  int count, pad[3];
};
static_assert(sizeof(Shared) == kTreeSharedBytes, "workspace size");

// Walks the segments of this CTA's share of the tiles: of W tiles, the first
// W % G of the G CTAs that take part get one more than W / G.
struct Cursor {
  uint32_t t, t1;   // next tile, end of the share
  uint32_t q, r;    // W / G, W % G
  int b;
  __device__ Cursor(const TreePlan& p, int B) {
    const uint32_t W = p.pre[B], G = min(W, gridDim.x), c = blockIdx.x;
    t = t1 = q = r = 0;
    b = 0;
    if (c >= G) return;
    q = W / G;
    r = W - q * G;
    t = c * q + min(c, r);
    t1 = t + q + (c < r);
    int hi = B;  // b: the last with pre[b] <= t
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (p.pre[mid] <= t) b = mid;
      else hi = mid;
    }
  }
  // The CTA whose share holds tile x.
  __device__ int cta_of(uint32_t x) const {
    const uint32_t wide = r * (q + 1);
    return (int)(x < wide ? x / (q + 1) : r + (x - wide) / q);
  }
  __device__ __forceinline__ bool next(const TreeLaunch& L, const TreePlan& p, int rows_per_unit, Seg* s) {
    if (t >= t1) return false;
    while (p.pre[b + 1] <= t) ++b;
    s->b = b;
    s->pos = p.pos[b];
    s->nodes = p.nodes[b];
    s->n = s->pos + s->nodes;
    const int all_rows = s->nodes * L.g;
    s->tiles = (s->n + kKeys - 1) / kKeys;
    const uint32_t off = t - p.pre[b];
    uint32_t slot = off / (uint32_t)s->tiles;
    s->k0 = (int)(off - slot * s->tiles);
    s->k1 = (int)min((uint32_t)s->tiles, s->k0 + (t1 - t));
    s->row0 = 0;
    if (all_rows > rows_per_unit) {
      const uint32_t blocks = (all_rows + rows_per_unit - 1) / rows_per_unit, unit = slot;
      slot = unit / blocks;
      s->row0 = (int)(unit - slot * blocks) * rows_per_unit;
    }
    s->rows = min(rows_per_unit, all_rows - s->row0);
    s->head = L.head_idx ? L.head_idx[(size_t)b * L.cap + slot] : (int)slot;
    s->ok = s->head >= 0 && s->head < L.h;
    t += s->k1 - s->k0;
    return true;
  }
  // The shared unit that begins in this CTA's share, once its last segment s
  // (the one that next() gave last) is done; called by one thread.
  __device__ void describe(const Seg& s, bool any, Shared* out) const {
    Shared d{};
    if (any && s.ok && s.k0 == 0 && s.k1 < s.tiles) {
      d.b = s.b; d.head = s.head; d.row0 = s.row0; d.rows = s.rows;
      d.count = cta_of(t - s.k1 + s.tiles - 1) - (int)blockIdx.x + 1;
    }
    reinterpret_cast<int4*>(out)[0] = make_int4(d.b, d.head, d.row0, d.rows);
    reinterpret_cast<int4*>(out)[1] = make_int4(d.count, 0, 0, 0);
  }
};

// Query row r of unit (b, head): its offset in q and out.
template <typename Unit>
__device__ __forceinline__ size_t row_offset(const TreeLaunch& L, const Unit& s, int r, int d_h) {
  const int rr = s.row0 + r, t = rr / L.g, e = rr - t * L.g;
  return (((size_t)s.b * L.T + t) * L.h * L.g + (size_t)s.head * L.g + e) * d_h;
}

// Whether node t sees slot u of the tree.
__device__ __forceinline__ bool sees(const TreeLaunch& L, const Seg& s, int t, int u) {
  if (u >= s.nodes) return false;
  if (!L.mask) return u <= t;
  return L.mask[s.b * L.mask_stride + (size_t)t * L.T + u] != 0;
}

__device__ __forceinline__ size_t piece_slot(int cta, bool first) { return (size_t)cta * 2 + (first ? 1 : 0); }

template <typename T>
__device__ __forceinline__ void store4(T* dst, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void store4<float>(float* dst, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
}
template <>
__device__ __forceinline__ void store4<__half>(__half* dst, float a, float b, float c, float d) {
  const __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* dst, float a, float b, float c, float d) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// Rows that no unit writes are zero: heads outside the list, nodes behind the
// last of a tree that is not full, sequences that were refused.
template <typename T, int DH>
__device__ void zero_rows(const TreeLaunch& L, const TreePlan& p, int worker, int workers, int lane, int lanes) {
  if (!L.head_idx && !L.nodes) {
    bool all = true;
    for (int b = lane; b < L.B; b += lanes) all &= p.nodes[b] == L.T;
    if (__all_sync(0xffffffffu, all)) return;
  }
  constexpr int kVec = 16 / sizeof(T);
  const int row_vecs = DH / kVec;
  for (int w = worker; w < L.B * L.h; w += workers) {
    const int b = w / L.h, i = w - b * L.h;
    bool mine = !L.head_idx;
    if (L.head_idx) {
      const int cnt = max(0, min(L.head_count[b], L.cap));
      bool found = false;
      for (int k = lane; k < cnt; k += lanes) found |= L.head_idx[(size_t)b * L.cap + k] == i;
      mine = __any_sync(0xffffffffu, found);
    }
    const int t0 = mine ? p.nodes[b] : 0;
    for (int e = lane; e < (L.T - t0) * L.g * row_vecs; e += lanes) {
      const int rr = e / row_vecs, c = e - rr * row_vecs;
      const int t = t0 + rr / L.g, x = rr % L.g;
      T* dst = static_cast<T*>(L.out) + (((size_t)b * L.T + t) * L.h * L.g + (size_t)i * L.g + x) * DH + c * kVec;
      *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
    }
  }
}

// Bit i: byte i of a 16-byte vector is not 0.
__device__ __forceinline__ uint32_t nonzero16(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = ((((w[i] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w[i]) >> 7) & 0x01010101u;
    bits |= ((top * 0x10204080u) >> 28) << (4 * i);
  }
  return bits;
}

// Bit i: the row sees key j0 + i.  t: the row's node.  The mask bytes come in
// the aligned vectors that cover them, all in flight together (64 byte loads,
// eight at a time, took 4500 cycles a tile); a vector that would reach outside
// the mask is read byte by byte.
__device__ __forceinline__ unsigned long long visible_keys(const TreeLaunch& L, const Seg& s, int j0, int t) {
  const int u0 = j0 - s.pos;                                   // tree slot of the tile's first key
  const int lo = min(max(-u0, 0), kKeys), hi = min(max(s.nodes - u0, 0), kKeys);
  const unsigned long long below = lo >= 64 ? ~0ull : (1ull << lo) - 1;
  if (!L.mask) {
    const int top = min(max(t + 1 - u0, lo), hi);
    return top >= 64 ? ~0ull : (1ull << top) - 1;
  }
  if (hi <= lo) return below;
  const uint8_t* first = L.mask;
  const uint8_t* end = first + (L.mask_stride ? L.B * L.mask_stride : (long long)L.T * L.T);
  const uint8_t* p = first + s.b * L.mask_stride + (long long)t * L.T + u0 + lo;
  const int n = hi - lo, off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint8_t* base = p - off;
  uint4 v[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    v[k] = make_uint4(0, 0, 0, 0);
    const uint8_t* at = base + 16 * k;
    if (16 * k < off + n && at >= first && at + 16 <= end) v[k] = __ldg(reinterpret_cast<const uint4*>(at));
  }
  unsigned long long bits = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) bits |= (unsigned long long)nonzero16(v[k]) << (16 * k);
  bits >>= off;
  if (off) bits |= (unsigned long long)nonzero16(v[4]) << (64 - off);
  for (int k = 0; k < 5; ++k) {
    const uint8_t* at = base + 16 * k;
    if (16 * k >= off + n || (at >= first && at + 16 <= end)) continue;
    for (int i = max(16 * k - off, 0); i < min(16 * k + 16 - off, n); ++i)
      bits |= (unsigned long long)(p[i] != 0) << i;
  }
  if (n < 64) bits &= (1ull << n) - 1;
  return below | (bits << lo);
}

// ---- CUDA cores (32-bit storage) ----------------------------------------------
//
// Units of 16 query rows.  K and V tiles come by cp.async into two buffers.
//   scores      thread = one key, four rows
//   softmax     a warp to two rows, a lane to two keys
//   numerators  thread = four columns and a group of a tile's keys, all rows in
//               registers over the whole segment (a key's V is read once, a
//               weight once for four columns); the key groups are added at the
//               segment's end.

constexpr int kSimtRows = 16;
constexpr int kSimtThreads = 256;

template <int DH>
struct SimtSmem {
  TreePlan plan;
  alignas(16) float q[kSimtRows][DH];
  alignas(16) float k[2][kKeys][DH + 4];       // at the segment's end: [8][kSimtRows][DH] partial numerators
  alignas(16) float v[2][kKeys][DH];
  alignas(16) float s[kSimtRows][kKeys + 4];   // scores, then weights
  float alpha[kSimtRows], m[kSimtRows], l[kSimtRows];
  u64 vis[kSimtRows];                          // edge tiles: the keys that a row sees
};

template <int DH>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<DH>& sm = *reinterpret_cast<SimtSmem<DH>*>(smem_raw);
  const TreeLaunch& L = a.L;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  constexpr int kChunks = DH / 4, kGroups = kSimtThreads / kChunks, kMine = kKeys / kGroups;
  constexpr int kCols = DH / 16;   // output columns of a thread at the end
  static_assert(8 * kSimtRows * DH <= 2 * kKeys * (DH + 4), "the partial numerators fit into the K buffers");
  grid_dep_wait();
  grid_dep_launch();
  tree_plan<kSimtThreads>(a, &sm.plan, kSimtRows);
  zero_rows<float, DH>(L, sm.plan, blockIdx.x * (kSimtThreads / 32) + wid, gridDim.x * (kSimtThreads / 32), lane, 32);
  Cursor cur(sm.plan, L.B);
  Seg s{};
  bool any = false;
  while (cur.next(L, sm.plan, kSimtRows, &s)) {
    any = true;
    if (!s.ok) {
      if (tid == 0) set_error(a.hdr, DV_ERR_INDEX_RANGE, s.head);
      continue;
    }
    const size_t kv0 = ((size_t)s.b * L.h + s.head) * L.n_max * DH;
    const auto fetch = [&](int kt, int buf) {
      const int j0 = kt * kKeys;
      for (int i = tid; i < kKeys * kChunks; i += kSimtThreads) {
        const int j = i / kChunks, c = (i % kChunks) * 4, there = j0 + j < s.n ? 16 : 0;
        const size_t at = kv0 + (size_t)(there ? j0 + j : j0) * DH + c;
        cp_async16_or_zero(&sm.k[buf][j][c], static_cast<const float*>(L.K) + at, there);
        cp_async16_or_zero(&sm.v[buf][j][c], static_cast<const float*>(L.V) + at, there);
      }
    };
    __syncthreads();  // the previous segment's shared memory is no longer read
    fetch(s.k0, 0);
    for (int i = tid; i < kSimtRows * kChunks; i += kSimtThreads) {
      const int r = i / kChunks, c = (i % kChunks) * 4;
      cp_async16_or_zero(&sm.q[r][c],
                         static_cast<const float*>(L.q) + (r < s.rows ? row_offset(L, s, r, DH) + c : (size_t)0),
                         r < s.rows ? 16 : 0);
    }
    cp_async_commit();
    if (tid < kSimtRows) {
      sm.m[tid] = -INFINITY;
      sm.l[tid] = 0.f;
    }
    const int c4 = tid % kChunks, grp = tid / kChunks;
    float acc[kSimtRows][4];
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.f;
    for (int kt = s.k0; kt < s.k1; ++kt) {
      const int j0 = kt * kKeys, buf = (kt - s.k0) & 1;
      const bool edge = j0 + kKeys > s.pos;   // the tile holds tree nodes, or ends behind the last
      if (kt + 1 < s.k1) fetch(kt + 1, buf ^ 1);
      cp_async_commit();
      if (edge && tid < s.rows) sm.vis[tid] = visible_keys(L, s, j0, (s.row0 + tid) / L.g);
      cp_async_wait<1>();
      __syncthreads();
      const int j = tid & (kKeys - 1), r0 = (tid / kKeys) * 4;
      if (r0 < s.rows) {  // scores
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int c = 0; c < DH; c += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[buf][j][c]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[r0 + r][c]);
            d[r] = fmaf(q4.x, k4.x, d[r]); d[r] = fmaf(q4.y, k4.y, d[r]);
            d[r] = fmaf(q4.z, k4.z, d[r]); d[r] = fmaf(q4.w, k4.w, d[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool seen = r0 + r < s.rows && (!edge || ((sm.vis[r0 + r] >> j) & 1));
          sm.s[r0 + r][j] = seen ? d[r] * a.scale_log2 : -INFINITY;
        }
      }
      __syncthreads();
#pragma unroll
      for (int rr = 0; rr < kSimtRows / 8; ++rr) {  // softmax
        const int r = wid + rr * 8;
        if (r >= s.rows) continue;
        const float s0 = sm.s[r][lane], s1 = sm.s[r][lane + 32];
        const float mo = sm.m[r], mn = fmaxf(mo, warp_max(fmaxf(s0, s1)));
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float p0 = exp2f(s0 - mu), p1 = exp2f(s1 - mu);
        const float sum = warp_sum(p0 + p1);
        sm.s[r][lane] = p0;
        sm.s[r][lane + 32] = p1;
        if (lane == 0) {
          const float al = mo == -INFINITY ? 0.f : exp2f(mo - mu);
          sm.alpha[r] = al;
          sm.m[r] = mn;
          sm.l[r] = fmaf(sm.l[r], al, sum);
        }
      }
      __syncthreads();
      {  // numerators
        float4 v[kMine];
#pragma unroll
        for (int k = 0; k < kMine; ++k) v[k] = *reinterpret_cast<const float4*>(&sm.v[buf][grp * kMine + k][c4 * 4]);
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) {
          if (r >= s.rows) break;
          const float al = sm.alpha[r];
          float o0 = acc[r][0] * al, o1 = acc[r][1] * al, o2 = acc[r][2] * al, o3 = acc[r][3] * al;
          // a V row that the row does not see must not reach it, whatever it
          // holds (0 x inf)
          const uint32_t seen = edge ? (uint32_t)(sm.vis[r] >> (grp * kMine)) : ~0u;
#pragma unroll
          for (int k = 0; k < kMine; k += 4) {
            const float4 p = *reinterpret_cast<const float4*>(&sm.s[r][grp * kMine + k]);
            const float pk[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (edge && !((seen >> (k + x)) & 1)) continue;
              o0 = fmaf(pk[x], v[k + x].x, o0); o1 = fmaf(pk[x], v[k + x].y, o1);
              o2 = fmaf(pk[x], v[k + x].z, o2); o3 = fmaf(pk[x], v[k + x].w, o3);
            }
          }
          acc[r][0] = o0; acc[r][1] = o1; acc[r][2] = o2; acc[r][3] = o3;
        }
      }
      __syncthreads();  // the buffers are read
    }
    // the key groups' numerators: lanes 16 apart first where a warp holds two
    float* red = &sm.k[0][0][0];
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) {
      if (r >= s.rows) break;
      if (kGroups == 16) {
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[r][x] += __shfl_xor_sync(0xffffffffu, acc[r][x], 16);
      }
      if (kGroups == 8 || lane < 16)
        *reinterpret_cast<float4*>(red + (wid * kSimtRows + r) * DH + c4 * 4) =
            make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    }
    __syncthreads();
    const int r = tid / 16, c0 = (tid % 16) * 4;
    if (r < s.rows) {
      const bool whole = s.k1 - s.k0 == s.tiles;
      const float l = sm.l[r], inv = l == 0.f ? 0.f : 1.f / l;
      const size_t slot = piece_slot(blockIdx.x, s.k0 == 0);
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 x = *reinterpret_cast<const float4*>(red + (g * kSimtRows + r) * DH + c0 + c * 16);
          o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
        }
        if (whole)
          store4<float>(static_cast<float*>(L.out) + row_offset(L, s, r, DH) + c0 + c * 16, o.x * inv, o.y * inv,
                        o.z * inv, o.w * inv);
        else
          __stcg(reinterpret_cast<float4*>(L.part) + (slot * (DH / 4) + (c0 + c * 16) / 4) * L.rows_pad + r, o);
      }
      if (!whole && c0 == 0) __stcg(&L.ml[slot * L.rows_pad + r], make_float2(sm.m[r], l));
    }
  }
  if (tid == 0) cur.describe(s, any, static_cast<Shared*>(L.shared) + blockIdx.x);
}

// ---- tensor cores (16-bit storage) ------------------------------------------------
//
// S = Q K^T and O += P V on tcgen05: M = 128 query rows (rows behind the unit's
// last hold anything: a row of the product depends on its own row of Q and P
// alone), fp32 accumulators in tensor memory.  Tiles go in pairs: one S of 128
// keys (half as many reads of Q from shared memory as two of 64, and those
// bound the product at N = 64), then one softmax group and one P V for each
// tile of the pair.
//   warp 8   one thread issues the TMA loads: K by pairs, V by tiles, two rings
//   warp 9   issues the MMAs
//   warp 10  copies the next unit's query rows (swizzled, two buffers)
//   warps 0-3 and 4-7  the two softmax groups, a thread to a row: no value
//            crosses threads.  Each group has its own maximum, sum and
//            accumulator O; they are joined at the end of the segment.  S is
//            read into registers at once, so that the next pair's S is
//            computed while the groups work on this one's.
// P goes back to tensor memory (the A operand of the second product) as the
// sum of two 16-bit halves hi + lo: one rounding of P to bf16 would put as
// large an error into O as the output's own rounding; the two halves leave
// 2^-17.  The second MMA is not free: without it 8 x 64 nodes took 153 us
// instead of 162.  A tile of 64 keys is 32 KB, about 1400 cycles at an SM's
// share of the memory; its three products take about 770 (4096 products a
// cycle), and the tensor pipe is busy 0.41 of the time.
// The reference maximum moves only when a tile's maximum exceeds it by 2^8
// (P <= 2^14 with the 2^6 that keeps small weights out of f16's subnormals):
// rescaling O is rare.

constexpr int kTcThreads = 352;
constexpr int kTcTmemCols = 512;
// columns of group w: O at w DH, S at 256 + 64 w, P (two halves of 32) at 384 + 64 w
constexpr uint32_t kColO = 0, kColS = 256, kColP = 384;
constexpr float kShift = 6.f, kSlack = 8.f;
constexpr long long kUnwindNs = 2000000000LL;

template <int DH>
struct TcSizes {
  static constexpr int kPairs = DH == 128 ? 2 : 4, kTiles = DH == 128 ? 5 : 8;   // ring depths: K pairs, V tiles
  static constexpr uint32_t kQBytes = kTreeRows * DH * 2;
  static constexpr uint32_t kTileBytes = kKeys * DH * 2, kPairBytes = 2 * kTileBytes;
  static constexpr size_t kSmem = 1024 + 2 * kQBytes + kPairs * kPairBytes + kTiles * kTileBytes;
};

// A wait that ends: at its phase, when another wait of the CTA gave up, or at
// the limit (recorded as DV_ERR_TIMEOUT; the CTA then unwinds, its results
// being void).  Returns whether the phase was reached.  Only the first try is
// inlined: the loop's dozen waits are on the path of every tile, and with their
// slow parts in line the kernel took 168 us instead of 160.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* stop, WsHeader* hdr,
                                       long long wait_ns, int code) {
  const unsigned long long t0 = globaltimer_ns();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if ((long long)(globaltimer_ns() - t0) > wait_ns) {
      *stop = 1;
      set_error(hdr, DV_ERR_TIMEOUT, code);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* stop, const TreeArgs& a,
                                         int code) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, stop, a.hdr, a.wait_ns, code);
}
// The same by a converged warp (lanes may differ in their answers).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* stop, const TreeArgs& a,
                                          int code) {
  const bool ok = wait_bar(bar, parity, stop, a, code);
  __syncwarp();
  return ok;
}

template <int N>
__device__ __forceinline__ void group_sync() {  // the eight softmax warps
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

template <typename T> struct Half2;
template <> struct Half2<__half> {
  static constexpr uint32_t kExp = 0x7c00u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 open(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
};
template <> struct Half2<__nv_bfloat16> {
  static constexpr uint32_t kExp = 0x7f80u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 open(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
};

// The V rows of a tile that not every row may see, in shared memory before the
// product reads them: rows behind the last node become 0, and so do values of
// tree nodes that are not finite (0 x inf would reach rows that do not see
// them); returns whether there were any of those.
template <typename T, int DH>
__device__ __forceinline__ bool clean_v(uint8_t* v, const Seg& s, int j0, int tid) {
  constexpr int kRowChunks = DH / 8;
  bool found = false;
  for (int i = tid; i < kKeys * kRowChunks; i += 128) {
    const int r = i / kRowChunks, c = i % kRowChunks, j = j0 + r;
    if (j < s.pos) continue;
    uint4* p = reinterpret_cast<uint4*>(v + (c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    if (j >= s.n) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 x = *p;
    uint32_t* w = &x.x;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      constexpr uint32_t lo = Half2<T>::kExp, hi = lo << 16;
      if ((w[e] & lo) == lo) { w[e] &= 0xffff0000u; bad = true; }
      if ((w[e] & hi) == hi) { w[e] &= 0x0000ffffu; bad = true; }
    }
    if (bad) *p = x;
    found |= bad;
  }
  return found;
}

// Makes an edge tile (tile j of the segment: it holds tree nodes, or ends behind
// the last) ready: its V rows, which are there, clean; returns the keys that the
// row sees.  By a softmax group.  The V stage's barrier was at this tile's phase
// or the one before when it was waited for: the product that freed the stage
// had been.
template <typename T, int DH>
__device__ __forceinline__ u64 prepare_edge(const TreeLaunch& L, int b, int pos, int nodes, uint8_t* v, int j0, int t,
                                         bool active, int* bad) {
  Seg s{};
  s.b = b; s.pos = pos; s.nodes = nodes; s.n = pos + nodes;
  const u64 seen = active ? visible_keys(L, s, j0, t) : ~0ull;
  if (clean_v<T, DH>(v, s, j0, threadIdx.x & 127)) *bad = 1;
  tc::fence_proxy_async();
  return seen;
}

template <typename T, int DH>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                   const __grid_constant__ TreeArgs a) {
  using Z = TcSizes<DH>;
  constexpr int NK = Z::kPairs, NV = Z::kTiles, kBoxes = DH / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TreePlan plan;
  __shared__ uint64_t kfull[NK], kempty[NK], vfull[NV], vempty[NV], qfull[2], qempty[2], sfull, sfree, pready[2],
      pdone[2], ofull, odone, done;
  __shared__ float2 sml[2][2][kTreeRows];   // [segment parity][group][row] maximum and sum
  __shared__ uint32_t tmem_base;
  __shared__ int stop_s, bad_v[4];
  const TreeLaunch& L = a.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * Z::kQBytes;
  uint8_t* sV = sK + NK * Z::kPairBytes;
  volatile int* stop = &stop_s;
  const long long unwind_ns = a.wait_ns > kUnwindNs ? a.wait_ns : kUnwindNs;

  if (tid == 0) {
    for (int q = 0; q < NK; ++q) {
      tc::mbar_init(&kfull[q], 1);
      tc::mbar_init(&kempty[q], 1);
    }
    for (int q = 0; q < NV; ++q) {
      tc::mbar_init(&vfull[q], 1);
      tc::mbar_init(&vempty[q], 1);
    }
    for (int q = 0; q < 2; ++q) {
      tc::mbar_init(&qfull[q], 32);
      tc::mbar_init(&qempty[q], 1);
      tc::mbar_init(&pready[q], 128);
      tc::mbar_init(&pdone[q], 1);
    }
    tc::mbar_init(&sfull, 1);
    tc::mbar_init(&sfree, 256);
    tc::mbar_init(&ofull, 1);
    tc::mbar_init(&odone, 256);
    tc::mbar_init(&done, 1);
    tc::fence_mbar_init();
    stop_s = 0;
    bad_v[0] = bad_v[1] = bad_v[2] = bad_v[3] = 0;
  }
  if (tid == 256) {
    tc::prefetch_map(&mapK);
    tc::prefetch_map(&mapV);
  }
  if (warp == 9) tc::tmem_alloc(&tmem_base, kTcTmemCols);
  grid_dep_wait();  // no global memory is touched before
  grid_dep_launch();
  tc::fence_before_sync();
  tree_plan<kTcThreads>(a, &plan, kTreeRows);  // ends with a barrier
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base;
  Cursor cur(plan, L.B);
  Seg s{};

  if (warp == 8) {
    if (lane == 0) {  // TMA producer
      int kp = 0, vt = 0;   // pairs and tiles issued
      while (!*stop && cur.next(L, plan, kTreeRows, &s)) {
        if (!s.ok) continue;
        const int z = s.b * L.h + s.head;
        for (int kt = s.k0; kt < s.k1 && !*stop; kt += 2) {
          const int two = min(2, s.k1 - kt);
          {
            const int st = kp % NK, use = kp / NK;
            if (use && !wait_bar(&kempty[st], (use - 1) & 1, stop, a, 31)) break;
            tc::mbar_arrive_expect_tx(&kfull[st], two * Z::kTileBytes);
            for (int h = 0; h < two; ++h)
#pragma unroll
              for (int x = 0; x < kBoxes; ++x)
                tc::tma_load_3d(sK + st * Z::kPairBytes + x * (2 * kKeys * 128) + h * (kKeys * 128), &mapK, x * 64,
                                (kt + h) * kKeys, z, &kfull[st]);
            ++kp;
          }
          for (int h = 0; h < two; ++h) {
            const int st = vt % NV, use = vt / NV;
            if (use && !wait_bar(&vempty[st], (use - 1) & 1, stop, a, 32)) break;
            tc::mbar_arrive_expect_tx(&vfull[st], Z::kTileBytes);
#pragma unroll
            for (int x = 0; x < kBoxes; ++x)
              tc::tma_load_3d(sV + st * Z::kTileBytes + x * (kKeys * 128), &mapV, x * 64, (kt + h) * kKeys, z,
                              &vfull[st]);
            ++vt;
          }
        }
      }
      // no copy into this CTA's shared memory may be in flight when it exits
      for (int q = max(0, kp - NK); q < kp; ++q)
        if (!tc::mbar_wait_soon(&kfull[q % NK], (q / NK) & 1, unwind_ns)) break;
      for (int q = max(0, vt - NV); q < vt; ++q)
        if (!tc::mbar_wait_soon(&vfull[q % NV], (q / NV) & 1, unwind_ns)) break;
    }
    __syncwarp();
  } else if (warp == 9) {  // MMA issuer
    // The whole warp walks the loop and one lane issues, so that counters and
    // descriptors are warp-uniform: issued from inside a one-lane branch, the
    // 16 MMAs of a tile took 1200 cycles to issue and bounded the kernel.
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t idS1 = tc::idesc_f16(kTreeRows, kKeys, kBf16, false, false),
                   idS2 = tc::idesc_f16(kTreeRows, 2 * kKeys, kBf16, false, false);
    const uint32_t idO = tc::idesc_f16(kTreeRows, DH, kBf16, false, /*B MN-major*/ true);
    const uint64_t qd0 = tc::smem_desc(tc::saddr(sQ), 16, 1024, 2), kd0 = tc::smem_desc(tc::saddr(sK), 16, 1024, 2);
    // V (MN-major): 16 keys = two 8-row groups (1024 B apart), the 64-column
    // halves kKeys * 128 bytes apart
    const uint64_t vd0 = tc::smem_desc(tc::saddr(sV), kKeys * 128, 1024, 2);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t ks = 0, kph = 0, vs = 0, vph = 0;   // ring stages and their phases
    uint32_t p_ph = 0;                           // bit w: group w
    int sg = 0, pairs = 0;                       // segments begun, S issued
    while (cur.next(L, plan, kTreeRows, &s)) {
      if (!s.ok) continue;
      const int nt = __shfl_sync(0xffffffffu, s.k1 - s.k0, 0);
      bool ok = wait_warp(&qfull[sg & 1], (sg >> 1) & 1, stop, a, 33);
      const uint64_t qd = qd0 + (sg & 1) * (Z::kQBytes >> 4);
      auto issue_s = [&](bool two) {
        if (pairs) ok &= wait_warp(&sfree, (pairs - 1) & 1, stop, a, 43);
        ++pairs;
        ok &= wait_warp(&kfull[ks], kph, stop, a, 34);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint64_t kd = kd0 + ks * (Z::kPairBytes >> 4);
          const uint32_t id = two ? idS2 : idS1;
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            tc::mma_f16(tm + kColS, qd + ((kk >> 2) * (kTreeRows * 128) + (kk & 3) * 32) / 16,
                        kd + ((kk >> 2) * (2 * kKeys * 128) + (kk & 3) * 32) / 16, id, kk != 0);
          tc::mma_commit(&sfull);
          tc::mma_commit(&kempty[ks]);
        }
        __syncwarp();
        if (++ks == NK) { ks = 0; kph ^= 1; }
      };
      if (ok) issue_s(nt > 1);
      // O is read to the end of the previous segment before it is begun anew
      if (sg > 0) ok &= wait_warp(&odone, (sg - 1) & 1, stop, a, 35);
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t w = j & 1;
        // S of the next pair while the groups work on this one
        if (w == 0 && j + 2 < nt) issue_s(j + 3 < nt);
        ok &= wait_warp(&pready[w], (p_ph >> w) & 1, stop, a, 36);
        p_ph ^= 1u << w;
        ok &= wait_warp(&vfull[vs], vph, stop, a, 37);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint64_t vd = vd0 + vs * (Z::kTileBytes >> 4);
          const uint32_t p = tm + kColP + w * kKeys, o = tm + kColO + w * DH;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk) {
            tc::mma_f16_ts(o, p + kk * 8, vd + kk * (2048 / 16), idO, j >= 2 || kk != 0);
            tc::mma_f16_ts(o, p + 32 + kk * 8, vd + kk * (2048 / 16), idO, 1);
          }
          tc::mma_commit(&vempty[vs]);
          tc::mma_commit(&pdone[w]);
        }
        __syncwarp();
        if (++vs == NV) { vs = 0; vph ^= 1; }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (tc::elect_one()) {
        tc::mma_commit(&qempty[sg & 1]);
        tc::mma_commit(&ofull);
      }
      __syncwarp();
      if (!ok) break;
      ++sg;
    }
    if (tc::elect_one()) {
      tc::mma_commit(&done);  // arrives once every MMA issued above has completed
      if (!tc::mbar_wait_soon(&done, 0, unwind_ns)) set_error(a.hdr, DV_ERR_TIMEOUT, 38);
    }
    __syncwarp();
  } else if (warp == 10) {  // query rows, then the rows of out that no unit writes
    constexpr int kRowChunks = DH / 8;
    int sg = 0;
    bool go = true;
    while (go && cur.next(L, plan, kTreeRows, &s)) {
      if (!s.ok) continue;
      if (sg >= 2) go = __all_sync(0xffffffffu, wait_warp(&qempty[sg & 1], ((sg >> 1) - 1) & 1, stop, a, 39));
      uint8_t* dst = sQ + (sg & 1) * Z::kQBytes;
      if (go) {
        for (int i = lane; i < s.rows * kRowChunks; i += 32) {
          const int r = i / kRowChunks, c = i % kRowChunks;
          cp_async16(dst + (c >> 3) * (kTreeRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                     static_cast<const T*>(L.q) + row_offset(L, s, r, DH) + c * 8);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      tc::fence_proxy_async();
      tc::mbar_arrive(&qfull[sg & 1]);
      ++sg;
    }
    __syncwarp();
    zero_rows<T, DH>(L, plan, blockIdx.x, gridDim.x, lane, 32);
  } else {  // softmax groups
    const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t tS = lanes + kColS + w * kKeys, tP = lanes + kColP + w * kKeys, tO = lanes + kColO + w * DH;
    int base = 0, sg = 0;
    uint32_t scount = 0, pcount = 0;   // pairs seen, tiles worked on
    bool any = false;
    while (cur.next(L, plan, kTreeRows, &s)) {
      any = true;
      if (!s.ok) {
        if (tid == 0) set_error(a.hdr, DV_ERR_INDEX_RANGE, s.head);
        continue;
      }
      const int nt = s.k1 - s.k0;
      const bool active = quad * 32 < s.rows;
      const int t = min(s.row0 + row, s.row0 + s.rows - 1) / L.g;
      float m = -INFINITY, l = 0.f;
      // what an edge tile needs besides its scores is made ready while the tile
      // before it is in the products
      bool there = true;
      const auto prepare = [&](int j) -> u64 {
        if (j >= nt || (s.k0 + j + 1) * kKeys <= s.pos) return ~0ull;
        const int it = base + j, st = it % NV;
        there &= wait_warp(&vfull[st], (it / NV) & 1, stop, a, 40);
        return prepare_edge<T, DH>(L, s.b, s.pos, s.nodes, sV + st * Z::kTileBytes, (s.k0 + j) * kKeys, t, active,
                                   &bad_v[sg & 3]);
      };
      u64 vis = prepare(w);
      for (int j = w; j - w < nt; j += 2) {
        there &= wait_warp(&sfull, scount & 1, stop, a, 41);
        ++scount;
        if (!__all_sync(0xffffffffu, there)) break;  // the whole warp, or none of it
        if (j >= nt) {  // a pair of one tile, the other group's
          tc::mbar_arrive(&sfree);
          break;
        }
        tc::fence_after_sync();
        if (active) {
          float v[kKeys];
          tc::tmem_ld32(tS, v);
          tc::tmem_ld32(tS + 32, v + 32);
          tc::tmem_ld_wait();
          tc::fence_before_sync();
          tc::mbar_arrive(&sfree);
          const float c = a.scale_log2;
          if (__any_sync(0xffffffffu, vis != ~0ull)) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i) v[i] = (vis >> i) & 1 ? v[i] : -INFINITY;
          }
          float mx[2] = {fmaxf(v[0], v[1]), fmaxf(v[2], v[3])};
#pragma unroll
          for (int i = 4; i < kKeys; i += 4) {
            mx[0] = max3(mx[0], v[i], v[i + 1]);
            mx[1] = max3(mx[1], v[i + 2], v[i + 3]);
          }
          const float top = fmaxf(mx[0], mx[1]) * c;
          // P and O of the group's tile before are read and written
          if (pcount) there &= wait_warp(&pdone[w], (pcount - 1) & 1, stop, a, 44);
          __syncwarp();
          tc::fence_after_sync();
          const bool move = row < s.rows && top > m + kSlack;
          if (__any_sync(0xffffffffu, move)) {
            // a row whose maximum was -inf has sums of 0: nothing to rescale
            const float alpha = move && m > -INFINITY ? ex2(m - top) : 1.f;
            if (move) m = top;
            l *= alpha;
            if (j >= 2 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int cc = 0; cc < DH; cc += 32) {
                float o[32];
                tc::tmem_ld32(tO + cc, o);
                tc::tmem_ld_wait();
                uint32_t r[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(o[i] * alpha);
                tc::tmem_st32(tO + cc, r);
              }
            }
          }
          const float off = kShift - (m == -INFINITY ? 0.f : m);
          u64 sum[2] = {0, 0};
          const u64 c2 = pack2(c, c), off2 = pack2(off, off), minus = pack2(-1.f, -1.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t hi[kKeys / 4], lo[kKeys / 4];
#pragma unroll
            for (int i = 0; i < kKeys / 2; i += 2) {
              float p0, p1;
              open2(fma2(pack2(v[half * 32 + i], v[half * 32 + i + 1]), c2, off2), &p0, &p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              const u64 p = pack2(p0, p1);
              sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], p);
              hi[i / 2] = Half2<T>::pack(p0, p1);
              const float2 h = Half2<T>::open(hi[i / 2]);
              float l0, l1;
              open2(fma2(pack2(h.x, h.y), minus, p), &l0, &l1);
              lo[i / 2] = Half2<T>::pack(l0, l1);
            }
            tc::tmem_st16(tP + half * 16, hi);
            tc::tmem_st16(tP + 32 + half * 16, lo);
          }
          float s0, s1;
          open2(add2(sum[0], sum[1]), &s0, &s1);
          l += s0 + s1;
          tc::tmem_st_wait();
        } else {
          // a warp without rows keeps step: it must not arrive for the next
          // tile while the others are still at this one
          tc::mbar_arrive(&sfree);
          if (pcount) wait_warp(&pdone[w], (pcount - 1) & 1, stop, a, 44);
        }
        ++pcount;
        tc::fence_before_sync();
        tc::mbar_arrive(&pready[w]);
        vis = prepare(j + 2);
      }
      // the segment's end: both groups' results joined, a group to each half of the columns
      sml[sg & 1][w][row] = make_float2(m, l);
      if (tid == 0) bad_v[(sg + 2) & 3] = 0;
      group_sync<256>();
      wait_warp(&ofull, sg & 1, stop, a, 42);
      tc::fence_after_sync();
      __syncwarp();
      const bool fix = bad_v[sg & 3] != 0;
      const float2 A = sml[sg & 1][0][row], Bv = sml[sg & 1][1][row];
      const float M = fmaxf(A.x, Bv.x);
      const float wA = A.x == -INFINITY ? 0.f : ex2(A.x - M), wB = Bv.x == -INFINITY ? 0.f : ex2(Bv.x - M);
      const float sum = fmaf(A.y, wA, Bv.y * wB);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;   // a row that sees nothing is zero
      const bool whole = nt == s.tiles;
      const size_t slot = piece_slot(blockIdx.x, s.k0 == 0);
#pragma unroll 1
      for (int cc = w * (DH / 2); cc < (w + 1) * (DH / 2); cc += 32) {
        if (!active) break;
        float o[32];
        {
          float ob[32];
          tc::tmem_ld32(lanes + kColO + cc, o);
          if (nt > 1) tc::tmem_ld32(lanes + kColO + DH + cc, ob);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            o[i] *= wA;
            if (nt > 1) o[i] = fmaf(ob[i], wB, o[i]);
          }
        }
        if (row < s.rows) {
          if (fix) {  // values that clean_v took out, for the rows that see them
            const int f0 = max(s.k0 * kKeys - s.pos, 0), f1 = min(s.k1 * kKeys - s.pos, s.nodes);
            for (int u = f0; u < f1; ++u) {
              if (!sees(L, s, t, u)) continue;
              const T* vr = static_cast<const T*>(L.V) +
                            (((size_t)s.b * L.h + s.head) * L.n_max + s.pos + u) * DH + cc;
  #pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = Elem<T>::to_f(vr[i]);
                if (!(fabsf(x) < INFINITY)) o[i] += x;
              }
            }
          }
          if (whole) {
            T* dst = static_cast<T*>(L.out) + row_offset(L, s, row, DH) + cc;
  #pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const uint4 x = make_uint4(Half2<T>::pack(o[i] * inv, o[i + 1] * inv),
                                         Half2<T>::pack(o[i + 2] * inv, o[i + 3] * inv),
                                         Half2<T>::pack(o[i + 4] * inv, o[i + 5] * inv),
                                         Half2<T>::pack(o[i + 6] * inv, o[i + 7] * inv));
              *reinterpret_cast<uint4*>(dst + i) = x;
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(L.part) + (slot * (DH / 4) + cc / 4) * L.rows_pad + row;
  #pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(dst + (size_t)(i / 4) * L.rows_pad, make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
            if (cc == 0) __stcg(&L.ml[slot * L.rows_pad + row], make_float2(M, sum));
          }
        }
        __syncwarp();
      }
      tc::fence_before_sync();
      tc::mbar_arrive(&odone);
      base += nt;
      ++sg;
    }
    if (tid == 0) cur.describe(s, any, static_cast<Shared*>(L.shared) + blockIdx.x);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 9) tc::tmem_dealloc(tmem, kTcTmemCols);
}

// ---- join ---------------------------------------------------------------------
//
// Block (c, part): the shared unit that begins in CTA c's share, kJoinThreads of its
// (row, four columns).

constexpr int kJoinThreads = 128;   // fits beside a CTA of the first kernel, to wait for its end there

template <typename T, int DH>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a) {
  const TreeLaunch& L = a.L;
  const int owner = blockIdx.x, i = blockIdx.y * kJoinThreads + threadIdx.x;
  grid_dep_launch();
  grid_dep_wait();
  const int4* d = reinterpret_cast<const int4*>(static_cast<const Shared*>(L.shared) + owner);
  const int4 d0 = __ldcg(d);
  const int pieces = __ldcg(d + 1).x;
  const Shared s{d0.x, d0.y, d0.z, d0.w, pieces, {0, 0, 0}};
  if (pieces < 2 || i >= s.rows * (DH / 4)) return;
  constexpr int kP = 4;  // pieces whose loads are in flight together
  {
    const int r = i % s.rows, c4 = i / s.rows;
    float M = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
    for (int q0 = 0; q0 < pieces; q0 += kP) {
      float2 ml[kP];
      float4 x[kP];
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q0 + q < pieces) {
          const size_t slot = piece_slot(owner + q0 + q, q0 + q == 0);
          ml[q] = __ldcg(&L.ml[slot * L.rows_pad + r]);
          x[q] = __ldcg(reinterpret_cast<const float4*>(L.part) + (slot * (DH / 4) + c4) * L.rows_pad + r);
        }
      }
      float m = M;
#pragma unroll
      for (int q = 0; q < kP; ++q) m = fmaxf(m, ml[q].x);
      const float keep = M == -INFINITY ? 1.f : ex2(M - m);   // (sums of 0, or a NaN, where M is -inf)
      M = m;
      l *= keep; o0 *= keep; o1 *= keep; o2 *= keep; o3 *= keep;
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const float w = ml[q].x == -INFINITY ? 1.f : ex2(ml[q].x - m);
        l = fmaf(ml[q].y, w, l);
        o0 = fmaf(x[q].x, w, o0); o1 = fmaf(x[q].y, w, o1);
        o2 = fmaf(x[q].z, w, o2); o3 = fmaf(x[q].w, w, o3);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees nothing is zero
    store4<T>(static_cast<T*>(L.out) + row_offset(L, s, r, DH) + 4 * c4, o0 * inv, o1 * inv, o2 * inv, o3 * inv);
  }
}

// ---- host ------------------------------------------------------------------------

template <typename T, int DH>
cudaError_t run_join(const TreeArgs& a, int ctas, int rows_per_unit, cudaStream_t stream) {
  const int items = min(rows_per_unit, a.L.T * a.L.g) * (DH / 4);
  return launch_k(tree_join_kernel<T, DH>, dim3(ctas, (items + kJoinThreads - 1) / kJoinThreads), dim3(kJoinThreads), 0,
                  stream, true, 1, a);
}

template <typename T, int DH>
cudaError_t run_tc(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  CUtensorMap mK, mV;
  const uint64_t mats = (uint64_t)a.L.B * a.L.h;
  if (!make_map_3d(&mK, a.L.K, DH, a.L.n_max, mats, kKeys, bf16) ||
      !make_map_3d(&mV, a.L.V, DH, a.L.n_max, mats, kKeys, bf16))
    return cudaErrorInvalidValue;
  constexpr size_t smem = TcSizes<DH>::kSmem;
  static PerDevice attr;  // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(tree_tc_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (ea != cudaSuccess) return ea;
  const int ctas = min(num_sms, kTreeCtas);
  const cudaError_t e = launch_k(tree_tc_kernel<T, DH>, dim3(ctas), dim3(kTcThreads), smem, stream, true, 1, mK, mV, a);
  return e == cudaSuccess ? run_join<T, DH>(a, ctas, kTreeRows, stream) : e;
}

template <int DH>
cudaError_t run_simt(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr size_t smem = sizeof(SimtSmem<DH>);
  static PerDevice attr;  // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(tree_simt_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (ea != cudaSuccess) return ea;
  const int ctas = min(num_sms, kTreeCtas);
  const cudaError_t e = launch_k(tree_simt_kernel<DH>, dim3(ctas), dim3(kSimtThreads), smem, stream, true, 1, a);
  return e == cudaSuccess ? run_join<float, DH>(a, ctas, kSimtRows, stream) : e;
}

}  // namespace

cudaError_t launch_tree_attn(const TreeLaunch& L, dv_dtype dt, WsHeader* hdr, int num_sms, cudaStream_t stream) {
  const TreeArgs a{L, L.scale * kLog2e, hdr, wait_limit_ns()};
  const bool wide = L.d_h == 128;
  switch (dt) {
    case DV_F32: return wide ? run_simt<128>(a, num_sms, stream) : run_simt<64>(a, num_sms, stream);
    case DV_F16: return wide ? run_tc<__half, 128>(a, num_sms, stream) : run_tc<__half, 64>(a, num_sms, stream);
    case DV_BF16:
      return wide ? run_tc<__nv_bfloat16, 128>(a, num_sms, stream) : run_tc<__nv_bfloat16, 64>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dv
