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
// numerator) per CTA, and the last CTA to finish joins them in tile order, so
// results do not depend on timing.

#include <type_traits>

#include "dv_kernels.h"

namespace dv {
namespace {

constexpr int kKeys = 64;      // keys per tile
constexpr float kLog2e = 1.4426950408889634f;

struct TreeArgs {
  TreeLaunch L;
  float scale_log2;            // scale log2(e): exponentials are taken to base 2
  WsHeader* hdr;
};

// What every role of a CTA needs to walk its share of the tiles.
struct TreePlan {
  long long pre[kTreeMaxB + 1];  // tiles of the sequences before b
  int pos[kTreeMaxB], nodes[kTreeMaxB];
};

struct Seg {
  int b, head, row0, rows;       // rows row0 .. row0 + rows - 1 of the sequence's T g
  int pos, nodes, n;             // committed positions, tree nodes, their sum
  int k0, k1, tiles;             // tiles [k0, k1) of the unit's `tiles`
  int owner, pieces;             // CTA of the unit's first tile, CTAs that share it
  bool ok;                       // the head index is in range
};

// One block-wide pass over the sequences: checks, lengths and the prefix sums
// of their tiles.  NT threads; ends with a barrier.
template <int NT>
__device__ void tree_plan(const TreeArgs& a, TreePlan* p, int rows_per_unit) {
  __shared__ long long warp_tot[NT / 32];
  const TreeLaunch& L = a.L;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  long long carry = 0;
  for (int b0 = 0; b0 < L.B; b0 += NT) {
    const int b = b0 + tid;
    long long work = 0;
    if (b < L.B) {
      const int n = L.pos[b];
      int nd = L.nodes ? L.nodes[b] : L.T;
      int cnt = L.head_idx ? L.head_count[b] : L.h;
      const bool report = blockIdx.x == 0;
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
      if (nd > 0 && cnt > 0)
        work = (long long)cnt * ((nd * L.g + rows_per_unit - 1) / rows_per_unit) * ((n + nd + kKeys - 1) / kKeys);
      p->pos[b] = n;
      p->nodes[b] = nd;
    }
    long long v = work;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_tot[wid] = v;
    __syncthreads();
    long long before = carry;
    for (int q = 0; q < wid; ++q) before += warp_tot[q];
    if (b < L.B) p->pre[b + 1] = before + v;
    long long all = carry;
    for (int q = 0; q < NT / 32; ++q) all += warp_tot[q];
    carry = all;
    __syncthreads();
  }
  if (tid == 0) p->pre[0] = 0;
  __syncthreads();
}

// Walks the segments of this CTA's share of the tiles.
struct Cursor {
  long long t, t1, W;
  int G, b;
  __device__ Cursor(const TreePlan& p, int B) {
    W = p.pre[B];
    G = (int)(W < (long long)gridDim.x ? W : (long long)gridDim.x);
    const int c = blockIdx.x;
    t = c < G ? W * c / G : 0;
    t1 = c < G ? W * (c + 1) / G : 0;
    int lo = 0, hi = B;  // the last b with pre[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.pre[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  __device__ bool next(const TreeLaunch& L, const TreePlan& p, int rows_per_unit, Seg* s) {
    if (t >= t1) return false;
    while (p.pre[b + 1] <= t) ++b;
    s->b = b;
    s->pos = p.pos[b];
    s->nodes = p.nodes[b];
    s->n = s->pos + s->nodes;
    const int all_rows = s->nodes * L.g;
    const int blocks = (all_rows + rows_per_unit - 1) / rows_per_unit;
    s->tiles = (s->n + kKeys - 1) / kKeys;
    const long long off = t - p.pre[b];
    const long long unit = off / s->tiles;
    s->k0 = (int)(off - unit * s->tiles);
    s->k1 = (int)min((long long)s->tiles, s->k0 + (t1 - t));
    const int slot = (int)(unit / blocks);
    s->row0 = (int)(unit - (long long)slot * blocks) * rows_per_unit;
    s->rows = min(rows_per_unit, all_rows - s->row0);
    s->head = L.head_idx ? L.head_idx[(size_t)b * L.cap + slot] : slot;
    s->ok = s->head >= 0 && s->head < L.h;
    const long long u0 = t - s->k0, u1 = u0 + s->tiles - 1;
    s->owner = (int)(((u0 + 1) * G - 1) / W);
    s->pieces = (int)(((u1 + 1) * G - 1) / W) - s->owner + 1;
    t += s->k1 - s->k0;
    return true;
  }
};

// Query row r of unit (b, head): its offset in q and out.
__device__ __forceinline__ size_t row_offset(const TreeLaunch& L, const Seg& s, int r, int d_h) {
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

// Joins the partial results of a unit, in tile order, and writes its rows.
// Called by NT threads of the CTA that finished last.
template <typename T, int DH, int NT>
__device__ void join_unit(const TreeLaunch& L, const Seg& s, int tid) {
  for (int i = tid; i < s.rows * (DH / 4); i += NT) {
    const int r = i % s.rows, c4 = i / s.rows;
    float M = -INFINITY;
    for (int q = 0; q < s.pieces; ++q)
      M = fmaxf(M, __ldcg(&L.ml[piece_slot(s.owner + q, q == 0) * L.rows_pad + r].x));
    float l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
    for (int q = 0; q < s.pieces; ++q) {
      const size_t slot = piece_slot(s.owner + q, q == 0);
      const float2 ml = __ldcg(&L.ml[slot * L.rows_pad + r]);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(L.part) + (slot * (DH / 4) + c4) * L.rows_pad + r);
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      l = fmaf(ml.y, w, l);
      o0 = fmaf(o.x, w, o0); o1 = fmaf(o.y, w, o1);
      o2 = fmaf(o.z, w, o2); o3 = fmaf(o.w, w, o3);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees nothing is zero
    store4<T>(static_cast<T*>(L.out) + row_offset(L, s, r, DH) + 4 * c4, o0 * inv, o1 * inv, o2 * inv, o3 * inv);
  }
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

// ---- CUDA cores ---------------------------------------------------------------

constexpr int kSimtRows = 16;
constexpr int kSimtThreads = 256;

template <int DH>
struct SimtSmem {
  TreePlan plan;
  alignas(16) float q[kSimtRows][DH];
  alignas(16) float k[kKeys][DH + 4];
  alignas(16) float v[kKeys][DH];
  float s[kSimtRows][kKeys + 1];   // scores, then p; -1 marks a masked key
  float alpha[kSimtRows];
  float m[kSimtRows], l[kSimtRows];
  int last;
};

template <typename T, int DH>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<DH>& sm = *reinterpret_cast<SimtSmem<DH>*>(smem_raw);
  const TreeLaunch& L = a.L;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  constexpr int kVec = Elem<T>::kVec, kChunks = DH / kVec;
  constexpr int kCols = DH / 16;   // output columns of a thread
  tree_plan<kSimtThreads>(a, &sm.plan, kSimtRows);
  zero_rows<T, DH>(L, sm.plan, blockIdx.x * (kSimtThreads / 32) + wid, gridDim.x * (kSimtThreads / 32), lane, 32);
  Cursor cur(sm.plan, L.B);
  Seg s;
  while (cur.next(L, sm.plan, kSimtRows, &s)) {
    if (!s.ok) {
      if (tid == 0) set_error(a.hdr, DV_ERR_INDEX_RANGE, s.head);
      continue;
    }
    __syncthreads();
    for (int i = tid; i < kSimtRows * kChunks; i += kSimtThreads) {
      const int r = i / kChunks, c = i % kChunks;
      float f[kVec];
      if (r < s.rows) {
        unpack<T>(ld_cached(static_cast<const T*>(L.q) + row_offset(L, s, r, DH) + c * kVec), f);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) f[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) sm.q[r][c * kVec + e] = f[e];
    }
    if (tid < kSimtRows) {
      sm.m[tid] = -INFINITY;
      sm.l[tid] = 0.f;
    }
    float acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
    const size_t kv0 = ((size_t)s.b * L.h + s.head) * L.n_max * DH;
    for (int kt = s.k0; kt < s.k1; ++kt) {
      const int j0 = kt * kKeys, nk = min(kKeys, s.n - j0);
      __syncthreads();   // the previous tile is no longer read
      for (int i = tid; i < kKeys * kChunks; i += kSimtThreads) {
        const int j = i / kChunks, c = i % kChunks;
        float fk[kVec], fv[kVec];
        if (j < nk) {
          unpack<T>(ld_stream(static_cast<const T*>(L.K) + kv0 + (size_t)(j0 + j) * DH + c * kVec), fk);
          unpack<T>(ld_stream(static_cast<const T*>(L.V) + kv0 + (size_t)(j0 + j) * DH + c * kVec), fv);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) fk[e] = fv[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          sm.k[j][c * kVec + e] = fk[e];
          sm.v[j][c * kVec + e] = fv[e];
        }
      }
      __syncthreads();
      {  // scores: thread = one key, four rows
        const int j = tid & (kKeys - 1), r0 = (tid / kKeys) * 4;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int c = 0; c < DH; c += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[j][c]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[r0 + r][c]);
            d[r] = fmaf(q4.x, k4.x, d[r]); d[r] = fmaf(q4.y, k4.y, d[r]);
            d[r] = fmaf(q4.z, k4.z, d[r]); d[r] = fmaf(q4.w, k4.w, d[r]);
          }
        }
        const int u = j0 + j - s.pos;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool vis = r0 + r < s.rows && j < nk && (u < 0 || sees(L, s, (s.row0 + r0 + r) / L.g, u));
          sm.s[r0 + r][j] = vis ? d[r] * a.scale_log2 : -INFINITY;
        }
      }
      __syncthreads();
#pragma unroll
      for (int rr = 0; rr < kSimtRows / 8; ++rr) {  // softmax: a warp takes two rows, a lane two keys
        const int r = wid * (kSimtRows / 8) + rr;
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
      {  // numerators: thread = one row, kCols columns
        const int r = tid / 16, c0 = (tid % 16) * 4;
        const float al = sm.alpha[r];
        const int t = (s.row0 + r) / L.g;
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] *= al;
        for (int j = 0; j < nk; ++j) {
          const float p = sm.s[r][j];
          // 0 x inf: a masked V row must not reach the sum, whatever it holds
          if (p == 0.f && (r >= s.rows || (j0 + j >= s.pos && !sees(L, s, t, j0 + j - s.pos)))) continue;
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float4 v4 = *reinterpret_cast<const float4*>(&sm.v[j][c0 + c * 16]);
            acc[c] = fmaf(p, v4.x, acc[c]); acc[c + 1] = fmaf(p, v4.y, acc[c + 1]);
            acc[c + 2] = fmaf(p, v4.z, acc[c + 2]); acc[c + 3] = fmaf(p, v4.w, acc[c + 3]);
          }
        }
      }
    }
    const int r = tid / 16, c0 = (tid % 16) * 4;
    if (s.pieces == 1) {
      if (r < s.rows) {
        const float l = sm.l[r], inv = l == 0.f ? 0.f : 1.f / l;
        T* dst = static_cast<T*>(L.out) + row_offset(L, s, r, DH) + c0;
#pragma unroll
        for (int c = 0; c < kCols; c += 4)
          store4<T>(dst + c * 16, acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv);
      }
      continue;
    }
    const size_t slot = piece_slot(blockIdx.x, s.k0 == 0);
    if (r < s.rows) {
      float4* dst = reinterpret_cast<float4*>(L.part) + slot * (DH / 4) * L.rows_pad + r;
#pragma unroll
      for (int c = 0; c < kCols; c += 4)
        __stcg(dst + (size_t)((c0 + c * 16) / 4) * L.rows_pad, make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]));
      if (c0 == 0) __stcg(&L.ml[slot * L.rows_pad + r], make_float2(sm.m[r], sm.l[r]));
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      sm.last = atomicAdd(&L.ctr[s.owner], 1) == s.pieces - 1;
      if (sm.last) L.ctr[s.owner] = 0;
      __threadfence();
    }
    __syncthreads();
    if (sm.last) join_unit<T, DH, kSimtThreads>(L, s, tid);
  }
}

// ---- host ------------------------------------------------------------------------

template <typename T, int DH>
cudaError_t run_simt(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr size_t smem = sizeof(SimtSmem<DH>);
  static PerDevice attr;  // function attributes are per device
  const cudaError_t ea = (cudaError_t)attr.get(current_device(), [] {
    return (int)cudaFuncSetAttribute(tree_simt_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (ea != cudaSuccess) return ea;
  return launch_k(tree_simt_kernel<T, DH>, dim3(min(num_sms, kTreeCtas)), dim3(kSimtThreads), smem, stream, false, 1, a);
}

template <typename T>
cudaError_t run_t(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  return a.L.d_h == 128 ? run_simt<T, 128>(a, num_sms, stream) : run_simt<T, 64>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_tree_attn(const TreeLaunch& L, dv_dtype dt, WsHeader* hdr, int num_sms, cudaStream_t stream) {
  TreeArgs a{L, L.scale * kLog2e, hdr};
  switch (dt) {
    case DV_F32: return run_t<float>(a, num_sms, stream);
    case DV_F16: return run_t<__half>(a, num_sms, stream);
    case DV_BF16: return run_t<__nv_bfloat16>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dv
