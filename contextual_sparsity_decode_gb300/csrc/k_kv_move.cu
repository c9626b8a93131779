// Moving rows of the KV cache in place: K, V, the token embeddings X and the
// valid flags of a cache position go together.
//
//   compact  the accepted nodes of a drafted tree, slots idx[0] < idx[1] < ...
//            behind the committed positions, become positions pos, pos + 1, ...
//            dst(k) = pos + k <= src(k) = pos + idx[k] < src(k + 1), so a
//            thread that walks k upwards never overwrites a row that it (or
//            any other thread: a thread keeps its 16-byte column) still reads.
//   reorder  beam w of a sequence continues beam parent[w]: positions
//            [start, pos of the parent) of row w become those of row
//            parent[w].  The same parent may be taken several times and the
//            rows may form cycles; a thread holds its 16-byte column of every
//            beam that is read in registers before it writes any, so no second
//            cache is needed.
//
// A (head, position) whose valid flag is 0 has no K/V: only its flag moves
// (a sequence that keeps 20 % of the heads then moves a fifth of the K/V).
// Both kernels are bounded by memory: every moved row is read once and
// written once, with 16-byte accesses, each thread's loads all issued before
// its first store.

#include "dv_kernels.h"

namespace dv {
namespace {

constexpr int kMoveThreads = 256;

__device__ __forceinline__ uint4 ld16(const void* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void st16(void* p, const uint4& v) { __stcg(reinterpret_cast<uint4*>(p), v); }

// Advances pos once every CTA has read it: the last CTA to finish writes
// new_pos (which may be pos itself).
__device__ __forceinline__ bool last_cta(int* ctr, int total) {
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ctr, 1) == total - 1;
    if (last) *ctr = 0;
  }
  __syncthreads();
  return last != 0;
}

struct CompactArgs {
  KvPtrs kv[kKvLayers];
  int B, h, n_max, kv_chunks, x_chunks;  // 16-byte chunks of a K/V row and of an X row
  const int32_t* pos;
  const int32_t* idx;
  int cap;
  const int32_t* count;
  int32_t* new_pos;  // null in all but the last launch of a call
  WsHeader* hdr;
};

// Number of accepted nodes of sequence b, or -1 when its list is refused.
__device__ int compact_count(const CompactArgs& a, int b, int* pos_out, bool report) {
  int n = a.count[b];
  if (n > a.cap) {
    if (report) set_error(a.hdr, DV_ERR_CAPACITY, n);
    n = a.cap;
  }
  const int p = a.pos[b];
  *pos_out = p;
  if (n <= 0) return 0;
  if (p < 0 || p >= a.n_max) {
    if (report) set_error(a.hdr, DV_ERR_POSITION, p);
    return -1;
  }
  int prev = -1;
  for (int k = 0; k < n; ++k) {
    const int u = a.idx[(size_t)b * a.cap + k];
    if (u <= prev) {
      if (report) set_error(a.hdr, DV_ERR_INDEX_RANGE, u);
      return -1;
    }
    if (u >= a.n_max - p) {
      if (report) set_error(a.hdr, DV_ERR_POSITION, p);
      return -1;
    }
    prev = u;
  }
  return n;
}

// grid (part, b, layer): part 0..h-1 a head's K and V rows, part h the X rows
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const __grid_constant__ CompactArgs a) {
  const int part = blockIdx.x, b = blockIdx.y, layer = blockIdx.z;
  int p;
  const int n = compact_count(a, b, &p, part == 0 && layer == 0 && threadIdx.x == 0);
  const KvPtrs& kv = a.kv[layer];
  const int32_t* idx = a.idx + (size_t)b * a.cap;
  if (n > 0) {
    if (part < a.h) {
      uint8_t* flags = kv.valid + ((size_t)b * a.h + part) * a.n_max + p;
      char* rows[2] = {kv.K, kv.V};
      const size_t pitch = (size_t)a.kv_chunks * 16;
      const size_t base = (((size_t)b * a.h + part) * a.n_max + p) * pitch;
      for (int c = threadIdx.x; c < 2 * a.kv_chunks; c += blockDim.x) {
        char* row = rows[c >= a.kv_chunks] + base + (size_t)(c % a.kv_chunks) * 16;
        for (int k = 0; k < n; ++k) {
          const int u = idx[k];
          if (u != k && flags[u]) st16(row + k * pitch, ld16(row + u * pitch));
        }
      }
      __syncthreads();
      if (threadIdx.x == 0)
        for (int k = 0; k < n; ++k) flags[k] = flags[idx[k]];
    } else {
      const size_t pitch = (size_t)a.x_chunks * 16;
      char* base = kv.X + ((size_t)b * a.n_max + p) * pitch;
      for (int c = threadIdx.x; c < a.x_chunks; c += blockDim.x)
        for (int k = 0; k < n; ++k)
          if (idx[k] != k) st16(base + k * pitch + (size_t)c * 16, ld16(base + idx[k] * pitch + (size_t)c * 16));
    }
  }
  if (a.new_pos) {
    if (last_cta(&a.hdr->pad[0], gridDim.x * gridDim.y * gridDim.z)) {
      for (int s = threadIdx.x; s < a.B; s += blockDim.x) {
        int q;
        const int m = compact_count(a, s, &q, false);
        a.new_pos[s] = q + max(m, 0);
      }
    }
  }
}

struct ReorderArgs {
  KvPtrs kv[kKvLayers];
  int S, W, h, n_max, kv_chunks, x_chunks;
  const int32_t* pos;
  const int32_t* start;
  const int32_t* parent;
  WsHeader* hdr;
};

// grid (part, position block, layer * S + s)
template <int WM>
__global__ void __launch_bounds__(kMoveThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int par[WM], hi[WM];
  __shared__ int lo_s;
  const int part = blockIdx.x, s = blockIdx.z % a.S, layer = blockIdx.z / a.S;
  const KvPtrs& kv = a.kv[layer];
  if (threadIdx.x < WM) {
    const int w = threadIdx.x;
    int p = w, top = 0;
    if (w < a.W) {
      p = a.parent[s * a.W + w];
      if (p < 0 || p >= a.W) {
        if (part == 0 && layer == 0 && blockIdx.y == 0) set_error(a.hdr, DV_ERR_INDEX_RANGE, p);
        p = w;
      }
      top = a.pos[s * a.W + p];
      if (top < 0 || top > a.n_max) {
        if (part == 0 && layer == 0 && blockIdx.y == 0) set_error(a.hdr, DV_ERR_POSITION, top);
        top = 0;
      }
    }
    par[w] = p;
    hi[w] = p == w ? 0 : top;   // a beam that continues itself stays as it is
    if (w == 0) lo_s = a.start ? max(a.start[s], 0) : 0;
  }
  __syncthreads();
  int top = 0;
  for (int w = 0; w < a.W; ++w) top = max(top, hi[w]);
  const bool is_x = part == a.h;
  const int chunks = is_x ? a.x_chunks : a.kv_chunks;
  const size_t pitch = (size_t)chunks * 16;
  const int tensors = is_x ? 1 : 2;
  const size_t row0 = (size_t)s * a.W;
  const size_t beam_rows = is_x ? a.n_max : (size_t)a.h * a.n_max;       // rows between two beams
  const size_t first = is_x ? row0 * a.n_max : (row0 * a.h + part) * a.n_max;
  const uint8_t* flags = kv.valid + (row0 * a.h + (is_x ? 0 : part)) * a.n_max;
  const int per = kMoveThreads / chunks > 0 ? kMoveThreads / chunks : 1;  // positions a block handles at once
  const int lanes = chunks < kMoveThreads ? chunks : kMoveThreads;
  const int sub = threadIdx.x / lanes, c0 = threadIdx.x % lanes;
  for (int j = lo_s + blockIdx.y * per + sub; j < top && sub < per; j += gridDim.y * per) {
    for (int t = 0; t < tensors; ++t) {
      char* base = (is_x ? kv.X : t ? kv.V : kv.K) + (first + j) * pitch;
      for (int c = c0; c < chunks; c += lanes) {
        uint4 v[WM];
        bool take[WM];
#pragma unroll
        for (int w = 0; w < WM; ++w) {
          const int p = par[w];
          take[w] = j < hi[w] && (is_x || flags[(size_t)p * a.h * a.n_max + j]);
          if (take[w]) v[w] = ld16(base + p * beam_rows * pitch + (size_t)c * 16);
        }
#pragma unroll
        for (int w = 0; w < WM; ++w)
          if (take[w]) st16(base + w * beam_rows * pitch + (size_t)c * 16, v[w]);
      }
    }
  }
}

// the flags move after the rows that they describe
template <int WM>
__global__ void __launch_bounds__(kMoveThreads) reorder_flags_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int par[WM], hi[WM];
  const int i = blockIdx.x, s = blockIdx.y, layer = blockIdx.z;
  if (threadIdx.x < WM) {
    const int w = threadIdx.x;
    int p = w, top = 0;
    if (w < a.W) {
      p = a.parent[s * a.W + w];
      if (p < 0 || p >= a.W) p = w;
      top = a.pos[s * a.W + p];
      if (top < 0 || top > a.n_max) top = 0;
    }
    par[w] = p;
    hi[w] = p == w ? 0 : top;
  }
  __syncthreads();
  int top = 0;
  for (int w = 0; w < a.W; ++w) top = max(top, hi[w]);
  const int lo = a.start ? max(a.start[s], 0) : 0;
  const size_t beam = (size_t)a.h * a.n_max;
  uint8_t* flags = a.kv[layer].valid + ((size_t)s * a.W * a.h + i) * a.n_max;
  for (int j = lo + threadIdx.x; j < top; j += blockDim.x) {
    uint8_t f[WM];
#pragma unroll
    for (int w = 0; w < WM; ++w) f[w] = j < hi[w] ? flags[par[w] * beam + j] : 0;
#pragma unroll
    for (int w = 0; w < WM; ++w)
      if (j < hi[w]) flags[w * beam + j] = f[w];
  }
}

template <int WM>
cudaError_t run_reorder(const ReorderArgs& a, int n_kv, cudaStream_t stream) {
  const int blocks = max(1, min(64, a.n_max / 16));
  reorder_kernel<WM><<<dim3(a.h + 1, blocks, n_kv * a.S), kMoveThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  reorder_flags_kernel<WM><<<dim3(a.h, a.S, n_kv), kMoveThreads, 0, stream>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(2);
  return e;
}

}  // namespace

cudaError_t launch_kv_compact(const KvMove& m, const int32_t* idx, int cap, const int32_t* count, int32_t* new_pos,
                              WsHeader* hdr, cudaStream_t stream) {
  for (int l0 = 0; l0 < m.n_kv; l0 += kKvLayers) {
    const int n = min(kKvLayers, m.n_kv - l0);
    CompactArgs a{};
    for (int l = 0; l < n; ++l) a.kv[l] = m.kv_at(l0 + l);
    a.B = m.B; a.h = m.h; a.n_max = m.n_max; a.kv_chunks = m.kv_chunks; a.x_chunks = m.x_chunks;
    a.pos = m.pos; a.idx = idx; a.cap = cap; a.count = count; a.hdr = hdr;
    a.new_pos = l0 + n == m.n_kv ? new_pos : nullptr;
    compact_kernel<<<dim3(m.h + 1, m.B, n), kMoveThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaSuccess;
}

cudaError_t launch_kv_reorder(const KvMove& m, int width, const int32_t* start, const int32_t* parent, WsHeader* hdr,
                              cudaStream_t stream) {
  for (int l0 = 0; l0 < m.n_kv; l0 += kKvLayers) {
    const int n = min(kKvLayers, m.n_kv - l0);
    ReorderArgs a{};
    for (int l = 0; l < n; ++l) a.kv[l] = m.kv_at(l0 + l);
    a.S = m.B / width; a.W = width; a.h = m.h; a.n_max = m.n_max;
    a.kv_chunks = m.kv_chunks; a.x_chunks = m.x_chunks;
    a.pos = m.pos; a.start = start; a.parent = parent; a.hdr = hdr;
    const cudaError_t e = width <= 4    ? run_reorder<4>(a, n, stream)
                          : width <= 8  ? run_reorder<8>(a, n, stream)
                          : width <= 16 ? run_reorder<16>(a, n, stream)
                                        : run_reorder<32>(a, n, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dv
