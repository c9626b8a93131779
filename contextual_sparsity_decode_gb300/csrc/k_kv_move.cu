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
// its first store.  Measured on GB300: eight layers of 32 sequences, 1 to 12
// rows each, 92 MB read and written: 27 us, 3.4 TB/s (waits for loads); three
// layers of 4 x 8 beams, 2.06 GB: 370 us, 5.6 TB/s, 0.82 of a plain copy's rate.

#include "dv_kernels.h"

namespace dv {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;

__device__ __forceinline__ uint4 ld16(const void* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void st16(void* p, const uint4& v) { __stcg(reinterpret_cast<uint4*>(p), v); }

// ---- compact ------------------------------------------------------------------
//
// A warp to a head's K, V and flags, or to 512 bytes of the X rows, of one
// sequence and layer: eight rows at a time, their loads issued together.  What
// bounds it is the chain of small reads (count and position, list, flags, rows,
// stores: each a round trip), so all layers go in one launch and the rest is
// left to the number of warps.

constexpr int kRowsAtOnce = 8;

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

// Accepted nodes of sequence b and its position, found by one warp; -1: the
// list is refused.
__device__ int compact_count(const CompactArgs& a, int b, int lane, bool report, int* pos_out) {
  // three reads at once: the list's first entries do not wait for its length
  const int32_t* idx = a.idx + (size_t)b * a.cap;
  const int u0 = lane < a.cap ? idx[lane] : 0;
  int n = a.count[b];
  const int p = a.pos[b];
  *pos_out = p;
  if (n > a.cap) {
    if (report && lane == 0) set_error(a.hdr, DV_ERR_CAPACITY, n);
    n = a.cap;
  }
  if (n <= 0) return 0;
  const bool outside = p < 0 || p >= a.n_max;
  int bad = 0, what = 0, before = -1;
  for (int k0 = 0; k0 < n && !outside && !bad; k0 += 32) {
    const int k = k0 + lane;
    const int u = k0 == 0 ? u0 : k < n ? idx[k] : 0;
    int prev = __shfl_up_sync(0xffffffffu, u, 1);
    if (lane == 0) prev = before;
    const int mine = k >= n ? 0 : u <= prev ? DV_ERR_INDEX_RANGE : u >= a.n_max - p ? DV_ERR_POSITION : 0;
    const uint32_t ball = __ballot_sync(0xffffffffu, mine != 0);
    if (ball) {
      const int src = __ffs(ball) - 1;
      bad = __shfl_sync(0xffffffffu, mine, src);
      what = __shfl_sync(0xffffffffu, u, src);
    }
    before = __shfl_sync(0xffffffffu, u, 31);
  }
  if (outside) bad = DV_ERR_POSITION;
  if (bad && report && lane == 0) set_error(a.hdr, bad, bad == DV_ERR_POSITION ? p : what);
  return bad ? -1 : n;
}

// grid (groups of eight warp items, b, layer)
__global__ void __launch_bounds__(kMoveThreads, 4) compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int last;
  const int b = blockIdx.y, layer = blockIdx.z;
  const int lane = threadIdx.x & 31, item = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  const bool first = blockIdx.x == 0 && layer == 0 && threadIdx.x < 32;
  int p;
  const int n = compact_count(a, b, lane, first, &p);
  const KvPtrs& kv = a.kv[layer];
  const int32_t* idx = a.idx + (size_t)b * a.cap;
  const bool head = item < a.h;
  const int x0 = (item - a.h) * 32;                       // first chunk of an X item
  const int items = head ? 2 * a.kv_chunks : min(32, a.x_chunks - x0);
  const size_t pitch = (size_t)(head ? a.kv_chunks : a.x_chunks) * 16;
  const size_t row0 = head ? ((size_t)b * a.h + item) * a.n_max + p : (size_t)b * a.n_max + p;
  uint8_t* flags = head ? kv.valid + row0 : nullptr;
  for (int k0 = 0; k0 < n && items > 0; k0 += kRowsAtOnce) {
    // lane k: slot and flag of row k0 + k
    const bool live = lane < kRowsAtOnce && k0 + lane < n;
    const int my_u = live ? idx[k0 + lane] : 0;
    const uint8_t flag = live && head ? flags[my_u] : 0;
    const uint32_t move = __ballot_sync(0xffffffffu, live && my_u != k0 + lane && (!head || flag));
    for (int c = lane; c - lane < items; c += 32) {
      char* col = nullptr;
      if (c < items)
        col = head ? (c < a.kv_chunks ? kv.K + c * 16 : kv.V + (c - a.kv_chunks) * 16) + row0 * pitch
                   : kv.X + row0 * pitch + (size_t)(x0 + c) * 16;
      uint4 v[kRowsAtOnce];
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k) {
        const int u = __shfl_sync(0xffffffffu, my_u, k);
        if (((move >> k) & 1) && col) v[k] = ld16(col + u * pitch);
      }
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k)
        if (((move >> k) & 1) && col) st16(col + (k0 + k) * pitch, v[k]);
    }
    if (live && head) flags[k0 + lane] = flag;
    __syncwarp();
  }
  if (!a.new_pos) return;
  if (a.new_pos != a.pos) {
    if (first && lane == 0) a.new_pos[b] = p + max(n, 0);
    return;
  }
  // in place: once every CTA has read pos, the last one advances it
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(&a.hdr->pad[0], 1) == (int)(gridDim.x * gridDim.y * gridDim.z) - 1;
    if (last) a.hdr->pad[0] = 0;
  }
  __syncthreads();
  if (!last) return;
  for (int s = threadIdx.x >> 5; s < a.B; s += kMoveWarps) {
    int q;
    const int m = compact_count(a, s, lane, false, &q);
    if (lane == 0) a.new_pos[s] = q + max(m, 0);
  }
}

// ---- reorder ------------------------------------------------------------------
//
// A CTA takes 128 positions of one head's K, V and flags, or of 512 bytes of the
// X rows, of one sequence and layer.  Every parent that is taken is read once
// and written to each of the beams that continue it.

constexpr int kSpan = 128;     // positions of a CTA, at most

struct ReorderArgs {
  KvPtrs kv[kKvLayers];
  int S, W, h, n_max, kv_chunks, x_chunks;
  int span;                      // positions of a CTA
  const int32_t* pos;
  const int32_t* start;
  const int32_t* parent;
  WsHeader* hdr;
};

// grid (heads and X parts, position blocks, layer * S + s)
template <int WM>
__global__ void __launch_bounds__(kMoveThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ uint32_t heirs[WM];   // the beams that continue beam p, itself apart
  __shared__ int upto[WM];         // positions held by beam p, 0 where it has no heirs
  __shared__ uint32_t there[kSpan];  // bit p: beam p's K/V at the position are present (and wanted)
  const int part = blockIdx.x, s = blockIdx.z % a.S, layer = blockIdx.z / a.S;
  const KvPtrs& kv = a.kv[layer];
  const bool is_x = part >= a.h;
  const size_t row0 = (size_t)s * a.W, flag_beam = (size_t)a.h * a.n_max;
  const size_t first = is_x ? row0 * a.n_max : (row0 * a.h + part) * a.n_max;
  uint8_t* flags = is_x ? nullptr : kv.valid + first;
  const int lo = a.start ? min(max(a.start[s], 0), a.n_max) : 0;
  const bool report = part == 0 && layer == 0 && blockIdx.y == 0;   // this CTA's sequence, once, whatever moves
  const int j0 = lo + blockIdx.y * a.span;
  if (j0 >= a.n_max && !report) return;
  if (threadIdx.x >= 128 && threadIdx.x < 128 + a.span) {  // the flags do not wait for the parents
    const int j = j0 + threadIdx.x - 128;
    uint32_t m = is_x ? ~0u : 0u;
    if (!is_x && j < a.n_max) {
#pragma unroll
      for (int p = 0; p < WM; ++p)
        if (p < a.W && flags[p * flag_beam + j]) m |= 1u << p;
    }
    there[threadIdx.x - 128] = m;
  }
  if (threadIdx.x < 32) {
    const int w = threadIdx.x;
    int p = w;
    if (w < a.W) {
      int top = a.pos[s * a.W + w];
      p = a.parent[s * a.W + w];
      if (p < 0 || p >= a.W) {
        if (report) set_error(a.hdr, DV_ERR_INDEX_RANGE, p);
        p = w;
      }
      if (top < 0 || top > a.n_max) top = -1;  // an error only where another beam continues this one
      if (w < WM) upto[w] = top;
    }
    uint32_t mine = 0;
    for (int q = 0; q < a.W; ++q) {
      const int pq = __shfl_sync(0xffffffffu, p, q);
      if (pq == w && q != w) mine |= 1u << q;
    }
    if (w < a.W) {
      if (mine && upto[w] < 0 && report) set_error(a.hdr, DV_ERR_POSITION, a.pos[s * a.W + w]);
      heirs[w] = mine;
      if (!mine || upto[w] < 0) upto[w] = 0;
    } else if (w < WM) {
      heirs[w] = 0;
      upto[w] = 0;
    }
  }
  __syncthreads();
  int top = 0;
#pragma unroll
  for (int p = 0; p < WM; ++p) top = max(top, upto[p]);
  const int j1 = min(j0 + a.span, top);
  if (j0 >= j1) return;
  const int c_first = is_x ? (part - a.h) * 32 : 0;
  const int chunks = is_x ? min(32, a.x_chunks - c_first) : a.kv_chunks;
  const size_t pitch = (size_t)(is_x ? a.x_chunks : a.kv_chunks) * 16;
  const size_t beam_rows = is_x ? (size_t)a.n_max : flag_beam;  // rows between two beams
  const int lanes = min(chunks, kMoveThreads), per = kMoveThreads / lanes;  // positions at once
  const int sub = threadIdx.x / lanes, c0 = threadIdx.x % lanes;
  if (sub < per) {
    for (int j = j0 + sub; j < j1; j += per) {
      uint32_t take = there[j - j0];
#pragma unroll
      for (int p = 0; p < WM; ++p)
        if (j >= upto[p]) take &= ~(1u << p);
      for (int c = c0; c < chunks; c += lanes) {
        const size_t at = (first + j) * pitch + (size_t)(c_first + c) * 16, step = beam_rows * pitch;
        // up to eight beams: K and V together (128 bytes in flight a thread)
        constexpr int kTogether = WM <= 8 ? 2 : 1;
        const int tensors = is_x ? 1 : 2;
        for (int t = 0; t < tensors; t += kTogether) {
          char* b0 = (is_x ? kv.X : t ? kv.V : kv.K) + at;
          char* b1 = kTogether == 2 && !is_x ? kv.V + at : nullptr;
          uint4 v[WM], u[kTogether == 2 ? WM : 1];
#pragma unroll
          for (int p = 0; p < WM; ++p) {
            if ((take >> p) & 1) {
              v[p] = ld16(b0 + p * step);
              if (kTogether == 2 && b1) u[p % (kTogether == 2 ? WM : 1)] = ld16(b1 + p * step);
            }
          }
#pragma unroll
          for (int p = 0; p < WM; ++p) {
            if ((take >> p) & 1) {
              for (uint32_t m = heirs[p]; m; m &= m - 1) {
                const size_t to = (__ffs(m) - 1) * step;
                st16(b0 + to, v[p]);
                if (kTogether == 2 && b1) st16(b1 + to, u[p % (kTogether == 2 ? WM : 1)]);
              }
            }
          }
        }
      }
    }
  }
  if (is_x) return;
  __syncthreads();  // the flags of these positions are read
  for (int j = j0 + threadIdx.x; j < j1; j += kMoveThreads) {
    uint8_t f[WM];
#pragma unroll
    for (int p = 0; p < WM; ++p) f[p] = j < upto[p] ? flags[p * flag_beam + j] : 0;
#pragma unroll
    for (int p = 0; p < WM; ++p)
      if (j < upto[p])
        for (uint32_t m = heirs[p]; m; m &= m - 1) flags[(__ffs(m) - 1) * flag_beam + j] = f[p];
  }
}

template <int WM>
cudaError_t run_reorder(const ReorderArgs& r, int n_kv, cudaStream_t stream) {
  ReorderArgs a = r;
  const int parts = a.h + (a.x_chunks + 31) / 32;
  // Long spans spread a CTA's start (parents, flags) over more rows; a small
  // problem is spread over the SMs instead (four beams of one layer, 112
  // positions: 10.7 us with 128 positions a CTA, 5.1 with 16; eight beams of
  // 56 heads: 454 us with 64, 370 with 128).  The host knows n_max, not the
  // positions: in a cache that is mostly empty the blocks behind the last
  // position are counted too, and read their flags before they leave.
  const auto blocks = [&](int span) { return (a.n_max + span - 1) / span; };
  a.span = kSpan;
  while (a.span > 16 && (long long)parts * blocks(a.span) * n_kv * a.S < 4 * num_sms_current()) a.span /= 2;
  reorder_kernel<WM><<<dim3(parts, blocks(a.span), n_kv * a.S), kMoveThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
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
    const int items = m.h + (m.x_chunks + 31) / 32;
    compact_kernel<<<dim3((items + kMoveWarps - 1) / kMoveWarps, m.B, n), kMoveThreads, 0, stream>>>(a);
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
