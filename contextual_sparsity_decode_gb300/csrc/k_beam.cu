// Beam selection: the K best continuations of a sequence over its W beams and
// the vocabulary,
//     score(w, v) = cum[w] + x[w][v] - logsumexp(x[w][:]),
// by score descending, ties to the lower w V + v.
//
// Within a beam the order is that of the logits themselves (the log-sum-exp is
// one number per row), so the selection inside a row is exact and needs no
// arithmetic; only the candidates of different beams are compared by score, in
// double precision.
//
// One CTA takes kChunk consecutive tokens of a row into registers, reduces
// their maximum and sum of exponentials and lists their K largest; the last
// CTA of a sequence to finish joins the chunks (log-sum-exp in double, chunk
// by chunk in order) and picks the K best of the listed candidates.  The
// elements of a thread and the order of every sum depend on the token index
// alone, so rows with equal logits get equal sums.

#include "dv_kernels.h"

namespace dv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 32;                      // tokens per thread
static_assert(kThreads * kPer == kBeamChunk, "tokens per CTA");

// Order-preserving map of a float to unsigned; NaN is treated elsewhere.
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  return v;
}

// A candidate of the join: score, then the lower flat index.
struct Cand {
  double s;
  long long f;  // w V + v, or -1: none
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  if (b.f < 0) return a.f >= 0;
  if (a.f < 0) return false;
  return a.s > b.s || (a.s == b.s && a.f < b.f);
}
__device__ __forceinline__ Cand warp_best(Cand c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Cand d;
    d.s = __shfl_xor_sync(0xffffffffu, c.s, o);
    d.f = __shfl_xor_sync(0xffffffffu, c.f, o);
    if (before(d, c)) c = d;
  }
  return c;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_kernel(const BeamLaunch a) {
  __shared__ float redf[kThreads / 32];
  __shared__ unsigned long long red64[kThreads / 32];
  __shared__ Cand redc[kThreads / 32];
  __shared__ double base[kBeamMaxWidth];   // cum - lse of a row
  __shared__ int kind[kBeamMaxWidth];      // 0: listed tokens, 1: every token at -inf, 2: ended
  __shared__ int last;
  const int chunk = blockIdx.x, w = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row = s * a.W + w;
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.ld;
  const int v0 = chunk * kBeamChunk;

  float f[kPer];
  float m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = v0 + i * kThreads + tid;
    f[i] = v < a.V ? Elem<T>::to_f(x[v]) : -INFINITY;
    bad |= !(f[i] < INFINITY);   // NaN or +inf
    m = fmaxf(m, f[i]);
  }
  m = warp_max(m);
  if (lane == 0) redf[wid] = m;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int q = 0; q < kThreads / 32; ++q) m = fmaxf(m, redf[q]);
  __syncthreads();
  float sum = 0.f;
  if (m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += expf(f[i] - m);
  }
  sum = warp_sum(sum);
  if (lane == 0) redf[wid] = sum;
  __syncthreads();
  const size_t slot = (size_t)row * a.chunks + chunk;
  if (tid == 0) {
    double t = 0.0;
    for (int q = 0; q < kThreads / 32; ++q) t += (double)redf[q];
    a.stat[slot] = make_float2(bad ? NAN : m, (float)t);
  }
  // the K largest, by (value, lower index): one more each round
  unsigned long long prev = ~0ull;
  for (int k = 0; k < a.K; ++k) {
    unsigned long long best = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int v = v0 + i * kThreads + tid;
      const unsigned long long key = ((unsigned long long)ord32(f[i]) << 32) | (uint32_t)~v;
      if (v < a.V && key < prev && key > best) best = key;
    }
    best = warp_max_u64(best);
    if (lane == 0) red64[wid] = best;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kThreads / 32; ++q) best = red64[q] > best ? red64[q] : best;
    __syncthreads();
    if (tid == 0) a.cand[slot * a.K + k] = make_int2(best ? __float_as_int(unord32(best >> 32)) : 0, best ? (int)~(uint32_t)best : -1);
    prev = best;
  }

  // the sequence's last CTA joins
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(&a.ctr[s], 1) == a.W * a.chunks - 1;
    if (last) {
      a.ctr[s] = 0;
      __threadfence();
    }
  }
  __syncthreads();
  if (!last) return;
  if (tid < a.W) {
    const int r = s * a.W + tid;
    float M = -INFINITY;
    bool nan = false;
    for (int c = 0; c < a.chunks; ++c) {
      const float2 st = __ldcg(&a.stat[(size_t)r * a.chunks + c]);
      nan |= st.x != st.x;
      M = fmaxf(M, st.x);
    }
    double t = 0.0;
    for (int c = 0; c < a.chunks; ++c) {
      const float2 st = __ldcg(&a.stat[(size_t)r * a.chunks + c]);
      if (st.y > 0.f) t += (double)st.y * exp((double)st.x - (double)M);
    }
    const float cum = a.cum[r];
    const bool open = cum > -INFINITY && cum < INFINITY;   // NaN and +inf count as -inf
    if (a.done && a.done[r]) {
      kind[tid] = 2;
      base[tid] = open ? (double)cum : -INFINITY;
    } else if (nan || !(M > -INFINITY) || !open) {
      kind[tid] = 1;
    } else {
      kind[tid] = 0;
      base[tid] = (double)M + log(t);
    }
  }
  __syncthreads();
  const int per_row = a.chunks * a.K;
  Cand prevc{INFINITY, -1};
  for (int k = 0; k < a.K; ++k) {
    Cand best{-INFINITY, -1};
    for (int i = tid; i < a.W * per_row; i += kThreads) {
      const int bw = i / per_row, e = i - bw * per_row;
      Cand c{-INFINITY, -1};
      if (kind[bw] == 0) {
        const int2 p = __ldcg(&a.cand[(size_t)(s * a.W + bw) * per_row + e]);
        if (p.y >= 0) {
          c.s = (double)a.cum[s * a.W + bw] + ((double)__int_as_float(p.x) - base[bw]);
          c.f = (long long)bw * a.V + p.y;
        }
      } else if (e < a.K) {
        // the K lowest tokens at -inf; an ended beam's end token at its score
        // takes the place of itself, or of the last of them
        if (e < a.V) c.f = (long long)bw * a.V + e;
        if (kind[bw] == 2 && (e == a.end || (e == a.K - 1 && a.end >= a.K))) {
          c.f = (long long)bw * a.V + a.end;
          c.s = base[bw];
        }
      }
      if (c.f >= 0 && (prevc.f < 0 || before(prevc, c)) && before(c, best)) best = c;
    }
    best = warp_best(best);
    if (lane == 0) redc[wid] = best;
    __syncthreads();
    best = redc[0];
#pragma unroll
    for (int q = 1; q < kThreads / 32; ++q)
      if (before(redc[q], best)) best = redc[q];
    __syncthreads();
    if (tid == 0) {
      a.score[(size_t)s * a.K + k] = (float)best.s;
      a.token[(size_t)s * a.K + k] = (int)(best.f % a.V);
      a.beam[(size_t)s * a.K + k] = (int)(best.f / a.V);
    }
    prevc = best;
  }
}

}  // namespace

cudaError_t launch_beam_select(const BeamLaunch& a, dv_dtype dt, cudaStream_t stream) {
  const dim3 grid(a.chunks, a.W, a.S);
  switch (dt) {
    case DV_F32: beam_kernel<float><<<grid, kThreads, 0, stream>>>(a); break;
    case DV_F16: beam_kernel<__half><<<grid, kThreads, 0, stream>>>(a); break;
    case DV_BF16: beam_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a); break;
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dv
