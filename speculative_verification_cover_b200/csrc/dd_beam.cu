// Beam search's selection over beams and vocabulary (dd_beam_select).
//
// score(k, v) = score_k + x_kv - lse_k with lse_k = log sum_u e^{x_ku}. Within a beam the
// order of the candidates is the order of the logits, so the scan of a row needs no lse:
// each CTA reads one piece of one row once, leaves the piece's maximum, its sum of
// exponentials and its K best logits, and a merge CTA per request joins the sums and picks
// the K best candidates by score, in 64 bits.
//
// Bound: HBM, B K V logits read once.
#include "dd_common.cuh"
#include "dd_internal.h"

namespace dd {

namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamVecs = 4;  // 16-byte vectors per thread
constexpr uint32_t kNone = 0x007FFFFFu;  // key of -inf

template <typename T>
constexpr int beam_piece() { return kBeamThreads * kBeamVecs * (16 / (int)sizeof(T)); }

__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// NaN is no candidate; -0 ties with 0.
__device__ __forceinline__ float clean_logit(float x) { return x == x ? x + 0.f : -INFINITY; }

template <typename T, int PV>
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[PV]) {
  if constexpr (PV == 4) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  } else {
    x[0] = bf16lo(r.x); x[1] = bf16hi(r.x); x[2] = bf16lo(r.y); x[3] = bf16hi(r.y);
    x[4] = bf16lo(r.z); x[5] = bf16hi(r.z); x[6] = bf16lo(r.w); x[7] = bf16hi(r.w);
  }
}

__device__ __forceinline__ bool scans(const float* score_in, const uint8_t* done_in, int row) {
  const float s = score_in[row];
  return s > -INFINITY && !(done_in && done_in[row]);
}

// One piece of one row. The K-th largest of the 256 threads' maxima is a lower bound of the
// piece's K-th largest logit, and only the fewer than K threads whose maximum lies above it
// hold logits above it: those are collected and ranked by counting, and the lowest indices
// of the logits equal to it (a bitmap) fill up.
template <typename T>
__global__ void __launch_bounds__(kBeamThreads)
beam_scan_kernel(const T* __restrict__ logits, int K, int V, int64_t ld, int pieces,
                 const float* __restrict__ score_in, const uint8_t* __restrict__ done_in,
                 float2* __restrict__ ml, uint2* __restrict__ cand) {
  constexpr int PV = 16 / (int)sizeof(T);
  constexpr int kPiece = beam_piece<T>();
  constexpr int kMost = (kBeamMaxK - 1) * kBeamVecs * PV;  // logits above the bound
  __shared__ uint32_t s_key[kBeamThreads];
  __shared__ uint32_t s_gt_key[kMost];
  __shared__ int s_gt_idx[kMost];
  __shared__ uint32_t s_tie[kPiece / 32];
  __shared__ float s_red[kBeamThreads / 32];
  __shared__ int s_scan[kBeamThreads / 32];
  __shared__ uint32_t s_bound;
  __shared__ int s_n;
  const int row = blockIdx.x / pieces, piece = blockIdx.x - row * pieces;
  if (!scans(score_in, done_in, row)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* x0 = logits + (int64_t)row * ld;
  const int base = piece * kPiece;
  uint4 raw[kBeamVecs];
#pragma unroll
  for (int i = 0; i < kBeamVecs; ++i) {
    const int v = base + (i * kBeamThreads + threadIdx.x) * PV;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < V) raw[i] = *reinterpret_cast<const uint4*>(x0 + v);
  }
  const auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kBeamVecs; ++i) {
      float x[PV];
      unpack<T, PV>(raw[i], x);
      const int at = (i * kBeamThreads + threadIdx.x) * PV;
#pragma unroll
      for (int e = 0; e < PV; ++e) f(base + at + e < V ? clean_logit(x[e]) : -INFINITY, at + e);
    }
  };
  float mx = -INFINITY;
  each([&](float x, int) { mx = fmaxf(mx, x); });
  s_key[threadIdx.x] = logit_key(mx);
  for (int i = threadIdx.x; i < kPiece / 32; i += kBeamThreads) s_tie[i] = 0u;
  float m = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_red[warp] = m;
  if (threadIdx.x == 0) { s_bound = kNone; s_n = 0; }
  __syncthreads();
  m = s_red[0];
#pragma unroll
  for (int w = 1; w < kBeamThreads / 32; ++w) m = fmaxf(m, s_red[w]);
  const float mb = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
  each([&](float x, int) { sum += exp2f((x - mb) * kLog2e); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  // the K-th largest thread maximum
  const uint32_t mine = s_key[threadIdx.x];
  int above = 0;
  for (int t = 0; t < kBeamThreads; ++t) {
    const uint32_t k = s_key[t];
    above += k > mine || (k == mine && t < (int)threadIdx.x);
  }
  if (above == K - 1) s_bound = mine;
  __syncthreads();
  if (lane == 0) s_red[warp] = sum;
  const uint32_t bound = s_bound;
  if (mine >= bound && mine > kNone)
    each([&](float x, int at) {
      const uint32_t k = logit_key(x);
      if (k > bound) {
        const int i = atomicAdd(&s_n, 1);
        if (DD_IN_BOUNDS(i < kMost)) { s_gt_key[i] = k; s_gt_idx[i] = at; }
      } else if (k == bound && bound > kNone) {
        atomicOr(&s_tie[at >> 5], 1u << (at & 31));
      }
    });
  __syncthreads();
  const int n = min(s_n, kMost);
  uint2* out = cand + (int64_t)blockIdx.x * K;
  for (int i = threadIdx.x; i < n; i += kBeamThreads) {
    const uint32_t k = s_gt_key[i];
    const int at = s_gt_idx[i];
    int r = 0;
    for (int t = 0; t < n; ++t) r += s_gt_key[t] > k || (s_gt_key[t] == k && s_gt_idx[t] < at);
    if (r < K) out[r] = make_uint2(k, (uint32_t)(base + at));
  }
  // ties fill up from the lowest index
  uint32_t bits = threadIdx.x < kPiece / 32 ? s_tie[threadIdx.x] : 0u;
  const int cnt = __popc(bits);
  int incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int r = n + incl - cnt, all = n;
#pragma unroll
  for (int w = 0; w < kBeamThreads / 32; ++w) {
    if (w < warp) r += s_scan[w];
    all += s_scan[w];
  }
  for (; bits && r < K; ++r, bits &= bits - 1u)
    out[r] = make_uint2(bound, (uint32_t)(base + threadIdx.x * 32 + __ffs(bits) - 1));
  for (int i = all + threadIdx.x; i < K; i += kBeamThreads) out[i] = make_uint2(kNone, 0u);
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBeamThreads / 32; ++w) s += s_red[w];
    ml[blockIdx.x] = make_float2(m, s);
  }
}

struct Best {
  double score;
  int64_t at;  // k V + v
  int list;
};
__device__ __forceinline__ bool better(double s, int64_t at, double s2, int64_t at2) {
  return s > s2 || (s == s2 && at < at2);
}

// One CTA per request: K rounds, each taking the best head of the sorted lists (one per
// beam and piece) and stepping that list on.
__global__ void __launch_bounds__(kBeamThreads)
beam_merge_kernel(int K, int V, int pieces, const float* __restrict__ score_in,
                  const uint8_t* __restrict__ done_in, int eos, const float2* __restrict__ ml,
                  const uint2* __restrict__ cand, int32_t* __restrict__ parent,
                  int32_t* __restrict__ token, float* __restrict__ score_out,
                  uint8_t* __restrict__ done_out) {
  pdl_wait();
  extern __shared__ uint8_t head[];  // [K * pieces]
  __shared__ double s_base[kBeamMaxK];
  __shared__ uint8_t s_kind[kBeamMaxK];  // 0 no candidate, 1 live, 2 done
  __shared__ Best s_best[kBeamThreads / 32];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int k = warp; k < K; k += kBeamThreads / 32) {
    const int row = b * K + k;
    const float s = score_in[row];
    if (!scans(score_in, done_in, row)) {
      if (lane == 0) {
        s_kind[k] = s > -INFINITY ? 2 : 0;
        s_base[k] = (double)s;
      }
      continue;
    }
    float m = -INFINITY;
    for (int i = lane; i < pieces; i += 32) m = fmaxf(m, ml[(int64_t)row * pieces + i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double z = 0.0;
    if (m > -INFINITY)
      for (int i = lane; i < pieces; i += 32) {
        const float2 p = ml[(int64_t)row * pieces + i];
        z += (double)p.y * exp((double)p.x - (double)m);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) {
      s_kind[k] = m > -INFINITY ? 1 : 0;
      s_base[k] = (double)s - ((double)m + log(z));
    }
  }
  const int lists = K * pieces;
  for (int i = threadIdx.x; i < lists; i += kBeamThreads) head[i] = 0;
  __syncthreads();
  const auto find = [&](Best& best) {
    best = Best{-INFINITY, INT64_MAX, -1};
    for (int i = threadIdx.x; i < lists; i += kBeamThreads) {
      const int k = i / pieces, h = head[i];
      double s;
      int64_t at;
      if (s_kind[k] == 1) {
        if (h >= K) continue;
        const uint2 c = cand[((int64_t)b * lists + i) * K + h];
        if (c.x <= kNone) continue;
        s = s_base[k] + (double)key_logit(c.x);
        at = (int64_t)k * V + c.y;
      } else {
        if (s_kind[k] == 0 || i != k * pieces || h > 0) continue;
        s = s_base[k];
        at = (int64_t)k * V + (eos > 0 ? eos : 0);
      }
      if (better(s, at, best.score, best.at)) best = Best{s, at, i};
    }
  };
  Best own;
  find(own);
  for (int r = 0; r < K; ++r) {
    Best best = own;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double s = __shfl_xor_sync(0xffffffffu, best.score, o);
      const int64_t at = __shfl_xor_sync(0xffffffffu, best.at, o);
      const int list = __shfl_xor_sync(0xffffffffu, best.list, o);
      if (better(s, at, best.score, best.at)) best = Best{s, at, list};
    }
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    best = s_best[0];
    for (int w = 1; w < kBeamThreads / 32; ++w)
      if (better(s_best[w].score, s_best[w].at, best.score, best.at)) best = s_best[w];
    __syncthreads();
    const bool found = best.list >= 0;
    if (threadIdx.x == 0) {
      const int64_t o = (int64_t)b * K + r;
      const int k = found ? best.list / pieces : -1;
      const bool was_done = found && s_kind[k] == 2;
      const int v = !found ? -1 : was_done ? eos : (int)(best.at - (int64_t)k * V);
      parent[o] = k;
      token[o] = v;
      score_out[o] = found ? (float)best.score : -INFINITY;
      if (done_out) done_out[o] = was_done || (found && v == eos) ? 1 : 0;
    }
    if (found && best.list % kBeamThreads == (int)threadIdx.x) {
      head[best.list] += 1;
      find(own);
    }
  }
}

}  // namespace

namespace {
int beam_pieces(int V, dd_dtype dtype) {
  const int piece = dtype == DD_BF16 ? beam_piece<__nv_bfloat16>() : beam_piece<float>();
  return (V + piece - 1) / piece;
}
}  // namespace

size_t beam_select_workspace(int B, int K, int V, dd_dtype dtype) {
  const size_t lists = (size_t)B * K * beam_pieces(V, dtype);
  return ((lists * 8 + 255) & ~(size_t)255) + ((lists * K * 8 + 255) & ~(size_t)255);
}

cudaError_t launch_beam_select(const BeamCall& p, cudaStream_t stream) {
  const int pieces = beam_pieces(p.V, p.dtype);
  const size_t lists = (size_t)p.B * p.K * pieces;
  float2* ml = static_cast<float2*>(p.workspace);
  uint2* cand = reinterpret_cast<uint2*>(static_cast<char*>(p.workspace) + ((lists * 8 + 255) & ~(size_t)255));
  if (p.dtype == DD_BF16)
    beam_scan_kernel<__nv_bfloat16><<<(unsigned)lists, kBeamThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(p.logits), p.K, p.V, p.ld, pieces, p.score_in, p.done_in, ml, cand);
  else
    beam_scan_kernel<float><<<(unsigned)lists, kBeamThreads, 0, stream>>>(
        static_cast<const float*>(p.logits), p.K, p.V, p.ld, pieces, p.score_in, p.done_in, ml, cand);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  static thread_local int configured_for = -1;
  if (configured_for != device_info().device) {
    e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kBeamMaxK * (kBeamMaxV / beam_piece<float>()));
    if (e != cudaSuccess) return e;
    configured_for = device_info().device;
  }
  return launch_dependent(beam_merge_kernel, dim3(p.B), dim3(kBeamThreads), (size_t)p.K * pieces, stream, p.K,
                          p.V, pieces, p.score_in, p.done_in, p.eos, (const float2*)ml, (const uint2*)cand,
                          p.parent, p.token, p.score_out, p.done_out);
}

}  // namespace dd
