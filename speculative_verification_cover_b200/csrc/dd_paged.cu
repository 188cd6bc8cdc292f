// Attention of one new token per sequence over a paged K/V cache (dd_paged_attention).
//
// With s_hj = scale q_h . k_j over the slots j of a sequence, the softmax over any
// partition of the slots is joined from each part's maximum m, sum l = sum e^{s - m}
// and o = sum e^{s - m} v: m' = max m_i, l' = sum l_i e^{m_i - m'}, o' likewise.
//
// Work decomposition. The unit is a tile of 64 slots of one (sequence, kv head, block of
// query heads); the tiles of all of them form one index space, cut into equal contiguous
// ranges, one per CTA. So ragged batches, one long sequence and many short ones all
// spread evenly, and a range crosses at most from the end of one sequence-head through
// whole ones into the start of another: whole ones are finished in place, and at most
// two partial results per CTA are left in the workspace for the join kernel.
// Lengths are read on the device (a captured call follows them); only the launch
// depends on max_len.
//
// Bound: HBM, 2 Hkv d elements per slot read once.
#include "dd_paged.cuh"

namespace dd {

namespace {

constexpr int kTile = 64;        // slots per tile
constexpr int kPagedThreads = 128;
constexpr int kPagedWarps = kPagedThreads / 32;
constexpr int kMaxPagedGrid = 1024;  // bounds the workspace on any device
constexpr int kMaxHeads = 16;    // query heads of one block at most

struct PagedArgs {
  PagedView c;
  const char* q;
  const char* k_new;
  const char* v_new;
  int64_t q_bytes, new_bytes;  // sequence strides
  const int32_t* lengths;
  int B, Hq, G, heads, blocks;  // query heads per kv head; per block; blocks per kv head
  int max_len;
  float scale2;                // softmax scale * log2(e)
  char* out;
  float* lse;
  const float* mass_in;
  float* mass_out;
  int64_t mass_stride;
  // workspace
  int32_t* prefix;             // [B + 1] first tile of each sequence
  float2* part_ml;             // [2 grid][heads] (m, l) of the partial results, log2 units
  float* part_o;               // [2 grid][heads][d]
  float* lse2;                 // [B, Hq] in log2 units, of unsplit sequence-heads
  float* scores;               // [B, Hkv, max_len, G], log2 units (masses only)
  int grid;
};

// First tile of every sequence into smem prefix[0 .. B] (and CTA 0: the workspace, for
// the join), the tiles per CTA as the result.
__device__ int plan_tiles(const PagedArgs& a, int32_t* prefix, int* warp_tmp) {
  const int per_tile = a.c.Hkv * a.blocks;
  const int chunk = (a.B + kPagedThreads - 1) / kPagedThreads;
  const int b0 = min(a.B, (int)threadIdx.x * chunk), b1 = min(a.B, b0 + chunk);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = checked_length(a.lengths, b, a.max_len);
    prefix[b] = sum;
    sum += (n + kTile - 1) / kTile * per_tile;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) warp_tmp[warp] = incl;
  __syncthreads();
  int before = incl - sum;
  for (int w = 0; w < warp; ++w) before += warp_tmp[w];
  for (int b = b0; b < b1; ++b) prefix[b] += before;
  if (threadIdx.x == kPagedThreads - 1) prefix[a.B] = before + sum;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.B; b += kPagedThreads) a.prefix[b] = prefix[b];
  return (prefix[a.B] + a.grid - 1) / a.grid;
}

// The sequence that tile u belongs to: prefix[b] <= u < prefix[b + 1].
__device__ __forceinline__ int find_sequence(const int32_t* prefix, int B, int u) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Rows of sequences without slots: out = 0, lse = -inf.
template <typename T>
__device__ void write_empty_rows(const PagedArgs& a, const int32_t* prefix, int d) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    T* out = reinterpret_cast<T*>(a.out) + (int64_t)b * a.Hq * d;
    for (int i = threadIdx.x; i < a.Hq * d; i += kPagedThreads) store_out(out + i, 0.f);
    if (a.lse)
      for (int h = threadIdx.x; h < a.Hq; h += kPagedThreads) a.lse[(int64_t)b * a.Hq + h] = -INFINITY;
  }
}

// ------------------------------------------------------------------ CUDA-core form
template <typename T, int N>
struct LaneRow {
  float v[N];
};
template <int N>
__device__ __forceinline__ LaneRow<float, N> load_vec(const float* p) {
  LaneRow<float, N> r;
  if constexpr (N == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    r.v[0] = x.x; r.v[1] = x.y; r.v[2] = x.z; r.v[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(p);
    r.v[0] = x.x; r.v[1] = x.y;
  }
  return r;
}
template <int N>
__device__ __forceinline__ LaneRow<__nv_bfloat16, N> load_vec(const __nv_bfloat16* p) {
  LaneRow<__nv_bfloat16, N> r;
  if constexpr (N == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    r.v[0] = bf16lo(x.x); r.v[1] = bf16hi(x.x); r.v[2] = bf16lo(x.y); r.v[3] = bf16hi(x.y);
  } else {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
    r.v[0] = bf16lo(x); r.v[1] = bf16hi(x);
  }
  return r;
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const LaneRow<float, N>& x) {
#pragma unroll
  for (int e = 0; e < N; ++e) p[e] = x.v[e];
}
template <int N>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const LaneRow<__nv_bfloat16, N>& x) {
#pragma unroll
  for (int e = 0; e < N; ++e) p[e] = __float2bfloat16_rn(x.v[e]);  // came from bf16: exact
}

// Each lane holds d / 32 elements of a row. U slots at a time, a warp forms the U GB
// partial dot products and sums them over the lanes by halving: after step i a lane
// keeps the half of the products its lane bit names, so the sums cost U GB - 1 exchanges
// rather than 5 U GB, and the product of (slot u, head g) ends in the lanes whose top
// bits are u GB + g. Softmax and mass scores are then one value per lane.
template <typename T, int D, int GB>
__global__ void __launch_bounds__(kPagedThreads)
paged_simt_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int N = D / 32;
  constexpr int U = GB >= 8 ? 4 : 8;  // slots in flight per warp
  constexpr int C = U * GB;           // 8 .. 32
  constexpr int SH = C == 32 ? 0 : C == 16 ? 1 : 2;
  extern __shared__ int32_t prefix[];
  __shared__ int warp_tmp[kPagedWarps];
  __shared__ float s_m[kPagedWarps][GB], s_l[kPagedWarps][GB];
  __shared__ float s_o[kPagedWarps][GB][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = plan_tiles(a, prefix, warp_tmp);
  write_empty_rows<T>(a, prefix, D);
  const int total = prefix[a.B];
  int u = blockIdx.x * share;
  const int u_end = min(total, u + share);
  while (u < u_end) {
    const int b = find_sequence(prefix, a.B, u);
    const int len = checked_length(a.lengths, b, a.max_len);
    const int tiles = (len + kTile - 1) / kTile;
    const int rel = u - prefix[b];
    const int pair = rel / tiles, tile0 = rel - pair * tiles;
    const int n_tiles = min(tiles - tile0, u_end - u);
    const int kvh = pair / a.blocks, blk = pair - kvh * a.blocks;
    const int h0 = kvh * a.G + blk * a.heads;          // first query head of the block
    const int nh = min(a.heads, a.G - blk * a.heads);  // heads of this block
    const int j0 = tile0 * kTile, j1 = min(len, (tile0 + n_tiles) * kTile);
    const int32_t* row = a.c.table + (int64_t)b * a.c.table_stride;
    const int64_t head_off = (int64_t)kvh * a.c.head_bytes;

    float q[GB][N];
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      const T* qp = reinterpret_cast<const T*>(a.q + (int64_t)b * a.q_bytes) +
                    (int64_t)(h0 + min(g, nh - 1)) * D + lane * N;
      const auto x = load_vec<N>(qp);
#pragma unroll
      for (int e = 0; e < N; ++e) q[g][e] = x.v[e] * a.scale2;
    }
    float m = -INFINITY, l = 0.f;  // of head (lane >> SH) % GB
    float o[GB][N];
#pragma unroll
    for (int g = 0; g < GB; ++g)
#pragma unroll
      for (int e = 0; e < N; ++e) o[g][e] = 0.f;

    for (int j = j0 + warp * U; j < j1; j += kPagedWarps * U) {
      LaneRow<T, N> kr[U], vr[U];
      unsigned held = 0;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t off = j + i < j1 ? slot_offset(a.c, row, j + i) : -1;
#pragma unroll
        for (int e = 0; e < N; ++e) kr[i].v[e] = vr[i].v[e] = 0.f;
        if (off < 0) continue;
        held |= 1u << i;
        T* kp = reinterpret_cast<T*>(a.c.k + off + head_off) + lane * N;
        T* vp = reinterpret_cast<T*>(a.c.v + off + head_off) + lane * N;
        if (a.k_new && j + i == len - 1) {  // the new token: read from the caller, kept in the cache
          const int64_t at = (int64_t)b * a.new_bytes;
          kr[i] = load_vec<N>(reinterpret_cast<const T*>(a.k_new + at) + kvh * D + lane * N);
          vr[i] = load_vec<N>(reinterpret_cast<const T*>(a.v_new + at) + kvh * D + lane * N);
          if (blk == 0) {
            store_vec<N>(kp, kr[i]);
            store_vec<N>(vp, vr[i]);
          }
        } else {
          kr[i] = load_vec<N>(kp);
          vr[i] = load_vec<N>(vp);
        }
      }
      float s[C];
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          float t = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) t = fmaf(q[g][e], kr[i].v[e], t);
          s[i * GB + g] = t;
        }
      int n = C;
#pragma unroll
      for (int bit = 16; bit > 0; bit >>= 1) {
        if (n > 1) {
          n >>= 1;
          const bool up = lane & bit;
#pragma unroll
          for (int i = 0; i < C / 2; ++i)
            if (i < n) {
              const float mine = up ? s[i + n] : s[i], give = up ? s[i] : s[i + n];
              s[i] = mine + __shfl_xor_sync(0xffffffffu, give, bit);
            }
        } else {
          s[0] += __shfl_xor_sync(0xffffffffu, s[0], bit);
        }
      }
      const int c = lane >> SH, iu = c / GB, ig = c % GB;
      const float sc = (held >> iu) & 1u ? s[0] : -INFINITY;
      if (a.scores && (lane & ((1 << SH) - 1)) == 0 && ig < nh && j + iu < j1)
        a.scores[(((int64_t)b * a.c.Hkv + kvh) * a.max_len + j + iu) * a.G + blk * a.heads + ig] = sc;
      float mx = sc;
#pragma unroll
      for (int bit = 16; bit >= 32 / U; bit >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, bit));
      const float m_new = fmaxf(m, mx);
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float p = exp2f(sc - base);
      const float alpha = exp2f(m - base);
      float ps = p;
#pragma unroll
      for (int bit = 16; bit >= 32 / U; bit >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, bit);
      l = l * alpha + ps;
      m = m_new;
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        const float al = __shfl_sync(0xffffffffu, alpha, g << SH);
#pragma unroll
        for (int e = 0; e < N; ++e) o[g][e] *= al;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float pi = __shfl_sync(0xffffffffu, p, (i * GB + g) << SH);
#pragma unroll
          for (int e = 0; e < N; ++e) o[g][e] = fmaf(pi, vr[i].v[e], o[g][e]);
        }
      }
    }
    // ---- join the four warps
    __syncthreads();  // the previous piece's reads of s_* are over
    if (lane < (GB << SH) && (lane & ((1 << SH) - 1)) == 0) {
      s_m[warp][lane >> SH] = m;
      s_l[warp][lane >> SH] = l;
    }
#pragma unroll
    for (int g = 0; g < GB; ++g)
#pragma unroll
      for (int e = 0; e < N; ++e) s_o[warp][g][lane * N + e] = o[g][e];
    __syncthreads();
    const bool starts = tile0 == 0, whole = starts && n_tiles == tiles;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (starts ? 1 : 0);
    for (int i = threadIdx.x; i < nh * D; i += kPagedThreads) {
      const int g = i / D, e = i - g * D;
      float mm = s_m[0][g];
#pragma unroll
      for (int w = 1; w < kPagedWarps; ++w) mm = fmaxf(mm, s_m[w][g]);
      const float base = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f, oo = 0.f;
#pragma unroll
      for (int w = 0; w < kPagedWarps; ++w) {
        const float f = exp2f(s_m[w][g] - base);
        ll = fmaf(s_l[w][g], f, ll);
        oo = fmaf(s_o[w][g][e], f, oo);
      }
      if (whole) {
        const int64_t h = (int64_t)b * a.Hq + h0 + g;
        store_out(reinterpret_cast<T*>(a.out) + h * D + e, ll > 0.f ? oo / ll : 0.f);
        if (e == 0) {
          const float z2 = ll > 0.f ? mm + log2f(ll) : -INFINITY;
          a.lse2[h] = z2;
          if (a.lse) a.lse[h] = z2 * kLn2;
        }
      } else if (DD_IN_BOUNDS(slot < 2ll * a.grid)) {
        a.part_o[(slot * a.heads + g) * D + e] = oo;
        if (e == 0) a.part_ml[slot * a.heads + g] = make_float2(mm, ll);
      }
    }
    u += n_tiles;
  }
}

// ------------------------------------------------------------------ join and masses
// CTAs whose tiles hold a sequence-head: first and last, from the plan of the main kernel.
struct Span {
  int c0, c1, tiles;
};
__device__ __forceinline__ Span split_of(const PagedArgs& a, int b, int pair) {
  Span s;
  const int p0 = a.prefix[b], p1 = a.prefix[b + 1];
  const int share = (a.prefix[a.B] + a.grid - 1) / a.grid;
  s.tiles = (p1 - p0) / (a.c.Hkv * a.blocks);
  if (s.tiles == 0) return s;
  const int first = p0 + pair * s.tiles;
  s.c0 = first / share;
  s.c1 = (first + s.tiles - 1) / share;
  return s;
}
__device__ __forceinline__ int64_t part_slot(const Span& s, int c) {
  return 2 * (int64_t)c + (c == s.c0 ? 1 : 0);
}

constexpr int kJoinThreads = 128;
constexpr int kMassChunk = 256;  // slots per step of a mass CTA

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(const __grid_constant__ PagedArgs a, int out_ctas, int mass_ctas) {
  pdl_wait();
  constexpr int N = D / 32;
  extern __shared__ float z2[];  // [Hq] of this sequence, log2 units (mass CTAs)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x < out_ctas) {  // one warp per (sequence, query head)
    const int64_t i = (int64_t)blockIdx.x * (kJoinThreads / 32) + warp;
    if (i >= (int64_t)a.B * a.Hq) return;
    const int b = (int)(i / a.Hq), h = (int)(i - (int64_t)b * a.Hq);
    const int kvh = h / a.G, g = h - kvh * a.G, blk = g / a.heads, gi = g - blk * a.heads;
    const Span s = split_of(a, b, kvh * a.blocks + blk);
    if (s.tiles == 0 || s.c0 == s.c1) return;  // already whole
    float m = -INFINITY;
    for (int c = s.c0 + lane; c <= s.c1; c += 32)
      m = fmaxf(m, a.part_ml[part_slot(s, c) * a.heads + gi].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int c = s.c0; c <= s.c1; ++c) {
      const int64_t at = part_slot(s, c) * a.heads + gi;
      const float2 ml = a.part_ml[at];
      const float f = exp2f(ml.x - base);
      const auto x = load_vec<N>(a.part_o + at * D + lane * N);
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = fmaf(x.v[e], f, acc[e]);
    }
    T* out = reinterpret_cast<T*>(a.out) + i * D + lane * N;
#pragma unroll
    for (int e = 0; e < N; ++e) store_out(out + e, l > 0.f ? acc[e] / l : 0.f);
    if (lane == 0 && a.lse) a.lse[i] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    return;
  }
  // ---- masses of one sequence's slots
  const int k = blockIdx.x - out_ctas, b = k / mass_ctas, part = k - b * mass_ctas;
  const int len = checked_length(a.lengths, b, a.max_len);
  if (part * kMassChunk >= len) return;
  for (int h = warp; h < a.Hq; h += kJoinThreads / 32) {
    const int kvh = h / a.G, g = h - kvh * a.G, blk = g / a.heads, gi = g - blk * a.heads;
    const Span s = split_of(a, b, kvh * a.blocks + blk);
    float z;
    if (s.c0 == s.c1) {
      z = a.lse2[(int64_t)b * a.Hq + h];
    } else {
      float m = -INFINITY, l = 0.f;
      for (int c = s.c0 + lane; c <= s.c1; c += 32) {
        const float2 ml = a.part_ml[part_slot(s, c) * a.heads + gi];
        const float mn = fmaxf(m, ml.x);
        const float base = mn == -INFINITY ? 0.f : mn;
        l = l * exp2f(m - base) + ml.y * exp2f(ml.x - base);
        m = mn;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        const float mn = fmaxf(m, m2);
        const float base = mn == -INFINITY ? 0.f : mn;
        l = l * exp2f(m - base) + l2 * exp2f(m2 - base);
        m = mn;
      }
      z = l > 0.f ? m + log2f(l) : -INFINITY;
    }
    if (lane == 0) z2[h] = z;
  }
  __syncthreads();
  const float inv = 1.f / (float)a.Hq;
  for (int j = part * kMassChunk + threadIdx.x; j < len; j += kMassChunk * mass_ctas) {
#pragma unroll
    for (int half = 0; half < kMassChunk / kJoinThreads; ++half) {
      const int jj = j + half * kJoinThreads;
      if (jj >= len) break;
      float sum = 0.f;
      for (int kvh = 0; kvh < a.c.Hkv; ++kvh) {
        const float* sp = a.scores + (((int64_t)b * a.c.Hkv + kvh) * a.max_len + jj) * a.G;
        for (int g = 0; g < a.G; ++g) {
          const float z = z2[kvh * a.G + g];
          if (z > -INFINITY) sum += exp2f(sp[g] - z);
        }
      }
      const int64_t at = (int64_t)b * a.mass_stride + jj;
      const bool fresh = a.k_new && jj == len - 1;
      const float before = a.mass_in && !fresh ? a.mass_in[at] : 0.f;
      a.mass_out[at] = before + sum * inv;
    }
  }
}

struct PagedWorkspace {
  size_t prefix, ml, o, lse2, scores, total;
};
// Heads of one block: a kv head's query heads in as few equal blocks as the limit allows.
int head_blocks(int G, int limit) { return (G + limit - 1) / limit; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

PagedWorkspace paged_layout(int B, int Hq, int d, int max_len, bool mass, int heads) {
  PagedWorkspace w;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align256(bytes);
    return r;
  };
  w.prefix = take(((size_t)B + 1) * 4);
  w.ml = take((size_t)2 * kMaxPagedGrid * heads * 8);
  w.o = take((size_t)2 * kMaxPagedGrid * heads * d * 4);
  w.lse2 = take((size_t)B * Hq * 4);
  w.scores = take(mass ? (size_t)B * Hq * max_len * 4 : 0);
  w.total = at;
  return w;
}

template <typename T, int D>
cudaError_t launch_simt(const PagedArgs& a, size_t smem, cudaStream_t stream) {
  switch (a.heads) {
    case 1: paged_simt_kernel<T, D, 1><<<a.grid, kPagedThreads, smem, stream>>>(a); break;
    case 2: paged_simt_kernel<T, D, 2><<<a.grid, kPagedThreads, smem, stream>>>(a); break;
    case 3: case 4: paged_simt_kernel<T, D, 4><<<a.grid, kPagedThreads, smem, stream>>>(a); break;
    default: paged_simt_kernel<T, D, 8><<<a.grid, kPagedThreads, smem, stream>>>(a); break;
  }
  return cudaGetLastError();
}

int heads_per_block(int G) {
  const int blocks = head_blocks(G, 8);
  return (G + blocks - 1) / blocks;
}

}  // namespace

PagedView make_paged_view(const dd_paged_cache& c) {
  const int64_t e = c.dtype == DD_BF16 ? 2 : 4;
  PagedView v{};
  v.k = static_cast<char*>(c.k);
  v.v = static_cast<char*>(c.v);
  v.layer_bytes = c.layer_stride * e;
  v.page_bytes = c.page_stride * e;
  v.token_bytes = c.token_stride * e;
  v.head_bytes = c.head_stride * e;
  v.layers = c.layers;
  v.n_pages = c.n_pages;
  v.Hkv = c.Hkv;
  const int64_t cap = (int64_t)c.max_pages * c.page_size;
  v.cap = cap > 0x7fffffffll ? 0x7fffffff : (int)cap;
  v.page = make_fast_div(c.page_size);
  v.table = c.page_table;
  v.table_stride = c.table_stride;
  v.max_pages = c.max_pages;
  return v;
}

size_t paged_attention_workspace(int B, int Hq, int Hkv, int d, int max_len, bool mass) {
  return paged_layout(B, Hq, d, max_len, mass, heads_per_block(Hq / Hkv)).total;
}

int64_t paged_attention_tiles(int B, int Hq, int max_len) {
  return (int64_t)B * Hq * ((max_len + kTile - 1) / kTile);
}

cudaError_t launch_paged_attention(const PagedCall& p, cudaStream_t stream) {
  const dd_paged_cache& c = *p.cache;
  PagedArgs a{};
  a.c = make_paged_view(c);
  const int64_t e = c.dtype == DD_BF16 ? 2 : 4;
  a.q = static_cast<const char*>(p.q);
  a.k_new = static_cast<const char*>(p.k_new);
  a.v_new = static_cast<const char*>(p.v_new);
  a.q_bytes = p.q_stride * e;
  a.new_bytes = p.new_stride * e;
  a.lengths = p.lengths;
  a.B = p.B; a.Hq = p.Hq; a.G = p.Hq / c.Hkv;
  a.heads = heads_per_block(a.G);
  a.blocks = (a.G + a.heads - 1) / a.heads;
  a.max_len = p.max_len;
  a.scale2 = (p.scale > 0.f ? p.scale : 1.f / sqrtf((float)c.d)) * kLog2e;
  a.out = static_cast<char*>(p.out);
  a.lse = p.lse;
  a.mass_in = p.mass_in; a.mass_out = p.mass_out; a.mass_stride = p.mass_stride;
  const PagedWorkspace w = paged_layout(p.B, p.Hq, c.d, p.max_len, p.mass_out != nullptr, a.heads);
  char* ws = static_cast<char*>(p.workspace);
  a.prefix = reinterpret_cast<int32_t*>(ws + w.prefix);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  a.scores = p.mass_out ? reinterpret_cast<float*>(ws + w.scores) : nullptr;
  const int64_t tiles = (int64_t)p.B * c.Hkv * a.blocks * ((p.max_len + kTile - 1) / kTile);
  const int64_t most = min((int64_t)kMaxPagedGrid, (int64_t)device_info().sm_count * 4);
  a.grid = (int)(tiles < most ? tiles : most);
  const size_t smem = ((size_t)p.B + 1) * 4;
  cudaError_t err;
  if (c.dtype == DD_BF16)
    err = c.d == 128 ? launch_simt<__nv_bfloat16, 128>(a, smem, stream)
                     : launch_simt<__nv_bfloat16, 64>(a, smem, stream);
  else
    err = c.d == 128 ? launch_simt<float, 128>(a, smem, stream) : launch_simt<float, 64>(a, smem, stream);
  if (err != cudaSuccess) return err;
  // join: one warp per query head; masses: enough CTAs a sequence to fill the GPU a few times
  const int out_ctas = (int)(((int64_t)p.B * p.Hq + 3) / 4);
  int mass_ctas = 0;
  if (p.mass_out) {
    const int chunks = (p.max_len + kMassChunk - 1) / kMassChunk;
    const int fill = (device_info().sm_count * 8 + p.B - 1) / p.B;
    mass_ctas = chunks < fill ? chunks : fill;
  }
  const dim3 grid(out_ctas + mass_ctas * p.B);
  const size_t zmem = p.mass_out ? (size_t)p.Hq * 4 : 0;
  const auto join = [&](auto kernel) {
    return launch_dependent(kernel, grid, dim3(kJoinThreads), zmem, stream, a, out_ctas, mass_ctas);
  };
  if (c.dtype == DD_BF16)
    return c.d == 128 ? join(paged_join_kernel<__nv_bfloat16, 128>)
                      : join(paged_join_kernel<__nv_bfloat16, 64>);
  return c.d == 128 ? join(paged_join_kernel<float, 128>) : join(paged_join_kernel<float, 64>);
}

}  // namespace dd
