// Eviction from a paged cache by accumulated attention mass (dd_cache_evict), and what
// beams do to caches and states (dd_paged_fork, dd_beam_reorder).
#include "dd_paged.cuh"

namespace dd {

namespace {

constexpr int kEvictThreads = 512;

// Ranking key of a slot: protected slots above everything, then the mass (as an
// order-preserving integer; NaN below every number).
__device__ __forceinline__ uint32_t evict_key(float mass, int pos, int sink, int64_t newest,
                                              int recent) {
  if (pos < sink || (int64_t)pos > newest - recent) return 0xFFFFFFFFu;
  if (mass != mass) return 0u;
  const uint32_t u = __float_as_uint(mass + 0.f);  // -0 ranks as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Bits of the slots below `limit` in word w of a slot bitmap.
__device__ __forceinline__ uint32_t below_mask(int w, int limit) {
  const int n = limit - w * 32;
  return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// Exclusive prefix sum of f(w) over the words [w0, w1) into out[w].
template <typename F>
__device__ void scan_words(int w0, int w1, uint32_t* out, int* warp_tmp, F f) {
  const int n = w1 - w0, chunk = (n + kEvictThreads - 1) / kEvictThreads;
  const int a = w0 + min(n, (int)threadIdx.x * chunk), e = min(w1, a + chunk);
  int sum = 0;
  for (int w = a; w < e; ++w) sum += f(w);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) warp_tmp[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += warp_tmp[w];
  for (int w = a; w < e; ++w) {
    const int c = f(w);  // before out[w] is written: out may be what f reads
    out[w] = (uint32_t)run;
    run += c;
  }
  __syncthreads();
}

// Grid (CTAs per sequence, sequences). The selection reads 8 bytes a slot; every CTA of a
// sequence repeats it (the repeats come from L2) and then does its share of the moves, so
// nothing has to be handed from one CTA to another. The budget-th largest key is found by
// a radix select, 8 bits a pass; kept slots become a bitmap in shared memory, and the i-th
// freed slot below the new length takes the i-th kept slot at or beyond it: both are ranks
// over the bitmap (a prefix count per word and a bit count).
__global__ void __launch_bounds__(kEvictThreads)
evict_kernel(PagedView c, const int32_t* __restrict__ lengths, int max_len, int budget, int sink,
             int recent, const float* __restrict__ mass_in, const int32_t* __restrict__ pos_in,
             int64_t stride, float* __restrict__ mass_out, int32_t* __restrict__ pos_out,
             int32_t* __restrict__ src_out, int32_t* __restrict__ lengths_out, int chunk16_log2) {
  extern __shared__ uint32_t words[];
  __shared__ unsigned int hist[256];
  __shared__ int warp_tmp[kEvictThreads / 32];
  __shared__ uint32_t prefix_s;
  __shared__ int need_s, newest_s, moves_s;
  __shared__ int2 moves[kEvictThreads];
  const int n = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = checked_length(lengths, n, max_len);
  const int left = min(len, budget);
  const float* mass = mass_in + (int64_t)n * stride;
  const int32_t* pos = pos_in + (int64_t)n * stride;
  if (blockIdx.x == 0 && threadIdx.x == 0) lengths_out[n] = left;
  const int W = (len + 31) >> 5, wl = left >> 5;
  uint32_t* kept = words;         // [W] bitmap
  uint32_t* rank = words + W;     // [W] freed slots before word w (w <= wl), else movers before it
  uint32_t* tie = words + 2 * W;  // [W] bitmap of slots at the threshold
  if (len > budget) {
    if (threadIdx.x == 0) newest_s = INT32_MIN;
    for (int t = threadIdx.x; t < 256; t += kEvictThreads) hist[t] = 0u;
    __syncthreads();
    int top = INT32_MIN;
    for (int j = threadIdx.x; j < len; j += kEvictThreads) top = max(top, pos[j]);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&newest_s, top);
    __syncthreads();
    const int64_t newest = newest_s;
    uint32_t prefix = 0u;
    int want = budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
      const uint32_t hmask = shift == 24 ? 0u : (0xFFFFFFFFu << (shift + 8));
      for (int j = threadIdx.x; j < len; j += kEvictThreads) {
        const uint32_t key = evict_key(mass[j], pos[j], sink, newest, recent);
        if ((key & hmask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {
        unsigned int cnt[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) { cnt[e] = hist[255 - 8 * lane - e]; sum += cnt[e]; }
        unsigned int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        unsigned int run = incl - sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (run < (unsigned)want && run + cnt[e] >= (unsigned)want) {
            prefix_s = prefix | ((uint32_t)(255 - 8 * lane - e) << shift);
            need_s = want - (int)run;
          }
          run += cnt[e];
        }
      }
      __syncthreads();
      prefix = prefix_s;
      want = need_s;
      for (int t = threadIdx.x; t < 256; t += kEvictThreads) hist[t] = 0u;
      __syncthreads();
    }
    // kept: above the threshold, and the `want` lowest of the slots at it
    for (int w = warp; w < W; w += kEvictThreads / 32) {
      const int j = w * 32 + lane;
      const uint32_t key = j < len ? evict_key(mass[j], pos[j], sink, newest, recent) : 0u;
      const uint32_t gt = __ballot_sync(0xffffffffu, j < len && key > prefix);
      const uint32_t eq = __ballot_sync(0xffffffffu, j < len && key == prefix);
      if (lane == 0) { kept[w] = gt; tie[w] = eq; }
    }
    __syncthreads();
    scan_words(0, W, rank, warp_tmp, [&](int w) { return __popc(tie[w]); });
    for (int w = threadIdx.x; w < W; w += kEvictThreads) {
      uint32_t bits = tie[w], take = 0u;
      for (int left_over = want - (int)rank[w]; left_over > 0 && bits; --left_over) {
        take |= bits & (0u - bits);
        bits &= bits - 1u;
      }
      kept[w] |= take;
    }
    __syncthreads();
    scan_words(0, wl + 1 < W ? wl + 1 : W, rank, warp_tmp,
               [&](int w) { return __popc(~kept[w] & below_mask(w, left)); });
    const uint32_t first = wl < W ? kept[wl] & ~below_mask(wl, left) : 0u;  // movers of the word `left` is in
    scan_words(wl + 1 < W ? wl + 1 : W, W, rank, warp_tmp, [&](int w) { return __popc(kept[w]); });
    for (int w = wl + 1 + threadIdx.x; w < W; w += kEvictThreads) rank[w] += __popc(first);
    __syncthreads();
  }
  // ---- this CTA's share of the new slots
  for (int base = blockIdx.x * kEvictThreads; base < left; base += gridDim.x * kEvictThreads) {
    if (threadIdx.x == 0) moves_s = 0;
    __syncthreads();
    const int j = base + threadIdx.x;
    if (j < left) {
      int src = j;
      if (len > budget) {
        const int w = j >> 5;
        if (!((kept[w] >> (j & 31)) & 1u)) {
          int r = (int)rank[w] + __popc(~kept[w] & below_mask(w, j));  // this freed slot's rank
          int lo = wl, hi = W - 1;  // the last word with at most r movers before it
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int)rank[mid] <= r) lo = mid; else hi = mid - 1;
          }
          uint32_t bits = kept[lo] & ~below_mask(lo, left);
          if (lo > wl) r -= (int)rank[lo];
          for (; r > 0; --r) bits &= bits - 1u;
          src = lo * 32 + __ffs(bits) - 1;
          if (DD_IN_BOUNDS(bits != 0u && src < len)) {
            moves[atomicAdd(&moves_s, 1)] = make_int2(j, src);
          } else {
            src = j;
          }
        }
      }
      const int64_t at = (int64_t)n * stride;
      mass_out[at + j] = mass[src];
      pos_out[at + j] = pos[src];
      if (src_out) src_out[at + j] = src;
    }
    __syncthreads();
    const int n_moves = moves_s;
    const int32_t* row = c.table + (int64_t)n * c.table_stride;
    const int per = c.Hkv << chunk16_log2;  // 16-byte chunks of a row
    for (int i = warp; i < n_moves; i += kEvictThreads / 32) {
      const int64_t to = slot_offset(c, row, moves[i].x), from = slot_offset(c, row, moves[i].y);
      if (to < 0 || from < 0) continue;
      for (int x = lane; x < per; x += 32) {
        const int64_t off = (int64_t)(x >> chunk16_log2) * c.head_bytes +
                            (int64_t)(x & ((1 << chunk16_log2) - 1)) * 16;
        const uint4 kx = *reinterpret_cast<const uint4*>(c.k + from + off);
        const uint4 vx = *reinterpret_cast<const uint4*>(c.v + from + off);
        *reinterpret_cast<uint4*>(c.k + to + off) = kx;
        *reinterpret_cast<uint4*>(c.v + to + off) = vx;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ beams
struct RowStates {
  dd_row_state s[kMaxRowStates];
  int unit[kMaxRowStates];  // bytes copied at a time: 16, 4 or 1
};

__device__ __forceinline__ int parent_row(const int32_t* parent, int n, int K) {
  const int b = n / K, p = parent[n];
  return b * K + (p >= 0 && p < K ? p : n - b * K);
}

constexpr int kCopyThreads = 128;

template <typename U>
__device__ __forceinline__ void copy_units(char* dst, const char* src, int64_t bytes, int64_t first,
                                           int64_t step) {
  const U* s = reinterpret_cast<const U*>(src);
  U* d = reinterpret_cast<U*>(dst);
  const int64_t units = bytes / (int64_t)sizeof(U);
#pragma unroll 4
  for (int64_t i = first; i < units; i += step) d[i] = s[i];
}

// Grid (rows, states, parts of a row).
__global__ void __launch_bounds__(kCopyThreads)
beam_reorder_kernel(const int32_t* __restrict__ parent, int K,
                    const __grid_constant__ RowStates st) {
  pdl_wait();
  const dd_row_state& s = st.s[blockIdx.y];
  const int n = blockIdx.x, p = parent_row(parent, n, K);
  const char* src = static_cast<const char*>(s.src) + (int64_t)p * s.src_stride;
  char* dst = static_cast<char*>(s.dst) + (int64_t)n * s.dst_stride;
  const int64_t first = (int64_t)blockIdx.z * kCopyThreads + threadIdx.x;
  const int64_t step = (int64_t)gridDim.z * kCopyThreads;
  const int unit = st.unit[blockIdx.y];
  if (unit == 16) copy_units<uint4>(dst, src, s.row_bytes, first, step);
  else if (unit == 4) copy_units<uint32_t>(dst, src, s.row_bytes, first, step);
  else copy_units<uint8_t>(dst, src, s.row_bytes, first, step);
}

// Grid (beams, layers, parts of a page).
__global__ void __launch_bounds__(kCopyThreads)
paged_fork_kernel(PagedView c, const int32_t* __restrict__ parent, int K,
                  const int32_t* __restrict__ lengths, const int32_t* __restrict__ fresh,
                  int32_t* __restrict__ table_out, int64_t out_stride,
                  int32_t* __restrict__ lengths_out, int chunk16_log2) {
  pdl_wait();
  const int n = blockIdx.x, p = parent_row(parent, n, K);
  const int len = checked_length(lengths, p, c.cap);
  const int full = div_fast(c.page, len), rest = len - full * c.page.n;
  const int32_t* row = c.table + (int64_t)p * c.table_stride;
  const int old = rest > 0 ? checked_page(row[full], c.n_pages) : -1;
  int fr = -1;
  if (full < c.max_pages && (rest == 0 || old >= 0)) {
    fr = fresh[n];
    if (fr < 0 || fr >= c.n_pages) {
      record_error(DD_ERR_BOUNDS);
      fr = -1;
    }
  }
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    int32_t* out = table_out + (int64_t)n * out_stride;
    for (int i = threadIdx.x; i < full; i += kCopyThreads) out[i] = row[i];
    if (threadIdx.x == 0) {
      if (full < c.max_pages) out[full] = fr;
      lengths_out[n] = len;
    }
  }
  if (fr < 0 || rest == 0) return;
  const int per = c.Hkv << chunk16_log2;
  const int64_t layer = (int64_t)blockIdx.y * c.layer_bytes;
  const int64_t from = layer + (int64_t)old * c.page_bytes, to = layer + (int64_t)fr * c.page_bytes;
  const int64_t units = (int64_t)rest * per;
#pragma unroll 2
  for (int64_t x = (int64_t)blockIdx.z * kCopyThreads + threadIdx.x; x < units;
       x += (int64_t)gridDim.z * kCopyThreads) {
    const int r = (int)(x / per), y = (int)(x - (int64_t)r * per);
    const int64_t off = (int64_t)r * c.token_bytes + (int64_t)(y >> chunk16_log2) * c.head_bytes +
                        (int64_t)(y & ((1 << chunk16_log2) - 1)) * 16;
    const uint4 kx = *reinterpret_cast<const uint4*>(c.k + from + off);
    const uint4 vx = *reinterpret_cast<const uint4*>(c.v + from + off);
    *reinterpret_cast<uint4*>(c.k + to + off) = kx;
    *reinterpret_cast<uint4*>(c.v + to + off) = vx;
  }
}

int chunk_log2(const dd_paged_cache& c) {  // log2 of the 16-byte chunks of a head's row
  const int chunks = c.d * (c.dtype == DD_BF16 ? 2 : 4) / 16;  // 8, 16 or 32
  return chunks == 8 ? 3 : chunks == 16 ? 4 : 5;
}

}  // namespace

cudaError_t launch_cache_evict(const EvictCall& p, cudaStream_t stream) {
  static thread_local int configured_for = -1;
  const DeviceInfo& dev = device_info();
  if (configured_for != dev.device) {
    cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kEvictMaxLen / 32 * 3 * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    configured_for = dev.device;
  }
  const int most = p.budget < p.max_len ? p.budget : p.max_len;
  const int parts = (most + kEvictThreads - 1) / kEvictThreads;
  const int fill = (2 * dev.sm_count + p.N - 1) / p.N;
  const size_t smem = (size_t)((p.max_len + 31) / 32) * 3 * sizeof(uint32_t);
  evict_kernel<<<dim3(parts < fill ? parts : fill, p.N), kEvictThreads, smem, stream>>>(
      make_paged_view(*p.cache), p.lengths, p.max_len, p.budget, p.sink, p.recent, p.mass_in,
      p.pos_in, p.stride, p.mass_out, p.pos_out, p.src_out, p.lengths_out, chunk_log2(*p.cache));
  return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const int32_t* parent, int B, int K, const dd_row_state* states,
                                int n_states, cudaStream_t stream) {
  RowStates st{};
  int64_t longest = 1;
  const int64_t rows = (int64_t)B * K;
  for (int i = 0; i < n_states; ++i) {
    const dd_row_state& s = st.s[i] = states[i];
    uintptr_t bits = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) |
                     (uintptr_t)s.row_bytes;
    if (rows > 1) bits |= (uintptr_t)s.src_stride | (uintptr_t)s.dst_stride;
    st.unit[i] = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
    const int64_t units = s.row_bytes / st.unit[i];
    if (units > longest) longest = units;
  }
  int64_t parts = (longest + kCopyThreads * 16 - 1) / (kCopyThreads * 16);
  if (parts > 64) parts = 64;
  return launch_dependent(beam_reorder_kernel, dim3((unsigned)rows, n_states, (unsigned)parts),
                          dim3(kCopyThreads), 0, stream, parent, K, st);
}

cudaError_t launch_paged_fork(const dd_paged_cache& cache, const int32_t* parent, int B, int K,
                              const int32_t* lengths, const int32_t* fresh, int32_t* table_out,
                              int64_t out_stride, int32_t* lengths_out, cudaStream_t stream) {
  const int lg = chunk_log2(cache);
  const int64_t units = (int64_t)(cache.page_size - 1) * (cache.Hkv << lg);
  int64_t parts = (units + kCopyThreads * 4 - 1) / (kCopyThreads * 4);
  parts = parts < 1 ? 1 : parts > 64 ? 64 : parts;
  return launch_dependent(paged_fork_kernel, dim3(B * K, cache.layers, (unsigned)parts),
                          dim3(kCopyThreads), 0, stream, make_paged_view(cache), parent, K, lengths,
                          fresh, table_out, out_stride, lengths_out, lg);
}

}  // namespace dd
