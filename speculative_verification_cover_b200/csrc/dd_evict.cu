// Eviction from a paged cache by accumulated attention mass (dd_cache_evict), and what
// beams do to caches and states (dd_paged_fork, dd_beam_reorder).
#include "dd_paged.cuh"

namespace dd {

namespace {

// Threads of a CTA: for short sequences the barriers of fewer warps are cheaper.
constexpr int kEvictFew = 256, kEvictMany = 1024;
constexpr int kEvictRegs = 8;      // slots a thread holds from its first load
constexpr int kEvictKeySlots = 45056;  // slots whose keys fit shared memory (176 KB)
constexpr int kEvictBins = 2048;
constexpr int kEvictList = 1024;   // keys of one bin ranked by counting

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

// Exclusive prefix sums of f(0) .. f(n - 1) into out; returns the total. out may be what f
// reads.
template <typename F>
__device__ int scan_block(int n, uint32_t* out, int* warp_tmp, F f) {
  const int chunk = (n + blockDim.x - 1) / blockDim.x;
  const int a = min(n, (int)threadIdx.x * chunk), e = min(n, a + chunk);
  int sum = 0;
  for (int w = a; w < e; ++w) sum += f(w);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) warp_tmp[warp] = incl;
  __syncthreads();
  int x = lane < warps ? warp_tmp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  const int total = __shfl_sync(0xffffffffu, x, 31);
  const int before = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
  int run = incl - sum + (warp > 0 ? before : 0);
  for (int w = a; w < e; ++w) {
    const int c = f(w);
    out[w] = (uint32_t)run;
    run += c;
  }
  __syncthreads();
  return total;
}

// Grid (CTAs per sequence, sequences). The selection reads 8 bytes a slot; every CTA of a
// sequence repeats it (the repeats come from L2) and then does its share of the moves, so
// nothing has to be handed from one CTA to another.
// The budget-th largest key is found by histograms of 11 bits; the first leaves, with
// attention masses, a bin of few keys, which are ranked by counting (a bin of more than
// kEvictList keys gets another histogram). Kept slots become a bitmap, and the i-th freed
// slot below the new length takes the i-th kept slot at or beyond it: both are ranks over
// the bitmap (one prefix count per word and a bit count).
__global__ void __launch_bounds__(kEvictMany)
evict_kernel(PagedView c, const int32_t* __restrict__ lengths, int max_len, int budget, int sink,
             int recent, const float* __restrict__ mass_in, const int32_t* __restrict__ pos_in,
             int64_t stride, float* __restrict__ mass_out, int32_t* __restrict__ pos_out,
             int32_t* __restrict__ src_out, int32_t* __restrict__ lengths_out, int chunk16_log2,
             bool keys_fit) {
  extern __shared__ uint32_t words[];
  __shared__ int hist[kEvictBins];
  __shared__ uint32_t list[kEvictList];
  __shared__ int warp_tmp[32];
  __shared__ uint32_t prefix_s;
  __shared__ int want_s, ties_s, newest_s, n_s;
  __shared__ int64_t s_to[kEvictMany], s_from[kEvictMany];
  const int n = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = blockDim.x;
  const int len = checked_length(lengths, n, max_len);
  const int left = min(len, budget);
  const float* mass = mass_in + (int64_t)n * stride;
  const int32_t* pos = pos_in + (int64_t)n * stride;
  if (blockIdx.x == 0 && threadIdx.x == 0) lengths_out[n] = left;
  const int W = (len + 31) >> 5, wl = left >> 5;
  uint32_t* kept = words;          // [W] bitmap
  uint32_t* rank = words + W;      // [W] freed slots and movers before word w
  uint32_t* tie = words + 2 * W;   // [W] bitmap of slots at the threshold
  uint32_t* keys = words + 3 * W;  // [len], where they fit
  int moves_total = 0;
  if (len > budget) {
    // ---- keys
    if (threadIdx.x == 0) newest_s = INT32_MIN;
    for (int t = threadIdx.x; t < kEvictBins; t += threads) hist[t] = 0;
    float m[kEvictRegs];
    int p[kEvictRegs];
    const auto load = [&](int base) {
#pragma unroll
      for (int e = 0; e < kEvictRegs; ++e) {
        const int j = base + e * threads + threadIdx.x;
        m[e] = j < len ? mass[j] : 0.f;
        p[e] = j < len ? pos[j] : INT32_MIN;
      }
    };
    const int step = kEvictRegs * threads;
    load(0);
    int top = p[0];
#pragma unroll
    for (int e = 1; e < kEvictRegs; ++e) top = max(top, p[e]);
    for (int base = step; base < len; base += step) {
      int q[kEvictRegs];
#pragma unroll
      for (int e = 0; e < kEvictRegs; ++e) {
        const int j = base + e * threads + threadIdx.x;
        q[e] = j < len ? pos[j] : INT32_MIN;
      }
#pragma unroll
      for (int e = 0; e < kEvictRegs; ++e) top = max(top, q[e]);
    }
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&newest_s, top);
    __syncthreads();
    const int64_t newest = newest_s;
    const auto key_at = [&](int j) {
      return keys_fit ? keys[j] : evict_key(mass[j], pos[j], sink, newest, recent);
    };
    // first histogram (the top 11 bits) as the keys are formed
    int safe = 0;
    for (int base = 0; base < len; base += step) {
      if (base > 0) load(base);
#pragma unroll
      for (int e = 0; e < kEvictRegs; ++e) {
        const int j = base + e * threads + threadIdx.x;
        if (j >= len) continue;
        const uint32_t key = evict_key(m[e], p[e], sink, newest, recent);
        if (keys_fit) keys[j] = key;
        if (key == 0xFFFFFFFFu) ++safe;
        else atomicAdd(&hist[key >> 21], 1);
      }
    }
    safe = __reduce_add_sync(0xffffffffu, safe);
    if (lane == 0 && safe) atomicAdd(&hist[kEvictBins - 1], safe);
    __syncthreads();
    uint32_t prefix = 0u;  // bits of the threshold found so far
    int want = budget, bits = 21;
    while (true) {
      // the bin, from the top, that the want-th largest key falls into
      const int bins = bits == 21 || bits == 10 ? kEvictBins : 1024;
      int count = 0;
      {
        // thread t holds bins from the top: bins - 1 - t * per ...
        const int per = (bins + threads - 1) / threads;
        const int b0 = (int)threadIdx.x * per, b1 = min(bins, b0 + per);
        int sum = 0;
        for (int x = b0; x < b1; ++x) sum += hist[bins - 1 - x];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        if (lane == 31) warp_tmp[warp] = incl;
        __syncthreads();
        int x = lane < (threads >> 5) ? warp_tmp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += t;
        }
        const int before = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
        int run = incl - sum + (warp > 0 ? before : 0);
        if (run < want && run + sum >= want)
          for (int y = b0; y < b1; ++y) {
            const int h = hist[bins - 1 - y];
            if (run < want && run + h >= want) {
              prefix_s = prefix | ((uint32_t)(bins - 1 - y) << bits);
              want_s = want - run;
              ties_s = h;
            }
            run += h;
          }
        if (threadIdx.x == 0) n_s = 0;
        __syncthreads();
        prefix = prefix_s;
        want = want_s;
        count = ties_s;
      }
      const uint32_t mask = bits == 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << bits;
      if (bits == 0 || count <= kEvictList) {
        if (bits > 0) {  // rank the bin's keys
          for (int j = threadIdx.x; j < len; j += threads) {
            const uint32_t key = key_at(j);
            if ((key & mask) == prefix) {
              const int at = atomicAdd(&n_s, 1);
              if (DD_IN_BOUNDS(at < kEvictList)) list[at] = key;
            }
          }
          __syncthreads();
          for (int i = threadIdx.x; i < count; i += threads) {
            const uint32_t key = list[i];
            int above = 0, equal = 0;
            for (int t = 0; t < count; ++t) {
              above += list[t] > key;
              equal += list[t] == key;
            }
            if (above < want && above + equal >= want) {  // the same from each equal key
              prefix_s = key;
              want_s = want - above;
              ties_s = equal;
            }
          }
          __syncthreads();
          prefix = prefix_s;
          want = want_s;
        }
        break;
      }
      // another 11 (then 10) bits
      const int next = bits == 21 ? 10 : 0;
      for (int t = threadIdx.x; t < kEvictBins; t += threads) hist[t] = 0;
      __syncthreads();
      for (int j = threadIdx.x; j < len; j += threads) {
        const uint32_t key = key_at(j);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> next) & (next == 10 ? 2047u : 1023u)], 1);
      }
      bits = next;
      __syncthreads();
    }
    const bool all_ties = ties_s == want;
    // ---- kept: above the threshold, and the `want` lowest of the slots at it
    for (int w = warp; w < W; w += threads >> 5) {
      const int j = w * 32 + lane;
      const uint32_t key = j < len ? key_at(j) : 0u;
      const uint32_t gt = __ballot_sync(0xffffffffu, j < len && key > prefix);
      const uint32_t eq = __ballot_sync(0xffffffffu, j < len && key == prefix);
      if (lane == 0) {
        kept[w] = all_ties ? gt | eq : gt;
        tie[w] = eq;
      }
    }
    __syncthreads();
    if (!all_ties) {
      scan_block(W, rank, warp_tmp, [&](int w) { return __popc(tie[w]); });
      for (int w = threadIdx.x; w < W; w += threads) {
        uint32_t from = tie[w], take = 0u;
        for (int more = want - (int)rank[w]; more > 0 && from; --more) {
          take |= from & (0u - from);
          from &= from - 1u;
        }
        kept[w] |= take;
      }
      __syncthreads();
    }
    // freed slots lie below `left`, movers at or beyond it; there are as many of each
    moves_total = scan_block(W, rank, warp_tmp, [&](int w) {
      const uint32_t b = below_mask(w, left);
      return __popc((~kept[w] & b) | (kept[w] & ~b));
    }) / 2;
  }
  // ---- this CTA's share of the new slots
  const int share = ((left + gridDim.x - 1) / gridDim.x + 31) & ~31;
  const int end = min(left, (int)(blockIdx.x + 1) * share);
  const int32_t* row = c.table + (int64_t)n * c.table_stride;
  const int per = c.Hkv << chunk16_log2;  // 16-byte chunks of a row
  const int64_t at = (int64_t)n * stride;
  for (int base = blockIdx.x * share; base < end; base += threads) {
    if (threadIdx.x == 0) n_s = 0;
    __syncthreads();
    const int j = base + threadIdx.x;
    if (j < end) {
      int src = j;
      if (moves_total > 0) {
        const int w = j >> 5;
        if (!((kept[w] >> (j & 31)) & 1u)) {
          // this freed slot's rank among them, and the mover of the same rank: the last word
          // with at most that many movers before it
          int r = (int)rank[w] + __popc(~kept[w] & below_mask(w, j));
          int lo = wl, hi = W - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int)rank[mid] - moves_total <= r) lo = mid; else hi = mid - 1;
          }
          uint32_t b = kept[lo] & ~below_mask(lo, left);
          if (lo > wl) r -= (int)rank[lo] - moves_total;
          for (; r > 0; --r) b &= b - 1u;
          const int from = lo * 32 + __ffs(b) - 1;
          if (DD_IN_BOUNDS(b != 0u && from < len)) {
            src = from;
            const int64_t ot = slot_offset(c, row, j), of = slot_offset(c, row, src);
            if (ot >= 0 && of >= 0) {
              const int i = atomicAdd(&n_s, 1);
              s_to[i] = ot;
              s_from[i] = of;
            }
          }
        }
      }
      mass_out[at + j] = mass[src];
      pos_out[at + j] = pos[src];
      if (src_out) src_out[at + j] = src;
    }
    __syncthreads();
    // rows that move: K and V, 16 bytes a thread and step
    const int units = n_s * per;
    for (int u = threadIdx.x; u < units; u += 4 * threads) {
      uint4 kx[4], vx[4];
      int64_t to[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = u + e * threads;
        if (x >= units) continue;
        const int i = x / per, y = x - i * per;
        const int64_t off = (int64_t)(y >> chunk16_log2) * c.head_bytes +
                            (int64_t)(y & ((1 << chunk16_log2) - 1)) * 16;
        kx[e] = *reinterpret_cast<const uint4*>(c.k + s_from[i] + off);
        vx[e] = *reinterpret_cast<const uint4*>(c.v + s_from[i] + off);
        to[e] = s_to[i] + off;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (u + e * threads >= units) continue;
        *reinterpret_cast<uint4*>(c.k + to[e]) = kx[e];
        *reinterpret_cast<uint4*>(c.v + to[e]) = vx[e];
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
  constexpr int kBitmaps = kEvictMaxLen / 32 * 3 * 4;
  constexpr int kWithKeys = kEvictKeySlots * 4 + (kEvictKeySlots + 31) / 32 * 3 * 4;
  if (configured_for != dev.device) {
    cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBitmaps > kWithKeys ? kBitmaps : kWithKeys);
    if (e != cudaSuccess) return e;
    configured_for = dev.device;
  }
  const int threads = p.max_len <= kEvictFew * kEvictRegs ? kEvictFew : kEvictMany;
  const bool keys_fit = p.max_len <= kEvictKeySlots;
  const size_t smem = (size_t)((p.max_len + 31) / 32) * 3 * 4 + (keys_fit ? (size_t)p.max_len * 4 : 0);
  // CTAs per sequence: one per 32 rows that may move, and per 8192 slots that stay, until
  // the GPU is full
  const int most = p.budget < p.max_len ? p.budget : p.max_len;
  const int movers = most < p.max_len - most ? most : p.max_len - most;
  const int parts = (movers + 31) / 32 > (most + 8191) / 8192 ? (movers + 31) / 32 : (most + 8191) / 8192;
  const int fill = (2 * dev.sm_count + p.N - 1) / p.N;
  evict_kernel<<<dim3(parts < fill ? parts : fill, p.N), threads, smem, stream>>>(
      make_paged_view(*p.cache), p.lengths, p.max_len, p.budget, p.sink, p.recent, p.mass_in,
      p.pos_in, p.stride, p.mass_out, p.pos_out, p.src_out, p.lengths_out, chunk_log2(*p.cache),
      keys_fit);
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
