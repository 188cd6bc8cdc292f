// Eviction from a paged cache by accumulated attention mass (dd_cache_evict), and what
// beams do to caches and states (dd_paged_fork, dd_beam_reorder).
#include <cooperative_groups.h>

#include "dd_paged.cuh"

namespace dd {

namespace {

// Sequences of up to kEvictShort slots are selected by one CTA (whose barriers, with few
// warps, are cheap), longer ones by a cluster.
constexpr int kEvictFew = 256;
constexpr int kEvictRegs = 8;      // slots a thread holds from its first load
constexpr int kEvictShort = kEvictFew * kEvictRegs;
constexpr int kEvictMany = 512;    // threads of a cluster's CTA
constexpr int kCluster = 8;
constexpr int kEvictBins = 2048;
constexpr int kEvictList = 256;    // keys of one bin ranked by counting (their square is the work)

struct EvictArgs {
  PagedView c;
  const int32_t* lengths;
  int max_len, budget, sink, recent;
  const float* mass_in;
  const int32_t* pos_in;
  int64_t stride;
  float* mass_out;
  int32_t *pos_out, *src_out, *lengths_out;
  int chunk16_log2;
  int mover_share;  // cluster: movers' slots kept per CTA
  bool keys_fit;    // cluster: a CTA's keys are in shared memory
};

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

// The bin that holds the want-th key from the top: counts(x) is bin x's count, x < bins.
// Returns the bin; want becomes the rank within it, count its count. `bins` is a multiple
// of the block's threads or below it.
struct Crossing {
  int bin, want, count;
};
template <typename F>
__device__ Crossing find_bin(int bins, int want, int* warp_tmp, int* found, F counts) {
  const int per = (bins + blockDim.x - 1) / blockDim.x;  // at most 8: 2048 bins, 256 threads; 4096, 512
  const int first = (int)threadIdx.x * per;              // counted from the top
  int c[8], sum = 0;
#pragma unroll
  for (int y = 0; y < 8; ++y) {
    c[y] = y < per && first + y < bins ? counts(bins - 1 - first - y) : 0;
    sum += c[y];
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
  int x = lane < (int)(blockDim.x >> 5) ? warp_tmp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  const int before = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
  int run = incl - sum + (warp > 0 ? before : 0);
#pragma unroll
  for (int y = 0; y < 8; ++y) {
    if (run < want && run + c[y] >= want) {
      found[0] = bins - 1 - first - y;
      found[1] = want - run;
      found[2] = c[y];
    }
    run += c[y];
  }
  __syncthreads();
  return Crossing{found[0], found[1], found[2]};
}

// The want-th largest of `count` keys, and how many are equal to it; found as in find_bin.
__device__ Crossing rank_list(const uint32_t* list, int count, int want, int* found) {
  for (int i = threadIdx.x; i < count; i += blockDim.x) {
    const uint32_t key = list[i];
    int above = 0, equal = 0;
    for (int t = 0; t < count; ++t) {
      above += list[t] > key;
      equal += list[t] == key;
    }
    if (above < want && above + equal >= want) {  // the same from each equal key
      found[0] = (int)key;
      found[1] = want - above;
      found[2] = equal;
    }
  }
  __syncthreads();
  return Crossing{found[0], found[1], found[2]};
}

// The `more` lowest bits of `from`.
__device__ __forceinline__ uint32_t lowest_bits(uint32_t from, int more) {
  uint32_t take = 0u;
  for (; more > 0 && from; --more) {
    take |= from & (0u - from);
    from &= from - 1u;
  }
  return take;
}

struct MoveList {
  int64_t to[kEvictMany], from[kEvictMany];
  int n;
};

// New slots [begin, end) of sequence n: mass and position (and origin) of each, and the K and
// V rows of those that came from elsewhere. source(j): the old slot of new slot j.
template <typename F>
__device__ void write_slots(const EvictArgs& a, int n, int begin, int end, MoveList& list, F source) {
  const float* mass = a.mass_in + (int64_t)n * a.stride;
  const int32_t* pos = a.pos_in + (int64_t)n * a.stride;
  const int32_t* row = a.c.table + (int64_t)n * a.c.table_stride;
  const int per = a.c.Hkv << a.chunk16_log2;  // 16-byte chunks of a row
  const int64_t at = (int64_t)n * a.stride;
  const int threads = blockDim.x;
  for (int base = begin; base < end; base += threads) {
    if (threadIdx.x == 0) list.n = 0;
    __syncthreads();
    const int j = base + threadIdx.x;
    if (j < end) {
      const int src = source(j);
      if (src != j) {
        const int64_t to = slot_offset(a.c, row, j), from = slot_offset(a.c, row, src);
        if (to >= 0 && from >= 0) {
          const int i = atomicAdd(&list.n, 1);
          list.to[i] = to;
          list.from[i] = from;
        }
      }
      a.mass_out[at + j] = mass[src];
      a.pos_out[at + j] = pos[src];
      if (a.src_out) a.src_out[at + j] = src;
    }
    __syncthreads();
    // rows that move: K and V, 16 bytes a thread and step
    const int units = list.n * per;
    for (int u = threadIdx.x; u < units; u += 4 * threads) {
      uint4 kx[4], vx[4];
      int64_t to[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = u + e * threads;
        if (x >= units) continue;
        const int i = x / per, y = x - i * per;
        const int64_t off = (int64_t)(y >> a.chunk16_log2) * a.c.head_bytes +
                            (int64_t)(y & ((1 << a.chunk16_log2) - 1)) * 16;
        kx[e] = *reinterpret_cast<const uint4*>(a.c.k + list.from[i] + off);
        vx[e] = *reinterpret_cast<const uint4*>(a.c.v + list.from[i] + off);
        to[e] = list.to[i] + off;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (u + e * threads >= units) continue;
        *reinterpret_cast<uint4*>(a.c.k + to[e]) = kx[e];
        *reinterpret_cast<uint4*>(a.c.v + to[e]) = vx[e];
      }
    }
    __syncthreads();
  }
}

// Up to kEvictShort slots. Grid (CTAs per sequence, sequences): every CTA of a sequence
// repeats the selection, which reads 8 bytes a slot, and does its share of the moves, so
// nothing has to be handed from one CTA to another.
// The budget-th largest key is found by a histogram of its top 11 bits, which leaves a bin
// of keys to rank by counting (a bin of more than kEvictList gets another histogram). Kept
// slots become a bitmap, and the i-th freed slot below the new length takes the i-th kept
// slot at or beyond it: both are ranks over the bitmap (one prefix count per word and a bit
// count). Bound: the latency of its steps: 7.2 us for 16 sequences of 1025 slots of 8 heads of
// 128, one leaving each.
__global__ void __launch_bounds__(kEvictFew)
evict_short_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kWords = kEvictShort / 32;
  __shared__ int hist[kEvictBins];
  __shared__ uint32_t list[kEvictList];
  __shared__ uint32_t keys[kEvictShort];
  __shared__ uint32_t kept[kWords], tie[kWords], rank[kWords];
  __shared__ int warp_tmp[32], found[3];
  __shared__ int newest_s, n_s;
  __shared__ MoveList moves;
  const int n = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = checked_length(a.lengths, n, a.max_len);
  const int left = min(len, a.budget);
  const float* mass = a.mass_in + (int64_t)n * a.stride;
  const int32_t* pos = a.pos_in + (int64_t)n * a.stride;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.lengths_out[n] = left;
  const int W = (len + 31) >> 5, wl = left >> 5;
  int moves_total = 0;
  if (len > a.budget) {
    float m[kEvictRegs];
    int p[kEvictRegs];
#pragma unroll
    for (int e = 0; e < kEvictRegs; ++e) {
      const int j = e * kEvictFew + threadIdx.x;
      m[e] = j < len ? mass[j] : 0.f;
      p[e] = j < len ? pos[j] : INT32_MIN;
    }
    if (threadIdx.x == 0) { newest_s = INT32_MIN; n_s = 0; }
    for (int t = threadIdx.x; t < kEvictBins; t += kEvictFew) hist[t] = 0;
    int top = p[0];
#pragma unroll
    for (int e = 1; e < kEvictRegs; ++e) top = max(top, p[e]);
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (lane == 0) atomicMax(&newest_s, top);
    __syncthreads();
    const int64_t newest = newest_s;
    int safe = 0;
#pragma unroll
    for (int e = 0; e < kEvictRegs; ++e) {
      const int j = e * kEvictFew + threadIdx.x;
      if (j >= len) continue;
      const uint32_t key = evict_key(m[e], p[e], a.sink, newest, a.recent);
      keys[j] = key;
      if (key == 0xFFFFFFFFu) ++safe;
      else atomicAdd(&hist[key >> 21], 1);
    }
    safe = __reduce_add_sync(0xffffffffu, safe);
    if (lane == 0 && safe) atomicAdd(&hist[kEvictBins - 1], safe);
    __syncthreads();
    Crossing x = find_bin(kEvictBins, a.budget, warp_tmp, found, [&](int b) { return hist[b]; });
    uint32_t prefix = (uint32_t)x.bin << 21;
    int bits = 21;
    while (x.count > kEvictList && bits > 0) {
      const uint32_t mask = 0xFFFFFFFFu << bits;
      const int next = bits == 21 ? 10 : 0;
      for (int t = threadIdx.x; t < kEvictBins; t += kEvictFew) hist[t] = 0;
      __syncthreads();
      for (int j = threadIdx.x; j < len; j += kEvictFew)
        if ((keys[j] & mask) == prefix) atomicAdd(&hist[(keys[j] >> next) & (next == 10 ? 2047u : 1023u)], 1);
      __syncthreads();
      x = find_bin(next == 10 ? 2048 : 1024, x.want, warp_tmp, found, [&](int b) { return hist[b]; });
      prefix |= (uint32_t)x.bin << next;
      bits = next;
    }
    if (bits > 0) {
      const uint32_t mask = 0xFFFFFFFFu << bits;
      for (int j = threadIdx.x; j < len; j += kEvictFew)
        if ((keys[j] & mask) == prefix) {
          const int at = atomicAdd(&n_s, 1);
          if (DD_IN_BOUNDS(at < kEvictList)) list[at] = keys[j];
        }
      __syncthreads();
      x = rank_list(list, x.count, x.want, found);
      prefix = (uint32_t)x.bin;
    }
    // ---- kept: above the threshold, and the x.want lowest of the slots at it
    const bool all_ties = x.count == x.want;
    for (int w = warp; w < W; w += kEvictFew / 32) {
      const int j = w * 32 + lane;
      const uint32_t key = j < len ? keys[j] : 0u;
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
      for (int w = threadIdx.x; w < W; w += kEvictFew) kept[w] |= lowest_bits(tie[w], x.want - (int)rank[w]);
      __syncthreads();
    }
    // freed slots lie below `left`, movers at or beyond it; there are as many of each
    moves_total = scan_block(W, rank, warp_tmp, [&](int w) {
      const uint32_t b = below_mask(w, left);
      return __popc((~kept[w] & b) | (kept[w] & ~b));
    }) / 2;
  }
  const int share = ((left + gridDim.x - 1) / gridDim.x + 31) & ~31;
  write_slots(a, n, blockIdx.x * share, min(left, (int)(blockIdx.x + 1) * share), moves, [&](int j) {
    const int w = j >> 5;
    if (moves_total == 0 || ((kept[w] >> (j & 31)) & 1u)) return j;
    // this freed slot's rank among them, and the mover of the same rank: the last word with
    // at most that many movers before it
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
    return DD_IN_BOUNDS(b != 0u && from < len) ? from : j;
  });
}

// Longer sequences: a cluster of 8 CTAs selects, each from an eighth of the slots, with
// histograms, lists and counts summed through distributed shared memory; the movers' slots
// are laid out by rank over the cluster's CTAs, so a freed slot finds its mover in one
// remote read. Grid (8 x clusters per sequence, sequences): where there are few sequences
// several clusters repeat a selection and share the moves.
// Bound: the chain of about ten steps, 2 to 7 K cycles each (7 cluster barriers among them),
// and the rows that move: 16 sequences of up to 8192 slots, 4 heads of 128 bf16, cut to 1024
// (46 MB): 20.0 us; one of 30001 cut to 9999: 20.7 us. A CTA for each sequence took 70 and 115.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kEvictMany)
evict_cluster_kernel(const __grid_constant__ EvictArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t words[];
  constexpr int kBins = 4096;  // 12 bits first, then 10, then 10
  __shared__ int hist[kBins], sums[kBins];  // this CTA's, the cluster's
  __shared__ uint32_t list[kEvictList];
  __shared__ int warp_tmp[32], found[3];
  __shared__ int s_top[kCluster], s_listed, s_ties, s_moves;
  __shared__ MoveList moves;
  uint32_t* all = reinterpret_cast<uint32_t*>(moves.to);  // the cluster's lists, before any move
  static_assert(sizeof(moves.to) >= kEvictList * 4);
  const cg::cluster_group cluster = cg::this_cluster();
  const int n = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = (int)cluster.block_rank();
  const int len = checked_length(a.lengths, n, a.max_len);
  const int left = min(len, a.budget);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.lengths_out[n] = left;
  const int share = ((left + gridDim.x - 1) / gridDim.x + 31) & ~31;
  const int begin = blockIdx.x * share, end = min(left, begin + share);
  if (len <= a.budget) {  // the whole cluster
    write_slots(a, n, begin, end, moves, [](int j) { return j; });
    return;
  }
  const float* mass = a.mass_in + (int64_t)n * a.stride;
  const int32_t* pos = a.pos_in + (int64_t)n * a.stride;
  const int Wc = ((len + 31) / 32 + kCluster - 1) / kCluster;  // words, and slots, of a CTA
  const int j0 = me * Wc * 32, j1 = min(len, j0 + Wc * 32), mine = max(0, j1 - j0);
  uint32_t* kept = words;          // [Wc]
  uint32_t* rank = words + Wc;     // [Wc] freed slots and movers before the word, in this CTA
  uint32_t* mover = words + 2 * Wc;                // [mover_share]
  uint32_t* keys = mover + a.mover_share;          // [Wc * 32], where they fit
  // ---- the newest position
  float m[kEvictRegs];
  int p[kEvictRegs];
  const int step = kEvictRegs * kEvictMany;
  const auto load = [&](int base) {
#pragma unroll
    for (int e = 0; e < kEvictRegs; ++e) {
      const int j = j0 + base + e * kEvictMany + threadIdx.x;
      m[e] = j < j1 ? mass[j] : 0.f;
      p[e] = j < j1 ? pos[j] : INT32_MIN;
    }
  };
  load(0);
  if (threadIdx.x == 0) s_top[me] = INT32_MIN;
  for (int t = threadIdx.x; t < kBins; t += kEvictMany) hist[t] = sums[t] = 0;
  int top = p[0];
#pragma unroll
  for (int e = 1; e < kEvictRegs; ++e) top = max(top, p[e]);
#pragma unroll 8
  for (int j = j0 + step + (int)threadIdx.x; j < j1; j += kEvictMany) top = max(top, pos[j]);
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) atomicMax(&s_top[me], top);
  if (threadIdx.x == 0) s_listed = s_ties = s_moves = 0;
  cluster.sync();
  int64_t newest = INT32_MIN;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) newest = max(newest, (int64_t)*cluster.map_shared_rank(&s_top[c], c));
  // ---- keys and the first histogram
  const auto key_at = [&](int i) {  // i-th slot of this CTA
    return a.keys_fit ? keys[i] : evict_key(mass[j0 + i], pos[j0 + i], a.sink, newest, a.recent);
  };
  int safe = 0;
  for (int base = 0; base < mine; base += step) {
    if (base > 0) load(base);
#pragma unroll
    for (int e = 0; e < kEvictRegs; ++e) {
      const int i = base + e * kEvictMany + threadIdx.x;
      if (i >= mine) continue;
      const uint32_t key = evict_key(m[e], p[e], a.sink, newest, a.recent);
      if (a.keys_fit) keys[i] = key;
      if (key == 0xFFFFFFFFu) ++safe;
      else atomicAdd(&hist[key >> 20], 1);
    }
  }
  safe = __reduce_add_sync(0xffffffffu, safe);
  if (lane == 0 && safe) atomicAdd(&hist[kBins - 1], safe);
  // a CTA adds its bins that hold any (tens of them: masses cluster in a few octaves) to
  // every CTA's sums
  const auto add_up = [&]() {
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kEvictMany) {
      const int k = hist[b];
      if (!k) continue;
#pragma unroll
      for (int c = 0; c < kCluster; ++c) atomicAdd(cluster.map_shared_rank(&sums[b], c), k);
    }
    cluster.sync();
  };
  add_up();
  const auto total = [&](int b) { return sums[b]; };
  Crossing x = find_bin(kBins, a.budget, warp_tmp, found, total);
  uint32_t prefix = (uint32_t)x.bin << 20;
  int bits = 20;
  while (x.count > kEvictList && bits > 0) {  // the same in every CTA
    const uint32_t mask = 0xFFFFFFFFu << bits;
    const int next = bits == 20 ? 10 : 0;
    __syncthreads();
    for (int t = threadIdx.x; t < kBins; t += kEvictMany) hist[t] = sums[t] = 0;
    cluster.sync();  // before anyone adds to these sums
    for (int i = threadIdx.x; i < mine; i += kEvictMany) {
      const uint32_t key = key_at(i);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> next) & 1023u], 1);
    }
    add_up();
    x = find_bin(1024, x.want, warp_tmp, found, total);
    prefix |= (uint32_t)x.bin << next;
    bits = next;
  }
  if (bits > 0) {  // the bin's keys, from every CTA's list into one
    const uint32_t mask = 0xFFFFFFFFu << bits;
    for (int i = threadIdx.x; i < mine; i += kEvictMany) {
      const uint32_t key = key_at(i);
      if ((key & mask) == prefix) {
        const int at = atomicAdd(&s_listed, 1);
        if (DD_IN_BOUNDS(at < kEvictList)) list[at] = key;
      }
    }
    cluster.sync();
    // 64 threads to each CTA's list
    const int c = threadIdx.x / (kEvictMany / kCluster), i0 = threadIdx.x % (kEvictMany / kCluster);
    int at = 0, k = 0;
#pragma unroll
    for (int y = 0; y < kCluster; ++y) {
      const int ky = *cluster.map_shared_rank(&s_listed, y);
      if (y < c) at += ky;
      if (y == c) k = ky;
    }
    const uint32_t* from = cluster.map_shared_rank(list, c);
    for (int i = i0; i < k; i += kEvictMany / kCluster)
      if (DD_IN_BOUNDS(at + i < kEvictList)) all[at + i] = from[i];
    __syncthreads();
    x = rank_list(all, min(x.count, kEvictList), x.want, found);
    prefix = (uint32_t)x.bin;
  }
  // ---- kept: above the threshold, and the x.want lowest of the slots at it
  const bool all_ties = x.count == x.want;
  int ties = 0;
  for (int w = warp; w < Wc; w += kEvictMany / 32) {
    const int i = w * 32 + lane;
    const uint32_t key = i < mine ? key_at(i) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, i < mine && key > prefix);
    const uint32_t eq = __ballot_sync(0xffffffffu, i < mine && key == prefix);
    if (lane == 0) {
      kept[w] = all_ties ? gt | eq : gt;
      rank[w] = eq;  // until it is known which of them stay
      ties += __popc(eq);
    }
  }
  if (lane == 0 && ties) atomicAdd(&s_ties, ties);
  if (!all_ties) {
    cluster.sync();
    int want = x.want;
    for (int c = 0; c < me; ++c) want -= *cluster.map_shared_rank(&s_ties, c);
    // ranks of the ties in this CTA: the bitmap is read before its prefix count is written
    const int per = (Wc + kEvictMany - 1) / kEvictMany;
    const int w0 = min(Wc, (int)threadIdx.x * per), w1 = min(Wc, w0 + per);
    int sum = 0;
    for (int w = w0; w < w1; ++w) sum += __popc(rank[w]);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) warp_tmp[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += warp_tmp[w];
    for (int w = w0; w < w1; ++w) {
      const uint32_t eq = rank[w];
      kept[w] |= lowest_bits(eq, want - run);
      run += __popc(eq);
    }
  }
  __syncthreads();
  // ---- ranks of freed slots (below `left`) and movers (at or beyond it)
  const int word0 = me * Wc;
  const int here = scan_block(Wc, rank, warp_tmp, [&](int w) {
    const uint32_t b = below_mask(word0 + w, left);
    return __popc((~kept[w] & b) | (kept[w] & ~b));
  });
  if (threadIdx.x == 0) s_moves = here;
  cluster.sync();
  int before = 0, both = 0;
  int counts[kCluster];
#pragma unroll
  for (int c = 0; c < kCluster; ++c) counts[c] = *cluster.map_shared_rank(&s_moves, c);
#pragma unroll
  for (int c = 0; c < kCluster; ++c) {
    if (c < me) before += counts[c];
    both += counts[c];
  }
  const int moves_total = both / 2;
  // ---- movers by rank
  const int wl = left >> 5;
  for (int w = threadIdx.x; w < Wc; w += kEvictMany) {
    uint32_t b = kept[w] & ~below_mask(word0 + w, left);
    if (!b) continue;
    int r = word0 + w > wl ? before + (int)rank[w] - moves_total : 0;
    int c = r / a.mover_share, at = r - c * a.mover_share;
    for (; b; b &= b - 1u) {
      if (DD_IN_BOUNDS(r >= 0 && c < kCluster))
        cluster.map_shared_rank(mover, c)[at] = (uint32_t)((word0 + w) * 32 + __ffs(b) - 1);
      if (++at == a.mover_share) {
        at = 0;
        ++c;
      }
    }
  }
  cluster.sync();
  // freed slots before the first word of each CTA
  int first[kCluster];
#pragma unroll
  for (int c = 0, sum = 0; c < kCluster; ++c) {
    first[c] = sum;
    sum += counts[c];
  }
  write_slots(a, n, begin, end, moves, [&](int j) {
    const int w = j >> 5, c = w / Wc, i = w - c * Wc;
    const uint32_t k = cluster.map_shared_rank(kept, c)[i];
    if ((k >> (j & 31)) & 1u) return j;
    int r = (int)cluster.map_shared_rank(rank, c)[i] + __popc(~k & below_mask(w, j));
#pragma unroll
    for (int y = 0; y < kCluster; ++y)
      if (y == c) r += first[y];
    const int o = r / a.mover_share;
    return DD_IN_BOUNDS(o < kCluster) ? (int)cluster.map_shared_rank(mover, o)[r - o * a.mover_share] : j;
  });
  cluster.sync();  // no CTA leaves while another reads its shared memory
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

// Grid (rows, states, parts of a row). Bound: latency (3 us); HBM for large states.
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

// Grid (beams, layers, parts of a page). Bound: HBM, the copied rows read and written (512
// beams, two layers, pages of 32 slots of 8 heads of 128: 130 MB in 18 us, part of it from L2).
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
  const DeviceInfo& dev = device_info();
  EvictArgs a{};
  a.c = make_paged_view(*p.cache);
  a.lengths = p.lengths;
  a.max_len = p.max_len; a.budget = p.budget; a.sink = p.sink; a.recent = p.recent;
  a.mass_in = p.mass_in; a.pos_in = p.pos_in; a.stride = p.stride;
  a.mass_out = p.mass_out; a.pos_out = p.pos_out; a.src_out = p.src_out; a.lengths_out = p.lengths_out;
  a.chunk16_log2 = chunk_log2(*p.cache);
  const int most = p.budget < p.max_len ? p.budget : p.max_len;
  const int movers = most < p.max_len - most ? most : p.max_len - most;
  if (p.max_len <= kEvictShort) {
    // CTAs per sequence: one per 32 rows that may move, until the GPU is full
    const int parts = (movers + 31) / 32 > 1 ? (movers + 31) / 32 : 1;
    const int fill = (2 * dev.sm_count + p.N - 1) / p.N;
    evict_short_kernel<<<dim3(parts < fill ? parts : fill, p.N), kEvictFew, 0, stream>>>(a);
    return cudaGetLastError();
  }
  static thread_local int configured_for = -1, resident = 1;  // clusters at once, one CTA an SM
  constexpr int kDynamic = 168 * 1024;
  if (configured_for != dev.device) {
    cudaError_t e = cudaFuncSetAttribute(evict_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamic);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kEvictMany);
    cfg.dynamicSmemBytes = kDynamic;
    e = cudaOccupancyMaxActiveClusters(&resident, evict_cluster_kernel, &cfg);
    if (e != cudaSuccess) return e;
    configured_for = dev.device;
  }
  const int Wc = ((p.max_len + 31) / 32 + kCluster - 1) / kCluster;
  a.mover_share = (movers + kCluster - 1) / kCluster > 1 ? (movers + kCluster - 1) / kCluster : 1;
  size_t smem = ((size_t)2 * Wc + a.mover_share) * 4;
  a.keys_fit = smem + (size_t)Wc * 32 * 4 <= (size_t)kDynamic;
  if (a.keys_fit) smem += (size_t)Wc * 32 * 4;
  // clusters per sequence: one per 256 rows that may move, as long as all of them run at
  // once (a second round of clusters doubles the time of the selection)
  const int parts = (movers + 255) / 256 > 1 ? (movers + 255) / 256 : 1;
  const int fill = resident / p.N > 1 ? resident / p.N : 1;
  evict_cluster_kernel<<<dim3(kCluster * (parts < fill ? parts : fill), p.N), kEvictMany, smem, stream>>>(a);
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
