// Attention of one new token per sequence over a paged K/V cache (dd_paged_attention).
//
// With s_hj = scale q_h . k_j over the slots j of a sequence, the softmax over any
// partition of the slots is joined from each part's maximum m, sum l = sum e^{s - m}
// and o = sum e^{s - m} v: m' = max m_i, l' = sum l_i e^{m_i - m'}, o' likewise.
//
// Work decomposition. The unit is a tile of 64 slots (32 of 128 fp32 elements) of one (sequence, kv head, block of
// query heads); the tiles of all of them form one index space, cut into equal contiguous
// ranges, one per CTA. So ragged batches, one long sequence and many short ones all
// spread evenly, and a range crosses at most from the end of one sequence-head through
// whole ones into the start of another: whole ones are finished in place, and at most
// two partial results per CTA are left in the workspace for the join kernel.
// Lengths are read on the device (a captured call follows them); only the launch
// depends on max_len.
//
// Bound: HBM, 2 Hkv d elements per slot read once. Measured (one B200, calls in a graph; of
// the copy bandwidth): one sequence of 131071 slots, 8 kv heads of 128 bf16, 86.9 us (95%); 64
// sequences of 17 to 8191, 4 kv heads, with masses, 110.4 us (75%; the scores' way to the join
// and back is 58 of 600 MB); 7 of 101 to 2047, 32 kv heads, 26.5 us (71%): there the first
// lengths, page ids and slots arriving, and the ends of sequence-heads, are a third of it.
#include <cooperative_groups.h>

#include <algorithm>

#include "dd_paged.cuh"
#include "dd_tc.cuh"

namespace dd {

namespace {

constexpr int kTileBytes = 32768;  // K and V of a tile of one head, at most
constexpr int kTileSlots = 64;     // slots of a tile (32 where a row has 512 bytes)
constexpr int kPagedThreads = 128;
constexpr int kPagedWarps = kPagedThreads / 32;
constexpr int kMaxPagedGrid = 1024;  // bounds the workspace on any device
constexpr int kMaxHeads = 16;    // query heads of one block at most
constexpr int kWholeLen = 512;   // sequences up to here are not split
constexpr int kPairCtas = 8;     // CTAs of a sequence-head's cluster (few short sequences)

// How the tiles are given to CTAs: equal ranges, joined by a second kernel; whole
// sequence-heads; or a cluster of CTAs for each.
enum class PagedSplit { kRanges, kWhole, kCluster };

struct PagedArgs {
  PagedView c;
  const char* q;
  const char* k_new;
  const char* v_new;
  int64_t q_bytes, new_bytes;  // sequence strides
  const int32_t* lengths;
  int B, Hq, G, heads, blocks;  // query heads per kv head; per block; blocks per kv head
  int max_len;
  bool even_pages;             // a page holds whole groups of 16 slots
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
  float* scores;               // [B, Hq, row], log2 units (masses only)
  int64_t score_row;           // max_len rounded up to 4
  int grid;
  PagedSplit split;
};

// The tiles of a CTA: [u0, u1).
struct Share {
  int u0, u1;
};
__host__ __device__ constexpr int tile_count(int len, int tile) { return (len + tile - 1) / tile; }

// First tile of every sequence into smem prefix[0 .. B] (and CTA 0: the workspace, for
// the join), and this CTA's share of the tiles.
template <int TILE>
__device__ Share plan_tiles(const PagedArgs& a, int32_t* prefix, int* warp_tmp) {
  const int per_tile = a.c.Hkv * a.blocks;
  const int chunk = (a.B + kPagedThreads - 1) / kPagedThreads;
  const int b0 = min(a.B, (int)threadIdx.x * chunk), b1 = min(a.B, b0 + chunk);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = checked_length(a.lengths, b, a.max_len);
    prefix[b] = sum;
    sum += tile_count(n, TILE) * per_tile;
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
  if (a.split == PagedSplit::kCluster) return Share{0, 0};  // the caller's
  if (a.split == PagedSplit::kWhole) {  // as many sequence-heads a CTA as any other, give or take one
    const int per = a.c.Hkv * a.blocks;
    const auto start = [&](int64_t i) {  // first tile of the first sequence-head of CTA i
      const int64_t p = i * ((int64_t)a.B * per) / a.grid;
      const int b = (int)(p / per);
      return b == a.B ? prefix[b] : prefix[b] + (prefix[b + 1] - prefix[b]) / per * (int)(p - (int64_t)b * per);
    };
    return Share{start(blockIdx.x), start(blockIdx.x + 1)};
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.B; b += kPagedThreads) a.prefix[b] = prefix[b];
  const int64_t total = prefix[a.B], share = (total + a.grid - 1) / a.grid;
  const int64_t u0 = min(total, blockIdx.x * share);
  return Share{(int)u0, (int)min(total, u0 + share)};
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

// ------------------------------------------------------------------ the slots' ring
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The slot of a sequence's new token: its last, or -1 without one (or with a length out of
// range, which is clamped to read by but not to write by).
__device__ __forceinline__ int new_slot(const PagedArgs& a, int b, int len) {
  return a.k_new && a.lengths[b] == len ? len - 1 : -1;
}

// A place in the tile space: tile `tile` of (sequence b, pair = kv head and head block).
template <int TILE>
struct Cursor {
  int b, len, tiles, fresh, pair, tile;  // fresh: the new token's slot
  __device__ __forceinline__ void enter(const PagedArgs& a, int at) {
    b = at;
    len = checked_length(a.lengths, b, a.max_len);
    tiles = tile_count(len, TILE);
    fresh = new_slot(a, b, len);
  }
  __device__ __forceinline__ void seek(const PagedArgs& a, const int32_t* prefix, int u) {
    enter(a, find_sequence(prefix, a.B, u));
    const int rel = u - prefix[b];
    pair = rel / tiles;
    tile = rel - pair * tiles;
  }
  // The next tile; u is its index, below the total.
  __device__ __forceinline__ void next(const PagedArgs& a, const int32_t* prefix, int u) {
    if (++tile < tiles) return;
    tile = 0;
    if (++pair < a.c.Hkv * a.blocks) return;
    pair = 0;
    int n = b + 1;
    while (prefix[n + 1] <= u) ++n;  // sequences without slots
    enter(a, n);
  }
};

// A warp's slots, SLOTS of each tile of its CTA's range, through S stages of shared memory
// (cp.async; K, then V, a group each), on and on across sequence-heads: warps wait for one
// another only where a sequence-head ends. Rows are swizzled by 16-byte chunks (chunk c of
// row r at c ^ (r % 8)). Page ids are fetched one tile ahead of the copies that need them.
// Slots in holes or behind the end arrive as zeros.
template <int ROW, int SLOTS, int S>
struct SlotRing {
  static constexpr int kTile = kPagedWarps * SLOTS;
  static constexpr int kHalf = SLOTS * ROW;  // K, or V, of one stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kBytes = kPagedWarps * S * kStage;
  static constexpr int CH = ROW / 16;        // chunks of a row
  static constexpr int RPI = 32 / CH;        // rows a warp copies per instruction
  static_assert(S * SLOTS <= 64 && kTile * ROW * 2 <= kTileBytes);

  const PagedArgs& a;
  const int32_t* prefix;
  int64_t* new_at;  // [S] where a stage's new token goes
  uint32_t ring;
  int lane, warp, lu, u_end, id;
  uint64_t held_q;  // SLOTS bits per stage: slots that count
  Cursor<kTile> lc;  // the tile whose page ids are held

  __device__ __forceinline__ SlotRing(const PagedArgs& args, const int32_t* pre, uint8_t* smem, int64_t* s_new,
                                      int u0, int u1)
      : a(args), prefix(pre), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), lu(u0), u_end(u1), id(-1), held_q(0) {
    new_at = s_new + warp * S;
    ring = smem_u32(smem) + warp * (S * kStage);
    if (u0 < u1) {
      lc.seek(a, prefix, u0);
      fetch_id();
    }
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s);
  }
  __device__ __forceinline__ int slot() const { return lc.tile * kTile + warp * SLOTS + lane % SLOTS; }
  __device__ __forceinline__ void fetch_id() {
    id = slot() < lc.len ? a.c.table[(int64_t)lc.b * a.c.table_stride + div_fast(a.c.page, slot())] : -1;
  }
  // The queries of a sequence-head are read when its tiles come up: into L2 before that.
  __device__ __forceinline__ void prefetch_q() const {
    const int kvh = lc.pair / a.blocks, blk = lc.pair - kvh * a.blocks;
    const char* q = a.q + (int64_t)lc.b * a.q_bytes + (int64_t)(kvh * a.G + blk * a.heads) * ROW;
    for (int x = lane; x < min(a.heads, a.G - blk * a.heads) * (ROW / 128); x += 32) prefetch_l2(q + x * 128);
  }
  // Whether slot r of a stage counts.
  __device__ __forceinline__ uint32_t held(int stage) const {
    return (uint32_t)(held_q >> (SLOTS * stage)) & ((1u << SLOTS) - 1u);
  }
  __device__ __forceinline__ uint32_t k_at(int stage) const { return ring + stage * kStage; }
  __device__ __forceinline__ uint32_t v_at(int stage) const { return ring + stage * kStage + kHalf; }
  static __device__ __forceinline__ uint32_t chunk(int r, int c) { return r * ROW + ((c ^ (r & 7)) << 4); }

  // Start the copies of the next tile (or of nothing: empty groups keep the count).
  __device__ __forceinline__ void issue(int stage) {
    if (lu >= u_end) {
      cp_async_commit();
      cp_async_commit();
      return;
    }
    constexpr uint32_t kAll = (1u << SLOTS) - 1u;
    const int j = slot(), kvh = lc.pair / a.blocks;
    const int page = checked_page(id, a.c.n_pages);
    const bool ok = page >= 0;  // j < len is in the id
    int64_t off = 0;
    if (ok)
      off = (int64_t)page * a.c.page_bytes + (int64_t)kvh * a.c.head_bytes +
            (int64_t)(j - div_fast(a.c.page, j) * a.c.page.n) * a.c.token_bytes;
    const uint32_t rows = __ballot_sync(0xffffffffu, ok) & kAll;
    const uint32_t fresh = __ballot_sync(0xffffffffu, ok && j == lc.fresh) & kAll;
    held_q = (held_q & ~((uint64_t)kAll << (SLOTS * stage))) | ((uint64_t)rows << (SLOTS * stage));
    if ((fresh >> (lane % SLOTS)) & 1u) new_at[stage] = off;  // the slot's lanes: the same
    const uint32_t dst = k_at(stage);
    const int c = lane % CH, r0 = lane / CH;
    if (a.even_pages && !fresh) {  // the rows are of one page: one address and a stride
      const int64_t o = __shfl_sync(0xffffffffu, off, 0) + r0 * a.c.token_bytes + c * 16;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const char* src = (kv ? a.c.v : a.c.k) + o;
#pragma unroll
        for (int i = 0; i < SLOTS / RPI; ++i) {
          const int r = i * RPI + r0;
          cp_async16(dst + kv * kHalf + chunk(r, c), src, (rows >> r) & 1u ? 16 : 0);
          src += RPI * a.c.token_bytes;
        }
        cp_async_commit();
      }
    } else {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const char* base = kv ? a.c.v : a.c.k;
#pragma unroll
        for (int i = 0; i < SLOTS / RPI; ++i) {
          const int r = i * RPI + r0;
          const char* src = base + __shfl_sync(0xffffffffu, off, r);
          if ((fresh >> r) & 1u)  // the new token: read from the caller
            src = (kv ? a.v_new : a.k_new) + (int64_t)lc.b * a.new_bytes + kvh * ROW;
          cp_async16(dst + kv * kHalf + chunk(r, c), src + c * 16, (rows >> r) & 1u ? 16 : 0);
        }
        cp_async_commit();
      }
    }
    if (++lu < u_end) {
      lc.next(a, prefix, lu);
      fetch_id();
      if (lc.tile == 0 && warp == 0) prefetch_q();
    }
  }
  // The new token, from its row of a stage, into the cache.
  __device__ __forceinline__ void keep_new(int stage, int r) const {
    const int64_t to = new_at[stage] + (lane % CH) * 16;
    if (lane >= CH) return;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4 w;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "r"(k_at(stage) + kv * kHalf + chunk(r, lane % CH)) : "memory");
      *reinterpret_cast<uint4*>((kv ? a.c.v : a.c.k) + to) = w;
    }
  }
};

// ------------------------------------------------------------------ the end of a sequence-head
__device__ __forceinline__ void store4(float* p, const float4& x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16(x.x, x.y), tc::pack_bf16(x.z, x.w));
}
__device__ __forceinline__ void add_scaled(float4& o, const float4& x, float f) {
  o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y);
  o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
}
// Head h's output from its sums.
template <typename T, int D>
__device__ __forceinline__ void write_out(const PagedArgs& a, int64_t h, int e, float m, float l, float4 o) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  store4(reinterpret_cast<T*>(a.out) + h * D + e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (e != 0) return;
  const float z2 = l > 0.f ? m + log2f(l) : -INFINITY;
  if (a.scores) a.lse2[h] = z2;
  if (a.lse) a.lse[h] = z2 * kLn2;
}

// A cluster's CTA results: (m, l) per head and [head][d], where its joined results go.
template <int H>
struct ClusterPart {
  float m[H], l[H];
};

// A piece: the tiles of one sequence-head a CTA has.
struct Piece {
  int b, h0, heads;      // sequence, first query head, heads
  bool starts, whole;    // it has the head's first tile; all of them
};

// Join the four warps' results of up to 8 heads, heads t0 .. of the piece: joined(w) is warp
// w's [8][D], element e of a row at e ^ (8 * (head / 2 % 4)) (which spreads the heads that
// lanes write at once over the banks), s_m / s_l its maxima and sums. Whole sequence-heads
// are written out; a cluster's CTA keeps its part; else it goes to the workspace.
template <typename T, int D, int H, bool CL, typename J>
__device__ __forceinline__ void join_warps(const PagedArgs& a, const Piece& p, int t0, const float (*s_m)[H],
                                           const float (*s_l)[H], J joined, ClusterPart<CL ? H : 1>& part,
                                           float* part_o) {
  const int64_t slot = 2 * (int64_t)blockIdx.x + (p.starts ? 1 : 0);
  for (int i = threadIdx.x; i < min(p.heads - t0, 8) * (D / 4); i += kPagedThreads) {
    const int gt = i / (D / 4), e = (i - gt * (D / 4)) * 4, g = t0 + gt;
    float mm = s_m[0][g];
#pragma unroll
    for (int w = 1; w < kPagedWarps; ++w) mm = fmaxf(mm, s_m[w][g]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) {
      const float f = exp2f(s_m[w][g] - base);
      ll = fmaf(s_l[w][g], f, ll);
      add_scaled(oo, *reinterpret_cast<const float4*>(joined(w) + gt * D + (e ^ (((gt >> 1) & 3) << 3))), f);
    }
    if constexpr (CL) {
      *reinterpret_cast<float4*>(part_o + gt * D + e) = oo;
      if (e == 0) { part.m[g] = mm; part.l[g] = ll; }
    } else if (p.whole) {
      write_out<T, D>(a, (int64_t)p.b * a.Hq + p.h0 + g, e, mm, ll, oo);
    } else if (DD_IN_BOUNDS(slot < 2ll * a.grid)) {
      *reinterpret_cast<float4*>(a.part_o + (slot * a.heads + g) * D + e) = oo;
      if (e == 0) a.part_ml[slot * a.heads + g] = make_float2(mm, ll);
    }
  }
}

// Cluster launches: this CTA's share of a sequence-head's tiles. Returns false where the
// sequence has no slots.
template <int TILE>
__device__ __forceinline__ bool cluster_share(const PagedArgs& a, const int32_t* prefix, int& b, int& pair, Share& share) {
  const int per = a.c.Hkv * a.blocks, p = blockIdx.x / kPairCtas, rank = blockIdx.x - p * kPairCtas;
  b = p / per;
  pair = p - b * per;
  const int tiles = (prefix[b + 1] - prefix[b]) / per;
  const int each = tile_count(tiles, kPairCtas), first = prefix[b] + pair * tiles;
  share = Share{first + min(tiles, rank * each), first + min(tiles, (rank + 1) * each)};
  return tiles > 0;
}
// The cluster's CTAs join their parts, an eighth of the elements each. part_at(g): head g's
// row of the CTA's own shared memory.
template <typename T, int D, int H, typename P>
__device__ __forceinline__ void join_cluster(const PagedArgs& a, int b, int pair, bool has_part, ClusterPart<H>& part,
                                             P part_at) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int kvh = pair / a.blocks, blk = pair - kvh * a.blocks;
  const int h0 = kvh * a.G + blk * a.heads, nh = min(a.heads, a.G - blk * a.heads);
  if (!has_part && threadIdx.x < H) { part.m[threadIdx.x] = -INFINITY; part.l[threadIdx.x] = 0.f; }
  cluster.sync();
  for (int i = (int)cluster.block_rank() * kPagedThreads + threadIdx.x; i < nh * (D / 4); i += kPairCtas * kPagedThreads) {
    const int g = i / (D / 4), e = (i - g * (D / 4)) * 4;
    float mr[kPairCtas], lr[kPairCtas];
    float4 x[kPairCtas];
#pragma unroll
    for (int r = 0; r < kPairCtas; ++r) {
      mr[r] = *cluster.map_shared_rank(&part.m[g], r);
      lr[r] = *cluster.map_shared_rank(&part.l[g], r);
      x[r] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part_at(g) + e, r));
    }
    float mm = mr[0];
#pragma unroll
    for (int r = 1; r < kPairCtas; ++r) mm = fmaxf(mm, mr[r]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kPairCtas; ++r) {
      if (mr[r] == -INFINITY) continue;  // its shared memory may hold no result
      const float f = exp2f(mr[r] - base);
      ll = fmaf(lr[r], f, ll);
      add_scaled(oo, x[r], f);
    }
    write_out<T, D>(a, (int64_t)b * a.Hq + h0 + g, e, mm, ll, oo);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// Shapes of a kernel: slots of a warp's stage (8 KB of K and V, or less), stages, CTAs an SM.
template <typename T, int D, int S_, int CTAS>
struct PagedCfg {
  static constexpr int S = S_, kCtas = CTAS;
  static constexpr int ROW = D * (int)sizeof(T);
  static constexpr int SLOTS = ROW == 512 ? 8 : 16;
  using Ring = SlotRing<ROW, SLOTS, S>;
  static constexpr int kSmem = Ring::kBytes;
  static_assert(8 * D * 4 <= Ring::kHalf);  // a warp's results, in the place of a stage's K
};

// ------------------------------------------------------------------ tensor-core form (bf16)
// Per warp and tile: 16 slots. S^T [16 slots x heads] = K Q^T and O^T [d x heads] += V^T P^T
// as m16n8k16 products whose 16-row operand is the cache (8 heads, or 16 in two column
// tiles, are the narrow side: as the 16-row operand they would waste half of it, and twice
// the instructions). The call is bound by reading K and V, about 23 bytes a cycle and SM,
// which leaves these instructions an idle pipe: a 128-row tcgen05 tile would wait for 128
// slots before its first product, where a warp's 16 slots start as they arrive.
// P is carried as two bf16 terms (16 bits of a weight), so the output has fp32 weights'
// accuracy; one term alone would add as much error again as the output's own rounding.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NT column tiles of 8 query heads. CL: a cluster of kPairCtas CTAs for each sequence-head,
// its tiles split among them, their results joined through distributed shared memory: one
// launch, for few short sequences, where the latency of the call is what counts.
template <typename C, int D, int NT, bool CL>
__global__ void __launch_bounds__(kPagedThreads, C::kCtas)
paged_mma_kernel(const __grid_constant__ PagedArgs a) {
  using Ring = typename C::Ring;
  constexpr int H = NT * 8, KS = D / 16;  // heads, padded; k-steps of S and row tiles of O
  constexpr int S = C::S, ROW = C::ROW;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int warp_tmp[kPagedWarps];
  __shared__ float s_m[kPagedWarps][H], s_l[kPagedWarps][H];
  __shared__ int64_t s_new[kPagedWarps * S];
  __shared__ ClusterPart<CL ? H : 1> part;
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + C::kSmem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  Share share = plan_tiles<Ring::kTile>(a, prefix, warp_tmp);
  write_empty_rows<__nv_bfloat16>(a, prefix, D);
  [[maybe_unused]] int cl_b = 0, cl_pair = 0;
  // a cluster's part goes to the V of the first stages of warps 0 (heads 0 - 7) and 1, which
  // nobody reads any more by then
  const auto part_at = [&](int g) {
    return reinterpret_cast<float*>(smem + (g / 8) * (S * Ring::kStage) + Ring::kHalf) + (g % 8) * D;
  };
  if constexpr (CL) {
    if (!cluster_share<Ring::kTile>(a, prefix, cl_b, cl_pair, share)) return;  // the whole cluster
  } else if (share.u0 >= share.u1) {
    return;
  }
  const int u_end = share.u1;
  Ring ring(a, prefix, smem, s_new, share.u0, u_end);
  Cursor<Ring::kTile> cc;
  if (!CL || share.u0 < u_end) cc.seek(a, prefix, share.u0);
  int stage = 0;
  for (int u = share.u0; u < u_end;) {
    const int b = cc.b, len = cc.len, tiles = cc.tiles, tile0 = cc.tile;
    const int n_tiles = min(tiles - tile0, u_end - u);
    const int kvh = cc.pair / a.blocks, blk = cc.pair - kvh * a.blocks;
    const Piece piece{b, kvh * a.G + blk * a.heads, min(a.heads, a.G - blk * a.heads), tile0 == 0,
                      n_tiles == tiles};
    const int h0 = piece.h0, nh = piece.heads;
    // the tile of this piece, if any, whose slots of this warp hold the new token
    const int new_tile =
        cc.fresh >= 0 && blk == 0 && cc.fresh % Ring::kTile / C::SLOTS == warp ? tiles - 1 - tile0 : -1;
    const int new_row = cc.fresh % C::SLOTS;
    uint32_t q[NT][KS][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = t * 8 + (lane >> 2);
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(
          a.q + (int64_t)b * a.q_bytes + (int64_t)(h0 + min(h, nh - 1)) * ROW) + (lane & 3);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        q[t][k][0] = h < nh ? qp[k * 8] : 0u;
        q[t][k][1] = h < nh ? qp[k * 8 + 4] : 0u;
      }
    }
    float o[KS][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][t][e] = 0.f;
    }
    for (int i = 0; i < n_tiles; ++i) {
      __syncwarp();  // every lane has read the stage that is filled next
      ring.issue(stage == 0 ? S - 1 : stage - 1);
      const uint32_t kb = ring.k_at(stage), vb = ring.v_at(stage);
      const uint32_t held = ring.held(stage);
      cp_async_wait<2 * S - 1>();
      __syncwarp();
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
      const int kr = lane & 15;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t f[4];
        ldsm4(kb + Ring::chunk(kr, 2 * k + (lane >> 4)), f);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(s[t], f, q[t][k][0], q[t][k][1]);
      }
      // rows lane / 4 and + 8; heads 2 (lane % 4) and + 1
      const bool in0 = (held >> (lane >> 2)) & 1u, in1 = (held >> ((lane >> 2) + 8)) & 1u;
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = (e < 2 ? in0 : in1) ? s[t][e] * a.scale2 : -INFINITY;
        if (a.scores) {
          const int j = (tile0 + i) * Ring::kTile + warp * C::SLOTS + (lane >> 2);
          const int g = t * 8 + 2 * (lane & 3);
          float* sp = a.scores + ((int64_t)b * a.Hq + h0 + g) * a.score_row + j;
          if (g < nh && j < len) sp[0] = s[t][0];
          if (g < nh && j + 8 < len) sp[8] = s[t][2];
          if (g + 1 < nh && j < len) sp[a.score_row] = s[t][1];
          if (g + 1 < nh && j + 8 < len) sp[a.score_row + 8] = s[t][3];
        }
        float mx[2] = {fmaxf(s[t][0], s[t][2]), fmaxf(s[t][1], s[t][3])};
        float p[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
          const float mn = fmaxf(m[t][e], mx[e]);
          const float base = mn == -INFINITY ? 0.f : mn;
          const float alpha = exp2f(m[t][e] - base);
          m[t][e] = mn;
          p[e] = exp2f(s[t][e] - base);
          p[e + 2] = exp2f(s[t][e + 2] - base);
          l[t][e] = fmaf(l[t][e], alpha, p[e] + p[e + 2]);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[k][t][e] *= alpha;
            o[k][t][e + 2] *= alpha;
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t hi = tc::pack_bf16(p[2 * r], p[2 * r + 1]);
          const uint32_t lo = tc::pack_bf16(p[2 * r] - bf16lo(hi), p[2 * r + 1] - bf16hi(hi));
          ph[t][r] = transpose8x8(hi);
          pl[t][r] = transpose8x8(lo);
        }
      }
      cp_async_wait<2 * S - 2>();
      __syncwarp();
      const int vr = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t f[4];
        ldsm4_trans(vb + Ring::chunk(vr, 2 * k + ((lane >> 3) & 1)), f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816(o[k][t], f, ph[t][0], ph[t][1]);
          mma16816(o[k][t], f, pl[t][0], pl[t][1]);
        }
      }
      if (i == new_tile && ((held >> new_row) & 1u)) ring.keep_new(stage, new_row);
      stage = stage + 1 == S ? 0 : stage + 1;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[t][e] = x;
      }
    // the stage read last is not refilled before the join: its K takes a warp's results
    const int last = stage == 0 ? S - 1 : stage - 1;
    const auto joined = [&](int w) { return reinterpret_cast<float*>(smem + (w * S + last) * Ring::kStage); };
    __syncwarp();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t > 0) __syncthreads();  // the first eight heads' results are read
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = 2 * (lane & 3) + e;
        if (lane < 4) {
          s_m[warp][t * 8 + g] = m[t][e];
          s_l[warp][t * 8 + g] = l[t][e];
        }
        float* op = joined(warp) + g * D;
        const int x = (lane & 3) << 3;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          op[(k * 16 + (lane >> 2)) ^ x] = o[k][t][e];
          op[(k * 16 + 8 + (lane >> 2)) ^ x] = o[k][t][e + 2];
        }
      }
      __syncthreads();
      join_warps<__nv_bfloat16, D, H, CL>(a, piece, t * 8, s_m, s_l, joined, part, part_at(t * 8));
    }
    u += n_tiles;
    if (!CL && u < u_end) {
      __syncthreads();  // every warp has read the results: the stage is free
      cc.tile = tile0 + n_tiles - 1;
      cc.next(a, prefix, u);
    }
  }
  if constexpr (CL) join_cluster<__nv_bfloat16, D, H>(a, cl_b, cl_pair, share.u0 < u_end, part, part_at);
}

// ------------------------------------------------------------------ CUDA-core form (fp32)
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

// Each lane holds d / 32 elements of a row. U slots at a time, a warp forms the U GB
// partial dot products and sums them over the lanes by halving: after step i a lane
// keeps the half of the products its lane bit names, so the sums cost U GB - 1 exchanges
// rather than 5 U GB, and the product of (slot u, head g) ends in the lanes whose top
// bits are u GB + g. Softmax and mass scores are then one value per lane.
// Bound: HBM while a kv head has few query heads (16 sequences of 2000 to 4000 slots, 8 kv
// heads of 128: 1 or 4 query heads each 68 us, 89% of the copy bandwidth); at 8 its issue slots
// (the same: 89 us, 68%; 12 sequences of 8000 slots, 4 kv heads of 64: 64 us, 47%). More than 8
// are blocks of up to 8 that each read the cache (16: 169 us, 36%).
template <typename C, int D, int GB, bool CL>
__global__ void __launch_bounds__(kPagedThreads, C::kCtas)
paged_fp32_kernel(const __grid_constant__ PagedArgs a) {
  using Ring = typename C::Ring;
  constexpr int N = D / 32, S = C::S, SLOTS = C::SLOTS;
  constexpr int U = GB >= 8 ? 4 : 8;  // slots at a time
  constexpr int P = U * GB;           // products: 8 .. 32
  constexpr int SH = P == 32 ? 0 : P == 16 ? 1 : 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int warp_tmp[kPagedWarps];
  __shared__ float s_m[kPagedWarps][8], s_l[kPagedWarps][8];
  __shared__ __align__(16) float s_p[kPagedWarps][32];
  __shared__ int64_t s_new[kPagedWarps * S];
  __shared__ ClusterPart<CL ? 8 : 1> part;
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + C::kSmem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  Share share = plan_tiles<Ring::kTile>(a, prefix, warp_tmp);
  write_empty_rows<float>(a, prefix, D);
  [[maybe_unused]] int cl_b = 0, cl_pair = 0;
  const auto part_at = [&](int g) { return reinterpret_cast<float*>(smem + Ring::kHalf) + g * D; };
  if constexpr (CL) {
    if (!cluster_share<Ring::kTile>(a, prefix, cl_b, cl_pair, share)) return;  // the whole cluster
  } else if (share.u0 >= share.u1) {
    return;
  }
  const int u_end = share.u1;
  Ring ring(a, prefix, smem, s_new, share.u0, u_end);
  Cursor<Ring::kTile> cc;
  if (!CL || share.u0 < u_end) cc.seek(a, prefix, share.u0);
  int stage = 0;
  for (int u = share.u0; u < u_end;) {
    const int b = cc.b, len = cc.len, tiles = cc.tiles, tile0 = cc.tile;
    const int n_tiles = min(tiles - tile0, u_end - u);
    const int kvh = cc.pair / a.blocks, blk = cc.pair - kvh * a.blocks;
    const Piece piece{b, kvh * a.G + blk * a.heads, min(a.heads, a.G - blk * a.heads), tile0 == 0,
                      n_tiles == tiles};
    const int new_tile =
        cc.fresh >= 0 && blk == 0 && cc.fresh % Ring::kTile / SLOTS == warp ? tiles - 1 - tile0 : -1;
    const int new_row = cc.fresh % SLOTS;
    float q[GB][N];
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      const auto x = load_vec<N>(reinterpret_cast<const float*>(a.q + (int64_t)b * a.q_bytes) +
                                 (int64_t)(piece.h0 + min(g, piece.heads - 1)) * D + lane * N);
#pragma unroll
      for (int e = 0; e < N; ++e) q[g][e] = x.v[e] * a.scale2;
    }
    float m = -INFINITY, l = 0.f;  // of head (lane >> SH) % GB
    float o[GB][N];
#pragma unroll
    for (int g = 0; g < GB; ++g)
#pragma unroll
      for (int e = 0; e < N; ++e) o[g][e] = 0.f;
    for (int i = 0; i < n_tiles; ++i) {
      __syncwarp();  // every lane has read the stage that is filled next
      ring.issue(stage == 0 ? S - 1 : stage - 1);
      const uint32_t held = ring.held(stage);
      const uint8_t* kb = smem + (warp * S + stage) * Ring::kStage;
      const auto row = [&](const uint8_t* base, int r) {  // this lane's elements of a staged row
        return load_vec<N>(reinterpret_cast<const float*>(base + Ring::chunk(r, lane * N / 4)) + lane * N % 4);
      };
      cp_async_wait<2 * S - 2>();
      __syncwarp();
#pragma unroll 1
      for (int r0 = 0; r0 < SLOTS; r0 += U) {
        float s[P];
#pragma unroll
        for (int i2 = 0; i2 < U; ++i2) {
          const auto k = row(kb, r0 + i2);
#pragma unroll
          for (int g = 0; g < GB; ++g) {
            float t = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) t = fmaf(q[g][e], k.v[e], t);
            s[i2 * GB + g] = t;
          }
        }
        int n = P;
#pragma unroll
        for (int bit = 16; bit > 0; bit >>= 1) {
          if (n > 1) {
            n >>= 1;
            const bool up = lane & bit;
#pragma unroll
            for (int i2 = 0; i2 < P / 2; ++i2)
              if (i2 < n) {
                const float mine = up ? s[i2 + n] : s[i2], give = up ? s[i2] : s[i2 + n];
                s[i2] = mine + __shfl_xor_sync(0xffffffffu, give, bit);
              }
          } else {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], bit);
          }
        }
        const int c = lane >> SH, iu = c / GB, ig = c % GB;
        const float sc = (held >> (r0 + iu)) & 1u ? s[0] : -INFINITY;
        if (a.scores && (lane & ((1 << SH) - 1)) == 0) {
          const int j = (tile0 + i) * Ring::kTile + warp * SLOTS + r0 + iu;
          if (ig < piece.heads && j < len) a.scores[((int64_t)b * a.Hq + piece.h0 + ig) * a.score_row + j] = sc;
        }
        float mx = sc;
#pragma unroll
        for (int bit = 16; bit >= 32 / U; bit >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, bit));
        const float mn = fmaxf(m, mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float p = exp2f(sc - base), alpha = exp2f(m - base);
        float ps = p;
#pragma unroll
        for (int bit = 16; bit >= 32 / U; bit >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, bit);
        l = l * alpha + ps;
        m = mn;
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          const float al = __shfl_sync(0xffffffffu, alpha, g << SH);
#pragma unroll
          for (int e = 0; e < N; ++e) o[g][e] *= al;
        }
        if constexpr (GB >= 4) {  // a slot's weights of four heads in one broadcast read
          __syncwarp();
          s_p[warp][lane] = p;  // P = 32: the lane is the product
          __syncwarp();
        }
#pragma unroll
        for (int i2 = 0; i2 < U; ++i2) {
          const auto v = row(kb + Ring::kHalf, r0 + i2);
          float w[GB];
          if constexpr (GB >= 4) {
#pragma unroll
            for (int g = 0; g < GB; g += 4) {
              const float4 x = *reinterpret_cast<const float4*>(&s_p[warp][i2 * GB + g]);
              w[g] = x.x; w[g + 1] = x.y; w[g + 2] = x.z; w[g + 3] = x.w;
            }
          } else {
#pragma unroll
            for (int g = 0; g < GB; ++g) w[g] = __shfl_sync(0xffffffffu, p, (i2 * GB + g) << SH);
          }
#pragma unroll
          for (int g = 0; g < GB; ++g)
#pragma unroll
            for (int e = 0; e < N; ++e) o[g][e] = fmaf(w[g], v.v[e], o[g][e]);
        }
      }
      if (i == new_tile && ((held >> new_row) & 1u)) ring.keep_new(stage, new_row);
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    const int last = stage == 0 ? S - 1 : stage - 1;
    const auto joined = [&](int w) { return reinterpret_cast<float*>(smem + (w * S + last) * Ring::kStage); };
    __syncwarp();
    if (lane < (GB << SH) && (lane & ((1 << SH) - 1)) == 0) {
      s_m[warp][lane >> SH] = m;
      s_l[warp][lane >> SH] = l;
    }
#pragma unroll
    for (int g = 0; g < GB; ++g)
#pragma unroll
      for (int e = 0; e < N; ++e) joined(warp)[g * D + ((lane * N + e) ^ (((g >> 1) & 3) << 3))] = o[g][e];
    __syncthreads();
    join_warps<float, D, 8, CL>(a, piece, 0, s_m, s_l, joined, part, part_at(0));
    u += n_tiles;
    if (!CL && u < u_end) {
      __syncthreads();  // every warp has read the results: the stage is free
      cc.tile = tile0 + n_tiles - 1;
      cc.next(a, prefix, u);
    }
  }
  if constexpr (CL) join_cluster<float, D, 8>(a, cl_b, cl_pair, share.u0 < u_end, part, part_at);
}

// ------------------------------------------------------------------ join and masses
// CTAs whose tiles hold a sequence-head: first and last, from the plan of the main kernel.
struct Span {
  int c0, c1;
};
// What the plan says of a sequence: its first tile, the tiles of each of its heads (or head
// blocks), and the tiles of a CTA.
struct SequenceTiles {
  int first, tiles, share;
  __device__ __forceinline__ SequenceTiles(const PagedArgs& a, int b) {
    first = a.prefix[b];
    tiles = (a.prefix[b + 1] - first) / (a.c.Hkv * a.blocks);
    share = (int)(((uint32_t)a.prefix[a.B] + (uint32_t)a.grid - 1u) / (uint32_t)a.grid);
  }
  __device__ __forceinline__ Span span(int pair) const {
    const int at = first + pair * tiles;
    return Span{at / share, (at + tiles - 1) / share};
  }
};
__device__ __forceinline__ int64_t part_slot(const Span& s, int c) {
  return 2 * (int64_t)c + (c == s.c0 ? 1 : 0);
}

constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kMassChunk = 128;  // slots per step of a mass CTA: four to a lane, warps share the heads

// (m, l) of the union of two parts.
__device__ __forceinline__ void merge_ml(float& m, float& l, float m2, float l2) {
  const float mn = fmaxf(m, m2);
  const float base = mn == -INFINITY ? 0.f : mn;
  l = l * exp2f(m - base) + l2 * exp2f(m2 - base);
  m = mn;
}

// Bound: latency (4 us; with masses 6 us at 16 sequences of 1024 slots, 32 heads) and, with
// masses in long caches, the scores' bytes (16 us at 64 sequences of up to 8191, 28 heads).
// CTAs [0, out_ctas = B Hq, or none where no sequence-head is split): the output of one
// (sequence, query head) that was split, its parts over four warps. The rest, mass_ctas to a
// sequence: the masses, from the scores the main kernel left and the joined log-sums. Each
// warp takes eight heads at a time, forms their log-sums (4 lanes to a head) rather than
// waiting for another kernel's, and adds up their part of the CTA's slots.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(const __grid_constant__ PagedArgs a, int out_ctas, int mass_ctas) {
  pdl_wait();
  constexpr int N = D / 32;
  extern __shared__ float z2[];  // [Hq rounded up to 8] of this sequence, log2 units (mass CTAs);
                                // a warp's heads are written and read by that warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x < out_ctas) {
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ float s_o[kJoinWarps][D];
    const int i = blockIdx.x, b = i / a.Hq, h = i - b * a.Hq;
    const int kvh = h / a.G, g = h - kvh * a.G, blk = g / a.heads, gi = g - blk * a.heads;
    const SequenceTiles plan(a, b);
    if (plan.tiles == 0) return;
    const Span s = plan.span(kvh * a.blocks + blk);
    if (s.c0 == s.c1) return;  // already whole
    float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    for (int c = s.c0 + warp; c <= s.c1; c += 4 * kJoinWarps) {
      float2 ml[4];
      LaneRow<float, N> x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int cc = c + k * kJoinWarps;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (cc > s.c1) continue;
        const int64_t at = part_slot(s, cc) * a.heads + gi;
        ml[k] = a.part_ml[at];
        x[k] = load_vec<N>(a.part_o + at * D + lane * N);
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < 4; ++k) mn = fmaxf(mn, ml[k].x);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f0 = exp2f(m - base);
      l *= f0;
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] *= f0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (c + k * kJoinWarps > s.c1) continue;
        const float f = exp2f(ml[k].x - base);
        l = fmaf(ml[k].y, f, l);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(x[k].v[e], f, acc[e]);
      }
      m = mn;
    }
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
    for (int e = 0; e < N; ++e) s_o[warp][lane * N + e] = acc[e];
    __syncthreads();
    m = s_m[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, s_m[w]);
    const float base = m == -INFINITY ? 0.f : m;
    l = 0.f;
    float o = 0.f;
    const int e = threadIdx.x < D ? threadIdx.x : 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = exp2f(s_m[w] - base);
      l = fmaf(s_l[w], f, l);
      o = fmaf(s_o[w][e], f, o);
    }
    if (threadIdx.x < D) store_out(reinterpret_cast<T*>(a.out) + (int64_t)i * D + e, l > 0.f ? o / l : 0.f);
    if (threadIdx.x == 0 && a.lse) a.lse[i] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    return;
  }
  // ---- masses of one sequence's slots
  const int k = (int)(blockIdx.x - out_ctas), b = k / mass_ctas, part = k - b * mass_ctas;
  const int len = checked_length(a.lengths, b, a.max_len);
  if (part * kMassChunk >= len) return;
  __shared__ float4 s_sum[kJoinWarps][32];
  const float* scores = a.scores + (int64_t)b * a.Hq * a.score_row;
  int j = part * kMassChunk + 4 * lane;
  // the scores of eight heads; the first eight are under way while the log-sums are formed
  float4 x[8];
  const auto load = [&](int h) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j < len)
        x[e] = *reinterpret_cast<const float4*>(scores + min(h + e, a.Hq - 1) * a.score_row + j);
  };
  load(8 * warp);
  // a head without weights (or behind the last) adds none: e^{s - inf} = 0
  if (a.split != PagedSplit::kRanges) {  // whole heads: four times this warp's eight at once
    for (int h = 8 * warp + (lane & 7) + 8 * kJoinWarps * (lane >> 3); h < (a.Hq + 7) / 8 * 8; h += 32 * kJoinWarps) {
      const float m = h < a.Hq ? a.lse2[(int64_t)b * a.Hq + h] : -INFINITY;
      z2[h] = m == -INFINITY ? INFINITY : m;
    }
  } else {
    const SequenceTiles plan(a, b);
    for (int h0 = 8 * warp; h0 < a.Hq; h0 += 8 * kJoinWarps) {
      const int h = h0 + (lane >> 2);
      float m = -INFINITY, l = 0.f;
      bool whole = false;
      if (h < a.Hq) {
        const int kvh = h / a.G, g = h - kvh * a.G, blk = g / a.heads, gi = g - blk * a.heads;
        const Span s = plan.span(kvh * a.blocks + blk);
        whole = s.c0 == s.c1;
        if (whole) {
          m = a.lse2[(int64_t)b * a.Hq + h];
        } else {
#pragma unroll 4
          for (int c = s.c0 + (lane & 3); c <= s.c1; c += 4) {
            const float2 ml = a.part_ml[part_slot(s, c) * a.heads + gi];
            merge_ml(m, l, ml.x, ml.y);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        if (!whole) merge_ml(m, l, m2, l2);
      }
      if ((lane & 3) == 0)
        z2[h] = h >= a.Hq || m == -INFINITY ? INFINITY : whole ? m : m + log2f(l);
    }
  }
  __syncwarp();
  const float inv = 1.f / (float)a.Hq;
  const int fresh = new_slot(a, b, len);
  for (int first = part * kMassChunk; first < len; first += kMassChunk * mass_ctas) {
    j = first + 4 * lane;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int h = 8 * warp; h < a.Hq; h += 8 * kJoinWarps) {
      if (h > 8 * warp || first > part * kMassChunk) load(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = z2[h + e];
        sum.x += exp2f(x[e].x - z);
        sum.y += exp2f(x[e].y - z);
        sum.z += exp2f(x[e].z - z);
        sum.w += exp2f(x[e].w - z);
      }
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    const int at = first + threadIdx.x;  // a slot a thread
    if (at < len) {
      float total = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) total += reinterpret_cast<const float*>(s_sum[w])[threadIdx.x];
      const int64_t o = (int64_t)b * a.mass_stride + at;
      const float before = a.mass_in && at != fresh ? a.mass_in[o] : 0.f;
      a.mass_out[o] = before + total * inv;
    }
    __syncthreads();
  }
}

struct PagedWorkspace {
  size_t prefix, ml, o, lse2, scores, total;
};
// Heads of one block: a kv head's query heads in as few equal blocks as the limit allows.
int head_blocks(int G, int limit) { return (G + limit - 1) / limit; }

int64_t score_row(int max_len) { return ((int64_t)max_len + 3) & ~3ll; }
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
  w.scores = take(mass ? (size_t)B * Hq * score_row(max_len) * 4 : 0);
  w.total = at;
  return w;
}

int64_t sequence_heads(const PagedArgs& a) { return (int64_t)a.B * a.c.Hkv * a.blocks; }

// bf16: up to 16 heads in one pass over the cache (two column tiles); fp32: 8.
int heads_per_block(int G, bool bf16) {
  const int blocks = head_blocks(G, bf16 ? kMaxHeads : 8);
  return (G + blocks - 1) / blocks;
}

template <typename C, bool CL>
cudaError_t launch_split(void (*kernel)(PagedArgs), int& configured_for, PagedArgs& a, cudaStream_t stream) {
  const DeviceInfo& dev = device_info();
  if (configured_for != dev.device) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C::kSmem + (kPagedMaxBatch + 1) * 4);
    if (e != cudaSuccess) return e;
    configured_for = dev.device;
  }
  a.even_pages = a.c.page.n % C::SLOTS == 0;
  const int64_t pairs = sequence_heads(a);
  int64_t ctas = a.split == PagedSplit::kWhole ? pairs : pairs * tile_count(a.max_len, C::Ring::kTile);
  const int64_t most = std::min<int64_t>((int64_t)dev.sm_count * C::kCtas, kMaxPagedGrid);
  ctas = CL ? pairs * kPairCtas : std::min(ctas, most);
  a.grid = (int)ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kPagedThreads);
  cfg.dynamicSmemBytes = C::kSmem + ((size_t)a.B + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPairCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <typename C, int D, int NT, bool CL = false>
cudaError_t launch_mma(PagedArgs& a, cudaStream_t stream) {
  static thread_local int configured_for = -1;
  return launch_split<C, CL>(paged_mma_kernel<C, D, NT, CL>, configured_for, a, stream);
}
template <typename C, int D, int GB, bool CL>
cudaError_t launch_fp32_heads(PagedArgs& a, cudaStream_t stream) {
  static thread_local int configured_for = -1;
  return launch_split<C, CL>(paged_fp32_kernel<C, D, GB, CL>, configured_for, a, stream);
}

// Stages of a warp's ring. Two CTAs an SM with three stages keep the most bytes in flight,
// which one long sequence wants (bf16, 131071 slots, 8 kv heads: 88.7 us, against 92.9 with
// three CTAs of two stages). Where there are as many sequence-heads as SMs their ends and
// starts cost more, and a third CTA works through them (7 sequences of 32 kv heads: 26.9 us
// against 29.0; 64 of 4: 109.5 against 111.0). Both sides of each were measured in one run.
// 9 to 16 query heads leave registers for two CTAs, and two stages at d = 128: 32 sequences of
// 4096 slots, 4 kv heads of 128, take 54.5 us with 9 and 56.8 with 16, 51.4 with 8 (75, 72 and
// 80% of the copy bandwidth); with 8 kv heads of 64, 16 query heads each, 78 us (53%).
template <int D>
cudaError_t launch_bf16(PagedArgs& a, cudaStream_t stream) {
  using T = __nv_bfloat16;
  using Deep = PagedCfg<T, D, 3, 2>;
  using Wide = PagedCfg<T, D, 2, 3>;
  using Heads16 = PagedCfg<T, D, D == 128 ? 2 : 3, 2>;  // registers: two CTAs
  if (a.split == PagedSplit::kCluster)
    return a.heads > 8 ? launch_mma<Heads16, D, 2, true>(a, stream) : launch_mma<Deep, D, 1, true>(a, stream);
  if (a.heads > 8) return launch_mma<Heads16, D, 2>(a, stream);
  return sequence_heads(a) >= device_info().sm_count ? launch_mma<Wide, D, 1>(a, stream)
                                                     : launch_mma<Deep, D, 1>(a, stream);
}

template <int D, bool CL>
cudaError_t launch_fp32(PagedArgs& a, cudaStream_t stream) {
  using C = PagedCfg<float, D, 3, 2>;
  switch (a.heads) {
    case 1: return launch_fp32_heads<C, D, 1, CL>(a, stream);
    case 2: return launch_fp32_heads<C, D, 2, CL>(a, stream);
    case 3: case 4: return launch_fp32_heads<C, D, 4, CL>(a, stream);
    default: return launch_fp32_heads<C, D, 8, CL>(a, stream);
  }
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
  // the type is not known here: room for either
  const size_t x = paged_layout(B, Hq, d, max_len, mass, heads_per_block(Hq / Hkv, false)).total;
  const size_t y = paged_layout(B, Hq, d, max_len, mass, heads_per_block(Hq / Hkv, true)).total;
  return x > y ? x : y;
}

int64_t paged_attention_tiles(int B, int Hq, int max_len) {
  return (int64_t)B * Hq * tile_count(max_len, 32);  // the smaller tile
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
  a.heads = heads_per_block(a.G, c.dtype == DD_BF16);
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
  a.score_row = score_row(p.max_len);
  a.scores = p.mass_out ? reinterpret_cast<float*>(ws + w.scores) : nullptr;
  // Short sequences are not split, so that nothing is left to a join (with masses: but those).
  // Whole sequence-heads fill the GPU where there are as many as SMs and not a few more than
  // CTAs at once, whose second round runs on a nearly idle GPU; what that costs is compared with
  // the join, about four tiles of a CTA (none with masses: their join stays), or small against
  // eight rounds. fp32 with masses is bound by its issue slots, which ragged whole ones leave
  // idle (64 of 4, 100 to 512 slots: 37.5, 32.4 split): short ones only. (bf16, 28 heads: 64
  // sequences of 4 kv heads, 512 slots: 15.1 us, 19.5 split; with masses 17.5, 20.6; of 100 to
  // 250, 96 of them: 14.4, 19.0. 64 of 8, 256 slots: 15.5, 18.5; but 512 slots: 22.4, 19.6
  // split. fp32: 64 of 4, 250 slots: 13.4, 15.5; 64 of 8, 512 slots: 39.6, 33.4 split; 96 of 32,
  // 1 to 400 slots: 148, 160.) With few, a CTA would walk through its tiles alone (one sequence
  // of 8 kv heads, 200 slots: 8.2 us whole, 6.7 split and joined) and a cluster shares them (6.2
  // us, and 2 us less of the host's time than two launches), unless there is one tile (64 slots:
  // 5.1 us whole, 6.2 split). With masses, which take a second launch anyway, a cluster gains
  // nothing (200 slots: 8.2 us, 7.8 split). Clusters beyond what is resident at once would
  // queue: those are split (8 sequences, 256 slots: 7.7 us; whole 8.5).
  a.split = PagedSplit::kRanges;
  const int tile = c.d * e == 512 ? kTileSlots / 2 : kTileSlots;
  const int64_t pairs = sequence_heads(a), sms = device_info().sm_count;
  const int64_t resident = sms * (c.dtype == DD_BF16 && a.heads <= 8 ? 3 : 2);
  const int64_t idle = pairs <= resident ? 0 : (resident - pairs % resident) % resident;
  const int whole_len = p.mass_out && c.dtype == DD_F32 ? 4 * tile : kWholeLen;
  const bool even = pairs >= 8 * resident ||
                    idle * tile_count(p.max_len, tile) <= (p.mass_out ? 0 : 4 * resident);
  if (p.max_len <= tile || (p.max_len <= whole_len && pairs >= sms && even))
    a.split = PagedSplit::kWhole;
  else if (p.max_len <= kWholeLen && !p.mass_out && pairs * kPairCtas <= 2 * sms)
    a.split = PagedSplit::kCluster;
  cudaError_t err;
  if (c.dtype == DD_BF16)
    err = c.d == 128 ? launch_bf16<128>(a, stream) : launch_bf16<64>(a, stream);
  else if (a.split == PagedSplit::kCluster)
    err = c.d == 128 ? launch_fp32<128, true>(a, stream) : launch_fp32<64, true>(a, stream);
  else
    err = c.d == 128 ? launch_fp32<128, false>(a, stream) : launch_fp32<64, false>(a, stream);
  if (err != cudaSuccess || (a.split != PagedSplit::kRanges && !p.mass_out)) return err;
  // join: a CTA per query head that may be split; masses: enough CTAs a sequence to fill the GPU a few times
  int mass_ctas = 0;
  if (p.mass_out) {
    const int chunks = (p.max_len + kMassChunk - 1) / kMassChunk;
    const int fill = (device_info().sm_count * 8 + p.B - 1) / p.B;
    mass_ctas = chunks < fill ? chunks : fill;
  }
  const int out_ctas = a.split == PagedSplit::kRanges ? p.B * p.Hq : 0;
  const dim3 grid((unsigned)(out_ctas + mass_ctas * p.B));
  const size_t zmem = p.mass_out ? ((size_t)p.Hq + 7) / 8 * 8 * 4 : 0;
  const auto join = [&](auto kernel) {
    return launch_dependent(kernel, grid, dim3(kJoinThreads), zmem, stream, a, out_ctas, mass_ctas);
  };
  if (c.dtype == DD_BF16)
    return c.d == 128 ? join(paged_join_kernel<__nv_bfloat16, 128>)
                      : join(paged_join_kernel<__nv_bfloat16, 64>);
  return c.d == 128 ? join(paged_join_kernel<float, 128>) : join(paged_join_kernel<float, 64>);
}

}  // namespace dd
