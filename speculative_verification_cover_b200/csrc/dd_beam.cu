// Beam search's selection over beams and vocabulary (dd_beam_select).
//
// score(k, v) = score_k + x_kv - lse_k with lse_k = log sum_u e^{x_ku}, summed and compared
// relative to the beam's largest logit: (x_kv - m_k) - log sum_u e^{x_ku - m_k}. Within a beam the
// order of the candidates is the order of the logits, so the scan of a row needs no lse:
// each CTA reads one piece of one row once, leaves the piece's maximum, its sum of
// exponentials and its K best logits, and a merge CTA per request joins the sums and picks
// the K best candidates by score, in 64 bits.
//
// Bound: HBM, B K V logits read once. Measured (one B200): 32 requests of 16 beams, 152064
// tokens, a tenth of the beams done: scan 43.5 us for 140 MB (half of the copy bandwidth; see
// the scan), merge 12.6 us; a whole step with reordered states 76.7 us. 16 requests of 16 beams
// in fp32, none done: scan and merge 54 us for 156 MB. One request of 4 beams, 1000 tokens, the
// whole step: 13.4 us, four launches.
#include "dd_common.cuh"
#include "dd_internal.h"
#include "dd_tc.cuh"

namespace dd {

namespace {

constexpr int kBeamThreads = 256;  // of the merge
constexpr int kBeamWarps = kBeamThreads / 32;
// The scan: pieces of 32 KB, six CTAs an SM, which is what bounds it: about 12 K cycles of
// latency a piece (half of its issue slots are taken).
constexpr int kScanThreads = 256;
constexpr int kScanCtas = 6;       // an SM
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanVecs = 8;       // 16-byte vectors per thread: a segment of 128 bytes
constexpr int kPieceBytes = kScanThreads * kScanVecs * 16;
constexpr int kBeamList = 512;  // candidates ranked by counting
constexpr uint32_t kNone = 0x007FFFFFu;  // key of -inf

template <typename T>
constexpr int beam_piece() { return kPieceBytes / (int)sizeof(T); }

__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// NaN and +inf are no candidates; -0 ties with 0.
__device__ __forceinline__ float clean_logit(float x) { return x < INFINITY ? x + 0.f : -INFINITY; }

// The two (bf16) or one (fp32) logits of a 32-bit word.
template <typename T>
struct Word;
template <>
struct Word<__nv_bfloat16> {
  static constexpr int n = 2;
  static __device__ __forceinline__ float get(uint32_t w, int e) { return e ? bf16hi(w) : bf16lo(w); }
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
};
template <>
struct Word<float> {
  static constexpr int n = 1;
  static __device__ __forceinline__ float get(uint32_t w, int) { return __uint_as_float(w); }
  static constexpr uint32_t kNegInf = 0xFF800000u;
};

// Largest logit of four words, NaN ignored (NaN only if all are).
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b, float) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ float max_of(uint32_t w, __nv_bfloat16) { return fmaxf(bf16lo(w), bf16hi(w)); }
__device__ __forceinline__ float max_of(uint32_t w, float) { return __uint_as_float(w); }

__device__ __forceinline__ bool scans(const float* score_in, const uint8_t* done_in, int row) {
  const float s = score_in[row];
  const uint8_t d = done_in ? done_in[row] : 0;  // both loads in flight at once
  return isfinite(s) && !d;
}

// The largest 16-bit p that at least `want` of the block's keys reach, bit by bit; all threads
// call it. (A barrier that counts costs 60 to 110 cycles a bit; one warp over all keys, 300
// for two bits.)
__device__ __forceinline__ void kth_bit(uint32_t key, int want, int bit, uint32_t& p) {
  if (__syncthreads_count(key >= (p | (1u << bit))) >= want) p |= 1u << bit;
}
__device__ __forceinline__ uint32_t kth_key16(uint32_t key, int want) {
  uint32_t p = 0;
#pragma unroll 1  // a kernel's first pass waits for its instructions: short code
  for (int bit = 15; bit >= 0; --bit) kth_bit(key, want, bit, p);
  return p;
}

// One piece of one row, copied into shared memory by one bulk copy; several CTAs share an
// SM, so their copies and their arithmetic overlap. A thread reads a segment of the piece
// (eight vectors), keeps its maximum and sums exponentials relative to that maximum. The
// K-th largest of the 256 maxima (its top 16 bits) is a lower bound of the piece's K-th
// largest logit, so only the segments whose maximum reaches it, about K of them, are
// looked at again, a warp to a segment; what reaches the bound there is ranked by counting.
// Where more than kBeamList logits reach the bound (long runs of equal logits), the K-th
// largest is found by a radix select over the piece instead, whose counts of equal logits meet
// in one bin: 32 requests of 16 beams, 152064 tokens, all but 20 at the lowest finite value:
// 634 us, where -inf, which is no candidate, takes 49.
template <typename T>
__global__ void __launch_bounds__(kScanThreads, kScanCtas)
beam_scan_kernel(const T* __restrict__ logits, int K, int V, int64_t ld, int pieces,
                 const float* __restrict__ score_in, const uint8_t* __restrict__ done_in,
                 float2* __restrict__ ml, uint2* __restrict__ cand, uint32_t spin) {
  using W = Word<T>;
  constexpr int kPiece = beam_piece<T>();
  extern __shared__ __align__(128) uint8_t piece_smem[];  // [kPieceBytes]
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint2 s_list[kBeamList];   // (key, index in the piece)
  __shared__ uint8_t s_seg[kScanThreads];
  __shared__ float2 s_ml[kScanWarps + kScanWarps / 2];  // and the radix select's scan
  __shared__ int s_n, s_segs, s_want;
  __shared__ uint32_t s_bound;
  const int row = blockIdx.x / pieces, piece = blockIdx.x - row * pieces;
  if (!scans(score_in, done_in, row)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int base = piece * kPiece, n_here = min(kPiece, V - base);
  uint32_t* words = reinterpret_cast<uint32_t*>(piece_smem);
  const T* from = logits + (int64_t)row * ld + base;
  // whole vectors by the bulk copy, the logits of a last, partly filled one by threads: nothing
  // is read behind the vocabulary
  const int copied = n_here & ~(16 / (int)sizeof(T) - 1);
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    tc::fence_barrier_init();
    if (copied > 0) {
      const uint32_t bytes = (uint32_t)copied * sizeof(T);
      tc::mbar_expect_tx(&bar, bytes);
      tc::bulk_load(piece_smem, from, bytes, &bar);
    }
    s_n = 0;
    s_segs = 0;
  }
  if (n_here < kPiece) {
    T* x = reinterpret_cast<T*>(piece_smem);
    for (int i = copied + threadIdx.x; i < kPiece; i += kScanThreads)
      x[i] = i < n_here ? from[i] : static_cast<T>(-INFINITY);
  }
  __syncthreads();
  const bool here = copied == 0 || mbar_wait_bounded(&bar, 0, spin);
  if (__syncthreads_or(!here)) return;  // recorded; uniform over the CTA
  const uint4* seg = reinterpret_cast<const uint4*>(piece_smem) + threadIdx.x;  // every 256th vector
  uint32_t mw[4] = {W::kNegInf, W::kNegInf, W::kNegInf, W::kNegInf};
#pragma unroll
  for (int i = 0; i < kScanVecs; ++i) {
    const uint4 v = seg[i * kScanThreads];
    mw[0] = max_word(mw[0], v.x, T{});
    mw[1] = max_word(mw[1], v.y, T{});
    mw[2] = max_word(mw[2], v.z, T{});
    mw[3] = max_word(mw[3], v.w, T{});
  }
  float mx = max_of(max_word(max_word(mw[0], mw[1], T{}), max_word(mw[2], mw[3], T{}), T{}), T{}) + 0.f;
  if (mx == INFINITY) {  // not a candidate: again, without such logits
    mx = -INFINITY;
    for (int i = 0; i < kScanVecs; ++i) {
      const uint4 v = seg[i * kScanThreads];
      const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int h = 0; h < W::n; ++h) mx = fmaxf(mx, clean_logit(W::get(r[e], h)));
    }
  }
  const uint32_t mine = logit_key(mx) >> 16;
  uint32_t bound = 0;
  // sum of exponentials relative to the segment's maximum. The maximum is subtracted before
  // the change of base: a difference below 0, exact to half a step of its own, whatever the
  // logits' size, where log2(e) times a logit may overflow or lose all that lies between two.
  const float ref = mx > -INFINITY ? mx : 0.f;
  float sum = 0.f;
  {
    // two logits at a time, packed; the bound's bits are counted in between, so that its
    // barriers' latency is spent on them
    float2 part[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) part[e] = make_float2(0.f, 0.f);
    const float2 scale = make_float2(kLog2e, kLog2e), shift = make_float2(-ref, -ref);
    static_assert(kScanVecs == 8);  // two of the 16 bits a vector
#pragma unroll 1
    for (int i = 0; i < kScanVecs; ++i) {
      const uint4 v = seg[i * kScanThreads];
      kth_bit(mine, K, 15 - 2 * i, bound);
      const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; e += 2 / W::n) {
        const float2 x = W::n == 2 ? make_float2(W::get(r[e], 0), W::get(r[e], 1))
                                   : make_float2(W::get(r[e], 0), W::get(r[e + 2 / W::n - 1], 0));
        const float2 y = __fmul2_rn(__fadd2_rn(x, shift), scale);
        part[e] = __fadd2_rn(part[e], make_float2(fast_exp2(y.x), fast_exp2(y.y)));
      }
      kth_bit(mine, K, 14 - 2 * i, bound);
    }
    sum = ((part[0].x + part[0].y) + (part[1].x + part[1].y)) + ((part[2].x + part[2].y) + (part[3].x + part[3].y));
    if (!(sum < INFINITY)) {  // NaN and +inf logits add nothing
      sum = 0.f;
      for (int i = 0; i < kScanVecs; ++i) {
        const uint4 v = seg[i * kScanThreads];
        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int h = 0; h < W::n; ++h)
            sum += fast_exp2((clean_logit(W::get(r[e], h)) - ref) * kLog2e);
      }
    }
  }
  // (maximum, sum) of the piece
  float m = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  sum *= mx > -INFINITY ? fast_exp2((mx - m) * kLog2e) : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_ml[warp] = make_float2(m, sum);
  __syncthreads();
  if (mine >= bound && mx > -INFINITY) s_seg[atomicAdd(&s_segs, 1)] = (uint8_t)threadIdx.x;
  __syncthreads();
  const int segs = s_segs;
  for (int i = warp; i < segs; i += kScanWarps) {
    const int t = s_seg[i];
    const int at = (((lane >> 2) * kScanThreads + t) << 2) + (lane & 3);
    const uint32_t w = words[at];
#pragma unroll
    for (int h = 0; h < W::n; ++h) {
      const uint32_t k = logit_key(clean_logit(W::get(w, h)));
      if ((k >> 16) >= bound && k > kNone) {  // few do
        const int place = atomicAdd(&s_n, 1);
        if (place < kBeamList) s_list[place] = make_uint2(k, (uint32_t)(at * W::n + h));
      }
    }
  }
  __syncthreads();
  int n = s_n;
  if (n > kBeamList) {
    // ---- radix select over the piece
    int* hist = reinterpret_cast<int*>(s_list);  // the list is empty again
    int* scan = reinterpret_cast<int*>(s_ml + kScanWarps);
    const T* x = reinterpret_cast<const T*>(piece_smem);
    uint32_t prefix = 0u;
    int want = K;
    for (int shift = 24; shift >= 0; shift -= 8) {
      const uint32_t hmask = shift == 24 ? 0u : (0xFFFFFFFFu << (shift + 8));
      for (int i = threadIdx.x; i < 256; i += kScanThreads) hist[i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < kPiece; i += kScanThreads) {
        const uint32_t k = logit_key(clean_logit((float)x[i]));
        if (k > kNone && (k & hmask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int run = 0, dgt = 255;
        for (; dgt > 0 && run + hist[dgt] < want; --dgt) run += hist[dgt];
        s_bound = prefix | ((uint32_t)dgt << shift);
        s_want = want - run;
      }
      __syncthreads();
      prefix = s_bound;
      want = s_want;
    }
    // more than kBeamList >= K logits are candidates, so `prefix` is the K-th largest key and
    // `want` >= 1 of the logits equal to it are taken, from the lowest index
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();  // also: the histogram is read
    constexpr int kRun = kPiece / kScanThreads;
    int ties = 0;
    for (int i = threadIdx.x * kRun; i < (threadIdx.x + 1) * kRun; ++i) {
      const uint32_t k = logit_key(clean_logit((float)x[i]));
      if (k > prefix) {
        const int at = atomicAdd(&s_n, 1);
        if (DD_IN_BOUNDS(at < kBeamList)) s_list[at] = make_uint2(k, (uint32_t)i);
      }
      ties += k == prefix;
    }
    int incl = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = incl - ties;
    for (int w = 0; w < warp; ++w) before += scan[w];
    const int above = s_n;
    for (int i = threadIdx.x * kRun; i < (threadIdx.x + 1) * kRun && before < want; ++i)
      if (logit_key(clean_logit((float)x[i])) == prefix) {
        if (DD_IN_BOUNDS(above + before < kBeamList)) s_list[above + before] = make_uint2(prefix, (uint32_t)i);
        ++before;
      }
    __syncthreads();
    n = min(above + want, kBeamList);
  }
  uint2* out = cand + (int64_t)blockIdx.x * K;
  for (int i = threadIdx.x; i < n; i += kScanThreads) {
    const uint2 c = s_list[i];
    int r = 0;
    for (int t = 0; t < n; ++t) {
      const uint2 o = s_list[t];
      r += o.x > c.x || (o.x == c.x && o.y < c.y);
    }
    if (r < K) out[r] = make_uint2(c.x, (uint32_t)base + c.y);
  }
  for (int i = n + threadIdx.x; i < K; i += kScanThreads) out[i] = make_uint2(kNone, 0u);
  if (threadIdx.x == 0) {
    m = s_ml[0].x;
#pragma unroll
    for (int w = 1; w < kScanWarps; ++w) m = fmaxf(m, s_ml[w].x);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w)
      if (s_ml[w].x > -INFINITY) s = fmaf(s_ml[w].y, fast_exp2((s_ml[w].x - m) * kLog2e), s);
    ml[blockIdx.x] = make_float2(m, s);
  }
}

// A candidate's place among those of equal score, smaller first: the beam, then the larger
// logit (which a 64-bit score far from zero no longer tells apart), then the token.
__device__ __forceinline__ int64_t place_of(int k, uint32_t key, int v) {
  return ((int64_t)k << 55) | ((int64_t)(0xFFFFFFFFu - key) << 23) | v;
}
__device__ __forceinline__ int place_beam(int64_t at) { return (int)(at >> 55); }
__device__ __forceinline__ int place_token(int64_t at) { return (int)(at & ((1 << 23) - 1)); }
static_assert(kBeamMaxV <= 1 << 23 && kBeamMaxK <= 1 << 7);

struct Best {
  double score;
  int64_t at;
  int list;
};
__device__ __forceinline__ bool better(double s, int64_t at, double s2, int64_t at2) {
  return s > s2 || (s == s2 && at < at2);
}

// What the merge holds in shared memory from its first loads: entries, and lists' sums (more
// are read again where they are needed).
constexpr int kHeldEntries = 4096;
constexpr int kHeldLists = 512;

struct BeamOut {
  int32_t* parent;
  int32_t* token;
  float* score;
  uint8_t* done;
  int eos;
};
// Rank r of a request: token v of beam k (k < 0: none).
__device__ __forceinline__ void write_beam(const BeamOut& o, int64_t r, int k, bool was_done, double score,
                                           int token) {
  const int v = k < 0 ? -1 : was_done ? o.eos : token;
  o.parent[r] = k < 0 ? -1 : k;
  o.token[r] = v;
  o.score[r] = k < 0 ? -INFINITY : (float)score;
  if (o.done) o.done[r] = k >= 0 && (was_done || v == o.eos) ? 1 : 0;
}

// One CTA per request. Candidates are the lists' entries (K per beam and piece) and one of
// each beam that is done. The K-th largest of the threads' best scores bounds the K-th best
// from below; the few candidates that reach it are ranked by counting. (The bound compares
// distances below the best score by their top 16 bits: 1 part in 128, whatever the scores'
// size.) Should more than kBeamList reach it, K rounds over the lists' heads pick one each.
__global__ void __launch_bounds__(kBeamThreads)
beam_merge_kernel(int K, int pieces, const float* __restrict__ score_in,
                  const uint8_t* __restrict__ done_in, const float2* __restrict__ ml,
                  const uint2* __restrict__ cand, BeamOut res) {
  pdl_wait();
  extern __shared__ uint8_t head[];  // [K * pieces]
  __shared__ double s_base[kBeamMaxK];
  __shared__ uint8_t s_kind[kBeamMaxK];  // 0 no candidate, 1 live, 2 done
  __shared__ float s_max[kBeamMaxK];
  __shared__ double s_sum[kBeamMaxK];
  __shared__ Best s_best[kBeamWarps];
  __shared__ float2 s_ml[kHeldLists];
  __shared__ uint2 s_cand[kHeldEntries];
  __shared__ double s_score[kBeamList];
  __shared__ int64_t s_at[kBeamList];
  __shared__ int s_n;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lists = K * pieces;
  const uint2* mine = cand + (int64_t)b * lists * K;
  // everything is loaded at once: the lists' entries do not wait for the sums
  const int per_beam = pieces * K, entries = K * per_beam;
#pragma unroll 4
  for (int i = threadIdx.x; i < min(entries, kHeldEntries); i += kBeamThreads) s_cand[i] = mine[i];
  const bool small = lists <= kHeldLists;
  if (small)
    for (int i = threadIdx.x; i < lists; i += kBeamThreads) s_ml[i] = ml[(int64_t)b * lists + i];
  if (threadIdx.x < K) {
    const float s = score_in[b * K + threadIdx.x];
    const bool done = done_in && done_in[b * K + threadIdx.x];
    s_kind[threadIdx.x] = !isfinite(s) ? 0 : done ? 2 : 1;
    s_base[threadIdx.x] = (double)s;
  }
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  for (int k = warp; k < K; k += kBeamWarps) {
    if (s_kind[k] != 1) continue;
    const float2* p = small ? s_ml + k * pieces : ml + ((int64_t)b * K + k) * pieces;
    float m = -INFINITY;
    for (int i = lane; i < pieces; i += 32) m = fmaxf(m, p[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double z = 0.0;
    if (m > -INFINITY)
      for (int i = lane; i < pieces; i += 32) z += (double)p[i].y * (double)expf(p[i].x - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) {
      s_max[k] = m;
      s_sum[k] = z;
    }
  }
  __syncthreads();
  if (threadIdx.x < K && s_kind[threadIdx.x] == 1) {
    const float m = s_max[threadIdx.x];
    if (m > -INFINITY) s_base[threadIdx.x] -= log(s_sum[threadIdx.x]);
    else s_kind[threadIdx.x] = 0;
  }
  __syncthreads();
  // An entry of live beam k, from its distance to the beam's largest logit (next to which score
  // and log-sum may be lost in 64 bits); the one candidate of done beam k.
  const auto entry = [&](int k, double base, double largest, const uint2& c, double& s, int64_t& at) {
    if (c.x <= kNone) return false;
    s = base + ((double)key_logit(c.x) - largest);
    at = place_of(k, c.x, (int)c.y);
    return true;
  };
  const auto ended = [&](int k, double& s, int64_t& at) {
    if (s_kind[k] != 2) return false;
    s = s_base[k];
    at = place_of(k, 0u, 0);
    return true;
  };
  // this thread's candidates: warp w has beams w, w + 8, ..., a lane every 32nd entry
  const auto each = [&](auto f) {
    double s;
    int64_t at;
#pragma unroll 1
    for (int k = warp; k < K; k += kBeamWarps) {
      if (s_kind[k] == 1) {
        const double base = s_base[k], largest = s_max[k];
#pragma unroll 2
        for (int i = k * per_beam + lane; i < (k + 1) * per_beam; i += 32)
          if (entry(k, base, largest, i < kHeldEntries ? s_cand[i] : mine[i], s, at)) f(s, at);
      }
      if (lane == 0 && ended(k, s, at)) f(s, at);
    }
  };
  double top = -INFINITY;
  each([&](double s, int64_t) { top = fmax(top, s); });
  double best = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmax(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s_best[warp].score = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBeamWarps; ++w) best = fmax(best, s_best[w].score);
  const auto near = [&](double s) {  // 16 bits, larger nearer to the best; 0: none
    return s > -INFINITY ? 0xFFFFu - (__float_as_uint((float)(best - s)) >> 16) : 0u;
  };
  const uint32_t bound = kth_key16(near(top), K);
  if (near(top) >= bound)
    each([&](double s, int64_t at) {
      if (near(s) < bound) return;
      const int n = atomicAdd(&s_n, 1);
      if (n < kBeamList) {
        s_score[n] = s;
        s_at[n] = at;
      }
    });
  __syncthreads();
  const int n = s_n;
  if (n <= kBeamList) {
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
      const double s = s_score[i];
      const int64_t at = s_at[i];
      int r = 0;
      for (int t = 0; t < n; ++t) r += better(s_score[t], s_at[t], s, at);
      const int k = place_beam(at);
      if (r < K) write_beam(res, (int64_t)b * K + r, k, s_kind[k] == 2, s, place_token(at));
    }
    for (int r = n + threadIdx.x; r < K; r += kBeamThreads)
      write_beam(res, (int64_t)b * K + r, -1, false, 0.0, 0);
    return;
  }
  // ---- K rounds: the best head of the sorted lists, whose list steps on
  for (int i = threadIdx.x; i < lists; i += kBeamThreads) head[i] = 0;
  __syncthreads();
  const auto find = [&](Best& o) {
    o = Best{-INFINITY, INT64_MAX, -1};
    for (int i = threadIdx.x; i < lists; i += kBeamThreads) {
      const int k = i / pieces, h = head[i];
      double s;
      int64_t at;
      if (s_kind[k] == 1 ? h < K && entry(k, s_base[k], s_max[k], mine[i * K + h], s, at)
                         : h == 0 && i == k * pieces && ended(k, s, at))
        if (better(s, at, o.score, o.at)) o = Best{s, at, i};
    }
  };
  Best own;
  find(own);
  for (int r = 0; r < K; ++r) {
    Best x = own;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double s = __shfl_xor_sync(0xffffffffu, x.score, o);
      const int64_t at = __shfl_xor_sync(0xffffffffu, x.at, o);
      const int list = __shfl_xor_sync(0xffffffffu, x.list, o);
      if (better(s, at, x.score, x.at)) x = Best{s, at, list};
    }
    if (lane == 0) s_best[warp] = x;
    __syncthreads();
    x = s_best[0];
    for (int w = 1; w < kBeamWarps; ++w)
      if (better(s_best[w].score, s_best[w].at, x.score, x.at)) x = s_best[w];
    __syncthreads();
    if (threadIdx.x == 0) {
      const int k = x.list >= 0 ? x.list / pieces : -1;
      write_beam(res, (int64_t)b * K + r, k, k >= 0 && s_kind[k] == 2, x.score, place_token(x.at));
    }
    if (x.list >= 0 && x.list % kBeamThreads == (int)threadIdx.x) {
      head[x.list] += 1;
      find(own);
    }
  }
}

int beam_pieces(int V, dd_dtype dtype) {
  const int piece = dtype == DD_BF16 ? beam_piece<__nv_bfloat16>() : beam_piece<float>();
  return (V + piece - 1) / piece;
}

template <typename T>
cudaError_t launch_scan(const BeamCall& p, unsigned grid, int pieces, float2* ml, uint2* cand,
                        cudaStream_t stream) {
  beam_scan_kernel<T><<<grid, kScanThreads, kPieceBytes, stream>>>(
      static_cast<const T*>(p.logits), p.K, p.V, p.ld, pieces, p.score_in, p.done_in, ml, cand, spin_limit());
  return cudaGetLastError();
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
  cudaError_t e = p.dtype == DD_BF16 ? launch_scan<__nv_bfloat16>(p, (unsigned)lists, pieces, ml, cand, stream)
                                     : launch_scan<float>(p, (unsigned)lists, pieces, ml, cand, stream);
  if (e != cudaSuccess) return e;
  static thread_local int configured_for = -1;
  if (configured_for != device_info().device) {
    e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kBeamMaxK * (kBeamMaxV / beam_piece<float>()));
    if (e != cudaSuccess) return e;
    configured_for = device_info().device;
  }
  const BeamOut res{p.parent, p.token, p.score_out, p.done_out, p.eos};
  return launch_dependent(beam_merge_kernel, dim3(p.B), dim3(kBeamThreads), (size_t)p.K * pieces, stream, p.K, pieces,
                          p.score_in, p.done_in, (const float2*)ml, (const uint2*)cand, res);
}

}  // namespace dd
