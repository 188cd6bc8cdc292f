// C ABI of the cached-decoding operators (include/dd.h): argument validation and launches.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "dd_common.cuh"
#include "dd_internal.h"

using namespace dd;

namespace {

// Sizes, alignment and strides every call on a paged cache checks.
dd_status check_cache(const dd_paged_cache* c) {
  if (!c || !c->k || !c->v || !c->page_table) return DD_ERR_INVALID_ARG;
  if (!valid_dtype(c->dtype)) return DD_ERR_INVALID_ARG;
  if (c->layers < 1 || c->n_pages < 1 || c->page_size < 1 || c->Hkv < 1 || c->max_pages < 1)
    return DD_ERR_INVALID_ARG;
  if (c->d < 1) return DD_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return DD_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return DD_ERR_INVALID_ARG;
  const int64_t e = (int64_t)elem_size(c->dtype);
  for (const int64_t s : {c->layer_stride, c->page_stride, c->token_stride, c->head_stride})
    if (s < 0 || s > (1ll << 60) || (s * e) % 16 != 0) return DD_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages) return DD_ERR_INVALID_ARG;
  return DD_OK;
}

// Slots a table row has room for.
int64_t table_slots(const dd_paged_cache* c) { return (int64_t)c->max_pages * c->page_size; }

using wide = __int128;  // offsets of any strides
wide floor_div(wide a, wide b) { return a / b - (a % b < 0); }

// n rows of `bytes` each, `stride` bytes apart: what a call reads or writes of an argument.
struct Rows {
  uintptr_t at, end;  // all of them lie in [at, end); empty where there is none
  int64_t n, bytes, stride;
  Rows(const void* p, int64_t rows, int64_t row_bytes, int64_t row_stride)
      : at(reinterpret_cast<uintptr_t>(p)), end(at), n(rows), bytes(row_bytes), stride(row_stride) {
    int64_t extent;
    if (p && (__builtin_mul_overflow(n - 1, stride, &extent) || __builtin_add_overflow(extent, bytes, &extent) ||
              __builtin_add_overflow(at, (uintptr_t)extent, &end)))
      end = UINTPTR_MAX;
  }
};
Rows flat(const void* p, int64_t bytes) { return Rows(p, 1, bytes, bytes); }

// Whether a row of x and a row of y, whose extents meet, have a byte in common: rows of one
// may lie between those of the other (columns of a wider table).
bool rows_meet(const Rows& x, const Rows& y) {
  if (x.n > y.n) return rows_meet(y, x);
  const wide step = y.n > 1 ? y.stride : 1;
  for (int64_t i = 0; i < x.n; ++i) {  // rows j of y with j step in (lo - y.bytes, lo + x.bytes)
    const wide lo = (wide)x.at + (wide)i * x.stride - (wide)y.at;
    const wide first = floor_div(lo - y.bytes, step) + 1, last = floor_div(lo + x.bytes - 1, step);
    if (std::max<wide>(first, 0) <= std::min<wide>(last, y.n - 1)) return true;
  }
  return false;
}
bool overlap(const Rows& x, const Rows& y) { return x.at < y.end && y.at < x.end && rows_meet(x, y); }

// Whether an output lies in the memory of an input or of another output. CTAs read inputs
// while others write, so such a call would depend on timing.
bool clash(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows& in : ins)
      if (overlap(*o, in)) return true;
    for (auto other = o + 1; other != outs.end(); ++other)
      if (overlap(*o, *other)) return true;
  }
  return false;
}

Rows table_rows(const dd_paged_cache* c, int64_t n) {
  return Rows(c->page_table, n, (int64_t)c->max_pages * 4, c->table_stride * 4);
}

}  // namespace

extern "C" {

size_t dd_paged_attention_workspace_size(int B, int Hq, int Hkv, int d, int max_len,
                                         int with_mass) {
  if (B < 1 || Hq < 1 || Hkv < 1 || d < 1 || max_len < 1 || Hq % Hkv != 0) return 0;
  if (max_len > kPagedMaxLen) return 0;
  return paged_attention_workspace(B, Hq, Hkv, d, max_len, with_mass != 0);
}

dd_status dd_paged_attention(const void* q, int64_t q_stride, const void* k_new,
                             const void* v_new, int64_t new_stride, const dd_paged_cache* cache,
                             const int32_t* lengths, int B, int Hq, int max_len,
                             float softmax_scale, void* out, float* lse, const float* mass_in,
                             float* mass_out, int64_t mass_stride, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const dd_status st = check_cache(cache);
  if (st != DD_OK) return st;
  if (!q || !lengths || !out || cache->layers != 1) return DD_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hq % cache->Hkv != 0) return DD_ERR_INVALID_ARG;
  if (max_len < 1 || max_len > table_slots(cache)) return DD_ERR_INVALID_ARG;
  if (!k_new != !v_new) return DD_ERR_INVALID_ARG;
  const int64_t e = (int64_t)elem_size(cache->dtype);
  if (!aligned16(q) || !aligned16(out) || (k_new && (!aligned16(k_new) || !aligned16(v_new))))
    return DD_ERR_INVALID_ARG;
  if (B > 1 && (q_stride < (int64_t)Hq * cache->d || (q_stride * e) % 16 != 0))
    return DD_ERR_INVALID_ARG;
  if (B > 1 && k_new && (new_stride < (int64_t)cache->Hkv * cache->d || (new_stride * e) % 16 != 0))
    return DD_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || isinf(softmax_scale)) return DD_ERR_INVALID_ARG;
  if (!mass_out && mass_in) return DD_ERR_INVALID_ARG;
  if (mass_out && mass_stride < max_len) return DD_ERR_INVALID_ARG;
  if (B > kPagedMaxBatch || Hq > kPagedMaxHeads || max_len > kPagedMaxLen) return DD_ERR_UNSUPPORTED;
  if (paged_attention_tiles(B, Hq, max_len) >= (1ll << 31)) return DD_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return DD_ERR_INVALID_ARG;
  const size_t need = paged_attention_workspace(B, Hq, cache->Hkv, cache->d, max_len, mass_out != nullptr);
  if (workspace_bytes < need) return DD_ERR_INVALID_ARG;
  // in place: a block of heads is written after its queries are read, a mass by its reader
  const int64_t q_row = (int64_t)Hq * cache->d * e, new_row = (int64_t)cache->Hkv * cache->d * e;
  const bool in_place = out == q && (B == 1 || q_stride == (int64_t)Hq * cache->d);
  if (clash({flat(out, B * q_row), flat(lse, (int64_t)B * Hq * 4), Rows{mass_out, B, (int64_t)max_len * 4, mass_stride * 4},
             flat(workspace, (int64_t)need)},
            {Rows{in_place ? nullptr : q, B, q_row, q_stride * e}, Rows{k_new, B, new_row, new_stride * e},
             Rows{v_new, B, new_row, new_stride * e}, flat(lengths, (int64_t)B * 4), table_rows(cache, B),
             Rows{mass_in == mass_out ? nullptr : mass_in, B, (int64_t)max_len * 4, mass_stride * 4}}))
    return DD_ERR_INVALID_ARG;
  PagedCall p{};
  p.q = q; p.q_stride = B > 1 ? q_stride : 0;
  p.k_new = k_new; p.v_new = v_new; p.new_stride = B > 1 ? new_stride : 0;
  p.cache = cache; p.lengths = lengths;
  p.B = B; p.Hq = Hq; p.max_len = max_len; p.scale = softmax_scale;
  p.out = out; p.lse = lse;
  p.mass_in = mass_in; p.mass_out = mass_out; p.mass_stride = mass_stride;
  p.workspace = workspace;
  return from_cuda(launch_paged_attention(p, static_cast<cudaStream_t>(stream)));
}

dd_status dd_cache_evict(const dd_paged_cache* cache, const int32_t* lengths, int N, int max_len,
                         int budget, int sink, int recent, const float* mass_in,
                         const int32_t* pos_in, int64_t stride, float* mass_out,
                         int32_t* pos_out, int32_t* src_out, int32_t* lengths_out, void* stream) {
  const dd_status st = check_cache(cache);
  if (st != DD_OK) return st;
  if (!lengths || !mass_in || !pos_in || !mass_out || !pos_out || !lengths_out)
    return DD_ERR_INVALID_ARG;
  if (cache->layers != 1 || N < 1 || max_len < 1 || max_len > table_slots(cache))
    return DD_ERR_INVALID_ARG;
  if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget)
    return DD_ERR_INVALID_ARG;
  if (stride < max_len || lengths == lengths_out || mass_in == mass_out || pos_in == pos_out)
    return DD_ERR_INVALID_ARG;
  if (N > 65535 || max_len > kEvictMaxLen) return DD_ERR_UNSUPPORTED;
  const auto rows = [&](const void* x, int slots) { return Rows{x, N, (int64_t)slots * 4, stride * 4}; };
  const int left = std::min(budget, max_len);
  if (clash({rows(mass_out, left), rows(pos_out, left), rows(src_out, left), flat(lengths_out, (int64_t)N * 4)},
            {rows(mass_in, max_len), rows(pos_in, max_len), flat(lengths, (int64_t)N * 4), table_rows(cache, N)}))
    return DD_ERR_INVALID_ARG;
  EvictCall p{cache, lengths, N, max_len, budget, sink, recent, mass_in, pos_in, stride,
              mass_out, pos_out, src_out, lengths_out};
  return from_cuda(launch_cache_evict(p, static_cast<cudaStream_t>(stream)));
}

size_t dd_beam_select_workspace_size(int B, int K, int V, dd_dtype dtype) {
  if (B < 1 || K < 1 || V < 1 || !valid_dtype(dtype)) return 0;
  if (K > kBeamMaxK || V > kBeamMaxV || (int64_t)B * K > (1ll << 20)) return 0;
  return beam_select_workspace(B, K, V, dtype);
}

dd_status dd_beam_select(const void* logits, dd_dtype dtype, int B, int K, int V, int64_t ld,
                         const float* score_in, const uint8_t* done_in, int eos, int32_t* parent,
                         int32_t* token, float* score_out, uint8_t* done_out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!logits || !score_in || !parent || !token || !score_out) return DD_ERR_INVALID_ARG;
  if (!valid_dtype(dtype) || B < 1 || K < 1 || V < 1 || ld < V) return DD_ERR_INVALID_ARG;
  if (eos < -1 || eos >= V) return DD_ERR_INVALID_ARG;
  if (!aligned16(logits) || ld > (1ll << 40) || (ld * (int64_t)elem_size(dtype)) % 16 != 0)
    return DD_ERR_INVALID_ARG;
  if (score_out == score_in || (done_out && done_out == done_in)) return DD_ERR_INVALID_ARG;
  if (K > kBeamMaxK || V > kBeamMaxV || (int64_t)B * K > (1ll << 20)) return DD_ERR_UNSUPPORTED;
  if ((int64_t)B * K * ((V + 4095) / 4096) >= (1ll << 31)) return DD_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return DD_ERR_INVALID_ARG;
  const size_t need = beam_select_workspace(B, K, V, dtype);
  if (workspace_bytes < need) return DD_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * K, e = (int64_t)elem_size(dtype);
  if (clash({flat(parent, n * 4), flat(token, n * 4), flat(score_out, n * 4), flat(done_out, n),
             flat(workspace, (int64_t)need)},
            {Rows{logits, n, V * e, ld * e}, flat(score_in, n * 4), flat(done_in, n)}))
    return DD_ERR_INVALID_ARG;
  BeamCall p{logits, dtype, B, K, V, ld, score_in, done_in, eos, parent, token, score_out,
             done_out, workspace};
  return from_cuda(launch_beam_select(p, static_cast<cudaStream_t>(stream)));
}

dd_status dd_beam_reorder(const int32_t* parent, int B, int K, const dd_row_state* states,
                          int n_states, void* stream) {
  if (!parent || !states || B < 1 || K < 1 || n_states < 1) return DD_ERR_INVALID_ARG;
  if (n_states > kMaxRowStates || (int64_t)B * K > (1ll << 20)) return DD_ERR_UNSUPPORTED;
  for (int i = 0; i < n_states; ++i) {
    const dd_row_state& s = states[i];
    if (!s.src || !s.dst || s.src == s.dst || s.row_bytes < 1) return DD_ERR_INVALID_ARG;
    if ((int64_t)B * K > 1 && (s.src_stride < s.row_bytes || s.dst_stride < s.row_bytes))
      return DD_ERR_INVALID_ARG;
  }
  const int64_t n = (int64_t)B * K;
  for (int i = 0; i < n_states; ++i) {
    const Rows dst{states[i].dst, n, states[i].row_bytes, states[i].dst_stride};
    if (overlap(dst, flat(parent, n * 4))) return DD_ERR_INVALID_ARG;
    for (int j = 0; j < n_states; ++j) {
      const dd_row_state& s = states[j];
      if (overlap(dst, Rows{s.src, n, s.row_bytes, s.src_stride}) ||
          (j > i && overlap(dst, Rows{s.dst, n, s.row_bytes, s.dst_stride})))
        return DD_ERR_INVALID_ARG;
    }
  }
  return from_cuda(
      launch_beam_reorder(parent, B, K, states, n_states, static_cast<cudaStream_t>(stream)));
}

dd_status dd_paged_fork(const dd_paged_cache* cache, const int32_t* parent, int B, int K,
                        const int32_t* lengths, const int32_t* fresh, int32_t* table_out,
                        int64_t out_stride, int32_t* lengths_out, void* stream) {
  const dd_status st = check_cache(cache);
  if (st != DD_OK) return st;
  if (!parent || !lengths || !fresh || !table_out || !lengths_out) return DD_ERR_INVALID_ARG;
  if (B < 1 || K < 1 || out_stride < cache->max_pages) return DD_ERR_INVALID_ARG;
  if (table_out == cache->page_table || lengths_out == lengths) return DD_ERR_INVALID_ARG;
  if ((int64_t)B * K > 65535) return DD_ERR_UNSUPPORTED;
  const int64_t n = (int64_t)B * K;
  if (clash({Rows{table_out, n, (int64_t)cache->max_pages * 4, out_stride * 4}, flat(lengths_out, n * 4)},
            {table_rows(cache, n), flat(parent, n * 4), flat(lengths, n * 4), flat(fresh, n * 4)}))
    return DD_ERR_INVALID_ARG;
  return from_cuda(launch_paged_fork(*cache, parent, B, K, lengths, fresh, table_out, out_stride,
                                     lengths_out, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
