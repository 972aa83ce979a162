// C ABI of rotary positions and of the cache in 8 or 4 bits (declared in
// spd.h): argument checks, the split of the work over the GPU and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "api_util.h"
#include "quant.h"
#include "spd.h"
#include "spd_internal.h"

using namespace spd;

namespace {

constexpr int kMaxTokens = 1 << 28;
constexpr long long kMaxPlaces = 1LL << 30;  // tiles of one attention launch

bool aligned(const void *p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
bool bad_stride(long long s, long long row) { return s < row || s % 8 || s > (1LL << 31); }

const char *check_table(const spd_rotary_table *t) {
  if (!t) return "the rotary table is NULL";
  if ((t->head_dim != 64 && t->head_dim != 128) || t->rotary_dim < 16 || t->rotary_dim % 16 ||
      t->rotary_dim > t->head_dim || t->axes < 1 || t->axes > 4 ||
      (t->neighbours != 0 && t->neighbours != 1))
    return "the rotary table was not made by spd_rotary_make";
  for (int i = 0; i < t->rotary_dim / 2; ++i)
    if (t->axis[i] >= t->axes) return "the rotary table was not made by spd_rotary_make";
  return nullptr;
}

spd_status need_quant(spd_ctx *c, const CtxView &v) {
  if (v.quant) return SPD_OK;
  return fail_message(c, SPD_ERR_INVALID_ARG, "the context has no kv_quant");
}

// CTAs that share a tile's heads, kQuantWriteWarps at once each: as many as make 14 CTAs an SM;
// each makes the tile's sines again.  (2,048 tokens of 32 and 8 heads of 128 channels into 8 bits
// 16.9 us, 17.6 with 6; 4,096, where the queries are in the launch, 30.8 and 26.2; 8,192 into 4 bits
// 54.1 and 56.9, 16,385 92.0 and 95.0; 30 is as 14.)
int parts_of(long long tiles, int works, int sms) {
  const int most = (works + kQuantWriteWarps - 1) / kQuantWriteWarps;
  return (int)std::max<long long>(1, std::min<long long>(most, 14LL * sms / std::max(tiles, 1LL)));
}

// A rotary launch takes up to kRotaryTokens tokens a CTA, fewer where that leaves SMs idle.
int rotary_tokens(long long n, int sms) {
  return (int)std::max(1LL, std::min<long long>(kRotaryTokens, n / (4 * sms)));
}

// Tiles that tokens [first, first + n) touch.
long long tiles_of(long long first, long long n) {
  return (first + n + kQuantTile - 1) / kQuantTile - first / kQuantTile;
}

}  // namespace

namespace spd {

// Queries of few tokens are rotated by the appending launch, those of many by one of their own,
// whose threads need a third of the registers.  Tokens of 32 query heads, apart and together: with 8
// kv heads of 128 channels in 8 bits 2,048 tokens 22.0 and 16.7 us, 4,096 27.2 and 31.2, 4,880 29.9
// and 33.9, 16,385 79.6 and 88.7; in 4 bits 27.0 and 21.5, 31.1 and 36.2, 34.1 and 40.0, 92.6 and
// 100.7; with 4 kv heads of 64 channels in 4 bits 14.7 and 11.0, 16.7 and 16.4, 17.3 and 16.8, 38.0
// and 43.7.  Before a launch of their own the new pages go by themselves (16,385 tokens with reading
// back 102 us, 105 with the pages in the second launch).
static bool queries_apart(const QuantWrite &w, long long tiles, int sms) {
  return w.table && tiles > 2LL * sms;
}

bool quant_takes(spd_ctx *c, const QuantWrite &w, const int *ids, int n, int n_tokens,
                 const PtUpdate *updates, int n_updates) {
  if (n > kQuantSeqs || n_updates > kQuantUpdates) return false;
  CtxView v;
  ctx_view(c, &v);
  long long tiles = 0;
  for (int i = 0; i < n; ++i) tiles += tiles_of(seq_length(c, ids[i]), n_tokens);
  if (queries_apart(w, tiles, v.num_sms)) return false;
  // entries of one sequence follow one another, in order
  for (int u = 1; u < n_updates; ++u) {
    const bool same = updates[u].slot == updates[u - 1].slot;
    if (same ? updates[u].index != updates[u - 1].index + 1 : false) return false;
    for (int k = 0; !same && k + 1 < u; ++k)
      if (updates[k].slot == updates[u].slot) return false;
  }
  return true;
}

// Writes n_tokens tokens of each listed sequence (their pages are there, the context's device is
// current); lengths are the caller's to set.
spd_status quant_append(spd_ctx *c, const QuantWrite &w, const int *ids, int n, int n_tokens,
                        const PtUpdate *updates, int n_updates, cudaStream_t st) {
  CtxView v;
  const spd_status r = ctx_device(c, st, &v);
  if (r != SPD_OK) return r;
  const spd_config &cfg = *v.cfg;
  for (int b = 0; b < n; b += kQuantSeqs) {
    static thread_local QuantAppendParams p;
    p.n_seqs = std::min(kQuantSeqs, n - b);
    long long tiles = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
      const long long L = seq_length(c, ids[b + i]);
      p.seqs[i] = QuantAppendSeq{ids[b + i], (int)L, (int)tiles, 0, 0, 0};
      tiles += tiles_of(L, n_tokens);
    }
    p.n_updates = n_updates;  // (one launch where there are any: quant_takes)
    for (int u = 0, at = 0; u < n_updates; ++u) {
      p.updates[u] = updates[u];
      if (u > 0 && updates[u].slot == updates[at].slot) continue;
      at = u;
      int many = 1;
      while (u + many < n_updates && updates[u + many].slot == updates[u].slot) ++many;
      for (int i = 0; i < p.n_seqs; ++i)
        if (p.seqs[i].slot == updates[u].slot) {
          p.seqs[i].page = updates[u].index;
          p.seqs[i].pages = many;
          p.seqs[i].upd = u;
        }
    }
    const bool apart = queries_apart(w, tiles, v.num_sms);
    p.hq = w.table && !apart ? cfg.num_q_heads : 0;
    p.parts = parts_of(tiles, cfg.num_kv_heads + p.hq, v.num_sms);
    if (tiles * p.parts > 0x7fffffffLL)
      return fail_message(c, SPD_ERR_CAPACITY, "append too large for one launch");
    if (w.table) p.table = *w.table;
    p.rotate = w.table != nullptr;
    p.k = w.k;
    p.v = w.v;
    p.q = w.q;
    p.q_out = w.q_out;
    p.k_stride = w.k_stride;
    p.v_stride = w.v_stride;
    p.q_stride = w.q_stride;
    p.positions = w.positions;
    p.pool = v.buf->k_pool;
    p.page_table = static_cast<int *>(v.buf->page_table);
    p.err = v.err;
    p.n_tokens = n_tokens;
    p.hkv = cfg.num_kv_heads;
    p.P = cfg.physical_page;
    p.max_pp = v.max_pp;
    p.num_phys = cfg.num_physical_pages;
    p.total_seqs = n;
    p.seq0 = b;
    p.tiles = (int)tiles;
    cudaError_t e = cudaSuccess;
    if (apart) {
      static thread_local RotaryParams x;
      static thread_local RotaryPlaces places;
      const long long before = (long long)b * n_tokens, row = (long long)cfg.num_q_heads * cfg.head_dim;
      if ((long long)p.n_seqs * n_tokens > 0x7fffffffLL)
        return fail_message(c, SPD_ERR_CAPACITY, "append too large for one launch");
      x.table = *w.table;
      x.q = static_cast<const char *>(w.q) + 2 * before * w.q_stride;
      x.q_out = static_cast<char *>(w.q_out) + 2 * before * row;
      x.q_stride = w.q_stride;
      x.q_out_stride = row;
      x.positions = w.positions ? w.positions + before : nullptr;
      x.axis_stride = (long long)n * n_tokens;
      x.n = p.n_seqs * n_tokens;
      x.hq = cfg.num_q_heads;
      x.tokens_per_cta = rotary_tokens(x.n, v.num_sms);
      places.n_tokens = n_tokens;
      for (int i = 0; i < p.n_seqs; ++i) places.first[i] = p.seqs[i].first;
      e = launch_rotary(x, w.positions ? nullptr : &places, cfg.dtype, st);
      note_launches(c, st, 1);
    }
    if (e == cudaSuccess) {
      e = launch_quant_append(p, cfg.dtype, cfg.head_dim, v.quant, st);
      note_launches(c, st, 1);
    }
    if (e != cudaSuccess) return fail_message(c, SPD_ERR_CUDA, cudaGetErrorString(e));
  }
  return SPD_OK;
}

}  // namespace spd

extern "C" {

spd_status spd_rotary_make(const spd_rotary_rule *r, spd_rotary_table *out) {
  if (!r || !out) return SPD_ERR_INVALID_ARG;
  if ((r->head_dim != 64 && r->head_dim != 128) || r->rotary_dim < 16 || r->rotary_dim % 16 ||
      r->rotary_dim > r->head_dim || r->axes < 1 || r->axes > 4)
    return SPD_ERR_INVALID_ARG;
  if ((r->axes_in_turn != 0 && r->axes_in_turn != 1) || (r->neighbours != 0 && r->neighbours != 1))
    return SPD_ERR_INVALID_ARG;
  const int pairs = r->rotary_dim / 2;
  int left[4] = {0, 0, 0, 0}, sum = 0;
  for (int a = 0; a < r->axes; ++a) {
    if (r->sections[a] < 0 || r->sections[a] > pairs) return SPD_ERR_INVALID_ARG;
    sum += left[a] = r->sections[a];
  }
  if (sum != pairs) return SPD_ERR_INVALID_ARG;
  if (!r->inv_freq && !(r->base >= 1.0 && r->base <= 1e300)) return SPD_ERR_INVALID_ARG;
  if (r->inv_freq)
    for (int i = 0; i < pairs; ++i)
      if (!(r->inv_freq[i] >= 0.0 && r->inv_freq[i] <= 1000.0)) return SPD_ERR_INVALID_ARG;
  spd_rotary_table t;
  memset(&t, 0, sizeof t);
  t.head_dim = r->head_dim;
  t.rotary_dim = r->rotary_dim;
  t.axes = r->axes;
  t.neighbours = r->neighbours;
  int a = 0;
  for (int i = 0; i < pairs; ++i) {
    while (left[a] == 0) a = (a + 1) % r->axes;
    t.axis[i] = (unsigned char)a;
    --left[a];
    if (r->axes_in_turn) a = (a + 1) % r->axes;
    const double f = r->inv_freq ? r->inv_freq[i] : std::pow(r->base, -2.0 * i / r->rotary_dim);
    const double turns = f / 6.283185307179586476925286766559;
    const double x = std::nearbyint(std::ldexp(turns - std::floor(turns), 64));
    t.turns[i] = x >= 18446744073709551616.0 ? 0ull : (unsigned long long)x;
  }
  *out = t;
  return SPD_OK;
}

spd_status spd_rotary(const spd_rotary_table *table, spd_dtype dtype, int n_tokens,
                      const int *positions, const void *q, long long q_stride, int q_heads,
                      const void *k, long long k_stride, int kv_heads, void *q_out,
                      long long q_out_stride, void *k_out, long long k_out_stride, int inverse,
                      spd_stream stream) {
  if (check_table(table) || (dtype != SPD_F16 && dtype != SPD_BF16) || n_tokens < 1 ||
      !aligned(positions, 4) || (inverse != 0 && inverse != 1))
    return SPD_ERR_INVALID_ARG;
  const bool has_k = k || k_out;
  const int hkv = has_k ? kv_heads : 0;
  if (q_heads < 1 || q_heads > 1024 || (has_k && (kv_heads < 1 || kv_heads > 1024)))
    return SPD_ERR_INVALID_ARG;
  const long long qr = (long long)q_heads * table->head_dim, kr = (long long)hkv * table->head_dim;
  if (!aligned(q, 16) || !aligned(q_out, 16) || bad_stride(q_stride, qr) ||
      bad_stride(q_out_stride, qr))
    return SPD_ERR_INVALID_ARG;
  if (has_k && (!aligned(k, 16) || !aligned(k_out, 16) || bad_stride(k_stride, kr) ||
                bad_stride(k_out_stride, kr)))
    return SPD_ERR_INVALID_ARG;
  if ((q == q_out && q_stride != q_out_stride) || (has_k && k == k_out && k_stride != k_out_stride))
    return SPD_ERR_INVALID_ARG;
  if (n_tokens > kMaxTokens) return SPD_ERR_CAPACITY;
  int device = 0;
  if (!device_of(q_out, &device)) return SPD_ERR_INVALID_ARG;
  DeviceGuard guard;
  const spd_status s = guard.bind(device);
  if (s != SPD_OK) return s;
  static thread_local RotaryParams p;
  p.table = *table;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.positions = positions;
  p.n = n_tokens;
  p.hq = q_heads;
  p.hkv = hkv;
  p.inverse = inverse;
  p.axis_stride = n_tokens;
  p.tokens_per_cta = rotary_tokens(n_tokens, sm_count(device));
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = launch_rotary(p, nullptr, dtype, st);
  note_prompt_launch(st);
  return e == cudaSuccess ? SPD_OK : SPD_ERR_CUDA;
}

spd_status spd_kv_append_rotary(spd_ctx *c, const spd_rotary_table *table, const int *seq_ids,
                                int n_seqs, int n_tokens, const int *positions, const void *q,
                                long long q_stride, const void *k, long long k_stride,
                                const void *v, long long v_stride, void *q_out,
                                spd_stream stream) {
  if (!c) return SPD_ERR_INVALID_ARG;
  CtxView w;
  ctx_view(c, &w);
  spd_status r = need_quant(c, w);
  if (r != SPD_OK) return r;
  const spd_config &cfg = *w.cfg;
  if (const char *bad = check_table(table)) return fail_message(c, SPD_ERR_INVALID_ARG, bad);
  if (table->head_dim != cfg.head_dim)
    return fail_message(c, SPD_ERR_INVALID_ARG, "the rotary table is of another head_dim");
  const long long qr = (long long)cfg.num_q_heads * cfg.head_dim,
                  kr = (long long)cfg.num_kv_heads * cfg.head_dim;
  if (!aligned(q, 16) || !aligned(q_out, 16) || bad_stride(q_stride, qr) ||
      bad_stride(k_stride, kr) || bad_stride(v_stride, kr))
    return fail_message(c, SPD_ERR_INVALID_ARG,
                        "q, k, v and q_out must be 16-byte aligned, strides multiples of 8 and at "
                        "least a row");
  if (q == q_out && q_stride != qr)
    return fail_message(c, SPD_ERR_INVALID_ARG, "q_out may be q only where its rows are contiguous");
  if (positions && !aligned(positions, 4))
    return fail_message(c, SPD_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  QuantWrite x{};
  x.table = table;
  x.k = k;
  x.v = v;
  x.q = q;
  x.q_out = q_out;
  x.k_stride = k_stride;
  x.v_stride = v_stride;
  x.q_stride = q_stride;
  x.positions = positions;
  return append_quantised(c, x, seq_ids, n_seqs, n_tokens, (cudaStream_t)stream);
}

spd_status spd_kv_read(spd_ctx *c, const int *seq_ids, int n_seqs, int begin, int n_tokens,
                       void *k, void *v, spd_stream stream) {
  if (!c) return SPD_ERR_INVALID_ARG;
  CtxView w;
  ctx_view(c, &w);
  spd_status r = need_quant(c, w);
  if (r != SPD_OK) return r;
  if (n_tokens < 1 || !aligned(k, 16) || !aligned(v, 16))
    return fail_message(c, SPD_ERR_INVALID_ARG,
                        "n_tokens >= 1 and 16-byte aligned k and v required");
  if ((r = check_live(c, seq_ids, n_seqs)) != SPD_OK) return r;
  for (int i = 0; i < n_seqs; ++i) {
    const long long L = seq_length(c, seq_ids[i]), first = begin < 0 ? L + begin : begin;
    if (first < 0 || first + n_tokens > L)
      return fail_message(c, SPD_ERR_CAPACITY, "a sequence does not hold all of these tokens");
  }
  const cudaStream_t st = (cudaStream_t)stream;
  if ((r = ctx_device(c, st, &w)) != SPD_OK) return r;
  DeviceGuard guard;
  if ((r = guard.bind(w.device)) != SPD_OK) return fail_message(c, r, "cudaSetDevice failed");
  const spd_config &cfg = *w.cfg;
  const size_t row = (size_t)n_tokens * cfg.num_kv_heads * cfg.head_dim * 2;  // of a sequence
  for (int b = 0; b < n_seqs; b += kQuantSeqs) {
    static thread_local QuantReadParams p;
    p.n_seqs = std::min(kQuantSeqs, n_seqs - b);
    long long tiles = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
      const long long L = seq_length(c, seq_ids[b + i]), first = begin < 0 ? L + begin : begin;
      p.seqs[i] = QuantSeq{seq_ids[b + i], (int)first, (int)tiles};
      tiles += tiles_of(first, n_tokens);
    }
    if (tiles * 2 * cfg.num_kv_heads > 0x7fffffffLL)
      return fail_message(c, SPD_ERR_CAPACITY, "read too large for one launch");
    p.pool = w.buf->k_pool;
    p.k = static_cast<char *>(k) + (size_t)b * row;
    p.v = static_cast<char *>(v) + (size_t)b * row;
    p.page_table = static_cast<const int *>(w.buf->page_table);
    p.err = w.err;
    p.n_tokens = n_tokens;
    p.hkv = cfg.num_kv_heads;
    p.P = cfg.physical_page;
    p.max_pp = w.max_pp;
    p.num_phys = cfg.num_physical_pages;
    p.tiles = (int)tiles;
    const cudaError_t e = launch_quant_read(p, cfg.dtype, cfg.head_dim, w.quant, st);
    note_launches(c, st, 1);
    if (e != cudaSuccess) return fail_message(c, SPD_ERR_CUDA, cudaGetErrorString(e));
  }
  return SPD_OK;
}

spd_status spd_quant_decode_attention(spd_ctx *c, const void *q, const int *seq_ids, int n_seqs,
                                      int window, const spd_score_rule *rule, spd_out out_type,
                                      void *out, spd_stream stream) {
  if (!c) return SPD_ERR_INVALID_ARG;
  CtxView v;
  ctx_view(c, &v);
  spd_status r = need_quant(c, v);
  if (r != SPD_OK) return r;
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail_message(c, SPD_ERR_INVALID_ARG, "q and out must be 16-byte aligned pointers");
  if (out_type != SPD_OUT_F32 && out_type != SPD_OUT_DTYPE)
    return fail_message(c, SPD_ERR_INVALID_ARG, "out_type must be SPD_OUT_F32 or SPD_OUT_DTYPE");
  if (window < 0) return fail_message(c, SPD_ERR_INVALID_ARG, "window must be >= 0");
  if (const char *bad = check_rule(rule)) return fail_message(c, SPD_ERR_INVALID_ARG, bad);
  if ((r = check_live(c, seq_ids, n_seqs)) != SPD_OK) return r;
  for (int i = 0; i < n_seqs; ++i)
    if (seq_length(c, seq_ids[i]) < 1)
      return fail_message(c, SPD_ERR_STATE, "a sequence has no tokens");
  const cudaStream_t st = (cudaStream_t)stream;
  if ((r = ctx_device(c, st, &v)) != SPD_OK) return r;
  DeviceGuard guard;
  if ((r = guard.bind(v.device)) != SPD_OK) return fail_message(c, r, "cudaSetDevice failed");
  const spd_config &cfg = *v.cfg;
  const size_t oe = out_type == SPD_OUT_F32 ? 4 : 2, row = (size_t)cfg.num_q_heads * cfg.head_dim;
  const int Hkv = cfg.num_kv_heads, most_ctas = std::min(kQuantCtas, kQuantPerSm * v.num_sms);
  for (int b = 0; b < n_seqs;) {
    static thread_local QuantAttendParams p;
    // as many sequences as fit one launch
    int n = 0;
    long long total = 0;
    while (n < kQuantSeqs && b + n < n_seqs) {
      const int L = (int)seq_length(c, seq_ids[b + n]);
      const int first = window > 0 && window < L ? L - window : 0;
      const int tiles = (int)tiles_of(first, L - first);
      if (n > 0 && total + (long long)tiles * Hkv > kMaxPlaces) break;
      p.seqs[n] = QuantAttendSeq{seq_ids[b + n], L, first, tiles, tiles, 0};
      total += (long long)tiles * Hkv;
      ++n;
    }
    if (total > kMaxPlaces)
      return fail_message(c, SPD_ERR_CAPACITY, "a sequence is too long for one launch");
    // Every warp takes per_warp tiles, whole steps of them.  Where one step (or a sixteenth) more
    // lets all units begin at a CTA of their own they do, so that no unit has a stray part
    // elsewhere, and fewer are joined over CTAs: 16 windows of 4,096 tokens that begin inside a tile
    // (257 tiles a unit) take 29.9 us with 22 tiles a warp on 128 CTAs, 33.0 with 20 on all SMs (fp32
    // out; 27.0 and 29.5 for 16 bits).
    const long long warps = (long long)most_ctas * kQuantWarps;
    const int step = quant_step_tiles(cfg.head_dim);
    p.per_warp = (int)((total + warps - 1) / warps + step - 1) / step * step;
    auto ctas_of = [&](int per_warp) {  // with units that begin at CTAs
      long long k = 0;
      for (int i = 0; i < n; ++i)
        k += (long long)Hkv * ((p.seqs[i].tiles + per_warp * kQuantWarps - 1) /
                               (per_warp * kQuantWarps));
      return k;
    };
    int whole = p.per_warp;
    const int give = std::max(whole + whole / 16, whole + step);
    while (whole < give && ctas_of(whole) > most_ctas) whole += step;
    if (ctas_of(whole) <= most_ctas) {
      p.per_warp = whole;
      const int per_cta = whole * kQuantWarps;
      for (int i = 0; i < n; ++i)
        p.seqs[i].stride = (p.seqs[i].tiles + per_cta - 1) / per_cta * per_cta;
    }
    long long places = 0;
    for (int i = 0; i < n; ++i) {
      p.seqs[i].off = (int)places;
      places += (long long)p.seqs[i].stride * Hkv;
    }
    p.total = (int)places;
    p.ctas = (int)((places + (long long)p.per_warp * kQuantWarps - 1) /
                   ((long long)p.per_warp * kQuantWarps));
    p.pool = v.buf->k_pool;
    p.q = static_cast<const char *>(q) + (size_t)b * row * 2;
    p.out = static_cast<char *>(out) + (size_t)b * row * oe;
    p.page_table = static_cast<const int *>(v.buf->page_table);
    p.parts = v.parts;
    p.firsts = v.firsts;
    p.tickets = v.tickets;
    p.err = v.err;
    p.rule = make_rule(rule, cfg.head_dim);
    p.out_f32 = out_type == SPD_OUT_F32;
    p.precise_cap = p.out_f32 || cfg.dtype == SPD_F16 || !p.rule.rough;
    p.n = n;
    p.hkv = Hkv;
    p.P = cfg.physical_page;
    p.max_pp = v.max_pp;
    p.num_phys = cfg.num_physical_pages;
    const auto launch = cfg.dtype == SPD_F16 ? launch_quant_attend_f16 : launch_quant_attend_bf16;
    const cudaError_t e = launch(p, cfg.head_dim, v.quant, v.G, st);
    note_launches(c, st, 1);
    if (e != cudaSuccess) return fail_message(c, SPD_ERR_CUDA, cudaGetErrorString(e));
    b += n;
  }
  return SPD_OK;
}

}  // extern "C"
