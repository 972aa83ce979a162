// C ABI of dense attention with score rules (prompts, shared prefixes) and of
// eviction (declared in spd.h): argument checks, the split of the work over
// the GPU, workspace layouts and launches.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <new>

#include "api_util.h"
#include "dense.h"
#include "spd.h"
#include "spd_internal.h"

using namespace spd;

namespace {

constexpr int kMaxTokens = 1 << 28;
constexpr int kMaxKeep = 1 << 28;  // no sequence is longer (max_context is bounded by it)

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void *p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
}

// 4-D map, boxes of 128-byte rows, 128-byte swizzle.
bool encode4(CUtensorMap *m, CUtensorMapDataType t, const void *base, const cuuint64_t (&dims)[4],
             const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
  const auto encode = map_encoder();
  if (!encode) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(m, t, 4, const_cast<void *>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

CUtensorMapDataType map_type(spd_dtype t) {
  return t == SPD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Rows [tokens][heads][d] at `stride` elements, boxes of `bh` heads x `bt`
// tokens x 128 bytes of channels.
bool encode_rows(CUtensorMap *m, CUtensorMapDataType t, const void *base, int d, int heads,
                 int tokens, long long stride, int bh, int bt) {
  const cuuint64_t e = t == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2, c = 128 / e;
  const cuuint64_t dims[4] = {c, (cuuint64_t)d / c, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[3] = {128, (cuuint64_t)d * e, (cuuint64_t)stride * e};
  const cuuint32_t box[4] = {(cuuint32_t)c, 1, (cuuint32_t)bh, (cuuint32_t)bt};
  return encode4(m, t, base, dims, strides, box);
}

// Partial sums [rows][d] fp32 in boxes of a warp's 32 rows.
bool encode_partials(CUtensorMap *m, const float *base, int d, size_t rows) {
  const cuuint64_t dims[4] = {32, (cuuint64_t)d / 32, 1, (cuuint64_t)rows};
  const cuuint64_t strides[3] = {128, (cuuint64_t)d * 4, (cuuint64_t)d * 4};
  const cuuint32_t box[4] = {32, 1, 1, 32};
  return encode4(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, dims, strides, box);
}

// ---- prompt attention ------------------------------------------------------------

struct PromptPlan {
  int G = 0, HP = 0, lhp = 0, HG = 0, tiles = 0, nsplit = 1, dup = 0;
  bool partial = false;
  size_t po = 0, pml = 0, total = 0;
};

bool valid_dense(const spd_dense_config *c) {
  if (!c || c->num_kv_heads < 1 || c->num_kv_heads > kMaxKvHeads || c->num_q_heads < 1 ||
      c->num_q_heads % c->num_kv_heads)
    return false;
  if (c->num_q_heads > 1024) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->dtype != SPD_F16 && c->dtype != SPD_BF16) return false;
  if (c->out != SPD_OUT_F32 && c->out != SPD_OUT_DTYPE) return false;
  return check_rule(&c->rule) == nullptr;
}

// Heads that share K and V lie in one matrix (a power of two of them, so that
// a matrix's 128 rows hold whole tokens).  Few units over a long axis are cut
// along the keys until the GPU is full, at least four blocks per cut; at most
// 128 rows are held twice, both matrices taking turns at the keys.
spd_status plan_prompt(const spd_dense_config *c, int Lq, int Lk, int sms, PromptPlan *z) {
  if (!valid_dense(c) || Lq < 1 || Lk < 1) return SPD_ERR_INVALID_ARG;
  if (Lq > kMaxTokens || Lk > kMaxTokens) return SPD_ERR_CAPACITY;
  z->G = c->num_q_heads / c->num_kv_heads;
  while (z->lhp < 3 && z->G % (2 << z->lhp) == 0) ++z->lhp;
  z->HP = 1 << z->lhp;
  z->HG = z->G / z->HP;
  const int blocks = (Lk + kDenseBlock - 1) / kDenseBlock;
  z->dup = (long long)Lq * z->HP <= 128 && blocks >= 8 ? 1 : 0;
  const int per = (z->dup ? 128 : kDenseRows) / z->HP;
  z->tiles = (Lq + per - 1) / per;
  const long long units = (long long)z->tiles * c->num_kv_heads * z->HG;
  const int most = kDenseMaxSplits / (z->dup ? 2 : 1);
  // Cuts along the keys.  A block takes 0.85 us, a CTA 8 us besides; where the CTAs
  // of a full GPU leave partial sums, 5.2 more, and as much to join them (a fit to
  // about 30 shapes).  Over a much longer row the units are even and run in whole
  // rounds; a square causal prompt's run longest first, and either the longest or
  // the average bounds them.  (Whole and in the cuts taken: 2,048 queries over 49,152
  // keys with 32 heads 1,292 and 1,202 us, 8,192 causal with 4 heads 114 and 75,
  // 4,096 with 8 heads 62 and 53, 128 over 1,024 keys 20 and 15.  Kept whole: 7,000
  // with 8 heads 101, in two cuts 123; 2,048 with 32 heads 38 and 76; 512 13.6 and
  // 18.7.)
  const double work = Lk > Lq ? 1.0 - 0.5 * Lq / Lk : 0.5;  // of units x blocks
  auto cost = [&](long long s) {
    const bool cut = z->dup || s > 1;
    const double part = cut ? 5.2 * std::min(1.0, (double)(units * s) / sms) : 0.0;
    const double block = 0.85, fixed = 8.0 + part, join = part;
    const double one = block * blocks / (double)s + fixed;
    if (Lk >= 4LL * Lq) return (double)((units * s + sms - 1) / sms) * one + join;
    const double all = block * work * blocks * (double)units / sms +
                       (cut ? fixed * (double)(units * s) / sms : 0.0);
    return std::max(one, all) + join;
  };
  for (int s = 2; s <= most && s * 4 <= blocks && units <= 8LL * sms; ++s)
    if (cost(s) < cost(z->nsplit)) z->nsplit = s;
  z->partial = z->dup || z->nsplit > 1;
  if (units * z->nsplit > 0x7fffffffLL || (long long)Lq * c->num_q_heads > 0x7fffffffLL * 8)
    return SPD_ERR_CAPACITY;
  if (z->partial) {
    const size_t rows = (size_t)units * z->nsplit * kDenseRows;
    z->po = 0;
    z->pml = round_up(rows * c->head_dim * 4, 256);
    z->total = round_up(z->pml + rows * 8, 256);
  }
  return SPD_OK;
}

// ---- shared prefix ------------------------------------------------------------------

// Query rows (sequences x heads per kv head) of a prefix: up to kFewRows go
// with the sequences' own tokens (dense_decode), up to kManyRows over dense_few
// (128 channels; 64 stay with dense_decode), more over dense_tc.
// A brief prefix (tokens times groups of 16 rows) goes with the own tokens
// whatever its rows: one kernel (12 and 48 rows over 1,000 tokens 14 and 16 us
// against 16 and 19; 96 over 1,000 23 against 20, 12 over 4,099 20 against 18).
constexpr int kFewRows = 8, kManyRows = 32, kFewTile = 32, kBriefWork = 4000;

struct SharedPlan {
  bool tc = false, few = false;                // the prefix by dense_tc, dense_few
  bool own_first = false;                      // dense_few after the own tokens
  int tiles = 0, nsplit = 0, dup = 0;          // dense_tc
  int prefix_items = 0, prefix_ns = 0, prefix_tpi = 1, prefix_rows = 0;
  int own_items = 0, longest = 0;
  size_t pre_o = 0, pre_ml = 0, part_o = 0, part_ml = 0, logits = 0, total = 0;
};

// The split of one launch's sequences: an item gets the tiles that fill the
// CTAs that the GPU holds at once evenly, at least two per warp (of 16 keys) or
// two (of 128).
void plan_shared(const spd_ctx *c, const CtxView &v, int prefix_len, const int *ids, int n,
                 bool weights, bool f32, DecodeSeq *seqs, SharedPlan *z) {
  const int Hkv = v.cfg->num_kv_heads, d = v.cfg->head_dim, rows = n * v.G;
  const bool brief = (long long)((rows + kDecodeRows - 1) / kDecodeRows) * prefix_len <= kBriefWork;
  z->tc = !brief && rows > kManyRows;
  z->few = !brief && !z->tc && rows > kFewRows && d == 128;
  const int tk = z->few ? kFewKeys : kDecodeTile;  // keys per tile of the prefix
  z->prefix_rows = z->few ? std::min(rows, kFewTile) : kDecodeRows;
  const int pt = prefix_len > 0 && !z->tc ? (prefix_len + tk - 1) / tk : 0;
  const int pu = pt > 0 ? Hkv * ((rows + z->prefix_rows - 1) / z->prefix_rows) : 0;
  auto tiles_of = [](int tokens) { return (tokens + kDecodeTile - 1) / kDecodeTile; };
  int most = 0;
  long long own_work = 0;
  z->longest = 0;
  for (int i = 0; i < n; ++i) {
    const int L = (int)seq_length(c, ids[i]), t = tiles_of(L);
    seqs[i].slot = ids[i];
    seqs[i].L = L;
    z->longest = std::max(z->longest, L);
    most = std::max(most, t);
    own_work += (long long)Hkv * t;
  }
  // the tiles per item: one wave if whole units leave room for it (the least
  // that fit), else four finer ones
  auto per_item = [&](long long work, int longest, int per_sm, int least, auto items_for) {
    const long long slots = (long long)per_sm * v.num_sms;
    int tpi = (int)std::max<long long>(least, (work + slots - 1) / slots);
    if (items_for(std::max(longest, 1)) > slots)
      return (int)std::max<long long>(least, (work + 4 * slots - 1) / (4 * slots));
    int lo = tpi, hi = std::max(tpi, longest);
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (items_for(mid) <= slots) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };
  auto pre_items = [&](int tpi) { return (long long)pu * ((pt + tpi - 1) / tpi); };
  auto own_items = [&](int tpi) {
    long long k = 0;
    for (int i = 0; i < n; ++i) k += (long long)Hkv * ((tiles_of(seqs[i].L) + tpi - 1) / tpi);
    return k;
  };
  const long long pre_work = (long long)pu * pt;
  int tpi, tpi_pre = 1;
  if (z->few) {
    tpi = per_item(own_work, most, 2, 8, own_items);
    tpi_pre = per_item(pre_work, pt, rows <= 16 && !f32 ? 3 : 2, 2, pre_items);
    z->own_first = own_work * kDecodeTile < pre_work * kFewKeys;
  } else {
    tpi = tpi_pre = per_item(pre_work + own_work, std::max(pt, most), 2, 8,
                             [&](int x) { return pre_items(x) + own_items(x); });
  }
  tpi = std::max(tpi, (most + kOwnMaxSplits - 1) / kOwnMaxSplits);
  tpi_pre = std::max(tpi_pre, (pt + kDenseMaxSplits - 1) / kDenseMaxSplits);
  z->prefix_tpi = tpi_pre;
  z->prefix_ns = pt > 0 ? (pt + tpi_pre - 1) / tpi_pre : 0;
  z->prefix_items = pu * z->prefix_ns;
  z->own_items = 0;
  for (int i = 0; i < n; ++i) {
    const int t = tiles_of(seqs[i].L);
    seqs[i].item_off = z->own_items;
    seqs[i].ns = (t + tpi - 1) / tpi;
    seqs[i].tpi = tpi;
    z->own_items += Hkv * seqs[i].ns;
  }
  size_t pre_rows = (size_t)z->prefix_items * z->prefix_rows;
  if (z->tc) {
    const int blocks = (prefix_len + kDenseBlock - 1) / kDenseBlock;
    z->dup = rows <= 128 && blocks >= 8 ? 1 : 0;
    z->tiles = (rows + (z->dup ? 128 : kDenseRows) - 1) / (z->dup ? 128 : kDenseRows);
    const int units = z->tiles * Hkv;
    z->nsplit = std::max(1, std::min({kDenseMaxSplits / (z->dup ? 2 : 1), v.num_sms / units,
                                      blocks / 4}));
    z->prefix_rows = z->dup ? 128 : kDenseRows;
    z->prefix_ns = z->nsplit * (z->dup ? 2 : 1);
    pre_rows = (size_t)units * z->nsplit * kDenseRows;
  }
  const size_t own_rows = (size_t)z->own_items * v.G;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  z->pre_o = take(pre_rows * d * 4);
  z->pre_ml = take(pre_rows * 8);
  z->part_o = take(own_rows * d * 4);
  z->part_ml = take(own_rows * 8);
  long long tokens = 0;
  for (int i = 0; i < n; ++i) {
    seqs[i].l_off = tokens;
    tokens += (long long)round_up(seqs[i].L, 4);
  }
  z->logits = take(weights ? (size_t)tokens * Hkv * v.G * 4 : 0);
  z->total = off;
}

// Workspace of a whole call: its launches run one after the other in the same
// one.  The type of the output may change the split: the larger of both.
size_t shared_bytes(const spd_ctx *c, const CtxView &v, int prefix_id, const int *ids, int n,
                    bool weights) {
  DecodeSeq seqs[kDenseSeqs];
  size_t most = 0;
  for (int b = 0; b < n; b += kDenseSeqs)
    for (int f32 = 0; f32 < 2; ++f32) {
      SharedPlan z;
      plan_shared(c, v, prefix_id >= 0 ? (int)seq_length(c, prefix_id) : 0, ids + b,
                  std::min(kDenseSeqs, n - b), weights, f32 != 0, seqs, &z);
      most = std::max(most, z.total);
    }
  return most;
}

spd_status check_shared(spd_ctx *c, const CtxView &v, int prefix_id, const int *ids, int n) {
  if (v.Hs > 0)
    return fail_message(c, SPD_ERR_INVALID_ARG, "a context with streaming heads keeps no whole cache");
  if (v.kv_fp8) return fail_message(c, SPD_ERR_INVALID_ARG, "fp8 KV storage is not supported here");
  if (v.quant)
    return fail_message(c, SPD_ERR_INVALID_ARG, "a cache with kv_quant is attended by spd_quant_decode_attention");
  spd_status r = check_live(c, ids, n);
  if (r != SPD_OK) return r;
  long long lp = 0;
  if (prefix_id >= 0) {
    if ((r = check_live(c, &prefix_id, 1)) != SPD_OK) return r;
    for (int i = 0; i < n; ++i)
      if (ids[i] == prefix_id)
        return fail_message(c, SPD_ERR_BAD_SEQ, "the prefix is listed as a sequence too");
    lp = seq_length(c, prefix_id);
    if (lp < 1) return fail_message(c, SPD_ERR_STATE, "the prefix has no tokens");
  } else if (prefix_id != -1) {
    return fail_message(c, SPD_ERR_BAD_SEQ, "prefix_id must be a live sequence or -1");
  }
  if (lp == 0)
    for (int i = 0; i < n; ++i)
      if (seq_length(c, ids[i]) < 1)
        return fail_message(c, SPD_ERR_STATE, "a sequence has no tokens and there is no prefix");
  return SPD_OK;
}

}  // namespace

extern "C" {

spd_status spd_prefill_attention_sizes(const spd_dense_config *cfg, int q_len, int kv_len,
                                       size_t *workspace_bytes) {
  PromptPlan z;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) (void)cudaGetLastError();
  const spd_status s = plan_prompt(cfg, q_len, kv_len, sm_count(device), &z);
  if (s != SPD_OK) return s;
  if (workspace_bytes) *workspace_bytes = z.total;
  return SPD_OK;
}

spd_status spd_prefill_attention(const spd_dense_config *cfg, int q_len, int kv_len, const void *q,
                                 long long q_stride, const void *k, long long k_stride,
                                 const void *v, long long v_stride, const int *key_begin,
                                 const int *key_end, void *out, void *workspace,
                                 size_t workspace_bytes, spd_stream stream) {
  if (!valid_dense(cfg) || q_len < 1 || kv_len < 1) return SPD_ERR_INVALID_ARG;
  const long long qrow = (long long)cfg->num_q_heads * cfg->head_dim,
                  kvrow = (long long)cfg->num_kv_heads * cfg->head_dim;
  for (long long x : {q_stride, k_stride, v_stride})
    if (x % 8 || x > (1LL << 32)) return SPD_ERR_INVALID_ARG;
  if (q_stride < qrow || k_stride < kvrow || v_stride < kvrow) return SPD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      (key_begin == nullptr) != (key_end == nullptr) ||
      (key_begin && (!aligned(key_begin, 4) || !aligned(key_end, 4))))
    return SPD_ERR_INVALID_ARG;
  int device = 0;
  if (!device_of(out, &device)) return SPD_ERR_INVALID_ARG;
  PromptPlan z;
  spd_status s = plan_prompt(cfg, q_len, kv_len, sm_count(device), &z);
  if (s != SPD_OK) return s;
  if (z.partial) {
    int wd = -1;
    if (!aligned(workspace, 256) || !device_of(workspace, &wd) || wd != device)
      return SPD_ERR_INVALID_ARG;
    if (workspace_bytes < z.total) return SPD_ERR_CAPACITY;
  }
  DeviceGuard guard;
  if ((s = guard.bind(device)) != SPD_OK) return s;
  DenseTcParams p{};
  const int d = cfg->head_dim;
  const CUtensorMapDataType mt = map_type(cfg->dtype);
  float *part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + z.po);
  if (!encode_rows(&p.tm_q, mt, q, d, cfg->num_q_heads, q_len, q_stride, z.HP, 128 / z.HP) ||
      !encode_rows(&p.tm_k, mt, k, d, cfg->num_kv_heads, kv_len, k_stride, 1, kDenseBlock) ||
      !encode_rows(&p.tm_v, mt, v, d, cfg->num_kv_heads, kv_len, v_stride, 1, kDenseBlock) ||
      !(z.partial ? encode_partials(&p.tm_out, part_o, d,
                                    (size_t)z.tiles * cfg->num_kv_heads * z.HG * z.nsplit * kDenseRows)
                  : encode_rows(&p.tm_out, cfg->out == SPD_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : mt,
                                out, d, cfg->num_q_heads, q_len, qrow, z.HP, 32 / z.HP)))
    return SPD_ERR_CUDA;
  p.partial = z.partial;
  p.part_o = part_o;
  p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + z.pml);
  p.v = v;
  p.v_stride = v_stride;
  p.key_begin = key_begin;
  p.key_end = key_end;
  p.rule = make_rule(&cfg->rule, d);
  p.out_f32 = cfg->out == SPD_OUT_F32;
  p.Lq = q_len;
  p.Lk = kv_len;
  p.Hq = cfg->num_q_heads;
  p.Hkv = cfg->num_kv_heads;
  p.G = z.G;
  p.lhp = z.lhp;
  p.HG = z.HG;
  p.tiles = z.tiles;
  p.nsplit = z.nsplit;
  p.dup = z.dup;
  p.pos0 = kv_len - q_len;
  cudaStream_t st = (cudaStream_t)stream;
  note_prompt_launch(st);
  if (launch_dense_tc(p, cfg->dtype, d, p.out_f32 != 0, st) != cudaSuccess) return SPD_ERR_CUDA;
  if (z.partial && launch_dense_prompt_combine(p, cfg->dtype, d, out, st) != cudaSuccess)
    return SPD_ERR_CUDA;
  return SPD_OK;
}

spd_status spd_prefill_attention_check(const void *out, spd_stream stream) {
  int device = 0;
  if (!out || !device_of(out, &device)) return SPD_ERR_INVALID_ARG;
  DeviceGuard guard;
  const spd_status s = guard.bind(device);
  if (s != SPD_OK) return s;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return SPD_ERR_CUDA;
  int w[4] = {0, 0, 0, 0};
  if (dense_error_word(w) != cudaSuccess) return SPD_ERR_CUDA;
  return w[0] == 0 ? SPD_OK : SPD_ERR_DEVICE_CHECK;
}

spd_status spd_document_key_ranges(const int *offsets, const int *prefix, int n_docs, int n_tokens,
                                   int *key_begin, int *key_end, spd_stream stream) {
  if (!aligned(offsets, 4) || (prefix && !aligned(prefix, 4)) || !aligned(key_begin, 4) ||
      !aligned(key_end, 4) || n_docs < 1 || n_tokens < 1 || n_tokens > kMaxTokens)
    return SPD_ERR_INVALID_ARG;
  int device = 0;
  if (!device_of(key_end, &device)) return SPD_ERR_INVALID_ARG;
  DeviceGuard guard;
  const spd_status s = guard.bind(device);
  if (s != SPD_OK) return s;
  note_prompt_launch((cudaStream_t)stream);
  return launch_document_ranges(offsets, prefix, n_docs, n_tokens, key_begin, key_end,
                                (cudaStream_t)stream) == cudaSuccess
             ? SPD_OK
             : SPD_ERR_CUDA;
}

spd_status spd_shared_prefix_sizes(spd_ctx *c, int prefix_id, const int *seq_ids, int n_seqs,
                                   int weights, size_t *workspace_bytes) {
  if (!c || !workspace_bytes) return SPD_ERR_INVALID_ARG;
  CtxView v;
  ctx_view(c, &v);
  const spd_status r = check_shared(c, v, prefix_id, seq_ids, n_seqs);
  if (r != SPD_OK) return r;
  v.num_sms = sm_count(v.device);
  *workspace_bytes = shared_bytes(c, v, prefix_id, seq_ids, n_seqs, weights != 0);
  return SPD_OK;
}

spd_status spd_shared_prefix_attention(spd_ctx *c, const void *q, int prefix_id,
                                       const int *seq_ids, int n_seqs, const spd_score_rule *rule,
                                       spd_out out_type, void *out, const float *weights_in,
                                       float *weights_out, long long weights_stride,
                                       void *workspace, size_t workspace_bytes,
                                       spd_stream stream) {
  if (!c) return SPD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail_message(c, SPD_ERR_INVALID_ARG, "q and out must be 16-byte aligned pointers");
  if (const char *e = check_rule(rule)) return fail_message(c, SPD_ERR_INVALID_ARG, e);
  if (out_type != SPD_OUT_F32 && out_type != SPD_OUT_DTYPE)
    return fail_message(c, SPD_ERR_INVALID_ARG, "out_type must be SPD_OUT_F32 or SPD_OUT_DTYPE");
  if (weights_in && !weights_out)
    return fail_message(c, SPD_ERR_INVALID_ARG, "weights_in needs weights_out");
  if ((weights_in && !aligned(weights_in, 4)) || (weights_out && !aligned(weights_out, 4)))
    return fail_message(c, SPD_ERR_INVALID_ARG, "weights must be 4-byte aligned");
  CtxView v;
  ctx_view(c, &v);
  spd_status r = check_shared(c, v, prefix_id, seq_ids, n_seqs);
  if (r != SPD_OK) return r;
  if (weights_out)
    for (int i = 0; i < n_seqs; ++i)
      if (seq_length(c, seq_ids[i]) > weights_stride)
        return fail_message(c, SPD_ERR_CAPACITY, "weights_stride is below a sequence's length");
  if (!aligned(workspace, 256))
    return fail_message(c, SPD_ERR_INVALID_ARG, "workspace must be a 256-byte aligned pointer");
  cudaStream_t st = (cudaStream_t)stream;
  if ((r = ctx_device(c, st, &v)) != SPD_OK) return r;
  // (a call of one launch is held to the plan that it uses, below)
  if (n_seqs > kDenseSeqs &&
      workspace_bytes < shared_bytes(c, v, prefix_id, seq_ids, n_seqs, weights_out != nullptr))
    return fail_message(c, SPD_ERR_CAPACITY, "workspace is smaller than spd_shared_prefix_sizes");
  DeviceGuard guard;
  if ((r = guard.bind(v.device)) != SPD_OK) return fail_message(c, r, "cudaSetDevice failed");
  const spd_config &cfg = *v.cfg;
  const int d = cfg.head_dim, lp = prefix_id >= 0 ? (int)seq_length(c, prefix_id) : 0;
  char *ws = static_cast<char *>(workspace);
  static thread_local DenseDecodeParams p;
  static thread_local DenseTcParams t;
  for (int b = 0; b < n_seqs; b += kDenseSeqs) {
    const int n = std::min(kDenseSeqs, n_seqs - b);
    SharedPlan z;
    plan_shared(c, v, lp, seq_ids + b, n, weights_out != nullptr, out_type == SPD_OUT_F32, p.seqs,
                &z);
    if (workspace_bytes < z.total)
      return fail_message(c, SPD_ERR_CAPACITY, "workspace is smaller than spd_shared_prefix_sizes");
    const char *qb = static_cast<const char *>(q) + (size_t)b * cfg.num_q_heads * d * 2;
    const size_t oe = out_type == SPD_OUT_F32 ? 4 : 2;
    p.tm_k = *v.tm_k;
    p.tm_v = *v.tm_v;
    p.q = qb;
    p.out = static_cast<char *>(out) + (size_t)b * cfg.num_q_heads * d * oe;
    p.part_o = reinterpret_cast<float *>(ws + z.part_o);
    p.part_ml = reinterpret_cast<float2 *>(ws + z.part_ml);
    p.pre_o = reinterpret_cast<float *>(ws + z.pre_o);
    p.pre_ml = reinterpret_cast<float2 *>(ws + z.pre_ml);
    const size_t wb = (size_t)b * cfg.num_kv_heads * weights_stride;
    p.logits = weights_out ? reinterpret_cast<float *>(ws + z.logits) : nullptr;
    p.w_in = weights_in ? weights_in + wb : nullptr;
    p.w_out = weights_out ? weights_out + wb : nullptr;
    p.page_table = static_cast<const int *>(v.buf->page_table);
    p.err = v.err;
    p.rule = make_rule(rule, d);
    p.w_stride = weights_stride;
    p.out_f32 = out_type == SPD_OUT_F32;
    p.n = n;
    p.Hq = cfg.num_q_heads;
    p.Hkv = cfg.num_kv_heads;
    p.G = v.G;
    p.P = cfg.physical_page;
    p.max_pp = v.max_pp;
    p.num_phys = cfg.num_physical_pages;
    p.prefix_slot = prefix_id;
    p.prefix_len = lp;
    p.prefix_items = z.prefix_items;
    p.prefix_ns = z.prefix_ns;
    p.prefix_tpi = z.prefix_tpi;
    p.prefix_rows = z.prefix_rows;
    p.own_items = z.own_items;
    p.precise = p.out_f32 || weights_out || !p.rule.rough;
    p.w_chunks = (z.longest + 1023) / 1024;
    if ((long long)n * (p.Hq + (weights_out ? (long long)p.Hkv * p.w_chunks : 0)) > 0x7fffffffLL)
      return fail_message(c, SPD_ERR_CAPACITY, "too many weights for one launch");
    int launches = 0;
    cudaError_t e = cudaSuccess;
    const CUtensorMapDataType mt = map_type(cfg.dtype);
    const int br = cfg.physical_page % 64 == 0 ? 64 : cfg.physical_page % 32 == 0 ? 32 : 16;
    if (z.tc || z.few) {
      const cuuint64_t dims[4] = {64, (cuuint64_t)cfg.physical_page, (cuuint64_t)d / 64,
                                  (cuuint64_t)cfg.num_physical_pages * cfg.num_kv_heads};
      const cuuint64_t strides[3] = {(cuuint64_t)d * 2, 128, (cuuint64_t)cfg.physical_page * d * 2};
      const cuuint32_t box[4] = {64, (cuuint32_t)br, 1, 1};
      if (!encode4(&t.tm_k, mt, v.buf->k_pool, dims, strides, box) ||
          !encode4(&t.tm_v, mt, v.buf->v_pool, dims, strides, box))
        return fail_message(c, SPD_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    }
    p.box_rows = br;
    if (z.tc) {
      t.rule = p.rule;
      if (!encode_rows(&t.tm_q, mt, qb, d, cfg.num_q_heads, n, (long long)cfg.num_q_heads * d, v.G,
                       128 / v.G) ||
          !encode_partials(&t.tm_out, p.pre_o, d,
                           (size_t)z.tiles * cfg.num_kv_heads * z.nsplit * kDenseRows))
        return fail_message(c, SPD_ERR_CUDA, "cuTensorMapEncodeTiled failed");
      t.partial = 1;
      t.part_o = p.pre_o;
      t.part_ml = p.pre_ml;
      t.v = nullptr;
      t.v_stride = 0;
      t.key_begin = t.key_end = nullptr;
      t.page_row = p.page_table + (size_t)prefix_id * v.max_pp;
      t.err = v.err;
      t.paged = 1;
      t.out_f32 = p.out_f32;
      t.Lq = n;
      t.Lk = lp;
      t.Hq = p.Hq;
      t.Hkv = p.Hkv;
      t.G = v.G;
      t.lhp = v.G == 8 ? 3 : v.G == 4 ? 2 : v.G == 2 ? 1 : 0;
      t.HG = 1;
      t.tiles = z.tiles;
      t.nsplit = z.nsplit;
      t.dup = z.dup;
      t.P = p.P;
      t.max_pp = p.max_pp;
      t.num_phys = p.num_phys;
      t.box_rows = br;
      t.pos0 = 0;
      for (int i = 0; i < n; ++i) t.lens[i] = p.seqs[i].L;
      // weights that are kept show the cap in their denominator: the precise form, which
      // is the split one's (64 sequences over 32,768 tokens with a cap 86 -> 113 us)
      const bool fine = p.out_f32 || (weights_out && p.rule.cap_out > 0.f);
      e = launch_dense_tc(t, cfg.dtype, d, fine, st);
      ++launches;
    }
    p.follow = z.tc;
    // one kernel where it takes all items (the weights need every split first)
    const bool joins = !z.tc && !z.few && !weights_out && n <= v.ticket_seqs;
    p.tickets = joins ? v.tickets : nullptr;
    if (z.few) {
      // the shorter one first: the other, which does not wait for it, hides it
      for (int k = 0; k < 2 && e == cudaSuccess; ++k) {
        const bool own = (k == 0) == z.own_first;
        if (own && z.own_items == 0) continue;
        if (own) {
          p.tm_k = *v.tm_k;
          p.tm_v = *v.tm_v;
          p.prefix_items = 0;  // (the decode kernel takes the own items alone)
          e = launch_dense_decode(p, cfg.dtype, d, st);
        } else {
          p.tm_k = t.tm_k;
          p.tm_v = t.tm_v;
          p.prefix_items = z.prefix_items;
          e = launch_dense_few(p, cfg.dtype, st);
        }
        p.follow = 1;
        ++launches;
      }
    } else if (e == cudaSuccess && z.prefix_items + z.own_items > 0) {
      e = launch_dense_decode(p, cfg.dtype, d, st);
      ++launches;
    }
    if (e == cudaSuccess && !joins) {
      e = launch_dense_decode_combine(p, cfg.dtype, d, st);
      ++launches;
    }
    note_launches(c, st, launches);
    if (e != cudaSuccess) return fail_message(c, SPD_ERR_CUDA, cudaGetErrorString(e));
  }
  return SPD_OK;
}

spd_status spd_kv_evict(spd_ctx *c, const int *src_ids, const int *dst_ids, int n_seqs, int keep,
                        int recent, const float *weights, long long weights_stride, int *kept,
                        float *kept_weights, spd_stream stream) {
  if (!c) return SPD_ERR_INVALID_ARG;
  if (keep < 1 || recent < 0 || recent > keep)
    return fail_message(c, SPD_ERR_INVALID_ARG, "keep >= 1 and 0 <= recent <= keep required");
  if (keep > kMaxKeep) return fail_message(c, SPD_ERR_CAPACITY, "keep exceeds 2^28");
  if (!aligned(weights, 4) || !aligned(kept, 4) || (kept_weights && !aligned(kept_weights, 4)))
    return fail_message(c, SPD_ERR_INVALID_ARG, "weights and kept must be 4-byte aligned pointers");
  CtxView v;
  ctx_view(c, &v);
  if (v.Hs > 0)
    return fail_message(c, SPD_ERR_INVALID_ARG, "a context with streaming heads keeps no whole cache");
  if (v.quant) return fail_message(c, SPD_ERR_INVALID_ARG, "a cache with kv_quant is not evicted from");
  spd_status r = check_live(c, src_ids, n_seqs);
  if (r != SPD_OK) return r;
  if ((r = check_live(c, dst_ids, n_seqs)) != SPD_OK) return r;
  const std::unique_ptr<int[]> m(new (std::nothrow) int[n_seqs]);
  if (!m) return fail_message(c, SPD_ERR_CAPACITY, "out of host memory");
  for (int i = 0; i < n_seqs; ++i) {
    for (int j = 0; j < n_seqs; ++j)
      if (src_ids[i] == dst_ids[j])
        return fail_message(c, SPD_ERR_BAD_SEQ, "a sequence is listed as source and destination");
    const long long L = seq_length(c, src_ids[i]);
    if (L < 1) return fail_message(c, SPD_ERR_STATE, "a source sequence has no tokens");
    if (seq_length(c, dst_ids[i]) != 0)
      return fail_message(c, SPD_ERR_STATE, "a destination sequence is not empty");
    if (L > weights_stride)
      return fail_message(c, SPD_ERR_CAPACITY, "weights_stride is below a sequence's length");
    m[i] = (int)std::min<long long>(keep, L);
  }
  // (below 2^30: the copying CTAs count on by the grid behind the last group)
  const long long groups = ((long long)keep + 63) / 64;
  if (groups * std::min(n_seqs, kDenseSeqs) * v.Hd > (1LL << 30))
    return fail_message(c, SPD_ERR_CAPACITY, "keep is too large for one launch");
  if ((r = check_fill(c, dst_ids, m.get(), n_seqs)) != SPD_OK) return r;
  cudaStream_t st = (cudaStream_t)stream;
  if ((r = ctx_device(c, st, &v)) != SPD_OK) return r;
  DeviceGuard guard;
  if ((r = guard.bind(v.device)) != SPD_OK) return fail_message(c, r, "cudaSetDevice failed");
  if ((r = fill_pages(c, dst_ids, m.get(), n_seqs, st)) != SPD_OK) return r;
  const spd_config &cfg = *v.cfg;
  static thread_local EvictParams p;
  for (int b = 0; b < n_seqs; b += kDenseSeqs) {
    p.n = std::min(kDenseSeqs, n_seqs - b);
    p.k_pool = v.buf->k_pool;
    p.v_pool = v.buf->v_pool;
    p.meta = v.buf->meta;
    p.page_table = static_cast<const int *>(v.buf->page_table);
    p.weights = weights + (size_t)b * v.Hd * weights_stride;
    p.kept = kept + (size_t)b * v.Hd * keep;
    p.kept_weights = kept_weights ? kept_weights + (size_t)b * v.Hd * keep : nullptr;
    p.err = v.err;
    p.w_stride = weights_stride;
    p.Hkv = v.Hd;
    p.keep = keep;
    p.recent = recent;
    p.ell = cfg.logical_page;
    p.P = cfg.physical_page;
    p.R = v.R;
    p.max_pp = v.max_pp;
    p.num_phys = cfg.num_physical_pages;
    p.kv_fp8 = v.kv_fp8;
    p.P_log2 = -1;
    for (int x = 0; x < 31; ++x)
      if (p.P == 1 << x) p.P_log2 = x;
    for (int i = 0; i < p.n; ++i)
      p.seqs[i] = EvictSeq{src_ids[b + i], dst_ids[b + i], (int)seq_length(c, src_ids[b + i]),
                           m[b + i]};
    const cudaError_t e = launch_evict(p, cfg.dtype, cfg.head_dim, v.num_sms, st);
    note_launches(c, st, 2);
    if (e != cudaSuccess) return fail_message(c, SPD_ERR_CUDA, cudaGetErrorString(e));
  }
  set_filled(c, dst_ids, m.get(), n_seqs);
  return SPD_OK;
}

}  // extern "C"
