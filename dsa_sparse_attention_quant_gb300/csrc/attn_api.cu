// attn_api.cu — the C entry points of the attention, the KV cache's writer and
// the page calls: argument checks, workspace carving, tensor maps, launches.
// Host code only.
#include <climits>
#include <cmath>
#include <cstring>

#include "attn.h"
#include "host.h"
#include "kernels.h"

using namespace dsa;

namespace {

constexpr int64_t kMaxStride = int64_t{1} << 39;  // elements of 2 bytes: tensor-map strides end at 2^40 bytes

bool stride_ok(int64_t s, int head_dim) { return s >= head_dim && s % 8 == 0 && s < kMaxStride; }

// The cache's description with the strides of one-element axes made valid.
int check_kv(const DsaKv* kv, bool packed, DsaKv* out) {
  if (kv == nullptr) return DSA_EINVAL;
  *out = *kv;
  if (kv->dtype != DSA_BF16 && kv->dtype != DSA_FP16) return DSA_EINVAL;
  if (kv->num_kv_heads < 1 || kv->num_kv_heads > 65535 || (kv->head_dim != 64 && kv->head_dim != 128))
    return DSA_EINVAL;
  if (kv->num_blocks < 1 || kv->num_blocks > (packed ? INT_MAX : INT_MAX / kBlock)) return DSA_EINVAL;
  if (!kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return DSA_EINVAL;
  const int d = kv->head_dim;
  if (kv->num_kv_heads == 1) out->k_head_stride = out->v_head_stride = d;
  if (packed || kv->num_blocks == 1) out->k_page_stride = out->v_page_stride = d;
  if (packed && kv->num_blocks == 1) out->k_slot_stride = out->v_slot_stride = d;
  for (int64_t s : {out->k_page_stride, out->k_slot_stride, out->k_head_stride, out->v_page_stride,
                    out->v_slot_stride, out->v_head_stride})
    if (!stride_ok(s, d)) return DSA_EINVAL;
  return DSA_OK;
}

// rows: the rows of q and out that the call may reach, from the first.
int check_attn(const DsaAttn* at, const DsaKv& kv, int64_t rows, DsaAttn* out) {
  if (at == nullptr) return DSA_EINVAL;
  *out = *at;
  if (!at->q || !at->out || !aligned16(at->q) || !aligned16(at->out)) return DSA_EINVAL;
  if (at->lse != nullptr && reinterpret_cast<uintptr_t>(at->lse) % 4 != 0) return DSA_EINVAL;
  if (at->num_heads < 1 || at->num_heads > 65535 || at->num_heads % kv.num_kv_heads != 0) return DSA_EINVAL;
  if (at->num_heads == 1) out->q_head_stride = out->out_head_stride = kv.head_dim;
  if (rows == 1) out->q_row_stride = out->out_row_stride = kv.head_dim;
  for (int64_t s : {out->q_row_stride, out->q_head_stride, out->out_row_stride, out->out_head_stride})
    if (!stride_ok(s, kv.head_dim)) return DSA_EINVAL;
  if (!std::isfinite(at->scale * 1.4426950408889634f) && !(at->scale < 0)) return DSA_EINVAL;
  if (!(at->scale > 0.0f)) out->scale = kv.head_dim == 128 ? 0.08838834764831845f : 0.125f;
  return DSA_OK;
}

// pages: the call reads the block table.
int check_step(const DsaBatch* b, bool pages) {
  if (b == nullptr) return DSA_EINVAL;
  if (b->num_reqs < 0 || b->num_decodes < 0 || b->num_decodes > b->num_reqs || b->num_tokens < 0) return DSA_EINVAL;
  if (b->num_decode_tokens < 0 || b->num_decode_tokens > b->num_tokens) return DSA_EINVAL;
  if (b->num_tokens > 0 && b->num_reqs == 0) return DSA_EINVAL;
  if (b->max_seq_len < 0) return DSA_EINVAL;
  if (b->num_reqs > 0 && (!b->query_start_loc || !b->seq_lens)) return DSA_EINVAL;
  if (b->num_reqs > 0 && pages && (!b->block_table || b->bt_stride < 1)) return DSA_EINVAL;
  if (b->num_tokens > 0 && b->req_id_per_token == nullptr) return DSA_EINVAL;
  return DSA_OK;
}

// Keys that both the block-table row and max_seq_len allow.
int max_keys(const DsaBatch* b) {
  const int64_t row = b->bt_stride > INT_MAX / kBlock ? INT_MAX : b->bt_stride * kBlock;
  return static_cast<int>(row < b->max_seq_len ? row : b->max_seq_len);
}

// ---- single rows: how the work is cut, from the host's bounds alone.
struct RowsPlan {
  int passes, rows;  // passes over the keys, rows of the workspace per pass
  int64_t slices;    // split: slices of the tile list, else the tokens
  int64_t ctas;      // per slice, KV head and pass
  bool split;
  size_t off_ml, off_o, bytes;
};

// Two CTAs per SM on a part of up to 160 SMs.
constexpr int kRowsCtas = 320;
// Tokens of up to this many tiles are not cut while the CTAs are few: one streams
// such a row in about the time that the join's launch takes. GPU time, 32/8 heads
// of 128: one request of 256 keys 5.7 us (cut from 2 tiles on: 7.1), of 768 7.9 (cut
// from 16 on: 11.5); one of 512 takes 8.5, cut 7.5.
constexpr int kDirectTiles = 8;
// More CTAs than this run as slices, whose loads go on across tokens: two on each of
// a GB300's 152 SMs. It is a number, not the device's, so that the scratch's size
// and the run decide alike. 32 requests of 512 keys, 32/8 heads: 10.6 us (with 152:
// 15.2); 64 of them 29.3 (with 608: 26.5).
constexpr int kDirectCtas = 304;
// The least slice, in tiles: shorter ones pay more for their partials than they save
// (2 requests of 4096 keys, 40/1 heads: 14.3 us, with 1 tile 18.5; one of 768,
// 32/8: 7.9, with 4 tiles 9.1).
constexpr int kMinTiles = 2;

// One slice per CTA place: cut two or four times finer, so that CTAs that stream
// slower take less, the partials and the CTAs' starts cost more than that gains
// (32 requests of 4K to 8K keys: 130.8, 134.4, 145.0 us).
RowsPlan rows_plan(int64_t tokens, int64_t keys, int heads, int hkv, int head_dim, int ctas) {
  RowsPlan p{};
  const int group = heads / hkv;
  p.rows = group <= 16 ? 16 : 32;
  p.passes = (group + p.rows - 1) / p.rows;
  const int64_t tiles = keys > 0 ? (keys + kBlock - 1) / kBlock : 1;
  p.split = tiles > kDirectTiles || tokens * hkv * p.passes > kDirectCtas;
  p.slices = tokens;
  if (p.split) {
    const int64_t most = (tokens * tiles + kMinTiles - 1) / kMinTiles;
    int64_t s = ctas / (static_cast<int64_t>(hkv) * p.passes);
    if (s < 1) s = 1;
    p.slices = s < most ? s : most;
  }
  p.ctas = p.slices * hkv * p.passes;
  if (p.split) {
    const size_t n = static_cast<size_t>(p.ctas);
    p.off_ml = align_up(n * sizeof(int2), 256);
    p.off_o = p.off_ml + align_up(2 * n * p.rows * sizeof(float2), 256);
    p.bytes = p.off_o + 2 * n * p.rows * head_dim * sizeof(float);
  }
  return p;
}

bool heads_ok(int32_t heads, int32_t hkv, int32_t head_dim) {
  return hkv >= 1 && heads >= 1 && heads <= 65535 && heads % hkv == 0 && (head_dim == 64 || head_dim == 128);
}

RowsArgs rows_args(const DsaKv& kv, const DsaAttn& at) {
  RowsArgs a{};
  a.q = at.q;
  a.k = kv.k;
  a.v = kv.v;
  a.out = at.out;
  a.lse = at.lse;
  a.q_row = at.q_row_stride;
  a.q_head = at.q_head_stride;
  a.out_row = at.out_row_stride;
  a.out_head = at.out_head_stride;
  a.k_page = kv.k_page_stride;
  a.k_slot = kv.k_slot_stride;
  a.k_head = kv.k_head_stride;
  a.v_page = kv.v_page_stride;
  a.v_slot = kv.v_slot_stride;
  a.v_head = kv.v_head_stride;
  a.heads = at.num_heads;
  a.hkv = kv.num_kv_heads;
  a.group = at.num_heads / kv.num_kv_heads;
  a.scale_log2 = at.scale * 1.4426950408889634f;
  a.num_blocks = kv.num_blocks;
  a.num_slots = kv.num_blocks * kBlock;
  a.min_tiles = kMinTiles;
  return a;
}

int run_rows(RowsArgs& a, int64_t tokens, int64_t keys, const DsaKv& kv, bool selected, void* ws, size_t ws_bytes,
             cudaStream_t stream) {
  RowsPlan need = rows_plan(tokens, keys, a.heads, a.hkv, kv.head_dim, kRowsCtas);
  if (need.ctas > INT_MAX) return DSA_EINVAL;
  if (need.bytes > 0 && (ws == nullptr || !aligned16(ws))) return DSA_EINVAL;
  if (ws_bytes < need.bytes) return DSA_ENOSPACE;
  int sms;
  int st = device_sms(&sms);
  if (st != DSA_OK) return st;
  const RowsPlan p = rows_plan(tokens, keys, a.heads, a.hkv, kv.head_dim, 2 * sms < kRowsCtas ? 2 * sms : kRowsCtas);
  a.n_tokens = static_cast<int>(tokens);
  a.passes = p.passes;
  a.slices = static_cast<int>(p.slices);
  a.split = p.split;
  if (p.split) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.desc = reinterpret_cast<int2*>(base);
    a.part_ml = reinterpret_cast<float2*>(base + p.off_ml);
    a.part_o = reinterpret_cast<float*>(base + p.off_o);
  }
  return from_cuda(launch_attn_rows(a, kv.head_dim, kv.dtype, selected, stream));
}

// K or V as a 4-D tensor {head_dim, heads, slots, pages} (packed: {head_dim,
// heads, rows, 1}): one box is 64 columns (128 bytes) of 64 slots of a head,
// landed with the 128-byte swizzle.
int make_kv_map(CUtensorMap* m, const DsaKv& kv, const void* base, int64_t page, int64_t slot, int64_t head,
                bool packed) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  int st = tensor_map_encoder(&enc);
  if (st != DSA_OK) return st;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(kv.num_kv_heads),
                        static_cast<cuuint64_t>(packed ? kv.num_blocks : kBlock),
                        static_cast<cuuint64_t>(packed ? 1 : kv.num_blocks)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(head * 2), static_cast<cuuint64_t>(slot * 2),
                           static_cast<cuuint64_t>(page * 2)};
  cuuint32_t box[4] = {64, 1, kBlock, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, kv.dtype == DSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DSA_OK : DSA_ECUDA;
}

// q as a 3-D tensor {head_dim, heads, tokens}: one box is 64 columns of 128 tokens of a head.
int make_prompt_q_map(CUtensorMap* m, const DsaAttn& at, const DsaKv& kv, int64_t tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  int st = tensor_map_encoder(&enc);
  if (st != DSA_OK) return st;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(at.num_heads),
                        static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(at.q_head_stride * 2), static_cast<cuuint64_t>(at.q_row_stride * 2)};
  cuuint32_t box[3] = {64, 1, 128};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, kv.dtype == DSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(at.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DSA_OK : DSA_ECUDA;
}

// ---- pages
struct PagesWs {
  int32_t *w0, *w1, *w2, *counts, *fresh;
  int4* entry;
  size_t bytes;
};

PagesWs pages_carve(int64_t num_blocks, int32_t n, void* base) {
  PagesWs w{};
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void* r = p ? p + off : nullptr;
    off = align_up(off + bytes, 256);
    return r;
  };
  const size_t nb = static_cast<size_t>(num_blocks), m = static_cast<size_t>(n);
  w.w0 = static_cast<int32_t*>(take(nb * 4));
  w.w1 = static_cast<int32_t*>(take(nb * 4));
  w.w2 = static_cast<int32_t*>(take(nb * 4));
  w.counts = static_cast<int32_t*>(take(((nb + kPageChunk - 1) / kPageChunk + 1) * 4));
  w.entry = static_cast<int4*>(take(m * sizeof(int4)));
  w.fresh = static_cast<int32_t*>(take(m * 4));
  w.bytes = off;
  return w;
}

constexpr int64_t kMaxBlocks = INT_MAX / kBlock;

constexpr int kMaxLists = 16;

int check_caches(const DsaCacheDesc* caches, int32_t n) {
  if (n < 0 || n > kMaxLists * kMaxCaches || (n > 0 && caches == nullptr)) return DSA_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    const DsaCacheDesc& c = caches[i];
    if (!c.base || !aligned16(c.base) || c.page_bytes < 16 || c.page_bytes % 16 != 0 || c.page_stride % 16 != 0 ||
        c.page_stride < c.page_bytes || c.page_bytes > (int64_t{1} << 30))
      return DSA_EINVAL;
  }
  return DSA_OK;
}

int check_pages(const DsaPages* g, bool lens) {
  if (g == nullptr || g->num_blocks < 1 || g->num_blocks > kMaxBlocks || g->n_rows < 0 || g->bt_stride < 1 ||
      g->bt_stride > INT_MAX / kBlock)
    return DSA_EINVAL;
  if (!g->refs || !aligned16(g->refs)) return DSA_EINVAL;
  if (g->n_rows > 0 && (!g->block_table || (lens && !g->seq_lens))) return DSA_EINVAL;
  return DSA_OK;
}

// Calls f(lists, n) with the caches in lists of kMaxCaches; one empty list without caches.
template <typename F>
int with_lists(const DsaCacheDesc* caches, int32_t n, F f) {
  CacheList lists[kMaxLists];
  int m = 0;
  for (int32_t i = 0; i < n || m == 0; ++m) {
    CacheList& l = lists[m];
    std::memset(&l, 0, sizeof(l));
    for (; i < n && l.n < kMaxCaches; ++i, ++l.n) {
      l.base[l.n] = static_cast<uint8_t*>(caches[i].base);
      l.page_bytes[l.n] = caches[i].page_bytes;
      l.page_stride[l.n] = caches[i].page_stride;
      l.parts += static_cast<int>((caches[i].page_bytes + kPartBytes - 1) / kPartBytes);
      l.parts_end[l.n] = l.parts;
    }
  }
  return f(lists, m);
}

PagesArgs pages_args(const DsaPages& g, const PagesWs& w, const int32_t* a, const int32_t* b, int32_t n,
                     int32_t* err) {
  PagesArgs p{};
  p.refs = g.refs;
  p.num_blocks = g.num_blocks;
  p.block_table = g.block_table;
  p.bt_stride = g.bt_stride;
  p.n_rows = g.n_rows;
  p.seq_lens = g.seq_lens;
  p.a = a;
  p.b = b;
  p.n = n;
  p.w0 = w.w0;
  p.w1 = w.w1;
  p.w2 = w.w2;
  p.counts = w.counts;
  p.entry = w.entry;
  p.fresh = w.fresh;
  p.err = err;
  return p;
}

}  // namespace

extern "C" {

int dsa_kv_write(const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                 int64_t v_head_stride, int64_t n_tokens, const int64_t* slot_mapping, const DsaKv* kv,
                 int32_t* dev_err, dsa_stream_t stream) {
  DsaKv c;
  int st = check_kv(kv, false, &c);
  if (st != DSA_OK) return st;
  if (n_tokens < 0) return DSA_EINVAL;
  if (c.num_kv_heads == 1) k_head_stride = v_head_stride = c.head_dim;
  if (n_tokens <= 1) k_row_stride = v_row_stride = c.head_dim;
  // rows may overlap as views do, but not share a head's elements
  for (int64_t s : {k_row_stride, k_head_stride, v_row_stride, v_head_stride})
    if (!stride_ok(s, c.head_dim)) return DSA_EINVAL;
  if (n_tokens == 0) return DSA_OK;
  if (!k || !v || !slot_mapping || !aligned16(k) || !aligned16(v)) return DSA_EINVAL;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  const KvWriteArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                      k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                      static_cast<uint16_t*>(c.k), static_cast<uint16_t*>(c.v),
                      c.k_page_stride, c.k_slot_stride, c.k_head_stride,
                      c.v_page_stride, c.v_slot_stride, c.v_head_stride,
                      c.num_kv_heads, n_tokens, c.num_blocks * kBlock, slot_mapping, dev_err};
  return from_cuda(launch_kv_write(a, c.head_dim, sms, stream));
}

size_t dsa_attn_decode_workspace_size(const DsaBatch* batch, int32_t num_heads, int32_t num_kv_heads,
                                      int32_t head_dim) {
  if (check_step(batch, true) != DSA_OK || !heads_ok(num_heads, num_kv_heads, head_dim)) return 0;
  return rows_plan(batch->num_decode_tokens, batch->num_reqs > 0 ? max_keys(batch) : 0, num_heads, num_kv_heads,
                   head_dim, kRowsCtas)
      .bytes;
}

int dsa_attn_decode(const DsaBatch* batch, const DsaKv* kv, const DsaAttn* attn, void* ws, size_t ws_bytes,
                    int32_t* dev_err, dsa_stream_t stream) {
  DsaKv c;
  DsaAttn at;
  int st = check_step(batch, true);
  if (st != DSA_OK) return st;
  if (batch->num_decode_tokens == 0) return DSA_OK;
  if ((st = check_kv(kv, false, &c)) != DSA_OK ||
      (st = check_attn(attn, c, batch->num_decode_tokens, &at)) != DSA_OK)
    return st;
  if (batch->num_blocks != c.num_blocks || batch->num_decodes < 1) return DSA_EINVAL;
  RowsArgs a = rows_args(c, at);
  a.qsl = batch->query_start_loc;
  a.seq_lens = batch->seq_lens;
  a.req_id = batch->req_id_per_token;
  a.block_table = batch->block_table;
  a.bt_stride = batch->bt_stride;
  a.num_reqs = batch->num_decodes;
  a.max_keys = max_keys(batch);
  a.err = dev_err;
  return run_rows(a, batch->num_decode_tokens, a.max_keys, c, false, ws, ws_bytes, stream);
}

size_t dsa_attn_selected_workspace_size(int64_t n_tokens, int32_t topk, int32_t num_heads, int32_t num_kv_heads,
                                        int32_t head_dim) {
  if (n_tokens < 0 || n_tokens > INT_MAX || topk < 1 || !heads_ok(num_heads, num_kv_heads, head_dim)) return 0;
  return rows_plan(n_tokens, topk, num_heads, num_kv_heads, head_dim, kRowsCtas).bytes;
}

int dsa_attn_selected(const DsaKv* kv, const DsaAttn* attn, const int32_t* physical, int64_t n_tokens, int32_t topk,
                      void* ws, size_t ws_bytes, int32_t* dev_err, dsa_stream_t stream) {
  DsaKv c;
  DsaAttn at;
  if (n_tokens < 0 || n_tokens > INT_MAX || topk < 1) return DSA_EINVAL;
  if (n_tokens == 0) return DSA_OK;
  int st = check_kv(kv, false, &c);
  if (st != DSA_OK || (st = check_attn(attn, c, n_tokens, &at)) != DSA_OK) return st;
  if (physical == nullptr) return DSA_EINVAL;
  RowsArgs a = rows_args(c, at);
  a.physical = physical;
  a.topk = topk;
  a.err = dev_err;
  return run_rows(a, n_tokens, topk, c, true, ws, ws_bytes, stream);
}

int dsa_attn_prompt(const DsaBatch* batch, const DsaKv* kv, const int32_t* kv_start, const DsaAttn* attn,
                    int32_t* dev_err, dsa_stream_t stream) {
  DsaKv c;
  DsaAttn at;
  const bool packed = kv_start != nullptr;
  int st = check_step(batch, !packed);
  if (st != DSA_OK) return st;
  const int reqs = batch->num_reqs - batch->num_decodes;
  const int64_t rows = batch->num_tokens - batch->num_decode_tokens;
  if (rows == 0) return DSA_OK;
  if ((st = check_kv(kv, packed, &c)) != DSA_OK ||
      (st = check_attn(attn, c, batch->num_tokens, &at)) != DSA_OK)
    return st;
  if (reqs < 1 || (!packed && batch->num_blocks != c.num_blocks)) return DSA_EINVAL;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  CUtensorMap mq, mk, mv;
  if ((st = make_prompt_q_map(&mq, at, c, batch->num_tokens)) != DSA_OK) return st;
  if ((st = make_kv_map(&mk, c, c.k, c.k_page_stride, c.k_slot_stride, c.k_head_stride, packed)) != DSA_OK) return st;
  if ((st = make_kv_map(&mv, c, c.v, c.v_page_stride, c.v_slot_stride, c.v_head_stride, packed)) != DSA_OK) return st;
  PromptArgs a{};
  a.out = at.out;
  a.lse = at.lse;
  a.out_row = at.out_row_stride;
  a.out_head = at.out_head_stride;
  a.v = c.v;
  a.v_page = c.v_page_stride;
  a.v_slot = c.v_slot_stride;
  a.v_head = c.v_head_stride;
  a.heads = at.num_heads;
  a.hkv = c.num_kv_heads;
  a.group = at.num_heads / c.num_kv_heads;
  a.scale_log2 = at.scale * 1.4426950408889634f;
  a.qsl = batch->query_start_loc;
  a.seq_lens = batch->seq_lens;
  a.block_table = batch->block_table;
  a.kv_start = kv_start;
  a.bt_stride = batch->bt_stride;
  a.num_blocks = c.num_blocks;
  a.num_reqs = batch->num_reqs;
  a.num_decodes = batch->num_decodes;
  a.num_tokens = batch->num_tokens;
  a.first_token = batch->num_decode_tokens;
  a.max_keys = packed ? batch->max_seq_len : max_keys(batch);
  a.pair_heads = a.group % 2 == 0;
  a.head_units = a.pair_heads ? a.heads / 2 : a.heads;
  const int64_t unit = a.pair_heads ? 128 : 256;
  const int64_t units = rows / unit + reqs;  // at least the sum of ceil(q_len / unit)
  if (units * a.head_units > INT_MAX) return DSA_EINVAL;
  a.tile_units = static_cast<int>(units);
  a.err = dev_err;
  return from_cuda(launch_attn_prompt(a, &mq, &mk, &mv, c.head_dim, c.dtype, stream));
}

size_t dsa_pages_workspace_size(int64_t num_blocks, int32_t n) {
  if (num_blocks < 1 || num_blocks > kMaxBlocks || n < 0) return 0;
  return pages_carve(num_blocks, n, nullptr).bytes;
}

int dsa_pages_copy(const DsaCacheDesc* caches, int32_t n_caches, int64_t num_blocks, const int32_t* src,
                   const int32_t* dst, int32_t n, void* ws, size_t ws_bytes, int32_t* dev_err, dsa_stream_t stream) {
  int st = check_caches(caches, n_caches);
  if (st != DSA_OK) return st;
  if (num_blocks < 1 || num_blocks > kMaxBlocks || n < 0 || n > (1 << 30)) return DSA_EINVAL;
  if (n == 0) return DSA_OK;
  if (!src || !dst || !ws || !aligned16(ws)) return DSA_EINVAL;
  const PagesWs w = pages_carve(num_blocks, n, ws);
  if (ws_bytes < w.bytes) return DSA_ENOSPACE;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  DsaPages g{};
  g.num_blocks = num_blocks;
  const PagesArgs p = pages_args(g, w, src, dst, n, dev_err);
  return with_lists(caches, n_caches, [&](const CacheList* l, int m) {
    return from_cuda(launch_pages_copy(p, l, m, sms, stream));
  });
}

int dsa_pages_fork(const DsaPages* pages, const int32_t* parents, const int32_t* children, int32_t n,
                   const DsaCacheDesc* caches, int32_t n_caches, void* ws, size_t ws_bytes, int32_t* dev_err,
                   dsa_stream_t stream) {
  int st = check_pages(pages, true);
  if (st != DSA_OK || (st = check_caches(caches, n_caches)) != DSA_OK) return st;
  if (n < 0) return DSA_EINVAL;
  if (n == 0) return DSA_OK;
  if (!parents || !children || !ws || !aligned16(ws)) return DSA_EINVAL;
  const PagesWs w = pages_carve(pages->num_blocks, n, ws);
  if (ws_bytes < w.bytes) return DSA_ENOSPACE;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  const PagesArgs p = pages_args(*pages, w, parents, children, n, dev_err);
  return with_lists(caches, n_caches, [&](const CacheList* l, int m) {
    return from_cuda(launch_pages_fork(p, l, m, sms, stream));
  });
}

int dsa_pages_free(const DsaPages* pages, const int32_t* rows, int32_t n, int32_t* dev_err, dsa_stream_t stream) {
  int st = check_pages(pages, true);
  if (st != DSA_OK) return st;
  if (n < 0) return DSA_EINVAL;
  if (n == 0) return DSA_OK;
  if (!rows) return DSA_EINVAL;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  return from_cuda(launch_pages_free(pages_args(*pages, PagesWs{}, rows, nullptr, n, dev_err), stream));
}

int dsa_pages_compact(const DsaPages* pages, const DsaCacheDesc* caches, int32_t n_caches, void* ws, size_t ws_bytes,
                      int32_t* dev_err, dsa_stream_t stream) {
  int st = check_pages(pages, false);
  if (st != DSA_OK || (st = check_caches(caches, n_caches)) != DSA_OK) return st;
  if (!ws || !aligned16(ws)) return DSA_EINVAL;
  const PagesWs w = pages_carve(pages->num_blocks, 0, ws);
  if (ws_bytes < w.bytes) return DSA_ENOSPACE;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  const PagesArgs p = pages_args(*pages, w, nullptr, nullptr, 0, dev_err);
  return with_lists(caches, n_caches, [&](const CacheList* l, int m) {
    return from_cuda(launch_pages_compact(p, l, m, sms, stream));
  });
}

}  // extern "C"
