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

// The 8-bit cache's description with the strides of one-element axes made valid;
// sizes: heads, head_dim, pages and type as DsaKv has them.
int check_kv8(const DsaKv8* kv, DsaKv8* out, DsaKv* sizes) {
  if (kv == nullptr) return DSA_EINVAL;
  *out = *kv;
  if (kv->dtype != DSA_BF16 && kv->dtype != DSA_FP16) return DSA_EINVAL;
  if (kv->num_kv_heads < 1 || kv->num_kv_heads > 65535 || (kv->head_dim != 64 && kv->head_dim != 128))
    return DSA_EINVAL;
  if (kv->num_blocks < 1 || kv->num_blocks > INT_MAX / kBlock) return DSA_EINVAL;
  if (!kv->k || !kv->v || !kv->scale || !aligned16(kv->k) || !aligned16(kv->v) || !aligned16(kv->scale))
    return DSA_EINVAL;
  const int d = kv->head_dim;
  if (kv->num_kv_heads == 1) {
    out->k_head_stride = out->v_head_stride = d;
    out->s_head_stride = 2;
  }
  if (kv->num_blocks == 1) {
    out->k_page_stride = out->v_page_stride = d;
    out->s_page_stride = 2;
  }
  for (int64_t s : {out->k_page_stride, out->k_slot_stride, out->k_head_stride, out->v_page_stride,
                    out->v_slot_stride, out->v_head_stride})
    if (!stride_ok(s, d) || s % 16 != 0) return DSA_EINVAL;
  for (int64_t s : {out->s_page_stride, out->s_block_stride, out->s_head_stride})
    if (s < 2 || s % 2 != 0 || s >= kMaxStride) return DSA_EINVAL;
  *sizes = DsaKv{};
  sizes->dtype = kv->dtype;
  sizes->num_kv_heads = kv->num_kv_heads;
  sizes->head_dim = d;
  sizes->num_blocks = kv->num_blocks;
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
enum Cache { kIn16, kIn8 };
struct RowsPlan {
  int passes, rows;  // passes over the keys, rows of the workspace per pass
  int64_t slices;    // split: slices of the tile list, else the tokens
  int64_t ctas;      // per slice, KV head and pass
  bool split;
  int cluster;       // not split: CTAs that share a token (8 bits)
  size_t off_ml, off_o, bytes;
};

// The scratch is sized for parts of up to 160 SMs.
constexpr int kMostSms = 160;
// Tokens of up to this many tiles are not cut while the CTAs are few: one streams
// such a row in about the time that the join's launch takes. GPU time, 32/8 heads
// of 128: one request of 256 keys 5.7 us (cut from 2 tiles on: 7.1), of 768 7.9 (cut
// from 16 on: 11.5); one of 512 takes 8.5, cut 7.5.
constexpr int kDirectTiles = 8;
// More CTAs than there are places on a GB300's 152 SMs run as slices, whose loads go on
// across tokens. It is a number, not the device's, so that the scratch's size
// and the run decide alike. 16 bits, two places an SM: 32 requests of 512 keys, 32/8
// heads: 10.6 us (with 152: 15.2); 64 of them 29.3 (with 608: 26.5).
constexpr int kDirectSms = 152;
// The least slice, in tiles: shorter ones pay more for their partials than they save
// (2 requests of 4096 keys, 40/1 heads: 14.3 us, with 1 tile 18.5; one of 768,
// 32/8: 7.9, with 4 tiles 9.1).
constexpr int kMinTiles = 2;
// 8 bits: tokens of up to this many tiles are shared by clusters of up to 8 CTAs, two
// tiles each at least, while all of them have places: a cluster joins its token's rows
// through shared memory, without a second launch. 2 requests of 4096 keys, 40/8 heads of
// 128: 11.5 us, cut into slices 14.3; 16 tokens of 1024 slots, 32/8: 15.8, 18.1; but one
// request of 8192, 32/8: 15.9, 13.5; and with more than 8 query heads a KV head one
// token of 2048 slots, 40/2: 12.6, 11.7.
constexpr int kClusterTiles = 64;

int64_t row_tiles(int64_t keys) { return keys > 0 ? (keys + kBlock - 1) / kBlock : 1; }

// The kernels count a call's (token, tile) pairs in 32 bits.
bool rows_fit(int64_t tokens, int64_t keys) { return tokens <= INT_MAX / row_tiles(keys); }

// One slice per CTA place: cut two or four times finer, so that CTAs that stream
// slower take less, the partials and the CTAs' starts cost more than that gains
// (32 requests of 4K to 8K keys: 130.8, 134.4, 145.0 us).
// joint: KV heads a CTA takes.
RowsPlan rows_plan(int64_t tokens, int64_t keys, int heads, int hkv, int head_dim, Cache cache, int joint,
                   int sms) {
  RowsPlan p{};
  const int group = heads / hkv;
  p.rows = cache == kIn8 ? rows8_of(group) : rows_of(group);
  const int per_sm = cache == kIn8 ? rows8_ctas(p.rows, joint) : kRowsCtas;
  p.passes = (group + p.rows - 1) / p.rows;
  const int64_t across = static_cast<int64_t>(hkv / joint) * p.passes;  // CTAs a slice
  const int64_t tiles = row_tiles(keys);
  p.split = tiles > kDirectTiles || tokens * across > per_sm * kDirectSms;
  p.slices = tokens;
  p.cluster = 1;
  if (cache == kIn8 && p.rows == 8 && tiles <= kClusterTiles) {
    while (p.cluster < kMostCluster && tiles >= 4 * p.cluster &&
           2 * p.cluster * tokens * across <= per_sm * kDirectSms)
      p.cluster *= 2;
    // more than 8 tiles a CTA are cut into slices all the same
    if (tiles > kDirectTiles * p.cluster) p.cluster = 1;
    if (p.cluster > 1) p.split = false;
  }
  if (p.split) {
    const int64_t most = (tokens * tiles + kMinTiles - 1) / kMinTiles;
    int64_t s = per_sm * (sms < kMostSms ? sms : kMostSms) / across;
    if (s < 1) s = 1;
    p.slices = s < most ? s : most;
  }
  p.ctas = p.slices * across;
  if (p.split) {
    const size_t n = static_cast<size_t>(p.ctas) * joint;
    p.off_ml = align_up(static_cast<size_t>(p.ctas) * sizeof(int2), 256);
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
  a.joint = 1;
  return a;
}

// Heads of 64 that lie side by side, two to a row of 128 bytes.
bool pairs_of_64(const DsaKv8& kv) {
  return kv.head_dim == 64 && kv.num_kv_heads % 2 == 0 && kv.k_head_stride == 64 && kv.v_head_stride == 64;
}

// Codes of K or V as a 4-D tensor {row, rows of heads, slots, pages} with `pair` heads a
// row: one box is 16 slots of a row.
int make_kv8_map(CUtensorMap* m, const DsaKv8& kv, int pair, const void* base, int64_t page, int64_t slot,
                 int64_t head) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  int st = tensor_map_encoder(&enc);
  if (st != DSA_OK) return st;
  const int row = pair * kv.head_dim;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(kv.num_kv_heads / pair), kBlock,
                        static_cast<cuuint64_t>(kv.num_blocks)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(head * pair), static_cast<cuuint64_t>(slot),
                           static_cast<cuuint64_t>(page)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(row), 1, DSA_SCALE_BLOCK, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE,
                   row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DSA_OK : DSA_ECUDA;
}

Rows8Args rows8_args(const DsaKv8& kv, const DsaKv& sizes, const DsaAttn& at) {
  Rows8Args a{};
  static_cast<RowsArgs&>(a) = rows_args(sizes, at);
  a.k = kv.k;
  a.v = kv.v;
  a.k_page = kv.k_page_stride;
  a.k_slot = kv.k_slot_stride;
  a.k_head = kv.k_head_stride;
  a.v_page = kv.v_page_stride;
  a.v_slot = kv.v_slot_stride;
  a.v_head = kv.v_head_stride;
  a.scale = kv.scale;
  a.s_page = kv.s_page_stride;
  a.s_block = kv.s_block_stride;
  a.s_head = kv.s_head_stride;
  a.bf16 = kv.dtype == DSA_BF16;
  return a;
}

Cache8Args cache8_args(const DsaKv8& kv) {
  return Cache8Args{kv.k,
                    kv.v,
                    kv.scale,
                    kv.k_page_stride,
                    kv.k_slot_stride,
                    kv.k_head_stride,
                    kv.v_page_stride,
                    kv.v_slot_stride,
                    kv.v_head_stride,
                    kv.s_page_stride,
                    kv.s_block_stride,
                    kv.s_head_stride,
                    kv.num_kv_heads,
                    kv.num_blocks};
}

// launch(): the kernels with the finished arguments.
template <typename F>
int run_rows(RowsArgs& a, int* cluster, int64_t tokens, int64_t keys, int head_dim, Cache cache, size_t need, void* ws,
             size_t ws_bytes, F launch) {
  if (!rows_fit(tokens, keys)) return DSA_EINVAL;
  const RowsPlan most = rows_plan(tokens, keys, a.heads, a.hkv, head_dim, cache, a.joint, kMostSms);
  if (most.ctas > INT_MAX || most.slices * a.hkv * most.passes > INT_MAX) return DSA_EINVAL;
  if (need > 0 && (ws == nullptr || !aligned16(ws))) return DSA_EINVAL;
  if (ws_bytes < need) return DSA_ENOSPACE;
  int sms;
  int st = device_sms(&sms);
  if (st != DSA_OK) return st;
  const RowsPlan p = rows_plan(tokens, keys, a.heads, a.hkv, head_dim, cache, a.joint, sms);
  a.n_tokens = static_cast<int>(tokens);
  a.passes = p.passes;
  a.slices = static_cast<int>(p.slices);
  a.split = p.split;
  if (cluster != nullptr) *cluster = p.cluster;
  if (p.split) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.desc = reinterpret_cast<int2*>(base);
    a.part_ml = reinterpret_cast<float2*>(base + p.off_ml);
    a.part_o = reinterpret_cast<float*>(base + p.off_o);
  }
  return launch();
}

// Scratch of a call over a cache in 16 bits, and in 8: the latter whatever the cache's
// strides, which decide how many heads a CTA takes.
size_t rows_bytes(int64_t tokens, int64_t keys, int heads, int hkv, int head_dim) {
  if (!rows_fit(tokens, keys)) return 0;
  return rows_plan(tokens, keys, heads, hkv, head_dim, kIn16, 1, kMostSms).bytes;
}
size_t rows8_bytes(int64_t tokens, int64_t keys, int heads, int hkv, int head_dim) {
  if (!rows_fit(tokens, keys)) return 0;
  const size_t one = rows_plan(tokens, keys, heads, hkv, head_dim, kIn8, 1, kMostSms).bytes;
  if (head_dim == 128 || hkv % 2 != 0) return one;
  const size_t two = rows_plan(tokens, keys, heads, hkv, head_dim, kIn8, 2, kMostSms).bytes;
  return one > two ? one : two;
}

// What a batch's decode tokens read.
void set_decode(RowsArgs& a, const DsaBatch* batch, int32_t* dev_err) {
  a.qsl = batch->query_start_loc;
  a.seq_lens = batch->seq_lens;
  a.req_id = batch->req_id_per_token;
  a.block_table = batch->block_table;
  a.bt_stride = batch->bt_stride;
  a.num_reqs = batch->num_decodes;
  a.max_keys = max_keys(batch);
  a.err = dev_err;
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
  return rows_bytes(batch->num_decode_tokens, batch->num_reqs > 0 ? max_keys(batch) : 0, num_heads, num_kv_heads,
                    head_dim);
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
  set_decode(a, batch, dev_err);
  return run_rows(a, nullptr, batch->num_decode_tokens, a.max_keys, c.head_dim, kIn16,
                  rows_bytes(batch->num_decode_tokens, a.max_keys, a.heads, a.hkv, c.head_dim), ws, ws_bytes,
                  [&] { return from_cuda(launch_attn_rows(a, c.head_dim, c.dtype, false, stream)); });
}

size_t dsa_attn_selected_workspace_size(int64_t n_tokens, int32_t topk, int32_t num_heads, int32_t num_kv_heads,
                                        int32_t head_dim) {
  if (n_tokens < 0 || n_tokens > INT_MAX || topk < 1 || !heads_ok(num_heads, num_kv_heads, head_dim)) return 0;
  return rows_bytes(n_tokens, topk, num_heads, num_kv_heads, head_dim);
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
  return run_rows(a, nullptr, n_tokens, topk, c.head_dim, kIn16,
                  rows_bytes(n_tokens, topk, a.heads, a.hkv, c.head_dim), ws, ws_bytes,
                  [&] { return from_cuda(launch_attn_rows(a, c.head_dim, c.dtype, true, stream)); });
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
  if (a.max_keys > INT_MAX - 127) a.max_keys = INT_MAX - 127;  // whole tiles of 128 keys are counted in 32 bits
  a.pair_heads = a.group % 2 == 0;
  a.head_units = a.pair_heads ? a.heads / 2 : a.heads;
  const int64_t unit = a.pair_heads ? 128 : 256;
  const int64_t units = rows / unit + reqs;  // at least the sum of ceil(q_len / unit)
  if (units * a.head_units > INT_MAX) return DSA_EINVAL;
  a.tile_units = static_cast<int>(units);
  a.err = dev_err;
  return from_cuda(launch_attn_prompt(a, &mq, &mk, &mv, c.head_dim, c.dtype, stream));
}

size_t dsa_kv_write8_workspace_size(int64_t n_tokens, int64_t num_blocks) {
  if (n_tokens <= kWrite8Few || n_tokens > INT_MAX || num_blocks < 1 || num_blocks > INT_MAX / kBlock) return 0;
  return static_cast<size_t>(num_blocks) * kBlock * sizeof(int32_t);
}

int dsa_kv_write8(const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                  int64_t v_head_stride, int64_t n_tokens, const int64_t* slot_mapping, const DsaKv8* kv, void* ws,
                  size_t ws_bytes, int32_t* dev_err, dsa_stream_t stream) {
  DsaKv8 c;
  DsaKv sizes;
  int st = check_kv8(kv, &c, &sizes);
  if (st != DSA_OK) return st;
  if (n_tokens < 0 || n_tokens > INT_MAX) return DSA_EINVAL;
  if (c.num_kv_heads == 1) k_head_stride = v_head_stride = c.head_dim;
  if (n_tokens <= 1) k_row_stride = v_row_stride = c.head_dim;
  for (int64_t s : {k_row_stride, k_head_stride, v_row_stride, v_head_stride})
    if (!stride_ok(s, c.head_dim)) return DSA_EINVAL;
  if (n_tokens == 0) return DSA_OK;
  if (!k || !v || !slot_mapping || !aligned16(k) || !aligned16(v)) return DSA_EINVAL;
  const size_t need = dsa_kv_write8_workspace_size(n_tokens, c.num_blocks);
  if (need > 0 && (ws == nullptr || !aligned16(ws))) return DSA_EINVAL;
  if (ws_bytes < need) return DSA_ENOSPACE;
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  const Write8Args a{cache8_args(c), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                     k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                     n_tokens, slot_mapping, need > 0 ? static_cast<int32_t*>(ws) : nullptr, dev_err};
  return from_cuda(launch_kv_write8(a, c.head_dim, c.dtype, sms, stream));
}

int dsa_kv_read8(const DsaBatch* batch, const DsaKv8* kv, const int32_t* kv_start, const DsaKv* rows, int32_t past,
                 int32_t* dev_err, dsa_stream_t stream) {
  DsaKv8 c;
  DsaKv sizes, out;
  if (batch == nullptr || batch->num_reqs < 0 || batch->max_seq_len < 0) return DSA_EINVAL;
  if (batch->num_reqs == 0) return DSA_OK;
  int st = check_kv8(kv, &c, &sizes);
  if (st != DSA_OK || (st = check_kv(rows, true, &out)) != DSA_OK) return st;
  if (out.dtype != c.dtype || out.num_kv_heads != c.num_kv_heads || out.head_dim != c.head_dim) return DSA_EINVAL;
  if (!batch->seq_lens || !batch->block_table || batch->bt_stride < 1 || batch->num_blocks != c.num_blocks ||
      !kv_start || (past && !batch->query_start_loc))
    return DSA_EINVAL;
  const int keys = max_keys(batch);
  if (keys > (1 << 27) - kBlock) return DSA_EINVAL;  // the blocks of 256 requests are counted in 32 bits
  int sms;
  if ((st = device_sms(&sms)) != DSA_OK) return st;
  const Read8Args a{cache8_args(c), static_cast<uint16_t*>(out.k), static_cast<uint16_t*>(out.v),
                    out.k_slot_stride, out.k_head_stride, out.v_slot_stride, out.v_head_stride,
                    out.num_blocks, batch->query_start_loc, batch->seq_lens, batch->block_table, kv_start,
                    batch->bt_stride, batch->num_reqs, keys, past != 0, dev_err};
  return from_cuda(launch_kv_read8(a, c.head_dim, c.dtype, sms, stream));
}

size_t dsa_attn_decode8_workspace_size(const DsaBatch* batch, int32_t num_heads, int32_t num_kv_heads,
                                       int32_t head_dim) {
  if (check_step(batch, true) != DSA_OK || !heads_ok(num_heads, num_kv_heads, head_dim)) return 0;
  return rows8_bytes(batch->num_decode_tokens, batch->num_reqs > 0 ? max_keys(batch) : 0, num_heads, num_kv_heads,
                     head_dim);
}

int dsa_attn_decode8(const DsaBatch* batch, const DsaKv8* kv, const DsaAttn* attn, void* ws, size_t ws_bytes,
                     int32_t* dev_err, dsa_stream_t stream) {
  DsaKv8 c;
  DsaKv sizes;
  DsaAttn at;
  int st = check_step(batch, true);
  if (st != DSA_OK) return st;
  if (batch->num_decode_tokens == 0) return DSA_OK;
  if ((st = check_kv8(kv, &c, &sizes)) != DSA_OK ||
      (st = check_attn(attn, sizes, batch->num_decode_tokens, &at)) != DSA_OK)
    return st;
  if (batch->num_blocks != c.num_blocks || batch->num_decodes < 1) return DSA_EINVAL;
  Rows8Args a = rows8_args(c, sizes, at);
  set_decode(a, batch, dev_err);
  a.pairs = pairs_of_64(c);
  a.joint = a.pairs ? 2 : 1;
  return run_rows(a, &a.cluster, batch->num_decode_tokens, a.max_keys, c.head_dim, kIn8,
                  rows8_bytes(batch->num_decode_tokens, a.max_keys, a.heads, a.hkv, c.head_dim), ws, ws_bytes,
                  [&] {
                    CUtensorMap maps[2];
                    int e = make_kv8_map(&maps[0], c, a.joint, c.k, c.k_page_stride, c.k_slot_stride, c.k_head_stride);
                    if (e != DSA_OK) return e;
                    e = make_kv8_map(&maps[1], c, a.joint, c.v, c.v_page_stride, c.v_slot_stride, c.v_head_stride);
                    if (e != DSA_OK) return e;
                    return from_cuda(launch_attn_rows8(a, c.head_dim, false, maps, stream));
                  });
}

size_t dsa_attn_selected8_workspace_size(int64_t n_tokens, int32_t topk, int32_t num_heads, int32_t num_kv_heads,
                                         int32_t head_dim) {
  if (n_tokens < 0 || n_tokens > INT_MAX || topk < 1 || !heads_ok(num_heads, num_kv_heads, head_dim)) return 0;
  return rows8_bytes(n_tokens, topk, num_heads, num_kv_heads, head_dim);
}

int dsa_attn_selected8(const DsaKv8* kv, const DsaAttn* attn, const int32_t* physical, int64_t n_tokens, int32_t topk,
                       void* ws, size_t ws_bytes, int32_t* dev_err, dsa_stream_t stream) {
  DsaKv8 c;
  DsaKv sizes;
  DsaAttn at;
  if (n_tokens < 0 || n_tokens > INT_MAX || topk < 1) return DSA_EINVAL;
  if (n_tokens == 0) return DSA_OK;
  int st = check_kv8(kv, &c, &sizes);
  if (st != DSA_OK || (st = check_attn(attn, sizes, n_tokens, &at)) != DSA_OK) return st;
  if (physical == nullptr) return DSA_EINVAL;
  Rows8Args a = rows8_args(c, sizes, at);
  a.physical = physical;
  a.topk = topk;
  a.err = dev_err;
  a.pairs = pairs_of_64(c);
  a.joint = a.pairs ? 2 : 1;
  return run_rows(a, &a.cluster, n_tokens, topk, c.head_dim, kIn8,
                  rows8_bytes(n_tokens, topk, a.heads, a.hkv, c.head_dim), ws, ws_bytes, [&] {
                    const CUtensorMap maps[2] = {};
                    return from_cuda(launch_attn_rows8(a, c.head_dim, true, maps, stream));
                  });
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
