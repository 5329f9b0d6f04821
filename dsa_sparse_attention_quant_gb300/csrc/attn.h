// attn.h — host-side launchers of the attention and page kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dsaidx.h"

namespace dsa {

// All but the page copies' kernels are launched while the stream's previous kernel
// runs, and wait for it before they read anything. What they read behind that wait
// is read with plain loads: __ldg and const __restrict__ are for what nobody writes
// as long as the kernel lives, and such loads may move ahead of the wait.

// Single query rows over the paged cache (attn_rows.cu). Strides in elements.
struct RowsArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;  // [rows, heads] or nullptr
  int64_t q_row, q_head, out_row, out_head;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
  int heads, hkv, group;  // query heads, KV heads, query heads per KV head
  int passes;             // passes over the keys: the group's heads in 16- or 32-row tiles
  float scale_log2;       // softmax scale * log2(e)
  int n_tokens;
  // dense: the decode tokens' pages
  const int32_t *qsl, *seq_lens, *req_id, *block_table;
  int64_t bt_stride, num_blocks;
  int num_reqs;   // decode requests
  int max_keys;   // keys a block-table row can name
  // selected
  const int32_t* physical;  // [n_tokens, topk]
  int topk;
  int64_t num_slots;
  // work: split: slices of at least min_tiles tiles of the flat tile list, else
  // a token per slice; a CTA per slice, `joint` KV heads and pass
  int slices, min_tiles;
  int joint;  // 1 or 2
  bool split;
  int2* desc;       // [CTAs]: {token begun here and continued, its last slice}
  float2* part_ml;  // [2 * CTAs][joint][rows of a pass]
  float* part_o;    // [2 * CTAs][joint][rows of a pass][D]
  int32_t* err;
};
// How the kernels take work, for the host's plan, which sizes the scratch that they write:
// a pass's rows (query heads of a KV head), and CTAs per SM.
constexpr int rows_of(int group) { return group <= 16 ? 16 : 32; }
constexpr int rows8_of(int group) { return group <= 8 ? 8 : 16; }
constexpr int kRowsCtas = 2;
constexpr int rows8_ctas(int rows, int joint) { return rows * joint > 16 ? 2 : 3; }  // what registers allow
constexpr int kMostCluster = 8;
cudaError_t launch_attn_rows(const RowsArgs& a, int head_dim, int dtype, bool selected, cudaStream_t stream);

// The parts that the slices of attn_rows8.cu left, added (attn_rows.cu): krows rows of the
// workspace a CTA and KV head.
cudaError_t launch_attn_join8(const RowsArgs& a, int head_dim, bool bf16, int krows, cudaStream_t stream);

// The same rows over a cache of E4M3 codes (attn_rows8.cu): k, v and their strides
// count bytes, the scales' strides count fp32 numbers.
struct Rows8Args : RowsArgs {
  const float* scale;  // [pages, 4, heads, 2]: a block of 16 slots' K and V scale
  int64_t s_page, s_block, s_head;
  bool bf16;   // of q and out; else fp16
  bool pairs;  // heads of 64 side by side, an even number of them
  int cluster;  // not split: CTAs that share a token's keys and join its rows among themselves
};
// maps: K and V as {row, rows of heads, 64 slots, pages}; not used for selected slots.
cudaError_t launch_attn_rows8(const Rows8Args& a, int head_dim, bool selected, const CUtensorMap* maps,
                              cudaStream_t stream);

// The cache of E4M3 codes, written and read back (kv8.cu). Strides as in Rows8Args;
// those of 16-bit rows in elements of 2 bytes.
struct Cache8Args {
  uint8_t *k, *v;
  float* scale;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head, s_page, s_block, s_head;
  int hkv;
  int64_t num_blocks;
};
struct Write8Args {
  Cache8Args c;
  const uint16_t *k, *v;
  int64_t k_row, k_rhead, v_row, v_rhead;
  int64_t n_tokens;
  const int64_t* slot_mapping;
  int32_t* token_of;  // [slots]: the last token with that slot, or anything; nullptr: few tokens
  int32_t* err;
};
// Up to this many tokens: one launch, without token_of. 8 heads of 128: 1000 rows of 2 sequences
// 8.5 us (with it 11), 600 of 600 sequences 8.6 (11); 2000 of 2 without it 11.5 (10.5), 1500 of
// 1500 16.3 (14.9).
constexpr int kWrite8Few = 1024;
cudaError_t launch_kv_write8(const Write8Args& a, int head_dim, int dtype, int num_sms, cudaStream_t stream);

struct Read8Args {
  Cache8Args c;
  uint16_t *k, *v;
  int64_t k_row, k_rhead, v_row, v_rhead;
  int64_t rows;  // of k and v
  const int32_t *qsl, *seq_lens, *block_table, *kv_start;
  int64_t bt_stride;
  int num_reqs, max_keys;
  bool past;  // without the requests' own query tokens
  int32_t* err;
};
cudaError_t launch_kv_read8(const Read8Args& a, int head_dim, int dtype, int num_sms, cudaStream_t stream);

// K and V rows into the paged cache (pages.cu). Strides in elements of 2 bytes.
struct KvWriteArgs {
  const uint16_t *k, *v;
  int64_t k_row, k_rhead, v_row, v_rhead;  // of the new rows
  uint16_t *kc, *vc;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
  int hkv;
  int64_t n_tokens, num_slots;
  const int64_t* slot_mapping;
  int32_t* err;
};
cudaError_t launch_kv_write(const KvWriteArgs& a, int head_dim, int num_sms, cudaStream_t stream);

// Page moves (pages.cu).
constexpr int kMaxCaches = 64;  // caches per copy launch
constexpr int kPartBytes = 32768;  // a CTA's piece of a page: what the lists count and the copies step by
struct CacheList {
  uint8_t* base[kMaxCaches];
  int64_t page_bytes[kMaxCaches];
  int64_t page_stride[kMaxCaches];
  int parts_end[kMaxCaches];  // running sum of the caches' copy parts per page
  int n;
  int parts;  // copy parts of one page over all caches
};
struct PagesArgs {
  int32_t* refs;
  int64_t num_blocks;
  int32_t* block_table;
  int64_t bt_stride;
  int32_t n_rows;
  int32_t* seq_lens;
  const int32_t *a, *b;  // parents/children, sources/destinations, rows/unused
  int32_t n;
  // workspace
  int32_t *w0, *w1, *w2;  // [num_blocks] each
  int32_t* counts;        // chunk counts, then the number of moved pages
  int4* entry;            // [n]
  int32_t* fresh;         // [n]
  int32_t* err;
};
constexpr int kPageChunk = 2048;  // pages per CTA of the compaction's scans
cudaError_t launch_pages_copy(const PagesArgs& p, const CacheList* lists, int n_lists, int num_sms, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesArgs& p, const CacheList* lists, int n_lists, int num_sms, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesArgs& p, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesArgs& p, const CacheList* lists, int n_lists, int num_sms,
                                 cudaStream_t stream);

// Prompts (attn_prompt.cu).
struct PromptArgs {
  void* out;
  float* lse;
  int64_t out_row, out_head;
  const void* v;  // plain access to V (the rare non-finite elements, see the kernel)
  int64_t v_page, v_slot, v_head;
  int heads, hkv, group;
  float scale_log2;
  const int32_t *qsl, *seq_lens, *block_table, *kv_start;  // kv_start: packed keys, else nullptr
  int64_t bt_stride, num_blocks;  // packed: num_blocks = rows of k and v
  int num_reqs, num_decodes, num_tokens, first_token;
  int max_keys;
  int head_units;  // CTAs across the heads
  int tile_units;  // CTAs across the query tiles (upper bound)
  bool pair_heads; // a CTA's two query tiles: two heads, or two token tiles of one head
  int32_t* err;
};
cudaError_t launch_attn_prompt(const PromptArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                               const CUtensorMap* mv, int head_dim, int dtype, cudaStream_t stream);

}  // namespace dsa
