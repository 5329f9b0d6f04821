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
  // a token per slice; a CTA per slice, KV head and pass
  int slices, min_tiles;
  bool split;
  int2* desc;       // [CTAs]: {token begun here and continued, its last slice}
  float2* part_ml;  // [2 * CTAs][rows of a pass]
  float* part_o;    // [2 * CTAs][rows of a pass][D]
  int32_t* err;
};
cudaError_t launch_attn_rows(const RowsArgs& a, int head_dim, int dtype, bool selected, cudaStream_t stream);

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
