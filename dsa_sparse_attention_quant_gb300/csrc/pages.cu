// pages.cu — the paged KV cache's upkeep (sm_103a): writing the step's rows,
// and copying, forking, freeing and compacting pages.
//
// Bookkeeping is a reference count per page (0 = free), a block-table row and
// a length per sequence. All results are whole numbers or moved bytes and do
// not depend on the order in which threads run: free pages are taken lowest
// first in the order of the request list, and the k-th page that compaction
// moves goes to the k-th hole. The byte moves are bound by HBM, one read and
// one write of every moved page; the bookkeeping by a few dependent reads.
// Measured: 32768 rows of 8 x 128 written in 40 us (6.7 TB/s, read and write);
// 0.5 GB of pages moved by a compaction over 8 caches in 170 to 174 us (5.8 TB/s with
// the plan); 1024 pages copied over 4 caches in 180 us (6.0 TB/s with the claims), 64
// over 16 in 54; 64 forks over 16 caches 12 us on the GPU, about 30 us of host time.
// Each call's first kernel is launched while the stream's previous one drains (rows
// 44.2 -> 41.6 us), but for the page copies, whose claims begin with memsets.
#include "attn.h"
#include "common.cuh"

namespace dsa {

namespace {

// ------------------------------------------------------------------ kv write
// A warp per token: both rows' 16-byte chunks, eight in flight per lane. Bound
// by HBM, one read and one write of the rows.
constexpr int kWriteThreads = 256;

template <int D>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const __grid_constant__ KvWriteArgs a) {
  pdl_wait();
  constexpr int CH = D / 8;
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kWriteThreads + threadIdx.x) >> 5;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kWriteThreads / 32);
  const int chunks = a.hkv * CH;
  for (int64_t t = warp; t < a.n_tokens; t += warps) {
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0 || slot >= a.num_slots) {
      if (slot != -1 && lane == 0) flag_error(a.err, DSA_DEVERR_SLOT_RANGE);
      continue;
    }
    const int64_t page = slot / kBlock, off = slot % kBlock;
    const uint16_t *ks = a.k + t * a.k_row, *vs = a.v + t * a.v_row;
    uint16_t *kd = a.kc + page * a.k_page + off * a.k_slot, *vd = a.vc + page * a.v_page + off * a.v_slot;
    for (int c0 = lane; c0 < chunks; c0 += 32 * U) {
      uint4 kx[U], vx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * u;
        if (c < chunks) {
          kx[u] = *reinterpret_cast<const uint4*>(ks + (c / CH) * a.k_rhead + (c % CH) * 8);
          vx[u] = *reinterpret_cast<const uint4*>(vs + (c / CH) * a.v_rhead + (c % CH) * 8);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * u;
        if (c < chunks) {
          *reinterpret_cast<uint4*>(kd + (c / CH) * a.k_head + (c % CH) * 8) = kx[u];
          *reinterpret_cast<uint4*>(vd + (c / CH) * a.v_head + (c % CH) * 8) = vx[u];
        }
      }
    }
  }
}

// ----------------------------------------------------------------- the copies
// A page of a cache is copied in parts of 32 KB, a CTA's eight 16-byte chunks
// per thread in flight; parts are numbered pair-major over all caches.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
static_assert(kPartBytes == kCopyThreads * kCopyUnroll * 16, "a CTA copies a whole part");

__device__ __forceinline__ void copy_part(const CacheList& cl, int part, int64_t src, int64_t dst) {
  int c = 0;
  while (c + 1 < cl.n && part >= cl.parts_end[c]) ++c;
  const int64_t off = static_cast<int64_t>(part - (c > 0 ? cl.parts_end[c - 1] : 0)) * kPartBytes;
  const int64_t left = cl.page_bytes[c] - off;
  const uint8_t* s = cl.base[c] + src * cl.page_stride[c] + off;
  uint8_t* d = cl.base[c] + dst * cl.page_stride[c] + off;
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int64_t at = (static_cast<int64_t>(u) * kCopyThreads + threadIdx.x) * 16;
    if (at < left) v[u] = *reinterpret_cast<const uint4*>(s + at);
  }
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int64_t at = (static_cast<int64_t>(u) * kCopyThreads + threadIdx.x) * 16;
    if (at < left) *reinterpret_cast<uint4*>(d + at) = v[u];
  }
}

// Which pairs of a copy list stand: the lowest entry of each destination, and
// none whose destination is also a source.
__global__ void __launch_bounds__(256) copy_claim_kernel(const __grid_constant__ PagesArgs p) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.n) return;
  const int32_t s = p.a[i], d = p.b[i];
  if (s < 0 || d < 0 || s >= p.num_blocks || d >= p.num_blocks || s == d) return;
  atomicMin(p.w0 + d, i);
  p.w1[s] = 0;
}

__global__ void __launch_bounds__(kCopyThreads) copy_pairs_kernel(const __grid_constant__ PagesArgs p,
                                                                  const __grid_constant__ CacheList cl) {
  const int64_t units = static_cast<int64_t>(p.n) * cl.parts;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = static_cast<int>(u / cl.parts), part = static_cast<int>(u - static_cast<int64_t>(i) * cl.parts);
    const int32_t s = p.a[i], d = p.b[i];
    if (s == -1 || d == -1 || s == d) continue;
    if (s < 0 || d < 0 || s >= p.num_blocks || d >= p.num_blocks) {
      if (threadIdx.x == 0) flag_error(p.err, DSA_DEVERR_BLOCK_RANGE);
      continue;
    }
    if (p.w0[d] != i || p.w1[d] == 0) {
      if (threadIdx.x == 0) flag_error(p.err, DSA_DEVERR_PAGE_STATE);
      continue;
    }
    copy_part(cl, part, s, d);
  }
}

// ----------------------------------------------------------------------- fork
constexpr int kForkThreads = 1024;
constexpr int kForkUnclaim = 2;  // an entry's state until its child is empty again

// One CTA: checks the list, takes the fresh pages. entry[i] = {parent's last
// page, fresh page, parent's length, state}; state 0 = skipped. A child that was
// claimed and then skipped is empty again.
__global__ void __launch_bounds__(kForkThreads) fork_plan_kernel(const __grid_constant__ PagesArgs p) {
  __shared__ int scan[33];
  const int tid = threadIdx.x;
  pdl_wait();
  const int64_t most = p.bt_stride * kBlock;
  // lengths before any child is written
  for (int i = tid; i < p.n; i += kForkThreads) {
    const int32_t a = p.a[i], b = p.b[i];
    int state = 0, len = 0;
    if (a < 0 || a >= p.n_rows || b < 0 || b >= p.n_rows) {
      flag_error(p.err, DSA_DEVERR_SEQ_RANGE);
    } else {
      len = p.seq_lens[a];
      if (len < 0 || len > most)
        flag_error(p.err, DSA_DEVERR_SEQ_RANGE);
      else if (p.seq_lens[b] != 0)
        flag_error(p.err, DSA_DEVERR_PAGE_STATE);
      else
        state = 1;
    }
    p.entry[i] = make_int4(-1, -1, len, state);
  }
  __syncthreads();
  // a child named twice is the first entry's: the claims are negative lengths
  for (int i = tid; i < p.n; i += kForkThreads)
    if (p.entry[i].w) atomicMin(p.seq_lens + p.b[i], i - p.n);
  __syncthreads();
  int need = 0, tot;
  for (int i0 = 0; i0 < p.n; i0 += kForkThreads) {
    const int i = i0 + tid;
    int part = 0;
    if (i < p.n && p.entry[i].w) {
      if (*reinterpret_cast<volatile int32_t*>(p.seq_lens + p.b[i]) != i - p.n) {
        p.entry[i].w = 0;
        flag_error(p.err, DSA_DEVERR_PAGE_STATE);
      } else if (p.entry[i].z % kBlock != 0) {
        const int32_t src = p.block_table[p.a[i] * p.bt_stride + p.entry[i].z / kBlock];
        const bool in = src >= 0 && src < p.num_blocks;
        part = in && p.refs[src] > 0;
        p.entry[i].x = src;
        if (!part) {  // nothing to copy, or a page that may be another child's fresh one
          p.entry[i].w = kForkUnclaim;
          flag_error(p.err, in ? DSA_DEVERR_PAGE_STATE : DSA_DEVERR_BLOCK_RANGE);
        }
      }
    }
    const int incl = block_scan_incl(part, scan, &tot);
    if (part) p.entry[i].y = need + incl - 1;  // rank among the fresh pages
    need += tot;
  }
  // the lowest free pages
  int found = 0;
  for (int64_t c0 = 0; c0 < p.num_blocks && found < need; c0 += kForkThreads * 8) {
    const int64_t at = c0 + tid * 8;
    uint32_t bits = 0;
    if (at + 8 <= p.num_blocks) {
      const int4 x = *reinterpret_cast<const int4*>(p.refs + at), y = *reinterpret_cast<const int4*>(p.refs + at + 4);
      bits = (x.x == 0) | (x.y == 0) << 1 | (x.z == 0) << 2 | (x.w == 0) << 3 | (y.x == 0) << 4 | (y.y == 0) << 5 |
             (y.z == 0) << 6 | (y.w == 0) << 7;
    } else {
      for (int e = 0; e < 8 && at + e < p.num_blocks; ++e) bits |= static_cast<uint32_t>(p.refs[at + e] == 0) << e;
    }
    int k = found + block_scan_incl(__popc(bits), scan, &tot) - __popc(bits);
    for (; bits != 0 && k < need; bits &= bits - 1) p.fresh[k++] = static_cast<int32_t>(at + __ffs(bits) - 1);
    found += tot;
  }
  if (tid == 0) p.counts[0] = found < need ? found : need;  // fresh pages taken
  __syncthreads();
  for (int i = tid; i < p.n; i += kForkThreads) {
    int4 e = p.entry[i];
    if (!e.w) continue;
    const int32_t b = p.b[i];
    if (e.z % kBlock != 0) {
      if (e.w != kForkUnclaim && e.y >= found) {  // no page left
        flag_error(p.err, DSA_DEVERR_NO_PAGE);
        e.w = kForkUnclaim;
      }
      if (e.w == kForkUnclaim) {
        p.seq_lens[b] = 0;
        p.entry[i].w = 0;
        continue;
      }
      const int32_t dst = p.fresh[e.y];
      p.refs[dst] = 1;
      p.w0[dst] = e.y;
      p.block_table[b * p.bt_stride + e.z / kBlock] = dst;
      e.y = dst;
    }
    p.seq_lens[b] = e.z;
    p.entry[i] = e;
  }
}

// The children's shared pages (CTAs [0, n), first launch only) and the copies
// of the part-filled last pages. A shared page whose count was not positive is
// flagged; one that the plan took has count 1 by now, and is known as taken by its
// rank: w0 may hold anything for other pages, but then the rank's page is another.
__global__ void __launch_bounds__(kCopyThreads) fork_move_kernel(const __grid_constant__ PagesArgs p,
                                                                 const __grid_constant__ CacheList cl, int tables) {
  pdl_wait();
  if (static_cast<int>(blockIdx.x) < tables) {
    const int taken = p.counts[0];
    for (int i = blockIdx.x; i < p.n; i += tables) {
      const int4 e = p.entry[i];
      if (!e.w) continue;
      const int32_t *from = p.block_table + p.a[i] * p.bt_stride;
      int32_t* to = p.block_table + p.b[i] * p.bt_stride;
      for (int j = threadIdx.x; j < e.z / kBlock; j += kCopyThreads) {
        const int32_t id = from[j];
        to[j] = id;
        if (id < 0 || id >= p.num_blocks) {
          flag_error(p.err, DSA_DEVERR_BLOCK_RANGE);
          continue;
        }
        const int k = p.w0[id];
        if (atomicAdd(p.refs + id, 1) <= 0 || (k >= 0 && k < taken && p.fresh[k] == id))
          flag_error(p.err, DSA_DEVERR_PAGE_STATE);
      }
    }
    return;
  }
  const int64_t units = static_cast<int64_t>(p.n) * cl.parts;
  for (int64_t u = blockIdx.x - tables; u < units; u += gridDim.x - tables) {
    const int i = static_cast<int>(u / cl.parts);
    const int4 e = p.entry[i];
    if (!e.w || e.x < 0) continue;
    copy_part(cl, static_cast<int>(u - static_cast<int64_t>(i) * cl.parts), e.x, e.y);
  }
}

// ----------------------------------------------------------------------- free
// A CTA per row. Each table entry is taken by an exchange, so a row named
// twice gives its pages back once.
__global__ void __launch_bounds__(256) pages_free_kernel(const __grid_constant__ PagesArgs p) {
  pdl_wait();
  const int32_t row = p.a[blockIdx.x];
  if (row < 0 || row >= p.n_rows) {
    if (threadIdx.x == 0) flag_error(p.err, DSA_DEVERR_SEQ_RANGE);
    return;
  }
  const int32_t len = *reinterpret_cast<volatile int32_t*>(p.seq_lens + row);
  __syncthreads();  // read by all before it is cleared
  if (len < 0 || len > p.bt_stride * kBlock) {
    if (threadIdx.x == 0) flag_error(p.err, DSA_DEVERR_SEQ_RANGE);
    return;
  }
  int32_t* bt = p.block_table + row * p.bt_stride;
  const int pages = (len + kBlock - 1) / kBlock;
  for (int j = threadIdx.x; j < pages; j += 256) {
    const int32_t id = atomicExch(bt + j, -1);
    if (id == -1) continue;  // taken by the row's other entry
    if (id < 0 || id >= p.num_blocks) {
      flag_error(p.err, DSA_DEVERR_BLOCK_RANGE);
    } else if (atomicSub(p.refs + id, 1) <= 0) {
      atomicAdd(p.refs + id, 1);
      flag_error(p.err, DSA_DEVERR_PAGE_STATE);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.seq_lens[row] = 0;
}

// -------------------------------------------------------------------- compact
constexpr int kScanThreads = 256;
constexpr int kPerThread = kPageChunk / kScanThreads;

// Live bits of this thread's pages [at, at + kPerThread).
__device__ __forceinline__ uint32_t live_bits(const PagesArgs& p, int64_t at) {
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e)
    if (at + e < p.num_blocks) bits |= static_cast<uint32_t>(p.refs[at + e] > 0) << e;
  return bits;
}

__global__ void __launch_bounds__(kScanThreads) compact_count_kernel(const __grid_constant__ PagesArgs p) {
  __shared__ int scan[33];
  pdl_wait();
  const uint32_t bits = live_bits(p, static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x * kPerThread);
  int tot;
  block_scan_incl(__popc(bits), scan, &tot);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = tot;
}

// With U live pages: the k-th hole below U into w0[k], the k-th live page at
// or above U into w1[k], and w2[page] = k for those (-1 for every other page).
__global__ void __launch_bounds__(kScanThreads) compact_rank_kernel(const __grid_constant__ PagesArgs p) {
  __shared__ int scan[33];
  pdl_wait();
  int tot, before = 0, all = 0;
  for (int c0 = 0; c0 < static_cast<int>(gridDim.x); c0 += kScanThreads) {
    const int c = c0 + threadIdx.x;
    const int v = c < static_cast<int>(gridDim.x) ? p.counts[c] : 0;
    block_scan_incl(v, scan, &tot);
    all += tot;
    block_scan_incl(c < static_cast<int>(blockIdx.x) ? v : 0, scan, &tot);
    before += tot;
  }
  const int64_t U = all;
  // live pages below U: whole chunks, then the chunk that U falls into
  const int cu = static_cast<int>(U / kPageChunk);
  int below = 0;
  for (int c0 = 0; c0 < cu; c0 += kScanThreads) {
    const int c = c0 + threadIdx.x;
    block_scan_incl(c < cu ? p.counts[c] : 0, scan, &tot);
    below += tot;
  }
  {
    const int64_t at = static_cast<int64_t>(cu) * kPageChunk + threadIdx.x * kPerThread;
    uint32_t bits = live_bits(p, at);
    const int64_t keep = U - at;
    if (keep < kPerThread) bits = keep <= 0 ? 0 : bits & ((1u << keep) - 1u);
    block_scan_incl(__popc(bits), scan, &tot);
    below += tot;
  }
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x * kPerThread;
  const uint32_t bits = live_bits(p, at);
  int live = before + block_scan_incl(__popc(bits), scan, &tot) - __popc(bits);  // live pages before `at`
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int64_t i = at + e;
    if (i >= p.num_blocks) break;
    const bool on = (bits >> e) & 1;
    int k = -1;
    if (!on && i < U) p.w0[i - live] = static_cast<int32_t>(i);
    if (on && i >= U) {
      k = live - below;
      p.w1[k] = static_cast<int32_t>(i);
    }
    p.w2[i] = k;
    live += on;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.counts[gridDim.x] = all - below;
}

// The moves: bytes, counts and table entries (the latter two by `books` CTAs,
// first launch only).
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const __grid_constant__ PagesArgs p,
                                                                    const __grid_constant__ CacheList cl, int chunks,
                                                                    int books) {
  pdl_wait();
  const int moved = p.counts[chunks];
  if (static_cast<int>(blockIdx.x) < books) {
    const int64_t step = static_cast<int64_t>(books) * kCopyThreads;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
    for (int64_t k = t0; k < moved; k += step) {
      const int32_t s = p.w1[k];
      p.refs[p.w0[k]] = p.refs[s];
      p.refs[s] = 0;
    }
    const int64_t entries = static_cast<int64_t>(p.n_rows) * p.bt_stride;
    for (int64_t j = t0; j < entries; j += step) {
      const int32_t id = p.block_table[j];
      if (id < 0 || id >= p.num_blocks) continue;
      const int32_t k = p.w2[id];
      if (k >= 0) p.block_table[j] = p.w0[k];
    }
    return;
  }
  const int64_t units = static_cast<int64_t>(moved) * cl.parts;
  for (int64_t u = blockIdx.x - books; u < units; u += gridDim.x - books) {
    const int64_t k = u / cl.parts;
    copy_part(cl, static_cast<int>(u - k * cl.parts), p.w1[k], p.w0[k]);
  }
}

// CTAs that copy: eight per SM, fewer for little work. (Five of them fit at
// once; with four per SM, all resident, a 1 GB move took 184 us, so 178.)
int copy_ctas(int64_t units, int num_sms) {
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(units < cap ? (units > 0 ? units : 1) : cap);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  const int64_t per = kWriteThreads / 32;
  int64_t grid = (a.n_tokens + per - 1) / per;
  // a warp per token as a rule: with eight CTAs per SM looping over the tokens,
  // 32768 tokens of 8 x 128 took 45.8 us, so 44.1
  const int64_t cap = static_cast<int64_t>(num_sms) * 64;
  if (grid > cap) grid = cap;
  if (head_dim == 128)
    return launch_pdl(kv_write_kernel<128>, dim3(static_cast<unsigned>(grid)), dim3(kWriteThreads), 0, stream, a);
  return launch_pdl(kv_write_kernel<64>, dim3(static_cast<unsigned>(grid)), dim3(kWriteThreads), 0, stream, a);
}

cudaError_t launch_pages_copy(const PagesArgs& p, const CacheList* lists, int n_lists, int num_sms,
                              cudaStream_t stream) {
  // claims start above every entry; 0x7F bytes are larger than any index, and nonzero marks "not a source"
  cudaError_t e = cudaMemsetAsync(p.w0, 0x7F, static_cast<size_t>(p.num_blocks) * 4, stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(p.w1, 0x7F, static_cast<size_t>(p.num_blocks) * 4, stream);
  if (e != cudaSuccess) return e;
  copy_claim_kernel<<<(p.n + 255) / 256, 256, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  for (int i = 0; i < n_lists; ++i) {
    copy_pairs_kernel<<<copy_ctas(static_cast<int64_t>(p.n) * lists[i].parts, num_sms), kCopyThreads, 0, stream>>>(
        p, lists[i]);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_pages_fork(const PagesArgs& p, const CacheList* lists, int n_lists, int num_sms,
                              cudaStream_t stream) {
  cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kForkThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n_lists; ++i) {
    const int tables = i == 0 ? (p.n < num_sms ? p.n : num_sms) : 0;
    const int grid = tables + (lists[i].n > 0 ? copy_ctas(static_cast<int64_t>(p.n) * lists[i].parts, num_sms) : 0);
    if ((e = launch_pdl(fork_move_kernel, dim3(grid), dim3(kCopyThreads), 0, stream, p, lists[i], tables)) !=
        cudaSuccess)
      return e;
  }
  return cudaSuccess;
}

cudaError_t launch_pages_free(const PagesArgs& p, cudaStream_t stream) {
  return launch_pdl(pages_free_kernel, dim3(p.n), dim3(256), 0, stream, p);
}

cudaError_t launch_pages_compact(const PagesArgs& p, const CacheList* lists, int n_lists, int num_sms,
                                 cudaStream_t stream) {
  const int chunks = static_cast<int>((p.num_blocks + kPageChunk - 1) / kPageChunk);
  cudaError_t e = launch_pdl(compact_count_kernel, dim3(chunks), dim3(kScanThreads), 0, stream, p);
  if (e == cudaSuccess) e = launch_pdl(compact_rank_kernel, dim3(chunks), dim3(kScanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  const int64_t entries = static_cast<int64_t>(p.n_rows) * p.bt_stride;
  for (int i = 0; i < n_lists; ++i) {
    const int64_t want = (entries + 8 * kCopyThreads - 1) / (8 * kCopyThreads) + 1;
    const int books = i == 0 ? static_cast<int>(want < num_sms ? want : num_sms) : 0;
    // the number of moved pages is not known here: CTAs without a part return at once
    const int copies = lists[i].n > 0 ? copy_ctas((p.num_blocks + 1) / 2 * lists[i].parts, num_sms) : 0;
    if ((e = launch_pdl(compact_move_kernel, dim3(books + copies), dim3(kCopyThreads), 0, stream, p, lists[i], chunks,
                        books)) != cudaSuccess)
      return e;
  }
  return cudaSuccess;
}

}  // namespace dsa
