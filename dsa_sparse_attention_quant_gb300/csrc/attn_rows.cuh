// attn_rows.cuh — what the kernels over single query rows share (attn_rows.cu for
// caches in 16 bits, attn_rows8.cu in 8): the element types, the asynchronous loads,
// and how the (token, 64-key tile) list is cut into slices.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace dsa {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 64;                 // keys per tile = slots per page
constexpr int kWarpKeys = kTile / kWarps;  // 16: one MMA k step
static_assert(kTile == kBlock, "a tile is one page");

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  // p_j <= 2^8 while M lags by up to 8; bf16 has fp32's exponents.
  static constexpr float kHead = 0.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Elem<__half> {
  // M sits 6 below the maximum, so p_j reaches 2^14 at most (fp16 holds
  // 65504) and fp16's smallest step, 2^-24, is 2^-30 of the largest weight.
  static constexpr float kHead = 6.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
// M moves only when a score passes it by more than this many powers of two:
// rescaling O costs more than the range it saves.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes global -> shared, zeros when `in` is false (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Half of 2^d's exponent: sums that have to come further down than 2^-126 at a time are multiplied
// by it twice. Where V's scales are in the weights (attn_rows8.cu), a part's sum may be 2^78 a key
// and its reference 190 below the row's, and it a good part of the row's sum all the same.
__device__ __forceinline__ float half_way(float d) { return ex2(0.5f * d); }

// What a stage holds, written by the loader and read when it is consumed.
enum : int { kFirst = 1, kLast = 2, kStartsItem = 4, kEndsItem = 8 };

// Keys a decode token sees, or 0 (a padding token, or flagged metadata), and
// its request's block-table row.
__device__ __forceinline__ int token_keys(const RowsArgs& a, int t, int* req, bool flag) {
  // token t mostly belongs to request t: that one's metadata is read beside its id, not after it
  const int r = a.req_id[t];
  const bool guess = t < a.num_reqs;
  int q0 = guess ? a.qsl[t] : 0, q1 = guess ? a.qsl[t + 1] : 0, sl = guess ? a.seq_lens[t] : 0;
  *req = 0;
  if (r < 0 || r >= a.num_reqs) {
    if (flag) flag_error(a.err, DSA_DEVERR_SEQ_RANGE);
    return 0;
  }
  *req = r;
  if (r != t) {
    q0 = a.qsl[r];
    q1 = a.qsl[r + 1];
    sl = a.seq_lens[r];
  }
  if (t < q0 || t >= q1 || sl < 0 || sl > a.max_keys) {
    if (flag) flag_error(a.err, DSA_DEVERR_SEQ_RANGE);
    return 0;
  }
  return max(0, sl - (q1 - t) + 1);
}

// (n up to 2^31 - 1)
__device__ __forceinline__ int tiles_of(int n) { return n > 0 ? (n - 1) / kTile + 1 : 1; }

// The tiles of a CTA's slice, in order.
struct Cursor {
  int t, kt;     // token, tile of the token
  int tiles, n;  // of this token
  int req;
  int left;      // tiles of the slice not yet taken
  bool fresh;    // the next tile is the first of its item in this slice
};

template <bool SEL>
__device__ __forceinline__ void enter_token(const RowsArgs& a, Cursor& c) {
  if (SEL) {
    c.n = a.topk;
    c.tiles = tiles_of(a.topk);
    c.req = 0;
  } else {
    c.n = token_keys(a, c.t, &c.req, false);
    c.tiles = tiles_of(c.n);
  }
}

// What find_slice() finds, in shared memory.
struct Slice {
  int64_t all, end;  // tiles in all, end of this slice
  int t, kt;         // its first token and that token's tile
  int left;          // its tiles
  int in_use;        // slices in use
  int n, req;        // of the first token
};

// Split mode: slice `part` of the flat tile list, many tokens counted in rounds of
// kPer a thread: their metadata's latency is what a round takes (4096 requests of
// 300 keys, 32/8 heads of 128: 801 us with rounds of one a thread and a second
// pass over all of them, so 780). All THREADS threads call; rounds[kRounds] is scratch.
constexpr int kPer = 4, kRounds = 1024;
template <bool SEL, int THREADS = kThreads>
__device__ void find_slice(const RowsArgs& a, int part, bool flag, Slice* s, int* scan, int* rounds) {
  const int T = a.n_tokens, tid = threadIdx.x;
  int tot, n[kPer], req[kPer], tiles[kPer], first = 0;  // of this thread's tokens of the last counted round
  int64_t total = 0;
  const int per = T <= THREADS ? 1 : kPer;
  auto count = [&](int c0, bool f) {
    int sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = c0 + tid * per + e;
      n[e] = req[e] = tiles[e] = 0;
      if (e < per && t < T) {
        n[e] = token_keys(a, t, &req[e], f);
        tiles[e] = tiles_of(n[e]);
      }
      sum += tiles[e];
    }
    first = block_scan_incl(sum, scan, &tot) - sum;
  };
  constexpr int R = THREADS * kPer;
  if (SEL) {
    total = static_cast<int64_t>(T) * tiles_of(a.topk);
  } else {
    for (int c0 = 0, i = 0; c0 < T; c0 += R, ++i) {
      count(c0, flag);
      if (tid == 0 && i < kRounds) rounds[i] = tot;
      total += tot;
    }
    __syncthreads();
  }
  const int64_t most = (total + a.min_tiles - 1) / a.min_tiles;
  const int use = static_cast<int>(most < a.slices ? most : a.slices);
  const int64_t b0 = part < use ? total * part / use : total, b1 = part < use ? total * (part + 1) / use : total;
  if (tid == 0) {
    s->all = total;
    s->end = b1;
    s->left = static_cast<int>(b1 - b0);
    s->in_use = use;
  }
  if (b0 < b1) {
    if (SEL) {
      if (tid == 0) {
        const int each = tiles_of(a.topk);
        s->t = static_cast<int>(b0 / each);
        s->kt = static_cast<int>(b0 % each);
        s->n = a.topk;
        s->req = 0;
      }
    } else {
      int64_t carry = 0;
      int c0 = 0;
      for (int i = 0; i < kRounds && c0 < T && carry + rounds[i] <= b0; ++i, c0 += R) carry += rounds[i];
      for (; c0 < T && carry <= b0; c0 += R) {
        if (T > R) count(c0, false);
        int64_t at = carry + first;
#pragma unroll
        for (int e = 0; e < kPer; at += tiles[e], ++e) {
          if (at <= b0 && b0 < at + tiles[e]) {
            s->t = c0 + tid * per + e;
            s->kt = static_cast<int>(b0 - at);
            s->n = n[e];
            s->req = req[e];
          }
        }
        carry += tot;
      }
    }
  }
  __syncthreads();
}

}  // namespace dsa
