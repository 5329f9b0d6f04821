// attn_prompt.cu — causal attention over prompts on the tcgen05 tensor cores
// (sm_103a), keys in the paged cache or packed beside the queries.
//
//   S = Q K^T,  P = 2^(S scale log2(e) - M),  O = P V,  out = O / sum(P),
//   lse = ln 2 * (M + log2 sum(P))
// tile by tile over the keys. Any M gives the same quotient; it only has to
// keep P in range. So a row's M is the maximum of the first 32 columns it sees
// (all 128 of the tile: 2000 cycles more per unit; 512 prompts of 128, 16/2 heads
// of 128, 171 us, so 153), and P of a tile is computed by the M at hand:
// only when a row's weights come out too large is M raised (its O and sum
// rescaled) and P computed again. M never sits above a score that was seen, so
// the weights cannot all underflow. The rescaling of O, a round trip through
// TMEM, is rare, and the softmax warps do it themselves.
//
// What bounds it: 4*D operations per (query head, visible pair), the bf16 /
// fp16 rate of the tensor cores, with 128x128 tiles of S needing one exponential
// per 4*D operations beside it. Measured: 4 x 8192, 64/8 heads of 128, 2.54 ms in
// single calls at 2070 MHz (1730 TFLOP/s), 2.75 ms one call after the other under the
// power cap, at 1840 MHz in the median (1600);
// 2 x 8192, 32/8 heads of 64, 497 us (1105 TFLOP/s): there a tile pair's
// exponentials and the rest of its softmax, 2100 cycles, outlast its MMAs, 1024.
// Short prompts are a chain per unit (scores, weights, P V, the store), 9000
// cycles: 512 prompts of 128, 16/2 heads of 128, 144 us; one of 509, 11.4 us
// (14.4 when it did not start while the previous kernel drained).
// A unit's keys are not split: few query rows behind many keys are as many chains
// as there are units (128 tokens behind 128K keys, 32/8 heads: 16 units, 1.33 ms for
// 0.14 of operations; 8 tokens the same, 0.08 of bytes).
//
// Mapping: a CTA holds two query tiles of 128 rows that share one stream of
// K and V tiles (128 keys): two query heads of one KV head where the group is
// even, else two consecutive token tiles of one head. While one tile's softmax
// runs, the tensor cores run the other tile's P V and next Q K^T.
//  * warps 0-3 / 4-7: softmax of tile 0 / 1, a row per thread: S from TMEM, P
//    back to TMEM as the A operand of P V (never through shared memory),
//    rescaling, and the final store.
//  * warp 8: TMA. K and V tiles take turns in one ring (D = 128: five 32 KB
//    stages, D = 64: twelve of 16 KB); a page (64 slots of a head) is one box per
//    64 columns.
//  * warp 9: issues the MMAs, the tiles taking turns. V is read as stored, keys
//    along rows: B is "MN-major", K and Q are K-major; all in the 128-byte
//    swizzle.
//  * TMEM: O of both tiles (2 x D columns) and buffers of S (128 columns), P over
//    its S. D = 128: a buffer for each tile. D = 64: room for three that all steps
//    take in turn, so that a step's Q K^T is issued three steps ahead and the
//    softmax warps, which bound it there, find their next scores ready (5% less
//    at 2 x 8192, 32/8 heads, than two buffers and P beside them).
// CTAs are numbered from the last query tile of the last request down, so the
// longest tiles start first and the short ones fill the tail.
//
// V rows a tile holds but a row may not see meet P = 0 in the MMA, and 0 * NaN
// is NaN: in the tiles cut by the causal edge or by the sequence's end, the
// softmax warps first clear the rows behind the sequence and any non-finite V
// element; rows that do see such an element get it added back at the end, but
// for rows whose scores are all -infinity.
#include "attn.h"
#include "common.cuh"

namespace dsa {

namespace {

constexpr int kRowsTile = 128;  // query rows per tile
constexpr int kKeys = 128;      // keys per tile
constexpr int kSoftWarps = 8;
// Three warpgroups, the third with two idle warps: registers move between
// warpgroups (PromptCfg), from 168 a thread at launch (384 * 168 = 64512).
constexpr int kPromptThreads = 32 * (kSoftWarps + 4);
constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;

template <int D>
struct PromptCfg {
  static constexpr int kTileBytes = kKeys * D * 2;      // a Q, K or V tile
  static constexpr int kBoxBytes = kBlock * 128;        // 64 slots of 64 columns
  static constexpr int kColBytes = kKeys * 128;         // 64 columns of a tile
  static constexpr int kStages = D == 128 ? 5 : 12;
  static constexpr int kOffKv = 2 * kTileBytes;
  static constexpr int kOffBar = kOffKv + kStages * kTileBytes;
  // Buffers of S that the tiles take in turn, P over its S. D = 128: TMEM holds
  // one for each tile. D = 64: three for both, so a tile's next scores are there
  // when its weights are done.
  static constexpr bool kRing = D == 64;
  static constexpr int kBufs = kRing ? 3 : 1;  // of a tile at a time, at most
  static constexpr int kNumBars = 2 * kStages + 2 * 2 + 2 * kBufs + 3 + 2 * 2 + 2 * 2 + 1 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffNext = (kOffMisc + 16 + 15) / 16 * 16;  // the 16 bytes of a taken-over CTA's index
  static constexpr int kOffCta = kOffNext + 16;
  static constexpr int kSmemBytes = kOffCta + 2 * 96 + 1024;  // + slack to align the base to 1024
  // Registers of the softmax warps (a row of S) and of the others. At 2 x 8192, 32/8
  // heads: D = 64 with 208/88 508 us, so 501; D = 128 with 200/104 651 us, so 638.
  static constexpr int kSoftRegs = D == 128 ? 208 : 200, kIssueRegs = D == 128 ? 88 : 104;
  static_assert(32 * kSoftWarps * kSoftRegs + 128 * kIssueRegs <= kPromptThreads * 168, "register split");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kO = kRing ? 3 * kKeys : 2 * kKeys;  // first column of O
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(kO + 2 * D <= kTmemCols, "TMEM budget");
};

template <typename T>
struct PElem;
template <>
struct PElem<__nv_bfloat16> {
  static constexpr uint32_t kFmt = 1;
  // bf16 has fp32's exponents: a tile's weights may sum to 2^30 before the reference
  // moves. O is their product with V, not yet divided: |v| < 2^98 / tiles stays finite.
  static constexpr float kHead = 0.0f, kMaxSum = 1073741824.0f;
  static constexpr uint32_t kExp = 0x7F80u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct PElem<__half> {
  static constexpr uint32_t kFmt = 0;
  // The reference is set 4 below a maximum and moves when a row's weights in a
  // tile sum to more than 2^15 (fp16 holds 65504): the least step of a weight,
  // 2^-24, is 2^-28 of the largest or less.
  static constexpr float kHead = 4.0f, kMaxSum = 32768.0f;
  static constexpr uint32_t kExp = 0x7C00u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// Volatile: the order in which weights() issues them is kept.
__device__ __forceinline__ float pex2(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Instruction descriptor of kind::f16 -> fp32, M = 128.
__host__ __device__ constexpr uint32_t f16_idesc(uint32_t fmt, int N, bool b_mn_major) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (128u >> 4 << 24);
}

// Shared-memory matrix descriptors, both with the 128-byte swizzle and 8-row
// groups 1024 bytes apart: the high word is one constant, the low word holds
// the start address (16-byte units) and, for a tile stored row by row along the
// reduction (V, keys along rows: "MN-major"), the distance of the next 64
// columns. K-major: sw128_kmajor_desc of the shared header, split.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t kmajor_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (static_cast<uint32_t>((kKeys * 128) >> 4) << 16);
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
      "%6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// This warp's 32 TMEM lanes, 32 columns (the counterpart of tmem_ld32).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32}; " ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The request and query tile of one unit, found from the metadata.
struct PromptTile {
  int req;
  int t0, ntok;   // first token (row of q) of the CTA's rows, tokens left in the request from there
  int pos0;       // position of the first token
  int keys;       // the request's keys
  int kv0;        // packed: row of key 0
  bool found;
};

// Where a search ended: 32 requests from the base-th last one, `before` units
// behind them, and the number of all units once it is known. A CTA's units come
// in rising order as a rule, so the next search starts there (4096 prompts of
// 128, 16/2 heads of 128: 1.33 ms; from the last request each time 8.8).
struct PromptFind {
  int base = 0, before = 0, end = 0x7FFFFFFF;
};

__device__ __forceinline__ PromptTile find_tile(const PromptArgs& a, int rank, PromptFind* at) {
  const int lane = threadIdx.x & 31;
  const int unit = a.pair_heads ? kRowsTile : 2 * kRowsTile;
  PromptTile p{};
  if (rank >= at->end) return p;
  if (rank < at->before) at->base = at->before = 0;
  int before = at->before;  // units of the requests behind this one
  for (int base = at->base; base < a.num_reqs - a.num_decodes; base += 32) {
    at->base = base;
    at->before = before;
    const int r = a.num_reqs - 1 - base - lane;
    int q0 = 0, q1 = 0, sl = 0, s0 = 0;
    bool bad = false;
    if (r >= a.num_decodes) {
      q0 = a.qsl[r];
      q1 = a.qsl[r + 1];
      sl = a.seq_lens[r];
      if (a.kv_start != nullptr) s0 = a.kv_start[r];
      if (q1 < q0 || q0 < a.first_token || q1 > a.num_tokens) {
        bad = true;
        q1 = q0;  // no rows of its own to write
      }
      if (sl < 0 || sl > a.max_keys || (a.kv_start != nullptr && (s0 < 0 || s0 > a.num_blocks - sl))) {
        bad = true;
        sl = 0;
      }
      if (bad) flag_error(a.err, DSA_DEVERR_SEQ_RANGE);
    }
    const int units = (q1 - q0 + unit - 1) / unit;
    int incl = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    const int first = before + incl - units;
    const uint32_t hit = __ballot_sync(0xffffffffu, rank >= first && rank < first + units);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      const int u = units - 1 - (rank - first);
      p.req = __shfl_sync(0xffffffffu, r, src);
      p.t0 = __shfl_sync(0xffffffffu, q0 + u * unit, src);
      p.ntok = __shfl_sync(0xffffffffu, q1 - q0 - u * unit, src);
      p.pos0 = __shfl_sync(0xffffffffu, sl - (q1 - q0) + u * unit, src);
      p.keys = __shfl_sync(0xffffffffu, sl, src);
      p.kv0 = __shfl_sync(0xffffffffu, s0, src);
      p.found = true;
      return p;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  at->end = before;
  return p;
}

// Keys visible to the row at position pos.
__device__ __forceinline__ int visible(int pos, int keys) { return min(max(pos + 1, 0), keys); }

// A row's weights of one tile, packed as the A operand, and their sum: S from
// TMEM, 2^(s * scale + ref); columns from lim on are out (EDGE only). Written as
// a software pipeline, eight columns' exponentials issued ahead of the previous
// eight's sums and packing, 32 columns of S on the way while the previous ones
// are worked on: left to the compiler's order a tile took 1000 cycles and more,
// so 780 (the exponentials alone are 512).
template <typename T, bool EDGE>
__device__ __forceinline__ float weights(uint32_t ts, int lim, uint64_t sc2, uint64_t ref2, uint32_t (&p)[2][32]) {
  using E = PElem<T>;
  constexpr int G = 4;  // pairs of columns per step
  uint64_t sum[4] = {0, 0, 0, 0};
  uint32_t s[4][32];
  tmem_ld32(ts, s[0]);
  tmem_wait32(s[0]);
  tmem_ld32(ts + 32, s[1]);
  float2 w[2][G];
#pragma unroll
  for (int g = 0; g <= 64 / G; ++g) {
    if (g < 64 / G) {
      if (g % (16 / G) == 0 && g > 0 && g < 64 / G) {
        const int c = g * G / 16;
        tmem_wait32(s[c]);
        if (c < 3) tmem_ld32(ts + (c + 1) * 32, s[c + 1]);
      }
      float2 x[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int q = g * G + i;
        float a = __uint_as_float(s[q / 16][(q % 16) * 2]), b = __uint_as_float(s[q / 16][(q % 16) * 2 + 1]);
        if (EDGE) {
          a = 2 * q < lim ? a : -INFINITY;
          b = 2 * q + 1 < lim ? b : -INFINITY;
        }
        x[i] = unpack_f32x2(fma_f32x2(pack_f32x2(a, b), sc2, ref2));
      }
#pragma unroll
      for (int i = 0; i < G; ++i) w[g & 1][i] = make_float2(pex2(x[i].x), pex2(x[i].y));
    }
    if (g > 0) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int q = (g - 1) * G + i;
        const float2 e = w[(g - 1) & 1][i];
        // summed before P is rounded for the MMA: the rounding enters the numerator only
        sum[i & 3] = add_f32x2(sum[i & 3], pack_f32x2(e.x, e.y));
        p[q / 32][q % 32] = E::pack(e.x, e.y);
      }
    }
  }
  const float2 l = unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])));
  return l.x + l.y;
}

// Between lanes 2n and 2n + 1: lane 2n gets both rows' first halves, 2n + 1 their
// second ones; in: the lane's own row.
__device__ __forceinline__ void exchange2(uint32_t (&lo)[8], uint32_t (&hi)[8]) {
  const bool up = threadIdx.x & 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = __shfl_xor_sync(0xffffffffu, up ? lo[i] : hi[i], 1);
    lo[i] = up ? v : lo[i];
    hi[i] = up ? hi[i] : v;
  }
}

// 32 bytes: one store where their address allows it.
__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

// What a CTA works on: one unit of the grid, its own or a taken-over one.
struct PromptCta {
  PromptTile tile;
  // the two query tiles: head, first row of q, rows, position of the first, key tiles
  int head[2], t0[2], rows[2], pos0[2], nt[2];
  // key tiles in which a non-finite V element was cleared: lowest and highest
  int bad_lo, bad_hi;
  int stop;  // no unit: the end
};
static_assert(sizeof(PromptCta) <= 96, "room for two");

// Ask for the index of a CTA that has not started yet, which then will not
// start: *next and bar get the answer (16 bytes).
__device__ __forceinline__ void ask_next(void* next, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(next)),
      "r"(smem_u32(bar))
      : "memory");
}
// The answer: that CTA's index, or -1 when none was left.
__device__ __forceinline__ int read_next(const void* next) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "mov.s32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
      : "=r"(x)
      : "r"(smem_u32(next))
      : "memory");
  return x;
}

// Add V's elements of keys [k0, k1) to a stored row of D values, as far as they
// are not finite: what was cleared for the MMA.
template <int D, typename T>
__device__ __forceinline__ void add_non_finite(const PromptArgs& a, const PromptCta& cta, int k0, int k1, T* out) {
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    int64_t at;
    if (a.kv_start == nullptr) {
      const int id = a.block_table[static_cast<int64_t>(cta.tile.req) * a.bt_stride + k / kBlock];
      if (id < 0 || id >= a.num_blocks) continue;
      at = id * a.v_page + static_cast<int64_t>(k % kBlock) * a.v_slot;
    } else {
      at = static_cast<int64_t>(cta.tile.kv0 + k) * a.v_slot;
    }
    const T* v = static_cast<const T*>(a.v) + at + cta.head[0] / a.group * a.v_head;
#pragma unroll 1
    for (int i = 0; i < D; ++i) {
      const float x = static_cast<float>(v[i]);
      if (!isfinite(x)) out[i] = static_cast<T>(static_cast<float>(out[i]) + x);
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kPromptThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ PromptArgs a) {
  using C = PromptCfg<D>;
  using E = PElem<T>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* kv = smem + C::kOffKv;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + S;
  uint64_t* qfull = empty + S;
  uint64_t* qempty = qfull + 2;
  uint64_t* sfull = qempty + 2;          // tile x's nth scores: [x * kBufs + n % kBufs]
  uint64_t* pfull = sfull + 2 * C::kBufs;  // the weights in a buffer
  uint64_t* ofull = pfull + 3;             // its O, complete up to the nth tile (kRing) or unit: [x + 2 * (n % 2)]
  uint64_t* ufull = ofull + 4;   // a unit's PromptCta is written
  uint64_t* uempty = ufull + 2;  // and read by all
  uint64_t* asked = uempty + 2;
  uint64_t* done = asked + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  uint8_t* next = smem + C::kOffNext;
  PromptCta* ctas = reinterpret_cast<PromptCta*>(smem + C::kOffCta);  // two, taking turns

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // both tiles' softmax warps, whether they use the stage or not
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&qfull[x], 1);
      mbar_init(&qempty[x], 1);
      for (int b = 0; b < C::kBufs; ++b) mbar_init(&sfull[x * C::kBufs + b], 1);
      mbar_init(&ofull[x], 1);
      mbar_init(&ofull[x + 2], 1);
      mbar_init(&ufull[x], 1);
      mbar_init(&uempty[x], kSoftWarps + 1);
    }
    for (int b = 0; b < 3; ++b) mbar_init(&pfull[b], kSoftWarps / 2);
    mbar_init(asked, 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // launched while the stream's previous kernel drains: nothing is read or written before it has ended

  // The next unit for a warp that follows the TMA warp, or false at the end.
  int units = 0;
  auto next_unit = [&](const volatile PromptCta** w) {
    const int u = units & 1;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&ufull[u], (units >> 1) & 1, abort_flag, a.err)) != 0;
    *w = &ctas[u];
    ++units;
    return ok && !(*w)->stop;
  };
  auto unit_read = [&]() {  // of the unit that next_unit gave last
    __syncwarp();
    if (lane == 0) mbar_arrive(&uempty[(units - 1) & 1]);
  };

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
    if (warp == kTmaWarp) {
      // --------------------------------------------------------------- TMA
      int seq = 0;       // ring stages filled so far
      int nq[2] = {0, 0};  // units that loaded query tile x
      int item = blockIdx.x;
      int asks = 0;  // answers read
      PromptFind found_at;
      bool ok = true, pending = false;
      while (ok) {
        const int u = units & 1;
        if (units >= 2)
          ok = __all_sync(0xffffffffu, mbar_wait(&uempty[u], ((units >> 1) - 1) & 1, abort_flag, a.err)) != 0;
        if (!ok) break;
        PromptCta& c = ctas[u];
        const int hu = item < 0 ? 0 : item % a.head_units;
        PromptTile tile{};
        if (item >= 0) tile = find_tile(a, item / a.head_units, &found_at);
        const bool none = item >= 0 && !tile.found;  // the grid is an upper bound
        if (none) {  // pass over it
          if (lane == 0) {
            mbar_arrive_expect_tx(asked, 16);
            ask_next(next, asked);
          }
          pending = true;
        }
        int nt[2] = {0, 0};
        if (tile.found) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int shift = a.pair_heads ? 0 : x * kRowsTile;
            const int rows = min(kRowsTile, max(0, tile.ntok - shift));
            nt[x] = rows > 0 ? (visible(tile.pos0 + shift + rows - 1, tile.keys) + kKeys - 1) / kKeys : 0;
            if (lane == 0) {
              c.head[x] = a.pair_heads ? 2 * hu + x : hu;
              c.t0[x] = tile.t0 + shift;
              c.rows[x] = rows;
              c.pos0[x] = tile.pos0 + shift;
              c.nt[x] = nt[x];
            }
          }
        }
        if (!none) {
          if (lane == 0) {
            c.tile = tile;
            c.bad_lo = 0x7FFFFFFF;
            c.bad_hi = -1;
            c.stop = item < 0;
            mbar_arrive(&ufull[u]);
            if (item >= 0) {
              mbar_arrive_expect_tx(asked, 16);
              ask_next(next, asked);
            }
          }
          pending = item >= 0;
          ++units;
          if (item < 0) break;
          const int n_tiles = max(nt[0], nt[1]);
          const int h = (a.pair_heads ? 2 * hu : hu) / a.group;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (nt[x] == 0 || !ok) continue;
            if (nq[x] > 0)
              ok = __all_sync(0xffffffffu, mbar_wait(&qempty[x], (nq[x] - 1) & 1, abort_flag, a.err)) != 0;
            ++nq[x];
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(&qfull[x], C::kTileBytes);
#pragma unroll
              for (int b = 0; b < D / 64; ++b)
                tma_load_3d(smem + x * C::kTileBytes + b * C::kColBytes, &tmap_q, &qfull[x], b * 64,
                            a.pair_heads ? 2 * hu + x : hu, tile.t0 + (a.pair_heads ? 0 : x * kRowsTile));
            }
          }
          const int n_pages = (tile.keys + kBlock - 1) / kBlock;
          int32_t ids = 0;
          for (int j = 0; j < n_tiles && ok; ++j) {
            int c2[2], c3[2], boxes;
            if (a.kv_start == nullptr) {
              if ((j & 15) == 0) {  // the next 32 pages
                const int pg = 2 * j + lane;
                ids = pg < n_pages ? a.block_table[static_cast<int64_t>(tile.req) * a.bt_stride + pg] : 0;
                if (ids < 0 || ids >= a.num_blocks) {
                  flag_error(a.err, DSA_DEVERR_BLOCK_RANGE);
                  ids = 0;
                }
              }
              c3[0] = __shfl_sync(0xffffffffu, ids, 2 * (j & 15));
              c3[1] = __shfl_sync(0xffffffffu, ids, 2 * (j & 15) + 1);
              c2[0] = c2[1] = 0;
              boxes = 2 * j + 1 < n_pages ? 2 : 1;
            } else {
              c2[0] = tile.kv0 + j * kKeys;
              c2[1] = c2[0] + kBlock;
              c3[0] = c3[1] = 0;
              // a box may begin behind the last packed row only if it is not loaded at all
              boxes = j * kKeys + kBlock < tile.keys ? 2 : 1;
            }
            if (lane == 0) {
#pragma unroll
              for (int kvi = 0; kvi < 2; ++kvi) {
                const int st = seq % S, round = seq / S;
                if (round > 0 && !mbar_wait(&empty[st], (round - 1) & 1, abort_flag, a.err)) {
                  ok = false;
                  break;
                }
                uint8_t* dst = kv + st * C::kTileBytes;
                mbar_arrive_expect_tx(&full[st], boxes * C::kBoxBytes * (D / 64));
                for (int b = 0; b < boxes; ++b)
#pragma unroll
                  for (int k = 0; k < D / 64; ++k)
                    tma_load_4d(dst + k * C::kColBytes + b * C::kBoxBytes, kvi == 0 ? &tmap_k : &tmap_v, &full[st],
                                k * 64, h, c2[b], c3[b]);
                ++seq;
              }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
          }
        }
        // the unit after this one
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(asked, asks & 1, abort_flag, a.err)) != 0;
        if (ok) {
          ++asks;
          pending = false;
          item = read_next(next);
          fence_proxy_async();  // read before the next answer is written
          __syncwarp();
        }
      }
      if (lane == 0 && *abort_flag) {  // giving up: no copy may land after the CTA's end
        const unsigned long long until = global_ns() + kWaitLimitNs;
        if (pending)
          while (!mbar_try_wait(smem_u32(asked), asks & 1) && global_ns() < until) {
          }
        for (int i = max(0, seq - S); i < seq; ++i)
          while (!mbar_try_wait(smem_u32(&full[i % S]), (i / S) & 1) && global_ns() < until) {
          }
        for (int x = 0; x < 2; ++x)
          if (nq[x] > 0)
            while (!mbar_try_wait(smem_u32(&qfull[x]), (nq[x] - 1) & 1) && global_ns() < until) {
            }
      }
    } else if (warp == kMmaWarp) {
      // --------------------------------------------------------------- MMA
      // The warp waits as one and an elected thread issues: with one lane alone
      // in the loop each MMA took about 115 cycles to issue, whatever its size.
      // One warp for both tiles keeps them out of step, one's softmax under the
      // other's MMAs: with a warp per tile they fell into step (1350 -> 1230
      // TFLOP/s at 4 x 8192, 64/8 heads of 128).
      {
        constexpr uint32_t kIdS = f16_idesc(E::kFmt, kKeys, false), kIdO = f16_idesc(E::kFmt, D, true);
        const uint32_t qd = kmajor_lo(smem_u32(smem)), kv0 = smem_u32(kv);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err)) != 0;
        };
        int seq = 0, nq[2] = {0, 0}, np[2] = {0, 0};  // ring stages, units and tiles so far
        int on[2] = {0, 0};  // which of the two ofull the tile completes next
        // ring stages and parities of the next K and V; kRing: buffers of the next S
        // and P, and which of its sfull a tile completes next
        int kst = 0, vst = 1, sbuf = 0, pbuf = 0, sn[2] = {0, 0};
        uint32_t kpar = 0, vpar = 0, ppar = 0;
        auto scores = [&](int x, int st, int buf, uint64_t* bar) {
          const uint32_t kd = kmajor_lo(kv0 + st * C::kTileBytes), qx = qd + ((x * C::kTileBytes) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k / 4) * C::kColBytes + (k % 4) * 32) >> 4;
              mma_f16_ss(tmem + buf * kKeys, qx + off, kd + off, kIdS, k > 0);
            }
            mma_commit(bar);
          }
          __syncwarp();
        };
        auto values = [&](int x, int st, int buf, bool acc) {
          const uint32_t vd = mnmajor_lo(kv0 + st * C::kTileBytes);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_f16_ts(tmem + C::kO + x * D, tmem + buf * kKeys + k * 8, vd + ((k * 16 * 128) >> 4), kIdO,
                         acc || k > 0);
            if constexpr (C::kRing) mma_commit(&ofull[x + 2 * on[x]]);  // elsewhere a unit's last alone
          }
          __syncwarp();
        };
        auto release = [&](uint64_t* bar) {
          if (elect_one()) mma_commit(bar);
          __syncwarp();
        };
        bool ok = true;
        const volatile PromptCta* w;
        while (ok && next_unit(&w)) {
          const int nt[2] = {w->nt[0], w->nt[1]};
          unit_read();
          const int n_tiles = max(nt[0], nt[1]);
          if (n_tiles == 0) continue;
          if constexpr (C::kRing) {
            // Steps (tile x, key tile j) in turn, each: P V, then Q K^T of the third
            // step after it, into the buffer just read. Stages and parities are kept
            // as running values, and a step's MMAs issued in one piece: this warp's
            // instructions are between a step's weights and the scores that follow
            // (8 x 2048, 32/8 heads: 172 us with two pieces, so 166; 188 with every
            // step by next_scores).
            auto bump = [&](int& st, uint32_t& par) {
              st += 2;
              if (st >= S) st -= S, par ^= 1;
            };
            auto step_scores = [&](int x) {  // of tile x, K in stage kst, S to buffer sbuf
              scores(x, kst, sbuf, &sfull[x * 3 + sn[x]]);
              sn[x] = sn[x] == 2 ? 0 : sn[x] + 1;
              sbuf = sbuf == 2 ? 0 : sbuf + 1;
            };
            auto step_values = [&](int x, int j) {  // of tile x, V in stage vst, P in buffer pbuf
              ok = wait(&pfull[pbuf], ppar);
              if (!ok) return;
              tc_fence_after();
              values(x, vst, pbuf, j > 0);
              on[x] ^= 1;
              if (++pbuf == 3) pbuf = 0, ppar ^= 1;
            };
            auto step_both = [&](int x, int j) {  // values of (x, j), then scores of the other tile
              const int y = x ^ 1;
              ok = ok && wait(&pfull[pbuf], ppar);
              if (!ok) return;
              tc_fence_after();
              const uint32_t vd = mnmajor_lo(kv0 + vst * C::kTileBytes), kd = kmajor_lo(kv0 + kst * C::kTileBytes);
              const uint32_t sp = tmem + pbuf * kKeys, qy = qd + ((y * C::kTileBytes) >> 4);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  mma_f16_ts(tmem + C::kO + x * D, sp + k * 8, vd + ((k * 16 * 128) >> 4), kIdO, j > 0 || k > 0);
                mma_commit(&ofull[x + 2 * on[x]]);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint32_t off = ((k / 4) * C::kColBytes + (k % 4) * 32) >> 4;
                  mma_f16_ss(sp, qy + off, kd + off, kIdS, k > 0);
                }
                mma_commit(&sfull[y * 3 + sn[y]]);
              }
              __syncwarp();
              on[x] ^= 1;
              sn[y] = sn[y] == 2 ? 0 : sn[y] + 1;
              if (++pbuf == 3) pbuf = 0, ppar ^= 1;
              sbuf = pbuf;
            };
            int qj = 0, j = 0;  // key tiles of the next scores and P V
            bool q1 = false;    // the next scores are tile 1's
            auto next_scores = [&]() {  // wherever they are
              if (qj >= n_tiles || !ok) return;
              if (!q1 && qj >= nt[0]) q1 = true;
              if (q1 && qj >= nt[1]) {
                q1 = qj + 1 >= nt[0];
                ++qj;
                bump(kst, kpar);
              }
              if (qj >= n_tiles) return;
              const int x = q1;
              if (qj == 0) ok = wait(&qfull[x], x == 0 ? nq[0]++ & 1 : nq[1]++ & 1);
              ok = ok && wait(&full[kst], kpar);
              if (!ok) return;
              if (x == 0)
                step_scores(0);
              else
                step_scores(1);
              if (qj + 1 == (x == 0 ? nt[0] : nt[1])) release(&qempty[x]);  // the unit's last use of this query tile
              if (q1) {
                ++qj;
                bump(kst, kpar);
              }
              q1 = !q1;
            };
            for (int i = 0; i < 3; ++i) next_scores();
            while (j < n_tiles && ok) {
              ok = wait(&full[vst], vpar);
              if (j + 2 < nt[0] && j + 1 < nt[1]) {  // both tiles go on: scores of (1, j + 1) and (0, j + 2)
                step_both(0, j);
                if (j + 2 == nt[1]) release(&qempty[1]);
                bump(kst, kpar);
                ok = ok && wait(&full[kst], kpar);
                step_both(1, j);
                if (j + 3 == nt[0]) release(&qempty[0]);
                ++qj;
              } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  if (j >= nt[x] || !ok) continue;
                  step_values(x, j);
                  next_scores();
                }
              }
              ++j;
              bump(vst, vpar);
            }
            // kst has passed, or passes, the unit's last K
            for (; qj < n_tiles; ++qj) bump(kst, kpar);
          } else {
            ok = wait(&full[seq % S], (seq / S) & 1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (nt[x] == 0 || !ok) continue;
              ok = wait(&qfull[x], nq[x]++ & 1);
              if (ok) scores(x, seq % S, x, &sfull[x]);
              if (nt[x] == 1) release(&qempty[x]);
            }
            vst = (seq + 1) % S, kst = (seq + 2) % S;
            vpar = ((seq + 1) / S) & 1, kpar = ((seq + 2) / S) & 1;
            ok = ok && wait(&full[vst], vpar);
            for (int j = 0; j < n_tiles && ok; ++j) {
              bool have_k = false;
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                if (j >= nt[x]) continue;
                ok = ok && wait(&pfull[x], np[x]++ & 1);
                if (!ok) break;
                tc_fence_after();
                values(x, vst, x, j > 0);
                if (j == nt[x] - 1) {
                  release(&ofull[x + 2 * on[x]]);
                  on[x] ^= 1;
                }
                if (j + 1 >= nt[x]) continue;
                if (!have_k) ok = wait(&full[kst], kpar);
                have_k = true;
                if (ok) scores(x, kst, x, &sfull[x]);
                if (j + 2 == nt[x]) release(&qempty[x]);  // the unit's last use of this query tile
              }
              for (int i = 0; i < 2; ++i) {
                if (++vst == S) vst = 0, vpar ^= 1;
                if (++kst == S) kst = 0, kpar ^= 1;
              }
              if (ok && j + 1 < n_tiles) ok = wait(&full[vst], vpar);
            }
          }
          seq += 2 * n_tiles;
        }
        if (*abort_flag) {  // giving up: let the MMAs in flight end before TMEM is freed
          if (elect_one()) mma_commit(done);
          __syncwarp();
          const unsigned long long until = global_ns() + kWaitLimitNs;
          while (!mbar_try_wait(smem_u32(done), 0) && global_ns() < until) {
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    // ------------------------------------------------------------- softmax
    // A row per thread, the row's TMEM lane in the quarter that its warp may read.
    const int x = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + C::kO + x * D;
    const float NEG = -INFINITY;
    const bool leader = (warp & 3) == 0 && lane == 0;
    bool ok = true;
    int seq = 0;  // ring stages so far
    int ns = 0;         // tiles so far
    int base = 0, no = 0;  // kRing: both tiles' tiles in the units before; rounds of ofull waited for
    const volatile PromptCta* wp;
    while (ok && next_unit(&wp)) {
      const volatile PromptCta& w = *wp;
      PromptCta& cta = ctas[(units - 1) & 1];
      const int my_nt = w.nt[x], other_nt = w.nt[x ^ 1];
      const int vis = visible(w.pos0[x] + min(r, w.rows[x] - 1), w.tile.keys);
      float M = NEG, L = 0.0f;
      bool fresh = true;  // some row of the warp may have no reference yet
      // uniform bounds of what only some tiles need: the first tile that a row of
      // the warp, and of the tile, does not see whole
      const int edge_from = __reduce_min_sync(0xffffffffu, vis) / kKeys;
      const int fix_from = x == 0 ? visible(w.pos0[0], w.tile.keys) / kKeys
                                  : max(visible(w.pos0[1], w.tile.keys) / kKeys, other_nt);
      int kst = seq % S, vst = (seq + 1) % S;  // ring stages of tile j
      uint32_t vpar = ((seq + 1) / S) & 1;
      // O complete up to the unit's tile j, or (not kRing, j = 0) its last
      const int first_o = C::kRing ? ns : no;
      auto wait_o = [&](int j) {
        bool k = true;
        for (; k && no <= first_o + j; ++no)
          k = __all_sync(0xffffffffu, mbar_wait(&ofull[x + 2 * (no & 1)], (no >> 1) & 1, abort_flag, a.err)) != 0;
        tc_fence_after();
        return k;
      };
      // V in a tile cut by the causal edge or the sequence's end, before its first
      // use: D = 128 while the tile's scores are on the way (8 x 2048, 32/8 heads:
      // 233 -> 228 us); D = 64, whose scores are there by then, behind the weights
      // (2 x 8192, 32/8 heads: 536 us, in front 562)
      auto clear_v = [&](int j) {
        if (j < fix_from) return true;
        ok = __all_sync(0xffffffffu, mbar_wait(&full[vst], vpar, abort_flag, a.err)) != 0;
        if (!ok) return false;
        // thread r: key row r of the tile, which lies at 128-byte row r of each
        // 64-column block; its 16-byte pieces in another order in each lane, so
        // that the lanes' banks differ
        uint8_t* v = kv + vst * C::kTileBytes + r * 128;
        bool bad = false;
        if (j * kKeys + r >= w.tile.keys) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint4*>(v + (i / 8) * C::kColBytes + ((i ^ r) % 8) * 16) = make_uint4(0, 0, 0, 0);
        } else {
          // an exponent of all ones, plus its last bit's weight, carries into the sign's place
          constexpr uint32_t kOnes = E::kExp * 0x10001u, kOne = (E::kExp & (0u - E::kExp)) * 0x10001u;
          uint32_t hit = 0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(v + (i / 8) * C::kColBytes + ((i ^ r) % 8) * 16);
            hit |= ((u.x & kOnes) + kOne) | ((u.y & kOnes) + kOne) | ((u.z & kOnes) + kOne) | ((u.w & kOnes) + kOne);
          }
          bad = hit & 0x80008000u;
          if (bad) {
            for (int i = 0; i < D / 2; ++i) {
              uint32_t* at = reinterpret_cast<uint32_t*>(v + (i / 32) * C::kColBytes + (i % 32) * 4);
              const uint32_t e = (*at & kOnes) + kOne;
              *at &= ((e & 0x8000u) ? 0u : 0xFFFFu) | ((e & 0x80000000u) ? 0u : 0xFFFF0000u);
            }
          }
        }
        if (bad) {
          atomicMin(&cta.bad_lo, j);
          atomicMax(&cta.bad_hi, j);
        }
        fence_proxy_async();
        return true;
      };
      for (int j = 0; j < my_nt; ++j, ++ns) {
        // its step's buffer: the steps before it are the tiles before it, and the other tile's
        const int buf = C::kRing ? (base + j + min(j + x, other_nt)) % 3 : x;
        const uint32_t ts = tmem + lanes + buf * kKeys;
        if constexpr (!C::kRing) {  // while its scores are on the way
          if (!clear_v(j)) break;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&sfull[x * C::kBufs + ns % C::kBufs], (ns / C::kBufs) & 1, abort_flag,
                                               a.err)) != 0;
        if (!ok) break;
        tc_fence_after();
        if (leader) {  // the scores are complete, and with one buffer all that this tile's MMAs read before
          mbar_arrive(&empty[kst]);
          if (!C::kRing && j > 0) mbar_arrive(&empty[kst == 0 ? S - 1 : kst - 1]);
        }
        const int lim = vis - j * kKeys;  // visible columns
        // The weights by the reference at hand, without looking for the maximum
        // first: only where a row has none yet, or its weights come out too large
        // (or not a number), the tile's is taken and the weights once more. A
        // row's decision is its own: no other row has a part in its bits. The way
        // of most tiles is short and in one piece, the rest out of its way: with
        // all in one loop, 2 x 8192, 32/8 heads took 652 us (D = 128) and 538
        // (D = 64), so 638 and 508.
        if (__builtin_expect(fresh, 0)) {  // a first reference: the maximum of the columns in front
          uint32_t s[32];
          tmem_ld32(ts, s);
          tmem_wait32(s);
          float mx[4];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float v = i < lim ? __uint_as_float(s[i]) : NEG;
            mx[i & 3] = i < 4 ? v : fmaxf(mx[i & 3], v);
          }
          // (no weight was above 0 so far: nothing to rescale)
          if (M == NEG) M = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2 - E::kHead;
          fresh = __any_sync(0xffffffffu, M == NEG);
        }
        uint32_t p[2][32];
        float add;
        const bool whole = j < edge_from && !fresh;
        bool done = false;
        if (__builtin_expect(whole, 1)) {
          add = weights<T, false>(ts, lim, pack_f32x2(a.scale_log2, a.scale_log2), pack_f32x2(-M, -M), p);
          done = __all_sync(0xffffffffu, add <= E::kMaxSum);
        }
        if (__builtin_expect(!done, 0)) {
          bool raise = whole ? !(add <= E::kMaxSum) : M == NEG && lim > 0;
          for (int attempt = __any_sync(0xffffffffu, raise) ? 1 : 0;; ++attempt) {
            if (attempt > 0) {
              float top = NEG;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t s[32];
                tmem_ld32(ts + c * 32, s);
                tmem_wait32(s);
                const int end = lim - c * 32;
                float mx[4];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float v = i < end ? __uint_as_float(s[i]) : NEG;
                  mx[i & 3] = i < 4 ? v : fmaxf(mx[i & 3], v);
                }
                top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
              }
              const float n = raise ? fmaxf(M, top * a.scale_log2 - E::kHead) : M;
              const float f = !raise ? 1.0f : M == NEG ? 0.0f : pex2(M - n);
              M = n;
              L *= f;
              fresh = __any_sync(0xffffffffu, M == NEG);
              if (j > 0) {
                if (C::kRing && !wait_o(j - 1)) {  // (with one buffer, its MMAs precede this tile's scores)
                  ok = false;
                  break;
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t o[32];
                  tmem_ld32(to + c * 32, o);
                  tmem_wait32(o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st32(to + c * 32, o);
                }
              }
            }
            const float ref = M == NEG ? 0.0f : M;
            const uint64_t sc2 = pack_f32x2(a.scale_log2, a.scale_log2), ref2 = pack_f32x2(-ref, -ref);
            add = weights<T, true>(ts, lim, sc2, ref2, p);
            raise = !raise && !(add <= E::kMaxSum);
            if (attempt == 2 || !__any_sync(0xffffffffu, raise)) break;
          }
          if (!ok) break;
        }
        L += add;
        if (C::kRing && j > 1) {  // P V of the tile before the previous one: V was read (mostly long ago)
          ok = wait_o(j - 2);
          if (leader) mbar_arrive(&empty[kst < 3 ? kst + S - 3 : kst - 3]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) tmem_st32(ts + half * 32, p[half]);
        if constexpr (C::kRing) {
          if (!clear_v(j)) break;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[buf]);
        kst += 2;
        if (kst >= S) kst -= S;
        vst += 2;
        if (vst >= S) vst -= S, vpar ^= 1;
      }
      // ---- the row's result
      if (ok && my_nt > 0) {
        ok = wait_o(C::kRing ? my_nt - 1 : 0);
      }
      base += my_nt + other_nt;
      if (leader && ok) {  // the last V's, then the stages that only the other tile reads
        for (int i = C::kRing ? 2 : 1; i > 0; --i)
          if (my_nt >= i) mbar_arrive(&empty[(seq + 2 * (my_nt - i) + 1) % S]);
        for (int i = seq + 2 * my_nt; i < seq + 2 * other_nt && ok; ++i) {
          ok = mbar_wait(&full[i % S], (i / S) & 1, abort_flag, a.err);
          mbar_arrive(&empty[i % S]);
        }
      }
      seq += 2 * max(my_nt, other_nt);
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (ok) {
        tc_fence_after();
        const int my_head = w.head[x], my_t0 = w.t0[x];
        const int my_rows = w.rows[x];
        // (no score but NaN leaves M alone, and a sum of NaN)
        const bool mine = r < my_rows, any = M != NEG || L != 0.0f;
        const float inv = any ? 1.0f / L : 0.0f;
        const int blo = my_nt > 0 ? w.bad_lo : 0x7FFFFFFF, bhi = my_nt > 0 ? w.bad_hi : -1;
        // after the exchange below this lane stores 32 bytes of rows r / 2 * 2 and the
        // next (16 bytes of four rows, by two exchanges: 512 prompts of 128 took 152
        // us, so 146)
        T* out = static_cast<T*>(a.out) + static_cast<int64_t>(my_t0 + (r & ~1)) * a.out_row + my_head * a.out_head +
                 (lane & 1) * 16;
        const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | a.out_row * 2 | a.out_head * 2) & 31) == 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c, out += 32) {
          uint32_t o[32];
          if (my_nt > 0) {
            tmem_ld32(to + c * 32, o);
            tmem_wait32(o);
          }
          uint32_t u[2][8];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            u[i / 8][i % 8] = any ? E::pack(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0u;
          exchange2(u[0], u[1]);
          if ((r & ~1) < my_rows) store32(out, u[0], wide);
          if ((r | 1) < my_rows) store32(out + a.out_row, u[1], wide);
        }
        if (blo <= bhi) {
          __syncwarp();  // the row was stored by two lanes
          if (mine && any)
            add_non_finite<D, T>(a, cta, blo * kKeys, min(vis, (bhi + 1) * kKeys),
                                 static_cast<T*>(a.out) + static_cast<int64_t>(my_t0 + r) * a.out_row +
                                     my_head * a.out_head);
        }
        if (mine && a.lse != nullptr)
          a.lse[static_cast<int64_t>(my_t0 + r) * a.heads + my_head] = any ? (M + log2f(L)) * 0.6931471805599453f : NEG;
      }
      unit_read();
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, typename T>
cudaError_t launch(const PromptArgs& a, const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv,
                   cudaStream_t stream) {
  static uint64_t done = 0;
  auto* fn = attn_prompt_kernel<D, T>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(fn), PromptCfg<D>::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, dim3(a.head_units * a.tile_units), dim3(kPromptThreads), PromptCfg<D>::kSmemBytes, stream, *mq,
                    *mk, *mv, a);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                               const CUtensorMap* mv, int head_dim, int dtype, cudaStream_t stream) {
  if (dtype == DSA_BF16)
    return head_dim == 128 ? launch<128, __nv_bfloat16>(a, mq, mk, mv, stream)
                           : launch<64, __nv_bfloat16>(a, mq, mk, mv, stream);
  return head_dim == 128 ? launch<128, __half>(a, mq, mk, mv, stream) : launch<64, __half>(a, mq, mk, mv, stream);
}

}  // namespace dsa
