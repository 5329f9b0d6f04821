// kv8.cu — the paged KV cache in 8 bits (sm_103a): rows quantised as they are
// written, and sequences' rows read back in 16 bits.
//
// A block is 16 slots of a page and one KV head, K and V apart; its scale is a power
// of two 2^e, a row's values are codes * 2^e. For the rows that a call writes into a
// block, with amax their largest finite magnitude,
//   need = the least 2^e, e >= -64, with amax / 2^e <= 448 (E4M3's largest code),
//   scale = need if the block's first slot is written, else max(need, old scale),
//   code = RN(x / scale), and RN(code * old / scale) for the block's other slots
//   where the scale rises.
// Powers of two make x / scale exact, so each value is rounded once, and a code that
// moves to a higher scale is rounded again only where it falls below 2^-6. A scale of
// another kind that a block brings along stays while it suffices: its quotients and
// products come in 32 bits in a way that leaves the rounding to a code right
// (odd), as those that are read back are. All of it depends on the call's rows and the block alone, not on the order of
// the list or of the threads.
//
// What bounds both: HBM, 4*D bytes of rows and 2*D of codes a (token, head). 8 heads of
// 128: 30572 rows of 8 requests written in 35 us (5.4 TB/s; the claims are a launch of
// their own), 113K rows of 8 requests of up to 16K read back in 107 us (6.6 TB/s, two
// thirds of it writes). 64 rows written, or 301 read back, take 8 us, the host's
// time for the call, of which the GPU's is 3 to 4.
#include "attn.h"
#include "common.cuh"

namespace dsa {

namespace {

constexpr int kScaleBlock = DSA_SCALE_BLOCK;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The least power of two 2^e, e >= -64, with amax <= 448 * 2^e: amax = m*2^E (1 <= m
// < 2) and 448 = 1.75*2^8, so e = E - 8, plus one when m > 1.75.
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t u = __float_as_uint(fmaxf(amax, 0x1p-64f));
  return fmaxf(__uint_as_float(((u >> 23) - 8u + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u)) << 23), 0x1p-64f);
}

// Two 16-bit values as fp32.
__device__ __forceinline__ float2 wide(uint32_t x, __nv_bfloat16) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
__device__ __forceinline__ float2 wide(uint32_t x, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ uint32_t narrow(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t narrow(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Bits of the type's infinity: magnitudes at or above it are not finite.
__device__ __forceinline__ uint32_t inf_bits(__nv_bfloat16) { return 0x7F80u; }
__device__ __forceinline__ uint32_t inf_bits(__half) { return 0x7C00u; }

// Four codes as fp32.
__device__ __forceinline__ void values(uint32_t codes, float2* lo, float2* hi) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(codes));
  *lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
  *hi = __half22float2(*reinterpret_cast<const __half2*>(&b));
}
// Eight codes' values in the type.
template <typename T>
__device__ __forceinline__ uint4 row_of(uint2 codes, float s, T type) {
  float2 f[4];
  values(codes.x, &f[0], &f[1]);
  values(codes.y, &f[2], &f[3]);
  return make_uint4(narrow(f[0].x * s, f[0].y * s, type), narrow(f[1].x * s, f[1].y * s, type),
                    narrow(f[2].x * s, f[2].y * s, type), narrow(f[3].x * s, f[3].y * s, type));
}
__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float f) {
  float2 lo, hi;
  values(codes, &lo, &hi);
  return e4m3x4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7FFFFFu) == 0; }

// A number q that stands for q + r, for a rounding to fewer bits: where r is not 0 its last
// bit is set, towards r, so that it lies on the side of every halfway point that q + r lies
// on. (Rounding to odd, after which a second rounding gives what one would: Boldo and Melquiond.)
__device__ __forceinline__ float odd(float q, float r) {
  uint32_t u = __float_as_uint(q);
  if (r != 0.0f && !(u & 1u)) u += (__float_as_uint(r) ^ u) >> 31 ? 0xffffffffu : 1u;
  return __uint_as_float(u);
}
__device__ __forceinline__ float product(float a, float b) { return odd(a * b, fmaf(a, b, -(a * b))); }
// x / s as a number that rounds to the same code: x * inv rounded to five bits (Veltkamp's
// splitting), among which are all codes and all points halfway between them, and moved to the
// side of it that x / s lies on, which x - five * s tells without a rounding of its sign.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv, c = __fmul_rn(q, 524289.0f), five = __fsub_rn(c, __fsub_rn(c, q));
  return odd(five, fmaf(-five, s, x));
}

// ---------------------------------------------------------------------- write
// Who writes a block: the call's tokens of a block are found by its slots, whatever
// their places in the list. With few tokens each CTA looks the list through; with many
// a first kernel leaves each slot's last token in token_of, which needs no clearing:
// an entry counts only if it names a token whose slot this is. Either way the token
// at the block's lowest written slot takes the whole block.
__global__ void __launch_bounds__(kThreads) write8_claim_kernel(const __grid_constant__ Write8Args a) {
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (t >= a.n_tokens) return;
  const int64_t slot = a.slot_mapping[t], slots = a.c.num_blocks * kBlock;
  if (slot < 0 || slot >= slots) return;
  int32_t* at = a.token_of + slot;
  int32_t seen = *reinterpret_cast<volatile int32_t*>(at);
  while (true) {
    // an entry of this call that is later in the list stands; each exchange that fails meets another token's
    if (seen >= static_cast<int32_t>(t) && seen < a.n_tokens && a.slot_mapping[seen] == slot) return;
    const int32_t was = atomicCAS(at, seen, static_cast<int32_t>(t));
    if (was == seen) return;
    seen = was;
  }
}

// The codes of a block whose scale was no power of two, which this file does not make: the
// rows at `rows` over the scale s, and the codes that are there moved from `old` to it. A
// function of its own, a value at a time: as a branch of write_block it costs the rows that
// never take it 13% (30572 rows: 39.3 us, so 34.9).
template <int D, typename T>
__device__ __noinline__ void write_odd(const uint16_t* rows, int64_t row, uint8_t* codes, int64_t slot,
                                       const int32_t* src, float s, float old) {
  const float inv = 1.0f / s, f = old * inv;  // where s is above old it is a power of two, and f exact
  const uint32_t inf = inf_bits(T());
#pragma unroll 1
  for (int i = 2 * (threadIdx.x & 31); i < kScaleBlock * D; i += 64) {
    const int r = i / D, c = i % D, t = src[r];
    uint16_t* at = reinterpret_cast<uint16_t*>(codes + r * slot + c);
    float2 lo, hi;
    if (t >= 0) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(rows + t * row + c);
      lo = wide(w, T());
      lo.x = (w & 0x7FFFu) < inf ? quotient(lo.x, s, inv) : NAN;
      lo.y = (w >> 16 & 0x7FFFu) < inf ? quotient(lo.y, s, inv) : NAN;
    } else {
      if (!(s > old)) continue;
      values(*at, &lo, &hi);
      lo = make_float2(product(lo.x, f), product(lo.y, f));
    }
    *at = static_cast<uint16_t>(e4m3x4(lo.x, lo.y, 0.0f, 0.0f));
  }
}

// A warp: the rows of one block and head, K or V; src[r] = the token of slot r, or -1.
template <int D, typename T>
__device__ __forceinline__ void write_block(const Write8Args& a, int64_t block, const int32_t* src, int h, bool isv) {
  constexpr int CH = D / 8;                  // 16-byte chunks of a new row
  constexpr int RPI = 32 / CH;               // rows per load of the warp
  constexpr int N = kScaleBlock / RPI;       // loads
  const int lane = threadIdx.x & 31, ch = lane % CH, r0 = lane / CH;
  const uint16_t* rows = (isv ? a.v : a.k) + h * (isv ? a.v_rhead : a.k_rhead);
  const int64_t row = isv ? a.v_row : a.k_row;
  const int64_t page = block / (kBlock / kScaleBlock), part = block % (kBlock / kScaleBlock);
  const int64_t slot = isv ? a.c.v_slot : a.c.k_slot;
  uint8_t* codes = (isv ? a.c.v + page * a.c.v_page + h * a.c.v_head : a.c.k + page * a.c.k_page + h * a.c.k_head) +
                   part * kScaleBlock * slot;
  float* scale = a.c.scale + page * a.c.s_page + part * a.c.s_block + h * a.c.s_head + (isv ? 1 : 0);

  uint4 x[N];
  bool in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int32_t t = src[i * RPI + r0];
    in[i] = t >= 0;
    x[i] = in[i] ? *reinterpret_cast<const uint4*>(rows + t * row + ch * 8) : make_uint4(0, 0, 0, 0);
  }
  const bool opened = src[0] >= 0;
  float old = opened ? 0.0f : *scale;
  if (!(old > 0.0f && old < INFINITY)) old = 0.0f;  // nothing was written here
  // the largest magnitude, by its bits; values that are not finite do not count
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (uint32_t w : {x[i].x, x[i].y, x[i].z, x[i].w}) most = __vmaxu2(most, w & 0x7FFF7FFFu);
  const uint32_t inf = inf_bits(T());
  const bool finite = !__any_sync(0xffffffffu, (most & 0xFFFFu) >= inf || (most >> 16) >= inf);
  if (!finite) {
    most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (uint32_t w : {x[i].x, x[i].y, x[i].z, x[i].w}) {
        const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
        most = __vmaxu2(most, (lo < inf ? lo : 0u) | (hi < inf ? hi << 16 : 0u));
      }
  }
  most = max(most & 0xFFFFu, most >> 16);
  most = __reduce_max_sync(0xffffffffu, most);
  const float s = fmaxf(scale_of(wide(most, T()).x), old);
  const float inv = 1.0f / s;
  if (!power_of_two(old)) {
    write_odd<D, T>(rows, row, codes, slot, src, s, old);
    __syncwarp();  // as below
    if (lane == 0) *scale = s;
    return;
  }
  if (old > 0.0f && s > old) {
    // the rows that are there move to the higher scale
    const float f = old * inv;
    constexpr int CC = D / 16, RC = 32 / CC;
    const int cc = lane % CC, q0 = lane / CC;
#pragma unroll
    for (int i = 0; i < kScaleBlock / RC; ++i) {
      const int r = i * RC + q0;
      if (src[r] >= 0) continue;
      uint4* at = reinterpret_cast<uint4*>(codes + r * slot + cc * 16);
      uint4 v = *at;
      v = make_uint4(rescaled(v.x, f), rescaled(v.y, f), rescaled(v.z, f), rescaled(v.w, f));
      *at = v;
    }
  }
  uint8_t* at = codes + r0 * slot + ch * 8;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!in[i]) continue;
    float2 f[4] = {wide(x[i].x, T()), wide(x[i].y, T()), wide(x[i].z, T()), wide(x[i].w, T())};
    if (!finite) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // x - x: 0, or NaN for what is not finite, which has NaN as its code
        f[k].x += f[k].x - f[k].x;
        f[k].y += f[k].y - f[k].y;
      }
    }
    *reinterpret_cast<uint2*>(at + i * RPI * slot) =
        make_uint2(e4m3x4(f[0].x * inv, f[0].y * inv, f[1].x * inv, f[1].y * inv),
                   e4m3x4(f[2].x * inv, f[2].y * inv, f[3].x * inv, f[3].y * inv));
  }
  __syncwarp();  // all have read the old scale
  if (lane == 0) *scale = s;
}

// The blocks of a CTA's tokens: src[i][r] = the token of slot r of block[i], or -1;
// list[0, n) = those that are taken here.
template <int PER>
struct Blocks {
  int32_t src[PER][kScaleBlock];
  int64_t block[PER];
  int list[PER], n;
  bool lead[PER];
};

// All warps share the blocks' heads, those of the grid's other CTAs with these tokens too.
template <int D, typename T, bool SHARED, int PER>
__device__ __forceinline__ void write_blocks(const Write8Args& a, const Blocks<PER>& s) {
  const int each = 2 * a.c.hkv, units = s.n * each;
#pragma unroll 1
  for (int u = (SHARED ? blockIdx.y * kWarps : 0) + (threadIdx.x >> 5); u < units;
       u += SHARED ? gridDim.y * kWarps : kWarps) {
    const int i = PER == 1 ? 0 : s.list[u / each], hv = PER == 1 ? u : u % each;
    write_block<D, T>(a, s.block[i], s.src[i], hv >> 1, hv & 1);
  }
}

// Few tokens: a CTA each, whose threads look the list through.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, D == 128 ? 3 : 4) write8_few_kernel(const __grid_constant__ Write8Args a) {
  __shared__ Blocks<1> s;
  pdl_wait();
  const int64_t slot = a.slot_mapping[blockIdx.x], slots = a.c.num_blocks * kBlock, b = slot / kScaleBlock;
  if (slot < 0 || slot >= slots) {
    if (slot != -1 && threadIdx.x == 0) flag_error(a.err, DSA_DEVERR_SLOT_RANGE);
    return;
  }
  if (threadIdx.x < kScaleBlock) s.src[0][threadIdx.x] = -1;
  if (threadIdx.x == 0) {
    s.block[0] = b;
    s.n = 1;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < a.n_tokens; j += kThreads) {
    const int64_t other = a.slot_mapping[j];
    if (other >= 0 && other / kScaleBlock == b) atomicMax(&s.src[0][other % kScaleBlock], j);
  }
  __syncthreads();
  int first = 0;
  while (s.src[0][first] < 0) ++first;  // this token's slot is there
  if (s.src[0][first] != static_cast<int32_t>(blockIdx.x)) return;
  write_blocks<D, T, false>(a, s);
}

// Many: a CTA per 16 tokens of the list, 16 threads a token, a thread a slot of its block.
constexpr int kPer = kThreads / kScaleBlock;
template <int D, typename T, bool SHARED>
__global__ void __launch_bounds__(kThreads, 4) write8_many_kernel(const __grid_constant__ Write8Args a) {
  __shared__ Blocks<kPer> s;
  pdl_wait();
  const int lane = threadIdx.x & 31, i = threadIdx.x / kScaleBlock, r = threadIdx.x % kScaleBlock;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kPer + i, slots = a.c.num_blocks * kBlock;
  const int64_t slot = t < a.n_tokens ? a.slot_mapping[t] : -1, first = slot / kScaleBlock * kScaleBlock;
  const bool ok = slot >= 0 && slot < slots;
  if (slot != -1 && !ok && r == 0 && blockIdx.y == 0) flag_error(a.err, DSA_DEVERR_SLOT_RANGE);
  int32_t mine = -1;
  if (ok) {
    const int32_t v = a.token_of[first + r];
    if (v >= 0 && v < a.n_tokens && a.slot_mapping[v] == first + r) mine = v;
  }
  const uint32_t there = (__ballot_sync(0xffffffffu, mine >= 0) >> (lane & 16)) & 0xffffu;
  const int32_t lowest = __shfl_sync(0xffffffffu, mine, (lane & 16) + (there ? __ffs(there) - 1 : 0));
  s.src[i][r] = mine;
  if (r == 0) {
    s.block[i] = slot / kScaleBlock;
    s.lead[i] = there && lowest == t;
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // in order, alike in the CTAs that share them
    const bool lead = lane < kPer && s.lead[lane];
    const uint32_t m = __ballot_sync(0xffffffffu, lead);
    if (lead) s.list[__popc(m & ((1u << lane) - 1u))] = lane;
    if (lane == 0) s.n = __popc(m);
  }
  __syncthreads();
  write_blocks<D, T, SHARED>(a, s);
}

// ----------------------------------------------------------------------- read
// A block's first `have` rows where a scale is no power of two, or V's below 2^-64: each
// product is rounded once to the type. Apart from the others as write_odd is (V's least scale
// taken there, for all blocks: 113K rows 114.4 us, so 107.6).
template <int D, typename T>
__device__ __noinline__ void read_odd(const uint8_t* codes, int64_t slot, uint16_t* rows, int64_t row, int have,
                                      float s) {
#pragma unroll 1
  for (int i = 2 * (threadIdx.x & 31); i < have * D; i += 64) {
    const int r = i / D, c = i % D;
    float2 lo, hi;
    values(*reinterpret_cast<const uint16_t*>(codes + r * slot + c), &lo, &hi);
    *reinterpret_cast<uint32_t*>(rows + r * row + c) = narrow(product(lo.x, s), product(lo.y, s), T());
  }
}

// A warp per (block of a request, head), K and V, in order; lengths are counted in
// rounds of kThreads requests.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) read8_kernel(const __grid_constant__ Read8Args a) {
  constexpr int CH = D / 8;  // 8-byte chunks of a row of codes: 16 bytes of a row read
  constexpr int RPI = 32 / CH;
  constexpr int N = kScaleBlock / RPI;
  __shared__ int scan[33];
  __shared__ int ends[kThreads], keys[kThreads];
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ch = lane % CH, r0 = lane / CH;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + warp;  // this warp's unit, from the round's first one
  for (int q0 = 0; q0 < a.num_reqs; q0 += kThreads) {
    int n = 0;
    if (q0 + tid < a.num_reqs) {
      const int r = q0 + tid;
      const int64_t start = a.kv_start[r];
      if (start >= 0) {  // below 0: this request is not read
        const int sl = a.seq_lens[r];
        n = sl;
        const int ql = a.past ? a.qsl[r + 1] - a.qsl[r] : 0;
        n -= ql;
        if (sl < 0 || ql < 0 || n < 0 || n > a.max_keys || start + n > a.rows) {
          if (blockIdx.x == 0) flag_error(a.err, DSA_DEVERR_SEQ_RANGE);
          n = 0;
        }
      }
    }
    int tot;
    const int incl = block_scan_incl((n + kScaleBlock - 1) / kScaleBlock, scan, &tot);
    ends[tid] = incl;
    keys[tid] = n;
    __syncthreads();
    const int64_t units = static_cast<int64_t>(tot) * a.c.hkv;
    int i = 0;
    for (; at < units; at += warps) {
      const int b = static_cast<int>(at / a.c.hkv), h = static_cast<int>(at - static_cast<int64_t>(b) * a.c.hkv);
      while (ends[i] <= b) ++i;
      const int first = (b - (i > 0 ? ends[i - 1] : 0)) * kScaleBlock, have = min(kScaleBlock, keys[i] - first);
      const int64_t page = a.block_table[static_cast<int64_t>(q0 + i) * a.bt_stride + first / kBlock];
      if (page < 0 || page >= a.c.num_blocks) {
        if (lane == 0) flag_error(a.err, DSA_DEVERR_BLOCK_RANGE);
        continue;
      }
      const int part = first % kBlock / kScaleBlock;
      const uint8_t* kp = a.c.k + page * a.c.k_page + h * a.c.k_head + (part * kScaleBlock + r0) * a.c.k_slot + ch * 8;
      const uint8_t* vp = a.c.v + page * a.c.v_page + h * a.c.v_head + (part * kScaleBlock + r0) * a.c.v_slot + ch * 8;
      uint2 x[N], y[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (u * RPI + r0 < have) {
          x[u] = *reinterpret_cast<const uint2*>(kp + u * RPI * a.c.k_slot);
          y[u] = *reinterpret_cast<const uint2*>(vp + u * RPI * a.c.v_slot);
        }
      }
      const float* sp = a.c.scale + page * a.c.s_page + part * a.c.s_block + h * a.c.s_head;
      const float2 s = *reinterpret_cast<const float2*>(sp);
      const int64_t row = static_cast<int64_t>(a.kv_start[q0 + i]) + first + r0;
      if (!power_of_two(s.x) || !power_of_two(s.y) || !(s.y >= 0x1p-64f)) {
        const int64_t r = row - r0;
        read_odd<D, T>(kp - r0 * a.c.k_slot - ch * 8, a.c.k_slot, a.k + h * a.k_rhead + r * a.k_row, a.k_row, have, s.x);
        read_odd<D, T>(vp - r0 * a.c.v_slot - ch * 8, a.c.v_slot, a.v + h * a.v_rhead + r * a.v_row, a.v_row, have,
                       fmaxf(s.y, 0x1p-64f));  // as attention takes it
        continue;
      }
      uint16_t* ko = a.k + h * a.k_rhead + row * a.k_row + ch * 8;
      uint16_t* vo = a.v + h * a.v_rhead + row * a.v_row + ch * 8;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (u * RPI + r0 >= have) continue;
        *reinterpret_cast<uint4*>(ko + u * RPI * a.k_row) = row_of(x[u], s.x, T());
        *reinterpret_cast<uint4*>(vo + u * RPI * a.v_row) = row_of(y[u], s.y, T());
      }
    }
    at -= units;
    __syncthreads();  // the round's lengths are read
  }
}

template <int D, typename T>
cudaError_t write8(const Write8Args& a, int num_sms, cudaStream_t stream) {
  if (a.token_of == nullptr)
    return launch_pdl(write8_few_kernel<D, T>, dim3(static_cast<unsigned>(a.n_tokens)), dim3(kThreads), 0, stream, a);
  cudaError_t e = launch_pdl(write8_claim_kernel, dim3(static_cast<unsigned>((a.n_tokens + kThreads - 1) / kThreads)),
                             dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  // tokens may lie in one block or each in its own: few CTAs' blocks are shared by more, up to
  // 8 CTAs an SM (1500 rows of 1500 sequences 14.9 us; up to 2 17.5, up to 32 16.8)
  const int64_t chunks = (a.n_tokens + kPer - 1) / kPer, want = static_cast<int64_t>(num_sms) * 8 / chunks;
  const int64_t most = (static_cast<int64_t>(kPer) * 2 * a.c.hkv + kWarps - 1) / kWarps;
  const int64_t across = want < 1 ? 1 : want < most ? want : most;
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(across)), block(kThreads);
  // (the shared form's loop takes 40.5 us, so 35.3, for the 30572 rows)
  return across > 1 ? launch_pdl(write8_many_kernel<D, T, true>, grid, block, 0, stream, a)
                    : launch_pdl(write8_many_kernel<D, T, false>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_kv_write8(const Write8Args& a, int head_dim, int dtype, int num_sms, cudaStream_t stream) {
  if (dtype == DSA_BF16)
    return head_dim == 128 ? write8<128, __nv_bfloat16>(a, num_sms, stream)
                           : write8<64, __nv_bfloat16>(a, num_sms, stream);
  return head_dim == 128 ? write8<128, __half>(a, num_sms, stream) : write8<64, __half>(a, num_sms, stream);
}

cudaError_t launch_kv_read8(const Read8Args& a, int head_dim, int dtype, int num_sms, cudaStream_t stream) {
  // at most so many blocks are read, whatever the lengths
  const int64_t blocks = static_cast<int64_t>(a.num_reqs) * ((a.max_keys + kScaleBlock - 1) / kScaleBlock);
  int64_t grid = (blocks * a.c.hkv + kWarps - 1) / kWarps;
  // so many CTAs an SM that those at the end are short (113K rows, 8 heads of 128: 107.3 us;
  // with 16 109.0, with 8 110.9)
  const int64_t cap = static_cast<int64_t>(num_sms) * 32;
  if (grid > cap) grid = cap;
  if (grid < 1) grid = 1;
  const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
  if (dtype == DSA_BF16)
    return head_dim == 128 ? launch_pdl(read8_kernel<128, __nv_bfloat16>, g, b, 0, stream, a)
                           : launch_pdl(read8_kernel<64, __nv_bfloat16>, g, b, 0, stream, a);
  return head_dim == 128 ? launch_pdl(read8_kernel<128, __half>, g, b, 0, stream, a)
                         : launch_pdl(read8_kernel<64, __half>, g, b, 0, stream, a);
}

}  // namespace dsa
