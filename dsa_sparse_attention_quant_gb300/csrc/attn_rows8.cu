// attn_rows8.cu — attention of single query rows over a paged KV cache in 8 bits
// (sm_103a): every decode token over its request's pages, or any token over the
// slots that the indexer selected for it.
//
// A key's row is sk * ck: E4M3 codes ck and a scale sk per block of 16 slots and KV
// head, K and V apart. With query head e sharing KV head h,
//   s_j = scale * sk_j * (q[t,e].ck_j),  out[t,e] = sum_j e^(s_j) sv_j cv_j / sum_j e^(s_j).
// K's scale multiplies the fp32 scores. V's goes into the exponent:
//   t_j = s_j log2(e) + log2(sv_j),  w_j = 2^(t_j - M),
//   out = sum_j w_j cv_j / L,  L = sum_j w_j / sv_j,  lse = ln(2^M L)
// for any reference M, a running maximum of the t_j that may lag (kSlack); so the
// sums rescale, split and join as those of attn_rows.cu do, and one number per key
// is all that the scales cost.
//
// E4M3 codes are exact in fp16, so both products run as fp16 MMAs with fp32 sums
// whatever q's type: bf16 rows of q are multiplied by the power of two that brings
// their largest magnitude into [2^14, 2^15) (what falls below 2^-24 then is 2^-38 of
// that element or less), taken back with the scores' scale. The weights w_j are
// rounded to fp16 for the second product (2^-11 relative, 2^-24 in absolute terms
// where the largest is 2^6 at least).
//
// What bounds it: one read of the codes, 2*D bytes a (key, KV head), and 0.5 of
// scales for 4*G*D operations.
//
// Mapping: slices, warps and rings as in attn_rows.cu. The MMAs take the keys as
// their 16 rows and the query heads as their 8 columns (S^T = K q^T, O^T = V^T P^T):
// G <= 8 query heads fill the tile that a 16-row tile of heads would half fill, and
// K's and V's fragments, which have to be made from codes, are A operands that
// several tiles of heads share. A lane's four codes of a K row are four columns
// d..d+3: two of them are taken as the MMA's k slots 2c, 2c+1 and two as 2c+8, 2c+9,
// and q's columns are loaded in that order. V comes through the transposing ldmatrix
// as pairs of codes (2d, 2d+1): even columns become the tile's rows 0-7, odd ones
// rows 8-15, so that no byte moves between lanes. P^T is S^T's fragment transposed
// (movmatrix).
#include "attn_rows.cuh"

namespace dsa {

namespace {

constexpr int kScaleBlock = DSA_SCALE_BLOCK;
static_assert(kWarpKeys == kScaleBlock, "a warp's keys of a tile share their scales");
constexpr float kLeastScale = 0x1p-64f, kMostScale = 0x1p126f;

template <int D, int NT>
struct Rows8Cfg {
  static constexpr int kRows = 8 * NT;                  // query heads of a pass
  static constexpr int kStageBytes = 2 * kWarpKeys * D;  // a warp's K codes, then its V codes
  static constexpr int kStages = (D == 128 ? 5 : 10) - (NT == 4 ? (D == 128 ? 1 : 2) : 0);
  static constexpr int kORow = D + 4;  // floats between rows of obuf: lanes of a store on 32 banks
  static constexpr int kOffMeta = kWarps * kStages * kStageBytes;
  static constexpr int kOffScale = kOffMeta + kWarps * kStages * 16;             // float2 [kWarps][kStages][16]
  static constexpr int kOffMl = kOffScale + kWarps * kStages * kWarpKeys * 8;    // float2 [kWarps][kRows]
  static constexpr int kOffO = kOffMl + kWarps * kRows * 8;                      // float [2][kRows][kORow]
  static constexpr int kOffScan = kOffO + 2 * kRows * kORow * 4;                 // the slice, scan scratch
  static constexpr int kSmemBytes = kOffScan + 48 * 4;
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(kOffMeta >= 4096, "find_slice's rounds lie in the ring");
};

// Where 16-byte chunk c of row r lies in a row of D codes: eight rows' chunks c on all banks.
template <int D>
__device__ __forceinline__ int swz(int r, int c) {
  return (D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4;
}

// Two E4M3 codes as fp16, exact.
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(codes));
  return h;
}
__device__ __forceinline__ uint32_t half2_of_high(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(codes));
  return h;
}
// An 8x8 tile of 16-bit elements transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// 8 bytes global -> shared, zeros when `in` is false.
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0) : "memory");
}

// A row of q as the MMA's B fragments: q4 of four columns each, in fp16. Returns what
// the scores have to be multiplied by. All lanes of a row (4) call.
template <int KS>
__device__ __forceinline__ float q_fragments(uint2 (&q4)[KS], __half) {
  return 1.0f;
}
template <int KS>
__device__ __forceinline__ float q_fragments(uint2 (&q4)[KS], __nv_bfloat16) {
  uint32_t most = 0;  // of the magnitudes' bits: NaN above infinity above the rest
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    most = __vmaxu2(most, q4[k].x & 0x7FFF7FFFu);
    most = __vmaxu2(most, q4[k].y & 0x7FFF7FFFu);
  }
  most = max(most & 0xFFFFu, most >> 16);
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  // 2^(14 - e) for magnitudes of exponent e, which is held above -100: what is smaller scores 0
  const int e = max(static_cast<int>(most >> 7) - 127, -100);
  const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q4[k].x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q4[k].y));
    q4[k].x = Elem<__half>::pack(a.x * up, a.y * up);
    q4[k].y = Elem<__half>::pack(b.x * up, b.y * up);
  }
  return __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

template <int D, typename T, int NT, bool SEL>
__global__ void __launch_bounds__(kThreads, 2) attn_rows8_kernel(const __grid_constant__ Rows8Args a) {
  using C = Rows8Cfg<D, NT>;
  using E = Elem<__half>;
  constexpr int S = C::kStages;
  constexpr int CH = D / 16;    // 16-byte chunks per row of codes
  constexpr int KS = D / 16;    // MMA k steps of q.k
  constexpr int RPI = 32 / CH;  // rows one cp.async instruction of a warp covers
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring_u = smem_u32(smem + warp * S * C::kStageBytes);
  int4* meta = reinterpret_cast<int4*>(smem + C::kOffMeta) + warp * S;
  float2* scales = reinterpret_cast<float2*>(smem + C::kOffScale) + warp * S * kWarpKeys;
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  float* obuf = reinterpret_cast<float*>(smem + C::kOffO);
  Slice* slice = reinterpret_cast<Slice*>(smem + C::kOffScan);

  const int col = blockIdx.x / a.passes, pass = blockIdx.x - col * a.passes;
  const int part = col / a.hkv, h = col - part * a.hkv;  // slice (split) or token, KV head
  const int head0 = pass * C::kRows;                     // first query head of the group in this pass
  const int rows = min(C::kRows, a.group - head0);       // its query heads

  // Launched while the stream's previous kernel drains: nothing is read before
  // it has ended. The join's CTAs in turn may take the places of CTAs that have
  // ended, and wait there.
  pdl_wait();
  if (a.split) pdl_launch_dependents();
  // ---- this CTA's slice
  Cursor cur;
  cur.fresh = true;
  if (a.split) {
    find_slice<SEL>(a, part, blockIdx.x == 0, slice, reinterpret_cast<int*>(slice + 1), reinterpret_cast<int*>(smem));
    cur.left = slice->left;
    if (cur.left == 0) {  // fewer tiles than slices
      if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int2(-1, 0);
      return;
    }
    cur.t = slice->t;
    cur.kt = slice->kt;
    cur.n = slice->n;
    cur.req = slice->req;
    cur.tiles = tiles_of(cur.n);
  } else {
    cur.t = part;
    cur.kt = 0;
    if (SEL) {
      cur.n = a.topk;
      cur.req = 0;
    } else {
      cur.n = token_keys(a, cur.t, &cur.req, threadIdx.x == 0 && h == 0 && pass == 0);
    }
    cur.tiles = tiles_of(cur.n);
    cur.left = cur.tiles;
  }
  int desc_token = -1, desc_last = 0;  // the slice ends inside a token that it began: which, and its last slice

  // ---- the loader: one tile of this warp's 16 keys and their scales into a stage
  const uint8_t* kbase = static_cast<const uint8_t*>(a.k);
  const uint8_t* vbase = static_cast<const uint8_t*>(a.v);
  int32_t nid = -1;  // dense: the next tile's page; selected: this lane's slot of the next tile (lane & 15)
  auto fetch_id = [&]() {
    nid = -1;
    if (cur.left <= 0) return;
    if (SEL) {
      const int j = cur.kt * kTile + warp * kWarpKeys + (lane & 15);
      if (j < a.topk) nid = a.physical[static_cast<int64_t>(cur.t) * a.topk + j];
    } else if (cur.n > 0) {
      nid = a.block_table[static_cast<int64_t>(cur.req) * a.bt_stride + cur.kt];
    }
  };
  auto issue = [&](int stage) {
    if (cur.left > 0) {
      const uint32_t kdst = ring_u + stage * C::kStageBytes;
      const uint32_t vdst = kdst + kWarpKeys * D;
      const uint32_t sdst = smem_u32(scales + stage * kWarpKeys);
      const int ch = lane % CH, r0 = lane / CH;
      uint32_t mask = 0;
      if (SEL) {
        const bool in = nid >= 0 && static_cast<int64_t>(nid) < a.num_slots;
        if (nid < -1 || (nid >= 0 && !in)) flag_error(a.err, DSA_DEVERR_ID_RANGE);
        mask = __ballot_sync(0xffffffffu, in) & 0xffffu;
        // lanes 0-15 hold the K rows' offsets, lanes 16-31 the V rows'
        const bool isv = lane >= 16;
        const int64_t page = in ? nid / kBlock : 0, slot = in ? nid % kBlock : 0;
        const int64_t off = isv ? page * a.v_page + slot * a.v_slot + h * a.v_head
                                : page * a.k_page + slot * a.k_slot + h * a.k_head;
        if (mask != 0) {
          if (!isv) cp8(sdst + lane * 8, a.scale + page * a.s_page + slot / kScaleBlock * a.s_block + h * a.s_head, in);
#pragma unroll
          for (int i = 0; i < kWarpKeys / RPI; ++i) {
            const int r = i * RPI + r0;
            const int64_t ko = __shfl_sync(0xffffffffu, off, r);
            const int64_t vo = __shfl_sync(0xffffffffu, off, r + 16);
            const bool ok = (mask >> r) & 1;
            const uint32_t d = r * D + swz<D>(r, ch);
            cp16(kdst + d, kbase + ko + ch * 16, ok);
            cp16(vdst + d, vbase + vo + ch * 16, ok);
          }
        }
      } else {
        const int j0 = cur.kt * kTile + warp * kWarpKeys;
        int have = min(kWarpKeys, cur.n - j0);
        if (cur.n > 0 && (nid < 0 || static_cast<int64_t>(nid) >= a.num_blocks)) {
          if (lane == 0) flag_error(a.err, DSA_DEVERR_BLOCK_RANGE);
          have = 0;
        }
        if (have > 0) {
          mask = (1u << have) - 1u;
          if (lane == 0) cp8(sdst, a.scale + nid * a.s_page + warp * a.s_block + h * a.s_head, true);
          const uint8_t* kp = kbase + nid * a.k_page + static_cast<int64_t>(warp * kWarpKeys + r0) * a.k_slot +
                              h * a.k_head + ch * 16;
          const uint8_t* vp = vbase + nid * a.v_page + static_cast<int64_t>(warp * kWarpKeys + r0) * a.v_slot +
                              h * a.v_head + ch * 16;
#pragma unroll
          for (int i = 0; i < kWarpKeys / RPI; ++i) {
            const int r = i * RPI + r0;
            const bool ok = r < have;
            const uint32_t d = r * D + swz<D>(r, ch);
            cp16(kdst + d, ok ? kp + i * RPI * a.k_slot : kbase, ok);
            cp16(vdst + d, ok ? vp + i * RPI * a.v_slot : vbase, ok);
          }
        }
      }
      const bool ends = cur.kt == cur.tiles - 1, last = ends || cur.left == 1;
      if (lane == 0) {
        const int flags = (cur.fresh ? kFirst : 0) | (last ? kLast : 0) | (cur.kt == 0 ? kStartsItem : 0) |
                          (ends ? kEndsItem : 0);
        meta[stage] = make_int4(static_cast<int>(mask) | (flags << 16), cur.t, cur.tiles - 1 - cur.kt, 0);
      }
      // advance
      cur.fresh = last;
      --cur.left;
      if (!ends) {
        ++cur.kt;
      } else {
        cur.kt = 0;
        ++cur.t;
        if (cur.left > 0) enter_token<SEL>(a, cur);
      }
      fetch_id();
    }
    cp_commit();
  };

  const int total = cur.left;
  fetch_id();
#pragma unroll 1
  for (int s = 0; s < S - 1; ++s) issue(s);

  // ---- the consumer: lane (g, c) has keys g, g + 8 of a tile, query heads 2c, 2c + 1
  // of each eight, and columns 16y + 2g, 16y + 2g + 1 of O
  float o[NT][CH][4];
  float m[NT][2], l[NT][2], rf[NT][2];
  uint2 qf[NT][KS];
  bool starts = true;
  const float NEG = -INFINITY;
  int stage = 0, into = S - 1;
#pragma unroll 1
  for (int it = 0; it < total; ++it) {
    cp_wait<S - 2>();
    __syncwarp();
    const int4 mt = meta[stage];
    const uint32_t mask = static_cast<uint32_t>(mt.x) & 0xffffu;
    const int flags = mt.x >> 16;
    issue(into);  // the stage consumed in the previous step
    if (++into == S) into = 0;

    if (flags & kFirst) {
      starts = flags & kStartsItem;
      const T* q = static_cast<const T*>(a.q) + mt.y * a.q_row + static_cast<int64_t>(h * a.group + head0) * a.q_head;
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        m[x][0] = m[x][1] = NEG;
        l[x][0] = l[x][1] = 0.0f;
#pragma unroll
        for (int y = 0; y < CH; ++y) o[x][y][0] = o[x][y][1] = o[x][y][2] = o[x][y][3] = 0.0f;
        const bool in = x * 8 + g < rows;
        const T* qp = q + (in ? x * 8 + g : 0) * a.q_head + c * 4;
#pragma unroll
        for (int k = 0; k < KS; ++k)
          qf[x][k] = in ? *reinterpret_cast<const uint2*>(qp + k * 16) : make_uint2(0, 0);
        const float f = q_fragments<KS>(qf[x], T()) * a.scale_log2;  // of row x * 8 + g
        rf[x][0] = __shfl_sync(0xffffffffu, f, 8 * c);
        rf[x][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
      }
    }

    if (mask != 0) {
      const uint32_t ks = ring_u + stage * C::kStageBytes, vs = ks + kWarpKeys * D;
      // S^T = K q^T
      float s[NT][4];
#pragma unroll
      for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.0f;
      {
        const int row = (lane & 7) + ((lane >> 4) << 3), cb = (lane >> 3) & 1;
        const uint32_t base = ks + row * D;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t b[4];  // keys 0-7 chunks k, k + 1; keys 8-15 chunks k, k + 1
          ldsm4(b, base + swz<D>(row, k + cb));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t f[4] = {half2_of(b[u]), half2_of(b[2 + u]), half2_of_high(b[u]), half2_of_high(b[2 + u])};
#pragma unroll
            for (int x = 0; x < NT; ++x) E::mma(s[x], f, qf[x][k + u].x, qf[x][k + u].y);
          }
        }
      }
      // scores in powers of two with V's scale in them; absent keys out
      const float2* sc = scales + stage * kWarpKeys;
      const float2 s0 = sc[SEL ? g : 0], s1 = SEL ? sc[g + 8] : s0;
      const float v0 = fminf(fmaxf(s0.y, kLeastScale), kMostScale), v1 = fminf(fmaxf(s1.y, kLeastScale), kMostScale);
      const float lv0 = __log2f(v0), lv1 = __log2f(v1);
      const float iv0 = __frcp_rn(v0), iv1 = __frcp_rn(v1);
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        s[x][0] = fmaf(s[x][0], rf[x][0] * s0.x, lv0);
        s[x][1] = fmaf(s[x][1], rf[x][1] * s0.x, lv0);
        s[x][2] = fmaf(s[x][2], rf[x][0] * s1.x, lv1);
        s[x][3] = fmaf(s[x][3], rf[x][1] * s1.x, lv1);
      }
      if (mask != 0xffffu) {
        const bool in0 = (mask >> g) & 1, in1 = (mask >> (g + 8)) & 1;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (!in0) s[x][0] = s[x][1] = NEG;
          if (!in1) s[x][2] = s[x][3] = NEG;
        }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float t0 = fmaxf(s[x][0], s[x][2]), t1 = fmaxf(s[x][1], s[x][3]);
        const bool move = t0 > m[x][0] + (E::kHead + kSlack) || t1 > m[x][1] + (E::kHead + kSlack);
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int i = 4; i < 32; i *= 2) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, i));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, i));
          }
          const float n0 = fmaxf(m[x][0], t0 - E::kHead), n1 = fmaxf(m[x][1], t1 - E::kHead);
          const float f0 = m[x][0] == NEG ? 0.0f : ex2(m[x][0] - n0), f1 = m[x][1] == NEG ? 0.0f : ex2(m[x][1] - n1);
          m[x][0] = n0;
          m[x][1] = n1;
          l[x][0] *= f0;
          l[x][1] *= f1;
#pragma unroll
          for (int y = 0; y < CH; ++y) {
            o[x][y][0] *= f0;
            o[x][y][1] *= f1;
            o[x][y][2] *= f0;
            o[x][y][3] *= f1;
          }
        }
        const float m0 = m[x][0] == NEG ? 0.0f : m[x][0], m1 = m[x][1] == NEG ? 0.0f : m[x][1];
        const float e0 = ex2(s[x][0] - m0), e1 = ex2(s[x][1] - m1), e2 = ex2(s[x][2] - m0), e3 = ex2(s[x][3] - m1);
        // the sums are taken before the weights are rounded for the MMA: the
        // rounding errors (half a step each, unbiased) enter the numerator only
        l[x][0] = fmaf(e0, iv0, fmaf(e2, iv1, l[x][0]));
        l[x][1] = fmaf(e1, iv0, fmaf(e3, iv1, l[x][1]));
        p[x][0] = transpose8(E::pack(e0, e1));
        p[x][1] = transpose8(E::pack(e2, e3));
      }
      // O^T += V^T P^T
      {
        const int row = (lane & 7) + (((lane >> 3) & 1) << 3), cb = lane >> 4;
        const uint32_t base = vs + row * D;
#pragma unroll
        for (int y = 0; y < CH; y += 2) {
          uint32_t b[4];  // chunk y: keys 0-7, 8-15; chunk y + 1: keys 0-7, 8-15
          ldsm4_t(b, base + swz<D>(row, y + cb));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            // codes (key 2c: even, odd column; key 2c + 1: even, odd) -> a column's two keys
            const uint32_t w0 = __byte_perm(b[2 * u], 0, 0x3120), w1 = __byte_perm(b[2 * u + 1], 0, 0x3120);
            const uint32_t f[4] = {half2_of(w0), half2_of_high(w0), half2_of(w1), half2_of_high(w1)};
#pragma unroll
            for (int x = 0; x < NT; ++x) E::mma(o[x][y + u], f, p[x][0], p[x][1]);
          }
        }
      }
    }
    if (++stage == S) stage = 0;

    if (flags & kLast) {
      // ---- the four warps' partial results into one
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = l[x][e];
#pragma unroll
          for (int i = 4; i < 32; i *= 2) t += __shfl_xor_sync(0xffffffffu, t, i);
          l[x][e] = t;
        }
      __syncthreads();  // the previous item's buffers are read
      if (g == 0) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) ml[warp * C::kRows + x * 8 + 2 * c + e] = make_float2(m[x][e], l[x][e]);
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = NEG, L = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * C::kRows + x * 8 + 2 * c + e].x);
          const float Ms = M == NEG ? 0.0f : M;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 v = ml[w * C::kRows + x * 8 + 2 * c + e];
            L += v.y * ex2(v.x - Ms);
          }
          const float f = ex2(m[x][e] - Ms);
#pragma unroll
          for (int y = 0; y < CH; ++y) {
            o[x][y][e] *= f;
            o[x][y][2 + e] *= f;
          }
          m[x][e] = M;
          l[x][e] = L;
        }
      // O of warps 2, 3 into 0, 1, then of 1 into 0
#pragma unroll
      for (int step = 2; step >= 1; step >>= 1) {
        if (warp >= step && warp < 2 * step) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int y = 0; y < CH; ++y)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2*>(obuf + ((warp - step) * C::kRows + x * 8 + 2 * c + e) * C::kORow + y * 16 +
                                           2 * g) = make_float2(o[x][y][e], o[x][y][2 + e]);
        }
        __syncthreads();
        if (warp < step) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int y = 0; y < CH; ++y)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float2 v = *reinterpret_cast<const float2*>(
                    obuf + (warp * C::kRows + x * 8 + 2 * c + e) * C::kORow + y * 16 + 2 * g);
                o[x][y][e] += v.x;
                o[x][y][2 + e] += v.y;
              }
        }
        if (step == 2) __syncthreads();
      }
      const bool whole = starts && (flags & kEndsItem);
      if (warp == 0) {
        // slot 2c: a part that continues an earlier CTA's item; 2c + 1: the beginning of one
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0);
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = x * 8 + 2 * c + e;
            if (r >= rows) continue;
            const float L = l[x][e], M = m[x][e];
            if (whole) {
              const int64_t head = static_cast<int64_t>(h) * a.group + head0 + r;
              T* out = static_cast<T*>(a.out) + mt.y * a.out_row + head * a.out_head;
              // L = 0: no key, or only scores of -infinity (O is then 0, or NaN by 0 times
              // a V that is NaN); no score but NaN leaves M alone and L NaN
              const float inv = 1.0f / L;
#pragma unroll
              for (int y = 0; y < CH; ++y)
                *reinterpret_cast<uint32_t*>(out + y * 16 + 2 * g) =
                    L == 0.0f ? 0u : Elem<T>::pack(o[x][y][e] * inv, o[x][y][2 + e] * inv);
              if (a.lse != nullptr && g == 0)
                a.lse[static_cast<int64_t>(mt.y) * a.heads + head] =
                    L == 0.0f ? NEG : (M + log2f(L)) * 0.6931471805599453f;
            } else {
              float* po = a.part_o + (slot * C::kRows + r) * D;
#pragma unroll
              for (int y = 0; y < CH; ++y)
                *reinterpret_cast<float2*>(po + y * 16 + 2 * g) = make_float2(o[x][y][e], o[x][y][2 + e]);
              if (g == 0) a.part_ml[slot * C::kRows + r] = make_float2(M, L);
            }
          }
      }
      if (!whole && starts) {  // it began here and goes on: mt.z tiles after this one, in the next slices
        desc_token = mt.y;
        const int64_t end = slice->end + mt.z;
        desc_last = static_cast<int>((end * slice->in_use + slice->all - 1) / slice->all) - 1;
      }
    }
  }
  cp_wait<0>();
  if (a.split && threadIdx.x == 0) a.desc[blockIdx.x] = make_int2(desc_token, desc_last);
}

template <int D, typename T, int NT, bool SEL>
cudaError_t launch(const Rows8Args& a, int grid, int dtype, cudaStream_t stream) {
  static uint64_t done = 0;
  using C = Rows8Cfg<D, NT>;
  auto* fn = attn_rows8_kernel<D, T, NT, SEL>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(fn), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(fn, dim3(grid), dim3(kThreads), C::kSmemBytes, stream, a)) != cudaSuccess || !a.split) return e;
  return launch_attn_join(a, D, dtype, grid, C::kRows, stream);
}

template <int D, typename T>
cudaError_t launch_dt(const Rows8Args& a, int grid, int dtype, bool sel, cudaStream_t stream) {
  if (a.group <= 8)
    return sel ? launch<D, T, 1, true>(a, grid, dtype, stream) : launch<D, T, 1, false>(a, grid, dtype, stream);
  if (a.group <= 16)
    return sel ? launch<D, T, 2, true>(a, grid, dtype, stream) : launch<D, T, 2, false>(a, grid, dtype, stream);
  return sel ? launch<D, T, 4, true>(a, grid, dtype, stream) : launch<D, T, 4, false>(a, grid, dtype, stream);
}

}  // namespace

cudaError_t launch_attn_rows8(const Rows8Args& a, int head_dim, int dtype, bool selected, cudaStream_t stream) {
  const int grid = a.slices * a.hkv * a.passes;
  if (dtype == DSA_BF16)
    return head_dim == 128 ? launch_dt<128, __nv_bfloat16>(a, grid, dtype, selected, stream)
                           : launch_dt<64, __nv_bfloat16>(a, grid, dtype, selected, stream);
  return head_dim == 128 ? launch_dt<128, __half>(a, grid, dtype, selected, stream)
                         : launch_dt<64, __half>(a, grid, dtype, selected, stream);
}

}  // namespace dsa
