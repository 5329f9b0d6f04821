// attn_rows.cu — attention of single query rows over the paged KV cache
// (sm_103a): every decode token over its request's pages, or any token over
// the slots that the indexer selected for it.
//
// For query head e of token t, with the KV head h = e / G it shares (G query
// heads per KV head) and the keys j that the token sees,
//   s_j = scale * q[t,e].k[j,h],   out[t,e] = sum_j p_j v[j,h] / sum_j p_j,
//   p_j = 2^(s_j log2(e) - M),     lse[t,e] = ln sum_j e^(s_j),
// for any M: numerator and denominator carry the same factor 2^-M. M only has
// to keep the p_j in range, so it is a running maximum that may lag the true
// one (kSlack below); the sums O and L are rescaled by 2^(M_old - M_new) when
// it moves. Partial results (M, L, O) over disjoint key sets add up the same
// way, which is what splits a long context over CTAs and a tile over warps.
//
// What bounds it: one read of the K and V rows, 4*D bytes per (key, KV head)
// for 4*G*D operations: HBM for the usual G. Measured, 64/8 heads of 128: 8
// requests of 128K keys 606 us (7.06 TB/s), 32 of 4K to 8K keys 127 us
// (6.4 TB/s), 64 tokens of 2048 selected slots 100 us (5.4 TB/s: single 256-byte
// rows); one request of 300 keys 9 to 10 us, the host's time for the call. 8 requests
// of 32K keys: 64/1 heads 64 us, 128/1 101, the keys alone 20: there the MMAs and
// their fragments bound it. 4096 tokens of one request, 2048 of 32K slots each,
// 64/8 heads: 4.5 ms, every row fetched through L2 for each token (34 GB, 7.5 TB/s).
// The G query heads of a KV head
// form one 16-row MMA tile, so K and V are read once for all of them; G > 16
// takes 32-row tiles (two 16-row MMA tiles on the same K and V fragments) and
// one pass over the keys per 32 heads, the passes' CTAs next to each other so
// that the later pass finds K and V in L2. Tokens of one request share nothing: n
// decode tokens read its pages n times (8 requests of 128K, 32/8 heads: one token
// each 0.62 ms, four 2.36).
//
// Mapping: the (token, 64-key tile) pairs form one flat list, cut into equally
// long slices whatever the mix of lengths; a slice is run by one CTA per KV
// head (and pass), next to each other, so that the heads' rows of a slot, which
// lie side by side in memory, are fetched at about the same time. Two CTAs of
// four warps sit on an SM. A warp owns 16 keys of every tile and
// streams them through its own ring of cp.async stages (zero-filled where a
// key is absent, so garbage or NaN bits in unwritten slots never reach an
// MMA); no block barrier sits in the stream. The stream runs on across items:
// the ring already loads the next item while one is reduced. At an item's end
// the four warps' (M, L, O) meet in shared memory; an item cut by a slice
// boundary leaves partials in the workspace, which a second small kernel adds
// in a fixed order (results do not depend on timing).
#include "attn_rows.cuh"

namespace dsa {

namespace {

template <int D, int MT>
struct RowsCfg {
  static constexpr int kRows = 16 * MT;
  static_assert(kRows == rows_of(kRows) && rows_of(kRows - 15) == kRows, "the host's plan has these rows a pass");
  static constexpr int kRowBytes = D * 2;
  static constexpr int kStageBytes = 2 * kWarpKeys * kRowBytes;  // a warp's K rows, then its V rows
  // As many stages as leave room for two CTAs on an SM (D = 128: three of 8 KB
  // per warp, 192 KB in flight on the SM).
  static constexpr int kStages = (D == 128 ? 3 : 6) - (MT == 2 ? (D == 128 ? 1 : 2) : 0);
  static constexpr int kOffMeta = kWarps * kStages * kStageBytes;
  static constexpr int kOffMl = kOffMeta + kWarps * kStages * 16;       // float2 [kWarps][kRows]
  static constexpr int kOffO = kOffMl + kWarps * kRows * 8;             // float [2][kRows][D]
  static constexpr int kOffQ = kOffO + 2 * kRows * D * 4;               // MT = 2: the item's q rows
  static constexpr int kOffScan = kOffQ + (MT == 2 ? kRows * kRowBytes : 0);  // the slice, scan scratch
  static constexpr int kSmemBytes = kOffScan + 48 * 4;
  static_assert(kRowsCtas * (kSmemBytes + 1024) <= 228 * 1024, "CTAs per SM");
  static_assert(kOffMeta >= 4096, "find_slice's rounds lie in the ring");
};

template <int D, typename T, int MT, bool SEL>
__global__ void __launch_bounds__(kThreads, kRowsCtas) attn_rows_kernel(const __grid_constant__ RowsArgs a) {
  using C = RowsCfg<D, MT>;
  using E = Elem<T>;
  constexpr int S = C::kStages;
  constexpr int CH = D / 8;          // 16-byte chunks per row
  constexpr int KS = D / 16;         // MMA k steps of q.k
  constexpr int RPI = 32 / CH;       // rows one cp.async instruction of a warp covers
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * S * C::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  int4* meta = reinterpret_cast<int4*>(smem + C::kOffMeta) + warp * S;
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  float* obuf = reinterpret_cast<float*>(smem + C::kOffO);
  uint8_t* qbuf = smem + C::kOffQ;
  Slice* slice = reinterpret_cast<Slice*>(smem + C::kOffScan);

  const int col = blockIdx.x / a.passes, pass = blockIdx.x - col * a.passes;
  const int part = col / a.hkv, h = col - part * a.hkv;    // slice (split) or token, KV head
  const int head0 = pass * C::kRows;                       // first query head of the group in this pass
  const int rows = min(C::kRows, a.group - head0);         // its query heads

  // Launched while the stream's previous kernel drains: nothing is read before
  // it has ended. The join's CTAs in turn may take the places of CTAs that have
  // ended, and wait there.
  pdl_wait();
  if (a.split) pdl_launch_dependents();
  // ---- this CTA's slice
  Cursor cur;
  cur.fresh = true;
  if (a.split) {
    find_slice<SEL>(a, part, blockIdx.x == 0, slice, reinterpret_cast<int*>(slice + 1),
                    reinterpret_cast<int*>(smem));
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

  // ---- the loader: one tile of this warp's 16 keys into a stage
  const T* kbase = static_cast<const T*>(a.k);
  const T* vbase = static_cast<const T*>(a.v);
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
      const uint32_t vdst = kdst + kWarpKeys * C::kRowBytes;
      const int c = lane % CH, r0 = lane / CH;
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
#pragma unroll
          for (int i = 0; i < kWarpKeys / RPI; ++i) {
            const int r = i * RPI + r0;
            const int64_t ko = __shfl_sync(0xffffffffu, off, r);
            const int64_t vo = __shfl_sync(0xffffffffu, off, r + 16);
            const bool ok = (mask >> r) & 1;
            const uint32_t d = r * C::kRowBytes + ((c ^ (r & 7)) << 4);
            cp16(kdst + d, kbase + ko + c * 8, ok);
            cp16(vdst + d, vbase + vo + c * 8, ok);
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
          const T* kp = kbase + nid * a.k_page + static_cast<int64_t>(warp * kWarpKeys + r0) * a.k_slot +
                        h * a.k_head + c * 8;
          const T* vp = vbase + nid * a.v_page + static_cast<int64_t>(warp * kWarpKeys + r0) * a.v_slot +
                        h * a.v_head + c * 8;
#pragma unroll
          for (int i = 0; i < kWarpKeys / RPI; ++i) {
            const int r = i * RPI + r0;
            const bool ok = r < have;
            const uint32_t d = r * C::kRowBytes + ((c ^ (r & 7)) << 4);
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

  // ---- the consumer
  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2];
  uint32_t qf[MT == 1 ? KS : 1][4];
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
#pragma unroll
      for (int x = 0; x < MT; ++x) {
        m[x][0] = m[x][1] = NEG;
        l[x][0] = l[x][1] = 0.0f;
#pragma unroll
        for (int y = 0; y < D / 8; ++y) o[x][y][0] = o[x][y][1] = o[x][y][2] = o[x][y][3] = 0.0f;
      }
      const T* q = static_cast<const T*>(a.q) + mt.y * a.q_row + static_cast<int64_t>(h * a.group + head0) * a.q_head;
      if constexpr (MT == 1) {
        const int g = lane >> 2, c2 = (lane & 3) * 2;
        const bool v0 = g < rows, v1 = g + 8 < rows;
        const T* q0 = q + (v0 ? g : 0) * a.q_head + c2;
        const T* q1 = q + (v1 ? g + 8 : 0) * a.q_head + c2;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[k][0] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + k * 16) : 0u;
          qf[k][1] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + k * 16) : 0u;
          qf[k][2] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + k * 16 + 8) : 0u;
          qf[k][3] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + k * 16 + 8) : 0u;
        }
      } else {
        // (no warp reads the previous item's rows any more: all have met at its end)
#pragma unroll 2
        for (int i = threadIdx.x; i < C::kRows * CH; i += kThreads) {
          const int r = i / CH, c = i % CH;
          const uint4 v =
              r < rows ? *reinterpret_cast<const uint4*>(q + r * a.q_head + c * 8) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(qbuf + r * C::kRowBytes + ((c ^ (r & 7)) << 4)) = v;
        }
        __syncthreads();
      }
    }

    if (mask != 0) {
      const uint32_t ks = ring_u + stage * C::kStageBytes, vs = ks + kWarpKeys * C::kRowBytes;
      // S = Q K^T: 16 keys, two 8-key MMA tiles
      float s[MT][2][4];
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) s[x][y][0] = s[x][y][1] = s[x][y][2] = s[x][y][3] = 0.0f;
      {
        const int row = (lane & 7) + ((lane >> 4) << 3), cb = (lane >> 3) & 1;
        const uint32_t base = ks + row * C::kRowBytes;
        const int qr = lane & 15, qc = lane >> 4;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          ldsm4(b, base + (((2 * k + cb) ^ (row & 7)) << 4));
#pragma unroll
          for (int x = 0; x < MT; ++x) {
            if constexpr (MT == 1) {
              E::mma(s[x][0], qf[k], b[0], b[1]);
              E::mma(s[x][1], qf[k], b[2], b[3]);
            } else {
              uint32_t q4[4];
              ldsm4(q4, smem_u32(qbuf) + (x * 16 + qr) * C::kRowBytes + (((2 * k + qc) ^ (qr & 7)) << 4));
              E::mma(s[x][0], q4, b[0], b[1]);
              E::mma(s[x][1], q4, b[2], b[3]);
            }
          }
        }
      }
      // scores in powers of two; absent keys out
      const float sc = a.scale_log2;
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][y][e] *= sc;
      if (mask != 0xffffu) {
        const int c2 = (lane & 3) * 2;
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((mask >> (y * 8 + c2 + (e & 1))) & 1)) s[x][y][e] = NEG;
      }
#pragma unroll
      for (int x = 0; x < MT; ++x) {
        float t0 = fmaxf(fmaxf(s[x][0][0], s[x][0][1]), fmaxf(s[x][1][0], s[x][1][1]));
        float t1 = fmaxf(fmaxf(s[x][0][2], s[x][0][3]), fmaxf(s[x][1][2], s[x][1][3]));
        const bool move = t0 > m[x][0] + (E::kHead + kSlack) || t1 > m[x][1] + (E::kHead + kSlack);
        if (__any_sync(0xffffffffu, move)) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
          const float n0 = fmaxf(m[x][0], t0 - E::kHead), n1 = fmaxf(m[x][1], t1 - E::kHead);
          const float f0 = m[x][0] == NEG ? 0.0f : ex2(m[x][0] - n0), f1 = m[x][1] == NEG ? 0.0f : ex2(m[x][1] - n1);
          m[x][0] = n0;
          m[x][1] = n1;
          l[x][0] *= f0;
          l[x][1] *= f1;
#pragma unroll
          for (int y = 0; y < D / 8; ++y) {
            o[x][y][0] *= f0;
            o[x][y][1] *= f0;
            o[x][y][2] *= f1;
            o[x][y][3] *= f1;
          }
        }
      }
      uint32_t p[MT][4];
#pragma unroll
      for (int x = 0; x < MT; ++x) {
        const float m0 = m[x][0] == NEG ? 0.0f : m[x][0], m1 = m[x][1] == NEG ? 0.0f : m[x][1];
        float e[8];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          e[4 * y + 0] = ex2(s[x][y][0] - m0);
          e[4 * y + 1] = ex2(s[x][y][1] - m0);
          e[4 * y + 2] = ex2(s[x][y][2] - m1);
          e[4 * y + 3] = ex2(s[x][y][3] - m1);
        }
        // the sum is taken before the weights are rounded for the MMA: the
        // rounding errors (half a step each, unbiased) enter the numerator only
        l[x][0] += (e[0] + e[1]) + (e[4] + e[5]);
        l[x][1] += (e[2] + e[3]) + (e[6] + e[7]);
        p[x][0] = E::pack(e[0], e[1]);
        p[x][1] = E::pack(e[2], e[3]);
        p[x][2] = E::pack(e[4], e[5]);
        p[x][3] = E::pack(e[6], e[7]);
      }
      // O += P V
      {
        const int row = (lane & 7) + (((lane >> 3) & 1) << 3), cb = lane >> 4;
        const uint32_t base = vs + row * C::kRowBytes;
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
          uint32_t b[4];
          ldsm4_t(b, base + (((2 * y + cb) ^ (row & 7)) << 4));
#pragma unroll
          for (int x = 0; x < MT; ++x) {
            E::mma(o[x][2 * y], p[x], b[0], b[1]);
            E::mma(o[x][2 * y + 1], p[x], b[2], b[3]);
          }
        }
      }
    }
    if (++stage == S) stage = 0;

    if (flags & kLast) {
      // ---- the four warps' partial results into one
      const int g = lane >> 2;
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = l[x][e];
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          l[x][e] = t;
        }
      __syncthreads();  // the previous item's buffers are read
      if ((lane & 3) == 0) {
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          ml[warp * C::kRows + x * 16 + g] = make_float2(m[x][0], l[x][0]);
          ml[warp * C::kRows + x * 16 + g + 8] = make_float2(m[x][1], l[x][1]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = NEG, L = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * C::kRows + x * 16 + g + 8 * e].x);
          const float Ms = M == NEG ? 0.0f : M;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 v = ml[w * C::kRows + x * 16 + g + 8 * e];
            L += v.y * ex2(v.x - Ms);
          }
          const float f = ex2(m[x][e] - Ms);
#pragma unroll
          for (int y = 0; y < D / 8; ++y) {
            o[x][y][2 * e] *= f;
            o[x][y][2 * e + 1] *= f;
          }
          m[x][e] = M;
          l[x][e] = L;
        }
      // O of warps 2, 3 into 0, 1, then of 1 into 0
      const int c2 = (lane & 3) * 2;
#pragma unroll
      for (int step = 2; step >= 1; step >>= 1) {
        if (warp >= step && warp < 2 * step) {
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int y = 0; y < D / 8; ++y)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2*>(obuf + ((warp - step) * C::kRows + x * 16 + g + 8 * e) * D +
                                           (y ^ g) * 8 + c2) =
                    make_float2(o[x][y][2 * e], o[x][y][2 * e + 1]);
        }
        __syncthreads();
        if (warp < step) {
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int y = 0; y < D / 8; ++y)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float2 v = *reinterpret_cast<const float2*>(
                    obuf + (warp * C::kRows + x * 16 + g + 8 * e) * D + (y ^ g) * 8 + c2);
                o[x][y][2 * e] += v.x;
                o[x][y][2 * e + 1] += v.y;
              }
        }
        if (step == 2) __syncthreads();
      }
      const bool whole = starts && (flags & kEndsItem);
      if (warp == 0) {
        // slot 2c: a part that continues an earlier CTA's item; 2c + 1: the beginning of one
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0);
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = x * 16 + g + 8 * e;
            if (r >= rows) continue;
            const float L = l[x][e], M = m[x][e];
            if (whole) {
              const int64_t head = static_cast<int64_t>(h) * a.group + head0 + r;
              T* out = static_cast<T*>(a.out) + mt.y * a.out_row + head * a.out_head;
              // L = 0: no key, or only scores of -infinity (O is then 0, or NaN by 0 times
              // a V that is not finite); no score but NaN leaves M alone and L NaN
              const float inv = 1.0f / L;
#pragma unroll
              for (int y = 0; y < D / 8; ++y)
                *reinterpret_cast<uint32_t*>(out + y * 8 + c2) =
                    L == 0.0f ? 0u : E::pack(o[x][y][2 * e] * inv, o[x][y][2 * e + 1] * inv);
              if (a.lse != nullptr && (lane & 3) == 0)
                a.lse[static_cast<int64_t>(mt.y) * a.heads + head] =
                    L == 0.0f ? NEG : (M + log2f(L)) * 0.6931471805599453f;
            } else {
              float* po = a.part_o + (slot * C::kRows + r) * D;
#pragma unroll
              for (int y = 0; y < D / 8; ++y)
                *reinterpret_cast<float2*>(po + y * 8 + c2) = make_float2(o[x][y][2 * e], o[x][y][2 * e + 1]);
              if ((lane & 3) == 0) a.part_ml[slot * C::kRows + r] = make_float2(M, L);
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

// The tokens cut by slice boundaries: for the token and head that main CTA b
// began, CTA (b, y) adds the partials of rows y * 8 / WAYS and following. WAYS
// warps share a row, taking its slices in turn, each in order; their sums are
// added in warp order. More than four slices per token want all eight warps on a
// row (one of 131072 keys, 32/8 heads: 38 partials a row, 83 us, with a warp per row
// 93), fewer a warp per row (32 of 2048, 64/8: 48.4 us, with eight 50.4).
constexpr int kJoinWarps = 8;

// SCALED: V's scales are in the weights, and the sums come further down than O does.
template <int D, typename T, int WAYS, bool SCALED>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const __grid_constant__ RowsArgs a, int krows,
                                                                    bool early) {
  constexpr int V = D / 32;
  constexpr int kRowsCta = kJoinWarps / WAYS;
  __shared__ float so[WAYS > 1 ? kJoinWarps : 1][D];
  __shared__ float2 sml[kJoinWarps];
  const int col = blockIdx.x / a.passes, pass = blockIdx.x - col * a.passes;
  const int part = col / a.hkv, h = col - part * a.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kRowsCta + warp / WAYS, head0 = pass * krows;
  const bool in = head0 + r < a.group && r < krows;
  if (early) pdl_launch_dependents();
  pdl_wait();
  // the main kernel's CTA of slice c with this head; a CTA has one head or two
  const int two = a.joint - 1, across = a.hkv >> two, mine = h >> two;
  auto cta = [&](int64_t c) { return (c * across + mine) * a.passes + pass; };
  const int2 d = a.desc[cta(part)];
  if (d.x < 0) return;
  float M = -INFINITY, L = 0.0f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  if (in) {
#pragma unroll 4
    for (int c = part + warp % WAYS; c <= d.y; c += WAYS) {
      const int64_t slot = ((2 * cta(c) + (c == part ? 1 : 0)) << two) + (h & two);
      const float2 v = a.part_ml[slot * krows + r];
      const float* p = a.part_o + (slot * krows + r) * D + lane * V;
      float w[V];
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = p[i];
      // a part without a weight adds 0, or NaN where V is not finite: as within a CTA
      const float n = fmaxf(M, v.x), ref = n == -INFINITY ? 0.0f : n;
      float f, e;  // -inf: 0
      if constexpr (SCALED) {
        const float hf = half_way(M - ref), he = half_way(v.x - ref);
        f = hf * hf;
        e = he * he;
        L = L * hf * hf + v.y * he * he;
      } else {
        f = ex2(M - ref);
        e = ex2(v.x - ref);
        L = L * f + v.y * e;
      }
      M = n;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * f + w[i] * e;
    }
  }
  if constexpr (WAYS > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) so[warp][lane * V + i] = o[i];
    if (lane == 0) sml[warp] = make_float2(M, L);
    __syncthreads();
    if (warp % WAYS != 0) return;
    M = -INFINITY;
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < WAYS; ++w) M = fmaxf(M, sml[warp + w].x);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < WAYS; ++w) {
      float f;
      if constexpr (SCALED) {
        const float half = half_way(sml[warp + w].x - ref);
        f = half * half;
        L += sml[warp + w].y * half * half;
      } else {
        f = ex2(sml[warp + w].x - ref);
        L += sml[warp + w].y * f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] += so[warp + w][lane * V + i] * f;
    }
  }
  if (!in) return;
  const int64_t head = static_cast<int64_t>(h) * a.group + head0 + r;
  const float inv = 1.0f / L;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + d.x * a.out_row + head * a.out_head + lane * V);
#pragma unroll
  for (int i = 0; i < V; i += 2) out[i / 2] = L == 0.0f ? 0u : Elem<T>::pack(o[i] * inv, o[i + 1] * inv);
  if (a.lse != nullptr && lane == 0)
    a.lse[static_cast<int64_t>(d.x) * a.heads + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// krows: rows of the workspace per main CTA and KV head; early: the next kernel's CTAs may begin.
template <int D, typename T, bool SCALED>
cudaError_t join(const RowsArgs& a, int krows, bool early, cudaStream_t stream) {
  const int grid = a.slices * a.hkv * a.passes;
  const int rows = a.group < krows ? a.group : krows;
  if (a.slices > 4 * static_cast<int64_t>(a.n_tokens))
    return launch_pdl(attn_join_kernel<D, T, 8, SCALED>, dim3(grid, rows), dim3(32 * kJoinWarps), 0, stream, a, krows,
                      early);
  return launch_pdl(attn_join_kernel<D, T, 1, SCALED>, dim3(grid, (rows + 7) / 8), dim3(32 * kJoinWarps), 0, stream, a, krows,
                      early);
}

template <int D, typename T, int MT, bool SEL>
cudaError_t launch(const RowsArgs& a, int grid, cudaStream_t stream) {
  static uint64_t done = 0;
  using C = RowsCfg<D, MT>;
  auto* fn = attn_rows_kernel<D, T, MT, SEL>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(fn), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(fn, dim3(grid), dim3(kThreads), C::kSmemBytes, stream, a)) != cudaSuccess || !a.split) return e;
  return join<D, T, false>(a, C::kRows, true, stream);
}

template <int D, typename T>
cudaError_t launch_dt(const RowsArgs& a, int grid, bool sel, cudaStream_t stream) {
  if (rows_of(a.group) == 16)
    return sel ? launch<D, T, 1, true>(a, grid, stream) : launch<D, T, 1, false>(a, grid, stream);
  return sel ? launch<D, T, 2, true>(a, grid, stream) : launch<D, T, 2, false>(a, grid, stream);
}

}  // namespace

cudaError_t launch_attn_rows(const RowsArgs& a, int head_dim, int dtype, bool selected, cudaStream_t stream) {
  const int grid = a.slices * a.hkv * a.passes;
  if (dtype == DSA_BF16)
    return head_dim == 128 ? launch_dt<128, __nv_bfloat16>(a, grid, selected, stream)
                           : launch_dt<64, __nv_bfloat16>(a, grid, selected, stream);
  return head_dim == 128 ? launch_dt<128, __half>(a, grid, selected, stream)
                         : launch_dt<64, __half>(a, grid, selected, stream);
}

cudaError_t launch_attn_join8(const RowsArgs& a, int head_dim, bool bf16, int krows, cudaStream_t stream) {
  if (bf16)
    return head_dim == 128 ? join<128, __nv_bfloat16, true>(a, krows, false, stream)
                           : join<64, __nv_bfloat16, true>(a, krows, false, stream);
  return head_dim == 128 ? join<128, __half, true>(a, krows, false, stream)
                         : join<64, __half, true>(a, krows, false, stream);
}

}  // namespace dsa
