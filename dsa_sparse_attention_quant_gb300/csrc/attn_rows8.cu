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
// is all that the scales cost. Scales of V may be 2^184 apart (a block of zeros has the
// least), and a key that is nothing to O still has its share e^(s_j) of L. So that w_j
// does not end before the share counts for nothing, a scale below 2^-96 of one that has
// moved M is taken as that (kSpread): O is off by 2^-96 of that scale's weight of e^(s_j)
// at most. And parts' L are joined by factors that do not end where O's do (half_way).
//
// E4M3 codes are exact in fp16, so both products run as fp16 MMAs with fp32 sums
// whatever q's type: bf16 rows of q are multiplied by the power of two that brings
// their largest magnitude into [2^14, 2^15) (what falls below 2^-24 then is 2^-38 of
// that element or less), taken back with the scores' scale. The weights w_j are
// rounded to fp16 for the second product (2^-11 relative, 2^-24 in absolute terms
// where the largest is 2^6 at least).
//
// What bounds it: one read of the codes, 2*D bytes a (key, KV head), and 0.5 of
// scales for 4*G*D operations: HBM, in the large calls. 64/8 heads of 128: 8 requests of 128K
// keys 316 us (6.8 TB/s), 32 of 4K to 8K 73 us (5.6: 4 us until all CTAs stream,
// 4 between their ends, 3 of the join); 64 tokens of 2048 selected slots 63 us (4.3 TB/s:
// rows of 128 bytes, in an order of their own: place_slots); 24 requests of 1
// to 4001, 16/16 heads of 64, 28 us. One request of 300 keys takes 9 to 10 us, the host's time for
// the call. More than 16 query heads a KV head: the making of fragments and the MMAs (8
// requests of 32K keys, 64/1 heads of 128: 61 us, the keys alone 10).
//
// Fragments: the MMAs take the keys as their 16 rows and the query heads as their 8
// columns (S^T = K q^T, O^T = V^T P^T): G <= 8 query heads fill the tile that a 16-row
// tile of heads would half fill, and K's and V's fragments, which have to be made from
// codes, are A operands that two tiles of heads share (G > 8). More than 16 query heads
// take a pass over the keys per 16 of them: with tiles for 32 the registers do not suffice
// (8 requests of 32K keys, 64/1 heads of 128: 61 us, so 74; 40/2 of 64: 52, so 98). A
// lane's four codes of a K row are four columns d..d+3: two of them are taken as the MMA's
// k slots 2c, 2c+1 and two as 2c+8, 2c+9, and q's columns are loaded in that order. V
// comes through the transposing ldmatrix as pairs of codes (2d, 2d+1): even columns become
// the tile's rows 0-7, odd ones rows 8-15, so that no byte moves between lanes. P^T is
// S^T's fragment transposed (movmatrix).
//
// Mapping: the (token, 64-key tile) list is cut into slices, and parts are joined, as in
// attn_rows.cu. A CTA has four consumer warps, which own 16 keys of a tile each (a scale
// block), and a loader warp, which finds tokens, pages and slots ahead, 32 tiles at a time,
// and fills the stages with TMA boxes of 16 slots; so the consumers' registers hold only
// what the products need, and three CTAs sit on an SM, or two for pairs of heads with G > 8 (each
// warp with copies of its own, two CTAs: 8 requests of 128K keys 361 us, 32 of 4K to 8K 84).
// Selected slots' rows the consumers fetch themselves (Load, below), from addresses that
// the loader has made. Heads of 64 are taken two at a time where they lie side by side, so
// that a row in shared memory is 128 bytes (the ragged requests: 39 us, so 27).
//
// Short tokens (rows_plan) are shared by the CTAs of a cluster, which join a token's rows
// out of each other's shared memory: one launch and no scratch.
#include "attn_rows.cuh"

namespace dsa {

namespace {

constexpr int kScaleBlock = DSA_SCALE_BLOCK;
static_assert(kWarpKeys == kScaleBlock, "a warp's keys of a tile share their scales");
constexpr float kLeastScale = 0x1p-64f, kMostScale = 0x1p126f;
// With the key k that made M (w_k = 2^6 or more) and a key j: w_j >= 2^6 e^(s_j - s_k) kSpread, which
// is a number down to a share of 2^-36. Nothing in the stream pays for it but a register; where
// the shares of such keys were added apart, by a branch for each tile, 8 requests of 32K keys, 64/4
// heads of 128, took 65.4 us, so 64.4, and 24 of 1 to 4001 keys, 16/16 of 64, 28.4, so 27.7.
constexpr float kSpread = 0x1p-96f;

// How codes come into shared memory: TMA boxes of a page's 16 slots, asked for by the
// loader; or 16 bytes a lane from the selected slots, asked for by the warps that use them
// (64 tokens of 2048 slots: TMA gathers of four slots' rows 90 us, bulk copies of four
// heads a slot 93, single rows 184).
enum Load : int { kPages, kSlots };

constexpr int kFirstTiles = 6;    // a CTA's first tiles of slots, read in the list's order
constexpr int kOrderedTiles = 8;  // fewer tiles of slots at a time are there sooner than they are in order
constexpr int64_t kApart = 1 << 28;
constexpr int kThreads8 = kThreads + 32;  // the consumers, and the loader

// A row in shared memory is HP heads of a slot, 128 bytes: one head of 128, or two of 64
// that lie side by side in the cache (64 bytes, where they do not). A tile is four blocks
// of 16 rows, a warp's each.
template <int D, int HP, int NT, int LOAD>
struct Rows8Cfg {
  static constexpr int kRows = 8 * NT;                         // query heads of a KV head in a pass
  static constexpr int kRowBytes = HP * D;
  static constexpr int kCtas = rows8_ctas(kRows, HP);           // per SM
  static_assert(kRows == rows8_of(kRows) && rows8_of(kRows - 7) == kRows, "the host's plan has these rows a pass");
  // q's fragments in shared memory, each thread's its own, where registers do not hold them: three CTAs
  // then (8 requests of 32K keys, 64/1 heads of 128: 60.7 us, two with q in registers 64.9; 128/1 97.6,
  // 108.3; but pairs of 40/2 heads of 64 67.5, two 58.3)
  static constexpr bool kKeptQ = HP == 1 && NT * D > 128;
  static constexpr int kStageBytes = 2 * kTile * kRowBytes;    // a tile's K codes, then its V codes
  // D = 128: 8 requests of 128K keys, 64/8 heads: 321 us, with four stages 349
  static constexpr int kStages = LOAD == kSlots ? (kRowBytes == 64 ? 5 : kCtas == 3 ? 3 : 4)
                                                : (kRowBytes == 128 ? 1 : 2) * (kCtas == 3 ? 3 : 6);
  // what a tile's consumers have to know besides, made by the loader: as far ahead as
  // the codes are, or with slots further, since their addresses come this way
  static constexpr int kInfos = LOAD == kSlots ? (kKeptQ ? 5 : 8) : kStages;
  static constexpr int kScales = kTile * HP;
  static constexpr int kOffMeta = kStages * kStageBytes;                  // int4 [kInfos]
  static constexpr int kOffBar = kOffMeta + kInfos * 16;                 // full, empty, scaled [kInfos], meeting
  static constexpr int kOffScale = kOffBar + kInfos * 32;                 // float2 [kInfos][kScales]
  static constexpr int kOffAt = kOffScale + kInfos * kScales * 8;         // slots: longlong2 [kInfos][kTile]
  // slots: the next tiles' (a window), in the order in which they are read
  static constexpr int kWindow = kKeptQ ? kFirstTiles : 12;  // (kKeptQ: no room for more)
  static constexpr int kOffIds = kOffAt + (LOAD == kSlots ? kInfos * kTile * 16 : 0);      // int [kWindow][kTile]
  static constexpr int kOffMl = kOffIds + (LOAD == kSlots ? kWindow * kTile * 4 : 0);      // float2 [kWarps][HP][kRows]
  static constexpr int kOffParts = kOffMl + kWarps * HP * kRows * 8;      // cluster: float2 [HP][kRows]
  static constexpr int kOffScan = kOffParts + HP * kRows * 8;             // the slice, scan scratch, abort flag
  static constexpr int kOffQ = (kOffScan + 49 * 4 + 15) / 16 * 16;        // uint4 [NT * D / 32][kThreads]
  static constexpr int kSmemBytes = kKeptQ ? kOffQ + NT * D / 32 * kThreads * 16 : kOffScan + 49 * 4;
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "CTAs per SM");
  static_assert(kWarps * HP * 8 * D * 4 == kStageBytes, "O of four warps' eight heads fits a stage");
  static_assert(kOffMeta >= 4096, "find_slice's rounds lie in the ring");
  static_assert(kInfos > kStages || LOAD == kPages, "the loader runs ahead");
};

// Where 16-byte chunk c of row r lies in a row of BYTES: eight rows' chunks c on all
// banks; what the 128- and 64-byte swizzles of TMA copies give.
template <int BYTES>
__device__ __forceinline__ int swz(int r, int c) {
  return (BYTES == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4;
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
// A box of a 4-D tensor map into shared memory, completing on an mbarrier.
__device__ __forceinline__ void tma_box_4d(void* dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1,
                                           int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
      "%6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// This thread's plain accesses to shared memory before later TMA copies there.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 8 bytes global -> shared.
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A weight as fp16 rounds it, but with all its bits however small it is: weights that are little
// of O, by V's scale, may be a good part of L.
__device__ __forceinline__ float to_11_bits(float e) {
  return __uint_as_float((__float_as_uint(e) + 0x1000u) & 0xFFFFE000u);
}
// This thread's cp.async copies so far, as an arrival at the barrier when they have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A bf16 row of q as fp16: q4 of four columns each. Returns what the scores have to be
// multiplied by. All lanes of a row (4) call.
template <int KS>
__device__ __forceinline__ float to_half(uint2 (&q4)[KS]) {
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

// W columns of a finished row, O = 2^M sum over L. L = 0: no key, or only scores of
// -infinity (O is then 0, or NaN by 0 times a V that is NaN); no score but NaN leaves M
// alone and L NaN.
template <int W>
__device__ __forceinline__ void store_row(const Rows8Args& a, int token, int64_t head, int c0, const float (&sum)[W],
                                          float M, float L) {
  uint16_t* out = static_cast<uint16_t*>(a.out) + token * a.out_row + head * a.out_head + c0;
  const float inv = 1.0f / L;
  uint32_t w[W / 2];
#pragma unroll
  for (int i = 0; i < W; i += 2)
    w[i / 2] = L == 0.0f ? 0u
               : a.bf16  ? Elem<__nv_bfloat16>::pack(sum[i] * inv, sum[i + 1] * inv)
                         : Elem<__half>::pack(sum[i] * inv, sum[i + 1] * inv);
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  if (a.lse != nullptr && c0 == 0)
    a.lse[static_cast<int64_t>(token) * a.heads + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// All threads of the cluster's CTAs that have not ended; what they wrote before is seen.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of the cluster's CTA `rank`: the same place in its shared memory.
template <typename V>
__device__ __forceinline__ V remote(const V* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  if constexpr (sizeof(V) == 16) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
  } else {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
  }
}
template <typename V>
__device__ __forceinline__ V remote(const float* p, int rank) {
  return remote<V>(reinterpret_cast<const V*>(p), rank);
}

// The dense tiles of a slice, 32 at a time: tile i of the slice belongs to the token
// whose tiles end behind it. Tokens are looked at 32 at a time too, so that a slice of
// many short ones reads their metadata once per 32.
struct Tile8 {
  int t, kt, n;  // token, tile of the token, keys of the token
  int32_t page;
};
struct TileWindow {
  int t0, n, req, begin, end;  // the first token; of token t0 + lane: keys, request, its tiles within the slice

  // from token t on, whose first tile would be tile `at` of the slice
  __device__ __forceinline__ void open(const RowsArgs& a, int t, int at) {
    const int lane = threadIdx.x & 31;
    t0 = t;
    n = req = 0;
    int tiles = 0;
    if (t + lane < a.n_tokens) {
      n = token_keys(a, t + lane, &req, false);
      tiles = tiles_of(n);
    }
    end = tiles;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, end, i);
      if (lane >= i) end += v;
    }
    end += at;
    begin = end - tiles;
  }
  // lane i: tile `first` + i of the slice's `total`
  __device__ __forceinline__ Tile8 batch(const RowsArgs& a, int first, int total) {
    const int i = first + (threadIdx.x & 31);
    Tile8 d{0, 0, 0, -1};
    int of = 0;
    bool found = i >= total;
    while (true) {
      const int all = __shfl_sync(0xffffffffu, end, 31);
      int k = 0;  // the tokens that end before tile i
#pragma unroll
      for (int step = 16; step > 0; step /= 2)
        if (__shfl_sync(0xffffffffu, end, k + step - 1) <= i) k += step;
      const int b = __shfl_sync(0xffffffffu, begin, k), r = __shfl_sync(0xffffffffu, req, k);
      const int keys = __shfl_sync(0xffffffffu, n, k);
      if (!found && i < all) {
        found = true;
        d.t = t0 + k;
        d.kt = i - b;
        d.n = keys;
        of = r;
      }
      if (__all_sync(0xffffffffu, found) || t0 + 32 >= a.n_tokens) break;
      open(a, t0 + 32, all);
    }
    if (i < total && d.n > 0) d.page = a.block_table[static_cast<int64_t>(of) * a.bt_stride + d.kt];
    return d;
  }
};

// A window's slots (id[i] of lane l: place 32 i + l, -1 behind the list) into ids[], brought
// into 16 stretches of the cache from its lower to its upper end, if they lie in kApart
// bytes of K or more (page: a page's). One warp.
template <int TILES>
__device__ __forceinline__ bool order_slots(const int (&id)[2 * TILES], int tiles, int64_t page, int32_t* ids) {
  const int lane = threadIdx.x & 31;
  int lo = INT_MAX, hi = 0;
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i) {
    lo = min(lo, id[i] >= 0 ? id[i] : INT_MAX);
    hi = max(hi, id[i]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (hi <= lo || (hi - lo) / kBlock * page < kApart) return false;
  const int shift = max(0, 28 - __clz(hi - lo));  // (hi - lo) >> shift < 16
  auto stretch = [&](int x) { return x >= 0 ? (x - lo) >> shift : 15; };  // absent ones come last
  // lane b (and b + 16): the slots of stretch b so far; q: a slot's place in its stretch
  int count = 0, q[2 * TILES];
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i) {
    if (i >= 2 * tiles) break;
    const int b = stretch(id[i]);
    uint32_t m = 0xffffffffu;  // the lanes whose slot lies in stretch `lane % 16`
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = __ballot_sync(0xffffffffu, (b >> k) & 1);
      m &= (lane >> k) & 1 ? v : ~v;
    }
    q[i] = __shfl_sync(0xffffffffu, count, b) + __popc(__shfl_sync(0xffffffffu, m, b) & ((1u << lane) - 1u));
    count += __popc(m);
  }
  int first = count;  // of stretch `lane`, all stretches before it
#pragma unroll
  for (int k = 1; k < 16; k *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, first, k);
    if (lane >= k) first += v;
  }
  first -= count;
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i) {
    if (i >= 2 * tiles) break;
    ids[__shfl_sync(0xffffffffu, first, stretch(id[i])) + q[i]] = id[i];
  }
  __syncwarp();
  return true;
}

// The slots of a window of tiles, from place j of a token's list on, into ids[]: in order,
// or, of kOrderedTiles tiles or more that lie far apart, in the cache's. CTAs that begin
// together then go through the cache together, and what they read at a time lies in few of
// the memory's pages, whose translations they share. 64 tokens of 2048 slots, 64/8 heads of
// 128, from 64, 16 and 8 requests of 32K (2.1, 0.54 and 0.27 GB of K): 63.4, 58.6 and 57.7 us,
// in the list's order 70.1, 63.6 and 56.1; 512 tokens of one 369, 352. Windows of 8, 12 and 16
// tiles, in a run of their own: 65.7, 64.4 and 63.4, heads of 64 43.4, 43.1 and 46.4. Which keys
// make a tile changes by it, and so the sums' order, but not from run to run. The forms with q in
// shared memory have no room for such windows and read in the list's order. One warp.
template <int TILES>
__device__ __forceinline__ void place_slots(const int32_t* list, int j, int n, int tiles, int64_t page, int32_t* ids) {
  const int lane = threadIdx.x & 31;
  int id[2 * TILES];
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i)
    id[i] = i < 2 * tiles && j + i * 32 + lane < n ? list[j + i * 32 + lane] : -1;
  if constexpr (TILES >= kOrderedTiles)
    if (tiles >= kOrderedTiles && order_slots<TILES>(id, tiles, page, ids)) return;
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i)
    if (i < 2 * tiles) ids[i * 32 + lane] = id[i];
  __syncwarp();
}

template <int D, int HP, int NT, int LOAD>
__global__ void __launch_bounds__(kThreads8, Rows8Cfg<D, HP, NT, LOAD>::kCtas)
    attn_rows8_kernel(const __grid_constant__ Rows8Args a, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv) {
  using C = Rows8Cfg<D, HP, NT, LOAD>;
  using E = Elem<__half>;
  constexpr bool SEL = LOAD == kSlots;
  constexpr int S = C::kStages, I = C::kInfos, RB = C::kRowBytes;
  constexpr int CH = D / 16;  // 16-byte chunks of a head's codes: MMA k steps of q.k
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + I;
  uint64_t* scaled = SEL ? empty + I : full;  // slots: their places are used before their scales are there
  uint64_t* meeting = empty + 2 * I;          // of the consumers
  int4* meta = reinterpret_cast<int4*>(smem + C::kOffMeta);
  float2* scales = reinterpret_cast<float2*>(smem + C::kOffScale);
  Slice* slice = reinterpret_cast<Slice*>(smem + C::kOffScan);
  int* abort_flag = reinterpret_cast<int*>(smem + C::kOffScan) + 48;

  const int cluster = NT == 1 ? a.cluster : 1;
  const int place = blockIdx.x / cluster, rank = blockIdx.x - place * cluster;  // a token's CTAs side by side
  const int col = place / a.passes, pass = place - col * a.passes;
  // slice (split) or token, and the first of its KV heads
  const int part = col / (a.hkv / HP), h0 = (col - part * (a.hkv / HP)) * HP;

  if (threadIdx.x < I) {
    // lane 0 with the copies' bytes or the slots' places, and every lane's scales
    mbar_init(&full[threadIdx.x], SEL ? 1 : 33);
    if (SEL) mbar_init(&scaled[threadIdx.x], 32);
    mbar_init(&empty[threadIdx.x], kWarps);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    mbar_init(meeting, kWarps);
    fence_barrier_init();
    *abort_flag = 0;
  }
  // Launched while the stream's previous kernel drains: nothing is read before it has ended.
  pdl_wait();
  // ---- this CTA's slice
  if (a.split) {
    find_slice<SEL, kThreads8>(a, part, blockIdx.x == 0, slice, reinterpret_cast<int*>(slice + 1),
                               reinterpret_cast<int*>(smem));
    if (slice->left == 0) {  // fewer tiles than slices
      if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int2(-1, 0);
      return;
    }
    fence_async();  // its scratch lies where copies will
  } else if (threadIdx.x == 0) {
    int req = 0;
    slice->t = part;
    slice->n = SEL ? a.topk : token_keys(a, part, &req, h0 == 0 && pass == 0 && rank == 0);
    slice->req = req;
    const int tiles = tiles_of(slice->n);
    slice->kt = tiles * rank / cluster;  // (a cluster's tokens are short)
    slice->left = tiles * (rank + 1) / cluster - slice->kt;
  }
  __syncthreads();
  const int total = slice->left;

  if (warp == kWarps) {
    // ---- the loader: a tile's codes and scales into a stage, stage after stage. What it
    // has to know first comes in whole batches, so that no tile waits for it by itself:
    // dense: lane i has tile i of 32: its token, tile of the token, keys and page;
    // selected: the slots of a window of tiles
    TileWindow win;
    Tile8 mine;
    int32_t* ids = reinterpret_cast<int32_t*>(smem + C::kOffIds);
    int w = 0, wn = 0;  // tiles of the window: taken, in all
    const int each = SEL ? tiles_of(a.topk) : 0;  // a token's tiles
    int t = slice->t, kt = slice->kt;
    const int t1 = t, kt1 = kt, n1st = slice->n, left1st = tiles_of(n1st) - kt;  // the first token, its tiles here
    int32_t page1st = -1;
    if (!SEL && lane < left1st && n1st > 0)
      page1st = a.block_table[static_cast<int64_t>(slice->req) * a.bt_stride + kt + lane];
    bool fresh = true, opened = false;
    int stage = 0, phase = 1;  // of the I
#pragma unroll 1
    for (int it = 0; it < total; ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, abort_flag, a.err))) break;
      const uint32_t sdst = smem_u32(scales + stage * C::kScales);
      int n = a.topk, tiles = each;
      int32_t page = -1;
      if (!SEL) {
        if (it % 32 == 0) {
          if (it == 0 && (left1st >= 32 || left1st >= total)) {
            mine = Tile8{t1, kt1 + lane, n1st, page1st};
          } else {
            if (!opened) win.open(a, t1, -kt1);
            opened = true;
            mine = win.batch(a, it, total);
          }
        }
        t = __shfl_sync(0xffffffffu, mine.t, it % 32);
        kt = __shfl_sync(0xffffffffu, mine.kt, it % 32);
        n = __shfl_sync(0xffffffffu, mine.n, it % 32);
        page = __shfl_sync(0xffffffffu, mine.page, it % 32);
        tiles = tiles_of(n);
      }
      const bool ends = kt == tiles - 1, last = ends || it == total - 1;
      const int flags =
          (fresh ? kFirst : 0) | (last ? kLast : 0) | (kt == 0 ? kStartsItem : 0) | (ends ? kEndsItem : 0);
      const int more = (tiles - 1 - kt) << 4;
      if (SEL) {
        if (w == wn) {
          w = 0;
          wn = min(min(each - kt, total - it), it == 0 ? kFirstTiles : C::kWindow);
          place_slots<C::kWindow>(a.physical + static_cast<int64_t>(t) * a.topk, kt * kTile, a.topk, wn, a.k_page, ids);
        }
        const int32_t n0 = ids[w * kTile + lane], n1 = ids[w * kTile + 32 + lane];
        ++w;
        const bool in0 = n0 >= 0 && static_cast<int64_t>(n0) < a.num_slots;
        const bool in1 = n1 >= 0 && static_cast<int64_t>(n1) < a.num_slots;
        if ((n0 != -1 && !in0) || (n1 != -1 && !in1)) flag_error(a.err, DSA_DEVERR_ID_RANGE);
        const uint32_t lo = __ballot_sync(0xffffffffu, in0), hi = __ballot_sync(0xffffffffu, in1);
        longlong2* at = reinterpret_cast<longlong2*>(smem + C::kOffAt) + stage * kTile;  // K's and V's rows
        const uint32_t id0 = in0 ? n0 : 0, id1 = in1 ? n1 : 0;
        const uint32_t p0 = id0 / kBlock, s0 = id0 % kBlock, p1 = id1 / kBlock, s1 = id1 % kBlock;
        at[lane] = make_longlong2(p0 * a.k_page + s0 * a.k_slot, p0 * a.v_page + s0 * a.v_slot);
        at[lane + 32] = make_longlong2(p1 * a.k_page + s1 * a.k_slot, p1 * a.v_page + s1 * a.v_slot);
        __syncwarp();  // the rows' places are written
        if (lane == 0) {
          meta[stage] = make_int4(lo, hi, t, more | flags);
          mbar_arrive(&full[stage]);
        }
        // scales [block][head of the row][key of the block]
        const float* sp = a.scale + h0 * a.s_head;
        const float* sc0 = sp + p0 * a.s_page + s0 / kScaleBlock * a.s_block;
        const float* sc1 = sp + p1 * a.s_page + s1 / kScaleBlock * a.s_block;
        const uint32_t d0 = sdst + (lane / kScaleBlock * HP * kScaleBlock + lane % kScaleBlock) * 8;
#pragma unroll
        for (int z = 0; z < HP; ++z) {
          if (in0) cp8(d0 + z * kScaleBlock * 8, sc0 + z * a.s_head);
          if (in1) cp8(d0 + (2 * HP + z) * kScaleBlock * 8, sc1 + z * a.s_head);
        }
      } else {
        int have = max(0, min(kTile, n - kt * kTile));
        if (have > 0 && (page < 0 || static_cast<int64_t>(page) >= a.num_blocks)) {
          if (lane == 0) flag_error(a.err, DSA_DEVERR_BLOCK_RANGE);
          have = 0;
        }
        const int blocks = (have + kScaleBlock - 1) / kScaleBlock;
        if (lane == 0) {
          const uint32_t lo = have >= 32 ? 0xffffffffu : (1u << have) - 1u;
          const uint32_t hi = have >= 64 ? 0xffffffffu : have > 32 ? (1u << (have - 32)) - 1u : 0u;
          meta[stage] = make_int4(lo, hi, t, more | flags);
          mbar_arrive_expect_tx(&full[stage], blocks * 2 * kScaleBlock * RB);
        }
        __syncwarp();
        uint8_t* kdst = smem + stage * C::kStageBytes;
        uint8_t* vdst = kdst + kTile * RB;
        // lanes 0-3 a block of K each, 4-7 of V; lanes 0-4HP a block's and head's scales
        const int b = lane & 3;
        if (lane < 8 && b < blocks)
          tma_box_4d((lane < 4 ? kdst : vdst) + b * kScaleBlock * RB, lane < 4 ? &mk : &mv, &full[stage], 0, h0 / HP,
                      b * kScaleBlock, page);
        if (lane < 4 * HP && b < blocks)
          cp8(sdst + (b * HP + lane / 4) * kScaleBlock * 8,
              a.scale + page * a.s_page + b * a.s_block + (h0 + lane / 4) * a.s_head);
      }
      cp_arrive(&scaled[stage]);
      fresh = last;
      if (SEL) {
        if (++kt == each) {
          kt = 0;
          ++t;
        }
      }
      if (++stage == I) {
        stage = 0;
        phase ^= 1;
      }
    }
    cp_wait<0>();
    return;
  }

  // ---- the consumers: a warp has a block of 16 keys and HP heads; lane (g, c) of it keys
  // g, g + 8, query heads 2c, 2c + 1 of each eight, and columns 16y + 2g, 16y + 2g + 1 of O
  const int g = lane >> 2, c = lane & 3;
  const int head0 = pass * C::kRows;                // first query head of the group in this pass
  const int rows = min(C::kRows, a.group - head0);  // its query heads
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  float2* parts_ml = reinterpret_cast<float2*>(smem + C::kOffParts);
  int desc_token = -1, desc_last = 0;  // the slice ends inside a token that it began: which, and its last slice
  float o[HP][NT][CH][4];
  float m[HP][NT][2], l[HP][NT][2], lr[HP][NT][2], rf[HP][NT][2];  // lr: fp16: l of the rounded weights
  uint2 qf[HP][C::kKeptQ ? 1 : NT][CH];
  uint4* const kept = reinterpret_cast<uint4*>(smem + C::kOffQ) + threadIdx.x;
  bool starts = true;
  float least[HP];  // V's scales count as this at least
  const float NEG = -INFINITY;
  // where ldmatrix's rows lie in a stage; chunk k of them is at the address with k << 4 flipped
  const int krow = warp * kWarpKeys + (lane & 7) + ((lane >> 4) << 3);
  const uint32_t kaddr = smem_u32(smem) + krow * RB + swz<RB>(krow, (lane >> 3) & 1);
  const int vrow = warp * kWarpKeys + (lane & 7) + (((lane >> 3) & 1) << 3);
  const uint32_t vaddr = smem_u32(smem) + (kTile + vrow) * RB + swz<RB>(vrow, lane >> 4);
  // slots: the copies of this warp's rows of a tile, whose places the loader has left
  constexpr int RC = RB / 16, RPI = 32 / RC;  // 16-byte pieces of a row, rows that a copy of the warp covers
  const int ch = lane % RC, r0 = lane / RC;
  const uint8_t* kb = static_cast<const uint8_t*>(a.k) + h0 * a.k_head + ch * 16;
  const uint8_t* vb = static_cast<const uint8_t*>(a.v) + h0 * a.v_head + ch * 16;
  int info = 0, into = 0, next = 0, nphase = 0;  // of the tile at hand; of the next to be copied: stage, info
  auto issue = [&](bool in) {
    if (in) {
      const bool here = __all_sync(0xffffffffu, mbar_wait(&full[next], nphase, abort_flag, a.err));
      const int4 mt = meta[next];
      const uint32_t mask =
          here ? (static_cast<uint32_t>(warp < 2 ? mt.x : mt.y) >> (16 * (warp & 1))) & 0xffffu : 0u;
      const longlong2* at = reinterpret_cast<const longlong2*>(smem + C::kOffAt) + next * kTile + warp * kWarpKeys;
      const uint32_t dst = smem_u32(smem) + into * C::kStageBytes + warp * kWarpKeys * RB;
#pragma unroll
      for (int i = 0; i < kWarpKeys / RPI; ++i) {
        const int r = i * RPI + r0;
        if ((mask >> r) & 1) {
          const longlong2 o = at[r];
          const uint32_t d = dst + r * RB + swz<RB>(r, ch);
          cp16(d, kb + o.x, true);
          cp16(d + kTile * RB, vb + o.y, true);
        }
      }
      if (++into == S) into = 0;
      if (++next == I) {
        next = 0;
        nphase ^= 1;
      }
    }
    cp_commit();
  };
  if (SEL) {
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) issue(i < total);
  }
  // the consumers meet; a wait of theirs in vain is flagged, and all go on
  int mphase = 0;
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(meeting);
    mbar_wait(meeting, mphase, abort_flag, a.err);
    __syncwarp();
    mphase ^= 1;
  };
  int stage = 0, phase = 0;
#pragma unroll 1
  for (int it = 0; it < total; ++it) {
    if (SEL) {
      cp_wait<S - 2>();
      __syncwarp();
      issue(it + S - 1 < total);  // into the stage consumed in the previous step
    }
    // a wait in vain is flagged; the tile is left out and its rows are unspecified
    const bool here = __all_sync(0xffffffffu, mbar_wait(&scaled[info], phase, abort_flag, a.err));
    const int4 mt = here ? meta[info] : make_int4(0, 0, 0, 0);
    const uint32_t mask = (static_cast<uint32_t>(warp < 2 ? mt.x : mt.y) >> (16 * (warp & 1))) & 0xffffu;
    const int flags = mt.w & 15;

    if (flags & kFirst) {
      starts = flags & kStartsItem;
#pragma unroll
      for (int z = 0; z < HP; ++z) {
        least[z] = kLeastScale;
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + mt.z * a.q_row +
                            (static_cast<int64_t>(h0 + z) * a.group + head0) * a.q_head;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          m[z][x][0] = m[z][x][1] = NEG;
          l[z][x][0] = l[z][x][1] = lr[z][x][0] = lr[z][x][1] = 0.0f;
#pragma unroll
          for (int y = 0; y < CH; ++y) o[z][x][y][0] = o[z][x][y][1] = o[z][x][y][2] = o[z][x][y][3] = 0.0f;
          uint2(&q4)[CH] = qf[z][C::kKeptQ ? 0 : x];
          const bool in = x * 8 + g < rows;
          const uint16_t* qp = q + (in ? x * 8 + g : 0) * a.q_head + c * 4;
#pragma unroll
          for (int k = 0; k < CH; ++k) q4[k] = in ? *reinterpret_cast<const uint2*>(qp + k * 16) : make_uint2(0, 0);
          const float f = (a.bf16 ? to_half<CH>(q4) : 1.0f) * a.scale_log2;  // of row x * 8 + g
          rf[z][x][0] = __shfl_sync(0xffffffffu, f, 8 * c);
          rf[z][x][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
          if constexpr (C::kKeptQ) {
#pragma unroll
            for (int k = 0; k < CH; k += 2)
              kept[(x * (CH / 2) + k / 2) * kThreads] = make_uint4(q4[k].x, q4[k].y, q4[k + 1].x, q4[k + 1].y);
          }
        }
      }
    }

    if (mask != 0) {
      if (mask != 0xffffu) {
        // an absent key's V may be anything, NaN among it, and 0 * NaN is NaN
        const int r = lane & 15;
        if (!((mask >> r) & 1)) {
          uint4* row = reinterpret_cast<uint4*>(smem + stage * C::kStageBytes + (kTile + warp * kWarpKeys + r) * RB +
                                                (lane >> 4) * (RB / 2));
#pragma unroll
          for (int i = 0; i < RB / 32; ++i) row[i] = make_uint4(0, 0, 0, 0);
        }
        if (!SEL) fence_async();  // before the copies that follow into this stage
        __syncwarp();
      }
      // S^T = K q^T
      float s[HP][NT][4];
#pragma unroll
      for (int z = 0; z < HP; ++z)
#pragma unroll
        for (int x = 0; x < NT; ++x) s[z][x][0] = s[z][x][1] = s[z][x][2] = s[z][x][3] = 0.0f;
      {
        const uint32_t base = kaddr + stage * C::kStageBytes;
#pragma unroll
        for (int j = 0; j < HP * CH; j += 2) {
          const int z = j / CH, k = j % CH;
          uint32_t b[4];  // keys 0-7 chunks j, j + 1; keys 8-15 chunks j, j + 1
          ldsm4(b, base ^ (j << 4));
          uint4 q2[NT];  // chunks k and k + 1 of q
#pragma unroll
          for (int x = 0; x < NT; ++x)
            if constexpr (C::kKeptQ) {
              q2[x] = kept[(x * (CH / 2) + k / 2) * kThreads];
            } else {
              const uint2 q0 = qf[z][x][k], q1 = qf[z][x][k + 1];
              q2[x] = make_uint4(q0.x, q0.y, q1.x, q1.y);
            }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t f[4] = {half2_of(b[u]), half2_of(b[2 + u]), half2_of_high(b[u]), half2_of_high(b[2 + u])};
#pragma unroll
            for (int x = 0; x < NT; ++x) E::mma(s[z][x], f, u ? q2[x].z : q2[x].x, u ? q2[x].w : q2[x].y);
          }
        }
      }
      uint32_t p[HP][NT][2];
#pragma unroll
      for (int z = 0; z < HP; ++z) {
        // scores in powers of two with V's scale in them; absent keys out
        const float2* sc = scales + info * C::kScales + (warp * HP + z) * kScaleBlock + (SEL ? g : 0);
        const float2 s0 = sc[0], s1 = SEL ? sc[8] : s0;
        const float v0 = fminf(fmaxf(s0.y, least[z]), kMostScale), v1 = fminf(fmaxf(s1.y, least[z]), kMostScale);
        float lv0 = lg2(v0), lv1 = lg2(v1);
        float iv0 = rcp(v0), iv1 = rcp(v1);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          float(&w)[4] = s[z][x];
          w[0] = fmaf(w[0], rf[z][x][0] * s0.x, lv0);
          w[1] = fmaf(w[1], rf[z][x][1] * s0.x, lv0);
          w[2] = fmaf(w[2], rf[z][x][0] * s1.x, lv1);
          w[3] = fmaf(w[3], rf[z][x][1] * s1.x, lv1);
          if (mask != 0xffffu) {
            if (!((mask >> g) & 1)) w[0] = w[1] = NEG;
            if (!((mask >> (g + 8)) & 1)) w[2] = w[3] = NEG;
          }
          float t0 = fmaxf(w[0], w[2]), t1 = fmaxf(w[1], w[3]);
          float(&mm)[2] = m[z][x];
          const bool move = t0 > mm[0] + (E::kHead + kSlack) || t1 > mm[1] + (E::kHead + kSlack);
          if (__any_sync(0xffffffffu, move)) {
            float top = v0;  // the largest scale of the warp's keys
            if constexpr (SEL) {
              top = fmaxf((mask >> g) & 1 ? v0 : 0.0f, (mask >> (g + 8)) & 1 ? v1 : 0.0f);
              top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            }
            if (top * kSpread > least[z]) {
              least[z] = top * kSpread;
              if constexpr (SEL) {  // (pages: they have one scale)
                const float a0 = fmaxf(v0, least[z]), a1 = fmaxf(v1, least[z]), b0 = lg2(a0), b1 = lg2(a1);
                w[0] += b0 - lv0;
                w[1] += b0 - lv0;
                w[2] += b1 - lv1;
                w[3] += b1 - lv1;
                t0 = fmaxf(w[0], w[2]);
                t1 = fmaxf(w[1], w[3]);
                lv0 = b0;
                lv1 = b1;
                iv0 = rcp(a0);
                iv1 = rcp(a1);
              }
            }
#pragma unroll
            for (int i = 4; i < 32; i *= 2) {
              t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, i));
              t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, i));
            }
            const float n0 = fmaxf(mm[0], t0 - E::kHead), n1 = fmaxf(mm[1], t1 - E::kHead);
            const float g0 = mm[0] == NEG ? 0.0f : half_way(mm[0] - n0), g1 = mm[1] == NEG ? 0.0f : half_way(mm[1] - n1);
            const float f0 = g0 * g0, f1 = g1 * g1;
            mm[0] = n0;
            mm[1] = n1;
            l[z][x][0] = l[z][x][0] * g0 * g0;
            l[z][x][1] = l[z][x][1] * g1 * g1;
            lr[z][x][0] *= f0;
            lr[z][x][1] *= f1;
#pragma unroll
            for (int y = 0; y < CH; ++y) {
              o[z][x][y][0] *= f0;
              o[z][x][y][1] *= f1;
              o[z][x][y][2] *= f0;
              o[z][x][y][3] *= f1;
            }
          }
          const float m0 = mm[0] == NEG ? 0.0f : mm[0], m1 = mm[1] == NEG ? 0.0f : mm[1];
          const float e0 = ex2(w[0] - m0), e1 = ex2(w[1] - m1), e2 = ex2(w[2] - m0), e3 = ex2(w[3] - m1);
          l[z][x][0] = fmaf(e0, iv0, fmaf(e2, iv1, l[z][x][0]));
          l[z][x][1] = fmaf(e1, iv0, fmaf(e3, iv1, l[z][x][1]));
          const uint32_t p0 = E::pack(e0, e1), p1 = E::pack(e2, e3);
          if (!a.bf16) {
            lr[z][x][0] = fmaf(to_11_bits(e0), iv0, fmaf(to_11_bits(e2), iv1, lr[z][x][0]));
            lr[z][x][1] = fmaf(to_11_bits(e1), iv0, fmaf(to_11_bits(e3), iv1, lr[z][x][1]));
          }
          p[z][x][0] = transpose8(p0);
          p[z][x][1] = transpose8(p1);
        }
      }
      // O^T += V^T P^T
      {
        const uint32_t base = vaddr + stage * C::kStageBytes;
#pragma unroll
        for (int j = 0; j < HP * CH; j += 2) {
          const int z = j / CH, y = j % CH;
          uint32_t b[4];  // chunk j: keys 0-7, 8-15; chunk j + 1: keys 0-7, 8-15
          ldsm4_t(b, base ^ (j << 4));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            // codes (key 2c: even, odd column; key 2c + 1: even, odd) -> a column's two keys
            const uint32_t w0 = __byte_perm(b[2 * u], 0, 0x3120), w1 = __byte_perm(b[2 * u + 1], 0, 0x3120);
            const uint32_t f[4] = {half2_of(w0), half2_of_high(w0), half2_of(w1), half2_of_high(w1)};
#pragma unroll
            for (int x = 0; x < NT; ++x) E::mma(o[z][x][y + u], f, p[z][x][0], p[z][x][1]);
          }
        }
      }
    }

    if (flags & kLast) {
      // ---- the partial results of the warps that share a head into one: each leaves its
      // O, eight query heads at a time, in the stage that has just been read; then 16
      // threads a row add them
      const bool whole = starts && (flags & kEndsItem);
      float* parts = reinterpret_cast<float*>(smem + (stage + 1) % S * C::kStageBytes);
      const int r8 = threadIdx.x / 16;                                  // row of the eight
      constexpr int W = D / 16;                                         // columns of a thread
      const int at = r8 * D + ((threadIdx.x % 16 * W) ^ (r8 / 2 * 8));  // where they lie in eight rows of O
      float* os = reinterpret_cast<float*>(smem + stage * C::kStageBytes);
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        meet();  // all have read the stage, or the rows before
#pragma unroll
        for (int z = 0; z < HP; ++z) {
          float even[2] = {1.0f, 1.0f};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float sum = l[z][x][e], rounded = lr[z][x][e];
#pragma unroll
            for (int i = 4; i < 32; i *= 2) {
              sum += __shfl_xor_sync(0xffffffffu, sum, i);
              rounded += __shfl_xor_sync(0xffffffffu, rounded, i);
            }
            if (g == 0) ml[(warp * HP + z) * C::kRows + x * 8 + 2 * c + e] = make_float2(m[z][x][e], sum);
            // fp16: O is divided by the sum of the weights that made it, so that a row with few
            // keys has not their rounding and the result's (2 requests of 53 to 167 keys: 1.47 times
            // the error of 32-bit arithmetic, so 1.1); that sum is finite and as near where all is well
            if (!a.bf16 && fabsf(rounded - sum) <= 0x1p-10f * sum && sum > 0.0f) even[e] = sum / rounded;
          }
          float* mine = os + (warp * HP + z) * 8 * D;
#pragma unroll
          for (int y = 0; y < CH; ++y)
#pragma unroll
            for (int e = 0; e < 2; ++e)  // columns moved by eights: four rows' stores on 32 banks
              *reinterpret_cast<float2*>(mine + (2 * c + e) * D + ((y * 16 + 2 * g) ^ (c * 8))) =
                  make_float2(o[z][x][y][e] * even[e], o[z][x][y][2 + e] * even[e]);
        }
        meet();
        const int r = x * 8 + r8;
        if (r < rows) {
#pragma unroll
          for (int z = 0; z < HP; ++z) {
            float M = NEG, L = 0.0f, sum[W];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[(w * HP + z) * C::kRows + r].x);
            const float Ms = M == NEG ? 0.0f : M;
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float2 v = ml[(w * HP + z) * C::kRows + r];
              const float half = half_way(v.x - Ms), f = half * half;
              const float* p = os + (w * HP + z) * 8 * D + at;
              L = fmaf(v.y * half, half, L);
#pragma unroll
              for (int i = 0; i < W; i += 4) {
                const float4 u = *reinterpret_cast<const float4*>(p + i);
                sum[i] = fmaf(u.x, f, sum[i]);
                sum[i + 1] = fmaf(u.y, f, sum[i + 1]);
                sum[i + 2] = fmaf(u.z, f, sum[i + 2]);
                sum[i + 3] = fmaf(u.w, f, sum[i + 3]);
              }
            }
            const int c0 = threadIdx.x % 16 * W;
            if (NT == 1 && cluster > 1) {
              // for the cluster's CTAs to read: in the next stage, which no copy is left for
              float* px = parts + (z * C::kRows + r) * D + c0;
#pragma unroll
              for (int i = 0; i < W; i += 4)
                *reinterpret_cast<float4*>(px + i) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
              if (c0 == 0) parts_ml[z * C::kRows + r] = make_float2(M, L);
            } else if (whole) {
              store_row<W>(a, mt.z, static_cast<int64_t>(h0 + z) * a.group + head0 + r, c0, sum, M, L);
            } else {
              // slot 2c: a part that continues an earlier CTA's item; 2c + 1: the beginning of one
              const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0)) * HP + z;
              float* po = a.part_o + (slot * C::kRows + r) * D + c0;
#pragma unroll
              for (int i = 0; i < W; i += 4)
                *reinterpret_cast<float4*>(po + i) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
              if (c0 == 0) a.part_ml[slot * C::kRows + r] = make_float2(M, L);
            }
          }
        }
      }
      if (SEL)
        meet();  // all have read it, before the copies that follow into this stage
      else
        fence_async();
      if (a.split && !whole && starts) {  // it began here and goes on: so many tiles after this one, in the next slices
        desc_token = mt.z;
        const int64_t end = slice->end + (mt.w >> 4);
        desc_last = static_cast<int>((end * slice->in_use + slice->all - 1) / slice->all) - 1;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[info]);
    if (++stage == S) stage = 0;
    if (++info == I) {
      info = 0;
      phase ^= 1;
    }
  }
  if (SEL) cp_wait<0>();
  if (*static_cast<volatile int*>(abort_flag)) {
    // a wait gave up: copies in flight land in this CTA's memory, so they get their time again
    const unsigned long long t0 = global_ns();
    for (int s = 0; s < I && s < total; ++s)
      while (!mbar_try_wait(smem_u32(&scaled[s]), ((total - 1 - s) / I) & 1) && global_ns() - t0 < kWaitLimitNs) {
      }
  }
  if (a.split && threadIdx.x == 0) a.desc[blockIdx.x] = make_int2(desc_token, desc_last);
  if (NT > 1 || cluster == 1) return;
  // ---- a cluster's CTAs have a token's keys in turn: its rows are shared out, and each
  // CTA adds its rows' parts out of the others' shared memory
  if (total == 0 && threadIdx.x < HP * C::kRows) parts_ml[threadIdx.x] = make_float2(NEG, 0.0f);  // no keys, no part
  cluster_sync();
  constexpr int W = D / 16;
  const int c0 = threadIdx.x % 16 * W, tiles = tiles_of(slice->n);
  for (int i = (threadIdx.x / 16) * cluster + rank; i < HP * rows; i += kThreads / 16 * cluster) {
    const int z = i / rows, row = z * C::kRows + i - z * rows;
    float M = NEG, L = 0.0f, sum[W];
    float2 v[kMostCluster];
#pragma unroll
    for (int k = 0; k < kMostCluster; ++k) {
      v[k] = k < cluster ? remote<float2>(parts_ml + row, k) : make_float2(NEG, 0.0f);
      M = fmaxf(M, v[k].x);
    }
    const float ref = M == NEG ? 0.0f : M;
#pragma unroll
    for (int j = 0; j < W; ++j) sum[j] = 0.0f;
#pragma unroll
    for (int k0 = 0; k0 < kMostCluster; k0 += 4) {
      if (k0 >= cluster) break;
      float4 u[4][W / 4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // the stage that a CTA's parts lie in is behind its last tile's
        const int left = tiles * (k0 + k + 1) / cluster - tiles * (k0 + k) / cluster;
        const float* px = reinterpret_cast<const float*>(smem + left % S * C::kStageBytes) + row * D + c0;
#pragma unroll
        for (int j = 0; j < W / 4; ++j)
          u[k][j] = k0 + k < cluster && left > 0 ? remote<float4>(px + 4 * j, k0 + k) : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float half = half_way(v[k0 + k].x - ref), e = half * half;
        L = fmaf(v[k0 + k].y * half, half, L);
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          sum[4 * j] = fmaf(u[k][j].x, e, sum[4 * j]);
          sum[4 * j + 1] = fmaf(u[k][j].y, e, sum[4 * j + 1]);
          sum[4 * j + 2] = fmaf(u[k][j].z, e, sum[4 * j + 2]);
          sum[4 * j + 3] = fmaf(u[k][j].w, e, sum[4 * j + 3]);
        }
      }
    }
    store_row<W>(a, part, static_cast<int64_t>(h0 + z) * a.group + head0 + i - z * rows, c0, sum, M, L);
  }
  cluster_sync();  // all have read this CTA's
}

template <int D, int HP, int NT, int LOAD>
cudaError_t launch(const Rows8Args& a, int grid, const CUtensorMap* maps, cudaStream_t stream) {
  static uint64_t done = 0;
  using C = Rows8Cfg<D, HP, NT, LOAD>;
  auto* fn = attn_rows8_kernel<D, HP, NT, LOAD>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(fn), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  if (a.cluster > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads8);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, a, maps[0], maps[1]);
  }
  e = launch_pdl(fn, dim3(grid), dim3(kThreads8), C::kSmemBytes, stream, a, maps[0], maps[1]);
  if (e != cudaSuccess || !a.split) return e;
  // the next kernel is not let in while the join runs: its CTAs would take places
  // where one of this kernel's three would have to go (8 x 128K keys: 321 us, so 315)
  return launch_attn_join8(a, D, a.bf16, C::kRows, stream);
}

template <int D, int HP, int LOAD>
cudaError_t launch_rows(const Rows8Args& a, int grid, const CUtensorMap* maps, cudaStream_t stream) {
  return rows8_of(a.group) == 8 ? launch<D, HP, 1, LOAD>(a, grid, maps, stream)
                                : launch<D, HP, 2, LOAD>(a, grid, maps, stream);
}

}  // namespace

cudaError_t launch_attn_rows8(const Rows8Args& a, int head_dim, bool selected, const CUtensorMap* maps,
                              cudaStream_t stream) {
  const int grid = a.slices * (a.hkv / a.joint) * a.passes * a.cluster;
  if (!selected) {
    if (head_dim == 128) return launch_rows<128, 1, kPages>(a, grid, maps, stream);
    return a.pairs ? launch_rows<64, 2, kPages>(a, grid, maps, stream)
                   : launch_rows<64, 1, kPages>(a, grid, maps, stream);
  }
  if (head_dim == 128) return launch_rows<128, 1, kSlots>(a, grid, maps, stream);
  return a.pairs ? launch_rows<64, 2, kSlots>(a, grid, maps, stream)
                 : launch_rows<64, 1, kSlots>(a, grid, maps, stream);
}

}  // namespace dsa
