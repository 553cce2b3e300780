// DCA decode over a paged 4-bit cache (kv4.cuh): one new query per sequence.
//
// Mathematics.  With key j stored as khat = c * scale + offset per group g,
//     S_j = sum_g scale_jg <q_g, c_jg> + offset_jg * sum(q_g),
// so the matrix product runs on the bare codes and a key costs one FMA pair a
// group and head instead of a conversion an element.  The codes 0 .. 15 are
// exact as fp16 SUBNORMALS: a nibble masked into the low mantissa bits of each
// half of a word is c * 2^-24 (bits 4-7: 16 c * 2^-24, undone by a query
// pre-scaled by 1/16), so eight codes cost four logic operations and a shift.
// q, scaled per head by a power of two to below 2^11, is kept as its nearest
// integers and the fp16 remainders: 22 bits and more of the head's largest.  The
// products of the integers are integers below 2^21, so their sum is exact; those
// of the remainders are summed apart.  (Rounded to fp16 and summed as one, the
// sums, whose codes are not centred, lost up to 1e-5 of a score to the tensor
// core's truncation.)  For the values,
//     O = sum_j (p_j scale_j) c_j + sum_j p_j offset_j,
// again on the bare codes, with p_j scale_j rounded to fp16 after a
// normalisation by the largest scale of the 64-key tile (a power of two), so
// that scales of any size from 2^-113 on fit; the second sum stays in fp32 outside
// the matrix product.  A tile's product is formed from zero and then added to O in
// fp32: the codes are not centred, so a long sum inside the tensor core, which
// truncates, would drift by more than the result can bear.
//
// Kernel 1, a CTA per share of the tiles of all (sequence, kv head, group of <= 8
// query heads): four warps take its 64-key tiles in turn, each fetching its own
// (K part and V part, 36 * D contiguous bytes each, one bulk copy) through a small
// ring, so that the running maximum, its shuffles and the update of O are paid
// once per 64 keys of a warp.  The tiles are shared out evenly on the device from
// t[b], whatever the caches' capacity.  Kernel 2 merges the shares.  Where the
// caches are short a CTA takes a (sequence, kv head, group) whole and there is no
// second kernel.
//
// What bounds it.  A key costs 144 bytes of cache a kv head (D = 128) and, with
// eight query heads on it, about 18 instructions a warp (1148 for 64 keys, 96 of
// them matrix products, half of the rest unpacking nibbles).  With one query
// head memory bounds it: 24 sequences of 16k keys, 32 kv heads, take 317 us, 5.6
// TB/s, 85 % of the copy rate.  With eight no pipe is full: 16 sequences of 33k to
// 65k keys, 8 kv heads, take 203 to 206 us at 1965 MHz, 4.4 TB/s, the logic pipe
// busy for 51 % and the matrix pipe for 37 % of it, an instruction issued in 0.55 of
// the cycles; at 2.7 warps a scheduler the latency between dependent instructions
// is what remains.  (One call after another takes 222 us: the power cap then holds
// the clock near 1760 MHz.)  One sequence of 100k keys takes 38 us in a graph, 43
// with a cold cache, against 17.6 of bytes: about 9 us pass before the first and
// after the last tile, and seven or eight tiles a warp follow.
#include <atomic>

#include "dca_common.cuh"
#include "dca_index.cuh"
#include "dca_kernels.cuh"
#include "kv4.cuh"

namespace dca {
namespace kv4 {

constexpr int kHeads = 8;   // query heads per CTA (MMA N)
// Three CTAs of four warps an SM, a ring of three half tiles (K or V part) a
// warp, caches cold: 64.5 us for 24 x 4k keys of 32 kv heads, 44 for 1 x 100k and 206
// for 16 x 64k of 8.  Two CTAs with rings of four take 66.5, 44 and 208, two of six
// warps 68, 48 and 218, one of twelve 101, 48 and 241.  The 168 registers that this
// leaves a thread make the compiler spill at D = 128: 100 bytes a thread with
// eight query heads a kv head (20 with at most four), 284 (64) in the form that
// takes units whole.
constexpr int kWarps = 4;
constexpr int kRing = 3;
constexpr int kCtasPerSm = 3;
constexpr int kMany = 2;    // 16-key steps whose score products run interleaved: with one, 46 and
                            // 210 us for the last two of those
constexpr int kMaxTiles = 512;  // of a CTA's share, so that their places fit in shared memory

// Work.  A unit is a (sequence, kv head, group of <= 8 query heads).  The tiles
// of all units, one unit after another, are cut into equal shares, a CTA each,
// so neither unequal sequences nor few of them leave SMs idle.  Every unit
// counts kSetup tiles besides its own, before them, for what it costs to begin
// one (rotating the queries, the first fetch, the merge).  A share may hold the
// end of one unit and the beginning of the next; each piece gives a partial
// result.  Share c of unit U writes slot U + c: along the line of tiles each new
// piece raises one of the two, so no slot is used twice.  Over 22 batches of 1 to
// 40 sequences of 1k to 30k keys, a setup of 6, 8, 9, 10 and 12 tiles differed by
// at most 1.4 % in the mean, 8 the fastest.
constexpr int kSetup = 8;
// Where the caches are short, a unit is not cut: a CTA takes it whole, writes its
// outputs, and there is nothing to merge.  In a graph, against equal shares, 8 query
// heads a unit:
//     keys      8 units        32             63             128            512
//      250   7.7 /  9.6    7.9 / 10.2    8.1 / 12.3    8.5 / 15.0   20.4 / 29.6 us
//      500   8.5 /  9.9    8.6 / 10.5    8.6 / 12.8    8.9 / 17.1   24.9 / 33.7
//     1000  11.2 / 10.1   11.5 / 11.9   11.4 / 15.9   11.6 / 20.6   35.4 / 42.5
//     2000       -              -        16.1 / 19.0  16.3 / 24.4   57.9 / 58.7
//     3000       -              -        21.2 / 20.6  21.5 / 28.9   79.2 / 73.6
// (63 units: 64 from 2000 keys on.)  Below 48 units shares are faster from 750 keys
// on, by 1.5 us at most up to 1024 rows; but one launch fewer saves 2.6 us of the
// host's time at every count of units (15.7 against 18.4 us a call), which is what
// so short a call waits for outside a graph.  The choice goes by the table's width,
// which the host knows, not by the lengths, which lie on the device: a short
// sequence in a wide table takes the shares' time.
constexpr int kWide = 8;  // warps of such a CTA where every unit has an SM to itself: 148 units of
                          // 1000 keys take 11.6 us, 13.2 with twelve, 15.2 with four
constexpr long long kWholeUnits = 0x7FFFFFFF;  // the launch grid
inline bool takes_whole(long long units, long long cap) {  // cap: rows of a cache
  return units <= kWholeUnits && cap <= (units < 64 ? 1024 : 2048);
}
struct Split {
  long long shares, each, extra;  // the first `extra` shares hold one tile more
};
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (unsigned)a / (unsigned)b : a / b;
}
__device__ __forceinline__ Split make_split(long long tiles, long long shares) {
  Split sp;
  sp.shares = shares;
  sp.each = quotient(tiles, shares);
  sp.extra = tiles - sp.each * shares;
  return sp;
}
__device__ __forceinline__ long long share_begin(const Split& sp, long long c) {
  return c * sp.each + (c < sp.extra ? c : sp.extra);
}
// The share that holds tile g.
__device__ __forceinline__ long long share_of(const Split& sp, long long g) {
  const long long most = sp.extra * (sp.each + 1);
  return g < most ? quotient(g, sp.each + 1) : sp.extra + quotient(g - most, sp.each);
}
inline int head_groups(int Hq, int Hkv) { return (Hq / Hkv + kHeads - 1) / kHeads; }
// Shares of `tiles` tiles: one for every four (a tile a warp), at most `most`.
__host__ __device__ inline long long share_count(long long tiles, long long most) {
  const long long n = tiles / kWarps < most ? tiles / kWarps : most;
  return n > 0 ? n : 1;
}
// Shares of a call whose caches are full (the grid): at most all SMs once, or
// more where a share would pass kMaxTiles.
inline long long decode_shares(int B, int Hq, int Hkv, long long cap) {
  const long long tiles = (long long)B * Hkv * head_groups(Hq, Hkv) *
                          ((cap + kTileKeys - 1) / kTileKeys + kSetup);
  const long long need = (tiles + kMaxTiles - 1) / kMaxTiles;
  return share_count(tiles, need > 148 * kCtasPerSm ? need : 148 * kCtasPerSm);
}

template <int D, int W>
struct DecodeSmem {
  static constexpr int kHalf = Tile<D>::kBytes / 2;
  static constexpr int kRings = W * kRing * kHalf;
  // [piece][hi, lo][group][head][word] x 16 bytes of query fragments
  static constexpr int kQ = 3 * 2 * (D / 64) * kHeads * 8 * 16;
  static constexpr int kCs = 3 * (D / 2) * 8;          // cos, sin
  static constexpr int kRaw = kHeads * D * 2;          // queries as they came
  static constexpr int kSums = 3 * kHeads * (D / 64) * 4;  // sum of q per group
  static constexpr int kF = 2 * kHeads * 4;  // power of two of a head's scores, in two parts
  static constexpr int kBars = W * kRing * 8 + 16;  // + abort and page words
  static constexpr int kPlaces = kMaxTiles * 4;  // pool tile of every tile of the share
  static constexpr int kTotal = kRings + kQ + kRaw + kCs + kSums + kF + kBars + kPlaces;
  static_assert(W * kHeads * (D + 2) * 4 <= kRings, "merge area");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// m16n8k16 on fp16, fp32 accumulate; volatile, which keeps the products in the
// order written (two independent ones in turn): left to itself the compiler
// gathers all loads of a tile first and spills.
__device__ __forceinline__ void mma_codes(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum (C = 0).
__device__ __forceinline__ void mma_codes_first(float (&d)[4], const uint32_t (&a)[4],
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Greater of either bf16 half (NaN only against NaN).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

constexpr float kMostF = 1.7014118346046923e38f;  // 2^127
// 2^e for e > -127; infinite above 127.
__device__ __forceinline__ float power2(int e) {
  return __uint_as_float((unsigned)min(e + 127, 255) << 23);
}

__device__ __forceinline__ int tiles_of(int t, long long cap) {
  return t >= 0 && t < cap ? t / kTileKeys + 1 : 0;
}
// The same with its setup, on the line of shares; 0 for a bad position.
__device__ __forceinline__ int span_of(int t, long long cap) {
  const int n = tiles_of(t, cap);
  return n ? n + kSetup : 0;
}
// Spans of sequences 0 .. n-1 (units of one sequence counted once), by the block.
__device__ __forceinline__ long long spans_before(const int* t, int n, long long cap,
                                                  long long* sums) {
  long long x = 0;
  for (int b = threadIdx.x; b < n; b += blockDim.x) x += span_of(__ldg(t + b), cap);
#pragma unroll
  for (int sh = 16; sh >= 1; sh >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, sh);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) x += sums[w];
  return x;
}

// O += weights * values of group gr over a 64-key tile: wgt holds the MMA columns
// of each 16-key step.  With one head a lane (kOwn = 1) its groups are the two
// columns, of which this group's is taken.
template <int D, int kOut>
__device__ __forceinline__ void pv(float (&o)[D / 16][kOut], const uint32_t (&wgt)[4][2],
                                   const uint8_t* tile, int gr, int g, int t4, float down) {
  using TL = Tile<D>;
  float acc[4][4];
#pragma unroll
  for (int sub = 0; sub < 4; ++sub) {
    // word g of the group for keys 4 t4 .. 4 t4 + 3: MMA k rows 2 t4, 2 t4 + 1 and
    // 2 t4 + 8, 2 t4 + 9
    const uint4 v = *reinterpret_cast<const uint4*>(
        tile + TL::v_word(0, 0, 0) + (((sub * TL::kGroups + gr) * 8 + g) * 16 + 4 * t4) * 4);
#pragma unroll
    for (int m = 0; m < 4; ++m) {  // dims 2m (rows g) and 2m + 1 (rows g + 8)
      const uint32_t sel = m | ((4 + m) << 8);  // byte m of either word, 16 bits apart
      const uint32_t ra = __byte_perm(v.x, v.y, sel), rb = __byte_perm(v.z, v.w, sel);
      const uint32_t a[4] = {ra & 0x000F000Fu, ra & 0x00F000F0u, rb & 0x000F000Fu,
                             rb & 0x00F000F0u};
      if (sub == 0) mma_codes_first(acc[m], a, wgt[sub][0], wgt[sub][1]);
      else mma_codes(acc[m], a, wgt[sub][0], wgt[sub][1]);
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float* out = o[gr * 4 + m];
    if (kOut == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = fmaf(acc[m][e], down, out[e]);
    } else {
      out[0] = fmaf(acc[m][gr], down, out[0]);
      out[1] = fmaf(acc[m][2 + gr], down, out[1]);
    }
  }
}

// kFew: at most four query heads a kv head.  Eight MMA columns then hold both
// parts of every query, half the score products: 64.5 us for 24 x 4k keys of 32 kv
// heads with a query head each, against 77 as eight columns of high parts.
template <int D, bool kFew, int W, bool kWhole>
__global__ void __launch_bounds__(W * 32, W == kWarps ? kCtasPerSm : 1) decode_kernel(
    const __nv_bfloat16* __restrict__ q, Pages pg, const int* __restrict__ t,
    float* __restrict__ Opart, float2* __restrict__ MLpart, __nv_bfloat16* __restrict__ O,
    float* __restrict__ LSE, int B, int Hq, int s, int c, float scale_log2, int n_hg,
    const __grid_constant__ Theta theta) {
  using TL = Tile<D>;
  using SM = DecodeSmem<D, W>;
  constexpr int kThreads = W * 32;
  constexpr int kGr = TL::kGroups, kOwn = kFew ? 1 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long sums[W];
  uint8_t* qf = smem + SM::kRings;
  __nv_bfloat16* qraw = reinterpret_cast<__nv_bfloat16*>(qf + SM::kQ);
  float2* cs = reinterpret_cast<float2*>(qf + SM::kQ + SM::kRaw);
  float* qsum = reinterpret_cast<float*>(qf + SM::kQ + SM::kRaw + SM::kCs);  // [piece][head][group]
  float* qexp = qsum + 3 * kHeads * kGr;                          // [2][head]
  uint8_t* bars = reinterpret_cast<uint8_t*>(qexp + 2 * kHeads);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + W * kRing * 8);
  volatile int* bad_pages = abort_flag + 1;  // [2], of this piece and of the next
  uint32_t* places = reinterpret_cast<uint32_t*>(bars + SM::kBars);

  cudaTriggerProgrammaticLaunchCompletion();  // the merge may take its places
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = Hq / pg.Hkv, per_seq = pg.Hkv * n_hg;
  const int tpb = pg.block_rows / kTileKeys;
  const long long cap = (long long)pg.max_blocks * pg.block_rows;
  if (tid == 0) {
    *abort_flag = 0;
    bad_pages[0] = bad_pages[1] = 0;
    for (int i = 0; i < W * kRing; ++i) mbar_init(smem_u32(bars) + 8 * i, 1);
    fence_barrier_init();
  }
  for (int i = tid; i < SM::kQ / 16; i += kThreads)  // heads a unit does not have
    reinterpret_cast<uint4*>(qf)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < 3 * kHeads * kGr + 2 * kHeads; i += kThreads) qsum[i] = 0.f;
  // spans of 32 sequences, and those of the ones up to the lane's
  long long mine, sum;
  auto scan = [&](int first) {
    mine = first + lane < B ? (long long)span_of(__ldg(t + first + lane), cap) * per_seq : 0;
    sum = mine;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, sh);
      if (lane >= sh) sum += y;
    }
  };
  long long at, end, b_at = 0;  // the share, and where its first sequence begins
  int b = 0;
  if (kWhole) {
    // a unit a CTA, as if its sequence were alone
    b = blockIdx.x / per_seq;
    const int u = blockIdx.x % per_seq, span = span_of(__ldg(t + b), cap);
    at = (long long)u * span;
    end = at + span;
    if (span == 0) {  // a position outside the cache: reported, NaN
      if (tid == 0 && u == 0) report_error(kDevBadArg, 207);
      const int h0 = u / n_hg * G + u % n_hg * kHeads;
      const int h1 = min(h0 + kHeads, u / n_hg * G + G);
      for (int x = h0 * D + tid; x < h1 * D; x += kThreads)
        O[(size_t)b * Hq * D + x] = __ushort_as_bfloat16(0x7FC0);
      if (tid < h1 - h0) LSE[(size_t)b * Hq + h0 + tid] = __int_as_float(0x7fc00000);
    }
  } else {
    scan(0);
    const long long all = B <= 32 ? __shfl_sync(0xFFFFFFFFu, sum, 31)
                                  : spans_before(t, B, cap, sums) * per_seq;
    const Split split = make_split(all, share_count(all, gridDim.x));
    if (blockIdx.x == 0) {  // positions outside the cache: reported, no work
      for (int k = tid; k < B; k += kThreads)
        if (tiles_of(__ldg(t + k), cap) == 0) report_error(kDevBadArg, 207);
    }
    if (blockIdx.x >= split.shares || all == 0) return;
    at = share_begin(split, blockIdx.x);
    end = share_begin(split, blockIdx.x + 1);
    for (;;) {  // every warp looks for the sequence at the share's begin
      const unsigned past = __ballot_sync(0xFFFFFFFFu, at < b_at + sum);
      if (past) {
        const int k = __ffs(past) - 1;
        b_at += __shfl_sync(0xFFFFFFFFu, sum - mine, k);
        b += k;
        break;
      }
      b_at += __shfl_sync(0xFFFFFFFFu, sum, 31);
      b += 32;
      if (b >= B) return;  // t has changed meanwhile
      scan(b);
    }
  }
  // This warp's ring: the K and V parts of its tiles pass in turn through its
  // buffers; a part is fetched as soon as the one kRing before it is read.
  const uint8_t* ring = smem + warp * kRing * SM::kHalf;
  const uint32_t full0 = smem_u32(bars) + warp * kRing * 8;
  int buf = 0, phase = 0;
  int turned = -1, turns = 0;  // the sequence whose rotations cs holds, and for which DCA pieces

  for (int piece = 0; at < end; ++piece) {
  volatile int* bad_page = bad_pages + (piece & 1);
  const int tb = __ldg(t + b), all_tiles = tiles_of(tb, cap), span = all_tiles + kSetup;
  const int unit = (int)quotient(at - b_at, span);
  const long long unit_at = b_at + (long long)unit * span;
  const int tile0 = max(0, (int)(at - unit_at) - kSetup);
  const int tile1 = max(0, (int)(min(end - unit_at, (long long)span)) - kSetup);
  const int n_tiles = tile1 - tile0;
  at = unit_at + span < end ? unit_at + span : end;
  const int seq = b;
  if (at == b_at + (long long)span * per_seq) {
    b_at = at;
    do ++b;
    while (b < B && tiles_of(__ldg(t + b), cap) == 0);
  }
  if (n_tiles == 0) continue;  // the share ends inside the unit's setup
  const int hg = unit % n_hg, hk = unit / n_hg;
  const int h_base = hk * G + hg * kHeads;
  const int n_heads = min(kHeads, G - hg * kHeads);
  __syncthreads();  // the piece before is done
  if (tid == 0) bad_pages[~piece & 1] = 0;
  // first keys of the query's own chunk and of the one before; the DCA pieces that
  // the share's keys lie in, p_lo for the last key and p_hi for the first
  const int own0 = tb - tb % s, prev0 = own0 - s;
  auto dca_piece = [&](int j) { return j < prev0 ? 2 : (j < own0 ? 1 : 0); };
  const int p_lo = dca_piece(min(tile1 * kTileKeys - 1, tb)), p_hi = dca_piece(tile0 * kTileKeys);
  // everything that is fetched to begin with, in flight at once behind the rotations:
  // the first of the pages and the queries
  const int* pages = pg.table + (size_t)seq * pg.max_blocks;
  int blk = tid < n_tiles ? __ldg(pages + (tile0 + tid) / tpb) : 0;
  const bool has_q = tid < n_heads * D / 8;
  uint4 q8 = {};
  if (has_q)
    q8 = __ldg(reinterpret_cast<const uint4*>(q + ((size_t)seq * Hq + h_base) * D) + tid);
  if (turned != seq) turns = 0;
  turned = seq;
  const int missing = ((2 << p_hi) - (1 << p_lo)) & ~turns;
  if (missing) {
    const int im = tb % s;
#pragma unroll 1
    for (int x = tid; x < 3 * (D / 2); x += kThreads) {
      const int p = x / (D / 2), k = x % (D / 2);
      if (!(missing >> p & 1)) continue;
      double cd, sd;
      sincos64((double)query_pos_for_piece(p, im, s, c) * theta.v[k], cd, sd);
      cs[x] = make_float2((float)cd, (float)sd);
    }
    turns |= missing;
  }
  for (int i = tid; i < n_tiles; i += kThreads) {
    const int tile = tile0 + i;
    if (i != tid) blk = __ldg(pages + tile / tpb);
    if ((unsigned)blk >= (unsigned)pg.num_blocks) {
      report_error(kDevBadArg, 208);  // the outputs become NaN
      *bad_page = 1;
      blk = 0;
    }
    places[i] = (uint32_t)(((size_t)blk * pg.Hkv + hk) * tpb + tile % tpb);
  }
  if (has_q) reinterpret_cast<uint4*>(qraw)[tid] = q8;
  __syncthreads();
  const int parts = n_tiles > warp ? 2 * ((n_tiles - warp + W - 1) / W) : 0;
  // lane 0: fetch part i of this warp's tiles into buffer `to`
  auto fetch = [&](int i, int to) {
    const uint8_t* src = pg.pool + (size_t)places[warp + (i >> 1) * W] * TL::kBytes +
                         (i & 1) * SM::kHalf;
    const uint32_t bar = full0 + 8 * to;
    mbar_arrive_expect_tx(bar, SM::kHalf);
    bulk_load(smem_u32(ring) + to * SM::kHalf, src, SM::kHalf, bar);
  };
  if (lane == 0)
    for (int i = 0, to = buf; i < min(parts, kRing); ++i, to = to == kRing - 1 ? 0 : to + 1)
      fetch(i, to);

  // ---------------- queries: rotations, fragments, group sums ----------------
  {
    constexpr int kPairs = D / 64;  // (k, k + D/2) pairs a lane owns of a head
#pragma unroll 1
    for (int job = warp; job < (p_hi - p_lo + 1) * n_heads; job += W) {
      const int p = p_lo + job / n_heads, hh = job % n_heads;  // a piece and a head
      float x0[kPairs], x1[kPairs], big = 0.f;
      // by the head's largest element first, so that queries of any size have the
      // same bits behind them
#pragma unroll
      for (int u = 0; u < kPairs; ++u) {
        x0[u] = __bfloat162float(qraw[hh * D + lane + 32 * u]);
        x1[u] = __bfloat162float(qraw[hh * D + lane + 32 * u + D / 2]);
        big = fmaxf(big, fmaxf(fabsf(x0[u]), fabsf(x1[u])));
      }
      const int most = (int)(__reduce_max_sync(~0u, __float_as_uint(big)) >> 23) - 127;
      const int er = max(-126, min(most, 126));
      const float whole_q = power2(-er);
      big = 0.f;
#pragma unroll
      for (int u = 0; u < kPairs; ++u) {
        x0[u] = x0[u] * whole_q * scale_log2;
        x1[u] = x1[u] * whole_q * scale_log2;
        big = fmaxf(big, fabsf(x0[u]) + fabsf(x1[u]));
      }
      big = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(big)));
      // every rotated value times 2^-e stays below 2^11; scores come times 2^-(e + er + 24),
      // which is to be a normal number (smaller ones are nothing to any key)
      const int e = max(big > 0.f ? (int)(__float_as_uint(big) >> 23) - 127 - 10 : 0, -150 - er);
      const float down = power2(-(e / 2)), down2 = power2(-(e - e / 2));
      {
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kPairs; ++u) {
          const int k = lane + 32 * u;
          const float2 r = cs[p * (D / 2) + k];
          const float y[2] = {fmaf(x0[u], r.x, -x1[u] * r.y), fmaf(x1[u], r.x, x0[u] * r.y)};
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int d = k + v * (D / 2);
            // nibbles 0..3 of a word go to the low halves of four registers,
            // 4..7 to the high halves; odd nibbles arrive times 16
            const int g = d / 64, i = (d % 64) / 8, n = d % 8;
            const float z = y[v] * down * down2, whole = rintf(z), by = (n & 1) ? 0.0625f : 1.f;
            sum[D == 128 ? v : 0] += z;
            const __half hi = __float2half_rn(whole * by);
            const __half lo = __float2half_rn((z - whole) * by);
            const int at =
                ((((p * 2) * kGr + g) * kHeads + hh) * 8 + i) * 8 + (n & 3) * 2 + (n >> 2);
            reinterpret_cast<__half*>(qf)[at] = hi;
            reinterpret_cast<__half*>(qf)[at + kGr * kHeads * 64] = lo;
          }
        }
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1)
#pragma unroll
          for (int g = 0; g < kGr; ++g) sum[g] += __shfl_xor_sync(~0u, sum[g], sh);
        // in the units of the code products
        const float unit = 5.9604644775390625e-8f;  // 2^-24
        if (lane < kGr) qsum[(p * kHeads + hh) * kGr + lane] = (lane == 0 ? sum[0] : sum[1]) * unit;
      }
      if (lane == 0 && p == p_lo) {
        qexp[hh] = power2(min(e + er + 24, 127));
        qexp[kHeads + hh] = power2(max(0, min(e + er + 24 - 127, 127)));
      }
    }
    __syncthreads();
  }

  // A lane owns the scores of keys kr and kr + 2 of a 16-key step (MMA rows g and
  // g + 8) and kOwn heads: 2 t4 and 2 t4 + 1, the MMA columns; or, with at most
  // four heads, head t4, whose high part and remainder are the two columns.
  const int g = lane >> 2, t4 = lane & 3;
  const int kr = 4 * (g >> 1) + (g & 1);
  const int head0 = kFew ? t4 : 2 * t4;
  float m_run[kOwn], l_run[kOwn];
  float off[kGr][kOwn];       // sum of p * offset, by group
  // O of 16 dims: rows g and g + 8, each kOwn heads; times 2^-10, rows g + 8 times
  // 16 besides.  (Products come times 2^14 for the weights and 2^-24 for the codes;
  // the two together, left alone, keep the least and the largest scales in range.)
  float o[kGr * 4][2 * kOwn];
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    m_run[e] = -INFINITY;
    l_run[e] = 0.f;
#pragma unroll
    for (int gr = 0; gr < kGr; ++gr) off[gr][e] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < kGr * 4; ++i)
#pragma unroll
    for (int e = 0; e < 2 * kOwn; ++e) o[i][e] = 0.f;

  {
    // ---------------- tiles ----------------
    float F[kOwn];
#pragma unroll
    for (int e = 0; e < kOwn; ++e) F[e] = qexp[head0 + e];
    int part = 0;
    auto next_part = [&]() {  // the part just read is free: fetch another in its place
      __syncwarp();
      if (lane == 0 && part + kRing < parts) fetch(part + kRing, buf);
      ++part;
      if (++buf == kRing) {
        buf = 0;
        phase ^= 1;
      }
    };
#pragma unroll 1
    for (int it = warp; it < n_tiles; it += W) {
      if (!warp_wait(full0 + 8 * buf, phase, abort_flag, 402)) break;
      const int j0 = (tile0 + it) * kTileKeys;
      const int j1 = min(j0 + kTileKeys - 1, tb);  // last valid key of the tile
      // scores over F: [16-key step][key kr + 2 u, head e] at u * kOwn + e
      float x[4][2 * kOwn];
#pragma unroll
      for (int sub = 0; sub < 4; ++sub)
#pragma unroll
        for (int e = 0; e < 2 * kOwn; ++e) x[sub][e] = 0.f;
      // Scores of piece p, whose keys of the tile are p0 .. p1 - 1; in a tile of
      // several pieces the other keys take part with parameters of 0.
      auto scores = [&](auto several, int p, int p0, int p1) {
        // the same codes again for the next piece: an offset that the compiler
        // cannot follow keeps it from holding them all in registers meanwhile
        uint32_t place = buf * SM::kHalf;
        asm volatile("" : "+r"(place));
        const uint8_t* codes = ring + place;
#pragma unroll
        for (int gr = 0; gr < kGr; ++gr) {
          // column g of the lane's two words of this group: head g's high part and
          // its remainder, or one of the two of head g / 2
          const uint4* qa = reinterpret_cast<const uint4*>(qf) + 2 * t4 +
                            (kFew ? (((p * 2 + (g & 1)) * kGr + gr) * kHeads + (g >> 1)) * 8
                                  : (((p * 2) * kGr + gr) * kHeads + g) * 8);
          const uint4 h[2] = {qa[0], qa[1]};
          uint4 l[2];
          if (!kFew) {
            l[0] = qa[kGr * kHeads * 8];
            l[1] = qa[kGr * kHeads * 8 + 1];
          }
          float qs[kOwn];
#pragma unroll
          for (int e = 0; e < kOwn; ++e) qs[e] = qsum[(p * kHeads + head0 + e) * kGr + gr];
#pragma unroll
          for (int pair = 0; pair < 4; pair += kMany) {  // 16-key steps, interleaved
            uint2 wa[kMany], wb[kMany];
            uint32_t par[kMany][2];
            float acc[kMany][4], low[kFew ? 1 : kMany][4];
#pragma unroll
            for (int n = 0; n < kMany; ++n) {
              const int r0 = (pair + n) * 16 + kr;
              const uint8_t* ka = codes + TL::k_word(0, gr, 0) + r0 * (D / 2) + t4 * (D / 8);
              const uint8_t* kp = codes + TL::k_param(0, gr) + r0 * (kGr * 4);
              wa[n] = *reinterpret_cast<const uint2*>(ka);
              wb[n] = *reinterpret_cast<const uint2*>(ka + D);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                par[n][u] = *reinterpret_cast<const uint32_t*>(kp + u * kGr * 8);
                if (several && (r0 + 2 * u < p0 || r0 + 2 * u >= p1)) par[n][u] = 0u;
              }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t u[kMany], v[kMany];
#pragma unroll
              for (int n = 0; n < kMany; ++n) {
                u[n] = w ? wa[n].y : wa[n].x;
                v[n] = w ? wb[n].y : wb[n].x;
              }
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t a[kMany][4];
#pragma unroll
                for (int n = 0; n < kMany; ++n) {
                  const uint32_t uu = u[n] >> (8 * half), vv = v[n] >> (8 * half);
                  a[n][0] = uu & 0x000F000Fu;
                  a[n][1] = vv & 0x000F000Fu;
                  a[n][2] = uu & 0x00F000F0u;
                  a[n][3] = vv & 0x00F000F0u;
                }
                const uint32_t h0 = half ? h[w].z : h[w].x, h1 = half ? h[w].w : h[w].y;
#pragma unroll
                for (int n = 0; n < kMany; ++n) {
                  if (w == 0 && half == 0) mma_codes_first(acc[n], a[n], h0, h1);
                  else mma_codes(acc[n], a[n], h0, h1);
                }
                if (!kFew) {
                  const uint32_t l0 = half ? l[w].z : l[w].x, l1 = half ? l[w].w : l[w].y;
#pragma unroll
                  for (int n = 0; n < kMany; ++n) {
                    if (w == 0 && half == 0) mma_codes_first(low[kFew ? 0 : n], a[n], l0, l1);
                    else mma_codes(low[kFew ? 0 : n], a[n], l0, l1);
                  }
                }
              }
            }
#pragma unroll
            for (int n = 0; n < kMany; ++n)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < kOwn; ++e) {
                  const float sum = kFew ? acc[n][2 * u] + acc[n][2 * u + 1]
                                         : acc[n][2 * u + e] + low[kFew ? 0 : n][2 * u + e];
                  float& z = x[pair + n][u * kOwn + e];
                  z = fmaf(bf16_lo(par[n][u]), sum, fmaf(bf16_hi(par[n][u]), qs[e], z));
                }
          }
        }
      };
      const int first = dca_piece(j1), last = dca_piece(j0);  // of the last key, the first one
      const bool whole = j1 - j0 == kTileKeys - 1;
      if (first == last && whole) {
        scores(std::false_type(), first, 0, kTileKeys);
      } else {
        int p1 = kTileKeys;
#pragma unroll 1
        for (int p = first; p <= last; ++p) {
          const int p0 = p == last ? 0 : (p == 0 ? own0 : prev0) - j0;
          scores(std::true_type(), p, p0, p1);
          p1 = p0;
        }
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < kOwn; ++e)
              if (j0 + sub * 16 + kr + 2 * u > j1) x[sub][u * kOwn + e] = -INFINITY;
      }
      next_part();
      // a query too large for one power of two (above about 2^115)
      if (fmaxf(F[0], F[kOwn - 1]) == kMostF) {
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int e = 0; e < 2 * kOwn; ++e) x[sub][e] *= qexp[kHeads + head0 + e % kOwn];
      }
      float mx[kOwn];
      bool higher = false;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        mx[e] = fmax3(fmax3(x[0][e], x[0][kOwn + e], x[1][e]),
                      fmax3(x[1][kOwn + e], x[2][e], x[2][kOwn + e]),
                      fmaxf(x[3][e], x[3][kOwn + e]));
#pragma unroll
        for (int sh = 4; sh <= 16; sh <<= 1)
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], sh));
        mx[e] *= F[e];
        higher |= mx[e] > m_run[e];
      }
      if (__any_sync(0xFFFFFFFFu, higher)) {
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
          const float mn = fmaxf(m_run[e], mx[e]);
          const float al = fast_exp2(m_run[e] - (mn == -INFINITY ? 0.f : mn));
          m_run[e] = mn;
          l_run[e] *= al;
#pragma unroll
          for (int gr = 0; gr < kGr; ++gr) off[gr][e] *= al;
#pragma unroll
          for (int i = 0; i < kGr * 4; ++i) {
            o[i][e] *= al;
            o[i][kOwn + e] *= al;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        const float mu = m_run[e] == -INFINITY ? 0.f : -m_run[e];
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float& z = x[sub][u * kOwn + e];
            z = fast_exp2(fmaf(z, F[e], mu));
            l_run[e] += z;
          }
      }
      if (!warp_wait(full0 + 8 * buf, phase, abort_flag, 403)) break;
      const uint8_t* tile = ring + buf * SM::kHalf - SM::kHalf;  // V offsets count from the tile
      if (!whole) {  // rows past the sequence hold anything, NaN too
        for (int r = j1 - j0 + 1 + lane; r < kTileKeys; r += 32)
#pragma unroll
          for (int gr = 0; gr < kGr; ++gr)
            *reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(tile) + TL::v_param(r, gr)) = 0u;
        __syncwarp();
      }
      // Weights p * scale of every 16-key step as MMA columns: the lane's two heads,
      // a set for each group; or both groups of its one head.
      float down[kGr];
      uint32_t wgt[kFew ? 1 : kGr][4][2];
      float few[kFew ? 4 : 1][2][2];
#pragma unroll
      for (int gr = 0; gr < kGr; ++gr) {
        uint32_t par[4][2], most = 0;
        const uint8_t* vp = tile + TL::v_param(0, gr) + kr * (kGr * 4);
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            par[sub][u] = *reinterpret_cast<const uint32_t*>(vp + (sub * 16 + 2 * u) * (kGr * 4));
            most = max_bf16x2(most, par[sub][u]);
          }
        // scale * 2^(14 - exponent of the tile's largest scale) < 2^15: a product, not
        // a sum of exponents, which a scale of 0 or one far below the largest would
        // leave; its factor is a normal number for every ex (from a largest scale of
        // 2^-113 on; smaller ones count as that)
        const uint32_t ex =
            max(__reduce_max_sync(0xFFFFFFFFu, most & 0xFFFFu) >> 7, 14u);
        const float up = __uint_as_float((268u - ex) << 23);
        down[gr] = __uint_as_float(ex << 23);
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float sc = bf16_lo(par[sub][u]) * up;
            const float* pr = x[sub] + u * kOwn;
#pragma unroll
            for (int e = 0; e < kOwn; ++e)
              off[gr][e] = fmaf(pr[e], bf16_hi(par[sub][u]), off[gr][e]);
            if (kFew) few[kFew ? sub : 0][u][gr] = pr[0] * sc;
            else
              wgt[kFew ? 0 : gr][sub][u] =
                  transpose8x8(pack_half(pr[0] * sc, pr[kOwn - 1] * sc));
          }
        if (!kFew) pv<D>(o, wgt[kFew ? 0 : gr], tile, gr, g, t4, down[gr]);
      }
      if (kFew) {
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            wgt[0][sub][u] = transpose8x8(pack_half(few[kFew ? sub : 0][u][0],
                                                    kGr == 2 ? few[kFew ? sub : 0][u][1] : 0.f));
#pragma unroll
        for (int gr = 0; gr < kGr; ++gr) pv<D>(o, wgt[0], tile, gr, g, t4, down[gr]);
      }
      next_part();
    }
#pragma unroll
    for (int sh = 4; sh <= 16; sh <<= 1) {
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        l_run[e] += __shfl_xor_sync(0xFFFFFFFFu, l_run[e], sh);
#pragma unroll
        for (int gr = 0; gr < kGr; ++gr)
          off[gr][e] += __shfl_xor_sync(0xFFFFFFFFu, off[gr][e], sh);
      }
    }
  }
  __syncthreads();  // every part is read: the rings hold the merge now
  if (*abort_flag) {  // a wait gave up: let the copies in flight land, within limits
    if (lane == 0)
      for (int i = 0; i < kRing; ++i)
        mbar_wait(full0 + 8 * i, i < buf ? phase ^ 1 : phase, nullptr, 404, kWaitDeadlineNs / 8);
    return;
  }

  float* mo = reinterpret_cast<float*>(smem);   // [warp][head][D]
  float* mm = mo + W * kHeads * D;         // [warp][head]
  float* ml = mm + W * kHeads;             // [warp][head]
  {
#pragma unroll
    for (int gr = 0; gr < kGr; ++gr)
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
          // rows g and g + 8 are dims 2m and 2m + 1 of word g
          float* at = mo + (warp * kHeads + head0 + e) * D + gr * 64 + 8 * g + 2 * m;
          at[0] = fmaf(o[gr * 4 + m][e], 1024.f, off[gr][e]);        // 2^10
          at[1] = fmaf(o[gr * 4 + m][kOwn + e], 64.f, off[gr][e]);   // 2^10 / 16
        }
    if (g == 0) {
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        mm[warp * kHeads + head0 + e] = m_run[e];
        ml[warp * kHeads + head0 + e] = l_run[e];
      }
    }
  }
  __syncthreads();
  const float poison = *bad_page ? __int_as_float(0x7fc00000) : 0.f;
  for (int idx = tid; idx < n_heads * D; idx += kThreads) {
    const int hh = idx / D, d = idx % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, mm[w * kHeads + hh]);
    const float mu = M == -INFINITY ? 0.f : M;
    float acc = poison, lsum = poison;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = fast_exp2(mm[w * kHeads + hh] - mu);
      acc += f * mo[(w * kHeads + hh) * D + d];
      lsum += f * ml[w * kHeads + hh];
    }
    if (kWhole) {
      const size_t row = (size_t)seq * Hq + h_base + hh;
      O[row * D + d] = __float2bfloat16_rn(acc / lsum);
      if (d == 0) LSE[row] = (mu + log2f(lsum)) * 0.69314718055994530942f;
    } else {
      const size_t slot = ((size_t)seq * per_seq + unit + blockIdx.x) * kHeads + hh;
      Opart[slot * D + d] = acc;
      if (d == 0) MLpart[slot] = make_float2(M, lsum);
    }
  }
  // the buffers go back to the copies of the next piece
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
}

// O = sum_p e^{m_p - m} O_p / sum_p e^{m_p - m} l_p over the partial results of
// a unit, LSE = m + ln(sum).  kRows heads of a sequence a block, 8 / kRows warps a
// head over its partials in turn, a row of D a warp.  It starts beside the decode
// kernel, finds its place from t and waits for the results.
constexpr int kMergeThreads = 256;

template <int D, int kRows>
__global__ void __launch_bounds__(kMergeThreads) decode_merge(
    const float* __restrict__ Opart, const float2* __restrict__ MLpart,
    const int* __restrict__ t, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE, int B,
    int Hq, int Hkv, int n_hg, long long cap, int grid_shares) {
  constexpr int kW = kMergeThreads / 32 / kRows, kEach = D / 32;
  __shared__ float part[kMergeThreads / 32][D];
  __shared__ float2 stat[kMergeThreads / 32];
  __shared__ long long sums[kMergeThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, h = blockIdx.x * kRows + warp / kW;
  const int tb = __ldg(t + b);
  const int G = Hq / Hkv, per_seq = Hkv * n_hg;
  const long long all = spans_before(t, B, cap, sums) * per_seq;
  const long long b_at = spans_before(t, b, cap, sums) * per_seq;
  const int tiles = tiles_of(tb, cap);
  cudaGridDependencySynchronize();
  // this warp's partials' sum, relative to their own maximum
  float m = -INFINITY, l = 0.f, acc[kEach] = {};
  if (tiles > 0 && h < Hq) {
    const int unit = h / G * n_hg + h % G / kHeads, hh = h % G % kHeads;
    const long long g0 = b_at + (long long)unit * (tiles + kSetup) + kSetup;
    const Split split = make_split(all, share_count(all, grid_shares));
    const long long c0 = share_of(split, g0);
    const int n = (int)(share_of(split, g0 + tiles - 1) - c0) + 1;
    const size_t slot0 = ((size_t)b * per_seq + unit + c0) * kHeads + hh;
#pragma unroll 4
    for (int p = warp % kW; p < n; p += kW) {
      const size_t slot = slot0 + (size_t)p * kHeads;
      const float2 ml = MLpart[slot];
      float v[kEach];
      const float* from = Opart + slot * D + lane * kEach;
      if (D == 128) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(from);
      else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(from);
      const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
      const float old = fast_exp2(m - mu), now = fast_exp2(ml.x - mu);
      m = mn;
      l = l * old + ml.y * now;
#pragma unroll
      for (int e = 0; e < kEach; ++e) acc[e] = acc[e] * old + v[e] * now;
    }
  }
  if (kW > 1) {  // the head's warps: all sums to the first
#pragma unroll
    for (int e = 0; e < kEach; ++e) part[warp][lane * kEach + e] = acc[e];
    if (lane == 0) stat[warp] = make_float2(m, l);
    __syncthreads();
    if (warp % kW) return;
    for (int w = 1; w < kW; ++w) m = fmaxf(m, stat[warp + w].x);
    const float mu = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
    for (int w = 0; w < kW; ++w) {
      const float f = fast_exp2(stat[warp + w].x - mu);
      l += f * stat[warp + w].y;
#pragma unroll
      for (int e = 0; e < kEach; ++e) acc[e] += f * part[warp + w][lane * kEach + e];
    }
  }
  if (h >= Hq) return;
  const float nan = __int_as_float(0x7fc00000);
  const size_t row = (size_t)b * Hq + h;
  uint32_t out[kEach / 2];
#pragma unroll
  for (int e = 0; e < kEach; e += 2)
    out[e / 2] = tiles ? pack_bf16(acc[e] / l, acc[e + 1] / l) : pack_bf16(nan, nan);
  __nv_bfloat16* to = O + row * D + lane * kEach;
  if (D == 128) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(out);
  else *reinterpret_cast<uint32_t*>(to) = out[0];
  if (lane == 0)
    LSE[row] = tiles ? ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.69314718055994530942f : nan;
}

namespace {
std::atomic<unsigned long long> g_smem_set[12];  // by kernel: a bit a device
}

template <int D>
cudaError_t launch_decode_t(const void* q, const Pages& pg, const int* t, void* O, float* LSE,
                            int B, int Hq, int s, int c, float base, float scale,
                            void* workspace, cudaStream_t stream) {
  const long long cap = (long long)pg.max_blocks * pg.block_rows;
  const int shares = (int)decode_shares(B, Hq, pg.Hkv, cap);
  const int n_hg = head_groups(Hq, pg.Hkv);
  const size_t slots = ((size_t)B * pg.Hkv * n_hg + shares) * kHeads;
  float* Opart = static_cast<float*>(workspace);
  float2* MLpart = reinterpret_cast<float2*>(Opart + slots * D);
  const long long units = (long long)B * pg.Hkv * n_hg;
  const bool few = Hq / pg.Hkv <= 4, whole_units = takes_whole(units, cap);
  const bool wide = whole_units && units <= 148;
  auto kern =
      wide ? (few ? decode_kernel<D, true, kWide, true> : decode_kernel<D, false, kWide, true>)
      : whole_units
          ? (few ? decode_kernel<D, true, kWarps, true> : decode_kernel<D, false, kWarps, true>)
          : (few ? decode_kernel<D, true, kWarps, false> : decode_kernel<D, false, kWarps, false>);
  const int threads = (wide ? kWide : kWarps) * 32;
  const int smem = wide ? DecodeSmem<D, kWide>::kTotal : DecodeSmem<D, kWarps>::kTotal;
  // once a device: the attribute stays with the function there
  std::atomic<unsigned long long>& set = g_smem_set[D / 128 * 6 + (wide + whole_units) * 2 + few];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(set.load() >> dev & 1))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) set.fetch_or(1ull << dev);
  }
  if (e != cudaSuccess) return e;
  kern<<<whole_units ? (int)units : shares, threads, smem, stream>>>(
      static_cast<const __nv_bfloat16*>(q), pg, t, Opart, MLpart, static_cast<__nv_bfloat16*>(O),
      LSE, B, Hq, s, c, scale * 1.4426950408889634f, n_hg, make_theta(D, base));
  e = cudaGetLastError();
  if (e != cudaSuccess || whole_units) return e;
  // Warps by the partials a unit has on average.  A block a head against a warp a
  // head, 8 heads a unit, in a graph: 4 / 64 / 128 / 440 units of 4000 keys 11.0 / 23.8 /
  // 34.5 / 91.6 us against 13.7 / 24.2 / 33.2 / 78.8, of 16000 keys 13.4 / 46.3 / 81.4 /
  // 242 against 27.1 / 46.8 / 79.5 / 236.  They meet where a unit has four to eight.
  auto merge = shares > 4 * units ? decode_merge<D, 1> : decode_merge<D, 8>;
  const int rows = shares > 4 * units ? 1 : 8;
  return launch_early(merge, dim3((Hq + rows - 1) / rows, B), kMergeThreads, stream,
                      static_cast<const float*>(Opart), static_cast<const float2*>(MLpart), t,
                      static_cast<__nv_bfloat16*>(O), LSE, B, Hq, pg.Hkv, n_hg, cap, shares);
}

}  // namespace kv4

// Units, shares and a sequence's query elements (with a block's step) are counted in
// ints.
bool kv4_decode_fits(int B, int Hq, int Hkv, int D, long long cap) {
  constexpr long long kMost = 0x7FFFFFFF;
  return (long long)Hq * D <= 1 << 30 && (long long)B * Hkv * kv4::head_groups(Hq, Hkv) <= kMost &&
         kv4::decode_shares(B, Hq, Hkv, cap) <= kMost;
}

size_t kv4_decode_workspace_bytes(int B, int Hq, int Hkv, int D, long long cap) {
  const size_t units = (size_t)B * Hkv * kv4::head_groups(Hq, Hkv);
  const size_t slots = units + (size_t)kv4::decode_shares(B, Hq, Hkv, cap);
  return B == 0 ? 0 : slots * kv4::kHeads * (D + 2) * sizeof(float);
}

cudaError_t launch_kv4_decode(const void* q, const void* pool, const int* block_table,
                              int max_blocks, int block_rows, int num_blocks, const int* t,
                              void* O, float* LSE, int B, int Hq, int Hkv, int D, int s, int c,
                              float base, float scale, void* workspace, cudaStream_t stream) {
  const kv4::Pages pg{static_cast<uint8_t*>(const_cast<void*>(pool)), block_table, max_blocks,
                      block_rows, num_blocks, Hkv};
  return D == 64 ? kv4::launch_decode_t<64>(q, pg, t, O, LSE, B, Hq, s, c, base, scale, workspace,
                                            stream)
                 : kv4::launch_decode_t<128>(q, pg, t, O, LSE, B, Hq, s, c, base, scale,
                                             workspace, stream);
}

}  // namespace dca
