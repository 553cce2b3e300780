// DCA decode over a paged 4-bit cache (kv4.cuh): one new query per sequence.
//
// Mathematics.  With key j stored as khat = c * scale + offset per group g,
//     S_j = sum_g scale_jg <q_g, c_jg> + offset_jg * sum(q_g),
// so the matrix product runs on the bare codes and a key costs one FMA pair a
// group and head instead of a conversion an element.  The codes 0 .. 15 are
// exact as fp16 SUBNORMALS: a nibble masked into the low mantissa bits of each
// half of a word is c * 2^-24 (bits 4-7: 16 c * 2^-24, undone by a query
// pre-scaled by 1/16), so eight codes cost four logic operations and a shift.
// q is kept as an fp16 high part and remainder (normalised per head by a power
// of two), about 22 significant bits.  For the values,
//     O = sum_j p_j (c_j - 8) scale_j + sum_j p_j (offset_j + 8 scale_j):
// centred codes are exact in bf16 and keep the sums near the size of the
// result; p_j scale_j is rounded to bf16 (as P is in the bf16 decode) and the
// second sum stays in fp32 outside the matrix product.
//
// Kernel 1, one CTA per (share of the cache, kv head, group of <= 8 query
// heads, sequence): a producer warp brings whole 64-key tiles (K and V codes
// and their parameters, 72 * D contiguous bytes) with one bulk copy each into a
// ring; four consumer warps take tiles in turn, so that the running maximum, its
// shuffles and the rescaling of O are paid once per 64 keys of a warp.  The
// sequence's tiles are shared out evenly on the device from t[b], whatever the
// cache's capacity.  Kernel 2 merges the shares.
#include "dca_common.cuh"
#include "dca_index.cuh"
#include "dca_kernels.cuh"
#include "kv4.cuh"

namespace dca {
namespace kv4 {

constexpr int kHeads = 8;        // query heads per CTA (MMA N)
constexpr int kWarps = 4;        // consumer warps
constexpr int kDecodeThreads = (kWarps + 1) * 32;
constexpr int kStages = 6;

// CTAs wanted in flight over the whole call: three fit an SM, and shares of
// unequal sequences even out over a few waves.
constexpr int kWantCtas = 148 * 3 * 2;
inline int decode_shares(int B, int Hq, int Hkv, long long cap) {
  if (B == 0) return 1;
  const int G = Hq / Hkv;
  const long long units = (long long)B * Hkv * ((G + kHeads - 1) / kHeads);
  const long long tiles = (cap + kTileKeys - 1) / kTileKeys;
  long long n = (kWantCtas + units - 1) / units;
  if (n > tiles) n = tiles;
  if (n > 256) n = 256;
  return n < 1 ? 1 : (int)n;
}

template <int D>
struct DecodeSmem {
  static constexpr int kRing = kStages * Tile<D>::kBytes;
  // [piece][hi, lo][group][head][word] x 16 bytes of query fragments
  static constexpr int kQ = 3 * 2 * (D / 64) * kHeads * 8 * 16;
  static constexpr int kCs = 3 * (D / 2) * 8;          // cos, sin
  static constexpr int kSums = 3 * kHeads * (D / 64) * 4;  // sum of q per group
  static constexpr int kF = kHeads * 4;
  static constexpr int kBars = 2 * kStages * 8 + 16;  // + abort, page and copy words
  static constexpr int kTotal = 128 + kRing + kQ + kCs + kSums + kF + kBars;
  static_assert(kWarps * kHeads * (D + 2) * 4 <= kRing, "merge area");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void lds64(uint32_t& x, uint32_t& y, uint32_t a) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}

// Shares of a sequence of n_tiles tiles: tiles per share; share sp holds tiles
// sp * per .. (sp + 1) * per - 1.
__device__ __forceinline__ int tiles_per_share(int n_tiles, int shares) {
  return (n_tiles + shares - 1) / shares;
}

// Codes of one nibble position as bf16 pairs c - 8 (exact).
__device__ __forceinline__ uint32_t centred(uint32_t w) {
  const uint32_t v = (w & 0x000F000Fu) | 0x43004300u;  // 128 + c
  const uint32_t bias = 0x43084308u;                   // 136
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&d);
}

template <int D>
__global__ void __launch_bounds__(kDecodeThreads, 3) decode_kernel(
    const __nv_bfloat16* __restrict__ q, Pages pg, const int* __restrict__ t,
    float* __restrict__ Opart, float* __restrict__ MLpart, int Hq, int s, int c, float scale_log2,
    int shares, int n_hg, const __grid_constant__ Theta theta) {
  using TL = Tile<D>;
  using SM = DecodeSmem<D>;
  constexpr int kGr = TL::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 127) & ~(uintptr_t)127);
  const uint32_t ring = smem_u32(smem);
  uint8_t* qf = smem + SM::kRing;
  float2* cs = reinterpret_cast<float2*>(qf + SM::kQ);
  float* qsum = reinterpret_cast<float*>(qf + SM::kQ + SM::kCs);  // [piece][head][group]
  float* qexp = qsum + 3 * kHeads * kGr;                          // [head]
  uint8_t* bars = reinterpret_cast<uint8_t*>(qexp + kHeads);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + kStages * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * kStages * 8);
  volatile int* bad_page = abort_flag + 1;
  volatile int* issued = abort_flag + 2;  // copies started

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sp = blockIdx.x;
  const int hg = blockIdx.y % n_hg, hk = blockIdx.y / n_hg, b = blockIdx.z;
  const int G = Hq / pg.Hkv;
  const int tb = __ldg(t + b);
  if (tb < 0 || tb >= pg.max_blocks * pg.block_rows) {
    if (tid == 0 && sp == 0 && blockIdx.y == 0) report_error(kDevBadArg, 207);
    return;
  }
  const int all_tiles = tb / kTileKeys + 1;
  const int per = tiles_per_share(all_tiles, shares);
  const int tile0 = sp * per;
  if (tile0 >= all_tiles) return;
  const int n_tiles = min(per, all_tiles - tile0);
  const int h_base = hk * G + hg * kHeads;
  const int n_heads = min(kHeads, G - hg * kHeads);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    *abort_flag = 0;
    *bad_page = 0;
    *issued = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ---------------- producer ----------------
    const int tpb = pg.block_rows / kTileKeys;
    for (int it0 = 0; it0 < n_tiles; it0 += 32) {
      // the pages of the next 32 tiles, one lookup a lane
      const int mine = tile0 + it0 + lane;
      const uint8_t* src = nullptr;
      if (it0 + lane < n_tiles) {
        int blk = __ldg(pg.table + (size_t)b * pg.max_blocks + mine / tpb);
        if (blk < 0 || blk >= pg.num_blocks) {  // reported; the outputs become NaN
          report_error(kDevBadArg, 208);
          *bad_page = 1;
          blk = 0;
        }
        src = pg.pool + (((size_t)blk * pg.Hkv + hk) * tpb + mine % tpb) * TL::kBytes;
      }
      const int n = min(32, n_tiles - it0);
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        const int it = it0 + j, st = it % kStages;
        const uint8_t* from = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xFFFFFFFFu, (unsigned long long)src, j));
        if (it >= kStages)
          ok = warp_wait(empty0 + 8 * st, ((it / kStages) + 1) & 1, abort_flag, 401);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(full0 + 8 * st, TL::kBytes);
          bulk_load(ring + st * TL::kBytes, from, TL::kBytes, full0 + 8 * st);
          *issued = it + 1;
        }
      }
      if (!ok) break;
    }
  }

  // ---------------- queries: three rotations, fragments, group sums ----------------
  if (warp < kWarps) {
    const int im = tb % s;
    for (int x = tid; x < 3 * (D / 2); x += kWarps * 32) {
      const int p = x / (D / 2), k = x % (D / 2);
      constexpr double kTwoPi = 6.283185307179586476925286766559;
      const double a = (double)query_pos_for_piece(p, im, s, c) * theta.v[k];
      float sf, cf;
      sincosf((float)fma(-rint(a * (1.0 / kTwoPi)), kTwoPi, a), &sf, &cf);
      cs[x] = make_float2(cf, sf);
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    constexpr int kPairs = D / 64;  // (k, k + D/2) pairs a lane owns of a head
    for (int hh = warp; hh < kHeads; hh += kWarps) {
      float x0[kPairs], x1[kPairs], big = 0.f;
#pragma unroll
      for (int u = 0; u < kPairs; ++u) {
        x0[u] = x1[u] = 0.f;
        if (hh < n_heads) {
          const __nv_bfloat16* row = q + ((size_t)b * Hq + h_base + hh) * D + lane + 32 * u;
          x0[u] = __bfloat162float(row[0]) * scale_log2;
          x1[u] = __bfloat162float(row[D / 2]) * scale_log2;
        }
        big = fmaxf(big, fabsf(x0[u]) + fabsf(x1[u]));
      }
#pragma unroll
      for (int sh = 16; sh >= 1; sh >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, sh));
      // every rotated value times 2^-e stays below 2^13
      const int e = big > 0.f ? (int)(__float_as_uint(big) >> 23) - 127 - 12 : 0;
      const float down = ldexpf(1.f, -(e / 2)), down2 = ldexpf(1.f, -(e - e / 2));
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kPairs; ++u) {
          const int k = lane + 32 * u;
          const float2 r = cs[p * (D / 2) + k];
          const float y[2] = {fmaf(x0[u], r.x, -x1[u] * r.y), fmaf(x1[u], r.x, x0[u] * r.y)};
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int d = k + v * (D / 2);
            sum[D == 128 ? v : 0] += y[v];
            // nibbles 0..3 of a word go to the low halves of four registers,
            // 4..7 to the high halves; odd nibbles arrive times 16
            const int g = d / 64, i = (d % 64) / 8, n = d % 8;
            const float z = y[v] * down * down2 * ((n & 1) ? 0.0625f : 1.f);
            const __half hi = __float2half_rn(z);
            const __half lo = __float2half_rn(z - __half2float(hi));
            const int at = ((((p * 2) * kGr + g) * kHeads + hh) * 8 + i) * 8 + (n & 3) * 2 + (n >> 2);
            reinterpret_cast<__half*>(qf)[at] = hi;
            reinterpret_cast<__half*>(qf)[at + kGr * kHeads * 64] = lo;
          }
        }
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1)
#pragma unroll
          for (int g = 0; g < kGr; ++g) sum[g] += __shfl_xor_sync(~0u, sum[g], sh);
        if (lane < kGr) qsum[(p * kHeads + hh) * kGr + lane] = lane == 0 ? sum[0] : sum[1];
      }
      if (lane == 0) qexp[hh] = ldexpf(1.f, e + 24);
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
  }

  const int g = lane >> 2, t4 = lane & 3;
  float m_run[2] = {-INFINITY, -INFINITY};  // heads 2 t4, 2 t4 + 1
  float l_run[2] = {0.f, 0.f};
  float off[kGr][2];                        // sum of p (offset + 8 scale), by group
  float o[kGr * 4][4];
#pragma unroll
  for (int i = 0; i < kGr * 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
  for (int i = 0; i < kGr; ++i) off[i][0] = off[i][1] = 0.f;

  if (warp < kWarps) {
    // ---------------- consumers ----------------
    const int ci = tb / s;
    const float F[2] = {qexp[2 * t4], qexp[2 * t4 + 1]};
    int cur = -1;
    uint32_t qh[kGr][2][4], ql[kGr][2][4];
    float qs[kGr][2];
    const int kr = 4 * (g >> 1) + (g & 1);  // MMA row g holds key kr, row g + 8 key kr + 2
    for (int it = warp; it < n_tiles; it += kWarps) {
      const int st = it % kStages;
      if (!warp_wait(full0 + 8 * st, (it / kStages) & 1, abort_flag, 402)) break;
      const uint32_t tile = ring + st * TL::kBytes;
      const int j0 = (tile0 + it) * kTileKeys;
      const int j1 = min(j0 + kTileKeys - 1, tb);  // last valid key of the tile
      float x[4][4];  // [16-key step][(kr, head 0), (kr, head 1), (kr + 2, ..), ..]
      // pieces of the tile, nearest first; distances of 2 and more are one piece
      const int dlo = min(ci - j1 / s, 2), dhi = min(ci - j0 / s, 2);
#pragma unroll 1
      for (int p = dlo; p <= dhi; ++p) {
        if (p != cur) {
          cur = p;
#pragma unroll
          for (int gr = 0; gr < kGr; ++gr) {
            const uint32_t a = smem_u32(qf) +
                               ((((p * 2) * kGr + gr) * kHeads + g) * 8 + 2 * t4) * 16;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              lds128(qh[gr][w], a + w * 16);
              lds128(ql[gr][w], a + kGr * kHeads * 128 + w * 16);
            }
            qs[gr][0] = qsum[(p * kHeads + 2 * t4) * kGr + gr];
            qs[gr][1] = qsum[(p * kHeads + 2 * t4 + 1) * kGr + gr];
          }
        }
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          const int r0 = sub * 16 + kr;
          uint32_t wa[4], wb[4];
          const uint32_t ka = tile + TL::k_word(0, 0, 0) + r0 * (D / 2) + t4 * (D / 8);
          if (D == 128) {
            lds128(wa, ka);
            lds128(wb, ka + 2 * (D / 2));
          } else {
            lds64(wa[0], wa[1], ka);
            lds64(wb[0], wb[1], ka + 2 * (D / 2));
          }
          float acc[kGr][4];
#pragma unroll
          for (int gr = 0; gr < kGr; ++gr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[gr][e] = 0.f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t u = wa[gr * 2 + w], v = wb[gr * 2 + w];
              const uint32_t a0[4] = {u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u,
                                      v & 0x00F000F0u};
              u >>= 8;
              v >>= 8;
              const uint32_t a1[4] = {u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u,
                                      v & 0x00F000F0u};
              const uint32_t h0[2] = {qh[gr][w][0], qh[gr][w][1]};
              const uint32_t h1[2] = {qh[gr][w][2], qh[gr][w][3]};
              const uint32_t l0[2] = {ql[gr][w][0], ql[gr][w][1]};
              const uint32_t l1[2] = {ql[gr][w][2], ql[gr][w][3]};
              mma_f16_16816(acc[gr], a0, h0);
              mma_f16_16816(acc[gr], a0, l0);
              mma_f16_16816(acc[gr], a1, h1);
              mma_f16_16816(acc[gr], a1, l1);
            }
          }
          uint32_t pa[2], pb[2];
          if (D == 128) {
            lds64(pa[0], pa[1], tile + TL::k_param(0, 0) + r0 * 8);
            lds64(pb[0], pb[1], tile + TL::k_param(0, 0) + r0 * 8 + 16);
          } else {
            pa[0] = lds32(tile + TL::k_param(0, 0) + r0 * 4);
            pb[0] = lds32(tile + TL::k_param(0, 0) + r0 * 4 + 8);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float main = 0.f, rest = 0.f;
#pragma unroll
            for (int gr = 0; gr < kGr; ++gr) {
              const uint32_t w = e < 2 ? pa[gr] : pb[gr];
              main = fmaf(bf16_lo(w), acc[gr][e], main);
              rest = fmaf(bf16_hi(w), qs[gr][e & 1], rest);
            }
            const float y = fmaf(main, F[e & 1], rest);
            if (dlo == dhi) {
              x[sub][e] = y;
            } else {  // keep the keys of piece p
              const int j = j0 + r0 + (e & 2);
              if (min(ci - j / s, 2) == p || p == dlo) x[sub][e] = y;
            }
          }
        }
      }
      if (j1 - j0 != kTileKeys - 1) {  // the sequence's last tile
#pragma unroll
        for (int sub = 0; sub < 4; ++sub)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j0 + sub * 16 + kr + (e & 2) > j1) x[sub][e] = -INFINITY;
      }
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(fmaxf(fmaxf(x[0][e], x[0][e + 2]), fmaxf(x[1][e], x[1][e + 2])),
                      fmaxf(fmaxf(x[2][e], x[2][e + 2]), fmaxf(x[3][e], x[3][e + 2])));
#pragma unroll
        for (int sh = 4; sh <= 16; sh <<= 1)
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], sh));
      }
      if (__any_sync(0xFFFFFFFFu, mx[0] > m_run[0] || mx[1] > m_run[1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m_run[e], mx[e]);
          const float al = fast_exp2(m_run[e] - (mn == -INFINITY ? 0.f : mn));
          m_run[e] = mn;
          l_run[e] *= al;
#pragma unroll
          for (int gr = 0; gr < kGr; ++gr) off[gr][e] *= al;
#pragma unroll
          for (int i = 0; i < kGr * 4; ++i) {
            o[i][e] *= al;
            o[i][e + 2] *= al;
          }
        }
      }
      const float mu[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0],
                           m_run[1] == -INFINITY ? 0.f : m_run[1]};
      const bool whole = j1 - j0 == kTileKeys - 1;
#pragma unroll
      for (int sub = 0; sub < 4; ++sub) {
        const int r0 = sub * 16 + kr;
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = fast_exp2(x[sub][e] - mu[e & 1]);
          l_run[e & 1] += pr[e];
        }
        uint32_t pa[2], pb[2];
        if (D == 128) {
          lds64(pa[0], pa[1], tile + TL::v_param(0, 0) + r0 * 8);
          lds64(pb[0], pb[1], tile + TL::v_param(0, 0) + r0 * 8 + 16);
        } else {
          pa[0] = lds32(tile + TL::v_param(0, 0) + r0 * 4);
          pb[0] = lds32(tile + TL::v_param(0, 0) + r0 * 4 + 8);
        }
        if (!whole) {  // rows past the sequence hold anything, NaN too
#pragma unroll
          for (int gr = 0; gr < kGr; ++gr) {
            if (j0 + r0 > j1) pa[gr] = 0u;
            if (j0 + r0 + 2 > j1) pb[gr] = 0u;
          }
        }
#pragma unroll
        for (int gr = 0; gr < kGr; ++gr) {
          const float sa = bf16_lo(pa[gr]), sb = bf16_lo(pb[gr]);
          const float ca = fmaf(8.f, sa, bf16_hi(pa[gr])), cb = fmaf(8.f, sb, bf16_hi(pb[gr]));
#pragma unroll
          for (int e = 0; e < 2; ++e)
            off[gr][e] = fmaf(pr[e], ca, fmaf(pr[e + 2], cb, off[gr][e]));
          const uint32_t bw[2] = {movmatrix_t(pack_bf16(pr[0] * sa, pr[1] * sa)),
                                  movmatrix_t(pack_bf16(pr[2] * sb, pr[3] * sb))};
          // word g of the group for keys 4 t4 .. 4 t4 + 3: MMA k rows
          // 2 t4, 2 t4 + 1 and 2 t4 + 8, 2 t4 + 9
          uint32_t v[4];
          lds128(v, tile + TL::v_word(0, 0, 0) + (((sub * kGr + gr) * 8 + g) * 16 + 4 * t4) * 4);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t ra = __byte_perm(v[0], v[1], half ? 0x7632 : 0x5410);
            uint32_t rb = __byte_perm(v[2], v[3], half ? 0x7632 : 0x5410);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t a[4] = {centred(ra), centred(ra >> 4), centred(rb),
                                     centred(rb >> 4)};
              mma_bf16_16816(o[gr * 4 + half * 2 + m], a, bw);
              ra >>= 8;
              rb >>= 8;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * st);
    }
#pragma unroll
    for (int sh = 4; sh <= 16; sh <<= 1) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l_run[e] += __shfl_xor_sync(0xFFFFFFFFu, l_run[e], sh);
#pragma unroll
        for (int gr = 0; gr < kGr; ++gr)
          off[gr][e] += __shfl_xor_sync(0xFFFFFFFFu, off[gr][e], sh);
      }
    }
  }
  __syncthreads();  // every stage is consumed: the ring holds the merge now
  if (*abort_flag) {  // a wait gave up: let the copies in flight land, within limits
    if (tid == 0) {
      const int n = *issued;
      for (int it = max(0, n - kStages); it < n; ++it)
        mbar_wait(full0 + 8 * (it % kStages), (it / kStages) & 1, nullptr, 403, kWaitDeadlineNs / 8);
    }
    return;
  }

  float* mo = reinterpret_cast<float*>(smem);   // [warp][head][D]
  float* mm = mo + kWarps * kHeads * D;         // [warp][head]
  float* ml = mm + kWarps * kHeads;             // [warp][head]
  if (warp < kWarps) {
#pragma unroll
    for (int gr = 0; gr < kGr; ++gr)
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // rows g and g + 8 are dims 2m and 2m + 1 of word g
          float* at = mo + (warp * kHeads + 2 * t4 + e) * D + gr * 64 + 8 * g + 2 * m;
          at[0] = o[gr * 4 + m][e] + off[gr][e];
          at[1] = o[gr * 4 + m][e + 2] + off[gr][e];
        }
    if (g == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mm[warp * kHeads + 2 * t4 + e] = m_run[e];
        ml[warp * kHeads + 2 * t4 + e] = l_run[e];
      }
    }
  }
  __syncthreads();
  const float poison = *bad_page ? __int_as_float(0x7fc00000) : 0.f;
  for (int idx = tid; idx < n_heads * D; idx += kDecodeThreads) {
    const int hh = idx / D, d = idx % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mm[w * kHeads + hh]);
    const float mu = M == -INFINITY ? 0.f : M;
    float acc = poison, lsum = poison;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = fast_exp2(mm[w * kHeads + hh] - mu);
      acc += f * mo[(w * kHeads + hh) * D + d];
      lsum += f * ml[w * kHeads + hh];
    }
    const size_t slot = ((size_t)b * Hq + h_base + hh) * shares + sp;
    Opart[slot * D + d] = acc;
    if (d == 0) {
      MLpart[slot * 2] = M;
      MLpart[slot * 2 + 1] = lsum;
    }
  }
}

// O = sum_p e^{m_p - m} O_p / sum_p e^{m_p - m} l_p over the shares that hold
// keys, LSE = m + ln(sum): one block a (head, sequence), four rows of D/4
// threads over the shares in turn.
template <int D>
__global__ void __launch_bounds__(D) decode_merge(const float* __restrict__ Opart,
                                                  const float* __restrict__ MLpart,
                                                  const int* __restrict__ t,
                                                  __nv_bfloat16* __restrict__ O,
                                                  float* __restrict__ LSE, int Hq, int cap,
                                                  int shares) {
  __shared__ float4 part[4][D / 4];
  __shared__ float stat[2];
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  const int tb = __ldg(t + b);
  const size_t row = (size_t)b * Hq + h;
  if (tb < 0 || tb >= cap) {
    O[row * D + d] = __float2bfloat16_rn(__int_as_float(0x7fc00000));
    if (d == 0) LSE[row] = __int_as_float(0x7fc00000);
    return;
  }
  const int tiles = tb / kTileKeys + 1, per = tiles_per_share(tiles, shares);
  const int n = (tiles + per - 1) / per;
  const float2* ml = reinterpret_cast<const float2*>(MLpart) + row * shares;
  if (d < 32) {
    float M = -INFINITY;
    for (int p = d; p < n; p += 32) M = fmaxf(M, ml[p].x);
#pragma unroll
    for (int sh = 16; sh >= 1; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, sh));
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int p = d; p < n; p += 32) l += fast_exp2(ml[p].x - mu) * ml[p].y;
#pragma unroll
    for (int sh = 16; sh >= 1; sh >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, sh);
    if (d == 0) {
      stat[0] = mu;
      stat[1] = l;
    }
  }
  __syncthreads();
  const float M = stat[0], l = stat[1];
  const int lane = d % (D / 4), first = d / (D / 4);
  const float4* src = reinterpret_cast<const float4*>(Opart) + row * shares * (D / 4) + lane;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = first; p < n; p += 4) {
    const float f = fast_exp2(ml[p].x - M);
    const float4 v = src[(size_t)p * (D / 4)];
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  part[first][lane] = acc;
  __syncthreads();
  const float* col = reinterpret_cast<const float*>(part);
  const float sum = (col[d] + col[D + d]) + (col[2 * D + d] + col[3 * D + d]);
  O[row * D + d] = __float2bfloat16_rn(sum / l);
  if (d == 0) LSE[row] = (M + log2f(l)) * 0.69314718055994530942f;
}

template <int D>
cudaError_t launch_decode_t(const void* q, const Pages& pg, const int* t, void* O, float* LSE,
                            int B, int Hq, int s, int c, float base, float scale,
                            void* workspace, cudaStream_t stream) {
  const int cap = pg.max_blocks * pg.block_rows;
  const int shares = decode_shares(B, Hq, pg.Hkv, cap);
  const int n_hg = (Hq / pg.Hkv + kHeads - 1) / kHeads;
  float* Opart = static_cast<float*>(workspace);
  float* MLpart = Opart + (size_t)B * Hq * shares * D;
  auto kern = decode_kernel<D>;
  constexpr int smem = DecodeSmem<D>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(shares, pg.Hkv * n_hg, B), kDecodeThreads, smem, stream>>>(
      static_cast<const __nv_bfloat16*>(q), pg, t, Opart, MLpart, Hq, s, c,
      scale * 1.4426950408889634f, shares, n_hg, make_theta(D, base));
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  decode_merge<D><<<dim3(Hq, B), D, 0, stream>>>(Opart, MLpart, t,
                                                 static_cast<__nv_bfloat16*>(O), LSE, Hq, cap,
                                                 shares);
  return cudaGetLastError();
}

}  // namespace kv4

size_t kv4_decode_workspace_bytes(int B, int Hq, int Hkv, int D, long long cap) {
  return (size_t)B * Hq * kv4::decode_shares(B, Hq, Hkv, cap) * (D + 2) * sizeof(float);
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
