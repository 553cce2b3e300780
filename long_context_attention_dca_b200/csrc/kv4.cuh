// The 4-bit key/value cache: its tile, its quantiser and the fp64 rotation
// angles its kernels share.
//
// A cache row (one token, one kv head) of D values is cut into D/64 groups of
// 64.  A group keeps a bf16 offset (its least value, which is a bf16 already),
// a bf16 scale (the smallest bf16 with 15 * scale >= greatest - least) and 64
// codes c in 0 .. 15:
//     c = rint((x - offset) / scale)  (half to even),  value = c * scale + offset,
// so |x - value| <= scale / 2 for every finite input.  A group that holds an
// infinity or a NaN keeps NaN parameters and reads back as NaN.
//
// 64 rows of one kv head form a tile of 72 * D bytes, contiguous, so that one
// bulk copy brings everything a warp of the decode kernel needs:
//     K codes   [64 keys][4 chunks][D/64][2 words]    row-wise: chunk t holds
//               words 2t, 2t+1 of every group, 16 bytes at D = 128
//     K params  [64 keys][D/64]    scale in the low, offset in the high half
//     V codes   [4][D/64][8 words][16 keys]           transposed per 16 keys
//     V params  [64 keys][D/64]
// Word i of a group holds its dims 8i .. 8i+7, lowest nibble first; a word
// belongs to one token, so an append writes whole words.  In these orders the
// decode kernel reads nothing but a lane's own MMA fragments from shared memory:
// values in 16-byte loads without conflicts; keys in 8-byte loads, a group at a
// time, two lanes of a half warp to a bank (rows 0 and 4, 1 and 5 of each eight lie
// a multiple of 128 bytes apart); parameters in 4-byte loads without conflicts.
// A page is [Hkv][block_rows / 64] tiles.
#pragma once

#include <cmath>

#include "dca_common.cuh"
#include "softmax_sm100.cuh"

namespace dca {
namespace kv4 {

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

constexpr int kTileKeys = 64;
constexpr int kGroup = 64;

template <int D>
struct Tile {
  static constexpr int kGroups = D / kGroup;
  static constexpr int kCodeBytes = kTileKeys * D / 2;
  static constexpr int kParamBytes = kTileKeys * kGroups * 4;
  static constexpr int kKCodes = 0;
  static constexpr int kKParams = kCodeBytes;
  static constexpr int kVCodes = kKParams + kParamBytes;
  static constexpr int kVParams = kVCodes + kCodeBytes;
  static constexpr int kBytes = kVParams + kParamBytes;
  // byte offset of word i of group g of key r (0 .. 63)
  __host__ __device__ static constexpr int k_word(int r, int g, int i) {
    return kKCodes + (((r * 4 + (i >> 1)) * kGroups + g) * 2 + (i & 1)) * 4;
  }
  __host__ __device__ static constexpr int v_word(int r, int g, int i) {
    return kVCodes + ((((r >> 4) * kGroups + g) * 8 + i) * 16 + (r & 15)) * 4;
  }
  __host__ __device__ static constexpr int k_param(int r, int g) {
    return kKParams + (r * kGroups + g) * 4;
  }
  __host__ __device__ static constexpr int v_param(int r, int g) {
    return kVParams + (r * kGroups + g) * 4;
  }
};
inline size_t tile_bytes(int D) { return (size_t)72 * D; }

// RoPE frequencies base^(-2k/D) in fp64, computed once on the host and passed
// by value (the device never evaluates a power).
struct Theta {
  double v[64];
};
inline Theta make_theta(int D, float base) {
  // base^(-2k/D), k = 8 i + j, as a product of two powers: 16 calls, a last
  // place of fp64 in accuracy
  Theta t;
  double big[8], small[8];
  for (int i = 0; i < 8; ++i) {
    big[i] = std::pow((double)base, -16.0 * i / D);
    small[i] = std::pow((double)base, -2.0 * i / D);
  }
  for (int k = 0; k < 64; ++k) t.v[k] = k < D / 2 ? big[k / 8] * small[k % 8] : 0.0;
  return t;
}

// cos and sin of a double angle (any size up to about 2^31 radians): reduced to
// |r| <= pi/4 by the nearest multiple of pi/2 (in two parts), then the Taylor
// series to r^16 (truncation below 1e-15).
__device__ __forceinline__ void sincos64(double a, double& c, double& s) {
  const double n = rint(a * 0.63661977236758134308);
  double r = fma(-n, 1.57079632679489655800, a);
  r = fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double p = fma(z, 1.0 / 355687428096000.0, -1.0 / 1307674368000.0);
  p = fma(z, p, 1.0 / 6227020800.0);
  p = fma(z, p, -1.0 / 39916800.0);
  p = fma(z, p, 1.0 / 362880.0);
  p = fma(z, p, -1.0 / 5040.0);
  p = fma(z, p, 1.0 / 120.0);
  p = fma(z, p, -1.0 / 6.0);
  const double sr = fma(r * z, p, r);
  double q = fma(z, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  q = fma(z, q, 1.0 / 479001600.0);
  q = fma(z, q, -1.0 / 3628800.0);
  q = fma(z, q, 1.0 / 40320.0);
  q = fma(z, q, -1.0 / 720.0);
  q = fma(z, q, 1.0 / 24.0);
  q = fma(z, q, -0.5);
  const double cr = fma(z, q, 1.0);
  const int k = (int)((long long)n & 3);
  const double u = (k & 1) ? sr : cr, v = (k & 1) ? cr : sr;
  c = (k == 1 || k == 2) ? -u : u;
  s = (k >= 2) ? -v : v;
}

// Where a paged cache lives: pool of num_blocks pages, block_table [B][max_blocks].
struct Pages {
  uint8_t* pool;
  const int* table;
  int max_blocks, block_rows, num_blocks, Hkv;
};
// The tile of position pos of sequence b and kv head h; null when the table
// names no page of the pool.
template <int D>
__device__ __forceinline__ uint8_t* tile_of(const Pages& pg, int b, int pos, int h) {
  const int blk = __ldg(pg.table + (size_t)b * pg.max_blocks + pos / pg.block_rows);
  if (blk < 0 || blk >= pg.num_blocks) return nullptr;
  const int tpb = pg.block_rows / kTileKeys;
  return pg.pool + (((size_t)blk * pg.Hkv + h) * tpb + (pos % pg.block_rows) / kTileKeys) *
                       Tile<D>::kBytes;
}

}  // namespace kv4
}  // namespace dca
