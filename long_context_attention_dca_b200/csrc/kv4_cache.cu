// Writing to and reading from the paged 4-bit key/value cache (kv4.cuh).
//
// Append: packed new tokens (sequence b at rows cu_seqlens[b] ..
// cu_seqlens[b+1]-1, absolute index t0[b] + local row).  A key is rotated at
// its index mod s and rounded once to bf16, exactly as the bf16 caches store
// it, then quantised; a value is quantised as it is.  Both roundings are those
// of the exact result: the rotation runs in fp32 on operands split so that its
// error is a few 2^-24 of the result, and an element that comes that close to
// the border between two bf16 values, or a quotient that close to the border
// between two codes, is decided again in fp64.  A step of the 4-bit grid is a
// tenth of a typical value, so without this two builds of the same cache could
// differ visibly.
//
// Mapping: D/16 lanes own one (token, kv head) row; lane i holds dims 8i .. 8i+7
// and their rotation partners D/2 further on, i.e. one code word of either
// half, and its eight angles serve all kv heads the thread walks.
#include "dca_common.cuh"
#include "dca_kernels.cuh"
#include "kv4.cuh"

namespace dca {
namespace kv4 {

constexpr int kThreads = 256;

// A double rounded once to bf16 (nearest even): to fp32 toward zero with the
// lost bits kept as a sticky last bit, which the second rounding cannot confuse
// with a tie.
__device__ __forceinline__ uint32_t bf16_bits_of(double x) {
  const float f = __double2float_rz(x);
  uint32_t b = __float_as_uint(f);
  if ((double)f != x && (b & 0x7F800000u) != 0x7F800000u) b |= 1u;
  return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(b)));
}

// A float with a 16-bit significand and the rest, of a double in [-1, 1].
__device__ __forceinline__ void split16(double x, float& hi, float& lo) {
  hi = __uint_as_float(__float_as_uint((float)x) & 0xFFFFFF00u);
  lo = (float)(x - (double)hi);
}

// True when y may lie within `tol` of the midpoint of two bf16 values.
__device__ __forceinline__ bool near_bf16_border(float y, float tol) {
  const float mid = __uint_as_float((__float_as_uint(y) & 0xFFFF0000u) | 0x8000u);
  return fabsf(y - mid) <= tol;
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) {
  return *reinterpret_cast<__nv_bfloat162*>(&w);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}

// (least, -greatest) of 8 bf16 values as a bf16 pair; NaN if any is NaN.
__device__ __forceinline__ uint32_t min_negmax(const uint32_t (&w)[4]) {
  const __nv_bfloat162 a = __hmin2_nan(__hmin2_nan(as_bf162(w[0]), as_bf162(w[1])),
                                       __hmin2_nan(as_bf162(w[2]), as_bf162(w[3])));
  const __nv_bfloat162 b = __hmax2_nan(__hmax2_nan(as_bf162(w[0]), as_bf162(w[1])),
                                       __hmax2_nan(as_bf162(w[2]), as_bf162(w[3])));
  const uint32_t ua = as_u32(a), ub = as_u32(b) ^ 0x80008000u;
  // (a.lo, -b.lo) against (a.hi, -b.hi)
  const uint32_t lo = __byte_perm(ua, ub, 0x5410), hi = __byte_perm(ua, ub, 0x7632);
  return as_u32(__hmin2_nan(as_bf162(lo), as_bf162(hi)));
}

struct Params {
  float off, scale;  // bf16 values
  float k1, k0;      // quotient = x * k1 + k0
  float tol;         // how close to a border the fp32 quotient decides nothing
  uint32_t word;     // as stored
};
// Parameters of a group from its (least, -greatest).
__device__ __forceinline__ Params make_params(uint32_t mm) {
  Params p;
  // (-0 becomes 0, so that a stored parameter never carries a stray sign)
  const float lo = __fadd_rn(bf16_lo(mm), 0.f), hi = __fadd_rn(-bf16_hi(mm), 0.f);
  // halves, so that the range of any two finite bf16 stays finite; rounded up
  // twice in fp32 and then to bf16, which gives the smallest bf16 >= range / 15
  // (15 * bf16 fits fp32, so no intermediate step can jump over it)
  const float r = __fdiv_ru(__fsub_ru(hi * 0.5f, lo * 0.5f), 7.5f);
  const uint32_t sb = (__float_as_uint(r) + 0xFFFFu) & 0xFFFF0000u;
  p.off = lo;
  p.scale = __uint_as_float(sb);
  if (!(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY)) {
    p.word = 0x7FFF7FFFu;
    p.k1 = p.k0 = p.tol = 0.f;
    return p;
  }
  const bool plain = p.scale >= 1e-30f;
  const float inv = plain ? 1.f / p.scale : 0.f;
  p.k1 = inv;
  p.k0 = -(lo * inv);
  // |error of the quotient| <= 2^-24 (3 |k0| + 31); a scale whose reciprocal
  // could overflow leaves every element to the exact rule
  p.tol = plain ? fmaf(fabsf(p.k0), 4e-7f, 8e-6f) : (p.scale > 0.f ? INFINITY : 0.f);
  p.word = (sb >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
  return p;
}

// Code of x in exact arithmetic.  off, scale and x are bf16, so -off - (n+.5)
// scale is exact in fp64 and the last addition keeps the sign of the real sum.
__device__ __forceinline__ uint32_t exact_code(float x, const Params& p) {
  if (!(p.scale > 0.f)) return 0u;
  const double q = ((double)x - (double)p.off) / (double)p.scale;
  int n = (int)q;  // q in [0, 15]
  n = max(0, min(n, 14));
  // the border nearest to q is n + 0.5 for n = floor(q)
  const double d = (double)x + (-(double)p.off - ((double)n + 0.5) * (double)p.scale);
  return d > 0.0 ? n + 1 : (d < 0.0 ? n : n + (n & 1));
}

// Eight values (four bf16 pairs) to a code word.
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&w)[4], const Params& p) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: rounds to an integer
  float c[8], far = 0.f;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const float x = (n & 1) ? bf16_hi(w[n >> 1]) : bf16_lo(w[n >> 1]);
    const float q = fmaf(x, p.k1, p.k0);
    c[n] = __fsub_rn(__fadd_rn(q, kMagic), kMagic);
    far = fmaxf(far, fabsf(q - c[n]));
  }
  if (far < 0.5f - p.tol) {
    const float lo = fmaf(c[3], 4096.f, fmaf(c[2], 256.f, fmaf(c[1], 16.f, c[0])));
    const float hi = fmaf(c[7], 4096.f, fmaf(c[6], 256.f, fmaf(c[5], 16.f, c[4])));
    return (uint32_t)__float2uint_rz(lo) | ((uint32_t)__float2uint_rz(hi) << 16);
  }
  uint32_t out = 0;
  if (p.word == 0x7FFF7FFFu) return out;
#pragma unroll 1
  for (int n = 0; n < 8; ++n) {
    const uint32_t pair = n < 4 ? (n < 2 ? w[0] : w[1]) : (n < 6 ? w[2] : w[3]);
    out |= exact_code((n & 1) ? bf16_hi(pair) : bf16_lo(pair), p) << (4 * n);
  }
  return out;
}

// Packed row r: its sequence b and absolute index, or b = -1 for a row of no
// sequence and for one whose span does not fit the cache.
struct RowAt {
  int b, pos;
};
__device__ __forceinline__ RowAt locate(int r, int T, const int* cu, const int* t0, int B,
                                        long long cap) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  const int a = __ldg(cu + lo), e = __ldg(cu + lo + 1), first = __ldg(t0 + lo);
  RowAt at{-1, 0};
  if (a < 0 || r < a || r >= e || e > T) return at;
  if (first < 0 || (long long)first + (e - a) > cap) return at;
  at.b = lo;
  at.pos = first + (r - a);
  return at;
}
// The packed offsets as a whole, by the first block: a fault is reported once.
__device__ __forceinline__ void check_offsets(int T, const int* cu, const int* t0, int B,
                                              long long cap) {
  bool bad = false;
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int a = __ldg(cu + b), e = __ldg(cu + b + 1), first = __ldg(t0 + b);
    bad |= a < 0 || e < a || e > T || first < 0 || (long long)first + ((long long)e - a) > cap;
  }
  if (bad) report_error(kDevBadArg, 204);
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(
    const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new, Pages pg,
    const int* __restrict__ cu, const int* __restrict__ t0, int B, int T, int s,
    int heads_per_cta, const __grid_constant__ Theta theta) {
  using TL = Tile<D>;
  constexpr int kLanes = D / 16;  // lanes of a row
  const long long cap = (long long)pg.max_blocks * pg.block_rows;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(T, cu, t0, B, cap);
  const int i = threadIdx.x % kLanes;
  const int row = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  RowAt at{-1, 0};
  if (row < T) at = locate(row, T, cu, t0, B, cap);
  const int pos = at.pos % s;
  float c1[8], c2[8], s1[8], s2[8];
  if (at.b >= 0) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      double c, sn;
      sincos64((double)pos * theta.v[8 * i + n], c, sn);
      split16(c, c1[n], c2[n]);
      split16(sn, s1[n], s2[n]);
    }
  }
  const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, pg.Hkv);
  const unsigned lanes = 0xFFFFFFFFu;
  for (int h = h0; h < h1; ++h) {
    uint32_t k[2][4] = {}, v[2][4] = {};
    const size_t src = ((size_t)row * pg.Hkv + h) * D + 8 * i;
    if (at.b >= 0) {
      const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(k_new + src));
      const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(k_new + src + D / 2));
      const uint4 y0 = __ldg(reinterpret_cast<const uint4*>(v_new + src));
      const uint4 y1 = __ldg(reinterpret_cast<const uint4*>(v_new + src + D / 2));
      v[0][0] = y0.x, v[0][1] = y0.y, v[0][2] = y0.z, v[0][3] = y0.w;
      v[1][0] = y1.x, v[1][1] = y1.y, v[1][2] = y1.z, v[1][3] = y1.w;
      const uint32_t a[4] = {x0.x, x0.y, x0.z, x0.w}, b[4] = {x1.x, x1.y, x1.z, x1.w};
      uint32_t again = 0;  // elements next to a border, by pair
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        float o0[2], o1[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float p = u ? bf16_hi(a[n / 2]) : bf16_lo(a[n / 2]);
          const float q = u ? bf16_hi(b[n / 2]) : bf16_lo(b[n / 2]);
          const int m = n + u;
          // products with the 16-bit parts are exact in fp32
          o0[u] = fmaf(p, c1[m], -(q * s1[m])) + fmaf(p, c2[m], -(q * s2[m]));
          o1[u] = fmaf(q, c1[m], p * s1[m]) + fmaf(q, c2[m], p * s2[m]);
          const float tiny = (fabsf(p) + fabsf(q)) * 1e-11f;
          if (near_bf16_border(o0[u], fmaf(fabsf(o0[u]), 2.4e-7f, tiny)) ||
              near_bf16_border(o1[u], fmaf(fabsf(o1[u]), 2.4e-7f, tiny)))
            again |= 1u << m;
        }
        k[0][n / 2] = pack_bf16(o0[0], o0[1]);
        k[1][n / 2] = pack_bf16(o1[0], o1[1]);
      }
      while (again) {
        const int m = __ffs(again) - 1;
        again &= again - 1;
        double c, sn;
        sincos64((double)pos * theta.v[8 * i + m], c, sn);
        const double p = (double)__bfloat162float(k_new[src + m]);
        const double q = (double)__bfloat162float(k_new[src + D / 2 + m]);
        const int sh = (m & 1) * 16;
        const uint32_t keep = ~(0xFFFFu << sh);
        const uint32_t z0 = bf16_bits_of(fma(p, c, -(q * sn))) << sh;
        const uint32_t z1 = bf16_bits_of(fma(q, c, p * sn)) << sh;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j == m / 2) {
            k[0][j] = (k[0][j] & keep) | z0;
            k[1][j] = (k[1][j] & keep) | z1;
          }
        }
      }
    }
    // ranges of the groups: D = 128 has a group in either half, D = 64 one over both
    uint32_t mk[2] = {min_negmax(k[0]), min_negmax(k[1])};
    uint32_t mv[2] = {min_negmax(v[0]), min_negmax(v[1])};
    if (D == 64) {
      mk[0] = mk[1] = as_u32(__hmin2_nan(as_bf162(mk[0]), as_bf162(mk[1])));
      mv[0] = mv[1] = as_u32(__hmin2_nan(as_bf162(mv[0]), as_bf162(mv[1])));
    }
#pragma unroll
    for (int sh = kLanes / 2; sh >= 1; sh >>= 1) {
#pragma unroll
      for (int g = 0; g < TL::kGroups; ++g) {
        mk[g] = as_u32(__hmin2_nan(as_bf162(mk[g]), as_bf162(__shfl_xor_sync(lanes, mk[g], sh))));
        mv[g] = as_u32(__hmin2_nan(as_bf162(mv[g]), as_bf162(__shfl_xor_sync(lanes, mv[g], sh))));
      }
    }
    if (at.b < 0) continue;
    uint8_t* tile = tile_of<D>(pg, at.b, at.pos, h);
    if (tile == nullptr) {
      if (i == 0 && h == h0) report_error(kDevBadArg, 205);
      continue;
    }
    const int r = at.pos % kTileKeys;
#pragma unroll
    for (int g = 0; g < TL::kGroups; ++g) {
      const Params pk = make_params(mk[g]), pv = make_params(mv[g]);
      if (i == g) {
        *reinterpret_cast<uint32_t*>(tile + TL::k_param(r, g)) = pk.word;
        *reinterpret_cast<uint32_t*>(tile + TL::v_param(r, g)) = pv.word;
      }
#pragma unroll
      for (int half = g; half < 2; half += TL::kGroups) {
        const int word = D == 128 ? i : i + 4 * half;
        *reinterpret_cast<uint32_t*>(tile + TL::k_word(r, g, word)) = quantise8(k[half], pk);
        *reinterpret_cast<uint32_t*>(tile + TL::v_word(r, g, word)) = quantise8(v[half], pv);
      }
    }
  }
}

// Rows of the cache back as bf16: the stored keys (rotated) and values, to
// packed rows [T][Hkv][D], or with out_rows > 0 to row `index` of entry b of
// [B][out_rows][Hkv][D].  code * scale + offset is formed in fp32, where it is
// exact unless the offset is over 2^11 steps away, and rounded once.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(
    __nv_bfloat16* __restrict__ Ko, __nv_bfloat16* __restrict__ Vo, Pages pg,
    const int* __restrict__ cu, const int* __restrict__ t0, int B, int T, int out_rows) {
  using TL = Tile<D>;
  constexpr int kLanes = D / 16;
  const long long cap = out_rows > 0
                            ? min((long long)pg.max_blocks * pg.block_rows, (long long)out_rows)
                            : (long long)pg.max_blocks * pg.block_rows;
  if (blockIdx.x == 0) check_offsets(T, cu, t0, B, cap);
  const long long gid = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int i = threadIdx.x % kLanes;
  if (gid >= (long long)T * pg.Hkv) return;
  // heads outermost inside a run of rows, so that a block reads whole tiles
  const int run = 64;
  const long long per = (long long)run * pg.Hkv;
  const int r0 = (int)(gid / per) * run, n = min(run, T - r0);
  const int h = (int)((gid % per) / n), row = r0 + (int)((gid % per) % n);
  const RowAt at = locate(row, T, cu, t0, B, cap);
  if (at.b < 0) return;
  const uint8_t* tile = tile_of<D>(pg, at.b, at.pos, h);
  if (tile == nullptr) {
    if (i == 0 && h == 0) report_error(kDevBadArg, 206);
    return;
  }
  const int r = at.pos % kTileKeys;
  const long long orow = out_rows > 0 ? (long long)at.b * out_rows + at.pos : row;
  const size_t dst = ((size_t)orow * pg.Hkv + h) * D + 8 * i;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int g = D == 128 ? half : 0, word = D == 128 ? i : i + 4 * half;
    const uint32_t wk = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::k_word(r, g, word)));
    const uint32_t wv = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::v_word(r, g, word)));
    const uint32_t pk = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::k_param(r, g)));
    const uint32_t pv = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::v_param(r, g)));
    uint32_t k[4], v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a0 = (float)((wk >> (8 * j)) & 15u), a1 = (float)((wk >> (8 * j + 4)) & 15u);
      const float b0 = (float)((wv >> (8 * j)) & 15u), b1 = (float)((wv >> (8 * j + 4)) & 15u);
      k[j] = pack_bf16(fmaf(a0, bf16_lo(pk), bf16_hi(pk)), fmaf(a1, bf16_lo(pk), bf16_hi(pk)));
      v[j] = pack_bf16(fmaf(b0, bf16_lo(pv), bf16_hi(pv)), fmaf(b1, bf16_lo(pv), bf16_hi(pv)));
    }
    *reinterpret_cast<uint4*>(Ko + dst + half * (D / 2)) = make_uint4(k[0], k[1], k[2], k[3]);
    *reinterpret_cast<uint4*>(Vo + dst + half * (D / 2)) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

template <int D>
cudaError_t launch_append_t(const void* k_new, const void* v_new, const Pages& pg, const int* cu,
                            const int* t0, int B, int T, int s, float base, cudaStream_t stream) {
  constexpr int kRows = kThreads / (D / 16);
  const unsigned gx = (unsigned)((T + kRows - 1) / kRows);
  // The angles of a row serve all heads of a block, so a block takes as many
  // heads as leave 4 blocks an SM.
  int hpc = pg.Hkv;
  while (hpc > 1 && (long long)gx * ((pg.Hkv + hpc - 1) / hpc) < 148 * 4) hpc = (hpc + 1) / 2;
  const unsigned gy = (unsigned)((pg.Hkv + hpc - 1) / hpc);
  append_kernel<D><<<dim3(gx, gy), kThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new), pg, cu,
      t0, B, T, s, hpc, make_theta(D, base));
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_read_t(void* K, void* V, const Pages& pg, const int* cu, const int* t0, int B,
                          int T, int out_rows, cudaStream_t stream) {
  constexpr int kRows = kThreads / (D / 16);
  const unsigned grid = (unsigned)(((long long)T * pg.Hkv + kRows - 1) / kRows);
  read_kernel<D><<<grid, kThreads, 0, stream>>>(static_cast<__nv_bfloat16*>(K),
                                                static_cast<__nv_bfloat16*>(V), pg, cu, t0, B, T,
                                                out_rows);
  return cudaGetLastError();
}

}  // namespace kv4

cudaError_t launch_kv4_append(const void* k_new, const void* v_new, void* pool,
                              const int* block_table, int max_blocks, int block_rows,
                              int num_blocks, const int* cu, const int* t0, int B, int T, int Hkv,
                              int D, int s, float base, cudaStream_t stream) {
  const kv4::Pages pg{static_cast<uint8_t*>(pool), block_table, max_blocks, block_rows,
                      num_blocks, Hkv};
  return D == 64 ? kv4::launch_append_t<64>(k_new, v_new, pg, cu, t0, B, T, s, base, stream)
                 : kv4::launch_append_t<128>(k_new, v_new, pg, cu, t0, B, T, s, base, stream);
}

cudaError_t launch_kv4_read(const void* pool, const int* block_table, int max_blocks,
                            int block_rows, int num_blocks, const int* cu, const int* t0,
                            void* K, void* V, int B, int T, int Hkv, int D, int out_rows,
                            cudaStream_t stream) {
  const kv4::Pages pg{static_cast<uint8_t*>(const_cast<void*>(pool)), block_table, max_blocks,
                      block_rows, num_blocks, Hkv};
  return D == 64 ? kv4::launch_read_t<64>(K, V, pg, cu, t0, B, T, out_rows, stream)
                 : kv4::launch_read_t<128>(K, V, pg, cu, t0, B, T, out_rows, stream);
}

}  // namespace dca
