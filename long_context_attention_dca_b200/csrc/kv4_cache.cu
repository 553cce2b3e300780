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
//
// What bounds it: instructions, not memory.  34816 rows of 8 heads of 128 (182 MB
// in and out, 28 us at the copy rate) take 74 us, with an instruction issued in
// 0.69 of the cycles: about 775 a warp for 4 rows of K and V, 24 a value.  Of the
// 74, the tests of the rotation's roundings cost 2, those of the codes 8, both 12, and
// the second part of the angles 2 more (timed without each, results then not
// exact); loads, stores and the groups' ranges alone take 34.  What is left, some 26
// us, is the arithmetic of the rotation and of the quantiser itself.  Packed pairs
// of fp32 (two elements an instruction) and the fp64 path behind a test are what
// brought it there from 226 us.  Reading back the same rows takes 37 us, 4.9 TB/s:
// the logic pipe, which takes the nibbles apart, is busy for 71 % of it and an
// instruction is issued in 0.71 of the cycles, so that memory is not alone.
#include "dca_common.cuh"
#include "dca_kernels.cuh"
#include "kv4.cuh"

namespace dca {
namespace kv4 {

constexpr int kThreads = 64;  // small blocks fill the last wave: against 128, 23 -> 21 us for
                              // 3525 rows of 32 heads of 64, the same for the case above

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

// Two results rounded to bf16, and where their errors leave that open: bits that
// differ between the roundings of the two ends.  Errors below 2.9 * 2^-24 of a
// result, and the widening's own 2^-24, fit the factors, 1 +- 4 * 2^-24.
__device__ __forceinline__ uint32_t rounded(uint64_t y, uint32_t& open) {
  float a, b, c, d;
  f2_unpack(f2_mul(y, f2_pack(1.00000024f, 1.00000024f)), a, b);
  f2_unpack(f2_mul(y, f2_pack(0.99999976f, 0.99999976f)), c, d);
  const uint32_t one = pack_bf16(a, b), other = pack_bf16(c, d);
  open = one ^ other;
  return one;
}

struct Params {
  float off, scale;     // halves of the bf16 values: ranges of any size stay finite
  float inv;            // 1 / scale (of the halves)
  uint32_t word;        // as stored
};
// 1 / x within a few last places (quantise8 corrects the quotient); infinite for
// a subnormal x.
__device__ __forceinline__ float approx_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Parameters of a group from its (least, -greatest).
__device__ __forceinline__ Params make_params(uint32_t mm) {
  Params p;
  // (-0 becomes 0, so that a stored parameter never carries a stray sign)
  const float lo = __fadd_rn(bf16_lo(mm), 0.f), hi = __fadd_rn(-bf16_hi(mm), 0.f);
  // The smallest bf16 b with 15 b >= the range: from an approximate quotient cut
  // to bf16, stepped up while 7.5 b, exact in fp32, is below half the range.
  const float range = __fsub_ru(hi * 0.5f, lo * 0.5f);
  uint32_t sb = __float_as_uint(range * (1.f / 7.5f)) & 0xFFFF0000u;
  if (__uint_as_float(sb) * 7.5f < range) sb += 0x10000u;
  if (__uint_as_float(sb) * 7.5f < range) sb += 0x10000u;
  p.off = lo * 0.5f;
  p.scale = __uint_as_float(sb) * 0.5f;
  p.inv = p.scale > 0.f ? approx_rcp(p.scale) : 0.f;
  p.word = (sb >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
  if (!(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY)) {  // codes 0 (of x = 0 and of NaN)
    p.word = 0x7FFF7FFFu;
    p.off = p.scale = p.inv = 0.f;
  }
  return p;
}

// Codes of eight values in exact arithmetic: off, scale and x are bf16 halves, so
// -off - (n + .5) scale is exact in fp64 and the last addition keeps the sign of
// the real sum.
__device__ __noinline__ uint32_t mend_codes(uint4 v, float off, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out = 0;
  for (int i = 0; i < 8; ++i) {
    const uint32_t pair = i < 4 ? (i < 2 ? w[0] : w[1]) : (i < 6 ? w[2] : w[3]);
    const double x = 0.5 * (double)((i & 1) ? bf16_hi(pair) : bf16_lo(pair));
    const int n = max(0, min((int)((x - (double)off) / (double)scale), 14));
    const double d = x + (-(double)off - ((double)n + 0.5) * (double)scale);
    out |= (uint32_t)(d > 0.0 ? n + 1 : (d < 0.0 ? n : n + (n & 1))) << (4 * i);
  }
  return out;
}

// Eight values (four bf16 pairs) to a code word.  With d = x - off, the quotient
// from the reciprocal and one correction is an exact half wherever d / scale is
// one, so rounding it to even is right on every border that d reaches exactly;
// and c is right whenever the remainder d - c * scale, which the fused
// multiply-add forms exactly, is at most half a step.  What is left is mended: a
// quotient next to a border, and a border that d reached only by rounding (|x|
// far below |off|; a zero among the values counts as one, which costs time only).
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&w)[4], const Params& p) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: rounds to an integer
  const uint64_t off2 = f2_pack(-p.off, -p.off), inv2 = f2_pack(p.inv, p.inv);
  const uint64_t neg_scale2 = f2_pack(-p.scale, -p.scale), half2 = f2_pack(0.5f, 0.5f);
  const uint64_t magic2 = f2_pack(kMagic, kMagic);
  uint64_t c2[4];
  float far = 0.f;
#pragma unroll
  for (int n = 0; n < 4; ++n) {  // two elements an instruction
    const uint64_t x = f2_pack(bf16_lo(w[n]), bf16_hi(w[n]));
    const uint64_t d = f2_fma(x, half2, off2);
    uint64_t q = f2_mul(d, inv2);
    q = f2_fma(f2_fma(q, neg_scale2, d), inv2, q);
    c2[n] = f2_sub(f2_add(q, magic2), magic2);
    float r0, r1;
    f2_unpack(f2_fma(c2[n], neg_scale2, d), r0, r1);
    far = fmax3(far, fabsf(r0), fabsf(r1));
  }
  const float half = 0.5f * p.scale;
  if (half > 0.f && (far >= half || p.inv == INFINITY)) {
    // Only a value far below the offset makes d inexact, which matters on a border.
    const __nv_bfloat162 least =
        __hmin2(__hmin2(__habs2(as_bf162(w[0])), __habs2(as_bf162(w[1]))),
                __hmin2(__habs2(as_bf162(w[2])), __habs2(as_bf162(w[3]))));
    const bool small = fminf(bf16_lo(as_u32(least)), bf16_hi(as_u32(least))) <
                       fabsf(p.off) * 1.220703125e-4f;  // 2^-13 of half the offset
    // (an infinite reciprocal: a subnormal scale)
    if (far > half || small || p.inv == INFINITY)
      return mend_codes(make_uint4(w[0], w[1], w[2], w[3]), p.off, p.scale);
  }
  // c0 + 16 c1 + 256 c2 + 4096 c3 on 2^23, whose low half is the integer
  float a0, a1, b0, b1, lo, hi;
  const uint64_t by256 = f2_pack(256.f, 256.f);
  f2_unpack(f2_fma(c2[1], by256, c2[0]), a0, a1);
  f2_unpack(f2_fma(c2[3], by256, c2[2]), b0, b1);
  lo = fmaf(a1, 16.f, a0 + 8388608.f);
  hi = fmaf(b1, 16.f, b0 + 8388608.f);
  // (no scale: a constant group, or one that is not finite, whose sums are NaN)
  return half > 0.f ? __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410) : 0u;
}

// Packed row r: its sequence b and absolute index, or b = -1 for a row of no
// sequence and for one whose span does not fit the cache.
struct RowAt {
  int b, pos;
};
__device__ __forceinline__ RowAt locate(int r, int T, const int* cu, const int* t0, int B,
                                        long long cap) {
  // with one new token a sequence, row r is sequence r's
  int lo = 0, hi = B - 1;
  if (r < B && __ldg(cu + r) <= r && r < __ldg(cu + r + 1)) lo = hi = r;
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
// The packed offsets as a whole, by one block.
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
  if (blockIdx.x == gridDim.x - 1) {  // a block of its own, beside the work
    if (blockIdx.y == 0) check_offsets(T, cu, t0, B, cap);
    return;
  }
  const int i = threadIdx.x % kLanes;
  const int row = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  // this head's rows, fetched one head ahead
  uint4 x0 = {}, x1 = {}, y0 = {}, y1 = {};
  auto load = [&](int h) {
    const size_t from = ((size_t)row * pg.Hkv + h) * D + 8 * i;
    x0 = __ldg(reinterpret_cast<const uint4*>(k_new + from));
    x1 = __ldg(reinterpret_cast<const uint4*>(k_new + from + D / 2));
    y0 = __ldg(reinterpret_cast<const uint4*>(v_new + from));
    y1 = __ldg(reinterpret_cast<const uint4*>(v_new + from + D / 2));
  };
  const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, pg.Hkv);
  if (row < T) load(h0);
  RowAt at{-1, 0};
  if (row < T) at = locate(row, T, cu, t0, B, cap);
  const int pos = at.pos % s;
  // cos and sin of two angles each, in two parts: the thread's own, kept in
  // shared memory, which leaves registers for more warps
  __shared__ ulonglong2 turn[4][2][kThreads];
  if (at.b >= 0) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float ch[2], cl[2], sh[2], sl[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        double c, sn;
        sincos64((double)pos * theta.v[8 * i + 2 * n + u], c, sn);
        split16(c, ch[u], cl[u]);
        split16(sn, sh[u], sl[u]);
      }
      turn[n][0][threadIdx.x] = make_ulonglong2(f2_pack(ch[0], ch[1]), f2_pack(cl[0], cl[1]));
      turn[n][1][threadIdx.x] = make_ulonglong2(f2_pack(sh[0], sh[1]), f2_pack(sl[0], sl[1]));
    }
  }
  // the row's place in the tile of head 0
  uint8_t* tile0 = nullptr;
  if (at.b >= 0) {
    tile0 = tile_of<D>(pg, at.b, at.pos, 0);
    if (tile0 == nullptr) {
      if (i == 0 && blockIdx.y == 0) report_error(kDevBadArg, 205);
      at.b = -1;
    }
  }
  const int r = at.pos % kTileKeys;
  const size_t head_bytes = (size_t)(pg.block_rows / kTileKeys) * TL::kBytes;
  const unsigned lanes = 0xFFFFFFFFu;
  for (int h = h0; h < h1; ++h) {
    uint32_t k[2][4] = {}, v[2][4] = {};
    const size_t src = ((size_t)row * pg.Hkv + h) * D + 8 * i;
    if (at.b >= 0) {
      v[0][0] = y0.x, v[0][1] = y0.y, v[0][2] = y0.z, v[0][3] = y0.w;
      v[1][0] = y1.x, v[1][1] = y1.y, v[1][2] = y1.z, v[1][3] = y1.w;
      const uint32_t a[4] = {x0.x, x0.y, x0.z, x0.w}, b[4] = {x1.x, x1.y, x1.z, x1.w};
      if (h + 1 < h1) load(h + 1);
      uint32_t again = 0;  // elements next to a border, by pair
#pragma unroll
      for (int n = 0; n < 4; ++n) {  // two elements an instruction
        const uint64_t p2 = f2_pack(bf16_lo(a[n]), bf16_hi(a[n]));
        const uint64_t q2 = f2_pack(bf16_lo(b[n]), bf16_hi(b[n]));
        const uint64_t n2 = f2_pack(bf16_lo(b[n] ^ 0x80008000u), bf16_hi(b[n] ^ 0x80008000u));
        const ulonglong2 c = turn[n][0][threadIdx.x], sn = turn[n][1][threadIdx.x];
        // products with the 16-bit parts are exact in fp32
        uint32_t b0, b1;  // not 0 next to a border
        const uint64_t o0 = f2_add(f2_fma(p2, c.x, f2_mul(n2, sn.x)),
                                   f2_fma(p2, c.y, f2_mul(n2, sn.y)));
        const uint64_t o1 = f2_add(f2_fma(q2, c.x, f2_mul(p2, sn.x)),
                                   f2_fma(q2, c.y, f2_mul(p2, sn.y)));
        k[0][n] = rounded(o0, b0);
        k[1][n] = rounded(o1, b1);
        // The errors are 2^-24 of the first sum, 3 * 2^-39 of the operands for the
        // second and 2^-24 for the last addition: under 2.76 * 2^-24 of a result that
        // is above 2^-13 of its operands.  One below that is a border too.
        const __nv_bfloat162 size = __hadd2(__habs2(as_bf162(a[n])), __habs2(as_bf162(b[n])));
        const __nv_bfloat162 much = __float2bfloat162_rn(8192.f);
        b0 |= as_u32(__hsub2(__hmul2(__habs2(as_bf162(k[0][n])), much), size)) & 0x80008000u;
        b1 |= as_u32(__hsub2(__hmul2(__habs2(as_bf162(k[1][n])), much), size)) & 0x80008000u;
        if (b0 | b1) again |= 1u << n;
      }
      while (again) {  // both elements of the pair once more, in fp64
        const int n = __ffs(again) - 1;
        again &= again - 1;
        uint32_t z0 = 0, z1 = 0;
        for (int u = 0; u < 2; ++u) {
          double c, sn;
          sincos64((double)pos * theta.v[8 * i + 2 * n + u], c, sn);
          const double p = (double)__bfloat162float(k_new[src + 2 * n + u]);
          const double q = (double)__bfloat162float(k_new[src + D / 2 + 2 * n + u]);
          z0 |= bf16_bits_of(fma(p, c, -(q * sn))) << (16 * u);
          z1 |= bf16_bits_of(fma(q, c, p * sn)) << (16 * u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j == n) {
            k[0][j] = z0;
            k[1][j] = z1;
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
    // Every group's parameters are the same in all lanes of the row: lane j forms
    // those of group j (keys first), the others take them from it.
    const int j = i % (2 * TL::kGroups);
    const Params own = make_params(j < TL::kGroups ? mk[j % TL::kGroups] : mv[j % TL::kGroups]);
    uint8_t* tile = tile0 + h * head_bytes;
    if (at.b >= 0 && i < 2 * TL::kGroups)
      *reinterpret_cast<uint32_t*>(tile + (i < TL::kGroups ? TL::k_param(r, i)
                                                           : TL::v_param(r, i - TL::kGroups))) =
          own.word;
#pragma unroll
    for (int g = 0; g < 2 * TL::kGroups; ++g) {
      Params p;
      p.off = __shfl_sync(lanes, own.off, g, kLanes);
      p.scale = __shfl_sync(lanes, own.scale, g, kLanes);
      p.inv = __shfl_sync(lanes, own.inv, g, kLanes);
      const int gr = g % TL::kGroups;
      const bool key = g < TL::kGroups;
#pragma unroll
      for (int half = gr; half < 2; half += TL::kGroups) {
        const int word = D == 128 ? i : i + 4 * half;
        const uint32_t codes = quantise8(key ? k[half] : v[half], p);
        if (at.b >= 0)
          *reinterpret_cast<uint32_t*>(tile + (key ? TL::k_word(r, gr, word)
                                                   : TL::v_word(r, gr, word))) = codes;
      }
    }
  }
}

// The eight values of a code word as bf16 pairs: code * scale + offset in fp32,
// where it is exact unless the offset is over 2^11 steps away, rounded once.  A
// nibble masked in place under the exponent of 2^23 is 2^23 + c * 16^n, so the
// code comes out by a subtraction and its place goes into the scale.
__device__ __forceinline__ void dequantise8(uint32_t w, uint32_t param, uint32_t (&out)[4]) {
  const float scale = bf16_lo(param), off = bf16_hi(param);
  const uint64_t off2 = f2_pack(off, off), base2 = f2_pack(8388608.f, 8388608.f);
  const uint64_t s01 = f2_pack(scale, scale * 0.0625f);
  const uint64_t s23 = f2_pack(scale * 0.00390625f, scale * 0.000244140625f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t u = w >> (16 * j);
    const uint64_t c01 = f2_pack(__uint_as_float((u & 0xFu) | 0x4B000000u),
                                 __uint_as_float((u & 0xF0u) | 0x4B000000u));
    const uint64_t c23 = f2_pack(__uint_as_float((u & 0xF00u) | 0x4B000000u),
                                 __uint_as_float((u & 0xF000u) | 0x4B000000u));
    float a, b;
    f2_unpack(f2_fma(f2_sub(c01, base2), s01, off2), a, b);
    out[2 * j] = pack_bf16(a, b);
    f2_unpack(f2_fma(f2_sub(c23, base2), s23, off2), a, b);
    out[2 * j + 1] = pack_bf16(a, b);
  }
}

// Rows of the cache back as bf16: the stored keys (rotated) and values, to
// packed rows [T][Hkv][D], or with out_rows > 0 to row `index` of entry b of
// [B][out_rows][Hkv][D].  code * scale + offset is formed in fp32, where it is
// exact unless the offset is over 2^11 steps away, and rounded once.
// One block a (run of rows, kv head), so that it reads whole tiles; a thread
// takes kReadRows rows of the run, all their loads in flight at once (one row: 39 us
// for the case above; two: 37).
constexpr int kReadRows = 2;

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(
    __nv_bfloat16* __restrict__ Ko, __nv_bfloat16* __restrict__ Vo, Pages pg,
    const int* __restrict__ cu, const int* __restrict__ t0, int B, int T, int out_rows) {
  using TL = Tile<D>;
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;
  const long long cap = out_rows > 0
                            ? min((long long)pg.max_blocks * pg.block_rows, (long long)out_rows)
                            : (long long)pg.max_blocks * pg.block_rows;
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) check_offsets(T, cu, t0, B, cap);
    return;
  }
  const int i = threadIdx.x % kLanes, h = blockIdx.y;
  size_t dst[kReadRows];
  uint32_t w[kReadRows][2][4];
  bool live[kReadRows];
#pragma unroll
  for (int n = 0; n < kReadRows; ++n) {
    const int row = (blockIdx.x * kReadRows + n) * kRows + threadIdx.x / kLanes;
    live[n] = false;
    if (row >= T) continue;
    const RowAt at = locate(row, T, cu, t0, B, cap);
    if (at.b < 0) continue;
    const uint8_t* tile = tile_of<D>(pg, at.b, at.pos, h);
    if (tile == nullptr) {
      if (i == 0 && h == 0) report_error(kDevBadArg, 206);
      continue;
    }
    const int r = at.pos % kTileKeys;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int g = D == 128 ? half : 0, word = D == 128 ? i : i + 4 * half;
      w[n][half][0] = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::k_word(r, g, word)));
      w[n][half][1] = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::v_word(r, g, word)));
      w[n][half][2] = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::k_param(r, g)));
      w[n][half][3] = __ldg(reinterpret_cast<const uint32_t*>(tile + TL::v_param(r, g)));
    }
    const long long orow = out_rows > 0 ? (long long)at.b * out_rows + at.pos : row;
    dst[n] = ((size_t)orow * pg.Hkv + h) * D + 8 * i;
    live[n] = true;
  }
#pragma unroll
  for (int n = 0; n < kReadRows; ++n) {
    if (!live[n]) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t k[4], v[4];
      dequantise8(w[n][half][0], w[n][half][2], k);
      dequantise8(w[n][half][1], w[n][half][3], v);
      const size_t to = dst[n] + half * (D / 2);
      *reinterpret_cast<uint4*>(Ko + to) = make_uint4(k[0], k[1], k[2], k[3]);
      *reinterpret_cast<uint4*>(Vo + to) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Heads of a block: what a thread works out for its row serves them all, so as
// many as leave 4 blocks an SM (3525 rows of 32 heads of 64: 27 us with 2 blocks
// an SM, 21 with 4, 23 with 8).
inline int heads_per_block(long long row_blocks, int Hkv) {
  int n = Hkv;
  while (n > 1 && row_blocks * ((Hkv + n - 1) / n) < 148 * 4) n = (n + 1) / 2;
  return n;
}

template <int D>
cudaError_t launch_append_t(const void* k_new, const void* v_new, const Pages& pg, const int* cu,
                            const int* t0, int B, int T, int s, float base, cudaStream_t stream) {
  constexpr int kRows = kThreads / (D / 16);
  const unsigned gx = (unsigned)(((long long)T + kRows - 1) / kRows);
  const int hpc = heads_per_block(gx, pg.Hkv);
  const unsigned gy = (unsigned)((pg.Hkv + hpc - 1) / hpc);
  append_kernel<D><<<dim3(gx + 1, gy), kThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new), pg, cu,
      t0, B, T, s, hpc, make_theta(D, base));
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_read_t(void* K, void* V, const Pages& pg, const int* cu, const int* t0, int B,
                          int T, int out_rows, cudaStream_t stream) {
  constexpr int kRows = kThreads / (D / 16);
  const unsigned gx = (unsigned)(((long long)T + kRows * kReadRows - 1) / (kRows * kReadRows));
  read_kernel<D><<<dim3(gx + 1, pg.Hkv), kThreads, 0, stream>>>(
      static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), pg, cu, t0, B, T, out_rows);
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
