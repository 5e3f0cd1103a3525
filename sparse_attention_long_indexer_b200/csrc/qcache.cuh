// The 8-bit latent cache: rows quantised as they are written, and read back.
//
// A row of the cache is d_latent E4M3 codes, one fp32 scale per group of 128 of them, and the
// RoPE part in bf16 (656 B at the production dims, against 1152 B in bf16). With amax the
// largest finite magnitude of a group,
//   scale = 2^e, e the smallest integer with amax <= 448 * 2^e, held to -100 .. 100 (1 if amax = 0)
//   code  = E4M3(x / scale), to nearest even, magnitudes above 448 * scale held to 448
// A power of two costs nothing (E4M3's spacing is relative) and makes x / scale exact, so the
// code is the only rounding; and code * scale is exact in bf16 (E4M3 has 4 significant bits),
// so reading back rounds nothing. A group that holds a NaN gets the scale NaN and reads as NaN.
// Index keys are quantised by the same rule with one scale per token, the form the indexer takes.
//
// Both kernels move bytes and compute next to nothing: one warp per row, every lane one 16-code
// chunk, all loads of a row issued before the first use.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace dsa {

constexpr int kScaleGroup = 128;         // latent dims per scale
constexpr int kScaleExpMax = 100;        // |exponent| of a scale
constexpr int kRowThreads = 256;         // 8 warps = 8 rows per CTA and pass
constexpr int kRowWarps = kRowThreads / 32;
// Resident CTAs per SM, and the most that are launched. 32768 rows written, from inputs that change, take 15.8 to
// 16.1 us (4.5 TB/s of the 6.5 a copy reaches); with 8 launched per SM, of which 6 fit, 18.3, and with the next
// row's loads ahead of the current row's stores, at 4 per SM, 18.2.
constexpr int kRowCtas = 6;

struct QCacheView {
  uint8_t* codes;        // E4M3 [B, max_len, d_latent]
  float* scales;         // fp32 [B, max_len, ceil(d_latent / 128)]
  __nv_bfloat16* rope;   // bf16 [B, max_len, d_rope]
};

// ------------------------------------------------------------------------- conversions
// Bit patterns of bf16 magnitudes order like the magnitudes; from kNonFinite on they are no numbers.
constexpr uint32_t kNonFinite = 0x7F80u;
// Two packed magnitudes, those of infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite_mag2(uint32_t v) {
  uint32_t m = v & 0x7FFF7FFFu;
  if ((m & 0xFFFFu) >= kNonFinite) m &= 0xFFFF0000u;
  if ((m >> 16) >= kNonFinite) m &= 0x0000FFFFu;
  return m;
}
__device__ __forceinline__ uint32_t max4(const uint4& v, uint32_t mask) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & mask, v.y & mask), __vmaxu2(v.z & mask, v.w & mask));
  return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ uint32_t max4_finite(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(finite_mag2(v.x), finite_mag2(v.y)), __vmaxu2(finite_mag2(v.z), finite_mag2(v.w)));
  return max(m & 0xFFFFu, m >> 16);
}
// Exponent of the scale from the bf16 bit pattern of amax: 448 = 1.75 * 2^8, so the smallest e
// is (exponent of amax) - 8, one more where amax's significand is above 1.75 (mantissa 0x60).
// Subnormal magnitudes end at the lower bound either way.
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  const int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
  return max(-kScaleExpMax, min(kScaleExpMax, e));
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Two fp32 in one 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// Four bf16 (two words) times `inv` (packed twice), rounded to E4M3 (to nearest even, magnitudes held to 448).
__device__ __forceinline__ uint32_t e4m3x4(uint32_t a, uint32_t b, uint64_t inv2) {
  uint64_t x = pack_f32x2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
  uint64_t y = pack_f32x2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(inv2));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(inv2));
  float x0, x1, y0, y1;
  unpack_f32x2(x, x0, x1);
  unpack_f32x2(y, y0, y1);
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
  return r;
}
// Two E4M3 codes times a scale (packed twice), as two bf16. Codes convert to fp16 and fp16 to fp32
// exactly; the product with a power of two, and its bf16 form, are exact too. An SM takes 3.3 clocks for a
// warp's words of four codes (512 threads); moving sign, exponent and mantissa into a bf16's places and multiplying
// there takes fewer instructions but 4.5 clocks, as most of them are integer ones.
__device__ __forceinline__ uint32_t expand2(uint16_t codes, uint64_t scale2) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  float lo, hi;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(h));
  uint64_t v = pack_f32x2(lo, hi);
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(scale2));
  unpack_f32x2(v, lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 codes -> 16 bf16
__device__ __forceinline__ void expand16(const uint4& c, float scale, uint4& lo, uint4& hi) {
  const uint64_t s2 = pack_f32x2(scale, scale);
  auto two = [&](uint32_t w, uint32_t& a, uint32_t& b) {
    a = expand2(static_cast<uint16_t>(w), s2);
    b = expand2(static_cast<uint16_t>(w >> 16), s2);
  };
  two(c.x, lo.x, lo.y);
  two(c.y, lo.z, lo.w);
  two(c.z, hi.x, hi.y);
  two(c.w, hi.z, hi.w);
}

// ------------------------------------------------------------------------- write
struct QCacheWriteParams {
  const __nv_bfloat16* latent;   // [B, n_src, d_latent + d_rope], or null
  const __nv_bfloat16* keys;     // [B, n_src, idx_dim], or null
  const int32_t* src;            // [B, n] source row of each written row (< 0: none), or null: row j
  const int32_t* start;          // [B] position of the first written row, or null: 0
  const int32_t* lengths;        // [B] end of each sequence, or null: max_len
  QCacheView cache;
  uint8_t* k_idx;                // E4M3 [B, max_len, idx_dim]
  float* k_scale;                // fp32 [B, max_len]
  uint32_t* status;
  int32_t n, n_src, max_len, d_latent, d_rope, idx_dim;
  int64_t rows;                  // B * n
};

template <int kWidth>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
  for (int o = kWidth / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__global__ void __launch_bounds__(kRowThreads, kRowCtas) qcache_write_kernel(const QCacheWriteParams p) {
  const uint32_t lane = lane_id();
  const int groups = (p.d_latent + kScaleGroup - 1) / kScaleGroup;
  const bool has_lat = p.latent != nullptr && static_cast<int32_t>(16 * lane) < p.d_latent;
  const bool has_rope = p.latent != nullptr && static_cast<int32_t>(8 * lane) < p.d_rope;
  const bool has_key = p.keys != nullptr && static_cast<int32_t>(8 * lane) < p.idx_dim;
  struct Row {
    uint4 a0, a1, r, k;    // 16 latent dims, 8 RoPE dims, 8 key dims
    int64_t to;            // row of the cache, or -1
  };
  // all loads of a row
  auto fetch = [&](int64_t row) {
    Row x;
    x.a0 = x.a1 = x.r = x.k = make_uint4(0, 0, 0, 0);
    x.to = -1;
    const int32_t b = static_cast<int32_t>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.n));
    const int32_t j = static_cast<int32_t>(row - static_cast<int64_t>(b) * p.n);
    const int32_t s = p.src != nullptr ? __ldg(p.src + row) : j;
    const int64_t pos = (p.start != nullptr ? static_cast<int64_t>(__ldg(p.start + b)) : 0) + j;
    if (s < 0 || pos < 0 || (p.lengths != nullptr && pos >= __ldg(p.lengths + b))) return x;
    if (s >= p.n_src || pos >= p.max_len) {
      if (lane == 0) record_error(p.status, DSA_ERR_INDEX_RANGE, static_cast<uint32_t>(row));
      return x;
    }
    const int64_t from = static_cast<int64_t>(b) * p.n_src + s;
    x.to = static_cast<int64_t>(b) * p.max_len + pos;
    const __nv_bfloat16* lat = p.latent + from * (p.d_latent + p.d_rope);
    if (has_lat) {
      const uint4* src = reinterpret_cast<const uint4*>(lat + 16 * lane);
      x.a0 = __ldg(src);
      x.a1 = __ldg(src + 1);
    }
    if (has_rope) x.r = __ldg(reinterpret_cast<const uint4*>(lat + p.d_latent + 8 * lane));
    if (has_key) x.k = __ldg(reinterpret_cast<const uint4*>(p.keys + from * p.idx_dim + 8 * lane));
    return x;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowWarps;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp_id(); row < p.rows; row += step) {
    const Row x = fetch(row);
    if (x.to < 0) continue;
    // magnitudes as they are; in the rare row with an infinity or a NaN, those left out
    uint32_t m = max(max4(x.a0, 0x7FFF7FFFu), max4(x.a1, 0x7FFF7FFFu)), mk = max4(x.k, 0x7FFF7FFFu);
    uint32_t nans = 0;                                     // lanes whose latents hold a NaN
    if (__any_sync(0xffffffffu, max(m, mk) >= kNonFinite)) {
      nans = __ballot_sync(0xffffffffu, m > kNonFinite);
      m = max(max4_finite(x.a0), max4_finite(x.a1));
      mk = max4_finite(x.k);
    }
    if (p.latent != nullptr) {
      const int e = scale_exp(group_max<8>(m));            // 8 lanes hold a group of 128
      const uint64_t inv2 = pack_f32x2(pow2f(-e), pow2f(-e));
      if (has_lat) {
        reinterpret_cast<uint4*>(p.cache.codes + x.to * p.d_latent)[lane] =
            make_uint4(e4m3x4(x.a0.x, x.a0.y, inv2), e4m3x4(x.a0.z, x.a0.w, inv2), e4m3x4(x.a1.x, x.a1.y, inv2),
                       e4m3x4(x.a1.z, x.a1.w, inv2));
        if ((lane & 7u) == 0)
          p.cache.scales[x.to * groups + (lane >> 3)] = ((nans >> lane) & 0xFFu) ? __int_as_float(0x7FC00000) : pow2f(e);
      }
      if (has_rope) reinterpret_cast<uint4*>(p.cache.rope + x.to * p.d_rope)[lane] = x.r;
    }
    if (p.keys != nullptr) {
      const int e = scale_exp(group_max<16>(mk));          // 16 lanes hold the key (idx_dim <= 128)
      const uint64_t inv2 = pack_f32x2(pow2f(-e), pow2f(-e));
      if (has_key)
        reinterpret_cast<uint2*>(p.k_idx + x.to * p.idx_dim)[lane] =
            make_uint2(e4m3x4(x.k.x, x.k.y, inv2), e4m3x4(x.k.z, x.k.w, inv2));
      if (lane == 0) p.k_scale[x.to] = pow2f(e);
    }
  }
}

// ------------------------------------------------------------------------- read
struct QCacheReadParams {
  QCacheView cache;
  const int32_t* listed;         // [B, n] positions (< 0: a zero row), or null: start[b] + j
  const int32_t* start;          // [B], or null: 0
  const int32_t* lengths;        // [B], or null: max_len
  __nv_bfloat16* out;            // [B, n, d_latent + d_rope]
  uint32_t* status;
  int32_t n, max_len, d_latent, d_rope;
  int64_t rows;                  // B * n
};

__global__ void __launch_bounds__(kRowThreads, kRowCtas) qcache_read_kernel(const QCacheReadParams p) {
  const uint32_t lane = lane_id();
  const int groups = (p.d_latent + kScaleGroup - 1) / kScaleGroup;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp_id(); row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const int64_t b = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.n);
    int64_t pos;
    bool ok;
    if (p.listed != nullptr) {
      pos = __ldg(p.listed + row);
      ok = pos >= 0 && pos < p.max_len;
      if (pos >= p.max_len && lane == 0) record_error(p.status, DSA_ERR_INDEX_RANGE, static_cast<uint32_t>(row));
    } else {
      pos = (p.start != nullptr ? static_cast<int64_t>(__ldg(p.start + b)) : 0) + (row - b * p.n);
      const int64_t end = p.lengths != nullptr ? static_cast<int64_t>(__ldg(p.lengths + b)) : p.max_len;
      ok = pos >= 0 && pos < end && pos < p.max_len;
    }
    const int64_t at = b * p.max_len + pos;
    const bool has_lat = static_cast<int32_t>(16 * lane) < p.d_latent;
    const bool has_rope = static_cast<int32_t>(8 * lane) < p.d_rope;
    uint4 c = zero, r = zero;
    float s = 0.f;
    if (ok && has_lat) {
      c = __ldg(reinterpret_cast<const uint4*>(p.cache.codes + at * p.d_latent) + lane);
      s = __ldg(p.cache.scales + at * groups + (lane >> 3));
    }
    if (ok && has_rope) r = __ldg(reinterpret_cast<const uint4*>(p.cache.rope + at * p.d_rope) + lane);
    __nv_bfloat16* dst = p.out + row * (p.d_latent + p.d_rope);
    if (has_lat) {
      uint4 lo, hi;
      expand16(c, s, lo, hi);
      uint4* o = reinterpret_cast<uint4*>(dst + 16 * lane);
      o[0] = lo;
      o[1] = hi;
    }
    if (has_rope) reinterpret_cast<uint4*>(dst + p.d_latent)[lane] = r;
  }
}

}  // namespace dsa
