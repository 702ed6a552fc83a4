// fp4_quant.cu -- rows of numbers to blocks of 4-bit values (spec_quantize_fp4).
//
// A value is c * S: c one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (sign, two exponent
// bits, one mantissa bit), S the scale of its block.
//   SV_FP4_E8M0_32  blocks of 32, S = 2^e with e = floor(log2 max|x|) - 2 (the largest value lands
//                   in [4, 8), above 6 it saturates).
//   SV_FP4_E4M3_16  blocks of 16, S = s g: g = 2^k the row's scale, the smallest power of two with
//                   row maximum <= 6 * 448 g, and s = max|x| / (6 g) rounded to the nearest e4m3.
// c is x / S rounded to nearest, ties to the even code.  Every rounding is decided on the exact
// quotient: a division by a power of two is exact, the other two are rounded to odd in binary32
// (truncated, the last bit set when inexact) before the conversion rounds them, which keeps a
// quotient from being rounded onto the middle between two codes and then away from its side.
#include "fp4.cuh"
#include "sv_host.h"

namespace sv {
namespace {

struct QuantParams {
  const uint8_t* x;
  int64_t rows, H, ldx;
  uint8_t* packed;
  int64_t row_bytes;
  uint8_t* scales;
  int32_t groups;  // scale groups (of four blocks) per row
  float* row_scales;
  uint16_t* values;
  int64_t ldv;
  int32_t* status;
};

constexpr int kQuantThreads = 128;

template <typename E>
struct In;
template <>
struct In<float> {
  static constexpr int kBytes = 4;
  __device__ static __forceinline__ uint32_t one(const uint8_t* p) {
    return __ldg(reinterpret_cast<const uint32_t*>(p));
  }
};
template <>
struct In<bf16_tag> {
  static constexpr int kBytes = 2;
  __device__ static __forceinline__ uint32_t one(const uint8_t* p) {
    return uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p))) << 16;
  }
};

// Elements e0 .. e0 + kN - 1 of a row as binary32 bit patterns, zeros past H.
template <typename E, int kN, bool kVec>
__device__ __forceinline__ void load_block(const uint8_t* row, int64_t e0, int64_t H,
                                           uint32_t* v) {
  constexpr int kPer = 16 / In<E>::kBytes;
  if (kVec && e0 + kN <= H) {
    const uint4* p = reinterpret_cast<const uint4*>(row + e0 * In<E>::kBytes);
#pragma unroll
    for (int q = 0; q < kN / kPer; ++q) {
      float f[kPer];
      Elem<E>::unpack(__ldg(p + q), f);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[q * kPer + j] = __float_as_uint(f[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) v[j] = e0 + j < H ? In<E>::one(row + (e0 + j) * In<E>::kBytes) : 0u;
}

// Largest magnitude as a bit pattern: above 0x7F800000 for a NaN, so neither NaN nor infinity is
// lost among finite values.
template <int kN>
__device__ __forceinline__ uint32_t amax_bits(const uint32_t* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kN; ++j) m = max(m, v[j] & 0x7FFFFFFFu);
  return m;
}

constexpr uint32_t kInfBits = 0x7F800000u;

// |x| / S rounded to odd, for S with few significant bits: q the nearest quotient, then one step
// towards the exact one if it is inexact and its last bit is even.
__device__ __forceinline__ float div_odd(float x, float S) {
  const float q = __fdiv_rn(x, S);
  const float d = fmaf(-q, S, x);  // exact remainder
  uint32_t b = __float_as_uint(q);
  if (d != 0.f && !(b & 1u)) b = d > 0.f ? b + 1u : b - 1u;
  return __uint_as_float(b);
}

// Writes one block: codes, and the values they stand for.
template <int kN, bool kVec>
__device__ __forceinline__ void store_block(const QuantParams& p, int64_t r, int64_t e0,
                                            const float* t, float S) {
  uint32_t w[kN / 8];
#pragma unroll
  for (int q = 0; q < kN / 8; ++q) w[q] = fp4x8(t + 8 * q);
  uint8_t* dst = p.packed + r * p.row_bytes + (e0 >> 1);
  if constexpr (kN == 32) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  }
  if (!p.values) return;
  uint16_t* vd = p.values + r * p.ldv + e0;
#pragma unroll
  for (int q = 0; q < kN / 8; ++q) {
    float f[8];
    fp4x8_values(w[q], f);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j] * S, f[2 * j + 1] * S);  // exact
      h[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (kVec && e0 + 8 * q + 8 <= p.H) {
      *reinterpret_cast<uint4*>(vd + 8 * q) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e0 + 8 * q + j < p.H) vd[8 * q + j] = static_cast<uint16_t>(h[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// Where row r's scale of block k lies.
__device__ __forceinline__ size_t scale_at(int64_t r, int64_t k, int32_t groups) {
  return (size_t(r >> 7) * groups + size_t(k >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 +
         (k & 3);
}

// Blocks of 32: a thread per (row, block), the padding blocks and rows of the scale tiles included.
template <typename E, bool kVec>
__global__ void __launch_bounds__(kQuantThreads) quant_e8m0_kernel(QuantParams p) {
  const int64_t nb = int64_t(p.groups) * 4;
  const int64_t i = int64_t(blockIdx.x) * kQuantThreads + threadIdx.x;
  const int64_t r = i / nb, k = i % nb;
  if (r >= ((p.rows + 127) & ~int64_t(127))) return;
  uint8_t* sc = p.scales + scale_at(r, k, p.groups);
  if (r >= p.rows || k * 32 >= p.H) {
    *sc = 0;
    return;
  }
  uint32_t v[32];
  load_block<E, 32, kVec>(p.x + r * p.ldx * In<E>::kBytes, k * 32, p.H, v);
  const uint32_t m = amax_bits<32>(v);
  float t[32];
  float S;
  if (m >= kInfBits) {
    report(p.status, SV_ERR_BAD_INPUT);
    *sc = 0xFF;  // the scale that stands for NaN
    S = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j] = 0.f;
  } else {
    // floor(log2 m) - 2, biased; below 2^-125 (and for a block of zeros) the smallest scale
    const int32_t e = max(int32_t(m >> 23) - 2, 0);
    *sc = static_cast<uint8_t>(e);
    S = e ? __uint_as_float(uint32_t(e) << 23) : __uint_as_float(1u << 22);
    const float inv = __uint_as_float(uint32_t(254 - e) << 23);  // 2^(127 - e), exact
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j] = __uint_as_float(v[j]) * inv;
  }
  store_block<32, kVec>(p, r, k * 32, t, S);
}

// Blocks of 16 under a row scale: a CTA per row, two passes over it (the second from L1).
template <typename E, bool kVec>
__global__ void __launch_bounds__(kQuantThreads) quant_e4m3_kernel(QuantParams p) {
  __shared__ uint32_t s_max[kQuantThreads / 32];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t nb = int64_t(p.groups) * 4;
  if (r >= p.rows) {
    for (int64_t k = tid; k < nb; k += kQuantThreads) p.scales[scale_at(r, k, p.groups)] = 0;
    return;
  }
  const uint8_t* row = p.x + r * p.ldx * In<E>::kBytes;
  uint32_t m = 0;
  for (int64_t k = tid; k * 16 < p.H; k += kQuantThreads) {
    uint32_t v[16];
    load_block<E, 16, kVec>(row, k * 16, p.H, v);
    m = max(m, amax_bits<16>(v));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, s_max[w]);
  const bool bad = m >= kInfBits;
  // 6 * 448 = 1.3125 * 2^11: the smallest k with m <= 1.3125 * 2^(11 + k)
  int32_t k2 = 0;
  if (!bad && m) {
    const int32_t e = int32_t(m >> 23) - 127;
    k2 = e - 11 + ((m & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    k2 = min(max(k2, -120), 120);
  }
  const float g = __uint_as_float(uint32_t(k2 + 127) << 23);
  const float ginv = __uint_as_float(uint32_t(127 - k2) << 23);
  if (tid == 0) {
    p.row_scales[r] = g;
    if (bad) report(p.status, SV_ERR_BAD_INPUT);
  }
  for (int64_t k = tid; k < nb; k += kQuantThreads) {
    uint8_t* sc = p.scales + scale_at(r, k, p.groups);
    if (k * 16 >= p.H) {
      *sc = 0;
      // the packed row is padded to 32 elements: its second half block is zeros
      if (k * 8 < p.row_bytes)
        *reinterpret_cast<uint2*>(p.packed + r * p.row_bytes + k * 8) = make_uint2(0, 0);
      continue;
    }
    uint32_t v[16];
    load_block<E, 16, kVec>(row, k * 16, p.H, v);
    float t[16];
    uint32_t code;
    float s;
    if (bad) {
      code = 0x7Fu;
      s = __uint_as_float(0x7FC00000u);
    } else {
      const float a = __uint_as_float(amax_bits<16>(v)) * ginv;
      code = e4m3_of(div_odd(a, 6.f));
      s = e4m3_value(code);
    }
    const float S = s * g;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = __uint_as_float(v[j]);
      t[j] = (bad || code == 0) ? 0.f : copysignf(div_odd(fabsf(x), S), x);
    }
    *sc = static_cast<uint8_t>(code);
    store_block<16, kVec>(p, r, k * 16, t, S);
  }
}

template <typename E>
sv_status launch_quant(const QuantParams& p, int32_t format, bool vec, cudaStream_t s) {
  const int64_t padded = (p.rows + 127) / 128 * 128;
  if (format == SV_FP4_E8M0_32) {
    const int64_t blocks = (padded * p.groups * 4 + kQuantThreads - 1) / kQuantThreads;
    if (blocks > INT32_MAX) return SV_ERR_UNSUPPORTED;
    if (vec)
      quant_e8m0_kernel<E, true><<<unsigned(blocks), kQuantThreads, 0, s>>>(p);
    else
      quant_e8m0_kernel<E, false><<<unsigned(blocks), kQuantThreads, 0, s>>>(p);
  } else {
    if (padded > INT32_MAX) return SV_ERR_UNSUPPORTED;
    if (vec)
      quant_e4m3_kernel<E, true><<<unsigned(padded), kQuantThreads, 0, s>>>(p);
    else
      quant_e4m3_kernel<E, false><<<unsigned(padded), kQuantThreads, 0, s>>>(p);
  }
  return launch_status(cudaGetLastError());
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int64_t spec_fp4_row_bytes(int64_t H) { return H < 1 ? 0 : (H + 31) / 32 * 16; }

extern "C" size_t spec_fp4_scale_bytes(int64_t rows, int64_t H, int32_t format) {
  if (rows < 1 || H < 1 || (format != SV_FP4_E8M0_32 && format != SV_FP4_E4M3_16)) return 0;
  return size_t((rows + 127) / 128) * fp4_groups(H, format) * 512;
}

extern "C" sv_status spec_quantize_fp4(const void* x, sv_dtype dtype, int64_t rows, int64_t H,
                                       int64_t ldx, int32_t format, uint8_t* packed,
                                       uint8_t* scales, float* row_scales, void* values,
                                       int64_t ld_values, int32_t* status, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID;
  if (format != SV_FP4_E8M0_32 && format != SV_FP4_E4M3_16) return SV_ERR_INVALID;
  if (rows < 0 || H < 1 || ldx < H || (values && ld_values < H)) return SV_ERR_INVALID;
  if (H > INT32_MAX || rows > INT32_MAX) return SV_ERR_UNSUPPORTED;
  if (rows == 0) return SV_OK;
  if (!x || !packed || !scales || (format == SV_FP4_E4M3_16 && !row_scales))
    return SV_ERR_INVALID;
  const int eb = elem_bytes(dtype);
  if (!aligned16(packed) || !aligned16(scales) ||
      reinterpret_cast<uintptr_t>(x) % eb != 0 || reinterpret_cast<uintptr_t>(values) % 2 != 0)
    return SV_ERR_UNSUPPORTED;
  const bool vec = aligned16(x) && (ldx * eb) % 16 == 0 &&
                   (!values || (aligned16(values) && ld_values % 8 == 0));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, sizeof(int32_t), s) != cudaSuccess) return SV_ERR_CUDA;
  const QuantParams p = {static_cast<const uint8_t*>(x),
                         rows,
                         H,
                         ldx,
                         packed,
                         spec_fp4_row_bytes(H),
                         scales,
                         fp4_groups(H, format),
                         row_scales,
                         static_cast<uint16_t*>(values),
                         ld_values,
                         status};
  return dtype == SV_BF16 ? launch_quant<bf16_tag>(p, format, vec, s)
                          : launch_quant<float>(p, format, vec, s);
}
