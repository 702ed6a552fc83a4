// fp4_quant.cu -- rows of numbers to blocks of 4-bit values (spec_quantize_fp4).
//
// A value is c * S: c one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (sign, two exponent
// bits, one mantissa bit), S the scale of its block.
//   SV_FP4_E8M0_32  blocks of 32, S = 2^e with e = floor(log2 max|x|) - 2 (the largest value lands
//                   in [4, 8), above 6 it saturates).
//   SV_FP4_E4M3_16  blocks of 16, S = s g: g = 2^k the row's scale, the smallest power of two with
//                   row maximum <= 6 * 448 g, and s = max|x| / (6 g) rounded to the nearest e4m3.
// c is x / S rounded to nearest, ties to the even code, decided on the exact quotient without
// dividing: see fp4_quotients.
//
// A lane takes 8 neighbouring elements (16 bytes of bf16, of packed codes 4, of values 16), so that
// every load and store of a warp is contiguous; 4 or 2 lanes share a block.
#include <algorithm>

#include "dependent.cuh"
#include "fp4.cuh"

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

// A CTA that is alone first resets the status, which saves a few rows a second launch, and clears the
// one tile row of scales there is, padding rows and all.
__device__ __forceinline__ void begin_alone(const QuantParams& p) {
  if (threadIdx.x == 0 && p.status) *p.status = 0;
  for (int32_t i = threadIdx.x; i < p.groups * 32; i += blockDim.x)
    reinterpret_cast<uint4*>(p.scales)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();  // the rows' scales come after
}

constexpr uint32_t kInfBits = 0x7F800000u;

// Eight elements: as they lie in memory (bf16 pairs, or binary32 patterns).
template <typename E>
struct In;

template <>
struct In<float> {
  static constexpr int kBytes = 4, kWords = 8;
  static constexpr bool kFew = false;  // 24 significant bits
  __device__ static __forceinline__ void load(const uint8_t* p, uint32_t* w) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint4 b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  using Raw = uint32_t;
  // Largest magnitude as a binary32 pattern: a NaN exceeds infinity, which exceeds finite values.
  __device__ static __forceinline__ uint32_t amax(const uint32_t* w) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, w[j] & 0x7FFFFFFFu);
    return m;
  }
  __device__ static __forceinline__ float get(const uint32_t* w, int j) {
    return __uint_as_float(w[j]);
  }
};

template <>
struct In<bf16_tag> {
  static constexpr int kBytes = 2, kWords = 4;
  static constexpr bool kFew = true;  // 8 significant bits
  __device__ static __forceinline__ void load(const uint8_t* p, uint32_t* w) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  using Raw = uint16_t;
  __device__ static __forceinline__ uint32_t amax(const uint32_t* w) {
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ static __forceinline__ float get(const uint32_t* w, int j) {
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
  }
};

// How far vectors may be trusted: 0, rows on any element boundary; 1, rows 16-byte aligned; 2, and
// H a multiple of 256, so that no vector needs a check.

// One warp loads kN spans of 256 elements (span[q] < 0: none) of a row, each lane 8 neighbouring
// elements of every span, zeros past H.  Rows off the 16-byte boundary (kAlign 0) come element by
// element, neighbours to neighbouring lanes, and change hands in shared memory (`stage`, kN spans):
// with lanes that load and store their own 8 one by one, 5000 x 8191 bf16 took 91 us, now 50.
template <typename E, int kAlign, int kN, typename Span>
__device__ __forceinline__ void load_spans(const uint8_t* row, int64_t H, int lane, Span&& span,
                                           typename In<E>::Raw* stage,
                                           uint32_t (*w)[In<E>::kWords]) {
  using Raw = typename In<E>::Raw;
  if constexpr (kAlign == 0) {
    Raw raw[kN][8];
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int64_t e0 = span(q) * 256;
      const Raw* const from = reinterpret_cast<const Raw*>(row) + e0 + lane;
      const int32_t there = e0 < 0 ? 0 : int32_t(min(H - e0, int64_t(256)));
      if (there == 256) {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[q][i] = from[i * 32];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[q][i] = i * 32 + lane < there ? from[i * 32] : Raw(0);
      }
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kN; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) stage[q * 256 + i * 32 + lane] = raw[q][i];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kN; ++q)
#pragma unroll
      for (int i = 0; i < In<E>::kWords; i += 4) {
        const uint4 v = *(reinterpret_cast<const uint4*>(stage + q * 256 + lane * 8) + i / 4);
        w[q][i] = v.x, w[q][i + 1] = v.y, w[q][i + 2] = v.z, w[q][i + 3] = v.w;
      }
  } else {
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int64_t e0 = span(q) * 256 + lane * 8;
      if (e0 >= 0 && (kAlign == 2 || e0 + 8 <= H)) {
        In<E>::load(row + e0 * In<E>::kBytes, w[q]);
      } else {
#pragma unroll
        for (int i = 0; i < In<E>::kWords; ++i) w[q][i] = 0;
        if (e0 >= 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (e0 + j >= H) continue;
            const uint32_t x = reinterpret_cast<const Raw*>(row)[e0 + j];
            if constexpr (sizeof(Raw) == 4)
              w[q][j] = x;
            else
              w[q][j >> 1] |= x << (16 * (j & 1));
          }
        }
      }
    }
  }
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight elements times 2^60.
template <typename E>
__device__ __forceinline__ void scale_up(const uint32_t* w, uint32_t* y) {
  if constexpr (In<E>::kFew) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __float_as_uint(In<E>::get(w, 2 * i) * 0x1p60f);
      const uint32_t b = __float_as_uint(In<E>::get(w, 2 * i + 1) * 0x1p60f);
      y[i] = (a >> 16) | (b & 0xFFFF0000u);  // exact: still 8 significant bits
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(__uint_as_float(w[i]) * 0x1p60f);
  }
}

// Numbers that round to the same codes as the quotients x / S, S = s g.  The codes' borders are
// 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.  q = x / S is first approximated (x r, r near 1 / S, off by
// less than 2^-19) and put on the grid of multiples of 2^-13, which holds the borders.
//   8 significant bits (bf16): a border has 3 significant bits and S has 4, so x is either S times
//   the border or off it by at least 2^-8 of it; on the grid q is then the border itself, or at
//   least 7 steps away on its side.
//   24 significant bits: the sign of the exact remainder x - q' S of the grid point q' says on which
//   side of q' the quotient lies; half a step to that side keeps it off the border.
template <typename E>
__device__ __forceinline__ void fp4_quotients(const uint32_t* w, float S, float r, float* t) {
  constexpr float kGrid = 1536.f;  // one unit in the last place of 1024 .. 2048 is 2^-13
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 x = make_float2(In<E>::get(w, j), In<E>::get(w, j + 1));
    const float2 q = add2(fma2(x, splat2(r), splat2(kGrid)), splat2(-kGrid));
    t[j] = q.x;
    t[j + 1] = q.y;
    if constexpr (!In<E>::kFew) {
      const float2 d = fma2(make_float2(-q.x, -q.y), splat2(S), x);
      if (d.x != 0.f) t[j] += copysignf(6.103515625e-05f, d.x);  // 2^-14
      if (d.y != 0.f) t[j + 1] += copysignf(6.103515625e-05f, d.y);
    }
  }
}

// The e4m3 code of a / 6, rounded to nearest, ties to even: a / 6 is rounded to odd for 24
// significant bits (truncated, the last bit set if inexact), so that no quotient lands on the
// middle of two codes; for 8 bits a rounding to 12 significant bits is enough (a middle times 6 has
// at most 7, so a is it or at least 2^-8 away).
template <typename E>
__device__ __forceinline__ uint32_t scale_code(float a) {
  if constexpr (In<E>::kFew) {
    const float q = a * 0.16666667163372039794921875f;  // 1 / 6 rounded
    return e4m3_of(__uint_as_float((__float_as_uint(q) + 0x800u) & ~0xFFFu));
  } else {
    const float q = __fdiv_rn(a, 6.f);
    const float d = fmaf(-q, 6.f, a);  // exact remainder
    uint32_t b = __float_as_uint(q);
    if (d != 0.f && !(b & 1u)) b = d > 0.f ? b + 1u : b - 1u;
    return e4m3_of(__uint_as_float(b));
  }
}

// The values that eight codes stand for, as bf16 pairs (exact).
__device__ __forceinline__ uint4 fp4x8_bf16(uint32_t codes, float S) {
  float f[8];
  fp4x8_values(codes, f);
  uint32_t h[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 v = mul2(make_float2(f[2 * q], f[2 * q + 1]), splat2(S));
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    h[q] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// Where a lane's vectors of one row go: vector j0 of the row, later ones at multiples of 32 from it.
struct RowOut {
  uint8_t* packed;
  uint8_t* values;  // null: not asked for
  uint8_t* scales;  // of the group that vector j0 lies in (kPerGroup vectors to a group)
};

template <int kPerGroup>
__device__ __forceinline__ RowOut row_out(const QuantParams& p, int64_t r, int64_t j0) {
  RowOut o;
  o.packed = p.packed + r * p.row_bytes + j0 * 4;
  o.values = p.values ? reinterpret_cast<uint8_t*>(p.values + r * p.ldv + j0 * 8) : nullptr;
  o.scales = p.scales + (size_t(r >> 7) * p.groups + size_t(j0) / kPerGroup) * 512 + (r & 31) * 16 +
             ((r >> 5) & 3) * 4;
  return o;
}

// Codes and values of the vector `ahead` spans of 32 vectors behind the row's first; `left` elements
// of the row from it on, `room` bytes of the packed row (kAlign 2: no end in sight).  The whole warp
// takes part; with kAlign 0 values change hands in `stage` as elements do when they are loaded.
template <int kAlign>
__device__ __forceinline__ void store_vec(const RowOut& o, int64_t ahead, const float* t, float S,
                                          int64_t left, int64_t room, int lane, uint16_t* stage) {
  const uint32_t w = fp4x8(t);
  if (kAlign == 2 || room > 0) *reinterpret_cast<uint32_t*>(o.packed + ahead * 128) = w;
  if (!o.values) return;
  const uint4 h = fp4x8_bf16(w, S);
  uint8_t* vd = o.values + ahead * 512;
  if constexpr (kAlign == 0) {
    __syncwarp();
    *reinterpret_cast<uint4*>(stage + lane * 8) = h;
    __syncwarp();
    uint16_t* const to = reinterpret_cast<uint16_t*>(vd) - lane * 7;  // the span's element `lane`
    const int32_t there = int32_t(min(left + lane * 8, int64_t(256)));  // elements of the span
    if (there == 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) to[i * 32] = stage[i * 32 + lane];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * 32 + lane < there) to[i * 32] = stage[i * 32 + lane];
    }
  } else if (kAlign == 2 || left >= 8) {
    *reinterpret_cast<uint4*>(vd) = h;
  } else {
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < left)
        reinterpret_cast<uint16_t*>(vd)[q] = static_cast<uint16_t>(hw[q >> 1] >> (16 * (q & 1)));
  }
}

constexpr int kQuantThreads = 256;

// Latency bounds the hidden rows of a round: 384 x 2560 take 4.3 to 4.8 us a call, most of it the two
// launches.
//
// Blocks of 32: a warp takes kN spans of 256 elements (two scale groups) of one row; the padding
// rows of the last scale tile get scales of zero.
template <typename E, int kAlign, int kN, int kThreads>
__global__ void __launch_bounds__(kThreads) quant_e8m0_kernel(QuantParams p, int32_t spans) {
  constexpr bool kAlone = kThreads == 1024;
  dependent_start();
  if constexpr (kAlone) begin_alone(p);
  const int lane = threadIdx.x & 31;
  const int32_t per_row = (spans + kN - 1) / kN;
  __shared__ __align__(16) typename In<E>::Raw
      s_stage[kAlign == 0 ? kThreads / 32 : 1][kAlign == 0 ? kN * 256 : 8];
  static_assert(sizeof(s_stage) <= 48 * 1024);
  auto* const stage = s_stage[kAlign == 0 ? threadIdx.x >> 5 : 0];
  int64_t warp = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  do {
    const int64_t r = warp / per_row;
    const int32_t s0 = static_cast<int32_t>(warp % per_row) * kN;
    if (r >= (kAlone ? p.rows : (p.rows + 127) & ~int64_t(127))) break;
    const bool real = r < p.rows;
    const int64_t j0 = int64_t(s0) * 32 + lane;
    uint32_t w[kN][In<E>::kWords];
    load_spans<E, kAlign, kN>(
        p.x + r * p.ldx * In<E>::kBytes, p.H, lane,
        [&](int q) { return real && s0 + q < spans ? int64_t(s0 + q) : int64_t(-1); }, stage, w);
    const RowOut o = row_out<16>(p, r, j0);
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      if (s0 + q >= spans) break;
      uint32_t m = In<E>::amax(w[q]);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const bool bad = m >= kInfBits;
      // floor(log2 m) - 2, biased; below 2^-125 (and for a block of zeros) the smallest scale
      const int32_t e = max(int32_t(m >> 23) - 2, 0);
      uint32_t four = (bad ? 0xFFu : uint32_t(e)) << (8 * ((lane >> 2) & 3));
      four |= __shfl_xor_sync(0xffffffffu, four, 4);
      four |= __shfl_xor_sync(0xffffffffu, four, 8);
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(o.scales + q * 1024) = four;
      if (!real) continue;
      if (bad) report(p.status, SV_ERR_BAD_INPUT);
      const float S = bad ? __uint_as_float(0x7FC00000u)  // the scale 0xFF stands for NaN
                          : e ? __uint_as_float(uint32_t(e) << 23) : __uint_as_float(1u << 22);
      const float inv = __uint_as_float(uint32_t(254 - e) << 23);  // 2^(127 - e): exact products
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = bad ? 0.f : In<E>::get(w[q], i) * inv;
      const int64_t j = j0 + q * 32;
      store_vec<kAlign>(o, q, t, S, p.H - j * 8, p.row_bytes - j * 4, lane,
                        reinterpret_cast<uint16_t*>(stage));
    }
    warp += kThreads / 32;
  } while (kAlone);
}

// Whether the staging of kN vectors a lane fits in 48 KB with a CTA of `threads`.
template <typename E, int kAlign, int kN>
constexpr bool staging_fits(int threads) {
  return kAlign != 0 || threads / 32 * (kN * 256 * In<E>::kBytes + 4) <= 48 * 1024;
}

// Memory and issue slots bound it alike: 151936 x 2560 bf16 with values take 263 us, 6.8 TB/s (the
// rate of a copy) at 74% of the issue slots.  A persistent form with the next row in registers took
// 368: 112 registers leave too few warps.
//
// Blocks of 16 under a row scale: `warps` warps of a CTA per row, each lane with kN vectors of it in
// registers between the row's maximum and the codes (kN = 0: any number, read twice).
template <typename E, int kAlign, int kN, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    quant_e4m3_kernel(QuantParams p, int32_t spans, int32_t warps) {
  __shared__ uint32_t s_max[kThreads / 32];
  dependent_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t rows_here = (kThreads >> 5) / warps;
  if constexpr (kThreads == 1024) begin_alone(p);
  const int64_t r = int64_t(blockIdx.x) * rows_here + warp / warps;
  const int32_t mine = warp % warps;
  const bool real = r < p.rows, tile = r < ((p.rows + 127) & ~int64_t(127));
  const int64_t j0 = int64_t(mine) * 32 + lane;
  const uint8_t* row = p.x + r * p.ldx * In<E>::kBytes;
  constexpr int kHold = kN ? kN : 1;
  __shared__ __align__(16) typename In<E>::Raw
      s_stage[kAlign == 0 ? kThreads / 32 : 1][kAlign == 0 ? kHold * 256 : 8];
  static_assert(sizeof(s_stage) + sizeof(s_max) <= 48 * 1024);
  auto* const stage = s_stage[kAlign == 0 ? warp : 0];
  uint32_t w[kHold][In<E>::kWords], am[kHold];
  auto fetch = [&](int32_t q0) {  // kHold spans from q0 on
    load_spans<E, kAlign, kHold>(
        row, p.H, lane,
        [&](int q) {
          const int32_t span = (q0 + q) * warps + mine;
          return real && span < spans ? int64_t(span) : int64_t(-1);
        },
        stage, w);
  };
  uint32_t m = 0;
  if constexpr (kN > 0) {
    fetch(0);
#pragma unroll
    for (int q = 0; q < kN; ++q) m = max(m, am[q] = In<E>::amax(w[q]));
  } else {
    for (int32_t q = 0; q * warps + mine < spans; ++q) {
      fetch(q);
      m = max(m, In<E>::amax(w[0]));
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (warps > 1) {
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    for (int i = 0; i < warps; ++i) m = max(m, s_max[warp - mine + i]);
  }
  if (!tile) return;
  const RowOut o = row_out<8>(p, r, j0);
  if (!real) {  // a padding row of the last scale tile
    for (int32_t q = 0; q * warps + mine < spans; ++q)
      if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(o.scales + int64_t(q) * warps * 2048) = 0;
    return;
  }
  const bool bad = m >= kInfBits;
  // 6 * 448 = 1.3125 * 2^11: the smallest k with m <= 1.3125 * 2^(11 + k)
  int32_t k2 = 0;
  if (!bad && m) {
    k2 = int32_t(m >> 23) - 127 - 11 + ((m & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    k2 = min(max(k2, -120), 120);
  }
  const float g = __uint_as_float(uint32_t(k2 + 127) << 23);
  const float ginv = __uint_as_float(uint32_t(127 - k2) << 23);
  if (mine == 0 && lane == 0) {
    p.row_scales[r] = g;
    if (bad) report(p.status, SV_ERR_BAD_INPUT);
  }
  const uint32_t byte = 8 * ((lane >> 1) & 3);
  auto emit = [&](int32_t q, const uint32_t* x, uint32_t amax) {
    if (q * warps + mine >= spans) return;
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const uint32_t code = bad ? 0x7Fu : scale_code<E>(__uint_as_float(amax) * ginv);
    uint32_t four = code << byte;
    four |= __shfl_xor_sync(0xffffffffu, four, 2);
    four |= __shfl_xor_sync(0xffffffffu, four, 4);
    if ((lane & 7) == 0)
      *reinterpret_cast<uint32_t*>(o.scales + int64_t(q) * warps * 2048) = four;
    const float s = e4m3_value(code);
    const float S = bad ? __uint_as_float(0x7FC00000u) : s * g;
    const float rs = code ? rcp_approx(s) : 0.f;  // a block of zero scale has codes of zero
    float t[8];
    if (bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = 0.f;
    } else if (k2 > -110) {
      fp4_quotients<E>(x, S, rs * ginv, t);
    } else {
      // 1 / S would overflow at the smallest scales: both are taken 2^60 larger (x and S stay exact,
      // they are far below the largest number)
      uint32_t y[In<E>::kWords];
      scale_up<E>(x, y);
      fp4_quotients<E>(y, S * 0x1p60f, rs * (ginv * 0x1p-60f), t);
    }
    const int64_t j = j0 + int64_t(q) * warps * 32;
    store_vec<kAlign>(o, int64_t(q) * warps, t, S, p.H - j * 8, p.row_bytes - j * 4, lane,
                      reinterpret_cast<uint16_t*>(stage));
  };
  if constexpr (kN > 0) {
#pragma unroll
    for (int q = 0; q < kN; ++q) emit(q, w[q], am[q]);
  } else {
    for (int32_t q = 0; q * warps + mine < spans; ++q) {
      fetch(q);
      emit(q, w[0], In<E>::amax(w[0]));
    }
  }
}

template <typename E, int kAlign>
sv_status launch_e8m0(const QuantParams& p, cudaStream_t s) {
  const int32_t spans = int32_t((p.H + 255) / 256);
  const int64_t padded = (p.rows + 127) / 128 * 128;
  // two spans per warp where there is enough work for the GPU, else one
  const bool two = padded * spans >= 2 * 16384;
  const int64_t warps = padded * (two ? (spans + 1) / 2 : spans);
  const int64_t blocks = (warps * 32 + kQuantThreads - 1) / kQuantThreads;
  if (blocks > INT32_MAX) return SV_ERR_UNSUPPORTED;
  // Few spans go to one CTA and one launch (us a call, bf16 with values: 2 x 2560 3.0, 6 x 2560 3.5; 8
  // x 2560, 80 spans, 4.4 and 16 x 2560 6.8, where two launches take 4.4 for all of them).
  if (p.rows * spans <= 64)
    return launch_dependent(quant_e8m0_kernel<E, kAlign, 1, 1024>, 1, 1024, 0, s, p, spans);
  const sv_status reset = reset_status(p.status, s);
  if (reset != SV_OK) return reset;
  return launch_dependent(two ? quant_e8m0_kernel<E, kAlign, 2, kQuantThreads>
                              : quant_e8m0_kernel<E, kAlign, 1, kQuantThreads>,
                          unsigned(blocks), kQuantThreads, 0, s, p, spans);
}

// `warps` warps to a row, CTAs of 128 threads or a row.
template <typename E, int kAlign, int kN>
sv_status launch_e4m3(const QuantParams& p, int32_t spans, int32_t warps, cudaStream_t s) {
  const int32_t threads = warps <= 4 ? 128 : warps * 32;
  const int64_t rows = (p.rows + 127) / 128 * 128, here = threads / 32 / warps;
  const int64_t blocks = (rows + here - 1) / here;
  if (blocks > INT32_MAX) return SV_ERR_UNSUPPORTED;
  auto* kernel = quant_e4m3_kernel<E, kAlign, kN, 128>;
  if (threads == 256) kernel = quant_e4m3_kernel<E, kAlign, kN, 256>;
  if constexpr (staging_fits<E, kAlign, kN>(512)) {
    if (threads == 512) kernel = quant_e4m3_kernel<E, kAlign, kN, 512>;
  } else if (threads == 512) {
    return SV_ERR_UNSUPPORTED;  // not asked for below
  }
  return launch_dependent(kernel, unsigned(blocks), unsigned(threads), 0, s, p, spans, warps);
}

template <typename E, int kAlign>
sv_status launch_e4m3(const QuantParams& p, cudaStream_t s) {
  constexpr int kMost = In<E>::kFew ? 5 : 4;  // vectors a lane holds
  const int32_t spans = int32_t((p.H + 255) / 256);
  // the fewest warps per row that hold it; more where the rows alone would leave the GPU idle
  int32_t warps = 1;
  while (warps < 16 && (warps * kMost < spans || (warps < spans && p.rows * warps < 2048)))
    warps *= 2;
  // Few spans go to one CTA and one launch (us a call, with values: 2 x 2560 3.0, 8 x 2560 bf16 3.8, 6 x
  // 2560 fp32 4.3; 16 x 2560 5.1 and 7.5, where two launches take 4.4 for all of them).
  constexpr int kHeld = staging_fits<E, kAlign, kMost>(1024) ? kMost
                        : staging_fits<E, kAlign, 2>(1024)   ? 2
                                                             : 1;
  int32_t each = 1;  // warps per row of that CTA: 32 over the next power of two of the rows
  while (each * 2 * p.rows <= 32) each *= 2;
  if (p.rows <= 32 && p.rows * spans <= (In<E>::kFew ? 80 : 48) && spans <= kHeld * each) {
    const int32_t hold = (spans + each - 1) / each;
    return launch_dependent(hold == 1   ? quant_e4m3_kernel<E, kAlign, 1, 1024>
                            : hold == 2 ? quant_e4m3_kernel<E, kAlign, kHeld < 2 ? 1 : 2, 1024>
                                        : quant_e4m3_kernel<E, kAlign, kHeld, 1024>,
                            1, 1024, 0, s, p, spans, each);
  }
  const sv_status reset = reset_status(p.status, s);
  if (reset != SV_OK) return reset;
  // a kernel for each number of vectors: in one for up to five or three of them the others' turns
  // cost, and with fewer held rows need CTAs of eight warps or more (40000 x 4096 fp32 223 -> 157 us,
  // 100000 x 1025 bf16 197 -> 113, 20000 x 7168 bf16 131 -> 116)
  const int32_t hold = (spans + warps - 1) / warps;
  if (hold == 1) return launch_e4m3<E, kAlign, 1>(p, spans, warps, s);
  if (hold == 2) return launch_e4m3<E, kAlign, 2>(p, spans, warps, s);
  if (warps < 16 || staging_fits<E, kAlign, kMost>(512)) {
    if (hold == 3) return launch_e4m3<E, kAlign, 3>(p, spans, warps, s);
    if (hold == 4) return launch_e4m3<E, kAlign, 4>(p, spans, warps, s);
    if (hold <= kMost) return launch_e4m3<E, kAlign, kMost>(p, spans, warps, s);
  }
  return launch_e4m3<E, kAlign, 0>(p, spans, warps, s);
}

template <typename E>
sv_status launch_quant(const QuantParams& p, int32_t format, bool vec, cudaStream_t s) {
  const int align = !vec ? 0 : p.H % 256 ? 1 : 2;
  if (format == SV_FP4_E8M0_32)
    return align == 0   ? launch_e8m0<E, 0>(p, s)
           : align == 1 ? launch_e8m0<E, 1>(p, s)
                        : launch_e8m0<E, 2>(p, s);
  return align == 0   ? launch_e4m3<E, 0>(p, s)
         : align == 1 ? launch_e4m3<E, 1>(p, s)
                      : launch_e4m3<E, 2>(p, s);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return reset_status(status, s);
  if (!x || !packed || !scales || (format == SV_FP4_E4M3_16 && !row_scales))
    return SV_ERR_INVALID;
  const int eb = elem_bytes(dtype);
  if (!aligned16(packed) || !aligned16(scales) ||
      reinterpret_cast<uintptr_t>(x) % eb != 0 || reinterpret_cast<uintptr_t>(values) % 2 != 0)
    return SV_ERR_UNSUPPORTED;
  const bool vec = aligned16(x) && (ldx * eb) % 16 == 0 &&
                   (!values || (aligned16(values) && ld_values % 8 == 0));
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
