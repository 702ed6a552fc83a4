// fp4_project.cu -- logits from 4-bit hidden rows and a 4-bit output projection
// (spec_project_fp4): out[m][v] = sum_k x[m][k] w[v][k], both operands as quantised by
// spec_quantize_fp4.
//
// A persistent, warp-specialised tcgen05 GEMM.  W is the A operand (128 vocabulary rows per tile,
// TMEM lanes), the hidden rows the B operand (up to 192 rows per tile, TMEM columns), K in blocks
// of 256 elements: 128 bytes, one row of the 128-byte swizzle.
//   warp 0     TMA loads of the k-blocks of W and of the hidden rows, and bulk copies of their
//              scale tiles, into a ring;
//   warp 1     per k-block, tcgen05.cp of the scale tiles to TMEM and four block-scaled
//              tcgen05.mma (K = 64) into one of two accumulators;
//   warps 2-9  the epilogue: a lane quadrant and a column half each.
// The tensor cores apply the block scales and add in fp32; the row scales of SV_FP4_E4M3_16 are
// powers of two, applied to the sum in the epilogue.
#include <algorithm>

#include "fp4.cuh"
#include "sv_host.h"
#include "tc.cuh"
#include "tmap.h"

namespace sv {
namespace {

constexpr int kPjRows = 128;     // vocabulary rows per tile (UMMA M)
constexpr int kPjMaxN = 192;     // hidden rows per tile at most
constexpr int kPjEpiWarps = 8;
constexpr int kPjThreads = 32 * (2 + kPjEpiWarps);
constexpr uint32_t kPjABytes = kPjRows * 128;
constexpr uint32_t kPjSmem = 225 * 1024;  // ring and alignment slack
constexpr int kPjMaxStages = 10;
constexpr uint32_t kPjTmemCols = 512;

struct PjParams {
  int32_t n_vt, n_nt, nt;  // vocabulary tiles, hidden-row tiles, rows of a hidden-row tile
  int32_t kblocks;
  int64_t H, V;
  int32_t M;
  int32_t m_tiles;  // scale tiles of the hidden rows
  int32_t stages;
  uint32_t stage_bytes, b_off, sfa_off, sfb_off;
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  const float* w_row;
  const float* x_row;
  void* out;
  int64_t ld;
  int32_t* status;
};

// mbar_wait with a suspend-time hint: the waiting thread sleeps until the phase completes.  Bounded:
// after kWaitLimitNs it reports SV_ERR_TIMEOUT and gives up.
__device__ __forceinline__ bool pj_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ bool pj_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  if (pj_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!pj_try_wait(bar, parity)) {
    if (global_ns() - t0 > kWaitLimitNs) {
      report(status, SV_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Shared-memory descriptor of a 512-byte scale tile (32 rows of 16 bytes, no swizzle): core
// matrices of 8 rows by 16 bytes are 128 bytes, the stride between them.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_byte_addr) {
  uint64_t d = 0;
  d |= uint64_t((smem_byte_addr & 0x3FFFFu) >> 4);
  d |= uint64_t(128 >> 4) << 32;  // stride byte offset: eight rows of 16 bytes
  d |= uint64_t(1) << 46;         // descriptor version
  return d;
}

// 512 bytes of scales to four TMEM columns, the 32 lanes repeated in every lane quadrant.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// Instruction descriptor of the block-scaled 4-bit kinds: e2m1 A and B (1 in bits [7,10) and
// [10,12)), both K-major, N >> 3 in [17,23), scale type in bit 23 (1: e8m0, 0: e4m3), M >> 7 in
// [27,29); the scale ids of B and A go to [4,6) and [29,31).
constexpr uint32_t pj_idesc(int32_t n, bool e8m0) {
  return (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (e8m0 ? 1u << 23 : 0u) | (1u << 27);
}

template <int kFmt>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  if constexpr (kFmt == SV_FP4_E8M0_32) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(sfa), "r"(sfb)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(sfa), "r"(sfb)
        : "memory");
  }
}

template <int kFmt, typename Out>
__global__ void __launch_bounds__(kPjThreads, 1)
    project_kernel(const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x, PjParams p) {
  constexpr int kGroups = kFmt == SV_FP4_E8M0_32 ? 2 : 4;  // scale groups per k-block
  constexpr uint32_t kTileBytes = kGroups * 512;           // scales of 128 rows and one k-block
  constexpr uint32_t kSfaCols = kGroups * 4;
  constexpr uint32_t kSfCols = kSfaCols * 3;  // W's tile and at most two of the hidden rows'
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kPjMaxStages], empty[kPjMaxStages];
  __shared__ uint64_t acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_base;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t n_items = p.n_vt * p.n_nt;
  const int32_t stages = p.stages;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], kPjEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(&tmem_base, kPjTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base;
  const uint32_t sf_base = tmem + kPjTmemCols - 2 * kSfCols;  // two buffers of scale columns

  // Scale tiles of the hidden rows n0 .. n0 + nt - 1 that exist.
  auto x_tiles = [&](int32_t n0) {
    return min(p.m_tiles, (n0 + p.nt + 127) >> 7) - (n0 >> 7);
  };

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t keep = tc::policy_evict_last(), once = tc::policy_evict_first();
      const uint64_t w_policy = p.n_nt > 1 ? keep : once;
      uint32_t it = 0;
      bool ok = true;
      for (int32_t item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
        const int32_t vt = item / p.n_nt, n0 = (item % p.n_nt) * p.nt;
        const int32_t nx = x_tiles(n0);
        const uint32_t bytes = kPjABytes + uint32_t(p.nt) * 128 + (1 + nx) * kTileBytes;
        const size_t per_tile = size_t(p.kblocks) * kTileBytes;
        const uint8_t* ws = p.w_scales + size_t(vt) * per_tile;
        const uint8_t* xs = p.x_scales + size_t(n0 >> 7) * per_tile;
        for (int32_t kb = 0; kb < p.kblocks; ++kb, ++it) {
          const uint32_t s = it % stages, use = it / stages;
          if (use > 0 && !pj_wait(&empty[s], (use - 1) & 1, p.status)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + size_t(s) * p.stage_bytes;
          mbar_expect_tx(&full[s], bytes);
          tc::tma_load_2d_hint(st, &map_w, kb * 128, vt * kPjRows, &full[s], w_policy);
          tc::tma_load_2d_hint(st + p.b_off, &map_x, kb * 128, n0, &full[s], keep);
          bulk_g2s(st + p.sfa_off, ws + size_t(kb) * kTileBytes, kTileBytes, &full[s]);
          for (int32_t t = 0; t < nx; ++t)
            bulk_g2s(st + p.sfb_off + t * kTileBytes, xs + t * per_tile + size_t(kb) * kTileBytes,
                     kTileBytes, &full[s]);
        }
      }
      // the copies in flight land before the block may end
      for (uint32_t k = it > uint32_t(stages) ? it - stages : 0; k < it; ++k)
        pj_wait(&full[k % stages], (k / stages) & 1, p.status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0;
      int t = 0;
      bool ok = true;
      for (int32_t item = blockIdx.x; item < n_items && ok; item += gridDim.x, ++t) {
        const int32_t n0 = (item % p.n_nt) * p.nt;
        const int32_t nx = x_tiles(n0);
        const int32_t n = min(p.nt, (p.M - n0 + 15) & ~15);
        const uint32_t idesc = pj_idesc(n, kFmt == SV_FP4_E8M0_32);
        const uint32_t acc = tmem + (t & 1) * p.nt;
        if (t >= 2 && !pj_wait(&acc_empty[t & 1], ((t >> 1) - 1) & 1, p.status)) break;
        tc::fence_after_sync();
        for (int32_t kb = 0; kb < p.kblocks; ++kb, ++it) {
          const uint32_t s = it % stages;
          if (!pj_wait(&full[s], (it / stages) & 1, p.status)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t base = smem_addr(ring + size_t(s) * p.stage_bytes);
          const uint32_t sfa = sf_base + (it & 1) * kSfCols, sfb = sfa + kSfaCols;
#pragma unroll
          for (int gq = 0; gq < kGroups; ++gq) {
            copy_scales(sfa + gq * 4, scale_desc(base + p.sfa_off + gq * 512));
            for (int32_t x = 0; x < nx; ++x)
              copy_scales(sfb + (gq * 2 + x) * 4,
                          scale_desc(base + p.sfb_off + x * kTileBytes + gq * 512));
          }
          const int32_t ksteps = min(4, int32_t((p.H - int64_t(kb) * 256 + 63) >> 6));
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            if (ks >= ksteps) break;
            const int gq = kGroups == 4 ? ks : ks >> 1;
            const uint32_t id = kGroups == 4 ? 0u : uint32_t(ks & 1) * 2u;
            mma_fp4<kFmt>(acc, tc::smem_desc_sw128(base + ks * 32),
                          tc::smem_desc_sw128(base + p.b_off + ks * 32),
                          idesc | (id << 4) | (id << 29), sfa + gq * 4,
                          sfb + gq * 8 + ((n0 & 127) >> 5), (kb | ks) != 0);
          }
          tc::mma_commit(&empty[s]);
        }
        if (ok) tc::mma_commit(&acc_full[t & 1]);
      }
      // nothing reads shared or tensor memory once this has passed
      tc::mma_commit(&drain);
      pj_wait(&drain, 0, p.status);
    }
  } else {
    const int q = warp & 3, h = (warp - 2) >> 2;
    bool failed = false;
    int t = 0;
    for (int32_t item = blockIdx.x; item < n_items; item += gridDim.x, ++t) {
      const int32_t vt = item / p.n_nt, n0 = (item % p.n_nt) * p.nt;
      const int64_t v = int64_t(vt) * kPjRows + 32 * q + lane;
      const int32_t n = min(p.nt, p.M - n0);
      float ws = 1.f;
      if (kFmt == SV_FP4_E4M3_16 && v < p.V) ws = __ldg(p.w_row + v);
      if (!failed && !pj_wait(&acc_full[t & 1], (t >> 1) & 1, p.status)) failed = true;
      __syncwarp();
      tc::fence_after_sync();
      // 16-column pieces, alternating between the two warps of a quadrant
      for (int32_t c = 16 * h; c < n; c += 32) {
        float a[16];
        tc::tmem_load16(tmem + (uint32_t(32 * q) << 16) + (t & 1) * p.nt + c, a);
        if (v < p.V) {
          Out* o = static_cast<Out*>(p.out) + int64_t(n0 + c) * p.ld + v;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c + j >= n) break;
            float y = a[j];
            if (kFmt == SV_FP4_E4M3_16) y = y * ws * __ldg(p.x_row + n0 + c + j);
            if constexpr (sizeof(Out) == 2)
              o[j * p.ld] = __float2bfloat16_rn(y);
            else
              o[j * p.ld] = y;
          }
        }
        __syncwarp();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[t & 1]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kPjTmemCols);
  }
}

template <int kFmt, typename Out>
sv_status launch_project(const CUtensorMap& map_w, const CUtensorMap& map_x, const PjParams& p,
                         int grid, cudaStream_t s) {
  auto* kern = project_kernel<kFmt, Out>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kPjSmem)) !=
      cudaSuccess)
    return SV_ERR_CUDA;
  kern<<<grid, kPjThreads, kPjSmem, s>>>(map_w, map_x, p);
  return launch_status(cudaGetLastError());
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status spec_project_fp4(const uint8_t* x_packed, const uint8_t* x_scales,
                                      const float* x_row_scales, int64_t M,
                                      const uint8_t* w_packed, const uint8_t* w_scales,
                                      const float* w_row_scales, int64_t V, int64_t H,
                                      int32_t format, void* logits, sv_dtype dtype, int64_t ld,
                                      int32_t* status, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID;
  if (format != SV_FP4_E8M0_32 && format != SV_FP4_E4M3_16) return SV_ERR_INVALID;
  if (M < 0 || V < 1 || H < 1 || ld < V) return SV_ERR_INVALID;
  if (V > INT32_MAX - 256 || M > (1 << 24) || H > (1 << 24)) return SV_ERR_UNSUPPORTED;
  if (M == 0) return SV_OK;
  if (!x_packed || !x_scales || !w_packed || !w_scales || !logits) return SV_ERR_INVALID;
  if (format == SV_FP4_E4M3_16 && (!x_row_scales || !w_row_scales)) return SV_ERR_INVALID;
  if (!aligned16(x_packed) || !aligned16(x_scales) || !aligned16(w_packed) ||
      !aligned16(w_scales) || !aligned16(logits) || (ld * elem_bytes(dtype)) % 16)
    return SV_ERR_UNSUPPORTED;
  PjParams p = {};
  p.V = V;
  p.H = H;
  p.M = int32_t(M);
  p.kblocks = int32_t((H + 255) / 256);
  p.n_vt = int32_t((V + kPjRows - 1) / kPjRows);
  // tiles of equal size; where there is more than one, they start on whole 64-row halves of a
  // scale tile
  p.n_nt = int32_t((M + kPjMaxN - 1) / kPjMaxN);
  if (p.n_nt == 1) {
    p.nt = int32_t((M + 15) / 16 * 16);
  } else {
    p.nt = int32_t(((M + p.n_nt - 1) / p.n_nt + 63) / 64 * 64);
    p.n_nt = int32_t((M + p.nt - 1) / p.nt);
  }
  if (int64_t(p.n_vt) * p.n_nt > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
  p.m_tiles = int32_t((M + 127) / 128);
  const uint32_t tile_bytes = format == SV_FP4_E8M0_32 ? 1024 : 2048;
  p.b_off = kPjABytes;
  p.sfa_off = p.b_off + uint32_t(p.nt) * 128;
  p.sfb_off = p.sfa_off + tile_bytes;
  p.stage_bytes = (p.sfb_off + 2 * tile_bytes + 1023) / 1024 * 1024;
  p.stages = int32_t(std::min<uint32_t>(kPjMaxStages, (kPjSmem - 1024) / p.stage_bytes));
  p.w_scales = w_scales;
  p.x_scales = x_scales;
  p.w_row = w_row_scales;
  p.x_row = x_row_scales;
  p.out = logits;
  p.ld = ld;
  p.status = status;
  const int sms = device_sm_count();
  if (sms <= 0) return SV_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const uint64_t row_bytes = uint64_t(spec_fp4_row_bytes(H));
  CUtensorMap map_w, map_x;
  {
    const uint64_t dims[2] = {row_bytes, uint64_t(V)};
    const uint64_t strides[1] = {row_bytes};
    const uint32_t box[2] = {128, kPjRows};
    if (!make_map(&map_w, w_packed, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return SV_ERR_CUDA;
  }
  {
    const uint64_t dims[2] = {row_bytes, uint64_t(M)};
    const uint64_t strides[1] = {row_bytes};
    const uint32_t box[2] = {128, uint32_t(p.nt)};
    if (!make_map(&map_x, x_packed, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_DATA_TYPE_UINT8))
      return SV_ERR_CUDA;
  }
  if (status && cudaMemsetAsync(status, 0, sizeof(int32_t), s) != cudaSuccess) return SV_ERR_CUDA;
  const int grid = int(std::min<int64_t>(sms, int64_t(p.n_vt) * p.n_nt));
  if (format == SV_FP4_E8M0_32)
    return dtype == SV_BF16 ? launch_project<SV_FP4_E8M0_32, __nv_bfloat16>(map_w, map_x, p, grid, s)
                            : launch_project<SV_FP4_E8M0_32, float>(map_w, map_x, p, grid, s);
  return dtype == SV_BF16 ? launch_project<SV_FP4_E4M3_16, __nv_bfloat16>(map_w, map_x, p, grid, s)
                          : launch_project<SV_FP4_E4M3_16, float>(map_w, map_x, p, grid, s);
}
