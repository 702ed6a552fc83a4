// fp4_project.cu -- logits from 4-bit hidden rows and a 4-bit output projection
// (spec_project_fp4): out[m][v] = sum_k x[m][k] w[v][k], both operands as quantised by
// spec_quantize_fp4.
//
// A persistent, warp-specialised tcgen05 GEMM on pairs of CTAs (cta_group::2).  W is the A operand
// (256 vocabulary rows per tile: TMEM lanes, 128 in each CTA), the hidden rows the B operand (up to
// 256 rows per tile: TMEM columns, half of them in each CTA's shared memory), K in blocks of 256
// elements: 128 bytes, one row of the 128-byte swizzle.
//   warp 0      TMA loads of this CTA's k-blocks of W, of its half of the hidden rows and of the
//               scale tiles into a ring; both CTAs' copies complete on the leader's barrier;
//   warp 1      in the leader, per k-block, tcgen05.cp of the scale tiles to both CTAs' TMEM and
//               four block-scaled tcgen05.mma (K = 64) into an accumulator;
//   warps 2-17  the epilogue: a lane quadrant and every fourth 16-column piece each, moved to
//               registers at once so that the accumulator is free again, then through shared
//               memory to the logits by TMA stores.
// The tensor cores apply the block scales and add in fp32; the row scales of SV_FP4_E4M3_16 are
// powers of two, applied to the sum in the epilogue (with kMinRow, kMaxRow, so that neither alone
// takes it out of binary32's range).
//
// Few rows are bound by reading W: 6 rows of 2560 on V = 151936 take 33.6 us, 6.2 TB/s.  384 rows with
// fp32 logits (207 MB read, 233 MB written) take 82 us, 5.4 TB/s.  1024 rows of 4096 on V = 129280 take
// 209 us in a loop of calls, 5.2 PFLOP/s, where the power cap holds the SMs at 1.77 GHz (the first
// hundred calls, at 2.07 GHz, 192); the tensor pipe is 62% active.  Wide tiles are bound by the ring: a
// stage's way round is longer than the products of the stages that fit (see where they are counted).
// At 1024 x 2560 on V = 151936, e8m0 (163 us), the hidden rows loaded for the first tile only give 158, the scale copies left out 163, two of four
// products left out with no loads but the scales' 101, with 40 us of products.  Scales copied a
// k-block ahead, with both k-blocks waited for, took 180.  What made the difference on the way:
//   - the issuing warps stay converged around elect.sync; in a branch on lane 0 each product took
//     125 ns to issue (6 rows 48 us, loads or not);
//   - pairs of CTAs: half of the hidden rows per SM (1024 rows of 4096: 432 -> 355 us);
//   - the accumulator is emptied at once and stored by TMA (355 -> 199, with the item before).
#include <algorithm>

#include "dependent.cuh"
#include "fp4.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace sv {
namespace {

constexpr int kPjRows = 128;    // vocabulary rows per CTA and tile
constexpr int kPjMaxN = 256;    // hidden rows per tile at most
constexpr int kPjEpiWarps = 16;
constexpr int kPjThreads = 32 * (2 + kPjEpiWarps);
constexpr uint32_t kPjABytes = kPjRows * 128;
constexpr uint32_t kPjSmem = 225 * 1024;  // ring and alignment slack
constexpr int kPjMaxStages = 10;
constexpr uint32_t kPjTmemCols = 512;

// Row scales of W between which a sum f of products may be multiplied by them first and by the row
// scale of the hidden row then.  f is 0 or 2^-20 <= |f| < 2^47 (codes of 0.5 under two scales of
// 2^-9, and 2^24 products of 2688^2), so f * w is a normal number and exact, and the second product
// rounds the logit once.  Other row scales (2^-120 .. 2^117 are possible) go through binary64; real
// weights never do.
constexpr float kMinRow = 0x1p-100f, kMaxRow = 0x1p64f;

struct PjParams {
  int32_t n_vt, n_nt, nt;  // tiles of 256 vocabulary rows, hidden-row tiles, their rows
  int32_t kblocks;
  int64_t H, V;
  int32_t M;
  int32_t n_acc;  // accumulators in TMEM
  int32_t stages;
  uint32_t stage_bytes, b_off, sfa_off, sfb_off;
  uint32_t out_off;  // the epilogue's staging buffers, behind the ring
  int32_t out_bufs;  // of them per warp, 1 or 2
  uint32_t tx_bytes;  // bytes both CTAs load per stage
  int32_t groups;     // scale groups per row
  const float* w_row;
  const float* x_row;
  void* out;
  int64_t ld;
  int32_t* status;
};

// ---- cluster pieces ------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The cluster-window address of `local` (a shared::cta address) in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// TMA loads of a CTA pair: the destination is this CTA's, `bar` the leader's barrier.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                             int32_t c1, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                             int32_t c1, int32_t c2, uint32_t bar,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void store_2d(const CUtensorMap* map, const void* src, int32_t c0,
                                         int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(c0), "r"(c1)
               : "memory");
}

// Tiles towards L2 ahead of their loads.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1)
               : "memory");
}

__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int32_t c0, int32_t c1,
                                            int32_t c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Arrive once on `bar` (the same offset in both CTAs) when all tcgen05 work issued so far is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

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

// One thread of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// pj_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool pj_wait_warp(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, pj_wait(bar, parity, status));
}

// Shared-memory descriptors by halves: the low word holds the address (>> 4) and the leading
// offset, the high word is a constant of the layout, so that moving to another stage, tile or
// K-step is one 32-bit addition.  Operands: 128-byte swizzle (tc.cuh).  Scale tiles: 32 rows of 16
// bytes without swizzle, core matrices of 8 rows by 16 bytes 128 bytes apart.
constexpr uint32_t kOperandHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kOperandLo = 1u << 16;
constexpr uint32_t kScaleHi = (128u >> 4) | (1u << 14);

__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}

// 512 bytes of scales to four TMEM columns, the 32 lanes repeated in every lane quadrant.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(desc_of(lo, kScaleHi))
               : "memory");
}

// Instruction descriptor of the block-scaled 4-bit kinds: e2m1 A and B (1 in bits [7,10) and
// [10,12)), both K-major, N >> 3 in [17,23), scale type in bit 23 (1: e8m0, 0: e4m3), M >> 7 in
// [27,29) (M = 256 over the pair); the scale ids of B and A go to [4,6) and [29,31).
constexpr uint32_t pj_idesc(int32_t n, bool e8m0) {
  return (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (e8m0 ? 1u << 23 : 0u) | (2u << 27);
}

// 16 columns of this thread's TMEM lane, in flight until the next tcgen05.wait::ld.
__device__ __forceinline__ void tmem_load16_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

// Uses of v stay behind the wait before this.
__device__ __forceinline__ void tmem_landed(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                 "+f"(v[13]), "+f"(v[14]), "+f"(v[15])::"memory");
}

template <int kFmt>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  if constexpr (kFmt == SV_FP4_E8M0_32) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(sfa), "r"(sfb)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(sfa), "r"(sfb)
        : "memory");
  }
}

// One k-block: the scale tiles of W and of kX tiles of the hidden rows to TMEM, then `ksteps`
// products of K = 64.  Everything but the K-steps of the last k-block is known at compile time: a
// single thread issues all of this, and its instructions, not the tensor cores, set the pace of
// small tiles.
template <int kFmt, int kX>
__device__ __forceinline__ void k_block(uint32_t stage, uint32_t b_off, uint32_t sfa_off,
                                        uint32_t sfb_off, uint32_t acc, uint32_t sfa,
                                        uint32_t sfb_shift, uint32_t idesc, int32_t ksteps,
                                        bool accumulate) {
  constexpr int kGroups = kFmt == SV_FP4_E8M0_32 ? 2 : 4;
  const uint32_t sfb = sfa + kGroups * 4;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    copy_scales(sfa + g * 4, stage + sfa_off + g * 32);
#pragma unroll
    for (int x = 0; x < kX; ++x)
      copy_scales(sfb + (g * kX + x) * 4, stage + sfb_off + (x * kGroups + g) * 32);
  }
  const uint32_t a_lo = stage + kOperandLo, b_lo = a_lo + b_off;
  const uint32_t sfbs = sfb + sfb_shift;
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    if (ks >= ksteps) break;
    const int g = kGroups == 4 ? ks : ks >> 1;
    const uint32_t id = kGroups == 4 ? 0u : (ks & 1) ? (2u << 4) | (2u << 29) : 0u;
    mma_fp4<kFmt>(acc, desc_of(a_lo + ks * 2, kOperandHi), desc_of(b_lo + ks * 2, kOperandHi),
                  idesc | id, sfa + g * 4, sfbs + g * kX * 4, accumulate || ks != 0);
  }
}

__device__ __forceinline__ void put(float* o, float y) { *o = y; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float y) { *o = __float2bfloat16_rn(y); }

template <int kFmt, int kX, typename Out>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPjThreads, 1)
    project_kernel(const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_ws,
                   const __grid_constant__ CUtensorMap map_xs,
                   const __grid_constant__ CUtensorMap map_out, PjParams p) {
  constexpr int kGroups = kFmt == SV_FP4_E8M0_32 ? 2 : 4;  // scale groups per k-block
  constexpr uint32_t kSfCols = kGroups * 4 * (1 + kX);
  constexpr int kPieces = kX == 1 ? 2 : 4;  // 16-column pieces per epilogue warp
  constexpr uint32_t kOutBytes = 16 * 32 * sizeof(Out);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kPjMaxStages], empty[kPjMaxStages];  // full: the leader's
  __shared__ uint64_t acc_full[2], acc_empty[2], drain;         // acc_empty: the leader's
  __shared__ uint32_t tmem_base;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int32_t n_items = p.n_vt * p.n_nt;
  const int32_t stages = p.stages;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 2 * kPjEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base)),
                 "r"(kPjTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  // Programmatic dependent of the work before it: all above ran beside that work's end, and nothing
  // it wrote (or that still reads the logits) is touched before dependent_start.  W's first tiles
  // are on their way to L2 meanwhile; should that work still write W, its writes meet them there.
  if (warp == 0 && elect_one()) {
    const int32_t vt = (pair / p.n_nt) * 2 + int32_t(rank);
    for (int32_t kb = 0; kb < min(stages, p.kblocks); ++kb) {
      prefetch_2d(&map_w, kb * 128, vt * kPjRows);
      prefetch_3d(&map_ws, 0, kb * kGroups, vt);
    }
  }
  __syncwarp();
  dependent_start();
  // the only report is of a wait that ran out, a second after the start at the earliest
  if (blockIdx.x == 0 && tid == 0 && p.status) *p.status = 0;
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before anything arrives on them
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base;
  const uint32_t sf_base = tmem + kPjTmemCols - 2 * kSfCols;  // two buffers of scale columns

  if (warp == 0) {
    const uint64_t keep = tc::policy_evict_last(), once = tc::policy_evict_first();
    const uint64_t w_policy = p.n_nt > 1 ? keep : once;
    const uint32_t ring_at = smem_addr(ring);
    int32_t st = 0;
    uint32_t phase = 1;  // a ring stage starts out empty
    int32_t issued = 0;  // stages filled at least once
    uint32_t dst = ring_at, bar = map_rank(smem_addr(&full[0]), 0);
    const uint32_t bar0 = bar;
    bool ok = true;
    for (int32_t item = pair; item < n_items && ok; item += n_pairs) {
      const int32_t vt = (item / p.n_nt) * 2 + int32_t(rank), n0 = (item % p.n_nt) * p.nt;
      // the products take their N columns half from each CTA
      const int32_t x0 = n0 + int32_t(rank) * (min(p.nt, (p.M - n0 + 15) & ~15) >> 1);
      for (int32_t kb = 0; kb < p.kblocks; ++kb) {
        if (!pj_wait_warp(&empty[st], phase, p.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(&full[st], p.tx_bytes);
          pair_load_2d(dst, &map_w, kb * 128, vt * kPjRows, bar, w_policy);
          pair_load_2d(dst + p.b_off, &map_x, kb * 128, x0, bar, keep);
          pair_load_3d(dst + p.sfa_off, &map_ws, 0, kb * kGroups, vt, bar, w_policy);
          pair_load_3d(dst + p.sfb_off, &map_xs, 0, kb * kGroups, n0 >> 7, bar, keep);
        }
        __syncwarp();
        issued = max(issued, st + 1);
        dst += p.stage_bytes;
        bar += 8;
        if (++st == stages) {
          st = 0;
          phase ^= 1;
          dst = ring_at;
          bar = bar0;
        }
      }
    }
    // both CTAs' copies in flight land before either block may end: of each stage that was
    // filled, the last fill (of this turn of the ring below st, of the one before from st on)
    if (rank == 0)
      for (int32_t k = 0; k < issued; ++k)
        pj_wait_warp(&full[k], k < st ? phase ^ 1 : phase, p.status);
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t ring_lo = smem_addr(ring) >> 4, stage_lo = p.stage_bytes >> 4;
      const uint32_t b_off = p.b_off >> 4, sfa_off = p.sfa_off >> 4, sfb_off = p.sfb_off >> 4;
      const int32_t last_steps = int32_t((p.H - int64_t(p.kblocks - 1) * 256 + 63) >> 6);
      int32_t st = 0, a = 0;
      uint32_t phase = 0, stage = ring_lo, sfa = sf_base;
      uint32_t acc_phase = 1;  // the accumulators start out empty
      bool ok = true;
      for (int32_t item = pair; item < n_items && ok; item += n_pairs) {
        const int32_t n0 = (item % p.n_nt) * p.nt;
        const uint32_t idesc =
            pj_idesc(min(p.nt, (p.M - n0 + 15) & ~15), kFmt == SV_FP4_E8M0_32);
        const uint32_t shift = (n0 & 127) >> 5;
        const uint32_t acc = tmem + a * p.nt;
        if (!pj_wait_warp(&acc_empty[a], acc_phase, p.status)) break;
        tc::fence_after_sync();
        for (int32_t kb = 0; kb < p.kblocks; ++kb) {
          if (!pj_wait_warp(&full[st], phase, p.status)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          if (elect_one()) {
            k_block<kFmt, kX>(stage, b_off, sfa_off, sfb_off, acc, sfa, shift, idesc,
                              kb + 1 == p.kblocks ? last_steps : 4, kb != 0);
            pair_commit(&empty[st]);
          }
          __syncwarp();
          sfa = sfa == sf_base ? sf_base + kSfCols : sf_base;
          stage += stage_lo;
          if (++st == stages) {
            st = 0;
            phase ^= 1;
            stage = ring_lo;
          }
        }
        if (ok && elect_one()) pair_commit(&acc_full[a]);
        __syncwarp();
        if (++a == p.n_acc) {
          a = 0;
          acc_phase ^= 1;
        }
      }
      // nothing reads shared or tensor memory once this has passed
      if (elect_one()) pair_commit(&drain);
      __syncwarp();
      pj_wait_warp(&drain, 0, p.status);
    }
  } else {
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t lanes = tmem + (uint32_t(32 * q) << 16);
    const uint32_t freed = map_rank(smem_addr(acc_empty), 0);
    // this warp's staging buffers of 16 rows of 32 logits
    const bool two = p.out_bufs == 2;
    uint8_t* const stage0 = ring + p.out_off + (warp - 2) * p.out_bufs * kOutBytes;
    bool failed = false;
    int32_t a = 0, buf = 0;
    uint32_t phase = 0;
    for (int32_t item = pair; item < n_items; item += n_pairs) {
      const int32_t vt = (item / p.n_nt) * 2 + int32_t(rank), n0 = (item % p.n_nt) * p.nt;
      const int32_t v0 = vt * kPjRows + 32 * q;
      const int32_t n = min(p.nt, p.M - n0);
      float ws = 1.f, xs[kPieces];
      if constexpr (kFmt == SV_FP4_E4M3_16) {
        if (v0 + lane < p.V) ws = p.w_row[v0 + lane];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {  // lane j holds column j's row scale
          const int32_t c = 16 * (h + 4 * i) + (lane & 15);
          xs[i] = c < n ? p.x_row[n0 + c] : 0.f;
        }
      }
      if (!failed && !pj_wait(&acc_full[a], phase, p.status)) failed = true;
      __syncwarp();
      tc::fence_after_sync();
      float f[kPieces][16];
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (16 * (h + 4 * i) < n) tmem_load16_async(lanes + a * p.nt + 16 * (h + 4 * i), f[i]);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int i = 0; i < kPieces; ++i) tmem_landed(f[i]);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_cluster(freed + a * 8);
      if (++a == p.n_acc) {
        a = 0;
        phase ^= 1;
      }
      if (v0 >= p.V) continue;
      const bool plain_rows =
          kFmt != SV_FP4_E4M3_16 || __all_sync(0xffffffffu, ws >= kMinRow && ws <= kMaxRow);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int32_t c = 16 * (h + 4 * i);
        if (c >= n) break;
        if constexpr (kFmt == SV_FP4_E4M3_16) {
          if (plain_rows) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              f[i][j] = f[i][j] * ws * __shfl_sync(0xffffffffu, xs[i], j);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              f[i][j] = static_cast<float>(double(f[i][j]) * double(ws) *
                                           double(__shfl_sync(0xffffffffu, xs[i], j)));
          }
        }
        if (v0 + 32 > p.V) {  // a TMA store clips a row at 16 bytes only: these 32 one by one
          Out* const o = static_cast<Out*>(p.out) + int64_t(n0 + c) * p.ld + v0 + lane;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < n && v0 + lane < p.V) put(o + j * p.ld, f[i][j]);
          continue;
        }
        uint8_t* const st = stage0 + buf * kOutBytes;
        if (two) {
          buf ^= 1;
          tc::bulk_wait_read<1>();  // the store before the last has read this buffer
        } else {
          tc::bulk_wait_read<0>();
        }
        __syncwarp();
        if constexpr (sizeof(Out) == 4) {
#pragma unroll
          for (int j = 0; j < 16; ++j) reinterpret_cast<float*>(st)[j * 32 + lane] = f[i][j];
        } else {
          // rows j and j + 1 at once: an even lane takes (v, v + 1) of row j, an odd one
          // (v - 1, v) of row j + 1
          uint32_t* const o = reinterpret_cast<uint32_t*>(st) + (lane & 1) * 16 + (lane >> 1);
          const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(f[i][j], f[i][j + 1]);
            const uint32_t mine = *reinterpret_cast<const uint32_t*>(&two);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
            o[j * 16] = __byte_perm(mine, other, pick);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (elect_one()) {
          store_2d(&map_out, st, v0, n0 + c);  // clipped at M
          tc::bulk_commit();
        }
        __syncwarp();
      }
    }
    tc::bulk_wait_all();
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // neither CTA's memory goes away while the other's work may touch it
  if (warp == 1) {
    tc::fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kPjTmemCols)
                 : "memory");
  }
}

struct PjMaps {
  CUtensorMap w, x, ws, xs, out;
};

template <int kFmt, int kX, typename Out>
sv_status launch_project(const PjMaps& m, const PjParams& p, int grid, cudaStream_t s) {
  auto* kern = project_kernel<kFmt, kX, Out>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kPjSmem)) !=
      cudaSuccess)
    return SV_ERR_CUDA;
  return launch_dependent(kern, unsigned(grid), kPjThreads, kPjSmem, s, m.w, m.x, m.ws, m.xs, m.out,
                          p);
}

template <int kFmt, int kX>
sv_status launch_project(const PjMaps& m, const PjParams& p, sv_dtype dtype, int grid,
                         cudaStream_t s) {
  return dtype == SV_BF16 ? launch_project<kFmt, kX, __nv_bfloat16>(m, p, grid, s)
                          : launch_project<kFmt, kX, float>(m, p, grid, s);
}

// A tensor map of `type` elements; dims[0] is the contiguous one, strides in bytes for dims 1 ..;
// what lies outside loads as zero.
bool typed_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
               const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle,
               CUtensorMapDataType type) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3], es[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
  }
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return fn(map, type, rank, const_cast<void*>(base), d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rows_map(CUtensorMap* map, const uint8_t* base, int64_t rows, uint64_t row_bytes,
              uint32_t box_rows) {
  const uint64_t dims[2] = {row_bytes, uint64_t(rows)};
  const uint64_t strides[1] = {row_bytes};
  const uint32_t box[2] = {128, box_rows};
  return typed_map(map, base, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_DATA_TYPE_UINT8);
}

// Scale tiles as [row tile][group][128 words]; a row tile that does not exist loads as zeros.
bool scales_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int32_t groups,
                uint32_t box_groups, uint32_t box_tiles) {
  const uint64_t dims[3] = {128, uint64_t(groups), uint64_t((rows + 127) / 128)};
  const uint64_t strides[2] = {512, uint64_t(groups) * 512};
  const uint32_t box[3] = {128, box_groups, box_tiles};
  return typed_map(map, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_DATA_TYPE_UINT32);
}

bool logits_map(CUtensorMap* map, const void* out, sv_dtype dtype, int64_t M, int64_t V,
                int64_t ld) {
  const uint64_t dims[2] = {uint64_t(V), uint64_t(M)};
  const uint64_t strides[1] = {uint64_t(ld) * uint64_t(elem_bytes(dtype))};
  const uint32_t box[2] = {32, 16};
  return typed_map(map, out, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                  dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) return reset_status(status, s);
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
  p.n_vt = int32_t((V + 2 * kPjRows - 1) / (2 * kPjRows));
  // tiles of equal size; where there is more than one, they start on whole 64-row halves of a
  // scale tile
  p.n_nt = int32_t((M + kPjMaxN - 1) / kPjMaxN);
  // (narrower, down to 64 rows, while there are fewer tiles than pairs of SMs: 1100 rows on V = 1000,
  // H = 7168 15.9 -> 12.5 us)
  const int sms = device_sm_count();
  if (sms < 2) return SV_ERR_CUDA;
  p.n_nt = std::max(p.n_nt, int32_t(std::min<int64_t>((M + 63) / 64, sms / 2 / p.n_vt)));
  if (p.n_nt == 1) {
    p.nt = int32_t((M + 15) / 16 * 16);
  } else {
    p.nt = int32_t(((M + p.n_nt - 1) / p.n_nt + 63) / 64 * 64);
    p.n_nt = int32_t((M + p.nt - 1) / p.nt);
  }
  if (int64_t(p.n_vt) * p.n_nt > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
  const bool e8m0 = format == SV_FP4_E8M0_32;
  const uint32_t box_groups = e8m0 ? 2 : 4;
  const uint32_t x_tiles = p.nt > 128 ? 2 : 1;  // scale tiles that a tile's rows can lie in
  const uint32_t sf_cols = box_groups * 4 * (1 + x_tiles);
  p.n_acc = 2 * p.nt + 2 * sf_cols <= kPjTmemCols ? 2 : 1;
  p.groups = fp4_groups(H, format);
  p.b_off = kPjABytes;
  p.sfa_off = p.b_off + uint32_t(p.nt / 2) * 128;
  p.sfb_off = p.sfa_off + box_groups * 512;
  const uint32_t bytes = p.sfb_off + x_tiles * box_groups * 512;
  p.tx_bytes = 2 * bytes;
  p.stage_bytes = (bytes + 1023) / 1024 * 1024;
  // A stage is away for 1.6 us or more, from the products that free it to the arrival of its next
  // copies, and the products of five stages take 1.3 (256 rows), so every stage counts (1024 rows of
  // 2560: 206 us with three, 175 with four, 164 with five).  Wide tiles give up their second staging
  // buffers where that makes room for a stage: 384 rows with fp32 logits 84.6 -> 81.2 us (e4m3 93.8 ->
  // 85.7), 1024 rows of 4096 6% less.  A single tile with five stages and up to 128 rows do better
  // with both (160 rows 52.1 for 54.7, 128 rows 49.5 for 52.4).
  const uint32_t out_bytes = kPjEpiWarps * 16 * 32 * uint32_t(elem_bytes(dtype));
  auto stages_with = [&](uint32_t bufs) {
    return std::min<uint32_t>(kPjMaxStages, (kPjSmem - 1024 - bufs * out_bytes) / p.stage_bytes);
  };
  const bool wide = p.nt > 128 && (p.n_nt > 1 || stages_with(2) < 5);
  p.out_bufs = wide && stages_with(1) > stages_with(2) ? 1 : 2;
  p.stages = int32_t(stages_with(uint32_t(p.out_bufs)));
  p.out_off = uint32_t(p.stages) * p.stage_bytes;
  p.w_row = w_row_scales;
  p.x_row = x_row_scales;
  p.out = logits;
  p.ld = ld;
  p.status = status;

  const uint64_t row_bytes = uint64_t(spec_fp4_row_bytes(H));
  PjMaps m;
  if (!rows_map(&m.w, w_packed, V, row_bytes, kPjRows) ||
      !rows_map(&m.x, x_packed, M, row_bytes, uint32_t(p.nt / 2)) ||
      !scales_map(&m.ws, w_scales, V, p.groups, box_groups, 1) ||
      !scales_map(&m.xs, x_scales, M, p.groups, box_groups, x_tiles) ||
      !logits_map(&m.out, logits, dtype, M, V, ld))
    return SV_ERR_CUDA;
  const int grid = 2 * int(std::min<int64_t>(sms / 2, int64_t(p.n_vt) * p.n_nt));
  if (e8m0)
    return x_tiles == 1 ? launch_project<SV_FP4_E8M0_32, 1>(m, p, dtype, grid, s)
                        : launch_project<SV_FP4_E8M0_32, 2>(m, p, dtype, grid, s);
  return x_tiles == 1 ? launch_project<SV_FP4_E4M3_16, 1>(m, p, dtype, grid, s)
                      : launch_project<SV_FP4_E4M3_16, 2>(m, p, dtype, grid, s);
}
