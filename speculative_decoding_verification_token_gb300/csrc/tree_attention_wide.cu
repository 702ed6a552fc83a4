// tree_attention_wide.cu -- attention of many rows over the paged cache: the kernel of
// spec_tree_attention for more than 64 rows a key head (trees under many query heads, prompts).
//
// With rows enough to fill a matrix instruction the products, not the cache's bytes, are what counts, and
// operands that shared memory must deliver (128 bytes a clock, just what 128 x 128 products with both
// operands there read).  So here rows lie in the TMEM lanes, S = Q K^T and O += P V, and P, which is
// computed from S, goes back to tensor memory, over the S it came from, and is read there.  A thread has
// a row to itself: maxima and sums need no other thread.
//   Two streams share the tensor cores, each with its S, its O and four softmax warps: while one takes
//   exponentials, the other's products run.  They are two tiles of 128 rows over the same keys, or, where
//   an item has one tile only, its odd and even key tiles, joined at the end.
//   warps 0-3, 4-7  softmax and results of stream 0, 1; 8, 11 loads; 9 products; 10 items.
// m is raised, and O scaled, only when a row's score passes it by more than 8 (as in tree_attention.cu).
#include "tree_attention.cuh"

namespace sv {
namespace attn {
namespace {

// A warp's results go out through shared memory, 64 bytes of each of its 32 rows at a time, so that four
// lanes write a row's 64 bytes (16 bytes of 32 rows at once take four times as long).  80 bytes apart the
// rows' pieces lie in different banks.
constexpr int kStageRow = 80;
constexpr int kBadWords = kWide / 32;  // (an item has up to 256 rows of a chain, with a head a key head)

template <int kD>
struct WideShared {
  static constexpr uint32_t kSlot = kTile * kD * 2;
  static constexpr uint32_t kQTile = kTile * kD * 2;
  struct Small {
    uint64_t full[16], empty[16], item_full[2], item_empty[2], table_full[2];
    uint64_t q_full, q_empty, s_full[2], p_half[2], p_full[2], o_full[2], drain;
    Item item[2];
    alignas(16) uint32_t above[2][SV_MAX_TREE_ROWS][4];
    int32_t up[SV_MAX_TREE_ROWS];
    uint32_t bad[2][2][kBadWords];  // an item's rows whose values are not all finite, by who found it
    float m[kTile], l[kTile];                   // of stream 1, for joining
    alignas(16) uint8_t stage[kSoftWarps][32 * kStageRow];  // results on their way out
    uint32_t tmem;
    int32_t err, cut_columns;
  };
  static constexpr uint32_t kSmall = (sizeof(Small) + 127) / 128 * 128;
  static constexpr int kStages() {
    const int s = int((kAttnSmem - 1024 - kSmall - 2 * kQTile) / kSlot);
    return s < 16 ? s : 16;
  }
};

// 32 columns of this thread's TMEM lane, in flight until wait_loads; uses stay behind landed.
__device__ __forceinline__ void load32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wait_loads() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void landed(float* v) {
#pragma unroll
  for (int j = 0; j < 32; j += 8)
    asm volatile(""
                 : "+f"(v[j]), "+f"(v[j + 1]), "+f"(v[j + 2]), "+f"(v[j + 3]), "+f"(v[j + 4]),
                   "+f"(v[j + 5]), "+f"(v[j + 6]), "+f"(v[j + 7])::"memory");
}

__device__ __forceinline__ void store16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void wait_stores() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] B[smem]: A's rows in the lanes, two 16-bit elements of the contraction a column.
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                              bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

// Barrier of all softmax warps that also tells whether `x` held in any thread.
__device__ __forceinline__ bool both_any(bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, 3, 256, q;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(uint32_t(x))
      : "memory");
  return any != 0;
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&two);
}

template <int kD, int kLoaders>
__global__ void __launch_bounds__(kAttnThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap map_q,
                const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  using Sh = WideShared<kD>;
  constexpr int kStages = Sh::kStages();
  static_assert(kStages >= 3, "a ring of three tiles");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const q_at = ring + kStages * Sh::kSlot;
  typename Sh::Small& sm = *reinterpret_cast<typename Sh::Small*>(q_at + 2 * Sh::kQTile);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], kLoaders);  // their parts
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.item_full[b], 1);
      mbar_init(&sm.item_empty[b], 3 + kLoaders);  // the loads, the products, the streams
      mbar_init(&sm.table_full[b], 1);
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.p_half[b], 4);
      mbar_init(&sm.p_full[b], 4);
      mbar_init(&sm.o_full[b], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    fence_barrier_init();
    sm.err = 0;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&sm.tmem, 512);
  if (warp == kLoadWarp && elect()) {
    prefetch_map(&map_q);
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  __syncwarp();
  tc::fence_before_sync();
  dependent_start();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;  // S (and P) of the streams at 0 and 128, O at 256 and 384
  int32_t* const err = &sm.err;
  const WsLayout wl = ws_layout(gridDim.x, kWide, kD);
  const int32_t tile_rows = p.tile_tokens * p.group;
  if (warp == kItemWarp) {
    // ---- the items ---------------------------------------------------------------------------------
    int64_t built[2] = {-1, -1};
    const int32_t columns = walk_items<1>(
        p, reinterpret_cast<Cut*>(p.ws + wl.cuts), sm.item, sm.item_full, sm.item_empty, err,
        [&](int b, const Item& x, int64_t first) {
          if (!p.rd.parents) return;
          const int64_t key = int64_t(x.r) << 32 | x.tok0;
          if (x.t1 * int64_t(kTile) > x.base0 && built[b] != key) {
            built[b] = key;
            build_above(p, first, x.end - x.ctx, sm.up, sm.above[b], err);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.table_full[b]);
        });
    if (lane == 0) sm.cut_columns = columns;
  } else if (warp == kLoadWarp || (kLoaders == 2 && warp == kLoadWarp2)) {
    // ---- the loads -----------------------------------------------------------------------------------
    // in the order of use: K of the first tile (two streams of tiles: the first two), then V of a tile
    // and K of the next one that its stream needs
    const uint64_t once = tc::policy_evict_first();
    const int part = kLoaders == 2 && warp == kLoadWarp2;
    int32_t slot = 0, filled = 0, items = 0;
    uint32_t phase = 1;
    bool ok = true;
    auto load = [&](const CUtensorMap* map, int32_t page, int32_t from, int32_t boxes, int32_t head) {
      if (!wait_for_warp(&sm.empty[slot], phase, err)) return false;
      load_tile<kD, kLoaders, true>(p, ring + slot * Sh::kSlot, map, part, page, from, boxes, head,
                              &sm.full[slot], once);
      filled = max(filled, slot + 1);
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
      return true;
    };
    for (int32_t it = 0; ok; ++it) {
      const int b = it & 1;
      if (!wait_for_warp(&sm.item_full[b], (it >> 1) & 1, err)) break;
      const Item x = sm.item[b];
      if (x.stop) break;
      const bool twin = x.columns <= tile_rows;
      const int32_t n = x.t1 - x.t0, ahead = min(n, twin ? 2 : 1);
      // pages of the tiles whose V is still to come
      int32_t page[2] = {}, from[2] = {}, boxes[2] = {};
      for (int32_t i = 0; i < n + ahead && ok; ++i) {
        if (i >= ahead) ok = load(&map_v, page[0], from[0], boxes[0], x.head);
        if (i >= ahead) page[0] = page[1], from[0] = from[1], boxes[0] = boxes[1];
        if (i < n && ok) {
          int32_t pg, fr;
          const int32_t bx = tile_boxes<kD, kLoaders>(p, x, x.t0 + i, part, pg, fr, err);
          ok = load(&map_k, pg, fr, bx, x.head);
          const bool second = i >= 1 && ahead == 2;
          if (second) page[1] = pg, from[1] = fr, boxes[1] = bx;
          else page[0] = pg, from[0] = fr, boxes[0] = bx;
        }
        if (i == ahead - 1 && ok && part == 0) {
          ok = it == 0 || wait_for_warp(&sm.q_empty, (it - 1) & 1, err);
          if (ok && elect()) {
            // (rows behind the request's last hold anything: nobody reads what becomes of them)
            const int tiles = twin ? 1 : 2;
            mbar_expect_tx(&sm.q_full, uint32_t(tiles * tile_rows) * kD * 2);
            for (int s = 0; s < tiles; ++s) {
#pragma unroll
              for (int k = 0; k < kD / 64; ++k)
                tc::tma_load_3d(q_at + s * Sh::kQTile + k * 16384, &map_q, k * 64,
                                x.head * p.group, int32_t(x.first_row) + s * p.tile_tokens,
                                &sm.q_full);
            }
          }
          __syncwarp();
          if (ok) items = it + 1;
        }
      }
      if (lane == 0) mbar_arrive(&sm.item_empty[b]);
    }
    // every copy in flight lands before the CTA may end
    for (int32_t k = 0; k < filled; ++k)
      wait_for_warp(&sm.full[k], k < slot ? phase ^ 1 : phase, err);
    if (items > 0) wait_for_warp(&sm.q_full, (items - 1) & 1, err);
  } else if (warp == kMmaWarp) {
    // ---- the products --------------------------------------------------------------------------------
    // (bit 13: Q negated, so that the scale is positive)
    const uint32_t kIdS = tc::idesc_bf16_f32(128, 128) | (p.scale2 < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t kIdO = tc::idesc_bf16_f32(128, kD) | (1u << 16);
    const uint32_t ring_lo = desc_at(ring), q_lo = desc_at(q_at);
    int32_t slot = 0;
    uint32_t phase = 0, p_phase[2] = {0, 0};
    bool ok = true;
    auto next_slot = [&] {
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto scores = [&](int s, int q, int32_t at) {  // S of stream s from row tile q and ring slot `at`
      const uint32_t k_lo = (ring_lo + at * (Sh::kSlot >> 4)) | kAlongK;
      const uint32_t a_lo = (q_lo + q * (Sh::kQTile >> 4)) | kAlongK;
#pragma unroll
      for (int k = 0; k < kD / 16; ++k)
        tc::mma_bf16(tmem + s * 128, desc_of(a_lo + (k >> 2) * 1024 + (k & 3) * 2),
                     desc_of(k_lo + (k >> 2) * 1024 + (k & 3) * 2), kIdS, k > 0);
      tc::mma_commit(&sm.s_full[s]);
    };
    // O of stream s (+)= P V, for the first or second half of the places
    auto values = [&](int s, int32_t at, int half, bool first) {
      const uint32_t v_lo = ring_lo + at * (Sh::kSlot >> 4) + kAcross;
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) {
        const int k = half * (kTile / 32) + i;
        mma_from_tmem(tmem + 256 + s * 128, tmem + s * 128 + k * 8, desc_of(v_lo + k * 128), kIdO,
                      !first || k > 0);
      }
    };
    for (int32_t it = 0; ok; ++it) {
      const int b = it & 1;
      if (!wait_for_warp(&sm.item_full[b], (it >> 1) & 1, err)) break;
      const Item x = sm.item[b];
      if (x.stop) break;
      const bool twin = x.columns <= tile_rows;
      const int32_t n = x.t1 - x.t0;
      if (!wait_for_warp(&sm.q_full, it & 1, err)) break;
      const int32_t ahead = min(n, twin ? 2 : 1);
      for (int32_t i = 0; i < ahead && ok; ++i) {
        ok = wait_for_warp(&sm.full[slot], phase, err);
        if (!ok) break;
        tc::fence_after_sync();
        if (elect()) {
          scores(i, 0, slot);
          if (!twin) scores(1, 1, slot);
          tc::mma_commit(&sm.empty[slot]);
          if (i + 1 == n) tc::mma_commit(&sm.q_empty);
        }
        __syncwarp();
        next_slot();
      }
      for (int32_t i = 0; i < n && ok; ++i) {
        const int32_t v_slot = slot;
        ok = wait_for_warp(&sm.full[slot], phase, err);
        next_slot();
        const bool more = i + 1 < n;  // (of a pair)
        if (twin) {
          const int s = i & 1;
          ok = ok && wait_for_warp(&sm.p_half[s], p_phase[s], err);
          if (!ok) break;
          tc::fence_after_sync();
          if (elect()) values(s, v_slot, 0, i < 2);
          __syncwarp();
          ok = wait_for_warp(&sm.p_full[s], p_phase[s], err);
          if (!ok) break;
          p_phase[s] ^= 1;
          tc::fence_after_sync();
          if (elect()) {
            values(s, v_slot, 1, i < 2);
            tc::mma_commit(&sm.empty[v_slot]);
            if (i + 2 >= n) tc::mma_commit(&sm.o_full[s]);
          }
          __syncwarp();
          if (i + 2 < n) {
            ok = wait_for_warp(&sm.full[slot], phase, err);
            if (!ok) break;
            tc::fence_after_sync();
            if (elect()) {
              scores(s, 0, slot);
              tc::mma_commit(&sm.empty[slot]);
              if (i + 3 == n) tc::mma_commit(&sm.q_empty);
            }
            __syncwarp();
            next_slot();
          }
        } else {
          // a tile whose values are looked through waits for both streams' look
          const bool masked = (x.t0 + i + 1) * int64_t(kTile) > x.base0;
          ok = ok && wait_for_warp(&sm.p_half[0], p_phase[0], err) &&
               (!masked || wait_for_warp(&sm.p_half[1], p_phase[1], err));
          if (!ok) break;
          tc::fence_after_sync();
          if (elect()) values(0, v_slot, 0, i == 0);
          __syncwarp();
          ok = wait_for_warp(&sm.p_full[0], p_phase[0], err);
          if (!ok) break;
          tc::fence_after_sync();
          if (elect()) {
            values(0, v_slot, 1, i == 0);
            if (!more) tc::mma_commit(&sm.o_full[0]);
          }
          __syncwarp();
          const int32_t k_slot = slot;
          if (more) {
            ok = wait_for_warp(&sm.full[slot], phase, err);
            if (!ok) break;
            next_slot();
            tc::fence_after_sync();
            if (elect()) scores(0, 0, k_slot);
            __syncwarp();
          }
          ok = wait_for_warp(&sm.p_half[1], p_phase[1], err);
          if (!ok) break;
          tc::fence_after_sync();
          if (elect()) values(1, v_slot, 0, i == 0);
          __syncwarp();
          ok = wait_for_warp(&sm.p_full[1], p_phase[1], err);
          if (!ok) break;
          p_phase[0] ^= 1;
          p_phase[1] ^= 1;
          tc::fence_after_sync();
          if (elect()) {
            values(1, v_slot, 1, i == 0);
            tc::mma_commit(&sm.empty[v_slot]);
            if (!more) {
              tc::mma_commit(&sm.o_full[1]);
            } else {
              scores(1, 1, k_slot);
              tc::mma_commit(&sm.empty[k_slot]);
              if (i + 2 == n) tc::mma_commit(&sm.q_empty);
            }
          }
          __syncwarp();
        }
      }
      if (lane == 0) mbar_arrive(&sm.item_empty[b]);
    }
    // nothing reads shared or tensor memory once this has passed
    if (elect()) tc::mma_commit(&sm.drain);
    __syncwarp();
    wait_for_warp(&sm.drain, 0, err);
  } else if (warp < kSoftWarps) {
    // ---- softmax and results -------------------------------------------------------------------------
    const int s = warp >> 2, quad = warp & 3;
    const int row = tid & 127;  // of the stream's tile; place of a key tile where values are looked through
    const uint32_t lanes = tmem + (uint32_t(32 * quad) << 16);
    const uint32_t s_at = lanes + s * 128, o_at = lanes + 256 + s * 128;
    const float scale1 = fabsf(p.scale2);
    const float2 scale = splat2(scale1);
    uint32_t s_phase = 0, o_phase = 0;
    int32_t loads = 0;  // tiles that went through the ring before this item
    bool failed = false;  // a wait ran out: no further ones, on to where all meet
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!failed && !wait_for(bar, parity, err)) failed = true;
    };
    for (int32_t it = 0;; ++it) {
      const int b = it & 1;
      wait(&sm.item_full[b], (it >> 1) & 1);
      if (both_any(failed)) break;
      const Item& x = sm.item[b];  // (not in registers: a row's scores want them)
      if (x.stop) break;
      const bool twin = x.columns <= tile_rows;
      const int32_t n = x.t1 - x.t0, ahead = twin ? 2 : 1;
      // this thread's token in the item, and its column
      auto token = [&] { return (twin ? 0 : s * p.tile_tokens) + row / p.group; };
      auto column_of = [&] { return (twin ? 0 : s * tile_rows) + row; };
      auto is_mine = [&] { return row < tile_rows && column_of() < x.columns; };
      if (row < kBadWords) sm.bad[b][s][row] = 0;
      soft_sync(s);
      float m = kM2Empty, l = 0.f;
      bool table = !p.rd.parents, fresh = true;
      const int32_t mask_from = x.base0 / kTile - x.t0;  // tiles from here on hold places not all see
      for (int32_t i = twin ? s : 0; i < n; i += ahead) {
        const bool masked = i >= mask_from;
        wait(&sm.s_full[s], s_phase);
        s_phase ^= 1;
        uint32_t seen[4];  // bit c of word w: this row sees place 32 w + c of the tile
        if (masked) {
          if (!table) wait(&sm.table_full[b], (it >> 1) & 1);
          table = true;
          const int32_t i_item = token();
          const bool mine = is_mine();
          const int32_t kt = x.t0 + i, j0 = kt * kTile - x.base0;  // the tile's first place among those of the rows
          if (p.rd.parents) {
            // the row's 128 bits from j0 on: ones before them, zeros behind them
            const uint4 v = *reinterpret_cast<const uint4*>(
                sm.above[b][min(x.tok0 + i_item, SV_MAX_TREE_ROWS - 1)]);
            const uint32_t above[4] = {v.x, v.y, v.z, v.w};
            const int32_t k0 = j0 >> 5;
            uint32_t word[5];
#pragma unroll
            for (int w = 0; w < 5; ++w) {
              const int32_t k = k0 + w;
              word[w] = k < 0 ? ~0u : 0u;
#pragma unroll
              for (int e = 0; e < 4; ++e) word[w] = k == e ? above[e] : word[w];
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) seen[w] = __funnelshift_r(word[w], word[w + 1], j0 & 31);
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {  // places up to the row's own
              const int32_t count = i_item + 1 - (j0 + 32 * w);
              seen[w] = count <= 0 ? 0u : count >= 32 ? ~0u : (1u << count) - 1;
            }
          }
          const int32_t load = loads + min(n, i + ahead) + i;
          wait(&sm.full[load % kStages], (load / kStages) & 1);
          const int32_t place = kt * kTile + row;
          if (place >= x.base0 && !failed) {
            uint8_t* const v = ring + (load % kStages) * Sh::kSlot;
            const bool found = twin ? make_finite<kD / 8>(v, row, 0, place >= x.end)
                                    : make_finite<kD / 16>(v, row, s * (kD / 16), place >= x.end);
            if (found) atomicOr(&sm.bad[b][s][(place - x.base0) >> 5], 1u << ((place - x.base0) & 31));
          }
          fence_proxy_async();
        }
        __syncwarp();
        tc::fence_after_sync();
        // the row's largest score
        float a[128];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) load32(s_at + 32 * ch, a + 32 * ch);
        wait_loads();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) landed(a + 32 * ch);
        if (masked) {
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) hide<32>(a + 32 * ch, seen[ch]);
        }
        float t[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = max3(t[e], a[c + 2 * e], a[c + 2 * e + 1]);
        }
        float top = max3(max3(t[0], t[1], a[124]), max3(t[2], t[3], a[125]), fmaxf(a[126], a[127]));
        top *= scale1;  // (an infinite score makes m infinite, and the row's weights NaN, as a NaN does itself)
        if (__any_sync(0xffffffffu, top > m + kSlack)) {
          const float now = fmaxf(m, top), factor = fast_exp2(m - now);
          m = now;
          l *= factor;
          if (!fresh) {
#pragma unroll 1
            for (int d = 0; d < kD; d += 8) {
              float o[8];
              tmem_load<8>(o_at + d, o);
#pragma unroll
              for (int c = 0; c < 8; ++c) o[c] *= factor;
              tmem_store<8>(o_at + d, o);
            }
          }
        }
        fresh = false;
        // P, rounded to bf16 for the product (half a step of 2^-8 a weight); its sum takes what it was
        // before that.  It goes over S, which is in registers by now.
        const float2 minus = splat2(-m);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float* const f = a + 32 * ch;
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 e = exp2_2(fma2(make_float2(f[c], f[c + 1]), scale, minus));
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], e);
            w[c / 2] = bf16_pair(e.x, e.y);
          }
          store16(s_at + 16 * ch, w);
          if (ch == 1) {
            wait_stores();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_half[s]);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        wait_stores();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[s]);
      }
      loads += 2 * n;
      // the item's results
      const bool had = !fresh;
      if (had) {
        wait(&sm.o_full[s], o_phase);
        o_phase ^= 1;
      }
      if (twin && s == 1) sm.m[row] = m, sm.l[row] = l;
      if (both_any(failed)) break;
      tc::fence_after_sync();
      const bool writes = !twin || s == 0, mine = is_mine();
      const int32_t i_item = token(), column = column_of();
      if (writes) {
        float mine_f = 1.f, other_f = 0.f;
        if (twin) {
          const float m1 = sm.m[row], now = fmaxf(m, m1);
          mine_f = fast_exp2(m - now);
          other_f = fast_exp2(m1 - now);
          l = l * mine_f + sm.l[row] * other_f;
          m = now;
        }
        const bool other = twin && n > 1;
        const int32_t head = x.head * p.group + row % p.group;
        const int64_t out_row = x.first_row + i_item;
        float* const part = reinterpret_cast<float*>(p.ws + wl.parts) +
                            (2 * int64_t(blockIdx.x) + x.begins) * wl.part_floats;
        if (mine) {
          if (!x.whole) {
            part[kWide * kD + column] = m;
            part[kWide * kD + kWide + column] = l;
          } else if (p.lse) {
            p.lse[out_row * p.ld_lse + head] = (log2f(l) + m) * kLn2;
          }
        }
        const float inv = 1.f / l;
        const int64_t out_at = mine ? out_row * p.ldo + head * p.o_head : -1;
        // the rows' values that were left out of the product for not being finite: elements d0 .. of what
        // is on its way out
        bool any_bad = false;
#pragma unroll
        for (int w = 0; w < kBadWords; ++w)
          any_bad |= (sm.bad[b][0][w] | sm.bad[b][1][w]) != 0;
        auto add_bad = [&](auto* to, int n, int d0) {
#pragma unroll 1
          for (int32_t j = 0; j < 32 * kBadWords; ++j) {
            if (!((sm.bad[b][0][j >> 5] | sm.bad[b][1][j >> 5]) >> (j & 31) & 1u)) continue;
            if (!mine || !(p.rd.parents ? sm.above[b][x.tok0 + i_item][j >> 5] >> (j & 31) & 1u
                                        : j <= i_item))
              continue;
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
              const float v = value_at(p, x, j, d0 + c);
              if (!isfinite(v)) to[c] = float(to[c]) + v;
            }
          }
        };
        // the warp's columns: from column0 on, the first rows_here of its lanes'
        const int32_t column0 = column - lane;
        const int32_t rows_here = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll 1
        for (int d = 0; d < kD; d += 32) {
          float o[32];
          __syncwarp();
          load32(o_at + d, o);
          wait_loads();
          landed(o);
          if (twin) {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] *= mine_f;
            if (other) {
              float o1[32];
              load32(o_at + 128 + d, o1);
              wait_loads();
              landed(o1);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] += o1[c] * other_f;
            }
          }
          // this lane's row into the stage, and 16 bytes of row 8 q + lane / 4 out of it
          uint8_t* const in = sm.stage[warp] + lane * kStageRow;
          const uint8_t* const from = sm.stage[warp] + (lane >> 2) * kStageRow + (lane & 3) * 16;
          if (x.whole) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 32; c += 8)
              *reinterpret_cast<uint4*>(in + 2 * c) =
                  make_uint4(bf16_pair(o[c] * inv, o[c + 1] * inv),
                             bf16_pair(o[c + 2] * inv, o[c + 3] * inv),
                             bf16_pair(o[c + 4] * inv, o[c + 5] * inv),
                             bf16_pair(o[c + 6] * inv, o[c + 7] * inv));
            if (any_bad) add_bad(reinterpret_cast<__nv_bfloat16*>(in), 32, d);
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int64_t to = __shfl_sync(0xffffffffu, out_at, 8 * q + (lane >> 2));
              if (to >= 0)
                *reinterpret_cast<uint4*>(p.out + to + d + (lane & 3) * 8) =
                    *reinterpret_cast<const uint4*>(from + q * 8 * kStageRow);
            }
          } else {
#pragma unroll
            for (int part_of = 0; part_of < 2; ++part_of) {  // 16 elements at a time
              __syncwarp();
#pragma unroll
              for (int c = 0; c < 16; c += 4)
                *reinterpret_cast<float4*>(in + 4 * c) =
                    make_float4(o[16 * part_of + c], o[16 * part_of + c + 1], o[16 * part_of + c + 2],
                                o[16 * part_of + c + 3]);
              if (any_bad) add_bad(reinterpret_cast<float*>(in), 16, d + 16 * part_of);
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int32_t col = column0 + 8 * q + (lane >> 2);
                if (8 * q + (lane >> 2) < rows_here)
                  *reinterpret_cast<float4*>(part + col * kD + d + 16 * part_of + (lane & 3) * 4) =
                      *reinterpret_cast<const float4*>(from + q * 8 * kStageRow);
              }
            }
          }
        }
      }
      tc::fence_before_sync();
      if (twin) both_any(false);  // stream 1's sums are not overwritten before they are read
      else soft_sync(s);
      if (row == 0) mbar_arrive(&sm.item_empty[b]);
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0) reinterpret_cast<int32_t*>(p.ws)[blockIdx.x] = sm.err * 512 + sm.cut_columns;
}

template <int kD, int kLoaders>
sv_status launch(const AttnMaps& m, const AttnParams& p, int grid, cudaStream_t s) {
  auto* kern = wide_kernel<kD, kLoaders>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kAttnSmem)) !=
      cudaSuccess)
    return SV_ERR_CUDA;
  return launch_dependent(kern, unsigned(grid), kAttnThreads, kAttnSmem, s, m.q, m.k, m.v, p);
}

}  // namespace

// Two loading warps for pages of at most 16 places, where one's issue is the bound; where it is not, the other
// costs the products 2% (8 x 64 rows, 16000 to 32768 places, one warp and two: 355 and 306 us in pages of
// 16, 298 and 319 of 32; 8 prompts of 2048 rows: 345 and 308, 301 and 309).
sv_status launch_wide(int32_t D, const AttnMaps& m, const AttnParams& p, int grid, cudaStream_t s) {
  if (p.box_rows <= 16) return D == 64 ? launch<64, 2>(m, p, grid, s) : launch<128, 2>(m, p, grid, s);
  return D == 64 ? launch<64, 1>(m, p, grid, s) : launch<128, 1>(m, p, grid, s);
}

}  // namespace attn
}  // namespace sv
