// tree_attention.cu -- attention of a round's rows over the paged cache (spec_tree_attention).
//
// The rows of a request are few and its keys many, so a tile puts the keys where a matrix instruction
// is wide and the rows where it is narrow: with K a tile of 128 places, Q the rows of all query heads of
// one key head (kN columns: token i, head g in column i G + g) and V the tile's values,
//   S^T = K Q^T   (128 x kN, TMEM lane = place, column = row),
//   P^T = 2^(scale log2(e) S^T - m)   in bf16 to shared memory,
//   O^T += V^T P^T   (D x kN, lane = element of the head).
// K and V go in as they lie in the cache (K with its elements, V with its places along the contraction);
// a row costs a 16th of the narrowest instruction, where it would be padded to 128 the other way round.
//   warps 0-7  softmax: a place a thread, half of the columns for warps 0-3, the others for 4-7.  m is
//              a bound of a column's maximum that is raised only when a score passes it by more than 8
//              (P then reaches 2^8, in 16 bits as exact as 1), so that nearly every tile costs no
//              reduction over the places; the sums of P stay with the places and are added over them at
//              the end;
//   warps 8, 11  TMA loads: an item's queries, then K and V, page by page, into a ring;
//   warp 9     tcgen05.mma: S of a tile ahead of the product with V of the one before;
//   warp 10    the work items: their sizes, and for trees who sees whom.
// The work -- (request, key head, row tile, key tile) -- is one list, cut into equal runs for a
// persistent CTA on every SM, wherever the cuts fall; what a cut leaves in parts goes to the workspace
// and is joined by a second kernel.  Where there are few items of few tiles, a cluster takes each, and its
// CTAs, a run of the tiles each, join their parts through one another's shared memory: one launch.
#include "tree_attention.cuh"

#include "tmap.h"

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

namespace sv {
namespace {

using namespace attn;

// Items whose descriptions are there at once: of short ones several lie in the ring, and the loads wait for the
// results of none (256 rows over 100 to 400 places each: 80 us with two, 66 with four).
constexpr int kItemsLog = 2, kItems = 1 << kItemsLog;

template <int kD, int kN>
struct AttnShared {
  static constexpr uint32_t kSlot = kTile * kD * 2;
  static constexpr uint32_t kQBytes = kN * kD * 2;
  static constexpr uint32_t kPBytes = (kN + 63) / 64 * 16384;
  static constexpr int kWords = (kN + 31) / 32;
  struct Small {
    uint64_t full[16], empty[16], item_full[kItems], item_empty[kItems], table_full[kItems];
    uint64_t q_full[2], q_empty[2], s_full[2];
    uint64_t p_full, p_free, drain;
    int64_t col_off[kItems][kN];  // of a column's output
    Item item[kItems];
    alignas(16) float minus[kN];  // -m; read four at a time, as the next two
    alignas(16) float factor[kN];
    alignas(16) float inv[kN];
    float part[4][kN];
    uint32_t seen[kItems][SV_MAX_TREE_ROWS][kWords];  // bit c: column c sees the tree's row
    uint32_t above[SV_MAX_TREE_ROWS][4];         // rows above a row, itself included
    int32_t up[SV_MAX_TREE_ROWS];
    uint32_t bad[kItems][2][SV_MAX_TREE_ROWS / 32];  // an item's rows whose values (of a half of D) are
                                                     // not all finite
    uint32_t tmem;
    int32_t err, cut_columns;
    uint32_t had;  // this CTA of a cluster has a part
  };
  static constexpr uint32_t kSmall = (sizeof(Small) + 127) / 128 * 128;
  static constexpr int kStages() {
    const int s = int((kAttnSmem - 1024 - kSmall - 2 * kQBytes - kPBytes) / kSlot);
    return s < 16 ? s : 16;
  }
};

// Who sees whom in a tree, by one warp: seen[j] = columns that see row j.
template <int kWords>
__device__ __forceinline__ void build_seen(const AttnParams& p, const Item& x, uint32_t (*above)[4],
                                           uint32_t (*seen)[kWords]) {
  const int lane = threadIdx.x & 31;
  const int32_t nodes = x.end - x.ctx, columns = x.columns;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int32_t c = w * 32 + lane, i = c / p.group;
    const bool in = c < columns;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k * 32 >= nodes) break;
      const uint32_t mine = in ? above[i][k] : 0u;
      uint32_t row = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const uint32_t word = __ballot_sync(0xffffffffu, mine >> j & 1u);
        if (lane == j) row = word;
      }
      seen[k * 32 + lane][w] = row;
    }
  }
}

// The item of this CTA's cluster of kCtas, a key head of a request, and the CTA's tiles of it.
template <int kCtas>
__device__ __forceinline__ Item cluster_item(const AttnParams& p, int64_t& first) {
  const int32_t cluster = blockIdx.x / kCtas, rank = blockIdx.x % kCtas, r = cluster / p.n_kv;
  Request q;
  Item x = {};
  if (round_request(p.rd, r, q) && q.n > 0) {
    first = q.first;
    x.head = cluster - r * p.n_kv, x.r = r;
    x.first_row = q.first;
    x.columns = q.n * p.group;
    x.ctx = x.base0 = q.ctx;
    x.end = q.ctx + q.n;
    const int64_t all = tiles_of(q, 0, p.tokens);
    x.t0 = int32_t(all * rank / kCtas), x.t1 = int32_t(all * (rank + 1) / kCtas);
  }
  x.begins = x.last = 1;
  x.stop = x.t0 == x.t1;
  return x;
}

// All there is to check of a call of at most 32 requests, by one warp: whether it is bad.  A lane looks at
// a request's sizes, then all of them at everybody's pages and parents.
__device__ __forceinline__ bool bad_round(const RoundParams& rd) {
  const int lane = threadIdx.x & 31;
  Request q = {};
  bool bad = lane < rd.B && !round_request(rd, lane, q);
  const int32_t pages =
      q.n ? int32_t((int64_t(q.ctx) + q.n + rd.page_size - 1) / rd.page_size) : 0;
#pragma unroll 8
  for (int32_t i0 = 0; i0 < rd.B * rd.max_pages; i0 += 32) {
    const int32_t r = (i0 + lane) / rd.max_pages, i = i0 + lane - r * rd.max_pages;
    const int32_t n = __shfl_sync(0xffffffffu, pages, r & 31);
    if (r < rd.B && i < n) {
      const int32_t g = rd.page_table[r * rd.ld_pages + i];
      bad |= g < 0 || g >= rd.n_pages;
    }
  }
  if (rd.parents) {
    const int32_t rows = rd.max_draft_len + rd.bonus_row;
#pragma unroll 4
    for (int32_t i0 = 0; i0 < rd.B * rows; i0 += 32) {
      const int32_t r = (i0 + lane) / rows, i = i0 + lane - r * rows;
      const int32_t n = __shfl_sync(0xffffffffu, q.n, r & 31);
      const int64_t first = __shfl_sync(0xffffffffu, q.first, r & 31);
      if (r < rd.B && i < n) {
        const int32_t up = rd.parents[first + i];
        bad |= up < -1 || up >= i;
      }
    }
  }
  return __any_sync(0xffffffffu, bad);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t at, int rank) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
  return to;
}
__device__ __forceinline__ float peer_load(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// The parts of a cluster's item joined by all of its threads: CTA `rank` takes
// every kCtas-th column.
template <int kD, int kN, int kCtas>
__device__ __forceinline__ void cluster_join(const AttnParams& p, const Item& x, const float* part,
                                             const uint32_t* had, const int64_t* col_off) {
  const uint32_t at = smem_addr(part), had_at = smem_addr(had);
  for (int32_t u = threadIdx.x;; u += kAttnThreads) {
    const int32_t col = blockIdx.x % kCtas + kCtas * (u / (kD / 2)), d = u % (kD / 2) * 2;
    if (col >= x.columns) return;
    float m[kCtas], l[kCtas], a[kCtas], b[kCtas];
    bool has[kCtas];
#pragma unroll
    for (int r = 0; r < kCtas; ++r) {
      const uint32_t from = peer(at, r);
      has[r] = __float_as_uint(peer_load(peer(had_at, r))) != 0;
      m[r] = peer_load(from + 4 * (kN * kD + col));
      l[r] = peer_load(from + 4 * (kN * kD + kN + col));
      a[r] = peer_load(from + 4 * (col * kD + d));
      b[r] = peer_load(from + 4 * (col * kD + d + 1));
    }
    float top = kM2Empty, sum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int r = 0; r < kCtas; ++r)
      if (has[r]) top = fmaxf(top, m[r]);
#pragma unroll
    for (int r = 0; r < kCtas; ++r) {
      if (!has[r]) continue;
      const float w = fast_exp2(m[r] - top);
      sum += w * l[r];
      y0 += w * a[r];
      y1 += w * b[r];
    }
    const float inv = 1.f / sum;
    *reinterpret_cast<__nv_bfloat162*>(p.out + col_off[col] + d) =
        __floats2bfloat162_rn(y0 * inv, y1 * inv);
    if (d == 0 && p.lse) {
      const int32_t i = col / p.group;
      p.lse[(x.first_row + i) * p.ld_lse + x.head * p.group + col - i * p.group] =
          (top + log2f(sum)) * kLn2;
    }
  }
}

template <int kD, int kN, int kCtas>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  using Sh = AttnShared<kD, kN>;
  constexpr bool kShort = kCtas > 0;
  constexpr int kC = kN / 2;  // columns of a half
  constexpr int kStages = Sh::kStages();
  constexpr uint32_t kCols = kN <= 16 ? 64 : kN <= 32 ? 128 : 256;
  static_assert(kStages >= 3, "a ring of three tiles");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const q_at = ring + kStages * Sh::kSlot;
  uint8_t* const p_at = q_at + 2 * Sh::kQBytes;
  typename Sh::Small& sm = *reinterpret_cast<typename Sh::Small*>(p_at + Sh::kPBytes);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 2);  // either loading warp's part
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < kItems; ++b) {
      mbar_init(&sm.item_full[b], 1);
      mbar_init(&sm.item_empty[b], 5);  // the loads, the products with Q, the softmax's halves
      mbar_init(&sm.table_full[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.q_full[b], 1);
      mbar_init(&sm.q_empty[b], 1);
      mbar_init(&sm.s_full[b], 1);
    }
    mbar_init(&sm.p_full, kSoftWarps);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.drain, 1);
    fence_barrier_init();
    sm.err = 0;
    sm.had = 0;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&sm.tmem, kCols);
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
  const uint32_t tmem = sm.tmem;
  int32_t* const err = &sm.err;
  const WsLayout wl = ws_layout(gridDim.x, kN, kD);
  if (warp == kItemWarp) {
    // ---- the items ---------------------------------------------------------------------------------
    int32_t built[kItems];  // the request whose tree a slot has
#pragma unroll
    for (int b = 0; b < kItems; ++b) built[b] = -1;
    auto details = [&](int b, const Item& x, int64_t first) {
      for (int32_t c = lane; c < x.columns; c += 32) {
        const int32_t i = c / p.group, g = c - i * p.group;
        sm.col_off[b][c] = (x.first_row + i) * p.ldo + int64_t(x.head * p.group + g) * p.o_head;
      }
      if (p.rd.parents && x.t1 * int64_t(kTile) > x.base0 && built[b] != x.r) {
        built[b] = x.r;
        build_above(p, first, x.end - x.ctx, sm.up, sm.above, err);
        build_seen<Sh::kWords>(p, x, sm.above, sm.seen[b]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.table_full[b]);
    };
    if constexpr (kShort) {
      int64_t first = 0;
      const Item x = cluster_item<kCtas>(p, first);
      if (lane == 0) {
        sm.item[0] = x;
        mbar_arrive(&sm.item_full[0]);
        sm.item[1].stop = 1;  // there is no other
        mbar_arrive(&sm.item_full[1]);
      }
      __syncwarp();
      details(0, x, first);
    } else {
      const int32_t columns = walk_items<kItemsLog>(p, reinterpret_cast<Cut*>(p.ws + wl.cuts), sm.item,
                                                 sm.item_full, sm.item_empty, err, details);
      if (lane == 0) sm.cut_columns = columns;
    }
  } else if (warp == kLoadWarp || warp == kLoadWarp2) {
    // ---- the loads -----------------------------------------------------------------------------------
    const uint64_t once = tc::policy_evict_first();
    const int part = warp == kLoadWarp2;
    int32_t slot = 0, filled = 0, items = 0;
    uint32_t phase = 1;
    // a tile's boxes, one a lane: its page and first place in it
    int32_t v_page = 0, v_from = 0, v_boxes = 0, v_head = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap* map, int32_t pg, int32_t fr, int32_t n, int32_t hd) {
      if (!wait_for_warp(&sm.empty[slot], phase, err)) return false;
      load_tile<kD, 2, false>(p, ring + slot * Sh::kSlot, map, part, pg, fr, n, hd, &sm.full[slot], once);
      filled = max(filled, slot + 1);
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
      return true;
    };
    for (int32_t it = 0; ok; ++it) {
      const int b = it & (kItems - 1), qb = it & 1;
      if (!wait_for_warp(&sm.item_full[b], (it >> kItemsLog) & 1, err)) break;
      const Item x = sm.item[b];
      if (x.stop) break;
      if (part == 0 && it >= 2 && !wait_for_warp(&sm.q_empty[qb], ((it >> 1) - 1) & 1, err)) break;
      if (part == 0 && elect()) {
        // (rows behind the request's last, and columns behind those, hold anything: nobody reads them)
        mbar_expect_tx(&sm.q_full[qb], uint32_t(p.tile_tokens * p.group) * kD * 2);
#pragma unroll
        for (int k = 0; k < kD / 64; ++k)
          tc::tma_load_3d(q_at + qb * Sh::kQBytes + k * kN * 128, &map_q, k * 64, x.head * p.group,
                          int32_t(x.first_row), &sm.q_full[qb]);
      }
      __syncwarp();
      if (part == 0) items = it + 1;
      for (int32_t t = x.t0; t < x.t1 && ok; ++t) {
        int32_t page, from;
        const int32_t boxes = tile_boxes<kD, 2>(p, x, t, part, page, from, err);
        ok = load(&map_k, page, from, boxes, x.head) &&
             (v_boxes == 0 || load(&map_v, v_page, v_from, v_boxes, v_head));
        v_page = page, v_from = from, v_boxes = boxes, v_head = x.head;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[b]);
    }
    if (ok && v_boxes) load(&map_v, v_page, v_from, v_boxes, v_head);
    // every copy in flight lands before the CTA may end
    for (int32_t k = 0; k < filled; ++k)
      wait_for_warp(&sm.full[k], k < slot ? phase ^ 1 : phase, err);
    for (int32_t k = max(0, items - 2); k < items; ++k)
      wait_for_warp(&sm.q_full[k & 1], (k >> 1) & 1, err);
  } else if (warp == kMmaWarp) {
    // ---- the products --------------------------------------------------------------------------------
    constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, kN);
    constexpr uint32_t kIdO = tc::idesc_bf16_f32(128, kN) | (1u << 15) | (1u << 16);
    const uint32_t ring_lo = desc_at(ring), q_lo = desc_at(q_at);
    const uint32_t p_lo = desc_at(p_at) | kAcross;
    int32_t slot = 0, t = 0;
    uint32_t phase = 0;
    bool ok = true, fresh = false, v_fresh = false;
    auto next_slot = [&] {
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
    };
    // O of the tile before: (+)= V^T P^T
    auto values = [&] {
      if (!wait_for_warp(&sm.p_full, (t - 1) & 1, err) || !wait_for_warp(&sm.full[slot], phase, err))
        return false;
      tc::fence_after_sync();
      if (elect()) {
        const uint32_t v_lo = ring_lo + slot * (Sh::kSlot >> 4) + kAcross;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tc::mma_bf16(tmem + 2 * kN, desc_of(v_lo + k * 128), desc_of(p_lo + k * 128), kIdO,
                       !v_fresh || k > 0);
        tc::mma_commit(&sm.p_free);
        tc::mma_commit(&sm.empty[slot]);
      }
      __syncwarp();
      next_slot();
      return true;
    };
    for (int32_t it = 0; ok; ++it) {
      const int b = it & (kItems - 1), qb = it & 1;
      if (!wait_for_warp(&sm.item_full[b], (it >> kItemsLog) & 1, err)) break;
      if (sm.item[b].stop) break;
      const int32_t n = sm.item[b].t1 - sm.item[b].t0;
      if (!wait_for_warp(&sm.q_full[qb], (it >> 1) & 1, err)) break;
      for (int32_t k = 0; k < n && ok; ++k, ++t) {
        if (!wait_for_warp(&sm.full[slot], phase, err)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (elect()) {
          const uint32_t k_lo = (ring_lo + slot * (Sh::kSlot >> 4)) | kAlongK;
          const uint32_t b_lo = (q_lo + qb * (Sh::kQBytes >> 4)) | kAlongK;
#pragma unroll
          for (int s = 0; s < kD / 16; ++s)
            tc::mma_bf16(tmem + (t & 1) * kN, desc_of(k_lo + (s >> 2) * 1024 + (s & 3) * 2),
                         desc_of(b_lo + (s >> 2) * (kN * 8) + (s & 3) * 2), kIdS, s > 0);
          tc::mma_commit(&sm.s_full[t & 1]);
          tc::mma_commit(&sm.empty[slot]);
          if (k + 1 == n) {
            tc::mma_commit(&sm.q_empty[qb]);
            tc::mma_commit(&sm.item_empty[b]);
          }
        }
        __syncwarp();
        next_slot();
        v_fresh = fresh;
        fresh = k == 0;
        if (t > 0) ok = values();
      }
    }
    if (ok && t > 0) {
      v_fresh = fresh;
      ok = values();
    }
    // nothing reads shared or tensor memory once this has passed
    if (elect()) tc::mma_commit(&sm.drain);
    __syncwarp();
    wait_for_warp(&sm.drain, 0, err);
  } else if (warp < kSoftWarps) {
    // ---- softmax and results -------------------------------------------------------------------------
    const int half = warp >> 2, quad = warp & 3;
    const int row = tid & 127;       // place of a key tile; element of the head
    const int col0 = half * kC;      // this half's first column
    const uint32_t lanes = tmem + (uint32_t(32 * quad) << 16) + col0;
    float* const minus = sm.minus + col0;
    float* const factor = sm.factor + col0;
    float* const inv = sm.inv + col0;
    float l[kC];
    int32_t t = 0;
    bool ok = true;
    for (int32_t it = 0; ok; ++it) {
      const int b = it & (kItems - 1);
      if (soft_any(half, !wait_for(&sm.item_full[b], (it >> kItemsLog) & 1, err))) break;
      const Item x = sm.item[b];
      if (x.stop) break;
      if (row < kC) minus[row] = -kM2Empty;
      if (row < SV_MAX_TREE_ROWS / 32) sm.bad[b][half][row] = 0;
#pragma unroll
      for (int c = 0; c < kC; ++c) l[c] = 0.f;
      bool table = false;
      soft_sync(half);
      for (int32_t kt = x.t0; kt < x.t1; ++kt, ++t) {
        const uint32_t s_at = lanes + (t & 1) * kN;
        bool free = t == 0;  // P's buffer
        // (a wait that ran out leaves the loop in all four warps together)
        bool late = !wait_for(&sm.s_full[t & 1], (t >> 1) & 1, err);
        const bool masked = (kt + 1) * int64_t(kTile) > x.base0;
        uint32_t seen = ~0u;  // bit c: column c of this half sees this thread's place
        if (masked) {
          if (!table) late |= !wait_for(&sm.table_full[b], (it >> kItemsLog) & 1, err);
          table = true;
          const int32_t place = kt * kTile + row, j = place - x.base0;
          if (place >= x.end) {
            seen = 0u;
          } else if (j >= 0 && p.rd.parents) {
            seen = sm.seen[b][j][col0 >> 5] >> (col0 & 31);
          } else if (j >= 0) {  // columns of token j and later ones
            const int32_t from = j * p.group - col0;
            seen = from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
          }
          // each half looks through half of the elements
          const int32_t load = kt + 1 == x.t1 && x.last ? 2 * t + 1 : 2 * t + 2;
          late |= !wait_for(&sm.full[load % kStages], (load / kStages) & 1, err);
          if (place >= x.base0 && !late &&
              make_finite<kD / 16>(ring + (load % kStages) * Sh::kSlot, row, half * (kD / 16),
                                   place >= x.end))
            atomicOr(&sm.bad[b][half][j >> 5], 1u << (j & 31));
        }
        tc::fence_after_sync();
        // does any score pass its column's m by more than the slack?
        float s[kC], m[kC], top = kt == x.t0 ? INFINITY : -INFINITY;  // (the first tile's surely do)
        if (kt > x.t0) {
          broadcast<kC>(minus, m);
          tmem_load<kC>(s_at, s);
          scaled<kC>(s, p.scale2, m);
          if (masked) hide<kC>(s, seen);
#pragma unroll
          for (int c = 0; c < kC; c += 2) top = max3(top, s[c], s[c + 1]);
        }
        const bool raise = soft_any(half, late || top > kSlack);
        if (raise) {
          if (soft_any(half, late)) {
            ok = false;
            break;
          }
          tmem_load<kC>(s_at, s);
#pragma unroll
          for (int c = 0; c < kC; ++c) s[c] *= p.scale2;
          if (masked) hide<kC>(s, seen);
          const float most = over_lanes<kC>(s, [](float a, float b) { return fmaxf(a, b); });
          if (lane < kC) sm.part[quad][col0 + lane] = most;
          soft_sync(half);
          if (row < kC) {
            const int c = col0 + row;
            const float old = -minus[row];
            const float most = fmaxf(fmaxf(sm.part[0][c], sm.part[1][c]),
                                     fmaxf(sm.part[2][c], sm.part[3][c]));
            const float now = fmaxf(old, most);
            minus[row] = -now;
            factor[row] = fast_exp2(old - now);
          }
          soft_sync(half);
          if (kt > x.t0) {  // there are sums
            if (soft_any(half, !wait_for(&sm.p_free, (t - 1) & 1, err))) {
              ok = false;
              break;
            }
            free = true;
            tc::fence_after_sync();
            broadcast<kC>(factor, m);
#pragma unroll
            for (int c = 0; c < kC; ++c) l[c] *= m[c];
            tmem_load<kC>(lanes + 2 * kN, s);
#pragma unroll
            for (int c = 0; c < kC; ++c) s[c] *= m[c];
            tmem_store<kC>(lanes + 2 * kN, s);
          }
        }
        if (!free && soft_any(half, !wait_for(&sm.p_free, (t - 1) & 1, err))) {
          ok = false;
          break;
        }
        // P, rounded to bf16 for the product (half a step of 2^-8 a weight); its sums take what it was
        // before that
        if (raise) {
          broadcast<kC>(minus, m);
          tmem_load<kC>(s_at, s);
          scaled<kC>(s, p.scale2, m);
          if (masked) hide<kC>(s, seen);
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) s[c] = fast_exp2(s[c]);
#pragma unroll
        for (int c = 0; c < kC; c += 2) {
          const float2 sum = add2(make_float2(l[c], l[c + 1]), make_float2(s[c], s[c + 1]));
          l[c] = sum.x, l[c + 1] = sum.y;
        }
#pragma unroll
        for (int c = 0; c < kC; c += 8) {
          uint4 w;
          uint32_t* const wp = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(s[c + 2 * e], s[c + 2 * e + 1]);
            wp[e] = *reinterpret_cast<const uint32_t*>(&two);
          }
          const int col = col0 + c;
          *reinterpret_cast<uint4*>(p_at + (col >> 6) * 16384 + tc::sw128(row, (col & 63) >> 3)) = w;
        }
        fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
      }
      if (!ok) break;
      // the item's denominators (while the last product is on its way), then its sums
      bool late = !table && !wait_for(&sm.table_full[b], (it >> kItemsLog) & 1, err);
      const float sum = over_lanes<kC>(l, [](float a, float b) { return a + b; });
      if (lane < kC) sm.part[quad][col0 + lane] = sum;
      late |= !wait_for(&sm.p_free, (t - 1) & 1, err);
      if (soft_any(half, late)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      // (a cluster's CTA has a single item, and its ring is free)
      float* const part = kShort ? reinterpret_cast<float*>(ring)
                                 : reinterpret_cast<float*>(p.ws + wl.parts) +
                                       (2 * int64_t(blockIdx.x) + x.begins) * wl.part_floats;
      if (kShort && tid == 0) sm.had = 1;
      if (row < kC && col0 + row < x.columns) {
        const int c = col0 + row;
        const float sum = (sm.part[0][c] + sm.part[1][c]) + (sm.part[2][c] + sm.part[3][c]);
        if (x.whole) {
          inv[row] = 1.f / sum;
          if (p.lse) {
            const int32_t i = c / p.group;
            p.lse[(x.first_row + i) * p.ld_lse + x.head * p.group + c - i * p.group] =
                (log2f(sum) - minus[row]) * kLn2;
          }
        } else {
          part[kN * kD + c] = -minus[row];
          part[kN * kD + kN + c] = sum;
        }
      }
      soft_sync(half);
      bool any_bad = false;
#pragma unroll
      for (int w = 0; w < SV_MAX_TREE_ROWS / 32; ++w)
        any_bad |= (sm.bad[b][0][w] | sm.bad[b][1][w]) != 0;
      if (32 * quad < kD && col0 < x.columns) {
        float s[kC], f[kC];
        tmem_load<kC>(lanes + 2 * kN, s);
        if (any_bad) {  // values that were left out of the product for not being finite
#pragma unroll 1
          for (int32_t j = 0; j < SV_MAX_TREE_ROWS; ++j) {
            if (!((sm.bad[b][0][j >> 5] | sm.bad[b][1][j >> 5]) >> (j & 31) & 1u)) continue;
            const float v = value_at(p, x, j, row);
            if (isfinite(v)) continue;
            const uint32_t sees = p.rd.parents ? sm.seen[b][j][col0 >> 5] >> (col0 & 31)
                                  : j * p.group <= col0 ? ~0u
                                  : j * p.group >= col0 + 32 ? 0u
                                                           : ~0u << (j * p.group - col0);
#pragma unroll
            for (int c = 0; c < kC; ++c)
              if (sees >> c & 1u) s[c] += v;
          }
        }
        if (x.whole) {
          // two columns at once: an even lane takes elements (d, d + 1) of one, an odd lane (d - 1,
          // d) of the next
          const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;
          broadcast<kC>(inv, f);
          __nv_bfloat16* to[kC / 2];
#pragma unroll
          for (int c = 0; c < kC; c += 2)
            to[c / 2] = p.out + sm.col_off[b][col0 + c + (lane & 1)] + (row & ~1);
#pragma unroll
          for (int c = 0; c < kC; c += 2) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(s[c] * f[c], s[c + 1] * f[c + 1]);
            const uint32_t mine = *reinterpret_cast<const uint32_t*>(&two);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
            if (col0 + c + (lane & 1) < x.columns)
              *reinterpret_cast<uint32_t*>(to[c / 2]) = __byte_perm(mine, other, pick);
          }
        } else {
          float* const to = part + col0 * kD + row;
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (col0 + c < x.columns) to[c * kD] = s[c];
        }
      }
      tc::fence_before_sync();
      soft_sync(half);
      if (row == 0) mbar_arrive(&sm.item_empty[b]);
    }
  }
  if constexpr (kShort) {
    // CTA 0 looks at all there is to check, and the status is its own; what ran out of time says so later
    if (warp == kItemWarp && blockIdx.x == 0 && p.status) {
      const bool bad = bad_round(p.rd);
      if (lane == 0) *p.status = bad ? SV_ERR_BAD_INPUT : SV_OK;
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kCols);
  }
  if constexpr (kShort) {
    if (tid == 0 && sm.err == SV_ERR_TIMEOUT) report(p.status, SV_ERR_TIMEOUT);
    __syncwarp();
    cluster_sync();
    cluster_join<kD, kN, kCtas>(p, sm.item[0], reinterpret_cast<const float*>(ring), &sm.had, sm.col_off[0]);
    __syncwarp();
    cluster_sync();  // nobody's shared memory goes away while others read it
  } else {
    if (tid == 0) reinterpret_cast<int32_t*>(p.ws)[blockIdx.x] = sm.err * 512 + sm.cut_columns;
  }
}

constexpr int kJoinThreads = 256;
// Columns of a warp: one where there are few columns, and many parts of each.
constexpr int join_columns_of(int n) { return n <= 64 ? 1 : 4; }

// Columns from col0 on of the item that CTA `cta` begins, by one warp.
template <int kD, int kN>
__device__ __forceinline__ void join_columns(const AttnParams& p, const WsLayout& wl, const Cut& cut,
                                             int32_t columns, int32_t ctas, int32_t cta, int32_t col0) {
  constexpr int kE = kD / 32;
  constexpr int kC = join_columns_of(kN), kParts = 32 / kC;
  const int lane = threadIdx.x & 31;
  const float* const parts = reinterpret_cast<const float*>(p.ws + wl.parts);
  // CTA k's part
  auto part_of = [&](int32_t k) { return parts + (2 * int64_t(k) + (k == cta)) * wl.part_floats; };
  // CTA k has none where its run is empty
  auto has = [&](int32_t k) {
    return k <= cut.last &&
           (k == cta || cut.total >= ctas || cut.total * k / ctas != cut.total * (k + 1) / ctas);
  };
  // kParts parts at a time: lane l looks at part l / kC of them and column l % kC
  const int32_t my_col = min(col0 + lane % kC, columns - 1);
  float top = kM2Empty, sum = 0.f;  // of this lane's column
  float y[kC][kE] = {};
  for (int32_t k0 = cta; k0 <= cut.last; k0 += kParts) {
    const int32_t k = k0 + lane / kC;
    const bool mine = has(k);
    const float* const x = part_of(mine ? k : cta) + kN * kD + my_col;
    const float m = mine ? x[0] : kM2Empty, d = mine ? x[kN] : 0.f;
    float most = m;
#pragma unroll
    for (int o = kC; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    most = fmaxf(most, top);
    const float old = fast_exp2(top - most), w = mine ? fast_exp2(m - most) : 0.f;
    float all = d * w;
#pragma unroll
    for (int o = kC; o < 32; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    sum = sum * old + all;
    top = most;
    if (k0 > cta) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const float f = __shfl_sync(0xffffffffu, old, c);
#pragma unroll
        for (int e = 0; e < kE; ++e) y[c][e] *= f;
      }
    }
    const uint32_t there = __ballot_sync(0xffffffffu, mine);
    const int32_t n = min(kParts, cut.last - k0 + 1);
    for (int32_t i0 = 0; i0 < n; i0 += 8 / kC) {
      float v[8][kE];  // in flight together
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int32_t i = i0 + q / kC;
        const bool is = i < n && (there >> (kC * i) & 1u);
        // (columns behind the last are there too, and are not written)
        const float* const o = part_of(is ? k0 + i : cta) + (col0 + q % kC) * kD + lane * kE;
        if constexpr (kE == 4) {
          const float4 z = *reinterpret_cast<const float4*>(o);
          v[q][0] = z.x, v[q][1] = z.y, v[q][2] = z.z, v[q][3] = z.w;
        } else {
          const float2 z = *reinterpret_cast<const float2*>(o);
          v[q][0] = z.x, v[q][1] = z.y;
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int32_t i = i0 + q / kC;
        const bool is = i < n && (there >> (kC * i) & 1u);
        const float f = __shfl_sync(0xffffffffu, w, (kC * i + q % kC) & 31);
#pragma unroll
        for (int e = 0; e < kE; ++e) y[q % kC][e] += is ? f * v[q][e] : 0.f;
      }
    }
  }
  const float my_inv = 1.f / sum, my_lse = (top + log2f(sum)) * kLn2;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const float inv = __shfl_sync(0xffffffffu, my_inv, c);
    if (col0 + c >= columns) break;
    const int32_t i = (col0 + c) / p.group, h = cut.head * p.group + col0 + c - i * p.group;
    const int64_t row = cut.first_row + i;
    __nv_bfloat16* const o = p.out + row * p.ldo + h * p.o_head + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(o + e) = __floats2bfloat162_rn(y[c][e] * inv, y[c][e + 1] * inv);
    if (lane == c && p.lse) p.lse[row * p.ld_lse + h] = my_lse;
  }
}

// A warp for every kC columns that there can be; the first ones, spread over the SMs, take those of
// the cut items.  Block 0 also gathers the CTAs' errors.
template <int kD, int kN>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnParams p, int32_t ctas) {
  constexpr int kRounds = (kMaxCtas + 31) / 32, kC = join_columns_of(kN);
  dependent_start();
  const WsLayout wl = ws_layout(ctas, kN, kD);
  const int lane = threadIdx.x & 31;
  int32_t word[kRounds], all = 0, code = 0;  // of CTA 32 k + lane
#pragma unroll
  for (int k = 0; k < kRounds; ++k)
    word[k] = k * 32 + lane < ctas ? reinterpret_cast<const int32_t*>(p.ws)[k * 32 + lane] : 0;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    code = max(code, word[k] >> 9);
    word[k] &= 511;
    all += (word[k] + kC - 1) / kC;
  }
  if (blockIdx.x == 0 && threadIdx.x < 32 && p.status) {
    code = __reduce_max_sync(0xffffffffu, code);
    if (lane == 0) *p.status = code;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  int32_t cta = -1, group = blockIdx.x + gridDim.x * (threadIdx.x >> 5), columns = 0;
  if (group >= all) return;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    if (cta < 0) {
      const int32_t mine = (word[k] + kC - 1) / kC;
      int32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, group < upto);
      if (past) {
        const int l = __ffs(past) - 1;
        group -= __shfl_sync(0xffffffffu, upto - mine, l);
        columns = __shfl_sync(0xffffffffu, word[k], l);
        cta = k * 32 + l;
      } else {
        group -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  join_columns<kD, kN>(p, wl, reinterpret_cast<const Cut*>(p.ws + wl.cuts)[cta], columns, ctas, cta,
                       group * kC);
}

// ---- host ----------------------------------------------------------------------------------------------

// Columns of a row tile: the narrowest that takes all of a request's rows.
int32_t columns_for(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : kWide; }

// [D][heads][places][pages] of a cache, boxes of 64 elements of one head of `box_rows` places.
bool cache_map(CUtensorMap* map, const void* base, int32_t D, int32_t heads, int32_t page_size,
               int64_t pages, int64_t head_stride, int64_t token_stride, int64_t page_stride,
               int32_t box_rows) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(page_size),
                              cuuint64_t(pages)};
  // (the stride of an axis of one says nothing)
  const cuuint64_t st[3] = {heads > 1 ? cuuint64_t(head_stride) * 2 : 16,
                            page_size > 1 ? cuuint64_t(token_stride) * 2 : 16,
                            pages > 1 ? cuuint64_t(page_stride) * 2 : 16};
  const cuuint32_t box[4] = {64, 1, cuuint32_t(box_rows), 1}, es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, st, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [D][heads][rows] of the queries, boxes of 64 elements of `tokens` rows of a key head's query heads.
bool query_map(CUtensorMap* map, const void* q, int32_t D, int32_t heads, int64_t rows, int64_t q_head,
               int64_t ldq, int32_t group, int32_t tokens) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(rows)};
  const cuuint64_t st[2] = {heads > 1 ? cuuint64_t(q_head) * 2 : 16,
                            rows > 1 ? cuuint64_t(ldq) * 2 : 16};
  const cuuint32_t box[3] = {64, cuuint32_t(group), cuuint32_t(tokens)}, es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, st, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, int kN>
sv_status launch_join(const AttnParams& p, int grid, cudaStream_t s) {
  constexpr int kPerBlock = kJoinThreads / 32 * join_columns_of(kN);
  return launch_dependent(join_kernel<kD, kN>, unsigned(grid * kN + kPerBlock - 1) / kPerBlock,
                          kJoinThreads, 0, s, p, grid);
}

// Few items of few tiles: a cluster of 8 CTAs for each, or of 4.  They have to be there at once (see
// clusters_at_once); more tiles are worth more SMs than a cluster has; and one warp looks through all the
// pages.  Rows of 6 under 32 heads (8 key heads): one request 8.4 us over 1000 places (14.6 from the list),
// two 12.2 over 2000 each (14.7), four 12.6 (17.7).  Eight in clusters of 2: 18.4 over 2000 places each (22.6),
// but 17.9 over 1 to 2000 (16.3), the list's runs being equal.
constexpr int kShortItems = 48, kShortRun = 8, kShortPages = 1024;

struct ShortLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ShortLaunch(int items, int ctas, cudaStream_t s) {
    cfg.gridDim = dim3(unsigned(items * ctas));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = kAttnSmem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// Clusters of kCtas that the current device runs at once (asked once per device; 0 if it cannot be asked).
template <int kD, int kN, int kCtas>
int clusters_at_once() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // and one
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    auto* kern = attention_kernel<kD, kN, kCtas>;
    ShortLaunch l(1, kCtas, nullptr);
    l.cfg.numAttrs = 1;
    int most = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kAttnSmem)) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&most, kern, &l.cfg) != cudaSuccess)
      most = 0;
    n = most + 1;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

// Sets `taken` where the call is one for clusters of kCtas, and makes it.
template <int kD, int kN, int kCtas>
sv_status launch_short(const AttnMaps& m, const AttnParams& p, int64_t items, int64_t tiles,
                       cudaStream_t s, bool& taken) {
  auto* kern = attention_kernel<kD, kN, kCtas>;
  static_assert(kN * (kD + 2) * 4 <= AttnShared<kD, kN>::kStages() * AttnShared<kD, kN>::kSlot,
                "a part fits the ring");
  if (tiles > kShortRun * kCtas || items > clusters_at_once<kD, kN, kCtas>()) return SV_OK;
  taken = true;
  ShortLaunch l(int(items), kCtas, s);
  return launch_status(cudaLaunchKernelEx(&l.cfg, kern, m.q, m.k, m.v, p));
}

template <int kD, int kN>
sv_status launch_short(const AttnMaps& m, const AttnParams& p, int64_t items, int64_t tiles,
                       cudaStream_t s, bool& taken) {
  const sv_status st = launch_short<kD, kN, 8>(m, p, items, tiles, s, taken);
  return taken ? st : launch_short<kD, kN, 4>(m, p, items, tiles, s, taken);
}

template <int kD>
sv_status launch_short(int32_t n, const AttnMaps& m, const AttnParams& p, int64_t items, int64_t tiles,
                       cudaStream_t s, bool& taken) {
  return n == 16   ? launch_short<kD, 16>(m, p, items, tiles, s, taken)
         : n == 32 ? launch_short<kD, 32>(m, p, items, tiles, s, taken)
                   : launch_short<kD, 64>(m, p, items, tiles, s, taken);
}

template <int kD, int kN>
sv_status launch(const AttnMaps& m, const AttnParams& p, int grid, cudaStream_t s) {
  auto* kern = attention_kernel<kD, kN, 0>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kAttnSmem)) !=
      cudaSuccess)
    return SV_ERR_CUDA;
  const sv_status st =
      launch_dependent(kern, unsigned(grid), kAttnThreads, kAttnSmem, s, m.q, m.k, m.v, p);
  if (st != SV_OK) return st;
  return launch_join<kD, kN>(p, grid, s);
}

template <int kD>
sv_status launch(int32_t n, const AttnMaps& m, const AttnParams& p, int grid, cudaStream_t s) {
  if (n == 16) return launch<kD, 16>(m, p, grid, s);
  if (n == 32) return launch<kD, 32>(m, p, grid, s);
  if (n == 64) return launch<kD, 64>(m, p, grid, s);
  const sv_status st = launch_wide(kD, m, p, grid, s);
  return st != SV_OK ? st : launch_join<kD, kWide>(p, grid, s);
}

}  // namespace
}  // namespace sv

using namespace sv;
using namespace sv::attn;

extern "C" size_t spec_tree_attention_workspace_bytes(int32_t B, int32_t max_draft_len,
                                                      int32_t bonus_row, int32_t n_heads,
                                                      int32_t n_kv_heads, int32_t D) {
  if (B < 0 || max_draft_len < 0 || bonus_row < 0 || bonus_row > 1 || n_heads < 1 ||
      n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 128 ||
      (D != 64 && D != 128))
    return 0;
  const int64_t rows = (max_draft_len + int64_t(bonus_row)) * (n_heads / n_kv_heads);
  return ws_layout(kMaxCtas, columns_for(rows), D).bytes;
}

extern "C" sv_status spec_tree_attention(
    const void* q, int64_t ldq, int64_t q_head, int64_t n_rows, int32_t n_heads,
    int32_t n_kv_heads, int32_t D, float scale, const int64_t* row0, const int32_t* draft_len,
    int32_t max_draft_len, int32_t bonus_row, const int32_t* parents, int32_t B,
    const int32_t* ctx_len, const int32_t* page_table, int64_t ld_pages, int32_t max_pages,
    const void* k_cache, const void* v_cache, int64_t n_pages, int32_t page_size,
    int64_t page_stride, int64_t token_stride, int64_t head_stride, void* out, int64_t ldo,
    int64_t o_head, float* lse, int64_t ld_lse, int32_t* status, void* workspace,
    size_t workspace_bytes, void* stream) {
  if (!round_sizes_ok(max_draft_len, bonus_row, B, n_rows, ld_pages, max_pages, n_pages, page_size))
    return SV_ERR_INVALID;
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || D < 1 || !std::isfinite(scale * kLog2e) ||
      (lse && ld_lse < n_heads))
    return SV_ERR_INVALID;
  if (parents && max_draft_len + int64_t(bonus_row) > SV_MAX_TREE_ROWS) return SV_ERR_UNSUPPORTED;
  const int32_t group = n_heads / n_kv_heads;
  if ((D != 64 && D != 128) || group > 128 || page_size < 8 || (page_size & (page_size - 1)))
    return SV_ERR_UNSUPPORTED;
  if (n_rows > INT32_MAX - kWide) return SV_ERR_UNSUPPORTED;  // (the end of a row tile fits 32 bits)
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || max_draft_len + int64_t(bonus_row) == 0 || n_rows == 0)
    return reset_status(status, s);
  if (!q || !out || !k_cache || !v_cache || !row0 || !draft_len || !ctx_len ||
      (!page_table && max_pages > 0) || !workspace || n_pages < 1)
    return SV_ERR_INVALID;
  if (!aligned_bf16(q, ldq, q_head, 0) || !aligned_bf16(out, ldo, o_head, 0) ||
      !aligned_bf16(k_cache, page_stride, token_stride, head_stride) || !aligned16(v_cache) ||
      !aligned256(workspace))
    return SV_ERR_UNSUPPORTED;
  if (workspace_bytes < spec_tree_attention_workspace_bytes(B, max_draft_len, bonus_row, n_heads,
                                                            n_kv_heads, D))
    return SV_ERR_INVALID;
  AttnParams p = {};
  max_draft_len = round_most_drafts(max_draft_len);
  p.rd = {row0,    draft_len, parents,       ctx_len,   page_table, ld_pages, n_rows,
          n_pages, B,         max_draft_len, bonus_row, max_pages,  page_size};
  p.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  p.page_stride = page_stride, p.token_stride = token_stride, p.head_stride = head_stride;
  p.n_kv = n_kv_heads, p.group = group;
  const int64_t rows = (max_draft_len + int64_t(bonus_row)) * group;
  const int32_t n = columns_for(rows);
  p.tile_tokens = std::min(n, kTile) / group;
  p.tokens = p.tile_tokens * (n / std::min(n, kTile));
  p.box_rows = std::min(page_size, kTile);
  p.scale2 = scale * kLog2e;
  if (p.scale2 == 0.f) p.scale2 = FLT_MIN;  // (so that -inf, a place not seen, stays -inf)
  p.out = static_cast<__nv_bfloat16*>(out), p.ldo = ldo, p.o_head = o_head;
  p.lse = lse, p.ld_lse = ld_lse, p.status = status;
  p.ws = static_cast<uint8_t*>(workspace);
  const int sms = std::min(device_sm_count(), kMaxCtas);
  if (sms < 1) return SV_ERR_CUDA;
  AttnMaps m;
  if (!query_map(&m.q, q, D, n_heads, n_rows, q_head, ldq, group, p.tile_tokens) ||
      !cache_map(&m.k, k_cache, D, n_kv_heads, page_size, n_pages, head_stride, token_stride,
                 page_stride, p.box_rows) ||
      !cache_map(&m.v, v_cache, D, n_kv_heads, page_size, n_pages, head_stride, token_stride,
                 page_stride, p.box_rows))
    return SV_ERR_UNSUPPORTED;
  // no more CTAs than there can be tiles
  const int64_t row_tiles = (max_draft_len + int64_t(bonus_row) + p.tokens - 1) / p.tokens;
  const int64_t key_tiles = (int64_t(max_pages) * page_size + kTile - 1) / kTile;
  const double items = double(B) * n_kv_heads * double(row_tiles), most = items * double(key_tiles);
  if (most > 9e15) return SV_ERR_UNSUPPORTED;
  const int grid = int(std::max(1.0, std::min(double(sms), most)));
  p.reread = row_tiles > 1;
  // (17 x 9 narrow rows over up to 3000 places: 0 33.9 us, 1 24.0, 2 19.8, 4 19.6; 32 trees of 64 rows
  // over up to 4096: 0 198 us, 2 182, 4 176, 6 171)
  p.item_cost = n == kWide ? 6 : 4;
  p.big = most + p.item_cost * items >= double(1 << 22);  // (times 192 CTAs it fits 32 bits)
  if (n <= 64 && B <= 32 && items <= kShortItems && max_pages > 0 &&
      int64_t(B) * max_pages <= kShortPages) {
    bool taken = false;
    const sv_status st = D == 64 ? launch_short<64>(n, m, p, int64_t(items), key_tiles, s, taken)
                                 : launch_short<128>(n, m, p, int64_t(items), key_tiles, s, taken);
    if (taken) return st;
  }
  return D == 64 ? launch<64>(n, m, p, grid, s) : launch<128>(n, m, p, grid, s);
}
