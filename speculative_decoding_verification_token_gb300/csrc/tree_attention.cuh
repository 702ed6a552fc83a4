// tree_attention.cuh -- what the two kernels of spec_tree_attention share: the list of work, waits,
// descriptors and tensor-memory accesses, and the parts of cut items.
#pragma once

#include "round.cuh"
#include "tc.cuh"

namespace sv {
namespace attn {

constexpr int kTile = 128;        // places of a tile
constexpr int kAttnThreads = 384;
constexpr int kSoftWarps = 8;     // warps 0-7: two halves of four, a TMEM lane a thread
constexpr int kLoadWarp = 8, kMmaWarp = 9, kItemWarp = 10, kLoadWarp2 = 11;
constexpr uint32_t kAttnSmem = 232448 - 1024;  // dynamic shared memory of a CTA, less what is static
constexpr int kWide = 256;        // rows of an item of the wide kernel: two tiles of 128
constexpr int kMaxCtas = 192;     // the workspace's size does not depend on the current device
// log2 of what P may reach before m is raised.  (m is a rounded product and P's exponent an unrounded one less
// m: with scores of 2^27, of 2^28 in base 2, P may be 2^8 off besides, the same for all of a row's.)
constexpr float kSlack = 8.f;

struct AttnParams {
  RoundParams rd;
  const __nv_bfloat16* v_cache;
  int64_t page_stride, token_stride, head_stride;
  int32_t n_kv, group;
  int32_t tokens;       // tokens of a work item: of a row tile, or of a pair of them
  int32_t tile_tokens;  // tokens of a row tile
  int32_t box_rows;  // places of a TMA box
  int32_t reread;    // several row tiles read the same keys
  int32_t item_cost; // what an item costs beside its key tiles, in key tiles
  int32_t big;       // the call's cost may pass 2^22
  float scale2;  // scale * log2(e)
  __nv_bfloat16* out;
  int64_t ldo, o_head;
  float* lse;
  int64_t ld_lse;
  int32_t* status;
  uint8_t* ws;
};

// A cut item: what the joining kernel needs of it, left by the CTA that its first part lies in.
struct Cut {
  int64_t total;      // tiles of the whole call
  int64_t first_row;  // the row tile's first row
  int32_t head, last;
};

// Workspace: per CTA its error (times 512) and the columns of its cut item (0: it begins none that it
// does not end), its cut, and two parts (0: of an item begun before it, 1: of one it
// begins) of kN x (D + 2) binary32: [kN][D] sums, [kN] maxima, [kN] denominators.
struct WsLayout {
  size_t cuts, parts, part_floats, bytes;
};
__host__ __device__ inline WsLayout ws_layout(int ctas, int n, int d) {
  WsLayout w;
  w.cuts = (size_t(ctas) * 4 + 255) / 256 * 256;
  w.parts = w.cuts + (size_t(ctas) * sizeof(Cut) + 255) / 256 * 256;
  w.part_floats = size_t(n) * (d + 2);
  w.bytes = w.parts + size_t(ctas) * 2 * w.part_floats * 4;
  return w;
}

// ---- the list of work ------------------------------------------------------------------------------

__device__ __forceinline__ int32_t tiles_of(const Request& q, int32_t rt, int32_t tokens) {
  return int32_t((int64_t(q.ctx) + min(q.n, (rt + 1) * tokens) + kTile - 1) / kTile);
}

// Items and key tiles of one key head of a request.
__device__ __forceinline__ int64_t tiles_of_head(const Request& q, int32_t tokens, int32_t& items) {
  int64_t t = 0;
  items = 0;
  for (; items * tokens < q.n; ++items) t += tiles_of(q, items, tokens);
  return t;
}

// The list is cut into runs of equal cost: an item counts its key tiles and `cost` units ahead of them.
struct Span {
  int64_t total, begin, end;  // units of the call, of this CTA
  int64_t before;             // units before request `r`
  int32_t cost;
  int32_t r;                  // the request that `begin` lies in
  Request q;                  // and its sizes
};

__device__ __forceinline__ int32_t warp_add(int32_t x, int32_t) {
  return __reduce_add_sync(0xffffffffu, x);
}
__device__ __forceinline__ int64_t warp_add(int64_t x, int32_t steps) {
  for (int o = 1; o < steps; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return __shfl_sync(0xffffffffu, x, 0);
}

// One warp: this CTA's run of the list, from the requests in chunks of 32, a lane each.  T holds the
// call's cost times the number of CTAs; the loads of kU chunks are in flight together.
template <typename T, int kU>
__device__ __forceinline__ Span find_span(const AttnParams& p, int32_t* err) {
  const int lane = threadIdx.x & 31;
  const int32_t steps = min(p.rd.B, 32);
  Span span = {};
  Request q[kU];
  T tiles[kU], items[kU];  // of the lane's requests
  auto chunks = [&](int32_t r0, bool tell) {
    int32_t drafts[kU], ctx[kU];
    int64_t first[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int32_t r = r0 + 32 * u + lane;
      if (r < p.rd.B) drafts[u] = p.rd.draft_len[r], ctx[u] = p.rd.ctx_len[r], first[u] = p.rd.row0[r];
    }
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      tiles[u] = items[u] = 0;
      q[u] = {};
      if (r0 + 32 * u + lane < p.rd.B) {
        bad |= !round_request(p.rd, drafts[u], ctx[u], first[u], q[u]);
        int32_t n;
        tiles[u] = T(tiles_of_head(q[u], p.tokens, n)) * p.n_kv;
        items[u] = T(n) * p.n_kv;
      }
    }
    if (bad && tell) report(err, SV_ERR_BAD_INPUT);
  };
  T all_tiles = 0, all_items = 0;
  for (int32_t r0 = 0; r0 < p.rd.B; r0 += 32 * kU) {
    chunks(r0, blockIdx.x == 0);
#pragma unroll
    for (int u = 1; u < kU; ++u) tiles[0] += tiles[u], items[0] += items[u];
    all_tiles += warp_add(tiles[0], steps);
    all_items += warp_add(items[0], steps);
#pragma unroll
    for (int u = 1; u < kU; ++u) tiles[0] -= tiles[u], items[0] -= items[u];
  }
  // (with few tiles for each CTA their number alone counts)
  span.cost = all_tiles > 2 * T(gridDim.x) ? p.item_cost : 0;
  const T total = all_tiles + span.cost * all_items;
  const T begin = total * T(blockIdx.x) / T(gridDim.x), end = total * T(blockIdx.x + 1) / T(gridDim.x);
  span.total = total, span.begin = begin, span.end = end;
  if (begin == end) return span;
  T before = 0;
  for (int32_t r0 = 0; r0 < p.rd.B; r0 += 32 * kU) {
    if (p.rd.B > 32 * kU) chunks(r0, false);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (r0 + 32 * u >= p.rd.B) break;
      const T mine = tiles[u] + span.cost * items[u];
      T upto = mine;
      for (int o = 1; o < steps; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const T a = before + upto - mine;
      const uint32_t hit = __ballot_sync(0xffffffffu, mine > 0 && a <= begin && begin < a + mine);
      if (hit) {
        const int l = __ffs(hit) - 1;
        span.before = __shfl_sync(0xffffffffu, a, l);
        span.r = r0 + 32 * u + l;
        span.q.first = __shfl_sync(0xffffffffu, q[u].first, l);
        span.q.n = __shfl_sync(0xffffffffu, q[u].n, l);
        span.q.ctx = __shfl_sync(0xffffffffu, q[u].ctx, l);
        return span;
      }
      before += __shfl_sync(0xffffffffu, upto, steps - 1);
    }
  }
  return span;
}

// ---- small pieces ----------------------------------------------------------------------------------

__device__ __forceinline__ bool try_wait_for(uint64_t* bar, uint32_t parity) {
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

// Wait for phase `parity`, asleep; gives up after kWaitLimitNs and reports it.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int32_t* err) {
  if (try_wait_for(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!try_wait_for(bar, parity)) {
    if (global_ns() - t0 > kWaitLimitNs) {
      report(err, SV_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The same by a whole warp: one answer.
__device__ __forceinline__ bool wait_for_warp(uint64_t* bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, err));
}

__device__ __forceinline__ bool elect() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// Barrier of a half's four softmax warps (1 or 2) that also tells whether `x` held in any thread.
__device__ __forceinline__ bool soft_any(int half, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(uint32_t(x)), "r"(1 + half)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void soft_sync(int half) { named_sync(1 + half, 128); }

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* map, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3, uint64_t* bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar)),
      "l"(policy)
      : "memory");
}

// Shared-memory descriptors of 128-byte swizzled operands by halves (low word: address >> 4 and leading
// offset, high word: stride offset 1024, version 1, swizzle).  Operands whose rows run along the
// contraction (K, Q) leave the leading offset unused; in those whose rows run along M or N (V, P: a row
// of 64 elements a place) it is the distance between groups of 64, and eight places are 1024 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kAlongK = 1u << 16;
constexpr uint32_t kAcross = (16384u >> 4) << 16;  // groups of 64: 128 places of 128 bytes
// A descriptor's address bits (a CTA of a cluster has its rank in the upper ones of its own addresses).
__device__ __forceinline__ uint32_t desc_at(const void* p) { return (smem_addr(p) & 0x3FFFFu) >> 4; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kDescHi));
  return d;
}

// C columns of this thread's TMEM lane.
template <int C>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float* v) {
  if constexpr (C == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7])
        : "r"(taddr)
        : "memory");
  } else if constexpr (C == 16) {
    tc::tmem_load16(taddr, v);
  } else {
    tc::tmem_load32(taddr, v);
  }
}

template <int C>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const float* v) {
#pragma unroll
  for (int j = 0; j < C; j += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     taddr + j),
                 "f"(v[j]), "f"(v[j + 1]), "f"(v[j + 2]), "f"(v[j + 3]), "f"(v[j + 4]),
                 "f"(v[j + 5]), "f"(v[j + 6]), "f"(v[j + 7])
                 : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// C columns a lane joined over the lanes by `op`: column lane % C's result in every lane.  Half of what
// a lane holds goes to the lane that keeps it, in every step.
template <int C, typename Op>
__device__ __forceinline__ float over_lanes(float* v, Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o >= C; o >>= 1) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = op(v[j], __shfl_xor_sync(0xffffffffu, v[j], o));
  }
#pragma unroll
  for (int o = C / 2; o > 0; o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float give = upper ? v[j] : v[j + o], keep = upper ? v[j + o] : v[j];
      v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return v[0];
}

// C consecutive values of shared memory, the same in every lane.
template <int C>
__device__ __forceinline__ void broadcast(const float* at, float* v) {
#pragma unroll
  for (int j = 0; j < C; j += 4) {
    const float4 x = *reinterpret_cast<const float4*>(at + j);
    v[j] = x.x, v[j + 1] = x.y, v[j + 2] = x.z, v[j + 3] = x.w;
  }
}

// s scale + minus, in pairs.
template <int C>
__device__ __forceinline__ void scaled(float* s, float scale, const float* minus) {
  const float2 f = splat2(scale);
#pragma unroll
  for (int j = 0; j < C; j += 2) {
    const float2 y = fma2(make_float2(s[j], s[j + 1]), f, make_float2(minus[j], minus[j + 1]));
    s[j] = y.x, s[j + 1] = y.y;
  }
}

// -inf in the columns whose bit is clear.
template <int C>
__device__ __forceinline__ void hide(float* y, uint32_t seen) {
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (!(seen >> j & 1u)) y[j] = -INFINITY;
}

// A work item as the warps of a CTA share it.
struct Item {
  int64_t first_row;  // row of the tile's first token
  int32_t r, head, columns;
  int32_t tok0, ctx;  // the request's rows before it, places filled before
  int32_t base0;   // places below it are seen by every column
  int32_t end;     // places from it on by none
  int32_t t0, t1;  // its key tiles in this CTA
  int32_t whole, begins, last;
  int32_t stop;    // no item: the list is at its end
};

// The items of this CTA's run, by one warp: item_full says that an item's description is there (of 2^kLog
// at a time), item_empty that nobody needs it any more.  `after` adds what is not needed at once.
// Ends the list with an item that says so, and leaves the CTA's cut item in the workspace; returns its
// columns.
template <int kLog, typename After>
__device__ __forceinline__ int32_t walk_items(const AttnParams& p, Cut* cuts, Item* item,
                                              uint64_t* item_full, uint64_t* item_empty,
                                              int32_t* err, After after) {
  constexpr int kItems = 1 << kLog;
  const int lane = threadIdx.x & 31;
  const Span span = p.big          ? find_span<int64_t, 4>(p, err)
                    : p.rd.B > 32 ? find_span<int32_t, 4>(p, err)
                                  : find_span<int32_t, 1>(p, err);
  Cut cut = {};
  int32_t cut_columns = 0;
  bool ok = true;
  int32_t it = 0;
  if (span.begin < span.end) {
    int64_t at = span.begin, off = at - span.before;  // units of the call, and of the request's first item
    int32_t r = span.r, h = 0, rt = 0;
    Request rq = span.q;
    int32_t n_items;
    int64_t per_head = tiles_of_head(rq, p.tokens, n_items);
    per_head += int64_t(span.cost) * n_items;
    h = p.big ? int32_t(off / per_head) : int32_t(uint32_t(off) / uint32_t(per_head));
    off -= h * per_head;
    while (off >= tiles_of(rq, rt, p.tokens) + span.cost)
      off -= tiles_of(rq, rt++, p.tokens) + span.cost;
    while (at < span.end && ok) {
      const int32_t tiles = tiles_of(rq, rt, p.tokens);
      const int64_t units = min(tiles + span.cost - off, span.end - at);
      const int64_t t0 = max(off - span.cost, int64_t(0)), t1 = off + units - span.cost;
      if (t1 > t0) {  // (else the run ends within what stands for the item's own cost)
        const int b = it & (kItems - 1);
        const int32_t tok0 = rt * p.tokens, ntok = min(p.tokens, rq.n - tok0);
        const int32_t columns = ntok * p.group;
        Item x;
        x.first_row = rq.first + tok0;
        x.r = r, x.head = h, x.columns = columns;
        x.tok0 = tok0, x.ctx = rq.ctx;
        x.base0 = rq.ctx + (p.rd.parents ? 0 : tok0);
        x.end = rq.ctx + tok0 + ntok;
        x.t0 = int32_t(t0);
        x.t1 = int32_t(t1);
        x.whole = x.t0 == 0 && x.t1 == tiles;
        x.begins = x.t0 == 0;
        x.last = span.end - (at + units) <= span.cost;
        x.stop = 0;
        if (it >= kItems && !wait_for_warp(&item_empty[b], ((it >> kLog) - 1) & 1, err)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          item[b] = x;
          mbar_arrive(&item_full[b]);
        }
        __syncwarp();
        after(b, x, rq.first);
        if (x.begins && !x.whole) {
          cut.total = span.total;
          cut.first_row = x.first_row;
          cut.head = h;
          // the CTA that the item's last unit lies in
          const int64_t end = (at - off + tiles + span.cost) * gridDim.x - 1;
          cut.last = p.big ? int32_t(end / cut.total) : int32_t(uint32_t(end) / uint32_t(cut.total));
          cut_columns = columns;
        }
        ++it;
      }
      at += units;
      off = 0;
      if (at < span.end && ++rt * p.tokens >= rq.n) {
        rt = 0;
        if (++h == p.n_kv) {
          h = 0;
          do {
            if (++r == p.rd.B) break;
            round_request(p.rd, r, rq);
          } while (rq.n == 0);
          ok = r < p.rd.B;
        }
      }
    }
  }
  const int b = it & (kItems - 1);
  if (ok && (it < kItems || wait_for_warp(&item_empty[b], ((it >> kLog) - 1) & 1, err)) && lane == 0) {
    item[b].stop = 1;
    mbar_arrive(&item_full[b]);
  }
  if (lane == 0 && cut_columns) cuts[blockIdx.x] = cut;
  return cut_columns;
}

// above[i] = rows above row i of a tree, itself included, for its first `nodes` rows; one warp.
__device__ __forceinline__ void build_above(const AttnParams& p, int64_t first, int32_t nodes,
                                            int32_t* up, uint32_t (*above)[4], int32_t* err) {
  const int lane = threadIdx.x & 31;
  for (int32_t i = lane; i < nodes; i += 32) {
    int32_t u = p.rd.parents[first + i];
    if (u < -1 || u >= i) {
      report(err, SV_ERR_BAD_INPUT);
      u = -1;
    }
    up[i] = u;
#pragma unroll
    for (int w = 0; w < 4; ++w) above[i][w] = i >> 5 == w ? 1u << (i & 31) : 0u;
  }
  __syncwarp();
  // the way up doubles its length a round: a row takes over what the row at its end has
  for (int round = 0; round < 7; ++round) {
    uint32_t a[4][4];
    int32_t next[4];
    bool more = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t i = k * 32 + lane;
      next[k] = -1;
      if (i < nodes && up[i] >= 0) {
        more = true;
        next[k] = up[up[i]];
#pragma unroll
        for (int w = 0; w < 4; ++w) a[k][w] = above[i][w] | above[up[i]][w];
      }
    }
    if (!__any_sync(0xffffffffu, more)) break;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t i = k * 32 + lane;
      if (i < nodes && up[i] >= 0) {
#pragma unroll
        for (int w = 0; w < 4; ++w) above[i][w] = a[k][w];
        up[i] = next[k];
      }
    }
    __syncwarp();
  }
}

// The boxes of a tile, one a lane, are loaded by kLoaders warps: of two, each takes 64 of the 128 elements, or
// every other box of 64.  One warp's issue is what bounds small pages -- 256 requests of one token over up
// to 4096 places in pages of 16: 449 us by one warp, 361 by two.
template <int kD, int kLoaders>
__device__ __forceinline__ int box_of_lane(int part) {
  const int lane = threadIdx.x & 31;
  return kLoaders == 1 || kD == 128 ? lane : 2 * lane + part;
}

// The TMA boxes of key tile t, one a lane: page and first place in it.  Returns how many.
template <int kD, int kLoaders>
__device__ __forceinline__ int32_t tile_boxes(const AttnParams& p, const Item& x, int32_t t,
                                              int part, int32_t& page, int32_t& from, int32_t* err) {
  const int box = box_of_lane<kD, kLoaders>(part);
  const int32_t boxes = (min(kTile, x.end - t * kTile) + p.box_rows - 1) / p.box_rows;
  const int32_t place = t * kTile + box * p.box_rows;
  page = 0;
  if (box < boxes) {
    page = round_page(p.rd, x.r, place);
    if (page < 0) {
      report(err, SV_ERR_BAD_INPUT);
      page = 0;
    }
  }
  from = place & (p.rd.page_size - 1);
  return boxes;
}

// A warp's part of a tile of K or V into a ring slot of [D / 64][128 places][64 elements], swizzled.
template <int kD, int kLoaders, bool kRowTiles>
__device__ __forceinline__ void load_tile(const AttnParams& p, uint8_t* dst, const CUtensorMap* map,
                                          int part, int32_t page, int32_t from, int32_t boxes,
                                          int32_t head, uint64_t* full, uint64_t once) {
  constexpr int kEach = kLoaders == 2 ? 1 : kD / 64;  // loads of a box
  const int box = box_of_lane<kD, kLoaders>(part), k0 = kD == 128 ? part : 0;
  const int32_t mine = kLoaders == 1 || kD == 128 ? boxes : (boxes + 1 - part) / 2;
  if (elect()) mbar_expect_tx(full, uint32_t(mine) * p.box_rows * kEach * 128);
  __syncwarp();
  if (box < boxes) {
#pragma unroll
    for (int k = k0; k < k0 + kEach; ++k) {
      uint8_t* const to = dst + k * 16384 + box * p.box_rows * 128;
      // (keys that other row tiles of the request read too stay in L2 like anything else)
      if (kRowTiles && p.reread) tma_load_4d(to, map, k * 64, head, from, page, full);
      else tma_load_4d_hint(to, map, k * 64, head, from, page, full, once);
    }
  }
  __syncwarp();
}

// Values that are seen by some rows only must be finite for the product: a weight of 0 would not rid the
// others of them.  Of place `row` of a V tile, 16-byte chunks k0 .. k0 + kCount - 1: zeros if it is
// past the end, zeros for what is not finite otherwise; returns whether there was such a thing, which
// is added to the rows that do see it at the end.
template <int kCount>
__device__ __forceinline__ bool make_finite(uint8_t* v, int row, int k0, bool past) {
  auto chunk = [&](int i) {
    const int k = k0 + i;
    return reinterpret_cast<uint4*>(v + (k >> 3) * 16384 + tc::sw128(row, k & 7));
  };
  if (past) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) *chunk(i) = make_uint4(0, 0, 0, 0);
    return false;
  }
  // an exponent of all ones carries into the sign's place
  auto ones = [](uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; };
  uint32_t found = 0;
#pragma unroll
  for (int i = 0; i < kCount; ++i) {
    const uint4 y = *chunk(i);
    found |= ones(y.x) | ones(y.y) | ones(y.z) | ones(y.w);
  }
  if (!(found & 0x80008000u)) return false;
#pragma unroll 1
  for (int i = 0; i < kCount; ++i) {
    uint4 y = *chunk(i);
    uint32_t* const w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t o = ones(w[e]);
      w[e] &= (o & 0x8000u ? 0u : 0xFFFFu) | (o & 0x80000000u ? 0u : 0xFFFF0000u);
    }
    *chunk(i) = y;
  }
  return true;
}

// Element d of row j (of those that not everybody sees) in the cache.
__device__ __forceinline__ float value_at(const AttnParams& p, const Item& x, int32_t j, int32_t d) {
  const int32_t place = x.base0 + j, page = max(round_page(p.rd, x.r, place), 0);
  return __bfloat162float(p.v_cache[page * p.page_stride +
                                    (place & (p.rd.page_size - 1)) * p.token_stride +
                                    x.head * p.head_stride + d]);
}

struct AttnMaps {
  CUtensorMap q, k, v;
};

// tree_attention_wide.cu: more than 64 rows a key head.
sv_status launch_wide(int32_t D, const AttnMaps& m, const AttnParams& p, int grid, cudaStream_t s);

}  // namespace attn
}  // namespace sv
