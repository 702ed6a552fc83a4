// cache.cu -- a round's keys and values in the paged cache: written with the position rotation
// (spec_cache_append), and the accepted path's moved together (spec_cache_keep).  Between the two
// lies the walk down the tree of drafts (spec_tree_accept).
#include "round.cuh"

#include <algorithm>

namespace sv {
namespace {

// ---- append ----------------------------------------------------------------------------------------

struct AppendParams {
  RoundParams rd;
  CacheParams cache;
  const void *q, *k, *v;
  int64_t ldq, q_head, ldk, k_head, ldv, v_head;
  __nv_bfloat16* q_out;
  int64_t ldqo, qo_head;
  const float* cos_sin;
  int64_t ld_cos_sin, n_positions;  // (without a rotation any position will do)
  int32_t n_heads, n_kv_heads, D, rot;
  int32_t rows;    // of a CTA
  int32_t chunks;  // CTAs of a request
  int32_t* status;
  bool one;
};

constexpr int kAppendThreads = 256;
constexpr int kRowThreads = 128;  // of a row
constexpr int kAppendGroups = kAppendThreads / kRowThreads;
// Heads whose loads a thread has in flight, and CTAs an SM, within the registers there are: 8 prompts of
// up to 8192 tokens (bf16) 136 us (5.8 TB/s of the 784 MB that have to move; two CTAs 149), in fp32 203 us (5.8
// TB/s); 64 trees of 16 rows (fp32) 8.1 us where everything lies in L2 (three CTAs spill: 16.6), 9 to 12 from memory.
template <typename T>
constexpr int kAppendUnroll = sizeof(T) == 2 ? 3 : 2;
template <typename T>
constexpr int kAppendCtas = sizeof(T) == 2 ? 3 : 2;
constexpr int kAppendMostRows = 16;  // of a CTA

// 8 consecutive elements: as they lie, and as binary32.
template <typename T>
struct Eight {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (int j = 0; j < int(sizeof(T) / 2); ++j) raw[j] = reinterpret_cast<const uint4*>(x)[j];
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (sizeof(T) == 2) {
      Elem<bf16_tag>::unpack(raw[0], f);
    } else {
      Elem<float>::unpack(raw[0], f);
      Elem<float>::unpack(raw[1], f + 4);
    }
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* o, const float* f) {
  uint4 v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(o) = v;
}

// 128 threads a row: a thread keeps one sixteen-element part of the heads (two runs of 8: the pairs
// of a rotation, or neighbours) with that part's cosines and sines, and goes through the heads of q, k
// and v with it.  Returns whether it found bad data.
template <typename T, bool kAdjacent>
__device__ __forceinline__ bool append_body(const AppendParams& p, int32_t* parents) {
  const int32_t r = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int32_t sub = threadIdx.x / kRowThreads, t = threadIdx.x % kRowThreads;
  Request rq;
  if (!round_request(p.rd, r, rq)) return chunk == 0;
  const int32_t begin = chunk * p.rows, end = min(begin + p.rows, rq.n);
  if (begin >= end) return false;
  bool bad = false;
  if (p.rd.parents) {
    for (int32_t j = threadIdx.x; j < end; j += kAppendThreads) {
      int32_t up = p.rd.parents[rq.first + j];
      if (up < -1 || up >= j) {
        bad = true;
        up = -1;
      }
      parents[j] = up;
    }
    __syncthreads();
  }
  const int32_t parts = p.D >> 4, rot_parts = p.rot >> 4;
  const int32_t part = t % parts, step = kRowThreads / parts;
  if (t >= parts * step) return bad;
  const bool turn = part < rot_parts;
  const bool halves = turn && !kAdjacent;
  const int32_t e0 = halves ? part * 8 : part * 16, e1 = halves ? e0 + (p.rot >> 1) : e0 + 8;
  const int32_t all = p.n_heads + 2 * p.n_kv_heads;
  for (int32_t i = begin + sub; i < end; i += kAppendGroups) {
    int32_t depth = i;
    if (p.rd.parents) {
      depth = 0;
      for (int32_t j = parents[i]; j >= 0; j = parents[j]) ++depth;
    }
    Eight<float> c8, s8;
    const int64_t pos = int64_t(rq.ctx) + depth;
    if (pos >= p.n_positions) {  // (for the threads of parts that do not turn too)
      bad = true;
      continue;
    }
    if (turn) {
      const float* row = p.cos_sin + pos * p.ld_cos_sin + part * 8;
      c8.load(row);
      s8.load(row + (p.rot >> 1));
    }
    const int32_t place = rq.ctx + i, page = round_page(p.rd, r, place);
    bad |= page < 0;
    const int64_t at = page * p.cache.page_stride + (place % p.rd.page_size) * p.cache.token_stride;
    const int64_t row = rq.first + i;
    for (int32_t h0 = t / parts; h0 < all; h0 += step * kAppendUnroll<T>) {
      Eight<T> x[kAppendUnroll<T>], y[kAppendUnroll<T>];
#pragma unroll
      for (int u = 0; u < kAppendUnroll<T>; ++u) {
        const int32_t h = h0 + u * step, kv = h - p.n_heads;
        if (h < all) {
          const bool v_head = kv >= p.n_kv_heads;
          const T* src = kv < 0 ? static_cast<const T*>(p.q) + row * p.ldq + h * p.q_head
                         : v_head ? static_cast<const T*>(p.v) + row * p.ldv + (kv - p.n_kv_heads) * p.v_head
                                  : static_cast<const T*>(p.k) + row * p.ldk + kv * p.k_head;
          x[u].load(src + (v_head ? part * 16 : e0));
          y[u].load(src + (v_head ? part * 16 + 8 : e1));
        }
      }
#pragma unroll
      for (int u = 0; u < kAppendUnroll<T>; ++u) {
        const int32_t h = h0 + u * step, kv = h - p.n_heads;
        if (h >= all || (kv >= 0 && page < 0)) continue;
        const bool v_head = kv >= p.n_kv_heads;
        __nv_bfloat16* dst = kv < 0   ? p.q_out + row * p.ldqo + h * p.qo_head
                             : v_head ? p.cache.v + at + (kv - p.n_kv_heads) * p.cache.head_stride
                                      : p.cache.k + at + kv * p.cache.head_stride;
        float a[8], b[8];
        x[u].get(a);
        y[u].get(b);
        if (turn && !v_head) {
          float c[8], s[8];
          c8.get(c);
          s8.get(s);
          if constexpr (kAdjacent) {  // pairs within each run of 8: angles 0-3 and 4-7
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = a[2 * j], g = a[2 * j + 1];
              a[2 * j] = f * c[j] - g * s[j];
              a[2 * j + 1] = f * s[j] + g * c[j];
              const float z = b[2 * j], w = b[2 * j + 1];
              b[2 * j] = z * c[4 + j] - w * s[4 + j];
              b[2 * j + 1] = z * s[4 + j] + w * c[4 + j];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float f = a[j], g = b[j];
              a[j] = f * c[j] - g * s[j];
              b[j] = f * s[j] + g * c[j];
            }
          }
        }
        store8(dst + (v_head ? part * 16 : e0), a);
        store8(dst + (v_head ? part * 16 + 8 : e1), b);
      }
    }
  }
  return bad;
}

template <typename T, bool kAdjacent>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas<T>) append_kernel(AppendParams p) {
  __shared__ int32_t parents[SV_MAX_TREE_ROWS];
  dependent_start();
  round_status(p.status, append_body<T, kAdjacent>(p, parents), p.one);
}

// ---- accept ----------------------------------------------------------------------------------------

struct AcceptParams {
  const int32_t *sampled, *tokens, *parents, *draft_len;
  const int64_t *row0, *draft_row0;
  int64_t n_rows, n_drafts;
  int32_t B, max_draft_len;
  int32_t *accepted_len, *out_tokens, *correction, *path;
  int64_t out_ld, ld_path;
  int32_t* status;
  bool one;
};

constexpr int kTreeWords = SV_MAX_TREE_ROWS / 32;

// A warp per request: the rows' parents, tokens and samples in registers, row i in lane i % 32.  A
// step compares every row with the one the walk stands on; children follow their parents, so the
// first match is the lowest child.
// Returns whether the data are bad.
__device__ __forceinline__ bool accept_body(const AcceptParams& p) {
  const int32_t r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= p.B) return false;
  const int32_t drafts = p.draft_len[r];
  const int64_t first = p.row0[r], dfirst = p.draft_row0[r];
  bool bad = drafts < 0 || drafts > p.max_draft_len || first < 0 || first >= p.n_rows ||
             drafts >= p.n_rows - first ||
             (drafts > 0 && (dfirst < 0 || dfirst > p.n_drafts || drafts > p.n_drafts - dfirst));
  int32_t* const out = p.out_tokens + r * p.out_ld;
  int32_t* const path = p.path ? p.path + r * p.ld_path : nullptr;
  // Nothing is emitted: a length of -1, with which spec_cache_keep leaves the request as it was, and no token
  // of an earlier round for the history.
  auto nothing = [&] {
    __syncwarp();  // (over what a walk has written)
    if (lane == 0) {
      p.accepted_len[r] = -1;
      if (p.correction) p.correction[r] = -1;
    }
    for (int32_t i = lane; i <= p.max_draft_len; i += 32) out[i] = -1;
    if (path)
      for (int32_t i = lane; i < p.max_draft_len; i += 32) path[i] = -1;
    return true;
  };
  if (bad) return nothing();
  int32_t parent[kTreeWords], token[kTreeWords], sample[kTreeWords];
#pragma unroll
  for (int k = 0; k < kTreeWords; ++k) {
    const int32_t i = k * 32 + lane;
    parent[k] = -2;  // nobody's child
    token[k] = sample[k] = -1;
    if (i <= drafts) {
      sample[k] = p.sampled[first + i];
      if (i > 0) token[k] = p.tokens[dfirst + i - 1];
      parent[k] = p.parents ? p.parents[first + i] : i - 1;
      bad |= parent[k] < -1 || parent[k] >= i;
    }
  }
  int32_t at = 0, n = 0, t = 0;
  for (;;) {
    const int32_t word = at >> 5;
    const int32_t mine = word == 0 ? sample[0] : word == 1 ? sample[1] : word == 2 ? sample[2] : sample[3];
    t = __shfl_sync(0xffffffffu, mine, at & 31);
    if (t < 0) return nothing();
    int32_t next = -1;
#pragma unroll
    for (int k = kTreeWords - 1; k >= 0; --k) {
      // (a row with a bad parent, not below it, must not lead the walk round)
      const int32_t i = k * 32 + lane;
      const uint32_t hit =
          __ballot_sync(0xffffffffu, parent[k] == at && token[k] == t && i > at);
      if (hit) next = k * 32 + __ffs(hit) - 1;
    }
    if (next < 0) break;
    if (lane == 0) {
      out[n] = t;
      if (path) path[n] = next;
    }
    ++n;
    at = next;
  }
  if (lane == 0) {
    out[n] = t;
    p.accepted_len[r] = n;
    if (p.correction) p.correction[r] = t;
  }
  for (int32_t i = n + 1 + lane; i <= p.max_draft_len; i += 32) out[i] = -1;
  if (path)
    for (int32_t i = n + lane; i < p.max_draft_len; i += 32) path[i] = -1;
  return bad;
}

__global__ void __launch_bounds__(1024) accept_kernel(AcceptParams p) {
  dependent_start();
  round_status(p.status, accept_body(p), p.one);
}

// ---- keep ------------------------------------------------------------------------------------------

struct KeepParams {
  RoundParams rd;  // tables and lengths only
  CacheParams cache;
  const int32_t *accepted_len, *path;
  int64_t ld_path;
  int32_t n_path, n_layers;
  int32_t layers;  // of a CTA
  int64_t layer_stride;
  int32_t columns;       // 16-byte columns of a place in one cache
  int32_t head_columns;  // of a head
  int32_t* new_len;
  int32_t* status;
  bool one;
};

constexpr int kKeepThreads = 256;
constexpr int kKeepBatch = 8;
// CTAs aimed at an SM: 64 requests in 32 layers 10.2 us where the rows lie in L2 (2: 13.4, 16: 11.7), 15 from memory.
constexpr int kKeepCtas = 6;

// A CTA per request and run of layers.  A path ascends from 1 or more, so row path[i] lies at or behind the
// place i + 1 it goes to, and a thread that takes its own 16-byte column through the moves in order
// never reads what it has overwritten; it reads a batch of rows ahead of writing them.
// Returns whether the data are bad.
__device__ __forceinline__ bool keep_body(const KeepParams& p, int64_t* src, int64_t* dst) {
  const int32_t r = blockIdx.x % p.rd.B, tid = threadIdx.x;
  const int32_t layer0 = blockIdx.x / p.rd.B * p.layers;
  const int32_t ctx = p.rd.ctx_len[r], n = p.accepted_len[r];
  const int64_t room = min(int64_t(p.rd.max_pages) * p.rd.page_size, int64_t(INT32_MAX));
  bool bad = n < 0 || n > p.n_path || ctx < 0 || int64_t(ctx) + 1 + n > room;
  int32_t from = 0, page_from = 0, page_to = 0;
  if (!bad && p.path && tid < n) {
    const int32_t* const path = p.path + r * p.ld_path;
    from = path[tid];
    bad = from <= (tid > 0 ? path[tid - 1] : 0) || ctx + int64_t(from) >= room;
    if (!bad) {
      page_from = round_page(p.rd, r, ctx + from);
      page_to = round_page(p.rd, r, ctx + 1 + tid);
      bad = page_from < 0 || page_to < 0;
    }
  }
  bad = __syncthreads_or(bad);
  if (layer0 == 0 && tid == 0 && p.new_len) p.new_len[r] = bad ? ctx : ctx + 1 + n;
  if (bad) return layer0 == 0 && tid == 0;
  if (!p.path) return false;
  // a path starts with the rows that lie in place; from its first gap on every row moves
  const bool move = tid < n && from != tid + 1;
  const int32_t count = __syncthreads_count(move);
  if (move) {
    const int32_t m = tid - (n - count), ps = p.rd.page_size;
    src[m] = page_from * p.cache.page_stride + ((ctx + from) % ps) * p.cache.token_stride;
    dst[m] = page_to * p.cache.page_stride + ((ctx + 1 + tid) % ps) * p.cache.token_stride;
  }
  __syncthreads();
  const int32_t layers = min(p.layers, p.n_layers - layer0);
  for (int32_t c = tid; c < 2 * p.columns; c += kKeepThreads) {
    const int32_t col = c < p.columns ? c : c - p.columns;
    __nv_bfloat16* base = (c < p.columns ? p.cache.k : p.cache.v) + layer0 * p.layer_stride +
                          (col / p.head_columns) * p.cache.head_stride +
                          (col % p.head_columns) * 8;
    for (int32_t layer = 0; layer < layers; ++layer, base += p.layer_stride) {
      for (int32_t m0 = 0; m0 < count; m0 += kKeepBatch) {
        uint4 x[kKeepBatch];
#pragma unroll
        for (int u = 0; u < kKeepBatch; ++u)
          if (m0 + u < count) x[u] = *reinterpret_cast<const uint4*>(base + src[m0 + u]);
#pragma unroll
        for (int u = 0; u < kKeepBatch; ++u)
          if (m0 + u < count) *reinterpret_cast<uint4*>(base + dst[m0 + u]) = x[u];
      }
    }
  }
  return false;
}

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(KeepParams p) {
  __shared__ int64_t src[SV_MAX_TREE_ROWS], dst[SV_MAX_TREE_ROWS];
  dependent_start();
  round_status(p.status, keep_body(p, src, dst), p.one);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status spec_cache_append(
    const void* q, int64_t ldq, int64_t q_head, const void* k, int64_t ldk, int64_t k_head,
    const void* v, int64_t ldv, int64_t v_head, sv_dtype dtype, int64_t n_rows, int32_t n_heads,
    int32_t n_kv_heads, int32_t D, const float* cos_sin, int64_t ld_cos_sin, int64_t n_positions,
    int32_t rot, int32_t adjacent, const int64_t* row0, const int32_t* draft_len,
    int32_t max_draft_len, int32_t bonus_row, const int32_t* parents, int32_t B,
    const int32_t* ctx_len, const int32_t* page_table, int64_t ld_pages, int32_t max_pages,
    void* q_out, int64_t ldqo, int64_t qo_head, void* k_cache, void* v_cache, int64_t n_pages,
    int32_t page_size, int64_t page_stride, int64_t token_stride, int64_t head_stride,
    int32_t* status, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID;
  if (!round_sizes_ok(max_draft_len, bonus_row, B, n_rows, ld_pages, max_pages, n_pages, page_size))
    return SV_ERR_INVALID;
  if (n_heads < 0 || n_kv_heads < 1 || D < 1 || (adjacent != 0 && adjacent != 1))
    return SV_ERR_INVALID;
  if (cos_sin ? rot < 1 || rot > D || ld_cos_sin < rot || n_positions < 0 : rot != 0)
    return SV_ERR_INVALID;
  if (parents && max_draft_len + int64_t(bonus_row) > SV_MAX_TREE_ROWS) return SV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || max_draft_len + int64_t(bonus_row) == 0 || n_rows == 0) return reset_status(status, s);
  if (!k || !v || !k_cache || !v_cache || !row0 || !draft_len || !ctx_len ||
      (!page_table && max_pages > 0) ||
      (n_heads > 0 && (!q || !q_out)))
    return SV_ERR_INVALID;
  if (D % 16 || D > 256 || rot % 16) return SV_ERR_UNSUPPORTED;
  if (int64_t(n_heads) + 2 * int64_t(n_kv_heads) > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
  const int64_t in = 16 / elem_bytes(dtype);
  if (!aligned16(k) || !aligned16(v) || ldk % in || k_head % in || ldv % in || v_head % in ||
      (n_heads > 0 && (!aligned16(q) || ldq % in || q_head % in ||
                       !aligned_bf16(q_out, ldqo, qo_head, 0))) ||
      (cos_sin && (!aligned16(cos_sin) || ld_cos_sin % 4)) ||
      !aligned_bf16(k_cache, page_stride, token_stride, head_stride) || !aligned16(v_cache))
    return SV_ERR_UNSUPPORTED;
  if (n_heads > 0 && q_out == q && (dtype != SV_BF16 || ldqo != ldq || qo_head != q_head))
    return SV_ERR_INVALID;
  AppendParams p = {};
  max_draft_len = round_most_drafts(max_draft_len);
  p.rd = {row0,    draft_len, parents,       ctx_len,   page_table, ld_pages, n_rows,
          n_pages, B,         max_draft_len, bonus_row, max_pages,  page_size};
  p.cache = {static_cast<__nv_bfloat16*>(k_cache), static_cast<__nv_bfloat16*>(v_cache),
             page_stride, token_stride, head_stride};
  p.q = q, p.k = k, p.v = v;
  p.ldq = ldq, p.q_head = q_head, p.ldk = ldk, p.k_head = k_head, p.ldv = ldv, p.v_head = v_head;
  p.q_out = static_cast<__nv_bfloat16*>(q_out), p.ldqo = ldqo, p.qo_head = qo_head;
  p.cos_sin = cos_sin, p.ld_cos_sin = ld_cos_sin;
  p.n_positions = cos_sin ? n_positions : INT64_MAX;
  p.n_heads = n_heads, p.n_kv_heads = n_kv_heads, p.D = D, p.rot = rot;
  const int64_t most = max_draft_len + int64_t(bonus_row);
  // a CTA takes several rows where there are enough of them for two rounds of CTAs: what it finds out of
  // its request first costs as much as a row (prompts as above 165 -> 136 us)
  if ((most + kAppendMostRows - 1) / kAppendMostRows * B > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms < 1) return SV_ERR_CUDA;
  p.rows = kAppendGroups;
  while (p.rows < kAppendMostRows && most * B >= int64_t(4) * 3 * sms * p.rows) p.rows *= 2;
  p.chunks = int32_t((most + p.rows - 1) / p.rows);
  p.status = status;
  auto* kernel = dtype == SV_BF16
                     ? (adjacent ? append_kernel<__nv_bfloat16, true>
                                 : append_kernel<__nv_bfloat16, false>)
                     : (adjacent ? append_kernel<float, true> : append_kernel<float, false>);
  return launch_round(kernel, int64_t(p.chunks) * B, kAppendThreads, s, p);
}

extern "C" sv_status spec_tree_accept(const int32_t* sampled, const int32_t* draft_tokens,
                                      const int32_t* parents, const int64_t* row0,
                                      const int64_t* draft_row0, const int32_t* draft_len,
                                      int32_t max_draft_len, int32_t B, int64_t n_rows,
                                      int64_t n_drafts, int32_t* accepted_len,
                                      int32_t* out_tokens, int64_t out_ld,
                                      int32_t* correction_token, int32_t* path, int64_t ld_path,
                                      int32_t* status, void* stream) {
  if (max_draft_len < 0 || B < 0 || n_rows < 0 || n_drafts < 0 ||
      out_ld < int64_t(max_draft_len) + 1 || (path && ld_path < max_draft_len))
    return SV_ERR_INVALID;
  if (max_draft_len >= SV_MAX_TREE_ROWS) return SV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0) return reset_status(status, s);
  if (!sampled || !row0 || !draft_row0 || !draft_len || !accepted_len || !out_tokens ||
      (max_draft_len > 0 && !draft_tokens))
    return SV_ERR_INVALID;
  AcceptParams p = {sampled,  draft_tokens, parents,       draft_len,    row0,
                    draft_row0, n_rows,     n_drafts,      B,            max_draft_len,
                    accepted_len, out_tokens, correction_token, path,    out_ld,
                    ld_path,  status,       false};
  // one cluster as far as it goes, then CTAs of four
  const int warps = B <= 32 * kOneCluster ? (B + kOneCluster - 1) / kOneCluster : 4;
  return launch_round(accept_kernel, (B + int64_t(warps) - 1) / warps, 32u * unsigned(warps), s, p);
}

extern "C" sv_status spec_cache_keep(const int32_t* accepted_len, const int32_t* path,
                                     int64_t ld_path, int32_t n_path, int32_t B,
                                     const int32_t* ctx_len, const int32_t* page_table,
                                     int64_t ld_pages, int32_t max_pages, void* k_cache,
                                     void* v_cache, int32_t n_layers, int64_t layer_stride,
                                     int64_t n_pages, int32_t page_size, int64_t page_stride,
                                     int64_t token_stride, int64_t head_stride, int32_t n_kv_heads,
                                     int32_t D, int32_t* new_len, int32_t* status, void* stream) {
  if (!round_sizes_ok(0, 1, B, 0, ld_pages, max_pages, n_pages, page_size)) return SV_ERR_INVALID;
  if (n_path < 0 || (path && ld_path < n_path) || n_layers < 0 || n_kv_heads < 1 || D < 1)
    return SV_ERR_INVALID;
  if (n_path >= SV_MAX_TREE_ROWS && path) return SV_ERR_UNSUPPORTED;
  if (new_len && (new_len == ctx_len || new_len == accepted_len)) return SV_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0) return reset_status(status, s);
  if (!accepted_len || !ctx_len || (!page_table && max_pages > 0)) return SV_ERR_INVALID;
  if (path && n_layers > 0 && (!k_cache || !v_cache)) return SV_ERR_INVALID;
  if (D % 8 || D > (1 << 16) || n_kv_heads > (1 << 12)) return SV_ERR_UNSUPPORTED;
  if (path && (!aligned_bf16(k_cache, page_stride, token_stride, head_stride) ||
               !aligned16(v_cache) || layer_stride % 8))
    return SV_ERR_UNSUPPORTED;
  KeepParams p = {};
  p.rd.ctx_len = ctx_len, p.rd.page_table = page_table, p.rd.ld_pages = ld_pages;
  p.rd.max_pages = max_pages, p.rd.n_pages = n_pages, p.rd.page_size = page_size, p.rd.B = B;
  p.cache = {static_cast<__nv_bfloat16*>(k_cache), static_cast<__nv_bfloat16*>(v_cache),
             page_stride, token_stride, head_stride};
  p.accepted_len = accepted_len, p.path = path, p.ld_path = ld_path, p.n_path = n_path;
  // (a chain moves nothing: its lengths are one layer's work)
  p.n_layers = path ? n_layers : 1, p.layer_stride = layer_stride;
  p.columns = n_kv_heads * (D / 8), p.head_columns = D / 8;
  p.new_len = new_len, p.status = status;
  if (p.n_layers == 0) p.path = nullptr;
  p.n_layers = std::max(p.n_layers, 1);
  // several layers a CTA once there are CTAs enough: what it finds out first is the same for all
  if (int64_t(p.n_layers) * B > int64_t(INT32_MAX)) return SV_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms < 1) return SV_ERR_CUDA;
  p.layers = int32_t(std::max<int64_t>(1, int64_t(p.n_layers) * B / (kKeepCtas * sms)));
  return launch_round(keep_kernel, int64_t((p.n_layers + p.layers - 1) / p.layers) * B, kKeepThreads, s,
                      p);
}
