// tree_attention.cu -- attention of a round's rows over the paged cache (spec_tree_attention).
//
// A CTA per (row, query head): its warps share the keys out, each keeps a running maximum, sum and
// output, and they are joined at the end.
#include "round.cuh"

#include <cmath>

namespace sv {
namespace {

struct AttnParams {
  RoundParams rd;
  CacheParams cache;
  const __nv_bfloat16* q;
  int64_t ldq, q_head;
  int32_t n_heads, group, D;
  float scale2;  // scale * log2(e)
  __nv_bfloat16* out;
  int64_t ldo, o_head;
  float* lse;
  int64_t ld_lse;
  int32_t* status;
};

constexpr int kAttnWarps = 4;

template <int kD>
__global__ void __launch_bounds__(32 * kAttnWarps) attention_kernel(AttnParams p, int32_t max_rows) {
  constexpr int kE = kD / 32;
  __shared__ uint32_t seen[SV_MAX_TREE_ROWS / 32];
  __shared__ float part[kAttnWarps][kD + 2];
  dependent_start();
  const int32_t h = blockIdx.x % p.n_heads, i = blockIdx.x / p.n_heads % max_rows;
  const int32_t r = blockIdx.x / p.n_heads / max_rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Request rq;
  if (!round_request(p.rd, r, rq)) {
    if (i == 0 && h == 0 && threadIdx.x == 0) report(p.status, SV_ERR_BAD_INPUT);
    return;
  }
  if (i >= rq.n) return;
  if (p.rd.parents && threadIdx.x == 0) {
    for (int w = 0; w < SV_MAX_TREE_ROWS / 32; ++w) seen[w] = 0;
    for (int32_t j = i; j >= 0;) {
      seen[j >> 5] |= 1u << (j & 31);
      int32_t up = p.rd.parents[rq.first + j];
      if (up < -1 || up >= j) {
        report(p.status, SV_ERR_BAD_INPUT);
        up = -1;
      }
      j = up;
    }
  }
  __syncthreads();
  const int64_t row = rq.first + i;
  float q[kE], o[kE] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < kE; ++e)
    q[e] = __bfloat162float(p.q[row * p.ldq + h * p.q_head + lane + 32 * e]) * p.scale2;
  for (int32_t j = warp; j <= rq.ctx + i; j += kAttnWarps) {
    if (j >= rq.ctx && p.rd.parents) {
      const int32_t t = j - rq.ctx;
      if (!(seen[t >> 5] >> (t & 31) & 1u)) continue;
    }
    const int32_t page = round_page(p.rd, r, j);
    if (page < 0) {
      if (lane == 0) report(p.status, SV_ERR_BAD_INPUT);
      continue;
    }
    const int64_t at = page * p.cache.page_stride + (j % p.rd.page_size) * p.cache.token_stride +
                       (h / p.group) * p.cache.head_stride;
    float x = 0.f;
    for (int e = 0; e < kE; ++e) x += q[e] * __bfloat162float(p.cache.k[at + lane + 32 * e]);
    x = warp_sum(x);
    const float mn = fmaxf(m, x);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(x - (mn == -INFINITY ? 0.f : mn));  // NaN stays
    l = l * f + w;
    for (int e = 0; e < kE; ++e)
      o[e] = o[e] * f + w * __bfloat162float(p.cache.v[at + lane + 32 * e]);
    m = mn;
  }
  for (int e = 0; e < kE; ++e) part[warp][lane + 32 * e] = o[e];
  if (lane == 0) part[warp][kD] = m, part[warp][kD + 1] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, part[w][kD]);
  for (int d = threadIdx.x; d < kD; d += 32 * kAttnWarps) {
    float y = 0.f;
    sum = 0.f;
    for (int w = 0; w < kAttnWarps; ++w) {
      const float f = part[w][kD] == -INFINITY ? 0.f : exp2f(part[w][kD] - top);
      y += f * part[w][d];
      sum += f * part[w][kD + 1];
    }
    p.out[row * p.ldo + h * p.o_head + d] = __float2bfloat16_rn(sum == 0.f ? 0.f : y / sum);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[row * p.ld_lse + h] = (top + log2f(sum)) * kLn2;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_tree_attention_workspace_bytes(int32_t B, int32_t max_draft_len,
                                                      int32_t bonus_row, int32_t n_heads,
                                                      int32_t n_kv_heads, int32_t D) {
  if (B < 0 || max_draft_len < 0 || bonus_row < 0 || bonus_row > 1 || n_heads < 1 ||
      n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 128 ||
      (D != 64 && D != 128))
    return 0;
  return 256;
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
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || D < 1 || !std::isfinite(scale) ||
      (lse && ld_lse < n_heads))
    return SV_ERR_INVALID;
  if (parents && max_draft_len + int64_t(bonus_row) > SV_MAX_TREE_ROWS) return SV_ERR_UNSUPPORTED;
  if ((D != 64 && D != 128) || n_heads / n_kv_heads > 128 || page_size < 8 ||
      (page_size & (page_size - 1)))
    return SV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || max_draft_len + bonus_row == 0 || n_rows == 0) return reset_status(status, s);
  if (!q || !out || !k_cache || !v_cache || !row0 || !draft_len || !ctx_len || !page_table ||
      !workspace)
    return SV_ERR_INVALID;
  if (!aligned_bf16(q, ldq, q_head, 0) || !aligned_bf16(out, ldo, o_head, 0) ||
      !aligned_bf16(k_cache, page_stride, token_stride, head_stride) || !aligned16(v_cache) ||
      !aligned256(workspace))
    return SV_ERR_UNSUPPORTED;
  if (workspace_bytes < spec_tree_attention_workspace_bytes(B, max_draft_len, bonus_row, n_heads,
                                                            n_kv_heads, D))
    return SV_ERR_INVALID;
  AttnParams p = {};
  p.rd = {row0,    draft_len, parents,       ctx_len,   page_table, ld_pages, n_rows,
          n_pages, B,         max_draft_len, bonus_row, max_pages,  page_size};
  p.cache = {static_cast<__nv_bfloat16*>(const_cast<void*>(k_cache)),
             static_cast<__nv_bfloat16*>(const_cast<void*>(v_cache)), page_stride, token_stride,
             head_stride};
  p.q = static_cast<const __nv_bfloat16*>(q), p.ldq = ldq, p.q_head = q_head;
  p.n_heads = n_heads, p.group = n_heads / n_kv_heads, p.D = D;
  p.scale2 = scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(out), p.ldo = ldo, p.o_head = o_head;
  p.lse = lse, p.ld_lse = ld_lse, p.status = status;
  const int64_t blocks = int64_t(n_heads) * (max_draft_len + int64_t(bonus_row)) * B;
  if (blocks > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const sv_status st = reset_status(status, s);
  if (st != SV_OK) return st;
  return launch_dependent(D == 64 ? attention_kernel<64> : attention_kernel<128>, unsigned(blocks),
                          32 * kAttnWarps, 0, s, p, max_draft_len + bonus_row);
}
