// process.cu -- penalties, logit biases and grammar masks on the logits of a speculative round
// (spec_process_logits).
//
// Row i of request r is conditioned on the request's history and on its first i drafted tokens.
// With n(v) the number of times v was emitted (counts[slot][v] plus its occurrences among those i
// tokens), for every token v:
//   l = seen(v) ? (l > 0 ? l / repetition : l * repetition) : l     seen: in the prompt, or n > 0
//   l = l - frequency * n - (n > 0 ? presence : 0)
//   l = l + bias(v)
//   l = allowed(v) ? l : -inf
// computed in binary32 and rounded once to the logits' type.  An element that nothing touches is
// left (or copied) bit for bit.
#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {
namespace {

struct ProcParams {
  const uint8_t* logits;
  int64_t ld;
  uint8_t* out;
  int64_t ld_out;
  int64_t V;
  const int64_t* row0;
  const int64_t* draft_row0;
  const int32_t* draft_len;
  int32_t gmax, first_row, bonus_row;
  const int32_t* draft_tokens;
  int32_t chunks;
  const int32_t* slots;
  int32_t n_slots;
  const int32_t* counts;
  int64_t ld_counts;
  const uint8_t* prompt_bits;
  const uint8_t* output_bits;
  int64_t ld_bits;  // bytes
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_start;
  const int32_t* bias_tokens;
  const float* bias_values;
  int64_t n_bias;
  const uint8_t* mask;
  int64_t ld_mask;  // bytes
  int32_t n_mask;
  const int32_t* mask_row;
  int32_t* status;
};

constexpr int kProcThreads = 256;
constexpr int kProcRows = 4;  // rows whose loads are in flight together

template <typename E>
struct ProcElem;

template <>
struct ProcElem<float> {
  static constexpr int kBytes = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  __device__ static __forceinline__ float get(const uint4& v, int j) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return __uint_as_float(w[j]);
  }
  __device__ static __forceinline__ void put(uint4& v, int j, float y) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    w[j] = __float_as_uint(y);
  }
};

template <>
struct ProcElem<bf16_tag> {
  static constexpr int kBytes = 2;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  __device__ static __forceinline__ float get(const uint4& v, int j) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
  }
  __device__ static __forceinline__ void put(uint4& v, int j, float y) {
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    w[j >> 1] = (j & 1) ? ((w[j >> 1] & 0xFFFFu) | (h << 16)) : ((w[j >> 1] & 0xFFFF0000u) | h);
  }
};

// The kVec bits of tokens v0 .. v0 + kVec - 1 (v0 a multiple of kVec) of a bit row.
template <int kVec>
__device__ __forceinline__ uint32_t bits_of(const uint8_t* row, int64_t v0) {
  const uint32_t b = __ldg(row + (v0 >> 3));
  return kVec == 8 ? b : (b >> (v0 & 4)) & 0xFu;
}

// One CTA per (request, chunk of kProcThreads vectors); a thread owns one 16-byte vector of the
// vocabulary in every row of the request, so history, counts and biases are read once for all of
// them.  In place, a vector that nothing touches costs two bytes of bits and no logit traffic.
template <typename E, bool kInPlace>
__global__ void __launch_bounds__(kProcThreads) process_kernel(ProcParams p) {
  using X = ProcElem<E>;
  constexpr int kVec = 16 / X::kBytes;
  constexpr int kChunk = kProcThreads * kVec;
  __shared__ int32_t s_tok[SV_MAX_DRAFT_LEN], s_pos[SV_MAX_DRAFT_LEN];
  __shared__ int32_t s_n;
  __shared__ float s_bias[kChunk];
  __shared__ uint32_t s_bbits[kChunk / 32];
  const int32_t r = blockIdx.x / p.chunks;
  const int32_t c = blockIdx.x % p.chunks;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t lo = int64_t(c) * kChunk;
  const bool first = c == 0 && tid == 0;  // reports what does not depend on the chunk

  int32_t g = p.draft_len[r];
  if (g < 0 || g > p.gmax) {
    if (first) report(p.status, SV_ERR_BAD_INPUT);
    g = g < 0 ? 0 : p.gmax;
  }
  const int32_t rows = g + p.bonus_row;
  const float theta = p.repetition ? p.repetition[r] : 1.f;
  const float pres = p.presence ? p.presence[r] : 0.f;
  const float freq = p.frequency ? p.frequency[r] : 0.f;
  bool pen = theta != 1.f || pres != 0.f || freq != 0.f;
  int32_t slot = 0;
  if (pen) {
    slot = p.slots ? p.slots[r] : r;
    const bool ok = theta > 0.f && theta < INFINITY && fabsf(pres) < INFINITY &&
                    fabsf(freq) < INFINITY && slot >= 0 && slot < p.n_slots;
    if (!ok) {
      if (first) report(p.status, SV_ERR_BAD_INPUT);
      pen = false;
    }
  }
  int64_t b0 = 0, b1 = 0;
  if (p.bias_start) {
    b0 = p.bias_start[r];
    b1 = p.bias_start[r + 1];
    if (b0 < 0 || b1 < b0 || b1 > p.n_bias) {
      if (first) report(p.status, SV_ERR_BAD_INPUT);
      b1 = b0 = 0;
    }
  }

  // ---- the drafted tokens and the biases of this chunk
  if (tid == 0) s_n = 0;
  if (tid < kChunk / 32) s_bbits[tid] = 0;
  __syncthreads();
  if (pen && tid < 32 && g > 0) {
    const int64_t d0 = p.draft_row0[r];
    int n = 0;
    for (int32_t k0 = 0; k0 < g; k0 += 32) {
      const int32_t k = k0 + lane;
      const int32_t x = k < g ? p.draft_tokens[d0 + k] : -1;
      if (k < g && (x < 0 || x >= p.V)) report(p.status, SV_ERR_BAD_INPUT);
      const bool in = k < g && x >= lo && x < lo + kChunk && x < p.V;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (in) {
        const int at = n + __popc(m & ((1u << lane) - 1u));
        s_tok[at] = static_cast<int32_t>(x - lo);
        s_pos[at] = k + 1;
      }
      n += __popc(m);
    }
    if (lane == 0) s_n = n;
  }
  for (int64_t k = b0 + tid; k < b1; k += kProcThreads) {
    const int32_t x = p.bias_tokens[k];
    if (c == 0 && (x < 0 || x >= p.V || (k > b0 && p.bias_tokens[k - 1] >= x)))
      report(p.status, SV_ERR_BAD_INPUT);
    if (x >= lo && x < lo + kChunk) {
      s_bias[x - lo] = p.bias_values[k];
      atomicOr(&s_bbits[(x - lo) >> 5], 1u << ((x - lo) & 31));
    }
  }
  __syncthreads();

  const int64_t v0 = lo + int64_t(tid) * kVec;
  if (v0 >= p.V) return;
  const uint32_t valid = p.V - v0 >= kVec ? (1u << kVec) - 1u : (1u << (p.V - v0)) - 1u;
  const bool whole = valid == (1u << kVec) - 1u;
  uint32_t emitted = 0, seen = 0;
  int32_t cnt[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) cnt[j] = 0;
  if (pen) {
    emitted = bits_of<kVec>(p.output_bits + slot * p.ld_bits, v0) & valid;
    seen = (bits_of<kVec>(p.prompt_bits + slot * p.ld_bits, v0) & valid) | emitted;
    if (emitted) {
      const int32_t* cr = p.counts + slot * p.ld_counts + v0;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (emitted >> j & 1u) cnt[j] = __ldg(cr + j);
    }
  }
  const uint32_t biased =
      (s_bbits[(tid * kVec) >> 5] >> ((tid * kVec) & 31)) & ((1u << kVec) - 1u);
  const int n_draft = s_n;
  int next = 0;       // drafted tokens of the chunk already counted
  int next_bits = 0;  // the same, for the bits only (they run ahead with the loads)
  uint32_t touched = seen | biased;

  const int64_t row = p.row0[r];
  for (int32_t i0 = p.first_row; i0 < rows; i0 += kProcRows) {
    uint4 x[kProcRows];
    uint32_t ok[kProcRows], act[kProcRows];
#pragma unroll
    for (int u = 0; u < kProcRows; ++u) {
      const int32_t i = i0 + u;
      ok[u] = valid;
      act[u] = 0;
      if (i >= rows) continue;
      if (p.mask_row) {
        const int32_t m = p.mask_row[row + i];
        if (m >= p.n_mask || m < -1) {
          if (first) report(p.status, SV_ERR_BAD_INPUT);
        } else if (m >= 0) {
          ok[u] = bits_of<kVec>(p.mask + m * p.ld_mask, v0) & valid;
        }
      }
      while (next_bits < n_draft && s_pos[next_bits] <= i) {
        const uint32_t j = static_cast<uint32_t>(s_tok[next_bits++] - tid * kVec);
        if (j < uint32_t(kVec)) touched |= 1u << j;
      }
      act[u] = (touched & ok[u]) | (valid & ~ok[u]);
      if ((!kInPlace || act[u]) && (ok[u] || !whole)) {
        const uint8_t* src = p.logits + ((row + i) * p.ld + v0) * X::kBytes;
        if (whole) {
          x[u] = kInPlace ? *reinterpret_cast<const uint4*>(src)
                          : __ldg(reinterpret_cast<const uint4*>(src));
        } else {
          x[u] = make_uint4(0, 0, 0, 0);
          for (int j = 0; j < kVec; ++j)
            if (valid >> j & 1u) {
              if constexpr (X::kBytes == 4)
                X::put(x[u], j, reinterpret_cast<const float*>(src)[j]);
              else
                reinterpret_cast<uint16_t*>(&x[u])[j] = reinterpret_cast<const uint16_t*>(src)[j];
            }
        }
      } else {
        x[u] = make_uint4(X::kNegInf, X::kNegInf, X::kNegInf, X::kNegInf);
      }
    }
#pragma unroll
    for (int u = 0; u < kProcRows; ++u) {
      const int32_t i = i0 + u;
      if (i >= rows) continue;
      while (next < n_draft && s_pos[next] <= i) {
        const uint32_t j = static_cast<uint32_t>(s_tok[next++] - tid * kVec);
        if (j < uint32_t(kVec)) {
          emitted |= 1u << j;
          seen |= 1u << j;
#pragma unroll
          for (int q = 0; q < kVec; ++q)
            if (uint32_t(q) == j) ++cnt[q];
        }
      }
      if (kInPlace && !act[u]) continue;
      if (act[u]) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (!(act[u] >> j & 1u)) continue;
          float y = X::get(x[u], j);
          if (seen >> j & 1u) y = y > 0.f ? __fdiv_rn(y, theta) : y * theta;
          if (emitted >> j & 1u) y = y - freq * static_cast<float>(cnt[j]) - pres;
          if (biased >> j & 1u) y += s_bias[tid * kVec + j];
          if (!(ok[u] >> j & 1u)) y = -INFINITY;
          X::put(x[u], j, y);
        }
      }
      uint8_t* dst = p.out + ((row + i) * p.ld_out + v0) * X::kBytes;
      if (whole) {
        *reinterpret_cast<uint4*>(dst) = x[u];
      } else {
        for (int j = 0; j < kVec; ++j)
          if (valid >> j & 1u) {
            if constexpr (X::kBytes == 4)
              reinterpret_cast<uint32_t*>(dst)[j] = reinterpret_cast<const uint32_t*>(&x[u])[j];
            else
              reinterpret_cast<uint16_t*>(dst)[j] = reinterpret_cast<const uint16_t*>(&x[u])[j];
          }
      }
    }
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status spec_process_logits(
    const void* logits, int64_t ld, void* out, int64_t ld_out, sv_dtype dtype, int64_t V,
    const int64_t* row0, const int64_t* draft_row0, const int32_t* draft_len,
    int32_t max_draft_len, int32_t first_row, int32_t bonus_row, const int32_t* draft_tokens,
    int32_t B, const int32_t* slots, int32_t n_slots, const int32_t* counts, int64_t ld_counts,
    const uint32_t* prompt_bits, const uint32_t* output_bits, int64_t ld_bits,
    const float* repetition, const float* presence, const float* frequency,
    const int32_t* bias_start, const int32_t* bias_tokens, const float* bias_values,
    int64_t n_bias, const uint32_t* mask, int64_t ld_mask, int32_t n_mask,
    const int32_t* mask_row, int32_t* status, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID;
  if (B < 0 || V < 1 || max_draft_len < 0 || max_draft_len > SV_MAX_DRAFT_LEN || ld < V ||
      ld_out < V || first_row < 0 || (bonus_row != 0 && bonus_row != 1))
    return SV_ERR_INVALID;
  if (!logits || !out || (out == logits && ld_out != ld)) return SV_ERR_INVALID;
  if (V > INT32_MAX - 4096) return SV_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned16(logits) || !aligned16(out) || (ld * eb) % 16 || (ld_out * eb) % 16)
    return SV_ERR_UNSUPPORTED;
  if (B == 0) return SV_OK;
  if (!row0 || !draft_len) return SV_ERR_INVALID;
  if (repetition || presence || frequency) {
    if (!counts || !prompt_bits || !output_bits || n_slots < 1 || ld_counts < V ||
        ld_bits < (V + 31) / 32)
      return SV_ERR_INVALID;
    if (max_draft_len > 0 && (!draft_tokens || !draft_row0)) return SV_ERR_INVALID;
  }
  if (bias_start && (n_bias < 0 || (n_bias > 0 && (!bias_tokens || !bias_values))))
    return SV_ERR_INVALID;
  if (mask_row && (n_mask < 0 || (n_mask > 0 && (!mask || ld_mask < (V + 31) / 32))))
    return SV_ERR_INVALID;
  const int64_t chunk = int64_t(kProcThreads) * (16 / eb);
  const int64_t chunks = (V + chunk - 1) / chunk;
  if (chunks * B > INT32_MAX) return SV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, sizeof(int32_t), s) != cudaSuccess) return SV_ERR_CUDA;
  const ProcParams p = {static_cast<const uint8_t*>(logits),
                        ld,
                        static_cast<uint8_t*>(out),
                        ld_out,
                        V,
                        row0,
                        draft_row0,
                        draft_len,
                        max_draft_len,
                        first_row,
                        bonus_row,
                        draft_tokens,
                        int32_t(chunks),
                        slots,
                        n_slots,
                        counts,
                        ld_counts,
                        reinterpret_cast<const uint8_t*>(prompt_bits),
                        reinterpret_cast<const uint8_t*>(output_bits),
                        ld_bits * 4,
                        repetition,
                        presence,
                        frequency,
                        bias_start,
                        bias_tokens,
                        bias_values,
                        n_bias,
                        reinterpret_cast<const uint8_t*>(mask),
                        ld_mask * 4,
                        n_mask,
                        mask_row,
                        status};
  const unsigned grid = unsigned(chunks * B);
  const bool in_place = out == logits;
  if (dtype == SV_BF16) {
    if (in_place)
      process_kernel<bf16_tag, true><<<grid, kProcThreads, 0, s>>>(p);
    else
      process_kernel<bf16_tag, false><<<grid, kProcThreads, 0, s>>>(p);
  } else {
    if (in_place)
      process_kernel<float, true><<<grid, kProcThreads, 0, s>>>(p);
    else
      process_kernel<float, false><<<grid, kProcThreads, 0, s>>>(p);
  }
  return launch_status(cudaGetLastError());
}
