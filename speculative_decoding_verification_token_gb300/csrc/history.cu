// history.cu -- the token history that penalties are computed from (spec_history_append).
//
// State of a slot: how often each token was emitted (counts), and two bit rows, token v in bit
// v % 32 of word v / 32: the tokens of the prompt and the tokens emitted (set exactly where the
// count is positive).  Appending adds integers and sets bits, so the result does not depend on the
// order in which the atomics land.
#include "dependent.cuh"

namespace sv {
namespace {

struct HistParams {
  const int32_t* tokens;
  int64_t ld_tokens;
  const int32_t* lens;
  int32_t n;
  const int32_t* slots;
  int32_t B;
  int32_t prompt;
  int64_t V;
  int32_t n_slots;
  int32_t* counts;
  int64_t ld_counts;
  uint32_t* prompt_bits;
  uint32_t* output_bits;
  int64_t ld_bits;
  int32_t* status;
  bool one_row;  // reset = 1 with one row
};

constexpr int kHistThreads = 256;  // of a CTA, where there are several

// Row r's slot and number of columns; a bad value of either is reported and leaves the row alone.
__device__ __forceinline__ bool hist_row(const HistParams& p, int32_t r, int32_t* status,
                                         int32_t& slot, int32_t& n) {
  slot = p.slots ? p.slots[r] : r;
  n = p.lens ? p.lens[r] : p.n;
  if (slot < 0 || slot >= p.n_slots || n < 0 || n > p.n) {
    report(status, SV_ERR_BAD_INPUT);
    return false;
  }
  return true;
}

// Where a CTA that clears reports.  Of a single row's CTAs the first, which sees all there is to
// report, resets the status and reports: that saves the call a launch (100 tokens, V = 32000: 4.1 ->
// 2.8 us).
__device__ __forceinline__ int32_t* reset_reports(const HistParams& p, int32_t c) {
  if (!p.one_row || !p.status) return p.status;
  if (c != 0) return nullptr;
  if (threadIdx.x == 0) *p.status = 0;
  __syncthreads();
  return p.status;
}

// One thread per token: a round appends a few hundred, so the call is one launch of one or two
// dependent loads and two atomics, and the launch is what it costs (64 x 6 tokens: 2.5 us a call in
// a loop, host time included).  A single CTA (one = true) resets the status itself, which saves the
// short call a second launch.
__global__ void __launch_bounds__(1024) history_append_kernel(HistParams p, bool one) {
  dependent_start();
  if (one) {
    if (threadIdx.x == 0 && p.status) *p.status = 0;
    __syncthreads();
  }
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= int64_t(p.B) * p.n) return;
  const int32_t r = static_cast<int32_t>(i / p.n);
  const int32_t t = static_cast<int32_t>(i % p.n);
  const int32_t x = p.tokens[r * p.ld_tokens + t];
  int32_t slot, n;
  if (!hist_row(p, r, p.status, slot, n) || t >= n) return;
  if (x < 0) return;  // padding
  if (x >= p.V) {
    report(p.status, SV_ERR_BAD_INPUT);
    return;
  }
  uint32_t* word = (p.prompt ? p.prompt_bits : p.output_bits) + slot * p.ld_bits + (x >> 5);
  atomicOr(word, 1u << (x & 31));
  if (!p.prompt) atomicAdd(p.counts + slot * p.ld_counts + x, 1);
}

constexpr int kResetThreads = 256;
constexpr int kResetWords = 256;  // 32-token words of a slot that one CTA owns
constexpr int kResetAhead = 8;    // tokens a thread has in flight

// Clear, then append emitted tokens (prompts: history_prompt_kernel): each CTA owns kResetWords words
// of one slot and the counts below them, so the two steps need no order between CTAs.  It clears its
// counts, reads the row's tokens (at most a few tens of KB, from L2 for all CTAs of a slot but the
// first) and keeps those in its range.
__global__ void __launch_bounds__(kResetThreads) history_reset_kernel(HistParams p,
                                                                      int32_t chunks) {
  __shared__ uint32_t s_bits[kResetWords];
  dependent_start();
  const int32_t r = blockIdx.x / chunks;
  const int32_t c = blockIdx.x % chunks;
  const int tid = threadIdx.x;
  int32_t* const status = reset_reports(p, c);
  int32_t slot, n;
  if (!hist_row(p, r, status, slot, n)) return;  // the whole CTA
  const int32_t* row = p.tokens + r * p.ld_tokens;
  int32_t x[kResetAhead];
  auto fetch = [&](int32_t t0) {
#pragma unroll
    for (int q = 0; q < kResetAhead; ++q) {
      const int32_t t = t0 + tid + q * kResetThreads;
      x[q] = t < n ? row[t] : -1;
    }
  };
  fetch(0);
  int32_t twice = 0;
  if (p.slots)
    for (int32_t q = tid; q < p.B; q += kResetThreads) twice |= q != r && p.slots[q] == slot;
  static_assert(kResetWords == kResetThreads, "a word per thread");
  s_bits[tid] = 0;
  if (__syncthreads_or(twice)) {  // two rows would clear and fill the same slot
    if (tid == 0) report(status, SV_ERR_BAD_INPUT);
    return;
  }
  const int64_t w0 = int64_t(c) * kResetWords;
  const int64_t v0 = w0 * 32, v1 = min(p.V, v0 + int64_t(kResetWords) * 32);
  int32_t* cnt = p.counts + slot * p.ld_counts;
  if ((reinterpret_cast<uintptr_t>(cnt) & 15u) == 0) {
    const int64_t full = v1 & ~int64_t(3);
    for (int64_t v = v0 + 4 * tid; v < full; v += 4 * kResetThreads)
      *reinterpret_cast<int4*>(cnt + v) = make_int4(0, 0, 0, 0);
    for (int64_t v = full + tid; v < v1; v += kResetThreads) cnt[v] = 0;
  } else {
    for (int64_t v = v0 + tid; v < v1; v += kResetThreads) cnt[v] = 0;
  }
  __syncthreads();  // the counts are zero before this CTA's atomics reach them
  for (int32_t t0 = 0; t0 < n; t0 += kResetAhead * kResetThreads) {
    if (t0) fetch(t0);
#pragma unroll
    for (int q = 0; q < kResetAhead; ++q) {
      if (x[q] >= p.V) report(status, SV_ERR_BAD_INPUT);
      if (x[q] < v0 || x[q] >= v1) continue;
      const uint32_t b = 1u << (x[q] & 31);
      uint32_t* word = &s_bits[(x[q] - v0) >> 5];
      if (!(*reinterpret_cast<volatile uint32_t*>(word) & b)) atomicOr(word, b);
      atomicAdd(cnt + x[q], 1);
    }
  }
  __syncthreads();
  if (w0 + tid < (p.V + 31) / 32) {
    p.prompt_bits[slot * p.ld_bits + w0 + tid] = 0u;
    p.output_bits[slot * p.ld_bits + w0 + tid] = s_bits[tid];
  }
}

constexpr int kPromptThreads = 1024;
constexpr int kPromptWords = 8192;   // words of prompt bits one CTA collects: 262144 tokens
constexpr int kPromptAhead = 8;      // tokens a thread has in flight
constexpr int kClearTokens = 16384;  // counts one CTA clears

// A slot's history replaced by a prompt.  The prompt touches no counts, so clearing them and
// collecting the tokens need no order: of each slot's CTAs the first `marks` read the tokens, once,
// and write the bit rows whole, the others clear 64 KB of counts each.  32 prompts of up to 8192
// tokens, V = 129280: 6.3 us a call, of which the 18 MB written would take 2.7; the rest is the two
// launches and the CTAs that mark, whose 32 warps compete for their SM's issue slots ("not selected"
// leads the stalls, then the tokens' latency; with the kernel above, whose CTAs each read all tokens,
// 9.5).
__global__ void __launch_bounds__(kPromptThreads) history_prompt_kernel(HistParams p,
                                                                        int32_t marks,
                                                                        int32_t ctas) {
  __shared__ uint32_t s_bits[kPromptWords];
  dependent_start();
  const int32_t r = blockIdx.x / ctas;
  const int32_t c = blockIdx.x % ctas;
  const int tid = threadIdx.x;
  int32_t* const status = reset_reports(p, c);
  const int32_t* row = p.tokens + r * p.ld_tokens;
  int32_t x[kPromptAhead];
  auto fetch = [&](int32_t t0) {
#pragma unroll
    for (int q = 0; q < kPromptAhead; ++q) {
      const int32_t t = t0 + tid + q * kPromptThreads;
      x[q] = t < p.n ? row[t] : -1;
    }
  };
  if (c < marks) fetch(0);  // beside the row's slot and length; columns behind the length are dropped
  int32_t slot, n;
  if (!hist_row(p, r, status, slot, n)) return;  // the whole CTA
  int32_t twice = 0;
  if (p.slots)
    for (int32_t q = tid; q < p.B; q += kPromptThreads) twice |= q != r && p.slots[q] == slot;
  if (c >= marks) {
    if (__syncthreads_or(twice)) return;
    const int64_t v0 = int64_t(c - marks) * kClearTokens, v1 = min(p.V, v0 + kClearTokens);
    int32_t* cnt = p.counts + slot * p.ld_counts;
    const int64_t full = (reinterpret_cast<uintptr_t>(cnt) & 15u) ? v0 : v1 & ~int64_t(3);
    for (int64_t v = v0 + 4 * tid; v < full; v += 4 * kPromptThreads)
      *reinterpret_cast<int4*>(cnt + v) = make_int4(0, 0, 0, 0);
    for (int64_t v = full + tid; v < v1; v += kPromptThreads) cnt[v] = 0;
    return;
  }
  const int64_t w0 = int64_t(c) * kPromptWords;
  const int32_t words =
      static_cast<int32_t>(min(int64_t(kPromptWords), (p.V + 31) / 32 - w0));
  const int64_t v0 = w0 * 32, v1 = min(p.V, v0 + int64_t(kPromptWords) * 32);
  for (int w = tid; w < words; w += kPromptThreads) s_bits[w] = 0;
  if (__syncthreads_or(twice)) {
    if (tid == 0) report(status, SV_ERR_BAD_INPUT);
    return;
  }
  for (int32_t t0 = 0; t0 < n; t0 += kPromptAhead * kPromptThreads) {
    if (t0) fetch(t0);
#pragma unroll
    for (int q = 0; q < kPromptAhead; ++q) {
      if (t0 + tid + q * kPromptThreads >= n) continue;
      if (x[q] >= p.V) report(status, SV_ERR_BAD_INPUT);
      if (x[q] < v0 || x[q] >= v1) continue;
      const uint32_t b = 1u << (x[q] & 31);
      uint32_t* word = &s_bits[(x[q] - v0) >> 5];
      if (!(*reinterpret_cast<volatile uint32_t*>(word) & b)) atomicOr(word, b);  // often there
    }
  }
  __syncthreads();
  uint32_t* pb = p.prompt_bits + slot * p.ld_bits + w0;
  uint32_t* ob = p.output_bits + slot * p.ld_bits + w0;
  for (int w = tid; w < words; w += kPromptThreads) {
    pb[w] = s_bits[w];
    ob[w] = 0;
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status spec_history_append(const int32_t* tokens, int64_t ld_tokens,
                                         const int32_t* lens, int32_t n, const int32_t* slots,
                                         int32_t B, int32_t kind, int32_t reset, int64_t V,
                                         int32_t n_slots, int32_t* counts, int64_t ld_counts,
                                         uint32_t* prompt_bits, uint32_t* output_bits,
                                         int64_t ld_bits, int32_t* status, void* stream) {
  if (B < 0 || n < 0 || V < 1 || n_slots < 0 || ld_tokens < n || ld_counts < V ||
      ld_bits < (V + 31) / 32 || (kind != SV_HISTORY_OUTPUT && kind != SV_HISTORY_PROMPT) ||
      (reset != 0 && reset != 1))
    return SV_ERR_INVALID;
  if (V > INT32_MAX || n > INT32_MAX - 8192) return SV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || (n == 0 && !reset)) return reset_status(status, s);  // nothing else to do
  if ((n > 0 && !tokens) || !counts || !prompt_bits || !output_bits) return SV_ERR_INVALID;
  const bool fill = reset && kind == SV_HISTORY_PROMPT;
  const int64_t marks = ((V + 31) / 32 + kPromptWords - 1) / kPromptWords;
  const int64_t chunks = fill ? marks + (V + kClearTokens - 1) / kClearTokens
                              : ((V + 31) / 32 + kResetWords - 1) / kResetWords;
  const int64_t blocks =
      reset ? chunks * B : (int64_t(B) * n + kHistThreads - 1) / kHistThreads;
  if (blocks > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const bool one = !reset && int64_t(B) * n <= 1024, one_row = reset && B == 1;
  if (!one && !one_row) {
    const sv_status st = reset_status(status, s);
    if (st != SV_OK) return st;
  }
  const HistParams p = {tokens, ld_tokens, lens, n,         slots,       B,           kind,
                        V,      n_slots,   counts, ld_counts, prompt_bits, output_bits, ld_bits,
                        status, one_row};
  if (fill)
    return launch_dependent(history_prompt_kernel, unsigned(blocks), kPromptThreads, 0, s, p,
                            int32_t(marks), int32_t(chunks));
  if (reset)
    return launch_dependent(history_reset_kernel, unsigned(blocks), kResetThreads, 0, s, p,
                            int32_t(chunks));
  if (one)
    return launch_dependent(history_append_kernel, 1u, unsigned(B * n + 31) / 32 * 32, 0, s, p, true);
  return launch_dependent(history_append_kernel, unsigned(blocks), kHistThreads, 0, s, p, false);
}
