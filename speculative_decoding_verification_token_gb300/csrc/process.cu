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
#include <algorithm>

#include "dependent.cuh"

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
  int32_t chunks, splits;  // CTAs per request: chunks of the row times groups of rows
  int32_t group_rows;
  const int32_t* slots;
  int32_t n_slots;
  const int32_t* counts;
  int64_t ld_counts;
  const uint32_t* prompt_bits;
  const uint32_t* output_bits;
  int64_t ld_bits;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_start;
  const int32_t* bias_tokens;
  const float* bias_values;
  int64_t n_bias;
  const uint32_t* mask;
  int64_t ld_mask;
  int32_t n_mask;
  const int32_t* mask_row;
  int32_t* status;
  // Who resets the status and reports: each request's first CTA reports, after a kernel that resets
  // it; with kSingle the only request's first CTA does both; with kApart CTA 0, which does nothing
  // else, does both for all requests.
  int32_t reports;
};
enum { kFirst = 0, kSingle = 1, kApart = 2 };

constexpr int kProcThreads = 128;
constexpr int kProcRows = 4;  // rows handled together

// How a call moves its logits, and the bytes of a row that one CTA takes where there are many.
enum ProcMode {
  kCopy = 0,     // out of place: every row moves
  kMasked = 1,   // in place with masks: banned elements are written
  kSparse = 2    // in place without masks: only touched elements move
};
constexpr uint32_t proc_row_bytes(int mode) {
  return mode == kCopy ? 4096 : 8192;
}

constexpr uint32_t kSmallRowBytes = 1024;  // where there are few

template <typename E>
struct ProcElem;

template <>
struct ProcElem<float> {
  using T = float;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  __device__ static __forceinline__ float up(float x) { return x; }
  __device__ static __forceinline__ float down(float y) { return y; }
};

template <>
struct ProcElem<bf16_tag> {
  using T = uint16_t;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  __device__ static __forceinline__ float up(uint16_t h) {
    return __uint_as_float(uint32_t(h) << 16);
  }
  __device__ static __forceinline__ uint16_t down(float y) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
};

// Byte permutation whose selector nibbles 8 .. 11 spread the top bit of byte 0 .. 3 over a byte.
__device__ __forceinline__ uint32_t spread_sign(uint32_t x, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "r"(sel));
  return r;
}

// The elements of a 16-byte vector whose bit in `ok` is clear become -inf.  Four bits are multiplied
// to the tops of four bytes, one permutation makes a word's mask of them, one logic operation
// selects: 14 instructions a vector (testing bit by bit took about 40, and the masked rows were
// bound by them).
template <typename E>
__device__ __forceinline__ uint4 ban(uint4 x, uint32_t ok) {
  constexpr uint32_t kInf = ProcElem<E>::kNegInf;
  const uint32_t lo = ((ok & 0xFu) * 0x10204080u) & 0x80808080u;
  uint32_t m[4];
  if constexpr (sizeof(typename ProcElem<E>::T) == 4) {
    m[0] = spread_sign(lo, 0x8888u);
    m[1] = spread_sign(lo, 0x9999u);
    m[2] = spread_sign(lo, 0xAAAAu);
    m[3] = spread_sign(lo, 0xBBBBu);
  } else {
    const uint32_t hi = ((ok >> 4) * 0x10204080u) & 0x80808080u;
    m[0] = spread_sign(lo, 0x9988u);
    m[1] = spread_sign(lo, 0xBBAAu);
    m[2] = spread_sign(hi, 0x9988u);
    m[3] = spread_sign(hi, 0xBBAAu);
  }
  return make_uint4((x.x & m[0]) | (kInf & ~m[0]), (x.y & m[1]) | (kInf & ~m[1]),
                    (x.z & m[2]) | (kInf & ~m[2]), (x.w & m[3]) | (kInf & ~m[3]));
}

// All of a small call's requests checked by one CTA, a thread for each row and bias entry: saves the
// call the launch that would reset the status.
__device__ __forceinline__ void check_requests(const ProcParams& p, int32_t B, bool masked) {
  dependent_start();
  if (threadIdx.x == 0) *p.status = 0;
  bool bad = false;
  const int32_t per = p.gmax + 1;
  for (int32_t j = threadIdx.x; j < B * per; j += kProcThreads) {
    const int32_t i = j % per;
    const int32_t r = j / per, g = p.draft_len[r], slot = p.slots ? p.slots[r] : r;
    const float theta = p.repetition ? p.repetition[r] : 1.f;
    const float pres = p.presence ? p.presence[r] : 0.f;
    const float freq = p.frequency ? p.frequency[r] : 0.f;
    bool pen = theta != 1.f || pres != 0.f || freq != 0.f;
    if (pen && !(theta > 0.f && theta < INFINITY && fabsf(pres) < INFINITY &&
                 fabsf(freq) < INFINITY && slot >= 0 && slot < p.n_slots)) {
      bad = true;
      pen = false;
    }
    bad |= g < 0 || g > p.gmax;
    const int32_t drafts = min(max(g, 0), p.gmax);
    if (pen && i < drafts) {
      const int32_t x = p.draft_tokens[p.draft_row0[r] + i];
      bad |= x < 0 || x >= p.V;
    }
    if (masked && i >= p.first_row && i < drafts + p.bonus_row) {
      const int32_t m = p.mask_row[p.row0[r] + i];
      bad |= m < -1 || m >= p.n_mask;
    }
    if (p.bias_start) {
      const int32_t b0 = p.bias_start[r], b1 = p.bias_start[r + 1];
      bad |= b0 < 0 || b1 < b0 || b1 > p.n_bias;
    }
  }
  if (p.bias_start) {  // the lists follow one another: neighbours ascend unless a list starts there
    const int64_t k0 = max(int64_t(p.bias_start[0]), int64_t(0));
    const int64_t k1 = min(int64_t(p.bias_start[B]), p.n_bias);
    for (int64_t k = k0 + threadIdx.x; k < k1; k += kProcThreads) {
      const int32_t x = p.bias_tokens[k];
      bad |= x < 0 || x >= p.V;
      if (k > k0 && p.bias_tokens[k - 1] >= x) {
        int32_t r = 0;  // the first list that starts at k or behind it
        for (int32_t end = B; r < end;) {
          const int32_t mid = (r + end) >> 1;
          if (p.bias_start[mid] < k)
            r = mid + 1;
          else
            end = mid;
        }
        bad |= r == B || p.bias_start[r] != k;
      }
    }
  }
  __syncthreads();
  if (bad) report(p.status, SV_ERR_BAD_INPUT);
}

// One CTA per (request, chunk of a row), for all rows of the request: the history, biases
// and drafted tokens of the chunk are read once.  What they touch -- a few tokens in a hundred --
// is gathered into a list of offsets, one thread per listed token edits it in every row, and the
// rest of the logits moves (or, in place, does not move) without passing through a register:
//   out of place  bulk copies bring kProcRows row parts to shared memory, masks and edits work
//                 there, bulk copies take them to `out`;
//   in place      masks store -inf where they ban and edits touch single elements.
// Memory traffic bounds it where rows move: 384 rows of 151936 bf16 with histories of up to 2000
// tokens and 300 biases take 41.5 us, 5.7 TB/s of logits (without histories and biases 37); a CTA
// is a chain of four dependent loads (parameters; bits and tokens; counts and mask words; rows), so
// ten small CTAs an SM, four rows each time, do better than fewer with more rows (eight: 165 us for
// the 256 ragged requests that take 118).  In place it is sectors: a banned or edited element costs
// the 32 or 64 bytes around it, read and written, so that 512 masked rows of 129280 (2% allowed) and
// the edits of 512 others move 340 MB for 144 MB of elements: 62 us.
template <typename E, int kMode, uint32_t kRowBytes>
__global__ void __launch_bounds__(kProcThreads, 10)
    process_kernel(ProcParams p) {
  constexpr bool kInPlace = kMode != kCopy;
  using X = ProcElem<E>;
  using T = typename X::T;
  constexpr int kVec = 16 / sizeof(T);
  constexpr uint32_t kAll = (1u << kVec) - 1u;
  constexpr int kChunk = kRowBytes / sizeof(T);
  constexpr int kWords = kChunk / 32;
  constexpr int kOwn = (kWords + kProcThreads - 1) / kProcThreads;  // bit words per thread
  extern __shared__ __align__(128) uint8_t s_rows[];  // row parts, out of place
  __shared__ uint32_t s_mask[kMode == kSparse ? 1 : kProcRows][kWords];
  __shared__ uint16_t s_off[kChunk];
  __shared__ uint32_t s_touch[kWords], s_prompt[kWords], s_out[kWords], s_bbits[kWords],
      s_drafted[kWords];
  __shared__ int32_t s_tok[SV_MAX_DRAFT_LEN], s_pos[SV_MAX_DRAFT_LEN];
  __shared__ int32_t s_mrow[SV_MAX_DRAFT_LEN + 1];
  __shared__ int32_t s_n, s_nd;
  __shared__ uint32_t s_bias0;  // first entry of the bias list in this chunk, from b0
  __shared__ uint64_t s_bar;
  static_assert(kProcThreads > SV_MAX_DRAFT_LEN, "a thread for each row and drafted token");
  constexpr bool kSmall = kRowBytes == kSmallRowBytes;
  // (one dimension: with a grid of three, which needs no division, 128 requests in place took 65 us
  // where they take 62, and the ragged ones 122 for 120)
  const uint32_t part = blockIdx.x - (kSmall && p.reports == kApart ? 1u : 0u);
  const int32_t r = part / (p.chunks * p.splits);
  const int32_t c = part / p.splits % p.chunks;
  const int32_t group = part % p.splits;
  const int tid = threadIdx.x;
  const int64_t lo = int64_t(c) * kChunk;
  const int32_t n_tok = static_cast<int32_t>(min(int64_t(kChunk), p.V - lo));
  const uint32_t full = uint32_t(n_tok) * sizeof(T) & ~15u;  // bytes in whole vectors
  const int32_t n_vec = full >> 4, n_tail = n_tok - n_vec * kVec;

  if (kSmall && part == ~0u) {
    check_requests(p, int32_t(gridDim.x - 1) / (p.chunks * p.splits), kMode != kSparse && p.mask_row);
    return;
  }
  dependent_start();
  // ---- first loads: the request's parameters
  int32_t g = p.draft_len[r];
  const int64_t row = p.row0[r];
  const int64_t d0 = p.draft_row0 ? p.draft_row0[r] : 0;
  const float theta = p.repetition ? p.repetition[r] : 1.f;
  const float pres = p.presence ? p.presence[r] : 0.f;
  const float freq = p.frequency ? p.frequency[r] : 0.f;
  const int32_t slot = p.slots ? p.slots[r] : r;
  int64_t b0 = 0, b1 = 0;
  if (p.bias_start) {
    b0 = p.bias_start[r];
    b1 = p.bias_start[r + 1];
  }
  for (int w = tid; w < kWords; w += kProcThreads) s_touch[w] = s_bbits[w] = s_drafted[w] = 0;
  const bool first = c == 0 && group == 0 && !(kSmall && p.reports == kApart);
  if (tid == 0) {
    s_n = s_nd = 0;
    s_bias0 = ~0u;
    if (first && p.reports == kSingle && p.status) *p.status = 0;
    if (!kInPlace) {
      mbar_init(&s_bar, 1);
      fence_barrier_init();
    }
  }
  bool bad = g < 0 || g > p.gmax;
  g = min(max(g, 0), p.gmax);
  // rows of the request, and those of this CTA's group
  const int32_t all_rows = g + p.bonus_row;
  const int32_t row_a = p.first_row + group * p.group_rows;
  const int32_t rows = min(all_rows, row_a + p.group_rows);
  bool pen = theta != 1.f || pres != 0.f || freq != 0.f;
  if (pen && !(theta > 0.f && theta < INFINITY && fabsf(pres) < INFINITY &&
               fabsf(freq) < INFINITY && slot >= 0 && slot < p.n_slots)) {
    bad = true;
    pen = false;
  }
  if (b0 < 0 || b1 < b0 || b1 > p.n_bias) {
    bad = true;
    b1 = b0 = 0;
  }
  const uint8_t* const src = p.logits + (row * p.ld + lo) * int64_t(sizeof(T));
  uint8_t* const dst = p.out + (row * p.ld_out + lo) * int64_t(sizeof(T));
  const int64_t src_ld = p.ld * int64_t(sizeof(T)), dst_ld = p.ld_out * int64_t(sizeof(T));

  auto load_rows = [&](int32_t i0) {  // thread 0
    const int32_t n = min(kProcRows, rows - i0);
    if (full == 0) return;
    mbar_expect_tx(&s_bar, uint32_t(n) * full);
    for (int32_t u = 0; u < n; ++u)
      bulk_g2s(s_rows + u * kRowBytes, src + (i0 + u) * src_ld, full, &s_bar);
  };
  // ---- second loads, all in flight together: row parts, bits, drafted tokens, mask rows, biases
  if (!kInPlace && tid == 0 && row_a < rows) load_rows(row_a);
  uint32_t pb[kOwn], ob[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int w = tid + q * kProcThreads;
    pb[q] = ob[q] = 0;
    if (pen && w < kWords && w * 32 < n_tok) {
      const uint32_t valid = n_tok - w * 32 >= 32 ? ~0u : (1u << (n_tok - w * 32)) - 1u;
      pb[q] = p.prompt_bits[slot * p.ld_bits + (lo >> 5) + w] & valid;
      ob[q] = p.output_bits[slot * p.ld_bits + (lo >> 5) + w] & valid;
    }
  }
  const int role = kProcThreads - 1 - tid;  // the threads least busy with bits
  const bool drafted = pen && role < g;
  const int32_t x_draft = drafted ? p.draft_tokens[d0 + role] : -1;
  const bool masked = kMode != kSparse && p.mask_row != nullptr;
  int32_t mrow = -1;
  if (masked && tid < all_rows - p.first_row) {
    mrow = p.mask_row[row + p.first_row + tid];
    if (mrow < -1 || mrow >= p.n_mask) {
      bad = true;
      mrow = -1;
    }
  }
  constexpr int kAhead = 3;  // bias entries per thread loaded with the rest
  int32_t bt[kAhead];
#pragma unroll
  for (int q = 0; q < kAhead; ++q) {
    const int64_t k = b0 + tid + q * kProcThreads;
    bt[q] = k < b1 ? p.bias_tokens[k] : -1;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int w = tid + q * kProcThreads;
    if (w >= kWords) break;
    s_prompt[w] = pb[q];
    s_out[w] = ob[q];
    if (pb[q] | ob[q]) atomicOr(&s_touch[w], pb[q] | ob[q]);
  }
  if (tid <= SV_MAX_DRAFT_LEN) s_mrow[tid] = mrow;
  if (drafted) {
    bad |= x_draft < 0 || x_draft >= p.V;
    const int64_t o = x_draft - lo;
    if (o >= 0 && o < n_tok) {  // an unordered list: rows count the entries before them
      const int at = atomicAdd(&s_nd, 1);
      s_tok[at] = static_cast<int32_t>(o);
      s_pos[at] = role + 1;
      atomicOr(&s_touch[o >> 5], 1u << (o & 31));
      atomicOr(&s_drafted[o >> 5], 1u << (o & 31));
    }
  }
  auto add_bias = [&](int64_t k, int32_t x) {
    if (first) bad |= x < 0 || x >= p.V || (k > b0 && p.bias_tokens[k - 1] >= x);
    const int64_t o = x - lo;
    if (o >= 0 && o < n_tok) {
      atomicMin(&s_bias0, static_cast<uint32_t>(k - b0));
      atomicOr(&s_bbits[o >> 5], 1u << (o & 31));
      atomicOr(&s_touch[o >> 5], 1u << (o & 31));
    }
  };
#pragma unroll
  for (int q = 0; q < kAhead; ++q) {
    const int64_t k = b0 + tid + q * kProcThreads;
    if (k < b1) add_bias(k, bt[q]);
  }
  for (int64_t k = b0 + tid + kAhead * kProcThreads; k < b1; k += kProcThreads)
    add_bias(k, p.bias_tokens[k]);
  if (first && bad) report(p.status, SV_ERR_BAD_INPUT);
  __syncthreads();
  // The masks' words of this chunk (1 behind the vocabulary) for the batch of rows from i0 on: loads,
  // then stores to shared memory, with other work between them.  Tells whether any mask applies.
  constexpr int kMaskOwn = (kProcRows * kWords + kProcThreads - 1) / kProcThreads;
  uint32_t mw[kMode == kSparse ? 1 : kMaskOwn];
  auto load_masks = [&](int32_t i0) {
    const int32_t* mr = s_mrow + (i0 - p.first_row);
    const int32_t n = min(kProcRows, rows - i0);
    bool any = false;
#pragma unroll
    for (int u = 0; u < kProcRows; ++u) any |= u < n && mr[u] >= 0;
    if (!any) return false;
#pragma unroll
    for (int q = 0; q < kMaskOwn; ++q) {
      const int u = (tid + q * kProcThreads) / kWords, w = (tid + q * kProcThreads) % kWords;
      const int32_t m = u < n ? mr[u] : -1;
      mw[q] = ~0u;
      if (m >= 0 && w * 32 < n_tok) {
        mw[q] = p.mask[m * p.ld_mask + (lo >> 5) + w];
        if (n_tok - w * 32 < 32) mw[q] |= ~0u << (n_tok - w * 32);
      }
    }
    return true;
  };
  bool next_masked = false;
  if constexpr (kMode != kSparse) {
    if (masked && row_a < rows) next_masked = load_masks(row_a);
  }
  for (int w = tid; w < kWords; w += kProcThreads) {  // the list of touched offsets, in any order
    uint32_t t = s_touch[w];
    if (!t) continue;
    int at = atomicAdd(&s_n, __popc(t));
    while (t) {
      s_off[at++] = static_cast<uint16_t>(w * 32 + __ffs(t) - 1);
      t &= t - 1;
    }
  }
  __syncthreads();
  const int32_t n_list = s_n, nd = s_nd;
  auto count_of = [&](int o) {
    return s_out[o >> 5] >> (o & 31) & 1u ? p.counts[slot * p.ld_counts + lo + o] : 0;
  };
  // a biased token's value: the chunk's entries are neighbours in the ascending list
  auto bias_of = [&](int o) {
    if (!(s_bbits[o >> 5] >> (o & 31) & 1u)) return 0.f;
    int k = __popc(s_bbits[o >> 5] & ((1u << (o & 31)) - 1u));
    for (int w = 0; w < o >> 5; ++w) k += __popc(s_bbits[w]);
    return p.bias_values[b0 + s_bias0 + k];
  };
  // the count and bias of this thread's first listed token, while the rows are on their way
  int32_t count0 = 0;
  float bias0 = 0.f;
  if (tid < n_list) {
    count0 = count_of(s_off[tid]);
    bias0 = bias_of(s_off[tid]);
  }

  uint32_t phase = 0;
  for (int32_t i0 = row_a; i0 < rows; i0 += kProcRows) {
    const int32_t n = min(kProcRows, rows - i0);
    const bool now_masked = next_masked;  // the same in every thread
    if constexpr (kMode != kSparse) {
      if (now_masked) {
#pragma unroll
        for (int q = 0; q < kMaskOwn; ++q)
          if (tid + q * kProcThreads < kProcRows * kWords)
            (&s_mask[0][0])[tid + q * kProcThreads] = mw[q];
      }
      next_masked = masked && i0 + kProcRows < rows && load_masks(i0 + kProcRows);
    }
    if constexpr (!kInPlace) {
      for (int q = tid; q < n * n_tail; q += kProcThreads) {
        const int u = q / n_tail, j = n_vec * kVec + q % n_tail;
        reinterpret_cast<T*>(s_rows + u * kRowBytes)[j] =
            reinterpret_cast<const T*>(src + (i0 + u) * src_ld)[j];
      }
      if (full) mbar_wait(&s_bar, phase, p.status);
      phase ^= 1;
    }
    __syncthreads();
    // ---- masks: whole vectors, then the row's last few elements
    if (kMode != kSparse && now_masked) {
      auto piece = [&](int u, int v) {  // the bits of vector v
        return s_mask[u][(v * kVec) >> 5] >> ((v * kVec) & 31) & kAll;
      };
      if constexpr (kInPlace) {
        // A vector banned as a whole is stored, a partly banned one read first.  Both in one store
        // instruction: halves of a 32-byte sector stored by two take five times as long in all.
        // (Masked rows through shared memory by bulk copies took 83 us where this then took 73.)
        for (int v = tid; v < n_vec; v += kProcThreads) {
          uint4 x[kProcRows];
          uint32_t ok[kProcRows];
          uint8_t* const at = dst + i0 * dst_ld + v * 16;
#pragma unroll
          for (int u = 0; u < kProcRows; ++u) {
            ok[u] = u < n ? piece(u, v) : kAll;
            x[u] = make_uint4(0, 0, 0, 0);
            if (ok[u] && ok[u] != kAll) x[u] = *reinterpret_cast<const uint4*>(at + u * dst_ld);
          }
#pragma unroll
          for (int u = 0; u < kProcRows; ++u)
            if (ok[u] != kAll)
              *reinterpret_cast<uint4*>(at + u * dst_ld) = ban<E>(x[u], ok[u]);
        }
        for (int q = tid; q < n * n_tail; q += kProcThreads) {
          const int u = q / n_tail, j = n_vec * kVec + q % n_tail;
          if (!(s_mask[u][j >> 5] >> (j & 31) & 1u))
            reinterpret_cast<T*>(dst + (i0 + u) * dst_ld)[j] = X::down(-INFINITY);
        }
      } else {
        for (int q = tid; q < n * int(kRowBytes / 16); q += kProcThreads) {
          const int u = q / int(kRowBytes / 16), v = q % int(kRowBytes / 16);
          const uint32_t ok = piece(u, v);
          if (ok == kAll) continue;
          uint4* at = reinterpret_cast<uint4*>(s_rows + u * kRowBytes) + v;
          *at = ban<E>(*at, ok);
        }
      }
      __syncthreads();
    }
    // ---- edits: a thread per listed token
    for (int e = tid; e < n_list; e += kProcThreads) {
      const int o = s_off[e];
      const uint32_t w = o >> 5, b = 1u << (o & 31);
      const bool in_prompt = s_prompt[w] & b, biased = s_bbits[w] & b;
      const int drafts = s_drafted[w] & b ? nd : 0;
      const int32_t base = e == tid ? count0 : count_of(o);
      const float add = e == tid ? bias0 : bias_of(o);
      T* const at = reinterpret_cast<T*>(kInPlace ? dst + i0 * dst_ld : s_rows) + o;
      const int64_t step = kInPlace ? p.ld_out : int64_t(kRowBytes / sizeof(T));
      T x[kProcRows];
#pragma unroll
      for (int u = 0; u < kProcRows; ++u)
        if (u < n) x[u] = at[u * step];
#pragma unroll
      for (int u = 0; u < kProcRows; ++u) {
        if (u >= n || (now_masked && !(s_mask[u][w] & b))) continue;
        int32_t cnt = base;
        for (int k = 0; k < drafts; ++k) cnt += s_tok[k] == o && s_pos[k] <= i0 + u;
        const bool seen = in_prompt || cnt > 0;
        if (!seen && !biased) continue;
        float y = X::up(x[u]);
        if (seen) y = y > 0.f ? __fdiv_rn(y, theta) : y * theta;
        if (cnt > 0) y = y - freq * static_cast<float>(cnt) - pres;
        if (biased) y += add;
        at[u * step] = X::down(y);
      }
    }
    if constexpr (!kInPlace) {
      fence_proxy_async();  // the edits before the bulk copies that read them
      __syncthreads();
      for (int q = tid; q < n * n_tail; q += kProcThreads) {
        const int u = q / n_tail, j = n_vec * kVec + q % n_tail;
        reinterpret_cast<T*>(dst + (i0 + u) * dst_ld)[j] =
            reinterpret_cast<const T*>(s_rows + u * kRowBytes)[j];
      }
      if (tid == 0 && full) {
        for (int32_t u = 0; u < n; ++u)
          bulk_s2g(dst + (i0 + u) * dst_ld, s_rows + u * kRowBytes, full);
        bulk_group_commit();
        bulk_group_wait_read();  // the rows may be overwritten, or the CTA end
        if (i0 + kProcRows < rows) load_rows(i0 + kProcRows);
      }
    }
    if (i0 + kProcRows < rows) __syncthreads();  // masks and tails of the next rows
  }
}

template <typename E, int kMode, uint32_t kRowBytes>
sv_status launch_process(ProcParams p, int32_t B, int sms, cudaStream_t s) {
  constexpr int64_t chunk = kRowBytes / sizeof(typename ProcElem<E>::T);
  const int64_t chunks = (p.V + chunk - 1) / chunk;
  // One CTA takes all rows of a chunk, unless that leaves SMs with fewer than twelve CTAs: then groups
  // of kProcRows rows go to CTAs of their own, each with the lists built anew (1 request of 17 rows
  // of 152000, masked in place: 23.6 -> 7.5 us; 256 requests of 17 rows of 1000: 59 -> 29; with four
  // CTAs per SM as the limit 7.6 and 54).
  const int64_t most = std::max(1, p.gmax + p.bonus_row - p.first_row);
  const int64_t batches = (most + kProcRows - 1) / kProcRows;
  const int64_t splits = std::min(batches, std::max<int64_t>(1, 12 * sms / (chunks * B)));
  p.group_rows = int32_t((batches + splits - 1) / splits) * kProcRows;
  p.splits = int32_t((most + p.group_rows - 1) / p.group_rows);
  p.chunks = int32_t(chunks);
  // CTA 0 checks a call of at most 512 rows and 1024 bias entries (fewer with many requests, whose
  // lists' ends have to be looked up) while the others are at work (8 requests of 5 rows of 32000
  // 7.1 -> 4.8 us, 21 of 17 rows of 4298 6.6 -> 4.7); a larger call would wait for it (256 requests
  // with 4 biases each 6.4 -> 10.3).
  const bool few = int64_t(B) * (p.gmax + 1) <= 512 &&
                   (!p.bias_start || p.n_bias + 8 * int64_t(B) <= 1024);
  p.reports = B == 1 || !p.status ? kSingle
              : kRowBytes == kSmallRowBytes && few ? kApart
                                                   : kFirst;
  if (p.reports == kFirst) {
    const sv_status st = reset_status(p.status, s);
    if (st != SV_OK) return st;
  }
  const size_t smem = kMode == kCopy ? std::min<int64_t>(kProcRows, most) * kRowBytes : 0;
  const unsigned ctas = unsigned(chunks * B * p.splits) + (p.reports == kApart);
  return launch_dependent(process_kernel<E, kMode, kRowBytes>, ctas, kProcThreads, smem, s, p);
}

template <typename E, int kMode>
sv_status launch_process(const ProcParams& p, int32_t B, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return SV_ERR_CUDA;
  // Parts of 1 KB while they make one wave (eight CTAs an SM), so that long lists of touched tokens
  // are spread as far as they go: 9 requests of 5 rows of 8217 bf16 with 6382 tokens of history and
  // 300 biases, masked in place, 26.3 -> 7.9 us; 2 of 14 rows of 1709 fp32 13.7 -> 6.3; 8 of 5 rows of
  // 32000 7.1 -> 6.2 (the status reset by a launch of its own).  Beyond a wave every part's own lists
  // cost more: 13 rows of 113249 fp32 (11.7 CTAs an SM) 5.2 -> 5.8.
  constexpr int64_t kFew = kSmallRowBytes / sizeof(typename ProcElem<E>::T);
  const int64_t most = std::max(1, p.gmax + p.bonus_row - p.first_row);
  const int64_t batches = (most + kProcRows - 1) / kProcRows;
  if ((p.V + kFew - 1) / kFew * B * batches <= int64_t(8) * sms)
    return launch_process<E, kMode, kSmallRowBytes>(p, B, sms, s);
  return launch_process<E, kMode, proc_row_bytes(kMode)>(p, B, sms, s);
}

template <typename E>
sv_status launch_process(const ProcParams& p, int32_t B, cudaStream_t s) {
  if (p.out != p.logits) return launch_process<E, kCopy>(p, B, s);
  return p.mask_row ? launch_process<E, kMasked>(p, B, s) : launch_process<E, kSparse>(p, B, s);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0) return reset_status(status, s);
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
  // the most CTAs any mode launches
  if ((V + 4095 / eb) / (4096 / eb) * B > INT32_MAX / 32) return SV_ERR_UNSUPPORTED;
  const ProcParams p = {static_cast<const uint8_t*>(logits),
                        ld,
                        static_cast<uint8_t*>(out),
                        ld_out,
                        V,
                        row0,
                        draft_row0,
                        draft_len,
                        max_draft_len,
                        std::min(first_row, max_draft_len + 1),  // no row is that far
                        bonus_row,
                        draft_tokens,
                        0,
                        1,
                        0,
                        slots,
                        n_slots,
                        counts,
                        ld_counts,
                        prompt_bits,
                        output_bits,
                        ld_bits,
                        repetition,
                        presence,
                        frequency,
                        bias_start,
                        bias_tokens,
                        bias_values,
                        n_bias,
                        mask,
                        ld_mask,
                        n_mask,
                        mask_row,
                        status,
                        kFirst};
  return dtype == SV_BF16 ? launch_process<bf16_tag>(p, B, s) : launch_process<float>(p, B, s);
}
