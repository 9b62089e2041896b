// spec_logits.cu — spec_process_logits: penalties for repeated tokens, biases and grammar masks on the
// logits of every drafted position, before they are verified.
//
// One block owns a stretch of the vocabulary for one request and all its positions.  It counts the
// request's history over that stretch in shared memory (integer adds: their order changes nothing), so
// the [V] table of counts never exists in memory, and then streams the positions' logits through
// registers.  A thread keeps the effect of its tokens' counts in registers from position to position and
// adds the drafts as it passes them.
//
// Measured, against a copy at 6772 GB/s: 256 requests of 3 to 9 positions, V = 152064 in fp32, histories of
// 2000 to 4000 tokens: 279 us, 6.2 TB/s (0.91), bound by reading and writing the logits once; 64 x 7, V = 128256
// in bf16 with masks: 54 us, 4.4 TB/s (0.65; 39 us without penalties, bias and mask), bound by instructions,
// most of all in the stretch of the frequent tokens.

#include <type_traits>

#include "decode_common.cuh"

namespace sv {

constexpr int kRuleThreads = 256;
constexpr int kRowsAhead = 4;            // positions whose logits a thread loads before it uses them
// Tokens of one block: a long stretch shares one scan of the history among more tokens (the two batches above: 279
// and 54 us; 289 and 54 with 4096 at most, 283 and 58 with shorter ones until there are 16 blocks per SM).
constexpr int kStretches[] = {8192, 4096, 2048};

// A token's word of counts: bit 31 = in the prompt, bits 20..30 = 1 + index of its bias entry (0: none),
// bits 0..19 = times among the output tokens.
constexpr uint32_t kPromptBit = 1u << 31;
constexpr int kBiasShift = 20;
constexpr uint32_t kCountMask = (1u << kBiasShift) - 1;
static_assert(SPEC_MAX_HISTORY + SPEC_MAX_NEW <= (int)kCountMask, "counts fit their field");
static_assert(SPEC_MAX_BIAS + 1 < (1 << (31 - kBiasShift)), "bias indices fit their field");

struct RuleParams {
  const void* logits;
  void* out;
  spec_logit_rules_t r;
  int B, T, V, words, stretch;
};

// 16 bytes of logits.  The loads are not read-only ones: out may be logits.
struct Raw {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
};

template <bool BF16, int VEC>
__device__ __forceinline__ void unpack(const uint32_t* w, float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    x[i] = !BF16 ? __uint_as_float(w[i]) : i % 2 ? bf16_high(w[i / 2]) : bf16_low(w[i / 2]);
}
template <bool BF16, int VEC>
__device__ __forceinline__ void pack(uint32_t* w, const float (&x)[VEC]) {
  if constexpr (!BF16) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) w[i / 2] = pack_bf16(x[i], i + 1 < VEC ? x[i + 1] : 0.0f);
  }
}

// A block's request, its stretch of the vocabulary and what the request asks for.
struct Stretch {
  int b, first, len, rows;
  float rep, pre, fre, inv;
  bool penal;
};

// Counts the request's history, bias entries and prompt over the stretch into `word`; `draft` gets the drafts
// relative to the stretch (-1: elsewhere).
__device__ __forceinline__ Stretch count_rules(const RuleParams& P, uint32_t* word, int* draft) {
  Stretch s;
  s.b = blockIdx.x, s.first = blockIdx.y * P.stretch;
  s.len = min(P.stretch, P.V - s.first);
  const int b = s.b, first = s.first, len = s.len;
  const spec_logit_rules_t& R = P.r;
  pdl_launch_next();
  for (int i = threadIdx.x; i < (len + 3) / 4; i += kRuleThreads) reinterpret_cast<uint4*>(word)[i] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  s.rows = R.t_per_row ? min(max(__ldg(R.t_per_row + b), 0), P.T) : P.T;
  s.rep = R.repetition ? __ldg(R.repetition + b) : 1.0f;
  s.pre = R.presence ? __ldg(R.presence + b) : 0.0f;
  s.fre = R.frequency ? __ldg(R.frequency + b) : 0.0f;
  const int held = R.history ? min(max(__ldg(R.history_len + b), 0), R.history_stride) : 0;
  const int prompt = R.history && R.prompt_len ? __ldg(R.prompt_len + b) : 0;
  s.penal = s.rep != 1.0f || s.pre != 0.0f || s.fre != 0.0f;
  s.inv = 1.0f / s.rep;
  if (threadIdx.x < SPEC_MAX_NEW) {
    int d = -1;
    if (s.penal && R.draft && (int)threadIdx.x < s.rows - 1) d = __ldg(R.draft + (int64_t)b * (P.T - 1) + threadIdx.x);
    draft[threadIdx.x] = d >= first && d - first < len ? d - first : -1;
  }
  __syncthreads();
  if (R.bias_n > 0) {  // of two entries with one id the later holds
    const int32_t* ids = R.bias_ids + (int64_t)b * R.bias_n;
    for (int i = threadIdx.x; i < R.bias_n; i += kRuleThreads) {
      const uint32_t v = (uint32_t)__ldg(ids + i) - (uint32_t)first;
      if (v < (uint32_t)len) atomicMax(&word[v], (uint32_t)(i + 1) << kBiasShift);
    }
    __syncthreads();
  }
  if (s.penal) {
    const int32_t* ids = R.history + (int64_t)b * R.history_stride;
    constexpr int kAhead = 8;  // entries a thread loads before it counts the first
    for (int i0 = threadIdx.x; i0 < held; i0 += kRuleThreads * kAhead) {
      uint32_t v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * kRuleThreads;
        v[j] = i < held ? (uint32_t)__ldg(ids + i) - (uint32_t)first : ~0u;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (v[j] < (uint32_t)len) {
          if (i0 + j * kRuleThreads < prompt)
            atomicOr(&word[v[j]], kPromptBit);
          else
            atomicAdd(&word[v[j]], 1u);
        }
    }
  }
  __syncthreads();
  return s;
}

// A repeated token's logit: x / rep or x * rep.  The quotient is the product with the reciprocal, twice corrected by its
// residual (P. Markstein, IBM Journal of Research and Development 34, 1990): the first leaves it within a unit in the
// last place, so the second rounds it correctly.  Where the residual may not be exact the product stands, within 2 units.
// (64 x 7 x 128256 in bf16: 53.3 us without the corrections, 54.4 with them, 56.7 with divisions.)
__device__ __forceinline__ float repeated(float x, const Stretch& s) {
  float q = x * s.inv;
  if (fabsf(x) > 0x1p-60f && fabsf(q) < 0x1p60f) {
    q = fmaf(fmaf(-q, s.rep, x), s.inv, q);
    q = fmaf(fmaf(-q, s.rep, x), s.inv, q);
  }
  return x > 0.0f ? q : x * s.rep;
}

// What a token's word makes of its logit: (seen ? repeated(x) : x) + off.  The terms of off are summed before they meet
// the logit.
__device__ __forceinline__ float effect(const RuleParams& P, const Stretch& s, uint32_t w, bool& seen) {
  const uint32_t count = w & kCountMask, e = (w & ~kPromptBit) >> kBiasShift;
  seen = s.rep != 1.0f && (count > 0 || (w & kPromptBit));
  float off = e ? __ldg(P.r.bias + (int64_t)s.b * P.r.bias_n + e - 1) : 0.0f;
  if (count > 0) off = off - s.fre * (float)count - s.pre;
  return off;
}

// Rows on 16-byte boundaries.  A thread takes a run of VEC tokens through all positions, with their counts' effect
// in registers.
template <bool BF16>
__global__ void __launch_bounds__(kRuleThreads, 5) rules_kernel(const __grid_constant__ RuleParams P) {
  constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
  extern __shared__ __align__(16) uint32_t word[];  // [stretch]
  __shared__ int draft[SPEC_MAX_NEW];
  const Stretch s = count_rules(P, word, draft);
  const int b = s.b, first = s.first, len = s.len, rows = s.rows;

  const int64_t row_bytes = (int64_t)P.V * ES;
  const int64_t base = ((int64_t)b * P.T * P.V + first) * ES;
  const char* in = static_cast<const char*>(P.logits) + base;
  char* out = static_cast<char*>(P.out) + base;
  const int32_t* mask = P.r.mask ? P.r.mask + (int64_t)b * P.T * P.words + (first >> 5) : nullptr;
  constexpr uint32_t kAll = (1u << VEC) - 1;
  for (int v = threadIdx.x * VEC; v < len; v += kRuleThreads * VEC) {  // VEC divides V and the stretch
    float off[VEC];
    uint32_t w[VEC], any = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[i] = word[v + i];
      any |= w[i];
      off[i] = 0.0f;
    }
    uint32_t seen = any ? 1u << 31 : 0;  // bit i: token i is; bit 31: some token's logit changes
    if (any) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        bool is;
        off[i] = effect(P, s, w[i], is);
        seen |= (uint32_t)is << i;
      }
    }
    for (int t0 = 0; t0 < rows; t0 += kRowsAhead) {
      uint32_t allowed[kRowsAhead];
      Raw raw[kRowsAhead];
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r) {
        allowed[r] = kAll;
        if (mask && t0 + r < rows)
          allowed[r] = ((uint32_t)__ldg(mask + (int64_t)(t0 + r) * P.words + (v >> 5)) >> (v & 31)) & kAll;
      }
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[r].w[i] = 0;
        // a run that the mask forbids throughout is not read: the load then waits for the mask, but a mask that allows
        // tokens in 1 of its words in 100 leaves most memory sectors unread (64 x 7 x 128256 in bf16, such masks: 46.8 us
        // against 51.1; 1 token in 16 for half of the requests, 15 for the others: 53.9 against 51.8)
        if (allowed[r] && t0 + r < rows) raw[r].load(in + (t0 + r) * row_bytes + v * ES);
      }
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r) {
        const int t = t0 + r;
        if (t >= rows) break;
        const int d = t > 0 ? draft[t - 1] : -1;
        if (d >= v && d < v + VEC) {  // this thread's word alone: from here on the draft counts
          const uint32_t u = ++word[d];
          bool is;
          const float o = effect(P, s, u, is);
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (i == d - v) off[i] = o;
          seen |= 1u << 31 | 1u << (d - v);
        }
        if (seen || allowed[r] != kAll) {
          float x[VEC];
          unpack<BF16, VEC>(raw[r].w, x);
          if (seen) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              if ((seen >> i) & 1u) x[i] = repeated(x[i], s);
              x[i] += off[i];
            }
          }
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (!((allowed[r] >> i) & 1u)) x[i] = -INFINITY;
          pack<BF16, VEC>(raw[r].w, x);
        }
        raw[r].store(out + t * row_bytes + v * ES);
      }
    }
  }
}

// Rows that begin anywhere.  The runs of a row lie on its own 16-byte boundaries, so a token's run and thread
// change from position to position: every token's effect lies in shared memory, with bitmaps of the tokens that have
// one and that are seen.  The drafts' logits behind them are worked out beforehand and written last.  Runs that
// reach past the stretch, and all where out lies otherwise than logits on 16 bytes, are read and written an element
// at a time.  (Four blocks an SM, not the three that its registers would leave: 64 x 7 x 128257 in bf16: 115 us against 133.)
template <bool BF16>
__global__ void __launch_bounds__(kRuleThreads, 4) rules_odd_kernel(const __grid_constant__ RuleParams P) {
  constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
  using Element = typename std::conditional<BF16, uint16_t, uint32_t>::type;
  extern __shared__ __align__(16) uint32_t word[];  // [stretch], then the bitmaps
  __shared__ int draft[SPEC_MAX_NEW];
  __shared__ uint32_t draft_word[SPEC_MAX_NEW];      // the counts of the drafts
  const int map = P.stretch / 32 + 2;                // words of a bitmap, [-1 .. stretch / 32]
  uint32_t* marks = word + P.stretch + 1;            // tokens with an effect
  uint32_t* seen = marks + map;                      // tokens among the prompt or the output
  for (int i = threadIdx.x; i < 2 * map; i += kRuleThreads) marks[i - 1] = 0;
  const Stretch s = count_rules(P, word, draft);
  const int b = s.b, first = s.first, len = s.len, rows = s.rows;
  if ((int)threadIdx.x < rows - 1 && draft[threadIdx.x] >= 0) draft_word[threadIdx.x] = word[draft[threadIdx.x]];
  __syncthreads();
  const int lane = threadIdx.x % 32;
  for (int i = threadIdx.x - lane; i < len; i += kRuleThreads) {  // 32 neighbours a warp; a word becomes its effect
    const int v = i + lane;
    const uint32_t w = v < len ? word[v] : 0;
    bool is = false;
    float off = 0.0f;
    if (w) off = effect(P, s, w, is);
    if (v < len) word[v] = __float_as_uint(off);
    const uint32_t any = __ballot_sync(~0u, w != 0), all = __ballot_sync(~0u, is);
    if (lane == 0) marks[i / 32] = any, seen[i / 32] = all;
  }
  __syncthreads();

  const char* in = static_cast<const char*>(P.logits) + ((int64_t)b * P.T * P.V + first) * ES;
  char* out = static_cast<char*>(P.out) + ((int64_t)b * P.T * P.V + first) * ES;
  const int32_t* mask = P.r.mask ? P.r.mask + (int64_t)b * P.T * P.words + (first >> 5) : nullptr;
  const int words = (len + 31) / 32;  // of the mask, and of the bitmaps
  const bool alike = (((uintptr_t)in ^ (uintptr_t)out) & 15) == 0;
  constexpr uint32_t kAll = (1u << VEC) - 1;
  const auto bits_at = [&](const uint32_t* p, int v) {  // bits v .. v + VEC - 1 of a bitmap, v > -32
    const int at = v >> 5;
    return __funnelshift_r(p[at], p[at + 1], v & 31) & kAll;
  };
  const auto shaped = [&](float x, bool is, float off) { return (is ? repeated(x, s) : x) + off; };
  // draft i at a position t > i counts with all drafts of its token before t
  constexpr int kPairs = SPEC_MAX_NEW * (SPEC_MAX_NEW - 1) / 2, kPairsEach = (kPairs + kRuleThreads - 1) / kRuleThreads;
  Element fixed[kPairsEach];
  int64_t place[kPairsEach];  // -1: none
#pragma unroll
  for (int k = 0; k < kPairsEach; ++k) {
    place[k] = -1;
    const int pair = threadIdx.x + k * kRuleThreads;
    if (pair >= rows * (rows - 1) / 2) continue;
    int t = (int)((1.0f + sqrtf(1.0f + 8.0f * pair)) * 0.5f);  // t (t - 1) / 2 <= pair < t (t + 1) / 2
    while (t * (t - 1) / 2 > pair) --t;
    while (t * (t + 1) / 2 <= pair) ++t;
    const int d = draft[pair - t * (t - 1) / 2];
    if (d < 0) continue;
    uint32_t w = 0, more = 0;
    for (int i = 0; i < t; ++i)
      if (draft[i] == d) w = draft_word[i], ++more;
    const uint32_t raw[1] = {reinterpret_cast<const Element*>(in)[(int64_t)t * P.V + d]};
    float x[1];
    unpack<BF16, 1>(raw, x);
    bool is;
    const float off = effect(P, s, w + more, is);
    x[0] = shaped(x[0], is, off);
    if (mask && !(((uint32_t)__ldg(mask + (int64_t)t * P.words + d / 32) >> (d % 32)) & 1)) x[0] = -INFINITY;
    uint32_t packed[1];
    pack<BF16, 1>(packed, x);
    fixed[k] = (Element)packed[0];
    place[k] = (int64_t)t * P.V + d;
  }
  __syncthreads();  // out may be logits: they are read before any is written
  for (int t0 = 0; t0 < rows; t0 += kRowsAhead)
    for (int j = threadIdx.x; j * VEC < len + VEC - 1; j += kRuleThreads) {
      uint32_t allowed[kRowsAhead];
      Raw raw[kRowsAhead];
      int v[kRowsAhead];
      bool whole[kRowsAhead];
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r) {
        const char* row = in + (int64_t)(t0 + r) * P.V * ES;
        v[r] = j * VEC - (int)(((uintptr_t)row & 15) / ES);
        whole[r] = alike && t0 + r < rows && v[r] >= 0 && v[r] + VEC <= len;
        allowed[r] = kAll;
        if (mask && t0 + r < rows) {
          const int32_t* m = mask + (int64_t)(t0 + r) * P.words;
          const int at = v[r] >> 5;
          const uint32_t lo = at >= 0 && at < words ? (uint32_t)__ldg(m + at) : 0, hi = at + 1 < words ? (uint32_t)__ldg(m + at + 1) : 0;
          allowed[r] = __funnelshift_r(lo, hi, v[r] & 31) & kAll;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[r].w[i] = 0;
        if (t0 + r >= rows || !allowed[r] || v[r] >= len || v[r] + VEC <= 0) continue;
        if (whole[r]) {
          raw[r].load(row + v[r] * ES);
        } else {  // (elements outside are replaced by one of this run's)
          Element e[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) e[i] = reinterpret_cast<const volatile Element*>(row)[min(max(v[r] + i, 0), len - 1)];
#pragma unroll
          for (int i = 0; i < VEC; ++i) raw[r].w[i * ES / 4] |= (uint32_t)e[i] << (i * ES % 4 * 8);
        }
      }
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r) {
        const int t = t0 + r;
        if (t >= rows) break;
        char* to = out + (int64_t)t * P.V * ES;
        const uint32_t marked = bits_at(marks, v[r]);
        if (marked || allowed[r] != kAll) {
          float x[VEC];
          unpack<BF16, VEC>(raw[r].w, x);
          if (marked) {
            const uint32_t is = bits_at(seen, v[r]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = shaped(x[i], (is >> i) & 1, __uint_as_float(word[min(max(v[r] + i, 0), len - 1)]));
          }
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (!((allowed[r] >> i) & 1u)) x[i] = -INFINITY;
          pack<BF16, VEC>(raw[r].w, x);
        }
        if (whole[r]) {
          raw[r].store(to + v[r] * ES);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (v[r] + i >= 0 && v[r] + i < len)
              reinterpret_cast<Element*>(to)[v[r] + i] = (Element)(raw[r].w[i * ES / 4] >> (i * ES % 4 * 8));
        }
      }
    }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPairsEach; ++k)
    if (place[k] >= 0) reinterpret_cast<Element*>(out)[place[k]] = fixed[k];
}

}  // namespace sv

using namespace sv;

extern "C" spec_status_t spec_process_logits(const void* logits, void* out, const spec_logit_rules_t* rules, int32_t B,
                                             int32_t T, int32_t V, spec_dtype_t dtype, void* stream) {
  if (!rules || B < 0 || T < 0 || V <= 0) return SPEC_ERR_INVALID_ARG;
  const spec_logit_rules_t& r = *rules;
  if (r.history_stride < 0 || r.bias_n < 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (V > SPEC_MAX_V || B > SPEC_MAX_BATCH || T > SPEC_MAX_NEW || r.history_stride > SPEC_MAX_HISTORY ||
      r.bias_n > SPEC_MAX_BIAS)
    return SPEC_ERR_UNSUPPORTED;
  if (r.history && !r.history_len) return SPEC_ERR_INVALID_ARG;
  if (r.bias_n > 0 && (!r.bias_ids || !r.bias)) return SPEC_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SPEC_OK;
  if (!logits || !out) return SPEC_ERR_INVALID_ARG;
  const int es = dtype == SPEC_DTYPE_BF16 ? 2 : 4;
  if ((uintptr_t)logits % es || (uintptr_t)out % es) return SPEC_ERR_INVALID_ARG;

  RuleParams P = {};
  P.logits = logits, P.out = out, P.r = r;
  P.B = B, P.T = T, P.V = V, P.words = (V + 31) / 32;
  // A long stretch shares one scan of the history among more tokens; a shorter one is taken when there would
  // be fewer than 8 blocks per SM.
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  for (int s : kStretches) {
    P.stretch = s;
    if ((int64_t)B * ((V + s - 1) / s) >= 8 * sms) break;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // all requests' first stretches first: vocabularies tend to begin with the frequent tokens, whose stretches take
  // the longest
  const dim3 grid(B, (V + P.stretch - 1) / P.stretch), block(kRuleThreads);
  const bool even = (uintptr_t)logits % 16 == 0 && (uintptr_t)out % 16 == 0 && (int64_t)V * es % 16 == 0;
  const bool bf16 = dtype == SPEC_DTYPE_BF16;
  const size_t counts = P.stretch * sizeof(uint32_t), marks = 2 * (P.stretch / 32 + 2) * sizeof(uint32_t);
  const cudaError_t e = even ? launch_early(bf16 ? rules_kernel<true> : rules_kernel<false>, grid, block, counts, st, P)
                             : launch_early(bf16 ? rules_odd_kernel<true> : rules_odd_kernel<false>, grid, block, counts + marks, st, P);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
