// spec_logits.cu — spec_process_logits: penalties for repeated tokens, biases and grammar masks on the
// logits of every drafted position, before they are verified.
//
// One block owns a stretch of the vocabulary for one request and all its positions.  It counts the
// request's history over that stretch in shared memory (integer adds: their order changes nothing), so
// the [V] table of counts never exists in memory, and then streams the positions' logits through
// registers.  A thread keeps its tokens' counts in registers from position to position and adds the
// drafts as it passes them.  Bound by reading and writing the logits once.

#include "decode_common.cuh"

namespace sv {

constexpr int kRuleThreads = 256;
constexpr int kRowsAhead = 4;            // positions whose logits a thread loads before it uses them
constexpr int kStretches[] = {8192, 4096, 2048};  // tokens of one block

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

// VEC logits as one load and store of 2 to 16 bytes.  The loads are not read-only ones: out may be logits.
template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
};
template <>
struct Raw<8> {
  uint32_t w[2];
  __device__ __forceinline__ void load(const void* p) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]); }
};
template <>
struct Raw<4> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const void* p) { asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p)); }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint32_t*>(p) = w[0]; }
};
template <>
struct Raw<2> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const void* p) {
    uint16_t h;
    asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
    w[0] = h;
  }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0]; }
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

// A thread takes GROUPS runs of VEC tokens, kRuleThreads * VEC apart, through all positions.
template <bool BF16, int VEC, int GROUPS>
__global__ void __launch_bounds__(kRuleThreads) rules_kernel(const __grid_constant__ RuleParams P) {
  constexpr int ES = BF16 ? 2 : 4;
  extern __shared__ __align__(16) uint32_t word[];  // [stretch]
  __shared__ int draft[SPEC_MAX_NEW];               // relative to the stretch; -1: elsewhere
  const int b = blockIdx.y, first = blockIdx.x * P.stretch;
  const int len = min(P.stretch, P.V - first);
  pdl_launch_next();
  for (int i = threadIdx.x; i < (len + 3) / 4; i += kRuleThreads) reinterpret_cast<uint4*>(word)[i] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  const spec_logit_rules_t& R = P.r;
  const int rows = R.t_per_row ? min(max(__ldg(R.t_per_row + b), 0), P.T) : P.T;
  const float rep = R.repetition ? __ldg(R.repetition + b) : 1.0f;
  const float pre = R.presence ? __ldg(R.presence + b) : 0.0f;
  const float fre = R.frequency ? __ldg(R.frequency + b) : 0.0f;
  const int held = R.history ? min(max(__ldg(R.history_len + b), 0), R.history_stride) : 0;
  const int prompt = R.history && R.prompt_len ? __ldg(R.prompt_len + b) : 0;
  const bool penal = rep != 1.0f || pre != 0.0f || fre != 0.0f;

  if (threadIdx.x < SPEC_MAX_NEW) {
    int d = -1;
    if (penal && R.draft && (int)threadIdx.x < rows - 1) d = __ldg(R.draft + (int64_t)b * (P.T - 1) + threadIdx.x);
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
  if (penal) {
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

  const int64_t row_bytes = (int64_t)P.V * ES;
  const int64_t base = ((int64_t)b * P.T * P.V + first) * ES;
  const char* in = static_cast<const char*>(P.logits) + base;
  char* out = static_cast<char*>(P.out) + base;
  const int32_t* mask = R.mask ? R.mask + (int64_t)b * P.T * P.words + (first >> 5) : nullptr;
  constexpr uint32_t kAll = VEC == 32 ? ~0u : (1u << VEC) - 1;
  // What a token's word makes of its logit x: (seen ? x * (x > 0 ? 1 / rep : rep) : x) + off.  The reciprocal
  // is within 2^-23 of the division, and the terms of off are summed before they meet the logit.
  const float inv = 1.0f / rep;
  const auto effect = [&](uint32_t w, bool& seen) {
    const uint32_t count = w & kCountMask, e = (w & ~kPromptBit) >> kBiasShift;
    seen = penal && (count > 0 || (w & kPromptBit));
    float off = e ? __ldg(R.bias + (int64_t)b * R.bias_n + e - 1) : 0.0f;
    if (count > 0) off = off - fre * (float)count - pre;
    return off;
  };
  for (int v0 = threadIdx.x * VEC; v0 < len; v0 += kRuleThreads * VEC * GROUPS) {  // VEC divides V and the stretch
    float off[GROUPS][VEC];
    uint32_t seen[GROUPS];  // bit i: token i is; bit 31: some token's logit changes
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int v = v0 + g * kRuleThreads * VEC;
      uint32_t w[VEC], any = 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        w[i] = v < len ? word[v + i] : 0;
        any |= w[i];
        off[g][i] = 0.0f;
      }
      seen[g] = any ? 1u << 31 : 0;
      if (any) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          bool s;
          off[g][i] = effect(w[i], s);
          seen[g] |= (uint32_t)s << i;
        }
      }
    }
    for (int t0 = 0; t0 < rows; t0 += kRowsAhead) {
      uint32_t allowed[kRowsAhead][GROUPS];
      Raw<VEC * ES> raw[kRowsAhead][GROUPS];
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r)
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const int v = v0 + g * kRuleThreads * VEC;
          allowed[r][g] = kAll;
          if (mask && t0 + r < rows && v < len)
            allowed[r][g] = ((uint32_t)__ldg(mask + (int64_t)(t0 + r) * P.words + (v >> 5)) >> (v & 31)) & kAll;
        }
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r)
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const int v = v0 + g * kRuleThreads * VEC;
#pragma unroll
          for (int i = 0; i < (VEC * ES + 3) / 4; ++i) raw[r][g].w[i] = 0;
          // a run that the mask forbids throughout is not read
          if (allowed[r][g] && t0 + r < rows && v < len) raw[r][g].load(in + (t0 + r) * row_bytes + v * ES);
        }
#pragma unroll
      for (int r = 0; r < kRowsAhead; ++r) {
        const int t = t0 + r;
        if (t >= rows) break;
        const int d = t > 0 ? draft[t - 1] : -1;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const int v = v0 + g * kRuleThreads * VEC;
          if (v >= len) continue;
          if (d >= v && d < v + VEC) {  // this thread's word alone: from here on the draft counts
            const uint32_t w = ++word[d];
            bool s;
            const float o = effect(w, s);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (i == d - v) off[g][i] = o;
            seen[g] |= 1u << 31 | 1u << (d - v);
          }
          if (seen[g] || allowed[r][g] != kAll) {
            float x[VEC];
            unpack<BF16, VEC>(raw[r][g].w, x);
            if (seen[g]) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                const float f = x[i] > 0.0f ? inv : rep;
                x[i] = fmaf(x[i], (seen[g] >> i) & 1u ? f : 1.0f, off[g][i]);
              }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (!((allowed[r][g] >> i) & 1u)) x[i] = -INFINITY;
            pack<BF16, VEC>(raw[r][g].w, x);
          }
          raw[r][g].store(out + t * row_bytes + v * ES);
        }
      }
    }
  }
}

template <bool BF16>
static cudaError_t launch_rules(const RuleParams& P, int align, cudaStream_t st) {
  // the widest vector that divides the rows and their addresses; narrow ones take several runs a thread to
  // keep as many bytes in flight
  constexpr int ES = BF16 ? 2 : 4;
  void (*kern)(RuleParams) = nullptr;
  if (align % 16 == 0) kern = rules_kernel<BF16, 16 / ES, 1>;
  else if (align % 8 == 0) kern = rules_kernel<BF16, 8 / ES, 2>;
  else if (align % 4 == 0) kern = rules_kernel<BF16, 4 / ES, 4>;
  else kern = rules_kernel<BF16, 1, 4>;
  const dim3 grid((P.V + P.stretch - 1) / P.stretch, P.B);
  return launch_early(kern, grid, dim3(kRuleThreads), P.stretch * sizeof(uint32_t), st, P);
}

}  // namespace sv

using namespace sv;

extern "C" spec_status_t spec_process_logits(const void* logits, void* out, const spec_logit_rules_t* rules, int32_t B,
                                             int32_t T, int32_t V, spec_dtype_t dtype, void* stream) {
  if (!rules || B < 0 || T < 0 || V <= 0) return SPEC_ERR_INVALID_ARG;
  const spec_logit_rules_t& r = *rules;
  if (r.history_stride < 0 || r.bias_n < 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (V > SPEC_MAX_V || B > 65535 || T > SPEC_MAX_NEW || r.history_stride > SPEC_MAX_HISTORY ||
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
  // the largest power of two that divides every row's address
  const uint64_t bits = (uint64_t)(uintptr_t)logits | (uint64_t)(uintptr_t)out | (uint64_t)((int64_t)V * es) | 16u;
  const int align = (int)(bits & (~bits + 1));
  const cudaError_t e = dtype == SPEC_DTYPE_BF16 ? launch_rules<true>(P, align, st) : launch_rules<false>(P, align, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
