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
constexpr int kStretch = 8192;  // tokens of one block: 32 KB of counts, 6 blocks per SM

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
  int B, T, V, words;
};

template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 4> {
  using W = float4;
  static __device__ __forceinline__ void get(const W& w, float (&x)[4]) { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
  static __device__ __forceinline__ W put(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Pack<float, 1> {
  using W = float;
  static __device__ __forceinline__ void get(const W& w, float (&x)[1]) { x[0] = w; }
  static __device__ __forceinline__ W put(const float (&x)[1]) { return x[0]; }
};
template <>
struct Pack<__nv_bfloat16, 8> {
  using W = uint4;
  static __device__ __forceinline__ void get(const W& w, float (&x)[8]) { unpack8(w, x); }
  static __device__ __forceinline__ W put(const float (&x)[8]) { return pack8(x); }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  using W = __nv_bfloat16;
  static __device__ __forceinline__ void get(const W& w, float (&x)[1]) { x[0] = __bfloat162float(w); }
  static __device__ __forceinline__ W put(const float (&x)[1]) { return __float2bfloat16(x[0]); }
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kRuleThreads) rules_kernel(const __grid_constant__ RuleParams P) {
  __shared__ __align__(16) uint32_t word[kStretch];
  const int b = blockIdx.y, first = blockIdx.x * kStretch;
  const int len = min(kStretch, P.V - first);
  const spec_logit_rules_t& R = P.r;
  const int rows = R.t_per_row ? min(max(__ldg(R.t_per_row + b), 0), P.T) : P.T;
  const float rep = R.repetition ? __ldg(R.repetition + b) : 1.0f;
  const float pre = R.presence ? __ldg(R.presence + b) : 0.0f;
  const float fre = R.frequency ? __ldg(R.frequency + b) : 0.0f;
  const bool penal = rep != 1.0f || pre != 0.0f || fre != 0.0f;

  for (int i = threadIdx.x; i < kStretch; i += kRuleThreads) word[i] = 0;
  __syncthreads();
  if (R.bias_n > 0) {  // of two entries with one id the later holds
    const int32_t* ids = R.bias_ids + (int64_t)b * R.bias_n;
    for (int i = threadIdx.x; i < R.bias_n; i += kRuleThreads) {
      const int64_t v = (int64_t)__ldg(ids + i) - first;
      if (v >= 0 && v < len) atomicMax(&word[v], (uint32_t)(i + 1) << kBiasShift);
    }
    __syncthreads();
  }
  if (penal && R.history) {
    const int held = min(max(__ldg(R.history_len + b), 0), R.history_stride);
    const int prompt = R.prompt_len ? __ldg(R.prompt_len + b) : 0;
    const int32_t* ids = R.history + (int64_t)b * R.history_stride;
    for (int i = threadIdx.x; i < held; i += kRuleThreads) {
      const int64_t v = (int64_t)__ldg(ids + i) - first;
      if (v >= 0 && v < len) {
        if (i < prompt)
          atomicOr(&word[v], kPromptBit);
        else
          atomicAdd(&word[v], 1u);
      }
    }
  }
  __syncthreads();

  using K = Pack<T, VEC>;
  const int64_t base = (int64_t)b * P.T * P.V + first;
  for (int v0 = threadIdx.x * VEC; v0 < len; v0 += kRuleThreads * VEC) {  // VEC > 1: V is a multiple of it
    uint32_t c[VEC], any = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      c[i] = word[v0 + i];
      any |= c[i];
    }
    for (int t = 0; t < rows; ++t) {
      if (penal && R.draft && t > 0) {
        const int64_t d = (int64_t)__ldg(R.draft + (int64_t)b * (P.T - 1) + t - 1) - first - v0;
        if (d >= 0 && d < VEC) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) c[i] += i == (int)d;
          any |= 1;
        }
      }
      const int64_t at = base + (int64_t)t * P.V + v0;
      float x[VEC];
      K::get(*reinterpret_cast<const typename K::W*>(static_cast<const T*>(P.logits) + at), x);
      if (any) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const uint32_t count = c[i] & kCountMask;
          if (penal) {
            if (count > 0 || (c[i] & kPromptBit)) x[i] = x[i] > 0.0f ? x[i] / rep : x[i] * rep;
            if (count > 0) x[i] = x[i] - fre * (float)count - pre;
          }
          const uint32_t e = (c[i] & ~kPromptBit) >> kBiasShift;
          if (e) x[i] += __ldg(R.bias + (int64_t)b * R.bias_n + e - 1);
        }
      }
      if (R.mask) {
        const uint32_t bits =
            (uint32_t)__ldg(R.mask + ((int64_t)b * P.T + t) * P.words + ((first + v0) >> 5)) >> ((first + v0) & 31);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (!((bits >> i) & 1u)) x[i] = -INFINITY;
      }
      *reinterpret_cast<typename K::W*>(static_cast<T*>(P.out) + at) = K::put(x);
    }
  }
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
  const dim3 grid((V + kStretch - 1) / kStretch, B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = (uintptr_t)logits % 16 == 0 && (uintptr_t)out % 16 == 0 && (int64_t)V * es % 16 == 0;
  if (dtype == SPEC_DTYPE_BF16) {
    if (vec) rules_kernel<__nv_bfloat16, 8><<<grid, kRuleThreads, 0, st>>>(P);
    else rules_kernel<__nv_bfloat16, 1><<<grid, kRuleThreads, 0, st>>>(P);
  } else {
    if (vec) rules_kernel<float, 4><<<grid, kRuleThreads, 0, st>>>(P);
    else rules_kernel<float, 1><<<grid, kRuleThreads, 0, st>>>(P);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
