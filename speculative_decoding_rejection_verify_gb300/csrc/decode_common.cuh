// decode_common.cuh — what the decode-step operators' translation units share: the batch and cache as
// kernels see them, host-side checks of their structs, and loads, stores and conversions of 8 elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "spec_decode.h"

namespace sv {

// Heads of a batch of tokens (spec_heads_t) as a kernel sees them.
struct Heads {
  char* data;
  int64_t row, token, head;  // strides in bytes
};

struct Cache {
  char* k;
  char* v;
  int64_t layer, page, slot, head;  // strides in bytes
  int num_pages, page_shift;
  const float* k_scale;
  const float* v_scale;
};

struct Batch {
  const int32_t* pages;
  const int32_t* ctx_len;
  const int32_t* t_per_row;
  int B, T, max_pages;
  int slots;  // max_pages * page_size
};

// The request's valid new tokens and its context, clamped into the table (a context that overfills it
// leaves slots past it, which every user of a slot checks).
__device__ __forceinline__ int batch_tokens(const Batch& b, int row) {
  const int t = b.t_per_row ? __ldg(b.t_per_row + row) : b.T;
  return min(max(t, 0), b.T);
}
__device__ __forceinline__ int batch_context(const Batch& b, int row) {
  return min(max(__ldg(b.ctx_len + row), 0), b.slots);
}

// Programmatic dependent launch: a kernel lets the next one of the stream start launching, and waits
// itself until the one before it has finished and its writes are visible.
__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_low(w.x), x[1] = bf16_high(w.x), x[2] = bf16_low(w.y), x[3] = bf16_high(w.y);
  x[4] = bf16_low(w.z), x[5] = bf16_high(w.z), x[6] = bf16_low(w.w), x[7] = bf16_high(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Four E4M3 codes: round to nearest even, what is beyond +-448 cut to it, NaN kept.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four E5M2 codes, likewise.
__device__ __forceinline__ uint32_t pack_e5m2(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E5M2);
  return lo | (hi << 16);
}

// Four E4M3 codes as fp16 pairs, exactly.
__device__ __forceinline__ void e4m3_to_half(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ float4 unpack_e4m3(uint32_t x) {
  uint32_t lo, hi;
  e4m3_to_half(x, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Where slot `slot` of a request lies in the cache: its byte offset within a head, or -1.
__device__ __forceinline__ int64_t slot_offset(const Batch& b, const Cache& c, int row, int slot) {
  if (slot < 0 || slot >= b.slots) return -1;
  const int page = __ldg(b.pages + (int64_t)row * b.max_pages + (slot >> c.page_shift));
  if (page < 0 || page >= c.num_pages) return -1;
  return page * c.page + (slot & ((1 << c.page_shift) - 1)) * c.slot;
}

// x / s for E4M3's rounding: the product with the reciprocal is up to 1.5 units in the last place off, which puts a
// quotient that lies halfway between two codes on either side; corrected by its residual x - q s (P. Markstein, IBM Journal
// of Research and Development 34, 1990) it is the quotient.  For s within 2^+-80 the residual is exact for all quotients
// that are neither under half of the smallest code nor over the largest.  (4 x 2047 tokens, interleaved: 22.5 us without
// the correction, 23.0 with it, 24.9 with divisions.)
__device__ __forceinline__ float quotient(float x, float s, float inverse) {
  const float q = x * inverse;
  return fabsf(q) < 512.0f ? fmaf(fmaf(-q, s, x), inverse, q) : q;  // beyond 448, infinite or NaN: q says it
}

// The same, with -0 kept.
__device__ __forceinline__ float signed_quotient(float x, float s, float inverse) { return x == 0.0f ? x : quotient(x, s, inverse); }

// Page scales (spec_kv_page_scales_t): [layers][num_pages, heads].
struct PageScales {
  float* k;
  float* v;
  int64_t layer;
};
constexpr float kLeastPageScale = 0x1p-24f, kMostPageScale = 0x1p24f;
__device__ __forceinline__ bool scale_counts(float s) { return s >= kLeastPageScale && s <= kMostPageScale; }
// The smallest power of two s in range with most <= 448 s.  448 is 1.75 * 2^8.
__device__ __forceinline__ float scale_need(float most) {
  const int bits = __float_as_int(most);
  const int power = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000);
  return __int_as_float((min(max(power, -24), 24) + 127) << 23);
}

// 16 codes at another scale: each times `ratio`, a power of two in 2^-24 .. 2^15, and rounded.  In fp16 a code and its
// product are exact down to 2^-14, and what is below 2^-10 is 0 whatever its last bits.
__device__ __forceinline__ uint4 rescaled_half(uint4 w, __half2 r) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    e4m3_to_half(x[i], lo, hi);
    const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&lo), r), b = __hmul2(*reinterpret_cast<const __half2*>(&hi), r);
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\tmov.b32 %0, {a, b};\n\t}"
        : "=r"(x[i])
        : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
  }
  return w;
}
__device__ __forceinline__ bool half_ratio(float ratio) {  // whether rescaled_half does it
  return (__float_as_int(ratio) & 0x7FFFFF) == 0 && ratio >= 0x1p-24f && ratio <= 0x1p15f;
}
// The same for any ratio.
__device__ __forceinline__ uint4 rescaled(uint4 w, float ratio) {
  if (half_ratio(ratio)) return rescaled_half(w, __float2half2_rn(ratio));
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = unpack_e4m3(x[i]);
    x[i] = pack_e4m3(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio);
  }
  return w;
}

// Weights and positions of the cache's entries (spec_kv_record_t): [layers][num_pages, heads, page_size].
struct Record {
  float* weight;
  int32_t* position;
  int64_t layer;
};

// ------------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------------
inline bool heads_ok(const spec_heads_t* h) {
  return h && h->data && ((uintptr_t)h->data & 15u) == 0 && h->row_stride % 8 == 0 && h->token_stride % 8 == 0 &&
         h->head_stride % 8 == 0 && h->row_stride >= 0 && h->token_stride >= 0 && h->head_stride >= 0;
}
inline Heads heads_of(const spec_heads_t* h) {
  if (!h) return Heads{nullptr, 0, 0, 0};
  return Heads{static_cast<char*>(h->data), h->row_stride * 2, h->token_stride * 2, h->head_stride * 2};
}

inline spec_status_t check_cache(const spec_kv_cache_t* c, bool scales) {
  if (!c) return SPEC_ERR_INVALID_ARG;
  if (c->layers < 1 || c->num_pages < 1 || c->heads < 1 || c->page_size < 1) return SPEC_ERR_INVALID_ARG;
  if (c->dtype != SPEC_DTYPE_BF16 && c->dtype != SPEC_DTYPE_E4M3) return SPEC_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > SPEC_MAX_PAGE || (c->page_size & (c->page_size - 1)))
    return SPEC_ERR_UNSUPPORTED;
  if (c->heads > 65535) return SPEC_ERR_UNSUPPORTED;
  if (!c->k || !c->v) return SPEC_ERR_INVALID_ARG;
  const int vec = c->dtype == SPEC_DTYPE_BF16 ? 8 : 16;
  if (((uintptr_t)c->k & 15u) || ((uintptr_t)c->v & 15u) || c->layer_stride % vec || c->page_stride % vec ||
      c->slot_stride % vec || c->head_stride % vec)
    return SPEC_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0 || c->layer_stride < 0) return SPEC_ERR_INVALID_ARG;
  if (scales && c->dtype != SPEC_DTYPE_E4M3 && (c->k_scale || c->v_scale)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}
inline Cache cache_of(const spec_kv_cache_t* c) {
  const int64_t es = c->dtype == SPEC_DTYPE_BF16 ? 2 : 1;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  return Cache{static_cast<char*>(c->k), static_cast<char*>(c->v), c->layer_stride * es, c->page_stride * es,
               c->slot_stride * es, c->head_stride * es, c->num_pages, shift, c->k_scale, c->v_scale};
}

// scales may be NULL
inline spec_status_t check_scales(const spec_kv_page_scales_t* s, const spec_kv_cache_t* c) {
  if (!s) return SPEC_OK;
  if (c->dtype != SPEC_DTYPE_E4M3 || c->k_scale || c->v_scale) return SPEC_ERR_INVALID_ARG;
  if (!s->k || !s->v || ((uintptr_t)s->k & 3u) || ((uintptr_t)s->v & 3u) || s->layer_stride < 0) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}
inline PageScales scales_of(const spec_kv_page_scales_t* s) { return s ? PageScales{s->k, s->v, s->layer_stride} : PageScales{}; }

// The sizes of a record alone; with a cache, whether they are the cache's.
inline spec_status_t check_record(const spec_kv_record_t* r, const spec_kv_cache_t* c) {
  if (!r) return SPEC_OK;
  if (((uintptr_t)r->weight & 3u) || ((uintptr_t)r->position & 3u) || r->layer_stride < 0) return SPEC_ERR_INVALID_ARG;
  if (r->layers < 1 || r->num_pages < 1 || r->heads < 1 || r->page_size < 1) return SPEC_ERR_INVALID_ARG;
  if (r->page_size < 8 || r->page_size > SPEC_MAX_PAGE || (r->page_size & (r->page_size - 1)) || r->heads > 65535)
    return SPEC_ERR_UNSUPPORTED;
  if (c && (r->layers != c->layers || r->num_pages != c->num_pages || r->page_size != c->page_size || r->heads != c->heads))
    return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}
inline Record record_of(const spec_kv_record_t* r) { return r ? Record{r->weight, r->position, r->layer_stride} : Record{}; }

// B = 0 is an empty batch: nothing is read.
inline spec_status_t check_batch(const spec_decode_batch_t* b, const spec_kv_cache_t* c) {
  if (!b || b->B < 0 || b->T < 0 || b->max_pages < 0) return SPEC_ERR_INVALID_ARG;
  if ((int64_t)b->max_pages * c->page_size > SPEC_MAX_SLOTS || b->T > SPEC_MAX_SLOTS) return SPEC_ERR_UNSUPPORTED;
  if (b->B > 0 && (!b->ctx_len || (b->max_pages > 0 && !b->pages))) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}
inline Batch batch_of(const spec_decode_batch_t* b, const spec_kv_cache_t* c) {
  return Batch{b->pages, b->ctx_len, b->t_per_row, b->B, b->T, b->max_pages, b->max_pages * c->page_size};
}

// Launches a kernel that begins with pdl_wait: its blocks may come up while the kernel before it drains.
template <typename P>
inline cudaError_t launch_early(void (*kern)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, params);
}

// The current device and its SMs (looked up once per device).
constexpr int kMaxGpus = 64;
inline cudaError_t device_sms(int* dev, int* sms) {
  static std::atomic<int> known[kMaxGpus];
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= kMaxGpus) return cudaErrorInvalidDevice;
  *sms = known[*dev].load(std::memory_order_relaxed);
  if (*sms == 0) {
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess) known[*dev].store(*sms, std::memory_order_relaxed);
  }
  return e;
}

}  // namespace sv
