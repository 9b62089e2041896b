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
