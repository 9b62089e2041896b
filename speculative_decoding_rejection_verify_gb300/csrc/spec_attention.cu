// spec_attention.cu — spec_paged_attention: the new tokens of a step attend over the paged cache.

#include "decode_common.cuh"

namespace sv {

constexpr int kRowWarps = 4;

struct AttnParams {
  Heads q, out;
  Cache cache;
  Batch batch;
  const int64_t* mask;
  int q_heads, group;
  float scale;
};

// One block per query row; each warp takes every kRowWarps-th slot with its own running maximum, and the
// warps' parts are joined at the end.
template <int D, bool F8>
__global__ void __launch_bounds__(kRowWarps * 32) attn_row_kernel(const __grid_constant__ AttnParams P) {
  constexpr int E = D / 32;  // elements per lane
  __shared__ float part[kRowWarps][D + 2];
  const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tb = batch_tokens(P.batch, b), ctx = batch_context(P.batch, b);
  char* out = P.out.data + b * P.out.row + t * P.out.token + h * P.out.head;
  float m = -INFINITY, l = 0.0f, o[E] = {};
  if (t < tb) {
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(P.q.data + b * P.q.row + t * P.q.token + h * P.q.head);
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __bfloat162float(q[lane + 32 * i]);
    const int kvh = h / P.group;
    const float ks = F8 && P.cache.k_scale ? P.cache.k_scale[kvh] : 1.0f;
    const float vs = F8 && P.cache.v_scale ? P.cache.v_scale[kvh] : 1.0f;
    const uint64_t rule = P.mask ? (uint64_t)P.mask[(int64_t)b * P.batch.T + t] : (t >= 63 ? ~0ull : (2ull << t) - 1);
    const int end = min(ctx + tb, P.batch.slots);
    for (int s = warp; s < end; s += kRowWarps) {
      if (s >= ctx && !((rule >> (s - ctx)) & 1)) continue;
      const int page = P.batch.pages[(int64_t)b * P.batch.max_pages + (s >> P.cache.page_shift)];
      const bool in = page >= 0 && page < P.cache.num_pages;
      const int64_t at = page * P.cache.page + (s & ((1 << P.cache.page_shift) - 1)) * P.cache.slot + kvh * P.cache.head;
      float dot = 0.0f, v[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        float k = 0.0f;
        v[i] = 0.0f;
        if (in) {
          if constexpr (F8) {
            k = (float)reinterpret_cast<const __nv_fp8_e4m3*>(P.cache.k + at)[lane + 32 * i] * ks;
            v[i] = (float)reinterpret_cast<const __nv_fp8_e4m3*>(P.cache.v + at)[lane + 32 * i] * vs;
          } else {
            k = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(P.cache.k + at)[lane + 32 * i]);
            v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(P.cache.v + at)[lane + 32 * i]);
          }
        }
        dot += x[i] * k;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
      const float z = dot * P.scale;
      const float top = fmaxf(m, z), base = top == -INFINITY ? 0.0f : top;
      const float keep = expf(m - base), w = expf(z - base);
      l = l * keep + w;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * v[i];
      m = top;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) part[warp][lane + 32 * i] = o[i];
  if (lane == 0) part[warp][D] = m, part[warp][D + 1] = l;
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kRowWarps * 32) {
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, part[w][D]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kRowWarps; ++w) {
      const float f = expf(part[w][D] - base);
      sum += f * part[w][D + 1];
      acc += f * part[w][d];
    }
    reinterpret_cast<__nv_bfloat16*>(out)[d] = __float2bfloat16(sum == 0.0f ? 0.0f : acc / sum);
  }
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_paged_attention_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t heads, int32_t head_dim) {
  if (B < 0 || T < 0 || T > SPEC_MAX_NEW || heads < 1 || q_heads < 1 || q_heads % heads) return 0;
  if (q_heads / heads > SPEC_MAX_GROUP) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return 256;
}

spec_status_t spec_paged_attention(const spec_heads_t* q, const spec_heads_t* out, int32_t q_heads,
                                   const spec_kv_cache_t* cache, const spec_decode_batch_t* batch,
                                   const int64_t* mask, float scale, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  spec_status_t s = check_cache(cache, true);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (q_heads < 1 || q_heads % cache->heads || !isfinite(scale)) return SPEC_ERR_INVALID_ARG;
  if (batch->T > SPEC_MAX_NEW || batch->B > 65535 || q_heads / cache->heads > SPEC_MAX_GROUP) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0 || batch->T == 0) return SPEC_OK;
  if (!heads_ok(q) || !heads_ok(out)) return SPEC_ERR_INVALID_ARG;
  const size_t need = spec_paged_attention_workspace_bytes(batch->B, batch->T, q_heads, cache->heads, cache->head_dim);
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < need) return SPEC_ERR_WORKSPACE;
  AttnParams P = {};
  P.q = heads_of(q), P.out = heads_of(out);
  P.cache = cache_of(cache);
  P.batch = batch_of(batch, cache);
  P.mask = mask;
  P.q_heads = q_heads, P.group = q_heads / cache->heads;
  P.scale = scale;
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  auto kern = cache->head_dim == 128 ? (f8 ? attn_row_kernel<128, true> : attn_row_kernel<128, false>)
                                     : (f8 ? attn_row_kernel<64, true> : attn_row_kernel<64, false>);
  kern<<<dim3(q_heads, batch->T, batch->B), kRowWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
