// spec_evict.cu — which entries of a cache attention looks at, and which stay: spec_kv_weigh adds up the weights that the
// new tokens of a step give every entry, spec_kv_select picks a head's entries of largest weight.

#include "decode_common.cuh"

namespace sv {

// ------------------------------------------------------------------------------------------------
// spec_kv_weigh
// ------------------------------------------------------------------------------------------------
struct WeighParams {
  Heads q;
  Cache cache;
  PageScales scales;
  Record record;
  Batch batch;
  const int64_t* mask;
  const float* lse;
  const int32_t* positions;
  int heads, group;
  float scale;
};

constexpr int kWeighRows = 16;  // rows of q in shared memory at a time

// A thread per slot, its key in registers; rows of q go by in shared memory.
template <int D, bool F8>
__global__ void __launch_bounds__(128) weigh_kernel(const __grid_constant__ WeighParams P) {
  __shared__ float4 rows[kWeighRows][D / 4];
  __shared__ float lse[kWeighRows];
  pdl_launch_next();
  pdl_wait();
  for (int item = blockIdx.y; item < P.batch.B * P.heads; item += gridDim.y) {
    const int b = item / P.heads, head = item % P.heads;
    const int tb = batch_tokens(P.batch, b), ctx = batch_context(P.batch, b);
    const int end = (int)min((int64_t)ctx + tb, (int64_t)P.batch.slots);
    if (tb == 0) continue;
    for (int slot0 = blockIdx.x * 128; slot0 < end; slot0 += gridDim.x * 128) {
      const int slot = slot0 + threadIdx.x;
      float4 k[D / 4];
      int page = -1;
      if (slot < end) {
        page = __ldg(P.batch.pages + (int64_t)b * P.batch.max_pages + (slot >> P.cache.page_shift));
        if (page < 0 || page >= P.cache.num_pages) page = -1;
      }
      float scale = P.scale;
      if (page >= 0) {
        const char* p = P.cache.k + page * P.cache.page + (slot & ((1 << P.cache.page_shift) - 1)) * P.cache.slot + head * P.cache.head;
        if constexpr (F8) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + i * 16);
            k[4 * i] = unpack_e4m3(w.x), k[4 * i + 1] = unpack_e4m3(w.y), k[4 * i + 2] = unpack_e4m3(w.z), k[4 * i + 3] = unpack_e4m3(w.w);
          }
          if (P.scales.k) {
            const float s = P.scales.k[(int64_t)page * P.heads + head];
            scale *= scale_counts(s) ? s : NAN;
          } else if (P.cache.k_scale) {
            scale *= __ldg(P.cache.k_scale + head);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            float x[8];
            unpack8(*reinterpret_cast<const uint4*>(p + i * 16), x);
            k[2 * i] = make_float4(x[0], x[1], x[2], x[3]), k[2 * i + 1] = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      }
      float sum = 0.0f;
      for (int r0 = 0; r0 < tb * P.group; r0 += kWeighRows) {
        __syncthreads();
        const int n = min(kWeighRows, tb * P.group - r0);
        for (int u = threadIdx.x; u < n * (D / 8); u += 128) {
          const int r = r0 + u / (D / 8), t = r / P.group, g = r % P.group;
          float x[8];
          unpack8(*reinterpret_cast<const uint4*>(P.q.data + b * P.q.row + t * P.q.token + (int64_t)(head * P.group + g) * P.q.head + u % (D / 8) * 16), x);
          rows[u / (D / 8)][u % (D / 8) * 2] = make_float4(x[0], x[1], x[2], x[3]);
          rows[u / (D / 8)][u % (D / 8) * 2 + 1] = make_float4(x[4], x[5], x[6], x[7]);
        }
        if (threadIdx.x < n) {
          const int r = r0 + threadIdx.x, t = r / P.group, g = r % P.group;
          const float x = P.lse[((int64_t)b * P.batch.T + t) * (P.heads * P.group) + head * P.group + g];
          lse[threadIdx.x] = x == -INFINITY ? INFINITY : x;
        }
        __syncthreads();
        if (page >= 0)
          for (int r = 0; r < n; ++r) {
            const int t = (r0 + r) / P.group, fresh = slot - ctx;
            if (fresh >= 0 && !(P.mask ? (P.mask[(int64_t)b * P.batch.T + t] >> fresh) & 1 : fresh <= t)) continue;
            if (lse[r] == INFINITY) continue;
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
              const float4 q = rows[r][i];
              z += q.x * k[i].x + q.y * k[i].y + q.z * k[i].z + q.w * k[i].w;
            }
            sum += expf(z * scale - lse[r]);
          }
      }
      if (page >= 0) {
        const int64_t at = (((int64_t)page * P.heads + head) << P.cache.page_shift) + (slot & ((1 << P.cache.page_shift) - 1));
        P.record.weight[at] = (slot < ctx ? P.record.weight[at] : 0.0f) + sum;
        if (slot >= ctx && P.record.position) P.record.position[at] = P.positions ? P.positions[(int64_t)b * P.batch.T + slot - ctx] : slot;
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// spec_kv_select
// ------------------------------------------------------------------------------------------------
struct SelectParams {
  Record record;
  Batch batch;
  const int32_t* budget;
  const int32_t* seen;
  int32_t* source;
  int32_t* target;
  int32_t* moves;
  int32_t* new_len;
  int heads, num_pages, page_shift, first, recent, max_moves;
};

constexpr int kSelectThreads = 1024;

// A block per (layer, request, head): the budget-th largest key by its digits of 8 bits from the top, then one pass in the
// order of the slots that numbers the ties and the moves.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams P) {
  __shared__ int bins[256];
  __shared__ int digit, above;
  __shared__ int sums[3][32];
  pdl_launch_next();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int list = blockIdx.x, head = list % P.heads, rest = list / P.heads, b = rest % P.batch.B, layer = rest / P.batch.B;
  const int ctx = batch_context(P.batch, b), m = min(ctx, max(__ldg(P.budget + b), 0));
  if (threadIdx.x == 0 && head == 0 && layer == 0) P.new_len[b] = m;
  if (m == ctx || m == 0) {
    if (threadIdx.x == 0) P.moves[list] = 0;
    return;
  }
  // positions from here on stay
  const int64_t recent = P.recent > 0 ? (int64_t)(P.seen ? __ldg(P.seen + b) : ctx) - P.recent : INT64_MAX;
  const int32_t* table = P.batch.pages + (int64_t)b * P.batch.max_pages;
  const int mask = (1 << P.page_shift) - 1;
  const int64_t base = layer * P.record.layer;
  // A larger key is a larger weight; +0 and -0 are one.
  const auto key_of = [&](int slot) -> uint32_t {
    const int page = __ldg(table + (slot >> P.page_shift));
    float w = -INFINITY;
    if (page >= 0 && page < P.num_pages) {
      const int64_t at = base + (((int64_t)page * P.heads + head) << P.page_shift) + (slot & mask);
      w = P.record.weight[at] + 0.0f;
      if (w != w) w = -INFINITY;
      if (P.record.position) {
        const int position = P.record.position[at];
        if (position < P.first || position >= recent) w = INFINITY;
      }
    }
    const uint32_t bits = __float_as_uint(w);
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
  };
  uint32_t prefix = 0;
  int left = m;  // of the keys that agree with the prefix, how many stay
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSelectThreads) bins[i] = 0;
    __syncthreads();
    for (int slot = threadIdx.x; slot < ctx; slot += kSelectThreads) {
      const uint32_t key = key_of(slot);
      if (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&bins[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {  // the bin that holds the left-th key from the top
      int mine = 0;
      for (int i = 0; i < 8; ++i) mine += bins[255 - lane * 8 - i];
      int before = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(~0u, before, d);
        if (lane >= d) before += x;
      }
      before -= mine;
      if (before < left && before + mine >= left) {
        int i = 255 - lane * 8;
        while (before + bins[i] < left) before += bins[i--];
        digit = i, above = before;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)digit << shift;
    left -= above;
    __syncthreads();
  }
  // `left` of the keys equal to prefix stay, the lowest slots first
  int ties = 0, sources = 0, targets = 0;  // in the slots before
  int32_t* source = P.source + (int64_t)list * P.max_moves;
  int32_t* target = P.target + (int64_t)list * P.max_moves;
  for (int slot0 = 0; slot0 < ctx; slot0 += kSelectThreads) {
    const int slot = slot0 + threadIdx.x;
    const uint32_t key = slot < ctx ? key_of(slot) : 0;
    const bool tie = slot < ctx && key == prefix;
    const uint32_t tied = __ballot_sync(~0u, tie);
    if (lane == 0) sums[0][warp] = __popc(tied);
    __syncthreads();
    int before = ties, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += sums[0][w];
      all += sums[0][w];
    }
    const bool stays = slot < ctx && (key > prefix || (tie && before + __popc(tied & ((1u << lane) - 1)) < left));
    const bool is_source = stays && slot >= m, is_target = slot < m && !stays;
    const uint32_t s = __ballot_sync(~0u, is_source), t = __ballot_sync(~0u, is_target);
    if (lane == 0) sums[1][warp] = __popc(s), sums[2][warp] = __popc(t);
    __syncthreads();
    int at_s = sources, at_t = targets;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at_s += sums[1][w], at_t += sums[2][w];
      sources += sums[1][w], targets += sums[2][w];
    }
    at_s += __popc(s & ((1u << lane) - 1)), at_t += __popc(t & ((1u << lane) - 1));
    if (is_source && at_s < P.max_moves) source[at_s] = slot;
    if (is_target && at_t < P.max_moves) target[at_t] = slot;
    ties += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) P.moves[list] = min(sources, P.max_moves);
}

}  // namespace sv

using namespace sv;

extern "C" {

spec_status_t spec_kv_weigh(const spec_heads_t* q, int32_t q_heads, const spec_kv_cache_t* given,
                            const spec_kv_page_scales_t* scales, const spec_decode_batch_t* batch, const int64_t* mask,
                            float scale, const float* lse, const spec_kv_record_t* record, const int32_t* positions,
                            void* stream) {
  if (!given) return SPEC_ERR_INVALID_ARG;
  spec_kv_cache_t keys = *given;
  keys.v = keys.k, keys.v_scale = keys.k_scale;
  const spec_kv_cache_t* cache = &keys;
  spec_status_t s = check_cache(cache, true);
  spec_kv_page_scales_t only;
  if (scales) {
    only = *scales, only.v = only.k;
    scales = &only;
  }
  if (s == SPEC_OK) s = check_scales(scales, cache);
  if (s == SPEC_OK) s = check_record(record, cache);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (q_heads < 1 || q_heads % cache->heads || !isfinite(scale) || !record || !record->weight) return SPEC_ERR_INVALID_ARG;
  if (batch->T > SPEC_MAX_NEW || batch->B > SPEC_MAX_BATCH || q_heads / cache->heads > SPEC_MAX_GROUP) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0 || batch->T == 0) return SPEC_OK;
  if (!heads_ok(q) || !lse) return SPEC_ERR_INVALID_ARG;
  WeighParams P = {};
  P.q = heads_of(q), P.cache = cache_of(cache), P.scales = scales_of(scales), P.record = record_of(record), P.batch = batch_of(batch, cache);
  P.mask = mask, P.lse = lse, P.positions = positions;
  P.heads = cache->heads, P.group = q_heads / cache->heads, P.scale = scale;
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  auto kern = cache->head_dim == 128 ? (f8 ? weigh_kernel<128, true> : weigh_kernel<128, false>)
                                     : (f8 ? weigh_kernel<64, true> : weigh_kernel<64, false>);
  const int64_t items = (int64_t)batch->B * cache->heads, tiles = ((int64_t)P.batch.slots + 127) / 128;
  if (tiles == 0) return SPEC_OK;
  const unsigned y = (unsigned)(items < 65535 ? items : 65535), x = (unsigned)(tiles < 1024 ? tiles : 1024);
  return launch_early(kern, dim3(x, y), dim3(128), 0, static_cast<cudaStream_t>(stream), P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status_t spec_kv_select(const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* budget,
                             const int32_t* seen, int32_t first, int32_t recent, int32_t* source, int32_t* target,
                             int32_t max_moves, int32_t* moves, int32_t* new_len, void* stream) {
  if (!record) return SPEC_ERR_INVALID_ARG;
  spec_status_t s = check_record(record, nullptr);
  if (s != SPEC_OK) return s;
  spec_kv_cache_t sizes = {};
  sizes.page_size = record->page_size;
  s = check_batch(batch, &sizes);
  if (s != SPEC_OK) return s;
  if (first < 0 || recent < 0 || max_moves < 0 || !record->weight || ((first > 0 || recent > 0) && !record->position))
    return SPEC_ERR_INVALID_ARG;
  const int64_t lists = (int64_t)record->layers * batch->B * record->heads;
  if (lists > 0x3fffffffll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0) return SPEC_OK;
  if ((int64_t)max_moves < (int64_t)batch->max_pages * record->page_size / 2) return SPEC_ERR_INVALID_ARG;
  if (!budget || !moves || !new_len || (max_moves > 0 && (!source || !target))) return SPEC_ERR_INVALID_ARG;
  SelectParams P = {};
  P.record = record_of(record);
  if (first == 0 && recent == 0) P.record.position = nullptr;
  P.batch = batch_of(batch, &sizes);
  P.budget = budget, P.seen = seen, P.source = source, P.target = target, P.moves = moves, P.new_len = new_len;
  P.heads = record->heads, P.num_pages = record->num_pages, P.first = first, P.recent = recent, P.max_moves = max_moves;
  while ((1 << P.page_shift) < record->page_size) ++P.page_shift;
  return launch_early(select_kernel, dim3((unsigned)lists), dim3(kSelectThreads), 0, static_cast<cudaStream_t>(stream), P) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // extern "C"
