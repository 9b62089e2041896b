// spec_kv.cu — the writes to the paged key-value cache: spec_kv_append (the new tokens' rotated keys and
// their values, with the queries rotated on the way) and spec_kv_keep (the accepted branch moved up
// behind the context).  Both are streams of 16-byte vectors, bound by memory traffic on large calls and
// by their launch on small ones.

#include "decode_common.cuh"

namespace sv {

constexpr int kAppendThreads = 256;

struct AppendParams {
  Heads q, k, v, q_out;
  Cache cache;
  Batch batch;
  const float* cos_table;
  const float* sin_table;
  const int32_t* positions;
  int32_t* flags;
  int q_heads, heads;      // heads of q; heads of k (and of v)
  int rot, max_positions;  // rot = rot_dim
  int per_task;            // heads that one thread takes in turn
  int tasks;               // ceil((q_heads + 2 heads) / per_task)
  int64_t total;           // B * T * tasks * units
};

// Where new token t of a request goes in the cache: its byte offset within a head, or -1.
__device__ __forceinline__ int64_t slot_offset(const Batch& b, const Cache& c, int row, int slot) {
  if (slot < 0 || slot >= b.slots) return -1;
  const int page = __ldg(b.pages + (int64_t)row * b.max_pages + (slot >> c.page_shift));
  if (page < 0 || page >= c.num_pages) return -1;
  return page * c.page + (slot & ((1 << c.page_shift) - 1)) * c.slot;
}

// 8 elements of a key or value into the cache.
template <bool F8>
__device__ __forceinline__ void store_entry(char* p, float (&x)[8], float scale) {
  if constexpr (F8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] / scale;
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
  } else {
    *reinterpret_cast<uint4*>(p) = pack8(x);
  }
}

// One thread owns one unit of the head dimension -- the 8 elements at `lo`, and with half-split rotation
// also their partners at lo + rot/2 -- for per_task heads of one token, so a token's cos and sin are loaded
// once for them, and an element's partner is always in the same thread (q_out may be q itself).
template <int D, bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams P) {
  const int paired = INTERLEAVED ? 0 : P.rot / 16;  // units that hold a vector and its partner
  const int units = D / 8 - paired;
  const int64_t id = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  if (id >= P.total) return;
  const int unit = (int)(id % units);
  const int64_t rest = id / units;
  const int task = (int)(rest % P.tasks);
  const int64_t token = rest / P.tasks;
  const int b = (int)(token / P.batch.T), t = (int)(token % P.batch.T);
  const int h_end = min((task + 1) * P.per_task, P.q_heads + 2 * P.heads);
  int h = task * P.per_task;

  const bool pair = unit < paired;
  const int lo = pair || INTERLEAVED ? unit * 8 : P.rot + (unit - paired) * 8;
  const bool turns = pair || (INTERLEAVED && lo < P.rot);
  const int tb = batch_tokens(P.batch, b);
  if (t >= tb) {  // a padded token: its rotated query is 0
    for (; h < h_end && h < P.q_heads; ++h) {
      char* o = P.q_out.data + b * P.q_out.row + t * P.q_out.token + h * P.q_out.head;
      *reinterpret_cast<uint4*>(o + lo * 2) = make_uint4(0, 0, 0, 0);
      if (pair) *reinterpret_cast<uint4*>(o + (lo + P.rot / 2) * 2) = make_uint4(0, 0, 0, 0);
    }
    if (P.flags && t == P.batch.T - 1 && task == 0 && unit == 0 && P.batch.t_per_row &&
        __ldg(P.batch.t_per_row + b) < 0)
      atomicOr(P.flags + b, SPEC_FLAG_BAD_K);
    return;
  }
  const int ctx = batch_context(P.batch, b);
  const int64_t at = slot_offset(P.batch, P.cache, b, ctx + t);
  int flag = at < 0 ? SPEC_FLAG_BAD_SLOT : 0;
  if (P.flags && P.batch.t_per_row && __ldg(P.batch.t_per_row + b) > P.batch.T) flag |= SPEC_FLAG_BAD_K;
  if (P.flags && __ldg(P.batch.ctx_len + b) < 0) flag |= SPEC_FLAG_BAD_SLOT;

  // cos and sin of the unit: 8 pairs half-split, 4 pairs interleaved
  float co[8], si[8];
  if (P.rot > 0) {
    int pos = P.positions ? __ldg(P.positions + (int64_t)b * P.batch.T + t) : ctx + t;
    if (pos < 0 || pos >= P.max_positions) {
      flag |= SPEC_FLAG_BAD_POSITION;
      pos = min(max(pos, 0), P.max_positions - 1);
    }
    if (turns) {
      const int64_t base = (int64_t)pos * (P.rot / 2) + (INTERLEAVED ? lo / 2 : lo);
#pragma unroll
      for (int i = 0; i < (INTERLEAVED ? 4 : 8); i += 4) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(P.cos_table + base + i));
        const float4 s = __ldg(reinterpret_cast<const float4*>(P.sin_table + base + i));
        co[i] = c.x, co[i + 1] = c.y, co[i + 2] = c.z, co[i + 3] = c.w;
        si[i] = s.x, si[i + 1] = s.y, si[i + 2] = s.z, si[i + 3] = s.w;
      }
    }
  }
  if (P.flags && flag && task == 0 && unit == 0) atomicOr(P.flags + b, flag);

  const int far = P.rot / 2;  // distance to the partner
  for (; h < h_end; ++h) {
    const bool is_q = h < P.q_heads;
    const bool is_k = !is_q && h < P.q_heads + P.heads;
    const int hh = is_q ? h : is_k ? h - P.q_heads : h - P.q_heads - P.heads;
    if (!is_q && at < 0) break;  // k and v heads follow the q heads
    const Heads& in = is_q ? P.q : is_k ? P.k : P.v;
    const char* p = in.data + b * in.row + t * in.token + hh * in.head;
    const uint4 w0 = *reinterpret_cast<const uint4*>(p + lo * 2);
    uint4 w1 = make_uint4(0, 0, 0, 0);
    if (pair) w1 = *reinterpret_cast<const uint4*>(p + (lo + far) * 2);
    float x[8], y[8];
    unpack8(w0, x);
    unpack8(w1, y);
    if (turns && (is_q || is_k)) {
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], c = x[2 * i + 1];
          x[2 * i] = a * co[i] - c * si[i];
          x[2 * i + 1] = c * co[i] + a * si[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[i], c = y[i];
          x[i] = a * co[i] - c * si[i];
          y[i] = c * co[i] + a * si[i];
        }
      }
    }
    if (is_q) {
      char* o = P.q_out.data + b * P.q_out.row + t * P.q_out.token + hh * P.q_out.head;
      *reinterpret_cast<uint4*>(o + lo * 2) = pack8(x);
      if (pair) *reinterpret_cast<uint4*>(o + (lo + far) * 2) = pack8(y);
    } else {
      constexpr int ES = F8 ? 1 : 2;
      const float* scales = is_k ? P.cache.k_scale : P.cache.v_scale;
      const float scale = F8 && scales ? __ldg(scales + hh) : 1.0f;
      char* o = (is_k ? P.cache.k : P.cache.v) + at + hh * P.cache.head;
      store_entry<F8>(o + lo * ES, x, scale);
      if (pair) store_entry<F8>(o + (lo + far) * ES, y, scale);
    }
  }
}

// ------------------------------------------------------------------------------------------------
// spec_kv_keep
// ------------------------------------------------------------------------------------------------
struct KeepParams {
  Cache cache;
  Batch batch;
  const int32_t* path;
  const int32_t* n_keep;
  int max_keep, heads, vecs;  // 16-byte vectors per head
  int64_t total;              // layers * B * 2 * heads * vecs
};

constexpr int kKeepThreads = 256;

// One thread owns one 16-byte column of one request's entries (layer, k or v, head, vector) and moves it
// through the path in order.  A strictly increasing path has path[i] >= i, so what move i overwrites
// (slot i) is never read by a later move: loads may run ahead of stores, and columns are independent.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams P) {
  const int64_t id = (int64_t)blockIdx.x * kKeepThreads + threadIdx.x;
  if (id >= P.total) return;
  const int vec = (int)(id % P.vecs);
  int64_t rest = id / P.vecs;
  const int h = (int)(rest % P.heads);
  rest /= P.heads;
  const bool is_v = rest & 1;
  rest >>= 1;
  const int b = (int)(rest % P.batch.B);
  const int64_t layer = rest / P.batch.B;
  const int n = min(max(__ldg(P.n_keep + b), 0), P.max_keep);
  const int ctx = batch_context(P.batch, b);
  char* column = (is_v ? P.cache.v : P.cache.k) + layer * P.cache.layer + h * P.cache.head + vec * 16;
  for (int i = 0; i < n; ++i) {
    const int from = __ldg(P.path + (int64_t)b * P.max_keep + i);
    if (from == i || from < 0 || from >= P.batch.slots) continue;
    const int64_t src = ctx + from >= 0 ? slot_offset(P.batch, P.cache, b, ctx + from) : -1;
    const int64_t dst = slot_offset(P.batch, P.cache, b, ctx + i);
    if (src < 0 || dst < 0) continue;
    *reinterpret_cast<uint4*>(column + dst) = *reinterpret_cast<const uint4*>(column + src);
  }
}

}  // namespace sv

using namespace sv;

extern "C" {

spec_status_t spec_kv_append(const spec_heads_t* q, const spec_heads_t* k, const spec_heads_t* v,
                             const spec_heads_t* q_out, int32_t q_heads, const spec_kv_cache_t* cache,
                             const spec_decode_batch_t* batch, const spec_rotary_t* rotary, int32_t* out_flags,
                             void* stream) {
  spec_status_t s = check_cache(cache, true);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (q_heads < 0 || (q_heads == 0) != (q == nullptr) || (q_heads == 0) != (q_out == nullptr))
    return SPEC_ERR_INVALID_ARG;
  const int rot = rotary ? rotary->rot_dim : 0;
  if (rot < 0 || rot > cache->head_dim || rot % 16) return SPEC_ERR_INVALID_ARG;
  if (rot > 0 && (!rotary->cos_table || !rotary->sin_table || rotary->max_positions < 1 ||
                  ((uintptr_t)rotary->cos_table & 15u) || ((uintptr_t)rotary->sin_table & 15u)))
    return SPEC_ERR_INVALID_ARG;
  if (batch->B == 0 || batch->T == 0) return SPEC_OK;
  if (!heads_ok(k) || !heads_ok(v) || (q && (!heads_ok(q) || !heads_ok(q_out)))) return SPEC_ERR_INVALID_ARG;

  AppendParams P = {};
  P.q = heads_of(q), P.k = heads_of(k), P.v = heads_of(v), P.q_out = heads_of(q_out);
  P.cache = cache_of(cache);
  P.batch = batch_of(batch, cache);
  P.rot = rot;
  if (rot > 0) {
    P.cos_table = rotary->cos_table, P.sin_table = rotary->sin_table;
    P.positions = rotary->positions, P.max_positions = rotary->max_positions;
  }
  P.flags = out_flags;
  P.q_heads = q_heads, P.heads = cache->heads;
  const bool inter = rot > 0 && rotary->interleaved != 0;
  const int units = cache->head_dim / 8 - (inter ? 0 : rot / 16);
  const int all = q_heads + 2 * cache->heads;
  P.per_task = 4;
  P.tasks = (all + P.per_task - 1) / P.per_task;
  P.total = (int64_t)batch->B * batch->T * P.tasks * units;
  const int64_t blocks = (P.total + kAppendThreads - 1) / kAppendThreads;
  if (blocks > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  auto kern = cache->head_dim == 128
                  ? (f8 ? (inter ? append_kernel<128, true, true> : append_kernel<128, true, false>)
                        : (inter ? append_kernel<128, false, true> : append_kernel<128, false, false>))
                  : (f8 ? (inter ? append_kernel<64, true, true> : append_kernel<64, true, false>)
                        : (inter ? append_kernel<64, false, true> : append_kernel<64, false, false>));
  kern<<<(unsigned)blocks, kAppendThreads, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status_t spec_kv_keep(const spec_kv_cache_t* cache, const spec_decode_batch_t* batch, const int32_t* path,
                           const int32_t* n_keep, int32_t max_keep, void* stream) {
  spec_status_t s = check_cache(cache, false);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (max_keep < 0) return SPEC_ERR_INVALID_ARG;
  if (batch->B == 0 || max_keep == 0) return SPEC_OK;
  if (!path || !n_keep) return SPEC_ERR_INVALID_ARG;
  KeepParams P = {};
  P.cache = cache_of(cache);
  P.batch = batch_of(batch, cache);
  P.path = path, P.n_keep = n_keep, P.max_keep = max_keep;
  P.heads = cache->heads;
  P.vecs = cache->head_dim * (cache->dtype == SPEC_DTYPE_BF16 ? 2 : 1) / 16;
  P.total = (int64_t)cache->layers * batch->B * 2 * P.heads * P.vecs;
  const int64_t blocks = (P.total + kKeepThreads - 1) / kKeepThreads;
  if (blocks > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  keep_kernel<<<(unsigned)blocks, kKeepThreads, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
