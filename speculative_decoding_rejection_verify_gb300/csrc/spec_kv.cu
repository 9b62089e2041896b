// spec_kv.cu — the writes to the paged key-value cache: spec_kv_append (the new tokens' rotated keys and
// their values, with the queries rotated on the way) and spec_kv_keep (the accepted branch moved up
// behind the context).  Both are streams of 16-byte vectors, bound by memory traffic on large calls and
// by their launch on small ones.  Measured: 4 x 2047 tokens of 32 + 2 x 8 heads of 128, half-split, bf16: 33 us,
// 6.2 TB/s of the bytes read and written (0.92 of a copy's 6772 GB/s); 8 x 6 tokens: 2.8 us.  64 requests' 1 to 5
// entries in 32 layers: 5.0 us, 3.8 TB/s, bound by the chain of two dependent loads before the first entry.

#include "decode_common.cuh"

namespace sv {

// Threads of a token's block.  Few tokens: as many as load all of a token at once.  Many: small blocks, which start
// and end more smoothly (4 x 2047 tokens of 32 + 2 x 8 heads, half-split: 46 us with 256, 36 with 128, 33 with 64;
// 8 x 6 tokens: 2.8, 3.0, 3.7).
constexpr int kAppendThreads = 256, kAppendThreadsMany = 64;

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
};

// Where new token t of a request goes in the cache: its byte offset within a head, or -1.
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
constexpr float kLeastScale = 0x1p-80f, kMostScale = 0x1p80f;
// A power of two that brings another scale to [1, 2), or a subnormal one as near as it reaches; 0 and NaN stay.
__device__ __forceinline__ float scale_power(float s) {
  return __int_as_float(max((254 - ((__float_as_int(s) >> 23) & 255)) << 23, 1 << 22));
}

// 8 elements of a key or value into the cache.
template <bool F8>
__device__ __forceinline__ void store_entry(char* p, float (&x)[8], float scale, float inverse) {
  if constexpr (F8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = quotient(x[i], scale, inverse);
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
  } else {
    *reinterpret_cast<uint4*>(p) = pack8(x);
  }
}

// One block per token.  A thread owns one unit of the head dimension -- the 8 elements at `lo`, and with
// half-split rotation also their partners at lo + rot/2 -- for every lanes-th head, so a token's cos and
// sin are loaded once a thread and an element's partner is always in the same thread (q_out may be q
// itself).  kAhead heads are loaded before the first is used.
template <int D, bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int kAhead = INTERLEAVED ? 4 : 2;
  pdl_launch_next();
  pdl_wait();
  const int paired = INTERLEAVED ? 0 : P.rot / 16;  // units that hold a vector and its partner
  const int units = D / 8 - paired, lanes = blockDim.x / units;
  const int head0 = threadIdx.x / units, unit = threadIdx.x - head0 * units;
  const int b = blockIdx.x / P.batch.T, t = blockIdx.x - b * P.batch.T;
  if (head0 >= lanes) return;

  const bool pair = unit < paired;
  const int lo = pair || INTERLEAVED ? unit * 8 : P.rot + (unit - paired) * 8;
  const bool turns = pair || (INTERLEAVED && lo < P.rot);
  const int far = P.rot / 2;  // distance to the partner
  const int given = P.batch.t_per_row ? __ldg(P.batch.t_per_row + b) : P.batch.T;
  const int held = __ldg(P.batch.ctx_len + b);
  const int tb = min(max(given, 0), P.batch.T), ctx = min(max(held, 0), P.batch.slots);
  int flag = given < 0 || given > P.batch.T ? SPEC_FLAG_BAD_K : 0;
  if (t >= tb) {  // a padded token: its rotated query is 0
    for (int h = head0; h < P.q_heads; h += lanes) {
      char* o = P.q_out.data + b * P.q_out.row + t * P.q_out.token + h * P.q_out.head;
      *reinterpret_cast<uint4*>(o + lo * 2) = make_uint4(0, 0, 0, 0);
      if (pair) *reinterpret_cast<uint4*>(o + (lo + far) * 2) = make_uint4(0, 0, 0, 0);
    }
    if (P.flags && flag && threadIdx.x == 0) atomicOr(P.flags + b, flag);
    return;
  }
  const char* q = P.q.data + b * P.q.row + t * P.q.token;
  const char* k = P.k.data + b * P.k.row + t * P.k.token;
  const char* v = P.v.data + b * P.v.row + t * P.v.token;
  const int k_end = P.q_heads + P.heads, end = k_end + P.heads;
  uint4 w0[kAhead], w1[kAhead];
  const auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * lanes;
      if (h >= end) break;
      const char* p = h < P.q_heads ? q + h * P.q.head : h < k_end ? k + (h - P.q_heads) * P.k.head : v + (h - k_end) * P.v.head;
      w0[i] = *reinterpret_cast<const uint4*>(p + lo * 2);
      if (pair) w1[i] = *reinterpret_cast<const uint4*>(p + (lo + far) * 2);
    }
  };
  load(head0);  // before the page and the angles are known

  // cos and sin of the unit: 8 pairs half-split, 4 pairs interleaved
  float co[8], si[8];
  if (P.rot > 0) {
    // (of the context as it is given, which the table may not hold)
    int pos = P.positions ? __ldg(P.positions + (int64_t)b * P.batch.T + t) : (int)min((int64_t)max(held, 0) + t, (int64_t)INT32_MAX);
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
  const int64_t at = slot_offset(P.batch, P.cache, b, ctx + t);
  if (at < 0 || held < 0) flag |= SPEC_FLAG_BAD_SLOT;
  if (P.flags && flag && threadIdx.x == 0) atomicOr(P.flags + b, flag);

  char* o = P.q_out.data + b * P.q_out.row + t * P.q_out.token;
  for (int h0 = head0; h0 < end; h0 += lanes * kAhead) {
    if (h0 > head0) load(h0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * lanes;
      if (h >= end) break;
      float x[8], y[8];
      unpack8(w0[i], x);
      if (pair) unpack8(w1[i], y);
      if (turns && h < k_end) {
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], c = x[2 * e + 1];
            x[2 * e] = a * co[e] - c * si[e];
            x[2 * e + 1] = c * co[e] + a * si[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[e], c = y[e];
            x[e] = a * co[e] - c * si[e];
            y[e] = c * co[e] + a * si[e];
          }
        }
      }
      if (h < P.q_heads) {
        *reinterpret_cast<uint4*>(o + h * P.q_out.head + lo * 2) = pack8(x);
        if (pair) *reinterpret_cast<uint4*>(o + h * P.q_out.head + (lo + far) * 2) = pack8(y);
      } else if (at >= 0) {
        constexpr int ES = F8 ? 1 : 2;
        const int hh = h < k_end ? h - P.q_heads : h - k_end;
        const float* scales = h < k_end ? P.cache.k_scale : P.cache.v_scale;
        float scale = F8 && scales ? __ldg(scales + hh) : 1.0f;
        if (F8 && !(fabsf(scale) >= kLeastScale && fabsf(scale) <= kMostScale)) {
          const float power = scale_power(scale);
          scale *= power;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            x[n] *= power;
            if (pair) y[n] *= power;
          }
        }
        const float inverse = 1.0f / scale;
        char* e = (h < k_end ? P.cache.k : P.cache.v) + at + hh * P.cache.head;
        store_entry<F8>(e + lo * ES, x, scale, inverse);
        if (pair) store_entry<F8>(e + (lo + far) * ES, y, scale, inverse);
      }
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
  int columns;                // layers * 2 * heads * vecs
};

constexpr int kKeepThreads = 256;
// Columns a thread takes together, and entries of each that it loads before it stores the first (64 requests, 32
// layers, 0 to 4 moves: 5.0 us; 6.4 with 4 columns and 4 entries, 5.8 with 1 and 4; up to 12 moves: 15.4, 18.5, 15.6).
constexpr int kKeepColumns = 2, kKeepAhead = 3;
constexpr int kKeepRound = 64;   // moves whose places the block works out at a time

// Block (x, y): every gridDim.x-th run of 256 columns of request y's entries.  A column is one 16-byte
// vector (layer, k or v, head, vector) of every slot, and one thread moves it through the path in order.  A
// strictly increasing path has path[i] >= i, so what move i overwrites (slot i) is never read by a later
// move: loads may run ahead of stores, and columns are independent.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams P) {
  __shared__ int64_t from[kKeepRound], to[kKeepRound];
  __shared__ int moves;
  pdl_launch_next();
  pdl_wait();
  const int b = blockIdx.y;
  const int32_t* path = P.path + (int64_t)b * P.max_keep;
  const int ahead = threadIdx.x < 32 && (int)threadIdx.x < P.max_keep ? __ldg(path + threadIdx.x) : 0;  // before n is known
  const int n = min(max(__ldg(P.n_keep + b), 0), P.max_keep);
  const int ctx = batch_context(P.batch, b);
  for (int i0 = 0; i0 < n; i0 += kKeepRound) {
    // the moves of this round that move something, in the path's order
    if (threadIdx.x < 32) {
      int count = 0;
      for (int i1 = i0; i1 < min(n, i0 + kKeepRound); i1 += 32) {
        const int i = i1 + threadIdx.x;
        int64_t src = -1, dst = -1;
        if (i < n) {
          const int p = i < 32 ? ahead : __ldg(path + i);
          if (p != i && p >= 0 && p < P.batch.slots) {
            dst = slot_offset(P.batch, P.cache, b, ctx + i);
            src = slot_offset(P.batch, P.cache, b, ctx + p);
          }
        }
        const bool is = src >= 0 && dst >= 0;
        const uint32_t all = __ballot_sync(~0u, is);
        if (is) {
          const int at = count + __popc(all & ((1u << threadIdx.x) - 1));
          from[at] = src, to[at] = dst;
        }
        count += __popc(all);
      }
      if (threadIdx.x == 0) moves = count;
    }
    __syncthreads();
    const int round = moves;
    for (int c0 = blockIdx.x * kKeepThreads * kKeepColumns + threadIdx.x; c0 < P.columns;
         c0 += gridDim.x * kKeepThreads * kKeepColumns) {
      char* column[kKeepColumns];
#pragma unroll
      for (int k = 0; k < kKeepColumns; ++k) {
        const int c = c0 + k * kKeepThreads;
        const int head = c / P.vecs, vec = c - head * P.vecs;
        const int side = head / P.heads, layer = side / 2;
        column[k] = c < P.columns ? (side % 2 ? P.cache.v : P.cache.k) + layer * P.cache.layer +
                                        (head - side * P.heads) * P.cache.head + vec * 16
                                  : nullptr;
      }
      for (int i = 0; i < round; i += kKeepAhead) {
        uint4 w[kKeepColumns][kKeepAhead];
#pragma unroll
        for (int k = 0; k < kKeepColumns; ++k)
#pragma unroll
          for (int j = 0; j < kKeepAhead; ++j)
            if (column[k] && i + j < round) w[k][j] = *reinterpret_cast<const uint4*>(column[k] + from[i + j]);
#pragma unroll
        for (int k = 0; k < kKeepColumns; ++k)
#pragma unroll
          for (int j = 0; j < kKeepAhead; ++j)
            if (column[k] && i + j < round) *reinterpret_cast<uint4*>(column[k] + to[i + j]) = w[k][j];
      }
    }
    __syncthreads();
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
  const int64_t blocks = (int64_t)batch->B * batch->T;
  if (blocks > 0x7fffffffll || q_heads > 65535) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  auto kern = cache->head_dim == 128
                  ? (f8 ? (inter ? append_kernel<128, true, true> : append_kernel<128, true, false>)
                        : (inter ? append_kernel<128, false, true> : append_kernel<128, false, false>))
                  : (f8 ? (inter ? append_kernel<64, true, true> : append_kernel<64, true, false>)
                        : (inter ? append_kernel<64, false, true> : append_kernel<64, false, false>));
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  const int threads = blocks >= 16 * sms ? kAppendThreadsMany : kAppendThreads;
  return launch_early(kern, dim3((unsigned)blocks), dim3(threads), 0, st, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
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
  const int64_t columns = (int64_t)cache->layers * 2 * P.heads * P.vecs;
  if (columns > 0x40000000ll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;  // column indices stay in 32 bits
  P.columns = (int)columns;
  const int64_t run = kKeepThreads * kKeepColumns;
  const dim3 grid((unsigned)((columns + run - 1) / run), batch->B);
  return launch_early(keep_kernel, grid, dim3(kKeepThreads), 0, static_cast<cudaStream_t>(stream), P) == cudaSuccess ? SPEC_OK
                                                                                                                    : SPEC_ERR_CUDA;
}

}  // extern "C"
