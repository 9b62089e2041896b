// spec_kv.cu — the writes to the paged key-value cache: spec_kv_append (the new tokens' rotated keys and
// their values, with the queries rotated on the way) and spec_kv_keep (the accepted branch moved up
// behind the context).  Both are streams of 16-byte vectors, bound by memory traffic on large calls and
// by their launch on small ones.  Measured: 4 x 2047 tokens of 32 + 2 x 8 heads of 128, half-split, bf16: 33 us,
// 6.2 TB/s of the bytes read and written (0.92 of a copy's 6772 GB/s); 8 x 6 tokens: 2.8 us.  With page scales, pages of 32:
// 28 us interleaved, 3.3 TB/s (0.49), 30 half-split, bound by instructions; 8 x 6 tokens: 3.4 us.  64 requests' 1 to 5
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
__device__ __forceinline__ void append_token(const AppendParams& P, int block) {
  constexpr int kAhead = INTERLEAVED ? 4 : 2;
  const int paired = INTERLEAVED ? 0 : P.rot / 16;  // units that hold a vector and its partner
  const int units = D / 8 - paired, lanes = blockDim.x / units;
  const int head0 = threadIdx.x / units, unit = threadIdx.x - head0 * units;
  const int b = block / P.batch.T, t = block - b * P.batch.T;
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

template <int D, bool F8, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams P) {
  pdl_launch_next();
  pdl_wait();
  append_token<D, F8, INTERLEAVED>(P, blockIdx.x);
}

// ------------------------------------------------------------------------------------------------
// spec_kv_append_ex: a page's scale follows what goes into it
// ------------------------------------------------------------------------------------------------
// Threads of a page's block, by the tokens that it can get (4 x 2047 tokens, pages of 8: 38 us with 64, 46 with 128; of 32: 30, 31, and
// 49 with 256; of 256: 106, 58, 43).
constexpr int kPageThreadsMost = 256;
static int page_threads(int tokens) { return tokens <= 32 ? 64 : tokens <= 128 ? 128 : 256; }

struct PageAppendParams {
  Heads k, v;
  Cache cache;
  PageScales scales;
  Batch batch;
  const float* cos_table;
  const float* sin_table;
  const int32_t* positions;
  int heads, touched;  // touched: pages that T tokens can lie in
  int rot, max_positions;
};

// One block per (request, page that gets tokens, head, k or v), `index`: the largest magnitude of what goes in, then the page's
// scale, then the codes.  A thread owns one unit of the head dimension as in append_kernel, for every lanes-th token; the
// products of a rotation are rounded one by one, so the magnitude does not depend on how they are fused.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void append_page(const PageAppendParams& P, int index) {
  constexpr int kHeld = INTERLEAVED ? 4 : 2;  // tokens that a thread holds between the two passes
  __shared__ float most_of[kPageThreadsMost / 32];
  const bool is_v = index & 1;
  index >>= 1;
  const int head = index % P.heads;
  index /= P.heads;
  const int nth = index % P.touched, b = index / P.touched;

  const int page_size = 1 << P.cache.page_shift;
  const int held = __ldg(P.batch.ctx_len + b);
  const int tb = batch_tokens(P.batch, b), ctx = min(max(held, 0), P.batch.slots);
  const int ordinal = (ctx >> P.cache.page_shift) + nth;
  if (ordinal >= P.batch.max_pages) return;
  const int from = ordinal << P.cache.page_shift;  // the page's first slot
  const int t0 = max(from - ctx, 0), t1 = (int)min((int64_t)tb, (int64_t)from + page_size - ctx);
  if (t0 >= t1) return;
  const int page = __ldg(P.batch.pages + (int64_t)b * P.batch.max_pages + ordinal);
  if (page < 0 || page >= P.cache.num_pages) return;

  const int rot = is_v ? 0 : P.rot;
  const int paired = INTERLEAVED ? 0 : rot / 16, units = D / 8 - paired, lanes = blockDim.x / units;
  const int lane0 = threadIdx.x / units, unit = threadIdx.x - lane0 * units;
  const bool works = lane0 < lanes, pair = unit < paired;
  const int lo = pair || INTERLEAVED ? unit * 8 : rot + (unit - paired) * 8, far = rot / 2;
  const bool turns = pair || (INTERLEAVED && lo < rot);
  const Heads& in = is_v ? P.v : P.k;
  const char* src = in.data + b * in.row + head * in.head;

  const auto load = [&](int t, uint4& a, uint4& c) {
    const char* p = src + t * in.token;
    a = *reinterpret_cast<const uint4*>(p + lo * 2);
    if (pair) c = *reinterpret_cast<const uint4*>(p + (lo + far) * 2);
  };
  const auto turned = [&](int t, const uint4& a, const uint4& c, float (&x)[8], float (&y)[8]) {
    unpack8(a, x);
    if (pair) unpack8(c, y);
    if (!turns) return;
    int pos = P.positions ? __ldg(P.positions + (int64_t)b * P.batch.T + t) : (int)min((int64_t)max(held, 0) + t, (int64_t)INT32_MAX);
    pos = min(max(pos, 0), P.max_positions - 1);
    const int64_t base = (int64_t)pos * (rot / 2) + (INTERLEAVED ? lo / 2 : lo);
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 4 : 8); i += 4) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(P.cos_table + base + i));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(P.sin_table + base + i));
      const float co[4] = {c4.x, c4.y, c4.z, c4.w}, si[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& first = INTERLEAVED ? x[2 * e] : x[i + e];
        float& second = INTERLEAVED ? x[2 * e + 1] : y[i + e];
        const float u = first, v = second;
        first = __fsub_rn(__fmul_rn(u, co[e]), __fmul_rn(v, si[e]));
        second = __fadd_rn(__fmul_rn(v, co[e]), __fmul_rn(u, si[e]));
      }
    }
  };

  float most = 0.0f;  // of the finite magnitudes
  const auto look = [&](const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (fabsf(x[e]) < INFINITY) most = fmaxf(most, fabsf(x[e]));
      if (!INTERLEAVED && pair && fabsf(y[e]) < INFINITY) most = fmaxf(most, fabsf(y[e]));
    }
  };
  float x[kHeld][8], y[kHeld][8];  // the first tokens, turned
  if (works) {
    uint4 a[kHeld], c[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (t0 + lane0 + i * lanes < t1) load(t0 + lane0 + i * lanes, a[i], c[i]);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (t0 + lane0 + i * lanes < t1) {
        turned(t0 + lane0 + i * lanes, a[i], c[i], x[i], y[i]);
        look(x[i], y[i]);
      }
    for (int t = t0 + lane0 + kHeld * lanes; t < t1; t += lanes) {
      uint4 a, c;
      float x[8], y[8];
      load(t, a, c);
      turned(t, a, c, x, y);
      look(x, y);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  if ((threadIdx.x & 31) == 0) most_of[threadIdx.x >> 5] = most;
  float* place = (is_v ? P.scales.v : P.scales.k) + (int64_t)page * P.heads + head;
  const int before = nth == 0 ? ctx - from : 0;  // rows of the page that hold tokens already
  const float old = before > 0 ? *place : 0.0f;
  __syncthreads();  // every thread has read the old scale
  for (int w = 0; w < blockDim.x / 32; ++w) most = fmaxf(most, most_of[w]);
  const bool counts = before > 0 && scale_counts(old);
  const float need = scale_need(most), scale = counts ? fmaxf(old, need) : need, inverse = 1.0f / scale;
  if (threadIdx.x == 0) *place = scale;

  char* out = (is_v ? P.cache.v : P.cache.k) + page * P.cache.page + head * P.cache.head;
  if (counts && need > old) {  // the rows before: their codes at the new scale, a power of two
    const float ratio = old * inverse;
    for (int u = threadIdx.x; u < before * (D / 16); u += blockDim.x) {
      uint4* p = reinterpret_cast<uint4*>(out + (u / (D / 16)) * P.cache.slot + (u % (D / 16)) * 16);
      *p = rescaled(*p, ratio);
    }
  }
  if (!works) return;
  const auto store = [&](int t, const float (&x)[8], const float (&y)[8]) {
    char* p = out + (int64_t)(ctx + t - from) * P.cache.slot;
    const auto put = [&](char* at, const float (&z)[8]) {
      float c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = signed_quotient(z[e], scale, inverse);
      *reinterpret_cast<uint2*>(at) = make_uint2(pack_e4m3(c[0], c[1], c[2], c[3]), pack_e4m3(c[4], c[5], c[6], c[7]));
    };
    put(p + lo, x);
    if (!INTERLEAVED && pair) put(p + lo + far, y);
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (t0 + lane0 + i * lanes < t1) store(t0 + lane0 + i * lanes, x[i], y[i]);
  for (int t = t0 + lane0 + kHeld * lanes; t < t1; t += lanes) {
    uint4 a, c;
    float x[8], y[8];
    load(t, a, c);
    turned(t, a, c, x, y);
    store(t, x, y);
  }
}

struct PageStepParams {
  AppendParams queries;  // heads = 0: the queries and the flags
  PageAppendParams pages;
  int page_blocks;
};

// The pages' blocks, then the tokens' that rotate the queries: in one launch they run beside one another (4 x 2047 tokens of 32 +
// 2 x 8 heads, pages of 32: 30 us, 31 in two; 8 x 6 tokens: a launch less).  Four blocks of 256 threads an SM: 28 us
// instead of 30.6 interleaved.  Half-split, with a few registers spilled: 30 us, 36 at pages of 256; 29 and 40 with three blocks, 36 and 53 with
// two, which spill nothing.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kPageThreadsMost, 4) page_append_kernel(const __grid_constant__ PageStepParams P) {
  pdl_launch_next();
  pdl_wait();
  if (blockIdx.x < P.page_blocks) append_page<D, INTERLEAVED>(P.pages, blockIdx.x);
  else append_token<D, true, INTERLEAVED>(P.queries, blockIdx.x - P.page_blocks);
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

spec_status_t spec_kv_append_ex(const spec_heads_t* q, const spec_heads_t* k, const spec_heads_t* v,
                                const spec_heads_t* q_out, int32_t q_heads, const spec_kv_cache_t* cache,
                                const spec_kv_page_scales_t* scales, const spec_decode_batch_t* batch,
                                const spec_rotary_t* rotary, int32_t* out_flags, void* stream) {
  spec_status_t s = check_cache(cache, true);
  if (s == SPEC_OK) s = check_scales(scales, cache);
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
  P.q_heads = q_heads, P.heads = scales ? 0 : cache->heads;  // with page scales: the queries and flags alone
  const bool inter = rot > 0 && rotary->interleaved != 0;
  const int64_t blocks = (int64_t)batch->B * batch->T;
  const int64_t touched = ((int64_t)batch->T + cache->page_size - 2) / cache->page_size + 1;
  const int64_t page_blocks = batch->B * touched * cache->heads * 2;
  if (scales && page_blocks + blocks > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  if (blocks > 0x7fffffffll || q_heads > 65535) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  auto kern = cache->head_dim == 128
                  ? (f8 ? (inter ? append_kernel<128, true, true> : append_kernel<128, true, false>)
                        : (inter ? append_kernel<128, false, true> : append_kernel<128, false, false>))
                  : (f8 ? (inter ? append_kernel<64, true, true> : append_kernel<64, true, false>)
                        : (inter ? append_kernel<64, false, true> : append_kernel<64, false, false>));
  if (scales) {
    const bool tokens = q_heads > 0 || out_flags;
    const PageStepParams A = {P, {P.k, P.v, P.cache, scales_of(scales), P.batch, P.cos_table, P.sin_table, P.positions, cache->heads,
                              (int)touched, rot, P.max_positions}, (int)page_blocks};
    auto pages = cache->head_dim == 128 ? (inter ? page_append_kernel<128, true> : page_append_kernel<128, false>)
                                        : (inter ? page_append_kernel<64, true> : page_append_kernel<64, false>);
    const dim3 grid((unsigned)(page_blocks + (tokens ? blocks : 0)));
    const int threads = page_threads(batch->T < cache->page_size ? batch->T : cache->page_size);
    return launch_early(pages, grid, dim3(threads), 0, st, A) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  }
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  const int threads = blocks >= 16 * sms ? kAppendThreadsMany : kAppendThreads;
  return launch_early(kern, dim3((unsigned)blocks), dim3(threads), 0, st, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status_t spec_kv_append(const spec_heads_t* q, const spec_heads_t* k, const spec_heads_t* v,
                             const spec_heads_t* q_out, int32_t q_heads, const spec_kv_cache_t* cache,
                             const spec_decode_batch_t* batch, const spec_rotary_t* rotary, int32_t* out_flags,
                             void* stream) {
  return spec_kv_append_ex(q, k, v, q_out, q_heads, cache, nullptr, batch, rotary, out_flags, stream);
}

spec_status_t spec_kv_keep(const spec_kv_cache_t* cache, const spec_decode_batch_t* batch, const int32_t* path,
                           const int32_t* n_keep, int32_t max_keep, void* stream) {
  spec_status_t s = check_cache(cache, false);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (max_keep < 0) return SPEC_ERR_INVALID_ARG;
  if (max_keep > SPEC_MAX_SLOTS) return SPEC_ERR_UNSUPPORTED;
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
