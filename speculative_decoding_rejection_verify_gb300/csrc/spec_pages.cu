// spec_pages.cu — moves of cache entries: spec_kv_keep_ex (the accepted branch in a cache with page scales, and what is
// recorded of the entries) and spec_kv_move (the entries that stay, after spec_kv_select).  An entry that moves into
// another page of an E4M3 cache with page scales is a code of that page's scale from then on, which may have to grow, and
// then the page's other codes change with it; so a page's moves are one warp's work: their codes into registers, the largest
// magnitude (only where a source's scale is above the target's: else nothing can grow it), the new scale, the codes.
//
// Measured: 32 requests x 8 heads of 128, 6000 of 8000 to 16000 entries kept, E4M3 with page scales: 262 us on a new cache, two
// thirds of whose pages grow, and 143 us where none does: 2.8 TB/s of the bytes moved (0.41 of a copy's 6749 GB/s), bound by
// instructions and by the chain list -> page -> scale and codes -> store at 24 warps an SM (two warps' work for keys and values:
// 225 us with both in one, which takes 162 registers).  A scale per head 88 us, bf16 149.  64 requests' 1 to 5 entries in 32 layers:
// 29 us on a new cache, 12 where no page grows (17 with weights and positions); up to 31 entries 42 and 17, up to 61 171 and 150.

#include "decode_common.cuh"

namespace sv {

// The values of 16 codes at scale `from`, as codes at scale `to` (by way of fp16 where both are powers of two).
__device__ __forceinline__ uint4 recoded(uint4 w, float from, float to) {
  const float inverse = 1.0f / to, ratio = from * inverse;
  if (((__float_as_int(from) | __float_as_int(to)) & 0x7FFFFF) == 0 && half_ratio(ratio)) return rescaled_half(w, __float2half2_rn(ratio));
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const float4 f = unpack_e4m3(x[i]);
    x[i] = pack_e4m3(signed_quotient(f.x * from, to, inverse), signed_quotient(f.y * from, to, inverse),
                     signed_quotient(f.z * from, to, inverse), signed_quotient(f.w * from, to, inverse));
  }
  return w;
}

// One lane's move of a warp's 32: where its entry lies and goes, as byte offsets from row 0 of page 0 of the head.  Moves
// into one page are neighbours, lanes lo .. hi; a lane whose move is left out still belongs to its page.
struct Move {
  bool is;
  int64_t src, dst;
  int from, to;   // pages; to < 0: the page is outside the pool
  int lo, hi;
};

// A warp's view of the keys or values of one head of a cache with page scales.
struct Side {
  char* base;       // row 0 of page 0
  float* scales;    // of page 0
  int heads;        // from page to page
  int64_t slot, page;
  int page_size;
};

// What a warp's lanes tell one another.
struct Exchange {
  int64_t src[32], dst[32];
  float2 scales[32];                    // an entry's, old and new
  uint32_t ratio[32];                   // the old over the new, twice in fp16; 0: fp16 does not do it
  uint32_t taken[SPEC_MAX_PAGE / 32];   // rows of a page that entries move into
};

__device__ __forceinline__ void tell_places(Exchange& x, const Move& m) {
  const int lane = threadIdx.x & 31;
  x.src[lane] = m.is ? m.src : -1, x.dst[lane] = m.dst;
  __syncwarp();
}
// The entries' codes: lane l has vector l % (D / 16) of entries j * 32 / (D / 16) + l / (D / 16).  n: the moves are lanes 0 .. n - 1.
template <int D>
__device__ __forceinline__ void load_entries(const char* base, const Exchange& x, int n, uint4 (&w)[D / 16]) {
  constexpr int kVecs = D / 16, kAtOnce = 32 / kVecs;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    w[j] = make_uint4(0, 0, 0, 0);
    if (j * kAtOnce >= n) continue;
    const int64_t at = x.src[j * kAtOnce + lane / kVecs];
    if (at >= 0) w[j] = *reinterpret_cast<const uint4*>(base + at + lane % kVecs * 16);
  }
}
// Bytes 1 and 3 of the largest codes among a vector's, without their signs: a larger one is a larger magnitude.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t largest_of(const uint4& w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) top = max_u16x2(top, max_u16x2(x[k] & 0x7F007F00u, (x[k] << 8) & 0x7F007F00u));
  return top;
}
__device__ __forceinline__ uint4 without_nan(uint4 w) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] &= ~__vcmpeq4(x[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return w;
}
// The largest code of this lane's entry that is not NaN (0x7F), without its sign.
template <int D>
__device__ __forceinline__ uint32_t largest_code(const uint4 (&w)[D / 16], int n) {
  constexpr int kVecs = D / 16, kAtOnce = 32 / kVecs;
  const int lane = threadIdx.x & 31;
  uint32_t top[kVecs], all = 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    top[j] = j * kAtOnce < n ? largest_of(w[j]) : 0;
    all = max_u16x2(all, top[j]);
  }
  if (__any_sync(~0u, all >= 0x7F000000u || (all & 0xFFFF) >= 0x7F00u)) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) top[j] = largest_of(without_nan(w[j]));
  }
  // over the lanes of an entry, each of which ends with the entry of its own number
#pragma unroll
  for (int d = kVecs / 2; d > 0; d /= 2) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < d; ++k) {
      const uint32_t keep = up ? top[k + d] : top[k], send = up ? top[k] : top[k + d];
      top[k] = max_u16x2(keep, __shfl_xor_sync(~0u, send, d));
    }
  }
  const uint32_t mine = __shfl_sync(~0u, top[0], lane % kAtOnce * kVecs + lane / kAtOnce);
  return max(mine >> 24, (mine >> 8) & 0xFF);
}
__device__ __forceinline__ float magnitude(uint32_t code, float scale) {  // a finite one, or 0
  const float x = unpack_e4m3(code).x * fabsf(scale);
  return x < INFINITY ? x : 0.0f;
}
__device__ __forceinline__ void tell_scales(Exchange& x, float from, float to) {
  const int lane = threadIdx.x & 31;
  const float ratio = from * (1.0f / to);
  const __half2 r = __float2half2_rn(ratio);
  const bool half = ((__float_as_int(from) | __float_as_int(to)) & 0x7FFFFF) == 0 && half_ratio(ratio);
  x.scales[lane] = make_float2(from, to);
  x.ratio[lane] = from == to ? 0x3C003C00u : half ? *reinterpret_cast<const uint32_t*>(&r) : 0;
  __syncwarp();
}
template <int D>
__device__ __forceinline__ void store_entries(char* base, const Exchange& x, int n, const uint4 (&w)[D / 16]) {
  constexpr int kVecs = D / 16, kAtOnce = 32 / kVecs;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    if (j * kAtOnce >= n) continue;
    const int e = j * kAtOnce + lane / kVecs;
    if (x.src[e] < 0) continue;
    const uint32_t ratio = x.ratio[e];
    uint4 y = w[j];
    if (ratio == 0) y = recoded(y, x.scales[e].x, x.scales[e].y);
    else if (ratio != 0x3C003C00u) y = rescaled_half(y, *reinterpret_cast<const __half2*>(&ratio));
    *reinterpret_cast<uint4*>(base + x.dst[e] + lane % kVecs * 16) = y;
  }
}
// The page's scale with `most` in it, and what its codes have to be multiplied by.
struct NewScale {
  float scale, ratio;  // ratio 1: the codes stay
};
__device__ __forceinline__ NewScale new_scale(float old, float most) {
  const bool counts = scale_counts(old);
  const float need = scale_need(most), scale = counts ? fmaxf(old, need) : need;
  return {scale, counts && need > old ? old / need : 1.0f};
}
// Whether a page of scale `old` holds whatever a page of scale `from` does: a power of two that is not less.
__device__ __forceinline__ bool holds(float old, float from) {
  return scale_counts(old) && (__float_as_int(old) & 0x7FFFFF) == 0 && from >= 0.0f && from <= old;
}
// A warp rescales the rows < end of a page but for those marked in `taken`.  (Several rows in flight a thread cost registers that
// the moves without it want more: 195 us against 150 with four.)
template <int D>
__device__ __forceinline__ void rescale_page(char* page, int64_t slot, int end, const uint32_t* taken, float ratio) {
  constexpr int kVecs = D / 16, kAtOnce = 32 / kVecs;
  const int lane = threadIdx.x & 31;
  for (int r = lane / kVecs; r < end; r += kAtOnce) {
    if ((taken[r >> 5] >> (r & 31)) & 1) continue;
    uint4* p = reinterpret_cast<uint4*>(page + r * slot + lane % kVecs * 16);
    *p = rescaled(*p, ratio);
  }
  __syncwarp();
}
__device__ __forceinline__ void clear_taken(uint32_t* taken, int page_size) {
  for (int i = threadIdx.x & 31; i < (page_size + 31) / 32; i += 32) taken[i] = 0;
  __syncwarp();
}

// A warp's n moves, whole pages' of them, at most 32: every entry is in registers before the first is written.  row: the
// target's row in its page; end: the rows of that page that hold what stays.
template <int D>
__device__ __forceinline__ void move_batch(const Side& c, const Move& m, int n, int row, int end, Exchange& x) {
  const int lane = threadIdx.x & 31;
  tell_places(x, m);
  uint4 w[D / 16];
  load_entries<D>(c.base, x, n, w);
  const float from = m.is ? c.scales[(int64_t)m.from * c.heads] : 0.0f, old = m.to >= 0 ? c.scales[(int64_t)m.to * c.heads] : 1.0f;
  const uint32_t page_lanes = (m.hi == 31 ? ~0u : (2u << m.hi) - 1) & (~0u << m.lo);
  const bool any = __ballot_sync(~0u, m.is) & page_lanes;  // of the lane's page
  float scale = old;
  if (__any_sync(~0u, m.is && !holds(old, from))) {
    float most = magnitude(largest_code<D>(w, n), from);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const float y = __shfl_up_sync(~0u, most, d);
      if (lane - d >= m.lo) most = fmaxf(most, y);
    }
    const NewScale s = new_scale(old, __shfl_sync(~0u, most, m.hi));
    scale = s.scale;
    uint32_t grown = __ballot_sync(~0u, any && lane == m.lo && s.ratio != 1.0f);
    while (grown) {
      const int leader = __ffs(grown) - 1;
      grown &= grown - 1;
      clear_taken(x.taken, c.page_size);
      if (m.is && m.lo == leader) atomicOr(&x.taken[row >> 5], 1u << (row & 31));
      __syncwarp();
      rescale_page<D>(c.base + __shfl_sync(~0u, m.to, leader) * c.page, c.slot, __shfl_sync(~0u, end, leader), x.taken,
                      __shfl_sync(~0u, s.ratio, leader));
    }
  }
  tell_scales(x, from, scale);
  store_entries<D>(c.base, x, n, w);
  // an entry may come from a page that others go to: its old scale was needed until here, and is in registers
  if (any && lane == m.lo && scale != old) c.scales[(int64_t)m.to * c.heads] = scale;
  __syncwarp();
}

// A warp's n moves into one page: info(i) is lane's move i (is = false behind the last), row(move) its row.
template <int D, typename Info, typename Row>
__device__ __noinline__ void move_page(const Side& c, int n, int to, int end, Exchange& x, Info info, Row row) {
  const int lane = threadIdx.x & 31;
  float* place = c.scales + (int64_t)to * c.heads;
  const float old = *place;
  float most = 0.0f;
  bool any = false, look = false;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const Move m = info(i0 + lane);
    const float from = m.is ? c.scales[(int64_t)m.from * c.heads] : 0.0f;
    any |= m.is;
    if (!__any_sync(~0u, m.is && !holds(old, from))) continue;
    look = true;
    tell_places(x, m);
    uint4 w[D / 16];
    load_entries<D>(c.base, x, n - i0, w);
    most = fmaxf(most, magnitude(largest_code<D>(w, n - i0), from));
    __syncwarp();
  }
  if (!__any_sync(~0u, any)) return;
  NewScale s = {old, 1.0f};
  if (look) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
    s = new_scale(old, most);
  }
  if (s.ratio != 1.0f) {
    clear_taken(x.taken, c.page_size);
    for (int i0 = 0; i0 < n; i0 += 32) {
      const Move m = info(i0 + lane);
      if (m.is) atomicOr(&x.taken[row(m) >> 5], 1u << (row(m) & 31));
    }
    __syncwarp();
    rescale_page<D>(c.base + to * c.page, c.slot, end, x.taken, s.ratio);
  }
  for (int i0 = 0; i0 < n; i0 += 32) {
    const Move m = info(i0 + lane);
    tell_places(x, m);
    uint4 w[D / 16];
    load_entries<D>(c.base, x, n - i0, w);
    tell_scales(x, m.is ? c.scales[(int64_t)m.from * c.heads] : 1.0f, s.scale);
    store_entries<D>(c.base, x, n - i0, w);
    __syncwarp();
  }
  // an entry may come from the same page: its old scale was needed until here
  if (lane == 0 && s.scale != old) *place = s.scale;
  __syncwarp();
}

// ------------------------------------------------------------------------------------------------
// spec_kv_keep_ex
// ------------------------------------------------------------------------------------------------
struct PageKeepParams {
  Cache cache;
  PageScales scales;
  Batch batch;
  const int32_t* path;
  const int32_t* n_keep;
  int max_keep, heads;
  int lists;  // layers * heads * 2
};

constexpr int kPageKeepWarps = 4;

// Where the moves of a request's path go, of all its layers and heads.
struct PathMoves {
  int64_t src[SPEC_MAX_NEW], dst[SPEC_MAX_NEW];
  int from[SPEC_MAX_NEW], to[SPEC_MAX_NEW];  // from < 0: left out
};

// A block's warps take the (layer, head, k or v) of one request.  Nothing is written before everything is read, since a path's
// targets may be its later sources: up to 32 entries wait in registers; more (BIG) are copied to shared memory first, which takes
// the place of the cache as their source.
template <int D, bool BIG>
__global__ void __launch_bounds__(kPageKeepWarps * 32, 6) page_keep_kernel(const __grid_constant__ PageKeepParams P) {
  __shared__ PathMoves path;
  __shared__ Exchange exchange[kPageKeepWarps];
  __shared__ float scales_of[kPageKeepWarps][BIG ? SPEC_MAX_NEW : 1];
  extern __shared__ uint4 copies[];  // BIG: [warps][SPEC_MAX_NEW][D / 16]
  pdl_launch_next();
  pdl_wait();
  constexpr int kVecs = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y, shift = P.cache.page_shift, page_size = 1 << shift;
  const int n = min(max(__ldg(P.n_keep + b), 0), P.max_keep), ctx = batch_context(P.batch, b);
  if (threadIdx.x < SPEC_MAX_NEW) {
    const int i = threadIdx.x;
    int from = -1, to = -1;
    int64_t src = 0, dst = 0;
    if (i < n) {
      const int p = __ldg(P.path + (int64_t)b * P.max_keep + i);
      const int64_t t = slot_offset(P.batch, P.cache, b, ctx + i);
      if (t >= 0) to = __ldg(P.batch.pages + (int64_t)b * P.batch.max_pages + ((ctx + i) >> shift)), dst = t;
      if (t >= 0 && p != i && p >= 0 && p < P.batch.slots) {
        const int64_t s = slot_offset(P.batch, P.cache, b, ctx + p);
        if (s >= 0) from = __ldg(P.batch.pages + (int64_t)b * P.batch.max_pages + ((ctx + p) >> shift)), src = s;
      }
    }
    path.src[i] = src, path.dst[i] = dst, path.from[i] = from, path.to[i] = to;
  }
  const bool any = __syncthreads_or(threadIdx.x < n && path.from[threadIdx.x] >= 0);
  if (!any) return;
  const int end = (int)min((int64_t)ctx + n, (int64_t)P.batch.slots);
  const auto rows_of = [&](int ordinal) { return min(end - (ordinal << shift), page_size); };
  Exchange& x = exchange[warp];
  for (int list = blockIdx.x * kPageKeepWarps + warp; list < P.lists; list += gridDim.x * kPageKeepWarps) {
    const bool is_v = list & 1;
    const int head = (list >> 1) % P.heads, layer = (list >> 1) / P.heads;
    const Side c = {(is_v ? P.cache.v : P.cache.k) + layer * P.cache.layer + head * P.cache.head,
                    (is_v ? P.scales.v : P.scales.k) + layer * P.scales.layer + head, P.heads, P.cache.slot, P.cache.page, page_size};
    if constexpr (!BIG) {
      const int ordinal = (ctx + lane) >> shift;
      Move m = {lane < n && path.from[lane] >= 0, path.src[lane], path.dst[lane], path.from[lane], lane < n ? path.to[lane] : -1, lane, lane};
      if (lane < n) m.lo = max((ordinal << shift) - ctx, 0), m.hi = min(((ordinal + 1) << shift) - ctx, n) - 1;
      move_batch<D>(c, m, n, (ctx + lane) & (page_size - 1), rows_of(ordinal), x);
    } else {
      uint4* mine = copies + warp * SPEC_MAX_NEW * kVecs;
      for (int u = lane; u < n * kVecs; u += 32)
        if (path.from[u / kVecs] >= 0) mine[u] = *reinterpret_cast<const uint4*>(c.base + path.src[u / kVecs] + u % kVecs * 16);
      for (int i = lane; i < n; i += 32)
        if (path.from[i] >= 0) scales_of[warp][i] = c.scales[(int64_t)path.from[i] * P.heads];
      __syncwarp();
      for (int i = 0; i < n;) {  // a page at a time
        const int ordinal = (ctx + i) >> shift, first = i, to = path.to[i];
        float most = 0.0f;
        bool moves = false;
        for (; i < n && (ctx + i) >> shift == ordinal; ++i) {
          if (path.from[i] < 0) continue;
          moves = true;
          uint32_t top = lane < kVecs ? largest_of(without_nan(mine[i * kVecs + lane])) : 0;
          top = max(top >> 24, (top >> 8) & 0xFF);
          most = fmaxf(most, magnitude(__reduce_max_sync(~0u, top), scales_of[warp][i]));
        }
        if (!moves) continue;
        float* place = c.scales + (int64_t)to * P.heads;
        const NewScale s = new_scale(*place, most);
        if (s.ratio != 1.0f) {
          clear_taken(x.taken, page_size);
          for (int k = first + lane; k < i; k += 32) {
            const int row = (ctx + k) & (page_size - 1);
            if (path.from[k] >= 0) atomicOr(&x.taken[row >> 5], 1u << (row & 31));
          }
          __syncwarp();
          rescale_page<D>(c.base + to * c.page, c.slot, rows_of(ordinal), x.taken, s.ratio);
        }
        for (int u = first * kVecs + lane; u < i * kVecs; u += 32) {
          const int k = u / kVecs;
          if (path.from[k] < 0) continue;
          const float from = scales_of[warp][k];
          *reinterpret_cast<uint4*>(c.base + path.dst[k] + u % kVecs * 16) = from == s.scale ? mine[u] : recoded(mine[u], from, s.scale);
        }
        __syncwarp();
        if (lane == 0) *place = s.scale;
        __syncwarp();
      }
    }
  }
}

struct RecordKeepParams {
  Cache cache;  // its pages' number and size
  Record record;
  Batch batch;
  const int32_t* path;
  const int32_t* n_keep;
  int max_keep, heads;
  int64_t lists;  // layers * B * heads
};

// A thread per (layer, request, head) goes through the path in order: what move i overwrites no later one reads.
__global__ void __launch_bounds__(128) record_keep_kernel(const __grid_constant__ RecordKeepParams P) {
  pdl_launch_next();
  pdl_wait();
  int64_t list = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (list >= P.lists) return;
  const int head = list % P.heads;
  list /= P.heads;
  const int b = list % P.batch.B;
  const int64_t layer = list / P.batch.B * P.record.layer;
  const int n = min(max(__ldg(P.n_keep + b), 0), P.max_keep), ctx = batch_context(P.batch, b);
  const int mask = (1 << P.cache.page_shift) - 1;
  const auto place = [&](int slot) -> int64_t {
    if (slot < 0 || slot >= P.batch.slots) return -1;
    const int page = __ldg(P.batch.pages + (int64_t)b * P.batch.max_pages + (slot >> P.cache.page_shift));
    if (page < 0 || page >= P.cache.num_pages) return -1;
    return layer + (((int64_t)page * P.heads + head) << P.cache.page_shift) + (slot & mask);
  };
  for (int i = 0; i < n; ++i) {
    const int p = __ldg(P.path + (int64_t)b * P.max_keep + i);
    if (p == i || p < 0 || p >= P.batch.slots) continue;
    const int64_t dst = place(ctx + i), src = place(ctx + p);
    if (dst < 0 || src < 0) continue;
    if (P.record.weight) P.record.weight[dst] = P.record.weight[src];
    if (P.record.position) P.record.position[dst] = P.record.position[src];
  }
}

// ------------------------------------------------------------------------------------------------
// spec_kv_move
// ------------------------------------------------------------------------------------------------
struct MoveParams {
  Cache cache;
  PageScales scales;
  Record record;
  Batch batch;
  const int32_t* source;
  const int32_t* target;
  const int32_t* moves;
  int max_moves, heads;
  int lists;  // layers * B * heads
  int vecs;   // 16-byte vectors of an entry
  int last;   // page scales: this launch moves into the page that the context ends in, and the other one into the others
};

constexpr int kMoveWarps = 4;

// One (layer, request, head) of a move.
struct MoveList {
  int b, head, n, end;
  int64_t layer;
  const int32_t* source;
  const int32_t* target;
  const int32_t* table;
  __device__ MoveList(const MoveParams& P, int list) {
    head = list % P.heads;
    const int rest = list / P.heads;
    b = rest % P.batch.B, layer = rest / P.batch.B;
    n = min(max(P.moves[list], 0), P.max_moves);
    end = batch_context(P.batch, b);
    source = P.source + (int64_t)list * P.max_moves;
    target = P.target + (int64_t)list * P.max_moves;
    table = P.batch.pages + (int64_t)b * P.batch.max_pages;
  }
  __device__ int page_of(const MoveParams& P, int slot) const {
    const int page = __ldg(table + (slot >> P.cache.page_shift));
    return page < 0 || page >= P.cache.num_pages ? -1 : page;
  }
  // Pages of move i; false: it is left out.
  __device__ bool pages(const MoveParams& P, int i, int& s, int& t, int& from, int& to) const {
    s = source[i], t = target[i];
    if (t < 0 || t >= end || s < end || s >= P.batch.slots) return false;
    from = page_of(P, s), to = page_of(P, t);
    return from >= 0 && to >= 0;
  }
};

__device__ __forceinline__ void move_record(const MoveParams& P, const MoveList& m, int s, int t, int from, int to) {
  const int mask = (1 << P.cache.page_shift) - 1;
  const int64_t base = m.layer * P.record.layer;
  const int64_t src = base + (((int64_t)from * P.heads + m.head) << P.cache.page_shift) + (s & mask);
  const int64_t dst = base + (((int64_t)to * P.heads + m.head) << P.cache.page_shift) + (t & mask);
  if (P.record.weight) P.record.weight[dst] = P.record.weight[src];
  if (P.record.position) P.record.position[dst] = P.record.position[src];
}

// Entries as they are.  A warp takes 32 moves: each lane works out one, then the warp copies their vectors, kAhead of
// keys and of values in flight.
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const __grid_constant__ MoveParams P) {
  constexpr int kAhead = 4;
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int mask = (1 << P.cache.page_shift) - 1;
  const int at_once = 32 / P.vecs, vec = lane % P.vecs;  // entries that the warp takes in one go, 2 to 8
  for (int list = blockIdx.y; list < P.lists; list += gridDim.y) {
    const MoveList m(P, list);
    for (int i0 = (blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * 32; i0 < m.n; i0 += gridDim.x * kMoveWarps * 32) {
      int s = 0, t = 0, from = 0, to = 0;
      const bool is = i0 + lane < m.n && m.pages(P, i0 + lane, s, t, from, to);
      const uint32_t all = __ballot_sync(~0u, is);
      const int64_t src = from * P.cache.page + (s & mask) * P.cache.slot, dst = to * P.cache.page + (t & mask) * P.cache.slot;
      if (is) move_record(P, m, s, t, from, to);
      const int64_t base = m.layer * P.cache.layer + m.head * P.cache.head + vec * 16;
      for (int e0 = lane / P.vecs; e0 < 32; e0 += at_once * kAhead) {
        uint4 k[kAhead], v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int e = e0 + j * at_once;
          const int64_t a = base + __shfl_sync(~0u, src, e & 31);
          if (e < 32 && ((all >> e) & 1))
            k[j] = *reinterpret_cast<const uint4*>(P.cache.k + a), v[j] = *reinterpret_cast<const uint4*>(P.cache.v + a);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int e = e0 + j * at_once;
          const int64_t d = base + __shfl_sync(~0u, dst, e & 31);
          if (e < 32 && ((all >> e) & 1))
            *reinterpret_cast<uint4*>(P.cache.k + d) = k[j], *reinterpret_cast<uint4*>(P.cache.v + d) = v[j];
        }
      }
    }
  }
}

// Moves among which a warp's pages begin: more for large pages, of which it then has whole ones (32 requests, half of 8000 to
// 16000 entries, pages of 32: 150 us with 32, 154 with 128; of 64: 253, 271; of 256: 347, 266).
constexpr int kMoveStretch = 32, kMoveStretchLong = 128, kLongPage = 128;

// Entries of a cache with page scales.  A warp takes the pages whose first move lies in its stretch of the list (targets
// are in ascending order), as many at a time as have 32 moves together; a page with more goes by itself.  The page that the
// context ends in holds sources of other pages' moves, whose scale is still needed: its own moves wait for a launch of their own.
template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32, 6) page_move_kernel(const __grid_constant__ MoveParams P) {
  __shared__ Exchange exchange[kMoveWarps];
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = P.cache.page_shift, page_size = 1 << shift, mask = page_size - 1;
  const int stretch = page_size >= kLongPage ? kMoveStretchLong : kMoveStretch;
  Exchange& x = exchange[warp];
  const bool is_v = blockIdx.y & 1;
  for (int list = blockIdx.y >> 1; list < P.lists; list += gridDim.y >> 1) {
    const MoveList m(P, list);
    const int last = m.end & mask ? m.end >> shift : -1;  // the page that the context ends in
    if (m.n == 0 || (P.last && last < 0)) continue;
    int begin = 0, stop = m.n;  // the moves that this launch takes
    if (last >= 0) {            // the first move into the last page: any number that are left out may be behind the page's own
      int first = m.n;
      for (int i = m.n - 1 - lane;; i -= 32) {
        const uint32_t in = __ballot_sync(~0u, i >= 0 && m.target[max(i, 0)] >> shift >= last);
        first -= in == ~0u ? 32 : __ffs(~in) - 1;
        if (in != ~0u) break;
      }
      if (P.last) begin = first;
      else stop = first;
    }
    const Side c = {(is_v ? P.cache.v : P.cache.k) + m.layer * P.cache.layer + m.head * P.cache.head,
                    (is_v ? P.scales.v : P.scales.k) + m.layer * P.scales.layer + m.head, P.heads, P.cache.slot, P.cache.page, page_size};
    const auto info = [&](int i) {
      Move y = {false, 0, 0, 0, -1, lane, lane};
      if (i >= stop) return y;
      int s, t;
      y.is = m.pages(P, i, s, t, y.from, y.to);
      if (y.is) y.src = y.from * P.cache.page + (s & mask) * P.cache.slot, y.dst = y.to * P.cache.page + (t & mask) * P.cache.slot;
      return y;
    };
    for (int i0 = begin + (blockIdx.x * kMoveWarps + warp) * stretch; i0 < stop; i0 += gridDim.x * kMoveWarps * stretch) {
      const int bound = min(i0 + stretch, stop);
      int before = i0 > begin ? m.target[i0 - 1] >> shift : -1 << 30;  // the page of the move before
      bool looking = true;  // for the first page that begins here
      for (int i = i0; i < bound;) {
        const int page = i + lane < stop ? m.target[i + lane] >> shift : 1 << 30, next = i + 32 < stop ? m.target[i + 32] >> shift : 1 << 30;
        int previous = __shfl_up_sync(~0u, page, 1);
        if (lane == 0) previous = before;
        const uint32_t starts = __ballot_sync(~0u, page != previous);
        if (looking && !(starts & 1)) {  // the stretch begins within a page that is another warp's
          const int skip = starts ? __ffs(starts) - 1 : 32;
          before = __shfl_sync(~0u, page, skip - 1);
          i += skip;
          continue;
        }
        looking = false;
        // pages that begin before `bound` and end within these 32 moves
        const int valid = min(32, stop - i);
        const uint32_t behind = bound - i < 32 ? starts & (~0u << (bound - i)) : 0;
        int n = behind ? __ffs(behind) - 1 : valid;
        if (n == 32 && next == __shfl_sync(~0u, page, 31)) n = 31 - __clz(starts);  // the last one goes on
        if (n > 0) {
          Move y = {false, 0, 0, 0, -1, lane, lane};
          int s = 0, t = 0;
          if (lane < n) {
            const uint32_t mine = starts & (lane == 31 ? ~0u : (2u << lane) - 1), after = lane == 31 ? 0u : starts & (~0u << (lane + 1));
            y.is = m.pages(P, i + lane, s, t, y.from, y.to);
            y.lo = 31 - __clz(mine | 1), y.hi = min(after ? __ffs(after) - 2 : 31, n - 1);
            if (page >= 0 && page << shift < m.end) y.to = m.page_of(P, page << shift);  // also where this move is left out
            if (y.is) {
              y.src = y.from * P.cache.page + (s & mask) * P.cache.slot, y.dst = y.to * P.cache.page + (t & mask) * P.cache.slot;
              if (!is_v) move_record(P, m, s, t, y.from, y.to);
            }
          }
          move_batch<D>(c, y, n, t & mask, lane < n ? min(m.end - (page << shift), page_size) : 0, x);
        } else {  // a page of more than 32 moves
          const int ordinal = __shfl_sync(~0u, page, 0);
          for (n = 32; i + n < stop;) {
            const uint32_t same = __ballot_sync(~0u, i + n + lane < stop && m.target[i + n + lane] >> shift == ordinal);
            n += same == ~0u ? 32 : __ffs(~same) - 1;
            if (same != ~0u) break;
          }
          if (ordinal >= 0 && ordinal << shift < m.end) {
            const int into = m.page_of(P, ordinal << shift);
            if (into >= 0)
              move_page<D>(
                  c, n, into, min(m.end - (ordinal << shift), page_size), x,
                  [&](int k) { return info(k < n ? i + k : stop); },
                  [&](const Move& y) { return (int)((y.dst - into * P.cache.page) / P.cache.slot); });
            for (int k = lane; k < n && !is_v; k += 32) {
              int s, t, from, to;
              if (m.pages(P, i + k, s, t, from, to)) move_record(P, m, s, t, from, to);
            }
          }
        }
        before = __shfl_sync(~0u, page, min(n, 32) - 1);
        i += n;
      }
    }
  }
}

}  // namespace sv

using namespace sv;

extern "C" {

spec_status_t spec_kv_keep_ex(const spec_kv_cache_t* cache, const spec_kv_page_scales_t* scales,
                              const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* path,
                              const int32_t* n_keep, int32_t max_keep, void* stream) {
  spec_status_t s = check_cache(cache, false);
  if (s == SPEC_OK) s = check_scales(scales, cache);
  if (s == SPEC_OK) s = check_record(record, cache);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (max_keep < 0) return SPEC_ERR_INVALID_ARG;
  if (max_keep > (scales ? SPEC_MAX_NEW : SPEC_MAX_SLOTS)) return SPEC_ERR_UNSUPPORTED;
  const int64_t lists = (int64_t)cache->layers * batch->B * cache->heads;
  if ((int64_t)cache->layers * cache->heads > 0x3fffffffll || lists > 0x3fffffffll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0 || max_keep == 0) return SPEC_OK;
  if (!path || !n_keep) return SPEC_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!scales) {
    s = spec_kv_keep(cache, batch, path, n_keep, max_keep, stream);
    if (s != SPEC_OK) return s;
  } else {
    const int D = cache->head_dim, lists_each = cache->layers * cache->heads * 2;
    const PageKeepParams P = {cache_of(cache), scales_of(scales), batch_of(batch, cache), path, n_keep, max_keep, cache->heads, lists_each};
    const int64_t most = (lists_each + kPageKeepWarps - 1) / kPageKeepWarps, rounds = (most * batch->B + 2047) / 2048;
    const dim3 grid((unsigned)((most + rounds - 1) / rounds), batch->B), block(kPageKeepWarps * 32);
    const bool big = max_keep > 32;
    const size_t smem = big ? (size_t)kPageKeepWarps * SPEC_MAX_NEW * D : 0;
    auto kern = big ? (D == 128 ? page_keep_kernel<128, true> : page_keep_kernel<64, true>)
                    : (D == 128 ? page_keep_kernel<128, false> : page_keep_kernel<64, false>);
    if (launch_early(kern, grid, block, smem, st, P) != cudaSuccess) return SPEC_ERR_CUDA;
  }
  if (record && (record->weight || record->position)) {
    const RecordKeepParams R = {cache_of(cache), record_of(record), batch_of(batch, cache), path, n_keep, max_keep, cache->heads, lists};
    if (launch_early(record_keep_kernel, dim3((unsigned)((lists + 127) / 128)), dim3(128), 0, st, R) != cudaSuccess) return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

spec_status_t spec_kv_move(const spec_kv_cache_t* cache, const spec_kv_page_scales_t* scales,
                           const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* source,
                           const int32_t* target, const int32_t* moves, int32_t max_moves, void* stream) {
  spec_status_t s = check_cache(cache, false);
  if (s == SPEC_OK) s = check_scales(scales, cache);
  if (s == SPEC_OK) s = check_record(record, cache);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (max_moves < 0) return SPEC_ERR_INVALID_ARG;
  const int64_t lists = (int64_t)cache->layers * batch->B * cache->heads;
  if (lists > 0x3fffffffll || batch->B > SPEC_MAX_BATCH || max_moves > SPEC_MAX_SLOTS) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0 || max_moves == 0) return SPEC_OK;
  if (!source || !target || !moves) return SPEC_ERR_INVALID_ARG;
  MoveParams P = {};
  P.cache = cache_of(cache), P.scales = scales_of(scales), P.record = record_of(record), P.batch = batch_of(batch, cache);
  P.source = source, P.target = target, P.moves = moves;
  P.max_moves = max_moves, P.heads = cache->heads, P.lists = (int)lists;
  P.vecs = cache->head_dim * (cache->dtype == SPEC_DTYPE_BF16 ? 2 : 1) / 16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 block(kMoveWarps * 32);
  // blocks for the lists, and more for each where there are few; a list's moves go round its blocks
  const int64_t most = ((int64_t)max_moves + kMoveWarps * 32 - 1) / (kMoveWarps * 32);
  const int64_t rows = lists * (scales ? 2 : 1);
  const unsigned y = (unsigned)(rows < 65534 ? rows : 65534);
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  int64_t x = (32 * (int64_t)sms + y - 1) / y;
  if (x > most) x = most;
  if (!scales) return launch_early(move_kernel, dim3((unsigned)x, y), block, 0, st, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  auto kern = cache->head_dim == 128 ? page_move_kernel<128> : page_move_kernel<64>;
  if (launch_early(kern, dim3((unsigned)x, y), block, 0, st, P) != cudaSuccess) return SPEC_ERR_CUDA;
  P.last = 1;
  return launch_early(kern, dim3(1, y), block, 0, st, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
