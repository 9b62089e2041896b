// spec_pages.cu — moves of cache entries: spec_kv_keep_ex (the accepted branch in a cache with page scales, and what is
// recorded of the entries) and spec_kv_move (the entries that stay, after spec_kv_select).  An entry that moves into
// another page of an E4M3 cache with page scales is a code of that page's scale from then on, which may have to grow, and
// then the page's other codes change with it; so a page's moves are one warp's work.  All of it is bound by memory
// traffic, or by the launch where little moves.

#include "decode_common.cuh"

namespace sv {

// What a warp needs of one page that entries move into.
struct Target {
  char* rows;       // row 0 of the page, of one head
  int64_t slot;     // bytes from row to row
  float* scale;
  int end;          // rows from here on hold nothing that stays
};

// The values of 16 codes at scale `from`, as codes at scale `to`.
__device__ __forceinline__ uint4 recoded(uint4 w, float from, float to, float inverse) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = unpack_e4m3(x[i]);
    x[i] = pack_e4m3(quotient(f.x * from, to, inverse), quotient(f.y * from, to, inverse), quotient(f.z * from, to, inverse),
                     quotient(f.w * from, to, inverse));
  }
  return w;
}

// A warp's moves into one page: entries 0 .. n - 1, of which fetch(i, vec, scale) gives 16 codes (vector vec) and their
// scale, and row(i) the page's row, or -1 for a move that is left out.  `taken` [page_size / 32] marks the rows.
template <int D, typename Fetch, typename Row>
__device__ void put_entries(const Target& to, int n, uint32_t* taken, int page_size, Fetch fetch, Row row) {
  constexpr int kVecs = D / 16, kAtOnce = 32 / kVecs;
  const int lane = threadIdx.x & 31, vec = lane % kVecs, mine = lane / kVecs;
  float most = 0.0f;  // of the finite magnitudes
  for (int i0 = 0; i0 < n; i0 += kAtOnce) {
    const int i = i0 + mine;
    if (i >= n || row(i) < 0) continue;
    float scale;
    const uint4 w = fetch(i, vec, scale);
    const uint32_t* x = reinterpret_cast<const uint32_t*>(&w);
    uint32_t top = 0;  // a larger code without its sign is a larger magnitude; 0x7F is NaN
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t size = x[j] & 0x7F7F7F7Fu;
      top = __vmaxu4(top, size & ~__vcmpeq4(size, 0x7F7F7F7Fu));
    }
    top = max(max(top & 0xFF, (top >> 8) & 0xFF), max((top >> 16) & 0xFF, top >> 24));
    const float size = unpack_e4m3(top).x * fabsf(scale);
    if (size < INFINITY) most = fmaxf(most, size);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  const float old = *to.scale;
  const bool counts = scale_counts(old);
  const float need = scale_need(most), scale = counts ? fmaxf(old, need) : need, inverse = 1.0f / scale;

  if (counts && need > old) {
    for (int i = lane; i < page_size / 32 + 1; i += 32) taken[i] = 0;
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
      const int r = row(i);
      if (r >= 0) atomicOr(&taken[r >> 5], 1u << (r & 31));
    }
    __syncwarp();
    const float ratio = old * inverse;
    for (int r0 = 0; r0 < to.end; r0 += kAtOnce) {
      const int r = r0 + mine;
      if (r >= to.end || ((taken[r >> 5] >> (r & 31)) & 1)) continue;
      uint4* p = reinterpret_cast<uint4*>(to.rows + r * to.slot + vec * 16);
      *p = rescaled(*p, ratio);
    }
  }
  for (int i0 = 0; i0 < n; i0 += kAtOnce) {
    const int i = i0 + mine, r = i < n ? row(i) : -1;
    if (r < 0) continue;
    float from;
    const uint4 w = fetch(i, vec, from);
    *reinterpret_cast<uint4*>(to.rows + r * to.slot + vec * 16) = from == scale ? w : recoded(w, from, scale, inverse);
  }
  __syncwarp();  // an entry may come from the same page: its old scale was needed until here
  if (lane == 0) *to.scale = scale;
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
  int64_t lists;  // layers * B * heads * 2
};

constexpr int kPageKeepWarps = 4;

// A warp per (layer, request, head, k or v).  The moved entries and their scales come into shared memory before the first
// one is written: a path's targets may be its later sources, and a page's scale may change.
template <int D>
__global__ void __launch_bounds__(kPageKeepWarps * 32) page_keep_kernel(const __grid_constant__ PageKeepParams P) {
  __shared__ uint4 entries[kPageKeepWarps][SPEC_MAX_NEW * (D / 16)];
  __shared__ float scales[kPageKeepWarps][SPEC_MAX_NEW];
  __shared__ int targets[kPageKeepWarps][SPEC_MAX_NEW];                // slots, -1: left out
  __shared__ uint32_t taken[kPageKeepWarps][SPEC_MAX_PAGE / 32 + 1];
  pdl_launch_next();
  pdl_wait();
  constexpr int kVecs = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t list = (int64_t)blockIdx.x * kPageKeepWarps + warp;
  if (list >= P.lists) return;
  const bool is_v = list & 1;
  list >>= 1;
  const int head = list % P.heads;
  list /= P.heads;
  const int b = list % P.batch.B, layer = list / P.batch.B;

  const int n = min(max(__ldg(P.n_keep + b), 0), P.max_keep);
  const int ctx = batch_context(P.batch, b), page_size = 1 << P.cache.page_shift;
  char* base = (is_v ? P.cache.v : P.cache.k) + layer * P.cache.layer + head * P.cache.head;
  float* scale = (is_v ? P.scales.v : P.scales.k) + layer * P.scales.layer + head;
  const int32_t* table = P.batch.pages + (int64_t)b * P.batch.max_pages;
  bool any = false;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    int64_t src = -1, dst = -1;
    if (i < n) {
      const int p = __ldg(P.path + (int64_t)b * P.max_keep + i);
      if (p != i && p >= 0 && p < P.batch.slots) {
        dst = slot_offset(P.batch, P.cache, b, ctx + i);
        src = slot_offset(P.batch, P.cache, b, ctx + p);
      }
      targets[warp][i] = src >= 0 && dst >= 0 ? ctx + i : -1;
      if (src >= 0 && dst >= 0) scales[warp][i] = scale[(int64_t)__ldg(table + ((ctx + p) >> P.cache.page_shift)) * P.heads];
    }
    const uint32_t moves = __ballot_sync(~0u, src >= 0 && dst >= 0);
    any |= moves != 0;
    for (int u = lane; u < 32 * kVecs; u += 32) {
      const int64_t from = __shfl_sync(~0u, src, u / kVecs);  // the same u / kVecs for lanes of one entry
      if ((moves >> (u / kVecs)) & 1) entries[warp][i0 * kVecs + u] = *reinterpret_cast<const uint4*>(base + from + (u % kVecs) * 16);
    }
  }
  __syncwarp();
  if (!any) return;
  const int end = (int)min((int64_t)ctx + n, (int64_t)P.batch.slots);
  for (int i = 0; i < n;) {  // a page at a time
    const int ordinal = (ctx + i) >> P.cache.page_shift, first = i;
    bool moves = false;
    for (; i < n && (ctx + i) >> P.cache.page_shift == ordinal; ++i) moves |= targets[warp][i] >= 0;
    if (!moves) continue;
    const int page = __ldg(table + ordinal);  // in the pool: a move into it is not left out
    const Target to = {base + page * P.cache.page, P.cache.slot, scale + (int64_t)page * P.heads,
                       min(end - (ordinal << P.cache.page_shift), page_size)};
    put_entries<D>(
        to, i - first, taken[warp], page_size,
        [&](int k, int vec, float& s) {
          s = scales[warp][first + k];
          return entries[warp][(first + k) * kVecs + vec];
        },
        [&](int k) {
          const int t = targets[warp][first + k];
          return t < 0 ? -1 : t & (page_size - 1);
        });
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

// Entries as they are.  A warp takes 32 moves: each lane works out one, then the warp copies their vectors.
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const __grid_constant__ MoveParams P) {
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int mask = (1 << P.cache.page_shift) - 1;
  for (int list = blockIdx.y; list < P.lists; list += gridDim.y) {
    const MoveList m(P, list);
    for (int i0 = (blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * 32; i0 < m.n; i0 += gridDim.x * kMoveWarps * 32) {
      int s = 0, t = 0, from = 0, to = 0;
      const bool is = i0 + lane < m.n && m.pages(P, i0 + lane, s, t, from, to);
      const uint32_t all = __ballot_sync(~0u, is);
      const int64_t src = from * P.cache.page + (s & mask) * P.cache.slot, dst = to * P.cache.page + (t & mask) * P.cache.slot;
      if (is) move_record(P, m, s, t, from, to);
      const int64_t base = m.layer * P.cache.layer + m.head * P.cache.head;
      for (int u = lane; u < 32 * P.vecs; u += 32) {
        const int64_t a = __shfl_sync(~0u, src, u / P.vecs), d = __shfl_sync(~0u, dst, u / P.vecs);
        if (!((all >> (u / P.vecs)) & 1)) continue;
        const int64_t at = base + (u % P.vecs) * 16;
        const uint4 k = *reinterpret_cast<const uint4*>(P.cache.k + at + a), v = *reinterpret_cast<const uint4*>(P.cache.v + at + a);
        *reinterpret_cast<uint4*>(P.cache.k + at + d) = k;
        *reinterpret_cast<uint4*>(P.cache.v + at + d) = v;
      }
    }
  }
}

// Entries of a cache with page scales.  A warp takes the pages whose first move lies among its 32 moves (targets are in
// ascending order), and all moves into them.  The page that the context ends in holds sources of other pages' moves, whose
// scale is still needed: its own moves wait for a launch of their own.
template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) page_move_kernel(const __grid_constant__ MoveParams P) {
  __shared__ uint32_t taken_of[kMoveWarps][SPEC_MAX_PAGE / 32 + 1];
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = P.cache.page_shift, page_size = 1 << shift, mask = page_size - 1;
  for (int list = blockIdx.y >> 1; list < P.lists; list += gridDim.y >> 1) {
    const MoveList m(P, list);
    const bool is_v = blockIdx.y & 1;
    const int last = m.end & mask ? m.end >> shift : -1;  // the page that the context ends in
    if (P.last && last < 0) continue;
    int first = 0, stop = m.n;  // the first moves of the pages that this launch takes
    // the first move into the last page
    if (last >= 0) {
      int lo = 0, hi = m.n;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (m.target[mid] >> shift < last) lo = mid + 1;
        else hi = mid;
      }
      if (P.last) first = lo;
      else stop = lo;
    }
    char* base = (is_v ? P.cache.v : P.cache.k) + m.layer * P.cache.layer + m.head * P.cache.head;
    float* scales = (is_v ? P.scales.v : P.scales.k) + m.layer * P.scales.layer + m.head;
    for (int i0 = first + (blockIdx.x * kMoveWarps + warp) * 32; i0 < stop; i0 += gridDim.x * kMoveWarps * 32) {
      const int i = i0 + lane;
      const int page = i < stop ? m.target[i] >> shift : -2;
      int before = __shfl_up_sync(~0u, page, 1);
      if (lane == 0) before = i0 > first ? m.target[i0 - 1] >> shift : -2;
      uint32_t starts = __ballot_sync(~0u, i < stop && page != before);
      while (starts) {
        const int begin = __ffs(starts) - 1;
        starts &= starts - 1;
        const int ordinal = __shfl_sync(~0u, page, begin);
        // its moves: up to the next start, or on beyond these 32
        int n = (starts ? __ffs(starts) - 1 : min(32, stop - i0)) - begin;
        if (!starts)
          for (int j = i0 + begin + n; j < stop; j += 32) {
            const bool same = j + lane < stop && m.target[j + lane] >> shift == ordinal;
            const uint32_t all = __ballot_sync(~0u, same);
            n += all == ~0u ? 32 : __ffs(~all) - 1;
            if (all != ~0u) break;
          }
        const int at = i0 + begin;
        if (ordinal < 0 || ordinal << shift >= m.end) continue;
        const int into = m.page_of(P, ordinal << shift);
        if (into < 0) continue;
        const Target to = {base + into * P.cache.page, P.cache.slot, scales + (int64_t)into * P.heads,
                           min(m.end - (ordinal << shift), page_size)};
        put_entries<D>(
            to, n, taken_of[warp], page_size,
            [&](int k, int vec, float& scale) {
              const int s = m.source[at + k], p = m.page_of(P, s);
              scale = scales[(int64_t)p * P.heads];
              return *reinterpret_cast<const uint4*>(base + p * P.cache.page + (s & mask) * P.cache.slot + vec * 16);
            },
            [&](int k) {
              int s, t, from, page;
              return m.pages(P, at + k, s, t, from, page) ? t & mask : -1;
            });
        if (!is_v)
          for (int k = lane; k < n; k += 32) {
            int s, t, from, page;
            if (m.pages(P, at + k, s, t, from, page)) move_record(P, m, s, t, from, page);
          }
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
  if (scales && max_keep > SPEC_MAX_NEW) return SPEC_ERR_UNSUPPORTED;
  const int64_t lists = (int64_t)cache->layers * batch->B * cache->heads;
  if (lists > 0x3fffffffll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0 || max_keep == 0) return SPEC_OK;
  if (!path || !n_keep) return SPEC_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!scales) {
    s = spec_kv_keep(cache, batch, path, n_keep, max_keep, stream);
    if (s != SPEC_OK) return s;
  } else {
    const PageKeepParams P = {cache_of(cache), scales_of(scales), batch_of(batch, cache), path, n_keep, max_keep, cache->heads, lists * 2};
    const dim3 grid((unsigned)((lists * 2 + kPageKeepWarps - 1) / kPageKeepWarps));
    auto kern = cache->head_dim == 128 ? page_keep_kernel<128> : page_keep_kernel<64>;
    if (launch_early(kern, grid, dim3(kPageKeepWarps * 32), 0, st, P) != cudaSuccess) return SPEC_ERR_CUDA;
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
  if (lists > 0x3fffffffll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;
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
  const int sides = scales ? 2 : 1;
  const int64_t rows = lists * sides, most = ((int64_t)max_moves + kMoveWarps * 32 - 1) / (kMoveWarps * 32);
  const unsigned y = (unsigned)(rows < 65534 ? rows : 65534);
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  int64_t x = (8 * sms + y - 1) / y;
  if (x > most) x = most;
  if (!scales) return launch_early(move_kernel, dim3((unsigned)x, y), block, 0, st, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  auto kern = cache->head_dim == 128 ? page_move_kernel<128> : page_move_kernel<64>;
  if (launch_early(kern, dim3((unsigned)x, y), block, 0, st, P) != cudaSuccess) return SPEC_ERR_CUDA;
  P.last = 1;
  return launch_early(kern, dim3(1, y), block, 0, st, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
