// tile_stream.cuh — what the kernels that stream the paged cache through the matrix unit share: PTX, descriptors and
// tensor maps, the split of queries for E4M3 products, and the line of tiles that is cut over the SMs.
#pragma once

#include <cuda.h>

#include <atomic>

#include "decode_common.cuh"

namespace sv {

extern std::atomic<int32_t> g_test_hooks;  // spec_verify_set_test_hooks

constexpr int kTileSlots = 128;  // slots per tile = rows of the matrix unit
constexpr int kMaxRows = 128;    // query rows of one item
constexpr float kLog2e = 1.4426950408889634f;

// What the cache holds: E4M3 with a scale per head, or per page and head.  (kBf16Lse: the attention over bf16 that leaves lse.)
enum { kBf16 = 0, kE4m3 = 1, kE4m3Pages = 2, kBf16Lse = 3 };
__host__ __device__ constexpr bool holds_e4m3(int kind) { return kind == kE4m3 || kind == kE4m3Pages; }

// ------------------------------------------------------------------------------------------------
// PTX
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {  // does not suspend
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Waits for the phase, `limit` tries at most; a wait that runs out marks the block dead, which ends every other
// wait in it soon after.  Nothing here waits on another block.
struct Patience {
  volatile int* dead;
  int limit;
};
constexpr int kWaitTries = 1 << 22;
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const Patience& w) {
  if (mbar_try(bar, parity)) return true;
  for (int i = 0; i < w.limit; ++i) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 255) == 0 && *w.dead) return false;
  }
  *w.dead = 1;
  return false;
}
// the same for a whole warp that goes on together
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, const Patience& w) {
  return __all_sync(~0u, mbar_wait(bar, parity, w));
}
// Behind a wait that ran out: sees what is in flight come to its end before the block goes.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < (1 << 16) && !mbar_try(bar, parity); ++i) {
  }
}

// A copy by one elected lane of a warp that goes through the code together (see tc_mma).
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                         uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Products are issued by one elected lane of a warp that goes through the code together: the descriptors then
// stay in uniform registers (measured: 43 to 55 cycles per product of 128 x 16..80 x 32 bytes, against 90 to
// 118 from a branch that one lane takes).
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// kind::f16 (fp16 or bf16 operands) or kind::f8f6f4 (E4M3, and E5M2 as B)
template <bool F8>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A load from TMEM and the wait for it, in one statement: nothing can use the registers in between.
template <int N>
__device__ __forceinline__ void tm_load(uint32_t addr, float (&x)[N]);
template <>
__device__ __forceinline__ void tm_load<8>(uint32_t addr, float (&x)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
}
template <>
__device__ __forceinline__ void tm_load<16>(uint32_t addr, float (&x)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tm_store(uint32_t addr, const float (&x)[N]);
template <>
__device__ __forceinline__ void tm_store<8>(uint32_t addr, const float (&x)[8]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <>
__device__ __forceinline__ void tm_store<16>(uint32_t addr, const float (&x)[16]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 128 threads of one warpgroup
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}

// In an instruction's descriptor: B is E5M2 (A and E4M3 are 0), for the remainders of split queries.
constexpr uint32_t kSecondE5m2 = 1u << 10;

// Shared-memory matrix descriptors: 128-byte swizzle (or 64-byte: E4M3 rows of 64), strides in bytes.  Along
// a swizzled row lies the reduction (Q and K) or the free dimension (V^T and P^T, "transposed" in the
// instruction).
template <int ROW = 128>
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
         1ull << 46 | (ROW == 128 ? 2ull : 4ull) << 61;
}

// Over an E4M3 cache the queries are 8-bit numbers too: a row is scaled by a power of two to a largest element in [128, 256), and
// its 8-bit significands split into E4M3's 4 bits and a remainder of at most 8 units in the last place, which are E5M2's 3 bits.
// That is exact where an element, scaled, is a normal E4M3 number, 2^-6 (2^-13 of the largest at least); below, what E4M3's step of
// 2^-9 leaves is 2^-10 at most and off by 2^-14, 2^-21 of the largest.  (E4M3 has no finer steps for the remainder than for the number
// itself: 2^-17.  One query channel that is 100 times the others is usual.)  The scale goes into the row's factor, beside `c`.
// rows: a multiple of 16.  The split overwrites the row (a TMA-loaded [halves][NT][128 bytes]): no other row's lines.
template <int D, int NT, int THREADS>
__device__ __forceinline__ void split_queries(char* q, int tid, int rows, float c, float* mult) {
  constexpr int kLanes = D / 16;  // threads per row, 16 elements each
  const int i = tid % kLanes;
#pragma unroll 1
  for (int row = tid / kLanes; row < rows; row += THREADS / kLanes) {
    const int sw = row & 7;
    const char* src = q + (i * 16 / 64) * (NT * 128) + row * 128;
    const int v0 = (i * 16 % 64) / 8;
    float x[16];
    unpack8(*reinterpret_cast<const uint4*>(src + ((v0 ^ sw) * 16)), reinterpret_cast<float(&)[8]>(x[0]));
    unpack8(*reinterpret_cast<const uint4*>(src + (((v0 + 1) ^ sw) * 16)), reinterpret_cast<float(&)[8]>(x[8]));
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(~0u, top, d));
    const int up = min(134 - (int)(top >> 23), 127);  // 7 minus the largest element's exponent
    const float scale = __uint_as_float((uint32_t)(up + 127) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e + k] *= scale;
      hi[e / 4] = pack_e4m3(x[e], x[e + 1], x[e + 2], x[e + 3]);
      const float4 u = unpack_e4m3(hi[e / 4]);
      lo[e / 4] = pack_e5m2(x[e] - u.x, x[e + 1] - u.y, x[e + 2] - u.z, x[e + 3] - u.w);
    }
    __syncwarp();  // the row is read
    *reinterpret_cast<uint4*>(q + row * 128 + ((i ^ sw) * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    char* rest = D == 128 ? q + NT * 128 + row * 128 + ((i ^ sw) * 16) : q + row * 128 + (((i + 4) ^ sw) * 16);
    *reinterpret_cast<uint4*>(rest) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (i == 0) mult[row] = top >= 0x7F800000u ? NAN : ldexpf(c, -up);  // infinite or NaN: the row is NaN
  }
}

// ------------------------------------------------------------------------------------------------
// the line of tiles
// ------------------------------------------------------------------------------------------------
struct Segment {
  int b, head, row_group;
  int tile0, tile1, tiles;  // this part of the item's tiles
  int ctx, tokens, end;     // context, valid new tokens, end of the slots
  int item_end;             // where the item ends on the line
};

// Slots of a request that anything reads, and its tiles (one at least: its rows are written there).
__device__ __forceinline__ int request_end(int ctx, int tokens, int slots) { return tokens > 0 ? min(ctx + tokens, slots) : 0; }
__device__ __forceinline__ int request_tiles(int end) { return max(1, (end + kTileSlots - 1) / kTileSlots); }
// An item's length on the line: its tiles, behind what beginning and ending it costs.
template <typename Params>
__device__ __forceinline__ int request_length(const Params& P, int ctx, int tokens) {
  return request_tiles(request_end(ctx, tokens, P.batch.slots)) + P.item_cost;
}

// Where CTA c's part of the line begins.
__device__ __forceinline__ int line_cut(int total, int c, int ctas) { return (int)((int64_t)total * c / ctas); }

// The part of the line that is this CTA's, by a scan over the requests' lengths; the whole block comes here, and what it
// wrote to shared memory before (and to TMEM's address) is there behind it.
struct LinePart {
  int first, count, total;
  int start_b, start_offset;  // the request it begins in, and where
};
template <int THREADS, typename Params>
__device__ __forceinline__ void find_part(const Params& P, int* warp_sum, int* found_b, int* found_offset, LinePart& part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_request = P.heads * P.row_groups;
  const int chunk = (P.batch.B + THREADS - 1) / THREADS;
  const int b_first = min((int)threadIdx.x * chunk, P.batch.B), b_last = min(b_first + chunk, P.batch.B);
  int mine = 0;
  for (int b = b_first; b < b_last; ++b)
    mine += request_length(P, batch_context(P.batch, b), batch_tokens(P.batch, b)) * per_request;
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int x = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) warp_sum[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int ctas = min((int)gridDim.x, total);  // the others have no part
  const int first = line_cut(total, min((int)blockIdx.x, ctas), ctas);
  const int count = line_cut(total, min((int)blockIdx.x + 1, ctas), ctas) - first;
  if (count > 0 && first >= before && first < before + mine) {
    int b = b_first, rest = first - before;
    for (;; ++b) {
      const int n = request_length(P, batch_context(P.batch, b), batch_tokens(P.batch, b)) * per_request;
      if (rest < n) break;
      rest -= n;
    }
    *found_b = b, *found_offset = rest;
  }
  __syncthreads();
  part = {first, count, total, count > 0 ? *found_b : 0, count > 0 ? *found_offset : 0};
}

// Every role of a CTA walks the same part of the line by itself.  (Params: batch, heads, row_groups, item_cost and whole.)
template <typename Params>
struct Walk {
  const Params& P;
  int b, head, row_group, at, left, stop;  // at: within the item
  int ctx, tokens, next_ctx, next_tokens;

  __device__ Walk(const Params& p, int b0, int offset, int first, int count) : P(p), b(b0), left(count), stop(first + count) {
    head = row_group = at = ctx = tokens = next_ctx = next_tokens = 0;
    if (left <= 0) return;
    ctx = batch_context(P.batch, b);
    tokens = batch_tokens(P.batch, b);
    const int n = request_length(P, ctx, tokens);
    const int index = offset / n;
    at = offset - index * n;
    head = index / P.row_groups;
    row_group = index - head * P.row_groups;
    prefetch();
  }
  __device__ void prefetch() {
    if (b + 1 < P.batch.B) {
      next_ctx = batch_context(P.batch, b + 1);
      next_tokens = batch_tokens(P.batch, b + 1);
    }
  }
  __device__ bool next(Segment& s) {
    while (left > 0) {
      s.b = b, s.head = head, s.row_group = row_group;
      s.ctx = ctx, s.tokens = tokens, s.end = request_end(ctx, tokens, P.batch.slots);
      s.tiles = request_tiles(s.end);
      const int length = s.tiles + P.item_cost;
      const int n = P.whole ? length - at : min(length - at, left);
      const bool other = P.whole && at > 0;  // it began in an earlier CTA
      s.tile0 = max(at - P.item_cost, 0), s.tile1 = max(at + n - P.item_cost, 0);
      left -= n;
      at += n;
      s.item_end = stop - left + length - at;
      if (at == length) {
        at = 0;
        if (++row_group == P.row_groups) row_group = 0, ++head;
        if (head == P.heads) {
          head = 0;
          ++b;
          ctx = next_ctx, tokens = next_tokens;
          prefetch();
        }
      }
      if (s.tile1 > s.tile0 && !other) return true;  // else it holds nothing but an item's cost
    }
    return false;
  }
};

// ------------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------------
// Tokens per row group: as few groups as 128 rows allow, of even size.
inline void row_groups(int T, int group, int* tokens, int* groups) {
  const int most = kMaxRows / group;
  *groups = (T + most - 1) / most;
  *tokens = (T + *groups - 1) / *groups;
  *groups = (T + *tokens - 1) / *tokens;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn encode_fn() {
  static std::atomic<void*> cached{nullptr};
  void* f = cached.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    cached.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// A 4-d map with the given extents, byte strides of dimensions 1..3 and box.  The stride of a dimension of
// one element is never used, and is set to a legal one.
inline bool encode(CUtensorMap* map, CUtensorMapDataType type, int es, void* data, const int64_t (&dim)[4],
                   const int64_t (&stride)[3], const int (&box)[4], CUtensorMapSwizzle swizzle) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < 4; ++i) d[i] = (cuuint64_t)dim[i], b[i] = (cuuint32_t)box[i];
  for (int i = 0; i < 3; ++i) s[i] = dim[i + 1] == 1 ? (cuuint64_t)dim[0] * es : (cuuint64_t)stride[i];
  return fn(map, type, 4, data, d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sv
