// spec_weigh.cu — spec_kv_weigh: the attention weight that the new tokens of a step give every entry of the paged cache.
//
// The sum over rows of exp(scale q.K_s - lse) needs each key once and nothing of the other slots, since the rows' sums are
// known.  So it is a stream over the keys, half of what the attention reads, with 2 R flops per byte (bf16) for R rows:
//
//   S^T = K Q^T   [128 slots x R]    tcgen05.mma, K from a TMA-fed ring, the accumulator in TMEM
//   w_s = sum over R of exp2(c S - lse)   one thread per slot: its R columns are its own, no reduction crosses threads
//
// with slots on the matrix unit's 128 rows as in spec_attention.cu, whose line of tiles, cut into equal parts over the
// SMs, this takes too; a cut item needs no join.  More than 128 rows go by in passes over the same tiles, which add to what the
// one before left: a slot's passes are the same thread's.
//
// Measured (requests x tokens, 8 kv heads x 4 of 128, 1000 to 16000 slots; time; of the bytes' 6749 GB/s):
//   64 x 7, E4M3 with page scales   105 us  0.84   memory; a launch's beginning and end are 10 us of it
//   64 x 7, bf16                    179 us  0.95   memory
//   64 x 17 (68 rows), E4M3         139 us  0.64   the sums: 68 columns of 128 slots a tile (page scales: 143)
//   8 x 6, 0 to 4001, bf16           11 us  0.45   the call's host part

#include <type_traits>

#include "tile_stream.cuh"

namespace sv {

struct WeighParams {
  CUtensorMap q_map, k_map;
  Cache cache;
  PageScales scales;
  Record record;
  Batch batch;
  const int64_t* mask;
  const float* lse;
  const int32_t* positions;
  int heads, group;
  int tokens;                // of a pass
  int rows;                  // group * tokens
  int row_groups;            // of the line's items: 1
  int item_cost;             // an item's beginning, in tiles
  int whole;                 // 0: items may be cut
  int wait_tries;            // the limit of every wait
  float scale_log2;          // scale * log2(e)
};

// The waits of this kernel.  A limit of 0, which a test sets, does not let the first try suspend.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const Patience& w) {
  if (w.limit > 0) return mbar_wait(bar, parity, w);
  if (mbar_test(bar, parity)) return true;
  *w.dead = 1;
  return false;
}
__device__ __forceinline__ bool wait_for_warp(uint32_t bar, uint32_t parity, const Patience& w) {
  return __all_sync(~0u, wait_for(bar, parity, w));
}

template <int D, bool F8, int NT>
struct WeighShape {
  static constexpr int kHalves = D / 64;
  static constexpr int kRing = kTileSlots * D * (F8 ? 1 : 2);
  static constexpr int kQ = NT * D * 2;
  static constexpr int kBudget = 232448 - 1024 - 6144;  // 227 KB, alignment, barriers and row states
  static constexpr int kFit = (kBudget - 2 * kQ) / kRing;
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;  // keys' tiles in flight
  static_assert(kSlots >= 3, "the ring holds three tiles at least");
  static constexpr int kGroups = 4;                     // warpgroups that add up, each every kGroups-th tile of an item,
  static constexpr int kColumns = NT * kGroups;         // with a buffer of scores of its own
  static constexpr int kAddWarps = 4 * kGroups;
  static constexpr int kProducer = kAddWarps, kProducers = 2;  // each every other tile
  static constexpr int kIssuer = kProducer + kProducers;
  static constexpr int kPrepare = kIssuer + 1, kPrepareWarps = F8 && NT > 32 ? 4 : 1;
  // 20 warps or 24, the last one idle: more rows take longer to split (64 requests x 17 tokens, 1000 to 4000 slots: 68 us with one
  // warp, 57 with four), fewer leave registers for twice as many scores at a time (64 x 7 tokens: 104 us against 110).
  static constexpr int kThreads = kPrepareWarps == 4 ? 768 : 640;
  static_assert(kThreads % 128 == 0, "whole warpgroups");
  static constexpr int kChunk = kPrepareWarps == 4 || NT < 32 ? 16 : 32;  // scores a thread has in registers

  struct State {
    uint64_t ring_full[12], ring_empty[12];
    uint64_t q_loaded[2], q_full[2], q_empty[2];  // by the pass's parity
    uint64_t rows_full[2], rows_empty[2];
    uint64_t s_full[4], s_empty[4];
    uint64_t products_done;                       // behind a wait that ran out
    uint32_t tmem;
    int dead;
    int copies[kProducers], queries;              // tiles and Qs whose copies were issued, up to the last one
    int start_b, start_offset;
    int warp_sum[kThreads / 32];
    alignas(16) float shift[2][NT];               // -lse in log2 units; -inf: the row has no part
    alignas(16) float mult[2][F8 ? NT : 4];       // E4M3: a score's factor to log2 units
    uint64_t rule[2][SPEC_MAX_NEW];               // which new tokens the pass's tokens attend to
    uint32_t active[2][(NT + 31) / 32];           // rows that have a part
  };
  static constexpr int kState = 2 * kQ + kSlots * kRing;
  static constexpr int kBytes = kState + (int)sizeof(State) + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

template <int D, int KIND, int NT>
__global__ void __launch_bounds__(WeighShape<D, KIND != kBf16, NT>::kThreads, 1) weigh_kernel(const __grid_constant__ WeighParams P) {
  constexpr bool F8 = KIND != kBf16, PAGES = KIND == kE4m3Pages;
  using S = WeighShape<D, F8, NT>;
  extern __shared__ char raw_smem[];
  char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  char* q_buf = smem;                  // [2][halves][NT][128 B]
  char* ring = q_buf + 2 * S::kQ;
  auto* st = reinterpret_cast<typename S::State*>(smem + S::kState);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_next();
  if (threadIdx.x == 0) {
    st->dead = st->queries = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(smem_addr(&st->ring_full[i]), 1);
      mbar_init(smem_addr(&st->ring_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&st->q_loaded[i]), 1);
      mbar_init(smem_addr(&st->q_full[i]), S::kPrepareWarps);
      mbar_init(smem_addr(&st->q_empty[i]), 1);
      mbar_init(smem_addr(&st->rows_full[i]), S::kPrepareWarps);
      mbar_init(smem_addr(&st->rows_empty[i]), S::kAddWarps);
    }
    for (int i = 0; i < S::kGroups; ++i) {
      mbar_init(smem_addr(&st->s_full[i]), 1);
      mbar_init(smem_addr(&st->s_empty[i]), 4);
    }
    mbar_init(smem_addr(&st->products_done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Nothing before this reads or writes what another kernel may, nor takes TMEM that one before it may still need.
  pdl_wait();
  if (warp == S::kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&st->tmem)), "r"(S::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  LinePart part;
  find_part<S::kThreads>(P, st->warp_sum, &st->start_b, &st->start_offset, part);
  const uint32_t tmem = st->tmem;
  const Patience dead = {&st->dead, P.wait_tries};
  Walk<WeighParams> walk(P, part.start_b, part.start_offset, part.first, part.count);
  Segment s;
  // Every role goes through the same passes: of each segment, as many as its tokens need.
  const auto passes_of = [&](const Segment& s) { return (s.tokens + P.tokens - 1) / P.tokens; };
  // The warpgroup that has a tile: the same in every pass, another for another head, as short items have but one.
  const auto owner = [](const Segment& s, int tile) { return (tile + s.head + s.b) & (S::kGroups - 1); };

  if (warp >= S::kProducer && warp < S::kIssuer) {
    // ---- TMA: K of every tile, page by page, by two warps in turn (copies of 8 or 16 slots take one longer than they take
    // the memory: 64 x 7 tokens, E4M3, pages of 16: 155 us with one, 122 with two) ----
    const auto uniform = [](int x) { return __shfl_sync(~0u, x, 0); };
    const int shift = uniform(P.cache.page_shift), page = 1 << shift;
    const int box = min(page, kTileSlots);  // slots of one copy
    const int copies = kTileSlots / box;    // copies of a tile (and half)
    constexpr int kParts = F8 ? 1 : S::kHalves;
    const uint32_t base = uniform(smem_addr(smem)), bars = uniform(smem_addr(st));
    const auto bar_of = [&](const uint64_t* x) { return bars + (uint32_t)(reinterpret_cast<const char*>(x) - reinterpret_cast<const char*>(st)); };
    const int me = uniform(warp - S::kProducer);
    int slot = 0, nth = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int head = uniform(s.head), tile0 = uniform(s.tile0), tile1 = uniform(s.tile1), passes = uniform(passes_of(s));
      const int32_t* table = P.batch.pages + (int64_t)s.b * P.batch.max_pages;
      const auto entry = [&](int tile) {  // the page of this lane's copy of a tile; one past the pool reads as zeros
        const int at = tile * kTileSlots + lane * box;
        if (lane >= copies || at >= s.end) return P.cache.num_pages;
        const int p = __ldg(table + (at >> shift));
        return p < 0 || p > P.cache.num_pages ? P.cache.num_pages : p;
      };
      for (int pass = 0; ok && pass < passes; ++pass) {
        const int mine = tile0 + ((nth ^ me) & 1);
        int next_page = mine < tile1 ? entry(mine) : P.cache.num_pages;
        for (int tile = tile0; tile < tile1; ++tile) {
          const bool other = (nth++ ^ me) & 1;
          const int at_slot = slot;
          const uint32_t at_phase = phase;
          if (++slot == S::kSlots) slot = 0, phase ^= 1;
          if (other) continue;
          const int my_page = next_page;
          if (tile + 2 < tile1) next_page = entry(tile + 2);
          ok = wait_for_warp(bar_of(&st->ring_empty[at_slot]), at_phase ^ 1, dead);
          if (!ok) break;
          const uint32_t bar = bar_of(&st->ring_full[at_slot]);
          if (lane == 0) mbar_expect(bar, S::kRing);
          __syncwarp();
          const uint32_t dst = base + 2 * S::kQ + at_slot * S::kRing;
          const auto bring = [&](auto tag) {
            constexpr int N = decltype(tag)::value;  // copies, of kTileSlots / N slots
            const int row = N == 1 ? (tile * kTileSlots) & (page - 1) : 0;
            int p[N];
#pragma unroll
            for (int c = 0; c < N; ++c) p[c] = __shfl_sync(~0u, my_page, c);
#pragma unroll
            for (int c = 0; c < N; ++c)
#pragma unroll
              for (int part = 0; part < kParts; ++part)
                tma_load(dst + c * (kTileSlots / N) * (F8 ? D : 128) + part * (kTileSlots * 128), &P.k_map, part * 64, row, head, p[c], bar);
          };
          if (copies == 1) bring(std::integral_constant<int, 1>{});
          else if (copies == 2) bring(std::integral_constant<int, 2>{});
          else if (copies == 4) bring(std::integral_constant<int, 4>{});
          else if (copies == 8) bring(std::integral_constant<int, 8>{});
          else bring(std::integral_constant<int, 16>{});
          issued = nth;
        }
      }
    }
    if (lane == 0) st->copies[me] = issued;
  } else if (warp == S::kIssuer) {
    // ---- scores: a tile as soon as it is there and a buffer is free ----
    const auto uniform = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };
    const uint32_t n16 = uniform((P.rows + 15) / 16 * 16);
    const uint32_t idesc = 1u << 4 | (n16 >> 3) << 17 | (128u >> 4) << 24 | (F8 ? 0u : 1u << 7 | 1u << 10);  // fp32, M = 128
    const uint32_t base = uniform(smem_addr(smem)), cols = uniform(tmem), bars = uniform(smem_addr(st));
    const auto bar_of = [&](const uint64_t* x) { return bars + (uint32_t)(reinterpret_cast<const char*>(x) - reinterpret_cast<const char*>(st)); };
    const uint64_t q_desc = matrix_desc(base, 16, 1024);
    const uint64_t k_desc = F8 ? matrix_desc<D>(base + 2 * S::kQ, 16, 8 * D) : matrix_desc(base + 2 * S::kQ, 16, 1024);
    const auto ahead = [](int bytes) { return (uint64_t)(bytes >> 4); };
    int slot = 0, nth = 0;
    uint32_t phase = 0, s_phase = 0;  // s_phase: a bit for each buffer
    bool ok = true;
    while (ok && uniform(walk.next(s))) {
      const int tiles = uniform(s.tile1 - s.tile0), passes = uniform(passes_of(s)), first = uniform(owner(s, s.tile0));
      for (int pass = 0; ok && pass < passes; ++pass, ++nth) {
        const int qb = nth & 1;
        ok = wait_for_warp(bar_of(F8 ? &st->q_full[qb] : &st->q_loaded[qb]), (nth >> 1) & 1, dead);
        for (int tile = 0; ok && tile < tiles; ++tile) {
          const int buffer = (first + tile) & (S::kGroups - 1);
          ok = wait_for_warp(bar_of(&st->ring_full[slot]), phase, dead) &&
               wait_for_warp(bar_of(&st->s_empty[buffer]), ((s_phase >> buffer) & 1) ^ 1, dead);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = k_desc + ahead(slot * S::kRing), b = q_desc + ahead(qb * S::kQ);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            if constexpr (F8) {
              const int part = k / (D / 32), in = (k % (D / 32)) * 32;  // of q: its 4 upper bits, then the others
              tc_mma<true>(cols + buffer * NT, a + ahead(in), b + ahead(part * (D == 128 ? NT * 128 : 64) + in),
                           idesc | (part ? kSecondE5m2 : 0u), k > 0);
            } else {
              const int half = k / 4, in = (k % 4) * 32;
              tc_mma<false>(cols + buffer * NT, a + ahead(half * (kTileSlots * 128) + in), b + ahead(half * (NT * 128) + in), idesc, k > 0);
            }
          }
          tc_commit(bar_of(&st->s_full[buffer]));
          tc_commit(bar_of(&st->ring_empty[slot]));
          if (++slot == S::kSlots) slot = 0, phase ^= 1;
          s_phase ^= 1u << buffer;
        }
        if (ok) tc_commit(bar_of(&st->q_empty[qb]));
      }
    }
    __syncwarp();
  } else if (warp >= S::kPrepare + S::kPrepareWarps) {
    // (so that the block has whole warpgroups)
  } else if (warp >= S::kPrepare) {
    // ---- what each pass knows of its rows, up to two passes ahead: Q (over E4M3 keys split), sums, factors, rules ----
    const auto uniform = [](int x) { return __shfl_sync(~0u, x, 0); };
    const uint32_t base = uniform(smem_addr(smem)), bars = uniform(smem_addr(st));
    const auto bar_of = [&](const uint64_t* x) { return bars + (uint32_t)(reinterpret_cast<const char*>(x) - reinterpret_cast<const char*>(st)); };
    const int tid = threadIdx.x - S::kPrepare * 32, me = uniform(tid / 32);
    constexpr int kCount = S::kPrepareWarps * 32;
    int nth = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int passes = passes_of(s);
      for (int pass = 0; ok && pass < passes; ++pass, ++nth) {
        const int qb = nth & 1, t0 = pass * P.tokens, rows = min(s.tokens - t0, P.tokens) * P.group;
        if (me == 0) {
          ok = wait_for_warp(bar_of(&st->q_empty[qb]), ((nth >> 1) & 1) ^ 1, dead);
          if (!ok) break;
          const uint32_t bar = bar_of(&st->q_loaded[qb]);
          if (lane == 0) mbar_expect(bar, P.rows * D * 2), st->queries = nth + 1;
          __syncwarp();
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            tma_load(base + qb * S::kQ + h * NT * 128, &P.q_map, h * 64, uniform(s.head) * P.group, uniform(t0), uniform(s.b), bar);
        }
        ok = wait_for_warp(smem_addr(&st->rows_empty[qb]), ((nth >> 1) & 1) ^ 1, dead);
        if (!ok) break;
        for (int r0 = me * 32; r0 < NT; r0 += kCount) {
          const int r = r0 + lane;
          float x = -INFINITY;
          if (r < rows) {
            const int t = t0 + r / P.group, g = r % P.group;
            x = -P.lse[(((int64_t)s.b * P.batch.T + t) * P.heads + s.head) * P.group + g] * kLog2e;
            if (fabsf(x) == INFINITY) x = -INFINITY;
          }
          if (r < NT) st->shift[qb][r] = x;
          const uint32_t word = __ballot_sync(~0u, r < rows && !(x == -INFINITY));
          if (lane == 0) st->active[qb][r0 / 32] = word;
        }
        for (int t = tid; t < min(P.tokens, s.tokens - t0); t += kCount)
          st->rule[qb][t] = P.mask ? (uint64_t)__ldg(P.mask + (int64_t)s.b * P.batch.T + t0 + t) : t0 + t >= 63 ? ~0ull : (2ull << (t0 + t)) - 1;
        if constexpr (F8) {
          ok = wait_for_warp(smem_addr(&st->q_loaded[qb]), (nth >> 1) & 1, dead);
          if (!ok) break;
          const float c = P.scale_log2 * (!PAGES && P.cache.k_scale ? __ldg(P.cache.k_scale + s.head) : 1.0f);
          split_queries<D, NT, kCount>(q_buf + qb * S::kQ, tid, (rows + 15) & ~15, c, st->mult[qb]);
          fence_async_shared();
        }
        __syncwarp();
        if (lane == 0) {
          if constexpr (F8) mbar_arrive(smem_addr(&st->q_full[qb]));
          mbar_arrive(smem_addr(&st->rows_full[qb]));
        }
      }
    }
  } else {
    // ---- the sums: a thread per slot, each warpgroup every kGroups-th tile ----
    const int wg = warp >> 2, key = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    constexpr int CK = S::kChunk;
    const float c = P.scale_log2;
    const int page_mask = (1 << P.cache.page_shift) - 1;
    int nth = 0;
    uint32_t parity = 0;  // of this warpgroup's buffer
    bool ok = true;
    while (walk.next(s)) {
      const int passes = passes_of(s);
      const int32_t* table = P.batch.pages + (int64_t)s.b * P.batch.max_pages;
      const auto page_of = [&](int tile) {  // -1: nothing is recorded
        const int at = tile * kTileSlots + key;
        if (tile >= s.tile1 || at >= s.end) return -1;
        const int p = __ldg(table + (at >> P.cache.page_shift));
        return p < 0 || p >= P.cache.num_pages ? -1 : p;
      };
      for (int pass = 0; pass < passes; ++pass, ++nth) {
        const int qb = nth & 1, t0 = pass * P.tokens, rows = min(s.tokens - t0, P.tokens) * P.group;
        ok = ok && wait_for(smem_addr(&st->rows_full[qb]), (nth >> 1) & 1, dead);
        __syncwarp();
        bool plain = true;  // every row has a part
#pragma unroll
        for (int r0 = 0; r0 < NT; r0 += 32)
          if (r0 < rows) plain = plain && st->active[qb][r0 / 32] == (rows - r0 >= 32 ? ~0u : (1u << (rows - r0)) - 1);
        plain = __all_sync(~0u, plain);
        // what a slot has and its page's scale come a tile (of this warpgroup) ahead, its page two
        const int mine = s.tile0 + ((wg - owner(s, s.tile0)) & (S::kGroups - 1));
        int page = page_of(mine), next_page = page_of(mine + S::kGroups);
        float* place = nullptr;
        float had = 0.0f, scale = 1.0f;
        const auto look = [&](int tile) {
          place = nullptr, had = 0.0f, scale = 1.0f;
          if (page < 0) return;
          const int slot = tile * kTileSlots + key;
          const int64_t at = (int64_t)page * P.heads + s.head;
          place = P.record.weight + (at << P.cache.page_shift) + (slot & page_mask);
          if (slot < s.ctx || pass > 0) had = *place;
          if constexpr (PAGES) scale = P.scales.k[at];
        };
        look(mine);
        for (int tile = mine; tile < s.tile1; tile += S::kGroups) {
          const int slot = tile * kTileSlots + key;
          float* const to = place;
          const float before = had, factor = PAGES && !scale_counts(scale) ? NAN : scale;
          const int at_page = page;
          page = next_page;
          look(tile + S::kGroups);
          next_page = page_of(tile + 2 * S::kGroups);

          ok = ok && wait_for(smem_addr(&st->s_full[wg]), parity, dead);
          parity ^= 1;
          __syncwarp();
          tc_fence_after();
          float2 sum = make_float2(0.0f, 0.0f);
          // columns four at a time, so that those past the rows cost nothing
          const auto add = [&](int c0, auto tag) {
            constexpr bool CHECKED = decltype(tag)::value;
            float z[CK];
            uint32_t see = ~0u;  // columns, from c0 on, that have a part in this slot
            if constexpr (CHECKED) {
              see = st->active[qb][c0 / 32] >> (c0 & 31);
              const int fresh = slot - s.ctx;
              if (fresh >= 0 && fresh < 64)
                for (int t = c0 / P.group; t * P.group < min(rows, c0 + CK); ++t)
                  if (!((st->rule[qb][t] >> fresh) & 1)) {
                    const int from = max(t * P.group - c0, 0), to = min((t + 1) * P.group - c0, CK);
                    see &= ~((to == 32 ? ~0u : (1u << to) - 1) & (~0u << from));
                  }
              __syncwarp();
            }
            if constexpr (CK == 32) {
              tm_load<16>(lanes + wg * NT + c0, reinterpret_cast<float(&)[16]>(z[0]));
              tm_load<16>(lanes + wg * NT + c0 + 16, reinterpret_cast<float(&)[16]>(z[CK - 16]));
            } else {
              tm_load<CK>(lanes + wg * NT + c0, z);
            }
            if (c0 + CK >= rows) {  // the last scores are in registers: the buffer is the next tile's
              tc_fence_before();
              if (lane == 0) mbar_arrive(smem_addr(&st->s_empty[wg]));
            }
#pragma unroll
            for (int i = 0; i < CK; i += 4) {
              if (c0 + i >= rows) break;
              const float4 m = *reinterpret_cast<const float4*>(&st->shift[qb][c0 + i]);
              const float4 f = F8 ? *reinterpret_cast<const float4*>(&st->mult[qb][c0 + i]) : make_float4(c, c, c, c);
              float2 z0 = make_float2(z[i], z[i + 1]), z1 = make_float2(z[i + 2], z[i + 3]);
              if constexpr (PAGES) z0 = mul2(z0, make_float2(factor, factor)), z1 = mul2(z1, make_float2(factor, factor));
              const float2 a = fma2(z0, make_float2(f.x, f.y), make_float2(m.x, m.y));
              const float2 b = fma2(z1, make_float2(f.z, f.w), make_float2(m.z, m.w));
              float2 w0 = make_float2(exp2_approx(a.x), exp2_approx(a.y)), w1 = make_float2(exp2_approx(b.x), exp2_approx(b.y));
              if (!CHECKED && c0 + i + 4 > rows) {  // columns past the rows may hold anything
                w0.y = c0 + i + 1 < rows ? w0.y : 0.0f, w1.x = c0 + i + 2 < rows ? w1.x : 0.0f, w1.y = 0.0f;
              }
              if constexpr (CHECKED) {  // so may rows without a part
                w0.x = (see >> i) & 1 ? w0.x : 0.0f, w0.y = (see >> (i + 1)) & 1 ? w0.y : 0.0f;
                w1.x = (see >> (i + 2)) & 1 ? w1.x : 0.0f, w1.y = (see >> (i + 3)) & 1 ? w1.y : 0.0f;
              }
              sum = add2(sum, add2(w0, w1));
            }
          };
          const bool checked = !plain || (tile + 1) * kTileSlots > s.ctx;
          if (checked)
            for (int c0 = 0; c0 < rows; c0 += CK) add(c0, std::true_type{});
          else
            for (int c0 = 0; c0 < rows; c0 += CK) add(c0, std::false_type{});
          if (to) {
            *to = ok ? before + (sum.x + sum.y) : NAN;
            if (pass == 0 && slot >= s.ctx && P.record.position) {
              const int64_t at = (((int64_t)at_page * P.heads + s.head) << P.cache.page_shift) + (slot & page_mask);
              P.record.position[at] = P.positions ? __ldg(P.positions + (int64_t)s.b * P.batch.T + slot - s.ctx) : slot;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&st->rows_empty[qb]));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  const bool lost = *dead.dead != 0;  // a wait ran out: products and copies may be in flight that nobody saw end
  if (warp == S::kIssuer) {
    tc_fence_after();
    if (lost) {
      tc_commit(smem_addr(&st->products_done));  // arrives behind every product of this warp
      mbar_drain(smem_addr(&st->products_done), 0);
      __syncwarp();
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kColumns));
  }
  if (lost && warp == S::kProducer) {
    // a slot is filled again only when its last filling was used: the last copy of each is the one that may be in flight
    const int copies = max(st->copies[0], st->copies[1]);
    for (int i = max(copies - S::kSlots - 1, 0); i < copies; ++i)
      if (i < st->copies[i & 1]) mbar_drain(smem_addr(&st->ring_full[i % S::kSlots]), (i / S::kSlots) & 1);
    for (int i = max(st->queries - 2, 0); i < st->queries; ++i) mbar_drain(smem_addr(&st->q_loaded[i & 1]), (i >> 1) & 1);
  }
}

// ------------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------------
template <int D, int KIND, int NT>
static cudaError_t launch_weigh(const WeighParams& P, int dev, int ctas, cudaStream_t st) {
  using S = WeighShape<D, KIND != kBf16, NT>;
  auto kern = weigh_kernel<D, KIND, NT>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel's shared memory is set
  if (!((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return launch_early(kern, dim3(ctas), dim3(S::kThreads), S::kBytes, st, P);
}

template <int D, int KIND>
static cudaError_t launch_weigh_rows(const WeighParams& P, int dev, int ctas, cudaStream_t st) {
  if (P.rows <= 16) return launch_weigh<D, KIND, 16>(P, dev, ctas, st);
  if (P.rows <= 32) return launch_weigh<D, KIND, 32>(P, dev, ctas, st);
  if (P.rows <= 64) return launch_weigh<D, KIND, 64>(P, dev, ctas, st);
  return launch_weigh<D, KIND, 128>(P, dev, ctas, st);
}

}  // namespace sv

using namespace sv;

extern "C" spec_status_t spec_kv_weigh(const spec_heads_t* q, int32_t q_heads, const spec_kv_cache_t* given,
                                       const spec_kv_page_scales_t* scales, const spec_decode_batch_t* batch, const int64_t* mask,
                                       float scale, const float* lse, const spec_kv_record_t* record, const int32_t* positions,
                                       void* stream) {
  if (!given) return SPEC_ERR_INVALID_ARG;
  spec_kv_cache_t keys = *given;  // the values are not used
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
  if (!heads_ok(q) || !lse || ((uintptr_t)lse & 3u)) return SPEC_ERR_INVALID_ARG;

  WeighParams P = {};
  P.cache = cache_of(cache), P.scales = scales_of(scales), P.record = record_of(record), P.batch = batch_of(batch, cache);
  P.mask = mask, P.lse = lse, P.positions = positions;
  const int D = cache->head_dim;
  P.heads = cache->heads, P.group = q_heads / cache->heads;
  int passes;
  row_groups(batch->T, P.group, &P.tokens, &passes);
  P.rows = P.group * P.tokens;
  P.row_groups = 1;
  P.scale_log2 = scale * kLog2e;
  // an item's beginning and its tile with new tokens (64 x 7 tokens, E4M3: 113 us at 1 tile, 110 at 2, 107 at 4, 106 at 6; 16 x 7:
  // 37, 36, 34, 34; 64 x 7, bf16, whose tiles take twice as long: 177, 178, 178, 180)
  P.item_cost = cache->dtype == SPEC_DTYPE_E4M3 ? 4 : 1;
  P.wait_tries = g_test_hooks.load(std::memory_order_relaxed) & 2 ? 0 : kWaitTries;
  const int64_t per = ((int64_t)P.batch.slots + kTileSlots - 1) / kTileSlots;
  const int64_t most = (int64_t)batch->B * cache->heads * ((per > 0 ? per : 1) + P.item_cost);
  if (most > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;

  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  const int box = cache->page_size < kTileSlots ? cache->page_size : kTileSlots;
  const Heads hq = heads_of(q);
  bool ok = encode(&P.q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, hq.data, {D, q_heads, batch->T, batch->B},
                   {hq.head, hq.token, hq.row}, {64, P.group, P.tokens, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
  ok = ok && encode(&P.k_map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f8 ? 1 : 2, P.cache.k,
                    {D, cache->page_size, cache->heads, cache->num_pages}, {P.cache.slot, P.cache.head, P.cache.page},
                    {f8 ? D : 64, box, 1, 1}, f8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return SPEC_ERR_CUDA;
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  const int ctas = most < sms ? (int)most : sms;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kind = scales ? kE4m3Pages : f8 ? kE4m3 : kBf16;
  const cudaError_t e = D == 128 ? (kind == kBf16 ? launch_weigh_rows<128, kBf16>(P, dev, ctas, st)
                                    : kind == kE4m3 ? launch_weigh_rows<128, kE4m3>(P, dev, ctas, st)
                                                    : launch_weigh_rows<128, kE4m3Pages>(P, dev, ctas, st))
                                 : (kind == kBf16 ? launch_weigh_rows<64, kBf16>(P, dev, ctas, st)
                                    : kind == kE4m3 ? launch_weigh_rows<64, kE4m3>(P, dev, ctas, st)
                                                    : launch_weigh_rows<64, kE4m3Pages>(P, dev, ctas, st));
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
