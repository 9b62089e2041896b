// spec_attention.cu — spec_paged_attention: the new tokens of a step attend over the paged cache.
//
// A request's new tokens and the q heads of a group share every key and value they read: their
// R = group * tokens rows are one small matrix against a long cache, so the work is a stream over the
// cache with 2 R flops per byte (bf16), memory bound up to R ~ 280 on this part.  Per kv head:
//
//   S^T = K Q^T   [128 slots x R]    tcgen05.mma, K from a TMA-fed ring, the accumulator in TMEM
//   P^T = exp2(c S^T - m)            one thread per slot, R columns in registers; fp32
//   O^T += V^T P^T [head_dim x R]    tcgen05.mma, V and P^T read with their slots as the reduction
//
// Slots lie on the 128 rows of the matrix unit and query rows on its free N side, so few rows cost little
// and nothing is padded to 128 query rows.  The maximum m of a row is taken over a tile only when
// some weight passes 2^8 (a vote per tile; the first tile always): rescaling is exact whatever m is, and
// this keeps the cross-thread reductions out of the stream.
//
// The tiles of all requests and heads form one line, cut into equal parts over the SMs (no part of the
// plan needs the host to know a length).  An item (request, kv head, row group) that a cut splits
// leaves its parts' (m, l, O) in the workspace, and a second kernel joins them.
//
// Within a CTA (one per SM) warps have roles that meet at mbarriers: one brings Q and K, one V (TMA, a
// ring of 2 to 4 tiles of each), one issues the products, two or four warpgroups are the softmax, and with
// an E4M3 cache four warps split Q and bring V to fp16.
//
// Measured (requests x tokens, kv heads x group, slots; time; of the copy bandwidth of 6772 GB/s):
//   64 x 7, 8 x 4, 1000 to 16000, bf16   330 us  6.8 TB/s  1.00   bound by memory
//   2 x 5, 4 x 8, 100003 to 131071, bf16  83 us  5.7 TB/s  0.84   memory, and 10 us to begin and join
//   64 x 7, 8 x 4, 1000 to 16000, E4M3 with page scales  219 us  5.1 TB/s  0.76   the softmax (a scale per head: 202 us)
//   32 x 17 (a tree), 8 x 4, 500 to 9000, E4M3  120 us  2.7 TB/s  0.39   the softmax: 68 rows at 128 slots a step
//   8 x 6, 8 x 4, 0 to 4001, bf16         21 us  3.1 TB/s  0.46   beginnings and ends of 64 items

#include <type_traits>

#include "tile_stream.cuh"

namespace sv {

// Where the page table could hold no item of more tiles, none is cut, which saves the join (the host knows the table's
// width, not the lengths, so short requests under a wide table are cut; 4 requests x 8 kv heads, 20 rows: 9.0 us against
// 11.8 at 300 slots, 10.5 against 12.0 at 600, 12.5 against 12.6 at 1000; one request x 2 heads: 7.2 / 8.6, 8.5 / 8.5, 10.3 / 9.1).
constexpr int kWholeTiles = 6;
constexpr int kMaxParts = 160;        // CTAs of the stream at most (one per SM), for the workspace's size
constexpr float kRescale = 8.0f;      // rescale when a score passes the maximum in use by 2^8
constexpr float kNone = 3e38f;        // shift of a row without a maximum yet: any score asks for one
constexpr int kConvertWarps = 4;      // E4M3 caches: E4M3 -> fp16
constexpr float kLn2 = 0.6931471805599453f;
// fp16 weights are lifted to a largest of 2^7 (2^15 before a rescale), so they reach down to 2^-31 of it
constexpr float kLift16 = 7.0f;

struct AttnParams {
  CUtensorMap q_map, k_map, v_map;
  Heads out;
  Cache cache;                 // for the rare reads of single entries, and the scales
  PageScales scales;
  Batch batch;
  const int64_t* mask;
  int heads, group;
  int tokens, row_groups;      // tokens per row group
  int rows;                    // group * tokens
  int item_cost;               // an item's beginning and end, in tiles
  int whole;                   // items are not cut: the CTA that one begins in takes all of it
  int wait_tries;              // the limit of every wait
  float scale_log2;            // scale * log2(e)
  float* lse;                  // [B, T, q heads] or null
  float* part;                 // [CTA][2][rows][D] unnormalised O
  float2* part_ml;             // [CTA][2][rows] (m in log2 units, l)
  float* part_raw;             // [CTA][2][rows] bf16 with lse: the sum of the weights before their rounding
  int4* cut;                   // [CTA] (b, head * row_groups + row group, item's end, total) on the line of an
                               //       item that begins in this CTA and ends in a later one; b = -1: none
};

// A row's log of its sum of exponentials: `sum` is of weights 2^(score - top + lift), scores in log2 units.
__device__ __forceinline__ float row_lse(float top, float lift, float sum) {
  return sum == 0.0f ? -INFINITY : (top - lift + log2f(sum)) * kLn2;
}
__device__ __forceinline__ int64_t lse_place(int b, int T, int t, int heads, int head, int group, int g) {
  return (((int64_t)b * T + t) * heads + head) * group + g;
}

// ------------------------------------------------------------------------------------------------
// shared memory
// ------------------------------------------------------------------------------------------------
template <int D, int KIND, int NT>
struct Shape {
  static constexpr bool F8 = holds_e4m3(KIND);
  static constexpr int kHalves = D / 64;                          // 128-byte columns of a 16-bit row
  static constexpr int kTile16 = kTileSlots * D * 2;              // a K or V tile in 16 bits
  static constexpr int kRing = kTileSlots * D * (F8 ? 1 : 2);     // a ring slot: a tile as the cache holds it
  static constexpr int kQ = NT * D * 2;                           // a Q buffer
  static constexpr int kQBufs = NT > 64 ? 1 : 2;                  // two, where the ring stays deep enough
  static constexpr int kP = kTileSlots * 128 * (NT > 64 ? 2 : 1); // P^T, 128 bytes a slot and 64 rows
  static constexpr int kFixed = kQBufs * kQ + kP + (F8 ? 2 * kTile16 : 0);
  static constexpr int kBudget = 232448 - 1024 - 6144;            // 227 KB, alignment, barriers and row states
  static constexpr int kFit = (kBudget - kFixed) / kRing;
  static constexpr int kSlots = kFit > 8 ? 8 : F8 ? kFit / 2 * 2 : kFit;  // K and V tiles in flight (E4M3: V in odd slots)
  static_assert(kSlots >= 4, "the ring holds two tiles of K and V at least");
  // Softmax warpgroups, each with every kGroups-th chunk of columns: a tile is a chain of short steps, and
  // warps are what hides their latencies (64 rows, E4M3: 93 us with 4 warpgroups, 112 with 2; 32 rows: the same).
  static constexpr int kGroups = NT >= 64 ? 4 : 2;
  static constexpr int kSoftmaxWarps = 4 * kGroups;
  static constexpr int kProducer = kSoftmaxWarps, kIssuer = kSoftmaxWarps + 1;  // the producer of K and Q,
  static constexpr int kProducerV = kIssuer + 1 + (F8 ? kConvertWarps : 0);     // and that of V
  static constexpr int kThreads = kSoftmaxWarps * 32 + (F8 ? 256 : 128);
  // Registers: the softmax warps take more than an even split of the SM's gives them, the others less.  Per
  // warpgroup of 128 threads: 4 x 128 = 512 = 2 x 176 + 2 x 80 and 6 x 80 = 480 = 4 x 88 + 2 x 64 with E4M3;
  // 5 x 96 = 480 = 4 x 104 + 64 with bf16.
  static constexpr bool kSplit = kGroups == 4 || (F8 && NT > 16);
  static constexpr int kLaunchRegs = kGroups == 4 ? (F8 ? 80 : 96) : F8 ? 128 : 168;
  static constexpr int kMoreRegs = kGroups == 4 ? (F8 ? 88 : 104) : 176, kFewRegs = kGroups == 4 ? 64 : 80;
  static_assert(!kSplit || kGroups * kMoreRegs + (kThreads / 128 - kGroups) * kFewRegs <= kThreads / 128 * kLaunchRegs,
                "register split");
  static constexpr int kColumns = 3 * NT <= 64 ? 64 : 3 * NT <= 128 ? 128 : 3 * NT <= 256 ? 256 : 512;
  static constexpr int kChunk = NT == 32 || NT == 128 ? 16 : 8;  // columns a warpgroup takes at a time
  static constexpr int kOwn = NT / kGroups;                      // columns of one warpgroup
  static constexpr int kChunks = kOwn / kChunk;
  static_assert(kOwn <= 32, "a warpgroup's columns fit a word");
  // A tile's weights stay in registers over the vote on them; with many columns, which would spill, the vote
  // is on scores that are then computed again (68 rows: 118 us against 125 in E4M3, 114 against 117 in bf16).
  static constexpr bool kHold = NT <= 64;
  static constexpr int kScales = kProducerV + 1;  // of page scales, which other caches leave idle
  static constexpr int kAheadScales = KIND == kE4m3Pages ? 8 : 1, kPageScales = KIND == kE4m3Pages ? kTileSlots / 8 : 1;
  static_assert(KIND != kE4m3Pages || kScales < kThreads / 32, "a warp for the scales");

  struct State {
    uint64_t ring_full[8], ring_empty[8];
    uint64_t q_loaded[2], q_full[2], q_empty[2], mult_full[2];
    uint64_t v16_full[2], v16_empty[2];
    uint64_t s_full[2], s_empty[2], p_full, o_full;
    uint64_t scales_full[kAheadScales], scales_empty[kAheadScales];
    uint64_t products_done;          // behind a wait that ran out
    uint32_t tmem;
    int dead;
    int copies[2], queries;          // tiles of K and V, and Qs, whose copies were issued
    int start_b, start_offset, total;
    uint32_t bad_value[4];           // segment + 1 whose new tokens hold a value that is not finite, by segment % 4
    int warp_sum[24];
    alignas(16) float shift[NT];     // what is added to a score: minus the row's maximum in use (see kNone, kLift)
    alignas(16) float top[NT];       // the maximum in use, -inf for none
    alignas(16) float factor[NT];    // a rescale's factor; 1 / l at the end
    float red[4][NT];
    alignas(16) float mult[2][NT];   // E4M3: a score's factor to log2 units, by the segment's parity
    alignas(16) int64_t place[NT];   // the row's offset in the item's output
    // Page scales: of every page of a tile, (a key's, the logarithm of a value's, its inverse)
    alignas(16) float4 scales[kAheadScales][kPageScales];
    uint32_t seen[kGroups][SPEC_MAX_NEW];  // which columns of each warpgroup attend to a new token
  };
  static constexpr int kState = kFixed + kSlots * kRing;
  static constexpr int kBytes = kState + (int)sizeof(State) + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

// Over the 32 lanes, `op` of every one of N values: lane l ends with that of value l % N.
template <int N, typename Op>
__device__ __forceinline__ float fold_lanes(float (&x)[N], int lane, Op op) {
#pragma unroll
  for (int w = N / 2; w > 0; w /= 2) {
    const bool up = lane & w;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float keep = up ? x[k + w] : x[k], send = up ? x[k] : x[k + w];
      x[k] = op(keep, __shfl_xor_sync(~0u, send, w));
    }
  }
  float r = x[0];
#pragma unroll
  for (int w = N; w < 32; w *= 2) r = op(r, __shfl_xor_sync(~0u, r, w));
  return r;
}

// ------------------------------------------------------------------------------------------------
// the stream over the cache
// ------------------------------------------------------------------------------------------------
template <int D, int KIND, int NT>
__global__ void __launch_bounds__(Shape<D, KIND, NT>::kThreads, 1) attn_kernel(const __grid_constant__ AttnParams P) {
  constexpr bool F8 = holds_e4m3(KIND), PAGES = KIND == kE4m3Pages, LSE = KIND == kBf16Lse;
  using S = Shape<D, KIND, NT>;
  extern __shared__ char raw_smem[];
  char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  char* q_buf = smem;                                     // [kQBufs][halves][NT][128 B]
  char* p_buf = q_buf + S::kQBufs * S::kQ;                     // [NT > 64 ? 2 : 1][128][128 B]
  char* v16 = p_buf + S::kP;                              // E4M3: V in fp16, [2][halves][128][128 B]
  char* ring = v16 + (F8 ? 2 * S::kTile16 : 0);
  auto* st = reinterpret_cast<typename S::State*>(smem + S::kState);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kSoftmaxWarps = S::kSoftmaxWarps, kProducer = S::kProducer, kIssuer = S::kIssuer;

  pdl_launch_next();

  if (threadIdx.x == 0) {
    st->dead = 0;
    for (int i = 0; i < 4; ++i) st->bad_value[i] = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(smem_addr(&st->ring_full[i]), 1);
      mbar_init(smem_addr(&st->ring_empty[i]), F8 && i % 2 ? kConvertWarps : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&st->q_loaded[i]), 1);
      mbar_init(smem_addr(&st->q_full[i]), kConvertWarps);
      mbar_init(smem_addr(&st->mult_full[i]), kConvertWarps);
      mbar_init(smem_addr(&st->q_empty[i]), 1);
      mbar_init(smem_addr(&st->s_full[i]), 1);
      mbar_init(smem_addr(&st->s_empty[i]), kSoftmaxWarps);
      mbar_init(smem_addr(&st->v16_full[i]), kConvertWarps);
      mbar_init(smem_addr(&st->v16_empty[i]), 1);
    }
    mbar_init(smem_addr(&st->p_full), kSoftmaxWarps);
    mbar_init(smem_addr(&st->o_full), 1);
    for (int i = 0; i < S::kAheadScales; ++i) {
      mbar_init(smem_addr(&st->scales_full[i]), 1);
      mbar_init(smem_addr(&st->scales_empty[i]), kSoftmaxWarps);
    }
    mbar_init(smem_addr(&st->products_done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Nothing before this reads or writes what another kernel may, nor takes TMEM that one before it may still need.
  pdl_wait();
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&st->tmem)),
                 "r"(S::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  LinePart part;
  find_part<S::kThreads>(P, st->warp_sum, &st->start_b, &st->start_offset, part);
  const int first = part.first, count = part.count, total = part.total, start_b = part.start_b, start_offset = part.start_offset;
  const uint32_t tmem = st->tmem;
  const Patience dead = {&st->dead, P.wait_tries};

  if (warp >= kSoftmaxWarps) {
    if constexpr (S::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kFewRegs));
    Walk<AttnParams> walk(P, start_b, start_offset, first, count);
    Segment s;
    if (warp == kProducer || warp == S::kProducerV) {
      // ---- TMA: one warp brings Q of every segment and K of every tile, another V, page by page ----
      const auto uniform = [](int x) { return __shfl_sync(~0u, x, 0); };
      const bool is_v = uniform(warp == S::kProducerV);
      const CUtensorMap* map = is_v ? &P.v_map : &P.k_map;
      const int shift = uniform(P.cache.page_shift), page = 1 << shift;
      const int box = min(page, kTileSlots);  // slots of one copy
      const int copies = kTileSlots / box;    // copies of a tile (and half)
      constexpr int kParts = F8 ? 1 : S::kHalves;
      const uint32_t base = uniform(smem_addr(smem)), bars = uniform(smem_addr(st));
      const auto bar_of = [&](const uint64_t* x) { return bars + (uint32_t)(reinterpret_cast<const char*>(x) - reinterpret_cast<const char*>(st)); };
      int slot = is_v;
      uint32_t phase = 0;  // of the ring
      bool ok = true;
      int issued = 0, queries = 0;
      for (int seg = 0; ok && walk.next(s); ++seg) {
        const int head = uniform(s.head), tile0 = uniform(s.tile0), tile1 = uniform(s.tile1);
        if (!is_v) {
          const int qb = seg % S::kQBufs;
          ok = mbar_wait_warp(bar_of(&st->q_empty[qb]), ((seg / S::kQBufs) & 1) ^ 1, dead);
          if (!ok) break;
          const uint32_t bar = bar_of(&st->q_loaded[qb]);
          if (lane == 0) mbar_expect(bar, P.rows * D * 2);
          __syncwarp();
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            tma_load(base + (uint32_t)(q_buf - smem) + qb * S::kQ + h * NT * 128, &P.q_map, h * 64, head * P.group,
                     uniform(s.row_group) * P.tokens, uniform(s.b), bar);
          ++queries;
        }
        const int32_t* table = P.batch.pages + (int64_t)s.b * P.batch.max_pages;
        const auto entry = [&](int tile) {  // the page of this lane's copy of a tile; one past the pool reads as zeros
          const int at = tile * kTileSlots + lane * box;
          if (lane >= copies || at >= s.end) return P.cache.num_pages;
          const int p = __ldg(table + (at >> shift));
          return p < 0 || p > P.cache.num_pages ? P.cache.num_pages : p;
        };
        int next_page = entry(tile0);
        for (int tile = tile0; tile < tile1; ++tile) {
          const int my_page = next_page;
          if (tile + 1 < tile1) next_page = entry(tile + 1);
          ok = mbar_wait_warp(bar_of(&st->ring_empty[slot]), phase ^ 1, dead);
          if (!ok) break;
          const uint32_t bar = bar_of(&st->ring_full[slot]);
          if (lane == 0) mbar_expect(bar, S::kRing);
          __syncwarp();
          const uint32_t dst = base + (uint32_t)(ring - smem) + slot * S::kRing;
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
                tma_load(dst + c * (kTileSlots / N) * (F8 ? D : 128) + part * (kTileSlots * 128), map, part * 64, row, head, p[c], bar);
          };
          if (copies == 1) bring(std::integral_constant<int, 1>{});
          else if (copies == 2) bring(std::integral_constant<int, 2>{});
          else if (copies == 4) bring(std::integral_constant<int, 4>{});
          else if (copies == 8) bring(std::integral_constant<int, 8>{});
          else bring(std::integral_constant<int, 16>{});
          ++issued;
          slot += 2;
          if (slot >= S::kSlots) slot -= S::kSlots, phase ^= 1;
        }
      }
      if (lane == 0) {
        st->copies[is_v] = issued;
        if (!is_v) st->queries = queries;
      }
    } else if (PAGES && warp == S::kScales) {
      // ---- page scales of every tile, by a warp of their own: K's producer would bring 64 KB an SM later for them (64 x 7
      // tokens, pages of 32: 236 us) ----
      const int shift = P.cache.page_shift, box = min(1 << shift, kTileSlots), pages = kTileSlots / box;
      int it = 0;
      bool ok = true;
      while (ok && walk.next(s)) {
        const int32_t* table = P.batch.pages + (int64_t)s.b * P.batch.max_pages;
        // a round of as many tiles as the warp has lanes for their pages (8 at most), scales a round ahead and pages two
        const int round = min(32 / pages, 8), mine = lane / pages;
        const auto page_of = [&](int first) {
          const int tile = first + mine, at = tile * kTileSlots + lane % pages * box;
          const int p = mine < round && tile < s.tile1 && at < s.end ? __ldg(table + (at >> shift)) : -1;
          return p < P.cache.num_pages ? p : -1;
        };
        const auto scales_of = [&](int page) {  // of a page outside the pool, which reads as zeros, 1
          const int64_t at = (int64_t)page * P.heads + s.head;
          return page >= 0 ? make_float2(P.scales.k[at], P.scales.v[at]) : make_float2(1.0f, 1.0f);
        };
        int far_page = page_of(s.tile0 + round);
        float2 next = scales_of(page_of(s.tile0));
        for (int first = s.tile0; ok && first < s.tile1; first += round) {
          const float2 x = next;
          next = scales_of(far_page);
          far_page = page_of(first + 2 * round);
          const bool counts = scale_counts(x.y);  // one that does not makes the slots' scores NaN
          const float4 told = make_float4(scale_counts(x.x) ? x.x : NAN, counts ? log2f(x.y) : NAN, counts ? 1.0f / x.y : 1.0f, 0.0f);
          for (int i = 0; i < min(round, s.tile1 - first); ++i, ++it) {
            const int at = it & (S::kAheadScales - 1);
            ok = mbar_wait_warp(smem_addr(&st->scales_empty[at]), ((it / S::kAheadScales) & 1) ^ 1, dead);
            if (!ok) break;
            if (mine == i) st->scales[at][lane % pages % S::kPageScales] = told;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&st->scales_full[at]));
          }
        }
      }
    } else if (warp == kIssuer) {
      // ---- matrix products: weighted values of a tile or scores of the next, as either is ready ----
      const auto uniform = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };
      const auto ready = [](uint32_t bar, uint32_t parity) { return __all_sync(~0u, mbar_test(bar, parity)); };
      const uint32_t n16 = uniform((P.rows + 15) / 16 * 16);
      const uint32_t shape = 1u << 4 | (n16 >> 3) << 17 | (128u >> 4) << 24;  // fp32 accumulators, M = 128
      const uint32_t s_idesc = shape | (F8 ? 0u : 1u << 7 | 1u << 10);        // E4M3 or bf16 operands
      // fp16 or bf16 operands, both with the reduction outside
      const uint32_t o_idesc = shape | (F8 ? 0u : 1u << 7 | 1u << 10) | 1u << 15 | 1u << 16;
      const uint32_t base = uniform(smem_addr(smem)), cols = uniform(tmem), bars = uniform(smem_addr(st));
      const auto bar_of = [&](const uint64_t* x) { return bars + (uint32_t)(reinterpret_cast<const char*>(x) - reinterpret_cast<const char*>(st)); };
      const uint32_t ring_at = base + (uint32_t)(ring - smem), v16_at = base + (uint32_t)(v16 - smem);
      const uint64_t q_desc = matrix_desc(base + (uint32_t)(q_buf - smem), 16, 1024);
      const uint64_t k_desc = F8 ? matrix_desc<D>(ring_at, 16, 8 * D) : matrix_desc(ring_at, 16, 1024);
      // head_dim 64: the instruction's rows 64..127 repeat rows 0..63 and are not read
      const uint64_t v_desc = matrix_desc(F8 ? v16_at : ring_at, D == 128 ? kTileSlots * 128 : 0, 1024);
      const uint64_t p_desc = matrix_desc(base + (uint32_t)(p_buf - smem), kTileSlots * 128, 1024);
      const auto ahead = [](int bytes) { return (uint64_t)(bytes >> 4); };  // of a descriptor's address
      uint32_t s_it = 0, v_it = 0;  // tiles whose scores, and whose values, are issued
      int k_slot = 0, v_slot = 1;
      uint32_t k_phase = 0, v_phase = 0, first_bits = 0;
      const auto advance = [&](int& slot, uint32_t& phase) {
        slot += 2;
        if (slot >= S::kSlots) slot -= S::kSlots, phase ^= 1;
      };
      int seg = 0, idle = 0;
      bool more = uniform(walk.next(s));
      int tile0 = uniform(s.tile0), tile1 = uniform(s.tile1), tile = tile0;
      while (more || v_it < s_it) {
        bool moved = false;
        if (v_it < s_it && ready(bar_of(&st->p_full), v_it & 1) &&
            (F8 ? ready(bar_of(&st->v16_full[v_it & 1]), (v_it >> 1) & 1) : ready(bar_of(&st->ring_full[v_slot]), v_phase))) {
          tc_fence_after();
          const uint32_t add = ((first_bits >> (v_it & 1)) & 1) ^ 1;
          const uint64_t a = v_desc + ahead(F8 ? (int)(v_it & 1) * S::kTile16 : v_slot * S::kRing);
#pragma unroll
          for (int k = 0; k < kTileSlots / 16; ++k)
            tc_mma<false>(cols + 2 * NT, a + ahead(k * 2048), p_desc + ahead(k * 2048), o_idesc, k > 0 ? 1u : add);
          tc_commit(bar_of(&st->o_full));
          tc_commit(bar_of(F8 ? &st->v16_empty[v_it & 1] : &st->ring_empty[v_slot]));
          advance(v_slot, v_phase);
          ++v_it;
          moved = true;
        }
        if (more && s_it - v_it < 2) {
          const int qb = seg % S::kQBufs, sb = s_it & 1;
          if (ready(bar_of(&st->ring_full[k_slot]), k_phase) &&
              (tile != tile0 || ready(bar_of(F8 ? &st->q_full[qb] : &st->q_loaded[qb]), (seg / S::kQBufs) & 1)) &&
              ready(bar_of(&st->s_empty[sb]), ((s_it >> 1) & 1) ^ 1)) {
            tc_fence_after();
            const uint64_t a = k_desc + ahead(k_slot * S::kRing), b = q_desc + ahead(qb * S::kQ);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              if constexpr (F8) {
                // q = (its 4 upper bits, E4M3) + (the others, E5M2): see split_queries
                const int part = k / (D / 32), in = (k % (D / 32)) * 32;
                tc_mma<true>(cols + sb * NT, a + ahead(in), b + ahead(part * (D == 128 ? NT * 128 : 64) + in),
                             s_idesc | (part ? kSecondE5m2 : 0u), k > 0);
              } else {
                const int half = k / 4, in = (k % 4) * 32;
                tc_mma<false>(cols + sb * NT, a + ahead(half * (kTileSlots * 128) + in), b + ahead(half * (NT * 128) + in),
                              s_idesc, k > 0);
              }
            }
            tc_commit(bar_of(&st->s_full[sb]));
            tc_commit(bar_of(&st->ring_empty[k_slot]));
            advance(k_slot, k_phase);
            first_bits = (first_bits & ~(1u << sb)) | (uint32_t)(tile == tile0) << sb;
            ++s_it;
            if (++tile == tile1) {
              tc_commit(bar_of(&st->q_empty[qb]));
              ++seg;
              more = uniform(walk.next(s));
              tile0 = uniform(s.tile0), tile1 = uniform(s.tile1), tile = tile0;
            }
            moved = true;
          }
        }
        if (moved) {
          idle = 0;
        } else if (++idle > 4 * P.wait_tries || ((idle & 255) == 0 && uniform(*dead.dead))) {
          *dead.dead = 1;
          break;
        }
      }
      __syncwarp();
    } else if (F8 && warp > kIssuer && warp <= kIssuer + kConvertWarps) {
      // ---- E4M3 caches: Q split for the product with K as it is; V to fp16 (exact) for that with P ----
      const int tid = threadIdx.x - (kIssuer + 1) * 32;  // 0..127
      int slot = 1;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int seg = 0; ok && walk.next(s); ++seg) {
        const int qb = seg % S::kQBufs;
        ok = mbar_wait_warp(smem_addr(&st->q_loaded[qb]), (seg / S::kQBufs) & 1, dead);
        // the tile before the last is done with: so are the factors of the segment before the last
        ok = ok && mbar_wait_warp(smem_addr(&st->v16_empty[it & 1]), ((it >> 1) & 1) ^ 1, dead);
        if (!ok) break;
        const float c = P.scale_log2 * (!PAGES && P.cache.k_scale ? __ldg(P.cache.k_scale + s.head) : 1.0f);
        split_queries<D, NT, kConvertWarps * 32>(q_buf + qb * S::kQ, tid, NT, c, st->mult[seg & 1]);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&st->q_full[qb]));
          mbar_arrive(smem_addr(&st->mult_full[seg & 1]));
        }

        for (int tile = s.tile0; ok && tile < s.tile1; ++tile, ++it) {
          ok = ok && mbar_wait_warp(smem_addr(&st->ring_full[slot]), phase, dead);
          ok = ok && mbar_wait_warp(smem_addr(&st->v16_empty[it & 1]), ((it >> 1) & 1) ^ 1, dead);
          if (!ok) break;
          // a slot per thread: its vectors lie in different banks from its neighbours' by the swizzle, in the
          // ring and in fp16
          const int row = tid;
          const char* src = ring + slot * S::kRing + row * D;
          const int sw = D == 128 ? row & 7 : (row >> 1) & 3;
          uint4 raw[D / 16];
#pragma unroll
          for (int v = 0; v < D / 16; ++v) raw[v] = *reinterpret_cast<const uint4*>(src + ((v ^ sw) * 16));
          const int at = tile * kTileSlots + row;
          if (at >= s.ctx) {
            // Slots past the end are zeroed: their weights are 0, but 0 times what they hold may not be.  New
            // tokens' values that are not finite are taken out here and added at the end to the rows that
            // attend to them.
            bool bad = false;
#pragma unroll
            for (int v = 0; v < D / 16; ++v) {
              uint32_t* x = reinterpret_cast<uint32_t*>(&raw[v]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {  // the code 0x7F of either sign is NaN
                const uint32_t nan = __vcmpeq4(x[j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                bad |= nan != 0;
                x[j] = at < s.end ? x[j] & ~nan : 0u;
              }
            }
            if (bad && at < s.end) st->bad_value[seg & 3] = seg + 1;
          }
          char* out = v16 + (it & 1) * S::kTile16 + row * 128;
          const int sw16 = row & 7;
#pragma unroll
          for (int v = 0; v < D / 16; ++v) {
            const uint32_t* x = reinterpret_cast<const uint32_t*>(&raw[v]);
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) e4m3_to_half(x[j], h[2 * j], h[2 * j + 1]);
            char* o = out + (v / 4) * (kTileSlots * 128);
            const int j0 = (v % 4) * 2;
            *reinterpret_cast<uint4*>(o + ((j0 ^ sw16) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(o + (((j0 + 1) ^ sw16) * 16)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&st->v16_full[it & 1]));
            mbar_arrive(smem_addr(&st->ring_empty[slot]));
          }
          slot += 2;
          if (slot >= S::kSlots) slot -= S::kSlots, phase ^= 1;
        }
      }
    }
  } else {
    if constexpr (S::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kMoreRegs));
    Walk<AttnParams> walk(P, start_b, start_offset, first, count);
    Segment s;
    // ---- softmax and output; no branch around a group_sync depends on anything but the plan and votes ----
    const int wg = warp >> 2, quad = warp & 3, bar = 1 + wg;
    const int key = quad * 32 + lane, wtid = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int CK = S::kChunk;
    const auto row_of = [&](int own) { return ((own / CK) * S::kGroups + wg) * CK + own % CK; };  // of the warpgroup's columns
    const int my_row = row_of(wtid);  // wtid < kOwn
    if (wtid < S::kOwn) {
      const int t = my_row / P.group, g = my_row - t * P.group;
      st->place[my_row] = (int64_t)t * P.out.token + (int64_t)g * P.out.head;
    }
    // this lane's column and its token, for the ballots
    const int rule_row = lane < S::kOwn ? row_of(lane) : kMaxRows, rule_token = rule_row / P.group;
    constexpr float kLift = F8 ? kLift16 : 0.0f;
    float l[S::kChunks][CK];
    // The sum that lse is the logarithm of: over bf16, where l is of rounded weights, a second one, of the weights before their
    // rounding (64 x 7 tokens, 28 rows, 1000 to 16000 slots: 333 us against 332 without; 32 x 16 to 32 x 32 tokens, 500 to 9000 slots:
    // 64 rows 115, 111; 68 rows 123, 116; 128 rows 162, 134, where the sums spill).
    float raw[LSE ? S::kChunks : 1][LSE ? CK : 1];
    uint32_t it = 0;
    int v_slot = 1;
    uint32_t v_phase = 0;
    const auto col = [&](int j) { return (S::kGroups * j + wg) * CK; };

    if (threadIdx.x == 0) P.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    for (int seg = 0; walk.next(s); ++seg) {
      const int t0 = s.row_group * P.tokens;
      const int rows = min(max((s.tokens - t0) * P.group, 0), P.rows);  // valid ones come first
      const float c = P.scale_log2;
      const float* mult = st->mult[seg & 1];
      const float v_scale = F8 && !PAGES && P.cache.v_scale ? __ldg(P.cache.v_scale + s.head) : 1.0f;
      group_sync(bar);  // the last segment's row states are read
      if (wtid < S::kOwn) {
        st->top[my_row] = -INFINITY;
        st->shift[my_row] = my_row < rows ? kNone : -INFINITY;  // rows that are none: weights 0, and no vote
      }
      if (s.tile1 * kTileSlots > s.ctx) {  // new tokens among the slots: who attends to which
        uint64_t rule = 0;
        const int t = t0 + rule_token;
        if (rule_row < rows)
          rule = P.mask ? (uint64_t)__ldg(P.mask + (int64_t)s.b * P.batch.T + t) : t >= 63 ? ~0ull : (2ull << t) - 1;
        for (int i = quad; i < s.tokens; i += 4) {
          const uint32_t word = __ballot_sync(~0u, (rule >> i) & 1);
          if (lane == 0) st->seen[wg][i] = word;
        }
      }
      if constexpr (F8) mbar_wait(smem_addr(&st->mult_full[seg & 1]), (seg >> 1) & 1, dead);
      group_sync(bar);
#pragma unroll
      for (int j = 0; j < S::kChunks; ++j)
#pragma unroll
        for (int i = 0; i < CK; ++i) {
          l[j][i] = 0.0f;
          if constexpr (LSE) raw[j][i] = 0.0f;
        }

      for (int tile = s.tile0; tile < s.tile1; ++tile, ++it) {
        const int sb = it & 1;
        const uint32_t s_col = lanes + sb * NT;
        mbar_wait(smem_addr(&st->s_full[sb]), (it >> 1) & 1, dead);
        // Page scales: a key's is a factor of its scores.  A value's goes into the weight, as an addend of the exponent, so
        // that the largest product of weight and scale is what a row's maximum follows and fp16 reaches down from; the sum of
        // the weights themselves takes it out again.
        float k_factor = 1.0f, v_log2 = 0.0f, v_inverse = 1.0f;
        if constexpr (PAGES) {
          mbar_wait(smem_addr(&st->scales_full[it & (S::kAheadScales - 1)]), (it / S::kAheadScales) & 1, dead);
          const float4 x = st->scales[it & (S::kAheadScales - 1)][key >> min(P.cache.page_shift, 7)];
          k_factor = x.x, v_log2 = x.y, v_inverse = x.z;
        }
        __syncwarp();
        if (PAGES && lane == 0) mbar_arrive(smem_addr(&st->scales_empty[it & (S::kAheadScales - 1)]));
        tc_fence_after();

        const auto weigh = [&](auto tag) {
          constexpr bool MASKED = decltype(tag)::value;  // the tile reaches past the context
          uint32_t see = ~0u;                            // columns that attend to this thread's slot
          if constexpr (MASKED) {
            const int slot = tile * kTileSlots + key, fresh = slot - s.ctx;
            see = slot >= s.end ? 0 : fresh < 0 ? ~0u : st->seen[wg][fresh];
          }
          const auto sees = [&](int j, int i) { return !MASKED || ((see >> (j * CK + i)) & 1); };
          const auto scores = [&](int j, float (&z)[CK]) {  // in log2 units, less the maximum in use
            tm_load<CK>(s_col + col(j), z);
#pragma unroll
            for (int i = 0; i < CK; i += 4) {
              const float4 m = *reinterpret_cast<const float4*>(&st->shift[col(j) + i]);
              const float4 f = F8 ? *reinterpret_cast<const float4*>(&mult[col(j) + i]) : make_float4(c, c, c, c);
              float2 z0 = make_float2(z[i], z[i + 1]), z1 = make_float2(z[i + 2], z[i + 3]), m0 = make_float2(m.x, m.y), m1 = make_float2(m.z, m.w);
              if constexpr (PAGES) {
                z0 = mul2(z0, make_float2(k_factor, k_factor)), z1 = mul2(z1, make_float2(k_factor, k_factor));
                m0 = add2(m0, make_float2(v_log2, v_log2)), m1 = add2(m1, make_float2(v_log2, v_log2));
              }
              const float2 a = fma2(z0, make_float2(f.x, f.y), m0);
              const float2 b = fma2(z1, make_float2(f.z, f.w), m1);
              z[i] = a.x, z[i + 1] = a.y, z[i + 2] = b.x, z[i + 3] = b.y;
            }
          };
          // One pass makes scores and weights with the maximum in use and adds the weights up; a vote on the
          // largest weight then says whether they stand.  (Without kHold: a vote on the scores, then the weights.)
          uint32_t p[S::kHold ? S::kChunks : 1][CK / 2];
          uint32_t over = 0;  // two fp16 or bf16 weights
          const auto store = [&](int j) {
            const uint32_t* w = p[S::kHold ? j : 0];
            char* row = p_buf + (col(j) / 64) * (kTileSlots * 128) + key * 128;
#pragma unroll
            for (int i = 0; i < CK / 8; ++i)
              *reinterpret_cast<uint4*>(row + ((((col(j) % 64) + i * 8) * 2) ^ ((key & 7) * 16))) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          };
          const auto weights = [&](int j) {
            float z[CK];
            scores(j, z);
#pragma unroll
            for (int i = 0; i < CK; i += 2) {
              if (!sees(j, i)) z[i] = -INFINITY;
              if (!sees(j, i + 1)) z[i + 1] = -INFINITY;
              float2 w = make_float2(exp2_approx(z[i]), exp2_approx(z[i + 1]));
              // the weights' rounding: bf16 to go with a bf16 cache (2^-8 of each at most), fp16 with E4M3
              if constexpr (F8) {
                const __half2 h = __floats2half2_rn(w.x, w.y), m = __hmax2(h, *reinterpret_cast<const __half2*>(&over));
                p[S::kHold ? j : 0][i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                over = *reinterpret_cast<const uint32_t*>(&m);
              } else {
                const uint32_t h = pack_bf16(w.x, w.y);
                if constexpr (LSE) {
                  const float2 s = add2(make_float2(raw[j][i], raw[j][i + 1]), w);
                  raw[j][i] = s.x, raw[j][i + 1] = s.y;
                }
                p[S::kHold ? j : 0][i / 2] = h;
                w = make_float2(bf16_low(h), bf16_high(h));
                const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&h), *reinterpret_cast<const __nv_bfloat162*>(&over));
                over = *reinterpret_cast<const uint32_t*>(&m);
              }
              // bf16 weights are summed as they were rounded, so that a row's normalised ones sum to 1: where one slot has
              // nearly all the weight, its rounding (2^-8 of it) leaves no error.  fp16's is below the output's rounding.
              const float2 old = make_float2(l[j][i], l[j][i + 1]);
              const float2 sum = PAGES ? fma2(w, make_float2(v_inverse, v_inverse), old) : add2(old, w);
              l[j][i] = sum.x, l[j][i + 1] = sum.y;
            }
          };
          bool raise = tile == s.tile0;
          if (!raise && !S::kHold) {
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < S::kChunks; ++j)
              if (col(j) < rows) {
                float z[CK];
                scores(j, z);
#pragma unroll
                for (int i = 0; i < CK; ++i) most = fmaxf(most, sees(j, i) ? z[i] : -INFINITY);
              }
            raise = group_any(bar, most > kRescale + kLift);
          } else if (!raise) {
#pragma unroll
            for (int j = 0; j < S::kChunks; ++j)
              if (col(j) < rows) weights(j);
            // in either type a larger non-negative weight has the larger bits
            const uint32_t most = F8 ? (uint32_t)(15 + kRescale + kLift) << 10 : (uint32_t)(127 + kRescale) << 7;
            raise = group_any(bar, (over & 0xFFFF) > most || (over >> 16) > most);
          }
          if (raise) {
#pragma unroll
            for (int j = 0; j < S::kChunks; ++j)
              if (col(j) < rows) {
                float x[CK];
                if (S::kHold && tile > s.tile0) {  // take the weights back; those over 2^100 (2^90) leave nothing of what was there before
                  scores(j, x);
#pragma unroll
                  for (int i = 0; i < CK; ++i) {
                    float w = sees(j, i) ? exp2_approx(x[i]) : 0.0f;
                    if constexpr (LSE) raw[j][i] = w < 0x1p100f ? raw[j][i] - w : 0.0f;
                    if constexpr (!F8) w = __bfloat162float(__float2bfloat16(w));  // as it was added
                    l[j][i] = w < (PAGES ? 0x1p90f : 0x1p100f) ? (PAGES ? fmaf(-w, v_inverse, l[j][i]) : l[j][i] - w) : 0.0f;
                  }
                }
                tm_load<CK>(s_col + col(j), x);
#pragma unroll
                for (int i = 0; i < CK; ++i) {
                  const float z = PAGES ? fmaf(x[i] * k_factor, mult[col(j) + i], v_log2) : x[i] * (F8 ? mult[col(j) + i] : c);
                  x[i] = sees(j, i) ? z : -INFINITY;
                }
                const float m = fold_lanes<CK>(x, lane, [](float a, float b) { return fmaxf(a, b); });
                if (lane < CK) st->red[quad][col(j) + lane] = m;
              }
            group_sync(bar);
            if (wtid < S::kOwn && my_row < rows) {
              const float old = st->top[my_row];
              float top = old;
#pragma unroll
              for (int w = 0; w < 4; ++w) top = fmaxf(top, st->red[w][my_row]);
              st->factor[my_row] = old == -INFINITY ? 0.0f : exp2_approx(old - top);
              st->top[my_row] = top;
              st->shift[my_row] = top == -INFINITY ? kNone : kLift - top;
            }
            group_sync(bar);
          }
          // the last product is done: P may be written again, and O rescaled
          if (it > 0) mbar_wait(smem_addr(&st->o_full), (it - 1) & 1, dead);
          __syncwarp();
          if (raise) {
            if (tile > s.tile0) {
              tc_fence_after();
#pragma unroll
              for (int j = 0; j < S::kChunks; ++j)
                if (col(j) < rows) {
                  float x[CK];
                  tm_load<CK>(lanes + 2 * NT + col(j), x);
#pragma unroll
                  for (int i = 0; i < CK; ++i) {
                    const float f = st->factor[col(j) + i];
                    x[i] *= f;
                    l[j][i] *= f;
                    if constexpr (LSE) raw[j][i] *= f;
                  }
                  tm_store<CK>(lanes + 2 * NT + col(j), x);
                }
              tm_wait_store();
            }
            if constexpr (S::kHold) {
#pragma unroll
              for (int j = 0; j < S::kChunks; ++j)
                if (col(j) < rows) weights(j);
            }
          }
#pragma unroll
          for (int j = 0; j < S::kChunks; ++j)
            if (col(j) < rows) {
              if constexpr (!S::kHold) weights(j);
              store(j);
            }
          tc_fence_before();
          if constexpr (!F8 && MASKED) {
            // V's slots past the end are zeroed: their weights are 0, but 0 times what they hold may not
            // be.  New tokens' values that are not finite are taken out here and added at the end to the
            // rows that attend to them.
            mbar_wait(smem_addr(&st->ring_full[v_slot]), v_phase, dead);
            char* v = ring + v_slot * S::kRing;
            const int from = max(s.ctx - tile * kTileSlots, 0), end = s.end - tile * kTileSlots;
            // pages behind the last one came as zeros
            const int stop = min(kTileSlots, end + (-s.end & ((1 << P.cache.page_shift) - 1)));
            constexpr int kVecs = D / 8;
            for (int u = from * kVecs + (int)threadIdx.x; u < stop * kVecs; u += kSoftmaxWarps * 32) {
              const int row = u / kVecs, vec = u % kVecs;
              uint4* p = reinterpret_cast<uint4*>(v + (vec / 8) * (kTileSlots * 128) + row * 128 + (((vec % 8) ^ (row & 7)) * 16));
              if (row >= end) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                uint4 w = *p;
                uint32_t* x = reinterpret_cast<uint32_t*>(&w);
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t odd = __vcmpeq2(x[i] & 0x7F807F80u, 0x7F807F80u);
                  bad |= odd != 0;
                  x[i] &= ~odd;
                }
                if (bad) {
                  *p = w;
                  st->bad_value[seg & 3] = seg + 1;
                }
              }
            }
          }
        };
        if ((tile + 1) * kTileSlots > s.ctx)
          weigh(std::true_type{});
        else
          weigh(std::false_type{});
        if constexpr (!F8) {
          v_slot += 2;
          if (v_slot >= S::kSlots) v_slot -= S::kSlots, v_phase ^= 1;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&st->s_empty[sb]));
          mbar_arrive(smem_addr(&st->p_full));
        }
      }

      // ---- the segment's end ----
#pragma unroll
      for (int j = 0; j < S::kChunks; ++j)
        if (col(j) < rows) {
          const float sum = fold_lanes<CK>(l[j], lane, [](float a, float b) { return a + b; });
          if (lane < CK) st->red[quad][col(j) + lane] = sum;
        }
      group_sync(bar);
      const bool whole = s.tile0 == 0 && s.tile1 == s.tiles;
      // parts: slot 0 for an item that an earlier CTA began, slot 1 for one that a later one ends
      const int64_t part_row = ((int64_t)blockIdx.x * 2 + (s.tile0 == 0)) * P.rows;
      float lse = -INFINITY;
      if (wtid < S::kOwn) {
        float f = 0.0f;
        if (my_row < rows) {
          const float sum = st->red[0][my_row] + st->red[1][my_row] + st->red[2][my_row] + st->red[3][my_row];
          f = sum == 0.0f ? 0.0f : v_scale / sum;
          if (!whole) P.part_ml[part_row + my_row] = make_float2(st->top[my_row], sum);
          else if (!LSE && P.lse) lse = row_lse(st->top[my_row], kLift, sum);
        }
        st->factor[my_row] = f;
      }
      if constexpr (LSE) {
        group_sync(bar);  // the sums of l are read
#pragma unroll
        for (int j = 0; j < S::kChunks; ++j)
          if (col(j) < rows) {
            const float part = fold_lanes<CK>(raw[j], lane, [](float a, float b) { return a + b; });
            if (lane < CK) st->red[quad][col(j) + lane] = part;
          }
        group_sync(bar);
        if (wtid < S::kOwn && my_row < rows) {
          const float sum = st->red[0][my_row] + st->red[1][my_row] + st->red[2][my_row] + st->red[3][my_row];
          if (whole) lse = row_lse(st->top[my_row], kLift, sum);
          else P.part_raw[part_row + my_row] = sum;
        }
      }
      mbar_wait(smem_addr(&st->o_full), (it - 1) & 1, dead);
      __syncwarp();
      tc_fence_after();
      group_sync(bar);
      const bool bad = st->bad_value[seg & 3] == (uint32_t)seg + 1;
      const bool lost = *dead.dead != 0;
      if (lost && !whole && wtid < S::kOwn && my_row < rows) {  // the join makes NaN of the row then (a NaN maximum it would pass over)
        P.part_ml[part_row + my_row].y = NAN;
        if constexpr (LSE) P.part_raw[part_row + my_row] = NAN;
      }
      char* out = P.out.data + s.b * P.out.row + (int64_t)t0 * P.out.token + (int64_t)s.head * P.group * P.out.head + key * 2;
      float* part = P.part + part_row * D + key;
      const int rows_all = min(P.rows, (P.batch.T - t0) * P.group);
      if (P.lse && whole && wtid < S::kOwn && my_row < rows_all)
        P.lse[lse_place(s.b, P.batch.T, t0 + my_row / P.group, P.heads, s.head, P.group, my_row % P.group)] = lost ? NAN : lse;
#pragma unroll
      for (int j = 0; j < S::kChunks; ++j) {
        const int n0 = col(j);
        if (n0 >= rows_all) continue;
        float x[CK];
#pragma unroll
        for (int i = 0; i < CK; ++i) x[i] = 0.0f;
        if (n0 < rows) tm_load<CK>(lanes + 2 * NT + n0, x);
        if (key >= D) continue;
        if (bad) {  // values that are not finite: each row takes those of the tokens it attends to
          for (int i = max(s.tile0 * kTileSlots - s.ctx, 0); s.ctx + i < min(s.tile1 * kTileSlots, s.end); ++i) {
            const int at = s.ctx + i;
            const int pg = __ldg(P.batch.pages + (int64_t)s.b * P.batch.max_pages + (at >> P.cache.page_shift));
            if (pg < 0 || pg >= P.cache.num_pages) continue;
            const char* p = P.cache.v + pg * P.cache.page + (at & ((1 << P.cache.page_shift) - 1)) * P.cache.slot +
                            s.head * P.cache.head + key * (F8 ? 1 : 2);
            const float v = F8 ? ((*reinterpret_cast<const uint8_t*>(p) & 0x7F) == 0x7F ? NAN : 0.0f)
                               : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
            if (isfinite(v)) continue;
            const uint32_t see = st->seen[wg][i];
#pragma unroll
            for (int n = 0; n < CK; ++n)
              if ((see >> (j * CK + n)) & 1) x[n] += v;
          }
        }
        if (lost) {
#pragma unroll
          for (int i = 0; i < CK; ++i) x[i] = NAN;
        }
        if (whole) {
          int64_t place[CK];
#pragma unroll
          for (int i = 0; i < CK; i += 2) {
            const longlong2 w = *reinterpret_cast<const longlong2*>(&st->place[n0 + i]);
            place[i] = w.x, place[i + 1] = w.y;
          }
#pragma unroll
          for (int i = 0; i < CK; ++i)  // rows past the request's tokens are 0 (their products may hold anything)
            x[i] = lost ? x[i] : n0 + i < rows ? x[i] * st->factor[n0 + i] : 0.0f;
#pragma unroll
          for (int i = 0; i < CK; ++i)
            if (n0 + i < rows_all) *reinterpret_cast<__nv_bfloat16*>(out + place[i]) = __float2bfloat16(x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < CK; ++i)
            if (n0 + i < rows) part[(n0 + i) * D] = x[i];
        }
      }
      tc_fence_before();
      // an item that begins here and is cut: who joins it finds it in this CTA's record
      if (threadIdx.x == 0 && s.tile0 == 0 && s.tile1 < s.tiles)
        P.cut[blockIdx.x] = make_int4(s.b, s.head * P.row_groups + s.row_group, s.item_end, total);
    }
  }

  tc_fence_before();
  __syncthreads();
  const bool lost = *dead.dead != 0;  // a wait ran out: products and copies may be in flight that nobody saw end
  if (warp == kIssuer) {
    tc_fence_after();
    if (lost) {
      tc_commit(smem_addr(&st->products_done));  // arrives behind every product of this warp
      mbar_drain(smem_addr(&st->products_done), 0);
      __syncwarp();
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kColumns));
  }
  if (lost && warp == kProducer) {
    // Tile i of K is copy 2 i of the ring, of V copy 2 i + 1; copy n goes to slot n % kSlots.  A slot is filled again only
    // when its last filling was used, so the last copy of each slot is the only one that may be in flight.
    for (int slot = 0; slot < S::kSlots; ++slot) {
      int last = -1;
      for (int kv = 0; kv < 2; ++kv) {
        const int issued = st->copies[kv];
        for (int i = issued - 1; i >= max(issued - S::kSlots, 0); --i)
          if ((2 * i + kv) % S::kSlots == slot) {
            last = max(last, 2 * i + kv);
            break;
          }
      }
      if (last >= 0) mbar_drain(smem_addr(&st->ring_full[slot]), (last / S::kSlots) & 1);
    }
    for (int i = max(st->queries - S::kQBufs, 0); i < st->queries; ++i)
      mbar_drain(smem_addr(&st->q_loaded[i % S::kQBufs]), (i / S::kQBufs) & 1);
  }
}

// ------------------------------------------------------------------------------------------------
// the join of cut items
// ------------------------------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

struct JoinParams {
  Heads out;
  Batch batch;
  const float* v_scale;
  const float* part;
  const float2* part_ml;
  const float* part_raw;  // null: lse is of part_ml's sums
  const int4* cut;
  float* lse;
  float lift;
  int heads, group, tokens, row_groups, rows, ctas;
};

// Block (x, y): the item that begins in CTA x and ends in a later one, rows 8 y .. 8 y + 7, a warp each.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ JoinParams P) {
  pdl_launch_next();
  pdl_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int n = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int4 cut = P.cut[c0];
  if (cut.x < 0 || n >= P.rows) return;
  const int b = cut.x, head = cut.y / P.row_groups, t0 = cut.y % P.row_groups * P.tokens;
  const int end = cut.z, total = cut.w;
  const int ctas = min(P.ctas, total);
  const int t = t0 + n / P.group;
  if (t >= P.batch.T) return;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(P.out.data + b * P.out.row + t * P.out.token +
                                                        (int64_t)(head * P.group + n % P.group) * P.out.head);
  constexpr int E = D / 32;
  float o[E] = {};
  float sum = 0.0f, raw = 0.0f, top = -INFINITY;
  if (t < batch_tokens(P.batch, b)) {
    // the last CTA of the item: the one whose part of the line holds tile end - 1
    int c1 = (int)(((int64_t)end * ctas - 1) / total);
    while (c1 + 1 < ctas && line_cut(total, c1 + 1, ctas) < end) ++c1;
    while (line_cut(total, c1, ctas) >= end) --c1;
    const auto row_of = [&](int c) { return ((int64_t)c * 2 + (c == c0)) * P.rows + n; };
    for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, P.part_ml[row_of(c)].x);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    for (int c = c0; c <= c1; c += 32) {
      float f = 0.0f, part = 0.0f, raw_part = 0.0f;
      if (c + lane <= c1) {
        const float2 ml = P.part_ml[row_of(c + lane)];
        f = exp2_approx(ml.x - base);
        part = f * ml.y;
        if (P.part_raw) raw_part = f * P.part_raw[row_of(c + lane)];
      }
#pragma unroll
      for (int d = 16; d > 0; d /= 2) part += __shfl_xor_sync(~0u, part, d), raw_part += __shfl_xor_sync(~0u, raw_part, d);
      sum += part, raw += raw_part;
      const int last = min(32, c1 + 1 - c);
#pragma unroll 4
      for (int i = 0; i < last; ++i) {
        const float g = __shfl_sync(~0u, f, i);
        const float* p = P.part + row_of(c + i) * D + lane * E;
        float x[E];
        if constexpr (E == 4) {
          const float4 w = *reinterpret_cast<const float4*>(p);
          x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        } else {
          const float2 w = *reinterpret_cast<const float2*>(p);
          x[0] = w.x, x[1] = w.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += g * x[e];
      }
    }
  }
  if (P.lse && lane == 0) P.lse[lse_place(b, P.batch.T, t, P.heads, head, P.group, n % P.group)] = row_lse(top, P.lift, P.part_raw ? raw : sum);
  const float v = P.v_scale ? __ldg(P.v_scale + head) : 1.0f;
  const float inv = sum == 0.0f ? 0.0f : v / sum;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(out + lane * E + e) = pack_bf16(o[e] * inv, o[e + 1] * inv);
}

// ------------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------------
struct AttnLayout {
  size_t part, ml, raw, cut, bytes;
};
static AttnLayout attn_layout(int rows, int D) {
  const auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  AttnLayout L;
  L.part = 0;
  L.ml = up(L.part + (size_t)kMaxParts * 2 * rows * D * sizeof(float));
  L.raw = up(L.ml + (size_t)kMaxParts * 2 * rows * sizeof(float2));
  L.cut = up(L.raw + (size_t)kMaxParts * 2 * rows * sizeof(float));
  L.bytes = up(L.cut + kMaxParts * sizeof(int4));
  return L;
}

template <int D, int KIND, int NT>
static cudaError_t launch_attention(const AttnParams& P, int dev, int ctas, cudaStream_t st) {
  constexpr bool F8 = holds_e4m3(KIND);
  using S = Shape<D, KIND, NT>;
  auto kern = attn_kernel<D, KIND, NT>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel's shared memory is set
  cudaError_t e = cudaSuccess;
  if (!((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    if constexpr (S::kSplit) {  // the split must not ask for more than the launch gets: the kernel would wait for it
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kern);
      if (e != cudaSuccess) return e;
      if (fa.numRegs < S::kLaunchRegs) return cudaErrorInvalidConfiguration;
    }
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  e = launch_early(kern, dim3(ctas), dim3(S::kThreads), S::kBytes, st, P);
  if (e != cudaSuccess || ctas == 1 || P.whole) return e;
  const JoinParams J = {P.out, P.batch, F8 ? P.cache.v_scale : nullptr, P.part, P.part_ml, KIND == kBf16Lse ? P.part_raw : nullptr, P.cut, P.lse, F8 ? kLift16 : 0.0f,
                        P.heads, P.group, P.tokens, P.row_groups, P.rows, ctas};
  return launch_early(join_kernel<D>, dim3(ctas, (P.rows + kJoinWarps - 1) / kJoinWarps), dim3(kJoinWarps * 32), 0, st, J);
}

template <int D, int KIND>
static cudaError_t launch_rows(const AttnParams& P, int dev, int ctas, cudaStream_t st) {
  if (P.rows <= 16) return launch_attention<D, KIND, 16>(P, dev, ctas, st);
  if (P.rows <= 32) return launch_attention<D, KIND, 32>(P, dev, ctas, st);
  if (P.rows <= 64) return launch_attention<D, KIND, 64>(P, dev, ctas, st);
  // a width of its own: 128 columns' sums spill where 96 do not (68 rows, E4M3: 118 us against 139; bf16: 114, 118)
  if (P.rows <= 96) return launch_attention<D, KIND, 96>(P, dev, ctas, st);
  return launch_attention<D, KIND, 128>(P, dev, ctas, st);
}

template <int D>
static cudaError_t launch_kind(int kind, const AttnParams& P, int dev, int ctas, cudaStream_t st) {
  if (kind == kBf16) return launch_rows<D, kBf16>(P, dev, ctas, st);
  if (kind == kBf16Lse) return launch_rows<D, kBf16Lse>(P, dev, ctas, st);
  if (kind == kE4m3) return launch_rows<D, kE4m3>(P, dev, ctas, st);
  return launch_rows<D, kE4m3Pages>(P, dev, ctas, st);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_paged_attention_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t heads, int32_t head_dim) {
  if (B < 0 || T < 0 || T > SPEC_MAX_NEW || heads < 1 || q_heads < 1 || q_heads % heads) return 0;
  if (q_heads / heads > SPEC_MAX_GROUP) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  if (T == 0) return 256;
  int tokens, groups;
  row_groups(T, q_heads / heads, &tokens, &groups);
  return attn_layout(tokens * (q_heads / heads), head_dim).bytes;
}

spec_status_t spec_paged_attention_ex(const spec_heads_t* q, const spec_heads_t* out, int32_t q_heads,
                                      const spec_kv_cache_t* cache, const spec_kv_page_scales_t* scales,
                                      const spec_decode_batch_t* batch, const int64_t* mask, float scale, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  spec_status_t s = check_cache(cache, true);
  if (s == SPEC_OK) s = check_scales(scales, cache);
  if (s == SPEC_OK) s = check_batch(batch, cache);
  if (s != SPEC_OK) return s;
  if (q_heads < 1 || q_heads % cache->heads || !isfinite(scale) || ((uintptr_t)lse & 3u)) return SPEC_ERR_INVALID_ARG;
  if (batch->T > SPEC_MAX_NEW || batch->B > SPEC_MAX_BATCH || q_heads / cache->heads > SPEC_MAX_GROUP) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0 || batch->T == 0) return SPEC_OK;
  if (!heads_ok(q) || !heads_ok(out)) return SPEC_ERR_INVALID_ARG;
  const int D = cache->head_dim, group = q_heads / cache->heads;
  const size_t need = spec_paged_attention_workspace_bytes(batch->B, batch->T, q_heads, cache->heads, D);
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < need) return SPEC_ERR_WORKSPACE;

  AttnParams P = {};
  P.out = heads_of(out);
  P.cache = cache_of(cache);
  P.scales = scales_of(scales);
  P.batch = batch_of(batch, cache);
  P.mask = mask;
  P.lse = lse;
  P.heads = cache->heads, P.group = group;
  row_groups(batch->T, group, &P.tokens, &P.row_groups);
  P.rows = group * P.tokens;
  P.scale_log2 = scale * kLog2e;
  const AttnLayout L = attn_layout(P.rows, D);
  char* ws = static_cast<char*>(workspace);
  P.part = reinterpret_cast<float*>(ws + L.part);
  P.part_ml = reinterpret_cast<float2*>(ws + L.ml);
  P.part_raw = reinterpret_cast<float*>(ws + L.raw);
  P.cut = reinterpret_cast<int4*>(ws + L.cut);

  // the line's length at most: what the page table could hold
  const int64_t per = ((int64_t)P.batch.slots + kTileSlots - 1) / kTileSlots;
  // E4M3 items and those of many rows take longer to begin and end (32 requests of 500 to 9000 slots, 68 rows, E4M3:
  // 125 us at 2 tiles, 118 at 4, 119 at 6; 24 rows in bf16, 0 to 4001 slots: 22.4 us at 1, 21.0 at 2, 21.5 at 3)
  P.item_cost = cache->dtype == SPEC_DTYPE_E4M3 || P.rows > 64 ? 4 : 2;
  P.whole = per <= kWholeTiles;
  P.wait_tries = g_test_hooks.load(std::memory_order_relaxed) & 2 ? 0 : kWaitTries;
  const int64_t most = (int64_t)batch->B * cache->heads * P.row_groups * ((per > 0 ? per : 1) + P.item_cost);
  if (most > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;

  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  const int es = f8 ? 1 : 2;
  const int box = cache->page_size < kTileSlots ? cache->page_size : kTileSlots;
  const Heads hq = heads_of(q);
  bool ok = encode(&P.q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, hq.data, {D, q_heads, batch->T, batch->B},
                   {hq.head, hq.token, hq.row}, {64, group, P.tokens, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
  for (int kv = 0; kv < 2; ++kv)
    ok = ok && encode(kv ? &P.v_map : &P.k_map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, es,
                      kv ? P.cache.v : P.cache.k, {D, cache->page_size, cache->heads, cache->num_pages},
                      {P.cache.slot, P.cache.head, P.cache.page}, {f8 ? D : 64, box, 1, 1},
                      f8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return SPEC_ERR_CUDA;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  int ctas = sms < kMaxParts ? sms : kMaxParts;
  if (most < ctas) ctas = (int)most;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kind = scales ? kE4m3Pages : f8 ? kE4m3 : lse ? kBf16Lse : kBf16;
  e = D == 128 ? launch_kind<128>(kind, P, dev, ctas, st) : launch_kind<64>(kind, P, dev, ctas, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status_t spec_paged_attention(const spec_heads_t* q, const spec_heads_t* out, int32_t q_heads,
                                   const spec_kv_cache_t* cache, const spec_decode_batch_t* batch,
                                   const int64_t* mask, float scale, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return spec_paged_attention_ex(q, out, q_heads, cache, nullptr, batch, mask, scale, nullptr, workspace, workspace_bytes, stream);
}

}  // extern "C"
