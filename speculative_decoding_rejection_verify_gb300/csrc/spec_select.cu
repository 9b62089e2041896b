// spec_select.cu — spec_kv_select: which entries of a head's context stay, those of largest weight up to a budget.
//
// A weight's bits, turned so that a larger one is the larger number, are a key; the budget-th largest key follows from
// three histograms of its digits of 11, 11 and 10 bits, from the top.  Then a slot stays where its key is larger, or equal and
// among the first such.  With G and E the larger and equal ones before a slot, K = G + min(E, left) stay before it, so the
// slots < m that go and those >= m that stay number themselves: s - K, and K less what stays below m.
//
// A cluster of 1 to 8 blocks per (layer, request, head), each with a stretch of the slots, whose keys it holds in shared
// memory as far as they fit: weights and positions are read once.  Bound by that read on long contexts, by the chain of
// histograms on short ones.

#include <cooperative_groups.h>

#include "decode_common.cuh"

namespace cg = cooperative_groups;

namespace sv {

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
  int held;  // keys that a block holds
};

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr uint32_t kNoKey = 0x007FFFFFu;  // of -infinity

struct SelectState {
  int bins[kBins];
  int warp_sum[kSelectWarps];
  int digit, above;
  int counts[4];                    // of the block: larger, equal; and of those the ones below m
  int warp_counts[2][kSelectWarps];
};

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams P) {
  extern __shared__ uint32_t keys[];  // [held]
  __shared__ SelectState st;
  pdl_launch_next();
  pdl_wait();
  const cg::cluster_group cluster = cg::this_cluster();
  const int blocks = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int list = blockIdx.x / blocks, head = list % P.heads, rest = list / P.heads, b = rest % P.batch.B, layer = rest / P.batch.B;
  const int ctx = batch_context(P.batch, b), m = min(ctx, max(__ldg(P.budget + b), 0));
  const bool tells = rank == 0 && threadIdx.x == 0;
  if (tells && head == 0 && layer == 0) P.new_len[b] = m;
  if (m == ctx || m == 0) {  // the whole cluster
    if (tells) P.moves[list] = 0;
    return;
  }
  // positions from here on stay
  const int64_t recent = P.recent > 0 ? (int64_t)(P.seen ? __ldg(P.seen + b) : ctx) - P.recent : INT64_MAX;
  const int32_t* table = P.batch.pages + (int64_t)b * P.batch.max_pages;
  const int mask = (1 << P.page_shift) - 1;
  const int64_t base = layer * P.record.layer;
  // A larger key is a larger weight; +0 and -0 are one.
  const auto key = [&](float w, int position) -> uint32_t {
    w += 0.0f;
    if (w != w) w = -INFINITY;
    if (P.record.position && (position < P.first || position >= recent)) w = INFINITY;
    const uint32_t bits = __float_as_uint(w);
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
  };
  const auto place_of = [&](int slot) -> int64_t {  // -1: in a page outside the pool
    const int page = __ldg(table + (slot >> P.page_shift));
    return page < 0 || page >= P.num_pages ? -1 : base + (((int64_t)page * P.heads + head) << P.page_shift) + (slot & mask);
  };
  const auto key_of = [&](int slot) {
    const int64_t at = place_of(slot);
    return at < 0 ? kNoKey : key(P.record.weight[at], P.record.position ? P.record.position[at] : 0);
  };
  // this block's slots, whole words of 32 of them, and this warp's
  const int words = (ctx + 31) / 32, share = (words + blocks - 1) / blocks;
  const int word0 = min(rank * share, words), word1 = min(word0 + share, words);
  const int slot0 = word0 * 32, n = min(word1 * 32, ctx) - slot0;
  const auto key_at = [&](int i) { return i < P.held ? keys[i] : key_of(slot0 + i); };

  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) st.bins[i] = 0;
  __syncthreads();
  // the keys, with the first digit's histogram: kAhead in flight a thread
  constexpr int kAhead = 8;
  for (int i0 = threadIdx.x; i0 < n; i0 += kSelectThreads * kAhead) {
    float weight[kAhead];
    int position[kAhead];
    uint32_t in = 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kSelectThreads;
      weight[k] = -INFINITY, position[k] = P.first;
      const int64_t at = i < n ? place_of(slot0 + i) : -1;
      if (at >= 0) {
        weight[k] = P.record.weight[at], in |= 1u << k;
        if (P.record.position) position[k] = P.record.position[at];
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kSelectThreads;
      if (i >= n) break;
      const uint32_t x = (in >> k) & 1 ? key(weight[k], position[k]) : kNoKey;
      if (i < P.held) keys[i] = x;
      atomicAdd(&st.bins[x >> 21], 1);
    }
  }
  uint32_t prefix = 0;
  int left = m;  // of the keys that agree with the prefix, how many stay
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    if (digit > 0) {
      for (int i = threadIdx.x; i < kBins; i += kSelectThreads) st.bins[i] = 0;
      __syncthreads();
      const int above = digit == 1 ? 21 : 10;  // bits that have to agree
      for (int i = threadIdx.x; i < n; i += kSelectThreads) {
        const uint32_t key = key_at(i);
        if (key >> above == prefix >> above) atomicAdd(&st.bins[(key >> shift) & (digit == 1 ? 2047 : 1023)], 1);
      }
    }
    cluster.sync();
    // this thread's four bins, from the top, over all blocks
    const int top = kBins - 4 - threadIdx.x * 4;
    int4 sum = make_int4(0, 0, 0, 0);
    for (int r = 0; r < blocks; ++r) {
      const int4 x = *reinterpret_cast<const int4*>(cluster.map_shared_rank(&st.bins[top], r));
      sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
    }
    const int mine = sum.x + sum.y + sum.z + sum.w;
    int before = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(~0u, before, d);
      if (lane >= d) before += x;
    }
    if (lane == 31) st.warp_sum[warp] = before;
    before -= mine;
    cluster.sync();  // every block has read the bins
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w)
      if (w < warp) before += st.warp_sum[w];
    if (before < left && before + mine >= left) {  // one thread's
      int bin = top + 3;
      const int four[4] = {sum.w, sum.z, sum.y, sum.x};
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (bin == top + 3 - k && before + four[k] < left) before += four[k], --bin;
      st.digit = bin, st.above = before;
    }
    __syncthreads();
    prefix |= (uint32_t)st.digit << shift;
    left -= st.above;
  }
  // `left` of the keys equal to prefix stay, the lowest slots first.  Counts: of each warp's stretch, of the block, of the cluster
  const int mine_words = (word1 - word0 + kSelectWarps - 1) / kSelectWarps;
  const int first_word = min(word0 + warp * mine_words, word1), last_word = min(first_word + mine_words, word1);
  int larger = 0, equal = 0, larger_below = 0, equal_below = 0;
  if (threadIdx.x < 4) st.counts[threadIdx.x] = 0;
  for (int w = first_word; w < last_word; ++w) {
    const int slot = w * 32 + lane;
    const uint32_t key = slot < ctx ? key_at(slot - slot0) : 0;
    const uint32_t gt = __ballot_sync(~0u, slot < ctx && key > prefix), eq = __ballot_sync(~0u, slot < ctx && key == prefix);
    const uint32_t below = m - w * 32 >= 32 ? ~0u : m <= w * 32 ? 0u : (1u << (m - w * 32)) - 1;
    larger += __popc(gt), equal += __popc(eq), larger_below += __popc(gt & below), equal_below += __popc(eq & below);
  }
  __syncthreads();
  if (lane == 0) {
    st.warp_counts[0][warp] = larger, st.warp_counts[1][warp] = equal;
    atomicAdd(&st.counts[0], larger), atomicAdd(&st.counts[1], equal);
    atomicAdd(&st.counts[2], larger_below), atomicAdd(&st.counts[3], equal_below);
  }
  cluster.sync();
  int G = 0, E = 0, G_below = 0, E_below = 0;
  for (int r = 0; r < blocks; ++r) {
    const int* c = cluster.map_shared_rank(st.counts, r);
    if (r < rank) G += c[0], E += c[1];
    G_below += c[2], E_below += c[3];
  }
  cluster.sync();  // no block leaves while its counts are read
  for (int w = 0; w < warp; ++w) G += st.warp_counts[0][w], E += st.warp_counts[1][w];
  const int below_m = G_below + min(E_below, left);  // what stays below m
  if (tells) P.moves[list] = min(m - below_m, P.max_moves);
  int32_t* source = P.source + (int64_t)list * P.max_moves;
  int32_t* target = P.target + (int64_t)list * P.max_moves;
  for (int w = first_word; w < last_word; ++w) {
    const int slot = w * 32 + lane;
    const uint32_t key = slot < ctx ? key_at(slot - slot0) : 0;
    const bool is_eq = slot < ctx && key == prefix;
    const uint32_t gt = __ballot_sync(~0u, slot < ctx && key > prefix), eq = __ballot_sync(~0u, is_eq), lower = (1u << lane) - 1;
    const int e = E + __popc(eq & lower), k = G + __popc(gt & lower) + min(e, left);
    const bool stays = ((gt >> lane) & 1) || (is_eq && e < left);
    if (slot < m && !stays && slot - k < P.max_moves) target[slot - k] = slot;
    if (slot >= m && stays && k - below_m < P.max_moves) source[k - below_m] = slot;
    G += __popc(gt), E += __popc(eq);
  }
}

}  // namespace sv

using namespace sv;

extern "C" spec_status_t spec_kv_select(const spec_kv_record_t* record, const spec_decode_batch_t* batch, const int32_t* budget,
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
  if (lists > 0x0fffffffll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0) return SPEC_OK;
  const int64_t slots = (int64_t)batch->max_pages * record->page_size;
  if ((int64_t)max_moves < slots / 2) return SPEC_ERR_INVALID_ARG;
  if (!budget || !moves || !new_len || (max_moves > 0 && (!source || !target))) return SPEC_ERR_INVALID_ARG;
  SelectParams P = {};
  P.record = record_of(record);
  if (first == 0 && recent == 0) P.record.position = nullptr;
  P.batch = batch_of(batch, &sizes);
  P.budget = budget, P.seen = seen, P.source = source, P.target = target, P.moves = moves, P.new_len = new_len;
  P.heads = record->heads, P.num_pages = record->num_pages, P.first = first, P.recent = recent, P.max_moves = max_moves;
  while ((1 << P.page_shift) < record->page_size) ++P.page_shift;

  constexpr int kMostHeld = 24576;  // 96 KB: two blocks an SM
  int blocks = 1;
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  while (blocks < kMaxCluster && slots > 4096 * blocks && (lists * blocks < 4 * sms || slots > (int64_t)kMostHeld * blocks)) blocks *= 2;
  const int64_t stretch = ((slots + 31) / 32 + blocks - 1) / blocks * 32;
  P.held = (int)(stretch < kMostHeld ? stretch : kMostHeld);
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel's shared memory is set
  if (!((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
    if (cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostHeld * 4) != cudaSuccess) return SPEC_ERR_CUDA;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(lists * blocks)), cfg.blockDim = dim3(kSelectThreads), cfg.dynamicSmemBytes = (size_t)P.held * 4;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = blocks, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel, P) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
