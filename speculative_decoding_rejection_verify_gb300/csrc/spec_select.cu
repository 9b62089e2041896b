// spec_select.cu — spec_kv_select: which entries of a head's context stay, those of largest weight up to a budget.
//
// A weight's bits, turned so that a larger one is the larger number, are a key; the budget-th largest key follows from
// three histograms of its digits of 11, 11 and 10 bits, from the top.  Then a slot stays where its key is larger, or equal and
// among the first such.  With G and E the larger and equal ones before a slot, K = G + min(E, left) stay before it, so the
// slots < m that go and those >= m that stay number themselves: s - K, and K less what stays below m.
//
// A cluster of 1 to 8 blocks per (layer, request, head), each with a stretch of the slots, whose keys it holds in shared
// memory as far as they fit: weights and positions are read once.
//
// Measured: 4 layers x 16 requests x 8 heads of 30000 to 65003 entries, 16384 kept: 177 us, 1.3 TB/s of the bytes read and
// written (0.20 of a copy's 6749 GB/s).  A block's 16000 keys take about 35000 cycles: 9000 to read and count, 3500 to exchange bins for
// each digit, 3000 to count each, 15000 to number and list; three blocks an SM.  One layer of 8 requests of
// about 1000 entries: 10.5 us, the call's host part.

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
  int32_t* new_len;  // null: lengths_kernel writes it
  int heads, num_pages, page_shift, first, recent, max_moves;
  int held;  // keys that a block holds
};

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kRun = 128;  // slots that a warp takes at a time
constexpr int kMaxCluster = 8;
constexpr uint32_t kNoKey = 0x007FFFFFu;  // of -infinity

struct SelectState {
  union {
    alignas(16) int bins[kBins];
    alignas(16) uint32_t turned[kSelectWarps][kRun];  // keys of a warp's run that the block does not hold (after the histograms)
  };
  int warp_sum[kSelectWarps];
  int digit, above, whole;
  alignas(16) int counts[4];                    // of the block: larger, equal; and of those the ones below m
  int warp_counts[2][kSelectWarps];
};

__global__ void __launch_bounds__(kSelectThreads, 3) select_kernel(const __grid_constant__ SelectParams P) {
  extern __shared__ __align__(16) uint32_t keys[];  // [held]
  __shared__ SelectState st;
  pdl_launch_next();
  pdl_wait();
  const cg::cluster_group cluster = cg::this_cluster();
  const int blocks = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int list = blockIdx.x / blocks, head = list % P.heads, rest = list / P.heads, b = rest % P.batch.B, layer = rest / P.batch.B;
  const int ctx = batch_context(P.batch, b), m = min(ctx, max(__ldg(P.budget + b), 0));
  const bool tells = rank == 0 && threadIdx.x == 0;
  if (tells && head == 0 && layer == 0 && P.new_len) P.new_len[b] = m;
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
    w = w != w ? -INFINITY : w + 0.0f;
    if (position < P.first || position >= recent) w = INFINITY;
    const int bits = __float_as_int(w);
    return bits ^ ((bits >> 31) | 0x80000000);
  };
  // The keys of four slots that lie in one page, of which the last may be behind the context.
  const auto keys_of = [&](int slot) -> uint4 {
    const int page = __ldg(table + (slot >> P.page_shift));
    if (page < 0 || page >= P.num_pages) return make_uint4(kNoKey, kNoKey, kNoKey, kNoKey);
    const int64_t at = base + (((int64_t)page * P.heads + head) << P.page_shift) + (slot & mask);
    const float4 w = *reinterpret_cast<const float4*>(P.record.weight + at);
    int4 p = make_int4(P.first, P.first, P.first, P.first);
    if (P.record.position) p = *reinterpret_cast<const int4*>(P.record.position + at);
    return make_uint4(key(w.x, p.x), key(w.y, p.y), key(w.z, p.z), key(w.w, p.w));
  };
  // this block's slots, whole runs of 128 of them
  const int runs = (ctx + kRun - 1) / kRun, share = (runs + blocks - 1) / blocks;
  const int run0 = min(rank * share, runs), run1 = min(run0 + share, runs);
  const int slot0 = run0 * kRun, n = max(min(run1 * kRun, ctx) - slot0, 0);
  // four keys from i on, 0 (less than any) behind the last one
  const auto keys_at = [&](int i) -> uint4 {
    if (i < P.held) return *reinterpret_cast<const uint4*>(&keys[i]);
    uint4 x = keys_of(slot0 + i);
    if (i + 3 >= n) x.y = i + 1 < n ? x.y : 0, x.z = i + 2 < n ? x.z : 0, x.w = 0;
    return x;
  };

  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) st.bins[i] = 0;
  __syncthreads();
  // the keys, with the first digit's histogram: kAhead loads in flight a thread
  constexpr int kAhead = 4;
  const int whole = (run1 - run0) * kRun;  // up to a run's end: 0 behind the last key
  for (int i0 = threadIdx.x * 4; i0 < whole; i0 += kSelectThreads * 4 * kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kSelectThreads * 4;
      x[k] = make_uint4(0, 0, 0, 0);
      if (i < n) x[k] = keys_of(slot0 + i);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kSelectThreads * 4;
      if (i >= whole) break;
      if (i + 3 >= n) x[k].y = i + 1 < n ? x[k].y : 0, x[k].z = i + 2 < n ? x[k].z : 0, x[k].w = 0;
      if (i < P.held) *reinterpret_cast<uint4*>(&keys[i]) = x[k];
      if (x[k].x) atomicAdd(&st.bins[x[k].x >> 21], 1);
      if (x[k].y) atomicAdd(&st.bins[x[k].y >> 21], 1);
      if (x[k].z) atomicAdd(&st.bins[x[k].z >> 21], 1);
      if (x[k].w) atomicAdd(&st.bins[x[k].w >> 21], 1);
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
      const uint32_t above = digit == 1 ? 0xFFE00000u : 0xFFFFFC00u;  // bits that have to agree
      const auto count = [&](uint32_t key) {
        if (((key ^ prefix) & above) == 0) atomicAdd(&st.bins[(key >> shift) & (digit == 1 ? 2047 : 1023)], 1);
      };
      for (int i = threadIdx.x * 4; i < n; i += kSelectThreads * 4) {
        const uint4 x = keys_at(i);
        count(x.x), count(x.y), count(x.z), count(x.w);
      }
    }
    cluster.sync();
    // this thread's four bins, from the top, over all blocks
    const int top = kBins - 4 - threadIdx.x * 4;
    int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (int r0 = 0; r0 < blocks; r0 += 4) {  // four in flight: more take registers that a third block an SM needs
      int4 of_block[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < blocks) of_block[r] = *reinterpret_cast<const int4*>(cluster.map_shared_rank(&st.bins[top], r0 + r));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < blocks) sum.x += of_block[r].x, sum.y += of_block[r].y, sum.z += of_block[r].z, sum.w += of_block[r].w;
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
    before += __reduce_add_sync(~0u, lane < warp ? st.warp_sum[lane] : 0);
    if (before < left && before + mine >= left) {  // one thread's
      int bin = top + 3;
      const int four[4] = {sum.w, sum.z, sum.y, sum.x};
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (bin == top + 3 - k && before + four[k] < left) before += four[k], --bin;
      const int in_bin = bin == top + 3 ? sum.w : bin == top + 2 ? sum.z : bin == top + 1 ? sum.y : sum.x;
      st.digit = bin, st.above = before, st.whole = before + in_bin == left;
    }
    __syncthreads();
    prefix |= (uint32_t)st.digit << shift;
    left -= st.above;
    if (st.whole) {  // all of the bin's keys stay, and the lower digits do not matter
      prefix -= 1, left = 0;
      break;
    }
  }
  // `left` of the keys equal to prefix stay, the lowest slots first.  A warp takes runs of 128 slots, a word of 32 at a time:
  // what stays is a word of bits, and its counts are the warp's, of the block, of the cluster.
  const int mine_runs = (run1 - run0 + kSelectWarps - 1) / kSelectWarps;
  const int first_run = min(run0 + warp * mine_runs, run1), last_run = min(first_run + mine_runs, run1);
  const auto run_keys = [&](int r, uint32_t (&x)[4]) {  // lane l has slots r * 128 + l, + 32, ...
    const int i = r * kRun - slot0;
    if (i < P.held) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = keys[i + j * 32 + lane];
    } else {  // turned from four slots a lane
      const uint4 y = i + lane * 4 < n ? keys_at(i + lane * 4) : make_uint4(0, 0, 0, 0);
      __syncwarp();
      *reinterpret_cast<uint4*>(&st.turned[warp][lane * 4]) = y;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = st.turned[warp][j * 32 + lane];
    }
  };
  int larger = 0, equal = 0, larger_below = 0, equal_below = 0;  // this lane's, then the warp's
  if (threadIdx.x < 4) st.counts[threadIdx.x] = 0;
  for (int r = first_run; r < last_run; ++r) {
    uint32_t x[4];
    run_keys(r, x);
    if (r * kRun <= m && m < r * kRun + kRun) {  // m lies in it
      larger_below = larger, equal_below = equal;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r * kRun + j * 32 + lane < m) larger_below += x[j] > prefix, equal_below += x[j] == prefix;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) larger += x[j] > prefix, equal += x[j] == prefix;
  }
  if (last_run * kRun <= m) larger_below = larger, equal_below = equal;
  larger = __reduce_add_sync(~0u, larger), equal = __reduce_add_sync(~0u, equal);
  larger_below = __reduce_add_sync(~0u, larger_below), equal_below = __reduce_add_sync(~0u, equal_below);
  __syncthreads();
  if (lane == 0) {
    st.warp_counts[0][warp] = larger, st.warp_counts[1][warp] = equal;
    atomicAdd(&st.counts[0], larger), atomicAdd(&st.counts[1], equal);
    atomicAdd(&st.counts[2], larger_below), atomicAdd(&st.counts[3], equal_below);
  }
  cluster.sync();
  int G = 0, E = 0, G_below = 0, E_below = 0;
  int4 of_block[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < blocks) of_block[r] = *reinterpret_cast<const int4*>(cluster.map_shared_rank(st.counts, r));
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < blocks) {
      if (r < rank) G += of_block[r].x, E += of_block[r].y;
      G_below += of_block[r].z, E_below += of_block[r].w;
    }
  G += __reduce_add_sync(~0u, lane < warp ? st.warp_counts[0][lane] : 0), E += __reduce_add_sync(~0u, lane < warp ? st.warp_counts[1][lane] : 0);
  const int below_m = G_below + min(E_below, left);  // what stays below m
  if (tells) P.moves[list] = min(m - below_m, P.max_moves);
  int32_t* source = P.source + (int64_t)list * P.max_moves;
  int32_t* target = P.target + (int64_t)list * P.max_moves;
  const uint32_t lower = (1u << lane) - 1;
  for (int r = first_run; r < last_run; ++r) {
    uint32_t x[4];
    run_keys(r, x);
    const bool below = r * kRun + kRun <= m, above = r * kRun >= m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int slot = r * kRun + j * 32 + lane, before = G + min(E, left);  // `before` stay of the slots before these 32
      uint32_t stays = __ballot_sync(~0u, x[j] > prefix);
      const uint32_t eq = __ballot_sync(~0u, x[j] == prefix);
      if (eq) {  // few words have any
        G += __popc(stays);
        stays |= __ballot_sync(~0u, ((eq >> lane) & 1) && E + __popc(eq & lower) < left);
        E += __popc(eq);
      }
      const bool mine = (stays >> lane) & 1;
      const int k = __popc(stays & lower);
      if (!eq) G += __shfl_sync(~0u, k + mine, 31);  // (a count of bits takes longer)
      const int t = slot - before - k, c = before - below_m + k;
      if (!mine && (below || (!above && slot < m)) && t < P.max_moves) target[t] = slot;
      if (mine && (above || (!below && slot >= m)) && c < P.max_moves) source[c] = slot;
    }
  }
  cluster.sync();  // no block leaves while its counts are read
}

struct LengthsParams {
  Batch batch;
  const int32_t* budget;
  int32_t* new_len;
};

// The new lengths where they replace an input that the selection's blocks read until their end: behind all of them.
__global__ void __launch_bounds__(128) lengths_kernel(const __grid_constant__ LengthsParams P) {
  pdl_launch_next();
  pdl_wait();
  const int b = blockIdx.x * 128 + threadIdx.x;
  if (b < P.batch.B) P.new_len[b] = min(min(max(P.batch.ctx_len[b], 0), P.batch.slots), max(P.budget[b], 0));
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
  if (first < 0 || recent < 0 || max_moves < 0 || !record->weight || ((uintptr_t)record->weight & 15u) || ((uintptr_t)record->position & 15u) || record->layer_stride % 4 ||
      ((first > 0 || recent > 0) && !record->position))
    return SPEC_ERR_INVALID_ARG;
  const int64_t lists = (int64_t)record->layers * batch->B * record->heads;
  if (lists > 0x0fffffffll || batch->B > SPEC_MAX_BATCH) return SPEC_ERR_UNSUPPORTED;
  if (batch->B == 0) return SPEC_OK;
  const int64_t slots = (int64_t)batch->max_pages * record->page_size;
  if ((int64_t)max_moves < slots / 2) return SPEC_ERR_INVALID_ARG;
  if (!budget || !moves || !new_len || (max_moves > 0 && (!source || !target))) return SPEC_ERR_INVALID_ARG;
  // new_len may be an input itself, and must not overlap one in another way
  bool replaces = false;
  for (const int32_t* input : {batch->ctx_len, budget, seen}) {
    const uintptr_t a = (uintptr_t)input, n = (uintptr_t)new_len, bytes = (uintptr_t)batch->B * 4;
    if (input && a != n && a < n + bytes && n < a + bytes) return SPEC_ERR_INVALID_ARG;
    replaces |= a == n;
  }
  SelectParams P = {};
  P.record = record_of(record);
  if (first == 0 && recent == 0) P.record.position = nullptr;
  P.batch = batch_of(batch, &sizes);
  P.budget = budget, P.seen = seen, P.source = source, P.target = target, P.moves = moves;
  P.new_len = replaces ? nullptr : new_len;
  P.heads = record->heads, P.num_pages = record->num_pages, P.first = first, P.recent = recent, P.max_moves = max_moves;
  while ((1 << P.page_shift) < record->page_size) ++P.page_shift;

  // Blocks a list: more while they fit the GPU beside one another, as an exchange costs a block what 2000 keys do (8 lists of
  // 65000: 117 us with 1, 55 with 2, 25 with 4 or 8; 512 of 9000: 39, 54, 108, 344), and as many as hold the keys (512 of 65000, with
  // two blocks an SM: 272 with 1, 200 with 2, 209 with 4; with three 177 with 4).
  constexpr int kMostHeld = 24576;  // 96 KB
  int blocks = 1;
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPEC_ERR_CUDA;
  while (blocks < kMaxCluster && ((slots > 4096 * blocks && lists * blocks * 2 <= sms) || slots > (int64_t)kMostHeld * blocks)) blocks *= 2;
  const int64_t stretch = ((slots + kRun - 1) / kRun + blocks - 1) / blocks * kRun;
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
  if (cudaLaunchKernelEx(&cfg, select_kernel, P) != cudaSuccess) return SPEC_ERR_CUDA;
  if (!replaces) return SPEC_OK;
  const LengthsParams L = {P.batch, budget, new_len};
  return launch_early(lengths_kernel, dim3((unsigned)((batch->B + 127) / 128)), dim3(128), 0, cfg.stream, L) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
