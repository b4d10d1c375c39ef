// Pages of the paged caches planned on the GPU (kvarn_plan_pages) and new tokens written to their
// slots of the fp16 cache (kvarn_fp16_store).
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "kvarn.h"

namespace kvarn {
namespace pages {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxBatch = 16384;           // needs of all sequences are held in shared memory
constexpr int kMaxPoolLog = 23;            // pages of a pool
constexpr int kMaxBitsLog = 20;            // pages of a CTA's bitmap: 128 KB of shared memory
constexpr int kCluster = 8;                // CTAs of a large plan: the portable cluster size
constexpr uint32_t kManyPages = 1u << 30;  // needs are added up to here: no pool has as many pages
constexpr int kAhead = 8;                  // table entries that a lane has under way
constexpr int kSpan = 32 * kAhead;         // table entries that a warp marks at a time
// Slots that the planning CTAs write themselves; more take a kernel of their own (8192 slots: 7.6 against 9.2 us,
// 16384: 8.9 against 9.8, 24576: 10.0 against 10.5, 32768: 11.2 against 11.1, 65536: 13.1 against 11.3).
constexpr int64_t kSlotsHere = 16384;
// Up to these sizes (table entries, pages of the pool, tokens that come) one CTA plans, beyond them a cluster.  One
// CTA against a cluster: 1 row 4.3 / 5.8 us, 64 rows of 128 entries 5.3 / 5.9, 128 rows 6.8 / 6.2, 512 rows 15.7 / 7.6;
// 64 rows and a pool of 200,000 pages 5.8 / 6.8; 8 rows of 128 / 512 / 1024 tokens 5.1 / 7.1, 7.2 / 7.1, 10.2 / 7.1.
constexpr int64_t kSmallTable = 16384, kSmallPool = 262144, kSmallTokens = 4096;

struct PlanParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* block_table;
  int32_t* seq_lens_out;
  int64_t* slot_map;
  int32_t* status;
  int num_pool_pages;
  int batch, chunk, max_pages;
  int open_tiles;
  int ctas;   // 1, or kCluster
  int whole;  // a CTA's bitmap is the whole pool's (its marks are joined with the others'), or its share of it
  int share;  // words of the bitmap that a CTA counts and gives away
};

// All threads of the plan's CTAs: what they wrote (shared and global memory) is seen after it.
__device__ __forceinline__ void plan_sync(int ctas) {
  if (ctas == 1) {
    __syncthreads();
    return;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_smem(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Pages of a length.
__device__ __forceinline__ uint32_t pages_of(uint32_t len, int open_tiles) {
  return (len + (open_tiles ? 0 : kTile - 1)) / kTile;
}
__device__ __forceinline__ int held_pages(const PlanParams& p, int len) {
  return len < 0 ? 0 : (int)min(pages_of(len, p.open_tiles), (uint32_t)p.max_pages);
}

// One sequence: the tokens that come (-1 where it cannot be served whatever the pool holds), the pages that
// its table row names and those that it wants.
struct Request {
  int len, add, held, need, bad;
};
__device__ __forceinline__ Request request(const PlanParams& p, int b) {
  Request r;
  r.len = p.seq_lens[b];
  r.add = p.new_lens != nullptr ? p.new_lens[b] : p.chunk;
  r.bad = r.add < 0 || r.add > p.chunk ? KVARN_DEV_SEQ_TOO_LONG : 0;
  r.add = min(max(r.add, 0), p.chunk);
  r.held = held_pages(p, r.len);
  const uint32_t after = pages_of((uint32_t)r.len + (uint32_t)r.add, p.open_tiles);  // below 2^32: both are below 2^31
  if (r.len < 0 || after > (uint32_t)p.max_pages) {
    r.bad = KVARN_DEV_SEQ_TOO_LONG;
    r.add = -1;
    r.need = 0;
  } else {
    r.need = (int)after - r.held;
  }
  return r;
}

__device__ __forceinline__ uint32_t add_pages(uint32_t a, uint32_t b) { return min(a + b, kManyPages); }

// Sequence whose pages hold rank `r`: the first b with end[b] > r.
__device__ __forceinline__ int owner_of(const uint32_t* end, int batch, uint32_t r) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Slots of tokens first, first + stride, ... of the batch x chunk grid, once the lengths and the table
// rows are written.
template <class Index>
__device__ __forceinline__ void write_slots(const PlanParams& p, Index first, Index stride) {
  const Index total = (Index)p.batch * (Index)p.chunk;
  for (Index t = first; t < total; t += stride) {
    const int b = (int)(t / (Index)p.chunk);
    const uint32_t at = (uint32_t)p.seq_lens[b] + (uint32_t)(t - (Index)b * (Index)p.chunk);
    const int grown = __ldcg(p.seq_lens_out + b);
    const uint32_t page = at / kTile;
    int64_t slot = -1;
    if (grown >= 0 && at < (uint32_t)grown && page < pages_of(grown, p.open_tiles)) {
      const int32_t id = __ldcg(p.block_table + (int64_t)b * p.max_pages + page);
      if (id >= 0 && id < p.num_pool_pages) slot = (int64_t)id * kTile + at % kTile;
      else flag_error(p.status, KVARN_DEV_BAD_PAGE_ID);
    }
    p.slot_map[t] = slot;
  }
}

// One CTA, or a cluster of them, plans the whole batch.  The pages that the table rows name are marked in a
// bitmap of the pool in shared memory; its zero bits, in ascending order, go to the sequences in order.
// Bound by latency: a chain of loads, marks, two counts and the writes, with a meeting of all threads
// between them (512 rows of 16k tokens: 8.5 us, of which the loads take two trips to memory and the cluster's three
// meetings about 2 us).  A CTA of a cluster marks its rows in a bitmap of its own and reads the others' afterwards:
// marks sent to the CTA that owns the page took 10 us of 17, for they pass one by one.
__global__ void __launch_bounds__(kThreads) plan_kernel(PlanParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t warp_sum[kWarps], warp_free[kWarps];
  __shared__ uint32_t cta_free[kCluster];
  __shared__ uint32_t served_sum;
  const int rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x / 32;
  const int words = p.whole ? (p.num_pool_pages + 31) / 32 : p.share;
  const int first_word = p.whole ? 0 : rank * p.share;  // of the pool, at bitmap[0]
  uint32_t* bitmap = smem;
  uint32_t* end = smem + words;  // [batch] pages wanted by sequences 0..b
  for (int w = tid; w < words; w += blockDim.x) {
    // pages past the pool's end count as used
    const int left = p.num_pool_pages - 32 * (first_word + w);
    bitmap[w] = left >= 32 ? 0u : left <= 0 ? ~0u : ~0u << left;
  }
  if (tid == 0) served_sum = 0;
  __syncthreads();
  grid_dependency_wait();
  const int per = (p.batch + blockDim.x - 1) / blockDim.x;  // sequences of a thread, of every CTA
  const Request mine = tid < p.batch ? request(p, tid) : Request{0, 0, 0, 0, 0};  // of thread tid where per is 1

  // mark what the rows name: a CTA's rows in a bitmap of the whole pool, or all rows in its share of it
  const int spans = (p.max_pages + kSpan - 1) / kSpan;
  const int64_t items = (int64_t)p.batch * spans;
  const int lines = p.whole ? p.ctas : 1;
  int flags = 0;
  for (int64_t it = (int64_t)warp * lines + (p.whole ? rank : 0); it < items; it += (int64_t)warps * lines) {
    const int b = spans == 1 ? (int)it : (int)(it / spans);
    const int from = (int)(it - (int64_t)b * spans) * kSpan + lane;
    const int held = held_pages(p, p.seq_lens[b]);
    const int32_t* row = p.block_table + (int64_t)b * p.max_pages;
    int32_t id[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) id[j] = from + 32 * j < held ? row[from + 32 * j] : 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (from + 32 * j >= held) continue;
      if (id[j] < 0 || id[j] >= p.num_pool_pages) {
        flags |= KVARN_DEV_BAD_PAGE_ID;
        continue;
      }
      const int w = id[j] / 32 - first_word;
      if (w >= 0 && w < words) atomicOr(bitmap + w, 1u << (id[j] % 32));
    }
  }

  // pages wanted, added up over the sequences (every CTA by itself)
  uint32_t wanted = 0;
  for (int j = 0; j < per; ++j) {
    const int b = tid * per + j;
    if (b < p.batch) {
      const Request r = per == 1 ? mine : request(p, b);
      flags |= r.bad;
      wanted = add_pages(wanted, (uint32_t)r.need);
      end[b] = wanted;
    }
  }
  uint32_t scan = wanted;
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t o = __shfl_up_sync(~0u, scan, d);
    if (lane >= d) scan = add_pages(scan, o);
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  uint32_t before = __shfl_up_sync(~0u, scan, 1);
  if (lane == 0) before = 0;
  uint32_t others = lane < warp ? warp_sum[lane] : 0u;  // sums of the warps before this one
  for (int d = 16; d > 0; d /= 2) others = add_pages(others, __shfl_xor_sync(~0u, others, d));
  before = add_pages(before, others);
  for (int j = 0; j < per; ++j) {
    const int b = tid * per + j;
    if (b < p.batch) end[b] = add_pages(end[b], before);
  }
  plan_sync(p.ctas);

  // Free pages of this CTA's share of the pool, by warps: a run of words each.
  const int s0 = p.whole ? min(rank * p.share, words) : 0, s1 = min(s0 + p.share, words);
  const int run = (s1 - s0 + warps - 1) / warps;
  const int w0 = min(s0 + warp * run, s1), w1 = min(w0 + run, s1);
  uint32_t zeros = 0;
  for (int w = w0 + lane; w < w1; w += 32) {
    uint32_t used = bitmap[w];
    if (p.whole && p.ctas > 1) {
      for (int c = 1; c < kCluster; ++c) used |= peer_load(peer_smem(bitmap + w, (rank + c) % kCluster));
      bitmap[w] = used;  // no other CTA reads this CTA's share here
    }
    zeros += __popc(~used);
  }
  zeros = __reduce_add_sync(~0u, zeros);
  if (lane == 0) warp_free[warp] = zeros;
  __syncthreads();
  const uint32_t counted = lane < warps ? warp_free[lane] : 0u;
  const uint32_t in_cta = __reduce_add_sync(~0u, counted);
  uint32_t free_pages = in_cta, first = __reduce_add_sync(~0u, lane < warp ? counted : 0u);
  if (p.ctas > 1) {
    if (tid < p.ctas) peer_store(peer_smem(cta_free + rank, tid), in_cta);
    plan_sync(p.ctas);
    const uint32_t of = lane < p.ctas ? cta_free[lane] : 0u;
    free_pages = __reduce_add_sync(~0u, of);
    first += __reduce_add_sync(~0u, lane < rank ? of : 0u);
  }

  // Sequences are served in order while their pages last; one that needs none always is.
  uint32_t most = 0;
  if (end[p.batch - 1] <= free_pages) {
    most = end[p.batch - 1];
  } else {
    for (int b = tid; b < p.batch; b += blockDim.x)
      if (end[b] <= free_pages) most = max(most, end[b]);
    most = __reduce_max_sync(~0u, most);
    if (lane == 0 && most > 0) atomicMax(&served_sum, most);
    __syncthreads();
    most = served_sum;
  }
  for (int w = w0; w < w1 && first < most; w += 32) {
    const uint32_t z = w + lane < w1 ? ~bitmap[w + lane] : 0u;
    const uint32_t n = __popc(z);
    uint32_t at = n;
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(~0u, at, d);
      if (lane >= d) at += o;
    }
    const uint32_t all = __shfl_sync(~0u, at, 31);
    at -= n;
    const uint32_t give = min(all, most - first);
    for (uint32_t i0 = 0; i0 < give; i0 += 32) {
      // zero bit i of the warp's 32 words: the last lane with `at` <= i has it, then its bit by halves
      const uint32_t i = i0 + lane;
      int of = 0;
      for (int d = 16; d > 0; d /= 2)
        if (__shfl_sync(~0u, at, of + d) <= i) of += d;
      const uint32_t bits = __shfl_sync(~0u, z, of);
      uint32_t k = i - __shfl_sync(~0u, at, of);
      int bit = 0;
      for (int d = 16; d > 0; d /= 2) {
        const uint32_t low = __popc(bits >> bit & ((1u << d) - 1));
        if (k >= low) k -= low, bit += d;
      }
      if (i < give) {
        const int b = owner_of(end, p.batch, first + i);
        const uint32_t start = b > 0 ? end[b - 1] : 0u;
        p.block_table[(int64_t)b * p.max_pages + held_pages(p, p.seq_lens[b]) + (first + i - start)] =
            32 * (first_word + w + of) + bit;
      }
    }
    first += all;
  }
  if (rank == 0) {
    for (int j = 0; j < per; ++j) {
      const int b = per == 1 ? tid : tid + j * blockDim.x;
      if (b >= p.batch) continue;
      const Request r = per == 1 ? mine : request(p, b);
      const bool served = r.need == 0 || end[b] <= free_pages;
      if (!served) flags |= KVARN_DEV_NO_PAGES;
      p.seq_lens_out[b] = r.len + (served ? max(r.add, 0) : 0);
    }
  }
  if (flags != 0) flag_error(p.status, flags);
  if (p.slot_map == nullptr || p.batch * (int64_t)p.chunk > kSlotsHere) return;
  plan_sync(p.ctas);
  write_slots<uint32_t>(p, rank * blockDim.x + tid, p.ctas * blockDim.x);
}

// The slots of a large plan, over the whole GPU.
__global__ void __launch_bounds__(256) plan_slots_kernel(PlanParams p) {
  grid_dependency_wait();
  const uint64_t first = blockIdx.x * 256ull + threadIdx.x, stride = gridDim.x * 256ull;
  if ((uint64_t)p.batch * p.chunk + stride < (1ull << 32)) write_slots<uint32_t>(p, (uint32_t)first, (uint32_t)stride);
  else write_slots<uint64_t>(p, first, stride);
}

struct StoreParams {
  const __half* k;
  const __half* v;
  int64_t tok_stride, head_stride;
  const int64_t* slots;
  __half* pool;
  int64_t num_pool_pages;
  int64_t tokens;
  int num_kv_heads, dim, per_cta;
  int streaming;  // many tokens
  int32_t* status;
};

constexpr int kStoreThreads = 256, kStoreUnroll = 4;

// A CTA copies `per_cta` tokens, 16 bytes a thread and step.  A thread keeps its place within a token (key or
// value, head, channels), so that a copy costs a slot, two additions and the move: with the place worked out for
// every copy the kernel was bound by its 150 instructions a copy.
__global__ void __launch_bounds__(kStoreThreads) store_kernel(StoreParams p) {
  const int64_t t0 = (int64_t)blockIdx.x * p.per_cta;
  const int tokens = (int)min((int64_t)p.per_cta, p.tokens - t0);
  const int row = p.dim / 8, half = p.num_kv_heads * row, vecs = 2 * half;
  const int groups = vecs < kStoreThreads ? kStoreThreads / vecs : 1;  // tokens that the CTA copies side by side
  const int group = vecs < kStoreThreads ? (int)threadIdx.x / vecs : 0;
  const int64_t limit = p.num_pool_pages * kTile, page = (int64_t)p.num_kv_heads * 2 * kTile * p.dim;
  if (group >= groups) return;
  grid_dependency_wait();
  for (int i = (int)threadIdx.x - group * vecs; i < vecs; i += kStoreThreads) {
    const int kv = i >= half, hc = i - kv * half, h = hc / row, c = 8 * (hc - h * row);
    const __half* src = (kv ? p.v : p.k) + h * p.head_stride + c;
    __half* dst = p.pool + (int64_t)(2 * h + kv) * kTile * p.dim + c;
    for (int t = group; t < tokens; t += kStoreUnroll * groups) {
      uint4 x[kStoreUnroll];
      int64_t slot[kStoreUnroll];
#pragma unroll
      for (int u = 0; u < kStoreUnroll; ++u) {
        slot[u] = t + u * groups < tokens ? p.slots[t0 + t + u * groups] : -1;
        if (slot[u] >= 0 && slot[u] < limit)
          x[u] = __ldcs(reinterpret_cast<const uint4*>(src + (t0 + t + u * groups) * p.tok_stride));
      }
#pragma unroll
      for (int u = 0; u < kStoreUnroll; ++u) {
        if (slot[u] < 0) continue;
        if (slot[u] >= limit) {
          flag_error(p.status, KVARN_DEV_BAD_PAGE_ID);
          continue;
        }
        uint4* to = reinterpret_cast<uint4*>(dst + (slot[u] / kTile) * page + (slot[u] % kTile) * p.dim);
        // prompts pass through the L2 cache, a step's tokens stay
        if (p.streaming) __stcs(to, x[u]);
        else *to = x[u];
      }
    }
  }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pages
}  // namespace kvarn

using namespace kvarn;
using namespace kvarn::pages;

extern "C" {

int kvarn_plan_pages(int batch, int chunk_len, const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table,
                     int max_pages, int64_t num_pool_pages, int open_tiles, int32_t* seq_lens_out, int64_t* slot_map,
                     int32_t* dev_status, void* stream) {
  if (batch < 0 || chunk_len < 1 || max_pages < 1 || num_pool_pages < 1) return KVARN_ERR_INVALID_ARG;
  if (batch > kMaxBatch || max_pages > (1 << 23) || chunk_len > (1 << 30) ||
      num_pool_pages > (1 << kMaxPoolLog))
    return KVARN_ERR_UNSUPPORTED;
  if (batch == 0) return KVARN_OK;
  if (seq_lens == nullptr || block_table == nullptr || seq_lens_out == nullptr || seq_lens_out == seq_lens)
    return KVARN_ERR_INVALID_ARG;
  PlanParams p{};
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.block_table = block_table;
  p.seq_lens_out = seq_lens_out;
  p.slot_map = slot_map;
  p.status = dev_status;
  p.num_pool_pages = (int)num_pool_pages;
  p.batch = batch;
  p.chunk = chunk_len;
  p.max_pages = max_pages;
  p.open_tiles = open_tiles != 0;
  // One CTA where there is little to read, mark and write: the CTAs of a cluster meet three times.
  const int64_t slots = slot_map != nullptr ? (int64_t)batch * chunk_len : 0;
  const bool small = (int64_t)batch * max_pages <= kSmallTable && num_pool_pages <= kSmallPool &&
                     (int64_t)batch * chunk_len <= kSmallTokens;
  p.ctas = small ? 1 : kCluster;
  p.whole = num_pool_pages <= (1 << kMaxBitsLog);
  const int words = (int)((num_pool_pages + 31) / 32);
  p.share = (words + p.ctas - 1) / p.ctas;
  const int smem = 4 * ((p.whole ? words : p.share) + batch);
  static PerDeviceOnce smem_once;
  const void* fn = reinterpret_cast<const void*>(plan_kernel);
  if (const int st = set_smem_limit(smem_once, fn, (1 << (kMaxBitsLog - 3)) + 4 * kMaxBatch); st != KVARN_OK) return st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = p.ctas > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, plan_kernel, p) != cudaSuccess) return KVARN_ERR_CUDA;
  if (slots <= kSlotsHere) return KVARN_OK;
  const int64_t grid = (slots + 1023) / 1024;
  cfg.gridDim = dim3((unsigned)(grid < 152 * 8 ? grid : 152 * 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_slots_kernel, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

int kvarn_fp16_store(int head_dim, int num_kv_heads, int64_t num_tokens, const void* k, const void* v,
                     int64_t tok_stride, int64_t head_stride, const int64_t* slot_map, void* page_pool,
                     int64_t num_pool_pages, int32_t* dev_status, void* stream) {
  if (head_dim != 64 && head_dim != 128) return KVARN_ERR_UNSUPPORTED;
  if (num_kv_heads < 1 || num_tokens < 0 || num_pool_pages < 1) return KVARN_ERR_INVALID_ARG;
  if (num_kv_heads > 65535 || num_tokens > 0x7fffffffLL || num_pool_pages > 0x7fffffffLL) return KVARN_ERR_UNSUPPORTED;
  if (num_tokens == 0) return KVARN_OK;
  if (k == nullptr || v == nullptr || slot_map == nullptr || page_pool == nullptr) return KVARN_ERR_INVALID_ARG;
  if (!pages::aligned16(k) || !pages::aligned16(v) || !pages::aligned16(page_pool)) return KVARN_ERR_INVALID_ARG;
  if (tok_stride < 0 || head_stride < 0 || tok_stride % 8 != 0 || head_stride % 8 != 0) return KVARN_ERR_INVALID_ARG;
  StoreParams p{};
  p.k = static_cast<const __half*>(k);
  p.v = static_cast<const __half*>(v);
  p.tok_stride = tok_stride;
  p.head_stride = head_stride;
  p.slots = slot_map;
  p.pool = static_cast<__half*>(page_pool);
  p.num_pool_pages = num_pool_pages;
  p.tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.dim = head_dim;
  // Few tokens: as many CTAs as there are; many: enough copies a thread to keep their latency covered.  Few against many, 8
  // kv heads, head_dim 128: 64 tokens 1.5 / 1.7 us, 512 2.1 / 1.8, 1024 3.0 / 2.1, 1536 3.9 / 2.5, 16384 41 / 21; 2 kv heads,
  // head_dim 64: 1024 tokens 1.6 / 1.8, 4096 2.3 / 1.9.
  const int vecs = 2 * num_kv_heads * (head_dim / 8), groups = vecs < kStoreThreads ? kStoreThreads / vecs : 1;
  p.streaming = num_tokens > 1024;
  p.per_cta = (p.streaming ? kStoreUnroll : 1) * groups;
  p.status = dev_status;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((num_tokens + p.per_cta - 1) / p.per_cta));
  cfg.blockDim = dim3(kStoreThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, store_kernel, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // extern "C"
