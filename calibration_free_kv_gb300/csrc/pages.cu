// Pages of the paged caches planned on the GPU (kvarn_plan_pages) and new tokens written to their
// slots of the fp16 cache (kvarn_fp16_store).
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "kvarn.h"

namespace kvarn {
namespace pages {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxBatch = 16384;       // needs of all sequences are held in shared memory
constexpr int kMaxShardLog = 20;       // pages of one CTA's bitmap: 128 KB of shared memory
constexpr int kMaxCluster = 8;         // the portable cluster size
constexpr uint32_t kManyPages = 1u << 30;  // needs are added up to here: no pool has as many pages
constexpr int kSpan = 1024;            // table entries that a warp marks at a time

struct PlanParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* block_table;
  int32_t* seq_lens_out;
  int64_t* slot_map;
  int32_t* status;
  int64_t num_pool_pages;
  int batch, chunk, max_pages;
  int open_tiles;
  int shard_log;  // CTA r of the cluster keeps the bitmap of pages [r << shard_log, (r + 1) << shard_log)
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster: what they wrote (shared and global memory) is seen after it.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_smem(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void peer_or(uint32_t addr, uint32_t bits) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(bits) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Tokens and pages of one sequence: the length now, the tokens that come (0 where the sequence cannot
// be served whatever the pool holds), the pages that its table row names and will name.
struct Request {
  int64_t len, add;
  int held, after;
  int bad;  // KVARN_DEV_SEQ_TOO_LONG
};
__device__ __forceinline__ Request request(const PlanParams& p, int b) {
  Request r;
  r.len = p.seq_lens[b];
  r.add = p.new_lens != nullptr ? p.new_lens[b] : p.chunk;
  r.bad = 0;
  if (r.add < 0 || r.add > p.chunk) {
    r.add = r.add < 0 ? 0 : p.chunk;
    r.bad = KVARN_DEV_SEQ_TOO_LONG;
  }
  const int64_t up = p.open_tiles ? 0 : kTile - 1;
  int64_t held = r.len < 0 ? 0 : (r.len + up) / kTile, after = r.len < 0 ? 0 : (r.len + r.add + up) / kTile;
  if (r.len < 0 || after > p.max_pages) {
    r.bad = KVARN_DEV_SEQ_TOO_LONG;
    held = held < p.max_pages ? held : p.max_pages;
    after = held;
    r.add = -1;
  }
  r.held = (int)held;
  r.after = (int)after;
  return r;
}

__device__ __forceinline__ uint32_t add_pages(uint32_t a, uint32_t b) {
  return min(a + b, kManyPages);
}

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
__device__ __forceinline__ void write_slots(const PlanParams& p, int64_t first, int64_t stride) {
  const int64_t total = (int64_t)p.batch * p.chunk;
  for (int64_t t = first; t < total; t += stride) {
    const int b = (int)(t / p.chunk);
    const int64_t at = (int64_t)p.seq_lens[b] + (t - (int64_t)b * p.chunk);
    const int64_t grown = __ldcg(p.seq_lens_out + b);
    const int64_t page = at / kTile, pages = (grown + (p.open_tiles ? 0 : kTile - 1)) / kTile;
    int64_t slot = -1;
    if (at < grown && page < pages) {
      const int32_t id = __ldcg(p.block_table + (int64_t)b * p.max_pages + page);
      if (id >= 0 && id < p.num_pool_pages) slot = (int64_t)id * kTile + at % kTile;
      else flag_error(p.status, KVARN_DEV_BAD_PAGE_ID);
    }
    p.slot_map[t] = slot;
  }
}

// One cluster plans the whole batch.  The pages that the table rows name are marked in a bitmap of the
// pool that lies in the cluster's shared memory (a shard per CTA); its zero bits, in ascending order,
// go to the sequences in order.
__global__ void __launch_bounds__(kThreads) plan_kernel(PlanParams p) {
  extern __shared__ uint32_t smem[];
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = 1 << (p.shard_log - 5);
  uint32_t* bitmap = smem;
  uint32_t* end = smem + words;  // [batch] pages wanted by sequences 0..b
  __shared__ uint32_t warp_sum[kWarps];
  __shared__ uint32_t cta_free[kMaxCluster];
  __shared__ uint32_t served_sum;

  // pages past the pool's end count as used
  const int64_t base = (int64_t)rank << p.shard_log;
  for (int w = tid; w < words; w += kThreads) {
    const int64_t left = p.num_pool_pages - base - 32 * (int64_t)w;
    bitmap[w] = left >= 32 ? 0u : left <= 0 ? ~0u : ~0u << left;
  }
  grid_dependency_wait();
  cluster_sync();

  // mark what the rows name
  const int spans = (p.max_pages + kSpan - 1) / kSpan;
  int flags = 0;
  for (int64_t it = (int64_t)warp * ctas + rank; it < (int64_t)p.batch * spans; it += (int64_t)ctas * kWarps) {
    const int b = (int)(it / spans);
    const int from = (int)(it - (int64_t)b * spans) * kSpan;
    const Request r = request(p, b);
    const int to = min(r.held, from + kSpan);
    const int32_t* row = p.block_table + (int64_t)b * p.max_pages;
    for (int i = from + lane; i < to; i += 32) {
      const int32_t id = row[i];
      if (id >= 0 && id < p.num_pool_pages)
        peer_or(peer_smem(bitmap + ((id & ((1 << p.shard_log) - 1)) >> 5), (uint32_t)id >> p.shard_log), 1u << (id & 31));
      else
        flags |= KVARN_DEV_BAD_PAGE_ID;
    }
  }

  // pages wanted, added up over the sequences (every CTA by itself)
  const int per = (p.batch + kThreads - 1) / kThreads;
  uint32_t mine = 0;
  for (int j = 0; j < per; ++j) {
    const int b = tid * per + j;
    if (b < p.batch) {
      const Request r = request(p, b);
      flags |= r.bad;
      mine = add_pages(mine, (uint32_t)(r.after - r.held));
      end[b] = mine;
    }
  }
  uint32_t scan = mine;
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t o = __shfl_up_sync(~0u, scan, d);
    if (lane >= d) scan = add_pages(scan, o);
  }
  if (lane == 31) warp_sum[warp] = scan;
  if (tid == 0) served_sum = 0;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before = add_pages(before, warp_sum[w]);
  const uint32_t up = __shfl_up_sync(~0u, scan, 1);
  if (lane > 0) before = add_pages(before, up);
  for (int j = 0; j < per; ++j) {
    const int b = tid * per + j;
    if (b < p.batch) end[b] = add_pages(end[b], before);
  }
  cluster_sync();

  // free pages of this CTA's shard: a run of words per warp
  const int run = (words + kWarps - 1) / kWarps;
  const int w0 = warp * run, w1 = min(words, w0 + run);
  uint32_t zeros = 0;
  for (int w = w0 + lane; w < w1; w += 32) zeros += __popc(~bitmap[w]);
  zeros = __reduce_add_sync(~0u, zeros);
  __syncthreads();  // warp_sum is read above
  if (lane == 0) warp_sum[warp] = zeros;
  __syncthreads();
  if (warp == 0) {
    const uint32_t all = __reduce_add_sync(~0u, warp_sum[lane]);
    if (lane < ctas) peer_store(peer_smem(cta_free + rank, lane), all);
  }
  cluster_sync();
  uint32_t free_pages = 0, first = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    if (c == rank) first = free_pages;
    free_pages += cta_free[c];
  }

  // Sequences are served in order while their pages last; one that needs none always is.
  uint32_t most = 0;
  for (int b = tid; b < p.batch; b += kThreads)
    if (end[b] <= free_pages) most = max(most, end[b]);
  most = __reduce_max_sync(~0u, most);
  if (lane == 0 && most > 0) atomicMax(&served_sum, most);
  __syncthreads();
  const uint32_t taken = served_sum;
  for (int w = 0; w < warp; ++w) first += warp_sum[w];
  for (int w = w0; w < w1 && first < taken; w += 32) {
    uint32_t z = w + lane < w1 ? ~bitmap[w + lane] : 0u;
    const uint32_t n = __popc(z);
    uint32_t at = n;
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(~0u, at, d);
      if (lane >= d) at += o;
    }
    const uint32_t all = __shfl_sync(~0u, at, 31);
    at += first - n;
    for (; z != 0u && at < taken; z &= z - 1, ++at) {
      const int b = owner_of(end, p.batch, at);
      const uint32_t start = b > 0 ? end[b - 1] : 0u;
      const Request r = request(p, b);
      p.block_table[(int64_t)b * p.max_pages + r.held + (at - start)] =
          (int32_t)(base + 32 * (int64_t)(w + lane) + (__ffs(z) - 1));
    }
    first += all;
  }
  for (int b = (int)rank * kThreads + tid; b < p.batch; b += (int)ctas * kThreads) {
    const Request r = request(p, b);
    const bool served = r.after == r.held || end[b] <= free_pages;
    if (!served) flags |= KVARN_DEV_NO_PAGES;
    p.seq_lens_out[b] = (int32_t)(r.len + (served && r.add > 0 ? r.add : 0));
  }
  if (flags != 0) flag_error(p.status, flags);
  if (p.slot_map == nullptr) return;
  cluster_sync();
  write_slots(p, (int64_t)rank * kThreads + tid, (int64_t)ctas * kThreads);
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
  int32_t* status;
};

constexpr int kStoreThreads = 256, kStoreUnroll = 4;

// A CTA copies `per_cta` tokens, 16 bytes a thread and step.
__global__ void __launch_bounds__(kStoreThreads) store_kernel(StoreParams p) {
  const int64_t t0 = (int64_t)blockIdx.x * p.per_cta;
  const int tokens = (int)min((int64_t)p.per_cta, p.tokens - t0);
  const int row = p.dim / 8, half = p.num_kv_heads * row, vecs = 2 * half;
  grid_dependency_wait();
  for (int i0 = threadIdx.x; i0 < tokens * vecs; i0 += kStoreThreads * kStoreUnroll) {
    uint4 x[kStoreUnroll];
    int64_t to[kStoreUnroll];
#pragma unroll
    for (int u = 0; u < kStoreUnroll; ++u) {
      const int i = i0 + u * kStoreThreads;
      to[u] = -1;
      if (i >= tokens * vecs) continue;
      const int t = i / vecs, r = i - t * vecs, kv = r >= half, hc = r - kv * half, h = hc / row, c = hc - h * row;
      const int64_t slot = p.slots[t0 + t];
      if (slot < 0) continue;
      if (slot >= p.num_pool_pages * kTile) {
        flag_error(p.status, KVARN_DEV_BAD_PAGE_ID);
        continue;
      }
      const __half* src = (kv ? p.v : p.k) + (t0 + t) * p.tok_stride + h * p.head_stride + 8 * c;
      x[u] = __ldcs(reinterpret_cast<const uint4*>(src));
      to[u] = ((((slot / kTile) * p.num_kv_heads + h) * 2 + kv) * kTile + slot % kTile) * p.dim + 8 * c;
    }
#pragma unroll
    for (int u = 0; u < kStoreUnroll; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4*>(p.pool + to[u]) = x[u];
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
      num_pool_pages > ((int64_t)kMaxCluster << kMaxShardLog))
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
  p.num_pool_pages = num_pool_pages;
  p.batch = batch;
  p.chunk = chunk_len;
  p.max_pages = max_pages;
  p.open_tiles = open_tiles != 0;
  const int ctas = kMaxCluster;
  p.shard_log = 5;
  while (((int64_t)ctas << p.shard_log) < num_pool_pages) ++p.shard_log;
  const int smem = (1 << (p.shard_log - 3)) + 4 * batch;
  static PerDeviceOnce smem_once;
  const void* fn = reinterpret_cast<const void*>(plan_kernel);
  if (const int st = set_smem_limit(smem_once, fn, (1 << (kMaxShardLog - 3)) + 4 * kMaxBatch); st != KVARN_OK) return st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_kernel, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
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
  p.per_cta = num_tokens > 1024 ? 4 : 1;
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
