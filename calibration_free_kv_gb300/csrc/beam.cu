// Beam search over the paged cache: the best continuations over beams and vocabulary
// (kvarn_beam_select) and the state of the beams that go on (kvarn_beam_reorder).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"
#include "kvarn.h"
#include "params.cuh"

namespace kvarn {
namespace beam {

constexpr int kMaxBeams = 32, kMaxCount = 64;
constexpr int kMaxVocab = 1 << 26;     // beam * vocab + token stays within 31 bits
constexpr int kMergeEntries = 8192;    // candidates that the merge holds in shared memory

// ---- selection: one pass over the logits ----------------------------------------------------
// A row of logits (one beam) is cut into chunks, one CTA each.  A CTA streams its chunk in tiles held
// in registers (64 bytes a thread), keeps per-thread sums of exp(x - ref) in 32 bits, and keeps the
// chunk's `count` best logits in a short list: elements above the list's threshold are appended, the
// list is cut back to `count` when it grows.  The merge joins the chunks' sums in 64 bits and takes
// the best candidates off the sorted lists.

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kWords = 16;             // 32-bit words of a tile that a thread holds
constexpr int kCap = 512;              // entries of the list
constexpr int kPruneAt = 192;          // the list is cut back beyond this many
constexpr float kStep = 40.0f;         // a thread's reference moves when a logit exceeds it by more

enum DType { kF16 = 0, kBF16 = 1, kF32 = 2 };

struct SelectParams {
  const void* logits;
  int64_t row_stride;  // elements
  const float* scores;
  const uint8_t* done;
  float2* sums;      // [rows][chunks]: reference, sum
  float2* entries;   // [rows][chunks][count]: logit, token (bits), best first; token -1 past the last
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  uint8_t* out_done;
  int32_t* status;
  int batch, beams, vocab, count, end_token;
  int chunks, chunk_len;
};

// The greater one; NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

struct F16 {
  static constexpr int kPerWord = 2;
  static constexpr uint32_t kNone = 0xfc00fc00u;  // -inf
  using Elem = uint16_t;
  static __device__ __forceinline__ float2 get(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
};
struct BF16 {
  static constexpr int kPerWord = 2;
  static constexpr uint32_t kNone = 0xff80ff80u;
  using Elem = uint16_t;
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
};
struct F32 {
  static constexpr int kPerWord = 1;
  static constexpr uint32_t kNone = 0xff800000u;
  using Elem = uint32_t;
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order of floats as unsigned integers; both zeros are one value.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A tile's elements as a thread holds them.  kBytes: the width of its loads, so that rows whose start
// is aligned to no more still stream; the place of an element depends on its index and kBytes alone,
// which makes the sums of equal rows equal.
template <class T, int kBytes>
struct Tile {
  static constexpr int kPer = kBytes / (int)sizeof(typename T::Elem);         // elements of a load
  static constexpr int kLoads = 64 / kBytes;
  static constexpr int kElems = 64 / (int)sizeof(typename T::Elem);
  static constexpr int kSize = kThreads * kElems;
  uint32_t w[kWords];

  // index within the tile of element e of this thread
  static __device__ __forceinline__ int index(int e) { return ((e / kPer) * kThreads + (int)threadIdx.x) * kPer + e % kPer; }

  __device__ __forceinline__ void load(const typename T::Elem* row, int64_t at, int64_t end) {
    if (at + kSize <= end) {
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const typename T::Elem* src = row + at + index(l * kPer);
        if constexpr (kBytes == 16) {
          const uint4 x = __ldcs(reinterpret_cast<const uint4*>(src));
          w[4 * l] = x.x, w[4 * l + 1] = x.y, w[4 * l + 2] = x.z, w[4 * l + 3] = x.w;
        } else if constexpr (kBytes == 4) {
          w[l] = __ldcs(reinterpret_cast<const uint32_t*>(src));
        } else {
          const uint32_t x = __ldcs(reinterpret_cast<const uint16_t*>(src));
          if (l % 2 == 0) w[l / 2] = x;
          else w[l / 2] |= x << 16;
        }
      }
      return;
    }
    // the chunk's last tile: whole loads while they fit, then single elements
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int64_t i = at + index(l * kPer);
      const typename T::Elem* src = row + i;
      if constexpr (kBytes == 16) {
        uint4 x = make_uint4(T::kNone, T::kNone, T::kNone, T::kNone);
        if (i + kPer <= end) {
          x = __ldcs(reinterpret_cast<const uint4*>(src));
        } else if (i < end) {
          uint32_t v[4] = {T::kNone, T::kNone, T::kNone, T::kNone};
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (i + e < end) put(v[e / T::kPerWord], e % T::kPerWord, src[e]);
          x = make_uint4(v[0], v[1], v[2], v[3]);
        }
        w[4 * l] = x.x, w[4 * l + 1] = x.y, w[4 * l + 2] = x.z, w[4 * l + 3] = x.w;
      } else if constexpr (kBytes == 4) {
        w[l] = T::kNone;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (i + e < end) put(w[l], e % T::kPerWord, src[e]);
      } else {
        if (l % 2 == 0) w[l / 2] = T::kNone;
        if (i < end) put(w[l / 2], l % 2, *src);
      }
    }
  }
  static __device__ __forceinline__ void put(uint32_t& word, int part, typename T::Elem x) {
    if constexpr (T::kPerWord == 1) word = x;
    else word = part == 0 ? (word & 0xffff0000u) | x : (word & 0xffffu) | ((uint32_t)x << 16);
  }

  __device__ __forceinline__ float max() const {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < kWords; ++i) m = T::max(m, w[i]);
    if constexpr (T::kPerWord == 1) return __uint_as_float(m);
    else {
      const float2 f = T::get(m);
      return max_nan(f.x, f.y);
    }
  }
  __device__ __forceinline__ float value(int e) const {
    if constexpr (T::kPerWord == 1) return __uint_as_float(w[e]);
    else {
      const float2 f = T::get(w[e / 2]);
      return e % 2 == 0 ? f.x : f.y;
    }
  }
  // sum of exp(x - ref)
  __device__ __forceinline__ float sum(float ref) const {
    float2 a = make_float2(0.0f, 0.0f);
    const float2 r = make_float2(-ref, -ref), l = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kElems / 2; ++i) {
      float2 x;
      if constexpr (T::kPerWord == 1) x = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else x = T::get(w[i]);
      // the difference first: it is exact near the reference, where the sum is made
      x = mul2(add2(x, r), l);
      a = add2(a, make_float2(exp2_fast(x.x), exp2_fast(x.y)));
    }
    return a.x + a.y;
  }
};

struct List {
  float2 e[kCap];  // logit, token
  int n;
  float threshold;  // `count` elements seen so far are at least as great; -inf while there are fewer
};

__device__ __forceinline__ bool better(float xa, int ia, float xb, int ib) { return xa > xb || (xa == xb && ia < ib); }

// Cuts the list's `n` entries (<= kCap, the same value in all threads) to the `count` best, in order.
__device__ __forceinline__ void prune(List& list, int n, int count) {
  constexpr int kMine = kCap / kThreads;
  float2 mine[kMine];
  int rank[kMine];
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int i = threadIdx.x + m * kThreads;
    rank[m] = kCap;
    if (i >= n) continue;
    mine[m] = list.e[i];
    int r = 0;
    for (int j = 0; j < n; ++j) {
      const float2 o = list.e[j];
      r += better(o.x, __float_as_int(o.y), mine[m].x, __float_as_int(mine[m].y));
    }
    rank[m] = r;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kMine; ++m)
    if (rank[m] < count) {
      list.e[rank[m]] = mine[m];
      if (rank[m] == count - 1) list.threshold = mine[m].x;
    }
  if (threadIdx.x == 0) {
    list.n = n < count ? n : count;
    if (n < count) list.threshold = -CUDART_INF_F;
  }
  __syncthreads();
}

__device__ __forceinline__ void append(List& list, float x, int token) {
  const int at = atomicAdd(&list.n, 1);
  if (at < kCap) list.e[at] = make_float2(x, __int_as_float(token));
}

__device__ __forceinline__ uint64_t entry_key(float x, int token) {
  return ((uint64_t)order_key(x) << 32) | (uint32_t)~token;
}

// A tile with more candidates than the list holds (many equal logits, rising ones): the `count`-th
// greatest of the list's first `have` entries and the tile, bit by bit, then what is not below it.
template <class Tl>
__device__ __noinline__ void select_exact(List& list, int have, int count, const Tl& tile, int64_t at, int* counters) {
  uint64_t cut = 0;
  if (threadIdx.x < 2) counters[threadIdx.x] = 0;
  __syncthreads();
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t trial = cut | (1ull << bit);
    int n = 0;
    for (int i = threadIdx.x; i < have; i += kThreads)
      n += entry_key(list.e[i].x, __float_as_int(list.e[i].y)) >= trial;
    for (int e = 0; e < Tl::kElems; ++e) {
      const float x = tile.value(e);
      n += x > -CUDART_INF_F && entry_key(x, (int)at + Tl::index(e)) >= trial;
    }
    n = __reduce_add_sync(~0u, n);
    int* c = counters + (bit & 1);
    if ((threadIdx.x & 31) == 0 && n > 0) atomicAdd(c, n);
    __syncthreads();
    if (*c >= count) cut = trial;
    if (threadIdx.x == 0) counters[(bit & 1) ^ 1] = 0;
    __syncthreads();
  }
  float2 kept[kCap / kThreads];
  bool keep[kCap / kThreads];
#pragma unroll
  for (int m = 0; m < kCap / kThreads; ++m) {
    const int i = threadIdx.x + m * kThreads;
    keep[m] = i < have;
    if (keep[m]) kept[m] = list.e[i];
    keep[m] = keep[m] && entry_key(kept[m].x, __float_as_int(kept[m].y)) >= cut;
  }
  __syncthreads();
  if (threadIdx.x == 0) list.n = 0;
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kCap / kThreads; ++m)
    if (keep[m]) append(list, kept[m].x, __float_as_int(kept[m].y));
  for (int e = 0; e < Tl::kElems; ++e) {
    const float x = tile.value(e);
    const int token = (int)at + Tl::index(e);
    if (x > -CUDART_INF_F && entry_key(x, token) >= cut) append(list, x, token);
  }
  __syncthreads();
}

// A beam that has candidates of its own logits: not finished, its score finite.
__device__ __forceinline__ bool beam_open(const SelectParams& p, int row) {
  return !(p.done != nullptr && p.done[row] != 0) && fabsf(p.scores[row]) < CUDART_INF_F;
}

template <class T, int kBytes>
__global__ void __launch_bounds__(kThreads) select_kernel(SelectParams p) {
  using Tl = Tile<T, kBytes>;
  __shared__ List list;
  __shared__ uint32_t warp_key[kWarps];
  __shared__ int counters[2];
  __shared__ float2 warp_sum[kWarps];
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    list.n = 0;
    list.threshold = -CUDART_INF_F;
  }
  grid_dependency_wait();
  if (!beam_open(p, row)) return;  // the merge does not look at its lists
  const typename T::Elem* x = static_cast<const typename T::Elem*>(p.logits) + row * p.row_stride;
  const int64_t begin = (int64_t)chunk * p.chunk_len;
  const int64_t end = begin + p.chunk_len < p.vocab ? begin + p.chunk_len : p.vocab;
  float ref = -CUDART_INF_F, sum = 0.0f;
  int have = 0;
  bool nan = false;
  Tl next;
  next.load(x, begin, end);
  for (int64_t at = begin; at < end; at += Tl::kSize) {
    const Tl tile = next;
    if (at + Tl::kSize < end) next.load(x, at + Tl::kSize, end);
    const float top = tile.max();  // NaN if the tile holds one
    nan |= top != top;
    float least;
    if (at == begin) {
      // The m-th greatest of each warp's thread maxima, m = ceil(count / 8): the least of them over
      // the 8 warps has `count` elements at or above it.
      uint32_t key = order_key(top), mth = 0;
      for (int m = (p.count + kWarps - 1) / kWarps; m > 0; --m) {
        mth = __reduce_max_sync(~0u, key);
        if (lane == __ffs(__ballot_sync(~0u, key == mth)) - 1) key = 0;
      }
      if (lane == 0) warp_key[warp] = mth;
      __syncthreads();
      mth = warp_key[0];
      for (int w = 1; w < kWarps; ++w) mth = min(mth, warp_key[w]);
      least = nextafterf(fmaxf(key_value(mth), -FLT_MAX), -CUDART_INF_F);
    } else {
      least = list.threshold;
    }
    bool pushed = false;
    if (top > least) {
#pragma unroll
      for (int e = 0; e < Tl::kElems; ++e) {
        const float v = tile.value(e);
        if (v > least) append(list, v, (int)at + Tl::index(e));
      }
      pushed = true;
    }
    if (top > ref + kStep) {
      sum *= exp2_fast((ref - top) * kLog2e);
      ref = top;
    }
    if (ref > -CUDART_INF_F) sum += tile.sum(ref);
    if (__syncthreads_or(pushed)) {
      int n = list.n;
      __syncthreads();
      if (n > kCap) {
        select_exact(list, have, p.count, tile, at, counters);
        n = list.n;
        __syncthreads();
      }
      if (at == begin || n > kPruneAt) {
        prune(list, n, p.count);
        n = n < p.count ? n : p.count;
      }
      have = n;
    }
  }
  if (have > 0) {
    prune(list, have, p.count);
    have = have < p.count ? have : p.count;
  }
  // threads' sums on one reference
  float top = ref;
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) warp_sum[warp].x = top;
  __syncthreads();
  top = warp_sum[0].x;
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_sum[w].x);
  sum = nan ? CUDART_NAN_F : ref > -CUDART_INF_F ? sum * exp2f((ref - top) * kLog2e) : 0.0f;
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) warp_sum[warp].y = sum;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) sum += warp_sum[w].y;
    p.sums[blockIdx.x] = make_float2(top, sum);
  }
  float2* out = p.entries + (int64_t)blockIdx.x * p.count;
  for (int i = tid; i < p.count; i += kThreads)
    out[i] = i < have ? list.e[i] : make_float2(-CUDART_INF_F, __int_as_float(-1));
}

constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double key_value64(uint64_t k) {
  return __longlong_as_double((long long)(k >> 63 ? k ^ (1ull << 63) : ~k));
}

// One CTA a group of beams: log-sum-exp of each beam in 64 bits, then `count` times the best head of
// the sorted lists.
__global__ void __launch_bounds__(kMergeThreads) select_merge_kernel(SelectParams p) {
  extern __shared__ float2 entry[];  // [beams * chunks][count]
  // A candidate's score is offset + (logit - greatest): next to a logit of 1e38 a logarithm would be lost.
  __shared__ double offset[kMaxBeams];  // score - log(sum exp(logit - greatest)), or a finished beam's score
  __shared__ float greatest[kMaxBeams];
  __shared__ int kind[kMaxBeams];       // 0: no candidates, 1: those of its lists, 2: finished
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lists = p.beams * p.chunks;
  grid_dependency_wait();
  const float2* src = p.entries + (int64_t)group * lists * p.count;
  for (int i = tid; i < lists * p.count; i += kMergeThreads) {
    const int row = group * p.beams + i / (p.count * p.chunks);
    entry[i] = beam_open(p, row) ? src[i] : make_float2(-CUDART_INF_F, __int_as_float(-1));
  }
  for (int k = warp; k < p.beams; k += kMergeWarps) {
    const int row = group * p.beams + k;
    const float score = p.scores[row];
    int what = 0;
    double off = 0.0;
    float high = 0.0f;
    if (!(score < CUDART_INF_F)) {  // NaN, +inf
      if (lane == 0) flag_error(p.status, KVARN_DEV_BAD_LOGITS);
    } else if (score > -CUDART_INF_F && p.done != nullptr && p.done[row] != 0) {
      what = 2;
      off = score;
    } else if (score > -CUDART_INF_F) {
      const float2* s = p.sums + (int64_t)row * p.chunks;
      float top = -CUDART_INF_F;
      bool bad = false;
      for (int c = lane; c < p.chunks; c += 32) {
        const float2 v = s[c];
        top = fmaxf(top, v.x);
        bad |= !(v.y < CUDART_INF_F);
      }
      for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      bad = __any_sync(~0u, bad);
      if (bad) {
        if (lane == 0) flag_error(p.status, KVARN_DEV_BAD_LOGITS);
      } else if (top > -CUDART_INF_F) {
        double sum = 0.0;
        for (int c = lane; c < p.chunks; c += 32) {
          const float2 v = s[c];
          if (v.x > -CUDART_INF_F) sum += v.x == top ? (double)v.y : (double)v.y * exp((double)v.x - (double)top);
        }
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
        what = 1;
        off = (double)score - log(sum);
        high = top;
      }
    }
    if (lane == 0) {
      offset[k] = off;
      greatest[k] = high;
      kind[k] = what;
    }
  }
  __syncthreads();
  if (warp != 0) return;

  // Lane l keeps the heads of lists l, l + 32, ...: next[] counts what was taken of each.
  extern __shared__ float2 dynamic[];
  int* next = reinterpret_cast<int*>(dynamic + lists * p.count);
  for (int i = lane; i < lists; i += 32) next[i] = 0;
  __syncwarp();
  uint64_t best = 0;
  uint32_t best_at = ~0u;  // beam * vocab + token
  int best_list = 0;
  const auto scan = [&]() {
    best = 0, best_at = ~0u;
    for (int i = lane; i < lists; i += 32) {
      const int k = i / p.chunks, n = next[i];
      if (kind[k] == 0 || n >= p.count) continue;
      uint64_t key;
      uint32_t at;
      if (kind[k] == 2) {
        if (i != k * p.chunks || n > 0) continue;  // one candidate, in the first list
        key = order_key(offset[k]);
        at = (uint32_t)k * p.vocab + p.end_token;
      } else {
        const float2 e = entry[i * p.count + n];
        if (__float_as_int(e.y) < 0) continue;
        key = order_key(offset[k] + ((double)e.x - (double)greatest[k]));
        at = (uint32_t)k * p.vocab + __float_as_int(e.y);
      }
      if (key > best || (key == best && at < best_at)) best = key, best_at = at, best_list = i;
    }
  };
  scan();
  for (int j = 0; j < p.count; ++j) {
    const uint32_t hi = __reduce_max_sync(~0u, (uint32_t)(best >> 32));
    const bool in = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(~0u, in ? (uint32_t)best : 0u);
    const uint32_t at = __reduce_min_sync(~0u, in && (uint32_t)best == lo ? best_at : ~0u);
    const uint64_t key = ((uint64_t)hi << 32) | lo;
    const int64_t o = (int64_t)group * p.count + j;
    const bool found = at != ~0u;
    if (lane == 0) {
      const int k = found ? (int)(at / (uint32_t)p.vocab) : -1, token = found ? (int)(at - (uint32_t)k * p.vocab) : -1;
      p.out_scores[o] = found ? (float)key_value64(key) : -CUDART_INF_F;
      p.out_parents[o] = k;
      p.out_tokens[o] = token;
      if (p.out_done != nullptr) p.out_done[o] = found && (kind[k] == 2 || token == p.end_token);
    }
    if (found && best_at == at) {
      ++next[best_list];
      scan();
    }
  }
}

// Chunks of a row: enough CTAs to fill the GPU when the rows are few, each of some thousand logits at
// least, and no more lists than the merge holds.
static int chunks_of(int64_t rows, int beams, int vocab, int count) {
  int64_t c = (608 + rows - 1) / rows;
  const int64_t most = (vocab + 2047) / 2048, held = kMergeEntries / ((int64_t)beams * count);
  c = c < most ? c : most;
  c = c < held ? c : held;
  return c < 1 ? 1 : (int)c;
}
// Logits of a chunk: a multiple of 2048, so that all but the last end on a whole load.
static int chunk_len_of(int vocab, int chunks) { return (((vocab + chunks - 1) / chunks + 2047) / 2048) * 2048; }

struct SelectLayout {
  int chunks, chunk_len;
  size_t sum_bytes, entry_bytes;
};
static SelectLayout select_layout(int batch, int beams, int vocab, int count) {
  SelectLayout L;
  const int64_t rows = (int64_t)batch * beams;
  const int want = chunks_of(rows, beams, vocab, count);
  L.chunk_len = chunk_len_of(vocab, want);
  L.chunks = (vocab + L.chunk_len - 1) / L.chunk_len;
  L.sum_bytes = ((size_t)rows * L.chunks * sizeof(float2) + 15) / 16 * 16;
  L.entry_bytes = ((size_t)rows * L.chunks * count * sizeof(float2) + 15) / 16 * 16;
  return L;
}

static int select_shape_check(int batch, int beams, int vocab, int count) {
  if (batch < 0 || beams < 1 || vocab < 1 || count < 1) return KVARN_ERR_INVALID_ARG;
  if (beams > kMaxBeams || count > kMaxCount || vocab > kMaxVocab || batch > (1 << 20)) return KVARN_ERR_UNSUPPORTED;
  return KVARN_OK;
}

static cudaLaunchConfig_t config(unsigned grid, unsigned block, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <class T, int kBytes>
static int launch_select(const SelectParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config((unsigned)(p.batch * p.beams * (int64_t)p.chunks), kThreads, 0, stream, &attr);
  return cudaLaunchKernelEx(&cfg, select_kernel<T, kBytes>, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

// ---- reorder ----------------------------------------------------------------------------------

struct ReorderParams {
  const int32_t* parents;
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  const int32_t* table;
  int32_t* table_out;
  const __half* k;
  const __half* v;
  __half* k_out;
  __half* v_out;
  int32_t* status;
  int batch, beams, max_pages, layers, num_kv_heads, dim;
  int slices;  // CTAs of the rows of one (layer, K or V, group, kv head)
};

constexpr int kMoveThreads = 256;

// Every 16-byte vector of the open tiles, and every table entry, is moved for all beams of a group by
// one thread, which reads them all before it writes: the outputs may be the inputs' own buffers.
template <int kBeams>
__global__ void __launch_bounds__(kMoveThreads) reorder_kernel(ReorderParams p) {
  __shared__ int parent[kMaxBeams], length[kMaxBeams];
  const int tid = threadIdx.x;
  const int64_t unit = blockIdx.x;  // (group, kv head, slice)
  const int slice = (int)(unit % p.slices);
  const int head = (int)(unit / p.slices % p.num_kv_heads);
  const int group = (int)(unit / p.slices / p.num_kv_heads);
  const int rows0 = group * p.beams;
  grid_dependency_wait();
  if (tid < p.beams) {
    int of = p.parents[rows0 + tid], n = 0, bad = 0;
    if (of < -1 || of >= p.beams) bad = KVARN_DEV_BAD_BEAM, of = -1;
    if (of >= 0) {
      n = p.seq_lens[rows0 + of];
      if (n < 0 || n / kTile > p.max_pages) bad = KVARN_DEV_SEQ_TOO_LONG;
    }
    parent[tid] = of;
    length[tid] = n;
    if (blockIdx.y == 0 && slice == 0 && head == 0) {
      p.seq_lens_out[rows0 + tid] = n;
      if (bad) flag_error(p.status, bad);
    }
  }
  __syncthreads();
  if (blockIdx.y == 0) {
    // lengths and table rows
    const int step = p.slices * p.num_kv_heads * kMoveThreads;
    for (int64_t i = (int64_t)(head * p.slices + slice) * kMoveThreads + tid; i < p.max_pages; i += step) {
      int32_t x[kBeams];
#pragma unroll
      for (int b = 0; b < kBeams; ++b)
        if (b < p.beams && i < length[b] / kTile) x[b] = p.table[(int64_t)(rows0 + parent[b]) * p.max_pages + i];
#pragma unroll
      for (int b = 0; b < kBeams; ++b)
        if (b < p.beams && i < length[b] / kTile) p.table_out[(int64_t)(rows0 + b) * p.max_pages + i] = x[b];
    }
    return;
  }
  const int layer = (blockIdx.y - 1) >> 1, kv = (blockIdx.y - 1) & 1;
  const int vecs = p.dim / 8;
  const uint4* src = reinterpret_cast<const uint4*>(kv ? p.v : p.k);
  uint4* dst = reinterpret_cast<uint4*>(kv ? p.v_out : p.k_out);
  const int64_t seq = (int64_t)p.num_kv_heads * kTile * vecs;  // vectors of one sequence in one layer
  const int64_t first = (int64_t)layer * p.batch * p.beams * seq + (int64_t)rows0 * seq + (int64_t)head * kTile * vecs;
  const bool in_place = src == dst;
  for (int i = slice * kMoveThreads + tid; i < kTile * vecs; i += p.slices * kMoveThreads) {
    const int row = i / vecs;
    uint4 x[kBeams];
#pragma unroll
    for (int b = 0; b < kBeams; ++b)
      if (b < p.beams && length[b] > 0 && row < length[b] % kTile && !(in_place && parent[b] == b))
        x[b] = src[first + parent[b] * seq + i];
#pragma unroll
    for (int b = 0; b < kBeams; ++b)
      if (b < p.beams && length[b] > 0 && row < length[b] % kTile && !(in_place && parent[b] == b))
        dst[first + b * seq + i] = x[b];
  }
}

template <int kBeams>
static int launch_reorder(const ReorderParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config((unsigned)((int64_t)p.batch * p.num_kv_heads * p.slices), kMoveThreads, 0, stream, &attr);
  cfg.gridDim.y = 2 * p.layers + 1;
  return cudaLaunchKernelEx(&cfg, reorder_kernel<kBeams>, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace beam
}  // namespace kvarn

using namespace kvarn;
using namespace kvarn::beam;

extern "C" {

size_t kvarn_beam_select_workspace_bytes(int batch, int beams, int vocab, int count) {
  if (select_shape_check(batch, beams, vocab, count) != KVARN_OK || batch == 0) return 0;
  const SelectLayout L = select_layout(batch, beams, vocab, count);
  return L.sum_bytes + L.entry_bytes;
}

int kvarn_beam_select(int batch, int beams, int vocab, int count, const void* logits, int logits_type, int64_t row_stride,
                      const float* scores, const uint8_t* done, int end_token, float* out_scores, int32_t* out_parents,
                      int32_t* out_tokens, uint8_t* out_done, void* workspace, size_t workspace_bytes,
                      int32_t* dev_status, void* stream) {
  if (const int st = select_shape_check(batch, beams, vocab, count); st != KVARN_OK) return st;
  if (logits_type != KVARN_LOGITS_F16 && logits_type != KVARN_LOGITS_BF16 && logits_type != KVARN_LOGITS_F32)
    return KVARN_ERR_UNSUPPORTED;
  if (batch == 0) return KVARN_OK;
  if (logits == nullptr || scores == nullptr || out_scores == nullptr || out_parents == nullptr ||
      out_tokens == nullptr || workspace == nullptr)
    return KVARN_ERR_INVALID_ARG;
  if (end_token < -1 || end_token >= vocab || (done != nullptr && end_token < 0)) return KVARN_ERR_INVALID_ARG;
  const int size = logits_type == KVARN_LOGITS_F32 ? 4 : 2;
  const uintptr_t base = reinterpret_cast<uintptr_t>(logits);
  if (row_stride < vocab || base % size != 0 || !beam::aligned16(workspace)) return KVARN_ERR_INVALID_ARG;
  const SelectLayout L = select_layout(batch, beams, vocab, count);
  if (workspace_bytes < L.sum_bytes + L.entry_bytes) return KVARN_ERR_WORKSPACE_TOO_SMALL;
  if ((int64_t)batch * beams * L.chunks > 0x7fffffffLL) return KVARN_ERR_UNSUPPORTED;
  SelectParams p{};
  p.logits = logits;
  p.row_stride = row_stride;
  p.scores = scores;
  p.done = done;
  p.sums = static_cast<float2*>(workspace);
  p.entries = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + L.sum_bytes);
  p.out_scores = out_scores;
  p.out_parents = out_parents;
  p.out_tokens = out_tokens;
  p.out_done = out_done;
  p.status = dev_status;
  p.batch = batch;
  p.beams = beams;
  p.vocab = vocab;
  p.count = count;
  p.end_token = end_token;
  p.chunks = L.chunks;
  p.chunk_len = L.chunk_len;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the widest load that every row's start is aligned to
  const uint64_t both = (uint64_t)base | ((uint64_t)row_stride * size);
  int st;
  if (logits_type == KVARN_LOGITS_F32)
    st = both % 16 == 0 ? launch_select<F32, 16>(p, s) : launch_select<F32, 4>(p, s);
  else if (logits_type == KVARN_LOGITS_BF16)
    st = both % 16 == 0 ? launch_select<BF16, 16>(p, s) : both % 4 == 0 ? launch_select<BF16, 4>(p, s) : launch_select<BF16, 2>(p, s);
  else
    st = both % 16 == 0 ? launch_select<F16, 16>(p, s) : both % 4 == 0 ? launch_select<F16, 4>(p, s) : launch_select<F16, 2>(p, s);
  if (st != KVARN_OK) return st;
  const int lists = beams * L.chunks;
  static PerDeviceOnce smem_once;
  const int most = kMergeEntries * (int)sizeof(float2) + kMergeEntries * 4;
  if (const int e = set_smem_limit(smem_once, reinterpret_cast<const void*>(select_merge_kernel), most); e != KVARN_OK) return e;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      config((unsigned)batch, kMergeThreads, (size_t)lists * count * sizeof(float2) + (size_t)lists * 4, s, &attr);
  return cudaLaunchKernelEx(&cfg, select_merge_kernel, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

int kvarn_beam_reorder(const kvarn_desc* desc, int batch, int beams, int layers, const int32_t* parents,
                       const int32_t* seq_lens, int32_t* seq_lens_out, const int32_t* block_table,
                       int32_t* block_table_out, int max_pages, const void* partial_k, const void* partial_v,
                       void* partial_k_out, void* partial_v_out, int32_t* dev_status, void* stream) {
  if (const int st = desc_check(desc); st != KVARN_OK) return st;
  if (batch < 0 || beams < 1 || layers < 0 || max_pages < 1) return KVARN_ERR_INVALID_ARG;
  if (beams > kMaxBeams || layers > 16383 || max_pages > (1 << 23) || (int64_t)batch * beams > (1 << 24))
    return KVARN_ERR_UNSUPPORTED;
  if (batch == 0) return KVARN_OK;
  if (parents == nullptr || seq_lens == nullptr || seq_lens_out == nullptr || seq_lens_out == seq_lens ||
      block_table == nullptr || block_table_out == nullptr)
    return KVARN_ERR_INVALID_ARG;
  if (layers > 0 && (partial_k == nullptr || partial_v == nullptr || partial_k_out == nullptr || partial_v_out == nullptr))
    return KVARN_ERR_INVALID_ARG;
  if (!beam::aligned16(partial_k) || !beam::aligned16(partial_v) || !beam::aligned16(partial_k_out) || !beam::aligned16(partial_v_out))
    return KVARN_ERR_INVALID_ARG;
  ReorderParams p{};
  p.parents = parents;
  p.seq_lens = seq_lens;
  p.seq_lens_out = seq_lens_out;
  p.table = block_table;
  p.table_out = block_table_out;
  p.k = static_cast<const __half*>(partial_k);
  p.v = static_cast<const __half*>(partial_v);
  p.k_out = static_cast<__half*>(partial_k_out);
  p.v_out = static_cast<__half*>(partial_v_out);
  p.status = dev_status;
  p.batch = batch;
  p.beams = beams;
  p.max_pages = max_pages;
  p.layers = layers;
  p.num_kv_heads = desc->num_kv_heads;
  p.dim = desc->head_dim;
  p.slices = 4;
  if ((int64_t)batch * p.num_kv_heads * p.slices > 0x7fffffffLL) return KVARN_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (beams <= 4) return launch_reorder<4>(p, s);
  if (beams <= 8) return launch_reorder<8>(p, s);
  if (beams <= 16) return launch_reorder<16>(p, s);
  return launch_reorder<32>(p, s);
}

}  // extern "C"
