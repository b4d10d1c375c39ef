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
constexpr int kChunkEntries = 1024;    // candidates beyond which a group's rows are not divided further
static_assert(kChunkEntries <= kMaxBeams * kMaxCount && kMaxBeams * kMaxCount * 12 + 16384 <= 49152,
              "the merge takes its lists without a raised limit");

// ---- selection: one pass over the logits ----------------------------------------------------
// A row of logits (one beam) is cut into chunks, one CTA each.  A CTA streams its chunk through shared
// memory; a thread keeps its sum of exp(x - ref) in 32 bits and notes the greatest of every 32 elements.
// Then a bound is taken from these, below which none of the chunk's `count` best can be, and the few runs of
// 32 whose greatest reaches it are read again: what reaches the bound goes into a short list, which is cut
// to the `count` best.  The merge joins the chunks' sums and takes the best candidates of the lists.
//
// The logits are read once (the runs again, 64 bytes each, a few per chunk): 64 groups of 8 beams over 151936 logits of
// 16 bits, 156 MB, take 38 us.  A kernel that only reads them takes 23.5 us; the stream ends after 23 us on SMs with
// three CTAs, after up to 28 us on those with four, the end of the chunks takes 5 us, the merge 3.5 us.  While a CTA
// met at every tile to keep a list in order it took 93 us, with lists kept by appending 57 us: the threads now meet only
// after the stream.  Chunks cut so that every SM has the same share (a CTA then ends two of them) gained 4 us there and
// lost up to half elsewhere.

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kResident = 4;          // CTAs of the streaming kernel on an SM
constexpr int kWords = 8;              // 32-bit words of a tile that a thread holds
constexpr int kStages = 3;            // tiles on their way
constexpr int kCap = 512;              // entries of the list
// References stay within it where sums are kept by their products with log2(e): farther out the rounding of the
// product passes 0.004.  A warp whose logits are all below -kFar (a mask of finite values) keeps -kFar, against which
// they count as next to nothing; with the mask's own value the product overflows.  A chunk that ends with a reference
// of kFar or more, or of -kFar, takes the slower path.
constexpr float kFar = 65536.0f;
// A reference moves when a logit exceeds it by more: the greatest terms' arguments stay small, and with them
// their rounding (with 40 the logarithm of a sum was off by 3.1e-7 in the mean square, with 1 by 1.3e-7, by 7.6e-8 since
// tiles are added without an error, and by 7.5e-8 since a move is exact to a rounding of its factor).
constexpr float kStep = 1.0f;

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
  static __device__ __forceinline__ float one(Elem x) { return get(x).x; }
  static __device__ __forceinline__ Elem bits(float x) { return __half_as_ushort(__float2half_rn(x)); }  // x is an element
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
  static __device__ __forceinline__ float one(Elem x) { return get(x).x; }
  static __device__ __forceinline__ Elem bits(float x) { return (Elem)(__float_as_uint(x) >> 16); }
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
  static __device__ __forceinline__ float one(Elem x) { return __uint_as_float(x); }
  static __device__ __forceinline__ Elem bits(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sums and scores are pairs of floats (hi + lo, |lo| at most half a step of hi: 48 bits): 64-bit arithmetic
// runs at 1/64 of the 32-bit rate here and took two thirds of the merge's time.
struct Pair {
  float hi, lo;
};
// a + b without an error (Knuth); the intrinsics are never fused with a product before them
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  const Pair t = two_sum(a.lo, b.lo);
  s = two_sum(s.hi, s.lo + t.hi);
  return two_sum(s.hi, s.lo + t.lo);
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float h = a.hi * b.hi;
  return two_sum(h, fmaf(a.hi, b.hi, -h) + fmaf(a.hi, b.lo, a.lo * b.hi));
}
// exp(a - b), a <= b, the difference without an error: an error of its rounding would be the same for all that is
// joined at one step.  (With exp2f((a - b) * kLog2e) a peak 11.2 above 151935 equal logits was off by 5.5e-7.)
__device__ __forceinline__ float exp_difference(float a, float b) {
  const Pair d = two_sum(a, -b);
  const float e = expf(d.hi);
  return d.hi > -104.0f ? fmaf(e, d.lo, e) : 0.0f;
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
  static constexpr int kLoads = 4 * kWords / kBytes;
  static constexpr int kElems = 4 * kWords / (int)sizeof(typename T::Elem);
  static constexpr int kSize = kThreads * kElems;
  static constexpr int kRun = 32 / kElems;                            // tiles of a run of 32 elements
  // Runs of a thread that are noted at a time, 10 KB; a chunk with more ends a part more than once: 512 rows of 163840
  // 16-bit logits take 38.4 us, of 163848 45.0, of 200064 48.4; of 81920 32-bit ones 36.6, of 81928 40.0.
  static constexpr int kRuns = T::kPerWord == 1 ? 10 : 20;
  uint32_t w[kWords];

  // index within the tile of element e of this thread
  static __device__ __forceinline__ int index(int e) { return ((e / kPer) * kThreads + (int)threadIdx.x) * kPer + e % kPer; }

  __device__ __forceinline__ void load(const typename T::Elem* row, int at, int end) {
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
    // The row's last tile: loads past the end are moved back into the row, all of them under way at once, and
    // their elements replaced.
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int i = at + index(l * kPer);
      if constexpr (kBytes == 16) {
        uint4 x = make_uint4(T::kNone, T::kNone, T::kNone, T::kNone);
        if (i + kPer <= end) {
          x = __ldcs(reinterpret_cast<const uint4*>(row + i));
        } else if (i < end) {
          uint32_t v[4] = {T::kNone, T::kNone, T::kNone, T::kNone};
          typename T::Elem one[kPer];
#pragma unroll
          for (int e = 0; e < kPer; ++e) one[e] = row[::min(i + e, end - 1)];
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (i + e < end) put(v[e / T::kPerWord], e % T::kPerWord, one[e]);
          x = make_uint4(v[0], v[1], v[2], v[3]);
        }
        w[4 * l] = x.x, w[4 * l + 1] = x.y, w[4 * l + 2] = x.z, w[4 * l + 3] = x.w;
      } else if constexpr (kPer == 1) {
        const typename T::Elem x = row[::min(i, end - 1)];
        if constexpr (T::kPerWord == 1) {
          w[l] = i < end ? x : T::kNone;
        } else {
          const uint32_t v = i < end ? x : T::kNone & 0xffffu;
          if (l % 2 == 0) w[l / 2] = v;
          else w[l / 2] |= v << 16;
        }
      } else {  // two halves a word
        const uint32_t x = end >= 2 ? *reinterpret_cast<const uint32_t*>(row + ::min(i, (end & ~1) - 2)) : 0u;
        w[l] = i + 2 <= end ? x : T::kNone;
        if (i + 1 == end) put(w[l], 0, row[i]);
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
  // sum of exp(x - ref), in the order of the fast path's
  __device__ __forceinline__ float sum_of(float ref) const {
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < kElems; ++e) a[e % 4] += expf(value(e) - ref);
    return (a[0] + a[2]) + (a[1] + a[3]);
  }
};

struct List {
  float2 e[kCap];  // logit, token
  int n;
  float threshold;  // `count` elements seen so far are at least as great; -inf while there are fewer
  int far;          // a reference is kFar or more, or -kFar
};

// Tiles on their way through shared memory: a thread reads the words that it copied itself, so that it
// waits for its own copies only.  Word i of a thread lies in slot[i / 4][thread], part i % 4.
template <class T, int kBytes>
struct Ring {
  using Tl = Tile<T, kBytes>;
  uint4 slot[kStages][kWords / 4][kThreads];

  __device__ __forceinline__ void issue(int stage, const typename T::Elem* row, int at, int end) {
    if (at < end) {
      const uint32_t to = smem_u32(&slot[stage][0][threadIdx.x]);
      if (at + Tl::kSize <= end) {
        const char* src = reinterpret_cast<const char*>(row + at) + threadIdx.x * kBytes;
#pragma unroll
        for (int l = 0; l < Tl::kLoads; ++l) {
          const uint32_t dst = to + (kBytes == 16 ? l : l / 4) * kThreads * 16 + (kBytes == 16 ? 0 : l % 4 * 4);
          if constexpr (kBytes == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + l * kThreads * 16) : "memory");
          else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src + l * kThreads * 4) : "memory");
        }
      } else {
        Tl tile;
        tile.load(row, at, end);
        put(stage, tile);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void put(int stage, const Tl& tile) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      slot[stage][i][threadIdx.x] = make_uint4(tile.w[4 * i], tile.w[4 * i + 1], tile.w[4 * i + 2], tile.w[4 * i + 3]);
  }
  // the copies of all but the newest kStages - 1 tiles have arrived
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); }

  // element e of thread t
  __device__ __forceinline__ float value(int stage, int t, int e) const {
    const int i = e / T::kPerWord;
    const uint32_t w = reinterpret_cast<const uint32_t*>(&slot[stage][i / 4][t])[i % 4];
    if constexpr (T::kPerWord == 1) return __uint_as_float(w);
    else {
      const float2 f = T::get(w);
      return e % 2 == 0 ? f.x : f.y;
    }
  }
  __device__ __forceinline__ float top_of(uint32_t m) const {
    if constexpr (T::kPerWord == 1) return __uint_as_float(m);
    else {
      const float2 f = T::get(m);
      return max_nan(f.x, f.y);
    }
  }
  // The thread's sum of 2^(x log2(e) - base), log2(e) and the argument rounded to 32 bits, and its greatest x
  // (NaN if there is one).
  __device__ __forceinline__ float sum(int stage, float base, float& top) const {
    float2 a = make_float2(0.0f, 0.0f), b = a;
    const float2 r = make_float2(-base, -base), l = make_float2(kLog2e, kLog2e);
    const auto put = [&](float2& to, float2 x) {
      x = fma2(x, l, r);
      to = add2(to, make_float2(exp2_fast(x.x), exp2_fast(x.y)));
    };
    uint32_t m = T::kNone;
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = slot[stage][i][threadIdx.x];
      m = T::max(m, T::max(T::max(v.x, v.y), T::max(v.z, v.w)));
      if constexpr (T::kPerWord == 1) {
        put(a, make_float2(__uint_as_float(v.x), __uint_as_float(v.y)));
        put(b, make_float2(__uint_as_float(v.z), __uint_as_float(v.w)));
      } else {
        put(a, T::get(v.x));
        put(b, T::get(v.y));
        put(a, T::get(v.z));
        put(b, T::get(v.w));
      }
    }
    top = top_of(m);
    a = add2(a, b);
    return a.x + a.y;
  }
};

// Sum of exponentials of one thread: sum + rest = sum of 2^(x log2(e) - base) with base = ref log2(e) rounded.
// The tiles' sums are added without an error, so that a rounding is a share of one tile only.
struct Sum {
  float ref, base, sum, rest;
  __device__ __forceinline__ void start() { ref = -CUDART_INF_F, base = sum = rest = 0.0f; }
  __device__ __forceinline__ void add(float part) {
    const Pair s = two_sum(sum, part);
    sum = s.hi;
    rest += s.lo;
  }
  // Sum of exp(x - ref): what the rounding of base took, e^c with c = log(2) (base - ref log2(e)), is given back.
  // |ref| <= kFar: |c| < 0.005, so 1 + c + c^2/2 is off by less than 2^-25.
  __device__ __forceinline__ float of_ref() const {
    const float c = 0.6931472f * fmaf(-ref, kLog2e, base);
    return sum + fmaf(sum, fmaf(0.5f * c, c, c), rest);
  }
  // What is carried stays a sum of 2^(x log2(e) - base): it is multiplied by 2^(old base - new base), the difference
  // taken without an error, its whole part apart, the product kept with its rounding.
  __device__ __forceinline__ void move(float to) {
    const float next = __fmul_rn(to, kLog2e);
    const Pair d = two_sum(base, -next);
    const float n = rintf(d.hi);
    const bool carried = ref > -CUDART_INF_F && n >= -126.0f;
    const float by = carried ? expf(0.6931472f * ((d.hi - n) + d.lo)) * __int_as_float(((int)n + 127) << 23) : 0.0f;
    scale(by);
    ref = to;
    base = next;
  }
  // the product of 0 is 0: a sum against a reference within kFar is finite
  __device__ __forceinline__ void scale(float by) {
    const float s = sum * by;
    rest = fmaf(rest, by, fmaf(sum, by, -s));
    sum = s;
  }
};

// Without branches, as the ranks' loops want it.
__device__ __forceinline__ bool better(float xa, int ia, float xb, int ib) {
  return (xa > xb) | ((xa == xb) & (ia < ib));
}

// Entries of the list that are better than one of them; a warp counts together.
__device__ __forceinline__ int rank_of(const List& list, int n, float2 e) {
  int r = 0;
  for (int j = threadIdx.x & 31; j < n; j += 32) {
    const float2 o = list.e[j];
    r += better(o.x, __float_as_int(o.y), e.x, __float_as_int(e.y));
  }
  return __reduce_add_sync(~0u, r);
}
// Cuts the list's `n` entries (<= kCap, the same value in all threads) to the `count` best, in order.
__device__ __forceinline__ void prune(List& list, int n, int count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kCap <= 64 * kWarps, "a warp's entries, two a lane");
  float2 first = {}, second = {};
  int to_first = -1, to_second = -1, kept = 0;
  for (int i = warp; i < n; i += kWarps, ++kept) {
    const float2 e = list.e[i];
    const int r = rank_of(list, n, e), to = r < count ? r : -1;
    if (kept == lane) first = e, to_first = to;
    if (kept == lane + 32) second = e, to_second = to;
  }
  __syncthreads();
  const auto place = [&](float2 e, int to) {
    if (to < 0) return;
    list.e[to] = e;
    if (to == count - 1) list.threshold = e.x;
  };
  place(first, to_first);
  place(second, to_second);
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
__device__ __forceinline__ void select_exact(List& list, int have, int count, const Tl& tile, int at, int* counters) {
  uint64_t cut = 0;
  if (threadIdx.x < 2) counters[threadIdx.x] = 0;
  __syncthreads();
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t trial = cut | (1ull << bit);
    int n = 0;
    for (int i = threadIdx.x; i < have; i += kThreads)
      n += entry_key(list.e[i].x, __float_as_int(list.e[i].y)) >= trial;
#pragma unroll
    for (int e = 0; e < Tl::kElems; ++e) {
      const float x = tile.value(e);
      n += x > -CUDART_INF_F && entry_key(x, at + Tl::index(e)) >= trial;
    }
    n = __reduce_add_sync(~0u, n);
    int* c = counters + (bit & 1);
    if ((threadIdx.x & 31) == 0 && n > 0) atomicAdd(c, n);
    __syncthreads();
    const int found = *c;
    if (found >= count) cut = trial;
    if (found == count) break;
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
#pragma unroll
  for (int e = 0; e < Tl::kElems; ++e) {
    const float x = tile.value(e);
    const int token = at + Tl::index(e);
    if (x > -CUDART_INF_F && entry_key(x, token) >= cut) append(list, x, token);
  }
  __syncthreads();
}

// The rest of a chunk, from `at` on, where more of it reached the bound than the list holds or a reference is beyond
// kFar: tile by tile, references a thread's own.  sum.sum + sum.rest is the sum of exp(x - sum.ref) here, tiles added
// without an error (with plain additions 2^20 logits 17 below 4096 others were off by 1e-5).  Returns whether a logit
// was NaN or +inf.
template <class Tl, class Elem>
__device__ __noinline__ bool select_slow(List& list, int have, int count, const Elem* row, int at, int end,
                                         Sum& sum, int* counters) {
  bool bad = false;
  if (threadIdx.x == 0) list.n = have;
  __syncthreads();
  for (; at < end; at += Tl::kSize) {
    Tl tile;
    tile.load(row, at, end);
    const float top = tile.max(), least = list.threshold;
    bad |= !(top < CUDART_INF_F);
    if (top > least) {
#pragma unroll
      for (int e = 0; e < Tl::kElems; ++e)
        if (tile.value(e) > least) append(list, tile.value(e), at + Tl::index(e));
    }
    if (top > sum.ref + kStep) {
      sum.scale(exp_difference(sum.ref, top));
      sum.ref = top;
    }
    if (sum.ref > -CUDART_INF_F) sum.add(tile.sum_of(sum.ref));
    __syncthreads();
    int n = list.n;
    __syncthreads();
    if (n > kCap) {
      select_exact(list, have, count, tile, at, counters);
      n = count;
    }
    if (n > have) {
      prune(list, n, count);
      n = n < count ? n : count;
    }
    have = n;
  }
  return bad;
}

// Keys that come before number i of them, whose value is `mine`.
__device__ __forceinline__ int rank_of_key(const uint32_t* keys, int n, uint32_t mine, int i) {
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const uint32_t k = keys[j];
    rank += (k > mine) | ((k == mine) & (j < i));
  }
  return rank;
}

template <class T, int kBytes>
__global__ void __launch_bounds__(kThreads, kResident) select_kernel(SelectParams p) {
  using Tl = Tile<T, kBytes>;
  extern __shared__ __align__(16) uint8_t dynamic_smem[];
  Ring<T, kBytes>& ring = *reinterpret_cast<Ring<T, kBytes>*>(dynamic_smem);
  __shared__ typename T::Elem noted[Tl::kRuns][kThreads];
  __shared__ List list;
  __shared__ int runs[kCap];  // runs to read again: number x kThreads + thread
  __shared__ int num_runs;
  __shared__ uint32_t keys[kThreads], bound;
  __shared__ int counters[2];
  __shared__ float2 warp_sum[kWarps];
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    list.n = 0;
    list.threshold = -CUDART_INF_F;
    list.far = 0;
    num_runs = 0;
  }
  grid_dependency_wait();
  const float score = p.scores[row];
  const int finished = p.done != nullptr ? p.done[row] : 0;
  const typename T::Elem* x = static_cast<const typename T::Elem*>(p.logits) + row * p.row_stride;
  const int begin = chunk * p.chunk_len;
  const int end = min(begin + p.chunk_len, p.vocab);
  __syncthreads();  // the list is empty
  Sum sum;
  sum.start();
  int have = 0;
  bool nan = false;
  Tl next;  // rows aligned to 2 bytes: a tile in registers before it goes to the ring
  if constexpr (kBytes == 2) {
    next.load(x, begin, end);
  } else {
    for (int i = 0; i < kStages - 1; ++i) ring.issue(i, x, begin + i * Tl::kSize, end);
  }
  if (finished != 0 || !(fabsf(score) < CUDART_INF_F)) {  // no candidates of its logits: the merge does not look here
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  // the warp's sums on the greatest of its references
  const auto warp_total = [&](float ref, float total) {
    const float top = key_value(__reduce_max_sync(~0u, order_key(ref)));
    total = nan ? CUDART_NAN_F : ref > -CUDART_INF_F ? total * exp_difference(ref, top) : 0.0f;
    for (int d = 16; d > 0; d /= 2) total += __shfl_xor_sync(~0u, total, d);
    if (lane == 0) warp_sum[warp] = make_float2(top, total);
  };
  float2* out = p.entries + (int64_t)blockIdx.x * p.count;
  // the chunk's sum, and the rest of its list after the n best
  const auto finish = [&](int n) {
    for (int i = n + tid; i < p.count; i += kThreads) out[i] = make_float2(-CUDART_INF_F, __int_as_float(-1));
    if (warp != 0) return;
    const float2 v = lane < kWarps ? warp_sum[lane] : make_float2(-CUDART_INF_F, 0.0f);
    const float top = key_value(__reduce_max_sync(~0u, order_key(v.x)));
    Pair total = {v.x > -CUDART_INF_F || v.y != v.y ? v.x == top ? v.y : v.y * exp_difference(v.x, top) : 0.0f, 0.0f};
    for (int d = kWarps / 2; d > 0; d /= 2)
      total = add(total, {__shfl_xor_sync(~0u, total.hi, d), __shfl_xor_sync(~0u, total.lo, d)});
    if (lane == 0) p.sums[blockIdx.x] = make_float2(top, total.hi);
  };
  // One part for chunks of up to 20 x 8192 elements (fp32: 10 x 8192), which is nearly all of them.
  int at = begin, stage = 0;
  while (at < end) {
    const int part = at, part_end = min(at + Tl::kRuns * Tl::kRun * Tl::kSize, end);
    const Sum before = sum;
    float most = -CUDART_INF_F, run_top = -CUDART_INF_F;
    for (int t = 0; at < part_end; at += Tl::kSize, ++t, stage = stage == kStages - 1 ? 0 : stage + 1) {
      if constexpr (kBytes == 2) {
        ring.put(stage, next);
        if (at + Tl::kSize < end) next.load(x, at + Tl::kSize, end);
      } else {
        ring.issue(stage == 0 ? kStages - 1 : stage - 1, x, at + (kStages - 1) * Tl::kSize, end);
        ring.wait();
      }
      float top;
      float part_sum = ring.sum(stage, sum.base, top);
      if (__any_sync(~0u, top > sum.ref + kStep)) {  // also in the warp's first tile; its lanes have one reference
        const float to = key_value(__reduce_max_sync(~0u, order_key(top == top ? top : -CUDART_INF_F)));
        sum.move(fmaxf(to, -kFar));
        part_sum = ring.sum(stage, sum.base, top);
      }
      sum.add(part_sum);
      nan |= top != top;
      run_top = t % Tl::kRun == 0 ? top : fmaxf(run_top, top);
      noted[t / Tl::kRun][tid] = T::bits(run_top);
      most = fmaxf(most, top);
    }
    // The bound: the `take` greatest of the lanes' greatest ones of each warp (whose lanes all hold elements)
    // are put together, and of these the count-th is taken.  At least `count` elements are not below it, and
    // with twice as many taken as wanted it is most often the exact count-th of the threads' greatest.
    const int full = min(kWarps, (part_end - part) / (32 * Tl::kPer));
    const int take = full > 0 ? min(32, (2 * p.count + full - 1) / full) : 0, pool = full * take;
    uint32_t key = order_key(most);
    for (int m = 0; m < take; ++m) {
      const uint32_t mth = __reduce_max_sync(~0u, key);
      if (lane == __ffs(__ballot_sync(~0u, key == mth)) - 1) {
        if (warp < full) keys[warp * take + m] = mth;
        key = 0;
      }
    }
    if (fabsf(sum.ref) >= kFar && sum.ref > -CUDART_INF_F) list.far = 1;
    if (part_end == end) warp_total(sum.ref, sum.ref > -CUDART_INF_F ? sum.of_ref() : 0.0f);
    __syncthreads();
    float least = list.threshold;
    if (pool >= p.count) {
      if (tid < pool && rank_of_key(keys, pool, keys[tid], tid) == p.count - 1) bound = keys[tid];
      __syncthreads();
      least = fmaxf(least, nextafterf(fmaxf(key_value(bound), -FLT_MAX), -CUDART_INF_F));
    }
    const int tiles = (part_end - part + Tl::kSize - 1) / Tl::kSize, num_noted = (tiles + Tl::kRun - 1) / Tl::kRun;
    for (uint32_t lanes = __ballot_sync(~0u, most > least); lanes != 0; lanes &= lanes - 1) {
      const int thread = warp * 32 + __ffs(lanes) - 1;
      if (lane < num_noted && T::one(noted[lane][thread]) > least) {
        const int i = atomicAdd(&num_runs, 1);
        if (i < kCap) runs[i] = lane * kThreads + thread;
      }
    }
    __syncthreads();
    const int again = num_runs;
    bool slow = again > kCap || list.far != 0;
    if (!slow) {
      // element i of the runs: its token, where it is in the ring
      struct Place {
        int token, thread, tile, e;
      };
      const auto place = [&](int i) {
        const int r = runs[i / 32], thread = r % kThreads, e = i % Tl::kElems;
        const int t = r / kThreads * Tl::kRun + i % 32 / Tl::kElems;
        return Place{part + t * Tl::kSize + ((e / Tl::kPer) * kThreads + thread) * Tl::kPer + e % Tl::kPer, thread, t, e};
      };
      if (part_end == end && tiles <= kStages) {  // the whole part is still in the ring
        for (int i = tid; i < again * 32; i += kThreads) {
          const Place at_i = place(i);
          const int back = tiles - at_i.tile;
          if (back <= 0) continue;
          const float v = ring.value(stage - back + (stage < back ? kStages : 0), at_i.thread, at_i.e);
          if (v > least) append(list, v, at_i.token);
        }
      } else {
        constexpr int kAtOnce = 4;  // loads under way
        for (int i0 = tid; i0 < again * 32; i0 += kAtOnce * kThreads) {
          float v[kAtOnce];
          int token[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const int i = i0 + j * kThreads;
            token[j] = i < again * 32 ? place(i).token : part_end;
            v[j] = token[j] < part_end ? T::one(x[token[j]]) : -CUDART_INF_F;
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
            if (v[j] > least) append(list, v[j], token[j]);
        }
      }
    }
    __syncthreads();
    const int n = list.n;
    slow = slow || n > kCap;
    if (slow) {
      __syncthreads();
      sum = before;
      at = part;
      break;
    }
    if (part_end == end) {
      grid_launch_dependents();
      for (int i = warp; i < n; i += kWarps) {
        const float2 e = list.e[i];
        const int r = rank_of(list, n, e);
        if (lane == 0 && r < p.count) out[r] = e;
      }
      finish(n);
      return;
    }
    if (tid == 0) num_runs = 0;
    __syncthreads();
    prune(list, n, p.count);
    have = n < p.count ? n : p.count;
  }
  // the slow path, for the rest of the chunk
  asm volatile("cp.async.wait_all;" ::: "memory");
  sum.sum = sum.ref > -CUDART_INF_F ? sum.of_ref() : 0.0f;
  sum.rest = 0.0f;
  nan |= select_slow<Tl>(list, have, p.count, x, at, end, sum, counters);
  grid_launch_dependents();
  warp_total(sum.ref, sum.sum + sum.rest);
  __syncthreads();
  const int n = list.n;
  for (int i = tid; i < n; i += kThreads) out[i] = list.e[i];
  finish(n);
}

// ---- the merge --------------------------------------------------------------------------------
// exp(d) for -80 <= d.hi <= 80 to 2^-27: d = k log 2 + r, 1 + r exactly, r^2/2 + ... as Taylor's series to the ninth power in
// 32 bits (at most 0.07, so its rounding is 2^-28 of the result).  log 2 = 2839/4096 + 3.19461849e-5: k times
// the first part is exact.
__device__ __forceinline__ Pair exp_pair(Pair d) {
  const float k = rintf(d.hi * kLog2e);
  const float r = fmaf(k, -2839.0f / 4096.0f, d.hi);
  const Pair x = two_sum(r, fmaf(k, -3.194618494530941e-5f, d.lo));
  float q = 1.0f / 362880.0f;
  q = fmaf(q, x.hi, 1.0f / 40320.0f);
  q = fmaf(q, x.hi, 1.0f / 5040.0f);
  q = fmaf(q, x.hi, 1.0f / 720.0f);
  q = fmaf(q, x.hi, 1.0f / 120.0f);
  q = fmaf(q, x.hi, 1.0f / 24.0f);
  q = fmaf(q, x.hi, 1.0f / 6.0f);
  q = fmaf(q, x.hi, 0.5f);
  const Pair s = two_sum(1.0f, x.hi);
  const float rest = s.lo + fmaf(x.hi * x.hi, q, x.lo * s.hi);
  const Pair e = two_sum(s.hi, rest);
  const float scale = __int_as_float(((int)k + 127) << 23);
  return {e.hi * scale, e.lo * scale};
}
// log(s) for 1 <= s <= e^80 to 2^-26: one Newton step from the 32-bit logarithm
__device__ __forceinline__ Pair log_pair(Pair s) {
  const float y = logf(s.hi);
  const Pair t = mul(s, exp_pair({-y, 0.0f}));
  return two_sum(y, (t.hi - 1.0f) + t.lo);
}
__device__ __forceinline__ uint64_t order_key(Pair x) { return ((uint64_t)order_key(x.hi) << 32) | order_key(x.lo); }

constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kGather = kMergeThreads;  // candidates that count those before them, one a thread

// A candidate: its score's order, 0 for none, and beam * vocab + token.
struct Candidate {
  uint64_t key;
  uint32_t place;
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  return (a.key > b.key) | ((a.key == b.key) & (a.place < b.place));
}

// One CTA a group of beams: the log-sum-exp of each beam, the scores of all list entries, and the `count`
// best of them.  As in a chunk, the greatest of each thread give a bound; what reaches it is gathered, and every
// gathered candidate counts those before it, which is its place in the result.  Bound by latency.
__global__ void __launch_bounds__(kMergeThreads) select_merge_kernel(SelectParams p) {
  extern __shared__ uint64_t keys[];  // [beams * chunks][count]: score, 0: no candidate
  // A candidate's score is offset + (logit - greatest): next to a logit of 1e38 a logarithm would be lost.
  __shared__ Pair offset[kMaxBeams];  // score - log(sum exp(logit - greatest)), or a finished beam's score
  __shared__ float greatest[kMaxBeams];
  __shared__ int kind[kMaxBeams];  // 0: no candidates, 1: those of its lists, 2: finished
  __shared__ uint32_t pool[32 * kMergeWarps];
  __shared__ uint64_t near_key[kGather];  // entries that are not behind the bound
  __shared__ uint32_t near_place[kGather];
  __shared__ int near_beam[kGather];
  __shared__ uint32_t bound;
  __shared__ int gathered, valid, counters[2];
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lists = p.beams * p.chunks, entries = lists * p.count, per_beam = p.chunks * p.count;
  uint32_t* places = reinterpret_cast<uint32_t*>(keys + entries);        // [beams * chunks][count]
  if (tid == 0) {
    gathered = valid = counters[0] = counters[1] = 0;
    bound = 0;
  }
  grid_dependency_wait();
  const float2* src = p.entries + (int64_t)group * entries;
  constexpr int kAhead = 4;
  float2 ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (tid + j * kMergeThreads < entries) ahead[j] = __ldcg(src + tid + j * kMergeThreads);
  for (int k = warp; k < p.beams; k += kMergeWarps) {
    const int row = group * p.beams + k;
    const float2* s = p.sums + (int64_t)row * p.chunks;
    const float2 first = lane < p.chunks ? __ldcg(s + lane) : make_float2(-CUDART_INF_F, 0.0f);
    const float score = p.scores[row];
    const bool finished = p.done != nullptr && p.done[row] != 0;
    int what = 0;
    Pair off = {score, 0.0f};
    float high = 0.0f;
    if (!(score < CUDART_INF_F)) {  // NaN, +inf
      if (lane == 0) flag_error(p.status, KVARN_DEV_BAD_LOGITS);
    } else if (score > -CUDART_INF_F && finished) {
      what = 2;
    } else if (score > -CUDART_INF_F) {
      float top = first.x;
      bool bad = !(first.y < CUDART_INF_F);
      for (int c = lane + 32; c < p.chunks; c += 32) {
        const float2 v = s[c];
        top = fmaxf(top, v.x);
        bad |= !(v.y < CUDART_INF_F);
      }
      top = key_value(__reduce_max_sync(~0u, order_key(top)));
      bad = __any_sync(~0u, bad);
      if (bad) {
        if (lane == 0) flag_error(p.status, KVARN_DEV_BAD_LOGITS);
      } else if (top > -CUDART_INF_F) {
        Pair sum = {0.0f, 0.0f};
        if (first.x == top) sum.hi = first.y;
        else if (first.x > -CUDART_INF_F) sum.hi = first.y * exp_difference(first.x, top);
        for (int c = lane + 32; c < p.chunks; c += 32) {
          const float2 v = s[c];
          if (v.x > -CUDART_INF_F) sum = add(sum, {v.x == top ? v.y : v.y * exp_difference(v.x, top), 0.0f});
        }
        for (int d = 1; d < 32 && d < p.chunks; d *= 2)
          sum = add(sum, {__shfl_xor_sync(~0u, sum.hi, d), __shfl_xor_sync(~0u, sum.lo, d)});
        what = 1;
        high = top;
        const Pair l = log_pair(sum);
        off = add(off, {-l.hi, -l.lo});
      }
    }
    if (lane == 0) {
      offset[k] = off;
      greatest[k] = high;
      kind[k] = what;
    }
  }
  __syncthreads();
  const float per_inverse = 1.0f / (float)per_beam;
  int mine = 0;
  uint32_t most = 0;  // the greatest score of the thread's entries, in 32 bits
#pragma unroll 1
  for (int i = tid, j = 0; i < entries; i += kMergeThreads, ++j) {
    const float2 e = j == 0 ? ahead[0] : j == 1 ? ahead[1] : j == 2 ? ahead[2] : j == 3 ? ahead[3] : __ldcg(src + i);
    const int k = (int)(((float)i + 0.5f) * per_inverse);  // i / per_beam: entries <= 2048
    uint64_t key = 0;
    int t = __float_as_int(e.y);
    if (kind[k] == 1) {
      const Pair score = add(offset[k], two_sum(e.x, -greatest[k]));
      if (t >= 0 && fabsf(score.hi) < CUDART_INF_F) key = order_key(score);
    } else if (kind[k] == 2 && i == k * per_beam) {  // one candidate, first of the beam's first list
      t = p.end_token;
      key = order_key(offset[k]);
    }
    keys[i] = key;
    places[i] = (uint32_t)k * (uint32_t)p.vocab + (uint32_t)t;
    mine += key != 0;
    most = max(most, (uint32_t)(key >> 32));
  }
  mine = __reduce_add_sync(~0u, mine);
  if (lane == 0 && mine > 0) atomicAdd(&valid, mine);
  const int active = min(kMergeWarps, (entries + 31) / 32);  // warps that hold entries
  // twice as many as wanted: with a few more than wanted 64 candidates leave more than kGather (53 -> 75 us)
  const int take = min(32, (2 * p.count + active - 1) / active);
  for (int m = 0; m < take; ++m) {
    const uint32_t mth = __reduce_max_sync(~0u, most);
    if (lane == __ffs(__ballot_sync(~0u, most == mth)) - 1) {
      pool[warp * take + m] = mth;
      most = 0;
    }
  }
  __syncthreads();
  const int want = min(p.count, valid);
  if (tid < take * active && rank_of_key(pool, take * active, pool[tid], tid) == p.count - 1) bound = pool[tid];
  __syncthreads();
  const uint32_t least = max(bound, 1u);
  const auto gather = [&](int i) {
    const int at = atomicAdd(&gathered, 1);
    if (at >= kGather) return;
    near_key[at] = keys[i];
    near_place[at] = places[i];
    near_beam[at] = (int)(((float)i + 0.5f) * per_inverse);
  };
  for (int i = tid; i < entries; i += kMergeThreads)
    if ((uint32_t)(keys[i] >> 32) >= least) gather(i);
  __syncthreads();
  int total = gathered;
  if (total > kGather) {
    // Many equal scores: the last of the `want` candidates, bit by bit (a lower place first), and those not
    // behind it.
    Candidate cut = {0, ~0u};
    for (int bit = 95; bit >= 0; --bit) {
      Candidate trial = cut;
      if (bit >= 32) trial.key |= 1ull << (bit - 32);
      else trial.place &= ~(1u << bit);
      int n = 0;
      for (int i = tid; i < entries; i += kMergeThreads)
        n += (keys[i] != 0) & !before({trial.key, bit >= 32 ? ~0u : trial.place}, {keys[i], places[i]});
      n = __reduce_add_sync(~0u, n);
      if (lane == 0 && n > 0) atomicAdd(&counters[bit & 1], n);
      __syncthreads();
      if (counters[bit & 1] >= want) cut = trial;
      if (tid == 0) counters[(bit & 1) ^ 1] = 0;
      __syncthreads();
    }
    if (tid == 0) gathered = 0;
    __syncthreads();
    for (int i = tid; i < entries; i += kMergeThreads)
      if (keys[i] != 0 && !before(cut, {keys[i], places[i]})) gather(i);
    __syncthreads();
    total = gathered;
  }
  if (tid < total) {
    const Candidate c = {near_key[tid], near_place[tid]};
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < total; ++j) rank += before({near_key[j], near_place[j]}, c);
    if (rank < p.count) {
      const int64_t o = (int64_t)group * p.count + rank;
      const int k = near_beam[tid], t = (int)(c.place - (uint32_t)k * (uint32_t)p.vocab);
      p.out_scores[o] = key_value((uint32_t)(c.key >> 32));
      p.out_parents[o] = k;
      p.out_tokens[o] = t;
      if (p.out_done != nullptr) p.out_done[o] = kind[k] == 2 || t == p.end_token;
    }
  }
  for (int j = want + tid; j < p.count; j += kMergeThreads) {
    const int64_t o = (int64_t)group * p.count + j;
    p.out_scores[o] = -CUDART_INF_F;
    p.out_parents[o] = -1;
    p.out_tokens[o] = -1;
    if (p.out_done != nullptr) p.out_done[o] = 0;
  }
}

// Chunks of a row: two CTAs an SM when the rows are few, each of some thousand logits at least, and no more lists than
// the one CTA that merges a group joins quickly.  With 4 / 3 / 2 an SM 128 rows of 128000 take 15.8 / 15.7 / 15.2 us, 80 of
// 100000 14.0 / 12.7 / 12.8, 40 of 50001 11.2 / 11.1 / 10.4: more chunks end more often and leave the merge more lists.
// One group of 8 rows of 151936 with 16 candidates takes 21.2 us with lists of up to 8192 candidates, 14.7 with 4096, 10.9
// with 1024, 11.6 with 512, 12.8 with 256; one of 16 rows with 32 takes 48, 23, 19, 23 and 23 us.
static int chunks_of(int64_t rows, int beams, int vocab, int count) {
  int64_t c = 152 * 2 / rows;
  const int64_t most = (vocab + 2047) / 2048, held = kChunkEntries / ((int64_t)beams * count);
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
  static PerDeviceOnce smem_once;
  constexpr int kSmem = sizeof(Ring<T, kBytes>);
  if (const int st = set_smem_limit(smem_once, reinterpret_cast<const void*>(select_kernel<T, kBytes>), kSmem); st != KVARN_OK)
    return st;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config((unsigned)(p.batch * p.beams * (int64_t)p.chunks), kThreads, kSmem, stream, &attr);
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
// one thread, which reads them all before it writes: the outputs may be the inputs' own buffers.  The beams'
// sources and live rows are worked out once a CTA (worked out for every move, the kernel ran 135 instructions a
// move and was bound by them as much as by HBM).
template <int kBeams>
__global__ void __launch_bounds__(kMoveThreads) reorder_kernel(ReorderParams p) {
  __shared__ int parent[kMaxBeams], pages[kMaxBeams], live[kMaxBeams];
  __shared__ int64_t from[kMaxBeams];
  __shared__ int most;
  const int tid = threadIdx.x;
  const int64_t unit = blockIdx.x;  // (group, kv head, slice)
  const int slice = (int)(unit % p.slices);
  const int head = (int)(unit / p.slices % p.num_kv_heads);
  const int group = (int)(unit / p.slices / p.num_kv_heads);
  const int rows0 = group * p.beams;
  const int layer = ((int)blockIdx.y - 1) >> 1, kv = ((int)blockIdx.y - 1) & 1;
  const int vecs = p.dim / 8;
  const uint4* src = reinterpret_cast<const uint4*>(kv ? p.v : p.k);
  uint4* dst = reinterpret_cast<uint4*>(kv ? p.v_out : p.k_out);
  const int64_t seq = (int64_t)p.num_kv_heads * kTile * vecs;  // vectors of one sequence in one layer
  grid_dependency_wait();
  if (tid < 32) {
    int n = 0, rows = 0;
    if (tid < p.beams) {
      int of = p.parents[rows0 + tid], bad = 0;
      if (of < -1 || of >= p.beams) bad = KVARN_DEV_BAD_BEAM, of = -1;
      if (of >= 0) {
        n = p.seq_lens[rows0 + of];
        if (n < 0 || n / kTile > p.max_pages) bad = KVARN_DEV_SEQ_TOO_LONG;
      }
      rows = n > 0 && !(src == dst && of == tid) ? n % kTile : 0;
      parent[tid] = of;
      pages[tid] = max(n, 0) / kTile;
      live[tid] = rows;
      from[tid] = max(of, 0) * seq;
      if (blockIdx.y == 0 && slice == 0 && head == 0) {
        p.seq_lens_out[rows0 + tid] = n;
        if (bad) flag_error(p.status, bad);
      }
    }
    rows = __reduce_max_sync(~0u, rows);
    if (tid == 0) most = rows;
  }
  __syncthreads();
  if (blockIdx.y == 0) {
    // lengths and table rows
    const int step = p.slices * p.num_kv_heads * kMoveThreads;
    for (int64_t i = (int64_t)(head * p.slices + slice) * kMoveThreads + tid; i < p.max_pages; i += step) {
      int32_t x[kBeams];
#pragma unroll
      for (int b = 0; b < kBeams; ++b)
        if (b < p.beams && i < pages[b]) x[b] = p.table[(int64_t)(rows0 + parent[b]) * p.max_pages + i];
#pragma unroll
      for (int b = 0; b < kBeams; ++b)
        if (b < p.beams && i < pages[b]) p.table_out[(int64_t)(rows0 + b) * p.max_pages + i] = x[b];
    }
    return;
  }
  const int64_t first = (int64_t)layer * p.batch * p.beams * seq + (int64_t)rows0 * seq + (int64_t)head * kTile * vecs;
  src += first;
  dst += first;
  const float per_row = 1.0f / (float)vecs;
  for (int i = slice * kMoveThreads + tid; i < most * vecs; i += p.slices * kMoveThreads) {
    const int row = (int)(((float)i + 0.5f) * per_row);  // i / vecs: i < 4096
    uint4 x[kBeams];
#pragma unroll
    for (int b = 0; b < kBeams; ++b)
      if (b < p.beams && row < live[b]) x[b] = src[from[b] + i];
    uint4* to = dst + i;
#pragma unroll
    for (int b = 0; b < kBeams; ++b, to += seq)
      if (b < p.beams && row < live[b]) *to = x[b];
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
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      config((unsigned)batch, kMergeThreads, (size_t)lists * count * 12, s, &attr);
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
  // Few units: CTAs to fill the GPU; many: long-lived ones.  16 groups of 4 over 16 layers take 52 / 45 / 45 / 46 us in
  // 8 / 4 / 2 / 1 slices, 6 groups of 5 over 4 layers 5.3 / 4.1 / 3.8 / 4.2 us, one group in one layer 2.5 us in 4 or more,
  // 3.2 in 2.  4 / 2 / 1 slices of 8 kv heads: 4 groups of 4 in one layer 2.9 / 3.6 / 3.8 us, 16 groups 4.8 / 4.2 / 4.9, 16 groups
  // over 4 layers 14.8 / 15.1 / 15.3, 8 groups of 8 over 16 layers 91.0 / 92.8 / 95.6.
  p.slices = (int64_t)batch * p.num_kv_heads * (2 * layers + 1) <= 152 ? 4 : 2;
  if ((int64_t)batch * p.num_kv_heads * p.slices > 0x7fffffffLL) return KVARN_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (beams <= 4) return launch_reorder<4>(p, s);
  if (beams <= 8) return launch_reorder<8>(p, s);
  if (beams <= 16) return launch_reorder<16>(p, s);
  return launch_reorder<32>(p, s);
}

}  // extern "C"
