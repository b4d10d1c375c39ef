// Attention of a block of new tokens per sequence over the packed cache (sm_103a): the drafted
// tokens of a tree, each seeing the whole cache and its own ancestors, or a chunk of a prompt under
// a sliding window with a few first tokens that stay visible.
//
// Math (rotated basis, R = H_d / sqrt(d)): a sealed page's logit of query row r and token t is
//   tau r_t ( sum_j code_tj (q~_rj s'_j) + sum_j q~_rj z'_j ),  o~ = sum_t p_t V~_t,
//   V~_tj = c_j ( code_tj s'_t + z'_t )
// [vatt §四個步驟: the rotation keeps q.k unchanged; hotdry §非对称量化与尺度折叠: the folded scales
//  are multiplied back at read].  Three kernels:
//  block_raw_kernel    the open tile's raw tokens and the new tokens themselves, masked, on
//                      mma.sync: one partial (m, l, o) per query row, original basis;
//  block_cache_kernel  the sealed pages on tcgen05: partials in the rotated basis;
//  block_merge_kernel  joins the partials, undoes the rotation, rounds once to fp16.
//
// block_cache_kernel.  The G * block query rows of one (sequence, kv head) are cut into row tiles of
// NR = 16, 32, 48 or 64 rows.  The (row tile, visible page) pairs lie on a line that is cut into equal
// ranges, one per CTA and one CTA per SM.  Tokens sit on the MMA's M axis (a page is exactly its
// 128 rows) and query rows on N, so that the MMA time follows the rows a tile has.  Per page:
//  QK  S[t][r] = sum_j A_K[t][j] B[j][r]; A_K = the codes in tensor memory as exact fp16 subnormals
//      (one AND per two codes), B = q~ . s' as fp16 hi, then lo (2 x D/16 MMAs into one
//      accumulator).  hi + lo because keys with outlier channels give logits in the hundreds, and
//      one fp16 rounding of q~ s' (2^-11 relative) would move them by 0.1;
//  PV  O[c][r] += sum_t A_V[c][t] P[t][r]; A_V = V~ rounded twice to fp16 (once per product),
//      P = exp2 rounded once to fp16.  These roundings cost precision, and kvarn.h tells the caller:
//      against 64 bits the output is off by 3.1e-4 to 3.8e-4 (relative 2-norm), by 2.1e-4 where only it
//      is rounded.  Without either V~'s second rounding or P's it would still be near 3e-4, and going
//      without both takes fp32 conversions and a second PV pass on the pipes that bound this kernel.
// Softmax: a thread owns a token and half the rows of the tile; each row's reference, 2^7 below a maximum
// of the row, is kept from page to page and moved only when a logit passes that maximum by 2^8 (then O
// and l are rescaled), so no maximum is exchanged on the usual page; P stays below 2^15 and l is fp32.
// Warps: 0-7 softmax (two warpgroups, one per row half: also the rescale and the row tile's partial at
// its end), 8-11 K codes, 12-15 q~ . z' (both groups: half of B each), 16-23 V, 24 page records (1-D
// bulk copies into a ring), 25-26 QK and 27-28 PV (one warp per column part), 29-31 the walk and q~ of
// the next segment.  Operand and score buffers are double.  Every wait on an mbarrier is bounded; what
// follows when one runs out is in role_waits.h: all roles go on to the same end, the copies and MMAs in
// flight are waited for, and the call reports KVARN_DEV_WAIT_TIMEOUT.
// What bounds it: the conversion of codes and the softmax on the ordinary pipes, not memory and not the
// tensor cores.  With 64 rows, head_dim 128 and K4V2 a page takes about 1.31 us a SM (2520 cycles, 6820
// instructions; on 16 trees of 26 nodes issue slots 62 % used, shared memory's data pipe 52 %, tensor
// pipe 30 %, DRAM 13 %), a segment about 10 us on top: 16 trees of 64 nodes over 16k 624 us, a 2 x 2048-token
// windowed chunk 690 us of this kernel.
#include "common.cuh"
#include "decode_util.cuh"
#include "params.cuh"
#include "role_waits.h"
#include "tcgen05.cuh"

namespace kvarn {
namespace blk {

using namespace tc5;

constexpr int kThreads = 1024;
// warps: 0-7 softmax (4 per row half), 8-15 K, 16-23 V, 24 loader, 25-26 QK, 27-28 PV, 29-31 queries
constexpr int kKWarp = 8, kVWarp = 16, kMiscWarp = 24;
constexpr int kLoadWarp = 24, kQkWarp = 25, kPvWarp = 27, kQueryWarp = 29;
constexpr int kMaxSlots = 8;
// Segments in flight, a power of two: the query warps are at most two ahead of the K warps, and the
// roles that trail (V by up to six pages, each a segment of its own at worst) are within 8 of those.
constexpr int kSegs = 16;
// Named barriers.  Warps hand work to each other through them: a warp waiting at one issues nothing,
// while polls of mbarriers by 13 warps (one every ~23 cycles each) kept the arrivals of the others
// waiting and cost more than the work itself.  mbarriers remain where the hardware signals (bulk
// copies, MMA completion), polled by one warp of a role, which then meets the others.
//   0 the CTA; kQueryBar the query warps; kSmBar + half the softmax warps of a row half;
//   kKBar, kVBar the K and V warps; per stage kOpsK (K warps -> QK), kSFree (softmax -> QK),
//   kOpsV (V warps -> PV); kPFull + 2 part + stage (softmax -> PV).
constexpr int kQueryBar = 1, kSmBar = 2, kKBar = 4, kVBar = 5, kOpsK = 6, kSFree = 8, kOpsV = 10, kPFull = 12;
// Units of the line ahead of a row tile's pages for a segment's fixed work, and the smallest range
// (5, 8 and 14 units took no less time than 3).
constexpr int kFixUnits = 3, kMinUnits = 3;
// A row's reference lies kHead (log2 units) below the maximum it was set at, and a logit may pass that
// maximum by kSlack: P is at most 2^15.  fp16 ends at 2^-24, so that what is lost of a weight lies
// below 2^-32 of the row's largest (without the head 2^-25, which many tokens can add up to).
constexpr float kHead = 7.0f, kSlack = 8.0f;
// The raw tokens' reference follows the maximum from stage to stage: P is at most 2^12, what is lost of
// a weight lies below 2^-37 of the row's largest, and the logits' own rounding has room up to 2^16.
constexpr float kRawHead = 12.0f;
constexpr int kSmemMax = 232448 - 1536;  // the rest is for the static part

template <int D, int NR>
struct Shape {
  static constexpr int kSteps = D / 16;           // K steps of QK
  static constexpr int kHalves = D > 128 ? 2 : 1; // 128-channel blocks of PV
  static constexpr int kParts = NR % 32 == 0 ? 2 : 1; // column parts of the MMAs (N a multiple of 16)
  static constexpr int kVStages = D > 128 ? 1 : 2;
  static constexpr int kStep = NR * 32;           // bytes of one K step of a B operand
  static constexpr int kBHalf = NR * D * 2;       // q~ s' hi (or lo) of one page
  // P, MN-major: per 16 tokens two groups of 8 rows (tokens) of 16 bytes per 8 columns; the second
  // group is 32 bytes off so that the 8 lanes of a store phase, two groups of four, miss each other
  static constexpr int kPGroup = NR * 16 + 32, kPStep = 2 * kPGroup;
  static constexpr int kPBytes = 8 * kPStep;
  // shared memory: B (two stages, hi + lo), P (two stages), q~ hi + lo of two segments, small state, records
  static constexpr int kBOff = 0;
  static constexpr int kPOff = 2 * 2 * kBHalf;
  static constexpr int kQOff = kPOff + 2 * kPBytes;
  static constexpr int kSmallOff = kQOff + 2 * 2 * kBHalf;
  // floats: qz [4][NR], -reference, row maximum, rescale [NR] each, row limit [kSegs][NR], per warp
  // [4][NR], token factors [4][128]
  static constexpr int kSmallFloats = (4 + 3 + kSegs + 4) * NR + 4 * kTile;
  static constexpr int kBarOff = kSmallOff + kSmallFloats * 4;
  static constexpr int kNumBars = 2 * kMaxSlots + 2 * 4 + kSegs + 2;
  static constexpr int kRecOff = (kBarOff + kNumBars * 8 + 127) & ~127;
  // tensor memory columns
  static constexpr uint32_t kColK = 0, kColV = 2 * (D / 2);
  static constexpr uint32_t kColS = kColV + kVStages * 64 * kHalves;
  static constexpr uint32_t kColO = kColS + 2 * NR;
  static_assert(kColO + kHalves * NR <= 512, "fits tensor memory");
};

// kind::f16, f32 accumulate, f16 A and B, M = 128, N = NR; B K-major (QK) or MN-major (PV).
template <int NR>
constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(NR >> 3) << 17) | ((128u >> 4) << 24);
template <int NR>
constexpr uint32_t kIdescPV = kIdescQK<NR> | (1u << 16);

// Factors on q~ for channels 0..7 and 8..15 of every 16, whose 4- / 2-bit codes sit 4 / 2 bits
// apart in their subnormals (the same lifts as the decode kernels' operands).
__device__ __forceinline__ float lift0(int kb) { return kb == 8 ? 256.0f : (kb == 4 ? 16.0f : 4.0f); }
__device__ __forceinline__ float lift1(int kb) { return kb == 8 ? 256.0f : 1.0f; }

// These barriers are the aligned forms: a warp's threads come to them together.  Threads may leave a
// poll or an elected section one by one, so that __syncwarp() follows each (inside the three wrappers,
// ahead of every barrier, it cost 5 % on 16 trees of 64 nodes: 659 against 624 us).
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier of `threads` threads; returns whether any of them passed `flag`.
__device__ __forceinline__ bool bar_any(int id, int threads, bool flag) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, %2, %3, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out)
      : "r"((uint32_t)flag), "r"(id), "r"(threads)
      : "memory");
  return out != 0;
}

// Bounded wait (2 s, as the other kernels') on an mbarrier, for page `need` - 1 of the MMA warp whose
// count of issued pages is *issued (null: none, as for copies); see wait_page.
__device__ __forceinline__ void wait_one(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         const volatile int* issued, int need) {
  wait_page([&] { return mbar_try_wait(bar, parity); }, [&] { return issued == nullptr || *issued >= need; },
            [&] { return *abort_flag != 0; }, [&] { *abort_flag = 1; }, global_timer_ns);
}
// One lane of a converged warp.  MMAs are issued under it: the compiler then knows that a single
// thread runs them and keeps their operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {  // (a & b) | c
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

template <int N>
struct IntC {
  static constexpr int value = N;
};

__device__ __forceinline__ int cached_len(const BlockParams& p, int b) {
  const int cap = p.max_pages * kTile + (kTile - 1);
  const int len = p.seq_lens[b];
  return len < 0 ? 0 : (len > cap ? cap : len);
}
__device__ __forceinline__ int new_len(const BlockParams& p, int b) {
  if (p.new_lens == nullptr) return p.block;
  const int n = p.new_lens[b];
  return n < 0 ? 0 : (n > p.block ? p.block : n);
}

// The sealed pages row tile t of sequence b sees: 0 .. sinks - 1, then first ..; count in all.
struct Span {
  int sinks, first, count;
  __device__ __forceinline__ int page(int i) const { return i < sinks ? i : first + (i - sinks); }
};
__device__ __forceinline__ Span tile_span(const BlockParams& p, int len, int nl, int t) {
  const int n = len / kTile;
  const int c0 = t * p.tile_rows / p.group;  // the tile's first new token
  if (c0 >= nl) return {0, 0, 0};
  if (p.window <= 0) return {0, 0, n};
  const int start = max(0, len + c0 + 1 - p.window);
  const int first = min(start / kTile, n);
  const int sinks = min((p.sink + kTile - 1) / kTile, first);
  return {sinks, first, sinks + n - first};
}
__device__ __forceinline__ int tile_units(const Span& s, int fix) { return s.count > 0 ? s.count + fix : 0; }
// pages of all row tiles of one kv head of sequence b, and the tiles that have any
__device__ __forceinline__ int64_t head_pages(const BlockParams& p, int b, int& tiles) {
  const int len = cached_len(p, b), nl = new_len(p, b);
  const int live = (nl * p.group + p.tile_rows - 1) / p.tile_rows;
  tiles = 0;
  if (p.window <= 0) {
    if (len >= kTile) tiles = live;
    return (int64_t)live * (len / kTile);
  }
  int64_t n = 0;
  for (int t = 0; t < live; ++t) {
    const Span s = tile_span(p, len, nl, t);
    n += s.count;
    tiles += s.count > 0 ? 1 : 0;
  }
  return n;
}

struct Partition : PagePartition {
  int fix;  // units ahead of a row tile's pages
};

// A CTA's range of the line, as segments: runs of pages of one row tile.
struct TileWalk {
  int b, h, t, j;   // row tile t of (sequence b, kv head h), first visible page of the segment
  int len, nl;      // sequence b's cached and new tokens
  Span span;
  int64_t left;     // units of the range from page j on (0: nothing left)
  int64_t row0;     // unit at which the row tile starts
  __device__ int count() const { return (int)min((int64_t)(span.count - j), left); }
  __device__ int64_t row(const BlockParams& p) const { return ((int64_t)b * p.num_kv_heads + h) * p.tiles + t; }
  __device__ void next(const BlockParams& p, int fix) {
    left -= count();
    if (left <= 0) return;
    j = 0;
    row0 += tile_units(span, fix);
    for (;;) {
      if (++t >= p.tiles) {
        t = 0;
        if (++h == p.num_kv_heads) {
          h = 0;
          if (++b >= p.batch) {  // unreachable while the lengths stay as they were
            left = 0;
            return;
          }
          len = cached_len(p, b);
          nl = new_len(p, b);
        }
      }
      span = tile_span(p, len, nl, t);
      if (span.count > 0) {
        left -= fix;  // the range may end inside the row tile's fixed units
        if (left < 0) left = 0;
        return;
      }
    }
  }
};

// Warp-collective: the partition and this CTA's walk.
__device__ __forceinline__ TileWalk range_walk(const BlockParams& p, int64_t cta, int lane, Partition& pp) {
  TileWalk w = {};
  long long pages = 0, tiles = 0;
  for (int b = lane; b < p.batch; b += 32) {
    int t;
    pages += head_pages(p, b, t);
    tiles += t;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    pages += __shfl_xor_sync(0xffffffffu, pages, m);
    tiles += __shfl_xor_sync(0xffffffffu, tiles, m);
  }
  pages *= p.num_kv_heads;
  tiles *= p.num_kv_heads;
  // With few pages a CTA each the pages are spread one by one (a segment's fixed work then runs on
  // all SMs at once); with more the line charges each row tile for it.
  pp.fix = pages <= 2 * kBlockCtas ? 0 : kFixUnits;
  pp.total = pages + tiles * pp.fix;
  const int64_t c = pp.fix == 0 ? pp.total : pp.total / kMinUnits;
  pp.ctas = pp.total > 0 ? (c < 1 ? 1 : (c > kBlockCtas ? kBlockCtas : c)) : 0;
  if (cta >= pp.ctas) return w;
  const int64_t x0 = range_start(pp, cta), x1 = range_start(pp, cta + 1);
  long long cum = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int bb = b0 + lane;
    int ht = 0;
    long long hu = bb < p.batch ? head_pages(p, bb, ht) : 0;
    hu += (long long)ht * pp.fix;
    long long incl = hu * p.num_kv_heads;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += o;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > x0);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      const long long u = __shfl_sync(0xffffffffu, hu, l);
      long long at = cum + __shfl_sync(0xffffffffu, incl, l) - u * p.num_kv_heads;  // start of sequence b
      w.b = b0 + l;
      w.len = cached_len(p, w.b);
      w.nl = new_len(p, w.b);
      w.h = (int)((x0 - at) / u);
      at += (long long)w.h * u;
      for (w.t = 0;; ++w.t) {  // the row tile that holds x0
        w.span = tile_span(p, w.len, w.nl, w.t);
        const int tu = tile_units(w.span, pp.fix);
        if (x0 < at + tu || w.t + 1 >= p.tiles) break;
        at += tu;
      }
      w.row0 = at;
      const int64_t first = at + pp.fix;  // unit of the row tile's first page
      w.j = x0 < first ? 0 : (int)(x0 - first);
      w.left = x1 - (first + w.j);
      if (w.left < 0) w.left = 0;  // the range ends inside the fixed units
      return w;
    }
    cum += __shfl_sync(0xffffffffu, incl, 31);
  }
  return w;
}

}  // namespace blk

// ---- the sealed pages ----------------------------------------------------------------------
template <int D, int NR>
__global__ void __launch_bounds__(blk::kThreads, 1) block_cache_kernel(BlockParams p, int slots) {
  using namespace blk;
  using S = Shape<D, NR>;
  constexpr int NC = NR / 2;       // rows (columns of S, P and O) of one softmax warpgroup
  constexpr int NP = S::kParts;    // MMA column parts
  constexpr int NM = NR / NP;      // columns of one MMA
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ TileWalk seg_s[kSegs];
  __shared__ Partition part_s;
  __shared__ uint32_t tslot;
  __shared__ int abort_flag;
  __shared__ uint32_t gate_s;  // segments published, and kGateClosed (role_waits.h)
  __shared__ int issued_s[4];  // pages whose QK (parts 0, 1) and PV (parts 0, 1) are issued
  __shared__ __align__(8) uint64_t drained_s[4];  // every MMA of an issuing warp has completed
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RecordLayout RL = record_layout(D, p.kb, p.vb);
  const int rec = RL.bytes;
  uint64_t* rec_full = reinterpret_cast<uint64_t*>(sm + S::kBarOff);
  uint64_t* rec_empty = rec_full + kMaxSlots;
  uint64_t* qk_full = rec_empty + kMaxSlots;  // [part][stage]: QK done (K codes and B are free)
  uint64_t* pv_done = qk_full + 4;            // [part][stage]: PV done: V and P are free, O is up to date
  uint64_t* seg_full = pv_done + 4;           // [segment % kSegs]: its walk, q~ and row limits written
  uint64_t* q_empty = seg_full + kSegs;       // [segment % 2]: the K warps are done with its q~
  constexpr int kOpsThreads = 256 + 32 * NP;           // kOpsK, kSFree, kOpsV
  constexpr int kPThreads = 256 / NP + 32;             // kPFull
  float* qz_s = reinterpret_cast<float*>(sm + S::kSmallOff);  // [4][NR]: page g's at g % 4
  float* nref_s = qz_s + 4 * NR;   // minus the row's reference
  float* max_s = nref_s + NR;      // the row's maximum when the reference was set (-inf: none yet)
  float* alpha_s = max_s + NR;     // rescale of l and O
  int* lim_all = reinterpret_cast<int*>(alpha_s + NR);  // [kSegs][NR]: position from which a row's window sees
  float* warp_s = reinterpret_cast<float*>(lim_all + kSegs * NR);  // [4][NR]
  float* rt_s = warp_s + 4 * NR;  // [4][128]: the token factors of page g at g % 4
  uint8_t* recs = sm + S::kRecOff;
  auto q_of = [&](int k) { return sm + S::kQOff + (k & 1) * 2 * S::kBHalf; };  // hi, then lo

  // The kernel before this one (block_raw_kernel) waited for everything ahead of it before it let
  // this grid start, so the inputs are complete; its own partials are read by the merge only.
  if (warp == 1) {
    Partition pp;
    const TileWalk w = range_walk(p, blockIdx.x, lane, pp);
    if (lane == 0) {
      seg_s[0] = w;
      part_s = pp;
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&rec_full[i], 1);
      mbar_init(&rec_empty[i], 16);  // the K and V warps
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&qk_full[s], 2);
      mbar_init(&pv_done[s], 1);
    }
    for (int s = 0; s < kSegs; ++s) mbar_init(&seg_full[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&q_empty[s], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&drained_s[i], 1);
    abort_flag = 0;
    gate_s = 1;  // segment 0 is staged below, by all warps
    for (int i = 0; i < 4; ++i) issued_s[i] = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tslot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  grid_launch_dependents();
  const uint32_t tmem = tslot;
  volatile int* abort_v = &abort_flag;
  volatile int* issued = issued_s;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_one(bar, parity, abort_v, nullptr, 0); };
  // QK / PV of page j (j < 0: none) by the warp of column part m
  auto wait_qk = [&](int m, int j) {
    if (j >= 0) wait_one(&qk_full[2 * m + (j & 1)], (uint32_t)((j >> 1) & 1), abort_v, issued + m, j + 1);
  };
  auto wait_pv = [&](int m, int j) {
    if (j >= 0) wait_one(&pv_done[2 * m + (j & 1)], (uint32_t)((j >> 1) & 1), abort_v, issued + 2 + m, j + 1);
  };
  // Segments pass through a ring (their q~ through two buffers): the query warps write segment k + 1
  // while the others work on segment k.  These waits do not look at the abort flag: the query warps
  // and the roles keep going after it is set, for as long as pages are issued.
  auto seg = [&](int k) -> const TileWalk& { return seg_s[k & (kSegs - 1)]; };
  auto wait_handoff = [&](uint64_t* bar, uint32_t parity) -> bool {
    return wait_progress([&] { return mbar_try_wait(bar, parity); }, [&] { return issued[0]; }, global_timer_ns);
  };
  auto wait_segment = [&](int k) {
    if (wait_handoff(&seg_full[k & (kSegs - 1)], (uint32_t)(k / kSegs) & 1u)) return;
    *abort_v = 1;
    atomicOr(&gate_s, kGateClosed);
    __threadfence_block();
  };
  // Segment k, once waited for, is there: false past the end of the range, and for every role alike
  // past the segments published when some role gave up waiting.
  auto there = [&](int k) -> bool {
    return gate_open(*const_cast<volatile uint32_t*>(&gate_s), k) && seg(k).left > 0;
  };
  // Segment k for a group of warps that meets at barrier `id`.
  auto segment = [&](int k, int id, int threads, bool leader) -> bool {
    if (leader) wait_segment(k);
    __syncwarp();
    bar_sync(id, threads);
    return there(k);
  };
  // q~ of segment k, hi + lo, in the order and layout of the QK operand: passes n0, n0 + step, .. of
  // 512 / D rows.  A lane takes one 16-channel block of a row (four butterfly stages within the lane,
  // the rest across lanes, every shuffle of a stage in flight together), which is one K step's two
  // 16-byte chunks.
  auto stage_queries = [&](int k, int n0, int step) {
    constexpr int kRowsPass = 512 / D;
    const int row0 = seg(k).t * NR, nl = seg(k).nl, lim0 = seg(k).len + 1 - p.window;
    const __half* base = p.q + ((int64_t)seg(k).b * p.block * p.num_q_heads + seg(k).h * p.group) * p.d0;
    uint8_t* q_hi = q_of(k);
    int* lim_s = lim_all + (k & (kSegs - 1)) * NR;
    const float sc = p.qscale * inv_sqrt_d<D>();
    const bool q16 = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0u;
    const int shift = 31 - __clz(p.group);  // the group is a power of two
    const int blk = lane / kRowsPass;
#pragma unroll 1
    for (int pass = n0; pass < NR / kRowsPass; pass += step) {
      const int n = pass * kRowsPass + lane % kRowsPass;
      const int r = row0 + n, c = r >> shift;
      const bool live = c < nl;
      const __half* src = base + ((int64_t)c * p.num_q_heads + (r & (p.group - 1))) * p.d0 + 16 * blk;
      float v[16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // d0 is a multiple of 8
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (live && 16 * blk + 8 * h < p.d0) {
          if (q16) {
            w = *reinterpret_cast<const uint4*>(src + 8 * h);
          } else {
            const uint16_t* x = reinterpret_cast<const uint16_t*>(src + 8 * h);
            w = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
          }
        }
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(u2h2(ws[e]));
          v[8 * h + 2 * e] = f.x;
          v[8 * h + 2 * e + 1] = f.y;
        }
      }
#pragma unroll
      for (int st = 1; st < 16; st <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((i & st) == 0) {
            const float x = v[i], y = v[i + st];
            v[i] = x + y;
            v[i + st] = x - y;
          }
#pragma unroll
      for (int m = kRowsPass; m < 32; m <<= 1) {
        const float sign = (lane & m) != 0 ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = fmaf(sign, v[i], __shfl_xor_sync(0xffffffffu, v[i], m));
      }
      uint8_t* dst = q_hi + blk * S::kStep + (n >> 3) * 256 + (n & 7) * 16;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // channels 4kb + {0, 1}, {8, 9}, {2, 3}, {10, 11}
          const int ch = 4 * kb + 8 * (e & 1) + 2 * (e >> 1);
          const float f = sc * ((e & 1) ? lift1(p.kb) : lift0(p.kb));
          const float x = v[ch] * f, y = v[ch + 1] * f;
          const __half2 h2 = __floats2half2_rn(x, y);
          const float2 hf = __half22float2(h2);
          hi[e] = h2u(h2);
          lo[e] = h2u(__floats2half2_rn(x - hf.x, y - hf.y));
        }
        *reinterpret_cast<uint4*>(dst + 128 * kb) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + S::kBHalf + 128 * kb) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      // padding rows see everything: they get a reference on the first page
      if (blk == 0) lim_s[n] = live ? lim0 + c : INT32_MIN;
    }
  };
  // where the merge finds the partials of the row tile that segment w begins, if it begins one
  auto note_slots = [&](const TileWalk& w) {
    if (w.left <= 0 || w.j != 0) return;
    const int64_t row = w.row(p);
    const int64_t last = owner_cta(part_s, w.row0 + part_s.fix + w.span.count - 1);
    p.row_info[row] = make_int2((int)((int64_t)blockIdx.x + row), (int)(last - blockIdx.x + 1));
  };
  if (seg_s[0].left > 0) stage_queries(0, warp, kThreads / 32);
  __syncthreads();
  // the roles' place in the line of pages and in the ring of records
  int g = 0;
  int r = 0;
  uint32_t rph = 0;
  auto next_record = [&]() {
    if (++r == slots) {
      r = 0;
      rph ^= 1u;
    }
  };

  // Registers of the 65,536 the CTA is launched with: 104 a thread for the softmax, which holds a
  // token's NR / 2 logits and as many sums, 72 for K, which holds its share of q~, 40 for the rest.
  if (warp < kKWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---- softmax (thread = token, rows c0 ..), rescale and the segment's partial (thread = channel) ----
    const int u = threadIdx.x & 127, wq = warp & 3;
    const int half = warp >> 2;
    const int c0 = half * NC;
    const int part = NP == 2 ? half : 0;
    const int sbar = kSmBar + half;
    const uint32_t lanes = (uint32_t)(32 * wq) << 16;
    const int kpos = 4 * ((u >> 1) & 3) + 2 * ((u >> 3) & 1) + (u & 1);
    const int poff = (u >> 4) * S::kPStep + (kpos >> 3) * S::kPGroup + (kpos & 7) * 16 + 16 * c0;
    const float cf = kTwo24 / lift0(p.kb) * (p.kb == 2 && ((u >> 4) & 1) ? 0.0625f : 1.0f);
    for (int k = 0; segment(k, sbar, 128, wq == 0); ++k) {
      const TileWalk& w = seg(k);  // read where it is needed: registers are short here
      const int cnt = w.count();
      float2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = make_float2(0.0f, 0.0f);
      if (u < NC) {
        nref_s[c0 + u] = 0.0f;
        max_s[c0 + u] = -INFINITY;
      }
      bool unset = true;  // some row has no reference yet
      for (int i = 0; i < cnt; ++i, ++g) {
        const int s = (int)(g & 1);
        // S of the page, and PV of the page before the last, which has read this stage's P
        // (a poll takes ~150 cycles even when it succeeds, so each is another warp's)
        if (wq == 0) wait_qk(part, g);
        if (wq == 1) wait_pv(part, g - 2);
        __syncwarp();
        bar_sync(sbar, 128);
        fence_after();
        const uint32_t ts = tmem + S::kColS + (uint32_t)(s * NR + c0) + lanes;
        const float rt = rt_s[(g & 3) * kTile + u], at = rt * cf;
        const float* qz = qz_s + (g & 3) * NR + c0;
        const int* lim_s = nullptr;  // the rows' limits on an edge page of the window or the first tokens
        int pos = 0;
        if (p.window > 0) {
          pos = w.span.page(w.j + i) * kTile;
          // from `sure` on the window of the tile's last row sees
          const int sure = w.len + min((w.t * NR + NR - 1) / p.group, w.nl - 1) + 1 - p.window;
          if (pos + kTile > p.sink && pos < sure) lim_s = lim_all + (k & (kSegs - 1)) * NR + c0;
          pos += u;
          if (pos < p.sink) lim_s = nullptr;  // this token is one of the first
        }
        float x[NC];  // logits less their rows' references
        for (bool moved = false;; moved = true) {
          ld_cols<NC>(ts, x);
#pragma unroll
          for (int n = 0; n < NC; n += 4) {
            const float4 z = *reinterpret_cast<const float4*>(qz + n);
            const float4 m = *reinterpret_cast<const float4*>(nref_s + c0 + n);
            const float2 a = fma2(make_float2(at, at), make_float2(x[n], x[n + 1]),
                                  fma2(make_float2(rt, rt), make_float2(z.x, z.y), make_float2(m.x, m.y)));
            const float2 c = fma2(make_float2(at, at), make_float2(x[n + 2], x[n + 3]),
                                  fma2(make_float2(rt, rt), make_float2(z.z, z.w), make_float2(m.z, m.w)));
            x[n] = a.x;
            x[n + 1] = a.y;
            x[n + 2] = c.x;
            x[n + 3] = c.y;
          }
          if (lim_s != nullptr) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (pos < lim_s[n]) x[n] = -INFINITY;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < NC; n += 2) mx = fmax3(mx, x[n], x[n + 1]);
          if (!bar_any(sbar, 128, !moved && (unset || mx > kHead + kSlack))) break;
          // Move the references to the rows' maxima, then take the logits again.  This runs once or
          // twice a segment, from a cold instruction cache that costs ~200 cycles for eight
          // instructions: short loops over eight rows here, and the code above for the rest.
#pragma unroll 1
          for (int n0 = 0; n0 < NC; n0 += 8) {
            float y[8];
            ld_cols<8>(ts + n0, y);
            float mine = 0.0f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              y[n] = fmaf(at, y[n], rt * qz[n0 + n]);
              if (lim_s != nullptr && pos < lim_s[n0 + n]) y[n] = -INFINITY;
              const float v = warp_max(y[n]);
              if (lane == n) mine = v;
            }
            if (lane < 8) warp_s[wq * NR + c0 + n0 + lane] = mine;
          }
          bar_sync(sbar, 128);
          bool none = false;
          if (u < NC) {
            const int n = c0 + u;
            const float old = max_s[n];
            const float pm = fmaxf(fmaxf(warp_s[n], warp_s[NR + n]), fmaxf(warp_s[2 * NR + n], warp_s[3 * NR + n]));
            const float mn = fmaxf(old, pm);
            none = mn == -INFINITY;
            const float nref = none ? 0.0f : kHead - mn;
            alpha_s[n] = old == -INFINITY ? 0.0f : ex2_approx(nref - nref_s[n]);
            max_s[n] = mn;
            nref_s[n] = nref;
          }
          unset = bar_any(sbar, 128, none);
          if (i > 0) {  // l and O of the pages before this one
#pragma unroll
            for (int n = 0; n < NC; n += 2) {
              const float2 al = *reinterpret_cast<const float2*>(alpha_s + c0 + n);
              l[n / 2] = mul2(l[n / 2], al);
            }
            wait_pv(part, g - 1);
            __syncwarp();
            fence_after();
#pragma unroll 1
            for (int hf = 0; hf < S::kHalves; ++hf)
#pragma unroll 1
              for (int n0 = 0; n0 < NC; n0 += 8) {
                float o[8];
                const uint32_t ta = tmem + S::kColO + (uint32_t)(hf * NR + c0 + n0) + lanes;
                ld_cols<8>(ta, o);
                uint32_t ob[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) ob[n] = __float_as_uint(o[n] * alpha_s[c0 + n0 + n]);
                st_32x32b_x8(ta, ob);
              }
            wait_st();
          }
        }
        fence_before();
        bar_arrive(kSFree + s, kOpsThreads);
        uint8_t* pb = sm + S::kPOff + s * S::kPBytes + poff;
#pragma unroll
        for (int n = 0; n < NC; n += 8) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = make_float2(ex2_approx(x[n + 2 * e]), ex2_approx(x[n + 2 * e + 1]));
            l[n / 2 + e] = add2(l[n / 2 + e], v);
            h[e] = h2u(__floats2half2_rn(v.x, v.y));
          }
          *reinterpret_cast<uint4*>(pb + 16 * n) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        fence_before();
        bar_arrive(kPFull + 2 * part + s, kPThreads);
      }
      // the segment's partial: l over the tokens, O once its last PV is done
      // (a butterfly that halves the rows a lane holds: row lane ends in lane's first value)
      constexpr int kPow = NC == 24 ? 32 : NC;
      float v[kPow];
#pragma unroll
      for (int n = 0; n < kPow; n += 2) {
        v[n] = n < NC ? l[n / 2 < NC / 2 ? n / 2 : 0].x : 0.0f;
        v[n + 1] = n < NC ? l[n / 2 < NC / 2 ? n / 2 : 0].y : 0.0f;
      }
#pragma unroll
      for (int m = 16; m >= kPow; m >>= 1)
#pragma unroll
        for (int n = 0; n < kPow; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], m);
#pragma unroll
      for (int m = kPow / 2; m > 0; m >>= 1) {
        const bool up = (lane & m) != 0;
#pragma unroll
        for (int n = 0; n < m; ++n) {
          const float send = up ? v[n] : v[n + m];
          const float keep = up ? v[n + m] : v[n];
          v[n] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
      }
      if (lane < NC) warp_s[wq * NR + c0 + lane] = v[0];
      bar_sync(sbar, 128);
      const int live = min(NR, w.nl * p.group - w.t * NR) - c0;  // rows of this half that exist
      float* dst = p.part + (((int64_t)blockIdx.x + w.row(p)) * NR + c0) * (D + 4);
      if (u < min(live, NC)) {
        const int n = c0 + u;
        float* d = dst + (int64_t)u * (D + 4);
        d[0] = max_s[n] == -INFINITY ? -INFINITY : -nref_s[n];
        d[1] = (warp_s[n] + warp_s[NR + n]) + (warp_s[2 * NR + n] + warp_s[3 * NR + n]);
      }
      wait_pv(part, g - 1);
      __syncwarp();
      fence_after();
#pragma unroll 1
      for (int hf = 0; hf < S::kHalves; ++hf) {
#pragma unroll 1
        for (int n0 = 0; n0 < min(NC, live); n0 += 8) {
          float o[8];
          ld_cols<8>(tmem + S::kColO + (uint32_t)(hf * NR + c0 + n0) + lanes, o);
          if (D >= 128 || u < D) {
#pragma unroll
            for (int n = 0; n < 8; ++n)
              if (n0 + n < live) dst[(int64_t)(n0 + n) * (D + 4) + 4 + hf * 128 + u] = o[n];
          }
        }
      }
      fence_before();
    }
  } else if (warp < kVWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 72;");
    // ---- warps 8-11: K codes -> tensor memory; 12-15: q~ . z'; each half of the rows of B = q~ s' ----
    const int t = threadIdx.x & 127, q = warp & 3;
    const bool codes = warp < kKWarp + 4;
    const int grp = t >> 3, nl = t & 7;
    const int gq = lane >> 2, tq = lane & 3;
    const float i0 = 1.0f / lift0(p.kb), i1 = 1.0f / lift1(p.kb);
    // B rows n = 8 rg + nl over K indexes 8kb..8kb+7 of step kk (channels cb + {0, 1, 8, 9, 2, 3, 10,
    // 11}): the 16 thread groups of 8 take the D / 8 (kk, kb) pairs and, each warpgroup, half the rows.
    // A thread's q~ stay in registers for the segment.
    constexpr int kPairs = D > 128 ? 2 : 1;
    constexpr int kRows = D == 64 ? (NR / 16 + 1) / 2 : NR / 16;
    auto builds = [&](int e) { return D > 64 || 2 * e + (grp >> 3) < NR / 16; };  // whether row group e is there
    auto pair_of = [&](int c2) { return D == 64 ? (grp & 7) : grp + 16 * c2; };
    auto b_at = [&](int c2, int e) {
      const int oc = pair_of(c2);
      const int rg = (codes ? 0 : NR / 16) + (D == 64 ? 2 * e + (grp >> 3) : e);
      return (oc >> 1) * S::kStep + rg * 256 + (oc & 1) * 128 + nl * 16;
    };
    for (int k = 0; segment(k, kKBar, 256, warp == kKWarp); ++k) {
      const int cnt = seg(k).count();
      const uint8_t* q_hi = q_of(k);
      const uint8_t* q_lo = q_hi + S::kBHalf;
      if (k > 0 && t == 0 && codes) mbar_arrive(&q_empty[(k - 1) & 1]);  // every K warp is past it
      uint4 qh[kPairs][kRows], ql[kPairs][kRows];
#pragma unroll
      for (int c2 = 0; c2 < kPairs; ++c2)
#pragma unroll
        for (int e = 0; e < kRows; ++e) {
          qh[c2][e] = ql[c2][e] = make_uint4(0u, 0u, 0u, 0u);
          if (builds(e)) {
            qh[c2][e] = *reinterpret_cast<const uint4*>(q_hi + b_at(c2, e));
            ql[c2][e] = *reinterpret_cast<const uint4*>(q_lo + b_at(c2, e));
          }
        }
      for (int i = 0; i < cnt; ++i, ++g) {
        const int s = (int)(g & 1);
        // QK of the page before the last has read the codes and B
        if (warp == kKWarp) wait(&rec_full[r], rph);
        if (warp > kKWarp && warp <= kKWarp + NP) wait_qk(warp - kKWarp - 1, g - 2);
        __syncwarp();
        bar_sync(kKBar, 256);
        fence_after();
        const uint8_t* R = recs + r * rec;
        if (codes) {
          // fragment (o, i) of 16 tokens x 16 channels is lanes 16o.., columns 8i..8i+7; column
          // 2tq + h holds channels 16i + 8h + 2tq, +1 of its tokens g and g + 8
          const uint32_t ta = tmem + S::kColK + (uint32_t)(s * (D / 2)) + ((uint32_t)(32 * q) << 16);
          const uint4* kc = reinterpret_cast<const uint4*>(R + RL.kcodes);
          if (p.kb == 4) {
#pragma unroll
            for (int oo = 0; oo < 2; ++oo)
#pragma unroll 2
              for (int kq = 0; kq < D / 64; ++kq) {
                const uint4 w4 = kc[((2 * q + oo) * (D / 64) + kq) * 32 + lane];
                const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
                uint32_t rr[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t x = ws[e], y = x >> 8;
                  rr[4 * e] = x & 0x000F000Fu;
                  rr[4 * e + 1] = x & 0x00F000F0u;
                  rr[4 * e + 2] = y & 0x000F000Fu;
                  rr[4 * e + 3] = y & 0x00F000F0u;
                }
                st_16x256b_x4(ta + ((uint32_t)(16 * oo) << 16) + 32 * kq, rr);
              }
          } else if (p.kb == 8) {
#pragma unroll 1
            for (int oo = 0; oo < 2; ++oo)
#pragma unroll 2
              for (int kp = 0; kp < D / 32; ++kp) {
                const uint4 w4 = kc[((2 * q + oo) * (D / 32) + kp) * 32 + lane];
                uint32_t rr[8], a[4];
                unpack_k8(w4.x, w4.y, a);
                rr[0] = a[0];
                rr[1] = a[2];
                rr[2] = a[1];
                rr[3] = a[3];
                unpack_k8(w4.z, w4.w, a);
                rr[4] = a[0];
                rr[5] = a[2];
                rr[6] = a[1];
                rr[7] = a[3];
                st_16x256b_x2(ta + ((uint32_t)(16 * oo) << 16) + 16 * kp, rr);
              }
          } else {  // 2-bit: a word holds token blocks 2q and 2q + 1, the odd one's codes 4 bits higher
#pragma unroll 1
            for (int kq = 0; kq < D / 64; ++kq) {
              const uint4 w4 = kc[(q * (D / 64) + kq) * 32 + lane];
              const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
              for (int oo = 0; oo < 2; ++oo) {
                uint32_t rr[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t x = ws[e], y = x >> 8;
                  rr[4 * e] = x & (0x00030003u << (4 * oo));
                  rr[4 * e + 1] = x & (0x000C000Cu << (4 * oo));
                  rr[4 * e + 2] = y & (0x00030003u << (4 * oo));
                  rr[4 * e + 3] = y & (0x000C000Cu << (4 * oo));
                }
                st_16x256b_x4(ta + ((uint32_t)(16 * oo) << 16) + 32 * kq, rr);
              }
            }
          }
        } else if (16 * q < NR) {
          // q~ . z' of rows 16q..16q+15 on mma.sync: B column 0 holds z' of channels 0..7 of every
          // 16, column 1 of channels 8..15, whose q~ carry different lifts
          float acc[2][4] = {};  // q~ hi and lo: two chains
          const int m = lane >> 3;
          const uint32_t qa = smem_u32(q_hi) + (2 * q + (m & 1)) * 256 + (m >> 1) * 128 + (lane & 7) * 16;
          const bool mine = gq < 2 && (tq & 1) == gq;
          const uint8_t* zc = R + RL.kzero + 2 * (8 * (tq & 1) + 2 * (tq >> 1));
#pragma unroll 8
          for (int kk = 0; kk < S::kSteps; ++kk) {
            const uint32_t b0 = mine ? *reinterpret_cast<const uint32_t*>(zc + 32 * kk) : 0u;
            const uint32_t b1 = mine ? *reinterpret_cast<const uint32_t*>(zc + 32 * kk + 8) : 0u;
            uint32_t a[4];
            ldsm_x4(qa + kk * S::kStep, a);
            mma16816(acc[0], a, b0, b1);
            ldsm_x4(qa + S::kBHalf + kk * S::kStep, a);
            mma16816(acc[1], a, b0, b1);
          }
          if (tq == 0) {
            float* qz = qz_s + (g & 3) * NR + 16 * q + gq;
            qz[0] = (acc[0][0] + acc[1][0]) * i0 + (acc[0][1] + acc[1][1]) * i1;
            qz[8] = (acc[0][2] + acc[1][2]) * i0 + (acc[0][3] + acc[1][3]) * i1;
          }
        }
        if (!codes) rt_s[(g & 3) * kTile + t] = __half2float(reinterpret_cast<const __half*>(R + RL.kfactor)[t]);
        uint8_t* bs = sm + S::kBOff + s * 2 * S::kBHalf;
#pragma unroll
        for (int c2 = 0; c2 < kPairs; ++c2) {
          const int oc = pair_of(c2), cb = 16 * (oc >> 1) + 4 * (oc & 1);
          const uint2 sa = *reinterpret_cast<const uint2*>(R + RL.kscale + 2 * cb);
          const uint2 sb = *reinterpret_cast<const uint2*>(R + RL.kscale + 2 * (cb + 8));
          const __half2 sv[4] = {u2h2(sa.x), u2h2(sb.x), u2h2(sa.y), u2h2(sb.y)};
#pragma unroll
          for (int e = 0; e < kRows; ++e) {
            if (!builds(e)) continue;
            const __half2 h4[4] = {u2h2(qh[c2][e].x), u2h2(qh[c2][e].y), u2h2(qh[c2][e].z), u2h2(qh[c2][e].w)};
            const __half2 l4[4] = {u2h2(ql[c2][e].x), u2h2(ql[c2][e].y), u2h2(ql[c2][e].z), u2h2(ql[c2][e].w)};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 hv = __hmul2(h4[j], sv[j]);
              hi[j] = h2u(hv);
              lo[j] = h2u(__hfma2(l4[j], sv[j], __hfma2(h4[j], sv[j], __hneg2(hv))));
            }
            *reinterpret_cast<uint4*>(bs + b_at(c2, e)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(bs + S::kBHalf + b_at(c2, e)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_empty[r]);
        if (codes) wait_st();
        fence_proxy_async_smem();
        fence_before();
        bar_arrive(kOpsK + s, kOpsThreads);
        next_record();
      }
    }
  } else if (warp < kMiscWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // ---- V~ -> tensor memory: channels on the lanes, tokens along K; a warp takes its quarter's
    // 32 channels of each 128 and half the tokens ----
    const int q = warp & 3, th = (warp - kVWarp) >> 2;
    const int gq = lane >> 2;
    for (int k = 0; segment(k, kVBar, 256, warp == kVWarp); ++k) {
      const int cnt = seg(k).count();
      for (int i = 0; i < cnt; ++i, ++g) {
        const int s = (int)(g & 1);
        const int vs = S::kVStages == 2 ? s : 0;
        // PV of the page that last used this buffer
        if (warp == kVWarp) wait(&rec_full[r], rph);
        if (warp > kVWarp && warp <= kVWarp + NP) wait_pv(warp - kVWarp - 1, g - S::kVStages);
        __syncwarp();
        bar_sync(kVBar, 256);
        fence_after();
        const uint8_t* R = recs + r * rec;
        const uint32_t sz = smem_u32(R + RL.vscale) + 16 * (lane >> 3);  // group lane / 8 of a pair's four
        const __half* vch = reinterpret_cast<const __half*>(R + RL.vfactor);
        const uint32_t* vc = reinterpret_cast<const uint32_t*>(R + RL.vcodes);
        const uint32_t ta =
            tmem + S::kColV + (uint32_t)(vs * 64 * S::kHalves) + ((uint32_t)(32 * q) << 16);
        if (D >= 128 || q < D / 32) {
#pragma unroll 1
          for (int hf = 0; hf < S::kHalves; ++hf) {
            const int cb = 8 * hf + 2 * q;  // channel blocks cb and cb + 1: adjacent words
            __half2 cv[2][2];
#pragma unroll
            for (int ii = 0; ii < 2; ++ii)
#pragma unroll
              for (int rho = 0; rho < 2; ++rho) cv[ii][rho] = __half2half2(vch[16 * (cb + ii) + gq + 8 * rho]);
            const uint32_t* vw = vc + ((cb >> 2) * 32 + lane) * 4 + (cb & 3);
            auto tile = [&](auto vbc) {
              constexpr int VB = decltype(vbc)::value;
              constexpr int kMasks = VB == 2 ? 4 : 2;  // bit offsets of a code: 2-bit 0, 2, 4, 6, 4-bit 0, 4
              uint32_t mask[kMasks];
#pragma unroll
              for (int e = 0; e < kMasks; ++e) {
                mask[e] = VB == 2 ? 0x00030003u << (2 * e) : 0x000F000Fu << (4 * e);
                asm("" : "+r"(mask[e]));  // kept in registers: a LOP3 takes one immediate
              }
#pragma unroll
              for (int oo = 0; oo < 2; ++oo) {
                const int o2 = 2 * th + oo;  // pair of 16-token blocks
                // token scales and zeros of the pair's four 8-token groups: rows of one ldmatrix all
                // at the same 16 bytes leave lane (g, tq) tokens 2tq, 2tq + 1 of each group
                uint32_t s2[4], z2[4];
                ldsm_x4(sz + 64 * o2, s2);
                ldsm_x4(sz + 2 * kTile + 64 * o2, z2);
                uint2 x[2];  // words of blocks cb, cb + 1 (2-bit: both token blocks share one)
                x[0] = *reinterpret_cast<const uint2*>(vw + (VB == 2 ? o2 : 2 * o2) * (D / 64) * 128);
                if (VB == 4) x[1] = *reinterpret_cast<const uint2*>(vw + (2 * o2 + 1) * (D / 64) * 128);
#pragma unroll
                for (int ii = 0; ii < 2; ++ii) {
                  uint32_t rr[8];
#pragma unroll
                  for (int f = 0; f < 2; ++f) {
                    const uint2 w2 = x[VB == 2 ? 0 : f];
                    const uint32_t lo = ii ? w2.y : w2.x, hi = lo >> 8;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      // the code's bits under an exponent that makes them base + code, minus base
                      const int e = VB == 2 ? 2 * f + h : h;
                      const uint32_t base = 0x64006400u - (uint32_t)(VB == 2 ? 2 * e : 4 * e) * 0x04000400u;
#pragma unroll
                      for (int rho = 0; rho < 2; ++rho) {
                        const __half2 c = __hsub2(u2h2(and_or(rho ? hi : lo, mask[e], base)), u2h2(base));
                        rr[4 * f + 2 * rho + h] =
                            h2u(__hmul2(__hfma2(c, u2h2(s2[2 * f + h]), u2h2(z2[2 * f + h])), cv[ii][rho]));
                      }
                    }
                  }
                  st_16x256b_x2(ta + ((uint32_t)(16 * ii) << 16) + 64 * hf + 16 * o2, rr);
                }
              }
            };
            if (p.vb == 2) tile(IntC<2>{});
            else tile(IntC<4>{});
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_empty[r]);
        wait_st();
        fence_before();
        bar_arrive(kOpsV + s, kOpsThreads);
        next_record();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kLoadWarp) {
      // ---- page records -> the ring ----
      if (lane == 0) {
        CopyRing ring(slots);
        for (int k = 0;; ++k) {
          wait_segment(k);
          const TileWalk& w = seg(k);
          const int cnt = there(k) ? w.count() : 0;
          const int j = w.j, sinks = w.span.sinks, skip = w.span.first - w.span.sinks;
          const int32_t* bt = p.block_table + (int64_t)w.b * p.max_pages;
          const uint8_t* src = p.pool + (int64_t)w.h * rec;
          if (cnt == 0) break;
          for (int i = j; i < j + cnt; ++i) {
            int64_t id = bt[i < sinks ? i : i + skip];
            if (id < 0 || id >= p.num_pool_pages) {
              flag_error(p.status, KVARN_DEV_BAD_PAGE_ID);
              id = 0;
            }
            uint64_t* full = &rec_full[ring.slot];
            wait(&rec_empty[ring.slot], ring.phase ^ 1u);
            if (*abort_v != 0) continue;  // nobody waits for the copies any more
            fence_proxy_async_smem();
            mbar_expect_tx(full, (uint32_t)rec);
            bulk_copy_g2s(recs + ring.slot * rec, src + id * p.num_kv_heads * (int64_t)rec, (uint32_t)rec, full);
            ring.next();
          }
        }
        // The copies still in flight land before the CTA may leave, whatever has run out elsewhere:
        // these waits do not look at the abort flag.
        if (!ring.drain([&](int slot, uint32_t parity) { return mbar_wait(&rec_full[slot], parity); })) *abort_v = 1;
      }
      __syncwarp();
    } else if (warp >= kQueryWarp) {
      // ---- the segments' walk and queries, one segment ahead of the roles ----
      const bool lead = warp == kQueryWarp;
      if (lead && lane == 0) {
        mbar_arrive(&seg_full[0]);  // staged above
        note_slots(seg(0));
      }
      bool open = true;  // the segments so far were published before any role gave up
      for (int k = 1; seg(k - 1).left > 0; ++k) {
        if (lead) {
          TileWalk& w = seg_s[k & (kSegs - 1)];
          if (lane == 0) {
            w = seg(k - 1);
            w.next(p, part_s.fix);
          }
          // the K warps are done with the queries of the segment before the last (after a closed
          // gate they may have ended)
          const bool free_q = k < 2 || !open || wait_handoff(&q_empty[k & 1], (uint32_t)((k - 2) >> 1) & 1u);
          open = __all_sync(0xffffffffu, free_q) && open;
          if (!open) *abort_v = 1;
          if (lane == 0) {
            if (!open) w.left = 0;  // the last segment
            note_slots(w);
          }
          __syncwarp();
        }
        bar_sync(kQueryBar, 96);
        if (seg(k).left > 0) stage_queries(k, warp - kQueryWarp, 3);
        bar_sync(kQueryBar, 96);
        if (lead) {
          int published = 1;
          if (lane == 0) {
            __threadfence_block();
            published = gate_publish([&](uint32_t was, uint32_t is) { return atomicCAS(&gate_s, was, is); }, k);
            mbar_arrive(&seg_full[k & (kSegs - 1)]);
          }
          open = __shfl_sync(0xffffffffu, published, 0) != 0 && open;
        }
      }
    } else if (warp - (warp >= kPvWarp ? kPvWarp : kQkWarp) < NP) {
      // ---- MMA issue: QK and PV, a warp for each row half ----
      const bool is_pv = warp >= kPvWarp;
      const int part = is_pv ? warp - kPvWarp : warp - kQkWarp;
      for (int k = 0;; ++k) {
        wait_segment(k);
        __syncwarp();
        const int cnt = there(k) ? seg(k).count() : 0;
        if (cnt == 0) break;
        for (int i = 0; i < cnt; ++i, ++g) {
          const int s = g & 1;
          if (is_pv) {
            bar_sync(kOpsV + s, kOpsThreads);
            bar_sync(kPFull + 2 * part + s, kPThreads);
          } else {
            bar_sync(kOpsK + s, kOpsThreads);
            if (g >= 2) bar_sync(kSFree + s, kOpsThreads);  // S of the page before the last is read
          }
          fence_after();
          if (elect_one()) {
            if (is_pv) {
              const uint64_t pd = smem_desc(smem_u32(sm + S::kPOff + s * S::kPBytes) + part * NR * 8, S::kPGroup, 128);
              const uint32_t av = tmem + S::kColV + (S::kVStages == 2 ? (uint32_t)(s * 64 * S::kHalves) : 0u);
#pragma unroll 1
              for (int hf = 0; hf < S::kHalves; ++hf)
#pragma unroll
                for (int o = 0; o < 8; ++o)
                  mma_ts(tmem + S::kColO + hf * NR + part * NM, av + 64 * hf + 8 * o, pd + o * (S::kPStep >> 4),
                         kIdescPV<NM>, (uint32_t)(i > 0 || o > 0));
              mma_commit(&pv_done[2 * part + s]);
              issued[2 + part] = g + 1;
            } else {
              const uint64_t bd = smem_desc(smem_u32(sm + S::kBOff + s * 2 * S::kBHalf) + part * NR * 16, 128, 256);
              const uint32_t ak = tmem + S::kColK + (uint32_t)(s * (D / 2));
#pragma unroll 1
              for (int lo = 0; lo < 2; ++lo)
#pragma unroll 8
                for (int kk = 0; kk < S::kSteps; ++kk)
                  mma_ts(tmem + S::kColS + (uint32_t)(s * NR + part * NM), ak + 8 * kk,
                         bd + (lo * S::kSteps + kk) * (S::kStep >> 4), kIdescQK<NM>, (uint32_t)(lo + kk > 0));
              mma_commit(&qk_full[2 * part + s]);
              // this thread has seen the K warps' writes (q~ . z') and passes them on to the softmax
              mbar_arrive(&qk_full[2 * part + s]);
              issued[part] = g + 1;
            }
          }
          __syncwarp();  // the next page's barriers want the whole warp
        }
      }
      if (g > 0) {
        // The MMAs have completed before tensor memory is given back: one more commit arrives once
        // all of this thread's have, and the wait does not look at the abort flag (after an abort
        // the pages' own barriers say only what was issued).  The arrivals for pages that do not
        // follow are taken.
        uint64_t* drained = &drained_s[(is_pv ? 2 : 0) + part];
        if (elect_one()) mma_commit(drained);
        __syncwarp();
        if (!mbar_wait(drained, 0)) *abort_v = 1;
        __syncwarp();
        if (!is_pv)
          for (int i = g > 1 ? g - 2 : 0; i < g; ++i) bar_sync(kSFree + (i & 1), kOpsThreads);
      }
      __syncwarp();
    }
  }

  // ---- tear-down: every role is past its last wait ----
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_flag != 0) flag_error(p.status, KVARN_DEV_WAIT_TIMEOUT);
  if (warp == 2) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  grid_dependency_wait();  // block_raw_kernel has finished when this grid has
}

// ---- the open tile's raw tokens and the new tokens -------------------------------------------
// One CTA of 8 warps per (128 query rows, kv head, sequence), warp w taking rows 16w..16w+15; K and
// V rows stream through shared memory 64 tokens at a time (cp.async into swizzled fp16 rows, two
// stages), the open tile's first, then the new tokens'.  mma.sync m16n8k16: A = the fp16 queries
// (exact products; the scale applied to the fp32 sums) by ldmatrix, B = K rows by ldmatrix; online
// softmax in the log2 domain; PV with the probabilities, 2^12 at a row's maximum, rounded once to fp16
// (they move the output like its own rounding; as fp16 hi + lo the 2 x 2048-token chunk's call takes 1159
// instead of 1076 us).  A row that sees nothing leaves m = -inf, l = 0, o = 0.  The queries stay in
// shared memory so that two CTAs (16 warps) fit an SM at head_dim 64 and 128: with them in registers,
// one CTA an SM and fp16 hi + lo probabilities a 2 x 2048-token chunk took 482 us.  Masks are looked at
// only in stages that some row of the warp does not see whole: that chunk 386 -> 332 us; latency
// bounds it (8 x 256 tokens: issue slots 38 % used, tensor pipe 28 %, 16 warps an SM).  32 rows a
// warp took longer (395 against 386 us, before that step).
template <int D>
__global__ void __launch_bounds__(256, D <= 128 ? 2 : 1) block_raw_kernel(BlockParams p) {
  constexpr int NB = 64;      // tokens per stage
  constexpr int NN = D / 8;   // channel n-tiles
  constexpr int KK = D / 16;  // channel k-steps
  constexpr uint32_t kStage = 2 * NB * 2 * D;  // K rows then V rows, fp16
  extern __shared__ __align__(128) uint8_t cs[];
  const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
  const int g = lane >> 2, tq = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y;
  const int G = p.group;
  grid_dependency_wait();    // lengths, tiles and tokens may come from the previous kernel
  grid_launch_dependents();  // block_cache_kernel reads nothing of this one
  const int raw_len = p.seq_lens[b], len = blk::cached_len(p, b), nl = blk::new_len(p, b);
  int n_part = len % kTile;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    if (raw_len != len || (p.new_lens != nullptr && p.new_lens[b] != nl)) flag_error(p.status, KVARN_DEV_SEQ_TOO_LONG);
    if (n_part > 0 && p.partial_k == nullptr) flag_error(p.status, KVARN_DEV_NO_PARTIAL);
  }
  if (p.partial_k == nullptr) n_part = 0;
  const int part0 = len - len % kTile;  // position of the open tile's first token
  const int rows = nl * G;
  const int rbase = ((int)gridDim.x - 1 - (int)blockIdx.x) * 128;  // the longest causal rows first
  if (rbase >= rows) return;
  const int r0 = rbase + 16 * wi;  // this warp's first query row
  const bool warp_live = r0 < rows;
  const int c_first = rbase / G, c_last = min(rbase + 127, rows - 1) / G;  // the CTA's new tokens
  const int ra = r0 + g, rb = r0 + g + 8;
  const int ca = ra < rows ? ra / G : -1, cb = rb < rows ? rb / G : -1;  // -1: padding row
  const uint32_t sbase = smem_u32(cs);
  const uint32_t qbase = sbase + 2 * kStage;  // [128][D] fp16 query rows, swizzled
  const int64_t rstride = (int64_t)p.num_kv_heads * p.d0;
  const int64_t nbase = ((int64_t)b * p.block * p.num_kv_heads + h) * p.d0;
  const int64_t pbase = ((int64_t)b * p.num_kv_heads + h) * kTile * p.d0;
  const int dch = p.d0 / 8;  // 16-byte chunks of a row (d0 % 8 == 0)
  // stages: `pblk` of the open tile, then those of the new tokens any row of the CTA may see
  const int pblk = (n_part + NB - 1) / NB;
  const int n_new = p.mask != nullptr ? nl : c_last + 1;
  const int nblk = pblk + (n_new + NB - 1) / NB;
  // whether no row of the CTA sees a token of stage `blk` (windows only)
  auto skipped = [&](int blk) {
    if (p.window <= 0) return false;
    const int at = blk < pblk ? part0 + blk * NB : len + (blk - pblk) * NB;  // position of its first token
    return at >= p.sink && at + NB <= len + c_first + 1 - p.window;
  };
  auto next_blk = [&](int blk) {
    do ++blk;
    while (blk < nblk && skipped(blk));
    return blk;
  };
  auto stage = [&](int blk, int buf) {
    const uint32_t base = sbase + (uint32_t)buf * kStage;
    const bool part = blk < pblk;
    const int t0 = part ? blk * NB : (blk - pblk) * NB;
    const int n = part ? n_part : n_new;
    const __half* kg = part ? p.partial_k + pbase : p.new_k + nbase;
    const __half* vg = part ? p.partial_v + pbase : p.new_v + nbase;
    const int64_t stride = part ? p.d0 : rstride;
    for (int qi = threadIdx.x; qi < 2 * NB * (D / 8); qi += blockDim.x) {
      const int r = qi / (D / 8), c = qi - r * (D / 8);
      const int t = t0 + (r < NB ? r : r - NB);
      const bool in = t < n && c < dch;
      const __half* src = (r < NB ? kg : vg) + (int64_t)t * stride + 8 * c;
      cp_async_16(base + swz_row<D>(r, c), in ? src : p.new_k, in ? 16u : 0u);
    }
    cp_async_commit_all();
  };
  int blk = next_blk(-1);
  if (blk < nblk) stage(blk, 0);
  {
    // the CTA's queries (zero past the rows and past d0); rows start at multiples of 8 elements
    const bool q16 = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0u;
    for (int qi = threadIdx.x; qi < 128 * (D / 8); qi += blockDim.x) {
      const int n = qi / (D / 8), ch = qi - n * (D / 8);
      const int r = rbase + n, c = r / G;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && ch < dch) {
        const __half* src = p.q + (((int64_t)b * p.block + c) * p.num_q_heads + h * G + (r - c * G)) * p.d0 + 8 * ch;
        if (q16) {
          w = *reinterpret_cast<const uint4*>(src);
        } else {
          const uint16_t* x = reinterpret_cast<const uint16_t*>(src);
          w = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
        }
      }
      *reinterpret_cast<uint4*>(cs + 2 * kStage + swz_row<D>(n, ch)) = w;
    }
  }
  float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;  // l: this lane's share
  float o[NN][4];
#pragma unroll
  for (int n = 0; n < NN; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
  for (int buf = 0; blk < nblk; buf ^= 1) {
    const int nxt = next_blk(blk);
    if (nxt < nblk) {
      stage(nxt, buf ^ 1);  // its buffer was released by the barrier closing the stage before
      cp_async_wait_prev();
    } else {
      cp_async_wait_all();
    }
    __syncthreads();
    const bool part = blk < pblk;
    const int t0 = part ? blk * NB : (blk - pblk) * NB;
    const int n = part ? n_part : n_new;
    // bit 8nt + 2tq + e of va / vb: row ra / rb sees token t0 + 8nt + 2tq + e
    uint64_t va = 0, vb = 0;
    if (warp_live) {
      if (!part && p.mask != nullptr) {
        auto bits = [&](int c) -> uint64_t {
          if (c < 0) return 0;
          const uint32_t* m = p.mask + ((int64_t)b * p.block + c) * p.mask_words;
          const int w = t0 / 32;
          return (uint64_t)m[w] | ((uint64_t)(w + 1 < p.mask_words ? m[w + 1] : 0u) << 32);
        };
        va = bits(ca);
        vb = bits(cb);
      } else {
        const int at = part ? part0 + t0 : len + t0;  // position of the stage's first token
        auto bits = [&](int c) -> uint64_t {
          if (c < 0) return 0;
          const int upto = len + c + 1 - at;                            // tokens up to the query's own
          uint64_t v = upto >= 64 ? ~0ull : (upto <= 0 ? 0ull : (1ull << upto) - 1ull);
          if (p.window > 0) {
            const int drop = upto - p.window, keep = p.sink - at;       // tokens before the window / sinks
            const uint64_t old = drop >= 64 ? ~0ull : (drop <= 0 ? 0ull : (1ull << drop) - 1ull);
            const uint64_t snk = keep >= 64 ? ~0ull : (keep <= 0 ? 0ull : (1ull << keep) - 1ull);
            v &= ~old | snk;
          }
          return v;
        };
        va = bits(ca);
        vb = bits(cb);
      }
      const uint64_t in = n - t0 >= 64 ? ~0ull : (1ull << (n - t0)) - 1ull;
      va &= in;
      vb &= in;
    }
    if (__any_sync(0xffffffffu, (va | vb) != 0ull)) {
      const uint32_t base = sbase + (uint32_t)buf * kStage;
      float s[NB / 8][4];
#pragma unroll
      for (int nt = 0; nt < NB / 8; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        uint32_t a[4];  // rows 16wi + .., channels 16kk + ..
        ldsm_x4(qbase + swz_row<D>(16 * wi + (lane & 15), 2 * kk + (lane >> 4)), a);
#pragma unroll
        for (int np = 0; np < NB / 16; ++np) {  // token n-tiles 2np, 2np + 1
          uint32_t bk[4];
          ldsm_x4(base + swz_row<D>(16 * np + (lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1)), bk);
          mma16816(s[2 * np], a, bk[0], bk[1]);
          mma16816(s[2 * np + 1], a, bk[2], bk[3]);
        }
      }
      // masks, where some row does not see the whole stage (the bit tests are a third of the
      // instructions of a stage that needs them)
      if (!__all_sync(0xffffffffu, (va & vb) == ~0ull)) {
#pragma unroll
        for (int nt = 0; nt < NB / 8; ++nt) {
          const uint32_t ba = (uint32_t)(va >> (8 * nt)) >> (2 * tq), bb = (uint32_t)(vb >> (8 * nt)) >> (2 * tq);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (((ba >> e) & 1u) == 0u) s[nt][e] = -INFINITY;
            if (((bb >> e) & 1u) == 0u) s[nt][2 + e] = -INFINITY;
          }
        }
      }
      float mxa = -INFINITY, mxb = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NB / 8; ++nt) {
        mxa = fmax3(mxa, s[nt][0], s[nt][1]);
        mxb = fmax3(mxb, s[nt][2], s[nt][3]);
      }
      mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, 1));
      mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, 2));
      mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, 1));
      mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, 2));
      // references in the log2 domain, kRawHead below the maxima; qscale > 0
      const float na = fmaxf(ma, fmaf(mxa, p.qscale, -blk::kRawHead)), nb = fmaxf(mb, fmaf(mxb, p.qscale, -blk::kRawHead));
      const float sa = na == -INFINITY ? 0.0f : -na, sb = nb == -INFINITY ? 0.0f : -nb;
      const float aa = ma == -INFINITY ? 0.0f : exp2f(ma - na);
      const float ab = mb == -INFINITY ? 0.0f : exp2f(mb - nb);
      ma = na;
      mb = nb;
      float2 pa = make_float2(0.0f, 0.0f), pb = pa;
      const float2 q2 = make_float2(p.qscale, p.qscale), sa2 = make_float2(sa, sa), sb2 = make_float2(sb, sb);
#pragma unroll
      for (int nt = 0; nt < NB / 8; ++nt) {
        const float2 x = fma2(make_float2(s[nt][0], s[nt][1]), q2, sa2);
        const float2 y = fma2(make_float2(s[nt][2], s[nt][3]), q2, sb2);
        s[nt][0] = ex2_approx(x.x);
        s[nt][1] = ex2_approx(x.y);
        s[nt][2] = ex2_approx(y.x);
        s[nt][3] = ex2_approx(y.y);
        pa = add2(pa, make_float2(s[nt][0], s[nt][1]));
        pb = add2(pb, make_float2(s[nt][2], s[nt][3]));
      }
      la = fmaf(la, aa, pa.x + pa.y);
      lb = fmaf(lb, ab, pb.x + pb.y);
      if (__any_sync(0xffffffffu, aa != 1.0f || ab != 1.0f)) {  // some row's maximum moved
#pragma unroll
        for (int n2 = 0; n2 < NN; ++n2) {
          o[n2][0] *= aa;
          o[n2][1] *= aa;
          o[n2][2] *= ab;
          o[n2][3] *= ab;
        }
      }
#pragma unroll
      for (int ks = 0; ks < NB / 16; ++ks) {
        if (t0 + 16 * ks >= n) break;  // past the tokens (warp-uniform)
        // A = p of tokens t0 + 16ks..: n-tiles 2ks (k 0..7) and 2ks + 1 (k 8..15)
        uint32_t ah[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ah[i] = h2u(__floats2half2_rn(s[2 * ks + (i >> 1)][2 * (i & 1)], s[2 * ks + (i >> 1)][2 * (i & 1) + 1]));
#pragma unroll
        for (int np = 0; np < NN / 2; ++np) {  // channel n-tiles 2np, 2np + 1
          uint32_t bv[4];
          ldsm_x4_trans(base + swz_row<D>(NB + 16 * ks + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * np + (lane >> 4)), bv);
          mma16816(o[2 * np], ah, bv[0], bv[1]);
          mma16816(o[2 * np + 1], ah, bv[2], bv[3]);
        }
      }
    }
    __syncthreads();  // the stage buffer is refilled two stages on
    blk = nxt;
  }
  if (!warp_live) return;
  la += __shfl_xor_sync(0xffffffffu, la, 1);
  la += __shfl_xor_sync(0xffffffffu, la, 2);
  lb += __shfl_xor_sync(0xffffffffu, lb, 1);
  lb += __shfl_xor_sync(0xffffffffu, lb, 2);
  const int64_t row0 = ((int64_t)b * p.num_kv_heads + h) * p.tiles * p.tile_rows;
  auto store = [&](int r, int hf, float m, float l) {  // hf: o[.][2 hf..2 hf + 1]
    float* dst = p.raw_part + (row0 + r) * (D + 4);
#pragma unroll
    for (int n = 0; n < NN; ++n)
      *reinterpret_cast<float2*>(dst + 4 + 8 * n + 2 * tq) = make_float2(o[n][2 * hf], o[n][2 * hf + 1]);
    if (tq == 0) *reinterpret_cast<float2*>(dst) = make_float2(m, l);
  };
  if (ca >= 0) store(ra, 0, ma, la);
  if (cb >= 0) store(rb, 1, mb, lb);
}

// ---- the merge -------------------------------------------------------------------------------
// A warp takes one, or in large calls two neighbouring, (sequence, new token, query head) rows: the
// cache partials of the row's tile are summed with their weights and rotated back [R is orthonormal
// and symmetric], the raw partial joins in the original basis.  Rows past a sequence's new tokens are
// not written.  Two rows a warp cover each other's load latency (a 2 x 2048-token chunk 81 -> 64 us);
// where all warps fit the SMs at once one row a warp is quicker (8 nodes 7 -> 6 us).
template <int D, int kRows>
__global__ void __launch_bounds__(128) block_merge_kernel(BlockParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t gw0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * kRows;
  const int64_t step = (int64_t)p.tile_rows * (D + 4);
  const int64_t all_slots = kBlockCtas + (int64_t)p.batch * p.num_kv_heads * p.tiles;
  bool live[kRows];
  const float* raw[kRows];   // the row's raw partial
  const float* base[kRows];  // its first cache partial
  int slots[kRows];
  const int2* info_at[kRows];  // its row tile's slots, null where no sealed page is seen
  // The lengths come from before block_raw_kernel, which waited for their writer: they are read ahead
  // of the wait for the partials.
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t gw = gw0 + i;
    info_at[i] = nullptr;
    live[i] = gw < (int64_t)p.batch * p.block * p.num_q_heads;
    slots[i] = 0;
    base[i] = p.part;
    raw[i] = p.raw_part;
    if (!live[i]) continue;
    const int hq = (int)(gw % p.num_q_heads);
    const int64_t bc = gw / p.num_q_heads;
    const int b = (int)(bc / p.block), c = (int)(bc - (int64_t)b * p.block);
    const int len = blk::cached_len(p, b), nl = blk::new_len(p, b);
    live[i] = c < nl;
    if (!live[i]) continue;
    const int h = hq / p.group;
    const int r = c * p.group + (hq - h * p.group);
    const int t = r / p.tile_rows;
    const int64_t row = ((int64_t)b * p.num_kv_heads + h) * p.tiles + t;
    const int64_t in_tile = (int64_t)(r - t * p.tile_rows) * (D + 4);
    raw[i] += row * step + in_tile;
    base[i] += in_tile;
    if (blk::tile_span(p, len, nl, t).count > 0) info_at[i] = p.row_info + row;
  }
  grid_dependency_wait();
  grid_launch_dependents();
  int2 info[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) info[i] = info_at[i] != nullptr ? *info_at[i] : make_int2(0, 0);
  float2 rml[kRows];
  float ro[kRows][E], v[kRows][E], M[kRows], l[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    rml[i] = make_float2(-INFINITY, 0.0f);
    if (live[i]) rml[i] = *reinterpret_cast<const float2*>(raw[i]);
#pragma unroll
    for (int e = 0; e < E; ++e) ro[i][e] = v[i][e] = 0.0f;
    if (live[i]) load_f32<E>(raw[i] + 4 + lane * E, ro[i]);
    M[i] = rml[i].x;
    l[i] = 0.0f;
  }
  int most = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    // checked: a CTA of the cache kernel whose waits ran out may leave its entries unwritten
    if (info[i].y > 0 && info[i].x >= 0 && (int64_t)info[i].x + info[i].y <= all_slots) {
      slots[i] = info[i].y;
      base[i] += (int64_t)info[i].x * step;
      most = max(most, slots[i]);
    }
  }
#pragma unroll 2
  for (int s = 0; s < most; ++s) {
    float2 ml[kRows];
    float o[kRows][E];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      ml[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.0f;
      if (s < slots[i]) {
        ml[i] = *reinterpret_cast<const float2*>(base[i] + s * step);
        load_f32<E>(base[i] + s * step + 4 + lane * E, o[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      // a partial that saw no token; one whose logits are NaN has no maximum either, but its sum is NaN
      if (ml[i].x == -INFINITY && ml[i].y == 0.0f) continue;
      const float mn = fmaxf(M[i], ml[i].x);
      const float keep = M[i] == -INFINITY ? 0.0f : exp2f(M[i] - mn), w = exp2f(ml[i].x - mn);
      M[i] = mn;
      l[i] = fmaf(l[i], keep, w * ml[i].y);
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = fmaf(v[i][e], keep, w * o[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (slots[i] > 0) warp_fwht<D>(v[i], lane);
    const float wr = rml[i].x == -INFINITY ? 0.0f : exp2f(rml[i].x - M[i]);
    const float sum = fmaf(wr, rml[i].y, l[i]);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    if (!live[i]) continue;
    __half* dst = p.out + (gw0 + i) * p.d0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = lane * E + e;
      if (j < p.d0) dst[j] = __float2half_rn(fmaf(v[i][e], inv_sqrt_d<D>(), wr * ro[i][e]) * inv);
    }
  }
}

// ---- launches --------------------------------------------------------------------------------
template <int D, int NR>
static int launch_block_t(const BlockParams& p, cudaStream_t stream) {
  using S = blk::Shape<D, NR>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  {
    constexpr int kSmem = 2 * 2 * 64 * 2 * D + 128 * 2 * D;  // two stages of K and V rows, the queries
    static PerDeviceOnce once;
    const void* fn = reinterpret_cast<const void*>(block_raw_kernel<D>);
    if (const int st = set_smem_limit(once, fn, kSmem); st != KVARN_OK) return st;
    cfg.gridDim = dim3((unsigned)(((int64_t)p.block * p.group + 127) / 128), p.num_kv_heads, p.batch);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = kSmem;
    if (cudaLaunchKernelEx(&cfg, block_raw_kernel<D>, p) != cudaSuccess) return KVARN_ERR_CUDA;
  }
  {
    const int rec = record_layout(D, p.kb, p.vb).bytes;
    int slots = (blk::kSmemMax - S::kRecOff) / rec;
    slots = slots > blk::kMaxSlots ? blk::kMaxSlots : slots;
    if (slots < 2) return KVARN_ERR_UNSUPPORTED;
    static PerDeviceOnce once;
    const void* fn = reinterpret_cast<const void*>(block_cache_kernel<D, NR>);
    if (const int st = set_smem_limit(once, fn, blk::kSmemMax); st != KVARN_OK) return st;
    cfg.gridDim = dim3(kBlockCtas);
    cfg.blockDim = dim3(blk::kThreads);
    cfg.dynamicSmemBytes = S::kRecOff + slots * rec;
    if (cudaLaunchKernelEx(&cfg, block_cache_kernel<D, NR>, p, slots) != cudaSuccess) return KVARN_ERR_CUDA;
  }
  const int64_t rows = (int64_t)p.batch * p.block * p.num_q_heads;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  if (rows <= 4096) {  // 27 warps an SM
    cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
    return cudaLaunchKernelEx(&cfg, block_merge_kernel<D, 1>, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
  }
  cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
  return cudaLaunchKernelEx(&cfg, block_merge_kernel<D, 2>, p) == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

// The least tile that holds the rows, or 64 rows a tile: QK, PV, the softmax and B follow the rows of
// a tile, the K and V conversion does not.  Tiles of 48 rows against tiles of 64: 40 rows of 32
// sequences over 8k, head_dim 128, 186 -> 168 us; 33 rows of 8 sequences, head_dim 64, 42.5 -> 37.7 us.
// head_dim 256 has tensor memory for 32 rows, and with 12 bits a code pair shared memory for 16.
int block_tile_rows(int d, int64_t rows, int kb, int vb) {
  const int most = d <= 128 ? 64 : (kb + vb > 8 ? 16 : 32);
  return rows < most ? (int)((rows + 15) / 16 * 16) : most;
}

int launch_block_attention(int d, const BlockParams& p, cudaStream_t stream) {
  if (d == 64) {
    if (p.tile_rows == 16) return launch_block_t<64, 16>(p, stream);
    if (p.tile_rows == 32) return launch_block_t<64, 32>(p, stream);
    if (p.tile_rows == 48) return launch_block_t<64, 48>(p, stream);
    if (p.tile_rows == 64) return launch_block_t<64, 64>(p, stream);
  } else if (d == 128) {
    if (p.tile_rows == 16) return launch_block_t<128, 16>(p, stream);
    if (p.tile_rows == 32) return launch_block_t<128, 32>(p, stream);
    if (p.tile_rows == 48) return launch_block_t<128, 48>(p, stream);
    if (p.tile_rows == 64) return launch_block_t<128, 64>(p, stream);
  } else if (d == 256) {
    if (p.tile_rows == 16) return launch_block_t<256, 16>(p, stream);
    if (p.tile_rows == 32) return launch_block_t<256, 32>(p, stream);
  }
  return KVARN_ERR_UNSUPPORTED;
}

}  // namespace kvarn
