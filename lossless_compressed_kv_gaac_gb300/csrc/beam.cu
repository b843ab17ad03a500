// A beam search's selection over beams and vocabulary.
//
//   c(i, t) = score_i + x_it - ln sum_u exp x_iu,   the n_out largest over (i, t), ties to the lowest i * vocab + t.
//
// The logits are read once, in one launch:
//  1. A CTA takes up to kBmMostTiles runs of kBmTile consecutive logits of one beam, 32 a thread and run, the next run's loads
//     under way while one is worked on.  They give its part of the sum and its n_out largest logits: within a beam the order
//     of the logits is that of the candidates, so no candidate beyond these can be among the chosen.  The n_out-th largest
//     of the maxima of 32 groups of threads of the first run (for n_out > 32 of 64, half of them from either half) is a bound that at
//     least n_out logits reach.  Those of all runs that do, some tens, are put side by side in shared memory and ranked by
//     counting, after the first run too, which leaves the others the n_out-th largest itself for a bound.  A run that has more
//     of them than there is room for (logits that are all alike, or sorted) is searched for its largest one at a time.
//  2. The last CTA of a search adds up the sums in 64 bits, in a fixed order, and merges the sorted lists: the largest of
//     their heads is taken n_out times, by one warp.  The other searches are read meanwhile.
// Bound by its instructions and barriers where there is much to read: 32 searches of 8 beams, 128,511 bf16 logits at odd addresses,
// n_out 16, 66 MB: 38.5 us (490 instructions for 32 logits of a warp's lanes, of which the sum takes 110, loads and widening 100, the
// candidates 150).  Rows that rise all along, which every run searches, 515 us; five tokens left by a mask 575, one in a hundred 39.
// What it was: every CTA one run and the choice a launch of its own, 104 us; odd rows put together from
// aligned vectors of neighbouring lanes, 72 us; the bound by taking the largest maximum n_out times in place of a sort, 5 us
// more; the choice in a second launch, 8 us more.  One search of 4 beams, 32,000 fp32 logits: 7.7 us.
// Order: logits as unsigned numbers of the same order, the lower token first where they are equal; in the merge the
// candidate to 48 bits, so that logits that differ stay apart, then the lower i * vocab + t.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "f32x2.cuh"
#include "kv8.cuh"

namespace gaac {

constexpr int kBmThreads = 256;
constexpr int kBmPer = 32;                        // logits of a thread
constexpr int kBmTile = kBmThreads * kBmPer;
constexpr int kBmMostTiles = 8;                   // runs of a CTA
constexpr int kBmCtasPerSm = 2;                   // three spill: 87 us in place of 35
constexpr int kBmRoom = 512;                      // logits that are ranked by counting
constexpr int kBmMostOut = 64;
constexpr int kBmMostBeams = 32;
constexpr int kBmMostVocab = 1 << 20;
constexpr int kBmStage = 36 * 1024;               // bytes of candidates that a merge holds in shared memory
constexpr uint32_t kBmAll = 0xFFFFFFFFu;
constexpr uint32_t kBmLowest = 0x007FFFFFu;       // -infinity in the order of bm_order

struct BeamArgs {
  const char* logits;
  int64_t row;                // bytes between beams
  const float* scores;
  const uint8_t* ended;       // nullptr: none
  int end_token, beams, vocab, n_out, chunks, tiles;  // chunks of a beam, of so many runs each
  float2* sums;               // [beam][chunk]: maximum, sum of exp(x - maximum)
  int32_t* tickets;           // [search]: CTAs that are done, 0 between calls
  int staged;                 // a merge's candidates fit in shared memory
  uint64_t* lists;            // [beam][chunk][n_out]: order of the logit << 32 | ~token, descending; 0 behind the last
  float* out_scores;
  int32_t* parents;
  int32_t* tokens;
};

// Unsigned numbers in the order of x; zeros of both signs are equal, NaN counts as -infinity.
__device__ __forceinline__ uint32_t bm_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x != x ? kBmLowest : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float bm_value(uint32_t u) { return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u); }
// The exact sum of two numbers as the nearest one and what that leaves (Knuth).
__device__ __forceinline__ float2 bm_two_sum(float x, float y) {
  const float s = __fadd_rn(x, y), b = __fsub_rn(s, x);
  return make_float2(s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(y, b)));
}
// A beam's candidates: (x - peak) + hi + lo, the largest logit first so that its size takes nothing from the others.
struct BmShift {
  float peak, hi, lo;
};
// A candidate as a place in an order: its value to 48 bits, as the nearest fp32 number and what that leaves (64-bit arithmetic takes 16
// cycles an instruction and more on this GPU).
__device__ __forceinline__ uint64_t bm_candidate(float x, const BmShift& a) {
  const float2 d = bm_two_sum(x, -a.peak), c = bm_two_sum(d.x, a.hi);
  const float e = __fadd_rn(__fadd_rn(c.y, d.y), a.lo), r = __fadd_rn(c.x, e);
  if (!(fabsf(r) < INFINITY)) return static_cast<uint64_t>(bm_order(r)) << 32;
  return static_cast<uint64_t>(bm_order(r)) << 32 | bm_order(__fsub_rn(e, __fsub_rn(r, c.x)));
}

__device__ __forceinline__ float bm_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float bm_max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// The head of a list as a candidate: its place in the order (0: none), and i * vocab + t.
struct BmHead {
  uint64_t c;
  uint32_t at;
};
__device__ __forceinline__ bool bm_before(const BmHead& x, const BmHead& y) { return x.c > y.c || (x.c == y.c && x.at < y.at); }

// The largest of a warp's heads, in every lane.
__device__ __forceinline__ BmHead bm_warp_best(BmHead h) {
  const uint32_t hi = static_cast<uint32_t>(h.c >> 32), lo = static_cast<uint32_t>(h.c);
  const uint32_t mh = __reduce_max_sync(kBmAll, hi);
  const uint32_t ml = __reduce_max_sync(kBmAll, hi == mh ? lo : 0u);
  const uint32_t at = __reduce_min_sync(kBmAll, hi == mh && lo == ml ? h.at : ~0u);
  return BmHead{static_cast<uint64_t>(mh) << 32 | ml, at};
}

// The choice of one search, by the CTA that was the last to read its logits.
__device__ __noinline__ void beam_merge(const BeamArgs& a, int64_t search) {
  constexpr int kWarps = kBmThreads / 32;
  const bool staged = a.staged;
  extern __shared__ uint64_t stage[];
  __shared__ BmShift shift[kBmMostBeams];
  __shared__ int kind[kBmMostBeams];                             // of a beam
  __shared__ uint8_t taken[kBmMostBeams * (kBmMostVocab / kBmTile)];  // of each list
  enum { kAlive, kEnded, kDead };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = search * a.beams;
  const uint64_t* lists = a.lists + first * a.chunks * a.n_out;
  const int n_lists = a.beams * a.chunks;
  for (int l = tid; l < n_lists; l += kBmThreads) taken[l] = 0;
  for (int i = warp; i < a.beams; i += kWarps) {
    const bool end = a.ended != nullptr && a.ended[first + i];
    const float s = a.scores[first + i];
    double log_total = 0.0;  // of the sum relative to the peak
    float m = 0.f;
    if (!end) {
      const float2* p = a.sums + (first + i) * a.chunks;
      m = -INFINITY;
      for (int j = lane; j < a.chunks; j += 32) m = fmaxf(m, __ldcg(&p[j].x));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kBmAll, m, d));
      double total = 0.0;
      for (int j = lane; j < a.chunks; j += 32) {
        const float2 v = __ldcg(p + j);
        total += static_cast<double>(v.y) * static_cast<double>(expf(v.x - m));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kBmAll, total, d);
      // ln(total) from its exponent in 64 bits and the fp32 logarithm of its mantissa in [0.75, 1.5), which is off by 2^-25
      const float t = static_cast<float>(total);
      if (t > 0.f && t < INFINITY) {
        const int e = static_cast<int>((__float_as_uint(t) - 0x3F400000u)) >> 23;
        log_total = e * 0.693147180559945309 + static_cast<double>(logf(__uint_as_float(__float_as_uint(t) - (static_cast<uint32_t>(e) << 23))));
      } else {
        log_total = t == 0.f ? -INFINITY : NAN;
      }
    }
    if (lane == 0) {
      const double d = s - log_total;
      shift[i] = BmShift{m, static_cast<float>(d), static_cast<float>(d - static_cast<float>(d))};
      // without a finite score and, unless it has ended, a finite sum, every candidate counts as -infinity
      kind[i] = !isfinite(s) || (!end && !(isfinite(log_total) && isfinite(m))) ? kDead : end ? kEnded : kAlive;
    }
  }
  __syncthreads();
  // Candidate k of list l, which is of beam i.  Those at -infinity come in the order of their tokens; a beam that is dead has no
  // others, one that has ended the end token before them: their lists are made up in the first chunk's place.
  auto candidate = [&](int l, int i, int k) {
    BmHead h{0, ~0u};
    if (kind[i] != kAlive) {
      int t = k;
      if (kind[i] == kEnded) t = k == 0 ? a.end_token : k - 1 < a.end_token ? k - 1 : k;
      if (l == i * a.chunks && t < a.vocab) {
        h.c = kind[i] == kEnded && k == 0 ? bm_candidate(0.f, shift[i]) : static_cast<uint64_t>(kBmLowest) << 32;
        h.at = static_cast<uint32_t>(i) * a.vocab + t;
      }
    } else {
      const uint64_t e = __ldcg(lists + static_cast<int64_t>(l) * a.n_out + k);
      if (e != 0) {
        h.c = bm_candidate(bm_value(static_cast<uint32_t>(e >> 32)), shift[i]);
        h.at = static_cast<uint32_t>(i) * a.vocab + ~static_cast<uint32_t>(e);
      }
    }
    return h;
  };
  // All of them at once where there is room, else one by one as they are wanted.
  const int all = n_lists * a.n_out;
  uint32_t* const stage_at = reinterpret_cast<uint32_t*>(stage + all);
  if (staged) {
#pragma unroll 4
    for (int j = tid; j < all; j += kBmThreads) {
      const int l = j / a.n_out;
      const BmHead h = candidate(l, l / a.chunks, j - l * a.n_out);
      stage[j] = h.c;
      stage_at[j] = h.at;
    }
    __syncthreads();
  }
  if (warp != 0) return;
  BmHead mine{0, ~0u};
  int of = -1;  // the list that it is from
  auto look = [&]() {  // the best head of lists lane, lane + 32, ...
    mine = BmHead{0, ~0u};
    for (int l = lane; l < n_lists; l += 32) {
      const int k = taken[l];
      if (k == a.n_out) continue;
      const BmHead h = staged ? BmHead{stage[l * a.n_out + k], stage_at[l * a.n_out + k]} : candidate(l, l / a.chunks, k);
      if (bm_before(h, mine)) {
        mine = h;
        of = l;
      }
    }
  };
  uint64_t got_c[2] = {0, 0};  // choices lane and lane + 32
  uint32_t got_at[2] = {0, 0};
  auto keep = [&](int r, const BmHead& b) {
    if (lane == r) got_c[0] = b.c, got_at[0] = b.at;
    if (lane + 32 == r) got_c[1] = b.c, got_at[1] = b.at;
  };
  if (staged && n_lists <= 32) {  // a list to a lane, its next candidate in registers
    const int from = lane * a.n_out, end = lane < n_lists ? from + a.n_out : from;
    int at = from;
    mine = at < end ? BmHead{stage[at], stage_at[at]} : BmHead{0, ~0u};
    BmHead after = at + 1 < end ? BmHead{stage[at + 1], stage_at[at + 1]} : BmHead{0, ~0u};
    for (int r = 0; r < a.n_out; ++r) {
      const BmHead b = bm_warp_best(mine);
      keep(r, b);
      if (mine.at == b.at) {  // places are distinct
        mine = after;
        ++at;
        after = at + 1 < end ? BmHead{stage[at + 1], stage_at[at + 1]} : BmHead{0, ~0u};
      }
    }
  } else {
    look();
    for (int r = 0; r < a.n_out; ++r) {
      const BmHead b = bm_warp_best(mine);
      keep(r, b);
      if (of >= 0 && mine.at == b.at) {
        ++taken[of];
        look();
      }
      __syncwarp();
    }
  }
  for (int r = lane, k = 0; r < a.n_out; r += 32, ++k) {
    const int64_t at = search * a.n_out + r;
    a.out_scores[at] = bm_value(static_cast<uint32_t>((k ? got_c[1] : got_c[0]) >> 32));
    const uint32_t place = k ? got_at[1] : got_at[0];
    a.parents[at] = static_cast<int32_t>(place / a.vocab);
    a.tokens[at] = static_cast<int32_t>(place % a.vocab);
  }
}

// A thread's part of a run: kBmPer logits in loads of E each, kBmThreads * E apart.  E is 16 bytes' worth where all rows of the
// call lie so, 2 for 16-bit logits on 4-byte boundaries, else 1: what decides is the same for all rows, so that equal rows have equal
// sums whatever their places in memory.  (Vectors on 16-byte boundaries of every row, put together from two lanes' where a row
// begins between them, took 230 instructions a run, single loads take 32.)
template <typename T, int E>
struct BmRun {
  static constexpr bool kPacked = sizeof(T) == 2 && E >= 2;        // two logits to a word
  static constexpr int kWords = kPacked ? kBmPer / 2 : kBmPer, kLoads = kBmPer / E;
  uint32_t w[kWords];

  static __device__ __forceinline__ int token(int tile, int i) { return tile * kBmTile + (i / E * kBmThreads + static_cast<int>(threadIdx.x)) * E + i % E; }
  static __device__ __forceinline__ uint32_t one(const char* p) {
    if (sizeof(T) == 4) return __ldcs(reinterpret_cast<const uint32_t*>(p));
    return __ldcs(reinterpret_cast<const uint16_t*>(p));
  }
  static __device__ __forceinline__ float widen(uint32_t bits) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
    if constexpr (std::is_same<T, __half>::value) return kv8_pair<true>(bits).x;
    return __uint_as_float(bits << 16);
  }
  // Tokens of run `tile`; those behind the vocabulary are -infinity.
  __device__ __forceinline__ void load(const char* row, int tile, int vocab) {
    const char* const p = row + (static_cast<int64_t>(tile) * kBmTile + threadIdx.x * E) * static_cast<int64_t>(sizeof(T));
    const uint32_t low = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00u : 0xFF80u;
    const bool whole = (tile + 1) * kBmTile <= vocab;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const char* const q = p + j * kBmThreads * E * static_cast<int>(sizeof(T));
      const int left = vocab - token(tile, j * E);  // of this load's tokens
      if constexpr (E * sizeof(T) == 16) {
        uint4 v = make_uint4(low, low, low, low);
        if (sizeof(T) == 2) v = make_uint4(low * 0x10001u, low * 0x10001u, low * 0x10001u, low * 0x10001u);
        uint32_t* const to = w + j * 4;
        if (whole || left >= E) v = __ldcs(reinterpret_cast<const uint4*>(q));
        to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
        if (!whole && left > 0 && left < E) {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (i < left) {
              const uint32_t x = one(q + i * sizeof(T));
              if (sizeof(T) == 4)
                to[i % 4] = x;
              else
                to[i / 2] = i % 2 ? (to[i / 2] & 0xFFFFu) | x << 16 : (to[i / 2] & 0xFFFF0000u) | x;
            }
        }
      } else if constexpr (E == 2) {
        w[j] = low * 0x10001u;
        if (whole || left >= 2)
          w[j] = __ldcs(reinterpret_cast<const uint32_t*>(q));
        else if (left == 1)
          w[j] = low << 16 | one(q);
      } else {
        w[j] = whole || left > 0 ? one(q) : low;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (kPacked) return i % 2 ? (std::is_same<T, __half>::value ? kv8_pair<true>(w[i / 2]).y : __uint_as_float(w[i / 2] & 0xFFFF0000u)) : widen(w[i / 2] & 0xFFFFu);
    return widen(w[i]);
  }
  // The largest of logits 8 g .. 8 g + 7.
  __device__ __forceinline__ float top(int g) const {
    if constexpr (kPacked) {
      uint32_t x = w[4 * g];
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        if (std::is_same<T, __half>::value)
          asm("max.f16x2 %0, %0, %1;" : "+r"(x) : "r"(w[4 * g + i]));
        else
          asm("max.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(w[4 * g + i]));
      }
      const float2 f = kv8_pair<std::is_same<T, __half>::value>(x);
      return fmaxf(f.x, f.y);
    }
    float m = fmaxf(get(8 * g), get(8 * g + 1));
#pragma unroll
    for (int i = 2; i < 8; i += 2) m = bm_max3(m, get(8 * g + i), get(8 * g + i + 1));
    return m;
  }
};

// The k-th largest (k >= 1) of the lanes' numbers: a bitonic sort, largest first.
__device__ __forceinline__ uint32_t bm_kth(uint32_t x, int k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d > 0; d /= 2) {
      const uint32_t y = __shfl_xor_sync(kBmAll, x, d);
      x = ((lane & d) == 0) == ((lane & size) == 0) ? max(x, y) : min(x, y);
    }
  return __shfl_sync(kBmAll, x, k - 1);
}

template <typename T, int E>
__global__ void __launch_bounds__(kBmThreads, kBmCtasPerSm) beam_chunk_kernel(const BeamArgs a) {
  using Run = BmRun<T, E>;
  constexpr int kWarps = kBmThreads / 32;
  __shared__ uint32_t rep[2 * kBmMostBeams];
  __shared__ float warp_sum[kWarps], warp_base[kWarps];
  __shared__ int count[kBmMostTiles];  // logits that reach the bound, of each run
  __shared__ uint64_t found[kBmRoom];
  __shared__ uint64_t best[2][kWarps];
  __shared__ int last;
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t beam = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks);
  const int64_t search = beam / a.beams;
  // One more CTA of the search is done; the last one makes the choice.  Everybody's stores come before thread 0's release by the
  // barrier, and what the others released before what follows.
  auto done = [&]() {
    __syncthreads();
    if (tid == 0) {
      const unsigned all = static_cast<unsigned>(a.beams) * a.chunks;
      last = kv8_atomic_add_acq_rel(a.tickets + search, 1u) == all - 1;
      if (last) a.tickets[search] = 0;
    }
    __syncthreads();
    if (last) beam_merge(a, search);
  };
  if (a.ended != nullptr && a.ended[beam]) return done();  // its candidate needs no logits
  const char* const begin = a.logits + beam * a.row;
  uint64_t* const list = a.lists + (beam * a.chunks + chunk) * a.n_out;
  const int first = chunk * a.tiles, end = min(first + a.tiles, (a.vocab + kBmTile - 1) / kBmTile);
  if (tid < kBmMostTiles) count[tid] = 0;
  float base = -INFINITY, sum = 0.f;  // this thread's sum of exp(x - base)
  float floor = 0.f;            // the bound as a number
  uint64_t least = 0;           // of a key that is still looked at
  Run next;
  next.load(begin, first, a.vocab);
  int taken = 0;  // keys in `found`, the same for all threads
#pragma unroll 1
  for (int tile = first; tile < end; ++tile) {
    const Run now = next;
    if (tile + 1 < end) next.load(begin, tile + 1, a.vocab);
    float m[4], top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      m[g] = now.top(g);
      top = fmaxf(top, m[g]);
    }
    if (tile == first) {
      // ---- maxima of groups of threads; the n_out-th largest of them, by every warp
      uint32_t g = bm_order(top);
      const int reps = a.n_out > 32 ? 64 : 32;
      for (int d = 1; d < kBmThreads / reps; d *= 2) g = max(g, __shfl_xor_sync(kBmAll, g, d));
      if (lane % (kBmThreads / reps) == 0) rep[tid / (kBmThreads / reps)] = g;
      __syncthreads();
      const uint32_t r0 = rep[lane], r1 = reps == 64 ? rep[32 + lane] : 0u;
      const uint32_t peak = __reduce_max_sync(kBmAll, max(r0, r1));
      uint32_t bound;
      if (reps == 32) {
        bound = bm_kth(r0, a.n_out);
      } else {  // as many of either half: the smaller of the two is reached by all of these
        bound = min(bm_kth(r0, (a.n_out + 1) / 2), bm_kth(r1, (a.n_out + 1) / 2));
      }
      least = static_cast<uint64_t>(bound) << 32;
      floor = bm_value(bound);
      base = bm_value(peak);
    }
    // ---- the sum.  The difference first: a product with log2(e) would be off by the last bit of a large logit.
    // The base is this thread's largest logit so far: an exponent's error grows with the distance from it (with a base that
    // rose by steps of 60 only, a peak in a later run took 3e-6 of the sum), and what is far below has no weight.
    if (top > base) {  // rare behind the first run, whose peak all threads begin with
      sum *= bm_exp2((base - top) * 1.44269504f);
      base = top;
    }
    const uint64_t minus = f2_all(base == -INFINITY ? 0.f : -base), scale = f2_all(1.44269504f);
    uint64_t part[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kBmPer; i += 2) {
      const float2 e = f2_get(f2_mul(f2_add(f2_make(now.get(i), now.get(i + 1)), minus), scale));
      part[i / 2 & 1] = f2_add(part[i / 2 & 1], f2_make(bm_exp2(e.x), bm_exp2(e.y)));
    }
    sum += f2_sum(f2_add(part[0], part[1]));
    // ---- logits that reach the bound
    auto key = [&](float x, int t) { return static_cast<uint64_t>(bm_order(x)) << 32 | static_cast<uint32_t>(~t); };
    if (top >= floor) {
      uint32_t hit = 0;  // which do, a bit for each
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (m[g] >= floor) {
#pragma unroll
          for (int i = 8 * g; i < 8 * g + 8; ++i) hit |= now.get(i) >= floor ? 1u << i : 0u;
        }
      while (hit != 0u) {  // few: their logits are read again
        const int e = __ffs(hit) - 1, t = Run::token(tile, e);
        hit &= hit - 1u;
        if (t >= a.vocab) continue;
        const uint64_t k = key(Run::widen(Run::one(begin + t * static_cast<int64_t>(sizeof(T)))), t);
        if (k < least) continue;
        const int at = taken + atomicAdd(&count[tile - first], 1);
        if (at < kBmRoom) found[at] = k;
      }
    }
    __syncthreads();
    int n = taken + count[tile - first];
    if (n > kBmRoom) {  // this run's n_out largest one by one, in the place of what it has left in `found`
      uint64_t below = ~0ull;  // what has been taken
      n = taken;
      for (int r = 0; r < a.n_out; ++r) {
        uint64_t b = 0;
#pragma unroll
        for (int i = 0; i < kBmPer; ++i) {
          const int t = Run::token(tile, i);
          const uint64_t k = key(now.get(i), t);
          if (t < a.vocab && k < below && k > b) b = k;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) b = max(b, static_cast<uint64_t>(__shfl_xor_sync(kBmAll, static_cast<unsigned long long>(b), d)));
        if (lane == 0) best[r & 1][warp] = b;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) b = max(b, best[r & 1][i]);
        if (b == 0) break;  // the same for all
        if (tid == 0) found[n] = b;
        ++n;
        below = b;
      }
      __syncthreads();
    }
    taken = n;
    // ---- with more runs to come: the n_out largest so far alone, and a bound that their ties behind them do not reach
    if (tile + 1 < end && n > a.n_out && (tile == first || n > kBmRoom - kBmMostOut)) {
      uint64_t k[kBmRoom / kBmThreads];
      int rank[kBmRoom / kBmThreads];
#pragma unroll
      for (int q = 0; q < kBmRoom / kBmThreads; ++q) {
        const int i = tid + q * kBmThreads;
        k[q] = i < n ? found[i] : 0;
        rank[q] = i < n ? 0 : kBmRoom;
        if (i < n)
          for (int j = 0; j < n; ++j) rank[q] += found[j] > k[q];
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kBmRoom / kBmThreads; ++q)
        if (rank[q] < a.n_out) found[rank[q]] = k[q];
      __syncthreads();
      taken = a.n_out;
      least = found[a.n_out - 1];
      floor = bm_value(static_cast<uint32_t>(least >> 32));
      __syncthreads();
    }
  }
  // ---- the list and the sum
  for (int i = tid; i < taken; i += kBmThreads) {
    const uint64_t k = found[i];
    int rank = 0;
    for (int j = 0; j < taken; ++j) rank += found[j] > k;
    if (rank < a.n_out) list[rank] = k;
  }
  if (tid >= taken && tid < a.n_out) list[tid] = 0;
  // Threads' bases differ where one has met larger logits than the first run's: all go to the largest.
  float high = base;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(kBmAll, high, d));
  if (base != high) sum *= bm_exp2((base - high) * 1.44269504f);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kBmAll, sum, d);
  if (lane == 0) warp_sum[warp] = sum, warp_base[warp] = high;
  __syncthreads();
  if (tid == 0) {
    high = warp_base[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) high = fmaxf(high, warp_base[i]);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += warp_base[i] == high ? warp_sum[i] : warp_sum[i] * bm_exp2((warp_base[i] - high) * 1.44269504f);
    a.sums[beam * a.chunks + chunk] = make_float2(high, sum);
  }
  done();
}

// Runs of a CTA: as many as leave every SM three CTAs, of which two run at a time, up to kBmMostTiles, the same for all CTAs of a
// beam as nearly as it goes (32 searches of 8 beams, 16 runs a beam: 38.5 us with eight runs, 42.4 with four).  Two CTAs in place of
// three: 64 rows of 50,257 bf16 logits 10.6 us for 13.1, but 128 of 128,256 23.3 for 21.1; four: 41.5 for 38.7 with 256 of 128,511.
static int beam_tiles(int64_t rows, int vocab) {
  const int64_t tiles = (vocab + kBmTile - 1) / kBmTile;
  const int64_t least = (tiles + kBmMostTiles - 1) / kBmMostTiles;
  const int64_t chunks = std::max(least, std::min<int64_t>(tiles, (152 * 3 + rows - 1) / rows));
  return static_cast<int>((tiles + chunks - 1) / chunks);
}
static int beam_chunks(int64_t rows, int vocab) {
  const int per = kBmTile * beam_tiles(rows, vocab);
  return (vocab + per - 1) / per;
}

}  // namespace gaac

using namespace gaac;

extern "C" size_t gaac_beam_workspace(int batch, int beams, int vocab, int n_out) {
  if (batch < 1 || beams < 1 || beams > kBmMostBeams || vocab < 1 || vocab > kBmMostVocab || n_out < 1 || n_out > kBmMostOut) return 0;
  const size_t lists = static_cast<size_t>(batch) * beams * beam_chunks(static_cast<int64_t>(batch) * beams, vocab);
  const size_t tickets = (static_cast<size_t>(batch) + 3) / 4 * 4 * sizeof(int32_t);
  return (tickets + lists * (sizeof(float2) + n_out * sizeof(uint64_t)) + 15) & ~static_cast<size_t>(15);
}

extern "C" int gaac_beam_select(const void* logits, int dtype, int64_t row_stride, const float* scores, const uint8_t* ended,
                                int end_token, int batch, int beams, int vocab, int n_out, float* out_scores, int32_t* parents,
                                int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream) {
  if ((dtype != GAAC_BF16 && dtype != GAAC_F16 && dtype != GAAC_F32) || batch < 0 || beams < 1 || beams > kBmMostBeams || vocab < 1 ||
      vocab > kBmMostVocab || n_out < 1 || n_out > kBmMostOut || n_out > static_cast<int64_t>(beams) * vocab)
    return GAAC_EINVAL;
  if (row_stride < vocab || row_stride > (int64_t{1} << 40) || (ended != nullptr && (end_token < 0 || end_token >= vocab))) return GAAC_EINVAL;
  if (batch == 0) return GAAC_OK;
  const uintptr_t size = dtype == GAAC_F32 ? 4 : 2;
  if (logits == nullptr || scores == nullptr || out_scores == nullptr || parents == nullptr || tokens == nullptr || workspace == nullptr ||
      (reinterpret_cast<uintptr_t>(logits) & (size - 1)) || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
      ((reinterpret_cast<uintptr_t>(scores) | reinterpret_cast<uintptr_t>(out_scores) | reinterpret_cast<uintptr_t>(parents) |
        reinterpret_cast<uintptr_t>(tokens)) & 3u))
    return GAAC_EINVAL;
  const int64_t rows = static_cast<int64_t>(batch) * beams;
  const int chunks = beam_chunks(rows, vocab);
  const int64_t ctas = static_cast<int64_t>(batch) * beams * chunks;
  if (ctas > 0x7FFFFFFF || workspace_bytes < gaac_beam_workspace(batch, beams, vocab, n_out)) return GAAC_EINVAL;
  BeamArgs a;
  a.logits = static_cast<const char*>(logits);
  a.row = row_stride * static_cast<int64_t>(size);
  a.scores = scores;
  a.ended = ended;
  a.end_token = end_token;
  a.beams = beams;
  a.vocab = vocab;
  a.n_out = n_out;
  a.chunks = chunks;
  a.tiles = beam_tiles(rows, vocab);
  a.tickets = static_cast<int32_t*>(workspace);
  a.lists = reinterpret_cast<uint64_t*>(a.tickets + (batch + 3) / 4 * 4);
  a.sums = reinterpret_cast<float2*>(a.lists + ctas * n_out);
  a.out_scores = out_scores;
  a.parents = parents;
  a.tokens = tokens;
  const dim3 grid(static_cast<unsigned>(ctas));
  // What all rows begin on, in bytes.
  const uintptr_t lie = reinterpret_cast<uintptr_t>(logits) | (rows > 1 ? static_cast<uintptr_t>(a.row) : 0u);
  const size_t bytes = static_cast<size_t>(beams) * chunks * n_out * (sizeof(uint64_t) + sizeof(uint32_t));
  a.staged = bytes <= kBmStage;
  auto launch = [&](auto* wide, auto* pairs, auto* single) {
    return kv8_launch((lie & 15u) == 0 ? wide : (lie & 3u) == 0 ? pairs : single, grid, kBmThreads, a.staged ? bytes : 0, stream, a);
  };
  return dtype == GAAC_F32   ? launch(beam_chunk_kernel<float, 4>, beam_chunk_kernel<float, 1>, beam_chunk_kernel<float, 1>)
         : dtype == GAAC_F16 ? launch(beam_chunk_kernel<__half, 8>, beam_chunk_kernel<__half, 2>, beam_chunk_kernel<__half, 1>)
                             : launch(beam_chunk_kernel<__nv_bfloat16, 8>, beam_chunk_kernel<__nv_bfloat16, 2>, beam_chunk_kernel<__nv_bfloat16, 1>);
}
