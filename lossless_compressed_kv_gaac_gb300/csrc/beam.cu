// A beam search's selection over beams and vocabulary.
//
//   c(i, t) = score_i + x_it - ln sum_u exp x_iu,   the n_out largest over (i, t), ties to the lowest i * vocab + t.
//
// Memory bound: the logits are read once.  Two launches:
//  1. A CTA takes up to kBmMostTiles runs of kBmTile consecutive logits of one beam, 32 a thread and run, the next run's loads
//     under way while one is worked on.  They give its part of the sum and its n_out largest logits: within a beam the order
//     of the logits is that of the candidates, so no candidate beyond these can be among the chosen.  The n_out-th largest
//     of the maxima of 32 (64 for n_out > 32) groups of threads of the first run is a bound that at least n_out logits
//     reach; those of all runs that do (some tens of each run) are put side by side in shared memory and ranked by counting.
//     A run that has more of them than there is room for (logits that are all alike, or sorted) is searched for its largest
//     one at a time instead.
//  2. A CTA for each search adds up the sums in 64 bits, a fixed order, and merges the sorted lists: the largest of
//     their heads is taken n_out times, by one warp.
// Order: logits as unsigned numbers of the same order, the lower token first where they are equal; in the merge the
// candidate in 64 bits, so that logits that differ stay apart, then the lower i * vocab + t.
#include <algorithm>
#include <cmath>

#include "f32x2.cuh"
#include "kv8.cuh"

namespace gaac {

constexpr int kBmThreads = 256;
constexpr int kBmPer = 32;                        // logits of a thread
constexpr int kBmTile = kBmThreads * kBmPer;
constexpr int kBmMostTiles = 4;                   // runs of a CTA
constexpr int kBmRoom = 512;                      // logits that are ranked by counting
constexpr int kBmMostOut = 64;
constexpr int kBmMostBeams = 32;
constexpr int kBmMostVocab = 1 << 20;
constexpr int kBmMerge = 128;                     // threads of a merge
constexpr int kBmStage = 96 * 1024;               // bytes of lists that a merge holds in shared memory
constexpr uint32_t kBmAll = 0xFFFFFFFFu;
constexpr uint32_t kBmLowest = 0x007FFFFFu;       // -infinity in the order of bm_order

struct BeamArgs {
  const char* logits;
  int64_t row;                // bytes between beams
  const float* scores;
  const uint8_t* ended;       // nullptr: none
  int end_token, beams, vocab, n_out, chunks, tiles;  // chunks of a beam, of so many runs each
  float2* sums;               // [beam][chunk]: maximum, sum of exp(x - maximum)
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
__device__ __forceinline__ uint64_t bm_order64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double bm_value64(uint64_t u) {
  return __longlong_as_double(static_cast<long long>((u >> 63) ? u & ~(1ull << 63) : ~u));
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

template <typename T>
struct BmVec;
template <>
struct BmVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(uint4 w, float* f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint32_t bits(const char* p) { return *reinterpret_cast<const uint32_t*>(p); }
};
template <bool HALF>
struct BmVec16 {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(uint4 w, float* f) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = kv8_pair<HALF>(x[i]);
      f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint32_t bits(const char* p) { return *reinterpret_cast<const uint16_t*>(p); }
};
template <>
struct BmVec<__half> : BmVec16<true> {};
template <>
struct BmVec<__nv_bfloat16> : BmVec16<false> {};

// A thread's tokens are the same whatever the row's alignment, so that equal rows have equal sums.  Loads lie on
// 16-byte boundaries, the row's first logit being number `skip` of vector 0; where that is not 0, tokens are put together
// from a vector and the next lane's (the last lane loads one more).
template <typename T>
struct BmRow {
  using Vec = BmVec<T>;
  static constexpr int kN = Vec::kN, kVecs = kBmPer / kN;
  const char* row;
  int skip, vocab;

  __device__ __forceinline__ uint4 one(int v) const {
    const int t = v * kN - skip;
    const char* p = row + static_cast<int64_t>(t) * static_cast<int64_t>(sizeof(T));
    if (t >= 0 && t + kN <= vocab) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (t + i >= 0 && t + i < vocab) w[i * sizeof(T) / 4] |= Vec::bits(p + i * sizeof(T)) << (i * sizeof(T) % 4 * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Vectors of run `tile`: one of kVecs at kBmThreads apart.
  __device__ __forceinline__ void load(int tile, uint4 (&w)[kVecs], uint4 (&more)[kVecs]) const {
    const int v0 = tile * (kBmTile / kN) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) w[j] = one(v0 + j * kBmThreads);
    if (skip != 0 && threadIdx.x % 32 == 31) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) more[j] = one(v0 + j * kBmThreads + 1);
    }
  }
  // Words of vector j with the row's alignment taken out.
  __device__ __forceinline__ void align(uint4& w, const uint4& more) const {
    const int lane = threadIdx.x & 31, bytes = skip * static_cast<int>(sizeof(T));
    uint32_t n[8] = {w.x, w.y, w.z, w.w, 0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[4 + i] = __shfl_down_sync(kBmAll, n[i], 1);
      if (lane == 31) n[4 + i] = i == 0 ? more.x : i == 1 ? more.y : i == 2 ? more.z : more.w;
    }
    if (bytes & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) n[i] = n[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) n[i] = n[i + 1];
    }
    if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = __funnelshift_r(n[i], n[i + 1], 16);
    }
    w = make_uint4(n[0], n[1], n[2], n[3]);
  }
};

template <typename T>
__global__ void __launch_bounds__(kBmThreads, 2) beam_chunk_kernel(const BeamArgs a) {
  using Row = BmRow<T>;
  using Vec = BmVec<T>;
  constexpr int kN = Vec::kN, kVecs = Row::kVecs, kWarps = kBmThreads / 32;
  __shared__ uint32_t rep[2 * kBmMostBeams];
  __shared__ float warp_sum[kWarps], warp_base[kWarps];
  __shared__ int count[kBmMostTiles];  // logits that reach the bound, of each run
  __shared__ uint64_t found[kBmRoom];
  __shared__ uint64_t best[2][kWarps];
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t beam = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks);
  if (a.ended != nullptr && a.ended[beam]) return;  // its candidate needs no logits
  const char* const begin = a.logits + beam * a.row;
  const Row row{begin, static_cast<int>((reinterpret_cast<uintptr_t>(begin) & 15u) / sizeof(T)), a.vocab};
  uint64_t* const list = a.lists + (beam * a.chunks + chunk) * a.n_out;
  const int first = chunk * a.tiles, end = min(first + a.tiles, (a.vocab + kBmTile - 1) / kBmTile);
  if (tid < kBmMostTiles) count[tid] = 0;
  float base = -INFINITY, sum = 0.f;  // this thread's sum of exp(x - base)
  float floor = 0.f;            // the bound as a number
  uint64_t least = 0;           // of a key that is still looked at
  uint4 w[kVecs], more[kVecs];
  row.load(first, w, more);
  int taken = 0;  // keys in `found`, the same for all threads
#pragma unroll 1
  for (int tile = first; tile < end; ++tile) {
    uint4 now[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (row.skip != 0) row.align(w[j], more[j]);
      now[j] = w[j];
    }
    if (tile + 1 < end) row.load(tile + 1, w, more);
    float x[kBmPer], m[kVecs];
    const int t0 = tile * kBmTile + tid * kN;  // token of element i: t0 + i / kN * kBmThreads * kN + i % kN
    const bool whole = (tile + 1) * kBmTile <= a.vocab;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      Vec::get(now[j], x + j * kN);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (t0 + j * kBmThreads * kN + i >= a.vocab) x[j * kN + i] = -INFINITY;
      }
      m[j] = x[j * kN];
#pragma unroll
      for (int i = 1; i + 1 < kN; i += 2) m[j] = bm_max3(m[j], x[j * kN + i], x[j * kN + i + 1]);
      m[j] = fmaxf(m[j], x[j * kN + kN - 1]);
    }
    float top = m[0];
#pragma unroll
    for (int j = 1; j < kVecs; ++j) top = fmaxf(top, m[j]);
    if (tile == first) {
      // ---- maxima of groups of threads; the n_out-th largest of them, by every warp
      uint32_t g = bm_order(top);
      g = max(g, __shfl_xor_sync(kBmAll, g, 1));
      g = max(g, __shfl_xor_sync(kBmAll, g, 2));
      const int reps = a.n_out > 32 ? 64 : 32;  // groups of 4 or of 8 threads
      if (reps == 32) g = max(g, __shfl_xor_sync(kBmAll, g, 4));
      if (lane % (kBmThreads / reps) == 0) rep[tid / (kBmThreads / reps)] = g;
      __syncthreads();
      uint32_t r0 = rep[lane], r1 = reps == 64 ? rep[32 + lane] : 0u, bound = 0, peak = 0;
      for (int left = a.n_out;;) {
        bound = __reduce_max_sync(kBmAll, max(r0, r1));
        if (peak == 0) peak = bound;
        left -= __popc(__ballot_sync(kBmAll, r0 == bound)) + (reps == 64 ? __popc(__ballot_sync(kBmAll, r1 == bound)) : 0);
        if (left <= 0) break;
        if (r0 == bound) r0 = 0;
        if (r1 == bound) r1 = 0;
      }
      least = static_cast<uint64_t>(bound) << 32;
      floor = bm_value(bound);
      base = bm_value(peak);
    }
    // ---- the sum.  The difference first: a product with log2(e) would be off by the last bit of a large logit.
    if (top > base + 60.f) {  // rare: what comes is far above the runs before, or the first that is finite
      sum *= bm_exp2((base - top) * 1.44269504f);
      base = top;
    }
    const uint64_t minus = f2_all(base == -INFINITY ? 0.f : -base), scale = f2_all(1.44269504f);
    uint64_t part[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kBmPer; i += 2) {
      const float2 e = f2_get(f2_mul(f2_add(f2_make(x[i], x[i + 1]), minus), scale));
      part[i / 2 & 1] = f2_add(part[i / 2 & 1], f2_make(bm_exp2(e.x), bm_exp2(e.y)));
    }
    sum += f2_sum(f2_add(part[0], part[1]));
    // ---- logits that reach the bound
    auto key = [&](int i) {
      return static_cast<uint64_t>(bm_order(x[i])) << 32 | static_cast<uint32_t>(~(t0 + i / kN * kBmThreads * kN + i % kN));
    };
    auto real = [&](int i) { return t0 + i / kN * kBmThreads * kN + i % kN < a.vocab; };
    if (top >= floor) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (m[j] >= floor) {
#pragma unroll
          for (int i = j * kN; i < (j + 1) * kN; ++i)
            if (x[i] >= floor && real(i) && key(i) >= least) {
              const int at = taken + atomicAdd(&count[tile - first], 1);
              if (at < kBmRoom) found[at] = key(i);
            }
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
          const uint64_t k = key(i);
          if (real(i) && k < below && k > b) b = k;
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
    if (tile + 1 < end && n > kBmRoom - kBmMostOut) {
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
  // Threads' bases differ where one has met far larger logits: all go to the largest.
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

__global__ void __launch_bounds__(kBmMerge) beam_merge_kernel(const BeamArgs a, int staged) {
  constexpr int kWarps = kBmMerge / 32;
  extern __shared__ uint64_t stage[];
  __shared__ double log_sum[kBmMostBeams], score[kBmMostBeams];
  __shared__ int kind[kBmMostBeams];                             // of a beam
  __shared__ uint8_t taken[kBmMostBeams * (kBmMostVocab / kBmTile)];  // of each list
  enum { kAlive, kEnded, kDead };
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.beams;
  const uint64_t* lists = a.lists + first * a.chunks * a.n_out;
  const int n_lists = a.beams * a.chunks;
  if (staged)
    for (int i = tid; i < n_lists * a.n_out; i += kBmMerge) stage[i] = __ldcg(lists + i);
  for (int l = tid; l < n_lists; l += kBmMerge) taken[l] = 0;
  for (int i = warp; i < a.beams; i += kWarps) {
    const bool end = a.ended != nullptr && a.ended[first + i];
    const float s = a.scores[first + i];
    double log_total = 0.0;
    if (!end) {
      const float2* p = a.sums + (first + i) * a.chunks;
      float m = -INFINITY;
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
      log_total += m;
    }
    if (lane == 0) {
      log_sum[i] = log_total;
      score[i] = s;
      // without a finite score and, unless it has ended, a finite sum, every candidate counts as -infinity
      kind[i] = !isfinite(s) || (!end && !isfinite(log_total)) ? kDead : end ? kEnded : kAlive;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  if (staged) lists = stage;
  // The next candidate of list l, which is of beam i.  Candidates at -infinity come in the order of their tokens; a beam that is
  // dead has no others, one that has ended the end token before them: their lists are made up in the first chunk's place.
  auto head = [&](int l, int i) {
    const int k = taken[l];
    BmHead h{0, ~0u};
    if (kind[i] != kAlive) {
      int t = k;
      if (kind[i] == kEnded) t = k == 0 ? a.end_token : k - 1 < a.end_token ? k - 1 : k;
      if (l == i * a.chunks && k < a.n_out && t < a.vocab) {
        h.c = bm_order64(kind[i] == kEnded && k == 0 ? score[i] : -INFINITY);
        h.at = static_cast<uint32_t>(i) * a.vocab + t;
      }
    } else if (k < a.n_out) {
      const uint64_t e = staged ? stage[l * a.n_out + k] : __ldcg(lists + static_cast<int64_t>(l) * a.n_out + k);
      if (e != 0) {
        h.c = bm_order64(score[i] + (static_cast<double>(bm_value(static_cast<uint32_t>(e >> 32))) - log_sum[i]));
        h.at = static_cast<uint32_t>(i) * a.vocab + ~static_cast<uint32_t>(e);
      }
    }
    return h;
  };
  BmHead mine{0, ~0u};
  int of = -1;  // the list that it is from
  auto look = [&]() {  // the best head of lists lane, lane + 32, ...
    mine = BmHead{0, ~0u};
    for (int l = lane; l < n_lists; l += 32) {
      const BmHead h = head(l, l / a.chunks);
      if (bm_before(h, mine)) {
        mine = h;
        of = l;
      }
    }
  };
  look();
  uint64_t got_c[2] = {0, 0};  // choices lane and lane + 32
  uint32_t got_at[2] = {0, 0};
  for (int r = 0; r < a.n_out; ++r) {
    const BmHead b = bm_warp_best(mine);
    if (lane == r) got_c[0] = b.c, got_at[0] = b.at;
    if (lane + 32 == r) got_c[1] = b.c, got_at[1] = b.at;
    if (of >= 0 && mine.at == b.at) {  // places are distinct
      ++taken[of];
      look();
    }
    __syncwarp();
  }
  for (int r = lane, k = 0; r < a.n_out; r += 32, ++k) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * a.n_out + r;
    a.out_scores[at] = static_cast<float>(bm_value64(k ? got_c[1] : got_c[0]));
    const uint32_t place = k ? got_at[1] : got_at[0];
    a.parents[at] = static_cast<int32_t>(place / a.vocab);
    a.tokens[at] = static_cast<int32_t>(place % a.vocab);
  }
}

// Runs of a CTA: as many as leave every SM three CTAs.
static int beam_tiles(int64_t rows, int vocab) {
  const int64_t tiles = (vocab + kBmTile - 1) / kBmTile;
  return static_cast<int>(std::min<int64_t>(std::min<int64_t>(kBmMostTiles, tiles), std::max<int64_t>(1, rows * tiles / (152 * 3))));
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
  return (lists * (sizeof(float2) + n_out * sizeof(uint64_t)) + 15) & ~static_cast<size_t>(15);
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
  a.lists = static_cast<uint64_t*>(workspace);
  a.sums = reinterpret_cast<float2*>(a.lists + ctas * n_out);
  a.out_scores = out_scores;
  a.parents = parents;
  a.tokens = tokens;
  const dim3 grid(static_cast<unsigned>(ctas));
  const int e = dtype == GAAC_F32   ? kv8_launch(beam_chunk_kernel<float>, grid, kBmThreads, 0, stream, a)
                : dtype == GAAC_F16 ? kv8_launch(beam_chunk_kernel<__half>, grid, kBmThreads, 0, stream, a)
                                    : kv8_launch(beam_chunk_kernel<__nv_bfloat16>, grid, kBmThreads, 0, stream, a);
  if (e != GAAC_OK) return e;
  const size_t bytes = static_cast<size_t>(beams) * chunks * n_out * sizeof(uint64_t);
  const bool staged = bytes <= kBmStage;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GAAC_ECUDA;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBmStage) != cudaSuccess) return GAAC_ECUDA;
    done[dev] = true;
  }
  return kv8_launch(beam_merge_kernel, dim3(batch), kBmMerge, staged ? bytes : 0, stream, a, staged ? 1 : 0);
}
