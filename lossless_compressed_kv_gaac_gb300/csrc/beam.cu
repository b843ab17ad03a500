// A beam search's selection over beams and vocabulary.
//
//   c(i, t) = score_i + x_it - ln sum_u exp x_iu,   the n_out largest over (i, t), ties to the lowest i * vocab + t.
//
// Memory bound: the logits are read once.  Two launches:
//  1. A CTA takes kBmChunk consecutive logits of one beam, 32 a thread, and keeps them in registers.  They give its part
//     of the sum (relative to its own maximum) and its n_out largest logits: within a beam the order of the logits is
//     that of the candidates, so no candidate beyond these can be among the chosen.  The n_out-th largest of the maxima
//     of 32 (64 for n_out > 32) groups of threads is a bound that at least n_out logits reach; some tens do, they are put
//     side by side in shared memory and ranked by counting.  Where more do than there is room for (logits that are all
//     alike, or sorted), the largest are taken one at a time.
//  2. A CTA for each search adds up the sums in 64 bits, a fixed order, and merges the sorted lists: the largest of
//     their heads is taken n_out times.
// Order: logits as unsigned numbers of the same order, the lower token first where they are equal; in the merge the
// candidate in 64 bits, so that logits that differ stay apart, then the lower i * vocab + t.
#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace gaac {

constexpr int kBmThreads = 256;
constexpr int kBmPer = 32;                        // logits of a thread
constexpr int kBmChunk = kBmThreads * kBmPer;
constexpr int kBmRoom = 512;                      // logits that are ranked by counting
constexpr int kBmMostOut = 64;
constexpr int kBmMostBeams = 32;
constexpr int kBmMostVocab = 1 << 20;
constexpr int kBmMerge = 256;                     // threads of a merge
constexpr int kBmStage = 96 * 1024;               // bytes of lists that a merge holds in shared memory
constexpr uint32_t kBmAll = 0xFFFFFFFFu;
constexpr uint32_t kBmLowest = 0x007FFFFFu;       // -infinity in the order of bm_order

struct BeamArgs {
  const char* logits;
  int64_t row;                // bytes between beams
  const float* scores;
  const uint8_t* ended;       // nullptr: none
  int end_token, beams, vocab, n_out, chunks;
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

template <typename T>
__global__ void __launch_bounds__(kBmThreads) beam_chunk_kernel(const BeamArgs a) {
  using Vec = BmVec<T>;
  constexpr int kN = Vec::kN, kVecs = kBmPer / kN, kWarps = kBmThreads / 32;
  __shared__ uint32_t rep[2 * kBmMostBeams];
  __shared__ float warp_sum[kWarps];
  __shared__ int count;
  __shared__ uint64_t found[kBmRoom];
  __shared__ uint64_t best[2][kWarps];
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t beam = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x % a.chunks);
  if (a.ended != nullptr && a.ended[beam]) return;  // its candidate needs no logits
  // A thread's tokens are the same whatever the row's alignment, so that equal rows have equal sums.  Loads lie on
  // 16-byte boundaries, the row's first logit being number `skip` of vector 0; where that is not 0, tokens are put
  // together from a vector and the next lane's.
  const char* const row = a.logits + beam * a.row;
  const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  auto load = [&](int v) {
    const int t = v * kN - skip;
    const char* p = row + static_cast<int64_t>(t) * static_cast<int64_t>(sizeof(T));
    if (t >= 0 && t + kN <= a.vocab) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (t + i >= 0 && t + i < a.vocab) w[i * sizeof(T) / 4] |= Vec::bits(p + i * sizeof(T)) << (i * sizeof(T) % 4 * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  float x[kBmPer];
  const int v0 = chunk * (kBmChunk / kN) + tid, t0 = v0 * kN;
  {
    uint4 w[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) w[j] = load(v0 + j * kBmThreads);
    if (skip != 0) {
      uint4 more[kVecs];  // the next vector
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (lane == 31) more[j] = load(v0 + j * kBmThreads + 1);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        uint32_t n[8] = {w[j].x, w[j].y, w[j].z, w[j].w, 0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n[4 + i] = __shfl_down_sync(kBmAll, n[i], 1);
          if (lane == 31) n[4 + i] = i == 0 ? more[j].x : i == 1 ? more[j].y : i == 2 ? more[j].z : more[j].w;
        }
        const int bytes = skip * static_cast<int>(sizeof(T));
#pragma unroll
        for (int i = 0; i < 6; ++i) n[i] = (bytes & 8) ? n[i + 2] : n[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) n[i] = (bytes & 4) ? n[i + 1] : n[i];
        if (sizeof(T) == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) n[i] = (bytes & 2) ? __funnelshift_r(n[i], n[i + 1], 16) : n[i];
        }
        w[j] = make_uint4(n[0], n[1], n[2], n[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      Vec::get(w[j], x + j * kN);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (t0 + j * kBmThreads * kN + i >= a.vocab) x[j * kN + i] = -INFINITY;
    }
  }
  if (tid == 0) count = 0;
  // ---- maxima: of the thread, of groups of threads
  float m = x[0];
#pragma unroll
  for (int i = 1; i < kBmPer; ++i) m = fmaxf(m, x[i]);
  const uint32_t mine = bm_order(m);
  uint32_t g = mine;
  g = max(g, __shfl_xor_sync(kBmAll, g, 1));
  g = max(g, __shfl_xor_sync(kBmAll, g, 2));
  const int reps = a.n_out > 32 ? 64 : 32;  // groups of 4 or of 8 threads
  if (reps == 32) g = max(g, __shfl_xor_sync(kBmAll, g, 4));
  if (lane % (kBmThreads / reps) == 0) rep[tid / (kBmThreads / reps)] = g;
  __syncthreads();
  // ---- the n_out-th largest of them, by every warp
  uint32_t r0 = rep[lane], r1 = reps == 64 ? rep[32 + lane] : 0u;
  uint32_t top = 0, bound = 0;
  for (int left = a.n_out;;) {
    bound = __reduce_max_sync(kBmAll, max(r0, r1));
    if (top == 0) top = bound;
    left -= __popc(__ballot_sync(kBmAll, r0 == bound)) + (reps == 64 ? __popc(__ballot_sync(kBmAll, r1 == bound)) : 0);
    if (left <= 0) break;
    if (r0 == bound) r0 = 0;
    if (r1 == bound) r1 = 0;
  }
  // ---- the sum
  // The difference first: a product with log2(e) would be off by the last bit of a large logit.
  const float peak = bm_value(top), base = peak == -INFINITY ? 0.f : peak;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kBmPer; ++i) sum += bm_exp2((x[i] - base) * 1.44269504f);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kBmAll, sum, d);
  if (lane == 0) warp_sum[warp] = sum;
  // ---- logits that reach the bound
  auto token = [&](int i) { return t0 + i / kN * kBmThreads * kN + i % kN; };
  auto key = [&](int i) { return static_cast<uint64_t>(bm_order(x[i])) << 32 | static_cast<uint32_t>(~token(i)); };
  auto real = [&](int i) { return token(i) < a.vocab; };
  if (mine >= bound) {
#pragma unroll
    for (int i = 0; i < kBmPer; ++i)
      if (bm_order(x[i]) >= bound && real(i)) {
        const int at = atomicAdd(&count, 1);
        if (at < kBmRoom) found[at] = key(i);
      }
  }
  __syncthreads();
  uint64_t* const list = a.lists + (beam * a.chunks + chunk) * a.n_out;
  const int n = count;
  if (n <= kBmRoom) {
    for (int i = tid; i < n; i += kBmThreads) {
      const uint64_t k = found[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += found[j] > k;
      if (rank < a.n_out) list[rank] = k;
    }
    if (n < a.n_out && tid >= n && tid < a.n_out) list[tid] = 0;
  } else {
    uint64_t below = ~0ull;  // what has been taken
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
      if (tid == 0) list[r] = b;
      below = b;
    }
  }
  if (tid == 0) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += warp_sum[i];
    a.sums[beam * a.chunks + chunk] = make_float2(peak, sum);
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
  __shared__ int kind[kBmMostBeams];                                // of a beam
  __shared__ uint8_t taken[kBmMostBeams * (kBmMostVocab / kBmChunk)];  // of each list
  __shared__ BmHead best[2][kWarps];
  enum { kAlive, kEnded, kDead };
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.beams;
  const uint64_t* lists = a.lists + first * a.chunks * a.n_out;
  const int n_lists = a.beams * a.chunks;
  for (int i = warp; i < a.beams; i += kWarps) {
    const bool end = a.ended != nullptr && a.ended[first + i];
    const float s = a.scores[first + i];
    double total = 0.0, m = -INFINITY;
    if (!end) {
      const float2* p = a.sums + (first + i) * a.chunks;
      for (int j = lane; j < a.chunks; j += 32) m = fmax(m, static_cast<double>(__ldcg(&p[j].x)));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmax(m, __shfl_xor_sync(kBmAll, m, d));
      for (int j = lane; j < a.chunks; j += 32) {
        const float2 v = __ldcg(p + j);
        if (v.y != 0.f) total += static_cast<double>(v.y) * exp(static_cast<double>(v.x) - m);  // NaN goes on
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kBmAll, total, d);
      m += log(total);
    }
    if (lane == 0) {
      log_sum[i] = m;
      score[i] = s;
      // without a finite score and, unless it has ended, a finite sum, every candidate counts as -infinity
      kind[i] = !isfinite(s) || (!end && !isfinite(m)) ? kDead : end ? kEnded : kAlive;
    }
  }
  if (staged) {
    for (int i = tid; i < n_lists * a.n_out; i += kBmMerge) stage[i] = __ldcg(lists + i);
    lists = stage;
  }
  for (int l = tid; l < n_lists; l += kBmMerge) taken[l] = 0;
  __syncthreads();
  // The next candidate of list l.  Candidates at -infinity come in the order of their tokens; a beam that is dead has
  // no others, one that has ended the end token before them: their lists are made up in the first chunk's place.
  auto head = [&](int l) {
    const int i = l / a.chunks, k = taken[l];
    BmHead h{0, ~0u};
    if (kind[i] != kAlive) {
      int t = k;
      if (kind[i] == kEnded) t = k == 0 ? a.end_token : k - 1 < a.end_token ? k - 1 : k;
      if (l % a.chunks == 0 && k < a.n_out && t < a.vocab) {
        h.c = bm_order64(kind[i] == kEnded && k == 0 ? score[i] : -INFINITY);
        h.at = static_cast<uint32_t>(i) * a.vocab + t;
      }
    } else if (k < a.n_out) {
      const uint64_t e = staged ? lists[l * a.n_out + k] : __ldcg(lists + static_cast<int64_t>(l) * a.n_out + k);
      if (e != 0) {
        h.c = bm_order64(score[i] + (static_cast<double>(bm_value(static_cast<uint32_t>(e >> 32))) - log_sum[i]));
        h.at = static_cast<uint32_t>(i) * a.vocab + ~static_cast<uint32_t>(e);
      }
    }
    return h;
  };
  BmHead mine{0, ~0u};
  int of = -1;  // the list that it is from
  auto look = [&]() {
    mine = BmHead{0, ~0u};
    for (int l = tid; l < n_lists; l += kBmMerge) {
      const BmHead h = head(l);
      if (bm_before(h, mine)) {
        mine = h;
        of = l;
      }
    }
  };
  look();
  for (int r = 0; r < a.n_out; ++r) {
    const BmHead w = bm_warp_best(mine);
    if (lane == 0) best[r & 1][warp] = w;
    __syncthreads();
    const BmHead b = bm_warp_best(lane < kWarps ? best[r & 1][lane] : BmHead{0, ~0u});
    if (tid == 0) {
      const int64_t at = static_cast<int64_t>(blockIdx.x) * a.n_out + r;
      a.out_scores[at] = static_cast<float>(bm_value64(b.c));
      a.parents[at] = static_cast<int32_t>(b.at / a.vocab);
      a.tokens[at] = static_cast<int32_t>(b.at % a.vocab);
    }
    if (of >= 0 && mine.at == b.at) {  // places are distinct
      ++taken[of];
      look();
    }
  }
}

static int beam_chunks(int vocab) { return (vocab + kBmChunk - 1) / kBmChunk; }

}  // namespace gaac

using namespace gaac;

extern "C" size_t gaac_beam_workspace(int batch, int beams, int vocab, int n_out) {
  if (batch < 1 || beams < 1 || beams > kBmMostBeams || vocab < 1 || vocab > kBmMostVocab || n_out < 1 || n_out > kBmMostOut) return 0;
  const size_t lists = static_cast<size_t>(batch) * beams * beam_chunks(vocab);
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
  const int chunks = beam_chunks(vocab);
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
