// Append to the 8-bit paged cache: new tokens join each sequence's open block; blocks that fill are quantised
// into their pages, the rest stays in the tail in the model's type.
//
// Scale of a block (one for its K and one for its V of every kv-head): with A the largest finite magnitude of
// its 64 x 128 numbers and 1.75 * 2^t the format's largest value (t = 8 for E4M3, 15 for E5M2),
//   scale = the smallest 2^e with A <= 1.75 * 2^(t + e), e >= -126;  1 for a block without finite nonzero numbers.
// A power of two makes x / scale exact, so the only rounding is the one to FP8 (nearest, ties to even), and a
// floating format gains nothing from a finer scale but at its subnormal end.  A block is quantised once, from
// the numbers themselves, however its tokens arrive.  NaN stays NaN; an infinity stays one in E5M2 and becomes
// NaN in E4M3, which has none.
//
// One CTA for each (block touched, kv-head), K and V together: 256 threads hold the block's 32 KB in registers
// (eight 16-byte loads in flight each), so every number is read once and written once.  The first block's CTA
// also writes the new open block's rows, after it has read the old ones from the same tail.
#include "kv8.cuh"

namespace gaac {

struct Kv8AppendArgs {
  Kv8Dev c;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_tok, v_tok;  // elements between tokens
  const int32_t* cu;     // first token of each sequence, batch + 1; nullptr: one token each
  int64_t total;
  int32_t* status;
};

constexpr int kApThreads = 256;

template <int FMT>
__device__ __forceinline__ uint32_t to_fp8x2(float lo, float hi) {
  uint16_t r;
  if (FMT == GAAC_FP8_E4M3)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Infinities: NaN in E4M3, infinity in E5M2 (the conversion above would clamp them).
template <int FMT>
__device__ __forceinline__ uint32_t to_fp8_any(float x) {
  if (isinf(x)) return FMT == GAAC_FP8_E4M3 ? 0x7Fu : (x < 0.f ? 0xFCu : 0x7Cu);
  if (isnan(x)) return 0x7Fu;
  return to_fp8x2<FMT>(x, 0.f) & 0xFFu;
}

// The scale's exponent for the largest magnitude `bits` (a 16-bit number of the model's type).
template <bool HALF, int FMT>
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const float a = kv8_pair<HALF>(bits).x;
  if (a == 0.f) return 0;
  // a * 2^64 is a normal number whatever a is (the smallest bf16 is 2^-133); exact, and below 2^128 for a < 2^64
  const bool small = a < 0x1p-100f;
  const uint32_t f = __float_as_uint(small ? a * 0x1p64f : a);
  const int e = static_cast<int>(f >> 23) - 127 - (small ? 64 : 0);
  const int top = FMT == GAAC_FP8_E4M3 ? 8 : 15;
  return max(e - top + ((f & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
}

template <bool HALF, int FMT>
__global__ void __launch_bounds__(kApThreads) kv8_append_kernel(Kv8AppendArgs a) {
  __shared__ uint32_t sh_max[kApThreads / 32];
  dependent_wait();
  dependent_launch();
  const Kv8Dev& c = a.c;
  const int tid = threadIdx.x;
  const int h = static_cast<int>(blockIdx.x % c.heads);
  const int64_t tile = blockIdx.x / c.heads;
  // ---- the sequence and the block of this CTA
  // Sequence b owns tiles [cu[b]/64 + 2b, cu[b+1]/64 + 2b + 2): at least as many as its tokens can touch, wherever
  // its open block ends.
  int b, j, n, span;
  int64_t first;
  if (a.cu == nullptr) {
    b = static_cast<int>(tile);
    j = 0;
    n = 1;
    span = 1;
    first = b;
  } else {
    int count = 0, bad = 0;
    for (int i0 = 0; i0 < c.batch; i0 += kApThreads) {
      const int i = i0 + tid;
      int below = 0;
      if (i < c.batch) {
        const int64_t lo = a.cu[i], hi = a.cu[i + 1];
        if (lo < 0 || hi < lo || hi > a.total) bad = 1;
        below = hi / kBlock + 2 * (static_cast<int64_t>(i) + 1) <= tile;
      }
      count += __syncthreads_count(below);
    }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && tid == 0) report(a.status, GAAC_EINVAL);
      return;
    }
    b = count;
    if (b >= c.batch) return;
    first = a.cu[b];
    const int64_t t0 = first / kBlock + 2 * static_cast<int64_t>(b), t1 = a.cu[b + 1] / kBlock + 2 * (static_cast<int64_t>(b) + 1);
    if (tile < t0) return;
    j = static_cast<int>(tile - t0);
    span = static_cast<int>(t1 - t0);
    n = static_cast<int>(a.cu[b + 1] - first);
  }
  const int len = c.lens[b];
  const int64_t now = static_cast<int64_t>(len) + n;
  const int blk0 = len / kBlock, blk1 = static_cast<int>(now / kBlock);
  const int32_t* row = c.table + static_cast<int64_t>(b) * c.max_blocks;
  int fault = 0;
  if (len < 0 || now > static_cast<int64_t>(c.max_blocks) * kBlock) {
    fault = GAAC_EINVAL;
  } else {
    int missing = 0;
    for (int i = blk0 + tid; i < blk1; i += kApThreads) {
      const int32_t p = row[i];
      if (p < 0 || p >= c.n_pages) missing = 1;
    }
    if (__syncthreads_or(missing)) fault = GAAC_EPOOL;
  }
  if (fault && tid == 0) report(a.status, fault);
  const int touched = n == 0 || fault ? 0 : static_cast<int>((now + kBlock - 1) / kBlock) - blk0;
  if (j < touched) {
    const int blk = blk0 + j;
    const bool seal = blk < blk1;
    uint16_t* tail = c.tail + (static_cast<int64_t>(b) * c.heads + h) * 2 * kKv8Tile;
    const int t0 = tid >> 4, c8 = 8 * (tid & 15);
    const uint16_t* src[2] = {a.k + h * kD + c8, a.v + h * kD + c8};
    const int64_t step[2] = {a.k_tok, a.v_tok};
    if (seal) {
      uint4 w[2][4];
#pragma unroll
      for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 16 * i;
          const int64_t at = static_cast<int64_t>(blk) * kBlock + t - len;  // among the new tokens
          w[kind][i] = *reinterpret_cast<const uint4*>(at < 0 ? tail + kind * kKv8Tile + t * kD + c8
                                                              : src[kind] + (first + at) * step[kind]);
        }
      // largest finite magnitudes as 16-bit patterns (their order is the numbers'): K in the low half, V in the high
      uint32_t mx = 0, odd = 0;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t* x = reinterpret_cast<const uint32_t*>(&w[kind][i]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t mag = x[q] & 0x7FFF7FFFu;
            const uint32_t inf = __vcmpgeu2(mag, HALF ? 0x7C007C00u : 0x7F807F80u);
            odd |= inf;
            m = __vmaxu2(m, mag & ~inf);
          }
        }
        m = max(m & 0xFFFFu, m >> 16);
        mx |= m << (16 * kind);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
      if ((tid & 31) == 0) sh_max[tid >> 5] = mx;
      const bool any_odd = __syncthreads_or(odd != 0u);  // also: the old rows of the tail have been read
#pragma unroll
      for (int i = 0; i < kApThreads / 32; ++i) mx = __vmaxu2(mx, sh_max[i]);
      const int64_t page = row[blk];
      uint8_t* dst = c.pages + (page * c.heads + h) * kKv8Pair + t0 * kD + c8;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        const int e = scale_exponent<HALF, FMT>((mx >> (16 * kind)) & 0xFFFFu);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t* x = reinterpret_cast<const uint32_t*>(&w[kind][i]);
          uint32_t o[2] = {0u, 0u};
          if (!any_odd) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 f = kv8_pair<HALF>(x[q]);
              o[q >> 1] |= to_fp8x2<FMT>(f.x * inv, f.y * inv) << (16 * (q & 1));
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 f = kv8_pair<HALF>(x[q]);
              o[q >> 1] |= (to_fp8_any<FMT>(f.x * inv) | to_fp8_any<FMT>(f.y * inv) << 8) << (16 * (q & 1));
            }
          }
          *reinterpret_cast<uint2*>(dst + kind * kKv8Tile + 16 * i * kD) = make_uint2(o[0], o[1]);
        }
        if (tid == 0) c.scales[(page * c.heads + h) * 2 + kind] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
    }
    // the rows of the new open block
    if (j == 0 && blk1 < blk0 + touched) {
      const int64_t open = static_cast<int64_t>(blk1) * kBlock;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind)
        for (int t = t0; t < now - open; t += 16) {
          const int64_t at = open + t - len;
          if (at >= 0)
            *reinterpret_cast<uint4*>(tail + kind * kKv8Tile + t * kD + c8) =
                *reinterpret_cast<const uint4*>(src[kind] + (first + at) * step[kind]);
        }
    }
  }
  // ---- the length advances once every CTA of the sequence has read it
  if (tid == 0) {
    const unsigned int all = static_cast<unsigned int>(span) * c.heads;
    if (kv8_atomic_add_acq_rel(c.work + b, 1u) == all - 1) {
      c.work[b] = 0;
      if (!fault) c.lens[b] = static_cast<int32_t>(now);
    }
  }
}

}  // namespace gaac

using namespace gaac;

extern "C" size_t gaac_kv8_workspace(int batch, int64_t n_pages) {
  if (batch < 1 || n_pages < 1) return 0;
  return static_cast<size_t>(kv8_work(batch, n_pages).words) * sizeof(int32_t);
}

extern "C" int gaac_kv8_append(const gaac_kv8* cache, const void* k, const void* v, int64_t n_tokens,
                               int64_t k_tok_stride, int64_t v_tok_stride, const int32_t* cu_tokens, int32_t* d_status,
                               void* stream) {
  if (!kv8_ok(cache) || n_tokens < 0 || n_tokens > 0x7FFFFFFF || (cu_tokens == nullptr && n_tokens != cache->batch))
    return GAAC_EINVAL;
  if (n_tokens == 0) return GAAC_OK;
  const int64_t width = static_cast<int64_t>(cache->n_kv_heads) * kD;
  if (k == nullptr || v == nullptr || (reinterpret_cast<uintptr_t>(k) & 15u) || (reinterpret_cast<uintptr_t>(v) & 15u) ||
      (reinterpret_cast<uintptr_t>(cu_tokens) & 3u) || k_tok_stride < width || v_tok_stride < width ||
      (k_tok_stride & 7) || (v_tok_stride & 7) || k_tok_stride > (int64_t{1} << 40) || v_tok_stride > (int64_t{1} << 40))
    return GAAC_EINVAL;
  const int64_t tiles = cu_tokens == nullptr ? cache->batch : n_tokens / kBlock + 2 * static_cast<int64_t>(cache->batch);
  if (tiles * cache->n_kv_heads > 0x7FFFFFFF) return GAAC_EINVAL;
  const Kv8AppendArgs a{kv8_dev(cache), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_tok_stride,
                        v_tok_stride, cu_tokens, n_tokens, d_status};
  const dim3 grid(static_cast<unsigned>(tiles * cache->n_kv_heads));
  if (cache->dtype == GAAC_BF16)
    return cache->fmt == GAAC_FP8_E4M3 ? kv8_launch(kv8_append_kernel<false, GAAC_FP8_E4M3>, grid, kApThreads, 0, stream, a)
                                       : kv8_launch(kv8_append_kernel<false, GAAC_FP8_E5M2>, grid, kApThreads, 0, stream, a);
  return cache->fmt == GAAC_FP8_E4M3 ? kv8_launch(kv8_append_kernel<true, GAAC_FP8_E4M3>, grid, kApThreads, 0, stream, a)
                                     : kv8_launch(kv8_append_kernel<true, GAAC_FP8_E5M2>, grid, kApThreads, 0, stream, a);
}
