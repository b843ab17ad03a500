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
// Memory bound: 2 bytes read and 1 written per number.  A CTA takes a run of consecutive blocks of K or of V of one
// kv-head: 128 threads hold a block's 16 KB in registers and have the next block's loads in flight while they
// quantise it, so the reads never pause, few warps wait at a block's one barrier, and what the run's sequence and pages
// are is looked up once.  Runs are one block long where there are few (latency), longer where every SM has several.
// 113,000 tokens of 8 heads in chunks of up to 24,000: 105 us, 6.6 TB/s (a block's K and V in CTAs of 512 threads:
// 120 us; with lane-by-lane conversions and address arithmetic: 150 us).  One token for each of 32 sequences: 2.3 us.
// The first block's CTA also writes the new open block's rows, after it has read the old ones from the same tail.
#include <algorithm>

#include "kv8.cuh"

namespace gaac {

struct Kv8AppendArgs {
  Kv8Dev c;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_tok, v_tok;  // elements between tokens
  const int32_t* cu;     // first token of each sequence, batch + 1; nullptr: one token each
  int64_t total;
  int run;               // blocks of a CTA
  int32_t* status;
};

constexpr int kApThreads = 128;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApStep = kApThreads / 16;           // rows that the CTA covers with one 16-byte vector a thread
constexpr int kApRows = kBlock / kApStep;          // vectors of a thread in a block
constexpr int kApCtasPerSm = 5;

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

// The scale's exponent for the largest magnitude `bits` (a 16-bit number of the model's type).  A bf16 subnormal's
// exponent comes out too large by its leading zeros, but any such block takes the smallest scale.
template <bool HALF, int FMT>
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  constexpr int kTop = FMT == GAAC_FP8_E4M3 ? 8 : 15;
  const uint32_t f = __float_as_uint(kv8_pair<HALF>(bits).x);
  const int e = max(static_cast<int>(f >> 23) - 127 - kTop + ((f & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
  return bits == 0u ? 0 : e;
}

// A thread's part of a block that fills: channels c8 .. c8 + 7 of kApRows rows, and the block's page.
struct ApBlock {
  uint4 w[kApRows];
  int32_t page;
};

// The block's largest magnitude as a 16-bit pattern, whose order is the numbers'.  FINITE leaves out infinities and
// NaN, which are otherwise the largest.  One barrier.
template <bool HALF, bool FINITE>
__device__ __forceinline__ uint32_t ap_largest(const ApBlock& x, uint32_t* sh) {
  const int tid = threadIdx.x;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kApRows; ++i) {
    const uint32_t w[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t mag = w[q] & 0x7FFF7FFFu;
      m = __vmaxu2(m, FINITE ? mag & ~__vcmpgeu2(mag, HALF ? 0x7C007C00u : 0x7F807F80u) : mag);
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
  if ((tid & 31) == 0) sh[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kApWarps; ++i) m = max(m, sh[i]);
  return m;
}

// Four numbers of the model's type times `inv`, as FP8.
template <bool HALF, int FMT>
__device__ __forceinline__ uint32_t ap_four(uint32_t w0, uint32_t w1, float inv) {
  const float2 a = kv8_pair<HALF>(w0), b = kv8_pair<HALF>(w1);
  uint32_t r;
#define GAAC_AP_FOUR(FP8X2)                                                                                       \
  asm("{\n .reg .b64 x, y, f;\n .reg .f32 x0, x1, y0, y1;\n .reg .b16 lo, hi;\n mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n" \
      " mov.b64 f, {%5, %5};\n mul.rn.f32x2 x, x, f;\n mul.rn.f32x2 y, y, f;\n mov.b64 {x0, x1}, x;\n mov.b64 {y0, y1}, y;\n" \
      " cvt.rn.satfinite." FP8X2 ".f32 lo, x1, x0;\n cvt.rn.satfinite." FP8X2 ".f32 hi, y1, y0;\n mov.b32 %0, {lo, hi};\n}"     \
      : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(inv))
  if (FMT == GAAC_FP8_E4M3)
    GAAC_AP_FOUR("e4m3x2");
  else
    GAAC_AP_FOUR("e5m2x2");
#undef GAAC_AP_FOUR
  return r;
}

// Quantises the block into its page: tile = 2 (page, kv-head) + (K|V), dst = this thread's first number of it.  sh: two
// sets of the warps' maxima; a barrier at least, behind which the old rows of the tail have been read.
template <bool HALF, int FMT>
__device__ __forceinline__ void ap_seal(const ApBlock& x, uint8_t* dst, float* scale, uint32_t (*sh)[kApWarps]) {
  constexpr uint32_t kInf = HALF ? 0x7C00u : 0x7F80u;
  uint32_t mx = ap_largest<HALF, false>(x, sh[0]);
  const bool odd = mx >= kInf;  // the same for the whole CTA
  if (odd) mx = ap_largest<HALF, true>(x, sh[1]);
  const int e = scale_exponent<HALF, FMT>(mx);
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  if (!odd) {
#pragma unroll
    for (int i = 0; i < kApRows; ++i)
      *reinterpret_cast<uint2*>(dst + i * kApStep * kD) =
          make_uint2(ap_four<HALF, FMT>(x.w[i].x, x.w[i].y, inv), ap_four<HALF, FMT>(x.w[i].z, x.w[i].w, inv));
  } else {
#pragma unroll
    for (int i = 0; i < kApRows; ++i) {
      const uint4 w = x.w[i];
      uint2 o = make_uint2(0u, 0u);
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        const float2 f = kv8_pair<HALF>(q < 2 ? w.x : q < 4 ? w.y : q < 6 ? w.z : w.w);
        const uint32_t y = to_fp8_any<FMT>((q & 1 ? f.y : f.x) * inv) << (8 * (q & 3));
        if (q < 4) o.x |= y; else o.y |= y;
      }
      *reinterpret_cast<uint2*>(dst + i * kApStep * kD) = o;
    }
  }
  if (threadIdx.x == 0) *scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

template <bool HALF, int FMT>
__global__ void __launch_bounds__(kApThreads, kApCtasPerSm) kv8_append_kernel(const Kv8AppendArgs a) {
  __shared__ uint32_t sh_max[2][2][kApWarps];  // of a block and the next
  dependent_wait();
  dependent_launch();
  const Kv8Dev& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31;
  const int hk = static_cast<int>(blockIdx.x % (2 * c.heads)), h = hk >> 1, kind = hk & 1;
  const int64_t place = blockIdx.x / (2 * c.heads);
  // ---- the sequence and the run of this CTA
  // With R blocks in a run, sequence b owns places [cu[b]/64R + 2b, cu[b+1]/64R + 2b + 2): at least as many as its
  // tokens can touch, wherever its open block ends.  Every warp looks it up for itself.
  int b, j, span;
  int64_t n, first;  // new tokens, and the row of the first
  if (a.cu == nullptr) {
    b = static_cast<int>(place);
    j = 0;
    n = 1;
    span = 1;
    first = b;
  } else {
    const int64_t per = static_cast<int64_t>(kBlock) * a.run;
    int count = 0, bad = 0;
#pragma unroll 4
    for (int i0 = 0; i0 < c.batch; i0 += 32) {
      const int i = i0 + lane;
      bool below = false;
      if (i < c.batch) {
        const int64_t lo = a.cu[i], hi = a.cu[i + 1];
        if (lo < 0 || hi < lo || hi > a.total) bad = 1;
        below = hi / per + 2 * (static_cast<int64_t>(i) + 1) <= place;
      }
      count += __popc(__ballot_sync(0xFFFFFFFFu, below));
    }
    if (__any_sync(0xFFFFFFFFu, bad)) {
      if (blockIdx.x == 0 && tid == 0) report(a.status, GAAC_EINVAL);
      return;
    }
    b = count;
    if (b >= c.batch) return;
    first = a.cu[b];
    const int64_t end = a.cu[b + 1];
    const int64_t p0 = first / per + 2 * static_cast<int64_t>(b), p1 = end / per + 2 * (static_cast<int64_t>(b) + 1);
    if (place < p0) return;
    j = static_cast<int>(place - p0) * a.run;
    span = static_cast<int>(p1 - p0);
    n = end - first;
  }
  const int len = c.lens[b];
  const int64_t now = len + n;
  const bool fits = len >= 0 && now <= static_cast<int64_t>(c.max_blocks) * kBlock;
  const int blk0 = fits ? len / kBlock : 0, blk1 = fits ? static_cast<int>(now / kBlock) : 0;  // blocks [blk0, blk1) fill
  const int32_t* row = c.table + static_cast<int64_t>(b) * c.max_blocks;
  const int t0 = tid >> 4, c8 = 8 * (tid & 15);
  uint16_t* tail = c.tail + (static_cast<int64_t>(b) * 2 * c.heads + hk) * kKv8Tile + c8;
  const uint16_t* src = (kind == 0 ? a.k : a.v) + h * kD + c8;
  const int64_t step = kind == 0 ? a.k_tok : a.v_tok;
  const int blk_begin = blk0 + j, blk_end = min(blk_begin + a.run, blk1);
  // this thread's first row of the run's next block that is loaded
  const uint16_t* at = src + (first + static_cast<int64_t>(blk_begin) * kBlock + t0 - len) * step;
  auto load = [&](ApBlock& x, int blk) {
    const int old = len - blk * kBlock;  // a block that opened before this call: its first tokens are in the tail
    if (old > 0) {
#pragma unroll
      for (int i = 0; i < kApRows; ++i)
        x.w[i] = *reinterpret_cast<const uint4*>(t0 + kApStep * i < old ? tail + (t0 + kApStep * i) * kD : at + kApStep * i * step);
    } else {
#pragma unroll
      for (int i = 0; i < kApRows; ++i) x.w[i] = *reinterpret_cast<const uint4*>(at + kApStep * i * step);
    }
    x.page = row[blk];
    at += kBlock * step;
  };
  auto seal = [&](const ApBlock& x, uint32_t (*sh)[kApWarps]) {
    const int64_t tile = static_cast<int64_t>(x.page) * 2 * c.heads + hk;
    ap_seal<HALF, FMT>(x, c.pages + tile * kKv8Tile + t0 * kD + c8, c.scales + tile, sh);
  };
  ApBlock x, y;
  if (blk_begin < blk_end) load(x, blk_begin);  // under way while the pages are checked
  int missing = 0;
  for (int i = blk0 + tid; i < blk1; i += kApThreads) {
    const int32_t p = row[i];
    if (p < 0 || p >= c.n_pages) missing = 1;
  }
  const int fault = !fits ? GAAC_EINVAL : __syncthreads_or(missing) ? GAAC_EPOOL : 0;
  if (fault) {
    if (tid == 0) report(a.status, fault);
  } else if (n > 0) {
    for (int blk = blk_begin; blk < blk_end; blk += 2) {
      if (blk + 1 < blk_end) load(y, blk + 1);
      seal(x, sh_max[0]);
      if (blk + 1 < blk_end) {
        if (blk + 2 < blk_end) load(x, blk + 2);
        seal(y, sh_max[1]);
      }
    }
    // the rows of the new open block
    if (j == 0) {
      const int64_t open = static_cast<int64_t>(blk1) * kBlock;
      for (int t = t0; t < now - open; t += kApStep) {
        const int64_t i = open + t - len;  // among the new tokens
        if (i >= 0) *reinterpret_cast<uint4*>(tail + t * kD) = *reinterpret_cast<const uint4*>(src + (first + i) * step);
      }
    }
  }
  // ---- the length advances once every CTA of the sequence has read it
  if (tid == 0) {
    const unsigned int all = static_cast<unsigned int>(span) * 2 * c.heads;
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

static int kv8_append(const gaac_kv8* cache, const void* k, const void* v, int64_t n_tokens, int64_t k_tok_stride,
                      int64_t v_tok_stride, const int32_t* cu_tokens, bool reserve, int32_t* d_status, void* stream) {
  if (!kv8_ok(cache) || n_tokens < 0 || n_tokens > 0x7FFFFFFF || (cu_tokens == nullptr && n_tokens != cache->batch))
    return GAAC_EINVAL;
  if (n_tokens == 0) return GAAC_OK;
  const int64_t width = static_cast<int64_t>(cache->n_kv_heads) * kD;
  if (k == nullptr || v == nullptr || (reinterpret_cast<uintptr_t>(k) & 15u) || (reinterpret_cast<uintptr_t>(v) & 15u) ||
      (reinterpret_cast<uintptr_t>(cu_tokens) & 3u) || k_tok_stride < width || v_tok_stride < width ||
      (k_tok_stride & 7) || (v_tok_stride & 7) || k_tok_stride > (int64_t{1} << 40) || v_tok_stride > (int64_t{1} << 40))
    return GAAC_EINVAL;
  // Blocks of a run: one while the blocks leave an SM with fewer than sixteen, at most sixteen.
  const int64_t blocks = n_tokens / kBlock * cache->n_kv_heads * 2;
  const int run = cu_tokens == nullptr ? 1 : static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, blocks / (152 * 16))));
  const int64_t places = cu_tokens == nullptr ? cache->batch : n_tokens / (kBlock * run) + 2 * static_cast<int64_t>(cache->batch);
  if (places * cache->n_kv_heads > 0x3FFFFFFF) return GAAC_EINVAL;
  // every refusal by the arguments comes before the reserve changes anything
  if (reserve) {
    const int e = kv8_reserve_rows(cache, cu_tokens, n_tokens, d_status, stream);
    if (e != GAAC_OK) return e;
  }
  const Kv8AppendArgs a{kv8_dev(cache), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_tok_stride,
                        v_tok_stride, cu_tokens, n_tokens, run, d_status};
  const dim3 grid(static_cast<unsigned>(places * 2 * cache->n_kv_heads));
  if (cache->dtype == GAAC_BF16)
    return cache->fmt == GAAC_FP8_E4M3 ? kv8_launch(kv8_append_kernel<false, GAAC_FP8_E4M3>, grid, kApThreads, 0, stream, a)
                                       : kv8_launch(kv8_append_kernel<false, GAAC_FP8_E5M2>, grid, kApThreads, 0, stream, a);
  return cache->fmt == GAAC_FP8_E4M3 ? kv8_launch(kv8_append_kernel<true, GAAC_FP8_E4M3>, grid, kApThreads, 0, stream, a)
                                     : kv8_launch(kv8_append_kernel<true, GAAC_FP8_E5M2>, grid, kApThreads, 0, stream, a);
}

extern "C" int gaac_kv8_append(const gaac_kv8* cache, const void* k, const void* v, int64_t n_tokens,
                               int64_t k_tok_stride, int64_t v_tok_stride, const int32_t* cu_tokens, int32_t* d_status,
                               void* stream) {
  return kv8_append(cache, k, v, n_tokens, k_tok_stride, v_tok_stride, cu_tokens, false, d_status, stream);
}

extern "C" int gaac_kv8_reserve_append(const gaac_kv8* cache, const void* k, const void* v, int64_t n_tokens,
                                       int64_t k_tok_stride, int64_t v_tok_stride, const int32_t* cu_tokens,
                                       int32_t* d_status, void* stream) {
  return kv8_append(cache, k, v, n_tokens, k_tok_stride, v_tok_stride, cu_tokens, true, d_status, stream);
}
