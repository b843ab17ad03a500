// Decode attention over the 8-bit paged cache.
//
//   s_t = scale * sK * (q . k8_t),   out = sum_t softmax(s)_t * sV * v8_t
// with sK, sV the scales of t's block (1 for the open block, which is in the model's type).
//
// First form: one CTA per (sequence, kv-head), a warp per token, everything in 32-bit floats.
#include "kv8.cuh"

namespace gaac {

struct Kv8AttnArgs {
  Kv8Dev c;
  const uint16_t* q;
  int64_t q_seq;
  void* out;
  int out_f32, r;
  float scale;
  int32_t* status;
};

constexpr int kKaWarps = 8;

template <bool HALF, int FMT>
__global__ void __launch_bounds__(32 * kKaWarps) kv8_attention_kernel(Kv8AttnArgs a) {
  __shared__ float sm[kKaWarps][8], sl[kKaWarps][8];
  __shared__ float so[kKaWarps][8][kD];
  dependent_wait();
  dependent_launch();
  const Kv8Dev& c = a.c;
  const int b = blockIdx.x / c.heads, h = blockIdx.x % c.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int len = c.lens[b];
  if (len < 0 || len > static_cast<int64_t>(c.max_blocks) * kBlock) {
    if (threadIdx.x == 0) report(a.status, GAAC_EINVAL);
    len = 0;
  }
  float q[8][4], o[8][4], m[8], l[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[r][i] = q[r][i] = 0.f;
    if (r < a.r) {
      const uint2 w = *reinterpret_cast<const uint2*>(a.q + b * a.q_seq + (h * a.r + r) * kD + 4 * lane);
      const float2 x = kv8_pair<HALF>(w.x), y = kv8_pair<HALF>(w.y);
      q[r][0] = x.x, q[r][1] = x.y, q[r][2] = y.x, q[r][3] = y.y;
    }
  }
  for (int t = warp; t < len; t += kKaWarps) {
    const int blk = t / kBlock, row = t % kBlock;
    float k[4], v[4], sk = 1.f, sv = 1.f;
    if ((blk + 1) * kBlock <= len) {
      const int64_t p = c.table[static_cast<int64_t>(b) * c.max_blocks + blk];
      if (p < 0 || p >= c.n_pages) {
        if (lane == 0) report(a.status, GAAC_EFORMAT);
        continue;
      }
      const uint8_t* base = c.pages + (p * c.heads + h) * kKv8Pair + row * kD + 4 * lane;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(base), vw = *reinterpret_cast<const uint32_t*>(base + kKv8Tile);
      const uint32_t w[4] = {fp8x2_to_f16x2<FMT>(kw & 0xFFFF), fp8x2_to_f16x2<FMT>(kw >> 16), fp8x2_to_f16x2<FMT>(vw & 0xFFFF),
                             fp8x2_to_f16x2<FMT>(vw >> 16)};
      const float2 x = kv8_pair<true>(w[0]), y = kv8_pair<true>(w[1]), z = kv8_pair<true>(w[2]), u = kv8_pair<true>(w[3]);
      k[0] = x.x, k[1] = x.y, k[2] = y.x, k[3] = y.y;
      v[0] = z.x, v[1] = z.y, v[2] = u.x, v[3] = u.y;
      sk = c.scales[(p * c.heads + h) * 2];
      sv = c.scales[(p * c.heads + h) * 2 + 1];
    } else {
      const uint16_t* base = c.tail + (static_cast<int64_t>(b) * c.heads + h) * 2 * kKv8Tile + row * kD + 4 * lane;
      const uint2 kw = *reinterpret_cast<const uint2*>(base), vw = *reinterpret_cast<const uint2*>(base + kKv8Tile);
      const float2 x = kv8_pair<HALF>(kw.x), y = kv8_pair<HALF>(kw.y), z = kv8_pair<HALF>(vw.x), u = kv8_pair<HALF>(vw.y);
      k[0] = x.x, k[1] = x.y, k[2] = y.x, k[3] = y.y;
      v[0] = z.x, v[1] = z.y, v[2] = u.x, v[3] = u.y;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float s = q[r][0] * k[0] + q[r][1] * k[1] + q[r][2] * k[2] + q[r][3] * k[3];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      s *= a.scale * sk;
      const float mn = fmaxf(m[r], s), shift = mn == -INFINITY ? 0.f : mn;
      const float f = __expf(m[r] - shift), p = __expf(s - shift);
      m[r] = mn;
      l[r] = l[r] * f + p;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[r][i] = o[r][i] * f + p * sv * v[i];
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (lane == 0) {
      sm[warp][r] = m[r];
      sl[warp][r] = l[r];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) so[warp][r][4 * lane + i] = o[r][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.r * kD; i += 32 * kKaWarps) {
    const int r = i / kD, ch = i % kD;
    float mx = -INFINITY;
    for (int w = 0; w < kKaWarps; ++w) mx = fmaxf(mx, sm[w][r]);
    float den = 0.f, num = 0.f;
    for (int w = 0; w < kKaWarps; ++w) {
      const float f = __expf(sm[w][r] - (mx == -INFINITY ? 0.f : mx));
      den += f * sl[w][r];
      num += f * so[w][r][ch];
    }
    const float y = den == 0.f ? 0.f : num / den;
    const int64_t at = (static_cast<int64_t>(b) * c.heads * a.r + h * a.r) * kD + i;
    if (a.out_f32)
      static_cast<float*>(a.out)[at] = y;
    else if (HALF)
      static_cast<__half*>(a.out)[at] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace gaac

using namespace gaac;

extern "C" size_t gaac_kv8_attention_workspace(void) { return 16; }

extern "C" int gaac_kv8_decode_attention(const gaac_kv8* cache, const void* q, int n_q_heads, int64_t q_seq_stride,
                                         float scale, void* out, int out_dtype, void* workspace,
                                         size_t workspace_bytes, int32_t* d_status, void* stream) {
  if (!kv8_ok(cache) || q == nullptr || out == nullptr || workspace == nullptr || !std::isfinite(scale) ||
      (out_dtype != cache->dtype && out_dtype != GAAC_F32))
    return GAAC_EINVAL;
  if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads != 0 || n_q_heads / cache->n_kv_heads > GAAC_MAX_GQA ||
      q_seq_stride < static_cast<int64_t>(n_q_heads) * kD || (q_seq_stride & 7) || q_seq_stride > (int64_t{1} << 40) ||
      (reinterpret_cast<uintptr_t>(q) & 15u) || (reinterpret_cast<uintptr_t>(out) & 15u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < gaac_kv8_attention_workspace())
    return GAAC_EINVAL;
  const Kv8AttnArgs a{kv8_dev(cache), static_cast<const uint16_t*>(q), q_seq_stride, out, out_dtype == GAAC_F32,
                      n_q_heads / cache->n_kv_heads, scale, d_status};
  const dim3 grid(static_cast<unsigned>(cache->batch) * cache->n_kv_heads);
  if (cache->dtype == GAAC_BF16)
    return cache->fmt == GAAC_FP8_E4M3
               ? kv8_launch(kv8_attention_kernel<false, GAAC_FP8_E4M3>, grid, 32 * kKaWarps, 0, stream, a)
               : kv8_launch(kv8_attention_kernel<false, GAAC_FP8_E5M2>, grid, 32 * kKaWarps, 0, stream, a);
  return cache->fmt == GAAC_FP8_E4M3
             ? kv8_launch(kv8_attention_kernel<true, GAAC_FP8_E4M3>, grid, 32 * kKaWarps, 0, stream, a)
             : kv8_launch(kv8_attention_kernel<true, GAAC_FP8_E5M2>, grid, 32 * kKaWarps, 0, stream, a);
}
