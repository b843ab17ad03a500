// Rotary positions.
//
// Channels (a, b) of pair j at position p turn by the angle p * w_j:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin).
// The GAAC page's Appendix C studies rotary keys; this is the operator itself, applied before an append.
//
// Angles: w_j comes as a fraction of a turn in 64-bit fixed point, F_j = w_j / (2 pi) * 2^64.  The product
// p * F_j modulo 2^64 is the exact fraction of the turn whatever the position (32-bit floats would be off by
// 0.06 rad at a million), and its top 32 bits, as a signed number, are the angle in [-pi, pi): one float
// conversion, then sincospi.  The angle is off by at most 2^-26 turns for the conversion, 2^-33 for the bits left
// out, and p times the table's own error: 2^-65 where F_j is the nearest, 2^-52 of w_j / (2 pi) where it comes from
// 64-bit floats (2^-34 turns at a million for the fastest pair).
//
// Memory bound: every byte of input is read once and written once.  A thread owns V pairs (16-byte vectors where
// alignment allows) of one row and walks over up to five heads with them, so V sines and cosines serve all of these;
// neighbouring threads take neighbouring vectors, then neighbouring heads.  The loads of two heads are under way
// before the sines are computed.  CTAs of 64 threads, 16 to an SM (64 registers), keep the loads of many rows in
// flight: 32,768 tokens x 40 heads x 128 in bf16 take 100.3 us, 6.69 TB/s (104.1 us with 128 threads and eight
// heads, 106.2 us with 256); 32 tokens 2.1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace gaac {

struct RopeTensor {
  const char* x;
  char* out;
  int64_t x_seq, x_tok, x_head, out_seq, out_tok, out_head;  // bytes
  int copy;                                                  // out is other memory: the rest of the head is copied
};

struct RopeArgs {
  RopeTensor t[2];
  int heads0, heads;  // heads of the first tensor; of both
  unsigned n_seq, n_tok;
  int rot, dim;
  const void* pos;
  int pos64;
  int64_t pos_seq, pos_tok;
  const uint64_t* turns;
  float mscale;
  int inverse;
  unsigned units, rot_units;          // of a head: all units, the copied rest included; the rotated ones
  int walkers;                        // threads that share the heads of a row
  unsigned row_walkers;               // rows * walkers
  unsigned unit_threads, per_block;   // threads for the units of a (row, walker); those of a block
};

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T v[V];
};

__device__ __forceinline__ float2 rope_pair(__nv_bfloat162 w) { return __bfloat1622float2(w); }
__device__ __forceinline__ float2 rope_pair(__half2 w) { return __half22float2(w); }
template <typename T>
struct RopePair;
template <>
struct RopePair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ type pack(float a, float b) { return __floats2bfloat162_rn(a, b); }
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct RopePair<__half> {
  using type = __half2;
  static __device__ __forceinline__ type pack(float a, float b) { return __floats2half2_rn(a, b); }
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

template <typename T, int V>
__device__ __forceinline__ void rope_unpack(const RopeVec<T, V>& x, float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = x.v[i];
  } else if constexpr (V == 1) {
    f[0] = RopePair<T>::get(x.v[0]);
  } else {
    const auto* w = reinterpret_cast<const typename RopePair<T>::type*>(x.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 p = rope_pair(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void rope_pack(RopeVec<T, V>& x, const float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = f[i];
  } else if constexpr (V == 1) {
    x.v[0] = RopePair<T>::put(f[0]);
  } else {
    auto* w = reinterpret_cast<typename RopePair<T>::type*>(x.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = RopePair<T>::pack(f[2 * i], f[2 * i + 1]);
  }
}

constexpr int kRopeThreads = 64;
constexpr int kRopeBatch = 2;  // heads whose loads a thread has in flight
constexpr int kRopeMost = 5;   // most heads of a thread

// Thread (row, walker, unit): heads walker, walker + walkers, ... of one row, V pairs of each.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 16) rope_kernel(const RopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using Vec = RopeVec<T, V>;
  const unsigned local = threadIdx.x / a.unit_threads;
  const unsigned rw = blockIdx.x * a.per_block + local;
  if (local >= a.per_block || rw >= a.row_walkers) return;
  const unsigned row = rw / a.walkers;
  const int walker = static_cast<int>(rw - row * a.walkers);
  unsigned seq = 0, tok = row;
  if (a.n_seq > 1) {
    seq = row / a.n_tok;
    tok = row - seq * a.n_tok;
  }
  const char* const xq = a.t[0].x + seq * a.t[0].x_seq + tok * a.t[0].x_tok;
  const char* const xk = a.t[1].x + seq * a.t[1].x_seq + tok * a.t[1].x_tok;
  char* const outq = a.t[0].out + seq * a.t[0].out_seq + tok * a.t[0].out_tok;
  char* const outk = a.t[1].out + seq * a.t[1].out_seq + tok * a.t[1].out_tok;
  for (unsigned u = threadIdx.x - local * a.unit_threads; u < a.units; u += a.unit_threads) {
    // a unit is two vectors: of the rotated part, or of the channels behind it (the last may be one)
    const bool turned = u < a.rot_units;
    const int e0 = turned ? (INTER ? 2 * u * V : u * V) : a.rot + 2 * (u - a.rot_units) * V;
    const int e1 = turned && !INTER ? e0 + a.rot / 2 : e0 + V;
    const bool two = e1 < a.dim;
    const int64_t o0 = e0 * static_cast<int64_t>(sizeof(T)), o1 = e1 * static_cast<int64_t>(sizeof(T));
    Vec v[kRopeBatch][2];
    char* out[kRopeBatch];
    auto load = [&](int h0) {
#pragma unroll
      for (int j = 0; j < kRopeBatch; ++j) {
        const int h = h0 + j * a.walkers;
        out[j] = nullptr;
        if (h < a.heads) {
          const bool second = h >= a.heads0;
          if (turned || (second ? a.t[1].copy : a.t[0].copy)) {
            const char* x = second ? xk + (h - a.heads0) * a.t[1].x_head : xq + h * a.t[0].x_head;
            out[j] = second ? outk + (h - a.heads0) * a.t[1].out_head : outq + h * a.t[0].out_head;
            v[j][0] = *reinterpret_cast<const Vec*>(x + o0);
            if (two) v[j][1] = *reinterpret_cast<const Vec*>(x + o1);
          }
        }
      }
    };
    load(walker);  // under way while the sines are computed
    float c[V], s[V];
    if (turned) {
      const int64_t pi = seq * a.pos_seq + tok * a.pos_tok;
      uint64_t p = a.pos64 ? static_cast<uint64_t>(static_cast<const int64_t*>(a.pos)[pi])
                           : static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t*>(a.pos)[pi]));
      if (a.inverse) p = 0 - p;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t turn = p * a.turns[u * V + i] + (1ull << 31);
        const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        // A 16-bit result is rounded at 2^-12 or coarser, so the hardware's sine and cosine (2^-21.2 off at most in
        // [-pi, pi]) serve it; they take a tenth of the instructions, which bound the kernel otherwise.
        if constexpr (sizeof(T) == 2)
          __sincosf(half_turns * 3.14159265358979f, &s[i], &c[i]);
        else
          sincospif(half_turns, &s[i], &c[i]);
        s[i] *= a.mscale;
        c[i] *= a.mscale;
      }
    }
    // the loads of kRopeBatch heads come before the first store
    for (int h0 = walker;;) {
#pragma unroll
      for (int j = 0; j < kRopeBatch; ++j) {
        if (out[j] != nullptr) {
          if (turned) {
            float e[2 * V];
            rope_unpack<T, V>(v[j][0], e);
            rope_unpack<T, V>(v[j][1], e + V);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : V + i;
              const float x0 = e[ia], x1 = e[ib];
              e[ia] = x0 * c[i] - x1 * s[i];
              e[ib] = x1 * c[i] + x0 * s[i];
            }
            rope_pack<T, V>(v[j][0], e);
            rope_pack<T, V>(v[j][1], e + V);
          }
          *reinterpret_cast<Vec*>(out[j] + o0) = v[j][0];
          if (two) *reinterpret_cast<Vec*>(out[j] + o1) = v[j][1];
        }
      }
      h0 += kRopeBatch * a.walkers;
      if (h0 >= a.heads) break;
      load(h0);
    }
  }
}

template <typename T, int V>
static int rope_launch(const RopeArgs& a, bool inter, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.row_walkers + a.per_block - 1) / a.per_block);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = inter ? cudaLaunchKernelEx(&cfg, rope_kernel<T, V, true>, a)
                              : cudaLaunchKernelEx(&cfg, rope_kernel<T, V, false>, a);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? GAAC_OK : GAAC_ECUDA;
}

template <typename T>
static int rope_vec(RopeArgs& a, int v, bool inter, cudaStream_t st) {
  switch (v) {
    case 8:
      if constexpr (sizeof(T) == 2) return rope_launch<T, 8>(a, inter, st);
      return GAAC_EINVAL;
    case 4: return rope_launch<T, 4>(a, inter, st);
    case 2: return rope_launch<T, 2>(a, inter, st);
    default: return rope_launch<T, 1>(a, inter, st);
  }
}

// Elements (seq, tok, head) of the output are distinct: taken from the smallest stride up, each dimension
// steps over everything below it.  Dimensions of size 1 do not count.
static bool distinct(int64_t dim, int64_t n[3], int64_t s[3]) {
  int64_t extent = dim;
  bool used[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) return true;
    if (s[at] < extent) return false;
    extent = s[at] * (n[at] - 1) + extent;
    used[at] = true;
  }
  return true;
}

}  // namespace gaac

using namespace gaac;

extern "C" int gaac_rope(const gaac_rope_tensor* tensors, int n_tensors, int dtype, int64_t n_seq, int64_t n_tok,
                         int head_dim, int rot_dim, const void* positions, int pos_bits, int64_t pos_seq_stride,
                         int64_t pos_tok_stride, const uint64_t* turns, float mscale, unsigned flags, void* stream) {
  if (tensors == nullptr || n_tensors < 1 || n_tensors > 2 || (dtype != GAAC_BF16 && dtype != GAAC_F16 && dtype != GAAC_F32) ||
      (pos_bits != 32 && pos_bits != 64) || (flags & ~static_cast<unsigned>(GAAC_ROPE_INTERLEAVED | GAAC_ROPE_INVERSE)) ||
      !std::isfinite(mscale))
    return GAAC_EINVAL;
  if (n_seq < 0 || n_tok < 0 || n_seq > 0x7FFFFFFF || n_tok > 0x7FFFFFFF || head_dim < 2 || head_dim > 4096 || rot_dim < 2 ||
      rot_dim > head_dim || (rot_dim & 1))
    return GAAC_EINVAL;
  const int64_t rows = n_seq * n_tok;
  if (rows > 0x7FFFFFFF) return GAAC_EINVAL;
  const int size = dtype == GAAC_F32 ? 4 : 2;
  int64_t heads = 0;
  for (int i = 0; i < n_tensors; ++i) {
    if (tensors[i].n_heads < 1 || tensors[i].n_heads > 65536) return GAAC_EINVAL;
    heads += tensors[i].n_heads;
  }
  if (rows == 0) return GAAC_OK;
  if (positions == nullptr || turns == nullptr || pos_seq_stride < 0 || pos_tok_stride < 0 ||
      (reinterpret_cast<uintptr_t>(positions) & (pos_bits / 8 - 1)) || (reinterpret_cast<uintptr_t>(turns) & 7u))
    return GAAC_EINVAL;
  // Vector width: as many elements as one 16-byte access holds, halved until both halves of the rotated part,
  // the rest of the head and every pointer and stride are multiples of it.
  int v = 16 / size;
  while (v > 1 && ((rot_dim / 2) % v || (head_dim - rot_dim) % v)) v /= 2;
  RopeArgs a = {};
  bool copies = false;
  for (int i = 0; i < n_tensors; ++i) {
    const gaac_rope_tensor& t = tensors[i];
    if (t.x == nullptr || t.out == nullptr || t.x_seq < 0 || t.x_tok < 0 || t.x_head < 0) return GAAC_EINVAL;
    const int64_t most = int64_t{1} << 56;
    if (t.x_seq > most / n_seq || t.x_tok > most / n_tok || t.x_head > most / t.n_heads || t.out_seq > most / n_seq ||
        t.out_tok > most / n_tok || t.out_head > most / t.n_heads)
      return GAAC_EINVAL;
    int64_t n[3] = {n_seq, n_tok, t.n_heads}, so[3] = {t.out_seq, t.out_tok, t.out_head};
    if (t.out_seq < 0 || t.out_tok < 0 || t.out_head < 0 || !distinct(head_dim, n, so)) return GAAC_EINVAL;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(t.x), o0 = reinterpret_cast<uintptr_t>(t.out);
    if ((x0 | o0) & (size - 1)) return GAAC_EINVAL;
    // In place means the same elements; any other overlap of input and output would read rotated values.
    const bool same = x0 == o0 && (n_seq == 1 || t.x_seq == t.out_seq) && (n_tok == 1 || t.x_tok == t.out_tok) &&
                      (t.n_heads == 1 || t.x_head == t.out_head);
    const uintptr_t xe = x0 + ((n_seq - 1) * t.x_seq + (n_tok - 1) * t.x_tok + (t.n_heads - 1) * t.x_head + head_dim) * size;
    const uintptr_t oe = o0 + ((n_seq - 1) * t.out_seq + (n_tok - 1) * t.out_tok + (t.n_heads - 1) * t.out_head + head_dim) * size;
    if (!same && x0 < oe && o0 < xe) return GAAC_EINVAL;
    const uintptr_t all = (n_seq > 1 ? (t.x_seq | t.out_seq) : 0) | (n_tok > 1 ? (t.x_tok | t.out_tok) : 0) |
                          (t.n_heads > 1 ? (t.x_head | t.out_head) : 0);
    while (v > 1 && ((all % v) || ((x0 | o0) & (static_cast<uintptr_t>(v) * size - 1)))) v /= 2;
    a.t[i] = RopeTensor{static_cast<const char*>(t.x), static_cast<char*>(t.out), t.x_seq * size, t.x_tok * size,
                        t.x_head * size, t.out_seq * size, t.out_tok * size, t.out_head * size, same ? 0 : 1};
    copies = copies || !same;
  }
  // Two tensors with a first element in common, one of them an output.  Tensors that share others (slices of one
  // projection's output overlap as ranges and share none) are the caller's to keep apart.
  if (n_tensors == 2 && (tensors[0].out == tensors[1].out || tensors[0].out == tensors[1].x || tensors[1].out == tensors[0].x))
    return GAAC_EINVAL;
  a.heads0 = tensors[0].n_heads;
  a.heads = static_cast<int>(heads);
  a.n_seq = static_cast<unsigned>(n_seq);
  a.n_tok = static_cast<unsigned>(n_tok);
  a.rot = rot_dim;
  a.dim = head_dim;
  a.pos = positions;
  a.pos64 = pos_bits == 64;
  a.pos_seq = pos_seq_stride;
  a.pos_tok = pos_tok_stride;
  a.turns = turns;
  a.mscale = mscale;
  a.inverse = (flags & GAAC_ROPE_INVERSE) != 0;
  a.rot_units = rot_dim / 2 / v;
  a.units = a.rot_units + (copies ? ((head_dim - rot_dim) / v + 1) / 2 : 0);
  // Heads per thread: as many as leave twice the threads that 152 SMs hold at a time (16 CTAs of 64 each), so that
  // sines are shared where there is work for all, and single heads where latency counts.
  const int64_t want = int64_t{152} * 2048, per_row = rows * a.units;
  const int64_t walkers = std::max<int64_t>((heads + kRopeMost - 1) / kRopeMost, (want + per_row - 1) / per_row);
  a.walkers = static_cast<int>(std::min<int64_t>(heads, walkers));
  if (rows * a.walkers > 0x7FFFFFFF) return GAAC_EINVAL;
  a.row_walkers = static_cast<unsigned>(rows * a.walkers);
  a.unit_threads = std::min<unsigned>(a.units, kRopeThreads);
  a.per_block = kRopeThreads / a.unit_threads;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = (flags & GAAC_ROPE_INTERLEAVED) != 0;
  if (dtype == GAAC_BF16) return rope_vec<__nv_bfloat16>(a, v, inter, st);
  if (dtype == GAAC_F16) return rope_vec<__half>(a, v, inter, st);
  return rope_vec<float>(a, v, inter, st);
}
