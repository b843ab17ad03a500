// Norms of queries and keys for each head with the rotation by their positions in the same pass, and the gradient.
//
// A head x of n channels, weights w:
//   r = 1 / sqrt(mean x^2 + eps),  y = x r w,  the first rot_dim channels of y turned as in rope.cu.
// Backward, with dz the gradient of the result:
//   g = dz turned back,  h = g w,  dx = r (h - x r mean(h x r)),  dw = sum over tokens and heads of g x r.
//
// Memory bound: the forward pass reads and writes every element once, the backward pass reads x and dz and writes dx;
// r is computed again rather than kept, since x has to be read for dx anyway.  A group of 2 to 32 lanes owns the heads of
// a row that it walks over; a lane has two vectors of V elements of each (a unit: V pairs of the rotated part, or of the
// channels behind it), so that the mean takes a few shuffles and V sines serve all heads of the walk.  Vectors of
// neighbouring lanes are neighbours, so that an instruction takes whole sectors (with a lane's two side by side, the
// gradient of interleaved pairs took 34.1 us for 27.4).  V is 16 bytes where widths and alignment allow, else one element with four
// units a lane.
// Arithmetic is packed, two numbers an instruction; the forward pass multiplies the weights into the sines once for a row and
// tensor.  Each head's registers are loaded again, with the head four further on, as soon as they are unpacked.
// Forward, 32,768 tokens x 40 heads x 128, bf16: 119 us, 5.6 TB/s (83% of a copy).  One head at a time without packing: 148 us;
// walks of five heads 154-179 us by CTAs an SM, of ten 129-157, of twenty 120 (8 CTAs, four heads in flight) to 163 (spills).  32
// tokens: 3.0 us.
// The backward pass has no registers for loads in flight (two heads' in them leave three CTAs to an SM and take 116 us), so
// its next three heads, across walks, come by asynchronous copies into shared memory, and 128 registers leave four CTAs.
// 16,384 tokens x 40 heads x 128, bf16: 88 us, 5.7 TB/s (84% of a copy), of which 3 us are sines as fine as an fp32 dw wants them;
// walks of 16 heads 89, of 32 93.  With coarser sines, 85 us: shuffles of the two means one after the other 94, and of that form
// two heads ahead the same, walks of 4 heads 99, a row's heads in one walk that begins with empty hands 97.  4,999 tokens x 24
// heads, fp16, half turned, interleaved: 27 us; 512 tokens x 24: 9.6 us.
// Sums are fp32.  dw: every lane adds up its channels over its rows, a CTA its lanes in order, a second launch the
// CTAs in order, so the result is the same each time.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "f32x2.cuh"
#include "kv8.cuh"
#include "rope.cuh"

namespace gaac {

constexpr int kNrThreads = 64;
constexpr int kNrBatch = 4;        // heads whose loads a lane has in flight
constexpr int kNrMost = 20;         // most heads of a walk
constexpr int kNrCtasPerSm = 8;
constexpr int kNrMaxDim = 256;
constexpr int kNgThreads = 128;    // gradient
constexpr int kNgMost = 8;         // most heads of a walk
constexpr int kNgAhead = 3;        // heads whose copies a lane has under way, where they are vectors
constexpr int kNgCtasPerSm = 4;
constexpr int kNgMostCtas = 152 * kNgCtasPerSm;

struct NormTensor {
  const char* x;
  const char* dz;  // gradient only
  char* out;
  const void* w;   // nullptr: ones
  float* dw;       // gradient only; may be nullptr
  int64_t x_seq, x_tok, x_head, dz_seq, dz_tok, dz_head, out_seq, out_tok, out_head;  // bytes
};

struct NormArgs {
  NormTensor t[2];
  int heads0, heads;  // heads of the first tensor; of both
  unsigned n_seq, n_tok;
  int rot, dim, w_f32;
  const void* pos;
  int pos64;
  int64_t pos_seq, pos_tok;
  const uint64_t* turns;
  float mscale, eps;
  int rot_units, units, lanes;  // of a head; lanes of a group
  int walk, walkers;            // heads of a walk; groups that share the heads of a row (gradient: of the first tensor)
  int walk1, walkers1;          // gradient: of the second
  unsigned row_walkers;         // rows * walkers
  unsigned ctas0;               // gradient: CTAs of the first tensor
  float* part;                  // gradient: [CTA][dim]
};

// A lane's units of a head: element offsets of the two vectors of unit k, and whether they exist.
template <int V, int UPL, bool INTER>
struct NormUnits {
  int e0[UPL], e1[UPL];
  bool turned[UPL], one[UPL], two[UPL];
  __device__ __forceinline__ NormUnits(const NormArgs& a, int lane) {
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      const int u = lane + k * a.lanes;
      turned[k] = u < a.rot_units;
      if (V > 1 || !INTER) {  // neighbouring lanes have neighbouring vectors
        e0[k] = turned[k] ? u * V : a.rot + (u - a.rot_units) * V;
        e1[k] = e0[k] + (turned[k] ? a.rot_units : a.units - a.rot_units) * V;
      } else {
        e0[k] = turned[k] ? 2 * u : a.rot + 2 * (u - a.rot_units);
        e1[k] = e0[k] + 1;
      }
      one[k] = u < a.units;
      two[k] = one[k] && e1[k] < a.dim;
    }
  }
};

// A lane's channels of a head as UPL * V pairs (a, b), two of them to a packed number.  Pairs that are not turned have
// sine 0 and cosine 1, and take nothing of each other (of_partner).  PART: there are such pairs; where the whole head is
// turned the selects for that would take 2% (121.4 us for 119.1, gradient 86.9 for 85.2).
template <typename T, int V, int UPL, bool INTER, bool PART>
struct NormLane {
  using Vec = RopeVec<T, V>;
  using Units = NormUnits<V, UPL, INTER>;
  static constexpr int kPairs = UPL * V / 2;  // packed

  // The element of packed number q, half i, of the as (b = 0) or bs (1): unit, and place in its two vectors.
  static __device__ __forceinline__ constexpr int unit(int q) { return 2 * q / V; }
  static __device__ __forceinline__ constexpr int place(int q, int i, int b) {
    const int p = (2 * q + i) % V;
    return INTER ? 2 * p + b : p + b * V;
  }

  static __device__ __forceinline__ void load(Vec (&v)[UPL][2], const char* x, const Units& n) {
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      v[k][0] = v[k][1] = Vec{};
      if (n.one[k]) v[k][0] = *reinterpret_cast<const Vec*>(x + n.e0[k] * static_cast<int64_t>(sizeof(T)));
      if (n.two[k]) v[k][1] = *reinterpret_cast<const Vec*>(x + n.e1[k] * static_cast<int64_t>(sizeof(T)));
    }
  }
  static __device__ __forceinline__ void unpack(const Vec (&v)[UPL][2], uint64_t (&a)[kPairs], uint64_t (&b)[kPairs]) {
    float f[UPL][2 * V];
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      rope_unpack<T, V>(v[k][0], f[k]);
      rope_unpack<T, V>(v[k][1], f[k] + V);
    }
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      constexpr int kStep = V == 1 ? 1 : 0;  // V == 1: the halves are of two units
      a[q] = f2_make(f[unit(q)][place(q, 0, 0)], f[unit(q) + kStep][place(q, 1, 0)]);
      b[q] = f2_make(f[unit(q)][place(q, 0, 1)], f[unit(q) + kStep][place(q, 1, 1)]);
    }
  }
  static __device__ __forceinline__ void store(char* out, const Units& n, const uint64_t (&a)[kPairs], const uint64_t (&b)[kPairs]) {
    float f[UPL][2 * V];
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      constexpr int kStep = V == 1 ? 1 : 0;
      const float2 x = f2_get(a[q]), y = f2_get(b[q]);
      f[unit(q)][place(q, 0, 0)] = x.x, f[unit(q) + kStep][place(q, 1, 0)] = x.y;
      f[unit(q)][place(q, 0, 1)] = y.x, f[unit(q) + kStep][place(q, 1, 1)] = y.y;
    }
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      Vec y;
      if (n.one[k]) {
        rope_pack<T, V>(y, f[k]);
        *reinterpret_cast<Vec*>(out + n.e0[k] * static_cast<int64_t>(sizeof(T))) = y;
      }
      if (n.two[k]) {
        rope_pack<T, V>(y, f[k] + V);
        *reinterpret_cast<Vec*>(out + n.e1[k] * static_cast<int64_t>(sizeof(T))) = y;
      }
    }
  }
  // What a turned channel takes of its partner; 0 where it is not turned, since an infinity times the sine 0 is NaN.
  static __device__ __forceinline__ uint64_t of_partner(uint64_t x, const Units& n, int q) {
    if constexpr (!PART) return x;
    if constexpr (V > 1) return n.turned[unit(q)] ? x : 0;
    const float2 f = f2_get(x);
    return f2_make(n.turned[unit(q)] ? f.x : 0.f, n.turned[unit(q) + 1] ? f.y : 0.f);
  }
  // f(a or b (0, 1), q, half, channel) for every channel of the lane.
  template <typename F>
  static __device__ __forceinline__ void each(const Units& n, F f) {
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = unit(q) + (V == 1 ? i : 0);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int at = place(q, i, b);
          if (at < V ? n.one[k] : n.two[k]) f(b, q, i, at < V ? n.e0[k] + at : n.e1[k] + at - V);
        }
      }
  }
  static __device__ __forceinline__ void weights(uint64_t (&wa)[kPairs], uint64_t (&wb)[kPairs], const NormArgs& a, const void* p,
                                                 const Units& n) {
    float w[2][kPairs][2];
#pragma unroll
    for (int q = 0; q < kPairs; ++q) w[0][q][0] = w[0][q][1] = w[1][q][0] = w[1][q][1] = 1.f;
    if (p != nullptr && (a.w_f32 || sizeof(T) == 4)) {
      each(n, [&](int b, int q, int i, int ch) { w[b][q][i] = static_cast<const float*>(p)[ch]; });
    } else if (p != nullptr) {
      if constexpr (sizeof(T) == 2) {
        Vec v[UPL][2];
        if ((reinterpret_cast<uintptr_t>(p) & (V * 2 - 1)) == 0) {
          load(v, static_cast<const char*>(p), n);
          unpack(v, wa, wb);
          return;
        }
        each(n, [&](int b, int q, int i, int ch) { w[b][q][i] = RopePair<T>::get(static_cast<const T*>(p)[ch]); });
      }
    }
#pragma unroll
    for (int q = 0; q < kPairs; ++q) wa[q] = f2_make(w[0][q][0], w[0][q][1]), wb[q] = f2_make(w[1][q][0], w[1][q][1]);
  }
  // As accurate as results of type S want them.
  template <typename S>
  static __device__ __forceinline__ void sines(uint64_t (&s)[kPairs], uint64_t (&c)[kPairs], const NormArgs& a, const Units& n,
                                               int lane, int64_t pos_at) {
    const uint64_t p = rope_position(a.pos, a.pos64, pos_at);
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      float x[2] = {0.f, 0.f}, y[2] = {1.f, 1.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = unit(q) + (V == 1 ? i : 0);
        const int at = (2 * q + i) % V;  // interleaved pairs stay within a vector
        const int pair = !INTER || V == 1 ? (lane + k * a.lanes) * V + at : at < V / 2 ? n.e0[k] / 2 + at : n.e1[k] / 2 + at - V / 2;
        if (n.turned[k]) rope_sincos<S>(p * a.turns[pair], a.mscale, x[i], y[i]);
      }
      s[q] = f2_make(x[0], x[1]);
      c[q] = f2_make(y[0], y[1]);
    }
  }
};

// The sum of x over the group's lanes.
__device__ __forceinline__ float group_sum(float x, int lanes, uint32_t mask) {
  for (int d = lanes >> 1; d > 0; d >>= 1) x += __shfl_xor_sync(mask, x, d);
  return x;
}
// Of two numbers at a time, whose shuffles overlap.
__device__ __forceinline__ float2 group_sums(float x, float y, int lanes, uint32_t mask) {
  for (int d = lanes >> 1; d > 0; d >>= 1) {
    const float a = __shfl_xor_sync(mask, x, d), b = __shfl_xor_sync(mask, y, d);
    x += a, y += b;
  }
  return {x, y};
}
__device__ __forceinline__ uint32_t group_mask(int lanes) {
  const uint32_t low = lanes == 32 ? 0xFFFFFFFFu : (1u << lanes) - 1u;
  return low << (threadIdx.x & 31 & ~(lanes - 1));
}

// Group (row, walker): `walk` heads of one row, from walker * walk on.
template <typename T, int V, int UPL, bool INTER, bool PART>
__global__ void __launch_bounds__(kNrThreads, kNrCtasPerSm) qk_norm_rope_kernel(const NormArgs a) {
  dependent_wait();
  dependent_launch();
  using L = NormLane<T, V, UPL, INTER, PART>;
  constexpr int kP = L::kPairs;
  const int lane = threadIdx.x & (a.lanes - 1);
  const uint32_t mask = group_mask(a.lanes);
  const unsigned rw = blockIdx.x * (kNrThreads / a.lanes) + threadIdx.x / a.lanes;
  if (rw >= a.row_walkers) return;
  const unsigned row = rw / a.walkers;
  const int first = static_cast<int>(rw - row * a.walkers) * a.walk, end = min(first + a.walk, a.heads);
  unsigned seq = 0, tok = row;
  if (a.n_seq > 1) {
    seq = row / a.n_tok;
    tok = row - seq * a.n_tok;
  }
  const NormUnits<V, UPL, INTER> n(a, lane);
  const char* const xq = a.t[0].x + seq * a.t[0].x_seq + tok * a.t[0].x_tok;
  const char* const xk = a.t[1].x + seq * a.t[1].x_seq + tok * a.t[1].x_tok;
  char* const outq = a.t[0].out + seq * a.t[0].out_seq + tok * a.t[0].out_tok;
  char* const outk = a.t[1].out + seq * a.t[1].out_seq + tok * a.t[1].out_tok;
  RopeVec<T, V> v[kNrBatch][UPL][2];
  auto load = [&](RopeVec<T, V> (&to)[UPL][2], int h) {
    if (h < end) L::load(to, h >= a.heads0 ? xk + (h - a.heads0) * a.t[1].x_head : xq + h * a.t[0].x_head, n);
  };
#pragma unroll
  for (int j = 0; j < kNrBatch; ++j) load(v[j], first + j);
  uint64_t s[kP], c[kP];
  L::template sines<T>(s, c, a, n, lane, seq * a.pos_seq + tok * a.pos_tok);
  // a' = r (a ca + b sb),  b' = r (b cb + a sa): the weights are part of the sines
  uint64_t ca[kP], cb[kP], sa[kP], sb[kP];
  int of = -1;  // the tensor whose weights they hold
  const float mean = 1.f / a.dim;
#pragma unroll 1
  for (int h0 = first; h0 < end; h0 += kNrBatch) {
#pragma unroll
    for (int j = 0; j < kNrBatch; ++j) {
      const int h = h0 + j;
      if (h >= end) break;
      const int second = h >= a.heads0;
      if (second != of) {
        L::weights(ca, cb, a, a.t[second].w, n);
#pragma unroll
        for (int q = 0; q < kP; ++q) {
          sa[q] = f2_mul(s[q], ca[q]);
          sb[q] = f2_mul(f2_mul(s[q], f2_all(-1.f)), cb[q]);
          ca[q] = f2_mul(c[q], ca[q]);
          cb[q] = f2_mul(c[q], cb[q]);
        }
        of = second;
      }
      uint64_t x[kP], y[kP], sum = 0;
      L::unpack(v[j], x, y);
      load(v[j], h + kNrBatch);
#pragma unroll
      for (int q = 0; q < kP; ++q) sum = f2_fma(y[q], y[q], f2_fma(x[q], x[q], sum));
      const uint64_t r = f2_all(rsqrtf(group_sum(f2_sum(sum), a.lanes, mask) * mean + a.eps));
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const uint64_t t = x[q];
        x[q] = f2_mul(r, f2_fma(t, ca[q], L::of_partner(f2_mul(y[q], sb[q]), n, q)));
        y[q] = f2_mul(r, f2_fma(y[q], cb[q], L::of_partner(f2_mul(t, sa[q]), n, q)));
      }
      L::store(second ? outk + (h - a.heads0) * a.t[1].out_head : outq + h * a.t[0].out_head, n, x, y);
    }
  }
}

// The heads of x and dz that a lane works on next, kAhead of them, the oldest first.  Single elements wait in registers.
template <typename T, int V, int UPL, bool INTER, bool PART, bool kVectors = V * sizeof(T) == 16>
struct NormAhead {
  using Vec = RopeVec<T, V>;
  using L = NormLane<T, V, UPL, INTER, PART>;
  static constexpr int kAhead = 1, kBytes = 16;
  const typename L::Units& n;
  Vec x[UPL][2], dz[UPL][2];
  __device__ __forceinline__ NormAhead(const typename L::Units& n, char*) : n(n) {}
  __device__ __forceinline__ void fetch(const char* from, const char* dz_from, bool there) {
    if (!there) return;
    L::load(x, from, n);
    L::load(dz, dz_from, n);
  }
  __device__ __forceinline__ void take(uint64_t (&xa)[L::kPairs], uint64_t (&xb)[L::kPairs], uint64_t (&za)[L::kPairs],
                                       uint64_t (&zb)[L::kPairs]) {
    L::unpack(x, xa, xb);
    L::unpack(dz, za, zb);
  }
};

// Vectors wait in shared memory, at places that one lane alone fills, by asynchronous copies, and reads.
template <typename T, int V, int UPL, bool INTER, bool PART>
struct NormAhead<T, V, UPL, INTER, PART, true> {
  using Vec = RopeVec<T, V>;
  using L = NormLane<T, V, UPL, INTER, PART>;
  static constexpr int kAhead = kNgAhead, kStages = kAhead + 1, kStep = kNgThreads * 16, kStage = 4 * UPL * kStep;
  static constexpr int kBytes = kStages * kStage;
  const typename L::Units& n;
  const uint32_t base;
  uint32_t put = 0, get = 0;
  __device__ __forceinline__ NormAhead(const typename L::Units& n, char* ring)
      : n(n), base(static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * 16) {}
  // Each call is a group of copies, an empty one where there is nothing.
  __device__ __forceinline__ void fetch(const char* x, const char* dz, bool there) {
    if (there) {
#pragma unroll
      for (int k = 0; k < UPL; ++k) {
        const uint32_t to = base + put + k * 4 * kStep;
        copy(to, x, n.e0[k], n.one[k]);
        copy(to + kStep, x, n.e1[k], n.two[k]);
        copy(to + 2 * kStep, dz, n.e0[k], n.one[k]);
        copy(to + 3 * kStep, dz, n.e1[k], n.two[k]);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put + kStage == kBytes ? 0 : put + kStage;
  }
  __device__ __forceinline__ void take(uint64_t (&xa)[L::kPairs], uint64_t (&xb)[L::kPairs], uint64_t (&za)[L::kPairs],
                                       uint64_t (&zb)[L::kPairs]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    Vec x[UPL][2], dz[UPL][2];
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      const uint32_t at = base + get + k * 4 * kStep;
      read(x[k][0], at);
      read(x[k][1], at + kStep);
      read(dz[k][0], at + 2 * kStep);
      read(dz[k][1], at + 3 * kStep);
    }
    L::unpack(x, xa, xb);
    L::unpack(dz, za, zb);
    get = get + kStage == kBytes ? 0 : get + kStage;
  }
  // 16 bytes, zeros where there is nothing.
  static __device__ __forceinline__ void copy(uint32_t to, const char* from, int element, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                 "l"(from + (there ? element : 0) * static_cast<int64_t>(sizeof(T))), "r"(there ? 16 : 0)
                 : "memory");
  }
  static __device__ __forceinline__ void read(Vec& v, uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    memcpy(&v, &w, 16);
  }
};

// CTAs below ctas0 take the first tensor, the others the second; their groups take (row, walker) in turn.
template <typename T, int V, int UPL, bool INTER, bool PART>
__global__ void __launch_bounds__(kNgThreads, kNgCtasPerSm) qk_norm_rope_gradient_kernel(const NormArgs a) {
  using Ahead = NormAhead<T, V, UPL, INTER, PART>;
  constexpr int kAhead = Ahead::kAhead;
  constexpr int kSums = kNgThreads * UPL * 2 * V * static_cast<int>(sizeof(float));
  __shared__ __align__(16) char ring[Ahead::kBytes > kSums ? Ahead::kBytes : kSums];
  float* const sums = reinterpret_cast<float*>(ring);  // [group][dim], when the heads are through
  dependent_wait();
  dependent_launch();
  using L = NormLane<T, V, UPL, INTER, PART>;
  constexpr int kP = L::kPairs;
  const int lane = threadIdx.x & (a.lanes - 1), groups = kNgThreads / a.lanes, group = threadIdx.x / a.lanes;
  const uint32_t mask = group_mask(a.lanes);
  const bool second = blockIdx.x >= a.ctas0;
  const NormTensor& t = a.t[second];
  const int n_heads = second ? a.heads - a.heads0 : a.heads0, walk = second ? a.walk1 : a.walk;
  const unsigned walkers = second ? a.walkers1 : a.walkers;
  const unsigned cta = second ? blockIdx.x - a.ctas0 : blockIdx.x, ctas = second ? gridDim.x - a.ctas0 : a.ctas0;
  const unsigned rows = a.n_seq * a.n_tok;
  const NormUnits<V, UPL, INTER> n(a, lane);
  const float mean = 1.f / a.dim;
  uint64_t wa[kP], wb[kP], da[kP], db[kP];
  L::weights(wa, wb, a, t.w, n);
#pragma unroll
  for (int q = 0; q < kP; ++q) da[q] = db[q] = 0;
  Ahead in(n, ring);
  const unsigned walks = rows * walkers, step = ctas * groups;
  auto place = [&](unsigned rw, unsigned& seq, unsigned& tok, int& first) {  // -> heads of walk rw
    const unsigned row = rw / walkers;
    first = (rw - row * walkers) * walk;
    seq = 0, tok = row;
    if (a.n_seq > 1) {
      seq = row / a.n_tok;
      tok = row - seq * a.n_tok;
    }
    return min(walk, n_heads - first);
  };
  // What is fetched next: `left` more heads of walk `ahead`, at x and dz.
  unsigned ahead = cta * groups + group - step;
  int left = 0;
  const char *x = nullptr, *dz = nullptr;
  auto fetch = [&] {
    if (left == 0) {
      ahead += step;
      if (ahead < walks) {
        unsigned seq, tok;
        int first;
        left = place(ahead, seq, tok, first);
        x = t.x + seq * t.x_seq + tok * t.x_tok + first * t.x_head;
        dz = t.dz + seq * t.dz_seq + tok * t.dz_tok + first * t.dz_head;
      } else {
        ahead -= step;
      }
    }
    in.fetch(x, dz, left > 0);
    if (left > 0) --left, x += t.x_head, dz += t.dz_head;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) fetch();
#pragma unroll 1
  for (unsigned rw = cta * groups + group; rw < walks; rw += step) {
    unsigned seq, tok;
    int first;
    const int n_walk = place(rw, seq, tok, first);
    char* out = t.out + seq * t.out_seq + tok * t.out_tok + first * t.out_head;
    uint64_t s[kP], c[kP];
    L::template sines<float>(s, c, a, n, lane, seq * a.pos_seq + tok * a.pos_tok);  // dw is fp32
#pragma unroll 1
    for (int h = 0; h < n_walk; ++h, out += t.out_head) {
      uint64_t xa[kP], xb[kP], ga[kP], gb[kP], ta[kP], tb[kP], xx = 0, hx = 0;
      in.take(xa, xb, ga, gb);
      fetch();
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const uint64_t g0 = ga[q], minus = f2_mul(s[q], f2_all(-1.f));
        ga[q] = f2_fma(g0, c[q], L::of_partner(f2_mul(gb[q], s[q]), n, q));
        gb[q] = f2_fma(gb[q], c[q], L::of_partner(f2_mul(g0, minus), n, q));
        ta[q] = f2_mul(ga[q], xa[q]);
        tb[q] = f2_mul(gb[q], xb[q]);
        xx = f2_fma(xb[q], xb[q], f2_fma(xa[q], xa[q], xx));
        hx = f2_fma(tb[q], wb[q], f2_fma(ta[q], wa[q], hx));
      }
      const float2 sum = group_sums(f2_sum(xx), f2_sum(hx), a.lanes, mask);
      const float r = rsqrtf(sum.x * mean + a.eps);
      const float m = sum.y * mean * r;  // the mean of h x r
      const uint64_t r2 = f2_all(r), k2 = f2_all(-r * r * m);
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        da[q] = f2_fma(ta[q], r2, da[q]);
        db[q] = f2_fma(tb[q], r2, db[q]);
        xa[q] = f2_fma(f2_mul(ga[q], wa[q]), r2, f2_mul(xa[q], k2));
        xb[q] = f2_fma(f2_mul(gb[q], wb[q]), r2, f2_mul(xb[q], k2));
      }
      L::store(out, n, xa, xb);
    }
  }
  __syncthreads();  // no head waits any more
  L::each(n, [&](int b, int q, int i, int ch) {
    const float2 d = f2_get(b ? db[q] : da[q]);
    sums[group * a.dim + ch] = i ? d.y : d.x;
  });
  __syncthreads();
  for (int ch = threadIdx.x; ch < a.dim; ch += kNgThreads) {
    float sum = 0.f;
    for (int i = 0; i < groups; ++i) sum += sums[i * a.dim + ch];
    a.part[static_cast<int64_t>(blockIdx.x) * a.dim + ch] = sum;
  }
}

// dw of 32 channels of one tensor: 32 threads each, in 32 runs of its CTAs that are joined in order.
__global__ void __launch_bounds__(1024) norm_weights_kernel(const float* part, int ctas0, int ctas, int dim, float* dw0, float* dw1) {
  __shared__ float sums[32][33];
  dependent_wait();
  dependent_launch();
  const int ch = threadIdx.x & 31, run = threadIdx.x >> 5, at = blockIdx.x * 32 + ch;
  const int begin = blockIdx.y == 0 ? 0 : ctas0, end = blockIdx.y == 0 ? ctas0 : ctas;
  float* const dw = blockIdx.y == 0 ? dw0 : dw1;
  if (dw == nullptr) return;
  const int per = (end - begin + 31) / 32;
  float sum = 0.f;
  if (at < dim) {
#pragma unroll 16
    for (int i = begin + run * per; i < min(end, begin + (run + 1) * per); ++i) sum += __ldcg(part + static_cast<int64_t>(i) * dim + at);
  }
  sums[run][ch] = sum;
  __syncthreads();
  if (run == 0 && at < dim) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sums[i][ch];
    dw[at] = sum;
  }
}

template <typename T, int V, int UPL, bool INTER, bool PART>
static int norm_launch(const NormArgs& a, int grid, void* stream) {
  if (grid > 0) return kv8_launch(qk_norm_rope_gradient_kernel<T, V, UPL, INTER, PART>, dim3(grid), kNgThreads, 0, stream, a);
  const unsigned per = kNrThreads / a.lanes;
  return kv8_launch(qk_norm_rope_kernel<T, V, UPL, INTER, PART>, dim3((a.row_walkers + per - 1) / per), kNrThreads, 0, stream, a);
}
template <typename T>
static int norm_launch(const NormArgs& a, bool wide, bool inter, int grid, void* stream) {
  constexpr int V = 16 / sizeof(T);
  if (!wide) return inter ? norm_launch<T, 1, 4, true, true>(a, grid, stream) : norm_launch<T, 1, 4, false, true>(a, grid, stream);
  if (a.rot < a.dim) return inter ? norm_launch<T, V, 1, true, true>(a, grid, stream) : norm_launch<T, V, 1, false, true>(a, grid, stream);
  return inter ? norm_launch<T, V, 1, true, false>(a, grid, stream) : norm_launch<T, V, 1, false, false>(a, grid, stream);
}

struct Span {  // the elements of one tensor, in bytes
  uintptr_t begin, end;
};

// The arguments of either call.  grid: 0 for the forward pass, else where the gradient's CTAs go.
static int norm_rope(const gaac_norm_tensor* tensors, int n_tensors, int dtype, int weight_dtype, int64_t n_seq, int64_t n_tok,
                     int head_dim, int rot_dim, const void* positions, int pos_bits, int64_t pos_seq_stride,
                     int64_t pos_tok_stride, const uint64_t* turns, float mscale, float eps, unsigned flags, bool gradient,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (tensors == nullptr || n_tensors < 1 || n_tensors > 2 || (dtype != GAAC_BF16 && dtype != GAAC_F16 && dtype != GAAC_F32) ||
      (weight_dtype != dtype && weight_dtype != GAAC_F32) || (pos_bits != 32 && pos_bits != 64) ||
      (flags & ~static_cast<unsigned>(GAAC_ROPE_INTERLEAVED)) || !std::isfinite(mscale) || !std::isfinite(eps) || eps < 0.f)
    return GAAC_EINVAL;
  if (n_seq < 0 || n_tok < 0 || n_seq > 0x7FFFFFFF || n_tok > 0x7FFFFFFF || head_dim < 2 || head_dim > kNrMaxDim || (head_dim & 1) ||
      rot_dim < 2 || rot_dim > head_dim || (rot_dim & 1))
    return GAAC_EINVAL;
  const int64_t rows = n_seq * n_tok;
  if (rows > 0x7FFFFFFF) return GAAC_EINVAL;
  int64_t heads = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const gaac_norm_tensor& t = tensors[i];
    if (t.n_heads < 1 || t.n_heads > 65536 || (reinterpret_cast<uintptr_t>(t.weight) & (weight_dtype == GAAC_F32 ? 3u : 1u)) ||
        (gradient && (reinterpret_cast<uintptr_t>(t.dweight) & 3u)))
      return GAAC_EINVAL;
    heads += t.n_heads;
  }
  if (gradient && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
                   workspace_bytes < gaac_qk_norm_rope_workspace(head_dim)))
    return GAAC_EINVAL;
  if (gradient && n_tensors == 2 && tensors[0].dweight != nullptr && tensors[0].dweight == tensors[1].dweight) return GAAC_EINVAL;
  if (rows == 0 && !gradient) return GAAC_OK;
  if (rows > 0 && (positions == nullptr || turns == nullptr || pos_seq_stride < 0 || pos_tok_stride < 0 ||
                   (reinterpret_cast<uintptr_t>(positions) & (pos_bits / 8 - 1)) || (reinterpret_cast<uintptr_t>(turns) & 7u)))
    return GAAC_EINVAL;
  const int size = dtype == GAAC_F32 ? 4 : 2, full = 16 / size;
  bool wide = (rot_dim / 2) % full == 0 && (head_dim - rot_dim) % full == 0;
  NormArgs a = {};
  for (int i = 0; i < n_tensors && rows > 0; ++i) {
    const gaac_norm_tensor& t = tensors[i];
    if (t.x == nullptr || t.out == nullptr || (gradient && t.dz == nullptr)) return GAAC_EINVAL;
    const int64_t most = int64_t{1} << 56;
    const int64_t strides[9] = {t.x_seq, t.x_tok, t.x_head, t.out_seq, t.out_tok, t.out_head, t.dz_seq, t.dz_tok, t.dz_head};
    const int64_t counts[3] = {n_seq, n_tok, t.n_heads};
    int64_t all = 0;
    for (int k = 0; k < (gradient ? 9 : 6); ++k) {
      if (strides[k] < 0 || strides[k] > most / counts[k % 3]) return GAAC_EINVAL;
      if (counts[k % 3] > 1) all |= strides[k];
    }
    int64_t count[3] = {n_seq, n_tok, t.n_heads}, so[3] = {t.out_seq, t.out_tok, t.out_head};
    if (!distinct(head_dim, count, so)) return GAAC_EINVAL;
    auto span = [&](const void* p, const int64_t* s) {
      const uintptr_t b = reinterpret_cast<uintptr_t>(p);
      return Span{b, b + ((n_seq - 1) * s[0] + (n_tok - 1) * s[1] + (t.n_heads - 1) * s[2] + head_dim) * size};
    };
    const Span x = span(t.x, strides), o = span(t.out, strides + 3), z = gradient ? span(t.dz, strides + 6) : x;
    const uintptr_t addresses = x.begin | o.begin | z.begin;
    if (addresses & (size - 1)) return GAAC_EINVAL;
    // In place means the same elements, of x or of dz; any other overlap would read what has been written.
    auto clash = [&](const Span& in, const int64_t* s) {
      bool same = in.begin == o.begin;
      for (int k = 0; k < 3; ++k) same = same && (counts[k] == 1 || s[k] == strides[3 + k]);
      return !same && in.begin < o.end && o.begin < in.end;
    };
    if (clash(x, strides) || (gradient && clash(z, strides + 6))) return GAAC_EINVAL;
    wide = wide && all % full == 0 && (addresses & 15u) == 0;
    a.t[i] = NormTensor{static_cast<const char*>(t.x), static_cast<const char*>(t.dz), static_cast<char*>(t.out), t.weight, t.dweight,
                        t.x_seq * size, t.x_tok * size, t.x_head * size, t.dz_seq * size, t.dz_tok * size, t.dz_head * size,
                        t.out_seq * size, t.out_tok * size, t.out_head * size};
  }
  if (rows == 0)
    for (int i = 0; i < n_tensors; ++i) a.t[i].dw = tensors[i].dweight;
  // Two tensors with a first element in common, one of them an output (the caller keeps other overlaps apart).
  if (n_tensors == 2 && rows > 0) {
    const void* o[2] = {tensors[0].out, tensors[1].out};
    for (int i = 0; i < 2; ++i)
      if (o[i] == o[1 - i] || o[i] == tensors[1 - i].x || (gradient && o[i] == tensors[1 - i].dz)) return GAAC_EINVAL;
  }
  const int v = wide ? full : 1;
  a.heads0 = tensors[0].n_heads;
  a.heads = static_cast<int>(heads);
  a.n_seq = static_cast<unsigned>(n_seq);
  a.n_tok = static_cast<unsigned>(n_tok);
  a.rot = rot_dim;
  a.dim = head_dim;
  a.w_f32 = weight_dtype == GAAC_F32;
  a.pos = positions;
  a.pos64 = pos_bits == 64;
  a.pos_seq = pos_seq_stride;
  a.pos_tok = pos_tok_stride;
  a.turns = turns;
  a.mscale = mscale;
  a.eps = eps;
  a.rot_units = rot_dim / 2 / v;
  a.units = a.rot_units + ((head_dim - rot_dim) / v + 1) / 2;
  a.lanes = 2;
  while (a.lanes < 32 && a.lanes < a.units) a.lanes *= 2;
  // Heads of a walk: as many as leave four times the lanes that 152 SMs hold at a time (gradient: one walk for each group that
  // they hold), so that sines are shared where there is work for all, and single heads where latency counts.
  const int64_t want = int64_t{152} * (gradient ? kNgThreads * kNgCtasPerSm : 4 * kNrThreads * kNrCtasPerSm), lanes = std::max<int64_t>(rows, 1) * heads * a.lanes;
  const int64_t fair = std::max<int64_t>(1, gradient ? (lanes + want - 1) / want : lanes / want);
  const int64_t walkers_most = 0x7FFFFFFF / std::max<int64_t>(rows, 1);  // walks are counted in 31 bits
  if (gradient) {  // walks of like lengths
    auto of = [&](int n, int* walk) {
      const int most = static_cast<int>(std::max(std::min<int64_t>(fair, kNgMost), (n + walkers_most - 1) / walkers_most));
      const int walkers = (n + most - 1) / most;
      *walk = walkers > 0 ? (n + walkers - 1) / walkers : 1;
      return walkers;
    };
    a.walkers = of(a.heads0, &a.walk);
    a.walkers1 = of(a.heads - a.heads0, &a.walk1);
  } else {
    a.walk = static_cast<int>(std::max(std::min<int64_t>(kNrMost, fair), (heads + walkers_most - 1) / walkers_most));
    a.walkers = (a.heads + a.walk - 1) / a.walk;
  }
  a.row_walkers = static_cast<unsigned>(rows * a.walkers);
  a.part = static_cast<float*>(workspace);
  int grid = 0;
  if (gradient) {  // CTAs of either tensor in the ratio of their heads
    const int64_t per = kNgThreads / a.lanes;
    auto ctas = [&](int n, int walkers) {
      const int64_t share = std::max<int64_t>(1, (kNgMostCtas - 1) * static_cast<int64_t>(n) / heads);
      return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(share, (rows * walkers + per - 1) / per)));
    };
    a.ctas0 = ctas(a.heads0, a.walkers);
    grid = a.ctas0 + (n_tensors == 2 ? ctas(a.heads - a.heads0, a.walkers1) : 0);
  }
  const bool inter = (flags & GAAC_ROPE_INTERLEAVED) != 0;
  const int e = dtype == GAAC_BF16  ? norm_launch<__nv_bfloat16>(a, wide, inter, grid, stream)
                : dtype == GAAC_F16 ? norm_launch<__half>(a, wide, inter, grid, stream)
                                    : norm_launch<float>(a, wide, inter, grid, stream);
  if (e != GAAC_OK || !gradient) return e;
  if (a.t[0].dw == nullptr && a.t[1].dw == nullptr) return GAAC_OK;
  return kv8_launch(norm_weights_kernel, dim3((head_dim + 31) / 32, n_tensors), 1024, 0, stream, static_cast<const float*>(a.part),
                    static_cast<int>(a.ctas0), grid, head_dim, a.t[0].dw, a.t[1].dw);
}

}  // namespace gaac

using namespace gaac;

extern "C" size_t gaac_qk_norm_rope_workspace(int head_dim) {
  if (head_dim < 2 || head_dim > kNrMaxDim) return 0;
  return (static_cast<size_t>(kNgMostCtas + 1) * head_dim * sizeof(float) + 15) & ~static_cast<size_t>(15);
}

extern "C" int gaac_qk_norm_rope(const gaac_norm_tensor* tensors, int n_tensors, int dtype, int weight_dtype, int64_t n_seq,
                                 int64_t n_tok, int head_dim, int rot_dim, const void* positions, int pos_bits,
                                 int64_t pos_seq_stride, int64_t pos_tok_stride, const uint64_t* turns, float mscale, float eps,
                                 unsigned flags, void* stream) {
  return norm_rope(tensors, n_tensors, dtype, weight_dtype, n_seq, n_tok, head_dim, rot_dim, positions, pos_bits, pos_seq_stride,
                   pos_tok_stride, turns, mscale, eps, flags, false, nullptr, 0, stream);
}

extern "C" int gaac_qk_norm_rope_gradient(const gaac_norm_tensor* tensors, int n_tensors, int dtype, int weight_dtype,
                                          int64_t n_seq, int64_t n_tok, int head_dim, int rot_dim, const void* positions,
                                          int pos_bits, int64_t pos_seq_stride, int64_t pos_tok_stride, const uint64_t* turns,
                                          float mscale, float eps, unsigned flags, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  return norm_rope(tensors, n_tensors, dtype, weight_dtype, n_seq, n_tok, head_dim, rot_dim, positions, pos_bits, pos_seq_stride,
                   pos_tok_stride, turns, mscale, eps, flags, true, workspace, workspace_bytes, stream);
}
