// Decode attention over the 8-bit paged cache.
//
//   s_t = scale * sK * (q . k8_t),   out = sum_t softmax(s)_t * sV * v8_t
// with sK, sV the scales of t's block (1 for the open block, which is in the model's type).
//
// Memory bound: 256 bytes per token and kv-head are read once, and 4 * (query heads) * 128 operations per token
// hide under them.  Two CTAs per SM, each of four compute warps and one copy warp:
//  * Work is cut evenly, whatever the lengths: the (sequence, kv-head) pairs' blocks in one row of units (a page is
//    one unit, an open block two, an empty sequence one), CTA i of G takes units [i U/G, (i+1) U/G).  A pair that
//    spans CTAs is joined by the last of them to finish; a CTA has at most two such pairs, its first and its last.
//  * The copy warp walks the units: one tensor copy (TMA, 128-byte swizzle) brings K and V of a page and head, which
//    lie together (16 KB), into a ring of stages; the scales ride along as an 8-byte asynchronous copy, the
//    pair's queries as a bulk copy with its first unit.  Everything a unit's consumers need is in its stage.
//  * Compute warp w takes tokens [16w, 16w+16) of every block and keeps its own softmax state.  S = K q^T with K as
//    the 16-row operand (mma.sync m16n8k16, 8 columns = query heads of the kv-head): the decode step has at most
//    8 rows, so the wide operand is the cache and no tensor-core work is spent on padding tokens; tcgen05's 128-row
//    tile would be.  O^T = V^T P^T uses the transposed 8-bit V straight from ldmatrix.trans (pairs of channels).
//  * FP8 becomes f16 in registers (exact).  The query is scaled by a power of two per row into f16's range (exact
//    but for parts below 2^-28 of the row's largest), the scale is put back with sK.
//  * Two running maxima per row: m of the logits, for the softmax's sum l; and M of logit + log2 sV, for the
//    weights 2^(s + log2 sV - M + 15) that go to the tensor cores as f16: whatever the blocks' scales, the largest
//    weight is 2^15 and those down to 2^-29 of it keep f16's 11 bits.  m, l, M and O are fp32.
//  * The open block is multiplied in its own type (bf16: the weights as a high and a low part).
#include <cuda.h>

#include <algorithm>

#include "kv8.cuh"

namespace gaac {

constexpr int kKaWarps = 4;                  // compute warps
constexpr int kKaThreads = 32 * (kKaWarps + 1);
constexpr int kKaStages = 5;
constexpr int kKaCtasPerSm = 2;
constexpr int kKaRows = 8;                   // query heads per kv-head in the MMA columns
constexpr int kKaMinUnits = 2;               // fewer units than this are not worth a CTA
constexpr int kKaStride = kD + 4;            // floats per row of a warp's state in shared memory (bank spread)
constexpr int kKaQStride = 2 * kD + 8;       // bytes per query row kept for the open block
constexpr int kKaPart = 3 * kKaRows + kKaRows * kD;  // floats of a partial: m, l, M, O
constexpr uint32_t kKaFull = 0xFFFFFFFFu;

enum { kUnitPage = 0, kUnitOpen = 1, kUnitNone = 2, kUnitEnd = 3 };

struct KaMeta {
  int kind, first, last;
  int n_tok;               // open block: its tokens
  int b, h;
  int cta0, n_cta;         // the CTAs that share the pair
};

struct KaSmem {
  alignas(1024) uint8_t stage[kKaStages][kKv8Pair];
  alignas(128) uint16_t q[kKaStages][kKaRows * kD];
  alignas(16) float state[kKaWarps][kKaRows][kKaStride];
  alignas(16) uint8_t qraw[kKaRows][kKaQStride];
  alignas(16) float2 scale[kKaStages];
  KaMeta meta[kKaStages];
  float m[kKaWarps][kKaRows], l[kKaWarps][kKaRows], mv[kKaWarps][kKaRows];
  uint64_t full[kKaStages], empty[kKaStages], sync;
  int last;
};

struct KaArgs {
  Kv8Dev c;
  const uint16_t* q;
  int64_t q_seq;
  void* out;
  int out_f32, r;
  float c_log2;  // scale * log2(e)
  int32_t* counters;
  float* part;
  int32_t* status;
};

__device__ __forceinline__ void ka_mma_f16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ka_ldmatrix(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ka_ldmatrix_t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t ka_transpose(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ka_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t ka_pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t ka_pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void ka_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ------------------------------------------------------------------ units

struct KaSeq {  // a sequence's units per kv-head
  int full, open, units;
};
__device__ __forceinline__ KaSeq ka_seq(const Kv8Dev& c, int len) {
  if (len < 0 || len > static_cast<int64_t>(c.max_blocks) * kBlock) len = 0;
  KaSeq s;
  s.full = len / kBlock;
  s.open = len % kBlock;
  s.units = max(1, s.full + (s.open ? 2 : 0));
  return s;
}

__device__ __forceinline__ void ka_tma(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// A bounded wait that the whole warp takes alike.
__device__ __forceinline__ bool ka_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(kKaFull, mbar_wait(bar, parity, status));
}

// The copy warp's ring position; every call by the whole warp.
struct KaRing {
  int stage = 0;
  uint32_t phase = 0;
  int issued = 0;
};

// Waits for the next stage to be free.  false: gave up.
__device__ __forceinline__ bool ka_acquire(KaSmem& sm, KaRing& r, int32_t* status) {
  if (r.issued >= kKaStages) {
    if (!ka_wait(&sm.empty[r.stage], r.phase ^ 1u, status)) return false;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  return true;
}
__device__ __forceinline__ void ka_next(KaRing& r) {
  ++r.issued;
  if (++r.stage == kKaStages) {
    r.stage = 0;
    r.phase ^= 1u;
  }
}

__device__ void ka_copy_warp(const KaArgs& a, KaSmem& sm, const CUtensorMap* pages, const CUtensorMap* tail) {
  const Kv8Dev& c = a.c;
  const int lane = threadIdx.x & 31;
  KaRing ring;
  // ---- all units, then this CTA's and where they begin
  int64_t total = 0;
  for (int b0 = 0; b0 < c.batch; b0 += 32) {
    int u = 0;
    if (b0 + lane < c.batch) {
      const int len = c.lens[b0 + lane];
      if (blockIdx.x == 0 && (len < 0 || len > static_cast<int64_t>(c.max_blocks) * kBlock)) report(a.status, GAAC_EINVAL);
      u = ka_seq(c, len).units;
    }
    // 32 sequences of up to 2^24 + 2 units: 30 bits
    total += static_cast<int64_t>(__reduce_add_sync(kKaFull, u)) * c.heads;
  }
  const int64_t G = min(static_cast<int64_t>(gridDim.x), (total + kKaMinUnits - 1) / kKaMinUnits);
  const int64_t u_begin = static_cast<int64_t>(blockIdx.x) * total / G, u_end = (static_cast<int64_t>(blockIdx.x) + 1) * total / G;
  bool ok = true;
  if (blockIdx.x < G && u_begin < u_end) {
    int b = 0;
    int64_t base = 0;  // units before sequence b
    int len32 = 0, b32 = -1;
    for (int b0 = 0; b0 < c.batch; b0 += 32) {
      const int len = b0 + lane < c.batch ? c.lens[b0 + lane] : 0;
      const int64_t u = b0 + lane < c.batch ? static_cast<int64_t>(ka_seq(c, len).units) * c.heads : 0;
      int64_t incl = u;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(kKaFull, incl, d);
        if (lane >= d) incl += v;
      }
      const uint32_t past = __ballot_sync(kKaFull, base + incl > u_begin);
      if (past) {
        const int at = __ffs(past) - 1;
        base += __shfl_sync(kKaFull, incl - u, at);
        b = b0 + at;
        len32 = len;
        b32 = b0;
        break;
      }
      base += __shfl_sync(kKaFull, incl, 31);
    }
    KaSeq s = ka_seq(c, __shfl_sync(kKaFull, len32, b - b32));
    int h = static_cast<int>((u_begin - base) / s.units);
    int64_t seg = base + static_cast<int64_t>(h) * s.units;  // first unit of the pair
    int64_t u = u_begin;
    while (u < u_end && ok) {
      const int l0 = static_cast<int>(u - seg);
      int l1 = static_cast<int>(min(u_end, seg + s.units) - seg);
      // An open block's two units go together to the CTA that has the first.
      const bool skip = s.open && l0 == s.full + 1;
      if (!skip) {
        if (s.open && l1 > s.full) l1 = s.full + 2;
        const int64_t tail_unit = seg + s.units - (s.open ? 2 : 1);
        KaMeta meta;
        meta.b = b;
        meta.h = h;
        meta.cta0 = static_cast<int>(((seg + 1) * G - 1) / total);
        meta.n_cta = static_cast<int>(((tail_unit + 1) * G - 1) / total) - meta.cta0 + 1;
        meta.n_tok = s.open;
        const int blk_end = min(l1, s.full);
        const bool with_open = s.open && l1 > s.full;
        const uint32_t q_bytes = static_cast<uint32_t>(a.r) * kD * 2;
        const uint16_t* q = a.q + b * a.q_seq + static_cast<int64_t>(h) * a.r * kD;
        bool first = true;
        const int32_t* row = c.table + static_cast<int64_t>(b) * c.max_blocks;
        int32_t pg = l0 + lane < blk_end ? row[l0 + lane] : 0;
        for (int blk0 = l0; blk0 < blk_end && ok; blk0 += 32) {
          const int32_t pg_next = blk0 + 32 + lane < blk_end ? row[blk0 + 32 + lane] : 0;
          const int n = min(32, blk_end - blk0);
          for (int i = 0; i < n && ok; ++i) {
            const int32_t page = __shfl_sync(kKaFull, pg, i);
            ok = ka_acquire(sm, ring, a.status);
            if (lane == 0 && ok) {
              const bool valid = page >= 0 && page < c.n_pages;
              if (!valid) report(a.status, GAAC_EFORMAT);
              meta.kind = valid ? kUnitPage : kUnitNone;
              meta.first = first;
              meta.last = !with_open && blk0 + i + 1 == blk_end;
              sm.meta[ring.stage] = meta;
              uint64_t* full = &sm.full[ring.stage];
              const int64_t tile = static_cast<int64_t>(valid ? page : 0) * c.heads + h;
              if (valid) {
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(&sm.scale[ring.stage])),
                             "l"(c.scales + 2 * tile) : "memory");
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(full)) : "memory");
              } else {
                ka_arrive(full);
              }
              mbar_arrive_expect_tx(full, (valid ? kKv8Pair : 0) + (first ? q_bytes : 0));
              if (valid) ka_tma(sm.stage[ring.stage], pages, 0, static_cast<int>(tile * 2 * kBlock), full);
              if (first) bulk_g2s(sm.q[ring.stage], q, q_bytes, full);
            }
            first = false;
            ka_next(ring);
          }
          pg = pg_next;
        }
        if (with_open && ok) {
#pragma unroll 1
          for (int kind = 0; kind < 2 && ok; ++kind) {
            ok = ka_acquire(sm, ring, a.status);
            if (lane == 0 && ok) {
              meta.kind = kUnitOpen;
              meta.first = first;
              meta.last = 1;
              sm.meta[ring.stage] = meta;
              uint64_t* full = &sm.full[ring.stage];
              ka_arrive(full);
              mbar_arrive_expect_tx(full, kKv8Pair + (first ? q_bytes : 0));
              const int y = static_cast<int>(((static_cast<int64_t>(b) * c.heads + h) * 2 + kind) * kBlock);
              ka_tma(sm.stage[ring.stage], tail, 0, y, full);
              ka_tma(sm.stage[ring.stage] + kKv8Tile, tail, kD / 2, y, full);
              if (first) bulk_g2s(sm.q[ring.stage], q, q_bytes, full);
            }
            first = false;
            ka_next(ring);
          }
        } else if (s.units == 1 && s.full == 0 && ok) {  // an empty sequence
          ok = ka_acquire(sm, ring, a.status);
          if (lane == 0 && ok) {
            meta.kind = kUnitNone;
            meta.first = 1;
            meta.last = 1;
            sm.meta[ring.stage] = meta;
            ka_arrive(&sm.full[ring.stage]);
            mbar_arrive_expect_tx(&sm.full[ring.stage], q_bytes);
            bulk_g2s(sm.q[ring.stage], q, q_bytes, &sm.full[ring.stage]);
          }
          ka_next(ring);
        }
      }
      // ---- the next pair
      seg += s.units;
      u = seg;
      if (++h == c.heads) {
        h = 0;
        if (++b >= c.batch) break;
        if (b - b32 >= 32) {
          b32 += 32;
          len32 = b32 + lane < c.batch ? c.lens[b32 + lane] : 0;
        }
        s = ka_seq(c, __shfl_sync(kKaFull, len32, b - b32));
      }
    }
  }
  if (ok) ok = ka_acquire(sm, ring, a.status);
  if (ok) {
    if (lane == 0) {
      sm.meta[ring.stage].kind = kUnitEnd;
      ka_arrive(&sm.full[ring.stage]);
      ka_arrive(&sm.full[ring.stage]);
    }
  }
  // No copy may be in flight when the CTA ends, not even where a consumer's wait ran out: the last use of every stage
  // is waited for (bounded).  The end unit has taken the stage of the oldest of them, which was consumed.
  const int n = min(ring.issued, ok ? kKaStages - 1 : kKaStages);
  for (int i = 0; i < n; ++i) {
    const int j = ring.issued - 1 - i;
    mbar_wait(&sm.full[j % kKaStages], (j / kKaStages) & 1, a.status);
  }
}

// ------------------------------------------------------------------ compute warps

struct KaSync {
  uint32_t phase = 0;
};
// The four compute warps meet.  false: gave up.
__device__ __forceinline__ bool ka_meet(KaSmem& sm, KaSync& s, int32_t* status) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ka_arrive(&sm.sync);
  const bool ok = ka_wait(&sm.sync, s.phase, status);
  s.phase ^= 1u;
  return ok;
}

__device__ __forceinline__ float ka_finite(float m) { return m == -INFINITY ? 0.f : m; }

template <bool HALF>
__device__ __forceinline__ void ka_store(const KaArgs& a, int b, int h, int row, int ch, float4 y) {
  const int64_t at = (static_cast<int64_t>(b) * a.c.heads + h) * a.r * kD + row * kD + ch;
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
  else if (HALF)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(ka_pack_f16(y.x, y.y), ka_pack_f16(y.z, y.w));
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(ka_pack_bf16(y.x, y.y), ka_pack_bf16(y.z, y.w));
}

// O, in units of 2^M, over the sum l, in units of 2^m: halves of the exponent on either side of the division, so
// that neither leaves fp32 before the result does.
__device__ __forceinline__ float4 ka_result(float4 o, float m, float l, float mv) {
  if (l == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
  const float e = ka_exp2(0.5f * (ka_finite(mv) - ka_finite(m)));
  return make_float4(o.x * e / l * e, o.y * e / l * e, o.z * e / l * e, o.w * e / l * e);
}

template <bool HALF, int FMT>
__device__ void ka_compute(const KaArgs& a, KaSmem& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  KaSync meet;
  int stage = 0;
  uint32_t phase = 0;
  uint32_t qf[8][2];       // q^T operand: row g, channels 16 j + 4 tq .. + 3 of k-step j
  float qc[2];             // logit factor of rows 2 tq, 2 tq + 1 before sK: scale * log2(e) / (the row's power of two)
  float acc[8][4];         // O^T: [16-channel tile][(channel 2g, row 2tq), (2g, 2tq+1), (2g+1, 2tq), (2g+1, 2tq+1)]
  float m[2], l[2], mv[2];
#pragma unroll
  for (int j = 0; j < 8; ++j) qf[j][0] = qf[j][1] = 0u;
  qc[0] = qc[1] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  m[0] = m[1] = mv[0] = mv[1] = -INFINITY;
  l[0] = l[1] = 0.f;
  // addresses of this lane's ldmatrix rows within a stage
  const int i8 = lane >> 3, r8 = lane & 7;
  const uint32_t k_row = static_cast<uint32_t>(16 * warp + 8 * (i8 & 1) + r8);   // K: matrices (tokens 0-7, 8-15) x (chunk, chunk + 1)
  const uint32_t k_off = k_row * kD;
  const uint32_t v_off = kKv8Tile + k_off;                                        // V: the same tokens, read transposed
  const uint32_t half = static_cast<uint32_t>(i8 >> 1);

  while (true) {
    if (!ka_wait(&sm.full[stage], phase, a.status)) return;
    const KaMeta& meta = sm.meta[stage];
    const int kind = meta.kind;
    if (kind == kUnitEnd) return;
    const bool last = meta.last;
    if (meta.first) {
      // ---- the pair's queries
      const uint16_t* qs = sm.q[stage];
      uint32_t w[8][2];
      uint32_t big = 0;  // largest finite magnitude of this lane's part of row g, as a 16-bit pattern
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint2 x = make_uint2(0u, 0u);
        if (g < a.r) x = *reinterpret_cast<const uint2*>(qs + g * kD + 16 * j + 4 * tq);
        w[j][0] = x.x, w[j][1] = x.y;
        *reinterpret_cast<uint2*>(sm.qraw[g] + 2 * (16 * j + 4 * tq)) = x;  // every warp writes the same
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t mag = w[j][i] & 0x7FFF7FFFu;
          big = __vmaxu2(big, mag & ~__vcmpgeu2(mag, HALF ? 0x7C007C00u : 0x7F807F80u));
        }
      }
      big = max(big & 0xFFFFu, big >> 16);
      big = max(big, __shfl_xor_sync(kKaFull, big, 1));
      big = max(big, __shfl_xor_sync(kKaFull, big, 2));
      // row's power of two: its largest magnitude to [2^14, 2^15); both factors of it are normal numbers
      int e = 0;
      if (big != 0u) {
        const float f = kv8_pair<HALF>(big).x * 0x1p100f;  // a 16-bit number below 2^28 keeps clear of overflow ...
        const float f2 = kv8_pair<HALF>(big).x * 0x1p-100f;
        e = isinf(f) ? static_cast<int>(__float_as_uint(f2) >> 23) - 127 + 100 : static_cast<int>(__float_as_uint(f) >> 23) - 127 - 100;
        e = 14 - e;  // multiply by 2^e, in [-113, 147]
      }
      const float s1 = __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
      const float s2 = __uint_as_float(static_cast<uint32_t>(127 + e - e / 2) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 f = kv8_pair<HALF>(w[j][i]);
          qf[j][i] = ka_pack_f16(f.x * s1 * s2, f.y * s1 * s2);
        }
      // rows 2 tq and 2 tq + 1 live in lanes 8 tq and 8 tq + 4
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int er = -__shfl_sync(kKaFull, e, 8 * tq + 4 * i);
        qc[i] = a.c_log2 * __uint_as_float(static_cast<uint32_t>(127 + er / 2) << 23) *
                __uint_as_float(static_cast<uint32_t>(127 + er - er / 2) << 23);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
      m[0] = m[1] = mv[0] = mv[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }

    // ---- logits of this warp's 16 tokens: s[0], s[1] token g, rows 2tq, 2tq+1; s[2], s[3] token g + 8
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    float lv = 0.f;
    const uint32_t base = smem_addr(sm.stage[stage]);
    if (kind == kUnitPage) {
      const float2 sc = sm.scale[stage];
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t r[4];
        ka_ldmatrix(r, base + k_off + (((j + half) ^ (k_row & 7u)) << 4));
        const uint32_t a0[4] = {fp8x2_to_f16x2<FMT>(r[0] & 0xFFFFu), fp8x2_to_f16x2<FMT>(r[1] & 0xFFFFu),
                                fp8x2_to_f16x2<FMT>(r[0] >> 16), fp8x2_to_f16x2<FMT>(r[1] >> 16)};
        const uint32_t a1[4] = {fp8x2_to_f16x2<FMT>(r[2] & 0xFFFFu), fp8x2_to_f16x2<FMT>(r[3] & 0xFFFFu),
                                fp8x2_to_f16x2<FMT>(r[2] >> 16), fp8x2_to_f16x2<FMT>(r[3] >> 16)};
        ka_mma_f16(s, a0, qf[j][0], qf[j][1]);
        ka_mma_f16(t, a1, qf[j + 1][0], qf[j + 1][1]);
      }
      lv = log2f(sc.y);
      const float c0 = qc[0] * sc.x, c1 = qc[1] * sc.x;
      s[0] = (s[0] + t[0]) * c0, s[1] = (s[1] + t[1]) * c1, s[2] = (s[2] + t[2]) * c0, s[3] = (s[3] + t[3]) * c1;
    } else if (kind == kUnitOpen) {
      const int n_tok = meta.n_tok;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // token g (and g + 8), channels 16 j + 4 tq .. + 3: eight bytes of one 16-byte chunk
        const uint32_t chunk = static_cast<uint32_t>(2 * (j & 3) + (tq >> 1));
        const uint32_t row = static_cast<uint32_t>(16 * warp + g);  // (row + 8) & 7 == row & 7
        const uint32_t at = (j >> 2) * kKv8Tile + row * 128u + ((chunk ^ (row & 7u)) << 4) + 8u * (tq & 1);
        const uint2 x0 = *reinterpret_cast<const uint2*>(sm.stage[stage] + at);
        const uint2 x1 = *reinterpret_cast<const uint2*>(sm.stage[stage] + at + 8 * 128);
        const uint2 qw = *reinterpret_cast<const uint2*>(sm.qraw[g] + 2 * (16 * j + 4 * tq));
        const uint32_t aw[4] = {x0.x, x1.x, x0.y, x1.y};
        if (HALF)
          ka_mma_f16(s, aw, qw.x, qw.y);
        else
          mma_bf16(s, aw[0], aw[1], aw[2], aw[3], qw.x, qw.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = 16 * warp + g + 8 * (i >> 1) < n_tok ? s[i] * a.c_log2 : -INFINITY;
    }

    // ---- softmax state
    uint32_t pb[4];  // P^T operand (tokens 0-7, 8-15): f16, or bf16 high parts and then low parts
    if (kind != kUnitNone) {
      float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(kKaFull, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(kKaFull, x1, d));
      }
      const float n0 = fmaxf(m[0], x0), n1 = fmaxf(m[1], x1);
      const float w0 = fmaxf(mv[0], x0 + lv - 15.f), w1 = fmaxf(mv[1], x1 + lv - 15.f);
      if (__any_sync(kKaFull, n0 > m[0] || n1 > m[1] || w0 > mv[0] || w1 > mv[1])) {
        l[0] *= ka_exp2(m[0] - ka_finite(n0));
        l[1] *= ka_exp2(m[1] - ka_finite(n1));
        const float f0 = ka_exp2(mv[0] - ka_finite(w0)), f1 = ka_exp2(mv[1] - ka_finite(w1));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i][0] *= f0;
          acc[i][1] *= f1;
          acc[i][2] *= f0;
          acc[i][3] *= f1;
        }
        m[0] = n0, m[1] = n1, mv[0] = w0, mv[1] = w1;
      }
      const float m0 = ka_finite(m[0]), m1 = ka_finite(m[1]), v0 = ka_finite(mv[0]) - lv, v1 = ka_finite(mv[1]) - lv;
      l[0] += ka_exp2(s[0] - m0) + ka_exp2(s[2] - m0);
      l[1] += ka_exp2(s[1] - m1) + ka_exp2(s[3] - m1);
      const float p[4] = {ka_exp2(s[0] - v0), ka_exp2(s[1] - v1), ka_exp2(s[2] - v0), ka_exp2(s[3] - v1)};
      if (HALF || kind == kUnitPage) {
        pb[0] = ka_transpose(ka_pack_f16(p[0], p[1]));
        pb[1] = ka_transpose(ka_pack_f16(p[2], p[3]));
      } else {
        const uint32_t h0 = ka_pack_bf16(p[0], p[1]), h1 = ka_pack_bf16(p[2], p[3]);
        const float2 b0 = kv8_pair<false>(h0), b1 = kv8_pair<false>(h1);
        pb[0] = ka_transpose(h0);
        pb[1] = ka_transpose(h1);
        pb[2] = ka_transpose(ka_pack_bf16(p[0] - b0.x, p[1] - b0.y));
        pb[3] = ka_transpose(ka_pack_bf16(p[2] - b1.x, p[3] - b1.y));
      }
    }

    // ---- O^T += V^T P^T
    if (kind == kUnitPage) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        // matrices (tokens 0-7, 8-15) of channels 16 i .. and of 16 (i + 1) ..; a lane gets channels 2g, 2g+1 of
        // tokens 2tq (low half) and 2tq+1
        uint32_t r[4];
        ka_ldmatrix_t(r, base + v_off + (((i + half) ^ (k_row & 7u)) << 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = __byte_perm(r[k], 0u, 0x3120);
        const uint32_t a0[4] = {fp8x2_to_f16x2<FMT>(r[0] & 0xFFFFu), fp8x2_to_f16x2<FMT>(r[0] >> 16),
                                fp8x2_to_f16x2<FMT>(r[1] & 0xFFFFu), fp8x2_to_f16x2<FMT>(r[1] >> 16)};
        const uint32_t a1[4] = {fp8x2_to_f16x2<FMT>(r[2] & 0xFFFFu), fp8x2_to_f16x2<FMT>(r[2] >> 16),
                                fp8x2_to_f16x2<FMT>(r[3] & 0xFFFFu), fp8x2_to_f16x2<FMT>(r[3] >> 16)};
        ka_mma_f16(acc[i], a0, pb[0], pb[1]);
        ka_mma_f16(acc[i + 1], a1, pb[0], pb[1]);
      }
    } else if (kind == kUnitOpen) {
      // the next stage holds V
      const int n_tok = meta.n_tok;
      __syncwarp();
      if (lane == 0) ka_arrive(&sm.empty[stage]);
      if (++stage == kKaStages) {
        stage = 0;
        phase ^= 1u;
      }
      if (!ka_wait(&sm.full[stage], phase, a.status)) return;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t aw[4];
#pragma unroll
        for (int t8 = 0; t8 < 2; ++t8) {
          uint32_t x[2];
#pragma unroll
          for (int o = 0; o < 2; ++o) {  // token 2tq + o (+ 8): channels 16 i + 2g, + 1
            const uint32_t row = static_cast<uint32_t>(16 * warp + 8 * t8 + 2 * tq + o);
            const uint32_t chunk = static_cast<uint32_t>(2 * (i & 3) + (g >> 2));
            const uint32_t at = (i >> 2) * kKv8Tile + row * 128u + ((chunk ^ (row & 7u)) << 4) + 4u * (g & 3);
            x[o] = static_cast<int>(row) < n_tok ? *reinterpret_cast<const uint32_t*>(sm.stage[stage] + at) : 0u;
          }
          aw[2 * t8] = __byte_perm(x[0], x[1], 0x5410);
          aw[2 * t8 + 1] = __byte_perm(x[0], x[1], 0x7632);
        }
        if (HALF) {
          ka_mma_f16(acc[i], aw, pb[0], pb[1]);
        } else {
          mma_bf16(acc[i], aw[0], aw[1], aw[2], aw[3], pb[0], pb[1]);
          mma_bf16(acc[i], aw[0], aw[1], aw[2], aw[3], pb[2], pb[3]);
        }
      }
    }

    // ---- the end of the pair in this CTA
    if (last) {
      const int b = sm.meta[stage].b, h = sm.meta[stage].h, cta0 = sm.meta[stage].cta0, n_cta = sm.meta[stage].n_cta;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[0] += __shfl_xor_sync(kKaFull, l[0], d);
        l[1] += __shfl_xor_sync(kKaFull, l[1], d);
      }
      if (g == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sm.m[warp][2 * tq + i] = m[i];
          sm.l[warp][2 * tq + i] = l[i];
          sm.mv[warp][2 * tq + i] = mv[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        *reinterpret_cast<float2*>(&sm.state[warp][2 * tq][16 * i + 2 * g]) = make_float2(acc[i][0], acc[i][2]);
        *reinterpret_cast<float2*>(&sm.state[warp][2 * tq + 1][16 * i + 2 * g]) = make_float2(acc[i][1], acc[i][3]);
      }
      if (!ka_meet(sm, meet, a.status)) return;
      const bool whole = n_cta == 1;
      float* part = a.part + static_cast<int64_t>(2 * blockIdx.x + (static_cast<int>(blockIdx.x) == cta0 ? 1 : 0)) * kKaPart;
#pragma unroll
      for (int k = 0; k < kKaRows * kD / 4 / (32 * kKaWarps); ++k) {
        const int at = tid + 32 * kKaWarps * k, row = at / (kD / 4), ch = 4 * (at % (kD / 4));
        float mx = -INFINITY, vx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kKaWarps; ++w) {
          mx = fmaxf(mx, sm.m[w][row]);
          vx = fmaxf(vx, sm.mv[w][row]);
        }
        float den = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kKaWarps; ++w) {
          den += ka_exp2(sm.m[w][row] - ka_finite(mx)) * sm.l[w][row];
          const float f = ka_exp2(sm.mv[w][row] - ka_finite(vx));
          const float4 x = *reinterpret_cast<const float4*>(&sm.state[w][row][ch]);
          o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
        }
        if (whole) {
          if (row < a.r) ka_store<HALF>(a, b, h, row, ch, ka_result(o, mx, den, vx));
        } else {
          *reinterpret_cast<float4*>(part + 3 * kKaRows + row * kD + ch) = o;
          if (ch == 0) {
            part[row] = mx;
            part[kKaRows + row] = den;
            part[2 * kKaRows + row] = vx;
          }
        }
      }
      if (!whole) {
        __threadfence();
        if (!ka_meet(sm, meet, a.status)) return;
        if (tid == 0) sm.last = kv8_atomic_add_acq_rel(a.counters + cta0, 1u) == static_cast<unsigned int>(n_cta - 1);
        if (!ka_meet(sm, meet, a.status)) return;
        if (sm.last) {
          // ---- the last CTA of the pair joins the partials, in order
          auto slot = [&](int i) { return a.part + static_cast<int64_t>(2 * (cta0 + i) + (i == 0 ? 1 : 0)) * kKaPart; };
#pragma unroll 1
          for (int k = 0; k < kKaRows * kD / 4 / (32 * kKaWarps); ++k) {
            const int at = tid + 32 * kKaWarps * k, row = at / (kD / 4), ch = 4 * (at % (kD / 4));
            float mx = -INFINITY, vx = -INFINITY, den = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < n_cta; ++i) {
              mx = fmaxf(mx, __ldcg(slot(i) + row));
              vx = fmaxf(vx, __ldcg(slot(i) + 2 * kKaRows + row));
            }
#pragma unroll 8
            for (int i = 0; i < n_cta; ++i) {
              const float* p = slot(i);
              const float4 x = __ldcg(reinterpret_cast<const float4*>(p + 3 * kKaRows + row * kD + ch));
              den += ka_exp2(__ldcg(p + row) - ka_finite(mx)) * __ldcg(p + kKaRows + row);
              const float f = ka_exp2(__ldcg(p + 2 * kKaRows + row) - ka_finite(vx));
              o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
            }
            if (row < a.r) ka_store<HALF>(a, b, h, row, ch, ka_result(o, mx, den, vx));
          }
          if (tid == 0) a.counters[cta0] = 0;
        }
      }
      // the next pair's state may be written once everybody has read this one's
      if (!ka_meet(sm, meet, a.status)) return;
    }
    __syncwarp();
    if (lane == 0) ka_arrive(&sm.empty[stage]);
    if (++stage == kKaStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

template <bool HALF, int FMT>
__global__ void __launch_bounds__(kKaThreads, kKaCtasPerSm)
    kv8_attention_kernel(const KaArgs a, const __grid_constant__ CUtensorMap pages, const __grid_constant__ CUtensorMap tail) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  KaSmem& sm = *reinterpret_cast<KaSmem*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKaStages; ++i) {
      mbar_init(&sm.full[i], 2);
      mbar_init(&sm.empty[i], kKaWarps);
    }
    mbar_init(&sm.sync, kKaWarps);
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(&pages) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tail) : "memory");
  }
  __syncthreads();
  dependent_wait();
  dependent_launch();
  if (threadIdx.x >= 32 * kKaWarps)
    ka_copy_warp(a, sm, &pages, &tail);
  else
    ka_compute<HALF, FMT>(a, sm);
}

// ------------------------------------------------------------------ host

static int ka_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
    cached[dev] = n;
  }
  return cached[dev];
}

static size_t ka_counter_bytes(int grid) { return (static_cast<size_t>(grid) * 4 + 15) & ~static_cast<size_t>(15); }

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled ka_encode() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A map of [rows][128 bytes-wide column blocks]: boxes of box_x elements by box_y rows, 128-byte swizzle.
static bool ka_map(CUtensorMap* m, CUtensorMapDataType type, int elem, void* base, int64_t rows, unsigned box_x, unsigned box_y) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(kD * elem)};
  const cuuint32_t box[2] = {box_x, box_y}, one[2] = {1, 1};
  return ka_encode()(m, type, 2, base, dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool HALF, int FMT>
static int ka_launch(const KaArgs& a, const CUtensorMap& pages, const CUtensorMap& tail, int grid, void* stream) {
  constexpr size_t smem = sizeof(KaSmem) + 1024;  // room to align the stages
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GAAC_ECUDA;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kv8_attention_kernel<HALF, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return GAAC_ECUDA;
    done[dev] = true;
  }
  return kv8_launch(kv8_attention_kernel<HALF, FMT>, dim3(grid), kKaThreads, smem, stream, a, pages, tail);
}

}  // namespace gaac

using namespace gaac;

extern "C" size_t gaac_kv8_attention_workspace(void) {
  const int grid = kKaCtasPerSm * ka_sms();
  return ka_counter_bytes(grid) + static_cast<size_t>(2 * grid) * kKaPart * sizeof(float);
}

extern "C" int gaac_kv8_decode_attention(const gaac_kv8* cache, const void* q, int n_q_heads, int64_t q_seq_stride,
                                         float scale, void* out, int out_dtype, void* workspace,
                                         size_t workspace_bytes, int32_t* d_status, void* stream) {
  if (!kv8_ok(cache) || q == nullptr || out == nullptr || workspace == nullptr || !std::isfinite(scale) ||
      (out_dtype != cache->dtype && out_dtype != GAAC_F32))
    return GAAC_EINVAL;
  if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads != 0 || n_q_heads / cache->n_kv_heads > GAAC_MAX_GQA ||
      q_seq_stride < static_cast<int64_t>(n_q_heads) * kD || (q_seq_stride & 7) || q_seq_stride > (int64_t{1} << 40) ||
      (reinterpret_cast<uintptr_t>(q) & 15u) || (reinterpret_cast<uintptr_t>(out) & 15u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < 16)
    return GAAC_EINVAL;
  const int sms = ka_sms();
  if (sms <= 0 || ka_encode() == nullptr) return GAAC_ECUDA;
  if (workspace_bytes < gaac_kv8_attention_workspace()) return GAAC_EINVAL;
  const int grid = kKaCtasPerSm * sms;
  KaArgs a;
  a.c = kv8_dev(cache);
  a.q = static_cast<const uint16_t*>(q);
  a.q_seq = q_seq_stride;
  a.out = out;
  a.out_f32 = out_dtype == GAAC_F32;
  a.r = n_q_heads / cache->n_kv_heads;
  a.c_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.counters = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + ka_counter_bytes(grid));
  a.status = d_status;
  CUtensorMap pages, tail;
  const int64_t rows = int64_t{2} * kBlock * cache->n_kv_heads;
  if (!ka_map(&pages, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, cache->pages, cache->n_pages * rows, kD, 2 * kBlock) ||
      !ka_map(&tail, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, cache->tail, cache->batch * rows, kD / 2, kBlock))
    return GAAC_ECUDA;
  if (cache->dtype == GAAC_BF16)
    return cache->fmt == GAAC_FP8_E4M3 ? ka_launch<false, GAAC_FP8_E4M3>(a, pages, tail, grid, stream)
                                       : ka_launch<false, GAAC_FP8_E5M2>(a, pages, tail, grid, stream);
  return cache->fmt == GAAC_FP8_E4M3 ? ka_launch<true, GAAC_FP8_E4M3>(a, pages, tail, grid, stream)
                                     : ka_launch<true, GAAC_FP8_E5M2>(a, pages, tail, grid, stream);
}
