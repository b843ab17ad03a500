// Decode attention over the 8-bit paged cache.
//
//   s_t = scale * sK * (q . k8_t),   out = sum_t softmax(s)_t * sV * v8_t
// with sK, sV the scales of t's block (1 for the open block, which is in the model's type).
//
// Memory bound: 256 bytes per token and kv-head are read once, and 4 * (query heads) * 128 operations per token
// hide under them.  One CTA per SM: five groups of two compute warps, and two copy warps (one alone takes
// some 950 cycles for each 16 KB, which bounds the kernel at 4.9 TB/s; with two the memory does):
//  * Work is cut evenly, whatever the lengths: the blocks of all (sequence, kv-head) pairs in one row of units (a page
//    is one unit, half an open block one, an empty sequence one), every CTA a piece of it of the same size.  Pieces
//    begin with a pair where there are CTAs for that.  A pair that spans CTAs is joined by the last of them to
//    finish; a CTA has at most two such pairs, its first and its last.
//  * The copy warps walk the units: one tensor copy (TMA, 128-byte swizzle) brings K and V of a page and head, which
//    lie together (16 KB), into a ring of ten stages; the scales ride along as an 8-byte asynchronous copy, the
//    pair's queries as a bulk copy with its first unit.  Everything a unit's consumers need is in its stage.
//  * Units go round the groups.  Short pairs go to one group each, side by side, which saves the CTA-wide meetings
//    (64 sequences of 10-200 tokens, 8 kv-heads: 18.0 us, 25 without).
//  * A group's two warps take 32 tokens of a page each and keep their own softmax state until the pair ends.  S = K q^T
//    with K as the 16-row operand (mma.sync m16n8k16, 8 columns = query heads of the kv-head): the decode step has at
//    most 8 rows, so the wide operand is the cache and no tensor-core work goes to padding, as it would in
//    tcgen05's 128-row tile, whose operands would also have to be widened into shared memory first.  O^T = V^T P^T
//    takes the transposed 8-bit V straight from ldmatrix.trans (pairs of channels).
//  * FP8 becomes f16 in registers (exact).  The query is scaled by a power of two per row into f16's range (exact
//    but for parts below 2^-28 of the row's largest), the scale is put back with sK.
//  * Two running maxima per row: m of the logits, for the softmax's sum l; and M of logit + log2 sV, for the
//    weights 2^(s + log2 sV - M + 15) that go to the tensor cores as f16: whatever the blocks' scales, the largest
//    weight is 2^15 and those down to 2^-29 of it keep f16's 11 bits.  What the rounding leaves (2^-11 of the weight)
//    follows as a second operand, for every result type: 2^-11 is an eighth of bf16's own half step, and leaving it to
//    a bf16 result would save 0.1 us of 8 (1 x 777), 0.3 of 25 (1 x 65,536), 1.4 of 176 (the 1.2 GB below) and at most
//    3% where hundreds of short sequences leave the groups no pause.  m, l, M and O are fp32.
//  * The open block is multiplied in its own type, the weights in two parts as well.
// Measured: 32 sequences of 4,096-32,768 tokens, 8 kv-heads, 1.2 GB: 176 us, 6.9 TB/s; one of 65,536 tokens: 25.0 us,
// of which 3 us go by before the first data and 4 us from the last to the joined result; one of 777 tokens: 8.0 us.
#include <algorithm>

#include "kv8.cuh"
#include "tma.cuh"

namespace gaac {

constexpr int kKaGroups = 5;                 // pairs of compute warps, units dealt out in turn
constexpr int kKaWarps = 2 * kKaGroups;      // a warp takes 32 tokens of a page, 16 of half an open block
constexpr int kKaCompute = 32 * kKaWarps;
constexpr int kKaCopyWarps = 2;
constexpr int kKaThreads = kKaCompute + 32 * kKaCopyWarps;
constexpr int kKaStages = 10;                // unit i uses stage i % stages and belongs to group i % groups
constexpr int kKaHalf = kBlock / 2;          // tokens of an open block's unit
constexpr int kKaRows = 8;                   // query heads per kv-head in the MMA columns
// Fewer units than this are not worth a CTA: 1 x 777 tokens 8.3 us (five: 8.9), 4 x 500 8.8 us (five: 9.2; two:
// 13.7, where the pieces no longer fit pair by pair).
constexpr int kKaMinUnits = 4;
// Most units of a pair that one group may take alone (at most 32).  256 x 1,000 tokens, 17 units a pair: 95 us; left to
// all groups, with sixteen here, 7% more; 32 makes no difference where it was measured.
constexpr unsigned kKaSolo = 20;
constexpr int kKaStride = kD + 4;            // floats per row of a warp's state in shared memory (bank spread)
constexpr int kKaPart = 3 * kKaRows + kKaRows * kD;  // floats of a partial: m, l, M, O
// Partials in flight when they are joined: 1 x 65,536 tokens then 25.2 us (with eight 26.6, with twelve 26.0).
constexpr int kKaJoin = 10;
constexpr uint32_t kKaFull = 0xFFFFFFFFu;
static_assert(kKaStages % kKaGroups == 0, "a stage belongs to one group, which waits for all of its phases in turn");

enum { kUnitPage, kUnitOpen, kUnitNone, kUnitEnd };
enum { kLastAll = 1, kLastSolo = 2 };        // the pair ends for all groups of the CTA; for its one group

struct KaSmem {
  alignas(1024) uint8_t stage[kKaStages][kKv8Pair];
  alignas(128) uint16_t q[kKaStages][kKaRows * kD];
  alignas(16) float state[kKaWarps][kKaRows][kKaStride];
  alignas(16) int4 meta[kKaStages][2];  // {kind, first of the pair in its group (2: with queries), last, tokens}, {b, h, first CTA, CTAs}
  alignas(16) float2 scale[kKaStages];
  float m[kKaWarps][kKaRows], l[kKaWarps][kKaRows], mv[kKaWarps][kKaRows];
  alignas(16) float solo[2][kKaWarps][3][kKaRows];  // m, l, M of pairs that groups end alone
  // pairs side by side, for each copy warp: {full blocks, open tokens, b, h}, units, pages
  alignas(16) int4 side[kKaCopyWarps][kKaGroups];
  int side_units[kKaCopyWarps][kKaGroups];
  int32_t side_page[kKaCopyWarps][kKaGroups][kKaSolo];
  uint64_t full[kKaStages], empty[kKaStages], sync, pair_sync[kKaGroups];
  int last;
  // Units of each 32 sequences, while the work is cut and there are no states yet.
  static constexpr int kPlaces = 65536 / 32;
  __device__ unsigned* places() { return reinterpret_cast<unsigned*>(state); }
};
static_assert(sizeof(KaSmem::state) >= KaSmem::kPlaces * sizeof(unsigned), "places in the states' room");

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
__device__ __forceinline__ float ka_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four FP8 numbers as two f16x2: (0, 1), (2, 3), or with SPLIT (0, 2), (1, 3).
template <int FMT, bool SPLIT>
__device__ __forceinline__ void ka_widen(uint32_t w, uint32_t& x, uint32_t& y) {
  if (FMT == GAAC_FP8_E5M2) {  // an e5m2 byte is the high byte of the f16
    x = __byte_perm(w, 0u, SPLIT ? 0x2404 : 0x1404);
    y = __byte_perm(w, 0u, SPLIT ? 0x3414 : 0x3424);
  } else {
    if (SPLIT) w = __byte_perm(w, 0u, 0x3120);
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}"
        : "=r"(x), "=r"(y) : "r"(w));
  }
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
// Two numbers of f16 or bf16, infinities and NaN made finite: magnitudes are at most 65504 or 2^113, which a weight's
// second part (2^6 at most) does not take past fp32.
template <bool F16>
__device__ __forceinline__ uint32_t ka_finite_pair(uint32_t x) {
  uint32_t r;
  if (F16)
    asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7BFF7BFFu));
  else
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x78007800u));
  return r;
}
__device__ __forceinline__ void ka_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ------------------------------------------------------------------ units

struct KaSeq {  // a sequence's units per kv-head
  int full, open;
  unsigned units;
};
__device__ __forceinline__ KaSeq ka_seq(const Kv8Dev& c, int len) {
  if (len < 0 || len > static_cast<int64_t>(c.max_blocks) * kBlock) len = 0;
  KaSeq s;
  s.full = len / kBlock;
  s.open = len % kBlock;
  s.units = static_cast<unsigned>(max(1, s.full + (s.open + kKaHalf - 1) / kKaHalf));
  return s;
}

// The cache is read once a step: its lines leave L2 first (1 x 65536 tokens: 26.8 us, 28.3 without the hint).
__device__ __forceinline__ uint64_t ka_evict_first() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void ka_tma(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], "
      "[%4], %5;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// A bounded wait that the whole warp takes alike.
__device__ __forceinline__ bool ka_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(kKaFull, mbar_wait(bar, parity, status));
}

// Where a CTA's work lies.
struct KaCut {
  unsigned piece;            // units of a CTA at most
  bool aligned;
  int b, h, b32, len32;      // its first pair (b = batch: none); the lengths of sequences b32 .. b32 + 31, one a lane
  KaSeq s;                   // sequence b
  unsigned own, skipped;     // places of a pair of sequence b, and those of the first pair before this CTA's
  unsigned seg, u, u_end;    // in units: the pair's first, this CTA's first and its end
};

// Places of chunks of 32 sequences, piece units per place: put(j, sum) for chunks j0, j0 + step, ...  The lengths come
// from L2, so that a call ahead of the dependent-launch wait leaves nothing stale; eight loads are in flight.
template <class Put>
__device__ __forceinline__ void ka_sums(const Kv8Dev& c, int j0, int step, unsigned piece, int32_t* status, Put put) {
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 31, chunks = (c.batch + 31) / 32;
#pragma unroll 1
  for (; j0 < chunks; j0 += kAhead * step) {
    int len[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = 32 * (j0 + static_cast<int64_t>(k) * step) + lane;
      len[k] = i < c.batch ? __ldcg(c.lens + i) : 0;
      if (status != nullptr && (len[k] < 0 || len[k] > static_cast<int64_t>(c.max_blocks) * kBlock)) report(status, GAAC_EINVAL);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = j0 + k * step;
      if (j >= chunks) break;
      const unsigned u = 32 * j + lane < c.batch ? (ka_seq(c, len[k]).units + piece - 1) / piece : 0u;
      put(j, __reduce_add_sync(kKaFull, u));  // 32 sequences of up to 2^24 + 1 units: 30 bits
    }
  }
}

__device__ __forceinline__ unsigned ka_scan(unsigned v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned x = __shfl_up_sync(kKaFull, v, d);
    if (lane >= d) v += x;
  }
  return v;
}

// By a whole warp.  FEW: at most 32 sequences, one a lane, whose lengths are read once (as many sequences are, one of 777
// tokens takes 9.2 us, so 7.9).  Else places: the units of each 32 sequences, which all warps have added up (each copy
// warp for itself: 5,000 sequences of 100 tokens, 1 kv-head, take 160 us, so 105).
template <bool FEW>
__device__ __forceinline__ KaCut ka_cut(const Kv8Dev& c, const unsigned* places, int32_t* status) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x != 0) status = nullptr;  // one CTA reports lengths that are not valid
  // ---- the cut: pieces of at most `piece` units (all counts below 2^31: the host has checked)
  const int chunks = (c.batch + 31) / 32;
  unsigned sums = 0, total;  // sums, FEW: this lane's sequence's
  int len32 = 0;
  if (FEW) {
    if (lane < c.batch) {
      len32 = __ldcg(c.lens + lane);
      if (status != nullptr && (len32 < 0 || len32 > static_cast<int64_t>(c.max_blocks) * kBlock)) report(status, GAAC_EINVAL);
      sums = ka_seq(c, len32).units;
    }
    total = sums;
  } else {
    total = 0;
    for (int j = lane; j < chunks; j += 32) total += places[j];
  }
  total = __reduce_add_sync(kKaFull, total) * c.heads;
  const unsigned piece = max(static_cast<unsigned>(kKaMinUnits), (total + gridDim.x - 1) / gridDim.x);
  // Pieces begin with their pair where that needs no more CTAs: then none has parts of two pairs to bring to an
  // end.  Otherwise the row of all units is cut without regard to pairs.
  bool aligned = false;
  if (static_cast<unsigned>(c.batch) * c.heads <= min(gridDim.x, 1024u)) {
    unsigned pieces = (sums + piece - 1) / piece;  // else of a chunk: there are no more of them than lanes
    if (!FEW)
      ka_sums(c, 0, 1, piece, nullptr, [&](int j, unsigned sum) {
        if (lane == j) pieces = sum;
      });
    aligned = __reduce_add_sync(kKaFull, pieces) * c.heads <= gridDim.x;
    if (aligned) sums = pieces;
  }
  // In places (units, or pieces when aligned): where this CTA begins and ends.
  const unsigned begin = aligned ? blockIdx.x : blockIdx.x * piece;
  int b = c.batch, b32 = 0;
  unsigned base = 0;  // places before sequence b
  if (!FEW) {         // the 32 sequences that it begins in
    const unsigned per = aligned ? piece : 1u;
    for (int j0 = 0;; j0 += 32) {
      if (j0 >= chunks) {
        sums = 0;  // it begins behind all of them
        break;
      }
      const unsigned v = aligned ? sums : j0 + lane < chunks ? places[j0 + lane] : 0u;
      const unsigned incl = ka_scan(v, lane);
      const uint32_t past = __ballot_sync(kKaFull, base + incl * c.heads > begin);
      const int at = past ? __ffs(past) - 1 : 31;
      base += __shfl_sync(kKaFull, past ? incl - v : incl, at) * c.heads;
      if (past) {
        b32 = 32 * (j0 + at);
        len32 = b32 + lane < c.batch ? __ldcg(c.lens + b32 + lane) : 0;
        sums = b32 + lane < c.batch ? (ka_seq(c, len32).units + per - 1) / per : 0u;
        break;
      }
    }
  }
  const unsigned incl = ka_scan(sums, lane);
  const uint32_t past = __ballot_sync(kKaFull, base + incl * c.heads > begin);
  if (past) {
    const int at = __ffs(past) - 1;
    base += __shfl_sync(kKaFull, incl - sums, at) * c.heads;
    b = b32 + at;
  }
  KaSeq s = {};
  int h = 0;
  unsigned own = 1;      // places of a pair of sequence b
  unsigned skipped = 0;  // places of the first pair before this CTA's
  unsigned seg = 0, u = 0, u_end = 0;  // in units: the pair's first, this CTA's next and last
  if (b < c.batch) {
    s = ka_seq(c, __shfl_sync(kKaFull, len32, b - b32));
    own = aligned ? (s.units + piece - 1) / piece : s.units;
    h = static_cast<int>((begin - base) / own);
    skipped = begin - base - h * own;
    seg = aligned ? 0 : begin - skipped;
    u = aligned ? skipped * piece : begin;
    u_end = min(u + piece, aligned ? static_cast<unsigned>(s.units) : total);
  }
  return KaCut{piece, aligned, b, h, b32, len32, s, own, skipped, seg, u, u_end};
}

// Before the kernel ahead on the stream is done: the pages that this CTA will most likely read first are fetched into
// L2.  Lengths and table may still change, which wastes a prefetch; every address is checked.
__device__ __forceinline__ void ka_guess(const KaArgs& a) {
  const Kv8Dev& c = a.c;
  const int lane = threadIdx.x & 31;
  // More than 32 sequences: guessing as well takes 256 x 1,000 tokens from 96.6 to 95.2 us and, by the code that it
  // needs, 1 x 65,536 from 24.6 to 24.9; it is left to calls where the start is a larger part.
  if (c.batch > 32) return;
  const KaCut cut = ka_cut<true>(c, nullptr, nullptr);
  const int l = static_cast<int>(cut.u - cut.seg) + lane;
  if (cut.b < c.batch && lane < kKaStages && cut.u + lane < cut.u_end && l < cut.s.full) {
    const int32_t page = __ldcg(c.table + static_cast<int64_t>(cut.b) * c.max_blocks + l);
    if (page >= 0 && page < c.n_pages)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(c.pages + (static_cast<int64_t>(page) * c.heads + cut.h) * kKv8Pair),
                   "r"(kKv8Pair) : "memory");
  }
}

// A copy warp.  The CTA's units, of all its pairs, are numbered; unit j uses stage j % kKaStages, and copy warp w starts
// the copies of units w, w + kKaCopyWarps, ...: lane 0 does, the others help with what is warp-wide.
__device__ void ka_copy_warp(const KaArgs& a, KaSmem& sm, const CUtensorMap* pages, const CUtensorMap* tail, int copier) {
  static_assert(kKaStages % kKaCopyWarps == 0, "a stage belongs to one copy warp");
  constexpr int kOwn = kKaStages / kKaCopyWarps;
  const Kv8Dev& c = a.c;
  const int lane = threadIdx.x & 31;
  const KaCut cut = c.batch <= 32 ? ka_cut<true>(c, nullptr, a.status) : ka_cut<false>(c, sm.places(), nullptr);
  if (c.batch > 32) __syncthreads();  // the places are read
  KaSeq s = cut.s;
  int b = cut.b, h = cut.h, b32 = cut.b32, len32 = cut.len32;
  unsigned seg = cut.seg, u = cut.u, u_end = cut.u_end;
  const unsigned piece = cut.piece, own = cut.own, skipped = cut.skipped;
  const bool aligned = cut.aligned;
  const uint64_t policy = ka_evict_first();
  const uint32_t q_bytes = static_cast<uint32_t>(a.r) * kD * 2;
  bool ok = true;
  int count = 0;             // units of all copy warps, modulo kKaCopyWarps (all lanes)
  int st = copier, used = 0;  // lane 0: the next stage of this warp and how many it has used
  uint32_t parity = 1u;       // lane 0: of the phase that frees the stage
  auto acquire = [&]() {
    if (used >= kOwn) {
      ok = mbar_wait(&sm.empty[st], parity, a.status);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    return ok;
  };
  auto next_stage = [&]() {
    ++used;
    st += kKaCopyWarps;
    if (st >= kKaStages) {
      st -= kKaStages;
      parity ^= 1u;
    }
  };
  // Lane 0: one unit of pair (pb, ph) into the next stage.  unit: its place in the pair.
  auto issue = [&](const KaSeq& ps, int pb, int ph, int unit, int32_t page, bool empty, bool first, int last, int cta0, int n_cta) {
    if (!acquire()) return;
    uint64_t* full = &sm.full[st];
    int kind = kUnitNone, n_tok = kBlock;
    if (empty) {
    } else if (unit < ps.full) {
      kind = page >= 0 && page < c.n_pages ? kUnitPage : kUnitNone;
      if (kind == kUnitNone) report(a.status, GAAC_EFORMAT);
    } else if (ps.open) {
      kind = kUnitOpen;
      n_tok = min(kKaHalf, ps.open - kKaHalf * (unit - ps.full));
    }
    const bool with_q = first && !empty;
    sm.meta[st][0] = make_int4(kind, first ? 1 + with_q : 0, last, n_tok);
    if (last) sm.meta[st][1] = make_int4(pb, ph, cta0, n_cta);
    const int64_t tile = static_cast<int64_t>(page) * c.heads + ph;
    if (kind == kUnitPage) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(&sm.scale[st])), "l"(c.scales + 2 * tile) : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(full)) : "memory");
    } else {
      ka_arrive(full);
    }
    mbar_arrive_expect_tx(full, (kind == kUnitNone ? 0 : kKv8Pair) + (with_q ? q_bytes : 0));
    if (kind == kUnitPage) {
      ka_tma(sm.stage[st], pages, 0, static_cast<int>(tile * 2 * kBlock), full, policy);
    } else if (kind == kUnitOpen) {  // K channels 0-63, 64-127, V the same
      const int y = static_cast<int>((static_cast<int64_t>(pb) * c.heads + ph) * 2 * kBlock) + kKaHalf * (unit - ps.full);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ka_tma(sm.stage[st] + k * (kKv8Pair / 4), tail, (k & 1) * (kD / 2), y + (k >> 1) * kBlock, full, policy);
    }
    if (with_q) bulk_g2s(sm.q[st], a.q + pb * a.q_seq + static_cast<int64_t>(ph) * a.r * kD, q_bytes, full);
    next_stage();
  };
  // The first of the next units that is this warp's, when `count` have been before.
  auto first_own = [&]() { return (copier - count + kKaCopyWarps) % kKaCopyWarps; };
  auto next_pair = [&]() {  // (b, h), s, seg and u move on
    seg += s.units;
    u = seg;
    if (++h < c.heads) return;
    h = 0;
    if (++b >= c.batch) {
      u_end = u;
      return;
    }
    if (b - b32 >= 32) {
      b32 += 32;
      len32 = b32 + lane < c.batch ? c.lens[b32 + lane] : 0;
    }
    s = ka_seq(c, __shfl_sync(kKaFull, len32, b - b32));
  };
  // Lane 0: this warp's of the next n_all units, of the pairs side by side, or of pair (b, h) from unit l0 on with n
  // units of which the first n_pages are pages, row their table entries.
  auto start = [&](int n_all, bool sides, const int32_t* row, int l0, int n, int n_pages, int cta0, int n_cta) {
    if (lane == 0) {
      int i = first_own();
      const int plain_end = sides ? 0 : min(n_pages, n_all - kKaGroups);
      int32_t page_next = i < n_pages ? row[i] : 0;
#pragma unroll 1
      for (; i < n_all && ok; i += kKaCopyWarps) {
        int32_t page = page_next;  // one unit ahead
        page_next = i + kKaCopyWarps < n_pages ? row[i + kKaCopyWarps] : 0;
        if (i >= kKaGroups && i < plain_end && page >= 0 && page < c.n_pages) {  // most units: neither first nor last
          if (!acquire()) break;
          uint64_t* full = &sm.full[st];
          const int64_t tile = static_cast<int64_t>(page) * c.heads + h;
          sm.meta[st][0] = make_int4(kUnitPage, 0, 0, kBlock);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(&sm.scale[st])), "l"(c.scales + 2 * tile) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(full)) : "memory");
          mbar_arrive_expect_tx(full, kKv8Pair);
          ka_tma(sm.stage[st], pages, 0, static_cast<int>(tile * 2 * kBlock), full, policy);
          next_stage();
        } else {
          KaSeq ps = s;
          int pb = b, ph = h, unit = l0 + i, last = i >= n_all - kKaGroups ? kLastAll : 0;
          bool empty = i >= n, first = i < kKaGroups;
          if (sides) {
            const int k = i % kKaGroups;
            unit = i / kKaGroups;
            const int4 d = sm.side[copier][k];
            const int units = sm.side_units[copier][k];
            ps.full = d.x, ps.open = d.y, pb = d.z, ph = d.w;
            page = sm.side_page[copier][k][min(unit, static_cast<int>(kKaSolo) - 1)];
            empty = unit >= units;
            first = unit == 0;
            last = unit + 1 == units ? kLastSolo : 0;
          }
          issue(ps, pb, ph, unit, page, empty, first, last, cta0, n_cta);
        }
      }
    }
    count = (count + n_all) % kKaCopyWarps;
    ok = __shfl_sync(kKaFull, ok, 0);
  };
  while (u < u_end && ok) {
    if (!aligned && u == seg && s.units <= kKaSolo && u + s.units <= u_end &&
        (s.units <= 4 || (h + 3 <= c.heads && u_end - u >= 3 * s.units))) {
      // ---- short pairs: the next ones of about the same length, up to one for each group, side by side (three at
      // least, or few units)
      unsigned most = 0, least = kKaSolo;
      __syncwarp();  // lane 0 is done with the last ones
#pragma unroll 1
      for (int k = 0; k < kKaGroups; ++k) {
        const bool take = u < u_end && u + s.units <= u_end && s.units <= kKaSolo &&
                          4 * max(most, s.units) <= 5 * min(least, s.units) + 4;
        if (lane == 0) {
          sm.side[copier][k] = take ? make_int4(s.full, s.open, b, h) : make_int4(0, 0, 0, 0);
          sm.side_units[copier][k] = take ? static_cast<int>(s.units) : 0;
        }
        if (take) {
          if (lane < s.full) sm.side_page[copier][k][lane] = c.table[static_cast<int64_t>(b) * c.max_blocks + lane];
          most = max(most, s.units);
          least = min(least, s.units);
          next_pair();
        }
      }
      __syncwarp();
      start(kKaGroups * static_cast<int>(most), true, nullptr, 0, 0, 0, 0, 1);
      continue;
    }
    const int l0 = static_cast<int>(u - seg);
    const int n = static_cast<int>(min(u_end, seg + s.units) - u);
    const int cta0 = static_cast<int>(aligned ? blockIdx.x - skipped : seg / piece);
    const int n_cta = static_cast<int>(aligned ? own : (seg + s.units - 1) / piece - cta0 + 1);
    const int32_t* row = c.table + static_cast<int64_t>(b) * c.max_blocks + l0;
    // every group takes part in every pair, with an empty unit if need be
    start(max(n, kKaGroups), false, row, l0, n, max(0, min(n, s.full - l0)), cta0, n_cta);
    next_pair();
  }
  // No copy may be in flight when the CTA ends, not even where a consumer's wait ran out: the last use of every stage
  // is waited for (bounded) before the end is passed on.
  if (lane == 0) {
    for (int i = 1; i <= min(used, kOwn); ++i) {
      const int j = used - i;
      mbar_wait(&sm.full[copier + kKaCopyWarps * (j % kOwn)], (j / kOwn) & 1, a.status);
    }
    for (int i = first_own(); i < kKaGroups && ok; i += kKaCopyWarps) {
      if (!acquire()) break;
      sm.meta[st][0] = make_int4(kUnitEnd, 0, 0, 0);
      ka_arrive(&sm.full[st]);
      ka_arrive(&sm.full[st]);
      next_stage();
    }
  }
}

// ------------------------------------------------------------------ compute warps

struct KaSync {
  uint32_t phase = 0;
};
// The compute warps (or the two of a group) meet.  false: gave up.
__device__ __forceinline__ bool ka_meet_at(uint64_t* bar, KaSync& s, int32_t* status) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ka_arrive(bar);
  const bool ok = ka_wait(bar, s.phase, status);
  s.phase ^= 1u;
  return ok;
}
__device__ __forceinline__ bool ka_meet(KaSmem& sm, KaSync& s, int32_t* status) { return ka_meet_at(&sm.sync, s, status); }

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

template <bool HALF>
__device__ __forceinline__ void ka_store2(const KaArgs& a, int b, int h, int row, int ch, float y0, float y1) {
  const int64_t at = (static_cast<int64_t>(b) * a.c.heads + h) * a.r * kD + row * kD + ch;
  if (a.out_f32)
    *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(y0, y1);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) = HALF ? ka_pack_f16(y0, y1) : ka_pack_bf16(y0, y1);
}

// O, in units of 2^M, over the sum l, in units of 2^m: halves of the exponent on either side of the division, so
// that neither leaves fp32 before the result does.
__device__ __forceinline__ float4 ka_result(float4 o, float m, float l, float mv) {
  if (l == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
  const float e = ka_exp2(0.5f * (ka_finite(mv) - ka_finite(m)));
  return make_float4(o.x * e / l * e, o.y * e / l * e, o.z * e / l * e, o.w * e / l * e);
}

// Folds a partial (m, l, mv, o) into the running one.
__device__ __forceinline__ void ka_fold(float& m, float& l, float& mv, float4& o, float m1, float l1, float mv1, float4 o1) {
  const float mn = fmaxf(m, m1), vn = fmaxf(mv, mv1), z = ka_finite(mn), zv = ka_finite(vn);
  l = l * ka_exp2(m - z) + l1 * ka_exp2(m1 - z);
  const float f0 = ka_exp2(mv - zv), f1 = ka_exp2(mv1 - zv);
  o.x = o.x * f0 + o1.x * f1, o.y = o.y * f0 + o1.y * f1, o.z = o.z * f0 + o1.z * f1, o.w = o.w * f0 + o1.w * f1;
  m = mn;
  mv = vn;
}

// Folds n partials, the first at `head`, the others `step` floats apart from `rest` on.  Thread (share, row, four
// channels) takes partials share, share + shares, ... in order, kKaJoin of them in flight; the shares (as many as the
// threads allow for r rows) meet in shared memory.  Threads of share 0 get the result of their row and channels.
template <bool HALF>
__device__ __forceinline__ bool ka_fold_all(const KaArgs& a, KaSmem& sm, const float* head, const float* rest, int64_t step,
                                            int n, KaSync& meet, float& m, float& l, float& mv, float4& o) {
  const int per = a.r * (kD / 4), shares = kKaCompute / per;
  const int share = threadIdx.x / per, at = threadIdx.x % per, row = at / (kD / 4), ch = 4 * (at % (kD / 4));
  m = mv = -INFINITY;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (share < shares) {
#pragma unroll 1
    for (int i0 = share; i0 < n; i0 += kKaJoin * shares) {
      float m1[kKaJoin], l1[kKaJoin], mv1[kKaJoin];
      float4 o1[kKaJoin];
#pragma unroll
      for (int k = 0; k < kKaJoin; ++k) {
        const int i = i0 + k * shares;
        m1[k] = mv1[k] = -INFINITY;
        l1[k] = 0.f;
        o1[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
          const float* p = (i == 0 ? head : rest + (i - 1) * step) + row;
          m1[k] = __ldcg(p);
          l1[k] = __ldcg(p + kKaRows);
          mv1[k] = __ldcg(p + 2 * kKaRows);
          o1[k] = __ldcg(reinterpret_cast<const float4*>(p + 3 * kKaRows + row * (kD - 1) + ch));
        }
      }
      float mn = m, vn = mv;
#pragma unroll
      for (int k = 0; k < kKaJoin; ++k) {
        mn = fmaxf(mn, m1[k]);
        vn = fmaxf(vn, mv1[k]);
      }
      const float z = ka_finite(mn), zv = ka_finite(vn), f = ka_exp2(mv - zv);
      l *= ka_exp2(m - z);
      o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
      for (int k = 0; k < kKaJoin; ++k) {
        l += l1[k] * ka_exp2(m1[k] - z);
        const float g = ka_exp2(mv1[k] - zv);
        o.x += g * o1[k].x, o.y += g * o1[k].y, o.z += g * o1[k].z, o.w += g * o1[k].w;
      }
      m = mn;
      mv = vn;
    }
    if (share > 0) {
      *reinterpret_cast<float4*>(&sm.state[share][row][ch]) = o;
      if (ch == 0) {
        sm.m[share][row] = m;
        sm.l[share][row] = l;
        sm.mv[share][row] = mv;
      }
    }
  }
  if (shares > 1) {
    if (!ka_meet(sm, meet, a.status)) return false;
    if (share == 0) {
#pragma unroll 1
      for (int w = 1; w < shares; ++w)
        ka_fold(m, l, mv, o, sm.m[w][row], sm.l[w][row], sm.mv[w][row], *reinterpret_cast<const float4*>(&sm.state[w][row][ch]));
    }
  }
  return true;
}

// One more CTA has written its partial where `count` of them meet.  last: it was the last one.  Everybody's stores
// come before thread 0's release by the barrier, and what the others released comes before what follows.
__device__ __forceinline__ bool ka_arrived(KaSmem& sm, int32_t* counter, int count, KaSync& meet, int32_t* status, bool& last) {
  if (!ka_meet(sm, meet, status)) return false;
  if (threadIdx.x == 0) {
    sm.last = kv8_atomic_add_acq_rel(counter, 1u) == static_cast<unsigned int>(count - 1);
    if (sm.last) *counter = 0;
  }
  if (!ka_meet(sm, meet, status)) return false;
  last = sm.last;
  return true;
}

// The partial of a (CTA, pair): slot 1 where the pair begins in the CTA, 0 where it does not.
__device__ __forceinline__ int64_t ka_slot(int cta, int cta0) { return 2 * static_cast<int64_t>(cta) + (cta == cta0 ? 1 : 0); }

__device__ __forceinline__ void ka_put(float* slot, int row, int ch, float m, float l, float mv, float4 o) {
  *reinterpret_cast<float4*>(slot + 3 * kKaRows + row * kD + ch) = o;
  if (ch == 0) {
    slot[row] = m;
    slot[kKaRows + row] = l;
    slot[2 * kKaRows + row] = mv;
  }
}

// This CTA's partial of a pair that n CTAs share is in its slot: the last to come joins them.  Up to kKaJoin partials
// for each share of the threads are one round of loads; more than that are joined in teams of kKaJoin first, so that
// two rounds and two counters take the place of up to a dozen rounds.
template <bool HALF>
__device__ __forceinline__ bool ka_join(const KaArgs& a, KaSmem& sm, int b, int h, int cta0, int n, KaSync& meet) {
  const int per = a.r * (kD / 4), at = threadIdx.x % per, row = at / (kD / 4), ch = 4 * (at % (kD / 4));
  const bool writer = threadIdx.x < per;
  const int64_t grid = gridDim.x;
  const float* rest = a.part + 2 * static_cast<int64_t>(cta0 + 1) * kKaPart;
  float m, l, mv;
  float4 o;
  bool last;
  if (n <= kKaJoin * (kKaCompute / per)) {
    if (!ka_arrived(sm, a.counters + cta0, n, meet, a.status, last)) return false;
    if (last) {
      if (!ka_fold_all<HALF>(a, sm, a.part + ka_slot(cta0, cta0) * kKaPart, rest, 2 * kKaPart, n, meet, m, l, mv, o)) return false;
      if (writer) ka_store<HALF>(a, b, h, row, ch, ka_result(o, m, l, mv));
    }
    return true;
  }
  const int team = (static_cast<int>(blockIdx.x) - cta0) / kKaJoin, teams = (n + kKaJoin - 1) / kKaJoin;
  const int head = cta0 + team * kKaJoin, size = min(kKaJoin, n - team * kKaJoin);
  if (!ka_arrived(sm, a.counters + grid + ka_slot(head, cta0), size, meet, a.status, last)) return false;
  if (!last) return true;
  if (!ka_fold_all<HALF>(a, sm, a.part + ka_slot(head, cta0) * kKaPart, rest + 2 * static_cast<int64_t>(head - cta0) * kKaPart,
                         2 * kKaPart, size, meet, m, l, mv, o))
    return false;
  float* joined = a.part + 2 * grid * kKaPart;  // the teams' partials: slots like the CTAs', at a team's first CTA
  if (writer) ka_put(joined + ka_slot(head, cta0) * kKaPart, row, ch, m, l, mv, o);
  if (!ka_arrived(sm, a.counters + cta0, teams, meet, a.status, last)) return false;
  if (last) {
    if (!ka_fold_all<HALF>(a, sm, joined + ka_slot(cta0, cta0) * kKaPart, joined + 2 * static_cast<int64_t>(cta0 + kKaJoin) * kKaPart,
                           2 * kKaJoin * kKaPart, teams, meet, m, l, mv, o))
      return false;
    if (writer) ka_store<HALF>(a, b, h, row, ch, ka_result(o, m, l, mv));
  }
  return true;
}

// The P^T operands of 16 tokens from their weights in the logits' places: rounded to f16 or bf16, and what that
// leaves, rounded again (2^-22 of the weight is lost in f16, 2^-16 in bf16).
// An infinite V has to make its sum infinite, but 0 times infinity is NaN, as are two infinities of either sign.  So
// with INF the first part of a positive weight is not 0 (f16's smallest number at least; the second part takes back
// what that adds), and the second part is multiplied by V's numbers made finite (ka_finite_pair).  Over E5M2 pages
// that takes 1% (the 1.2 GB in FP16: 175.5 us without, 177.2 with; 256 sequences of 300-700 tokens 60.0 and 61.4); the
// open block's share does not show.
template <bool F16, bool INF>
__device__ __forceinline__ void ka_weights(const float w[4], uint32_t pb[4]) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = F16 && INF && w[i] > 0.f && w[i] < 0x1p-24f ? 0x1p-24f : w[i];
  const uint32_t h0 = F16 ? ka_pack_f16(f[0], f[1]) : ka_pack_bf16(f[0], f[1]);
  const uint32_t h1 = F16 ? ka_pack_f16(f[2], f[3]) : ka_pack_bf16(f[2], f[3]);
  pb[0] = ka_transpose(h0);
  pb[1] = ka_transpose(h1);
  const float2 b0 = kv8_pair<F16>(h0), b1 = kv8_pair<F16>(h1);
  const float r[4] = {w[0] - b0.x, w[1] - b0.y, w[2] - b1.x, w[3] - b1.y};
  pb[2] = ka_transpose(F16 ? ka_pack_f16(r[0], r[1]) : ka_pack_bf16(r[0], r[1]));
  pb[3] = ka_transpose(F16 ? ka_pack_f16(r[2], r[3]) : ka_pack_bf16(r[2], r[3]));
}

template <bool HALF, int FMT>
__device__ void ka_compute(const KaArgs& a, KaSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int warp = tid >> 5, part = warp & 1;  // part: which half of a unit's tokens
  KaSync meet, meet_pair;
  int turn = 0;
  bool gave = false;
  int stage = warp >> 1;
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
  // This lane's ldmatrix row of the first 16 tokens (matrices: tokens 0-7, 8-15 of chunk 0, then of chunk 1), its
  // 16-byte chunk swizzled by the row: chunk c of row t lies at c ^ (t & 7).
  const uint32_t lm_row = static_cast<uint32_t>(32 * part + 8 * ((lane >> 3) & 1) + (lane & 7));
  const uint32_t lm_off = lm_row * 128u + ((static_cast<uint32_t>(lane >> 4) ^ (lm_row & 7u)) << 4);

  while (true) {
    if (!ka_wait(&sm.full[stage], phase, a.status)) return;
    const int4 meta = sm.meta[stage][0];
    const int kind = meta.x, last = meta.z;
    if (kind == kUnitEnd) return;
    if (meta.y) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
      m[0] = m[1] = mv[0] = mv[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    if (meta.y == 2) {
      // ---- the pair's queries
      const uint16_t* qs = sm.q[stage];
      uint32_t w[8][2];
      uint32_t big = 0;  // largest finite magnitude of this lane's part of row g, as a 16-bit pattern
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint2 x = make_uint2(0u, 0u);
        if (g < a.r) x = *reinterpret_cast<const uint2*>(qs + g * kD + 16 * j + 4 * tq);
        w[j][0] = x.x, w[j][1] = x.y;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t mag = w[j][i] & 0x7FFF7FFFu;
          big = __vmaxu2(big, mag & ~__vcmpgeu2(mag, HALF ? 0x7C007C00u : 0x7F807F80u));
        }
      }
      big = max(big & 0xFFFFu, big >> 16);
      big = max(big, __shfl_xor_sync(kKaFull, big, 1));
      big = max(big, __shfl_xor_sync(kKaFull, big, 2));
      // The row's power of two takes its largest magnitude to [2^14, 2^15).  Its exponent is read after a scaling
      // that makes any 16-bit number normal in fp32; it is applied in two halves, both normal.
      int e = 0;
      if (big != 0u) {
        const float f = kv8_pair<HALF>(big).x;
        const bool low = f < 0x1p-60f;
        e = 14 - (static_cast<int>(__float_as_uint(low ? f * 0x1p80f : f) >> 23) - 127 - (low ? 80 : 0));
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
    }

    if (kind != kUnitNone) {
      // ---- logits: s[t][0], s[t][1] token 16 t + g, rows 2tq, 2tq+1; s[t][2], s[t][3] token 16 t + g + 8
      float s[2][4];
      float lv = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = kind == kUnitPage ? 0.f : -INFINITY;
      const uint32_t base = smem_addr(sm.stage[stage]);
      if (kind == kUnitPage) {
        const float2 sc = sm.scale[stage];
        float u[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < 8; j += 2)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t r[4], a0[4], a1[4];
            ka_ldmatrix(r, ((base + lm_off) ^ (j << 4)) + 16 * 128 * t);
            ka_widen<FMT, false>(r[0], a0[0], a0[2]);
            ka_widen<FMT, false>(r[1], a0[1], a0[3]);
            ka_widen<FMT, false>(r[2], a1[0], a1[2]);
            ka_widen<FMT, false>(r[3], a1[1], a1[3]);
            ka_mma_f16(s[t], a0, qf[j][0], qf[j][1]);
            ka_mma_f16(u[t], a1, qf[j + 1][0], qf[j + 1][1]);
          }
        lv = ka_log2(sc.y);
        const float c0 = qc[0] * sc.x, c1 = qc[1] * sc.x;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[t][0] = (s[t][0] + u[t][0]) * c0, s[t][1] = (s[t][1] + u[t][1]) * c1;
          s[t][2] = (s[t][2] + u[t][2]) * c0, s[t][3] = (s[t][3] + u[t][3]) * c1;
        }
      } else {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // token g (and g + 8), channels 16 j + 4 tq .. + 3: eight bytes of one 16-byte chunk
          const uint32_t chunk = static_cast<uint32_t>(2 * (j & 3) + (tq >> 1));
          const uint32_t row = static_cast<uint32_t>(16 * part + g);  // (row + 8) & 7 == row & 7
          const uint32_t at = (j >> 2) * (kKv8Pair / 4) + row * 128u + ((chunk ^ (row & 7u)) << 4) + 8u * (tq & 1);
          const uint2 x0 = *reinterpret_cast<const uint2*>(sm.stage[stage] + at);
          const uint2 x1 = *reinterpret_cast<const uint2*>(sm.stage[stage] + at + 8 * 128);
          const uint32_t aw[4] = {x0.x, x1.x, x0.y, x1.y};
          if (HALF) {
            ka_mma_f16(d, aw, qf[j][0], qf[j][1]);
          } else {  // the scaled query as bf16 again (exact), its largest magnitude in [1, 2)
            uint32_t qb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 f = kv8_pair<true>(qf[j][i]);
              qb[i] = ka_pack_bf16(f.x * 0x1p-14f, f.y * 0x1p-14f);
            }
            mma_bf16(d, aw[0], aw[1], aw[2], aw[3], qb[0], qb[1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * part + g + 8 * (i >> 1) < meta.w) s[0][i] = d[i] * (HALF ? qc[i & 1] : qc[i & 1] * 0x1p14f);
      }

      // ---- softmax state
      float x0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
      float x1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(kKaFull, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(kKaFull, x1, d));
      }
      const float y0 = x0 + (lv - 15.f), y1 = x1 + (lv - 15.f);
      if (__any_sync(kKaFull, x0 > m[0] || x1 > m[1] || y0 > mv[0] || y1 > mv[1])) {
        const float n0 = fmaxf(m[0], x0), n1 = fmaxf(m[1], x1), w0 = fmaxf(mv[0], y0), w1 = fmaxf(mv[1], y1);
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
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        l[0] += ka_exp2(s[t][0] - m0) + ka_exp2(s[t][2] - m0);
        l[1] += ka_exp2(s[t][1] - m1) + ka_exp2(s[t][3] - m1);
        s[t][0] = ka_exp2(s[t][0] - v0), s[t][1] = ka_exp2(s[t][1] - v1);
        s[t][2] = ka_exp2(s[t][2] - v0), s[t][3] = ka_exp2(s[t][3] - v1);
      }

      // ---- O^T += V^T P^T
      if (kind == kUnitPage) {
        constexpr bool kInf = FMT == GAAC_FP8_E5M2;  // E4M3 has no infinities
        uint32_t pb[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) ka_weights<true, kInf>(s[t], pb[t]);
#pragma unroll
        for (int i = 0; i < 8; i += 2)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            // matrices (tokens 0-7, 8-15) of channels 16 i .. and of 16 (i + 1) ..; a lane gets channels 2g, 2g+1 of
            // token 2tq (low half of the word) and of 2tq+1
            uint32_t r[4], a0[4], a1[4];
            ka_ldmatrix_t(r, ((base + lm_off) ^ (i << 4)) + kKv8Tile + 16 * 128 * t);
            ka_widen<FMT, true>(r[0], a0[0], a0[1]);
            ka_widen<FMT, true>(r[1], a0[2], a0[3]);
            ka_widen<FMT, true>(r[2], a1[0], a1[1]);
            ka_widen<FMT, true>(r[3], a1[2], a1[3]);
            ka_mma_f16(acc[i], a0, pb[t][0], pb[t][1]);
            ka_mma_f16(acc[i + 1], a1, pb[t][0], pb[t][1]);
            if (kInf) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                a0[j] = ka_finite_pair<true>(a0[j]);
                a1[j] = ka_finite_pair<true>(a1[j]);
              }
            }
            ka_mma_f16(acc[i], a0, pb[t][2], pb[t][3]);
            ka_mma_f16(acc[i + 1], a1, pb[t][2], pb[t][3]);
          }
      } else {
        uint32_t pb[4];
        ka_weights<HALF, true>(s[0], pb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t aw[4];
#pragma unroll
          for (int t8 = 0; t8 < 2; ++t8) {
            uint32_t x[2];
#pragma unroll
            for (int o = 0; o < 2; ++o) {  // token 2tq + o (+ 8): channels 16 i + 2g, + 1; rows behind the tokens are 0
              const uint32_t row = static_cast<uint32_t>(16 * part + 8 * t8 + 2 * tq + o);
              const uint32_t chunk = static_cast<uint32_t>(2 * (i & 3) + (g >> 2));
              const uint32_t at = kKv8Tile + (i >> 2) * (kKv8Pair / 4) + row * 128u + ((chunk ^ (row & 7u)) << 4) + 4u * (g & 3);
              x[o] = static_cast<int>(row) < meta.w ? *reinterpret_cast<const uint32_t*>(sm.stage[stage] + at) : 0u;
            }
            aw[2 * t8] = __byte_perm(x[0], x[1], 0x5410);
            aw[2 * t8 + 1] = __byte_perm(x[0], x[1], 0x7632);
          }
          if (HALF) {
            ka_mma_f16(acc[i], aw, pb[0], pb[1]);
          } else {
            mma_bf16(acc[i], aw[0], aw[1], aw[2], aw[3], pb[0], pb[1]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) aw[j] = ka_finite_pair<HALF>(aw[j]);
          if (HALF) {
            ka_mma_f16(acc[i], aw, pb[2], pb[3]);
          } else {
            mma_bf16(acc[i], aw[0], aw[1], aw[2], aw[3], pb[2], pb[3]);
          }
        }
      }
    }

    // ---- the end of the pair in this CTA
    if (last) {
      const int4 pair = sm.meta[stage][1];
      const int b = pair.x, h = pair.y, cta0 = pair.z, n_cta = pair.w;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[0] += __shfl_xor_sync(kKaFull, l[0], d);
        l[1] += __shfl_xor_sync(kKaFull, l[1], d);
      }
      if (last == kLastSolo) {
        // The group's two warps exchange halves: this one ends channels 64 part .. + 63, from its registers and the
        // other's state (5,000 x 100 tokens, 1 kv-head: 87 us; through shared memory as below 105).  Two buffers in
        // turn, so that one meeting a pair is enough.
        float(&st)[3][kKaRows] = sm.solo[turn][warp];
        const float(&st1)[3][kKaRows] = sm.solo[turn][warp ^ 1];
        float4* give = reinterpret_cast<float4*>(sm.state[warp]) + 128 * turn + lane;
        const float4* got = reinterpret_cast<const float4*>(sm.state[warp ^ 1]) + 128 * turn + lane;
        if (g == 0) {
          *reinterpret_cast<float2*>(&st[0][2 * tq]) = make_float2(m[0], m[1]);
          *reinterpret_cast<float2*>(&st[1][2 * tq]) = make_float2(l[0], l[1]);
          *reinterpret_cast<float2*>(&st[2][2 * tq]) = make_float2(mv[0], mv[1]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          give[32 * k] = part ? make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3])
                              : make_float4(acc[4 + k][0], acc[4 + k][1], acc[4 + k][2], acc[4 + k][3]);
        if (!ka_meet_at(&sm.pair_sync[warp >> 1], meet_pair, a.status)) return;
        const float2 m1 = *reinterpret_cast<const float2*>(&st1[0][2 * tq]), l1 = *reinterpret_cast<const float2*>(&st1[1][2 * tq]),
                     mv1 = *reinterpret_cast<const float2*>(&st1[2][2 * tq]);
        bool none[2];
        float f0[2], f1[2], e0[2], e1[2];  // O = f0 o + f1 o1 over the sum: O * e0 * e1, as in ka_result
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float ma = i ? m1.y : m1.x, la = i ? l1.y : l1.x, va = i ? mv1.y : mv1.x;
          const float mx = fmaxf(m[i], ma), vx = fmaxf(mv[i], va), z = ka_finite(mx), zv = ka_finite(vx);
          const float den = ka_exp2(m[i] - z) * l[i] + ka_exp2(ma - z) * la;
          f0[i] = ka_exp2(mv[i] - zv);
          f1[i] = ka_exp2(va - zv);
          e1[i] = ka_exp2(0.5f * (zv - z));
          e0[i] = e1[i] / den;
          none[i] = den == 0.f;
        }
        turn ^= 1;
        gave = true;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 x = got[32 * k];
          float y[4] = {part ? acc[4 + k][0] : acc[k][0], part ? acc[4 + k][1] : acc[k][1],
                        part ? acc[4 + k][2] : acc[k][2], part ? acc[4 + k][3] : acc[k][3]};
          y[0] = none[0] ? 0.f : (f0[0] * y[0] + f1[0] * x.x) * e0[0] * e1[0];
          y[1] = none[1] ? 0.f : (f0[1] * y[1] + f1[1] * x.y) * e0[1] * e1[1];
          y[2] = none[0] ? 0.f : (f0[0] * y[2] + f1[0] * x.z) * e0[0] * e1[0];
          y[3] = none[1] ? 0.f : (f0[1] * y[3] + f1[1] * x.w) * e0[1] * e1[1];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (2 * tq + i < a.r) ka_store2<HALF>(a, b, h, 2 * tq + i, 64 * part + 16 * k + 2 * g, y[i], y[2 + i]);
        }
      } else {
        // the other warp of the group may still read what this one gave
        if (gave && !ka_meet_at(&sm.pair_sync[warp >> 1], meet_pair, a.status)) return;
        gave = false;
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
        // this CTA's part of the pair: the states of all warps
        for (int at = tid; at < a.r * (kD / 4); at += kKaCompute) {
          const int row = at / (kD / 4), ch = 4 * (at % (kD / 4));
          float mx = -INFINITY, vx = -INFINITY, den = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
          for (int w = 0; w < kKaWarps; ++w) {
            mx = fmaxf(mx, sm.m[w][row]);
            vx = fmaxf(vx, sm.mv[w][row]);
          }
#pragma unroll 2
          for (int w = 0; w < kKaWarps; ++w) {
            den += ka_exp2(sm.m[w][row] - ka_finite(mx)) * sm.l[w][row];
            const float f = ka_exp2(sm.mv[w][row] - ka_finite(vx));
            const float4 x = *reinterpret_cast<const float4*>(&sm.state[w][row][ch]);
            o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
          }
          if (n_cta == 1)
            ka_store<HALF>(a, b, h, row, ch, ka_result(o, mx, den, vx));
          else
            ka_put(a.part + ka_slot(blockIdx.x, cta0) * kKaPart, row, ch, mx, den, vx, o);
        }
        if (n_cta != 1 && !ka_join<HALF>(a, sm, b, h, cta0, n_cta, meet)) return;
        // the next pair's state may be written once everybody has read this one's
        if (!ka_meet(sm, meet, a.status)) return;
      }
    }
    __syncwarp();
    if (lane == 0) ka_arrive(&sm.empty[stage]);
    stage += kKaGroups;
    if (stage >= kKaStages) {
      stage -= kKaStages;
      phase ^= 1u;
    }
  }
}

template <bool HALF, int FMT>
__global__ void __launch_bounds__(kKaThreads, 1)
    kv8_attention_kernel(const KaArgs a, const __grid_constant__ CUtensorMap pages, const __grid_constant__ CUtensorMap tail) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  KaSmem& sm = *reinterpret_cast<KaSmem*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKaStages; ++i) {
      mbar_init(&sm.full[i], 2);
      mbar_init(&sm.empty[i], 2);
    }
    mbar_init(&sm.sync, kKaWarps);
    for (int i = 0; i < kKaGroups; ++i) mbar_init(&sm.pair_sync[i], 2);
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(&pages) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tail) : "memory");
  }
  __syncthreads();
  if (threadIdx.x < 32) ka_guess(a);  // a compute warp: it has nothing to do before the first data
  dependent_wait();
  dependent_launch();
  if (a.c.batch > 32) {  // all warps add up the units (see ka_cut)
    unsigned* places = sm.places();
    ka_sums(a.c, threadIdx.x / 32, kKaThreads / 32, 1u, blockIdx.x == 0 ? a.status : nullptr, [&](int j, unsigned sum) {
      if (threadIdx.x % 32 == 0) places[j] = sum;
    });
    __syncthreads();
  }
  if (threadIdx.x >= 32 * kKaWarps) {
    ka_copy_warp(a, sm, &pages, &tail, threadIdx.x / 32 - kKaWarps);
  } else {
    if (a.c.batch > 32) __syncthreads();  // the copy warps have read them
    ka_compute<HALF, FMT>(a, sm);
  }
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

// Counters: one for each pair (at its first CTA) and two for the teams that begin at a CTA.
static size_t ka_counter_bytes(int grid) { return (static_cast<size_t>(3 * grid) * 4 + 15) & ~static_cast<size_t>(15); }

// A map of [rows][128 bytes-wide column blocks]: boxes of box_x elements by box_y rows, 128-byte swizzle.
static bool ka_map(CUtensorMap* m, CUtensorMapDataType type, int elem, void* base, int64_t rows, unsigned box_x, unsigned box_y) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(kD * elem)};
  const cuuint32_t box[2] = {box_x, box_y}, one[2] = {1, 1};
  return tma_encode()(m, type, 2, base, dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
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
  const int grid = ka_sms();
  return ka_counter_bytes(grid) + static_cast<size_t>(4 * grid) * kKaPart * sizeof(float);
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
  if (static_cast<int64_t>(cache->batch) * cache->n_kv_heads > 0x7FFFFFFF / (static_cast<int64_t>(cache->max_blocks) + 1))
    return GAAC_EINVAL;
  const int sms = ka_sms();
  if (sms <= 0 || tma_encode() == nullptr) return GAAC_ECUDA;
  if (workspace_bytes < gaac_kv8_attention_workspace()) return GAAC_EINVAL;
  const int grid = sms;
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
      !ka_map(&tail, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, cache->tail, cache->batch * rows, kD / 2, kKaHalf))
    return GAAC_ECUDA;
  const bool e4 = cache->fmt == GAAC_FP8_E4M3;
  if (cache->dtype == GAAC_F16)
    return e4 ? ka_launch<true, GAAC_FP8_E4M3>(a, pages, tail, grid, stream)
              : ka_launch<true, GAAC_FP8_E5M2>(a, pages, tail, grid, stream);
  return e4 ? ka_launch<false, GAAC_FP8_E4M3>(a, pages, tail, grid, stream)
            : ka_launch<false, GAAC_FP8_E5M2>(a, pages, tail, grid, stream);
}
