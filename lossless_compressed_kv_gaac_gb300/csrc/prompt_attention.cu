// Attention of whole prompts: causal, grouped heads, packed sequences of different lengths.
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   within a sequence, query head hq reading kv-head hq / G.
//
// Tensor bound where prompts are long: 4 * 128 operations for each pair (i, j <= i) and query head.  A CTA takes 2 x
// floor(128 / G) consecutive tokens of one sequence with all G query heads of one kv-head, as two tiles of up to 128
// rows (row r of a tile: token r / G, head r % G), so that a tile's rows share their keys, its diagonal is short
// and few tokens still fill a tile.  Warps:
//  * one issues the copies (TMA): both tiles' queries, then K and V of 128 tokens in turn into a ring of five slots;
//  * one for each tile multiplies (tcgen05.mma): S = Q K^T (128 x 128, both operands in shared memory), O += P V (P in TMEM, V's
//    rows as they lie, token-major).  While one tile's S is in its softmax, the tensor cores work for the other.
//  * four warps for each tile: a thread owns a row.  S comes from TMEM into its registers; P goes back, rounded to the
//    inputs' type, over the S it came from.  All of TMEM's 512 columns are used: S and O of both tiles.
//  * four look over V (below).
// Softmax: weights are 2^(c s - c m), c = |scale| log2 e, with a reference m that follows the running maximum only where
// that has grown by more than 2^8: then O and the sum are scaled.  Until then weights are at most 2^8, which costs
// nothing in either type (rounding is relative; f16 goes to 2^16, and loses those below 2^-25 of the reference, which is
// at most the row's maximum).  Sums are fp32 over the unrounded weights; a weight's rounding, 2^-8 at most in bf16 and
// 2^-11 in f16, is that of the result's type.
// Where a mask leaves keys out, V has to be finite there, or 0 * V would be NaN: four warps look such a block of V over
// before it is multiplied and put zeros in the place of what is not finite.  What of that rows may see is added
// to them at the end, from memory.
// 1 x 16,384 tokens, 32 / 8 heads, bf16: 1.39-1.42 ms, 1.55-1.58 PFLOP/s, 80% of the measured burst rate of a library product.  A block of
// keys takes both tiles some 3,000 cycles, of which the tensor cores work 2,048: a tile's chain is its softmax (1,200-1,300 cycles: the
// exponentials are a third of it), P V and Q K^T (768 behind the last weight) and the ways between warps (some 500).  What
// brought it there from 1.82 ms: a multiplying warp for each tile and converged issue (1.69), packed arithmetic and three-way
// maxima, weights multiplied in two parts, and the maximum off the chain with waits that poll (1.43).  Short prompts pay 7,000 cycles
// a unit for its start and end (32 x 1-2,048 tokens, 16 / 8 heads, f16: 240 us, 0.8 PFLOP/s; 1 x 777: 17.5 us).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <numeric>

#include "f32x2.cuh"
#include "kv8.cuh"
#include "tma.cuh"

namespace gaac {

constexpr int kPaRows = 128;                  // rows of a tile
constexpr int kPaKeys = 128;                  // keys of a block
constexpr int kPaTile = 128 * kD * 2;         // bytes of a tile of Q, K or V
constexpr int kPaHalf = kPaTile / 2;          // 64 channels of it: rows of 128 bytes, swizzled
constexpr int kPaSlots = 5;
constexpr int kPaSoftmax = 256;
constexpr int kPaCleaners = 128;
constexpr int kPaThreads = kPaSoftmax + 128 + kPaCleaners;   // 128: two multipliers, the copier, one warp idle
constexpr int kPaEarly = 64;                  // keys of a block whose weights are multiplied ahead of the others
constexpr int64_t kPaApartBytes = int64_t{64} << 20;  // of K and V, and units for each SM, from which kv-heads are taken one
constexpr int kPaApartUnits = 11;                     // after the other
constexpr int kPaLook = 3;                    // blocks of a unit that have masked keys, at most
constexpr uint32_t kPaFull = 0xFFFFFFFFu;
constexpr uint32_t kPaColS = 0, kPaColO = 256;  // TMEM columns: S of tile t at 128 t, P over it, O at 256 + 128 t

struct PaArgs {
  const int32_t* cu;
  int batch, hkv, g, per;      // per: tokens of a tile
  int g_inverse;               // row / g is row * g_inverse >> 16
  unsigned places;
  int heads_apart;             // one kv-head after the other
  int64_t n_tokens;
  float c;                     // |scale| log2 e
  int negate;                  // scale < 0: the logits' sign turns
  const char* v;
  int64_t v_tok, v_head;       // bytes
  char* out;
  int64_t out_tok, out_head;   // bytes
  float* lse;                  // [n_tokens][hkv * g], or nullptr
  int32_t* status;
};

struct PaSmem {
  alignas(1024) uint8_t q[2][kPaTile];
  alignas(1024) uint8_t kv[kPaSlots][kPaTile];
  uint64_t q_full[2], kv_full[kPaSlots], kv_empty[kPaSlots], s_full[2], p_early[2], p_full[2], o_full[2], due[kPaLook], clean[kPaLook], done[2];
  uint32_t tmem;
  int odd;  // a V that some row may see is not finite in a block with masked keys
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void t5_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a),
      "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void t5_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a),
      "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// `bar` is arrived at once all that this thread has issued so far is done.
__device__ __forceinline__ void t5_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void t5_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void t5_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void t5_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define GAAC_W8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define GAAC_W32(x, i) GAAC_W8(x, i), GAAC_W8(x, i + 8), GAAC_W8(x, i + 16), GAAC_W8(x, i + 24)
#define GAAC_I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])

// Columns of this warp's 32 lanes, one lane a thread: the wait is part of the load, so nothing uses a register before it.
__device__ __forceinline__ void t5_ld32(uint32_t* x, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : GAAC_W8(x, 0), GAAC_W8(x, 8), GAAC_W8(x, 16), GAAC_W8(x, 24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void t5_ld128(uint32_t* x, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : GAAC_W32(x, 0), GAAC_W32(x, 32), GAAC_W32(x, 64), GAAC_W32(x, 96)
      : "r"(at), "r"(at + 32), "r"(at + 64), "r"(at + 96)
      : "memory");
}
__device__ __forceinline__ void t5_st32(uint32_t at, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      GAAC_I8(x, 0), GAAC_I8(x, 8), GAAC_I8(x, 16), GAAC_I8(x, 24)
      : "memory");
}
__device__ __forceinline__ void t5_st16(uint32_t at, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      GAAC_I8(x, 0), GAAC_I8(x, 8)
      : "memory");
}

// Shared-memory operand, 128-byte swizzle.  Rows of 64 channels, channels along the contraction (Q, K): groups of eight
// rows 1,024 bytes apart.  Contraction over the rows (V): the same, and the next 64 channels kPaHalf further.
__device__ __forceinline__ uint64_t pa_desc(uint32_t addr, uint32_t leading) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(leading >> 4) << 16 | static_cast<uint64_t>(1024 >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}
// 128 x 128 with fp32 sums; v: B is V, whose rows run along the contraction.
__device__ __forceinline__ uint32_t pa_idesc(bool bf16, bool v) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (v ? 1u << 16 : 0u) | (128u >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void pa_tma(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float pa_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool HALF>
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
  uint32_t r;
  if (HALF)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ------------------------------------------------------------------ units

// What a CTA works on: tokens t0 .. t0 + 2 per - 1 of a sequence that begins at row `first` and has len tokens.
struct PaUnit {
  int first, len, t0, h;
  int blocks[2];  // of keys, for each tile; 0: no tokens
  int look;       // the first block with keys that some row does not see; less than kPaLook from the last
};

// Units of 2 per tokens, numbered (x) by a rule that puts those with many keys first, so that the last CTAs to run are short
// ones.  By a whole warp.  false: nothing to do here.
//  * Up to 32 sequences, one a lane: the units that are number `level` of their sequence, for all sequences, from the highest
//    level down.  There are C(l) = sum_b max(0, units_b - l) of level l and above.
//  * More: from the last sequence back, and from the last unit of each.  Sequence b owns places [cu[b] / T + b, cu[b + 1] / T +
//    b + 1), T = 2 per: as many as it can need, some are empty.
__device__ __forceinline__ bool pa_unit(const PaArgs& a, PaUnit& u) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = 2 * a.per;
  int64_t lo, hi, t0;
  if (a.batch <= 32) {
    const int64_t from = lane < a.batch ? a.cu[lane] : 0, to = lane < a.batch ? a.cu[lane + 1] : 0;
    if (__any_sync(kPaFull, from < 0 || to < from || to > a.n_tokens)) {
      if (blockIdx.x == 0 && lane == 0) report(a.status, GAAC_EINVAL);
      return false;
    }
    const int units = static_cast<int>((to - from + unit - 1) / unit);
    const int total = __reduce_add_sync(kPaFull, units), top = __reduce_max_sync(kPaFull, units);
    int x = static_cast<int>(blockIdx.x);
    if (a.heads_apart) {
      u.h = total > 0 ? x / total : a.hkv;
      x -= u.h * total;
    } else {
      u.h = x % a.hkv;
      x /= a.hkv;
    }
    if (u.h >= a.hkv || x >= total) return false;
    int low = 0, high = top;  // C(low) > x >= C(high)
    while (high - low > 1) {
      const int mid = (low + high) / 2;
      if (static_cast<int>(__reduce_add_sync(kPaFull, max(0, units - mid))) > x)
        low = mid;
      else
        high = mid;
    }
    x -= static_cast<int>(__reduce_add_sync(kPaFull, max(0, units - high)));
    uint32_t have = __ballot_sync(kPaFull, units > low);
    for (; x > 0; --x) have &= have - 1u;
    const int b = __ffs(have) - 1;
    lo = __shfl_sync(kPaFull, from, b);
    hi = __shfl_sync(kPaFull, to, b);
    t0 = low * unit;
  } else {
    u.h = static_cast<int>(blockIdx.x / a.places);
    const int64_t place = a.places - 1 - (blockIdx.x - u.h * a.places);
    int count = 0, bad = 0;
#pragma unroll 4
    for (int i0 = 0; i0 < a.batch; i0 += 32) {
      const int i = i0 + lane;
      bool below = false;
      if (i < a.batch) {
        const int64_t from = a.cu[i], to = a.cu[i + 1];
        if (from < 0 || to < from || to > a.n_tokens) bad = 1;
        below = to / unit + i + 1 <= place;
      }
      count += __popc(__ballot_sync(kPaFull, below));
    }
    if (__any_sync(kPaFull, bad)) {
      if (blockIdx.x == 0 && lane == 0) report(a.status, GAAC_EINVAL);
      return false;
    }
    if (count >= a.batch) return false;
    lo = a.cu[count];
    hi = a.cu[count + 1];
    const int64_t p0 = lo / unit + count;
    t0 = (place - p0) * unit;
    if (place < p0 || t0 >= hi - lo) return false;
  }
  u.first = static_cast<int>(lo);
  u.len = static_cast<int>(hi - lo);
  u.t0 = static_cast<int>(t0);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int from = u.t0 + t * a.per;
    u.blocks[t] = from < u.len ? (min(u.len, from + a.per) + kPaKeys - 1) / kPaKeys : 0;
  }
  u.look = u.t0 / kPaKeys;
  return true;
}

// The copy that brings K (kind 0) or V of block i is number 2 i + kind.
__device__ __forceinline__ int pa_slot(int n) { return n % kPaSlots; }
__device__ __forceinline__ uint32_t pa_phase(int n) { return (n / kPaSlots) & 1; }

__device__ __forceinline__ void pa_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ void pa_load(const PaArgs& a, PaSmem& sm, const PaUnit& u, const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv) {
  const int blocks = max(u.blocks[0], u.blocks[1]);
  const uint32_t q_bytes = static_cast<uint32_t>(a.g) * a.per * kD * 2;
  auto q = [&](int t) {
    if (u.blocks[t] == 0) return;
    mbar_arrive_expect_tx(&sm.q_full[t], q_bytes);
#pragma unroll
    for (int half = 0; half < 2; ++half)
      pa_tma(sm.q[t] + half * kPaHalf, mq, half * (kD / 2), u.h * a.g, u.first + u.t0 + t * a.per, &sm.q_full[t]);
  };
  q(0);
  int n = 0;
  bool ok = true;
  for (; n < 2 * blocks && ok; ++n) {
    const int slot = pa_slot(n);
    if (n >= kPaSlots) ok = mbar_wait(&sm.kv_empty[slot], pa_phase(n) ^ 1u, a.status);
    if (!ok) break;
    mbar_arrive_expect_tx(&sm.kv_full[slot], kPaTile);
#pragma unroll
    for (int half = 0; half < 2; ++half)
      pa_tma(sm.kv[slot] + half * kPaHalf, n & 1 ? mv : mk, half * (kD / 2), u.h, u.first + (n >> 1) * kPaKeys, &sm.kv_full[slot]);
    if (n == 0) q(1);
    // the slot's barrier is now in the phase of this copy, whoever waits for it without having seen those before
    if ((n & 1) && (n >> 1) >= u.look) pa_arrive(&sm.due[(n >> 1) - u.look]);
  }
  // no copy may be in flight when the CTA ends, not even where a wait ran out
  for (int i = max(0, n - kPaSlots); i < n; ++i) mbar_wait(&sm.kv_full[pa_slot(i)], pa_phase(i), a.status);
  for (int t = 0; t < 2; ++t)
    if (u.blocks[t]) mbar_wait(&sm.q_full[t], 0, a.status);
}

// A bounded wait that the whole warp takes alike.  The first polls come back at once: a phase that is nearly over is met
// without the time that a sleeping warp needs to wake.
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    if (__all_sync(kPaFull, ok)) return true;
  }
  return __all_sync(kPaFull, mbar_wait(bar, parity, status));
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool pa_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0u;
}

// Tile t's multiplier.  All of the warp walks along and one lane issues, so that addresses and descriptors are known to be
// the same for the warp: with a branch that one lane alone takes, an instruction took some 75 cycles to issue, and its
// thread, not the tensor cores, was what the kernel waited for.  One warp for both tiles spends as long in its waits
// and commits as the tensor cores need for the products; with one for each, either's fall under the other's products.
template <bool HALF>
__device__ void pa_mma(const PaArgs& a, PaSmem& sm, const PaUnit& u, uint32_t tmem, int t) {
  const uint32_t id_qk = pa_idesc(!HALF, false), id_pv = pa_idesc(!HALF, true);
  const int blocks = u.blocks[t], all = max(u.blocks[0], u.blocks[1]);
  const uint32_t col_s = tmem + kPaColS + 128 * t, col_o = tmem + kPaColO + 128 * t;
  const uint64_t q0 = pa_desc(smem_addr(sm.q[t]), 16), k0 = pa_desc(smem_addr(sm.kv[0]), 16), v0 = pa_desc(smem_addr(sm.kv[0]), kPaHalf);
  auto qk = [&](int slot) {
    const uint64_t k = k0 + slot * (kPaTile / 16);
#pragma unroll
    for (int j = 0; j < kD / 16; ++j) {
      const uint32_t at = ((j / 4) * kPaHalf + (j % 4) * 32) / 16;
      t5_mma_ss(col_s, q0 + at, k + at, id_qk, j > 0);
    }
    t5_commit(&sm.s_full[t]);
  };
  auto pv = [&](int slot, uint32_t add, int j0, int j1) {
    const uint64_t v = v0 + slot * (kPaTile / 16);
#pragma unroll
    for (int j = j0; j < j1; ++j) t5_mma_ts(col_o, col_s + 8 * j, v + j * (2048 / 16), id_pv, j > 0 ? 1u : add);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return pa_wait(bar, parity, a.status); };
  // A slot is handed back by the multipliers of both tiles (of the one that has tokens), where there is a copy that waits for
  // it.  The first tile has one block less than the second at most, which no copy waits for.
  bool ok = true;
  if (blocks > 0) {
    ok = wait(&sm.q_full[t], 0) && wait(&sm.kv_full[0], 0);
    if (ok && pa_elect()) {
      qk(0);
      if (kPaSlots < 2 * all) t5_commit(&sm.kv_empty[0]);
    }
    __syncwarp();
  }
  int slot = 1;  // of V of block i
  uint32_t phase = 0;
  for (int i = 0; i < blocks && ok; ++i) {
    const int v_slot = slot;
    ok = wait(&sm.kv_full[v_slot], phase);
    if (++slot == kPaSlots) slot = 0, phase ^= 1u;
    const int k_slot = slot;
    ok = ok && (i + 1 >= blocks || wait(&sm.kv_full[k_slot], phase)) && (i < u.look || wait(&sm.clean[i - u.look], 0)) &&
         wait(&sm.p_early[t], i & 1);
    if (++slot == kPaSlots) slot = 0, phase ^= 1u;
    if (!ok) break;
    t5_after();
    if (pa_elect()) pv(v_slot, i > 0, 0, kPaEarly / 16);
    __syncwarp();
    ok = wait(&sm.p_full[t], i & 1);
    if (!ok) break;
    t5_after();
    if (pa_elect()) {
      pv(v_slot, 1u, kPaEarly / 16, kPaKeys / 16);
      t5_commit(&sm.o_full[t]);
      if (2 * i + 1 + kPaSlots < 2 * all) t5_commit(&sm.kv_empty[v_slot]);
      if (i + 1 < blocks) {
        qk(k_slot);
        if (2 * i + 2 + kPaSlots < 2 * all) t5_commit(&sm.kv_empty[k_slot]);
      }
    }
    __syncwarp();
  }
  // nothing may be under way when TMEM is given back
  if (pa_elect()) t5_commit(&sm.done[t]);
  __syncwarp();
  wait(&sm.done[t], 0);
}

// Four warps (one takes 8,500 cycles for a block, longer than a short prompt's whole softmax): infinities and NaN become 0 in the blocks of V with masked keys.
template <bool HALF>
__device__ void pa_look(const PaArgs& a, PaSmem& sm, const PaUnit& u) {
  constexpr uint32_t kCarry = HALF ? 0x04000400u : 0x00800080u;  // takes an exponent of ones into the sign's place
  const int tid = threadIdx.x % kPaCleaners, blocks = max(u.blocks[0], u.blocks[1]);
  for (int i = u.look; i < blocks; ++i) {
    const int n = 2 * i + 1;
    if (!__all_sync(kPaFull, mbar_wait(&sm.due[i - u.look], 0, a.status) && mbar_wait(&sm.kv_full[pa_slot(n)], pa_phase(n), a.status)))
      return;
    uint4* const v = reinterpret_cast<uint4*>(sm.kv[pa_slot(n)]) + tid;
#pragma unroll 4
    for (int k = 0; k < kPaTile / 16; k += kPaCleaners) {
      const uint4 w = v[k];
      const uint32_t any = ((w.x & 0x7FFF7FFFu) + kCarry) | ((w.y & 0x7FFF7FFFu) + kCarry) | ((w.z & 0x7FFF7FFFu) + kCarry) |
                           ((w.w & 0x7FFF7FFFu) + kCarry);
      if (any & 0x80008000u) {
        auto fix = [](uint32_t x) {
          const uint32_t y = ((x & 0x7FFF7FFFu) + kCarry) & 0x80008000u;  // the sign's place of what is not finite
          return x & ~((y >> 15) * 0xFFFFu);
        };
        v[k] = make_uint4(fix(w.x), fix(w.y), fix(w.z), fix(w.w));
        if (i * kPaKeys + (k + tid) % (kPaHalf / 16) / 8 < u.len) sm.odd = 1;  // eight vectors of a token in each half
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) pa_arrive(&sm.clean[i - u.look]);
  }
}

template <bool HALF>
__device__ void pa_softmax(const PaArgs& a, PaSmem& sm, const PaUnit& u, uint32_t tmem, int t) {
  const int row = threadIdx.x % kPaRows, blocks = u.blocks[t];
  const int from = u.t0 + t * a.per, in_tile = row / a.g, token = from + in_tile;
  const bool real = in_tile < a.per && token < u.len;
  const uint32_t lane_at = tmem + (static_cast<uint32_t>(row & ~31) << 16);  // this warp's lanes
  const uint32_t at_s = lane_at + kPaColS + 128 * t, at_o = lane_at + kPaColO + 128 * t;
  float m = -INFINITY, l = 0.f;  // the reference, times c; the sum
  bool ok = true;
  for (int i = 0; i < blocks && ok; ++i) {
    ok = pa_wait(&sm.s_full[t], i & 1, a.status);
    if (!ok) break;
    t5_after();
    uint32_t s[128];
    t5_ld128(s, at_s);
    if (a.negate) {
#pragma unroll
      for (int k = 0; k < 128; ++k) s[k] ^= 0x80000000u;
    }
    const bool masked = i * kPaKeys + kPaKeys - 1 > from;  // for some row
    if (masked) {
      const int last = token - i * kPaKeys;  // the last key that this row sees
#pragma unroll
      for (int k = 0; k < 128; ++k)
        if (k > last) s[k] = 0xFF800000u;
    }
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = max3(__uint_as_float(s[j]), __uint_as_float(s[8 + j]), __uint_as_float(s[16 + j]));
#pragma unroll
    for (int k = 24; k < 120; k += 16)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = max3(x[j], __uint_as_float(s[k + j]), __uint_as_float(s[k + 8 + j]));
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaxf(x[j], __uint_as_float(s[120 + j]));
    const float top = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7])) * a.c;
    // Nothing below but the check needs this block's maximum, so it is found while the exponentials are taken with the
    // reference as it is; where that turns out to be too far below, they are taken again.
    if (i == 0) m = top;
    const uint64_t c2 = f2_make(a.c, a.c);
    uint64_t sum[2];
    float base;
    auto weights = [&](int k, uint32_t (&p)[16]) {
      const uint64_t base2 = f2_make(-base, -base);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 e = f2_get(f2_fma(f2_make(__uint_as_float(s[32 * k + 2 * j]), __uint_as_float(s[32 * k + 2 * j + 1])), c2, base2));
        const float p0 = pa_exp2(e.x), p1 = pa_exp2(e.y);
        sum[j & 1] = f2_add(sum[j & 1], f2_make(p0, p1));
        p[j] = pa_pack<HALF>(p0, p1);
      }
    };
    uint32_t p[16];
    while (true) {
      base = m == -INFINITY ? 0.f : m;
      sum[0] = sum[1] = 0;
      weights(0, p);
      t5_st16(at_s, p);
      weights(1, p);
      t5_st16(at_s + 16, p);
      const bool up = top > m + 8.f;
      if (!__any_sync(kPaFull, up)) break;
      const float to = up ? top : m, f = up ? pa_exp2(m - to) : 1.f;
      l *= f;
      m = to;
      if (i > 0) {
        ok = pa_wait(&sm.o_full[t], (i - 1) & 1, a.status);
        if (!ok) break;
        t5_after();
#pragma unroll 1
        for (int k = 0; k < 128; k += 32) {
          uint32_t o[32];
          t5_ld32(o, at_o + k);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          t5_st32(at_o + k, o);
        }
      }
    }
    if (!ok) break;
    weights(2, p);
    // the weights of the first keys are where the tensor cores read them
    t5_wait_st();
    t5_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) pa_arrive(&sm.p_early[t]);
    t5_st16(at_s + 32, p);
    weights(3, p);
    t5_st16(at_s + 48, p);
    const float2 sums = f2_get(f2_add(sum[0], sum[1]));
    l += sums.x + sums.y;
    t5_wait_st();
    t5_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) pa_arrive(&sm.p_full[t]);
  }
  if (blocks == 0 || !ok) return;
  if (!pa_wait(&sm.o_full[t], (blocks - 1) & 1, a.status)) return;
  t5_after();
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t token_at = static_cast<int64_t>(u.first) + token;
  const int head = u.h * a.g + row % a.g;
  // A thread has a row; stores of neighbouring channels by neighbouring threads need a turn through shared memory (stored by
  // rows, the two tiles of a unit take 4,000 cycles).  The queries have been multiplied: a warp's rows take their place, 16-byte
  // pieces swizzled by the row.
  uint8_t* const stage = sm.q[t] + (row & ~31) * (2 * kD);
  const int lane = row & 31;
#pragma unroll 1
  for (int k = 0; k < 128; k += 32) {
    uint32_t o[32];
    t5_ld32(o, at_o + k);
    float y[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) y[j] = l == 0.f ? 0.f : __uint_as_float(o[j]) * inv;
    if (real && l != 0.f && *reinterpret_cast<volatile int*>(&sm.odd)) {  // V that is not finite, of the blocks that were looked over
      for (int key = u.look * kPaKeys; key <= token; ++key) {
        const uint16_t* v = reinterpret_cast<const uint16_t*>(a.v + (static_cast<int64_t>(u.first) + key) * a.v_tok + u.h * a.v_head) + k;
#pragma unroll 1
        for (int j = 0; j < 32; ++j) {
          const float w = kv8_pair<HALF>(v[j]).x;
          if (!isfinite(w)) {
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (q == j) y[q] += w;
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4*>(stage + lane * (2 * kD) + (((k / 8 + j) ^ (lane & 7)) << 4)) =
          make_uint4(pa_pack<HALF>(y[8 * j], y[8 * j + 1]), pa_pack<HALF>(y[8 * j + 2], y[8 * j + 3]),
                     pa_pack<HALF>(y[8 * j + 4], y[8 * j + 5]), pa_pack<HALF>(y[8 * j + 6], y[8 * j + 7]));
  }
  __syncwarp();
  const int piece = lane & 15;
  char* const out = a.out + (static_cast<int64_t>(u.first) + from) * a.out_tok + u.h * a.g * a.out_head + piece * 16;
  const int left = min(a.per, u.len - from);
#pragma unroll
  for (int k0 = 0; k0 < 16; k0 += 8) {  // eight loads, then eight stores: one after the other, a step takes 225 cycles
    uint4 y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 2 * (k0 + k) + (lane >> 4);
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(y[k].x), "=r"(y[k].y), "=r"(y[k].z), "=r"(y[k].w) : "r"(smem_addr(stage) + r * (2 * kD) + ((piece ^ (r & 7)) << 4)));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int of = (row & ~31) + 2 * (k0 + k) + (lane >> 4), tok = of * a.g_inverse >> 16;
      if (tok < left)
        asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(out + tok * a.out_tok + (of - tok * a.g) * a.out_head), "r"(y[k].x),
                     "r"(y[k].y), "r"(y[k].z), "r"(y[k].w) : "memory");
    }
  }
  if (real && a.lse != nullptr) a.lse[token_at * (static_cast<int64_t>(a.hkv) * a.g) + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147181f;
}

template <bool HALF>
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const PaArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                            const __grid_constant__ CUtensorMap mv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PaSmem& sm = *reinterpret_cast<PaSmem*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 32 * 10) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mq) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mv) : "memory");
  }
  dependent_wait();
  dependent_launch();
  PaUnit u;
  if (!pa_unit(a, u)) return;  // the same for all warps
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_full[t], 1);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_early[t], 4);
      mbar_init(&sm.p_full[t], 4);
      mbar_init(&sm.o_full[t], 1);
      mbar_init(&sm.done[t], 1);
    }
    sm.odd = 0;
    for (int i = 0; i < kPaLook; ++i) {
      mbar_init(&sm.due[i], 1);
      mbar_init(&sm.clean[i], kPaCleaners / 32);
    }
    for (int i = 0; i < kPaSlots; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], u.blocks[1] > 0 ? 2 : 1);
    }
    fence_mbar_init();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  t5_before();
  __syncthreads();
  t5_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sm.tmem);
  // Registers go from the eight warps that need few to the softmax, whose rows fill 128 of them: 256 * 208 + 128 * (56 + 40) is
  // what 512 threads are launched with.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    pa_softmax<HALF>(a, sm, u, tmem, warp / 4);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < 10) {
      pa_mma<HALF>(a, sm, u, __shfl_sync(kPaFull, tmem, 0), warp - 8);
    } else if (warp == 10) {
      if ((threadIdx.x & 31) == 0) pa_load(a, sm, u, &mq, &mk, &mv);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    pa_look<HALF>(a, sm, u);
  }
  __syncwarp();
  t5_before();
  __syncthreads();
  if (warp == 8) {
    t5_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ host

// [tokens][heads][128] of a 16-bit type: boxes of 64 channels, `heads_box` heads and `tokens_box` tokens.
static bool pa_map(CUtensorMap* m, const void* base, int64_t tokens, int64_t heads, int64_t tok, int64_t head, unsigned heads_box,
                   unsigned tokens_box) {
  const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head * 2 : kD * 2), static_cast<cuuint64_t>(tokens > 1 ? tok * 2 : kD * 2)};
  const cuuint32_t box[3] = {kD / 2, heads_box, tokens_box}, one[3] = {1, 1, 1};
  return tma_encode()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a tensor's elements lie between and how they repeat: [tokens][heads][128], strides in elements.
struct PaSpan {
  int64_t at, tok, head, heads, end;  // the addresses in bytes
  PaSpan(const void* base, int64_t n, int64_t heads, int64_t tok, int64_t head)
      : at(static_cast<int64_t>(reinterpret_cast<uintptr_t>(base))), tok(n > 1 ? tok : 0), head(heads > 1 ? head : 0), heads(heads),
        end(at + ((n - 1) * this->tok + (heads - 1) * this->head + kD) * 2) {}
  int64_t row() const { return (heads - 1) * head + kD; }
};
// No element in common, shown in one of three ways: the ranges are apart; tokens lie alike and a token's heads are apart, as the slices
// of one projection; or all strides are multiples of a period in which the heads' channels have places of their own.
static bool pa_apart(const PaSpan& x, const PaSpan& y) {
  if (x.end <= y.at || y.end <= x.at) return true;
  const int64_t d = (y.at - x.at) / 2;
  auto within = [d](int64_t period, int64_t first, int64_t second) {
    if (period == 0) return false;
    const int64_t r = ((d % period) + period) % period;
    return r >= first && r + second <= period;
  };
  return (x.tok == y.tok && within(x.tok, x.row(), y.row())) ||
         within(std::gcd(std::gcd(x.tok, y.tok), std::gcd(x.head, y.head)), kD, kD);
}

template <bool HALF>
static int pa_launch(const PaArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, void* stream) {
  constexpr size_t smem = sizeof(PaSmem) + 1024;  // room to align the tiles
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GAAC_ECUDA;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(prompt_attention_kernel<HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return GAAC_ECUDA;
    done[dev] = true;
  }
  return kv8_launch(prompt_attention_kernel<HALF>, dim3(grid), kPaThreads, smem, stream, a, q, k, v);
}

}  // namespace gaac

using namespace gaac;

extern "C" int gaac_prompt_attention(const gaac_prompt* p, int dtype, int64_t n_tokens, int n_q_heads, int n_kv_heads,
                                     const int32_t* cu_tokens, int batch, float scale, int32_t* d_status, void* stream) {
  const double c = std::fabs(static_cast<double>(scale)) * 1.4426950408889634;
  if (p == nullptr || (dtype != GAAC_BF16 && dtype != GAAC_F16) || n_tokens < 0 || n_tokens > 0x7FFFFFFF - 65536 || batch < 0 ||
      batch > 65535 || !(c <= FLT_MAX) || n_kv_heads < 1 || n_kv_heads > 1024 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0 ||
      n_q_heads / n_kv_heads > GAAC_MAX_GQA)
    return GAAC_EINVAL;
  if (n_tokens == 0 || batch == 0) return GAAC_OK;
  const uintptr_t all = reinterpret_cast<uintptr_t>(p->q) | reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v) |
                        reinterpret_cast<uintptr_t>(p->out);
  if (p->q == nullptr || p->k == nullptr || p->v == nullptr || p->out == nullptr || cu_tokens == nullptr || (all & 15u) ||
      ((reinterpret_cast<uintptr_t>(cu_tokens) | reinterpret_cast<uintptr_t>(p->lse)) & 3u))
    return GAAC_EINVAL;
  const int64_t heads[4] = {n_q_heads, n_kv_heads, n_kv_heads, n_q_heads};
  const int64_t tok[4] = {p->q_tok, p->k_tok, p->v_tok, p->out_tok}, head[4] = {p->q_head, p->k_head, p->v_head, p->out_head};
  const void* base[4] = {p->q, p->k, p->v, p->out};
  for (int i = 0; i < 4; ++i) {
    const int64_t st = n_tokens > 1 ? tok[i] : kD, sh = heads[i] > 1 ? head[i] : kD;
    if (st < kD || sh < kD || ((st | sh) & 7) || st > std::min(int64_t{1} << 38, (int64_t{1} << 56) / n_tokens) ||
        sh > (int64_t{1} << 38))
      return GAAC_EINVAL;
  }
  // Heads of one token and tokens of one head of the result are apart, and no input has a part of the results.
  if (n_tokens > 1 && n_q_heads > 1 && tok[3] < static_cast<int64_t>(n_q_heads - 1) * head[3] + kD && head[3] < (n_tokens - 1) * tok[3] + kD)
    return GAAC_EINVAL;
  const PaSpan out(p->out, n_tokens, n_q_heads, p->out_tok, p->out_head);
  const int64_t lse = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p->lse)), lse_end = lse + n_tokens * n_q_heads * 4;
  for (int i = 0; i < 4; ++i) {
    const PaSpan t(base[i], n_tokens, heads[i], tok[i], head[i]);
    if ((i < 3 && !pa_apart(t, out)) || (lse != 0 && lse < t.end && t.at < lse_end)) return GAAC_EINVAL;
  }
  if (tma_encode() == nullptr) return GAAC_ECUDA;
  PaArgs a;
  a.cu = cu_tokens;
  a.batch = batch;
  a.hkv = n_kv_heads;
  a.g = n_q_heads / n_kv_heads;
  a.per = kPaRows / a.g;
  a.g_inverse = 65536 / a.g + 1;
  const int64_t places = n_tokens / (2 * a.per) + batch;
  if (places * n_kv_heads > 0x7FFFFFFF) return GAAC_EINVAL;
  a.places = static_cast<unsigned>(places);
  // The CTAs that run at a time share one kv-head's keys where K and V are more than half of L2 and there are units enough to
  // level out what every head ends with.  One head after the other against all in turn, in % of the time: 4 x 16,384 tokens,
  // 32 / 8 heads, -11 to -16; 32 of 1-4,096, 16 / 8, -6 to -9; 32 of 1-2,048, 16 / 8, -1 to -6; 8 of 1-12,000, 16 / 8, -8 to +6 by
  // their lengths; 1 x 16,384, 32 / 8 (64 MB), within 1.  Less data: 1 x 8,192, 32 / 8, +5 to +9.  Fewer units (of an SM): 8 of
  // 1-5,000, 16 / 8 (7-9), +8 to +12; 8 of 600-10,000, 8 / 8 (7-10), +3 to +10; 1 x 24,576, 16 / 16 (10), +1 to +3.
  a.heads_apart = n_tokens * n_kv_heads * (2 * kD * 2) > kPaApartBytes && places * n_kv_heads >= int64_t{152} * kPaApartUnits;
  a.n_tokens = n_tokens;
  // Not 0, which would make NaN of the masked logits: with the smallest number above it no finite logit moves a weight.
  a.c = scale == 0.f ? 0x1p-149f : static_cast<float>(c);
  a.negate = scale < 0.f;
  a.v = static_cast<const char*>(p->v);
  a.v_tok = p->v_tok * 2;
  a.v_head = p->v_head * 2;
  a.out = static_cast<char*>(p->out);
  a.out_tok = p->out_tok * 2;
  a.out_head = p->out_head * 2;
  a.lse = p->lse;
  a.status = d_status;
  CUtensorMap q, k, v;
  if (!pa_map(&q, p->q, n_tokens, n_q_heads, p->q_tok, p->q_head, a.g, a.per) ||
      !pa_map(&k, p->k, n_tokens, n_kv_heads, p->k_tok, p->k_head, 1, kPaKeys) ||
      !pa_map(&v, p->v, n_tokens, n_kv_heads, p->v_tok, p->v_head, 1, kPaKeys))
    return GAAC_ECUDA;
  const unsigned grid = static_cast<unsigned>(places * n_kv_heads);
  return dtype == GAAC_F16 ? pa_launch<true>(a, q, k, v, grid, stream) : pa_launch<false>(a, q, k, v, grid, stream);
}
