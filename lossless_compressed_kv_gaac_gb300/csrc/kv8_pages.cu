// Pages of the 8-bit cache: reserve, release, fork, reorder, compact.
//
// refs[p] counts the sequences that hold page p; a page with none is free.  There is no free list to keep: the
// lowest free pages are found by counting refs, so every result is a function of the tables alone (no order of
// atomics shows).  Full blocks never change, so a fork shares them by counting and copies only the open block's
// rows; nothing ever has to be copied on a write.
//
// All of it is bound by latency but the moves of a compaction, which are bound by memory.  Measured: release of 8 of
// 32 sequences 1.3 us, fork of as many 4.9 us (one CTA a pair: 8.5 us), reserve without a need 3.8 us (65,536 pages:
// 3.6 us), with 4,096 pages handed to 256 empty sequences 11.6 us; moving 2,000 pages of 8 heads (0.54 GB read and written)
// 77 us, 6.9 TB/s (1,216 CTAs that walk over the moves: 92 us).
#include <algorithm>

#include "kv8.cuh"

namespace gaac {

constexpr int kPgThreads = 1024;
constexpr int kPgPer = kKv8Chunk / kPgThreads;  // pages per thread of a chunk
constexpr unsigned kCompactAlone = 4;           // most chunks that every CTA counts for itself

// Exclusive prefix of x over the CTA's 1024 threads and the total.
__device__ __forceinline__ int block_exclusive(int x, int* total) {
  __shared__ int warp_sum[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  __syncthreads();  // the previous call's readers are done
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int s = warp_sum[lane];
    int t = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, t, d);
      if (lane >= d) t += v;
    }
    warp_sum[lane] = t - s;
    if (lane == 31) warp_sum[32] = t;
  }
  __syncthreads();
  *total = warp_sum[32];
  return warp_sum[warp] + incl - x;
}

// Bit i of the result: page p0 + i (of this thread's kPgPer) is held by a sequence; bits of pages that do not
// exist are clear in both masks.
__device__ __forceinline__ uint32_t held_mask(const int32_t* refs, int64_t p0, int64_t n_pages, uint32_t* exists) {
  uint32_t held = 0, ex = 0;
  if (p0 + kPgPer <= n_pages) {
    int32_t r[kPgPer];
#pragma unroll
    for (int i = 0; i < kPgPer / 4; ++i) {
      const int4 v = reinterpret_cast<const int4*>(refs + p0)[i];
      r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < kPgPer; ++i) held |= (r[i] > 0 ? 1u : 0u) << i;
    ex = (1u << kPgPer) - 1u;
  } else {
    for (int i = 0; i < kPgPer; ++i)
      if (p0 + i < n_pages) {
        ex |= 1u << i;
        held |= (refs[p0 + i] > 0 ? 1u : 0u) << i;
      }
  }
  *exists = ex;
  return held;
}

// This CTA's chunk: counts its free (or held) pages, and says whether it is the last CTA to do so (kLast), and whether a
// thread of any CTA came with `bad` (kLastBad).  What the CTA's threads have written before is visible to the last one.
enum { kNotLast, kLast, kLastBad };
__device__ __forceinline__ int count_chunk(const Kv8Dev& c, const Kv8Work& w, bool free_ones, int32_t* ticket, bool bad = false) {
  constexpr int kBad = 1 << 16;  // beside a chunk's count in a sum over threads, and beside the count of CTAs in the ticket
  static_assert(kKv8Chunk < kBad, "a chunk's count below the mark");
  __shared__ int last;
  uint32_t ex;
  const uint32_t held = held_mask(c.refs, static_cast<int64_t>(blockIdx.x) * kKv8Chunk + threadIdx.x * kPgPer, c.n_pages, &ex);
  int total;
  block_exclusive(__popc(free_ones ? ex & ~held : held) + (bad ? kBad : 0), &total);
  if (threadIdx.x == 0) {
    c.work[w.chunks + blockIdx.x] = total % kBad;
    const unsigned add = total >= kBad ? kBad + 1u : 1u, sum = kv8_atomic_add_acq_rel(ticket, add) + add;
    last = sum % kBad != gridDim.x ? kNotLast : sum >= kBad ? kLastBad : kLast;  // at most 2^11 CTAs
    if (last != kNotLast) *ticket = 0;
  }
  __syncthreads();
  return last;
}

// Blocks of sequence b that the next tokens fill: [lo, hi).  false: the lengths are not valid.  bad: nor are the offsets
// of `rows` rows, with which the append refuses the whole call.
__device__ __forceinline__ bool fill_range(const Kv8Dev& c, const int32_t* cu, int b, int* lo, int* hi, int64_t rows, bool* bad) {
  const int len = c.lens[b];
  const int64_t from = cu == nullptr ? 0 : cu[b], to = cu == nullptr ? 1 : cu[b + 1], n = to - from;
  const int64_t now = len + n;
  *lo = *hi = 0;
  *bad = from < 0 || n < 0 || to > rows;
  if (len < 0 || n < 0 || now > static_cast<int64_t>(c.max_blocks) * kBlock) return false;
  *lo = len / kBlock;
  *hi = static_cast<int>(now / kBlock);
  return true;
}

// For sequences b, b + step, ... (at most 32, one a lane, with blocks [lo, hi) each): visit(k, i, miss) for every 32
// blocks i .. of the k-th one, miss: this lane's block is there and has no page.  The first table entries of eight
// sequences are fetched at a time.
template <typename F>
__device__ __forceinline__ void for_missing(const Kv8Dev& c, int b, int step, int lo, int hi, F visit) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 31;
  uint32_t todo = __ballot_sync(kAll, hi > lo);
  while (todo != 0u) {
    int k[kAhead], entry[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      k[j] = todo ? __ffs(todo) - 1 : -1;
      todo &= todo - 1u;
      const int l = __shfl_sync(kAll, lo, max(k[j], 0)), h = __shfl_sync(kAll, hi, max(k[j], 0));
      entry[j] = k[j] >= 0 && l + lane < h ? c.table[static_cast<int64_t>(b + k[j] * step) * c.max_blocks + l + lane] : 0;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k[j] < 0) break;
      const int l = __shfl_sync(kAll, lo, k[j]), h = __shfl_sync(kAll, hi, k[j]);
      visit(k[j], l, entry[j] < 0);
      const int32_t* row = c.table + static_cast<int64_t>(b + k[j] * step) * c.max_blocks;
      for (int i = l + 32; i < h; i += 32) visit(k[j], i, i + lane < h && row[i + lane] < 0);
    }
  }
}

// Entries without a page among the blocks that fill, in order of sequence and block, get the lowest free pages
// in order.  Every CTA counts the free pages of its chunk and the missing entries of some sequences, a warp each; the
// last one to finish ranks them, lists the pages and hands them out, unless some CTA has found offsets that the append
// of `rows` rows would refuse as a whole.
__global__ void __launch_bounds__(kPgThreads) kv8_reserve_kernel(Kv8Dev c, const int32_t* cu, int64_t rows, int32_t* status) {
  __shared__ int sh_free;
  dependent_wait();
  dependent_launch();
  const Kv8Work w = kv8_work(c.batch, c.n_pages);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* need = c.work + w.need;
  const int warps = gridDim.x * (kPgThreads / 32);
  bool bad = false;
  for (int b0 = blockIdx.x * (kPgThreads / 32) + warp; b0 < c.batch; b0 += 32 * warps) {
    int lo = 0, hi = 0, mine = 0;
    const int64_t b = b0 + static_cast<int64_t>(lane) * warps;
    bool odd = false;
    if (b < c.batch && !fill_range(c, cu, static_cast<int>(b), &lo, &hi, rows, &odd)) report(status, GAAC_EINVAL);
    bad = bad || odd;
    for_missing(c, b0, warps, lo, hi, [&](int k, int, bool miss) {
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, miss));
      if (lane == k) mine += n;
    });
    if (b < c.batch) need[b] = mine;
  }
  const int last = count_chunk(c, w, true, c.work + w.tickets, bad);
  if (last != kLast) {
    if (last == kLastBad && tid == 0) report(status, GAAC_EINVAL);
    return;
  }
  // ---- the rank of each sequence's first one
  int total = 0;
  for (int b0 = 0; b0 < c.batch; b0 += kPgThreads) {
    const int x = b0 + tid < c.batch ? __ldcg(need + b0 + tid) : 0;
    int sum;
    const int at = total + block_exclusive(x, &sum);
    if (b0 + tid < c.batch) need[b0 + tid] = at;
    total += sum;
  }
  if (total == 0) return;
  // this warp's first sequences, under way while the pages are listed
  int lo0 = 0, hi0 = 0;
  if (warp + lane * (kPgThreads / 32) < c.batch) fill_range(c, cu, warp + lane * (kPgThreads / 32), &lo0, &hi0, rows, &bad);
  // ---- the lowest free pages, as many as are lacking
  int32_t* list = c.work + w.list_a;
  int found = 0;
  for (unsigned ch = 0; ch < gridDim.x && found < total; ++ch) {
    if (tid == 0) sh_free = __ldcg(c.work + w.chunks + ch);
    __syncthreads();
    const int n_free = sh_free;
    __syncthreads();
    if (n_free == 0) continue;
    const int64_t p0 = static_cast<int64_t>(ch) * kKv8Chunk + tid * kPgPer;
    uint32_t ex;
    const uint32_t held = held_mask(c.refs, p0, c.n_pages, &ex);
    uint32_t m = ex & ~held;
    int sum, r = found + block_exclusive(__popc(m), &sum);
    while (m != 0u && r < total) {
      list[r++] = static_cast<int32_t>(p0 + __ffs(m) - 1);
      m &= m - 1u;
    }
    found += sum;
  }
  if (found < total && tid == 0) report(status, GAAC_EPOOL);
  __syncthreads();
  // ---- into the table
  for (int b0 = warp; b0 < c.batch; b0 += 32 * (kPgThreads / 32)) {
    int lo = lo0, hi = hi0, rank = 0;
    const int b = b0 + lane * (kPgThreads / 32);
    if (b0 != warp) {
      lo = hi = 0;
      if (b < c.batch) fill_range(c, cu, b, &lo, &hi, rows, &bad);
    }
    if (b < c.batch) rank = need[b];
    for_missing(c, b0, kPgThreads / 32, lo, hi, [&](int k, int i, bool miss) {
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, miss);
      const int at = __shfl_sync(0xFFFFFFFFu, rank, k) + __popc(m & ((1u << lane) - 1u));
      if (miss && at < found) {
        const int32_t p = list[at];
        c.table[static_cast<int64_t>(b0 + k * (kPgThreads / 32)) * c.max_blocks + i + lane] = p;
        c.refs[p] = 1;
      }
      if (lane == k) rank += __popc(m);
    });
  }
}

constexpr int kRelThreads = 256;

// One CTA per listed sequence.  A sequence listed twice is released once: whoever takes an entry out of the
// table gives its page back.
__global__ void __launch_bounds__(kRelThreads) kv8_release_kernel(Kv8Dev c, const int32_t* seqs, int32_t* status) {
  dependent_wait();
  dependent_launch();
  const int b = seqs[blockIdx.x];
  if (b < 0 || b >= c.batch) {
    if (threadIdx.x == 0) report(status, GAAC_EINVAL);
    return;
  }
  int32_t* row = c.table + static_cast<int64_t>(b) * c.max_blocks;
  for (int i = threadIdx.x; i < c.max_blocks; i += kRelThreads) {
    if (row[i] == -1) continue;
    const int32_t p = atomicExch(row + i, -1);
    if (p == -1) continue;
    if (p < 0 || p >= c.n_pages) {
      report(status, GAAC_EFORMAT);
    } else if (atomicSub(c.refs + p, 1) <= 0) {
      atomicAdd(c.refs + p, 1);
      report(status, GAAC_EFORMAT);
    }
  }
  if (threadIdx.x == 0) c.lens[b] = 0;
}

constexpr int kFkThreads = 512;
constexpr int kFkCtas = 8;  // a cluster for each pair

// One cluster per pair (src, dst).  A pair is refused as a whole (and reported) when an index is out of range, dst is
// not empty, dst is listed before, src is the dst of some pair, or src's own row is not valid.  Every CTA of the
// cluster checks; none writes before all have (the cluster's barrier), since what is written is what is checked.
__global__ void __launch_bounds__(kFkThreads) kv8_fork_kernel(Kv8Dev c, const int32_t* src, const int32_t* dst, int n,
                                                              int32_t* status) {
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x, i = blockIdx.x / kFkCtas, part = blockIdx.x % kFkCtas;
  const int s = src[i], d = dst[i];
  const bool in = s >= 0 && s < c.batch && d >= 0 && d < c.batch;
  int bad = !in, odd = 0, len = 0;
  const int32_t* from = c.table + (in ? static_cast<int64_t>(s) * c.max_blocks : 0);
  int32_t* to = c.table + (in ? static_cast<int64_t>(d) * c.max_blocks : 0);
  if (in) {
    len = c.lens[s];
    if (c.lens[d] != 0) bad = 1;
    for (int j = tid; j < n; j += kFkThreads)
      if (dst[j] == s || (j < i && dst[j] == d)) bad = 1;
    for (int k = tid; k < c.max_blocks; k += kFkThreads)
      if (to[k] != -1) bad = 1;
    if (len < 0 || len > static_cast<int64_t>(c.max_blocks) * kBlock) {
      odd = 1;
    } else {
      for (int k = tid; k < len / kBlock; k += kFkThreads)
        if (from[k] < 0 || from[k] >= c.n_pages) odd = 1;
    }
  }
  bad = __syncthreads_or(bad);
  odd = __syncthreads_or(odd);
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (bad || odd) {
    if (tid == 0 && part == 0) report(status, bad ? GAAC_EINVAL : GAAC_EFORMAT);
    return;
  }
  const int full = len / kBlock, open = len % kBlock;
  for (int k = part * kFkThreads + tid; k < full; k += kFkCtas * kFkThreads) {
    const int32_t p = from[k];
    to[k] = p;
    atomicAdd(c.refs + p, 1);
  }
  // open rows of every (kv-head, K|V): 16 vectors of 16 bytes each
  constexpr int kRow = kD / 8;
  const uint4* ts = reinterpret_cast<const uint4*>(c.tail) + static_cast<int64_t>(s) * c.heads * 2 * kBlock * kRow;
  uint4* td = reinterpret_cast<uint4*>(c.tail) + static_cast<int64_t>(d) * c.heads * 2 * kBlock * kRow;
  const int per = open * kRow, all = per * 2 * c.heads;
#pragma unroll 4
  for (int k = part * kFkThreads + tid; k < all; k += kFkCtas * kFkThreads) {
    const int at = k / per * (kBlock * kRow) + k % per;
    td[at] = ts[at];
  }
  if (tid == 0 && part == 0) c.lens[d] = len;
}

// ------------------------------------------------------------------ reorder
// Sequence g * beams + i becomes what g * beams + parents[g][i] was.  A thread takes one place (a column of the table,
// 16 bytes of an open row) of all the beams of a group: it has read every beam's old value before it writes the first
// new one, so the exchange needs no second copy of anything.  BEAMS: the beams at most.  32 searches of 8 beams, rows of 512
// pages, open blocks of 8 heads half full, 59 MB moved: 11.0 us in a graph, 5.4 TB/s (13.4-14.6 us one by one; then eight
// or sixteen CTAs an SM in place of four 15.5 and 17.1 us, table and open rows by the same CTAs 15.4-16.7).  4 searches of 4: 3.9 us.

constexpr int kRoThreads = 128;

template <int BEAMS>
__global__ void __launch_bounds__(kRoThreads) kv8_reorder_kernel(Kv8Dev c, const int32_t* parents, int beams, unsigned table_parts,
                                                                 unsigned parts, int32_t* status) {
  __shared__ int parent[BEAMS], len[BEAMS];  // len: what a sequence becomes; -1 where it stays as it is
  dependent_wait();
  dependent_launch();
  const int tid = threadIdx.x;
  const int64_t group = blockIdx.x / parts, first = group * beams;
  const unsigned part = blockIdx.x % parts;
  if (tid < beams) {
    const int p = parents[first + tid];
    const bool in = p >= 0 && p < beams;
    const int n = in ? c.lens[first + p] : 0;
    const bool fits = n >= 0 && n <= static_cast<int64_t>(c.max_blocks) * kBlock;
    if (part == 0 && (!in || !fits)) report(status, in ? GAAC_EFORMAT : GAAC_EINVAL);
    parent[tid] = in ? p : tid;
    len[tid] = in && fits && p != tid ? n : -1;
  }
  __syncthreads();
  int most = 0;  // open rows
  for (int i = 0; i < beams; ++i) most = max(most, len[i] % kBlock);
  // ---- tables and counts, by the first CTAs: a sequence gives up its old row and holds its parent's full blocks
  for (int64_t col = part * kRoThreads + tid; part < table_parts && col < c.max_blocks; col += table_parts * kRoThreads) {
    int32_t was[BEAMS], now[BEAMS];
#pragma unroll
    for (int i = 0; i < BEAMS; ++i)
      if (i < beams) was[i] = c.table[(first + i) * c.max_blocks + col];
#pragma unroll
    for (int i = 0; i < BEAMS; ++i)
      if (i < beams) now[i] = len[i] < 0 ? was[i] : col < len[i] / kBlock ? c.table[(first + parent[i]) * c.max_blocks + col] : -1;
#pragma unroll
    for (int i = 0; i < BEAMS; ++i)
      if (i < beams && len[i] >= 0) {
        const bool held = now[i] >= 0 && now[i] < c.n_pages;
        if (!held && col < len[i] / kBlock) report(status, GAAC_EFORMAT);
        if (now[i] != was[i]) {
          if (was[i] >= 0 && was[i] < c.n_pages) atomicSub(c.refs + was[i], 1);
          if (held) atomicAdd(c.refs + now[i], 1);
          c.table[(first + i) * c.max_blocks + col] = now[i];
        }
      }
  }
  // ---- open rows of every (kv-head, K|V), by the others: 16 vectors of 16 bytes each
  constexpr int kRow = kD / 8;
  uint4* const tail = reinterpret_cast<uint4*>(c.tail);
  const int64_t seq = static_cast<int64_t>(c.heads) * 2 * kBlock * kRow;
  const unsigned per = most * kRow, all = per * 2 * c.heads;
  for (unsigned k = (part - table_parts) * kRoThreads + tid; part >= table_parts && k < all; k += (parts - table_parts) * kRoThreads) {
    const unsigned in = k % per;
    uint4* const t = tail + first * seq + k / per * (kBlock * kRow) + in;
    const int row = in / kRow;
    uint4 x[BEAMS];
#pragma unroll
    for (int i = 0; i < BEAMS; ++i)
      if (i < beams && row < len[i] % kBlock) x[i] = t[parent[i] * seq];
#pragma unroll
    for (int i = 0; i < BEAMS; ++i)
      if (i < beams && row < len[i] % kBlock) t[i * seq] = x[i];
  }
  // ---- the lengths change once every CTA of the group has read them
  if (tid == 0 && kv8_atomic_add_acq_rel(c.work + first, 1u) == parts - 1) {
    c.work[first] = 0;
    for (int i = 0; i < beams; ++i)
      if (len[i] >= 0) c.lens[first + i] = len[i];
  }
}

// ------------------------------------------------------------------ compact
// With n held pages, the held pages at n and above move into the holes below n: the lowest hole takes the highest
// page, and so on.  Source and target never overlap.
//   1. (pools of more than kCompactAlone chunks) every CTA counts the held pages of its chunk; the last one makes the
//      counts prefixes
//   2. holes and movers into two lists by rank; moved_to of the pages that stay
//   3. contents, counts and the table

__global__ void __launch_bounds__(kPgThreads) kv8_compact_count_kernel(Kv8Dev c) {
  dependent_wait();
  dependent_launch();
  const Kv8Work w = kv8_work(c.batch, c.n_pages);
  if (count_chunk(c, w, false, c.work + w.tickets + 1) == kNotLast) return;
  int run = 0;
  for (unsigned c0 = 0; c0 < gridDim.x; c0 += kPgThreads) {
    const unsigned ch = c0 + threadIdx.x;
    const int x = ch < gridDim.x ? __ldcg(c.work + w.chunks + ch) : 0;
    int sum;
    const int at = run + block_exclusive(x, &sum);
    if (ch < gridDim.x) c.work[w.chunks + ch] = at;
    run += sum;
  }
  if (threadIdx.x == 0) {
    c.work[w.chunks + gridDim.x] = run;  // held pages
    if (run == c.n_pages) c.work[w.tickets + 2] = 0;  // nothing moves; otherwise step 2 says how many do
  }
}

// ALONE: no counts from step 1; every CTA counts the whole pool itself, which for a few chunks is quicker than a
// launch more.
template <bool ALONE>
__global__ void __launch_bounds__(kPgThreads) kv8_compact_list_kernel(Kv8Dev c, int32_t* moved_to) {
  dependent_wait();
  dependent_launch();
  const Kv8Work w = kv8_work(c.batch, c.n_pages);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kKv8Chunk + threadIdx.x * kPgPer;
  uint32_t ex;
  const uint32_t held = held_mask(c.refs, p0, c.n_pages, &ex);
  int sum, in_chunk = block_exclusive(__popc(held), &sum);
  int64_t held_all;
  int before;
  if (ALONE) {
    int earlier = 0, all = 0, total;
    for (unsigned ch = 0; ch < gridDim.x; ++ch) {
      uint32_t e;
      const int n = ch == blockIdx.x ? __popc(held)
                                     : __popc(held_mask(c.refs, static_cast<int64_t>(ch) * kKv8Chunk + threadIdx.x * kPgPer, c.n_pages, &e));
      all += n;
      if (ch < blockIdx.x) earlier += n;
    }
    if (gridDim.x > 1) {
      block_exclusive(earlier, &before);
      block_exclusive(all, &total);
    } else {
      before = 0;
      total = sum;
    }
    held_all = total;
    if (blockIdx.x == 0 && threadIdx.x == 0 && held_all == c.n_pages) c.work[w.tickets + 2] = 0;
  } else {
    held_all = c.work[w.chunks + gridDim.x];
    before = c.work[w.chunks + blockIdx.x];
  }
  before += in_chunk;
  int32_t* holes = c.work + w.list_a;
  int32_t* movers = c.work + w.list_b;
#pragma unroll
  for (int i = 0; i < kPgPer; ++i) {
    if (!((ex >> i) & 1u)) continue;
    const int64_t p = p0 + i;
    const bool h = (held >> i) & 1u;
    if (p == held_all) c.work[w.tickets + 2] = static_cast<int32_t>(held_all) - before;  // pages that move
    int32_t to = h ? static_cast<int32_t>(p) : -1;
    if (h && p >= held_all) {
      const int rank = static_cast<int>(held_all) - 1 - before;
      movers[rank] = static_cast<int32_t>(p);
      to = -2 - rank;  // the hole of that rank, known when every list is written
    } else if (!h && p < held_all) {
      holes[p - before] = static_cast<int32_t>(p);
    }
    moved_to[p] = to;
    before += h;
  }
}

constexpr int kMvThreads = 256;
constexpr int kMvCtasPerSm = 8;
constexpr int kMvMost = 152 * 64;

// A CTA copies one (page, kv-head) at a time, 16 KB with four 16-byte loads a thread in flight; where the next one
// lies is fetched meanwhile.
__global__ void __launch_bounds__(kMvThreads, kMvCtasPerSm) kv8_compact_move_kernel(Kv8Dev c, int32_t* moved_to) {
  dependent_wait();
  dependent_launch();
  const Kv8Work w = kv8_work(c.batch, c.n_pages);
  const int32_t* holes = c.work + w.list_a;
  const int32_t* movers = c.work + w.list_b;
  const int tid = threadIdx.x;
  const unsigned heads = c.heads, items = static_cast<unsigned>(c.work[w.tickets + 2]) * heads;  // below 2^24
  unsigned it = blockIdx.x;
  int64_t from = 0, to = 0;
  if (it < items) {
    from = movers[it / heads];
    to = holes[it / heads];
  }
  while (it < items) {
    const unsigned h = it % heads;
    const uint4* s = reinterpret_cast<const uint4*>(c.pages + (from * c.heads + h) * kKv8Pair);
    uint4* d = reinterpret_cast<uint4*>(c.pages + (to * c.heads + h) * kKv8Pair);
    uint4 x[kKv8Pair / 16 / kMvThreads];
#pragma unroll
    for (int i = 0; i < kKv8Pair / 16 / kMvThreads; ++i) x[i] = __ldcs(s + tid + kMvThreads * i);
    const unsigned next = it + gridDim.x;
    int64_t from2 = 0, to2 = 0;
    if (next < items) {
      from2 = movers[next / heads];
      to2 = holes[next / heads];
    }
    if (tid == 0) {
      reinterpret_cast<float2*>(c.scales)[to * c.heads + h] = reinterpret_cast<const float2*>(c.scales)[from * c.heads + h];
      if (h == 0) {
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
        moved_to[from] = static_cast<int32_t>(to);
      }
    }
#pragma unroll
    for (int i = 0; i < kKv8Pair / 16 / kMvThreads; ++i) __stcs(d + tid + kMvThreads * i, x[i]);
    it = next;
    from = from2;
    to = to2;
  }
  // The table.  moved_to of a page that moves may or may not have been replaced above yet: both forms say the same.
  const int64_t entries = static_cast<int64_t>(c.batch) * c.max_blocks;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMvThreads + tid; i < entries; i += static_cast<int64_t>(gridDim.x) * kMvThreads) {
    const int32_t p = c.table[i];
    if (p < 0 || p >= c.n_pages) continue;
    int32_t q = *reinterpret_cast<volatile int32_t*>(moved_to + p);
    if (q <= -2) q = holes[-2 - q];
    if (q != p) c.table[i] = q;
  }
}

}  // namespace gaac

using namespace gaac;

static unsigned chunks_of(const gaac_kv8* c) { return static_cast<unsigned>((c->n_pages + kKv8Chunk - 1) / kKv8Chunk); }

int gaac::kv8_reserve_rows(const gaac_kv8* cache, const int32_t* cu_tokens, int64_t n_tokens, int32_t* d_status, void* stream) {
  return kv8_launch(kv8_reserve_kernel, dim3(chunks_of(cache)), kPgThreads, 0, stream, kv8_dev(cache), cu_tokens, n_tokens, d_status);
}

extern "C" int gaac_kv8_reserve(const gaac_kv8* cache, const int32_t* cu_tokens, int32_t* d_status, void* stream) {
  if (!kv8_ok(cache) || (reinterpret_cast<uintptr_t>(cu_tokens) & 3u)) return GAAC_EINVAL;
  return kv8_reserve_rows(cache, cu_tokens, 0x7FFFFFFF, d_status, stream);
}

extern "C" int gaac_kv8_release(const gaac_kv8* cache, const int32_t* seqs, int n, int32_t* d_status, void* stream) {
  if (!kv8_ok(cache) || n < 0) return GAAC_EINVAL;
  if (n == 0) return GAAC_OK;
  if (seqs == nullptr || (reinterpret_cast<uintptr_t>(seqs) & 3u)) return GAAC_EINVAL;
  return kv8_launch(kv8_release_kernel, dim3(n), kRelThreads, 0, stream, kv8_dev(cache), seqs, d_status);
}

extern "C" int gaac_kv8_fork(const gaac_kv8* cache, const int32_t* src, const int32_t* dst, int n, int32_t* d_status,
                             void* stream) {
  if (!kv8_ok(cache) || n < 0 || n > cache->batch) return GAAC_EINVAL;
  if (n == 0) return GAAC_OK;
  if (src == nullptr || dst == nullptr || ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 3u))
    return GAAC_EINVAL;
  return kv8_launch_cluster(kv8_fork_kernel, dim3(kFkCtas * n), kFkThreads, 0, kFkCtas, stream, kv8_dev(cache), src, dst, n,
                            d_status);
}

extern "C" int gaac_kv8_reorder(const gaac_kv8* cache, const int32_t* parents, int beams, int32_t* d_status, void* stream) {
  if (!kv8_ok(cache) || parents == nullptr || (reinterpret_cast<uintptr_t>(parents) & 3u) || beams < 1 || beams > GAAC_MAX_BEAMS ||
      cache->batch % beams != 0)
    return GAAC_EINVAL;
  if (beams == 1) return GAAC_OK;  // nothing has another parent
  // CTAs of a group: those that its table columns fill and those that its open rows may, up to four of either kind for each SM
  const int groups = cache->batch / beams;
  const int64_t most = std::max<int64_t>(1, (152 * 4 + groups - 1) / groups);
  auto ctas = [&](int64_t places) { return static_cast<unsigned>(std::min(most, (places + kRoThreads - 1) / kRoThreads)); };
  const unsigned table_parts = ctas(cache->max_blocks), parts = table_parts + ctas(int64_t{2} * cache->n_kv_heads * (kBlock - 1) * (kD / 8));
  const dim3 grid(parts * groups);
  const Kv8Dev c = kv8_dev(cache);
  if (beams <= 4) return kv8_launch(kv8_reorder_kernel<4>, grid, kRoThreads, 0, stream, c, parents, beams, table_parts, parts, d_status);
  if (beams <= 8) return kv8_launch(kv8_reorder_kernel<8>, grid, kRoThreads, 0, stream, c, parents, beams, table_parts, parts, d_status);
  if (beams <= 16) return kv8_launch(kv8_reorder_kernel<16>, grid, kRoThreads, 0, stream, c, parents, beams, table_parts, parts, d_status);
  return kv8_launch(kv8_reorder_kernel<32>, grid, kRoThreads, 0, stream, c, parents, beams, table_parts, parts, d_status);
}

extern "C" int gaac_kv8_compact(const gaac_kv8* cache, int32_t* moved_to, void* stream) {
  if (!kv8_ok(cache) || moved_to == nullptr || (reinterpret_cast<uintptr_t>(moved_to) & 3u)) return GAAC_EINVAL;
  const Kv8Dev c = kv8_dev(cache);
  const unsigned chunks = chunks_of(cache);
  int e;
  if (chunks <= kCompactAlone) {
    e = kv8_launch(kv8_compact_list_kernel<true>, dim3(chunks), kPgThreads, 0, stream, c, moved_to);
  } else {
    e = kv8_launch(kv8_compact_count_kernel, dim3(chunks), kPgThreads, 0, stream, c);
    if (e == GAAC_OK) e = kv8_launch(kv8_compact_list_kernel<false>, dim3(chunks), kPgThreads, 0, stream, c, moved_to);
  }
  // At most half the pages move: a CTA for each (page, kv-head) of those, up to kMvMost.
  const int64_t most = (c.n_pages / 2 + 1) * c.heads;
  if (e == GAAC_OK)
    e = kv8_launch(kv8_compact_move_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(most, kMvMost))), kMvThreads, 0, stream, c, moved_to);
  return e;
}
