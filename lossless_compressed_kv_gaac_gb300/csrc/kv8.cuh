// Shared pieces of the 8-bit paged cache: argument checks, the device view of a cache, and FP8 conversions.
//
// A block of 64 tokens is a page once it is full: FP8 numbers [kv-head][K|V][64][128] with one scale for each
// (page, kv-head, K|V).  The block that is still open lives in the tail, in the model's type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"

namespace gaac {

struct Kv8Dev {
  uint8_t* pages;
  float* scales;
  uint16_t* tail;
  int32_t* table;
  int32_t* refs;
  int32_t* lens;
  int32_t* work;
  int64_t n_pages;
  int batch, heads, max_blocks;
};

constexpr int kKv8Tile = kBlock * kD;       // FP8 bytes of one (page, kv-head, K|V)
constexpr int kKv8Pair = 2 * kKv8Tile;      // K and V of one (page, kv-head), contiguous
constexpr int kKv8Chunk = 8192;             // pages that one CTA counts (reserve, compact)

// Workspace (int32 words): the append's counters per sequence and the two tickets, which are zero between calls,
// then scratch that every call writes before it reads.
struct Kv8Work {
  int64_t tickets, need, chunks, list_a, list_b, words;
};
__host__ __device__ inline Kv8Work kv8_work(int64_t batch, int64_t n_pages) {
  Kv8Work w;
  w.tickets = batch;
  w.need = w.tickets + 4;
  w.chunks = w.need + batch + 1;
  w.list_a = w.chunks + (n_pages + kKv8Chunk - 1) / kKv8Chunk + 4;
  w.list_b = w.list_a + n_pages;
  w.words = w.list_b + n_pages;
  return w;
}

inline bool kv8_ok(const gaac_kv8* c) {
  if (c == nullptr || c->pages == nullptr || c->scales == nullptr || c->tail == nullptr || c->table == nullptr ||
      c->refs == nullptr || c->seq_lens == nullptr || c->work == nullptr)
    return false;
  if (c->n_pages < 1 || c->batch < 1 || c->batch > 65535 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 ||
      c->max_blocks < 1 || c->max_blocks > (1 << 24))
    return false;
  // rows of 128 numbers are counted in 32 bits by the copy engine's coordinates
  const int64_t rows = int64_t{2} * kBlock * c->n_kv_heads;
  if (c->n_pages > 0x7FFFFFFF / rows || c->batch > 0x7FFFFFFF / rows) return false;
  if ((c->fmt != GAAC_FP8_E4M3 && c->fmt != GAAC_FP8_E5M2) || (c->dtype != GAAC_BF16 && c->dtype != GAAC_F16)) return false;
  const uintptr_t a16 = reinterpret_cast<uintptr_t>(c->pages) | reinterpret_cast<uintptr_t>(c->tail) |
                        reinterpret_cast<uintptr_t>(c->refs) | reinterpret_cast<uintptr_t>(c->work);
  const uintptr_t a4 = reinterpret_cast<uintptr_t>(c->table) | reinterpret_cast<uintptr_t>(c->seq_lens);
  return (a16 & 15u) == 0 && (a4 & 3u) == 0 && (reinterpret_cast<uintptr_t>(c->scales) & 7u) == 0;
}

// gaac_kv8_reserve for appends of n_tokens rows; the cache has been checked.
int kv8_reserve_rows(const gaac_kv8* cache, const int32_t* cu_tokens, int64_t n_tokens, int32_t* d_status, void* stream);

inline Kv8Dev kv8_dev(const gaac_kv8* c) {
  return Kv8Dev{c->pages, c->scales, static_cast<uint16_t*>(c->tail), c->table, c->refs, c->seq_lens, c->work,
                c->n_pages, c->batch, c->n_kv_heads, c->max_blocks};
}

__device__ __forceinline__ unsigned int kv8_atomic_add_acq_rel(int32_t* p, unsigned int v) {
  unsigned int old;
  asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// One launch that may be set up while its predecessor on the stream drains; the kernel waits for it
// (griddepcontrol.wait) before it touches memory.  cluster: CTAs of a thread-block cluster.
template <typename... P, typename... A>
inline int kv8_launch_cluster(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? GAAC_OK : GAAC_ECUDA;
}
template <typename... P, typename... A>
inline int kv8_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, void* stream, A... args) {
  return kv8_launch_cluster(kernel, grid, threads, smem, 1, stream, args...);
}

__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependent_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <bool HALF>
__device__ __forceinline__ float2 kv8_pair(uint32_t w) {  // two 16-bit numbers of the model's type
  if (HALF) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

}  // namespace gaac
