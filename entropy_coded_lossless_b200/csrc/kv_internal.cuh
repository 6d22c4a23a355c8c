// kv_internal.cuh — what the kernels of the paged KV cache (include/shn_kv.h) share.
#pragma once

#include <cuda_bf16.h>

#include "../../include/shn_kv.h"
#include "shn_internal.cuh"

namespace shn {

// The cache as kernels take it.
struct KvPages {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  uint32_t n_pages;
  uint32_t kv_heads;
  uint32_t log2_pt;  // log2(page_tokens)
};

// Row (head h) of a slot, in rows of head_dim values: also the index of its scale. Slots stay below
// 2^31, rows can pass 2^32.
__device__ __forceinline__ uint64_t kv_row(const KvPages& c, uint32_t page, uint32_t h, uint32_t t_in_page) {
  return (((uint64_t)page * c.kv_heads + h) << c.log2_pt) + t_in_page;
}
__device__ __forceinline__ uint64_t kv_row_of_slot(const KvPages& c, uint32_t slot, uint32_t h) {
  return kv_row(c, slot >> c.log2_pt, h, slot & ((1u << c.log2_pt) - 1));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// (lo, hi) rounded to nearest even, packed
__device__ __forceinline__ uint32_t bf16_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// An error into the status, which is 0 before: of several of one kind the first request's (token's) stays, whoever comes
// first, and a wait that gave up stands above what is wrong with the input.
__device__ __forceinline__ void report_first(DeviceStatus* st, uint32_t code, uint32_t detail) {
  unsigned long long *word = reinterpret_cast<unsigned long long*>(st), old = 0;
  const unsigned long long mine = code | (unsigned long long)detail << 32;
  for (;;) {
    const unsigned long long now = atomicCAS(word, old, mine);
    if (now == old) return;
    const uint32_t is = (uint32_t)now;
    if (is == code ? (uint32_t)(now >> 32) <= detail : is != 0 && code != SHN_ERR_TIMEOUT) return;
    old = now;
  }
}

// A call's first kernel is launched as any other; the next ones are launched so that they start while the one before still
// runs (programmatic dependent launch) and hide their start behind it. A kernel launched so reads nothing that the one
// before writes, and writes nothing that it reads, until after_previous(); let_next() lets the one after it start.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_behind_in_clusters(void (*kernel)(P...), uint32_t cluster, dim3 grid, uint32_t threads, size_t smem, cudaStream_t s,
                                      const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_first(void (*kernel)(P...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t s, const A&... args) {
  kernel<<<grid, threads, smem, s>>>(P(args)...);
  return cudaGetLastError();
}
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t s, const A&... args) {
  return launch_behind_in_clusters(kernel, 1, grid, threads, smem, s, args...);
}
cudaError_t launch_kv_begin(DeviceStatus* st, cudaStream_t s);

struct KvPlanArgs {
  const int32_t *ctx, *fresh;
  uint32_t n, log2_pt, max_blocks, n_free, max_tokens;
  int32_t* table;
  const int32_t *free_pages, *free_head;
  int32_t *free_next, *cu, *kv_len, *positions, *slots;
  DeviceStatus* st;
};
cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t s);

struct KvStoreArgs {
  const uint16_t *q, *k, *v;
  uint64_t q_stride, k_stride, v_stride;
  uint32_t q_heads, n_tokens;
  const int32_t *positions, *slots;
  const uint16_t *q_weight, *k_weight;
  float eps;
  const float* cos_sin;
  uint32_t n_positions, rot, pairs;
  uint16_t* q_out;
  uint64_t q_out_stride;
  DeviceStatus* st;
};
cudaError_t launch_kv_store(const KvPages& c, uint32_t head_dim, const KvStoreArgs& a, int sm_count, cudaStream_t s);

struct KvLoadArgs {
  const int32_t* slots;
  uint32_t n_tokens;
  uint16_t *k_out, *v_out;
  uint64_t k_stride, v_stride;
  DeviceStatus* st;
};
cudaError_t launch_kv_load(const KvPages& c, uint32_t head_dim, const KvLoadArgs& a, cudaStream_t s);

// Both attention calls. cu_q is null for single tokens (request r has query r).
struct KvAttnArgs {
  const uint16_t* q;
  uint64_t q_stride;
  uint32_t n_tokens, q_heads;
  const int32_t* table;
  uint32_t max_blocks;
  const int32_t *cu_q, *kv_len;
  uint32_t n_reqs;
  const int32_t* prefix_pages;  // null: no prefix
  uint32_t n_prefix_pages;
  const int32_t* prefix_len;
  float scale;
  uint16_t* out;
  uint64_t out_stride;
  DeviceStatus* st;
};
cudaError_t launch_kv_prompt(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, int sm_count, cudaStream_t s);

}  // namespace shn
