// kv_attn.cu — attention over the paged INT8 cache (shn_kv_attn_prompt, shn_kv_attn_shared).
//
// One warp per query and head: a lane holds D/32 of the query's values and of the output; one pass
// over the keys with the running maximum and sum of the softmax, all in float32.
#include "kv_internal.cuh"

namespace shn {
namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) kv_attn_simple_kernel(KvPages c, KvAttnArgs a) {
  constexpr int E = D / 32;
  const uint64_t item = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const uint32_t lane = threadIdx.x & 31;
  if (item >= (uint64_t)a.n_tokens * a.q_heads) return;
  const uint32_t row = (uint32_t)(item / a.q_heads), head = (uint32_t)(item % a.q_heads);
  const uint32_t hk = head / (a.q_heads / c.kv_heads);
  // the request of this row, and how many tokens the row sees
  uint32_t r = row;
  int64_t seen;
  const int64_t holds = (int64_t)a.max_blocks << c.log2_pt;
  if (a.cu_q) {
    for (r = 0; r < a.n_reqs; ++r) {
      const int64_t b = a.cu_q[r], e = a.cu_q[r + 1];
      if (b < 0 || e < b || e > (int64_t)a.n_tokens) {
        if (lane == 0) report(a.st, SHN_ERR_INVALID_ARG, r);
      } else if (row >= b && row < e) {
        break;
      }
    }
    if (r == a.n_reqs) return;
  }
  int64_t len = a.kv_len[r];
  if (len < 0 || len > holds) {
    int64_t most = holds;
    if (a.prefix_len) {
      // a row may be shorter than its prefix
      const int64_t pl = min((int64_t)max(0, *a.prefix_len), (int64_t)a.n_prefix_pages << c.log2_pt);
      most = max(most, pl);
    }
    if (len < 0 || len > most) {
      if (lane == 0) report(a.st, SHN_ERR_INVALID_ARG, r);
      len = len < 0 ? 0 : most;
    }
  }
  seen = a.cu_q ? len - (a.cu_q[r + 1] - a.cu_q[r]) + (row - a.cu_q[r]) + 1 : len;
  int64_t prefix = 0;
  if (a.prefix_len) {
    prefix = *a.prefix_len;
    const int64_t most = (int64_t)a.n_prefix_pages << c.log2_pt;
    if (prefix < 0 || prefix > most) {
      if (lane == 0) report(a.st, SHN_ERR_INVALID_ARG, 0);
      prefix = prefix < 0 ? 0 : most;
    }
  }
  float q[E], o[E], m = -INFINITY, l = 0.f;
  const uint16_t* src = a.q + (uint64_t)row * a.q_stride + (uint64_t)head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __uint_as_float((uint32_t)src[e] << 16), o[e] = 0.f;
  for (int64_t j = 0; j < seen; ++j) {
    const uint32_t b = (uint32_t)(j >> c.log2_pt);
    const int32_t p = j < prefix ? a.prefix_pages[b] : a.table[(uint64_t)r * a.max_blocks + b];
    float s = 0.f, vs = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
    if (p < 0 || (uint32_t)p >= c.n_pages) {
      if (lane == 0) report(a.st, SHN_ERR_INVALID_ARG, r);
    } else {
      const uint64_t at = kv_row(c, (uint32_t)p, hk, (uint32_t)j & ((1u << c.log2_pt) - 1));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s = fmaf(q[e], (float)c.k[at * D + lane * E + e], s);
        v[e] = (float)c.v[at * D + lane * E + e];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      s *= c.k_scale[at] * a.scale;
      vs = c.v_scale[at];
    }
    const float top = fmaxf(m, s);
    const float keep = top == -INFINITY ? 1.f : __expf(m - top), w = top == -INFINITY ? 0.f : __expf(s - top);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w * vs, v[e], o[e] * keep);
    m = top;
  }
  uint16_t* dst = a.out + (uint64_t)row * a.out_stride + (uint64_t)head * D + lane * E;
  const float inv = l > 0.f ? 1.f / l : (seen > 0 ? 1.f / l : 0.f);
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = (uint16_t)bf16_pack(o[e] * inv, 0.f);
}

}  // namespace

cudaError_t launch_kv_attn(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, cudaStream_t s) {
  const uint64_t warps = (uint64_t)a.n_tokens * a.q_heads;
  const uint64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (head_dim == 128) kv_attn_simple_kernel<128><<<(uint32_t)blocks, kThreads, 0, s>>>(c, a);
  else kv_attn_simple_kernel<64><<<(uint32_t)blocks, kThreads, 0, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace shn
