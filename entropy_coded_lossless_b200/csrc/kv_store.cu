// kv_store.cu — a step's queries, keys and values through norm and rotation, keys and values quantised
// into their pages (shn_kv_store), and rows of the pages back as bf16 (shn_kv_load).
#include "kv_internal.cuh"

namespace shn {
namespace {

__global__ void kv_begin_kernel(DeviceStatus* st) {
  let_next();
  if (threadIdx.x == 0) st->status = 0, st->detail = 0;
}

// ---- shn_kv_store -------------------------------------------------------------------------------
// HBM-bound: every value is read and written once and costs about ten operations. A head row of D values
// is held by D/8 lanes, 8 values (16 bytes) each, so that a row's sum of squares and its largest
// magnitude are four shuffles away and a rotation's partner lane one; a lane covers the same dimensions in
// every row it takes, so the token's cosines and sines and the weights are loaded once.
// All arithmetic is float32; the query is rounded once to bf16, key and value once to INT8.
constexpr int kStoreThreads = 256;

template <int D>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(KvPages c, KvStoreArgs a) {
  constexpr uint32_t kLanes = D / 8, kGroups = kStoreThreads / kLanes;
  after_previous();
  const uint32_t token = blockIdx.x, lane = threadIdx.x % kLanes;
  const uint32_t rows = a.q_heads + 2 * c.kv_heads;
  const uint32_t warp_lane = threadIdx.x & 31u;
  const int32_t slot = a.slots[token];
  const bool rotate = a.rot != 0;
  const int32_t pos = rotate ? a.positions[token] : 0;
  if ((slot >= 0 && ((uint32_t)slot >> c.log2_pt) >= c.n_pages) ||
      (rotate && (pos < 0 || (uint32_t)pos >= a.n_positions))) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(a.st, SHN_ERR_INVALID_ARG, token);
    return;
  }
  // the lane's rotation: cosines and sines of its dimensions, and where its partners are
  const uint32_t half = a.rot / 2, d0 = lane * 8;
  float cs[8], sn[8];
  uint32_t partner = warp_lane;
  float sign = 0.f;
  const bool turns = rotate && d0 < a.rot;
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (turns) {
    const float* row = a.cos_sin + (uint64_t)pos * a.rot;
    if (a.pairs) {
      const float4 x = *reinterpret_cast<const float4*>(row + d0 / 2);
      const float4 y = *reinterpret_cast<const float4*>(row + half + d0 / 2);
      cs[0] = x.x, cs[1] = x.y, cs[2] = x.z, cs[3] = x.w;
      sn[0] = y.x, sn[1] = y.y, sn[2] = y.z, sn[3] = y.w;
    } else {
      const uint32_t at = d0 < half ? d0 : d0 - half;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float4 x = *reinterpret_cast<const float4*>(row + at + 4 * v);
        const float4 y = *reinterpret_cast<const float4*>(row + half + at + 4 * v);
        cs[4 * v] = x.x, cs[4 * v + 1] = x.y, cs[4 * v + 2] = x.z, cs[4 * v + 3] = x.w;
        sn[4 * v] = y.x, sn[4 * v + 1] = y.y, sn[4 * v + 2] = y.z, sn[4 * v + 3] = y.w;
      }
      partner = d0 < half ? warp_lane + half / 8 : warp_lane - half / 8;
      sign = d0 < half ? -1.f : 1.f;
    }
  }
  // a block's rows are consecutive; all lanes of a warp run the same number of turns (the shuffles are full)
  const uint32_t per_block = (rows + gridDim.y - 1) / gridDim.y;
  const uint32_t first = blockIdx.y * per_block, last = min(rows, first + per_block);
  for (uint32_t base = first; base < last; base += kGroups) {
    const uint32_t row = base + threadIdx.x / kLanes;
    const bool real = row < last;
    const bool is_q = row < a.q_heads, is_k = !is_q && row < a.q_heads + c.kv_heads;
    const uint32_t h = is_q ? row : is_k ? row - a.q_heads : row - a.q_heads - c.kv_heads;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (real) {
      const uint16_t* src = is_q   ? a.q + (uint64_t)token * a.q_stride
                            : is_k ? a.k + (uint64_t)token * a.k_stride
                                   : a.v + (uint64_t)token * a.v_stride;
      raw = *reinterpret_cast<const uint4*>(src + (uint64_t)h * D + d0);
    }
    float x[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y),
                  bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
    const uint16_t* weight = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
    if (weight) {
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const uint4 w = *reinterpret_cast<const uint4*>(weight + d0);
      const float wf[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                           bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * wf[i];
    }
    if (rotate) {
      if (a.pairs) {
        if (turns && (is_q || is_k)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = x[2 * i], w = x[2 * i + 1];
            x[2 * i] = u * cs[i] - w * sn[i];
            x[2 * i + 1] = w * cs[i] + u * sn[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_sync(~0u, x[i], partner);
          if (turns && (is_q || is_k)) x[i] = x[i] * cs[i] + sign * (other * sn[i]);
        }
      }
    }
    // largest magnitude as an integer maximum of the bits: a NaN is larger than infinity and stays
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
    if (!real) continue;
    if (is_q) {
      const uint4 o = make_uint4(bf16_pack(x[0], x[1]), bf16_pack(x[2], x[3]), bf16_pack(x[4], x[5]), bf16_pack(x[6], x[7]));
      *reinterpret_cast<uint4*>(a.q_out + (uint64_t)token * a.q_out_stride + (uint64_t)h * D + d0) = o;
    } else if (slot >= 0) {
      const float scale = (top > 0x7F800000u ? __uint_as_float(top) : fmaxf(__uint_as_float(top), 1e-30f)) / 127.f;
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // |x / scale| <= 127 up to rounding; x / inf = 0 and NaN -> 0, so a poisoned row is 0 * its scale = NaN
        const int v = max(-127, min(127, __float2int_rn(x[i] / scale)));
        w[i / 4] |= ((uint32_t)v & 0xFFu) << (8 * (i % 4));
      }
      const uint64_t at = kv_row_of_slot(c, (uint32_t)slot, h);
      *reinterpret_cast<uint2*>((is_k ? c.k : c.v) + at * D + d0) = make_uint2(w[0], w[1]);
      if (lane == 0) (is_k ? c.k_scale : c.v_scale)[at] = scale;
    }
  }
}

// ---- shn_kv_load --------------------------------------------------------------------------------
// HBM-bound copy with a scale: 16 INT8 values (16 bytes) in and 32 bytes out per lane, D/16 lanes to a row.
constexpr int kLoadThreads = 256;

__device__ __forceinline__ float int8_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

template <int D>
__global__ void __launch_bounds__(kLoadThreads) kv_load_kernel(KvPages c, KvLoadArgs a) {
  constexpr uint32_t kLanes = D / 16;
  after_previous();
  const uint64_t step = (uint64_t)gridDim.x * kLoadThreads / kLanes;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint64_t rows = (uint64_t)a.n_tokens * c.kv_heads;
  for (uint64_t i = ((uint64_t)blockIdx.x * kLoadThreads + threadIdx.x) / kLanes; i < rows; i += step) {
    const uint32_t token = (uint32_t)(i / c.kv_heads), h = (uint32_t)(i % c.kv_heads);
    const int32_t slot = a.slots[token];
    if (slot < 0) continue;
    if (((uint32_t)slot >> c.log2_pt) >= c.n_pages) {
      if (lane == 0) report(a.st, SHN_ERR_INVALID_ARG, token);
      continue;
    }
    const uint64_t at = kv_row_of_slot(c, (uint32_t)slot, h);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint16_t* out = kv ? a.v_out : a.k_out;
      if (!out) continue;
      const uint4 raw = *reinterpret_cast<const uint4*>((kv ? c.v : c.k) + at * D + lane * 16);
      const float s = (kv ? c.v_scale : c.k_scale)[at];
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = bf16_pack(int8_of(w[j / 2], 2 * (j % 2)) * s, int8_of(w[j / 2], 2 * (j % 2) + 1) * s);
      uint4* dst = reinterpret_cast<uint4*>(out + (uint64_t)token * (kv ? a.v_stride : a.k_stride) + (uint64_t)h * D + lane * 16);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace

cudaError_t launch_kv_begin(DeviceStatus* st, cudaStream_t s) {
  kv_begin_kernel<<<1, 32, 0, s>>>(st);
  return cudaGetLastError();
}

cudaError_t launch_kv_store(const KvPages& c, uint32_t head_dim, const KvStoreArgs& a, int sm_count, cudaStream_t s) {
  const uint32_t groups = kStoreThreads * 8 / head_dim, rows = a.q_heads + 2 * c.kv_heads;
  // few tokens: their rows over several blocks, until the SMs have two blocks each or a block has one row per group
  uint32_t parts = 1;
  while ((uint64_t)parts * a.n_tokens < 2ull * sm_count && parts * groups < rows) ++parts;
  const dim3 grid(a.n_tokens, parts);
  return head_dim == 128 ? launch_behind(kv_store_kernel<128>, grid, kStoreThreads, 0, s, c, a)
                         : launch_behind(kv_store_kernel<64>, grid, kStoreThreads, 0, s, c, a);
}

cudaError_t launch_kv_load(const KvPages& c, uint32_t head_dim, const KvLoadArgs& a, int sm_count, cudaStream_t s) {
  const uint64_t threads = (uint64_t)a.n_tokens * c.kv_heads * (head_dim / 16);
  uint64_t blocks = (threads + kLoadThreads - 1) / kLoadThreads;
  if (blocks > 8ull * sm_count) blocks = 8ull * sm_count;
  const dim3 grid((uint32_t)blocks);
  return head_dim == 128 ? launch_behind(kv_load_kernel<128>, grid, kLoadThreads, 0, s, c, a)
                         : launch_behind(kv_load_kernel<64>, grid, kLoadThreads, 0, s, c, a);
}

}  // namespace shn
