// kv_store.cu — a step's queries, keys and values through norm and rotation, keys and values quantised
// into their pages (shn_kv_store), and rows of the pages back as bf16 (shn_kv_load).
#include "kv_tc.cuh"

namespace shn {
namespace {

__global__ void kv_begin_kernel(DeviceStatus* st) {
  let_next();
  if (threadIdx.x == 0) st->status = 0, st->detail = 0;
}

// ---- shn_kv_store -------------------------------------------------------------------------------
// HBM-bound: every value is read and written once. A head row of D values is held by D/8 lanes, 8 values each: 4
// consecutive ones twice, the second 4 where the rotation's partners of the first are (half the rotated part further on), so a
// rotation needs no other lane; what is not rotated is dealt to the lanes behind. A row's sum of squares and its largest
// magnitude are log2(D/8) shuffles away. A lane covers the same dimensions in every row it takes, so the token's cosines and
// sines and the weights are loaded once, and a block's rows are asked for before anything else is waited for.
// All arithmetic is float32 (two values an instruction); the query is rounded once to bf16, key and value once to INT8.
constexpr int kStoreThreads = 256;
constexpr int kAtOnce = 4;  // rows of a lane that are on their way together

template <int D>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(KvPages c, KvStoreArgs a) {
  using namespace tc;
  constexpr uint32_t kLanes = D / 8, kGroups = kStoreThreads / kLanes;
  const uint32_t token = blockIdx.x, lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const uint32_t rows = a.q_heads + 2 * c.kv_heads;
  // a block's rows are consecutive; all lanes of a warp run the same number of turns (the shuffles are full)
  const uint32_t per_block = (rows + gridDim.y - 1) / gridDim.y;
  const uint32_t first = blockIdx.y * per_block, last = min(rows, first + per_block);
  // the lane's dimensions: 4 from d_lo, 4 from d_hi
  const uint32_t pair = a.rot / 8;  // lanes that rotate
  const bool turns = lane < pair;
  const uint32_t d_lo = turns ? 4 * lane : a.rot + 8 * (lane - pair), d_hi = turns ? d_lo + a.rot / 2 : d_lo + 4;

  uint2 raw[kAtOnce][2];
  auto ask = [&](uint32_t base) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t row = base + i * kGroups + sub;
      raw[i][0] = raw[i][1] = make_uint2(0, 0);
      if (row < last) {
        const uint16_t* src = row < a.q_heads                 ? a.q + (uint64_t)token * a.q_stride + (uint64_t)row * D
                              : row < a.q_heads + c.kv_heads ? a.k + (uint64_t)token * a.k_stride + (uint64_t)(row - a.q_heads) * D
                                                             : a.v + (uint64_t)token * a.v_stride + (uint64_t)(row - a.q_heads - c.kv_heads) * D;
        raw[i][0] = *reinterpret_cast<const uint2*>(src + d_lo);
        raw[i][1] = *reinterpret_cast<const uint2*>(src + d_hi);
      }
    }
  };
  ask(first);
  const int32_t slot = a.slots[token];
  const int32_t pos = a.rot ? a.positions[token] : 0;
  auto weights = [&](const uint16_t* w, uint64_t* f) {
    if (!w) return;
    const uint2 x = *reinterpret_cast<const uint2*>(w + d_lo), y = *reinterpret_cast<const uint2*>(w + d_hi);
    f[0] = pack2(bf16_lo(x.x), bf16_hi(x.x)), f[1] = pack2(bf16_lo(x.y), bf16_hi(x.y));
    f[2] = pack2(bf16_lo(y.x), bf16_hi(y.x)), f[3] = pack2(bf16_lo(y.y), bf16_hi(y.y));
  };
  uint64_t wq[4] = {0, 0, 0, 0}, wk[4] = {0, 0, 0, 0};
  weights(a.q_weight, wq);
  weights(a.k_weight, wk);
  after_previous();
  if ((slot >= 0 && ((uint32_t)slot >> c.log2_pt) >= c.n_pages) || (a.rot && (pos < 0 || (uint32_t)pos >= a.n_positions))) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(a.st, SHN_ERR_INVALID_ARG, token);
    return;
  }
  // cosines and sines of the lane's pairs: (x_i, x_{i+4}) by angle d_lo + i, or with a.pairs (x_0, x_1), (x_2, x_3) by angles
  // d_lo / 2, + 1 and (x_4, x_5), (x_6, x_7) by d_hi / 2, + 1
  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turns) {
    const float *cp = a.cos_sin + (uint64_t)pos * a.rot, *sp = cp + a.rot / 2;
    if (a.pairs) {
      const float2 c0 = *reinterpret_cast<const float2*>(cp + d_lo / 2), c1 = *reinterpret_cast<const float2*>(cp + d_hi / 2);
      const float2 s0 = *reinterpret_cast<const float2*>(sp + d_lo / 2), s1 = *reinterpret_cast<const float2*>(sp + d_hi / 2);
      cs = make_float4(c0.x, c0.y, c1.x, c1.y), sn = make_float4(s0.x, s0.y, s1.x, s1.y);
    } else {
      cs = *reinterpret_cast<const float4*>(cp + d_lo), sn = *reinterpret_cast<const float4*>(sp + d_lo);
    }
  }
  for (uint32_t base = first; base < last; base += kAtOnce * kGroups) {
    if (base != first) ask(base);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (base + i * kGroups >= last) break;
      const uint32_t row = base + i * kGroups + sub;
      const bool real = row < last;
      const bool is_q = row < a.q_heads, is_k = !is_q && row < a.q_heads + c.kv_heads;
      // x[0], x[1]: the first 4 values, x[2], x[3]: the other 4
      uint64_t x[4] = {pack2(bf16_lo(raw[i][0].x), bf16_hi(raw[i][0].x)), pack2(bf16_lo(raw[i][0].y), bf16_hi(raw[i][0].y)),
                       pack2(bf16_lo(raw[i][1].x), bf16_hi(raw[i][1].x)), pack2(bf16_lo(raw[i][1].y), bf16_hi(raw[i][1].y))};
      if (a.q_weight || a.k_weight) {
        uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(x[e], x[e], s2);
        float s0, s1;
        unpack2(s2, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
        if (is_q ? a.q_weight != nullptr : is_k && a.k_weight) {
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const uint64_t r2 = pack2(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = mul2(mul2(x[e], r2), is_q ? wq[e] : wk[e]);
        }
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) unpack2(x[e], y[2 * e], y[2 * e + 1]);
      if (turns && (is_q || is_k)) {
        auto turn = [&](float& u, float& w, float co, float si) {
          const float u0 = u, w0 = w;
          u = u0 * co - w0 * si;
          w = w0 * co + u0 * si;
        };
        if (a.pairs) {
          turn(y[0], y[1], cs.x, sn.x), turn(y[2], y[3], cs.y, sn.y), turn(y[4], y[5], cs.z, sn.z), turn(y[6], y[7], cs.w, sn.w);
        } else {
          turn(y[0], y[4], cs.x, sn.x), turn(y[1], y[5], cs.y, sn.y), turn(y[2], y[6], cs.z, sn.z), turn(y[3], y[7], cs.w, sn.w);
        }
      }
      uint32_t top = 0;
      if (__any_sync(~0u, real && !is_q)) {
        // largest magnitude as an integer maximum of the bits: a NaN is larger than infinity and stays
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
      }
      if (!real) continue;
      if (is_q) {
        uint16_t* dst = a.q_out + (uint64_t)token * a.q_out_stride + (uint64_t)row * D;
        *reinterpret_cast<uint2*>(dst + d_lo) = make_uint2(bf16_pack(y[0], y[1]), bf16_pack(y[2], y[3]));
        *reinterpret_cast<uint2*>(dst + d_hi) = make_uint2(bf16_pack(y[4], y[5]), bf16_pack(y[6], y[7]));
      } else if (slot >= 0) {
        const float scale = (top > 0x7F800000u ? __uint_as_float(top) : fmaxf(__uint_as_float(top), 1e-30f)) / 127.f;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // |y / scale| <= 127 up to rounding; y / inf = 0 and NaN -> 0, so a poisoned row is 0 * its scale = NaN
          const int v = max(-127, min(127, __float2int_rn(y[e] / scale)));
          w[e / 4] |= ((uint32_t)v & 0xFFu) << (8 * (e % 4));
        }
        const uint64_t at = kv_row_of_slot(c, (uint32_t)slot, row - a.q_heads - (is_k ? 0 : c.kv_heads));
        int8_t* dst = (is_k ? c.k : c.v) + at * D;
        *reinterpret_cast<uint32_t*>(dst + d_lo) = w[0];
        *reinterpret_cast<uint32_t*>(dst + d_hi) = w[1];
        if (lane == 0) (is_k ? c.k_scale : c.v_scale)[at] = scale;
      }
    }
  }
}

// ---- shn_kv_load --------------------------------------------------------------------------------
// HBM-bound copy with a scale: 16 INT8 values (16 bytes) in and 32 bytes out per lane, D/16 lanes to a row, keys and values of
// the row together. A token's rows are a block's neighbours, so its slot is read from L1 by all but the first.
constexpr int kLoadThreads = 256;

__device__ __forceinline__ float int8_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

template <int D>
__global__ void __launch_bounds__(kLoadThreads) kv_load_kernel(KvPages c, KvLoadArgs a) {
  constexpr uint32_t kLanes = D / 16;
  const uint32_t lane = threadIdx.x % kLanes;
  // rows of the block: tokens from blockIdx.x * tokens on, `parts` blocks to a token with more rows than a block has
  const uint32_t sub = threadIdx.x / kLanes, kSubs = kLoadThreads / kLanes;
  const uint32_t tokens = max(1u, kSubs / c.kv_heads);
  const uint32_t token = blockIdx.x * tokens + (tokens > 1 ? sub / c.kv_heads : 0);
  const uint32_t h = tokens > 1 ? sub % c.kv_heads : blockIdx.y * kSubs + sub;
  const bool real = token < a.n_tokens && h < c.kv_heads && (tokens == 1 || sub / c.kv_heads < tokens);
  const int32_t slot = real ? a.slots[token] : -1;
  after_previous();
  if (slot < 0) return;
  if (((uint32_t)slot >> c.log2_pt) >= c.n_pages) {
    if (lane == 0) report(a.st, SHN_ERR_INVALID_ARG, token);
    return;
  }
  const uint64_t at = kv_row_of_slot(c, (uint32_t)slot, h);
  uint4 raw[2];
  float s[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    raw[kv] = *reinterpret_cast<const uint4*>((kv ? c.v : c.k) + at * D + lane * 16);
    s[kv] = (kv ? c.v_scale : c.k_scale)[at];
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? a.v_out : a.k_out;
    if (!out) continue;
    const uint32_t w[4] = {raw[kv].x, raw[kv].y, raw[kv].z, raw[kv].w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = bf16_pack(int8_of(w[j / 2], 2 * (j % 2)) * s[kv], int8_of(w[j / 2], 2 * (j % 2) + 1) * s[kv]);
    uint4* dst = reinterpret_cast<uint4*>(out + (uint64_t)token * (kv ? a.v_stride : a.k_stride) + (uint64_t)h * D + lane * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
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

cudaError_t launch_kv_load(const KvPages& c, uint32_t head_dim, const KvLoadArgs& a, cudaStream_t s) {
  const uint32_t subs = kLoadThreads / (head_dim / 16), tokens = c.kv_heads < subs ? subs / c.kv_heads : 1;
  const dim3 grid((a.n_tokens + tokens - 1) / tokens, tokens > 1 ? 1 : (c.kv_heads + subs - 1) / subs);
  return head_dim == 128 ? launch_behind(kv_load_kernel<128>, grid, kLoadThreads, 0, s, c, a)
                         : launch_behind(kv_load_kernel<64>, grid, kLoadThreads, 0, s, c, a);
}

}  // namespace shn
