// kv_store.cu — a step's queries, keys and values through norm and rotation, keys and values quantised
// into their pages (shn_kv_store), and rows of the pages back as bf16 (shn_kv_load).
#include "kv_tc.cuh"

namespace shn {
namespace {

__global__ void kv_begin_kernel(DeviceStatus* st) {
  let_next();
  if (threadIdx.x == 0) st->status = 0, st->detail = 0;
}

// The status of a call whose errors its indexes alone show: one block looks at all of them and is the only one to write the
// status, so no kernel has to clear it first (64 tokens stored and loaded again 4.97 us against 5.99 with one in front of each).
// A store always does so, since its tokens take longer than their indexes (one key head of 64: 8192 tokens 7.5 us, with a kernel
// in front and every block reporting 8.4; 262,144 tokens 196 and 205; 32 query and 8 key heads of 128, 65,536 tokens 262 and 279).
// In a load of many small rows that block would be the last to end, so it does up to kOneTokens tokens (kOne); with more the kernel
// in front clears the status and every block reports. Measured, the one block / the kernel in front: one head of 64, 4096 tokens
// 2.65 / 2.91 us, 8192 3.80 / 3.30, 65,536 21.3 / 8.0; 8 heads of 128, 8192 tokens 10.2 / 10.8, 12,288 14.7 / 14.8, 16,384 18.8 / 18.4.
constexpr uint32_t kOneTokens = 8192;
constexpr int kAhead = 8;  // 16-byte loads of a thread on their way together
// The first of the n indexes that is outside [0, end); negative ones are fine where kNone.
template <bool kNone, int kThreads>
__device__ __forceinline__ uint32_t first_outside(const int32_t* p, uint32_t n, uint32_t end) {
  const uint32_t t = threadIdx.x;
  const uint32_t lead = min(n, (uint32_t)(-(reinterpret_cast<uintptr_t>(p) >> 2) & 3)), quads = (n - lead) / 4, tail = lead + 4 * quads;
  uint32_t first = 0xFFFFFFFFu;
  auto look = [&](int32_t x, uint32_t at) {
    if (!(kNone && x < 0) && (uint32_t)x >= end) first = min(first, at);
  };
  if (t < lead) look(p[t], t);
  if (tail + t < n) look(p[tail + t], tail + t);
  const int4* v = reinterpret_cast<const int4*>(p + lead);
#pragma unroll 1
  for (uint32_t i0 = t; i0 < quads; i0 += kAhead * kThreads) {
    int4 x[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const uint32_t i = i0 + e * kThreads;
      if (i < quads) x[e] = v[i];
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const uint32_t i = i0 + e * kThreads, at = lead + 4 * i;
      if (i < quads) look(x[e].x, at), look(x[e].y, at + 1), look(x[e].z, at + 2), look(x[e].w, at + 3);
    }
  }
  return first;
}
template <int kThreads>
__device__ __forceinline__ void write_status(DeviceStatus* st, uint32_t first) {
  __shared__ uint32_t least[kThreads / 32];
  first = __reduce_min_sync(~0u, first);
  if ((threadIdx.x & 31) == 0) least[threadIdx.x >> 5] = first;
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < kThreads / 32; ++i) first = min(first, least[i]);
  st->status = first == 0xFFFFFFFFu ? SHN_OK : SHN_ERR_INVALID_ARG;
  st->detail = first == 0xFFFFFFFFu ? 0 : first;
}

// ---- shn_kv_store -------------------------------------------------------------------------------
// HBM-bound: every value is read and written once. A head row of D values is held by D/8 lanes, 8 values each: 4
// consecutive ones twice, the second 4 where the rotation's partners of the first are (half the rotated part further on), so a
// rotation needs no other lane; what is not rotated is dealt to the lanes behind. A row's sum of squares and its largest
// magnitude are log2(D/8) shuffles away. A lane covers the same dimensions in every row it takes, so the token's cosines and
// sines and the weights are loaded once, and a block's rows are asked for before anything else is waited for.
// All arithmetic is float32 (two values an instruction); the query is rounded once to bf16, key and value once to INT8:
// issuing instructions bounds this about as much as memory, so a row has one division and one reciprocal, and y / scale is
// rounded by adding 1.5 * 2^23, which leaves the integer in the last byte.
// Measured (8191 tokens, 32 query and 8 key heads of 128): 43 us for 190 MB, 4.4 TB/s, 67 % of the measured copy rate.
// Small blocks, each with its token: what a warp does once for a token (rotation, addresses) then serves more rows, and
// tokens of few rows leave no warp idle. 64 threads, 14 blocks to an SM: 42.9 us, and 8191 tokens of 8 query and 8 key heads
// of 64 11.8; 128 threads, 6 blocks 44.4 and 14.3; 256 threads, 3 blocks 53.5 and 23.0; 32 threads, 24 blocks 48.5 and 9.6.
constexpr int kStoreThreads = 64, kStoreBlocks = 14;
constexpr int kAtOnce = 4;  // query rows of a lane that are on their way together

// A lane's 8 values of a row, two by two: [0], [1] the first 4, [2], [3] the other 4.
struct Row8 {
  uint64_t x[4];
};
struct RawRow {
  uint2 lo, hi;
  __device__ __forceinline__ Row8 values() const {
    using tc::pack2;
    return Row8{{pack2(bf16_lo(lo.x), bf16_hi(lo.x)), pack2(bf16_lo(lo.y), bf16_hi(lo.y)), pack2(bf16_lo(hi.x), bf16_hi(hi.x)),
                 pack2(bf16_lo(hi.y), bf16_hi(hi.y))}};
  }
};
// The token's rotation of the lane's values: (x_i, x_{i+4}) by the angle of c[i / 2]'s i mod 2; or (pairs) (x_0, x_1), (x_2, x_3),
// (x_4, x_5), (x_6, x_7) by the four angles in order.
struct Turn {
  uint64_t c[2], s[2], minus_s[2];
  __device__ __forceinline__ void apply(Row8& v, bool pairs) const {
    using namespace tc;
    if (!pairs) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t u = v.x[e], w = v.x[e + 2];
        v.x[e] = fma2(u, c[e], mul2(w, minus_s[e]));
        v.x[e + 2] = fma2(w, c[e], mul2(u, s[e]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float u, w, c0, c1, s0, s1;
        unpack2(v.x[e], u, w);
        unpack2(c[e / 2], c0, c1);
        unpack2(s[e / 2], s0, s1);
        const float co = e & 1 ? c1 : c0, si = e & 1 ? s1 : s0;
        v.x[e] = pack2(u * co - w * si, w * co + u * si);
      }
    }
  }
};
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kStoreThreads, kStoreBlocks) kv_store_kernel(KvPages c, KvStoreArgs a) {
  using namespace tc;
  constexpr uint32_t kLanes = D / 8, kGroups = kStoreThreads / kLanes;
  if (blockIdx.x == 0) {
    if (blockIdx.y) return;
    uint32_t first = first_outside<true, kStoreThreads>(a.slots, a.n_tokens, c.n_pages << c.log2_pt);
    if (a.rot) first = min(first, first_outside<false, kStoreThreads>(a.positions, a.n_tokens, a.n_positions));
    return write_status<kStoreThreads>(a.st, first);
  }
  const uint32_t block = blockIdx.x - 1, blocks = gridDim.x - 1;
  const uint32_t lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  // The block's share of the query rows, and of the key and value rows (keys first); all lanes of a warp run the same
  // number of turns (the shuffles are full).
  const uint32_t q_share = (a.q_heads + gridDim.y - 1) / gridDim.y, kv_share = (2 * c.kv_heads + gridDim.y - 1) / gridDim.y;
  const uint32_t q0 = blockIdx.y * q_share, q1 = min(a.q_heads, q0 + q_share);
  const uint32_t kv0 = blockIdx.y * kv_share, kv1 = min(2 * c.kv_heads, kv0 + kv_share);
  // the lane's dimensions: 4 from d_lo, 4 from d_hi
  const uint32_t pair = a.rot / 8;  // lanes that rotate
  const bool turns = lane < pair;
  const uint32_t d_lo = turns ? 4 * lane : a.rot + 8 * (lane - pair), d_hi = turns ? d_lo + a.rot / 2 : d_lo + 4;

  const uint32_t further = d_hi - d_lo;
  RawRow raw[kAtOnce], raw_kv;
  auto ask = [&](const uint16_t* src, RawRow& r) {
    r.lo = *reinterpret_cast<const uint2*>(src);
    r.hi = *reinterpret_cast<const uint2*>(src + further);
  };
  const uint16_t *q_src, *k_src, *v_src;  // the token's rows
  auto ask_q = [&](uint32_t base) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t row = base + i * kGroups + sub;
      raw[i].lo = raw[i].hi = make_uint2(0, 0);
      if (row < q1) ask(q_src + row * D, raw[i]);
    }
  };
  auto ask_kv = [&](uint32_t row) {
    raw_kv.lo = raw_kv.hi = make_uint2(0, 0);
    if (row < kv1) ask(row < c.kv_heads ? k_src + row * D : v_src + (row - c.kv_heads) * D, raw_kv);
  };
  auto weights = [&](const uint16_t* w) {
    RawRow r = {make_uint2(0, 0), make_uint2(0, 0)};
    if (w) r.lo = *reinterpret_cast<const uint2*>(w + d_lo), r.hi = *reinterpret_cast<const uint2*>(w + d_hi);
    return r.values();
  };
  const Row8 wq = weights(a.q_weight), wk = weights(a.k_weight);
  auto normed = [&](Row8& v, const Row8& w, bool is) {
    uint64_t s2 = mul2(v.x[0], v.x[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s2 = fma2(v.x[e], v.x[e], s2);
    float s0, s1;
    unpack2(s2, s0, s1);
    float ss = s0 + s1;
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
    const uint64_t r2 = pack2(r, r);
    if (is) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v.x[e] = mul2(mul2(v.x[e], r2), w.x[e]);
    }
  };
  // a block's tokens one after another; the next one's slot and position are read a turn ahead
  int32_t slot = a.slots[block], pos = a.rot ? a.positions[block] : 0;
  for (uint32_t token = block; token < a.n_tokens; token += blocks) {
    q_src = a.q + (uint64_t)token * a.q_stride + d_lo;
    k_src = a.k + (uint64_t)token * a.k_stride + d_lo, v_src = a.v + (uint64_t)token * a.v_stride + d_lo;
    ask_q(q0);
    ask_kv(kv0 + sub);
    const int32_t slot_now = slot, pos_now = pos;
    if (token + blocks < a.n_tokens) {
      slot = a.slots[token + blocks];
      if (a.rot) pos = a.positions[token + blocks];
    }
    if ((slot_now >= 0 && ((uint32_t)slot_now >> c.log2_pt) >= c.n_pages) || (a.rot && (uint32_t)pos_now >= a.n_positions)) continue;
    Turn turn = {};
    if (turns) {
      const float *cp = a.cos_sin + (uint64_t)pos_now * a.rot, *sp = cp + a.rot / 2;
      float4 cs, sn;
      if (a.pairs) {
        const float2 c0 = *reinterpret_cast<const float2*>(cp + d_lo / 2), c1 = *reinterpret_cast<const float2*>(cp + d_hi / 2);
        const float2 s0 = *reinterpret_cast<const float2*>(sp + d_lo / 2), s1 = *reinterpret_cast<const float2*>(sp + d_hi / 2);
        cs = make_float4(c0.x, c0.y, c1.x, c1.y), sn = make_float4(s0.x, s0.y, s1.x, s1.y);
      } else {
        cs = *reinterpret_cast<const float4*>(cp + d_lo), sn = *reinterpret_cast<const float4*>(sp + d_lo);
      }
      turn = {{pack2(cs.x, cs.y), pack2(cs.z, cs.w)}, {pack2(sn.x, sn.y), pack2(sn.z, sn.w)}, {pack2(-sn.x, -sn.y), pack2(-sn.z, -sn.w)}};
    }
    // ---- queries
    uint16_t* q_dst = a.q_out + (uint64_t)token * a.q_out_stride + d_lo;
    for (uint32_t base = q0; base < q1; base += kAtOnce * kGroups) {
      if (base != q0) ask_q(base);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (base + i * kGroups >= q1) break;
        const uint32_t row = base + i * kGroups + sub;
        Row8 v = raw[i].values();
        if (a.q_weight) normed(v, wq, true);
        if (turns) turn.apply(v, a.pairs);
        if (row < q1) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) unpack2(v.x[e], y[2 * e], y[2 * e + 1]);
          uint16_t* dst = q_dst + row * D;
          *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pack(y[0], y[1]), bf16_pack(y[2], y[3]));
          *reinterpret_cast<uint2*>(dst + further) = make_uint2(bf16_pack(y[4], y[5]), bf16_pack(y[6], y[7]));
        }
      }
    }
    // ---- keys and values
    if (slot_now < 0) continue;
    for (uint32_t base = kv0; base < kv1; base += kGroups) {
      const uint32_t row = base + sub;
      const bool is_k = row < c.kv_heads;
      Row8 v = raw_kv.values();
      if (base + kGroups < kv1) ask_kv(row + kGroups);
      if (a.k_weight && base < c.kv_heads) normed(v, wk, is_k);
      if (turns && is_k) turn.apply(v, a.pairs);
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) unpack2(v.x[e], y[2 * e], y[2 * e + 1]);
      float top = fabsf(y[0]);  // a NaN among them stays
#pragma unroll
      for (int e = 1; e < 8; ++e) top = max_nan(top, fabsf(y[e]));
#pragma unroll
      for (int d = kLanes / 2; d; d >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, d));
      if (row >= kv1) continue;
      const float scale = max_nan(top, 1e-30f) / 127.f, inverse = 1.f / scale;
      // y / scale in float32: times the reciprocal, and one residual step that leaves it correctly rounded but for rare
      // last-bit cases (P. Markstein, IBM J. Res. Dev. 34, 1990)
      const uint64_t by = pack2(inverse, inverse), minus = pack2(-scale, -scale), round = pack2(12582912.f, 12582912.f);
      uint64_t n[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t near = mul2(v.x[e], by);
        n[e] = add2(fma2(fma2(near, minus, v.x[e]), by, near), round);
      }
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float f[4];
        unpack2(n[2 * e], f[0], f[1]);
        unpack2(n[2 * e + 1], f[2], f[3]);
        w[e] = __byte_perm(__byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040),
                           __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040), 0x5410);
      }
      const uint64_t at = kv_row_of_slot(c, (uint32_t)slot_now, is_k ? row : row - c.kv_heads);
      int8_t* dst = (is_k ? c.k : c.v) + at * D + d_lo;
      *reinterpret_cast<uint32_t*>(dst) = w[0];
      *reinterpret_cast<uint32_t*>(dst + further) = w[1];
      if (lane == 0) (is_k ? c.k_scale : c.v_scale)[at] = scale;
    }
  }
}

// ---- shn_kv_load --------------------------------------------------------------------------------
// HBM-bound copy with a scale: 16 INT8 values (16 bytes) in and 32 bytes out per lane, D/16 lanes to a row, keys and values of
// the row together. A token's rows are a block's neighbours, so its slot is read from L1 by all but the first.
// Read and written once, so as streaming data that leaves the L2 first, and in small blocks, which end and begin more evenly.
// Measured (65,536 tokens, 8 heads of 128): 67 us for 407 MB, 6.0 TB/s, 92 % of the measured copy rate; blocks of 128 threads
// 69.5, of 256 70.9, those without the streaming hints 76.1; a loop over rows with one of them on its way 97.
constexpr int kLoadThreads = 64;

__device__ __forceinline__ float int8_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

template <int D, bool kOne>
__global__ void __launch_bounds__(kLoadThreads) kv_load_kernel(KvPages c, KvLoadArgs a) {
  constexpr uint32_t kLanes = D / 16;
  if (kOne && blockIdx.x == 0) {
    if (blockIdx.y == 0) write_status<kLoadThreads>(a.st, first_outside<true, kLoadThreads>(a.slots, a.n_tokens, c.n_pages << c.log2_pt));
    return;
  }
  const uint32_t lane = threadIdx.x % kLanes;
  // rows of the block: so many tokens, or a part of one token's rows where it has more than a block
  const uint32_t sub = threadIdx.x / kLanes, kSubs = kLoadThreads / kLanes;
  const uint32_t tokens = max(1u, kSubs / c.kv_heads);
  const uint32_t token = (blockIdx.x - kOne) * tokens + (tokens > 1 ? sub / c.kv_heads : 0);
  const uint32_t h = tokens > 1 ? sub % c.kv_heads : blockIdx.y * kSubs + sub;
  const bool real = token < a.n_tokens && h < c.kv_heads && (tokens == 1 || sub / c.kv_heads < tokens);
  const int32_t slot = real ? a.slots[token] : -1;
  if constexpr (!kOne) after_previous();
  if (slot < 0) return;
  if (((uint32_t)slot >> c.log2_pt) >= c.n_pages) {
    if (!kOne && lane == 0) report_first(a.st, SHN_ERR_INVALID_ARG, token);
    return;
  }
  const uint64_t at = kv_row_of_slot(c, (uint32_t)slot, h);
  uint4 raw[2];
  float s[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    raw[kv] = __ldcs(reinterpret_cast<const uint4*>((kv ? c.v : c.k) + at * D + lane * 16));
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
    __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
  }
}

}  // namespace

cudaError_t launch_kv_begin(DeviceStatus* st, cudaStream_t s) {
  kv_begin_kernel<<<1, 32, 0, s>>>(st);
  return cudaGetLastError();
}

cudaError_t launch_kv_store(const KvPages& c, uint32_t head_dim, const KvStoreArgs& a, int sm_count, cudaStream_t s) {
  const uint32_t groups = kStoreThreads * 8 / head_dim, rows = a.q_heads > 2 * c.kv_heads ? a.q_heads : 2 * c.kv_heads;
  // few tokens: their rows over several blocks, until the SMs have 8 blocks each or a block has one row per group (a token, 32
  // query and 8 key heads of 128, 2.3 us; 2.5 with fewer and larger blocks)
  uint32_t parts = 1;
  while ((uint64_t)parts * a.n_tokens < 8ull * sm_count && parts * groups < rows) ++parts;
  // as many blocks as the SMs have places, each with its tokens (or the status)
  const uint32_t most = kStoreBlocks * (uint32_t)sm_count - 1;
  const dim3 grid(1 + (a.n_tokens < most ? a.n_tokens : most), parts);
  return head_dim == 128 ? launch_first(kv_store_kernel<128>, grid, kStoreThreads, 0, s, c, a) : launch_first(kv_store_kernel<64>, grid, kStoreThreads, 0, s, c, a);
}

cudaError_t launch_kv_load(const KvPages& c, uint32_t head_dim, const KvLoadArgs& a, cudaStream_t s) {
  const uint32_t subs = kLoadThreads / (head_dim / 16), tokens = c.kv_heads < subs ? subs / c.kv_heads : 1;
  const uint32_t blocks = (a.n_tokens + tokens - 1) / tokens, parts = tokens > 1 ? 1 : (c.kv_heads + subs - 1) / subs;
  if (a.n_tokens > kOneTokens) {
    const cudaError_t e = launch_kv_begin(a.st, s);
    if (e != cudaSuccess) return e;
    return head_dim == 128 ? launch_behind(kv_load_kernel<128, false>, dim3(blocks, parts), kLoadThreads, 0, s, c, a)
                           : launch_behind(kv_load_kernel<64, false>, dim3(blocks, parts), kLoadThreads, 0, s, c, a);
  }
  if (head_dim == 128) kv_load_kernel<128, true><<<dim3(1 + blocks, parts), kLoadThreads, 0, s>>>(c, a);
  else kv_load_kernel<64, true><<<dim3(1 + blocks, parts), kLoadThreads, 0, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace shn
