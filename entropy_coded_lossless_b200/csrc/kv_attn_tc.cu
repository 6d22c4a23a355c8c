// kv_attn_tc.cu — attention of many query rows over the paged INT8 cache on the tensor cores: packed causal
// prompts (shn_kv_attn_prompt).
//
// A block takes 256 rows of one key head: row = (query, head of the group), so every key and value it reads serves all
// heads of the group, whatever their number. It walks the sequence in tiles of 128 tokens:
//   S = Q K^T      tcgen05.mma, bf16, M = 128 rows, N = 128 tokens, two of them (rows 0-127, rows 128-255), into TMEM
//   s = S * k_scale_j * softmax_scale * log2(e);  p = 2^(s - m);  l += p;  P = bf16(p * v_scale_j)   one thread per row
//   O += P V       tcgen05.mma with P read from TMEM (it takes the place of S), V as the integers
// K and V enter as the integers, which bf16 holds exactly, so nothing is rounded on the way in; their scales are
// applied to the float32 scores and weights. The one rounding inside is P's to bf16: the tensor cores multiply
// 16-bit operands, and bf16 (8 bits, float32's range) needs no care for the scales' size where fp16 would.
//
// Softmax in one pass: m is a running maximum in units of log2. It is only raised when a row's maximum grows by more
// than 8, i.e. a weight may reach 2^8 before the sums are scaled down: that is exact in float32 and bf16 alike
// (a power-of-two range, no rounding) and spares almost every rescaling of O after a row's first tiles.
//
// Roles (512 threads): warps 0-3 and 4-7 the softmax of the two row tiles, warps 8-11 fetch the tiles and turn INT8 into
// bf16 operands in shared memory, warp 12 issues the products. While the softmax of one row tile works, the
// products of the other run. Two K and two V buffers; the next tile's bytes are on their way in registers while the present
// one is converted.
// TMEM (512 columns): S0, S1 (128 each; P in their first 64), O0, O1 (D each).
#include "kv_tc.cuh"

namespace shn {
namespace {

using namespace tc;

constexpr uint32_t kThreads = 512;
constexpr uint32_t kTile = 128;      // tokens of a tile
constexpr uint32_t kRows = 256;      // query rows of a block
constexpr uint32_t kHalf = 128 * 128;  // bytes of 128 rows of 64 bf16

template <int D>
struct Layout {
  static constexpr uint32_t kOperand = 128 * D * 2;  // one 128 x D bf16 operand
  static constexpr uint32_t q = 0, k = 2 * kOperand, v = 4 * kOperand, k_scale = 6 * kOperand, v_scale = k_scale + 4 * 512,
                            bars = v_scale + 4 * 512, misc = bars + 256, scan = misc + 64, total = scan + 192;
};
// barriers
enum : uint32_t { kQFull = 0, kKFull = 8, kKEmpty = 24, kVFull = 40, kVEmpty = 56, kScaleFull = 72, kSFull = 104, kPFull = 120, kOFull = 136, kDrain = 152 };

struct Work {
  uint32_t req, row0, rows;  // request, first row of the block within it, rows of the request
  int32_t q0;                // first query of the request
  int32_t len, nq;           // its tokens and queries
};

// Which request's rows a block takes: tiles of 256 rows, request after request, the last tile first (a
// prompt's last rows see the most tokens, and long blocks belong in front). False: no such tile.
__device__ __forceinline__ bool find_work(const KvPages& c, const KvAttnArgs& a, uint32_t group, uint32_t tile_from_end,
                                          uint32_t* scan, Work& w) {
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t run = (a.n_reqs + kThreads - 1) / kThreads;
  const uint32_t r0 = min(a.n_reqs, t * run), r1 = min(a.n_reqs, r0 + run);
  uint32_t own = 0;
  for (uint32_t r = r0; r < r1; ++r) {
    const int32_t b = a.cu_q[r], e = a.cu_q[r + 1];
    if (b < 0 || e < b || (uint32_t)e > a.n_tokens) report(a.st, SHN_ERR_INVALID_ARG, r);
    else own += ((uint32_t)(e - b) * group + kRows - 1) / kRows;
  }
  uint32_t inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(~0u, inc, d);
    if (lane >= (uint32_t)d) inc += x;
  }
  if (lane == 31) scan[warp] = inc;
  if (t == 0) scan[17] = 0xFFFFFFFFu;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (uint32_t i = 0; i < kThreads / 32; ++i) {
    const uint32_t x = scan[i];
    before += i < warp ? x : 0;
    total += x;
  }
  if (tile_from_end >= total) return false;
  const uint32_t tile = total - 1 - tile_from_end;
  before += inc - own;
  if (tile >= before && tile < before + own) {
    uint32_t left = tile - before;
    for (uint32_t r = r0; r < r1; ++r) {
      const int32_t b = a.cu_q[r], e = a.cu_q[r + 1];
      if (b < 0 || e < b || (uint32_t)e > a.n_tokens) continue;
      const uint32_t n = ((uint32_t)(e - b) * group + kRows - 1) / kRows;
      if (left < n) {
        scan[17] = r;
        scan[18] = left;
        break;
      }
      left -= n;
    }
  }
  __syncthreads();
  w.req = scan[17];
  if (w.req >= a.n_reqs) return false;
  w.row0 = scan[18] * kRows;
  w.q0 = a.cu_q[w.req];
  w.nq = a.cu_q[w.req + 1] - w.q0;
  w.rows = (uint32_t)w.nq * group;
  const int64_t holds = (int64_t)a.max_blocks << c.log2_pt;
  int32_t len = a.kv_len[w.req];
  if (len < 0 || len > holds) {
    if (t == 0) report(a.st, SHN_ERR_INVALID_ARG, w.req);
    len = len < 0 ? 0 : (int32_t)holds;
  }
  w.len = len;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(KvPages c, KvAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Layout<D>;
  const uint32_t base = smem_addr(smem), bars = base + L::bars, stop = base + L::misc;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t group = a.q_heads / c.kv_heads, hk = blockIdx.x % c.kv_heads;

  // after a wait that gave up the call has failed: the other blocks do not start on it
  if (__syncthreads_or(*reinterpret_cast<volatile uint32_t*>(&a.st->status) == SHN_ERR_TIMEOUT)) return;
  Work w;
  if (!find_work(c, a, group, blockIdx.x / c.kv_heads, reinterpret_cast<uint32_t*>(smem + L::scan), w)) return;
  const uint32_t rows_here = min(kRows, w.rows - w.row0);
  // tokens the block's last row sees; every row of the block sees at most as many
  const int32_t shift = w.len - w.nq + 1;  // query i sees shift + i tokens
  const int32_t most = max(0, min(w.len, shift + (int32_t)((w.row0 + rows_here - 1) / group)));
  const uint32_t tiles = ((uint32_t)most + kTile - 1) / kTile;

  if (tid == 0) {
    bar_init(bars + kQFull, 256);
    bar_init(bars + kDrain, 1);
    for (uint32_t i = 0; i < 2; ++i) {
      bar_init(bars + kKFull + 8 * i, 128);
      bar_init(bars + kKEmpty + 8 * i, 1);
      bar_init(bars + kVFull + 8 * i, 128);
      bar_init(bars + kVEmpty + 8 * i, 1);
      bar_init(bars + kSFull + 8 * i, 1);
      bar_init(bars + kPFull + 8 * i, 128);
      bar_init(bars + kOFull + 8 * i, 1);
    }
    for (uint32_t i = 0; i < 4; ++i) bar_init(bars + kScaleFull + 8 * i, 128);
    sts32(stop, 0);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(stop + 4) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = lds32(stop + 4);

  if (warp < 8) {
    // ---- softmax: thread = row -----------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // the queries of the block as an operand, zeros behind the last row
    for (uint32_t i = tid; i < kRows * (D / 8); i += 256) {
      const uint32_t row = i / (D / 8), piece = i % (D / 8);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < rows_here) {
        const uint32_t g = w.row0 + row;
        x = *reinterpret_cast<const uint4*>(a.q + (uint64_t)(w.q0 + g / group) * a.q_stride + (uint64_t)(hk * group + g % group) * D + piece * 8);
      }
      sts128(base + L::q + (row / 128) * L::kOperand + (piece / 8) * kHalf + swizzled(row % 128, piece % 8), x);
    }
    fence_smem();
    bar_arrive(bars + kQFull);

    const uint32_t half = warp >> 2;  // which 128 rows
    const uint32_t row = half * 128 + (warp & 3) * 32 + lane;
    const uint32_t at = tmem + (((warp & 3) * 32) << 16);  // the warp's lanes of TMEM
    const uint32_t s_col = at + half * 128, o_col = at + 256 + half * D;
    const uint32_t g = w.row0 + row;
    const int32_t seen = row < rows_here ? max(0, min(w.len, shift + (int32_t)(g / group))) : 0;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (uint32_t j = 0; j < tiles; ++j) {
      ok = bar_wait(bars + kScaleFull + 8 * (j & 3), (j >> 2) & 1, stop) && bar_wait(bars + kSFull + 8 * half, j & 1, stop);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      fence_after();
      uint32_t s[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) ld32(s_col + 32 * q, s + 32 * q);
      wait_ld();
      const uint32_t ks = base + L::k_scale + (j & 3) * 512, vs = base + L::v_scale + (j & 3) * 512;
      float top = -INFINITY;
      const bool edge = __any_sync(~0u, (int32_t)((j + 1) * kTile) > seen);
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        const uint4 f = lds128(ks + 16 * q);
        float x[4];
        unpack2(mul2(pack2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])), pack2(__uint_as_float(f.x), __uint_as_float(f.y))), x[0], x[1]);
        unpack2(mul2(pack2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])), pack2(__uint_as_float(f.z), __uint_as_float(f.w))), x[2], x[3]);
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = (int32_t)(j * kTile + 4 * q + e) < seen ? x[e] : -INFINITY;
        }
        top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * q + e] = __float_as_uint(x[e]);
      }
      if (j == 0) {
        m = top;
      } else if (__any_sync(~0u, top > m + 8.f)) {
        const float next = top > m + 8.f ? top : m;
        const float keep = next == m ? 1.f : exp2_approx(m - next);
        m = next;
        l *= keep;
        ok = __all_sync(~0u, bar_wait(bars + kOFull + 8 * half, (j - 1) & 1, stop));
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          ld32(o_col + 32 * q, o);
          wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
          st32(o_col + 32 * q, o);
        }
      }
      const float neg = m == -INFINITY ? 0.f : -m;
      const uint64_t neg2 = pack2(neg, neg);
      uint64_t sum2[2] = {0, 0};
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        const uint4 f = lds128(vs + 16 * q);
        float x[4];
        unpack2(add2(pack2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])), neg2), x[0], x[1]);
        unpack2(add2(pack2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])), neg2), x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = exp2_approx(x[e]);
        const uint64_t p01 = pack2(x[0], x[1]), p23 = pack2(x[2], x[3]);
        sum2[0] = add2(sum2[0], p01);
        sum2[1] = add2(sum2[1], p23);
        unpack2(mul2(p01, pack2(__uint_as_float(f.x), __uint_as_float(f.y))), x[0], x[1]);
        unpack2(mul2(p23, pack2(__uint_as_float(f.z), __uint_as_float(f.w))), x[2], x[3]);
        if (edge) {  // a scale behind the row's end may be anything: 0 * infinity
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = (int32_t)(j * kTile + 4 * q + e) < seen ? x[e] : 0.f;
        }
        s[2 * q] = bf16_pack(x[0], x[1]);  // (columns 2q and 2q+1 are behind us)
        s[2 * q + 1] = bf16_pack(x[2], x[3]);
      }
      st32(s_col, s);
      st32(s_col + 32, s + 32);
      float e0, e1, e2, e3;
      unpack2(sum2[0], e0, e1);
      unpack2(sum2[1], e2, e3);
      l += (e0 + e1) + (e2 + e3);
      wait_st();
      fence_before();
      bar_arrive(bars + kPFull + 8 * half);
    }
    if (ok && tiles) ok = __all_sync(~0u, bar_wait(bars + kOFull + 8 * half, (tiles - 1) & 1, stop));
    if (ok) {
      fence_after();
      // no token seen: zeros. (A sum that is not positive although tokens were seen is a NaN's or an infinity's.)
      const float inv = seen > 0 ? 1.f / l : 0.f;
      uint16_t* dst = a.out + (uint64_t)(w.q0 + g / group) * a.out_stride + (uint64_t)(hk * group + g % group) * D;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        if (tiles) {
          ld32(o_col + 32 * q, o);
          wait_ld();
        }
        if (row < rows_here) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = seen > 0 ? bf16_pack(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv) : 0u;
            *reinterpret_cast<uint4*>(dst + 32 * q + 8 * e) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      fence_before();
    }
  } else if (warp < 12) {
    // ---- fetch and convert ---------------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    constexpr int kLoads = D / 16;  // 16-byte loads of a thread per operand
    const uint32_t t = tid - 256, cw = t >> 5;
    // A warp's load: 4 lanes on 64 values of a row, 8 rows. For D = 128 even warps take the rows' first 64 values.
    const uint32_t part = D == 128 ? (cw & 1) : 0, first = D == 128 ? (cw >> 1) * 64 : cw * 32;
    const uint32_t chunk = lane & 3, sub = lane >> 2;
    const float k_mul = a.scale * 1.44269504088896340736f;  // log2(e)
    const int32_t* table = a.table + (uint64_t)w.req * a.max_blocks;
    const uint32_t pt_mask = (1u << c.log2_pt) - 1;

    // page of the tile's 16-token group `lane` (lanes 0-7), -1 where there are no tokens
    auto pages_of = [&](uint32_t j) -> int32_t {
      const int32_t tok = (int32_t)(j * kTile + (lane & 7) * 16);
      int32_t p = -1;
      if (j < tiles && tok < most) {
        p = table[tok >> c.log2_pt];
        if (p < 0 || (uint32_t)p >= c.n_pages) {
          if (lane < 8) report(a.st, SHN_ERR_INVALID_ARG, w.req);
          p = -1;
        }
      }
      return p;
    };
    auto fetch = [&](const int8_t* src, uint32_t j, int32_t pages, uint4* raw) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t row = first + i * 8 + sub, tok = j * kTile + row;
        const int32_t p = __shfl_sync(~0u, pages, (first + i * 8) >> 4);
        raw[i] = make_uint4(0, 0, 0, 0);
        if (p >= 0 && (int32_t)tok < most)
          raw[i] = *reinterpret_cast<const uint4*>(src + kv_row(c, (uint32_t)p, hk, tok & pt_mask) * D + part * 64 + chunk * 16);
      }
    };
    auto convert = [&](const uint4* raw, uint32_t dst) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t row = first + i * 8 + sub;
        const uint2 x = bf16x4_of_int8(raw[i].x), y = bf16x4_of_int8(raw[i].y), z = bf16x4_of_int8(raw[i].z), u = bf16x4_of_int8(raw[i].w);
        sts128(dst + part * kHalf + swizzled(row, 2 * chunk), make_uint4(x.x, x.y, y.x, y.y));
        sts128(dst + part * kHalf + swizzled(row, 2 * chunk + 1), make_uint4(z.x, z.y, u.x, u.y));
      }
      fence_smem();
    };
    uint4 kr[kLoads], vr[kLoads];
    float ksc = 0.f, vsc = 0.f;
    // scales of token t of the tile
    auto fetch_scales = [&](uint32_t j, int32_t pages) {
      const int32_t p = __shfl_sync(~0u, pages, t >> 4);
      const uint32_t tok = j * kTile + t;
      ksc = vsc = 0.f;
      if (p >= 0 && (int32_t)tok < most) {
        const uint64_t at = kv_row(c, (uint32_t)p, hk, tok & pt_mask);
        ksc = c.k_scale[at];
        vsc = c.v_scale[at];
      }
    };
    int32_t pages = pages_of(0);
    if (tiles) {
      fetch(c.k, 0, pages, kr);
      fetch_scales(0, pages);
    }
    for (uint32_t j = 0; j < tiles; ++j) {
      const uint32_t buf = j & 1, use = j >> 1;
      fetch(c.v, j, pages, vr);
      const int32_t next = pages_of(j + 1);
      if (!__all_sync(~0u, bar_wait(bars + kKEmpty + 8 * buf, (use & 1) ^ 1, stop))) break;
      // The scales have four places: those of tile j - 4 were read before the products of tile j - 3 could begin, and
      // this K buffer is free since those of tile j - 2 are done.
      sts32(base + L::k_scale + (j & 3) * 512 + 4 * t, __float_as_uint(ksc * k_mul));
      sts32(base + L::v_scale + (j & 3) * 512 + 4 * t, __float_as_uint(vsc));
      bar_arrive(bars + kScaleFull + 8 * (j & 3));
      convert(kr, base + L::k + buf * L::kOperand);
      bar_arrive(bars + kKFull + 8 * buf);
      pages = next;
      if (j + 1 < tiles) {
        fetch(c.k, j + 1, pages, kr);
        fetch_scales(j + 1, pages);
      }
      if (!__all_sync(~0u, bar_wait(bars + kVEmpty + 8 * buf, (use & 1) ^ 1, stop))) break;
      convert(vr, base + L::v + buf * L::kOperand);
      bar_arrive(bars + kVFull + 8 * buf);
    }
  } else {
    // ---- products: one thread issues -----------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (tid == 12 * 32 && tiles) {
      constexpr uint32_t kS = instr_desc(128, 128, false), kO = instr_desc(128, D, true);
      auto scores = [&](uint32_t i, uint32_t j) {
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const uint32_t off = (e / 4) * kHalf + (e % 4) * 32;
          mma_ss(tmem + 128 * i, smem_desc(base + L::q + i * L::kOperand + off, 16), smem_desc(base + L::k + (j & 1) * L::kOperand + off, 16), kS, e > 0);
        }
        commit(bars + kSFull + 8 * i);
      };
      auto values = [&](uint32_t i, uint32_t j) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          mma_ts(tmem + 256 + D * i, tmem + 128 * i + 8 * e, smem_desc(base + L::v + (j & 1) * L::kOperand + e * 2048, kHalf), kO, j > 0 || e > 0);
        commit(bars + kOFull + 8 * i);
      };
      bool ok = bar_wait(bars + kQFull, 0, stop) && bar_wait(bars + kKFull, 0, stop);
      if (ok) {
        fence_after();
        scores(0, 0);
        scores(1, 0);
        commit(bars + kKEmpty);
      }
      for (uint32_t j = 0; ok && j < tiles; ++j) {
        const uint32_t buf = j & 1, nbuf = buf ^ 1;
        ok = bar_wait(bars + kVFull + 8 * buf, (j >> 1) & 1, stop) && bar_wait(bars + kPFull, j & 1, stop);
        if (!ok) break;
        fence_after();
        values(0, j);
        if (j + 1 < tiles) {
          ok = bar_wait(bars + kKFull + 8 * nbuf, ((j + 1) >> 1) & 1, stop);
          if (!ok) break;
          fence_after();
          scores(0, j + 1);
        }
        ok = bar_wait(bars + kPFull + 8, j & 1, stop);
        if (!ok) break;
        fence_after();
        values(1, j);
        commit(bars + kVEmpty + 8 * buf);
        if (j + 1 < tiles) {
          scores(1, j + 1);
          commit(bars + kKEmpty + 8 * nbuf);
        }
      }
      if (!ok) {
        // gave up: let the products in flight end (again with a limit) before TMEM goes back
        report(a.st, SHN_ERR_TIMEOUT, w.req);
        commit(bars + kDrain);
        for (uint32_t i = 0; i < kWaitTries && !bar_try(bars + kDrain, 0); ++i) {
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (tid == 0 && lds32(stop) != 0) report(a.st, SHN_ERR_TIMEOUT, w.req);
}

template <int D>
cudaError_t launch(const KvPages& c, const KvAttnArgs& a, cudaStream_t s) {
  // more shared memory than the default 48 KB: an attribute of the kernel on each device, so it is set for the one that
  // is current on every call
  cudaError_t e = cudaFuncSetAttribute(kv_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::total);
  if (e != cudaSuccess) return e;
  const uint64_t group = a.q_heads / c.kv_heads;
  // at most so many tiles, however the queries are spread over the requests
  const uint64_t tiles = (uint64_t)a.n_tokens * group / kRows + (a.n_reqs < a.n_tokens ? a.n_reqs : a.n_tokens);
  if (tiles * c.kv_heads >= (1ull << 31)) return cudaErrorInvalidConfiguration;
  kv_prompt_kernel<D><<<(uint32_t)(tiles * c.kv_heads), kThreads, Layout<D>::total, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_prompt(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, cudaStream_t s) {
  return head_dim == 128 ? launch<128>(c, a, s) : launch<64>(c, a, s);
}

}  // namespace shn
