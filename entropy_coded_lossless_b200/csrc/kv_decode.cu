// kv_decode.cu — attention of single tokens over the paged INT8 cache, with a prefix that the requests share
// (shn_kv_attn_shared).
//
// Bound by reading the cache: a token's keys and values of one key head are 2 (head_dim + 4) bytes, used by few rows. Each
// warp brings its own 16 tokens a step through a ring of stages in shared memory with cp.async, the next steps on their
// way while one is worked on, and no warp waits for another. With the order of the contracted dimension free (as long as
// both operands agree) a lane's 16 consecutive bytes are its operands of several mma.sync steps. Rows are the narrow side:
//   S' = K Q'   m16 (tokens) n8 (query rows) k16, 16 tokens a step
//   O' = V' P'  m16 (values of a head) n8 (query rows) k16 (the 16 tokens); P' is S' transposed by movmatrix
// INT8 enters as fp16, exactly (1024 + u with u = x + 128 is a byte put into fp16's last bits; minus 1152 it is x). A query row
// is scaled by a power of two into fp16, exactly but for parts 2^-25 of its largest. Scales meet the float32 scores: with
// x = s k_scale softmax_scale log2(e),
//   p = 2^(x - m),   l += p,   P = fp16(p v_scale 2^-E)   (2^-11, the one rounding before the sums)
// The reference m is raised only when a score passes it by 8, and E, the exponent the sums are held in, when a value scale
// is 2^7 above it (2^15 together, within fp16); then E is 5 below that scale's. Almost every step does without a reduction
// across lanes. What fp16 cannot hold of a token's part is 2^-25 of that range, so the sums are exact to n 2^-30 of the largest
// value of the n tokens that the row sees: in a shared prefix a step that holds the end of what some row sees is taken in parts
// that end there, so that a row's own tokens are summed before larger ones that it does not see raise E.
//
// Measured (32 query and 8 key heads of 128, 128 requests with 1024 own tokens each): 54 us for 282 MB, 5.2 TB/s, 80 % of
// the measured copy rate. The join then reads what the parts of the prefix and the pieces left for each row: 16 us.
#include <type_traits>

#include "kv_decode.cuh"
#include "kv_tc.cuh"

namespace shn {
namespace {

using namespace tc;

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// A warp's ring: stages of 16 tokens' keys, values and scales; two blocks of 8 warps to an SM.
template <int D>
struct Ring {
  static constexpr uint32_t kStages = D == 128 ? 3 : 6, kStage = 32 * D + 128, kBytes = kDecodeThreads / 32 * kStages * kStage;
};
// What a row's chunk numbers are XORed with. Rows of 128 bytes: the 8 lanes that read at a time have rows g, g + 1 and 4
// chunks of keys (the lowest bit of the row moves them to the other half), or rows 2 cc and chunks g, g + 1 of values (the
// other bits spread them). Rows of 64 bytes lie in pairs; only values meet a bank twice there.
template <int D>
__device__ __forceinline__ uint32_t chunk_swap(uint32_t tok) {
  return D == 128 ? (tok & 2) | (((tok >> 2) ^ tok) & 1) << 2 : tok >> 1 & 3;
}
__device__ __forceinline__ void cp16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(kDecodeThreads, NT == 1 ? 2 : 1) kv_decode_kernel(KvPages c, KvAttnArgs a, DecodePlan pl) {
  constexpr uint32_t kRows = 8 * NT;
  constexpr int kKLoads = D / 64;  // 16-byte loads of a token's keys per lane
  constexpr uint32_t kStages = Ring<D>::kStages, kStage = Ring<D>::kStage;
  __shared__ UnitScan scan;
  __shared__ uint32_t error;
  const uint32_t lane = threadIdx.x & 31, g = lane >> 2, cc = lane & 3;
  const uint32_t w = blockIdx.x * (kDecodeThreads / 32) + (threadIdx.x >> 5);
  const uint32_t group = a.q_heads / c.kv_heads;
  // Nothing here reads what the prefix's kernel writes, if there is one before; only the end of this kernel has to come after
  // it (the join is behind both).
  let_next();
  if (threadIdx.x == 0) error = kNoError;
  __syncthreads();
  bool bad;
  const int32_t prefix = decode_prefix(c, a, bad);
  if (bad && threadIdx.x == 0) error = 0;
  scan_units(c, a, prefix, scan, blockIdx.x == 0 ? &error : nullptr);

  const uint32_t prefix_units = pl.prefix_groups ? ((uint32_t)prefix + kUnit - 1) / kUnit : 0;
  const uint32_t prefix_segs = c.kv_heads * pl.prefix_groups, seg_per_req = c.kv_heads * pl.own_groups;
  const unsigned long long own0 = (unsigned long long)prefix_segs * prefix_units;
  const unsigned long long units = own0 + scan.before[kDecodeThreads] * seg_per_req;
  const Line line(units, pl.warps);
  unsigned long long u = line.first(w);
  const unsigned long long u_end = line.first(w + 1);

  // the segment of unit u
  uint32_t r = 0, sub = 0;              // request (own tokens) and segment within it; or the prefix segment
  unsigned long long seg0 = 0;          // its first unit
  bool own = false;
  if (u < u_end) {
    if (u < own0) {
      sub = (uint32_t)(u / prefix_units);
      seg0 = (unsigned long long)sub * prefix_units;
    } else {
      own = true;
      const unsigned long long v = u - own0;
      uint32_t lo = 0, hi = kDecodeThreads;
      while (hi - lo > 1) {
        const uint32_t m = (lo + hi) >> 1;
        if (scan.before[m] * seg_per_req <= v) lo = m; else hi = m;
      }
      const uint32_t run = (a.n_reqs + kDecodeThreads - 1) / kDecodeThreads;
      unsigned long long at = scan.before[lo] * seg_per_req;
      for (r = lo * run;; ++r) {
        const uint32_t n = own_units(prefix, decode_len(c, a, prefix, r, bad));
        if (v < at + (unsigned long long)n * seg_per_req) {
          sub = (uint32_t)((v - at) / n);
          seg0 = own0 + at + (unsigned long long)sub * n;
          break;
        }
        at += (unsigned long long)n * seg_per_req;
      }
    }
  }
  const float log2e_scale = a.scale * 1.44269504088896340736f;
  extern __shared__ __align__(128) uint8_t stages[];
  const uint32_t ring = smem_addr(stages) + (threadIdx.x >> 5) * kStages * kStage;
  uint32_t stage = 0;

  while (u < u_end) {
    // ---- a piece: units [u, piece_end) of one segment ----
    const uint32_t groups = own ? pl.own_groups : pl.prefix_groups;
    const uint32_t hk = sub / groups, row0 = sub % groups * kRows;
    const int32_t len = own ? decode_len(c, a, prefix, r, bad) : prefix;
    const uint32_t n_units = own ? own_units(prefix, len) : prefix_units;
    const unsigned long long piece_end = min(u_end, seg0 + n_units);
    const uint32_t origin = own ? own_start(prefix) : 0;
    const uint32_t t_first = origin + (uint32_t)(u - seg0) * kUnit;
    const uint32_t t_last = min((uint32_t)len, origin + (uint32_t)(piece_end - seg0) * kUnit);
    const int32_t t_from = own ? prefix : 0;
    const int32_t* pages = own ? a.table + (uint64_t)r * a.max_blocks : a.prefix_pages;

    // 16 tokens a step: the row of the first in the cache, ~0 where there is none (warp-uniform)
    auto page_of = [&](uint32_t t) -> int32_t { return t < t_last ? __ldg(pages + (t >> c.log2_pt)) : -1; };
    auto row_of = [&](uint32_t t, int32_t p) -> uint64_t {
      if (t >= t_last) return ~0ull;
      if (p < 0 || (uint32_t)p >= c.n_pages) {
        if (lane == 0) atomicMin(&error, r);
        return ~0ull;
      }
      return kv_row(c, (uint32_t)p, hk, t & ((1u << c.log2_pt) - 1));
    };
    // One step into a stage: rows in order, the 16-byte chunks of a row exchanged so that the lanes of a fragment load meet no
    // bank twice. Where there is no page the bytes stay what they were and the scales are zeros: scores of 0, values of 0.
    auto fetch = [&](uint32_t stage, uint64_t row) {
      const uint32_t at = ring + stage * kStage;
      if (row != ~0ull) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t x = i * 32 + lane, tok = x / (D / 16), chunk = x % (D / 16);
          const uint32_t to = tok * D + ((chunk ^ chunk_swap<D>(tok)) << 4);
          cp16(at + to, c.k + row * D + x * 16);
          cp16(at + 16 * D + to, c.v + row * D + x * 16);
        }
        if (lane < 8) cp16(at + 32 * D + lane * 16, (lane < 4 ? c.k_scale : c.v_scale) + row + (lane & 3) * 4);
      } else if (lane < 8) {
        sts128(at + 32 * D + lane * 16, make_uint4(0, 0, 0, 0));
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int32_t page_next;
    {
      int32_t first_pages[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) first_pages[i] = page_of(t_first + 16 * i);
      page_next = first_pages[kStages - 1];
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) fetch((stage + i) % kStages, row_of(t_first + 16 * i, first_pages[i]));
    }

    // queries: B operands. Lane (g, cc) holds row g's values 16 cc + 4 k + j (and 64 + ...) for step k
    uint32_t qb[NT][D / 16][2];
    float mul[NT][2];     // scale of query columns 2 cc, 2 cc + 1
    int32_t limit_at[NT][2];  // tokens they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t row = row0 + 8 * nt + g;
      const bool real = own ? row < group : row < a.n_reqs * group;
      const uint32_t req = own ? r : row / group, head = hk * group + (own ? row : row % group);
      uint2 v[D / 16];
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        v[k] = real ? *reinterpret_cast<const uint2*>(a.q + (uint64_t)req * a.q_stride + (uint64_t)head * D + (k / 4) * 64 + cc * 16 + (k % 4) * 4)
                    : make_uint2(0, 0);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t x = v[k].x & 0x7FFF7FFFu, y = v[k].y & 0x7FFF7FFFu;
        top = max(max(top, max(x & 0xFFFFu, x >> 16)), max(y & 0xFFFFu, y >> 16));
      }
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      // exponent of the row's largest, kept where its power of two and the inverse are normal
      const int32_t e = max(-100, min(126, (int32_t)(top >> 7) - 127));
      const float by = pow2((float)-e);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qb[nt][k][0] = fp16_pack(bf16_lo(v[k].x) * by, bf16_hi(v[k].x) * by);
        qb[nt][k][1] = fp16_pack(bf16_lo(v[k].y) * by, bf16_hi(v[k].y) * by);
      }
      int32_t sees = 0x7FFFFFFF;  // (nobody's rows hold no step back)
      if (real) sees = own ? len : min(prefix, decode_len(c, a, prefix, req, bad));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t src = (2 * cc + i) * 4;
        mul[nt][i] = log2e_scale * pow2((float)__shfl_sync(~0u, e, src));
        limit_at[nt][i] = __shfl_sync(~0u, sees, src);
      }
    }

    // steps from full_from on and below full_to need no mask
    int32_t least = limit_at[0][0];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) least = min(least, limit_at[nt][i]);
    const int32_t full_to = min((int32_t)t_last, __reduce_min_sync(~0u, least));

    float o[NT][D / 16][4], l[NT][2], m[NT][2], above[NT][2];  // above: m + 8
    float held = -200.f, ceiling = 0.f, unit = 0.f;            // E, 2^(E + 7), 2^-E
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) l[nt][i] = m[nt][i] = 0.f, above[nt][i] = -INFINITY;  // (a reference of 0 until there is one)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.f;
    }

    int32_t from = t_from;  // the first token that is not summed yet
    bool again = false;     // the rest of a step
#pragma unroll 1
    for (uint32_t t = t_first; t < t_last;) {
      if (!again) {
        // the step kStages - 1 ahead into the stage that the last step left
        const uint32_t ahead = t + 16 * (kStages - 1);
        fetch((stage + kStages - 1) % kStages, row_of(ahead, page_next));
        page_next = page_of(ahead + 16);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
      }
      const uint32_t at = ring + stage * kStage;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      // keys of tokens g, g + 8 -> scores
#pragma unroll
      for (int h = 0; h < kKLoads; ++h) {
        uint4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = lds128(at + (g + 8 * i) * D + (((h * 4 + cc) ^ chunk_swap<D>(g + 8 * i)) << 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t af[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t wd = (k == 0 ? x[i].x : k == 1 ? x[i].y : k == 2 ? x[i].z : x[i].w) ^ 0x80808080u;
            af[i] = minus1152(__byte_perm(wd, 0x64646464u, 0x4140));
            af[i + 2] = minus1152(__byte_perm(wd, 0x64646464u, 0x4342));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], af, qb[nt][h * 4 + k][0], qb[nt][h * 4 + k][1]);
        }
      }
      float ks[2], vs_now[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ks[i] = __uint_as_float(lds32(at + 32 * D + 4 * (g + 8 * i)));
        vs_now[i] = __uint_as_float(lds32(at + 32 * D + 64 + 4 * (g + 8 * i)));
      }
      // scores -> x: s[2 i + e] is token g + 8 i, query column 2 cc + e
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] *= ks[i >> 1] * mul[nt][i & 1];
      const bool edge = (int32_t)t < from || (int32_t)t + 16 > full_to;
      again = false;
      if (edge) {
        const int32_t begin = max(from, (int32_t)t);
        int32_t end = min((int32_t)t_last, (int32_t)t + 16);
        const int32_t step_end = end;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (limit_at[nt][e] > begin) end = min(end, limit_at[nt][e]);
        end = __reduce_min_sync(~0u, end);
        again = end < step_end;
        from = end;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int32_t tok = (int32_t)(t + g + 8 * i);
          const bool in = tok >= begin && tok < end;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!in || tok >= limit_at[nt][e]) s[nt][2 * i + e] = -INFINITY;
          if (!in) vs_now[i] = 0.f;  // what stands there is nobody's
        }
      }
      bool rise = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) rise |= fabsf(vs_now[i]) > ceiling && fabsf(vs_now[i]) < INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) rise |= fmaxf(s[nt][e], s[nt][2 + e]) > above[nt][e];
      if (__any_sync(~0u, rise)) {
        uint32_t big = 0;  // the largest finite value scale of the step
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (fabsf(vs_now[i]) < INFINITY) big = max(big, __float_as_uint(fabsf(vs_now[i])));
        big = __reduce_max_sync(~0u, big);
        float lower = 1.f;
        if (__uint_as_float(big) > ceiling) {
          const float to = (float)max(-126, min(121, (int32_t)(big >> 23) - 132));
          const float down = held - to;  // (in two steps: what a row has summed stays right even where it is not normal any more)
          lower = held < -150.f ? 0.f : pow2(fmaxf(down, -126.f)) * pow2(fmaxf(fminf(down + 126.f, 0.f), -126.f));
          held = to;
          ceiling = pow2(held + 7.f);
          unit = pow2(-held);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[nt][e], s[nt][2 + e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
            float keep = 1.f;
            if (x > above[nt][e]) {
              keep = above[nt][e] == -INFINITY ? 0.f : exp2_approx(m[nt][e] - x);
              m[nt][e] = x;
              above[nt][e] = x + 8.f;
            }
            l[nt][e] *= keep;
            keep *= lower;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) o[nt][k][e] *= keep, o[nt][k][2 + e] *= keep;
          }
      }
      uint32_t pb[NT][2];
      const float f[2] = {vs_now[0] * unit, vs_now[1] * unit};
      auto weights = [&](auto edge_tag) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = s[nt][2 * i + e];
              p[e] = exp2_approx(x - m[nt][e]);
              l[nt][e] += p[e];
              p[e] *= f[i];
              if constexpr (decltype(edge_tag)::value) p[e] = x == -INFINITY ? 0.f : p[e];  // (a scale may be infinite)
            }
            pb[nt][i] = transposed8x8(fp16_pack(p[0], p[1]));
          }
      };
      if (edge) weights(std::true_type{});
      else weights(std::false_type{});
      // values -> sums: a lane's bytes are values g D/8 + 2k, + 1 of step k, for tokens 2 cc, 2 cc + 1 (and + 8, + 9)
      uint32_t vr[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t tok = 2 * cc + (i & 1) + 8 * (i >> 1), byte = g * (D / 8);
        const uint32_t from = at + 16 * D + tok * D + ((((byte >> 4) ^ chunk_swap<D>(tok)) << 4) | (byte & 15));
        if constexpr (D == 128) {
          const uint4 x = lds128(from);
          vr[i][0] = x.x, vr[i][1] = x.y, vr[i][D / 32 - 2] = x.z, vr[i][D / 32 - 1] = x.w;
        } else {
          const uint2 x = lds64(from);
          vr[i][0] = x.x, vr[i][1] = x.y;
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t af[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = vr[2 * i][k / 2], y = vr[2 * i + 1][k / 2];
          const uint32_t b = 2 * (k & 1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t v = __byte_perm(x, y, (b + e) | (b + e) << 4 | (4 + b + e) << 8 | (4 + b + e) << 12);
            af[2 * i + e] = minus1152((v & 0x00FF00FFu) ^ 0x64806480u);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][k], af, pb[nt][0], pb[nt][1]);
      }
      if (again) continue;
      __syncwarp();  // the stage is read: the next turn may fill it
      stage = (stage + 1) % kStages;
      t += 16;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // (what was fetched ahead of the end is nothing)
    __syncwarp();

    // ---- the piece's result ----
    const uint32_t seg = own ? prefix_segs + r * seg_per_req + sub : sub;
    const uint64_t piece = (uint64_t)(w + seg) * kRows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = l[nt][e];
        const uint32_t row = 8 * nt + 2 * cc + e;
        if (own ? row0 + row >= group : row0 + row >= a.n_reqs * group) continue;  // nobody's row
        const uint64_t q = piece + row;
        float* dst = pl.out + q * D + g * (D / 8);
#pragma unroll
        for (int k = 0; k < D / 16; k += 2)
          *reinterpret_cast<float4*>(dst + 2 * k) = make_float4(o[nt][k][e], o[nt][k][2 + e], o[nt][k + 1][e], o[nt][k + 1][2 + e]);
        if (g == 0) pl.ml[q] = make_float4(held < -150.f ? -INFINITY : m[nt][e] + held, above[nt][e] == -INFINITY ? -INFINITY : m[nt][e], x, 0.f);
      }

    // ---- on to the next segment ----
    u = piece_end;
    if (u < u_end) {
      seg0 = u;
      if (!own) {
        if (++sub == prefix_segs) own = true, r = 0, sub = 0;
      } else if (++sub == seg_per_req) {
        sub = 0, ++r;
      }
      if (own)
        while (own_units(prefix, decode_len(c, a, prefix, r, bad)) == 0) ++r;  // ends: there are units left
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) pl.errors[pl.n_errors - gridDim.x + blockIdx.x] = error;
  if (pl.splits) after_previous();
}

// Joins the pieces of a row (request, head): kTeam warps to a row, lanes across its values.
template <int D, uint32_t kTeam>
__global__ void __launch_bounds__(kDecodeThreads) kv_join_kernel(KvPages c, KvAttnArgs a, DecodePlan pl) {
  constexpr uint32_t kWarps = kDecodeThreads / 32;
  __shared__ UnitScan scan;
  __shared__ float sum_o[kWarps][D], sum_m[kWarps], sum_l[kWarps];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t group = a.q_heads / c.kv_heads;
  if (blockIdx.x == gridDim.x - 1) {  // the call's status
    __shared__ uint32_t first;
    if (threadIdx.x == 0) first = kNoError;
    __syncthreads();
    after_previous();
    uint32_t least = kNoError;
    bool gave_up = false;
    for (uint32_t i = threadIdx.x; i < pl.n_errors; i += kDecodeThreads) {
      const uint32_t x = pl.errors[i];
      gave_up |= x == kGaveUp;
      least = min(least, x);
    }
    if (least < kGaveUp) atomicMin(&first, least);
    gave_up = __syncthreads_or(gave_up);
    if (threadIdx.x == 0) {
      a.st->status = gave_up ? SHN_ERR_TIMEOUT : first != kNoError ? SHN_ERR_INVALID_ARG : SHN_OK;
      a.st->detail = !gave_up && first != kNoError ? first : 0;
    }
    return;
  }
  bool bad;
  const int32_t prefix = decode_prefix(c, a, bad);
  scan_units(c, a, prefix, scan, nullptr);
  const uint32_t wanted = blockIdx.x * (kWarps / kTeam) + warp / kTeam, items = a.n_reqs * a.q_heads;
  const uint32_t item = min(wanted, items - 1);  // (no warp leaves: there is a barrier ahead)
  const uint32_t r = item / a.q_heads, head = item % a.q_heads, hk = head / group, g = head % group;
  const int32_t len = decode_len(c, a, prefix, r, bad);
  const uint32_t prefix_units = pl.prefix_groups ? ((uint32_t)prefix + kUnit - 1) / kUnit : 0;
  const uint32_t prefix_segs = c.kv_heads * pl.prefix_groups, seg_per_req = c.kv_heads * pl.own_groups;
  const unsigned long long own0 = (unsigned long long)prefix_segs * prefix_units;
  const unsigned long long units = own0 + scan.before[kDecodeThreads] * seg_per_req;

  const Line line(units, pl.warps);
  // the row's results, in this order: pieces of the prefix's segment, parts of the prefix, pieces of its own tokens' segment
  const uint32_t prow = r * group + g, psub = pl.prefix_groups ? hk * pl.prefix_groups + prow / pl.rows : 0;
  const uint32_t osub = hk * pl.own_groups + g / pl.rows;
  const uint32_t n = own_units(prefix, len);
  uint32_t pw = 0, pn = 0, ow = 0, on = 0;  // first warp and number of pieces
  if (prefix_units) {
    const unsigned long long u0 = (unsigned long long)psub * prefix_units;
    pw = line.warp_of(u0);
    pn = line.warp_of(u0 + prefix_units - 1) - pw + 1;
  }
  if (n) {
    const unsigned long long u0 = own0 + units_before(c, a, prefix, scan, r) * seg_per_req + (unsigned long long)osub * n;
    ow = line.warp_of(u0);
    on = line.warp_of(u0 + n - 1) - ow + 1;
  }
  const uint32_t all = pn + pl.splits + on;
  constexpr int E = D / 32;
  float o[E], l = 0.f, m = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  after_previous();
  // Each warp of the team takes its share of them in a row, 32 at a time: a lane finds one's place and reads its (mt, ms, l);
  // then all lanes add them up one after another.
  const uint32_t share_n = (all + kTeam - 1) / kTeam, k_end = min(all, share_n * (warp % kTeam + 1));
  for (uint32_t k0 = share_n * (warp % kTeam); k0 < k_end; k0 += 32) {
    const uint32_t k = k0 + lane;
    const float* src = nullptr;
    float4 x = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
    if (k < k_end) {
      const bool part = k >= pn && k < pn + pl.splits;
      if (part) {
        const uint64_t q = (uint64_t)(k - pn) * a.n_reqs * a.q_heads + item;
        src = pl.split_out + q * D;
        x = pl.split_ml[q];
      } else {
        const bool mine = k >= pn;
        const uint32_t w = mine ? ow + (k - pn - pl.splits) : pw + k;
        if (line.first(w) != line.first(w + 1)) {  // (there are warps without units)
          const uint64_t q = (uint64_t)(w + (mine ? prefix_segs + r * seg_per_req + osub : psub)) * pl.rows + (mine ? g : prow) % pl.rows;
          src = pl.out + q * D;
          x = pl.ml[q];
        }
      }
      if (x.y == -INFINITY && x.z == 0.f) src = nullptr;  // it saw nothing
    }
    float top = src ? x.y : -INFINITY;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (top > m) {
      const float keep = exp2_approx(m - top);
      l *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= keep;
      m = top;
    }
    float share = src ? x.z * exp2_approx(x.y - m) : 0.f;
    const float by = src && x.x != -INFINITY ? exp2_approx(x.x - m) : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) share += __shfl_xor_sync(~0u, share, d);
    l += share;
    const uint32_t have = __ballot_sync(~0u, src != nullptr);
    const uint32_t last = min(32u, k_end - k0);
#pragma unroll 8
    for (uint32_t i = 0; i < last; ++i) {
      const float* from = reinterpret_cast<const float*>(__shfl_sync(~0u, (unsigned long long)src, i));
      const float f = __shfl_sync(~0u, by, i);
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
      if (have >> i & 1) {
        if constexpr (E == 4) {
          const float4 x4 = reinterpret_cast<const float4*>(from)[lane];  // (written while this kernel may have run: no __ldg)
          v[0] = x4.x, v[1] = x4.y, v[E - 2] = x4.z, v[E - 1] = x4.w;
        } else {
          const float2 x2 = reinterpret_cast<const float2*>(from)[lane];
          v[0] = x2.x, v[1] = x2.y;
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(v[e], f, o[e]);
    }
  }
  if constexpr (kTeam > 1) {
    if (lane == 0) sum_m[warp] = m, sum_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) sum_o[warp][lane * E + e] = o[e];
    __syncthreads();
    if (warp % kTeam) return;
#pragma unroll
    for (uint32_t i = 1; i < kTeam; ++i) m = fmaxf(m, sum_m[warp + i]);
    const float own = sum_m[warp] == -INFINITY ? 0.f : exp2_approx(sum_m[warp] - m);
    l *= own;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= own;
#pragma unroll
    for (uint32_t i = 1; i < kTeam; ++i) {
      const float f = sum_m[warp + i] == -INFINITY ? 0.f : exp2_approx(sum_m[warp + i] - m);
      l = fmaf(sum_l[warp + i], f, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(sum_o[warp + i][lane * E + e], f, o[e]);
    }
  }
  if (wanted >= items) return;
  uint16_t* dst = a.out + (uint64_t)r * a.out_stride + (uint64_t)head * D + lane * E;
  const float inv = len > 0 ? 1.f / l : 0.f;  // (a sum of 0 although tokens were seen: every score was -infinity, the result is NaN)
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = len > 0 ? bf16_pack(o[e] * inv, o[e + 1] * inv) : 0u;
}

template <int D>
cudaError_t launch(const KvPages& c, const KvAttnArgs& a, const DecodePlan& pl, cudaStream_t s) {
  const dim3 blocks(pl.warps / (kDecodeThreads / 32));
  const auto kernel = pl.rows == 8 ? kv_decode_kernel<D, 1> : kv_decode_kernel<D, 2>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kBytes);
  if (e != cudaSuccess) return e;
  e = pl.splits ? launch_behind(kernel, blocks, kDecodeThreads, Ring<D>::kBytes, s, c, a, pl)
                : launch_first(kernel, blocks, kDecodeThreads, Ring<D>::kBytes, s, c, a, pl);
  if (e != cudaSuccess) return e;
  // Few rows may have hundreds of pieces each, many rows only a few. A row gets 2, 4 or 8 warps while fewer than that share of
  // the decoding warps' number is asked for: so the join has about the warps that the decode had, up to twice as many.
  // Measured: 128 rows, a call 11.5 us against 21.6 with one warp to a row; 792 rows 25.2, one warp 33.8, eight 27.6; 4096
  // rows 126 (one warp), eight 145.
  const uint64_t rows = (uint64_t)a.n_reqs * a.q_heads;
  const uint32_t n = (uint32_t)rows;
  // (one block more, for the status)
  if (rows > pl.warps) return launch_behind(kv_join_kernel<D, 1>, dim3((n + 7) / 8 + 1), kDecodeThreads, 0, s, c, a, pl);
  if (2 * rows > pl.warps) return launch_behind(kv_join_kernel<D, 2>, dim3((n + 3) / 4 + 1), kDecodeThreads, 0, s, c, a, pl);
  if (4 * rows > pl.warps) return launch_behind(kv_join_kernel<D, 4>, dim3((n + 1) / 2 + 1), kDecodeThreads, 0, s, c, a, pl);
  return launch_behind(kv_join_kernel<D, 8>, dim3(n + 1), kDecodeThreads, 0, s, c, a, pl);
}

}  // namespace

cudaError_t launch_kv_decode(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, const DecodePlan& pl, cudaStream_t s) {
  return head_dim == 128 ? launch<128>(c, a, pl, s) : launch<64>(c, a, pl, s);
}

}  // namespace shn
