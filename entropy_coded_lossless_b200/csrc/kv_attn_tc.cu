// kv_attn_tc.cu — attention of many query rows over the paged INT8 cache on the tensor cores: packed causal
// prompts (shn_kv_attn_prompt), and parts of a prefix that many single-token requests share (shn_kv_attn_shared).
//
// A block takes 256 rows of one key head: row = (query, head of the group), so every key and value it reads serves all
// heads of the group, whatever their number. It walks the sequence in tiles of 128 tokens:
//   S = Q K^T      tcgen05.mma, fp16, M = 128 rows, N = 64 tokens, for rows 0-127 and 128-255 and both halves, into TMEM
//   s = S * k_scale_j * softmax_scale * log2(e);  p = 2^(s - m);  l += p;  P = fp16(p)
//   O += P V       tcgen05.mma, fp16, P read from TMEM (it takes the place of S)
// Queries enter with one power of two for the block taken out, which fp16 then holds exactly down to 2^-32 of the largest;
// keys as the integers, and their scales are applied to the float32 scores: scores have float32's error. Values enter as
// fp16(int8 * fp16(v_scale * 2^-e)), e the exponent of the largest value scale of 32 tokens; weights, values and their
// scales are rounded to fp16's 11 bits each (with bf16's 8 the results, rounded to bf16 themselves, were off by 0.0024 instead
// of 0.0017 in the mean). The power of two goes into the weights: P = p 2^(e - E), with E the exponent a row's O is held in: 6 below
// that of the largest value scale it has seen, and raised like the softmax's reference when one is more than 2^6 larger. What
// fp16 cannot hold of a weight is 2^-25 of that range, so O is exact to n 2^-30 + 2^-24 of the largest value of the n tokens that
// the row sees.
// Tokens that a row does not see are nothing to it, whatever their size. So a tile that some row of the block does not see whole
// has the integers as values and the scales on the float32 weights, P = fp16(p * v_scale 2^-E), and each row's E is of what it sees.
// (All tiles that way would round once for three times: the mean error stays 0.0017, 8192 tokens take 761 us a call instead
// of 663.)
//
// Softmax in one pass over the scores, without a search for the maximum: m is the maximum of a row's first 64 scores, and a
// thread's sum of 16 weights shows whether one of the later ones is above it by 2^8; only then m is raised, and what is
// summed scaled down. Sums of weights are float32.
//
// Roles (896 threads): warps 0-7 and 8-15 the softmax of the two row tiles (16 rows to a warp, so that each scheduler
// has four of them to hide their latencies), warps 16-23 fetch the tiles and turn INT8 into fp16 operands in shared memory,
// warps 24 and 25 issue the products of a row tile each. Two K and two V buffers; the next operand's bytes are on their
// way in registers while the present one is converted. TMEM (512 columns): O0, O1 (D each) and for each row tile 128
// columns in which a tile's two halves of S, the weights in their place and the next tile's first half take turns.
//
// Where a call has too few rows to fill the SMs, up to 8 blocks of a cluster share a row tile's tokens and join their sums in
// each other's shared memory (join_parts): no workspace, no second launch.
//
// What bounds it. 8192 causal tokens, 32 query and 8 key heads of 128: 663 us in a run of calls, 829 TFLOP/s, 50 % of the
// measured bf16 rate (598 us and 56 % for the call alone in a graph). A tile of 256 x 128 scores costs a block about 4400
// cycles; the products would take 2048 of them (1024 at D = 64) and so would the exponentials, at 16 a cycle; issuing the
// instructions of softmax, conversion and waits takes some 3000 of each scheduler. So the softmax sets the pace, by its
// instructions and their latency, and products and fetches run behind it.
// The steps, same case: a thread per row with its 128 scores in registers 1458 us; a row shared by four threads, so that a
// column's scale is read for two rows, 1193; 16 softmax warps 759; two issuing warps, halves with scores formed ahead and no
// search for the maximum 716; whole lines out and a shorter block start 690; tiles in front of the edge in a loop of their
// own 663. Tried and not kept: 8 softmax warps of 32 rows, and blocks of all requests in the order of their lengths.
#include <type_traits>

#include "kv_decode.cuh"
#include "kv_tc.cuh"

namespace shn {
namespace {

using namespace tc;

constexpr uint32_t kSoftWarps = 16, kConvertWarps = 8;
constexpr uint32_t kSoftThreads = 32 * kSoftWarps;
constexpr uint32_t kIssueWarp = kSoftWarps + kConvertWarps;  // in a warpgroup of its own
constexpr uint32_t kThreads = 32 * (kIssueWarp + 4);
constexpr uint32_t kTile = 128;      // tokens of a tile
constexpr uint32_t kRows = 256;      // query rows of a block
constexpr float kRise = 256.f;       // how far a weight may pass 1 before the reference is raised,
constexpr float kValueRise = 6.f;    // and (log2) the exponent of a value scale E: with the scale's own factor 2^15, within fp16
constexpr float kValueFall = -60.f, kValueFall2 = 1ull << 60;  // a tile this far below adds nothing to O in fp16
constexpr float kValueClimb = 110.f, kValueClimb2 = 0x1p-110f;  // 32 tokens may be above E as a whole: those that the row does not see
constexpr uint32_t kHalf = 128 * 128;  // bytes of 128 rows of 64 fp16

template <int D>
struct Layout {
  static constexpr uint32_t kOperand = 128 * D * 2;  // one 128 x D fp16 operand
  static constexpr uint32_t q = 0, k = 2 * kOperand, v = 4 * kOperand, scale = 6 * kOperand, info = scale + 4 * 1024, row_sum = info + 128, bars = row_sum + 12 * kRows, misc = bars + 256, scan = misc + 64, total = scan + 192;
};
// barriers
enum : uint32_t { kQFull = 0, kKFull = 8, kKEmpty = 24, kVFull = 40, kVEmpty = 56, kScaleFull = 72, kSFull = 104, kPFull = 136, kOFull = 168, kDrain = 200 };

struct Work {
  uint32_t req, row0, rows;  // request, first row of the block within it, rows of the request
  int32_t q0;                // first query of the request
  int32_t len, nq;           // its tokens and queries
  uint32_t t0;               // first token (in pages) of the block's part of the sequence
};

// In front of the others, which start beside it: what is wrong with the requests' ranges and lengths into the status. (Asked by every
// block of the kernel that follows, it cost a call of three short prompts 2 us of 16 and one of 8192 tokens 20 us of 690.)
__global__ void kv_prompt_begin_kernel(KvPages c, KvAttnArgs a) {
  let_next();
  __shared__ uint32_t least[32];
  const uint32_t t = threadIdx.x;
  const int64_t holds = (int64_t)a.max_blocks << c.log2_pt;
  uint32_t first = kNoError;
  for (uint32_t r = t; r < a.n_reqs; r += blockDim.x) {
    const int32_t b = a.cu_q[r], e = a.cu_q[r + 1], len = a.kv_len[r];
    if (b < 0 || e < b || (uint32_t)e > a.n_tokens || (e > b && (len < 0 || len > holds))) first = min(first, r);
  }
  first = __reduce_min_sync(~0u, first);
  if ((t & 31) == 0) least[t >> 5] = first;
  __syncthreads();
  if (t) return;
  for (uint32_t i = 1; i < blockDim.x / 32; ++i) first = min(first, least[i]);
  a.st->status = first == kNoError ? SHN_OK : SHN_ERR_INVALID_ARG;
  a.st->detail = first == kNoError ? 0 : first;
}

// Which request's rows a block takes: tiles of 256 rows, request after request, the last tile first (a
// prompt's last rows see the most tokens, and long blocks belong in front). False: no such tile.
__device__ __forceinline__ bool find_work(const KvPages& c, const KvAttnArgs& a, uint32_t group, uint32_t tile_from_end,
                                          uint32_t* scan, Work& w, uint32_t& status) {
  // The status as the kernel in front left it, asked for behind the first loads: both are on their way together.
  auto look = [&] {
    after_previous();
    status = *reinterpret_cast<volatile uint32_t*>(&a.st->status);
  };
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int32_t len;
  if (a.n_reqs <= 32) {
    // every warp finds it by itself, a request to a lane
    const bool is = lane < a.n_reqs;
    const int32_t b = is ? a.cu_q[lane] : 0, e = is ? a.cu_q[lane + 1] : 0;
    len = is ? a.kv_len[lane] : 0;
    look();
    const bool bad = b < 0 || e < b || (uint32_t)e > a.n_tokens;
    const uint32_t own = bad ? 0 : ((uint32_t)(e - b) * group + kRows - 1) / kRows;
    uint32_t inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, inc, d);
      if (lane >= (uint32_t)d) inc += x;
    }
    const uint32_t total = __shfl_sync(~0u, inc, 31);
    if (tile_from_end >= total) return false;
    const uint32_t tile = total - 1 - tile_from_end;
    w.req = __ffs(__ballot_sync(~0u, tile < inc)) - 1;  // the first whose tiles reach it
    w.row0 = (tile - __shfl_sync(~0u, inc - own, w.req)) * kRows;
    w.q0 = __shfl_sync(~0u, b, w.req);
    w.nq = __shfl_sync(~0u, e, w.req) - w.q0;
    len = __shfl_sync(~0u, len, w.req);
    w.rows = (uint32_t)w.nq * group;
  } else {
    const uint32_t run = (a.n_reqs + kThreads - 1) / kThreads;
    const uint32_t r0 = min(a.n_reqs, t * run), r1 = min(a.n_reqs, r0 + run);
    uint32_t own = 0;
    int32_t kv_len = 0;  // of the run's last request: with up to kThreads requests the one that is meant
    for (uint32_t r = r0; r < r1; ++r) {
      const int32_t b = a.cu_q[r], e = a.cu_q[r + 1];
      kv_len = a.kv_len[r];
      if (b >= 0 && e >= b && (uint32_t)e <= a.n_tokens) own += ((uint32_t)(e - b) * group + kRows - 1) / kRows;
    }
    look();
    uint32_t inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, inc, d);
      if (lane >= (uint32_t)d) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    if (t == 0) scan[30] = 0xFFFFFFFFu;
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
          scan[28] = (uint32_t)b;
          scan[29] = (uint32_t)(e - b);
          scan[30] = r;
          scan[31] = left;
          scan[32] = (uint32_t)(run == 1 ? kv_len : a.kv_len[r]);
          break;
        }
        left -= n;
      }
    }
    __syncthreads();
    w.req = scan[30];
    if (w.req >= a.n_reqs) return false;
    w.row0 = scan[31] * kRows;
    w.q0 = (int32_t)scan[28];
    w.nq = (int32_t)scan[29];
    w.rows = (uint32_t)w.nq * group;
    len = (int32_t)scan[32];
  }
  const int64_t holds = (int64_t)a.max_blocks << c.log2_pt;
  w.len = len < 0 ? 0 : len > holds ? (int32_t)holds : len;
  w.t0 = 0;
  return true;
}

// The same for a part of a shared prefix: blockIdx = (key head, tile of 256 rows, split), rows = (request, head of the group),
// tokens = the split's tiles of the prefix.
__device__ __forceinline__ void find_part(const KvPages& c, const KvAttnArgs& a, const DecodePlan& pl, uint32_t group, Work& w) {
  bool bad;
  const int32_t prefix = decode_prefix(c, a, bad);
  const uint32_t tiles = ((uint32_t)prefix + kTile - 1) / kTile;
  const uint32_t rest = blockIdx.x / c.kv_heads, split = rest % pl.splits;
  w.req = 0, w.q0 = 0, w.nq = (int32_t)a.n_reqs;
  w.row0 = rest / pl.splits * kRows;
  w.rows = a.n_reqs * group;
  w.t0 = (uint32_t)((uint64_t)split * tiles / pl.splits) * kTile;
  w.len = min(prefix, (int32_t)((uint64_t)(split + 1) * tiles / pl.splits * kTile)) - (int32_t)w.t0;
}

// A sequence's tiles over the blocks of a cluster. Joining costs about as much as a tile, so three tiles stay with one block (4
// requests of 55 to 262 tokens 17.1 us, 18.8 when they are shared) and from four on a block may have one (3 requests of 83 to
// 673 tokens 17.1 us; 19.2 with two tiles to a block at least, 21.8 with all in one).
__device__ __forceinline__ uint32_t parts_of(uint32_t tiles, uint32_t most) { return tiles > 3 ? min(most, tiles) : 1; }
__device__ __forceinline__ uint32_t first_tile(uint32_t tiles, uint32_t parts, uint32_t rank) { return min(rank, parts) * tiles / parts; }

// The parts' sums, sums of weights l, references m and exponents E of their rows lie in their blocks' shared memory. Each block of
// the cluster joins 256 / ranks rows, a warp 16 / ranks of them, half of these at a time: 8 loads of 32 lanes (a row of a block
// each) are on their way together.
//   out = sum O_i 2^(m_i - m + E_i - E) 2^E / sum l_i 2^(m_i - m)
template <int D, typename F>
__device__ __forceinline__ void join_parts(uint32_t base, uint32_t ranks, uint32_t parts, uint32_t tiles, uint32_t rank, uint32_t warp,
                                           uint32_t lane, F put) {
  using L = Layout<D>;
  const uint32_t mask = ranks - 1, log2 = 31 - __clz(ranks), each = 8 >> log2;  // rows at a time
  const uint32_t from = lane & mask;  // the block whose row a lane looks at: row (lane & 7) >> log2
  const bool has = first_tile(tiles, parts, from + 1) > first_tile(tiles, parts, from);
#pragma unroll 1
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t row0 = rank * (kRows >> log2) + (warp * 2 + i) * each, row = row0 + ((lane & 7) >> log2);
    float l = 0.f, m = -INFINITY, size = -INFINITY;
    if (has) {
      l = __uint_as_float(ld_cluster32(base + L::row_sum + 4 * row, from));
      m = __uint_as_float(ld_cluster32(base + L::row_sum + 4 * (kRows + row), from));
      size = m == -INFINITY ? m : __uint_as_float(ld_cluster32(base + L::row_sum + 4 * (2 * kRows + row), from));  // (no sums: no range)
    }
    uint4 v[8];
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      const uint32_t r = row0 + (e >> log2), of = e & mask;
      v[e] = make_uint4(0, 0, 0, 0);
      if (first_tile(tiles, parts, of + 1) > first_tile(tiles, parts, of)) {
        if constexpr (D == 128) {
          v[e] = ld_cluster128(base + L::q + r * 512 + ((lane ^ (r & 7)) << 4), of);
        } else {
          const uint2 x = ld_cluster64(base + L::q + r * 256 + (((lane >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8, of);
          v[e].x = x.x, v[e].y = x.y;
        }
      }
    }
    float top = m, held = size;
    for (uint32_t d = 1; d < ranks; d <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      held = fmaxf(held, __shfl_xor_sync(~0u, held, d));
    }
    float by = exp2_approx(m - top);
    float sum = has ? l * by : 0.f;
    by = has ? exp2_approx(m - top + (size - held)) : 0.f;
    for (uint32_t d = 1; d < ranks; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
    const float inv = pow2(held) / sum;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      const float f = __shfl_sync(~0u, by, e), g = __shfl_sync(~0u, inv, e);
      o[0] = fmaf(__uint_as_float(v[e].x), f, o[0]), o[1] = fmaf(__uint_as_float(v[e].y), f, o[1]);
      o[2] = fmaf(__uint_as_float(v[e].z), f, o[2]), o[3] = fmaf(__uint_as_float(v[e].w), f, o[3]);
      if ((e & mask) == mask) {
        put(row0 + (e >> log2), o, g);
        o[0] = o[1] = o[2] = o[3] = 0.f;
      }
    }
  }
}

// kSplit (grids of no more blocks than SMs): pl.splits blocks of a cluster, or one, share the tokens of 256 rows, and the rows
// of the result (join_parts).
template <int D, bool kPart, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(KvPages c, KvAttnArgs a, DecodePlan pl) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Layout<D>;
  const uint32_t base = smem_addr(smem), bars = base + L::bars, stop = base + L::misc;
  // Roles are counted from the second warpgroup on: the issuing warp is the block's first, which the schedulers serve
  // before younger ones.
  const uint32_t lane = threadIdx.x & 31, warp = ((threadIdx.x >> 5) + kIssueWarp) % (kThreads / 32), tid = warp * 32 + lane;
  const uint32_t place = kSplit ? blockIdx.x / pl.splits : blockIdx.x, rank = kSplit ? blockIdx.x % pl.splits : 0;
  const uint32_t group = a.q_heads / c.kv_heads, hk = place % c.kv_heads;

  Work w;
  uint32_t status = 0;
  if constexpr (kPart) {
    let_next();  // the call's first kernel
    find_part(c, a, pl, group, w);
  } else {  // the last: only the status is the other one's
    if (!find_work(c, a, group, place / c.kv_heads, reinterpret_cast<uint32_t*>(smem + L::scan), w, status)) return;
  }
  const uint32_t rows_here = min(kRows, w.rows - w.row0);
  // tokens the block's last row sees; every row of the block sees at most as many
  // row i of the block is query base_q + x and head y of the group, x = (rest + i) / group: with i + rest < 320 and group <= 64 that
  // is a multiplication by 2^16 / group, rounded up
  const uint32_t base_q = w.row0 / group, rest = w.row0 - base_q * group, inv_group = (65536u + group - 1) / group;
  auto query_of = [&](uint32_t i, uint32_t& head) -> uint32_t {
    const uint32_t x = ((rest + i) * inv_group) >> 16;
    head = rest + i - x * group;
    return base_q + x;
  };
  const int32_t shift = w.len - w.nq + 1;  // query i sees shift + i tokens
  int32_t most = kPart ? max(0, w.len) : max(0, min(w.len, shift + (int32_t)((w.row0 + rows_here - 1) / group)));
  uint32_t tiles = ((uint32_t)most + kTile - 1) / kTile;
  const uint32_t all_tiles = tiles;
  const uint32_t parts = kSplit ? parts_of(all_tiles, pl.splits) : 1;
  if constexpr (kSplit) {
    if (parts == 1 && rank > 0) return;  // (with one part no block waits for another or looks at its memory)
    if (parts > 1) {
      const uint32_t first = first_tile(all_tiles, parts, rank);
      tiles = first_tile(all_tiles, parts, rank + 1) - first;
      w.t0 = first * kTile;
      most = max(0, min(most - (int32_t)w.t0, (int32_t)(tiles * kTile)));
    }
  }

  if (tid == 0) {
    bar_init(bars + kQFull, kSoftThreads);
    bar_init(bars + kDrain, 1);
    bar_init(bars + kDrain + 8, 1);
    for (uint32_t i = 0; i < 2; ++i) {
      bar_init(bars + kKFull + 8 * i, kConvertWarps);
      bar_init(bars + kKEmpty + 8 * i, 2);
      bar_init(bars + kVFull + 8 * i, kConvertWarps);
      bar_init(bars + kVEmpty + 8 * i, 2);
      bar_init(bars + kSFull + 16 * i, 1);
      bar_init(bars + kSFull + 16 * i + 8, 1);
      bar_init(bars + kPFull + 16 * i, kSoftWarps / 2);
      bar_init(bars + kPFull + 16 * i + 8, kSoftWarps / 2);
      bar_init(bars + kOFull + 16 * i, 1);
      bar_init(bars + kOFull + 16 * i + 8, 1);
    }
    for (uint32_t i = 0; i < 4; ++i) bar_init(bars + kScaleFull + 8 * i, kConvertWarps);
    sts32(stop, 0);
    sts32(base + L::misc + 8, 0);
    sts32(base + L::misc + 12, 0x7FFFFFFFu);
    sts32(base + L::misc + 16, kNoError);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(stop + 4) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  // after a wait that gave up the call has failed: the other blocks do not start on it
  const bool failed = __syncthreads_or(status == SHN_ERR_TIMEOUT);
  fence_after();
  if (kSplit && parts > 1) {
    if (failed) tiles = 0;  // (the cluster's barriers need every block)
  } else if (failed) {
    if (warp == kIssueWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(lds32(stop + 4)));
    return;
  }
  // all 512 columns are this block's, so its addresses begin at 0 (nothing that follows has to carry the base)
  const uint32_t tmem = 0;
  if (lds32(stop + 4) != 0) sts32(stop, 1);

  if (warp < kSoftWarps) {
    // ---- softmax -------------------------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    // A warp has 16 rows (TMEM lanes); a thread has two of them, `quad` and quad + 8, and of each 8 columns two: a column's
    // scales, read from shared memory, serve two rows, and a row's maximum is two shuffles away.
    const uint32_t half = warp >> 3;  // which 128 rows
    const uint32_t lanes = (warp & 3) * 32 + (warp & 4) * 4, quad = lane >> 2, col = 2 * (lane & 3);
    const uint32_t at = tmem + (lanes << 16);
    const uint32_t s_at = at + half * 128, o_at = at + 256 + half * D;
    auto seen_by = [&](uint32_t row) -> int32_t {
      if (row >= rows_here) return 0;
      uint32_t head;
      const uint32_t q = query_of(row, head);
      if constexpr (kPart) {
        bool bad;
        return max(0, min(w.len, decode_len(c, a, (int32_t)w.t0 + w.len, q, bad) - (int32_t)w.t0));
      }
      if constexpr (kSplit) return max(0, min(most, min(w.len, shift + (int32_t)q) - (int32_t)w.t0));
      return max(0, min(w.len, shift + (int32_t)q));
    };
    // the queries of the block as an operand, zeros behind the last row
    const uint16_t* q_src = a.q + (uint64_t)w.q0 * a.q_stride + (uint64_t)hk * group * D;
    uint4 qx[kRows * D / 8 / kSoftThreads];  // all loads first: one wait for them
#pragma unroll
    for (uint32_t i = 0; i < kRows * D / 8 / kSoftThreads; ++i) {
      const uint32_t at = tid + i * kSoftThreads, row = at / (D / 8), piece = at % (D / 8);
      uint32_t head;
      const uint32_t query = query_of(row, head);
      qx[i] = make_uint4(0, 0, 0, 0);
      if (row < rows_here) qx[i] = *reinterpret_cast<const uint4*>(q_src + (uint64_t)query * a.q_stride + head * D + piece * 8);
    }
    int32_t seen[2];  // (rows behind the last one: all tokens); from here to the edge's tiles in shared memory
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t row = half * 128 + lanes + quad + 8 * r;
      seen[r] = row < rows_here ? seen_by(row) : 0x7FFFFFFF;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if ((lane & 3) == 0) sts32(base + L::row_sum + 4 * (half * 128 + lanes + quad + 8 * r), (uint32_t)seen[r]);
    const int32_t least_seen = __reduce_min_sync(~0u, min(seen[0], seen[1]));
    if (lane == 0) atomicMin(reinterpret_cast<int32_t*>(smem + L::misc + 12), least_seen);
    // One power of two brings the block's largest query value just below 2^15; fp16 then holds every bf16 down to 2^-32
    // of it exactly. (Values that are not finite set no size and stay what they are.)
    uint32_t top2 = 0;
#pragma unroll
    for (uint32_t i = 0; i < kRows * D / 8 / kSoftThreads; ++i) {
      top2 = __vmaxu2(__vmaxu2(top2, qx[i].x & 0x7FFF7FFFu), qx[i].y & 0x7FFF7FFFu);
      top2 = __vmaxu2(__vmaxu2(top2, qx[i].z & 0x7FFF7FFFu), qx[i].w & 0x7FFF7FFFu);
    }
    uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    if (top >= 0x7F80u) {
      top = 0;
#pragma unroll
      for (uint32_t i = 0; i < kRows * D / 8 / kSoftThreads; ++i) {
        const uint32_t x[4] = {qx[i].x, qx[i].y, qx[i].z, qx[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = x[e] & 0x7FFFu, hi = x[e] >> 16 & 0x7FFFu;
          top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
        }
      }
    }
    top = __reduce_max_sync(~0u, top);
    if (lane == 0) atomicMax(reinterpret_cast<uint32_t*>(smem + L::misc + 8), top);
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
    const int32_t q_exp = max(-100, (int32_t)(lds32(base + L::misc + 8) >> 7) - 127) - 14;  // of the power of two taken out
    const float down = pow2i(-q_exp);
#pragma unroll
    for (uint32_t i = 0; i < kRows * D / 8 / kSoftThreads; ++i) {
      const uint32_t at = tid + i * kSoftThreads, row = at / (D / 8), piece = at % (D / 8);
      const uint32_t x[4] = {qx[i].x, qx[i].y, qx[i].z, qx[i].w};
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fp16_pack(bf16_lo(x[e]) * down, bf16_hi(x[e]) * down);
      sts128(base + L::q + (row / 128) * L::kOperand + (piece / 8) * kHalf + swizzled(row % 128, piece % 8), make_uint4(y[0], y[1], y[2], y[3]));
    }
    fence_smem();
    bar_arrive(bars + kQFull);

    // Tiles that all rows of the block see whole come first: all rows hold their sums in the same range (held[0]), and no column's
    // place is looked at. In the others a row has its own. What only those need is kept out of the first ones' registers (8192
    // tokens 640 -> 598 us).
    const uint32_t whole = min(tiles, lds32(base + L::misc + 12) / kTile);
    float m[2], l[2];
    float neg[2];    // minus the reference (0 while there is none)
    float limit[2];  // how large a sum of weights may be before it is raised
    float held[2] = {-300.f, -300.f}, held2[2] = {1.f, 1.f};  // E and 2^E: a row's O is in units of it (none yet)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m[r] = -INFINITY, l[r] = 0.f, neg[r] = 0.f, limit[r] = seen[r] ? -1.f : INFINITY;  // (no reference yet: any sum passes)
    }
    // A warp whose rows are all behind the last one keeps step and does no more: its places in TMEM hold anything, and so do
    // these rows' sums, which nobody reads (one query after 5102 tokens 29.6 -> 25.8 us, 24 short requests 14.4 -> 12.8). Not for
    // full grids, whose blocks have few such rows: there the question alone costs 7 % (8192 tokens 627 -> 673 us).
    const bool skip = kSplit && half * 128 + lanes >= rows_here;
    bool ok = true;
    // Half a tile (64 tokens) at a time. The first half's scores lie in the 64 columns `here`, the second's in the other 64; both
    // halves' weights go into `here` (32 columns each). So the columns of the second half are free as soon as its scores
    // are in registers, and the next tile's first half is put there while this one is still worked on: next to no scores are
    // ever waited for. `grows`: some row's range may have to be raised (the same in all threads of the warp).
    auto half_tile = [&](auto edge_tag, uint32_t j, int h, uint32_t info, bool grows) {
      constexpr bool kEdge = decltype(edge_tag)::value;
      const uint32_t here = s_at + (j & 1) * 64;
      ok = __all_sync(~0u, bar_wait(bars + kSFull + 16 * half + 8 * h, j & 1, stop));
      if (!ok) return;
      if (skip) {  // (see above)
        if (lane == 0 && h == 1) bar_arrive(bars + kPFull + 16 * half);
        return;
      }
      fence_after();
      // s[4n + 2r + e]: row quad + 8r, column 64h + 8n + col + e
      uint32_t s[32];
      ld_quad32(s_at + ((j + h) & 1) * 64, s);
      wait_ld();
      if (h == 1) {
        // the first half's weights are stored and the second's scores loaded
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bars + kPFull + 16 * half);
      }
      const uint32_t scales = after_here(base + L::scale + (j & 3) * 1024 + h * 256 + 4 * col);
      const int32_t first = (int32_t)(j * kTile + 64 * h + col);
      bool rise = j == 0 && h == 0;  // (there is no reference yet)
      float lower[2] = {1.f, 1.f};   // what O is scaled by
      if (grows) {
        float top[2];  // (log2) the largest value scale of the tile, or of what the row sees of the half
        if constexpr (!kEdge) {
          const uint4 sizes = lds128(info);
          top[0] = top[1] = fmaxf(fmaxf(__uint_as_float(sizes.x), __uint_as_float(sizes.y)), fmaxf(__uint_as_float(sizes.z), __uint_as_float(sizes.w)));
        } else {
          float most_v[2] = {0.f, 0.f};
#pragma unroll 2
          for (int n = 0; n < 8; ++n) {
            float x, y;
            unpack2(lds64_free(scales + 512 + 32 * n), x, y);
            const float unit = pow2(lds32_free(info + 8 * h + 4 * (n >> 2)));
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (first + 8 * n < seen[r]) most_v[r] = fmaxf(most_v[r], fabsf(x) * unit);
              if (first + 8 * n + 1 < seen[r]) most_v[r] = fmaxf(most_v[r], fabsf(y) * unit);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            most_v[r] = fmaxf(most_v[r], __shfl_xor_sync(~0u, most_v[r], 1));
            most_v[r] = fmaxf(most_v[r], __shfl_xor_sync(~0u, most_v[r], 2));
            top[r] = (float)((int32_t)(__float_as_uint(most_v[r]) >> 23) - 127);
          }
        }
        bool raised = false;
#pragma unroll
        for (int r = 0; r < (kEdge ? 2 : 1); ++r) {
          if (!(top[r] > held[r] + kValueRise)) continue;
          const float to = fmaxf(top[r] - kValueRise, -126.f);
          lower[r] = pow2(fmaxf(held[r] - to, -126.f));
          held[r] = to;
          held2[r] = pow2(to);
          raised = true;
        }
        if constexpr (!kEdge) lower[1] = lower[0];
        rise |= __any_sync(~0u, raised);
      }
      float sum[2];
      // Weights against the reference that stands; no maximum is searched first. A thread's sum of a row's 16 weights shows
      // whether one of them has passed the limit, which almost never happens: this one pass is all then.
      auto weights = [&](auto mask_tag) {
        constexpr bool kMask = decltype(mask_tag)::value;
#pragma unroll
        for (int r = 0; r < 2; ++r) sum[r] = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // 32 columns: 16 of packed pairs
          // their weights' power of two, and its inverse
          const float size = lds32_free(info + 8 * h + 4 * b), inverse = lds32_free(info + 16 + 8 * h + 4 * b);
          float by[2], unby[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int of = kMask ? r : 0;  // (no mask: the warp's rows have the same range)
            by[r] = fmaxf(size - held[of], kValueFall);
            unby[r] = fminf(held2[of] * inverse, kValueFall2);
            if constexpr (kMask) by[r] = fminf(by[r], kValueClimb), unby[r] = fmaxf(unby[r], kValueClimb2);
          }
          uint64_t part[2] = {0, 0}, ref[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) ref[r] = pack2(neg[r] + by[r], neg[r] + by[r]);
          uint32_t p[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = 4 * b + i;
            const uint64_t ks = lds64_free(scales + 32 * n);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t* v = &s[4 * n + 2 * r];
              float x, y;
              unpack2(fma2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), ks, ref[r]), x, y);
              if constexpr (kMask) {
                x = first + 8 * n < seen[r] ? x : -INFINITY;
                y = first + 8 * n + 1 < seen[r] ? y : -INFINITY;
              }
              x = exp2_approx(x), y = exp2_approx(y);
              part[r] = add2(part[r], pack2(x, y));
              if constexpr (kEdge) unpack2(mul2(pack2(x, y), lds64_free(scales + 512 + 32 * n)), x, y);  // (values without their scales)
              p[2 * i + r] = fp16_pack(x, y);
            }
          }
          st_pairs8(here + 32 * h + 16 * b, p);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x, y;
            unpack2(part[r], x, y);
            sum[r] = fmaf(x + y, unby[r], sum[r]);
          }
        }
      };
      bool masked = false;  // some row of the warp does not see the half whole
      if constexpr (kEdge) masked = __any_sync(~0u, first - (int32_t)col + 64 > min(seen[0], seen[1]));
      auto form_weights = [&] {
        if constexpr (kEdge) {
          if (masked) return weights(std::true_type{});
        }
        weights(std::false_type{});
      };
      if (!rise) {
        form_weights();
        rise = __any_sync(~0u, sum[0] > limit[0] || sum[1] > limit[1]);
      }
      if (rise) {
        // the reference rises to the row's maximum of this half: what is summed is scaled down, and the weights formed again
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const uint64_t ks = lds64_free(scales + 32 * n);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x, y;
            unpack2(mul2(pack2(__uint_as_float(s[4 * n + 2 * r]), __uint_as_float(s[4 * n + 2 * r + 1])), ks), x, y);
            if (!kEdge || first + 8 * n < seen[r]) top[r] = fmaxf(top[r], x);
            if (!kEdge || first + 8 * n + 1 < seen[r]) top[r] = fmaxf(top[r], y);
          }
        }
        float keep[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
          keep[r] = 1.f;
          if (top[r] > m[r]) {
            keep[r] = exp2_approx(m[r] - top[r]);
            m[r] = top[r];
            neg[r] = -top[r];
            limit[r] = kRise;
          }
          l[r] *= keep[r];
          keep[r] *= lower[r];
        }
        if (j > 0 || h > 0) {
          ok = __all_sync(~0u, bar_wait(bars + kOFull + 16 * half + 8 * (h ^ 1), (j + h + 1) & 1, stop));  // the part before this one
          if (!ok) return;
          fence_after();
#pragma unroll 1
          for (uint32_t o_q = o_at; o_q < o_at + D; o_q += 16) {  // few registers a time
            uint32_t o[8];
            ld_quad8(o_q, o);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep[(e >> 1) & 1]);
            st_quad8(o_q, o);
          }
        }
        form_weights();
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) l[r] += sum[r];
    };
    auto end_tile = [&] {
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bars + kPFull + 16 * half + 8);
    };
    // The sizes (log2) of a tile's value scales, 32 tokens a time, as an address; and the largest.
    auto begin_tile = [&](uint32_t j, uint32_t& info) -> float {
      ok = __all_sync(~0u, bar_wait(bars + kScaleFull + 8 * (j & 3), (j >> 2) & 1, stop));
      info = after_here(base + L::info + (j & 3) * 32);
      const uint4 sizes = lds128(info);
      return fmaxf(fmaxf(__uint_as_float(sizes.x), __uint_as_float(sizes.y)), fmaxf(__uint_as_float(sizes.z), __uint_as_float(sizes.w)));
    };
    uint32_t j = 0;
    for (; j < whole && ok; ++j) {
      uint32_t info;
      const bool grows = begin_tile(j, info) > held[0] + kValueRise;
      if (!ok) break;
      half_tile(std::false_type{}, j, 0, info, grows);
      if (ok) half_tile(std::false_type{}, j, 1, info, false);
      if (ok) end_tile();
    }
    held[1] = held[0], held2[1] = held2[0];
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; ++r)
      seen[r] = (int32_t)lds32(base + L::row_sum + 4 * (half * 128 + lanes + quad + 8 * r));
#pragma unroll 1
    for (; j < tiles && ok; ++j) {
      uint32_t info;
      const float largest = begin_tile(j, info);
      const bool grows = __any_sync(~0u, largest > fminf(held[0], held[1]) + kValueRise);
      if (!ok) break;
      half_tile(std::true_type{}, j, 0, info, grows);
      if (ok) half_tile(std::true_type{}, j, 1, info, grows);
      if (ok) end_tile();
    }
    wait_st();  // (weights that a wait which gave up left on their way: TMEM goes back behind them)
    // the rows' sums, through shared memory to the threads that write the rows: warps of the same 32 rows take half of the
    // columns each (the barrier comes first: no warp may miss it)
    const uint32_t rows32 = (warp & 3) * 32;
    const uint32_t sums = base + L::row_sum + 4 * (half * 128), refs = sums + 4 * kRows, ranges = refs + 4 * kRows;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
      if ((lane & 3) == 0) sts32(sums + 4 * (lanes + quad + 8 * r), __float_as_uint(l[r]));
      if ((lane & 3) == 0) sts32(ranges + 4 * (lanes + quad + 8 * r), __float_as_uint(held[r]));
      if ((kPart || kSplit) && (lane & 3) == 0) sts32(refs + 4 * (lanes + quad + 8 * r), __float_as_uint(m[r]));
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(kSoftThreads / 2) : "memory");
    if (ok && tiles) ok = __all_sync(~0u, bar_wait(bars + kOFull + 16 * half + 8, (tiles - 1) & 1, stop));
    if (kSplit && parts > 1) {
      fence_after();
      asm volatile("bar.sync 3, %0;" ::"n"(kSoftThreads) : "memory");  // all products are done with shared memory
      // O where the queries and keys were, a row's 16-byte chunks exchanged so that 8 lanes' rows meet no bank twice
      const uint32_t row = half * 128 + rows32 + lane, first = (warp >> 2 & 1) * (D / 2);
#pragma unroll 1
      for (uint32_t q = 0; ok && tiles && q < D / 2; q += 32) {
        uint32_t o[32];
        ld32(tmem + (rows32 << 16) + 256 + half * D + first + q, o);
        wait_ld();
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
          sts128(base + L::q + row * (4 * D) + ((((first + q) / 4 + e) ^ (row & 7)) << 4), make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
      }
      fence_before();
      cluster_sync();
      join_parts<D>(base, pl.splits, parts, all_tiles, rank, warp, lane, [&](uint32_t at, const float* o, float inv) {
        if (at >= rows_here) return;
        uint32_t head;
        const uint32_t query = query_of(at, head);
        const bool any = min(w.len, shift + (int32_t)query) > 0;  // no token seen: zeros
        uint32_t x[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) x[i] = any ? bf16_pack(o[2 * i] * inv, o[2 * i + 1] * inv) : 0u;
        uint16_t* dst = a.out + (uint64_t)(w.q0 + query) * a.out_stride + (uint64_t)(hk * group + head) * D + lane * (D / 32);
        if constexpr (D == 128) *reinterpret_cast<uint2*>(dst) = make_uint2(x[0], x[1]);
        else *reinterpret_cast<uint32_t*>(dst) = x[0];
      });
      cluster_sync();  // nobody leaves while its memory is read
    } else if (ok) {
      fence_after();
      // Each warp takes half the columns of its 32 rows, 32 at a time: a thread has a row, and a row a thread is written as lines
      // would be, so the values change hands in shared memory (the queries' place, which no product reads any more: 4 KB a warp).
      const uint32_t row = half * 128 + rows32 + lane;
      const bool any = seen_by(row) > 0;
      // no token seen: zeros. (A sum that is not positive although tokens were seen is a NaN's or an infinity's.)
      const float sum = __uint_as_float(lds32(sums + 4 * (rows32 + lane)));
      const float range = __uint_as_float(lds32(ranges + 4 * (rows32 + lane)));
      const float inv = any ? pow2(range) / sum : 0.f;
      const uint32_t first = (warp >> 2 & 1) * (D / 2), mine = base + L::q + half * L::kOperand + (warp & 7) * (L::kOperand / 8);
      const uint64_t part0 = kPart ? (uint64_t)(blockIdx.x / c.kv_heads % pl.splits) * a.n_reqs : 0;
      if constexpr (kPart) {
        uint32_t head;
        const uint32_t query = query_of(row, head);
        if (row < rows_here && first == 0) {
          const float ref = __uint_as_float(lds32(refs + 4 * (rows32 + lane)));
          pl.split_ml[(part0 + query) * a.q_heads + hk * group + head] = make_float4(tiles ? ref + range : -INFINITY, ref, tiles ? sum : 0.f, 0.f);
        }
      }
      // a row's 32 columns are `kChunks` pieces of 16 bytes; a turn of the warp writes 32 / kChunks rows of them
      constexpr uint32_t kColumns = kPart && D == 64 ? 16 : 32, kChunks = kPart ? kColumns / 4 : kColumns / 8;
#pragma unroll 1
      for (uint32_t q = 0; q < D / 2; q += kColumns) {
        uint32_t o[32];
        if (tiles) {
          const uint32_t from = tmem + (rows32 << 16) + 256 + half * D + first + q;
          if constexpr (kColumns == 32) {
            ld32(from, o);
          } else {
            ld8(from, o);
            ld8(from + 8, o + 8);
          }
          wait_ld();
        }
#pragma unroll
        for (uint32_t e = 0; e < kChunks; ++e) {
          uint4 y;
          if constexpr (kPart) {
            y = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else {
            uint32_t z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              z[i] = any ? bf16_pack(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv) : 0u;
            y = make_uint4(z[0], z[1], z[2], z[3]);
          }
          sts128(mine + (lane * kChunks + (e ^ (lane / (8 / kChunks) % kChunks))) * 16, y);
        }
        __syncwarp();
#pragma unroll
        for (uint32_t i = 0; i < kChunks; ++i) {
          const uint32_t r = i * (32 / kChunks) + lane / kChunks, e = lane % kChunks, at = half * 128 + rows32 + r;
          const uint4 y = lds128(mine + (r * kChunks + (e ^ (r / (8 / kChunks) % kChunks))) * 16);
          uint32_t head;
          const uint32_t query = query_of(at, head);
          if (at < rows_here) {
            if constexpr (kPart) {
              if (tiles)
                *reinterpret_cast<uint4*>(pl.split_out + ((part0 + query) * a.q_heads + hk * group + head) * D + first + q + 4 * e) = y;
            } else {
              *reinterpret_cast<uint4*>(a.out + (uint64_t)(w.q0 + query) * a.out_stride + (uint64_t)(hk * group + head) * D + first + q + 8 * e) = y;
            }
          }
        }
        __syncwarp();
      }
      fence_before();
    }
  } else if (warp < kIssueWarp) {
    // ---- fetch and convert ---------------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    constexpr int kLoads = D / 32;  // 16-byte loads of a thread per operand
    const uint32_t t = tid - kSoftThreads, cw = t >> 5;
    // A warp's load: 4 lanes on 64 values of a row, 8 rows. For D = 128 even warps take the rows' first 64 values.
    const uint32_t part = D == 128 ? (cw & 1) : 0, first = (cw >> (D == 128 ? 1 : 0)) * kLoads * 8;
    const uint32_t chunk = lane & 3, sub = lane >> 2;
    const int32_t* table = (kPart ? a.prefix_pages : a.table + (uint64_t)w.req * a.max_blocks) + (kPart || kSplit ? w.t0 >> c.log2_pt : 0);
    const uint32_t skip = kPart || kSplit ? w.t0 & ((1u << c.log2_pt) - 1) : 0;  // (pages longer than a tile: the part begins inside one)
    const uint32_t pt_mask = (1u << c.log2_pt) - 1;

    // page of the tile's 16-token group `lane` (lanes 0-7), -1 where there are no tokens
    auto pages_of = [&](uint32_t j) -> int32_t {
      const int32_t tok = (int32_t)(j * kTile + (lane & 7) * 16);
      int32_t p = -1;
      if (j < tiles && tok < most) {
        p = table[(tok + skip) >> c.log2_pt];
        if (p < 0 || (uint32_t)p >= c.n_pages) {
          sts32(base + L::misc + 16, 0);
          p = -1;
        }
      }
      return p;
    };
    // Where the warp's rows of a tile lie: their 16-token groups' offsets in the cache, for keys and values alike (-1: nothing
    // there; the bytes behind a sequence's end in its last group are read and masked).
    constexpr int kGroups = kLoads / 2;
    const uint32_t lane_at = sub * D + part * 64 + chunk * 16;
    auto offsets = [&](uint32_t j, int32_t pages, int64_t* off) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const uint32_t group16 = (first >> 4) + i;
        const int32_t p = __shfl_sync(~0u, pages, group16);
        off[i] = p < 0 ? -1 : (int64_t)(kv_row(c, (uint32_t)p, hk, (j * kTile + group16 * 16 + skip) & pt_mask) * D + lane_at);
      }
    };
    // Converts the thread's pieces of an operand, and as each one's registers are read asks for the same piece of the
    // operand after it: one operand's worth of loads is always on its way and no more registers hold it.
    uint4 raw[kLoads];
    auto fetch = [&](const int8_t* src, const int64_t* off, int i) {
      return off[i / 2] < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(src + off[i / 2] + (i % 2) * 8 * D);
    };
    const uint32_t write_at = part * kHalf + (first + sub) * 128 + (((2 * chunk) ^ sub) << 4);
    auto turn = [&](auto value_tag, uint32_t row_scale, uint32_t dst, const int8_t* src, const int64_t* off) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        uint4 x = raw[i];
        uint32_t f = 0;
        if constexpr (decltype(value_tag)::value) f = __shfl_sync(~0u, row_scale, (first + i * 8 + sub) & 31);
        uint2 y[4] = {fp16x4_of_int8(x.x), fp16x4_of_int8(x.y), fp16x4_of_int8(x.z), fp16x4_of_int8(x.w)};
        if constexpr (decltype(value_tag)::value) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = make_uint2(fp16x2_times(y[e].x, f), fp16x2_times(y[e].y, f));
        }
        raw[i] = fetch(src, off, i);
        sts128(dst + write_at + i * 1024, make_uint4(y[0].x, y[0].y, y[1].x, y[1].y));  // row mod 8 is sub: swizzled(row, 2 * chunk)
        sts128((dst + write_at + i * 1024) ^ 16u, make_uint4(y[2].x, y[2].y, y[3].x, y[3].y));
      }
      fence_smem();
      __syncwarp();
    };
    // Scales: a lane holds the two of one token of the warp's 32 (two warps share them; the even one publishes).
    const uint32_t own32 = (cw >> 1) * 32 + lane;
    float factor = a.scale * 1.44269504088896340736f;  // log2(e); later with the queries' power of two
    float k_scale = 0.f, v_scale = 0.f;  // as loaded: nothing waits for them here
    auto fetch_scales = [&](uint32_t j, int32_t pages) {
      const int32_t p = __shfl_sync(~0u, pages, own32 >> 4);
      k_scale = v_scale = 0.f;
      if (p >= 0 && (int32_t)(j * kTile + own32) < most) {
        const uint64_t at = kv_row(c, (uint32_t)p, hk, (j * kTile + own32 + skip) & pt_mask);
        k_scale = c.k_scale[at];
        v_scale = c.v_scale[at];
      }
    };
    int32_t pages = pages_of(0);
    int64_t off[kGroups];
    offsets(0, pages, off);
    if (tiles) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) raw[i] = fetch(c.k, off, i);
      fetch_scales(0, pages);
    }
    uint32_t whole = 0;
    if (tiles && __all_sync(~0u, bar_wait(bars + kQFull, 0, stop))) {
      whole = lds32(base + L::misc + 12) / kTile;
      factor *= pow2i(max(-100, (int32_t)(lds32(base + L::misc + 8) >> 7) - 127) - 14);
    }
    for (uint32_t j = 0; j < tiles; ++j) {
      const uint32_t buf = j & 1, use = j >> 1;
      pages = pages_of(j + 1);  // -1 behind the last tile: nothing is fetched for it
      if (!__all_sync(~0u, bar_wait(bars + kKEmpty + 8 * buf, (use & 1) ^ 1, stop))) break;
      // The scales have four places: those of tile j - 4 were read before the products of tile j - 3 could begin, and
      // this K buffer is free since those of tile j - 2 are done.
      // A value scale that is not finite (or so large that its values would not be) makes the token's key scale NaN, and its values
      // zeros: whoever sees the token gets NaN, and a masked weight of 0 meets no infinity.
      const bool bad = !(fabsf(v_scale) < 1e36f);
      const float v = bad ? 0.f : v_scale;
      // 2^(e_v - 127) <= the largest of the 32 < 2^(e_v - 126)
      const uint32_t e_v = max(__reduce_max_sync(~0u, __float_as_uint(fabsf(v))) >> 23, 1u);
      const float in_range = v * __uint_as_float((254u - e_v) << 23);  // the lane's scale, in (-2, 2)
      uint32_t row_scale = fp16_pack(in_range, in_range);
      if (j >= whole) {  // values stay integers, their scales meet the weights
        row_scale = 0x3C003C00u;
        if (cw & 1) sts32(base + L::scale + (j & 3) * 1024 + 512 + 4 * own32, __float_as_uint(in_range));
      }
      if ((cw & 1) == 0) {
        sts32(base + L::scale + (j & 3) * 1024 + 4 * own32, bad ? 0x7FC00000u : __float_as_uint(k_scale * factor));
        if (lane == 0) {
          sts32(base + L::info + (j & 3) * 32 + 2 * cw, __float_as_uint((float)(int32_t)(e_v - 127)));
          sts32(base + L::info + (j & 3) * 32 + 16 + 2 * cw, (254u - e_v) << 23);  // 2^-(e_v - 127)
        }
      }
      turn(std::false_type{}, 0u, base + L::k + buf * L::kOperand, c.v, off);
      if (lane == 0) {
        bar_arrive(bars + kScaleFull + 8 * (j & 3));
        bar_arrive(bars + kKFull + 8 * buf);
      }
      offsets(j + 1, pages, off);
      fetch_scales(j + 1, pages);
      if (!__all_sync(~0u, bar_wait(bars + kVEmpty + 8 * buf, (use & 1) ^ 1, stop))) break;
      turn(std::true_type{}, row_scale, base + L::v + buf * L::kOperand, c.k, off);
      if (lane == 0) bar_arrive(bars + kVFull + 8 * buf);
    }
    if (kSplit && parts > 1) cluster_sync(), cluster_sync();
  } else {
    // ---- products: a warp for each row tile runs the loop as one, an elected thread issues ---------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp < kIssueWarp + 2 && tiles) {
      const uint32_t i = warp - kIssueWarp;
      constexpr uint32_t kS = instr_desc(128, 64, false), kO = instr_desc(128, D, true);
      const bool lead = elect_one();
      const bool real = !kSplit || i * 128 < rows_here;  // (a row tile without rows has no products, only their barriers)
      // Both for the tokens 64 h .. 64 h + 63 of tile j.
      auto scores = [&](uint32_t j, uint32_t h) {
        const uint32_t q = smem_desc(base + L::q + i * L::kOperand, 16), k = smem_desc(base + L::k + (j & 1) * L::kOperand + h * 8192, 16);
        const uint32_t d = tmem + 128 * i + 64 * ((j + h) & 1);
#pragma unroll
        for (int e = 0; real && e < D / 16; ++e) {
          const uint32_t off = ((e / 4) * kHalf + (e % 4) * 32) >> 4;
          if (e == 0) mma_ss<false>(d, q + off, k + off, kS, lead);
          else mma_ss<true>(d, q + off, k + off, kS, lead);
        }
        commit(bars + kSFull + 16 * i + 8 * h, lead);
      };
      auto values = [&](uint32_t j, uint32_t h) {
        const uint32_t v = smem_desc(base + L::v + (j & 1) * L::kOperand, kHalf) + h * (4 * 2048 >> 4);
        const uint32_t p = tmem + 128 * i + 64 * (j & 1) + 32 * h;
#pragma unroll
        for (int e = 0; real && e < 4; ++e) mma_ts(tmem + 256 + D * i, p + 8 * e, v + e * (2048 >> 4), kO, j > 0 || h > 0 || e > 0, lead);
        commit(bars + kOFull + 16 * i + 8 * h, lead);
      };
      auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(~0u, bar_wait(bars + bar, parity, stop)); };
      bool ok = wait(kQFull, 0) && wait(kKFull, 0);
      if (ok) {
        fence_after();
        scores(0, 0);
        scores(0, 1);
        commit(bars + kKEmpty, lead);
      }
      for (uint32_t j = 0; ok && j < tiles; ++j) {
        const uint32_t buf = j & 1, nbuf = buf ^ 1;
        ok = wait(kVFull + 8 * buf, (j >> 1) & 1);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          ok = ok && wait(kPFull + 16 * i + 8 * h, j & 1);
          if (!ok) break;
          fence_after();
          values(j, h);
          if (h == 1) commit(bars + kVEmpty + 8 * buf, lead);
          if (j + 1 < tiles) {
            if (h == 0) ok = wait(kKFull + 8 * nbuf, ((j + 1) >> 1) & 1);
            if (!ok) break;
            fence_after();
            scores(j + 1, h);
            if (h == 1) commit(bars + kKEmpty + 8 * nbuf, lead);
          }
        }
      }
      if (!ok) {
        // gave up: let the products in flight end (again with a limit) before TMEM goes back
        commit(bars + kDrain + 8 * i, lead);
        for (uint32_t n = 0; n < kDrainTries && !bar_try(bars + kDrain + 8 * i, 0); ++n) {
        }
      }
    }
    if (kSplit && parts > 1) cluster_sync(), cluster_sync();
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kIssueWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if constexpr (kPart) {
    if (tid == 0) pl.errors[blockIdx.x] = lds32(stop) != 0 ? kGaveUp : lds32(base + L::misc + 16);
  } else {
    const bool gave_up = lds32(stop) != 0;
    if (tid == 0 && (gave_up || lds32(base + L::misc + 16) != kNoError)) report_first(a.st, gave_up ? SHN_ERR_TIMEOUT : SHN_ERR_INVALID_ARG, w.req);
  }
}

// More shared memory than the default 48 KB: an attribute of the kernel on each device, so it is set for the one that is
// current on every call.
template <int D, bool kPart, bool kSplit>
cudaError_t launch(uint64_t blocks, const KvPages& c, const KvAttnArgs& a, const DecodePlan& pl, cudaStream_t s) {
  if (blocks >= (1ull << 31)) return cudaErrorInvalidConfiguration;
  const auto kernel = kv_prompt_kernel<D, kPart, kSplit>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::total);
  if (e != cudaSuccess) return e;
  if constexpr (kSplit) return launch_behind_in_clusters(kernel, pl.splits, dim3((uint32_t)blocks * pl.splits), kThreads, Layout<D>::total, s, c, a, pl);
  else if constexpr (kPart) return launch_first(kernel, dim3((uint32_t)blocks), kThreads, Layout<D>::total, s, c, a, pl);
  else return launch_behind(kernel, dim3((uint32_t)blocks), kThreads, Layout<D>::total, s, c, a, pl);
}

}  // namespace

cudaError_t launch_kv_prompt(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, int sm_count, cudaStream_t s) {
  const uint64_t group = a.q_heads / c.kv_heads;
  // at most so many tiles, however the queries are spread over the requests
  const uint64_t blocks = ((uint64_t)a.n_tokens * group / kRows + (a.n_reqs < a.n_tokens ? a.n_reqs : a.n_tokens)) * c.kv_heads;
  DecodePlan pl = {};
  pl.splits = 1;
  // Few blocks, and requests that may be long: several blocks to the same rows, as many as the SMs have places and the longest
  // sequence tiles. Measured, with and without: one query after 5102 tokens (8 heads on one) 25.5 / 118.8 us, 700 after 2551 (8 on
  // 2) 33.8 / 74.6, 40 after 5102 (32 on 8, of 64) 27.5 / 102.1. With 4 blocks to a row at most they take 42.4, 34.2 and
  // 37.8, with up to twice the blocks that have places 29.7, 49.1 and 27.0.
  const uint64_t tokens = (uint64_t)a.max_blocks << c.log2_pt;  // what a request can have
  kv_prompt_begin_kernel<<<1, a.n_reqs < 1024 ? (a.n_reqs + 31) / 32 * 32 : 1024, 0, s>>>(c, a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  while (pl.splits < 8 && blocks * pl.splits * 2 <= (uint64_t)sm_count && tokens > 2 * pl.splits * kTile) pl.splits *= 2;
  if (blocks <= (uint64_t)sm_count) return head_dim == 128 ? launch<128, false, true>(blocks, c, a, pl, s) : launch<64, false, true>(blocks, c, a, pl, s);
  return head_dim == 128 ? launch<128, false, false>(blocks, c, a, pl, s) : launch<64, false, false>(blocks, c, a, pl, s);
}

cudaError_t launch_kv_prefix(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, const DecodePlan& pl, cudaStream_t s) {
  const uint64_t group = a.q_heads / c.kv_heads;
  const uint64_t blocks = (a.n_reqs * group + kRows - 1) / kRows * c.kv_heads * pl.splits;
  return head_dim == 128 ? launch<128, true, false>(blocks, c, a, pl, s) : launch<64, true, false>(blocks, c, a, pl, s);
}

}  // namespace shn
