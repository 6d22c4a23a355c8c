// kv_decode.cuh — how the attention of single tokens is cut up: segments, units, pieces and their partial results.
//
// A segment is a run of tokens with the query rows that read it: the tokens of one request that are its own (rows: the
// heads of a group), or the shared prefix (rows: all requests' heads of a group). Its tokens are counted in units of
// kUnit, all segments' units lie in one line, and each of the W warps takes the same number in a row (or one more),
// whatever the lengths. A warp's part of a segment is a piece; pieces are numbered w + segment, which is
// unique because both only grow along the line. A piece's result for a row is (O, mt, ms, l):
//   sum of weights = l 2^ms,  sum of weighted values = O 2^mt
// and a last kernel joins a row's pieces in their order, so results do not depend on timing.
#pragma once

#include "kv_internal.cuh"

namespace shn {

constexpr uint32_t kUnit = 32;           // tokens
constexpr uint32_t kDecodeThreads = 256;
constexpr uint32_t kDecodeMaxWarps = 148 * 16;  // two blocks on each of a B200's SMs; the workspace has room for their pieces

struct DecodePlan {
  uint32_t rows;           // query rows of a segment: 8 or 16
  uint32_t own_groups;     // row groups of a request's heads per key head
  uint32_t prefix_groups;  // row groups of all requests' heads per key head (0: the prefix is not among the segments)
  uint32_t warps;          // W
  uint32_t splits;         // parts of the prefix in the other kernel (0: none)
  float* out;              // [pieces][rows][head_dim]
  float4* ml;              // [pieces][rows] (mt, ms, l, -)
  float* split_out;        // [splits][n_reqs * q_heads][head_dim]
  float4* split_ml;
  uint32_t* errors;        // [n_errors], what each block found: the prefix kernel's blocks, then the single-token kernel's
  uint32_t n_errors;
};
// A block's error: none, a wait that gave up, or the (first) request with something invalid. Every block writes its word, and
// the last kernel makes the status of them: nothing has to be cleared in front of the first.
constexpr uint32_t kNoError = 0xFFFFFFFFu, kGaveUp = 0xFFFFFFFEu;

// Effective lengths: what the tables can hold. `bad` is set where the caller's value is not that.
__device__ __forceinline__ int32_t decode_prefix(const KvPages& c, const KvAttnArgs& a, bool& bad) {
  const int64_t most = (int64_t)a.n_prefix_pages << c.log2_pt;
  const int32_t p = *a.prefix_len;
  bad = p < 0 || p > most;
  return bad ? (p < 0 ? 0 : (int32_t)most) : p;
}
__device__ __forceinline__ int32_t decode_len(const KvPages& c, const KvAttnArgs& a, int32_t prefix, uint32_t r, bool& bad) {
  const int64_t most = max((int64_t)a.max_blocks << c.log2_pt, (int64_t)prefix);
  const int32_t n = a.kv_len[r];
  bad = n < 0 || n > most;
  return bad ? (n < 0 ? 0 : (int32_t)most) : n;
}
__device__ __forceinline__ uint32_t own_start(int32_t prefix) { return (uint32_t)prefix & ~15u; }
__device__ __forceinline__ uint32_t own_units(int32_t prefix, int32_t len) {
  return len > prefix ? ((uint32_t)len - own_start(prefix) + kUnit - 1) / kUnit : 0;
}

// Units in front of each thread's run of requests, for kDecodeThreads threads; [kDecodeThreads] is their total. Units of one
// row group and key head: the line holds each request's kv_heads * own_groups times.
struct UnitScan {
  unsigned long long before[kDecodeThreads + 1];
  unsigned long long warp_sum[kDecodeThreads / 32];
};
// first_bad: where the first request with a bad length goes (shared memory), or null.
__device__ __forceinline__ void scan_units(const KvPages& c, const KvAttnArgs& a, int32_t prefix, UnitScan& s, uint32_t* first_bad) {
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t run = (a.n_reqs + kDecodeThreads - 1) / kDecodeThreads;
  const uint32_t r0 = min(a.n_reqs, t * run), r1 = min(a.n_reqs, r0 + run);
  unsigned long long own = 0;
  for (uint32_t r = r0; r < r1; ++r) {
    bool bad;
    const int32_t len = decode_len(c, a, prefix, r, bad);
    if (bad && first_bad) atomicMin(first_bad, r);
    own += own_units(prefix, len);
  }
  unsigned long long inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long x = __shfl_up_sync(~0u, inc, d);
    if (lane >= (uint32_t)d) inc += x;
  }
  if (lane == 31) s.warp_sum[warp] = inc;
  __syncthreads();
  unsigned long long base = 0;
#pragma unroll
  for (uint32_t i = 0; i < kDecodeThreads / 32; ++i) base += i < warp ? s.warp_sum[i] : 0;
  s.before[t] = base + inc - own;
  if (t == kDecodeThreads - 1) s.before[kDecodeThreads] = base + inc;
  __syncthreads();
}
// Units in front of request r.
__device__ __forceinline__ unsigned long long units_before(const KvPages& c, const KvAttnArgs& a, int32_t prefix, const UnitScan& s, uint32_t r) {
  const uint32_t run = (a.n_reqs + kDecodeThreads - 1) / kDecodeThreads;
  unsigned long long u = s.before[r / run];
  for (uint32_t i = r / run * run; i < r; ++i) {
    bool bad;
    u += own_units(prefix, decode_len(c, a, prefix, i, bad));
  }
  return u;
}
// The line of units and the warps' shares of it: the first `rest` warps take one unit more than the others.
struct Line {
  unsigned long long units, cut;  // cut: units of the first `rest` warps
  unsigned long long each;
  uint32_t rest;
  __device__ __forceinline__ Line(unsigned long long n, uint32_t warps) : units(n) {
    if (n >> 32) each = n / warps;
    else each = (uint32_t)n / warps;  // (the 64-bit division is many times as long)
    rest = (uint32_t)(n - each * warps);
    cut = rest * (each + 1);
  }
  __device__ __forceinline__ unsigned long long first(uint32_t w) const { return w * each + min(w, rest); }
  // The warp that takes unit u (u < units).
  __device__ __forceinline__ uint32_t warp_of(unsigned long long u) const {
    const bool in = u < cut;
    const unsigned long long x = in ? u : u - cut, y = in ? each + 1 : each;
    return (in ? 0 : rest) + (uint32_t)(units >> 32 ? x / y : (uint32_t)x / (uint32_t)y);
  }
};

// The prefix in pl.splits parts (kv_attn_tc.cu): parts' sums into pl.split_out, pl.split_ml.
cudaError_t launch_kv_prefix(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, const DecodePlan& pl, cudaStream_t s);
cudaError_t launch_kv_decode(const KvPages& c, uint32_t head_dim, const KvAttnArgs& a, const DecodePlan& pl, cudaStream_t s);

}  // namespace shn
