// kv_plan.cu — block tables and slot maps of a step from the requests' lengths (shn_kv_plan).
//
// Two exclusive sums over the requests (new tokens; pages to take), then one independent item per new
// token and per new page, each finding its request by a search in the sums. Little is read or written
// (about 16 bytes per request and 8 per token), so the call is bound by latency. Every block forms the sums
// for itself, which costs less than handing them around, and takes a token per thread. A step that one block
// covers is one launch. With more blocks the first of them looks at everything that can be wrong and is the only one to
// write the status; only where the caller has the free-list head updated in place a small kernel in front keeps it
// as it was before the call. Measured: 256 requests with a token each 4.1 us, 1000 with 131,072 in all 6.4 us; one
// cluster of 8 blocks with 16 tokens a thread took 24.6 for the latter.
#include "kv_internal.cuh"

namespace shn {
namespace {

constexpr int kThreads = 1024;

struct Sum2 {
  long long tokens, pages;
};

__device__ __forceinline__ long long pages_of(long long tokens, uint32_t log2_pt) {
  return (tokens + (1ll << log2_pt) - 1) >> log2_pt;
}

// Keeps the head (behind the status word) for the kernel that follows.
__global__ void kv_plan_begin_kernel(KvPlanArgs a, int32_t* kept) {
  let_next();
  if (threadIdx.x == 0) *kept = *a.free_head;
}

template <bool kOne>  // one block
__global__ void __launch_bounds__(kThreads) kv_plan_kernel(KvPlanArgs a) {
  __shared__ Sum2 before[kThreads + 1];  // sums in front of each thread's run of requests
  __shared__ Sum2 warp_sum[32];
  __shared__ uint32_t bad_code, bad_detail;
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // (several blocks: the first is for the status)
  const bool looks = !kOne && blockIdx.x == 0;
  const uint32_t rank = kOne ? 0 : blockIdx.x - 1, ranks = kOne ? 1 : gridDim.x - 1;
  const uint32_t run = (a.n + kThreads - 1) / kThreads;
  const uint32_t r0 = min(a.n, t * run), r1 = min(a.n, r0 + run);
  if (t == 0) bad_code = 0, bad_detail = 0xFFFFFFFFu;
  long long head = 0;
  if constexpr (kOne) head = *a.free_head;
  __syncthreads();

  Sum2 own = {0, 0};
  bool negative = false, wide = false;
  uint32_t bad_r = 0xFFFFFFFFu;
  for (uint32_t r = r0; r < r1; ++r) {
    const long long c = a.ctx[r], f = a.fresh[r];
    const long long p = pages_of(c + f, a.log2_pt);
    const bool neg = c < 0 || f < 0 || c + f > 0x7FFFFFFFll, wd = p > (long long)a.max_blocks;
    if ((neg || wd) && bad_r == 0xFFFFFFFFu) bad_r = r;
    negative |= neg;
    wide |= wd;
    own.tokens += f;
    own.pages += p - pages_of(c, a.log2_pt);
  }
  if (negative || wide) {
    atomicMin(&bad_detail, bad_r);
    atomicMax(&bad_code, negative ? 2u : 1u);
  }
  Sum2 inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, inc.tokens, d), y = __shfl_up_sync(~0u, inc.pages, d);
    if (lane >= (uint32_t)d) inc.tokens += x, inc.pages += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sum2 w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(~0u, w.tokens, d), y = __shfl_up_sync(~0u, w.pages, d);
      if (lane >= (uint32_t)d) w.tokens += x, w.pages += y;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  const Sum2 base = warp ? warp_sum[warp - 1] : Sum2{0, 0};
  before[t] = {base.tokens + inc.tokens - own.tokens, base.pages + inc.pages - own.pages};
  if (t == 0) before[kThreads] = warp_sum[31];
  __syncthreads();
  const Sum2 total = before[kThreads];

  if constexpr (!kOne) {
    after_previous();
    head = *reinterpret_cast<const volatile int32_t*>(a.free_head);
  }
  uint32_t code = bad_code == 2 ? SHN_ERR_INVALID_ARG : bad_code == 1 ? SHN_ERR_CAPACITY : SHN_OK;
  uint32_t detail = code ? bad_detail : 0;
  if (code == SHN_OK && (head < 0 || head > (long long)a.n_free)) code = SHN_ERR_INVALID_ARG;
  if (code == SHN_OK && (total.tokens > (long long)a.max_tokens || head + total.pages > (long long)a.n_free))
    code = SHN_ERR_CAPACITY;
  const bool ok = code == SHN_OK;
  if constexpr (kOne) __syncthreads();  // the head and what was found are read before anything is written
  const int32_t page_limit = (int32_t)(0x7FFFFFFFu >> a.log2_pt);
  const uint32_t pt_mask = (1u << a.log2_pt) - 1;
  if (looks) {
    // pages that are begun, and new ones
    if (ok) {
      for (uint32_t r = r0; r < r1; ++r) {
        const int32_t c = a.ctx[r];
        if (a.fresh[r] > 0 && (c & pt_mask)) {
          const int32_t p = a.table[(uint64_t)r * a.max_blocks + (c >> a.log2_pt)];
          if (p < 0 || p >= page_limit) atomicMin(&bad_detail, r);
        }
      }
      constexpr int kAhead = 8;
      for (long long i0 = t; i0 < total.pages; i0 += kAhead * kThreads) {
        int32_t p[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) p[e] = i0 + e * kThreads < total.pages ? a.free_pages[head + i0 + e * kThreads] : 0;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          if (p[e] >= 0 && p[e] < page_limit) continue;
          const long long i = i0 + e * kThreads;
          uint32_t r = 0;  // the request that takes it
          while (before[r / run + 1].pages <= i) r += run;
          for (long long j = i - before[r / run].pages;; ++r) {
            j -= pages_of((long long)a.ctx[r] + a.fresh[r], a.log2_pt) - pages_of(a.ctx[r], a.log2_pt);
            if (j < 0) break;
          }
          atomicMin(&bad_detail, r);
        }
      }
      __syncthreads();
      detail = bad_detail;
      if (detail != 0xFFFFFFFFu) code = SHN_ERR_INVALID_ARG;
      else detail = 0;
    }
    if (t == 0) a.st->status = code, a.st->detail = detail;
    return;
  }
  if (rank == 0 && t == 0) {
    *a.free_next = (int32_t)(ok ? head + total.pages : head);
    a.cu[a.n] = (int32_t)(ok ? total.tokens : 0);
  }
  if (t % ranks == rank) {
    long long tok = before[t].tokens;
    for (uint32_t r = r0; r < r1; ++r) {
      a.cu[r] = (int32_t)(ok ? tok : 0);
      a.kv_len[r] = ok ? a.ctx[r] + a.fresh[r] : 0;
      tok += a.fresh[r];
    }
  }
  // new pages into the table
  if (ok) {
    for (long long i = rank * kThreads + t; i < total.pages; i += (long long)ranks * kThreads) {
      uint32_t lo = 0, hi = kThreads;
      while (hi - lo > 1) {
        const uint32_t m = (lo + hi) >> 1;
        if (before[m].pages <= i) lo = m; else hi = m;
      }
      long long j = i - before[lo].pages;
      for (uint32_t r = lo * run;; ++r) {
        const long long have = pages_of(a.ctx[r], a.log2_pt);
        const long long need = pages_of((long long)a.ctx[r] + a.fresh[r], a.log2_pt) - have;
        if (j < need) {
          const int32_t p = a.free_pages[head + i];
          a.table[(uint64_t)r * a.max_blocks + have + j] = p;
          if (kOne && (p < 0 || p >= page_limit)) atomicMin(&bad_detail, r);
          break;
        }
        j -= need;
      }
    }
  }
  for (uint32_t i = rank * kThreads + t; i < a.max_tokens; i += ranks * kThreads) {
    int32_t pos = 0, slot = -1;
    if (ok && i < total.tokens) {
      uint32_t lo = 0, hi = kThreads;
      while (hi - lo > 1) {
        const uint32_t m = (lo + hi) >> 1;
        if (before[m].tokens <= i) lo = m; else hi = m;
      }
      long long j = i - before[lo].tokens, pages = before[lo].pages;
      for (uint32_t r = lo * run;; ++r) {
        const long long c = a.ctx[r], f = a.fresh[r], have = pages_of(c, a.log2_pt);
        if (j < f) {
          pos = (int32_t)(c + j);
          const long long b = pos >> a.log2_pt;
          const int32_t p = b < have ? a.table[(uint64_t)r * a.max_blocks + b] : a.free_pages[head + pages + b - have];
          if (p >= 0 && p < page_limit) slot = (int32_t)(((uint32_t)p << a.log2_pt) + (pos & pt_mask));
          else if (kOne) atomicMin(&bad_detail, r);
          break;
        }
        j -= f;
        pages += pages_of(c + f, a.log2_pt) - have;
      }
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
  if constexpr (kOne) {
    __syncthreads();
    if (t) return;
    const bool page = ok && bad_detail != 0xFFFFFFFFu;  // (the first request with one that is bad)
    a.st->status = page ? SHN_ERR_INVALID_ARG : code;
    a.st->detail = page ? bad_detail : detail;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t s) {
  // one block up to a token a thread (256 tokens 4.1 us, 4.4 with a block more for the status; 900 tokens 4.5 and 4.8; with two
  // tokens a thread 1500 tokens 5.5 and 4.7)
  if (a.max_tokens <= kThreads) {
    kv_plan_kernel<true><<<1, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const uint32_t most = 2u * sm_count_for_launch() - 1, blocks = (a.max_tokens + kThreads - 1) / kThreads;
  const dim3 grid(1 + (blocks < most ? blocks : most));
  if (a.free_head != a.free_next) return launch_first(kv_plan_kernel<false>, grid, kThreads, 0, s, a);
  KvPlanArgs b = a;
  int32_t* kept = reinterpret_cast<int32_t*>(a.st) + 2;
  b.free_head = kept;
  kv_plan_begin_kernel<<<1, 32, 0, s>>>(a, kept);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_behind(kv_plan_kernel<false>, grid, kThreads, 0, s, b) : e;
}

}  // namespace shn
