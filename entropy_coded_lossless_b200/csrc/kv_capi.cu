// kv_capi.cu — the extern "C" entry points of include/shn_kv.h: argument checks and launches.
// No device allocation and no synchronisation.
#include "kv_decode.cuh"

using namespace shn;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool power_of_two(uint32_t x) { return x && (x & (x - 1)) == 0; }
uint32_t log2_of(uint32_t x) {
  uint32_t l = 0;
  while ((1u << l) < x) ++l;
  return l;
}

// Largest group of query heads per key head: 64 rows of one query fit every kernel's row tile.
constexpr uint32_t kMaxGroup = 64;

int check_cache(const shn_kv_cache* c) {
  if (!c || !c->d_k || !c->d_v || !c->d_k_scale || !c->d_v_scale) return SHN_ERR_INVALID_ARG;
  if (!aligned(c->d_k, 16) || !aligned(c->d_v, 16) || !aligned(c->d_k_scale, 16) || !aligned(c->d_v_scale, 16))
    return SHN_ERR_INVALID_ARG;
  if (c->n_pages == 0 || c->kv_heads == 0 || c->kv_heads > 1024) return SHN_ERR_INVALID_ARG;
  if (!power_of_two(c->page_tokens) || c->page_tokens < 16 || c->page_tokens > 1024) return SHN_ERR_INVALID_ARG;
  if ((uint64_t)c->n_pages * c->page_tokens >= (1ull << 31)) return SHN_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return SHN_ERR_UNSUPPORTED;
  return SHN_OK;
}

KvPages pages_of(const shn_kv_cache* c) {
  return KvPages{c->d_k, c->d_v, c->d_k_scale, c->d_v_scale, c->n_pages, c->kv_heads, log2_of(c->page_tokens)};
}

// The workspace's status word, cleared on the stream. Null on failure (err set).
DeviceStatus* clear_status(void* d_work, cudaStream_t s) {
  DeviceStatus* st = static_cast<DeviceStatus*>(d_work);
  return launch_kv_begin(st, s) == cudaSuccess ? st : nullptr;
}

int check_work(const void* d_work, size_t have, size_t need) {
  if (!d_work || !aligned(d_work, 256)) return SHN_ERR_INVALID_ARG;
  return have < need ? SHN_ERR_WORKSPACE : SHN_OK;
}

// rows of activations: 16-byte aligned, token stride a multiple of 8 values that holds a token
bool rows_ok(const void* p, uint64_t stride, uint64_t heads, uint32_t head_dim, uint64_t n_tokens) {
  return p && aligned(p, 16) && stride % 8 == 0 && (n_tokens <= 1 || stride >= heads * head_dim);
}

int check_attn(const uint16_t* d_q, uint64_t q_stride, uint32_t n_tokens, uint32_t q_heads, const shn_kv_cache* cache,
               const int32_t* d_block_table, uint32_t max_blocks, const int32_t* d_kv_len, uint32_t n_reqs,
               const uint16_t* d_out, uint64_t out_stride) {
  const int e = check_cache(cache);
  if (e != SHN_OK) return e;
  if (q_heads == 0 || q_heads % cache->kv_heads || q_heads / cache->kv_heads > kMaxGroup) return SHN_ERR_INVALID_ARG;
  if (n_tokens >= (1u << 31) / q_heads || n_reqs >= (1u << 31) - 1) return SHN_ERR_INVALID_ARG;
  if (n_reqs && (!d_kv_len || (max_blocks && !d_block_table))) return SHN_ERR_INVALID_ARG;
  if ((uint64_t)max_blocks * cache->page_tokens >= (1ull << 31)) return SHN_ERR_INVALID_ARG;
  if (n_tokens && (!rows_ok(d_q, q_stride, q_heads, cache->head_dim, n_tokens) ||
                   !rows_ok(d_out, out_stride, q_heads, cache->head_dim, n_tokens)))
    return SHN_ERR_INVALID_ARG;
  return SHN_OK;
}

// Which kernel the prefix goes to. The single-token kernel reads it once for each 8 (16) query rows, about 1.5 ns a unit of 32
// tokens; the tensor core kernel serves 256 rows at once but takes some 12 us to start and end. Measured (32 query and 8
// key heads of 128, microseconds of GPU time with 16 own tokens each, single-token kernel / tensor cores): 8 requests 1024 tokens
// 13.3 / 18.0, 8192 tokens 22.8 / 26.6; 16 requests 1024 tokens 15.8 / 19.3, 8192 tokens 33.2 / 28.0. So tensor cores from
// kPrefixUnits units on, and for more row groups than the workspace keeps places for.
constexpr uint64_t kPrefixUnits = 12288, kPrefixGroups = 64;
// As many parts as give each of a B200's SMs a block: a number and not a question to the device, since the size query is for any device
// and makes no CUDA call. (Fewer or more SMs get the same parts, and right results.)
constexpr uint64_t kSplitBlocks = 148;

// How shn_kv_attn_shared is cut up, and its workspace: [status 256][pieces' sums][pieces' (mt, ms, l)][the same of the prefix's
// parts][blocks' errors]. For one request at least: an empty batch has no layout, only a status word.
struct SharedLayout {
  DecodePlan pl;
  size_t out_off, ml_off, split_off, split_ml_off, errors_off, total;
  uint64_t prefix_tiles;  // of 256 rows, all key heads'
};

SharedLayout shared_layout(const shn_kv_cache* c, uint32_t n_reqs, uint32_t q_heads) {
  SharedLayout x = {};
  const uint32_t group = q_heads / c->kv_heads;
  // The rows of one mma are 8; 16 share what is done for a token's bytes (groups of 16, 32 requests of 2048 tokens: 36.9 us
  // against 41.0 with two groups of 8 each).
  x.pl.rows = group <= 8 ? 8 : 16;
  x.pl.own_groups = (group + x.pl.rows - 1) / x.pl.rows;
  const uint64_t rows = (uint64_t)n_reqs * group;
  // for the tensor cores: as many parts as give every SM one block
  const uint64_t blocks = (rows + 255) / 256 * c->kv_heads;
  x.pl.splits = blocks >= kSplitBlocks ? 1 : (uint32_t)(kSplitBlocks / blocks);
  const uint64_t groups = (rows + x.pl.rows - 1) / x.pl.rows;
  x.pl.prefix_groups = groups <= kPrefixGroups ? (uint32_t)groups : 0;
  // Places for the most that any number of requests up to this one needs (a workspace serves smaller batches too), although
  // splits and prefix_groups fall as rows are added: prefix_groups are at most kPrefixGroups; parts' rows are at most
  // kSplitBlocks * 256 where there are several splits (256 rows to a block), and blocks * splits at most kSplitBlocks.
  const uint64_t segs = (uint64_t)c->kv_heads * ((groups < kPrefixGroups ? groups : kPrefixGroups) + (uint64_t)n_reqs * x.pl.own_groups);
  const uint64_t pieces = (kDecodeMaxWarps + segs) * x.pl.rows;
  const uint64_t all_rows = (uint64_t)n_reqs * q_heads, most_splits = c->kv_heads < kSplitBlocks ? kSplitBlocks / c->kv_heads : 1;
  const uint64_t split_rows = all_rows * most_splits < kSplitBlocks * 256 ? all_rows * most_splits : kSplitBlocks * 256;
  const uint64_t parts = all_rows > split_rows ? all_rows : split_rows;
  const uint64_t part_blocks = blocks > kSplitBlocks ? blocks : kSplitBlocks;
  x.out_off = 256;
  x.ml_off = x.out_off + round_up(pieces * c->head_dim * sizeof(float), 256);
  x.split_off = x.ml_off + round_up(pieces * sizeof(float4), 256);
  x.split_ml_off = x.split_off + round_up(parts * c->head_dim * sizeof(float), 256);
  x.errors_off = x.split_ml_off + round_up(parts * sizeof(float4), 256);
  x.prefix_tiles = blocks;
  x.total = x.errors_off + round_up((part_blocks + kDecodeMaxWarps / (kDecodeThreads / 32)) * sizeof(uint32_t), 256);
  return x;
}

}  // namespace

extern "C" {

int shn_kv_check_cache(const shn_kv_cache* c) { return check_cache(c); }

int shn_kv_plan(const int32_t* d_ctx_len, const int32_t* d_new_len, uint32_t n_reqs, uint32_t page_tokens,
                int32_t* d_block_table, uint32_t max_blocks, const int32_t* d_free_pages, uint32_t n_free,
                const int32_t* d_free_head, int32_t* d_free_next, int32_t* d_cu_new, int32_t* d_kv_len,
                int32_t* d_positions, int32_t* d_slots, uint32_t max_tokens, void* d_work, size_t work_bytes,
                void* stream) {
  if (!power_of_two(page_tokens) || page_tokens < 16 || page_tokens > 1024) return SHN_ERR_INVALID_ARG;
  if (n_reqs >= (1u << 31) - 1 || max_tokens >= (1u << 31) || n_free >= (1u << 31) ||
      (uint64_t)max_blocks * page_tokens >= (1ull << 31))
    return SHN_ERR_INVALID_ARG;
  if (!d_free_head || !d_free_next || !d_cu_new || (n_free && !d_free_pages)) return SHN_ERR_INVALID_ARG;
  if (n_reqs && (!d_ctx_len || !d_new_len || !d_kv_len || (max_blocks && !d_block_table))) return SHN_ERR_INVALID_ARG;
  if (max_tokens && (!d_positions || !d_slots)) return SHN_ERR_INVALID_ARG;
  const int e = check_work(d_work, work_bytes, SHN_KV_WORKSPACE_BYTES);
  if (e != SHN_OK) return e;
  if (n_reqs && (d_kv_len == d_ctx_len || d_kv_len == d_new_len)) return SHN_ERR_INVALID_ARG;  // every block reads these
  KvPlanArgs a;
  a.ctx = d_ctx_len, a.fresh = d_new_len, a.n = n_reqs, a.log2_pt = log2_of(page_tokens);
  a.max_blocks = max_blocks, a.n_free = n_free, a.max_tokens = max_tokens;
  a.table = d_block_table, a.free_pages = d_free_pages, a.free_head = d_free_head, a.free_next = d_free_next;
  a.cu = d_cu_new, a.kv_len = d_kv_len, a.positions = d_positions, a.slots = d_slots;
  a.st = static_cast<DeviceStatus*>(d_work);  // the kernel sets it, without a launch to clear it
  return launch_kv_plan(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SHN_OK : SHN_ERR_CUDA;
}

int shn_kv_store(const uint16_t* d_q, uint64_t q_stride, uint32_t q_heads, const uint16_t* d_k, uint64_t k_stride,
                 const uint16_t* d_v, uint64_t v_stride, uint32_t n_tokens, const int32_t* d_positions,
                 const int32_t* d_slots, const uint16_t* d_q_weight, const uint16_t* d_k_weight, float eps,
                 const float* d_cos_sin, uint32_t n_positions, uint32_t rot_dim, uint32_t pairs,
                 const shn_kv_cache* cache, uint16_t* d_q_out, uint64_t q_out_stride, void* d_work,
                 size_t work_bytes, void* stream) {
  int e = check_cache(cache);
  if (e != SHN_OK) return e;
  const uint32_t d = cache->head_dim;
  if (n_tokens >= (1u << 31) || q_heads > 65536 || pairs > 1) return SHN_ERR_INVALID_ARG;
  if (rot_dim > d || rot_dim % 16 || (rot_dim != 0) != (d_cos_sin != nullptr)) return SHN_ERR_INVALID_ARG;
  if (!aligned(d_cos_sin, 16) || !aligned(d_q_weight, 16) || !aligned(d_k_weight, 16)) return SHN_ERR_INVALID_ARG;
  if ((d_q_weight || d_k_weight) && !(eps >= 0.f)) return SHN_ERR_INVALID_ARG;
  if ((d_q == nullptr) != (q_heads == 0) && n_tokens) return SHN_ERR_INVALID_ARG;
  if (n_tokens) {
    if (!rows_ok(d_k, k_stride, cache->kv_heads, d, n_tokens) || !rows_ok(d_v, v_stride, cache->kv_heads, d, n_tokens))
      return SHN_ERR_INVALID_ARG;
    if (q_heads && (!rows_ok(d_q, q_stride, q_heads, d, n_tokens) || !rows_ok(d_q_out, q_out_stride, q_heads, d, n_tokens)))
      return SHN_ERR_INVALID_ARG;
    if (d_q == d_q_out && q_stride != q_out_stride && n_tokens > 1) return SHN_ERR_INVALID_ARG;
    if (!d_slots || (rot_dim && !d_positions)) return SHN_ERR_INVALID_ARG;
  }
  e = check_work(d_work, work_bytes, SHN_KV_WORKSPACE_BYTES);
  if (e != SHN_OK) return e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KvStoreArgs a;
  a.q = d_q, a.k = d_k, a.v = d_v, a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.q_heads = q_heads, a.n_tokens = n_tokens, a.positions = d_positions, a.slots = d_slots;
  a.q_weight = d_q_weight, a.k_weight = d_k_weight, a.eps = eps;
  a.cos_sin = d_cos_sin, a.n_positions = n_positions, a.rot = rot_dim, a.pairs = pairs;
  a.q_out = d_q_out, a.q_out_stride = q_out_stride;
  a.st = static_cast<DeviceStatus*>(d_work);  // set or cleared by the launches
  if (n_tokens == 0) return clear_status(d_work, s) ? SHN_OK : SHN_ERR_CUDA;
  return launch_kv_store(pages_of(cache), d, a, sm_count_for_launch(), s) == cudaSuccess ? SHN_OK : SHN_ERR_CUDA;
}

int shn_kv_load(const shn_kv_cache* cache, const int32_t* d_slots, uint32_t n_tokens, uint16_t* d_k_out,
                uint64_t k_stride, uint16_t* d_v_out, uint64_t v_stride, void* d_work, size_t work_bytes,
                void* stream) {
  int e = check_cache(cache);
  if (e != SHN_OK) return e;
  if (n_tokens >= (1u << 31)) return SHN_ERR_INVALID_ARG;
  if (n_tokens) {
    if (!d_slots || (d_k_out && !rows_ok(d_k_out, k_stride, cache->kv_heads, cache->head_dim, n_tokens)) ||
        (d_v_out && !rows_ok(d_v_out, v_stride, cache->kv_heads, cache->head_dim, n_tokens)))
      return SHN_ERR_INVALID_ARG;
  }
  e = check_work(d_work, work_bytes, SHN_KV_WORKSPACE_BYTES);
  if (e != SHN_OK) return e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KvLoadArgs a;
  a.slots = d_slots, a.n_tokens = n_tokens, a.k_out = d_k_out, a.v_out = d_v_out;
  a.k_stride = k_stride, a.v_stride = v_stride;
  a.st = static_cast<DeviceStatus*>(d_work);  // as above
  if (n_tokens == 0 || (!d_k_out && !d_v_out)) return clear_status(d_work, s) ? SHN_OK : SHN_ERR_CUDA;
  return launch_kv_load(pages_of(cache), cache->head_dim, a, s) == cudaSuccess ? SHN_OK : SHN_ERR_CUDA;
}

int shn_kv_attn_prompt(const uint16_t* d_q, uint64_t q_stride, uint32_t n_tokens, uint32_t q_heads,
                       const shn_kv_cache* cache, const int32_t* d_block_table, uint32_t max_blocks,
                       const int32_t* d_cu_q, const int32_t* d_kv_len, uint32_t n_reqs, float softmax_scale,
                       uint16_t* d_out, uint64_t out_stride, void* d_work, size_t work_bytes, void* stream) {
  int e = check_attn(d_q, q_stride, n_tokens, q_heads, cache, d_block_table, max_blocks, d_kv_len, n_reqs, d_out,
                     out_stride);
  if (e != SHN_OK) return e;
  if (n_reqs && !d_cu_q) return SHN_ERR_INVALID_ARG;
  e = check_work(d_work, work_bytes, SHN_KV_WORKSPACE_BYTES);
  if (e != SHN_OK) return e;
  if (n_tokens && d_q == d_out) return SHN_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KvAttnArgs a = {};
  a.q = d_q, a.q_stride = q_stride, a.n_tokens = n_tokens, a.q_heads = q_heads;
  a.table = d_block_table, a.max_blocks = max_blocks, a.cu_q = d_cu_q, a.kv_len = d_kv_len, a.n_reqs = n_reqs;
  a.scale = softmax_scale, a.out = d_out, a.out_stride = out_stride;
  a.st = static_cast<DeviceStatus*>(d_work);  // set by the first launch
  if (n_tokens == 0 || n_reqs == 0) return clear_status(d_work, s) ? SHN_OK : SHN_ERR_CUDA;
  return launch_kv_prompt(pages_of(cache), cache->head_dim, a, sm_count_for_launch(), s) == cudaSuccess ? SHN_OK : SHN_ERR_CUDA;
}

size_t shn_kv_attn_shared_workspace_bytes(const shn_kv_cache* cache, uint32_t n_reqs, uint32_t q_heads) {
  if (check_cache(cache) != SHN_OK || q_heads == 0 || q_heads % cache->kv_heads ||
      q_heads / cache->kv_heads > kMaxGroup || n_reqs >= (1u << 31) / q_heads)
    return 0;
  return n_reqs ? shared_layout(cache, n_reqs, q_heads).total : SHN_KV_WORKSPACE_BYTES;
}

int shn_kv_attn_shared(const uint16_t* d_q, uint64_t q_stride, uint32_t n_reqs, uint32_t q_heads,
                       const shn_kv_cache* cache, const int32_t* d_prefix_pages, uint32_t n_prefix_pages,
                       const int32_t* d_prefix_len, const int32_t* d_block_table, uint32_t max_blocks,
                       const int32_t* d_kv_len, float softmax_scale, uint16_t* d_out, uint64_t out_stride,
                       void* d_work, size_t work_bytes, void* stream) {
  int e = check_attn(d_q, q_stride, n_reqs, q_heads, cache, d_block_table, max_blocks, d_kv_len, n_reqs, d_out,
                     out_stride);
  if (e != SHN_OK) return e;
  if (!d_prefix_len || (n_prefix_pages && !d_prefix_pages) ||
      (uint64_t)n_prefix_pages * cache->page_tokens >= (1ull << 31))
    return SHN_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_reqs == 0) {
    e = check_work(d_work, work_bytes, SHN_KV_WORKSPACE_BYTES);
    return e != SHN_OK ? e : clear_status(d_work, s) ? SHN_OK : SHN_ERR_CUDA;
  }
  SharedLayout x = shared_layout(cache, n_reqs, q_heads);
  e = check_work(d_work, work_bytes, x.total);
  if (e != SHN_OK) return e;
  if (d_q == d_out) return SHN_ERR_INVALID_ARG;
  KvAttnArgs a = {};
  a.q = d_q, a.q_stride = q_stride, a.n_tokens = n_reqs, a.q_heads = q_heads;
  a.table = d_block_table, a.max_blocks = max_blocks, a.kv_len = d_kv_len, a.n_reqs = n_reqs;
  a.prefix_pages = d_prefix_pages, a.n_prefix_pages = n_prefix_pages, a.prefix_len = d_prefix_len;
  a.scale = softmax_scale, a.out = d_out, a.out_stride = out_stride;
  a.st = static_cast<DeviceStatus*>(d_work);  // the last kernel sets it
  uint8_t* wb = static_cast<uint8_t*>(d_work);
  x.pl.out = reinterpret_cast<float*>(wb + x.out_off);
  x.pl.ml = reinterpret_cast<float4*>(wb + x.ml_off);
  x.pl.split_out = reinterpret_cast<float*>(wb + x.split_off);
  x.pl.split_ml = reinterpret_cast<float4*>(wb + x.split_ml_off);
  x.pl.errors = reinterpret_cast<uint32_t*>(wb + x.errors_off);
  const uint64_t prefix_cap = (uint64_t)n_prefix_pages * cache->page_tokens;
  const uint64_t prefix_units = x.pl.prefix_groups * (uint64_t)cache->kv_heads * ((prefix_cap + kUnit - 1) / kUnit);
  if (prefix_cap && (!x.pl.prefix_groups || prefix_units >= kPrefixUnits)) {
    x.pl.prefix_groups = 0;
    // no more parts than the prefix can have tiles of 128 tokens
    if (x.pl.splits > (prefix_cap + 127) / 128) x.pl.splits = (uint32_t)((prefix_cap + 127) / 128);
  } else {
    x.pl.splits = 0;
    if (!prefix_cap) x.pl.prefix_groups = 0;
  }
  // warps: two blocks on each SM (one for 16 rows, which takes more registers), but no more than there can be units
  const uint64_t units = (uint64_t)cache->kv_heads * x.pl.prefix_groups * (((uint64_t)n_prefix_pages * cache->page_tokens + kUnit - 1) / kUnit) +
                         (uint64_t)n_reqs * cache->kv_heads * x.pl.own_groups * (((uint64_t)max_blocks * cache->page_tokens + kUnit - 1) / kUnit + 1);
  const uint64_t per_block = kDecodeThreads / 32;
  uint64_t blocks = (uint64_t)sm_count_for_launch() * (x.pl.rows == 8 ? 2 : 1);
  if (blocks > (units + per_block - 1) / per_block) blocks = (units + per_block - 1) / per_block;
  if (blocks > kDecodeMaxWarps / per_block) blocks = kDecodeMaxWarps / per_block;
  x.pl.warps = (uint32_t)(blocks * per_block);
  x.pl.n_errors = (uint32_t)(x.prefix_tiles * x.pl.splits + blocks);
  if (x.pl.splits && launch_kv_prefix(pages_of(cache), cache->head_dim, a, x.pl, s) != cudaSuccess) return SHN_ERR_CUDA;
  return launch_kv_decode(pages_of(cache), cache->head_dim, a, x.pl, s) == cudaSuccess ? SHN_OK : SHN_ERR_CUDA;
}

}  // extern "C"
