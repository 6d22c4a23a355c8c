// kv_tc.cuh — the tensor core and barrier instructions of the cache attention (sm_100a), packed float32 arithmetic, and the
// exact INT8 -> fp16 step in front of the products.
#pragma once

#include <cuda_fp16.h>

#include "kv_internal.cuh"

namespace shn {
namespace tc {

// ---- mbarriers, with bounded waits ---------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared.b64 p, [%1], %2, 2000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits for the phase of this parity, at most kWaitTries tries of 2000 ns each: a quarter of a second, where a legitimate
// wait here is microseconds. False: gave up, or another warp of the block did, which *stop tells. (A build for tests may set
// fewer tries; the products that a block has in flight are waited for with the full limit all the same.)
#ifndef SHN_KV_WAIT_TRIES
#define SHN_KV_WAIT_TRIES (1u << 17)
#endif
constexpr uint32_t kWaitTries = SHN_KV_WAIT_TRIES, kDrainTries = 1u << 17;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t stop) {
  for (uint32_t i = 0; i != kWaitTries; ++i) {
    if (bar_try(bar, parity)) return true;
    if ((i & 63u) == 63u && lds32(stop) != 0) return false;
  }
  sts32(stop, 1u);
  return false;
}

// ---- blocks of a cluster -------------------------------------------------------------------------
// Every thread of every block that has not left; what was written before is seen by all behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The same place in shared memory of another block
__device__ __forceinline__ uint32_t in_block(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_cluster32(uint32_t a, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_block(a, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_cluster64(uint32_t a, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(in_block(a, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster128(uint32_t a, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(in_block(a, rank))
               : "memory");
  return v;
}

// ---- tcgen05 -------------------------------------------------------------------------------------
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// true in one thread of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// The instructions below are issued by the thread whose `lead` is set, the rest of the warp passing over them under a
// predicate: control flow stays the warp's, and operands that are the same in all its threads stay in uniform registers.
__device__ __forceinline__ void commit(uint32_t bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"((uint32_t)lead)
      : "memory");
}

// Shared-memory operand in the 128-byte swizzle: rows of 128 bytes (64 fp16), the 16-byte pieces of row r exchanged by
// XOR with r mod 8, 8 rows (1024 bytes) to an atom. `lbo`: bytes between blocks of 64 along the other axis
// (only an operand whose rows run along K, i.e. an MN-major one, wider than 64 uses it).
// The descriptor's low word; the high one is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16; }
// kind::f16 instruction descriptor: f32 accumulator, fp16 operands, M x N; b_rows_along_k: B is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(uint32_t m, uint32_t n, bool b_rows_along_k) {
  return (1u << 4) | ((b_rows_along_k ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "n"(kAdd), "r"((uint32_t)lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add, bool lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "r"((uint32_t)add), "r"((uint32_t)lead)
      : "memory");
}

#define SHN_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define SHN_I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
// 32 columns of the warp's 32 lanes: thread = lane, register = column
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SHN_R8(v, 0), SHN_R8(v, 8), SHN_R8(v, 16), SHN_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void ld8(uint32_t addr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : SHN_R8(v, 0) : "r"(addr));
}
// 16 lanes: thread t holds rows t/4 (registers 0, 1) and t/4 + 8 (registers 2, 3) of columns 2(t%4), 2(t%4) + 1 of
// each 8 columns; 4 registers per 8 columns
__device__ __forceinline__ void ld_quad32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SHN_R8(v, 0), SHN_R8(v, 8), SHN_R8(v, 16), SHN_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void ld_quad8(uint32_t addr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : SHN_R8(v, 0) : "r"(addr));
}
__device__ __forceinline__ void st_quad8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), SHN_I8(v, 0) : "memory");
}
// 16 lanes, packed pairs: thread t holds rows t/4 and t/4 + 8 (registers 0, 1) of column t%4 of each 4 columns
__device__ __forceinline__ void st_pairs8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), SHN_I8(v, 0) : "memory");
}

// ---- arithmetic ----------------------------------------------------------------------------------
// Two float32 per instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Shared memory that nothing writes while they are read. The compiler may place the load freely after what
// the address depends on; `after_here` makes an address depend on a place in the program (behind a wait).
__device__ __forceinline__ uint32_t after_here(uint32_t a) {
  asm volatile("" : "+r"(a)::"memory");
  return a;
}
__device__ __forceinline__ float lds32_free(uint32_t a) {
  float v;
  asm("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint64_t lds64_free(uint32_t a) {
  uint64_t v;
  asm("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^n, exactly, for a whole number n in [-126, 127]
__device__ __forceinline__ float pow2(float n) { return __int_as_float(((int)n + 127) << 23); }

__device__ __forceinline__ float pow2i(int32_t n) { return __int_as_float((n + 127) << 23); }

// (lo, hi) rounded to fp16, packed
__device__ __forceinline__ uint32_t fp16_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp16 of 1024 + u, u = x + 128 (a byte in the last bits of 0x6400), minus 1152: x, exactly.
__device__ __forceinline__ uint32_t minus1152(uint32_t t) {
  uint32_t x;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(t), "r"(0x64806480u));
  return x;
}
// The 4 bytes of w in order, as 2 x fp16x2, exactly.
__device__ __forceinline__ uint2 fp16x4_of_int8(uint32_t w) {
  w ^= 0x80808080u;
  return make_uint2(minus1152(__byte_perm(w, 0x64646464u, 0x4140)), minus1152(__byte_perm(w, 0x64646464u, 0x4342)));
}
__device__ __forceinline__ uint32_t fp16x2_times(uint32_t x, uint32_t f) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(f));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t piece) { return row * 128u + ((piece ^ (row & 7u)) << 4); }

}  // namespace tc
}  // namespace shn
