// The fifth-generation tensor cores: descriptors, matrix instructions, tensor
// memory, and tiled bulk copies, as the paged attention uses them.
#pragma once

#include <cuda.h>

#include "dd_internal.cuh"

namespace dd {
namespace tc {

// ------------------------------------------------------------------ TMA
// Load a box of a 3-D tensor map; completion on `bar`.  x times the element
// size is a multiple of 16 bytes; coordinates outside the tensor read zeros.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
// Store a box; tracked by the issuing thread's bulk async-groups.  No negative
// coordinates; what lies outside the tensor is not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y,
                                             int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::
                   "l"(map),
               "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
using dd::fence_async_smem;

// -------------------------------------------------------------- descriptors
// Shared-memory matrix descriptor for the 128-byte swizzle: bits 0-13 the
// address, 16-29 the leading and 32-45 the stride byte offset (all in units of
// 16 bytes), 46-47 the descriptor version (1), 61-63 the swizzle (2 = 128 B).
// A tile is stored as panels of 64 two-byte elements (128 bytes) by its rows.
//   contraction along the 128 bytes: 8-row groups 1024 bytes apart (stride);
//     16 elements further along are 32 bytes further on;
//   contraction along the rows: 8-row groups 1024 bytes apart (stride), panels
//     `panel` bytes apart (leading); 16 rows further are 2048 bytes further on.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t panel) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)((panel >> 4) & 0x3FFF) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// A descriptor `bytes` further on (a multiple of 16 that stays in shared memory):
// only the address field changes, and it does not overflow.
__device__ __forceinline__ uint64_t further(uint64_t desc, uint32_t bytes) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(desc));
  lo += bytes >> 4;
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
// True for one thread of a converged warp.  Code behind it is known to run in a
// single thread, so descriptors stay in the uniform registers that the matrix
// instructions take; behind `lane == 0` each would be moved there every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r));
  return r != 0;
}
// Instruction descriptor: bf16 A and B, fp32 D, M x N; b_rows: B's contraction
// runs along its rows.
__host__ __device__ constexpr uint32_t instr_bf16(int M, int N, bool b_rows) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_rows ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ----------------------------------------------------- matrix instructions
// D[tmem] (+)= A B with A and B in shared memory / A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// One arrival on `bar` once every matrix instruction this thread issued is done.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ----------------------------------------------------------- tensor memory
// By one whole warp; the address comes back through shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
// 32 columns of the warp's 32 lanes: thread i has lane i's.
#define DD_R8(f, n) f(n), f(n + 1), f(n + 2), f(n + 3), f(n + 4), f(n + 5), f(n + 6), f(n + 7)
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
#define DD_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : DD_R8(DD_OUT, 0), DD_R8(DD_OUT, 8), DD_R8(DD_OUT, 16), DD_R8(DD_OUT, 24)
      : "r"(addr)
      : "memory");
#undef DD_OUT
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
#define DD_IN(i) "r"(r[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          addr),
      DD_R8(DD_IN, 0), DD_R8(DD_IN, 8), DD_R8(DD_IN, 16), DD_R8(DD_IN, 24)
      : "memory");
#undef DD_IN
}
// Registers that a load fills are used only behind this (it names them, so no
// use of them can be moved ahead of the wait before it).
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_loaded32(uint32_t* r) {
#define DD_IO(i) "+r"(r[i])
  asm volatile("" : DD_R8(DD_IO, 0), DD_R8(DD_IO, 8), DD_R8(DD_IO, 16), DD_R8(DD_IO, 24));
#undef DD_IO
}
#undef DD_R8
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Registers of the warpgroup's threads (all four warps call it).
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------- work of waiting CTAs
// A running CTA asks for the place of a CTA of this grid that has not started
// (it then never does) and computes that CTA's work itself: 16 bytes of answer
// on `bar`.  After an answer of "none" it must not ask again.
__device__ __forceinline__ void ask_for_work(uint4* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(smem_addr(answer)),
      "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ bool work_given(const uint4* answer, int& x, int& y, int& z) {
  uint32_t given, a, b, c;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
      " ld.shared.b128 r, [%4];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, r;\n}\n"
      : "=r"(given), "=r"(a), "=r"(b), "=r"(c)
      : "r"(smem_addr(answer))
      : "memory");
  x = (int)a;
  y = (int)b;
  z = (int)c;
  return given != 0;
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace tc
}  // namespace dd
