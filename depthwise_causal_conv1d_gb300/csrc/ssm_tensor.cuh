// Building blocks of the chunked scan and of the 4-bit products: the fifth-generation tensor cores (tcgen05) and their
// memory (TMEM), shared-memory operand descriptors, and tiled copies.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "ccu_bulk.cuh"
#include "ssm_internal.cuh"

namespace ccu {

// Tensor map of a 16-bit tensor [rows, groups, inner] (inner contiguous; base and strides multiples of 16 bytes),
// boxes of box_rows x 1 x box_inner.
cudaError_t encode_tiles(CUtensorMap *map, const void *data, int64_t inner, int64_t groups, int64_t rows, int64_t stride_group,
                         int64_t stride_row, int box_inner, int box_rows, CUtensorMapSwizzle swizzle);

namespace tensor {

// ---------------------------------------------------------------- operands in shared memory
//
// An operand tile is stored as blocks of rows of 128 bytes (64 BF16), whose eight 16-byte
// chunks are permuted within a row: chunk c of row r sits at c ^ (r % 8) (the 128-byte swizzle;
// a block starts on a 1024-byte boundary). Read along its rows (K-major) or across them
// (MN-major), a tile serves as either operand.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

constexpr uint64_t kSwizzle128 = uint64_t(2) << 61, kDescVersion = uint64_t(1) << 46;
constexpr uint64_t kEightRows = uint64_t(1024 >> 4) << 32;  // 8 rows of 128 bytes to the next 8

// K-major: a row of the tile is a row of the operand; the next 16 K are 32 bytes on.
__device__ __forceinline__ uint64_t desc_k_major(uint32_t smem) {
  return kSwizzle128 | kDescVersion | kEightRows | (uint64_t(1) << 16) | ((smem >> 4) & 0x3fff);
}
// MN-major: a row of the tile is one K; the next 16 K are 16 rows on, the next 64 rows of the
// operand `block` bytes on.
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t smem, uint32_t block) {
  return kSwizzle128 | kDescVersion | kEightRows | (uint64_t(block >> 4) << 16) | ((smem >> 4) & 0x3fff);
}

// Instruction descriptor: BF16 operands, FP32 accumulator, shapes, and which operands are MN-major.
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) |
         (uint32_t(m >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// A in TMEM: lane = row, two K to a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// True for one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// Arrives on the mbarrier when all tensor work this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bulk::smem_addr(bar)) : "memory");
}

// ---------------------------------------------------------------- TMEM

// Whole warps. `columns` a power of two >= 32; the address is written to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bulk::smem_addr(where)), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Behind wait_loads(): the compiler knows the loaded registers but not the wait, and could use
// them before it; passing through here keeps their uses behind.
template <int N>
__device__ __forceinline__ void loaded(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: lane l of the warp gets row l's 32 values. The address
// names the warp's first lane (bits 16..) and the first column.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// ---------------------------------------------------------------- copies and barriers

// Two (three) waits in one: a wait that is over takes some 200 cycles in a full SM, and those of a
// loop's turn one after the other take longer than the tensor cores' work. False: the limit ran out.
__device__ __forceinline__ bool wait_phases(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1, uint64_t *bar2,
                                            uint32_t parity2) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %7;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
      "and.pred p, p, q;\n\t"
      "and.pred p, p, r;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bulk::smem_addr(bar0)), "r"(parity0), "r"(bulk::smem_addr(bar1)), "r"(parity1), "r"(bulk::smem_addr(bar2)), "r"(parity2),
        "n"(bulk::kMaxSpins)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_phases(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %5;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bulk::smem_addr(bar0)), "r"(parity0), "r"(bulk::smem_addr(bar1)), "r"(parity1), "n"(bulk::kMaxSpins)
      : "memory");
  return done != 0;
}

// One box of a rank-3 tensor map into a swizzled tile; completes its bytes on `bar`. The first
// coordinate is a multiple of 8 BF16 (16 bytes).
__device__ __forceinline__ void tile_load(uint32_t smem, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bulk::smem_addr(bar))
      : "memory");
}

// The same box into L2 only.
__device__ __forceinline__ void tile_prefetch(const CUtensorMap *map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(c0), "r"(c1), "r"(c2) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) { asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory"); }

}  // namespace tensor
}  // namespace ccu
