// What the GEMM sources share: tensor-core instructions (tcgen05) and their
// descriptors, the staging of stores, and on the host the operands' tensor maps.
#pragma once

#include "common.cuh"

namespace mxq {
namespace gemm {

constexpr int BM = 128;
constexpr int BKB = 128;                 // bytes of codes per row per stage
constexpr int STG_BYTES = BM * 64;       // one staging buffer: 128 rows x 64 B

// Operand kinds (a template parameter of the kernels).
constexpr int KIND_MXF8 = 0;   // block-scaled E4M3 / E5M2: kind::mxf8f6f4, scale_vec::1X
constexpr int KIND_MXF4 = 1;   // block-scaled E2M1 (packed): kind::mxf4, scale_vec::2X
constexpr int KIND_F8 = 2;     // per-tensor E4M3 / E5M2: kind::f8f6f4, no block scales

// ---------------------------------------------------------------- tcgen05 wrappers
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

__device__ __forceinline__ void tc_cp_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

template <int KIND>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t acc) {
  if constexpr (KIND == KIND_MXF4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
  } else if constexpr (KIND == KIND_MXF8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  }
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// CTA-pair forms: issued by one thread of the pair's first CTA (alloc and
// dealloc by one warp of each CTA); shared-memory descriptors and tensor
// memory addresses name the same offsets in both CTAs.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// arrive on the mbarrier at this offset in both CTAs once the issued work is done
__device__ __forceinline__ void tc_commit_pair_both(uint32_t bar) {
  const uint16_t mask = 3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void tc_commit_pair_self(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_cp_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
template <int KIND>
__device__ __forceinline__ void tc_mma_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  if constexpr (KIND == KIND_MXF4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
  } else if constexpr (KIND == KIND_MXF8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  }
}

__device__ __forceinline__ void named_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// Shared-memory matrix descriptor (tcgen05 format): start address, leading
// and stride byte offsets (>> 4), fixed version field 1 at bit 46, swizzle
// mode at bits 61-63 (2 = 128-byte swizzle, 0 = none).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swz) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  d |= static_cast<uint64_t>(swz & 7u) << 61;
  return d;
}

// Instruction descriptor of the block-scaled MMA: A and B element type codes
// at bits 7-9 and 10-12 (kind::mxf8f6f4: E4M3 0, E5M2 1; kind::mxf4: E2M1 1),
// K-major operands, N >> 3 at bits 17-22, scale type UE8M0 (bit 23), M >> 4
// at bits 24-28, scale-factor byte selectors for B (bits 4-5) and A (29-30).
__host__ __device__ constexpr uint32_t instr_desc(uint32_t a_type, uint32_t b_type, int n, int m, uint32_t sf_id) {
  return (sf_id << 4) | (a_type << 7) | (b_type << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 4) << 24) | (sf_id << 29);
}

// Instruction descriptor of the unscaled kind::f8f6f4 MMA: float32
// accumulator (bits 4-5 = 1), A / B element types at bits 7-9 / 10-12,
// A / B major-ness at bits 15 / 16 (0 K-major, 1 MN-major), N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t instr_desc_f8(uint32_t a_type, uint32_t b_type, int n, int m, uint32_t a_mn,
                                                     uint32_t b_mn) {
  return (1u << 4) | (a_type << 7) | (b_type << 10) | (a_mn << 15) | (b_mn << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Shared-memory descriptor of an operand tile and the descriptor step from
// one 32-byte K slice to the next (16-byte units).  Both layouts are what a
// TMA load with the 128-byte swizzle writes: K-major -- 128-byte rows along
// K, one per M (N) index, 8-row groups 1024 bytes apart; MN-major -- 128-byte
// rows along M (N), one per K index (the tile is 128 elements wide: a single
// swizzle atom across), 8-row groups along K 1024 bytes apart, so a 32-deep
// K slice is 32 rows = 4096 bytes.  An MN-major tile has one atom across,
// so the atom stride across M (N) is never used; it is set to the 8-row
// group stride as well.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, int mn) {
  return mn ? smem_desc(addr, 1024, 1024, 2) : smem_desc(addr, 16, 1024, 2);
}
__device__ __forceinline__ uint32_t k_slice_step(int mn) { return mn ? 256u : 2u; }

// Before a staging buffer is rewritten: with two buffers the bulk store
// issued from this one two chunks ago must have read it (at most one store
// group still reading); with one buffer the last store must have.
template <int NBUF>
__device__ __forceinline__ void bulk_wait_read_staging() {
  if constexpr (NBUF == 2) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

}  // namespace gemm
}  // namespace mxq

// ---------------------------------------------------------------- host side
namespace mxq_host {

// An operand's code map: 128-byte K steps of `box_rows` rows, 128-byte
// swizzle.  Codes are bytes (8-bit formats, or packed E2M1 for kind::mxf4,
// kbytes = K / 2).  Packed E2M1 beside an 8-bit operand (kind::mxf8f6f4)
// goes through the 16 x 4-bit type that widens every 8 packed bytes to a
// 16-byte slot: a K step is then 128 elements in the same 128 bytes of
// shared memory per row as an 8-bit operand, the layout the tensor core
// reads for 4-bit elements of that kind, and the map's x coordinate counts
// elements, so the kernels' coordinates (kb * 128) are unchanged.
inline bool encode_operand(CUtensorMap* m, const void* q, bool u4, int64_t K, int64_t kbytes, uint64_t rows,
                    uint32_t box_rows) {
  using namespace mxq::gemm;
  if (u4)
    return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, q, K, rows, K / 2, 128, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
  return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, kbytes, rows, kbytes, BKB, box_rows,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

// Transaction bytes of one operand tile: the widened E2M1 load completes the
// packed bytes it reads (half its shared-memory footprint; the padding
// slots are not written).
constexpr uint32_t tx_bytes(int smem_bytes, bool u4) { return static_cast<uint32_t>(u4 ? smem_bytes / 2 : smem_bytes); }

// Element type code of the MMA's instruction descriptor: E4M3 0 and E5M2 1
// (kind::mxf8f6f4 / f8f6f4); E2M1 1 in kind::mxf4 and 5 in kind::mxf8f6f4.
inline uint32_t mma_type(int fmt, bool kind_mxf4) {
  if (fmt == MXQ_E2M1) return kind_mxf4 ? 1u : 5u;
  return fmt == MXQ_E4M3 ? 0u : 1u;
}

inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

inline bool valid_fmt(int f) { return f == MXQ_E4M3 || f == MXQ_E5M2 || f == MXQ_E2M1; }

}  // namespace mxq_host
