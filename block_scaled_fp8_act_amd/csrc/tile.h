// Building blocks of the tiled products: the LDS layout of a K-block's rows,
// direct-to-LDS loads, and the mapping of workgroups to tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsfp8 {
namespace {

constexpr int BK = 128;
constexpr int kXcds = 8;
constexpr int kGroupM = 8;

// Byte offset of 16-byte chunk c of tile row r in LDS.  The chunk index is
// XOR-ed with (r & 7) ^ ((r >> 3) & 1), which gives distinct chunks to the 8
// rows of each aligned group of 8 and distinct (row parity, chunk) pairs to
// the 16 rows of each aligned group of 16.  An MFMA fragment read (16
// consecutive rows, one logical chunk) is then free of bank conflicts whether
// the LDS serves it as 8 lanes over 128 bytes of banks or as 16 lanes over
// 256 bytes (measured: no SQ_LDS_BANK_CONFLICT cycles, against 42% of the
// LDS's active cycles with (r >> 1) & 7 or r & 7).  The key repeats every 16
// rows, so all fragment reads of a wave share their lane offsets.
__device__ __forceinline__ int swz_key(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swz(int r, int c) { return r * BK + ((c ^ swz_key(r)) << 4); }

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The loads are issued from inline assembly so that the compiler, which
// cannot tell the stages of the ring apart, does not add a vmcnt(0) wait in
// front of every LDS read; the kernel waits for each stage itself.  M0 holds
// the wave's LDS destination and is set in the same statement (and declared
// clobbered, so the compiler keeps nothing of its own in M0 across it); the
// s_nop provides the wait state required between an SALU write of M0 and an
// LDS DMA that reads it.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

// M0 is a reserved register, so clang warns that a clobber of it is not
// saved and restored around the statement; that is intended (nothing needs
// the old value), and the clobber still records the write of M0 in the
// statement's dependencies, so no instruction of the compiler's that reads
// M0 is moved across it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// Byte address of lane l: rsrc base + voff + soff (the scalar part carries the
// K-block offset, so the per-lane offsets stay fixed over the K loop).
__device__ __forceinline__ void dma_b128(i32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

// Four bytes per lane (for rows that are only 4-byte aligned).
__device__ __forceinline__ void dma_b32(i32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

// The same with the nontemporal hint: for weight panels that one tile
// streams once (the short, wide tiles of the grouped and gated products).
__device__ __forceinline__ void dma_b128_nt(i32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

// Per-lane 64-bit addresses: each active lane fetches one dword from anywhere.
__device__ __forceinline__ void dma_gather_b32(uint32_t lds, const float* addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(addr)
               : "memory", "m0");
}

#pragma clang diagnostic pop

// The lane index behind an empty statement: values derived from it are
// computed where they are used instead of being hoisted out of a persistent
// kernel's tile loop, where they would stay live across the K loop.
__device__ __forceinline__ int lane_id() {
  int l = (int)(threadIdx.x & 63);
  asm volatile("" : "+v"(l));
  return l;
}

constexpr uint32_t kOob = 0x80000000u;  // above every descriptor's size

__device__ __forceinline__ i32x4 make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));  // stride 0: raw buffer
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

// Wait until at most n vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Workgroup i runs on XCD i % 8.  Renumber ids 0..total-1 so that each XCD
// owns one contiguous range (and so shares its L2 among neighbouring tiles).
__device__ __forceinline__ int64_t xcd_contiguous(int64_t pid, int64_t total) {
  const int64_t q = total / kXcds, r = total % kXcds;
  const int64_t xcd = pid % kXcds, idx = pid / kXcds;
  return (xcd < r) ? xcd * (q + 1) + idx : r * (q + 1) + (xcd - r) * q + idx;
}

// x / d for x >= 0, d > 0 (tile-index arithmetic at the start of a tile):
// the 32-bit division whenever both fit, since a 64-bit integer division is
// a long instruction sequence that delays the tile's first loads.
__device__ __forceinline__ int64_t div_u(int64_t x, int64_t d) {
  if ((uint64_t)(x | d) <= 0xffffffffull) return (int64_t)((uint32_t)x / (uint32_t)d);
  return x / d;
}

// Map a linear workgroup id to (tile_m, tile_n): XCD-contiguous ranges, then
// GROUP_M-row groups inside a range.
__device__ __forceinline__ void tile_of(int64_t pid, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
  const int64_t total = tiles_m * tiles_n;
  pid = xcd_contiguous(pid, total);
  const int64_t per_group = (int64_t)kGroupM * tiles_n;
  const int64_t gid = div_u(pid, per_group);
  const int64_t first_m = gid * kGroupM;
  const int64_t gsize = (tiles_m - first_m) < kGroupM ? (tiles_m - first_m) : kGroupM;
  const int64_t in = pid - gid * per_group;
  tn = div_u(in, gsize);
  tm = first_m + (in - tn * gsize);
}

}  // namespace
}  // namespace dsfp8
