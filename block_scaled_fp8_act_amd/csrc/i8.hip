// int8 linear layer on gfx950: row quantisation and the product of int8
// matrices with a scale for each row of both.
//
// Quantisation of a row x (a token, or an output channel of a weight):
//   a = max(max |x|, 2^-100),  s = a / 127,  y = rne(x * (127 / a)),
// each step one fp32 operation, so the codes can be stated bit for bit.  The
// maximum is taken over the bit patterns of |x| as integers, in which NaN >
// infinity > every finite value: a row that holds one gets a scale that shows
// it.
//
// Product: C = bf16((sum_k A B) * (a_s * b_s)).  The integer sums are exact,
// so nothing depends on their order.
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "tile.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));  // an access at any address
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr float kAmaxFloor = 0x1p-100f;  // 127 / a and a / 127 stay normal

// ---- row quantisation ----------------------------------------------------------------

typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

enum Src { kBf16, kF32, kGated };

// SiLU(g) * u in fp32, within (|g| + 8) 2^-23 of it: the exponential's argument
// is rounded once, everything else is within a few 2^-24.
__device__ __forceinline__ float gate(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Eight consecutive input elements as loaded, and as fp32 values.
template <Src SRC>
struct Chunk {
  u32x4 r[SRC == kBf16 ? 1 : 2];

  // Elements k .. k + 7 of row m, all of them in the row; zeros if not `on`.
  __device__ __forceinline__ void load(const RowQuantArgs& a, int64_t m, int64_t k, bool on) {
#pragma unroll
    for (auto& w : r) w = u32x4{0u, 0u, 0u, 0u};
    if (!on) return;
    if constexpr (SRC == kF32) {
      const float* src = static_cast<const float*>(a.x) + m * a.ldx + k;
      r[0] = *reinterpret_cast<const u32x4u*>(src);
      r[1] = *reinterpret_cast<const u32x4u*>(src + 4);
    } else {
      r[0] = *reinterpret_cast<const u32x4u*>(static_cast<const uint16_t*>(a.x) + m * a.ldx + k);
      if constexpr (SRC == kGated) r[1] = *reinterpret_cast<const u32x4u*>(a.u + m * a.ldu + k);
    }
  }

  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (SRC == kF32) {
        v[i] = __uint_as_float(r[0][i]);
        v[4 + i] = __uint_as_float(r[1][i]);
      } else {
        v[2 * i] = bf16_lo(r[0][i]);
        v[2 * i + 1] = bf16_hi(r[0][i]);
        if constexpr (SRC == kGated) {
          v[2 * i] = gate(v[2 * i], bf16_lo(r[1][i]));
          v[2 * i + 1] = gate(v[2 * i + 1], bf16_hi(r[1][i]));
        }
      }
    }
  }

  // Keep the gate's result in place of its inputs.
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i >> 2][i & 3] = __float_as_uint(v[i]);
  }
};

// The largest |v| as a bit pattern (NaN > infinity > finite).
__device__ __forceinline__ uint32_t max_abs(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  return top;
}

__device__ __forceinline__ uint32_t max_u32_wave(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// Eight codes.  Adding 1.5 * 2^23 rounds a product to an integer (nearest
// even) and leaves it in the low bits as two's complement.
__device__ __forceinline__ u32x2u codes8(const float (&v)[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(v[i] * inv + 0x1.8p23f);
  u32x2u r;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    r[h] = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u) |
           __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000c0cu);
  return r;
}

// TPR threads per row, NC chunks of 8 elements per thread: the row stays in
// registers between the maximum and the codes, so it is read once (NC = 0: a
// longer row is read twice).  A row's last chunk starts at K - 8: where it
// overlaps the one before, the same codes are written twice.  K >= 8.
// Bound by memory: bf16 [4096, 7168] 16.9 us, 5.2 TB/s of its 88 MB (reading the
// row twice, 54.9 us), gated [4096, 18432] 68-73 us, 5.2-5.5 TB/s (275 us), fp32
// [4096, 7168] 26.7 us, 5.5 TB/s of 147 MB; a few rows are bound by the launch and
// one trip to memory (32 rows of 7168: 3.5 us).
template <Src SRC, int TPR, int NC>
__global__ __launch_bounds__(256) void row_quant_kernel(RowQuantArgs a) {
  constexpr int RPB = 256 / TPR;
  constexpr int N = NC > 0 ? NC : 4;
  constexpr Src kHeld = SRC == kGated ? kF32 : SRC;  // what a held chunk contains
  __shared__ uint32_t red[4];
  const int t = threadIdx.x % TPR;
  const int nch = (int)((a.K + 7) >> 3);
  const int passes = NC > 0 ? 1 : (nch + N * TPR - 1) / (N * TPR);
  auto at = [&](int c) { return c < nch - 1 ? 8 * (int64_t)c : a.K - 8; };
  for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < a.M; m += (int64_t)gridDim.x * RPB) {
    Chunk<kHeld> held[N];
    uint32_t top = __float_as_uint(kAmaxFloor);
    auto fetch = [&](int p) __attribute__((always_inline)) {
      Chunk<SRC> in[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = t + TPR * (i + N * p);
        in[i].load(a, m, at(c), c < nch);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v[8];
        in[i].values(v);
        top = max_abs(v, top);
        if constexpr (SRC == kGated) held[i].set(v);
        else held[i] = in[i];
      }
    };
    for (int p = 0; p < passes; ++p) fetch(p);
    top = max_u32_wave(top);
    if constexpr (TPR == 256) {
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; ++w) top = red[w] > top ? red[w] : top;
      __syncthreads();
    }
    const float amax = __uint_as_float(top);
    const float inv = 127.0f / amax;
    for (int p = 0; p < passes; ++p) {
      if constexpr (NC == 0) fetch(p);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = t + TPR * (i + N * p);
        float v[8];
        held[i].values(v);
        if (c < nch) *reinterpret_cast<u32x2u*>(a.y + m * a.ldy + at(c)) = codes8(v, inv);
      }
    }
    if (t == 0) a.s[m] = amax / 127.0f;
  }
}

// Rows of fewer than 8 elements: one thread each, bound by the launch.
__global__ __launch_bounds__(256) void row_quant_short_kernel(RowQuantArgs a) {
  for (int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x; m < a.M; m += (int64_t)gridDim.x * 256) {
    float v[8];
    for (int k = 0; k < 8; ++k) {
      v[k] = 0.0f;
      if (k >= a.K) continue;
      if (a.f32) {
        v[k] = static_cast<const float*>(a.x)[m * a.ldx + k];
      } else {
        v[k] = bf16_lo(static_cast<const uint16_t*>(a.x)[m * a.ldx + k]);
        if (a.u != nullptr) v[k] = gate(v[k], bf16_lo(a.u[m * a.ldu + k]));
      }
    }
    const float amax = __uint_as_float(max_abs(v, __float_as_uint(kAmaxFloor)));
    const u32x2u c = codes8(v, 127.0f / amax);
    for (int k = 0; k < a.K; ++k) a.y[m * a.ldy + k] = (int8_t)(c[k >> 2] >> (8 * (k & 3)));
    a.s[m] = amax / 127.0f;
  }
}

// ---- product ---------------------------------------------------------------------------

// 16 bytes of a row of K >= 16 bytes from column k, at any address; those past
// the row are zero.  Nothing outside the row is read: a chunk that the row's
// end cuts is taken from the last 16 bytes and shifted.
template <bool TAIL>
__device__ __forceinline__ u32x4 load16(const int8_t* row, int64_t k, int64_t K) {
  if (!TAIL || k + 16 <= K) return *reinterpret_cast<const u32x4u*>(row + k);
  const int64_t past = k + 16 - K;
  if (past >= 16) return u32x4{0u, 0u, 0u, 0u};
  const u32x4 v = *reinterpret_cast<const u32x4u*>(row + K - 16);
  const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v) >> (8 * (int)past);
  return __builtin_bit_cast(u32x4, w);
}

// ---- tiles ---------------------------------------------------------------------------
//
// BM x BN tiles, each wave WM x WN of it, as in the block-scaled products: a
// ring of STAGES K-blocks of 128 bytes per row, filled by buffer_load ... lds
// (rows past the matrix and chunks past K read as zero through the
// descriptor), one barrier per K-block, the loads of a later K-block issued
// between the MFMAs of the current one.  Nothing is rescaled inside the K
// loop, so the accumulators stay where the matrix instruction leaves them.
// The weight fragment is the instruction's first operand, so a lane's results
// are runs of four columns of one row.
// Large products are bound by the matrix cores at the clock that the card's power
// allows: 4096x18432x7168 455 us (2380 TOPS) and 4096x7168x18432 430 us (2520),
// in 256x256 tiles of eight 128x64 waves; waves of 64x128, sixteen of 64x64 or
// four of 128x128 were slower.  Smaller tiles serve products whose 256x256 tiles
// would leave CUs idle (kVariants).
//
// Operands whose rows are aligned to 4 bytes alone take the same path in loads
// of 4 bytes (through registers instead, 333x2500x1000 took 11.0 us against 7.7).
// A weight with rows at any address is loaded as aligned dwords where the
// activations are the quantiser's (I8LoaderShift: 700x4097x4099 with its
// quantisation 41.9 us against 48.9 through registers, 4096x7169x2051 101.6
// against 105.6).  Other operands go through registers (I8RegLoader): the next
// K-block's chunks are loaded before the MFMAs of the current one and written to
// the other stage after them.

typedef int v16i __attribute__((ext_vector_type(16)));

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct I8Cfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
  static constexpr int NW = WAVES_M * WAVES_N;
  static constexpr int kThreads = 64 * NW;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int TM = WM / 32, TN = WN / 32;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int A_INSTR = A_BYTES / 1024 / NW, B_INSTR = B_BYTES / 1024 / NW, LOADS = A_INSTR + B_INSTR;
  static constexpr int C_BYTES = 32 * WN * 2;  // 32 rows of a wave's output
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole 1 KB segments per wave");
  static_assert(WM % 32 == 0 && WN % 32 == 0, "32x32 subtiles");
  static_assert(NW % 2 == 0, "a wave's segments start at rows that agree modulo 16");
  static_assert(STAGES >= 2 && STAGES <= 4 && LOADS * (STAGES - 2) < 64, "the waits of the K loop");
};

template <class CF>
struct I8Loader {
  static constexpr int LOADS = CF::LOADS, STAGE_BYTES = CF::STAGE_BYTES;
  i32x4 rsA, rsB;
  uint32_t off[CF::LOADS];
  uint32_t kc;  // byte within the K-block of every load's chunk (a wave's rows agree modulo 16)
  uint32_t lds0;
  uint32_t K;
  int wave;

  __device__ __forceinline__ void init(const GemmI8Args& p, int64_t m0, int64_t n0, uint8_t* smem) {
    const int lane = lane_id();
    wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    K = (uint32_t)p.K;
    const int64_t ra = p.M - m0 < CF::BM ? p.M - m0 : CF::BM, rb = p.N - n0 < CF::BN ? p.N - n0 : CF::BN;
    rsA = make_rsrc(p.A + m0 * p.lda, (uint32_t)((ra - 1) * p.lda + p.K));
    rsB = make_rsrc(p.B + n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb + p.K));
    kc = (uint32_t)((lane & 7) ^ swz_key(wave * 8 + (lane >> 3))) * 16;
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n) {
      const bool a = n < CF::A_INSTR;
      const int r = (wave + CF::NW * (a ? n : n - CF::A_INSTR)) * 8 + (lane >> 3);
      off[n] = r < (a ? ra : rb) ? (uint32_t)(r * (a ? p.lda : p.ldb)) + kc : kOob;
    }
    lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem));
  }

  template <bool KFULL>
  __device__ __forceinline__ void issue(int n, int kb, int stage) const {
    const bool a = n < CF::A_INSTR;
    const uint32_t kbyte = (uint32_t)kb * BK;
    const bool in = KFULL || kbyte + kc < K;
    const uint32_t at = lds0 + (uint32_t)(stage * CF::STAGE_BYTES + (a ? 0 : CF::A_BYTES) +
                                          (wave + CF::NW * (a ? n : n - CF::A_INSTR)) * 1024);
    dma_b128(a ? rsA : rsB, at, in ? off[n] : kOob, kbyte);
  }
  __device__ __forceinline__ void finish(uint8_t*, int) const {}
};

// The same with four bytes per lane, for rows that are only 4-byte aligned (K a
// multiple of 4): a load fetches two rows.  A row past the matrix lies past the
// descriptor's end by itself.
template <class CF>
struct I8Loader4 {
  static constexpr int A_INSTR = 4 * CF::A_INSTR, LOADS = 4 * CF::LOADS, STAGE_BYTES = CF::STAGE_BYTES;
  static_assert(LOADS * (CF::STAGES - 2) < 64, "the waits of the K loop");
  i32x4 rsA, rsB;
  uint32_t offA, offB, stepA, stepB;  // of the wave's first row, and from load to load
  uint32_t kc;
  uint32_t lds0;
  uint32_t K;

  __device__ __forceinline__ void init(const GemmI8Args& p, int64_t m0, int64_t n0, uint8_t* smem) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    K = (uint32_t)p.K;
    const int64_t ra = p.M - m0 < CF::BM ? p.M - m0 : CF::BM, rb = p.N - n0 < CF::BN ? p.N - n0 : CF::BN;
    rsA = make_rsrc(p.A + m0 * p.lda, (uint32_t)((ra - 1) * p.lda + p.K));
    rsB = make_rsrc(p.B + n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb + p.K));
    const int r = 2 * wave + (lane >> 5);
    kc = (uint32_t)(((lane & 31) >> 2) ^ swz_key(r)) * 16 + 4 * (lane & 3);
    offA = (uint32_t)(r * p.lda);
    offB = (uint32_t)(r * p.ldb);
    stepA = (uint32_t)(2 * CF::NW * p.lda);
    stepB = (uint32_t)(2 * CF::NW * p.ldb);
    lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem)) + (uint32_t)wave * 256;
  }

  template <bool>
  __device__ __forceinline__ void issue(int n, int kb, int stage) const {
    static_assert(CF::NW == 4 || CF::NW == 8, "a load's rows and the next's differ by 8 or 16");
    const bool a = n < A_INSTR;
    const int i = a ? n : n - A_INSTR;
    const uint32_t kbyte = (uint32_t)kb * BK, k = kc ^ (CF::NW == 4 ? 16u * (i & 1) : 0u);
    const uint32_t off = a ? offA + (uint32_t)i * stepA : offB + (uint32_t)i * stepB;
    const uint32_t at = lds0 + (uint32_t)(stage * CF::STAGE_BYTES + (a ? 0 : CF::A_BYTES) + i * CF::NW * 256);
    dma_b32(a ? rsA : rsB, at, kbyte + k < K ? off + k : kOob, kbyte);
  }
  __device__ __forceinline__ void finish(uint8_t*, int) const {}
};

template <class CF>
struct I8RegLoader {
  static constexpr int LOADS = CF::LOADS, STAGE_BYTES = CF::STAGE_BYTES;
  const int8_t* row[CF::LOADS];
  u32x4 v[CF::LOADS];
  uint32_t at[CF::LOADS];
  uint32_t kc;

  __device__ __forceinline__ void init(const GemmI8Args& p, int64_t m0, int64_t n0, uint8_t*) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    kc = (uint32_t)((lane & 7) ^ swz_key(wave * 8 + (lane >> 3))) * 16;
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n) {
      const bool a = n < CF::A_INSTR;
      const int seg = wave + CF::NW * (a ? n : n - CF::A_INSTR);
      int64_t r = (a ? m0 : n0) + seg * 8 + (lane >> 3);
      const int64_t last = (a ? p.M : p.N) - 1;
      r = r < last ? r : last;  // rows past the matrix repeat the last; their results are not stored
      row[n] = a ? p.A + r * p.lda : p.B + r * p.ldb;
      at[n] = (uint32_t)((a ? 0 : CF::A_BYTES) + seg * 1024 + lane * 16);
    }
  }
  __device__ __forceinline__ void load(int kb, int64_t K) {
    const int64_t k = (int64_t)kb * BK + kc;
    if ((int64_t)(kb + 1) * BK <= K) {
#pragma unroll
      for (int n = 0; n < CF::LOADS; ++n) v[n] = load16<false>(row[n], k, K);
    } else {
#pragma unroll
      for (int n = 0; n < CF::LOADS; ++n) v[n] = load16<true>(row[n], k, K);
    }
  }
  __device__ __forceinline__ void store(uint8_t* stage) const {
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n) *reinterpret_cast<u32x4*>(stage + at[n]) = v[n];
  }
};

// A's rows 16-byte aligned and readable up to the next multiple of 16, B's at any
// address: of B the aligned dwords that hold a row's bytes are loaded, so that
// the row lies in LDS behind the 0 to 3 bytes before it in memory, and whoever
// reads a fragment shifts it into place.  A K-block's last fragments then end up
// to 3 bytes into the next K-block: those dwords are fetched once more, into an
// area of one dword per row behind the stage (one load per wave).  Rows step by
// multiples of 4 from load to load, subtile to subtile and tile to tile, so a
// lane's misalignment never changes.
template <class CF>
struct I8LoaderShift {
  static constexpr int A_INSTR = CF::A_INSTR, LOADS = CF::A_INSTR + 4 * CF::B_INSTR + 1;
  static constexpr int STAGE_BYTES = CF::STAGE_BYTES + CF::NW * 256;
  static_assert(LOADS * (CF::STAGES - 2) < 64, "the waits of the K loop");
  static_assert(CF::NW == 4 || CF::NW == 8, "a load's rows of B and the next's differ by 8 or 16");
  static_assert(CF::BN <= 64 * CF::NW, "a lane per row of B");
  i32x4 rsA, rsB;
  uint32_t offA[A_INSTR], kcA, KA;
  uint32_t mis, ld, K;                   // B: its first row's misalignment, the row stride
  uint32_t offB, stepB, endB, kcB;       // the lane's row in the first load, the step; first byte past the row
  uint32_t offT, endT;
  uint32_t lds0;

  __device__ __forceinline__ void init(const GemmI8Args& p, int64_t m0, int64_t n0, uint8_t* smem) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t ra = p.M - m0 < CF::BM ? p.M - m0 : CF::BM, rb = p.N - n0 < CF::BN ? p.N - n0 : CF::BN;
    K = (uint32_t)p.K;
    KA = (K + 15) & ~15u;
    rsA = make_rsrc(p.A + m0 * p.lda, (uint32_t)((ra - 1) * p.lda) + KA);
    kcA = (uint32_t)((lane & 7) ^ swz_key(wave * 8 + (lane >> 3))) * 16;
#pragma unroll
    for (int n = 0; n < A_INSTR; ++n) {
      const int r = (wave + CF::NW * n) * 8 + (lane >> 3);
      offA[n] = r < ra ? (uint32_t)(r * p.lda) + kcA : kOob;
    }
    const int8_t* B = p.B + n0 * p.ldb;
    mis = (uint32_t)(reinterpret_cast<uintptr_t>(B) & 3);
    ld = (uint32_t)p.ldb;
    rsB = make_rsrc(B - mis, (uint32_t)((mis + (rb - 1) * p.ldb + p.K + 3) & ~(int64_t)3));
    const int r = 2 * wave + (lane >> 5);
    kcB = (uint32_t)(((lane & 31) >> 2) ^ swz_key(r)) * 16 + 4 * (lane & 3);
    offB = (mis + r * ld) & ~3u;
    endB = ((mis + r * ld) & 3) + K;
    stepB = 2 * CF::NW * ld;
    const int rt = 64 * wave + lane;
    offT = (mis + rt * ld) & ~3u;
    endT = rt < CF::BN ? ((mis + rt * ld) & 3) + K : 0;
    lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem)) + (uint32_t)wave * 256;
  }

  // B's K-block is part of the lane's offset, which the descriptor checks: a row
  // past the matrix may begin in the last row's last dword.
  template <bool>
  __device__ __forceinline__ void issue(int n, int kb, int stage) const {
    const uint32_t kbyte = (uint32_t)kb * BK, at = lds0 + (uint32_t)(stage * STAGE_BYTES);
    if (n < A_INSTR) {
      const uint32_t wave = threadIdx.x >> 6;
      dma_b128(rsA, at + (uint32_t)__builtin_amdgcn_readfirstlane((int)wave) * 768 + (uint32_t)(n * CF::NW * 1024),
               kbyte + kcA < KA ? offA[n] : kOob, kbyte);
    } else if (n < LOADS - 1) {
      const int i = n - A_INSTR;
      const uint32_t k = kbyte + (kcB ^ (CF::NW == 4 ? 16u * (i & 1) : 0u));
      dma_b32(rsB, at + (uint32_t)(CF::A_BYTES + i * CF::NW * 256), k < endB ? offB + (uint32_t)i * stepB + k : kOob, 0);
    } else {
      const uint32_t k = kbyte + BK;
      dma_b32(rsB, at + CF::STAGE_BYTES, k < endT ? offT + k : kOob, 0);
    }
  }

  // The dword with a row's last bytes may hold some of the next row's: clear
  // them, so that the last K-block's sums are those of the rows alone.
  __device__ __forceinline__ void finish(uint8_t* stage, int kb) const {
    const int r = threadIdx.x;
    const uint32_t end = ((mis + (uint32_t)r * ld) & 3) + K, d = (end >> 2) - 32u * kb;
    if (r < CF::BN && (end & 3)) {
      uint32_t* at = reinterpret_cast<uint32_t*>(d < 32 ? stage + CF::A_BYTES + swz(r, (int)d >> 2) + 4 * (d & 3)
                                                        : stage + CF::STAGE_BYTES + 4 * r);
      *at &= (1u << (8 * (end & 3))) - 1;
    }
    __syncthreads();
  }
};

// Where a lane's operand fragments lie in a stage: row r of a 32-row slice is
// held by lanes r and r + 32, the two 16-byte halves of each 32 bytes of K.
// Computed once per kernel, not once per K-block (+2.8% on 4096x18432x7168).
template <class CF>
struct I8Frag {
  int at, bt;
  int lf[4];

  __device__ __forceinline__ explicit I8Frag(const GemmI8Args&) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int fr = lane & 31, fg = lane >> 5;
    at = wave / CF::WAVES_N * CF::WM * BK;
    bt = CF::A_BYTES + wave % CF::WAVES_N * CF::WN * BK;
#pragma unroll
    for (int h = 0; h < 4; ++h) lf[h] = fr * BK + (((2 * h + fg) ^ swz_key(fr)) << 4);
  }
  // Fragment h of the wave's 32-row slice i of A, or j of B.
  __device__ __forceinline__ v4i a(const uint8_t* stage, int i, int h) const {
    return *reinterpret_cast<const v4i*>(stage + at + i * 32 * BK + lf[h]);
  }
  __device__ __forceinline__ v4i b(const uint8_t* stage, int j, int h) const {
    return *reinterpret_cast<const v4i*>(stage + bt + j * 32 * BK + lf[h]);
  }
};

// The same where B's rows lie behind 0 to 3 bytes: the dword after each fragment,
// which for the last of a K-block lies in the area behind the stage, and the shift.
template <class CF>
struct I8FragShift : I8Frag<CF> {
  int bn[4], next;  // next: from 32-row slice to slice, for the K-block's last fragment
  uint32_t shift;

  __device__ __forceinline__ explicit I8FragShift(const GemmI8Args& p) : I8Frag<CF>(p) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int fr = lane & 31, fg = lane >> 5;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int c = 2 * h + fg + 1;
      bn[h] = c < 8 ? this->bt + fr * BK + ((c ^ swz_key(fr)) << 4)
                    : CF::STAGE_BYTES + 4 * (wave % CF::WAVES_N * CF::WN + fr);
    }
    next = fg ? 32 * 4 : 32 * BK;
    shift = (uint32_t)(reinterpret_cast<uintptr_t>(p.B + fr * p.ldb) & 3);
  }
  __device__ __forceinline__ v4i b(const uint8_t* stage, int j, int h) const {
    const v4i w = I8Frag<CF>::b(stage, j, h);
    const int n = *reinterpret_cast<const int*>(stage + bn[h] + j * (h < 3 ? 32 * BK : next));
    return v4i{(int)__builtin_amdgcn_alignbyte(w[1], w[0], shift), (int)__builtin_amdgcn_alignbyte(w[2], w[1], shift),
               (int)__builtin_amdgcn_alignbyte(w[3], w[2], shift), (int)__builtin_amdgcn_alignbyte(n, w[3], shift)};
  }
};

// The MFMAs of one K-block from its LDS stage; step(s) is called after each of
// the 4 TM groups of them.
template <class CF, class FR, class Step>
__device__ __forceinline__ void i8_block(const uint8_t* stage, const FR& f, v16i (&acc)[CF::TM][CF::TN], Step&& step) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    v4i fb[CF::TN];
#pragma unroll
    for (int j = 0; j < CF::TN; ++j) fb[j] = f.b(stage, j, h);
#pragma unroll
    for (int i = 0; i < CF::TM; ++i) {
      const v4i fa = f.a(stage, i, h);
#pragma unroll
      for (int j = 0; j < CF::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa, acc[i][j], 0, 0, 0);
      step(h * CF::TM + i);
    }
  }
}

// The K loop of one tile; K-blocks 0 .. STAGES - 2 are already on their way.
template <class CF, bool KFULL, class LD, class FR>
__device__ __forceinline__ void i8_k_loop(const LD& ld, const FR& f, int nkb, uint8_t* smem,
                                          v16i (&acc)[CF::TM][CF::TN]) {
  constexpr int PER = (LD::LOADS + 4 * CF::TM - 1) / (4 * CF::TM);
  for (int kb = 0; kb < nkb; ++kb) {
    // Of the stages issued so far, only those behind K-block kb may be missing.
    const int later = nkb - 1 - kb < CF::STAGES - 2 ? nkb - 1 - kb : CF::STAGES - 2;
    if (kb == 0) wait_vmcnt<0>();  // and the scales, and the previous tile's stores
    else if (CF::STAGES >= 4 && later >= 2) wait_vmcnt<LD::LOADS * (CF::STAGES >= 4 ? 2 : 0)>();
    else if (CF::STAGES >= 3 && later >= 1) wait_vmcnt<LD::LOADS * (CF::STAGES >= 3 ? 1 : 0)>();
    else wait_vmcnt<0>();
    __syncthreads();
    uint8_t* stage = smem + (kb % CF::STAGES) * LD::STAGE_BYTES;
    if (kb == nkb - 1) ld.finish(stage, kb);
    const int kn = kb + CF::STAGES - 1;
    i8_block<CF>(stage, f, acc, [&](int s) __attribute__((always_inline)) {
      if (kn >= nkb) return;
#pragma unroll
      for (int n = s * PER; n < (s + 1) * PER && n < LD::LOADS; ++n)
        ld.template issue<KFULL>(n, kn, kn % CF::STAGES);
    });
  }
}

// The scales of a lane's outputs: lane (fr, fg), value 4q + v of subtile (i, j)
// is row 32i + fr, column 32j + 8q + 4fg + v.
template <class CF>
struct I8Scales {
  float as[CF::TM], bs[CF::TN][16];

  __device__ __forceinline__ void load(const GemmI8Args& p, int64_t m0, int64_t n0) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t row = m0 + wave / CF::WAVES_N * CF::WM + (lane & 31);
    const int64_t col = n0 + wave % CF::WAVES_N * CF::WN + 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < CF::TM; ++i) as[i] = p.a_s[row + 32 * i < p.M ? row + 32 * i : p.M - 1];
#pragma unroll
    for (int j = 0; j < CF::TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int64_t c = col + 32 * j + 8 * (q >> 2) + (q & 3);
        bs[j][q] = p.b_s[c < p.N ? c : p.N - 1];
      }
  }
};

// Scale and round to bf16, and store 32 rows at a time through an LDS area of
// the wave's own (chunks of 16 bytes XOR-ed with the row), so that rows leave
// as 16-byte writes, at any address (as 2-byte writes where ldc or C is not
// 16-byte aligned, 4096x7169x2051 took 141 us against 105).
template <class CF>
__device__ __forceinline__ void i8_store(const GemmI8Args& p, int64_t m0, int64_t n0, const I8Scales<CF>& sc,
                                         const v16i (&acc)[CF::TM][CF::TN], uint8_t* area) {
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 31, fg = lane >> 5;
  const int64_t row0 = m0 + wave / CF::WAVES_N * CF::WM, col0 = n0 + wave % CF::WAVES_N * CF::WN;
  uint8_t* st = area + wave * CF::C_BYTES;
  constexpr int CPR = CF::WN / 8, IT = 32 * CPR / 64, MASK = CPR < 8 ? CPR - 1 : 7;
#pragma unroll
  for (int i = 0; i < CF::TM; ++i) {
#pragma unroll
    for (int j = 0; j < CF::TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float y[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = (float)acc[i][j][4 * q + v] * (sc.as[i] * sc.bs[j][4 * q + v]);
        *reinterpret_cast<uint2*>(st + fr * CF::WN * 2 + (((4 * j + q) ^ (fr & MASK)) << 4) + 8 * fg) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
    __builtin_amdgcn_wave_barrier();
    u32x4 v[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int r = (lane + 64 * it) / CPR, c = (lane + 64 * it) % CPR;
      v[it] = *reinterpret_cast<const u32x4*>(st + r * CF::WN * 2 + ((c ^ (r & MASK)) << 4));
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int64_t row = row0 + 32 * i + (lane + 64 * it) / CPR, col = col0 + (lane + 64 * it) % CPR * 8;
      if (row >= p.M || col >= p.N) continue;
      uint16_t* dst = p.C + row * p.ldc + col;
      if (col + 8 <= p.N) {
        *reinterpret_cast<u32x4u*>(dst) = v[it];
      } else {
        const uint32_t w[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
        for (int e = 0; e < 8 && col + e < p.N; ++e) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

template <class CF>
__device__ __forceinline__ void i8_zero(v16i (&acc)[CF::TM][CF::TN]) {
#pragma unroll
  for (int i = 0; i < CF::TM; ++i)
#pragma unroll
    for (int j = 0; j < CF::TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
}

// The operands: 16-byte aligned (K a multiple of 128, or of 16), 4-byte aligned
// (K a multiple of 4), A 16-byte aligned and padded, any (through registers).
enum Feed { kDmaFull, kDma, kDma4, kShift, kRegs };

template <class CF, Feed FEED>
using I8Feed = typename std::conditional<
    FEED == kRegs, I8RegLoader<CF>,
    typename std::conditional<FEED == kShift, I8LoaderShift<CF>,
                              typename std::conditional<FEED == kDma4, I8Loader4<CF>, I8Loader<CF>>::type>::type>::type;

// One workgroup per tile, or (with direct-to-LDS loads and room in LDS beside
// the ring for the output's staging) one per CU that walks its XCD's tiles:
// the next tile's first K-block is then on its way while the current tile is
// scaled and stored.  The scales are loaded before the K loop, whose waits
// cover them, so that the store waits for none of the next tile's loads.
template <class CF, Feed FEED>
__global__ __launch_bounds__(CF::kThreads) void gemm_i8_kernel(GemmI8Args p) {
  constexpr int RING = CF::STAGES * I8Feed<CF, FEED>::STAGE_BYTES;
  constexpr bool AHEAD = FEED != kRegs && RING + CF::NW * CF::C_BYTES <= 160 * 1024;
  constexpr int OUT = AHEAD ? RING : 0;
  constexpr int LDS = OUT + CF::NW * CF::C_BYTES > RING ? OUT + CF::NW * CF::C_BYTES : RING;
  __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
  const int64_t tiles_m = (p.M + CF::BM - 1) / CF::BM, tiles_n = (p.N + CF::BN - 1) / CF::BN;
  const int64_t total = tiles_m * tiles_n;
  const int nkb = (int)((p.K + BK - 1) / BK);
  const typename std::conditional<FEED == kShift, I8FragShift<CF>, I8Frag<CF>>::type f(p);
  int64_t tm, tn, pid = blockIdx.x;
  tile_of(pid, tiles_m, tiles_n, tm, tn);
  I8Feed<CF, FEED> ld;
  auto begin = [&]() __attribute__((always_inline)) {
    ld.init(p, tm * CF::BM, tn * CF::BN, smem);
    if constexpr (FEED != kRegs) {
      for (int s = 0; s < CF::STAGES - 1 && s < nkb; ++s)
#pragma unroll
        for (int n = 0; n < decltype(ld)::LOADS; ++n) ld.template issue<FEED == kDmaFull>(n, s, s);
    }
  };
  begin();
  for (;;) {
    v16i acc[CF::TM][CF::TN];
    i8_zero<CF>(acc);
    I8Scales<CF> sc;
    if constexpr (FEED == kRegs) {
      ld.load(0, p.K);
      ld.store(smem);
      for (int kb = 0; kb < nkb; ++kb) {
        __syncthreads();
        if (kb + 1 < nkb) ld.load(kb + 1, p.K);
        i8_block<CF>(smem + (kb & 1) * CF::STAGE_BYTES, f, acc, [](int) {});
        if (kb + 1 < nkb) ld.store(smem + ((kb + 1) & 1) * CF::STAGE_BYTES);
      }
      sc.load(p, tm * CF::BM, tn * CF::BN);
    } else {
      sc.load(p, tm * CF::BM, tn * CF::BN);
      i8_k_loop<CF, FEED == kDmaFull>(ld, f, nkb, smem, acc);
    }
    __syncthreads();
    const int64_t m0 = tm * CF::BM, n0 = tn * CF::BN;
    pid += gridDim.x;
    const bool more = pid < total;
    if (more) tile_of(pid, tiles_m, tiles_n, tm, tn);
    if (AHEAD && more) begin();
    i8_store<CF>(p, m0, n0, sc, acc, smem + OUT);
    if (!more) break;
    if constexpr (!AHEAD) {
      __syncthreads();
      begin();
    }
  }
}

// ---- few output tiles: K split over the waves of a workgroup ---------------------------
//
// A workgroup owns a 16 FM x 16 FN tile; its W waves take the K-blocks in turn
// (wave w: w, w + W, ...), each through a ring of D LDS slots of its own that
// hold one K-block of the tile's rows, so no wave waits for another until the
// sums are added up at the end, by integer additions in LDS, whose order does
// not matter.  All of a wave's first D K-blocks are in flight at once.
// Bound by trips to memory one after the other, as many as a wave's share of the
// K-blocks has of D, and by what one CU loads: the product 32x1536x7168 takes 5.1-5.3
// us (16x16 tiles, 192 workgroups, 7 K-blocks in 2 slots), 64x7168x2048 6.2-7.0 us (2
// in 1), 333x2500x1000 8.1 us, and the fused layer 1x1536x7168 6.3-6.5 us for 11 MB (7
// in 3, of which the first 3 are on their way beside the quantisation).
//
// FUSED: the activations come as the quantiser's input and every workgroup
// quantises all M <= 16 rows of it itself, while its first weights are on
// their way; the codes stay in LDS (rows of code_ld bytes after the ring).
// HALF (FN = 1): 8 columns per workgroup, so that a narrow product reaches
// more CUs.

constexpr int kSplitWaves = 8;
constexpr int kFusedCodes = 16384;  // room for the codes (M * K) of a fused launch

template <int FM, int FN, int D, bool FUSED, bool HALF>
struct SplitCfg {
  static constexpr int TM = 16 * FM, TN = HALF ? 8 : 16 * FN;
  static constexpr int AROWS = FUSED ? 0 : TM;
  static constexpr int SLOT = (AROWS + TN) * BK;
  static constexpr int RING = kSplitWaves * D * SLOT;
  static constexpr int SUM = TM * 16 * FN * 4;
  static constexpr int LDS = RING > SUM ? RING : SUM;
  static constexpr int CODES = FUSED ? kFusedCodes + 16 * (BK - 1 + 16) : 0;  // rows padded to whole K-blocks, and 16 bytes
};

template <class SRC_TAG, int FM, int FN, int D, bool HALF, int W>
__global__ __launch_bounds__(64 * kSplitWaves) void gemm_i8_split_kernel(GemmI8Args p, RowQuantArgs x, int code_ld) {
  constexpr bool FUSED = !std::is_void<SRC_TAG>::value;
  constexpr bool DMA = W > 0;
  static_assert(D <= 3 && (DMA || D == 1), "waits of the ring; one K-block in registers");
  using CF = SplitCfg<FM, FN, D, FUSED, HALF>;
  constexpr int BYTES = W == 4 ? 256 : 1024, LOADS = CF::SLOT / BYTES;  // of a load: 8 rows, or 2
  static_assert(LOADS * (D - 1) < 64, "waits of the ring");
  __shared__ __attribute__((aligned(16))) uint8_t smem[CF::LDS + CF::CODES];
  __shared__ uint32_t row_top[16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 15, fg = lane >> 4;
  const uint32_t tiles_n = (uint32_t)((p.N + CF::TN - 1) / CF::TN);
  const int64_t m0 = FUSED ? 0 : (int64_t)(blockIdx.x / tiles_n) * CF::TM;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * CF::TN;
  const int nkb = (int)((p.K + BK - 1) / BK);
  const uint32_t K = (uint32_t)p.K;
  const int64_t ra = p.M - m0 < CF::TM ? p.M - m0 : CF::TM, rb = p.N - n0 < CF::TN ? p.N - n0 : CF::TN;
  // Load n fetches rows 8n .. 8n + 7 of the slot (A's rows, then B's; W = 4:
  // rows 2n, 2n + 1); a lane's chunk depends on the row modulo 16 alone.
  const uint32_t kc[2] = {(uint32_t)((lane & 7) ^ swz_key(lane >> 3)) * 16,
                          (uint32_t)((lane & 7) ^ swz_key(8 + (lane >> 3))) * 16};
  i32x4 rsA, rsB;
  uint32_t off[W == 16 ? LOADS : 1];
  const int8_t* row[DMA ? 1 : LOADS];
  u32x4 reg[DMA ? 1 : LOADS];
  if constexpr (DMA) {
    rsA = make_rsrc(p.A + (FUSED ? 0 : m0 * p.lda), FUSED ? 0u : (uint32_t)((ra - 1) * p.lda + p.K));
    rsB = make_rsrc(p.B + n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb + p.K));
  }
  const uint32_t k4 = (uint32_t)(((lane & 31) >> 2) ^ (lane >> 5)) * 16 + 4 * (lane & 3);
  const uint32_t off4[2] = {(uint32_t)((lane >> 5) * p.lda), (uint32_t)((lane >> 5) * p.ldb)};
#pragma unroll
  for (int n = 0; n < LOADS && W != 4; ++n) {
    const bool a = 8 * n < CF::AROWS;
    const int r = 8 * n - (a ? 0 : CF::AROWS) + (lane >> 3);
    if constexpr (DMA) {
      off[n] = r < (a ? ra : rb) ? (uint32_t)(r * (a ? p.lda : p.ldb)) + kc[n & 1] : kOob;
    } else {
      const int64_t g = r < (a ? ra : rb) ? r : (a ? ra : rb) - 1;
      row[n] = a ? p.A + (m0 + g) * p.lda : p.B + (n0 + g) * p.ldb;
    }
  }
  const uint32_t lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem)) + (uint32_t)(wave * D * CF::SLOT);
  auto issue = [&](int kb, int slot) __attribute__((always_inline)) {
    if constexpr (W == 4) {
      const uint32_t kbyte = (uint32_t)kb * BK;
#pragma unroll
      for (int n = 0; n < LOADS; ++n) {
        const bool a = 2 * n < CF::AROWS;
        const int r = 2 * n - (a ? 0 : CF::AROWS);  // even; the key of r + 1 is that of r, its lowest bit flipped
        const uint32_t k = k4 ^ (uint32_t)(16 * swz_key(r)), o = off4[a ? 0 : 1] + (uint32_t)(r * (a ? p.lda : p.ldb)) + k;
        dma_b32(a ? rsA : rsB, lds0 + (uint32_t)(slot * CF::SLOT + n * 256), kbyte + k < K ? o : kOob, kbyte);
      }
    } else if constexpr (DMA) {
      const uint32_t kbyte = (uint32_t)kb * BK;
#pragma unroll
      for (int n = 0; n < LOADS; ++n)
        dma_b128(8 * n < CF::AROWS ? rsA : rsB, lds0 + (uint32_t)(slot * CF::SLOT + n * 1024),
                 kbyte + kc[n & 1] < K ? off[n] : kOob, kbyte);
    } else {
      const int64_t k = (int64_t)kb * BK;
      if (k + BK <= p.K) {
#pragma unroll
        for (int n = 0; n < LOADS; ++n) reg[n] = load16<false>(row[n], k + kc[n & 1], p.K);
      } else {
#pragma unroll
        for (int n = 0; n < LOADS; ++n) reg[n] = load16<true>(row[n], k + kc[n & 1], p.K);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wave + d * kSplitWaves < nkb) issue(wave + d * kSplitWaves, d);

  uint8_t* codes = smem + CF::LDS;
  if constexpr (FUSED) {
    // Units of 64 chunks of one row, dealt to the waves in turn; held in
    // registers between the row's maximum and its codes.
    constexpr Src SRC = SRC_TAG::value;
    constexpr Src kHeld = SRC == kGated ? kF32 : SRC;
    const int nch = (int)((x.K + 7) >> 3), segs = (nch + 63) >> 6, units = (int)p.M * segs;
    if (threadIdx.x < 16) row_top[threadIdx.x] = __float_as_uint(kAmaxFloor);
    __syncthreads();
    constexpr int HOLD = 4;
    Chunk<kHeld> held[HOLD];
    auto place = [&](int u, int& m, int& c) { m = u / segs, c = (u - m * segs) * 64 + lane; };
    auto at = [&](int c) { return c < nch - 1 ? 8 * c : (int)x.K - 8; };
    auto fetch = [&](int u0) __attribute__((always_inline)) {
      Chunk<SRC> in[HOLD];
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        int m, c;
        place(u0 + i * kSplitWaves, m, c);
        in[i].load(x, m, at(c), u0 + i * kSplitWaves < units && c < nch);
      }
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        if constexpr (SRC == kGated) {
          float v[8];
          in[i].values(v);
          held[i].set(v);
        } else {
          held[i] = in[i];
        }
      }
    };
    const bool once = units <= HOLD * kSplitWaves;
    for (int u0 = wave; u0 < units; u0 += HOLD * kSplitWaves) {
      fetch(u0);
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        const int u = u0 + i * kSplitWaves;
        if (u >= units) continue;
        float v[8];
        held[i].values(v);
        const uint32_t top = max_u32_wave(max_abs(v, 0u));
        if (lane == 0) atomicMax(&row_top[u / segs], top);
      }
    }
    // Zero the codes between the row's end and its last K-block's: their
    // weights read as zero, but the codes must be defined.
    const int pad = nkb * BK - (int)x.K;
    for (int i = threadIdx.x; i < (int)p.M * pad; i += 64 * kSplitWaves)
      codes[(i / pad) * code_ld + x.K + i % pad] = 0;
    __syncthreads();
    for (int u0 = wave; u0 < units; u0 += HOLD * kSplitWaves) {
      if (!once) fetch(u0);
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        const int u = u0 + i * kSplitWaves;
        if (u >= units) continue;
        int m, c;
        place(u, m, c);
        float v[8];
        held[i].values(v);
        if (c < nch)
          *reinterpret_cast<u32x2u*>(codes + m * code_ld + at(c)) = codes8(v, 127.0f / __uint_as_float(row_top[m]));
      }
    }
    __syncthreads();
  }

  v4i acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  const uint8_t* ring = smem + wave * D * CF::SLOT;
  for (int kb = wave, slot = 0; kb < nkb; kb += kSplitWaves) {
    // loads of the later K-blocks in flight behind this one's
    if constexpr (DMA) {
      const int left = (nkb - 1 - kb) / kSplitWaves;
      if (D >= 3 && left >= 2) wait_vmcnt<LOADS * (D >= 3 ? 2 : 0)>();
      else if (D >= 2 && left >= 1) wait_vmcnt<LOADS * (D >= 2 ? 1 : 0)>();
      else wait_vmcnt<0>();
      asm volatile("" ::: "memory");
    } else {
#pragma unroll
      for (int n = 0; n < LOADS; ++n)
        *reinterpret_cast<u32x4*>(smem + wave * D * CF::SLOT + n * 1024 + lane * 16) = reg[n];
      __builtin_amdgcn_wave_barrier();
    }
    const uint8_t* at = ring + slot * CF::SLOT;
    const uint8_t* bt = at + CF::AROWS * BK;
    v4i fa[FM][2], fb[FN][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[j][h] = *reinterpret_cast<const v4i*>(bt + swz(HALF ? fr & 7 : 16 * j + fr, 4 * h + fg));
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (FUSED) {
          const int r = fr < (int)p.M ? fr : 0;
          fa[i][h] = *reinterpret_cast<const v4i*>(codes + r * code_ld + kb * BK + 64 * h + 16 * fg);
        } else {
          fa[i][h] = *reinterpret_cast<const v4i*>(at + swz(16 * i + fr, 4 * h + fg));
        }
      }
    }
    // the slot is free once its fragments have arrived
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (kb + D * kSplitWaves < nkb) issue(kb + D * kSplitWaves, slot);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j][h], fa[i][h], acc[i][j], 0, 0, 0);
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  __syncthreads();
  // sum[subtile][v][lane] over the waves
  int* sum = reinterpret_cast<int*>(smem);
  for (int i = threadIdx.x; i < FM * FN * 256; i += 64 * kSplitWaves) sum[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) atomicAdd(&sum[((i * FN + j) * 4 + v) * 64 + lane], acc[i][j][v]);
  __syncthreads();
  constexpr int CPR = CF::TN / 4;  // runs of four columns per row
  for (int q = threadIdx.x; q < CF::TM * CPR; q += 64 * kSplitWaves) {
    const int r = q / CPR, c4 = q % CPR;
    const int64_t row = m0 + r, col = n0 + 4 * c4;
    if (row >= p.M || col >= p.N) continue;
    const int* src = sum + (((r >> 4) * FN + (c4 >> 2)) * 4) * 64 + (c4 & 3) * 16 + (r & 15);
    const float as = FUSED ? __uint_as_float(row_top[r & 15]) / 127.0f : p.a_s[row];
    uint32_t w[2];
    float y[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) y[v] = (float)src[64 * v] * (as * p.b_s[col + v < p.N ? col + v : p.N - 1]);
    w[0] = pack_bf16x2(y[0], y[1]);
    w[1] = pack_bf16x2(y[2], y[3]);
    uint16_t* dst = p.C + row * p.ldc + col;
    if (col + 4 <= p.N) {
      *reinterpret_cast<u32x2u*>(dst) = u32x2u{w[0], w[1]};
    } else {
      for (int v = 0; v < 4 && col + v < p.N; ++v) dst[v] = (uint16_t)(w[v >> 1] >> (16 * (v & 1)));
    }
  }
}

// ---- K < 16 ----------------------------------------------------------------------------

// A row is shorter than one load: one output per thread, byte by byte.  Bound by
// the launch for what such K is used for.
__global__ __launch_bounds__(256) void gemm_i8_short_kernel(GemmI8Args p) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M * p.N; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / p.N, n = i - m * p.N;
    int sum = 0;
    for (int k = 0; k < p.K; ++k) sum += (int)p.A[m * p.lda + k] * (int)p.B[n * p.ldb + k];
    p.C[m * p.ldc + n] = (uint16_t)pack_bf16x2((float)sum * (p.a_s[m] * p.b_s[n]), 0.0f);
  }
}

}  // namespace

namespace {

template <class Kernel>
hipError_t launch_rows(Kernel kernel, int rows_per_block, const RowQuantArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.M + rows_per_block - 1) / rows_per_block;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < (1 << 22) ? blocks : (1 << 22))), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <Src SRC>
hipError_t launch_quant(const RowQuantArgs& a, hipStream_t stream) {
  if (a.K <= 512) return launch_rows(row_quant_kernel<SRC, 64, 1>, 4, a, stream);
  if (a.K <= 1024) return launch_rows(row_quant_kernel<SRC, 64, 2>, 4, a, stream);
  if (a.K <= 2048) return launch_rows(row_quant_kernel<SRC, 256, 1>, 1, a, stream);
  if (a.K <= 4096) return launch_rows(row_quant_kernel<SRC, 256, 2>, 1, a, stream);
  if (a.K <= 8192) return launch_rows(row_quant_kernel<SRC, 256, 4>, 1, a, stream);
  if (a.K <= 20480) return launch_rows(row_quant_kernel<SRC, 256, 10>, 1, a, stream);
  return launch_rows(row_quant_kernel<SRC, 256, 0>, 1, a, stream);
}

}  // namespace

hipError_t launch_row_quant_i8(const RowQuantArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  if (a.K < 8) return launch_rows(row_quant_short_kernel, 256, a, stream);
  if (a.f32) return launch_quant<kF32>(a, stream);
  return a.u != nullptr ? launch_quant<kGated>(a, stream) : launch_quant<kBf16>(a, stream);
}

namespace {

using Plain = std::integral_constant<Src, kBf16>;
using Gated = std::integral_constant<Src, kGated>;
constexpr int64_t kMaxGrid = (int64_t)1 << 22;  // workgroups of a launch whose workgroups loop

inline bool aligned16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 16 == 0; }

// A weight (or activation) for the direct-to-LDS loads: 16-byte chunks, and a
// tile's rows within 31-bit offsets.
inline bool dma_ok(const void* p, int64_t ld, int64_t K) { return K % 16 == 0 && aligned16(p, ld) && ld < (1 << 23); }

// For the same loads of 4 bytes.
inline bool dma4_ok(const void* p, int64_t ld, int64_t K) {
  return K % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 3) == 0 && ld % 4 == 0 && ld < (1 << 23);
}

// For loads of B's aligned dwords.
inline bool shifted(const GemmI8Args& a) { return a.a_padded && a.ldb < (1 << 23); }

// Bytes per lane of the operands' direct-to-LDS loads; 0: neither holds.
inline int feed_bytes(const GemmI8Args& a, bool with_a) {
  if ((!with_a || dma_ok(a.A, a.lda, a.K)) && dma_ok(a.B, a.ldb, a.K)) return 16;
  return (!with_a || dma4_ok(a.A, a.lda, a.K)) && dma4_ok(a.B, a.ldb, a.K) ? 4 : 0;
}

template <class CF>
hipError_t launch_tiles(const GemmI8Args& a, int w, hipStream_t stream) {
  const int64_t t = ((a.M + CF::BM - 1) / CF::BM) * ((a.N + CF::BN - 1) / CF::BN);
  // the large tile: one workgroup per CU, a multiple of the XCDs
  const int64_t most = CF::BM * CF::BN == 65536 ? (device_cu_count() + kXcds - 1) / kXcds * kXcds : kMaxGrid;
  const dim3 grid((unsigned)(t < most ? t : most)), blk(CF::kThreads);
  if (w == 0 && shifted(a)) hipLaunchKernelGGL((gemm_i8_kernel<CF, kShift>), grid, blk, 0, stream, a);
  else if (w == 0) hipLaunchKernelGGL((gemm_i8_kernel<CF, kRegs>), grid, blk, 0, stream, a);
  else if (w == 4) hipLaunchKernelGGL((gemm_i8_kernel<CF, kDma4>), grid, blk, 0, stream, a);
  else if (a.K % BK == 0) hipLaunchKernelGGL((gemm_i8_kernel<CF, kDmaFull>), grid, blk, 0, stream, a);
  else hipLaunchKernelGGL((gemm_i8_kernel<CF, kDma>), grid, blk, 0, stream, a);
  return hipGetLastError();
}

template <class SRC_TAG, int FM, int FN, int D, bool HALF, int W = 16>
hipError_t launch_split_dma(const GemmI8Args& a, const RowQuantArgs& x, int code_ld, hipStream_t stream) {
  using CF = SplitCfg<FM, FN, D, !std::is_void<SRC_TAG>::value, HALF>;
  const int64_t t = (a.M + CF::TM - 1) / CF::TM * ((a.N + CF::TN - 1) / CF::TN);
  hipLaunchKernelGGL((gemm_i8_split_kernel<SRC_TAG, FM, FN, D, HALF, W>), dim3((unsigned)t), dim3(64 * kSplitWaves),
                     0, stream, a, x, code_ld);
  return hipGetLastError();
}

template <class SRC_TAG, int FM, int FN, int D, bool HALF>
hipError_t launch_split(const GemmI8Args& a, const RowQuantArgs& x, int w, hipStream_t stream) {
  // fused: rows of codes 16 bytes apart modulo the LDS's 128-byte bank row
  const int code_ld = std::is_void<SRC_TAG>::value ? 0 : (int)((a.K + BK - 1) / BK * BK + 16);
  if (w == 16) return launch_split_dma<SRC_TAG, FM, FN, D, HALF, 16>(a, x, code_ld, stream);
  if (w == 4) return launch_split_dma<SRC_TAG, FM, FN, D, HALF, 4>(a, x, code_ld, stream);
  return launch_split_dma<SRC_TAG, FM, FN, 1, HALF, 0>(a, x, code_ld, stream);
}

// The variants and what each costs: a CU runs up to `resident` workgroups at
// once, so it works through its share of the tiles in rounds; a round costs
// 1 us, a K-block of a tile per_kb (an eighth of the K-blocks for the split
// variants, whose eight waves share them), the launch and the store `fixed`;
// for direct-to-LDS operands in loads of 16 and of 4 bytes, with B's aligned
// dwords, and through registers (the split variants load the third kind through
// registers too).  The constants are fitted to 250 products (1 to 4096 rows, ten
// weights from 512x512 to 18432x7168), 118 with rows aligned to 4 bytes alone and
// twice 110 with odd sizes, each timed with every variant: the choice takes 2.9%
// (1.1%, 2.4%, 2.2%) longer than the fastest variant in the geometric mean; the
// best single variant would take 60% (29%, 70%, 67%) longer.  resident = 0: not
// for such operands (the 64x64 split variant spills with its loads in registers;
// with loads of 4 bytes the 64x32 one, at 2.14 and 1.658, was never the cheapest).
struct Cost {
  int resident;
  float fixed, per_kb;
};
struct Variant {
  int bm, bn;
  bool split;
  Cost dma, dma4, shift, regs;
};
constexpr Variant kVariants[] = {{16, 8, true, {2, 1.30f, 0.327f}, {2, 1.99f, 0.280f},
                                  {2, 2.27f, 0.305f}, {2, 2.22f, 0.412f}},
                                 {16, 16, true, {2, 1.38f, 0.470f}, {2, 1.80f, 0.433f},
                                  {2, 2.46f, 0.488f}, {2, 2.46f, 0.588f}},
                                 {32, 32, true, {2, 1.52f, 0.966f}, {2, 2.19f, 0.761f},
                                  {1, 3.56f, 1.150f}, {1, 3.48f, 1.416f}},
                                 {64, 32, true, {1, 1.69f, 1.465f}, {0, 0.0f, 0.0f},
                                  {1, 4.65f, 1.668f}, {1, 4.57f, 2.171f}},
                                 {64, 64, true, {1, 2.60f, 2.164f}, {1, 3.35f, 2.380f},
                                  {0, 0.0f, 0.0f}, {0, 0.0f, 0.0f}},
                                 {64, 64, false, {2, 2.62f, 0.271f}, {2, 3.31f, 0.435f},
                                  {2, 3.98f, 0.471f}, {2, 4.01f, 0.556f}},
                                 {128, 128, false, {1, 2.49f, 0.607f}, {1, 3.14f, 0.953f},
                                  {1, 2.96f, 0.998f}, {1, 2.31f, 1.388f}},
                                 {128, 256, false, {1, 3.54f, 0.897f}, {1, 4.54f, 1.432f},
                                  {1, 4.13f, 1.595f}, {1, 3.77f, 1.912f}},
                                 {256, 256, false, {1, 4.72f, 1.556f}, {1, 6.71f, 2.282f},
                                  {1, 5.64f, 2.178f}, {1, 6.72f, 2.484f}}};

float variant_us(const Variant& v, const GemmI8Args& a, int w, int cus) {
  const Cost& c = w == 16 ? v.dma : w == 4 ? v.dma4 : shifted(a) ? v.shift : v.regs;
  const int64_t tiles = (a.M + v.bm - 1) / v.bm * ((a.N + v.bn - 1) / v.bn);
  // a split launch has one workgroup per tile
  if (c.resident == 0 || (v.split && tiles > kMaxGrid)) return 1e30f;
  const int64_t full = tiles / ((int64_t)cus * c.resident), rest = tiles - full * cus * c.resident;
  const int64_t per_cu = full * c.resident + (rest + cus - 1) / cus;
  int64_t kbs = (a.K + BK - 1) / BK;
  if (v.split) kbs = (kbs + kSplitWaves - 1) / kSplitWaves;
  return c.fixed + (float)(full + (rest > 0)) + c.per_kb * (float)kbs * (float)per_cu;
}

}  // namespace

// The int8 linear layer in one launch: few rows, whose quantisation every
// workgroup repeats.
// By measurement the quantisation's own launch costs 2 us, and quantising M K
// elements in every workgroup as much where M K, doubled for the gated input and
// times the rounds of workgroups, is about 16384 (1x1536x7168 6.6 against 8.7 us,
// 4x7168x2048 8.0 against 8.7, but 8x7168x2048 9.4 against 8.8 and 2x18432x7168
// 30.8 against 29.4; gated 2x7168x2048 8.8 against 8.3 for twice its rows in two
// launches, which from Python take 4 us more).
// The rounds are those of 256 CUs, on any device: the workspace's size follows
// from the same rule, and that has to be a function of the sizes alone.
bool linear_i8_fused(int64_t M, int64_t N, int64_t K, bool gated) {
  if (M < 1 || M > 16 || K < 16 || M * K > kFusedCodes) return false;  // what the kernel has room for
  const int64_t rounds = ((N + 15) / 16 + 255) / 256;
  return M * K * (gated ? 2 : 1) * (rounds < 1 ? 1 : rounds) <= 16384;
}

hipError_t launch_linear_i8_fused(const GemmI8Args& g, const RowQuantArgs& q, hipStream_t stream) {
  const I8Variant v = linear_i8_fused_variant(g);
  const bool half = v.columns == 8;
  const int w = v.feed;
  if (q.u != nullptr)
    return half ? launch_split<Gated, 1, 1, 3, true>(g, q, w, stream)
                : launch_split<Gated, 1, 1, 3, false>(g, q, w, stream);
  return half ? launch_split<Plain, 1, 1, 3, true>(g, q, w, stream)
              : launch_split<Plain, 1, 1, 3, false>(g, q, w, stream);
}

namespace {

// The cheapest variant for operands that are loaded w bytes at a time.
int choose(const GemmI8Args& a, int w) {
  const int cus = device_cu_count();
  int best = 0;
  for (int i = 1; i < (int)(sizeof(kVariants) / sizeof(kVariants[0])); ++i)
    if (variant_us(kVariants[i], a, w, cus) < variant_us(kVariants[best], a, w, cus)) best = i;
  return best;
}

}  // namespace

I8Variant gemm_i8_variant(const GemmI8Args& a) {
  if (a.K < 16) return {DSFP8_I8_SHORT, 0, 0, 0};
  const int w = feed_bytes(a, true);
  const Variant& v = kVariants[choose(a, w)];
  return {v.split ? DSFP8_I8_SPLIT : DSFP8_I8_TILES, v.bm, v.bn, w == 0 && !v.split && shifted(a) ? 1 : w};
}

I8Variant linear_i8_fused_variant(const GemmI8Args& a) {
  return {DSFP8_I8_FUSED, 16, (a.N + 15) / 16 < device_cu_count() ? 8 : 16, feed_bytes(a, false)};
}

hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  if (a.K < 16) {
    const int64_t blocks = (a.M * a.N + 255) / 256;
    hipLaunchKernelGGL(gemm_i8_short_kernel, dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid)), dim3(256), 0,
                       stream, a);
    return hipGetLastError();
  }
  const int w = feed_bytes(a, true);
  const RowQuantArgs none{};
  switch (choose(a, w)) {
    case 0: return launch_split<void, 1, 1, 2, true>(a, none, w, stream);
    case 1: return launch_split<void, 1, 1, 2, false>(a, none, w, stream);
    case 2: return launch_split<void, 2, 2, 1, false>(a, none, w, stream);
    case 3:
      return w == 16 ? launch_split_dma<void, 4, 2, 1, false>(a, none, 0, stream)
                     : launch_split_dma<void, 4, 2, 1, false, 0>(a, none, 0, stream);
    case 4:
      return w == 4 ? launch_split_dma<void, 4, 4, 1, false, 4>(a, none, 0, stream)
                    : launch_split_dma<void, 4, 4, 1, false>(a, none, 0, stream);
    case 5: return launch_tiles<I8Cfg<64, 64, 2, 2, 4>>(a, w, stream);
    case 6: return launch_tiles<I8Cfg<128, 128, 2, 4, 3>>(a, w, stream);
    case 7: return launch_tiles<I8Cfg<128, 256, 2, 4, 3>>(a, w, stream);
    default: return launch_tiles<I8Cfg<256, 256, 2, 4, 2>>(a, w, stream);
  }
}

}  // namespace dsfp8
