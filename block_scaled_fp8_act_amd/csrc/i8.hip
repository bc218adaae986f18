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

// SiLU(g) * u in fp32.
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

// Rows of fewer than 8 elements: one thread each.
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

// 16 bytes of a row of K bytes from column k; bytes past the row, or of a row
// outside the matrix, are zero.
__device__ __forceinline__ u32x4 load16(const int8_t* row, int64_t k, int64_t K, bool ok) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (!ok || k >= K) return v;
  if (k + 16 <= K) return *reinterpret_cast<const u32x4u*>(row + k);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < K) w[i >> 2] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
  return u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ int chunk_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// ---- 16-byte aligned operands: tiles fed by direct-to-LDS loads ----------------------
//
// BM x BN tiles, each wave WM x WN of it, as in the block-scaled products: a
// ring of STAGES K-blocks of 128 bytes per row, filled by buffer_load ... lds
// (rows past the matrix and chunks past K read as zero through the
// descriptor), one barrier per K-block, the loads of a later K-block issued
// between the MFMAs of the current one.  Nothing is rescaled inside the K
// loop, so the accumulators stay where the matrix instruction leaves them.
// The weight fragment is the instruction's first operand, so a lane's results
// are runs of four columns of one row.

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
  static constexpr int CS = WN + 8;  // staged C row, in bf16 elements
  static constexpr int C_BYTES = NW * WM * CS * 2;
  static constexpr int LDS_BYTES = STAGES * STAGE_BYTES > C_BYTES ? STAGES * STAGE_BYTES : C_BYTES;
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole 1 KB segments per wave");
  static_assert(WM % 32 == 0 && WN % 32 == 0, "32x32 subtiles");
  static_assert(LOADS * (STAGES - 2) < 64 && LOADS <= 10, "vmcnt range, packed chunk indices");
};

template <class CF>
struct I8Loader {
  i32x4 rsA, rsB;
  uint32_t off[CF::LOADS];
  uint32_t kc;  // logical chunk (0..7) of load n at bits 3n
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
    kc = 0;
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n) {
      const bool a = n < CF::A_INSTR;
      const int r = (wave + CF::NW * (a ? n : n - CF::A_INSTR)) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ swz_key(r);
      off[n] = r < (a ? ra : rb) ? (uint32_t)(r * (a ? p.lda : p.ldb) + c * 16) : kOob;
      kc |= (uint32_t)c << (3 * n);
    }
    lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem));
  }

  template <bool KFULL>
  __device__ __forceinline__ void issue(int n, int kb, int stage) const {
    const bool a = n < CF::A_INSTR;
    const uint32_t kbyte = (uint32_t)kb * BK;
    const bool in = KFULL || kbyte + ((kc >> (3 * n)) & 7u) * 16u < K;
    const uint32_t at = lds0 + (uint32_t)(stage * CF::STAGE_BYTES + (a ? 0 : CF::A_BYTES) +
                                          (wave + CF::NW * (a ? n : n - CF::A_INSTR)) * 1024);
    dma_b128(a ? rsA : rsB, at, in ? off[n] : kOob, kbyte);
  }
};

// The K loop of one tile; K-blocks 0 .. STAGES - 2 are already on their way.
template <class CF, bool KFULL>
__device__ __forceinline__ void i8_k_loop(const I8Loader<CF>& ld, int nkb, const uint8_t* smem,
                                          v16i (&acc)[CF::TM][CF::TN]) {
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave / CF::WAVES_N, wn = wave % CF::WAVES_N;
  // Operand row r of a 32-row slice: lane r and lane r + 32 hold the two
  // 16-byte halves of each 32 bytes of K.
  const int fr = lane & 31, fg = lane >> 5;
  uint32_t lf[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) lf[h] = (uint32_t)(fr * BK + (((2 * h + fg) ^ swz_key(fr)) << 4));
#pragma unroll
  for (int i = 0; i < CF::TM; ++i)
#pragma unroll
    for (int j = 0; j < CF::TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  constexpr int STEPS = 4 * CF::TM;
  constexpr int PER = (CF::LOADS + STEPS - 1) / STEPS;
  for (int kb = 0; kb < nkb; ++kb) {
    if (CF::STAGES > 2 && kb + 1 < nkb) wait_vmcnt<CF::LOADS * (CF::STAGES - 2)>();
    else wait_vmcnt<0>();
    __syncthreads();
    const int kn = kb + CF::STAGES - 1, slot = kn % CF::STAGES;
    const uint8_t* at = smem + (kb % CF::STAGES) * CF::STAGE_BYTES + wm * CF::WM * BK;
    const uint8_t* bt = smem + (kb % CF::STAGES) * CF::STAGE_BYTES + CF::A_BYTES + wn * CF::WN * BK;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v4i fb[CF::TN];
#pragma unroll
      for (int j = 0; j < CF::TN; ++j) fb[j] = *reinterpret_cast<const v4i*>(bt + j * 32 * BK + lf[h]);
#pragma unroll
      for (int i = 0; i < CF::TM; ++i) {
        const v4i fa = *reinterpret_cast<const v4i*>(at + i * 32 * BK + lf[h]);
#pragma unroll
        for (int j = 0; j < CF::TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa, acc[i][j], 0, 0, 0);
        if (kn < nkb) {
#pragma unroll
          for (int n = (h * CF::TM + i) * PER; n < (h * CF::TM + i + 1) * PER && n < CF::LOADS; ++n)
            ld.template issue<KFULL>(n, kn, slot);
        }
      }
    }
  }
}

// Scale, round to bf16, stage in LDS (every wave is done with the ring) and
// store rows with 16-byte writes where the output allows.
template <class CF>
__device__ __forceinline__ void i8_store(const GemmI8Args& p, int64_t m0, int64_t n0,
                                         const v16i (&acc)[CF::TM][CF::TN], uint8_t* smem) {
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave / CF::WAVES_N, wn = wave % CF::WAVES_N;
  const int fr = lane & 31, fg = lane >> 5;
  const int64_t row0 = m0 + wm * CF::WM, col0 = n0 + wn * CF::WN;
  uint16_t* st = reinterpret_cast<uint16_t*>(smem) + wave * CF::WM * CF::CS;
  // lane (fr, fg), value 4q + v of subtile (i, j): row 32i + fr, column 32j + 8q + 4fg + v
  float as[CF::TM];
#pragma unroll
  for (int i = 0; i < CF::TM; ++i) {
    const int64_t r = row0 + 32 * i + fr;
    as[i] = p.a_s[r < p.M ? r : p.M - 1];
  }
#pragma unroll
  for (int j = 0; j < CF::TN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float bs[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t c = col0 + 32 * j + 8 * q + 4 * fg + v;
        bs[v] = p.b_s[c < p.N ? c : p.N - 1];
      }
#pragma unroll
      for (int i = 0; i < CF::TM; ++i) {
        float y[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = (float)acc[i][j][4 * q + v] * (as[i] * bs[v]);
        *reinterpret_cast<uint2*>(st + (32 * i + fr) * CF::CS + 32 * j + 8 * q + 4 * fg) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
    }
  __builtin_amdgcn_wave_barrier();
  const bool vec = (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 && p.ldc % 8 == 0;
  constexpr int CPR = CF::WN / 8, IT = CF::WM * CPR / 64;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int c = lane + 64 * it;
    const u32x4 v = *reinterpret_cast<const u32x4*>(st + (c / CPR) * CF::CS + (c % CPR) * 8);
    const int64_t row = row0 + c / CPR, col = col0 + (c % CPR) * 8;
    if (row >= p.M || col >= p.N) continue;
    uint16_t* dst = p.C + row * p.ldc + col;
    if (vec && col + 8 <= p.N) {
      *reinterpret_cast<u32x4*>(dst) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      for (int e = 0; e < 8 && col + e < p.N; ++e) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <class CF, bool KFULL>
__global__ __launch_bounds__(CF::kThreads) void gemm_i8_kernel(GemmI8Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[CF::LDS_BYTES];
  const int64_t tiles_m = (p.M + CF::BM - 1) / CF::BM, tiles_n = (p.N + CF::BN - 1) / CF::BN;
  const int nkb = (int)((p.K + BK - 1) / BK);
  for (int64_t pid = blockIdx.x; pid < tiles_m * tiles_n; pid += gridDim.x) {
    int64_t tm, tn;
    tile_of(pid, tiles_m, tiles_n, tm, tn);
    I8Loader<CF> ld;
    ld.init(p, tm * CF::BM, tn * CF::BN, smem);
    for (int s = 0; s < CF::STAGES - 1 && s < nkb; ++s)
#pragma unroll
      for (int n = 0; n < CF::LOADS; ++n) ld.template issue<KFULL>(n, s, s);
    v16i acc[CF::TM][CF::TN];
    i8_k_loop<CF, KFULL>(ld, nkb, smem, acc);
    __syncthreads();
    i8_store<CF>(p, tm * CF::BM, tn * CF::BN, acc, smem);
    __syncthreads();
  }
}

using I8Big = I8Cfg<256, 256, 2, 4, 2>;
using I8Mid = I8Cfg<128, 128, 2, 2, 2>;
using I8Small = I8Cfg<64, 64, 2, 2, 2>;

// ---- few output tiles: K split over the waves of a workgroup ---------------------------
//
// A workgroup owns a 16 FM x 16 FN tile; its W waves take the K-blocks in turn
// (wave w: w, w + W, ...), each through a ring of D LDS slots of its own that
// hold one K-block of the tile's rows, so no wave waits for another until the
// sums are added up at the end, by integer additions in LDS, whose order does
// not matter.  All of a wave's first D K-blocks are in flight at once.
//
// FUSED: the activations come as the quantiser's input and every workgroup
// quantises all M <= 16 rows of it itself, while its first weights are on
// their way; the codes stay in LDS (rows of code_ld bytes after the ring).
// HALF (FN = 1): 8 columns per workgroup, so that a narrow product reaches
// more CUs.

constexpr int kSplitWaves = 8;
constexpr int kFusedCodes = 16384;  // most codes (M * K) of a fused launch, which keeps two workgroups per CU

template <int FM, int FN, int D, bool FUSED, bool HALF>
struct SplitCfg {
  static constexpr int TM = 16 * FM, TN = HALF ? 8 : 16 * FN;
  static constexpr int AROWS = FUSED ? 0 : TM;
  static constexpr int SLOT = (AROWS + TN) * BK;
  static constexpr int LOADS = SLOT / 1024;  // 8 rows per load
  static constexpr int RING = kSplitWaves * D * SLOT;
  static constexpr int SUM = TM * 16 * FN * 4;
  static constexpr int LDS = RING > SUM ? RING : SUM;
  static constexpr int CODES = FUSED ? kFusedCodes + 16 * (BK - 16 + 16) : 0;
};

template <class SRC_TAG, int FM, int FN, int D, bool HALF>
__global__ __launch_bounds__(64 * kSplitWaves) void gemm_i8_split_kernel(GemmI8Args p, RowQuantArgs x, int code_ld) {
  constexpr bool FUSED = !std::is_void<SRC_TAG>::value;
  using CF = SplitCfg<FM, FN, D, FUSED, HALF>;
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
  const i32x4 rsA = make_rsrc(p.A + (FUSED ? 0 : m0 * p.lda), FUSED ? 0u : (uint32_t)((ra - 1) * p.lda + p.K));
  const i32x4 rsB = make_rsrc(p.B + n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb + p.K));
  uint32_t off[CF::LOADS], kc = 0;
#pragma unroll
  for (int n = 0; n < CF::LOADS; ++n) {
    const bool a = 8 * n < CF::AROWS;
    const int r = 8 * n - (a ? 0 : CF::AROWS) + (lane >> 3);
    const int c = (lane & 7) ^ swz_key(r);
    off[n] = r < (a ? ra : rb) ? (uint32_t)(r * (a ? p.lda : p.ldb) + c * 16) : kOob;
    kc |= (uint32_t)c << (3 * (n & 1));  // the chunk depends on the row modulo 16 alone
  }
  const uint32_t lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem)) + (uint32_t)(wave * D * CF::SLOT);
  auto issue = [&](int kb, int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n) {
      const uint32_t kbyte = (uint32_t)kb * BK;
      const bool in = kbyte + ((kc >> (3 * (n & 1))) & 7u) * 16u < K;
      dma_b128(8 * n < CF::AROWS ? rsA : rsB, lds0 + (uint32_t)(slot * CF::SLOT + n * 1024), in ? off[n] : kOob, kbyte);
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
    const int left = (nkb - 1 - kb) / kSplitWaves;
    if (D >= 4 && left >= 3) wait_vmcnt<CF::LOADS * (D >= 4 ? 3 : 0)>();
    else if (D >= 3 && left >= 2) wait_vmcnt<CF::LOADS * (D >= 3 ? 2 : 0)>();
    else if (D >= 2 && left >= 1) wait_vmcnt<CF::LOADS * (D >= 2 ? 1 : 0)>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
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
  const bool vec = (reinterpret_cast<uintptr_t>(p.C) & 7) == 0 && p.ldc % 4 == 0;
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
    if (vec && col + 4 <= p.N) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
      for (int v = 0; v < 4 && col + v < p.N; ++v) dst[v] = (uint16_t)(w[v >> 1] >> (16 * (v & 1)));
    }
  }
}

// ---- any alignment ---------------------------------------------------------------------

// 64x64 tiles, 4 waves of 32x32, any alignment: 16-byte chunks through
// registers into LDS.
__global__ __launch_bounds__(256) void gemm_i8_any_kernel(GemmI8Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2][64 * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int fr = lane & 15, fg = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  v4i acc[2][2];
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  for (int64_t k0 = 0; k0 < p.K; k0 += 128) {
    u32x4 ra[2], rb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 3) + 32 * i, c = tid & 7;
      const bool oa = m0 + r < p.M, ob = n0 + r < p.N;
      ra[i] = load16(p.A + (oa ? m0 + r : 0) * p.lda, k0 + 16 * c, p.K, oa);
      rb[i] = load16(p.B + (ob ? n0 + r : 0) * p.ldb, k0 + 16 * c, p.K, ob);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 3) + 32 * i, c = tid & 7;
      *reinterpret_cast<u32x4*>(smem[0] + chunk_at(r, c)) = ra[i];
      *reinterpret_cast<u32x4*>(smem[1] + chunk_at(r, c)) = rb[i];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4i fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const v4i*>(smem[0] + chunk_at(wm + 16 * i + fr, 4 * h + fg));
        fb[i] = *reinterpret_cast<const v4i*>(smem[1] + chunk_at(wn + 16 * i + fr, 4 * h + fg));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  // lane (fr, fg) holds row 16i + fr, columns 16j + 4fg ..+3
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = m0 + wm + 16 * i + fr;
    if (row >= p.M) continue;
    const float as = p.a_s[row];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t col = n0 + wn + 16 * j + 4 * fg + v;
        if (col < p.N)
          p.C[row * p.ldc + col] = (uint16_t)pack_bf16x2((float)acc[i][j][v] * (as * p.b_s[col]), 0.0f);
      }
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

inline bool aligned16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 16 == 0; }

template <class CF>
int64_t tiles(const GemmI8Args& a) {
  return ((a.M + CF::BM - 1) / CF::BM) * ((a.N + CF::BN - 1) / CF::BN);
}

template <class CF>
hipError_t launch_tiles(const GemmI8Args& a, hipStream_t stream) {
  const int64_t t = tiles<CF>(a);
  const dim3 grid((unsigned)(t < (1 << 20) ? t : (1 << 20)));
  if (a.K % BK == 0) hipLaunchKernelGGL((gemm_i8_kernel<CF, true>), grid, dim3(CF::kThreads), 0, stream, a);
  else hipLaunchKernelGGL((gemm_i8_kernel<CF, false>), grid, dim3(CF::kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

namespace {

// Operands for the direct-to-LDS loads, with a tile's rows within 31-bit offsets.
bool dma_ok(const GemmI8Args& a) {
  return a.K > 0 && a.K % 16 == 0 && aligned16(a.B, a.ldb) && a.ldb < (1 << 23) && aligned16(a.A, a.lda) &&
         a.lda < (1 << 23);
}

template <class SRC_TAG, int FM, int FN, int D, bool HALF>
hipError_t launch_split(const GemmI8Args& a, const RowQuantArgs& x, hipStream_t stream) {
  constexpr bool FUSED = !std::is_void<SRC_TAG>::value;
  using CF = SplitCfg<FM, FN, D, FUSED, HALF>;
  auto kernel = gemm_i8_split_kernel<SRC_TAG, FM, FN, D, HALF>;
  // rows of codes 16 bytes apart modulo the LDS's 128-byte bank row
  const int code_ld = FUSED ? (int)((a.K + BK - 1) / BK * BK + 16) : 0;
  const int64_t grid = (a.M + CF::TM - 1) / CF::TM * ((a.N + CF::TN - 1) / CF::TN);
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * kSplitWaves), 0, stream, a, x, code_ld);
  return hipGetLastError();
}

}  // namespace

// The int8 linear layer in one launch: few rows, whose quantisation every
// workgroup repeats.
bool linear_i8_fused(const GemmI8Args& g, const RowQuantArgs& q) {
  return g.M <= 16 && g.K >= 8 && g.K % 16 == 0 && aligned16(g.B, g.ldb) && g.ldb < (1 << 23) &&
         g.M * g.K <= kFusedCodes && !q.f32;
}

hipError_t launch_linear_i8_fused(const GemmI8Args& g, const RowQuantArgs& q, hipStream_t stream) {
  using Plain = std::integral_constant<Src, kBf16>;
  using Gated = std::integral_constant<Src, kGated>;
  const bool half = (g.N + 15) / 16 < device_cu_count();
  if (q.u != nullptr)
    return half ? launch_split<Gated, 1, 1, 4, true>(g, q, stream) : launch_split<Gated, 1, 1, 3, false>(g, q, stream);
  return half ? launch_split<Plain, 1, 1, 4, true>(g, q, stream) : launch_split<Plain, 1, 1, 3, false>(g, q, stream);
}

hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  if (dma_ok(a)) {
    const int cus = device_cu_count();
    const RowQuantArgs none{};
    if (tiles<I8Big>(a) >= cus) return launch_tiles<I8Big>(a, stream);
    if (tiles<I8Mid>(a) >= cus) return launch_tiles<I8Mid>(a, stream);
    if (a.M <= 16)
      return (a.N + 15) / 16 < cus ? launch_split<void, 1, 1, 4, true>(a, none, stream)
                                   : launch_split<void, 1, 1, 2, false>(a, none, stream);
    if (a.M <= 32) return launch_split<void, 2, 1, 2, false>(a, none, stream);
    if (tiles<I8Small>(a) >= cus) return launch_tiles<I8Small>(a, stream);
    return launch_split<void, 4, 2, 1, false>(a, none, stream);
  }
  const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64));
  hipLaunchKernelGGL(gemm_i8_any_kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dsfp8
