// MXFP4 linear layer on gfx950: rows in blocks of 32 columns, each block with
// one power-of-two scale (a byte, biased by 127) and 4-bit e2m1 codes (the
// OCP microscaling format), and products of such matrices.
//
// Quantisation of a block x of 32 columns:
//   e = max(floor(log2 max |x|) - 2, -127),  q = e2m1(x / 2^e),
// nearest-even, |q| <= 6; the scale byte is e + 127.  floor(log2) of an fp32
// value is its exponent field, so the scale byte is that field minus 2, and
// the division is part of the hardware's conversion, which rounds exactly
// (its tests hold every bf16 value against every scale it can have).  A block that
// holds a NaN or an infinity has the field 255 and gets the scale byte 255, the
// format's NaN.
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "tile.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));  // an access at any address
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kMx = 32;  // elements of a block

// ---- quantisation ----------------------------------------------------------------------

enum Src { kBf16, kF32, kGated };

// SiLU(g) * u in fp32, not rounded before the quantisation.
__device__ __forceinline__ float gate(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Eight consecutive elements of a row as loaded; zeros past the row.
template <Src SRC>
struct Chunk {
  u32x4 r[SRC == kBf16 ? 1 : 2];

  __device__ __forceinline__ void load(const MxQuantArgs& a, int64_t m, int64_t k, bool on) {
#pragma unroll
    for (auto& w : r) w = u32x4{0u, 0u, 0u, 0u};
    if (!on || k >= a.K) return;
    const bool full = k + 8 <= a.K;
    if constexpr (SRC == kF32) {
      const uint32_t* src = static_cast<const uint32_t*>(a.x) + m * a.ldx + k;
      if (full) {
        r[0] = *reinterpret_cast<const u32x4u*>(src);
        r[1] = *reinterpret_cast<const u32x4u*>(src + 4);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < a.K) r[i >> 2][i & 3] = src[i];
      }
    } else {
#pragma unroll
      for (int h = 0; h < (SRC == kGated ? 2 : 1); ++h) {
        const uint16_t* src = h ? a.u + m * a.ldu + k : static_cast<const uint16_t*>(a.x) + m * a.ldx + k;
        if (full) {
          r[h] = *reinterpret_cast<const u32x4u*>(src);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (k + i < a.K) r[h][i >> 1] |= (uint32_t)src[i] << (16 * (i & 1));
        }
      }
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
};

// Four lanes per block, eight columns each.  UNITS blocks of a lane are in
// flight together, a grid's width apart.
template <Src SRC, int UNITS>
__global__ __launch_bounds__(256) void mx_quant_kernel(MxQuantArgs a, FastDiv per_row, uint32_t total) {
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t t0 = blockIdx.x * 256u + threadIdx.x; t0 < total; t0 += UNITS * step) {
    Chunk<SRC> c[UNITS];
    uint32_t m[UNITS], k[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const uint32_t t = t0 + i * step;
      m[i] = fastdiv(t, per_row);
      k[i] = t - m[i] * per_row.d;
      c[i].load(a, m[i], (int64_t)k[i] * 8, t < total);
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      float v[8];
      c[i].values(v);
      const uint32_t s = mx_scale(mx_quad_top(v));
      if (t0 + i * step < total) {
        reinterpret_cast<uint32_t*>(a.y + (int64_t)m[i] * a.ldy)[k[i]] = mx_codes8(v, mx_scale_f32(s));
        if ((k[i] & 3) == 0) a.s[(int64_t)m[i] * a.lds + (k[i] >> 2)] = (uint8_t)s;
      }
    }
  }
}

// ---- dequantisation --------------------------------------------------------------------

// Eight columns per lane: code times scale, exact in bf16 (a product beyond its
// range is an infinity; the scale byte 255 gives NaN).
template <int UNITS>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxDequantArgs a, FastDiv per_row, uint32_t total) {
  const uint32_t step = gridDim.x * 256u;
  for (uint32_t t0 = blockIdx.x * 256u + threadIdx.x; t0 < total; t0 += UNITS * step) {
    uint32_t q[UNITS], m[UNITS], k[UNITS], s[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const uint32_t t = t0 + i * step < total ? t0 + i * step : total - 1;
      m[i] = fastdiv(t, per_row);
      k[i] = t - m[i] * per_row.d;
      q[i] = reinterpret_cast<const uint32_t*>(a.q + (int64_t)m[i] * a.ldq)[k[i]];
      s[i] = a.s[(int64_t)m[i] * a.lds + (k[i] >> 2)];
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      if (t0 + i * step >= total) break;
      const float scale = s[i] == 255 ? __uint_as_float(0x7fc00000u) : mx_scale_f32(s[i]);
      u32x4 w;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        // both codes of byte h as fp32 values: a shift of the sign and an exact product
        float v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t c = (q[i] >> (8 * h + 4 * e)) & 15u, mag = c & 7u;
          const float f = mag < 2 ? 0.5f * (float)mag : __uint_as_float(((mag >> 1) + 126u) << 23 | (mag & 1u) << 22);
          v[e] = __uint_as_float(__float_as_uint(f) | (c & 8u) << 28) * scale;
        }
        w[h] = pack_bf16x2(v[0], v[1]);
      }
      uint16_t* dst = a.out + (int64_t)m[i] * a.ldo + (int64_t)k[i] * 8;
      if ((int64_t)k[i] * 8 + 8 <= a.K) {
        *reinterpret_cast<u32x4u*>(dst) = w;
      } else {
        for (int e = 0; e < 8 && (int64_t)k[i] * 8 + e < a.K; ++e) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

// ---- where a workgroup's tile lies -------------------------------------------------------

// Rows [m0, m1) of the product and columns from n0, with the weight they multiply.
struct MxTile {
  int64_t m0, m1, n0;
  const uint8_t *B, *b_s;
};

// Row tile `want` of the experts' row ranges, every expert's range cut into
// tiles of BM rows; false behind the last one.  A wave reads 64 experts'
// offsets at a time and adds up their tiles.  Offsets are clamped to [0, M],
// so that malformed ones cannot name a row outside.
template <int BM>
__device__ __forceinline__ bool mx_find(const MxGemmArgs& p, int64_t want, MxTile& t) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int64_t base = 0; base < p.E; base += 64) {
    const int64_t e = base + lane;
    int lo = 0, hi = 0;
    if (e < p.E) {
      lo = p.offsets[e];
      hi = p.offsets[e + 1];
    }
    lo = lo < 0 ? 0 : (lo > (int)p.M ? (int)p.M : lo);
    hi = hi < lo ? lo : (hi > (int)p.M ? (int)p.M : hi);
    const uint32_t n = ((uint32_t)(hi - lo) + BM - 1) / BM;
    uint32_t sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)sum, d);
      sum += lane >= d ? o : 0u;
    }
    const uint64_t past = __ballot(before + (int64_t)sum > want);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      const int64_t first = before + __builtin_amdgcn_readlane((int)(sum - n), l);
      const int64_t e0 = base + l;
      t.m0 = __builtin_amdgcn_readlane(lo, l) + (want - first) * BM;
      t.m1 = __builtin_amdgcn_readlane(hi, l);
      t.B = p.B + e0 * p.N * p.ldb;
      t.b_s = p.b_s + e0 * p.N * p.ldbs;
      return want >= first && t.m0 < t.m1;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
  }
  return false;
}

// ---- tiles -----------------------------------------------------------------------------
//
// BM x BN tiles, each wave WM x WN of it in 32x32 subtiles of
// v_mfma_scale_f32_32x32x64_f8f6f4.  Lane (fr, fg) of an instruction holds 16
// bytes, the 32 columns of one block of row fr, and that block's scale byte, which
// the instruction applies.
//
// The operands go through the same ring of LDS stages as the other tiled
// products', filled by buffer_load ... lds; a stage is a K-block of 128 bytes a row,
// 256 columns, four matrix instructions deep, read without bank conflicts through
// the XOR swizzle.  The scale bytes of two K-blocks (16 bytes a row) are loaded
// together, one load per 64 rows, into buffers of their own behind the stages.
//
// A matrix instruction of this format takes half as long as one of 8 bits, so
// its operands are read one step (64 columns) ahead into registers, and over the
// K-blocks' border too: the barrier that hands over the next K-block comes before
// the last step of the current one, whose operands are in registers by then.
// The stage it leaves is refilled behind that step's instructions.
//
// 256x256 tiles, 4096x7168x18432: 269 us (4.0 PFLOP/s; 4096x18432x7168 297-301).  Two
// things bound it, close together: without the loads the rest takes 228 us (the matrix
// cores at the clock that the power allows: 6.1-7.1 PFLOP/s from registers alone),
// without the matrix instructions 230 us (of which the scales' loads, a line per
// row, are 27; LDS reads alone take 116).  Two more add to both: the last round of
// workgroups (1.75 rounds over the CUs run as two, an eighth of their time idle;
// 4096x18432x7168 4.5 as five, a tenth), and reading the scales from LDS, dwords at a
// stride of 16 bytes: without these reads 254 us (283), and of the bank conflicts, 14% of
// the cycles, 1% stay.  Stages of 64 bytes a row, four of
// them or three, took 294 us; waves of 128x128, four a workgroup, 290.

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct MxCfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
  static constexpr int NW = WAVES_M * WAVES_N;
  static constexpr int kThreads = 64 * NW;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int TM = WM / 32, TN = WN / 32;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int A_INSTR = A_BYTES / 1024 / NW, B_INSTR = B_BYTES / 1024 / NW, LOADS = A_INSTR + B_INSTR;
  static constexpr int S_ROWS = BM + BN, S_INSTR = (S_ROWS / 64 + NW - 1) / NW;  // scale loads of a wave
  static constexpr int S_BYTES = S_INSTR * NW * 1024, S_BUFS = STAGES / 2 + 1;
  static constexpr int C_BYTES = 32 * WN * 2;  // 32 rows of a wave's output
  static constexpr int LDS = STAGES * STAGE_BYTES + S_BUFS * S_BYTES;
  static constexpr int PER_CU = 160 * 1024 / LDS;  // workgroups that share a CU
  // Scale loads that go with K-blocks a .. b (every second one).
  static constexpr int scales_in(int a, int b) { return b < a ? 0 : (b / 2 - (a + 1) / 2 + 1) * S_INSTR; }
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole 1 KB segments per wave");
  static_assert(WM % 32 == 0 && WN % 32 == 0 && BM % 64 == 0 && BN % 64 == 0, "32x32 subtiles, scale loads of 64 rows");
  static_assert(NW % 2 == 0, "a wave's segments start at rows that agree modulo 16");
  static_assert(STAGES >= 2 && (STAGES - 1) * LOADS + S_BUFS * S_INSTR < 64, "the waits of the K loop");
  static_assert(NW * C_BYTES <= STAGE_BYTES, "the output's staging");
  static_assert(PER_CU >= 1, "LDS");
};

template <class CF, bool GROUPED>
struct MxLoader {
  i32x4 rsA, rsB, rsAS, rsBS;
  // A lane's row in load 0 of each operand and the step from load to load (a row
  // past the matrix lies past the descriptor's end by itself); grouped rows may
  // be anywhere.
  uint32_t offA[GROUPED ? CF::A_INSTR : 1], offB, stepA, stepB, soff[CF::S_INSTR];
  uint32_t kc;  // byte within the K-block of every load's chunk (a wave's rows agree modulo 16)
  uint32_t lds0, sds0;
  uint32_t KR;  // bytes of a row's codes
  int wave;

  __device__ __forceinline__ void init(const MxGemmArgs& p, const MxTile& t, uint8_t* smem) {
    const int lane = lane_id();
    wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    KR = (uint32_t)(p.KB * 16);
    const int64_t ra = t.m1 - t.m0 < CF::BM ? t.m1 - t.m0 : CF::BM, rb = p.N - t.n0 < CF::BN ? p.N - t.n0 : CF::BN;
    // rows through an index: the whole matrix behind one descriptor
    const bool at = GROUPED && p.rows;
    const int64_t m0 = at ? 0 : t.m0, ha = at ? p.a_rows : ra;
    rsA = make_rsrc(p.A + m0 * p.lda, (uint32_t)((ha - 1) * p.lda) + KR);
    rsB = make_rsrc(t.B + t.n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb) + KR);
    rsAS = make_rsrc(p.a_s + m0 * p.ldas, (uint32_t)(ha * p.ldas));
    rsBS = make_rsrc(t.b_s + t.n0 * p.ldbs, (uint32_t)(rb * p.ldbs));
    auto a_row = [&](int64_t r) __attribute__((always_inline)) {
      if (!at) return (uint32_t)r;
      const int32_t v = p.rows[t.m0 + r];
      return (uint32_t)(v < 0 ? 0 : (v < p.a_rows ? v : p.a_rows - 1));
    };
    const int r0 = wave * 8 + (lane >> 3);
    kc = (uint32_t)((lane & 7) ^ swz_key(r0)) * 16;
    if constexpr (GROUPED) {
#pragma unroll
      for (int n = 0; n < CF::A_INSTR; ++n) {
        const int r = r0 + CF::NW * 8 * n;
        offA[n] = r < ra ? a_row(r) * (uint32_t)p.lda + kc : kOob;
      }
    } else {
      offA[0] = (uint32_t)(r0 * p.lda) + kc;
    }
    offB = (uint32_t)(r0 * p.ldb) + kc;
    stepA = (uint32_t)(CF::NW * 8 * p.lda);
    stepB = (uint32_t)(CF::NW * 8 * p.ldb);
#pragma unroll
    for (int n = 0; n < CF::S_INSTR; ++n) {
      const int g = (wave + CF::NW * n) * 64 + lane, r = g < CF::BM ? g : g - CF::BM;
      soff[n] = kOob;
      if (g < CF::S_ROWS && r < (g < CF::BM ? ra : rb))
        soff[n] = g < CF::BM ? a_row(r) * (uint32_t)p.ldas : (uint32_t)(r * p.ldbs);
    }
    lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem));
    sds0 = lds0 + (uint32_t)(CF::STAGES * CF::STAGE_BYTES + wave * 1024);
  }

  // Load n of K-block kb into ring place `place`; one past the row's end fetches
  // nothing (its lanes are out of range and read as zero).
  __device__ __forceinline__ void issue(int n, int kb, int place) const {
    const bool a = n < CF::A_INSTR;
    const int i = a ? n : n - CF::A_INSTR;
    const uint32_t kbyte = (uint32_t)kb * BK;
    const uint32_t at = lds0 + (uint32_t)(place * CF::STAGE_BYTES + (a ? 0 : CF::A_BYTES) + (wave + CF::NW * i) * 1024);
    const uint32_t off = !a ? offB + (uint32_t)i * stepB : (GROUPED ? offA[GROUPED ? i : 0] : offA[0] + (uint32_t)i * stepA);
    dma_b128(a ? rsA : rsB, at, kbyte + kc < KR ? off : kOob, kbyte);
  }
  // The scales of K-blocks kb and kb + 1 (kb even).
  __device__ __forceinline__ void issue_scales(int kb) const {
    const bool in = (uint32_t)kb * BK < KR;
    const int q = kb / 2;
#pragma unroll
    for (int n = 0; n < CF::S_INSTR; ++n)
      dma_b128((wave + CF::NW * n) * 64 < CF::BM ? rsAS : rsBS,
               sds0 + (uint32_t)(q % CF::S_BUFS * CF::S_BYTES + CF::NW * n * 1024), in ? soff[n] : kOob, (uint32_t)q * 16);
  }
};

// A wave's operands: fragments of one step, and the scale bytes of two.
template <class CF>
struct MxOperands {
  const uint8_t* smem;
  int at, bt, sat, sbt;  // in a stage, and in a buffer of scales
  int lf[4];
  int shift;

  __device__ __forceinline__ explicit MxOperands(const uint8_t* smem) : smem(smem) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int fr = lane & 31, fg = lane >> 5;
    const int wm = wave / CF::WAVES_N * CF::WM, wn = wave % CF::WAVES_N * CF::WN;
    at = wm * BK;
    bt = CF::A_BYTES + wn * BK;
    sat = CF::STAGES * CF::STAGE_BYTES + (wm + fr) * 16;
    sbt = CF::STAGES * CF::STAGE_BYTES + (CF::BM + wn + fr) * 16;
    shift = 8 * fg;
#pragma unroll
    for (int h = 0; h < 4; ++h) lf[h] = fr * BK + (((2 * h + fg) ^ swz_key(fr)) << 4);
  }
  __device__ __forceinline__ u32x4 a(int place, int h, int i) const {
    return *reinterpret_cast<const u32x4*>(smem + place * CF::STAGE_BYTES + lf[h] + at + 32 * i * BK);
  }
  __device__ __forceinline__ u32x4 b(int place, int h, int j) const {
    return *reinterpret_cast<const u32x4*>(smem + place * CF::STAGE_BYTES + lf[h] + bt + 32 * j * BK);
  }
  // Dword d of the rows' scales in K-block kb, for steps 2d and 2d + 1: step h uses
  // byte 2h + fg of a row's eight, byte 0 or 2 of the dword shifted by fg bytes.
  // `mask` clears the blocks that a short last K-block does not have: their codes
  // read as zero, but their scale bytes may hold anything, and 255 would make NaN
  // of them.
  __device__ __forceinline__ void scales(int kb, int d, uint32_t mask, uint32_t (&sa)[CF::TM], uint32_t (&sb)[CF::TN]) const {
    const uint8_t* b = smem + kb / 2 % CF::S_BUFS * CF::S_BYTES + kb % 2 * 8 + 4 * d;
#pragma unroll
    for (int i = 0; i < CF::TM; ++i) sa[i] = (*reinterpret_cast<const uint32_t*>(b + sat + 32 * i * 16) & mask) >> shift;
#pragma unroll
    for (int j = 0; j < CF::TN; ++j) sb[j] = (*reinterpret_cast<const uint32_t*>(b + sbt + 32 * j * 16) & mask) >> shift;
  }
};

// One step of a 32x32 subtile, the weight first, so that a lane's results are
// runs of four columns of a row.
template <int H>
__device__ __forceinline__ v16f mx_mfma(u32x4 b, uint32_t sb, u32x4 a, uint32_t sa, v16f c) {
  const v8i b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const v8i a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, c, 4, 4, 2 * (H & 1), (int)sb, 2 * (H & 1), (int)sa);
}

// C values of a wave, rounded to bf16 and stored 32 rows at a time through an
// LDS area of the wave's own, so that rows leave as 16-byte writes at any address.
// Lane (fr, fg), value 4q + v of subtile (i, j) is row 32i + fr, column
// 32j + 8q + 4fg + v.
template <class CF>
__device__ __forceinline__ void mx_store(const MxGemmArgs& p, const MxTile& t, const v16f (&acc)[CF::TM][CF::TN],
                                         uint8_t* area) {
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 31, fg = lane >> 5;
  const int64_t row0 = t.m0 + wave / CF::WAVES_N * CF::WM, col0 = t.n0 + wave % CF::WAVES_N * CF::WN;
  uint8_t* st = area + wave * CF::C_BYTES;
  constexpr int CPR = CF::WN / 8, IT = 32 * CPR / 64, MASK = CPR < 8 ? CPR - 1 : 7;
#pragma unroll
  for (int i = 0; i < CF::TM; ++i) {
#pragma unroll
    for (int j = 0; j < CF::TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint2*>(st + fr * CF::WN * 2 + (((4 * j + q) ^ (fr & MASK)) << 4) + 8 * fg) =
            make_uint2(pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                       pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
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
      if (row >= t.m1 || col >= p.N) continue;
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

// Step H of a K-block; follow(i) is called behind the instructions of each
// subtile row i, whose operand is then free.
template <class CF, int H, class Follow>
__device__ __forceinline__ void mx_step(v16f (&acc)[CF::TM][CF::TN], u32x4 (&fa)[CF::TM], const u32x4 (&fb)[CF::TN],
                                        const uint32_t (&sa)[CF::TM], const uint32_t (&sb)[CF::TN], Follow&& follow) {
#pragma unroll
  for (int i = 0; i < CF::TM; ++i) {
#pragma unroll
    for (int j = 0; j < CF::TN; ++j) acc[i][j] = mx_mfma<H>(fb[j], sb[j], fa[i], sa[i], acc[i][j]);
    follow(i);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Workgroups walk the tiles, a grid's width apart: the next tile's first stages
// are on their way while the current one is stored, through the place of the
// last stage.
template <class CF, bool GROUPED>
__global__ __launch_bounds__(CF::kThreads) void mx_gemm_kernel(MxGemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[CF::LDS];
  constexpr int S = CF::STAGES, L = CF::LOADS;
  const int64_t tiles_m = (p.M + CF::BM - 1) / CF::BM, tiles_n = (p.N + CF::BN - 1) / CF::BN;
  const int nkb = (int)((p.KB + 7) / 8), left = (int)(p.KB & 7);
  const uint64_t tail = left ? (1ull << (8 * left)) - 1 : ~0ull;  // the blocks of the last K-block
  const MxOperands<CF> op(smem);
  int64_t pid = blockIdx.x;
  auto locate = [&](MxTile& t) __attribute__((always_inline)) {
    if constexpr (GROUPED) {
      const int64_t rt = div_u(pid, tiles_n);
      if (!mx_find<CF::BM>(p, rt, t)) return false;
      t.n0 = (pid - rt * tiles_n) * CF::BN;
    } else {
      if (pid >= tiles_m * tiles_n) return false;
      int64_t tm, tn;
      tile_of(pid, tiles_m, tiles_n, tm, tn);
      t = MxTile{tm * CF::BM, p.M, tn * CF::BN, p.B, p.b_s};
    }
    return true;
  };
  MxTile t;
  if (!locate(t)) return;
  MxLoader<CF, GROUPED> ld;
  auto begin = [&](int from, int to) __attribute__((always_inline)) {
#pragma unroll
    for (int kb = 0; kb < S; ++kb) {
      if (kb < from || kb >= to) continue;
#pragma unroll
      for (int n = 0; n < L; ++n) ld.issue(n, kb, kb);
      if (kb % 2 == 0) ld.issue_scales(kb);
    }
  };
  ld.init(p, t, smem);
  begin(0, S - 1);
  for (;;) {
    v16f acc[CF::TM][CF::TN];
#pragma unroll
    for (int i = 0; i < CF::TM; ++i)
#pragma unroll
      for (int j = 0; j < CF::TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    // The loop over the K-blocks has no branch inside, since the compiler would
    // move matrix instructions across it: loads past the row's end fetch nothing,
    // and the same numbers of them are in flight at every wait.
    if (nkb > 0) {
      u32x4 fa[CF::TM], fb[2][CF::TN];
      uint32_t sa[2][CF::TM], sb[2][CF::TN];
      begin(S - 1, S);
      // K-block 0 has arrived when only the S - 1 later ones may be missing
      wait_vmcnt<(S - 1) * L + CF::scales_in(1, S - 1)>();
      __syncthreads();
#pragma unroll
      for (int j = 0; j < CF::TN; ++j) fb[0][j] = op.b(0, 0, j);
#pragma unroll
      for (int i = 0; i < CF::TM; ++i) fa[i] = op.a(0, 0, i);
      op.scales(0, 0, nkb == 1 ? (uint32_t)tail : ~0u, sa[0], sb[0]);
      constexpr int PER = (L + CF::TM - 1) / CF::TM;
      int place = 0;
      auto run = [&](int kb, auto odd) __attribute__((always_inline)) {
        constexpr int X = decltype(odd)::value;
        const int next = place + 1 == S ? 0 : place + 1;
        auto ahead = [&](int h) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < CF::TN; ++j) fb[h & 1][j] = op.b(place, h, j);
        };
        op.scales(kb, 1, kb + 1 >= nkb ? (uint32_t)(tail >> 32) : ~0u, sa[1], sb[1]);
        ahead(1);
        mx_step<CF, 0>(acc, fa, fb[0], sa[0], sb[0], [&](int i) { fa[i] = op.a(place, 1, i); });
        ahead(2);
        mx_step<CF, 1>(acc, fa, fb[1], sa[0], sb[0], [&](int i) { fa[i] = op.a(place, 2, i); });
        ahead(3);
        mx_step<CF, 2>(acc, fa, fb[0], sa[1], sb[1], [&](int i) { fa[i] = op.a(place, 3, i); });
        // K-block kb + 1, when kb + 2 .. kb + S - 1 are missing
        wait_vmcnt<(S - 2) * L + CF::scales_in(X + 2, X + S - 1)>();
        __syncthreads();
        op.scales(kb + 1, 0, kb + 2 >= nkb ? (uint32_t)tail : ~0u, sa[0], sb[0]);
#pragma unroll
        for (int j = 0; j < CF::TN; ++j) fb[0][j] = op.b(next, 0, j);
        mx_step<CF, 3>(acc, fa, fb[1], sa[1], sb[1], [&](int i) __attribute__((always_inline)) {
          fa[i] = op.a(next, 0, i);
#pragma unroll
          for (int n = i * PER; n < (i + 1) * PER && n < L; ++n) ld.issue(n, kb + S, place);
          if (i == CF::TM - 1 && (X + S) % 2 == 0) ld.issue_scales(kb + S);
        });
        place = next;
      };
      int kb = 0;
      for (; kb + 1 < nkb; kb += 2) {
        run(kb, std::integral_constant<int, 0>{});
        run(kb + 1, std::integral_constant<int, 1>{});
      }
      if (kb < nkb) run(kb, std::integral_constant<int, 0>{});
    }
    // what has been loaded past the row's end is no longer on its way
    wait_vmcnt<0>();
    __syncthreads();
    MxTile u;
    pid += gridDim.x;
    const bool more = locate(u);
    if (more) {
      ld.init(p, u, smem);
      begin(0, S - 1);
    }
    mx_store<CF>(p, t, acc, smem + (S - 1) * CF::STAGE_BYTES);
    if (!more) break;
    t = u;
    __syncthreads();
  }
}

// ---- few rows or few tiles: K split over the waves of a workgroup -----------------------
//
// A workgroup owns a 16 FM x 16 FN tile; its eight waves take the K-blocks of 128
// bytes a row (256 columns) in turn, each through a ring of D LDS slots of its own
// that hold one K-block of the tile's rows and of their scales, so no wave waits for another
// until the sums are added up at the end, in the order of the waves.  All of a wave's
// first D K-blocks are in flight at once.  v_mfma_scale_f32_16x16x128_f8f6f4: lane
// (fr, fg) holds block fg of the four of row fr.
//
// FUSED: the activations come as bf16 rows and every workgroup quantises all M <=
// 16 of them itself, while its first weights are on their way; codes and
// scales stay in LDS.

constexpr int kSplitWaves = 8;
constexpr int kFusedBytes = 16384;  // room for the codes and scales of a fused launch

// Bytes of a row of codes and of scales in LDS: whole K-blocks, and a few more so
// that rows do not start in the same bank.
__host__ __device__ constexpr int mx_code_ld(int nkb) { return nkb * BK + 16; }
__host__ __device__ constexpr int mx_scale_ld(int nkb) { return nkb * 8 + 8; }

template <int FM, int FN, int D, bool FUSED>
struct SplitCfg {
  static constexpr int TM = 16 * FM, TN = 16 * FN;
  static constexpr int AROWS = FUSED ? 0 : TM, ROWS = AROWS + TN;
  static constexpr int LOADS = ROWS / 8;  // 8 rows each
  static constexpr int AS_LOADS = (AROWS + 31) / 32, S_LOADS = AS_LOADS + (TN + 31) / 32;  // scales of 32 rows each
  static constexpr int SLOT = ROWS * BK + S_LOADS * 256;
  static constexpr int RING = kSplitWaves * D * SLOT;
  static constexpr int SUM = kSplitWaves * FM * FN * 1024;
  static constexpr int LDS = (RING > SUM ? RING : SUM) + (FUSED ? kFusedBytes : 0);
  static_assert(D <= 4 && (LOADS + S_LOADS) * (D - 1) < 64, "waits of the ring");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <int FM, int FN, int D, bool FUSED, bool GROUPED>
__global__ __launch_bounds__(64 * kSplitWaves) void mx_split_kernel(MxGemmArgs p, MxQuantArgs x) {
  static_assert(!(FUSED && GROUPED), "grouped operands are quantised already");
  using CF = SplitCfg<FM, FN, D, FUSED>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[CF::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 15, fg = lane >> 4;
  const uint32_t tiles_n = (uint32_t)((p.N + CF::TN - 1) / CF::TN);
  const uint32_t tm = blockIdx.x / tiles_n;
  MxTile t;
  if constexpr (GROUPED) {
    if (!mx_find<CF::TM>(p, tm, t)) return;
  } else {
    t = MxTile{FUSED ? 0 : (int64_t)tm * CF::TM, p.M, 0, p.B, p.b_s};
  }
  t.n0 = (int64_t)(blockIdx.x - tm * tiles_n) * CF::TN;
  const int nkb = (int)((p.KB + 7) / 8);
  const uint32_t KR = (uint32_t)(p.KB * 16);
  const int64_t ra = t.m1 - t.m0 < CF::TM ? t.m1 - t.m0 : CF::TM, rb = p.N - t.n0 < CF::TN ? p.N - t.n0 : CF::TN;
  const bool at = GROUPED && p.rows;
  const int64_t m0 = at ? 0 : t.m0, ha = at ? p.a_rows : ra;
  i32x4 rsA, rsAS;
  if constexpr (!FUSED) {
    rsA = make_rsrc(p.A + m0 * p.lda, (uint32_t)((ha - 1) * p.lda) + KR);
    rsAS = make_rsrc(p.a_s + m0 * p.ldas, (uint32_t)(ha * p.ldas));
  }
  const i32x4 rsB = make_rsrc(t.B + t.n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb) + KR);
  const i32x4 rsBS = make_rsrc(t.b_s + t.n0 * p.ldbs, (uint32_t)(rb * p.ldbs));
  auto a_row = [&](int r) __attribute__((always_inline)) {
    if (!at) return (uint32_t)r;
    const int32_t v = p.rows[t.m0 + r];
    return (uint32_t)(v < 0 ? 0 : (v < p.a_rows ? v : p.a_rows - 1));
  };
  // Load n fetches rows 8n .. 8n + 7 of the slot (A's rows, then B's); a lane's
  // chunk depends on the row modulo 16 alone.
  const uint32_t kc[2] = {(uint32_t)((lane & 7) ^ swz_key(lane >> 3)) * 16,
                          (uint32_t)((lane & 7) ^ swz_key(8 + (lane >> 3))) * 16};
  uint32_t off[CF::LOADS];
#pragma unroll
  for (int n = 0; n < CF::LOADS; ++n) {
    const bool a = 8 * n < CF::AROWS;
    const int r = 8 * n - (a ? 0 : CF::AROWS) + (lane >> 3);
    off[n] = kOob;
    if (r < (a ? ra : rb)) off[n] = (a ? a_row(r) * (uint32_t)p.lda : (uint32_t)(r * p.ldb)) + kc[n & 1];
  }
  // Lane l of a load of scales: four of the eight bytes of row l / 2 (A's rows,
  // then B's, in loads of their own).
  uint32_t soff[CF::S_LOADS];
#pragma unroll
  for (int n = 0; n < CF::S_LOADS; ++n) {
    const bool a = n < CF::AS_LOADS;
    const int r = 32 * (a ? n : n - CF::AS_LOADS) + (lane >> 1);
    soff[n] = kOob;
    if (r < (a ? ra : rb)) soff[n] = (a ? a_row(r) * (uint32_t)p.ldas : (uint32_t)(r * p.ldbs)) + 4 * (lane & 1);
  }
  const uint32_t lds0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(smem)) + (uint32_t)(wave * D * CF::SLOT);
  auto issue = [&](int kb, int slot) __attribute__((always_inline)) {
    const uint32_t kbyte = (uint32_t)kb * BK, to = lds0 + (uint32_t)(slot * CF::SLOT);
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n)
      dma_b128(8 * n < CF::AROWS ? rsA : rsB, to + (uint32_t)(n * 1024), kbyte + kc[n & 1] < KR ? off[n] : kOob, kbyte);
#pragma unroll
    for (int n = 0; n < CF::S_LOADS; ++n)
      dma_b32(n < CF::AS_LOADS ? rsAS : rsBS, to + (uint32_t)(CF::ROWS * BK + n * 256), soff[n], (uint32_t)kb * 8);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wave + d * kSplitWaves < nkb) issue(wave + d * kSplitWaves, d);

  uint8_t* codes = smem + CF::LDS - (FUSED ? kFusedBytes : 0);
  uint8_t* scales = codes + (FUSED ? (int)p.M * mx_code_ld(nkb) : 0);
  if constexpr (FUSED) {
    // Chunks of 8 columns of all rows, dealt to the threads in turn, four
    // loads of a thread in flight.
    constexpr int HOLD = 4;
    const int per_row = (int)p.KB * 4, units = (int)p.M * per_row;
    for (int u0 = threadIdx.x; u0 < units; u0 += HOLD * 64 * kSplitWaves) {
      Chunk<kBf16> c[HOLD];
      int m[HOLD], k[HOLD];
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        const int u = u0 + i * 64 * kSplitWaves;
        m[i] = u / per_row;
        k[i] = u - m[i] * per_row;
        c[i].load(x, m[i], (int64_t)k[i] * 8, u < units);
      }
#pragma unroll
      for (int i = 0; i < HOLD; ++i) {
        float v[8];
        c[i].values(v);
        const uint32_t sc = mx_scale(mx_quad_top(v));
        if (u0 + i * 64 * kSplitWaves < units) {
          reinterpret_cast<uint32_t*>(codes + m[i] * mx_code_ld(nkb))[k[i]] = mx_codes8(v, mx_scale_f32(sc));
          if ((k[i] & 3) == 0) scales[m[i] * mx_scale_ld(nkb) + (k[i] >> 2)] = (uint8_t)sc;
        }
      }
    }
    __syncthreads();
  }

  v4f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const uint8_t* ring = smem + wave * D * CF::SLOT;
  const int left = (int)(p.KB & 7);
  for (int kb = wave, slot = 0; kb < nkb; kb += kSplitWaves) {
    // loads of the later K-blocks in flight behind this one's
    constexpr int PER = CF::LOADS + CF::S_LOADS;
    const int later = (nkb - 1 - kb) / kSplitWaves;
    if (D >= 4 && later >= 3) wait_vmcnt<PER * (D >= 4 ? 3 : 0)>();
    else if (D >= 3 && later >= 2) wait_vmcnt<PER * (D >= 3 ? 2 : 0)>();
    else if (D >= 2 && later >= 1) wait_vmcnt<PER * (D >= 2 ? 1 : 0)>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    const uint8_t* at = ring + slot * CF::SLOT;
    const uint8_t* bt = at + CF::AROWS * BK;
    const uint8_t* st = at + CF::ROWS * BK;
    // the scale bytes of blocks that a short last K-block does not have may hold anything
    const uint64_t mask = left && kb == nkb - 1 ? (1ull << (8 * left)) - 1 : ~0ull;
    u32x4 fa[FM][2], fb[FN][2];
    uint64_t sa[FM], sb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      sb[j] = (*reinterpret_cast<const uint64_t*>(st + CF::AS_LOADS * 256 + (16 * j + fr) * 8) & mask) >> (8 * fg);
#pragma unroll
      for (int h = 0; h < 2; ++h) fb[j][h] = *reinterpret_cast<const u32x4*>(bt + swz(16 * j + fr, 4 * h + fg));
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = FUSED ? (fr < (int)p.M ? fr : 0) : 16 * i + fr;
      sa[i] = (*reinterpret_cast<const uint64_t*>(FUSED ? scales + r * mx_scale_ld(nkb) + kb * 8 : st + r * 8) & mask) >> (8 * fg);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        fa[i][h] = *reinterpret_cast<const u32x4*>(FUSED ? codes + r * mx_code_ld(nkb) + kb * BK + 64 * h + 16 * fg
                                                         : at + swz(r, 4 * h + fg));
    }
    // the slot is free once its fragments have arrived
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (kb + D * kSplitWaves < nkb) issue(kb + D * kSplitWaves, slot);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v8i b8 = {(int)fb[j][h][0], (int)fb[j][h][1], (int)fb[j][h][2], (int)fb[j][h][3], 0, 0, 0, 0};
          const v8i a8 = {(int)fa[i][h][0], (int)fa[i][h][1], (int)fa[i][h][2], (int)fa[i][h][3], 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, acc[i][j], 4, 4, 0, (int)(sb[j] >> (32 * h)), 0,
                                                                       (int)(sa[i] >> (32 * h)));
        }
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  __syncthreads();
  // the waves' sums, added in the order of the waves: sum[wave][subtile][lane]
  v4f* sum = reinterpret_cast<v4f*>(smem);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sum[(wave * FM * FN + i * FN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int q = threadIdx.x; q < FM * FN * 64; q += 64 * kSplitWaves) {
    const int l = q & 63, i = (q >> 6) / FN, j = (q >> 6) % FN;
    const int64_t row = t.m0 + 16 * i + (l & 15), col = t.n0 + 16 * j + 4 * (l >> 4);
    if (row >= t.m1 || col >= p.N) continue;
    v4f y = sum[q];
#pragma unroll
    for (int w = 1; w < kSplitWaves; ++w) y += sum[w * FM * FN * 64 + q];
    const uint32_t w2[2] = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    uint16_t* dst = p.C + row * p.ldc + col;
    if (col + 4 <= p.N) {
      *reinterpret_cast<u32x2u*>(dst) = u32x2u{w2[0], w2[1]};
    } else {
      for (int v = 0; v < 4 && col + v < p.N; ++v) dst[v] = (uint16_t)(w2[v >> 1] >> (16 * (v & 1)));
    }
  }
}

inline unsigned grid_of(uint32_t total, int units) {
  const uint64_t per = 256u * (uint64_t)units;
  uint64_t g = (total + per - 1) / per;
  const uint64_t most = (uint64_t)device_cu_count() * 64;
  return (unsigned)(g < most ? g : most);
}

// Rows whose 8-column chunks number less than 2^31 go in one launch.
template <class Args, class F>
hipError_t by_rows(Args a, int64_t per_row, F&& launch) {
  const int64_t most = ((int64_t)1 << 30) / per_row;
  const int64_t M = a.M;
  for (int64_t m = 0; m < M; m += most) {
    a.M = M - m < most ? M - m : most;
    launch(a, m, (uint32_t)(a.M * per_row));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_quant(const MxQuantArgs& args, hipStream_t stream) {
  const int64_t per_row = (args.K + kMx - 1) / kMx * 4;
  if (args.M == 0 || per_row == 0) return hipSuccess;
  return by_rows(args, per_row, [&](MxQuantArgs a, int64_t m, uint32_t total) {
    const FastDiv d = make_fastdiv((uint32_t)per_row);
    a.x = static_cast<const uint8_t*>(args.x) + m * args.ldx * (args.f32 ? 4 : 2);
    if (args.u) a.u = args.u + m * args.ldu;
    a.y = args.y + m * args.ldy;
    a.s = args.s + m * args.lds;
    const unsigned grid = grid_of(total, 2);
    if (args.u) hipLaunchKernelGGL((mx_quant_kernel<kGated, 2>), dim3(grid), dim3(256), 0, stream, a, d, total);
    else if (args.f32) hipLaunchKernelGGL((mx_quant_kernel<kF32, 2>), dim3(grid), dim3(256), 0, stream, a, d, total);
    else hipLaunchKernelGGL((mx_quant_kernel<kBf16, 2>), dim3(grid), dim3(256), 0, stream, a, d, total);
  });
}

hipError_t launch_mx_dequant(const MxDequantArgs& args, hipStream_t stream) {
  const int64_t per_row = (args.K + 7) / 8;
  if (args.M == 0 || per_row == 0) return hipSuccess;
  return by_rows(args, per_row, [&](MxDequantArgs a, int64_t m, uint32_t total) {
    const FastDiv d = make_fastdiv((uint32_t)per_row);
    a.q = args.q + m * args.ldq;
    a.s = args.s + m * args.lds;
    a.out = args.out + m * args.ldo;
    hipLaunchKernelGGL((mx_dequant_kernel<2>), dim3(grid_of(total, 2)), dim3(256), 0, stream, a, d, total);
  });
}

// The variants and the cost of a product in each, in us:
//   launch + rounds * (start + step * K-blocks) + traffic * MB
// with rounds of workgroups over the CUs, K-blocks of 256 columns that one wave
// walks (split: an eighth of them), and the MB that all tiles load (rows of both
// operands).  Fitted to 108 dense products of 1 to 4096 rows and 93 grouped ones of
// 0.3 to 1500 rows an expert, weights past the caches: taking the least is within
// 5.3% (grouped 2.8%) of the best of thirteen variants in the mean, 32% (19%) at
// most.  Grouped products take five of the seven.
struct MxCost {
  float launch, start, step, traffic;
};
struct MxVariant {
  int rows, columns, per_cu;  // tile, workgroups that share a CU
  bool split;
  MxCost dense, grouped;
};
constexpr MxCost kNever = {1e30f, 0.0f, 0.0f, 0.0f};
constexpr MxVariant kMxVariants[] = {
    {16, 16, 2, true, {1.899f, 0.838f, 0.430f, 0.0479f}, kNever},
    {16, 32, 3, true, {2.277f, 0.307f, 0.706f, 0.0642f}, {2.777f, 1.567f, 0.0f, 0.0690f}},
    {32, 32, 2, true, {2.125f, 0.598f, 0.911f, 0.0491f}, {2.877f, 1.822f, 0.0f, 0.0588f}},
    {64, 64, 2, false, {2.009f, 1.881f, 0.313f, 0.0382f}, kNever},
    {64, 128, 2, false, {1.935f, 1.786f, 0.467f, 0.0457f}, {5.626f, 0.817f, 0.262f, 0.0711f}},
    {128, 128, 2, false, {3.529f, 0.0f, 0.845f, 0.0327f}, {6.981f, 0.026f, 0.533f, 0.0530f}},
    {256, 256, 1, false, {5.583f, 0.0f, 1.745f, 0.0f}, {12.626f, 0.243f, 0.892f, 0.0492f}},
};

// Row tiles of a grouped product: a short one for every expert that may have
// rows, and the rest in whole ones; never fewer than there are.
static int64_t grouped_tiles(const MxGemmArgs& a, int rows) {
  const int64_t some = a.E < a.M ? a.E : a.M;
  return some + (a.M - some) / rows;
}

constexpr double kMaxSplitTiles = 1 << 22;  // a workgroup each: a launch holds fewer than 2^32 threads

static int mx_choose(const MxGemmArgs& a) {
  const bool grouped = a.offsets != nullptr;
  const int64_t kbs = (a.KB + 7) / 8;
  int best = 0;
  double least = 1e30;
  for (int v = 0; v < (int)(sizeof kMxVariants / sizeof *kMxVariants); ++v) {
    const MxVariant& m = kMxVariants[v];
    const MxCost& c = grouped ? m.grouped : m.dense;
    const double tiles = (double)(grouped ? grouped_tiles(a, m.rows) : (a.M + m.rows - 1) / m.rows) *
                         (double)((a.N + m.columns - 1) / m.columns);
    if (m.split && tiles > kMaxSplitTiles) continue;
    const double part = tiles / ((double)device_cu_count() * m.per_cu);
    const double rounds = grouped ? (part > 1 ? part : 1) : __builtin_ceil(part);
    const double deep = (double)(m.split ? (kbs + kSplitWaves - 1) / kSplitWaves : kbs);
    const double cost =
        c.launch + rounds * (c.start + c.step * deep) + c.traffic * tiles * (m.rows + m.columns) * (double)kbs * BK * 1e-6;
    if (cost < least) best = v, least = cost;
  }
  return best;
}

template <class CF>
static hipError_t launch_mx_tiles(const MxGemmArgs& a, hipStream_t stream) {
  const int64_t tiles_m = a.offsets ? grouped_tiles(a, CF::BM) : (a.M + CF::BM - 1) / CF::BM;
  const int64_t tiles = tiles_m * ((a.N + CF::BN - 1) / CF::BN), slots = (int64_t)device_cu_count() * CF::PER_CU;
  const dim3 grid((unsigned)(tiles < slots ? tiles : slots)), blk(CF::kThreads);
  if constexpr (CF::BN > 64) {
    if (a.offsets) {
      hipLaunchKernelGGL((mx_gemm_kernel<CF, true>), grid, blk, 0, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_gemm_kernel<CF, false>), grid, blk, 0, stream, a);
  return hipGetLastError();
}

template <int FM, int FN, int D, bool FUSED>
static hipError_t launch_mx_split(const MxGemmArgs& a, const MxQuantArgs& x, hipStream_t stream) {
  using CF = SplitCfg<FM, FN, D, FUSED>;
  const int64_t tiles_m = a.offsets ? grouped_tiles(a, CF::TM) : (FUSED ? 1 : (a.M + CF::TM - 1) / CF::TM);
  const dim3 grid((unsigned)(tiles_m * ((a.N + CF::TN - 1) / CF::TN))), blk(64 * kSplitWaves);
  if constexpr (FN > 1 && !FUSED) {
    if (a.offsets) {
      hipLaunchKernelGGL((mx_split_kernel<FM, FN, D, false, true>), grid, blk, 0, stream, a, x);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_split_kernel<FM, FN, D, FUSED, false>), grid, blk, 0, stream, a, x);
  return hipGetLastError();
}

MxTileSize mx_gemm_tile(const MxGemmArgs& a) {
  const MxVariant& v = kMxVariants[mx_choose(a)];
  return {v.rows, v.columns};
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const MxQuantArgs none{};
  switch (mx_choose(a)) {
    case 0: return launch_mx_split<1, 1, 2, false>(a, none, stream);
    case 1: return launch_mx_split<1, 2, 1, false>(a, none, stream);
    case 2: return launch_mx_split<2, 2, 1, false>(a, none, stream);
    case 3: return launch_mx_tiles<MxCfg<64, 64, 2, 2, 4>>(a, stream);
    case 4: return launch_mx_tiles<MxCfg<64, 128, 1, 4, 3>>(a, stream);
    case 5: return launch_mx_tiles<MxCfg<128, 128, 2, 2, 2>>(a, stream);
    default: return launch_mx_tiles<MxCfg<256, 256, 2, 4, 2>>(a, stream);
  }
}

// The quantisation costs every workgroup a pass over all rows, 16384 elements at a time.
// One launch takes 4.6 us against 6.1 in two for 1x1536x7168, 5.3 against 7.1 for
// 8x7168x2048, 17.4 against 19.2 for 3x18432x7168, 87 against 90 for 3x129280x7168.  The
// bounds on M and K do not weigh N, and with many rows and very many columns two
// launches are faster: 16x18432x1536 8.9 us against 11.0, 8x129280x2048 29 against 36.
bool linear_mx_fused(int64_t M, int64_t N, int64_t K) {
  const int64_t nkb = (K + 255) / 256;
  return M <= 16 && N <= 16 * (int64_t)kMaxSplitTiles && M * nkb * 256 <= 24576 && M * (mx_code_ld((int)nkb) + mx_scale_ld((int)nkb)) <= kFusedBytes;
}

// 16 columns a workgroup where those are one round over the CUs (1x1536x7168 5.4 us,
// with 32 6.9; 1x4096x7168 6.3 and 7.3), else 32, which quantise half as often
// (3x18432x7168 16.9 us, with 16 19.2; 1x18432x7168 15.6 and 15.3).
hipError_t launch_linear_mx_fused(const MxGemmArgs& g, const MxQuantArgs& q, hipStream_t stream) {
  if (g.N <= 16 * (int64_t)device_cu_count()) return launch_mx_split<1, 1, 2, true>(g, q, stream);
  return launch_mx_split<1, 2, 1, true>(g, q, stream);
}

}  // namespace dsfp8
