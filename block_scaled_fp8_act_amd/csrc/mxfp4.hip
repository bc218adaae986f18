// MXFP4 linear layer on gfx950: rows in blocks of 32 columns, each block with
// one power-of-two scale (a byte, biased by 127) and 4-bit e2m1 codes (the
// OCP microscaling format), and products of such matrices.
//
// Quantisation of a block x of 32 columns:
//   e = max(floor(log2 max |x|) - 2, -127),  q = e2m1(x / 2^e),
// nearest-even, |q| <= 6; the scale byte is e + 127.  floor(log2) of an fp32
// value is its exponent field, so the scale byte is that field minus 2, and
// the division is part of the hardware's conversion, which rounds exactly
// (checked over every bf16 value and every scale).  A block that holds a NaN
// or an infinity has the field 255 and gets the scale byte 255, the format's
// NaN.
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
// v_mfma_scale_f32_32x32x64_f8f6f4.  A K-block is 128 bytes of a row, 256
// columns: four matrix instructions deep.  Lane (fr, fg) of an instruction
// holds 16 bytes, the 32 columns of one block of row fr, and that block's scale
// byte, which the instruction applies.  The operands go through the same ring of LDS
// stages as the other tiled products', filled by buffer_load ... lds and read
// without bank conflicts through the XOR swizzle.  The scale bytes of two K-blocks
// (16 bytes a row) are loaded together, one load per 64 rows, into a ring of
// two buffers behind the stages.

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
  static constexpr int S_BYTES = S_INSTR * NW * 1024;
  static constexpr int C_BYTES = 32 * WN * 2;  // 32 rows of a wave's output
  static constexpr int RING = STAGES * STAGE_BYTES + 2 * S_BYTES;
  static constexpr int LDS = RING > NW * C_BYTES ? RING : NW * C_BYTES;
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "whole 1 KB segments per wave");
  static_assert(WM % 32 == 0 && WN % 32 == 0 && BM % 64 == 0 && BN % 64 == 0, "32x32 subtiles, scale loads of 64 rows");
  static_assert(NW % 2 == 0, "a wave's segments start at rows that agree modulo 16");
  static_assert(STAGES == 2 || STAGES == 3, "the waits of the K loop");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <class CF>
struct MxLoader {
  i32x4 rsA, rsB, rsAS, rsBS;
  uint32_t off[CF::LOADS], soff[CF::S_INSTR];
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
    const int64_t m0 = p.rows ? 0 : t.m0, ha = p.rows ? p.a_rows : ra;
    rsA = make_rsrc(p.A + m0 * p.lda, (uint32_t)((ha - 1) * p.lda) + KR);
    rsB = make_rsrc(t.B + t.n0 * p.ldb, (uint32_t)((rb - 1) * p.ldb) + KR);
    rsAS = make_rsrc(p.a_s + m0 * p.ldas, (uint32_t)(ha * p.ldas));
    rsBS = make_rsrc(t.b_s + t.n0 * p.ldbs, (uint32_t)(rb * p.ldbs));
    auto a_row = [&](int64_t r) __attribute__((always_inline)) {
      if (!p.rows) return (uint32_t)r;
      const int32_t v = p.rows[t.m0 + r];
      return (uint32_t)(v < 0 ? 0 : (v < p.a_rows ? v : p.a_rows - 1));
    };
    kc = (uint32_t)((lane & 7) ^ swz_key(wave * 8 + (lane >> 3))) * 16;
#pragma unroll
    for (int n = 0; n < CF::LOADS; ++n) {
      const bool a = n < CF::A_INSTR;
      const int r = (wave + CF::NW * (a ? n : n - CF::A_INSTR)) * 8 + (lane >> 3);
      off[n] = kOob;
      if (r < (a ? ra : rb)) off[n] = (a ? a_row(r) * (uint32_t)p.lda : (uint32_t)(r * p.ldb)) + kc;
    }
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

  // Load n of K-block kb; the scales go with every other K-block.
  __device__ __forceinline__ void issue(int n, int kb, int stage) const {
    const bool a = n < CF::A_INSTR;
    const uint32_t kbyte = (uint32_t)kb * BK;
    const uint32_t at = lds0 + (uint32_t)(stage * CF::STAGE_BYTES + (a ? 0 : CF::A_BYTES) +
                                          (wave + CF::NW * (a ? n : n - CF::A_INSTR)) * 1024);
    dma_b128(a ? rsA : rsB, at, kbyte + kc < KR ? off[n] : kOob, kbyte);
  }
  __device__ __forceinline__ void issue_scales(int kb) const {
    if (kb & 1) return;
#pragma unroll
    for (int n = 0; n < CF::S_INSTR; ++n)
      dma_b128((wave + CF::NW * n) * 64 < CF::BM ? rsAS : rsBS,
               sds0 + (uint32_t)((kb >> 1 & 1) * CF::S_BYTES + CF::NW * n * 1024), soff[n], (uint32_t)(kb >> 1) * 16);
  }
};

// The scale bytes of a short last K-block's missing blocks may hold anything;
// their codes read as zero, but the scale byte 255 would make NaN of them.
template <class CF>
__device__ __forceinline__ void mx_clear_tail(uint8_t* smem, int kb, int blocks) {
  uint8_t* s = smem + CF::STAGES * CF::STAGE_BYTES + (kb >> 1 & 1) * CF::S_BYTES + 8 * (kb & 1);
  for (int r = threadIdx.x; r < CF::S_ROWS; r += CF::kThreads)
    *reinterpret_cast<uint64_t*>(s + r * 16) &= (1ull << (8 * blocks)) - 1;
  __syncthreads();
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

// One workgroup per tile (grouped: per CU, walking the tiles of every expert).
template <class CF, bool GROUPED>
__global__ __launch_bounds__(CF::kThreads) void mx_gemm_kernel(MxGemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[CF::LDS];
  const int64_t tiles_n = (p.N + CF::BN - 1) / CF::BN;
  const int nkb = (int)((p.KB + 7) / 8), tail = (int)(p.KB & 7);
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 31, fg = lane >> 5;
  const int wm = wave / CF::WAVES_N * CF::WM, wn = wave % CF::WAVES_N * CF::WN;
  int lf[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) lf[h] = fr * BK + (((2 * h + fg) ^ swz_key(fr)) << 4);
  for (int64_t pid = blockIdx.x;; pid += gridDim.x) {
    MxTile t;
    if constexpr (GROUPED) {
      const int64_t rt = div_u(pid, tiles_n);
      if (!mx_find<CF::BM>(p, rt, t)) break;
      t.n0 = (pid - rt * tiles_n) * CF::BN;
    } else {
      int64_t tm, tn;
      tile_of(pid, (p.M + CF::BM - 1) / CF::BM, tiles_n, tm, tn);
      t = MxTile{tm * CF::BM, p.M, tn * CF::BN, p.B, p.b_s};
    }
    MxLoader<CF> ld;
    ld.init(p, t, smem);
    for (int s = 0; s < CF::STAGES - 1 && s < nkb; ++s) {
#pragma unroll
      for (int n = 0; n < CF::LOADS; ++n) ld.issue(n, s, s);
      ld.issue_scales(s);
    }
    v16f acc[CF::TM][CF::TN];
#pragma unroll
    for (int i = 0; i < CF::TM; ++i)
#pragma unroll
      for (int j = 0; j < CF::TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    constexpr int PER = (CF::LOADS + 4 * CF::TM - 1) / (4 * CF::TM);
    for (int kb = 0; kb < nkb; ++kb) {
      // Of the stages issued so far, only the one behind K-block kb may be missing.
      if (CF::STAGES == 2 || kb + 1 >= nkb) wait_vmcnt<0>();
      else if (kb & 1) wait_vmcnt<CF::LOADS + CF::S_INSTR>();
      else wait_vmcnt<CF::LOADS>();
      __syncthreads();
      if (tail && kb == nkb - 1) mx_clear_tail<CF>(smem, kb, tail);
      const uint8_t* stage = smem + (kb % CF::STAGES) * CF::STAGE_BYTES;
      const uint8_t* sc = smem + CF::STAGES * CF::STAGE_BYTES + (kb >> 1 & 1) * CF::S_BYTES + 8 * (kb & 1);
      // Scale bytes of instruction h: byte 2h + fg of the row's eight.
      uint32_t sa[CF::TM][2], sb[CF::TN][2];
#pragma unroll
      for (int i = 0; i < CF::TM; ++i) {
        const uint2 w = *reinterpret_cast<const uint2*>(sc + (wm + 32 * i + fr) * 16);
        sa[i][0] = w.x >> (8 * fg), sa[i][1] = w.y >> (8 * fg);
      }
#pragma unroll
      for (int j = 0; j < CF::TN; ++j) {
        const uint2 w = *reinterpret_cast<const uint2*>(sc + (CF::BM + wn + 32 * j + fr) * 16);
        sb[j][0] = w.x >> (8 * fg), sb[j][1] = w.y >> (8 * fg);
      }
      const int kn = kb + CF::STAGES - 1;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        u32x4 fb[CF::TN];
#pragma unroll
        for (int j = 0; j < CF::TN; ++j)
          fb[j] = *reinterpret_cast<const u32x4*>(stage + CF::A_BYTES + (wn + 32 * j) * BK + lf[h]);
#pragma unroll
        for (int i = 0; i < CF::TM; ++i) {
          const u32x4 fa = *reinterpret_cast<const u32x4*>(stage + (wm + 32 * i) * BK + lf[h]);
          const v8i a8 = {(int)fa[0], (int)fa[1], (int)fa[2], (int)fa[3], 0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < CF::TN; ++j) {
            const v8i b8 = {(int)fb[j][0], (int)fb[j][1], (int)fb[j][2], (int)fb[j][3], 0, 0, 0, 0};
            // the weight first, so that a lane's results are runs of four columns of a row
            if (h & 1)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[i][j], 4, 4, 2, (int)sb[j][h >> 1],
                                                                          2, (int)sa[i][h >> 1]);
            else
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[i][j], 4, 4, 0, (int)sb[j][h >> 1],
                                                                          0, (int)sa[i][h >> 1]);
          }
          if (kn < nkb) {
            const int s = h * CF::TM + i;
#pragma unroll
            for (int n = s * PER; n < (s + 1) * PER && n < CF::LOADS; ++n) ld.issue(n, kn, kn % CF::STAGES);
            if (s == 4 * CF::TM - 1) ld.issue_scales(kn);
          }
        }
      }
    }
    __syncthreads();
    mx_store<CF>(p, t, acc, smem);
    if constexpr (!GROUPED) break;
    __syncthreads();
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

template <class CF>
static hipError_t launch_mx_tiles(const MxGemmArgs& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + CF::BN - 1) / CF::BN;
  if (a.offsets) {
    const int64_t some = a.E < a.M ? a.E : a.M;  // at most one short tile per expert that has rows
    const int64_t most = (some + (a.M - some) / CF::BM) * tiles_n, cus = device_cu_count();
    hipLaunchKernelGGL((mx_gemm_kernel<CF, true>), dim3((unsigned)(most < cus ? most : cus)), dim3(CF::kThreads), 0,
                       stream, a);
  } else {
    hipLaunchKernelGGL((mx_gemm_kernel<CF, false>), dim3((unsigned)((a.M + CF::BM - 1) / CF::BM * tiles_n)),
                       dim3(CF::kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int64_t t256 = (a.M + 255) / 256 * ((a.N + 255) / 256);
  if (t256 >= device_cu_count()) return launch_mx_tiles<MxCfg<256, 256, 2, 4, 2>>(a, stream);
  return launch_mx_tiles<MxCfg<64, 64, 2, 2, 2>>(a, stream);
}

bool linear_mx_fused(int64_t, int64_t, int64_t) { return false; }
hipError_t launch_linear_mx_fused(const MxGemmArgs&, const MxQuantArgs&, hipStream_t) { return hipErrorInvalidValue; }

}  // namespace dsfp8
