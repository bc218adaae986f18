// RMS norms around a residual connection on gfx950, with the quantisation of
// what follows:
//   t = x, or x / rms(x) * post_w    (rms(v) = sqrt(mean v^2 + eps))
//   h = residual + scale * gate * t
//   y = h / rms(h) * w
// in fp32; y is taken from h before h is rounded to bf16, and quantised
// without being rounded to bf16 in between.
//
// A row stays in registers between its two sums and its outputs, so every
// input is read once.  Lane l holds chunks of 8 columns, so that the 128
// columns of an e4m3 block lie in 16 lanes of a DPP row and the 32 of an MXFP4
// block in a quad.
//
// Bytes bound it: 8192x7168 with both norms and a gate 106 us, 5.5 TB/s; residual
// to e4m3 80-84 us, 4.9-5.2 TB/s, to MXFP4 71 us (a copy reaches 4.96).  32x7168 4.1 us:
// one trip to memory and one sum over the workgroup.  Rows that do not start at
// multiples of 16 bytes are read and written at their own addresses, 16 bytes a lane,
// which touch more lines: 8192x7167 with both norms and a gate 178 us, 3.3 TB/s.
#include "device.h"
#include "launch.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));  // an access at any address
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

// Columns k .. k + 7 of a row of K as loaded, zeros past it.
template <bool F32>
struct Eight {
  u32x4 r[F32 ? 2 : 1];

  __device__ __forceinline__ void load(const void* from, int k, int K) {
#pragma unroll
    for (auto& w : r) w = u32x4{0u, 0u, 0u, 0u};
    if constexpr (F32) {
      const uint32_t* row = static_cast<const uint32_t*>(from);
      if (k + 8 <= K) {
        r[0] = *reinterpret_cast<const u32x4u*>(row + k);
        r[1] = *reinterpret_cast<const u32x4u*>(row + k + 4);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < K) r[i >> 2][i & 3] = row[k + i];
      }
    } else {
      const uint16_t* row = static_cast<const uint16_t*>(from);
      if (k + 8 <= K) {
        r[0] = *reinterpret_cast<const u32x4u*>(row + k);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < K) r[0][i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (F32) return __uint_as_float(r[i >> 2][i & 3]);
    else return i & 1 ? bf16_hi(r[0][i >> 1]) : bf16_lo(r[0][i >> 1]);
  }
};

__device__ __forceinline__ void store_bf16x8(uint16_t* row, int k, int K, const float (&v)[8]) {
  const u32x4 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  if (k + 8 <= K) {
    *reinterpret_cast<u32x4u*>(row + k) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) row[k + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Sum over a wave, in every lane.
__device__ __forceinline__ float sum_wave(float v) {
  v += dpp_f32<0x111>(v);  // row_shr 1
  v += dpp_f32<0x112>(v);  // row_shr 2
  v += dpp_f32<0x114>(v);  // row_shr 4
  v += dpp_f32<0x118>(v);  // row_shr 8
  v += dpp_f32<0x142>(v);  // row_bcast 15
  v += dpp_f32<0x143>(v);  // row_bcast 31
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum of squares of a row, in every one of its threads: over a chunk, over the 512
// columns of a wave's chunks, and over those, so that the order does not depend
// on how many threads share the row.
template <int TPR, int NC>
__device__ __forceinline__ float sum_squares(const float (&v)[NC][8], float* red) {
  float s[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    s[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[c] = __builtin_fmaf(v[c][i], v[c][i], s[c]);
    s[c] = sum_wave(s[c]);
  }
  if constexpr (TPR == 64) {
    static_assert(NC == 1, "one wave, one sum");
    return s[0];
  } else {
    constexpr int WAVES = TPR / 64, N = NC * WAVES;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    __syncthreads();  // the area may hold the previous sum
    if (lane == 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) red[c * WAVES + wave] = s[c];
    }
    __syncthreads();
    float t = lane < N ? red[lane] : 0.0f;
    if constexpr (N > 64) t += lane + 64 < N ? red[lane + 64] : 0.0f;
    return sum_wave(t);
  }
}

__device__ __forceinline__ float inverse_rms(float sum, const NormArgs& a) {
  return 1.0f / __fsqrt_rn(sum / (float)a.D + a.eps);
}

// TPR threads per row, NC chunks of 8 columns per thread.  All operands are on
// their way before the first sum is waited for (32x7168 7.0 -> 4.1 us, 8192x7168 with both
// norms 129 -> 107, loads where they are used against this), as far as the
// registers of 1024 threads hold them.
template <int TPR, int NC, bool W_F32>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_kernel(NormArgs a) {
  constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
  static_assert(RPB == 1 || TPR == 64, "rows of a workgroup do not share its barriers");
  __shared__ float red[TPR > 64 ? NC * TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int D = (int)a.D;
  const int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (m >= a.T) return;
  constexpr bool EARLY = TPR * NC <= 4096, EARLY_W = EARLY && !(W_F32 && TPR * NC == 4096);
  Eight<false> x[NC], res[NC], gate[NC];
  Eight<W_F32> post[NC], w[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = (t + c * TPR) * 8;
    x[c].load(a.x + m * a.ldx, k, D);
    if (EARLY_W && a.post_w) post[c].load(a.post_w, k, D);
    if (EARLY && a.residual) res[c].load(a.residual + m * a.ldr, k, D);
    if (EARLY && a.gate) gate[c].load(a.gate + m * a.ldg, k, D);
    if (EARLY_W) w[c].load(a.w, k, D);
  }
  float v[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = x[c][i];
  if (a.post_w) {
    const float r = inverse_rms(sum_squares<TPR, NC>(v, red), a);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (!EARLY_W) post[c].load(a.post_w, (t + c * TPR) * 8, D);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r * post[c][i];
    }
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (t + c * TPR) * 8;
      if (a.gate) {
        if (!EARLY) gate[c].load(a.gate + m * a.ldg, k, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= gate[c][i];
      }
      if (!EARLY) res[c].load(a.residual + m * a.ldr, k, D);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = __builtin_fmaf(a.scale, v[c][i], res[c][i]);
      store_bf16x8(a.h + m * a.ldh, k, D, v[c]);
    }
  }
  const float r = inverse_rms(sum_squares<TPR, NC>(v, red), a);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = (t + c * TPR) * 8;
    if (!EARLY_W) w[c].load(a.w, k, D);
    if (a.fmt == DSFP8_NORM_BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r * w[c][i];
      store_bf16x8(static_cast<uint16_t*>(a.y) + m * a.ldy, k, D, v[c]);
      continue;
    }
    if (a.fmt == DSFP8_NORM_MXFP4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r * w[c][i];
      const uint32_t s = mx_scale(mx_quad_top(v[c]));
      if (k < (D + 31) / 32 * 32) {
        reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + m * a.ldy)[k >> 3] = mx_codes8(v[c], mx_scale_f32(s));
        if ((k & 31) == 0) static_cast<uint8_t*>(a.s)[m * a.s_rs + (k >> 5)] = (uint8_t)s;
      }
    } else {
      // From h on in 64 bits: h w is exact, 1 / rms is a factor of the scale and
      // cancels in the code, and what is left is rounded to fp32 on its way to e4m3,
      // which puts a value halfway between two codes exactly there again (its 64-bit
      // error is some 2^-50).  Where h and w have 8 significant bits each (no residual,
      // bf16 weights) nothing else gets there: with hw = a 2^i and the largest b 2^j, a
      // and b below 2^16, and a halfway point c of 5 bits, 448 hw / top and c differ by
      // 2^-21 or more, relative, or not at all, so the code is that of the exact y.  With
      // more bits a quotient within 2^-24 of a halfway point counts as one.  In 32 bits 5
      // in 10^6 codes, all halfway cases, go by chance (8192x7168 101 us against 104).
      // With a power-of-two scale, and where the clamp makes the scale, r does not cancel
      // and its error stays in the quotient.
      // The maximum is over bit patterns, in which NaN > infinity > every finite value, so
      // that a block that holds one gets a scale that shows it.
      double hw[8];
      uint64_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hw[i] = (double)v[c][i] * (double)w[c][i];
        const uint64_t b = (uint64_t)__double_as_longlong(hw[i]) & 0x7fffffffffffffffull;
        top = b > top ? b : top;
      }
      const uint32_t hi32 = max_row16_u32((uint32_t)(top >> 32));
      const uint32_t lo32 = max_row16_u32((uint32_t)(top >> 32) == hi32 ? (uint32_t)top : 0u);
      const double amax = __longlong_as_double((long long)((uint64_t)hi32 << 32 | lo32)) * (double)r;
      double scale = amax;
      if (amax == amax)
        scale = a.fmt == DSFP8_NORM_E4M3_UE8M0 ? (double)block_scale((float)amax, true)
                                               : fmax(amax, (double)kScaleFloor) * (1.0 / (double)kE4m3Max);
      const float s = (float)scale;
      const double inv = (double)r / scale;
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (float)(hw[i] * inv);
      const uint32_t lo = pack_e4m3x4(q[0], q[1], q[2], q[3]), hi = pack_e4m3x4(q[4], q[5], q[6], q[7]);
      uint8_t* dst = static_cast<uint8_t*>(a.y) + m * a.ldy + k;
      if (k + 8 <= D) {
        *reinterpret_cast<u32x2u*>(dst) = u32x2u{lo, hi};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < D) dst[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
      if ((k & 127) == 0 && k < D) static_cast<float*>(a.s)[m * a.s_rs + (int64_t)(k >> 7) * a.s_ks] = s;
    }
  }
}

template <int TPR, int NC>
hipError_t launch_norm_of(const NormArgs& a, hipStream_t stream) {
  constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
  // A launch holds fewer than 2^32 threads.  (A loop over rows in the kernel
  // instead: 8192x7168 with both norms 319 us against 130.)
  constexpr int64_t kMost = (int64_t)1 << 21;
  const int64_t ys = a.fmt == DSFP8_NORM_BF16 ? 2 : 1, ss = a.fmt == DSFP8_NORM_MXFP4 ? 1 : 4;
  for (int64_t m = 0; m < a.T; m += kMost) {
    NormArgs b = a;
    b.T = a.T - m < kMost ? a.T - m : kMost;
    b.x += m * a.ldx;
    if (a.residual) b.residual += m * a.ldr, b.h += m * a.ldh;
    if (a.gate) b.gate += m * a.ldg;
    b.y = static_cast<uint8_t*>(a.y) + m * a.ldy * ys;
    if (a.s) b.s = static_cast<uint8_t*>(a.s) + m * a.s_rs * ss;
    const dim3 grid((unsigned)((b.T + RPB - 1) / RPB)), blk(TPR > 256 ? TPR : 256);
    if (a.w_f32) hipLaunchKernelGGL((norm_kernel<TPR, NC, true>), grid, blk, 0, stream, b);
    else hipLaunchKernelGGL((norm_kernel<TPR, NC, false>), grid, blk, 0, stream, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.D == 0) return hipSuccess;
  if (a.D <= 512) return launch_norm_of<64, 1>(a, stream);
  if (a.D <= 2048) return launch_norm_of<256, 1>(a, stream);
  // Up to two rows a CU, four times the threads share a row: 32x7168 4.2 us against 7.0,
  // 512x7168 8.3 against 10.3; 1024x7168 14.7 in the narrow form, three rows a CU.
  const bool few = a.T <= 2 * (int64_t)device_cu_count();
  if (a.D <= 4096) return few ? launch_norm_of<512, 1>(a, stream) : launch_norm_of<256, 2>(a, stream);
  if (a.D <= 8192) return few ? launch_norm_of<1024, 1>(a, stream) : launch_norm_of<256, 4>(a, stream);
  if (a.D <= 16384) return few ? launch_norm_of<1024, 2>(a, stream) : launch_norm_of<512, 4>(a, stream);
  if (a.D <= 32768) return launch_norm_of<1024, 4>(a, stream);
  return launch_norm_of<1024, 8>(a, stream);
}

}  // namespace dsfp8
