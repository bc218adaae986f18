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
#include "device.h"
#include "launch.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));  // an access at any address
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

// Columns k .. k + 7 of a row of K, zeros past it.
__device__ __forceinline__ void load8(const uint16_t* row, int k, int K, float (&v)[8]) {
  u32x4 r = {0u, 0u, 0u, 0u};
  if (k + 8 <= K) {
    r = *reinterpret_cast<const u32x4u*>(row + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) r[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(r[i]), v[2 * i + 1] = bf16_hi(r[i]);
}

__device__ __forceinline__ void load8(const float* row, int k, int K, float (&v)[8]) {
  u32x4 r[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (k + 8 <= K) {
    r[0] = *reinterpret_cast<const u32x4u*>(row + k);
    r[1] = *reinterpret_cast<const u32x4u*>(row + k + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) r[i >> 2][i & 3] = __float_as_uint(row[k + i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i >> 2][i & 3]);
}

__device__ __forceinline__ void load_weight(const void* w, bool f32, int k, int K, float (&v)[8]) {
  if (f32) load8(static_cast<const float*>(w), k, K, v);
  else load8(static_cast<const uint16_t*>(w), k, K, v);
}

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

// Sum over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ float sum_row(float v, float* red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if constexpr (TPR > 64) {
    __syncthreads();  // the area may hold the previous sum
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += red[w];
  }
  return v;
}

__device__ __forceinline__ float inverse_rms(float sum, const NormArgs& a) {
  return 1.0f / __fsqrt_rn(sum / (float)a.D + a.eps);
}

// TPR threads per row, NC chunks of 8 columns per thread.
template <int TPR, int NC>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_kernel(NormArgs a) {
  constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
  static_assert(RPB == 1 || TPR == 64, "rows of a workgroup do not share its barriers");
  __shared__ float red[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int D = (int)a.D;
  const int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (m >= a.T) return;
  float v[NC][8];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) load8(a.x + m * a.ldx, (t + c * TPR) * 8, D, v[c]);
  if (a.post_w) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[c][i], v[c][i], sum);
    const float r = inverse_rms(sum_row<TPR>(sum, red), a);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float w[8];
      load_weight(a.post_w, a.w_f32, (t + c * TPR) * 8, D, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r * w[i];
    }
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (t + c * TPR) * 8;
      float q[8];
      if (a.gate) {
        load8(a.gate + m * a.ldg, k, D, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= q[i];
      }
      load8(a.residual + m * a.ldr, k, D, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = __builtin_fmaf(a.scale, v[c][i], q[i]);
      store_bf16x8(a.h + m * a.ldh, k, D, v[c]);
    }
  }
  sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[c][i], v[c][i], sum);
  const float r = inverse_rms(sum_row<TPR>(sum, red), a);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = (t + c * TPR) * 8;
    float w[8];
    load_weight(a.w, a.w_f32, k, D, w);
    if (a.fmt == DSFP8_NORM_BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r * w[i];
      store_bf16x8(static_cast<uint16_t*>(a.y) + m * a.ldy, k, D, v[c]);
      continue;
    }
    if (a.fmt == DSFP8_NORM_MXFP4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * r * w[i];
      const uint32_t s = mx_scale(mx_quad_top(v[c]));
      if (k < (D + 31) / 32 * 32) {
        reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + m * a.ldy)[k >> 3] = mx_codes8(v[c], mx_scale_f32(s));
        if ((k & 31) == 0) static_cast<uint8_t*>(a.s)[m * a.s_rs + (k >> 5)] = (uint8_t)s;
      }
    } else {
      // From h on in 64 bits: h w is exact, 1 / rms is a factor of the scale and
      // cancels in the code, and what is left is rounded to fp32 on its way to e4m3,
      // which puts a value halfway between two codes exactly there again.  So a code is
      // that of the exact y wherever h is exact (in 32 bits 5 in 10^6 codes, all halfway
      // cases, go by chance; 8192x7168 101 us against 104).  The maximum is over
      // bit patterns, in which NaN > infinity > every finite value, so that a block
      // that holds one gets a scale that shows it.
      double hw[8];
      uint64_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hw[i] = (double)v[c][i] * (double)w[i];
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
    hipLaunchKernelGGL((norm_kernel<TPR, NC>), dim3((unsigned)((b.T + RPB - 1) / RPB)), dim3(TPR > 256 ? TPR : 256), 0,
                       stream, b);
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
  if (a.D <= 4096) return launch_norm_of<256, 2>(a, stream);
  if (a.D <= 8192) return launch_norm_of<256, 4>(a, stream);
  if (a.D <= 16384) return launch_norm_of<512, 4>(a, stream);
  if (a.D <= 32768) return launch_norm_of<1024, 4>(a, stream);
  return launch_norm_of<1024, 8>(a, stream);
}

}  // namespace dsfp8
