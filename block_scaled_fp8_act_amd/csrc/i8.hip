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
#include "device.h"
#include "launch.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr float kAmaxFloor = 0x1p-100f;  // 127 / a and a / 127 stay normal

// ---- row quantisation ----------------------------------------------------------------

// Input element k of row m as fp32.
struct RowSrc {
  const RowQuantArgs& a;
  int64_t m;
  __device__ __forceinline__ float operator()(int64_t k) const {
    if (a.f32) return static_cast<const float*>(a.x)[m * a.ldx + k];
    const float g = bf16_lo(static_cast<const uint16_t*>(a.x)[m * a.ldx + k]);
    if (a.u == nullptr) return g;
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * bf16_lo(a.u[m * a.ldu + k]);
  }
};

__global__ __launch_bounds__(256) void row_quant_kernel(RowQuantArgs a) {
  __shared__ uint32_t red[256];
  const RowSrc x{a, (int64_t)blockIdx.x};
  uint32_t top = __float_as_uint(kAmaxFloor);
  for (int64_t k = threadIdx.x; k < a.K; k += 256) {
    const uint32_t b = __float_as_uint(x(k)) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  red[threadIdx.x] = top;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if ((int)threadIdx.x < d && red[threadIdx.x + d] > red[threadIdx.x]) red[threadIdx.x] = red[threadIdx.x + d];
    __syncthreads();
  }
  const float amax = __uint_as_float(red[0]);
  const float inv = 127.0f / amax;
  // Adding 1.5 * 2^23 rounds to an integer (nearest even) and leaves it in
  // the low bits as two's complement.
  for (int64_t k = threadIdx.x; k < a.K; k += 256)
    a.y[x.m * a.ldy + k] = (int8_t)__float_as_uint(x(k) * inv + 0x1.8p23f);
  if (threadIdx.x == 0) a.s[x.m] = amax / 127.0f;
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

hipError_t launch_row_quant_i8(const RowQuantArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  hipLaunchKernelGGL(row_quant_kernel, dim3((unsigned)a.M), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64));
  hipLaunchKernelGGL(gemm_i8_any_kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dsfp8
