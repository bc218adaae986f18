// A whole routed-expert layer for a few tokens on gfx950, in two kernels
// ("DeepSeek-V3 Administrator & Developer Guide", sections 6.4 and 8.4 with the
// expert of 1.2): for token t and slot j with expert e = indices[t, j],
//   h = SiLU(W1[e] x[t]) * (W3[e] x[t]),   out[t] = sum_j weights[t, j] W2[e] h.
//
// With a few tokens every expert that is hit has a few rows, so the layer is
// bound by the bytes of the experts' weights, 3 D F each, read once.  The
// products therefore run with the weights as the matrix instruction's first
// operand, straight from memory to registers (no weight is used twice by a
// workgroup, so LDS would only add a trip), converted to bf16, which holds
// every e4m3 and int8 value exactly, and with up to 16 tokens as the columns
// of its second operand.  Activations stay bf16; h is carried as the sum of two
// bf16 values (16 significant bits), since the matrix cores are far from
// busy and a second product per weight costs nothing that shows.
//
//   up    one workgroup per (leader pair, 32 columns of h).  The leader of an
//         expert is its first (token, slot) pair; workgroups of other pairs
//         end at once, so no list of experts has to be made first and no host
//         synchronisation is needed.  The eight waves split D and join through
//         LDS in a fixed order.
//   down  one workgroup per 16 columns of the output; its waves take the
//         (leader, piece of F) units in turn and add into an accumulator each,
//         joined at the end in a fixed order.
//
// The second kernel reads from the workspace, for each leader pair, the number
// of its tokens (0 for any other pair) and for each of them its row of h, the
// token and the sum of the token's weights for the expert.
#include <type_traits>

#include "device.h"
#include "launch.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kUpRows = 32;    // columns of h per workgroup (rows of w1, and as many of w3)
constexpr int kDownRows = 16;  // output columns per workgroup

struct TokenRef {
  int32_t row_tok;  // row of h (the pair index) * 64 + token
  float w;          // the token's weight for this expert
};

// Workspace: counts int32 [P] (padded to 16 bytes), refs TokenRef [P, T],
// h as hi bf16 [P, Fp] then lo bf16 [P, Fp], Fp = F rounded up to 128.
struct Work {
  int32_t* count;
  TokenRef* ref;
  uint16_t* hi;
  uint16_t* lo;
  int64_t Fp;
};

__host__ __device__ inline int64_t pad128(int64_t n) { return (n + 127) / 128 * 128; }

__host__ __device__ inline int64_t ref_offset(int64_t P) { return (P * 4 + 15) / 16 * 16; }
__host__ __device__ inline int64_t h_offset(int64_t P, int64_t T) {
  return ref_offset(P) + (P * T * (int64_t)sizeof(TokenRef) + 15) / 16 * 16;
}

__device__ __forceinline__ Work work_of(const MoeFewArgs& a) {
  const int64_t P = (int64_t)a.T * a.k;
  uint8_t* b = static_cast<uint8_t*>(a.work);
  Work w;
  w.Fp = pad128(a.F);
  w.count = reinterpret_cast<int32_t*>(b);
  w.ref = reinterpret_cast<TokenRef*>(b + ref_offset(P));
  w.hi = reinterpret_cast<uint16_t*>(b + h_offset(P, a.T));
  w.lo = w.hi + P * w.Fp;
  return w;
}

// 16 bytes from element k (of SZ bytes) of a row of K elements; elements past
// the row are zero.  TAIL = false promises that all of them lie in the row.
template <int SZ, bool TAIL>
__device__ __forceinline__ u32x4 load16(const uint8_t* row, int64_t k, int64_t K) {
  constexpr int n = 16 / SZ;
  if (!TAIL || k + n <= K) return *reinterpret_cast<const u32x4u*>(row + k * SZ);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < n; ++i) {
    if (k + i >= K) continue;
    const uint32_t v = SZ == 1 ? (uint32_t)row[k + i] : (uint32_t) reinterpret_cast<const uint16_t*>(row)[k + i];
    w[i * SZ / 4] |= v << (8 * (i * SZ % 4));
  }
  return u32x4{w[0], w[1], w[2], w[3]};
}

// Eight stored weights as bf16 (exact for both formats).
template <bool I8>
__device__ __forceinline__ bf16x8 widen(uint32_t a, uint32_t b) {
  u32x4 r;
  if constexpr (I8) {
    auto two = [](uint32_t w, int sh) {
      const uint32_t f0 = __float_as_uint((float)(int8_t)(w >> sh));
      const uint32_t f1 = __float_as_uint((float)(int8_t)(w >> (sh + 8)));
      return __builtin_amdgcn_perm(f1, f0, 0x07060302u);
    };
    r = u32x4{two(a, 0), two(a, 16), two(b, 0), two(b, 16)};
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true));
  }
  return __builtin_bit_cast(bf16x8, r);
}

// The 16x16 product of 128 elements: lane (r, g) = (lane % 16, lane / 16) holds
// elements 32g .. 32g+31 of weight row r (w) and of column r's activations (b);
// both operands take the elements in the same order, so the order in which
// the instruction consumes them does not matter.  Result: row 4g + v, column r.
template <bool I8>
__device__ __forceinline__ v4f block_product(const u32x4 (&w)[2], const u32x4 (&b)[4], v4f acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<I8>(w[s >> 1][2 * (s & 1)], w[s >> 1][2 * (s & 1) + 1]),
                                                  __builtin_bit_cast(bf16x8, b[s]), acc, 0, 0, 0);
  return acc;
}

template <bool I8, int CT>
__global__ __launch_bounds__(kThreads) void moe_few_up_kernel(MoeFewArgs a) {
  __shared__ float red[kWaves][2 * kUpRows][17];
  __shared__ int tok[kMoeFewTokens], pair[kMoeFewTokens];
  const Work wk = work_of(a);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int p0 = blockIdx.y;
  const int e = __builtin_amdgcn_readfirstlane(a.indices[(int64_t)(p0 / a.k) * a.ldi + p0 % a.k]);
  // This expert's tokens: lane t looks through token t's slots.
  int first = -1;
  float wsum = 0.0f;
  if (lane < a.T)
    for (int j = 0; j < a.k; ++j)
      if (a.indices[(int64_t)lane * a.ldi + j] == e) {
        if (first < 0) first = j;
        wsum += bf16_lo(a.weights[(int64_t)lane * a.ldwt + j]);
      }
  const uint64_t mask = __ballot(first >= 0);
  const int lead = __builtin_ctzll(mask);
  const bool mine = e >= 0 && e < a.E && lead * a.k + __shfl(first, lead) == p0;
  const int n = mine ? __popcll(mask) : 0;
  if (wave == 0) {
    const int c = __popcll(mask & ((1ull << lane) - 1));
    if (mine && first >= 0) {
      tok[c] = lane;
      pair[c] = lane * a.k + first;
      if (blockIdx.x == 0) wk.ref[(int64_t)p0 * a.T + c] = TokenRef{pair[c] * 64 + lane, wsum};
    }
    if (blockIdx.x == 0 && lane == 0) wk.count[p0] = n;
  }
  if (n == 0) return;
  __syncthreads();

  const int fr = lane & 15, fg = lane >> 4;
  const int64_t f0 = (int64_t)blockIdx.x * kUpRows;
  const int nct = (n + 15) >> 4;
  const int nkb = (int)((a.D + 127) >> 7);
  const uint8_t* we = a.w13 + (int64_t)e * 2 * a.F * a.ldw13;
  // Row tile i (0, 1: w1; 2, 3: w3); rows past F read row 0 and are not stored.
  const uint8_t* row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t f = f0 + 16 * (i & 1) + fr;
    row[i] = we + (f < a.F ? (i >> 1) * a.F + f : 0) * a.ldw13;
  }
  const uint8_t* xr[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
    xr[c] = reinterpret_cast<const uint8_t*>(a.x + (int64_t)(16 * c + fr < n ? tok[16 * c + fr] : 0) * a.ldx);
  v4f acc[4][CT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[i][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t kbn = (2 * a.F + 127) >> 7;
  const float* se = I8 ? nullptr : a.s13 + (int64_t)e * kbn * a.lds13;

  auto block = [&](int kb, auto tail) __attribute__((always_inline)) {
    constexpr bool TAIL = decltype(tail)::value;
    const int64_t k = (int64_t)kb * 128 + 32 * fg;
    u32x4 w[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[i][h] = load16<1, TAIL>(row[i], k + 16 * h, a.D);
    // the scale of each of a lane's four result rows: a 128-row block may
    // begin inside the w3 rows when F is no multiple of 128
    v4f sc[4];
    if constexpr (!I8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          int64_t r = f0 + 16 * (i & 1) + 4 * fg + v;
          r = (i >> 1) * a.F + (r < a.F ? r : a.F - 1);
          sc[i][v] = se[(r >> 7) * a.lds13 + kb];
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (c >= nct) continue;
      u32x4 b[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        b[s] = 16 * c + fr < n ? load16<2, TAIL>(xr[c], k + 8 * s, a.D) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (I8) {
          acc[i][c] = block_product<I8>(w[i], b, acc[i][c]);
        } else {
          const v4f part = block_product<I8>(w[i], b, v4f{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][c][v] = __builtin_fmaf(part[v], sc[i][v], acc[i][c][v]);
        }
      }
    }
  };
  for (int kb = wave; kb < nkb; kb += kWaves) {
    if ((int64_t)(kb + 1) * 128 <= a.D) block(kb, std::false_type{});
    else block(kb, std::true_type{});
  }

  // Join the waves' sums, gate, and write h.
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    if (c >= nct) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][16 * i + 4 * fg + v][fr] = acc[i][c][v];
    __syncthreads();
    const int r = threadIdx.x & 31, col = threadIdx.x >> 5;
    if (16 * c + col >= n) continue;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      g += red[w][r][col];
      u += red[w][kUpRows + r][col];
    }
    const int64_t f = f0 + r;
    float h = 0.0f;
    if (f < a.F) {
      if constexpr (I8) {
        const float* sr = a.s13 + (int64_t)e * a.lds13;
        g *= sr[f];
        u *= sr[a.F + f];
      }
      h = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
    }
    const float hi = bf16_lo(pack_bf16x2(h, 0.0f));
    // an infinite or NaN h stays so in hi alone
    const float lo = fabsf(hi) < __builtin_inff() ? h - hi : 0.0f;
    const int64_t at = (int64_t)pair[16 * c + col] * wk.Fp + f;
    wk.hi[at] = (uint16_t)pack_bf16x2(hi, 0.0f);
    wk.lo[at] = (uint16_t)pack_bf16x2(lo, 0.0f);
  }
}

template <bool I8, int CT>
__global__ __launch_bounds__(kThreads) void moe_few_down_kernel(MoeFewArgs a) {
  __shared__ float sum[kWaves][16 * CT][kDownRows + 4];
  __shared__ int list[kMoeFewTokens * 16];
  __shared__ int wave_n[kWaves];
  const Work wk = work_of(a);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int P = a.F > 0 ? a.T * a.k : 0;  // F = 0: the up kernel did not run, the output is zero
  for (int i = lane; i < 16 * CT * (kDownRows + 4); i += 64) (&sum[wave][0][0])[i] = 0.0f;
  // The leaders, in pair order.
  int total = 0;
  for (int base = 0; base < P; base += kThreads) {
    const int p = base + threadIdx.x;
    const bool is = p < P && wk.count[p] > 0;
    const uint64_t m = __ballot(is);
    if (lane == 0) wave_n[wave] = __popcll(m);
    __syncthreads();
    int at = total;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) at += wave_n[w];
      total += wave_n[w];
    }
    if (is) list[at + __popcll(m & ((1ull << lane) - 1))] = p;
    __syncthreads();
  }

  const int fr = lane & 15, fg = lane >> 4;
  const int64_t d0 = (int64_t)blockIdx.x * kDownRows;
  const int nkb = (int)(wk.Fp >> 7);
  const int64_t kbd = (a.D + 127) >> 7;
  // With fewer leaders than waves an expert's F is cut into pieces.
  const int pieces = total > 0 && total < kWaves ? (kWaves + total - 1) / total : 1;
  for (int unit = wave; unit < total * pieces; unit += kWaves) {
    const int p0 = __builtin_amdgcn_readfirstlane(list[unit / pieces]);
    const int piece = unit % pieces;
    const int e = __builtin_amdgcn_readfirstlane(a.indices[(int64_t)(p0 / a.k) * a.ldi + p0 % a.k]);
    const int n = __builtin_amdgcn_readfirstlane(wk.count[p0]);
    const int64_t d = d0 + fr;
    const uint8_t* row = a.w2 + ((int64_t)e * a.D + (d < a.D ? d : 0)) * a.ldw2;
    const float* se = I8 ? nullptr : a.s2 + ((int64_t)e * kbd + (d0 >> 7)) * a.lds2;
    const int b0 = nkb * piece / pieces, b1 = nkb * (piece + 1) / pieces;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (16 * c >= n) continue;
      const bool on = 16 * c + fr < n;
      const TokenRef ref = on ? wk.ref[(int64_t)p0 * a.T + 16 * c + fr] : TokenRef{0, 0.0f};
      const int64_t hrow = (int64_t)(ref.row_tok >> 6) * wk.Fp;
      v4f acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      for (int kb = b0; kb < b1; ++kb) {
        const int64_t k = (int64_t)kb * 128 + 32 * fg;
        u32x4 w[2], hh[4], hl[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = load16<1, true>(row, k + 16 * h, a.F);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          hh[s] = on ? *reinterpret_cast<const u32x4*>(wk.hi + hrow + k + 8 * s) : u32x4{0u, 0u, 0u, 0u};
          hl[s] = on ? *reinterpret_cast<const u32x4*>(wk.lo + hrow + k + 8 * s) : u32x4{0u, 0u, 0u, 0u};
        }
        if constexpr (I8) {
          acc = block_product<I8>(w, hl, block_product<I8>(w, hh, acc));
        } else {
          const v4f part = block_product<I8>(w, hl, block_product<I8>(w, hh, v4f{0.0f, 0.0f, 0.0f, 0.0f}));
          const float s = se[kb];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(part[v], s, acc[v]);
        }
      }
      if (!on) continue;
      // One lane of each row group per token: no two lanes share an address.
      float* dst = &sum[wave][ref.row_tok & 63][4 * fg];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float y = acc[v];
        if constexpr (I8) {
          const int64_t dv = d0 + 4 * fg + v;
          y *= a.s2[(int64_t)e * a.lds2 + (dv < a.D ? dv : a.D - 1)];
        }
        dst[v] = __builtin_fmaf(y, ref.w, dst[v]);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * kDownRows; i += kThreads) {
    const int t = i / kDownRows, r = i % kDownRows;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) y += sum[w][t][r];
    if (d0 + r < a.D) a.out[(int64_t)t * a.ldo + d0 + r] = (uint16_t)pack_bf16x2(y, 0.0f);
  }
}

template <bool I8, int CT>
hipError_t launch(const MoeFewArgs& a, hipStream_t stream) {
  if (a.F > 0) {
    const dim3 up((unsigned)(pad128(a.F) / kUpRows), (unsigned)(a.T * a.k));
    hipLaunchKernelGGL((moe_few_up_kernel<I8, CT>), up, dim3(kThreads), 0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const dim3 down((unsigned)((a.D + kDownRows - 1) / kDownRows));
  hipLaunchKernelGGL((moe_few_down_kernel<I8, CT>), down, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <bool I8>
hipError_t launch_ct(const MoeFewArgs& a, hipStream_t stream) {
  if (a.T <= 16) return launch<I8, 1>(a, stream);
  if (a.T <= 32) return launch<I8, 2>(a, stream);
  return launch<I8, 4>(a, stream);
}

}  // namespace

size_t moe_few_workspace_bytes(int64_t T, int64_t k, int64_t F) {
  return (size_t)(h_offset(T * k, T) + T * k * pad128(F) * 4);
}

hipError_t launch_moe_few(const MoeFewArgs& a, hipStream_t stream) {
  return a.i8 ? launch_ct<true>(a, stream) : launch_ct<false>(a, stream);
}

}  // namespace dsfp8
