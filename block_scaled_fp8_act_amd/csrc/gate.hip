// Choice of a token's experts from its router logits on gfx950.
//
// A wavefront per token; lane l holds VPT consecutive experts from l * VPT, so
// that among equal keys the lowest lane, and in it the first, is the lowest
// expert.  The scores are evaluated in 64 bits and rounded once, so that the
// choice does not depend on how an exponential is computed: an expert's key is
// the same fp32 value wherever it is evaluated.  Keys are compared as unsigned
// integers of the same order, 0 for an expert that is not available.  The
// maximum over the wave is six DPP steps, and each of the k rounds takes the first
// lane that holds it.
#include "device.h"
#include "launch.h"

namespace dsfp8 {
namespace {

constexpr int kGateWaves = 4;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

// Maximum over the wavefront, as a scalar.  Lanes without a source get 0, the least.
__device__ __forceinline__ uint32_t max_u32_wave(uint32_t v) {
  auto up = [&](uint32_t o) __attribute__((always_inline)) { v = o > v ? o : v; };
  up(dpp_u32<0x111>(v));  // row_shr 1
  up(dpp_u32<0x112>(v));  // row_shr 2
  up(dpp_u32<0x114>(v));  // row_shr 4
  up(dpp_u32<0x118>(v));  // row_shr 8
  up(dpp_u32<0x142>(v));  // row_bcast 15
  up(dpp_u32<0x143>(v));  // row_bcast 31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Unsigned integer in the order of the fp32 value (-0 and +0 alike); 0 for -inf.
__device__ __forceinline__ uint32_t order_u32(float key) {
  const uint32_t b = __float_as_uint(key + 0.0f);
  return key == -__builtin_inff() ? 0u : ((b >> 31) ? ~b : b | 0x80000000u);
}

template <int VPT, bool SOFTMAX>
__global__ __launch_bounds__(64 * kGateWaves) void gate_kernel(GateArgs a, FastDiv per_group) {
  __shared__ float keys[kGateWaves][64 * VPT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = (int64_t)blockIdx.x * kGateWaves + wave;
  if (t >= a.T) return;
  const float kNone = -__builtin_inff();
  float l[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane * VPT + j;
    l[j] = kNone;
    if (e < a.E)
      l[j] = a.bf16_in ? bf16_lo(static_cast<const uint16_t*>(a.logits)[t * a.ldl + e])
                       : static_cast<const float*>(a.logits)[t * a.ldl + e];
  }
  // scores, rounded once to fp32; 0 for an expert whose logit is -inf
  float score[VPT];
  bool bad = false;
  if constexpr (SOFTMAX) {
    float m = kNone;
#pragma unroll
    for (int j = 0; j < VPT; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    double p[VPT], sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      p[j] = l[j] == kNone ? 0.0 : exp((double)l[j] - (double)m);
      sum += p[j];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
#pragma unroll
    for (int j = 0; j < VPT; ++j) score[j] = l[j] == kNone ? 0.0f : (float)(p[j] / sum);
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) score[j] = l[j] == kNone ? 0.0f : (float)(1.0 / (1.0 + exp(-(double)l[j])));
  }
  uint32_t u[VPT];
  float key[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane * VPT + j;
    key[j] = score[j];
    if (a.bias && e < a.E) key[j] += a.bias[e];
    if (l[j] == kNone) key[j] = kNone;
    bad |= key[j] != key[j];
    u[j] = key[j] != key[j] ? 1u : order_u32(key[j]);  // NaN: available, after every number
  }
  if (a.groups > 1) {
    // Group g's score on lane g, from the keys in LDS; a group stays if fewer
    // than top_groups come before it.
#pragma unroll
    for (int j = 0; j < VPT; ++j) keys[wave][lane * VPT + j] = key[j];
    __builtin_amdgcn_wave_barrier();
    float t1 = kNone, t2 = kNone;
    const int gs = (int)per_group.d;
    if (lane < a.groups) {
      for (int i = 0; i < gs; ++i) {
        const float v = keys[wave][lane * gs + i];
        t2 = v > t1 ? t1 : (v > t2 ? v : t2);
        t1 = v > t1 ? v : t1;
      }
    }
    const float gsc = a.bias && t2 != kNone ? t1 + t2 : t1;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(gsc), g));
      ahead += o > gsc || (o == gsc && g < lane);
    }
    const uint64_t keep = __ballot(lane < a.groups && ahead < a.top_groups);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const uint32_t g = fastdiv((uint32_t)(lane * VPT + j), per_group);
      if (g < 64 && !(keep >> g & 1)) u[j] = 0;
    }
  }
  bad = __ballot(bad) != 0;

  float sum = 0.0f, w = 0.0f;
  int idx = -1;
  for (int i = 0; i < a.k; ++i) {
    uint32_t bu = u[0];
    int bj = 0;
    float bs = score[0];
#pragma unroll
    for (int j = 1; j < VPT; ++j)
      if (u[j] > bu) bu = u[j], bj = j, bs = score[j];
    const uint32_t top = max_u32_wave(bu);
    if (top == 0) break;  // no expert left
    const int from = __ffsll((unsigned long long)__ballot(bu == top)) - 1;
    const int e = __builtin_amdgcn_readlane(lane * VPT + bj, from);
    const float s = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(bs), from));
    sum += s;
    if (lane == i) idx = e, w = s;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (lane == from && j == bj) u[j] = 0;
  }
  if (lane < a.k) {
    if (a.renormalize) w = sum > 0.0f ? w / sum : 0.0f;
    w *= a.scale;
    if (bad) w = __uint_as_float(0x7fc00000u);
    a.indices[t * a.ldi + lane] = idx;
    a.weights[t * a.ldw + lane] = (uint16_t)pack_bf16x2(w, 0.0f);
  }
}

template <int VPT>
hipError_t launch_gate_of(const GateArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kGateWaves - 1) / kGateWaves)), blk(64 * kGateWaves);
  const FastDiv d = make_fastdiv((uint32_t)(a.E / a.groups));
  if (a.softmax) hipLaunchKernelGGL((gate_kernel<VPT, true>), grid, blk, 0, stream, a, d);
  else hipLaunchKernelGGL((gate_kernel<VPT, false>), grid, blk, 0, stream, a, d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.E <= 64) return launch_gate_of<1>(a, stream);
  if (a.E <= 128) return launch_gate_of<2>(a, stream);
  if (a.E <= 256) return launch_gate_of<4>(a, stream);
  if (a.E <= 512) return launch_gate_of<8>(a, stream);
  if (a.E <= 1024) return launch_gate_of<16>(a, stream);
  return launch_gate_of<64>(a, stream);
}

}  // namespace dsfp8
