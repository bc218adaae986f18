// Choice of a token's experts from its router logits on gfx950.
//
// LPT lanes per token, the whole wavefront or a quarter of it; each holds VPT
// consecutive experts, so that among equal keys the lowest lane, and in it the first,
// is the lowest expert.  The scores are evaluated in 64 bits (within 2^-45) and rounded
// once, so that the choice does not depend on how an exponential is computed: two
// evaluations give the same fp32 key but for one in 10^6 that lie next to a
// halfway case.  Keys are compared as unsigned
// integers of the same order, 0 for an expert that is not available.  Each of the k
// rounds takes the maximum over the token's lanes (DPP steps) and its first
// holder, which puts itself into the round's slot in LDS.
//
// 16384x256 in 8 groups: 18.2 us (softmax without groups 16.4), 1.0 TB/s; its
// instructions bound it, not its 17.6 MB: the last seven of eight rounds are 5.1 us, the
// scores 4.7 (the logits in their place), the groups 2.1 (one group), the rest 5.3.  One
// token: 4.3 to 4.8 us, a chain of dependent steps.
#include "device.h"
#include "launch.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));  // an access at any address
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

constexpr int kGateWaves = 4;
constexpr int kMaxGateK = 16, kMaxGateGroups = 64;
constexpr float kNone = -__builtin_inff();  // logit or key of an expert that is not available

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

// Maximum over a token's lanes, in every one of them.  Lanes without a source
// get 0, the least.
template <int LPT>
__device__ __forceinline__ uint32_t max_token(uint32_t v) {
  if constexpr (LPT == 16) return max_row16_u32(v);
  auto up = [&](uint32_t o) __attribute__((always_inline)) { v = o > v ? o : v; };
  up(dpp_u32<0x111>(v));  // row_shr 1
  up(dpp_u32<0x112>(v));  // row_shr 2
  up(dpp_u32<0x114>(v));  // row_shr 4
  up(dpp_u32<0x118>(v));  // row_shr 8
  up(dpp_u32<0x142>(v));  // row_bcast 15
  up(dpp_u32<0x143>(v));  // row_bcast 31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Unsigned integer, never 0, in the order of the fp32 value (-0 and +0 alike).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
// The same of a key; 0 for -inf.
__device__ __forceinline__ uint32_t order_u32(float key) { return key == kNone ? 0u : order_of(key); }

// A group's score from its two best keys, in order; 0 for a group without an
// expert, which comes after one whose two keys add up to -inf.
__device__ __forceinline__ uint32_t order_group(float t1, float t2, bool sum) {
  return t1 == kNone ? 0u : order_of(sum && t2 != kNone ? t1 + t2 : t1);
}

// 1 / v for finite v >= 1 in 64 bits, within a few units in the last place: the
// hardware's reciprocal and two Newton steps.
__device__ __forceinline__ double reciprocal(double v) {
  double r = __builtin_amdgcn_rcp(v);
  r = __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
}

// e^x for |x| <= 800 within 2^-46: x = n ln 2 + r with |r| <= ln 2 / 2, and the series of
// e^r up to r^11.  No branch, so that the chains of a lane's experts overlap (16384x256
// in groups 19.7 us with the library's exponential, which has branches, 17.8 with this).
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
  double r = __builtin_fma(n, -0x1.62e42fefa38p-1, x);     // ln 2 to 42 bits, n times it is exact
  r = __builtin_fma(n, -0x1.ef35793c7673p-45, r);          // and the rest of it
  constexpr double kSeries[] = {1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720,
                                1.0 / 120, 1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
  double p = kSeries[0];
#pragma unroll
  for (int i = 1; i < 12; ++i) p = __builtin_fma(p, r, kSeries[i]);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// The two largest of two pairs, each in order.
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
  const float lo = fminf(a1, b1);
  a1 = fmaxf(a1, b1);
  a2 = fmaxf(lo, fmaxf(a2, b2));
}

template <int VPT, int LPT, bool SOFTMAX>
__global__ __launch_bounds__(64 * kGateWaves) void gate_kernel(GateArgs a, FastDiv per_group) {
  constexpr int TPW = 64 / LPT;  // tokens of a wave
  __shared__ float keys[kGateWaves][TPW][LPT * VPT];
  __shared__ uint32_t group_score[kGateWaves][TPW][kMaxGateGroups];
  __shared__ float4 best2[kGateWaves][TPW][LPT];
  __shared__ int2 slots[kGateWaves][TPW][kMaxGateK];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int sub = (threadIdx.x & 63) / LPT, lane = threadIdx.x % LPT;  // token of the wave, lane of the token
  const int64_t at = ((int64_t)blockIdx.x * kGateWaves + wave) * TPW + sub;
  const int64_t t = at < a.T ? at : a.T - 1;  // a row past the last repeats it and stores nothing
  float l[VPT];
  const int e0 = lane * VPT;
#pragma unroll
  for (int j = 0; j < VPT; ++j) l[j] = kNone;
#pragma unroll
  for (int j = 0; j < VPT; j += 4) {
    const int64_t from = t * a.ldl + e0 + j;
    if (VPT >= 4 && e0 + j + 4 <= a.E) {
      if (a.bf16_in) {
        const u32x2u w = *reinterpret_cast<const u32x2u*>(static_cast<const uint16_t*>(a.logits) + from);
#pragma unroll
        for (int i = 0; i < 4 && j + i < VPT; ++i) l[j + i] = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
      } else {
        const u32x4u w = *reinterpret_cast<const u32x4u*>(static_cast<const float*>(a.logits) + from);
#pragma unroll
        for (int i = 0; i < 4 && j + i < VPT; ++i) l[j + i] = __uint_as_float(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 && j + i < VPT; ++i)
        if (e0 + j + i < a.E)
          l[j + i] = a.bf16_in ? bf16_lo(static_cast<const uint16_t*>(a.logits)[from + i])
                               : static_cast<const float*>(a.logits)[from + i];
    }
  }
  // keys, of scores rounded once to fp32 (0 for an expert whose logit is -inf)
  float key[VPT];
  bool bad = false;
  if constexpr (SOFTMAX) {
    float m = kNone;
#pragma unroll
    for (int j = 0; j < VPT; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    double p[VPT], sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const double d = (double)l[j] - (double)m, e = exp64(fmax(d, -800.0));  // e^-800 is 0 in fp32
      p[j] = l[j] == kNone ? 0.0 : (d != d ? d : e);
      sum += p[j];
    }
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) sum += __shfl_xor(sum, d);
    const double r = reciprocal(sum);  // the largest is 1, so the sum is, unless no expert is available
#pragma unroll
    for (int j = 0; j < VPT; ++j) key[j] = l[j] == kNone ? 0.0f : (float)(p[j] * r);
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      // past +-110 the score is 1 or, rounded to fp32, 0
      const float s = (float)reciprocal(1.0 + exp64((double)__builtin_amdgcn_fmed3f(-l[j], -110.0f, 110.0f)));
      key[j] = l[j] != l[j] ? l[j] : s;
    }
  }
  float score[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) score[j] = key[j];
  float b[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) b[j] = 0.0f;
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < VPT; j += 4) {
      if (VPT >= 4 && e0 + j + 4 <= a.E) {
        const u32x4u w = *reinterpret_cast<const u32x4u*>(a.bias + e0 + j);
#pragma unroll
        for (int i = 0; i < 4 && j + i < VPT; ++i) b[j + i] = __uint_as_float(w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4 && j + i < VPT; ++i)
          if (e0 + j + i < a.E) b[j + i] = a.bias[e0 + j + i];
      }
    }
  }
  uint32_t u[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (a.bias) key[j] += b[j];
    if (l[j] == kNone) key[j] = kNone;
    bad |= key[j] != key[j];
    u[j] = key[j] != key[j] ? 1u : order_u32(key[j]);  // NaN: available, after every number
  }
  if (a.groups > 1) {
    // A group's score, then its rank: a group stays if fewer than top_groups
    // come before it.
    if (__ballot(bad)) {
      // an expert whose key is NaN is available: in its group's score, the least number
#pragma unroll
      for (int j = 0; j < VPT; ++j) key[j] = key[j] != key[j] ? -0x1.fffffep127f : key[j];
    }
    const int gs = (int)per_group.d, gl = gs / VPT;
    uint32_t* gsc = group_score[wave][sub];
    const bool lanes = gs % VPT == 0;  // gl lanes hold a group
    // else, where gs > VPT, a lane's experts belong to group g0 and, from `border` on, the next
    // (16384x250 in 5 groups 18.3 us; one lane per group over all of its experts 39.5)
    const bool two = !lanes && gs > VPT;
    const int g0 = (int)fastdiv((uint32_t)e0, per_group), border = (g0 + 1) * gs;
    if (lanes && (gl & (gl - 1)) == 0) {
      float t1 = kNone, t2 = kNone;
#pragma unroll
      for (int j = 0; j < VPT; ++j) merge2(t1, t2, key[j], kNone);
      for (int d = 1; d < gl; d <<= 1) merge2(t1, t2, __shfl_xor(t1, d), __shfl_xor(t2, d));
      if (lane % gl == 0 && e0 < a.E) gsc[lane / gl] = order_group(t1, t2, a.bias != nullptr);
    } else if (lanes) {
      float t1 = kNone, t2 = kNone;
#pragma unroll
      for (int j = 0; j < VPT; ++j) merge2(t1, t2, key[j], kNone);
      best2[wave][sub][lane] = make_float4(t1, t2, kNone, kNone);
      __builtin_amdgcn_wave_barrier();
      for (int g = lane; g < a.groups; g += LPT) {
        t1 = t2 = kNone;
        for (int i = 0; i < gl; ++i) {
          const float4 o = best2[wave][sub][g * gl + i];
          merge2(t1, t2, o.x, o.y);
        }
        gsc[g] = order_group(t1, t2, a.bias != nullptr);
      }
    } else if (two) {
      float4 o = make_float4(kNone, kNone, kNone, kNone);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const bool next = e0 + j >= border;
        merge2(o.x, o.y, next ? kNone : key[j], kNone);
        merge2(o.z, o.w, next ? key[j] : kNone, kNone);
      }
      best2[wave][sub][lane] = o;
      __builtin_amdgcn_wave_barrier();
      for (int g = lane; g < a.groups; g += LPT) {
        const int first = g * gs / VPT, last = (g * gs + gs - 1) / VPT;
        o = best2[wave][sub][first];
        float t1 = first * VPT < g * gs ? o.z : o.x, t2 = first * VPT < g * gs ? o.w : o.y;
        for (int i = first + 1; i <= last; ++i) {
          o = best2[wave][sub][i];
          merge2(t1, t2, o.x, o.y);
        }
        gsc[g] = order_group(t1, t2, a.bias != nullptr);
      }
    } else {
      // fewer experts in a group than a lane holds: their keys through LDS
#pragma unroll
      for (int j = 0; j < VPT; ++j) keys[wave][sub][e0 + j] = key[j];
      __builtin_amdgcn_wave_barrier();
      for (int g = lane; g < a.groups; g += LPT) {
        float t1 = kNone, t2 = kNone;
        for (int i = 0; i < gs; ++i) merge2(t1, t2, keys[wave][sub][g * gs + i], kNone);
        gsc[g] = order_group(t1, t2, a.bias != nullptr);
      }
    }
    __builtin_amdgcn_wave_barrier();
    uint64_t keep = 0;
    for (int base = 0; base < a.groups; base += LPT) {
      const int mine = base + lane;
      const uint32_t v = mine < a.groups ? gsc[mine] : 0u;
      int ahead = 0;
      for (int g = 0; g < a.groups; ++g) {
        const uint32_t o = gsc[g];
        ahead += o > v || (o == v && g < mine);
      }
      const uint64_t stay = __ballot(mine < a.groups && ahead < a.top_groups) >> (LPT * sub);
      keep |= (LPT == 64 ? stay : stay & 0xffffu) << base;
    }
    if (lanes) {
      const bool out = e0 < a.E && !(keep >> (lane / gl) & 1);
#pragma unroll
      for (int j = 0; j < VPT; ++j) u[j] = out ? 0u : u[j];
    } else if (two) {
      // a lane past the last expert holds none, whatever it reads here
      const bool out0 = !(keep >> (g0 & 63) & 1), out1 = !(keep >> (g0 + 1 & 63) & 1);
#pragma unroll
      for (int j = 0; j < VPT; ++j) u[j] = (e0 + j >= border ? out1 : out0) ? 0u : u[j];
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const uint32_t g = fastdiv((uint32_t)(e0 + j), per_group);
        if (g < 64 && !(keep >> g & 1)) u[j] = 0;
      }
    }
  }
  {
    const uint64_t b = __ballot(bad) >> (LPT * sub);
    bad = (LPT == 64 ? b : b & 0xffffu) != 0;
  }

  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < VPT; ++j) keys[wave][sub][e0 + j] = score[j];  // for the weights
  int2* slot = slots[wave][sub];
  if (lane < kMaxGateK) slot[lane] = make_int2(-1, 0);
  __builtin_amdgcn_wave_barrier();
  for (int i = 0; i < a.k; ++i) {
    uint32_t best = u[0];
#pragma unroll
    for (int j = 1; j < VPT; ++j) best = u[j] > best ? u[j] : best;
    const uint32_t top = max_token<LPT>(best);
    const uint64_t have = __ballot(best == top && top != 0) >> (LPT * sub);
    const int from = __ffsll((unsigned long long)(LPT == 64 ? have : have & 0xffffu)) - 1;  // -1: no expert left
    if (lane == from) {
      int first = 0;
#pragma unroll
      for (int j = VPT - 1; j >= 0; --j) first = u[j] == best ? j : first;
#pragma unroll
      for (int j = 0; j < VPT; ++j) u[j] = j == first ? 0u : u[j];
      slot[i] = make_int2(e0 + first, __float_as_int(keys[wave][sub][e0 + first]));
    }
  }
  __builtin_amdgcn_wave_barrier();
  // Slot i on lane i; the sum over a row of 16 lanes, in a fixed order.
  const int2 s = slot[lane < kMaxGateK ? lane : kMaxGateK - 1];
  const int idx = s.x;
  float w = lane < a.k ? __int_as_float(s.y) : 0.0f;
  float sum = w;
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d);
  if (lane < a.k && at < a.T) {
    if (a.renormalize) w = sum > 0.0f ? w / sum : 0.0f;
    w *= a.scale;
    if (bad) w = __uint_as_float(0x7fc00000u);
    a.indices[t * a.ldi + lane] = idx;
    a.weights[t * a.ldw + lane] = (uint16_t)pack_bf16x2(w, 0.0f);
  }
}

template <int VPT, int LPT>
hipError_t launch_gate_of(const GateArgs& a, hipStream_t stream) {
  constexpr int TPB = kGateWaves * 64 / LPT;
  const dim3 grid((unsigned)((a.T + TPB - 1) / TPB)), blk(64 * kGateWaves);
  const FastDiv d = make_fastdiv((uint32_t)(a.E / a.groups));
  if (a.softmax) hipLaunchKernelGGL((gate_kernel<VPT, LPT, true>), grid, blk, 0, stream, a, d);
  else hipLaunchKernelGGL((gate_kernel<VPT, LPT, false>), grid, blk, 0, stream, a, d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  // A quarter of a wave per token issues less for a token but takes longer for it:
  // 16384x256 in groups 18.4 us against 20.0, 8192x256 10.0 against 11.0, 16384x64 5.4
  // against 7.8, but 4096x128 4.0 against 3.9.  Past 256 experts it has not been
  // made: 24 a lane would take 16384x384 in 19.6 us against 25.2 (8192x384 12.7
  // against 14.5), 32 a lane 16384x512 in 28.5 against 24.2.
  if (a.T >= 8192 && a.E <= 256) {
    if (a.E <= 64) return launch_gate_of<4, 16>(a, stream);
    if (a.E <= 128) return launch_gate_of<8, 16>(a, stream);
    return launch_gate_of<16, 16>(a, stream);
  }
  if (a.E <= 64) return launch_gate_of<1, 64>(a, stream);
  if (a.E <= 128) return launch_gate_of<2, 64>(a, stream);
  if (a.E <= 256) return launch_gate_of<4, 64>(a, stream);
  if (a.E <= 512) return launch_gate_of<8, 64>(a, stream);
  if (a.E <= 1024) return launch_gate_of<16, 64>(a, stream);
  return launch_gate_of<64, 64>(a, stream);
}

}  // namespace dsfp8
