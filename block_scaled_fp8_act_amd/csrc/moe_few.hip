// A whole routed-expert layer for a few tokens on gfx950, in two kernels
// ("DeepSeek-V3 Administrator & Developer Guide", sections 6.4 and 8.4 with the
// expert of 1.2): for token t and slot j with expert e = indices[t, j],
//   h = SiLU(W1[e] x[t]) * (W3[e] x[t]),   out[t] = sum_j weights[t, j] W2[e] h.
//
// With a few tokens every expert that is hit has a few rows, so the layer is
// bound by the bytes of the hit experts' weights, 3 D F each, read once.  The
// products run with the weights as the matrix instruction's first operand and
// some of the expert's tokens as the columns of its second (an expert with more
// tokens makes several units, whose weights come from the caches after the
// first).  Weights are widened to bf16, which holds every e4m3 and int8 value
// exactly; activations stay bf16, and h is carried as the sum of two bf16
// values (16 significant bits), which take two columns of the second product.
//
// Every wave streams its own share of the weights through an LDS slot of its
// own: direct-to-LDS loads fetch whole 128-byte lines (8 rows each; loading
// the operands straight into registers touches 16 lines for 64 bytes each),
// the fragments of a step are read back, and the next step's loads are issued
// before the step's products, so a slot is almost always on its way.  Weights
// whose rows are not 16-byte aligned take the register loads instead.
//
//   up    tasks of (unit, 32 columns of h): 32 rows of w1 and of w3 over D.
//         KS of a workgroup's eight waves share a task and join through LDS in
//         a fixed order.
//   down  one workgroup per 16 RT columns of the output.  The steps (unit, 128
//         elements of F) of all units are dealt to the sixteen waves in equal
//         consecutive ranges; a wave keeps its sums for all tokens in
//         registers over its whole range, and the waves join once at the end
//         in a fixed order, so no sum depends on timing.  The ranges, and with
//         them where a token's sums are cut, follow from all tokens' indices.
//
// Which experts are hit is found by every workgroup for itself from the
// indices, so nothing has to be sorted first and the host waits for nothing.
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "tile.h"

namespace dsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x4d __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kUpWaves = 8, kDownWaves = 16;
constexpr int kUpRows = 32;           // columns of h per task (rows of w1, and as many of w3)
constexpr int kUpSlot = 2 * kUpRows * BK;
constexpr int kMaxPairs = kMoeFewTokens * 16;

// Workspace: h as hi bf16 [T * k, Fp], then lo bf16 [T * k, Fp], by the first
// pair of each (token, expert); Fp = F rounded up to 128, zeros past F.
__host__ __device__ inline int64_t pad128(int64_t n) { return (n + 127) / 128 * 128; }

// The work units: a hit expert and up to COLS of its tokens, experts in the
// order of their first (token, slot) pair.  list[i] = expert | group << 16 |
// kAgain if the expert has several; its g-th group holds its COLS g-th to COLS
// g + COLS - 1-th token.  idx[p] = expert of pair p (-1: none here); wt[p], if
// asked for, its weight.
constexpr int kUpCols = 16, kDownCols = 8;
constexpr int kAgain = 1 << 24;
constexpr int kMaxUnits = kMaxPairs;  // at most one per pair

// At most 64 pairs of at most COLS tokens (so every expert is one unit): every
// wave finds the units by itself, in registers, lane p holding pair p.
// Lanes naming the same expert are found with ballots over the bits of the
// expert; the lowest of them leads.
__device__ __forceinline__ int find_units_wave(const MoeFewArgs& a, int* idx, int* list, float* wt) {
  const int lane = threadIdx.x & 63;
  const int P = a.T * a.k;
  int e = -1;
  if (lane < P) {
    const int t = (int)((uint32_t)lane / (uint32_t)a.k), j = lane - t * a.k;
    e = a.indices[(int64_t)t * a.ldi + j];
    if (e < 0 || e >= a.E) e = -1;
    if (wt != nullptr) wt[lane] = bf16_lo(a.weights[(int64_t)t * a.ldwt + j]);
  }
  idx[lane] = e;
  uint64_t same = ~0ull;
#pragma unroll
  for (int b = 0; b < 12; ++b) {
    const uint64_t m = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? m : ~m;
  }
  const uint64_t valid = __ballot(e >= 0);
  const bool lead = e >= 0 && __builtin_ctzll(same & valid) == lane;
  const uint64_t leads = __ballot(lead);
  if (lead) list[__popcll(leads & ((1ull << lane) - 1))] = e;
  __builtin_amdgcn_wave_barrier();
  return __popcll(leads);
}

// Any number of pairs, by the whole workgroup; table: 2 E ints of scratch.
template <int THREADS, int COLS>
__device__ __forceinline__ int find_units(const MoeFewArgs& a, int* table, int* idx, int* list, float* wt,
                                          int* wave_n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int P = a.T * a.k;
  int* lead = table;             // [E]: first pair of each expert
  int* count = table + a.E;      // [E]: tokens of each expert
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    lead[e] = P;
    count[e] = 0;
  }
  for (int p = threadIdx.x; p < P; p += THREADS) {
    const int t = (int)((uint32_t)p / (uint32_t)a.k), j = p - t * a.k;
    const int e = a.indices[(int64_t)t * a.ldi + j];
    idx[p] = e >= 0 && e < a.E ? e : -1;
    if (wt != nullptr) wt[p] = bf16_lo(a.weights[(int64_t)t * a.ldwt + j]);
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += THREADS) {
    const int e = idx[p];
    if (e < 0) continue;
    atomicMin(&lead[e], p);
    // a token that names the expert twice counts once
    bool again = false;
    for (int q = p - (int)((uint32_t)p % (uint32_t)a.k); q < p; ++q) again |= idx[q] == e;
    if (!again) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  int total = 0;
  for (int base = 0; base < P; base += THREADS) {
    const int p = base + threadIdx.x;
    const int e = p < P ? idx[p] : -1;
    const int groups = e >= 0 && lead[e] == p ? (count[e] + COLS - 1) / COLS : 0;
    int below = 0, sum = 0;
#pragma unroll
    for (int g = 0; g < kMoeFewTokens / COLS; ++g) {
      const uint64_t m = __ballot(groups > g);
      below += __popcll(m & ((1ull << lane) - 1));
      sum += __popcll(m);
    }
    if (lane == 0) wave_n[wave] = sum;
    __syncthreads();
    int at = total + below;
    for (int w = 0; w < THREADS / 64; ++w) {
      const int n = wave_n[w];
      at += w < wave ? n : 0;
      total += n;
    }
    for (int g = 0; g < groups; ++g) list[at + g] = e | g << 16 | (groups > 1 ? kAgain : 0);
    __syncthreads();
  }
  return total;
}

// A unit's columns.  Lane t: the first of token t's slots that names the expert
// (first, -1: none or another group) and the token's column (rank); lane c
// (modulo COLS) holds column c's token and pair, cols says how many there are.
struct Unit {
  int e, first, rank, cols, tok, pair;

  template <int COLS>
  __device__ __forceinline__ void set(const MoeFewArgs& a, const int* idx, int entry, int* scratch) {
    const int lane = threadIdx.x & 63;
    e = __builtin_amdgcn_readfirstlane(entry & 0xffff);
    const int g = __builtin_amdgcn_readfirstlane((entry >> 16) & 15);
    first = -1;
    if (lane < a.T)
      for (int j = a.k - 1; j >= 0; --j) first = idx[lane * a.k + j] == e ? j : first;
    const uint64_t all = __ballot(first >= 0);
    rank = __popcll(all & ((1ull << lane) - 1)) - COLS * g;
    if (rank < 0 || rank >= COLS) first = -1;
    cols = __popcll(all) - COLS * g;
    cols = cols < COLS ? cols : COLS;
    if (first >= 0) scratch[rank] = (lane * a.k + first) << 8 | lane;
    __builtin_amdgcn_wave_barrier();
    const int v = scratch[lane & (COLS - 1)];
    const bool on = (lane & (COLS - 1)) < cols;
    tok = on ? v & 255 : 0;
    pair = on ? v >> 8 : 0;
    __builtin_amdgcn_wave_barrier();
  }
};

// 16 bytes from element k (of SZ bytes) of a row of K elements, at any address;
// elements past the row are zero and nothing outside the row is read.  TAIL =
// false promises that all of them lie in the row; otherwise elements that the
// row's end cuts are taken from its last 16 bytes and shifted (a row shorter
// than that is read element by element).
template <int SZ, bool TAIL>
__device__ __forceinline__ u32x4 load16(const uint8_t* row, int64_t k, int64_t K) {
  constexpr int n = 16 / SZ;
  if (!TAIL || k + n <= K) return *reinterpret_cast<const u32x4u*>(row + k * SZ);
  if (k >= K) return u32x4{0u, 0u, 0u, 0u};
  unsigned __int128 w = 0;
  if (K >= n) {
    w = __builtin_bit_cast(unsigned __int128, *reinterpret_cast<const u32x4u*>(row + (K - n) * SZ));
    w >>= 8 * SZ * (int)(k + n - K);
  } else {
#pragma unroll 1
    for (int64_t i = K - 1; i >= k; --i)
      w = w << (8 * SZ) |
          (SZ == 1 ? (uint32_t)row[i] : (uint32_t) reinterpret_cast<const uint16_t*>(row)[i]);
  }
  return __builtin_bit_cast(u32x4, w);
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
__device__ __forceinline__ v4f block_product(const u32x4 (&w)[2], const u32x4* b, v4f acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<I8>(w[s >> 1][2 * (s & 1)], w[s >> 1][2 * (s & 1) + 1]),
                                                  __builtin_bit_cast(bf16x8, b[s]), acc, 0, 0, 0);
  return acc;
}

// Up to 32 consecutive rows of a weight, for one task or expert.
template <bool DMA>
struct Panel {
  const uint8_t* base;
  i32x4 rs;
  int rows;
  bool whole;  // no row past the matrix
  bool once;   // no other unit reads it

  __device__ __forceinline__ void set(const uint8_t* p, int64_t ld, int n, int full, int64_t K, int entry) {
    base = p;
    rows = n;
    whole = n == full;
    once = !(entry & kAgain);
    if constexpr (DMA) rs = make_rsrc(p, (uint32_t)((n - 1) * ld + K));
  }
};

// A wave's stream of weight blocks, NB blocks of 16 rows x 128 elements per
// step, through its LDS slot or (weights that are not 16-byte aligned)
// straight into the fragment registers.
template <int NB, bool DMA>
struct Stream {
  u32x4 w[NB][2];  // the step's fragments: lane (r, g) elements 32g .. 32g+31 of row r
  uint32_t behind[DMA ? 1 : NB], shift[DMA ? 1 : NB];  // the dword after them, and where in the dwords they begin
  uint32_t lds;
  const uint8_t* slot;
  uint32_t voff[2], kc[2];

  __device__ __forceinline__ void init(const uint8_t* s, int64_t ld) {
    slot = s;
    lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(s));
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + (lane >> 3);
      kc[h] = 16 * (uint32_t)((lane & 7) ^ swz_key(r));
      voff[h] = (uint32_t)(r * ld) + kc[h];
    }
  }

  // Block b of the step: rows 16 i .. of the panel, elements k .. k + 127 of K.
  __device__ __forceinline__ void issue(int b, const Panel<DMA>& p, int i, int64_t ld, uint32_t k, uint32_t K) {
    const int lane = threadIdx.x & 63;
    if constexpr (DMA) {
      const bool edge = !p.whole || k + BK > K;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v = voff[h], from = (uint32_t)(16 * i * ld) + k;
        if (edge) {
          // all of it in the lane's offset: a block that begins past the panel's
          // last row would have a scalar offset above the descriptor's size, and
          // a check that subtracts it from the size would wrap
          v = 16 * i + 8 * h + (lane >> 3) < p.rows && k + kc[h] < K ? v + from : kOob;
          from = 0;
        }
        const uint32_t to = lds + (uint32_t)(b * 2048 + h * 1024);
        // nontemporal where nothing is read again: one token 78.1 -> 72.3 us,
        // 16 tokens 521.7 -> 485.1; with it also for experts of several
        // units, 64 tokens over 8 experts took 84.3 against 69.8 us
        if (p.once) dma_b128_nt(p.rs, to, v, from);
        else dma_b128(p.rs, to, v, from);
      }
    } else {
      const int r = 16 * i + (lane & 15);
      const uint8_t* row = p.base + (r < p.rows ? r : 0) * ld;
      const int64_t kk = k + 32 * (lane >> 4);
      shift[b] = behind[b] = 0;
      if (k + BK <= K && ((reinterpret_cast<uintptr_t>(p.base) | (uintptr_t)ld) & 3) != 0) {
        // The aligned dwords that hold the 32 bytes, shifted in take(): loads at
        // any other address pass at half the rate (2 tokens, 8 experts of
        // 5001 x 1501, 87.1 -> 61.3 us; 16 tokens, 2049 x 700, 63.4 -> 44.8).
        shift[b] = (uint32_t)(reinterpret_cast<uintptr_t>(row + kk) & 3);
        const uint8_t* at = row + kk - shift[b];
        w[b][0] = *reinterpret_cast<const u32x4d*>(at);
        w[b][1] = *reinterpret_cast<const u32x4d*>(at + 16);
        behind[b] = *reinterpret_cast<const uint32_t*>(at + (shift[b] ? 32 : 28));
      } else if (k + BK <= K) {
        w[b][0] = load16<1, false>(row, kk, K);
        w[b][1] = load16<1, false>(row, kk + 16, K);
      } else {
        w[b][0] = load16<1, true>(row, kk, K);
        w[b][1] = load16<1, true>(row, kk + 16, K);
      }
    }
  }

  // The step's loads have arrived; afterwards the slot is free.
  __device__ __forceinline__ void take() {
    if constexpr (DMA) {
      const int lane = threadIdx.x & 63, fr = lane & 15, fg = lane >> 4;
      wait_vmcnt<0>();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[b][h] = *reinterpret_cast<const u32x4*>(slot + b * 2048 + swz(fr, 2 * fg + h));
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t next = e < 7 ? w[b][(e + 1) >> 2][(e + 1) & 3] : behind[b];
          w[b][e >> 2][e & 3] = __builtin_amdgcn_alignbyte(next, w[b][e >> 2][e & 3], shift[b]);
        }
    }
  }
};

// SiLU(g) * u, split into the two bf16 values hi + lo: 16 significant bits of it,
// an error of 2^-17 each and 2.5e-6 of a sum over 2048 of them, where the output's
// rounding to bf16 is 1.7e-3.  The two parts for eight tokens fill the sixteen
// columns of one matrix instruction; a third part, for all 24 bits, would need a
// second product per block, and products of their own for two parts already held
// the stream of weights up.
__device__ __forceinline__ void split_gate(float g, float u, uint16_t& hi, uint16_t& lo) {
  const float h = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
  const float top = bf16_lo(pack_bf16x2(h, 0.0f));
  // an infinite or NaN h stays so in hi alone
  hi = (uint16_t)pack_bf16x2(top, 0.0f);
  lo = (uint16_t)pack_bf16x2(fabsf(top) < __builtin_inff() ? h - top : 0.0f, 0.0f);
}

// Bound by the weights' bytes.  256 experts of 7168 x 2048, e4m3, 8 per token: one
// token 37-39 us for 235 MB (6.0-6.3 TB/s; a read alone reaches 7.1), 16 tokens
// (69 experts hit) 316 us (6.4 TB/s); 64 tokens, 17 of 32 experts hit, 83 us (6.0
// TB/s).  Rows that are not 16-byte aligned come through registers: 5 tokens, 8
// experts of 1000 x 714, 7.9-8.1 us.
template <bool I8, bool DMA>
__global__ __launch_bounds__(64 * kUpWaves, DMA ? 4 : 2) void moe_few_up_kernel(MoeFewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[kUpWaves * kUpSlot];
  __shared__ int idx[kMaxPairs], list[kMaxUnits];
  __shared__ int wave_n[kUpWaves], scratch[kUpWaves][kUpCols];
  static_assert(kMaxRouteExperts * 8 <= kUpWaves * kUpSlot, "the table of experts lies in the ring");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 15, fg = lane >> 4;
  int *my_idx = idx, *my_list = list;
  int units;
  if (a.T * a.k <= 64 && a.T <= kUpCols) {
    my_idx = idx + 64 * wave;
    my_list = list + 64 * wave;
    units = find_units_wave(a, my_idx, my_list, nullptr);
  } else {
    units = find_units<64 * kUpWaves, kUpCols>(a, reinterpret_cast<int*>(ring), idx, list, nullptr, wave_n);
  }
  units = __builtin_amdgcn_readfirstlane(units);
  const int nkb = (int)((a.D + BK - 1) / BK);
  const uint32_t tiles = (uint32_t)((a.F + kUpRows - 1) / kUpRows);
  const int64_t tasks = (int64_t)units * tiles, Fp = pad128(a.F);
  uint16_t* hi = static_cast<uint16_t*>(a.work);
  uint16_t* lo = hi + (int64_t)a.T * a.k * Fp;
  // KS waves per task, up to all of them: the more share a task, the longer the
  // run of each weight row that is read at one time (16 tokens: 462 us with
  // eight waves per task, 485 with the one to eight that would balance best).
  int ks = 1;
  while (ks < kUpWaves && 2 * ks <= nkb) ks *= 2;
  const int sub = wave & (ks - 1), per = kUpWaves / ks;
  Stream<4, DMA> st;
  st.init(ring + wave * kUpSlot, a.ldw13);
  float(*red)[17] = reinterpret_cast<float(*)[17]>(ring + wave * kUpSlot);
  static_assert(2 * kUpRows * 17 * 4 <= kUpSlot, "a wave's sums fit its slot");

  for (int64_t base = (int64_t)blockIdx.x * per; base < tasks; base += (int64_t)gridDim.x * per) {
    const int64_t task = base + wave / ks;
    const bool live = task < tasks;
    const uint32_t ui = live ? (uint32_t)task / tiles : 0;
    const int64_t f0 = live ? (int64_t)((uint32_t)task - ui * tiles) * kUpRows : 0;
    const int entry = __builtin_amdgcn_readfirstlane(my_list[ui]);
    Unit u;
    u.set<kUpCols>(a, my_idx, entry, scratch[wave]);
    const int e = u.e;
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
      const int rows = (int)(a.F - f0 < kUpRows ? a.F - f0 : kUpRows);
      Panel<DMA> w1, w3;
      const uint8_t* at1 = a.w13 + ((int64_t)e * 2 * a.F + f0) * a.ldw13;
      w1.set(at1, a.ldw13, rows, kUpRows, a.D, entry);
      w3.set(at1 + a.F * a.ldw13, a.ldw13, rows, kUpRows, a.D, entry);
      auto issue = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) st.issue(i, i < 2 ? w1 : w3, i & 1, a.ldw13, (uint32_t)kb * BK, (uint32_t)a.D);
      };
      // x of the lane's column, elements of K-block kb (a lane past the unit's
      // columns reads token 0, and its column is never used)
      const uint8_t* xrow = reinterpret_cast<const uint8_t*>(a.x + (int64_t)u.tok * a.ldx);
      u32x4 b[4];
      auto columns = [&](int kb) __attribute__((always_inline)) {
        const int64_t k = (int64_t)kb * BK + 32 * fg;
        if ((int64_t)(kb + 1) * BK <= a.D) {
#pragma unroll
          for (int s = 0; s < 4; ++s) b[s] = load16<2, false>(xrow, k + 8 * s, a.D);
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) b[s] = load16<2, true>(xrow, k + 8 * s, a.D);
        }
      };
      // Block scales: w1's 32 rows lie in one 128-row block; w3's may span two,
      // when F is no multiple of 32.
      const int64_t r3 = a.F + f0;
      const float* se = a.s13 + (I8 ? 0 : (int64_t)e * ((2 * a.F + BK - 1) / BK) * a.lds13);
      const float* s1p = se + (f0 >> 7) * a.lds13;
      const float* s3p = se + (r3 >> 7) * a.lds13;
      const float* s3q = se + ((r3 + rows - 1) >> 7) * a.lds13;
      const int cut = (int)(BK - (r3 & (BK - 1)));  // first w3 row of the second block
      if (sub < nkb) {
        issue(sub);
        columns(sub);
      }
      for (int kb = sub; kb < nkb; kb += ks) {
        float s1 = 1.0f, s3a = 1.0f, s3b = 1.0f;
        if constexpr (!I8) {
          s1 = s1p[kb];
          s3a = s3p[kb];
          s3b = s3q[kb];
        }
        st.take();
        const bool more = kb + ks < nkb;
        if (DMA && more) issue(kb + ks);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (I8) {
            acc[i] = block_product<I8>(st.w[i], b, acc[i]);
          } else {
            const v4f part = block_product<I8>(st.w[i], b, v4f{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float s = i < 2 ? s1 : (16 * (i & 1) + 4 * fg + v < cut ? s3a : s3b);
              acc[i][v] = __builtin_fmaf(part[v], s, acc[i][v]);
            }
          }
        }
        if (more) {
          if (!DMA) issue(kb + ks);
          columns(kb + ks);
        }
      }
    }

    // Join the waves' sums, gate, and write h: 32 x 16 values per task.
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[16 * i + 4 * fg + v][fr] = acc[i][v];
    __syncthreads();
    const float* group = reinterpret_cast<const float*>(ring + (wave - sub) * kUpSlot);
    for (int q = sub * 64 + lane; q < kUpRows * kUpCols; q += ks * 64) {
      const int r = q & (kUpRows - 1), c = q >> 5;
      const int pair = __shfl(u.pair, c);
      const int64_t f = f0 + r;
      if (!live || c >= u.cols || f >= Fp) continue;
      uint16_t vh = 0, vl = 0;
      if (f < a.F) {
        float g = 0.0f, up = 0.0f;
        for (int w = 0; w < ks; ++w) {
          g += group[w * (kUpSlot / 4) + r * 17 + c];
          up += group[w * (kUpSlot / 4) + (kUpRows + r) * 17 + c];
        }
        if constexpr (I8) {
          g *= a.s13[(int64_t)e * a.lds13 + f];
          up *= a.s13[(int64_t)e * a.lds13 + a.F + f];
        }
        split_gate(g, up, vh, vl);
      }
      hi[(int64_t)pair * Fp + f] = vh;
      lo[(int64_t)pair * Fp + f] = vl;
    }
    // the last task of a unit clears its rows from there to Fp
    const int rest = live && f0 + kUpRows >= a.F ? (int)(Fp - f0) - kUpRows : 0;
    for (int q = sub * 64 + lane; q < rest * kUpCols; q += ks * 64) {
      const int c = q & (kUpCols - 1);
      const int pair = scratch[wave][c] >> 8;
      if (c >= u.cols) continue;
      const int64_t at = (int64_t)pair * Fp + f0 + kUpRows + (q >> 4);
      hi[at] = 0;
      lo[at] = 0;
    }
    __syncthreads();
  }
}

// `rows` output columns per workgroup in RT row tiles of 16 (rows a multiple of
// 4); CT column tiles of 16 tokens.
// Bound by the weights' bytes, and with one token by filling the CUs: for the
// sizes above 23-24 us for 117 MB (5.0 TB/s), 167 us (6.1 TB/s), 64 us (3.9 TB/s:
// an expert of nine tokens or more is several units, whose weights pass through
// LDS and are widened once for each) and 6.7-7.9 us.
// Interleaving the units among the waves instead of consecutive ranges, two
// K-blocks in flight per wave, and 16-row tiles with two workgroups per CU were
// the same or slower.
template <bool I8, int CT, int RT, bool DMA>
__global__ __launch_bounds__(64 * kDownWaves) void moe_few_down_kernel(MoeFewArgs a, int wg_rows) {
  constexpr int SLOT = RT * 16 * BK;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kDownWaves * SLOT];
  __shared__ int idx[kMaxPairs], list[kMaxUnits];
  __shared__ float wt[kMaxPairs];
  __shared__ int wave_n[kDownWaves], scratch[kDownWaves][kDownCols];
  static_assert(kMaxRouteExperts * 8 <= kDownWaves * SLOT, "the table of experts lies in the ring");
  static_assert(64 * kDownWaves <= kMaxPairs, "a list of 64 per wave");
  constexpr int CJ = CT < 2 ? CT : 2;  // column tiles joined at a time
  static_assert(16 * CJ * 16 * RT * 4 <= SLOT, "a wave's sums fit its slot");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int fr = lane & 15, fg = lane >> 4;
  int *my_idx = idx, *my_list = list;
  float* my_wt = wt;
  int units = 0;  // F = 0: the up kernel did not run, and the output is zero
  if (a.F > 0) {
    if (a.T * a.k <= 64 && a.T <= kDownCols) {
      my_idx = idx + 64 * wave;
      my_list = list + 64 * wave;
      my_wt = wt + 64 * wave;
      units = find_units_wave(a, my_idx, my_list, my_wt);
    } else {
      units = find_units<64 * kDownWaves, kDownCols>(a, reinterpret_cast<int*>(ring), idx, list, wt, wave_n);
    }
  }
  units = __builtin_amdgcn_readfirstlane(units);
  const int64_t d0 = (int64_t)blockIdx.x * wg_rows, Fp = pad128(a.F);
  const int rows = (int)(a.D - d0 < wg_rows ? a.D - d0 : wg_rows);
  const uint16_t* hi = static_cast<const uint16_t*>(a.work);
  const int per = (int)((a.F + BK - 1) / BK);
  const int64_t steps = (int64_t)units * per, s0 = steps * wave / kDownWaves;
  const int n = (int)(steps * (wave + 1) / kDownWaves - s0);  // this wave's steps
  int at = n > 0 ? (int)(s0 / per) : 0, kp = (int)(s0 - (int64_t)at * per);

  Stream<RT, DMA> st;
  st.init(ring + wave * SLOT, a.ldw2);
  v4f acc[RT], sum[RT][CT];  // the current unit's columns; every token's
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CT; ++c) sum[i][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  Panel<DMA> w2;
  auto panel = [&](int entry) __attribute__((always_inline)) {
    w2.set(a.w2 + ((int64_t)(entry & 0xffff) * a.D + d0) * a.ldw2, a.ldw2, rows, 16 * RT, a.F, entry);
  };
  auto issue = [&](int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i) st.issue(i, w2, i, a.ldw2, (uint32_t)k * BK, (uint32_t)a.F);
  };
  // Columns 0 .. 7 hold the high parts of the unit's rows of h, columns 8 .. 15
  // the low parts, so one product serves both (with a product each, of 16
  // columns, the matrix and vector instructions held the stream up: 16 tokens
  // 208 us against 180).  A lane past the unit's columns reads some row of h;
  // what its column makes of it is never used.
  u32x4 b[4];
  float sca = 1.0f, scb = 1.0f;  // the step's block scales, of this block of rows and the next
  const int64_t kbd = (a.D + BK - 1) / BK;
  const int cut = (int)(BK - (d0 & (BK - 1)));  // first row of the next block
  Unit u;
  const uint16_t* hp = nullptr;
  const float *spa = nullptr, *spb = nullptr;
  auto enter = [&](int entry, int k) __attribute__((always_inline)) {
    u.template set<kDownCols>(a, my_idx, entry, scratch[wave]);
    hp = hi + (fr < kDownCols ? 0 : (int64_t)a.T * a.k * Fp) + (int64_t)u.pair * Fp + (int64_t)k * BK + 32 * fg;
    if constexpr (!I8) {
      spa = a.s2 + ((int64_t)u.e * kbd + (d0 >> 7)) * a.lds2 + k;
      spb = a.s2 + ((int64_t)u.e * kbd + ((d0 + rows - 1) >> 7)) * a.lds2 + k;
    }
  };
  auto columns = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 4; ++s) b[s] = *reinterpret_cast<const u32x4*>(hp + 8 * s);
    hp += BK;
    if constexpr (!I8) {
      sca = *spa++;
      scb = *spb++;
    }
  };
  // Add a finished unit's columns to their tokens, times the tokens' weights.
  auto leave = [&]() __attribute__((always_inline)) {
    float w = 0.0f;
    if (u.first >= 0)
      for (int j = u.first; j < a.k; ++j)
        if (my_idx[lane * a.k + j] == u.e) w += my_wt[lane * a.k + j];
    if constexpr (I8) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int r = 16 * i + 4 * fg + v;
          acc[i][v] *= a.s2[(int64_t)u.e * a.lds2 + d0 + (r < rows ? r : rows - 1)];
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int has = __shfl(u.first, 16 * c + fr), col = __shfl(u.rank, 16 * c + fr);
      const float wc = __shfl(w, 16 * c + fr);
      const int from = (lane & 48) | (col & (kDownCols - 1));
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float y = __shfl(acc[i][v], from) + __shfl(acc[i][v], from + kDownCols);
          if (has >= 0) sum[i][c][v] = __builtin_fmaf(y, wc, sum[i][c][v]);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };

  __syncthreads();  // the table of experts gives way to the ring
  if (n > 0) {
    const int entry = __builtin_amdgcn_readfirstlane(my_list[at]);
    panel(entry);
    issue(kp);
    enter(entry, kp);
    columns();
  }
  for (int s = 0; s < n; ++s) {
    const bool more = s + 1 < n, turn = ++kp == per;
    int entry = 0;
    if (turn) {
      kp = 0;
      ++at;
      if (more) {
        entry = __builtin_amdgcn_readfirstlane(my_list[at]);
        panel(entry);
      }
    }
    st.take();
    if (DMA && more) issue(kp);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const v4f part = block_product<I8>(st.w[i], b, v4f{0.0f, 0.0f, 0.0f, 0.0f});
      const float sc = 16 * i + 4 * fg < cut ? sca : scb;
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][v] = I8 ? acc[i][v] + part[v] : __builtin_fmaf(part[v], sc, acc[i][v]);
    }
    if (turn || !more) leave();
    if (more) {
      if (!DMA) issue(kp);
      if (turn) enter(entry, 0);
      columns();
    }
  }
  __syncthreads();

  // sums[wave][token][row], in the waves' slots
#pragma unroll
  for (int c0 = 0; c0 < CT; c0 += CJ) {
    float* mine = reinterpret_cast<float*>(ring + wave * SLOT);
    if (c0 > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CJ; ++c)
        *reinterpret_cast<v4f*>(mine + (16 * c + fr) * (16 * RT) + 16 * i + 4 * fg) = sum[i][c0 + c];
    __syncthreads();
    for (int q = threadIdx.x; q < 16 * CJ * 16 * RT; q += 64 * kDownWaves) {
      float y = 0.0f;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) y += reinterpret_cast<const float*>(ring + w * SLOT)[q];
      const int t = 16 * c0 + q / (16 * RT), r = q % (16 * RT);
      if (t < a.T && r < rows) a.out[(int64_t)t * a.ldo + d0 + r] = (uint16_t)pack_bf16x2(y, 0.0f);
    }
  }
}

template <bool I8, int CT, bool DMA>
hipError_t launch(const MoeFewArgs& a, hipStream_t stream) {
  const int cus = device_cu_count();
  if (a.F > 0) {
    // at most two workgroups per CU, which is what fits
    const int64_t tasks = (int64_t)a.T * a.k * ((a.F + kUpRows - 1) / kUpRows);
    const int64_t grid = tasks < 2 * cus ? tasks : 2 * cus;
    hipLaunchKernelGGL((moe_few_up_kernel<I8, DMA>), dim3((unsigned)grid), dim3(64 * kUpWaves), 0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  // As many output columns per workgroup as spread them over all CUs, up to 32
  // (7168 columns: 256 workgroups of 28 rather than 224 of 32).
  const int64_t want = ((a.D + cus - 1) / cus + 3) / 4 * 4;
  const int rows = (int)(want < 32 ? want : 32);
  const dim3 grid((unsigned)((a.D + rows - 1) / rows)), blk(64 * kDownWaves);
  if (rows > 16) hipLaunchKernelGGL((moe_few_down_kernel<I8, CT, 2, DMA>), grid, blk, 0, stream, a, rows);
  else hipLaunchKernelGGL((moe_few_down_kernel<I8, CT, 1, DMA>), grid, blk, 0, stream, a, rows);
  return hipGetLastError();
}

// 16-byte aligned weight rows, 16 of them within 31-bit offsets.
inline bool dma_ok(const void* p, int64_t ld, int64_t K) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 16 == 0 && K % 16 == 0 && ld < ((int64_t)1 << 26);
}

template <bool I8, int CT>
hipError_t launch_feed(const MoeFewArgs& a, hipStream_t stream) {
  return dma_ok(a.w13, a.ldw13, a.D) && dma_ok(a.w2, a.ldw2, a.F) ? launch<I8, CT, true>(a, stream)
                                                                  : launch<I8, CT, false>(a, stream);
}

template <bool I8>
hipError_t launch_ct(const MoeFewArgs& a, hipStream_t stream) {
  return a.T <= 16 ? launch_feed<I8, 1>(a, stream) : launch_feed<I8, 4>(a, stream);
}

}  // namespace

size_t moe_few_workspace_bytes(int64_t T, int64_t k, int64_t F) { return (size_t)(T * k * pad128(F) * 4); }

hipError_t launch_moe_few(const MoeFewArgs& a, hipStream_t stream) {
  return a.i8 ? launch_ct<true>(a, stream) : launch_ct<false>(a, stream);
}

}  // namespace dsfp8
