// The whole MoE layer for a few tokens (T <= 64), in two launches.
//
// With few tokens the layer is a walk over the selected experts' weights: each
// is read once from memory and multiplied by the handful of rows that chose
// it, so the kernel is bound by the weights' bytes and, for one token, by
// latency (75 MB at the 30B shape in bf16: 36 us; 64 tokens reach nearly all of
// the 1.2 GB: 259 us, 4.6 TB/s). Everything here serves that: the
// weights go straight from memory into registers in 16-byte loads, several
// steps ahead and on into the next unit; gate/up and down are one launch, so
// that the down weights' first loads are in flight while the last gate/up
// units finish; no activation row but the selected experts' (T k I bf16) is
// ever written.
//
//   few_router_kernel: logits, one workgroup per expert and 8 tokens.
//     Products and sums are taken in fp64, where a product of two bf16
//     numbers is exact at both ends of the range (in fp32 it overflows or
//     vanishes there). It also clears the second kernel's counters.
//   few_kernel: one persistent workgroup of 8 wavefronts per CU. Each selects
//     the experts of all tokens for itself (no third launch), then takes
//     its share of the units:
//     - gate/up unit: one expert, 8 or 16 columns (8 rows of W_gate and 8 of
//       W_up per wavefront). The reduction is split over the wavefronts, so
//       each token row's part is loaded by one or two of them (eight that work
//       side by side on one expert's columns wait for each other's pending
//       lines in the vector cache: 300 instead of 165 us for 64 tokens' gate
//       and up). The partial sums meet in LDS; a = bf16(w silu(g) u) goes to
//       the workspace: bf16 because the down product takes bf16 operands, its
//       weights being bf16 or 8 bits wide (y off by 0.0023 to 0.0024 in the norm,
//       0.0016 with a in fp32).
//     - down unit: one group of experts, 16 columns of y. The (expert, k)
//       steps are split over the wavefronts, each adding its experts' products
//       into its own y tile in LDS; the eight tiles are then summed in order.
//       With one group (up to 8 experts) that is y; otherwise the groups'
//       fp32 partial sums go to the workspace and the last workgroup to
//       finish a column block adds them in group order.
//     A wavefront's loads run two batches of steps ahead of its products and
//     on into the next units; nothing in that stream is conditional (a step
//     that does not exist reads out of range, which costs nothing), since only
//     then do the compiler's waits leave the newer loads running.
//
// Order and progress: the gate/up units come in as many shares as there are
// workgroups; a workgroup claims one at its start, and another whenever it is
// done, as long as one is left (eight counters, one per XCD, each first asked
// by its own workgroups). It goes on to the down units only once all shares
// are claimed. A down unit waits for its group's gate/up units; by then
// running workgroups hold all of those, and gate/up units wait for nothing:
// the wait ends whatever else occupies the device. (If another call
// overwrites the workspace, against the interface, the count may never be
// reached: the wait gives up after kFewPolls looks, seconds of running, and y
// becomes NaN there.) Claiming unit by unit instead stalls the loads: an atomic's
// answer comes back behind all loads issued before it.
//
// Tile: v_mfma_f32_16x16x32_bf16 with the weights as A (16 rows) and up to 16
// token rows as B, so a lane's four results are four consecutive columns of
// one row. A step is 128 bytes of each weight row: 64 bf16 or 128 E4M3 codes
// (one scale block; a last half block reads zeros). Loads take a row's 128
// bytes with eight neighbouring lanes (a load in the product's own layout,
// neighbouring lanes in different rows, costs the address unit 64 cycles
// instead of 16), and the steps change layout through LDS of the wavefront's
// own, weights and token rows alike: no barrier, and the registers stay the
// prefetch buffer. E4M3 weights are widened to bf16 (exact) and each step's
// product is multiplied by its block's scale in fp32.
#include "moe_internal.h"
#include "select.h"

#include <type_traits>

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBf16 = 0, kFp8 = 1;  // weight formats
constexpr int kNW = 8;              // wavefronts per workgroup
constexpr int kThreads = kNW * kWave;
constexpr int kGC = 8, kDC = 16;   // columns per gate/up and per down unit
constexpr int kLists = 8;           // counters of claimed shares, one per XCD
constexpr int kLine = 32;           // counters that workgroups add to lie 128 bytes apart
constexpr int kMaxPairs = kFewMaxT * kFewMaxK;
constexpr uint32_t kNoRow = 0x80000000u;  // an offset past every row, whatever is added to it

// The workspace's counters (uint32, in lines): [0, 8) gate/up shares claimed,
// then gate/up tiles done per group; after the lines, down units done per
// column block.
struct FewParams {
  int T, H, E, k, I;
  const bf16_t* x;
  const void *w0, *w1, *w2;     // gate, up, down: bf16 or E4M3 codes
  const float *s0, *s1, *s2;    // block scales (E4M3)
  const float* logits;
  int32_t* topk_idx;
  float* topk_w;
  bf16_t* y;
  uint32_t* cnt;
  uint32_t* cnt_down;
  uint32_t polls;               // looks at a count before a wait gives up
  bf16_t* act;                  // [T*k][I], weighted
  float* part;                  // [groups][T][H]
};

// Data that workgroups hand to each other inside the launch (activations, the
// groups' partial sums) is stored and loaded at device scope (sc1: written
// through, and not served from a cache that another XCD's store has not
// reached). A store counts as done once it is there, so the writer only waits
// for its stores before it counts its unit, and neither side has to write
// back or drop a whole L2 (a release or acquire fence of agent scope does, and
// a few hundred of them per launch took most of its time).
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kDeviceScope = 16;  // sc1
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}
__device__ __forceinline__ void stores_done() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  asm volatile("" ::: "memory");
}

// ---- router -----------------------------------------------------------------

constexpr int kRouterTokens = 8;
constexpr int kRouterWaves = 4;  // one expert's reduction is split over them: one load's latency at H = 2048

__global__ __launch_bounds__(kRouterWaves* kWave) void few_router_kernel(int T, int H, int E,
                                                                         const bf16_t* __restrict__ x,
                                                                         const bf16_t* __restrict__ wr,
                                                                         const float* __restrict__ bias,
                                                                         float* __restrict__ logits,
                                                                         uint32_t* __restrict__ cnt, int ncnt) {
  constexpr int N = kRouterWaves * kWave;
  __shared__ double part[kRouterWaves][kRouterTokens];
  const int e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int stride = gridDim.x * gridDim.y * N;
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * N + tid; i < ncnt; i += stride) cnt[i] = 0;
  double acc[kRouterTokens];
#pragma unroll
  for (int i = 0; i < kRouterTokens; ++i) acc[i] = 0.0;
  const u32x4* w4 = reinterpret_cast<const u32x4*>(wr + static_cast<int64_t>(e) * H);
  const u32x4* x4 = reinterpret_cast<const u32x4*>(x + static_cast<int64_t>(t0) * H);
  const int nt = min(kRouterTokens, T - t0), chunks = H / 8;
  for (int c = tid; c < chunks; c += N) {
    const u32x4 wv = w4[c];
    u32x4 xv[kRouterTokens];
#pragma unroll
    for (int i = 0; i < kRouterTokens; ++i) xv[i] = i < nt ? x4[static_cast<int64_t>(i) * chunks + c] : wv;
    double lo[4], hi[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      lo[q] = static_cast<double>(__uint_as_float(wv[q] << 16));
      hi[q] = static_cast<double>(__uint_as_float(wv[q] & 0xffff0000u));
    }
#pragma unroll
    for (int i = 0; i < kRouterTokens; ++i) {
      if (i >= nt) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[i] = fma(static_cast<double>(__uint_as_float(xv[i][q] << 16)), lo[q], acc[i]);
        acc[i] = fma(static_cast<double>(__uint_as_float(xv[i][q] & 0xffff0000u)), hi[q], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRouterTokens; ++i) {
    if (i >= nt) break;
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) acc[i] += __shfl_xor(acc[i], o, kWave);
    if (lane == 0) part[wave][i] = acc[i];
  }
  __syncthreads();
  if (tid < nt) {
    double v = part[0][tid];
#pragma unroll
    for (int w = 1; w < kRouterWaves; ++w) v += part[w][tid];
    logits[static_cast<int64_t>(t0 + tid) * E + e] = static_cast<float>(v + (bias ? static_cast<double>(bias[e]) : 0.0));
  }
}

// ---- the layer --------------------------------------------------------------

// One step in registers as loaded: 16 weight rows x 128 bytes, lane l the
// 16-byte chunk l % 8 of rows l / 8 and 8 + l / 8; and up to 16 token rows x
// the same k (kXL lanes per row, XR rows).
template <int FMT> constexpr int kStep = FMT == kBf16 ? 64 : 128;   // k per step
template <int FMT> constexpr int kXL = FMT == kBf16 ? 8 : 16;
template <int FMT> constexpr int kRPI = kWave / kXL<FMT>;           // token rows per load
template <int FMT, int XR>
struct Step {
  u32x4 w[2];
  u32x4 x[XR / kRPI<FMT>];
};

// The wavefront's LDS for one step: weight rows, then token rows, chunks
// swizzled by row so that both sides touch every bank once.
template <int FMT> constexpr int kStepBytes = 2048 + kXL<FMT> * 256;
__device__ __forceinline__ int w_slot(int row, int chunk) { return row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4); }
template <int FMT>
__device__ __forceinline__ int x_slot(int row, int chunk) {
  return 2048 + row * (kXL<FMT> * 16) + ((chunk ^ (FMT == kBf16 ? (row >> 1) & 7 : row)) << 4);
}

__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b) {  // eight E4M3 codes
  const bf16x2 r0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2 r1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2 r2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2 r3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf16x8{r0.x, r0.y, r1.x, r1.y, r2.x, r2.y, r3.x, r3.y};
}

__device__ __forceinline__ void put_w(char* lds, const u32x4 (&w)[2]) {
  const int lane = threadIdx.x % kWave, row = lane / 8, chunk = lane % 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(lds + w_slot(row + 8 * i, chunk)) = w[i];
}
template <int FMT, int XN>
__device__ __forceinline__ void put_x(char* lds, const u32x4 (&x)[XN], int row0) {
  const int lane = threadIdx.x % kWave, row = row0 + lane / kXL<FMT>, chunk = lane % kXL<FMT>;
#pragma unroll
  for (int i = 0; i < XN; ++i) *reinterpret_cast<u32x4*>(lds + x_slot<FMT>(row + kRPI<FMT> * i, chunk)) = x[i];
}

// acc += (scale) weight rows x token rows over the step in LDS.
template <int FMT>
__device__ __forceinline__ void multiply(f32x4& acc, const char* lds, float scale) {
  const int lane = threadIdx.x % kWave, row = lane % 16, g = lane / 16;
  auto at = [&](int o) { return *reinterpret_cast<const u32x4*>(lds + o); };
  if constexpr (FMT == kBf16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 w = at(w_slot(row, 4 * h + g)), x = at(x_slot<FMT>(row, 4 * h + g));
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc,
                                                    0, 0, 0);
    }
  } else {
    f32x4 p = f32x4{};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 w = at(w_slot(row, 4 * h + g));
      const u32x4 x0 = at(x_slot<FMT>(row, 2 * (4 * h + g))), x1 = at(x_slot<FMT>(row, 2 * (4 * h + g) + 1));
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w.x, w.y), __builtin_bit_cast(bf16x8, x0), p, 0, 0, 0);
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w.z, w.w), __builtin_bit_cast(bf16x8, x1), p, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(scale, p[i], acc[i]);
  }
}

__device__ __forceinline__ float lane_value(float v, int src) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), src));
}

struct FewLists {  // in LDS: the pairs (token, slot) sorted by expert
  int na;                          // experts that some token selected
  int share;                       // the next share of gate/up units
  int last;
  uint16_t expert[1024];           // active expert a -> expert
  uint16_t start[1025];            // its pairs: list[start[a] .. start[a + 1])
  uint16_t list[kMaxPairs];        // pair t * k + j
  uint16_t token[kMaxPairs];       // t, by place in the list
  uint16_t sel[kMaxPairs];         // expert of each pair
  float weight[kMaxPairs];         // by pair
};

// Scratch: the selection's, then the units'.
template <int TILES>
union FewScratch {
  struct {
    int count[1024];               // pairs per expert, then a cursor
    int wave_sum[kNW];
  } lists;
  float red[2][TILES][kNW][16][20];      // gate/up, by turns: [row tile][wave][row][8 gate, 8 up columns]
  float tile[kNW][16 * TILES][kDC + 4];  // down: [wave][token][column]
};

// Barrier for LDS traffic: unlike __syncthreads it leaves loads in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Unsigned maximum or minimum over a 16-lane row, in every lane of it.
template <bool MAX>
__device__ __forceinline__ uint32_t row_extreme(uint32_t v) {
  auto pick = [](uint32_t a, uint32_t b) { return MAX ? (a > b ? a : b) : (a < b ? a : b); };
  v = pick(v, dpp32<0xB1>(v));
  v = pick(v, dpp32<0x4E>(v));
  v = pick(v, dpp32<0x141>(v));
  return pick(v, dpp32<0x140>(v));
}

// Selection for more than 16 tokens: one token per 16-lane row (wavefronts
// past the last token skip it). A lane holds the order bits
// of logits n + 16 c (sel_key's upper word; 0 for a NaN). A round takes the
// largest, then the lowest index that has it, and marks that one as taken. The
// weights follow at once: softmax and renormalisation as moe_route.
template <int NC>
__device__ __forceinline__ void few_select_rows(const FewParams& P, FewLists& L) {
  const int tid = threadIdx.x, n = tid % 16;
  const int E = P.E, k = P.k;
  for (int t0 = 0; t0 < P.T; t0 += kThreads / 16) {
    const int tw = __builtin_amdgcn_readfirstlane(t0 + tid / kWave * 4);
    if (tw >= P.T) break;
    const int t = t0 + tid / 16;
    const bool active = t < P.T;
    const float* l = P.logits + static_cast<int64_t>(active ? t : 0) * E;
    uint32_t o[NC];
    uint64_t left = 0;  // bit c: a logit that is not taken
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = n + 16 * c;
      o[c] = 0;  // absent: below every number's bits, and not in `left`
      if (e < E) o[c] = static_cast<uint32_t>(sel_key(l[e], 0) >> 32);
      if (e < E) left |= 1ull << c;
    }
    float sel_v = 0.0f, vmax = 0.0f;
    int sel_i = 0;
    for (int j = 0; j < k; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < NC; ++c) m = o[c] > m ? o[c] : m;
      m = row_extreme<true>(m);
      uint32_t at = ~0u;
#pragma unroll
      for (int c = NC - 1; c >= 0; --c) at = o[c] == m && (left >> c & 1) ? n + 16 * c : at;
      at = row_extreme<false>(at);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (at == static_cast<uint32_t>(n + 16 * c)) {
          o[c] = 0;
          left &= ~(1ull << c);
        }
      }
      const float bv = key_value(static_cast<uint64_t>(m) << 32);
      if (j == 0) vmax = bv;
      if (n == j) {
        sel_v = bv;
        sel_i = static_cast<int>(at);
      }
    }
    // The softmax denominator: the selected logits and the ones left.
    const float top = n < k ? expf(sel_v - vmax) : 0.0f;
    float z = top;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (left >> c & 1) z += expf(key_value(static_cast<uint64_t>(o[c]) << 32) - vmax);
    z = row_sum(z);
    const float p = top / z;
    const float den = row_sum(p) + 1e-20f;
    if (active && n < k) {
      L.sel[t * k + n] = static_cast<uint16_t>(sel_i);
      L.weight[t * k + n] = p / den;
    }
  }
}

// Selection for up to 16 tokens: a wavefront per token, logits lane + 64 c.
// The rounds are the same; the lowest index comes from a ballot.
template <int NC>
__device__ __forceinline__ void few_select_waves(const FewParams& P, FewLists& L) {
  const int lane = threadIdx.x % kWave;
  const int E = P.E, k = P.k;
  for (int t = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); t < P.T; t += kNW) {
    const float* l = P.logits + static_cast<int64_t>(t) * E;
    uint32_t o[NC];
    uint32_t left = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = lane + kWave * c;
      o[c] = 0;  // absent: below every number's bits, and not in `left`
      if (e < E) o[c] = static_cast<uint32_t>(sel_key(l[e], 0) >> 32);
      if (e < E) left |= 1u << c;
    }
    int sel_i = 0;
    for (int j = 0; j < k; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < NC; ++c) m = o[c] > m ? o[c] : m;
      m = row_extreme<true>(m);
      const uint32_t m0 = __builtin_amdgcn_readlane(m, 0), m1 = __builtin_amdgcn_readlane(m, 16),
                     m2 = __builtin_amdgcn_readlane(m, 32), m3 = __builtin_amdgcn_readlane(m, 48);
      m = max(max(m0, m1), max(m2, m3));
      int at = -1;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (at < 0) {
          const uint64_t hit = __ballot(o[c] == m && (left >> c & 1));
          if (hit) {
            const int src = __builtin_ctzll(hit);
            at = src + kWave * c;
            if (lane == src) {
              o[c] = 0;
              left &= ~(1u << c);
            }
          }
        }
      }
      if (lane == j) sel_i = at;
    }
    if (lane < k) L.sel[t * k + lane] = static_cast<uint16_t>(sel_i);
  }
}

// The weights of up to 16 tokens' experts: one token per wavefront. Off the way of the first weight loads;
// the values are needed at the end of the first unit.
__device__ __forceinline__ void few_weights(const FewParams& P, FewLists& L) {
  const int lane = threadIdx.x % kWave;
  const int E = P.E, k = P.k;
  for (int t = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); t < P.T; t += kNW) {
    const float* l = P.logits + static_cast<int64_t>(t) * E;
    const float v0 = lane < E ? l[lane] : 0.0f, v1 = kWave + lane < E ? l[kWave + lane] : 0.0f;
    const int mine = lane < k ? L.sel[t * k + lane] : 0;
    const float sel = l[mine];
    const float vmax = lane_value(sel, 0);  // the first is the largest
    float z = (lane < E ? expf(v0 - vmax) : 0.0f) + (kWave + lane < E ? expf(v1 - vmax) : 0.0f);
    for (int e = 2 * kWave + lane; e < E; e += kWave) z += expf(l[e] - vmax);
    z = wave_sum(z);
    const float p = lane < k ? expf(sel - vmax) / z : 0.0f;
    const float den = row_sum(p) + 1e-20f;  // k <= 16: all of p lies in the first row
    if (lane < k) {
      const int pair = t * k + lane;
      L.weight[pair] = p / den;
    }
  }
}

// The experts of all tokens, and the lists of the pairs by expert. A row's
// place in its expert's list changes no result: every row is summed on its
// own, a token's experts in expert order.
template <int TILES, int NC>
__device__ __forceinline__ void few_select(const FewParams& P, FewLists& L, FewScratch<TILES>& S) {
  const int tid = threadIdx.x, lane = tid % kWave;
  const int E = P.E, pairs = P.T * P.k;
  if constexpr (TILES == 1) few_select_waves<(NC + 3) / 4>(P, L);
  else few_select_rows<NC>(P, L);
  __syncthreads();
  if (pairs <= kWave) {  // one wavefront, a pair per lane
    if (tid < kWave) {
      const int mine = lane < pairs ? L.sel[lane] : 0xffff;
      int at = 0, a = 0;
      bool repeat = false;
      for (int i = 0; i < pairs; ++i) {
        const int other = __builtin_amdgcn_readlane(mine, i);
        at += other < mine || (other == mine && i < lane);
        repeat |= other == mine && i < lane;
      }
      const uint64_t firsts = __ballot(lane < pairs && !repeat);
      for (int i = 0; i < pairs; ++i) a += __builtin_amdgcn_readlane(mine, i) < mine && (firsts >> i & 1);
      if (lane < pairs) {
        L.list[at] = static_cast<uint16_t>(lane);
        L.token[at] = static_cast<uint16_t>(lane / P.k);
        if (!repeat) {
          L.expert[a] = static_cast<uint16_t>(mine);
          L.start[a] = static_cast<uint16_t>(at);
        }
      }
      if (lane == 0) {
        L.na = __builtin_popcountll(firsts);
        L.start[__builtin_popcountll(firsts)] = static_cast<uint16_t>(pairs);
      }
    }
    __syncthreads();
    return;
  }
  for (int e = tid; e < E; e += kThreads) S.lists.count[e] = 0;
  __syncthreads();
  for (int q = tid; q < pairs; q += kThreads) atomicAdd(&S.lists.count[L.sel[q]], 1);
  __syncthreads();
  // Active experts in order, with their list starts: a scan over the experts,
  // two per thread, of (active, pairs) packed into one word.
  const int e0 = 2 * tid;
  const int c0 = e0 < E ? S.lists.count[e0] : 0, c1 = e0 + 1 < E ? S.lists.count[e0 + 1] : 0;
  const int mine = ((c0 > 0) + (c1 > 0)) << 16 | (c0 + c1);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += up;
  }
  if (lane == kWave - 1) S.lists.wave_sum[tid / kWave] = incl;
  __syncthreads();
  int before = incl - mine;
  for (int w = 0; w < tid / kWave; ++w) before += S.lists.wave_sum[w];
  int a = before >> 16, p = before & 0xffff;
  if (c0 > 0) {
    L.expert[a] = static_cast<uint16_t>(e0);
    L.start[a++] = static_cast<uint16_t>(p);
    S.lists.count[e0] = p;
    p += c0;
  }
  if (c1 > 0) {
    L.expert[a] = static_cast<uint16_t>(e0 + 1);
    L.start[a++] = static_cast<uint16_t>(p);
    S.lists.count[e0 + 1] = p;
    p += c1;
  }
  if (tid == kThreads - 1) {
    L.na = a;
    L.start[a] = static_cast<uint16_t>(p);
  }
  __syncthreads();
  for (int q = tid; q < pairs; q += kThreads) {
    const int at = atomicAdd(&S.lists.count[L.sel[q]], 1);
    L.list[at] = static_cast<uint16_t>(q);
    L.token[at] = static_cast<uint16_t>(q / P.k);
  }
  __syncthreads();
}

// Experts per group of the down phase: up to 8 selected experts, one group
// and no partial sums; beyond 64, groups of 16 halve the partial sums.
__host__ __device__ __forceinline__ int few_group(int na) { return na > 64 ? 16 : 8; }

// Claims of gate/up shares, handled by wavefront 0 (lane 0 claims, lanes 0 to
// 7 look at the counters). Counter l hands out shares l, l + 8, ..., n of them
// in all.
struct Claims {
  int list;          // the counter that is asked
  uint32_t ticket;   // lane 0: its answer
  uint32_t seen;     // lane l: counter l at that time

  static __device__ __forceinline__ uint32_t add(uint32_t* c) {
    uint32_t v = 0;
    if (threadIdx.x % kWave == 0) v = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return v;
  }
  static __device__ __forceinline__ int size(int n, int list) { return (n - list + kLists - 1) / kLists; }
  __device__ __forceinline__ void request(const FewParams& P) {
    ticket = add(P.cnt + list * kLine);
    const int l = threadIdx.x % kWave;
    if (l < kLists) seen = __hip_atomic_load(P.cnt + l * kLine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // The requested share, or -1 once all are claimed. A counter that has run
  // out is left for one that had not at the last look.
  __device__ __forceinline__ int take(const FewParams& P, int n) {
    for (;;) {
      const int t = __builtin_amdgcn_readfirstlane(min(ticket, 0x7fffffffu));
      if (t < size(n, list)) return t * kLists + list;
      const int l = threadIdx.x % kWave;
      const uint64_t open = __ballot(l < kLists && l != list && seen < static_cast<uint32_t>(size(n, l)));
      if (open == 0) return -1;
      list = __builtin_ctzll(open);
      request(P);
    }
  }
};

// Waits until *p reaches `want`; false after `polls` looks at it (a count of
// the wavefront's own, so that time in which it is suspended does not pass).
__device__ __forceinline__ bool wait_count(const uint32_t* p, uint32_t want, uint32_t polls) {
  bool there = false;
  for (uint32_t n = 0; n < polls && !there; ++n) {
    there = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= want;
    if (!there) __builtin_amdgcn_s_sleep(1);
  }
  asm volatile("" ::: "memory");  // what follows is read after it
  return there;
}

// TILES: 16-row tiles of one expert's tokens (one for T <= 16, else four); XR:
// the token rows whose values travel with the weights (an expert's further
// rows are loaded when their step is multiplied); NB: steps per batch (two
// batches are in flight per wavefront); NC: logits per lane of a 16-lane row
// (E <= 16 NC).
template <int FMT, int TILES, int XR, int NB, int NC>
__global__ __launch_bounds__(kThreads, 2) void few_kernel(const FewParams P) {
  constexpr int ESZ = FMT == kBf16 ? 2 : 1;
  constexpr int RPI = kRPI<FMT>, XN = XR / RPI;
  // A gate/up unit: GW times 8 columns, each 8 split along k over KW
  // wavefronts. Two share a unit's end and its barrier, at twice the loads of
  // token rows (us, one / two: 64 tokens in bf16 266 / 259, 33 in E4M3 184 / 174
  // at 128 experts, k = 8); not for a few units (1 token, E4M3: 34 / 43), nor
  // where the token rows are many (64 tokens, 8 experts, k = 2: 58 / 83).
  constexpr int GW = TILES > 1 && XR == 8 ? 2 : 1, GC = kGC * GW, KW = kNW / GW;
  constexpr int kBatchLoads = NB * (2 + XN);
  __shared__ FewLists L;
  __shared__ __attribute__((aligned(16))) FewScratch<TILES> S;
  __shared__ __attribute__((aligned(16))) char step_lds[kNW][kStepBytes<FMT>];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane % 16, g = lane / 16;
  const int wr = lane / 8, wc = lane % 8, xrow = lane / kXL<FMT>, xc = lane % kXL<FMT>;
  const int T = P.T, H = P.H, I = P.I, k = P.k;
  char* lds = step_lds[wave];

  const int shares = gridDim.x;
  Claims claims{static_cast<int>(blockIdx.x % kLists), 0, 0};
  if (wave == 0) claims.request(P);
  few_select<TILES, NC>(P, L, S);
  const int na = L.na, size = few_group(na), ngrp = (na + size - 1) / size;
  const int part = wave / KW, kw = wave % KW;  // columns and reduction part of a gate/up unit
  const int gpe = I / GC, dpg = H / kDC;  // gate/up units per expert, down units per group
  const int hsteps = (H + kStep<FMT> - 1) / kStep<FMT>, spe = (I + kStep<FMT> - 1) / kStep<FMT>;
  const bool hhalf = H % kStep<FMT> != 0, ihalf = I % kStep<FMT> != 0;
  const int down = ngrp * dpg;
  // The next share (barriers for all).
  auto claim = [&]() {
    if (wave == 0) {
      const int share = claims.take(P, shares);
      if (lane == 0) L.share = share;
      if (share >= 0) claims.request(P);  // the one after, answered long before it is asked for
    }
    __syncthreads();
    const int share = __builtin_amdgcn_readfirstlane(L.share);
    lds_barrier();  // everyone has read it
    return share;
  };

  const rsrc_t xs = make_rsrc(P.x, static_cast<int64_t>(T) * H * 2);
  Step<FMT, XR> st[2][NB];
  float sa[2] = {1.0f, 1.0f}, sb[2] = {1.0f, 1.0f};  // E4M3: lane d, the scales of the batch's step d
  f32x4 acc[TILES];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[t] = f32x4{};
  };
  auto load_b128 = [&](auto scope, const rsrc_t& r, uint32_t off) __attribute__((always_inline)) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, decltype(scope)::value));
  };
  bool weighed = false;
  typedef std::integral_constant<int, 0> Cached;
  typedef std::integral_constant<int, kDeviceScope> Fresh;

  // The product of the step in LDS with row tile t.
  auto multiply_tile = [&](int t, float f) __attribute__((always_inline)) {
    if (TILES == 1 || t == 0) multiply<FMT>(acc[0], lds, f);
    else if (t == 1) multiply<FMT>(acc[TILES > 1 ? 1 : 0], lds, f);
    else if (t == 2) multiply<FMT>(acc[TILES > 1 ? 2 : 0], lds, f);
    else multiply<FMT>(acc[TILES > 1 ? 3 : 0], lds, f);
  };
  // ---- gate/up units: the steps [q0, q1) of each are this wavefront's
  const int q0 = kw * hsteps / KW, q1 = (kw + 1) * hsteps / KW;
  const int batches = ((hsteps + KW - 1) / KW + NB - 1) / NB;  // the same for all wavefronts
  // Batch j of unit u into set B (u < 0: reads nothing).
  auto fetch = [&](auto setc, int u, int j) __attribute__((always_inline)) {
    constexpr int B = decltype(setc)::value;
    const int v = max(u, 0), a = v / gpe, c = v - a * gpe, e = L.expert[a], first = L.start[a];
    const int rows = u < 0 ? 0 : L.start[a + 1] - first;
    const int64_t at = (static_cast<int64_t>(e) * I + c * GC + part * kGC) * H * ESZ;
    const rsrc_t r0 = make_rsrc(static_cast<const char*>(P.w0) + at, u < 0 ? 0 : kGC * H * ESZ);
    const rsrc_t r1 = make_rsrc(static_cast<const char*>(P.w1) + at, u < 0 ? 0 : kGC * H * ESZ);
    const uint32_t wo = static_cast<uint32_t>(wr) * H * ESZ + 16 * wc;
    uint32_t xo[XN];
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int row = xrow + RPI * i;
      xo[i] = row < rows ? static_cast<uint32_t>(L.token[first + row]) * H * 2 + 16 * xc : kNoRow;
    }
    const int qb = q0 + j * NB;
#pragma unroll
    for (int d = 0; d < NB; ++d) {
      const int q = qb + d;
      const bool half = hhalf && q == hsteps - 1;
      const uint32_t wd = q >= q1 || (half && wc >= 4) ? kNoRow : wo + q * 128;
      st[B][d].w[0] = load_b128(Cached{}, r0, wd);
      st[B][d].w[1] = load_b128(Cached{}, r1, wd);
      const uint32_t xd = q >= q1 || (half && xc >= kXL<FMT> / 2) ? kNoRow : static_cast<uint32_t>(q) * (2 * kStep<FMT>);
#pragma unroll
      for (int i = 0; i < XN; ++i) st[B][d].x[i] = load_b128(Cached{}, xs, (xd & kNoRow) | (xo[i] + xd));
    }
    if constexpr (FMT == kFp8) {
      const int64_t sc = (static_cast<int64_t>(e) * ((I + 127) / 128) + c * GC / 128) * hsteps +
                         min(qb + lane % NB, hsteps - 1);
      sa[B] = P.s0[sc];
      sb[B] = P.s1[sc];
    }
  };
  // The products of batch j of unit u, in set B.
  auto use = [&](auto setc, int u, int j) __attribute__((always_inline)) {
    constexpr int B = decltype(setc)::value;
    const int a = u / gpe, first = L.start[a], rows = L.start[a + 1] - first;
#pragma unroll
    for (int d = 0; d < NB; ++d) {
      float f = 1.0f;
      if constexpr (FMT == kFp8) {
        const float fg = lane_value(sa[B], d), fu = lane_value(sb[B], d);
        f = lane < 32 ? fg : fu;  // result rows 8 .. 15 are up's
      }
      put_w(lds, st[B][d].w);
      put_x<FMT>(lds, st[B][d].x, 0);
      const int q = q0 + j * NB + d;
      int t = 0;
      // Past the wavefront's steps nothing is multiplied: its zeros would meet
      // rows that an earlier unit left in LDS, and zero times their NaN is NaN.
      if (q < q1) {
        for (int r0 = XR; r0 < rows; r0 += XR) {
          if (r0 % 16 == 0) multiply_tile(t++, f);
          u32x4 x[XN];
#pragma unroll
          for (int i = 0; i < XN; ++i) {
            const int row = r0 + xrow + RPI * i;
            const bool dead = row >= rows || (hhalf && q == hsteps - 1 && xc >= kXL<FMT> / 2);
            x[i] = load_b128(Cached{}, xs,
                             dead ? kNoRow
                                  : static_cast<uint32_t>(L.token[first + row]) * H * 2 + 16 * xc + q * (2 * kStep<FMT>));
          }
          put_x<FMT>(lds, x, r0 % 16);
        }
        multiply_tile(t, f);
      }
    }
  };
  // A unit's end: the partial sums to LDS; wavefront t then sums row tile t,
  // in wavefront order, two columns of a row per lane.
  uint32_t* pending = nullptr;  // counter of a tile whose stores may still be under way
  int turn = 0;
  auto finish = [&](int u) __attribute__((always_inline)) {
    const int a = u / gpe, c = u - a * gpe, first = L.start[a], rows = L.start[a + 1] - first, tiles = (rows + 15) / 16;
    if (pending != nullptr) {  // older than the last batch's loads
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0F70 | (kBatchLoads & 15) | (kBatchLoads >> 4) << 14);  // vmcnt(kBatchLoads)
      asm volatile("" ::: "memory");
      Claims::add(pending);
      pending = nullptr;
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t)
      if (t < tiles) *reinterpret_cast<f32x4*>(&S.red[turn][t][wave][col][4 * g]) = acc[t];
    lds_barrier();
    if (kw < tiles) {
      const int t = kw < TILES ? kw : 0, row = lane / 4, c0 = 2 * (lane % 4);
      float2 vg = make_float2(0.0f, 0.0f), vu = vg;
#pragma unroll
      for (int v = 0; v < KW; ++v) {
        const float2 x = *reinterpret_cast<const float2*>(&S.red[turn][t][part * KW + v][row][c0]);
        const float2 y = *reinterpret_cast<const float2*>(&S.red[turn][t][part * KW + v][row][8 + c0]);
        vg.x += x.x;
        vg.y += x.y;
        vu.x += y.x;
        vu.y += y.y;
      }
      if (16 * t + row < rows) {
        const int pair = L.list[first + 16 * t + row];
        const float pw = L.weight[pair];
        __hip_atomic_store(reinterpret_cast<uint32_t*>(P.act + static_cast<int64_t>(pair) * I + c * GC + part * kGC + c0),
                           pack_bf16x2(pw * (vg.x * sigmoidf_dev(vg.x) * vu.x), pw * (vg.y * sigmoidf_dev(vg.y) * vu.y)),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      pending = P.cnt + (kLists + a / size) * kLine;
    }
    turn ^= 1;
  };
  {
    typedef std::integral_constant<int, 0> Set0;
    typedef std::integral_constant<int, 1> Set1;
    const int units = na * gpe;
    for (int share = claim(); share >= 0; share = claim()) {
      int u = share < units ? share : -1;
      auto after = [&](int v) { return v >= 0 && v + shares < units ? v + shares : -1; };
      int un = after(u);
      fetch(Set0{}, u, 0);
      if (batches > 1) fetch(Set1{}, u, 1);
      else fetch(Set1{}, un, 0);
      clear();
      if (TILES == 1 && !weighed) few_weights(P, L);
      weighed = true;
      if (share == 0) {  // the routing's outputs
        __syncthreads();
        for (int i = tid; i < T * k; i += kThreads) {
          P.topk_idx[i] = L.sel[i];
          P.topk_w[i] = L.weight[i];
        }
      }
      int j = 0;
      auto turn_over = [&](auto setc) __attribute__((always_inline)) {
        use(setc, u, j);
        if (++j == batches) {
          finish(u);
          u = un;
          un = after(u);
          j = 0;
          clear();
        }
        // The set just used takes the batch after the next: batch j + 1 of u,
        // or the first of its successor.
        const int f = j + 1;
        fetch(setc, f < batches ? u : un, f < batches ? f : 0);
      };
      while (u >= 0) {
        turn_over(Set0{});
        if (u < 0) break;
        turn_over(Set1{});
      }
    }
    if (pending != nullptr) {  // before this workgroup waits for others
      stores_done();
      Claims::add(pending);
    }
  }

  // ---- down units
  __syncthreads();
  const rsrc_t act = make_rsrc(P.act, static_cast<int64_t>(T) * k * I * 2);
  for (int u = blockIdx.x; u < down; u += gridDim.x) {
    const int grp = u / dpg, c = u - grp * dpg, a0 = grp * size, a_end = a0 + min(size, na - a0);
    const int total = (a_end - a0) * spe, d0 = wave * total / kNW, d1 = (wave + 1) * total / kNW;
    // Cursors over the group's steps, expert by expert: of the weights'
    // loads, the activations' and the products.
    struct Cursor {
      int q, a, s;
    };
    Cursor cw{d0, a0 + d0 / spe, d0 % spe}, cx = cw, cu = cw;
    const uint32_t wo = static_cast<uint32_t>(wr) * I * ESZ + 16 * wc;
    auto weights_of = [&](int a) {
      return make_rsrc(static_cast<const char*>(P.w2) + (static_cast<int64_t>(L.expert[a]) * H + c * kDC) * I * ESZ,
                       kDC * I * ESZ);
    };
    rsrc_t rw = cw.q < d1 ? weights_of(cw.a) : make_rsrc(P.w2, 0);
    float sc[2][NB];  // E4M3: the steps' scales
    auto fetch_w = [&](auto setc) __attribute__((always_inline)) {
      constexpr int B = decltype(setc)::value;
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        const uint32_t o = ihalf && cw.s == spe - 1 && wc >= 4 ? kNoRow : wo + cw.s * 128;
        st[B][d].w[0] = load_b128(Cached{}, rw, o);
        st[B][d].w[1] = load_b128(Cached{}, rw, o + 8 * I * ESZ);
        if constexpr (FMT == kFp8)
          sc[B][d] = P.s2[(static_cast<int64_t>(L.expert[min(cw.a, a_end - 1)]) * ((H + 127) / 128) + c * kDC / 128) * spe +
                          cw.s];
        if (++cw.s == spe) {
          cw.s = 0;
          if (++cw.a < a_end) rw = weights_of(cw.a);
        }
        if (++cw.q >= d1) rw = make_rsrc(P.w2, 0);
      }
    };
    // The activations' offsets of rows r0 on of active expert a.
    auto row_offsets = [&](int a, int r0, uint32_t(&o)[XN]) __attribute__((always_inline)) {
      const int f0 = L.start[a], n = L.start[a + 1] - f0;
#pragma unroll
      for (int i = 0; i < XN; ++i) {
        const int row = r0 + xrow + RPI * i;
        o[i] = row < n ? static_cast<uint32_t>(L.list[f0 + row]) * I * 2 + 16 * xc : kNoRow;
      }
    };
    auto row_loads = [&](const uint32_t(&o)[XN], int s, u32x4(&x)[XN]) __attribute__((always_inline)) {
      const uint32_t dead = ihalf && s == spe - 1 && xc >= kXL<FMT> / 2 ? kNoRow : 0;
#pragma unroll
      for (int i = 0; i < XN; ++i) x[i] = load_b128(Fresh{}, act, (o[i] | dead) + s * (2 * kStep<FMT>));
    };
    uint32_t xo[XN];
    auto fetch_x = [&](auto setc) __attribute__((always_inline)) {
      constexpr int B = decltype(setc)::value;
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        row_loads(xo, cx.s, st[B][d].x);
        if (++cx.s == spe) {
          cx.s = 0;
          if (++cx.a < a_end) row_offsets(cx.a, 0, xo);
        }
        if (++cx.q >= d1) {
#pragma unroll
          for (int i = 0; i < XN; ++i) xo[i] = kNoRow;
        }
      }
    };
    float* tile = &S.tile[wave][0][0];
    constexpr int TS = kDC + 4;
    int first = 0, rows = 0;
    auto open = [&](int a) __attribute__((always_inline)) {
      first = L.start[a];
      rows = L.start[a + 1] - first;
    };
    auto use_down = [&](auto setc) __attribute__((always_inline)) {
      constexpr int B = decltype(setc)::value;
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        if (cu.q < d1) {
          const float f = FMT == kFp8 ? sc[B][d] : 1.0f;
          put_w(lds, st[B][d].w);
          put_x<FMT>(lds, st[B][d].x, 0);
          int t = 0;
          for (int r0 = XR; r0 < rows; r0 += XR) {
            if (r0 % 16 == 0) multiply_tile(t++, f);
            uint32_t o[XN];
            u32x4 x[XN];
            row_offsets(cu.a, r0, o);
            row_loads(o, cu.s, x);
            put_x<FMT>(lds, x, r0 % 16);
          }
          multiply_tile(t, f);
          ++cu.q;
          if (++cu.s == spe || cu.q == d1) {  // this expert's products into the tile, row by row
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (16 * t + col < rows) {
                f32x4* to = reinterpret_cast<f32x4*>(tile + L.token[first + 16 * t + col] * TS + 4 * g);
                f32x4 v = *to;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += acc[t][i];
                *to = v;
              }
            }
            clear();
            cu.s = 0;
            if (cu.q < d1) open(++cu.a);
          }
        }
      }
    };
    typedef std::integral_constant<int, 0> Set0;
    typedef std::integral_constant<int, 1> Set1;
    fetch_w(Set0{});
    fetch_w(Set1{});
    auto fill = [&](float v) __attribute__((always_inline)) {
      for (int i = lane; i < T * kDC; i += kWave) tile[i / kDC * TS + i % kDC] = v;
    };
    fill(0.0f);
    // The group's activations are there once all its tiles are counted.
    uint32_t want = 0;
    for (int a = a0; a < a_end; ++a) want += (L.start[a + 1] - L.start[a] + 15) / 16 * gpe * GW;
    if (!wait_count(P.cnt + (kLists + grp) * kLine, want, P.polls)) fill(__builtin_nanf(""));
    if (cx.q < d1) {
      row_offsets(cx.a, 0, xo);
      open(cu.a);
    } else {
#pragma unroll
      for (int i = 0; i < XN; ++i) xo[i] = kNoRow;
    }
    fetch_x(Set0{});
    fetch_x(Set1{});
    clear();
    while (cu.q < d1) {
      use_down(Set0{});
      fetch_w(Set0{});
      fetch_x(Set0{});
      use_down(Set1{});
      fetch_w(Set1{});
      fetch_x(Set1{});
    }
    lds_barrier();
    for (int i = tid; i < T * kDC / 2; i += kThreads) {
      const int t = i / (kDC / 2), h = 2 * (i % (kDC / 2));
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int v = 0; v < kNW; ++v) {
        v0 += S.tile[v][t][h];
        v1 += S.tile[v][t][h + 1];
      }
      const int64_t at = static_cast<int64_t>(t) * H + c * kDC + h;
      if (ngrp == 1) {
        *reinterpret_cast<uint32_t*>(P.y + at) = pack_bf16x2(v0, v1);
      } else {
        uint64_t* to = reinterpret_cast<uint64_t*>(P.part + static_cast<int64_t>(grp) * T * H + at);
        __hip_atomic_store(to, static_cast<uint64_t>(__float_as_uint(v1)) << 32 | __float_as_uint(v0),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (ngrp > 1) {
      stores_done();
      lds_barrier();
      if (tid == 0)
        L.last = __hip_atomic_fetch_add(P.cnt_down + c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 static_cast<uint32_t>(ngrp) - 1;
      lds_barrier();
      if (L.last) {
        for (int i = tid; i < T * kDC / 2; i += kThreads) {
          const int64_t at = static_cast<int64_t>(i / (kDC / 2)) * H + c * kDC + 2 * (i % (kDC / 2));
          float v0 = 0.0f, v1 = 0.0f;
          for (int v = 0; v < ngrp; ++v) {
            const uint64_t b =
                __hip_atomic_load(reinterpret_cast<uint64_t*>(P.part + static_cast<int64_t>(v) * T * H + at),
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            v0 += __uint_as_float(static_cast<uint32_t>(b));
            v1 += __uint_as_float(static_cast<uint32_t>(b >> 32));
          }
          *reinterpret_cast<uint32_t*>(P.y + at) = pack_bf16x2(v0, v1);
        }
      }
    }
    lds_barrier();  // the tiles are free
  }
}

template <int FMT, int NC>
void launch_layer(const FewParams& P, unsigned grid, hipStream_t st) {
  // An expert has at most T rows, and T k / E on average: up to 4 on average,
  // few have more than 8. Rows loaded 8 / 16 at a time (us, 2048 x 768, bf16):
  // 128 experts, k = 8: 1 token 36.6 / 37.5, 16 tokens 164 / 172, 64 tokens
  // (4 rows each) 263 / 270; 32 experts, k = 8: 16 tokens (4 rows) 85.7 / 86.7,
  // 32 (8 rows) 97 / 89, 64 (16 rows) 128 / 116.
  constexpr int NB = FMT == kBf16 ? 4 : 2;
  const bool thin = P.T <= 8 || P.T * P.k <= 4 * P.E;
  if (P.T <= 16) {
    if (thin) few_kernel<FMT, 1, 8, NB, NC><<<grid, kThreads, 0, st>>>(P);
    else few_kernel<FMT, 1, 16, NB, NC><<<grid, kThreads, 0, st>>>(P);
  } else {
    if (thin) few_kernel<FMT, 4, 8, NB, NC><<<grid, kThreads, 0, st>>>(P);
    else few_kernel<FMT, 4, 16, NB, NC><<<grid, kThreads, 0, st>>>(P);
  }
}

int few_max_active(const moe_shape& s) { return s.T * s.k < s.E ? s.T * s.k : s.E; }
int few_max_groups(const moe_shape& s) {  // the most over the active counts: groups of 8 up to 64 experts
  const int na = few_max_active(s);
  return na <= 64 ? ceil_div(na, 8) : (ceil_div(na, 16) > 8 ? ceil_div(na, 16) : 8);
}

}  // namespace

FewLayout few_layout(const moe_shape& s) {
  FewLayout l{};
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  l.groups = few_max_groups(s);
  l.counters = (kLists + l.groups) * kLine + s.H / 16;
  l.act = up(static_cast<size_t>(l.counters) * 4);
  l.part = up(l.act + static_cast<size_t>(s.T) * s.k * s.I * 2);
  l.total = up(l.part + static_cast<size_t>(l.groups) * s.T * s.H * 4);
  return l;
}

hipError_t launch_few(const moe_shape& s, const FewArgs& a, void* ws, hipStream_t st) {
  const FewLayout l = few_layout(s);
  char* base = static_cast<char*>(ws);
  FewParams P{};
  P.T = s.T;
  P.H = s.H;
  P.E = s.E;
  P.k = s.k;
  P.I = s.I;
  P.x = static_cast<const bf16_t*>(a.x);
  P.w0 = a.w_gate;
  P.w1 = a.w_up;
  P.w2 = a.w_down;
  P.s0 = a.gate_scale;
  P.s1 = a.up_scale;
  P.s2 = a.down_scale;
  P.logits = a.logits;
  P.topk_idx = a.topk_idx;
  P.topk_w = a.topk_w;
  P.y = static_cast<bf16_t*>(a.y);
  P.polls = a.polls;
  P.cnt = reinterpret_cast<uint32_t*>(base);
  P.act = reinterpret_cast<bf16_t*>(base + l.act);
  P.part = reinterpret_cast<float*>(base + l.part);
  P.cnt_down = P.cnt + (kLists + l.groups) * kLine;
  const dim3 rg(static_cast<unsigned>(s.E), static_cast<unsigned>(ceil_div(s.T, kRouterTokens)));
  few_router_kernel<<<rg, kRouterWaves * kWave, 0, st>>>(s.T, s.H, s.E, P.x, static_cast<const bf16_t*>(a.w_router), a.bias, a.logits,
                                          P.cnt, l.counters);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const unsigned grid = static_cast<unsigned>(gemm_grid());
  if (a.gate_scale != nullptr) {
    if (s.E <= 128) launch_layer<kFp8, 8>(P, grid, st);
    else if (s.E <= 256) launch_layer<kFp8, 16>(P, grid, st);
    else launch_layer<kFp8, 64>(P, grid, st);
  } else {
    if (s.E <= 128) launch_layer<kBf16, 8>(P, grid, st);
    else if (s.E <= 256) launch_layer<kBf16, 16>(P, grid, st);
    else launch_layer<kBf16, 64>(P, grid, st);
  }
  return hipGetLastError();
}

}  // namespace moe
