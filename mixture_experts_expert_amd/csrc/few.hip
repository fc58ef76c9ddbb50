// The whole MoE layer for a few tokens (T <= 64), in two launches.
//
// With few tokens the layer is a walk over the selected experts' weights: each
// is read once from memory and multiplied by the handful of rows that chose
// it, so the kernel is bound by the weights' bytes and, for one token, by
// latency (75 MB at the 30B shape in bf16). Everything here serves that: the
// weights go straight from memory into registers in 16-byte loads, several
// steps ahead and on into the next unit; gate/up and down are one launch, so
// that the down weights' first loads are in flight while the last gate/up
// units finish; no activation row but the selected experts' (T k I bf16) is
// ever written.
//
//   few_router_kernel: logits, one wavefront per expert and 8 tokens. x and
//     w_router products are exact in fp32 (bf16 factors) and summed in fp64,
//     so the logit is the exact sum rounded once, whatever the split. It also
//     clears the second kernel's counters.
//   few_kernel: one persistent workgroup of 8 wavefronts per CU. Each selects
//     the experts of all tokens for itself (no third launch), then takes
//     units by ticket:
//     - gate/up unit: one expert, 8 F columns of gate and of up. The reduction
//       is split over the 8 wavefronts; the partial sums meet in LDS, and
//       a = bf16(w silu(g) u) goes to the workspace per (token, slot).
//     - down unit: one group of experts, 16 F columns of y. The (expert, k)
//       steps are split over the wavefronts, each adding its experts' products
//       into its own y tile in LDS; the eight tiles are then summed in order.
//       With one group (up to 8 experts) that is y; otherwise the groups'
//       fp32 partial sums go to the workspace and the last workgroup to
//       finish a column block adds them in group order.
//
// Order and progress: tickets come from 16 counters, 8 for gate/up and 8 for
// down (one counter would serialise the first 256 tickets, about 10 ns each).
// A workgroup starts at its own XCD's counter, and takes a down ticket only
// once all 8 gate/up counters have run out. A down unit waits for its group's
// gate/up units; by then running workgroups hold all of those, and gate/up
// units wait for nothing: the wait ends whatever else occupies the device.
// (If another call overwrites the workspace, against the interface, the wait
// gives up after two seconds.)
//
// Tile: v_mfma_f32_16x16x32_bf16 with the weights as A (16 rows; a gate/up
// fragment with F = 1 is 8 rows of gate and 8 of up) and up to 16 token rows
// as B, so a lane's four results are four consecutive columns of one row. A
// step is 64 k: lane group g = lane / 16 takes k 16 g .. 16 g + 15 of it (the
// first 8 in one product, the others in the next; any assignment of k to
// lanes serves as long as both operands share it), so a row's 128 bytes are
// read together. E4M3 weights are widened to bf16 (exact) in registers and
// each step's partial product is multiplied by its block's scale in fp32.
//
// In flight: 64 to 128 KB per CU. Twice that is slower (measured with two
// workgroups per CU: 64 instead of 43 us for one token at the 30B shape), as
// the units' stores and counters then queue behind everyone's weights.
#include "moe_internal.h"
#include "select.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBf16 = 0, kFp8 = 1;  // weight formats
constexpr int kNW = 8;              // wavefronts per workgroup
constexpr int kThreads = kNW * kWave;
constexpr int kStep = 64;           // k per step
constexpr int kLists = 8;           // ticket counters per phase, one per XCD
constexpr int kLine = 32;           // counters that workgroups add to lie 128 bytes apart
constexpr int kMaxPairs = kFewMaxT * kFewMaxK;
constexpr uint64_t kSpinTicks = 200000000;  // two seconds of the 100 MHz clock

// The workspace's counters (uint32, in lines): [0, 8) gate/up tickets, [8, 16)
// down tickets, then gate/up tiles done per group; after the lines, down units
// done per column block.
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

__global__ __launch_bounds__(kWave) void few_router_kernel(int T, int H, int E, const bf16_t* __restrict__ x,
                                                           const bf16_t* __restrict__ wr,
                                                           const float* __restrict__ bias, float* __restrict__ logits,
                                                           uint32_t* __restrict__ cnt, int ncnt) {
  const int e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
  const int lane = threadIdx.x;
  const int stride = gridDim.x * gridDim.y * kWave;
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * kWave + lane; i < ncnt; i += stride) cnt[i] = 0;
  double acc[kRouterTokens];
#pragma unroll
  for (int i = 0; i < kRouterTokens; ++i) acc[i] = 0.0;
  const uint4* w4 = reinterpret_cast<const uint4*>(wr + static_cast<int64_t>(e) * H);
  const int nt = min(kRouterTokens, T - t0);
#pragma unroll 2
  for (int c = lane; c < H / 8; c += kWave) {
    const uint4 wv = w4[c];
    const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int i = 0; i < kRouterTokens; ++i) {
      if (i >= nt) break;
      const uint4 xv = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t0 + i) * H)[c];
      const uint32_t xu[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[i] += static_cast<double>(__uint_as_float(xu[q] << 16) * __uint_as_float(wu[q] << 16));
        acc[i] += static_cast<double>(__uint_as_float(xu[q] & 0xffff0000u) * __uint_as_float(wu[q] & 0xffff0000u));
      }
    }
  }
  const double b = bias ? static_cast<double>(bias[e]) : 0.0;
#pragma unroll
  for (int i = 0; i < kRouterTokens; ++i) {
    if (i >= nt) break;
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) acc[i] += __shfl_xor(acc[i], o, kWave);
    if (lane == 0) logits[static_cast<int64_t>(t0 + i) * E + e] = static_cast<float>(acc[i] + b);
  }
}

// ---- the layer --------------------------------------------------------------

// 16 weight rows' share of one step, in the lane that multiplies it.
template <int FMT> struct Frag;
template <> struct Frag<kBf16> {
  uint4 v[2];
  // p: this lane's row, at k = 16 g of step 0
  __device__ __forceinline__ void load(const void* p, int s) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const bf16_t*>(p) + s * kStep);
    v[0] = q[0];
    v[1] = q[1];
  }
  __device__ __forceinline__ bf16x8 half(int h) const { return __builtin_bit_cast(bf16x8, v[h]); }
};
template <> struct Frag<kFp8> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, int s) {
    v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + s * kStep);
  }
  __device__ __forceinline__ bf16x8 half(int h) const {
    const uint32_t a = h ? v.z : v.x, b = h ? v.w : v.y;
    const bf16x2 r0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2 r1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2 r2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2 r3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf16x8{r0.x, r0.y, r1.x, r1.y, r2.x, r2.y, r3.x, r3.y};
  }
};

struct Rows {  // a token row's share of one step
  uint4 v[2];
  __device__ __forceinline__ void load(const bf16_t* p, int s) {
    const uint4* q = reinterpret_cast<const uint4*>(p + s * kStep);
    v[0] = q[0];
    v[1] = q[1];
  }
  __device__ __forceinline__ void load(const rsrc_t& r, uint32_t off, int s) {  // another workgroup's row
    const uint32_t o = off + static_cast<uint32_t>(s) * (kStep * 2);
    v[0] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, kDeviceScope));
    v[1] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, o + 16, 0, kDeviceScope));
  }
  __device__ __forceinline__ bf16x8 half(int h) const { return __builtin_bit_cast(bf16x8, v[h]); }
};

// acc += (scale) W rows x token rows over one step.
template <int FMT>
__device__ __forceinline__ void multiply(f32x4& acc, const Frag<FMT>& w, const Rows& r, float scale) {
  if constexpr (FMT == kBf16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.half(0), r.half(0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.half(1), r.half(1), acc, 0, 0, 0);
  } else {
    f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.half(0), r.half(0), f32x4{}, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.half(1), r.half(1), p, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(scale, p[i], acc[i]);
  }
}

__device__ __forceinline__ float lane_value(float v, int src) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), src));
}

struct FewLists {  // in LDS: the pairs (token, slot) sorted by expert
  int na;                          // experts that some token selected
  int unit;                        // the next unit
  int last;
  uint16_t expert[1024];           // active expert a -> expert
  uint16_t start[1025];            // its pairs: list[start[a] .. start[a + 1])
  uint16_t list[kMaxPairs];        // pair t * k + j
  float weight[kMaxPairs];         // by pair
};

// Scratch, reused by the phases of a unit.
template <int TILES, int F>
union FewScratch {
  struct {
    uint16_t sel[kMaxPairs];       // expert of each pair
    int count[1024];               // pairs per expert, then a cursor
    int wave_sum[kNW];
  } lists;
  float red[TILES][kNW][16][16 * F + 4];      // gate/up: [tile][wave][row][gate columns, up columns]
  float tile[kNW][16 * TILES][16 * F + 4];    // down: [wave][token][column]
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
// largest, then the lowest index that has it, and marks that one as taken.
template <int NC, class S_t>
__device__ __forceinline__ void few_select_rows(const FewParams& P, FewLists& L, S_t& S) {
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
      const int pair = t * k + n;
      S.lists.sel[pair] = static_cast<uint16_t>(sel_i);
      L.weight[pair] = p / den;
      if (blockIdx.x == 0) {
        P.topk_idx[pair] = sel_i;
        P.topk_w[pair] = p / den;
      }
    }
  }
}

// Selection for up to 16 tokens: a wavefront per token, logits lane + 64 c.
// The rounds are the same; the lowest index comes from a ballot.
template <int NC, class S_t>
__device__ __forceinline__ void few_select_waves(const FewParams& P, FewLists& L, S_t& S) {
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
    float sel_v = 0.0f, vmax = 0.0f;
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
      const float bv = key_value(static_cast<uint64_t>(m) << 32);
      if (j == 0) vmax = bv;
      if (lane == j) {
        sel_v = bv;
        sel_i = at;
      }
    }
    const float top = lane < k ? expf(sel_v - vmax) : 0.0f;
    float z = top;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (left >> c & 1) z += expf(key_value(static_cast<uint64_t>(o[c]) << 32) - vmax);
    z = wave_sum(z);
    const float p = top / z;
    const float den = row_sum(p) + 1e-20f;  // k <= 16: all of p lies in the first row
    if (lane < k) {
      const int pair = t * k + lane;
      S.lists.sel[pair] = static_cast<uint16_t>(sel_i);
      L.weight[pair] = p / den;
      if (blockIdx.x == 0) {
        P.topk_idx[pair] = sel_i;
        P.topk_w[pair] = p / den;
      }
    }
  }
}

// The experts of all tokens, and the lists of the pairs by expert. A row's
// place in its expert's list changes no result: every row is summed on its
// own, a token's experts in expert order.
template <int TILES, int F, int NC>
__device__ __forceinline__ void few_select(const FewParams& P, FewLists& L, FewScratch<TILES, F>& S) {
  const int tid = threadIdx.x, lane = tid % kWave;
  const int E = P.E, pairs = P.T * P.k;
  if constexpr (TILES == 1) few_select_waves<(NC + 3) / 4>(P, L, S);
  else few_select_rows<NC>(P, L, S);
  __syncthreads();
  if (pairs <= kWave) {  // one wavefront, a pair per lane
    if (tid < kWave) {
      const int mine = lane < pairs ? S.lists.sel[lane] : 0xffff;
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
  for (int q = tid; q < pairs; q += kThreads) atomicAdd(&S.lists.count[S.lists.sel[q]], 1);
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
  for (int q = tid; q < pairs; q += kThreads)
    L.list[atomicAdd(&S.lists.count[S.lists.sel[q]], 1)] = static_cast<uint16_t>(q);
  __syncthreads();
}

// Experts per group of the down phase: up to 8 selected experts, one group
// and no partial sums; beyond 64, groups of 16 halve the partial sums.
__host__ __device__ __forceinline__ int few_group(int na) { return na > 64 ? 16 : 8; }

// Tickets (thread 0). list_size: units u = list, list + 8, ... below n.
__device__ __forceinline__ int list_size(int n, int list) { return (n - list + kLists - 1) / kLists; }

struct Tickets {
  int gu, down;    // units of each phase
  int phase, list;
  uint32_t ticket; // requested of the current list
  __device__ __forceinline__ uint32_t* counter(const FewParams& P, int l) const {
    return P.cnt + (phase * kLists + l) * kLine;
  }
  __device__ __forceinline__ void request(const FewParams& P) {
    ticket = __hip_atomic_fetch_add(counter(P, list), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // The unit of the requested ticket: a gate/up unit, gu + a down unit, or -1.
  // A list that has run out is left for one that still has units.
  __device__ __forceinline__ int take(const FewParams& P) {
    for (;;) {
      const int n = phase == 0 ? gu : down;
      if (ticket < static_cast<uint32_t>(list_size(n, list))) return phase * gu + static_cast<int>(ticket) * kLists + list;
      uint32_t c[kLists];
#pragma unroll
      for (int l = 0; l < kLists; ++l)
        c[l] = __hip_atomic_load(counter(P, l), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      int next = -1;
#pragma unroll
      for (int l = kLists - 1; l >= 0; --l)
        if (c[l] < static_cast<uint32_t>(list_size(n, l))) next = l;
      if (next >= 0) {
        list = next;
      } else if (phase == 0) {
        phase = 1;
        list = blockIdx.x % kLists;
      } else {
        return -1;
      }
      request(P);
    }
  }
};

// Waits until *p reaches `want` (one thread; the caller's barrier follows).
__device__ __forceinline__ void wait_count(const uint32_t* p, uint32_t want) {
  const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
  while (__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < want) {
    if (__builtin_amdgcn_s_memrealtime() - t0 > kSpinTicks) break;
    __builtin_amdgcn_s_sleep(1);
  }
}

// TILES: 16-row tiles of one expert's tokens (one for T <= 16, else four); F:
// weight fragments per step; AHEAD: steps of weights in flight per wavefront;
// NC: logits per lane of a 16-lane row (E <= 16 NC).
template <int FMT, int TILES, int F, int AHEAD, int NC>
__global__ __launch_bounds__(kThreads, 2) void few_kernel(const FewParams P) {
  constexpr int GC = 8 * F, DC = 16 * F;  // columns per gate/up and per down unit
  constexpr int ESZ = FMT == kBf16 ? 2 : 1;
  __shared__ FewLists L;
  __shared__ __attribute__((aligned(16))) FewScratch<TILES, F> S;
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane % 16, g = lane / 16;
  const int T = P.T, H = P.H, I = P.I, k = P.k;

  Tickets tk{};
  tk.list = blockIdx.x % kLists;
  if (tid == 0) tk.request(P);
  few_select<TILES, F, NC>(P, L, S);
  const int na = L.na, size = few_group(na), ngrp = (na + size - 1) / size;
  tk.gu = na * (I / GC);
  tk.down = ngrp * (H / DC);
  if (tid == 0) L.unit = tk.take(P);
  __syncthreads();

  // The stream of a unit's steps: this wavefront's steps q of [q0, q1), its
  // weights in w and the first 16 rows' values in r, AHEAD steps deep. The
  // load cursors (p, left, la for weights; pr for x) are ahead of the
  // multiplications.
  Frag<FMT> w[AHEAD][F];
  Rows r[AHEAD];
  const char* p[F];
  const bf16_t* pr = nullptr;
  int q0 = 0, q1 = 0, left = 0, la = 0;
  float sa = 1.0f, sb = 1.0f;            // E4M3: lane l holds the scales of step l (of the current 64)
  const int spe = I / kStep;             // down: steps per expert
  const int gpe = I / GC, dpg = H / DC;  // gate/up units per expert, down units per group
  const rsrc_t act = make_rsrc(P.act, static_cast<int64_t>(T) * k * I * 2);

  auto load_w = [&](int d) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      w[d][f].load(p[f], 0);
      p[f] += kStep * ESZ;
    }
  };
  auto down_rows = [&](int c, int a) __attribute__((always_inline)) {  // weight rows of active expert a
#pragma unroll
    for (int f = 0; f < F; ++f)
      p[f] = static_cast<const char*>(P.w2) +
             ((static_cast<int64_t>(L.expert[a]) * H + c * DC + 16 * f + col) * I + 16 * g) * ESZ;
  };
  // The finished unit: its partial results are in the scratch.
  int fin = -1;
  uint32_t* pending = nullptr;  // counter of a gate/up tile whose stores may still be under way
  auto signal = [&]() __attribute__((always_inline)) {
    if (pending != nullptr) {
      stores_done();
      if (lane == 0) __hip_atomic_fetch_add(pending, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      pending = nullptr;
    }
  };
  // A gate/up unit: wavefront t sums the partial products of row tile t, in
  // wavefront order: 2 F columns of one row per lane.
  auto finish_gate_up = [&](int v) __attribute__((always_inline)) {
    const int a = v / gpe, c = v - a * gpe;
    const int first = L.start[a], rows = L.start[a + 1] - first;
    if (16 * wave >= rows) return;
    const int row = lane / 4, c0 = 2 * F * (lane % 4);
    float vg[2 * F], vu[2 * F];
#pragma unroll
    for (int i = 0; i < 2 * F; ++i) vg[i] = vu[i] = 0.0f;
#pragma unroll
    for (int x = 0; x < kNW; ++x)
#pragma unroll
      for (int i = 0; i < 2 * F; ++i) {
        vg[i] += S.red[wave < TILES ? wave : 0][x][row][c0 + i];
        vu[i] += S.red[wave < TILES ? wave : 0][x][row][GC + c0 + i];
      }
    if (16 * wave + row < rows) {
      const int pair = L.list[first + 16 * wave + row];
      const float pw = L.weight[pair];
#pragma unroll
      for (int i = 0; i < 2 * F; ++i) vg[i] = pw * (vg[i] * sigmoidf_dev(vg[i]) * vu[i]);
      const int64_t at = static_cast<int64_t>(pair) * I + c * GC + c0;
#pragma unroll
      for (int i = 0; i < F; ++i)
        __hip_atomic_store(reinterpret_cast<uint32_t*>(P.act + at + 2 * i), pack_bf16x2(vg[2 * i], vg[2 * i + 1]),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    pending = P.cnt + (2 * kLists + a / size) * kLine;
  };
  // A down unit: the wavefronts' tiles, in order.
  auto finish_down = [&](int v) __attribute__((always_inline)) {
    const int grp = (v - tk.gu) / dpg, c = v - tk.gu - grp * dpg;
    for (int i = tid; i < T * DC / 2; i += kThreads) {
      const int t = i / (DC / 2), h = 2 * (i % (DC / 2));
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int x = 0; x < kNW; ++x) {
        v0 += S.tile[x][t][h];
        v1 += S.tile[x][t][h + 1];
      }
      const int64_t at = static_cast<int64_t>(t) * H + c * DC + h;
      if (ngrp == 1) {
        *reinterpret_cast<uint32_t*>(P.y + at) = pack_bf16x2(v0, v1);
      } else {
        uint64_t* to = reinterpret_cast<uint64_t*>(P.part + static_cast<int64_t>(grp) * T * H + at);
        __hip_atomic_store(to, static_cast<uint64_t>(__float_as_uint(v1)) << 32 | __float_as_uint(v0),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (ngrp == 1) return;
    stores_done();
    lds_barrier();
    if (tid == 0)
      L.last = __hip_atomic_fetch_add(P.cnt_down + c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               static_cast<uint32_t>(ngrp) - 1;
    lds_barrier();
    if (!L.last) return;
    for (int i = tid; i < T * DC / 2; i += kThreads) {
      const int64_t at = static_cast<int64_t>(i / (DC / 2)) * H + c * DC + 2 * (i % (DC / 2));
      float v0 = 0.0f, v1 = 0.0f;
      for (int x = 0; x < ngrp; ++x) {
        const uint64_t b =
            __hip_atomic_load(reinterpret_cast<uint64_t*>(P.part + static_cast<int64_t>(x) * T * H + at),
                              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v0 += __uint_as_float(static_cast<uint32_t>(b));
        v1 += __uint_as_float(static_cast<uint32_t>(b >> 32));
      }
      *reinterpret_cast<uint32_t*>(P.y + at) = pack_bf16x2(v0, v1);
    }
  };

  int u = __builtin_amdgcn_readfirstlane(L.unit);
  for (;;) {
    // First loads of unit u, then the finished unit's results.
    const bool down = u >= tk.gu;
    int first = 0, rows = 0, tiles = 0;  // the expert whose steps are multiplied
    int grp = 0, c = 0, a0 = 0, a_end = 0;
    auto scales = [&](int q) __attribute__((always_inline)) {
      if constexpr (FMT == kFp8) {
        if (!down) {
          const int kb = (H + 127) / 128;
          const int64_t at = (static_cast<int64_t>(L.expert[a0]) * ((I + 127) / 128) + c * GC / 128) * kb;
          const int b = min((q + lane) / 2, kb - 1);
          sa = P.s0[at + b];
          sb = P.s1[at + b];
        } else {
          const int kb = (I + 127) / 128, s = min(q + lane, (a_end - a0) * spe - 1);
          sa = P.s2[(static_cast<int64_t>(L.expert[a0 + s / spe]) * ((H + 127) / 128) + c * DC / 128) * kb +
                    s % spe / 2];
        }
      }
    };
    // The next step's weights into slot d; a down unit's cursor moves on to
    // the group's next expert.
    auto load_down = [&](int d) __attribute__((always_inline)) {
      load_w(d);
      if (--left == 0) {
        left = spe;
        if (++la < a_end) down_rows(c, la);
      }
    };
    auto load_gate_up = [&](int d) __attribute__((always_inline)) {
      load_w(d);
      r[d].load(pr, 0);
      pr += kStep;
    };
    if (u >= 0 && !down) {
      a0 = u / gpe;
      c = u - a0 * gpe;
      const int e = L.expert[a0], steps = H / kStep;
      first = L.start[a0];
      rows = L.start[a0 + 1] - first;
      tiles = (rows + 15) / 16;
      q0 = wave * steps / kNW;
      q1 = (wave + 1) * steps / kNW;
#pragma unroll
      for (int f = 0; f < F; ++f) {  // F = 1: 8 rows of gate, 8 of up; F = 2: 16 of each
        const bool up = F == 1 ? col >= 8 : f == 1;
        const int n = c * GC + (F == 1 ? col % 8 : col);
        p[f] = static_cast<const char*>(up ? P.w1 : P.w0) +
               ((static_cast<int64_t>(e) * I + n) * H + q0 * kStep + 16 * g) * ESZ;
      }
      pr = P.x + static_cast<int64_t>(L.list[first + min(col, rows - 1)] / k) * H + q0 * kStep + 16 * g;
#pragma unroll
      for (int d = 0; d < AHEAD; ++d)
        if (q0 + d < q1) load_gate_up(d);
      scales(q0);
    } else if (u >= 0) {
      grp = (u - tk.gu) / dpg;
      c = u - tk.gu - grp * dpg;
      a0 = grp * size;
      a_end = a0 + min(size, na - a0);
      const int total = (a_end - a0) * spe;
      q0 = wave * total / kNW;
      q1 = (wave + 1) * total / kNW;
      la = a0 + q0 / spe;
      left = spe - q0 % spe;
      if (q0 < q1) {
        down_rows(c, la);
#pragma unroll
        for (int f = 0; f < F; ++f) p[f] += (q0 % spe) * kStep * ESZ;
      }
#pragma unroll
      for (int d = 0; d < AHEAD; ++d)
        if (q0 + d < q1) load_down(d);
      scales(q0);
    }
    if (fin >= tk.gu) finish_down(fin);
    else if (fin >= 0) finish_gate_up(fin);
    if (u < 0) break;
    if (tid == 0) tk.request(P);  // the next ticket travels while this unit is computed

    f32x4 acc[TILES][F];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int f = 0; f < F; ++f) acc[t][f] = f32x4{};
    if (!down) {
      for (int q = q0; q < q1; q += AHEAD) {
        if (FMT == kFp8 && q > q0 && (q - q0) % 64 == 0) scales(q);
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
          if (q + d < q1) {
            float fa = 1.0f, fb = 1.0f;
            if constexpr (FMT == kFp8) {
              fa = lane_value(sa, (q + d - q0) % 64);
              fb = lane_value(sb, (q + d - q0) % 64);
              if constexpr (F == 1) fa = g < 2 ? fa : fb;  // result rows 8 .. 15 are up's
            }
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (t < tiles) {
                Rows x = r[d];
                if (t > 0)
                  x.load(P.x + static_cast<int64_t>(L.list[first + min(16 * t + col, rows - 1)] / k) * H + 16 * g,
                         q + d);
#pragma unroll
                for (int f = 0; f < F; ++f) multiply<FMT>(acc[t][f], w[d][f], x, f == 0 ? fa : fb);
              }
            }
            if (q + d + AHEAD < q1) load_gate_up(d);
          }
        }
      }
      signal();  // the previous unit's tile: its stores are older than the loads used above
      lds_barrier();  // everyone is done with the scratch
#pragma unroll
      for (int t = 0; t < TILES; ++t)
        if (t < tiles)
#pragma unroll
          for (int f = 0; f < F; ++f) *reinterpret_cast<f32x4*>(&S.red[t][wave][col][16 * f + 4 * g]) = acc[t][f];
    } else {
      float* tile = &S.tile[wave][0][0];
      constexpr int TS = DC + 4;
      signal();  // before this workgroup waits for others
      lds_barrier();  // everyone is done with the scratch
      for (int i = lane; i < T * DC; i += kWave) tile[i / DC * TS + i % DC] = 0.0f;
      // The group's activations are there once all its tiles are counted.
      if (tid == 0) {
        uint32_t want = 0;
        for (int a = a0; a < a_end; ++a) want += (L.start[a + 1] - L.start[a] + 15) / 16 * gpe;
        wait_count(P.cnt + (2 * kLists + grp) * kLine, want);
      }
      lds_barrier();
      int ca = a0 + q0 / spe, cs = q0 % spe;
      int ra = ca, rs = cs;  // row load cursor
      uint32_t rr = 0;
      auto row_at = [&](int a, int t) __attribute__((always_inline)) {
        const int f0 = L.start[a], n = L.start[a + 1] - f0;
        return (static_cast<uint32_t>(L.list[f0 + min(16 * t + col, n - 1)]) * I + 16 * g) * 2;
      };
      auto load_rows = [&](int d) __attribute__((always_inline)) {
        r[d].load(act, rr, rs);
        if (++rs == spe) {
          rs = 0;
          if (++ra < a_end) rr = row_at(ra, 0);
        }
      };
      if (q0 < q1) rr = row_at(ra, 0);
#pragma unroll
      for (int d = 0; d < AHEAD; ++d)
        if (q0 + d < q1) load_rows(d);
      if (q0 < q1) {
        first = L.start[ca];
        rows = L.start[ca + 1] - first;
        tiles = (rows + 15) / 16;
      }
      for (int q = q0; q < q1; q += AHEAD) {
        if (FMT == kFp8 && q > q0 && (q - q0) % 64 == 0) scales(q);
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
          if (q + d < q1) {
            const float fa = FMT == kFp8 ? lane_value(sa, (q + d - q0) % 64) : 1.0f;
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (t < tiles) {
                Rows x = r[d];
                if (t > 0) x.load(act, row_at(ca, t), cs);
#pragma unroll
                for (int f = 0; f < F; ++f) multiply<FMT>(acc[t][f], w[d][f], x, fa);
              }
            }
            if (++cs == spe || q + d + 1 == q1) {  // this expert's products into the tile, row by row
#pragma unroll
              for (int t = 0; t < TILES; ++t) {
                if (t < tiles && 16 * t + col < rows) {
                  float* to = tile + L.list[first + 16 * t + col] / k * TS + 4 * g;
#pragma unroll
                  for (int f = 0; f < F; ++f) {
                    f32x4 v = *reinterpret_cast<f32x4*>(to + 16 * f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += acc[t][f][i];
                    *reinterpret_cast<f32x4*>(to + 16 * f) = v;
                  }
                }
#pragma unroll
                for (int f = 0; f < F; ++f) acc[t][f] = f32x4{};
              }
              cs = 0;
              if (++ca < a_end) {
                first = L.start[ca];
                rows = L.start[ca + 1] - first;
                tiles = (rows + 15) / 16;
              }
            }
            if (q + d + AHEAD < q1) {
              load_down(d);
              load_rows(d);
            }
          }
        }
      }
    }
    fin = u;
    if (tid == 0) L.unit = tk.take(P);
    lds_barrier();
    u = __builtin_amdgcn_readfirstlane(L.unit);
  }
  signal();
}

template <int FMT, int NC>
void launch_layer(const FewParams& P, unsigned grid, hipStream_t st) {
  constexpr int A = FMT == kBf16 ? 4 : 8;
  if (P.T <= 16) few_kernel<FMT, 1, 1, A, NC><<<grid, kThreads, 0, st>>>(P);
  else few_kernel<FMT, 4, 2, A / 2, NC><<<grid, kThreads, 0, st>>>(P);
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
  l.counters = (2 * kLists + l.groups) * kLine + s.H / 16;
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
  P.cnt = reinterpret_cast<uint32_t*>(base);
  P.act = reinterpret_cast<bf16_t*>(base + l.act);
  P.part = reinterpret_cast<float*>(base + l.part);
  P.cnt_down = P.cnt + (2 * kLists + l.groups) * kLine;
  const dim3 rg(static_cast<unsigned>(s.E), static_cast<unsigned>(ceil_div(s.T, kRouterTokens)));
  few_router_kernel<<<rg, kWave, 0, st>>>(s.T, s.H, s.E, P.x, static_cast<const bf16_t*>(a.w_router), a.bias, a.logits,
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
