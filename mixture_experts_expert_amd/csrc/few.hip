// The whole MoE layer for a few tokens (T <= 64), in two launches.
//
// With few tokens the layer is a walk over the selected experts' weights: each
// is read once from memory and multiplied by the handful of rows that chose
// it, so the kernel is bound by the weights' bytes and, for one token, by
// latency (75 MB at the 30B shape in bf16). Everything here serves that: the
// weights go straight from memory into registers in 16-byte loads, several
// steps ahead; gate/up and down are one launch, so that the down weights'
// first loads are in flight while the last gate/up units finish; no
// activation row but the selected experts' (T k I bf16) is ever written.
//
//   few_router_kernel: logits, one wavefront per expert and 8 tokens. x and
//     w_router products are exact in fp32 (bf16 factors) and summed in fp64,
//     so the logit is the exact sum rounded once, whatever the split. It also
//     clears the second kernel's counters.
//   few_kernel: persistent workgroups of 8 wavefronts. Each selects the
//     experts of all tokens for itself (logits to LDS lists; a few hundred
//     nanoseconds, no third launch), then takes units from a ticket counter:
//     - gate/up unit: one expert, 16 columns of gate and of up. The reduction
//       is split over the 8 wavefronts; the partial sums meet in LDS, and
//       a = bf16(w silu(g) u) goes to the workspace per (token, slot).
//     - down unit: one group of experts, 16 columns of y. The (expert, k)
//       steps are split over the wavefronts, each adding its experts' products
//       into its own y tile in LDS; the eight tiles are then summed in order.
//       With one group (up to 8 experts) that is y; otherwise the groups'
//       fp32 partial sums go to the workspace and the last workgroup to
//       finish a column block adds them in group order.
//
// Order and progress: all gate/up units come before all down units in the
// ticket order, and a down unit waits for its group's gate/up units. Those
// have lower tickets, so running workgroups hold them and never wait
// themselves: the wait ends whatever else occupies the device. (If another
// call overwrites the workspace, against the interface, the wait gives up
// after two seconds.)
//
// Tile: v_mfma_f32_16x16x32_bf16 with the weights as A (16 rows) and up to 16
// token rows as B, so a lane's four results are four consecutive columns of
// one row. A step is 64 k: lane group g = lane / 16 takes k 16 g .. 16 g + 15
// of it (the first 8 in one product, the others in the next; any assignment
// of k to lanes serves as long as both operands share it), so a row's 128
// bytes are read together. E4M3 weights are widened to bf16 (exact) in
// registers and each step's partial product is multiplied by its block's
// scale in fp32.
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
constexpr int kCols = 16;           // columns (weight rows) per unit
constexpr int kMaxPairs = kFewMaxT * kFewMaxK;
constexpr uint64_t kSpinTicks = 200000000;  // two seconds of the 100 MHz clock

struct FewParams {
  int T, H, E, k, I;
  const bf16_t* x;
  const void *w0, *w1, *w2;     // gate, up, down: bf16 or E4M3 codes
  const float *s0, *s1, *s2;    // block scales (E4M3)
  const float* logits;
  int32_t* topk_idx;
  float* topk_w;
  bf16_t* y;
  uint32_t* cnt;                // [0] tickets, [1 + g] gate/up units done of group g, then [.. + c] down units done
  bf16_t* act;                  // [T*k][I], weighted
  float* part;                  // [groups][T][H]
  int cnt_down;                 // offset of the down counters
};

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
  int ticket;
  int last;
  uint16_t expert[1024];           // active expert a -> expert
  uint16_t start[1025];            // its pairs: list[start[a] .. start[a + 1])
  uint16_t list[kMaxPairs];        // pair t * k + j
  float weight[kMaxPairs];         // by pair
};

// Per-lane scratch, reused by the phases of a unit.
union FewScratch {
  struct {
    uint16_t sel[kMaxPairs];       // expert of each pair
    int count[1024];               // pairs per expert, then a cursor
    int wave_sum[kNW];
  } lists;
  float red[kNW][2][kCols][kCols + 4];   // gate/up: [wave][gate, up][token row][column]
  float tile[kNW][kFewMaxT][kCols + 4];  // down: [wave][token][column]
};

// Every workgroup selects the experts of all tokens: one token per 16-lane
// row; a round takes the largest key below the previous round's.
__device__ __forceinline__ void few_select(const FewParams& P, FewLists& L, FewScratch& S) {
  const int tid = threadIdx.x, n = tid % 16;
  const int E = P.E, k = P.k, pairs = P.T * k;
  constexpr int NC = 16;  // logits per lane held in registers (E <= 256)
  for (int e = tid; e < E; e += kThreads) S.lists.count[e] = 0;
  __syncthreads();
  for (int t0 = 0; t0 < P.T; t0 += kThreads / 16) {
    const int t = t0 + tid / 16;
    const bool active = t < P.T;
    const float* l = P.logits + static_cast<int64_t>(active ? t : 0) * E;
    float v[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) v[c] = n + 16 * c < E ? l[n + 16 * c] : 0.0f;
    uint64_t prev = ~0ull;
    float sel_v = 0.0f, vmax = 0.0f;
    int sel_i = 0;
    for (int j = 0; j < k; ++j) {
      uint64_t b = 0;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = n + 16 * c;
        const uint64_t key = sel_key(v[c], e);
        if (e < E && key < prev && key > b) b = key;
      }
      for (int e = n + 16 * NC; e < E; e += 16) {
        const uint64_t key = sel_key(l[e], e);
        if (key < prev && key > b) b = key;
      }
      b = row_max_key(b);
      prev = b;
      const float bv = key_value(b);
      if (j == 0) vmax = bv;
      if (n == j) {
        sel_v = bv;
        sel_i = static_cast<int>(~static_cast<uint32_t>(b));
      }
    }
    float z = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (n + 16 * c < E) z += expf(v[c] - vmax);
    for (int e = n + 16 * NC; e < E; e += 16) z += expf(l[e] - vmax);
    z = row_sum(z);
    const float p = n < k ? expf(sel_v - vmax) / z : 0.0f;
    const float den = row_sum(p) + 1e-20f;
    if (active && n < k) {
      const int pair = t * k + n;
      S.lists.sel[pair] = static_cast<uint16_t>(sel_i);
      L.weight[pair] = p / den;
      atomicAdd(&S.lists.count[sel_i], 1);
      if (blockIdx.x == 0) {
        P.topk_idx[pair] = sel_i;
        P.topk_w[pair] = p / den;
      }
    }
  }
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
    if (tid % kWave >= o) incl += up;
  }
  if (tid % kWave == kWave - 1) S.lists.wave_sum[tid / kWave] = incl;
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
  // A row's place in its expert's list changes no result: every row is
  // summed on its own, a token's experts in expert order.
  for (int q = tid; q < pairs; q += kThreads)
    L.list[atomicAdd(&S.lists.count[S.lists.sel[q]], 1)] = static_cast<uint16_t>(q);
  __syncthreads();
}

// Experts per group of the down phase: up to 8 selected experts, one group
// and no partial sums; beyond 64, groups of 16 halve the partial sums.
__host__ __device__ __forceinline__ int few_group(int na) { return na > 64 ? 16 : 8; }

template <int FMT, int TILES, int AHEAD>
__device__ __forceinline__ void gate_up_unit(const FewParams& P, const FewLists& L, FewScratch& S, int a, int c) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane % 16, g = lane / 16;
  const int H = P.H, I = P.I;
  const int e = L.expert[a], first = L.start[a], rows = L.start[a + 1] - first;
  const int steps = H / kStep;
  const int q0 = wave * steps / kNW, q1 = (wave + 1) * steps / kNW;
  constexpr int ESZ = FMT == kBf16 ? 2 : 1;
  const int64_t wrow = (static_cast<int64_t>(e) * I + c * kCols + col) * H + 16 * g;
  const char* pg = static_cast<const char*>(P.w0) + wrow * ESZ;
  const char* pu = static_cast<const char*>(P.w1) + wrow * ESZ;
  Frag<FMT> wg[AHEAD], wu[AHEAD];
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (q0 + d < q1) {
      wg[d].load(pg, q0 + d);
      wu[d].load(pu, q0 + d);
    }
  // Scales of up to 64 steps, one per lane.
  const int kb = (H + 127) / 128;
  const int64_t srow = (static_cast<int64_t>(e) * ((I + 127) / 128) + c * kCols / 128) * kb;
  float sg = 1.0f, su = 1.0f;
  auto scales = [&](int q) {
    if constexpr (FMT == kFp8) {
      const int b = min((q + lane) / 2, kb - 1);
      sg = P.s0[srow + b];
      su = P.s1[srow + b];
    }
  };
  scales(q0);
  const int tiles = (rows + 15) / 16;
  const bf16_t* xr[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int r = min(16 * t + col, rows - 1);
    xr[t] = P.x + static_cast<int64_t>(L.list[first + r] / P.k) * H + 16 * g;
  }
  f32x4 ag[TILES], au[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) ag[t] = au[t] = f32x4{};
  for (int q = q0; q < q1; q += AHEAD) {
    if (FMT == kFp8 && q > q0 && (q - q0) % 64 == 0) scales(q);
    Rows r0[AHEAD];
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
      if (q + d < q1) r0[d].load(xr[0], q + d);
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (q + d >= q1) break;
      const float fg = FMT == kFp8 ? lane_value(sg, (q + d - q0) % 64) : 1.0f;
      const float fu = FMT == kFp8 ? lane_value(su, (q + d - q0) % 64) : 1.0f;
      multiply<FMT>(ag[0], wg[d], r0[d], fg);
      multiply<FMT>(au[0], wu[d], r0[d], fu);
#pragma unroll
      for (int t = 1; t < TILES; ++t) {
        if (t >= tiles) break;
        Rows r;
        r.load(xr[t], q + d);
        multiply<FMT>(ag[t], wg[d], r, fg);
        multiply<FMT>(au[t], wu[d], r, fu);
      }
      if (q + d + AHEAD < q1) {
        wg[d].load(pg, q + d + AHEAD);
        wu[d].load(pu, q + d + AHEAD);
      }
    }
  }
  // The wavefronts' partial sums, in order; two columns of one row per thread.
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    if (t >= tiles) break;
    __syncthreads();
    *reinterpret_cast<f32x4*>(&S.red[wave][0][col][4 * g]) = ag[t];
    *reinterpret_cast<f32x4*>(&S.red[wave][1][col][4 * g]) = au[t];
    __syncthreads();
    const int r = tid / 8, c2 = 2 * (tid % 8);
    if (tid < 128 && 16 * t + r < rows) {
      float v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sgate = 0.0f, sup = 0.0f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
          sgate += S.red[w][0][r][c2 + i];
          sup += S.red[w][1][r][c2 + i];
        }
        v[i] = sgate * sigmoidf_dev(sgate) * sup;
      }
      const int pair = L.list[first + 16 * t + r];
      const float w = L.weight[pair];
      uint32_t* dst = reinterpret_cast<uint32_t*>(P.act + static_cast<int64_t>(pair) * I + c * kCols + c2);
      __hip_atomic_store(dst, pack_bf16x2(w * v[0], w * v[1]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

// Waits until *p reaches `want` (thread 0; the caller's barrier follows).
__device__ __forceinline__ void wait_count(const uint32_t* p, uint32_t want) {
  const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
  while (__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < want) {
    if (__builtin_amdgcn_s_memrealtime() - t0 > kSpinTicks) break;
    __builtin_amdgcn_s_sleep(1);
  }
}

template <int FMT, int TILES, int AHEAD>
__device__ __forceinline__ void down_unit(const FewParams& P, FewLists& L, FewScratch& S, int grp, int ngrp, int c) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane % 16, g = lane / 16;
  const int T = P.T, H = P.H, I = P.I;
  const int size = few_group(L.na), a0 = grp * size, na = min(size, L.na - a0);
  const int spe = I / kStep;  // steps per expert
  const int total = na * spe;
  const int q0 = wave * total / kNW, q1 = (wave + 1) * total / kNW;
  constexpr int ESZ = FMT == kBf16 ? 2 : 1;
  // The load cursor runs AHEAD steps before the compute cursor.
  int la = q0 / spe, ls = q0 % spe;
  const char* lp = nullptr;
  auto row_of = [&](int a) {
    return static_cast<const char*>(P.w2) +
           ((static_cast<int64_t>(L.expert[a0 + a]) * H + c * kCols + col) * I + 16 * g) * ESZ;
  };
  Frag<FMT> wd[AHEAD];
  if (q0 < q1) lp = row_of(la);
  auto load_next = [&](Frag<FMT>& f) {
    f.load(lp, ls);
    if (++ls == spe) {
      ls = 0;
      if (++la < na) lp = row_of(la);
    }
  };
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (q0 + d < q1) load_next(wd[d]);
  const int kb = (I + 127) / 128, hb = (H + 127) / 128;
  float sd = 1.0f;
  auto scales = [&](int q) {
    if constexpr (FMT == kFp8) {
      const int s = min(q + lane, total - 1);
      sd = P.s2[(static_cast<int64_t>(L.expert[a0 + s / spe]) * hb + c * kCols / 128) * kb + s % spe / 2];
    }
  };
  scales(q0);
  float* tile = &S.tile[wave][0][0];
  constexpr int TS = kCols + 4;
  for (int i = lane; i < T * kCols; i += kWave) tile[i / kCols * TS + i % kCols] = 0.0f;
  // All of the group's activations are there once its gate/up units are.
  if (tid == 0) {
    wait_count(P.cnt + 1 + grp, static_cast<uint32_t>(na) * (I / kCols));
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  }
  __syncthreads();
  f32x4 acc[TILES];
  const bf16_t* ar[TILES];
  int rows = 0, first = 0, tiles = 0;
  int ca = q0 / spe, cs = q0 % spe;
  auto open = [&]() {
    first = L.start[a0 + ca];
    rows = L.start[a0 + ca + 1] - first;
    tiles = (rows + 15) / 16;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      ar[t] = P.act + static_cast<int64_t>(L.list[first + min(16 * t + col, rows - 1)]) * I + 16 * g;
      acc[t] = f32x4{};
    }
  };
  auto close = [&]() {  // this expert's products into the tile, row by row
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      if (t >= tiles) break;
      if (16 * t + col < rows) {
        f32x4* d = reinterpret_cast<f32x4*>(tile + L.list[first + 16 * t + col] / P.k * TS + 4 * g);
        f32x4 v = *d;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += acc[t][i];
        *d = v;
      }
    }
  };
  if (q0 < q1) open();
  for (int q = q0; q < q1; q += AHEAD) {
    if (FMT == kFp8 && q > q0 && (q - q0) % 64 == 0) scales(q);
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (q + d >= q1) break;
      const float f = FMT == kFp8 ? lane_value(sd, (q + d - q0) % 64) : 1.0f;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        if (t >= tiles) break;
        Rows r;
        r.load(ar[t], cs);
        multiply<FMT>(acc[t], wd[d], r, f);
      }
      if (++cs == spe || q + d + 1 == q1) {
        close();
        cs = 0;
        if (++ca < na && q + d + 1 < q1) open();
      }
      if (q + d + AHEAD < q1) load_next(wd[d]);
    }
  }
  __syncthreads();
  for (int i = tid; i < T * kCols / 2; i += kThreads) {
    const int t = i / (kCols / 2), h = 2 * (i % (kCols / 2));
    float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      v0 += S.tile[w][t][h];
      v1 += S.tile[w][t][h + 1];
    }
    const int64_t at = static_cast<int64_t>(t) * H + c * kCols + h;
    if (ngrp == 1) {
      *reinterpret_cast<uint32_t*>(P.y + at) = pack_bf16x2(v0, v1);
    } else {
      uint64_t* d = reinterpret_cast<uint64_t*>(P.part + static_cast<int64_t>(grp) * T * H + at);
      __hip_atomic_store(d, static_cast<uint64_t>(__float_as_uint(v1)) << 32 | __float_as_uint(v0), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (ngrp == 1) return;
  __syncthreads();
  if (tid == 0) {
    const uint32_t n = __hip_atomic_fetch_add(P.cnt + P.cnt_down + c, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    L.last = n == static_cast<uint32_t>(ngrp) - 1;
  }
  __syncthreads();
  if (!L.last) return;
  for (int i = tid; i < T * kCols / 2; i += kThreads) {
    const int64_t at = static_cast<int64_t>(i / (kCols / 2)) * H + c * kCols + 2 * (i % (kCols / 2));
    float v0 = 0.0f, v1 = 0.0f;
    for (int q = 0; q < ngrp; ++q) {
      const float2 v = *reinterpret_cast<const float2*>(P.part + static_cast<int64_t>(q) * T * H + at);
      v0 += v.x;
      v1 += v.y;
    }
    *reinterpret_cast<uint32_t*>(P.y + at) = pack_bf16x2(v0, v1);
  }
}

// TILES: 16-row tiles of one expert's tokens (one for T <= 16, else four);
// AHEAD: steps of weights in flight per wavefront.
template <int FMT, int TILES, int AHEAD>
__global__ __launch_bounds__(kThreads, TILES == 1 ? 4 : 2) void few_kernel(FewParams P) {
  __shared__ FewLists L;
  __shared__ __attribute__((aligned(16))) FewScratch S;
  const int tid = threadIdx.x;
  uint32_t mine = 0;
  if (tid == 0) mine = __hip_atomic_fetch_add(P.cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  few_select(P, L, S);
  const int per_expert = P.I / kCols, per_group = P.H / kCols;
  const int size = few_group(L.na), ngrp = (L.na + size - 1) / size;
  const uint32_t gu = static_cast<uint32_t>(L.na) * per_expert, all = gu + static_cast<uint32_t>(ngrp) * per_group;
  for (;;) {
    if (tid == 0) L.ticket = static_cast<int>(min(mine, 0x7fffffffu));
    __syncthreads();
    const uint32_t u = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(L.ticket));
    if (u >= all) return;
    // The next ticket travels while this unit is computed.
    if (tid == 0) mine = __hip_atomic_fetch_add(P.cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (u < gu) {
      const int a = static_cast<int>(u) / per_expert;
      gate_up_unit<FMT, TILES, AHEAD>(P, L, S, a, static_cast<int>(u) % per_expert);
      __syncthreads();  // every thread's activations are written
      if (tid == 0)
        __hip_atomic_fetch_add(P.cnt + 1 + a / size, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    } else {
      const int d = static_cast<int>(u - gu);
      down_unit<FMT, TILES, AHEAD>(P, L, S, d / per_group, ngrp, d % per_group);
    }
    __syncthreads();
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
  l.counters = 1 + l.groups + s.H / kCols;
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
  P.cnt_down = 1 + l.groups;
  const dim3 rg(static_cast<unsigned>(s.E), static_cast<unsigned>(ceil_div(s.T, kRouterTokens)));
  few_router_kernel<<<rg, kWave, 0, st>>>(s.T, s.H, s.E, P.x, static_cast<const bf16_t*>(a.w_router), a.bias, a.logits,
                                          P.cnt, l.counters);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t units = static_cast<int64_t>(few_max_active(s)) * (s.I / kCols) +
                        static_cast<int64_t>(l.groups) * (s.H / kCols);
  const int64_t slots = 2 * gemm_grid();
  const unsigned grid = static_cast<unsigned>(units < slots ? units : slots);
  const bool one = s.T <= 16;
  if (a.gate_scale != nullptr) {
    if (one) few_kernel<kFp8, 1, 4><<<grid, kThreads, 0, st>>>(P);
    else few_kernel<kFp8, 4, 4><<<grid, kThreads, 0, st>>>(P);
  } else {
    if (one) few_kernel<kBf16, 1, 4><<<grid, kThreads, 0, st>>>(P);
    else few_kernel<kBf16, 4, 4><<<grid, kThreads, 0, st>>>(P);
  }
  return hipGetLastError();
}

}  // namespace moe
