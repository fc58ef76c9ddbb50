// Grouped products of E4M3 operands with one fp32 scale per block of 128:
// activations 1 x 128, weights 128 x 128.
//
//   out[p,n] = sum over blocks b of sa[p,b] sw[n/128,b] (sum_{k in b} a[p,k] w[n,k])
//
// The scales are not powers of two, so the matrix core cannot apply them: one
// v_mfma_f32_16x16x128_f8f6f4 covers exactly one block of k, and its partial
// product goes into the fp32 accumulators with one fma per element. With the
// weights as the A operand a lane's four results belong to one row of a, so
// the block's factor sa * sw is one register per 16 rows, and the fmas take
// half the matrix core's time on the vector units beside it.
//
// That instruction adds the products of 8 consecutive k aligned to the largest
// one's exponent and drops what lies 13 bits below (seen by cancelling large
// products against each other; sums of eights keep fp32's bits): against 64
// bits a block maximum of silu(g) u is off by 1.5e-5 (rms), where fp32 products
// give 5e-7. The older 32-deep instructions would halve the rate; E4M3 operands,
// off by 2^-4 themselves, do not ask for it.
//
// Two kernels:
//
// block_tile_kernel: a persistent workgroup of 8 wavefronts (two per SIMD, so
// that one's fmas run under the other's products) on BM x 256 tiles, 2 x 4
// wavefronts of BM/2 x 64. Operands go from memory straight into LDS, two
// stages of one 128-wide k-step in halves that are refilled as soon as they
// are read (see there). A row's 128 bytes are eight 16-byte chunks,
// XOR-swizzled by row so that a 16-lane read touches every bank once. Which
// weight row sits at which LDS row is chosen so that a lane ends with 8
// consecutive output columns. Measured: 8192 x 4096 x 4096 in 139 us, 2.0
// PFLOP/s (2.2 to 2.5 in the steady state of a longer reduction; without the
// loads it would be 112 us, so the way from L2 to LDS costs the rest); 65536
// rows over 128 experts, 2048 x 768, 178 us, of which the 520 MB are 101 us.
//
// block_stream_kernel, for a few rows: bound by the weights' bytes or by
// latency. Weights go from memory into registers two steps ahead; with few
// workgroups of work the reduction is split over the wavefronts of one, and
// the parts meet in LDS in a fixed order. One row, 2048 x 2048: 4.4 us.
//
// The gate/up forms end with a = silu(g) u quantised: a workgroup holds whole
// 1 x 128 blocks of a, whose maxima meet in LDS.
#include <type_traits>

#include "shared8.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int KS = 128;                     // k per step: one scale block
constexpr uint32_t kOutside = 0x80000000u;  // past every buffer's range: loads read zeros

struct Params {
  int M, E, N, K, KB, NB;   // KB, NB: blocks of the reduction and of the weight rows
  int arows;                // rows of a behind row_token
  const int32_t* offsets;
  const int32_t* row_token;
  const uint8_t *a, *w0, *w1;
  const float *sa, *sw0, *sw1;
  const float* row_weight;
  bf16_t* out;
  bool shared8;             // out in shared8.h's form
  uint8_t* aq;
  float* sout;
};

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

__device__ __forceinline__ i32x8 join(const u32x4& lo, const u32x4& hi) {
  return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
               static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
}

// The unscaled E4M3 x E4M3 product of one block.
__device__ __forceinline__ f32x4 block_product(const i32x8& w, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, f32x4{}, 0, 0, 0, 0, 0, 0);
}

// silu(g) u with the hardware exponential and reciprocal (about 1 ulp each;
// the result is rounded to 8 bits).
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f)) * u;
}

// 448 / amax (0 for amax = 0), and the power of two that keeps it finite for
// blocks below 2^-64.
__device__ __forceinline__ float code_factor(float amax, float& up) {
  up = amax < 0x1p-64f ? 0x1p64f : 1.0f;
  return amax > 0.0f ? 448.0f / (amax * up) : 0.0f;
}

// The largest magnitude rounds to at most one ulp past 448: clamped, because
// the conversion turns values past the range into NaN. NaN stays NaN.
__device__ __forceinline__ float to_code_range(float v, float up, float r) {
  const float t = v * up * r;
  return t == t ? __builtin_amdgcn_fmed3f(t, -448.0f, 448.0f) : t;
}

__device__ __forceinline__ uint32_t codes4(const float (&v)[4], float up, float r) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = to_code_range(v[i], up, r);
  int q = 0;
  q = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], q, false);
  q = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], q, true);
  return static_cast<uint32_t>(q);
}

// ---- many rows per expert ---------------------------------------------------

constexpr int BN = 256;
constexpr int kBand = 8;  // row tiles that run side by side over all columns: what an XCD's workgroups read meets in its L2

// GU: N columns of each of w0 and w1 (128 per tile), else N of w0 (256 per tile).
//
// A tile's rows come in two halves; a wavefront has half of each. Step s lives
// in stage s % 2, and its loads leave a step and a half before they are used:
// the weights and the first half's rows as soon as every wavefront has taken
// step s - 2's into registers (after that step's middle barrier), the second
// half's rows once step s - 2 has ended. In order of issue:
//   .. | W, A0 of s+1 | A1 of s+1 | W, A0 of s+2 | A1 of s+2 | ..
//         step s-1, 2nd  step s, 1st   step s, 2nd  step s+1, 1st half
// so at each barrier all but the last two groups have landed.
template <bool GU, int BM>
__global__ __launch_bounds__(kThreads, 2) void block_tile_kernel(const Params P) {
  constexpr int FM = BM / 32, HM = FM / 2;  // 16-row tiles of a per wavefront, and of those per half
  constexpr int HA = BM / 128;              // load instructions of half a's rows per wavefront
  constexpr int OS = BM / 2 * KS;
  constexpr int TN = GU ? BN / 2 : BN;
  constexpr int G1 = HA + 1, G2 = 4 + HA + 1, STORES = 2 * FM;
  // A stage, in three arrays, so that the compiler sees which reads follow
  // which loads: the weights' rows; the first half's rows of a and 8 x 64 scales
  // (waves 0 ..: rows; 6 and 7: the weights'); the second half's rows and scales.
  __shared__ __attribute__((aligned(1024))) uint8_t w0[BN * KS];
  __shared__ __attribute__((aligned(1024))) uint8_t w1[BN * KS];
  __shared__ __attribute__((aligned(1024))) uint8_t x0[OS + kThreads * 4];
  __shared__ __attribute__((aligned(1024))) uint8_t x1[OS + kThreads * 4];
  __shared__ __attribute__((aligned(1024))) uint8_t y0[OS + kThreads * 4];
  __shared__ __attribute__((aligned(1024))) uint8_t y1[OS + kThreads * 4];
  __shared__ int tstart[1025];
  __shared__ int eoff[1025];
  __shared__ int wsum[kWaves];
  __shared__ float amax[GU ? BM : 1][4];
  __shared__ __attribute__((aligned(256))) int per_row[kThreads];  // GU: the next tile's tokens, else this one's weights

  const int tid = threadIdx.x;
  const int lane_id = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int E = P.E, K = P.K, KB = P.KB;

  // tstart[e]: row tiles of the experts before e (two experts per thread).
  {
    int c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      const int b = e < E && P.offsets ? P.offsets[e] : 0;
      const int t = e < E ? (P.offsets ? P.offsets[e + 1] : P.M) : 0;
      c[i] = e < E ? (t - b + BM - 1) / BM : 0;
      if (e < E) eoff[e] = b;
      if (e == E - 1) eoff[E] = t;
    }
    const int mine = c[0] + c[1];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane_id >= o) incl += v;
    }
    if (lane_id == kWave - 1) wsum[wave] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < wave; ++w) at += wsum[w];
    if (2 * tid < E) tstart[2 * tid] = at;
    if (2 * tid + 1 < E) tstart[2 * tid + 1] = at + c[0];
    if (tid == kThreads - 1) tstart[E] = at + mine;
    __syncthreads();
  }
  const int ntn = (P.N + TN - 1) / TN;
  const int total = tstart[E] * ntn;
  // Eighths of the tile list per XCD, neighbouring tiles on one XCD.
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, nslots = gridDim.x >> 3;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * xcd / 8);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (xcd + 1) / 8);
  const int steps = KB, padded = (steps + 1) & ~1;
  const int tail = K - (steps - 1) * KS;  // k of the last step
  int L = lo + slot;
  if (L >= hi) return;

  // The arguments, read again where a tile begins or ends: kept in scalar
  // registers through the loop they cost spills, whose reloads wait for every
  // load in flight.
  auto args = [&]() __attribute__((always_inline)) {
    uintptr_t u = reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(u));
    return reinterpret_cast<const __attribute__((address_space(4))) Params*>(u);
  };
  struct Tile {
    int e, row0, valid, n0;
  };
  auto find = [&](int at) __attribute__((always_inline)) {
    int l = 0, h = E - 1;
    while (l < h) {
      const int mid = (l + h + 1) >> 1;
      if (tstart[mid] * ntn <= at) l = mid; else h = mid - 1;
    }
    const int rem = at - tstart[l] * ntn, mte = tstart[l + 1] - tstart[l];
    const int band = rem / (kBand * ntn), bm = min(kBand, mte - band * kBand);
    const int nt = (rem - band * kBand * ntn) / bm, mt = band * kBand + rem - band * kBand * ntn - nt * bm;
    Tile t;
    t.e = __builtin_amdgcn_readfirstlane(l);
    t.row0 = __builtin_amdgcn_readfirstlane(eoff[l] + mt * BM);
    t.valid = __builtin_amdgcn_readfirstlane(min(BM, eoff[l + 1] - eoff[l] - mt * BM));
    t.n0 = __builtin_amdgcn_readfirstlane(nt * TN);
    return t;
  };
  // The loads' state: resources of their tile, and the lane's offsets.
  rsrc_t ra, rb, rs;
  uint32_t aoff[2 * HA], boff[4], soff[2];
  auto aim = [&](const Tile& t) __attribute__((always_inline)) {
    const auto* A = args();
    int lane = lane_id;  // opaque: the lane terms are recomputed here, not kept alive
    asm volatile("" : "+v"(lane));
    const int64_t first = GU ? 0 : t.row0, rows = GU ? A->arows : t.valid;
    ra = make_rsrc(A->a + first * K, rows * K);
    rb = make_rsrc((GU && (wave & 1) ? A->w1 : A->w0) + static_cast<int64_t>(t.e) * A->N * K, static_cast<int64_t>(A->N) * K);
    const float* scales = A->sa + first * KB;
    int64_t n_scales = rows * KB;
    if (wave >= 6) {
      const int nb = GU ? t.n0 / 128 : min(t.n0 + (wave - 6) * 128, A->N - 1) / 128;
      scales = (GU && wave == 7 ? A->sw1 : A->sw0) + (static_cast<int64_t>(t.e) * A->NB + nb) * KB;
      n_scales = KB;
    }
    rs = make_rsrc(scales, n_scales * 4);
#pragma unroll
    for (int i = 0; i < 2 * HA; ++i) {
      const int r = (i / HA) * (BM / 2) + (wave * HA + i % HA) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      const int row = GU ? (r < t.valid ? per_row[r] : 0) : r;
      aoff[i] = r < t.valid ? static_cast<uint32_t>(row) * K + c * 16 : kOutside;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h * (BM / 2) + wave * 64 + lane;
      const bool in = wave < BM / 128 && r < t.valid;
      const int row = GU ? (in ? per_row[r] : 0) : r;
      soff[h] = in ? static_cast<uint32_t>(row) * KB * 4 : kOutside;
    }
    if (wave >= 6 && lane == 0) soff[0] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (wave * 4 + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      const int j = (r >> 4) & 3, q = r & 15;
      const int n = t.n0 + (r >> 6) * (GU ? 32 : 64) + (GU ? 0 : (j >> 1) * 32) + 8 * (q >> 2) + 4 * (j & 1) + (q & 3);
      boff[i] = n < A->N ? static_cast<uint32_t>(n) * K + c * 16 : kOutside;
    }
  };
  // Load instruction v of step s, of the first (weights W, rows, scales) or the
  // second half's group (rows, scales). Every wavefront issues every one in
  // every step (a branch in the loop costs more than the instruction): chunks
  // past a row's end, and all of a step that is not there, lie outside and
  // read zeros.
  typedef __attribute__((address_space(3))) void* lds_ptr;
  auto load = [&](int h, int v, uint8_t* S, uint8_t* W, int s, bool live) __attribute__((always_inline)) {
    if (v == (h ? G1 : G2) - 1) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(S + OS + wave * 256), 4, live ? soff[h] : kOutside, s * 4, 0,
                                               0);
      return;
    }
    const bool weights = !h && v < 4;
    const int i = weights ? v : h ? v : v - 4, blk = wave * (weights ? 4 : HA) + i;  // eight rows of its array
    const uint32_t to = weights ? boff[i & 3] : aoff[(h * HA + i) % (2 * HA)];
    const int c = (lane_id & 7) ^ (lane_id >> 4) ^ ((blk & 1) * 4);
    const uint32_t off = c * 16 < (!live ? 0 : s == steps - 1 ? tail : KS) ? to : kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(weights ? rb : ra, (lds_ptr)((weights ? W : S) + blk * 1024), 16, off, s * KS,
                                             0, 0);
  };
  // All but the last PENDING memory instructions are done, and every wavefront is here.
  auto landed = [&](auto pending) __attribute__((always_inline)) {
    constexpr int n = decltype(pending)::value;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);  // vmcnt(n) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  using none = std::integral_constant<int, 0>;
  using one = std::integral_constant<int, 1>;
  auto row_of = [&](int i, int q) __attribute__((always_inline)) {  // of the wavefront's 16-row tile i
    return (i / HM) * (BM / 2) + wm * (BM / 4) + (i % HM) * 16 + q;
  };
  auto per_row_load = [&](const void* base, int row0, int valid) __attribute__((always_inline)) {
    const int r = wave * 64 + lane_id;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(static_cast<const char*>(base) + static_cast<int64_t>(row0) * 4,
                                                       valid * 4),
                                             (lds_ptr)(reinterpret_cast<char*>(per_row) + wave * 256), 4, r * 4, 0, 0, 0);
  };

  f32x4 acc[FM][4];
  i32x8 wf[4];
  float fg = 0.0f, fu = 0.0f;
  // Half a step on stage C (the wavefront's 16-row tiles of half h, if NI has
  // them), while the group of step sn goes out into stage D. a's fragments are
  // read one tile ahead. The empty asm keeps the order as written: the
  // compiler otherwise joins the steps and spills.
  auto half = [&](auto nic, auto hc, const uint8_t* C, const uint8_t* CW, uint8_t* D, uint8_t* DW,
                  int sn, bool live) __attribute__((always_inline)) {
    constexpr int NI = decltype(nic)::value, h = decltype(hc)::value;
    constexpr int LD = h ? G2 : G1;  // the second half of a step sends the first half's group
    using group = std::integral_constant<int, h ? 0 : 1>;
    if constexpr (h * HM < NI) {
      int lane = lane_id;
      asm volatile("" : "+v"(lane));
      const int q = lane & 15, o = ((2 * (lane >> 4)) ^ ((q >> 1) & 7)) << 4;  // rows 16 apart: the same swizzle
      auto chunk = [&](const uint8_t* p) __attribute__((always_inline)) {
        return join(*reinterpret_cast<const u32x4*>(p + o), *reinterpret_cast<const u32x4*>(p + (o ^ 16)));
      };
      const uint8_t* wrow = CW + (wn * 64 + q) * KS;
      const uint8_t* arow = C + (wm * (BM / 4) + q) * KS;
      const uint8_t* srow = C + OS + (wm * (BM / 4) + q) * 4;
      i32x8 af[2];
      float sr[2];
      af[0] = chunk(arow);
      sr[0] = *reinterpret_cast<const float*>(srow);
      if constexpr (h == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) wf[j] = chunk(wrow + j * 16 * KS);
        fg = *reinterpret_cast<const float*>(C + OS + (GU ? 6 : 6 + (wn >> 1)) * 256);
        if constexpr (GU) fu = *reinterpret_cast<const float*>(C + OS + 7 * 256);
      }
      f32x4 pr[2][4];
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int i = 0; i <= HM; ++i) {
        if (i + 1 < HM) {
          af[(i + 1) & 1] = chunk(arow + (i + 1) * 16 * KS);
          sr[(i + 1) & 1] = *reinterpret_cast<const float*>(srow + (i + 1) * 64);
        }
        const float f = i > 0 ? s0 : 0.0f, f1 = i > 0 ? s1 : 0.0f;
        if (i < HM) {
          s0 = sr[i & 1] * fg;
          s1 = GU ? sr[i & 1] * fu : s0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i < HM) pr[i & 1][j] = block_product(wf[j], af[i & 1]);
          if (i > 0)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              acc[h * HM + i - 1][j][x] = fmaf(j < 2 ? f : f1, pr[(i - 1) & 1][j][x], acc[h * HM + i - 1][j][x]);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (i < HM)
#pragma unroll
          for (int v = i * LD / HM; v < (i + 1) * LD / HM; ++v) load(group::value, v, D, DW, sn, live);
        __builtin_amdgcn_sched_barrier(0);
        if (i > 0)
          asm volatile("" : "+v"(acc[h * HM + i - 1][0]), "+v"(acc[h * HM + i - 1][1]), "+v"(acc[h * HM + i - 1][2]),
                       "+v"(acc[h * HM + i - 1][3]));
      }
    } else {
#pragma unroll
      for (int v = 0; v < LD; ++v) load(group::value, v, D, DW, sn, live);
    }
  };

  Tile now = find(L), nx = now;
  auto tile = [&](auto nic) __attribute__((always_inline)) {
    constexpr int NI = decltype(nic)::value;
    const int next = L + nslots;
    const bool more = next < hi;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
    // Steps s (x0, y0) and s + 1 (x1, y1). From the middle of the last
    // pair on the loads are the next tile's.
    auto pair = [&](auto firstc, int s) __attribute__((always_inline)) {
      constexpr bool first = decltype(firstc)::value != 0;
      using pending = std::integral_constant<int, G1 + G2 + (first ? STORES : 0)>;
      const bool last = s + 2 == padded;
      half(nic, none{}, x0, w0, y1, nullptr, s + 1, s + 1 < steps);  // an odd count's last step: zeros
      landed(pending{});
      if constexpr (first) {
        if constexpr (GU) {
          if (more) {
            nx = find(next);
            per_row_load(args()->row_token, nx.row0, nx.valid);
          }
        } else if (const float* w = args()->row_weight; w != nullptr) {
          per_row_load(w, now.row0, now.valid);
        }
      }
      if (last && more) {
        if constexpr (!GU) nx = find(next);
        if (GU && first) landed(none{});  // a reduction of one pair: the tokens were only just sent for
        aim(nx);
      }
      half(nic, one{}, y0, nullptr, x0, w0, last ? 0 : s + 2, last ? more : s + 2 < steps);
      landed(pending{});
      half(nic, none{}, x1, w1, y0, nullptr, last ? 0 : s + 2, last ? more : s + 2 < steps);
      landed(std::integral_constant<int, G1 + G2>{});
      half(nic, one{}, y1, nullptr, x1, w1, last ? 1 : s + 3, last ? more && steps > 1 : s + 3 < steps);
      landed(std::integral_constant<int, G1 + G2>{});
    };
    pair(one{}, 0);
    for (int s = 2; s < padded; s += 2) pair(none{}, s);
    // ---- epilogue; stores of rows and columns outside go out of range, so
    // that their count is fixed: they run on under the next tile's first step.
    const auto* A = args();
    const int lane = lane_id, g = lane >> 4, q = lane & 15;
    const int row0 = now.row0, valid = now.valid, n0 = now.n0;
    if constexpr (GU) {
      const int NBo = (A->N + 127) / 128;
      const rsrc_t rq = make_rsrc(A->aq + static_cast<int64_t>(row0) * A->N, static_cast<int64_t>(valid) * A->N);
      const rsrc_t rm = make_rsrc(A->sout + static_cast<int64_t>(row0) * NBo, static_cast<int64_t>(valid) * NBo * 4);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float v = silu_mul(acc[i][j][x], acc[i][j + 2][x]);
            acc[i][j][x] = v;
            m = fmaxf(m, fabsf(v));
          }
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        if (g == 0) amax[row_of(i, q)][wn] = m;
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = row_of(i, q);
        uint2 codes = make_uint2(0, 0);
        float m = 0.0f;
        if (i < NI) {
          m = fmaxf(fmaxf(amax[r][0], amax[r][1]), fmaxf(amax[r][2], amax[r][3]));
          float up;
          const float f = code_factor(m, up);
          const float v0[4] = {acc[i][0][0], acc[i][0][1], acc[i][0][2], acc[i][0][3]};
          const float v1[4] = {acc[i][1][0], acc[i][1][1], acc[i][1][2], acc[i][1][3]};
          codes = make_uint2(codes4(v0, up, f), codes4(v1, up, f));
        }
        const int n = n0 + wn * 32 + 8 * g;
        const bool row = i < NI && r < valid;
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{codes.x, codes.y}, rq,
                                              row && n < A->N ? static_cast<uint32_t>(r) * A->N + n : kOutside, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(m / 448.0f), rm,
            row && wn == 0 && g == 0 ? (static_cast<uint32_t>(r) * NBo + n0 / 128) * 4 : kOutside, 0, 0);
      }
    } else {
      const rsrc_t ro = make_rsrc(A->out + static_cast<int64_t>(row0) * A->N, static_cast<int64_t>(valid) * A->N * 2);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = row_of(i, q);
        const float x = A->row_weight != nullptr ? __int_as_float(per_row[r]) : 1.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = n0 + wn * 64 + 32 * h + 8 * g;
          u32x4 o{};
          if (i < NI && row_of(i, 0) < valid) {  // 16 rows past the end are not packed
            float v[8], m = 0.0f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              v[c] = x * acc[i][2 * h + c / 4][c % 4];
              m = __builtin_elementwise_maximum(m, fabsf(v[c]));  // NaN if one is
            }
            float f = 0.0f;
            const uint32_t s = A->shared8 ? shared8_exponent(m, f) : 0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              o[c] = A->shared8 ? shared8_word(v[2 * c], v[2 * c + 1], s, f, c) : pack_bf16x2(v[2 * c], v[2 * c + 1]);
          }
          __builtin_amdgcn_raw_buffer_store_b128(
              o, ro, i < NI && r < valid && n < A->N ? (static_cast<uint32_t>(r) * A->N + n) * 2 : kOutside, 0, 0);
        }
      }
    }
    now = nx;
    L = next;
  };

  if constexpr (GU) {
    per_row_load(P.row_token, now.row0, now.valid);
    landed(none{});
  }
  aim(now);
#pragma unroll
  for (int v = 0; v < G2; ++v) load(0, v, x0, w0, 0, true);
#pragma unroll
  for (int v = 0; v < G1; ++v) load(1, v, y0, nullptr, 0, true);
#pragma unroll
  for (int v = 0; v < G2; ++v) load(0, v, x1, w1, 1, steps > 1);
  landed(none{});
  while (L < hi) {
    if (now.valid > BM / 2) tile(std::integral_constant<int, FM>{});
    else tile(std::integral_constant<int, HM>{});  // the first half holds every row
  }
}

// ---- few rows per expert ----------------------------------------------------

constexpr int kTiles = 2;  // 16-row tiles of a per pass over the weights
constexpr int kAhead = 2;  // steps in registers before their products

// One workgroup: expert e, and 16 columns per wavefront of w0 and w1 (GU), or
// (kWaves / ks) * 16 columns of w0, each split over ks wavefronts along k.
//
// Eight lanes load a row's 128 bytes of a step (loads whose neighbouring lanes
// are in different rows take four times the address cycles), kAhead steps ahead
// into registers; a wavefront's own piece of LDS turns them into fragments.
// Every load is issued in every step, outside the matrix where there is
// nothing to load: behind a condition the compiler waits for all of them.
template <bool GU>
__global__ __launch_bounds__(kThreads, 2) void block_stream_kernel(const Params P, int ks, int groups) {
  __shared__ __attribute__((aligned(16))) float red[kWaves][16][20];
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][GU ? 3 : 2][16 * KS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane & 15, g = lane >> 4;
  const int lr = lane >> 3, lc = lane & 7;  // as a loader: row, chunk
  const int e = blockIdx.x / groups, grp = blockIdx.x - e * groups;
  const int first = P.offsets ? P.offsets[e] : 0;
  const int rows = (P.offsets ? P.offsets[e + 1] : P.M) - first;
  if (rows <= 0) return;
  const int K = P.K, KB = P.KB, N = P.N;
  const int cw = GU ? wave : wave / ks, kp = GU ? 0 : wave - cw * ks;
  const int n0 = (grp * (GU ? kWaves : kWaves / ks) + cw) * 16;
  const int s0 = kp * KB / ks, s1 = (kp + 1) * KB / ks;
  const int64_t wbytes = static_cast<int64_t>(N) * K;
  const rsrc_t r0 = make_rsrc(P.w0 + e * wbytes, wbytes);
  const rsrc_t r1 = make_rsrc((GU ? P.w1 : P.w0) + e * wbytes, wbytes);
  const int64_t srow = (static_cast<int64_t>(e) * P.NB + min(n0, N - 1) / 128) * KB;
  const rsrc_t rs0 = make_rsrc(P.sw0 + srow, KB * 4), rs1 = make_rsrc((GU ? P.sw1 : P.sw0) + srow, KB * 4);
  uint32_t woff[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    woff[i] = n0 + lr + 8 * i < N ? static_cast<uint32_t>(n0 + lr + 8 * i) * K + lc * 16 : kOutside;
  auto b128 = [&](const rsrc_t& r, uint32_t off) __attribute__((always_inline)) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  };
  // A row's chunk of step s: outside past the wavefront's steps and the row's end.
  auto at = [&](uint32_t off, int s) __attribute__((always_inline)) {
    return s < s1 && s * KS + lc * 16 < K ? off + s * KS : kOutside;
  };
  struct Step {
    u32x4 w0[2], w1[GU ? 2 : 1], x[2];
    float sw0, sw1, sx;
  };
  auto put = [&](uint8_t* to, const u32x4(&v)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lr + 8 * i;
      *reinterpret_cast<u32x4*>(to + r * KS + ((lc ^ ((r >> 1) & 7)) << 4)) = v[i];
    }
  };
  auto fragment = [&](const uint8_t* from) __attribute__((always_inline)) {
    const uint8_t* p = from + q * KS;
    const int o = ((2 * g) ^ ((q >> 1) & 7)) << 4;
    return join(*reinterpret_cast<const u32x4*>(p + o), *reinterpret_cast<const u32x4*>(p + (o ^ 16)));
  };
  for (int p0 = 0; p0 < rows; p0 += 16 * kTiles) {
    const int tiles = min(kTiles, (rows - p0 + 15) / 16);
    const int64_t base = GU ? 0 : first + p0;
    const int64_t left = GU ? P.arows : min(rows - p0, 16 * kTiles);
    const rsrc_t ra = make_rsrc(P.a + base * K, left * K), rsa = make_rsrc(P.sa + base * KB, left * KB * 4);
    uint32_t xoff[kTiles][2], soff[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      auto row = [&](int i) {  // i: of the 16 rows
        const int r = p0 + 16 * t + i;
        return r < rows ? (GU ? P.row_token[first + r] : r - p0) : -1;
      };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = row(lr + 8 * i);
        xoff[t][i] = x >= 0 ? static_cast<uint32_t>(x) * K + lc * 16 : kOutside;
      }
      const int x = row(q);
      soff[t] = x >= 0 ? static_cast<uint32_t>(x) * KB * 4 : kOutside;
    }
    auto f32 = [&](const rsrc_t& r, uint32_t off) __attribute__((always_inline)) {
      return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    };
    Step st[kAhead];
    auto fetch = [&](Step& f, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f.w0[i] = b128(r0, at(woff[i], s));
        if constexpr (GU) f.w1[i] = b128(r1, at(woff[i], s));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) f.x[i] = b128(ra, at(xoff[0][i], s));
      f.sw0 = f32(rs0, s * 4);
      if constexpr (GU) f.sw1 = f32(rs1, s * 4);
      f.sx = f32(rsa, s < s1 ? soff[0] + s * 4 : kOutside);
    };
    f32x4 a0[kTiles], a1[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) a0[t] = a1[t] = f32x4{};
#pragma unroll
    for (int d = 0; d < kAhead; ++d) fetch(st[d], s0 + d);
    auto batch = [&](auto more, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        const float f0 = st[d].sw0, f1 = GU ? st[d].sw1 : 0.0f;
        uint8_t* own = stage[wave][0];
        put(own, st[d].w0);
        if constexpr (GU) put(own + 2 * 16 * KS, st[d].w1);
        put(own + 16 * KS, st[d].x);
        const i32x8 wf0 = fragment(own), wf1 = GU ? fragment(own + 2 * 16 * KS) : i32x8{};
        const float sx = st[d].sx;
        auto tile = [&](int t, float sr) __attribute__((always_inline)) {
          const i32x8 x = fragment(own + 16 * KS);
          const f32x4 m0 = block_product(wf0, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) a0[t][i] = fmaf(sr * f0, m0[i], a0[t][i]);
          if constexpr (GU) {
            const f32x4 m1 = block_product(wf1, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) a1[t][i] = fmaf(sr * f1, m1[i], a1[t][i]);
          }
        };
        if (s + d < s1) {  // past the steps, zeros could meet an infinite scale
          tile(0, sx);
#pragma unroll
          for (int t = 1; t < kTiles; ++t) {
            if (t >= tiles) break;
            const u32x4 x[2] = {b128(ra, at(xoff[t][0], s + d)), b128(ra, at(xoff[t][1], s + d))};
            const float sr = f32(rsa, soff[t] + (s + d) * 4);
            put(own + 16 * KS, x);
            tile(t, sr);
          }
        }
        if constexpr (decltype(more)::value) fetch(st[d], s + d + kAhead);
      }
    };
    int s = s0;
    for (; s + kAhead < s1; s += kAhead) batch(std::true_type{}, s);
    batch(std::false_type{}, s);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (t >= tiles) break;
      const int r = p0 + 16 * t + q;
      const int n = n0 + 4 * g;
      const int64_t p = first + r;
      if constexpr (GU) {
        float v[4], m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = silu_mul(a0[t][i], a1[t][i]);
          m = fmaxf(m, fabsf(v[i]));
        }
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        __syncthreads();  // the previous tile's maxima are read
        if (g == 0) red[wave][q][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = fmaxf(m, red[w][q][0]);
        float up;
        const float f = code_factor(m, up);
        if (r < rows) {
          if (n < N) *reinterpret_cast<uint32_t*>(P.aq + p * N + n) = codes4(v, up, f);
          if (wave == 0 && g == 0) P.sout[p * ((N + 127) / 128) + grp] = m / 448.0f;
        }
      } else {
        f32x4 v = a0[t];
        if (ks > 1) {  // the parts along k, in order
          __syncthreads();
          *reinterpret_cast<f32x4*>(&red[wave][q][4 * g]) = v;
          __syncthreads();
          if (kp != 0) continue;
          for (int w = 1; w < ks; ++w) {
            const f32x4 o = *reinterpret_cast<const f32x4*>(&red[wave + w][q][4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += o[i];
          }
        }
        const float w = P.row_weight && r < rows ? P.row_weight[p] : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= w;
        uint2 o = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        if (P.shared8) {  // eight columns: this lane's four and those of the lane 16 beside it
          float m = 0.0f, f;
#pragma unroll
          for (int i = 0; i < 4; ++i) m = __builtin_elementwise_maximum(m, fabsf(v[i]));
          const uint32_t s8 = shared8_exponent(__builtin_elementwise_maximum(m, __shfl_xor(m, 16, kWave)), f);
          o = make_uint2(shared8_word(v[0], v[1], s8, f, 2 * (g & 1)), shared8_word(v[2], v[3], s8, f, 2 * (g & 1) + 1));
        }
        if (r < rows && n < N) *reinterpret_cast<uint2*>(P.out + p * N + n) = o;
      }
    }
  }
}

template <bool GU>
hipError_t launch(const BlockGemmArgs& a, hipStream_t st) {
  Params P{};
  P.M = a.M;
  P.E = a.E;
  P.N = a.N;
  P.K = a.K;
  P.KB = ceil_div(a.K, 128);
  P.NB = ceil_div(a.N, 128);
  P.arows = a.arows;
  P.offsets = a.offsets;
  P.row_token = a.row_token;
  P.a = a.a;
  P.w0 = a.w0;
  P.w1 = a.w1;
  P.sa = a.a_scale;
  P.sw0 = a.w0_scale;
  P.sw1 = a.w1_scale;
  P.row_weight = a.row_weight;
  P.out = static_cast<bf16_t*>(a.out);
  P.shared8 = a.shared8;
  P.aq = a.aq;
  P.sout = a.a_out_scale;
  const unsigned grid = static_cast<unsigned>(gemm_grid());
  // Which kernel (times in us: gate/up + down at 128 experts, 2048 x 768,
  // unless said otherwise; evenly spread rows / rows spread as 1 / rank^1.2):
  //  - few rows: the stream kernel. At 2 rows per expert 65 / 70 against 99 / 69
  //    for 128-row tiles, at 4 71 / 118 against 100 / 93, at 8 71 / 219 against
  //    99 / 105: a long expert's rows pass 32 at a time through the few
  //    workgroups of its columns. One expert has no such skew, and few tiles
  //    fill few CUs: at 4096 x 4096 32 rows take 9 against 34, 192 rows 30
  //    against 41, 256 rows 38 against 41, 512 rows 73 against 43.
  //  - 256-row tiles against 128-row ones: at 96 rows per expert 146 / 232
  //    against 128 / 181, at 128 180 / 250 against 192 / 217, at 256 295 / 340
  //    against 297 / 308, at 512 493 / 487 against 521 / 524.
  const int64_t avg = (a.M + a.E - 1) / a.E;
  const bool one = a.E == 1 && a.M <= 192 && ceil_div(a.N, GU ? BN / 2 : BN) <= 32;
  const bool fits = static_cast<int64_t>(a.E) * ceil_div(a.N, 128) < 1 << 20;  // a launch has less than 2^32 threads
  if ((avg <= 4 || a.M <= 64 || one) && fits) {
    // Enough workgroups to fill the device: split the reduction when there
    // are too few columns.
    int ks = 1;
    if (!GU)
      while (ks < kWaves && static_cast<int64_t>(a.E) * ceil_div(a.N, 16 * kWaves / ks) < 2 * grid && ks < P.KB) ks *= 2;
    const int groups = ceil_div(a.N, 16 * kWaves / ks);
    block_stream_kernel<GU><<<static_cast<unsigned>(a.E) * groups, kThreads, 0, st>>>(P, ks, groups);
  } else if (avg <= 96) {
    block_tile_kernel<GU, 128><<<grid, kThreads, 0, st>>>(P);
  } else {
    block_tile_kernel<GU, 256><<<grid, kThreads, 0, st>>>(P);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp8_block(const BlockGemmArgs& a, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  return a.w1 != nullptr ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace moe
