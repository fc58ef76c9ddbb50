// Grouped products of 8-bit integer operands with one fp32 scale per row of each:
// activations per token, weights per output channel.
//
//   out[p,n] = sa[p] sw[n] sum_k a[p,k] w[n,k]
//
// The sums are whole numbers of at most 2^14 K < 2^31: exact in the matrix
// core's int32 accumulators (v_mfma_i32_16x16x64_i8). The scales multiply the
// finished sums, so nothing but products, LDS reads and loads is in the loop.
//
// Three kernels (launch says which):
//
// i8_tile_kernel, the plain product of many rows: a persistent workgroup of 8
// wavefronts per CU on 256 x 256 tiles, 2 x 4 wavefronts of 128 x 64. Operands go
// from memory straight into LDS, two stages of one 128-wide k-step in halves that
// are refilled as soon as they are read (see there). A row's 128 bytes are eight
// 16-byte chunks, XOR-swizzled by row so that a pass of a read touches every bank
// once. Which weight row sits at which LDS row is chosen so that a lane ends with
// 8 consecutive output columns.
//
// i8_duo_kernel, everything between: two workgroups per CU on 128 x 256 tiles
// (duo.h), gate/up and down.
//
// i8_stream_kernel, for a few rows: bound by the weights' bytes or by latency.
// Weights go from memory into registers steps ahead; with few workgroups of
// work the reduction is split over the wavefronts of one, and the parts meet
// in LDS.
//
// The gate/up forms end with v = silu(g) u, which the down product takes as
// 8-bit codes with one scale per row. A workgroup holds 128 columns of a row,
// not all of them: it writes v in 24 bits (16 and 8 apart), scaled by those 128
// columns' largest magnitude, and launch_requantize_i8_rows (i8.hip) makes the
// codes once all maxima are there. With 16 bits one code in 500 falls on the
// other side of its border, and since a code's step is large beside most of a
// row's values (silu(g) u has long tails) that is y's error 0.0026 instead of
// 0.0017 (192 tokens, 30B shape; bf16 y alone is 0.0016); bf16 in between would move a tenth of them.
#include <type_traits>

#include "duo.h"
#include "shared8.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int KS = 128;                     // k per step
constexpr uint32_t kOutside = 0x80000000u;  // past every buffer's range: loads read zeros

struct Params {
  int M, E, N, K;
  int arows;                // rows of a behind row_token
  const int32_t* offsets;
  const int32_t* row_token;
  const int8_t *a, *w0, *w1;
  const float *sa, *sw0, *sw1;
  const float* row_weight;
  bf16_t* out;
  bool shared8;             // out in shared8.h's form
  int16_t* v16;             // the upper 16 bits of silu(g) u, the lower 8, the maxima
  uint8_t* v8;
  float* amax;
};

// Rows of 128 bytes in LDS: chunk c of row r is at c ^ place8(r). A lane reads a row's
// chunks 2 g and 2 g + 1 (lane / 16 = g), so that places go by pairs (place4).
__device__ __forceinline__ int place8(int r) { return 2 * duo::place4(r >> 2) | (r >> 1 & 1); }

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

__device__ __forceinline__ i32x4 product64(const u32x4& w, const u32x4& a, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
}

// silu(g) u with the hardware exponential and reciprocal (about 1 ulp each;
// the result is rounded to 8 bits).
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f)) * u;
}

// The 24-bit form of values whose largest magnitude is m: kFull24 v / m. A block
// with a NaN has m NaN, and with it the row's scale.
struct Factor24 {
  float up, r;  // up lifts blocks below 2^-64 by 2^64 (exact), so that 2^23 / m stays finite
  __device__ __forceinline__ explicit Factor24(float m) {
    up = m < 0x1p-64f ? 0x1p64f : 1.0f;
    r = m > 0.0f ? kFull24 / (m * up) : 0.0f;
  }
};
// Four values: the upper 16 bits of each, and the lower 8.
struct Packed24 {
  uint32_t hi[2], lo;
  __device__ __forceinline__ Packed24(const f32x4& v, const Factor24& f) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = static_cast<uint32_t>(static_cast<int>(__builtin_rintf(v[i] * f.up * f.r)));
#pragma unroll
    for (int i = 0; i < 2; ++i) hi[i] = __builtin_amdgcn_perm(c[2 * i + 1], c[2 * i], 0x06050201u);
    lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u), __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u),
                               0x05040100u);
  }
};

__device__ __forceinline__ float max4(float m, const f32x4& v) {  // NaN if one is
#pragma unroll
  for (int x = 0; x < 4; ++x) m = __builtin_elementwise_maximum(m, fabsf(v[x]));
  return m;
}
__device__ __forceinline__ float across_groups(float m) {  // lanes 16, 32 and 48 apart
  m = __builtin_elementwise_maximum(m, __shfl_xor(m, 16, kWave));
  return __builtin_elementwise_maximum(m, __shfl_xor(m, 32, kWave));
}

// ---- many rows per expert ---------------------------------------------------

constexpr int BN = 256;
constexpr int kBand = 8;  // row tiles that run side by side over all columns: what an XCD's workgroups read meets in its L2

// A tile's rows come in two halves; a wavefront has half of each. Step s lives
// in stage s % 2, and its loads leave a step and a half before they are used:
// the weights and the first half's rows as soon as every wavefront has taken
// step s - 2's into registers (after that step's middle barrier), the second
// half's rows once step s - 2 has ended. In order of issue:
//   .. | W, A0 of s+1 | A1 of s+1 | W, A0 of s+2 | A1 of s+2 | ..
//         step s-1, 2nd  step s, 1st   step s, 2nd  step s+1, 1st half
// so at each barrier all but the last two groups have landed. A tile's stores run
// on under the next one's first step; the three groups that are on their way by
// then land before the first store (duo.h says why), so that its first two
// barriers wait for none.
__global__ __launch_bounds__(kThreads, 2) void i8_tile_kernel(const Params P) {
  constexpr int BM = 256;
  constexpr int FM = BM / 32, HM = FM / 2;  // 16-row tiles of a per wavefront, and of those per half
  constexpr int HA = BM / 128;              // load instructions of half a's rows per wavefront
  constexpr int OS = BM / 2 * KS;
  constexpr int G1 = HA, G2 = 4 + HA;
  // A stage, in three arrays, so that the compiler sees which reads follow
  // which loads: the weights' rows, the first and the second half's rows of a.
  __shared__ __attribute__((aligned(1024))) uint8_t w0[BN * KS];
  __shared__ __attribute__((aligned(1024))) uint8_t w1[BN * KS];
  __shared__ __attribute__((aligned(1024))) uint8_t x0[OS];
  __shared__ __attribute__((aligned(1024))) uint8_t x1[OS];
  __shared__ __attribute__((aligned(1024))) uint8_t y0[OS];
  __shared__ __attribute__((aligned(1024))) uint8_t y1[OS];
  __shared__ int tstart[1025];
  __shared__ int eoff[1025];
  __shared__ int wsum[kWaves];
  __shared__ __attribute__((aligned(256))) int per_row[kThreads];   // this tile's row weights
  __shared__ __attribute__((aligned(256))) float scale[kThreads];   // its scales: 256 rows, 256 columns

  const int tid = threadIdx.x;
  const int lane_id = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int E = P.E, K = P.K;

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
  const int ntn = (P.N + BN - 1) / BN;
  const int total = tstart[E] * ntn;
  // Eighths of the tile list per XCD, neighbouring tiles on one XCD.
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, nslots = gridDim.x >> 3;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * xcd / 8);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (xcd + 1) / 8);
  const int steps = (K + KS - 1) / KS, padded = (steps + 1) & ~1;
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
    t.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
    return t;
  };
  // The loads' state: resources of their tile, and the lane's offsets.
  rsrc_t ra, rb;
  uint32_t aoff[2 * HA], boff[4];
  auto aim = [&](const Tile& t) __attribute__((always_inline)) {
    const auto* A = args();
    int lane = lane_id;  // opaque: the lane terms are recomputed here, not kept alive
    asm volatile("" : "+v"(lane));
    ra = make_rsrc(A->a + static_cast<int64_t>(t.row0) * K, static_cast<int64_t>(t.valid) * K);
    rb = make_rsrc(A->w0 + static_cast<int64_t>(t.e) * A->N * K, static_cast<int64_t>(A->N) * K);
#pragma unroll
    for (int i = 0; i < 2 * HA; ++i) {
      const int r = (i / HA) * (BM / 2) + (wave * HA + i % HA) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ place8(r);
      aoff[i] = r < t.valid ? static_cast<uint32_t>(r) * K + c * 16 : kOutside;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (wave * 4 + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ place8(r);
      const int j = (r >> 4) & 3, q = r & 15;
      const int n = t.n0 + (r >> 6) * 64 + (j >> 1) * 32 + 8 * (q >> 2) + 4 * (j & 1) + (q & 3);
      boff[i] = n < A->N ? static_cast<uint32_t>(n) * K + c * 16 : kOutside;
    }
  };
  // Load instruction v of step s, of the first (weights W, rows) or the second
  // half's group (rows). Every wavefront issues every one in
  // every step (a branch in the loop costs more than the instruction): chunks
  // past a row's end, and all of a step that is not there, lie outside and
  // read zeros.
  typedef __attribute__((address_space(3))) void* lds_ptr;
  auto load = [&](int h, int v, uint8_t* S, uint8_t* W, int s, bool live) __attribute__((always_inline)) {
    const bool weights = !h && v < 4;
    const int i = weights ? v : h ? v : v - 4, blk = wave * (weights ? 4 : HA) + i;  // eight rows of its array
    const uint32_t to = weights ? boff[i & 3] : aoff[(h * HA + i) % (2 * HA)];
    const int c = (lane_id & 7) ^ place8((blk & 1) * 8 + (lane_id >> 3));
    const uint32_t off = c * 16 < (!live ? 0 : s == steps - 1 ? tail : KS) ? to : kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(weights ? rb : ra, (lds_ptr)((weights ? W : S) + blk * 1024), 16, off,
                                             min(s, steps - 1) * KS, 0, 0);
  };
  // All but the last PENDING memory instructions are done (kAny: as many as there are), and every wavefront is here.
  constexpr int kAny = 63;
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
  // The tile's scales: wavefronts 0 to 3 the rows', 4 to 7 the columns'. One instruction each.
  auto scale_load = [&](const Tile& t) __attribute__((always_inline)) {
    const auto* A = args();
    const int r = wave * 64 + lane_id;
    rsrc_t rs;
    uint32_t off;
    if (wave < 4) {
      rs = make_rsrc(A->sa + t.row0, t.valid * 4ll);
      off = static_cast<uint32_t>(r) * 4;
    } else {
      rs = make_rsrc(A->sw0 + static_cast<int64_t>(t.e) * A->N, A->N * 4ll);
      off = static_cast<uint32_t>(t.n0 + r - 256) * 4;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(reinterpret_cast<char*>(scale) + wave * 256), 4, off, 0, 0, 0);
  };

  i32x4 acc[FM][4];
  u32x4 wf[4][2];
  // Half a step on stage C (the wavefront's 16-row tiles of half h, if NI has
  // them), while the group of step sn goes out into stage D. a's fragments are
  // read one tile ahead.
  auto half = [&](auto nic, auto hc, const uint8_t* C, const uint8_t* CW, uint8_t* D, uint8_t* DW,
                  int sn, bool live) __attribute__((always_inline)) {
    constexpr int NI = decltype(nic)::value, h = decltype(hc)::value;
    constexpr int LD = h ? G2 : G1;  // the second half of a step sends the first half's group
    using group = std::integral_constant<int, h ? 0 : 1>;
    if constexpr (h * HM < NI) {
      int lane = lane_id;
      asm volatile("" : "+v"(lane));
      const int q = lane & 15, o = ((2 * (lane >> 4)) ^ place8(q)) << 4;  // rows 16 apart: the same swizzle
      auto chunk = [&](u32x4(&to)[2], const uint8_t* p) __attribute__((always_inline)) {
        to[0] = *reinterpret_cast<const u32x4*>(p + o);
        to[1] = *reinterpret_cast<const u32x4*>(p + (o ^ 16));
      };
      const uint8_t* wrow = CW + (wn * 64 + q) * KS;
      const uint8_t* arow = C + (wm * (BM / 4) + q) * KS;
      u32x4 af[2][2];
      chunk(af[0], arow);
      if constexpr (h == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) chunk(wf[j], wrow + j * 16 * KS);
      }
#pragma unroll
      for (int i = 0; i < HM; ++i) {
        if (i + 1 < HM) chunk(af[(i + 1) & 1], arow + (i + 1) * 16 * KS);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[h * HM + i][j] = product64(wf[j][k], af[i & 1][k], acc[h * HM + i][j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int v = i * LD / HM; v < (i + 1) * LD / HM; ++v) load(group::value, v, D, DW, sn, live);
        __builtin_amdgcn_sched_barrier(0);
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
      for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{};
    // Steps s (x0, y0) and s + 1 (x1, y1). From the middle of the last
    // pair on the loads are the next tile's.
    auto pair = [&](auto firstc, int s) __attribute__((always_inline)) {
      constexpr bool first = decltype(firstc)::value != 0;
      using pending = std::integral_constant<int, first ? kAny : G1 + G2>;
      const bool last = s + 2 == padded;
      half(nic, none{}, x0, w0, y1, nullptr, s + 1, s + 1 < steps);  // an odd count's last step: zeros
      landed(pending{});
      if constexpr (first) {  // every wavefront has left the previous tile's epilogue
        scale_load(now);
        if (const float* w = args()->row_weight; w != nullptr) per_row_load(w, now.row0, now.valid);
      }
      if (last && more) {
        nx = find(next);
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
    // ---- epilogue
    const auto* A = args();
    const int lane = lane_id, g = lane >> 4, q = lane & 15;
    const int row0 = now.row0, valid = now.valid, n0 = now.n0;
    auto columns = [&](int at) __attribute__((always_inline)) { return *reinterpret_cast<const f32x4*>(&scale[256 + at]); };
    const rsrc_t ro = make_rsrc(A->out + static_cast<int64_t>(row0) * A->N, static_cast<int64_t>(valid) * A->N * 2);
    f32x4 cs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[j] = columns(wn * 64 + (j >> 1) * 32 + 8 * g + 4 * (j & 1));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = row_of(i, q);
      const float rs = scale[r] * (A->row_weight != nullptr ? __int_as_float(per_row[r]) : 1.0f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = n0 + wn * 64 + 32 * h + 8 * g;
        u32x4 o;
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          v[c] = static_cast<float>(acc[i][2 * h + c / 4][c % 4]) * cs[2 * h + c / 4][c % 4] * rs;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
        if (i == 0 && h == 0) duo::loads_landed();
        __builtin_amdgcn_raw_buffer_store_b128(
            o, ro, r < valid && n < A->N ? (static_cast<uint32_t>(r) * A->N + n) * 2 : kOutside, 0, 0);
      }
    }
    now = nx;
    L = next;
  };

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
  landed(none{});  // nothing is on its way into LDS when the workgroup ends
}

// ---- up to some hundred rows per expert: two workgroups per CU (duo.h) ----------

struct DuoParams : duo::Base {
  const float *sa, *sw0, *sw1;
  const float* row_weight;
  bf16_t* out;
  int16_t* v16;
  uint8_t* v8;
  float* amax;
};

// GU: gate/up with silu(g) u in 24 bits; else the plain product, S8 in shared8.h's
// form. The extras: scales of 256 rows and 256 columns, then the rows' weights, or
// their maxima over each wavefront's columns.
template <bool GU, bool S8>
struct I8Op {
  typedef DuoParams Params;
  typedef const __attribute__((address_space(4))) Params* args_t;
  typedef i32x4 Acc;
  static constexpr bool PAIRED = GU, GATHER = GU, KROWS = false;
  static constexpr int EXTRA = 4 * (2 * duo::BN + (GU ? 2 * duo::BM : duo::BM));

  static __device__ __forceinline__ Acc product(const u32x4& w, const u32x4& a, const Acc& c) { return product64(w, a, c); }

  static __device__ __forceinline__ void begin(args_t A, const duo::Tile& t, const int* per_row, char* extra, int wave,
                                               int lane) {
    const int r = wave * 64 + lane;
    const rsrc_t rr = make_rsrc(A->sa + (GU ? 0 : t.row0), (GU ? A->arows : t.valid) * 4ll);
    duo::words_to_lds(rr, extra + wave * 256,
                      r < t.valid ? static_cast<uint32_t>(GU ? per_row[r & (duo::BM - 1)] : r) * 4 : kOutside);
    const int n = t.n0 + (GU ? r & 127 : r);
    const rsrc_t rc = make_rsrc((GU && wave >= 2 ? A->sw1 : A->sw0) + static_cast<int64_t>(t.e) * A->N, A->N * 4ll);
    duo::words_to_lds(rc, extra + 4 * duo::BN + wave * 256, n < A->N ? static_cast<uint32_t>(n) * 4 : kOutside);
    if constexpr (!GU)
      if (A->row_weight != nullptr && wave < duo::BM / kWave)
        duo::words_to_lds(make_rsrc(A->row_weight + t.row0, t.valid * 4ll), extra + 8 * duo::BN + wave * 256, r * 4);
  }

  template <int NI>
  static __device__ __forceinline__ void finish(args_t A, Acc (&acc)[duo::FM][duo::FN], const duo::Tile& t, char* extra,
                                                const duo::Where& w) {
    const int g = w.g, wn = w.wn, n0 = t.n0, valid = t.valid;
    const float* scale = reinterpret_cast<const float*>(extra);
    auto columns = [&](int at) __attribute__((always_inline)) {
      return *reinterpret_cast<const f32x4*>(&scale[duo::BN + at]);
    };
    f32x4 cs[8];
    if constexpr (GU) {
      float(&amax)[duo::BM][2] = *reinterpret_cast<float(*)[duo::BM][2]>(extra + 8 * duo::BN);
      const int NT = (A->N + 127) / 128;
      const rsrc_t rv = make_rsrc(A->v16 + static_cast<int64_t>(t.row0) * A->N, static_cast<int64_t>(valid) * A->N * 2);
      const rsrc_t rl = make_rsrc(A->v8 + static_cast<int64_t>(t.row0) * A->N, static_cast<int64_t>(valid) * A->N);
      const rsrc_t rm = make_rsrc(A->amax + static_cast<int64_t>(t.row0) * NT, static_cast<int64_t>(valid) * NT * 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = columns((j >> 2) * 128 + wn * 64 + ((j >> 1) & 1) * 32 + 8 * g + 4 * (j & 1));
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = w.row(i);
        const float rs = scale[r];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 v;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            v[x] = silu_mul(static_cast<float>(acc[i][j][x]) * (rs * cs[j][x]),
                            static_cast<float>(acc[i][j + 4][x]) * (rs * cs[j + 4][x]));
          m = max4(m, v);
          acc[i][j] = __builtin_bit_cast(i32x4, v);
        }
        m = across_groups(m);
        if (g == 0) amax[r][wn] = m;
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      duo::loads_landed();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = w.row(i);
        const bool row = r < valid;
        const float m = __builtin_elementwise_maximum(amax[r][0], amax[r][1]);
        const Factor24 f(m);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Packed24 p0(__builtin_bit_cast(f32x4, acc[i][2 * h]), f), p1(__builtin_bit_cast(f32x4, acc[i][2 * h + 1]), f);
          const u32x4 o{p0.hi[0], p0.hi[1], p1.hi[0], p1.hi[1]};
          const u32x2 low{p0.lo, p1.lo};
          const int n = n0 + wn * 64 + 32 * h + 8 * g;
          const uint32_t to = row && n < A->N ? static_cast<uint32_t>(r) * A->N + n : kOutside;
          __builtin_amdgcn_raw_buffer_store_b128(o, rv, to == kOutside ? to : 2 * to, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b64(low, rl, to, 0, 0);
        }
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(m), rm, row && wn == 0 && g == 0 ? (static_cast<uint32_t>(r) * NT + n0 / 128) * 4 : kOutside, 0,
            0);
      }
    } else {
      const rsrc_t ro = make_rsrc(A->out + static_cast<int64_t>(t.row0) * A->N, static_cast<int64_t>(valid) * A->N * 2);
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = columns(wn * 128 + (j >> 1) * 32 + 8 * g + 4 * (j & 1));
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = w.row(i);
        const float rs = scale[r] * (A->row_weight != nullptr ? scale[2 * duo::BN + r] : 1.0f);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int n = n0 + wn * 128 + 32 * h + 8 * g;
          u32x4 o;
          float v[8], m = 0.0f;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            v[c] = static_cast<float>(acc[i][2 * h + c / 4][c % 4]) * cs[2 * h + c / 4][c % 4] * rs;
            if constexpr (S8) m = __builtin_elementwise_maximum(m, fabsf(v[c]));  // NaN if one is
          }
          float f = 0.0f;
          uint32_t s = 0;
          if constexpr (S8) s = shared8_exponent(m, f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if constexpr (S8) o[c] = shared8_word(v[2 * c], v[2 * c + 1], s, f, c);
            else o[c] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
          }
          if (i == 0 && h == 0) duo::loads_landed();
          __builtin_amdgcn_raw_buffer_store_b128(
              o, ro, r < valid && n < A->N ? (static_cast<uint32_t>(r) * A->N + n) * 2 : kOutside, 0, 0);
        }
      }
    }
  }
};

template <bool GU, bool S8>
MOE_DUO_KERNEL void i8_duo_kernel(const DuoParams P) {
  duo::run<I8Op<GU, S8>>(P);
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
__global__ __launch_bounds__(kThreads, 2) void i8_stream_kernel(const Params P, int ks, int groups) {
  __shared__ __attribute__((aligned(16))) int red[kWaves][16][20];
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][GU ? 3 : 2][16 * KS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane & 15, g = lane >> 4;
  const int lr = lane >> 3, lc = lane & 7;  // as a loader: row, chunk
  const int e = blockIdx.x / groups, grp = blockIdx.x - e * groups;
  const int first = P.offsets ? P.offsets[e] : 0;
  const int rows = (P.offsets ? P.offsets[e + 1] : P.M) - first;
  if (rows <= 0) return;
  const int K = P.K, KB = (K + KS - 1) / KS, N = P.N;
  const int cw = GU ? wave : wave / ks, kp = GU ? 0 : wave - cw * ks;
  const int n0 = (grp * (GU ? kWaves : kWaves / ks) + cw) * 16;
  const int s0 = kp * KB / ks, s1 = (kp + 1) * KB / ks;
  const int64_t wbytes = static_cast<int64_t>(N) * K;
  const rsrc_t r0 = make_rsrc(P.w0 + e * wbytes, wbytes);
  const rsrc_t r1 = make_rsrc((GU ? P.w1 : P.w0) + e * wbytes, wbytes);
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
  };
  auto put = [&](uint8_t* to, const u32x4(&v)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lr + 8 * i;
      *reinterpret_cast<u32x4*>(to + r * KS + ((lc ^ place8(r)) << 4)) = v[i];
    }
  };
  auto fragment = [&](u32x4(&to)[2], const uint8_t* from) __attribute__((always_inline)) {
    const uint8_t* p = from + q * KS;
    const int o = ((2 * g) ^ place8(q)) << 4;
    to[0] = *reinterpret_cast<const u32x4*>(p + o);
    to[1] = *reinterpret_cast<const u32x4*>(p + (o ^ 16));
  };
  // The scales of this lane's four columns, the same for every row.
  f32x4 c0{}, c1{};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * g + i;
    if (n < N) c0[i] = P.sw0[static_cast<int64_t>(e) * N + n];
    if (GU && n < N) c1[i] = P.sw1[static_cast<int64_t>(e) * N + n];
  }
  for (int p0 = 0; p0 < rows; p0 += 16 * kTiles) {
    const int tiles = min(kTiles, (rows - p0 + 15) / 16);
    const int64_t base = GU ? 0 : first + p0;
    const int64_t left = GU ? P.arows : min(rows - p0, 16 * kTiles);
    const rsrc_t ra = make_rsrc(P.a + base * K, left * K);
    uint32_t xoff[kTiles][2];
    float sr[kTiles];
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
      sr[t] = x >= 0 ? P.sa[base + x] * (!GU && P.row_weight ? P.row_weight[first + p0 + 16 * t + q] : 1.0f) : 0.0f;
    }
    Step st[kAhead];
    auto fetch = [&](Step& f, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f.w0[i] = b128(r0, at(woff[i], s));
        if constexpr (GU) f.w1[i] = b128(r1, at(woff[i], s));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) f.x[i] = b128(ra, at(xoff[0][i], s));
    };
    i32x4 a0[kTiles], a1[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) a0[t] = a1[t] = i32x4{};
#pragma unroll
    for (int d = 0; d < kAhead; ++d) fetch(st[d], s0 + d);
    auto batch = [&](auto more, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        uint8_t* own = stage[wave][0];
        put(own, st[d].w0);
        if constexpr (GU) put(own + 2 * 16 * KS, st[d].w1);
        put(own + 16 * KS, st[d].x);
        u32x4 wf0[2], wf1[2];
        fragment(wf0, own);
        if constexpr (GU) fragment(wf1, own + 2 * 16 * KS);
        auto tile = [&](int t) __attribute__((always_inline)) {
          u32x4 x[2];
          fragment(x, own + 16 * KS);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            a0[t] = product64(wf0[k], x[k], a0[t]);
            if constexpr (GU) a1[t] = product64(wf1[k], x[k], a1[t]);
          }
        };
        tile(0);  // past the steps: zeros
#pragma unroll
        for (int t = 1; t < kTiles; ++t) {
          if (t >= tiles) break;
          const u32x4 x[2] = {b128(ra, at(xoff[t][0], s + d)), b128(ra, at(xoff[t][1], s + d))};
          put(own + 16 * KS, x);
          tile(t);
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
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = silu_mul(static_cast<float>(a0[t][i]) * (sr[t] * c0[i]), static_cast<float>(a1[t][i]) * (sr[t] * c1[i]));
        float m = across_groups(max4(0.0f, v));
        __syncthreads();  // the previous tile's maxima are read
        if (g == 0) red[wave][q][0] = __float_as_int(m);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = __builtin_elementwise_maximum(m, __int_as_float(red[w][q][0]));
        if (r < rows) {
          if (n < N) {
            const Packed24 o(v, Factor24(m));
            *reinterpret_cast<uint2*>(P.v16 + p * N + n) = make_uint2(o.hi[0], o.hi[1]);
            *reinterpret_cast<uint32_t*>(P.v8 + p * N + n) = o.lo;
          }
          if (wave == 0 && g == 0) P.amax[p * ((N + 127) / 128) + grp] = m;
        }
      } else {
        i32x4 sum = a0[t];
        if (ks > 1) {  // the parts along k: whole numbers, in any order
          __syncthreads();
          *reinterpret_cast<i32x4*>(&red[wave][q][4 * g]) = sum;
          __syncthreads();
          if (kp != 0) continue;
          for (int w = 1; w < ks; ++w) sum += *reinterpret_cast<const i32x4*>(&red[wave + w][q][4 * g]);
        }
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(sum[i]) * (sr[t] * c0[i]);
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

// Which kernel, in us:
//   Few rows: the weights are read once whatever the tile, so what counts is how
//   early their loads leave. stream | duo, one expert with N = K = 4096: 32 rows
//   8.4 | 26.4, 64 12.3 | 27.8, 128 20.9 | 31.1, 192 29.4 | 30.6, 256 37.8 | 31.2.
//   Several experts: the stream kernel takes an expert's rows 32 at a time and
//   reads its weights for each again, so that the longest expert sets the time.
//   16 of 2048 x 2048 with 4 rows each 13.6 | 16.6; a whole stage of 128 experts
//   (2048 x 768, top-8) of 65 tokens 123 | 133 evenly spread and 99 | 84 with
//   their ranks' 1.2th powers, of 128 tokens 127 | 137 and 142 | 95. Four rows per
//   expert is where the loss from skew passes the gain.
//   Many rows: 256-row tiles need full ones and enough of them for every CU.
//   tile | duo, one expert with N = K = 4096: 1024 rows 52 | 33, 2048 53 | 40, 4096
//   60 | 70, 8192 118 | 141; 128 experts, 2048 x 768, of 256 rows each 89 | 96, of
//   512 144 | 169; 32 experts of 512 rows 42 | 48, of 1024 73 | 89. Gate/up and the
//   shared8 form have longer epilogues, which the second workgroup hides: 4096
//   skewed tokens of the stage above 207 | 177 and 136 | 118 with the same LDS
//   places in both.
template <bool GU>
hipError_t launch(const I8GemmArgs& a, hipStream_t st) {
  Params P{};
  P.M = a.M;
  P.E = a.E;
  P.N = a.N;
  P.K = a.K;
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
  P.v16 = a.v16;
  P.v8 = a.v8;
  P.amax = a.amax;
  const unsigned grid = static_cast<unsigned>(gemm_grid());
  const int KB = ceil_div(a.K, KS);
  const int64_t avg = (a.M + a.E - 1) / a.E;
  const bool one = a.E == 1 && a.M <= 192 && ceil_div(a.N, GU ? BN / 2 : BN) <= 32;
  const bool fits = static_cast<int64_t>(a.E) * ceil_div(a.N, 128) < 1 << 20;  // a launch has less than 2^32 threads
  if ((avg <= 4 || a.M <= 64 || one) && fits) {
    // Enough workgroups to fill the device: split the reduction when there
    // are too few columns.
    int ks = 1;
    if (!GU)
      while (ks < kWaves && static_cast<int64_t>(a.E) * ceil_div(a.N, 16 * kWaves / ks) < 2 * grid && ks < KB) ks *= 2;
    const int groups = ceil_div(a.N, 16 * kWaves / ks);
    i8_stream_kernel<GU><<<static_cast<unsigned>(a.E) * groups, kThreads, 0, st>>>(P, ks, groups);
  } else if (!GU && !a.shared8 && avg >= 256 && (a.M / 256) * static_cast<int64_t>(ceil_div(a.N, BN)) >= grid) {
    i8_tile_kernel<<<grid, kThreads, 0, st>>>(P);
  } else {
    DuoParams D{};
    D.M = a.M;
    D.E = a.E;
    D.N = a.N;
    D.K = a.K;
    D.arows = a.arows;
    D.offsets = a.offsets;
    D.row_token = a.row_token;
    D.a = reinterpret_cast<const uint8_t*>(a.a);
    D.w0 = reinterpret_cast<const uint8_t*>(a.w0);
    D.w1 = reinterpret_cast<const uint8_t*>(a.w1);
    D.sa = a.a_scale;
    D.sw0 = a.w0_scale;
    D.sw1 = a.w1_scale;
    D.row_weight = a.row_weight;
    D.out = static_cast<bf16_t*>(a.out);
    D.v16 = a.v16;
    D.v8 = a.v8;
    D.amax = a.amax;
    if (!GU && a.shared8) i8_duo_kernel<GU, !GU><<<2 * grid, duo::kThreads, 0, st>>>(D);
    else i8_duo_kernel<GU, false><<<2 * grid, duo::kThreads, 0, st>>>(D);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const I8GemmArgs& a, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  return a.w1 != nullptr ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace moe
