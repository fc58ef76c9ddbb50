// The walk of a grouped product over its tiles with two workgroups per CU, for
// operands whose reduction rows are read 64 bytes at a time: whole numbers of 8
// bits (64 per step) and bf16 (32).
//
// A workgroup is 4 wavefronts on 128 x 256 tiles (128 rows of one expert), 2 x 2
// wavefronts of 64 x 128; it holds half of the CU's LDS and registers, so two of
// them run side by side and out of step: one's results (scaling, packing, stores)
// go out under the other's products, and what one waits for at its barrier the
// other fills. 256 x 256 tiles of 8 wavefronts, one workgroup per CU, read each
// operand half as often and are a tenth faster where the products are most of the
// work (int8 8192 x 4096 x 4096 118 us against 141, bf16 8192 rows per expert 391
// against 413), but stand still during their epilogue and half empty with few
// rows; where the kernels are chosen both sides are given.
//
// Operands go from memory straight into LDS, a ring of three stages of one step
// each; loads leave two steps before they are read. One barrier per step: after
// it every wavefront's loads for this step have landed, and the stage read in
// the step before is free.
//
// OP is the product: its operands' kind, what it keeps of a tile besides them and
// what becomes of the sums. It gives
//   Params    a struct that begins with Base; the kernel's only argument
//   PAIRED    columns of w0 and of w1 side by side, 128 of each (TN = 128)
//   GATHER    rows of a through row_token
//   KROWS     the weights' reduction index is their strided one ([K][N], bf16);
//             then acc[i][j][x] is column 16 j + 4 g + x
//   EXTRA     bytes of LDS for what begin() fetches
//   Acc, product(w, a, acc)
//   begin     sends for the tile's extras, into LDS; per_row: its tokens (GATHER)
//   finish    the epilogue; calls loads_landed() before its first store
//
// The counter of memory instructions says how many are left, not which. A tile's
// stores run on under the next one's first two steps, so those steps' loads have
// to be done before the first store goes out (loads_landed): no wait then counts
// stores, whose number is the compiler's affair (it joins equal neighbours). It
// costs up to 2% (int8 experts of 4096 skewed tokens 352 -> 356 us, 65536 rows over
// 128 experts none) beside a wait that counts them.
#pragma once
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace duo {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kThreads = 256;
constexpr int BM = 128, BN = 256;           // a tile's rows and weight rows
constexpr int FM = 4, FN = 8;               // a wavefront's 16-row tiles of a and of the weights
constexpr int KB = 64;                      // bytes of a reduction row per step
constexpr int kRing = 3;                    // stages of LDS
constexpr int LA = 2, LOADS = LA + 4;       // load instructions per wavefront and step: a's rows, all
constexpr int kEarly = LOADS / 2;           // of a step's, those sent before its products; the others go between them
constexpr int SA = BM * KB, STAGE = SA + BN * KB;
constexpr int kBand = 8;                    // row tiles that run side by side over all columns: what an XCD's workgroups read meets in its L2
constexpr uint32_t kOutside = 0x80000000u;  // past every buffer's range: loads read zeros, stores write nothing

struct Base {
  int M, E, N;
  int K;                    // bytes of a reduction row
  int arows;                // GATHER: rows of a
  const int32_t* offsets;   // NULL: one expert, every row
  const int32_t* row_token;
  const uint8_t *a, *w0, *w1;
};

// Which 16-byte chunk of LDS rows a read takes, by four rows: what rows t * 4 .. + 3
// XOR into the chunk's place. A ds_read_b128 goes through in four passes, the first
// two of lanes {0-3, 12-15, 20-23, 24-27} and {4-7, 8-11, 16-19, 28-31}, the others
// 32 on. With 16 rows in lanes 0-15 and the next chunk of the same rows in lanes
// 16-31, the places 0, 2, 3, 1 keep each pass on different banks (t itself does
// not: half of the LDS cycles were conflicts).
__device__ __forceinline__ int place4(int t) { return 0x78 >> 2 * (t & 3) & 3; }

__device__ __forceinline__ int kflip(int k) { return (k & 3) | (k >> 1 & 4); }

struct Tile {
  int e, row0, valid, n0;
};

// Where a wavefront's sums are: acc[i][j][x] is row (2 i + wm) * 16 + q and, for
// the pair h = j / 2 of weight tiles, column 32 h + 8 g + 4 (j % 2) + x of its
// 128 (PAIRED: of its 64 of w0 for j < 4, of w1 for the others).
struct Where {
  int wave, lane, wm, wn, g, q;
  __device__ __forceinline__ int row(int i) const { return (2 * i + wm) * 16 + q; }
};

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

// 64 words from base, one per lane, into LDS.
__device__ __forceinline__ void words_to_lds(const rsrc_t& r, char* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)to, 4, off, 0, 0, 0);
}

// Every load of this wavefront has landed.
__device__ __forceinline__ void loads_landed() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ float across_groups_max(float m) {  // lanes 16, 32 and 48 apart; NaN if one is
  m = __builtin_elementwise_maximum(m, __shfl_xor(m, 16, kWave));
  return __builtin_elementwise_maximum(m, __shfl_xor(m, 32, kWave));
}

template <class OP>
__device__ __forceinline__ void run(const typename OP::Params& P) {
  typedef typename OP::Acc Acc;
  typedef const __attribute__((address_space(4))) typename OP::Params* args_t;
  constexpr int TN = OP::PAIRED ? BN / 2 : BN;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[STAGE];
  __shared__ __attribute__((aligned(256))) char extra[OP::EXTRA];
  __shared__ __attribute__((aligned(256))) int per_row[OP::GATHER ? BM : 1];  // the next tile's tokens
  __shared__ int tstart[1025];
  __shared__ int wsum[kThreads / kWave];

  const int tid = threadIdx.x;
  const int lane_id = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int E = P.E, K = P.K;
  {  // tstart[e]: row tiles of the experts before e (four experts per thread)
    int c[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * tid + i;
      const int b = e < E && P.offsets ? P.offsets[e] : 0;
      const int t = e < E ? (P.offsets ? P.offsets[e + 1] : P.M) : 0;
      c[i] = e < E ? (t - b + BM - 1) / BM : 0;
      mine += c[i];
    }
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * tid + i < E) tstart[4 * tid + i] = at;
      at += c[i];
    }
    if (tid == kThreads - 1) tstart[E] = at;
    __syncthreads();
  }
  const int ntn = (P.N + TN - 1) / TN;
  const int total = tstart[E] * ntn;
  // Eighths of the tile list per XCD, neighbouring tiles on one XCD.
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, nslots = gridDim.x >> 3;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * xcd / 8);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (xcd + 1) / 8);
  const int steps = (K + KB - 1) / KB, padded = (steps + kRing - 1) / kRing * kRing;
  int L = lo + slot;
  if (L >= hi) return;

  // The arguments, read again where a tile begins or ends: kept in scalar
  // registers through the loop they cost spills, whose reloads wait for every
  // load in flight.
  auto args = [&]() __attribute__((always_inline)) {
    uintptr_t u = reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(u));
    return reinterpret_cast<args_t>(u);
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
    const int32_t* off = args()->offsets;
    const int begin = off ? off[t.e] : 0, end = off ? off[t.e + 1] : args()->M;
    t.row0 = __builtin_amdgcn_readfirstlane(begin + mt * BM);
    t.valid = __builtin_amdgcn_readfirstlane(min(BM, end - begin - mt * BM));
    t.n0 = __builtin_amdgcn_readfirstlane(nt * TN);
    return t;
  };
  // LDS of a stage. a, and weights whose rows are the output's columns: row r is
  // 64 bytes, chunk c of 16 at c ^ place4(r / 4); row r of the weights holds the
  // column that makes a lane's results neighbours (Where). KROWS: reduction row k is 256 columns,
  // chunk c at c ^ 2 kflip(k): a transposing read takes 32 bytes each of rows
  // 8 g .. 8 g + 3, which with those of two neighbouring g touch every bank once.
  rsrc_t ra, rb;
  uint32_t aoff[LA], boff[4];
  auto aim = [&](const Tile& t) __attribute__((always_inline)) {
    const args_t A = args();
    int lane = lane_id;  // opaque: the lane terms are recomputed here, not kept alive
    asm volatile("" : "+v"(lane));
    const int64_t first = OP::GATHER ? 0 : t.row0, rows = OP::GATHER ? A->arows : t.valid;
    ra = make_rsrc(A->a + first * K, rows * K);
    // KROWS: K / 2 rows of 2 N bytes, the same size
    const int64_t size = static_cast<int64_t>(A->N) * K;
    rb = make_rsrc((OP::PAIRED && (wave & 1) ? A->w1 : A->w0) + t.e * size, size);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = (wave * LA + i) * 16 + (lane >> 2);
      const int c = (lane & 3) ^ place4(r >> 2);
      const int row = OP::GATHER ? (r < t.valid ? per_row[r] : 0) : r;
      aoff[i] = r < t.valid ? static_cast<uint32_t>(row) * K + c * 16 : kOutside;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (OP::KROWS) {
        const int k = (wave * 4 + i) * 2 + (lane >> 5);
        const int n = t.n0 + ((lane & 31) ^ (kflip(k) << 1)) * 8;
        boff[i] = n < A->N ? (static_cast<uint32_t>(k) * A->N + n) * 2 : kOutside;
      } else {
        const int r = (wave * 4 + i) * 16 + (lane >> 2);
        const int c = (lane & 3) ^ place4(r >> 2);
        const int j = (r >> 4) & (OP::PAIRED ? 3 : 7), q = r & 15;
        const int n = t.n0 + (r >> 7) * (OP::PAIRED ? 64 : 128) + (j >> 1) * 32 + 8 * (q >> 2) + 4 * (j & 1) + (q & 3);
        boff[i] = n < A->N ? static_cast<uint32_t>(n) * K + c * 16 : kOutside;
      }
    }
  };
  // Load instruction v of a step whose bytes begin at sa (a's rows) and sb (the
  // weights) and of which k are there (0: a step that is not). Every wavefront
  // issues every one in every step.
  auto load = [&](int v, uint8_t* S, int sa, int sb, int k) __attribute__((always_inline)) {
    const bool weights = v < 4;
    const int i = weights ? v : v - 4, blk = weights ? wave * 4 + i : wave * LA + i;
    const int c = (lane_id & 3) ^ place4(lane_id >> 4);  // of the lane's row: r >> 2 & 3 = lane >> 4
    const uint32_t to = weights ? boff[i & 3] : aoff[i % LA];
    const uint32_t off = (weights && OP::KROWS ? 0 : c * 16) < k ? to : kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(weights ? rb : ra, (lds_ptr)(S + (weights ? SA : 0) + blk * 1024), 16, off,
                                             weights && OP::KROWS ? sb : sa, 0, 0);
  };
  struct From {
    int sa, sb, k;
  };
  auto step_at = [&](int s, bool live) __attribute__((always_inline)) {
    const int at = __builtin_amdgcn_readfirstlane(min(s, steps - 1));  // inside the rows also where nothing is read
    From f{at * KB, 0, __builtin_amdgcn_readfirstlane(live ? min(K - s * KB, KB) : 0)};
    if constexpr (OP::KROWS) f.sb = at * (KB / 2) * 2 * args()->N;
    asm volatile("" : "+s"(f.k));  // a select, not a branch
    return f;
  };
  auto landed = [&](auto pending) __attribute__((always_inline)) {
    constexpr int n = decltype(pending)::value;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);  // vmcnt(n) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  using none = std::integral_constant<int, 0>;
  auto tokens_load = [&](const Tile& t) __attribute__((always_inline)) {
    if (wave >= BM / kWave) return;
    words_to_lds(make_rsrc(args()->row_token + t.row0, t.valid * 4ll), reinterpret_cast<char*>(per_row) + wave * 256,
                 (wave * 64 + lane_id) * 4);
  };

  Acc acc[FM][FN];
  u32x4 fa[2], fb[FN];
  int fo, fk;  // the lane's byte in a 16-row tile, and in KROWS' weights
  {
    const int q = lane_id & 15, g = lane_id >> 4, k = 8 * g + (q >> 2);
    fo = q * KB + ((g ^ place4(q >> 2)) << 4);
    fk = k * (BN * 2) + ((wn * 16 + ((q & 3) >> 1)) ^ (kflip(k) << 1)) * 16 + (q & 1) * 8;
  }
  // The wavefront's 16-row tile i is the tile's 2 i + wm: both halves of a short tile have rows.
  auto read_a = [&](u32x4& to, const uint8_t* S, int i) __attribute__((always_inline)) {
    to = *reinterpret_cast<const u32x4*>(S + (2 * i + wm) * (16 * KB) + fo);
  };
  auto read_b = [&](u32x4& to, const uint8_t* S, int j) __attribute__((always_inline)) {
    if constexpr (OP::KROWS) {
      // Lane m of group g addresses four columns of reduction row 8 g + m / 4, then
      // of the fourth row after it (the same kflip), and gets four rows of column m.
      const uint8_t* p = S + SA + (fk ^ (j << 5));
      typedef __attribute__((address_space(3))) i16x4* tr_ptr;
      const i16x4 two[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)p),
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)(p + 4 * BN * 2))};
      to = __builtin_bit_cast(u32x4, two);
    } else {
      to = *reinterpret_cast<const u32x4*>(S + SA + (wn * 8 + j) * (16 * KB) + fo);
    }
  };
  // Step s on stage C, while the loads of step sn go out into stage D. `there`: the
  // step's loads were done before the last tile's stores, which are still under way.
  auto kstep = [&](auto nic, auto firstc, bool there, const uint8_t* C, uint8_t* D, int sn, bool live,
                   auto&& after) __attribute__((always_inline)) {
    constexpr int NI = decltype(nic)::value;
    constexpr bool first = decltype(firstc)::value != 0;
    asm volatile("" ::: "memory");
    if (there) __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    else __builtin_amdgcn_s_waitcnt(0x0070 | (LOADS & 15) | (LOADS >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    after();
    const From f = step_at(sn, live);
    read_a(fa[0], C, 0);
#pragma unroll
    for (int j = 0; j < FN; ++j) read_b(fb[j], C, j);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int v = 0; v < kEarly; ++v) load(v, D, f.sa, f.sb, f.k);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);  // products before the other workgroup's loads and results
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i + 1 < NI) read_a(fa[(i + 1) & 1], C, i + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = OP::product(fb[j], fa[i & 1], first ? Acc{} : acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = kEarly + i * (LOADS - kEarly) / NI; v < kEarly + (i + 1) * (LOADS - kEarly) / NI; ++v) load(v, D, f.sa, f.sb, f.k);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };

  Tile now = find(L), nx = now;
  using zero = std::integral_constant<int, 0>;
  using one = std::integral_constant<int, 1>;
  auto tile = [&](auto nic) __attribute__((always_inline)) {
    constexpr int NI = decltype(nic)::value;
    const int next = L + nslots;
    const bool more = next < hi;
    auto nothing = [] {};
    // Step s is read after its own barrier, at which all but step s + 1's loads
    // have landed (steps 0 and 1: all); step s + 2's go out then.
    auto send_tokens = [&]() __attribute__((always_inline)) {  // every wavefront has left begin()
      if (!more) return;
      nx = find(next);
      tokens_load(nx);
    };
    auto turn = [&]() __attribute__((always_inline)) {
      if (more) {
        if constexpr (!OP::GATHER) nx = find(next);
        if (OP::GATHER && padded == kRing) {  // there was no step to send for the tokens in
          send_tokens();
          landed(none{});
        }
        aim(nx);
      }
    };
    kstep(nic, one{}, true, lds0, lds2, 2, 2 < steps, [&]() __attribute__((always_inline)) {
      // Every wavefront has left the previous tile's epilogue.
      OP::begin(args(), now, per_row, extra, wave, lane_id);
    });
    for (int s = kRing; s < padded; s += kRing) {  // steps s - 2 .. s
      kstep(nic, zero{}, s == kRing, lds1, lds0, s, s < steps, [&]() __attribute__((always_inline)) {
        if (OP::GATHER && s == kRing) send_tokens();
      });
      kstep(nic, zero{}, false, lds2, lds1, s + 1, s + 1 < steps, nothing);
      kstep(nic, zero{}, false, lds0, lds2, s + 2, s + 2 < steps, nothing);
    }
    kstep(nic, zero{}, padded == kRing, lds1, lds0, 0, more, turn);
    kstep(nic, zero{}, false, lds2, lds1, 1, more && steps > 1, nothing);
    const Where w{wave, lane_id, wm, wn, lane_id >> 4, lane_id & 15};
    OP::template finish<NI>(args(), acc, now, extra, w);
    now = nx;
    L = next;
  };

  if constexpr (OP::GATHER) {
    tokens_load(now);
    landed(none{});
  }
  aim(now);
  {
    const From f0 = step_at(0, true), f1 = step_at(1, steps > 1);
#pragma unroll
    for (int v = 0; v < LOADS; ++v) load(v, lds0, f0.sa, f0.sb, f0.k);
#pragma unroll
    for (int v = 0; v < LOADS; ++v) load(v, lds1, f1.sa, f1.sb, f1.k);
  }
  landed(none{});
  while (L < hi) {
    if (now.valid > 64) tile(std::integral_constant<int, 4>{});
    else if (now.valid > 32) tile(std::integral_constant<int, 2>{});
    else tile(std::integral_constant<int, 1>{});
  }
  landed(none{});  // nothing is on its way into LDS when the workgroup ends
}

// A kernel's attributes.
#define MOE_DUO_KERNEL \
  __global__ __attribute__((amdgpu_flat_work_group_size(moe::duo::kThreads, moe::duo::kThreads), amdgpu_waves_per_eu(2, 2)))

}  // namespace duo
}  // namespace moe
