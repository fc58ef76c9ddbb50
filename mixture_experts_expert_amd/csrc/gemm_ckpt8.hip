// The two grouped products of a training step that keeps g and u in 8 bits: bf16
// products (v_mfma_f32_16x16x32_bf16, fp32 sums) on the walk of duo.h, and the
// codes in their epilogues.
//
//   gate/up:    g = x w_gate^T, u = x w_up^T  ->  codes of g and u, a = silu(g) u
//   down dgrad: dA = dy w_down  ->  with w the row's weight and a = silu(g) u from
//               the codes: dG = w dA u silu'(g), dU = w dA silu(g), a_w = w a and
//               each row's <dA, a>, which is the gradient of w
//
// Codes: per row and 64 columns scale = max |v| / 127 of the fp32 sums, code =
// the nearest whole number. A wavefront holds 64 columns of g and of u (or 128 of
// dA), so a block's maximum is two exchanges between lanes and nothing passes
// through LDS. The codes take half the bytes that bf16 values would, written here
// and read there.
//
// Gate/up has a second form, the 256 x 256 tiles of gemm_bf16.hip with one
// workgroup per CU (launch_gate_up_ckpt8 says when).
#include "duo.h"
#include "i8.h"

namespace moe {
namespace {

using duo::f32x4;
using duo::kOutside;
using duo::make_rsrc;
using duo::rsrc_t;
using duo::u32x2;
using duo::u32x4;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct CkptParams : duo::Base {
  const float* row_weight;
  int8_t *gq, *uq;
  float *gs, *us;
  bf16_t *a_out, *dgu;
  float* dot;
};

__device__ __forceinline__ float sigmoid(float g) {  // hardware exponential and reciprocal, about 1 ulp each
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

struct Bf16Product {
  typedef f32x4 Acc;
  static __device__ __forceinline__ Acc product(const u32x4& w, const u32x4& a, const Acc& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                   0);
  }
};

template <bool ROWS>  // rows of a through row_token
struct GateUpOp : Bf16Product {
  typedef CkptParams Params;
  typedef const __attribute__((address_space(4))) Params* args_t;
  static constexpr bool PAIRED = true, GATHER = ROWS, KROWS = false;
  static constexpr int EXTRA = 4;

  static __device__ __forceinline__ void begin(args_t, const duo::Tile&, const int*, char*, int, int) {}

  // The 16 values of one row's block that this lane holds, as codes.
  static __device__ __forceinline__ void block(const f32x4* v, u32x2 (&codes)[2], float& scale) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) m = __builtin_elementwise_maximum(m, fabsf(v[j][x]));
    const SumFactor f(duo::across_groups_max(m));
    scale = f.scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) c[x] = f.code(v[2 * h + x / 4][x % 4]);
      codes[h] = u32x2{bytes4(c[0], c[1], c[2], c[3]), bytes4(c[4], c[5], c[6], c[7])};
    }
  }

  template <int NI>
  static __device__ __forceinline__ void finish(args_t A, Acc (&acc)[duo::FM][duo::FN], const duo::Tile& t, char*,
                                                const duo::Where& w) {
    const int N = A->N, nblk = N / kCkptBlock, blk = t.n0 / kCkptBlock + w.wn;
    const int64_t base = static_cast<int64_t>(t.row0) * N, sbase = static_cast<int64_t>(t.row0) * nblk;
    const int64_t bytes = static_cast<int64_t>(t.valid) * N, sbytes = static_cast<int64_t>(t.valid) * nblk * 4;
    const rsrc_t rg = make_rsrc(A->gq + base, bytes), ru = make_rsrc(A->uq + base, bytes);
    const rsrc_t rgs = make_rsrc(A->gs + sbase, sbytes), rus = make_rsrc(A->us + sbase, sbytes);
    const rsrc_t ra = make_rsrc(A->a_out + base, 2 * bytes);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = w.row(i);
      const bool there = r < t.valid && blk < nblk;
      u32x2 gc[2], uc[2];
      u32x4 av[2];
      float sg, su;
      block(&acc[i][0], gc, sg);
      block(&acc[i][4], uc, su);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float a[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float g = acc[i][2 * h + x / 4][x % 4];
          a[x] = g * sigmoid(g) * acc[i][4 + 2 * h + x / 4][x % 4];
        }
        av[h] = pack8(a);
      }
      if (i == 0) duo::loads_landed();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t to = there ? static_cast<uint32_t>(r) * N + blk * kCkptBlock + 32 * h + 8 * w.g : kOutside;
        __builtin_amdgcn_raw_buffer_store_b64(gc[h], rg, to, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(uc[h], ru, to, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(av[h], ra, there ? 2 * to : kOutside, 0, 0);
      }
      const uint32_t to = there && w.g == 0 ? (static_cast<uint32_t>(r) * nblk + blk) * 4 : kOutside;
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sg), rgs, to, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(su), rus, to, 0, 0);
    }
  }
};

struct DownGradOp : Bf16Product {
  typedef CkptParams Params;
  typedef const __attribute__((address_space(4))) Params* args_t;
  static constexpr bool PAIRED = false, GATHER = true, KROWS = true;
  static constexpr int EXTRA = 4 * duo::BM;  // the rows' weights

  static __device__ __forceinline__ void begin(args_t A, const duo::Tile& t, const int*, char* extra, int wave, int lane) {
    if (wave < duo::BM / kWave)
      duo::words_to_lds(make_rsrc(A->row_weight + t.row0, t.valid * 4ll), extra + wave * 256, (wave * 64 + lane) * 4);
  }

  template <int NI>
  static __device__ __forceinline__ void finish(args_t A, Acc (&acc)[duo::FM][duo::FN], const duo::Tile& t, char* extra,
                                                const duo::Where& w) {
    const int N = A->N, nblk = N / kCkptBlock, ndot = (N + 127) / 128, c0 = t.n0 + w.wn * 128;
    const int64_t base = static_cast<int64_t>(t.row0) * N, sbase = static_cast<int64_t>(t.row0) * nblk;
    const int64_t bytes = static_cast<int64_t>(t.valid) * N, sbytes = static_cast<int64_t>(t.valid) * nblk * 4;
    const rsrc_t rg = make_rsrc(A->gq + base, bytes), ru = make_rsrc(A->uq + base, bytes);
    const rsrc_t rgs = make_rsrc(A->gs + sbase, sbytes), rus = make_rsrc(A->us + sbase, sbytes);
    const rsrc_t ro = make_rsrc(A->dgu + 2 * base, 4 * bytes), ra = make_rsrc(A->a_out + base, 2 * bytes);
    const rsrc_t rd = make_rsrc(A->dot + static_cast<int64_t>(t.row0) * ndot, static_cast<int64_t>(t.valid) * ndot * 4);
    // A lane's sums are four columns each of two tiles 16 apart; after an exchange
    // with the lane 16 on or back they are eight columns of one tile.
    const int col = 16 * (w.g & 1) + 8 * (w.g >> 1);
    struct Kept {
      u32x2 g[4], u[4];
      float gs[2], us[2];
    };
    auto fetch = [&](int i, Kept& k) __attribute__((always_inline)) {
      const int r = w.row(i);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int n = c0 + 32 * h + col;
        const uint32_t from = r < t.valid && n < N ? static_cast<uint32_t>(r) * N + n : kOutside;
        k.g[h] = __builtin_amdgcn_raw_buffer_load_b64(rg, from, 0, 0);
        k.u[h] = __builtin_amdgcn_raw_buffer_load_b64(ru, from, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int blk = c0 / kCkptBlock + b;
        const uint32_t from = r < t.valid && blk < nblk ? (static_cast<uint32_t>(r) * nblk + blk) * 4 : kOutside;
        k.gs[b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rgs, from, 0, 0));
        k.us[b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rus, from, 0, 0));
      }
    };
    Kept kept[2];  // a 16-row tile's are read during the arithmetic of the one before
    fetch(0, kept[0]);
    duo::loads_landed();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i + 1 < NI) fetch(i + 1, kept[(i + 1) & 1]);
      const Kept& k = kept[i & 1];
      const int r = w.row(i);
      const bool row = r < t.valid;
      const float rw = reinterpret_cast<const float*>(extra)[r];
      float sum = 0.0f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int n = c0 + 32 * h + col;
        u32x4 dg, du, aw;
        float d8[8], g8[8], u8[8], a8[8];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][2 * h][x]),
                                                          __float_as_uint(acc[i][2 * h + 1][x]), false, false);
          d8[x] = __uint_as_float(p[0]);
          d8[4 + x] = __uint_as_float(p[1]);
        }
        float part = 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float g = code_value(k.g[h][x / 4], x & 3) * k.gs[h / 2], u = code_value(k.u[h][x / 4], x & 3) * k.us[h / 2];
          const float s = sigmoid(g), silu = g * s, a = silu * u, d = rw * d8[x];
          part = fmaf(d8[x], a, part);
          a8[x] = rw * a;
          g8[x] = d * u * s * (1.0f + g * (1.0f - s));
          u8[x] = d * silu;
        }
        sum += n < N ? part : 0.0f;
        dg = pack8(g8);
        du = pack8(u8);
        aw = pack8(a8);
        const bool there = row && n < N;
        const uint32_t to = (static_cast<uint32_t>(r) * 2 * N + n) * 2;
        __builtin_amdgcn_raw_buffer_store_b128(dg, ro, there ? to : kOutside, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(du, ro, there ? to + 2u * N : kOutside, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(aw, ra, there ? (static_cast<uint32_t>(r) * N + n) * 2 : kOutside, 0, 0);
      }
      sum += __shfl_xor(sum, 16, kWave);
      sum += __shfl_xor(sum, 32, kWave);
      __builtin_amdgcn_raw_buffer_store_b32(
          __float_as_uint(sum), rd,
          row && c0 < N && w.g == 0 ? (static_cast<uint32_t>(r) * ndot + c0 / 128) * 4 : kOutside, 0, 0);
    }
  }
};

template <bool ROWS>
MOE_DUO_KERNEL void gate_up_ckpt8_kernel(const CkptParams P) {
  duo::run<GateUpOp<ROWS>>(P);
}

MOE_DUO_KERNEL void down_dgrad_ckpt8_kernel(const CkptParams P) { duo::run<DownGradOp>(P); }

// d_topk_w of each (token, slot) whose row some expert has: its row's dots in column order.
__global__ __launch_bounds__(256) void ckpt8_dots_kernel(int M, int n, int E, const int32_t* __restrict__ offsets,
                                                         const float* __restrict__ dot,
                                                         const int32_t* __restrict__ sorted_to_flat,
                                                         float* __restrict__ out) {
  const int p = blockIdx.x * 256 + threadIdx.x;
  if (p >= M || p < offsets[0] || p >= offsets[E]) return;
  float v = 0.0f;
  for (int i = 0; i < n; ++i) v += dot[static_cast<int64_t>(p) * n + i];
  out[sorted_to_flat[p]] = v;
}

CkptParams params(const moe_shape& s, const Ckpt8Args& a) {
  CkptParams P{};
  P.M = s.T * s.k;
  P.E = s.E;
  P.N = s.I;
  P.K = 2 * s.H;
  P.arows = s.T;
  P.offsets = a.offsets;
  P.row_token = a.row_token;
  P.a = static_cast<const uint8_t*>(a.in);
  P.w0 = static_cast<const uint8_t*>(a.w0);
  P.w1 = static_cast<const uint8_t*>(a.w1);
  P.row_weight = a.row_weight;
  P.gq = a.gq;
  P.gs = a.gs;
  P.uq = a.uq;
  P.us = a.us;
  P.a_out = static_cast<bf16_t*>(a.a_out);
  P.dgu = static_cast<bf16_t*>(a.dgu);
  P.dot = a.dot;
  return P;
}

}  // namespace

// From 256 rows per expert on 256-row tiles read the weights half as often and need
// less LDS per product; below them they stand half empty. Gate/up of 128 experts,
// 2048 x 768, top-8, us (256-row tiles | 128-row), the same rows for each: 512 tokens
// 164 | 158, 2048 tokens 217 | 198, 4096 tokens 248 | 269, 8192 tokens 450 | 470; 8
// experts, 8192 rows each 391 | 413. With rows spread as a random choice spreads
// them, 128 on average pass 128 as often as not: 2048 tokens 232 | 249, 1024 tokens
// 191 | 183. The data gradient has more to do in its epilogue, and the 128-row tiles'
// runs under the other workgroup's products: 97 | 96, 145 | 139, 203 | 176,
// 291 | 308 (343 | 337 where experts have 512 rows on average, not each), 249 | 269.
hipError_t launch_gate_up_ckpt8(const moe_shape& s, const Ckpt8Args& a, hipStream_t st) {
  if (static_cast<int64_t>(s.T) * s.k >= 256ll * s.E) {
    GemmArgs g{};
    g.offsets = a.offsets;
    g.a = a.in;
    g.row_token = a.row_token;
    g.b0 = a.w0;
    g.b1 = a.w1;
    g.out2 = a.a_out;
    g.gq = a.gq;
    g.gs = a.gs;
    g.uq = a.uq;
    g.us = a.us;
    return launch_gemm_bf16(GEMM_GATEUP, s, g, st);
  }
  const CkptParams P = params(s, a);
  if (a.row_token) gate_up_ckpt8_kernel<true><<<2 * gemm_grid(), duo::kThreads, 0, st>>>(P);
  else gate_up_ckpt8_kernel<false><<<2 * gemm_grid(), duo::kThreads, 0, st>>>(P);
  return hipGetLastError();
}

hipError_t launch_down_dgrad_ckpt8(const moe_shape& s, const Ckpt8Args& a, hipStream_t st) {
  down_dgrad_ckpt8_kernel<<<2 * gemm_grid(), duo::kThreads, 0, st>>>(params(s, a));
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int M = s.T * s.k;
  ckpt8_dots_kernel<<<static_cast<unsigned>(ceil_div64(M, 256)), 256, 0, st>>>(
      M, ceil_div(s.I, 128), s.E, a.offsets, a.dot, a.sorted_to_flat, a.d_topk_w);
  return hipGetLastError();
}

}  // namespace moe
