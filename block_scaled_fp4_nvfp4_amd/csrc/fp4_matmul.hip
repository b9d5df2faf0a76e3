// Dense matrix product with 4-bit weights (gfx950) behind fp4_matmul, and its
// gradient with respect to x behind fp4_matmul_grad:
//
//   y[m, n]  = S sum_k x[m, k]  g[n, k] s[n, k / B]
//   dx[m, k] = S sum_n dy[m, n] g[n, k] s[n, k / B]
//
// g the E2M1 values, s the block scales (NVFP4: E4M3, B = 16; MXFP4: a power of
// two, B = 32) and S the NVFP4 tensor scale.  Every g s is a bf16 value (E2M1 has
// two significant bits, E4M3 four), so weights are decoded to bf16 exactly and the
// products go through the bf16 MFMA, whose sums are f32.  S's power of two goes
// into the decoded weights, so that sums are of the size of the result, and its
// mantissa into the sum at the end.  bf16 x is taken as it is; f32 x is split into
// three bf16 terms, 8 of its 24 bits each: exactly, from 2^-109 on (bf16's smallest
// step is 2^-133).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"

namespace fp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kBK = 64;  // the sum's steps: 64 products at a time

struct Fp4MatmulArgs {
  const uint16_t* x;   // bf16 [terms][batch][M][ld], zeros from the sum's length to a multiple of 64
  const uint8_t* w;    // [batch][N][K / 2]
  const uint8_t* ws;   // [batch][N][K / 16] or [K / 32]
  const float* ts;     // [batch] (NVFP4)
  void* y;             // [batch][M][O]
  int64_t ld, term;    // x's row and term strides
  int64_t M, N, K, O;  // O: outputs (N, or K for the gradient)
  int steps, terms, y_f32;
};

// ------------------------------------------------------------ operands

// x [rows][len] (bf16 or f32, any alignment) as bf16 rows of `ld` values, zeros at
// their ends; f32 as three such arrays whose sum it is: each takes the next eight
// bits of what the ones before left (cut, not rounded: the largest f32 would round to infinity).
template <typename T>
__global__ void __launch_bounds__(256) fp4_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t len, int64_t ld, uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = ld / 8;
  if (i >= rows * per) return;
  const int64_t row = i / per, c = (i - row * per) * 8;
  constexpr int TERMS = sizeof(T) == 4 ? 3 : 1;
  uint32_t d[TERMS][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int t = 0; t < TERMS; ++t) d[t][j] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (c + j >= len) continue;
    if constexpr (TERMS == 1) {
      d[0][j >> 1] |= (uint32_t)x[row * len + c + j] << (16 * (j & 1));
    } else {
      float v = x[row * len + c + j];
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        const uint32_t top = __float_as_uint(v) & 0xFFFF0000u;
        d[t][j >> 1] |= (j & 1) ? top : top >> 16;
        v = __builtin_amdgcn_classf(v, 0x207) ? 0.0f : v - __uint_as_float(top);  // infinities and NaN leave nothing
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TERMS; ++t) st16(out + t * rows * ld + row * ld + c, u32x4{d[t][0], d[t][1], d[t][2], d[t][3]});
}

// 16 codes of a row (two dwords) and their block's scale byte to 16 bf16 values.
// `pow2`: the power of two of the tensor scale (NVFP4).
template <int FMT>
__device__ __forceinline__ void decode16(uint32_t a, uint32_t b, uint32_t scale, float pow2, uint32_t (&out)[8]) {
  if constexpr (FMT == FP4_FMT_MXFP4) {
    const float s = __uint_as_float(scale << 23);  // the conversion reads the exponent byte: 0 is 2^-127, 255 NaN
#define FP4_CVT(d, i) __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, i))
    out[0] = FP4_CVT(a, 0); out[1] = FP4_CVT(a, 1); out[2] = FP4_CVT(a, 2); out[3] = FP4_CVT(a, 3);
    out[4] = FP4_CVT(b, 0); out[5] = FP4_CVT(b, 1); out[6] = FP4_CVT(b, 2); out[7] = FP4_CVT(b, 3);
#undef FP4_CVT
  } else {
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)scale, 0) * pow2;
    float v[16];
    e2m1x8_to_f32x8(a, *reinterpret_cast<float(*)[8]>(v));
    e2m1x8_to_f32x8(b, *reinterpret_cast<float(*)[8]>(v + 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x2_t p{(__bf16)(v[2 * i] * s), (__bf16)(v[2 * i + 1] * s)};  // exact
      out[i] = __builtin_bit_cast(uint32_t, p);
    }
  }
}

// A tensor scale S as pow2 mant: the power of two goes into the weights (which stay
// bf16's normal numbers), the rest is applied to the sums.  S = 0 makes weights of 0,
// so that no sum of large x is infinite before it is multiplied by 0.
__device__ __forceinline__ void split_scale(float S, float& pow2, float& mant) {
  const int e = min(100, max(-100, __builtin_amdgcn_frexp_expf(S)));
  pow2 = S == 0.0f ? 0.0f : ldexpf(1.0f, e);
  mant = ldexpf(S, -e);
}

__device__ __forceinline__ bf16x8_t as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8_t, v); }

// ------------------------------------------------------------ tiles

// Tile of BM rows by BO outputs per workgroup of WM x WN waves, each owning 16 MS
// rows and 16 NS outputs.  Steps of 64 products: x's part comes by DMA, the
// weights' codes through registers, decoded on their way to LDS, both into the
// half of the LDS that the step before last used.  Weights are the A operand of
// the MFMA, so that a lane's four sums are four consecutive outputs of one row.
// The gradient sums over W's rows: its tile lies in LDS as W does and is turned by
// the transposing reads.
template <int WM, int WN, int MS, int NS, bool GRAD>
struct Fp4Tile {
  static constexpr int WAVES = WM * WN, TH = 64 * WAVES, BM = 16 * MS * WM, BO = 16 * NS * WN;
  static constexpr int XB = BM * 128;                              // bytes of x a step
  static constexpr int WROW = GRAD ? BO * 2 + 32 : 128;            // bytes of a row of the weight tile
  static constexpr int WB = GRAD ? 64 * WROW : BO * 128;
  static constexpr int CPT = BO * 4 / TH;                          // blocks of 16 codes a thread decodes a step
  static constexpr int XD = BM / 8 / WAVES;                        // DMA instructions of a wave a step
  static constexpr int LDS = 2 * (XB + WB);
  static_assert(CPT >= 1 && (BO * 4) % TH == 0 && (BM / 8) % WAVES == 0, "whole chunks");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <int FMT, bool GRAD, int WM, int WN, int MS, int NS>
__global__ void __launch_bounds__(64 * WM * WN, 2) fp4_tile_kernel(Fp4MatmulArgs a, int mt, int ot) {
  using C = Fp4Tile<WM, WN, MS, NS, GRAD>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, r = lane & 15;
  const int wm = wave / WN, wn = wave % WN;
  // workgroups b, b + 8, ... run on one XCD: give it consecutive tiles
  const int tiles = mt * ot, per = (tiles + 7) / 8;
  const int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (t >= tiles) return;
  const int grp = t / (8 * ot), in = t - grp * 8 * ot, rows = min(8, mt - grp * 8);
  const int64_t m0 = (int64_t)(grp * 8 + in % rows) * C::BM, o0 = (int64_t)(in / rows) * C::BO, b = blockIdx.z;
  const int64_t wrow = a.K / 2, srow = a.K / (FMT == FP4_FMT_NVFP4 ? 16 : 32);
  const uint8_t* w = a.w + b * a.N * wrow;
  const uint8_t* ws = a.ws + b * a.N * srow;
  float pow2 = 1.0f, mant = 1.0f;
  if constexpr (FMT == FP4_FMT_NVFP4) split_scale(a.ts[b], pow2, mant);

  // x rows past the end repeat the last one; their results are not stored
  const int mlast = (int)min((int64_t)C::BM - 1, a.M - 1 - m0);
  const int nsteps = a.steps * a.terms;
  uint32_t xoff[C::XD];
#pragma unroll
  for (int j = 0; j < C::XD; ++j) {
    const int row = wave * 8 * C::XD + 8 * j + (lane >> 3);
    xoff[j] = (uint32_t)min(row, mlast) * (uint32_t)(a.ld * 2) + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const uint16_t* xbase = a.x + (b * a.M + m0) * a.ld;
  auto load_x = [&](int step, int term, int half) __attribute__((always_inline)) {
    const auto buf = buffer_of(xbase + term * a.term, (uint32_t)(mlast + 1) * (uint32_t)(a.ld * 2));
#pragma unroll
    for (int j = 0; j < C::XD; ++j) dma_buffer(buf, xoff[j], 128 * step, lds + half * C::XB + (wave * C::XD + j) * 1024);
  };
  // this thread's blocks of 16 codes: consecutive ones of one row of the weight tile
  constexpr int PER_ROW = GRAD ? C::BO / 16 : 4;
  const int trow = tid * C::CPT / PER_ROW, tblk = tid * C::CPT % PER_ROW;
  uint32_t code[C::CPT][2], scale[C::CPT];
  auto load_w = [&](int step) __attribute__((always_inline)) {
    const int64_t n = GRAD ? (int64_t)step * kBK + trow : o0 + trow;
    const bool inside = n < a.N;
    const int64_t nn = min(n, a.N - 1);
#pragma unroll
    for (int c = 0; c < C::CPT; ++c) {
      const int64_t blk = (GRAD ? o0 / 16 : (int64_t)step * 4) + tblk + c;
      const bool ok = inside && blk * 16 < a.K;
      const int64_t bb = ok ? blk : 0;
      const u32x2 v = *reinterpret_cast<const u32x2*>(w + nn * wrow + bb * 8);
      const uint32_t s = ws[nn * srow + (FMT == FP4_FMT_NVFP4 ? bb : bb >> 1)];
      // what is past the end counts 0 (an infinity or NaN there would reach sums whose x is 0)
      code[c][0] = ok ? v.x : 0;
      code[c][1] = ok ? v.y : 0;
      scale[c] = ok ? s : 0;
    }
  };
  uint8_t* wlds = lds + 2 * C::XB;
  auto decode_w = [&](int half) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C::CPT; ++c) {
      uint32_t v[8];
      decode16<FMT>(code[c][0], code[c][1], scale[c], pow2, v);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int piece = 2 * (tblk + c) + h;
        uint8_t* to = wlds + half * C::WB + trow * C::WROW + 16 * (GRAD ? piece : piece ^ ((trow >> 1) & 7));
        st16(to, u32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]});
      }
    }
  };
  auto read_w = [&](int half, int s, int j) __attribute__((always_inline)) {
    const uint8_t* from = wlds + half * C::WB;
    if constexpr (GRAD) {
      // lane (g, r) names 4 values of row 32 j + 8 g + r / 4 and gets column r of the rows 32 j + 8 g .. + 3 (then + 4 .. + 7)
      const uint8_t* p = from + (32 * j + 8 * g + (r >> 2)) * C::WROW + (wn * 16 * NS + 16 * s + 4 * (r & 3)) * 2;
      typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * C::WROW));
      const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
      return as_bf16x8(u32x4{l.x, l.y, h.x, h.y});
    } else {
      const int row = wn * 16 * NS + 16 * s + r;
      return as_bf16x8(ld16(from + row * 128 + 16 * ((4 * j + g) ^ ((row >> 1) & 7))));
    }
  };
  floatx4 acc[MS][NS];
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[i][s] = floatx4{0.f, 0.f, 0.f, 0.f};
  load_x(0, 0, 0);
  load_w(0);
  decode_w(0);
  load_w(min(1, a.steps - 1));
  int step = 0, term = 0;
  for (int i = 0; i < nsteps; ++i) {
    __builtin_amdgcn_s_waitcnt(0);  // this step's x has arrived and its weights are written
    __syncthreads();
    const int next_term = term + 1 == a.terms ? 0 : term + 1, next_step = next_term ? step : step + 1;
    if (i + 1 < nsteps) load_x(next_step, next_term, (i + 1) & 1);
    if (term == 0) {
      decode_w((step + 1) & 1);
      load_w(min(step + 2, a.steps - 1));
    }
    const uint8_t* xr = lds + (i & 1) * C::XB;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bf16x8_t wf[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) wf[s] = read_w(step & 1, s, j);
#pragma unroll
      for (int q = 0; q < MS; ++q) {
        const int row = wm * 16 * MS + 16 * q + r;
        const bf16x8_t xf = as_bf16x8(ld16(xr + row * 128 + 16 * ((4 * j + g) ^ ((row >> 1) & 7))));
#pragma unroll
        for (int s = 0; s < NS; ++s) acc[q][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[s], xf, acc[q][s], 0, 0, 0);
      }
    }
    term = next_term;
    step = next_step;
  }
#pragma unroll
  for (int q = 0; q < MS; ++q) {
    const int64_t m = m0 + wm * 16 * MS + 16 * q + r;
    if (m >= a.M) continue;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t o = o0 + wn * 16 * NS + 16 * s + 4 * g + c;
        if (o >= a.O) continue;
        const float v = acc[q][s][c] * mant;
        const int64_t at = (b * a.M + m) * a.O + o;
        if (a.y_f32) static_cast<float*>(a.y)[at] = v;
        else static_cast<uint16_t*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
      }
  }
}

constexpr int64_t kMost = 0xFFFFFFFF;  // threads of a launch along x
constexpr int64_t kMostMatrices = 65535;

template <int FMT, bool GRAD>
static int launch_fp4(const Fp4MatmulArgs& a, int64_t batch, hipStream_t st) {
  using C = Fp4Tile<2, 2, 2, 2, GRAD>;
  const int64_t mt = (a.M + C::BM - 1) / C::BM, ot = (a.O + C::BO - 1) / C::BO, grid = (mt * ot + 7) / 8 * 8;
  if (grid * C::TH > kMost) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: too many rows or outputs");
  hipLaunchKernelGGL((fp4_tile_kernel<FMT, GRAD, 2, 2, 2, 2>), dim3((unsigned)grid, 1, (unsigned)batch), dim3(C::TH), 0, st, a, (int)mt, (int)ot);
  return check_launch("fp4_matmul");
}

// ------------------------------------------------------------ the calls

struct Fp4Plan {
  int64_t sum, out, ld, terms;  // length of the sum, outputs, row stride and terms of x as the kernels read it
  bool rows;                    // x is copied (split, padded) first
  size_t bytes;
};

static int plan_fp4(int w_fmt, int x_dtype, bool grad, int64_t batch, int64_t m, int64_t n, int64_t k, Fp4Plan& p) {
  if (w_fmt < FP4_FMT_NVFP4 || w_fmt > FP4_FMT_NONE) return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: unknown w_fmt %d", w_fmt);
  if (w_fmt != FP4_FMT_NVFP4 && w_fmt != FP4_FMT_MXFP4) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: weights in NVFP4 or MXFP4 only");
  if (x_dtype != FP4_DT_BF16 && x_dtype != FP4_DT_F32) return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: unknown dtype %d", x_dtype);
  if (batch < 0 || m < 0 || n < 0 || k < 0) return fail(FP4_ERR_SHAPE, "fp4_matmul: negative dimension");
  const int block = w_fmt == FP4_FMT_NVFP4 ? 16 : 32;
  if (k % block) return fail(FP4_ERR_SHAPE, "fp4_matmul: k = %lld is not a multiple of %d", (long long)k, block);
  const int64_t most = (int64_t)1 << 31;
  if (batch >= most || m >= most || n >= most || k >= most) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: a dimension of 2^31 or more");
  p.sum = grad ? n : k;
  p.out = grad ? k : n;
  if (p.sum > (int64_t)1 << 22) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: sums of more than 2^22 products");  // 32-bit offsets inside a tile
  if (batch > kMostMatrices) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: more than %lld matrices", (long long)kMostMatrices);
  const double elems = 0x1p46;
  if ((double)batch * m * k > elems || (double)batch * n * k > elems || (double)batch * m * n > elems)
    return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: an operand of more than 2^46 values");
  p.ld = (p.sum + kBK - 1) / kBK * kBK;
  p.terms = x_dtype == FP4_DT_F32 ? 3 : 1;
  p.rows = p.terms > 1 || p.ld != p.sum;
  p.bytes = p.rows ? (size_t)(2 * p.terms) * (size_t)(batch * m * p.ld) : 0;
  if (p.rows && batch * m * (p.ld / 8) > kMost) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: too many rows");
  return FP4_OK;
}

static int run_fp4(int w_fmt, const void* x, int x_dtype, bool grad, const uint8_t* w, const void* w_scales, const float* tensor_scale, int64_t batch,
                   int64_t m, int64_t n, int64_t k, void* y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  Fp4Plan p;
  FP4_CHECK(plan_fp4(w_fmt, x_dtype, grad, batch, m, n, k, p));
  if (y_dtype != FP4_DT_BF16 && y_dtype != FP4_DT_F32) return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: unknown dtype %d of the result", y_dtype);
  if (batch == 0 || m == 0 || p.out == 0) return FP4_OK;
  if (p.sum == 0) return fail(FP4_ERR_SHAPE, "fp4_matmul: sums of no products");
  if (!x || !w || !w_scales || !y || (w_fmt == FP4_FMT_NVFP4 && !tensor_scale)) return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: null pointer");
  if ((uintptr_t)x % (p.rows ? x_dtype == FP4_DT_F32 ? 4 : 2 : 16) || (uintptr_t)w % 8 || (uintptr_t)tensor_scale % 4 ||
      (uintptr_t)y % (y_dtype == FP4_DT_F32 ? 4 : 2))
    return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: misaligned pointer");
  if (p.bytes) {
    if (!workspace || workspace_bytes < p.bytes) return fail(FP4_ERR_WORKSPACE, "fp4_matmul: workspace of %zu bytes, %zu needed", workspace_bytes, p.bytes);
    if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: misaligned workspace");
  }
  hipStream_t st = as_stream(stream);
  if (p.rows) {
    const int64_t rows = batch * m;
    uint16_t* to = static_cast<uint16_t*>(workspace);
    const dim3 grid(grid_1d(rows * (p.ld / 8), 256));
    if (x_dtype == FP4_DT_F32) hipLaunchKernelGGL(fp4_rows_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(x), rows, p.sum, p.ld, to);
    else hipLaunchKernelGGL(fp4_rows_kernel<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(x), rows, p.sum, p.ld, to);
    FP4_CHECK(check_launch("fp4_rows"));
    x = to;
  }
  const Fp4MatmulArgs a{static_cast<const uint16_t*>(x), w, static_cast<const uint8_t*>(w_scales), tensor_scale, y, p.ld, batch * m * p.ld,
                        m, n, k, p.out, (int)(p.ld / kBK), (int)p.terms, y_dtype == FP4_DT_F32};
  if (w_fmt == FP4_FMT_NVFP4) return grad ? launch_fp4<FP4_FMT_NVFP4, true>(a, batch, st) : launch_fp4<FP4_FMT_NVFP4, false>(a, batch, st);
  return grad ? launch_fp4<FP4_FMT_MXFP4, true>(a, batch, st) : launch_fp4<FP4_FMT_MXFP4, false>(a, batch, st);
}

}  // namespace fp4

using namespace fp4;

extern "C" {

int fp4_matmul_workspace_size(int w_fmt, int x_dtype, int64_t batch, int64_t m, int64_t n, int64_t k, size_t* bytes) {
  Fp4Plan p;
  if (!bytes) return fail(FP4_ERR_INVALID_ARG, "null size pointer");
  FP4_CHECK(plan_fp4(w_fmt, x_dtype, false, batch, m, n, k, p));
  *bytes = p.bytes;
  return FP4_OK;
}

int fp4_matmul(int w_fmt, const void* x, int x_dtype, const uint8_t* w, const void* w_scales, const float* tensor_scale, int64_t batch, int64_t m,
               int64_t n, int64_t k, void* y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return run_fp4(w_fmt, x, x_dtype, false, w, w_scales, tensor_scale, batch, m, n, k, y, y_dtype, workspace, workspace_bytes, stream);
}

int fp4_matmul_grad_workspace_size(int w_fmt, int dy_dtype, int64_t batch, int64_t m, int64_t n, int64_t k, size_t* bytes) {
  Fp4Plan p;
  if (!bytes) return fail(FP4_ERR_INVALID_ARG, "null size pointer");
  FP4_CHECK(plan_fp4(w_fmt, dy_dtype, true, batch, m, n, k, p));
  *bytes = p.bytes;
  return FP4_OK;
}

int fp4_matmul_grad(int w_fmt, const void* dy, int dy_dtype, const uint8_t* w, const void* w_scales, const float* tensor_scale, int64_t batch, int64_t m,
                    int64_t n, int64_t k, void* dx, int dx_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return run_fp4(w_fmt, dy, dy_dtype, true, w, w_scales, tensor_scale, batch, m, n, k, dx, dx_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
