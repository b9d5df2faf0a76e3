// Dense matrix product in block FP8 (gfx950) behind fp8_block_matmul:
//
//   y[m, n] = sum_kb sx[m, kb] * sw[n / 128, kb] * sum_{k in block kb} cx[m, k] * cw[n, k]
//
// with E4M3 codes cx, cw, one f32 scale sx per (row, 128 columns) of x and one
// f32 scale sw per 128 x 128 tile of W (the block-FP8 pair of the retained
// layers, MXFP4-FP8-R12 card, runtime contract table).  Weights are the A
// operand of the MFMAs (their 16 rows the rows of C), activations the B
// operand, so that a lane's four accumulators are four consecutive outputs
// of one row of y, sx is one value per lane and sw one per wave.
//
// bf16 results sum each 128-block in the E4M3 MFMA: its sum carries about 16
// bits (1.6e-5 relative on normal data, measured), which bf16's rounding of
// the result (2^-8) covers; the blocks' sums are scaled and added in f32.
// f32 results convert the codes to fp16 (exact: E4M3's range and precision
// lie inside fp16's) and take the fp16 MFMA, whose f32 sum measured 7e-8.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"

namespace fp4 {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

struct MatmulArgs {
  const uint8_t* x;        // E4M3 codes [batch, M, K]
  const float* xs;         // [batch, M, K / 128]
  const uint8_t* w;        // E4M3 codes [batch, N, K]
  const float* ws;         // [batch, ceil(N / 128), K / 128]
  void* y;                 // [batch, M, N]
  int64_t M, N;
  int K;
};

// One MFMA fragment: 32 bytes of a row's 128-byte K step, chunks g and 4 + g
// of 16 bytes for lane group g (both operands take the same chunks, so any
// fixed assignment of K to lanes gives the same product).
__device__ __forceinline__ intx8 frag_of(u32x4 lo, u32x4 hi) {
  return intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Eight E4M3 codes (two dwords) as fp16, exactly.
__device__ __forceinline__ half8_t e4m3x8_to_f16(int a, int b) {
  const half2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const half2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const half2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const half2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return half8_t{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// The unscaled product of one 128-block (F32SUM: in fp16 MFMAs).
template <bool F32SUM>
__device__ __forceinline__ floatx4 block_product(const intx8& w, const intx8& x) {
  if constexpr (F32SUM) {
    floatx4 p{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      p = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3x8_to_f16(w[2 * q], w[2 * q + 1]),
                                                 e4m3x8_to_f16(x[2 * q], x[2 * q + 1]), p, 0, 0, 0);
    return p;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
  }
}

template <typename OutT>
__device__ __forceinline__ OutT out_of(float v);
template <>
__device__ __forceinline__ float out_of<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t out_of<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);  // to nearest even, NaN kept
}

// ------------------------------------------------------------ few rows

constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyAhead = 2;  // K steps whose loads are issued together

// 16 outputs x 16 MT rows of y per workgroup; its waves take every
// kSkinnyWaves-th 128-block of K straight from memory into registers and add
// their partial sums up in LDS.
template <int MT, typename OutT>
__global__ void __launch_bounds__(64 * kSkinnyWaves) fp8_skinny_kernel(MatmulArgs a) {
  constexpr bool F32SUM = sizeof(OutT) == 4;
  __shared__ float part[kSkinnyWaves][MT][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  const int64_t b = blockIdx.z, n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16 * MT;
  const int KB = a.K >> 7;
  const int64_t NB = (a.N + 127) >> 7;
  const uint8_t* wrow = a.w + (b * a.N + min(n0 + r, a.N - 1)) * a.K + 16 * g;  // rows past the end: the last one, unused
  const float* wsc = a.ws + (b * NB + (n0 >> 7)) * KB;
  const uint8_t* xrow[MT];
  const float* xsc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = min(m0 + 16 * i + r, a.M - 1);
    xrow[i] = a.x + (b * a.M + m) * a.K + 16 * g;
    xsc[i] = a.xs + (b * a.M + m) * KB;
  }
  floatx4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int kb0 = wave; kb0 < KB; kb0 += kSkinnyWaves * kSkinnyAhead) {
    u32x4 wv[kSkinnyAhead][2], xv[kSkinnyAhead][MT][2];
    float sw[kSkinnyAhead], sx[kSkinnyAhead][MT];
#pragma unroll
    for (int u = 0; u < kSkinnyAhead; ++u) {
      const int kb = min(kb0 + u * kSkinnyWaves, KB - 1);
      wv[u][0] = ld16(wrow + 128 * kb);
      wv[u][1] = ld16(wrow + 128 * kb + 64);
      sw[u] = wsc[kb];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xv[u][i][0] = ld16(xrow[i] + 128 * kb);
        xv[u][i][1] = ld16(xrow[i] + 128 * kb + 64);
        sx[u][i] = xsc[i][kb];
      }
    }
#pragma unroll
    for (int u = 0; u < kSkinnyAhead; ++u) {
      if (kb0 + u * kSkinnyWaves < KB) {
        const intx8 wf = frag_of(wv[u][0], wv[u][1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const floatx4 p = block_product<F32SUM>(wf, frag_of(xv[u][i][0], xv[u][i][1]));
          const float s = sx[u][i] * sw[u];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(p[q], s, acc[i][q]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) part[wave][i][r][4 * g + q] = acc[i][q];
  __syncthreads();
  for (int t = threadIdx.x; t < MT * 256; t += 64 * kSkinnyWaves) {
    const int m = t >> 4, n = t & 15;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kSkinnyWaves; ++w) s += part[w][m >> 4][m & 15][n];
    if (m0 + m < a.M && n0 + n < a.N)
      static_cast<OutT*>(a.y)[(b * a.M + m0 + m) * a.N + n0 + n] = out_of<OutT>(s);
  }
}

template <typename OutT>
static int launch_matmul(const MatmulArgs& a, int64_t batch, hipStream_t st) {
  const int64_t nx = (a.N + 15) / 16;
  const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  const int64_t ny = (a.M + 16 * mt - 1) / (16 * mt);
  if (nx > INT32_MAX || ny > 65535 || batch > 65535)
    return fail(FP4_ERR_UNSUPPORTED, "matmul: too many rows, outputs or matrices");
  const dim3 grid((unsigned)nx, (unsigned)ny, (unsigned)batch), block(64 * kSkinnyWaves);
  if (mt == 1) hipLaunchKernelGGL((fp8_skinny_kernel<1, OutT>), grid, block, 0, st, a);
  else if (mt == 2) hipLaunchKernelGGL((fp8_skinny_kernel<2, OutT>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((fp8_skinny_kernel<4, OutT>), grid, block, 0, st, a);
  return check_launch("fp8_block_matmul");
}

static size_t codes_bytes(int64_t batch, int64_t m, int64_t k) { return ((size_t)(batch * m * k) + 255) / 256 * 256; }

static int validate_matmul(int x_dtype, int64_t batch, int64_t m, int64_t n, int64_t k) {
  if (x_dtype != FP4_DT_BF16 && x_dtype != FP4_DT_F32 && x_dtype != FP4_DT_E4M3)
    return fail(FP4_ERR_INVALID_ARG, "matmul: unknown x_dtype %d", x_dtype);
  if (batch < 0 || m < 0 || n < 0 || k < 0) return fail(FP4_ERR_SHAPE, "matmul: negative dimension");
  if (k % 128) return fail(FP4_ERR_SHAPE, "matmul: k = %lld is not a multiple of 128", (long long)k);
  const int64_t most = (int64_t)1 << 31;
  if (batch >= most || m >= most || n >= most || k >= most)
    return fail(FP4_ERR_UNSUPPORTED, "matmul: a dimension of 2^31 or more");
  const double elems = 0x1p48;  // byte offsets stay far inside 64 bits
  if ((double)batch * m * k > elems || (double)batch * n * k > elems || (double)batch * m * n > elems)
    return fail(FP4_ERR_UNSUPPORTED, "matmul: an operand of more than 2^48 values");
  return FP4_OK;
}

}  // namespace fp4

using namespace fp4;

extern "C" {

int fp8_block_matmul_workspace_size(int x_dtype, int64_t batch, int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return fail(FP4_ERR_INVALID_ARG, "null size pointer");
  FP4_CHECK(validate_matmul(x_dtype, batch, m, n, k));
  *bytes = x_dtype == FP4_DT_E4M3 ? 0 : codes_bytes(batch, m, k) + sizeof(float) * (size_t)(batch * m * (k / 128));
  return FP4_OK;
}

int fp8_block_matmul(const void* x, int x_dtype, const float* x_scales, const uint8_t* w, const float* w_scales,
                     int64_t batch, int64_t m, int64_t n, int64_t k, void* y, int y_dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  size_t need = 0;
  FP4_CHECK(fp8_block_matmul_workspace_size(x_dtype, batch, m, n, k, &need));
  if (y_dtype != FP4_DT_BF16 && y_dtype != FP4_DT_F32) return fail(FP4_ERR_INVALID_ARG, "matmul: unknown y_dtype %d", y_dtype);
  if (batch == 0 || m == 0 || n == 0) return FP4_OK;
  if (k == 0) return fail(FP4_ERR_SHAPE, "matmul: k is 0");
  if (!x || !w || !w_scales || !y || (x_dtype == FP4_DT_E4M3 && !x_scales))
    return fail(FP4_ERR_INVALID_ARG, "matmul: null pointer");
  if ((uintptr_t)x % 16 || (uintptr_t)w % 16 || (uintptr_t)y % (y_dtype == FP4_DT_BF16 ? 2 : 4) ||
      (uintptr_t)x_scales % 4 || (uintptr_t)w_scales % 4)
    return fail(FP4_ERR_INVALID_ARG, "matmul: misaligned pointer");
  hipStream_t st = as_stream(stream);
  MatmulArgs a{static_cast<const uint8_t*>(x), x_scales, w, w_scales, y, m, n, (int)k};
  if (x_dtype != FP4_DT_E4M3) {
    if (!workspace || workspace_bytes < need)
      return fail(FP4_ERR_WORKSPACE, "matmul: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "matmul: misaligned workspace");
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(codes + codes_bytes(batch, m, k));
    FP4_CHECK(fp4_quantize(FP4_FMT_FP8_ROW, 0, 0, x, x_dtype, 1, batch * m, k, codes, scales, nullptr, nullptr, stream));
    a.x = codes;
    a.xs = scales;
  }
  return y_dtype == FP4_DT_BF16 ? launch_matmul<uint16_t>(a, batch, st) : launch_matmul<float>(a, batch, st);
}

}  // extern "C"
