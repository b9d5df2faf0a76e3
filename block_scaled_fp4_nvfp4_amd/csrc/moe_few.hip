// A whole routed-expert layer for a few tokens (at most 16), from the router's
// logits to y, behind moe_fp4_forward_few (gfx950):
//
//   l' = fp32(logit + bias), the k largest l' (ties: lower id), w = softmax over them
//   h_tj = Qh(SiLU(G_e x~_t) * (U_e x~_t)),  e = ids[t][j],  x~ = Qx(x)
//   y_t  = sum_j w_tj D_e h_tj  (+ sigmoid(x_t . g) * shared(x_t))
//
// Two kernels: routing, quantization of x and the gate_up products (every
// workgroup routes the tokens by itself); then the down products with the
// routing-weighted sum over experts kept in registers, so that neither a
// permutation nor per-pair down outputs exist.  Where h is quantized a small
// kernel between the two does it.
//
// What bounds it: the touched experts' weights, read once (2.76 MB an expert
// at hidden 2560, intermediate 640 in NVFP4).  All tokens of the call are the
// 16 columns of one 16x16x32 bf16 MFMA tile, so an expert's weights are
// decoded once whatever the number of its tokens, and no gather is needed:
// gate_up computes every column and keeps those of the expert's tokens, down
// reads zeros for the others.
//
// Everything the products read is exact in bf16: bf16 x, E4M3 values times
// powers of two (MXFP8), E4M3 codes alone (FP8 rows; their scales multiply the
// f32 sum of each 128-block), E2M1 codes times E4M3 block scales (6
// significant bits), E2M1 codes times powers of two.  An unquantized h (f32)
// is split into three bf16 terms whose sum is h (3 x 8 significant bits).
// Sums are f32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"
#include "moe_internal.h"

namespace fp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kFewTokens = 16;   // columns of the MFMA tile
constexpr int kGuWaves = 8;      // waves per workgroup of the gate_up kernel
constexpr int kGuAhead = 5;      // K steps loaded together
constexpr int kDnWaves = 16;     // waves per workgroup of the down kernel
constexpr int kDnAhead = 5;

// format pairs of the layer
enum FewMode { FM_NV = 0, FM_MX = 1, FM_NVNV = 2, FM_MXMX = 3, FM_FP8 = 4 };
constexpr int weight_fmt(int mode) {
  return mode == FM_NV || mode == FM_NVNV ? FP4_FMT_NVFP4 : mode == FM_FP8 ? FP4_FMT_FP8_BLOCK : FP4_FMT_MXFP4;
}
constexpr int act_fmt(int mode) {
  return mode == FM_NVNV ? FP4_FMT_NVFP4 : mode == FM_MXMX ? FP4_FMT_MXFP8 : mode == FM_FP8 ? FP4_FMT_FP8_ROW : FP4_FMT_NONE;
}

struct FewArgs {
  const uint16_t* x;       // bf16 [T, H]
  const float *logits, *bias;
  const uint8_t *w13, *w2;
  const void *w13s, *w2s;
  const float *w13s2, *w2s2;
  const float *x_scale, *h_scale;  // static NVFP4 activation tensor scales, or null
  const uint8_t *ws13, *ws13s, *ws2, *ws2s;
  const uint16_t* gate;
  int T, E, k, H, I, S;    // S: shared width, 0 without a shared expert
  int routed_wgs;          // gate_up workgroups of the routed experts; the rest take the shared expert
  int k_split;             // waves that share one unit of the routed gate_up
  // workspace
  int32_t *ids, *list, *slot;  // [T k], [1 + min(E, T k)] (count first), [.., 16] pair of (listed expert, token) or -1
  float *wts, *sgate, *amax_part, *h_ts;
  float* h;                // f32 [T k, I] (quantized modes)
  uint16_t* hb;            // bf16 [T k, I] quantized values, or [T k, 3, I] terms
  float* hf;               // FP8 rows: scales [T k, I / 128]
  float* sh;               // f32 [T, S]
  uint16_t* shb;           // bf16 [T, S]
  // outputs
  int32_t* ids_out;
  float* wts_out;
  void* y;
};

// ------------------------------------------------------------------ decoding

// Packs the bf16 values of two floats whose low 16 bits are zero.
__device__ __forceinline__ uint32_t pack_exact_bf16(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float ue8m0_f32(uint32_t c) {
  return c ? __uint_as_float(c << 23) : 5.877471754111438e-39f;  // 2^-127
}

// A lane's share of a weight row's 128-wide K step: 32 consecutive values
// (chunk g of lane group g) and their block scales.
template <int FMT>
struct WStep {
  u32x4 c[FMT == FP4_FMT_NVFP4 || FMT == FP4_FMT_MXFP4 ? 1 : 2];
  uint32_t s;
};

template <int FMT>
__device__ __forceinline__ void load_wstep(WStep<FMT>& v, const uint8_t* row, const uint8_t* srow, int kb, int g, int K) {
  const int k0 = 128 * kb + 32 * g;
  const int kk = k0 < K ? k0 : 0;  // past the row's end: its start, multiplied by zeros
  if constexpr (FMT == FP4_FMT_NVFP4) {
    v.c[0] = ld16(row + kk / 2);
    v.s = *reinterpret_cast<const uint16_t*>(srow + kk / 16);
  } else if constexpr (FMT == FP4_FMT_MXFP4) {
    v.c[0] = ld16(row + kk / 2);
    v.s = srow[kk / 32];
  } else {
    v.c[0] = ld16(row + kk);
    v.c[1] = ld16(row + kk + 16);
    v.s = FMT == FP4_FMT_MXFP8 ? srow[kk / 32] : 0;
  }
}

// Values 8j .. 8j+7 of the lane's 32 as bf16 (exact).
template <int FMT>
__device__ __forceinline__ bf16x8_t wstep_frag(const WStep<FMT>& v, int j) {
  u32x4 p;
  if constexpr (FMT == FP4_FMT_NVFP4) {
    const uint32_t d = v.c[0][j];
    const float s = j < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)v.s, 0) : __builtin_amdgcn_cvt_f32_fp8((int)v.s, 1);
    float f[8];
    e2m1x8_to_f32x8(d, f);
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] = pack_exact_bf16(f[2 * q] * s, f[2 * q + 1] * s);
  } else if constexpr (FMT == FP4_FMT_MXFP4) {
    const uint32_t d = v.c[0][j];
    const float s = ue8m0_f32(v.s);
    p.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0));
    p.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1));
    p.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2));
    p.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3));
  } else {
    const float s = FMT == FP4_FMT_MXFP8 ? ue8m0_f32(v.s) : 1.0f;
    const int a = (int)v.c[j >> 1][2 * (j & 1)], b = (int)v.c[j >> 1][2 * (j & 1) + 1];
    p.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false));
    p.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true));
    p.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false));
    p.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true));
  }
  return __builtin_bit_cast(bf16x8_t, p);
}

template <int FMT>
__device__ __forceinline__ int64_t code_row_bytes(int64_t K) {
  return FMT == FP4_FMT_NVFP4 || FMT == FP4_FMT_MXFP4 ? K / 2 : K;
}
template <int FMT>
__device__ __forceinline__ int64_t scale_row_bytes(int64_t K) {
  return FMT == FP4_FMT_NVFP4 ? K / 16 : FMT == FP4_FMT_FP8_BLOCK ? 0 : K / 32;
}

// ------------------------------------------------------------ quantization

// The values of 32 consecutive elements v (lane q of the four lanes of a
// 128-block) in activation format FMT, as bf16 in place of v; FP8 rows: the
// codes' values, with the block's scale returned.  ts: the NVFP4 tensor scale
// (its values come without it).
template <int FMT>
__device__ __forceinline__ float quantize32(float (&v)[32], float ts) {
  if constexpr (FMT == FP4_FMT_MXFP8) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
    const int e = mx_exponent(amax, kE4M3Max);
    const float up = ldexpf(1.0f, -e), down = ldexpf(1.0f, e);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float q = __builtin_amdgcn_cvt_f32_fp8((int)e4m3_hw(fminf(fabsf(v[i]) * up, kE4M3Max)), 0);
      v[i] = copysignf(q * down, v[i]);
    }
    return 1.0f;
  } else if constexpr (FMT == FP4_FMT_FP8_ROW) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, __shfl_xor(amax, 1));
    amax = fmaxf(amax, __shfl_xor(amax, 2));
    const float sigma = (float)((double)amax / 448.0);
    const float sg = sigma > 0.0f ? sigma : 1.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float q = __builtin_amdgcn_cvt_f32_fp8((int)e4m3_exact_quotient(fabsf(v[i]), sg), 0);
      v[i] = copysignf(sigma > 0.0f ? q : 0.0f, v[i]);
    }
    return sigma;
  } else if constexpr (FMT == FP4_FMT_NVFP4) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[16 * b + i]));
      const uint32_t sc = ts > 0.0f ? e4m3_rne_sat_f64((double)amax / (6.0 * (double)ts)) : 0u;
      const float s = __builtin_amdgcn_cvt_f32_fp8((int)sc, 0);
      const E2M1Thresholds th = e2m1_thresholds((double)s * (double)ts);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[16 * b + i] = copysignf(e2m1_mag_to_f32(e2m1_code(fabsf(v[16 * b + i]), th)) * s, v[16 * b + i]);
    }
    return 1.0f;
  }
  return 1.0f;
}

__device__ __forceinline__ void load_bf16x32(const uint16_t* p, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 w = ld16(p + 8 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void store_bf16x32(void* p, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_exact_bf16(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
    st16(static_cast<uint16_t*>(p) + 8 * i, w);
  }
}

// ---------------------------------------------------------------- routing

// Order-preserving key of a router value: larger value, larger key; 0 for
// what is never selected (-inf, NaN).
__device__ __forceinline__ uint32_t route_key(float v) {
  v += 0.0f;  // -0 and +0 tie
  const uint32_t u = __float_as_uint(v);
  const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (v > -__builtin_huge_valf()) ? key : 0u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  auto step = [&](auto ctrl) __attribute__((always_inline)) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xf, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>{});  // row_shr 1, 2, 4, 8: lane 15 of each row of 16
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  step(std::integral_constant<int, 0x142>{});  // row_bcast 15, 31: lane 63
  step(std::integral_constant<int, 0x143>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// One wave selects the k experts of one token: ids to LDS in order, and the
// j-th selected value's key in lane j.  PL: experts per lane.
template <int PL>
__device__ __forceinline__ uint32_t select_topk(const float* logits, const float* bias, int E, int k, int* s_ids) {
  const int lane = threadIdx.x & 63;
  uint32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? route_key(logits[e] + (bias ? bias[e] : 0.0f)) : 0u;
  }
  uint32_t mine = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) best = max(best, key[i]);
    const uint32_t top = wave_umax(best);
    int id = -1;
    if (top) {
      // lowest id among the equal: experts lane + 64 i, so the lowest i, then the lowest lane
#pragma unroll
      for (int i = PL - 1; i >= 0; --i) {
        const uint64_t m = __ballot(key[i] == top);
        if (m) id = 64 * i + __builtin_ctzll(m);
      }
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (id == lane + 64 * i) key[i] = 0u;
    }
    if (lane == j) mine = top;
    if (lane == 0) s_ids[j] = id;
  }
  return mine;
}

// ------------------------------------------------------------------ gate_up

struct GuSmem {
  int x, xf, ids, mask, list, red, total;
};
// byte offsets of the gate_up kernel's dynamic LDS
__host__ __device__ inline GuSmem gu_smem(int T, int E, int k, int K) {
  GuSmem s;
  const int kp = (K + 127) / 128 * 128;
  s.x = 0;  // rows padded by 16 bytes: 16 lanes that read one chunk of 16 rows hit different banks
  s.xf = s.x + T * (kp + 8) * 2;
  s.ids = s.xf + T * (kp / 128) * 4;
  s.mask = s.ids + T * k * 4;
  s.list = s.mask + E * 4;
  s.red = (s.list + (T * k + 1) * 4 + 15) / 16 * 16;
  s.total = s.red + kGuWaves * 64 * 8 * 4;
  return s;
}

// Prepares x~ in LDS: [T][kp + 8] bf16, K steps' factors in xf (FP8 rows).
// Returns the factor all products share (the NVFP4 tensor scale of x, or 1).
template <int AF>
__device__ float prepare_x(const FewArgs& a, uint8_t* sx, float* xf, float* tmp) {
  const int H = a.H, kp = (H + 127) / 128 * 128, T = a.T;
  float ts = 1.0f;
  if constexpr (AF == FP4_FMT_NVFP4) {
    if (a.x_scale) {
      ts = a.x_scale[0];
    } else {
      float m = 0.0f;
      for (int c = threadIdx.x; c < T * H / 32; c += 64 * kGuWaves) {
        float v[32];
        load_bf16x32(a.x + 32 * (int64_t)c, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = m;
      __syncthreads();
      m = tmp[0];
#pragma unroll
      for (int w = 1; w < kGuWaves; ++w) m = fmaxf(m, tmp[w]);
      ts = (float)((double)m / kNvTensorDivisor);
    }
  }
  const int per = kp / 32;
  for (int c = threadIdx.x; c < T * per; c += 64 * kGuWaves) {
    const int t = c / per, q = c - t * per;
    float v[32];
    if (32 * q < H) {
      load_bf16x32(a.x + (int64_t)t * H + 32 * q, v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    }
    const float f = quantize32<AF>(v, ts);
    store_bf16x32(sx + (t * (kp + 8) + 32 * q) * 2, v);
    if (AF == FP4_FMT_FP8_ROW && (q & 3) == 0) xf[t * (kp / 128) + (q >> 2)] = f;
  }
  return ts;
}

// 16 gate rows and the 16 up rows of one unit over the K steps [kb0, kb1) for
// all tokens.
template <int FMT>
__device__ __forceinline__ void gu_unit(const uint8_t* wg, const uint8_t* wu, const uint8_t* sg, const uint8_t* su,
                                        const float* fg, const float* fu, const uint8_t* sx, const float* xf, int K, int kb0, int kb1, int xt,
                                        int g, floatx4& accg, floatx4& accu) {
  const int kp = (K + 127) / 128 * 128;
  const uint8_t* xrow = sx + (xt * (kp + 8) + 32 * g) * 2;
  for (int kb = kb0; kb < kb1; kb += kGuAhead) {
    WStep<FMT> vg[kGuAhead], vu[kGuAhead];
#pragma unroll
    for (int u = 0; u < kGuAhead; ++u) {
      const int q = min(kb + u, kb1 - 1);
      load_wstep<FMT>(vg[u], wg, sg, q, g, K);
      load_wstep<FMT>(vu[u], wu, su, q, g, K);
    }
#pragma unroll
    for (int u = 0; u < kGuAhead; ++u) {
      if (kb + u < kb1) {
        floatx4 pg = accg, pu = accu;
        if (FMT == FP4_FMT_FP8_BLOCK) pg = pu = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t xv = __builtin_bit_cast(bf16x8_t, ld16(xrow + (128 * (kb + u) + 8 * j) * 2));
          pg = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(vg[u], j), xv, pg, 0, 0, 0);
          pu = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(vu[u], j), xv, pu, 0, 0, 0);
        }
        if (FMT == FP4_FMT_FP8_BLOCK) {
          const float f = xf[xt * (kp / 128) + kb + u];
          const float a = f * fg[kb + u], b = f * fu[kb + u];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            accg[q] = fmaf(pg[q], a, accg[q]);
            accu[q] = fmaf(pu[q], b, accu[q]);
          }
        } else {
          accg = pg;
          accu = pu;
        }
      }
    }
  }
}

// Sum over the k_split waves of a unit (LDS, one barrier before and one
// after); the first of them holds the result.
__device__ __forceinline__ void gu_reduce(floatx4& a, floatx4& b, float* red, int ks, int split) {
  if (split == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    red[(wave * 8 + q) * 64 + lane] = a[q];
    red[(wave * 8 + 4 + q) * 64 + lane] = b[q];
  }
  __syncthreads();
  if (ks == 0)
    for (int w = 1; w < split; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q] += red[((wave + w) * 8 + q) * 64 + lane];
        b[q] += red[((wave + w) * 8 + 4 + q) * 64 + lane];
      }
}

template <int MODE>
__global__ void __launch_bounds__(64 * kGuWaves, 4) few_gateup_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ float tmp[kGuWaves];
  __shared__ uint32_t s_amax;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, r = lane & 15;
  const int T = a.T, k = a.k, H = a.H, KB = (H + 127) / 128, P = T * k;
  const GuSmem sm = gu_smem(T, a.E, k, H);
  float* xf = reinterpret_cast<float*>(smem + sm.xf);
  float* red = reinterpret_cast<float*>(smem + sm.red);
  const int xt = min(r, T - 1);  // columns past the last token repeat it and are not kept
  const floatx4 zero{0.f, 0.f, 0.f, 0.f};

  if ((int)blockIdx.x >= a.routed_wgs) {  // shared expert
    const int S = a.S, units = S / 16, first = blockIdx.x - a.routed_wgs, step = gridDim.x - a.routed_wgs;
    prepare_x<FP4_FMT_MXFP8>(a, smem + sm.x, xf, tmp);
    if (first == 0) {  // sigmoid(x_t . g) on unquantized x
      for (int t = wave; t < T; t += kGuWaves) {
        float acc = 0.0f;
        for (int c = lane * 8; c < H; c += 512) {
          const u32x4 p = ld16(a.x + (int64_t)t * H + c), q = ld16(a.gate + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc = dot2_bf16(p[i], q[i], acc);
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) acc += __shfl_xor(acc, off);
        if (lane == 0) a.sgate[t] = 1.0f / (1.0f + __expf(-acc));
      }
    }
    __syncthreads();
    const int lo = wave * KB / kGuWaves, hi = (wave + 1) * KB / kGuWaves;
    for (int u = first; u < units; u += step) {
      const int64_t row = 16 * u + r;
      floatx4 ag = zero, au = zero;
      const uint8_t *wg = a.ws13 + row * H, *sg = a.ws13s + row * (H / 32);
      gu_unit<FP4_FMT_MXFP8>(wg, wg + (int64_t)S * H, sg, sg + (int64_t)S * (H / 32), nullptr, nullptr, smem + sm.x, xf, H,
                             lo, hi, xt, g, ag, au);
      gu_reduce(ag, au, red, wave, kGuWaves);
      if (wave == 0 && r < T) {
        floatx4 h;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = silu_f32(ag[q]) * au[q];
        *reinterpret_cast<floatx4*>(a.sh + (int64_t)r * S + 16 * u + 4 * g) = h;
      }
    }
    return;
  }

  int* ids = reinterpret_cast<int*>(smem + sm.ids);
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + sm.mask);
  int* list = reinterpret_cast<int*>(smem + sm.list);
  for (int e = tid; e < a.E; e += 64 * kGuWaves) mask[e] = 0;
  if (tid == 0) s_amax = 0;
  for (int t = wave; t < T; t += kGuWaves) {
    const float* lg = a.logits + (int64_t)t * a.E;
    uint32_t key;
    if (a.E <= 128) key = select_topk<2>(lg, a.bias, a.E, k, ids + t * k);
    else if (a.E <= 256) key = select_topk<4>(lg, a.bias, a.E, k, ids + t * k);
    else if (a.E <= 512) key = select_topk<8>(lg, a.bias, a.E, k, ids + t * k);
    else key = select_topk<16>(lg, a.bias, a.E, k, ids + t * k);
    if (blockIdx.x == 0) {  // softmax over the selected values in f64; slots left over: weight 0
      const uint32_t top = (uint32_t)__builtin_amdgcn_readfirstlane((int)key);
      const double z = key ? exp((double)key_value(key) - (double)key_value(top)) : 0.0;
      double sum = z;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
      sum = __shfl(sum, 0);
      if (lane < k) {
        const float w = key ? (float)(z / sum) : 0.0f;
        a.wts[t * k + lane] = w;
        if (a.wts_out) a.wts_out[t * k + lane] = w;
      }
    }
  }
  const float xs = prepare_x<AF>(a, smem + sm.x, xf, tmp);
  __syncthreads();
  for (int p = tid; p < P; p += 64 * kGuWaves)
    if (ids[p] >= 0) atomicOr(&mask[ids[p]], 1u << (p / k));
  __syncthreads();
  if (wave == 0) {  // the touched experts, by id
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const bool on = e0 + lane < a.E && mask[e0 + lane] != 0;
      const uint64_t m = __ballot(on);
      if (on) list[1 + n + __popcll(m & ((1ull << lane) - 1))] = e0 + lane;
      n += __popcll(m);
    }
    if (lane == 0) list[0] = n;
  }
  __syncthreads();
  const int nd = list[0];
  if (blockIdx.x == 0) {
    for (int p = tid; p < P; p += 64 * kGuWaves) {
      a.ids[p] = ids[p];
      if (a.ids_out) a.ids_out[p] = ids[p];
    }
    for (int i = tid; i <= nd; i += 64 * kGuWaves) a.list[i] = list[i];
    for (int i = tid; i < nd * kFewTokens; i += 64 * kGuWaves) {
      const int e = list[1 + (i >> 4)], t = i & 15;
      int p = -1;
      if (t < T && (mask[e] >> t & 1u))
        for (int j = 0; j < k; ++j)
          if (ids[t * k + j] == e) p = t * k + j;
      a.slot[i] = p;
    }
  }

  const int I = a.I, strips = I / 16, units = nd * strips;
  const int split = a.k_split, per = kGuWaves / split, ks = wave % split;
  const int lo = ks * KB / split, hi = (ks + 1) * KB / split;
  const int64_t rb = code_row_bytes<WF>(H), rs = scale_row_bytes<WF>(H);
  float hmax = 0.0f;
  for (int u0 = blockIdx.x * per; u0 < units; u0 += a.routed_wgs * per) {
    const int u = u0 + wave / split;
    const bool on = u < units;
    const int e = list[1 + (on ? u / strips : 0)], i0 = (on ? u % strips : 0) * 16;
    floatx4 ag = zero, au = zero;
    if (on) {
      const int64_t row = (int64_t)e * 2 * I + i0 + r;
      const uint8_t *wg = a.w13 + row * rb, *sg = static_cast<const uint8_t*>(a.w13s) + row * rs;
      const float *fg = nullptr, *fu = nullptr;
      if (WF == FP4_FMT_FP8_BLOCK) {
        fg = static_cast<const float*>(a.w13s) + ((int64_t)e * (2 * I / 128) + i0 / 128) * KB;
        fu = fg + (int64_t)(I / 128) * KB;
      }
      gu_unit<WF>(wg, wg + I * rb, sg, sg + I * rs, fg, fu, smem + sm.x, xf, H, lo, hi, xt, g, ag, au);
    }
    gu_reduce(ag, au, red, ks, split);
    if (on && ks == 0 && r < T && (mask[e] >> r & 1u)) {
      int p = 0;
      for (int j = 0; j < k; ++j)
        if (ids[r * k + j] == e) p = r * k + j;
      const float s = WF == FP4_FMT_NVFP4 ? a.w13s2[e] * xs : 1.0f;
      floatx4 h;
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = silu_f32(ag[q] * s) * (au[q] * s);
      if constexpr (AF == FP4_FMT_NONE) {
        uint16_t* d = a.hb + (int64_t)p * 3 * I + i0 + 4 * g;
        float rest[4] = {h[0], h[1], h[2], h[3]};
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // truncation, so that a finite rest never rounds up to infinity; what is left is exact
            const uint32_t b = __float_as_uint(rest[q]);
            w[q >> 1] |= (b >> 16) << (16 * (q & 1));
            const bool fin = (b & 0x7F800000u) != 0x7F800000u;
            rest[q] = fin ? rest[q] - __uint_as_float(b & 0xFFFF0000u) : 0.0f;
          }
          *reinterpret_cast<u32x2*>(d + (int64_t)term * I) = u32x2{w[0], w[1]};
        }
      } else {
        *reinterpret_cast<floatx4*>(a.h + (int64_t)p * I + i0 + 4 * g) = h;
#pragma unroll
        for (int q = 0; q < 4; ++q) hmax = fmaxf(hmax, fabsf(h[q]));
      }
    }
  }
  if constexpr (AF == FP4_FMT_NVFP4) {  // the largest |h| of this workgroup (non-negative floats order as integers)
    if (hmax > 0.0f) atomicMax(&s_amax, __float_as_uint(hmax));
    __syncthreads();
    if (tid == 0) a.amax_part[blockIdx.x] = __uint_as_float(s_amax);
  }
}

// ------------------------------------------------------------ h quantization

// Quantizes h of the pairs (format AF, f32 [P, I]) and of the shared expert
// (MXFP8, f32 [T, S]); a lane takes 32 values, the four lanes of a 128-block
// are neighbours.
template <int AF>
__global__ void __launch_bounds__(256) few_hquant_kernel(FewArgs a) {
  const int routed = AF == FP4_FMT_NONE ? 0 : a.T * a.k * (a.I / 32), shared = a.T * (a.S / 32);
  float ts = 1.0f;
  if constexpr (AF == FP4_FMT_NVFP4) {
    if (a.h_scale) {
      ts = a.h_scale[0];
    } else {
      float m = 0.0f;
      for (int i = threadIdx.x & 63; i < a.routed_wgs; i += 64) m = fmaxf(m, a.amax_part[i]);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      ts = (float)((double)m / kNvTensorDivisor);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.h_ts[0] = ts;
  }
  const int c = blockIdx.x * 256 + threadIdx.x;
  float v[32];
  auto load = [&](const float* p) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const floatx4 w = *reinterpret_cast<const floatx4*>(p + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
    }
  };
  if (c < routed) {
    load(a.h + 32 * (int64_t)c);
    const float f = quantize32<AF>(v, ts);
    store_bf16x32(a.hb + 32 * (int64_t)c, v);
    if (AF == FP4_FMT_FP8_ROW && (c & 3) == 0) a.hf[c >> 2] = f;
  } else if (c < routed + shared) {
    load(a.sh + 32 * (int64_t)(c - routed));
    quantize32<FP4_FMT_MXFP8>(v, ts);
    store_bf16x32(a.shb + 32 * (int64_t)(c - routed), v);
  }
}

// --------------------------------------------------------------------- down

// K steps [kb0, kb0 + kDnAhead) of 16 rows of one expert's down matrix times
// the expert's h: acc += f * product (FP8 blocks: f times the block's scales).
// hrow: the lane's pair's h (its first term), or null (a column of zeros).
template <int FMT, int NT>
__device__ __forceinline__ void dn_item(const uint8_t* row, const uint8_t* srow, const float* fw, const uint16_t* hrow, const float* hf,
                                        int K, int kb0, int g, float f, floatx4& acc) {
  const int KB = (K + 127) / 128;
  WStep<FMT> v[kDnAhead];
#pragma unroll
  for (int u = 0; u < kDnAhead; ++u) load_wstep<FMT>(v[u], row, srow, min(kb0 + u, KB - 1), g, K);
  floatx4 p[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) p[t] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < kDnAhead; ++u) {
    if (kb0 + u < KB) {
      const int k0 = 128 * (kb0 + u) + 32 * g;
      u32x4 hv[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) hv[t][j] = u32x4{0, 0, 0, 0};
      if (hrow && k0 < K) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) hv[t][j] = ld16(hrow + (int64_t)t * K + k0 + 8 * j);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8_t w = wstep_frag<FMT>(v[u], j);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8_t, hv[t][j]), p[t], 0, 0, 0);
      }
      if (FMT == FP4_FMT_FP8_BLOCK) {
        const float s = hrow ? hf[kb0 + u] * fw[kb0 + u] * f : 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = fmaf(p[0][q], s, acc[q]);
        p[0] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
  if (FMT != FP4_FMT_FP8_BLOCK) {
#pragma unroll
    for (int t = 1; t < NT; ++t) p[0] += p[t];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = fmaf(p[0][q], f, acc[q]);
  }
}

// 16 outputs of y for all tokens per workgroup; its waves share the touched
// experts (in chunks of kDnAhead K steps) and the shared expert.
template <int MODE, typename OutT>
__global__ void __launch_bounds__(64 * kDnWaves) few_down_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE), NT = AF == FP4_FMT_NONE ? 3 : 1;
  __shared__ float part[kDnWaves][kFewTokens][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, r = lane & 15;
  const int T = a.T, I = a.I, H = a.H, KB = (I + 127) / 128, chunks = (KB + kDnAhead - 1) / kDnAhead;
  const int n0 = blockIdx.x * 16;
  const int nd = a.list[0], items = nd * chunks;
  const int schunks = (a.S / 128 + kDnAhead - 1) / kDnAhead;
  const int64_t rb = code_row_bytes<WF>(I), rs = scale_row_bytes<WF>(I);
  floatx4 acc{0.f, 0.f, 0.f, 0.f};
  for (int it = wave; it < items + schunks; it += kDnWaves) {
    if (it < items) {
      const int ai = it / chunks, kb0 = (it - ai * chunks) * kDnAhead;
      const int e = a.list[1 + ai], p = a.slot[ai * kFewTokens + r];
      float f = p >= 0 ? a.wts[p] : 0.0f;
      if (WF == FP4_FMT_NVFP4) f *= a.w2s2[e];
      if (AF == FP4_FMT_NVFP4) f *= a.h_ts[0];
      const int64_t row = (int64_t)e * H + n0 + r;
      const float* fw = WF == FP4_FMT_FP8_BLOCK ? static_cast<const float*>(a.w2s) + ((int64_t)e * (H / 128) + n0 / 128) * KB : nullptr;
      dn_item<WF, NT>(a.w2 + row * rb, static_cast<const uint8_t*>(a.w2s) + row * rs, fw,
                      p >= 0 ? a.hb + (int64_t)p * NT * I : nullptr, a.hf + (int64_t)max(p, 0) * KB, I, kb0, g, f, acc);
    } else {
      const int S = a.S;
      const int64_t row = n0 + r;
      dn_item<FP4_FMT_MXFP8, 1>(a.ws2 + row * S, a.ws2s + row * (S / 32), nullptr, r < T ? a.shb + (int64_t)r * S : nullptr,
                                nullptr, S, (it - items) * kDnAhead, g, r < T ? a.sgate[r] : 0.0f, acc);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) part[wave][r][4 * g + q] = acc[q];
  __syncthreads();
  if (tid < 256 && (tid >> 4) < T) {
    const int t = tid >> 4, n = tid & 15;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kDnWaves; ++w) s += part[w][t][n];
    OutT* y = static_cast<OutT*>(a.y) + (int64_t)t * H + n0 + n;
    if constexpr (sizeof(OutT) == 4) *y = s;
    else *y = __builtin_bit_cast(uint16_t, (__bf16)s);
  }
}

// --------------------------------------------------------------------- host

struct FewPlan {
  int mode;
  size_t ids, wts, list, slot, sgate, amax_part, h_ts, h, hb, hf, sh, shb, total;
};

constexpr int kFewMaxWgs = 2048;

static int few_plan(const moe_fp4_layer* L, int64_t T, FewPlan* out) {
  FP4_CHECK(validate_layer(L, T));
  if (T > kFewTokens) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: %lld tokens, at most %d", (long long)T, kFewTokens);
  if (L->num_experts > 1024) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: more than 1024 experts");
  if (gu_smem((int)T, L->num_experts, L->top_k, L->hidden).total > 159 * 1024)
    return fail(FP4_ERR_UNSUPPORTED, "few-token forward: %lld tokens of width %d do not fit the LDS", (long long)T, L->hidden);
  const bool nv = L->w_fmt == FP4_FMT_NVFP4;
  FewPlan p{};
  p.mode = L->w_fmt == FP4_FMT_FP8_BLOCK ? FM_FP8 : L->a_fmt == FP4_FMT_NONE ? (nv ? FM_NV : FM_MX) : (nv ? FM_NVNV : FM_MXMX);
  const size_t P = (size_t)T * L->top_k, D = std::min<size_t>(P, L->num_experts), I = L->inter, S = L->shared_inter;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  p.ids = take(4 * P);
  p.wts = take(4 * P);
  p.list = take(4 * (1 + D));
  p.slot = take(4 * D * kFewTokens);
  p.sgate = take(4 * T);
  p.amax_part = take(4 * kFewMaxWgs);
  p.h_ts = take(4);
  p.h = take(L->a_fmt == FP4_FMT_NONE ? 0 : 4 * P * I);
  p.hb = take((L->a_fmt == FP4_FMT_NONE ? 6 : 2) * P * I);
  p.hf = take(L->a_fmt == FP4_FMT_FP8_ROW ? 4 * P * (I / 128) : 0);
  p.sh = take(4 * T * S);
  p.shb = take(2 * T * S);
  p.total = off;
  *out = p;
  return FP4_OK;
}

template <int MODE>
static int launch_few(FewArgs a, int y_dtype, hipStream_t st) {
  constexpr int AF = act_fmt(MODE);
  static std::atomic<uint64_t> lds_raised{0};
  FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_gateup_kernel<MODE>), 159 * 1024, lds_raised));
  const int cus = device_cu_count();
  const GuSmem sm = gu_smem(a.T, a.E, a.k, a.H);
  // workgroups that fit the chip at once, shared between the routed and the shared expert by bytes
  const int fit = cus * std::max(1, std::min(2, (160 * 1024) / (sm.total + 1024)));
  const int strips = a.I / 16;
  const int max_units = std::min(a.E, a.T * a.k) * strips;
  int shared = 0;
  if (a.S > 0) {
    const double sb = 2.0 * a.S, rb = (double)std::min(a.E, a.T * a.k) * 2 * a.I * (MODE == FM_FP8 ? 1.0 : 0.55);
    shared = std::max(1, std::min(a.S / 16, (int)(fit * sb / (sb + rb))));
  }
  // waves per unit: as many as leave every workgroup of the chip a unit
  a.k_split = 1;
  while (a.k_split < kGuWaves && max_units * a.k_split < fit * kGuWaves) a.k_split *= 2;
  const int per = kGuWaves / a.k_split;
  a.routed_wgs = std::max(1, std::min(std::min(fit - shared, kFewMaxWgs), (max_units + per - 1) / per));
  hipLaunchKernelGGL(few_gateup_kernel<MODE>, dim3((unsigned)(a.routed_wgs + shared)), dim3(64 * kGuWaves), (size_t)sm.total, st, a);
  FP4_CHECK(check_launch("few_gateup"));
  const int64_t lanes = (AF == FP4_FMT_NONE ? 0 : (int64_t)a.T * a.k * (a.I / 32)) + (int64_t)a.T * (a.S / 32);
  if (lanes > 0) {
    hipLaunchKernelGGL(few_hquant_kernel<AF>, dim3(grid_1d(lanes, 256)), dim3(256), 0, st, a);
    FP4_CHECK(check_launch("few_hquant"));
  }
  const dim3 grid((unsigned)(a.H / 16)), block(64 * kDnWaves);
  if (y_dtype == FP4_DT_F32) hipLaunchKernelGGL((few_down_kernel<MODE, float>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((few_down_kernel<MODE, uint16_t>), grid, block, 0, st, a);
  return check_launch("few_down");
}

}  // namespace fp4

using namespace fp4;

extern "C" {

int moe_fp4_few_workspace_size(const moe_fp4_layer* layer, int64_t tokens, size_t* bytes) {
  if (!bytes) return fail(FP4_ERR_INVALID_ARG, "null size pointer");
  FewPlan p;
  FP4_CHECK(few_plan(layer, tokens, &p));
  *bytes = p.total;
  return FP4_OK;
}

int moe_fp4_forward_few(const moe_fp4_layer* L, const uint16_t* x, int64_t tokens, const float* logits, const float* bias,
                        void* y, int y_dtype, int32_t* topk_ids, float* topk_weights, void* workspace,
                        size_t workspace_bytes, void* stream) {
  FewPlan p;
  FP4_CHECK(few_plan(L, tokens, &p));
  if (y_dtype != FP4_DT_BF16 && y_dtype != FP4_DT_F32) return fail(FP4_ERR_INVALID_ARG, "unknown y_dtype %d", y_dtype);
  if (tokens == 0) return FP4_OK;
  if (!x || !logits || !y) return fail(FP4_ERR_INVALID_ARG, "null tensor pointer");
  FP4_CHECK(validate_layer_pointers(L));
  // scales are read as pairs of bytes (NVFP4), bytes (MXFP4) or floats (block FP8)
  const uintptr_t sa = L->w_fmt == FP4_FMT_NVFP4 ? 2 : L->w_fmt == FP4_FMT_FP8_BLOCK ? 4 : 1;
  if ((uintptr_t)x % 16 || (uintptr_t)logits % 4 || (uintptr_t)bias % 4 || (uintptr_t)y % (y_dtype == FP4_DT_F32 ? 4 : 2) ||
      (uintptr_t)topk_ids % 4 || (uintptr_t)topk_weights % 4 || (uintptr_t)L->w13 % 16 || (uintptr_t)L->w2 % 16 ||
      (uintptr_t)L->w13_scale % sa || (uintptr_t)L->w2_scale % sa ||
      (L->shared_inter > 0 && ((uintptr_t)L->ws13 % 16 || (uintptr_t)L->ws2 % 16 || (uintptr_t)L->shared_gate % 16)))
    return fail(FP4_ERR_INVALID_ARG, "misaligned tensor pointer");
  if (!workspace || workspace_bytes < p.total)
    return fail(FP4_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, p.total);
  if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "misaligned workspace");
  char* b = static_cast<char*>(workspace);
  FewArgs a{};
  a.x = x; a.logits = logits; a.bias = bias;
  a.w13 = L->w13; a.w2 = L->w2; a.w13s = L->w13_scale; a.w2s = L->w2_scale;
  a.w13s2 = L->w13_scale_2; a.w2s2 = L->w2_scale_2;
  a.x_scale = L->input_scale; a.h_scale = L->inter_scale;
  a.ws13 = L->ws13; a.ws13s = L->ws13_scale; a.ws2 = L->ws2; a.ws2s = L->ws2_scale; a.gate = L->shared_gate;
  a.T = (int)tokens; a.E = L->num_experts; a.k = L->top_k; a.H = L->hidden; a.I = L->inter; a.S = L->shared_inter;
  a.ids = reinterpret_cast<int32_t*>(b + p.ids);
  a.list = reinterpret_cast<int32_t*>(b + p.list);
  a.slot = reinterpret_cast<int32_t*>(b + p.slot);
  a.wts = reinterpret_cast<float*>(b + p.wts);
  a.sgate = reinterpret_cast<float*>(b + p.sgate);
  a.amax_part = reinterpret_cast<float*>(b + p.amax_part);
  a.h_ts = reinterpret_cast<float*>(b + p.h_ts);
  a.h = reinterpret_cast<float*>(b + p.h);
  a.hb = reinterpret_cast<uint16_t*>(b + p.hb);
  a.hf = reinterpret_cast<float*>(b + p.hf);
  a.sh = reinterpret_cast<float*>(b + p.sh);
  a.shb = reinterpret_cast<uint16_t*>(b + p.shb);
  a.ids_out = topk_ids; a.wts_out = topk_weights; a.y = y;
  hipStream_t st = as_stream(stream);
  switch (p.mode) {
    case FM_NV: return launch_few<FM_NV>(a, y_dtype, st);
    case FM_MX: return launch_few<FM_MX>(a, y_dtype, st);
    case FM_NVNV: return launch_few<FM_NVNV>(a, y_dtype, st);
    case FM_MXMX: return launch_few<FM_MXMX>(a, y_dtype, st);
    default: return launch_few<FM_FP8>(a, y_dtype, st);
  }
}

}  // extern "C"
