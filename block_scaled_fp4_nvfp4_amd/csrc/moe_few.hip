// A whole routed-expert layer for a few tokens (at most 16), from the router's
// logits to y, behind moe_fp4_forward_few (gfx950):
//
//   l' = fp32(logit + bias), the k largest l' (ties: lower id), w = softmax over them
//   h_tj = Qh(SiLU(G_e x~_t) * (U_e x~_t)),  e = ids[t][j],  x~ = Qx(x)
//   y_t  = sum_j w_tj D_e h_tj  (+ sigmoid(x_t . g) * shared(x_t))
//
// Two kernels: routing, quantization of x and the gate_up products (every
// workgroup routes the tokens by itself); then the down products with the
// routing-weighted sum over experts kept on the chip, so that neither a
// permutation nor per-pair down outputs exist.  Where h is quantized a small
// kernel between the two does it.
//
// What bounds it: the touched experts' weights, read once (2.76 MB an expert
// at hidden 2560, intermediate 640 in NVFP4).  They stream through a ring of
// blocks in LDS that belongs to one wave (16 rows x 128 bytes of codes and
// their scales, by DMA, without barriers); loading MFMA fragments straight
// into registers touches four rows in every four lanes and measured twice the
// time.  All tokens of the call are the 16 columns of one 16x16x32 bf16 MFMA
// tile, so gate_up decodes an expert's weights once whatever the number of its
// tokens and gathers nothing: it computes every column and keeps those of the
// expert's tokens.
//
// Everything the products read is exact in bf16: bf16 x, E4M3 values times
// powers of two (MXFP8), E4M3 codes alone (FP8 rows; their scales multiply the
// f32 sum of each 128-block), E2M1 codes times E4M3 block scales (6
// significant bits), E2M1 codes times powers of two.  An h held in f32 (not
// quantized, or FP8 codes times their scales) is split into three bf16 terms
// whose sum is h (3 x 8 significant bits).  Sums are f32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"
#include "moe_internal.h"

namespace fp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kFewTokens = 16;  // columns of the MFMA tile
constexpr int kGuWaves = 8;     // most waves per workgroup of the gate_up kernel
constexpr int kDnWaves = 8;     // most waves per workgroup of the down kernel
constexpr int kDnSeg = 64;      // most experts of one split

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
  int splits, shared_splits;  // down workgroups of a strip: of the routed experts, of the shared expert
  int pass_pairs, seg_steps;  // pairs of an expert and 128-wide K steps that a wave of the down kernel takes at once
  // workspace
  int32_t *list, *pairs;   // touched experts [1 + min(E, T k)] (count first); [.., 16] their pairs, then -1
  int32_t* done;           // [H / 16] arrivals of the down kernel's splits
  float *wts, *sgate, *amax_part, *h_ts;
  float* h;                // f32 [T k, I] (quantized modes)
  uint16_t* hb;            // bf16 [T k, I] quantized values, or [T k, 3, I] terms
  float* sh;               // f32 [T, S]
  uint16_t* shb;           // bf16 [T, S]
  float* ypart;            // f32 [splits + shared_splits, T, H]
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

// Weight rows as the kernels copy them, in pieces of 128 bytes of codes: one
// 128-wide K step of E4M3, two of E2M1.  64-byte pieces with 8 bytes of scales
// (one step) measured 3.1 TB/s where these reach 4.4 TB/s (and 5.7 TB/s
// without any scales): every lane group of a copy that touches another row
// costs a cycle of its compute unit's address path.
template <int FMT>
struct Rows {
  static constexpr bool FP4 = FMT == FP4_FMT_NVFP4 || FMT == FP4_FMT_MXFP4;
  static constexpr int STEP = FP4 ? 64 : 128;  // code bytes of a K step
  static constexpr int STEPS = 128 / STEP;     // K steps of a piece
  static constexpr int SSTEP = FMT == FP4_FMT_NVFP4 ? 8 : FMT == FP4_FMT_FP8_BLOCK ? 0 : 4;  // scale bytes of a step
};

// A lane's 32 values of a K step (its values [32 g, + 32) of one row).
template <int FMT>
struct WStep {
  u32x4 c[Rows<FMT>::FP4 ? 1 : 2];
  uint32_t s;
  // chunk(i): the step's i-th 16-byte chunk of the row; sr: the row's scales of the step
  template <typename Chunk>
  __device__ __forceinline__ void read(Chunk chunk, const uint8_t* sr, int g) {
    if constexpr (Rows<FMT>::FP4) {
      c[0] = ld16(chunk(g));
    } else {
      c[0] = ld16(chunk(2 * g));
      c[1] = ld16(chunk(2 * g + 1));
    }
    if constexpr (FMT == FP4_FMT_NVFP4) s = *reinterpret_cast<const uint16_t*>(sr + 2 * g);
    else if constexpr (Rows<FMT>::SSTEP > 0) s = sr[g];
  }
};

// Values 8j .. 8j+7 of them as bf16 (exact).
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

// NVFP4 as fp16, exact too (6 significant bits between 2^-10 and 2688): half
// the instructions of bf16, whose product with the scale has no packed form.
__device__ __forceinline__ half8_t wstep_frag_f16(const WStep<FP4_FMT_NVFP4>& v, int j) {
  const uint32_t d = v.c[0][j];
  const half2_t both = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)v.s, 1.0f, false);
  const _Float16 s = j < 2 ? both.x : both.y;
  const half2_t sc{s, s};
  const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0) * sc, b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1) * sc;
  const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2) * sc, e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3) * sc;
  return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, e.x, e.y};
}

// acc + 16 rows of weights times 16 columns of x (bf16, or fp16 for NVFP4).
template <int FMT>
__device__ __forceinline__ floatx4 gu_mfma(const WStep<FMT>& w, int j, u32x4 x, floatx4 acc) {
  if constexpr (FMT == FP4_FMT_NVFP4)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(wstep_frag_f16(w, j), __builtin_bit_cast(half8_t, x), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(w, j), __builtin_bit_cast(bf16x8_t, x), acc, 0, 0, 0);
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
    uint32_t d[8];
    e4m3_codes<32>(v, sigma, d);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __builtin_amdgcn_cvt_f32_fp8((int)(d[i >> 2] >> (8 * (i & 3))), 0);
    return sigma;
  } else if constexpr (FMT == FP4_FMT_NVFP4) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[16 * b + i]));
      uint32_t sc = 0xFFu;
      if (ts > 0x1p-100f && ts < 0x1p100f) sc = e4m3_of_quotient(amax, amax / (6.0f * ts), 6.0f, ts);
      if (sc == 0xFFu) sc = ts > 0.0f ? e4m3_rne_sat_f64((double)amax / (6.0 * (double)ts)) : 0u;  // subnormal scales
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

// 32 values as fp16 (exact for those of NVFP4).
__device__ __forceinline__ void store_f16x32(void* p, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    half8_t h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (_Float16)v[8 * i + j];
    st16(static_cast<uint16_t*>(p) + 8 * i, __builtin_bit_cast(u32x4, h));
  }
}

// The three bf16 terms of v (their sum is v): by truncation, so that a finite
// rest never rounds up to infinity, and each rest is exact.  An infinity or
// NaN is its first term.
__device__ __forceinline__ void bf16_terms(float v, uint32_t (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t b = __float_as_uint(v);
    t[i] = b >> 16;
    v = (b & 0x7F800000u) != 0x7F800000u ? v - __uint_as_float(b & 0xFFFF0000u) : 0.0f;
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

// One wave selects the k experts of N tokens (logits and ids `step` tokens
// apart): ids to LDS in order, and the j-th selected value's key of each token
// in lane j.  Lane l holds experts l + 64 i, sorted once by key (stably: the
// lower id first); then each of the k rounds takes the largest of the lanes'
// heads and pops it.  Two tokens at once hide each other's latency.
template <int PL, int N>
__device__ __forceinline__ void select_topk(const float* logits, const float* bias, int E, int k, int step, int* s_ids, uint32_t (&mine)[N]) {
  const int lane = threadIdx.x & 63;
  uint32_t key[N][PL];
  int id[N][PL], my_id[N];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    const float b = bias && e < E ? bias[e] : 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      id[n][i] = e;
      key[n][i] = e < E ? route_key(logits[(int64_t)n * step * E + e] + b) : 0u;
    }
  }
#pragma unroll
  for (int pass = 0; pass < PL; ++pass)
#pragma unroll
    for (int i = pass & 1; i + 1 < PL; i += 2)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const bool swap = key[n][i + 1] > key[n][i];
        const uint32_t ka = key[n][i], kb = key[n][i + 1];
        const int ia = id[n][i], ib = id[n][i + 1];
        key[n][i] = swap ? kb : ka;
        key[n][i + 1] = swap ? ka : kb;
        id[n][i] = swap ? ib : ia;
        id[n][i + 1] = swap ? ia : ib;
      }
#pragma unroll
  for (int n = 0; n < N; ++n) { mine[n] = 0; my_id[n] = -1; }
  for (int j = 0; j < k; ++j) {
    uint32_t top[N];
#pragma unroll
    for (int n = 0; n < N; ++n) top[n] = wave_umax(key[n][0]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint64_t at = __ballot(key[n][0] == top[n]);
      int win = __builtin_ctzll(at), e = __builtin_amdgcn_readlane(id[n][0], win);
      if (top[n] != 0)
        for (at &= at - 1; at; at &= at - 1) {  // equal values: the lowest id
          const int l = __builtin_ctzll(at), o = __builtin_amdgcn_readlane(id[n][0], l);
          if (o < e) { e = o; win = l; }
        }
      if (lane == j) { mine[n] = top[n]; my_id[n] = top[n] ? e : -1; }  // nothing selectable left: -1
      if (lane == win) {
#pragma unroll
        for (int i = 0; i + 1 < PL; ++i) { key[n][i] = key[n][i + 1]; id[n][i] = id[n][i + 1]; }
        key[n][PL - 1] = 0u;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (lane < k) s_ids[n * step * k + lane] = my_id[n];
}

// ------------------------------------------------------------------ gate_up

struct GuSmem {
  int x, xf, ids, list, scale, slot, red, ring, total;
};
// byte offsets of the gate_up kernel's dynamic LDS: x~ (with `factors` one per
// token and K step), the routing's tables, nw waves with `ring` bytes each, their
// partial sums if a unit is split between waves
__host__ __device__ inline GuSmem gu_smem(int T, int E, int k, int K, bool factors, int nw, int ring, bool split) {
  GuSmem s;
  const int kp = (K + 127) / 128 * 128, D = E < T * k ? E : T * k;
  s.x = 0;  // rows padded by 16 bytes: 16 lanes that read one chunk of 16 rows hit different banks
  s.xf = s.x + T * (kp + 8) * 2;
  s.ids = s.xf + (factors ? T * (kp / 128) * 4 : 0);
  s.list = s.ids + T * k * 4;
  s.scale = s.list + D * 4;
  s.slot = s.scale + D * 4;
  s.red = (s.slot + D * kFewTokens + 15) / 16 * 16;
  s.ring = s.red + (split ? nw * 64 * 8 * 4 : 0);
  s.total = s.ring + nw * ring;
  return s;
}

// Prepares x~ in LDS, [T][kp + 8]: bf16, or fp16 for NVFP4 weights (WF). xs[t]
// gets the factor of a token's products, xf those of its K steps (FP8 rows).
// Plain x meets NVFP4 weights as fp16 scaled by the power of two that brings
// the token's largest value to [2^14, 2^15): exact down to 2^-29 of that
// value, and 2^-40 of it off below, far inside the f32 sums' own rounding.
template <int WF, int AF>
__device__ __forceinline__ void prepare_x(const FewArgs& a, uint8_t* sx, float* xf, float* xs, float* tmp) {
  const int H = a.H, kp = (H + 127) / 128 * 128, T = a.T, nw = (int)blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if constexpr (AF == FP4_FMT_NONE) {
    const auto xb = buffer_of(a.x, (uint32_t)(T * H * 2));
    for (int t = nw - 1 - wave; t < T; t += nw) {  // the waves that route fewer tokens first
      uint8_t* row = sx + t * (kp + 8) * 2;
      if constexpr (WF == FP4_FMT_NVFP4) {
        float m = 0.0f;
        for (int c0 = 0; c0 < H / 8; c0 += 8 * 64) {
          u32x4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = ld16(a.x + (int64_t)t * H + 8 * min(c0 + 64 * i + lane, H / 8 - 1));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i][j] << 16)), fabsf(__uint_as_float(w[i][j] & 0xFFFF0000u))));
            if (c0 + 64 * i + lane < H / 8) st16(row + 16 * (c0 + 64 * i + lane), w[i]);
          }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
        const int e = __builtin_amdgcn_frexp_expf(m);
        if (lane == 0) xs[t] = ldexpf(1.0f, e - 15);
        for (int c = lane; c < H / 8; c += 64) {
          const u32x4 w = ld16(row + 16 * c);
          half8_t h;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[2 * j] = (_Float16)ldexpf(__uint_as_float(w[j] << 16), 15 - e);
            h[2 * j + 1] = (_Float16)ldexpf(__uint_as_float(w[j] & 0xFFFF0000u), 15 - e);
          }
          st16(row + 16 * c, __builtin_bit_cast(u32x4, h));
        }
      } else {  // as it is, by DMA; the caller waits for it
        for (int c = 0; c < H / 8; c += 64)
          if (c + lane < H / 8) dma_buffer(xb, (uint32_t)(t * H * 2 + 16 * (c + lane)), 0, row + 16 * c);
        if (lane == 0) xs[t] = 1.0f;
      }
      if (H / 8 + lane < kp / 8) st16(row + 16 * (H / 8 + lane), u32x4{0, 0, 0, 0});
    }
    return;
  }
  float ts = 1.0f;
  if constexpr (AF == FP4_FMT_NVFP4) {
    if (a.x_scale) {
      ts = a.x_scale[0];
    } else {
      float m = 0.0f;
      for (int c = threadIdx.x; c < T * H / 8; c += (int)blockDim.x) {
        const u32x4 w = ld16(a.x + 8 * (int64_t)c);
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      if (lane == 0) tmp[wave] = m;
      __syncthreads();
      m = tmp[0];
#pragma unroll
      for (int w = 1; w < kGuWaves; ++w)
        if (w < nw) m = fmaxf(m, tmp[w]);
      ts = (float)((double)m / kNvTensorDivisor);
    }
  }
  if ((int)threadIdx.x < T) xs[threadIdx.x] = ts;
  const int per = H / 32;  // H is a multiple of 128 where x is quantized
  for (int c = threadIdx.x; c < T * per; c += (int)blockDim.x) {
    const int t = c / per, q = c - t * per;
    float v[32];
    load_bf16x32(a.x + (int64_t)t * H + 32 * q, v);
    const float f = quantize32<AF>(v, ts);
    if constexpr (WF == FP4_FMT_NVFP4) store_f16x32(sx + (t * (kp + 8) + 32 * q) * 2, v);
    else store_bf16x32(sx + (t * (kp + 8) + 32 * q) * 2, v);
    if (AF == FP4_FMT_FP8_ROW && (q & 3) == 0) xf[t * (kp / 128) + (q >> 2)] = f;
  }
}

// Sum over the `split` waves of a unit (in LDS, a barrier before and one
// after); the first of them holds the result.
__device__ __forceinline__ void gu_reduce(floatx4& a, floatx4& b, float* red, int ks, int split) {
  if (split == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto sync = []() __attribute__((always_inline)) {  // LDS only: the blocks on their way stay so
    __builtin_amdgcn_s_waitcnt(lgkmcnt0());
    asm volatile("s_barrier" ::: "memory");
  };
  sync();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    red[(wave * 8 + q) * 64 + lane] = a[q];
    red[(wave * 8 + 4 + q) * 64 + lane] = b[q];
  }
  sync();
  if (ks == 0)
    for (int w = 1; w < split; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q] += red[((wave + w) * 8 + q) * 64 + lane];
        b[q] += red[((wave + w) * 8 + 4 + q) * 64 + lane];
      }
}

// gate_up's ring slot: 128 bytes of codes of 16 gate rows, of 16 up rows (the
// rows' 16-byte chunks XOR-swizzled by the row), then the 32 rows' scales.
template <int FMT>
constexpr int gu_srow() { return Rows<FMT>::SSTEP * Rows<FMT>::STEPS; }
template <int FMT>
constexpr int gu_slot() { return 32 * (128 + gu_srow<FMT>()); }

// One wave's stream of gate_up units: in every round j < rounds it multiplies
// the pieces [lo, hi) of a unit's 16 gate rows and 16 up rows with all tokens'
// x~ (if j < mine) and hands the sums to finish(j, gate, up).  unit(j, codes,
// scales) gives a round's first gate row, factors(j, ..) its first block
// scales of block FP8, started() runs once the first loads are on their way.
// A ring of D slots; D - 1 are being loaded, over the rounds' borders.
template <int FMT, int D, typename Unit, typename Factors, typename Started, typename Finish>
__device__ __forceinline__ void gu_stream(int rounds, int mine, int lo, int hi, int K, int I, const uint8_t* sx, const float* xf, int xt, uint8_t* ring,
                                          Unit unit, Factors factors, Started started, Finish finish) {
  using R = Rows<FMT>;
  constexpr int SLOT = gu_slot<FMT>(), SR = gu_srow<FMT>();
  constexpr int W4 = 32 * SR / 4;                     // dwords of a slot's scales
  constexpr int ND = 4 + (W4 + 63) / 64, ND16 = SR == 16 ? 5 : ND;  // DMA instructions of a slot; with scales of 16 bytes a lane
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, kp = (K + 127) / 128 * 128, steps = kp / 128;
  const int rb = (int)code_row_bytes<FMT>(K), rs = (int)scale_row_bytes<FMT>(K);
  const uint32_t cup = (uint32_t)I * (uint32_t)rb, sup = (uint32_t)I * (uint32_t)rs;  // from the gate to the up rows
  const uint8_t* xrow = sx + (xt * (kp + 8) + 32 * g) * 2;
  const bool any = mine > 0 && hi > lo;
  const uint8_t *codes, *scales = nullptr;
  __amdgpu_buffer_rsrc_t bc, bs;
  // scales by DMA where rows begin at multiples of 16 bytes (4 bytes), else through registers
  unit(0, codes, scales);
  const uint32_t odd = (uint32_t)rs | (uint32_t)(uintptr_t)scales;
  const bool by16 = SR == 16 && (odd & 15) == 0, by4 = (odd & 3) == 0;
  int lj = 0, lb = lo;
  auto load_next = [&](int s) __attribute__((always_inline)) {
    uint8_t* to = ring + s * SLOT;
    if (lb == lo) {
      unit(min(lj, mine - 1), codes, scales);  // past the end the last unit again: every step issues as many loads
      bc = buffer_of(codes, (uint32_t)(I + 16) * (uint32_t)rb);
      if (SR > 0) bs = buffer_of(scales, (uint32_t)(I + 16) * (uint32_t)rs);
    }
    // chunks and scales past a row's end read the row's start (they meet zeros of x)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 8 * (j & 1) + lane / 8, at = 128 * lb + 16 * ((lane & 7) ^ (row >> 1));
      dma_buffer(bc, (uint32_t)(row * rb + (at < rb ? at : 0)), j < 2 ? 0 : cup, to + 1024 * j);
    }
    if constexpr (SR > 0) {
      to += 32 * 128;
      if (by16) {
        if (lane < 32) dma_buffer(bs, (uint32_t)((lane & 15) * rs + 16 * lb) + (lane < 16 ? 0 : sup), 0, to);
      } else if (by4) {
#pragma unroll
        for (int j = 0; j < (W4 + 63) / 64; ++j) {
          const int d = 64 * j + lane, row = d / (SR / 4), at = SR * lb + 4 * (d % (SR / 4));
          if (d < W4) dma_buffer4(bs, (uint32_t)((row & 15) * rs + (at < rs ? at : 0)) + (row < 16 ? 0 : sup), 0, to + 256 * j);
        }
      } else {
        for (int i = lane; i < 32 * SR; i += 64) {
          const int row = i / SR, at = SR * lb + i % SR;
          to[i] = at < rs ? scales[(row < 16 ? 0 : (int64_t)sup) + (row & 15) * rs + at] : 0;
        }
      }
    }
    if (++lb == hi) { lb = lo; ++lj; }
  };
  if (any) {
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load_next(d);
  }
  started();
  int slot = 0;
  for (int j = 0; j < rounds; ++j) {
    floatx4 ag{0.f, 0.f, 0.f, 0.f}, au = ag;
    if (any && j < mine) {
      const float *fg = nullptr, *fu = nullptr;
      if (FMT == FP4_FMT_FP8_BLOCK) factors(j, fg, fu);
      for (int b = lo; b < hi; ++b) {
        load_next(slot == 0 ? D - 1 : slot - 1);  // read a step ago: its values are in registers
        if (SR > 0 && !by4) __builtin_amdgcn_s_waitcnt(0);
        else if (by16) __builtin_amdgcn_s_waitcnt(vmcnt_only(ND16 * (D - 1)));
        else __builtin_amdgcn_s_waitcnt(vmcnt_only(ND * (D - 1)));
        asm volatile("" ::: "memory");
        const uint8_t *cg = ring + slot * SLOT + 128 * r, *sc = ring + slot * SLOT + 32 * 128 + SR * r;
        slot = slot == D - 1 ? 0 : slot + 1;
#pragma unroll
        for (int s = 0; s < R::STEPS; ++s) {
          const int kb = R::STEPS * b + s;
          if (s > 0 && kb >= steps) break;
          WStep<FMT> wg, wu;
          wg.read([&](int c) { return cg + 16 * ((R::STEP / 16 * s + c) ^ (r >> 1)); }, sc + R::SSTEP * s, g);
          wu.read([&](int c) { return cg + 2048 + 16 * ((R::STEP / 16 * s + c) ^ (r >> 1)); }, sc + 16 * SR + R::SSTEP * s, g);
          floatx4 pg = ag, pu = au;
          if (FMT == FP4_FMT_FP8_BLOCK) pg = pu = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x4 x = ld16(xrow + (128 * kb + 8 * q) * 2);
            pg = gu_mfma<FMT>(wg, q, x, pg);
            pu = gu_mfma<FMT>(wu, q, x, pu);
          }
          if (FMT == FP4_FMT_FP8_BLOCK) {
            const float f = xf[xt * steps + kb], fa = f * scalar_load(fg + kb), fb = f * scalar_load(fu + kb);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              ag[q] = fmaf(pg[q], fa, ag[q]);
              au[q] = fmaf(pu[q], fb, au[q]);
            }
          } else {
            ag = pg;
            au = pu;
          }
        }
      }
    }
    finish(j, ag, au);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // no DMA outlives the workgroup
}

// a wave's ring of D slots (the shared expert's MXFP8 slots share its bytes)
template <int MODE, int D>
__host__ __device__ constexpr int gu_ring(bool shared) {
  constexpr int own = D * gu_slot<weight_fmt(MODE)>(), sh = D * gu_slot<FP4_FMT_MXFP8>();
  return shared && sh > own ? sh : own;
}

template <int MODE, int D>
__global__ void __launch_bounds__(64 * kGuWaves, 2) few_gateup_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ float tmp[kGuWaves], xs[kFewTokens];
  __shared__ uint32_t s_amax;
  __shared__ unsigned long long touched[16];
  const int tid = threadIdx.x, th = blockDim.x, nw = th >> 6, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = a.T, k = a.k, H = a.H, P = T * k, split = a.k_split, ks = wave % split, per = nw / split;
  const GuSmem sm = gu_smem(T, a.E, k, H, AF == FP4_FMT_FP8_ROW, nw, gu_ring<MODE, D>(a.S > 0), split > 1);
  float* xf = reinterpret_cast<float*>(smem + sm.xf);
  float* red = reinterpret_cast<float*>(smem + sm.red);
  uint8_t* ring = smem + sm.ring + wave * gu_ring<MODE, D>(a.S > 0);
  const int xt = min(r, T - 1);  // columns past the last token repeat it and are not kept

  if ((int)blockIdx.x >= a.routed_wgs) {  // shared expert
    const int S = a.S, units = S / 16, wgs = gridDim.x - a.routed_wgs, first = (blockIdx.x - a.routed_wgs) * per + wave / split;
    prepare_x<FP4_FMT_MXFP8, FP4_FMT_MXFP8>(a, smem + sm.x, xf, xs, tmp);
    if ((int)blockIdx.x == a.routed_wgs) {  // sigmoid(x_t . g) on unquantized x
      for (int t = wave; t < T; t += nw) {
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
    const int NB = H / 128, lo = ks * NB / split, hi = (ks + 1) * NB / split;
    const int base = (blockIdx.x - a.routed_wgs) * per, rounds = (units - base + wgs * per - 1) / (wgs * per);
    const int mine = max(0, (units - first + wgs * per - 1) / (wgs * per));
    gu_stream<FP4_FMT_MXFP8, D>(
        rounds, mine, lo, hi, H, S, smem + sm.x, xf, xt, ring,
        [&](int j, const uint8_t*& codes, const uint8_t*& scales) __attribute__((always_inline)) {
          const int64_t row = 16 * (int64_t)(first + j * wgs * per);
          codes = a.ws13 + row * H;
          scales = a.ws13s + row * (H / 32);
        },
        [](int, const float*&, const float*&) {}, []() {},
        [&](int j, floatx4& ag, floatx4& au) __attribute__((always_inline)) {
          gu_reduce(ag, au, red, ks, split);
          if (j < mine && ks == 0 && r < T) {
            floatx4 h;
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = silu_f32(ag[q]) * au[q];
            *reinterpret_cast<floatx4*>(a.sh + (int64_t)r * S + 16 * (first + j * wgs * per) + 4 * g) = h;
          }
        });
    return;
  }

  int* ids = reinterpret_cast<int*>(smem + sm.ids);
  int* list = reinterpret_cast<int*>(smem + sm.list);
  float* scale = reinterpret_cast<float*>(smem + sm.scale);
  uint8_t* slots = smem + sm.slot;  // [listed expert][token]: the token's slot + 1
  if constexpr (AF == FP4_FMT_NONE) prepare_x<WF, AF>(a, smem + sm.x, xf, xs, tmp);
  for (int i = tid; i < min(a.E, P) * kFewTokens / 4; i += th) reinterpret_cast<uint32_t*>(slots)[i] = 0;
  if (tid == 0) s_amax = 0;
  if (tid < 16) touched[tid] = 0;
  auto weights = [&](int t, uint32_t key) __attribute__((always_inline)) {  // softmax over the selected values in f64; slots left over: weight 0
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
  };
  auto route = [&](auto n_, int t) __attribute__((always_inline)) {  // tokens t, t + nw, ..
    constexpr int N = decltype(n_)::value;
    const float* lg = a.logits + (int64_t)t * a.E;
    uint32_t key[N];
    if (a.E <= 128) select_topk<2, N>(lg, a.bias, a.E, k, nw, ids + t * k, key);
    else if (a.E <= 256) select_topk<4, N>(lg, a.bias, a.E, k, nw, ids + t * k, key);
    else if (a.E <= 512) select_topk<8, N>(lg, a.bias, a.E, k, nw, ids + t * k, key);
    else select_topk<16, N>(lg, a.bias, a.E, k, nw, ids + t * k, key);
    if (blockIdx.x == 0)
      for (int n = 0; n < N; ++n) weights(t + n * nw, key[n]);
  };
  for (int t = wave; t < T;) {
    if (t + nw < T) { route(std::integral_constant<int, 2>{}, t); t += 2 * nw; }
    else { route(std::integral_constant<int, 1>{}, t); t += nw; }
  }
  if constexpr (AF != FP4_FMT_NONE) prepare_x<WF, AF>(a, smem + sm.x, xf, xs, tmp);
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // x by DMA: a barrier alone does not wait for it
  __syncthreads();
  // the touched experts by id: a bit each, an expert's place in the list is the number of bits below its own
  for (int p = tid; p < P; p += th)
    if (ids[p] >= 0) atomicOr(&touched[ids[p] >> 6], 1ull << (ids[p] & 63));
  __syncthreads();
  uint64_t bits[16];
  int nd = 0;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    bits[c] = touched[c];
    nd += __popcll(bits[c]);
  }
  nd = __builtin_amdgcn_readfirstlane(nd);
  for (int p = tid; p < P; p += th) {
    const int e = ids[p];
    if (e < 0) continue;
    int at = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) at += __popcll(64 * c + 63 < e ? bits[c] : 64 * c < e ? bits[c] & ((1ull << (e & 63)) - 1) : 0ull);
    list[at] = e;
    slots[at * kFewTokens + p / k] = (uint8_t)(p % k + 1);
  }
  __syncthreads();
  if (blockIdx.x == 0) {  // for the down kernel
    for (int i = tid; i < H / 16; i += th) a.done[i] = 0;
    if (a.ids_out)
      for (int p = tid; p < P; p += th) a.ids_out[p] = ids[p];
    if (tid == 0) a.list[0] = nd;
    for (int i = tid; i < nd; i += th) a.list[1 + i] = list[i];
    for (int i = tid; i < nd; i += th) {
      int n = 0;
      for (int t = 0; t < T; ++t)
        if (const int j = slots[i * kFewTokens + t]) a.pairs[i * kFewTokens + n++] = t * k + j - 1;
      for (; n < kFewTokens; ++n) a.pairs[i * kFewTokens + n] = -1;
    }
  }

  const int I = a.I, strips = I / 16, units = nd * strips, base = blockIdx.x * per, first = base + wave / split, step = a.routed_wgs * per;
  const int64_t rb = code_row_bytes<WF>(H), rs = scale_row_bytes<WF>(H);
  constexpr int piece = 128 * Rows<WF>::STEPS;
  const int NB = (H + piece - 1) / piece, lo = ks * NB / split, hi = (ks + 1) * NB / split;
  float hmax = 0.0f;
  gu_stream<WF, D>(
      max(0, (units - base + step - 1) / step), max(0, (units - first + step - 1) / step), lo, hi, H, I, smem + sm.x, xf, xt, ring,
      [&](int j, const uint8_t*& codes, const uint8_t*& scales) __attribute__((always_inline)) {
        const int u = min(first + j * step, units - 1), e = __builtin_amdgcn_readfirstlane(list[u / strips]);
        const int64_t row = (int64_t)e * 2 * I + (u % strips) * 16;
        codes = a.w13 + row * rb;
        scales = static_cast<const uint8_t*>(a.w13s) + row * rs;
      },
      [&](int j, const float*& fg, const float*& fu) __attribute__((always_inline)) {
        const int u = first + j * step, e = __builtin_amdgcn_readfirstlane(list[u / strips]), KB = H / 128;
        fg = static_cast<const float*>(a.w13s) + ((int64_t)e * (2 * I / 128) + (u % strips) / 8) * KB;
        fu = fg + (int64_t)(I / 128) * KB;
      },
      [&]() __attribute__((always_inline)) {
        if constexpr (WF == FP4_FMT_NVFP4) {
          for (int i = tid; i < nd; i += th) scale[i] = a.w13s2[list[i]];
          __syncthreads();
        }
      },
      [&](int j, floatx4& ag, floatx4& au) __attribute__((always_inline)) {
        gu_reduce(ag, au, red, ks, split);
        const int u = first + j * step;
        if (u >= units || ks != 0) return;
        const int ai = u / strips, i0 = (u % strips) * 16, slot = slots[ai * kFewTokens + r];
        if (slot == 0) return;  // not a token of this expert
        const int64_t p = (int64_t)r * k + slot - 1;
        const float s = WF == FP4_FMT_NVFP4 ? scale[ai] * xs[r] : 1.0f;
        floatx4 h;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = silu_f32(ag[q] * s) * (au[q] * s);
        if constexpr (AF == FP4_FMT_NONE) {
          uint32_t t[4][3];
#pragma unroll
          for (int q = 0; q < 4; ++q) bf16_terms(h[q], t[q]);
#pragma unroll
          for (int i = 0; i < 3; ++i)
            *reinterpret_cast<u32x2*>(a.hb + (p * 3 + i) * I + i0 + 4 * g) = u32x2{t[0][i] | t[1][i] << 16, t[2][i] | t[3][i] << 16};
        } else {
          *reinterpret_cast<floatx4*>(a.h + p * I + i0 + 4 * g) = h;
#pragma unroll
          for (int q = 0; q < 4; ++q) hmax = fmaxf(hmax, fabsf(h[q]));
        }
      });
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
    if constexpr (AF == FP4_FMT_FP8_ROW) {  // code times scale, as three terms
      const int p = c / (a.I / 32), i0 = 32 * (c - p * (a.I / 32));
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        u32x4 w[3];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t lo[3], hi[3];
          bf16_terms(v[i + 2 * q] * f, lo);
          bf16_terms(v[i + 2 * q + 1] * f, hi);
#pragma unroll
          for (int t = 0; t < 3; ++t) w[t][q] = lo[t] | hi[t] << 16;
        }
#pragma unroll
        for (int t = 0; t < 3; ++t) st16(a.hb + ((int64_t)p * 3 + t) * a.I + i0 + i, w[t]);
      }
    } else {
      store_bf16x32(a.hb + 32 * (int64_t)c, v);
    }
  } else if (c < routed + shared) {
    load(a.sh + 32 * (int64_t)(c - routed));
    quantize32<FP4_FMT_MXFP8>(v, ts);
    store_bf16x32(a.shb + 32 * (int64_t)(c - routed), v);
  }
}

// --------------------------------------------------------------------- down

// A slot of the down kernel: one work item of a wave, a segment of m K steps of
// 16 weight rows (codes, then scales) and of h of up to PP pairs (NT terms
// each).  A row's 16-byte chunk c lies at place c + row (modulo the row), so
// that the 16 lanes that read one chunk of 16 rows hit different banks.
struct DnSlot {
  int cs, sd, hc;            // chunks of a code row, dwords of a scale row, chunks of an h row
  int scales, h, bytes, dmas;
};
template <int FMT>
__host__ __device__ inline DnSlot dn_slot(int m, int rows) {
  DnSlot s;
  s.cs = Rows<FMT>::STEP / 16 * m;
  s.sd = Rows<FMT>::SSTEP / 4 * m;
  s.hc = 16 * m;
  s.scales = 256 * s.cs;
  s.h = s.scales + 64 * s.sd;
  s.bytes = s.h + rows * s.hc * 16;
  s.dmas = s.cs / 4 + (16 * s.sd + 63) / 64 + rows * ((s.hc + 63) / 64);
  return s;
}
template <int FMT>
constexpr int dn_most_steps() { return Rows<FMT>::FP4 ? 8 : 4; }  // of an item: 8 DMA instructions of codes
constexpr int dn_terms(int mode) { return act_fmt(mode) == FP4_FMT_NONE || act_fmt(mode) == FP4_FMT_FP8_ROW ? 3 : 1; }

// Waits until at most n loads are on their way (more than 63: 63).
template <int LO = 0, int HI = 63>
__device__ __forceinline__ void wait_vm(int n) {
  if constexpr (LO == HI) {
    __builtin_amdgcn_s_waitcnt(vmcnt_only(LO));
  } else {
    constexpr int MID = (LO + HI + 1) / 2;
    if (n >= MID) wait_vm<MID, HI>(n);
    else wait_vm<LO, MID - 1>(n);
  }
}

// One wave's share of the down products of a strip of 16 outputs (rows n0 ..):
// experts i0, i0 + istep, .. < i1 of a list, up to PP of an expert's pairs at a
// time, segments [lo, hi) of m steps of K.  An item's weights and h come by
// DMA into one of the wave's two slots while the other is computed; nothing is
// shared between waves, so none waits for another.  h's rows (term * PP +
// pair) are the columns of the MFMA tile.  expert(i) gives the expert's number
// and pair count, pair(i, q) its q-th pair, factor(i, q) what multiplies that
// pair's product, token(p) its row of the wave's sums yl [T][16].
template <int FMT, int NT, typename Expert, typename Pair, typename Factor, typename Token>
__device__ __forceinline__ void dn_stream(const uint8_t* w, const uint8_t* ws, const float* wf, int H, int K, int n0, int m, int lo, int hi, int i0, int istep,
                                          int i1, const uint16_t* h, uint32_t h_bytes, int PP, uint8_t* slots, float* yl, Expert expert, Pair pair,
                                          Factor factor, Token token) {
  using R = Rows<FMT>;
  if (i0 >= i1 || lo >= hi) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int rb = (int)code_row_bytes<FMT>(K), rs = (int)scale_row_bytes<FMT>(K), rows = PP * NT, steps = (K + 127) / 128;
  const DnSlot sl = dn_slot<FMT>(m, rows);
  const bool by4 = (((uint32_t)rs | (uint32_t)(uintptr_t)ws) & 3) == 0;
  const auto hb = buffer_of(h, h_bytes);
  uint32_t coff[8], soff[4];  // a lane's byte offsets in the item's code rows and scale rows
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t at = 64 * j + lane, row = at / (uint32_t)sl.cs, c = at - row * sl.cs, rot = row % (uint32_t)sl.cs;
    coff[j] = row * rb + 16 * (c >= rot ? c - rot : c - rot + sl.cs);
  }
  if constexpr (R::SSTEP > 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = 64 * j + lane, row = at / (uint32_t)sl.sd;
      soff[j] = row * rs + 4 * (at - row * sl.sd);
    }
  }
  struct Item { int i, p0, seg; };
  auto issue = [&](const Item& it, uint8_t* slot) __attribute__((always_inline)) {
    const int2 ex = expert(it.i);
    const int64_t row = (int64_t)ex.x * H + n0;
    // rows and h past K give what lies behind them or zeros; the products skip it
    const int cat = 16 * sl.cs * it.seg, sat = 4 * sl.sd * it.seg;
    const auto bc = buffer_of(w + row * rb + cat, (uint32_t)(16 * rb - cat));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (4 * j < sl.cs) dma_buffer(bc, coff[j], 0, slot + 1024 * j);
    if constexpr (R::SSTEP > 0) {
      if (by4) {
        const auto bs = buffer_of(ws + row * rs + sat, (uint32_t)(16 * rs - sat));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (64 * j + lane < 16 * sl.sd) dma_buffer4(bs, soff[j], 0, slot + sl.scales + 256 * j);
      } else {
        for (int b = lane; b < 64 * sl.sd; b += 64) {
          const int q = b / (4 * sl.sd), at = sat + b - q * 4 * sl.sd;
          slot[sl.scales + b] = at < rs ? ws[(row + q) * rs + at] : 0;
        }
      }
    }
    for (int q = 0; q < rows; ++q) {
      const int t = q / PP, pq = q - t * PP, n = ex.y - it.p0;
      const int p = __builtin_amdgcn_readfirstlane(pair(it.i, it.p0 + (pq < n ? pq : 0)));  // rows past the pairs repeat the first
      const uint32_t at = (uint32_t)(2 * ((p * NT + t) * K + 128 * m * it.seg));
      for (int c0 = 0; c0 < sl.hc; c0 += 64) {
        const int c = c0 + lane - q;
        if (c0 + lane < sl.hc) dma_buffer(hb, at + 16 * (c < 0 ? c + sl.hc : c), 0, slot + sl.h + (q * sl.hc + c0) * 16);
      }
    }
  };
  auto advance = [&](Item& it) __attribute__((always_inline)) {
    if (++it.seg < hi) return;
    it.seg = lo;
    it.p0 += PP;
    if (it.p0 >= expert(it.i).y) { it.p0 = 0; it.i += istep; }
  };
  Item now{i0, 0, lo}, next = now;
  issue(next, slots);
  advance(next);
  uint8_t *slot = slots, *other = slots + sl.bytes;
  const int hr = r < rows ? r : 0;
  floatx4 acc{0.f, 0.f, 0.f, 0.f};
  while (now.i < i1) {
    if (next.i < i1) {
      __builtin_amdgcn_s_waitcnt(lgkmcnt0());  // the other slot's values are in registers
      issue(next, other);
      advance(next);
      if (R::SSTEP > 0 && !by4) __builtin_amdgcn_s_waitcnt(0);
      else wait_vm(sl.dmas);
    } else {
      __builtin_amdgcn_s_waitcnt(0);
    }
    asm volatile("" ::: "memory");
    const uint8_t *crow = slot + 16 * sl.cs * r, *srow = slot + sl.scales + 4 * sl.sd * r, *hrow = slot + sl.h + 16 * sl.hc * hr;
    const int rot = r % (uint32_t)sl.cs;
    const float* fw = FMT == FP4_FMT_FP8_BLOCK ? wf + ((int64_t)expert(now.i).x * (H / 128) + n0 / 128) * (K / 128) : nullptr;
    const int last = min(m, steps - m * now.seg);
    for (int s = 0; s < last; ++s) {
      const int kb = m * now.seg + s;
      const bool in = 128 * kb + 32 * g < K;
      WStep<FMT> v;
      v.read([&](int c) {
        c += R::STEP / 16 * s + rot;
        return crow + 16 * (c >= sl.cs ? c - sl.cs : c);
      }, srow + R::SSTEP * s, g);
      u32x4 x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int c = 16 * s + 4 * g + q + hr;
        c -= c >= sl.hc ? sl.hc : 0;
        x[q] = ld16(hrow + 16 * c);
      }
      if (128 * kb + 128 > K && !in) {  // what lies behind a row may be NaN: weights and h both give way to zeros
        v.c[0] = u32x4{0, 0, 0, 0};
        if constexpr (!R::FP4) v.c[1] = v.c[0];
        v.s = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = u32x4{0, 0, 0, 0};
      }
      floatx4 pr = FMT == FP4_FMT_FP8_BLOCK ? floatx4{0.f, 0.f, 0.f, 0.f} : acc;
#pragma unroll
      for (int q = 0; q < 4; ++q) pr = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(v, q), __builtin_bit_cast(bf16x8_t, x[q]), pr, 0, 0, 0);
      if (FMT == FP4_FMT_FP8_BLOCK) {
        const float f = scalar_load(fw + kb);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = fmaf(pr[q], f, acc[q]);
      } else {
        acc = pr;
      }
    }
    if (now.seg == hi - 1) {
      // the terms' columns of a pair add up, then go to its token's outputs (a token is in an expert's list once)
      floatx4 v = acc;
      if constexpr (NT == 3) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += __shfl(acc[q], lane + PP) + __shfl(acc[q], lane + 2 * PP);
      }
      if (r < PP && now.p0 + r < expert(now.i).y) {
        const float f = factor(now.i, now.p0 + r);
        floatx4* y = reinterpret_cast<floatx4*>(yl + token(pair(now.i, now.p0 + r)) * 16 + 4 * g);
        floatx4 o = *y;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = fmaf(v[q], f, o[q]);
        *y = o;
      }
      acc = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    advance(now);
    uint8_t* t = slot;
    slot = other;
    other = t;
  }
}

// Grid: (strips of 16 outputs, splits).  The waves of a workgroup share the
// experts of its split (a run of the touched ones), or (the last shared_splits)
// a run of the shared expert's K, then their sums are added in the waves'
// order.  More than one split: the sums go to ypart, and the last workgroup of
// a strip to arrive adds all splits up, in their order, and writes y.  Partial
// sums are stored and read at device scope, past the XCDs' L2s; no workgroup
// waits for another.
template <int MODE, typename OutT>
__global__ void __launch_bounds__(64 * kDnWaves, 2) few_down_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE), NT = dn_terms(MODE);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int2 s_expert[kDnSeg];                 // this split's experts: number, pairs
  __shared__ int16_t s_pair[kDnSeg][kFewTokens];
  __shared__ float s_factor[kDnSeg][kFewTokens];    // routing weight times the tensor scales
  __shared__ int s_last;
  const int tid = threadIdx.x, th = blockDim.x, nw = th >> 6, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = a.T, H = a.H, k = a.k, split = blockIdx.y, total = gridDim.y, n0 = blockIdx.x * 16;
  float* yl = reinterpret_cast<float*>(smem) + wave * T * 16;  // the waves' sums, then their slots
  uint8_t* slots = smem + nw * T * 64;
  for (int q = tid & 63; q < T * 16; q += 64) yl[q] = 0.0f;
  if (split < a.splits) {
    const int nd = a.list[0], a0 = split * nd / a.splits, a1 = (split + 1) * nd / a.splits;
    for (int i = tid; i < (a1 - a0) * kFewTokens; i += th) {
      const int e = a.list[1 + a0 + (i >> 4)], p = a.pairs[a0 * kFewTokens + i];
      float f = a.wts[max(p, 0)];
      if (WF == FP4_FMT_NVFP4) f *= a.w2s2[e];
      if (AF == FP4_FMT_NVFP4) f *= a.h_ts[0];
      s_pair[i >> 4][i & 15] = (int16_t)p;
      s_factor[i >> 4][i & 15] = f;
      const uint64_t on = __ballot(p >= 0) >> (threadIdx.x & 48) & 0xFFFFull;  // 16 lanes hold one expert's pairs
      if ((i & 15) == 0) s_expert[i >> 4] = int2{e, __popcll(on)};
    }
    __syncthreads();
    dn_stream<WF, NT>(
        a.w2, static_cast<const uint8_t*>(a.w2s), static_cast<const float*>(a.w2s), H, a.I, n0, a.seg_steps, 0,
        ((a.I + 127) / 128 + a.seg_steps - 1) / a.seg_steps, wave, nw, a1 - a0, a.hb, (uint32_t)(T * k) * NT * a.I * 2, a.pass_pairs,
        slots + wave * 2 * dn_slot<WF>(a.seg_steps, a.pass_pairs * NT).bytes, yl,
        [&](int i) __attribute__((always_inline)) {
          return int2{__builtin_amdgcn_readfirstlane(s_expert[i].x), __builtin_amdgcn_readfirstlane(s_expert[i].y)};
        },
        [&](int i, int q) __attribute__((always_inline)) { return (int)s_pair[i][q]; },
        [&](int i, int q) __attribute__((always_inline)) { return s_factor[i][q]; },
        [&](int p) __attribute__((always_inline)) { return p / k; });
  } else {
    const int S = a.S, NB = S / 128, part = (split - a.splits) * nw + wave, parts = a.shared_splits * nw;
    if (tid < T) s_factor[0][tid] = a.sgate[tid];
    __syncthreads();
    dn_stream<FP4_FMT_MXFP8, 1>(
        a.ws2, a.ws2s, nullptr, H, S, n0, 1, part * NB / parts, (part + 1) * NB / parts, 0, 1, 1, a.shb, (uint32_t)(T * S * 2), T,
        slots + wave * 2 * dn_slot<FP4_FMT_MXFP8>(1, T).bytes, yl,
        [&](int) __attribute__((always_inline)) { return int2{0, T}; }, [](int, int q) __attribute__((always_inline)) { return q; },
        [&](int, int q) __attribute__((always_inline)) { return s_factor[0][q]; }, [](int p) __attribute__((always_inline)) { return p; });
  }
  __syncthreads();
  for (int q0 = tid; q0 < T * 16; q0 += th) {
    const float* y0 = reinterpret_cast<const float*>(smem) + q0;
    float v = 0.0f;
    for (int i = 0; i < nw; ++i) v += y0[i * T * 16];
    const int64_t at = (int64_t)(q0 >> 4) * H + n0 + (q0 & 15);
    if (total > 1) __hip_atomic_store(a.ypart + (int64_t)split * T * H + at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else if constexpr (sizeof(OutT) == 4) static_cast<OutT*>(a.y)[at] = v;
    else static_cast<OutT*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
  if (total == 1) return;
  __builtin_amdgcn_s_waitcnt(0);  // this thread's stores acknowledged
  __syncthreads();
  if (tid == 0) s_last = __hip_atomic_fetch_add(a.done + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
  __syncthreads();
  if (!s_last) return;
  for (int q0 = tid; q0 < T * 16; q0 += th) {
    const int64_t at = (int64_t)(q0 >> 4) * H + n0 + (q0 & 15);
    float v = 0.0f;
    for (int s0 = 0; s0 < total; s0 += 8) {
      float t[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        t[s] = __hip_atomic_load(a.ypart + (int64_t)min(s0 + s, total - 1) * T * H + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int s = 0; s < 8; ++s) v += s0 + s < total ? t[s] : 0.0f;
    }
    if constexpr (sizeof(OutT) == 4) static_cast<OutT*>(a.y)[at] = v;
    else static_cast<OutT*>(a.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

// --------------------------------------------------------------------- host

struct FewPlan {
  int mode, splits, shared_splits, pass_pairs, seg_steps;
  int nw, depth, dn_waves;  // gate_up: waves of a workgroup, slots of a wave's ring; down: waves of a workgroup
  size_t wts, list, pairs, done, sgate, amax_part, h_ts, h, hb, sh, shb, ypart, total;
};

constexpr int kFewCus = 256;        // workgroups that a launch aims at: the card's compute units
constexpr int kLds = 160 * 1024;
constexpr int kGuLds = kLds - 256;  // dynamic LDS beside the gate_up kernel's static bytes
constexpr int kMoreSplits = 15;     // of a strip, above the fewest
constexpr int kDnLds = kLds - kDnSeg * (8 + kFewTokens * 6) - 64;

template <int D>
static int ring_bytes(int mode, bool shared) {
  switch (mode) {
    case FM_NV: case FM_NVNV: return gu_ring<FM_NV, D>(shared);
    case FM_MX: case FM_MXMX: return gu_ring<FM_MX, D>(shared);
    default: return gu_ring<FM_FP8, D>(shared);
  }
}

// LDS of a down workgroup: the waves' sums and two slots each
static size_t dn_smem(int mode, int T, int pairs, int m, int nw) {
  const int rows = pairs * dn_terms(mode);
  const DnSlot s = mode == FM_FP8 ? dn_slot<FP4_FMT_FP8_BLOCK>(m, rows)
                   : mode == FM_NV || mode == FM_NVNV ? dn_slot<FP4_FMT_NVFP4>(m, rows) : dn_slot<FP4_FMT_MXFP4>(m, rows);
  return (size_t)nw * (64 * T + 2 * s.bytes);
}
static size_t dn_smem_shared(int T, int nw) { return (size_t)nw * (64 * T + 2 * dn_slot<FP4_FMT_MXFP8>(1, T).bytes); }

static int few_plan(const moe_fp4_layer* L, int64_t T, FewPlan* out) {
  FP4_CHECK(validate_layer(L, T));
  if (T > kFewTokens) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: %lld tokens, at most %d", (long long)T, kFewTokens);
  if (L->num_experts > 1024) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: more than 1024 experts");
  if (L->hidden > 1 << 16 || L->inter > 1 << 16 || L->shared_inter > 1 << 16)
    return fail(FP4_ERR_UNSUPPORTED, "few-token forward: a width above 65536");
  const bool nv = L->w_fmt == FP4_FMT_NVFP4;
  FewPlan p{};
  p.mode = L->w_fmt == FP4_FMT_FP8_BLOCK ? FM_FP8 : L->a_fmt == FP4_FMT_NONE ? (nv ? FM_NV : FM_MX) : (nv ? FM_NVNV : FM_MXMX);
  const int nt = L->a_fmt == FP4_FMT_NONE || L->a_fmt == FP4_FMT_FP8_ROW ? 3 : 1;
  const size_t P = (size_t)T * L->top_k, D = std::min<size_t>(P, L->num_experts), I = L->inter, S = L->shared_inter, H = L->hidden;
  // gate_up: the most waves whose rings fit beside x, with the deepest rings that do
  const int rings[][2] = {{8, 4}, {8, 3}, {8, 2}, {4, 2}, {2, 2}, {1, 2}};
  for (auto& r : rings) {
    const int ring = r[1] == 4 ? ring_bytes<4>(p.mode, S > 0) : r[1] == 3 ? ring_bytes<3>(p.mode, S > 0) : ring_bytes<2>(p.mode, S > 0);
    if (p.nw == 0 && gu_smem((int)T, L->num_experts, L->top_k, L->hidden, p.mode == FM_FP8, r[0], ring, D * (I / 16) < (size_t)kFewCus * r[0]).total <= kGuLds) {
      p.nw = r[0];
      p.depth = r[1];
    }
  }
  if (p.nw == 0 && T > 0)
    return fail(FP4_ERR_UNSUPPORTED, "few-token forward: %lld tokens of width %d do not fit the LDS", (long long)T, L->hidden);
  // down: items as long in K as they may be (whole rows lie behind each other in memory) with enough waves beside each
  // other, as many pairs at once as a touched expert has on average
  const int steps = ((int)I + 127) / 128, strips = (int)H / 16, most = p.mode == FM_FP8 ? dn_most_steps<FP4_FMT_FP8_BLOCK>() : dn_most_steps<FP4_FMT_NVFP4>();
  const double touched = L->num_experts * (1.0 - std::pow(1.0 - (double)L->top_k / L->num_experts, (double)T));
  p.pass_pairs = (int)std::max(1.0, std::min({std::floor((double)P / std::max(touched, 1.0) + 0.5), 16.0 / dn_terms(p.mode), (double)std::max<int64_t>(T, 1)}));
  for (int segs = (steps + most - 1) / most; p.dn_waves < 6 && segs <= steps; ++segs) {
    p.seg_steps = (steps + segs - 1) / segs;
    for (p.dn_waves = kDnWaves; p.dn_waves > 1 && dn_smem(p.mode, (int)T, p.pass_pairs, p.seg_steps, p.dn_waves) > kDnLds;) --p.dn_waves;
  }
  // splits of a strip: the shortest rounds of the card, counting 1 us to begin a workgroup, 2 us to join splits, and items
  // at 24 GB/s a compute unit
  p.shared_splits = S ? (int)((S / 128 + 15) / 16) : 0;
  const double item = 16.0 * p.seg_steps * (p.mode == FM_FP8 ? 128 : 72) / 24e3, passes = (double)((steps + p.seg_steps - 1) / p.seg_steps);
  const int least = std::max(1, (int)((D + kDnSeg - 1) / kDnSeg));
  double best = 1e30;
  for (int s = least; s <= least + kMoreSplits; ++s) {
    const int wgs = strips * (s + p.shared_splits), per = (int)std::ceil(std::ceil(touched / s) / p.dn_waves);
    const double t = (wgs + kFewCus - 1) / kFewCus * (1.0 + per * passes * p.dn_waves * item) + (s + p.shared_splits > 1 ? 2.0 : 0.0);
    if (t < best) {
      best = t;
      p.splits = s;
    }
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  p.wts = take(4 * P);
  p.list = take(4 * (1 + D));
  p.pairs = take(4 * D * kFewTokens);
  p.done = take(4 * strips);
  p.sgate = take(4 * T);
  p.amax_part = take(4 * 2 * kFewCus);
  p.h_ts = take(4);
  p.h = take(L->a_fmt == FP4_FMT_NONE ? 0 : 4 * P * I);
  p.hb = take(2 * nt * P * I);
  p.sh = take(4 * T * S);
  p.shb = take(2 * T * S);
  p.ypart = take(4 * (size_t)(least + kMoreSplits + p.shared_splits) * T * H);  // for the most splits: more tokens, more bytes
  p.total = off;
  *out = p;
  return FP4_OK;
}

template <int MODE, int D>
static int launch_few(FewArgs a, const FewPlan& p, int y_dtype, hipStream_t st) {
  constexpr int AF = act_fmt(MODE);
  static std::atomic<uint64_t> gu_raised{0}, dn32_raised{0}, dn16_raised{0};
  FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_gateup_kernel<MODE, D>), kGuLds, gu_raised));
  const int ring = gu_ring<MODE, D>(a.S > 0), strips = a.I / 16, max_units = std::min(a.E, a.T * a.k) * strips;
  // a unit is split between waves (each a run of its pieces) until the units there may be fill the chip's waves
  a.k_split = 1;
  while (a.k_split < p.nw && max_units * a.k_split < kFewCus * p.nw) a.k_split *= 2;
  const int lds = gu_smem(a.T, a.E, a.k, a.H, MODE == FM_FP8, p.nw, ring, a.k_split > 1).total;
  const int per = p.nw / a.k_split, fit = kFewCus * std::max(1, std::min(2, kLds / (lds + 64)));
  int shared = 0;  // workgroups of the shared expert, by its share of the bytes
  if (a.S > 0) {
    const double sb = 2.0 * a.S, rb = (double)std::min(a.E, a.T * a.k) * 2 * a.I * (MODE == FM_FP8 ? 1.0 : 0.55);
    shared = std::max(1, std::min((a.S / 16 + per - 1) / per, (int)(fit * sb / (sb + rb))));
  }
  a.routed_wgs = std::max(1, std::min(fit - shared, (max_units + per - 1) / per));
  hipLaunchKernelGGL((few_gateup_kernel<MODE, D>), dim3((unsigned)(a.routed_wgs + shared)), dim3(64 * p.nw), (size_t)lds, st, a);
  FP4_CHECK(check_launch("few_gateup"));
  const int64_t lanes = (AF == FP4_FMT_NONE ? 0 : (int64_t)a.T * a.k * (a.I / 32)) + (int64_t)a.T * (a.S / 32);
  if (lanes > 0) {
    hipLaunchKernelGGL(few_hquant_kernel<AF>, dim3(grid_1d(lanes, 256)), dim3(256), 0, st, a);
    FP4_CHECK(check_launch("few_hquant"));
  }
  const size_t dn_lds = std::max(dn_smem(MODE, a.T, a.pass_pairs, a.seg_steps, p.dn_waves), a.S ? dn_smem_shared(a.T, p.dn_waves) : 0);
  const dim3 grid((unsigned)(a.H / 16), (unsigned)(a.splits + a.shared_splits)), block(64 * p.dn_waves);
  if (y_dtype == FP4_DT_F32) {
    FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_down_kernel<MODE, float>), kDnLds, dn32_raised));
    hipLaunchKernelGGL((few_down_kernel<MODE, float>), grid, block, dn_lds, st, a);
  } else {
    FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_down_kernel<MODE, uint16_t>), kDnLds, dn16_raised));
    hipLaunchKernelGGL((few_down_kernel<MODE, uint16_t>), grid, block, dn_lds, st, a);
  }
  return check_launch("few_down");
}

template <int MODE>
static int launch_few(const FewArgs& a, const FewPlan& p, int y_dtype, hipStream_t st) {
  if (p.depth == 4) return launch_few<MODE, 4>(a, p, y_dtype, st);
  if (p.depth == 3) return launch_few<MODE, 3>(a, p, y_dtype, st);
  return launch_few<MODE, 2>(a, p, y_dtype, st);
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
  a.splits = p.splits; a.shared_splits = p.shared_splits; a.pass_pairs = p.pass_pairs; a.seg_steps = p.seg_steps;
  a.list = reinterpret_cast<int32_t*>(b + p.list);
  a.pairs = reinterpret_cast<int32_t*>(b + p.pairs);
  a.done = reinterpret_cast<int32_t*>(b + p.done);
  a.wts = reinterpret_cast<float*>(b + p.wts);
  a.sgate = reinterpret_cast<float*>(b + p.sgate);
  a.amax_part = reinterpret_cast<float*>(b + p.amax_part);
  a.h_ts = reinterpret_cast<float*>(b + p.h_ts);
  a.h = reinterpret_cast<float*>(b + p.h);
  a.hb = reinterpret_cast<uint16_t*>(b + p.hb);
  a.sh = reinterpret_cast<float*>(b + p.sh);
  a.shb = reinterpret_cast<uint16_t*>(b + p.shb);
  a.ypart = reinterpret_cast<float*>(b + p.ypart);
  a.ids_out = topk_ids; a.wts_out = topk_weights; a.y = y;
  hipStream_t st = as_stream(stream);
  switch (p.mode) {
    case FM_NV: return launch_few<FM_NV>(a, p, y_dtype, st);
    case FM_MX: return launch_few<FM_MX>(a, p, y_dtype, st);
    case FM_NVNV: return launch_few<FM_NVNV>(a, p, y_dtype, st);
    case FM_MXMX: return launch_few<FM_MXMX>(a, p, y_dtype, st);
    default: return launch_few<FM_FP8>(a, p, y_dtype, st);
  }
}

}  // extern "C"
