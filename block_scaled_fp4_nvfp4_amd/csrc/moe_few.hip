// A whole routed-expert layer for a few tokens (at most 16), from the router's
// logits to y, behind moe_fp4_forward_few (gfx950):
//
//   l' = fp32(logit + bias), the k largest l' (ties: lower id), w = softmax over them
//   h_tj = Qh(SiLU(G_e x~_t) * (U_e x~_t)),  e = ids[t][j],  x~ = Qx(x)
//   y_t  = sum_j w_tj D_e h_tj  (+ sigmoid(x_t . g) * shared(x_t))
//
// Three kernels: routing, x~ and the gate_up products (every workgroup routes
// the tokens by itself, so none waits for another); the down products, whose
// waves make h~ themselves; the weighted sum of a token's products.
//
// What bounds it: the touched experts' weights, read once (2.76 MB an expert
// at hidden 2560, intermediate 640 in NVFP4).  They come by DMA into LDS slots
// that belong to one wave, without barriers; loading MFMA fragments straight
// into registers touches four rows in every four lanes and measured twice the
// time.  All tokens of the call are the 16 columns of one 16x16x32 MFMA tile,
// so gate_up decodes an expert's weights once whatever the number of its tokens
// and gathers nothing: it computes every column and keeps those of the
// expert's tokens.
//
// Measured at 512 experts, hidden 2560, intermediate 640, top 10, in graph
// replays over 16 sets of logits (us; in brackets the same layer through the
// router and the sorted forward): 1, 4, 8 and 16 tokens with NVFP4 weights 27
// [33], 45 [47], 70 [66], 111 [96]; MXFP4 25 [32], 41 [47], 62 [65], 100 [94];
// NVFP4/NVFP4 33 [72], 53 [86], 78 [114], 122 [190]; MXFP4/MXFP8 25 [38], 42
// [54], 64 [70], 101 [101]; block FP8 31 [58], 58 [85], 93 [115], 151 [175]; with a
// shared expert of 1280: NVFP4/NVFP4, top 5, 16 tokens 85 [129], block FP8, 7
// tokens 92 [126].  NVFP4 with little to read: 8 experts of 256 x 128, one token 16
// [14]; 64 experts, top 4, 16 tokens 54 [44].  So with plain activations the other
// way is faster above about 8 tokens or with few weights, with MXFP8 as fast at 16:
// every workgroup routes every token here, and plain h costs two or three columns
// a pair.  Of the time at one token of NVFP4 routing takes 4.5, the
// list of experts 1.3, gate_up 9, each gap between kernels 1.5, the down products
// 7, the sum 2; at 16 tokens routing and x~ 12, gate_up 56 (4.6 TB/s), the down
// products 34 (3.8 TB/s).
//
// Exactness.  Weights and x~ are exact where they meet: in fp16 for NVFP4
// weights (E2M1 codes times E4M3 scales, 6 significant bits) with x~ of NVFP4
// or a plain x scaled to fp16's range, in bf16 for MXFP4 (E2M1 codes times
// powers of two) and block FP8 (E4M3 codes alone; their scales multiply the f32
// sum of each 128-block).  An h held in f32 (not quantized, or FP8 codes times
// their scales) is split into terms: in bf16 three, whose sum is h down to bf16's
// smallest step, 2^-133 (all of an h of 2^-110 and more), for NVFP4 weights two in
// fp16 (dn_terms).  Sums are f32; scales whose product may leave f32 are applied one
// power of two at the end (scale_by, add_scaled).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

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

// format pairs of the layer
enum FewMode { FM_NV = 0, FM_MX = 1, FM_NVNV = 2, FM_MXMX = 3, FM_FP8 = 4 };
constexpr int weight_fmt(int mode) {
  return mode == FM_NV || mode == FM_NVNV ? FP4_FMT_NVFP4 : mode == FM_FP8 ? FP4_FMT_FP8_BLOCK : FP4_FMT_MXFP4;
}
constexpr int act_fmt(int mode) {
  return mode == FM_NVNV ? FP4_FMT_NVFP4 : mode == FM_MXMX ? FP4_FMT_MXFP8 : mode == FM_FP8 ? FP4_FMT_FP8_ROW : FP4_FMT_NONE;
}

// One pass of the down products: up to pass_pairs pairs of one expert.  gate_up's
// first workgroup writes a record for each.
struct DnPass {
  int32_t expert, n;
  uint16_t pair[kFewTokens];  // t * k + j | t << 9; those past n repeat the first
  float scale;                // the expert's tensor scale
  int32_t pad[5];
  float factor[kFewTokens];   // routing weight
};
static_assert(sizeof(DnPass) == 128);

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
  int down_wgs;            // down workgroups of the routed experts; the rest take the shared expert
  int pass_pairs, seg_steps;  // of the down kernel: pairs of an expert at once, 128-wide K steps of a slot
  // workspace
  int32_t* list;           // passes, then the selected experts of every token
  DnPass* passes;          // [T k]
  float *sgate, *amax_part;
  float* h;                // [T k, I]
  float* sh;               // [T, S]
  float* d;                // f32 [T k + S / 128 * T, H] weighted down products of the pairs, of the shared expert's K steps
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

// Values 8j .. 8j+7 of them as bf16 (exact): MXFP4 and the E4M3 formats.
template <int FMT>
__device__ __forceinline__ bf16x8_t wstep_frag(const WStep<FMT>& v, int j) {
  u32x4 p;
  if constexpr (FMT == FP4_FMT_MXFP4) {
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
__device__ __forceinline__ floatx4 w_mfma(const WStep<FMT>& w, int j, u32x4 x, floatx4 acc) {
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
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[16 * b + i]) & 0x7FFFFFFFu);
      float amax = __uint_as_float(top);
      const bool finite = top < 0x7F800000u;
      if (!finite) {
        amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[16 * b + i]));
      }
      uint32_t sc = 0xFFu;
      if (ts > 0x1p-100f && ts < 0x1p100f) sc = e4m3_of_quotient(amax, amax / (6.0f * ts), 6.0f, ts);
      if (sc == 0xFFu) sc = ts > 0.0f ? e4m3_rne_sat_f64((double)amax / (6.0 * (double)ts)) : 0u;  // subnormal scales
      const float s = __builtin_amdgcn_cvt_f32_fp8((int)sc, 0);
      // E2M1's borders have at most 8 significant bits.  q: the quotient |v| / (s ts) rounded to 8 bits (from an f32 one
      // that is less than 2^-21 off); the sign of the exact rest |v| - q s ts (q s has 12 bits, the fma rounds once) says
      // on which side of q the quotient lies, and q moves a quarter of its last place there: the hardware's rounding of
      // what results is the quotient's.
      const float unit = s * ts, inv = __builtin_amdgcn_rcpf(unit);
      if (finite && unit > 0x1p-100f && unit < 0x1p100f) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float* x = v + 16 * b + 8 * w;
          float q[8], f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = fabsf(x[i]);
            const uint32_t n = (__float_as_uint(fminf(y * inv, 8.0f)) + 0x8000u) & 0xFFFF0000u;
            const float rest = fmaf(-(__uint_as_float(n) * s), ts, y);
            q[i] = __uint_as_float(n + (rest > 0.0f ? 0x4000u : rest < 0.0f ? 0u - 0x4000u : 0u));
          }
          uint32_t d = 0;
          d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[0], q[1], 1.0f, 0);
          d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[2], q[3], 1.0f, 1);
          d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[4], q[5], 1.0f, 2);
          d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[6], q[7], 1.0f, 3);
          e2m1x8_to_f32x8(d, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = copysignf(f[i] * s, x[i]);
        }
      } else {
        const E2M1Thresholds th = e2m1_thresholds((double)s * (double)ts);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[16 * b + i] = copysignf(e2m1_mag_to_f32(e2m1_code(fabsf(v[16 * b + i]), th)) * s, v[16 * b + i]);
      }
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
  using Order = std::conditional_t<(PL > 8), uint64_t, uint32_t>;
  Order order[N];  // the i's of a lane's experts left, four bits each, the head's lowest
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    const float b = bias && e < E ? bias[e] : 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      id[n][i] = i;
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
  for (int n = 0; n < N; ++n) {
    mine[n] = 0;
    my_id[n] = -1;
    order[n] = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) order[n] |= (Order)id[n][i] << (4 * i);
  }
  for (int j = 0; j < k; ++j) {
    uint32_t top[N];
#pragma unroll
    for (int n = 0; n < N; ++n) top[n] = wave_umax(key[n][0]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint64_t at = __ballot(key[n][0] == top[n]);
      int win = __builtin_ctzll(at), e = 64 * (__builtin_amdgcn_readlane((int)order[n], win) & 15) + win;
      if (top[n] != 0)
        for (at &= at - 1; at; at &= at - 1) {  // equal values: the lowest id
          const int l = __builtin_ctzll(at), o = 64 * (__builtin_amdgcn_readlane((int)order[n], l) & 15) + l;
          if (o < e) { e = o; win = l; }
        }
      if (lane == j) { mine[n] = top[n]; my_id[n] = top[n] ? e : -1; }  // nothing selectable left: -1
      if (lane == win) {
#pragma unroll
        for (int i = 0; i + 1 < PL; ++i) key[n][i] = key[n][i + 1];
        key[n][PL - 1] = 0u;
        order[n] >>= 4;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (lane < k) s_ids[n * step * k + lane] = my_id[n];
}

// ------------------------------------------------------------------ gate_up

struct GuSmem {
  int x, xf, ids, wts, list, scale, slot, red, ring, total;
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
  s.wts = s.ids + T * k * 4;
  s.list = s.wts + T * k * 4;
  s.scale = s.list + D * 4;
  s.slot = s.scale + D * 4;
  s.red = (s.slot + D * kFewTokens + 15) / 16 * 16;
  s.ring = s.red + (split ? nw * 64 * 8 * 4 : 0);
  s.total = s.ring + nw * ring;
  return s;
}

// Copies x into LDS by DMA, [T][kp + 8] with zeros behind H; the last waves,
// which route fewer tokens, first.
__device__ __forceinline__ void copy_x(const FewArgs& a, uint8_t* sx) {
  const int H = a.H, kp = (H + 127) / 128 * 128, T = a.T, nw = (int)blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const auto xb = buffer_of(a.x, (uint32_t)(T * H * 2));
  for (int t = nw - 1 - wave; t < T; t += nw) {
    uint8_t* row = sx + t * (kp + 8) * 2;
    for (int c = 0; c < H / 8; c += 64)
      if (c + lane < H / 8) dma_buffer(xb, (uint32_t)(t * H * 2 + 16 * (c + lane)), 0, row + 16 * c);
    if (H / 8 + lane < kp / 8) st16(row + 16 * (H / 8 + lane), u32x4{0, 0, 0, 0});
  }
}

__device__ __forceinline__ float amax_bf16x8(u32x4 w, float m) {
#pragma unroll
  for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
  return m;
}
__device__ __forceinline__ float wave_amax(float m) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  return m;
}

// Makes x~ of the copied x, in place: bf16, or fp16 for NVFP4 weights (WF).
// xs[t] gets the factor of a token's products, xf those of its K steps (FP8
// rows).  Plain x meets NVFP4 weights as fp16 scaled by the power of two that
// brings the token's largest value to [2^14, 2^15): exact down to 2^-29 of
// that value, and 2^-39 of it off below: inside the f32 sums' own rounding,
// unless the weights of that largest value are zeros.
template <int WF, int AF>
__device__ __forceinline__ void prepare_x(const FewArgs& a, uint8_t* sx, float* xf, float* xs, float* tmp) {
  const int H = a.H, kp = (H + 127) / 128 * 128, T = a.T, nw = (int)blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // this wave's rows of x
  asm volatile("" ::: "memory");
  if constexpr (AF == FP4_FMT_NONE) {
    for (int t = nw - 1 - wave; t < T; t += nw) {
      uint8_t* row = sx + t * (kp + 8) * 2;
      int e = 15;
      if constexpr (WF == FP4_FMT_NVFP4) {
        float m = 0.0f;
        for (int c = lane; c < H / 8; c += 64) m = amax_bf16x8(ld16(row + 16 * c), m);
        e = __builtin_amdgcn_frexp_expf(fminf(wave_amax(m), 3.4028234663852886e38f));
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
      }
      if (lane == 0) xs[t] = ldexpf(1.0f, e - 15);
    }
    return;
  }
  __syncthreads();
  float ts = 1.0f;
  if constexpr (AF == FP4_FMT_NVFP4) {
    if (a.x_scale) {
      ts = a.x_scale[0];
    } else {
      float m = 0.0f;
      for (int t = wave; t < T; t += nw)
        for (int c = lane; c < H / 8; c += 64) m = amax_bf16x8(ld16(sx + t * (kp + 8) * 2 + 16 * c), m);
      m = wave_amax(m);
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
    uint8_t* at = sx + (t * (kp + 8) + 32 * q) * 2;
    float v[32];
    load_bf16x32(reinterpret_cast<const uint16_t*>(at), v);
    const float f = quantize32<AF>(v, ts);
    if constexpr (WF == FP4_FMT_NVFP4) store_f16x32(at, v);
    else store_bf16x32(at, v);
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
// Two slots: one is loaded, over the rounds' borders, while the other is
// multiplied (three and four slots measured the same).
template <int FMT, typename Unit, typename Factors, typename Started, typename Finish>
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
      unit(lj, codes, scales);
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
  if (any) load_next(0);
  started();
  int slot = 0;
  for (int j = 0; j < rounds; ++j) {
    floatx4 ag{0.f, 0.f, 0.f, 0.f}, au = ag;
    if (any && j < mine) {
      const float *fg = nullptr, *fu = nullptr;
      if (FMT == FP4_FMT_FP8_BLOCK) factors(j, fg, fu);
      for (int b = lo; b < hi; ++b) {
        const bool more = lj < mine;
        __builtin_amdgcn_s_waitcnt(lgkmcnt0());  // the other slot's values are in registers
        if (more) load_next(slot ^ 1);
        if (!more || (SR > 0 && !by4)) __builtin_amdgcn_s_waitcnt(0);
        else if (by16) __builtin_amdgcn_s_waitcnt(vmcnt_only(ND16));
        else __builtin_amdgcn_s_waitcnt(vmcnt_only(ND));
        asm volatile("" ::: "memory");
        const uint8_t *cg = ring + slot * SLOT + 128 * r, *sc = ring + slot * SLOT + 32 * 128 + SR * r;
        slot ^= 1;
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
            pg = w_mfma<FMT>(wg, q, x, pg);
            pu = w_mfma<FMT>(wu, q, x, pu);
          }
          if (FMT == FP4_FMT_FP8_BLOCK) {
            const float f = xf[xt * steps + kb], sg = scalar_load(fg + kb), su = scalar_load(fu + kb);
            add_scaled(ag, pg, f, sg);
            add_scaled(au, pu, f, su);
          } else {
            ag = pg;
            au = pu;
          }
        }
      }
    }
    finish(j, ag, au);
  }
}

// a wave's two slots (the shared expert's MXFP8 slots share their bytes)
template <int MODE>
__host__ __device__ constexpr int gu_ring(bool shared) {
  constexpr int own = 2 * gu_slot<weight_fmt(MODE)>(), sh = 2 * gu_slot<FP4_FMT_MXFP8>();
  return shared && sh > own ? sh : own;
}

template <int MODE>
__global__ void __launch_bounds__(64 * kGuWaves, 2) few_gateup_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ float tmp[kGuWaves], xs[kFewTokens];
  __shared__ uint32_t s_amax;
  __shared__ int s_np;
  __shared__ unsigned long long touched[16];
  const int tid = threadIdx.x, th = blockDim.x, nw = th >> 6, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = a.T, k = a.k, H = a.H, P = T * k, split = a.k_split, ks = wave % split, per = nw / split;
  const GuSmem sm = gu_smem(T, a.E, k, H, AF == FP4_FMT_FP8_ROW, nw, gu_ring<MODE>(a.S > 0), split > 1);
  float* xf = reinterpret_cast<float*>(smem + sm.xf);
  float* red = reinterpret_cast<float*>(smem + sm.red);
  uint8_t* ring = smem + sm.ring + wave * gu_ring<MODE>(a.S > 0);
  const int xt = min(r, T - 1);  // columns past the last token repeat it and are not kept

  if ((int)blockIdx.x >= a.routed_wgs) {  // shared expert
    const int S = a.S, units = S / 16, wgs = gridDim.x - a.routed_wgs, first = (blockIdx.x - a.routed_wgs) * per + wave / split;
    copy_x(a, smem + sm.x);
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
    gu_stream<FP4_FMT_MXFP8>(
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
  float* wts = reinterpret_cast<float*>(smem + sm.wts);
  float* scale = reinterpret_cast<float*>(smem + sm.scale);
  uint8_t* slots = smem + sm.slot;  // [listed expert][token]: the token's slot + 1
  copy_x(a, smem + sm.x);  // on its way while the tokens are routed
  for (int i = tid; i < min(a.E, P) * kFewTokens / 4; i += th) reinterpret_cast<uint32_t*>(slots)[i] = 0;
  if (tid == 0) s_amax = 0, s_np = 0;
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
      wts[t * k + lane] = w;
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
  prepare_x<WF, AF>(a, smem + sm.x, xf, xs, tmp);
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
    if (a.ids_out)
      for (int p = tid; p < P; p += th) a.ids_out[p] = ids[p];
    if (tid < T) {
      int n = 0;
      for (int j = 0; j < k; ++j) n += ids[tid * k + j] >= 0;
      a.list[1 + tid] = n;
    }
    for (int i = tid; i < nd; i += th) {  // the order of the passes does not matter: every pair's products have a row of their own
      const uint8_t* sl = slots + i * kFewTokens;
      int n = 0, q = 0;
      for (int t = 0; t < T; ++t) n += sl[t] != 0;
      DnPass* pass = a.passes + atomicAdd(&s_np, (n + a.pass_pairs - 1) / a.pass_pairs);
      const float f = WF == FP4_FMT_NVFP4 ? a.w2s2[list[i]] : 1.0f;
      for (int t = 0; t < T; ++t) {
        if (sl[t] == 0) continue;
        const int p = t * k + sl[t] - 1;
        pass->pair[q] = (uint16_t)(p | t << 9);
        pass->factor[q] = wts[p];
        --n;
        if (++q == a.pass_pairs || n == 0) {
          pass->expert = list[i];
          pass->scale = f;
          pass->n = q;
          for (; q < a.pass_pairs; ++q) pass->pair[q] = pass->pair[0];
          ++pass;
          q = 0;
        }
      }
    }
    __syncthreads();
    if (tid == 0) a.list[0] = s_np;
  }

  const int I = a.I, strips = I / 16, units = nd * strips, base = blockIdx.x * per, first = base + wave / split, step = a.routed_wgs * per;
  const int64_t rb = code_row_bytes<WF>(H), rs = scale_row_bytes<WF>(H);
  constexpr int piece = 128 * Rows<WF>::STEPS;
  const int NB = (H + piece - 1) / piece, lo = ks * NB / split, hi = (ks + 1) * NB / split;
  float hmax = 0.0f;
  gu_stream<WF>(
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
        floatx4 h;
        if constexpr (WF == FP4_FMT_NVFP4) {
          const float s = scale[ai], sx = xs[r];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            ag[q] = scale_by(ag[q], s, sx);
            au[q] = scale_by(au[q], s, sx);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = silu_f32(ag[q]) * au[q];
        *reinterpret_cast<floatx4*>(a.h + p * I + i0 + 4 * g) = h;
        if constexpr (AF == FP4_FMT_NVFP4) {
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

// --------------------------------------------------------------------- down

// A wave's LDS in the down kernel: two slots for a segment of m K steps of 16
// weight rows (codes, then scales), h of a pass (rows of `steps` K steps), its
// record, and the products of up to `hold` strips.  A row's 16-byte chunk c
// lies at place c + row (modulo the row), so that the 16 lanes that read one
// chunk of 16 rows hit different banks.
struct DnWave {
  int cs, sd, hc;  // chunks of a code row, dwords of a scale row, chunks of an h row
  int scales, slot, dmas, h, rec, out, hold, bytes;
};
template <int FMT>
__host__ __device__ inline DnWave dn_wave(int m, int steps, int pairs, int terms) {
  DnWave s;
  s.cs = Rows<FMT>::STEP / 16 * m;
  s.sd = Rows<FMT>::SSTEP / 4 * m;
  s.hc = 16 * steps;
  s.scales = 256 * s.cs;
  s.slot = s.scales + 64 * s.sd;
  s.dmas = s.cs / 4 + (16 * s.sd + 63) / 64;
  s.h = 2 * s.slot;
  s.rec = s.h + pairs * terms * s.hc * 16;
  s.out = s.rec + (int)sizeof(DnPass);
  s.hold = pairs > 2 ? 32 / pairs : 16;
  s.bytes = s.out + s.hold * pairs * 64;
  return s;
}
template <int FMT>
constexpr int dn_most_steps() { return Rows<FMT>::FP4 ? 8 : 4; }  // of a slot: 8 DMA instructions of codes
// terms whose sum is h: one where its quantized values are exact in a term, three in bf16 for codes times a scale (FP8)
// and for a plain h; a plain h meets NVFP4 weights as two fp16 terms, scaled by the power of two that brings the pair's
// largest value to [2^14, 2^15): off by less than 2^-22 of a value, or 2^-39 of that largest one, like the f32 sums' own
// roundings
constexpr int dn_terms(int mode) { return mode == FM_NV ? 2 : mode == FM_MX || mode == FM_FP8 ? 3 : 1; }

// Waits until at most n loads are on their way (more than 15: 15).
template <int LO = 0, int HI = 15>
__device__ __forceinline__ void wait_vm(int n) {
  if constexpr (LO == HI) {
    __builtin_amdgcn_s_waitcnt(vmcnt_only(LO));
  } else {
    constexpr int MID = (LO + HI + 1) / 2;
    if (n >= MID) wait_vm<MID, HI>(n);
    else wait_vm<LO, MID - 1>(n);
  }
}

// A word that the kernel before wrote, at an address all lanes share.
__device__ __forceinline__ uint32_t scalar_word(const void* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) uint32_t*>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ int pass_pair(const DnPass* p, int q) {
  return (int)(scalar_word(p->pair + (q & ~1)) >> (16 * (q & 1)) & 511);
}

// One wave's down products of one pass: strips [s0, s1) of 16 outputs of an
// expert (rows row0 + 16 strip of w), PP pairs of h, all of K or (the shared
// expert) its K steps [first, first + steps).  The wave quantizes the pass's h
// (format AF, tensor scale ts) itself, into NT bf16 terms: the rows term * PP +
// pair are the columns of the MFMA tile and stay in LDS.  The weights stream
// through two slots, one being copied while the other is computed.  Nothing is
// shared between waves, so none waits for another.  h_row(q) is where pair q's
// h begins; its product times factor(q), wscale and ts goes to row out_row(q) of d.
template <int FMT, int AF, int NT, typename HRow, typename Factor, typename OutRow>
__device__ __forceinline__ void dn_run(const uint8_t* w, const uint8_t* ws, const float* wf, int64_t row0, int H, int K, int first, int steps, int m, int s0, int s1,
                                       float ts, float wscale, const DnPass* rec, int n, int PP, uint8_t* lds, float* d, HRow h_row,
                                       Factor factor, OutRow out_row) {
  using R = Rows<FMT>;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int rb = (int)code_row_bytes<FMT>(K), rs = (int)scale_row_bytes<FMT>(K), rows = PP * NT, segs = (steps + m - 1) / m;
  const DnWave sl = dn_wave<FMT>(m, steps, PP, NT);
  const bool by4 = (((uint32_t)rs | (uint32_t)(uintptr_t)ws) & 3) == 0;
  // n / d = n (2^16 / d + 1) >> 16 for n < 512, d <= 32 (off by less than 512 / 2^16 < 1 / d)
  const uint32_t inv_cs = 65536u / sl.cs + 1, inv_sd = 65536u / max(sl.sd, 1) + 1;
  uint32_t coff[8], soff[4];  // a lane's byte offsets in a slot's code rows and scale rows
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t at = 64 * j + lane, row = at * inv_cs >> 16, c = at - row * sl.cs, rot = row - (row * inv_cs >> 16) * sl.cs;
    coff[j] = row * rb + 16 * (c >= rot ? c - rot : c - rot + sl.cs);
  }
  if constexpr (R::SSTEP > 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = 64 * j + lane, row = at * inv_sd >> 16;
      soff[j] = row * rs + 4 * (at - row * sl.sd);
    }
  }
  auto issue = [&](int strip, int seg, uint8_t* slot) __attribute__((always_inline)) {
    const int64_t row = row0 + 16 * strip;
    // rows past K give what lies behind them or zeros; the products skip it
    const int kb = first + m * seg, cat = R::STEP * kb, sat = R::SSTEP * kb;
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
  };
  const int hr = r < rows ? r : 0, rot = r - (int)(r * inv_cs >> 16) * sl.cs;
  const uint8_t* hrow = lds + sl.h + 16 * sl.hc * hr;
  float* out = reinterpret_cast<float*>(lds + sl.out);
  issue(s0, 0, lds);
  // the record, and h, 32 values a lane
  if (rec) {
    const auto b = buffer_of(rec, sizeof(DnPass));
    if (lane < (int)sizeof(DnPass) / 4) dma_buffer4(b, 4 * lane, 0, lds + sl.rec);
  }
  const int blocks = 4 * steps;
  auto load = [&](const float* p, int b, float (&v)[32]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const floatx4 w = *reinterpret_cast<const floatx4*>(p + min(128 * first + 32 * b, K - 32) + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
    }
  };
  auto store = [&](int pq, int b, int i, const u32x4 (&w)[NT]) __attribute__((always_inline)) {  // values 8 i .. of the block
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int q = t * PP + pq, c = 4 * b + i + q;
      st16(lds + sl.h + (q * sl.hc + (c >= sl.hc ? c - sl.hc : c)) * 16, w[t]);
    }
  };
  float unscale = 1.0f;  // of pair r
  if constexpr (NT == 2) {
    for (int pq = 0; pq < PP; ++pq) {
      const float* p = h_row(pq);
      float v[32], top = 0.0f;
      for (int b = (blocks - 1) / 64 * 64 + lane; b >= 0; b -= 64)  // the lane's first block last: its values stay
        if (b < blocks) {
          load(p, b, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(v[i]));
        }
      const int e = __builtin_amdgcn_frexp_expf(fminf(wave_amax(top), 3.4028234663852886e38f));
      if (r == pq) unscale = ldexpf(1.0f, e - 15);
      for (int b = lane; b < blocks; b += 64) {
        if (b != lane) load(p, b, v);
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          half8_t a, c;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = ldexpf(v[i + j], 15 - e);
            a[j] = (_Float16)x;
            const float rest = x - (float)a[j];  // exact; NaN after an infinity
            c[j] = (_Float16)(rest == rest ? rest : 0.0f);
          }
          store(pq, b, i / 8, {__builtin_bit_cast(u32x4, a), __builtin_bit_cast(u32x4, c)});
        }
      }
    }
  } else {
    for (int u = lane; u < PP * blocks; u += 64) {
      const int pq = u / blocks, b = u - pq * blocks;
      float v[32];
      load(h_row(pq), b, v);
      const float f = quantize32<AF>(v, ts);
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        u32x4 w[NT];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = v[i + 2 * j], y = v[i + 2 * j + 1];
          if constexpr (NT == 3) {
            uint32_t tx[3], ty[3];
            bf16_terms(x * f, tx);
            bf16_terms(y * f, ty);
#pragma unroll
            for (int t = 0; t < 3; ++t) w[t][j] = tx[t] | ty[t] << 16;
          } else if constexpr (FMT == FP4_FMT_NVFP4) {
            w[0][j] = __builtin_bit_cast(uint32_t, half2_t{(_Float16)x, (_Float16)y});
          } else {
            w[0][j] = pack_exact_bf16(x, y);
          }
        }
        store(pq, b, i / 8, w);
      }
    }
  }
  int strip = s0, seg = 0, base = s0;  // base: the first strip whose products `out` holds
  uint8_t *slot = lds, *other = lds + sl.slot;
  floatx4 acc{0.f, 0.f, 0.f, 0.f};
  while (strip < s1) {
    const bool end = seg + 1 == segs;
    const int nstrip = end ? strip + 1 : strip, nseg = end ? 0 : seg + 1;
    if (nstrip < s1) {
      __builtin_amdgcn_s_waitcnt(lgkmcnt0());  // the other slot's values are in registers
      issue(nstrip, nseg, other);
      if (R::SSTEP > 0 && !by4) __builtin_amdgcn_s_waitcnt(0);
      else wait_vm(sl.dmas);
    } else {
      __builtin_amdgcn_s_waitcnt(0);
    }
    asm volatile("" ::: "memory");
    const uint8_t *crow = slot + 16 * sl.cs * r, *srow = slot + sl.scales + 4 * sl.sd * r;
    const float* fw = FMT == FP4_FMT_FP8_BLOCK ? wf + ((row0 + 16 * strip) / 128) * (K / 128) + first + m * seg : nullptr;
    const int last = min(m, steps - m * seg);
    struct Step {
      WStep<FMT> w;
      u32x4 x[4];
    };
    auto read = [&](Step& v, int s) __attribute__((always_inline)) {
      v.w.read([&](int c) {
        c += R::STEP / 16 * s + rot;
        return crow + 16 * (c >= sl.cs ? c - sl.cs : c);
      }, srow + R::SSTEP * s, g);
      const int hs = m * seg + s, k0 = 128 * (first + hs);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int c = 16 * hs + 4 * g + q + hr;
        c -= c >= sl.hc ? sl.hc : 0;
        v.x[q] = ld16(hrow + 16 * c);
      }
      if (k0 + 128 > K && k0 + 32 * g >= K) {  // what lies behind a row may be NaN: weights and h both give way to zeros
        v.w.c[0] = u32x4{0, 0, 0, 0};
        if constexpr (!R::FP4) v.w.c[1] = v.w.c[0];
        v.w.s = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) v.x[q] = u32x4{0, 0, 0, 0};
      }
    };
    auto product = [&](const Step& v, int s) __attribute__((always_inline)) {
      floatx4 pr = FMT == FP4_FMT_FP8_BLOCK ? floatx4{0.f, 0.f, 0.f, 0.f} : acc;
#pragma unroll
      for (int q = 0; q < 4; ++q) pr = w_mfma<FMT>(v.w, q, v.x[q], pr);
      if (FMT == FP4_FMT_FP8_BLOCK) {
        const float f = scalar_load(fw + s);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = fmaf(pr[q], f, acc[q]);
      } else {
        acc = pr;
      }
    };
    Step a, b;  // a step's values leave LDS while the one before is multiplied
    read(a, 0);
    for (int s = 0;;) {
      if (s + 1 < last) read(b, s + 1);
      product(a, s);
      if (++s >= last) break;
      if (s + 1 < last) read(a, s + 1);
      product(b, s);
      if (++s >= last) break;
    }
    if (end) {
      floatx4 v = acc;  // the terms' columns of a pair add up
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (NT == 2) v[q] += __shfl(acc[q], lane + PP);
        if constexpr (NT == 3) v[q] += __shfl(acc[q], lane + PP) + __shfl(acc[q], lane + 2 * PP);
      }
      if (r < PP) {
        const float f = factor(r);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = scale_by(v[q] * f, wscale, NT == 2 ? unscale : ts);
        *reinterpret_cast<floatx4*>(out + (r * sl.hold + strip - base) * 16 + 4 * g) = v;
      }
      acc = floatx4{0.f, 0.f, 0.f, 0.f};
      const int held = strip + 1 - base;
      if (held == sl.hold || strip + 1 == s1) {  // a store's acknowledgement would hold up the loads behind it: few stores
        for (int q = 0; q < n; ++q) {
          const int64_t at = (int64_t)out_row(q) * H + 16 * base;
          if (lane < 4 * held) *reinterpret_cast<floatx4*>(d + at + 4 * lane) = *reinterpret_cast<const floatx4*>(out + q * sl.hold * 16 + 4 * lane);
        }
        base = strip + 1;
      }
    }
    strip = nstrip;
    seg = nseg;
    uint8_t* t = slot;
    slot = other;
    other = t;
  }
}

// The (pass, strip) pairs, pass by pass, are cut into one run a wave; the
// shared expert's (K step, strip) pairs go to the last workgroups in the same
// way.  The products of every pair (and of every K step of the shared expert)
// are rows of d in the workspace, which few_sum_kernel adds up: waves that added
// the strips they completed took 2.5 us for each, one after another, a tail
// of up to 27 us at 16 tokens.
template <int MODE>
__global__ void __launch_bounds__(64 * kDnWaves, 2) few_down_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE), NT = dn_terms(MODE);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int nw = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int T = a.T, H = a.H, S = a.S, P = T * a.k, strips = H / 16;
  const int np = (int)scalar_word(a.list), shared_parts = S / 128;
  const bool shared = (int)blockIdx.x >= a.down_wgs;
  const uint32_t waves = (shared ? gridDim.x - a.down_wgs : a.down_wgs) * nw, at = (shared ? blockIdx.x - a.down_wgs : blockIdx.x) * nw + wave;
  const uint64_t items = (uint64_t)(shared ? shared_parts : np) * strips;
  const uint32_t lo = (uint32_t)(items * at / waves), hi = (uint32_t)(items * (at + 1) / waves);
  if (!shared) {
    const int steps = (a.I + 127) / 128, PP = a.pass_pairs;
    const DnWave sl = dn_wave<WF>(a.seg_steps, steps, PP, NT);
    uint8_t* lds = smem + wave * sl.bytes;
    const DnPass* ldp = reinterpret_cast<const DnPass*>(lds + sl.rec);
    float ts = 1.0f;
    if constexpr (AF == FP4_FMT_NVFP4) {
      if (a.h_scale) {
        ts = a.h_scale[0];
      } else {
        float m = 0.0f;
        for (int i = lane; i < a.routed_wgs; i += 64) m = fmaxf(m, a.amax_part[i]);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
        ts = (float)((double)m / kNvTensorDivisor);
      }
    }
    for (uint32_t it = lo; it < hi;) {
      const uint32_t pass = it / strips, s0 = it - pass * strips, s1 = min((uint32_t)strips, s0 + hi - it);
      const DnPass* rec = a.passes + pass;
      const int n = (int)scalar_word(&rec->n);
      dn_run<WF, AF, NT>(
          a.w2, static_cast<const uint8_t*>(a.w2s), static_cast<const float*>(a.w2s), (int64_t)scalar_word(&rec->expert) * H, H, a.I, 0, steps, a.seg_steps, (int)s0, (int)s1,
          ts, __uint_as_float(scalar_word(&rec->scale)), rec, n, PP, lds, a.d,
          [&](int q) __attribute__((always_inline)) { return a.h + (int64_t)(PP == 1 ? pass_pair(rec, 0) : rec->pair[q] & 511) * a.I; },
          [&](int q) __attribute__((always_inline)) { return ldp->factor[q]; },
          [&](int q) __attribute__((always_inline)) { return pass_pair(rec, q); });
      it += s1 - s0;
    }
  } else {
    const DnWave sl = dn_wave<FP4_FMT_MXFP8>(1, 1, T, 1);
    const float gate = a.sgate[min(lane & 15, T - 1)];
    for (uint32_t it = lo; it < hi;) {
      const uint32_t part = it / strips, s0 = it - part * strips, s1 = min((uint32_t)strips, s0 + hi - it);
      dn_run<FP4_FMT_MXFP8, FP4_FMT_MXFP8, 1>(
          a.ws2, a.ws2s, nullptr, 0, H, S, (int)part, 1, 1, (int)s0, (int)s1, 1.0f, 1.0f, nullptr, T, T, smem + wave * sl.bytes, a.d,
          [&](int q) __attribute__((always_inline)) { return a.sh + (int64_t)q * S; }, [&](int) __attribute__((always_inline)) { return gate; },
          [&](int q) __attribute__((always_inline)) { return (int)(P + part * T) + q; });
      it += s1 - s0;
    }
  }
}

// y: the sum of a token's rows of d, in the order of its slots, then of the
// shared expert's K steps; a lane four outputs of a token.  Bound by latency:
// workgroups of one wave, over many compute units, took 1 us less than of four.
template <typename OutT>
__global__ void __launch_bounds__(64) few_sum_kernel(FewArgs a) {
  const int quads = a.H / 4, i = blockIdx.x * 64 + threadIdx.x;
  if (i >= a.T * quads) return;
  const int t = i / quads, c = 4 * (i - t * quads), P = a.T * a.k;
  floatx4 v{0.f, 0.f, 0.f, 0.f};
  auto rows = [&](int row, int step, int n) __attribute__((always_inline)) {
    for (int j0 = 0; j0 < n; j0 += 10) {
      floatx4 w[10];
#pragma unroll
      for (int j = 0; j < 10; ++j) w[j] = *reinterpret_cast<const floatx4*>(a.d + (int64_t)(row + min(j0 + j, n - 1) * step) * a.H + c);
#pragma unroll
      for (int j = 0; j < 10; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += j0 + j < n ? w[j][q] : 0.0f;
    }
  };
  rows(t * a.k, 1, a.list[1 + t]);
  rows(P + t, a.T, a.S / 128);
  OutT* y = static_cast<OutT*>(a.y) + (int64_t)t * a.H + c;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(OutT) == 4) y[q] = v[q];
    else y[q] = __builtin_bit_cast(uint16_t, (__bf16)v[q]);
  }
}

// --------------------------------------------------------------------- host

struct FewPlan {
  int mode, pass_pairs, seg_steps;
  int nw, dn_waves;  // waves of a gate_up, of a down workgroup
  size_t list, passes, sgate, amax_part, h, sh, d, total;
};

constexpr int kFewCus = 256;        // workgroups that a launch aims at: the card's compute units
constexpr int kLds = 160 * 1024;
constexpr int kGuLds = kLds - 256;  // dynamic LDS beside the gate_up kernel's static bytes

static int ring_bytes(int mode, bool shared) {
  switch (mode) {
    case FM_NV: case FM_NVNV: return gu_ring<FM_NV>(shared);
    case FM_MX: case FM_MXMX: return gu_ring<FM_MX>(shared);
    default: return gu_ring<FM_FP8>(shared);
  }
}

static size_t dn_smem(int mode, int steps, int pairs, int m, int nw) {
  const int terms = dn_terms(mode);
  const DnWave s = mode == FM_FP8 ? dn_wave<FP4_FMT_FP8_BLOCK>(m, steps, pairs, terms)
                   : mode == FM_NV || mode == FM_NVNV ? dn_wave<FP4_FMT_NVFP4>(m, steps, pairs, terms) : dn_wave<FP4_FMT_MXFP4>(m, steps, pairs, terms);
  return (size_t)nw * s.bytes;
}
static size_t dn_smem_shared(int T, int nw) { return (size_t)nw * dn_wave<FP4_FMT_MXFP8>(1, 1, T, 1).bytes; }

static int few_plan(const moe_fp4_layer* L, int64_t T, FewPlan* out) {
  FP4_CHECK(validate_layer(L, T));
  if (T > kFewTokens) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: %lld tokens, at most %d", (long long)T, kFewTokens);
  if (L->num_experts > 1024) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: more than 1024 experts");
  if (L->hidden > 1 << 16 || L->inter > 1 << 16 || L->shared_inter > 1 << 16)
    return fail(FP4_ERR_UNSUPPORTED, "few-token forward: a width above 65536");
  // one expert's gate and up rows lie behind one buffer descriptor
  if ((int64_t)(L->inter + 16) * L->hidden >> (L->w_fmt == FP4_FMT_FP8_BLOCK ? 31 : 32) || (int64_t)(L->shared_inter + 16) * L->hidden >> 31)
    return fail(FP4_ERR_UNSUPPORTED, "few-token forward: an expert's gate_up codes of more than 2 GiB");
  const bool nv = L->w_fmt == FP4_FMT_NVFP4;
  FewPlan p{};
  p.mode = L->w_fmt == FP4_FMT_FP8_BLOCK ? FM_FP8 : L->a_fmt == FP4_FMT_NONE ? (nv ? FM_NV : FM_MX) : (nv ? FM_NVNV : FM_MXMX);
  const size_t P = (size_t)T * L->top_k, D = std::min<size_t>(P, L->num_experts), I = L->inter, S = L->shared_inter, H = L->hidden;
  // gate_up: the most waves whose slots fit beside x
  const int ring = ring_bytes(p.mode, S > 0);
  for (int nw = kGuWaves; nw >= 1 && p.nw == 0; nw /= 2)
    if (gu_smem((int)T, L->num_experts, L->top_k, L->hidden, p.mode == FM_FP8, nw, ring, D * (I / 16) < (size_t)kFewCus * nw).total <= kGuLds) p.nw = nw;
  if (p.nw == 0 && T > 0)
    return fail(FP4_ERR_UNSUPPORTED, "few-token forward: %lld tokens of width %d do not fit the LDS", (long long)T, L->hidden);
  // down: slots as long in K as they may be (whole rows lie behind each other in memory) with enough waves beside each
  // other, as many pairs at once as a touched expert has on average
  const int steps = ((int)I + 127) / 128, most = p.mode == FM_FP8 ? dn_most_steps<FP4_FMT_FP8_BLOCK>() : dn_most_steps<FP4_FMT_NVFP4>();
  const double touched = std::max(1.0, L->num_experts * (1.0 - std::pow(1.0 - (double)L->top_k / L->num_experts, (double)T)));
  int pairs = (int)std::max(1.0, std::min({std::floor((double)P / touched + 0.5), 16.0 / dn_terms(p.mode), (double)std::max<int64_t>(T, 1)}));
  for (; p.dn_waves < 4 && pairs > 0; --pairs) {
    p.pass_pairs = pairs;
    for (int segs = (steps + most - 1) / most; p.dn_waves < 6 && segs <= steps; ++segs) {
      p.seg_steps = (steps + segs - 1) / segs;
      for (p.dn_waves = kDnWaves; p.dn_waves > 0 && dn_smem(p.mode, steps, pairs, p.seg_steps, p.dn_waves) > kLds;) --p.dn_waves;
    }
  }
  if (p.dn_waves == 0) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: intermediate width too large for the LDS");
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  p.list = take(4 * (1 + kFewTokens));
  p.passes = take(sizeof(DnPass) * P);
  p.sgate = take(4 * T);
  p.amax_part = take(4 * 2 * kFewCus);
  p.h = take(4 * P * I);
  p.sh = take(4 * T * S);
  p.d = take(4 * (P + S / 128 * T) * H);
  p.total = off;
  *out = p;
  return FP4_OK;
}

template <int MODE>
static int launch_few(FewArgs a, const FewPlan& p, int y_dtype, hipStream_t st) {
  static std::atomic<uint64_t> gu_raised{0}, dn_raised{0};
  FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_gateup_kernel<MODE>), kGuLds, gu_raised));
  const int ring = gu_ring<MODE>(a.S > 0), strips = a.I / 16, max_units = std::min(a.E, a.T * a.k) * strips;
  // a unit is split between waves (each a run of its pieces) until the units there may be fill the chip's waves
  a.k_split = 1;
  while (a.k_split < p.nw && max_units * a.k_split < kFewCus * p.nw) a.k_split *= 2;
  const int lds = gu_smem(a.T, a.E, a.k, a.H, MODE == FM_FP8, p.nw, ring, a.k_split > 1).total;
  const int per = p.nw / a.k_split, fit = kFewCus * std::max(1, std::min(2, kLds / (lds + 64)));
  int shared = 0;  // workgroups of the shared expert, by 1.5 times its share of the bytes: its waves stage all tokens' h
             // for each K step (shares of 1 / 1.5 / 2 in the header's graph replays: 16 tokens of NVFP4/NVFP4
             // 87.9 / 85.8 / 87.3 us, 7 of block FP8 98 / 93 / 94)
  double share = 0;
  if (a.S > 0) {
    const double sb = 1.5 * 2.0 * a.S, rb = (double)std::min(a.E, a.T * a.k) * 2 * a.I * (MODE == FM_FP8 ? 1.0 : 0.55);
    share = sb / (sb + rb);
    shared = std::max(1, std::min((a.S / 16 + per - 1) / per, (int)(fit * share)));
  }
  a.routed_wgs = std::max(1, std::min(fit - shared, (max_units + per - 1) / per));
  hipLaunchKernelGGL((few_gateup_kernel<MODE>), dim3((unsigned)(a.routed_wgs + shared)), dim3(64 * p.nw), (size_t)lds, st, a);
  FP4_CHECK(check_launch("few_gateup"));
  const size_t dn_lds = std::max(dn_smem(MODE, (a.I + 127) / 128, a.pass_pairs, a.seg_steps, p.dn_waves), a.S ? dn_smem_shared(a.T, p.dn_waves) : 0);
  const int64_t strips2 = a.H / 16;
  const int dn_fit = kFewCus * std::max(1, std::min(2, (int)(kLds / dn_lds)));
  shared = a.S > 0 ? std::max(1, (int)(dn_fit * share)) : 0;
  a.down_wgs = (int)std::min<int64_t>(dn_fit - shared, (strips2 * a.T * a.k + p.dn_waves - 1) / p.dn_waves);
  const dim3 grid((unsigned)(a.down_wgs + shared)), block(64 * p.dn_waves);
  FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_down_kernel<MODE>), kLds, dn_raised));
  hipLaunchKernelGGL(few_down_kernel<MODE>, grid, block, dn_lds, st, a);
  FP4_CHECK(check_launch("few_down"));
  const dim3 sum_grid(grid_1d((int64_t)a.T * (a.H / 4), 64));
  if (y_dtype == FP4_DT_F32) hipLaunchKernelGGL(few_sum_kernel<float>, sum_grid, dim3(64), 0, st, a);
  else hipLaunchKernelGGL(few_sum_kernel<uint16_t>, sum_grid, dim3(64), 0, st, a);
  return check_launch("few_sum");
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
  // a lane reads block scales as a pair of bytes (NVFP4), a byte (MXFP4) or a float (block FP8)
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
  a.pass_pairs = p.pass_pairs; a.seg_steps = p.seg_steps;
  a.list = reinterpret_cast<int32_t*>(b + p.list);
  a.passes = reinterpret_cast<DnPass*>(b + p.passes);
  a.sgate = reinterpret_cast<float*>(b + p.sgate);
  a.amax_part = reinterpret_cast<float*>(b + p.amax_part);
  a.h = reinterpret_cast<float*>(b + p.h);
  a.sh = reinterpret_cast<float*>(b + p.sh);
  a.d = reinterpret_cast<float*>(b + p.d);
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
