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

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"
#include "moe_internal.h"

namespace fp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kFewTokens = 16;  // columns of the MFMA tile
constexpr int kGuWaves = 8;     // most waves per workgroup of the gate_up kernel
constexpr int kDnWaves = 8;     // waves per workgroup of the down kernel, a strip of 16 outputs each
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
  int splits, shared_splits;  // down workgroups of a row group: of the routed experts, of the shared expert
  int pass_pairs, shared_pairs;  // pairs of an expert, tokens of the shared expert that the down kernel takes at once
  // workspace
  int32_t *list, *pairs;   // touched experts [1 + min(E, T k)] (count first); [.., 16] their pairs, then -1
  int32_t* done;           // [ceil(H / 128)] arrivals of the down kernel's splits
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

// A block: 16 weight rows (one strip) x one 128-wide K step, as a ring slot
// holds it: the rows' 16-byte chunks of codes XOR-swizzled by the row, then
// their block scales row by row.  gate_up's slots hold a gate and an up block:
// codes, codes, scales, scales.
template <int FMT>
struct Blk {
  static constexpr bool FP4 = FMT == FP4_FMT_NVFP4 || FMT == FP4_FMT_MXFP4;
  static constexpr int ROW = FP4 ? 64 : 128, CODES = 16 * ROW;  // code bytes of a row, of a block
  static constexpr int SROW = FMT == FP4_FMT_NVFP4 ? 8 : FMT == FP4_FMT_FP8_BLOCK ? 0 : 4;  // scale bytes of a row
  static constexpr int NC = CODES / 1024;  // DMA instructions of a block's codes
  static __device__ __forceinline__ int chunk(int c, int row) { return FP4 ? c ^ ((row >> 2) & 3) : c ^ (row >> 1); }
};
// bytes of a slot of `strips` blocks, and its DMA instructions
template <int FMT>
constexpr int slot_bytes(int strips) { return strips * (Blk<FMT>::CODES + 16 * Blk<FMT>::SROW); }
template <int FMT>
constexpr int slot_dmas(int strips) { return strips * Blk<FMT>::NC + (Blk<FMT>::SROW ? 1 : 0); }

// One or two strips' tensors (gate rows and the up rows `up` bytes behind).
template <int FMT>
struct Strip {
  __amdgpu_buffer_rsrc_t codes, scales;
  const uint8_t* srow;
  __device__ __forceinline__ void set(const uint8_t* c, const uint8_t* sc, uint32_t bytes, uint32_t sbytes) {
    codes = buffer_of(c, bytes);
    scales = buffer_of(sc, sbytes);
    srow = sc;
  }
};

// Loads K step kb of NS strips (the second cup / sup bytes behind the first)
// into `slot`.  Chunks and scales past a row's end read the row's start (they
// meet zeros of x or h).  Scale rows that are no multiple of 4 bytes (K not a
// multiple of 64 in NVFP4, of 128 in MXFP4) cannot be copied by DMA and go
// through registers.
template <int FMT, int NS>
__device__ __forceinline__ void load_slot(const Strip<FMT>& s, int kb, int rb, int rs, uint32_t cup, uint32_t sup, uint8_t* slot) {
  using B = Blk<FMT>;
  constexpr int CPR = B::ROW / 16, RPI = 64 / CPR;  // 16-byte chunks of a row, rows of an instruction
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int u = 0; u < NS; ++u)
#pragma unroll
    for (int j = 0; j < B::NC; ++j) {
      const int row = RPI * j + lane / CPR, at = B::ROW * kb + 16 * B::chunk(lane % CPR, row);
      dma_buffer(s.codes, (uint32_t)(row * rb + (at < rb ? at : 0)), u * cup, slot + u * B::CODES + 1024 * j);
    }
  if constexpr (B::SROW > 0) {
    uint8_t* to = slot + NS * B::CODES;
    if ((rs & 3) == 0) {
      constexpr int W = B::SROW / 4;  // dwords of a row's scales
      const int row = (lane / W) & 15, u = lane / (16 * W), at = B::SROW * kb + 4 * (lane % W);
      if (lane < NS * 16 * W) dma_buffer4(s.scales, (uint32_t)(row * rs + (at < rs ? at : 0)) + (uint32_t)u * sup, 0, to);
    } else {
      for (int i = lane; i < NS * 16 * B::SROW; i += 64) {
        const int row = (i / B::SROW) & 15, u = i / (16 * B::SROW), at = B::SROW * kb + i % B::SROW;
        to[i] = at < rs ? s.srow[(int64_t)u * sup + row * rs + at] : 0;
      }
    }
  }
}

// A lane's 32 values (K values [32 g, + 32) of the step, row r) of strip u.
template <int FMT>
struct WStep {
  u32x4 c[Blk<FMT>::FP4 ? 1 : 2];
  uint32_t s;
  template <int NS>
  __device__ __forceinline__ void read(const uint8_t* slot, int u, int g, int r) {
    using B = Blk<FMT>;
    const uint8_t* row = slot + u * B::CODES + B::ROW * r;
    if constexpr (B::FP4) {
      c[0] = ld16(row + 16 * B::chunk(g, r));
    } else {
      c[0] = ld16(row + 16 * B::chunk(2 * g, r));
      c[1] = ld16(row + 16 * B::chunk(2 * g + 1, r));
    }
    const uint8_t* sr = slot + NS * B::CODES + (16 * u + r) * B::SROW;
    if constexpr (FMT == FP4_FMT_NVFP4) s = *reinterpret_cast<const uint16_t*>(sr + 2 * g);
    else if constexpr (B::SROW > 0) s = sr[g];
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

// One wave selects the k experts of one token: ids to LDS in order, and the
// j-th selected value's key in lane j.  Lane l holds experts l + 64 i, sorted
// once by key (stably: the lower id first); then each of the k rounds takes the
// largest of the lanes' heads and pops it.
template <int PL>
__device__ __forceinline__ uint32_t select_topk(const float* logits, const float* bias, int E, int k, int* s_ids) {
  const int lane = threadIdx.x & 63;
  uint32_t key[PL];
  int id[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    id[i] = lane + 64 * i;
    key[i] = id[i] < E ? route_key(logits[id[i]] + (bias ? bias[id[i]] : 0.0f)) : 0u;
  }
#pragma unroll
  for (int pass = 0; pass < PL; ++pass)
#pragma unroll
    for (int i = pass & 1; i + 1 < PL; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const uint32_t ka = key[i], kb = key[i + 1];
      const int ia = id[i], ib = id[i + 1];
      key[i] = swap ? kb : ka;
      key[i + 1] = swap ? ka : kb;
      id[i] = swap ? ib : ia;
      id[i + 1] = swap ? ia : ib;
    }
  uint32_t mine = 0;
  int my_id = -1;
  for (int j = 0; j < k; ++j) {
    const uint32_t top = wave_umax(key[0]);
    if (top == 0) break;  // nothing selectable is left: ids -1
    uint64_t at = __ballot(key[0] == top);
    int win = __builtin_ctzll(at), e = __builtin_amdgcn_readlane(id[0], win);
    for (at &= at - 1; at; at &= at - 1) {  // equal values: the lowest id
      const int l = __builtin_ctzll(at), o = __builtin_amdgcn_readlane(id[0], l);
      if (o < e) { e = o; win = l; }
    }
    if (lane == j) { mine = top; my_id = e; }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i + 1 < PL; ++i) { key[i] = key[i + 1]; id[i] = id[i + 1]; }
      key[PL - 1] = 0u;
    }
  }
  if (lane < k) s_ids[lane] = my_id;
  return mine;
}

// ------------------------------------------------------------------ gate_up

struct GuSmem {
  int x, xf, ids, mask, place, list, scale, slot, red, ring, total;
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
  s.mask = s.ids + T * k * 4;
  s.place = s.mask + E * 4;
  s.list = s.place + (E + 1) / 2 * 4;
  s.scale = s.list + (D + 1) * 4;
  s.slot = s.scale + D * 4;
  s.red = (s.slot + D * kFewTokens + 15) / 16 * 16;
  s.ring = s.red + (split ? nw * 64 * 8 * 4 : 0);
  s.total = s.ring + nw * ring;
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
      for (int c = threadIdx.x; c < T * H / 32; c += (int)blockDim.x) {
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
      for (int w = 1; w < kGuWaves; ++w)
        if (w < (int)blockDim.x >> 6) m = fmaxf(m, tmp[w]);
      ts = (float)((double)m / kNvTensorDivisor);
    }
  }
  if constexpr (AF == FP4_FMT_NONE) {  // as it is, by DMA; the caller's barrier waits for it
    const auto xb = buffer_of(a.x, (uint32_t)(T * H * 2));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    for (int t = wave; t < T; t += (int)blockDim.x >> 6) {
      for (int c = 0; c < H / 8; c += 64)
        if (c + lane < H / 8) dma_buffer(xb, (uint32_t)(t * H * 2 + 16 * (c + lane)), 0, sx + t * (kp + 8) * 2 + 16 * c);
      if (H / 8 + lane < kp / 8) st16(sx + t * (kp + 8) * 2 + 16 * (H / 8 + lane), u32x4{0, 0, 0, 0});
    }
    return 1.0f;
  }
  const int per = kp / 32;
  for (int c = threadIdx.x; c < T * per; c += (int)blockDim.x) {
    const int t = c / per, q = c - t * per;
    float v[32];
    load_bf16x32(a.x + (int64_t)t * H + 32 * q, v);  // H is a multiple of 128 where x is quantized
    const float f = quantize32<AF>(v, ts);
    store_bf16x32(sx + (t * (kp + 8) + 32 * q) * 2, v);
    if (AF == FP4_FMT_FP8_ROW && (q & 3) == 0) xf[t * (kp / 128) + (q >> 2)] = f;
  }
  return ts;
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

// One wave's stream of gate_up units: in every round j < rounds it multiplies
// the K steps [lo, hi) of a unit's 16 gate rows and 16 up rows with all
// tokens' x~ (if j < mine) and hands the sums to finish(j, gate, up).
// strip(j, s) gives a round's weight rows, scales(j, ..) the first block scales
// of block FP8, started() runs once the first loads are on their way.  A ring
// of D slots; the next D - 1 are being loaded, over the rounds' borders.
template <int FMT, int D, typename SetStrip, typename Scales, typename Started, typename Finish>
__device__ __forceinline__ void gu_stream(int rounds, int mine, int lo, int hi, int K, int I, const uint8_t* sx, const float* xf, int xt, uint8_t* ring,
                                          SetStrip strip, Scales scales, Started started, Finish finish) {
  constexpr int SLOT = slot_bytes<FMT>(2), ND = slot_dmas<FMT>(2);
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, kp = (K + 127) / 128 * 128;
  const int rb = (int)code_row_bytes<FMT>(K), rs = (int)scale_row_bytes<FMT>(K);
  const uint32_t cup = (uint32_t)I * (uint32_t)rb, sup = (uint32_t)I * (uint32_t)rs;
  const uint8_t* xrow = sx + (xt * (kp + 8) + 32 * g) * 2;
  const bool any = mine > 0 && hi > lo, dma_scales = (rs & 3) == 0;
  Strip<FMT> st;
  int lj = 0, lb = lo;
  auto load_next = [&](int slot) __attribute__((always_inline)) {
    if (lb == lo) strip(min(lj, mine - 1), st);  // past the end the last unit again: every step issues as many loads
    load_slot<FMT, 2>(st, lb, rb, rs, cup, sup, ring + slot * SLOT);
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
      if (FMT == FP4_FMT_FP8_BLOCK) scales(j, fg, fu);
      for (int kb = lo; kb < hi; ++kb) {
        load_next(slot == 0 ? D - 1 : slot - 1);
        if (dma_scales) __builtin_amdgcn_s_waitcnt(vmcnt_only(ND * (D - 1)));
        else __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        const uint8_t* at = ring + slot * SLOT;
        slot = slot == D - 1 ? 0 : slot + 1;
        WStep<FMT> wg, wu;
        wg.template read<2>(at, 0, g, r);
        wu.template read<2>(at, 1, g, r);
        floatx4 pg = ag, pu = au;
        if (FMT == FP4_FMT_FP8_BLOCK) pg = pu = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8_t xv = __builtin_bit_cast(bf16x8_t, ld16(xrow + (128 * kb + 8 * q) * 2));
          pg = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(wg, q), xv, pg, 0, 0, 0);
          pu = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(wu, q), xv, pu, 0, 0, 0);
        }
        if (FMT == FP4_FMT_FP8_BLOCK) {
          const float f = xf[xt * (kp / 128) + kb], a = f * scalar_load(fg + kb), b = f * scalar_load(fu + kb);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            ag[q] = fmaf(pg[q], a, ag[q]);
            au[q] = fmaf(pu[q], b, au[q]);
          }
        } else {
          ag = pg;
          au = pu;
        }
      }
    }
    finish(j, ag, au);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // no DMA outlives the workgroup
}

// a wave's ring of D slots; the shared expert's larger MXFP8 slots share its bytes (two at least)
template <int MODE, int D>
__host__ __device__ constexpr int gu_ring(bool shared) {
  constexpr int own = D * slot_bytes<weight_fmt(MODE)>(2), sh = 2 * slot_bytes<FP4_FMT_MXFP8>(2);
  return shared && sh > own ? sh : own;
}
template <int MODE, int D>
constexpr int shared_depth() { return gu_ring<MODE, D>(true) / slot_bytes<FP4_FMT_MXFP8>(2); }

template <int MODE, int D>
__global__ void __launch_bounds__(64 * kGuWaves, 2) few_gateup_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ float tmp[kGuWaves];
  __shared__ uint32_t s_amax;
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
    prepare_x<FP4_FMT_MXFP8>(a, smem + sm.x, xf, tmp);
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
    gu_stream<FP4_FMT_MXFP8, shared_depth<MODE, D>()>(
        rounds, mine, lo, hi, H, S, smem + sm.x, xf, xt, ring,
        [&](int j, Strip<FP4_FMT_MXFP8>& st) __attribute__((always_inline)) {
          const int64_t row = 16 * (int64_t)(first + j * wgs * per);
          st.set(a.ws13 + row * H, a.ws13s + row * (H / 32), (uint32_t)(S + 16) * H, (uint32_t)(S + 16) * (H / 32));
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
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + sm.mask);    // tokens of an expert
  uint16_t* place = reinterpret_cast<uint16_t*>(smem + sm.place);  // of a touched expert in the list
  int* list = reinterpret_cast<int*>(smem + sm.list);
  float* scale = reinterpret_cast<float*>(smem + sm.scale);
  uint8_t* slots = smem + sm.slot;  // [listed expert][token]: the token's slot + 1
  if constexpr (AF == FP4_FMT_NONE) (void)prepare_x<AF>(a, smem + sm.x, xf, tmp);  // on its way while the tokens are routed
  for (int e = tid; e < a.E; e += th) mask[e] = 0;
  for (int i = tid; i < min(a.E, P) * kFewTokens / 4; i += th) reinterpret_cast<uint32_t*>(slots)[i] = 0;
  if (tid == 0) s_amax = 0;
  for (int t = wave; t < T; t += nw) {
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
  float xs = 1.0f;
  if constexpr (AF != FP4_FMT_NONE) xs = prepare_x<AF>(a, smem + sm.x, xf, tmp);
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // x by DMA: a barrier alone does not wait for it
  __syncthreads();
  for (int p = tid; p < P; p += th)
    if (ids[p] >= 0) atomicOr(&mask[ids[p]], 1u << (p / k));
  __syncthreads();
  // the touched experts by id: 64 to a ballot, every wave a run of them; the counts of the runs before come first
  const int runs = (a.E + 63) / 64;
  int before = 0;
  for (int c = 0; c < runs; ++c) {
    const int e = 64 * c + lane;
    const uint32_t m = e < a.E ? mask[e] & 0xFFFFu : 0u;
    const uint64_t on = __ballot(m != 0);
    if (m && c % nw == wave) {
      const int at = before + __popcll(on & ((1ull << lane) - 1));
      list[1 + at] = e;
      place[e] = (uint16_t)at;
    }
    before += __popcll(on);
  }
  const int nd = before;
  __syncthreads();
  for (int p = tid; p < P; p += th)
    if (ids[p] >= 0) slots[place[ids[p]] * kFewTokens + p / k] = (uint8_t)(p % k + 1);
  __syncthreads();
  if (blockIdx.x == 0) {  // for the down kernel
    for (int i = tid; i < (H + 127) / 128; i += th) a.done[i] = 0;
    if (a.ids_out)
      for (int p = tid; p < P; p += th) a.ids_out[p] = ids[p];
    if (tid == 0) a.list[0] = nd;
    for (int i = tid; i < nd; i += th) a.list[1 + i] = list[1 + i];
    for (int i = tid; i < nd; i += th) {
      int n = 0;
      for (int t = 0; t < T; ++t)
        if (const int j = slots[i * kFewTokens + t]) a.pairs[i * kFewTokens + n++] = t * k + j - 1;
      for (; n < kFewTokens; ++n) a.pairs[i * kFewTokens + n] = -1;
    }
  }

  const int I = a.I, strips = I / 16, units = nd * strips, base = blockIdx.x * per, first = base + wave / split, step = a.routed_wgs * per;
  const int64_t rb = code_row_bytes<WF>(H), rs = scale_row_bytes<WF>(H);
  const int NB = (H + 127) / 128, lo = ks * NB / split, hi = (ks + 1) * NB / split;
  float hmax = 0.0f;
  gu_stream<WF, D>(
      max(0, (units - base + step - 1) / step), max(0, (units - first + step - 1) / step), lo, hi, H, I, smem + sm.x, xf, xt, ring,
      [&](int j, Strip<WF>& st) __attribute__((always_inline)) {
        const int u = first + j * step, e = __builtin_amdgcn_readfirstlane(list[1 + u / strips]);
        const int64_t row = (int64_t)e * 2 * I + (u % strips) * 16;
        st.set(a.w13 + row * rb, static_cast<const uint8_t*>(a.w13s) + row * rs, (uint32_t)((I + 16) * rb), (uint32_t)((I + 16) * rs));
      },
      [&](int j, const float*& fg, const float*& fu) __attribute__((always_inline)) {
        const int u = first + j * step, e = __builtin_amdgcn_readfirstlane(list[1 + u / strips]), KB = H / 128;
        fg = static_cast<const float*>(a.w13s) + ((int64_t)e * (2 * I / 128) + (u % strips) / 8) * KB;
        fu = fg + (int64_t)(I / 128) * KB;
      },
      [&]() __attribute__((always_inline)) {
        if constexpr (WF == FP4_FMT_NVFP4) {
          for (int i = tid; i < nd; i += th) scale[i] = a.w13s2[list[1 + i]] * xs;
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
        const float s = WF == FP4_FMT_NVFP4 ? scale[ai] : 1.0f;
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

// LDS of the down kernel: the waves' rings, then h of two passes, then the
// waves' outputs (f32 [16 tokens][16]).
template <int FMT>
constexpr int dn_depth() { return Blk<FMT>::FP4 ? 8 : 4; }  // slots: 1 KB (E2M1) or 2 KB (E4M3) of codes
template <int FMT>
constexpr int dn_ring() { return dn_depth<FMT>() * slot_bytes<FMT>(1); }

// Waits until at most the loads of the last min(n, MOST) slots are on their way.
template <int MOST, int ND>
__device__ __forceinline__ void wait_vm(int n) {
  if (n >= MOST) __builtin_amdgcn_s_waitcnt(vmcnt_only(ND * MOST));
  else if constexpr (MOST > 0) wait_vm<MOST - 1, ND>(n);
}

// One workgroup's share of the down products: a row group (128 outputs, a
// strip of 16 a wave) times the passes of the experts [a0, a1) of a list; a
// pass is up to PP pairs of one expert, whose h rows (NT terms each) are
// copied into LDS one pass ahead and are the columns of the MFMA tile: row
// term * PP + pair.  expert(i) gives the expert's number and pair count,
// pair(i, q) its q-th pair, factor(p) what multiplies a pair's product, token(p)
// its row of y; blocks [lo, hi) of K.
template <int FMT, int NT, typename Expert, typename Pair, typename Factor, typename Token>
__device__ __forceinline__ void dn_stream(const uint8_t* w, const uint8_t* ws, const float* wf, int H, int K, int n0, int lo, int hi, int a0, int a1,
                                          const uint16_t* h, uint32_t h_bytes, int PP, uint8_t* smem, Expert expert, Pair pair, Factor factor, Token token) {
  constexpr int D = dn_depth<FMT>(), ND = slot_dmas<FMT>(1), SLOT = slot_bytes<FMT>(1);
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rb = (int)code_row_bytes<FMT>(K), rs = (int)scale_row_bytes<FMT>(K);
  uint8_t* ring = smem + wave * dn_ring<FMT>();
  uint8_t* hbuf = smem + kDnWaves * dn_ring<FMT>();
  const int RC = K / 8, rows = PP * NT, hbytes = rows * RC * 16;  // 16-byte chunks of a row of h
  float* yl = reinterpret_cast<float*>(hbuf + 2 * hbytes) + wave * 256;
#pragma unroll
  for (int q = 0; q < 4; ++q) yl[q * 64 + lane] = 0.0f;
  const bool strip_on = n0 < H, dma_scales = (rs & 3) == 0;  // H is a multiple of 32, not of 128: a wave may have no strip
  // load cursor of the weights: (expert, pass, block)
  Strip<FMT> st;
  int li = a0, lp = 0, lb = lo;
  auto set_strip = [&](int i) __attribute__((always_inline)) {
    const int64_t row = (int64_t)expert(i).x * H + n0;
    st.set(w + row * rb, ws + row * rs, 16 * rb, 16 * rs);
  };
  auto load_next = [&](int slot) __attribute__((always_inline)) {
    if (lb == lo) set_strip(min(li, a1 - 1));
    load_slot<FMT, 1>(st, lb, rb, rs, 0, 0, ring + slot * SLOT);
    if (++lb == hi) {
      lb = lo;
      lp += PP;
      if (li < a1 && lp >= expert(li).y) { lp = 0; ++li; }
    }
  };
  // h of the pass (expert i, pairs from p0) into buffer `buf`: chunk c of row q at place c + q (mod RC), so that the
  // 16 lanes that read one chunk of 16 rows hit different banks
  const uint32_t inv = 0xFFFFFFFFu / (uint32_t)RC + 1;  // s / RC = (s inv) >> 32 for s < 2^16
  const auto hb = buffer_of(h, h_bytes);
  auto load_h = [&](int i, int p0, int buf) __attribute__((always_inline)) {
    const int n = expert(i).y - p0;
    for (int s0 = wave * 64; s0 < rows * RC; s0 += kDnWaves * 64) {
      const uint32_t s = (uint32_t)min(s0 + lane, rows * RC - 1), row = __umulhi(s, inv), at = s - row * RC;
      const int rot = RC >= 16 ? (int)row : 0, c = (int)at - rot + ((int)at < rot ? RC : 0);
      const int t = (int)row / PP, q = (int)row - t * PP;
      const int p = pair(i, p0 + (q < n ? q : 0));  // rows past the pairs repeat the first; their columns are not kept
      if (s0 + lane < rows * RC) dma_buffer(hb, (uint32_t)(2 * ((p * NT + t) * K + 8 * c)), 0, hbuf + buf * hbytes + 16 * s0);
    }
  };
  if (a0 < a1) {
    load_h(a0, 0, 0);
    if (strip_on) {
#pragma unroll
      for (int d = 0; d < D - 1; ++d) load_next(d);
    }
  }
  int slot = 0, buf = 0;
  const int hr = r < rows ? r : 0, rot = RC >= 16 ? hr : 0;
  for (int i = a0, p0 = 0; i < a1;) {
    const int n = expert(i).y;
    int ni = i, np = p0 + PP;
    if (np >= n) { np = 0; ++ni; }
    // h of this pass was issued a pass ago (the first before the ring's first D - 1 blocks): only the weight blocks
    // issued since may still be on their way
    if (!strip_on || !dma_scales) __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    else wait_vm<D - 1, ND>(hi - lo);
    asm volatile("s_barrier" ::: "memory");  // h of this pass is there for every wave, and every wave is past the last one's
    if (ni < a1) load_h(ni, np, buf ^ 1);
    const uint8_t* hrow = hbuf + buf * hbytes + hr * RC * 16;
    floatx4 acc{0.f, 0.f, 0.f, 0.f};
    if (strip_on) {
      const float* fw = FMT == FP4_FMT_FP8_BLOCK ? wf + ((int64_t)expert(i).x * (H / 128) + n0 / 128) * (K / 128) : nullptr;
      for (int kb = lo; kb < hi; ++kb) {
        load_next(slot == 0 ? D - 1 : slot - 1);
        if (dma_scales) __builtin_amdgcn_s_waitcnt(vmcnt_only(ND * (D - 1)));
        else __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        WStep<FMT> v;
        v.template read<1>(ring + slot * SLOT, 0, g, r);
        slot = slot == D - 1 ? 0 : slot + 1;
        floatx4 pr = FMT == FP4_FMT_FP8_BLOCK ? floatx4{0.f, 0.f, 0.f, 0.f} : acc;
        const bool in = 128 * kb + 32 * g < K;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          int c = 16 * kb + 4 * g + q + rot;
          c -= c >= RC ? RC : 0;
          u32x4 hv = ld16(hrow + 16 * (in ? c : 0));
          if (!in) hv = u32x4{0, 0, 0, 0};
          pr = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wstep_frag<FMT>(v, q), __builtin_bit_cast(bf16x8_t, hv), pr, 0, 0, 0);
        }
        if (FMT == FP4_FMT_FP8_BLOCK) {
          const float f = scalar_load(fw + kb);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] = fmaf(pr[q], f, acc[q]);
        } else {
          acc = pr;
        }
      }
      // the terms' columns of a pair add up, then go to its token's outputs (a token is in an expert's list once)
      floatx4 v = acc;
      if constexpr (NT == 3) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += __shfl(acc[q], lane + PP) + __shfl(acc[q], lane + 2 * PP);
      }
      if (r < PP && p0 + r < n) {
        const float f = factor(i, p0 + r);
        floatx4* y = reinterpret_cast<floatx4*>(yl + token(pair(i, p0 + r)) * 16 + 4 * g);
        floatx4 o = *y;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = fmaf(v[q], f, o[q]);
        *y = o;
      }
    }
    buf ^= 1;
    i = ni;
    p0 = np;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // no DMA outlives the workgroup
}

// Grid: (row groups of 128 outputs, splits).  A split takes a run of the
// touched experts, or (the last shared_splits) a run of K of the shared
// expert, and leaves its sums in ypart; the last of a row group to arrive adds
// all splits up, in their order, and writes y.  Partial sums are stored and
// read at device scope, past the XCDs' L2s; no workgroup waits for another.
template <int MODE, typename OutT>
__global__ void __launch_bounds__(64 * kDnWaves, 2) few_down_kernel(FewArgs a) {
  constexpr int WF = weight_fmt(MODE), AF = act_fmt(MODE), NT = AF == FP4_FMT_NONE || AF == FP4_FMT_FP8_ROW ? 3 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int2 s_expert[kDnSeg];                 // this split's experts: number, pairs
  __shared__ int16_t s_pair[kDnSeg][kFewTokens];
  __shared__ float s_factor[kDnSeg][kFewTokens];    // routing weight times the tensor scales
  __shared__ int s_last;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = a.T, H = a.H, k = a.k, split = blockIdx.y, total = gridDim.y;
  const int n0 = blockIdx.x * 128 + wave * 16;
  const float* yl;
  if (split < a.splits) {
    const int nd = a.list[0], a0 = split * nd / a.splits, a1 = (split + 1) * nd / a.splits;
    for (int i = tid; i < (a1 - a0) * kFewTokens; i += 64 * kDnWaves) {
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
        a.w2, static_cast<const uint8_t*>(a.w2s), static_cast<const float*>(a.w2s), H, a.I, n0, 0, (a.I + 127) / 128, 0, a1 - a0,
        a.hb, (uint32_t)(T * k) * NT * a.I * 2, a.pass_pairs, smem,
        [&](int i) __attribute__((always_inline)) {
          return int2{__builtin_amdgcn_readfirstlane(s_expert[i].x), __builtin_amdgcn_readfirstlane(s_expert[i].y)};
        },
        [&](int i, int q) __attribute__((always_inline)) { return (int)s_pair[i][q]; },
        [&](int i, int q) __attribute__((always_inline)) { return s_factor[i][q]; },
        [&](int p) __attribute__((always_inline)) { return p / k; });
    yl = reinterpret_cast<const float*>(smem + kDnWaves * dn_ring<WF>() + 2 * a.pass_pairs * NT * a.I * 2);
  } else {
    const int S = a.S, NB = S / 128, sp = split - a.splits, PP = min(a.shared_pairs, T);
    if (tid < T) s_factor[0][tid] = a.sgate[tid];
    __syncthreads();
    dn_stream<FP4_FMT_MXFP8, 1>(
        a.ws2, a.ws2s, nullptr, H, S, n0, sp * NB / a.shared_splits, (sp + 1) * NB / a.shared_splits, 0, 1, a.shb, (uint32_t)(T * S * 2), PP, smem,
        [&](int) __attribute__((always_inline)) { return int2{0, T}; }, [](int, int q) __attribute__((always_inline)) { return q; },
        [&](int, int q) __attribute__((always_inline)) { return s_factor[0][q]; }, [](int p) __attribute__((always_inline)) { return p; });
    yl = reinterpret_cast<const float*>(smem + kDnWaves * dn_ring<FP4_FMT_MXFP8>() + 2 * PP * S * 2);
  }
  __syncthreads();
  // element q of this row group: token q / 128, output q % 128
  const int cols = min(128, H - (int)blockIdx.x * 128);
  auto own = [&](int q) __attribute__((always_inline)) { return yl[((q & 127) >> 4) * 256 + (q >> 7) * 16 + (q & 15)]; };
  auto store = [&](int q, float v) __attribute__((always_inline)) {
    OutT* y = static_cast<OutT*>(a.y) + (int64_t)(q >> 7) * H + blockIdx.x * 128 + (q & 127);
    if constexpr (sizeof(OutT) == 4) *y = v;
    else *y = __builtin_bit_cast(uint16_t, (__bf16)v);
  };
  if (total == 1) {
    for (int q = tid; q < T * 128; q += 64 * kDnWaves)
      if ((q & 127) < cols) store(q, own(q));
    return;
  }
  auto part = [&](int s, int q) __attribute__((always_inline)) { return a.ypart + ((int64_t)s * T + (q >> 7)) * H + blockIdx.x * 128 + (q & 127); };
  for (int q = tid; q < T * 128; q += 64 * kDnWaves)
    if ((q & 127) < cols) __hip_atomic_store(part(split, q), own(q), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __builtin_amdgcn_s_waitcnt(0);  // this thread's stores acknowledged
  __syncthreads();
  if (tid == 0) s_last = __hip_atomic_fetch_add(a.done + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
  __syncthreads();
  if (!s_last) return;
  for (int q = tid; q < T * 128; q += 64 * kDnWaves) {
    if ((q & 127) >= cols) continue;
    float v = 0.0f;
    for (int s0 = 0; s0 < total; s0 += 8) {
      float t[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) t[s] = __hip_atomic_load(part(min(s0 + s, total - 1), q), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int s = 0; s < 8; ++s) v += s0 + s < total ? t[s] : 0.0f;
    }
    store(q, v);
  }
}

// --------------------------------------------------------------------- host

struct FewPlan {
  int mode, splits, shared_splits, pass_pairs, shared_pairs;
  int nw, depth;  // gate_up: waves of a workgroup, slots of a wave's ring
  size_t wts, list, pairs, done, sgate, amax_part, h_ts, h, hb, sh, shb, ypart, total;
};

constexpr int kFewCus = 256;        // workgroups that a launch aims at: the card's compute units
constexpr int kLds = 160 * 1024;
constexpr int kGuLds = kLds - 64;   // dynamic LDS beside the gate_up kernel's static bytes
constexpr int kDnHBytes = 48 * 1024;  // LDS for h of two passes

template <int D>
static int ring_bytes(int mode, bool shared) {
  switch (mode) {
    case FM_NV: case FM_NVNV: return gu_ring<FM_NV, D>(shared);
    case FM_MX: case FM_MXMX: return gu_ring<FM_MX, D>(shared);
    default: return gu_ring<FM_FP8, D>(shared);
  }
}

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
  p.pass_pairs = (int)std::min<size_t>(std::min<size_t>(16 / nt, std::max<int64_t>(T, 1)), kDnHBytes / (4 * nt * I));
  p.shared_pairs = S ? (int)std::min<size_t>(8, kDnHBytes / (4 * S)) : 1;
  if (p.pass_pairs < 1 || p.shared_pairs < 1) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: intermediate width too large for the LDS");
  // down: splits of a row group, so that the launch has about a workgroup per compute unit
  const int64_t groups = (H + 127) / 128;
  p.shared_splits = S ? (int)std::max<size_t>(1, std::min<size_t>(S / 128, (S + 319) / 320)) : 0;
  p.splits = (int)std::max<int64_t>((D + kDnSeg - 1) / kDnSeg, std::min<int64_t>(D, std::max<int64_t>(1, kFewCus / groups - p.shared_splits)));
  p.splits = std::max(p.splits, 1);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  p.wts = take(4 * P);
  p.list = take(4 * (1 + D));
  p.pairs = take(4 * D * kFewTokens);
  p.done = take(4 * groups);
  p.sgate = take(4 * T);
  p.amax_part = take(4 * 2 * kFewCus);
  p.h_ts = take(4);
  p.h = take(L->a_fmt == FP4_FMT_NONE ? 0 : 4 * P * I);
  p.hb = take(2 * nt * P * I);
  p.sh = take(4 * T * S);
  p.shb = take(2 * T * S);
  p.ypart = take(4 * (size_t)(p.splits + p.shared_splits) * T * H);
  p.total = off;
  *out = p;
  return FP4_OK;
}

template <int MODE, int D>
static int launch_few(FewArgs a, const FewPlan& p, int y_dtype, hipStream_t st) {
  constexpr int AF = act_fmt(MODE), WF = weight_fmt(MODE), NT = AF == FP4_FMT_NONE || AF == FP4_FMT_FP8_ROW ? 3 : 1;
  static std::atomic<uint64_t> gu_raised{0}, dn32_raised{0}, dn16_raised{0};
  FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_gateup_kernel<MODE, D>), kGuLds, gu_raised));
  const int ring = gu_ring<MODE, D>(a.S > 0), strips = a.I / 16, max_units = std::min(a.E, a.T * a.k) * strips;
  // a unit is split between waves (each a run of K) until the units there may be fill the chip's waves
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
  const size_t routed_lds = kDnWaves * (dn_ring<WF>() + 1024) + 4 * (size_t)a.pass_pairs * NT * a.I;
  const size_t shared_lds = a.S ? kDnWaves * (dn_ring<FP4_FMT_MXFP8>() + 1024) + 4 * (size_t)std::min(a.shared_pairs, a.T) * a.S : 0;
  constexpr int dn_static = kDnSeg * (8 + kFewTokens * 6) + 64;
  const size_t dn_lds = std::max(routed_lds, shared_lds);
  if (dn_lds + dn_static > kLds) return fail(FP4_ERR_UNSUPPORTED, "few-token forward: down kernel needs %zu bytes of LDS", dn_lds);
  const dim3 grid((unsigned)((a.H + 127) / 128), (unsigned)(a.splits + a.shared_splits)), block(64 * kDnWaves);
  if (y_dtype == FP4_DT_F32) {
    FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_down_kernel<MODE, float>), kLds - dn_static, dn32_raised));
    hipLaunchKernelGGL((few_down_kernel<MODE, float>), grid, block, dn_lds, st, a);
  } else {
    FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(&few_down_kernel<MODE, uint16_t>), kLds - dn_static, dn16_raised));
    hipLaunchKernelGGL((few_down_kernel<MODE, uint16_t>), grid, block, dn_lds, st, a);
  }
  return check_launch("few_down");
}

template <int MODE>
static int launch_few(const FewArgs& a, const FewPlan& p, int y_dtype, hipStream_t st) {
  if (p.depth == 4) return launch_few<MODE, 4>(a, p, y_dtype, st);
  return p.depth == 3 ? launch_few<MODE, 3>(a, p, y_dtype, st) : launch_few<MODE, 2>(a, p, y_dtype, st);
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
  a.splits = p.splits; a.shared_splits = p.shared_splits; a.pass_pairs = p.pass_pairs; a.shared_pairs = p.shared_pairs;
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
