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
#include <atomic>
#include <cmath>
#include <type_traits>

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
  int each;            // steps of a workgroup
  float* parts;        // [splits][batch][M][O], where several workgroups share a tile's steps
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
        v -= __uint_as_float(top);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TERMS; ++t) st16(out + t * rows * ld + row * ld + c, u32x4{d[t][0], d[t][1], d[t][2], d[t][3]});
}

// The float that a block's scale byte stands for as decode2 takes it: MXFP4's
// conversion reads the exponent byte alone (0 is 2^-127, 255 NaN); `pow2` is the power
// of two of the NVFP4 tensor scale.
template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t byte, float pow2) {
  if constexpr (FMT == FP4_FMT_MXFP4) return __uint_as_float(byte << 23);
  else return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0) * pow2;
}
// The codes of byte I of a dword, scaled, as two bf16 values, exactly.
template <int FMT, int I>
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale) {
  if constexpr (FMT == FP4_FMT_MXFP4) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
  } else {
    const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, I);
    const bf16x2_t p{(__bf16)(v.x * scale), (__bf16)(v.y * scale)};
    return __builtin_bit_cast(uint32_t, p);
  }
}

// A tensor scale S as pow2 mant: the power of two goes into the weights (which stay
// bf16's normal numbers), the rest, 1 or more, is applied to the sums, which are
// no larger than the results then.  (Below 2^-100 mant is less than 1, and the results are
// far below f32's end.)  S = 0 makes weights of 0, so that no sum of large x is infinite
// before it is multiplied by 0.
__device__ __forceinline__ void split_scale(float S, float& pow2, float& mant) {
  const int e = min(100, max(-100, __builtin_amdgcn_frexp_expf(S) - 1));
  pow2 = S == 0.0f ? 0.0f : ldexpf(1.0f, e);
  mant = ldexpf(S, -e);
}

__device__ __forceinline__ bf16x8_t as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8_t, v); }

// ------------------------------------------------------------ few rows

constexpr int kFewK = 256;   // a wave's step: 128 bytes of codes of each of 16 rows of W
constexpr int kRing = 4;     // steps on their way to a wave (2, 3 and 6 measured the same)
constexpr int kSlot = 2304;  // bytes of a step: 2 KB of codes, scales
constexpr int kDirectRows = 4;  // up to these x's fragments come straight from memory: 1 x 2560 x 2560 5.3 us (6.3 by DMA), 16 x 131072 x 2560 42.5 (41.0)
// Waves that multiply: seven and the adding one have 256 registers each, eight and it 168.
constexpr int few_waves(int ms, int u, int terms) { return ms * u * terms > 2 ? 7 : 8; }
constexpr int few_per_simd(int ms, int u, int terms) { return ms * u * terms == 2 ? 4 : ms * u * terms == 1 ? 6 : ms * u * terms == 3 ? 3 : 2; }

struct Fp4FewArgs {
  const void* x;       // [batch][M][K]
  const uint8_t* w;    // [batch][N][K / 2]
  const uint8_t* ws;
  const float* ts;
  void* y;             // [batch][M][N]
  int64_t M, N;
  int K, y_f32;
};

// Eight values of x as TERMS bf16 fragments (f32: three, whose sum they are; see fp4_rows_kernel), zeros where not `ok`.
template <int TERMS>
struct XPiece {
  u32x4 v[TERMS == 3 ? 2 : 1];
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    if constexpr (TERMS == 1) {
      v[0] = ld16(static_cast<const uint16_t*>(x) + at);
    } else {
      v[0] = ld16(static_cast<const float*>(x) + at);
      v[1] = ld16(static_cast<const float*>(x) + at + 4);
    }
  }
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (int i = 0; i < (TERMS == 3 ? 2 : 1); ++i) asm volatile("" : "+v"(v[i]));
  }
  __device__ __forceinline__ void terms(bool ok, bf16x8_t (&f)[TERMS]) const {
    if constexpr (TERMS == 1) {
      f[0] = as_bf16x8(ok ? v[0] : u32x4{0, 0, 0, 0});
    } else {
      u32x4 d[3];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float a = ok ? __uint_as_float(v[p >> 1][2 * (p & 1)]) : 0.0f, b = ok ? __uint_as_float(v[p >> 1][2 * (p & 1) + 1]) : 0.0f;
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const uint32_t ta = __float_as_uint(a) & 0xFFFF0000u, tb = __float_as_uint(b) & 0xFFFF0000u;
          d[t][p] = __builtin_amdgcn_perm(tb, ta, 0x07060302);  // the upper halves
          a -= __uint_as_float(ta);
          b -= __uint_as_float(tb);
        }
      }
#pragma unroll
      for (int t = 0; t < 3; ++t) f[t] = as_bf16x8(d[t]);
    }
  }
};

// 16 MS rows of x: a workgroup walks over strips of 16 outputs; wave w takes the steps
// w, w + waves, ... of K (U at most) of every strip.  Its share of x is loaded once
// and stays in registers as MFMA fragments; its share of W streams through a ring of
// steps in LDS that belongs to the wave alone (DMA), is decoded in registers and goes
// into the MFMAs as their A operand.  A strip's partial sums meet in LDS.  Where rows
// of codes or scales are not whole pieces of DMA (DMA false), they are loaded
// straight into registers, without a step ahead.  Bound by W's bytes, or by latency
// where they are few: 16 x 131072 x 2560 MXFP4 in 39 us, 4.8 TB/s (the rings alone take
// 31); 1 x 2560 x 2560 NVFP4 in 5.6.  Strips in pairs or runs of neighbours took 43 to 45.
template <int FMT, int TERMS, int MS, int U, bool DMA>
__global__ void __launch_bounds__(64 * (few_waves(MS, U, TERMS) + 1), few_per_simd(MS, U, TERMS)) fp4_few_kernel(Fp4FewArgs a) {
  constexpr int SLOT = kSlot, RING = DMA ? kRing * SLOT : 8192, BLOCKS = FMT == FP4_FMT_NVFP4 ? 16 : 8;  // scales of a row and step
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (blockDim.x >> 6) - 1, g = lane >> 4, r = lane & 15;
  uint8_t* ring = few_lds + waves * (2 * MS * 1024) + wave * RING;  // W's steps; before them 8 KB of x
  const int64_t b = blockIdx.z, m0 = (int64_t)blockIdx.y * (16 * MS);
  const int KS = (a.K + kFewK - 1) / kFewK, strips = (int)((a.N + 15) >> 4), first = blockIdx.x, stride = gridDim.x;
  const int nu = max(0, (KS - wave + waves - 1) / waves), mine = (strips - first + stride - 1) / stride;
  const uint32_t wrow = (uint32_t)a.K / 2, srow = (uint32_t)a.K / (kFewK / BLOCKS);
  const uint8_t* wbase = a.w + b * a.N * wrow;
  const uint8_t* sbase = a.ws + b * a.N * srow;
  float pow2 = 1.0f, mant = 1.0f;
  if constexpr (FMT == FP4_FMT_NVFP4) split_scale(a.ts[b], pow2, mant);
  if (wave == waves) {  // the last wave adds up the others' sums of a strip while they are at the next one
    const bool vec = a.N % 4 == 0 && (uintptr_t)a.y % 16 == 0;
    const int m = lane >> 2, n = 4 * (lane & 3);
    for (int i = 0; i < mine; ++i) {
      asm volatile("s_barrier" ::: "memory");
      const float* part = reinterpret_cast<const float*>(few_lds) + (i & 1) * waves * (MS * 256);
      const int64_t n0 = (int64_t)(first + i * stride) * 16 + n;
#pragma unroll
      for (int s = 0; s < MS; ++s) {
        floatx4 v{0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < waves; ++w) v += *reinterpret_cast<const floatx4*>(part + (w * MS + s) * 256 + m * 16 + 4 * ((n >> 2) ^ ((m >> 1) & 3)));
        v *= mant;
        const int64_t row = m0 + 16 * s + m, at = (b * a.M + row) * a.N + n0;
        if (row >= a.M) continue;
        const bf16x2_t lo{(__bf16)v[0], (__bf16)v[1]}, hi{(__bf16)v[2], (__bf16)v[3]};
        const u32x2 h{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        if (vec && n0 < a.N) {
          if (a.y_f32) *reinterpret_cast<floatx4*>(static_cast<float*>(a.y) + at) = v;
          else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + at) = h;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (n0 + c < a.N) {
              if (a.y_f32) static_cast<float*>(a.y)[at + c] = v[c];
              else static_cast<uint16_t*>(a.y)[at + c] = (uint16_t)(h[c >> 1] >> (16 * (c & 1)));
            }
        }
      }
    }
    return;
  }

  // DMA of strip i's step u into a slot: row j of the strip at 128 j, its 16-byte chunks swizzled by the row so that
  // 16 rows' reads of a chunk touch all banks; then 16 rows of scales.  A lane's offsets are the same in every strip:
  // rows past the last one are left out by the buffer's bounds (their results are not stored), and what lies past the
  // end of a row is not used.
  constexpr int DW = BLOCKS / 4;  // dwords of scales of a row
  uint32_t at_code[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = 8 * j + (lane >> 3);
    at_code[j] = row * wrow + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const uint32_t at_scale = ((lane / DW) & 15) * srow + 4 * (lane % DW);
  int li = 0, lu = 0;  // the next step to load
  auto load_next = [&](int slot) __attribute__((always_inline)) {
    // past the end the last strip is loaded again, so that every step issues three instructions
    const int64_t n0 = (int64_t)(first + min(li, mine - 1) * stride) * 16;
    const int kb = wave + waves * lu, rows = (int)min((int64_t)16, a.N - n0);
    const auto codes = buffer_of(wbase + n0 * wrow, rows * wrow);
    const auto scales = buffer_of(sbase + n0 * srow, rows * srow);
#pragma unroll
    for (int j = 0; j < 2; ++j) dma_buffer(codes, at_code[j], 128 * kb, ring + SLOT * slot + 1024 * j);
    dma_buffer4(scales, at_scale, BLOCKS * kb, ring + SLOT * slot + 2048);
    if (++lu == nu) { lu = 0; ++li; }
  };
  bf16x8_t xf[U][2][4][MS][TERMS];
  if (nu > 0) {
    // 16 rows of x at a time, 512 bytes of each, come in by DMA (the ring is not in use yet): fragments straight from
    // memory would touch a row in every lane.  For a few rows those are fewer, and the same for many lanes.
    constexpr int XB = TERMS == 3 ? 4 : 2, PARTS = TERMS == 3 ? 2 : 1;
    const bool direct = a.M <= kDirectRows;
    if (DMA && direct) {
#pragma unroll
      for (int d = 0; d < kRing; ++d) load_next(d);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int s = 0; s < MS; ++s) {
        const int64_t m = b * a.M + min(m0 + 16 * s, a.M - 1);  // blocks past the end: the last row, not stored
        const int last = (int)max((int64_t)0, min((int64_t)15, a.M - 1 - m0 - 16 * s));
        const int k0 = kFewK * (wave + waves * u);
        XPiece<TERMS> piece[2][4];
        if (direct) {
          const int64_t row = (m + min(r, last)) * a.K;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int k = k0 + 128 * h + 32 * g + 8 * q;
              piece[h][q].load(a.x, row + (k < a.K ? k : 0));
            }
        } else {
          const uint32_t bytes = (uint32_t)a.K * XB;
          const auto rows = buffer_of(static_cast<const uint8_t*>(a.x) + m * bytes, (uint32_t)(last + 1) * bytes);
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const int at = k0 * XB + 512 * p;  // of the row's bytes
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int row = 2 * j + (lane >> 5), from = at + 16 * ((lane & 31) ^ row);
              dma_buffer(rows, (uint32_t)min(row, last) * bytes + ((uint32_t)from < bytes ? from : 0), 0, ring + 1024 * j);
            }
            __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
            asm volatile("" ::: "memory");
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (TERMS == 3 && h != p) continue;
                const int n = TERMS == 3 ? 8 * g + 2 * q : 16 * h + 4 * g + q;
                piece[h][q].v[0] = ld16(ring + r * 512 + 16 * (n ^ r));
                if constexpr (TERMS == 3) piece[h][q].v[1] = ld16(ring + r * 512 + 16 * ((n + 1) ^ r));
              }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (TERMS == 1 || h == p) piece[h][q].arrived();
            __builtin_amdgcn_s_waitcnt(lgkmcnt0());  // read: the place may be filled again
            asm volatile("" ::: "memory");
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) piece[h][q].terms(k0 + 128 * h + 32 * g + 8 * q < a.K, xf[u][h][q][s]);
        if constexpr (DMA && TERMS == 3) {
          // f32's terms stay as they are now: split anew in every strip, as the compiler has it otherwise, they do not fit
          // the registers (1 x 2560 x 2560 37 us, 8.3 so; 16 x 131072 x 2560 104 and 70)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int t = 0; t < TERMS; ++t) asm volatile("" : "+v"(xf[u][h][q][s][t]));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    if (DMA && !direct) {
#pragma unroll
      for (int d = 0; d < kRing; ++d) load_next(d);
    }
  }
  int slot = 0;
  for (int i = 0; i < mine; ++i) {
    const int64_t n0 = (int64_t)(first + i * stride) * 16;
    constexpr int CH = MS * TERMS >= 2 ? 2 : 4;  // independent sums: an MFMA waits for the one before in its own
    floatx4 acc[CH][MS];
#pragma unroll
    for (int h = 0; h < CH; ++h)
#pragma unroll
      for (int s = 0; s < MS; ++s) acc[h][s] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < nu) {
        const int kb = wave + waves * u;
        u32x4 code[2];
        uint32_t scale[2];  // NVFP4: the chunk's two blocks' bytes
        if constexpr (DMA) {
          __builtin_amdgcn_s_waitcnt(vmcnt_only(3 * (kRing - 1)));  // this step has arrived; the later ones may be on their way
          asm volatile("" ::: "memory");
          const uint8_t* from = ring + SLOT * slot;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int chunk = 4 * h + g;
            code[h] = ld16(from + r * 128 + 16 * (chunk ^ (r >> 1)));
            if constexpr (FMT == FP4_FMT_NVFP4) scale[h] = *reinterpret_cast<const uint16_t*>(from + 2048 + r * BLOCKS + 2 * chunk);
            else scale[h] = from[2048 + r * BLOCKS + chunk];
            asm volatile("" : "+v"(code[h]), "+v"(scale[h]));
          }
          __builtin_amdgcn_s_waitcnt(lgkmcnt0());  // read: the slot may be filled again
          asm volatile("" ::: "memory");
          load_next(slot);
          slot = slot == kRing - 1 ? 0 : slot + 1;
        } else {
          const int64_t n = min(n0 + r, a.N - 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = kFewK * kb + 32 * (4 * h + g), k1 = k < a.K ? k : 0, k2 = k + 16 < a.K ? k + 16 : 0;
            const uint8_t *c = wbase + n * wrow, *sc = sbase + n * srow;
            const u32x2 lo = *reinterpret_cast<const u32x2*>(c + k1 / 2), hi = *reinterpret_cast<const u32x2*>(c + k2 / 2);
            code[h] = u32x4{lo.x, lo.y, k + 16 < a.K ? hi.x : 0, k + 16 < a.K ? hi.y : 0};
            if constexpr (FMT == FP4_FMT_NVFP4) scale[h] = sc[k1 / 16] | (k + 16 < a.K ? (uint32_t)sc[k2 / 16] << 8 : 0);
            else scale[h] = sc[k1 / 32];
          }
        }
        if (kFewK * (kb + 1) > a.K) {  // what is past the end of the rows counts 0
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (kFewK * kb + 32 * (4 * h + g) >= a.K) {
              code[h] = u32x4{0, 0, 0, 0};
              scale[h] = 0;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float s = block_scale<FMT>(FMT == FP4_FMT_NVFP4 ? (scale[h] >> (8 * (q >> 1))) & 0xFF : scale[h], pow2);
            const uint32_t d = code[h][q];
            const bf16x8_t wf = as_bf16x8(u32x4{decode2<FMT, 0>(d, s), decode2<FMT, 1>(d, s), decode2<FMT, 2>(d, s), decode2<FMT, 3>(d, s)});
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
              for (int m = 0; m < MS; ++m) acc[q % CH][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[u][h][q][m][t], acc[q % CH][m], 0, 0, 0);
          }
      }
    }
    // [half][wave][16 MS rows][16 outputs], 16-byte pieces swizzled by the row; a half is written again two strips
    // later, when the adding wave has met the barrier after reading it
    float* part = reinterpret_cast<float*>(few_lds) + (i & 1) * waves * (MS * 256);
#pragma unroll
    for (int s = 0; s < MS; ++s) {
      floatx4 v = acc[0][s] + acc[1][s];
      if constexpr (CH == 4) v += acc[2][s] + acc[3][s];
      *reinterpret_cast<floatx4*>(part + (wave * MS + s) * 256 + r * 16 + 4 * (g ^ ((r >> 1) & 3))) = v;
    }
    __builtin_amdgcn_s_waitcnt(lgkmcnt0());
    asm volatile("s_barrier" ::: "memory");
  }
  if constexpr (DMA) __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // no DMA outlives the workgroup
}

// ------------------------------------------------------------ tiles

// NS fragments of 16 columns by 32 rows from a tile that lies row by row (ROW bytes each): the transposing reads, in one
// block with their wait, because the compiler lets such a read wait for all DMA that is on its way.
template <int NS, int ROW>
__device__ __forceinline__ void read_turned(const uint8_t* p, bf16x8_t (&f)[NS]) {
  const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
  u32x2 v[2 * NS];
  if constexpr (NS == 2) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n"
        "ds_read_b64_tr_b16 %1, %4 offset:%5\n"
        "ds_read_b64_tr_b16 %2, %4 offset:32\n"
        "ds_read_b64_tr_b16 %3, %4 offset:%6\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at), "n"(4 * ROW), "n"(4 * ROW + 32));
  } else {
    static_assert(NS == 4, "two or four fragments");
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n"
        "ds_read_b64_tr_b16 %1, %8 offset:%9\n"
        "ds_read_b64_tr_b16 %2, %8 offset:32\n"
        "ds_read_b64_tr_b16 %3, %8 offset:%10\n"
        "ds_read_b64_tr_b16 %4, %8 offset:64\n"
        "ds_read_b64_tr_b16 %5, %8 offset:%11\n"
        "ds_read_b64_tr_b16 %6, %8 offset:96\n"
        "ds_read_b64_tr_b16 %7, %8 offset:%12\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at), "n"(4 * ROW), "n"(4 * ROW + 32), "n"(4 * ROW + 64), "n"(4 * ROW + 96));
  }
#pragma unroll
  for (int s = 0; s < NS; ++s) f[s] = as_bf16x8(u32x4{v[2 * s].x, v[2 * s].y, v[2 * s + 1].x, v[2 * s + 1].y});
}

// Tile of BM rows by BO outputs per workgroup of WM x WN waves, each owning 16 MS
// rows and 16 NS outputs.  Steps of 64 products: x's part comes by DMA, the
// weights' codes through registers, decoded on their way to LDS, both into the
// half of the LDS that the step before last used.  Weights are the A operand of
// the MFMA, so that a lane's four sums are four consecutive outputs of one row.
// The gradient sums over W's rows: its tile lies in LDS as W does and is turned by
// the transposing reads.  Large products are bound by how far the CU's parts overlap:
// at 8192 x 10240 x 2560 (NVFP4, 256 x 256) 390 us, 1.1 PFLOP/s, where the MFMAs alone
// take 247, no loads of codes 340 and no decoding and writing of them 375; small ones
// by a step's latency, 0.4 to 0.5 us.
template <int R, int WM, int WN, int MS, int NS, bool GRAD>
struct Fp4Tile {
  static constexpr int WAVES = WM * WN, TH = 64 * WAVES, BM = 16 * MS * WM, BO = 16 * NS * WN;
  static constexpr int XB = BM * 128;                              // bytes of x a step
  static constexpr int WROW = GRAD ? BO * 2 + 32 : 128;            // bytes of a row of the weight tile
  static constexpr int WB = GRAD ? 64 * WROW : BO * 128;
  static constexpr int CPT = BO * 4 / TH;                          // blocks of 16 codes a thread decodes a step
  static constexpr int XD = BM / 8 < WAVES ? 1 : BM / 8 / WAVES;   // DMA instructions of a wave a step
  static constexpr int YROW = BO * 2 + 16;                         // bytes of a row of bf16 results on their way out
  static constexpr int LDS = R * XB + 2 * WB > BM * YROW ? R * XB + 2 * WB : BM * YROW;
  static_assert(CPT == 1 || CPT == 2, "a thread's codes");
  static_assert((BO * 4) % TH == 0 && ((BM / 8) % WAVES == 0 || WAVES % (BM / 8) == 0), "whole chunks");
  static_assert(R == 2 || R == 4, "the steps that the loop has written out");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <int FMT, bool GRAD, int TERMS, bool WIDE, int R, int WM, int WN, int MS, int NS>
__global__ void __launch_bounds__(64 * WM * WN, 2) fp4_tile_kernel(Fp4MatmulArgs a, int mt, int ot) {
  using C = Fp4Tile<R, WM, WN, MS, NS, GRAD>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, r = lane & 15;
  const int wm = wave / WN, wn = wave % WN;
  // workgroups b, b + 8, ... run on one XCD: give it consecutive tiles
  const int tiles = mt * ot, per = (tiles + 7) / 8;
  const int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (t >= tiles) return;
  const int grp = t / (8 * ot), in = t - grp * 8 * ot, rows = min(8, mt - grp * 8);
  const int64_t m0 = (int64_t)(grp * 8 + in % rows) * C::BM, o0 = (int64_t)(in / rows) * C::BO, b = blockIdx.z;
  const uint8_t* w = a.w + b * a.N * (a.K / 2);
  const uint8_t* ws = a.ws + b * a.N * (a.K / (FMT == FP4_FMT_NVFP4 ? 16 : 32));
  float pow2 = 1.0f, mant = 1.0f;
  if constexpr (FMT == FP4_FMT_NVFP4) split_scale(a.ts[b], pow2, mant);

  // x rows past the end repeat the last one; their results are not stored
  const int mlast = (int)min((int64_t)C::BM - 1, a.M - 1 - m0);
  uint32_t xoff[C::XD];
#pragma unroll
  for (int j = 0; j < C::XD; ++j) {
    const int row = 8 * ((wave * C::XD + j) % (C::BM / 8)) + (lane >> 3);
    xoff[j] = (uint32_t)min(row, mlast) * (uint32_t)(a.ld * 2) + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const uint16_t* xbase = a.x + (b * a.M + m0) * a.ld;
  const int first = blockIdx.y * a.each, last = min(a.steps, first + a.each) - 1;  // this workgroup's steps
  auto load_x = [&](int step, int term, int slot) __attribute__((always_inline)) {
    const auto buf = buffer_of(xbase + term * a.term, (uint32_t)(mlast + 1) * (uint32_t)(a.ld * 2));
#pragma unroll
    for (int j = 0; j < C::XD; ++j) dma_buffer(buf, xoff[j], 128 * step, lds + slot * C::XB + ((wave * C::XD + j) % (C::BM / 8)) * 1024);
  };
  // this thread's blocks of 16 codes: consecutive ones of one row of the weight tile
  constexpr int PER_ROW = GRAD ? C::BO / 16 : 4, CPT = C::CPT;
  const int trow = tid * CPT / PER_ROW, tblk = tid * CPT % PER_ROW;
  // Steps' codes and scales as they were loaded, one load each (8192 x 10240 x 2560: 400 us; 436 with two loads of codes
  // and two of scales, whose lines the L1 then passes twice as often), scales byte by byte where pairs are not aligned.
  // The large tiles (R = 2) load two steps' codes at a time, which lie in the same lines (390 us).
  constexpr int SB = FMT == FP4_FMT_NVFP4 ? CPT : (CPT + 1) / 2, SL = WIDE ? 1 : SB;  // bytes of scales, loads of them
  constexpr int CR = R == 2 ? 4 : R;  // steps whose codes are held or on their way
  uint32_t code[CR][2 * CPT], scale[CR][SL];
  const uint32_t wrow = (uint32_t)(a.K / 2), srow = (uint32_t)(a.K / (FMT == FP4_FMT_NVFP4 ? 16 : 32));  // bytes of a row
  const uint32_t at_code = trow * wrow + tblk * 8, at_scale = trow * srow + (FMT == FP4_FMT_NVFP4 ? tblk : tblk >> 1);
  const int blocks = (int)min((int64_t)1 << 30, a.K / 16 - (GRAD ? o0 / 16 : 0)) - tblk;  // of a row from this thread's first on
  auto load_w = [&](int step, int set) __attribute__((always_inline)) {
    // rows past the last one are left out by the buffers' bounds; blocks past a row's end are others, or left out
    const int64_t first_row = GRAD ? (int64_t)step * kBK : o0;
    const uint32_t rows = (uint32_t)min((int64_t)(GRAD ? kBK : C::BO), a.N - first_row);
    const uint32_t cs = GRAD ? (uint32_t)(o0 / 2) : 0, ss = GRAD ? (uint32_t)(o0 / (FMT == FP4_FMT_NVFP4 ? 16 : 32)) : 0;  // where the tile starts in a row
    const auto wb = buffer_of(w + first_row * wrow + cs, rows * wrow - cs);
    const auto sb = buffer_of(ws + first_row * srow + ss, rows * srow - ss);
    const uint32_t cat = GRAD ? 0 : step * 32, sat = GRAD ? 0 : step * (FMT == FP4_FMT_NVFP4 ? 4 : 2);
    if constexpr (CPT == 1) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(wb, at_code, cat, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) code[set][i] = v[i];
    } else {
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(wb, at_code, cat, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) code[set][i] = v[i];
    }
    if constexpr (SB / SL == 2) scale[set][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(sb, at_scale, sat, 0);
    else
#pragma unroll
      for (int i = 0; i < SL; ++i) scale[set][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sb, at_scale + i, sat, 0);
  };
  uint8_t* wlds = lds + R * C::XB;
  // The `part`-th of 2 CPT parts of the decoding: 8 codes, one 16-byte piece of the tile.
  float sc = 0.0f;
  uint32_t ok = 0;
  auto decode_w = [&](int step, int set, int part, int half) __attribute__((always_inline)) {
    const int c = part >> 1, h = part & 1;
    // what is past the end counts 0 (an infinity or NaN there would reach sums whose x is 0)
    if (h == 0) {
      ok = (GRAD ? 0 : 4 * step) + c < blocks ? 0xFFFFFFFFu : 0;
      const int i = FMT == FP4_FMT_NVFP4 ? c : c >> 1;  // its byte of the scales
      sc = block_scale<FMT>((SL == SB ? scale[set][SL == SB ? i : 0] : scale[set][0] >> 8 * i & 255) & ok, pow2);
    }
    const uint32_t d = code[set][2 * c + h] & ok;
    const int piece = 2 * (tblk + c) + h;
    uint8_t* to = wlds + half * C::WB + trow * C::WROW + 16 * (GRAD ? piece : piece ^ ((trow >> 1) & 7));
    st16(to, u32x4{decode2<FMT, 0>(d, sc), decode2<FMT, 1>(d, sc), decode2<FMT, 2>(d, sc), decode2<FMT, 3>(d, sc)});
  };
  // The weights' fragments of half a step.
  auto read_w = [&](int half, int j, bf16x8_t (&wf)[NS]) __attribute__((always_inline)) {
    const uint8_t* from = wlds + half * C::WB;
    if constexpr (GRAD) {
      // lane (g, r) names 4 values of row 32 j + 8 g + r / 4 and gets column r of the rows 32 j + 8 g .. + 3 (then + 4 .. + 7)
      read_turned<NS, C::WROW>(from + (32 * j + 8 * g + (r >> 2)) * C::WROW + (wn * 16 * NS + 4 * (r & 3)) * 2, wf);
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int row = wn * 16 * NS + 16 * s + r;
        wf[s] = as_bf16x8(ld16(from + row * 128 + 16 * ((4 * j + g) ^ ((row >> 1) & 7))));
      }
    }
  };
  floatx4 acc[MS][NS];
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[i][s] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int frag = r * 128 + 16 * (g ^ ((r >> 1) & 7));  // rows 16 apart lie alike
  int slot = 0;                                   // of this term's x
  int lstep = first, lterm = 0, lslot = 0;        // the next x to load
  auto load_next_x = [&]() __attribute__((always_inline)) {
    load_x(min(lstep, last), lterm, lslot);  // past the end the last step again
    lslot = lslot == R - 1 ? 0 : lslot + 1;
    if (++lterm == TERMS) { lterm = 0; ++lstep; }
  };
  // One step's products of one term of x, and on the way later steps' x and weights.  P: the set of the step's codes.
  auto body = [&](int step, auto P_, auto TERM_) __attribute__((always_inline)) {
    constexpr int P = decltype(P_)::value, TERM = decltype(TERM_)::value, NEXT = (P + 1) % CR;
    const int half = (step - first) & 1;
    // This term's x has arrived and its weights are written; what was asked for after that x may still be on its
    // way: its DMA, and of a step's codes and scales two loads at least (none is dropped, since all are used at the
    // end, and none passes a barrier).
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0((R - 2) * (C::XD + (TERMS == 1 ? 2 : 0))));
    asm volatile("s_barrier" ::: "memory");
    if (TERM == 0) {
      if constexpr (CR == R) {
        load_w(min(step + R, last), P);
      } else if constexpr (P & 1) {
        load_w(min(step + CR - 1, last), P - 1);
        load_w(min(step + CR, last), P);
      }
    }
    load_next_x();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* xr = lds + slot * C::XB + wm * (16 * MS * 128);
    bf16x8_t wf[2][NS], xf[3];
    auto read_x = [&](int i) __attribute__((always_inline)) { xf[i % 3] = as_bf16x8(ld16(xr + 2048 * (i % MS) + (frag ^ (64 * (i / MS))))); };
    read_w(half, 0, wf[0]);
    read_x(0);
    read_x(1);
    // The order is pinned: fragments are read two groups of MFMAs ahead, and the next
    // step's weights decoded between the MFMAs.
#pragma unroll
    for (int i = 0; i < 2 * MS; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i + 2 < 2 * MS) read_x(i + 2);
      if (i == MS - 1) read_w(half, 1, wf[1]);
      if (TERM == 0) {
#pragma unroll
        for (int part = 0; part < 2 * CPT; ++part)
          if (i == (part * 2 * MS) / (2 * CPT)) decode_w(min(step + 1, last), NEXT, part, half ^ 1);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) acc[i % MS][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i / MS][s], xf[i % 3], acc[i % MS][s], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    slot = slot == R - 1 ? 0 : slot + 1;
  };
  auto step_of = [&](int step, auto P_) __attribute__((always_inline)) {
    body(step, P_, std::integral_constant<int, 0>());
    if constexpr (TERMS == 3) {
      body(step, P_, std::integral_constant<int, 1>());
      body(step, P_, std::integral_constant<int, 2>());
    }
  };
  load_w(first, 0);
#pragma unroll
  for (int i = 0; i < R - 1; ++i) {  // in groups as the steps', which the waits count on
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    load_w(min(first + 1 + i, last), i + 1);
    load_next_x();
  }
  if constexpr (CR != R) {
    load_w(min(first + 2, last), 2);
    load_w(min(first + 3, last), 3);
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int part = 0; part < 2 * CPT; ++part) decode_w(first, 0, part, 0);
  for (int step = first; step <= last; step += CR) {
    step_of(step, std::integral_constant<int, 0>());
    if (step + 1 <= last) step_of(step + 1, std::integral_constant<int, 1>());
    if constexpr (CR >= 4) {
      if (step + 2 <= last) step_of(step + 2, std::integral_constant<int, 2>());
      if (step + 3 <= last) step_of(step + 3, std::integral_constant<int, 3>());
    }
  }
#pragma unroll
  for (int i = 0; i < CR; ++i)
#pragma unroll
    for (int c = 0; c < 2 * CPT; ++c) asm volatile("" ::"v"(code[i][c]), "v"(scale[i][c % SL]));
  __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0(0));  // no DMA outlives the workgroup
  if (a.y_f32 || a.parts) {
    const bool part = a.parts != nullptr;  // sums of some of the steps: joined, and scaled, by fp4_join_kernel
    if (part) mant = 1.0f;
    float* y = (part ? a.parts + (int64_t)blockIdx.y * gridDim.z * a.M * a.O : static_cast<float*>(a.y)) + (b * a.M + m0) * a.O + o0;
    const bool vec = a.O % 4 == 0 && (part || (uintptr_t)a.y % 16 == 0);
#pragma unroll
    for (int q = 0; q < MS; ++q) {
      const int m = wm * 16 * MS + 16 * q + r;
      if (m > mlast) continue;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int o = wn * 16 * NS + 16 * s + 4 * g;
        const floatx4 v = acc[q][s] * mant;
        if (vec) {
          if (o0 + o < a.O) *reinterpret_cast<floatx4*>(y + m * a.O + o) = v;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (o0 + o + c < a.O) y[m * a.O + o + c] = v[c];
        }
      }
    }
    return;
  }
  // bf16 results are turned in LDS, so that consecutive lanes store consecutive 16 bytes of a row
  __syncthreads();
#pragma unroll
  for (int q = 0; q < MS; ++q)
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const bf16x2_t lo{(__bf16)(acc[q][s][0] * mant), (__bf16)(acc[q][s][1] * mant)}, hi{(__bf16)(acc[q][s][2] * mant), (__bf16)(acc[q][s][3] * mant)};
      *reinterpret_cast<u32x2*>(lds + (wm * 16 * MS + 16 * q + r) * C::YROW + (wn * 16 * NS + 16 * s + 4 * g) * 2) =
          u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
  __syncthreads();
  uint16_t* y = static_cast<uint16_t*>(a.y) + (b * a.M + m0) * a.O + o0;
  const bool vec = a.O % 8 == 0 && (uintptr_t)a.y % 16 == 0;
  constexpr int PIECES = C::BO / 8;
#pragma unroll 4
  for (int q = tid; q < C::BM * PIECES; q += C::TH) {
    const int m = q / PIECES, o = q % PIECES * 8;
    if (m > mlast || o0 + o >= a.O) continue;
    const u32x4 v = ld16(lds + m * C::YROW + o * 2);
    if (vec) {
      st16(y + m * a.O + o, v);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (o0 + o + c < a.O) y[m * a.O + o + c] = (uint16_t)(v[c >> 1] >> (16 * (c & 1)));
    }
  }
}

// y = S sum of the parts, in their order.
__global__ void __launch_bounds__(256) fp4_join_kernel(const float* __restrict__ parts, int splits, int64_t per, int64_t batch, const float* __restrict__ ts,
                                                       void* __restrict__ y, int y_f32) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, total = per * batch;
  if (i >= total) return;
  float pow2 = 1.0f, mant[4] = {1.0f, 1.0f, 1.0f, 1.0f};
  if (ts)
#pragma unroll
    for (int c = 0; c < 4; ++c) split_scale(ts[min(i + c, total - 1) / per], pow2, mant[c]);
  const bool vec = total % 4 == 0;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const float* p = parts + s * total + i;
    if (vec) {
      const floatx4 q = *reinterpret_cast<const floatx4*>(p);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += q[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += i + c < total ? p[c] : 0.0f;
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] *= mant[c];
  if (y_f32) {
    float* o = static_cast<float*>(y) + i;
    if (vec && (uintptr_t)y % 16 == 0) {
      *reinterpret_cast<floatx4*>(o) = floatx4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < total) o[c] = v[c];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(y) + i;
    const bf16x2_t lo{(__bf16)v[0], (__bf16)v[1]}, hi{(__bf16)v[2], (__bf16)v[3]};
    const u32x2 h{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    if (vec && (uintptr_t)y % 8 == 0) {
      *reinterpret_cast<u32x2*>(o) = h;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < total) o[c] = (uint16_t)(h[c >> 1] >> (16 * (c & 1)));
    }
  }
}

constexpr int64_t kMost = 0xFFFFFFFF;  // threads of a launch along x
constexpr int64_t kMostMatrices = 65535;
constexpr int tile_threads(int rows) { return rows == 256 ? 512 : 256; }

template <int FMT, bool GRAD, int TERMS, int R, int WM, int WN, int MS, int NS>
static int launch_tile(const Fp4MatmulArgs& a, int64_t batch, int splits, hipStream_t st) {
  using C = Fp4Tile<R, WM, WN, MS, NS, GRAD>;
  static_assert(C::TH == tile_threads(C::BM), "what the plan counts");
  const int64_t mt = (a.M + C::BM - 1) / C::BM, ot = (a.O + C::BO - 1) / C::BO, grid = (mt * ot + 7) / 8 * 8;
  const dim3 wgs3((unsigned)grid, (unsigned)splits, (unsigned)batch);
  // a thread's two NVFP4 scales as one load
  constexpr bool PAIRS = FMT == FP4_FMT_NVFP4 && C::CPT == 2;
  if (!PAIRS || (a.K % 32 == 0 && (uintptr_t)a.ws % 2 == 0)) {
    hipLaunchKernelGGL((fp4_tile_kernel<FMT, GRAD, TERMS, true, R, WM, WN, MS, NS>), wgs3, dim3(C::TH), 0, st, a, (int)mt, (int)ot);
  } else if constexpr (PAIRS) {
    hipLaunchKernelGGL((fp4_tile_kernel<FMT, GRAD, TERMS, false, R, WM, WN, MS, NS>), wgs3, dim3(C::TH), 0, st, a, (int)mt, (int)ot);
  }
  FP4_CHECK(check_launch("fp4_matmul"));
  if (splits == 1) return FP4_OK;
  const int64_t wgs = (a.M * a.O * batch + 1023) / 1024;
  hipLaunchKernelGGL(fp4_join_kernel, dim3((unsigned)wgs), dim3(256), 0, st, a.parts, splits, a.M * a.O, batch, FMT == FP4_FMT_NVFP4 ? a.ts : nullptr, a.y, a.y_f32);
  return check_launch("fp4_join");
}

// The few-rows kernel's waves and steps a wave for K (0 waves: K is too long).
struct FewShape {
  int waves, steps;
};
static FewShape few_shape(int64_t k, int terms, int ms) {
  const int64_t ks = (k + kFewK - 1) / kFewK, most = terms == 3 ? 2 : 4 / ms;  // x of a wave: 128 registers, f32 192
  for (int u = 1; u <= most; u *= 2)
    if ((ks + u - 1) / u <= few_waves(ms, u, terms)) return {(int)((ks + u - 1) / u), u};
  return {0, 0};
}

template <int FMT, int TERMS, int MS, int U, bool DMA>
static int launch_few(const Fp4FewArgs& a, int64_t batch, int waves, hipStream_t st) {
  static std::atomic<uint64_t> raised{0};
  const int lds = waves * (2 * MS * 1024 + (DMA ? kRing * kSlot : 8192));
  void (*kernel)(Fp4FewArgs) = &fp4_few_kernel<FMT, TERMS, MS, U, DMA>;
  FP4_CHECK(raise_dyn_lds(reinterpret_cast<const void*>(kernel), 160 * 1024, raised));
  const int64_t strips = (a.N + 15) / 16, blocks = (a.M + 16 * MS - 1) / (16 * MS);
  // as many workgroups as stay on the card together, then the strips evenly
  const int64_t room = std::max<int64_t>(1, std::min<int64_t>(160 * 1024 / lds, 4 * few_per_simd(MS, U, TERMS) / (waves + 1))) * device_cu_count();
  const int64_t each = std::max<int64_t>(1, (strips * blocks * batch + room - 1) / room), wgs = (strips + each - 1) / each;
  hipLaunchKernelGGL(kernel, dim3((unsigned)wgs, (unsigned)blocks, (unsigned)batch), dim3(64 * (waves + 1)), lds, st, a);
  return check_launch("fp4_matmul");
}

template <int FMT, int TERMS, int MS, int U>
static int launch_few_dma(const Fp4FewArgs& a, int64_t batch, int waves, hipStream_t st) {
  // whole pieces of DMA: 16 bytes of codes and 4 of scales
  const bool whole = a.K % (FMT == FP4_FMT_NVFP4 ? 64 : 128) == 0 && (uintptr_t)a.w % 16 == 0 && (uintptr_t)a.ws % 4 == 0;
  return whole ? launch_few<FMT, TERMS, MS, U, true>(a, batch, waves, st) : launch_few<FMT, TERMS, MS, U, false>(a, batch, waves, st);
}

template <int FMT>
static int launch_few_rows(const Fp4FewArgs& a, int64_t batch, int terms, int ms, hipStream_t st) {
  const FewShape f = few_shape(a.K, terms, ms);
  if (terms == 3) return f.steps == 1 ? launch_few_dma<FMT, 3, 1, 1>(a, batch, f.waves, st) : launch_few_dma<FMT, 3, 1, 2>(a, batch, f.waves, st);
  if (ms == 1) {
    if (f.steps == 1) return launch_few_dma<FMT, 1, 1, 1>(a, batch, f.waves, st);
    if (f.steps == 2) return launch_few_dma<FMT, 1, 1, 2>(a, batch, f.waves, st);
    return launch_few_dma<FMT, 1, 1, 4>(a, batch, f.waves, st);
  }
  if (ms == 2) {
    if (f.steps == 1) return launch_few_dma<FMT, 1, 2, 1>(a, batch, f.waves, st);
    return launch_few_dma<FMT, 1, 2, 2>(a, batch, f.waves, st);
  }
  return launch_few_dma<FMT, 1, 4, 1>(a, batch, f.waves, st);
}

// The tiles there are: rows, outputs.
enum Fp4TileKind { TILE_16 = 0, TILE_32, TILE_64, TILE_128, TILE_256 };

template <int FMT, bool GRAD, int TERMS>
static int launch_tiles(const Fp4MatmulArgs& a, int64_t batch, int kind, int splits, hipStream_t st) {
  if (kind == TILE_16) return launch_tile<FMT, GRAD, TERMS, 4, 1, 4, 1, 2>(a, batch, splits, st);
  if (kind == TILE_32) return launch_tile<FMT, GRAD, TERMS, 4, 1, 4, 2, 2>(a, batch, splits, st);
  if (kind == TILE_64) return launch_tile<FMT, GRAD, TERMS, 4, 2, 2, 2, 2>(a, batch, splits, st);
  if (kind == TILE_128) return launch_tile<FMT, GRAD, TERMS, 2, 2, 2, 4, 4>(a, batch, splits, st);
  return launch_tile<FMT, GRAD, TERMS, 2, 2, 4, 8, 4>(a, batch, splits, st);
}
template <int FMT, bool GRAD>
static int launch_fp4(const Fp4MatmulArgs& a, int64_t batch, int kind, int splits, hipStream_t st) {
  return a.terms == 1 ? launch_tiles<FMT, GRAD, 1>(a, batch, kind, splits, st) : launch_tiles<FMT, GRAD, 3>(a, batch, kind, splits, st);
}

// ------------------------------------------------------------ the calls

// The few-rows kernel's blocks of 16 rows for a product, 0 where tiles are to take it.  Measured (us, graph replays, NVFP4,
// few-rows kernel and tiles): 1 x 2560 x 2560 5.8 and 11.6, 16 x 131072 x 2560 50 and 77, 32 x 10240 x 2560 12.9 and 18.3,
// 64 x 10240 x 2560 16.3 and 22.3, 64 x 2560 x 7168 17 and 22, 77 x 2560 x 2560 17 and 15.4, 256 x 10240 x 2560 28.8 and 22.2;
// f32 1 x 2560 x 2560 8.2 and 16.2, 64 x 2560 x 2560 14.3 and 19.6, 128 x 2560 x 3520 18.7 and 28.1.  Blocks of rows that
// pass a wide W four times or more lose (64 x 10240 x 5120 35 and 27, 64 x 131072 x 5120 364 and 194, MXFP4 204 and 186;
// f32 64 x 131072 x 2560 239 and 185, 128 x 131072 x 2560 468 and 244): the rule goes by rows and K alone.
static int few_blocks(int64_t m, int64_t n, int64_t k, int terms) {
  if (m > (terms == 3 ? 128 : 64)) return 0;
  for (int ms = terms == 3 || m <= 16 ? 1 : m <= 32 ? 2 : 4; ms > 0; ms /= 2)
    if (few_shape(k, terms, ms).waves) return ms;
  return 0;
}

struct Fp4Plan {
  int64_t sum, out, ld, terms;  // length of the sum, outputs, row stride and terms of x as the kernels read it
  bool rows;                    // x is copied (split, padded) first
  int few;                      // the few-rows kernel's blocks of 16 rows, or 0
  int kind, splits, each;       // the tile, workgroups that share one, their steps
  size_t row_bytes, bytes;      // of the workspace: x's rows, all
};

// One tile's modelled time: rounds of as many as the card holds at once at full load, and a last round between a lone
// tile's time and a full round's (microseconds a step of 64 products).
struct Fp4TileModel {
  int bm, bo, slots;
  double fixed, lone, loaded;
};
// A whole card's of 256 compute units, fitted at 40 and 160 steps before the codes came in wide loads (256 x 256 takes about
// 1.9 a step at full load since then, not 2.15); which tile is the fastest is still what they say, below.  Measured (us, graph replays) in this order, without splits: dx of 16 x 10240 ->
// 2560 80, 86, 77, 137, 276; y of 300 x 2560 -> 2560 36, 25, 18, 38, 76; of 1024 x 2560 -> 2560 85, 54, 33, 38, 77;
// 8192 x 2560 -> 10240 - , - , 764, 586, 435 (all before the wide loads).  Since then, the last three each
// with its best split: y of 1024 x 2560 -> 2560 33, 34, 39; of 2048 x 4096 -> 4096 124, 80, 82; of 600 x 2560 -> 10240 70,
// 51, 57; of 1024 x 2560 -> 10240 103, 77, 69; dx of 4096 x 2560 -> 2560 113, 79, 73: the model takes the fastest of each.
constexpr Fp4TileModel kTiles[] = {{16, 128, 768, 3.0, 0.50, 1.25}, {32, 128, 768, 3.0, 0.54, 1.40}, {64, 64, 768, 3.0, 0.37, 0.72},
                                   {128, 128, 512, 3.0, 0.85, 1.45}, {256, 256, 256, 4.0, 1.75, 2.15}};

// The tile and the number of workgroups that share one's steps whose modelled time is the least.  Parts of a tile are
// written, read and joined by a launch of its own: 4.5 us, and their bytes at 5 TB/s (4096 x 10240 -> 2560: 278 us in
// whole tiles, 251 in thirds; 16 x 10240 -> 2560 80 and, in eighths, 20).
static void choose_tile(int64_t m, int64_t out, int64_t steps, int64_t batch, int terms, Fp4Plan& p) {
  double best = 0;
  p.kind = TILE_64;
  p.splits = 1;
  for (int kind = TILE_16; kind <= TILE_256; ++kind) {
    const Fp4TileModel& t = kTiles[kind];
    const double tiles = (double)((m + t.bm - 1) / t.bm) * (double)((out + t.bo - 1) / t.bo) * (double)batch, terms_cost = terms == 3 ? 2.3 : 1.0;
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (s > 1 && (steps < 2 * s || tiles * s > 8192)) break;
      const double n = (double)((steps + s - 1) / s) * terms_cost, one = t.fixed + t.lone * n, full = t.fixed + t.loaded * n;
      const double rounds = std::floor(tiles * s / t.slots), rest = tiles * s - rounds * t.slots;
      double time = rounds * full + (rest > 0 ? one + (full - one) * rest / t.slots : 0.0);
      if (s > 1) time += 4.5 + 8.0 * s * (double)batch * (double)m * (double)out / 5e6;
      if (best == 0 || time < best) {
        best = time;
        p.kind = kind;
        p.splits = s;
      }
    }
  }
  p.each = (int)((steps + p.splits - 1) / p.splits);
  p.splits = p.each > 0 ? (int)((steps + p.each - 1) / p.each) : 1;
}

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
  if (p.sum > (int64_t)1 << 22 || k > (int64_t)1 << 26) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: sums of more than 2^22 products or k above 2^26");  // 32-bit offsets inside a tile
  if (batch > kMostMatrices) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: more than %lld matrices", (long long)kMostMatrices);
  const double elems = 0x1p46;
  if ((double)batch * m * k > elems || (double)batch * n * k > elems || (double)batch * m * n > elems)
    return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: an operand of more than 2^46 values");
  p.ld = (p.sum + kBK - 1) / kBK * kBK;
  p.terms = x_dtype == FP4_DT_F32 ? 3 : 1;
  p.few = grad ? 0 : few_blocks(m, n, k, (int)p.terms);
  p.rows = !p.few && (p.terms > 1 || p.ld != p.sum);
  p.kind = p.splits = p.each = 0;
  if (!p.few) choose_tile(m, p.out, p.ld / kBK, batch, (int)p.terms, p);
  p.row_bytes = p.rows ? ((size_t)(2 * p.terms) * (size_t)(batch * m * p.ld) + 255) / 256 * 256 : 0;
  p.bytes = p.row_bytes + (p.splits > 1 ? sizeof(float) * (size_t)p.splits * (size_t)(batch * m * p.out) : 0);
  // what no launch holds: workgroups of 256 threads that copy rows, of a tile (whose count is rounded up to a multiple of 8)
  if (p.rows && (batch * m * (p.ld / 8) + 255) / 256 * 256 > kMost) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: too many rows");
  if (!p.few) {
    const Fp4TileModel& t = kTiles[p.kind];
    const int64_t tiles = ((m + t.bm - 1) / t.bm) * ((p.out + t.bo - 1) / t.bo);
    if ((tiles + 7) / 8 * 8 * tile_threads(t.bm) > kMost) return fail(FP4_ERR_UNSUPPORTED, "fp4_matmul: too many rows or outputs");
  }
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
  if ((uintptr_t)x % (grad && p.rows ? x_dtype == FP4_DT_F32 ? 4 : 2 : 16) || (uintptr_t)w % 8 || (uintptr_t)tensor_scale % 4 ||
      (uintptr_t)y % (y_dtype == FP4_DT_F32 ? 4 : 2))
    return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: misaligned pointer");
  if (p.bytes) {
    if (!workspace || workspace_bytes < p.bytes) return fail(FP4_ERR_WORKSPACE, "fp4_matmul: workspace of %zu bytes, %zu needed", workspace_bytes, p.bytes);
    if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "fp4_matmul: misaligned workspace");
  }
  hipStream_t st = as_stream(stream);
  if (p.few) {
    const Fp4FewArgs a{x, w, static_cast<const uint8_t*>(w_scales), tensor_scale, y, m, n, (int)k, y_dtype == FP4_DT_F32};
    return w_fmt == FP4_FMT_NVFP4 ? launch_few_rows<FP4_FMT_NVFP4>(a, batch, (int)p.terms, p.few, st) : launch_few_rows<FP4_FMT_MXFP4>(a, batch, (int)p.terms, p.few, st);
  }
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
                        m, n, k, p.out, (int)(p.ld / kBK), (int)p.terms, y_dtype == FP4_DT_F32, p.each,
                        p.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.row_bytes) : nullptr};
  if (w_fmt == FP4_FMT_NVFP4) return grad ? launch_fp4<FP4_FMT_NVFP4, true>(a, batch, p.kind, p.splits, st) : launch_fp4<FP4_FMT_NVFP4, false>(a, batch, p.kind, p.splits, st);
  return grad ? launch_fp4<FP4_FMT_MXFP4, true>(a, batch, p.kind, p.splits, st) : launch_fp4<FP4_FMT_MXFP4, false>(a, batch, p.kind, p.splits, st);
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

// Not part of the interface: which kernel a call takes, for the tests that look at every one of them.  plan: blocks of 16
// rows of the few-rows kernel (0: tiles), a tile's rows, its outputs, workgroups that share its steps, whether x is copied.
int fp4_matmul_plan(int w_fmt, int x_dtype, int grad, int64_t batch, int64_t m, int64_t n, int64_t k, int* plan) {
  Fp4Plan p;
  FP4_CHECK(plan_fp4(w_fmt, x_dtype, grad != 0, batch, m, n, k, p));
  const int chosen[] = {p.few, p.few ? 0 : kTiles[p.kind].bm, p.few ? 0 : kTiles[p.kind].bo, p.few ? 1 : p.splits, p.rows};
  std::copy(chosen, chosen + 5, plan);
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
