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
// bf16 results sum each 128-block in the E4M3 MFMA.  As measured it adds eight
// consecutive products at a time, aligned to the largest of the eight and cut 14
// bits below its leading bit, and the eights in f32: 1.7e-5 of the products'
// magnitudes off on normal data, less than 7 2^-14 of them on any.  bf16's own
// rounding (2^-8 of the result) covers that unless a block's products cancel;
// fp16 MFMAs would cost twice the matrix time.  The blocks' sums are scaled and
// added in f32.  f32 results, for callers whose blocks cancel too, convert the
// codes to fp16 (exact: E4M3's range and precision lie inside fp16's) and take
// the fp16 MFMA, whose f32 sums measured 6.5e-8.
//
// Two scales whose product leaves f32's normal range are not multiplied with each
// other (add_far_scaled): a check by lane in the few-rows kernel, one of each
// table of scales in the tile kernel, 0 to 2 % of the time.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

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

// x as the few-rows kernel reads it: codes with their scales, or bf16 / f32
// values that each wave quantizes for its own K steps.
enum XKind { X_CODES = 0, X_BF16 = 1, X_F32 = 2 };

// V bf16 / f32 values from p (2 bf16 of 4 bytes upwards).
template <int XK, int V>
__device__ __forceinline__ void load_values(const uint8_t* p, float (&v)[V]) {
  constexpr int W = V * (XK == X_BF16 ? 2 : 4) / 4;
  uint32_t d[W];
  if constexpr (W == 1) {
    d[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const u32x2 t = *reinterpret_cast<const u32x2*>(p);
    d[0] = t.x;
    d[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4 t = ld16(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[4 * i + j] = t[j];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (XK == X_BF16) v[i] = __uint_as_float((i & 1) ? d[i >> 1] & 0xFFFF0000u : d[i >> 1] << 16);
    else v[i] = __uint_as_float(d[i]);
  }
}

// x [blocks, 128] to codes and one scale a block, 8 lanes of 16 values each
// per block (fp4_quantize's row kernel, with 4 lanes and IEEE divisions, takes
// 27 us for 8192 x 2560 bf16 and 5.1 us for 77 rows of f32 in a kernel trace;
// this one 13.4, 4.7 TB/s, and 3.1).
template <int XK>
__global__ void __launch_bounds__(256) fp8_rows_kernel(const uint8_t* __restrict__ x, int64_t blocks, uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales) {
  constexpr int XB = XK == X_BF16 ? 2 : 4;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if ((t >> 3) >= blocks) return;  // whole groups of 8 lanes
  float v[16];
  load_values<XK, 16>(x + t * 16 * XB, v);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const float sigma = (float)((double)amax / 448.0);
  uint32_t d[4];
  e4m3_codes<16>(v, sigma, d);
  st16(codes + t * 16, u32x4{d[0], d[1], d[2], d[3]});
  if ((t & 7) == 0) scales[t >> 3] = sigma;
}

// One wave quantizes its 128-block kb of P rows of x: 64 / P lanes a row, 2 P
// values a lane, so that the work follows the rows there are.  The codes pass
// through `stage` (2 KB of LDS of the wave) into the MFMA fragment; lane (g,
// r) gets row r mod P and its scale.
template <int XK, int P>
__device__ __forceinline__ intx8 quantized_frag(const uint8_t* x, int64_t row_bytes, int64_t M, int kb, uint8_t* stage, float& scale) {
  constexpr int V = 2 * P, LPR = 64 / P, XB = XK == X_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, row = lane / LPR, at = (lane % LPR) * V;
  float v[V];
  load_values<XK, V>(x + min((int64_t)row, M - 1) * row_bytes + (int64_t)(128 * kb + at) * XB, v);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const float sigma = (float)((double)amax / 448.0);
  uint32_t d[(V + 3) / 4];
  e4m3_codes<V>(v, sigma, d);
  uint8_t* to = stage + row * 128 + 16 * ((at >> 4) ^ (row >> 1)) + (at & 15);
  if constexpr (V == 2) *reinterpret_cast<uint16_t*>(to) = (uint16_t)d[0];
  else if constexpr (V == 8) *reinterpret_cast<u32x2*>(to) = u32x2{d[0], d[1]};
  else {
    st16(to, u32x4{d[0], d[1], d[2], d[3]});
    st16(stage + row * 128 + 16 * (((at >> 4) + 1) ^ (row >> 1)), u32x4{d[4], d[5], d[6], d[7]});
  }
  const int rr = r % P;
  scale = __shfl(sigma, rr * LPR);
  const uint8_t* from = stage + rr * 128 + 16 * (g ^ (rr >> 1));
  return frag_of(ld16(from), ld16(stage + rr * 128 + 16 * ((4 + g) ^ (rr >> 1))));
}

// At most 16 rows of x: a workgroup of NW waves walks over strips of 16
// outputs; wave w takes the 128-blocks w, w + NW, ... of K (U at most) of every
// strip.  Its share of x is loaded (and quantized) once and stays in
// registers as MFMA fragments; its share of the weights streams through a
// ring of D steps in LDS that belongs to the wave alone (16 rows x 128 bytes
// a step, by DMA, several strips ahead and without barriers: loading fragments
// straight into registers touches four rows in every four lanes, which
// measured 10.4 us against 7.5 at 16 x 10240 x 2560).  A strip's partial sums meet in
// LDS, one barrier a strip.  Bound by the weights' bytes, or by latency where
// they are few.
template <int U, int NW, int D, int XK, int P, typename OutT>
__global__ void __launch_bounds__(64 * NW) fp8_skinny_kernel(MatmulArgs a) {
  constexpr bool F32SUM = sizeof(OutT) == 4;
  constexpr int XB = XK == X_CODES ? 1 : XK == X_BF16 ? 2 : 4;
  constexpr int STAGED = XK == X_CODES ? 0 : 2048;  // a wave's staging of quantized x
  __shared__ __attribute__((aligned(16))) uint8_t lds[NW * (D * 2048 + STAGED) + 2 * NW * 1024];
  float* part = reinterpret_cast<float*>(lds + NW * (D * 2048 + STAGED));  // [2][NW][16 rows][16 outputs]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r = lane & 15;
  const int64_t b = blockIdx.z;
  const int KB = a.K >> 7, strips = (int)((a.N + 15) >> 4), first = blockIdx.x, step = gridDim.x;
  const int nu = max(0, (KB - wave + NW - 1) / NW);  // this wave's K steps of a strip
  const int mine = (strips - first + step - 1) / step;
  const uint8_t* wbase = a.w + b * a.N * a.K;
  const float* ws = a.ws + b * ((a.N + 127) >> 7) * KB;
  uint8_t* ring = lds + wave * (D * 2048 + STAGED);
  // item (strip i, step u) into ring slot `slot`: row j of the strip at 128 j, its chunks swizzled as in the tile kernel
  auto load = [&](int i, int u, int slot) __attribute__((always_inline)) {
    const int64_t n0 = (int64_t)(first + i * step) * 16;
    const int last = (int)min((int64_t)15, a.N - 1 - n0);  // rows past the end repeat the last one; their results are not stored
    const auto buf = buffer_of(wbase + n0 * a.K, (uint32_t)(last + 1) * (uint32_t)a.K);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 8 * j + (lane >> 3);
      dma_buffer(buf, (uint32_t)min(row, last) * (uint32_t)a.K + 16 * ((lane & 7) ^ (row >> 1)), 128 * (wave + NW * u), ring + 2048 * slot + 1024 * j);
    }
  };
  int li = 0, lu = 0;  // the next item to load
  auto load_next = [&](int slot) __attribute__((always_inline)) {
    // past the end the last item is loaded again, so that every step issues two instructions
    load(min(li, mine - 1), lu, slot);
    if (++lu == nu) { lu = 0; ++li; }
  };
  intx8 xf[U];
  float sx[U];
  if (nu > 0) {
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load_next(d);
    if constexpr (XK == X_CODES) {
      const int64_t m = b * a.M + min((int64_t)r, a.M - 1);
      const uint8_t* xrow = a.x + m * a.K + 16 * g;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kb = min(wave + NW * u, KB - 1);
        xf[u] = frag_of(ld16(xrow + 128 * kb), ld16(xrow + 128 * kb + 64));
        sx[u] = a.xs[m * KB + kb];
      }
    } else {
      const int64_t row_bytes = (int64_t)a.K * XB;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < nu) xf[u] = quantized_frag<XK, P>(a.x + b * a.M * row_bytes, row_bytes, a.M, wave + NW * u, ring + D * 2048, sx[u]);
    }
  }
  const int frag0 = r * 128 + 16 * (g ^ (r >> 1));
  int slot = 0;
  for (int i = 0; i < mine; ++i) {
    const int64_t n0 = (int64_t)(first + i * step) * 16;
    floatx4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < nu) {
        const float sw = scalar_load(ws + ((n0 >> 7) * KB + wave + NW * u));
        load_next(slot == 0 ? D - 1 : slot - 1);
        __builtin_amdgcn_s_waitcnt(vmcnt_only(2 * (D - 1)));  // this item has arrived; the D - 1 later ones may be on their way
        asm volatile("" ::: "memory");
        const uint8_t* w = ring + 2048 * slot;
        add_scaled(acc, block_product<F32SUM>(frag_of(ld16(w + frag0), ld16(w + (frag0 ^ 64))), xf[u]), sx[u], sw);
        // pinned here: the next item's loads overwrite a slot only after its values have reached an MFMA
        asm volatile("" ::"v"(acc));
        slot = slot == D - 1 ? 0 : slot + 1;
      }
    }
    float* pt = part + (i & 1) * (NW * 256);
    *reinterpret_cast<floatx4*>(pt + wave * 256 + r * 16 + 4 * (g ^ ((r >> 1) & 3))) = acc;
    __builtin_amdgcn_s_waitcnt(lgkmcnt0());
    // one barrier a strip: a wave writes this half of `part` again after the
    // next strip's barrier, which the readers below reach after reading
    asm volatile("s_barrier" ::: "memory");
    if (threadIdx.x < 256) {
      const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += pt[w * 256 + m * 16 + 4 * ((n >> 2) ^ ((m >> 1) & 3)) + (n & 3)];
      if (m < a.M && n0 + n < a.N) static_cast<OutT*>(a.y)[(b * a.M + m) * a.N + n0 + n] = out_of<OutT>(v);
    }
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // no DMA outlives the workgroup
}

// ------------------------------------------------------------ many rows

// Tile of BM rows of x by BN outputs per workgroup of WM x WN waves, each
// owning 16 MS rows and 16 NS outputs.  Both operands' tiles go through a ring
// of RING K steps in LDS by 16-byte DMA: eight consecutive lanes copy one
// row's 128 bytes, where loading MFMA fragments straight into registers would
// touch four rows in every four lanes (it measured 1.5 to 2 times slower, the
// more the larger the weights' share).  Chunks are XOR-swizzled by the row so
// that the 16 rows a fragment read touches hit all banks once.  One barrier a
// K step.  GROUPS groups of such waves share a tile, each with a run of its K
// steps and a ring of its own, and the first adds the groups' sums up: a lone
// step is mostly latency (0.33 us; deeper rings measured the same), so few
// tiles of many steps take GROUPS times fewer of them one after another.
constexpr int kTileTab = 24;  // K steps of scales held in LDS at once (even)

template <int WM, int WN, int MS, int NS, int RING, int GROUPS>
struct TileCfg {
  static constexpr int WAVES = WM * WN, BM = 16 * MS * WM, BN = 16 * NS * WN;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int XTAB = RING * STAGE;                    // f32 [kTileTab][BM]
  static constexpr int WTAB = XTAB + kTileTab * BM * 4;        // f32 [kTileTab][BN / 16]
  static constexpr int GLDS = WTAB + kTileTab * (BN / 16) * 4, FARTAB = GROUPS * GLDS;  // of a group; i32 [GROUPS * WAVES] of the workgroup
  static constexpr int LDS = FARTAB + GROUPS * WAVES * 4;
  static constexpr int ND = (BM + BN) / 8 / WAVES;             // DMA instructions of a wave per K step
  static_assert((BM / 8) % WAVES == 0 && (BN / 8) % WAVES == 0, "whole DMA instructions per wave");
  static_assert(LDS <= 160 * 1024, "LDS");
};

// One wave's 16 MS rows and 16 NS outputs from row m0 and output n0 on where
// scales are so far from 1 that their products may leave f32's normal range:
// from memory, 16 rows at a time, K's runs of `per_group` steps each summed up by
// itself, as the tile kernel's groups do.  It starts over, so that the tile
// kernel's registers need not hold both forms of a step (8192 x 2560 x 2560: 71 us,
// 212 with one such row and one such tile of W, 608 where all of them are).
template <int GROUPS, int MS, int NS, typename OutT>
__device__ __forceinline__ void far_tile(const MatmulArgs& a, int64_t b, int64_t m0, int64_t n0, int per_group) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15, KB = a.K >> 7;
  const float* ws = a.ws + b * ((a.N + 127) >> 7) * KB;
  // rows past the end of an operand repeat its last one; their results are not stored
  const uint8_t* w[NS];
  const float* sw[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int64_t n = n0 + 16 * s;
    w[s] = a.w + (b * a.N + min(n + r, a.N - 1)) * a.K + 16 * g;
    sw[s] = ws + (min(n, a.N - 1) >> 7) * KB;
  }
#pragma unroll 1
  for (int i = 0; i < MS; ++i) {
    const int64_t m = m0 + 16 * i + r, xm = b * a.M + min(m, a.M - 1);
    if (m0 + 16 * i >= a.M) break;
    const uint8_t* x = a.x + xm * a.K + 16 * g;
    const float* sx = a.xs + xm * KB;
    block_sums sum[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) sum[s] = block_sums{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int h = 0; h < GROUPS; ++h) {
      block_sums acc[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) acc[s] = block_sums{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
      for (int kb = h * per_group; kb < min(KB, (h + 1) * per_group); ++kb) {
        const intx8 xf = frag_of(ld16(x + 128 * kb), ld16(x + 128 * kb + 64));
#pragma unroll
        for (int s = 0; s < NS; ++s)
          add_far_scaled(acc[s], block_product<sizeof(OutT) == 4>(frag_of(ld16(w[s] + 128 * kb), ld16(w[s] + 128 * kb + 64)), xf), sx[kb], sw[s][kb]);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) sum[s] += acc[s];
    }
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (const int64_t n = n0 + 16 * s + 4 * g + c; m < a.M && n < a.N) static_cast<OutT*>(a.y)[(b * a.M + m) * a.N + n] = out_of<OutT>(sum[s][c]);
  }
}

template <int WM, int WN, int MS, int NS, int RING, int GROUPS, typename OutT>
__global__ void __launch_bounds__(64 * WM * WN * GROUPS, GROUPS > 2 ? GROUPS : 2) fp8_tile_kernel(MatmulArgs a, int mt, int nt) {
  using C = TileCfg<WM, WN, MS, NS, RING, GROUPS>;
  constexpr bool F32SUM = sizeof(OutT) == 4;
  constexpr int TH = 64 * C::WAVES, XD = C::BM / 8 / C::WAVES, WD = C::BN / 8 / C::WAVES;
  __shared__ __attribute__((aligned(16))) uint8_t tile_lds[C::LDS];
  const int group = GROUPS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TH) : 0;
  uint8_t* lds = tile_lds + group * C::GLDS;
  const int tid = threadIdx.x - group * TH, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, r = lane & 15;
  const int wm = wave / WN, wn = wave % WN;
  // workgroups b, b + 8, ... run on one XCD: give it consecutive tiles (they
  // share x and W tiles in its L2), in groups of 8 rows of tiles
  const int tiles = mt * nt, per = (tiles + 7) / 8;
  const int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (t >= tiles) return;
  const int grp = t / (8 * nt), in = t - grp * 8 * nt, rows = min(8, mt - grp * 8);
  const int64_t m0 = (int64_t)(grp * 8 + in % rows) * C::BM, n0 = (int64_t)(in / rows) * C::BN, b = blockIdx.z;
  const int K = a.K, KB = K >> 7;
  const int per_group = (KB + GROUPS - 1) / GROUPS, first = group * per_group, last = min(KB, first + per_group);  // this group's K steps
  const int64_t NB = (a.N + 127) >> 7;
  const float* xs = a.xs + (b * a.M + m0) * KB;
  const float* ws = a.ws + b * NB * KB;
  // rows past the end of an operand repeat its last one; their results are not stored
  const int mlast = (int)min((int64_t)C::BM - 1, a.M - 1 - m0), nlast = (int)min((int64_t)C::BN - 1, a.N - 1 - n0);
  const auto xb = buffer_of(a.x + (b * a.M + m0) * K, (uint32_t)(mlast + 1) * (uint32_t)K);
  const auto wb = buffer_of(a.w + (b * a.N + n0) * K, (uint32_t)(nlast + 1) * (uint32_t)K);
  uint32_t xoff[XD], woff[WD];
#pragma unroll
  for (int j = 0; j < XD; ++j) {
    const int row = wave * 8 * XD + 8 * j + (lane >> 3);
    xoff[j] = (uint32_t)min(row, mlast) * (uint32_t)K + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
#pragma unroll
  for (int j = 0; j < WD; ++j) {
    const int row = wave * 8 * WD + 8 * j + (lane >> 3);
    woff[j] = (uint32_t)min(row, nlast) * (uint32_t)K + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  auto load = [&](int kb, int stage) __attribute__((always_inline)) {
    uint8_t* st = lds + stage * C::STAGE;
#pragma unroll
    for (int j = 0; j < XD; ++j) dma_buffer(xb, xoff[j], 128 * kb, st + (wave * XD + j) * 1024);
#pragma unroll
    for (int j = 0; j < WD; ++j) dma_buffer(wb, woff[j], 128 * kb, st + C::BM * 128 + (wave * WD + j) * 1024);
  };
  float* xtab = reinterpret_cast<float*>(lds + C::XTAB);
  float* wtab = reinterpret_cast<float*>(lds + C::WTAB);
  int* fartab = reinterpret_cast<int*>(tile_lds + C::FARTAB);  // which bounds a wave's scales in the tables leave
  // Scales of the K steps [kb0, kb0 + kTileTab): every thread's loads are
  // issued together, consecutive threads along a row's K steps.
  auto fill_tables = [&](int kb0) __attribute__((always_inline)) {
    kb0 = min(kb0, KB - 1);
    const uint32_t n = min(kTileTab, KB - kb0), inv = ((1u << 20) + n - 1) / n;  // i / n = i inv >> 20 for i < 2^13
    constexpr int XI = (C::BM * kTileTab + TH - 1) / TH, WI = (C::BN / 16 * kTileTab + TH - 1) / TH;
    float xv[XI], wv[WI];
#pragma unroll
    for (int j = 0; j < XI; ++j) {
      const uint32_t i = min(tid + (uint32_t)TH * j, C::BM * n - 1), m = (i * inv) >> 20, q = i - m * n;
      xv[j] = xs[(int64_t)min((int)m, mlast) * KB + kb0 + q];
    }
#pragma unroll
    for (int j = 0; j < WI; ++j) {
      const uint32_t i = min(tid + (uint32_t)TH * j, C::BN / 16 * n - 1), s = (i * inv) >> 20, q = i - s * n;
      wv[j] = ws[min((n0 + 16 * s) >> 7, NB - 1) * KB + kb0 + q];
    }
    // no product leaves f32's normal range where x's scales lie in [2^-100, 2^120] and W's in [2^-24, 2^7] (as weights
    // have them, so that a padding row of anything does not matter), nor where both lie in [2^-62, 2^62]
    ScaleRange xr, wr;
#pragma unroll
    for (int j = 0; j < XI; ++j) xr.add(xv[j]);
#pragma unroll
    for (int j = 0; j < WI; ++j) wr.add(wv[j]);
    const int seen = (__any(xr.outside(-100, 120) || wr.outside(-24, 7)) ? 1 : 0) | (__any(xr.outside(-62, 62) || wr.outside(-62, 62)) ? 2 : 0);
    if (lane == 0) fartab[group * C::WAVES + wave] = seen;
#pragma unroll
    for (int j = 0; j < XI; ++j) {  // threads past the end repeat the last entry
      const uint32_t i = min(tid + (uint32_t)TH * j, C::BM * n - 1), m = (i * inv) >> 20, q = i - m * n;
      xtab[q * C::BM + m] = xv[j];
    }
#pragma unroll
    for (int j = 0; j < WI; ++j) {
      const uint32_t i = min(tid + (uint32_t)TH * j, C::BN / 16 * n - 1), s = (i * inv) >> 20, q = i - s * n;
      wtab[q * (C::BN / 16) + s] = wv[j];
    }
  };
  floatx4 acc[MS][NS];
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[i][s] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int v = 0; v < RING - 1; ++v) load(min(first + v, KB - 1), v);
  // row 16 i + r of a tile: chunks g and 4 + g
  const int frag0 = r * 128 + 16 * (g ^ (r >> 1));
  int stage = 0;
  bool far = false;  // whether the tables hold scales whose product may leave f32's normal range (of all groups)
  auto step = [&](int kb, int q) __attribute__((always_inline)) {
    // this wave's part of step kb has arrived; the RING - 2 later ones may still be on their way
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0(C::ND * (RING - 2)));
    asm volatile("s_barrier" ::: "memory");
    const uint8_t* xr = lds + stage * C::STAGE + wm * (16 * MS * 128) + frag0;
    const uint8_t* wr = lds + stage * C::STAGE + C::BM * 128 + wn * (16 * NS * 128);
    load(min(kb + RING - 1, KB - 1), stage == 0 ? RING - 1 : stage - 1);
    stage = stage == RING - 1 ? 0 : stage + 1;
    if (q == 0) {
      int any = 0;
#pragma unroll
      for (int w = 0; w < GROUPS * C::WAVES; ++w) any |= fartab[w];
      far = __builtin_amdgcn_readfirstlane(any) == 3;
      if (far) return;
    }
    if (GROUPS > 1 && kb >= last) return;  // the last groups may have fewer steps; every barrier is met
    float sw[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) sw[s] = wtab[q * (C::BN / 16) + wn * NS + s];
    intx8 wf[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) wf[s] = frag_of(ld16(wr + frag0 + 2048 * s), ld16(wr + (frag0 ^ 64) + 2048 * s));
    // Software pipeline over the row groups i: while the MFMAs of group i run,
    // the scaled sums of group i - 1 are added up and group i + 2 is read.
    intx8 xf[3];
    float sx[2];
    floatx4 p[2][NS];
    auto read_x = [&](int i) __attribute__((always_inline)) {
      xf[i % 3] = frag_of(ld16(xr + 2048 * i), ld16(xr - frag0 + (frag0 ^ 64) + 2048 * i));
    };
    auto add = [&](int i, int s) __attribute__((always_inline)) {
      const float f = sx[i & 1] * sw[s];
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][s][c] = fmaf(p[i & 1][s][c], f, acc[i][s][c]);
    };
    read_x(0);
    read_x(1);
    sx[0] = xtab[q * C::BM + wm * 16 * MS + r];
    // the order is pinned: left to itself the scheduler moves the reads next
    // to their uses and the sums next to their MFMAs, and waits for both
#pragma unroll
    for (int i = 0; i <= MS; ++i) {
      if (i + 2 < MS) read_x(i + 2);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        __builtin_amdgcn_sched_barrier(0);
        if (i < MS) p[i & 1][s] = block_product<F32SUM>(wf[s], xf[i % 3]);
        if (i > 0) add(i - 1, s);
      }
      if (i + 1 < MS) sx[(i + 1) & 1] = xtab[q * C::BM + wm * 16 * MS + 16 * (i + 1) + r];
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
      for (int s = 0; s < NS; ++s) asm volatile("" ::"v"(acc[i][s]));
  };
  for (int k0 = 0; k0 < per_group && !far; k0 += kTileTab) {
    if (k0 > 0) asm volatile("s_barrier" ::: "memory");  // every wave is past the tables' last use
    fill_tables(first + k0);
    const int n = min(kTileTab, per_group - k0);
    for (int q = 0; q < n && !far; ++q) step(first + k0 + q, q);  // the step's barrier follows the table stores
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // the last steps' DMA repeats step KB - 1: none outlives the workgroup
  if (far) {
    if (group == 0) far_tile<GROUPS, MS, NS, OutT>(a, b, m0 + wm * 16 * MS, n0 + wn * 16 * NS, per_group);
    return;
  }
  // The tile is turned in LDS: straight from the accumulators every four lanes
  // of a store would touch four rows of y (7 of the 22 us of a lone tile's
  // fixed cost); from LDS consecutive lanes store consecutive 16 bytes.
  __syncthreads();
  if constexpr (GROUPS > 1) {
    static_assert(TH * MS * NS * 16 <= C::GLDS, "a group's sums fit its ring");
    if (group > 0)
#pragma unroll
      for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int s = 0; s < NS; ++s) *reinterpret_cast<floatx4*>(lds + ((i * NS + s) * TH + tid) * 16) = acc[i][s];
    __syncthreads();
    if (group == 0)
#pragma unroll
      for (int h = 1; h < GROUPS; ++h)
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
          for (int s = 0; s < NS; ++s) acc[i][s] += *reinterpret_cast<const floatx4*>(lds + h * C::GLDS + ((i * NS + s) * TH + tid) * 16);
  }
  constexpr int ROW = C::BN * (int)sizeof(OutT) + 16, PV = 16 / (int)sizeof(OutT), PIECES = C::BN / PV;
  static_assert(C::BM * ROW <= C::GLDS, "the output tile fits a ring");
  if (group == 0)
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      struct alignas(4 * sizeof(OutT)) V4 { OutT v[4]; } v;
#pragma unroll
      for (int c = 0; c < 4; ++c) v.v[c] = out_of<OutT>(acc[i][s][c]);
      *reinterpret_cast<V4*>(lds + (wm * 16 * MS + 16 * i + r) * ROW + (wn * 16 * NS + 16 * s + 4 * g) * (int)sizeof(OutT)) = v;
    }
  __syncthreads();
  OutT* y = static_cast<OutT*>(a.y) + (b * a.M + m0) * a.N + n0;
  const bool vec = a.N % PV == 0 && (uintptr_t)a.y % 16 == 0;  // rows of y in whole 16-byte pieces
#pragma unroll 4
  for (int q = threadIdx.x; q < C::BM * PIECES; q += TH * GROUPS) {
    const int m = q / PIECES, n = (q % PIECES) * PV;
    if (m > mlast || n > nlast) continue;
    const u32x4 v = ld16(tile_lds + m * ROW + n * (int)sizeof(OutT));
    if (vec) {
      st16(y + (int64_t)m * a.N + n, v);
    } else {
#pragma unroll
      for (int c = 0; c < PV; ++c) {
        OutT o;
        if constexpr (sizeof(OutT) == 2) o = (OutT)(v[c >> 1] >> (16 * (c & 1)));
        else o = __uint_as_float(v[c]);
        if (n + c <= nlast) y[(int64_t)m * a.N + n + c] = o;
      }
    }
  }
}

constexpr int64_t kMaxThreads = 0xFFFFFFFF;  // of a launch along x
constexpr int64_t kMaxBatch = 65535;         // workgroups along z

template <int WM, int WN, int MS, int NS, int RING, int GROUPS, typename OutT>
static int launch_tile(const MatmulArgs& a, int64_t batch, hipStream_t st) {
  using C = TileCfg<WM, WN, MS, NS, RING, GROUPS>;
  const int64_t mt = (a.M + C::BM - 1) / C::BM, nt = (a.N + C::BN - 1) / C::BN;
  const int64_t grid = (mt * nt + 7) / 8 * 8;
  if (grid * (64 * C::WAVES * GROUPS) > kMaxThreads) return fail(FP4_ERR_UNSUPPORTED, "matmul: too many rows or outputs");
  hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, MS, NS, RING, GROUPS, OutT>), dim3((unsigned)grid, 1, (unsigned)batch), dim3(64 * C::WAVES * GROUPS), 0, st,
                     a, (int)mt, (int)nt);
  return check_launch("fp8_block_matmul");
}

template <int U, int NW, int D, int XK, int P, typename OutT>
static int launch_skinny(const MatmulArgs& a, int64_t batch, hipStream_t st) {
  // two workgroups a compute unit, as their LDS allows (f32 results with 8 K steps a wave: registers leave one)
  const int64_t strips = (a.N + 15) / 16, wgs = std::max<int64_t>(1, 2 * device_cu_count() / batch);
  hipLaunchKernelGGL((fp8_skinny_kernel<U, NW, D, XK, P, OutT>), dim3((unsigned)std::min(strips, wgs), 1, (unsigned)batch), dim3(64 * NW), 0, st, a);
  return check_launch("fp8_block_matmul");
}

constexpr int kSkinnyMaxK = 8 * 8 * 128;  // 8 K steps for each of 8 waves
template <int XK, int P, typename OutT>
static int launch_skinny_k(const MatmulArgs& a, int64_t batch, hipStream_t st) {
  constexpr int D = XK == X_CODES ? 4 : 3;  // with the staging of x, two workgroups share a CU's LDS either way
  const int kb = a.K / 128;
  if (kb <= 8) return launch_skinny<1, 8, D, XK, P, OutT>(a, batch, st);
  if (kb <= 24) return launch_skinny<3, 8, D, XK, P, OutT>(a, batch, st);
  return launch_skinny<8, 8, D, XK, P, OutT>(a, batch, st);
}

template <int XK, typename OutT>
static int launch_skinny_rows(const MatmulArgs& a, int64_t batch, hipStream_t st) {
  if (a.M == 1) return launch_skinny_k<XK, 1, OutT>(a, batch, st);
  if (a.M <= 4) return launch_skinny_k<XK, 4, OutT>(a, batch, st);
  return launch_skinny_k<XK, 16, OutT>(a, batch, st);
}

// One variant's modelled time: rounds of `slots` tiles at full load, and a last
// partial round between a lone tile's time and a full round's (microseconds).
struct TileModel {
  int bm, bn, slots_per_cu;
  double fixed, lone, loaded;  // per K step
  double time(const MatmulArgs& a, int64_t batch) const {
    const double tiles = (double)((a.M + bm - 1) / bm) * (double)((a.N + bn - 1) / bn) * (double)batch, slots = (double)slots_per_cu * device_cu_count();
    const double kb = a.K / 128, full = fixed + loaded * kb, one = fixed + lone * kb;
    const double rounds = std::floor(tiles / slots), rest = tiles - rounds * slots;
    return rounds * full + (rest > 0 ? one + (full - one) * rest / slots : 0.0);
  }
};

// The tile whose modelled time is the least.  The constants are this card's,
// fitted at K = 2560: a tile alone / a full round (us) 8.8 / 19.8 (64 x 64),
// 16 / 28 (128 x 128), 27 / 36 (192 x 256), 34 / 46 (256 x 256).  Measured (us),
// in that order: 1024 x 2560 15.4, 17.6, 28.8, 35.7; 8192 x 2560 98.8, 73.9, 68.4,
// 78.6; 8192 x 10240 (128 up) 268, 247, 230.  64 x 64 with the steps split over four
// groups against without: 77 x 1000 x 2560 7.7, 8.8; 300 x 2560 x 2560 8.6, 9.4; 64 x
// 2560 x 8192 14.8, 22.7; 512 x 2560 x 2560 15.5, 11.4.  f32 results take the fp16 MFMA, whose
// converted operands leave registers for 64 x 64 and 128 x 128 only.  The model has
// no term for the bytes written: at K = 128 a tile takes up to twice what it says
// (32 x (500 x 512 x 128): 5.2 modelled, 9.2 in a trace).
constexpr TileModel kTile64{64, 64, 4, 2.0, 0.34, 0.89}, kTile64Split{64, 64, 1, 4.4, 0.16, 0.26}, kTile128{128, 128, 2, 4.0, 0.60, 1.20}, kTile192{192, 256, 1, 4.4, 1.15, 1.58},
    kTile256{256, 256, 1, 5.0, 1.45, 2.05};

template <typename OutT>
static int launch_tiles(const MatmulArgs& a, int64_t batch, hipStream_t st) {
  const double t64 = kTile64.time(a, batch), t128 = kTile128.time(a, batch), t64s = kTile64Split.time(a, batch);
  if constexpr (sizeof(OutT) == 2) {
    const double t192 = kTile192.time(a, batch), t256 = kTile256.time(a, batch);
    if (t256 <= std::min({t192, t64, t64s, t128})) return launch_tile<2, 4, 8, 4, 2, 1, OutT>(a, batch, st);
    if (t192 <= std::min({t64, t64s, t128})) return launch_tile<2, 4, 6, 4, 2, 1, OutT>(a, batch, st);
  }
  if (t64s <= std::min(t64, t128)) return launch_tile<2, 2, 2, 2, 2, 4, OutT>(a, batch, st);
  return t64 <= t128 ? launch_tile<2, 2, 2, 2, 2, 1, OutT>(a, batch, st) : launch_tile<2, 2, 4, 4, 2, 1, OutT>(a, batch, st);
}

constexpr int64_t kFewRows = 16;

// bf16 / f32 x that the few-rows kernel quantizes by itself (one launch, no workspace)
static bool quantized_inside(int x_dtype, int64_t m, int64_t k) {
  return x_dtype != FP4_DT_E4M3 && m <= kFewRows && k <= kSkinnyMaxK;
}

template <typename OutT>
static int launch_matmul(const MatmulArgs& a, int xk, int64_t batch, hipStream_t st) {
  if (xk == X_BF16) return launch_skinny_rows<X_BF16, OutT>(a, batch, st);
  if (xk == X_F32) return launch_skinny_rows<X_F32, OutT>(a, batch, st);
  if (a.M <= kFewRows && a.K <= kSkinnyMaxK) return launch_skinny_k<X_CODES, 16, OutT>(a, batch, st);
  return launch_tiles<OutT>(a, batch, st);
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
  if (k > (int64_t)1 << 22) return fail(FP4_ERR_UNSUPPORTED, "matmul: k beyond 2^22");  // 32-bit offsets inside a tile of 256 rows
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
  *bytes = x_dtype == FP4_DT_E4M3 || quantized_inside(x_dtype, m, k) ? 0 : codes_bytes(batch, m, k) + sizeof(float) * (size_t)(batch * m * (k / 128));
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
  if (batch > kMaxBatch) return fail(FP4_ERR_UNSUPPORTED, "matmul: more than %lld matrices", (long long)kMaxBatch);
  hipStream_t st = as_stream(stream);
  MatmulArgs a{static_cast<const uint8_t*>(x), x_scales, w, w_scales, y, m, n, (int)k};
  int xk = X_CODES;
  if (quantized_inside(x_dtype, m, k)) {
    xk = x_dtype == FP4_DT_BF16 ? X_BF16 : X_F32;
  } else if (x_dtype != FP4_DT_E4M3) {
    if (!workspace || workspace_bytes < need)
      return fail(FP4_ERR_WORKSPACE, "matmul: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "matmul: misaligned workspace");
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(codes + codes_bytes(batch, m, k));
    const int64_t blocks = batch * m * (k / 128), wgs = (blocks * 8 + 255) / 256;
    if (wgs * 256 > kMaxThreads) return fail(FP4_ERR_UNSUPPORTED, "matmul: too many rows");
    if (x_dtype == FP4_DT_BF16)
      hipLaunchKernelGGL(fp8_rows_kernel<X_BF16>, dim3((unsigned)wgs), dim3(256), 0, st, static_cast<const uint8_t*>(x), blocks, codes, scales);
    else
      hipLaunchKernelGGL(fp8_rows_kernel<X_F32>, dim3((unsigned)wgs), dim3(256), 0, st, static_cast<const uint8_t*>(x), blocks, codes, scales);
    FP4_CHECK(check_launch("fp8_rows"));
    a.x = codes;
    a.xs = scales;
  }
  return y_dtype == FP4_DT_BF16 ? launch_matmul<uint16_t>(a, xk, batch, st) : launch_matmul<float>(a, xk, batch, st);
}

}  // extern "C"
