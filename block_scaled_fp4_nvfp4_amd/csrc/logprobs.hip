// Log probabilities of given tokens with entropy, rank and the most likely
// alternatives (token_logprobs), and their gradient (token_logprobs_grad), from
// rows of logits l at a temperature T (gfx950):
//
//   M = max l, z = (l - M) / T, Z = sum e^z = 1 + R
//   logprob = z_t - ln Z          entropy H = ln Z - sum z e^z / Z
//   dl_j = (g_lp ([j = t] - p_j) - g_H p_j (ln p_j + H)) / T,   p_j = e^(z_j) / Z
//
// R, the sum without the largest logit's 1, is held apart: where a token is all but
// certain, ln Z = log1p(R), H (all its terms are positive) and 1 - p_t = (R -
// expm1(z_t)) / Z keep their bits, which 1 + R would cut off at 2^-24.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"

namespace fp4 {

constexpr int kTopMost = 64;    // one lane of a wave each
constexpr int kSplitsMost = 64;  // parts of a row, one lane each when they meet
constexpr int kFewInserts = 6;   // alternatives that are inserted one by one; more are sorted and merged
constexpr float kLog2E = 1.44269504f, kLn2 = 0.693147181f;

struct LogprobArgs {
  const void* logits;
  int64_t stride, V;
  const int32_t* targets;
  float inv_t;
  int top, splits;
  float* logprobs;      // [T]
  int32_t* ranks;       // [T]
  int32_t* top_ids;     // [T, top]
  float* top_logprobs;  // [T, top]
  float* stats;         // [T, 3]: M, R, H
  float* parts;         // [T, splits, 8 + 2 top]: a part's Sums, its alternatives' logits and ids
};

__device__ __forceinline__ float logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit(const uint16_t* p, int64_t i) { return bf16_bits_to_f32(p[i]); }

// What a wave, a workgroup or a row has seen: the largest logit m, how many
// exponentials were 1 (the largest itself, and what equals it), the sum of the
// others, sum t 2^t with t = (l - m) log2(e) / T, and the logits before the target.
struct Sums {
  float m, R, E;
  int32_t ones, rank;
};
__device__ __forceinline__ Sums no_sums() { return Sums{-__builtin_huge_valf(), 0.0f, 0.0f, 0, 0}; }

// `b` taken into `a`, both brought to the larger maximum.
__device__ __forceinline__ void join(Sums& a, const Sums& b, float c) {
  const float m = fmaxf(a.m, b.m), at = m > -__builtin_huge_valf() ? m : 0.0f;
  // parts with nothing left have m = -inf and sums of 0: any small power does
  const float ta = fmaxf((a.m - at) * c, -200.0f), tb = fmaxf((b.m - at) * c, -200.0f);
  const float sa = exp2f(ta), sb = exp2f(tb), na = (float)a.ones, nb = (float)b.ones;
  const bool la = a.m == m, lb = b.m == m;
  a.E = sa * fmaf(ta, a.R + na, a.E) + sb * fmaf(tb, b.R + nb, b.E);
  a.R = sa * (a.R + (la ? 0.0f : na)) + sb * (b.R + (lb ? 0.0f : nb));
  a.ones = (la ? a.ones : 0) + (lb ? b.ones : 0);
  a.rank += b.rank;
  a.m = m;
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, 0xF, 0xF, false);
  return fmaxf(v, __int_as_float(o));
}
// The wave's largest value (NaN is not), the same for every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = dpp_max<0x111>(v);  // the lanes 1, 2, 4, 8 before in the row of 16
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);  // the last lane of the row before, of the rows before
  v = dpp_max<0x143>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ int from_lane_before(int v) { return __builtin_amdgcn_update_dpp(v, v, 0x138, 0xF, 0xF, false); }

// The best alternatives so far, lane j the j-th, largest first, ties by id; empty
// ones are (-inf, none).
constexpr int kNone = 0x7FFFFFFF;
__device__ __forceinline__ bool before(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

struct TopList {
  float v = -__builtin_huge_valf();
  int id = kNone;
  // One step of a sorting network: of each two lanes `d` apart the one with `first` gets the element that comes before.
  __device__ __forceinline__ void exchange(int d, bool first) {
    const float ov = __shfl_xor(v, d);
    const int oid = __shfl_xor(id, d);
    if (before(v, id, ov, oid) != first) v = ov, id = oid;
  }
  __device__ __forceinline__ void sort() {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 2; n <= 64; n *= 2)
#pragma unroll
      for (int d = n / 2; d > 0; d /= 2) exchange(d, ((lane & d) == 0) == ((lane & n) == 0));
  }
  // The first 64 of both lists: of the j-th here and the j-th last there the better, which
  // rise and fall once, so that the network's last six steps sort them.
  __device__ __forceinline__ void merge(float ov, int oid) {
    const int lane = threadIdx.x & 63;
    ov = __shfl_xor(ov, 63);
    oid = __shfl_xor(oid, 63);
    if (before(ov, oid, v, id)) v = ov, id = oid;
#pragma unroll
    for (int d = 32; d > 0; d /= 2) exchange(d, (lane & d) == 0);
  }
  __device__ __forceinline__ void insert(float cv, int cid) {  // cv, cid: the same for every lane
    const int lane = threadIdx.x & 63, at = __popcll(__ballot(before(v, id, cv, cid)));
    const int pv = from_lane_before(__float_as_int(v)), pid = from_lane_before(id);
    if (lane > at) v = __int_as_float(pv), id = pid;
    if (lane == at) v = cv, id = cid;
  }
};

// Of the lanes with the largest v the one with the lowest id.
__device__ __forceinline__ int lane_of_max(float v, int id, float most) {
  uint64_t which = __ballot(v == most);
  if (__popcll(which) > 1) {
    int low = v == most ? id : kNone;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) low = min(low, __shfl_xor(low, o));
    which = __ballot(v == most && id == low);
  }
  return (int)__ffsll((unsigned long long)which) - 1;
}

// The lists of a workgroup's WAVES waves (a power of two) into wave 0's, pair by pair.
template <int WAVES>
__device__ __forceinline__ void merge_waves(TopList& best, int wave, float (&v)[WAVES][kTopMost], int (&id)[WAVES][kTopMost]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < WAVES; d *= 2) {
    if ((wave & (2 * d - 1)) == d) v[wave][lane] = best.v, id[wave][lane] = best.id;
    __syncthreads();
    if ((wave & (2 * d - 1)) == 0) best.merge(v[wave + d][lane], id[wave + d][lane]);
  }
}

// A row's results from its sums and alternatives, by one wave.
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int64_t row, const Sums& s, const TopList& best, bool given, float lt) {
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_huge_valf(), at = s.m > ninf ? s.m : 0.0f;
  const float R = s.R + (float)(s.ones - 1);  // -1 for a row with nothing left
  const float Z = 1.0f + R, logZ = log1pf(R), H = Z == 0.0f ? 0.0f : logZ - s.E * kLn2 / Z;
  if (lane == 0) {
    if (a.logprobs) a.logprobs[row] = !given ? 0.0f : Z == 0.0f ? ninf : (lt - at) * a.inv_t - logZ;
    if (a.ranks) a.ranks[row] = given ? s.rank : -1;
    if (a.stats) {
      a.stats[3 * row] = s.m;
      a.stats[3 * row + 1] = R;
      a.stats[3 * row + 2] = H;
    }
  }
  if (lane < a.top) {
    const bool some = best.id != kNone;
    a.top_ids[row * a.top + lane] = some ? best.id : -1;
    a.top_logprobs[row * a.top + lane] = some ? (best.v - at) * a.inv_t - logZ : ninf;
  }
}

// The part `split` of a row by a workgroup of four waves.  A wave takes 2 x 64
// pieces of 16 bytes at a time, loaded one round ahead.  Its running maximum is one
// for all lanes, and a round whose logits all lie below it needs nothing but
// t = (l - m) c, 2^t, the two sums and the count of logits before the target, 10
// operations a bf16 value; a round that reaches it (few do) brings the sums to the
// new one and counts the exponentials that are 1.  Alternatives: a round with
// nothing above the wave's last one costs a comparison; else the lanes' largest values
// are taken out and inserted, or where they are many sorted and merged into the list.
template <typename T>
__global__ void __launch_bounds__(256) logprobs_kernel(LogprobArgs a) {
  constexpr int PV = 16 / (int)sizeof(T), NV = 2 * PV;  // values of a piece, of a lane's round
  __shared__ Sums sums_of[4];
  __shared__ float list_v[4][kTopMost];
  __shared__ int list_id[4][kTopMost];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x - row * a.splits);
  const T* l = static_cast<const T*>(a.logits) + row * a.stride;
  const float ninf = -__builtin_huge_valf(), c = a.inv_t * kLog2E;
  // pieces start at multiples of 16 bytes: the first one `skip` values before the row
  const int skip = (int)(((uintptr_t)l & 15) / sizeof(T)), V = (int)a.V;
  const int pieces = (int)((a.V + skip + PV - 1) / PV), per = ((pieces + a.splits - 1) / a.splits + 511) / 512 * 512;
  const int first = split * per, last = min(pieces, first + per);
  const int32_t t = a.targets ? a.targets[row] : -1;
  const bool given = t >= 0 && t < V;
  const float lt = given ? logit(l, t) : __builtin_nanf("");  // a NaN counts nothing before it
  // of ids below t those >= lt come before it, of others those > lt, which is >= the next float
  const int lb = __float_as_int(lt);
  const float above = lt != lt ? lt : lt == 0.0f ? __int_as_float(1) : __int_as_float(lb >= 0 ? lb + 1 : lb - 1);
  const int t_piece = given ? (t + skip) / PV : -1;

  Sums s = no_sums();
  float R = 0.0f, E = 0.0f, gate = ninf;  // a lane's sums; logits below `gate` have 2^t < 1
  TopList best;
  float least = ninf;                     // the last alternative
  int least_id = kNone;
  u32x4 raw[2];
  auto load = [&](int p0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int p = p0 + 64 * u + lane, i0 = p * PV - skip;
      if (p < last && i0 >= 0 && i0 + PV <= V) {
        raw[u] = *reinterpret_cast<const u32x4*>(l + i0);
      } else {  // past the part, or a piece that the row does not fill
        constexpr uint32_t kMasked = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        raw[u] = u32x4{kMasked, kMasked, kMasked, kMasked};
        if (p < last)
#pragma unroll
          for (int j = 0; j < PV; ++j)
            if (i0 + j >= 0 && i0 + j < V) {
              if constexpr (sizeof(T) == 4) raw[u][j] = __float_as_uint(l[i0 + j]);
              else raw[u][j >> 1] = (j & 1) ? (raw[u][j >> 1] & 0xFFFFu) | (uint32_t)l[i0 + j] << 16 : (raw[u][j >> 1] & 0xFFFF0000u) | l[i0 + j];
            }
      }
    }
  };
  int p0 = first + wave * 128;
  if (p0 < last) load(p0);
  for (; p0 < last; p0 += 512) {
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(raw[i >> 2][i & 3]);
      else v[i] = __uint_as_float((i & 1) ? raw[i >> 3][(i >> 1) & 3] & 0xFFFF0000u : raw[i >> 3][(i >> 1) & 3] << 16);
    }
    if (p0 + 512 < last) load(p0 + 512);
    float lm = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) lm = fmaxf(lm, v[i]);
    if (__any(!(lm < gate))) {
      const float most = wave_max(lm);
      if (most > s.m) {
        const float d = s.m > ninf ? fmaxf((s.m - most) * c, -200.0f) : 0.0f, f = exp2f(d);
        const float mine = lane == 0 ? (float)s.ones : 0.0f;  // the ones so far are below the new maximum (or as good as equal to it)
        E = f * fmaf(d, R + mine, E);
        R = f * (R + mine);
        s.ones = 0;
        s.m = most;
        gate = most - (0x1p-18f / c + fabsf(most) * 0x1p-22f);
      }
      const float at = s.m > ninf ? s.m : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float z = (v[i] - at) * c, e = __builtin_amdgcn_exp2f(z);
        const bool one = e == 1.0f;
        s.ones += __popcll(__ballot(one));
        R += one ? 0.0f : e;
        E = fmaf(e, fmaxf(z, -200.0f), E);
      }
    } else {
      float E1 = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float z = (v[i] - s.m) * c, e = __builtin_amdgcn_exp2f(z);
        R += e;
        E1 = fmaf(e, z, E1);
      }
      if (__any(E1 != E1)) {  // 0 times -inf: masked logits (or a NaN)
        E1 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float z = (v[i] - s.m) * c;
          E1 = fmaf(__builtin_amdgcn_exp2f(z), fmaxf(z, -200.0f), E1);
        }
      }
      E += E1;
    }
    if (t_piece >= p0 && t_piece < p0 + 128) {  // the target's own round
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int id = (p0 + 64 * (i / PV) + lane) * PV - skip + i % PV;
        s.rank += __popcll(__ballot(v[i] >= (id < t ? lt : above)));
      }
    } else {
      const float bar = p0 < t_piece ? lt : above;
#pragma unroll
      for (int i = 0; i < NV; ++i) s.rank += __popcll(__ballot(v[i] >= bar));
    }
    if (a.top > 0) {
      while (__any(lm >= least && lm > ninf)) {
        int k = NV;  // the first of this lane's values that is its largest
#pragma unroll
        for (int i = NV - 1; i >= 0; --i) k = v[i] == lm ? i : k;
        const int id = (p0 + 64 * (k / PV) + lane) * PV - skip + k % PV;
        const bool better = lm > ninf && before(lm, id, least, least_id);
        const uint64_t which = __ballot(better);
        if (which == 0) break;
        bool gone = better;
        if (__popcll(which) > kFewInserts) {  // every such lane's largest at once
          TopList some;
          if (better) some.v = lm, some.id = id;
          some.sort();
          best.merge(some.v, some.id);
        } else {
          const float most = wave_max(better ? lm : ninf);
          const int from = lane_of_max(better ? lm : ninf, id, most);
          best.insert(most, __builtin_amdgcn_readlane(id, from));
          gone = lane == from;
        }
        least = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(best.v), a.top - 1));
        least_id = __builtin_amdgcn_readlane(best.id, a.top - 1);
        if (gone) {
          lm = ninf;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            v[i] = i == k ? ninf : v[i];
            lm = fmaxf(lm, v[i]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    R += __shfl_xor(R, o);
    E += __shfl_xor(E, o);
  }
  s.R = R;
  s.E = E;
  if (lane == 0) sums_of[wave] = s;
  if (a.top > 0) merge_waves<4>(best, wave, list_v, list_id);
  else __syncthreads();
  if (wave != 0) return;
  s = sums_of[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) join(s, sums_of[w], c);
  // what the first piece holds before the row counted as masked logits of lower ids
  if (split == 0 && lt == ninf) s.rank -= skip;
  if (a.splits == 1) {
    finish_row(a, row, s, best, given, lt);
    return;
  }
  float* part = a.parts + (row * a.splits + split) * (8 + 2 * a.top);
  if (lane == 0) *reinterpret_cast<Sums*>(part) = s;
  if (lane < a.top) {
    part[8 + lane] = best.v;
    part[8 + a.top + lane] = __int_as_float(best.id);
  }
}

// The parts of a row: eight waves merge their alternatives, a wave taking every
// eighth part's, and one joins their sums.
template <typename T>
__global__ void __launch_bounds__(512) logprobs_join_kernel(LogprobArgs a) {
  constexpr int WAVES = 8, EACH = kSplitsMost / WAVES;
  __shared__ float list_v[WAVES][kTopMost];
  __shared__ int list_id[WAVES][kTopMost];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), size = 8 + 2 * a.top;
  const float* parts = a.parts + row * a.splits * size;
  const float c = a.inv_t * kLog2E;
  Sums s = no_sums();
  if (wave == 0 && lane < a.splits) s = *reinterpret_cast<const Sums*>(parts + lane * size);
  TopList best;
  if (a.top > 0) {
    TopList of[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if (wave + WAVES * i < a.splits && lane < a.top) {
        const float* p = parts + (wave + WAVES * i) * size + 8 + lane;
        of[i].v = p[0];
        of[i].id = __float_as_int(p[a.top]);
      }
    best = of[0];
#pragma unroll
    for (int i = 1; i < EACH; ++i)
      if (wave + WAVES * i < a.splits) best.merge(of[i].v, of[i].id);
    merge_waves<WAVES>(best, wave, list_v, list_id);
  }
  if (wave != 0) return;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {  // lane i takes lane i + o, in a fixed order
    Sums b;
    b.m = __shfl_down(s.m, o);
    b.R = __shfl_down(s.R, o);
    b.E = __shfl_down(s.E, o);
    b.ones = __shfl_down(s.ones, o);
    b.rank = __shfl_down(s.rank, o);
    if (lane < o) join(s, b, c);
  }
  s.m = __shfl(s.m, 0);
  s.R = __shfl(s.R, 0);
  s.E = __shfl(s.E, 0);
  s.ones = __shfl(s.ones, 0);
  s.rank = __shfl(s.rank, 0);
  const int32_t t = a.targets ? a.targets[row] : -1;
  const bool given = t >= 0 && t < a.V;
  const float lt = given ? logit(static_cast<const T*>(a.logits) + row * a.stride, t) : 0.0f;
  finish_row(a, row, s, best, given, lt);
}

// Parts of a row: enough workgroups to fill the card four times over (a workgroup
// holds 16 KB of loads in flight), a part being a round of its four waves at least.
static int logprob_splits(int dtype, int64_t tokens, int64_t vocab) {
  const int64_t rounds = (vocab + (dtype == FP4_DT_F32 ? 2047 : 4095)) / (dtype == FP4_DT_F32 ? 2048 : 4096);
  const int64_t wanted = (1024 + tokens - 1) / std::max<int64_t>(tokens, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({rounds, wanted, kSplitsMost}));
}
static size_t logprob_bytes(int64_t tokens, int splits, int top) { return splits == 1 ? 0 : sizeof(float) * (size_t)tokens * splits * (8 + 2 * top); }

struct LogprobGradArgs {
  const void* logits;
  int64_t stride, V;
  const int32_t* targets;
  const float *stats, *d_logprobs, *d_entropy;
  float inv_t;
  void* d_logits;
  int64_t d_stride;
  int splits;
};

// 2^t (A + B t) for all logits, the target's apart.  Bound by the bytes: pieces of
// 16 bytes where the rows of both sides lie alike, single values at their ends and
// where they do not.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(256) logprobs_grad_kernel(LogprobGradArgs a) {
  constexpr int PV = 16 / (int)sizeof(T);
  const int64_t row = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x - row * a.splits);
  const T* l = static_cast<const T*>(a.logits) + row * a.stride;
  T* d = static_cast<T*>(a.d_logits) + row * a.d_stride;
  const float R = a.stats[3 * row + 1], H = a.stats[3 * row + 2], Z = 1.0f + R;
  const bool none = Z == 0.0f;  // nothing left in the row
  const float m = none ? 0.0f : a.stats[3 * row];
  const int V = (int)a.V;
  const int32_t t = a.d_logprobs ? a.targets[row] : -1;
  const bool given = t >= 0 && t < V;
  const float glp = given ? a.d_logprobs[row] : 0.0f, gH = ENTROPY && a.d_entropy ? a.d_entropy[row] : 0.0f;
  const float logZ = none ? 0.0f : log1pf(R), scale = none ? 0.0f : a.inv_t / Z, c = a.inv_t * kLog2E;
  const float A = -scale * (ENTROPY ? glp + gH * (H - logZ) : glp), B = -scale * gH * kLn2;
  auto value = [&](float v) __attribute__((always_inline)) {
    const float z = (v - m) * c;
    float f = A;
    if constexpr (ENTROPY) f = fmaf(B, fmaxf(z, -200.0f), A);
    return __builtin_amdgcn_exp2f(z) * f;
  };
  auto target = [&](float v) __attribute__((always_inline)) {  // 1 - p_t without the subtraction
    const float z = (v - m) * a.inv_t, q = scale * (glp * (R - expm1f(z)));
    if constexpr (!ENTROPY) return q;
    const float f = gH * (fmaxf(z, -200.0f) + (H - logZ));
    return fmaf(-scale * f, __expf(z), q);
  };
  auto one = [&](int i) __attribute__((always_inline)) {
    const float v = logit(l, i), g = i == t ? target(v) : value(v);
    if constexpr (sizeof(T) == 2) d[i] = __builtin_bit_cast(uint16_t, (__bf16)g);
    else d[i] = g;
  };
  const int skip = (int)(((uintptr_t)l & 15) / sizeof(T));
  const int pieces = (V + skip + PV - 1) / PV, per = ((pieces + a.splits - 1) / a.splits + 255) / 256 * 256;
  const int last = min(pieces, (split + 1) * per);
  const bool alike = (((uintptr_t)l ^ (uintptr_t)d) & 15) == 0;
#pragma unroll 2
  for (int p = split * per + threadIdx.x; p < last; p += 256) {
    const int i0 = p * PV - skip;
    if (alike && i0 >= 0 && i0 + PV <= V) {
      const u32x4 raw = *reinterpret_cast<const u32x4*>(l + i0);
      float g[PV];
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        if constexpr (sizeof(T) == 4) g[j] = __uint_as_float(raw[j]);
        else g[j] = __uint_as_float((j & 1) ? raw[j >> 1] & 0xFFFF0000u : raw[j >> 1] << 16);
      }
      const bool has = given && (unsigned)(t - i0) < (unsigned)PV;
      float vt = 0.0f;
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        vt = j == t - i0 ? g[j] : vt;
        g[j] = value(g[j]);
      }
      if (has) {
        const float gt = target(vt);
#pragma unroll
        for (int j = 0; j < PV; ++j) g[j] = j == t - i0 ? gt : g[j];
      }
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          o[j] = __float_as_uint(g[j]);
        } else {
          const bf16x2_t pr{(__bf16)g[2 * j], (__bf16)g[2 * j + 1]};
          o[j] = __builtin_bit_cast(uint32_t, pr);
        }
      }
      *reinterpret_cast<u32x4*>(d + i0) = o;
    } else {
      for (int j = 0; j < PV; ++j)
        if (i0 + j >= 0 && i0 + j < V) one(i0 + j);
    }
  }
}

static int validate_logprobs(int dtype, int64_t tokens, int64_t vocab, int64_t stride, int top, float temperature) {
  if (dtype != FP4_DT_BF16 && dtype != FP4_DT_F32) return fail(FP4_ERR_INVALID_ARG, "logprobs: unknown dtype %d", dtype);
  if (tokens < 0 || vocab < 1) return fail(FP4_ERR_SHAPE, "logprobs: %lld rows of %lld logits", (long long)tokens, (long long)vocab);
  if (stride < vocab) return fail(FP4_ERR_SHAPE, "logprobs: rows of %lld logits at a stride of %lld", (long long)vocab, (long long)stride);
  if (vocab >= (int64_t)1 << 30 || tokens >= (int64_t)1 << 24 || stride >= (int64_t)1 << 40 || (double)tokens * stride > 0x1p46)
    return fail(FP4_ERR_UNSUPPORTED, "logprobs: 2^30 logits a row, 2^24 rows or more than 2^46 logits");
  if (top < 0 || top > kTopMost) return fail(FP4_ERR_INVALID_ARG, "logprobs: top = %d, 0 to %d expected", top, kTopMost);
  if (!(temperature > 0.0f && temperature < __builtin_huge_valf())) return fail(FP4_ERR_INVALID_ARG, "logprobs: temperature %g", (double)temperature);
  return FP4_OK;
}

}  // namespace fp4

using namespace fp4;

extern "C" {

int token_logprobs_workspace_size(int dtype, int64_t tokens, int64_t vocab, int top, size_t* bytes) {
  if (!bytes) return fail(FP4_ERR_INVALID_ARG, "null size pointer");
  FP4_CHECK(validate_logprobs(dtype, tokens, vocab, vocab, top, 1.0f));
  *bytes = logprob_bytes(tokens, logprob_splits(dtype, tokens, vocab), top);
  return FP4_OK;
}

int token_logprobs(const void* logits, int dtype, int64_t tokens, int64_t vocab, int64_t stride, const int32_t* targets, float temperature, int top,
                   float* logprobs, int32_t* ranks, int32_t* top_ids, float* top_logprobs, float* stats, void* workspace, size_t workspace_bytes,
                   void* stream) {
  FP4_CHECK(validate_logprobs(dtype, tokens, vocab, stride, top, temperature));
  if (tokens == 0) return FP4_OK;
  if (!logits || (top && (!top_ids || !top_logprobs)) || ((logprobs || ranks) && !targets)) return fail(FP4_ERR_INVALID_ARG, "logprobs: null pointer");
  if ((uintptr_t)logits % (dtype == FP4_DT_F32 ? 4 : 2) || (uintptr_t)targets % 4 || (uintptr_t)logprobs % 4 || (uintptr_t)ranks % 4 ||
      (uintptr_t)top_ids % 4 || (uintptr_t)top_logprobs % 4 || (uintptr_t)stats % 4)
    return fail(FP4_ERR_INVALID_ARG, "logprobs: misaligned pointer");
  const int splits = logprob_splits(dtype, tokens, vocab);
  const size_t need = logprob_bytes(tokens, splits, top);
  if (need) {
    if (!workspace || workspace_bytes < need) return fail(FP4_ERR_WORKSPACE, "logprobs: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "logprobs: misaligned workspace");
  }
  hipStream_t st = as_stream(stream);
  const LogprobArgs a{logits, stride, vocab, targets, 1.0f / temperature, top, splits, logprobs, ranks, top_ids, top_logprobs, stats, static_cast<float*>(workspace)};
  const dim3 grid((unsigned)(tokens * splits));
  if (dtype == FP4_DT_F32) hipLaunchKernelGGL(logprobs_kernel<float>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(logprobs_kernel<uint16_t>, grid, dim3(256), 0, st, a);
  FP4_CHECK(check_launch("token_logprobs"));
  if (splits == 1) return FP4_OK;
  if (dtype == FP4_DT_F32) hipLaunchKernelGGL(logprobs_join_kernel<float>, dim3((unsigned)tokens), dim3(512), 0, st, a);
  else hipLaunchKernelGGL(logprobs_join_kernel<uint16_t>, dim3((unsigned)tokens), dim3(512), 0, st, a);
  return check_launch("token_logprobs");
}

int token_logprobs_grad(const void* logits, int dtype, int64_t tokens, int64_t vocab, int64_t stride, const int32_t* targets, float temperature,
                        const float* stats, const float* d_logprobs, const float* d_entropy, void* d_logits, int64_t d_stride, void* stream) {
  FP4_CHECK(validate_logprobs(dtype, tokens, vocab, stride, 0, temperature));
  if (d_stride < vocab) return fail(FP4_ERR_SHAPE, "logprobs: gradients of %lld logits at a stride of %lld", (long long)vocab, (long long)d_stride);
  if (tokens == 0) return FP4_OK;
  if (!logits || !stats || !d_logits || (d_logprobs && !targets)) return fail(FP4_ERR_INVALID_ARG, "logprobs: null pointer");
  const uintptr_t size = dtype == FP4_DT_F32 ? 4 : 2;
  if ((uintptr_t)logits % size || (uintptr_t)d_logits % size || (uintptr_t)targets % 4 || (uintptr_t)stats % 4 || (uintptr_t)d_logprobs % 4 ||
      (uintptr_t)d_entropy % 4)
    return fail(FP4_ERR_INVALID_ARG, "logprobs: misaligned pointer");
  // parts of a row as in the forward pass, of four pieces a thread at least
  const int64_t pieces = (vocab + 7) / (dtype == FP4_DT_F32 ? 4 : 8) + 1;
  const int splits = (int)std::max<int64_t>(1, std::min<int64_t>((2048 + tokens - 1) / tokens, pieces / 1024));
  const LogprobGradArgs a{logits, stride, vocab, targets, stats, d_logprobs, d_entropy, 1.0f / temperature, d_logits, d_stride, splits};
  const dim3 grid((unsigned)(tokens * splits));
  hipStream_t st = as_stream(stream);
  if (dtype == FP4_DT_F32) {
    if (d_entropy) hipLaunchKernelGGL((logprobs_grad_kernel<float, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((logprobs_grad_kernel<float, false>), grid, dim3(256), 0, st, a);
  } else {
    if (d_entropy) hipLaunchKernelGGL((logprobs_grad_kernel<uint16_t, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((logprobs_grad_kernel<uint16_t, false>), grid, dim3(256), 0, st, a);
  }
  return check_launch("token_logprobs_grad");
}

}  // extern "C"
