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
constexpr int kFound = 1024;     // logits of a workgroup that may reach the floor before they are taken out wave by wave
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

// The sums of the first N lanes (a power of two), for every lane: lane i takes lane i + N / 2 and so on, in a fixed order.
template <int N>
__device__ __forceinline__ void join_lanes(Sums& s, float c) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const Sums b{__shfl_down(s.m, o), __shfl_down(s.R, o), __shfl_down(s.E, o), __shfl_down(s.ones, o), __shfl_down(s.rank, o)};
    if (lane < o) join(s, b, c);
  }
  s = Sums{__shfl(s.m, 0), __shfl(s.R, 0), __shfl(s.E, 0), __shfl(s.ones, 0), __shfl(s.rank, 0)};
}

// The value of the lane whose number differs in the bits D: within rows of 16 lanes by DPP, across them by the row and
// half swaps of gfx950 (a shuffle through LDS takes a wave about three times as long).
template <int D>
__device__ __forceinline__ int lane_xor(int v) {
  if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);         // quads 1 0 3 2
  else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);    // quads 2 3 0 1
  else if constexpr (D == 4) return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true);  // eights turned round, quads too
  else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, true);   // rows turned by 8
  else if constexpr (D == 15) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // rows turned round
  else if constexpr (D == 16) {  // the odd rows of one copy change places with the even rows of the other
    const auto p = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
    return (threadIdx.x & 16) ? (int)p[0] : (int)p[1];
  } else if constexpr (D == 32) {
    const auto p = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
    return (threadIdx.x & 32) ? (int)p[0] : (int)p[1];
  } else {
    static_assert(D == 63, "a power of two, 15 or 63");
    return lane_xor<32>(lane_xor<16>(lane_xor<15>(v)));
  }
}
template <int D>
__device__ __forceinline__ float lane_xor(float v) { return __int_as_float(lane_xor<D>(__float_as_int(v))); }

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
  // One step of a sorting network: of each two lanes D apart the one with `first` gets the element that comes before.
  template <int D>
  __device__ __forceinline__ void exchange(bool first) {
    const float ov = lane_xor<D>(v);
    const int oid = lane_xor<D>(id);
    if (before(v, id, ov, oid) != first) v = ov, id = oid;
  }
  template <int N, int D>
  __device__ __forceinline__ void sort_steps() {
    const int lane = threadIdx.x & 63;
    exchange<D>(((lane & D) == 0) == ((lane & N) == 0));
    if constexpr (D > 1) sort_steps<N, D / 2>();
    else if constexpr (N < 64) sort_steps<2 * N, N>();
  }
  __device__ __forceinline__ void sort() { sort_steps<2, 1>(); }
  // The first 64 of both lists: of the j-th here and the j-th last there the better, which
  // rise and fall once, so that the network's last six steps sort them.
  __device__ __forceinline__ void merge(float ov, int oid) {
    ov = lane_xor<63>(ov);
    oid = lane_xor<63>(oid);
    if (before(ov, oid, v, id)) v = ov, id = oid;
    sort_steps<64, 32>();
  }
  __device__ __forceinline__ void insert(float cv, int cid) {  // cv, cid: the same for every lane
    const int lane = threadIdx.x & 63, at = __popcll(__ballot(before(v, id, cv, cid)));
    const int pv = from_lane_before(__float_as_int(v)), pid = from_lane_before(id);
    if (lane > at) v = __int_as_float(pv), id = pid;
    if (lane == at) v = cv, id = cid;
  }
};

// The wave's values, largest first (a sorting network; no NaN).
template <int N, int D>
__device__ __forceinline__ float sorted_steps(float v) {
  const int lane = threadIdx.x & 63;
  const float o = lane_xor<D>(v);
  v = ((lane & D) == 0) == ((lane & N) == 0) ? fmaxf(v, o) : fminf(v, o);
  if constexpr (D > 1) return sorted_steps<N, D / 2>(v);
  else if constexpr (N < 64) return sorted_steps<2 * N, N>(v);
  else return v;
}
__device__ __forceinline__ float sorted(float v) { return sorted_steps<2, 1>(v); }

// Of the lanes with the largest v the one with the lowest id.
__device__ __forceinline__ int lane_of_max(float v, int id, float most) {
  uint64_t which = __ballot(v == most);
  if (__popcll(which) > 1) {
    int low = v == most ? id : kNone;
    low = min(low, lane_xor<1>(low));
    low = min(low, lane_xor<2>(low));
    low = min(low, lane_xor<4>(low));
    low = min(low, lane_xor<8>(low));
    low = min(low, lane_xor<16>(low));
    low = min(low, lane_xor<32>(low));
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

// The part `split` of a row by a workgroup of WAVES waves.  A wave takes 2 x 64
// pieces of 16 bytes at a time, loaded one round ahead.  Its running maximum is one
// for all lanes, and a round whose logits all lie below it needs nothing but
// t = (l - m) c, 2^t, the two sums and the count of logits before the target, 10
// operations a bf16 value; a round that reaches it (few do) brings the sums to the
// new one and counts the exponentials that are 1.  Alternatives: a round with
// nothing above the wave's last one costs a comparison; else the lanes' largest values
// are taken out and inserted, or where they are many sorted and merged into the list.
// 4096 x 65536 bf16 in 101 us, 5.3 TB/s of logits.
//
// HELD rounds at most (0: any number): all are loaded at once and stay in registers, so that the workgroup knows its largest
// logit before any sum, and a floor that no alternative lies below: the top-th largest of its 64 groups' largest.
template <typename T, int WAVES, int HELD>
__global__ void __launch_bounds__(64 * WAVES) logprobs_kernel(LogprobArgs a) {
  constexpr int ROUND = 128 * WAVES;  // pieces
  constexpr int PV = 16 / (int)sizeof(T), NV = 2 * PV;  // values of a piece, of a lane's round
  __shared__ Sums sums_of[WAVES];
  __shared__ float list_v[WAVES][kTopMost];
  __shared__ int list_id[WAVES][kTopMost];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x - row * a.splits);
  const T* l = static_cast<const T*>(a.logits) + row * a.stride;
  const float ninf = -__builtin_huge_valf(), c = a.inv_t * kLog2E;
  // pieces start at multiples of 16 bytes: the first one `skip` values before the row
  const int skip = (int)(((uintptr_t)l & 15) / sizeof(T)), V = (int)a.V;
  const int pieces = (int)((a.V + skip + PV - 1) / PV), per = ((pieces + a.splits - 1) / a.splits + ROUND - 1) / ROUND * ROUND;
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
  float least = ninf, floor = ninf;       // the last alternative; none lies below `floor`
  int least_id = kNone;
  auto load = [&](u32x4 (&raw)[2], int p0) __attribute__((always_inline)) {
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
  auto values = [&](const u32x4 (&raw)[2], float (&v)[NV]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(raw[i >> 2][i & 3]);
      else v[i] = __uint_as_float((i & 1) ? raw[i >> 3][(i >> 1) & 3] & 0xFFFF0000u : raw[i >> 3][(i >> 1) & 3] << 16);
    }
  };
  auto gate_at = [&](float m) __attribute__((always_inline)) { return m - (0x1p-18f / c + fabsf(m) * 0x1p-22f); };
  auto add_up = [&](int p0, const float (&v)[NV]) __attribute__((always_inline)) {
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
        gate = gate_at(most);
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
  };
  // The round's alternatives into the wave's list.
  auto select = [&](int p0, float (&v)[NV]) __attribute__((always_inline)) {
    float lm = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) lm = fmaxf(lm, v[i]);
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
      if (HELD && !before(least, least_id, floor, kNone)) least = floor, least_id = kNone;
      if (gone) {
        lm = ninf;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          v[i] = i == k ? ninf : v[i];
          lm = fmaxf(lm, v[i]);
        }
      }
    }
  };
  const int p0 = first + wave * 128;
  float v[NV];
  if constexpr (HELD == 0) {
    u32x4 raw[2];
    if (p0 < last) load(raw, p0);
    for (int p = p0; p < last; p += ROUND) {
      values(raw, v);
      if (p + ROUND < last) load(raw, p + ROUND);
      add_up(p, v);
      if (a.top > 0) select(p, v);
    }
  } else {
    static_assert(WAVES * 4 == 64, "64 groups of 16 lanes");
    __shared__ float groups[64], found_v[kFound];
    __shared__ int found_id[kFound], found;
    u32x4 raw[HELD][2];
    float most = ninf;
    if (threadIdx.x == 0) found = 0;
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if (p0 + h * ROUND < last) load(raw[h], p0 + h * ROUND);
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if (p0 + h * ROUND < last) {
        values(raw[h], v);
#pragma unroll
        for (int i = 0; i < NV; ++i) most = fmaxf(most, v[i]);
      }
    most = fmaxf(most, lane_xor<1>(most));
    most = fmaxf(most, lane_xor<2>(most));
    most = fmaxf(most, lane_xor<4>(most));
    most = fmaxf(most, lane_xor<8>(most));
    if ((lane & 15) == 0) groups[wave * 4 + (lane >> 4)] = most;
    __syncthreads();
    const float mine = groups[lane];
    s.m = wave_max(mine);
    gate = gate_at(s.m);
    if (a.top > 0) {
      floor = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sorted(mine)), a.top - 1));
      least = floor;
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if (p0 + h * ROUND < last) {
        values(raw[h], v);
        add_up(p0 + h * ROUND, v);
        if (a.top > 0) {  // what reaches the floor, in any order
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const bool in = v[i] >= floor && v[i] > ninf;
            const uint64_t which = __ballot(in);
            if (which == 0) continue;
            int at = 0;
            if (lane == 0) at = atomicAdd(&found, __popcll(which));
            at = __builtin_amdgcn_readfirstlane(at) + __popcll(which & ((1ull << lane) - 1));
            if (in && at < kFound) {
              found_v[at] = v[i];
              found_id[at] = (p0 + h * ROUND + 64 * (i / PV) + lane) * PV - skip + i % PV;
            }
          }
        }
      }
    if (a.top > 0) {
      __syncthreads();
      const int n = found;
      if (n <= kFound) {
        if (wave == 0)
          for (int j = 0; j < n; j += 64) {
            TopList some;
            if (j + lane < n) some.v = found_v[j + lane], some.id = found_id[j + lane];
            some.sort();
            if (j == 0) best = some;
            else best.merge(some.v, some.id);
          }
      } else {  // many equal ones
#pragma unroll
        for (int h = 0; h < HELD; ++h)
          if (p0 + h * ROUND < last) {
            values(raw[h], v);
            select(p0 + h * ROUND, v);
          }
        merge_waves<WAVES>(best, wave, list_v, list_id);
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
  if (HELD == 0 && a.top > 0) merge_waves<WAVES>(best, wave, list_v, list_id);
  else __syncthreads();
  if (wave != 0) return;
  if constexpr (WAVES == 4) {
    s = sums_of[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) join(s, sums_of[w], c);
  } else {
    s = lane < WAVES ? sums_of[lane] : no_sums();
    join_lanes<WAVES>(s, c);
  }
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
  join_lanes<kSplitsMost>(s, c);
  const int32_t t = a.targets ? a.targets[row] : -1;
  const bool given = t >= 0 && t < a.V;
  const float lt = given ? logit(static_cast<const T*>(a.logits) + row * a.stride, t) : 0.0f;
  finish_row(a, row, s, best, given, lt);
}

// Few rows: 16 waves a workgroup with up to four rounds in registers, a row of more in parts of two as long as there are
// fewer workgroups than compute units.  Else four waves, and parts that fill the card four times over.  Measured (us, graph
// replays, registers and else): 1 x 32000 bf16 top 5 11.4 and 12.1, 16 x 131000 f32 top 20 14.9 and 19.8, 300 x 50000 bf16
// top 20 28.6 and 42.2, 1 x 131072 bf16 16.2 both, 100 x 50000 f32 without alternatives 12.6 and 11.5, 16 x 131072 f32 top 64
// 27.6 and 23.9: what loses little is left to one rule.
constexpr int kHeld = 4;
struct LogprobShape {
  bool held;
  int splits;
};
static LogprobShape logprob_shape(int dtype, int64_t tokens, int64_t vocab) {
  const int64_t rounds = (vocab + 7) / (dtype == FP4_DT_F32 ? 4 : 8) / 512 + 1, held = (rounds + 3) / 4;  // of 4 waves, of 16
  const int64_t room = std::max<int64_t>(1, 256 / std::max<int64_t>(tokens, 1));
  const int64_t parts = held <= kHeld ? 1 : std::min<int64_t>({(held + 1) / 2, room, kSplitsMost});
  if (tokens < 768 && (held + parts - 1) / parts <= kHeld) return {true, (int)parts};
  const int64_t wanted = (1024 + tokens - 1) / std::max<int64_t>(tokens, 1);
  return {false, (int)std::max<int64_t>(1, std::min<int64_t>({rounds, wanted, kSplitsMost}))};
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
// where they do not.  4096 x 65536 bf16 in 213 us, 5.0 TB/s read and written: a copy's rate.
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
  const float logZ = none ? 0.0f : log1pf(R), c = a.inv_t * kLog2E;
  // f / (Z T) by the mantissas first and the powers of two last: 1 / (Z T) alone may be a subnormal of few bits
  auto by_row = [&](float f) __attribute__((always_inline)) {
    const float q = __builtin_amdgcn_frexp_mantf(f) * __builtin_amdgcn_frexp_mantf(a.inv_t) / Z;
    return none ? 0.0f : ldexpf(q, __builtin_amdgcn_frexp_expf(f) + __builtin_amdgcn_frexp_expf(a.inv_t));
  };
  const float A = -by_row(ENTROPY ? glp + gH * (H - logZ) : glp), B = ENTROPY ? -by_row(gH) * kLn2 : 0.0f;
  auto value = [&](float v) __attribute__((always_inline)) {
    const float z = (v - m) * c;
    float f = A;
    if constexpr (ENTROPY) f = fmaf(B, fmaxf(z, -200.0f), A);
    return __builtin_amdgcn_exp2f(z) * f;
  };
  auto target = [&](float v) __attribute__((always_inline)) {  // 1 - p_t without the subtraction
    const float z = (v - m) * a.inv_t, q = none ? 0.0f : scale_by((R - expm1f(z)) / Z, glp, a.inv_t);
    if constexpr (!ENTROPY) return q;
    const float f = gH * (fmaxf(z, -200.0f) + (H - logZ));
    return fmaf(-by_row(f), __expf(z), q);
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
  // far below, 1 / T and what is made of it overflow, and 0 times that is NaN
  if (!(temperature >= 0x1p-100f && temperature < __builtin_huge_valf())) return fail(FP4_ERR_INVALID_ARG, "logprobs: temperature %g", (double)temperature);
  return FP4_OK;
}

}  // namespace fp4

using namespace fp4;

extern "C" {

int token_logprobs_workspace_size(int dtype, int64_t tokens, int64_t vocab, int top, size_t* bytes) {
  if (!bytes) return fail(FP4_ERR_INVALID_ARG, "null size pointer");
  FP4_CHECK(validate_logprobs(dtype, tokens, vocab, vocab, top, 1.0f));
  *bytes = logprob_bytes(tokens, logprob_shape(dtype, tokens, vocab).splits, top);
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
  const LogprobShape shape = logprob_shape(dtype, tokens, vocab);
  const int splits = shape.splits;
  const size_t need = logprob_bytes(tokens, splits, top);
  if (need) {
    if (!workspace || workspace_bytes < need) return fail(FP4_ERR_WORKSPACE, "logprobs: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((uintptr_t)workspace % 16) return fail(FP4_ERR_INVALID_ARG, "logprobs: misaligned workspace");
  }
  hipStream_t st = as_stream(stream);
  const LogprobArgs a{logits, stride, vocab, targets, 1.0f / temperature, top, splits, logprobs, ranks, top_ids, top_logprobs, stats, static_cast<float*>(workspace)};
  const dim3 grid((unsigned)(tokens * splits));
  if (!shape.held) {
    if (dtype == FP4_DT_F32) hipLaunchKernelGGL((logprobs_kernel<float, 4, 0>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((logprobs_kernel<uint16_t, 4, 0>), grid, dim3(256), 0, st, a);
  } else {
    if (dtype == FP4_DT_F32) hipLaunchKernelGGL((logprobs_kernel<float, 16, kHeld>), grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((logprobs_kernel<uint16_t, 16, kHeld>), grid, dim3(1024), 0, st, a);
  }
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
