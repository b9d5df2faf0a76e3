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

#include "fp4_device.h"
#include "host_common.h"
#include "moe_common.h"

namespace fp4 {

constexpr int kTopMost = 64;

struct LogprobArgs {
  const void* logits;
  int64_t stride, V;
  const int32_t* targets;
  float inv_t;
  int top;
  float* logprobs;      // [T]
  int32_t* ranks;       // [T]
  int32_t* top_ids;     // [T, top]
  float* top_logprobs;  // [T, top]
  float* stats;         // [T, 3]: M, R, H
};

__device__ __forceinline__ float logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit(const uint16_t* p, int64_t i) { return bf16_bits_to_f32(p[i]); }

template <typename F>
__device__ __forceinline__ float block_sum(float v, float* part, F op) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return op(op(part[0], part[1]), op(part[2], part[3]));
}

// a before b in the order of the alternatives: larger, or equal with the lower id
__device__ __forceinline__ bool before(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

template <typename T>
__global__ void __launch_bounds__(256) logprobs_kernel(LogprobArgs a) {
  __shared__ float part[4];
  __shared__ int ids[4];
  const int64_t row = blockIdx.x;
  const T* l = static_cast<const T*>(a.logits) + row * a.stride;
  const float ninf = -__builtin_huge_valf();
  const auto add = [](float x, float y) { return x + y; };
  float m = ninf;
  for (int64_t i = threadIdx.x; i < a.V; i += 256) m = fmaxf(m, logit(l, i));
  m = block_sum(m, part, [](float x, float y) { return fmaxf(x, y); });
  const float at = m == ninf ? 0.0f : m;
  const int32_t t = a.targets ? a.targets[row] : -1;
  const bool given = t >= 0 && t < a.V;
  const float lt = given ? logit(l, t) : 0.0f;
  float R = 0.0f, ones = 0.0f, E = 0.0f, rank = 0.0f;
  for (int64_t i = threadIdx.x; i < a.V; i += 256) {
    const float v = logit(l, i), z = (v - at) * a.inv_t, e = __expf(z);
    if (e == 1.0f) ones += 1.0f;
    else R += e;
    E += e * fmaxf(z, -1000.0f);
    rank += (float)(v > lt || (v == lt && i < t));
  }
  R = block_sum(R, part, add);
  ones = block_sum(ones, part, add);
  E = block_sum(E, part, add);
  rank = block_sum(rank, part, add);
  R = R + (ones - 1.0f);  // -1 for a row with nothing left
  const float Z = 1.0f + R, logZ = log1pf(R), H = Z == 0.0f ? 0.0f : logZ - E / Z;
  if (threadIdx.x == 0) {
    if (a.logprobs) a.logprobs[row] = !given ? 0.0f : Z == 0.0f ? ninf : (lt - at) * a.inv_t - logZ;
    if (a.ranks) a.ranks[row] = given ? (int32_t)rank : -1;
    if (a.stats) {
      a.stats[3 * row] = m;
      a.stats[3 * row + 1] = R;
      a.stats[3 * row + 2] = H;
    }
  }
  float last = __builtin_huge_valf();
  int last_id = -1;
  for (int j = 0; j < a.top; ++j) {
    float best = ninf;
    int id = -1;
    for (int64_t i = threadIdx.x; i < a.V; i += 256) {
      const float v = logit(l, i);
      if (v > ninf && before(last, last_id, v, (int)i) && (id < 0 || before(v, (int)i, best, id))) best = v, id = (int)i;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float ob = __shfl_xor(best, o);
      const int oi = __shfl_xor(id, o);
      if (oi >= 0 && (id < 0 || before(ob, oi, best, id))) best = ob, id = oi;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = best, ids[threadIdx.x >> 6] = id;
    __syncthreads();
    best = part[0], id = ids[0];
    for (int w = 1; w < 4; ++w)
      if (ids[w] >= 0 && (id < 0 || before(part[w], ids[w], best, id))) best = part[w], id = ids[w];
    if (threadIdx.x == 0) {
      a.top_ids[row * a.top + j] = id;
      a.top_logprobs[row * a.top + j] = id < 0 ? ninf : (best - at) * a.inv_t - logZ;
    }
    last = id < 0 ? ninf : best;
    last_id = id < 0 ? 0x7FFFFFFF : id;
  }
}

struct LogprobGradArgs {
  const void* logits;
  int64_t stride, V;
  const int32_t* targets;
  const float *stats, *d_logprobs, *d_entropy;
  float inv_t;
  void* d_logits;
  int64_t d_stride;
};

template <typename T>
__global__ void __launch_bounds__(256) logprobs_grad_kernel(LogprobGradArgs a) {
  const int64_t row = blockIdx.x;
  const T* l = static_cast<const T*>(a.logits) + row * a.stride;
  T* d = static_cast<T*>(a.d_logits) + row * a.d_stride;
  const float m = a.stats[3 * row], R = a.stats[3 * row + 1], H = a.stats[3 * row + 2], Z = 1.0f + R;
  const int32_t t = a.targets ? a.targets[row] : -1;
  const float glp = a.d_logprobs && t >= 0 && t < a.V ? a.d_logprobs[row] : 0.0f, gH = a.d_entropy ? a.d_entropy[row] : 0.0f;
  const float logZ = log1pf(R), inv = 1.0f / Z;
  for (int64_t i = threadIdx.x; i < a.V; i += 256) {
    float v = 0.0f;
    if (Z != 0.0f) {
      const float z = (logit(l, i) - m) * a.inv_t, p = __expf(z) * inv;
      v = glp * (i == t ? (R - expm1f(z)) * inv : -p) - gH * p * (fmaxf(z, -1000.0f) - logZ + H);
    }
    v *= a.inv_t;
    if constexpr (sizeof(T) == 2) d[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else d[i] = v;
  }
}

static int validate_logprobs(int dtype, int64_t tokens, int64_t vocab, int64_t stride, int top, float temperature) {
  if (dtype != FP4_DT_BF16 && dtype != FP4_DT_F32) return fail(FP4_ERR_INVALID_ARG, "logprobs: unknown dtype %d", dtype);
  if (tokens < 0 || vocab < 1) return fail(FP4_ERR_SHAPE, "logprobs: %lld rows of %lld logits", (long long)tokens, (long long)vocab);
  if (stride < vocab) return fail(FP4_ERR_SHAPE, "logprobs: rows of %lld logits at a stride of %lld", (long long)vocab, (long long)stride);
  if (vocab >= (int64_t)1 << 30 || tokens >= (int64_t)1 << 31 || stride >= (int64_t)1 << 40 || (double)tokens * stride > 0x1p46)
    return fail(FP4_ERR_UNSUPPORTED, "logprobs: 2^30 logits a row, 2^31 rows or more than 2^46 logits");
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
  *bytes = 0;
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
  const LogprobArgs a{logits, stride, vocab, targets, 1.0f / temperature, top, logprobs, ranks, top_ids, top_logprobs, stats};
  if (dtype == FP4_DT_F32) hipLaunchKernelGGL(logprobs_kernel<float>, dim3((unsigned)tokens), dim3(256), 0, as_stream(stream), a);
  else hipLaunchKernelGGL(logprobs_kernel<uint16_t>, dim3((unsigned)tokens), dim3(256), 0, as_stream(stream), a);
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
  const LogprobGradArgs a{logits, stride, vocab, targets, stats, d_logprobs, d_entropy, 1.0f / temperature, d_logits, d_stride};
  if (dtype == FP4_DT_F32) hipLaunchKernelGGL(logprobs_grad_kernel<float>, dim3((unsigned)tokens), dim3(256), 0, as_stream(stream), a);
  else hipLaunchKernelGGL(logprobs_grad_kernel<uint16_t>, dim3((unsigned)tokens), dim3(256), 0, as_stream(stream), a);
  return check_launch("token_logprobs_grad");
}

}  // extern "C"
