// The router's choice of experts on gfx950: scores of each token's logits,
// an optional bias for balance, a choice of expert groups, the top K experts
// and their weights.
//
//   score_e  = softmax(logits)_e or sigmoid(logit_e)
//   choice_e = score_e + bias_e where a bias is given, else the order of the
//              logits themselves (both scores grow with the logit)
//   group g  = the sum of its group_top best choices (scores without a bias)
//   chosen   = the K largest choices inside the topk_group largest groups,
//              equal ones in ascending index
//   weight   = score (without the bias), over the chosen ones' sum if asked,
//              times scale
//
// An expert whose logit is NaN or -inf, or whose biased choice is NaN or
// -inf, is never chosen; slots that no expert is left for hold id -1 and
// weight 0, which the layer treats as dropped.
//
// One wave64 owns a token: lane l holds experts l, l + 64, ...  Which expert
// is chosen hangs on the order of close scores, so choices are compared in 64
// bits.
#include "device_common.h"
#include "fp8moe.h"
#include "launch.h"

namespace fp8moe {

constexpr int kRouterWaves = 4;   // tokens a workgroup

__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  return __hiloint2double(__shfl_xor(__double2hiint(v), o), __shfl_xor(__double2loint(v), o));
}

// The largest (key, lowest index on ties) over the wave, in every lane.
__device__ __forceinline__ void wave_argmax(double& key, int& idx) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const double k2 = shfl_xor_f64(key, o);
    const int i2 = __shfl_xor(idx, o);
    if (k2 > key || (k2 == key && i2 < idx)) {
      key = k2;
      idx = i2;
    }
  }
}

template <int NV, bool BF16>
__global__ __launch_bounds__(64 * kRouterWaves) void router_topk_kernel(
    const void* __restrict__ logits, const float* __restrict__ bias, int T, int E, int K, int score, int n_group,
    int topk_group, int group_top, int renormalize, float scale, int32_t* __restrict__ ids,
    float* __restrict__ weights) {
  extern __shared__ double keys_lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave;
  const bool live = t < T;
  const double kNone = -__longlong_as_double(0x7ff0000000000000ll);

  float l[NV];
  float m = -__uint_as_float(0x7f800000u);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    l[i] = -__uint_as_float(0x7f800000u);
    if (live && e < E) {
      float v;
      if constexpr (BF16) v = bf16_to_f32(static_cast<const uint16_t*>(logits)[t * E + e]);
      else v = static_cast<const float*>(logits)[t * E + e];
      if (v == v) l[i] = v;
    }
    m = fmaxf(m, l[i]);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  double z = 0.0;
  double sc[NV], key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool none = l[i] == -__uint_as_float(0x7f800000u);
    if (score == FP8MOE_SCORE_SOFTMAX) sc[i] = none ? 0.0 : l[i] == m ? 1.0 : exp((double)l[i] - (double)m);
    else sc[i] = none ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
    z += sc[i];
  }
  if (score == FP8MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int o = 32; o; o >>= 1) z += shfl_xor_f64(z, o);
#pragma unroll
    for (int i = 0; i < NV; ++i) sc[i] = z > 0.0 ? sc[i] / z : 0.0;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    key[i] = kNone;
    if (e < E && l[i] != -__uint_as_float(0x7f800000u)) {
      const double k = bias ? sc[i] + (double)bias[e] : (double)l[i];
      if (k == k) key[i] = k;
    }
  }

  if (n_group > 1) {
    double* mine = keys_lds + wave * E;
    const bool by_score = bias == nullptr && group_top > 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E) mine[e] = key[i] == kNone ? kNone : by_score ? sc[i] : key[i];
    }
    __syncthreads();
    const int G = E / n_group;
    double first = kNone, second = kNone;
    if (lane < n_group) {
      for (int i = 0; i < G; ++i) {
        const double v = mine[lane * G + i];
        if (v > first) {
          second = first;
          first = v;
        } else if (v > second) {
          second = v;
        }
      }
    }
    const double total = group_top > 1 ? first + second : first;
    bool taken = lane >= n_group;
    uint64_t kept = 0;
    for (int j = 0; j < topk_group; ++j) {
      double k = taken ? kNone : total;
      int g = taken ? 64 + lane : lane;
      wave_argmax(k, g);
      kept |= 1ull << (g & 63);
      if (lane == g) taken = true;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !(kept >> (e / G) & 1)) key[i] = kNone;
    }
  }

  // slot j's expert and weight end in lane j
  int my_id = -1;
  double my_w = 0.0, sum = 0.0;
  for (int j = 0; j < K; ++j) {
    double k = kNone;
    int e = E + lane;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > k) {
        k = key[i];
        e = lane + 64 * i;
      }
    wave_argmax(k, e);
    if (e >= E) break;   // nothing left
    double w = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 64 * i) {
        key[i] = kNone;
        w = sc[i];
      }
    w = __hiloint2double(__shfl(__double2hiint(w), e & 63), __shfl(__double2loint(w), e & 63));
    sum += w;
    if (lane == j) {
      my_id = e;
      my_w = w;
    }
  }
  if (live && lane < K) {
    double w = my_w;
    if (renormalize) w = sum > 0.0 ? w / sum : 0.0;
    ids[t * K + lane] = my_id;
    weights[t * K + lane] = (float)(w * (double)scale);
  }
}

template <int NV>
static void router_launch(const void* logits, bool bf16, const float* bias, int T, int E, int K, int score,
                          int n_group, int topk_group, int group_top, bool renormalize, float scale, int32_t* ids,
                          float* weights, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)T + kRouterWaves - 1) / kRouterWaves)), block(64 * kRouterWaves);
  const size_t lds = n_group > 1 ? sizeof(double) * kRouterWaves * E : 0;   // at most 32 KB
  if (bf16)
    hipLaunchKernelGGL((router_topk_kernel<NV, true>), grid, block, lds, stream, logits, bias, T, E, K, score,
                       n_group, topk_group, group_top, (int)renormalize, scale, ids, weights);
  else
    hipLaunchKernelGGL((router_topk_kernel<NV, false>), grid, block, lds, stream, logits, bias, T, E, K, score,
                       n_group, topk_group, group_top, (int)renormalize, scale, ids, weights);
}

hipError_t launch_router_topk(const void* logits, bool bf16, const float* bias, int T, int E, int K, int score,
                              int n_group, int topk_group, int group_top, bool renormalize, float scale,
                              int32_t* ids, float* weights, hipStream_t stream) {
#define FP8MOE_ROUTER(NV)                                                                                         \
  router_launch<NV>(logits, bf16, bias, T, E, K, score, n_group, topk_group, group_top, renormalize, scale, ids, \
                    weights, stream)
  if (E <= 64) FP8MOE_ROUTER(1);
  else if (E <= 128) FP8MOE_ROUTER(2);
  else if (E <= 256) FP8MOE_ROUTER(4);
  else if (E <= 512) FP8MOE_ROUTER(8);
  else FP8MOE_ROUTER(16);
#undef FP8MOE_ROUTER
  return hipGetLastError();
}

}  // namespace fp8moe
