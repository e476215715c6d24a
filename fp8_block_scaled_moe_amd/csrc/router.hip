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
// Which expert is chosen hangs on the order of close scores, and is decided as
// if in 64 bits.  Two paths give the same choices, and weights to fp32's
// rounding:
//
// Exact path (route_exact): one wave64 per token, every score and choice in
// fp64.  As the only path it measured 31 us for 8192 tokens of 256 experts in
// groups, 121 us for 65537 tokens of 128.
//
// Fast path (route_fast): L = 16 or 64 lanes per token, a lane holds up to NV
// experts of one group, choices in fp32.  Each is a 32-bit key: the
// order-preserving bits of the choice with the lowest IB replaced by the
// complement of the expert's index, so keys are unique, the largest key is the
// winner, and it is taken out by comparing.
//   * bf16 logits without a bias: 16 value bits and the index fit, always exact;
//   * else further keys are taken until the next cannot reach the last slot's,
//     and the candidates are put in order by their full choices: the logits
//     themselves, or, where neighbours lie closer than fp32's error, the
//     biased scores in fp64;
//   * groups of which a kept and a left one are closer than the error of both
//     are ranked by fp64 totals of their best choices;
//   * what is left for the exact path: more close candidates than lanes, and
//     chosen experts or close groups whose scores are next to fp32's smallest.
// In a graph, us for 8192 tokens of 256 experts, top-8: softmax 6.4 (bf16 logits
// 5.3), sigmoid with bias 8.2, softmax with bias 12.7, groups by their maximum
// 7.3, by the sum of two 9.8 (14 while close ones went the exact way); 65537
// tokens of 128: 15.2, 2.5 TB/s; one token of 256: 3.4; 64: 3.7.
// Bound by the K rounds of maximum and removal and their shuffles, at few tokens
// by the launch and one trip to memory.
#include "device_common.h"
#include "fp8moe.h"
#include "launch_ops.h"

namespace fp8moe {

constexpr int kRouterWaves = 4;   // waves a workgroup

struct RouterArgs {
  const void* logits;
  const float* bias;
  int T, E, K, score, n_group, topk_group, group_top, renormalize;
  // fast path: each group of `per` experts has `lanes` lanes (a power of two;
  // without groups the row's all), a lane up to `width` of them, read in vectors
  // of vec (1, 4, 8)
  int per, lanes, width, vec;
  float scale;
  int32_t* ids;
  float* weights;
};

__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  return __hiloint2double(__shfl_xor(__double2hiint(v), o), __shfl_xor(__double2loint(v), o));
}

constexpr float kRouterInf = __builtin_huge_valf();

template <bool BF16>
__device__ __forceinline__ float router_logit(const void* logits, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(logits)[i]);
  else return static_cast<const float*>(logits)[i];
}

// LDS of a wave is read by its own lanes only: the writes ahead of it have to
// be in order, which the hardware keeps and this asks of the compiler.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The largest of v over the row's L lanes, in each of them: rotations inside
// 16 lanes, then row and half swaps.
template <int L>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));   // rotate by 8 of 16
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  if constexpr (L == 64) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(h[0], h[1]);
  }
  return v;
}

// Bits of a double that order as unsigned integers; 0 for "never chosen",
// which -inf stands for.  + 0: zeros of both signs are equal.
__device__ __forceinline__ uint64_t sortable64(double v) {
  if (!(v > -__longlong_as_double(0x7ff0000000000000ll))) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// The lowest index among the lanes with the largest key; -1 where none has one.
__device__ __forceinline__ int wave_argmax(uint64_t key, int idx) {
  const uint32_t hi = row_max_u32<64>((uint32_t)(key >> 32));
  const uint32_t lo = row_max_u32<64>((uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
  const bool best = key != 0 && key == ((uint64_t)hi << 32 | lo);
  return (int)(0xffffffffu - row_max_u32<64>(best ? 0xffffffffu - (uint32_t)idx : 0u));
}

// Token t by one wave: expert lane + 64 i in register i; mine: E doubles of LDS.
template <int NV, bool BF16>
__device__ __forceinline__ void route_exact(const RouterArgs& a, int64_t t, int lane, double* mine) {
  const int E = a.E, K = a.K, score = a.score, n_group = a.n_group, topk_group = a.topk_group,
            group_top = a.group_top, renormalize = a.renormalize;
  const float scale = a.scale;
  const float* bias = a.bias;
  int32_t* ids = a.ids;
  float* weights = a.weights;
  const double kNone = -__longlong_as_double(0x7ff0000000000000ll);

  float l[NV];
  float m = -kRouterInf;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    l[i] = -kRouterInf;
    if (e < E) {
      const float v = router_logit<BF16>(a.logits, t * E + e);
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
    const bool none = l[i] == -kRouterInf;
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
    if (e < E && l[i] != -kRouterInf) {
      const double k = bias ? sc[i] + (double)bias[e] : (double)l[i];
      if (k == k) key[i] = k;
    }
  }

  if (n_group > 1) {
    wave_lds_fence();   // a row before this one has been read
    const bool by_score = bias == nullptr && group_top > 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E) mine[e] = key[i] == kNone ? kNone : by_score ? sc[i] : key[i];
    }
    wave_lds_fence();
    const int G = E / n_group;
    double first = kNone, second = kNone;
    if (lane < n_group) {
      for (int i = 0; i < G; i += 8) {
        double v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = mine[min(lane * G + i + k, E - 1)];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const double u = i + k < G ? v[k] : kNone;
          second = fmax(second, fmin(first, u));
          first = fmax(first, u);
        }
      }
    }
    const double total = group_top > 1 ? (second > kNone ? first + second : kNone) : first;
    // groups of no choice come last, in ascending order, by a key below all others
    uint64_t gkey = lane < n_group ? (sortable64(total) ? sortable64(total) : 1) : 0;
    uint64_t kept = 0;
    for (int j = 0; j < topk_group; ++j) {
      const int g = wave_argmax(gkey, lane);
      kept |= 1ull << g;
      if (lane == g) gkey = 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !(kept >> (e / G) & 1)) key[i] = kNone;
    }
  }

  // slot j's expert and weight end in lane j
  uint64_t left[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) left[i] = sortable64(key[i]);
  int my_id = -1;
  double my_w = 0.0, sum = 0.0;
  for (int j = 0; j < K; ++j) {
    uint64_t k = left[0];
    int e = lane;
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (left[i] > k) {
        k = left[i];
        e = lane + 64 * i;
      }
    e = wave_argmax(k, e);
    if (e < 0) break;   // nothing left
    double w = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 64 * i) {
        left[i] = 0;
        w = sc[i];
      }
    w = __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(w), e & 63),
                         __builtin_amdgcn_readlane(__double2loint(w), e & 63));
    sum += w;
    if (lane == j) {
      my_id = e;
      my_w = w;
    }
  }
  if (lane < K) {
    double w = my_w;
    if (renormalize) w = sum > 0.0 ? w / sum : 0.0;
    ids[t * K + lane] = my_id;
    weights[t * K + lane] = (float)(w * (double)scale);
  }
}

// Sum and maximum of floats over the row's L lanes.
template <int L, bool MAX>
__device__ __forceinline__ float row_reduce_f32(float v) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    const float w = __shfl_xor(v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  return v;
}

// Bits of a float that order as unsigned integers.
__device__ __forceinline__ uint32_t sortable(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t s) {
  return __uint_as_float(s ^ ((int32_t)s < 0 ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float shfl_any(float v, int l) { return __shfl(v, l); }
__device__ __forceinline__ double shfl_any(double v, int l) {
  return __hiloint2double(__shfl(__double2hiint(v), l), __shfl(__double2loint(v), l));
}

// exp(x) for x <= 0 (a few ulp plus |x| 2^-24) and the logistic function on
// the transcendental units.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)); }

// The tokens of a wave, 64 / L of them; true in the lanes of a row that the
// exact path has to decide.
template <int L, int NV, bool BF16>
__device__ __forceinline__ bool route_fast(const RouterArgs& a, int64_t t, int lane) {
  constexpr int IB = L * NV <= 256 ? 8 : 10;         // index bits of a key
  constexpr uint32_t kIdx = (1u << IB) - 1;
  const int E = a.E, K = a.K;
  const int rl = lane & (L - 1);                      // lane of the row
  const int gl = a.lanes, log_gl = __ffs(gl) - 1;     // lanes of a group
  const int g = rl >> log_gl, in = rl & (gl - 1), per = a.per;   // the lane's group, the lane in it
  // the lane's experts: base + step i, i < count; read in vectors they are
  // neighbours, else the group's lanes read neighbours
  const bool wide = a.vec > 1;
  const int base = g * per + (wide ? in * a.width : in), step = wide ? 1 : gl;
  const int count = g >= a.n_group ? 0 : wide ? min(a.width, per - in * a.width) : (per - in + gl - 1) >> log_gl;
  const bool live = t < a.T;
  const bool biased = a.bias != nullptr, softmax = a.score == FP8MOE_SCORE_SOFTMAX;
  const bool sums = a.n_group > 1 && a.group_top > 1 && !biased;   // groups by sums of scores
  const float kNone = -kRouterInf;

  float x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = kNone;
  if (live) {
    const char* src = static_cast<const char*>(a.logits) + (t * E + base) * (BF16 ? 2 : 4);
    if (a.vec == 8 && BF16) {
      if constexpr (BF16 && NV % 8 == 0) {
#pragma unroll
        for (int i = 0; i < NV; i += 8) {
          if (i >= count) break;
          const uint4 v = *reinterpret_cast<const uint4*>(src + 2 * i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[i + 2 * k] = __uint_as_float(w[k] << 16);
            x[i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
          }
        }
      }
    } else if (wide) {
      if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          if (i >= count) break;
          const uint2 v = *reinterpret_cast<const uint2*>(src + 2 * i);
          x[i] = __uint_as_float(v.x << 16);
          x[i + 1] = __uint_as_float(v.x & 0xffff0000u);
          x[i + 2] = __uint_as_float(v.y << 16);
          x[i + 3] = __uint_as_float(v.y & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          if (i >= count) break;
          const float4 v = *reinterpret_cast<const float4*>(src + 4 * i);
          x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < count) x[i] = router_logit<BF16>(a.logits, t * E + base + i * step);
    }
  }
  float m = kNone;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = x[i] == x[i] ? x[i] : kNone;
    m = fmaxf(m, x[i]);
  }
  // softmax: the row's maximum and sum; scores only where choices need them
  float z = 1.f;
  const bool scored = biased || sums;
  if (softmax) {
    m = row_reduce_f32<L, true>(m);
    if (scored || !a.renormalize) {
      float part[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (x[i] > kNone) part[i & 1] += x[i] == m ? 1.f : fast_exp(x[i] - m);
      z = row_reduce_f32<L, false>(part[0] + part[1]);
    }
  }
  const float zinv = 1.0f / z;
  auto score_of = [&](float v) __attribute__((always_inline)) -> float {
    if (v == kNone) return 0.f;
    return softmax ? (v == m ? 1.f : fast_exp(v - m)) * zinv : fast_sigmoid(v);
  };

  // Scores in fp64, for choices that fp32 cannot tell apart; a softmax's take the
  // row's sum in fp64, made where first needed.
  double z64 = 0.0;
  auto need_z64 = [&]() __attribute__((always_inline)) {
    if (!softmax || z64 != 0.0) return;
    for (int i = 0; i < a.width; ++i) {
      const float v = live && i < count ? router_logit<BF16>(a.logits, t * E + base + i * step) : kNone;
      if (v > kNone) z64 += v == m ? 1.0 : exp((double)v - (double)m);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) z64 += shfl_xor_f64(z64, o);
  };
  auto score64 = [&](float v) __attribute__((always_inline)) -> double {
    return softmax ? (v == m ? 1.0 : exp((double)v - (double)m)) / z64 : 1.0 / (1.0 + exp(-(double)v));
  };

  // choices: x itself without a bias; groups by sums look at the scores
  bool unsure = false;
  float c[NV];
  if (biased) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      if (wide && i < count) {
        const float4 v = *reinterpret_cast<const float4*>(a.bias + base + i);
        b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
      } else if (!wide) {
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = i + k < count ? a.bias[base + (i + k) * step] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = score_of(x[i + k]) + b[k];
        c[i + k] = x[i + k] > kNone && v == v ? v : kNone;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = x[i];
  }
  // Error of a choice c of score s, with margin: the logistic function is
  // within 2^-22, a softmax's score, of a logit d below the row's largest, within
  // 2^-19 + 2.25 d 2^-24 of itself (a sum of up to twice 16 terms a lane and 4
  // levels of lanes, or twice 8 and 6, and the exponential's argument), and the
  // bias adds half a step of c.  s = 1 and d = 0 bound every score.
  auto choice_tol = [&](float s, float c, float d) __attribute__((always_inline)) -> float {
    return (softmax ? s * (0x1p-18f + d * 0x1p-22f) : 0x1p-21f) + fabsf(c) * 0x1p-22f;
  };

  if (a.n_group > 1) {
    float first = kNone, second = kNone;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float v = sums ? (c[i] > kNone ? score_of(c[i]) : kNone) : c[i];
      second = fmaxf(second, fminf(first, v));
      first = fmaxf(first, v);
    }
    for (int o = 1; o < gl; o <<= 1) {
      const float f2 = __shfl_xor(first, o), s2 = __shfl_xor(second, o);
      second = fmaxf(fmaxf(second, s2), fminf(first, f2));
      first = fmaxf(first, f2);
    }
    const float total = a.group_top > 1 ? (second > kNone ? first + second : kNone) : first;
    // rank of the lane's group, and the distance of kept and left groups
    int rank = 0;
    for (int h = 0; h < a.n_group; ++h) {
      const float other = __shfl(total, (lane & ~(L - 1)) + h * gl);
      rank += other > total || (other == total && h < g);
    }
    bool keep = rank < a.topk_group;
    if (biased || sums) {
      const bool real = rl < a.n_group * gl;   // lanes of a group
      const float worst = -row_reduce_f32<L, true>(keep && real ? -total : kNone);
      const float best = row_reduce_f32<L, true>(keep || !real ? kNone : total);
      // two choices each (the tolerance has a margin of two), which may be far
      // larger than their sum; scores without a bias carry their argument's
      // roundings relative to themselves: two of |x| 2^-24 and log2 e's own, and a
      // softmax's |x - m| is up to 2 far
      float far = 0.f, tol;
      if (sums) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (fabsf(x[i]) < kRouterInf) far = fmaxf(far, fabsf(x[i]));
        tol = ((softmax ? 5.f : 2.f) * row_reduce_f32<L, true>(far) + 32.f) * 0x1p-23f * fabsf(worst);
      } else {
        if (first > kNone) far = fabsf(first);
        if (a.group_top > 1 && second > kNone) far += fabsf(second);
        tol = 2.f * choice_tol(1.f, row_reduce_f32<L, true>(far), 0.f);
      }
      const bool close = a.topk_group < a.n_group && best > kNone && !(worst - best > tol);
      // (sums of scores next to fp32's smallest have no relative bound)
      if (sums) unsure = close && worst < 0x1p-100f;
      if (__ballot(close && !unsure)) {
        need_z64();
        // Groups next to the border between kept and left ones are ranked by
        // their fp64 totals, from those of their choices that may be among the
        // largest; the others' places are certain.
        const bool border = close && real && !((keep ? total - best : worst - total) > tol);
        const float least = (a.group_top > 1 ? second : first) - tol;
        uint32_t able = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (border && c[i] > kNone && !((sums ? score_of(c[i]) : c[i]) < least)) able |= 1u << i;
        const double kNone64 = -__longlong_as_double(0x7ff0000000000000ll);
        double f64 = kNone64, s64 = kNone64;
        while (__ballot(able != 0)) {
          double u = kNone64;
          if (able != 0) {
            const int e = base + (__ffs(able) - 1) * step;
            able &= able - 1;
            u = score64(router_logit<BF16>(a.logits, t * E + e));
            if (biased) u += (double)a.bias[e];
          }
          s64 = fmax(s64, fmin(f64, u));
          f64 = fmax(f64, u);
        }
        for (int o = 1; o < gl; o <<= 1) {
          const double f2 = shfl_xor_f64(f64, o), s2 = shfl_xor_f64(s64, o);
          s64 = fmax(fmax(s64, s2), fmin(f64, f2));
          f64 = fmax(f64, f2);
        }
        const double sum64 = a.group_top == 1 ? f64 : s64 > kNone64 ? f64 + s64 : kNone64;   // no inf - inf
        const double total64 = border ? sum64 : (double)total;
        int rank64 = 0;
        for (int h = 0; h < a.n_group; ++h) {
          const double other = shfl_any(total64, (lane & ~(L - 1)) + h * gl);
          rank64 += other > total64 || (other == total64 && h < g);
        }
        if (close) keep = rank64 < a.topk_group;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!keep) c[i] = kNone;
  }

  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)   // + 0: zeros of both signs are equal
    key[i] = c[i] > kNone ? (sortable(c[i] + 0.f) & ~kIdx) | (kIdx - (uint32_t)(base + i * step)) : 0u;
  const bool cut = !BF16 || biased;   // keys hold a part of the choice
  uint32_t mine = 0, last = 0;
  auto take = [&](int j) __attribute__((always_inline)) {
    uint32_t w = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) w = max(w, key[i]);
    w = row_max_u32<L>(w);
    if (rl == j) mine = w;
    last = w;
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = key[i] == w ? 0u : key[i];
  };
  for (int j = 0; j < K; ++j) take(j);
  int taken = K;
  if (cut) {
    // Further candidates, until the last one's largest possible choice lies
    // below the smallest of slot K - 1's by more than both errors: the K best
    // are then among them.
    const uint32_t kth = last;
    const float kmin = key_value(kth & ~kIdx);
    const float margin = biased ? 2.f * choice_tol(1.f, kmin, 0.f) : 0.f;
    bool open = kth != 0;
    while (taken < L - 1 && __ballot(open)) {
      take(taken++);
      open = open && last != 0 && !(key_value(last | kIdx) < kmin - margin);
    }
    unsure = unsure || open;
  }
  int e = mine ? (int)(kIdx - (mine & kIdx)) : -1;
  float v = e >= 0 ? router_logit<BF16>(a.logits, t * E + e) : kNone;

  if (cut) {
    // candidates in the order of their choices (nearly so already): odd-even
    // exchanges until no neighbours are out of order
    auto sort = [&](auto ch) __attribute__((always_inline)) {
      for (int pass = 0; pass < L; ++pass) {
        const auto ch2 = shfl_any(ch, lane + 1);
        const int e2 = __shfl(e, lane + 1);
        const bool wrong = rl + 1 < taken && e2 >= 0 && (ch2 > ch || (ch2 == ch && e2 < e));
        if (!__ballot(wrong)) break;
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          const bool left = ((rl ^ odd) & 1) == 0;
          const int p = left ? lane + 1 : lane - 1, pr = left ? rl + 1 : rl - 1;
          const auto pch = shfl_any(ch, p);
          const float pv = __shfl(v, p);
          const int pe = __shfl(e, p);
          if (pr >= 0 && pr < taken && rl < taken && pe >= 0 && e >= 0) {
            const bool partner_first = pch > ch || (pch == ch && pe < e);
            if (left ? partner_first : !partner_first) {
              ch = pch;
              v = pv;
              e = pe;
            }
          }
        }
      }
      return ch;
    };
    if (!biased) {
      sort(v);
    } else {
      const float ch = sort(e >= 0 ? score_of(v) + a.bias[e] : kNone);
      const float tol = e >= 0 ? choice_tol(score_of(v), ch, m - v) : 0.f;
      const float ch2 = __shfl(ch, lane + 1), tol2 = __shfl(tol, lane + 1);
      const int e2 = __shfl(e, lane + 1);
      // (a softmax's errors grow with the score: a choice behind slot K - 1 may be
      // less sure than its neighbours)
      const bool close = (softmax || rl < K) && rl + 1 < taken && e2 >= 0 && !(ch - ch2 > tol + tol2);
      if (__ballot(close)) {
        // neighbours too close for fp32: in the order of their fp64 choices
        need_z64();
        sort(e >= 0 ? score64(v) + (double)a.bias[e] : -(double)kRouterInf);
      }
    }
  }

  float w = rl < K && e >= 0 ? (softmax ? (v == m ? 1.f : expf(v - m)) * zinv : 1.0f / (1.0f + expf(-v))) : 0.f;
  // next to fp32's smallest a score has lost bits, or all of them, which the sum
  // or the scale may bring back (logistic function below about -69; a softmax
  // whose choices lie as far below the row's largest logit)
  if (rl < K && e >= 0 && w < 0x1p-100f) unsure = true;
  if (a.renormalize) {
    const float sum = row_reduce_f32<L, false>(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  // one lane's doubt is the row's
  unsure = row_max_u32<L>(unsure ? 1u : 0u) != 0;
  if (live && rl < K && !unsure) {
    a.ids[t * K + rl] = e;
    a.weights[t * K + rl] = w * a.scale;
  }
  return live && unsure;
}

// FAST: the fast path, then the exact one for the rows it leaves; else the
// exact path alone.  PLAIN: neither bias nor groups, with nothing kept in
// registers for them (65537 tokens of 128 experts: 17.1 -> 15.8 us).
template <int L, int NV, bool BF16, bool FAST, bool PLAIN>
__global__ __launch_bounds__(64 * kRouterWaves) void router_topk_kernel(RouterArgs a) {
  extern __shared__ double keys_lds[];
  if constexpr (PLAIN) {
    a.bias = nullptr;
    a.n_group = a.topk_group = a.group_top = 1;
    a.per = a.E;
    a.lanes = L;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double* mine = keys_lds + wave * a.E;
  constexpr int ENV = (L * NV + 63) / 64;   // experts of a lane on the exact path
  const int64_t t0 = ((int64_t)blockIdx.x * kRouterWaves + wave) * (FAST ? 64 / L : 1);
  if constexpr (FAST) {
    const uint64_t left = __ballot(route_fast<L, NV, BF16>(a, t0 + lane / L, lane));
    if (left == 0) return;
    for (int r = 0; r < 64 / L; ++r)
      if (left >> (r * L) & 1) route_exact<ENV, BF16>(a, t0 + r, lane, mine);
  } else {
    if (t0 < a.T) route_exact<ENV, BF16>(a, t0, lane, mine);
  }
}

template <int L, int NV, bool FAST>
static void router_launch(const RouterArgs& a, bool bf16, hipStream_t stream) {
  constexpr int rows = kRouterWaves * (FAST ? 64 / L : 1);
  const dim3 grid((unsigned)(((int64_t)a.T + rows - 1) / rows)), block(64 * kRouterWaves);
  const size_t lds = a.n_group > 1 ? sizeof(double) * kRouterWaves * a.E : 0;   // at most 32 KB
  if constexpr (FAST) {
    if (a.bias == nullptr && a.n_group == 1) {
      if (bf16) hipLaunchKernelGGL((router_topk_kernel<L, NV, true, true, true>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((router_topk_kernel<L, NV, false, true, true>), grid, block, 0, stream, a);
      return;
    }
  }
  if (bf16) hipLaunchKernelGGL((router_topk_kernel<L, NV, true, FAST, false>), grid, block, lds, stream, a);
  else hipLaunchKernelGGL((router_topk_kernel<L, NV, false, FAST, false>), grid, block, lds, stream, a);
}

hipError_t launch_router_topk(const void* logits, bool bf16, const float* bias, int T, int E, int K, int score,
                              int n_group, int topk_group, int group_top, bool renormalize, float scale,
                              int32_t* ids, float* weights, hipStream_t stream) {
  // The fast path's rows: 16 lanes, or 64: beyond 512 experts, 14 slots (at
  // least one further candidate has a lane) or 16 groups, and, from 129 experts
  // on, where the tokens are few: fewer values a lane are the shorter way until
  // the waves queue.  16 and 64 lanes, us, fp32 softmax | biased sigmoid: 256
  // experts, T=64 5.2, 4.0 | 6.5, 4.4; T=4096 6.0, 5.7 | 7.4, 6.6; T=8192 6.6,
  // 8.4 | 8.2, 9.8.  512 experts, T=64 7.6, 4.6; T=8192 11.0, 10.4; T=16384
  // 15.5, 17.6.  128 experts, T=64 4.3, 4.2; T=2048 4.5, 4.7.
  const bool few = E > 128 && T <= 16 * E;
  const int L = !few && E <= 512 && K < 15 && n_group <= 16 ? 16 : 64;
  int NV = L == 16 ? (E <= 64 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : 32) : E <= 256 ? 4 : E <= 512 ? 8 : 16;
  const int per = E / n_group;
  int lanes = L;
  while (lanes * n_group > L) lanes /= 2;
  const bool aligned = (uintptr_t)logits % 16 == 0 && (uintptr_t)bias % 16 == 0;
  const int vec = !aligned || per % 4 ? 1 : per % 8 || NV % 8 ? 4 : 8;
  const int share = (per + lanes - 1) / lanes;
  const int width = (share + vec - 1) / vec * vec;
  while (NV < width && NV < (L == 16 ? 32 : 16)) NV *= 2;   // groups of a size that leaves lanes empty
  const bool fast = K < L - 1 && width <= NV;
  const RouterArgs a{logits, bias, T, E, K, score, n_group, topk_group, group_top, (int)renormalize,
                     per, lanes, width, vec, scale, ids, weights};
  if (fast) {
    if (L == 16) {
      if (NV == 4) router_launch<16, 4, true>(a, bf16, stream);
      else if (NV == 8) router_launch<16, 8, true>(a, bf16, stream);
      else if (NV == 16) router_launch<16, 16, true>(a, bf16, stream);
      else router_launch<16, 32, true>(a, bf16, stream);
    } else {
      if (NV == 4) router_launch<64, 4, true>(a, bf16, stream);
      else if (NV == 8) router_launch<64, 8, true>(a, bf16, stream);
      else router_launch<64, 16, true>(a, bf16, stream);
    }
  } else {
    if (E <= 64) router_launch<16, 4, false>(a, bf16, stream);
    else if (E <= 128) router_launch<16, 8, false>(a, bf16, stream);
    else if (E <= 256) router_launch<16, 16, false>(a, bf16, stream);
    else if (E <= 512) router_launch<64, 8, false>(a, bf16, stream);
    else router_launch<64, 16, false>(a, bf16, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8moe
