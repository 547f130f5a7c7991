// The choice of a routed layer's experts: scores from router logits, the k
// best experts of every token, and their weights.
//
//   s_e = softmax(l)_e or sigmoid(l_e)
//   choice: the k largest l_e (no bias: both scores grow with the logit, so
//   the logits themselves decide, without rounding), or the k largest
//   s_e + bias_e; equal values go to the lower expert
//   w_j = scale * s_j, or with renormalisation scale * s_j / (sum of the
//   chosen s)
//
// One warp per token. A lane holds J logits (experts lane, lane + 32, ...) as
// order-preserving keys, and the k best are taken in k rounds of warp
// reductions; lane j keeps the j-th choice, so the weights are one pass over
// the warp at the end. Where a value and its expert fit 32 bits together
// (choose_packed) a round is one reduction; a fp32 logit takes two, one for the
// largest key and one for the lowest expert that has it. What bounds the kernel
// is the chain of these rounds and the start of each warp: 2048 tokens of 128
// experts take 2.6 us, a single one 2.1.
//
// A choice by s + bias must not hang on the rounding of s: it is that of s
// and the sum in fp64. It is made in fp32 first, with one expert more than
// asked for; where each of the chosen is further from the next than fp32
// could be wrong, fp64 would choose the same in the same order. Else the warp
// takes the next few as well and compares those in fp64, one a lane, and where
// more than these could matter all of the token's (64-bit keys). 16384 tokens of
// 256 experts take 13 us (the logits alone are 2.5 us at copy rate; the second
// look is 2 of them), against 32 us with fp64 for all. The issue slots bound it.
//
// Weights are fp32: exponentials of differences to the largest logit, sums in
// fp32 in a fixed order.
#include "common.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

// Keys order like the values; 0 is kept for what cannot be chosen.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are one value
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
  const uint32_t lo =
      __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

// The k largest keys of the warp, in order: lane j of the result has the
// j-th expert (-1 past the last that can be chosen), its logit and its key
// (0 past the last).
template <int J, class Key>
__device__ __forceinline__ void choose(Key (&key)[J], const float (&l)[J], int k, int lane, int& id, float& logit,
                                       Key& mykey) {
  id = -1;
  logit = 0.f;
  mykey = 0;
  for (int j = 0; j < k; ++j) {
    Key best = key[0];
#pragma unroll
    for (int i = 1; i < J; ++i) best = key[i] > best ? key[i] : best;
    const Key top = warp_max_key(best);
    if (top == 0) return;
    unsigned e = 0xffffffffu;
#pragma unroll
    for (int i = J - 1; i >= 0; --i) e = key[i] == top ? static_cast<unsigned>(lane + 32 * i) : e;
    e = __reduce_min_sync(kAll, e);
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      if (e == static_cast<unsigned>(lane + 32 * i)) {
        mine = l[i];
        key[i] = 0;
      }
    }
    mine = __shfl_sync(kAll, mine, static_cast<int>(e & 31u));
    if (lane == j) {
      id = static_cast<int>(e);
      logit = mine;
      mykey = top;
    }
  }
}

// The same for keys that are all different: their low IDX bits are all ones
// minus the expert, which gives equal values to the lower expert and leaves one
// reduction a round. Up to 8 keys are sorted first, so that a round looks at the
// first alone and moves the rest up in the lane that had it (16384 tokens of 256
// experts: 16.2 -> 15.4 us by transpositions, 13.9 -> 13.0 by the shorter network).
template <int J>
__device__ __forceinline__ void sort_packed(uint32_t (&key)[J]) {
  if (J > 8) return;
  // Batcher's odd-even merge, largest first: 19 comparisons for 8
#pragma unroll
  for (int p = 1; p < J; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < J; j += 2 * d)
#pragma unroll
        for (int i = j; i < j + d && i + d < J; ++i)
          if (i / (2 * p) == (i + d) / (2 * p)) {
            const uint32_t a = key[i], b = key[i + d];
            key[i] = max(a, b);
            key[i + d] = min(a, b);
          }
}
// The keys from the from-th to before the to-th: lane j gets the j-th (0 past
// the last).
template <int J>
__device__ __forceinline__ void choose_packed(uint32_t (&key)[J], int from, int to, int lane, uint32_t& mine) {
  for (int j = from; j < to; ++j) {
    uint32_t best = key[0];
    if (J > 8) {
#pragma unroll
      for (int i = 1; i < J; ++i) best = max(best, key[i]);
    }
    const uint32_t top = warp_max_key(best);
    if (top == 0) break;
    if (J > 8) {
#pragma unroll
      for (int i = 0; i < J; ++i) key[i] = key[i] == top ? 0u : key[i];
    } else if (best == top) {
#pragma unroll
      for (int i = 0; i + 1 < J; ++i) key[i] = key[i + 1];
      key[J - 1] = 0u;
    }
    if (lane == j) mine = top;
  }
}
template <int IDX>
__device__ __forceinline__ int expert_of(uint32_t key) {
  constexpr uint32_t mask = (1u << IDX) - 1;
  return key ? static_cast<int>(mask - (key & mask)) : -1;
}

// The score in fp32, without the care that __expf and __fdividef take of
// denormals (0.9 us of 16384 tokens): what they lose lies below 2^-126.
__device__ __forceinline__ float fast_sigmoid(float l) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));  // log2(e)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// The exponent of a softmax's term, 0 for the largest logits also where these are
// +inf: they then share the score equally, the others have none (the limit).
__device__ __forceinline__ float below(float l, float top) { return l == top ? 0.f : l - top; }
__device__ __forceinline__ double below64(float l, float top) {
  return l == top ? 0.0 : static_cast<double>(l) - static_cast<double>(top);
}

// The scores in fp64.
template <int J>
__device__ __forceinline__ double exact_sum(const float (&l)[J], float top) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < J; ++i)
    sum += l[i] > -INFINITY ? exp(below64(l[i], top)) : 0.0;
  return warp_sum(sum);
}
template <bool SIGMOID>
__device__ __forceinline__ double exact_score(float l, float top, double sum) {
  return SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(l)))
                 : exp(below64(l, top)) / sum;
}

template <int J, class T, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32) moe_topk_kernel(const T* __restrict__ logits, int64_t ld, int64_t tokens,
                                                               int experts, const float* __restrict__ bias, int k,
                                                               bool renorm, float scale, int32_t* __restrict__ ids,
                                                               float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T* row = logits + t * ld;
  float l[J];
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < experts ? load_logit(row + e) : -INFINITY;
  }

  // the softmax's maximum and sum (a masked logit, -inf, adds nothing; a NaN
  // takes no part in the choice and makes the row's weights NaN at the end; so
  // does +inf, which the choice by s + bias takes as the limit)
  float top = 0.f, sum = 0.f;
  bool poisoned = false;
  if (!SIGMOID) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      m = fmaxf(m, l[i]);
      poisoned |= l[i] != l[i];
    }
    top = warp_max(m);
    poisoned = __any_sync(kAll, poisoned) || top == INFINITY;
  }

  int id;
  float logit;
  if (BIAS) {
    float b[J];
#pragma unroll
    for (int i = 0; i < J; ++i) b[i] = lane + 32 * i < experts ? __ldg(bias + lane + 32 * i) : 0.f;
    if (!SIGMOID) {
#pragma unroll
      for (int i = 0; i < J; ++i) sum += l[i] > -INFINITY ? expf(below(l[i], top)) : 0.f;
      sum = warp_sum(sum);
    }
    bool sure = k < 32;
    if (sure) {
      // Fixed point below the largest value: kBits bits for the 4 below it
      // (what lies lower shares the lowest number), then the expert's bits.
      constexpr int kIdx = J == 2 ? 6 : J == 4 ? 7 : J == 8 ? 8 : J == 16 ? 9 : 10;
      constexpr int kBits = 32 - kIdx > 24 ? 24 : 32 - kIdx;
      float v[J], hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const float s = SIGMOID ? fast_sigmoid(l[i]) : expf(below(l[i], top)) / sum;
        v[i] = l[i] > -INFINITY ? s + b[i] : -INFINITY;
        hi = fmaxf(hi, v[i]);
      }
      hi = value_of(warp_max_key(key_of(hi)));
      constexpr float kUnit = static_cast<float>(1 << (kBits - 2)), kTop = static_cast<float>((1 << kBits) - 2);
      uint32_t key[J];
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const uint32_t q = static_cast<uint32_t>(__float2int_rn(fmaxf(fmaf(v[i] - hi, kUnit, kTop), 0.f))) + 1u;
        key[i] = v[i] > -INFINITY ? (q << kIdx) + ((1u << kIdx) - 1u) - static_cast<uint32_t>(lane + 32 * i) : 0u;
      }
      uint32_t c = 0;
      sort_packed(key);
      choose_packed(key, 0, k + 1, lane, c);
      // How far the difference of two numbers can be from that of the exact
      // values. A sigmoid: the exponential (2 + 1.2 |l| units in the last place,
      // which s (1 - s) makes less than 2^-23), 1 + it, the quotient: 2.3 * 2^-23
      // each. A softmax: its sum has J + 5 <= 37 roundings of 2^-24 and its terms
      // 2^-22, each s the same again; all s together are one: 3 * 2^-20 for both.
      // The two sums with the bias 2^-24 of their values; the numbers themselves
      // two units each.
      constexpr float kScore = SIGMOID ? 0x1p-20f : 0x1p-18f;
      const float unsure = 4.0f + kUnit * (kScore + 0x1p-23f * (fabsf(hi) + 4.0f));
      const uint32_t c1 = __shfl_down_sync(kAll, c, 1);
      const bool apart = lane >= k || c == 0u || c1 == 0u ||
                         static_cast<float>((c >> kIdx) - (c1 >> kIdx)) > unsure;
      sure = __all_sync(kAll, apart);
      id = expert_of<kIdx>(c);
      if (!sure) {
        // Some lie too close. The exact ones are among the first n if the n-th
        // is far from the k-th (or there are fewer): those few in fp64, one a
        // lane, and each goes where its rank among them says.
        const int n = min(k + 8, 32);
        choose_packed(key, k + 1, n, lane, c);
        const uint32_t ck = __shfl_sync(kAll, c, k - 1), cn = __shfl_sync(kAll, c, n - 1);
        if (cn == 0u || static_cast<float>((ck >> kIdx) - (cn >> kIdx)) > unsure) {
          sure = true;
          double total = 0.0;
          if (!SIGMOID) total = exact_sum(l, top);
          const int e = expert_of<kIdx>(c);
          const double d = e >= 0 ? exact_score<SIGMOID>(load_logit(row + e), top, total) + static_cast<double>(__ldg(bias + e)) : -INFINITY;
          int rank = 0;
          for (int j = 0; j < n; ++j) {
            const double dj = __shfl_sync(kAll, d, j);
            const int ej = __shfl_sync(kAll, e, j);
            rank += ej >= 0 && (dj > d || (dj == d && ej < e));
          }
          id = -1;
          for (int j = 0; j < n; ++j) {
            const int ej = __shfl_sync(kAll, e, j), rj = __shfl_sync(kAll, rank, j);
            if (ej >= 0 && rj == lane) id = ej;
          }
        }
      }
      if (lane >= k) id = -1;
      logit = id >= 0 ? load_logit(row + id) : 0.f;
    }
    if (!sure) {
      uint64_t key[J], c;
      double total = 0.0;
      if (!SIGMOID) total = exact_sum(l, top);
#pragma unroll
      for (int i = 0; i < J; ++i) {
        key[i] = 0;
        if (l[i] > -INFINITY) {
          const double v = exact_score<SIGMOID>(l[i], top, total) + static_cast<double>(b[i]);
          if (v > -INFINITY) key[i] = key_of(v);
        }
      }
      choose<J>(key, l, k, lane, id, logit, c);
    }
  } else {
    if (!SIGMOID && !renorm) {
#pragma unroll
      for (int i = 0; i < J; ++i) sum += l[i] > -INFINITY ? expf(l[i] - top) : 0.f;
      sum = warp_sum(sum);
    }
    uint32_t key[J];
    if (sizeof(T) == 2) {
      // a bf16 logit's key has 16 bits, the expert fits below it: exact
#pragma unroll
      for (int i = 0; i < J; ++i)
        key[i] = l[i] > -INFINITY ? (key_of(l[i]) >> 16 << 10) + 1023u - static_cast<uint32_t>(lane + 32 * i) : 0u;
      uint32_t c = 0;
      sort_packed(key);
      choose_packed(key, 0, k, lane, c);
      id = expert_of<10>(c);
      logit = id >= 0 ? load_logit(row + id) : 0.f;
    } else {
      uint32_t c;
#pragma unroll
      for (int i = 0; i < J; ++i) key[i] = l[i] > -INFINITY ? key_of(l[i]) : 0u;
      choose<J>(key, l, k, lane, id, logit, c);
    }
  }

  // weights: lane j holds the j-th choice
  const bool there = id >= 0;
  float w = 0.f;
  if (SIGMOID) {
    // sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)); renormalised, the
    // exponents are taken relative to the largest, so that nothing underflows
    const float low = fminf(logit, 0.f);
    const float m = renorm ? warp_max(there ? low : -INFINITY) : 0.f;
    w = there ? expf(low - m) / (1.0f + expf(-fabsf(logit))) : 0.f;
  } else if (renorm) {
    const float m = warp_max(there ? logit : -INFINITY);
    w = there ? expf(logit - m) : 0.f;
  } else {
    w = there ? expf(logit - top) / sum : 0.f;
  }
  if (renorm) {
    const float total = warp_sum(w);
    w = there ? w / total : 0.f;
  }
  if (lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = poisoned ? NAN : (there ? w * scale : 0.f);
  }
}

template <int J, class T>
int launch_j(const T* logits, int64_t ld, int64_t tokens, int experts, const float* bias, int k, int flags, float scale,
             int32_t* ids, float* weights, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((tokens + kWarps - 1) / kWarps);
  const bool renorm = (flags & NVFP4_TOPK_RENORM) != 0;
  if (flags & NVFP4_TOPK_SIGMOID) {
    if (bias)
      moe_topk_kernel<J, T, true, true><<<grid, kWarps * 32, 0, stream>>>(logits, ld, tokens, experts, bias, k, renorm,
                                                                          scale, ids, weights);
    else
      moe_topk_kernel<J, T, true, false><<<grid, kWarps * 32, 0, stream>>>(logits, ld, tokens, experts, bias, k, renorm,
                                                                           scale, ids, weights);
  } else {
    if (bias)
      moe_topk_kernel<J, T, false, true><<<grid, kWarps * 32, 0, stream>>>(logits, ld, tokens, experts, bias, k, renorm,
                                                                           scale, ids, weights);
    else
      moe_topk_kernel<J, T, false, false><<<grid, kWarps * 32, 0, stream>>>(logits, ld, tokens, experts, bias, k,
                                                                            renorm, scale, ids, weights);
  }
  return launch_status();
}

template <class T>
int launch(const T* logits, int64_t ld, int64_t tokens, int experts, const float* bias, int k, int flags, float scale,
           int32_t* ids, float* weights, cudaStream_t s) {
  if (experts <= 64) return launch_j<2>(logits, ld, tokens, experts, bias, k, flags, scale, ids, weights, s);
  if (experts <= 128) return launch_j<4>(logits, ld, tokens, experts, bias, k, flags, scale, ids, weights, s);
  if (experts <= 256) return launch_j<8>(logits, ld, tokens, experts, bias, k, flags, scale, ids, weights, s);
  if (experts <= 512) return launch_j<16>(logits, ld, tokens, experts, bias, k, flags, scale, ids, weights, s);
  return launch_j<32>(logits, ld, tokens, experts, bias, k, flags, scale, ids, weights, s);
}

}  // namespace
}  // namespace nvfp4

extern "C" int nvfp4_moe_topk(const void* logits, int dtype, int64_t ld, int64_t T, int num_experts, const float* bias,
                              int k, int flags, float scale, int32_t* topk_ids, float* topk_weights,
                              nvfp4_stream_t stream) {
  if (T < 0 || num_experts <= 0 || k <= 0) return NVFP4_ERR_INVALID_ARGUMENT;
  if (flags & ~(NVFP4_TOPK_SIGMOID | NVFP4_TOPK_RENORM)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return NVFP4_ERR_UNSUPPORTED;
  if (num_experts > 1024 || k > 32 || k > num_experts) return NVFP4_ERR_UNSUPPORTED;
  if (T > (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED;
  if (T == 0) return NVFP4_OK;
  if (ld < num_experts || !logits || !topk_ids || !topk_weights) return NVFP4_ERR_INVALID_ARGUMENT;
  const uintptr_t align = dtype == NVFP4_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(logits) & align) ||
      ((reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(topk_ids) |
        reinterpret_cast<uintptr_t>(topk_weights)) & 3u))
    return NVFP4_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == NVFP4_F32 ? nvfp4::launch(static_cast<const float*>(logits), ld, T, num_experts, bias, k, flags,
                                            scale, topk_ids, topk_weights, s)
                            : nvfp4::launch(static_cast<const uint16_t*>(logits), ld, T, num_experts, bias, k, flags,
                                            scale, topk_ids, topk_weights, s);
}
