// Routing of tokens to experts: the router's logits -> the top_k experts of
// each token and their weights (lora_route_experts).
//
// Page "spark_model/lora/expert_apply.rs" puts the router LoRA on the logits
// before the top-k; this is that top-k. Per token, in fp32:
//   s = softmax(x) or sigmoid(x);  c = s + bias
//   with groups: a group (E / groups consecutive experts) is worth its best c
//   or the sum of its two best; experts outside the top_groups groups drop out
//   ids = the top_k experts by c;  w = s[ids] (/ their sum) * scaling
// An expert whose logit or c is NaN or -inf is not available: it is never
// chosen, and where fewer than top_k are left the rest is id -1, weight 0.
// Equal c go to the lowest expert.
//
// The softmax's sum is formed in fp64 and rounded to fp32 once: the fp64
// sum of at most 1024 fp32 terms is so near the true one that its rounding
// does not depend on the order, so neither do the scores and the choice
// between two near experts.
#include "lora_common.h"
#include "experts.h"

namespace lora {

namespace {

constexpr float kInf = __builtin_inff();

// Order-preserving map of the fp32 choice score to u32; 0 is "not available".
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t u = __float_as_uint(c + 0.0f);   // -0 -> +0: equal scores, equal keys
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < W; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
#pragma unroll
  for (int d = 1; d < W; d <<= 1) v = min(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

}  // namespace

// L lanes per token (16 or 64), V consecutive experts per lane (E <= L * V).
template <typename T, int L, int V>
__global__ __launch_bounds__(256) void k_route(const void* __restrict__ logits_,
                                               const float* __restrict__ bias, RouteArgs a,
                                               uint32_t gmagic, int32_t* __restrict__ ids,
                                               float* __restrict__ weights) {
  const int l = threadIdx.x % L;
  const int t = blockIdx.x * (256 / L) + threadIdx.x / L;
  const bool live = t < a.T;
  const int64_t base = (int64_t)(live ? t : a.T - 1) * a.E;
  const int e0 = l * V;

  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = -kInf;
    if (e0 + i < a.E) {
      if constexpr (sizeof(T) == 2)
        x[i] = __uint_as_float((uint32_t)((const uint16_t*)logits_)[base + e0 + i] << 16);
      else
        x[i] = ((const float*)logits_)[base + e0 + i];
      x[i] = x[i] != x[i] ? -kInf : fminf(x[i], __FLT_MAX__);
    }
  }

  // scores (0 where not available) and the order keys of the choice scores
  float s[V];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 1.0f / (1.0f + expf(-x[i]));
  } else {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int d = 1; d < L; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = x[i] == -kInf ? 0.0f : expf(x[i] - m);
      z += (double)s[i];
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) z += __shfl_xor(z, d);
    const float zf = (float)z;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = zf > 0.0f ? s[i] / zf : 0.0f;
  }
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float c = s[i];
    if (bias && e0 + i < a.E) c += bias[e0 + i];
    key[i] = (x[i] == -kInf || c != c || c == -kInf) ? 0u : order_key(c);
  }

  if (a.top_groups < a.groups) {
    // lane g of the token's lanes keeps the worth of group g, then its rank
    // among the groups says whether it stays
    float worth = -kInf;
    int grp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) grp[i] = (int)(((uint64_t)(uint32_t)(e0 + i) * gmagic) >> 21);
    for (int g = 0; g < a.groups; ++g) {
      uint32_t b0 = 0, b1 = 0;   // two best keys of the group
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t q = grp[i] == g ? key[i] : 0u;
        b1 = max(b1, min(b0, q));
        b0 = max(b0, q);
      }
#pragma unroll
      for (int d = 1; d < L; d <<= 1) {
        const uint32_t o0 = (uint32_t)__shfl_xor((int)b0, d);
        const uint32_t o1 = (uint32_t)__shfl_xor((int)b1, d);
        b1 = max(max(b1, o1), min(b0, o0));
        b0 = max(b0, o0);
      }
      auto val = [](uint32_t k) {
        return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
      };
      float wv = b0 ? val(b0) : -kInf;
      if (a.sum2 && b0 && b1) wv += val(b1);
      if (l == g) worth = wv;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __shfl(worth, g, L);
      rank += (o > worth || (o == worth && g < l)) ? 1 : 0;
    }
    const uint64_t all = __ballot(l < a.groups && rank < a.top_groups);
    const uint32_t keep = (uint32_t)(all >> (lane_id() & ~(L - 1)));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!((keep >> (grp[i] & 31)) & 1u)) key[i] = 0u;
  }

  // top_k rounds: the largest key, its lowest expert, out with it
  int my_id = -1;        // lane r keeps the r-th choice (r and r + L where top_k > L)
  float my_w = 0.0f;
  int my_id2 = -1;
  float my_w2 = 0.0f;
  float total = 0.0f;
  for (int r = 0; r < a.k; ++r) {
    uint32_t best = 0;
    int bi = 0;
    float bs = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) { best = key[i]; bi = i; bs = s[i]; }
    const uint32_t top = row_max<L>(best);
    // consecutive experts per lane: the lowest lane that holds the largest
    // key holds the lowest expert of that key
    const uint32_t lane = row_min<L>(top != 0u && best == top ? (uint32_t)l : 0xffffu);
    const int src = lane == 0xffffu ? 0 : (int)lane;
    const int id = lane == 0xffffu ? -1 : __shfl(e0 + bi, src, L);
    const float w = lane == 0xffffu ? 0.0f : __shfl(bs, src, L);
    if ((uint32_t)l == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == bi) key[i] = 0u;
    }
    if (l == r) { my_id = id; my_w = w; }
    if (l + L == r) { my_id2 = id; my_w2 = w; }
    total += w;
  }
  const float div = a.renorm ? total : 1.0f;
  auto put = [&](int r, int id, float w) {
    if (live && r < a.k) {
      ids[(int64_t)t * a.k + r] = id;
      weights[(int64_t)t * a.k + r] = div > 0.0f ? w / div * a.scaling : 0.0f;
    }
  };
  put(l, my_id, my_w);
  if (L < kMaxTopK) put(l + L, my_id2, my_w2);
}

hipError_t launch_route_experts(int dtype, const void* logits, const float* bias,
                                const RouteArgs& a, int32_t* ids, float* weights,
                                hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  // e / (E / groups) as a product: exact for e < 1024 and group sizes <= 1024
  const uint32_t gs = (uint32_t)(a.E / a.groups);
  const uint32_t gmagic = (1u << 21) / gs + 1u;
#define LAUNCH(TT, LV, VV)                                                                     \
  hipLaunchKernelGGL((k_route<TT, LV, VV>), dim3((unsigned)((a.T + 256 / LV - 1) / (256 / LV))), \
                     dim3(256), 0, stream, logits, bias, a, gmagic, ids, weights)
#define BY_E(TT)                              \
  do {                                        \
    if (a.E <= 16) LAUNCH(TT, 16, 1);         \
    else if (a.E <= 32) LAUNCH(TT, 16, 2);    \
    else if (a.E <= 64) LAUNCH(TT, 16, 4);    \
    else if (a.E <= 128) LAUNCH(TT, 16, 8);   \
    else if (a.E <= 256) LAUNCH(TT, 16, 16);  \
    else if (a.E <= 512) LAUNCH(TT, 64, 8);   \
    else LAUNCH(TT, 64, 16);                  \
  } while (0)
  if (dtype == 1) BY_E(uint16_t); else BY_E(float);
#undef BY_E
#undef LAUNCH
  return hipGetLastError();
}

}  // namespace lora
