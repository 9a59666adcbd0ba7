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
// between two near experts. The same holds for a sigmoid, which is one
// expression per expert.
//
// What bounds it: issued instructions, not bytes. 8192 tokens x 256 experts,
// top-8 of 4 of 8 groups, fp32: 7.7 us for 8.9 MB (1.9 us at the copy rate),
// of which 0.25 us a round of the top-k, 1.1 the groups. 16 lanes hold a token
// of up to 256 experts, so that the reductions stay in a row of lanes (DPP; by way
// of LDS shuffles with a wave's 64 lanes a row the same took 19 us) and a
// wave does 4 tokens at a time; 64 lanes hold it past that. One token of 64
// experts: 2.4 us on the GPU, the least that a launch takes.
#include <type_traits>
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

// v of the lane N places before in its row of 16 lanes (a rotation). Every
// lane has a source, so the old value and the bound never count; as 0 and
// true they let the compiler fold the move into the operation on it.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
  return dpp<0x120 | N>(v);
}
template <int N>
__device__ __forceinline__ float ror(float v) {
  return __uint_as_float(ror<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ double ror(double v) {
  const u32x2 u = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{ror<N>(u.x), ror<N>(u.y)});
}

// op over the L lanes (16 or 64) of a token, the result in all of them.
template <int L, typename T, typename Op>
__device__ __forceinline__ T over_lanes(T v, Op op) {
  v = op(v, ror<8>(v));
  v = op(v, ror<4>(v));
  v = op(v, ror<2>(v));
  v = op(v, ror<1>(v));
  if constexpr (L == 64) {
    v = op(v, __shfl_xor(v, 16));
    v = op(v, __shfl_xor(v, 32));
  }
  return v;
}

// b0 >= b1 become the two largest of b0, b1 and k; b1 their median.
__device__ __forceinline__ void two_largest(uint32_t& b0, uint32_t& b1, uint32_t k) {
  b1 = max(min(b0, b1), min(max(b0, b1), k));
  b0 = max(b0, k);
}

// The two largest of the keys of `per` (1 to 16, a power of two) lanes side by
// side, from each lane's two largest, in all of them: lanes 1 and 2 apart, then
// the mirrors of 8 and of 16 lanes, whose halves hold the same by then.
__device__ __forceinline__ void best_two(uint32_t& b0, uint32_t& b1, int per) {
  auto merge = [&](uint32_t o0, uint32_t o1) {
    b1 = max(max(b1, o1), min(b0, o0));
    b0 = max(b0, o0);
  };
  if (per >= 2) merge(dpp<0xb1>(b0), dpp<0xb1>(b1));
  if (per >= 4) merge(dpp<0x4e>(b0), dpp<0x4e>(b1));
  if (per >= 8) merge(dpp<0x141>(b0), dpp<0x141>(b1));
  if (per >= 16) merge(dpp<0x140>(b0), dpp<0x140>(b1));
}

// Is this lane the first of its token's L lanes with `is`? One of them has it.
template <int L>
__device__ __forceinline__ bool first_of(bool is, int l) {
  const uint64_t all = __ballot(is) >> (lane_id() & ~(L - 1));
  return l == (L <= 32 ? __builtin_ctz((uint32_t)all) : __builtin_ctzll(all));
}

// f(N) for N from 1 to 15, as constants.
template <int N = 1, typename F>
__device__ __forceinline__ void for_rotations(F f) {
  if constexpr (N < 16) {
    f(std::integral_constant<int, N>());
    for_rotations<N + 1>(f);
  }
}

// The choice score that an order key stands for.
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// One of a lane's V consecutive values of a row of E, -inf past its end. The
// row's V values start on ALIGN bytes where they are read as whole vectors.
template <typename T, int V, int ALIGN = sizeof(T) * V < 16 ? sizeof(T) * V : 16>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, float* x) {
  if (E % V == 0) {   // a row starts on V values: whole vectors
    if (e0 >= E) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = -kInf;
      return;
    }
    struct alignas(ALIGN) Pack { T v[V]; };
    const Pack p = *(const Pack*)(row + e0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 2) x[i] = __uint_as_float((uint32_t)p.v[i] << 16);
      else x[i] = p.v[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = -kInf;
    if (e0 + i < E) {
      if constexpr (sizeof(T) == 2) x[i] = __uint_as_float((uint32_t)row[e0 + i] << 16);
      else x[i] = row[e0 + i];
    }
  }
}

}  // namespace

// L lanes per token (16 or 64: reductions stay in the lanes' rows), V
// consecutive experts per lane (E <= L * V). The scores also go to LDS, where
// a choice's weight is looked up by its expert.
template <typename T, int L, int V>
__global__ __launch_bounds__(256) void k_route(const T* __restrict__ logits,
                                               const float* __restrict__ bias, RouteArgs a,
                                               int gs, uint32_t gmagic, int32_t* __restrict__ ids,
                                               float* __restrict__ weights) {
  __shared__ __attribute__((aligned(16))) float score[256 * V];
  __shared__ u32x4 held[V >= 8 ? V / 4 : 1][256];
  __shared__ int chosen[256 / L][kMaxTopK];
  const int l = threadIdx.x % L;
  const int tok = threadIdx.x / L;
  const uint32_t t = block_of_grid() * (256 / L) + tok;
  const bool live = t < (uint32_t)a.T;
  const int e0 = l * V;
  auto fmax2 = [](float p, float q) { return fmaxf(p, q); };
  auto umax2 = [](uint32_t p, uint32_t q) { return max(p, q); };

  float x[V];
  load_row<T, V>(logits + (int64_t)(live ? t : (uint32_t)a.T - 1) * a.E, e0, a.E, x);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = x[i] != x[i] ? -kInf : fminf(x[i], __FLT_MAX__);

  // scores (0 where not available) and the order keys of the choice scores
  float s[V];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 1.0f / (1.0f + expf(-x[i]));
  } else {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
    m = over_lanes<L>(m, fmax2);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = x[i] == -kInf ? 0.0f : expf(x[i] - m);
      z += (double)s[i];
    }
    const float zf = (float)over_lanes<L>(z, [](double p, double q) { return p + q; });
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = zf > 0.0f ? s[i] / zf : 0.0f;
  }
  uint32_t key[V];
  float b[V];
  if (bias) {
    load_row<float, V, 4>(bias, e0, a.E, b);   // a view of any element on
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] += s[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = s[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    score[threadIdx.x * V + i] = s[i];
    const float c = x[i] == -kInf ? -kInf : b[i];
    key[i] = c > -kInf ? order_key(c) : 0u;   // neither NaN nor -inf
  }

  if (a.top_groups < a.groups) {
    auto worth_of = [&](uint32_t b0, uint32_t b1) {
      const float v = b0 ? key_value(b0) : -kInf;
      return a.sum2 && b1 ? v + key_value(b1) : v;
    };
    // `per` lanes side by side hold the worth of a group, those past the groups
    // -inf. Where the lanes of a group are whole and a power of two they are
    // those of its experts; else lane g stands for group g, whose experts are
    // looked for in every lane (8192 x 256, 8 groups: 8.1 us against 11.3).
    const bool whole = gs % V == 0 && gs / V <= 16 && (gs / V & (gs / V - 1)) == 0;
    const int per = whole ? gs / V : 1;
    float worth = -kInf;
    if (whole) {
      uint32_t b0 = 0, b1 = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        two_largest(b0, b1, key[i]);
      }
      best_two(b0, b1, per);
      worth = worth_of(b0, b1);
    } else {
      for (int g = 0; g < a.groups; ++g) {
        uint32_t b0 = 0, b1 = 0;   // two best keys of the group
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int grp = (int)(((uint64_t)(uint32_t)(e0 + i) * gmagic) >> 21);
          two_largest(b0, b1, grp == g ? key[i] : 0u);
        }
        // the second best is the best but one lane's best, or that lane's second
        const uint32_t top = over_lanes<L>(b0, umax2);
        const uint32_t sec = over_lanes<L>(first_of<L>(b0 == top, l) ? b1 : b0, umax2);
        const float wv = worth_of(top, sec);
        if (l == g) worth = wv;
      }
    }
    // the lanes of better groups, of equal ones the lanes before
    const int first = l & -per;
    int rank = 0;
    if constexpr (L == 16) {
      for_rotations([&](auto n) {
        constexpr int N = decltype(n)::value;
        const float o = ror<N>(worth);
        rank += (int)(o > worth) | ((int)(o == worth) & (int)(l >= N));   // no branches
      });
      rank -= l - first;   // its own lanes before it
    } else {
      for (int g = 0; g < a.groups; ++g) {   // a wave a token
        const float o = __uint_as_float(
            (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(worth), g * per));
        rank += (int)(o > worth) | ((int)(o == worth) & (int)(g * per < first));
      }
      rank *= per;
    }
    const bool in = rank < a.top_groups * per;
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = in ? key[i] : 0u;
    } else {
      const uint32_t keep =
          (uint32_t)(__ballot(in && l < a.groups) >> (lane_id() & ~(L - 1)));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int grp = (int)(((uint64_t)(uint32_t)(e0 + i) * gmagic) >> 21);
        if (!((keep >> (grp & 31)) & 1u)) key[i] = 0u;
      }
    }
  }

  // top_k rounds: the largest key, its lowest expert, out with it. A lane
  // holds consecutive experts, so the lowest lane that holds the largest key
  // holds the lowest expert of that key. From 8 experts a lane on it holds the
  // best of each 4 of its keys in registers and the keys in LDS, and only the
  // 4 that lose one are looked at again (32768 x 256, top-8 without groups:
  // 17.2 us; all keys in registers, every one compared and masked a round: 20.1;
  // with 128 experts 11.1 and 12.6).
  if constexpr (V >= 8) {
    constexpr int NQ = V / 4;
    uint32_t best4[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      best4[q] = max(max(key[4 * q], key[4 * q + 1]), max(key[4 * q + 2], key[4 * q + 3]));
      held[q][threadIdx.x] = u32x4{key[4 * q], key[4 * q + 1], key[4 * q + 2], key[4 * q + 3]};
    }
    for (int r = 0; r < a.k; ++r) {
      uint32_t best = best4[0];
#pragma unroll
      for (int q = 1; q < NQ; ++q) best = max(best, best4[q]);
      const uint32_t top = over_lanes<L>(best, umax2);
      if (first_of<L>(best == top, l)) {
        int q = NQ - 1;
#pragma unroll
        for (int i = NQ - 2; i >= 0; --i) q = best4[i] == top ? i : q;
        u32x4 v = held[q][threadIdx.x];
        const int bi = v.x == top ? 0 : v.y == top ? 1 : v.z == top ? 2 : 3;
        chosen[tok][r] = top ? e0 + 4 * q + bi : -1;
        v.x = bi == 0 ? 0u : v.x;
        v.y = bi == 1 ? 0u : v.y;
        v.z = bi == 2 ? 0u : v.z;
        v.w = bi == 3 ? 0u : v.w;
        held[q][threadIdx.x] = v;
        const uint32_t left = max(max(v.x, v.y), max(v.z, v.w));
#pragma unroll
        for (int i = 0; i < NQ; ++i) best4[i] = i == q ? left : best4[i];
      }
    }
  } else {
    for (int r = 0; r < a.k; ++r) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
      const uint32_t top = over_lanes<L>(best, umax2);
      if (first_of<L>(best == top, l)) {
        int bi = V;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) bi = key[i] == top ? i : bi;
        chosen[tok][r] = top ? e0 + bi : -1;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = i == bi ? 0u : key[i];
      }
    }
  }
  // the token's lanes are lanes of one wave, whose LDS operations are in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  float total = 0.0f;
  if (a.renorm)
    for (int r = 0; r < a.k; ++r) {
      const int id = chosen[tok][r];
      total += id < 0 ? 0.0f : score[tok * L * V + id];
    }
  const float div = a.renorm ? total : 1.0f;
  for (int r = l; r < a.k; r += L) {
    const int id = chosen[tok][r];
    const float w = id < 0 ? 0.0f : score[tok * L * V + id];
    if (live) {
      ids[(int64_t)t * a.k + r] = id;
      weights[(int64_t)t * a.k + r] = div > 0.0f ? w / div * a.scaling : 0.0f;
    }
  }
}

hipError_t launch_route_experts(int dtype, const void* logits, const float* bias,
                                const RouteArgs& a, int32_t* ids, float* weights,
                                hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  // e / (E / groups) as a product: exact for e < 1024 and group sizes <= 1024
  const int gs = a.E / a.groups;
  const uint32_t gmagic = (1u << 21) / (uint32_t)gs + 1u;
#define LAUNCH(TT, LV, VV)                                                                     \
  hipLaunchKernelGGL((k_route<TT, LV, VV>),                                                    \
                     grid_of(((int64_t)a.T + 256 / LV - 1) / (256 / LV)), dim3(256), 0, stream, \
                     (const TT*)logits, bias, a, gs, gmagic, ids, weights)
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
