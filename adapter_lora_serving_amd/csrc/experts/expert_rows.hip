// The rows of the experts' products, and the way back to tokens.
//
// Page "spark_model/lora/expert_apply.rs" (module overview): the experts'
// products run on rows sorted by expert, each expert's rows between two of
// its offsets, and a reduction brings them back to tokens. expert_rows sorts
// the T * k (token, choice) pairs of a routed batch that way, on the device:
// the stable counting sort of the slot addressing with the expert as the key
// (a choice outside [0, E) is dead and comes after every expert), then each
// row's token, its token's adapter slot and each choice's row.
#include "lora_common.h"
#include "lora_kernels.h"
#include "experts.h"

namespace lora {

// Token of choice i: i / k as a product with kmul = ceil(2^32 / k) (0 for k =
// 1), exact where i k^2 < 2^32: for the 2^22 choices of one launch at most.
__device__ __forceinline__ int token_of(int i, uint32_t kmul) {
  return kmul ? (int)__umulhi((uint32_t)i, kmul) : i;
}

// Where the sort by expert puts choice i of token t: its row, or none for a
// dead one.
__device__ __forceinline__ void put_row(int i, int t, int row, bool live, int slot,
                                        int32_t* __restrict__ row_token,
                                        int32_t* __restrict__ positions,
                                        int32_t* __restrict__ row_slot) {
  row_token[row] = t;
  positions[i] = live ? row : -1;
  if (row_slot) row_slot[row] = live ? slot : -1;
}

// What a wave's lanes wrote to LDS before is what they read after it: LDS
// operations of a wave are in order, so this holds the compiler alone.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A decode step's few choices over few experts: one wave, no barrier (the
// one-wave sort of the slot addressing, with the rows written in its place and
// their slots asked for with the choices). 512 choices of 8 experts: 4.5 us
// on the GPU, 8 groups in turn; the addressing and a second launch took 18 us a
// call.
template <int G>
__global__ __launch_bounds__(64) void k_rows_wave(const int32_t* __restrict__ ids, int n,
                                                  uint32_t kmul, int E, const int32_t* __restrict__ token_slot,
                                                  int32_t* __restrict__ row_token,
                                                  int32_t* __restrict__ positions,
                                                  int32_t* __restrict__ offsets,
                                                  int32_t* __restrict__ row_slot) {
  __shared__ int hist[kWave];
  const int lane = lane_id();
  const int nbits = 32 - __clz(E);
  int raw[G], slot[G], key[G], off[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int i = g * kWave + lane;
    raw[g] = i < n ? ids[i] : -1;
    slot[g] = row_slot && i < n ? token_slot[token_of(i, kmul)] : -1;
  }
  hist[lane] = 0;
  wave_lds_order();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const GroupMatch m = match_raw(raw[g], g * kWave + lane < n, E, nbits);
    key[g] = m.key < 0 ? 0 : m.key;   // lanes past n: any valid index, never used
    off[g] = hist[key[g]] + m.rank;
    wave_lds_order();
    if (m.leader) hist[m.key] += m.count;   // distinct keys: no two leaders collide
    wave_lds_order();
  }
  const int c = lane <= E ? hist[lane] : 0;
  const int start = wave_inclusive_scan(c) - c;
  if (lane <= E) offsets[lane] = start;
  wave_lds_order();
  hist[lane] = start;
  wave_lds_order();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int i = g * kWave + lane;
    if (i < n)
      put_row(i, token_of(i, kmul), hist[key[g]] + off[g], key[g] < E, slot[g], row_token,
              positions, row_slot);
  }
}

// Larger batches in one launch: a workgroup places 1024 choices and counts
// all n of them for itself, those before its own apart from the rest, so no
// workgroup waits for another. The counting reads n ids from L2 a workgroup:
// 65536 choices are 64 workgroups of 256 KB each, 10.4 us for 256 experts,
// bound by the instructions and LDS adds of the counting. Past that, where the
// workspace of lora_expert_rows_workspace_bytes begins, the two passes of the
// addressing count once, and a third launch writes the rows. One launch would
// still be the shorter there (256 experts, 131072 choices: 15.7 us against
// 42.2; 262144: 25 against 75; 1048576: 246 against 387). The two passes hold a
// key a thread, 1023 experts and the dead choices; 1024 experts stay in one
// launch while token_of is exact (131072 choices: 17.3 us against 309 in the
// one workgroup that sorts any number of keys; 1048576: 348 against 2652).
// Neighbouring lanes add to other copies of the counters, since lanes
// that add to one address wait for each other: 4, 8 and 16 copies take 10.2,
// 10.2 and 10.4 us where the choices are spread evenly, 18.8, 12.1 and 9.5
// where all are of one expert (or dead). 16 fit the LDS up to 512 experts.
constexpr int kRowsBlock = 1024;
constexpr int kRowsOneLaunch = 1 << 16;
constexpr int kRowsOneLaunchAllKeys = 1 << 22;

template <int kCopies>
__global__ __launch_bounds__(kRowsBlock) void k_rows_block(
    const int32_t* __restrict__ ids, int n, uint32_t kmul, int E,
    const int32_t* __restrict__ token_slot, int32_t* __restrict__ row_token,
    int32_t* __restrict__ positions, int32_t* __restrict__ offsets,
    int32_t* __restrict__ row_slot) {
  extern __shared__ int smem[];
  const int S1 = E + 1;
  int* cnt = smem;                    // [16][S1] per-wave counts, then offsets in the workgroup
  int* before = cnt + 16 * S1;        // [kCopies][S1] choices before this workgroup's
  int* rest = before + kCopies * S1;  // [kCopies][S1] the others
  int* scratch = rest + kCopies * S1; // [20]
  const int tid = threadIdx.x;
  const int w = tid / kWave;
  const int nbits = 32 - __clz(E);
  const int own0 = blockIdx.x * kRowsBlock;
  for (int i = tid; i < (16 + 2 * kCopies) * S1; i += kRowsBlock) smem[i] = 0;
  const int i0 = own0 + tid;
  const GroupMatch g = match_raw(i0 < n ? ids[i0] : -1, i0 < n, E, nbits);
  const int t0 = token_of(min(i0, n), kmul);
  const int slot = row_slot && i0 < n ? token_slot[t0] : -1;
  __syncthreads();
  if (g.leader) cnt[w * S1 + g.key] += g.count;   // distinct keys: no collision
  // ids [lo, hi) into a histogram: whole vectors from the first 16-byte
  // boundary on, single ids around them
  auto count = [&](int lo, int hi, int* hist) {
    hist += tid % kCopies * S1;
    auto add = [&](uint32_t id) { atomicAdd(hist + min(id, (uint32_t)E), 1); };
    const int head = min(hi, lo + (int)(-(reinterpret_cast<intptr_t>(ids + lo) >> 2) & 3));
    const int tail = head + ((hi - head) & ~3);
#pragma unroll 4
    for (int i = head + tid * 4; i < tail; i += kRowsBlock * 4) {
      const u32x4 v = *(const u32x4*)(ids + i);
      add(v.x);
      add(v.y);
      add(v.z);
      add(v.w);
    }
    if (lo + tid < head) add((uint32_t)ids[lo + tid]);
    if (tail + tid < hi) add((uint32_t)ids[tail + tid]);
  };
  count(0, min(own0, n), before);
  count(min(own0, n), n, rest);
  __syncthreads();
  int tot = 0;   // key tid (S1 <= 1025: the last key by thread 0 below)
  auto offsets_of = [&](int key) {
    int run = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int c = cnt[q * S1 + key];
      cnt[q * S1 + key] = run;
      run += c;
    }
    int b = 0, r = 0;
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      b += before[q * S1 + key];
      r += rest[q * S1 + key];
    }
    before[key] = b;
    return b + r;
  };
  if (tid < E) tot = offsets_of(tid);
  if (tid == 0) offsets_of(E);
  int live = 0;
  const int start = block_exclusive_scan(tid < E ? tot : 0, scratch, &live);
  if (tid < E) {
    before[tid] += start;
    if (blockIdx.x == 0) offsets[tid] = start;
  }
  if (tid == 0) {
    before[E] += live;
    if (blockIdx.x == 0) offsets[E] = live;
  }
  __syncthreads();
  if (i0 < n)
    put_row(i0, t0, before[g.key] + cnt[w * S1 + g.key] + g.rank, g.key < E, slot, row_token,
            positions, row_slot);
}

// row_token holds the sorted choices (token * k + j) on entry and the tokens
// on return; every thread turns its own.
__global__ __launch_bounds__(256) void k_rows_finish(int n, int k, int E,
                                                     const int32_t* __restrict__ offsets,
                                                     const int32_t* __restrict__ token_slot,
                                                     int32_t* row_token,
                                                     int32_t* __restrict__ positions,
                                                     int32_t* __restrict__ row_slot) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= n) return;
  const int i = row_token[r], t = i / k;
  const bool live = r < offsets[E];
  put_row(i, t, r, live, row_slot && live ? token_slot[t] : -1, row_token, positions, row_slot);
}

size_t expert_rows_workspace_bytes(int64_t T, int k, int E) {
  return T * k <= kRowsOneLaunch ? 0 : addressing_workspace_bytes(T * k, E);
}

hipError_t launch_expert_rows(const int32_t* ids, int T, int k, int E, const int32_t* token_slot,
                              int32_t* row_token, int32_t* positions, int32_t* offsets,
                              int32_t* row_slot, void* ws, hipStream_t stream) {
  const int n = T * k;
  const uint32_t kmul = k == 1 ? 0u : (uint32_t)(((1ull << 32) + k - 1) / k);
  if (n <= 16 * kWave && E < kWave) {
#define W(GV)                                                                              \
  hipLaunchKernelGGL(k_rows_wave<GV>, dim3(1), dim3(kWave), 0, stream, ids, n, kmul, E,    \
                     token_slot, row_token, positions, offsets, row_slot)
    const int groups = (n + kWave - 1) / kWave;
    if (groups <= 1) W(1);
    else if (groups <= 2) W(2);
    else if (groups <= 4) W(4);
    else if (groups <= 8) W(8);
    else W(16);
#undef W
    return hipGetLastError();
  }
  const bool two_passes = addressing_workspace_bytes(n, E) > 0;   // E + 1 keys, one a thread
  if (n <= (two_passes ? kRowsOneLaunch : kRowsOneLaunchAllKeys)) {
    const int nb = n == 0 ? 1 : (n + kRowsBlock - 1) / kRowsBlock;
    const int copies = E <= 512 ? 16 : 8;
    auto* const f = copies == 16 ? k_rows_block<16> : k_rows_block<8>;
    const size_t lds = ((size_t)(16 + 2 * copies) * (E + 1) + 20) * sizeof(int);
    if (lds > 65536) {
      const hipError_t e = hipFuncSetAttribute((const void*)f,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(f, dim3(nb), dim3(kRowsBlock), lds, stream, ids, n, kmul, E, token_slot,
                       row_token, positions, offsets, row_slot);
    return hipGetLastError();
  }
  hipError_t e = launch_build_addressing(ids, n, E, row_token, offsets, ws,
                                         expert_rows_workspace_bytes(T, k, E), stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_rows_finish, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, n, k,
                     E, offsets, token_slot, row_token, positions, row_slot);
  return hipGetLastError();
}

// y[t] = residual[t] + sum over j of weights[t, j] * rows[positions[t, j]],
// j ascending in fp32, rounded once. A position outside [0, nrows) adds
// nothing. residual may be y (a thread reads its columns before it writes
// them), so neither is __restrict__. 16 bytes of columns per thread, a
// workgroup a token: the rows' bytes are the time. 8192 tokens x 8 rows x 4096
// bf16 onto the residual: 132 us for 671 MB, 5.1 TB/s.
template <typename D>
__global__ __launch_bounds__(256) void k_combine(const char* __restrict__ rows, int64_t nrows,
                                                 int H, const int32_t* __restrict__ positions,
                                                 const float* __restrict__ weights, int T, int k,
                                                 const char* residual, char* y) {
  const uint32_t t = block_of_grid();
  if (t >= (uint32_t)T) return;
  const int64_t rowb = (int64_t)H * D::kBytes;
  for (int c = threadIdx.x * 16; c < rowb; c += 256 * 16) {
    float acc[D::kVec];
    auto add = [&](u32x4 v, float w) {
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D::kVec == 8) {
          acc[2 * i] += w * bf16lo(q[i]);
          acc[2 * i + 1] += w * bf16hi(q[i]);
        } else {
          acc[i] += w * __uint_as_float(q[i]);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < D::kVec; ++i) acc[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int p = positions[(int64_t)t * k + j];
      if (p < 0 || p >= nrows) continue;
      add(*(const u32x4*)(rows + p * rowb + c), weights[(int64_t)t * k + j]);
    }
    if (residual) add(*(const u32x4*)(residual + t * rowb + c), 1.0f);
    u32x4 o;
    if constexpr (D::kVec == 8)
      o = u32x4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])};
    else
      o = u32x4{__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                __float_as_uint(acc[3])};
    *(u32x4*)(y + t * rowb + c) = o;
  }
}

hipError_t launch_combine_experts(int dtype, const void* rows, int64_t nrows, int H,
                                  const int32_t* positions, const float* weights, int T, int k,
                                  const void* residual, void* y, hipStream_t stream) {
  if (T == 0) return hipSuccess;
#define GO(D)                                                                                 \
  hipLaunchKernelGGL(k_combine<D>, grid_of(T), dim3(256), 0, stream, (const char*)rows, nrows, \
                     H, positions, weights, T, k, (const char*)residual, (char*)y)
  if (dtype == 1) GO(BF16); else GO(F32);
#undef GO
  return hipGetLastError();
}

}  // namespace lora
