// Routing to experts (moe_route) and the plan of a routing (moe_plan).
#include "moe.h"

#include <type_traits>
#include <utility>

namespace agg {

namespace {

constexpr float kNone = -__builtin_inff();   // the key of an expert that cannot be chosen

// The value of another lane of the same token: step 0 exchanges neighbours, step 1 pairs, step 2
// the quads of 8 lanes and step 3 the halves of 16 (mirrored; the lanes of a half agree by then);
// steps 4 and 5 exchange lanes 16 and 32 apart.
template <int STEP>
__device__ inline int other_lane(int v) {
  if constexpr (STEP == 0) return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, true);
  else if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, true);
  else if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xF, 0xF, true);
  else if constexpr (STEP == 3) return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xF, 0xF, true);
  else return __shfl_xor(v, 1 << STEP);
}

template <int I, int N, typename F>
__device__ inline void each_step(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each_step<I + 1, N>(f);
  }
}

// op over the 2^STEPS lanes of a token, the result on all of them
template <int STEPS, typename F>
__device__ inline float token_reduce(float v, F op) {
  each_step<0, STEPS>([&](auto i) {
    v = op(v, __builtin_bit_cast(float, other_lane<decltype(i)::value>(__builtin_bit_cast(int, v))));
  });
  return v;
}

__device__ inline float bf16_float(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

}  // namespace

// 2^STEPS lanes a token, each holding the keys of V experts in registers (expert v * L + lane).
// The k picks are k maxima over (key, lowest index); a picked key becomes kNone. Chosen experts'
// scores are computed again from their logits at the end, by the lane that writes them, so no
// second array is held. With groups the keys also go to LDS, where a lane scans a whole group for
// its score.
template <int STEPS, int V>
__global__ void __launch_bounds__(256) route_kernel(const RouteArgs a) {
  constexpr int L = 1 << STEPS, TOKENS = 256 / L, E = L * V;
  constexpr int OUT = AGG_MAX_TOP_K > L ? AGG_MAX_TOP_K / L : 1;   // choices a lane writes
  __shared__ float keys[TOKENS][E + 1];
  __shared__ float group_score[TOKENS][AGG_MAX_GROUPS];
  const int lane = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * TOKENS + slot;
  const bool live = t < a.tokens;
  const float* const xf = static_cast<const float*>(a.logits) + t * a.ld;
  const uint16_t* const xb = static_cast<const uint16_t*>(a.logits) + t * a.ld;
  auto logit = [&](int e) { return a.logits_bf16 ? bf16_float(xb[e]) : xf[e]; };

  float key[V];
  float top = kNone;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + lane;
    float x = kNone;
    if (live && e < a.experts) x = logit(e);
    if (x != x) x = kNone;                  // a NaN logit: never chosen
    key[v] = x;
    top = fmaxf(top, x);
  }
  float sum = 1.0f;
  if (!a.sigmoid) {
    top = token_reduce<STEPS>(top, [](float x, float y) { return fmaxf(x, y); });
    sum = 0.0f;
    if (!a.renorm || a.bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) sum += key[v] > kNone ? expf(key[v] - top) : 0.0f;
      sum = token_reduce<STEPS>(sum, [](float x, float y) { return x + y; });
    } else {
      sum = 1.0f;                           // (renormalised over the chosen: the sum cancels)
    }
  }
  auto score = [&](float x) { return a.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - top) / sum; };
  if (a.sigmoid || a.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!(key[v] > kNone)) continue;
      key[v] = score(key[v]);
      if (a.bias) key[v] += a.bias[v * L + lane];
      if (key[v] != key[v]) key[v] = kNone;
    }
  }

  if (a.groups > 1) {
    const int size = a.experts / a.groups;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + lane;
      if (e < a.experts) keys[slot][e] = key[v];
    }
    __syncthreads();
    for (int g = lane; g < a.groups; g += L) {
      float b0 = kNone, b1 = kNone;
      for (int i = 0; i < size; ++i) {
        const float x = keys[slot][g * size + i];
        b1 = fmaxf(b1, fminf(b0, x));
        b0 = fmaxf(b0, x);
      }
      group_score[slot][g] = a.sigmoid && b1 > kNone ? b0 + b1 : b0;
    }
    __syncthreads();
    uint32_t kept[2] = {0, 0};              // a bit for each group that stays
    for (int g = lane; g < a.groups; g += L) {
      const float mine = group_score[slot][g];
      int before = 0;
      for (int o = 0; o < a.groups; ++o) {
        const float x = group_score[slot][o];
        before += (x > mine || (x == mine && o < g)) ? 1 : 0;
      }
      if (before < a.top_groups) kept[g >> 5] |= 1u << (g & 31);
    }
    each_step<0, STEPS>([&](auto i) {
      kept[0] |= (uint32_t)other_lane<decltype(i)::value>((int)kept[0]);
      kept[1] |= (uint32_t)other_lane<decltype(i)::value>((int)kept[1]);
    });
    // e / size by a product: exact while e * size < 2^20
    const uint32_t inv = ((1u << 20) + (uint32_t)size - 1) / (uint32_t)size;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t g = ((uint32_t)(v * L + lane) * inv) >> 20;
      if (!((kept[(g >> 5) & 1] >> (g & 31)) & 1u)) key[v] = kNone;
    }
  }

  int mine[OUT];
#pragma unroll
  for (int o = 0; o < OUT; ++o) mine[o] = -1;
  for (int j = 0; j < a.top_k; ++j) {
    float best = key[0];
    int at = lane;
#pragma unroll
    for (int v = 1; v < V; ++v) {
      const bool more = key[v] > best;      // (equal keys: the lower index stays)
      best = more ? key[v] : best;
      at = more ? v * L + lane : at;
    }
    each_step<0, STEPS>([&](auto i) {
      const float ob = __builtin_bit_cast(float, other_lane<decltype(i)::value>(__builtin_bit_cast(int, best)));
      const int oa = other_lane<decltype(i)::value>(at);
      const bool take = ob > best || (ob == best && oa < at);
      best = take ? ob : best;
      at = take ? oa : at;
    });
    const int chosen = best > kNone ? at : -1;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * L + lane == at) key[v] = kNone;
#pragma unroll
    for (int o = 0; o < OUT; ++o)
      if (j == o * L + lane) mine[o] = chosen;
  }
  float w[OUT], total = 0.0f;
#pragma unroll
  for (int o = 0; o < OUT; ++o) {
    w[o] = live && mine[o] >= 0 ? score(logit(mine[o])) : 0.0f;
    total += w[o];
  }
  float scale = a.scale;
  if (a.renorm) {
    total = token_reduce<STEPS>(total, [](float x, float y) { return x + y; });
    scale = total > 0.0f ? a.scale / total : 0.0f;
  }
#pragma unroll
  for (int o = 0; o < OUT; ++o) {
    const int j = o * L + lane;
    if (!live || j >= a.top_k) continue;
    a.ids[t * a.top_k + j] = mine[o];
    a.weights[t * a.top_k + j] = w[o] * scale;
  }
}

template <int STEPS, int V>
static hipError_t launch_route_lv(const RouteArgs& a, hipStream_t stream) {
  constexpr int64_t tokens = 256 >> STEPS;
  hipLaunchKernelGGL((route_kernel<STEPS, V>), dim3((unsigned)((a.tokens + tokens - 1) / tokens)), dim3(256), 0,
                     stream, a);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, int cus, hipStream_t stream) {
  (void)cus;
  if (a.experts <= 64) return launch_route_lv<3, 8>(a, stream);
  if (a.experts <= 128) return launch_route_lv<4, 8>(a, stream);
  if (a.experts <= 256) return launch_route_lv<4, 16>(a, stream);
  if (a.experts <= 512) return launch_route_lv<5, 16>(a, stream);
  return launch_route_lv<6, 16>(a, stream);
}

// ---- the plan: a stable counting sort of the (token, choice) pairs by expert
//
// Pair p = token * top_k + choice goes into the bucket of its expert, or, where the expert is not
// one of this rank's n_local (or is -1), into a last bucket that gets no slot. Blocks of kPlanPairs
// pairs: the first kernel counts each block's buckets, the second adds up what comes before its
// block and gives every pair its place. One block needs the second kernel alone. Counts are sums
// of ones, so no order of additions changes them, and the places follow the pairs' order.

namespace {

__device__ inline int bucket_of(const PlanArgs& a, int64_t p) {
  const int64_t e = (int64_t)a.ids[p] - a.first;
  return a.ids[p] >= 0 && e >= 0 && e < a.n_local ? (int)e : a.n_local;
}

}  // namespace

__global__ void __launch_bounds__(256) plan_count_kernel(const PlanArgs a) {
  __shared__ int count[AGG_MAX_EXPERTS + 1];
  const int buckets = a.n_local + 1;
  for (int e = threadIdx.x; e < buckets; e += 256) count[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanPairs / 256; ++i) {
    const int64_t p = (int64_t)blockIdx.x * kPlanPairs + i * 256 + threadIdx.x;
    if (p < a.pairs) atomicAdd(&count[bucket_of(a, p)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += 256) a.work[(int64_t)blockIdx.x * buckets + e] = count[e];
}

__global__ void __launch_bounds__(256) plan_place_kernel(const PlanArgs a) {
  constexpr int W = 4, R = kPlanPairs / 256;         // waves; rounds of 64 pairs a wave
  __shared__ int count[W][AGG_MAX_EXPERTS + 1];      // pairs of this block, by wave and bucket
  __shared__ int total[AGG_MAX_EXPERTS + 1];         // pairs of all blocks, by bucket
  __shared__ int place[AGG_MAX_EXPERTS + 1];         // where the block's pairs of a bucket begin
  __shared__ int wave_sum[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int buckets = a.n_local + 1, blocks = (int)gridDim.x, block = (int)blockIdx.x;
  for (int e = tid; e < buckets; e += 256) {
    for (int w = 0; w < W; ++w) count[w][e] = 0;
    total[e] = place[e] = 0;
  }
  __syncthreads();

  // each wave takes 64 pairs after 64 of its quarter of the block, in order: the lanes of one
  // bucket find each other by comparing the bucket's bits over ballots
  int bucket[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t p = (int64_t)block * kPlanPairs + wave * (kPlanPairs / W) + r * 64 + lane;
    bucket[r] = p < a.pairs ? bucket_of(a, p) : -1;
    uint64_t same = __ballot(bucket[r] >= 0);
    for (int b = 0; (1 << b) <= a.n_local; ++b) {
      const bool bit = (bucket[r] >> b) & 1;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    rank[r] = 0;
    if (bucket[r] >= 0) {
      rank[r] = count[wave][bucket[r]] + before;
      if (before == 0) count[wave][bucket[r]] += __popcll(same);
    }
    __syncthreads();
  }

  // totals of every bucket and what the blocks before this one hold of it
  if (blocks > 1) {
    int e = tid % buckets, b = tid / buckets;
    const int step_e = 256 % buckets, step_b = 256 / buckets;
    for (int i = tid; i < blocks * buckets; i += 256) {
      const int c = a.work[i];
      if (c) {
        atomicAdd(&total[e], c);
        if (b < block) atomicAdd(&place[e], c);
      }
      e += step_e;
      b += step_b;
      if (e >= buckets) { e -= buckets; ++b; }
    }
  } else {
    for (int e = tid; e < buckets; e += 256) {
      int c = 0;
      for (int w = 0; w < W; ++w) c += count[w][e];
      total[e] = c;
    }
  }
  __syncthreads();
  constexpr int kRun = (AGG_MAX_EXPERTS + 1 + 255) / 256;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int e = tid * kRun + i;
    if (e < buckets) mine += total[e];
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int at = incl - mine;
  for (int w = 0; w < wave; ++w) at += wave_sum[w];
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int e = tid * kRun + i;
    if (e < buckets) {
      place[e] += at;
      if (block == 0) a.offsets[e] = at;
      at += total[e];
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (bucket[r] < 0) continue;
    const int64_t p = (int64_t)block * kPlanPairs + wave * (kPlanPairs / W) + r * 64 + lane;
    int s = place[bucket[r]] + rank[r];
    for (int w = 0; w < wave; ++w) s += count[w][bucket[r]];
    const bool held = bucket[r] < a.n_local;
    a.slot_token[s] = held ? (int)(p / a.top_k) : -1;
    a.token_slot[p] = held ? s : -1;
  }
}

hipError_t launch_plan(const PlanArgs& a, hipStream_t stream) {
  const int64_t blocks = a.pairs > 0 ? (a.pairs + kPlanPairs - 1) / kPlanPairs : 1;
  if (blocks > 1) {
    hipLaunchKernelGGL(plan_count_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  hipLaunchKernelGGL(plan_place_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace agg
