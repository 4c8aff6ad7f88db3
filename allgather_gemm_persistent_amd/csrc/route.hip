// Routing to experts (moe_route) and the plan of a routing (moe_plan).
#include "moe.h"

#include <type_traits>
#include <utility>

namespace agg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// Orders a wave's LDS accesses: what its lanes wrote before is what they read after (the lanes of a
// token share a wave, whose LDS operations run in order; this keeps the compiler to that order).
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ inline float bf16_float(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

// 1 / d for 1 <= d <= 2^126, rounded like the division: a reciprocal, one Newton step, and the
// residual's correction (Markstein); equal to the division for every such float (all were tried). The
// general division takes twice as many instructions for ranges that do not occur here.
__device__ inline float reciprocal(float d) {
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}
constexpr float kReciprocalMost = 8.5e37f;   // below 2^126
// Scores are lost below 2^-128 (a sigmoid's exponential overflows) or rounded to multiples of 2^-149: at
// most 2^-68 of a sum of 2^-60 or more. Below that sum sigmoid(x) is exp(x) to the last bit.
constexpr float kScoresLost = 8.673617380e-19f;   // 2^-60

// A group's score from its two largest keys.
__device__ inline float group_key(int sigmoid, float b0, float b1) { return sigmoid && b1 > kNone ? b0 + b1 : b0; }

// The groups before group g: larger scores, or equal ones at a lower index.
__device__ inline int group_rank(const float* score, int groups, int g) {
  const float mine = score[g];
  int before = 0;
  for (int o = 0; o < groups; ++o) {
    const float x = score[o];
    before += x > mine || (x == mine && o < g) ? 1 : 0;
  }
  return before;
}

// Drop the keys of the groups that do not stay, where a token's L * V experts fill its lanes and the
// groups' sizes are powers of two, no less than L and V. The keys cross LDS, so that lane i gets the V
// consecutive experts from i * V (padded by 16 bytes, which puts the lanes' 16-byte reads on different
// banks), all of one group; a group's lanes are neighbours. `room`: the token's LDS, L * (V + 4) floats;
// `score`: its groups' scores. (8 groups of 256 experts: 213 vector instructions a wave, 353 where each
// group's members are read from LDS one at a time; 19.8 us and 23.5 for the kernel at 32768 tokens.)
template <int STEPS, int V>
__device__ inline void keep_groups(float (&key)[V], int sigmoid, int groups, int top_groups, float* room,
                                   float* score, int lane) {
  constexpr int L = 1 << STEPS;
  static_assert(L >= V, "a row of experts across the lanes is whole chunks");
#pragma unroll
  for (int v = 0; v < V; ++v) room[v * (L + L / V * 4) + lane + lane / V * 4] = key[v];
  wave_sync();
  float b0 = kNone, b1 = kNone;
#pragma unroll
  for (int q = 0; q < V / 4; ++q) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(room + lane * (V + 4) + q * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b1 = __builtin_amdgcn_fmed3f(b0, b1, x[i]);        // (b1 <= b0: the new second)
      b0 = fmaxf(b0, x[i]);
    }
  }
  const int parts = L / groups;
  each_step<0, STEPS>([&](auto i) {
    if ((1 << decltype(i)::value) < parts) {
      const float o0 = __builtin_bit_cast(float, other_lane<decltype(i)::value>(__builtin_bit_cast(int, b0)));
      const float o1 = __builtin_bit_cast(float, other_lane<decltype(i)::value>(__builtin_bit_cast(int, b1)));
      b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
      b0 = fmaxf(b0, o0);
    }
  });
  const int g = lane / parts;
  if (lane % parts == 0) score[g] = group_key(sigmoid, b0, b1);
  wave_sync();
  uint32_t kept = lane % parts == 0 && group_rank(score, groups, g) < top_groups ? 1u << g : 0u;
  each_step<0, STEPS>([&](auto i) { kept |= (uint32_t)other_lane<decltype(i)::value>((int)kept); });
  // (v * L / size is the same on all lanes)
  const int shift = __builtin_ctz((uint32_t)(L * V / groups));
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (!(kept & (1u << ((v * L) >> shift)))) key[v] = kNone;
}

}  // namespace

// 2^STEPS lanes a token, each holding the keys of V experts in registers (expert v * L + lane). With
// groups the keys also go to LDS, where a lane scans a whole group for its score.
//
// The choice: with no more picks than half the lanes, the top_k-th largest of the lanes' own maxima is
// a bound that top_k keys reach, so only keys that reach it can be picked; they are few (about 10 for
// 8 of 256), go to a list in LDS, and each takes its place by counting the keys before it, (larger, or
// equal at a lower index). Otherwise, or where ties fill the list, the picks are top_k maxima over
// (key, lowest index) one after another, a picked key becoming kNone. Chosen experts' scores are
// computed again from their logits, by the lane that writes them.
//
// Bound by instructions at many tokens: 32768 tokens of 256 experts in fp32 are 33.6 MB, 6.6 us of
// copying. 6.2 us for top 1 over softmax, 13.3 for top 8, 16.5 over the sigmoid, 17.6 with a bias, 19.8
// with 8 groups of which 4 stay. FULL drops the bounds of experts that fill the lanes.
template <int STEPS, int V, bool BF16, bool FULL>
__global__ void __launch_bounds__(256) route_kernel(const RouteArgs a) {
  constexpr int L = 1 << STEPS, TOKENS = 256 / L;
  constexpr int OUT = AGG_MAX_TOP_K > L ? AGG_MAX_TOP_K / L : 1;   // choices a lane writes
  __shared__ __attribute__((aligned(16))) float keys[TOKENS][L * (V + 4)];
  __shared__ float group_score[TOKENS][AGG_MAX_GROUPS];
  constexpr int LIST = 2 * L;               // candidates a token's list holds
  struct __attribute__((aligned(8))) Candidate {
    float key;
    int at;
  };
  __shared__ Candidate list[TOKENS][LIST];
  __shared__ int picked[TOKENS][AGG_MAX_TOP_K];
  const int lane = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * TOKENS + slot;
  const bool live = t < a.tokens;
  const float* const xf = static_cast<const float*>(a.logits) + t * a.ld;
  const uint16_t* const xb = static_cast<const uint16_t*>(a.logits) + t * a.ld;
  auto logit = [&](int e) { return BF16 ? bf16_float(xb[e]) : xf[e]; };

  float key[V];
  float top = kNone;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + lane;
    float x = kNone;
    if (live && (FULL || e < a.experts)) x = logit(e);
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
  if (a.sigmoid) {
    float d[V], most = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] = 1.0f + expf(-key[v]);          // (kNone: infinity)
      most = fmaxf(most, key[v] > kNone ? d[v] : 0.0f);
    }
    const bool plain = __any(!(most <= kReciprocalMost));
    if (plain) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = 1.0f / d[v];
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = reciprocal(d[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] > kNone ? d[v] : kNone;
  } else if (a.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] > kNone ? score(key[v]) : kNone;
  }
  if (a.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + lane;
      if (FULL || e < a.experts) key[v] += a.bias[e];
      if (key[v] != key[v]) key[v] = kNone;
    }
  }

  if (a.groups > 1) {
    const int size = a.experts / a.groups;
    uint32_t kept[2] = {0, 0};              // a bit for each group that stays
    // (64 .. 1024 experts and up to 8 or 16 groups, both powers of two; else one member after another)
    if (FULL && (a.groups & (a.groups - 1)) == 0 && a.groups <= (L < V ? L : V)) {
      keep_groups<STEPS, V>(key, a.sigmoid, a.groups, a.top_groups, keys[slot], group_score[slot], lane);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * L + lane;
        if (e < a.experts) keys[slot][e] = key[v];
      }
      wave_sync();
      // `parts` lanes a group, each over its share of the members, starting at different members (the
      // groups' members lie a power of two apart in LDS: from the same one the lanes would meet in
      // its banks)
      int slots = 1;
      while (slots < a.groups && slots < L) slots *= 2;
      const int parts = L / slots, part = lane / slots;
      for (int g = lane & (slots - 1); g < a.groups; g += slots) {
        float b0 = kNone, b1 = kNone;
        int m = (g + part) % size;
        for (int i = part; i < size; i += parts) {
          const float x = keys[slot][g * size + m];
          b1 = fmaxf(b1, fminf(b0, x));
          b0 = fmaxf(b0, x);
          m += parts;
          if (m >= size) m -= size;
        }
        for (int d = slots; d < L; d *= 2) {
          const float o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
          b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
          b0 = fmaxf(b0, o0);
        }
        if (part == 0) group_score[slot][g] = group_key(a.sigmoid, b0, b1);
      }
      wave_sync();
      for (int g = lane; g < a.groups; g += L)
        if (group_rank(group_score[slot], a.groups, g) < a.top_groups) kept[g >> 5] |= 1u << (g & 31);
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
  }

  int mine[OUT];
  // (up to three picks one after another cost no more than the list: 6.3, 7.4, 8.9, 10.0, 12.8 and 15.5 us
  // for top 1, 2, 3, 4, 6 and 8 of 256 at 32768 tokens, the list 8.1, 8.8, 9.8, 9.8, 10.8 and 13.6)
  bool listed = 2 * a.top_k <= L && a.top_k > 3;
  if (listed) {
    // the bound: the top_k-th largest of the lanes' maxima (equal ones count for every lane)
    float best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = fmaxf(best, key[v]);
    wave_sync();                            // (the groups' scores were read from here)
    group_score[slot][lane] = best;
    wave_sync();
    int before = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) before += group_score[slot][i] > best ? 1 : 0;
    // lanes with fewer than top_k larger maxima hold the top_k largest; the least of them
    // (no less than the lowest float, which kNone does not reach)
    const float bound = fmaxf(token_reduce<STEPS>(before < a.top_k ? best : __builtin_inff(),
                                                  [](float x, float y) { return fminf(x, y); }),
                              -3.402823466e38f);
    int count = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) count += key[v] >= bound ? 1 : 0;
    int held = count;                       // becomes the lanes' inclusive prefix
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
      const int o = __shfl_up(held, d, L);
      if (lane >= d) held += o;
    }
    const int all = __shfl(held, L - 1, L);
    listed = !__any(all > LIST);
    if (listed) {
      int at = held - count;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] >= bound) {
          list[slot][at] = Candidate{key[v], v * L + lane};
          ++at;
        }
      for (int j = lane; j < a.top_k; j += L) picked[slot][j] = -1;
      wave_sync();
      for (int c = lane; c < all; c += L) {
        const Candidate own = list[slot][c];
        int place = 0;
#pragma unroll 4
        for (int i = 0; i < all; ++i) {
          const Candidate o = list[slot][i];
          place += o.key > own.key || (o.key == own.key && o.at < own.at) ? 1 : 0;
        }
        if (place < a.top_k) picked[slot][place] = own.at;
      }
      wave_sync();
#pragma unroll
      for (int o = 0; o < OUT; ++o) mine[o] = o * L + lane < a.top_k ? picked[slot][o * L + lane] : -1;
    }
  }
  if (!listed) {
#pragma unroll
    for (int o = 0; o < OUT; ++o) mine[o] = -1;
    for (int j = 0; j < a.top_k; ++j) {
      float best = key[0];
      int at = lane;
#pragma unroll
      for (int v = 1; v < V; ++v) {
        const bool more = key[v] > best;    // (equal keys: the lower index stays)
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
    if (total < kScoresLost) {
      // the chosen logits lie so far below the others (softmax, where a bias chooses) or below zero
      // (sigmoid) that their scores are lost or few bits are left of them: both scores are then
      // proportional to exp(x), which is taken from the largest chosen logit
      float most = kNone;
#pragma unroll
      for (int o = 0; o < OUT; ++o) most = fmaxf(most, live && mine[o] >= 0 ? logit(mine[o]) : kNone);
      most = token_reduce<STEPS>(most, [](float x, float y) { return fmaxf(x, y); });
      total = 0.0f;
#pragma unroll
      for (int o = 0; o < OUT; ++o) {
        w[o] = live && mine[o] >= 0 ? expf(logit(mine[o]) - most) : 0.0f;
        total += w[o];
      }
      total = token_reduce<STEPS>(total, [](float x, float y) { return x + y; });
    }
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
static hipError_t launch_route_lv(RouteArgs a, hipStream_t stream) {
  constexpr int64_t tokens = 256 >> STEPS;
  // (a launch holds fewer than 2^32 threads: more tokens go in further ones)
  constexpr int64_t most = tokens << 23;
  for (; a.tokens > most; a.tokens -= most) {
    RouteArgs p = a;
    p.tokens = most;
    if (hipError_t e = launch_route_lv<STEPS, V>(p, stream)) return e;
    a.logits = static_cast<const char*>(a.logits) + most * a.ld * (a.logits_bf16 ? 2 : 4);
    a.ids += most * a.top_k;
    a.weights += most * a.top_k;
  }
  const dim3 grid((unsigned)((a.tokens + tokens - 1) / tokens)), block(256);
  const bool full = a.experts == (V << STEPS);    // no lane without an expert
  if (a.logits_bf16) {
    if (full) hipLaunchKernelGGL((route_kernel<STEPS, V, true, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_kernel<STEPS, V, true, false>), grid, block, 0, stream, a);
  } else {
    if (full) hipLaunchKernelGGL((route_kernel<STEPS, V, false, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_kernel<STEPS, V, false, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
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
// pairs: the first kernel counts each block's buckets, the last gives every pair its place from what
// comes before its block, which it counts itself (up to kPlanAlone pairs, without the first kernel),
// adds up from the counts, or takes from a kernel between them that did.
// Counts are sums of ones, so no order of additions changes them, and the places follow the pairs' order.
//
// Bound by latency: the ids of 32768 tokens' 8 choices are 1 MB, and the two kernels take 4 and 6 us;
// a plan of one block takes 3 us.

namespace {

__device__ inline int bucket_of(const PlanArgs& a, int64_t p) {
  const int64_t e = (int64_t)a.ids[p] - a.first;
  return a.ids[p] >= 0 && e >= 0 && e < a.n_local ? (int)e : a.n_local;
}

}  // namespace

constexpr int kPlanThreads = 1024;
constexpr int64_t kPlanAlone = 12 * kPlanPairs;
constexpr int64_t kPlanCounts = 20000;               // counts that every block adds up

// Block b of R * kPlanPairs pairs.
template <int R>
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanArgs a) {
  __shared__ int count[AGG_MAX_EXPERTS + 1];
  const int buckets = a.n_local + 1;
  for (int e = threadIdx.x; e < buckets; e += kPlanThreads) count[e] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t p = ((int64_t)blockIdx.x * R + r) * kPlanPairs + threadIdx.x;
    if (p < a.pairs) atomicAdd(&count[bucket_of(a, p)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += kPlanThreads) a.work[(int64_t)blockIdx.x * buckets + e] = count[e];
}

// The counts of `blocks` blocks, in place, become the sums over the blocks before each; one more row gets
// the sums over all. A wave a bucket, its lanes over blocks.
__global__ void __launch_bounds__(256) plan_scan_kernel(const PlanArgs a, int blocks) {
  constexpr int U = 4;                               // loads on their way together
  const int lane = threadIdx.x & 63, buckets = a.n_local + 1;
  const int e = (int)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= buckets) return;
  int sum = 0;
  for (int b0 = 0; b0 < blocks; b0 += 64 * U) {
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * 64 + lane;
      c[u] = b < blocks ? a.work[(int64_t)b * buckets + e] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int incl = c[u];
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
      }
      const int b = b0 + u * 64 + lane;
      if (b < blocks) a.work[(int64_t)b * buckets + e] = sum + incl - c[u];
      sum += __shfl(incl, 63);
    }
  }
  if (lane == 0) a.work[(int64_t)blocks * buckets + e] = sum;
}

// How a block learns what comes before it: from all the pairs, from the blocks' counts, or from their sums.
enum PlanFrom { kFromPairs, kFromCounts, kFromSums };

template <int R, PlanFrom FROM>
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanArgs a) {
  constexpr int W = kPlanThreads / 64;               // waves
  __shared__ int count[W][AGG_MAX_EXPERTS + 1];      // pairs of this block, by wave and bucket
  __shared__ int total[AGG_MAX_EXPERTS + 1];         // pairs of all blocks, by bucket
  __shared__ int place[AGG_MAX_EXPERTS + 1];         // where the block's pairs of a bucket begin
  __shared__ int wave_sum[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int buckets = a.n_local + 1, blocks = (int)gridDim.x, block = (int)blockIdx.x;
  for (int e = tid; e < buckets; e += kPlanThreads) {
    for (int w = 0; w < W; ++w) count[w][e] = 0;
    total[e] = place[e] = 0;
  }
  // each wave takes 64 pairs after 64 of its part of the block, in order
  auto pair = [&](int r) { return ((int64_t)block * W + wave) * (R * 64) + r * 64 + lane; };
  int bucket[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) bucket[r] = pair(r) < a.pairs ? bucket_of(a, pair(r)) : -1;
  __syncthreads();
  // the lanes of one bucket find each other by comparing the bucket's bits over ballots
#pragma unroll
  for (int r = 0; r < R; ++r) {
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
      wave_sync();
      if (before == 0) count[wave][bucket[r]] += __popcll(same);
    }
    wave_sync();
  }

  // totals of every bucket and what the blocks before this one hold of it
  if (FROM == kFromSums) {
    for (int e = tid; e < buckets; e += kPlanThreads) {
      total[e] = a.work[(int64_t)blocks * buckets + e];
      place[e] = a.work[(int64_t)block * buckets + e];
    }
    __syncthreads();
  } else if (FROM == kFromPairs && blocks > 1) {
    // from the pairs themselves, kBatch loads on their way together
    constexpr int kBatch = 8;
    const int pairs = (int)a.pairs, mine = block * R * kPlanPairs;
    for (int p0 = tid; p0 < pairs; p0 += kPlanThreads * kBatch) {
      int b[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) b[u] = p0 + u * kPlanThreads < pairs ? bucket_of(a, p0 + u * kPlanThreads) : -1;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (b[u] < 0) continue;
        atomicAdd(p0 + u * kPlanThreads < mine ? &place[b[u]] : &total[b[u]], 1);
      }
    }
    __syncthreads();
    for (int e = tid; e < buckets; e += kPlanThreads) total[e] += place[e];
    __syncthreads();
  } else if (blocks > 1) {
    // kBatch loads on their way together; a thread steps through (block, bucket) by kPlanThreads
    constexpr int kBatch = 8;
    int e = tid % buckets, b = tid / buckets;
    const int step_e = kPlanThreads % buckets, step_b = kPlanThreads / buckets, words = blocks * buckets;
    for (int i0 = tid; i0 < words; i0 += kPlanThreads * kBatch) {
      int c[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) c[u] = i0 + u * kPlanThreads < words ? a.work[i0 + u * kPlanThreads] : 0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (c[u]) {
          atomicAdd(&total[e], c[u]);
          if (b < block) atomicAdd(&place[e], c[u]);
        }
        e += step_e;
        b += step_b;
        if (e >= buckets) { e -= buckets; ++b; }
      }
    }
    __syncthreads();
  } else {
    __syncthreads();
    for (int e = tid; e < buckets; e += kPlanThreads) {
      int c = 0;
      for (int w = 0; w < W; ++w) c += count[w][e];
      total[e] = c;
    }
    __syncthreads();
  }
  // a thread's run of buckets, and all runs before it
  constexpr int kRun = (AGG_MAX_EXPERTS + 1 + kPlanThreads - 1) / kPlanThreads;
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
    const int64_t p = pair(r);
    int s = place[bucket[r]] + rank[r];
    for (int w = 0; w < wave; ++w) s += count[w][bucket[r]];
    const bool held = bucket[r] < a.n_local;
    a.slot_token[s] = held ? (int)(p / a.top_k) : -1;
    a.token_slot[p] = held ? s : -1;
  }
}

template <int R, PlanFrom FROM>
static hipError_t launch_plan_r(const PlanArgs& a, hipStream_t stream) {
  const int64_t blocks = a.pairs > 0 ? (a.pairs + R * kPlanPairs - 1) / (R * kPlanPairs) : 1;
  if (FROM != kFromPairs) {
    hipLaunchKernelGGL(plan_count_kernel<R>, dim3((unsigned)blocks), dim3(kPlanThreads), 0, stream, a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (FROM == kFromSums) {
    hipLaunchKernelGGL(plan_scan_kernel, dim3((unsigned)((a.n_local + 4) / 4)), dim3(256), 0, stream, a, (int)blocks);
    if (hipError_t e = hipGetLastError()) return e;
  }
  hipLaunchKernelGGL((plan_place_kernel<R, FROM>), dim3((unsigned)blocks), dim3(kPlanThreads), 0, stream, a);
  return hipGetLastError();
}

// Up to kPlanAlone pairs every block counts them all. Beyond, it adds up the blocks' counts while these are
// few, and else takes them summed by a third launch (larger blocks then cost less). Microseconds:
//   pairs         4096  8192  12288  16384  131072   131072  262144  262144  262144   1048576  16777216
//   experts         64    64     64     64      64      256      64     256    1024       256       256
//   one launch     5.1   5.8    6.7    7.3
//   counts         6.7   6.8    7.1    7.1     8.3     12.7    10.3    19.3    51.1     131.5
//   sums, 2048 a block                        10.6     11.3    11.1    12.1    14.8      19.8       200
//   sums, 4096                                13.3     14.2    13.7    14.8    16.8      19.0       158
hipError_t launch_plan(const PlanArgs& a, hipStream_t stream) {
  static_assert(kPlanThreads == kPlanPairs, "a pair a thread and round");
  if (a.pairs <= kPlanAlone) return launch_plan_r<1, kFromPairs>(a, stream);
  if (a.pairs / kPlanPairs * (a.n_local + 1) <= kPlanCounts) return launch_plan_r<1, kFromCounts>(a, stream);
  if (a.pairs <= 1024 * kPlanPairs) return launch_plan_r<2, kFromSums>(a, stream);
  return launch_plan_r<4, kFromSums>(a, stream);
}

}  // namespace agg
