// Attention of new tokens over a paged cache (paged_attn): out = sum_i softmax(x)_i v_i, x_i = scale q . k_i,
// for every row (a new token) and head of queries.
#include <type_traits>

#include "attn.h"
#include "convert.h"

namespace agg {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4, kThreads = kAttnWaves * 64;
constexpr int kTile = 32;                      // tokens a wave takes at once: two runs of 16
constexpr int kBlock = 64;                     // tiles whose pages are looked up at once
constexpr int kBufferFlags = 0x00020000;       // word 3 of a raw buffer resource
constexpr uint32_t kOutOfRange = 0x80000000u;  // an offset past every descriptor
constexpr int kCoherent = 16;                  // an access that the whole GPU sees: past the L2, or written through it
constexpr uint32_t kFan = 32;                  // units joined in one step
constexpr int kChoices = 6;                    // lengths of a unit to choose from
constexpr float kUnitCost = 12;                // of a unit, beside its tiles, in tiles
constexpr float kJoinCost = 10;                // of units that are joined
constexpr float kLn2 = 0.693147181f;

__device__ inline f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

__device__ inline uint32_t pack2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ inline float low_half(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ inline float high_half(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// Over the wave's lanes, without LDS: f (of whole numbers, 0 for none) of the lanes up to this one.
template <typename F>
__device__ inline uint32_t lanes_upto(uint32_t x, F f) {
  auto step = [&](auto ctrl, auto rows) {
    x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, decltype(rows)::value, 0xF, false));
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});   // row_shr 1, 2, 4, 8
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // lane 15 of the row before, lane 31
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});
  return x;
}
__device__ inline uint32_t sum_upto(uint32_t x) {
  return lanes_upto(x, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ inline uint32_t most_upto(uint32_t x) {
  return lanes_upto(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ inline uint32_t last_lane(uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane((int)x, 63); }

// f over lanes l, l ^ 16, l ^ 32, l ^ 48. The swap exchanges the odd rows of 16 (or the upper 32 lanes) of one copy with the
// even rows (the lower lanes) of the other, so the two copies then hold what is to be joined. (In asm: given one
// value twice, the builtin's two results came out as one register. The nops are the wait between a vector write and
// the swap that reads it.)
template <typename F>
__device__ inline float over_rows(float x, F f) {
  float y = x;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  x = f(x, y);
  y = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return f(x, y);
}

// two e4m3 of a word as two bf16 (exact)
template <bool HIGH>
__device__ inline uint32_t widen8(uint32_t p) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p, 1.0f, HIGH));
}

}  // namespace

// An item is a row, a head of the cache, and up to 16 * RT of the queries that share it; its length counts in tiles of 32
// tokens. An item is cut into equal units of at most S tiles, S by the lengths of all rows (choose, below; lengths are read
// on the device, so a captured call follows them), so long sequences are split over many workgroups and short ones are
// not split at all; the workgroups take units in turn, a unit's tiles divided among the four waves. An item of one unit is written at once; the units of others go
// to the workspace (fp32, written through: output, maximum and sum), and the workgroup that finishes the last of them
// joins them in their order. More than kFan units are joined in two steps, groups of them first, so that no
// workgroup has many to read (one compute unit reads some 50 GB/s). Who is last depends on timing, what it
// computes does not.
//
// The loads of the next unit's first tile are on their way before the results of a unit are summed and stored.
//
// A wave takes 32 tokens at a time through the matrix units, transposed, so that nothing passes between
// lanes on the way: S^T = K Q^T with the tokens as rows and the (up to 16) queries as columns puts into lane
// l the products of query l % 16 with tokens 4 (l / 16) + i of both runs of 16, which is the order in which the
// second product O^T = V^T P^T wants its weights in that lane if token 4 (l / 16) + i of run u is called
// contraction index 8 (l / 16) + 4 u + i. V is read row by row (a lane holds VE channels of 8 tokens) and turned by
// byte permutes inside the lane: fragment m holds channel m of every lane's chunk.
//
// Softmax in one pass: a lane holds the running maximum and sum (in powers of 2) of its query, over its own
// tokens the sum, over all the maximum. The weights enter the second product in bf16 parts, each the bf16 of what the
// ones before leave: two, 16 bits, for a bf16 result, three, the whole fp32, for an fp32 one; the matrix units are far
// from busy (32 tokens of 128 channels are 8 KiB of K and of V, and 24 or 32 matrix instructions).
//
// Bound by reading K and V once. A kernel that only reads reaches 6.9 TB/s on the whole GPU, a copy 5.1:
//   4 rows of 131072 tokens, 8 heads of 128 in 8 bits (1.1 GB)             183 - 187 us    5.9 - 6.1 TB/s    matrix units 0.11 busy
//   61 rows up to 4000 in a window of 1000, 20 heads of 80 (212 MB)     44 - 52 us    4.1 - 4.8 TB/s
//   16 rows up to 8192, 64 heads on 8 of 128 (90 MB)                    25 - 30 us    3.0 - 3.6 TB/s
//   1 row of 500 tokens, 8 heads on 1                                     8.8 us    latency
// (one workgroup a row and head took 2108, 45, 105 and 12 us.) In the third of them planning takes 2.5 us, reading 15, and
// the joins, where one compute unit reads up to 26 results, 5. A short call is a chain of trips to memory: lengths, table,
// K, the results' way through the workspace, the counter, the results again.
template <bool FP8, int DP, int RT, bool OUT32, bool NT>
__global__ void __launch_bounds__(kThreads, RT == 1 && DP <= 128 ? 2 : 1) attn_kernel(const AttnArgs a) {
  constexpr int EL = FP8 ? 1 : 2;
  constexpr int PARTS = OUT32 ? 3 : 2;         // of the weights
  constexpr int KS = DP / 32;                  // contraction steps of the first product
  constexpr int VE = DP / 16;                  // channels of V a lane holds
  constexpr int KL = DP * EL / 64;             // 16-byte loads of a token's keys by a lane
  constexpr int VW = VE * EL / 4;              // words of a token's values in a lane
  constexpr int PO = DP + 4;                   // padded row of the partial results
  __shared__ __attribute__((aligned(16))) float s_o[kAttnWaves][16][PO];
  __shared__ float s_m[kAttnWaves][16], s_l[kAttnWaves][16];
  __shared__ uint32_t s_sum[kAttnWaves][kChoices], s_units[kThreads], s_slots[kThreads], s_last, s_next;

  const agg_kv_cache& cache = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int D = cache.head_dim, pg = cache.page_size;
  // ---- the lengths, and with them the units of each row
  const int room = (int)(a.seq_pages * pg);
  struct Row {
    int seq, lo, hi;                           // its tokens [lo, hi)
    uint32_t tiles;                            // one for an empty row, which has to be written too
  };
  auto row_of = [&](int seq, int n) {
    Row x;
    x.seq = seq;
    x.hi = seq < 0 || seq >= a.seqs || n < 0 ? 0 : n < room ? n : room;
    x.lo = a.window > 0 && x.hi > a.window ? (int)(x.hi - a.window) : 0;
    x.tiles = x.hi > x.lo ? ((uint32_t)x.hi + kTile - 1) / kTile - (uint32_t)x.lo / kTile : 1;
    return x;
  };
  auto row_at = [&](uint32_t r) { return row_of(a.row_seq ? a.row_seq[r] : (int)(a.first_row + r), a.lens[r]); };
  const uint32_t rows = (uint32_t)a.rows, grid = gridDim.x;
  const uint32_t splits = (uint32_t)((a.group + 16 * RT - 1) / (16 * RT)), items = splits * (uint32_t)cache.kv_heads;
  // lane t of every wave holds row t; more than 64 rows: thread t counts rows [t * chunk, + chunk)
  const bool few = rows <= 64;
  const uint32_t chunk = (rows + kThreads - 1) / kThreads;
  Row only{0, 0, 0, 0};
  if (few && (uint32_t)lane < rows) only = row_at((uint32_t)lane);
  auto each_row = [&](auto f) {
    if (few) {
      if (only.tiles) f(only);
    } else {
      for (uint32_t i = 0; i < chunk; ++i) {
        const uint32_t r = (uint32_t)tid * chunk + i;
        if (r < rows) f(row_at(r));
      }
    }
  };
  // sums over the rows
  auto sum_all = [&](auto& v) {
    constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = last_lane(sum_upto(v[k]));
    if (few) return;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) s_sum[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k)
      v[k] = __builtin_amdgcn_readfirstlane(s_sum[0][k] + s_sum[1][k] + s_sum[2][k] + s_sum[3][k]);
    __syncthreads();
  };
  uint32_t all_tiles[1] = {0};
  each_row([&](const Row& x) { all_tiles[0] += x.tiles; });
  sum_all(all_tiles);
  const uint32_t total = all_tiles[0] * items, share = (total + grid - 1) / grid;
  // ---- choose S: of some multiples of an even share, the one that is expected to end first. A unit costs its tiles and
  // as much as kUnitCost of them, and joining units as much as kJoinCost, or twice that in two steps; where every unit has a
  // workgroup of its own the longest one counts, else the mean and half of the longest
  const uint32_t some = share < (uint32_t)a.least ? (uint32_t)a.least : share;
  auto candidate = [&](int k) {
    constexpr uint32_t quarters[kChoices] = {2, 4, 5, 6, 8, 16};
    const uint32_t x = (some * quarters[k] + 3) / 4;
    return x < (uint32_t)a.least ? (uint32_t)a.least : x;
  };
  // (units of a row: tiles / S, rounded up but for 2^-21 of it, by which the reciprocal is shorter: never more)
  auto units_of = [&](uint32_t tiles, float inv) { return (uint32_t)ceilf((float)tiles * inv); };
  auto inverse = [](uint32_t s) { return (1.0f - 0x1p-21f) / (float)s; };
  float inv_most = 1.0f;
  if (few && total <= grid) {
    // a workgroup for every tile: latency counts. Rows that four waves finish in two turns are not split, others at most
    // into as many units as are joined in one step (against the choice below: one row of 500 tokens 9.8 -> 8.8 us, of 2000
    // 13.6 -> 12.5, 16 rows of 800 11.7 -> 10.6)
    const uint32_t longest = last_lane(most_upto(only.tiles)), s = (longest + kFan - 1) / kFan;
    inv_most = inverse(longest <= 8 ? longest : s < (uint32_t)a.least ? (uint32_t)a.least : s);
  } else {
    uint32_t n[kChoices] = {};
    float inv[kChoices];
#pragma unroll
    for (int k = 0; k < kChoices; ++k) inv[k] = inverse(candidate(k));
    each_row([&](const Row& x) {
#pragma unroll
      for (int k = 0; k < kChoices; ++k) n[k] += units_of(x.tiles, inv[k]);
    });
    sum_all(n);
    float best = INFINITY;
#pragma unroll
    for (int k = 0; k < kChoices; ++k) {
      const uint32_t u = n[k] * items;
      const float s = (float)candidate(k);
      const float cost = (u <= grid ? s + kUnitCost : (float)share + 0.5f * s + (float)u / (float)grid * kUnitCost) +
                         (n[k] > rows ? kJoinCost : 0.0f) + (n[k] > kFan * rows ? kJoinCost : 0.0f);
      if (cost < best) {
        best = cost;
        inv_most = inv[k];
      }
    }
  }
  // ---- units, and slots of the workspace, of the rows before each thread's. (An item of more units than one has fewer than
  // twice its tiles over S, and S is at least half of an even share: slots are no more than 4 * grid. An even share of one
  // tile: S is 4 or more, or nothing is split)
  uint32_t units = 0, slots = 0;
  each_row([&](const Row& x) {
    const uint32_t k = units_of(x.tiles, inv_most);
    units += k;
    slots += k > 1 ? k : 0;
  });
  uint32_t upto = sum_upto(units), slots_upto = sum_upto(slots), all_units = last_lane(upto) * items;
  if (!few) {
    if (lane == 63) {
      s_sum[wave][0] = upto;
      s_sum[wave][1] = slots_upto;
    }
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      if (w < wave) {
        upto += s_sum[w][0];
        slots_upto += s_sum[w][1];
      }
      all += s_sum[w][0];
    }
    s_units[tid] = upto;
    s_slots[tid] = slots_upto;
    __syncthreads();
    all_units = __builtin_amdgcn_readfirstlane(all) * items;
  }

  struct Unit {
    uint32_t row;
    int seq, lo, hi;
    int t_lo, t_hi;                            // this wave's tiles
    int head, q0, held;                        // the first of its queries in the head's group, and how many
    uint32_t part, parts;                      // which unit of the item, and of how many
    uint32_t slot;                             // the item's first place in the workspace
  };
  auto locate = [&](uint32_t u) {
    const uint32_t x = u / items;
    uint32_t r, before, slots_before;          // the unit's row, and the units and slots of the rows before it
    Row at;
    if (few) {
      // (rows past the last have the last one's sum, which x is below)
      r = (uint32_t)__popcll(__ballot(upto <= x));
      before = (uint32_t)__builtin_amdgcn_readlane((int)(upto - units), (int)r);
      slots_before = (uint32_t)__builtin_amdgcn_readlane((int)(slots_upto - slots), (int)r);
      at = row_of(__builtin_amdgcn_readlane(only.seq, (int)r), __builtin_amdgcn_readlane(only.hi, (int)r));
    } else {
      // the first thread whose rows reach past x: of every fourth, then of four
      const uint32_t four = (uint32_t)__popcll(__ballot(s_units[4 * lane + 3] <= x)) * 4;
      const uint32_t t = four + (uint32_t)__popcll(__ballot(lane < 4 && s_units[(four + lane) & (kThreads - 1)] <= x));
      before = __builtin_amdgcn_readfirstlane(t ? s_units[t - 1] : 0u);
      slots_before = __builtin_amdgcn_readfirstlane(t ? s_slots[t - 1] : 0u);
      for (r = t * chunk;; ++r) {
        at = row_at(r);
        at = row_of(__builtin_amdgcn_readfirstlane(at.seq), __builtin_amdgcn_readfirstlane(at.hi));
        const uint32_t k = __builtin_amdgcn_readfirstlane(units_of(at.tiles, inv_most));
        if (before + k > x || r + 1 >= rows) break;
        before += k;
        slots_before += k > 1 ? k : 0;
      }
    }
    Unit y;
    y.row = r;
    y.seq = at.seq;
    y.lo = at.lo;
    y.hi = at.hi;
    y.parts = __builtin_amdgcn_readfirstlane(units_of(at.tiles, inv_most));
    const uint32_t in = u - before * items, item = in / y.parts;
    y.part = in - item * y.parts;
    y.head = (int)(item / splits);
    y.q0 = (int)(item % splits) * 16 * RT;
    y.held = a.group - y.q0 < 16 * RT ? a.group - y.q0 : 16 * RT;
    y.slot = slots_before * items + item * y.parts;
    // equal parts, the first ones a tile longer
    const uint32_t base = at.tiles / y.parts, over = at.tiles - base * y.parts;
    const uint32_t from = base * y.part + (y.part < over ? y.part : over), len = base + (y.part < over ? 1 : 0);
    const int first = at.lo / kTile + (int)from;
    y.t_lo = first + (int)(len * (uint32_t)wave / kAttnWaves);
    y.t_hi = at.hi > at.lo ? first + (int)(len * (uint32_t)(wave + 1) / kAttnWaves) : y.t_lo;
    return y;
  };
  const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(a.ws, 0, (int)a.ws_bytes, kBufferFlags);

  // everything from here on, with the cache policy of the keys' and values' loads
  auto attend = [&](auto policy) {
  constexpr int kRead = decltype(policy)::value;
  // offsets of this lane in a run of 16 tokens
  const uint32_t token_bytes = (uint32_t)(cache.ld_token * EL);
  uint32_t koff[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) {
    const int d = FP8 ? i * 64 + g * 16 : i * 32 + g * 8;
    koff[i] = d < D ? (uint32_t)c * token_bytes + (uint32_t)(d * EL) : kOutOfRange;
  }
  // (256 channels of bf16: two loads of 16 bytes, 128 channels apart)
  constexpr int VL = VW > 4 ? VW / 4 : 1, VC = VE / VL;
  uint32_t voff[VL];
#pragma unroll
  for (int i = 0; i < VL; ++i) {
    const int d = i * 16 * VC + c * VC;
    voff[i] = d < D ? (uint32_t)(d * EL) : kOutOfRange;
  }

  // ---- the unit in work, or the next one
  int head = 0, lo = 0, hi = 0;
  const int32_t* table = a.table;
  // the page of each run of 16 tokens, and the place in it: the 128 runs of kBlock tiles from `block` on, in the lanes
  int pages[2] = {-1, -1}, inside[2] = {0, 0}, block = 0;
  auto look_up = [&](int tile) {
    block = tile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t own = (uint32_t)tile * 2 + (uint32_t)(h * 64 + lane), token = own * 16;
      const uint32_t n = (uint32_t)((uint64_t)own * a.page_magic >> a.page_shift);   // own / (page_size / 16)
      pages[h] = (int)token < hi ? table[n] : -1;
      inside[h] = (int)(token - n * (uint32_t)pg);
    }
  };
  struct Run {
    int page, inside;
    int held;                                  // of its 16 tokens, from the first; 0 past the `end` of the tiles
  };
  auto run_of = [&](int tile, int u, int end) {
    const int at = (tile - block) * 2 + u;
    const int p0 = __builtin_amdgcn_readlane(pages[0], at & 63), p1 = __builtin_amdgcn_readlane(pages[1], at & 63);
    const int i0 = __builtin_amdgcn_readlane(inside[0], at & 63), i1 = __builtin_amdgcn_readlane(inside[1], at & 63);
    const int page = at & 64 ? p1 : p0, left = hi - (tile * 2 + u) * 16;
    const bool is = page >= 0 && page < cache.pages && tile < end && left > 0;
    return Run{is ? page : 0, at & 64 ? i1 : i0, is ? (left < 16 ? left : 16) : 0};
  };
  // (readfirstlane: the compiler counts the bytes in vector registers and then loops over the lanes' descriptors, which are
  // the same. No tokens: a descriptor of no bytes, whose loads read nothing and give zeros. The loads stand in straight
  // lines, since behind a branch the compiler waits for all of them where it needs the older half)
  auto descriptor = [&](const void* pool, const Run& r) {
    const int64_t at = (int64_t)r.page * cache.ld_page + (int64_t)r.inside * cache.ld_token + (int64_t)head * cache.ld_head;
    const int bytes = (int)((uint32_t)(r.held - 1) * token_bytes + (uint32_t)(D * EL));
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(static_cast<const uint8_t*>(pool)) + at * EL, 0,
                                             __builtin_amdgcn_readfirstlane(r.held ? bytes : 0), kBufferFlags);
  };
  auto load_scales = [&](const float* scales, const Run& r) {
    const __amdgpu_buffer_rsrc_t d = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(scales) + ((int64_t)r.page * cache.kv_heads + head) * pg + r.inside, 0, r.held ? 64 : 0, kBufferFlags);
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(d, 16 * g, 0, 0));
  };

  struct Keys {
    u32x4 k[2][KL];
    f32x4 scale[2];
    int held[2];
  };
  struct Values {
    uint32_t v[2][4][VW];
    f32x4 scale[2];
  };
  auto load_keys = [&](Keys& x, int tile, int end) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Run r = run_of(tile, u, end);
      x.held[u] = r.held;
      const __amdgpu_buffer_rsrc_t d = descriptor(cache.k, r);
#pragma unroll
      for (int i = 0; i < KL; ++i)
        x.k[u][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(d, (int)koff[i], 0, kRead));
      if constexpr (FP8) x.scale[u] = load_scales(cache.k_scale, r);
    }
  };
  auto load_values = [&](Values& x, int tile, int end) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const Run r = run_of(tile, u, end);
      const __amdgpu_buffer_rsrc_t d = descriptor(cache.v, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (a value before the window may be anything, and zero times it a NaN: it is not read)
        const int token = tile * kTile + u * 16 + 4 * g + i;
        const uint32_t skip = token < lo ? kOutOfRange : 0u;
        const uint32_t base = (uint32_t)(4 * g + i) * token_bytes;
#pragma unroll
        for (int p = 0; p < VL; ++p) {
          const int off = (int)((voff[p] + base) | skip | (voff[p] & kOutOfRange));
          if constexpr (VW >= 4) {
            const u32x4 w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(d, off, 0, kRead));
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[u][i][4 * p + e] = w[e];
          } else if constexpr (VW == 2) {
            const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(d, off, 0, kRead));
            x.v[u][i][0] = w[0];
            x.v[u][i][1] = w[1];
          } else {
            x.v[u][i][0] = __builtin_amdgcn_raw_buffer_load_b32(d, off, 0, kRead);
          }
        }
      }
      if constexpr (FP8) x.scale[u] = load_scales(cache.v_scale, r);
    }
  };

  Keys kx;
  Values vx;
  u32x4 qf[RT][KS];
  auto begin = [&](const Unit& u) {
    head = u.head;
    lo = u.lo;
    hi = u.hi;
    table = a.table + (hi > 0 ? u.seq * a.ld_table : 0);
    look_up(u.t_lo);                           // (before Q: its wait is a wait for what was asked for earlier too)
    // Q: column c, steps of 32 channels; lane's 8 of step s as K's lane has them
    const uint16_t* const q = a.q + (int64_t)u.row * a.ld_q + (int64_t)(head * a.group + u.q0) * D;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d = FP8 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
        const int j = r * 16 + c;
        qf[r][s] = u32x4{};
        if (j < u.held && d < D) qf[r][s] = *reinterpret_cast<const u32x4*>(q + j * D + d);
      }
    load_keys(kx, u.t_lo, u.t_hi);
    load_values(vx, u.t_lo, u.t_hi);
  };

  // ---- the first unit by the workgroup's number; of further ones, where there are more units than workgroups, the
  // next that nobody has (asked for while a unit is in work)
  uint32_t number = blockIdx.x;
  if (number >= all_units) return;
  const bool claims = all_units > grid;
  uint32_t* const claimed = a.counts + 8 * grid;
  Unit now = locate(number);
  begin(now);
  for (;;) {
  uint32_t claim = 0;
  if (claims && tid == 0) claim = grid + __hip_atomic_fetch_add(claimed, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  f32x4 o[RT][VE];
  float m[RT], l[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < VE; ++e) o[r][e] = f32x4{};
  }
  for (int from = now.t_lo; from < now.t_hi; from += kBlock) {
  if (from > now.t_lo) {
    look_up(from);
    load_keys(kx, from, now.t_hi);
    load_values(vx, from, now.t_hi);
  }
  const int to = now.t_hi - from < kBlock ? now.t_hi : from + kBlock;
  for (int tile = from; tile < to; ++tile) {
    // ---- S^T, times the scale and in powers of 2
    f32x4 s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        s[r][u] = f32x4{};
#pragma unroll
        for (int st = 0; st < KS; ++st) {
          u32x4 f;
          if constexpr (FP8) {
            const u32x4 w = kx.k[u][st >> 1];
            const uint32_t x = w[(st & 1) * 2], y = w[(st & 1) * 2 + 1];
            f = u32x4{widen8<false>(x), widen8<true>(x), widen8<false>(y), widen8<true>(y)};
          } else {
            f = kx.k[u][st];
          }
          s[r][u] = mfma16(f, qf[r][st], s[r][u]);
        }
      }
    bool in[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        in[u][i] = 4 * g + i < kx.held[u] && tile * kTile + u * 16 + 4 * g + i >= lo;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[r][u][i] * a.scale2;
          if constexpr (FP8) x *= kx.scale[u][i];
          s[r][u][i] = in[u][i] ? x : -INFINITY;
        }
    // (the scheduling barriers keep the loads where they stand: the compiler otherwise moves them to the loop's end)
    __builtin_amdgcn_sched_barrier(0);
    load_keys(kx, tile + 1, to);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[r][u][i]);
      top = over_rows(top, [](float x, float y) { return fmaxf(x, y); });
      const float now = fmaxf(m[r], top);
      const float base = now == -INFINITY ? 0.0f : now;   // (nothing so far)
      const float shrink = __builtin_amdgcn_exp2f(m[r] - base);
      m[r] = now;
      l[r] *= shrink;
#pragma unroll
      for (int e = 0; e < VE; ++e) o[r][e] *= shrink;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[r][u][i] = __builtin_amdgcn_exp2f(s[r][u][i] - base);
          l[r] += s[r][u][i];
          if constexpr (FP8) s[r][u][i] = in[u][i] ? s[r][u][i] * vx.scale[u][i] : 0.0f;
        }
    }
    // ---- O^T
    u32x4 w[RT][PARTS];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float x = s[r][p >> 1][2 * (p & 1)], y = s[r][p >> 1][2 * (p & 1) + 1];
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
          w[r][t][p] = pack2(x, y);
          x -= low_half(w[r][t][p]);
          y -= high_half(w[r][t][p]);
        }
      }
    // fragments of two channels at a time
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      uint32_t v[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if constexpr (FP8) {
          const uint32_t x = vx.v[t >> 2][t & 3][e / 4];
          v[t] = e & 2 ? widen8<true>(x) : widen8<false>(x);
        } else {
          v[t] = vx.v[t >> 2][t & 3][e / 2];
        }
      }
      u32x4 f0, f1;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        f0[p] = __builtin_amdgcn_perm(v[2 * p + 1], v[2 * p], 0x05040100u);
        f1[p] = __builtin_amdgcn_perm(v[2 * p + 1], v[2 * p], 0x07060302u);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
          o[r][e] = mfma16(f0, w[r][t], o[r][e]);
          o[r][e + 1] = mfma16(f1, w[r][t], o[r][e + 1]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_values(vx, tile + 1, to);
    __builtin_amdgcn_sched_barrier(0);
  }
  }

  // ---- the waves' results, 16 queries at a time
  const Unit done = now;
  bool more = false;
  __syncthreads();                             // (everyone is past the last unit's s_o, s_m, s_l and s_last)
  if (claims) {
    if (tid == 0) s_next = claim;
    __syncthreads();
    number = __builtin_amdgcn_readfirstlane(s_next);
    more = number < all_units;
  }
  if (more) {
    now = locate(number);
    begin(now);
  }
  // a result: query j of the item, channels d .. d + 3
  auto finish = [&](int j, int d, float top, float sum, const f32x4& y) {
    const float inv = sum > 0.0f ? 1.0f / sum : sum;       // (a NaN stays one)
    const int qh = done.head * a.group + done.q0 + j;
    const int64_t to = (int64_t)done.row * a.ld_out + (int64_t)qh * D + d;
    const f32x4 v = y * inv;
    if constexpr (OUT32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to) = v;
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + to) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
    if (a.lse && d == 0) a.lse[(int64_t)done.row * a.q_heads + qh] = sum > 0.0f ? top * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
  };
  // a place of the workspace: its queries' outputs, then their maxima and sums, and the same of a group
  auto put = [&](uint32_t slot, int step, int j, int d, float top, float sum, const f32x4& y) {
    const uint32_t to = slot * (uint32_t)a.slot_bytes;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), ws, (int)(to + (uint32_t)(j * D + d) * 4), 0, kCoherent);
    if (d == 0)
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{top, sum}), ws,
                                            (int)(to + (uint32_t)(done.held * (D + 2 * step) + 2 * j) * 4), 0, kCoherent);
  };
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r * 16 >= done.held) break;
    const float sum = over_rows(l[r], [](float x, float y) { return x + y; });
    if (r > 0) __syncthreads();
    if (g == 0) {
      s_m[wave][c] = m[r];
      s_l[wave][c] = sum;
    }
    // row 4 g + i of fragment e is channel e of chunk 4 g + i
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < VE; e += 4)
        *reinterpret_cast<f32x4*>(&s_o[wave][c][e / VC * 16 * VC + (4 * g + i) * VC + e % VC]) =
            f32x4{o[r][e][i], o[r][e + 1][i], o[r][e + 2][i], o[r][e + 3][i]};
    __syncthreads();
    for (int x = tid; x < 16 * (DP / 4); x += kThreads) {
      const int j = x / (DP / 4), d = x % (DP / 4) * 4;
      if (r * 16 + j >= done.held || d >= D) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, s_m[w][j]);
      const float base = top == -INFINITY ? 0.0f : top;
      float all_sum = 0.0f;
      f32x4 y = f32x4{};
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        const float by = __builtin_amdgcn_exp2f(s_m[w][j] - base);
        all_sum += by * s_l[w][j];
        y += by * *reinterpret_cast<const f32x4*>(&s_o[w][j][d]);
      }
      if (done.parts == 1) finish(r * 16 + j, d, top, all_sum, y);
      else put(done.slot + done.part, 0, r * 16 + j, d, top, all_sum, y);
    }
  }
  if (done.parts > 1) {
    // ---- the units' results, in groups of `fan` and then the groups'
    auto arrive = [&](uint32_t counter, uint32_t expected) {
      // (the stores have completed, so no fence is needed: who reads them bypasses the caches too. The count is left at
      // zero for the next launch)
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = __hip_atomic_fetch_add(a.counts + counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = before == expected - 1;
        if (before == expected - 1) __hip_atomic_store(a.counts + counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      return __builtin_amdgcn_readfirstlane(s_last) != 0;
    };
    // the results in slots first, first + apart, ... (n of them) as one; `give` takes it
    auto join = [&](uint32_t first, uint32_t apart, uint32_t n, int step, auto give) {
      const int quads = D / 4;
      // threads of a quad: as many as there are to spare, up to 8, each every so manyth result
      uint32_t log2 = 0;
      while (log2 < 3 && (done.held * quads) << (log2 + 1) <= kThreads) ++log2;
      const uint32_t sub = (uint32_t)tid & ((1u << log2) - 1), stride = 1u << log2;
      for (int x = tid >> log2; x < (done.held * quads + (kThreads >> log2) - 1) / (kThreads >> log2) * (kThreads >> log2);
           x += kThreads >> log2) {
        const bool in = x < done.held * quads;
        const int j = in ? x / quads : 0, d = in ? x % quads * 4 : 0;
        float top = -INFINITY, sum = 0.0f;
        f32x4 y = f32x4{};
        auto take = [&](auto batch) {
        constexpr int B = decltype(batch)::value;
        for (uint32_t i0 = sub; i0 < n; i0 += B * stride) {
          f32x4 v[B];
          f32x2 ms[B];
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const uint32_t i = i0 + b * stride;
            const uint32_t from = i < n ? (first + i * apart) * (uint32_t)a.slot_bytes : kOutOfRange;
            v[b] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                ws, (int)((from + (uint32_t)(j * D + d) * 4) | (from & kOutOfRange)), 0, kCoherent));
            ms[b] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(
                ws, (int)((from + (uint32_t)(done.held * (D + 2 * step) + 2 * j) * 4) | (from & kOutOfRange)), 0, kCoherent));
            if (i >= n) ms[b][0] = -INFINITY;
          }
          float high = top;
#pragma unroll
          for (int b = 0; b < B; ++b) high = fmaxf(high, ms[b][0]);
          const float base = high == -INFINITY ? 0.0f : high;
          const float keep = __builtin_amdgcn_exp2f(top - base);
          sum *= keep;
          y *= keep;
          top = high;
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const float by = __builtin_amdgcn_exp2f(ms[b][0] - base);
            sum += by * ms[b][1];
            y += by * v[b];
          }
        }
        };
        // (as many loads in flight as there are registers; few where few are enough)
        if (n <= 4 * stride) take(std::integral_constant<int, 4>{});
        else take(std::integral_constant<int, RT == 1 && DP <= 128 ? 16 : 8>{});
        for (uint32_t s = 1; s < stride; s *= 2) {
          const float other = __shfl_xor(top, (int)s);
          const float both = fmaxf(top, other), base = both == -INFINITY ? 0.0f : both;
          const float keep = __builtin_amdgcn_exp2f(top - base), take = __builtin_amdgcn_exp2f(other - base);
          top = both;
          sum = keep * sum + take * __shfl_xor(sum, (int)s);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = keep * y[e] + take * __shfl_xor(y[e], (int)s);
        }
        if (in && sub == 0) give(j, d, top, sum, y);
      }
    };
    if (done.parts <= kFan) {
      if (arrive(done.slot, done.parts)) join(done.slot, 1, done.parts, 0, finish);
    } else {
      // (S is half an even share at least, so an item has twice as many units as there are workgroups at most: kFan^2. The
      // number itself is read where it is needed: as a constant it costs the loop registers, 16 rows up to 8192 29.5 -> 31.0 us)
      uint32_t fan = kFan;
      asm volatile("" : "+s"(fan));
      const uint32_t group = done.part / fan, lead = done.slot + group * fan, groups = (done.parts + fan - 1) / fan;
      const uint32_t n = done.parts - group * fan < fan ? done.parts - group * fan : fan;
      if (arrive(lead, n)) {
        // (the thread that reads an element of the leader's output writes it; the maxima and sums, which others
        // read too, have a second place)
        join(lead, 1, n, 0, [&](int j, int d, float top, float sum, const f32x4& y) { put(lead, 1, j, d, top, sum, y); });
        if (arrive(4 * grid + done.slot, groups)) join(done.slot, fan, groups, 1, finish);
      }
    }
  }
  if (!more) break;
  }
  if (!claims) return;
  // the last workgroup to end leaves the counters at zero (all claims came before)
  if (tid == 0 && __hip_atomic_fetch_add(claimed + 1, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == grid - 1) {
    __hip_atomic_store(claimed, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(claimed + 1, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  };

  // Non-temporal where the call reads more than the last level's 256 MB can hold, each token once: not more tokens than the
  // pool has, which rows that share pages would (measured at the launch, below)
  if constexpr (NT) {
    const float token = 2.0f * (float)(cache.kv_heads * D * EL), held = (float)cache.pages * (float)pg;
    if ((float)all_tiles[0] * (kTile * token) > 256e6f && (float)(all_tiles[0] - rows) * kTile <= held) {
      attend(std::integral_constant<int, 2>{});
      return;
    }
  }
  attend(std::integral_constant<int, 0>{});
}

template <bool FP8, int DP, int RT, bool NT>
static hipError_t launch_attn_nt(const AttnArgs& a, int grid, hipStream_t stream) {
  const dim3 g((unsigned)grid), b(kThreads);
  if (a.out_fp32) hipLaunchKernelGGL((attn_kernel<FP8, DP, RT, true, NT>), g, b, 0, stream, a);
  else hipLaunchKernelGGL((attn_kernel<FP8, DP, RT, false, NT>), g, b, 0, stream, a);
  return hipGetLastError();
}

template <bool FP8, int DP, int RT>
static hipError_t launch_attn_rt(const AttnArgs& a, int grid, hipStream_t stream) {
  // Non-temporal reads keep a cache that the last level's 256 MB cannot hold out of it. They pay where the lines of 128 bytes
  // are one head's each and neighbours, and every line is read once: 4 x 131072 tokens of 8 bits, heads first, 203 -> 189 us;
  // 32 x 8000 bf16 185 -> 170; 32 x 8000 of 16 heads of 64 bf16 180 -> 161; 256 wide 171 -> 163. Where a line is asked
  // for in parts at different times they cost: 80 wide 347 -> 420, tokens first 8 bits of 128 118 -> 124, bf16 of 128 189 and
  // 188. So they do where rows share pages (64 x 8000, 7200 shared, 151 -> 194; 32 x 32000, all but 160 shared, 285 -> 440), and
  // a little where a call reads little of a large pool (16 x 2000 bf16 27.5 -> 29.1): the kernel, which knows the lengths,
  // leaves them out there. Rows that share pages of a pool that could hold them apart are not told (32 x 16000 in 8 bits, 15200
  // shared, 120 -> 130). More queries than 16 to a head of the cache: what one workgroup reads another may
  if constexpr (RT == 1) {
    const int row = a.cache.head_dim * (FP8 ? 1 : 2);
    const double bytes = 2.0 * (double)a.cache.pages * a.cache.page_size * a.cache.kv_heads * row;
    if (bytes > 256e6 && row % 128 == 0 && (a.cache.ld_token == a.cache.head_dim || row >= 512))
      return launch_attn_nt<FP8, DP, 1, true>(a, grid, stream);
  }
  return launch_attn_nt<FP8, DP, RT, false>(a, grid, stream);
}

template <bool FP8, int DP>
static hipError_t launch_attn_dp(const AttnArgs& a, int grid, hipStream_t stream) {
  if (a.row_tiles == 1) return launch_attn_rt<FP8, DP, 1>(a, grid, stream);
  if (a.row_tiles == 2) return launch_attn_rt<FP8, DP, 2>(a, grid, stream);
  if constexpr (DP < 256) return launch_attn_rt<FP8, DP, 4>(a, grid, stream);
  else return hipErrorInvalidValue;
}

template <bool FP8>
static hipError_t launch_attn_type(const AttnArgs& a, int grid, hipStream_t stream) {
  if (a.cache.head_dim <= 64) return launch_attn_dp<FP8, 64>(a, grid, stream);
  if (a.cache.head_dim <= 128) return launch_attn_dp<FP8, 128>(a, grid, stream);
  return launch_attn_dp<FP8, 256>(a, grid, stream);
}

hipError_t launch_attn(const AttnArgs& a, int grid, hipStream_t stream) {
  return a.cache.dtype == AGG_FP8_E4M3 ? launch_attn_type<true>(a, grid, stream) : launch_attn_type<false>(a, grid, stream);
}

}  // namespace agg
