// The MoE FFN layer for a few tokens (a decode step): the same layer as the prefill call, on
// the same resident int4 banks, arranged around reading each chosen expert's weights once.
//   route    top-k gate and the chosen experts' rows (two blocks), e4m3 of x (a block a token)
//   gate_up  a unit is 16 hidden features of one expert: 8 gate rows and their 8 up rows are
//            the 16 rows of a warp-level MMA, twice; the expert's tokens are its 8-column
//            side; then silu(gate) * up, and who completes 128 features quantizes them
//   down     a unit is 32 output features of one expert; float32 results
//   combine  the gate-weighted sums of the results, in slot order
// For a few tokens of a small layer two launches do it all: every block of gate_up works out the
// routes and quantizes x for itself, down's blocks quantize the hidden rows of their segments, and
// the block that completes 32 output features of down sums them.
// A weight is used for at most 64 tokens, so the layer is bound by the weight stream (3 H I / 2
// bytes of codes and 3 H I / 32 of scales an expert).  gate_up and down are one kernel: the
// units of all segments (an expert and at most 8 NT of its rows) are cut into equal runs, one
// to an SM; a segment's activations lie in shared memory in the order the MMA reads them, and
// every warp keeps kDepth - 1 chunks of 32 rows x 128 weights in flight through its own ring in
// shared memory, each lane reading back what it copied, so the stream needs no block barrier.
// Two row tiles to a unit halve what each token tile costs (reading and widening its codes).
// Where there are few units, several warps share one unit's K.
//   Warp-level e4m3 MMAs take their operands apart into fp16 here, so the products are fp16
// MMAs from the start.  A nibble is an fp16 operand as it stands: with its sign bit flipped it
// is u = q + 8, and the bits 0..15 in the lowest places of a half are the subnormal u 2^-24, in
// the next four u 2^-20; a mask takes two weights at a time out of a word, and only every other
// pair needs a shift.  The sum of a u is brought back to that of a q by adding -8 times the
// group's sum of a, which the activation's quantizer leaves beside its scale.  The products are
// exact: a has 4 significant bits, u 4; the sums are float32.
//   Measured (device time of a call): H = 2048, I = 768, 64 experts, top-8: one token 20.8 us
// (20 MB: bound by the starts of two kernels and the steps of routing), 64 tokens 77 us.  H = 4096,
// I = 1536, 128 experts: 13 tokens 92 us (295 MB), 64 tokens 172 us (518 MB): gate_up 101 us at
// 3.5 TB/s and down 51 us at 3.4 TB/s, with the warps' MMAs 34%, the ALU 48% and the issue slots
// 47% busy and three warps a scheduler to hide their latencies; the registers of four column
// tiles leave no room for more (16 warps: 302 us).
#include <algorithm>

#include "chain.cuh"
#include "fge_device.cuh"
#include "quotient.cuh"

namespace fge {

namespace {

constexpr int kMaxRows = kMoeDecodeTokens * 32;
constexpr int kMaxSegments = kMaxExperts + kMaxRows / 8;
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kRouteThreads = 1024;
constexpr int kUnitRows = 32;                      // bank rows of a unit: two MMA row tiles
constexpr int kSlotBytes = kUnitRows * 64 + 128;   // a chunk: one 128 group of 32 rows, scales
constexpr int kDepth = 4;                          // chunks of a warp's ring (6: no faster)
constexpr int kRingBytes = kWarps * kDepth * kSlotBytes;
constexpr int kTiles = 8;                          // most column tiles in shared memory
constexpr int kSmemMost = 227 * 1024;

// At most 8 * tiles rows of one expert, the rows that a unit multiplies at a time.
struct alignas(16) Segment {
  int32_t expert, row0, rows, pad;
};
__device__ __forceinline__ Segment load_segment(const Segment* s) {
  const int4 v = __ldcg(reinterpret_cast<const int4*>(s));
  return Segment{v.x, v.y, v.z, 0};
}

// Routing results in the workspace.
constexpr int kMaxBlocks = 1024;
struct Routes {
  int2 run[2][kMaxBlocks];         // units [x, y) of every block of gate_up and of down
  Segment segment[2][kMaxSegments];
  int32_t row_token[kMaxRows];     // rows ordered by (expert, token)
  int32_t token_row[kMaxRows];     // [T, k]
  float gate[kMaxRows];            // [T, k]
};

struct Ws {
  Routes* routes;
  // finished units of 128 hidden features [segments of gate_up, I / 128]; with few tokens,
  // finished experts of 32 output features [H / 32]
  int32_t* count;
  uint8_t* xq;     // [T, H] codes, in the order of the bank's nibbles
  float2* xs;      // [T, H / 128] scale s and -8 * 2^-24 * s * sum of the codes
  float* h;        // [R, I] hidden values
  uint8_t* hq;     // [R, I] codes, likewise
  float2* hs;      // [R, I / 128]
  float* y;        // [R, H]
  size_t bytes;
};

// Segments that T tokens can make: one an expert, and one more for every 8 rows.
int64_t most_segments(int64_t T, int E, int k) {
  return std::min<int64_t>(T * k, E) + T * k / 8;
}

Ws carve(void* base, int64_t T, int64_t H, int64_t I, int E, int k) {
  Ws w{};
  const int64_t R = T * k;
  size_t off = 0;
  auto take = [&](size_t n) {
    void* p = base ? static_cast<uint8_t*>(base) + off : nullptr;
    off += align_up(n, 256);
    return p;
  };
  w.routes = static_cast<Routes*>(take(sizeof(Routes)));
  w.count = static_cast<int32_t*>(
      take(std::max<int64_t>(most_segments(T, E, k) * (I / 128), H / kUnitRows) * 4));
  w.xq = static_cast<uint8_t*>(take(T * H));
  w.xs = static_cast<float2*>(take(T * (H / 128) * 8));
  w.h = static_cast<float*>(take(R * I * 4));
  w.hq = static_cast<uint8_t*>(take(R * I));
  w.hs = static_cast<float2*>(take(R * (I / 128) * 8));
  w.y = static_cast<float*>(take(R * H * 4));
  w.bytes = off;
  return w;
}

// ------------------------------------------------------------------------------- route
// Sum of the values that 4 e4m3 codes stand for.
__device__ __forceinline__ float e4m3x4_sum(uint32_t codes) {
  const __half2_raw l = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&l));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return (a.x + a.y) + (b.x + b.y);
}

// The codes of 8 values in the order in which pairs of nibbles leave a bank's word: nibbles
// (0, 4) and (2, 6), then (1, 5) and (3, 7).  A byte of the subnormal bank holds elements b and
// b + 4; in the other one nibble i is element i.
template <bool SUB>
__device__ __forceinline__ uint2 nibble_order(uint2 q) {
  return SUB ? make_uint2(__byte_perm(q.x, q.x, 0x3120), __byte_perm(q.y, q.y, 0x3120))
             : make_uint2(__byte_perm(q.x, q.y, 0x6240), __byte_perm(q.x, q.y, 0x7351));
}

// e4m3 of one token, half a warp a 128 group.
template <bool SUB>
__device__ __forceinline__ void quantize_token(const uint16_t* __restrict__ x, int H,
                                               uint8_t* __restrict__ xq, float2* __restrict__ xs,
                                               int32_t* status) {
  const int lane = threadIdx.x & 15;
  for (int g = threadIdx.x >> 4; g < H / 128; g += kRouteThreads / 16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + g * 16 + lane);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((w[i] >> 16) & 0x7FFFu, w[i] & 0x7FFFu));
    const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(half, m, d));
    if (m >= 0x7F80u) set_device_error(status, FGE_ERR_NONFINITE);
    const float s = scale_from_amax(__uint_as_float(m << 16));
    const uint2 q = cast8(v, s, __frcp_rn(s), quot_fast_ok(s));
    float sum = e4m3x4_sum(q.x) + e4m3x4_sum(q.y);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(half, sum, d);
    reinterpret_cast<uint2*>(xq)[g * 16 + lane] = nibble_order<SUB>(q);
    if (lane == 0) xs[g] = make_float2(s, s * (sum * (-8.0f * 0x1p-24f)));
  }
}

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = f == 0.0f ? 0u : __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// Gates of a warp's first k lanes from their logits, the largest first.
__device__ __forceinline__ float top_gate(float logit, int k) {
  const float m = __shfl_sync(0xffffffffu, logit, 0);
  const float ex = (threadIdx.x & 31) < k ? expf(logit - m) : 0.0f;
  float sum = ex;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return __fdiv_rn(ex, sum);
}

// Top-k of one token (PER logits a lane): lane j < k gets slot j's expert and gate.
template <int PER>
__device__ __forceinline__ void topk_token(const float* __restrict__ logits, int E, int k,
                                           int* id, float* gate) {
  constexpr uint32_t kNone = 0x7fffffffu;
  const int lane = threadIdx.x & 31;
  // this lane's logits in order, equal ones by their number
  uint32_t key[PER], num[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool there = lane + 32 * i < E;
    key[i] = there ? order_key(__ldg(logits + lane + 32 * i)) : 0u;
    num[i] = there ? lane + 32 * i : kNone;
  }
  auto swap_if = [&](int i, int j) {
    if (key[j] > key[i]) {
      const uint32_t ks = key[i], ns = num[i];
      key[i] = key[j];
      num[i] = num[j];
      key[j] = ks;
      num[j] = ns;
    }
  };
  constexpr bool kSorted = PER <= 4;  // more would not fit the registers
  if constexpr (kSorted) {
#pragma unroll
    for (int n = PER - 1; n > 0; --n)
#pragma unroll
      for (int i = 0; i < n; ++i) swap_if(i, i + 1);
  }
  float my_val = 0.0f;
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    if constexpr (!kSorted) {  // the best one to the front; ties by number, as they lie apart
#pragma unroll
      for (int i = 1; i < PER; ++i)
        if (key[i] > key[0] || (key[i] == key[0] && num[i] < num[0])) {
          const uint32_t ks = key[0], ns = num[0];
          key[0] = key[i];
          num[0] = num[i];
          key[i] = ks;
          num[i] = ns;
        }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
    const uint32_t who = __ballot_sync(0xffffffffu, key[0] == top);
    const uint32_t win =
        (who & (who - 1)) ? __reduce_min_sync(0xffffffffu, key[0] == top ? num[0] : kNone)
                          : __shfl_sync(0xffffffffu, num[0], __ffs(who) - 1);
    if (win == num[0]) {
      if constexpr (kSorted) {
#pragma unroll
        for (int i = 0; i + 1 < PER; ++i) {
          key[i] = key[i + 1];
          num[i] = num[i + 1];
        }
      }
      key[kSorted ? PER - 1 : 0] = 0u;
      num[kSorted ? PER - 1 : 0] = kNone;
    }
    if (lane == j) {
      my_val = key_value(top);
      my_id = static_cast<int>(win);
    }
  }
  *id = my_id;
  *gate = top_gate(my_val, k);
}

struct RouteSmem {
  unsigned long long mask[kMaxExperts];  // tokens of an expert
  int32_t start[kMaxExperts];
  uint16_t id[kMaxRows];
  uint32_t warp_sum[kRouteThreads / 32];
  int32_t before[kMaxSegments + 1];      // cost of the segments before
  uint8_t tiles[kMaxSegments];
  int32_t fits;
};

// Exclusive sum over the block's threads; *total: of all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* total, uint32_t* warp_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t in = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, in, d);
    if (lane >= d) in += o;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = in;
  __syncthreads();
  uint32_t ws = warp_sum[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, ws, d);
    if (lane >= d) ws += o;
  }
  *total = __shfl_sync(0xffffffffu, ws, 31);
  return in - v + (warp ? __shfl_sync(0xffffffffu, ws, warp - 1) : 0);
}

// How one of the two kernels cuts its units.
struct CutArgs {
  int blocks, units, tiles;  // blocks; units of a segment; most column tiles of a segment
  int light;                 // shared memory holds two segments of at most so many tiles
};
// Cost of a unit by its column tiles, from the large layer: 2.0 us with one tile, 3.3 with two,
// and 1.7 against 3.7 with three where no warps share a unit.
__device__ __forceinline__ int unit_cost(int tiles) { return 2 + 3 * tiles; }

// The runs of units, one a block.  The light segments come first and are cut at equal cost: a
// block can hold the activations of both segments that its run spans.  A heavy segment gets a
// whole number of blocks (a run across its border would work off its two parts one after the
// other, half idle: 87 us instead of 50 us for 13 tokens of the large layer).  The blocks are
// shared out by the smallest largest run.
__device__ __forceinline__ void cut_runs(const CutArgs& c, int n_segments, int n_light,
                                         int2* __restrict__ run, RouteSmem& sm) {
  const int tid = threadIdx.x;
  const int cost = tid < n_segments ? unit_cost(sm.tiles[tid]) * c.units : 0;
  uint32_t total;
  const uint32_t before = block_scan(cost, &total, sm.warp_sum);
  if (tid <= n_segments && tid < kRouteThreads) sm.before[tid] = static_cast<int32_t>(before);
  if (n_segments - n_light + 1 > c.blocks) n_light = n_segments;
  if (tid == 0) sm.fits = 63;
  int light_blocks = c.blocks, high = 0;
  __syncthreads();
  if (n_light < n_segments) {
    // The smallest cost of a run among 64 candidates, half a warp each.  A run of twice the mean
    // is enough where the heavy segments are fewer than half the blocks: each adds less than one.
    const uint32_t light_cost = sm.before[n_light];
    const uint32_t low = (total + c.blocks - 1) / c.blocks;
    const uint32_t top = 2 * (n_segments - n_light + 1) <= c.blocks
                             ? 2 * low + 1
                             : max(static_cast<uint32_t>(unit_cost(kTiles) * c.units), light_cost);
    const uint32_t width = (max(top, low) - low + 63) / 64;
    const int half = tid >> 4, in_half = tid & 15;
    const uint32_t candidate = low + width * (half + 1);
    uint32_t need = in_half == 0 ? (light_cost + candidate - 1) / candidate : 0;
    for (int i = n_light + in_half; i < n_segments; i += 16)
      need += (static_cast<uint32_t>(unit_cost(sm.tiles[i]) * c.units) + candidate - 1) / candidate;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) need += __shfl_xor_sync(0xffffffffu, need, d);
    if (in_half == 0 && need <= static_cast<uint32_t>(c.blocks)) atomicMin(&sm.fits, half);
    __syncthreads();
    high = static_cast<int>(low + width * (min(sm.fits, 63) + 1));
    const int mine = tid >= n_light && tid < n_segments ? (cost + high - 1) / high : 0;
    uint32_t used_blocks;
    const int at = static_cast<int>(block_scan(mine, &used_blocks, sm.warp_sum));
    const int used = static_cast<int>(used_blocks);
    light_blocks = n_light ? c.blocks - used : 0;
    for (int j = 0; j < mine; ++j)
      run[light_blocks + at + j] = make_int2(tid * c.units + c.units * j / mine,
                                             tid * c.units + c.units * (j + 1) / mine);
    if (tid >= light_blocks + used && tid < c.blocks) run[tid] = make_int2(0, 0);
  }
  if (n_light) {
    const uint32_t light_cost = n_light == n_segments ? total : sm.before[n_light];
    auto unit_at = [&](int at) {
      int l = 0, h = n_light;  // the last segment that begins at or before `at`
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (sm.before[mid] <= at) l = mid; else h = mid;
      }
      return l * c.units + (at - sm.before[l]) / unit_cost(sm.tiles[l]);
    };
    if (tid < light_blocks) {
      // light_cost * i / light_blocks without leaving 32 bits
      const uint32_t each = light_cost / light_blocks, over = light_cost % light_blocks;
      auto share = [&](uint32_t i) {
        return static_cast<int>(each * i + over * i / static_cast<uint32_t>(light_blocks));
      };
      const int lo = unit_at(share(tid));
      const int hi = tid + 1 < light_blocks ? unit_at(share(tid + 1)) : n_light * c.units;
      run[tid] = make_int2(lo, hi);
    }
  }
  __syncthreads();
}

// Top-k of every token and the experts' rows in order of (expert, token): a warp a token (PER
// logits a lane), then per expert the set of its tokens as 64 bits, whose counts give every row
// its place.  Two blocks do it, one for each of the kernels that follow (`which`).
template <int PER>
__device__ __forceinline__ void route(const float* __restrict__ logits, int T, int E, int k,
                                      const CutArgs& cut, int which, Routes* __restrict__ out,
                                      RouteSmem& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kMaxExperts) sm.mask[tid] = 0;
  __syncthreads();
  for (int t = warp; t < T; t += kRouteThreads / 32) {
    int my_id;
    float gate;
    topk_token<PER>(logits + t * E, E, k, &my_id, &gate);
    if (lane < k) {
      sm.id[t * k + lane] = static_cast<uint16_t>(my_id);
      if (which) out->gate[t * k + lane] = gate;
      // half of the set: 64-bit atomics on shared memory are loops
      atomicOr(reinterpret_cast<uint32_t*>(&sm.mask[my_id]) + (t >> 5), 1u << (t & 31));
    }
  }
  __syncthreads();
  // an expert a thread: its first row, and its segments
  const int c = tid < kMaxExperts ? __popcll(sm.mask[tid]) : 0;
  // its segments: full ones and one of what is left, the light ones of all experts first
  const int most = 8 * cut.tiles, n = (c + most - 1) / most;
  const int rest = c - (n - 1) * most;  // rows of the last one
  const int full_light = cut.tiles <= cut.light;
  const int last_light = n && (rest + 7) / 8 <= cut.light;
  const int light = n ? (n - 1) * full_light + last_light : 0;
  // three sums in one word: rows, light segments, heavy ones
  static_assert(kMaxRows < 1 << 12 && kMaxSegments < 1 << 10, "fields of 12, 10 and 10 bits");
  uint32_t total;
  const uint32_t before = block_scan(static_cast<uint32_t>(c) << 20 | light << 10 | (n - light),
                                     &total, sm.warp_sum);
  const int row = static_cast<int>(before >> 20);
  if (tid < kMaxExperts) sm.start[tid] = row;
  const int n_light = total >> 10 & 1023, n_heavy = total & 1023;
  int at_light = static_cast<int>(before >> 10 & 1023);
  int at_heavy = static_cast<int>(before & 1023) + n_light;
  for (int i = 0; i < n; ++i) {
    const int rows = i + 1 < n ? most : rest;
    const int at = (i + 1 < n ? full_light : last_light) ? at_light++ : at_heavy++;
    out->segment[which][at] = Segment{tid, row + i * most, rows, 0};
    sm.tiles[at] = static_cast<uint8_t>((rows + 7) / 8);
  }
  __syncthreads();
  cut_runs(cut, n_light + n_heavy, n_light, out->run[which], sm);
  for (int i = tid; i < T * k; i += kRouteThreads) {
    const int t = i / k, e = sm.id[i];
    const int r = sm.start[e] + __popcll(sm.mask[e] & ((1ull << t) - 1ull));
    if (which) out->token_row[i] = r; else out->row_token[r] = t;
  }
}

// The routes of at most 8 tokens, in the shared memory of every block of gate_up.
constexpr int kFewTokens = 8, kFewRows = kFewTokens * 32;
constexpr int kRankExperts = 128;    // most whose keys are ranked side by side
struct FewRoutes {
  uint32_t key[kFewTokens * kRankExperts];
  uint16_t slot[kFewRows];         // [T, k] experts
  Segment segment[kFewRows];       // an expert and its rows
  float gate[kFewRows];            // [T, k]
  uint16_t token_row[kFewRows];    // [T, k]
  uint32_t mask[kMaxExperts];      // tokens of an expert
  int32_t warp_sum[2][kWarps];
  int32_t n_segments;
};

// All of a stream block's threads; leaves with the block in step.  `meanwhile` runs while the
// logits are on their way.
template <int PER, class F>
__device__ __forceinline__ void route_few(const float* __restrict__ logits, int T, int E, int k,
                                          FewRoutes& r, F&& meanwhile) {
  static_assert(kMaxExperts <= 2 * kThreads, "two experts a thread");
  constexpr bool kRank = 32 * PER <= kRankExperts;
  constexpr int kKeys = (kFewTokens * kRankExperts + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wide = (E + 3) & ~3;  // keys of a token, with places below any key at the end
  uint32_t key[kKeys];
  if constexpr (kRank) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int at = tid + i * kThreads, t = at / wide, e = at - t * wide;
      key[i] = t < T && e < E ? order_key(__ldg(logits + t * E + e)) : 0u;
    }
  }
  for (int e = tid; e < kMaxExperts; e += kThreads) r.mask[e] = 0;
  meanwhile();
  if constexpr (kRank) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (tid + i * kThreads < T * wide) r.key[tid + i * kThreads] = key[i];
    __syncthreads();
    // An expert a thread: its slot is the number of those before it, larger keys and equal ones
    // of a lower number.  No chain of maxima (with it, and x quantized only after it, a token
    // took 22.8 us instead of 20.8).
#pragma unroll 1
    for (int at = tid; at < T * wide; at += kThreads) {
      const int t = at / wide, e = at - t * wide;
      const uint32_t mine = r.key[at];
      const uint4* row = reinterpret_cast<const uint4*>(r.key + t * wide);
      int rank = e < E ? 0 : k;
#pragma unroll 4
      for (int j = 0; j < wide / 4; ++j) {
        const uint4 o = row[j];
        rank += (o.x > mine || (o.x == mine && 4 * j < e)) +
                (o.y > mine || (o.y == mine && 4 * j + 1 < e)) +
                (o.z > mine || (o.z == mine && 4 * j + 2 < e)) +
                (o.w > mine || (o.w == mine && 4 * j + 3 < e));
      }
      if (rank < k) r.slot[t * k + rank] = static_cast<uint16_t>(e);
    }
  }
  __syncthreads();
  int id = 0;
  if (warp < T) {
    float gate;
    if constexpr (kRank) {
      id = lane < k ? r.slot[warp * k + lane] : 0;
      gate = top_gate(lane < k ? key_value(r.key[warp * wide + id]) : 0.0f, k);
    } else {
      topk_token<PER>(logits + warp * E, E, k, &id, &gate);
    }
    if (lane < k) {
      r.gate[warp * k + lane] = gate;
      atomicOr(&r.mask[id], 1u << warp);
    }
  }
  __syncthreads();
  // two experts a thread: rows and experts before
  const uint32_t m0 = 2 * tid < kMaxExperts ? r.mask[2 * tid] : 0u;
  const uint32_t m1 = 2 * tid < kMaxExperts ? r.mask[2 * tid + 1] : 0u;
  const int rows = __popc(m0) + __popc(m1), experts = (m0 != 0) + (m1 != 0);
  int in = rows << 16 | experts;  // both sums in one word
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, in, d);
    if (lane >= d) in += o;
  }
  if (lane == 31) r.warp_sum[0][warp] = in;
  __syncthreads();
  int before = in - (rows << 16 | experts);
  for (int w = 0; w < warp; ++w) before += r.warp_sum[0][w];
  int row = before >> 16, at = before & 0xFFFF;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t m = i ? m1 : m0;
    if (!m) continue;
    r.segment[at++] = Segment{2 * tid + i, row, __popc(m), 0};
    row += __popc(m);
  }
  if (tid == kThreads - 1) r.n_segments = at;
  __syncthreads();
  if (warp < T && lane < k) {
    // the row of (token, expert): the expert's segment holds its tokens in order
    int l = 0, h = r.n_segments;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (r.segment[mid].expert <= id) l = mid; else h = mid;
    }
    r.token_row[warp * k + lane] = static_cast<uint16_t>(
        r.segment[l].row0 + __popc(r.mask[id] & ((1u << warp) - 1u)));
  }
  __syncthreads();
}

template <int PER, bool SUB>
__global__ void __launch_bounds__(kRouteThreads)
    moe_route_kernel(const float* __restrict__ logits, const uint16_t* __restrict__ x, int T,
                     int H, int E, int k, CutArgs gu, CutArgs dn, int counters, Ws w,
                     int32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ RouteSmem sm;
  if (blockIdx.x < 2) {
    if (blockIdx.x)
      for (int i = threadIdx.x; i < counters; i += kRouteThreads) w.count[i] = 0;
    route<PER>(logits, T, E, k, blockIdx.x ? dn : gu, blockIdx.x, w.routes, sm);
  } else {
    const int64_t t = blockIdx.x - 2;
    quantize_token<SUB>(x + t * H, H, w.xq + t * H, w.xs + t * (H / 128), status);
  }
}

// ------------------------------------------------------------------------ weight stream
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 codes as two fp16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d = a b, f16 operands.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// (x ^ flip) & keep in one instruction (the compiler does not merge the two here).
__device__ __forceinline__ uint32_t flip_keep(uint32_t x, uint32_t flip, uint32_t keep) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(d) : "r"(x), "r"(flip), "r"(keep));
  return d;
}

// acc += a chunk's weights times a segment's activations: b_codes [tile][group][half][lane] 16
// bytes, b_scales [tile][group][column] (scale, what to add); b_codes and b_scales at the chunk's
// group, tiles code_step bytes and scale_step columns apart.
template <int NT, bool SUB>
__device__ __forceinline__ void chunk_mma(float (&acc)[2][NT][4], const uint8_t* slot, int tiles,
                                          const uint8_t* b_codes, const float2* b_scales,
                                          int code_step, int scale_step, int lane) {
  const int g = lane >> 2, qd = lane & 3;
  // word i of a row: nibbles (0, 4) and (2, 6) in the lowest places, (1, 5) and (3, 7) next
  constexpr uint32_t kLo = 0x000F000Fu, kLoSign = 0x00080008u;
  uint32_t lo[2][4][4], hi[2][4][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 v = *reinterpret_cast<const uint4*>(slot + (2 * mt + half) * 512 + lane * 16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t up = w[i] >> 8;
        lo[mt][i][half] = flip_keep(w[i], kLoSign, kLo);
        hi[mt][i][half] = flip_keep(w[i], kLoSign << 4, kLo << 4);
        lo[mt][i][2 + half] = flip_keep(up, kLoSign, kLo);
        hi[mt][i][2 + half] = flip_keep(up, kLoSign << 4, kLo << 4);
      }
    }
  const float4 sw = *reinterpret_cast<const float4*>(slot + kUnitRows * 64 + g * 16);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (nt >= tiles) break;
    const uint4 b0 = *reinterpret_cast<const uint4*>(b_codes + nt * code_step + lane * 16);
    const uint4 b1 = *reinterpret_cast<const uint4*>(b_codes + nt * code_step + 512 + lane * 16);
    const float4 s = *reinterpret_cast<const float4*>(b_scales + nt * scale_step + 2 * qd);
    const uint32_t b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
    uint32_t f[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) e4m3x4_f16x4(b[i], f[i][0], f[i][1]);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float x[4], y[4];
      mma_f16_zero(x, lo[mt][0], f[0][0], f[0][1]);
      mma_f16_zero(y, hi[mt][0], f[1][0], f[1][1]);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        mma_f16(x, lo[mt][i], f[2 * i][0], f[2 * i][1]);
        mma_f16(y, hi[mt][i], f[2 * i + 1][0], f[2 * i + 1][1]);
      }
      const float s0 = mt ? sw.z : sw.x, s1 = mt ? sw.w : sw.y;
      float(&o)[4] = acc[mt][nt];
      o[0] = fmaf(fmaf(fmaf(y[0], 0.0625f, x[0]), s.x, s.y), s0, o[0]);
      o[1] = fmaf(fmaf(fmaf(y[1], 0.0625f, x[1]), s.z, s.w), s0, o[1]);
      o[2] = fmaf(fmaf(fmaf(y[2], 0.0625f, x[2]), s.x, s.y), s1, o[2]);
      o[3] = fmaf(fmaf(fmaf(y[3], 0.0625f, x[3]), s.z, s.w), s1, o[3]);
    }
  }
}

// The operands stand for u 2^-24; the subnormal bank's scales make up for 2^9 of it.
template <bool SUB>
__device__ __forceinline__ float bank_unit(float v) { return v * (SUB ? 0x1p15f : 0x1p24f); }

struct StreamArgs {
  const uint8_t* w;  // gate_up [E, 2I, H / 2]; down [E, H, I / 2]
  const float* sw;   // gate_up [E, H / 128, 2I]; down [E, I / 128, H]
  int N, K;          // 2I, H or H, I
  int tiles;         // column tiles that the shared memory has room for, of one or more segments
  int max_split;
  Ws ws;
  // few tokens only
  const float* logits;  // [T, E]
  const uint16_t* x;    // [T, H]
  int T, E, k, out_f32;
  void* out;
  int32_t* status;
};

// Quantizes 128 finished features of a segment's rows; one warp, a batch of rows at a time so
// that their loads overlap (row by row this cost a microsecond each).
template <bool SUB>
__device__ __forceinline__ void quantize_hidden(const Ws& ws, int I, int row0, int rows, int hg,
                                                int lane) {
  constexpr int kBatch = 8;
  for (int r0 = 0; r0 < rows; r0 += kBatch) {
    float4 v[kBatch];
    float amax[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      v[i] = r0 + i < rows ? __ldcg(reinterpret_cast<const float4*>(
                                        ws.h + static_cast<int64_t>(row0 + r0 + i) * I + hg * 128) +
                                    lane)
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      amax[i] = fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], d));
    uint32_t q[kBatch];
    float sum[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (r0 + i >= rows) break;
      amax[i] = scale_from_amax(amax[i]);
      q[i] = cvt_e4m3x4(__fdiv_rn(v[i].x, amax[i]), __fdiv_rn(v[i].y, amax[i]),
                        __fdiv_rn(v[i].z, amax[i]), __fdiv_rn(v[i].w, amax[i]));
      sum[i] = e4m3x4_sum(q[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (r0 + i >= rows) break;
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (r0 + i >= rows) break;
      // lanes 2 i and 2 i + 1 hold the two halves of 8 values
      const uint32_t other = __shfl_xor_sync(0xffffffffu, q[i], 1);
      const uint2 o =
          nibble_order<SUB>(lane & 1 ? make_uint2(other, q[i]) : make_uint2(q[i], other));
      const int64_t r = row0 + r0 + i;
      *reinterpret_cast<uint32_t*>(ws.hq + r * I + hg * 128 + lane * 4) = lane & 1 ? o.y : o.x;
      if (lane == 0) 
        ws.hs[r * (I / 128) + hg] =
            make_float2(amax[i], amax[i] * (sum[i] * (-8.0f * 0x1p-24f)));
    }
  }
}

// Few tokens: a block's columns, quantized straight into the order the MMA reads; gate_up from x
// (a column a token, whatever its experts; half a warp a 128 group), down from the hidden rows of
// its segments (a warp a group).
template <bool SUB, bool GATE_UP>
__device__ __forceinline__ void quantize_rows(const StreamArgs& p, int cols, const int* row_of,
                                              int groups, uint8_t* b_codes, float2* b_scales) {
  constexpr int kLanes = GATE_UP ? 16 : 32, kAhead = 2;
  constexpr float kSum = -8.0f * 0x1p-24f;
  const int team = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const uint32_t mask = GATE_UP ? 0xFFFFu << (threadIdx.x & 16) : 0xFFFFFFFFu;
  const int tasks = cols * groups;
  for (int task = team; task < tasks; task += kThreads / kLanes * kAhead) {
    int col[kAhead], grp[kAhead];
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = task + u * (kThreads / kLanes);
      col[u] = at / groups;
      grp[u] = at - col[u] * groups;
      const int64_t r = at >= tasks ? -1 : GATE_UP ? col[u] : row_of[col[u]];
      if (r < 0) col[u] = -1;
      v[u] = make_uint4(0, 0, 0, 0);
      if (r < 0) continue;
      if (GATE_UP)
        v[u] = __ldg(reinterpret_cast<const uint4*>(p.x + r * p.K + grp[u] * 128) + lane);
      else
        v[u] = __ldcg(reinterpret_cast<const uint4*>(p.ws.h + r * p.K + grp[u] * 128) + lane);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (col[u] < 0) continue;
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint8_t* to = b_codes + ((col[u] >> 3) * groups + grp[u]) * 1024 + (col[u] & 7) * 64;
      float s, sum;
      if constexpr (GATE_UP) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max((w[i] >> 16) & 0x7FFFu, w[i] & 0x7FFFu));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(mask, m, d));
        if (m >= 0x7F80u) set_device_error(p.status, FGE_ERR_NONFINITE);
        s = scale_from_amax(__uint_as_float(m << 16));
        const uint2 q = cast8(v[u], s, __frcp_rn(s), quot_fast_ok(s));
        sum = e4m3x4_sum(q.x) + e4m3x4_sum(q.y);
        // lane i: the 8 codes of half i & 1 of piece i / 2
        *reinterpret_cast<uint2*>(to + ((lane >> 1) & 1) * 512 + (lane >> 2) * 16 +
                                  (lane & 1) * 8) = nibble_order<SUB>(q);
      } else {
        const float f[4] = {__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]),
                            __uint_as_float(w[3])};
        float amax = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(mask, amax, d));
        s = scale_from_amax(amax);
        const uint32_t q = cvt_e4m3x4(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s), __fdiv_rn(f[2], s),
                                      __fdiv_rn(f[3], s));
        sum = e4m3x4_sum(q);
        // lanes 2 i and 2 i + 1 hold the two halves of 8 values
        const uint32_t other = __shfl_xor_sync(mask, q, 1);
        const uint2 o =
            nibble_order<SUB>(lane & 1 ? make_uint2(other, q) : make_uint2(q, other));
        *reinterpret_cast<uint32_t*>(to + ((lane >> 2) & 1) * 512 + (lane >> 3) * 16 +
                                     (lane & 3) * 4) = lane & 1 ? o.y : o.x;
      }
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(mask, sum, d);
      if (lane == 0)
        b_scales[((col[u] >> 3) * groups + grp[u]) * 8 + (col[u] & 7)] =
            make_float2(s, s * (sum * kSum));
    }
  }
}

// PER: with few tokens, the logits a lane (32 PER experts at most); 0: routes by a kernel before.
template <int NT, bool SUB, bool GATE_UP, int PER>
__global__ void __launch_bounds__(kThreads, 1) moe_stream_kernel(const StreamArgs p) {
  constexpr bool kFew = PER > 0;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  const int groups = p.K / 128;
  uint8_t* ring = smem + warp * (kDepth * kSlotBytes);
  const uint32_t ring_u = smem_u32(ring);
  uint8_t* b_codes = smem + kRingBytes;
  float2* b_scales = reinterpret_cast<float2*>(b_codes + p.tiles * groups * 1024);
  float4* red = reinterpret_cast<float4*>(b_scales + p.tiles * groups * 8) + 3 * kTiles;
  const int per_segment = p.N / kUnitRows;
  const Routes& rt = *p.ws.routes;
  FewRoutes& few = *reinterpret_cast<FewRoutes*>(red + (p.max_split > 1 ? kWarps * NT * 64 : 0));
  constexpr bool kOwnRoutes = kFew && GATE_UP;
  const Segment* segments = kOwnRoutes ? few.segment : rt.segment[GATE_UP ? 0 : 1];
  auto segment_at = [&](int s) { return kOwnRoutes ? segments[s] : load_segment(segments + s); };
  int lo, hi, n_segments = 0;
  if constexpr (kFew) {
    // every block of gate_up finds the routes for itself, and the first hands them on
    if constexpr (GATE_UP) {
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      route_few<PER>(p.logits, p.T, p.E, p.k, few, [&] {
        quantize_rows<SUB, true>(p, p.T, nullptr, groups, b_codes, b_scales);
      });
      n_segments = few.n_segments;
      if (blockIdx.x == 0) {
        Routes& to = *p.ws.routes;
        for (int i = threadIdx.x; i < p.K / kUnitRows; i += kThreads) p.ws.count[i] = 0;
        for (int i = threadIdx.x; i < n_segments; i += kThreads) to.segment[1][i] = few.segment[i];
        for (int i = threadIdx.x; i < p.T * p.k; i += kThreads) {
          to.token_row[i] = few.token_row[i];
          to.gate[i] = few.gate[i];
        }
        if (threadIdx.x == 0) to.run[1][0] = make_int2(n_segments, 0);
      }
    } else {
      // its blocks find room when gate_up's leave, too late for anything ahead of the wait
      asm volatile("griddepcontrol.wait;" ::: "memory");
      n_segments = __ldcg(&rt.run[1][0]).x;
    }
    const int total = n_segments * per_segment;
    lo = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
    hi = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  } else {
    // The routes are the work of the kernel before the one before (down) or of the one before
    // (gate_up), which lets its successor start only once it has waited itself: down reads
    // them, and its first weights, while gate_up still runs.
    if (GATE_UP) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    const int2 run = __ldcg(&rt.run[GATE_UP ? 0 : 1][blockIdx.x]);
    lo = run.x;
    hi = run.y;
  }
  // warps that share a unit: what gives the busiest warp the fewest groups
  int split = 1;
  {
    const int n = hi - lo;
    int best = (n + kWarps - 1) / kWarps * groups;
    for (int s = 2; s <= p.max_split && s <= groups; ++s) {
      if (kWarps % s) continue;
      const int teams = kWarps / s;
      const int cost = (n + teams - 1) / teams * ((groups + s - 1) / s);
      if (cost < best) {
        best = cost;
        split = s;
      }
    }
  }
  const int ks = warp % split, team = warp / split, teams = kWarps / split;
  const int64_t row_bytes = p.K / 2;

  // The warp's steps, (unit, group): units team, team + teams, ... of the run, groups ks,
  // ks + split, ...; copies run ahead.
  int in_seg = lo / per_segment, in_unit = lo + team, in_group = ks, slot_in = 0;
  const uint8_t* in_w = nullptr;  // row g of the unit's first 8, at this lane's 32 weights
  const float* in_s = nullptr;    // the scale this lane copies
  // the unit's rows in eights: gate_up 8 gate rows, 64 on in the interleaved bank their up
  // rows, and the same for the next 8 features; down 32 rows in turn
  constexpr int kBeside = GATE_UP ? 64 : 8, kNext = GATE_UP ? 8 : 16;
  Segment seg = lo < hi ? segment_at(in_seg) : Segment{};
  int64_t e = seg.expert;
  auto enter_unit = [&]() {
    if (in_unit >= hi) return;
    const int s = in_unit / per_segment, f = in_unit - s * per_segment;
    if (s != in_seg) e = segment_at(s).expert;
    in_seg = s;
    const int64_t row = (GATE_UP ? (f >> 2) * 128 + (f & 3) * 16 : f * 32) + g;
    in_w = p.w + (e * p.N + row) * row_bytes + ks * 64 + qd * 16;
    in_s = p.sw + (e * groups + ks) * p.N + row + (qd >> 1) * kNext + (qd & 1) * kBeside;
  };
  enter_unit();
  const int64_t beside = kBeside * row_bytes, next = kNext * row_bytes;
  const int64_t s_step = static_cast<int64_t>(split) * p.N;
  auto issue = [&]() {
    if (in_unit < hi) {
      const uint32_t to = ring_u + slot_in * kSlotBytes + lane * 16;
      copy16(to, in_w);
      copy16(to + 512, in_w + beside);
      copy16(to + 1024, in_w + next);
      copy16(to + 1536, in_w + next + beside);
      copy4(ring_u + slot_in * kSlotBytes + kUnitRows * 64 + lane * 4, in_s);
      slot_in = slot_in + 1 == kDepth ? 0 : slot_in + 1;
      in_group += split;
      in_w += split * 64;
      in_s += s_step;
      if (in_group >= groups) {
        in_group = ks;
        in_unit += teams;
        enter_unit();
      }
    }
    copy_commit();
  };
  // The activations of as many segments from unit `begin` on as there is room for: a warp a row,
  // 16 bytes of a group at a time.  Returns the unit after them.
  int4* part = reinterpret_cast<int4*>(b_scales + p.tiles * groups * 8);  // row0, rows, first tile
  int* row_of = reinterpret_cast<int*>(part + kTiles);
  auto load_activations = [&](int begin) {
    int s = begin / per_segment, n = 0, used = 0, end = begin;
    do {
      if (begin != lo || n) seg = segment_at(s);
      const int t = (seg.rows + 7) / 8;
      if (n && used + t > p.tiles) break;
      if (threadIdx.x == 0) part[n] = make_int4(seg.row0, seg.rows, used, 0);
      const int i = threadIdx.x;
      if (i < t * 8)
        row_of[used * 8 + i] = i >= seg.rows ? -1
                               : !GATE_UP    ? seg.row0 + i
                                             : __ldcg(&rt.row_token[seg.row0 + i]);
      used += t;
      ++n;
      end = min(hi, ++s * per_segment);
    } while (end < hi);
    __syncthreads();
    if constexpr (kFew && !GATE_UP) {
      quantize_rows<SUB, false>(p, used * 8, row_of, groups, b_codes, b_scales);
    } else {
      for (int col = warp; col < used * 8; col += kWarps) {
        const int64_t r = row_of[col];
        if (r < 0) continue;
        const uint8_t* codes = (GATE_UP ? p.ws.xq : p.ws.hq) + r * p.K;
        const float2* scales = (GATE_UP ? p.ws.xs : p.ws.hs) + r * groups;
        const uint32_t to = smem_u32(b_codes + (col >> 3) * groups * 1024 + (lane & 1) * 512 +
                                     ((col & 7) * 4 + ((lane & 7) >> 1)) * 16);
        const uint32_t to_s = smem_u32(b_scales + (col >> 3) * groups * 8 + (col & 7));
#pragma unroll 4
        for (int i = lane; i < groups * 8; i += 32) copy16(to + (i >> 3) * 1024, codes + i * 16);
        for (int i = lane; i < groups; i += 32) copy8(to_s + i * 64, scales + i);
      }
      copy_commit();
    }
    return end;
  };
  int end = lo;
  // gate_up: the activations first, which would else wait behind the ring's copies; down: the
  // weights first, while gate_up still runs
  if (GATE_UP && !kFew && lo < hi) end = load_activations(lo);
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) issue();
  if (!GATE_UP && !kFew) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  if (!GATE_UP && lo < hi) end = load_activations(lo);
  if (kOwnRoutes) end = hi;  // one tile of columns serves all segments

  int slot = 0, unit = lo + team;
  for (int begin = lo; begin < hi;) {
    if (begin != lo) {
      __syncthreads();  // the last activations are free
      end = load_activations(begin);
      if (!kFew) copy_wait<0>();
    } else if (!kFew) {
      copy_wait<GATE_UP ? kDepth - 1 : 0>();
    }
    __syncthreads();
    const int first = begin / per_segment;
    for (; unit < end; unit += teams) {
      const int s = unit / per_segment;
      int4 at;
      uint32_t members = 0;  // the columns that are rows of this segment
      if constexpr (kOwnRoutes) {
        const Segment of = few.segment[s];
        at = make_int4(of.row0, 8, 0, 0);
        members = few.mask[of.expert];
      } else {
        at = part[s - first];
      }
      const int row0 = at.x, m = at.y, tiles = (m + 7) / 8;
      float acc[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.0f;
      for (int c = ks; c < groups; c += split) {
        issue();
        copy_wait<kDepth - 1>();
        __syncwarp();
        const int b_group = at.z * groups + c;
        chunk_mma<NT, SUB>(acc, ring + slot * kSlotBytes, tiles, b_codes + b_group * 1024,
                           b_scales + b_group * 8, groups * 1024, groups * 8, lane);
        __syncwarp();
        slot = slot + 1 == kDepth ? 0 : slot + 1;
      }
      if (split > 1) {
        float4* mine = red + warp * (2 * NT * 32) + lane;
        if (ks) {
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) {
            const float(&o)[4] = acc[i & 1][i >> 1];
            if ((i >> 1) < tiles) mine[i * 32] = make_float4(o[0], o[1], o[2], o[3]);
          }
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * split) : "memory");
        if (!ks) {
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i)
            if ((i >> 1) < tiles)
              for (int w = 1; w < split; ++w) {
                const float4 v = mine[w * (2 * NT * 32) + i * 32];
                float(&o)[4] = acc[i & 1][i >> 1];
                o[0] += v.x;
                o[1] += v.y;
                o[2] += v.z;
                o[3] += v.w;
              }
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * split) : "memory");
        if (ks) continue;
      }
      const int f = unit - s * per_segment;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt >= tiles) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          int r = 8 * nt + 2 * qd + i;
          if (kOwnRoutes ? !(members >> r & 1u) : r >= m) continue;
          if (kOwnRoutes) r = __popc(members & ((1u << r) - 1u));
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const float v0 = bank_unit<SUB>(acc[mt][nt][i]);
            const float v1 = bank_unit<SUB>(acc[mt][nt][2 + i]);
            if constexpr (GATE_UP) {
              p.ws.h[static_cast<int64_t>(row0 + r) * (p.N / 2) + f * 16 + mt * 8 + g] =
                  __fdiv_rn(v0, 1.0f + expf(-v0)) * v1;
            } else {
              float* y = p.ws.y + static_cast<int64_t>(row0 + r) * p.N + f * 32 + mt * 16 + g;
              y[0] = v0;
              y[8] = v1;
            }
          }
        }
      }
    }
    begin = end;
  }
  if constexpr (GATE_UP && !kFew) {
    // Whoever brings the last of 128 features quantizes them, a warp at a time.  Once a block:
    // after every unit, the fence held up the warps that share it by two microseconds.
    if (lo >= hi) return;
    __threadfence();
    __syncthreads();
    constexpr int kGroupUnits = 8;
    for (int i = lo / kGroupUnits + warp; i * kGroupUnits < hi; i += kWarps) {
      const int mine = min(hi, (i + 1) * kGroupUnits) - max(lo, i * kGroupUnits);
      int last = 0;
      if (lane == 0) last = atomicAdd(p.ws.count + i, mine) + mine == kGroupUnits;
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      const int s = i * kGroupUnits / per_segment;
      const Segment of = load_segment(segments + s);
      quantize_hidden<SUB>(p.ws, p.N / 2, of.row0, of.rows, i - s * (p.N / 256), lane);
    }
  }
  if constexpr (!GATE_UP && kFew) {
    // The last of the experts' units of 32 features sums them, in slot order; a lane a feature.
    if (lo >= hi) return;
    __threadfence();
    __syncthreads();
    for (int i = lo + warp; i < hi; i += kWarps) {
      const int f = i % per_segment;
      int last = 0;
      if (lane == 0) last = atomicAdd(p.ws.count + f, 1) + 1 == n_segments;
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      for (int t = 0; t < p.T; ++t) {
        float sum = 0.0f;
#pragma unroll 8
        for (int j = 0; j < p.k; ++j)
          sum = fmaf(__ldcg(&rt.gate[t * p.k + j]),
                     __ldcg(p.ws.y + static_cast<int64_t>(__ldcg(&rt.token_row[t * p.k + j])) * p.N +
                            f * 32 + lane),
                     sum);
        const int64_t o = static_cast<int64_t>(t) * p.N + f * 32 + lane;
        if (p.out_f32)
          static_cast<float*>(p.out)[o] = sum;
        else
          static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(sum);
      }
    }
  }
}

// out[t] = sum over the token's slots of gate * y, in slot order; a thread 4 features.
__global__ void __launch_bounds__(128)
    moe_sum_kernel(const Ws ws, int T, int H, int k, int out_f32, void* __restrict__ out) {
  const int t = blockIdx.y, at = (blockIdx.x * 128 + threadIdx.x) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at >= H) return;
  const Routes& rt = *ws.routes;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int j = 0; j < k; ++j) {
    const float gate = __ldcg(&rt.gate[t * k + j]);
    const int64_t r = __ldcg(&rt.token_row[t * k + j]);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(ws.y + r * H + at));
    acc.x = fmaf(gate, v.x, acc.x);
    acc.y = fmaf(gate, v.y, acc.y);
    acc.z = fmaf(gate, v.z, acc.z);
    acc.w = fmaf(gate, v.w, acc.w);
  }
  const int64_t o = static_cast<int64_t>(t) * H + at;
  if (out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

// The shared memory of a block: rings, column tiles (8 rows of an expert each), their segments
// and rows, and the sums of warps that share a unit.
template <int NT>
struct StreamShape {
  // with few tokens there are few units: their K is shared by up to all warps; from 17 tokens
  // on the units outnumber the warps, and the room is worth more as another tile
  static constexpr int kSplit = NT == 1 ? kWarps : NT == 2 ? 4 : 1;
  static constexpr int kRed = NT <= 2 ? kWarps * NT * 1024 : 0;
  static constexpr int kFixed = kRingBytes + kRed + kTiles * (16 + 32) +
                                (NT == 1 ? static_cast<int>(sizeof(FewRoutes)) : 0);
  static int tile_bytes(int K) { return K / 128 * (1024 + 64); }
  static int tiles(int K) { return std::min(kTiles, (kSmemMost - kFixed) / tile_bytes(K)); }
  static int segment_tiles(int K) { return std::min(NT, tiles(K)); }
  static int smem(int K) { return kFixed + tiles(K) * tile_bytes(K); }
};

// The cut of N bank rows a segment, K values each, for at most `most` segments.
template <int NT>
CutArgs cut_args(int64_t most, int N, int K) {
  using Shape = StreamShape<NT>;
  const int tiles = Shape::tiles(K), seg = Shape::segment_tiles(K);
  return CutArgs{static_cast<int>(std::min<int64_t>({most * (N / kUnitRows), num_sms(), kMaxBlocks})),
                 N / kUnitRows, seg, tiles / 2};
}

template <int NT, bool SUB, bool GATE_UP, int PER>
cudaError_t launch_stream(const MoeDecodeArgs& a, const CutArgs& cut, const Ws& ws,
                          cudaStream_t s) {
  using Shape = StreamShape<NT>;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const auto kern = moe_stream_kernel<NT, SUB, GATE_UP, PER>;
  if (!device_kernel_ready(dev, reinterpret_cast<const void*>(kern), kSmemMost, 0))
    return cudaErrorInvalidConfiguration;
  const int H = static_cast<int>(a.H), I = static_cast<int>(a.I), K = GATE_UP ? H : I;
  const StreamArgs args{GATE_UP ? a.w_gu : a.w_dn, GATE_UP ? a.s_gu : a.s_dn, GATE_UP ? 2 * I : H, K,
                        Shape::tiles(K), Shape::kSplit, ws, a.logits, a.x, static_cast<int>(a.T),
                        a.E, a.k, a.out_f32, a.out, a.status};
  const dim3 grid(static_cast<unsigned>(cut.blocks)), block(kThreads);
  const size_t smem = static_cast<size_t>(Shape::smem(K));
  if (PER > 0 && GATE_UP) {  // the first kernel of the call
    kern<<<grid, block, smem, s>>>(args);
    return cudaGetLastError();
  }
  return launch_chained(kern, grid, block, smem, s, args);
}

// Two launches.
template <bool SUB, int PER>
cudaError_t run_few(const MoeDecodeArgs& a, const Ws& w, cudaStream_t s) {
  const int H = static_cast<int>(a.H), I = static_cast<int>(a.I);
  const int64_t most = std::min<int64_t>(a.T * a.k, a.E);
  const cudaError_t e = launch_stream<1, SUB, true, PER>(a, cut_args<1>(most, 2 * I, H), w, s);
  return e != cudaSuccess ? e : launch_stream<1, SUB, false, PER>(a, cut_args<1>(most, H, I), w, s);
}

template <int NT, bool SUB>
cudaError_t run(const MoeDecodeArgs& a, const Ws& w, cudaStream_t s) {
  const int T = static_cast<int>(a.T), H = static_cast<int>(a.H), I = static_cast<int>(a.I);
  const int per = (a.E + 31) / 32;
  const auto route = per <= 2   ? moe_route_kernel<2, SUB>
                     : per <= 4 ? moe_route_kernel<4, SUB>
                     : per <= 8 ? moe_route_kernel<8, SUB>
                                : moe_route_kernel<16, SUB>;
  const int64_t most = most_segments(T, a.E, a.k);
  const CutArgs gu = cut_args<NT>(most, 2 * I, H), dn = cut_args<NT>(most, H, I);
  route<<<static_cast<unsigned>(T + 2), kRouteThreads, 0, s>>>(
      a.logits, a.x, T, H, a.E, a.k, gu, dn, static_cast<int>(most * (I / 128)), w, a.status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_stream<NT, SUB, true, 0>(a, gu, w, s);
  if (e != cudaSuccess) return e;
  e = launch_stream<NT, SUB, false, 0>(a, dn, w, s);
  if (e != cudaSuccess) return e;
  return launch_chained(moe_sum_kernel, dim3(static_cast<unsigned>((H + 511) / 512), T), dim3(128),
                        0, s, w, T, H, a.k, a.out_f32, a.out);
}

template <bool SUB>
cudaError_t run_tokens(const MoeDecodeArgs& a, const Ws& w, cudaStream_t s) {
  // Two launches save the routing kernel but have every block quantize its own rows, which pays
  // while those are few and short: one token with H = 2048, I = 768 takes 20.8 us instead of
  // 26.7, three 29.2 instead of 32.3, six 40.7 instead of 37.4; with H = 4096, I = 1536 one takes
  // 43.4 instead of 42.2.
  if (a.T <= kFewTokens && a.T * a.H * a.I <= 5 << 20)
    return a.E <= 128 ? run_few<SUB, 4>(a, w, s) : run_few<SUB, 16>(a, w, s);
  // Column tiles of 8 tokens to a segment: with two, warps can share a unit's K; with four, an
  // expert of more than 16 tokens is read once, where shared memory has room for its rows (E = 64,
  // H = 2048: 32 tokens 60.0 us with two tiles, 69.9 with four; E = 128, H = 4096: 17 tokens
  // 109 and 111 us, 32 tokens 143 and 136 us, 64 tokens 205 and 181 us).
  if (a.T <= 24 || a.T * a.H <= 65536) return run<2, SUB>(a, w, s);
  return run<4, SUB>(a, w, s);
}

}  // namespace

size_t moe_decode_scratch_bytes(int64_t T, int64_t H, int64_t I, int E, int k) {
  // what the call refuses needs nothing
  if (T < 0 || T > kMoeDecodeTokens || H < 0 || H > kMoeDecodeWidth || I < 0 ||
      I > kMoeDecodeWidth || E < 0 || E > kMaxExperts || k < 0 || k > E || k > 32)
    return 0;
  return carve(nullptr, T, H, I, E, k).bytes;
}

cudaError_t launch_moe_decode(const MoeDecodeArgs& a, void* scratch, cudaStream_t s) {
  const Ws w = carve(scratch, a.T, a.H, a.I, a.E, a.k);
  return a.bank_format == kBankSubnormal ? run_tokens<true>(a, w, s) : run_tokens<false>(a, w, s);
}

}  // namespace fge
