// The shared prefix's part of single-token attention for a batch: many query rows (those of the
// whole batch that use one key/value head) over the same tokens, so unlike a sequence's own part
// it is a matrix product, and bound by the tensor cores and the exponentials.  A block takes two
// tiles of 128 rows and a run of 128-token tiles; the tiles' maxima, sums and outputs before the
// division go to the join kernel.
//   warps 0-7, 8-15  softmax of row tile 0 and 1: a thread has one row (its TMEM lane) and half
//                    of a tile's tokens
//   warps 16-19      load keys a tile ahead and widen the codes to fp16, once for 256 rows
//   warps 20-23      the same for values, transposed to [dim][token]
//   warp 24          issues the MMAs (tcgen05, kind::f16): S = Q K^T and O += P V, P from TMEM
// The two row tiles take turns: while one's scores go through the softmax the tensor core works
// for the other.  The probabilities overwrite the scores they come from.
//   Scores are q * k in fp16 operands and float32, both exact (the query after a power of two that
// brings the row's largest value to [128, 256)).  A weighted probability p vs is fp16 (2^-11):
// the row's reference M is max(x + log2 vs) of its first tile, x the score in base 2, so that
// 2^(x - M) vs begins at 1 at most; l sums 2^(x - M).  The next tiles keep M and only bound what
// they got, by their sum and the largest value scale; a tile that may pass 2^15 is done over with
// a new M.  Tokens of value zero count in l alone: a zero row's scale would set M for the others.
// vs is in units of the power of two of the run's first tile's largest, so that l keeps its range
// whatever the size of the values; one below 2^-90 of that is lost.
//   Bound by the exchange between tensor core and softmax: a token tile takes a block 3 us, of
// which the 32 MMAs are 1.1 (64 cycles each).  Measured for a batch of 96 (384 rows a head, 4
// heads) behind 16384 tokens, own tokens and join included: one softmax warpgroup a row tile and
// two looks at the scores 66 us; two warpgroups and one look, whole rows of the query loaded by
// neighbouring lanes (a row a lane, 16 bytes a time, read the query's sectors several times)
// 60 us; now 54 us, of which this kernel is about 30.
#include "attention.cuh"

namespace fge {

namespace {

constexpr int kRows = kPrefixTcRows;
constexpr int kTileWarps = 8;  // of a row tile's softmax
constexpr int kKeyWarp = 2 * kTileWarps, kValueWarp = kKeyWarp + 4, kMmaWarp = kValueWarp + 4;
constexpr int kThreads = (kMmaWarp + 1) * 32;  // whole warpgroups
constexpr int kHalfTile = kTile / 2;  // tokens of a softmax thread
constexpr int kConvertWarps = 4, kConvert = kConvertWarps * 32;

template <int D>
struct Layout {
  static constexpr int kHalf = kTile * D * 2;  // an fp16 tile
  static constexpr int kKey = 0, kValue = 2 * kHalf, kQuery = 4 * kHalf;
  // per tile: key scales, log2 of the value scales, value scales, the tokens that are there
  static constexpr int kScale = 6 * kHalf, kScaleBytes = 3 * kTile * 4 + 64;
  static constexpr int kTop = kScale + 2 * kScaleBytes;  // [row tile][half][row] float
  static constexpr int kBars = kTop + 4 * kRows * 4;
  static constexpr int kSmem = kBars + 256 + 1024;  // slack to align the base
};

// Barriers, two of each but the last: one a slot of two tiles, or one a row tile.
enum Bar {
  kKeyFull = 0, kKeyEmpty = 2, kValueFull = 4, kValueEmpty = 6, kScaleFull = 8, kScaleEmpty = 10,
  kScoreFull = 12, kProbFull = 14, kOutDone = 16, kQueryFull = 18, kDrain, kBarCount
};

// Instruction descriptor, kind::f16: D f32, A and B fp16, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// Both are for a whole warp to run, one lane of which (issue) does: no branch around them, so
// that their operands can stay in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}
// A from TMEM: its rows are the lanes, two fp16 values of K a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(issue)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// Values loaded from TMEM may be used only after the wait: this makes every use follow it.
__device__ __forceinline__ void wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// Pairs of floats, two lanes of one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pair_bits(uint32_t a, uint32_t b) {
  return pair(__uint_as_float(a), __uint_as_float(b));
}

// Byte offset of 16-byte chunk c (0..) of row r in an fp16 K-major tile of `rows` rows: 128-byte
// swizzle atoms of 64 values, one after the other.
__device__ __forceinline__ int half_tile(int rows, int r, int c) {
  return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

struct Args {
  AttentionArgs a;
  int groups;
  uint32_t splits, last;  // runs of the token tiles: of two groups together, of an odd last one
  float* partials;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const Args w) {
  extern __shared__ uint8_t raw_smem[];
  using L = Layout<D>;
  uint8_t* sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(sm), bars = base + L::kBars;
  int* s_int = reinterpret_cast<int*>(sm + L::kBars + kBarCount * 8);
  volatile int* s_abort = s_int;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_int + 1);
  float* s_unit = reinterpret_cast<float*>(s_int + 2);  // of the value scales
  float* s_most = reinterpret_cast<float*>(s_int + 4);  // largest scale of each value warp
  const AttentionArgs& a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return bars + 8 * i; };

  const int group = a.n_heads / a.c.n_kv;
  const int total_rows = static_cast<int>(a.B * group);  // partial results of 2^31 fit nowhere
  const uint32_t paired = (w.groups >> 1) * w.splits;  // a head's blocks with two row tiles
  const uint32_t per_head = paired + (w.groups & 1) * w.last;
  const int kv = blockIdx.x / per_head;
  const uint32_t in = blockIdx.x - kv * per_head;
  const int row_tiles = in < paired ? 2 : 1;  // of this block
  const uint32_t runs = in < paired ? w.splits : w.last;
  const int pr = in < paired ? in / w.splits : w.groups >> 1;
  const int split = in - pr * w.splits;
  // this block's run of token tiles
  const int len = threadIdx.x == 0 && blockIdx.x == 0
                      ? clamp_length(*a.prefix_length, a.prefix_width, a.c, a.status)
                      : quiet_length(*a.prefix_length, a.prefix_width, a.c.page_shift);
  const int all = tile_count(len);
  // at most 2^24 tiles, 64 runs
  const int t0 = static_cast<int>(static_cast<uint32_t>(all * split) / runs);
  const int n = static_cast<int>(static_cast<uint32_t>(all * (split + 1)) / runs) - t0;
  auto partial_of = [&](int tile) {
    return w.partials + (static_cast<int64_t>(kv * w.groups + 2 * pr + tile) *
                             max(w.splits, w.last) + split) * partial_floats(kRows, D);
  };
  // the cache row of a token of the prefix, or -1: not there, or its page number is bad
  auto row_of = [&](int tok) -> int64_t {
    if (tok >= len) return -1;
    const int page = __ldg(a.prefix_pages + (tok >> a.c.page_shift));
    if (page < 0 || page >= a.c.n_pages) return -1;
    return ((static_cast<int64_t>(page) * a.c.n_kv + kv) << a.c.page_shift) +
           (tok & (a.c.page_size - 1));
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (n == 0) {  // empty partial results
    for (int i = threadIdx.x; i < row_tiles * kRows; i += kThreads)
      partial_of(i / kRows)[kRows + i % kRows] = 0.0f;
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKeyFull + i), kConvertWarps);
      mbar_init(bar(kKeyEmpty + i), 1);
      mbar_init(bar(kValueFull + i), kConvertWarps);
      mbar_init(bar(kValueEmpty + i), 1);
      mbar_init(bar(kScaleFull + i), 2 * kConvertWarps);
      mbar_init(bar(kScaleEmpty + i), kTileWarps * row_tiles);
      mbar_init(bar(kScoreFull + i), 1);
      mbar_init(bar(kProbFull + i), kTileWarps);
      mbar_init(bar(kOutDone + i), 1);
    }
    mbar_init(bar(kQueryFull), kTileWarps * row_tiles);
    mbar_init(bar(kDrain), 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // scores (and probabilities) of row tile i at column 128 i, its outputs at 256 + 128 i
  bool dead = false;
  auto wait = [&](int b, int phase) {
    if (!dead) dead = !mbar_wait(bar(b), phase & 1, s_abort, a.status);
    return !dead;
  };

  if (warp >= kMmaWarp) {

    if (warp == kMmaWarp) {
    // the whole warp walks the loop, so that descriptors stay in uniform registers; one lane
    // issues
    constexpr uint32_t kScoreDesc = idesc_f16(kRows, kTile), kOutDesc = idesc_f16(kRows, D);
    const uint64_t query = make_sdesc_sw128(base + L::kQuery);
    const uint64_t key = make_sdesc_sw128(base + L::kKey);
    const uint64_t value = make_sdesc_sw128(base + L::kValue);
    const bool lead = lane == 0;
    auto score = [&](int tile, int slot, bool last) {
      const uint64_t q = query + tile * (L::kHalf >> 4), k = key + slot * (L::kHalf >> 4);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = ((i >> 2) * kTile * 128 + (i & 3) * 32) >> 4;
        mma_ss(tmem + 128 * tile, q + off, k + off, kScoreDesc, i > 0, lead);
      }
      if (lead) {
        mma_commit(bar(kScoreFull + tile));
        if (last) mma_commit(bar(kKeyEmpty + slot));
      }
      __syncwarp();
    };
    wait(kQueryFull, 0);
    wait(kKeyFull, 0);
    dead = __any_sync(0xffffffffu, dead);
    tc_fence_after();
    if (!dead)
      for (int tile = 0; tile < row_tiles; ++tile) score(tile, 0, tile + 1 == row_tiles);
    for (int i = 0; i < n && !dead; ++i) {
      const int st = i & 1, next = (i + 1) & 1;
      const uint64_t v = value + st * (L::kHalf >> 4);
      for (int tile = 0; tile < row_tiles; ++tile) {
        if (tile == 0) {
          wait(kValueFull + st, i >> 1);
          if (i + 1 < n) wait(kKeyFull + next, (i + 1) >> 1);
        }
        wait(kProbFull + tile, i);
        dead = __any_sync(0xffffffffu, dead);
        tc_fence_after();
        if (dead) break;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts(tmem + 256 + 128 * tile, tmem + 128 * tile + 8 * k + (k >> 2) * 32,
                 v + (((k >> 2) * D * 128 + (k & 3) * 32) >> 4), kOutDesc, i > 0 || k > 0, lead);
        if (lead) {
          mma_commit(bar(kOutDone + tile));
          if (tile + 1 == row_tiles) mma_commit(bar(kValueEmpty + st));
        }
        __syncwarp();
        if (i + 1 < n) score(tile, next, tile + 1 == row_tiles);
      }
    }
    // whatever was issued has to end, and its commits to arrive, before the memory is given
    // back
    if (lead) {
      int zero = 0;
      mma_commit(bar(kDrain));
      mbar_wait(bar(kDrain), 0, &zero, a.status);
    }
    __syncwarp();
    }
  } else if (warp >= kValueWarp) {
    // ------------------------------------------------------- values, and their scales
    // transposed: 8 tokens of 4 dims a time, a row of 64 tokens 128 bytes; lanes start at
    // different ones of their 4 dims so that 8 of them store to 8 different rows mod 8.  A
    // warp's words are whole tokens, 32 of them, of which each lane looks after one.
    constexpr int kWords = D / 4, kTasks = kTile / 8 * kWords / kConvert;
    const int tid = threadIdx.x - kValueWarp * 32;
    const int word = tid % kWords, turn = (word >> 1) & 3;
    constexpr int kPer = 32 / kTasks;  // of them a task
    const int token = 8 * ((tid / 32 * 32 + lane / kPer * kConvert) / kWords) + lane % kPer;
    uint32_t v[kTasks][8];
    float vs;
    bool here;
    auto load = [&](int t) {
      const int64_t mine = row_of(t * kTile + token);
      here = mine >= 0;
      vs = here ? __ldg(a.c.v_scales + mine) : 0.0f;
#pragma unroll
      for (int u = 0; u < kTasks; ++u) {
        const int tok = t * kTile + 8 * ((tid + u * kConvert) / kWords);
        const int64_t row = row_of(tok);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[u][j] = row >= 0 && tok + j < len
                        ? __ldg(reinterpret_cast<const uint32_t*>(a.c.v_codes + (row + j) * D) + word)
                        : 0u;
      }
    };
    load(t0);
    float down = 1.0f;  // 1 / *s_unit
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      if (i > 1) wait(kValueEmpty + st, (i >> 1) - 1);
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      // A token whose codes are all zero takes no part in the weights: its scale, which would
      // set the range of the others, is taken as zero.
      uint32_t some = 0;
#pragma unroll
      for (int u = 0; u < kTasks; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m |= (v[u][j] & 0x7F7F7F7Fu ? 1u : 0u) << j;
        m = __reduce_or_sync(0xffffffffu, m << (lane / kWords * 8));
        if (lane / kPer == u) some = m >> (lane % kPer) & 1u;
      }
      float weight = some ? vs : 0.0f;
      if (i == 0) {
        float most = fabsf(weight);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        if (lane == 0) s_most[warp - kValueWarp] = most;
        asm volatile("bar.sync 3, %0;" ::"n"(kConvert) : "memory");
        most = fmaxf(fmaxf(s_most[0], s_most[1]), fmaxf(s_most[2], s_most[3]));
        // biased exponents, both factors normal
        const uint32_t e = min(253u, __float_as_uint(most) >> 23);
        if (e) down = __uint_as_float((254u - e) << 23);
        if (tid == 0) *s_unit = e ? __uint_as_float(e << 23) : 1.0f;
      }
      weight *= down;
      float* sc = reinterpret_cast<float*>(sm + L::kScale + st * L::kScaleBytes);
      // a scale far below the others must not let the sum of 2^(x - M) overflow
      sc[kTile + token] = here ? fmaxf(log2f(fabsf(weight)), -90.0f) : -INFINITY;
      sc[2 * kTile + token] = weight;
      float most = fabsf(weight);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      if (lane == 0) sc[3 * kTile + 4 + (tid >> 5)] = most;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kScaleFull + st));
      uint8_t* to = sm + L::kValue + st * L::kHalf;
#pragma unroll
      for (int u = 0; u < kTasks; ++u) {
        const int octet = (tid + u * kConvert) / kWords;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int d0 = (2 * p + turn) & 3, d1 = (2 * p + 1 + turn) & 3;
          const uint32_t sel = d0 | (d0 + 4) << 4 | d1 << 8 | (d1 + 4) << 12;
          uint32_t x[4], y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            e4m3x4_f16x4(prmt(v[u][2 * j], v[u][2 * j + 1], sel), x[j], y[j]);
          *reinterpret_cast<uint4*>(to + half_tile(D, 4 * word + d0, octet)) =
              make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(to + half_tile(D, 4 * word + d1, octet)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kValueFull + st));
      if (i + 1 < n) load(t0 + i + 1);
    }
  } else if (warp >= kKeyWarp) {
    // --------------------------------------------------------- keys, and their scales
    constexpr int kChunks = D / 16, kTasks = kTile * kChunks / kConvert;
    const int tid = threadIdx.x - kKeyWarp * 32;
    const int c = tid % kChunks;
    uint4 k[kTasks];
    float ks;
    bool here;
    auto load = [&](int t) {
#pragma unroll
      for (int u = 0; u < kTasks; ++u) {
        const int64_t row = row_of(t * kTile + (tid + u * kConvert) / kChunks);
        k[u] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.c.k_codes + row * D) + c)
                        : make_uint4(0, 0, 0, 0);
      }
      const int64_t row = row_of(t * kTile + tid);
      here = row >= 0;
      if (!here && t * kTile + tid < len) set_device_error(a.status, FGE_ERR_BAD_INDEX);
      ks = here ? __ldg(a.c.k_scales + row) : 0.0f;
    };
    load(t0);
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      if (i > 1) {
        wait(kKeyEmpty + st, (i >> 1) - 1);
        wait(kScaleEmpty + st, (i >> 1) - 1);
      }
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      uint8_t* to = sm + L::kKey + st * L::kHalf;
#pragma unroll
      for (int u = 0; u < kTasks; ++u) {
        const int r = (tid + u * kConvert) / kChunks;
        uint4 lo, hi;
        e4m3x4_f16x4(k[u].x, lo.x, lo.y);
        e4m3x4_f16x4(k[u].y, lo.z, lo.w);
        e4m3x4_f16x4(k[u].z, hi.x, hi.y);
        e4m3x4_f16x4(k[u].w, hi.z, hi.w);
        // chunks of both parities a time: eight lanes store to eight different ones mod 8
        const int odd = c >> 2 & 1;
        *reinterpret_cast<uint4*>(to + half_tile(kTile, r, 2 * c + odd)) = odd ? hi : lo;
        *reinterpret_cast<uint4*>(to + half_tile(kTile, r, 2 * c + 1 - odd)) = odd ? lo : hi;
      }
      float* sc = reinterpret_cast<float*>(sm + L::kScale + st * L::kScaleBytes);
      sc[tid] = ks;
      const uint32_t m = __ballot_sync(0xffffffffu, here);
      if (lane == 0) reinterpret_cast<uint32_t*>(sc + 3 * kTile)[tid >> 5] = m;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kKeyFull + st));
        mbar_arrive(bar(kScaleFull + st));
      }
      if (i + 1 < n) load(t0 + i + 1);
    }
  } else {
    // ---------------------------------------------------------------------- softmax

    if (warp / kTileWarps < row_tiles) {
    const int tile = warp / kTileWarps, half = (warp >> 2) & 1, row = threadIdx.x & 127;
    const bool live = (2 * pr + tile) * kRows + row < total_rows;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t scores = tmem + 128 * tile + 64 * half + lanes;
    const uint32_t outs = tmem + 256 + 128 * tile + D / 2 * half + lanes;
    float* tops = reinterpret_cast<float*>(sm + L::kTop) + 2 * kRows * tile;
    // all of the row tile's threads, whatever became of their waits: none leaves early
    auto any_of_tile = [&](bool v) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
          : "=r"(r)
          : "r"(static_cast<uint32_t>(v)), "r"(1 + tile), "n"(kTileWarps * 32)
          : "memory");
      return r != 0;
    };
    float row_scale;
    {
      // The rows' queries, D / 8 lanes a row: the power of two that brings a row's largest value
      // to [128, 256), then fp16.
      constexpr int kLanes = D / 8, kRowsLoad = 32 / kLanes, kLoads = kRows / kTileWarps / kRowsLoad;
      const int r0 = (warp % kTileWarps) * (kRows / kTileWarps) + lane / kLanes;
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t r = static_cast<uint32_t>((2 * pr + tile) * kRows + r0 + i * kRowsLoad);
        const uint32_t b = r / static_cast<uint32_t>(group);
        x[i] = r < total_rows ? __ldg(reinterpret_cast<const uint4*>(
                                          a.q + b * a.q_stride + (kv * group + r - b * group) * D) +
                                      lane % kLanes)
                              : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t m = 0, f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max((w4[j] >> 16) & 0x7FFFu, w4[j] & 0x7FFFu));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const int up = min(253, max(1, 134 + 127 - static_cast<int>(m >> 7)));
        const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
        if (lane % kLanes == 0)
          tops[r0 + i * kRowsLoad] = __uint_as_float(static_cast<uint32_t>(254 - up) << 23) *
                                     a.scale * 1.4426950408889634f;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = pack_f16x2(bf16_lo(w4[j]) * mul, bf16_hi(w4[j]) * mul);
        *reinterpret_cast<uint4*>(sm + L::kQuery + tile * L::kHalf +
                                  half_tile(kRows, r0 + i * kRowsLoad, lane % kLanes)) =
            make_uint4(f[0], f[1], f[2], f[3]);
      }
      fence_proxy_async_smem();
      any_of_tile(false);
      row_scale = tops[row];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQueryFull));  // before tops is written again
    }
    const uint64_t rs2 = pair(row_scale, row_scale);
    float ref = -INFINITY;  // M, the same in both halves
    float l = 0.0f;         // of this half
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      wait(kScaleFull + st, i >> 1);
      wait(kScoreFull + tile, i);
      dead = __any_sync(0xffffffffu, dead);
      tc_fence_after();
      const float* scales = reinterpret_cast<const float*>(sm + L::kScale + st * L::kScaleBytes);
      const float* sc = scales + kHalfTile * half;
      const uint2 here = *reinterpret_cast<const uint2*>(scales + 3 * kTile + 2 * half);
      const bool full = (here.x & here.y) == 0xFFFFFFFFu;
      uint32_t p[kHalfTile / 2];
      float sum;
      bool again = i == 0;
      while (true) {
        if (again) {
          // ---- a new reference from the row's largest x + log2 vs
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kHalfTile / 16; ++c) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(scores + 16 * c, r);
            wait_ld16(r);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const ulonglong2 ks = *reinterpret_cast<const ulonglong2*>(sc + 16 * c + j);
              const ulonglong2 lv = *reinterpret_cast<const ulonglong2*>(sc + kTile + 16 * c + j);
              // the row's factor times the key's first: a score times a large key's scale alone
              // can pass float's range
              const float2 u = unpair(fma2(mul2(ks.x, rs2), pair_bits(r[j], r[j + 1]), lv.x));
              const float2 v = unpair(fma2(mul2(ks.y, rs2), pair_bits(r[j + 2], r[j + 3]), lv.y));
              top = fmaxf(fmaxf(top, fmaxf(u.x, u.y)), fmaxf(v.x, v.y));
            }
          }
          tops[half * kRows + row] = top;
          any_of_tile(false);
          top = fmaxf(top, tops[(half ^ 1) * kRows + row]);
          const float next = fmaxf(ref, top);
          const float factor = next == ref ? 1.0f : exp2_approx(ref - next);
          l *= factor;
          if (i > 0) {  // the MMAs of the tile before ended before the scores came
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[16];
              tmem_ld_32x32b_x16(outs + 16 * c, r);
              wait_ld16(r);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) * factor);
              tmem_st_32x32b_x16(outs + 16 * c, r);
            }
          }
          ref = next;
        }
        // ---- probabilities
        const float minus = ref == -INFINITY ? 0.0f : -ref;
        const uint64_t minus2 = pair(minus, minus);
        uint64_t sum2 = 0;
#pragma unroll
        for (int c = 0; c < kHalfTile / 16; ++c) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(scores + 16 * c, r);
          wait_ld16(r);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const ulonglong2 ks = *reinterpret_cast<const ulonglong2*>(sc + 16 * c + j);
            const ulonglong2 vs = *reinterpret_cast<const ulonglong2*>(sc + 2 * kTile + 16 * c + j);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 e = unpair(fma2(mul2(h ? ks.y : ks.x, rs2),
                                     pair_bits(r[j + 2 * h], r[j + 2 * h + 1]), minus2));
              e.x = exp2_approx(e.x);
              e.y = exp2_approx(e.y);
              if (!full) {
                // read again: in registers all the time, it made the loop spill 13 of them
                const uint32_t mask = reinterpret_cast<const volatile uint32_t*>(
                                          scales + 3 * kTile)[2 * half + (c >> 1)] >>
                                      (c & 1) * 16;
                if (!(mask >> (j + 2 * h) & 1u)) e.x = 0.0f;
                if (!(mask >> (j + 2 * h + 1) & 1u)) e.y = 0.0f;
              }
              const uint64_t e2 = pair(e.x, e.y);
              sum2 = add2(sum2, e2);
              const float2 pv = unpair(mul2(e2, h ? vs.y : vs.x));
              p[8 * c + j / 2 + h] = pack_f16x2(pv.x, pv.y);
            }
          }
        }
        // A weighted probability is at most the sum times the largest value scale: is that in
        // fp16's range, is the sum in float's, and is there a reference at all?
        const float2 s2 = unpair(sum2);
        const float4 most = *reinterpret_cast<const float4*>(scales + 3 * kTile + 4);
        sum = s2.x + s2.y;
        const bool over =
            !(sum * fmaxf(fmaxf(most.x, most.y), fmaxf(most.z, most.w)) <= 32768.0f &&
              sum <= 0x1p100f && ref != -INFINITY);
        if (again || !any_of_tile(over)) break;
        again = true;
      }
      // over the scores they come from
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = p[16 * c + j];
        tmem_st_32x32b_x16(scores + 16 * c, r);
      }
      tmem_wait_st();
      tc_fence_before();
      l += sum;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kProbFull + tile));
        mbar_arrive(bar(kScaleEmpty + st));
      }
    }
    wait(kOutDone + tile, n - 1);
    dead = __any_sync(0xffffffffu, dead);
    any_of_tile(false);  // the maxima have been read
    if (half) tops[row] = l;
    any_of_tile(false);
    if (!dead) {
      tc_fence_after();
      float* part = partial_of(tile);
      if (live && !half) {
        part[row] = ref;
        part[kRows + row] = l + tops[row];
      }
      float* o = part + 2 * kRows + row * D + half * (D / 2);
      const float unit = *s_unit;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(outs + 32 * c, r);
        wait_ld32(r);
        if (live)
#pragma unroll
          for (int j = 0; j < 32; j += 8)  // whole sectors
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             o + 32 * c + j),
                         "f"(__uint_as_float(r[j]) * unit), "f"(__uint_as_float(r[j + 1]) * unit),
                         "f"(__uint_as_float(r[j + 2]) * unit),
                         "f"(__uint_as_float(r[j + 3]) * unit),
                         "f"(__uint_as_float(r[j + 4]) * unit),
                         "f"(__uint_as_float(r[j + 5]) * unit),
                         "f"(__uint_as_float(r[j + 6]) * unit),
                         "f"(__uint_as_float(r[j + 7]) * unit)
                         : "memory");
      }
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t run(const Args& w, cudaStream_t s) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!device_kernel_ready(dev, reinterpret_cast<const void*>(prefix_kernel<D>), Layout<D>::kSmem,
                           0))
    return cudaErrorInvalidConfiguration;
  const int64_t grid = static_cast<int64_t>(w.a.c.n_kv) *
                       ((w.groups >> 1) * w.splits + (w.groups & 1) * w.last);
  prefix_kernel<D><<<static_cast<unsigned>(grid), kThreads, Layout<D>::kSmem, s>>>(w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_tc(const AttentionArgs& a, int groups, int splits, int last,
                             float* partials, cudaStream_t s) {
  const Args w{a, groups, static_cast<uint32_t>(splits), static_cast<uint32_t>(last), partials};
  return a.c.head_dim == 128 ? run<128>(w, s) : run<64>(w, s);
}

}  // namespace fge
