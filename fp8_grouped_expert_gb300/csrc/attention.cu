// Attention of single tokens over a paged e4m3 cache, optionally behind a prefix that the
// whole batch shares: out = sum_t p_t vs_t vc_t, p = softmax over the tokens t of
// scale * ks_t * (q . kc_t), with the running maximum and sum of the softmax in float32.
//
// One token per sequence reads every cached byte once and does 2 * heads / kv heads
// multiplications with it, so the kernel is built around the stream of cache pages: a
// producer warp keeps a ring of 128-token tiles in flight by TMA (one box a page piece,
// codes in the swizzled layout, scales beside them), a second one looks for tokens of value
// zero, and four warps each take 32 tokens of a tile, with their own running maximum, sum and
// output, joined at the end.
//   Scores.  mma m16n8k16 on the keys widened to fp16 (exact; an e4m3 MMA of this size takes its
// operands apart into fp16 as well, both of them and every time).  The query is an fp16 value
// too: a power of two brings the row's largest to [128, 256); the 8 significant bits of a bf16
// value fit down to 2^-24 of that, and smaller values are off by 2^-32 of it at most.
//   Output.  mma m16n8k16 on the values widened to fp16 (exact); p * vs is rounded to fp16
// (2^-11) after a power of two that keeps the largest that the row has had from this warp, as
// weighted against the present maximum, in [2^14, 2^15): what is lost lies below 2^-39 of it,
// whatever the size of the values.
// The tokens of all sequences form one list of tiles, cut into equal runs, one to a block, so
// that ragged batches and one long sequence fill the GPU alike; a sequence that a cut divides
// leaves partial results (maximum, sum, output) that a second kernel joins in order.
//   Bound by how fast the tiles come: 64 sequences of up to 16383 tokens (16 heads on 4, 318 MB)
// take 67 us, 54 of them in this kernel (5.8 TB/s: two blocks an SM with three tiles of 34 KB each
// in flight; scores and outputs keep its issue slots 41% and the MMA unit 25% busy); one of 131071
// tokens (138 MB) 35 us, 26 of them here, 4 of those before the first tile.  Short sequences are
// bound by the chain length, page number, tile, result: 300 tokens 6.2 us.
#include "attention.cuh"

namespace fge {

namespace {

constexpr int kWarps = 4;          // consumer warps, 32 tokens of a tile each
constexpr int kCopyWarp = kWarps, kZeroWarp = kWarps + 1;
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kStages = 3;
constexpr int kBlocksPerSm = 2;
constexpr int kMergeFloats = 2048;  // floats of the block's join buffer

template <int D>
struct Layout {
  static constexpr int kCodes = kTile * D;              // bytes of a tile's key or value codes
  static constexpr int kStage = 2 * kCodes + 2 * kTile * 4;
  static constexpr int kMerge = kStages * kStage;       // join buffer, then maxima and sums
  static constexpr int kBars = kMerge + kMergeFloats * 4 + 2 * kWarps * 16 * 4;
  static constexpr int kBytes = kBars + 3 * kStages * 8 + kStages * 4 + 32;
  static constexpr int kSmem = kBytes + 1024;           // slack to align the base
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The token list of one query-row group: which pages, how many tokens.
struct Segment {
  const int32_t* pages;
  int64_t width;
  int len;
};

// Tiles of a sequence: at least one, so that every row is written.
__device__ __forceinline__ int tiles_of(int len) { return max(1, tile_count(len)); }
// The tile list is cut by cost: an item (a sequence's row group) costs its tiles and kItemCost
// more, for its query and its result; those units come before its tiles.
constexpr int kItemCost = 1;

// a / b: 64-bit division costs hundreds of cycles, and few lists are that long.
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return a >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

struct Work {
  AttentionArgs a;
  int groups;         // row groups of a key/value head: blocks of ROWS of its query rows
  int group_rows;     // query rows of a key/value head (prefix: of the whole batch)
  int splits;         // prefix: runs that a row group's tiles are cut into
  int whole;          // each block one sequence and row group; nothing is divided
  // Partial results.  Prefix: [n_kv * groups * splits].  Decode: two for each of `blocks`
  // blocks (what it takes over from the block before, what it hands on), then, with a prefix,
  // one for each item that one block holds.
  float* partials;
  int blocks;
  const float* prefix_partials;
  int prefix_groups, prefix_splits, prefix_rows;  // how those are laid out (0: no prefix)
  int prefix_last;    // runs of a head's last group, prefix_splits those of the others
  int prefix_stride;  // partial results that a group has room for
};

constexpr int kPrefixRows = 16;  // query rows of a prefix item of this kernel

// Divides and writes N neighbouring outputs of a row, and at the first one its log-sum-exp.  A
// row without tokens (l = 0) is zeros.
template <int D, int N>
__device__ __forceinline__ void store_out(const AttentionArgs& a, int b, int h, int d, float m,
                                          float l, const float (&o)[N]) {
  const int64_t row = static_cast<int64_t>(b) * a.n_heads + h;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float x = l != 0.0f ? __fdiv_rn(o[i], l) : 0.0f;
    const float y = l != 0.0f ? __fdiv_rn(o[i + 1], l) : 0.0f;
    if (a.out_f32)
      reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + d)[i / 2] =
          make_float2(x, y);
    else
      reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D + d)[i / 2] =
          pack_bf16x2(x, y);
  }
  if (a.lse && d == 0) a.lse[row] = l != 0.0f ? 0.69314718056f * (m + log2f(l)) : -INFINITY;
}

// ROWS = 8: at most 8 query rows a group (half of a score MMA's rows idle); 16: up to 16.
template <int D, int ROWS, bool PREFIX>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    attention_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const Work w) {
  extern __shared__ uint8_t raw_smem[];
  using L = Layout<D>;
  uint8_t* sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  float* merge = reinterpret_cast<float*>(sm + L::kMerge);
  float* merge_ml = merge + kMergeFloats;
  const uint32_t bars = smem_u32(sm + L::kBars);
  const uint32_t zero_bars = bars + 2 * kStages * 8;
  uint32_t* chunk_mask = reinterpret_cast<uint32_t*>(sm + L::kBars + 3 * kStages * 8);
  int* shared_int = reinterpret_cast<int*>(chunk_mask + kStages);
  volatile int* s_abort = shared_int + 6;
  const AttentionArgs& a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = a.c.n_kv * w.groups;  // items of a sequence

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bars + 16 * i, 1);
      mbar_init(bars + 16 * i + 8, kWarps + 1);
      mbar_init(zero_bars + 8 * i, 1);
    }
    *s_abort = 0;
    fence_mbar_init();
  } else if (threadIdx.x == kCopyWarp * 32) {  // the first copies will want these
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  // This block's run of tiles: first sequence b, item hh (key/value head and row group) and
  // tile t of it, and how many tiles.
  if constexpr (PREFIX) {
    if (threadIdx.x == 0) {
      const int item = blockIdx.x / w.splits, s = blockIdx.x % w.splits;
      const int len = clamp_length(*a.prefix_length, a.prefix_width, a.c, a.status);
      const int tiles = tile_count(len);
      const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * s / w.splits);
      shared_int[0] = 0;
      shared_int[1] = item;
      shared_int[2] = t0;
      shared_int[3] = static_cast<int>(static_cast<int64_t>(tiles) * (s + 1) / w.splits) - t0;
    }
  } else if (w.whole) {
    if (threadIdx.x == 0) {
      const int b = blockIdx.x / per_seq;
      shared_int[0] = b;
      shared_int[1] = blockIdx.x % per_seq;
      shared_int[2] = 0;
      shared_int[3] = tiles_of(quiet_length(a.lengths[b], a.table_width, a.c.page_shift));
    }
  } else if (warp == 0) {
    auto units_of = [&](int i) {
      return i < a.B ? static_cast<int64_t>(per_seq) *
                           (kItemCost + tiles_of(quiet_length(a.lengths[i], a.table_width,
                                                              a.c.page_shift)))
                     : 0;
    };
    int64_t total = 0;
    for (int i = lane; i < a.B; i += 32) total += units_of(i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    const int blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
    const int64_t lo = quotient(total * block, blocks);
    const int64_t hi = quotient(total * (block + 1), blocks);
    if (lane == 0) shared_int[3] = 0;
    __syncwarp();
    int64_t before = 0;  // units of the sequences before the chunk of 32
    for (int i0 = 0; i0 < a.B; i0 += 32) {
      const int i = i0 + lane;
      const int64_t mine = units_of(i);
      int64_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      if (lo >= before + upto - mine && lo < before + upto) {
        const int per_item = static_cast<int>(quotient(mine, per_seq));
        const int64_t in = lo - (before + upto - mine);
        const int item = static_cast<int>(quotient(in, per_item));
        const int off = static_cast<int>(in - static_cast<int64_t>(item) * per_item);
        shared_int[0] = i;
        shared_int[1] = item;
        shared_int[2] = max(0, off - kItemCost);
        shared_int[3] = static_cast<int>(hi - lo) - max(0, kItemCost - off);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
      if (lo < before) break;
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int b = shared_int[0], hh = shared_int[1], t = shared_int[2], units = shared_int[3];
  if (!PREFIX && units <= 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  auto segment = [&](int bb) {
    Segment s;
    if (PREFIX) {
      s.pages = a.prefix_pages;
      s.width = a.prefix_width;
      s.len = quiet_length(*a.prefix_length, s.width, a.c.page_shift);
    } else {
      s.pages = a.page_table + static_cast<int64_t>(bb) * a.table_width;
      s.width = a.table_width;
      s.len = quiet_length(a.lengths[bb], s.width, a.c.page_shift);
    }
    return s;
  };

  if (warp == kCopyWarp) {
    // ---------------------------------------------------------------------- producer
    // lanes 0-7 copy key boxes, 8-15 value boxes, 16-23 and 24-31 their scales
    const int role = lane >> 3, box = lane & 7;
    const int box_shift = min(a.c.page_shift, 7), box_rows = 1 << box_shift;
    const int boxes = kTile >> box_shift, box_chunks = box_rows / 16;
    bool dead = false;
    int n_issued = 0;
    Segment seg = segment(b);
    if (!PREFIX && lane == 0 && t == 0 && hh == 0)
      clamp_length(a.lengths[b], a.table_width, a.c, a.status);
    auto page_of = [&](const Segment& s, int tile) {
      const int tok = tile * kTile + box * box_rows;
      return box < boxes && tok < s.len ? __ldg(s.pages + (tok >> a.c.page_shift)) : 0;
    };
    int page = page_of(seg, t);
    for (int it = 0; units > 0 && !dead; ++it) {
      const int st = it % kStages;
      if (it >= kStages) dead = !mbar_wait(bars + 16 * st + 8, ((it / kStages) - 1) & 1, s_abort, a.status);
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      const int tok = t * kTile + box * box_rows;
      const bool want = box < boxes && tok < seg.len;
      const bool ok = want && page >= 0 && page < a.c.n_pages;
      if (want && !ok && role == 0) set_device_error(a.status, FGE_ERR_BAD_INDEX);
      // bit c: tokens [16 c, 16 c + 16) of the tile are there
      const uint32_t chunks = __reduce_or_sync(
          0xffffffffu, ok ? ((1u << box_chunks) - 1u) << (box * box_chunks) : 0u);
      if (lane == 0) {
        chunk_mask[st] = chunks;
        mbar_arrive_expect_tx(bars + 16 * st,
                              static_cast<uint32_t>(__popc(chunks) * 16 * (2 * D + 8)));
      }
      __syncwarp();
      if (ok) {
        const int kv = hh / w.groups;
        const int row = ((page * a.c.n_kv + kv) << a.c.page_shift) + (tok & (a.c.page_size - 1));
        const uint32_t base = smem_u32(sm + st * L::kStage);
        const uint32_t bar = bars + 16 * st;
        if (role == 0)
          tma_load_2d(base + box * box_rows * D, &k_map, bar, 0, row);
        else if (role == 1)
          tma_load_2d(base + L::kCodes + box * box_rows * D, &v_map, bar, 0, row);
        else
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
              "[%3];" ::"r"(base + 2 * L::kCodes + (role - 2) * kTile * 4 + box * box_rows * 4),
              "l"(reinterpret_cast<uint64_t>((role == 2 ? a.c.k_scales : a.c.v_scales) + row)),
              "r"(box_rows * 4), "r"(bar)
              : "memory");
      }
      n_issued = it + 1;
      // the next tile's place, and its page number on the way
      int nb = b, nhh = hh, nt = t + 1;
      Segment nseg = seg;
      --units;
      if (nt >= tiles_of(seg.len)) {
        nt = 0;
        units -= kItemCost;
        if (++nhh == per_seq) {
          nhh = 0;
          ++nb;
          if (units > 0) {
            nseg = segment(nb);
            if (!PREFIX && lane == 0) clamp_length(a.lengths[nb], a.table_width, a.c, a.status);
          }
        }
      }
      const int npage = units > 0 ? page_of(nseg, nt) : 0;

      b = nb;
      hh = nhh;
      t = nt;
      seg = nseg;
      page = npage;
    }
    if (dead) {  // leave no copy of this block in flight
      int zero = 0;
      for (int i = max(0, n_issued - kStages); i < n_issued; ++i)
        mbar_wait(bars + 16 * (i % kStages), (i / kStages) & 1, &zero, a.status);
    }
    // this kernel needs nothing of the prefix's, which may still run, but who follows it
    // counts on both being finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  if (warp == kZeroWarp) {
    // ------------------------------------------------------------------- rows of value zero
    // A token whose codes are all zero takes no part in the weights: its scale, 1 from
    // kv_cache_write, must not set the range of the others.  It is taken as zero, while the
    // consumers work on the tile's scores.  (300 tokens take 6.2 us so, 6.0 without the look, 7.1
    // with the consumers looking for themselves wherever a range begins or moves; the ragged
    // batch 70.6, 70.5 and 73.1 us.)
    bool dead = false;
    for (int it = 0; units > 0;) {
      const int tiles = PREFIX ? t + units : tiles_of(segment(b).len);
      const int run = min(units, tiles - t);
      units -= run;
      t += run;
      for (const int end = it + run; it < end; ++it) {
        const int st = it % kStages;
        if (!dead) dead = !mbar_wait(bars + 16 * st, (it / kStages) & 1, s_abort, a.status);
        dead = __any_sync(0xffffffffu, dead);
        if (dead) continue;
        const uint8_t* vs = sm + st * L::kStage + L::kCodes;
        float* vscale = reinterpret_cast<float*>(sm + st * L::kStage + 2 * L::kCodes) + kTile;
#pragma unroll
        for (int r = lane; r < kTile; r += 32) {
          uint32_t some = 0;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(vs + swizzled<D>(r, c));
            some |= v.x | v.y | v.z | v.w;
          }
          if (!(some & 0x7F7F7F7Fu)) vscale[r] *= 0.0f;
        }
        fence_proxy_async_smem();  // before a later copy into this stage
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(zero_bars + 8 * st);
          mbar_arrive(bars + 16 * st + 8);
        }
      }
      if (t >= tiles) {
        t = 0;
        units -= kItemCost;
        if (++hh == per_seq) {
          hh = 0;
          ++b;
        }
      }
    }
    return;
  }

  // ------------------------------------------------------------------------ consumers
  constexpr int kSteps = D / 16;      // MMA steps of a score
  constexpr int kDt = D / 16;         // 16-dim tiles of the output
  constexpr int kOut = ROWS / 4;      // scores of a lane and 8 tokens
  const int g = lane >> 2, qd = lane & 3;
  const int group = a.n_heads / a.c.n_kv;
  bool dead = false;
  int it = 0;
  if (PREFIX && units <= 0) {  // a run without tiles leaves an empty partial result
    float* part = w.partials + static_cast<int64_t>(blockIdx.x) * partial_floats(ROWS, D);
    if (threadIdx.x < ROWS) part[ROWS + threadIdx.x] = 0.0f;
  }
  while (units > 0) {
    // ---- one item's run of tiles: row group hh of sequence b from tile t on
    const Segment seg = segment(b);
    const int tiles = PREFIX ? t + units : tiles_of(seg.len);
    const int first = t;
    const int run = min(units, tiles - t);
    units -= run;
    const int kv = hh / w.groups, row0 = (hh % w.groups) * ROWS;
    const int rows = min(ROWS, w.group_rows - row0);
    // query fragments: lane (g, qd) holds dims [D/4 qd, D/4 (qd + 1)) of row g; with 16 rows
    // those of row g + 8 wait in this warp's quarter of the join buffer
    uint32_t qa[kSteps][2];
    uint32_t* q_high = reinterpret_cast<uint32_t*>(merge) + warp * (kMergeFloats / kWarps);
    float row_scale[ROWS / 8];
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half) {
      const int r = row0 + g + 8 * half;
      const bool live = g + 8 * half < rows;
      uint32_t x[D / 8];
      const int qb = PREFIX ? r / group : b, qh = kv * group + (PREFIX ? r % group : r);
      const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(qb) * a.q_stride +
                                                        qh * D + qd * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
      }
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) m = max(m, max((x[i] >> 16) & 0x7FFFu, x[i] & 0x7FFFu));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // 2^k brings the largest value to [128, 256); biased exponents, both factors kept normal
      const int up = min(253, max(1, 134 + 127 - static_cast<int>(m >> 7)));
      const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
      row_scale[half] = __uint_as_float(static_cast<uint32_t>(254 - up) << 23) * a.scale *
                        1.4426950408889634f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t v = x[2 * s + p];
          const uint32_t f = pack_f16x2(bf16_lo(v) * mul, bf16_hi(v) * mul);
          if (half == 0) qa[s][p] = f;
          else q_high[(s * 32 + lane) * 2 + p] = f;
        }
    }
    // outputs transposed: tile i of 16 dims, query rows 2 qd, + 1 (of each 8); the softmax
    // state of row g (+ 8): reference maximum, sum, exponent of the output's scale
    float o[ROWS / 8][kDt][4], m_ref[ROWS / 8], l_run[ROWS / 8];
    int scale_exp[ROWS / 8];
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half) {
#pragma unroll
      for (int i = 0; i < kDt; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[half][i][x] = 0.0f;
      m_ref[half] = -INFINITY;
      l_run[half] = 0.0f;
      scale_exp[half] = 1;
    }

    for (int n = 0; n < run; ++n, ++t, ++it) {
      const int st = it % kStages;
      if (!dead) dead = !mbar_wait(bars + 16 * st, (it / kStages) & 1, s_abort, a.status);
      dead = __any_sync(0xffffffffu, dead);
      if (dead) continue;
      uint8_t* ks = sm + st * L::kStage;
      uint8_t* vs = ks + L::kCodes;
      const float* kscale = reinterpret_cast<const float*>(vs + L::kCodes) + 32 * warp;
      const float* vscale = kscale + kTile;
      const int avail = seg.len - t * kTile - 32 * warp;  // tokens of this warp that exist
      const uint32_t chunks = chunk_mask[st] >> (2 * warp);
      // bit r: token r of this warp's 32 is there
      const uint32_t there = (avail >= 32 ? ~0u : avail > 0 ? (1u << avail) - 1u : 0u) &
                             ((chunks & 1u ? 0xFFFFu : 0u) | (chunks & 2u ? 0xFFFF0000u : 0u));
      if (there) {
        const bool full = there == ~0u;
        if (!full) {
          // a value code that stands for no token may be anything, and 0 * NaN is NaN
          for (int r = 0; r < 32; ++r)
            if (!(there >> r & 1u) && lane < D / 4)
              *reinterpret_cast<uint32_t*>(vs + (32 * warp + r) * D + lane * 4) = 0;
          fence_proxy_async_smem();  // before a later copy into this stage
          __syncwarp();
        }
        // ---- scores of 32 tokens: lane holds tokens 8 j + 2 qd, + 1 of rows g (and g + 8)
        float s[4][kOut];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 32 * warp + 8 * j + g;
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint4 kw = *reinterpret_cast<const uint4*>(
                ks + swizzled<D>(r, D == 128 ? 2 * qd + h : qd));
            const uint32_t word[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t af[4] = {qa[4 * h + i][0], 0u, qa[4 * h + i][1], 0u}, b0, b1;
              if constexpr (ROWS == 16) {
                const uint2 high = *reinterpret_cast<const uint2*>(
                    q_high + ((4 * h + i) * 32 + lane) * 2);
                af[1] = high.x;
                af[3] = high.y;
              }
              e4m3x4_f16x4(word[i], b0, b1);
              mma_f16(c, af, b0, b1);
            }
          }
          const float2 sc = *reinterpret_cast<const float2*>(kscale + 8 * j + 2 * qd);
#pragma unroll
          for (int i = 0; i < kOut; ++i) s[j][i] = c[i] * ((i & 1 ? sc.y : sc.x) * row_scale[i >> 1]);
          if (!full) {
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
              const int tok = 8 * j + 2 * qd + (i & 1);
              if (!(there >> tok & 1u)) s[j][i] = -INFINITY;
            }
          }
        }
        // ---- softmax.  The reference maximum moves only when a score passes it by 8 (in base
        // 2), and the power of two that brings p * vs into fp16 only when one would pass 2^15 or
        // when the reference moves, so the output is rescaled rarely and the MMAs add straight
        // into it.  References are whole numbers: what came before falls by 2^-drop exactly, and
        // the range that it needed falls as much.  A range that only ever rose would go on
        // holding a large value that has lost its weight, and drop what has taken it.
        if (!dead) dead = !mbar_wait(zero_bars + 8 * st, (it / kStages) & 1, s_abort, a.status);
        uint32_t pf[ROWS / 8][4];
        float factor[ROWS / 8];  // of the outputs
        bool moved = false;
#pragma unroll
        for (int half = 0; half < ROWS / 8; ++half) {
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * half], s[j][2 * half + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const bool up_m = mx > m_ref[half] + 8.0f;
          const float mn = up_m ? ceilf(mx) : m_ref[half];
          const int drop = up_m ? static_cast<int>(fminf(mn - m_ref[half], 1024.0f)) : 0;
          l_run[half] *= up_m ? exp2_approx(m_ref[half] - mn) : 1.0f;
          m_ref[half] = mn;
          float sum = 0.0f, top = 0.0f;
          float pv[4][2];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 sc = *reinterpret_cast<const float2*>(vscale + 8 * j + 2 * qd);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p = exp2_approx(s[j][2 * half + i] - mn);
              sum += p;
              const float scale = i ? sc.y : sc.x;
              pv[j][i] = full || (there >> (8 * j + 2 * qd + i) & 1u) ? p * scale : 0.0f;
              top = fmaxf(top, fabsf(pv[j][i]));
            }
          }
          l_run[half] += sum;
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = static_cast<int>(__float_as_uint(top) >> 23) - 14;
          const int range = max(max(1, scale_exp[half] - drop), e);
          const int shift = drop + range - scale_exp[half];  // down by 2^shift; none below 0
          factor[half] = __uint_as_float(static_cast<uint32_t>(max(0, 127 - shift)) << 23);
          scale_exp[half] = range;
          moved |= shift != 0;
          const float up = __uint_as_float(static_cast<uint32_t>(254 - scale_exp[half]) << 23);
#pragma unroll
          for (int j = 0; j < 4; ++j) pf[half][j] = pack_f16x2(pv[j][0] * up, pv[j][1] * up);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int half = 0; half < ROWS / 8; ++half) {
            const float f0 = __shfl_sync(0xffffffffu, factor[half], 8 * qd);
            const float f1 = __shfl_sync(0xffffffffu, factor[half], 8 * qd + 4);
#pragma unroll
            for (int i = 0; i < kDt; ++i) {
              o[half][i][0] *= f0;
              o[half][i][1] *= f1;
              o[half][i][2] *= f0;
              o[half][i][3] *= f1;
            }
          }
        }
        // ---- output, transposed: values as the 16-row operand, 64 dims at a time.  Rows g and
        // g + 8 of tile 4 hw + 2 wd + pair are dims 64 hw + 8 g + 4 wd + 2 pair and the next;
        // the probabilities of row g are the 8-column operand as they lie in the registers.
#pragma unroll
        for (int hw = 0; hw < D / 64; ++hw) {
          uint32_t vw[2][4][2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 32 * warp + 16 * u + 8 * (k >> 1) + 2 * qd + (k & 1);
              const uint2 v = *reinterpret_cast<const uint2*>(
                  vs + swizzled<D>(r, 4 * hw + (g >> 1)) + 8 * (g & 1));
              vw[u][k][0] = v.x;
              vw[u][k][1] = v.y;
            }
#pragma unroll
          for (int wd = 0; wd < 2; ++wd)
#pragma unroll
            for (int pair = 0; pair < 2; ++pair)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t af[4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  e4m3x4_f16x4(prmt(vw[u][2 * k][wd], vw[u][2 * k + 1][wd],
                                    pair ? 0x7362u : 0x5140u),
                               af[2 * k], af[2 * k + 1]);
#pragma unroll
                for (int half = 0; half < ROWS / 8; ++half)
                  mma_f16(o[half][4 * hw + 2 * wd + pair], af, pf[half][2 * u],
                          pf[half][2 * u + 1]);
              }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 16 * st + 8);
    }

    // ---- join the four warps, kMergeFloats at a time, and write the result
    float inv[ROWS / 8][2];  // the outputs' scale, for rows 2 qd and 2 qd + 1
#pragma unroll
    for (int half = 0; half < ROWS / 8; ++half) {
      l_run[half] += __shfl_xor_sync(0xffffffffu, l_run[half], 1);
      l_run[half] += __shfl_xor_sync(0xffffffffu, l_run[half], 2);
      const float sc = __uint_as_float(static_cast<uint32_t>(scale_exp[half]) << 23);
      inv[half][0] = __shfl_sync(0xffffffffu, sc, 8 * qd);
      inv[half][1] = __shfl_sync(0xffffffffu, sc, 8 * qd + 4);
      if (qd == 0) {
        merge_ml[warp * 16 + g + 8 * half] = m_ref[half];
        merge_ml[kWarps * 16 + warp * 16 + g + 8 * half] = l_run[half];
      }
    }
    const bool divided = !PREFIX && !w.whole && (first > 0 || t < tiles);
    float* part = nullptr;
    if (PREFIX || divided || w.prefix_splits) {
      const int64_t slot =
          PREFIX ? static_cast<int64_t>(blockIdx.x)
          : divided
              ? 2 * static_cast<int64_t>(blockIdx.x) + (first > 0 ? 0 : 1)
              : 2 * static_cast<int64_t>(w.blocks) + static_cast<int64_t>(b) * per_seq + hh;
      part = w.partials + slot * partial_floats(ROWS, D);
    }
    // a round: kDims dims of every row; [warp][row][dim of the round].  A thread joins 4 dims of
    // one row, whose warps' weights it works out once.
    constexpr int kDims = kMergeFloats / (kWarps * ROWS);
    constexpr int kPer = kDims / 8;  // dims of a lane's g: 8 (rounds of 64 dims) or 4
    const int jr = threadIdx.x / (kDims / 4), at = threadIdx.x % (kDims / 4) * 4;
    float weight[kWarps], m_all = -INFINITY, l_all = 0.0f;
#pragma unroll 1
    for (int round = 0; round < D / kDims; ++round) {
#pragma unroll
      for (int i = 0; i < kDt; ++i) {
        if (i / (kPer / 2) != round) continue;
#pragma unroll
        for (int half = 0; half < ROWS / 8; ++half)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            *reinterpret_cast<float2*>(merge + (warp * ROWS + 8 * half + 2 * qd + x) * kDims +
                                       kPer * g + 2 * (i % (kPer / 2))) =
                make_float2(o[half][i][x] * inv[half][x], o[half][i][2 + x] * inv[half][x]);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
      if (round == 0) {
        // a warp without tokens has l = 0 and counts for nothing
        float mw[kWarps], lw[kWarps];
#pragma unroll
        for (int ww = 0; ww < kWarps; ++ww) {
          mw[ww] = merge_ml[ww * 16 + jr];
          lw[ww] = merge_ml[kWarps * 16 + ww * 16 + jr];
          if (lw[ww] != 0.0f) m_all = fmaxf(m_all, mw[ww]);
        }
#pragma unroll
        for (int ww = 0; ww < kWarps; ++ww) {
          weight[ww] = lw[ww] != 0.0f ? exp2_approx(mw[ww] - m_all) : 0.0f;
          if (lw[ww] != 0.0f) l_all = fmaf(lw[ww], weight[ww], l_all);
        }
      }
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ww = 0; ww < kWarps; ++ww) {
        const float4 x = *reinterpret_cast<const float4*>(merge + (ww * ROWS + jr) * kDims + at);
        v[0] = fmaf(x.x, weight[ww], v[0]);
        v[1] = fmaf(x.y, weight[ww], v[1]);
        v[2] = fmaf(x.z, weight[ww], v[2]);
        v[3] = fmaf(x.w, weight[ww], v[3]);
      }
      const int d =
          kPer == 8 ? round * 64 + at : (round >> 1) * 64 + 2 * at + 4 * (round & 1);
      if (jr < rows) {
        if (part) {
          if (d == 0) {
            part[jr] = m_all;
            part[ROWS + jr] = l_all;
          }
          *reinterpret_cast<float4*>(part + 2 * ROWS + jr * D + d) =
              make_float4(v[0], v[1], v[2], v[3]);
        } else {
          store_out<D, 4>(a, b, kv * group + row0 + jr, d, m_all, l_all, v);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    }
    if (t >= tiles) {
      t = 0;
      units -= kItemCost;
      if (++hh == per_seq) {
        hh = 0;
        ++b;
      }
    }
  }
}

// Joins the partial results of a query row: what the cuts of the tile list divided, and the
// prefix's.  LANES warps a row, each taking every LANES-th partial result: the weights first, a
// partial result a lane, then the outputs, D / 32 dims a lane.
constexpr int kJoinMost = 1024;  // partial results of a row

template <int D, int LANES>
__global__ void __launch_bounds__(LANES == 1 ? 128 : LANES * 32)
    attention_join_kernel(const Work w, int rows_per_group) {
  constexpr int kPer = D / 32, kRowsBlock = LANES == 1 ? 4 : 1;
  const AttentionArgs& a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = LANES == 1 ? 0 : warp;
  const int64_t query = static_cast<int64_t>(blockIdx.x) * kRowsBlock + (LANES == 1 ? warp : 0);
  const bool live = query < a.B * a.n_heads;
  const int b = live ? static_cast<int>(query / a.n_heads) : 0;
  const int h = live ? static_cast<int>(query - static_cast<int64_t>(b) * a.n_heads) : 0;
  const int group = a.n_heads / a.c.n_kv, kv = h / group;
  const int per_seq = a.c.n_kv * w.groups;
  const int hh = kv * w.groups + (h - kv * group) / rows_per_group;
  const int row = (h - kv * group) % rows_per_group;
  // the item's run of the tile list, and the blocks that hold its ends
  int c0 = 0, c1 = 0;
  int64_t total = 0;
  if (!w.whole) {
    int64_t before = 0;
    for (int i = lane; i < a.B; i += 32) {
      const int n =
          kItemCost + tiles_of(quiet_length(a.lengths[i], a.table_width, a.c.page_shift));
      total += n;
      if (i < b) before += n;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, x);
      before += __shfl_xor_sync(0xffffffffu, before, x);
    }
    total *= per_seq;
    const int tiles = tiles_of(quiet_length(a.lengths[b], a.table_width, a.c.page_shift));
    const int64_t start =
        before * per_seq + static_cast<int64_t>(hh) * (tiles + kItemCost) + kItemCost;
    // the block that holds unit x of the list: the largest c with total * c / blocks <= x
    auto block_of = [&](int64_t x) {
      int64_t c = (x * w.blocks + w.blocks - 1) / total;
      while (c > 0 && total * c / w.blocks > x) --c;
      while (c + 1 < w.blocks && total * (c + 1) / w.blocks <= x) ++c;
      return static_cast<int>(c);
    };
    c0 = block_of(start);
    c1 = block_of(start + tiles - 1);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // one row a block: all of its warps leave together
  if (!live || (c0 == c1 && !w.prefix_splits)) return;  // not divided: already written

  // Partial results: `own` of the tile list (the first handed on, the others taken over), then
  // the prefix's; each its maxima, its sums, its outputs.
  const int64_t rr = static_cast<int64_t>(b) * group + h - kv * group;  // rows of the batch
  const int prefix_group = w.prefix_splits ? static_cast<int>(rr / w.prefix_rows) : 0;
  const int runs = prefix_group + 1 < w.prefix_groups ? w.prefix_splits : w.prefix_last;
  const int own = c1 - c0 + 1, n = own + runs;
  const int64_t own_floats = rows_per_group * (D + 2);
  const float* own_first =
      w.partials + (c0 == c1 ? 2 * static_cast<int64_t>(w.blocks) +
                                   static_cast<int64_t>(b) * per_seq + hh
                             : 2 * static_cast<int64_t>(c0) + 1) * own_floats;
  const float* own_next = w.partials + 2 * static_cast<int64_t>(c0) * own_floats;
  const int prefix_row = w.prefix_splits ? static_cast<int>(rr - static_cast<int64_t>(prefix_group) *
                                                                     w.prefix_rows)
                                         : 0;
  const int64_t prefix_floats = partial_floats(w.prefix_rows, D);
  const float* prefix =
      w.prefix_splits ? w.prefix_partials +
                            (static_cast<int64_t>(kv) * w.prefix_groups + prefix_group) *
                                w.prefix_stride * prefix_floats
                      : nullptr;
  auto ml_of = [&](int i, float* l) {  // maximum and sum of partial result i
    const float* p = i >= own ? prefix + (i - own) * prefix_floats + prefix_row
                     : i == 0 ? own_first + row
                              : own_next + 2 * i * own_floats + row;
    // a block without tiles (there are fewer tiles than blocks) holds nothing of the list
    const bool empty = i < own && total < w.blocks && c0 != c1 &&
                       total * (c0 + i) / w.blocks == total * (c0 + i + 1) / w.blocks;
    *l = empty ? 0.0f : __ldcg(p + (i >= own ? w.prefix_rows : rows_per_group));
    const float m = __ldcg(p);
    // NaN sums (a NaN query) must reach the output: only an empty partial result is dropped
    return *l == 0.0f ? -INFINITY : m == -INFINITY ? NAN : m;
  };
  float m = -INFINITY, l = 0.0f, o[kPer] = {};
  // a round: up to 32 partial results of this warp, i = part + LANES (32 round + lane)
  for (int r0 = part; r0 < n; r0 += 32 * LANES) {
    const int mine = r0 + LANES * lane;
    float li = 0.0f, mi = -INFINITY;
    if (mine < n) mi = ml_of(mine, &li);
    float top = fmaxf(m, mi);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float scale = m == -INFINITY ? 0.0f : exp2_approx(m - top);
    const float f = mi == -INFINITY ? 0.0f : exp2_approx(mi - top);
    m = top;
    l = l * scale;
    l = fmaf(f, li, l);  // this lane's share
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] *= scale;
    const int count = min(32, (n - r0 + LANES - 1) / LANES);
#pragma unroll 8
    for (int j = 0; j < count; ++j) {
      const int i = r0 + LANES * j;
      const float fj = __shfl_sync(0xffffffffu, f, j);
      const float* p =
          (i >= own ? prefix + (i - own) * prefix_floats + 2 * w.prefix_rows + prefix_row * D
           : i == 0 ? own_first + 2 * rows_per_group + row * D
                    : own_next + 2 * i * own_floats + 2 * rows_per_group + row * D) +
          lane * kPer;
      // an empty partial result's outputs were never written: they may be anything
      if constexpr (kPer == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
        if (fj != 0.0f) {
          o[0] = fmaf(fj, v.x, o[0]);
          o[1] = fmaf(fj, v.y, o[1]);
          o[2] = fmaf(fj, v.z, o[2]);
          o[3] = fmaf(fj, v.w, o[3]);
        }
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
        if (fj != 0.0f) {
          o[0] = fmaf(fj, v.x, o[0]);
          o[1] = fmaf(fj, v.y, o[1]);
        }
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if constexpr (LANES > 1) {
    __shared__ float sm[LANES], sl[LANES], so[LANES][D];
    if (lane == 0) {
      sm[part] = m;
      sl[part] = l;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) so[part][lane * kPer + i] = o[i];
    __syncthreads();
    if (part) return;
    float top = -INFINITY, weight[LANES];
    l = 0.0f;
#pragma unroll
    for (int x = 0; x < LANES; ++x)
      if (sl[x] != 0.0f) top = fmaxf(top, sm[x]);
#pragma unroll
    for (int x = 0; x < LANES; ++x) {
      weight[x] = sl[x] != 0.0f ? exp2_approx(sm[x] - top) : 0.0f;
      if (sl[x] != 0.0f) l = fmaf(sl[x], weight[x], l);
    }
    m = top;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      o[i] = 0.0f;
#pragma unroll
      for (int x = 0; x < LANES; ++x)
        if (weight[x] != 0.0f) o[i] = fmaf(so[x][lane * kPer + i], weight[x], o[i]);
    }
  }
  store_out<D, kPer>(a, b, h, lane * kPer, m, l, o);
}

int blocks_of_list() { return std::min(num_sms() * kBlocksPerSm, kJoinMost - 64); }

// The prefix's query rows of a key/value head are those of the whole batch.  From 64 of them on
// they fill enough of a 128-row tcgen05 tile (4 heads, prefixes of 2048 and of 16384 tokens: 64
// rows 20.6 and 30.8 us for the whole call, 16 rows a time 22.7 and 31.0; 96 rows 18.6 and 31.0
// against 22.8 and 37.0; 800 rows 43 and 87 against 52 and 221; but 32 rows 20.3 and 29.1 against
// 20.6 and 26.7).
struct PrefixPlan {
  int rows, groups;  // rows of an item; items of a head
  int splits, last;  // runs of an item's tiles; of a head's last item
  int stride() const { return std::max(splits, last); }
};
PrefixPlan prefix_plan(int64_t B, int n_heads, int n_kv) {
  PrefixPlan p;
  const int64_t total = B * (n_heads / n_kv);
  p.rows = total >= 64 ? kPrefixTcRows : kPrefixRows;
  p.groups = static_cast<int>((total + p.rows - 1) / p.rows);
  // enough runs to fill the GPU, in whole waves where there are many row groups
  auto runs = [](int64_t n) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, n))); };
  if (p.rows != kPrefixTcRows) {
    p.splits = p.last = runs(blocks_of_list() / (static_cast<int64_t>(n_kv) * p.groups));
    return p;
  }
  // A tcgen05 block works on two items of 128 rows.  One that has an odd last item to itself takes
  // two thirds of the time a token tile, so it gets that part of the runs.
  const int64_t room = num_sms() / n_kv, pairs = p.groups / 2;
  if (p.groups % 2 == 0) {
    p.splits = p.last = runs(room / pairs);
  } else if (pairs == 0) {
    p.splits = p.last = runs(room);
  } else {
    p.splits = runs(3 * room / (3 * pairs + 2));
    p.last = runs(std::min<int64_t>(room - pairs * p.splits, p.splits));
  }
  return p;
}

template <int D, int ROWS, bool PREFIX>
cudaError_t launch_attention(const CUtensorMap& km, const CUtensorMap& vm, const Work& w,
                             int64_t grid, bool dependent, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const auto kern = attention_kernel<D, ROWS, PREFIX>;
  if (!device_kernel_ready(dev, reinterpret_cast<const void*>(kern), Layout<D>::kSmem, 0))
    return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, km, vm, w);
}

template <int D>
cudaError_t run_attention(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  CUtensorMap km, vm;
  if (!code_map(&km, a.c.k_codes, a.c) || !code_map(&vm, a.c.v_codes, a.c))
    return cudaErrorInvalidValue;
  const int group = a.n_heads / a.c.n_kv;
  const int rows = group <= 8 ? 8 : 16;
  Work w{};
  w.a = a;
  w.groups = (group + rows - 1) / rows;
  w.group_rows = group;
  w.partials = static_cast<float*>(scratch);
  const int64_t items = a.B * a.c.n_kv * w.groups;
  // Sequences of at most eight tiles are not divided: a block each costs less than the join
  // (16 heads on 4, all of the same length: 64 of 1024 tokens 20.4 us instead of 26.7 us, one of
  // 300 tokens 9.4 instead of 13.7, one of 1024 14.4 either way; one of 2048 would take 21.7 us
  // instead of 14.5).
  w.whole = (a.table_width << a.c.page_shift) <= 8 * kTile;
  w.blocks = blocks_of_list();
  const int64_t grid = w.whole ? items : w.blocks;
  cudaError_t e = cudaSuccess;
  if (a.shared) {
    PrefixPlan p = prefix_plan(a.B, a.n_heads, a.c.n_kv);
    // no more runs than tiles: an empty one still costs the join a look
    const int most = static_cast<int>(
        std::max<int64_t>(1, (a.prefix_width * a.c.page_size + kTile - 1) / kTile));
    p.splits = std::min(p.splits, most);
    p.last = std::min(p.last, most);
    Work pw = w;
    pw.groups = p.groups;
    pw.group_rows = static_cast<int>(a.B * group);
    pw.splits = p.splits;
    // on a 32-byte boundary, whatever the workspace's: the tcgen05 kernel writes whole sectors
    pw.partials = reinterpret_cast<float*>(align_up(
        reinterpret_cast<uintptr_t>(w.partials + (2 * w.blocks + items) * rows * (D + 2)), 32));
    e = p.rows == kPrefixTcRows
            ? launch_prefix_tc(a, p.groups, p.splits, p.last, pw.partials, s)
            : launch_attention<D, kPrefixRows, true>(
                  km, vm, pw, static_cast<int64_t>(p.groups) * a.c.n_kv * p.splits, false, s);
    if (e != cudaSuccess) return e;
    w.prefix_rows = p.rows;
    w.prefix_partials = pw.partials;
    w.prefix_groups = p.groups;
    w.prefix_splits = p.splits;
    w.prefix_last = p.last;
    w.prefix_stride = p.stride();
  }
  const bool dependent = a.shared;
  e = rows == 8 ? launch_attention<D, 8, false>(km, vm, w, grid, dependent, s)
                : launch_attention<D, 16, false>(km, vm, w, grid, dependent, s);
  if (e != cudaSuccess || (w.whole && !w.prefix_splits)) return e;
  // Few rows, or many partial results of each: several warps share a row's.  One sequence of
  // 131071 tokens took 38 us so, 64 us with one warp a row; 64 sequences of 4096 tokens 61 and
  // 54 us; 256 rows of a prefix in 38 runs 43 and 52 us, 384 rows in 19 runs 59 and 56 us.
  const int64_t queries = a.B * a.n_heads;
  if (queries * 16 >= 4LL * num_sms() * std::max(16, w.prefix_stride))
    return launch_chained(attention_join_kernel<D, 1>,
                          dim3(static_cast<unsigned>((queries + 3) / 4)), dim3(128), 0, s, w, rows);
  return launch_chained(attention_join_kernel<D, 8>, dim3(static_cast<unsigned>(queries)),
                        dim3(256), 0, s, w, rows);
}

}  // namespace

size_t attention_scratch_bytes(int64_t B, int n_heads, int head_dim, int n_kv, bool shared) {
  // what the call refuses needs nothing
  if (B <= 0 || B > kAttentionBatch || n_heads <= 0 || B * n_heads >= kAttentionRows ||
      head_dim <= 0 || n_kv <= 0 || n_heads % n_kv != 0)
    return 0;
  const int64_t group = n_heads / n_kv, rows = group <= 8 ? 8 : 16;
  size_t n = 2 * static_cast<size_t>(blocks_of_list()) * rows;
  if (shared) {
    const PrefixPlan p = prefix_plan(B, n_heads, n_kv);
    n += static_cast<size_t>(B) * n_kv * ((group + rows - 1) / rows) * rows +
         static_cast<size_t>(p.groups) * n_kv * p.stride() * p.rows;
  }
  return align_up(n * (head_dim + 2) * 4 + 32, 256);
}

cudaError_t launch_attention_decode(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  return a.c.head_dim == 128 ? run_attention<128>(a, scratch, s)
                             : run_attention<64>(a, scratch, s);
}

}  // namespace fge
