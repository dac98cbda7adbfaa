// Attention of every query token over its selected keys (forward).
//
//   z_j = scale * q_h . k[i_j];  z = cap * tanh(z / cap);  z -= slope_h |pos - i_j|
//   out_h = sum_j softmax(z)_j v[i_j],  lse_h = log sum_j exp z_j
// over the entries i_j of the token's index row that lie in [0, S) and in its
// key range; a row with none gives out = 0, lse = -inf.
//
// Every token has keys of its own, so a key row is read once per token and
// key head, and serves the G = H / Hk query heads that share it: G flops for
// every byte gathered.  Measured on GB300: 2048 queries x 64 heads x 128 with
// Top-2048 of a 128K cache 247 us (137 GFLOP: 556 TFLOP/s; 2.1 GB gathered: 8.7
// TB/s), 1024 x 128 heads of an 8K cache 124 us (1.11 PFLOP/s), one token 14 us in a
// graph.  A plain kernel gathers random 256-byte rows out of L2 at 20 TB/s (8.7
// with cp.async by 128 threads of an SM, 14 by 256; gather4 tensor copies issued
// by one warp reached 2.4), and the products of a tile take 1024 cycles; a tile
// takes 1560 in the middle of an item and 1900 on average.  What bounds it is the
// chain of hand-overs between the warps (S, P, P V, then the buffer's next S), and
// at an item's end the fetching of instructions that are not in the cache.

// An item is one token and one key head.  Its logits are a product of M = 128
// rows (query heads) with tiles of 128 gathered keys, tcgen05 with the
// accumulator in tensor memory, one row per softmax thread.  With fewer than
// 128 heads the rows are repeated: G <= 32 gives four copies, G <= 64 two.  A
// copy's threads take only their own quarter (half) of a tile's keys and keep
// their own running maximum and sum, the probabilities of the other keys stay
// zero, and the copies' partial results are joined at the end, as those of the
// CTAs of a cluster are: the softmax work spreads over all four warps at no
// cost in copies or barriers.
//
// One CTA per SM, persistent over items.  Warps:
//   0..7   softmax, two groups of four, tiles in turn: S from tensor memory,
//          running maximum and sum in FP32 (base 2), P rounded to the inputs'
//          16-bit type (the tensor core takes no wider operand beside 16-bit
//          values) into tensor memory.  The groups share each row's reference
//          maximum: a group settles its tile's before the other settles the
//          next one's.  It changes, and the accumulator is rescaled, only when
//          a maximum rises above it by more than 2^32 (BF16) or 2^15 (FP16:
//          P < 65504); a rescale stalls both groups and the tensor core, and at
//          2^8 sharp heads (logits of standard deviation 4) took 1.6 times as
//          long as flat ones.  In BF16 P is held 2^32 times smaller, so that it
//          never passes 1: sums overflow only where the values' own sum would
//   8..15  gather: cp.async of 16-byte pieces into rings of swizzled tiles,
//          four warps for the keys, four for the values
//   16..19 the finished items: O from tensor memory, joined and written, while
//          the softmax goes on with the next item
//   20     tensor core, S = Q K^T
//   21     index rows, compacted into tiles of valid keys
//   22     the items' query heads, one item ahead (the first item's: 16..19)
//   23     tensor core, P V (a warp of its own: the waits, the descriptors and the
//          commits of both took one warp 2500 cycles a tile, the products 1024)
// With few items a cluster of 2, 4 or 8 CTAs shares an item: CTA c takes the
// 128-entry chunks c, c + C, ... of the index row; the partial results are
// joined through distributed shared memory in a fixed order.
#include "per_device.h"
#include "sparse_attend.cuh"

#include <cmath>

namespace ta {

constexpr int THREADS = 768;
constexpr int GATHER = 128;  // gather threads of the keys, and as many of the values
// Registers of the six warpgroups after the split; launched with 80 each.
constexpr int REGS_SOFT = 88, REGS_GATHER = 40, REGS_END = 160, REGS_REST = 64;
static_assert(2 * REGS_SOFT + 2 * REGS_GATHER + REGS_END + REGS_REST <= 6 * 80, "register split");
constexpr int NI = 5;   // index tiles in flight
constexpr int NM = 4;   // items whose maxima and sums are kept: S(n) waits for P V of tile n - 3, so
                        // the item before that tile's has been read; the tiles from there to n
                        // can be of four items
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_O = 384;  // three buffers of 128 columns for S, then P in its place; O

// What the tensor-core warp tells a softmax group with a tile, and the last
// warps with an item.
struct Post {
  int32_t count, slot;   // valid keys, index slot
  int32_t nth, item;     // place in its item, which of this CTA's items with tiles
};
struct Done {
  int32_t tiles, first;  // tiles of the item, group of its first one
};
// An item's maxima and sums, by row: the reference, and each group's sum and the
// reference it goes by.
struct Rows {
  float ref[128];
  float sum[2][128], by[2][128];
};

template <int D>
struct Plan {
  static constexpr uint32_t BLOCK = KT * 128;             // 128 rows x 64 elements
  static constexpr uint32_t TILE = BLOCK * (D / 64);
  static constexpr uint32_t SLOTS = D == 128 ? 2 : 4;     // of K tiles, and as many of V tiles
  static constexpr uint32_t OFF_Q = 0;                    // two items' heads
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_STAGE = OFF_KV + 2 * SLOTS * TILE;   // [128][32] floats, swizzled
  static constexpr uint32_t OFF_IDX = OFF_STAGE + 128 * 32 * 4;
  static constexpr uint32_t OFF_ROWS = OFF_IDX + NI * sizeof(Tile);  // [NM]
  static constexpr uint32_t OFF_ML = OFF_ROWS + NM * sizeof(Rows);   // [2][128]: to be joined
  static constexpr uint32_t OFF_WT = OFF_ML + 2 * 128 * 4;           // [8][128]: CTAs' weights
  static constexpr uint32_t OFF_POST = OFF_WT + 8 * 128 * 4;         // [3] Post, Done
  static constexpr uint32_t OFF_BAR = OFF_POST + 64;
  static constexpr uint32_t NBAR = 4 * SLOTS + 2 * NI + 27;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 16 + 1008;  // + alignment slack
};
static_assert(Plan<128>::BYTES <= 232448 && Plan<64>::BYTES <= 232448, "shared memory plan");

// Infinite values.  A weight above zero times an infinite value is that infinity,
// but in the product such a value also meets weights that are zero (the other row
// copies', or one that underflowed), and 0 * inf is NaN.  A result that is NaN
// under a finite sum is therefore looked up in the values themselves: NaN or both
// signs selected, it stays; else it is the infinity.  Otherwise nothing but a check
// of 64 instructions per row is run.
//
// One warp: of the 32 columns from c0 on, in which does a selected value of token
// t, key head hk hold NaN, +inf, -inf (a bit per column each)?
template <bool BF16>
__device__ __forceinline__ void value_kinds(const Args& a, int32_t t, int32_t hk, uint32_t c0,
                                            uint32_t lane, uint32_t (&kinds)[3]) {
  constexpr uint32_t INF = BF16 ? 0x7f80u : 0x7c00u;
  const int32_t* idx = a.idx + (int64_t)t * a.ld_idx;
  const int32_t lo = a.lo ? max(a.lo[t], 0) : 0, hi = a.hi ? min(a.hi[t], a.S) : a.S;
  kinds[0] = kinds[1] = kinds[2] = 0u;
#pragma unroll 1
  for (int64_t j = lane; j < a.K; j += 32) {
    const int32_t i = idx[j];
    if (i < lo || i >= hi) continue;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) +
                                                          i * a.v_ts + hk * a.v_hs + c0 * 2u);
#pragma unroll 4
    for (uint32_t w = 0; w < 16; ++w) {
      const uint32_t two = __ldg(v + w);
#pragma unroll
      for (uint32_t s = 0; s < 2; ++s) {
        const uint32_t x = s ? two >> 16 : two & 0xffffu, bit = 1u << (2 * w + s);
        if ((x & 0x7fffu) > INF) kinds[0] |= bit;
        else if (x == INF) kinds[1] |= bit;
        else if (x == (0x8000u | INF)) kinds[2] |= bit;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) kinds[k] = __reduce_or_sync(0xffffffffu, kinds[k]);
}
// The result x of column c0 + column; `none`: the row's sum is zero.
template <bool BF16>
__device__ __forceinline__ uint16_t looked_up(uint16_t x, const uint32_t (&kinds)[3],
                                              uint32_t column, bool none) {
  constexpr uint32_t INF = BF16 ? 0x7f80u : 0x7c00u;
  if ((x & 0x7fffu) <= INF) return x;
  if (none) return 0;
  const bool pos = kinds[1] >> column & 1u, neg = kinds[2] >> column & 1u;
  if ((kinds[0] >> column & 1u) || pos == neg) return x;
  return (uint16_t)(pos ? INF : 0x8000u | INF);
}

// The warp's rows (lane's own at `row`, `odd`: it has such a NaN).  Not inlined: in
// the kernel's own code it took 280 us for 251 (2048 x 64 heads x 128, Top-2048)
// without ever running.
template <int D, bool BF16>
__device__ __noinline__ void look_up_rows(const Args* a, int32_t t, int32_t hk, uint32_t lane,
                                          uint16_t* row, bool odd, bool none) {
#pragma unroll 1
  for (uint32_t c0 = 0; c0 < (uint32_t)D; c0 += 32) {
    uint32_t kinds[3];
    value_kinds<BF16>(*a, t, hk, c0, lane, kinds);
    if (odd) {
#pragma unroll 1
      for (uint32_t i = 0; i < 32; ++i) row[c0 + i] = looked_up<BF16>(row[c0 + i], kinds, i, none);
    }
  }
}

// NC: key columns of a tile per row copy (128 / copies).  BENT: 1 a cap or a bias, 2 a cap
// above WIDE_CAP (a branch in one kernel instead took 288 us for 270).
// Chunks of 32 columns run in loops, not unrolled: five kinds of warps share the
// instruction cache, and 64 columns held in registers took longer than 32 read
// twice.
template <int D, int NC, bool BF16, int BENT>
__global__ void __launch_bounds__(THREADS, 1) k_attend(const __grid_constant__ Args a) {
  using P = Plan<D>;
  constexpr int PER = NC;  // rows per copy: with R = 128 / NC copies, 128 / R rows
  constexpr int COPIES = 128 / PER;
  // how far (base 2) a maximum may rise above its row's reference: P and the FP32
  // sums have the exponents for it, a relative error does not depend on them.  What
  // P is held smaller by: FP16 has no exponents to spare below, and its values do
  // not reach the end of FP32
  constexpr float GROWTH = BF16 ? 32.0f : 15.0f, SMALLER = BF16 ? 32.0f : 0.0f;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::saddr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  Tile* tiles = reinterpret_cast<Tile*>(sm + P::OFF_IDX);
  Rows* kept = reinterpret_cast<Rows*>(sm + P::OFF_ROWS);
  Post* posts = reinterpret_cast<Post*>(sm + P::OFF_POST);
  Done* done_post = reinterpret_cast<Done*>(sm + P::OFF_POST + 3 * sizeof(Post));
  const uint32_t bars = base + P::OFF_BAR;
  // slots 0 .. SLOTS - 1 hold K tiles, the next SLOTS V tiles
  auto kv_full = [&](uint32_t s) { return bars + 8u * s; };
  auto kv_empty = [&](uint32_t s) { return bars + 8u * (2 * P::SLOTS + s); };
  auto ix_full = [&](uint32_t s) { return bars + 8u * (4 * P::SLOTS + s); };
  auto ix_empty = [&](uint32_t s) { return bars + 8u * (4 * P::SLOTS + NI + s); };
  const uint32_t b0 = bars + 8u * (4 * P::SLOTS + 2 * NI);
  auto s_full = [&](uint32_t b) { return b0 + 8u * b; };
  auto p_full = [&](uint32_t b) { return b0 + 8u * (3 + b); };
  auto pv_done = [&](uint32_t b) { return b0 + 8u * (6 + b); };
  auto settled = [&](uint32_t g, uint32_t w) { return b0 + 8u * (9 + 4 * g + w); };
  auto q_full = [&](uint32_t b) { return b0 + 8u * (17 + b); };
  auto q_empty = [&](uint32_t b) { return b0 + 8u * (19 + b); };
  const uint32_t join = b0 + 168u, drain = b0 + 176u, meet = b0 + 184u, o_full = b0 + 192u,
                 o_empty = b0 + 200u, drain2 = b0 + 208u;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + P::OFF_MISC);
  volatile uint32_t* abort = misc + 1;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  uint32_t C;
  asm volatile("mov.u32 %0, %cluster_nctaid.x;" : "=r"(C));
  const uint32_t rank = C > 1 ? tc::cluster_rank() : 0u;
  const int32_t first = (int32_t)(blockIdx.x / C), step = (int32_t)(gridDim.x / C);
  // a whole warp waits, and goes on or gives up as one
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu,
                      tc::bar_wait(bar, parity, abort, &g_status, TOPK_FLAG_TIMEOUT)) != 0;
  };

  // the same for two barriers, which as a rule are both complete
  auto wait_both = [&](uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1) {
    const bool r0 = tc::bar_try(bar0, parity0), r1 = tc::bar_try(bar1, parity1);
    if (__all_sync(0xffffffffu, r0 && r1)) return true;
    return wait_warp(bar0, parity0) && wait_warp(bar1, parity1);
  };

  if (tid == 0) {
    for (uint32_t s = 0; s < 2 * P::SLOTS; ++s) {
      tc::bar_init(kv_full(s), GATHER);  // the gather threads' copies
      tc::bar_init(kv_empty(s), 1);
    }
    for (uint32_t s = 0; s < NI; ++s) {
      tc::bar_init(ix_full(s), 1);
      tc::bar_init(ix_empty(s), 10);  // 8 gather warps, two for the tensor-core warps
    }
    for (uint32_t b = 0; b < 3; ++b) {
      tc::bar_init(s_full(b), 2);  // the product and its post
      tc::bar_init(p_full(b), 4);
      tc::bar_init(pv_done(b), 1);
    }
    for (uint32_t w = 0; w < 8; ++w) tc::bar_init(settled(w >> 2, w & 3u), 1);
    for (uint32_t b = 0; b < 2; ++b) {
      tc::bar_init(q_full(b), 1);
      tc::bar_init(q_empty(b), 1);
    }
    tc::bar_init(drain, 1);
    tc::bar_init(drain2, 1);
    tc::bar_init(meet, 4);
    tc::bar_init(o_full, 2);  // the last product and its post
    tc::bar_init(o_empty, 4);
    tc::bar_init(join, 4 * C);
    *abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 20) tc::tm_alloc(tc::saddr(misc), TMEM_COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = misc[0];
  if (C > 1) tc::cluster_sync();

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    tc::regs_up<REGS_SOFT>();
    const uint32_t wg = warp >> 2, wq = warp & 3u;
    const uint32_t row = wq * 32u + lane, copy = row / PER, h = row % PER;
    const uint32_t lanes = (wq * 32u) << 16;
    const uint32_t col0 = copy * NC;
    const float sc = a.scale * LOG2E, mul = BENT ? 1.0f : sc;
    const float cap_in = a.cap > 0.0f ? a.scale / a.cap : 0.0f, cap_out = a.cap * LOG2E;
    float own = -INFINITY, l = 0.0f;  // this group's sum of the item, relative to 2^own
    int32_t item_seen = -1;
    float slope = 0.0f;
    int32_t pos = 0;
    // tile n of the CTA's, in buffer b, use number u of it
    for (uint32_t n = wg;; n += 2u) {
      const uint32_t u = n / 3u, b = n - 3u * u;
      if (!wait_warp(s_full(b), u & 1u)) break;
      const Post post = posts[b];
      if (post.count == 0) break;  // no more tiles
      tc::fence_after();
      const uint32_t tm_p = tmem + lanes + b * 128u, tm_s = tm_p + col0;
      const Tile* tile = tiles + post.slot;
      Rows* keep = kept + post.item % NM;
      if (post.item != item_seen) {
        item_seen = post.item;
        own = -INFINITY;
        l = 0.0f;
        if (BENT && a.slopes) {
          const int32_t t = tile->token, hk = tile->mark;
          slope = (int32_t)h < a.G ? a.slopes[hk * a.G + h] * LOG2E : 0.0f;
          pos = a.pos[t];
        }
      }
      // 32 raw products -> base-2 logits, where that takes more than a factor
      auto finish = [&](float (&x)[32], int at) {
        if (BENT) {
          if (BENT == 2) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = cap_out * tanh_near(x[i] * cap_in);
          } else if (a.cap > 0.0f) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = cap_out * tanh_of(x[i] * cap_in);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= sc;
          }
          if (a.slopes) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int4 key = *reinterpret_cast<const int4*>(tile->key + col0 + at + i);
              x[i] -= slope * fabsf((float)(pos - key.x));
              x[i + 1] -= slope * fabsf((float)(pos - key.y));
              x[i + 2] -= slope * fabsf((float)(pos - key.z));
              x[i + 3] -= slope * fabsf((float)(pos - key.w));
            }
          }
        }
        if (post.count < KT) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if ((int32_t)(col0 + at + i) >= post.count) x[i] = -INFINITY;
        }
      };
      auto largest = [](const float (&x)[32]) {
        float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[2], x[3]);
        float m2 = fmaxf(x[4], x[5]), m3 = fmaxf(x[6], x[7]);
#pragma unroll
        for (int i = 8; i < 32; i += 8) {
          m0 = fmaxf(m0, fmaxf(x[i], x[i + 1]));
          m1 = fmaxf(m1, fmaxf(x[i + 2], x[i + 3]));
          m2 = fmaxf(m2, fmaxf(x[i + 4], x[i + 5]));
          m3 = fmaxf(m3, fmaxf(x[i + 6], x[i + 7]));
        }
        return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
      };
      // 32 columns stay in registers; more are read twice
      float v[32];
      float mx = -INFINITY;
#pragma unroll 1
      for (int k = 0; k < NC; k += 32) {
        tc::tm_ld32(tm_s + k, v);
        tc::wait_ld();
        finish(v, k);
        mx = fmaxf(mx, largest(v));
      }
      mx *= mul;
      // the reference this tile goes by
      float ref = -INFINITY;
      // (an item's first tile waits too: the groups keep in step, neither can be
      // two phases ahead of the other's wait)
      if (n > 0 && !wait_warp(settled(wg ^ 1u, wq), ((n - 1u) >> 1) & 1u)) break;
      if (post.nth > 0) ref = keep->ref[row];
      const bool grow = mx > ref + GROWTH || (ref == -INFINITY && mx > -INFINITY);
      if (__any_sync(0xffffffffu, grow)) {
        const float to = grow ? mx : ref;
        if (post.nth > 0) {
          // O is complete up to tile n - 1, and P(n) V(n) waits for this P
          if (!wait_warp(pv_done((n - 1u) % 3u), ((n - 1u) / 3u) & 1u)) break;
          tc::fence_after();
          const float f = ref == to ? 1.0f : tc::ex2(ref - to);
#pragma unroll 1
          for (int k = 0; k < D; k += 16) {
            uint32_t u[16];
            tc::tm_ld16(tmem + lanes + TM_O + k, u);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
            tc::tm_st16(tmem + lanes + TM_O + k, u);
          }
          tc::wait_st();
        }
        ref = to;
        keep->ref[row] = ref;
      } else if (post.nth == 0) {
        keep->ref[row] = ref;
      }
      __syncwarp();
      if (lane == 0) tc::bar_arrive(settled(wg, wq));
      if (own != ref) {
        // (with no finite maximum yet, l is 0, or NaN where all scores so far were:
        // fmaxf drops them, and the sum has to keep them)
        if (own != -INFINITY) l *= tc::ex2(own - ref);
        own = ref;
      }
      const float zero = ref == -INFINITY ? 0.0f : ref + SMALLER;
      const uint64_t mul2 = tc::pack2(mul, mul), zero2 = tc::pack2(-zero, -zero);
      uint64_t l2 = 0ull;
      auto weigh = [&](const float (&x)[32], int at) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float p0, p1;
          tc::unpack2(tc::fma2(tc::pack2(x[2 * i], x[2 * i + 1]), mul2, zero2), &p0, &p1);
          p0 = tc::ex2(p0);
          p1 = tc::ex2(p1);
          l2 = tc::add2(l2, tc::pack2(p0, p1));
          u[i] = tc::pack16<BF16>(p0, p1);
        }
        tc::tm_st16(tm_p + (col0 + at) / 2, u);
      };
#pragma unroll 1
      for (int k = 0; k < NC; k += 32) {
        if (NC > 32) {
          tc::tm_ld32(tm_s + k, v);
          tc::wait_ld();
          finish(v, k);
        }
        weigh(v, k);
      }
      if (COPIES > 1) {
        // P of the other copies' keys is zero (over columns that were S)
        uint32_t z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll 1
        for (uint32_t k = 0; k < KT / 2; k += 16)
          if (k < col0 / 2 || k >= (col0 + NC) / 2) tc::tm_st16(tm_p + k, z);
      }
      float l0, l1;
      tc::unpack2(l2, &l0, &l1);
      l += l0 + l1;
      keep->sum[wg][row] = l;
      keep->by[wg][row] = own;
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(p_full(b));
    }
  } else if (warp < 16) {
    // -------------------------------------------------------------- gather
    tc::regs_down<REGS_GATHER>();
    // warps 8..11 the keys, 12..15 the values: V(n) waits for a place until
    // P(n - SLOTS) V is done, and K(n + 1) must not wait behind it
    const uint32_t gt = tid & 127u, kv = (warp - 8u) >> 2;
    const void* src = kv ? a.v : a.k;
    const int32_t row_bytes = (int32_t)(kv ? a.v_ts : a.k_ts);
    const int64_t head_bytes = kv ? a.v_hs : a.k_hs;
    uint32_t ti = 0, seq = 0;
    bool ok = true;
    for (int32_t item = first; item < a.items && ok; item += step) {
      const int32_t hk = item % a.Hk;
      for (;;) {
        const uint32_t is = ti % NI;
        if (!wait_warp(ix_full(is), (ti / NI) & 1u)) { ok = false; break; }
        const Tile* tile = tiles + is;
        const int32_t last = tile->last;
        if (tile->count > 0) {
          const uint32_t s = kv * P::SLOTS + seq % P::SLOTS;
          if (!wait_warp(kv_empty(s), ((seq / P::SLOTS) & 1u) ^ 1u)) { ok = false; break; }
          gather_rows<D, GATHER>(base + P::OFF_KV + s * P::TILE, src, row_bytes, head_bytes * hk,
                                 tile, gt);
          tc::cp_arrive(kv_full(s));
          ++seq;
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(ix_empty(is));
        ++ti;
        if (last) break;
      }
    }
    // nothing of this thread is in flight when it leaves
    tc::cp_commit();
    tc::cp_wait<0>();
  } else if (warp < 20) {
    // ------------------------------------------------------- finished items
    tc::regs_up<REGS_END>();
    const uint32_t wq = warp & 3u, row = wq * 32u + lane, copy = row / PER, h = row % PER;
    const uint32_t lanes = (wq * 32u) << 16;
    float* ml = reinterpret_cast<float*>(sm + P::OFF_ML);
    float* wt = reinterpret_cast<float*>(sm + P::OFF_WT);
    uint32_t phase = 0, met = 0, nd = 0, with = 0;  // join phases, meetings, items, items with tiles
    // these four warps meet, and with those of the cluster (waits are bounded)
    auto here = [&]() {
      __syncwarp();
      if (lane == 0) tc::bar_arrive(meet);
      return wait_warp(meet, met++ & 1u);
    };
    auto all = [&]() {
      __syncwarp();
      if (lane < C) tc::bar_arrive_remote(join, lane);
      return __all_sync(0xffffffffu, tc::bar_wait<true>(join, phase++ & 1u, abort, &g_status,
                                                        TOPK_FLAG_TIMEOUT)) != 0;
    };
    bool ok = true;
    if (first < a.items) {
      // these warps have time now: the first item's query heads
      const int32_t t = first / a.Hk, hk = first - t * a.Hk;
      clear_heads<D, 128>(sm + P::OFF_Q, a.G, PER, tid & 127u);
      clear_heads<D, 128>(sm + P::OFF_Q + P::TILE, a.G, PER, tid & 127u);
      load_heads<D, 128>(base + P::OFF_Q, a.q, t * a.q_ts, a.q_hs, hk * a.G, a.G, PER, tid & 127u);
      tc::cp_commit();
      tc::cp_wait<0>();
      tc::fence_async_shared();
      ok = here();
      if (ok && warp == 16 && lane == 0) tc::bar_arrive(q_full(0));
    }
    for (int32_t item = first; item < a.items && ok; item += step, ++nd) {
      const int32_t t = item / a.Hk, hk = item - t * a.Hk;
      if (!wait_warp(o_full, nd & 1u)) break;
      tc::fence_after();
      const Done done = *done_post;
      // the row's maximum and its sum over both groups
      float m = -INFINITY, l = 0.0f;
      if (done.tiles > 0) {
        const Rows* keep = kept + with % NM;
        ++with;
        m = keep->ref[row];
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (done.tiles > 1 || g == done.first) {
            const float by = keep->by[g][row];
            l += by == -INFINITY ? keep->sum[g][row] : keep->sum[g][row] * tc::ex2(by - m);
          }
      }
      if (C == 1) {
        // the whole row into registers: O is free after a few hundred cycles, and
        // the next item's P V need not wait for this one's stores
        float o[D];
        if (done.tiles > 0) {
#pragma unroll
          for (int k = 0; k < D; k += 16) tc::tm_ld16f(tmem + lanes + TM_O + k, o + k);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < D; ++k) o[k] = 0.0f;
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(o_empty);
        float mh = m, lh = l;
        if (COPIES > 1) {
          wt[row] = m;
          wt[128 + row] = l;
          if (!here()) break;
#pragma unroll
          for (int k = 0; k < COPIES; ++k) mh = fmaxf(mh, wt[k * PER + h]);
        }
        const float zero = mh == -INFINITY ? 0.0f : mh;
        if (COPIES > 1) {
          lh = 0.0f;
#pragma unroll
          for (int k = 0; k < COPIES; ++k)
            lh += wt[128 + k * PER + h] * tc::ex2(wt[k * PER + h] - zero);
        }
        const float f = lh != 0.0f ? tc::ex2(m - zero) / lh : 0.0f;  // NaN stays NaN
#pragma unroll
        for (int k = 0; k < D; ++k) o[k] *= f;
        if (COPIES > 1) {
          // the other copies' rows through shared memory, 32 columns at a time
#pragma unroll
          for (int part = 0; part < D / 32; ++part) {
            if (part > 0 && !here()) { ok = false; break; }
            if (copy > 0) {
              float* mine = reinterpret_cast<float*>(sm + P::OFF_STAGE) + (row - PER) * 32;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(mine + (((i >> 2) ^ (row & 7u)) << 2)) =
                    make_float4(o[part * 32 + i], o[part * 32 + i + 1], o[part * 32 + i + 2],
                                o[part * 32 + i + 3]);
            }
            if (!here()) { ok = false; break; }
            if (copy == 0) {
#pragma unroll
              for (int k = 1; k < COPIES; ++k) {
                const float* theirs =
                    reinterpret_cast<const float*>(sm + P::OFF_STAGE) + ((k - 1) * PER + h) * 32;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float4 x =
                      *reinterpret_cast<const float4*>(theirs + (((i >> 2) ^ (h & 7u)) << 2));
                  o[part * 32 + i] += x.x;
                  o[part * 32 + i + 1] += x.y;
                  o[part * 32 + i + 2] += x.z;
                  o[part * 32 + i + 3] += x.w;
                }
              }
            }
          }
          if (!ok) break;
        }
        bool odd = false;  // something is not finite although the sum is
        uint16_t* mine = static_cast<uint16_t*>(a.out) + ((int64_t)t * a.H + hk * a.G + h) * D;
        if (copy == 0 && (int32_t)h < a.G) {
          uint4* dst = reinterpret_cast<uint4*>(mine);
          uint64_t none2 = 0ull;
#pragma unroll
          for (int k = 0; k < D; k += 8) {
            dst[k / 8] = make_uint4(
                tc::pack16<BF16>(o[k], o[k + 1]), tc::pack16<BF16>(o[k + 2], o[k + 3]),
                tc::pack16<BF16>(o[k + 4], o[k + 5]), tc::pack16<BF16>(o[k + 6], o[k + 7]));
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              none2 = tc::fma2(tc::pack2(o[k + i], o[k + i + 1]), 0ull, none2);
          }
          if (a.lse)
            a.lse[(int64_t)t * a.H + hk * a.G + h] =
                lh != 0.0f ? (zero + SMALLER + log2f(lh)) * 0.6931471805599453f : -INFINITY;
          float n0, n1;
          tc::unpack2(none2, &n0, &n1);
          odd = n0 + n1 != 0.0f && lh == lh;
        }
        if (__any_sync(0xffffffffu, odd)) {
          asm volatile("" ::: "memory");  // the row is read back
          look_up_rows<D, BF16>(&a, t, hk, lane, mine, odd, lh == 0.0f);
        }
        continue;
      }
      // a cluster's item.  The copies of a head first, within the CTA: its maximum and
      // sum, and the factor of this row (the weights' table is free until they meet)
      wt[row] = m;
      wt[128 + row] = l;
      if (!here()) break;
      float scale_row;
      {
        float mh = -INFINITY, lh = 0.0f;
#pragma unroll
        for (int k = 0; k < COPIES; ++k) mh = fmaxf(mh, wt[k * PER + h]);
        const float zero = mh == -INFINITY ? 0.0f : mh;
#pragma unroll
        for (int k = 0; k < COPIES; ++k) lh += wt[128 + k * PER + h] * tc::ex2(wt[k * PER + h] - zero);
        scale_row = tc::ex2(wt[row] - zero);
        if (copy == 0) {
          ml[h] = mh;
          ml[128 + h] = lh;
        }
      }
      // 32 columns of the accumulator at a time: [128 rows][32] floats, 16-byte
      // pieces of row r at p ^ (r & 7) (stores of 8 rows then hit 8 bank groups).
      // The CTA's last item has the K and V rings to itself: all columns at once,
      // one meeting of the cluster instead of two for every 32.
      const bool spare = item + step >= a.items;
      const uint32_t to = spare ? P::OFF_KV : P::OFF_STAGE, stride = spare ? 128u * 32u * 4u : 0u;
#pragma unroll 1
      for (uint32_t part = 0; part < (uint32_t)D / 32u; ++part) {
        {
          float o[32];
          if (done.tiles > 0) {
            tc::tm_ld32(tmem + lanes + TM_O + part * 32u, o);
            tc::wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.0f;
          }
          float* mine = reinterpret_cast<float*>(sm + to + part * stride) + row * 32;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(mine + (((i >> 2) ^ (row & 7u)) << 2)) =
                make_float4(o[i] * scale_row, o[i + 1] * scale_row, o[i + 2] * scale_row,
                            o[i + 3] * scale_row);
        }
        if (part == D / 32u - 1u) {
          // O and the post may be replaced
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(o_empty);
        } else if (spare) {
          continue;
        }
        if (!all()) { ok = false; break; }  // everybody's rows are staged
        if (spare || part == 0) {
          // weights of the CTAs' results of head h: 2^(m - max) / sum
          float mc[8], lc[8], mm = -INFINITY, sum = 0.0f;
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c) {
            mc[c] = -INFINITY;
            lc[c] = 0.0f;
            if (c < C) {
              mc[c] = tc::ld_remote(base + P::OFF_ML + 4u * h, c);
              lc[c] = tc::ld_remote(base + P::OFF_ML + 4u * (128u + h), c);
            }
          }
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c) mm = fmaxf(mm, mc[c]);
          const float zero = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c) {
            mc[c] = tc::ex2(mc[c] - zero);
            sum += lc[c] * mc[c];
          }
          const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;  // NaN stays NaN
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c)
            if (c < C && copy == 0) wt[c * 128 + h] = mc[c] * inv;
          if (a.lse && rank == 0 && copy == 0 && (int32_t)h < a.G)
            a.lse[(int64_t)t * a.H + hk * a.G + h] =
                sum != 0.0f ? (zero + SMALLER + log2f(sum)) * 0.6931471805599453f : -INFINITY;
          if (!here()) { ok = false; break; }
        }
        // the joined rows, 4 elements per thread and step
#pragma unroll 1
        for (uint32_t q = spare ? 0u : part; q <= part; ++q) {
          float none = 0.0f;
#pragma unroll 1
          for (uint32_t e = rank * 128u + (tid & 127u); e < (uint32_t)a.G * 8u; e += C * 128u) {
            const uint32_t hh = e >> 3, p = e & 7u;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (uint32_t c = 0; c < C; ++c) {
              const float f = wt[c * 128 + hh];
#pragma unroll
              for (int k = 0; k < COPIES; ++k) {
                const uint32_t r = k * PER + hh;
                const uint32_t at = to + q * stride + (r * 32 + ((p ^ (r & 7u)) << 2)) * 4u;
                const float4 y = tc::ld_remote4(base + at, c);
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
              }
            }
            uint2 w;
            w.x = tc::pack16<BF16>(x.x, x.y);
            w.y = tc::pack16<BF16>(x.z, x.w);
            uint16_t* dst = static_cast<uint16_t*>(a.out) +
                            ((int64_t)t * a.H + hk * a.G + hh) * D + q * 32 + p * 4;
            *reinterpret_cast<uint2*>(dst) = w;
            none = fmaf(x.x, 0.0f, fmaf(x.y, 0.0f, fmaf(x.z, 0.0f, fmaf(x.w, 0.0f, none))));
          }
          if (__any_sync(0xffffffffu, none != 0.0f)) {
            asm volatile("" ::: "memory");  // the elements are read back
            uint32_t kinds[3];
            value_kinds<BF16>(a, t, hk, q * 32u, lane, kinds);
#pragma unroll 1
            for (uint32_t e = rank * 128u + (tid & 127u); e < (uint32_t)a.G * 8u; e += C * 128u) {
              const uint32_t hh = e >> 3, p = e & 7u;
              float sum = 0.0f;
              for (uint32_t c = 0; c < C; ++c) sum += wt[c * 128 + hh];
              if (sum != sum) continue;
              uint16_t* dst = static_cast<uint16_t*>(a.out) +
                              ((int64_t)t * a.H + hk * a.G + hh) * D + q * 32 + p * 4;
#pragma unroll 1
              for (uint32_t i = 0; i < 4; ++i)
                dst[i] = looked_up<BF16>(dst[i], kinds, p * 4 + i, sum == 0.0f);
            }
          }
        }
        // everybody has read the rows (the last ones stay until the cluster leaves)
        if (!spare && !all()) { ok = false; break; }
      }
    }
  } else {
    tc::regs_down<REGS_REST>();
    if (warp == 20) {
      // ------------------------------------------- tensor core: S = Q K^T
      constexpr uint32_t id_s = tc::idesc(BF16, 128, KT, false, false);
      const uint32_t lead = tc::elect_lane();
      uint32_t ti = 0, n = 0, nq = 0;
      int32_t with = 0;  // items with tiles
      bool ok = true;
      for (int32_t item = first; item < a.items && ok; item += step) {
        uint32_t nth = 0;
        const uint32_t qb = nq & 1u, qa = base + P::OFF_Q + qb * P::TILE;
        if (!wait_warp(q_full(qb), (nq >> 1) & 1u)) break;
        ++nq;
        for (;;) {
          const uint32_t is = ti % NI;
          if (!wait_warp(ix_full(is), (ti / NI) & 1u)) { ok = false; break; }
          const int32_t count = tiles[is].count, last = tiles[is].last;
          ++ti;
          if (count > 0) {
            // buffer b held P(n - 3)
            const uint32_t u = n / 3u, b = n - 3u * u, s = n % P::SLOTS;
            if (!wait_both(kv_full(s), (n / P::SLOTS) & 1u, pv_done(b), (u & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              posts[b] = Post{count, (int32_t)is, (int32_t)nth, with};
              tc::bar_arrive(s_full(b));
            }
            __syncwarp();
            tc::fence_async_shared();  // the gathered rows, for the tensor core
            tc::fence_after();
            const uint32_t kb = base + P::OFF_KV + s * P::TILE;
#pragma unroll
            for (uint32_t kk = 0; kk < D / 16; ++kk)
              tc::mma_ss(tmem + b * 128u, tc::desc_k(qa, P::BLOCK, kk),
                         tc::desc_k(kb, P::BLOCK, kk), id_s, kk > 0, lead);
            tc::mma_commit(s_full(b), lead);
            tc::mma_commit(kv_empty(s), lead);
            if (last) tc::mma_commit(q_empty(qb), lead);
            ++nth;
            ++n;
          } else {
            __syncwarp();
            if (lane == 0) {
              tc::bar_arrive(ix_empty(is));
              tc::bar_arrive(q_empty(qb));  // no tile: the heads' rows were not needed
            }
          }
          if (last) {
            if (nth > 0) ++with;
            break;
          }
        }
      }
      // the softmax groups leave
      for (uint32_t k = 0; k < 2 && ok; ++k) {
        const uint32_t u = (n + k) / 3u, b = n + k - 3u * u;
        if (!wait_warp(pv_done(b), (u & 1u) ^ 1u)) break;
        if (lane == 0) {
          posts[b].count = 0;
          tc::bar_arrive(s_full(b));
          tc::bar_arrive(s_full(b));
        }
      }
      // what was issued has completed before tensor memory is released
      if (n > 0) {
        tc::mma_commit(drain, lead);
        tc::bar_drain(drain, 0u);
      }
    } else if (warp == 23) {
      // ------------------------------------------------ tensor core: P V
      constexpr uint32_t id_o = tc::idesc(BF16, 128, D, false, true);
      const uint32_t lead = tc::elect_lane();
      uint32_t ti = 0, n = 0, no = 0;  // index tiles, tiles, items
      bool ok = true;
      for (int32_t item = first; item < a.items && ok; item += step, ++no) {
        uint32_t nth = 0;
        for (;;) {
          const uint32_t is = ti % NI;
          if (!wait_warp(ix_full(is), (ti / NI) & 1u)) { ok = false; break; }
          const int32_t count = tiles[is].count, last = tiles[is].last;
          ++ti;
          // the item before has been read
          if (nth == 0 && !wait_warp(o_empty, (no & 1u) ^ 1u)) { ok = false; break; }
          if (count > 0) {
            const uint32_t u = n / 3u, b = n - 3u * u, s = P::SLOTS + n % P::SLOTS;
            if (!wait_both(p_full(b), u & 1u, kv_full(s), (n / P::SLOTS) & 1u)) {
              ok = false;
              break;
            }
            tc::fence_async_shared();
            tc::fence_after();
            const uint32_t vb = base + P::OFF_KV + s * P::TILE;
#pragma unroll
            for (uint32_t kk = 0; kk < KT / 16; ++kk)
              tc::mma_ts(tmem + TM_O, tmem + b * 128u + kk * 8, tc::desc_mn(vb, P::BLOCK, kk),
                         id_o, nth > 0 || kk > 0, lead);
            tc::mma_commit(pv_done(b), lead);
            tc::mma_commit(kv_empty(s), lead);
            if (last) tc::mma_commit(o_full, lead);
            ++nth;
            ++n;
          } else if (lane == 0) {
            tc::bar_arrive(o_full);  // an item without a tile
          }
          __syncwarp();
          if (lane == 0) {
            // P is there: the softmax and the other tensor-core warp have read the tile
            tc::bar_arrive_n(ix_empty(is), count > 0 ? 2u : 1u);
            if (last) {
              done_post->tiles = (int32_t)nth;
              done_post->first = (int32_t)((n - nth) & 1u);
              tc::bar_arrive(o_full);
            }
          }
          if (last) break;
        }
      }
      if (n > 0) {
        tc::mma_commit(drain2, lead);
        tc::bar_drain(drain2, 0u);
      }
    } else if (warp == 21) {
      // --------------------------------------------------------- index rows
      uint32_t ti = 0;
      compact_rows(
          a, first, step, (int32_t)rank, (int32_t)C, lane, [](int32_t, int32_t hk) { return hk; },
          [&]() -> Tile* {
            return wait_warp(ix_empty(ti % NI), ((ti / NI) & 1u) ^ 1u) ? tiles + ti % NI : nullptr;
          },
          [&]() {
            __syncwarp();
            if (lane == 0) tc::bar_arrive(ix_full(ti % NI));
            ++ti;
          });
    } else if (warp == 22) {
      // ----------------------------------------- the items' query head rows
      uint32_t nq = 1;  // the first item's are not this warp's
      for (int32_t item = first + step; item < a.items; item += step, ++nq) {
        const int32_t t = item / a.Hk, hk = item - t * a.Hk;
        const uint32_t qb = nq & 1u;
        if (!wait_warp(q_empty(qb), ((nq >> 1) & 1u) ^ 1u)) break;
        load_heads<D, 32>(base + P::OFF_Q + qb * P::TILE, a.q, t * a.q_ts, a.q_hs, hk * a.G, a.G,
                          PER, lane);
        tc::cp_commit();
        tc::cp_wait<0>();
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(q_full(qb));
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == 20) {
    tc::fence_after();
    tc::tm_free(tmem, TMEM_COLS);
  }
  if (C > 1) tc::cluster_sync();  // nobody leaves while its rows are read
}

// ------------------------------------------------------------------ host side
int device_sms(int* sms) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TOPK_ERR_NO_DEVICE;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return TOPK_ERR_CUDA;
  return major == 10 && minor == 3 ? TOPK_OK : TOPK_ERR_NO_DEVICE;
}

int check_args(const Args& a, int32_t D, int32_t dtype) {
  if (a.T < 0 || a.H < 1 || a.Hk < 1 || a.K < 1 || a.S < 0 || (a.ld_idx < a.K && a.ld_idx != 0) ||
      (int64_t)a.T * a.H > INT32_MAX || !(a.scale > 0.0f) || !std::isfinite(a.scale) ||
      !std::isfinite(a.cap) || a.k_ts < 0 || a.k_ts > INT32_MAX || a.v_ts < 0 ||
      a.v_ts > INT32_MAX)
    return TOPK_ERR_ARG;
  if (a.H % a.Hk != 0 || a.H / a.Hk > 128 || (D != 64 && D != 128) ||
      (dtype != TOPK_BF16 && dtype != TOPK_FP16))
    return TOPK_ERR_UNSUPPORTED_SHAPE;
  if (a.T == 0) return TOPK_OK;
  if (!a.q || !a.idx || (a.S > 0 && (!a.k || !a.v)) || (a.slopes && !a.pos)) return TOPK_ERR_ARG;
  auto off = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (off(a.q, 16) || off(a.k, 16) || off(a.v, 16) ||
      ((a.q_ts | a.q_hs | a.k_ts | a.k_hs | a.v_ts | a.v_hs) & 15) || off(a.idx, 4) ||
      off(a.slopes, 4) || off(a.pos, 4) || off(a.lo, 4) || off(a.hi, 4))
    return TOPK_ERR_ALIGN;
  return TOPK_OK;
}

template <int D, int NC, bool BF16, int BENT>
int launch_kernel(const Args& a, int C, int sms, cudaStream_t st) {
  static OncePerDevice opted_in;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TOPK_ERR_NO_DEVICE;
  if (!opted_in.ensure(dev, [] {
        return cudaFuncSetAttribute(k_attend<D, NC, BF16, BENT>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)Plan<D>::BYTES) == cudaSuccess;
      }))
    return TOPK_ERR_CUDA;
  const int clusters = a.items < sms / C ? a.items : sms / C;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Plan<D>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attend<D, NC, BF16, BENT>, a) == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA;
}

template <int D, bool BF16, int BENT>
int launch_rows(const Args& a, int C, int sms, cudaStream_t st) {
  if (a.G <= 32) return launch_kernel<D, 32, BF16, BENT>(a, C, sms, st);
  if (a.G <= 64) return launch_kernel<D, 64, BF16, BENT>(a, C, sms, st);
  return launch_kernel<D, 128, BF16, BENT>(a, C, sms, st);
}

template <int D, bool BF16>
int launch_bent(const Args& a, int C, int sms, cudaStream_t st) {
  return a.cap > WIDE_CAP              ? launch_rows<D, BF16, 2>(a, C, sms, st)
         : a.cap > 0.0f || a.slopes ? launch_rows<D, BF16, 1>(a, C, sms, st)
                                    : launch_rows<D, BF16, 0>(a, C, sms, st);
}

// CTAs per item: the split with the least rounds of (chunks + one for the
// prologue and the join) over the SMs.
int cluster_size(int64_t items, int chunks, int sms) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int c = 1; c <= 8 && c <= chunks; c *= 2) {
    const int64_t rounds = (items + sms / c - 1) / (sms / c);
    const int64_t cost = rounds * ((chunks + c - 1) / c + (c > 1 ? 2 : 1));
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return best;
}

}  // namespace ta

extern "C" {

int topk_sparse_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                          const void* k, int64_t k_token_stride, int64_t k_head_stride,
                          const void* v, int64_t v_token_stride, int64_t v_head_stride,
                          const int32_t* idx, int64_t ld_idx, int64_t T, int64_t S, int32_t H,
                          int32_t Hk, int32_t D, int32_t K, int32_t dtype, float scale,
                          float softcap, const float* slopes, const int32_t* positions,
                          const int32_t* key_lo, const int32_t* key_hi, void* out, float* lse,
                          struct CUstream_st* stream) {
  if (T < 0 || T > INT32_MAX || S < 0 || S > INT32_MAX) return TOPK_ERR_ARG;
  ta::Args a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.idx = idx;
  a.slopes = slopes;
  a.pos = positions;
  a.lo = key_lo;
  a.hi = key_hi;
  a.q_ts = 2 * q_token_stride;
  a.q_hs = 2 * q_head_stride;
  a.k_ts = 2 * k_token_stride;
  a.k_hs = 2 * k_head_stride;
  a.v_ts = 2 * v_token_stride;
  a.v_hs = 2 * v_head_stride;
  a.ld_idx = ld_idx;
  a.T = (int32_t)T;
  a.S = (int32_t)S;
  a.H = H;
  a.Hk = Hk;
  a.K = K;
  a.scale = scale;
  a.cap = softcap;
  a.out = out;
  a.lse = lse;
  int rc = ta::check_args(a, D, dtype);
  if (rc != TOPK_OK || T == 0) return rc;
  if (!out) return TOPK_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(out) & 15u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return TOPK_ERR_ALIGN;
  a.G = H / Hk;
  a.chunks = (int32_t)(((int64_t)K + ta::KT - 1) / ta::KT);
  a.items = a.T * Hk;
  int sms = 0;
  rc = ta::device_sms(&sms);
  if (rc != TOPK_OK) return rc;
  const int C = ta::cluster_size(a.items, a.chunks, sms);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TOPK_BF16)
    return D == 64 ? ta::launch_bent<64, true>(a, C, sms, st) : ta::launch_bent<128, true>(a, C, sms, st);
  return D == 64 ? ta::launch_bent<64, false>(a, C, sms, st) : ta::launch_bent<128, false>(a, C, sms, st);
}

int topk_sparse_attention_read_status(struct CUstream_st* stream, uint32_t* flags) {
  if (!flags) return TOPK_ERR_ARG;
  uint32_t h = 0, g = 0, zero = 0;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyFromSymbolAsync(&h, ta::g_status, sizeof h, 0, cudaMemcpyDeviceToHost, st) !=
          cudaSuccess ||
      cudaMemcpyToSymbolAsync(ta::g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st) !=
          cudaSuccess)
    return TOPK_ERR_CUDA;
  const int rc = ta::take_status_grad(st, &g);  // synchronises the stream
  if (rc != TOPK_OK) return rc;
  *flags = h | g;
  return TOPK_OK;
}

}  // extern "C"
