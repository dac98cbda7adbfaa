// Gradients of the attention over selected keys.
//
//   p_j = exp(z_j - lse_h), dp_j = dout_h . v[i_j], delta_h = dout_h . out_h
//   ds_j = p_j (dp_j - delta_h) (1 - (cap part / cap)^2)
//   dq_h = scale sum_j ds_j k[i_j];  dk[i_j] += scale ds_j q_h;  dv[i_j] += p_j dout_h
// (z as in the forward pass; an entry that is masked there is skipped here).
//
// An item is one token and one key head, as in the forward kernel, with the
// same repeated head rows and tiles of 128 gathered keys.  A tile takes five
// products: S = Q K^T and dP = dO V^T (rows: heads), then, from P and dS
// rounded to the 16-bit type in shared memory, dQ += dS K (rows: heads) and
// dV = P^T dO, dK = dS^T Q (rows: the tile's keys).  P and dS are written once,
// [head][key]; the last two read the same bytes transposed.
//
// Keys are shared by many tokens, so dK and dV are summed in FP32 buffers with
// vector reductions to global memory: 8 D bytes per token, key and key head,
// against 4 D gathered.  Those bound the kernel, not the tensor core: on GB300 a
// kernel that does nothing else reaches 6.3 TB/s of reductions into 8 MB (L2), and
// this one 4.4-4.5 (1024 queries x 64 heads x 128, Top-2048 of 8192: 492 us, of
// them 341 us at that rate).  Without the reductions a tile takes 6700 cycles
// instead of 8400, without their way through tensor and shared memory 6000.  Their
// order is the scheduler's, so the sums differ by FP32 rounding between runs.
// P and dS are rounded to the inputs' 16-bit type before the last three products
// (the tensor core takes no wider operand beside 16-bit values; the error against
// 64 bits is 1.1 to 1.3 times that of FP32 products).  dS leaves the scale out until
// the FP32 results, and in FP16 it is held times a power of two that brings the
// item's largest |dout| into [4, 8) and is taken out of those results, exactly: with a
// scaled loss dS itself passes 65504 where dq, dk and dv do not.  8 (|v|_1 + |out|_1)
// bounds it then: finite for values whose absolute sum over D is below 4094.
//
// Tried and slower: twice the draining warps (8900 cycles a tile), dV and dK in
// halves of 64 columns with S and dP ahead of them (9400), bulk reductions of
// staged rows (one row in flight per thread is 2.7 TB/s, and shared memory has no
// room for four).
//
// One CTA per SM, persistent over items.  Warps:
//   0..3   P and dS from S and dP
//   4..7   dV and dK tiles from tensor memory to the sums (transposed through
//          shared memory to whole 128-byte lines), and the items' dQ
//   8..11  gather of keys, 12..15 of values
//   16     tensor core; 17 index rows; 18 the items' q and dout heads
// Tensor memory: three rotating buffers of 128 columns and dQ.  S(n) and dP(n)
// take the next two; once P and dS are written, dV(n) and dK(n) replace them.
#include "per_device.h"
#include "sparse_attend.cuh"

namespace ta {

constexpr int G_THREADS = 640;
constexpr int G_GATHER = 128;
constexpr int R_SOFT = 128, R_DRAIN = 112, R_GATHER = 72, R_REST = 80;
static_assert(R_SOFT + R_DRAIN + 2 * R_GATHER + R_REST <= 5 * 96, "register split");
constexpr int G_NI = 4;
constexpr uint32_t G_TMEM = 512, TM_DQ = 384;

template <int D>
struct GradPlan {
  static constexpr uint32_t BLOCK = KT * 128;
  static constexpr uint32_t TILE = BLOCK * (D / 64);
  static constexpr uint32_t SLOTS = D == 128 ? 1 : 2;
  static constexpr uint32_t OFF_Q = 0, OFF_DO = TILE, OFF_K = 2 * TILE;
  static constexpr uint32_t OFF_V = OFF_K + SLOTS * TILE;
  static constexpr uint32_t OFF_P = OFF_V + SLOTS * TILE;   // [128 heads][128 keys]
  static constexpr uint32_t OFF_DS = OFF_P + 2 * BLOCK;
  static constexpr uint32_t OFF_STAGE = OFF_DS + 2 * BLOCK;  // [128][32] floats, swizzled
  static constexpr uint32_t OFF_IDX = OFF_STAGE + 128 * 32 * 4;
  static constexpr uint32_t OFF_BAR = OFF_IDX + G_NI * sizeof(Tile);
  static constexpr uint32_t NBAR = 4 * SLOTS + 2 * G_NI + 3 + 6 + 4 + 2;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t BYTES = OFF_MISC + 64 + 1024;
};
static_assert(GradPlan<128>::BYTES <= 232448 && GradPlan<64>::BYTES <= 232448, "shared memory plan");

__device__ __forceinline__ void red4(float* p, float4 v) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// Infinite output gradients.  P is zero in the other copies' keys, and 0 * inf makes
// their part of dV NaN, where p * inf is that infinity.  So NaN in four neighbouring
// columns (from col on) of dV of token t, key head hk is looked up in the heads' dout:
// NaN or both signs there, it stays; else it is the infinity.  A head without a key
// (lse = -inf) takes no part; where a head's weights are NaN (lse is not finite) all
// stays.  Bits 0..3, 4..7: which columns become +inf, -inf.
template <bool BF16>
__device__ __forceinline__ uint32_t infinite_columns(const Args& a, int32_t t, int32_t hk,
                                                     uint32_t col) {
  constexpr uint32_t INF = BF16 ? 0x7f80u : 0x7c00u;
  uint32_t nan = 0u, pos = 0u, neg = 0u;
#pragma unroll 1
  for (int32_t h = hk * a.G; h < (hk + 1) * a.G; ++h) {
    const float lse = a.lse_in[(int64_t)t * a.H + h];
    if (lse == -INFINITY) continue;
    if (!(fabsf(lse) < INFINITY)) return 0u;
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.dout) +
                                                    t * a.do_ts + h * a.do_hs + col * 2u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = i < 2 ? w.x : w.y, x = i & 1 ? two >> 16 : two & 0xffffu;
      nan |= (uint32_t)((x & 0x7fffu) > INF) << i;
      pos |= (uint32_t)(x == INF) << i;
      neg |= (uint32_t)(x == (0x8000u | INF)) << i;
    }
  }
  return (pos & ~neg & ~nan) | (neg & ~pos & ~nan) << 4;
}
// The staged rows of a chunk of dV to the sums, such NaN replaced.  Not inlined: any
// code among the usual rows' loads and reductions costs them (568 us for 490 with
// 1024 x 64 heads x 128), although it never runs.
template <int D, bool BF16>
__device__ __noinline__ void add_odd_rows(const Args* a, int32_t t, int32_t hk, uint32_t c,
                                          uint32_t wq, uint32_t lane, const Tile* tile,
                                          const float* stage, float* sum) {
  const int64_t key_floats = (int64_t)a->Hk * D;
  const uint32_t inf = infinite_columns<BF16>(*a, t, hk, c + (lane & 7u) * 4u);
  auto put = [&](float& v, uint32_t i) {
    if (v != v && (inf >> i & 1u)) v = INFINITY;
    if (v != v && (inf >> (4 + i) & 1u)) v = -INFINITY;
  };
#pragma unroll 1
  for (uint32_t r = wq * 32u + (lane >> 3); r < wq * 32u + 32u; r += 4) {
    float4 x = *reinterpret_cast<const float4*>(stage + r * 32 + (((lane & 7u) ^ (r & 7u)) << 2));
    put(x.x, 0);
    put(x.y, 1);
    put(x.z, 2);
    put(x.w, 3);
    if ((int32_t)r < tile->count) red4(sum + tile->key[r] * key_floats, x);
  }
}

// One warp: the power of two that brings the largest |dout| of an item into [4, 8)
// (1 where there is none, or one that is not finite), as the bits of a float.
template <int D>
__device__ __forceinline__ int32_t factor_bits(const Args& a, int32_t t, int32_t hk, uint32_t lane) {
  constexpr uint32_t PIECES = D / 8;
  const uint8_t* src = static_cast<const uint8_t*>(a.dout) + t * a.do_ts + (int64_t)hk * a.G * a.do_hs;
  uint32_t top = 0u;  // largest magnitudes of the even and the odd elements
#pragma unroll 8
  for (uint32_t e = lane; e < (uint32_t)a.G * PIECES; e += 32) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src + (e / PIECES) * a.do_hs + e % PIECES * 16));
    top = __vmaxu2(__vmaxu2(top, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu)),
                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  }
  const uint32_t m = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  if (m == 0u || m >= 0x7c00u) return __float_as_int(1.0f);
  const int32_t exponent = (__float_as_int(__half2float(__ushort_as_half((uint16_t)m))) >> 23) - 127;
  return (127 + 2 - exponent) << 23;
}

template <int D, int NC, bool BF16>
__global__ void __launch_bounds__(G_THREADS, 1) k_attend_grad(const __grid_constant__ Args a) {
  using P = GradPlan<D>;
  constexpr int PER = NC, COPIES = 128 / PER;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::saddr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  Tile* tiles = reinterpret_cast<Tile*>(sm + P::OFF_IDX);
  const uint32_t bars = base + P::OFF_BAR;
  auto kv_full = [&](uint32_t s) { return bars + 8u * s; };
  auto kv_empty = [&](uint32_t s) { return bars + 8u * (2 * P::SLOTS + s); };
  auto ix_full = [&](uint32_t s) { return bars + 8u * (4 * P::SLOTS + s); };
  auto ix_empty = [&](uint32_t s) { return bars + 8u * (4 * P::SLOTS + G_NI + s); };
  const uint32_t b0 = bars + 8u * (4 * P::SLOTS + 2 * G_NI);
  const uint32_t s_full = b0, w_full = b0 + 8u, w_empty = b0 + 16u;  // S and dP; P and dS
  auto acc_full = [&](uint32_t b) { return b0 + 24u + 8u * b; };
  auto acc_free = [&](uint32_t b) { return b0 + 48u + 8u * b; };
  const uint32_t q_full = b0 + 72u, q_empty = b0 + 80u, dq_full = b0 + 88u, dq_free = b0 + 96u,
                 last_bar = b0 + 104u, meet = b0 + 112u;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + P::OFF_MISC);
  volatile uint32_t* abort = misc + 1;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  const int32_t first = (int32_t)blockIdx.x, step = (int32_t)gridDim.x;
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu,
                      tc::bar_wait(bar, parity, abort, &g_status, TOPK_FLAG_TIMEOUT)) != 0;
  };

  if (tid == 0) {
    for (uint32_t s = 0; s < 2 * P::SLOTS; ++s) {
      tc::bar_init(kv_full(s), G_GATHER);
      tc::bar_init(kv_empty(s), 1);
    }
    for (uint32_t s = 0; s < G_NI; ++s) {
      tc::bar_init(ix_full(s), 1);
      tc::bar_init(ix_empty(s), 17);  // 8 gather, 4 softmax and 4 draining warps, the MMA warp
    }
    tc::bar_init(s_full, 1);
    tc::bar_init(w_full, 4);
    tc::bar_init(w_empty, 1);
    for (uint32_t b = 0; b < 3; ++b) {
      tc::bar_init(acc_full(b), 1);
      tc::bar_init(acc_free(b), 4);
    }
    tc::bar_init(q_full, 1);
    tc::bar_init(q_empty, 1);
    tc::bar_init(dq_full, 1);
    tc::bar_init(dq_free, 4);
    tc::bar_init(last_bar, 1);
    tc::bar_init(meet, 4);
    *abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tc::tm_alloc(tc::saddr(misc), G_TMEM);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = misc[0];

  if (warp < 4) {
    // ------------------------------------------------------------ P and dS
    tc::regs_up<R_SOFT>();
    const uint32_t row = tid, copy = row / PER, h = row % PER, col0 = copy * NC;
    const uint32_t lanes = (warp * 32u) << 16;
    // the other copies' keys stay zero
    for (uint32_t p = 0; p < 16; ++p) {
      *reinterpret_cast<uint4*>(sm + P::OFF_P + piece_at(row, p, 128u)) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(sm + P::OFF_DS + piece_at(row, p, 128u)) = make_uint4(0, 0, 0, 0);
    }
    const float sc = a.scale * LOG2E;
    const float cap_in = a.cap > 0.0f ? a.scale / a.cap : 0.0f, cap_out = a.cap * LOG2E;
    uint32_t ti = 0, n = 0;
    bool ok = true;
    for (int32_t item = first; item < a.items && ok; item += step) {
      const int32_t t = item / a.Hk, hk = item - t * a.Hk;
      const bool live = (int32_t)h < a.G;
      const int64_t at = (int64_t)t * a.H + hk * a.G + h;
      const float slope = a.slopes && live ? a.slopes[hk * a.G + h] * LOG2E : 0.0f;
      const int32_t pos = a.slopes ? a.pos[t] : 0;
      // p = 0 in rows of no head, and where no key is left or all scores are -inf
      // (lse = -inf: 2^(-inf + inf) would be NaN)
      float lse = live ? a.lse_in[at] * LOG2E : INFINITY;
      if (lse == -INFINITY) lse = INFINITY;
      const float delta = live ? a.delta[at] : 0.0f;
      for (;;) {
        const uint32_t is = ti % G_NI;
        if (!wait_warp(ix_full(is), (ti / G_NI) & 1u)) { ok = false; break; }
        const Tile* tile = tiles + is;
        const int32_t count = tile->count, last = tile->last;
        if (count > 0) {
          if (!wait_warp(s_full, n & 1u) || !wait_warp(w_empty, (n & 1u) ^ 1u)) { ok = false; break; }
          tc::fence_after();
          const uint32_t ts = tmem + lanes + ((2u * n) % 3u) * 128u + col0;
          const uint32_t td = tmem + lanes + ((2u * n + 1u) % 3u) * 128u + col0;
          const float times = BF16 ? 1.0f : __int_as_float(tile->mark), less = -delta * times;
#pragma unroll 1
          for (int c = 0; c < NC; c += 32) {
            float us[32], ud[32];
            tc::tm_ld32(ts + c, us);
            tc::tm_ld32(td + c, ud);
            tc::wait_ld();
            float x[32];
            if (a.cap > WIDE_CAP) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float th = tanh_near(us[i] * cap_in);
                x[i] = cap_out * th;
                ud[i] = fmaf(ud[i], times, less) * fmaf(-th, th, 1.0f);
              }
            } else if (a.cap > 0.0f) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float th = tanh_of(us[i] * cap_in);
                x[i] = cap_out * th;
                // the cap's derivative goes with dP - delta
                ud[i] = fmaf(ud[i], times, less) * fmaf(-th, th, 1.0f);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                x[i] = us[i] * sc;
                ud[i] = fmaf(ud[i], times, less);
              }
            }
            if (a.slopes) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const int4 key = *reinterpret_cast<const int4*>(tile->key + col0 + c + i);
                x[i] -= slope * fabsf((float)(pos - key.x));
                x[i + 1] -= slope * fabsf((float)(pos - key.y));
                x[i + 2] -= slope * fabsf((float)(pos - key.z));
                x[i + 3] -= slope * fabsf((float)(pos - key.w));
              }
            }
            if (count < KT) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((int32_t)(col0 + c + i) >= count) x[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t wp[4], wd[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float p0 = tc::ex2(x[i + 2 * j] - lse), p1 = tc::ex2(x[i + 2 * j + 1] - lse);
                wp[j] = tc::pack16<BF16>(p0, p1);
                wd[j] = tc::pack16<BF16>(p0 * ud[i + 2 * j], p1 * ud[i + 2 * j + 1]);
              }
              const uint32_t to = piece_at(row, (col0 + c + i) / 8, 128u);
              *reinterpret_cast<uint4*>(sm + P::OFF_P + to) = make_uint4(wp[0], wp[1], wp[2], wp[3]);
              *reinterpret_cast<uint4*>(sm + P::OFF_DS + to) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
            }
          }
          tc::fence_before();
          tc::fence_async_shared();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(w_full);
          ++n;
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(ix_empty(is));
        ++ti;
        if (last) break;
      }
    }
  } else if (warp < 8) {
    // --------------------------------------------- dV, dK to the sums, and dQ
    tc::regs_up<R_DRAIN>();
    const uint32_t wq = warp - 4u, row = wq * 32u + lane, lanes = (wq * 32u) << 16;
    float* stage = reinterpret_cast<float*>(sm + P::OFF_STAGE);
    const int64_t key_floats = (int64_t)a.Hk * D;
    uint32_t ti = 0, n = 0, nq = 0, met = 0;
    // the four warps meet (a wait that is bounded, as all are here)
    auto drain_sync = [&]() {
      __syncwarp();
      if (lane == 0) tc::bar_arrive(meet);
      return wait_warp(meet, met++ & 1u);
    };
    bool ok = true;
    for (int32_t item = first; item < a.items && ok; item += step) {
      const int32_t t = item / a.Hk, hk = item - t * a.Hk;
      bool any = false;
      float undo = a.scale;  // dS's factor out of the results, and the scale in
      // an infinite or NaN dout leaves its mark in delta; without one dV needs no look
      // (looking at every row of dV took 615 us for 492 with 1024 x 64 heads x 128)
      bool mark = false;
      for (int32_t h = (int32_t)lane; h < a.G; h += 32)
        mark |= !(fabsf(a.delta[(int64_t)t * a.H + hk * a.G + h]) < INFINITY);
      for (;;) {
        const uint32_t is = ti % G_NI;
        if (!wait_warp(ix_full(is), (ti / G_NI) & 1u)) { ok = false; break; }
        const Tile* tile = tiles + is;
        const int32_t count = tile->count, last = tile->last;
        if (count > 0) {
          if (!BF16)  // the factor's inverse: a power of two
            undo = a.scale * __int_as_float((254 << 23) - tile->mark);
          // this lane's eight keys: row k * 4 + lane / 8 of the warp's 32
          int32_t key[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t r = wq * 32u + k * 4u + (lane >> 3);
            key[k] = (int32_t)r < count ? tile->key[r] : -1;
          }
#pragma unroll 1
          for (uint32_t e = 2u * n; e < 2u * n + 2u; ++e) {
            const uint32_t b = e % 3u;
            if (!wait_warp(acc_full(b), (e / 3u) & 1u)) { ok = false; break; }
            tc::fence_after();
            const bool odd = __any_sync(0xffffffffu, mark) && !(e & 1u);
            float* sum = ((e & 1u) ? a.dk32 : a.dv32) + (int64_t)hk * D + (lane & 7u) * 4u;
            const float f = (e & 1u) ? undo : 1.0f;
#pragma unroll 1
            for (uint32_t c = 0; c < (uint32_t)D; c += 32) {
              float u[32];
              tc::tm_ld32(tmem + lanes + b * 128u + c, u);
              tc::wait_ld();
              if (c + 32u == (uint32_t)D) {
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(acc_free(b));
              }
              __syncwarp();  // the last chunk's rows have been read
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(stage + row * 32 + (((i >> 2) ^ (row & 7u)) << 2)) =
                    make_float4(u[i] * f, u[i + 1] * f, u[i + 2] * f, u[i + 3] * f);
              __syncwarp();
              if (odd) {
                add_odd_rows<D, BF16>(&a, t, hk, c, wq, lane, tile, stage, sum + c);
                continue;
              }
              // four rows of 128 bytes per step; the reads of all eight steps first
              // (each waited for the one before it when they took turns)
              float4 x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t r = wq * 32u + k * 4u + (lane >> 3);
                x[k] = *reinterpret_cast<const float4*>(stage + r * 32 +
                                                        (((lane & 7u) ^ (r & 7u)) << 2));
              }
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (key[k] >= 0) red4(sum + key[k] * key_floats + c, x[k]);
            }
          }
          if (!ok) break;
          any = true;
          ++n;
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(ix_empty(is));
        ++ti;
        if (last) break;
      }
      if (!ok) break;
      if (any) {
        if (!wait_warp(dq_full, nq & 1u)) break;
        ++nq;
        tc::fence_after();
      }
#pragma unroll 1
      for (uint32_t c = 0; c < (uint32_t)D; c += 32) {
        float u[32];
        if (any) {
          tc::tm_ld32(tmem + lanes + TM_DQ + c, u);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = 0.0f;
        }
        if (any && c + 32u == (uint32_t)D) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(dq_free);
        }
        if (!drain_sync()) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(stage + row * 32 + (((i >> 2) ^ (row & 7u)) << 2)) =
              make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
        if (!drain_sync()) { ok = false; break; }
        for (uint32_t e = tid - 128u; e < (uint32_t)a.G * 8u; e += 128u) {
          const uint32_t hh = e >> 3, p = e & 7u;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < COPIES; ++k) {
            const uint32_t r = k * PER + hh;
            const float4 x = *reinterpret_cast<const float4*>(stage + r * 32 + ((p ^ (r & 7u)) << 2));
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
          }
          uint2 w;
          w.x = tc::pack16<BF16>(o.x * undo, o.y * undo);
          w.y = tc::pack16<BF16>(o.z * undo, o.w * undo);
          uint16_t* dst = static_cast<uint16_t*>(a.dq) +
                          ((int64_t)t * a.H + hk * a.G + hh) * D + c + p * 4;
          *reinterpret_cast<uint2*>(dst) = w;
        }
      }
      if (!ok || !drain_sync()) break;  // the rows have been read before the next tile takes their place
    }
  } else if (warp < 16) {
    // -------------------------------------------------------------- gather
    tc::regs_down<R_GATHER>();
    const uint32_t gt = tid & 127u, kv = (warp - 8u) >> 2;
    const void* src = kv ? a.v : a.k;
    const int32_t row_bytes = (int32_t)(kv ? a.v_ts : a.k_ts);
    const int64_t head_bytes = kv ? a.v_hs : a.k_hs;
    uint32_t ti = 0, seq = 0;
    bool ok = true;
    for (int32_t item = first; item < a.items && ok; item += step) {
      const int32_t hk = item % a.Hk;
      for (;;) {
        const uint32_t is = ti % G_NI;
        if (!wait_warp(ix_full(is), (ti / G_NI) & 1u)) { ok = false; break; }
        const Tile* tile = tiles + is;
        const int32_t last = tile->last;
        if (tile->count > 0) {
          const uint32_t s = kv * P::SLOTS + seq % P::SLOTS;
          if (!wait_warp(kv_empty(s), ((seq / P::SLOTS) & 1u) ^ 1u)) { ok = false; break; }
          gather_rows<D, G_GATHER>(base + P::OFF_K + s * P::TILE, src, row_bytes, head_bytes * hk,
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
  } else {
    tc::regs_down<R_REST>();
    if (warp == 16) {
      // ------------------------------------------------------- tensor core
      constexpr uint32_t id_s = tc::idesc(BF16, 128, KT, false, false);
      constexpr uint32_t id_q = tc::idesc(BF16, 128, D, false, true);
      constexpr uint32_t id_k = tc::idesc(BF16, 128, D, true, true);
      const uint32_t lead = tc::elect_lane();
      uint32_t ti = 0, n = 0, nq = 0, nd = 0;
      bool ok = true;
      for (int32_t item = first; item < a.items && ok; item += step) {
        uint32_t nth = 0;
        if (!wait_warp(q_full, nq & 1u)) break;
        ++nq;
        for (;;) {
          const uint32_t is = ti % G_NI;
          if (!wait_warp(ix_full(is), (ti / G_NI) & 1u)) { ok = false; break; }
          const int32_t count = tiles[is].count, last = tiles[is].last;
          __syncwarp();
          if (lane == 0) tc::bar_arrive(ix_empty(is));
          ++ti;
          if (count > 0) {
            const uint32_t s = n % P::SLOTS, full = (n / P::SLOTS) & 1u;
            const uint32_t e = 2u * n, bs = e % 3u, bd = (e + 1u) % 3u;
            const uint32_t kb = base + P::OFF_K + s * P::TILE, vb = base + P::OFF_V + s * P::TILE;
            if (!wait_warp(kv_full(s), full) ||
                !wait_warp(acc_free(bs), ((e / 3u) & 1u) ^ 1u)) { ok = false; break; }
            tc::fence_async_shared();
            tc::fence_after();
#pragma unroll
            for (uint32_t kk = 0; kk < D / 16; ++kk)
              tc::mma_ss(tmem + bs * 128u, tc::desc_k(base + P::OFF_Q, P::BLOCK, kk),
                         tc::desc_k(kb, P::BLOCK, kk), id_s, kk > 0, lead);
            if (!wait_warp(kv_full(P::SLOTS + s), full) ||
                !wait_warp(acc_free(bd), (((e + 1u) / 3u) & 1u) ^ 1u)) { ok = false; break; }
            tc::fence_async_shared();
            tc::fence_after();
#pragma unroll
            for (uint32_t kk = 0; kk < D / 16; ++kk)
              tc::mma_ss(tmem + bd * 128u, tc::desc_k(base + P::OFF_DO, P::BLOCK, kk),
                         tc::desc_k(vb, P::BLOCK, kk), id_s, kk > 0, lead);
            tc::mma_commit(kv_empty(P::SLOTS + s), lead);
            tc::mma_commit(s_full, lead);
            if (!wait_warp(w_full, n & 1u)) { ok = false; break; }
            if (nth == 0) {
              // the last item's dQ has been read
              if (!wait_warp(dq_free, (nd & 1u) ^ 1u)) { ok = false; break; }
              ++nd;
            }
            tc::fence_after();
#pragma unroll
            for (uint32_t kk = 0; kk < KT / 16; ++kk)
              tc::mma_ss(tmem + TM_DQ, tc::desc_k(base + P::OFF_DS, P::BLOCK, kk),
                         tc::desc_mn(kb, P::BLOCK, kk), id_q, nth > 0 || kk > 0, lead);
            tc::mma_commit(kv_empty(s), lead);
            if (last) tc::mma_commit(dq_full, lead);
#pragma unroll
            for (uint32_t kk = 0; kk < 8; ++kk)
              tc::mma_ss(tmem + bs * 128u, tc::desc_mn(base + P::OFF_P, P::BLOCK, kk),
                         tc::desc_mn(base + P::OFF_DO, P::BLOCK, kk), id_k, kk > 0, lead);
            tc::mma_commit(acc_full(bs), lead);
#pragma unroll
            for (uint32_t kk = 0; kk < 8; ++kk)
              tc::mma_ss(tmem + bd * 128u, tc::desc_mn(base + P::OFF_DS, P::BLOCK, kk),
                         tc::desc_mn(base + P::OFF_Q, P::BLOCK, kk), id_k, kk > 0, lead);
            tc::mma_commit(acc_full(bd), lead);
            tc::mma_commit(w_empty, lead);
            if (last) tc::mma_commit(q_empty, lead);
            ++n;
            ++nth;
          }
          if (last) {
            if (nth == 0 && lane == 0) tc::bar_arrive(q_empty);
            break;
          }
        }
      }
      if (n > 0) {
        tc::mma_commit(last_bar, lead);
        tc::bar_drain(last_bar, 0u);
      }
    } else if (warp == 17) {
      // --------------------------------------------------------- index rows
      uint32_t ti = 0;
      compact_rows(
          a, first, step, 0, 1, lane,
          [&](int32_t t, int32_t hk) { return BF16 ? 0 : factor_bits<D>(a, t, hk, lane); },
          [&]() -> Tile* {
            return wait_warp(ix_empty(ti % G_NI), ((ti / G_NI) & 1u) ^ 1u) ? tiles + ti % G_NI
                                                                           : nullptr;
          },
          [&]() {
            __syncwarp();
            if (lane == 0) tc::bar_arrive(ix_full(ti % G_NI));
            ++ti;
          });
    } else if (warp == 18) {
      // --------------------------------------- the items' q and dout head rows
      uint32_t nq = 0;
      clear_heads<D, 32>(sm + P::OFF_Q, a.G, PER, lane);
      clear_heads<D, 32>(sm + P::OFF_DO, a.G, PER, lane);
      for (int32_t item = first; item < a.items; item += step, ++nq) {
        const int32_t t = item / a.Hk, hk = item - t * a.Hk;
        if (nq > 0 && !wait_warp(q_empty, (nq - 1u) & 1u)) break;
        load_heads<D, 32>(base + P::OFF_Q, a.q, t * a.q_ts, a.q_hs, hk * a.G, a.G, PER, lane);
        load_heads<D, 32>(base + P::OFF_DO, a.dout, t * a.do_ts, a.do_hs, hk * a.G, a.G, PER, lane);
        tc::cp_commit();
        tc::cp_wait<0>();
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(q_full);
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == 16) {
    tc::fence_after();
    tc::tm_free(tmem, G_TMEM);
  }
}

__device__ __forceinline__ float2 widen(uint32_t u, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Clears the sums (n4 float4) and computes delta = dout . out: 8 or 16 lanes of
// 16 bytes per head row.
template <int D>
__global__ void __launch_bounds__(256) k_grad_begin(const __grid_constant__ Args a, int32_t bf16,
                                                    int64_t n4) {
  float4* sums = reinterpret_cast<float4*>(a.dk32);
  const int64_t start = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = start; i < n4; i += stride) sums[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int L = D / 8;
  const int64_t rows = (int64_t)a.T * a.H;
  const int lane = threadIdx.x % L;
  // whole warps run the same rounds: their shuffles meet
  for (int64_t r = start / L; r - (int64_t)(threadIdx.x % 32) / L < rows; r += stride / L) {
    float d = 0.0f;
    if (r < rows) {
      const int64_t t = r / a.H, h = r - t * a.H;
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.dout) +
                                                      t * a.do_ts + h * a.do_hs + lane * 16);
      const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.out) +
                                                      r * (2 * D) + lane * 16);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = widen(xs[i], bf16), q = widen(ys[i], bf16);
        d = fmaf(p.x, q.x, fmaf(p.y, q.y, d));
      }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (r < rows && lane == 0) a.delta[r] = d;
  }
}

// The FP32 sums rounded once to the keys' type, 8 elements per step.
template <bool BF16>
__global__ void __launch_bounds__(256) k_grad_end(const float4* dk32, const float4* dv32, uint4* dk,
                                                  uint4* dv, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < 2 * n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const bool second = i >= n;
    const int64_t j = second ? i - n : i;
    const float4* src = second ? dv32 : dk32;
    const float4 x = src[2 * j], y = src[2 * j + 1];
    (second ? dv : dk)[j] = make_uint4(tc::pack16<BF16>(x.x, x.y), tc::pack16<BF16>(x.z, x.w),
                                       tc::pack16<BF16>(y.x, y.y), tc::pack16<BF16>(y.z, y.w));
  }
}

// ------------------------------------------------------------------ host side
template <int D, int NC, bool BF16>
int launch_grad(const Args& a, int sms, cudaStream_t st) {
  static OncePerDevice opted_in;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TOPK_ERR_NO_DEVICE;
  if (!opted_in.ensure(dev, [] {
        return cudaFuncSetAttribute(k_attend_grad<D, NC, BF16>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)GradPlan<D>::BYTES) == cudaSuccess;
      }))
    return TOPK_ERR_CUDA;
  const int grid = a.items < sms ? a.items : sms;
  k_attend_grad<D, NC, BF16><<<grid, G_THREADS, GradPlan<D>::BYTES, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA;
}

template <int D, bool BF16>
int run_grad(const Args& a, void* dk, void* dv, int sms, cudaStream_t st) {
  const int64_t n = (int64_t)a.S * a.Hk * D;  // elements of dk and of dv
  k_grad_begin<D><<<sms * 8, 256, 0, st>>>(a, BF16, n / 2);
  if (cudaGetLastError() != cudaSuccess) return TOPK_ERR_CUDA;
  int rc = TOPK_OK;
  if (a.T > 0)
    rc = a.G <= 32   ? launch_grad<D, 32, BF16>(a, sms, st)
         : a.G <= 64 ? launch_grad<D, 64, BF16>(a, sms, st)
                     : launch_grad<D, 128, BF16>(a, sms, st);
  if (rc != TOPK_OK || n == 0) return rc;
  k_grad_end<BF16><<<sms * 8, 256, 0, st>>>(
      reinterpret_cast<const float4*>(a.dk32), reinterpret_cast<const float4*>(a.dv32),
      static_cast<uint4*>(dk), static_cast<uint4*>(dv), n / 8);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA;
}

int take_status_grad(cudaStream_t st, uint32_t* flags) {
  uint32_t h = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&h, g_status, sizeof h, 0, cudaMemcpyDeviceToHost, st) !=
          cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st) !=
          cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return TOPK_ERR_CUDA;
  *flags = h;
  return TOPK_OK;
}

}  // namespace ta

extern "C" {

size_t topk_sparse_attention_backward_workspace_bytes(int64_t T, int64_t S, int32_t H, int32_t Hk,
                                                      int32_t D) {
  if (T < 0 || S < 0 || H < 1 || Hk < 1 || D < 1) return 0;
  return 2 * (size_t)S * Hk * D * sizeof(float) + (size_t)T * H * sizeof(float);
}

int topk_sparse_attention_backward(
    const void* dout, int64_t do_token_stride, int64_t do_head_stride, const void* q,
    int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
    int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
    const int32_t* idx, int64_t ld_idx, const void* out, const float* lse, int64_t T, int64_t S,
    int32_t H, int32_t Hk, int32_t D, int32_t K, int32_t dtype, float scale, float softcap,
    const float* slopes, const int32_t* positions, const int32_t* key_lo, const int32_t* key_hi,
    void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
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
  a.do_ts = 2 * do_token_stride;
  a.do_hs = 2 * do_head_stride;
  a.ld_idx = ld_idx;
  a.T = (int32_t)T;
  a.S = (int32_t)S;
  a.H = H;
  a.Hk = Hk;
  a.K = K;
  a.scale = scale;
  a.cap = softcap;
  a.dout = dout;
  a.out = const_cast<void*>(out);
  a.lse_in = lse;
  a.dq = dq;
  int rc = ta::check_args(a, D, dtype);
  if (rc != TOPK_OK || (T == 0 && S == 0)) return rc;
  if ((T > 0 && (!dout || !out || !lse || !dq)) || (S > 0 && (!dk || !dv))) return TOPK_ERR_ARG;
  auto off = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (off(dout, 16) || off(out, 16) || off(lse, 4) || off(dq, 8) || off(dk, 16) || off(dv, 16) ||
      ((a.do_ts | a.do_hs) & 15) || off(workspace, 16))
    return TOPK_ERR_ALIGN;
  if (!workspace ||
      workspace_bytes < topk_sparse_attention_backward_workspace_bytes(T, S, H, Hk, D))
    return TOPK_ERR_WORKSPACE;
  a.dk32 = static_cast<float*>(workspace);
  a.dv32 = a.dk32 + S * (int64_t)Hk * D;
  a.delta = a.dv32 + S * (int64_t)Hk * D;
  a.G = H / Hk;
  a.chunks = (int32_t)(((int64_t)K + ta::KT - 1) / ta::KT);
  a.items = a.T * Hk;
  int sms = 0;
  rc = ta::device_sms(&sms);
  if (rc != TOPK_OK) return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TOPK_BF16)
    return D == 64 ? ta::run_grad<64, true>(a, dk, dv, sms, st) : ta::run_grad<128, true>(a, dk, dv, sms, st);
  return D == 64 ? ta::run_grad<64, false>(a, dk, dv, sms, st) : ta::run_grad<128, false>(a, dk, dv, sms, st);
}

}  // extern "C"
