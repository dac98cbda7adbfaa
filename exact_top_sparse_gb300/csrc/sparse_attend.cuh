// What the forward and the backward kernel of the attention over selected keys
// share: arguments, the compaction of index rows into key tiles, and the
// gather of key and value rows into swizzled shared memory.
#pragma once

#include "tc_ptx.cuh"
#include "topk.h"

namespace ta {

constexpr int KT = 128;                // keys per tile
constexpr float LOG2E = 1.4426950408889634f;

struct Args {
  const void* q;                       // [T][H][D], strides in bytes
  const void* k;                       // [S][Hk][D]
  const void* v;
  const int32_t* idx;                  // [T][ld_idx]
  const float* slopes;                 // [H] or nullptr
  const int32_t* pos;                  // [T], with slopes
  const int32_t* lo;                   // [T] or nullptr
  const int32_t* hi;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  int64_t ld_idx;
  int32_t T, H, Hk, G, K, S;           // G = H / Hk
  int32_t chunks;                      // ceil(K / KT)
  int32_t items;                       // T * Hk
  float scale, cap;                    // cap <= 0: none
  // forward
  void* out;                           // [T][H][D] contiguous
  float* lse;                          // [T][H] or nullptr
  // backward
  const void* dout;                    // strides in bytes
  int64_t do_ts, do_hs;
  const float* lse_in;                 // [T][H]
  float* delta;                        // [T][H]: sum of dout * out
  void* dq;                            // [T][H][D] contiguous
  float* dk32;                         // [S][Hk][D] FP32 sums
  float* dv32;
};

static __device__ uint32_t g_status;   // OR of error bits since the last read (one per direction)

// A tile of selected keys: slots of the cache, the first `count` of them valid.
struct Tile {
  int32_t key[KT];
  int32_t count;
  int32_t last;                        // 1: the item's last tile
  int32_t token;                       // the item's
  int32_t mark;                        // forward: its key head; gradient: dS's factor (bits)
};

// 16-byte piece `piece` of row `row` in a tile of 128-byte swizzled rows, one
// block of `rows` rows for every 64 elements.
__device__ __forceinline__ uint32_t piece_at(uint32_t row, uint32_t piece, uint32_t rows) {
  return (piece >> 3) * rows * 128u + row * 128u + (((piece & 7u) ^ (row & 7u)) << 4);
}

// One warp reads the index rows of the CTA's items (chunks c0, c0 + cstep, ... of
// each) and hands over tiles of valid keys: -1, anything outside [0, S) and
// anything outside the token's key range is dropped, so a masked key is neither
// read nor multiplied.  Every item gives at least one tile (count 0 where nothing
// is left).
//   acquire() -> Tile* (nullptr: gave up), publish() hands it over; mark(token, key
//   head) -> the item's Tile::mark, called by the whole warp.
// A lane takes four neighbouring entries (one 16-byte load where rows allow it),
// and two chunks are on their way while one is compacted, across items: with
// single loads, one chunk ahead, this warp took 1500 cycles a tile, more than the
// products.
template <class Mark, class Acquire, class Publish>
__device__ __forceinline__ void compact_rows(const Args& a, int32_t first, int32_t istep,
                                             int32_t c0, int32_t cstep, uint32_t lane, Mark mark,
                                             Acquire acquire, Publish publish) {
  struct Chunk {
    int4 v;
    int32_t lo, hi;
  };
  // the position two chunks ahead: its item, chunk, index row and key range
  int32_t pi = first, pc = c0, plo = 0, phi = a.S;
  const int32_t* prow = a.idx;
  bool wide = false;
  auto enter = [&]() {
    if (pi >= a.items) return;
    const int32_t t = pi / a.Hk;
    prow = a.idx + (int64_t)t * a.ld_idx;
    wide = (reinterpret_cast<uintptr_t>(prow) & 15u) == 0u;
    if (a.lo) plo = max(__ldg(a.lo + t), 0);
    if (a.hi) phi = min(__ldg(a.hi + t), a.S);
  };
  auto load = [&]() {
    Chunk k{make_int4(-1, -1, -1, -1), plo, phi};
    if (pi < a.items) {
      const int64_t j = (int64_t)pc * KT + (int64_t)lane * 4;
      if (wide && j + 4 <= a.K) {
        k.v = __ldg(reinterpret_cast<const int4*>(prow + j));
      } else {
        if (j < a.K) k.v.x = __ldg(prow + j);
        if (j + 1 < a.K) k.v.y = __ldg(prow + j + 1);
        if (j + 2 < a.K) k.v.z = __ldg(prow + j + 2);
        if (j + 3 < a.K) k.v.w = __ldg(prow + j + 3);
      }
      pc += cstep;
      if (pc >= a.chunks) {
        pc = c0;
        pi += istep;
        enter();
      }
    }
    return k;
  };
  enter();
  Chunk next = load();
  Chunk after = load();
  for (int32_t item = first; item < a.items; item += istep) {
    const int32_t t = item / a.Hk, its_mark = mark(t, item - t * a.Hk);
    Tile* tile = acquire();
    if (!tile) return;
    int32_t n = 0;
    auto close = [&](int32_t last) {
      if (lane == 0) {
        tile->count = last ? n : KT;
        tile->last = last;
        tile->token = t;
        tile->mark = its_mark;
      }
      publish();
    };
    for (int32_t c = c0;; ) {
      const Chunk now = next;
      next = after;
      after = load();
      const bool g0 = now.v.x >= now.lo && now.v.x < now.hi, g1 = now.v.y >= now.lo && now.v.y < now.hi;
      const bool g2 = now.v.z >= now.lo && now.v.z < now.hi, g3 = now.v.w >= now.lo && now.v.w < now.hi;
      const uint32_t m0 = __ballot_sync(0xffffffffu, g0), m1 = __ballot_sync(0xffffffffu, g1);
      const uint32_t m2 = __ballot_sync(0xffffffffu, g2), m3 = __ballot_sync(0xffffffffu, g3);
      const int32_t n0 = __popc(m0), n1 = __popc(m1), n2 = __popc(m2), n3 = __popc(m3);
      const int32_t total = n0 + n1 + n2 + n3;
      if (total > 0) {
        const uint32_t before = (1u << lane) - 1u;
        if (n == KT) {  // the tile is full and more follow: hand it over
          close(0);
          tile = acquire();
          if (!tile) return;
          n = 0;
        }
        if (n == 0 && total == KT) {
          *reinterpret_cast<int4*>(tile->key + lane * 4) = now.v;  // as it stands
          n = KT;
        } else {
          const int32_t p0 = n + __popc(m0 & before), p1 = n + n0 + __popc(m1 & before);
          const int32_t p2 = n + n0 + n1 + __popc(m2 & before);
          const int32_t p3 = n + n0 + n1 + n2 + __popc(m3 & before);
          if (g0 && p0 < KT) tile->key[p0] = now.v.x;
          if (g1 && p1 < KT) tile->key[p1] = now.v.y;
          if (g2 && p2 < KT) tile->key[p2] = now.v.z;
          if (g3 && p3 < KT) tile->key[p3] = now.v.w;
          n += total;
          if (n > KT) {
            close(0);
            tile = acquire();
            if (!tile) return;
            n -= KT;
            if (g0 && p0 >= KT) tile->key[p0 - KT] = now.v.x;
            if (g1 && p1 >= KT) tile->key[p1 - KT] = now.v.y;
            if (g2 && p2 >= KT) tile->key[p2 - KT] = now.v.z;
            if (g3 && p3 >= KT) tile->key[p3 - KT] = now.v.w;
          }
        }
      }
      c += cstep;
      if (c >= a.chunks) break;
    }
    close(1);
  }
}

// NT threads (tid 0..NT-1) start the copies of a tile's rows of k or v.  The
// lanes of one row take its 16-byte pieces; a thread's rows are consecutive, so
// that their keys come in a few vector loads ahead of the copies.
template <int D, int NT>
__device__ __forceinline__ void gather_rows(uint32_t dst, const void* base, int32_t row_bytes,
                                            int64_t head_bytes, const Tile* tile, uint32_t tid) {
  constexpr uint32_t PIECES = D / 8;             // 16-byte pieces of a row
  constexpr uint32_t ROWS = KT * PIECES / NT;    // rows of a thread
  const uint32_t piece = tid % PIECES, r0 = tid / PIECES * ROWS;
  const uint8_t* src = static_cast<const uint8_t*>(base) + head_bytes + piece * 16;
  const int32_t n = tile->count;
  dst += piece_at(r0, piece, KT);  // r0 is a multiple of 8: row r0 + i has swizzle i & 7
  if (n >= KT) {
    // four at a time in a loop: unrolled it took more in instruction fetches
#pragma unroll 1
    for (uint32_t i = 0; i < ROWS; i += 4) {
      const int4 key = *reinterpret_cast<const int4*>(tile->key + r0 + i);
      const uint32_t d = (dst ^ ((i & 7u) << 4)) + i * 128u;  // i & 7 is 0 or 4
      tc::cp_async16(d, src + (int64_t)key.x * row_bytes, 16u);
      tc::cp_async16((d ^ 16u) + 128u, src + (int64_t)key.y * row_bytes, 16u);
      tc::cp_async16((d ^ 32u) + 256u, src + (int64_t)key.z * row_bytes, 16u);
      tc::cp_async16((d ^ 48u) + 384u, src + (int64_t)key.w * row_bytes, 16u);
    }
  } else {
#pragma unroll 1
    for (uint32_t i = 0; i < ROWS; ++i) {
      const bool ok = (int32_t)(r0 + i) < n;
      tc::cp_async16((dst ^ ((i & 7u) << 4)) + i * 128u,
                     src + (ok ? (int64_t)tile->key[r0 + i] * row_bytes : 0), ok ? 16u : 0u);
    }
  }
}

// NT threads start the copies of a token's G heads into a 128-row operand: row r
// is head r % per.  The rows of no head stay as clear_heads() left them.
template <int D, int NT>
__device__ __forceinline__ void load_heads(uint32_t dst, const void* base, int64_t token_off,
                                           int64_t head_bytes, int32_t h0, int32_t G, int32_t per,
                                           uint32_t tid) {
  constexpr uint32_t PIECES = D / 8, ROWS = NT / PIECES;
  const uint32_t piece = tid % PIECES;
  const uint8_t* src = static_cast<const uint8_t*>(base) + token_off + h0 * head_bytes + piece * 16;
#pragma unroll 1
  for (uint32_t c = 0; c < 128u; c += (uint32_t)per)
#pragma unroll 4
    for (uint32_t h = tid / PIECES; h < (uint32_t)G; h += ROWS)
      tc::cp_async16(dst + piece_at(c + h, piece, 128u), src + h * head_bytes, 16u);
}
// NT threads write zeros to the rows of no head (once: the copies leave them alone).
template <int D, int NT>
__device__ __forceinline__ void clear_heads(uint8_t* dst, int32_t G, int32_t per, uint32_t tid) {
  constexpr uint32_t PIECES = D / 8;
#pragma unroll 1
  for (uint32_t e = tid; e < 128u * PIECES; e += NT) {
    const uint32_t r = e / PIECES;
    if ((int32_t)(r & (per - 1)) >= G)
      *reinterpret_cast<uint4*>(dst + piece_at(r, e % PIECES, 128u)) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// 1 - 2 / (1 + e^2x): absolute error of a few 2^-24 over the whole range.  NaN
// stays NaN (fminf would give 40 for it).
__device__ __forceinline__ float tanh_of(float x) {
  return 1.0f - __fdividef(2.0f, 1.0f + tc::ex2((x > 40.0f ? 40.0f : x) * (2.0f * LOG2E)));
}
// A cap far above the scores multiplies that error: above WIDE_CAP (where it is
// 2^-14 of a weight, still below P's rounding to 16 bits) the series to x^9 takes its
// place below 1/4 (next term: 2^-26 of the sum; error at most 2^-20 of tanh).  For
// every cap it took 334 us for 270 (512 x 32/8 heads x 64, Top-1024, cap 30).
constexpr float WIDE_CAP = 256.0f;
__device__ __forceinline__ float tanh_near(float x) {
  const float s = x * x;
  const float near = x * fmaf(s, fmaf(s, fmaf(s, fmaf(s, 62.0f / 2835.0f, -17.0f / 315.0f),
                                              2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
  return fabsf(x) < 0.25f ? near : tanh_of(x);
}

// Host side, shared by both directions.
int take_status_grad(cudaStream_t st, uint32_t* flags);
int check_args(const Args& a, int32_t D, int32_t dtype);
int device_sms(int* sms);

}  // namespace ta
