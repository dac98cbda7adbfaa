// Rotary positions, and the RMS norm of every query and key head with the
// rotation in the same pass, forward and backward.
//
//   phase_i = position * step_i  mod 2^64     (step_i: angle per position in
//                                              units of 2^-64 turns)
//   (x0, x1) -> scale * (x0 cos a - x1 sin a, x1 cos a + x0 sin a),
//               a = 2 pi phase_i / 2^64
//   norm: x_hat = x * rsqrt(mean(x^2) + eps), y = rotate(x_hat * w)
//   grad: g = rotate^-1(dy), dx = rstd * (g w - x_hat * mean(g w x_hat)),
//         dw = sum over rows of g x_hat
//
// The phase is a whole number and wraps where a turn ends, so it is exact at
// every position; an FP32 angle at position 10^6 would be off by 0.03 rad.
//
// All of it is bound by memory: one read and one write of every element.  A
// block takes a few whole tokens, puts their sines and cosines into shared
// memory once (sincospif of the phase's top 32 bits: 2^-32 turns; there is no
// table to read from memory), and turns all their heads with them.  A row (one
// head of one token) belongs to L lanes; a lane owns slots of two chunks of VEC
// elements.  A rotated slot holds VEC whole pairs (for the half layout its
// chunks lie rot/2 apart, for the interleaved one side by side), so the
// rotation needs no exchange between lanes; only the norm's sum does.  VEC is
// the widest of 16, 8, 4 bytes or one element that the sizes, strides and
// addresses allow.
//
// Measured on GB300 (BF16, in a graph): rotation of 8192 x 64 x 128 44 us (6.1
// TB/s, 0.90 of the measured copy rate), norm + rotation of 16384 x 36 x 128 63 us
// (4.8 TB/s; instructions bound it, two elements in each, and at the 64 registers of
// four blocks an SM the BF16 kernel spills 246 bytes a thread), its gradient of 8192 x
// 40 x 128 61 us (4.1 TB/s; two sums over the row between its loads and its stores,
// and 118 bytes spilled at 80 registers), one token 2.5 us.  Rows on their way through a ring of asynchronous
// copies in shared memory cost instructions and brought nothing (gradient 93 us
// with it and 94 without, before its blocks were balanced).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include <type_traits>

#include "tc_ptx.cuh"
#include "topk.h"

namespace tr {

constexpr int THREADS = 256;
constexpr int MAX_D = 512;
constexpr int MAX_BLOCKS = 456;  // of the backward pass, three for each of 152 SMs (rows of
                                 // partial sums of dw)
constexpr int TABLE_COST = 4;    // passes over the table to the time of a round of rows

struct Side {
  const void* x;
  const void* dy;       // backward only
  void* y;              // output, or dx
  const void* w;        // or nullptr
  int64_t x_ts, x_hs, dy_ts, dy_hs, y_ts, y_hs;  // strides in elements, below 2^31
  int32_t H;
  uint32_t inv_h;       // r / H = umulhi(r, inv_h) for a block's rows r < 2^16 (H > 1)
  int32_t blocks;       // backward
  int32_t tokens;       // of a block at a time
};
struct Args {
  Side side[2];
  const void* pos;
  const int64_t* freqs;
  float* partial;       // backward: [blocks of both sides][D]
  int64_t T;
  int32_t pos64, w32, w_vec;  // w_vec: weights readable as vectors
  int32_t D, rot, offset, interleaved, inverse;
  int32_t lanes;        // L, a power of two
  float scale, eps;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float f, float& x) { x = f; }
__device__ __forceinline__ void from_f(float f, __nv_bfloat16& x) { x = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_f(float f, __half& x) { x = __float2half_rn(f); }

// Whole packs, 16-bit types two elements per instruction.
template <int N>
__device__ __forceinline__ void widen(const Pack<float, N>& p, float* f) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = p.v[i];
}
template <typename T, int N>
__device__ __forceinline__ void widen(const Pack<T, N>& p, float* f) {
  if (N == 1) {
    f[0] = to_f(p.v[0]);
    return;
  }
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (std::is_same<T, __nv_bfloat16>::value) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(w + i));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}
template <int N>
__device__ __forceinline__ void narrow(const float* f, Pack<float, N>& p) {
#pragma unroll
  for (int i = 0; i < N; ++i) p.v[i] = f[i];
}
template <typename T, int N>
__device__ __forceinline__ void narrow(const float* f, Pack<T, N>& p) {
  if (N == 1) {
    from_f(f[0], p.v[0]);
    return;
  }
  uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    w[i] = tc::pack16<std::is_same<T, __nv_bfloat16>::value>(f[2 * i], f[2 * i + 1]);
}

enum { ROPE = 0, NORM = 1, NORM_GRAD = 2 };

// Two elements per instruction (each rounded as the plain form's).
__device__ __forceinline__ float2 two(const float* f) { return make_float2(f[0], f[1]); }
__device__ __forceinline__ void two(float* f, float2 v) {
  f[0] = v.x;
  f[1] = v.y;
}

// The pairs of a slot: f[0..2 VEC) as loaded (two chunks) is turned in place.
// The fused operations are spelled out: every vector width gives the same bits.
// cs, sn: VEC values in shared memory, aligned to VEC floats where VEC > 1.
template <int VEC>
__device__ __forceinline__ void turn(float* f, const float* cs, const float* sn, bool interleaved) {
  constexpr int W = VEC < 4 ? VEC : 4;
  float c[VEC], s[VEC];
#pragma unroll
  for (int i = 0; i < VEC; i += W) {
    *reinterpret_cast<Pack<float, W>*>(c + i) = *reinterpret_cast<const Pack<float, W>*>(cs + i);
    *reinterpret_cast<Pack<float, W>*>(s + i) = *reinterpret_cast<const Pack<float, W>*>(sn + i);
  }
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float a = f[2 * i], b = f[2 * i + 1];
      f[2 * i] = fmaf(a, c[i], -(b * s[i]));
      f[2 * i + 1] = fmaf(b, c[i], a * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += VEC > 1 ? 2 : 1) {
      if (VEC > 1) {
        const float2 a = two(f + i), b = two(f + VEC + i), ci = two(c + i), si = two(s + i);
        const float2 t = __fmul2_rn(b, make_float2(-si.x, -si.y));
        two(f + i, __ffma2_rn(a, ci, t));
        two(f + VEC + i, __ffma2_rn(b, ci, __fmul2_rn(a, si)));
      } else {
        const float a = f[i], b = f[VEC + i];
        f[i] = fmaf(a, c[i], -(b * s[i]));
        f[VEC + i] = fmaf(b, c[i], a * s[i]);
      }
    }
  }
}

template <typename T, int VEC, int NS, int MODE>
__global__ void __launch_bounds__(THREADS, NS > 1 ? 2 : MODE == NORM_GRAD ? 3 : 4)
    k_rope(const __grid_constant__ Args a) {
  using P = Pack<T, VEC>;
  constexpr int U = NS > 1 || MODE == NORM_GRAD ? 1 : 2;  // rows in flight per lane
  extern __shared__ float table[];   // [tokens][cos, sin][rot / 2]
  const int L = a.lanes, lane = threadIdx.x & (L - 1), per_block = THREADS / L;
  const int group = (int)threadIdx.x / L;
  const bool inter = a.interleaved != 0;
  const int pairs = a.rot / 2;
  const float inv_d = 1.0f / (float)a.D;

  // this lane's slots
  const int rot_slots = a.rot / (2 * VEC), pass_chunks = (a.D - a.rot) / VEC;
  int e[NS][2];
  bool ok[NS][2], turned[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int slot = lane + j * L;
    turned[j] = slot < rot_slots;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (turned[j]) {
        e[j][h] = a.offset + (inter ? (2 * slot + h) * VEC : slot * VEC + h * pairs);
        ok[j][h] = true;
      } else {
        const int c = 2 * (slot - rot_slots) + h;
        ok[j][h] = c < pass_chunks;
        e[j][h] = ok[j][h] ? (c * VEC < a.offset ? c * VEC : c * VEC + a.rot) : 0;
      }
    }
  }
  float dw[MODE == NORM_GRAD ? NS : 1][2 * VEC];
#pragma unroll
  for (int j = 0; j < (MODE == NORM_GRAD ? NS : 1); ++j)
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) dw[j][i] = 0.0f;

  // the gradient's blocks belong to one side each, the others' do both
  const int mine = MODE == NORM_GRAD && (int)blockIdx.x >= a.side[0].blocks ? 1 : 0;
  const int64_t first = MODE == NORM_GRAD && mine ? (int)blockIdx.x - a.side[0].blocks : blockIdx.x;
  const int64_t step = MODE == NORM_GRAD ? a.side[mine].blocks : gridDim.x;
  const int tokens = a.side[mine].tokens;
  for (int64_t t0 = first * tokens; t0 < a.T; t0 += step * tokens) {
    const int nt = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
    if (pairs > 0) {
      __syncthreads();
      for (int i = threadIdx.x; i < nt * pairs; i += THREADS) {
        const int t = i / pairs, p = i - t * pairs;
        const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.pos)[t0 + t]
                                    : (int64_t)static_cast<const int32_t*>(a.pos)[t0 + t];
        const uint64_t ph = (uint64_t)pos * (uint64_t)a.freqs[p];
        float si, co;  // the top 32 bits as half turns in [-1, 1)
        sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &si, &co);
        table[2 * t * pairs + p] = co * a.scale;
        table[(2 * t + 1) * pairs + p] = (a.inverse ? -si : si) * a.scale;
      }
      __syncthreads();
    }
#pragma unroll 1
    for (int sd = mine; sd < (MODE == NORM_GRAD ? mine + 1 : 2); ++sd) {
      const Side& s = a.side[sd];
      const int rows = nt * s.H;
      if (rows == 0) continue;
      const T* xb = static_cast<const T*>(s.x) + t0 * s.x_ts;
      const T* db = MODE == NORM_GRAD ? static_cast<const T*>(s.dy) + t0 * s.dy_ts : nullptr;
      T* yb = static_cast<T*>(s.y) + t0 * s.y_ts;
      const uint32_t x_ts = (uint32_t)s.x_ts, x_hs = (uint32_t)s.x_hs, d_ts = (uint32_t)s.dy_ts,
                     d_hs = (uint32_t)s.dy_hs, y_ts = (uint32_t)s.y_ts, y_hs = (uint32_t)s.y_hs;
      float w[NS][2 * VEC];
      if (MODE != ROPE) {
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (s.w && !a.w32 && ok[j][h] && VEC > 1 && a.w_vec) {
              const P q = *reinterpret_cast<const P*>(static_cast<const T*>(s.w) + e[j][h]);
              widen(q, w[j] + h * VEC);
            } else {
#pragma unroll
              for (int i = 0; i < VEC; ++i)
                w[j][h * VEC + i] = !ok[j][h] ? 0.0f
                                    : !s.w    ? 1.0f
                                    : a.w32   ? static_cast<const float*>(s.w)[e[j][h] + i]
                                              : to_f(static_cast<const T*>(s.w)[e[j][h] + i]);
            }
          }
      }
      // groups of one warp run the same number of rounds: their shuffles meet
      for (int base = 0; base < rows; base += per_block * U) {
        P px[U][NS][2], pd[MODE == NORM_GRAD ? U : 1][NS][2];
        uint32_t tok[U], head[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = base + u * per_block + group;
          in[u] = r < rows;
          tok[u] = !in[u] ? 0u : s.H == 1 ? (uint32_t)r : __umulhi((uint32_t)r, s.inv_h);
          head[u] = in[u] ? r - tok[u] * s.H : 0u;
          const T* x = xb + (uint64_t)tok[u] * x_ts + (uint64_t)head[u] * x_hs;
          const T* d = MODE == NORM_GRAD ? db + (uint64_t)tok[u] * d_ts + (uint64_t)head[u] * d_hs
                                         : nullptr;
          // (a lane beyond the rows reads the block's first one again; its sums and
          // its stores are dropped)
#pragma unroll
          for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (ok[j][h]) {
                px[u][j][h] = *reinterpret_cast<const P*>(x + e[j][h]);
                if (MODE == NORM_GRAD) pd[u][j][h] = *reinterpret_cast<const P*>(d + e[j][h]);
              } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                  from_f(0.0f, px[u][j][h].v[i]);
                  if (MODE == NORM_GRAD) from_f(0.0f, pd[u][j][h].v[i]);
                }
              }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u > 0 && base + u * per_block >= rows) break;  // the whole block
          const float* cs = table + 2 * tok[u] * pairs + lane * VEC;
          const float* sn = cs + pairs;
          float f[NS][2 * VEC];
#pragma unroll
          for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) widen(px[u][j][h], f[j] + h * VEC);
          if (MODE != ROPE) {
            float2 ss2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
              for (int i = 0; i < 2 * VEC; i += 2)
                ss2 = __ffma2_rn(two(f[j] + i), two(f[j] + i), ss2);
            float ss = ss2.x + ss2.y;
            for (int o = L >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
            const float2 rstd2 = make_float2(rstd, rstd);
            if (MODE == NORM) {
#pragma unroll
              for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 2 * VEC; i += 2)
                  two(f[j] + i, __fmul2_rn(__fmul2_rn(two(f[j] + i), rstd2), two(w[j] + i)));
            } else {
              float g[NS][2 * VEC];
              float2 dot2 = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int j = 0; j < NS; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h) widen(pd[u][j][h], g[j] + h * VEC);
                if (turned[j]) turn<VEC>(g[j], cs + j * L * VEC, sn + j * L * VEC, inter);
#pragma unroll
                for (int i = 0; i < 2 * VEC; i += 2) {
                  const float2 xh = __fmul2_rn(two(f[j] + i), rstd2), gi = two(g[j] + i);
                  const float2 gw = __fmul2_rn(gi, two(w[j] + i));
                  two(f[j] + i, xh);
                  two(dw[j] + i, in[u] ? __ffma2_rn(gi, xh, two(dw[j] + i)) : two(dw[j] + i));
                  two(g[j] + i, gw);
                  dot2 = __ffma2_rn(gw, xh, dot2);
                }
              }
              float dot = dot2.x + dot2.y;
              for (int o = L >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
              dot *= -inv_d;
#pragma unroll
              for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 2 * VEC; i += 2)
                  two(f[j] + i, __fmul2_rn(rstd2, __ffma2_rn(two(f[j] + i), make_float2(dot, dot),
                                                             two(g[j] + i))));
            }
          }
          if (MODE != NORM_GRAD) {
#pragma unroll
            for (int j = 0; j < NS; ++j)
              if (turned[j]) turn<VEC>(f[j], cs + j * L * VEC, sn + j * L * VEC, inter);
          }
          T* y = yb + (uint64_t)tok[u] * y_ts + (uint64_t)head[u] * y_hs;
#pragma unroll
          for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (in[u] && ok[j][h]) {
                P o;
                narrow(f[j] + h * VEC, o);
                *reinterpret_cast<P*>(y + e[j][h]) = o;
              }
        }
      }
    }
  }

  if (MODE == NORM_GRAD) {
    // dw: the warp's groups, then the block's warps in order, one row of
    // partial sums per block; the second kernel adds the rows in a fixed order
    __shared__ float acc[THREADS / 32][MAX_D];
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i)
        for (int o = L; o < 32; o <<= 1) dw[j][i] += __shfl_xor_sync(0xffffffffu, dw[j][i], o);
    if ((threadIdx.x & 31) < L) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i)
          if (ok[j][i / VEC]) acc[threadIdx.x >> 5][e[j][i / VEC] + i % VEC] = dw[j][i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += THREADS) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < THREADS / 32; ++k) v += acc[k][d];
      a.partial[(int64_t)blockIdx.x * a.D + d] = v;
    }
  }
}

// dw[d] = sum of the blocks' partial rows; 32 columns per block, 32 row lanes.
__global__ void __launch_bounds__(1024) k_weight_grad(const float* partial, int32_t D,
                                                      int32_t blocks0, int32_t blocks1,
                                                      float* dw0, float* dw1) {
  __shared__ float acc[32][33];
  const int sd = blockIdx.y, d = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
  const int n = sd ? blocks1 : blocks0;
  const float* p = partial + (sd ? (int64_t)blocks0 * D : 0);
  float* dw = sd ? dw1 : dw0;
  float v = 0.0f;
  if (d < D)
    for (int r = lane; r < n; r += 32) v += p[(int64_t)r * D + d];
  acc[lane][threadIdx.x & 31] = v;
  __syncthreads();
  v = acc[threadIdx.x & 31][lane];  // lane now is the column
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0 && dw && blockIdx.x * 32 + lane < D) dw[blockIdx.x * 32 + lane] = v;
}

// ------------------------------------------------------------------ host side
bool aligned(const Side& s, int64_t bytes, int64_t elem, bool grad) {
  auto ok = [&](const void* p, int64_t a, int64_t b) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && a * elem % bytes == 0 &&
                  b * elem % bytes == 0);
  };
  return s.H == 0 || (ok(s.x, s.x_ts, s.x_hs) && ok(s.y, s.y_ts, s.y_hs) &&
                      (!grad || ok(s.dy, s.dy_ts, s.dy_hs)));
}

template <typename T, int VEC, int NS>
void launch_vec(int mode, const Args& a, int blocks, cudaStream_t st) {
  const int most = a.side[0].tokens > a.side[1].tokens ? a.side[0].tokens : a.side[1].tokens;
  const size_t smem = (size_t)most * a.rot * sizeof(float);
  if (mode == ROPE) k_rope<T, VEC, NS, ROPE><<<blocks, THREADS, smem, st>>>(a);
  else if (mode == NORM) k_rope<T, VEC, NS, NORM><<<blocks, THREADS, smem, st>>>(a);
  else k_rope<T, VEC, NS, NORM_GRAD><<<blocks, THREADS, smem, st>>>(a);
}

// VEC by alignment, NS by the slots a lane of 32 has to take (one where the row
// fits; the wider forms hold more registers).
template <typename T>
void launch_type(int mode, const Args& a, int vec, int slots, int blocks, cudaStream_t st) {
  constexpr int FULL = 16 / (int)sizeof(T);
  if (vec == FULL && slots <= 32) launch_vec<T, FULL, 1>(mode, a, blocks, st);
  else if (vec == 4 && slots <= 32) launch_vec<T, 4, 1>(mode, a, blocks, st);
  else if (vec >= 4) launch_vec<T, 4, 2>(mode, a, blocks, st);  // 4 elements: D <= 512 is 64 slots
  else if (vec == 2 && slots <= 32) launch_vec<T, 2, 1>(mode, a, blocks, st);
  else if (vec == 2) launch_vec<T, 2, 4>(mode, a, blocks, st);
  else if (slots <= 64) launch_vec<T, 1, 2>(mode, a, blocks, st);
  else launch_vec<T, 1, 8>(mode, a, blocks, st);
}

int device_check() {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TOPK_ERR_NO_DEVICE;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return TOPK_ERR_CUDA;
  return major == 10 && minor == 3 ? TOPK_OK : TOPK_ERR_NO_DEVICE;
}

int check(const Args& a, int64_t T, int32_t dtype, int mode) {
  if (T < 0 || a.D < 1 || a.rot < 0 || (a.rot & 1) || a.offset < 0 ||
      (int64_t)a.offset + a.rot > a.D || dtype < TOPK_BF16 || dtype > TOPK_FP32)
    return TOPK_ERR_ARG;
  if (a.D > MAX_D) return TOPK_ERR_UNSUPPORTED_SHAPE;
  const int64_t elem = dtype == TOPK_FP32 ? 4 : 2;
  for (int i = 0; i < 2; ++i) {
    const Side& s = a.side[i];
    if (s.H < 0 || T * (int64_t)s.H > INT32_MAX) return TOPK_ERR_ARG;
    if (T == 0 || s.H == 0) continue;
    if (!s.x || !s.y || (mode == NORM_GRAD && !s.dy)) return TOPK_ERR_ARG;
    if (!aligned(s, elem, elem, mode == NORM_GRAD)) return TOPK_ERR_ALIGN;
    for (int64_t d : {s.x_ts, s.x_hs, s.y_ts, s.y_hs, s.dy_ts, s.dy_hs})
      if (d < 0 || d > INT32_MAX) return TOPK_ERR_ARG;
    if (s.w && (reinterpret_cast<uintptr_t>(s.w) % (a.w32 ? 4 : elem))) return TOPK_ERR_ALIGN;
  }
  if (T > 0 && a.rot > 0 && (!a.pos || !a.freqs)) return TOPK_ERR_ARG;
  if (a.rot > 0 && ((reinterpret_cast<uintptr_t>(a.freqs) & 7u) ||
                    (reinterpret_cast<uintptr_t>(a.pos) & (a.pos64 ? 7u : 3u))))
    return TOPK_ERR_ALIGN;
  return TOPK_OK;
}

// Chooses the vector width and the tokens of a block, and launches.
int launch(Args& a, int64_t T, int32_t dtype, int mode, cudaStream_t st) {
  const int elem = dtype == TOPK_FP32 ? 4 : 2;
  int vec = 16 / elem;
  for (; vec > 1; vec >>= 1) {
    if (a.D % vec == 0 && a.offset % vec == 0 && a.rot % (2 * vec) == 0 &&
        aligned(a.side[0], (int64_t)vec * elem, elem, mode == NORM_GRAD) &&
        aligned(a.side[1], (int64_t)vec * elem, elem, mode == NORM_GRAD))
      break;
  }
  const int slots = a.rot / (2 * vec) + ((a.D - a.rot) / vec + 1) / 2;
  int L = 1;
  while (L < slots && L < 32) L <<= 1;
  a.lanes = L;
  a.T = T;
  a.w_vec = 1;
  for (int i = 0; i < 2; ++i)
    if (reinterpret_cast<uintptr_t>(a.side[i].w) % (vec * elem)) a.w_vec = 0;
  // Tokens of a block at a time: about 8 rows to a group (the gradient: 4, of its
  // side), the count near that whose rows fill the groups best, at most 16 KB of
  // sines and cosines (a block's rows also stay below 2^16, for inv_h), and fewer
  // while that leaves some of 152 SMs without two blocks.
  const int per_block = THREADS / L;
  const int H0 = a.side[0].H, H1 = a.side[1].H;
  auto rounds = [&](int64_t t, int h) { return (t * h + per_block - 1) / per_block; };
  auto tokens_for = [&](int h0, int h1, int each) {
    const int64_t most = a.rot > 0 ? 4096 / a.rot : INT32_MAX;
    const int64_t about = (int64_t)each * per_block / (h0 + h1);
    int64_t best = about < most ? about : most;
    for (int64_t t = about / 2 + 1; t <= about * 3 / 2 && t <= most; ++t)
      if ((rounds(t, h0) + rounds(t, h1)) * best < (rounds(best, h0) + rounds(best, h1)) * t)
        best = t;
    while (best > 1 && (T + best - 1) / best < 304) best >>= 1;
    return (int32_t)(best < 1 ? 1 : best);
  };
  int64_t blocks = 0;
  if (mode != NORM_GRAD) {
    a.side[0].tokens = a.side[1].tokens = tokens_for(H0, H1, 8);
    blocks = (T + a.side[0].tokens - 1) / a.side[0].tokens;
  } else {
    // Blocks by the sides' shares of the work: rounds of rows and passes over the
    // table.  By rows alone, with one count of tokens for both sides, the blocks of
    // a few key heads came last: 282 us for 104 us with 16384 tokens of 32 and 4
    // heads, 261 for 60 with 16 and 1 of 256.
    int64_t work[2] = {0, 0}, chunks[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
      Side& s = a.side[i];
      if (s.H == 0) continue;
      s.tokens = tokens_for(s.H, 0, 4);
      chunks[i] = (T + s.tokens - 1) / s.tokens;
      const int64_t passes = ((int64_t)s.tokens * a.rot / 2 + THREADS - 1) / THREADS;
      work[i] = chunks[i] * (TABLE_COST * rounds(s.tokens, s.H) + passes);
    }
    for (int i = 0; i < 2; ++i) {
      if (a.side[i].H == 0) continue;
      int64_t share = (MAX_BLOCKS * work[i] + (work[0] + work[1]) / 2) / (work[0] + work[1]);
      if (share < 1) share = 1;
      if (share > MAX_BLOCKS - 1 && work[1 - i] > 0) share = MAX_BLOCKS - 1;
      a.side[i].blocks = (int32_t)(chunks[i] < share ? chunks[i] : share);
      blocks += a.side[i].blocks;
    }
  }
  for (int i = 0; i < 2; ++i) {
    Side& s = a.side[i];
    // a block with one token: every row is of token 0
    s.inv_h = s.tokens <= 1 || s.H < 2 ? 0u : (uint32_t)((1ull << 32) / s.H + 1);
  }
  if (blocks > INT32_MAX) return TOPK_ERR_ARG;
  if (dtype == TOPK_BF16) launch_type<__nv_bfloat16>(mode, a, vec, slots, (int)blocks, st);
  else if (dtype == TOPK_FP16) launch_type<__half>(mode, a, vec, slots, (int)blocks, st);
  else launch_type<float>(mode, a, vec, slots, (int)blocks, st);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA;
}

void fill(Args& a, const void* pos, int32_t pos64, const int64_t* freqs, int32_t D, int32_t rot,
          int32_t offset, int32_t interleaved, float scale, float eps) {
  a.pos = pos;
  a.pos64 = pos64;
  a.freqs = freqs;
  a.D = D;
  a.rot = rot;
  a.offset = offset;
  a.interleaved = interleaved;
  a.scale = scale;
  a.eps = eps;
}

}  // namespace tr

extern "C" {

int topk_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* y,
              int64_t y_token_stride, int64_t y_head_stride, int64_t T, int32_t H, int32_t D,
              int32_t dtype, const void* positions, int32_t positions64, const int64_t* freqs,
              int32_t rot_dim, int32_t offset, int32_t interleaved, int32_t inverse, float scale,
              struct CUstream_st* stream) {
  tr::Args a{};
  a.side[0].x = x;
  a.side[0].x_ts = x_token_stride;
  a.side[0].x_hs = x_head_stride;
  a.side[0].y = y;
  a.side[0].y_ts = y_token_stride;
  a.side[0].y_hs = y_head_stride;
  a.side[0].H = H;
  a.inverse = inverse;
  tr::fill(a, positions, positions64, freqs, D, rot_dim, offset, interleaved, scale, 0.0f);
  int rc = tr::check(a, T, dtype, tr::ROPE);
  if (rc != TOPK_OK || T == 0 || H == 0) return rc;
  rc = tr::device_check();
  if (rc != TOPK_OK) return rc;
  return tr::launch(a, T, dtype, tr::ROPE, reinterpret_cast<cudaStream_t>(stream));
}

int topk_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t H,
                      const void* k, int64_t k_token_stride, int64_t k_head_stride, int32_t Hk,
                      const void* q_weight, const void* k_weight, int32_t weights_fp32,
                      void* q_out, int64_t qo_token_stride, int64_t qo_head_stride, void* k_out,
                      int64_t ko_token_stride, int64_t ko_head_stride, int64_t T, int32_t D,
                      int32_t dtype, const void* positions, int32_t positions64,
                      const int64_t* freqs, int32_t rot_dim, int32_t offset, int32_t interleaved,
                      float scale, float eps, struct CUstream_st* stream) {
  tr::Args a{};
  a.side[0] = {q, nullptr, q_out, q_weight, q_token_stride, q_head_stride, 0, 0,
               qo_token_stride, qo_head_stride, H, 0, 0};
  a.side[1] = {k, nullptr, k_out, k_weight, k_token_stride, k_head_stride, 0, 0,
               ko_token_stride, ko_head_stride, Hk, 0, 0};
  a.w32 = weights_fp32;
  tr::fill(a, positions, positions64, freqs, D, rot_dim, offset, interleaved, scale, eps);
  int rc = tr::check(a, T, dtype, tr::NORM);
  if (rc != TOPK_OK || T == 0 || (H == 0 && Hk == 0)) return rc;
  rc = tr::device_check();
  if (rc != TOPK_OK) return rc;
  return tr::launch(a, T, dtype, tr::NORM, reinterpret_cast<cudaStream_t>(stream));
}

size_t topk_qk_norm_rope_backward_workspace_bytes(int32_t D) {
  return D < 1 || D > tr::MAX_D ? 0 : (size_t)(tr::MAX_BLOCKS + 2) * D * sizeof(float);
}

int topk_qk_norm_rope_backward(
    const void* dq_out, int64_t dqo_token_stride, int64_t dqo_head_stride, const void* dk_out,
    int64_t dko_token_stride, int64_t dko_head_stride, const void* q, int64_t q_token_stride,
    int64_t q_head_stride, int32_t H, const void* k, int64_t k_token_stride, int64_t k_head_stride,
    int32_t Hk, const void* q_weight, const void* k_weight, int32_t weights_fp32, int64_t T,
    int32_t D, int32_t dtype, const void* positions, int32_t positions64, const int64_t* freqs,
    int32_t rot_dim, int32_t offset, int32_t interleaved, float scale, float eps, void* dq,
    void* dk, float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
    struct CUstream_st* stream) {
  tr::Args a{};
  a.side[0] = {q, dq_out, dq, q_weight, q_token_stride, q_head_stride, dqo_token_stride,
               dqo_head_stride, (int64_t)H * D, D, H, 0, 0};
  a.side[1] = {k, dk_out, dk, k_weight, k_token_stride, k_head_stride, dko_token_stride,
               dko_head_stride, (int64_t)Hk * D, D, Hk, 0, 0};
  a.w32 = weights_fp32;
  a.inverse = 1;
  tr::fill(a, positions, positions64, freqs, D, rot_dim, offset, interleaved, scale, eps);
  int rc = tr::check(a, T, dtype, tr::NORM_GRAD);
  if (rc != TOPK_OK) return rc;
  if ((reinterpret_cast<uintptr_t>(dq_weight) & 3u) || (reinterpret_cast<uintptr_t>(dk_weight) & 3u))
    return TOPK_ERR_ALIGN;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T > 0 && (H > 0 || Hk > 0)) {
    if (!workspace || workspace_bytes < topk_qk_norm_rope_backward_workspace_bytes(D))
      return TOPK_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 3u) return TOPK_ERR_ALIGN;
    a.partial = static_cast<float*>(workspace);
  }
  rc = tr::device_check();
  if (rc != TOPK_OK) return rc;
  if (T > 0 && (H > 0 || Hk > 0)) {
    rc = tr::launch(a, T, dtype, tr::NORM_GRAD, st);
    if (rc != TOPK_OK) return rc;
  }
  if (dq_weight || dk_weight) {
    // a side without rows has no blocks: its gradient is zero
    tr::k_weight_grad<<<dim3((D + 31) / 32, 2), 1024, 0, st>>>(
        a.partial, D, a.side[0].blocks, a.side[1].blocks, dq_weight, dk_weight);
  }
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA;
}

}  // extern "C"
