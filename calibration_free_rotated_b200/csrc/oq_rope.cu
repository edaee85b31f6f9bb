// Rotary positions over several axes.
//
// Pair p of a head turns by phi = pos[t][axis_p] * f_p:
//   (a, b) -> (a cos phi - b sin phi, a sin phi + b cos phi)
// (the transposed turn, phi -> -phi, is the inverse and the gradient).
// The angle is exact for far positions: f_p is held in turns per position as a
// 64-bit fraction F = round(f_p / 2pi * 2^64), and pos * F mod 2^64 is the
// turn's fraction with an error below |pos| * 2^-65, reduced without a float
// division; rounded to fp32 (a small angle keeps its 24 bits) it goes through sincospif.
//
// Bound by memory (each value is read and written once).  A CTA takes a few
// tokens and a share of the heads: its threads first put the tokens' cosines
// and sines into shared memory (once for all heads), then each thread turns
// pairs of 16-byte vectors, two units under way at a time.  Inside a captured graph: 4608
// tokens, 48 heads of 128, bf16: 113 MB in 20.5 us, 5.5 TB/s; 32760 tokens, 24 heads, fp16:
// 403 MB in 67 us, 6.0 TB/s (halves: 19 and 64 us); a batch's step of 64 tokens: 2 us, the
// launch's latency.  In calls one by one 21.8, 73 and 6.5 us.
// (One unit at a time, neighbouring vectors and turns in plain order, read with four-way
// bank conflicts: 26 and 77 us.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "oq_cache.cuh"

namespace oq {
namespace {

using namespace cache;

constexpr int kThreads = 256;

struct RopeArgs {
  const char* x;
  char* y;
  const unsigned long long* freq;  // [pairs]
  const uint8_t* axis;             // [pairs]
  const int* pos;                  // [T][n_axes]
  long long xt, xh, yt, yh;        // strides in bytes
  int T, heads, n_axes, pairs, halves, inverse;
  int tokens, head_share;   // per CTA
  int units;                // vector pairs of a row
  unsigned div_units;       // ceil(2^32 / units)
};

template <typename T>
struct Vec;  // 16 bytes of T
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(uint4 w, float (&x)[8]) { unpack8<__nv_bfloat16>(w, x); }
  static __device__ __forceinline__ uint4 store(const float (&x)[8]) { return pack8<__nv_bfloat16>(x); }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(uint4 w, float (&x)[8]) { unpack8<__half>(w, x); }
  static __device__ __forceinline__ uint4 store(const float (&x)[8]) { return pack8<__half>(x); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(uint4 w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// Where pair p of a token has its turn: a thread's eight lanes' pieces lie 64 bytes apart,
// so 16-byte pieces are swapped within 64 bytes, and the eight come from different banks.
__device__ __forceinline__ int turn_at(int p) { return p ^ ((p >> 4 & 3) << 1); }

// A row's 16-byte vectors in units of two: HALVES: unit u < pairs / N holds the
// vectors N u and pairs + N u that turn into each other, the others what lies behind
// the turned part, two neighbouring vectors; otherwise vector u and the one half a row
// further on, so that lanes beside one another read what lies side by side.  An odd
// vector at the end stands alone.  A thread has two units under way, the first two
// while the token's turns are made.
template <typename T, bool HALVES>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int vecs) {
  constexpr int N = Vec<T>::N, BATCH = 2;
  extern __shared__ __align__(16) float2 turns[];  // [tokens][turn_at(pair)]
  chain();
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.T - t0);
  const int h0 = blockIdx.y * a.head_share, nh = min(a.head_share, a.heads - h0);
  const int row_units = a.units, total = nt * nh * row_units, stride = (a.pairs + 7) & ~7;
  const int first_pass = HALVES ? a.pairs / N : 0;  // units that pair two halves
  uint4 w[BATCH][2];
  int token[BATCH], unit[BATCH];
  char* to[BATCH];
  auto load = [&](int i, int k) {
    const int row = row_units == 1 ? i : (int)__umulhi((unsigned)i, a.div_units);
    const int u = i - row * row_units;
    const int t = row / nh, h = row - t * nh;
    const char* x = a.x + (t0 + t) * a.xt + (h0 + h) * a.xh;
    to[k] = a.y + (t0 + t) * a.yt + (h0 + h) * a.yh;
    token[k] = t, unit[k] = u;
    const bool pass = HALVES && u < first_pass;
    const int v0 = pass || !HALVES ? u : 2 * u, v1 = pass ? u + first_pass : HALVES ? v0 + 1 : u + row_units;
    w[k][0] = *reinterpret_cast<const uint4*>(x + 16 * v0);
    if (v1 < vecs) w[k][1] = *reinterpret_cast<const uint4*>(x + 16 * v1);
  };
#pragma unroll
  for (int k = 0; k < BATCH; ++k)
    if (threadIdx.x + k * kThreads < total) load(threadIdx.x + k * kThreads, k);
  for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
    const int t = i / a.pairs, p = i - t * a.pairs;
    const long long pos = a.pos[(size_t)(t0 + t) * a.n_axes + a.axis[p]];
    const unsigned long long turn = (unsigned long long)pos * a.freq[p];
    float s, c;
    sincospif((float)(long long)turn * 0x1p-63f, &s, &c);
    turns[t * stride + turn_at(p)] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < total; i0 += BATCH * kThreads) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (i0 + k * kThreads >= total) continue;
      const int u = unit[k];
      const float2* cs = turns + token[k] * stride;
      char* y = to[k];
      if (HALVES && u < first_pass) {
        float p[N], q[N];
        Vec<T>::load(w[k][0], p);
        Vec<T>::load(w[k][1], q);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float4 r = *reinterpret_cast<const float4*>(cs + turn_at(u * N + e));
          const float b0 = q[e], b1 = q[e + 1];
          q[e] = fmaf(p[e], r.y, b0 * r.x);
          p[e] = fmaf(p[e], r.x, -(b0 * r.y));
          q[e + 1] = fmaf(p[e + 1], r.w, b1 * r.z);
          p[e + 1] = fmaf(p[e + 1], r.z, -(b1 * r.w));
        }
        *reinterpret_cast<uint4*>(y + 16 * u) = Vec<T>::store(p);
        *reinterpret_cast<uint4*>(y + 16 * (u + first_pass)) = Vec<T>::store(q);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int v = HALVES ? 2 * u + j : u + j * row_units;
          if (v >= vecs) break;
          const int p0 = v * (N / 2);
          uint4 now4 = w[k][j];
          if (!HALVES && p0 < a.pairs) {  // the rest is carried over bit for bit
            float p[N];
            Vec<T>::load(now4, p);
#pragma unroll
            for (int e = 0; e < N / 2; e += 2) {
              const float4 r = *reinterpret_cast<const float4*>(cs + turn_at(p0 + e));
              const float b0 = p[2 * e + 1], b1 = p[2 * e + 3];
              p[2 * e + 1] = fmaf(p[2 * e], r.y, b0 * r.x);
              p[2 * e] = fmaf(p[2 * e], r.x, -(b0 * r.y));
              p[2 * e + 3] = fmaf(p[2 * e + 2], r.w, b1 * r.z);
              p[2 * e + 2] = fmaf(p[2 * e + 2], r.z, -(b1 * r.w));
            }
            now4 = Vec<T>::store(p);
            if (p0 + N / 2 > a.pairs) {  // the turned part ends inside this vector
              const uint32_t* old = &w[k][j].x;
              uint32_t* now = &now4.x;
              constexpr int words = (int)(sizeof(T) / 2);  // words of a pair
#pragma unroll
              for (int e = 0; e < N / 2; ++e)
#pragma unroll
                for (int x = 0; x < words; ++x)
                  if (p0 + e >= a.pairs) now[e * words + x] = old[e * words + x];
            }
          }
          *reinterpret_cast<uint4*>(y + 16 * v) = now4;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (i0 + (BATCH + k) * kThreads < total) load(i0 + (BATCH + k) * kThreads, k);
  }
}

}  // namespace

int launch_rope(const RopeCall& c) {
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  const int size = c.dtype == OQ_FP32 ? 4 : 2;
  a.x = static_cast<const char*>(c.x);
  a.y = static_cast<char*>(c.y);
  a.freq = c.freq;
  a.axis = c.axis;
  a.pos = c.pos;
  a.xt = c.x_token * size, a.xh = c.x_head * size, a.yt = c.y_token * size, a.yh = c.y_head * size;
  a.T = c.T, a.heads = c.heads, a.n_axes = c.n_axes, a.pairs = c.pairs, a.halves = c.halves, a.inverse = c.inverse;
  const int vecs = c.d * size / 16, n = 16 / size;
  const int lead = c.halves ? c.pairs / n : 0;
  a.units = lead + (vecs - 2 * lead + 1) / 2;
  a.div_units = (unsigned)((0x100000000ull + a.units - 1) / a.units);
  int nsm;
  if (int rc = sm_count(&nsm)) return rc;
  // A CTA turns about 1024 units (four a thread); with few tokens the heads are
  // shared out so that every SM has work.
  const int per_token = c.heads * a.units;
  a.tokens = std::max(1, std::min({1024 / std::max(1, per_token), 16, (c.T + nsm - 1) / nsm}));
  a.tokens = std::min(a.tokens, 4096 / a.pairs);
  int blocks = (c.T + a.tokens - 1) / a.tokens;
  int shares = std::max(1, std::max(std::min(c.heads, (2 * nsm) / blocks), (a.tokens * per_token + 2047) / 2048));
  shares = std::min(shares, std::min(c.heads, 65535));
  a.head_share = (c.heads + shares - 1) / shares;
  const dim3 grid((unsigned)blocks, (unsigned)((c.heads + a.head_share - 1) / a.head_share));
  const size_t smem = sizeof(float2) * (size_t)a.tokens * ((a.pairs + 7) & ~7);
  auto go = [&](auto kern) { return launch_chained("rope", kern, grid, kThreads, smem, c.stream, a, vecs); };
  if (c.dtype == OQ_BF16) return c.halves ? go(rope_kernel<__nv_bfloat16, true>) : go(rope_kernel<__nv_bfloat16, false>);
  if (c.dtype == OQ_FP16) return c.halves ? go(rope_kernel<__half, true>) : go(rope_kernel<__half, false>);
  return c.halves ? go(rope_kernel<float, true>) : go(rope_kernel<float, false>);
}

}  // namespace oq
