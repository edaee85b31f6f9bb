// Device helpers shared by the cache kernels (write, read back, attention).
//
// A row of head width D (64 or 128) is held by D / 8 neighbouring lanes, eight
// coordinates each: coordinate 8 l + i in register i of lane l of the row.  The
// block-Hadamard butterflies of strides 1, 2, 4 then stay in registers and the
// strides 8 .. h/2 are lane-xor shuffles.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "oq_internal.h"

namespace oq {
namespace cache {

// Exponents a page's scale may take: |value| <= 127 * 2^40 is held, steps below
// 2^-40 are not resolved.  The bounds keep 2^(e_max - e_min) and its products
// with exponentials of either sign inside fp32.
constexpr int kExpMin = -40, kExpMax = 40;

// Programmatic dependent launch: a kernel may start while the one before it in the
// stream finishes.  Every thread of these kernels first waits for that one's end
// (so the one after may rely on both), then lets the next one start: at once where
// the kernel is short, at its end where the next one's waiting blocks would take
// room beside a long one.
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain() {
  chain_wait();
  chain_next();
}
template <typename Kernel, typename... A>
int launch_chained(const char* what, Kernel kern, dim3 grid, int threads, size_t smem, void* stream, const A&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e == cudaSuccess ? OQ_OK : fail(OQ_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

struct Rotation {
  const uint16_t* perm;   // pi, or nullptr for no rotation
  const uint32_t* signs;  // bit j%32 of word j/32: sign_j = -1
  int h;
  float norm;  // 1 / sqrt(h)
};

struct View {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  int n_pages, heads, page;
};

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// Exponent of a power-of-two scale (any other bit pattern gives a finite value too).
__device__ __forceinline__ int scale_exp(float s) { return (int)((__float_as_uint(s) >> 23) & 0xFFu) - 127; }

// The least e with amax <= 127 * 2^e, within the bounds: with amax in
// [2^x, 2^(x+1)) that is x - 6 up to amax = (127/64) 2^x and x - 5 above.
__device__ __forceinline__ int step_exp(float amax) {
  const uint32_t b = __float_as_uint(amax) & 0x7FFFFFFFu;
  const int x = (int)(b >> 23) - 127;
  const int e = (b & 0x7FFFFFu) <= 0x7E0000u ? x - 6 : x - 5;  // 0x7E0000: the mantissa of 127/64
  return min(max(e, kExpMin), kExpMax);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);  // a in the low half
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  float2 t;
  t = unpack2<T>(w.x), x[0] = t.x, x[1] = t.y;
  t = unpack2<T>(w.y), x[2] = t.x, x[3] = t.y;
  t = unpack2<T>(w.z), x[4] = t.x, x[5] = t.y;
  t = unpack2<T>(w.w), x[6] = t.x, x[7] = t.y;
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// Eight coordinates of one lane: their gather places and signs, kept over the rows.
struct LaneTurn {
  uint32_t at[4];  // pi of coordinates 2 i (low half) and 2 i + 1
  uint32_t neg;    // bit i: coordinate i is negated
};
__device__ __forceinline__ LaneTurn lane_turn(const Rotation& r, int l) {
  LaneTurn t;
  if (r.perm) {
    const uint4 p = *reinterpret_cast<const uint4*>(r.perm + 8 * l);
    t.at[0] = p.x, t.at[1] = p.y, t.at[2] = p.z, t.at[3] = p.w;
    t.neg = (r.signs[l >> 2] >> (8 * (l & 3))) & 0xFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) t.at[i] = 0u;
    t.neg = 0u;
  }
  return t;
}
__device__ __forceinline__ int turn_at(const LaneTurn& t, int i) {
  return (int)((i & 1) ? t.at[i >> 1] >> 16 : t.at[i >> 1] & 0xFFFFu);
}

// Unnormalised Hadamard transform of every block of h coordinates (h = 32, 64
// or 128; all lanes of the warp take part).
__device__ __forceinline__ void fwht8(float (&x)[8], int l, int h) {
#pragma unroll
  for (int s = 1; s < 8; s <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & s)) {
        const float a = x[i], b = x[i + s];
        x[i] = a + b;
        x[i + s] = a - b;
      }
#pragma unroll
  for (int m = 1; m <= 8; m <<= 1) {
    if (8 * m < h) {
      const float sg = (l & m) ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(sg, x[i], __shfl_xor_sync(0xFFFFFFFFu, x[i], m));
    }
  }
}

// u = Pi x of the row of 16-bit values at `row` (shared memory, written by the row's
// lanes before a __syncwarp).
template <typename T>
__device__ __forceinline__ void rotate_row(const T* row, const LaneTurn& t, int l, const Rotation& rot, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = (float)row[turn_at(t, i)];
    x[i] = (t.neg >> i & 1u) ? -v : v;
  }
  fwht8(x, l, rot.h);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= rot.norm;
}

// x = Pi^T u: the transposed turn scatters the values, rounded to T, into the
// row at `row` (shared memory; the row's lanes read it after a __syncwarp).
template <typename T>
__device__ __forceinline__ void unrotate_row(float (&x)[8], const LaneTurn& t, int l, const Rotation& rot, T* row) {
  fwht8(x, l, rot.h);
#pragma unroll
  for (int i = 0; i < 8; ++i) row[turn_at(t, i)] = (T)(x[i] * ((t.neg >> i & 1u) ? -rot.norm : rot.norm));
}

// Records that an index on the device (a page, a length) was out of range.
__device__ __forceinline__ void bad_index(int* status) { atomicExch(status, OQ_ERR_ARG); }

}  // namespace cache
}  // namespace oq
