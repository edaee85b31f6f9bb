// The 8-bit cache: keys and values quantized as they are written, and read back.
//
// A page holds `page` tokens of one sequence; its tokens' rows of one head share
// one power-of-two scale 2^e for the keys and one for the values:
//   u = Pi x,  code = rne(u / 2^e),  e = the least with max|u| <= 127 * 2^e.
// A page that already holds tokens keeps its scale unless the new rows need a
// larger one; then its codes are halved as often as the scale doubled,
// code -> rne(code / 2^k).  Each such step adds at most half a step of the scale
// of its time, so no value is ever off by more than
// (1/2)(1 + 1/2 + 1/4 + ...) < 1 step of the scale that stands, in whatever
// portions the tokens came.  Powers of two make code * 2^e exact in bf16 and
// fp16 products, and the requantising exact integer work.
//
// Both directions are bound by memory for chunks and by latency for single tokens,
// if the turn costs little.  A warp turns 16 rows: half of the Hadamard transform
// (over four of a coordinate's bits) is a product with a 16 x 16 matrix of signs on
// the tensor cores (m16n8k16; the inputs are 16-bit values or codes, the entries 1,
// -1 and 0, the sums fp32: as exact as additions), the other bits are butterflies
// between accumulators.  Which bits: a lane's 16-byte piece of a row of codes is
// coordinates 64 j + 16 c + 4 w + e (c = lane % 4); the product of step (j, w) takes
// e and c together (bits 0, 1, 4, 5), so w and j (bits 2, 3, 6) stay between the
// lane's own accumulators, and it ends with the same 16 coordinates of the turned
// row: codes are read and written as they lie.  (With eight coordinates a lane and
// butterflies by shuffles, four times as many instructions, the write took 54 us and
// the read 42 us for 4608 tokens of 24 heads; now 52 us both (51 in a graph), 85 MB each.)  What is left
// above the 26 us of the bytes: the instructions of the turn (half of the issue slots)
// and, for the read, a page's scale before its codes; a step of 64 tokens waits for one
// chain of loads (page, scale, old codes).
//
// The permutation goes through shared memory on the 16-bit side, in 32-bit words of
// two rows (g and g + 8, as the product's operands and results have them).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "oq_cache.cuh"

namespace oq {
namespace {

using namespace cache;

constexpr int kThreads = 128;  // of the read kernel

__device__ __forceinline__ unsigned long long f2_add(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long f2_sub(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long f2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// c = a b
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
        "%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
        "%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two of four codes (bytes, sign bits turned) as fp16: see oq_cattn.cuh.
__device__ __forceinline__ uint32_t code_pair(uint32_t biased, uint32_t sel) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(biased, 0x64646464u, sel)), "r"(0x64806480u));
  return r;
}

// The 16 x 16 matrix of signs as two right operands (results e = 0, 1 and e = 2, 3):
// slot k of lane c stands for the coordinate bits (e, c), column n = 2 c' + b for
// (b + 2 tile, c').  Blocks of 32 leave bit 5 alone: entries between its halves are 0.
template <typename T>
__device__ __forceinline__ void sign_matrix(uint32_t (&m)[2][2], int lane, int h) {
  const int g = lane >> 2, c = lane & 3, c2 = g >> 1, b = g & 1;
  const uint32_t one = std::is_same<T, __nv_bfloat16>::value ? 0x3F80u : 0x3C00u;
  const bool zero = h == 32 && ((c ^ c2) & 2);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // slots 2 c, 2 c + 1: e = 0, 1; slots + 8: e = 2, 3
      uint32_t w = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t odd = (uint32_t)(__popc(c & (h == 32 ? 1 : 3) & c2) + (u & b) + (r & t)) & 1u;
        w |= (one | odd << 15) << (16 * u);
      }
      m[t][r] = zero ? 0u : w;
    }
}

// c = a b where the operand's lanes c < 2 and c >= 2 (`upper`) hold two blocks of 32 that
// may not meet: a zero entry times an infinity or a NaN would be NaN.  Each half by itself,
// of which a lane keeps its own half's results.
template <typename T>
__device__ __forceinline__ void mma_apart(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, bool upper) {
  float lo[4], hi[4];
  mma16816<T>(lo, upper ? 0u : a0, upper ? 0u : a1, upper ? 0u : a2, upper ? 0u : a3, b0, b1);
  mma16816<T>(hi, upper ? a0 : 0u, upper ? a1 : 0u, upper ? a2 : 0u, upper ? a3 : 0u, b0, b1);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = upper ? hi[i] : lo[i];
}

// The butterflies over bits 2, 3 and (blocks of 128) 6.
template <int KS>
__device__ __forceinline__ void butterflies(float (&acc)[KS][2][4], int h) {
#pragma unroll
  for (int s = 1; s < KS; s <<= 1) {
    if (s == 4 && h < 128) break;
#pragma unroll
    for (int k = 0; k < KS; ++k)
      if (!(k & s)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const unsigned long long a = f2(acc[k][t][i], acc[k][t][i + 1]);
            const unsigned long long b = f2(acc[k + s][t][i], acc[k + s][t][i + 1]);
            f2_split(f2_add(a, b), acc[k][t][i], acc[k][t][i + 1]);
            f2_split(f2_sub(a, b), acc[k + s][t][i], acc[k + s][t][i + 1]);
          }
      }
  }
}

struct WriteArgs {
  View c;
  Rotation r;
  const void* k;
  const void* v;
  long long kt, kh, vt, vh;  // strides in elements
  const int* cu;
  const int* past;
  const int* table;
  int* status;
  int B, T, width, units;
};

// The unit-th page that the sequences' new tokens touch; seq = -1 when there are
// fewer.  Each warp looks for itself.
struct Place {
  int seq, slot;  // sequence and the page's index in its table row
  int cu0, past, n;
};
template <int PLOG>
__device__ __forceinline__ Place find_place(const WriteArgs& a, int unit, bool report) {
  const int lane = threadIdx.x & 31;
  Place at;
  at.seq = -1, at.slot = 0, at.cu0 = 0, at.past = 0, at.n = 0;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 128) {
    int cu0[4], cu1[4], past[4];  // four groups of 32 sequences: their loads together
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int b = b0 + 32 * q + lane;
      const bool in = b < a.B;
      cu0[q] = in ? a.cu[b] : 0, cu1[q] = in ? a.cu[b + 1] : 0, past[q] = in ? a.past[b] : 0;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (b0 + 32 * q >= a.B) break;
      // a row of the batch whose numbers do not fit is left out, and reported
      const bool ok = cu0[q] >= 0 && cu1[q] >= cu0[q] && cu1[q] <= a.T && past[q] >= 0 &&
                      (long long)past[q] + (cu1[q] - cu0[q]) <= (long long)a.width << PLOG;
      const int n = ok ? cu1[q] - cu0[q] : 0;
      if (!ok && report) bad_index(a.status);
      const int pages = n > 0 ? ((past[q] + n - 1) >> PLOG) - (past[q] >> PLOG) + 1 : 0;
      int incl = pages;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        if (lane >= m) incl += o;
      }
      const int first = before + incl - pages;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, unit >= first && unit < first + pages);
      if (hit) {
        const int src = __ffs(hit) - 1;
        at.seq = b0 + 32 * q + src;
        at.cu0 = __shfl_sync(0xFFFFFFFFu, cu0[q], src);
        at.past = __shfl_sync(0xFFFFFFFFu, past[q], src);
        at.n = __shfl_sync(0xFFFFFFFFu, n, src);
        at.slot = (at.past >> PLOG) + (unit - __shfl_sync(0xFFFFFFFFu, first, src));
      }
      before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (unit < before && !report) break;
  }
  return at;
}

// WPU warps (one for every 16 tokens) write a page's rows of one head, keys or values.
// TURN: 0 none, 32 blocks of 32, 1 larger ones.  (Blocks of 32: the second product, taken
// only where something is not finite, is held to the first one's registers; 4608 tokens of
// 24 heads, written and read, 52.3 us against 50.9 without it, 53.7 if it were always taken.)
template <typename T, int D, int WPU, int TURN>
__global__ void __launch_bounds__(WPU < 4 ? 128 : 32 * WPU, TURN == 32 ? (D == 128 ? 5 : 8) / (WPU == 8 ? 2 : 1) : 0)
write_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int WARPS = WPU < 4 ? 4 : WPU, UNITS = WARPS / WPU, P = 16 * WPU;
  constexpr int KS = D / 16, PITCH = D + 4;  // words of a row pair in shared memory
  __shared__ __align__(16) uint32_t stage[WARPS][8 * PITCH];
  __shared__ uint32_t warp_top[WARPS];
  chain();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int unit = blockIdx.x * UNITS + warp / WPU, row0 = 16 * (warp % WPU);
  const int head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  Place at = find_place<WPU == 1 ? 4 : WPU == 2 ? 5 : WPU == 4 ? 6 : 7>(a, unit, blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && warp == 0);
  int page = 0;
  if (at.seq >= 0) {
    page = a.table[(size_t)at.seq * a.width + at.slot];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) bad_index(a.status);
      at.seq = -1;
      page = 0;
    }
  }
  const int start = at.slot * P;                                            // position of the page's first token
  const int held = at.seq < 0 ? 0 : min(max(at.past - start, 0), P);        // tokens it holds already
  const int end = at.seq < 0 ? 0 : min(at.past + at.n - start, P);          // and after this call
  const long long stride = values ? a.vt : a.kt;
  const long long first = (long long)at.cu0 + start - at.past;  // input row of the page's place 0
  uint32_t m[2][2];
  if constexpr (TURN != 0) sign_matrix<T>(m, lane, a.r.h);
  const T* src = static_cast<const T*>(values ? a.v : a.k) + head * (values ? a.vh : a.kh);
  float* scale = (values ? a.c.vs : a.c.ks) + (size_t)page * a.c.heads + head;
  const int e_old = held > 0 ? min(max(scale_exp(*scale), kExpMin), kExpMax) : kExpMin;
  const bool some = row0 < end && row0 + 16 > held;  // whether this warp has rows: the same for the warp

  // acc[4 j + w][t][i]: row g (i < 2) or g + 8, coordinate 64 j + 16 c + 4 w + 2 t + i % 2
  float acc[KS][2][4];
  if (some) {
    if constexpr (TURN != 0) {
      uint32_t* st = stage[warp];
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        const int id = lane + 32 * q, r = id / (D / 8), ch = id % (D / 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        const int lo = row0 + r, hi = lo + 8;
        if (lo >= held && lo < end) x = *reinterpret_cast<const uint4*>(src + (first + lo) * stride + 8 * ch);
        if (hi >= held && hi < end) y = *reinterpret_cast<const uint4*>(src + (first + hi) * stride + 8 * ch);
        uint4* to = reinterpret_cast<uint4*>(st + r * PITCH + 8 * ch);
        to[0] = make_uint4(__byte_perm(x.x, y.x, 0x5410), __byte_perm(x.x, y.x, 0x7632), __byte_perm(x.y, y.y, 0x5410),
                           __byte_perm(x.y, y.y, 0x7632));
        to[1] = make_uint4(__byte_perm(x.z, y.z, 0x5410), __byte_perm(x.z, y.z, 0x7632), __byte_perm(x.w, y.w, 0x5410),
                           __byte_perm(x.w, y.w, 0x7632));
      }
      __syncwarp();
      auto turn = [&](auto apart) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint4* pi = reinterpret_cast<const uint4*>(a.r.perm + 64 * j + 16 * c);
          const uint4 p0 = pi[0], p1 = pi[1];
          const uint32_t at16[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
          const uint32_t neg = a.r.signs[2 * j + (c >> 1)] >> (16 * (c & 1));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t lo[2], hi[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // e = 2 u, 2 u + 1
              const uint32_t p = at16[2 * w + u];
              const uint32_t w0 = st[g * PITCH + (p & 0xFFFFu)], w1 = st[g * PITCH + (p >> 16)];
              const uint32_t s2 = (neg >> (4 * w + 2 * u) & 3u) * 0x40008000u & 0x80008000u;  // two signs, to bits 15, 31
              lo[u] = __byte_perm(w0, w1, 0x5410) ^ s2;
              hi[u] = __byte_perm(w0, w1, 0x7632) ^ s2;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if constexpr (decltype(apart)::value)
                mma_apart<T>(acc[4 * j + w][t], lo[0], hi[0], lo[1], hi[1], m[t][0], m[t][1], c >= 2);
              else
                mma16816<T>(acc[4 * j + w][t], lo[0], hi[0], lo[1], hi[1], m[t][0], m[t][1]);
            }
          }
        }
        butterflies<KS>(acc, a.r.h);
      };
      turn(std::false_type());
      if constexpr (TURN == 32) {  // what is not finite may have come to a neighbouring block: once more
        bool nan = false;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) nan |= !(acc[k][t][i] == acc[k][t][i]);
        if (__any_sync(0xFFFFFFFFu, nan)) turn(std::true_type());
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + g + 8 * r;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (row >= held && row < end)
              y = *reinterpret_cast<const uint4*>(src + (first + row) * stride + 64 * j + 16 * c + 8 * u);
            float x[8];
            unpack8<T>(y, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[4 * j + 2 * u + (i >> 2)][(i >> 1) & 1][2 * r + (i & 1)] = x[i];
          }
      }
    }
  }
  // the largest magnitude; NaN counts as 0
  float top = 0.0f;
  if (some) {
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max_nan(top, fabsf(acc[k][t][i]));
    if (!(top == top)) {
      top = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = acc[k][t][i];
            if (!(x == x)) x = 0.0f;
            top = fmaxf(top, fabsf(x));
          }
    }
  }
  const uint32_t warp_most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
  if (lane == 0) warp_top[warp] = warp_most;
  __syncthreads();  // (the page's old scale was read before)
  uint32_t most = 0;
#pragma unroll
  for (int w = 0; w < WPU; ++w) most = max(most, warp_top[warp / WPU * WPU + w]);
  const float norm = TURN != 0 ? a.r.norm : 1.0f;
  const float amax = __uint_as_float(most) * norm;
  const int e = max(step_exp(amax), e_old);
  int8_t* dst = (values ? a.c.v : a.c.k) + ((size_t)page * a.c.heads + head) * P * D;

  if (held > 0 && e > e_old && end > 0) {  // the same for the page's warps
    const float f = pow2(e_old - e);
    for (int i = lane + 32 * (warp % WPU); i < held * (D / 4); i += 32 * WPU) {
      char4 v = reinterpret_cast<char4*>(dst)[i];
      v.x = (signed char)__float2int_rn((float)v.x * f);
      v.y = (signed char)__float2int_rn((float)v.y * f);
      v.z = (signed char)__float2int_rn((float)v.z * f);
      v.w = (signed char)__float2int_rn((float)v.w * f);
      reinterpret_cast<char4*>(dst)[i] = v;
    }
  }
  if (some) {
    // rne(u / 2^e) as the low byte of a sum with 1.5 * 2^23: one rounding, of the exact product
    const float to = norm * pow2(-e);
    if (amax > 127.0f * pow2(kExpMax)) {  // saturates
      const float lim = 127.0f * pow2(e) / norm;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[k][t][i] = fminf(fmaxf(acc[k][t][i], -lim), lim);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      const bool mine = row >= held && row < end;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(fmaf(acc[4 * j + w][i >> 1][2 * r + (i & 1)], to, 12582912.0f));
          o[w] = __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
        }
        if (mine) *reinterpret_cast<uint4*>(dst + (size_t)row * D + 64 * j + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (end > 0 && lane == 0 && warp % WPU == 0) *scale = pow2(e);
}

struct ReadArgs {
  View c;
  Rotation r;
  void* k;
  void* v;
  const int* cu;
  const int* first;
  const int* table;
  int* status;
  int B, T, width, heads_warp;
};

// A warp reads 16 output rows of heads_warp heads, keys or values.
template <typename T, int D, bool TURN>
__global__ void __launch_bounds__(kThreads, 4) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int KS = D / 16, PITCH = D + 4;
  __shared__ __align__(16) uint32_t stage[TURN ? kThreads / 32 : 1][8 * PITCH];
  chain();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int plog = 31 - __clz(a.c.page);
  uint32_t m[2][2];
  // where the lane's coordinates go, as byte offsets in a row of words; and the signs
  // of the eight coordinates that the lane stores in the end
  uint32_t to16[D / 64][8], flip[4];
  uint32_t* st = stage[TURN ? warp : 0];
  char* my_row = reinterpret_cast<char*>(st + g * PITCH);
  if constexpr (TURN) {
    sign_matrix<__half>(m, lane, a.r.h);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint4* pi = reinterpret_cast<const uint4*>(a.r.perm + 64 * j + 16 * c);
      const uint4 p0 = pi[0], p1 = pi[1];
      const uint32_t p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
      const uint32_t neg = a.r.signs[2 * j + (c >> 1)] >> (16 * (c & 1));
#pragma unroll
      for (int i = 0; i < 8; ++i) to16[j][i] = p[i] << 2;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<uint32_t*>(my_row + (i & 1 ? to16[j][i >> 1] >> 16 : to16[j][i >> 1] & 0xFFFFu)) = neg >> i & 1u;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      flip[i] = st[8 * (lane % (D / 8)) + 2 * i] << 15 | st[8 * (lane % (D / 8)) + 2 * i + 1] << 31;
  }

  const bool values = blockIdx.z != 0;
  const int t0 = (int)(blockIdx.x * (kThreads / 32) + warp) * 16;
  if (t0 >= a.T) return;  // (no barrier of the CTA below)
  const int h0 = blockIdx.y * a.heads_warp, h1 = min(h0 + a.heads_warp, a.c.heads);
  // the sequence of the first row: how many end at or before it.  Sequences from the first
  // on whose offsets fall or leave the tensor (`last`) are left out, so the ends that are
  // counted rise.
  const bool report = (blockIdx.x | blockIdx.y | blockIdx.z) == 0 && warp == 0;
  int before = 0, last = a.B;
  for (int b0 = 0; b0 < last; b0 += 128) {
    int s[4], e[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int b = b0 + 32 * q + lane;
      s[q] = b < a.B ? a.cu[b] : 0;
      e[q] = b < a.B ? a.cu[b + 1] : a.T;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (b0 + 32 * q >= last) break;
      const bool off = e[q] < s[q] || e[q] > a.T;
      if (report && (off || s[q] < 0)) bad_index(a.status);
      const uint32_t bad = __ballot_sync(0xFFFFFFFFu, off), ended = __ballot_sync(0xFFFFFFFFu, e[q] <= t0);
      if (bad) last = b0 + 32 * q + __ffs(bad) - 1;
      before += __popc(ended & ((bad & (0u - bad)) - 1u));  // (no bad one: all)
    }
  }
  // row of codes (page * page size + place) of the lane's row, or -1; lanes 16.. stand for nothing
  int at = -1;
  if (lane < 16 && t0 + lane < a.T) {
    const int t = t0 + lane;
    int b = before;
    while (b < last && a.cu[b + 1] <= t) ++b;
    const int from = b < last ? a.cu[b] : -1;
    if (from >= 0 && t >= from) {
      const long long p = (long long)a.first[b] + (t - from);
      if (p >= 0 && p < (long long)a.width * a.c.page) {
        const int page = a.table[(size_t)b * a.width + (int)(p >> plog)];
        if (page >= 0 && page < a.c.n_pages) at = (page << plog) + ((int)p & (a.c.page - 1));
      }
      if (at < 0) bad_index(a.status);
    }
  }
  const int at0 = __shfl_sync(0xFFFFFFFFu, at, g), at1 = __shfl_sync(0xFFFFFFFFu, at, g + 8);
  const int8_t* codes = values ? a.c.v : a.c.k;
  const float* scales = values ? a.c.vs : a.c.ks;
  T* out = static_cast<T*>(values ? a.v : a.k);
  // the codes and scales of the lane's two rows, fetched a head ahead
  uint4 next[2][D / 64];
  float next_f[2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = r ? at1 : at0;
      next_f[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) next[r][j] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= 0) {
        const size_t ph = (size_t)(row >> plog) * a.c.heads + h;
        const int8_t* from = codes + ((ph << plog) + (row & (a.c.page - 1))) * D + 16 * c;
        next_f[r] = scales[ph];
#pragma unroll
        for (int j = 0; j < D / 64; ++j) next[r][j] = *reinterpret_cast<const uint4*>(from + 64 * j);
      }
    }
  };
  fetch(h0);
  for (int h = h0; h < h1; ++h) {
    uint4 w0[D / 64], w1[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) w0[j] = next[0][j], w1[j] = next[1][j];
    float f0 = next_f[0], f1 = next_f[1];
    if (h + 1 < h1) fetch(h + 1);
    if constexpr (TURN) {
      float acc[KS][2][4];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint32_t x[4] = {w0[j].x, w0[j].y, w0[j].z, w0[j].w}, y[4] = {w1[j].x, w1[j].y, w1[j].z, w1[j].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t x8 = x[w] ^ 0x80808080u, y8 = y[w] ^ 0x80808080u;
          const uint32_t a0 = code_pair(x8, 0x4140), a1 = code_pair(y8, 0x4140), a2 = code_pair(x8, 0x4342),
                         a3 = code_pair(y8, 0x4342);
#pragma unroll
          for (int t = 0; t < 2; ++t) mma16816<__half>(acc[4 * j + w][t], a0, a1, a2, a3, m[t][0], m[t][1]);
        }
      }
      butterflies<KS>(acc, a.r.h);
      f0 *= a.r.norm, f1 *= a.r.norm;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float* v = acc[4 * j + (i >> 2)][(i >> 1) & 1];
          *reinterpret_cast<uint32_t*>(my_row + (i & 1 ? to16[j][i >> 1] >> 16 : to16[j][i >> 1] & 0xFFFFu)) =
              pack2<T>(v[i & 1] * f0, v[2 + (i & 1)] * f1);
        }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        const int id = lane + 32 * q, r = id / (D / 8), ch = id % (D / 8);
        const uint4* from = reinterpret_cast<const uint4*>(st + r * PITCH + 8 * ch);
        const uint4 x = from[0], y = from[1];
        const int lo = __shfl_sync(0xFFFFFFFFu, at, r), hi = __shfl_sync(0xFFFFFFFFu, at, r + 8);
        T* to = out + ((size_t)(t0 + r) * a.c.heads + h) * D + 8 * ch;
        if (lo >= 0)
          *reinterpret_cast<uint4*>(to) =
              make_uint4(__byte_perm(x.x, x.y, 0x5410) ^ flip[0], __byte_perm(x.z, x.w, 0x5410) ^ flip[1],
                         __byte_perm(y.x, y.y, 0x5410) ^ flip[2], __byte_perm(y.z, y.w, 0x5410) ^ flip[3]);
        if (hi >= 0)
          *reinterpret_cast<uint4*>(to + (size_t)8 * a.c.heads * D) =
              make_uint4(__byte_perm(x.x, x.y, 0x7632) ^ flip[0], __byte_perm(x.z, x.w, 0x7632) ^ flip[1],
                         __byte_perm(y.x, y.y, 0x7632) ^ flip[2], __byte_perm(y.z, y.w, 0x7632) ^ flip[3]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if ((r ? at1 : at0) < 0) continue;
        const float f = r ? f1 : f0;
        T* to = out + ((size_t)(t0 + g + 8 * r) * a.c.heads + h) * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint4 w = r ? w1[j] : w0[j];
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)(int)(signed char)(x[2 * u + (i >> 2)] >> (8 * (i & 3))) * f;
            *reinterpret_cast<uint4*>(to + 64 * j + 16 * c + 8 * u) = pack8<T>(v);
          }
        }
      }
    }
  }
}

View view_of(const oq_kvcache* c) {
  View v;
  v.k = c->k, v.v = c->v, v.ks = c->k_scale, v.vs = c->v_scale;
  v.n_pages = c->n_pages, v.heads = c->heads, v.page = c->page;
  return v;
}

}  // namespace

int cache_rotation(oq_rpbh_t r, void* rotation) {
  cache::Rotation& q = *static_cast<cache::Rotation*>(rotation);
  std::memset(&q, 0, sizeof(q));
  if (!r) return OQ_OK;
  if (int rc = rpbh_device_tables(r, &q.perm, &q.signs)) return rc;
  q.h = r->h;
  q.norm = (float)(1.0 / std::sqrt((double)r->h));
  return OQ_OK;
}

int launch_cache_write(const CacheCall& c) {
  WriteArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = view_of(c.cache);
  if (int rc = cache_rotation(c.r, &a.r)) return rc;
  if (int rc = device_status_word(&a.status)) return rc;
  a.k = c.k, a.v = c.v;
  a.kt = c.k_token, a.kh = c.k_head, a.vt = c.v_token, a.vh = c.v_head;
  a.cu = c.cu, a.past = c.at, a.table = c.table;
  a.B = c.B, a.T = c.T, a.width = c.width;
  const int P = c.cache->page, D = c.cache->d;
  // pages touched: at least one token each, and at most two partly filled for each sequence
  a.units = (int)std::min<long long>(c.T, (long long)c.T / P + 2ll * c.B);
  const int wpu = P / 16, per_cta = wpu < 4 ? 4 / wpu : 1;
  const dim3 grid((unsigned)((a.units + per_cta - 1) / per_cta), (unsigned)c.cache->heads, 2u);
  const int threads = wpu < 4 ? 128 : 32 * wpu;
  int rc = OQ_OK;
  auto go = [&](auto kern) { rc = launch_chained("cache write", kern, grid, threads, 0, c.stream, a); };
#define OQ_WRITE(T, DD, W) \
  !a.r.perm ? go(write_kernel<T, DD, W, 0>) : a.r.h == 32 ? go(write_kernel<T, DD, W, 32>) : go(write_kernel<T, DD, W, 1>)
#define OQ_WARPS(T, DD)                    \
  switch (wpu) {                           \
    case 1: OQ_WRITE(T, DD, 1); break;     \
    case 2: OQ_WRITE(T, DD, 2); break;     \
    case 4: OQ_WRITE(T, DD, 4); break;     \
    default: OQ_WRITE(T, DD, 8); break;    \
  }
  if (c.dtype == OQ_BF16) {
    if (D == 128) OQ_WARPS(__nv_bfloat16, 128) else OQ_WARPS(__nv_bfloat16, 64)
  } else {
    if (D == 128) OQ_WARPS(__half, 128) else OQ_WARPS(__half, 64)
  }
#undef OQ_WARPS
#undef OQ_WRITE
  return rc;
}

int launch_cache_read(const CacheCall& c) {
  ReadArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = view_of(c.cache);
  if (int rc = cache_rotation(c.r, &a.r)) return rc;
  if (int rc = device_status_word(&a.status)) return rc;
  a.k = c.k_out, a.v = c.v_out;
  a.cu = c.cu, a.first = c.at, a.table = c.table;
  a.B = c.B, a.T = c.T, a.width = c.width;
  const int D = c.cache->d;
  int nsm;
  if (int rc = sm_count(&nsm)) return rc;
  // A warp finds its rows' places (and what it keeps for the turn) once for several
  // heads, as long as there are 32 warps for each SM.  Measured, 4608 rows of 24 heads
  // with the turn: 1, 2, 3, 8 heads a warp 58, 52, 50, 49 us (write and read); 46
  // thousand rows of 8 narrow heads: 59, 44, 42, 38 us; without the turn 33, 30, 30, 40.
  const long long tiles = (c.T + 15) / 16;
  a.heads_warp = (int)std::max<long long>(1, std::min<long long>(a.r.perm ? 8 : 2, 2 * tiles * c.cache->heads / (32ll * nsm)));
  const dim3 grid((unsigned)((tiles + kThreads / 32 - 1) / (kThreads / 32)),
                  (unsigned)((c.cache->heads + a.heads_warp - 1) / a.heads_warp), 2u);
  int rc = OQ_OK;
  auto go = [&](auto kern) { rc = launch_chained("cache read", kern, grid, kThreads, 0, c.stream, a); };
#define OQ_READ(T, DD) a.r.perm ? go(read_kernel<T, DD, true>) : go(read_kernel<T, DD, false>)
  if (c.dtype == OQ_BF16) {
    if (D == 128) OQ_READ(__nv_bfloat16, 128);
    else OQ_READ(__nv_bfloat16, 64);
  } else {
    if (D == 128) OQ_READ(__half, 128);
    else OQ_READ(__half, 64);
  }
#undef OQ_READ
  return rc;
}

}  // namespace oq
