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
// Writing: a CTA takes one page, one head, keys or values.  Its rows' rotated
// values stay in registers between the two steps (the maximum, then the codes),
// so each input is read once.  Reading back: a CTA takes some rows of one head.
// Both are bound by memory for chunks and by latency for single tokens.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "oq_cache.cuh"

namespace oq {
namespace {

using namespace cache;

constexpr int kThreads = 256;

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
  int B, T, width;
};

// Finds the unit-th page that the sequences' new tokens touch.  All threads
// return the same answer; seq = -1 when there are fewer.
struct Place {
  int seq, slot;   // sequence and the page's index in its table row
  int cu0, past, n;
};
__device__ Place find_place(const WriteArgs& a, int unit, bool report) {
  __shared__ int warp_sum[kThreads / 32];
  __shared__ Place found;
  if (threadIdx.x == 0) found.seq = -1;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int cu0 = 0, n = 0, past = 0, pages = 0;
    if (b < a.B) {
      cu0 = a.cu[b];
      const int cu1 = a.cu[b + 1];
      past = a.past[b];
      // a row of the batch whose numbers do not fit is left out, and reported
      const bool ok = cu0 >= 0 && cu1 >= cu0 && cu1 <= a.T && past >= 0 &&
                      (long long)past + (cu1 - cu0) <= (long long)a.width * a.c.page;
      n = ok ? cu1 - cu0 : 0;
      if (!ok && report) bad_index(a.status);
      if (n > 0) pages = (past + n - 1) / a.c.page - past / a.c.page + 1;
    }
    int incl = pages;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
      if (lane >= m) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int base = before, all = before;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += warp_sum[w];
      all += warp_sum[w];
    }
    const int first = base + incl - pages;
    if (unit >= first && unit < first + pages) {
      found.seq = b;
      found.slot = past / a.c.page + (unit - first);
      found.cu0 = cu0, found.past = past, found.n = n;
    }
    __syncthreads();
    before = all;
    if (unit < all && !report) break;  // the same for all threads
  }
  return found;
}

template <typename T, int D, int PASSES>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int LPR = D / 8;               // lanes of a row
  constexpr int ROWS = kThreads / LPR;     // rows of a pass
  __shared__ __align__(16) T stage[ROWS][D];
  __shared__ float warp_max[kThreads / 32];
  const int head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const Place at = find_place(a, blockIdx.x, blockIdx.y == 0 && blockIdx.z == 0 && blockIdx.x == 0);
  if (at.seq < 0) return;
  const int page = a.table[(size_t)at.seq * a.width + at.slot];
  if (page < 0 || page >= a.c.n_pages) {
    if (threadIdx.x == 0) bad_index(a.status);
    return;
  }
  const int P = a.c.page;
  const int start = at.slot * P;                        // position of the page's first token
  const int held = min(max(at.past - start, 0), P);     // tokens it holds already
  const int end = min(at.past + at.n - start, P);       // and after this call
  const int l = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const T* src = static_cast<const T*>(values ? a.v : a.k) + head * (values ? a.vh : a.kh) + 8 * l;
  const long long stride = values ? a.vt : a.kt;
  const long long first = (long long)at.cu0 + start - at.past;  // input row of the page's place 0
  const LaneTurn turn = lane_turn(a.r, l);

  float u[PASSES][8];
  float top = 0.0f;
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    const int row = held + q * ROWS + r0;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (row < end) w = *reinterpret_cast<const uint4*>(src + (first + row) * stride);
    if (a.r.perm) {
      *reinterpret_cast<uint4*>(&stage[r0][8 * l]) = w;
      __syncwarp();
      rotate_row<T>(stage[r0], turn, l, a.r, u[q]);
      __syncwarp();
    } else {
      unpack8<T>(w, u[q]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(u[q][i]));
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
  float* scale = (values ? a.c.vs : a.c.ks) + (size_t)page * a.c.heads + head;
  const int e_old = held > 0 ? min(max(scale_exp(*scale), kExpMin), kExpMax) : kExpMin;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, warp_max[w]);
  const int e = max(step_exp(top), e_old);
  int8_t* dst = (values ? a.c.v : a.c.k) + ((size_t)page * a.c.heads + head) * P * D;

  if (held > 0 && e > e_old) {  // the same for all threads
    const float f = pow2(e_old - e);
    for (int i = threadIdx.x; i < held * (D / 4); i += kThreads) {
      char4 c = reinterpret_cast<char4*>(dst)[i];
      c.x = (signed char)__float2int_rn((float)c.x * f);
      c.y = (signed char)__float2int_rn((float)c.y * f);
      c.z = (signed char)__float2int_rn((float)c.z * f);
      c.w = (signed char)__float2int_rn((float)c.w * f);
      reinterpret_cast<char4*>(dst)[i] = c;
    }
  }
  const float inv = pow2(-e);
#pragma unroll
  for (int q = 0; q < PASSES; ++q) {
    const int row = held + q * ROWS + r0;
    if (row < end) {
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        int c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = u[q][4 * j + i];
          c[i] = __float2int_rn(fminf(fmaxf(x * inv, -127.0f), 127.0f));
          if (!(x == x)) c[i] = 0;
        }
        w[j] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
      }
      *reinterpret_cast<uint2*>(dst + (size_t)row * D + 8 * l) = make_uint2(w[0], w[1]);
    }
  }
  if (threadIdx.x == 0) *scale = pow2(e);  // read by this CTA alone, before the barrier above
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
  int B, T, width;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a, int rows_cta) {
  constexpr int LPR = D / 8;
  constexpr int ROWS = kThreads / LPR;
  __shared__ __align__(16) T stage[ROWS][D];
  __shared__ int place[128];  // row of codes (page * page size + place), or -1
  const int head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int t0 = blockIdx.x * rows_cta, nt = min(rows_cta, a.T - t0);
  // the sequence of the CTA's first row: how many end at or before it
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    before += __syncthreads_count(b < a.B && a.cu[b + 1] <= t0);
  }
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    int b = before;
    while (b < a.B && a.cu[b + 1] <= t) ++b;
    int at = -1;
    if (b < a.B && t >= a.cu[b]) {
      const long long p = (long long)a.first[b] + (t - a.cu[b]);
      if (p >= 0 && p < (long long)a.width * a.c.page) {
        const int page = a.table[(size_t)b * a.width + (int)(p / a.c.page)];
        if (page >= 0 && page < a.c.n_pages) at = page;
        if (at >= 0) place[threadIdx.x] = (int)(p % a.c.page);
      }
      if (at < 0) bad_index(a.status);
    }
    place[threadIdx.x] = at < 0 ? -1 : at * a.c.page + place[threadIdx.x];
  }
  __syncthreads();
  const int l = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const int8_t* codes = values ? a.c.v : a.c.k;
  const float* scales = values ? a.c.vs : a.c.ks;
  T* out = static_cast<T*>(values ? a.v : a.k);
  const LaneTurn turn = lane_turn(a.r, l);
  for (int q = 0; q < nt; q += ROWS) {
    const int row = q + r0;
    const int at = row < nt ? place[row] : -1;
    uint2 w = make_uint2(0u, 0u);
    float scale = 0.0f;
    if (at >= 0) {
      const int page = at / a.c.page, off = at - page * a.c.page;
      const size_t ph = (size_t)page * a.c.heads + head;
      w = *reinterpret_cast<const uint2*>(codes + (ph * a.c.page + off) * D + 8 * l);
      scale = scales[ph];
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = i < 4 ? w.x : w.y;
      x[i] = (float)(int)(signed char)(word >> (8 * (i & 3))) * scale;
    }
    uint4 o;
    if (a.r.perm) {
      unrotate_row<T>(x, turn, l, a.r, stage[r0]);
      __syncwarp();
      o = *reinterpret_cast<const uint4*>(&stage[r0][8 * l]);
      __syncwarp();
    } else {
      o = pack8<T>(x);
    }
    if (at >= 0) *reinterpret_cast<uint4*>(out + ((size_t)(t0 + row) * a.c.heads + head) * D + 8 * l) = o;
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
  const long long units = std::min<long long>(c.T, (long long)c.T / P + 2ll * c.B);
  const dim3 grid((unsigned)units, (unsigned)c.cache->heads, 2u);
  const int passes = (P * (D / 8) + kThreads - 1) / kThreads;
  cudaStream_t s = (cudaStream_t)c.stream;
  auto go = [&](auto kern) { kern<<<grid, kThreads, 0, s>>>(a); };
#define OQ_PASSES(T, DD)                               \
  switch (passes) {                                    \
    case 1: go(write_kernel<T, DD, 1>); break;         \
    case 2: go(write_kernel<T, DD, 2>); break;         \
    case 4: go(write_kernel<T, DD, 4>); break;         \
    default: go(write_kernel<T, DD, DD / 16>); break;  \
  }
  if (c.dtype == OQ_BF16) {
    if (D == 128) OQ_PASSES(__nv_bfloat16, 128) else OQ_PASSES(__nv_bfloat16, 64)
  } else {
    if (D == 128) OQ_PASSES(__half, 128) else OQ_PASSES(__half, 64)
  }
#undef OQ_PASSES
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(OQ_ERR_CUDA, "cache write launch: %s", cudaGetErrorString(e));
  return OQ_OK;
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
  // enough rows for a CTA to keep its loads in flight, fewer while SMs stand idle
  const int pass = kThreads / (D / 8);
  int rows = 128;
  while (rows > pass && (long long)((c.T + rows - 1) / rows) * c.cache->heads * 2 < 4ll * nsm) rows /= 2;
  const dim3 grid((unsigned)((c.T + rows - 1) / rows), (unsigned)c.cache->heads, 2u);
  cudaStream_t s = (cudaStream_t)c.stream;
  auto go = [&](auto kern) { kern<<<grid, kThreads, 0, s>>>(a, rows); };
  if (c.dtype == OQ_BF16)
    D == 128 ? go(read_kernel<__nv_bfloat16, 128>) : go(read_kernel<__nv_bfloat16, 64>);
  else
    D == 128 ? go(read_kernel<__half, 128>) : go(read_kernel<__half, 64>);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(OQ_ERR_CUDA, "cache read launch: %s", cudaGetErrorString(e));
  return OQ_OK;
}

}  // namespace oq
