// Attention over the 8-bit cache for few query rows (single tokens of a batch,
// or a few tokens checked together): bound by reading the cache once.
//
//   o_i = Pi^T sum_j p_ij v_j,  p = softmax_j(scale * (Pi q_i) . k_j)
// on codes: k_j = 2^ek ck_j, v_j = 2^ev cv_j with one ek, ev for a page and head.
// The turned query stands in fp16 beside a power of two of its own (largest
// value in [1, 2), so no range is lost; each value is rounded by at most 2^-12
// of itself, a sixteenth of a bf16 rounding; for fp16 tensors, where that would
// show, what the rounding leaves out is a second term), the codes are exact in
// fp16, sums are fp32.
//
// The running reference is taken over score + ev (logarithms to base 2), so the
// weights p * 2^ev that go to fp16 are at most 2^15.9, and right to 2^-12 down to
// 2^-26 of the largest (see kShift), whatever the pages' scales; the softmax sum
// takes them back times 2^-ev in fp32.  The reference is raised only when a weight
// would pass 2^15.9: the accumulators are rarely touched, and most tiles need no
// exchange at all.  (The running maximum and sum of a softmax in one pass: Milakov and
// Gimelshein, 2018; raising the maximum past a threshold only is published too.)  Weights
// of 2^-12 are a sixteenth of a bf16 result's rounding, but as much as an fp16 result's
// own: fp16 results are off from the exact ones by 1.3 times as much as with fp32 weights
// (2.8e-4 against 2.1e-4, chunks of D = 64).  A second term would double their products.
//
// Tensor tiles m16n8k16 with the cache as the left operand: keys (tokens x D)
// for the scores and transposed values (D x tokens) for the sum, eight query
// rows as the right one.  Nothing of the cache passes through a transposing
// step: the sum over D may take its coordinates in any order, so a lane's 16
// bytes of a key row serve four products as they lie; and the rows of the
// transposed values are any order of D, so a lane takes four tokens' bytes of
// the same 16 coordinates and pairs them with byte permutes.  (tcgen05 needs
// 64 rows at least and its operands expanded into shared memory; eight rows
// would leave it idle, and the kernel waits for memory, not for products.)
//
// A warp keeps a ring of 16-token stages of its own, filled by 16-byte
// asynchronous copies, so it never waits for other warps while tiles run; the
// four warps of a CTA take turns over the tokens and put their sums together at
// the end of an item.  Four CTAs fit an SM (three stages a warp), 128 KB of the
// cache under way on each: 64 sequences of 100 to 8200 tokens, 8 heads, group 4: 548 MB in
// 110 us inside a captured graph, 5.0 TB/s, and 119 us in calls one by one; one of 131072
// tokens: 269 MB in 60 us, 4.5 TB/s, and 61.  The median CTA is done after 85 % of that
// time; what is left is the unevenness of the memory's service between SMs, since shares
// are equal and fixed, and 8 us of the join.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "oq_cattn.cuh"

namespace oq {
namespace {

using namespace cattn;

constexpr int kThreads = 128, kWarps = 4;
constexpr int kTile = 64;  // keys of a tile: 16 for each warp
constexpr int kStart = 4;  // units of an item's beginning and end

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 (or 4) bytes into shared memory; zeros when `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Places of a stage's 16-byte chunks, so that the reads below meet no bank twice.
template <int D>
__device__ __forceinline__ int key_at(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ ((row & 1) << 2)) << 4) : row * 64 + (chunk << 4);
}
template <int D>
__device__ __forceinline__ int value_at(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ (row & 6)) << 4)
                  : (row >> 1) * 128 + (((row ^ (row >> 1)) & 1) << 6) + ((chunk ^ (((row >> 2) & 1) << 1)) << 4);
}

template <int D, int NQ, bool TWO>
struct Smem {
  static constexpr int RT = 8 * NQ;
  static constexpr int kStages = NQ == 1 ? 3 : 4;  // three: four CTAs an SM
  static constexpr int kStageBytes = 2 * 16 * D;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kScales = kRing;                             // [warps][stages][2] floats
  static constexpr int kQ = kScales + kWarps * kStages * 8;         // [RT][D + 8] halves
  static constexpr int kLow = kQ + RT * (D + 8) * 2;                // the same: the query's second term
  static constexpr int kRow = kLow + (TWO ? RT * (D + 8) * 2 : 0);  // [RT] factor, [RT] limit, [RT] start of the scores
  static constexpr int kStat = kRow + RT * 12;                      // [warps][RT] reference, sum
  static constexpr int kStageRow = kStat + kWarps * RT * 8;         // [128 / (D / 8)][D] 16-bit rows
  static constexpr int kTotal = kStageRow + kThreads / (D / 8) * D * 2;
  static constexpr int kSumStride = D + 4;
  static_assert(kWarps * RT * kSumStride * 4 <= kRing, "the warps' sums stand in the ring");
  static_assert(kQ % 16 == 0 && kRow % 16 == 0 && kStat % 16 == 0 && kStageRow % 16 == 0, "alignment");
};

template <typename T, int D, int NQ, bool TWO>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? 4 : 2)
step_kernel(const __grid_constant__ Args a) {
  using S = Smem<D, NQ, TWO>;
  constexpr int RT = S::RT, LPR = D / 8, KS = D / 16, kStages = S::kStages;
  extern __shared__ __align__(16) unsigned char sm[];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int cta = blockIdx.x;
  __half* qs = reinterpret_cast<__half*>(sm + S::kQ);
  __half* low = reinterpret_cast<__half*>(sm + S::kLow);
  float* row_fac = reinterpret_cast<float*>(sm + S::kRow);
  int* row_lim = reinterpret_cast<int*>(sm + S::kRow + RT * 4);
  float* row_bias = reinterpret_cast<float*>(sm + S::kRow + RT * 8);
  float* w_max = reinterpret_cast<float*>(sm + S::kStat);
  float* w_sum = w_max + kWarps * RT;
  float* sums = reinterpret_cast<float*>(sm);
  const uint32_t ring = smem_u32(sm) + warp * kStages * S::kStageBytes;
  const unsigned char* ring_p = sm + warp * kStages * S::kStageBytes;
  const float* scales_p = reinterpret_cast<const float*>(sm + S::kScales) + warp * kStages * 2;
  const uint32_t scales_s = smem_u32(sm) + S::kScales + warp * kStages * 8;

  const Share sh = find_share<RT, kTile, kStart, kThreads>(a, cta, gridDim.x);
  long long at = sh.size * cta;
  const long long stop = min(sh.total, at + sh.size);
  int4 desc = make_int4(0, 0, 0, 0);
  int b = sh.b;
  long long into = sh.into;
  const int l = lane % LPR;
  const LaneTurn turn = lane_turn(a.r, l);
  T* stage_row = reinterpret_cast<T*>(sm + S::kStageRow) + (threadIdx.x / LPR) * D;
  const int plog = 31 - __clz(a.c.page);
  // the lane's places in a stage: chunk lane + 32 j, of which j and j + 2 lie 1024 bytes apart
  uint32_t to_key[2], to_value[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int id = lane + 32 * j;
    to_key[j] = key_at<D>(id / KS, id % KS), to_value[j] = value_at<D>(id / KS, id % KS);
  }

  while (at < stop && b < a.B) {
    const Seq s = load_seq(a, b, false);
    const long long per_head = units_before<RT, kTile, kStart>(a, s, row_tiles<RT>(s));
    if (into >= per_head * a.c.heads) {
      ++b;
      into = 0;
      continue;
    }
    const Part part = find_part<RT, kTile, kStart>(a, s, per_head, into, stop - at);
    const int h = part.h, qt = part.qt, keys = part.keys, t0 = part.t0, take = part.t1 - part.t0;
    const bool first = t0 == 0, last = part.t1 == part.tiles;
    const size_t slot = ((size_t)2 * cta + (first ? 1 : 0)) * RT;
    const long long item_end = at - into + part.end;
    at += part.units;
    into += part.units;
    if (take == 0) {  // no key tile: nothing to do, but a piece that the join counts on says so
      if (t0 > 0 && threadIdx.x < RT) *reinterpret_cast<float2*>(a.stat + 2 * (slot + threadIdx.x)) = make_float2(-INFINITY, 0.0f);
      continue;
    }
    const int rows = min(RT, s.rows - qt * RT);

    // the item's query rows and the first codes are fetched together
    constexpr int PASS = kThreads / LPR, PASSES = (RT + PASS - 1) / PASS;
    uint4 q_row[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * PASS + threadIdx.x / LPR, gr = qt * RT + min(r, rows - 1), i = row_token(a, gr);
      q_row[p] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        q_row[p] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (long long)(s.cu0 + i) * a.qt +
                                                   ((long long)h * a.group + (gr - i * a.group)) * a.qh + 8 * l);
    }
    const int tok0 = t0 * kTile + warp * 16;
    const int* table = a.table + (size_t)b * a.width;
    auto issue = [&](int k, int st) {  // tokens of step k into stage st
      const int tok = tok0 + k * kTile;
      if (k < take && tok < keys) {
        int page = table[tok >> plog];
        const int have = (page >= 0 && page < a.c.n_pages) ? 16 : 0;  // else zeros: a key scale of 0
        if (!have) {
          if (lane == 0) bad_index(a.status);
          page = 0;
        }
        const size_t ph = (size_t)page * a.c.heads + h;
        const size_t from = ((ph << plog) + (tok & (a.c.page - 1))) * D + 16 * lane;
        const int8_t* ks = a.c.k + from;
        const int8_t* vs = a.c.v + from;
        const uint32_t dst = ring + st * S::kStageBytes;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          copy16(dst + to_key[j & 1] + (j >> 1) * 1024, ks + 512 * j, have);
          copy16(dst + 16 * D + to_value[j & 1] + (j >> 1) * 1024, vs + 512 * j, have);
        }
        if (lane < 2) copy4(scales_s + st * 8 + 4 * lane, (lane ? a.c.vs : a.c.ks) + ph, have / 4);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k, k);

    // the rows: turned, scaled by a power of two, fp16
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * PASS + threadIdx.x / LPR, i = row_token(a, qt * RT + min(r, rows - 1));
      const uint4 w = q_row[p];
      float x[8];
      if (a.r.perm) {
        *reinterpret_cast<uint4*>(stage_row + 8 * l) = w;
        __syncwarp();
        rotate_row<T>(stage_row, turn, l, a.r, x);
        __syncwarp();
      } else {
        unpack8<T>(w, x);
      }
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
#pragma unroll
      for (int m = LPR / 2; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
      const int e = min(max(scale_exp(top), -100), 120);
      float all = 0.0f;  // of the row's terms: see the keys' products
      if (r < RT) {
        const float f = pow2(-e);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= f;
        const uint4 hi = pack8<__half>(x);
        *reinterpret_cast<uint4*>(qs + r * (D + 8) + 8 * l) = hi;
        float y[8];
        unpack8<__half>(hi, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) all += y[k];
        if constexpr (TWO) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = x[k] - y[k];
          const uint4 lo = pack8<__half>(y);
          *reinterpret_cast<uint4*>(low + r * (D + 8) + 8 * l) = lo;
          unpack8<__half>(lo, y);
#pragma unroll
          for (int k = 0; k < 8; ++k) all += y[k];
        }
      }
#pragma unroll
      for (int m = LPR / 2; m >= 1; m >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, m);
      if (r < RT) {
        if (l == 0) {
          row_bias[r] = -1152.0f * all;
          row_fac[r] = pow2(e) * a.scale;
          row_lim[r] = r >= rows ? 0 : a.causal ? s.len - s.n + i + 1 : s.len;
        }
      }
    }
    __syncthreads();
    uint32_t qf[NQ][KS][2];
    float fac[NQ][2], bias[NQ][2];
    int lim[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        // product k takes, from lane c, coordinates 64 (k / 4) + 16 c + 4 (k % 4) + 0..3
        const uint2 w = *reinterpret_cast<const uint2*>(qs + (8 * n + g) * (D + 8) + 64 * (k / 4) + 16 * c + 4 * (k % 4));
        qf[n][k][0] = w.x, qf[n][k][1] = w.y;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * n + 2 * c + j;
        fac[n][j] = row_fac[r], lim[n][j] = row_lim[r], bias[n][j] = row_bias[r];
      }
    }
    const int sure = row_lim[0];  // keys before this are seen by every row of the tile

    float acc[KS][NQ][4];
    float top[NQ][2], sum[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[k][n][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) top[n][j] = -INFINITY, sum[n][j] = 0.0f;
    }

    int now = 0, then = kStages - 1;  // stages of step k, of the one that is fetched

    for (int k = 0; k < take; ++k) {
      const int tok = tok0 + k * kTile;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      issue(k + kStages - 1, then);
      if (tok >= keys) break;  // the same for the warp; only the item's last tile ends early
      const unsigned char* st = ring_p + now * S::kStageBytes;
      const float kscale = scales_p[now * 2], vscale = scales_p[now * 2 + 1];
      now = now + 1 == kStages ? 0 : now + 1, then = then + 1 == kStages ? 0 : then + 1;
      const int ev = min(max(scale_exp(vscale), -126), 126);

      // The keys' codes go into the products as 1152 + code (see oq_cattn.cuh) and the
      // sums begin at -1152 times the query's: the difference is the product with the
      // codes, to 2^-24 of ~2^13, far below what the query's rounding leaves.
      float sc[NQ][4], sd[NQ][4];  // two chains of products
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[n][j] = bias[n][j & 1], sd[n][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(st + key_at<D>(g, 4 * j + c));
        const uint4 k1 = *reinterpret_cast<const uint4*>(st + key_at<D>(g + 8, 4 * j + c));
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x0 = w0[i] ^ 0x80808080u, x1 = w1[i] ^ 0x80808080u;
          const uint32_t a0 = __byte_perm(x0, 0x64646464u, 0x4140), a1 = __byte_perm(x1, 0x64646464u, 0x4140),
                         a2 = __byte_perm(x0, 0x64646464u, 0x4342), a3 = __byte_perm(x1, 0x64646464u, 0x4342);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            mma16816(i & 1 ? sd[n] : sc[n], a0, a1, a2, a3, qf[n][4 * j + i][0], qf[n][4 * j + i][1]);
            if constexpr (TWO) {
              const uint2 w = *reinterpret_cast<const uint2*>(low + (8 * n + g) * (D + 8) + 64 * j + 16 * c + 4 * i);
              mma16816(i & 1 ? sd[n] : sc[n], a0, a1, a2, a3, w.x, w.y);
            }
          }
        }
      }
      // scores to base 2 plus the values' exponent; rows of sc: tokens g, g + 8; columns: rows 2 c, 2 c + 1
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          sc[n][j] = fmaf(sc[n][j] + sd[n][j], kscale * fac[n][j], (float)ev);
          sc[n][2 + j] = fmaf(sc[n][2 + j] + sd[n][2 + j], kscale * fac[n][j], (float)ev);
        }
      if (tok + 16 > sure || kscale == 0.0f) {  // the same for the warp
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (tok + g >= lim[n][j] || kscale == 0.0f) sc[n][j] = -INFINITY;
            if (tok + g + 8 >= lim[n][j] || kscale == 0.0f) sc[n][2 + j] = -INFINITY;
          }
      }
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) raise |= fmaxf(sc[n][j], sc[n][2 + j]) > top[n][j] + kRaise;
      if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float t = fmaxf(sc[n][j], sc[n][2 + j]);
#pragma unroll
            for (int m = 4; m <= 16; m <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, m));
            t = fmaxf(t - kShift, top[n][j]);
            f[j] = t == -INFINITY ? 1.0f : ex2(top[n][j] - t);
            top[n][j] = t;
            sum[n][j] *= f[j];
          }
#pragma unroll
          for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][n][j] *= f[j & 1];
        }
      }
      const float back = pow2(-ev);
      uint32_t pf[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float t = top[n][j] == -INFINITY ? 0.0f : top[n][j];
          p[j] = ex2(sc[n][j] - t), p[2 + j] = ex2(sc[n][2 + j] - t);
          sum[n][j] = fmaf(p[j] + p[2 + j], back, sum[n][j]);
        }
        pf[n][0] = transpose8x8(pack2<__half>(p[0], p[1]));
        pf[n][1] = transpose8x8(pack2<__half>(p[2], p[3]));
      }
      // transposed values: product m takes coordinates g D/8 + 2 m (rows g) and + 1 (rows g + 8)
      const unsigned char* vst = st + 16 * D;
      uint32_t v[4][D / 32];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 2 * c + (t & 1) + 8 * (t >> 1);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(vst + value_at<D>(row, g));
          v[t][0] = w.x, v[t][1] = w.y, v[t][2] = w.z, v[t][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vst + value_at<D>(row, g >> 1) + 8 * (g & 1));
          v[t][0] = w.x, v[t][1] = w.y;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t x0 = v[0][w] ^ 0x80808080u, x1 = v[1][w] ^ 0x80808080u;
        const uint32_t x2 = v[2][w] ^ 0x80808080u, x3 = v[3][w] ^ 0x80808080u;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t lo = __byte_perm(x0, x1, u ? 0x7362 : 0x5140), hi = __byte_perm(x2, x3, u ? 0x7362 : 0x5140);
          const uint32_t a0 = bytes2(lo, 0x4140), a1 = bytes2(lo, 0x4342), a2 = bytes2(hi, 0x4140),
                         a3 = bytes2(hi, 0x4342);
#pragma unroll
          for (int n = 0; n < NQ; ++n) mma16816(acc[2 * w + u][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // every warp is done with its ring: the sums go there

#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) sum[n][j] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][j], m);
        const int r = 8 * n + 2 * c + j;
        if (g == 0) w_max[warp * RT + r] = top[n][j], w_sum[warp * RT + r] = sum[n][j];
        float* o = sums + (warp * RT + r) * S::kSumStride + g * (D / 8);
#pragma unroll
        for (int m = 0; m < KS; ++m) *reinterpret_cast<float2*>(o + 2 * m) = make_float2(acc[m][n][j], acc[m][n][2 + j]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < RT; p += kThreads / LPR) {
      const int r = p + threadIdx.x / LPR, rr = min(r, RT - 1);
      float m4[kWarps], mx = -INFINITY, total = 0.0f, x[8];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m4[w] = w_max[w * RT + rr], mx = fmaxf(mx, m4[w]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(m4[w] - ref);
        total = fmaf(f, w_sum[w * RT + rr], total);
        const float* o = sums + (w * RT + rr) * S::kSumStride + 8 * l;
        const float4 lo = *reinterpret_cast<const float4*>(o), hi = *reinterpret_cast<const float4*>(o + 4);
        x[0] = fmaf(f, lo.x, x[0]), x[1] = fmaf(f, lo.y, x[1]), x[2] = fmaf(f, lo.z, x[2]), x[3] = fmaf(f, lo.w, x[3]);
        x[4] = fmaf(f, hi.x, x[4]), x[5] = fmaf(f, hi.y, x[5]), x[6] = fmaf(f, hi.z, x[6]), x[7] = fmaf(f, hi.w, x[7]);
      }
      if (first && last) {
        const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= inv;
        uint4 w;
        if (a.r.perm) {
          unrotate_row<T>(x, turn, l, a.r, stage_row);
          __syncwarp();
          w = *reinterpret_cast<const uint4*>(stage_row + 8 * l);
          __syncwarp();
        } else {
          w = pack8<T>(x);
        }
        const int gr = qt * RT + r, i = row_token(a, gr);
        if (r < rows)
          *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (long long)(s.cu0 + i) * a.ot +
                                    ((long long)h * a.group + (gr - i * a.group)) * a.oh + 8 * l) = w;
      } else if (r < rows) {
        float4* o = reinterpret_cast<float4*>(a.piece + (slot + r) * D + 8 * l);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (l == 0)  // (a NaN query leaves no reference; its piece must count all the same)
          *reinterpret_cast<float2*>(a.stat + 2 * (slot + r)) = make_float2(total == total ? mx : 0.0f, total);
      }
    }
    if (first && !last) desc = make_int4((int)((item_end - 1) / sh.size) - cta + 1, b, h, qt);
    __syncthreads();
  }
  chain_next();
  if (threadIdx.x == 0) a.desc[cta] = desc;
}

struct Plan {
  int rows;  // of a tile
  int ctas;  // most
};
Plan plan_of(int T, int B, int group) {
  Plan p;
  const long long per = ((long long)T * group + B - 1) / std::max(1, B);  // rows of a sequence, on average
  // 32 sequences of 3600 keys, 4 heads, fp16, D = 64, group 4; and one of 31200, 12 heads,
  // bf16, D = 128 (us with tiles of 8, 16, 256 rows):
  //   rows    4            8           16           24           32           48
  //        28, 33, 81   31, 35, 81   46, 39, 81   62, 61, 82   78, 64, 82   105, 83, 83
  //                     33, 31, 71   46, 34, 71   61, 51, 71   75, 51, 71   105, 69, 72
  // One choice for the call: where the sequences' rows lie on both sides of it, all pay for
  // the average.  63 single tokens over 4000 keys beside a chunk of 4096, 32 heads on 8: 576
  // us, and 106 and 249 in two calls; 127 beside a chunk of 1000: 416, and 191 and 54; with
  // 24 heads on 24, 1126, and 265 and 191.  The header sends such batches in two calls.
  p.rows = per <= 8 ? 8 : per <= 48 ? 16 : 256;
  p.ctas = p.rows == 256 ? kChunkCtas : kStepCtas;
  return p;
}

size_t piece_bytes(const Plan& p, int d) { return sizeof(float) * 2 * (size_t)p.ctas * p.rows * d; }
size_t stat_bytes(const Plan& p) { return sizeof(float) * 4 * (size_t)p.ctas * p.rows; }

template <typename T, int D, int NQ, bool TWO>
int launch_step(const Args& a, int ctas_most, void* stream) {
  auto kern = step_kernel<T, D, NQ, TWO>;
  const int smem = Smem<D, NQ, TWO>::kTotal;
  int per_sm = 0, nsm = 0;
  if (int rc = occupancy(reinterpret_cast<const void*>(kern), smem, kThreads, 0, &per_sm)) return rc;
  if (int rc = sm_count(&nsm)) return rc;
  if (per_sm < 1) return fail(OQ_ERR_UNSUPPORTED, "attention kernel does not fit");
  // no more CTAs than tiles that there can be
  const long long rows = (long long)a.T * a.group;
  const long long items = std::min<long long>((rows + 8 * NQ - 1) / (8 * NQ) + a.B, rows) * a.c.heads;
  const long long tiles = items * std::max<long long>(1, ((long long)a.width * a.c.page + kTile - 1) / kTile);
  const int ctas = (int)std::min<long long>(tiles, std::min(nsm * per_sm, ctas_most));
  if (int rc = launch_chained("attention", kern, dim3((unsigned)ctas), kThreads, smem, stream, a)) return rc;
  return launch_chained("attention join", join_kernel<T, D, 8 * NQ, 8>, dim3((unsigned)ctas, 8 * NQ), 256, 0, stream, a);
}

}  // namespace

size_t cattn_workspace(int T, int B, int group, int d) {
  const Plan p = plan_of(T, B, group);
  return piece_bytes(p, d) + stat_bytes(p) + sizeof(int4) * (size_t)p.ctas;
}

int launch_cattn(const AttnCall& c) {
  Args a;
  std::memset(&a, 0, sizeof(a));
  const oq_kvcache* v = c.cache;
  a.c.k = v->k, a.c.v = v->v, a.c.ks = v->k_scale, a.c.vs = v->v_scale;
  a.c.n_pages = v->n_pages, a.c.heads = v->heads, a.c.page = v->page;
  if (int rc = cache_rotation(c.r, &a.r)) return rc;
  if (int rc = device_status_word(&a.status)) return rc;
  a.q = c.q, a.out = c.out;
  a.qt = c.q_token, a.qh = c.q_head, a.ot = c.o_token, a.oh = c.o_head;
  a.cu = c.cu, a.lens = c.lens, a.table = c.table;
  a.B = c.B, a.T = c.T, a.width = c.width;
  a.group = c.heads / v->heads;
  a.div_group = a.group > 1 ? (unsigned)((0x100000000ull + a.group - 1) / a.group) : 0u;
  a.causal = c.causal;
  a.scale = (float)((double)c.scale * 1.4426950408889634);
  const Plan p = plan_of(c.T, c.B, a.group);
  a.piece = static_cast<float*>(c.workspace);
  a.stat = reinterpret_cast<float*>(static_cast<char*>(c.workspace) + piece_bytes(p, v->d));
  a.desc = reinterpret_cast<int4*>(static_cast<char*>(c.workspace) + piece_bytes(p, v->d) + stat_bytes(p));
  if (p.rows == 256) {
    a.stall = take_test_stall(7);
    return launch_cattn_chunk(a, c.dtype, v->d, c.stream);
  }
#define OQ_STEP(T, D, TWO) \
  return p.rows == 8 ? launch_step<T, D, 1, TWO>(a, p.ctas, c.stream) : launch_step<T, D, 2, TWO>(a, p.ctas, c.stream)
  if (c.dtype == OQ_BF16) {
    if (v->d == 128) OQ_STEP(__nv_bfloat16, 128, false);
    OQ_STEP(__nv_bfloat16, 64, false);
  }
  if (!a.r.perm) {  // fp16 rows that are not turned are exact in one term
    if (v->d == 128) OQ_STEP(__half, 128, false);
    OQ_STEP(__half, 64, false);
  }
  if (v->d == 128) OQ_STEP(__half, 128, true);
  OQ_STEP(__half, 64, true);
#undef OQ_STEP
}

}  // namespace oq
