// What the two attention kernels over the 8-bit cache share: how the work is
// shared out, and how the pieces of a split row are put together.
//
// An item is (sequence, head of the cache, tile of query rows): the rows of a
// tile are the new tokens' query heads that share the cache's head, row r being
// token r / group, head r % group of the group.  An item walks its key tiles.
// Its work is counted in units: a fixed number for its beginning and end (the
// query's turn, the first loads, the rows' turn back) and about one for each key
// tile.  The units of all items in a row (sequence, head, row tile) are cut into
// equal shares, one for each CTA, wherever the cut falls, so that ragged batches
// and a single long stream fill the machine alike.  A CTA finds its share from
// the lengths on the device: nothing about them is known on the host.  How many
// units the first q row tiles of a head have is a closed form (units_before), so
// no CTA walks over items that are not its own.
//
// An item that one CTA covers is finished there.  Of an item that is cut, each
// CTA leaves a piece in the workspace (for each row its reference, sum and
// weighted values, fp32): the CTA that has the first key tile in its slot 1, the
// ones that go on with it in their slot 0.  The first also writes down which CTAs
// hold pieces, and the joining kernel adds them up in the CTAs' order: no
// atomics, the same result every time.
#pragma once

#include "oq_cache.cuh"

namespace oq {
namespace cattn {

using namespace cache;

// Weights go to the products in fp16, beside a reference kept for each row and raised only
// when a weight would pass 2^kRaise (fp16 holds 65504, 2^15.99), so few steps have to rescale
// what is summed up.  A weight is right to 2^-12 of itself down to 2^-14 beside the reference,
// and off by up to 2^-25 below (the softmax's sum takes the weights in fp32).  So that weights
// far below a row's largest keep their bits, the reference, when it is raised, is set below
// the largest score: kShift below in the step kernel.  In the chunk kernel a raise is dear
// (4608 x 4608 rows whose scores spread by 3 to 5 nats: 320 us with the reference at the
// largest score, 393, 415 and 424 with it 8, 10 and 12 below), so it looks at the 64 keys at
// hand: up to kShift below, but no further than leaves the weakest 16 of them, by their
// largest, kRoom below.  Keys that spread as usual stay together and raise as seldom as
// before; where a few stand 17 nats above the others, these keep 10 bits and more.
constexpr float kShift = 12.0f, kRaise = 15.9f, kRoom = 10.0f;
// Most CTAs that the workspace has pieces for (the kernels' residency on 148 SMs).
constexpr int kStepCtas = 148 * 4, kChunkCtas = 148;

struct Args {
  View c;
  Rotation r;
  const void* q;
  void* out;
  long long qt, qh, ot, oh;  // strides in elements
  const int* cu;
  const int* lens;
  const int* table;
  int* status;
  float* piece;   // [2 ctas][rows of a tile][D]
  float* stat;    // [2 ctas][rows of a tile][2]: reference, sum
  int4* desc;     // [ctas]: (pieces, sequence, head, row tile)
  int B, T, width, group, causal;
  int stall;           // test hook: the chunk kernel's keys are never handed over (the waits run out)
  unsigned div_group;  // 2^32 / group, rounded up (group > 1)
  float scale;    // of the scores, times log2(e)
};

// Lengths of one sequence; rows = 0 where its numbers do not fit (reported) or it has no new token.
struct Seq {
  int cu0, n, len, rows;
};
__device__ __forceinline__ Seq load_seq(const Args& a, int b, bool report) {
  Seq s;
  s.cu0 = a.cu[b];
  s.n = a.cu[b + 1] - s.cu0;
  s.len = a.lens[b];
  const bool ok = s.cu0 >= 0 && s.n >= 0 && s.cu0 + (long long)s.n <= a.T && s.len >= 0 &&
                  s.len <= (long long)a.width * a.c.page;
  if (!ok) {
    if (report) bad_index(a.status);
    s.n = 0;
  }
  s.rows = s.n * a.group;
  return s;
}
// Token of a row: r / group.
__device__ __forceinline__ int row_token(const Args& a, int r) {
  if (a.group == 1) return r;
  const int q = (int)__umulhi((unsigned)r, a.div_group);  // right, or one too many
  return (long long)q * a.group > r ? q - 1 : q;
}
// Keys that the row tile's last row may see (causal: the tile's other rows see no more).
template <int RT>
__device__ __forceinline__ int tile_keys(const Args& a, const Seq& s, int qt) {
  if (!a.causal) return s.len;
  return max(0, s.len - s.n + row_token(a, min(s.rows - 1, qt * RT + RT - 1)) + 1);
}
template <int RT>
__device__ __forceinline__ int row_tiles(const Seq& s) {
  return (s.rows + RT - 1) / RT;
}
// Units of the first q row tiles of a head: START each, and the key tiles (for
// causal rows a smooth count, right but for roundings: row tile i sees
// len - n + (i + 1) RT / group keys).
template <int RT, int TILE, int START>
__device__ __forceinline__ long long units_before(const Args& a, const Seq& s, int q) {
  if (!a.causal) return (long long)q * (START + max(1, (s.len + TILE - 1) / TILE));
  // floor(q (2 group (len - n) + RT (q + 1)) / (2 group TILE)), whose product would pass 64 bits
  const unsigned long long past = (unsigned long long)q * (unsigned)max(0, s.len - s.n);
  const unsigned long long rest = past % TILE * 2u * a.group + (unsigned long long)RT * q * (q + 1ull);
  const unsigned den = 2u * a.group * TILE;
  const unsigned long long tiles = past / TILE + (rest >> 32 ? rest / den : (unsigned)rest / den);
  return (long long)q * (START + 1) + (long long)tiles;
}

// Where a CTA's share begins.
struct Share {
  long long total, size;  // units of all items, of a share
  int b;                  // sequence of the first unit; B when the share is empty
  long long into;         // units of that sequence before it
};

// All THREADS threads of the CTA take part and get the same answer.  SPARE: units that a
// share may grow by when that leaves no item cut.
template <int RT, int TILE, int START, int THREADS, int SPARE = 0>
__device__ Share find_share(const Args& a, int cta, int ctas) {
  __shared__ long long warp_sum[THREADS / 32];
  __shared__ Share found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.B <= 32) {  // each warp finds it for itself
    long long mine = 0;
    unsigned item = 0;  // units of an item of the sequence, where all its items are alike
    if (lane < a.B) {
      const Seq s = load_seq(a, lane, cta == 0 && warp == 0);
      mine = units_before<RT, TILE, START>(a, s, row_tiles<RT>(s)) * a.c.heads;
      if (SPARE > 0 && mine) item = (unsigned)units_before<RT, TILE, START>(a, s, 1);
    }
    long long incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
      if (lane >= m) incl += o;
    }
    Share s;
    s.total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    s.size = (s.total + ctas - 1) / ctas;
    if (SPARE > 0 && !a.causal) {  // whole items for each CTA, if they are all alike and cost little more
      const unsigned most = __reduce_max_sync(0xFFFFFFFFu, item);
      const unsigned least = __reduce_min_sync(0xFFFFFFFFu, item ? item : most);
      if (most && most == least) {
        const long long whole = (s.total / most + ctas - 1) / ctas * most;
        if (whole <= s.size + SPARE) s.size = whole;
      }
    }
    const long long start = s.size * cta;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, start >= incl - mine && start < incl);
    s.b = hit ? __ffs(hit) - 1 : a.B;
    s.into = start - __shfl_sync(0xFFFFFFFFu, incl - mine, hit ? s.b : 0);
    return s;
  }
  long long total = 0, mine = 0, start = 0, size = 0;
  if (threadIdx.x == 0) found.b = a.B;
  // two passes over the sequences: the sum, then the one that holds the start;
  // up to THREADS of them need their lengths only once
  for (int pass = 0; pass < 2; ++pass) {
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
      const int b = b0 + (int)threadIdx.x;
      if (pass == 0 || a.B > THREADS) {
        mine = 0;
        if (b < a.B) {
          const Seq s = load_seq(a, b, pass == 0 && cta == 0);
          mine = units_before<RT, TILE, START>(a, s, row_tiles<RT>(s)) * a.c.heads;
        }
      }
      long long incl = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        if (lane >= m) incl += o;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      long long base = before;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += warp_sum[w];
        before += warp_sum[w];
      }
      if (pass == 1) {
        const long long first = base + incl - mine;
        if (start >= first && start < first + mine) {
          found.b = b;
          found.into = start - first;
        }
      }
      __syncthreads();
    }
    total = before;
    size = (total + ctas - 1) / ctas;
    start = size * cta;
  }
  Share s = found;
  s.total = total, s.size = size;
  return s;
}

// The part of an item that a CTA has.
struct Part {
  int h, qt;          // head, row tile
  int keys, tiles;    // keys and key tiles of the item
  int t0, t1;         // key tiles of the part; none: t0 == t1
  long long units;    // how far the share goes on
  long long end;      // units of the sequence up to the item's end
};
// `into`: units of sequence s before the part, `left`: units of the share from there on.
template <int RT, int TILE, int START>
__device__ __forceinline__ Part find_part(const Args& a, const Seq& s, long long per_head, long long into, long long left) {
  Part p;
  p.h = (into | per_head) >> 32 ? (int)(into / per_head) : (int)((unsigned)into / (unsigned)per_head);
  const long long rem = into - p.h * per_head;
  int lo = 0, hi = row_tiles<RT>(s);  // units_before(lo) <= rem < units_before(hi)
  long long before = 0, after = per_head;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const long long u = units_before<RT, TILE, START>(a, s, mid);
    if (u <= rem) {
      lo = mid, before = u;
    } else {
      hi = mid, after = u;
    }
  }
  p.qt = lo;
  p.keys = tile_keys<RT>(a, s, lo);
  p.tiles = max(1, (p.keys + TILE - 1) / TILE);
  const long long item = after - before, at = rem - before;
  p.units = min(item - at, left);
  p.end = into - at + item;
  // the units behind the first START stand for the key tiles, in proportion
  const long long u0 = max(0ll, at - START), u1 = max(0ll, at + p.units - START), span = item - START;
  if (span == p.tiles) {
    p.t0 = (int)u0, p.t1 = (int)u1;
  } else {
    p.t0 = (int)(u0 * p.tiles / span), p.t1 = (int)(u1 * p.tiles / span);
  }
  return p;
}

// Puts the pieces of cut items together and writes their rows.  Block (i, j): rows
// of the item that CTA i began.  WPR = 8: one row at a time, whose pieces eight warps
// share (an item may have many); WPR = 1: a row for each of four warps (an item has
// many rows and few pieces).  The pieces' weights come first, all at once, so that
// the loads of the pieces wait for nothing.
template <typename T, int D, int RT, int WPR>
__global__ void __launch_bounds__(WPR == 8 ? 256 : 128) join_kernel(const __grid_constant__ Args a) {
  constexpr int WARPS = WPR == 8 ? 8 : 4, ROWS = WARPS / WPR, MOST = WPR == 8 ? kStepCtas : kChunkCtas;
  __shared__ __align__(16) float part[WARPS][D];
  __shared__ float2 weight[ROWS][MOST];  // of a piece: its factor, and that times its sum
  __shared__ float warp_max[WARPS];
  __shared__ __align__(16) T row_out[ROWS][D];
  chain();
  const int4 d = a.desc[blockIdx.x];
  if (d.x <= 0) return;
  const Seq s = load_seq(a, d.y, false);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % WPR, row = warp / WPR;
  const int rows = min(RT, s.rows - d.w * RT);
  constexpr int V = D / 32;  // values of a lane
  auto sync = [&] {
    if constexpr (WPR == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  for (int r0 = blockIdx.y * ROWS; r0 < rows; r0 += gridDim.y * ROWS) {
    const int r = min(r0 + row, rows - 1);
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * RT + r; };
    float top = -INFINITY;
    for (int i = 32 * w0 + lane; i < d.x; i += 32 * WPR) {
      weight[row][i] = *reinterpret_cast<const float2*>(a.stat + 2 * slot(i));
      top = fmaxf(top, weight[row][i].x);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    if constexpr (WPR > 1) {
      if (lane == 0) warp_max[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WPR; ++w) top = fmaxf(top, warp_max[w]);
    }
    if (top == -INFINITY) top = 0.0f;
    for (int i = 32 * w0 + lane; i < d.x; i += 32 * WPR) {
      const float2 st = weight[row][i];
      const float f = exp2f(st.x - top);
      weight[row][i] = make_float2(f, f == 0.0f ? 0.0f : f * st.y);
    }
    sync();
    float o[V], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = 0.0f;
    for (int i0 = w0; i0 < d.x; i0 += 8 * WPR) {
      float v[8][V];
      float2 f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = min(i0 + u * WPR, d.x - 1);
        f[u] = i0 + u * WPR < d.x ? weight[row][i] : make_float2(0.0f, 0.0f);
        const float* p = a.piece + slot(i) * D + V * lane;
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p);
          v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(p);
          v[u][0] = x.x, v[u][1] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sum += f[u].y;
#pragma unroll
        for (int k = 0; k < V; ++k)  // (a piece of no weight: its values may not even be written)
          o[k] = fmaf(f[u].x, f[u].x == 0.0f ? 0.0f : v[u][k], o[k]);
      }
    }
    // each piece's sum was counted by the one warp that took it
#pragma unroll
    for (int k = 0; k < V; ++k) part[warp][V * lane + k] = o[k];
    if constexpr (WPR > 1) {
      __syncthreads();
      if (lane == 0) warp_max[warp] = sum;
    }
    sync();
    if (w0 == 0) {
      const int l = lane % (D / 8);
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = part[warp][8 * l + k];
#pragma unroll
      for (int w = 1; w < WPR; ++w) {
        sum += warp_max[warp + w];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] += part[warp + w][8 * l + k];
      }
      const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // no key: 0; NaN stays
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] *= inv;
      uint4 w;
      if (a.r.perm) {
        unrotate_row<T>(x, lane_turn(a.r, l), l, a.r, row_out[row]);  // lanes of one l write the same values
        __syncwarp();
        w = *reinterpret_cast<const uint4*>(row_out[row] + 8 * l);
      } else {
        w = pack8<T>(x);
      }
      const int g = d.w * RT + r, i = row_token(a, g);
      if (lane < D / 8 && r0 + row < rows)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (long long)(s.cu0 + i) * a.ot +
                                  ((long long)d.z * a.group + (g - i * a.group)) * a.oh + 8 * l) = w;
    }
    sync();
  }
}

// Registers of four signed codes (bytes of w) as two fp16 pairs: a byte with its
// sign bit turned is code + 128, the low byte of the fp16 number 1024 + code + 128.
__device__ __forceinline__ uint32_t sub_bias(uint32_t h) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}
__device__ __forceinline__ uint32_t bytes2(uint32_t biased, uint32_t sel) {
  return sub_bias(__byte_perm(biased, 0x64646464u, sel));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace cattn

int launch_cattn_chunk(const cattn::Args& a, int dtype, int d, void* stream);  // oq_cattn_tc.cu

}  // namespace oq
