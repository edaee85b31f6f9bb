// Attention over the 8-bit cache for many query rows (chunks of new tokens,
// whole images): bound by the tensor cores and what feeds them.
//
// The same sums as oq_cattn.cu, on tcgen05: a CTA (one on each SM) takes 256 query
// rows as two tiles of 128 and walks KT keys a step.  Three roles:
//   warps 8..11  expand the step's codes to fp16 (exact) into the K-major
//                128-byte-swizzled layout of the tensor cores' operands, once for
//                both tiles: the keys as they lie, the values transposed by byte
//                permutes, with the codes of what comes next already in registers.
//   warps 0..7   four a tile, one thread a row: scores from TMEM, running reference
//                and sum, weights back into TMEM in two halves, so that the first
//                half's products run beside the second half's exponentials.
//   warp 12      issues the products; one tile's run beside the other tile's
//                exponentials.
// TMEM, all 512 columns: each tile's scores (KT columns), whose first half the
// weights take over (the left operand of the sum), and each tile's sum (D
// columns), which stays until the end.  The turned queries (fp16) are
// shared-memory operands.  The turns themselves are products too: the rows as they
// come times the matrix Pi (entries 0, 1, -1: exact), and at the end the sums, as
// two terms of the tensor's type (2^-17 and better), times its transpose; the
// matrix is written into the values' place when it is needed.  (Butterflies on the
// 256 rows took 33 thousand clocks an item, a tenth of a long one.)
//
// What bounds it (4608 x 4608 rows, D = 128, 24 heads, bf16: 329 us, 794 TFLOP/s; 31200 +
// 1560 keys for 1560 rows, 12 heads: 392 inside a captured graph and 414 to 428 in calls one by
// one; chunks of up to 511 rows, D = 64, fp16, causal: 84): 64 keys take 2150 clocks, of which
// the exponentials take 1024 (16 a clock), the tensor cores 1100, shared memory about as much
// (a 128-key step moves 256 KB: the scores' operands 128, the values 64, the expanded codes
// 64; at 128 bytes a clock 2048 of 4300 clocks), the issue slots 50 to 60 %.  Without the
// exponentials the first example takes 5 % less, without the expansion 12 %, without the
// weights altogether 15 %, with a quarter of the products 3 %: no single part holds it, but
// scores and weights share their columns, so a tile's scores, weights, sum and next scores
// follow one another.  An item's beginning and end take 25 thousand clocks (D = 64: 15), a
// sixth of the first example; a sequence of at most 128 rows leaves the second tile idle.
// Tried beside it (the first two examples, us, against 337 and 390 with cut items in
// both): 64 keys a step, with scores a step ahead, warps of their own for keys (2) and
// values (4), and a product warp for each tile, 330 and 395 (one by one 346 and 427, the chunks
// 87); the same with four warps for keys and values, 335 and 449; with two threads a row (24
// warps), 359 and 460; this one with a product warp for each tile and six expanding warps, 371
// and 447; two CTAs an SM of one tile each, 1.9 times as long.  (Two row tiles in turn, one's
// products beside the other's exponentials, is a published scheme for attention.)
//
// Scales: as in oq_cattn.cu the running reference is taken over score + ev, so
// the weights carry their page's value exponent; groups of 16 tokens (no page is
// smaller) have their own.  The accumulator is rescaled only when a weight would
// pass 2^15.9.
//
// fp16 queries keep a second term: the turn rounds them to 2^-12, which would
// show beside an fp16 result, so what the first operand leaves out goes into a
// second one and the scores take both.  (At D = 128 its 64 KB leave room for
// one stage of values instead of two.)
//
// Every wait is bounded (~1 s); one that gives up records OQ_ERR_TIMEOUT and raises a flag
// that lets all others return at once.  The CTA then leaves at its item's end, waits (bounded)
// for its own products under way, and frees its TMEM.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "oq_cattn.cuh"

namespace oq {
namespace {

using namespace cattn;

constexpr int kThreads = 416, kRows = 256, kTileRows = 128;
constexpr int kTmem = 512, kColS = 0, kColO = 256;  // a tile's columns begin 128 further on
constexpr int kStart = 4;  // units of an item's beginning and end (at D = 128 it takes nearer to six)
// A share may grow by kSpare units when that leaves no item cut: what a cut costs is another
// beginning and end, the pieces' way through memory and the join.  4608 x 4608 rows, D =
// 128, items cut or whole (us): 24 heads, 3 units more, 337 or 317; 23 heads, 8 units, 324 or
// 320; 22 heads, 13 units, 321 or 329; 1200 x 1200 rows, 24 heads, 2 units, 61 or 51.  (Between
// 8 and 13 units nothing was measured, nor shares of other lengths near the border; it is
// asked for up to 32 sequences, whose items every warp sees at once.)
constexpr int kSpare = 9;
constexpr unsigned long long kWaitLimitNs = 1000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const unsigned long long t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (*abort_flag || mbar_try_wait(bar, parity)) return;
    if ((i & 63u) == 0 && global_ns() - t0 > kWaitLimitNs) {
      atomicExch(status, OQ_ERR_TIMEOUT);
      *abort_flag = 1;
      return;
    }
  }
}
__device__ __forceinline__ void wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, abort_flag, status);
}
// The last wait of a CTA, for its own products and arrivals under way, whether or not it gave up.
__device__ __forceinline__ void wait_own(uint32_t bar) {
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, 0u) && global_ns() - t0 < kWaitLimitNs) {
  }
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}
// A value that is the same in all lanes, so that what follows from it stays in uniform
// registers, where the tensor instructions take their operands from.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xFFFFFFFFu, x); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Operand descriptor: K-major, 128-byte swizzle, groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Instruction descriptor: D f32, A and B f16, both K-major, M = 128.
template <int N>
__host__ __device__ constexpr uint32_t idesc() {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// The same with the type of a tensor's rows (the turn's products).
template <typename T, int N>
__host__ __device__ constexpr uint32_t idesc_of() {
  return idesc<N>() | (std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u);
}
template <int N>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc<N>()), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(t));
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(t));
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// 16 bytes from global to shared memory, asynchronously; zeros for those past `bytes`.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ unsigned long long f2_pack(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ unsigned long long u2_pack(uint32_t lo, uint32_t hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b,
                                                     unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long f2_add(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A row's weights 2^(score + ev - top) of KEYS keys from its scores in TMEM, as
// fp16 pairs, and into `sum` their part of the softmax's sum; `mx`: the largest
// exponent, `most`: that of every 16 keys.  sc: (key scale, ev, 2^-ev) of every 16 keys.  MASKED: only the first
// `left` keys are seen.
template <int KEYS, bool MASKED>
__device__ __forceinline__ float weigh(uint32_t scores, const float4* sc, float fac, float top, int left,
                                       uint32_t (&p)[KEYS / 2], float (&most)[KEYS / 16], float& mx) {
  uint32_t v[KEYS];
#pragma unroll
  for (int q = 0; q < KEYS / 32; ++q) tmem_ld32(scores + 32 * q, v + 32 * q);
  float4 s[KEYS / 16];
#pragma unroll
  for (int g = 0; g < KEYS / 16; ++g) s[g] = sc[g];
  wait_ld();
  float sum = 0.0f;
#pragma unroll
  for (int g = 0; g < KEYS / 16; ++g) {
    const float c = s[g].x * fac, d = s[g].x != 0.0f ? s[g].y - top : -INFINITY;  // an empty page's scores go
    const unsigned long long c2 = f2_pack(c, c), d2 = f2_pack(d, d);
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) f2_split(f2_fma(u2_pack(v[16 * g + 2 * j], v[16 * g + 2 * j + 1]), c2, d2), x[2 * j], x[2 * j + 1]);
    if constexpr (MASKED) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (16 * g + j >= left) x[j] = -INFINITY;
    }
    float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[2], x[3]);
#pragma unroll
    for (int j = 4; j < 16; j += 4) m0 = fmaxf(m0, fmaxf(x[j], x[j + 1])), m1 = fmaxf(m1, fmaxf(x[j + 2], x[j + 3]));
    most[g] = fmaxf(m0, m1);
    unsigned long long add[2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float e0 = ex2(x[2 * j]), e1 = ex2(x[2 * j + 1]);
      add[j & 1] = j < 2 ? f2_pack(e0, e1) : f2_add(add[j & 1], f2_pack(e0, e1));
      p[8 * g + j] = pack2<__half>(e0, e1);
    }
    float s0, s1;
    f2_split(f2_add(add[0], add[1]), s0, s1);
    sum = fmaf(s0 + s1, s[g].z, sum);
  }
  mx = most[0];
#pragma unroll
  for (int g = 1; g < KEYS / 16; ++g) mx = fmaxf(mx, most[g]);
  return sum;
}

// A block Hadamard matrix's column in the rows' order: coordinate pi(j) has j here,
// and the sign of j in bit 15.
__device__ __forceinline__ void invert(const Rotation& r, uint16_t* inv, int tid, int d) {
  if (r.perm && tid < d) inv[r.perm[tid]] = (uint16_t)(tid | ((r.signs[tid >> 5] >> (tid & 31) & 1u) << 15));
}
// Eight entries (16 bits each, `one` is 1 in their type) of Pi without its factor
// 1 / sqrt h, as a chunk of a K-major operand: row j, columns 8 c + 0..7 of Pi, or
// (TRANSPOSED) row i, columns 8 c + 0..7 of its transpose.
template <bool TRANSPOSED>
__device__ __forceinline__ uint4 turn_chunk(const uint16_t* inv, int row, int c, int h, uint32_t one) {
  uint32_t o[4];
  const uint4 w = TRANSPOSED ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(inv + 8 * c);
  const uint32_t its[4] = {w.x, w.y, w.z, w.w};
  const uint32_t own = TRANSPOSED ? inv[row] : 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t e[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t code = TRANSPOSED ? own : (its[k] >> (16 * u)) & 0xFFFFu;
      const uint32_t j = code & 0x7FFFu, j2 = TRANSPOSED ? 8u * c + 2 * k + u : (uint32_t)row;
      const uint32_t sign = (code ^ ((uint32_t)__popc(j & j2 & (uint32_t)(h - 1)) << 15)) & 0x8000u;
      e[u] = ((j ^ j2) & ~(uint32_t)(h - 1)) ? 0u : one | sign;
    }
    o[k] = e[0] | e[1] << 16;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D, bool TWO>
struct Smem {
  static constexpr int KT = 128;                             // keys of a step
  static constexpr int VST = TWO && D == 128 ? 1 : 2;        // stages of values
  static constexpr int kOperand = 2 * D * KT;                // bytes of a stage of keys, of values
  static constexpr int kTileQ = kTileRows * D * 2;           // of a tile's queries
  static constexpr int kKeys = 0, kValues = kOperand, kQuery = (1 + VST) * kOperand;
  static constexpr int kLow = kQuery + 2 * kTileQ;           // the queries' second term
  static constexpr int kScales = kLow + (TWO ? 2 * kTileQ : 0);             // [2][KT / 16] (key scale, ev, 2^-ev)
  static constexpr int kInverse = kScales + 2 * (KT / 16) * 16;             // [D] 16 bits: see invert
  static constexpr int kStat = kInverse + 2 * D;                            // [rows] reference, sum
  static constexpr int kBars = kStat + kRows * 8;
  static constexpr int kTotal = kBars + 192;
  static constexpr int kAlloc = kTotal + 1024;  // room to align the base
  // Outside the steps: the matrix in the values' first stage; the sums' second terms
  // in the queries' second terms' place, or the keys' and the values' second stage.
  static constexpr int kMatrix = kValues;
  static constexpr int kSumLow0 = TWO ? kLow : kKeys, kSumLow1 = TWO ? kLow + kTileQ : kValues + kOperand;
  static_assert(D * D * 2 <= kOperand && kTileQ <= kOperand, "what stands in the operands' place");
  static_assert(kRows * D * 4 <= kScales, "the rows' sums stand in the operands' place at the end");
  static_assert(kAlloc <= 227 * 1024, "shared memory of a CTA");
};

template <typename T, int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Args a) {
  using S = Smem<D, TWO>;
  constexpr int KT = S::KT, HK = KT / 2, LPR = D / 8, VST = S::VST;
  extern __shared__ unsigned char sm_raw[];
  chain_wait();
  unsigned char* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint16_t* inv = reinterpret_cast<uint16_t*>(sm + S::kInverse);
  float2* row_stat = reinterpret_cast<float2*>(sm + S::kStat);
  float4* scales = reinterpret_cast<float4*>(sm + S::kScales);
  const uint32_t bars = base + S::kBars;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + S::kBars + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::kBars + 164);
  auto bar = [&](int i) { return bars + 8u * i; };
  // of the two tiles (S_FULL + w) and of a tile's halves (P_FULL + 2 w + half)
  constexpr int K_FULL = 0, K_EMPTY = 1, V_FULL = 2, V_EMPTY = 4, S_FULL = 6, P_FULL = 8, HALF = 12, O_FULL = 14, TURN = 16, END = 18;

  if (tid == 0) {
    mbar_init(bar(K_FULL), 4), mbar_init(bar(K_EMPTY), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(V_FULL + i), 4), mbar_init(bar(V_EMPTY + i), 1);
      mbar_init(bar(S_FULL + i), 1), mbar_init(bar(HALF + i), 1), mbar_init(bar(O_FULL + i), 1);
      mbar_init(bar(P_FULL + 2 * i), 4), mbar_init(bar(P_FULL + 2 * i + 1), 4);
      mbar_init(bar(TURN + i), 1);
    }
    mbar_init(bar(END), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  invert(a.r, inv, tid, D);
  const int cta = blockIdx.x;
  const Share sh = find_share<kRows, KT, kStart, kThreads, kSpare>(a, cta, gridDim.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  long long at = sh.size * cta;
  const long long stop = min(sh.total, at + sh.size);
  int4 desc = make_int4(0, 0, 0, 0);
  int b = sh.b;
  long long into = sh.into;
  // the barriers' phases: steps of the keys, of each tile, items of each tile, turns
  uint32_t steps = 0, tile_steps[2] = {0, 0}, tile_items[2] = {0, 0}, turns = 0;
  const int l = tid % LPR;
  const int plog = 31 - __clz(a.c.page);

  while (at < stop && b < a.B) {
    const Seq s = load_seq(a, b, false);
    const long long per_head = units_before<kRows, KT, kStart>(a, s, row_tiles<kRows>(s));
    if (into >= per_head * a.c.heads) {
      ++b;
      into = 0;
      continue;
    }
    const Part part = find_part<kRows, KT, kStart>(a, s, per_head, into, stop - at);
    const int h = part.h, qt = part.qt, keys = part.keys, take = part.t1 - part.t0;
    const bool first = part.t0 == 0, last = part.t1 == part.tiles;
    const size_t slot = ((size_t)2 * cta + (first ? 1 : 0)) * kRows;
    const long long item_end = at - into + part.end;
    at += part.units;
    into += part.units;
    if (take == 0) {  // no key tile: nothing to do, but a piece that the join counts on says so
      if (part.t0 > 0 && tid < kRows)
        *reinterpret_cast<float2*>(a.stat + 2 * (slot + tid)) = make_float2(-INFINITY, 0.0f);
      continue;
    }
    const int rows = min(kRows, s.rows - qt * kRows);
    const int tok0 = part.t0 * KT;
    // steps of each tile: the second may have no rows, the first may see fewer keys
    int tile_take[2] = {take, rows > kTileRows ? take : 0};
    if (a.causal && rows > kTileRows) {
      const int seen = max(1, s.len - s.n + row_token(a, qt * kRows + kTileRows - 1) + 1);
      tile_take[0] = min(take, max(0, (seen + KT - 1) / KT - part.t0));
    }

    const int tiles = rows > kTileRows ? 2 : 1;
    const bool turned = a.r.perm != nullptr;
    constexpr uint32_t one = std::is_same<T, __nv_bfloat16>::value ? 0x3F80u : 0x3C00u;
    constexpr int PASS = 256 / LPR;
    if (warp < 8) {
      // the item's query rows as they come, as operands (zeros for rows that are not there)
      const T* q = static_cast<const T*>(a.q) + (long long)s.cu0 * a.qt + (long long)h * a.group * a.qh + 8 * l;
#pragma unroll 8
      for (int p = 0; p < tiles * kTileRows; p += PASS) {
        const int r = p + tid / LPR, tr = r & (kTileRows - 1), gr = qt * kRows + r, i = row_token(a, gr);
        copy16(base + S::kQuery + (r / kTileRows) * S::kTileQ + (l >> 3) * (kTileRows * 128) + tr * 128 +
                   (((l & 7) ^ (tr & 7)) << 4),
               r < rows ? q + i * a.qt + (gr - i * a.group) * a.qh : q, r < rows ? 16u : 0u);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }

    if (warp >= 8 && warp < 12) {
      // ---- expanding the codes ----
      // Keys: eight lanes beside one another have two rows' 16-byte pieces of one
      // 128-byte block, which lie in different banks.  Values: a lane takes eight
      // tokens and VB bytes of each; eight lanes beside one another have eight token
      // groups, whose chunks lie in different banks.
      const int ct = tid - 256;
      constexpr int KP = (KT / 32) * (D / 64);         // 16-byte pieces of keys of a lane
      constexpr int VB = KT * D / 1024, VW = VB / 4;   // bytes and words of a token's values
      const int kr = ct >> 2, kc = ct & 3;
      const int vt = 8 * (warp & 1) + (lane & 7);
      const int vd = (((warp - 8) >> 1) * 4 + (lane >> 3)) * VB;
      const int* table = a.table + (size_t)b * a.width;
      auto row_at = [&](int tok) -> size_t {  // row of codes of a token (some row where there is none)
        int page = 0;
        if (tok < keys) {
          page = table[tok >> plog];
          if (page < 0 || page >= a.c.n_pages) page = 0;
        }
        return (((size_t)page * a.c.heads + h) << plog) + (tok & (a.c.page - 1));
      };
      uint32_t code[4 * KP];  // of the keys or the values, whichever comes next
      static_assert(8 * VW == 4 * KP, "as many codes either way");
      auto load_k = [&](int t) {
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {
          const int8_t* p = a.c.k + row_at(tok0 + t * KT + 32 * i + kr) * D + 16 * kc;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + 64 * j);
            uint32_t* to = code + 4 * (i * (D / 64) + j);
            to[0] = w.x, to[1] = w.y, to[2] = w.z, to[3] = w.w;
          }
        }
      };
      auto load_v = [&](int t) {
        const int8_t* p = a.c.v + row_at(tok0 + t * KT + 8 * vt) * D + vd;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (VW == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + j * D);
            code[4 * j] = w.x, code[4 * j + 1] = w.y, code[4 * j + 2] = w.z, code[4 * j + 3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(p + j * D);
            code[2 * j] = w.x, code[2 * j + 1] = w.y;
          }
        }
      };
      float2 sc = make_float2(0.0f, 1.0f);
      auto load_scales = [&](int t) {  // a thread for each group of 16 tokens
        const int tok = tok0 + t * KT + 16 * ct;
        sc = make_float2(0.0f, 1.0f);  // a key scale of 0: no keys
        if (tok < keys) {
          const int page = table[tok >> plog];
          if (page >= 0 && page < a.c.n_pages) {
            const size_t ph = (size_t)page * a.c.heads + h;
            sc = make_float2(a.c.ks[ph], a.c.vs[ph]);
          } else {
            bad_index(a.status);
          }
        }
      };
      load_k(0);
      if (ct < KT / 16) load_scales(0);
      if (turned)
        for (int c = tid - 256; c < D * LPR; c += 160) {
          const uint4 w = turn_chunk<false>(inv, c / LPR, c % LPR, a.r.h, one);
          sts128(base + S::kMatrix + ((c % LPR) >> 3) * (D * 128) + (c / LPR) * 128 + (((c & 7) ^ (c / LPR & 7)) << 4), w.x, w.y,
                 w.z, w.w);
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      for (int t = 0; t < take; ++t) {
        const uint32_t it = steps + t;
        wait_bounded(bar(K_EMPTY), (it & 1u) ^ 1u, abort_flag, a.status);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {
          const int n = 32 * i + kr;
#pragma unroll
          for (int j = 0; j < D / 64; ++j)
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // eight codes: one 16-byte chunk
              const uint32_t* w = code + 4 * (i * (D / 64) + j) + 2 * u;
              const uint32_t w0 = w[0] ^ 0x80808080u, w1 = w[1] ^ 0x80808080u;
              sts128(base + S::kKeys + j * (KT * 128) + n * 128 + (((2 * kc + u) ^ (n & 7)) << 4), bytes2(w0, 0x4140),
                     bytes2(w0, 0x4342), bytes2(w1, 0x4140), bytes2(w1, 0x4342));
            }
        }
        load_v(t);
        if (ct < KT / 16) {
          const int ev = min(max(scale_exp(sc.y), -126), 126);
          scales[(it & 1u) * (KT / 16) + ct] = make_float4(sc.x, (float)ev, pow2(-ev), 0.0f);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && !a.stall) mbar_arrive(bar(K_FULL));
        if (t + 1 < take && ct < KT / 16) load_scales(t + 1);

        const uint32_t st = it % VST;
        if (t == 0 && turned) {  // the matrix stands in the values' place
          wait_bounded(bar(TURN), turns & 1u, abort_flag, a.status);
          wait_bounded(bar(TURN + 1), turns & 1u, abort_flag, a.status);
        }
        wait_bounded(bar(V_EMPTY + st), ((it / VST) & 1u) ^ 1u, abort_flag, a.status);
        __syncwarp();
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t o[4][4];  // [coordinate][pair of tokens]
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t x0 = code[VW * (2 * q) + w] ^ 0x80808080u, x1 = code[VW * (2 * q + 1) + w] ^ 0x80808080u;
            const uint32_t lo = __byte_perm(x0, x1, 0x5140), hi = __byte_perm(x0, x1, 0x7362);
            o[0][q] = bytes2(lo, 0x4140), o[1][q] = bytes2(lo, 0x4342);
            o[2][q] = bytes2(hi, 0x4140), o[3][q] = bytes2(hi, 0x4342);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int d = vd + 4 * w + k;
            sts128(base + S::kValues + st * S::kOperand + (vt >> 3) * (D * 128) + d * 128 + (((vt & 7) ^ (d & 7)) << 4),
                   o[k][0], o[k][1], o[k][2], o[k][3]);
          }
        }
        if (t + 1 < take) load_k(t + 1);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(V_FULL + st));
      }
    } else if (warp == 12) {
      // ---- products: a tile's sum, then its next scores, while the other tile's weights are made ----
      if (turned)
        for (int c = tid - 256; c < D * LPR; c += 160) {
          const uint4 w = turn_chunk<false>(inv, c / LPR, c % LPR, a.r.h, one);
          sts128(base + S::kMatrix + ((c % LPR) >> 3) * (D * 128) + (c / LPR) * 128 + (((c & 7) ^ (c / LPR & 7)) << 4), w.x, w.y,
                 w.z, w.w);
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      const uint64_t md = desc_sw128(base + S::kMatrix);
      if (turned) {
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint64_t qd = desc_sw128(base + S::kQuery + w * S::kTileQ);
            if (w < tiles) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                mma_ss(tmem + kColS + 128 * w, qd + (uint64_t)((k >> 2) * (kTileRows * 8) + (k & 3) * 2),
                       md + (uint64_t)((k >> 2) * (D * 8) + (k & 3) * 2), idesc_of<T, D>(), k > 0);
            }
            commit(bar(TURN + w));
          }
        }
        __syncwarp();
      }
      asm volatile("bar.sync 1, 288;" ::: "memory");  // with the rows' warps: the queries stand
      const uint32_t u_base = uniform(base), u_tmem = uniform(tmem), u_steps = uniform(steps), u_bars = u_base + S::kBars;
      const int u_take = (int)uniform((uint32_t)take);
      const int takes[2] = {(int)uniform((uint32_t)tile_take[0]), (int)uniform((uint32_t)tile_take[1])};
      const uint32_t phase[2] = {uniform(tile_steps[0]), uniform(tile_steps[1])};
      auto u_bar = [&](int i) { return u_bars + 8u * i; };
      const uint64_t kd = desc_sw128(u_base + S::kKeys), vd0 = desc_sw128(u_base + S::kValues);
      const uint64_t qd0 = desc_sw128(u_base + S::kQuery), ld0 = desc_sw128(u_base + S::kLow);
      auto scores = [&](int w, int t) {
        if (t == 0 || w == 0 || takes[0] <= t) wait_bounded(u_bar(K_FULL), (u_steps + t) & 1u, abort_flag, a.status);
        __syncwarp();
        tc_fence_after();
        const uint64_t qd = qd0 + (uint64_t)(w * (S::kTileQ / 16)), ld = ld0 + (uint64_t)(w * (S::kTileQ / 16));
        const uint32_t to = u_tmem + kColS + 128 * w, full = u_bar(S_FULL + w);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(to, qd + (uint64_t)((k >> 2) * (kTileRows * 8) + (k & 3) * 2),
                   kd + (uint64_t)((k >> 2) * (KT * 8) + (k & 3) * 2), idesc<KT>(), k > 0);
          if constexpr (TWO) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(to, ld + (uint64_t)((k >> 2) * (kTileRows * 8) + (k & 3) * 2),
                     kd + (uint64_t)((k >> 2) * (KT * 8) + (k & 3) * 2), idesc<KT>(), 1u);
          }
          commit(full);
        }
        __syncwarp();
      };
      auto keys_done = [&]() {
        const uint32_t empty = u_bar(K_EMPTY);
        if (elect_one()) commit(empty);
        __syncwarp();
      };
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (takes[w] > 0) scores(w, 0);
      keys_done();
      for (int t = 0; t < u_take; ++t) {
        const uint32_t it = u_steps + t, st = it % VST;
        wait_bounded(u_bar(V_FULL + st), (it / VST) & 1u, abort_flag, a.status);
        const uint64_t vd = vd0 + (uint64_t)(st * (S::kOperand / 16));
        const uint32_t empty = u_bar(V_EMPTY + st);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (t < takes[w]) {
            const uint32_t to = u_tmem + kColO + 128 * w, from = u_tmem + kColS + 128 * w;
            const uint32_t half = u_bar(HALF + w), done = u_bar(O_FULL + w);
            const bool end = t + 1 == takes[w];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              wait_bounded(u_bar(P_FULL + 2 * w + hf), (phase[w] + t) & 1u, abort_flag, a.status);
              __syncwarp();
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = hf * (HK / 16); k < (hf + 1) * (HK / 16); ++k)
                  mma_ts<D>(to, from + 8 * k, vd + (uint64_t)((k >> 2) * (D * 8) + (k & 3) * 2), t > 0 || k > 0);
                if (hf == 0)
                  commit(half);
                else if (end)
                  commit(done);
              }
              __syncwarp();
            }
          }
          if (w == 1) {
            if (elect_one()) commit(empty);
            __syncwarp();
          }
          if (t + 1 < takes[w]) scores(w, t + 1);
        }
        if (t + 1 < u_take) keys_done();
      }
    } else {
      // ---- weights ----
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      const int w = warp >> 2, tr = tid & (kTileRows - 1);
      const uint32_t tmem_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * w;  // this warp's lanes
      const int my_take = w ? tile_take[1] : tile_take[0];
      const uint32_t my_steps = w ? tile_steps[1] : tile_steps[0];
      const uint32_t my_query = base + S::kQuery + w * S::kTileQ + tr * 128;
      // this thread's row: turned, scaled by a power of two, fp16, back into the operand's place
      float fac = 0.0f;
      int lim = 0x7FFFFFFF;  // a row that is not there is not masked, and not used
      if (turned) {
        wait_bounded(bar(TURN + w), turns & 1u, abort_flag, a.status);
        __syncwarp();
        tc_fence_after();
      }
      if (w < tiles) {
        auto get = [&](int c, float (&x)[32]) {  // coordinates 32 c .. 32 c + 31
          if (turned) {
            uint32_t v[32];
            tmem_ld32(tmem_row + kColS + 32 * c, v);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float y[8];
              unpack8<T>(lds128(my_query + (c >> 1) * (kTileRows * 128) + (((4 * (c & 1) + j) ^ (tr & 7)) << 4)), y);
#pragma unroll
              for (int q = 0; q < 8; ++q) x[8 * j + q] = y[q];
            }
          }
        };
        float top = 0.0f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float x[32];
          get(c, x);
#pragma unroll
          for (int j = 0; j < 32; ++j) top = fmaxf(top, fabsf(x[j]));
        }
        const int e = min(max(scale_exp(top), -100), 120);
        const float f = pow2(-e);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float x[32];
          get(c, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = x[8 * j + q] * f;
            const uint4 hi = pack8<__half>(y);
            const uint32_t to = (c >> 1) * (kTileRows * 128) + (((4 * (c & 1) + j) ^ (tr & 7)) << 4);
            sts128(my_query + to, hi.x, hi.y, hi.z, hi.w);
            if constexpr (TWO) {
              float z[8];
              unpack8<__half>(hi, z);
#pragma unroll
              for (int q = 0; q < 8; ++q) z[q] = y[q] - z[q];
              const uint4 lo = pack8<__half>(z);
              sts128(base + S::kLow + w * S::kTileQ + tr * 128 + to, lo.x, lo.y, lo.z, lo.w);
            }
          }
        }
        if (tid < rows) {
          fac = pow2(e) * a.scale * (turned ? a.r.norm : 1.0f);
          lim = a.causal ? s.len - s.n + row_token(a, qt * kRows + tid) + 1 : s.len;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      asm volatile("bar.sync 1, 288;" ::: "memory");
      float top = 0.0f, sum = 0.0f;
      bool none = true;  // no key seen so far: the reference says nothing
      for (int t = 0; t < my_take; ++t) {
        const uint32_t ph = (my_steps + t) & 1u;
        wait_bounded(bar(S_FULL + w), ph, abort_flag, a.status);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float4* sc = scales + ((steps + t) & 1u) * (KT / 16) + hf * (HK / 16);
          const uint32_t from = tmem_row + kColS + HK * hf;
          const int left = lim - (tok0 + t * KT + HK * hf);  // keys of the half that the row may see
          const bool whole = __all_sync(0xFFFFFFFFu, left >= HK);
          // The weights at once, against the reference so far; in the rare step that
          // raises it (a weight above 2^15.9, or the first keys of a row) once more
          // from the scores, which still stand in TMEM.
          uint32_t p[HK / 2];
          for (int tries = 0; tries < 2; ++tries) {
            float most[HK / 16], mx;
            const float more = whole ? weigh<HK, false>(from, sc, fac, top, left, p, most, mx)
                                     : weigh<HK, true>(from, sc, fac, top, left, p, most, mx);
            const bool raise = mx > kRaise || (none && mx > -INFINITY);
            if (tries > 0 || !__any_sync(0xFFFFFFFFu, raise)) {
              sum += more;
              break;
            }
            float low = mx;  // the least of the groups' largest exponents
#pragma unroll
            for (int g = 0; g < HK / 16; ++g) low = most[g] > -INFINITY ? fminf(low, most[g]) : low;
            const float up = raise ? fmaxf(mx - kShift, fminf(mx, low + kRoom)) : 0.0f;
            const float f = none ? 1.0f : ex2(-up);  // nothing to rescale before the first key
            top += up;
            if (raise) none = false;
            sum *= f;
            if (hf == 1) {  // the first half's products must have been added
              wait_bounded(bar(HALF + w), ph, abort_flag, a.status);
              __syncwarp();
              tc_fence_after();
            }
            if (t > 0 || hf > 0) {  // the sum so far stands in TMEM, and no product is under way
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16(tmem_row + kColO + c, o);
                wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st16(tmem_row + kColO + c, o);
              }
            }
          }
          tmem_st32(tmem_row + kColS + 32 * hf, p);
          wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(P_FULL + 2 * w + hf));
        }
      }
      row_stat[tid] = make_float2(none && sum == sum ? -INFINITY : top, sum);  // (a NaN query's piece counts)
    }
    // Both tiles are done: what the operands stood in is free.
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (tile_take[w] > 0) wait_bounded(bar(O_FULL + w), tile_items[w] & 1u, abort_flag, a.status);
    __syncwarp();
    tc_fence_after();
    const bool whole_item = first && last;
    float row_back = 1.0f;  // this thread's row's power of two in the turn back
    turns += turned;
    if (warp < 8) {
      const int w = warp >> 2, tr = tid & (kTileRows - 1);
      const uint32_t tmem_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * w;
      const uint32_t my_query = base + S::kQuery + w * S::kTileQ + tr * 128;
      const bool some = (w ? tile_take[1] : tile_take[0]) > 0;
      if (whole_item && w < tiles) {
        // the rows as operands of the turn back, in two terms, or as they are stored
        const float y = row_stat[tid].y;
        float f = (y > 0.0f ? 1.0f / y : y == 0.0f ? 0.0f : y) * (turned ? a.r.norm : 1.0f);
        if (std::is_same<T, __half>::value && turned) {  // fp16 terms: beside a power of two, for their range
          float top = 0.0f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tmem_row + kColO + c, o);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, fabsf(__uint_as_float(o[j])));
          }
          const int e = min(max(scale_exp(top * f), -60), 60);
          f *= pow2(-e), row_back = pow2(e);
        }
        const uint32_t my_low = base + (w ? S::kSumLow1 : S::kSumLow0) + tr * 128;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(tmem_row + kColO + c, o);
          wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[8], z[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(o[8 * j + q]) * f;
            const uint4 hi = pack8<T>(x);
            const uint32_t to = (c >> 6) * (kTileRows * 128) + (((((c >> 3) & 7) + j) ^ (tr & 7)) << 4);
            sts128(my_query + to, hi.x, hi.y, hi.z, hi.w);
            if (turned) {
              unpack8<T>(hi, z);
#pragma unroll
              for (int q = 0; q < 8; ++q) z[q] = x[q] - z[q];
              const uint4 lo = pack8<T>(z);
              sts128(my_low + to, lo.x, lo.y, lo.z, lo.w);
            }
          }
        }
      } else if (!whole_item) {
        // a piece: the rows' sums as they are, 16-byte chunks turned by the row
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(tmem_row + kColO + c, o);
          wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t to = base + tid * (D * 4) + (((c / 4 + j) ^ (tid & 7)) << 4);
            if (some)
              sts128(to, o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            else
              sts128(to, 0u, 0u, 0u, 0u);
          }
        }
      }
    } else if (whole_item && turned) {
      for (int c = tid - 256; c < D * LPR; c += 160) {
        const uint4 w = turn_chunk<true>(inv, c / LPR, c % LPR, a.r.h, one);
        sts128(base + S::kMatrix + ((c % LPR) >> 3) * (D * 128) + (c / LPR) * 128 + (((c & 7) ^ (c / LPR & 7)) << 4), w.x, w.y, w.z,
               w.w);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (whole_item && turned) {
      if (warp == 12) {
        if (elect_one()) {
          const uint64_t md = desc_sw128(base + S::kMatrix);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w < tiles) {
#pragma unroll
              for (int term = 0; term < 2; ++term) {
                const uint64_t od = desc_sw128(base + (term == 0 ? S::kQuery + w * S::kTileQ : w ? S::kSumLow1 : S::kSumLow0));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_ss(tmem + kColS + 128 * w, od + (uint64_t)((k >> 2) * (kTileRows * 8) + (k & 3) * 2),
                         md + (uint64_t)((k >> 2) * (D * 8) + (k & 3) * 2), idesc_of<T, D>(), term > 0 || k > 0);
              }
            }
            commit(bar(TURN + w));
          }
        }
        __syncwarp();
      } else if (warp < 8) {
        const int w = warp >> 2, tr = tid & (kTileRows - 1);
        const uint32_t tmem_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * w;
        const uint32_t my_query = base + S::kQuery + w * S::kTileQ + tr * 128;
        wait_bounded(bar(TURN + w), turns & 1u, abort_flag, a.status);
        __syncwarp();
        tc_fence_after();
        if (w < tiles) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tmem_row + kColS + c, o);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float x[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(o[8 * j + q]) * row_back;
              const uint4 hi = pack8<T>(x);
              sts128(my_query + (c >> 6) * (kTileRows * 128) + (((((c >> 3) & 7) + j) ^ (tr & 7)) << 4), hi.x, hi.y, hi.z, hi.w);
            }
          }
        }
        tc_fence_before();
      }
      ++turns;
      __syncthreads();
    }
    if (warp < 8) {
      if (whole_item) {
        T* out = static_cast<T*>(a.out) + (long long)s.cu0 * a.ot + (long long)h * a.group * a.oh + 8 * l;
#pragma unroll 8
        for (int r = tid / LPR; r < rows; r += PASS) {
          const int tr = r & (kTileRows - 1), gr = qt * kRows + r, i = row_token(a, gr);
          *reinterpret_cast<uint4*>(out + i * a.ot + (gr - i * a.group) * a.oh) =
              lds128(base + S::kQuery + (r / kTileRows) * S::kTileQ + (l >> 3) * (kTileRows * 128) + tr * 128 +
                     (((l & 7) ^ (tr & 7)) << 4));
        }
      } else {
#pragma unroll 8
        for (int r = tid / (D / 4); r < rows; r += 256 / (D / 4)) {
          const int c = tid % (D / 4);
          *reinterpret_cast<uint4*>(a.piece + (slot + r) * D + 4 * c) = lds128(base + r * (D * 4) + ((c ^ (r & 7)) << 4));
        }
        if (tid < rows) *reinterpret_cast<float2*>(a.stat + 2 * (slot + tid)) = row_stat[tid];
      }
    }
    if (first && !last) desc = make_int4((int)((item_end - 1) / sh.size) - cta + 1, b, h, qt);
    if (__syncthreads_or(*abort_flag)) break;
    steps += take;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      tile_steps[w] += tile_take[w];
      tile_items[w] += tile_take[w] > 0;
    }
  }
  chain_next();
  if (tid == 0) a.desc[cta] = desc;
  if (warp == 12) {  // nothing may arrive in shared memory or TMEM that is given back
    if (elect_one()) commit(bar(END));
    __syncwarp();
    wait_own(bar(END));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
}

template <typename T, int D, bool TWO>
int launch(const Args& a, void* stream) {
  using S = Smem<D, TWO>;
  auto kern = chunk_kernel<T, D, TWO>;
  int per_sm = 0, nsm = 0;
  if (int rc = occupancy(reinterpret_cast<const void*>(kern), S::kAlloc, kThreads, 0, &per_sm)) return rc;
  if (int rc = sm_count(&nsm)) return rc;
  if (per_sm < 1) return fail(OQ_ERR_UNSUPPORTED, "attention kernel does not fit");
  // no more CTAs than units that there can be
  const long long rows = (long long)a.T * a.group;
  const long long items = std::min<long long>((rows + kRows - 1) / kRows + a.B, rows) * a.c.heads;
  const long long units = items * (kStart + 1 + (long long)a.width * a.c.page / S::KT);
  const int ctas = (int)std::min<long long>(units, std::min(nsm, kChunkCtas));
  if (int rc = launch_chained("attention", kern, dim3((unsigned)ctas), kThreads, S::kAlloc, stream, a)) return rc;
  return launch_chained("attention join", join_kernel<T, D, kRows, 1>, dim3((unsigned)ctas, kRows / 4), 128, 0, stream, a);
}

}  // namespace

int launch_cattn_chunk(const cattn::Args& a, int dtype, int d, void* stream) {
  if (dtype == OQ_BF16) return d == 128 ? launch<__nv_bfloat16, 128, false>(a, stream) : launch<__nv_bfloat16, 64, false>(a, stream);
  // fp16 rows that are not turned are exact in one term
  if (!a.r.perm) return d == 128 ? launch<__half, 128, false>(a, stream) : launch<__half, 64, false>(a, stream);
  return d == 128 ? launch<__half, 128, true>(a, stream) : launch<__half, 64, true>(a, stream);
}

}  // namespace oq
