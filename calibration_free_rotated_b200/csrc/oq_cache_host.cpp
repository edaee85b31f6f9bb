// Host side of the cache operators: the rope handle and the argument checks.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "oq_internal.h"

using namespace oq;

namespace {

// Most rows, and most tokens of a sequence: the kernels look a few tiles ahead in 32-bit
// places.
constexpr long long kMost = 0x7FFF0000ll;

int rope_table(oq_rope_t r, const unsigned long long** freq, const uint8_t** axis) {
  int dev;
  if (int rc = current_device(&dev)) return rc;
  std::lock_guard<std::mutex> lk(r->mu);
  const size_t n = r->freq.size();
  if (!r->dev_table[dev]) {
    unsigned char t[9 * 256];
    std::memcpy(t, r->freq.data(), 8 * n);
    std::memcpy(t + 8 * n, r->axis.data(), n);
    void* p = nullptr;
    if (int rc = device_alloc(&p, 9 * n, "rope table")) return rc;
    cudaError_t e = cudaMemcpy(p, t, 9 * n, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) {
      cudaFree(p);
      return fail(OQ_ERR_CUDA, "uploading the rope table: %s", cudaGetErrorString(e));
    }
    r->dev_table[dev] = static_cast<unsigned char*>(p);
  }
  *freq = reinterpret_cast<const unsigned long long*>(r->dev_table[dev]);
  *axis = r->dev_table[dev] + 8 * n;
  return OQ_OK;
}

// Base and strides (in elements of `size` bytes) of a tensor read or written in 16-byte vectors.
int check_rows(const char* what, const void* p, long long token, long long head, int size) {
  if (!p) return fail(OQ_ERR_ARG, "%s is NULL", what);
  if (!aligned16(p)) return fail(OQ_ERR_ALIGN, "%s must be 16-byte aligned", what);
  if ((token * size) % 16 != 0 || (head * size) % 16 != 0)
    return fail(OQ_ERR_ALIGN, "%s: strides (%lld, %lld) must be multiples of 16 bytes", what, token, head);
  return OQ_OK;
}

int check_cache(const oq_kvcache* c) {
  if (!c) return fail(OQ_ERR_ARG, "NULL cache");
  if (c->n_pages < 1 || c->heads < 1)
    return fail(OQ_ERR_ARG, "a cache needs n_pages >= 1 and heads >= 1 (got %d, %d)", c->n_pages, c->heads);
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
    return fail(OQ_ERR_UNSUPPORTED, "pages hold 16, 32, 64 or 128 tokens (got %d)", c->page);
  if (c->d != 64 && c->d != 128) return fail(OQ_ERR_UNSUPPORTED, "the cache needs d 64 or 128 (got %d)", c->d);
  if (c->heads > 65535) return fail(OQ_ERR_UNSUPPORTED, "heads <= 65535 (got %d)", c->heads);
  if ((long long)c->n_pages * c->page > 0x7FFFFFFFll)
    return fail(OQ_ERR_UNSUPPORTED, "a cache holds fewer than 2^31 tokens (%d pages of %d)", c->n_pages, c->page);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(OQ_ERR_ARG, "NULL cache buffer");
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return fail(OQ_ERR_ALIGN, "cache buffers must be 16-byte aligned");
  return OQ_OK;
}

int check_turn(const oq_kvcache* c, oq_rpbh_t r) {
  if (!r) return OQ_OK;
  if (r->d != c->d) return fail(OQ_ERR_ARG, "rotation of width %d on heads of %d", r->d, c->d);
  if (r->rounds != 1) return fail(OQ_ERR_UNSUPPORTED, "the cache takes one-round rotations (got %d rounds)", r->rounds);
  if (r->h < 32) return fail(OQ_ERR_UNSUPPORTED, "the cache needs a rotation block >= 32 (h=%d)", r->h);
  return OQ_OK;
}

int check_batch(const oq_kvcache* c, int dtype, int T, const void* cu, const void* at, int B, const void* table,
                int width) {
  if (dtype != OQ_BF16 && dtype != OQ_FP16)
    return fail(dtype == OQ_FP32 ? OQ_ERR_UNSUPPORTED : OQ_ERR_ARG, "dtype %d: the cache takes OQ_BF16 or OQ_FP16",
                dtype);
  if (T < 0 || B < 0) return fail(OQ_ERR_ARG, "T and B must be >= 0 (got %d, %d)", T, B);
  if (T == 0 || B == 0) return OQ_OK;
  if (width < 1) return fail(OQ_ERR_ARG, "the page table needs a width >= 1 (got %d)", width);
  if (T > kMost) return fail(OQ_ERR_UNSUPPORTED, "T must be at most %lld (got %d)", kMost, T);
  if ((long long)width * c->page > kMost)
    return fail(OQ_ERR_UNSUPPORTED, "a sequence holds at most %lld tokens (%d pages of %d)", kMost, width, c->page);
  if (!cu || !at || !table) return fail(OQ_ERR_ARG, "NULL index buffer");
  if (((uintptr_t)cu | (uintptr_t)at | (uintptr_t)table) & 3u)
    return fail(OQ_ERR_ALIGN, "index buffers must be 4-byte aligned");
  return OQ_OK;
}

}  // namespace

extern "C" {

int oq_make_rope(int pairs, const double* freq, const uint8_t* axis, int n_axes, int layout, oq_rope_t* out) {
  clear_error();
  if (!out) return fail(OQ_ERR_ARG, "out is NULL");
  *out = nullptr;
  if (pairs < 1 || pairs > 256) return fail(OQ_ERR_ARG, "pairs must be in 1..256 (got %d)", pairs);
  if (n_axes < 1 || n_axes > 8) return fail(OQ_ERR_ARG, "axes must be in 1..8 (got %d)", n_axes);
  if (layout != OQ_ROPE_INTERLEAVED && layout != OQ_ROPE_HALVES) return fail(OQ_ERR_ARG, "unknown layout %d", layout);
  if (!freq || !axis) return fail(OQ_ERR_ARG, "NULL table");
  for (int p = 0; p < pairs; ++p) {
    if (!std::isfinite(freq[p])) return fail(OQ_ERR_ARG, "frequency %d is not finite", p);
    if (axis[p] >= n_axes) return fail(OQ_ERR_ARG, "pair %d has axis %d of %d", p, axis[p], n_axes);
  }
  oq_rope_t r = new (std::nothrow) oq_rope_s;
  if (!r) return fail(OQ_ERR_NOMEM, "allocating the rope handle");
  r->n_axes = n_axes;
  r->halves = layout == OQ_ROPE_HALVES;
  try {
    r->axis.assign(axis, axis + pairs);
    r->freq.resize(pairs);
  } catch (const std::bad_alloc&) {
    delete r;
    return fail(OQ_ERR_NOMEM, "allocating the rope handle");
  }
  for (int p = 0; p < pairs; ++p) {
    // turns for each position; whole turns drop out, the fraction is kept to 2^-64
    // (long double: 64 bits of mantissa)
    const long double two_pi = 6.283185307179586476925286766559005768L;
    long double t = (long double)freq[p] / two_pi;
    t -= floorl(t);
    const long double v = roundl(t * 18446744073709551616.0L);  // 2^64
    r->freq[p] = v >= 18446744073709551616.0L ? 0u : (uint64_t)v;
  }
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) == cudaSuccess && ndev > 0) {
    const unsigned long long* f;
    const uint8_t* a;
    if (int rc = rope_table(r, &f, &a)) {
      delete r;
      return rc;
    }
  } else {
    cudaGetLastError();
  }
  *out = r;
  return OQ_OK;
}

int oq_rope_info(oq_rope_t rope, int* pairs, int* n_axes, int* layout) {
  clear_error();
  if (!rope) return fail(OQ_ERR_ARG, "NULL rope handle");
  if (pairs) *pairs = (int)rope->freq.size();
  if (n_axes) *n_axes = rope->n_axes;
  if (layout) *layout = rope->halves ? OQ_ROPE_HALVES : OQ_ROPE_INTERLEAVED;
  return OQ_OK;
}

void oq_free_rope(oq_rope_t r) {
  if (!r) return;
  int prev = -1;
  const bool have_prev = cudaGetDevice(&prev) == cudaSuccess;
  for (int dev = 0; dev < OQ_MAX_DEVICES; ++dev)
    if (r->dev_table[dev] && cudaSetDevice(dev) == cudaSuccess) cudaFree(r->dev_table[dev]);
  if (have_prev) cudaSetDevice(prev);
  delete r;
}

int oq_rope_apply(oq_rope_t rope, const void* X, long long x_token, long long x_head, void* Y, long long y_token,
                  long long y_head, int dtype, int T, int heads, int d, const int32_t* pos, int inverse,
                  void* stream) {
  clear_error();
  NvtxRange nvtx("oq_rope_apply");
  if (!rope) return fail(OQ_ERR_ARG, "NULL rope handle");
  if (dtype != OQ_BF16 && dtype != OQ_FP16 && dtype != OQ_FP32) return fail(OQ_ERR_ARG, "unknown dtype %d", dtype);
  if (T < 0 || heads < 0) return fail(OQ_ERR_ARG, "T and heads must be >= 0 (got %d, %d)", T, heads);
  const int pairs = (int)rope->freq.size();
  if (2 * pairs > d) return fail(OQ_ERR_ARG, "%d pairs do not fit into rows of %d", pairs, d);
  if (d % 8 != 0 || d > 512) return fail(OQ_ERR_UNSUPPORTED, "rope needs d %% 8 == 0 and d <= 512 (d=%d)", d);
  if (T > kMost || heads > 65535)
    return fail(OQ_ERR_UNSUPPORTED, "rope needs T <= %lld and heads <= 65535 (got %d, %d)", kMost, T, heads);
  if (rope->halves && pairs % 8 != 0)
    return fail(OQ_ERR_UNSUPPORTED, "the halves layout needs pairs %% 8 == 0 (pairs=%d)", pairs);
  if (T == 0 || heads == 0) return OQ_OK;
  const int size = dtype == OQ_FP32 ? 4 : 2;
  if (int rc = check_rows("X", X, x_token, x_head, size)) return rc;
  if (int rc = check_rows("Y", Y, y_token, y_head, size)) return rc;
  if (X == Y && (x_token != y_token || x_head != y_head))
    return fail(OQ_ERR_ARG, "in place, X and Y need the same strides");
  if (!pos) return fail(OQ_ERR_ARG, "pos is NULL");
  if ((uintptr_t)pos & 3u) return fail(OQ_ERR_ALIGN, "pos must be 4-byte aligned");
  RopeCall c;
  std::memset(&c, 0, sizeof(c));
  if (int rc = rope_table(rope, &c.freq, &c.axis)) return rc;
  c.x = X, c.y = Y, c.pos = pos;
  c.x_token = x_token, c.x_head = x_head, c.y_token = y_token, c.y_head = y_head;
  c.dtype = dtype, c.T = T, c.heads = heads, c.d = d;
  c.n_axes = rope->n_axes, c.pairs = pairs, c.halves = rope->halves, c.inverse = inverse != 0;
  c.stream = stream;
  return finish(launch_rope(c), stream);
}

int oq_cache_write(const oq_kvcache* cache, oq_rpbh_t r, const void* K, long long k_token, long long k_head,
                   const void* V, long long v_token, long long v_head, int dtype, int T, const int32_t* cu,
                   const int32_t* past, int B, const int32_t* table, int width, void* stream) {
  clear_error();
  NvtxRange nvtx("oq_cache_write");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_turn(cache, r)) return rc;
  if (int rc = check_batch(cache, dtype, T, cu, past, B, table, width)) return rc;
  if (T == 0 || B == 0) return OQ_OK;
  if (int rc = check_rows("K", K, k_token, k_head, 2)) return rc;
  if (int rc = check_rows("V", V, v_token, v_head, 2)) return rc;
  CacheCall c;
  std::memset(&c, 0, sizeof(c));
  c.cache = cache, c.r = r, c.k = K, c.v = V;
  c.k_token = k_token, c.k_head = k_head, c.v_token = v_token, c.v_head = v_head;
  c.dtype = dtype, c.B = B, c.T = T, c.width = width;
  c.cu = cu, c.at = past, c.table = table;
  c.stream = stream;
  return finish(launch_cache_write(c), stream);
}

int oq_cache_read(const oq_kvcache* cache, oq_rpbh_t r, void* K, void* V, int dtype, int T, const int32_t* cu,
                  const int32_t* first, int B, const int32_t* table, int width, void* stream) {
  clear_error();
  NvtxRange nvtx("oq_cache_read");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_turn(cache, r)) return rc;
  if (int rc = check_batch(cache, dtype, T, cu, first, B, table, width)) return rc;
  if (T == 0 || B == 0) return OQ_OK;
  if (int rc = check_rows("K", K, 0, 0, 2)) return rc;
  if (int rc = check_rows("V", V, 0, 0, 2)) return rc;
  CacheCall c;
  std::memset(&c, 0, sizeof(c));
  c.cache = cache, c.r = r, c.k_out = K, c.v_out = V;
  c.dtype = dtype, c.B = B, c.T = T, c.width = width;
  c.cu = cu, c.at = first, c.table = table;
  c.stream = stream;
  return finish(launch_cache_read(c), stream);
}

size_t oq_cache_attention_workspace_bytes(const oq_kvcache* cache, int T, int B, int heads) {
  if (!cache || cache->heads < 1 || heads < cache->heads || T <= 0 || B <= 0) return 0;
  return cattn_workspace(T, B, heads / cache->heads, cache->d);
}

int oq_cache_attention(const oq_kvcache* cache, oq_rpbh_t r, const void* Q, long long q_token, long long q_head,
                       void* O, long long o_token, long long o_head, int dtype, int heads, int T, const int32_t* cu,
                       const int32_t* lens, int B, const int32_t* table, int width, int causal, float scale,
                       void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  NvtxRange nvtx("oq_cache_attention");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_turn(cache, r)) return rc;
  if (int rc = check_batch(cache, dtype, T, cu, lens, B, table, width)) return rc;
  if (heads < 1 || heads % cache->heads != 0)
    return fail(OQ_ERR_ARG, "query heads (%d) must be a multiple of the cache's (%d)", heads, cache->heads);
  if (heads > 65535) return fail(OQ_ERR_UNSUPPORTED, "query heads <= 65535 (got %d)", heads);
  if (!std::isfinite(scale)) return fail(OQ_ERR_ARG, "scale must be finite");
  if (T == 0 || B == 0) return OQ_OK;
  if ((long long)T * heads > kMost)
    return fail(OQ_ERR_UNSUPPORTED, "T * heads must be at most %lld (%d, %d)", kMost, T, heads);
  if (int rc = check_rows("Q", Q, q_token, q_head, 2)) return rc;
  if (int rc = check_rows("O", O, o_token, o_head, 2)) return rc;
  if (Q == O) return fail(OQ_ERR_ARG, "O may not be Q");
  const size_t need = oq_cache_attention_workspace_bytes(cache, T, B, heads);
  if (!workspace || workspace_bytes < need)
    return fail(OQ_ERR_ARG, "workspace of %zu bytes is smaller than the %zu needed", workspace ? workspace_bytes : 0,
                need);
  if (!aligned16(workspace)) return fail(OQ_ERR_ALIGN, "workspace must be 16-byte aligned");
  AttnCall c;
  std::memset(&c, 0, sizeof(c));
  c.cache = cache, c.r = r, c.q = Q, c.out = O;
  c.q_token = q_token, c.q_head = q_head, c.o_token = o_token, c.o_head = o_head;
  c.dtype = dtype, c.heads = heads, c.B = B, c.T = T, c.width = width, c.causal = causal != 0;
  c.scale = scale;
  c.cu = cu, c.lens = lens, c.table = table;
  c.workspace = workspace;
  c.stream = stream;
  return finish(launch_cattn(c), stream);
}

}  // extern "C"
