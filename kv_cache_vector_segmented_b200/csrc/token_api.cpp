// C ABI of rotary positions and the exact token cache: argument validation
// (all of it on the host, before the first launch) and the rotary tables.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "internal.h"
#include "retroinfer.h"

using namespace ri;

namespace {

constexpr double kPi = 3.14159265358979323846;

ri_status check_cache(const ri_token_cache* c, const char* what) {
  RI_CHECK(c, RI_ERR_INVALID_ARG, "%s is NULL", what);
  RI_CHECK(c->batch >= 1 && c->num_kv_heads >= 1 && c->capacity >= 1, RI_ERR_INVALID_ARG,
           "%s: batch, num_kv_heads and capacity must be >= 1 (got %d, %d, %d)", what, c->batch,
           c->num_kv_heads, c->capacity);
  RI_CHECK(c->group_size >= 1 && c->group_size <= kMaxGroupHost, RI_ERR_INVALID_ARG,
           "%s: group_size must be in [1, %d] (got %d)", what, kMaxGroupHost, c->group_size);
  RI_CHECK(c->head_dim == 128, RI_ERR_INVALID_ARG, "%s: head_dim must be 128 (got %d)", what,
           c->head_dim);
  RI_CHECK((long long)c->batch * c->num_kv_heads <= 65536, RI_ERR_UNSUPPORTED,
           "%s: batch * num_kv_heads must be <= 65536", what);
  RI_CHECK(c->capacity <= 1 << 28, RI_ERR_UNSUPPORTED, "%s: capacity must be <= 2^28", what);
  return RI_OK;
}

ri_status check_arrays(const ri_token_cache* c, const char* what) {
  const ri_status s = check_cache(c, what);
  if (s != RI_OK) return s;
  const struct { const void* p; const char* name; } a[] = {
      {c->K, "K"}, {c->V, "V"}, {c->pos, "pos"}, {c->weight, "weight"}, {c->lens, "lens"}};
  for (const auto& x : a)
    RI_CHECK(x.p && aligned16(x.p), RI_ERR_INVALID_ARG,
             "%s: %s must be non-NULL and 16-byte aligned", what, x.name);
  return RI_OK;
}

ri_status check_workspace(const void* ws, size_t bytes, size_t need) {
  RI_CHECK(ws && aligned16(ws), RI_ERR_INVALID_ARG,
           "workspace must be non-NULL and 16-byte aligned");
  RI_CHECK(bytes >= need, RI_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", bytes, need);
  return RI_OK;
}

ri_status check_rope(const ri_rope* r, int head_dim) {
  RI_CHECK(r->turns && (reinterpret_cast<uintptr_t>(r->turns) & 7u) == 0, RI_ERR_INVALID_ARG,
           "rope: turns must be non-NULL and 8-byte aligned");
  RI_CHECK(r->rotary_dim >= 2 && r->rotary_dim % 2 == 0 && r->rotary_dim <= head_dim,
           RI_ERR_INVALID_ARG, "rope: rotary_dim must be even and in [2, head_dim] (got %d of %d)",
           r->rotary_dim, head_dim);
  RI_CHECK(std::isfinite(r->magnitude), RI_ERR_INVALID_ARG, "rope: magnitude must be finite");
  return RI_OK;
}

// Rows of 128 bf16 that 16-byte accesses can read.
ri_status check_rows(const ri_heads* x, const char* name) {
  RI_CHECK(x && x->data && aligned16(x->data), RI_ERR_INVALID_ARG,
           "%s must be non-NULL and 16-byte aligned", name);
  RI_CHECK(x->stride_b % 8 == 0 && x->stride_t % 8 == 0 && x->stride_h % 8 == 0,
           RI_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements", name);
  return RI_OK;
}

// Two arrays of one kind: the same one, or apart.
bool same_or_apart(const void* a, size_t na, const void* b, size_t nb) {
  if (a == b) return na == nb;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + na <= y || y + nb <= x;
}

// ri_token_attend; `hand_off` and `wait_ns` as its self-test sets them.
ri_status token_attend(const ri_token_cache* cache, const void* q, const ri_token_prefix* prefix,
                       void* out, float* lse, int32_t add_weight, void* workspace,
                       size_t workspace_bytes, int hand_off, unsigned long long wait_ns,
                       ri_stream_t stream) {
  ri_status st = check_arrays(cache, "token cache");
  if (st != RI_OK) return st;
  RI_CHECK(q && aligned16(q) && out && aligned16(out), RI_ERR_INVALID_ARG,
           "q and out must be non-NULL and 16-byte aligned");
  RI_CHECK(!lse || aligned4(lse), RI_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  TokenAttendArgs a = {};
  if (prefix && prefix->length != 0) {
    RI_CHECK(prefix->length > 0 && prefix->length <= 1 << 28, RI_ERR_INVALID_ARG,
             "prefix length must be in [0, 2^28] (got %d)", prefix->length);
    RI_CHECK(prefix->K && aligned16(prefix->K) && prefix->V && aligned16(prefix->V),
             RI_ERR_INVALID_ARG, "prefix K and V must be non-NULL and 16-byte aligned");
    RI_CHECK(prefix->reserved == 0, RI_ERR_INVALID_ARG, "prefix: reserved must be 0");
    RI_CHECK(prefix->stride_t >= 128 && prefix->stride_t % 8 == 0 &&
                 (cache->num_kv_heads == 1 ||
                  (prefix->stride_h >= 128 && prefix->stride_h % 8 == 0)),
             RI_ERR_INVALID_ARG,
             "prefix strides must be multiples of 8 elements and at least 128");
    a.p = *prefix;
    if (cache->num_kv_heads == 1) a.p.stride_h = a.p.stride_t;
  }
  const size_t need = token_attend_bytes(*cache, a.p.length);
  RI_CHECK(need, RI_ERR_UNSUPPORTED, "prefix of %d tokens: too much work for one call",
           a.p.length);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != RI_OK) return st;
  a.c = *cache;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.add_weight = add_weight != 0;
  a.ws = static_cast<char*>(workspace);
  a.wait_ns = wait_ns;
  a.hand_off = hand_off;
  const cudaError_t e = launch_token_attend(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RI_OK : cuda_fail(e, "token attend launch");
}

}  // namespace

extern "C" {

ri_status ri_rotary_table(const ri_rotary_config* cfg, uint64_t* turns, double* frequencies,
                          double* magnitude) {
  RI_CHECK(cfg && turns && magnitude, RI_ERR_INVALID_ARG,
           "rotary config, turns and magnitude must be non-NULL");
  const int n = cfg->rotary_dim;
  RI_CHECK(n >= 2 && n <= 256 && n % 2 == 0, RI_ERR_INVALID_ARG,
           "rotary_dim must be even and in [2, 256] (got %d)", n);
  RI_CHECK(cfg->scaling >= RI_ROPE_NONE && cfg->scaling <= RI_ROPE_YARN, RI_ERR_INVALID_ARG,
           "unknown rotary scaling %d", cfg->scaling);
  RI_CHECK(std::isfinite(cfg->base) && cfg->base > 1.0, RI_ERR_INVALID_ARG,
           "rotary base must be > 1 (got %g)", cfg->base);
  RI_CHECK(cfg->reserved == 0, RI_ERR_INVALID_ARG, "rotary config: reserved must be 0");
  const bool ramp = cfg->scaling == RI_ROPE_BANDS || cfg->scaling == RI_ROPE_YARN;
  const double factor = cfg->scaling == RI_ROPE_NONE ? 1.0 : cfg->factor;
  RI_CHECK(std::isfinite(factor) && factor > 0.0, RI_ERR_INVALID_ARG,
           "rotary factor must be > 0 (got %g)", cfg->factor);
  if (ramp) {
    RI_CHECK(cfg->original_len >= 1, RI_ERR_INVALID_ARG, "original_len must be >= 1 (got %d)",
             cfg->original_len);
    RI_CHECK(std::isfinite(cfg->low) && std::isfinite(cfg->high) && cfg->low > 0.0 &&
                 cfg->low < cfg->high,
             RI_ERR_INVALID_ARG, "rotary bounds need 0 < low < high (got %g, %g)", cfg->low,
             cfg->high);
  }
  double base = cfg->base;
  if (cfg->scaling == RI_ROPE_NTK) base *= std::pow(factor, n / std::fmax(1.0, n - 2.0));
  double first = 0.0, last = 0.0;
  if (cfg->scaling == RI_ROPE_YARN) {
    auto index = [&](double t) {
      return n * std::log(cfg->original_len / (t * 2 * kPi)) / (2 * std::log(cfg->base));
    };
    first = std::fmax(std::floor(index(cfg->high)), 0.0);
    last = std::fmin(std::ceil(index(cfg->low)), n - 1.0);
  }
  double f_of[128];
  for (int i = 0; i < n / 2; ++i) {
    double f = std::pow(base, -2.0 * i / n);
    if (cfg->scaling == RI_ROPE_LINEAR) {
      f /= factor;
    } else if (cfg->scaling == RI_ROPE_BANDS) {
      double t = (cfg->original_len * f / (2 * kPi) - cfg->low) / (cfg->high - cfg->low);
      t = std::fmin(std::fmax(t, 0.0), 1.0);
      f = (1 - t) * f / factor + t * f;
    } else if (cfg->scaling == RI_ROPE_YARN) {
      double r = (i - first) / std::fmax(last - first, 0.001);
      r = std::fmin(std::fmax(r, 0.0), 1.0);
      f = r * f / factor + (1 - r) * f;
    }
    RI_CHECK(std::isfinite(f) && f >= 0.0 && f < kPi, RI_ERR_INVALID_ARG,
             "rotary frequency %d is %g radians per position: it must be below pi", i, f);
    f_of[i] = f;
  }
  for (int i = 0; i < n / 2; ++i) {
    const long double t = (long double)f_of[i] / (2 * 3.141592653589793238462643383279502884L);
    turns[i] = (uint64_t)(t * 18446744073709551616.0L + 0.5L);
    if (frequencies) frequencies[i] = f_of[i];
  }
  *magnitude =
      cfg->scaling == RI_ROPE_YARN && factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return RI_OK;
}

ri_status ri_rotary(int32_t batch, int32_t tokens, int32_t heads, int32_t head_dim,
                    int32_t dtype, const ri_heads* x, const int32_t* pos, int64_t pos_stride,
                    const ri_rope* rope, const ri_heads* out, int32_t inverse,
                    ri_stream_t stream) {
  RI_CHECK(batch >= 1 && tokens >= 1 && heads >= 1, RI_ERR_INVALID_ARG,
           "batch, tokens and heads must be >= 1 (got %d, %d, %d)", batch, tokens, heads);
  RI_CHECK((long long)batch * tokens < 1ll << 31, RI_ERR_UNSUPPORTED,
           "batch * tokens must be < 2^31 (got %lld)", (long long)batch * tokens);
  RI_CHECK(heads <= 1 << 20, RI_ERR_UNSUPPORTED, "heads must be <= 2^20 (got %d)", heads);
  RI_CHECK(head_dim >= 2 && head_dim <= 256, RI_ERR_INVALID_ARG,
           "head_dim must be in [2, 256] (got %d)", head_dim);
  RI_CHECK(dtype == RI_BF16 || dtype == RI_FP16 || dtype == RI_FP32, RI_ERR_INVALID_ARG,
           "unknown dtype %d", dtype);
  const uintptr_t size = dtype == RI_FP32 ? 4 : 2;
  RI_CHECK(x && out && x->data && out->data &&
               (reinterpret_cast<uintptr_t>(x->data) & (size - 1)) == 0 &&
               (reinterpret_cast<uintptr_t>(out->data) & (size - 1)) == 0,
           RI_ERR_INVALID_ARG, "x and out must be non-NULL and aligned to their element");
  RI_CHECK(pos && aligned4(pos), RI_ERR_INVALID_ARG, "pos must be non-NULL and 4-byte aligned");
  RI_CHECK(rope, RI_ERR_INVALID_ARG, "rope is NULL");
  const ri_status st = check_rope(rope, head_dim);
  if (st != RI_OK) return st;
  RI_CHECK(x->data != out->data ||
               (x->stride_b == out->stride_b && x->stride_t == out->stride_t &&
                x->stride_h == out->stride_h),
           RI_ERR_INVALID_ARG, "out is x's memory with other strides");
  RotaryArgs a{batch, tokens, heads, head_dim, *x, *out, pos, pos_stride, *rope, inverse != 0};
  const cudaError_t e = launch_rotary(a, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RI_OK : cuda_fail(e, "rotary launch");
}

ri_status ri_token_append(const ri_token_cache* cache, int32_t tokens, const ri_heads* k,
                          const ri_heads* v, const int32_t* pos, int64_t pos_stride,
                          const ri_rope* rope, const ri_heads* q, void* q_out,
                          int32_t* lens_out, void* workspace, ri_stream_t stream) {
  ri_status st = check_arrays(cache, "token cache");
  if (st != RI_OK) return st;
  RI_CHECK(tokens >= 1, RI_ERR_INVALID_ARG, "tokens must be >= 1 (got %d)", tokens);
  RI_CHECK((long long)cache->batch * tokens < 1ll << 31, RI_ERR_UNSUPPORTED,
           "batch * tokens must be < 2^31 (got %lld)", (long long)cache->batch * tokens);
  if ((st = check_rows(k, "k")) != RI_OK || (st = check_rows(v, "v")) != RI_OK) return st;
  RI_CHECK(pos && aligned4(pos), RI_ERR_INVALID_ARG, "pos must be non-NULL and 4-byte aligned");
  if (rope && (st = check_rope(rope, 128)) != RI_OK) return st;
  RI_CHECK((q == nullptr) == (q_out == nullptr), RI_ERR_INVALID_ARG,
           "q and q_out must be given together");
  if (q) {
    if ((st = check_rows(q, "q")) != RI_OK) return st;
    RI_CHECK(aligned16(q_out), RI_ERR_INVALID_ARG, "q_out must be 16-byte aligned");
  }
  RI_CHECK(lens_out && aligned4(lens_out), RI_ERR_INVALID_ARG,
           "lens_out must be non-NULL and 4-byte aligned");
  const size_t lens_bytes = (size_t)cache->batch * cache->num_kv_heads * 4;
  RI_CHECK(same_or_apart(cache->lens, lens_bytes, lens_out, lens_bytes), RI_ERR_INVALID_ARG,
           "lens_out must be cache->lens or not overlap it");
  if ((st = check_workspace(workspace, kStatusBytesHost, kStatusBytesHost)) != RI_OK) return st;
  AppendTokensArgs a = {};
  a.c = *cache;
  a.T = tokens;
  a.k = *k;
  a.v = *v;
  if (q) a.q = *q;
  a.q_out = q_out;
  a.pos = pos;
  a.pos_stride = pos_stride;
  if (rope) a.rope = *rope;
  a.lens_out = lens_out;
  a.status = static_cast<int*>(workspace);
  const cudaError_t e = launch_token_append(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RI_OK : cuda_fail(e, "token append launch");
}

size_t ri_token_attend_workspace(const ri_token_cache* cache, int32_t prefix_len) {
  if (check_cache(cache, "token cache") != RI_OK) return 0;
  if (prefix_len < 0 || prefix_len > 1 << 28) {
    set_error("prefix length must be in [0, 2^28] (got %d)", prefix_len);
    return 0;
  }
  const size_t n = token_attend_bytes(*cache, prefix_len);
  if (n == 0) set_error("prefix of %d tokens: too much work for one call", prefix_len);
  return n;
}

ri_status ri_token_attend(const ri_token_cache* cache, const void* q,
                          const ri_token_prefix* prefix, void* out, float* lse,
                          int32_t add_weight, void* workspace, size_t workspace_bytes,
                          ri_stream_t stream) {
  return token_attend(cache, q, prefix, out, lse, add_weight, workspace, workspace_bytes, 0,
                      kWaitLimitNsHost, stream);
}

ri_status ri_selftest_token_attend_timeout(const ri_token_cache* cache, const void* q,
                                           const ri_token_prefix* prefix, void* out, float* lse,
                                           int32_t add_weight, void* workspace,
                                           size_t workspace_bytes, int32_t hand_off,
                                           uint64_t limit_ns, ri_stream_t stream) {
  RI_CHECK(prefix && prefix->length > 0, RI_ERR_INVALID_ARG, "the self-test needs a prefix");
  RI_CHECK(hand_off == RI_TOKEN_WAIT_TILE || hand_off == RI_TOKEN_WAIT_SCORES, RI_ERR_INVALID_ARG,
           "hand_off must be 1 or 2 (got %d)", hand_off);
  RI_CHECK(limit_ns > 0 && limit_ns <= 10ull * 1000000000ull, RI_ERR_INVALID_ARG,
           "limit_ns must be in (0, 10 s]");
  return token_attend(cache, q, prefix, out, lse, add_weight, workspace, workspace_bytes, hand_off,
                      limit_ns, stream);
}

size_t ri_token_evict_workspace(const ri_token_cache* cache, int32_t budget) {
  if (check_cache(cache, "token cache") != RI_OK) return 0;
  if (budget < 1) {
    set_error("budget must be >= 1 (got %d)", budget);
    return 0;
  }
  if (cache->capacity > kEvictMaxCapacity) {
    set_error("eviction handles capacities up to %d (got %d)", kEvictMaxCapacity,
              cache->capacity);
    return 0;
  }
  return token_evict_bytes(*cache, budget);
}

ri_status ri_token_evict(const ri_token_cache* cache, int32_t budget, int32_t keep_first,
                         int32_t keep_recent, const ri_token_cache* out, void* workspace,
                         size_t workspace_bytes, ri_stream_t stream) {
  ri_status st = check_arrays(cache, "token cache");
  if (st != RI_OK) return st;
  if ((st = check_arrays(out, "out cache")) != RI_OK) return st;
  RI_CHECK(budget >= 1 && keep_first >= 0 && keep_recent >= 0 &&
               (long long)keep_first + keep_recent <= budget,
           RI_ERR_INVALID_ARG,
           "budget must be >= 1 and hold keep_first + keep_recent (got %d, %d, %d)", budget,
           keep_first, keep_recent);
  RI_CHECK(out->batch == cache->batch && out->num_kv_heads == cache->num_kv_heads,
           RI_ERR_INVALID_ARG, "the caches must have equal batch and head counts");
  const int W = budget < cache->capacity ? budget : cache->capacity;
  RI_CHECK(out->capacity >= W, RI_ERR_CAPACITY, "out holds %d tokens, %d needed", out->capacity,
           W);
  RI_CHECK(cache->capacity <= kEvictMaxCapacity, RI_ERR_UNSUPPORTED,
           "eviction handles capacities up to %d (got %d)", kEvictMaxCapacity, cache->capacity);
  const size_t units = (size_t)cache->batch * cache->num_kv_heads;
  const size_t n = units * cache->capacity, m = units * out->capacity;
  const struct { const void *a, *b; size_t size; const char* name; } pairs[] = {
      {cache->K, out->K, 256, "K"}, {cache->V, out->V, 256, "V"}, {cache->pos, out->pos, 4, "pos"},
      {cache->weight, out->weight, 4, "weight"}};
  for (const auto& x : pairs)
    for (const auto& y : pairs)
      RI_CHECK((&x == &y || x.a != y.b) && same_or_apart(x.a, n * x.size, y.b, m * y.size),
               RI_ERR_INVALID_ARG,
               "out's %s must be the cache's own %s (equal capacity) or not overlap its %s",
               y.name, y.name, x.name);
  RI_CHECK(same_or_apart(cache->lens, units * 4, out->lens, units * 4), RI_ERR_INVALID_ARG,
           "out's lens must be the cache's own or not overlap it");
  if ((st = check_workspace(workspace, workspace_bytes, token_evict_bytes(*cache, budget))) !=
      RI_OK)
    return st;
  TokenEvictArgs a = {*cache, *out, budget, keep_first, keep_recent,
                      static_cast<char*>(workspace)};
  const cudaError_t e = launch_token_evict(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RI_OK : cuda_fail(e, "token evict launch");
}

}  // extern "C"
