// Attention of one token per sequence over a shared prefix and the sequence's
// own cached tokens (ri_token_attend).
//
// Split softmax: every block takes a share of one (sequence, KV head)'s
// tokens (prefix first, then own) and leaves (maximum, sum, weighted value
// sum) per query head; a second launch merges the shares by log-sum-exp,
// writes out and lse, and adds the own tokens' probabilities to their
// weights from the scores kept by the first.
#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr float kScale = 0.08838834764831845f;  // 1 / sqrt(128)

struct AttendLayout {
  int splits;
  size_t off_ml, off_num, off_score, total;
};

AttendLayout layout(const ri_token_cache& c, int prefix_len) {
  AttendLayout L;
  const size_t units = (size_t)c.batch * c.num_kv_heads;
  const long long tokens = (long long)prefix_len + c.capacity;
  long long splits = (1184 + units - 1) / units;
  if (splits > (tokens + 63) / 64) splits = (tokens + 63) / 64;
  if (splits < 1) splits = 1;
  L.splits = (int)splits;
  size_t off = kStatusBytesHost;
  L.off_ml = off;
  off = align_up(off + units * splits * c.group_size * 2 * sizeof(float), 256);
  L.off_num = off;
  off = align_up(off + units * splits * c.group_size * kHeadDim * sizeof(float), 256);
  L.off_score = off;
  off = align_up(off + units * c.capacity * c.group_size * sizeof(float), 256);
  L.total = off;
  return L;
}

struct AttendParams {
  ri_token_cache c;
  ri_token_prefix p;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  float* ml;     // [units][splits][G][2]
  float* num;    // [units][splits][G][128]
  float* score;  // [units][capacity][G]
  int* status;
  int splits, add_weight;
};

__device__ __forceinline__ int live_len(const ri_token_cache& c, int unit, int* status) {
  int len = c.lens[unit];
  if (len < 0 || len > c.capacity) {
    record_status(status, RI_ERR_INVALID_ARG);
    len = len < 0 ? 0 : c.capacity;
  }
  return len;
}

__global__ void __launch_bounds__(kThreads) attend_kernel(AttendParams p) {
  __shared__ float sh_m[kWarps][kMaxGroup], sh_l[kWarps][kMaxGroup];
  __shared__ float sh_o[kWarps][kMaxGroup][kHeadDim];
  const int unit = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int G = p.c.group_size, H = p.c.num_kv_heads;
  const int b = unit / H, h = unit % H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = live_len(p.c, unit, p.status);
  const int P = p.p.length;
  const long long n = (long long)P + len;
  const long long i0 = n * split / p.splits, i1 = n * (split + 1) / p.splits;
  float q[kMaxGroup][4], o[kMaxGroup][4], m[kMaxGroup], l[kMaxGroup];
  for (int g = 0; g < kMaxGroup; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    for (int e = 0; e < 4; ++e) {
      o[g][e] = 0.f;
      q[g][e] = g < G ? __bfloat162float(p.q[((size_t)b * H * G + h * G + g) * kHeadDim + lane * 4 + e])
                      : 0.f;
    }
  }
  for (long long i = i0 + warp; i < i1; i += kWarps) {
    const __nv_bfloat16 *k, *v;
    if (i < P) {
      k = static_cast<const __nv_bfloat16*>(p.p.K) + h * p.p.stride_h + i * p.p.stride_t;
      v = static_cast<const __nv_bfloat16*>(p.p.V) + h * p.p.stride_h + i * p.p.stride_t;
    } else {
      const size_t row = (size_t)unit * p.c.capacity + (i - P);
      k = static_cast<const __nv_bfloat16*>(p.c.K) + row * kHeadDim;
      v = static_cast<const __nv_bfloat16*>(p.c.V) + row * kHeadDim;
    }
    float kf[4], vf[4];
    for (int e = 0; e < 4; ++e) {
      kf[e] = __bfloat162float(k[lane * 4 + e]);
      vf[e] = __bfloat162float(v[lane * 4 + e]);
    }
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
      if (g >= G) break;
      float s = 0.f;
      for (int e = 0; e < 4; ++e) s += q[g][e] * kf[e];
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
      s *= kScale;
      if (i >= P && lane == 0)
        p.score[((size_t)unit * p.c.capacity + (i - P)) * G + g] = s;
      const float mn = fmaxf(m[g], s);
      const float a = __expf(m[g] - mn), w = __expf(s - mn);
      m[g] = mn;
      l[g] = l[g] * a + w;
      for (int e = 0; e < 4; ++e) o[g][e] = o[g][e] * a + w * vf[e];
    }
  }
  for (int g = 0; g < G; ++g) {
    if (lane == 0) {
      sh_m[warp][g] = m[g];
      sh_l[warp][g] = l[g];
    }
    for (int e = 0; e < 4; ++e) sh_o[warp][g][lane * 4 + e] = o[g][e];
  }
  __syncthreads();
  for (int g = 0; g < G; ++g) {
    float mx = -INFINITY, sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh_m[w][g]);
    if (mx > -INFINITY)
      for (int w = 0; w < kWarps; ++w) {
        const float f = __expf(sh_m[w][g] - mx);
        sum += f * sh_l[w][g];
        acc += f * sh_o[w][g][threadIdx.x];
      }
    const size_t at = ((size_t)unit * p.splits + split) * G + g;
    p.num[at * kHeadDim + threadIdx.x] = acc;
    if (threadIdx.x == 0) {
      p.ml[at * 2] = mx;
      p.ml[at * 2 + 1] = sum;
    }
  }
}

__global__ void __launch_bounds__(kThreads) merge_kernel(AttendParams p, int chunks) {
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int G = p.c.group_size, H = p.c.num_kv_heads;
  const int b = unit / H, h = unit % H;
  const int len = live_len(p.c, unit, p.status);
  float lse[kMaxGroup];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    if (g >= G) break;
    float m = -INFINITY, l = 0.f;
    for (int s = 0; s < p.splits; ++s)
      m = fmaxf(m, p.ml[(((size_t)unit * p.splits + s) * G + g) * 2]);
    if (m > -INFINITY)
      for (int s = 0; s < p.splits; ++s) {
        const float* ml = p.ml + (((size_t)unit * p.splits + s) * G + g) * 2;
        l += __expf(ml[0] - m) * ml[1];
      }
    lse[g] = l > 0.f ? m + logf(l) : -INFINITY;
    if (chunk == 0) {
      float acc = 0.f;
      if (l > 0.f)
        for (int s = 0; s < p.splits; ++s) {
          const size_t at = ((size_t)unit * p.splits + s) * G + g;
          acc += __expf(p.ml[at * 2] - m) * p.num[at * kHeadDim + threadIdx.x];
        }
      const size_t row = (size_t)b * H * G + h * G + g;
      p.out[row * kHeadDim + threadIdx.x] = __float2bfloat16_rn(l > 0.f ? acc / l : 0.f);
      if (p.lse && threadIdx.x == 0) p.lse[row] = lse[g];
    }
  }
  if (!p.add_weight) return;
  for (int i = chunk * kThreads + threadIdx.x; i < len; i += chunks * kThreads) {
    const size_t row = (size_t)unit * p.c.capacity + i;
    float w = 0.f;
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g)
      if (g < G) w += __expf(p.score[row * G + g] - lse[g]);
    p.c.weight[row] += w;
  }
}

}  // namespace

size_t token_attend_bytes(const ri_token_cache& c, int prefix_len) {
  return layout(c, prefix_len).total;
}

cudaError_t launch_token_attend(const TokenAttendArgs& a, cudaStream_t s) {
  const AttendLayout L = layout(a.c, a.p.length);
  AttendParams p;
  p.c = a.c;
  p.p = a.p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.ml = reinterpret_cast<float*>(a.ws + L.off_ml);
  p.num = reinterpret_cast<float*>(a.ws + L.off_num);
  p.score = reinterpret_cast<float*>(a.ws + L.off_score);
  p.status = reinterpret_cast<int*>(a.ws);
  p.splits = L.splits;
  p.add_weight = a.add_weight;
  const int units = a.c.batch * a.c.num_kv_heads;
  attend_kernel<<<units * L.splits, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int chunks = a.add_weight ? (a.c.capacity + kThreads * 4 - 1) / (kThreads * 4) : 1;
  merge_kernel<<<units * chunks, kThreads, 0, s>>>(p, chunks);
  return cudaGetLastError();
}

}  // namespace ri
