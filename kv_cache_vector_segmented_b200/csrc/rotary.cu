// Rotary positions: the rotation of query and key heads, alone (ri_rotary)
// and fused with the append to the exact token cache (ri_token_append).
//
// Mathematics: pair (a, b) of a head at position p turns by p * f_i radians.
// A position far out (p * f of 10^6 radians) loses all its fraction in fp32,
// so the table holds f / 2 pi as a 64-bit fraction of a turn: the product
// with the position, modulo 2^64, IS the angle's fraction of a turn, exact to
// 2^-64 * p, in two integer multiplications.  Its top 32 bits as a signed
// number of half turns go to sincospif.  The rotation runs in fp32 and is
// rounded once to the tensor's type.
//
// What bounds it: memory (each element read and written once); the angle of a
// pair is computed once per thread and used for every head the thread takes.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void turn_angle(unsigned long long turns, int pos, float magnitude,
                                           float* c, float* s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
  // [-2^31, 2^31) of 2^-31 half turns; the cut bits are 2^-32 of a turn
  const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
  float sv, cv;
  sincospif(half_turns, &sv, &cv);
  *c = cv * magnitude;
  *s = sv * magnitude;
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f<__half>(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f<float>(float v) {
  return v;
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}

// VEC elements moved by one access (16 bytes, or one element).
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load(const T* p) {
  return *reinterpret_cast<const Pack<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const Pack<T, VEC>& v) {
  *reinterpret_cast<Pack<T, VEC>*>(p) = v;
}

// A head's accesses ("items"): rotated ones first, then copies of the rest.
// Half layout: item i turns elements [i VEC, +VEC) with those n further on.
// Interleaved: item i turns the pairs inside elements [i W, +W), W = VEC (at
// least a pair).
template <int VEC>
struct Items {
  int n, turned, count, inter;  // pairs, rotated items, all items, layout
  __host__ __device__ Items(int rotary_dim, int interleaved, int d) {
    n = rotary_dim / 2;
    inter = interleaved;
    const int w = VEC > 1 ? VEC : 2;
    turned = interleaved ? rotary_dim / w : n / VEC;
    count = turned + (d - rotary_dim) / VEC;
  }
};

template <int VEC>
__device__ __forceinline__ void item_angles(const ri_rope& rope, const Items<VEC>& it, int item,
                                            int pos, float sign, float (&c)[VEC], float (&s)[VEC]) {
  if (item >= it.turned) return;
  constexpr int kInter = VEC > 1 ? VEC / 2 : 1;
  if (it.inter) {
#pragma unroll
    for (int i = 0; i < kInter; ++i) {
      turn_angle(__ldg(reinterpret_cast<const unsigned long long*>(rope.turns) + item * kInter + i),
                 pos, rope.magnitude, &c[i], &s[i]);
      s[i] *= sign;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      turn_angle(__ldg(reinterpret_cast<const unsigned long long*>(rope.turns) + item * VEC + i),
                 pos, rope.magnitude, &c[i], &s[i]);
      s[i] *= sign;
    }
  }
}

// One item of one head: src -> dst (which may be the same row).
template <typename T, int VEC>
__device__ __forceinline__ void turn_item(const T* src, T* dst, const Items<VEC>& it, int item,
                                          const float (&c)[VEC], const float (&s)[VEC]) {
  if (item >= it.turned) {
    const int at = 2 * it.n + (item - it.turned) * VEC;
    store<T, VEC>(dst + at, load<T, VEC>(src + at));
    return;
  }
  if (it.inter) {
    constexpr int W = VEC > 1 ? VEC : 2;
    const int at = item * W;
    T x[W];
    if constexpr (VEC > 1) {
      const Pack<T, VEC> p = load<T, VEC>(src + at);
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = p.v[i];
    } else {
      x[0] = src[at];
      x[1] = src[at + 1];
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const float a = to_f(x[2 * i]), b = to_f(x[2 * i + 1]);
      x[2 * i] = from_f<T>(a * c[i] - b * s[i]);
      x[2 * i + 1] = from_f<T>(b * c[i] + a * s[i]);
    }
    if constexpr (VEC > 1) {
      Pack<T, VEC> p;
#pragma unroll
      for (int i = 0; i < W; ++i) p.v[i] = x[i];
      store<T, VEC>(dst + at, p);
    } else {
      dst[at] = x[0];
      dst[at + 1] = x[1];
    }
    return;
  }
  const int at = item * VEC;
  Pack<T, VEC> p = load<T, VEC>(src + at), r = load<T, VEC>(src + at + it.n);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float a = to_f(p.v[i]), b = to_f(r.v[i]);
    p.v[i] = from_f<T>(a * c[i] - b * s[i]);
    r.v[i] = from_f<T>(b * c[i] + a * s[i]);
  }
  store<T, VEC>(dst + at, p);
  store<T, VEC>(dst + at + it.n, r);
}

// One thread per (token, group of `per` heads, item), items fastest so that
// neighbouring threads share rows; the angles are computed once and used for
// all heads of the group.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(RotaryArgs a, int per, int groups, int copy_rest) {
  const Items<VEC> it(a.rope.rotary_dim, a.rope.interleaved, a.d);
  const int items = copy_rest ? it.count : it.turned;
  const long long total = (long long)a.B * a.T * groups * items;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kThreads) {
    const int item = (int)(i % items);
    long long r = i / items;
    const int g = (int)(r % groups);
    r /= groups;
    const int t = (int)(r % a.T);
    const int b = (int)(r / a.T);
    float c[VEC], s[VEC];
    item_angles<VEC>(a.rope, it, item, a.pos[b * a.pos_stride + t], a.inverse ? -1.f : 1.f, c, s);
    const T* x = static_cast<const T*>(a.x.data) + b * a.x.stride_b + t * a.x.stride_t;
    T* y = static_cast<T*>(a.out.data) + b * a.out.stride_b + t * a.out.stride_t;
    const int h1 = min(a.heads, (g + 1) * per);
#pragma unroll 4
    for (int h = g * per; h < h1; ++h)
      turn_item<T, VEC>(x + h * a.x.stride_h, y + h * a.out.stride_h, it, item, c, s);
  }
}

template <typename T, int VEC>
cudaError_t rotary_typed(const RotaryArgs& a, cudaStream_t s) {
  const Items<VEC> it(a.rope.rotary_dim, a.rope.interleaved, a.d);
  const bool in_place = a.x.data == a.out.data;
  const int items = in_place ? it.turned : it.count;
  const int per = a.heads < 8 ? a.heads : 8;
  const int groups = (a.heads + per - 1) / per;
  const long long total = (long long)a.B * a.T * groups * items;
  long long blocks = (total + kThreads - 1) / kThreads;
  if (blocks > (1 << 30)) blocks = 1 << 30;
  rotary_kernel<T, VEC><<<(unsigned)blocks, kThreads, 0, s>>>(a, per, groups, !in_place);
  return cudaGetLastError();
}

bool vec_ok(const ri_heads& x, int size) {
  return aligned16(x.data) && x.stride_b * size % 16 == 0 && x.stride_t * size % 16 == 0 &&
         x.stride_h * size % 16 == 0;
}

template <typename T>
cudaError_t rotary_of(const RotaryArgs& a, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int run = a.rope.interleaved ? a.rope.rotary_dim : a.rope.rotary_dim / 2;
  // whole 16-byte accesses where every row and both halves start on one
  if (run % V == 0 && a.d % V == 0 && a.rope.rotary_dim % V == 0 && vec_ok(a.x, sizeof(T)) &&
      vec_ok(a.out, sizeof(T)))
    return rotary_typed<T, V>(a, s);
  return rotary_typed<T, 1>(a, s);
}

// ------------------------------------------------------------------- append
// One warp per (sequence, token, KV head): its G query heads, its key and its
// value.  The rows of a warp are dealt to groups of lanes, one item per lane.
template <int VEC>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendTokensArgs a, int advance) {
  using T = __nv_bfloat16;
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int H = a.c.num_kv_heads, G = a.c.group_size;
  if (w >= (long long)a.c.batch * a.T * H) return;
  const int h = (int)(w % H);
  const int t = (int)(w / H % a.T);
  const int b = (int)(w / H / a.T);
  const long long unit = (long long)b * H + h;
  const int cap = a.c.capacity;
  int len = a.c.lens[unit];
  if (len < 0 || len > cap) {
    if (lane == 0 && t == 0) record_status(a.status, RI_ERR_INVALID_ARG);
    len = len < 0 ? 0 : cap;
  }
  const bool room = len + (long long)a.T <= cap;
  if (!room && lane == 0 && t == 0) record_status(a.status, RI_ERR_CAPACITY);
  __syncwarp();  // every lane has the length before lane 0 may replace it
  const int pos = a.pos[b * a.pos_stride + t];
  const int n = a.rope.turns ? a.rope.rotary_dim : 0;
  const Items<VEC> it(n, a.rope.interleaved, kHeadDim);
  const long long row = unit * cap + len + t;
  const int q_rows = a.q.data ? G : 0;
  const int rows = q_rows + (room ? 1 : 0);
  // lanes of a row: the items' count rounded up to a power of two, at most 32
  int lpr = 1;
  while (lpr < it.count && lpr < 32) lpr <<= 1;
  const int sub = lane / lpr, subs = 32 / lpr;
  for (int item = lane % lpr; item < it.count; item += lpr) {
    float c[VEC], s[VEC];
    item_angles<VEC>(a.rope, it, item, pos, 1.f, c, s);
    for (int r = sub; r < rows; r += subs) {
      const T* src;
      T* dst;
      if (r < q_rows) {
        src = static_cast<const T*>(a.q.data) + b * a.q.stride_b + t * a.q.stride_t +
              (long long)(h * G + r) * a.q.stride_h;
        dst = static_cast<T*>(a.q_out) + (((long long)b * a.T + t) * H * G + h * G + r) * kHeadDim;
      } else {
        src = static_cast<const T*>(a.k.data) + b * a.k.stride_b + t * a.k.stride_t +
              h * a.k.stride_h;
        dst = static_cast<T*>(a.c.K) + row * kHeadDim;
      }
      turn_item<T, VEC>(src, dst, it, item, c, s);
    }
  }
  if (room) {
    const T* src = static_cast<const T*>(a.v.data) + b * a.v.stride_b + t * a.v.stride_t +
                   h * a.v.stride_h;
    T* dst = static_cast<T*>(a.c.V) + row * kHeadDim;
    if (lane < 16) store<T, 8>(dst + lane * 8, load<T, 8>(src + lane * 8));
    if (lane == 16) a.c.pos[row] = pos;
    if (lane == 17) a.c.weight[row] = 0.f;
  }
  if (advance && t == 0 && lane == 0) a.lens_out[unit] = room ? len + a.T : len;
}

// Advances the lengths in place once every token of append_kernel is stored.
__global__ void advance_kernel(int32_t* lens, int units, int cap, int T) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= units) return;
  const int len = min(max(lens[u], 0), cap);
  lens[u] = len + (long long)T <= cap ? len + T : len;
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t s) {
  switch (dtype) {
    case RI_BF16: return rotary_of<__nv_bfloat16>(a, s);
    case RI_FP16: return rotary_of<__half>(a, s);
    default: return rotary_of<float>(a, s);
  }
}

cudaError_t launch_token_append(const AppendTokensArgs& a, cudaStream_t s) {
  const long long warps = (long long)a.c.batch * a.T * a.c.num_kv_heads;
  const unsigned blocks = (unsigned)((warps * 32 + kThreads - 1) / kThreads);
  // one token per unit: the warp that reads a length is the one that replaces
  // it; several: other warps may still read it, so a second launch advances it
  const bool later = a.lens_out == a.c.lens && a.T > 1;
  const int n = a.rope.turns ? a.rope.rotary_dim : 0;
  const int run = a.rope.interleaved ? n : n / 2;
  if (run % 8 == 0 && n % 8 == 0)
    append_kernel<8><<<blocks, kThreads, 0, s>>>(a, !later);
  else
    append_kernel<1><<<blocks, kThreads, 0, s>>>(a, !later);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !later) return e;
  const int units = a.c.batch * a.c.num_kv_heads;
  advance_kernel<<<(units + 255) / 256, 256, 0, s>>>(a.c.lens, units, a.c.capacity, a.T);
  return cudaGetLastError();
}

}  // namespace ri
