// Rotary positions: the rotation of query and key heads, alone (ri_rotary)
// and fused with the append to the exact token cache (ri_token_append).
//
// Mathematics: pair (a, b) of a head at position p turns by p * f_i radians.
// A position far out (p * f of 10^6 radians) loses all its fraction in fp32,
// so the table holds f / 2 pi as a 64-bit fraction of a turn: the product
// with the position, modulo 2^64, IS the angle's fraction of a turn, exact to
// 2^-64 * p, in two integer multiplications.  The rotation runs in fp32 and is
// rounded once to the tensor's type.
//
// What bounds it: memory (each element read and written once).
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace ri {

namespace {

constexpr int kThreads = 256;
// blocks a grid has per SM: three fit at 64 KB of ring each, the fourth evens
// out the end (128K tokens of 8 heads: 93 us against 99 us with three)
constexpr int kBlocksPerSm = 4;
constexpr int kBatch = 4;  // rows of copies a thread issues at a time, one batch ahead

// Cosine and sine of pos * turns / 2^64 turns, times magnitude.  The fraction's
// top two bits (after adding an eighth) are the quadrant, the rest an angle x
// of at most pi / 4: sin x = x + x^3 p(x^2), cos x = 1 - x^2 / 2 + x^4 q(x^2)
// with p, q interpolated at Chebyshev nodes (off by 8.1e-9 and 5.9e-10).  The
// fraction needs no range reduction, which a call for any angle begins with.
__device__ __forceinline__ void turn_angle(unsigned long long turns, int pos, float magnitude,
                                           float* c, float* s) {
  const uint32_t t = static_cast<uint32_t>(
      (static_cast<unsigned long long>(static_cast<long long>(pos)) * turns) >> 32);
  const uint32_t q = (t + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(t - (q << 30))) * 1.4629180792671596e-9f;
  const float u = x * x;
  const float sx = fmaf(
      x * u, fmaf(u, fmaf(u, -0.00019587890710681677f, 0.008332747966051102f), -0.166666641831398f),
      x);
  const float cx = fmaf(
      u * u, fmaf(u, fmaf(u, 2.454794230288826e-05f, -0.001388830249197781f), 0.0416666641831398f),
      fmaf(u, -0.5f, 1.f));
  const float sv = (q & 1) ? cx : sx, cv = (q & 1) ? sx : cx;
  *s = __uint_as_float(__float_as_uint(sv * magnitude) ^ ((q & 2) << 30));
  *c = __uint_as_float(__float_as_uint(cv * magnitude) ^ (((q + 1) & 2) << 30));
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

// ------------------------------------------------- words of 2 x 16 or 32 bits
// An access moves N = 4 words (16 bytes) or one; its V elements as floats and
// back.
template <int N>
struct alignas(4 * N) Words {
  uint32_t w[N];
};
template <typename T, int N>
__device__ __forceinline__ void unpack(const Words<N>& x, float (&f)[4 * N / sizeof(T)]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(x.w[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x.w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    } else {
      f[2 * i] = __uint_as_float(x.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(x.w[i] & 0xFFFF0000u);
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void pack(const float (&f)[4 * N / sizeof(T)], Words<N>* x) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 4) {
      x->w[i] = __float_as_uint(f[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      x->w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      x->w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}
template <int N>
__device__ __forceinline__ void copy_async(Words<N>* smem, const void* g) {
  if constexpr (N == 4) cp_async16(smem, g);
  else cp_async4(smem, g);
}

// The rows (heads) of a token, in the order the kernels take them, and where
// they come from and go to.  A row without a source is skipped.
template <typename T>
struct HeadRows {  // ri_rotary
  static constexpr bool kAdvances = false;
  RotaryArgs a;
  __host__ __device__ int count() const { return a.heads; }
  __device__ __forceinline__ bool turned(int) const { return true; }
  __device__ __forceinline__ const T* from(int b, int t, int r) const {
    return static_cast<const T*>(a.x.data) + b * a.x.stride_b + t * a.x.stride_t +
           r * a.x.stride_h;
  }
  __device__ __forceinline__ T* to(int b, int t, int r, bool) const {
    return static_cast<T*>(a.out.data) + b * a.out.stride_b + t * a.out.stride_t +
           r * a.out.stride_h;
  }
};
struct StepRows {  // ri_token_append: the query heads, the keys, the values
  using T = __nv_bfloat16;
  static constexpr bool kAdvances = true;
  AppendTokensArgs a;
  int nq;  // query heads
  // Who writes the lengths after the call: `apart` (into an array of their
  // own), the thread that stores a unit's first key; in place with one token
  // per sequence, that sequence's block at its end; else a second launch, as
  // other blocks may still read them.
  bool apart;
  __host__ __device__ bool at_end() const { return !apart && a.T == 1; }
  __device__ __forceinline__ void advance(int u) const {
    const int cap = a.c.capacity, len = min(max(a.c.lens[u], 0), cap);
    a.lens_out[u] = len + (long long)a.T <= cap ? len + a.T : len;
  }
  __host__ __device__ int count() const { return nq + 2 * a.c.num_kv_heads; }
  __device__ __forceinline__ bool turned(int r) const { return r < nq + a.c.num_kv_heads; }
  __device__ __forceinline__ const T* from(int b, int t, int r) const {
    const bool q = r < nq, k = r < nq + a.c.num_kv_heads;
    const ri_heads& x = q ? a.q : k ? a.k : a.v;
    const int h = q ? r : k ? r - nq : r - nq - a.c.num_kv_heads;
    return static_cast<const T*>(x.data) + b * x.stride_b + t * x.stride_t + h * x.stride_h;
  }
  // `first`: the thread that also writes the token's position and weight and
  // reports a length out of range or a full head
  __device__ __forceinline__ T* to(int b, int t, int r, bool first) const {
    const int H = a.c.num_kv_heads, cap = a.c.capacity;
    if (r < nq) return static_cast<T*>(a.q_out) + (((long long)b * a.T + t) * nq + r) * kHeadDim;
    const bool k = r < nq + H;
    const long long unit = (long long)b * H + (k ? r - nq : r - nq - H);
    const int len = a.c.lens[unit];
    const bool live = len >= 0 && len <= cap;
    const int at = live ? len : len < 0 ? 0 : cap;
    const bool room = at + (long long)a.T <= cap;
    if (k && first && t == 0) {
      if (!live) record_status(a.status, RI_ERR_INVALID_ARG);
      if (!room) record_status(a.status, RI_ERR_CAPACITY);
      if (apart) a.lens_out[unit] = room ? at + a.T : at;
    }
    if (!room) return nullptr;
    const long long row = unit * cap + at + t;
    if (k && first) {
      a.c.pos[row] = a.pos[b * a.pos_stride + t];
      a.c.weight[row] = 0.f;
    }
    return static_cast<T*>(k ? a.c.K : a.c.V) + row * kHeadDim;
  }
};

// A block's 256 threads: `lanes` accesses of V elements ("items") of a row, fastest, so that
// a row is one contiguous piece; then `row_slots` rows; then tokens.  Items:
//  half layout  item i turns elements [i V, +V) with those n further on;
//  interleaved  item i turns the pairs inside elements [i V, +V);
//  the rest of the head is copied, V elements per item.
struct Shape {
  int lanes, row_slots;  // powers of two
  int items, turned;     // items of a row, those that turn
  int blocks;
};

Shape shape_of(int turned, int items, long long tokens, int rows) {
  Shape s;
  s.turned = turned;
  s.items = items;
  s.lanes = 1;
  while (s.lanes < items) s.lanes *= 2;
  const int slots = kThreads / s.lanes;
  const int fill = kBlocksPerSm * num_sms();
  // one row slot (angles serve all rows of a token) unless the grid would not
  // fill the machine
  s.row_slots = 1;
  while (s.row_slots < slots && s.row_slots < rows && tokens / (slots / s.row_slots) < fill)
    s.row_slots *= 2;
  const int token_slots = slots / s.row_slots;
  const long long tiles = (tokens + token_slots - 1) / token_slots;
  s.blocks = (int)(tiles < fill ? tiles : fill);
  return s;
}

// Every thread walks its tokens and their rows through a ring of its own in
// shared memory, kBatch to 2 kBatch rows of asynchronous copies ahead: no
// registers hold loads in flight and no barrier holds up the warps.  A token's
// angles are computed once per thread, for all its rows.  Measured: 128K
// tokens of 8 heads 93-97 us (5.5-5.8 TB/s), one row of copies at a time 104 us,
// rows held in registers behind a block's shared table of angles 96-104 us.
template <typename T, int N, bool INTER, class Rows>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    rows_kernel(const __grid_constant__ Rows rows, const ri_rope rope,
                const int32_t* __restrict__ pos, long long pos_stride, int T_, unsigned tokens,
                float sign, const Shape sh) {
  constexpr int V = 4 * N / (int)sizeof(T);
  static_assert(!INTER || V > 1, "an access holds whole pairs");
  constexpr int kRaws = INTER ? 1 : 2, kPairs = INTER ? V / 2 : V;
  extern __shared__ uint4 ring_[];  // [2 kBatch][kRaws][kThreads] accesses
  auto ring = [&](int stage, int raw) -> Words<N>& {
    return reinterpret_cast<Words<N>*>(ring_)[(stage * kRaws + raw) * kThreads + threadIdx.x];
  };
  const int lane = threadIdx.x & (sh.lanes - 1), slot = threadIdx.x / sh.lanes;
  const int token_slots = kThreads / sh.lanes / sh.row_slots;
  const unsigned tile0 = blockIdx.x * token_slots;
  const unsigned k_step = gridDim.x * token_slots;
  const int r0 = slot & (sh.row_slots - 1), n_rows = rows.count();
  // (a thread without an item or a row has no tokens)
  const unsigned k0 =
      lane < sh.items && r0 < n_rows ? tile0 + slot / sh.row_slots : tokens;
  const bool turns = lane < sh.turned;
  const int n = rope.rotary_dim / 2;
  const int at = turns ? lane * V : 2 * n + (lane - sh.turned) * V;

  // the row after next ones to copy: token ki (sequence bi, token ti), row ri
  unsigned ki = k0;
  int bi = ki / T_, ti = ki - bi * T_, ri = r0;
  auto copy_batch = [&](int first) {  // into slots first .. first + kBatch - 1
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (ki < tokens) {
        const T* src = rows.from(bi, ti, ri) + at;
        copy_async(&ring(first + j, 0), src);
        if (kRaws == 2 && turns) copy_async(&ring(first + j, kRaws - 1), src + n);
        ri += sh.row_slots;
        if (ri >= n_rows) {
          ri = r0;
          ki += k_step;
          if (ki < tokens) {
            bi = ki / T_;
            ti = ki - bi * T_;
          }
        }
      }
    cp_async_commit();
  };
  copy_batch(0);
  int stage = 0;  // row in use, modulo 2 kBatch
  unsigned long long turn_of[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    turn_of[i] = turns ? __ldg(reinterpret_cast<const unsigned long long*>(rope.turns) +
                               (INTER ? at / 2 : at) + i)
                       : 0ull;
  for (unsigned k = k0; k < tokens; k += k_step) {
    const int b = k / T_, t = k - b * T_;
    const int p = turns ? pos[b * pos_stride + t] : 0;
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      turn_angle(turn_of[i], p, rope.magnitude, &c[i], &s[i]);
      s[i] *= sign;
    }
#pragma unroll 1
    for (int r = r0; r < n_rows; r += sh.row_slots) {
      if (stage % kBatch == 0) {
        copy_batch(stage ^ kBatch);
        cp_async_wait<1>();
      }
      T* dst = rows.to(b, t, r, lane == 0);
      Words<N> x = ring(stage, 0);
      if (!turns) {
        if (dst) *reinterpret_cast<Words<N>*>(dst + at) = x;
      } else if constexpr (INTER) {
        if (rows.turned(r)) {
          float f[V];
          unpack<T>(x, f);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const float u = f[2 * i], v = f[2 * i + 1];
            f[2 * i] = u * c[i] - v * s[i];
            f[2 * i + 1] = v * c[i] + u * s[i];
          }
          pack<T>(f, &x);
        }
        if (dst) *reinterpret_cast<Words<N>*>(dst + at) = x;
      } else {
        Words<N> y = ring(stage, kRaws - 1);
        if (rows.turned(r)) {
          float u[V], v[V];
          unpack<T>(x, u);
          unpack<T>(y, v);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float w = u[i];
            u[i] = w * c[i] - v[i] * s[i];
            v[i] = v[i] * c[i] + w * s[i];
          }
          pack<T>(u, &x);
          pack<T>(v, &y);
        }
        if (dst) {
          *reinterpret_cast<Words<N>*>(dst + at) = x;
          *reinterpret_cast<Words<N>*>(dst + at + n) = y;
        }
      }
      stage = (stage + 1) % (2 * kBatch);
    }
  }
  cp_async_wait<0>();
  if constexpr (Rows::kAdvances) {
    if (rows.at_end()) {  // one token per sequence: token k is sequence k
      __syncthreads();
      const int H = rows.a.c.num_kv_heads;
      for (unsigned k = tile0; k < tokens; k += k_step)
        for (int i = threadIdx.x; i < token_slots * H; i += kThreads)
          if (k + i / H < tokens) rows.advance((int)(k * H + i));
    }
  }
}

// ------------------------------------------------ any strides and alignment
// One thread per element or pair: 16-bit heads whose rows or halves do not
// start on a word, interleaved fp32 ones that do not start on 16 bytes.  (15K
// tokens of 28 bf16 heads, 64 of 128 elements turned: 189 us here, 1.1 TB/s; 99 us
// a word at a time, 51 us 16 bytes at a time.)
template <typename T, class Rows>
__global__ void __launch_bounds__(kThreads)
    rows_any_kernel(const __grid_constant__ Rows rows, const ri_rope rope,
                    const int32_t* __restrict__ pos, long long pos_stride, int T_,
                    unsigned tokens, float sign, int d, int items) {
  const int n = rope.rotary_dim / 2, n_rows = rows.count();
  for (unsigned k = blockIdx.x; k < tokens; k += gridDim.x) {
    const int b = k / T_, t = k - b * T_;
    for (int i = threadIdx.x; i < items * n_rows; i += kThreads) {
      const int r = i / items, item = i - r * items;  // pairs first, then the rest of the head
      const T* src = rows.from(b, t, r);
      T* dst = rows.to(b, t, r, item == 0);
      if (!dst) continue;
      if (item >= n || !rows.turned(r)) {
        if (item >= n) {
          dst[n + item] = src[n + item];
        } else {
          const int ia = rope.interleaved ? 2 * item : item;
          const int ib = rope.interleaved ? ia + 1 : item + n;
          const T u = src[ia], v = src[ib];
          dst[ia] = u;
          dst[ib] = v;
        }
        continue;
      }
      float c, s;
      turn_angle(__ldg(reinterpret_cast<const unsigned long long*>(rope.turns) + item),
                 pos[b * pos_stride + t], rope.magnitude, &c, &s);
      s *= sign;
      const int ia = rope.interleaved ? 2 * item : item;
      const int ib = rope.interleaved ? ia + 1 : item + n;
      const float u = to_f(src[ia]), v = to_f(src[ib]);
      dst[ia] = from_f<T>(u * c - v * s);
      dst[ib] = from_f<T>(v * c + u * s);
    }
    if constexpr (Rows::kAdvances) {
      if (rows.at_end()) {
        __syncthreads();
        for (int h = threadIdx.x; h < rows.a.c.num_kv_heads; h += kThreads)
          rows.advance((int)(k * rows.a.c.num_kv_heads + h));
      }
    }
  }
}

// The widest access, in bytes, that every row, the second half's start and the
// rest's start allow: 16, 4, or less (0).
int width_of(const ri_rope& rope, int d, int size, const ri_heads* heads, int count) {
  unsigned long long bits = (unsigned)(rope.interleaved ? rope.rotary_dim : rope.rotary_dim / 2) *
                            size;
  bits |= (unsigned)(rope.rotary_dim * size) | (unsigned)(d * size);
  for (int i = 0; i < count; ++i)
    bits |= reinterpret_cast<uintptr_t>(heads[i].data) | (heads[i].stride_b * size) |
            (heads[i].stride_t * size) | (heads[i].stride_h * size);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 0;
}

struct RowsCall {
  ri_rope rope;
  const int32_t* pos;
  long long pos_stride;
  int T, B, d;
  bool inverse;
  bool rest;  // the elements behind the turned ones are copied too
  int slot;   // of the 16-byte kernel in set_smem_once's table
};

template <typename T, int N, bool INTER, class Rows>
cudaError_t launch_words(const Rows& rows, const RowsCall& c, cudaStream_t st) {
  constexpr int V = 4 * N / (int)sizeof(T);
  const int rd = c.rope.rotary_dim;
  const int turned = INTER ? rd / V : rd / 2 / V;
  const int items = turned + (c.rest ? (c.d - rd) / V : 0);
  const unsigned tokens = (unsigned)c.B * c.T;  // below 2^31 (checked by the calls)
  const Shape sh = shape_of(turned, items, tokens, rows.count());
  constexpr size_t ring = 2 * kBatch * (INTER ? 1 : 2) * kThreads * sizeof(Words<N>);
  auto kernel = rows_kernel<T, N, INTER, Rows>;
  if (ring > 48 << 10) {
    const cudaError_t e = set_smem_once(c.slot, reinterpret_cast<const void*>(kernel), (int)ring);
    if (e != cudaSuccess) return e;
  }
  kernel<<<sh.blocks, kThreads, ring, st>>>(rows, c.rope, c.pos, c.pos_stride, c.T, tokens,
                                            c.inverse ? -1.f : 1.f, sh);
  return cudaGetLastError();
}

template <typename T, class Rows>
cudaError_t launch_rows(const Rows& rows, const RowsCall& c, int width, cudaStream_t st) {
  const bool inter = c.rope.interleaved;
  if (width == 16)
    return inter ? launch_words<T, 4, true>(rows, c, st) : launch_words<T, 4, false>(rows, c, st);
  if (width == 4 && !inter) return launch_words<T, 1, false>(rows, c, st);
  if constexpr (sizeof(T) == 2)  // (a word of fp32 holds no pair)
    if (width == 4) return launch_words<T, 1, true>(rows, c, st);
  const unsigned tokens = (unsigned)c.B * c.T, fill = 8u * num_sms();
  const int rd = c.rope.rotary_dim, items = rd / 2 + (c.rest ? c.d - rd : 0);
  rows_any_kernel<T, Rows><<<tokens < fill ? tokens : fill, kThreads, 0, st>>>(
      rows, c.rope, c.pos, c.pos_stride, c.T, tokens, c.inverse ? -1.f : 1.f, c.d, items);
  return cudaGetLastError();
}

template <typename T>
cudaError_t rotary_of(const RotaryArgs& a, int slot, cudaStream_t s) {
  const ri_heads both[2] = {a.x, a.out};
  // in place the rest of the head stays where it is
  const RowsCall c{a.rope, a.pos, a.pos_stride, a.T, a.B, a.d, a.inverse, a.x.data != a.out.data,
                   slot};
  return launch_rows<T>(HeadRows<T>{a}, c, width_of(a.rope, a.d, sizeof(T), both, 2), s);
}

// The lengths after the call, once every token of it is stored.
__global__ void advance_kernel(const StepRows rows, int units) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u < units) rows.advance(u);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t s) {
  switch (dtype) {
    case RI_BF16: return rotary_of<__nv_bfloat16>(a, 8, s);
    case RI_FP16: return rotary_of<__half>(a, 9, s);
    default: return rotary_of<float>(a, 10, s);
  }
}

cudaError_t launch_token_append(const AppendTokensArgs& a, cudaStream_t s) {
  ri_rope rope = a.rope;
  if (!rope.turns) rope = ri_rope{nullptr, 0, 0, 1.f};  // nothing turns, all is copied
  const int H = a.c.num_kv_heads;
  const StepRows rows{a, a.q.data ? H * a.c.group_size : 0, a.lens_out != a.c.lens};
  const ri_heads given[3] = {a.k, a.v, a.q.data ? a.q : a.k};
  const RowsCall c{rope, a.pos, a.pos_stride, a.T, a.c.batch, kHeadDim, false, true, 11};
  const cudaError_t e =
      launch_rows<__nv_bfloat16>(rows, c, width_of(rope, kHeadDim, 2, given, 3), s);
  if (e != cudaSuccess || rows.apart || rows.at_end()) return e;
  const int units = a.c.batch * H;
  advance_kernel<<<(units + 255) / 256, 256, 0, s>>>(rows, units);
  return cudaGetLastError();
}

}  // namespace ri
