// Shared by the group norm's kernels (ctcpb_gnorm.cu, ctcpb_gnorm_split.cu).
#pragma once

#include "ctcpb_head.cuh"

namespace ctcpb {

constexpr int kGnThreads = 384;  // of a block at most (with two blocks an SM: 85 registers, three of 256 threads)

// What a launch works on.  A block takes a slab: some whole groups' channels, or
// (pieces > 1) a piece of one group's, of one utterance at a time.
struct GnArgs {
  const void *x, *dy;
  void* y;  // or dx
  long long x_b, x_t, dy_b, dy_t, y_b, y_t;
  const void *weight, *bias;
  int ptype;
  const int* lengths;
  int B, T, C, G, D;
  float eps;
  int act;
  float *mean, *rstd;
  float* cols;   // column sums [by * parts][2][C] (null: not wanted)
  float* group;  // split: groups' sums of the parts of an utterance's frames [B][parts][G * pieces]
  // geometry
  int gs;      // groups of a slab
  int pieces;  // slabs of a group
  int tw;      // vectors of a slab's row
  int rs;      // rows that a block takes at once
  int slots;   // rows of a thread that shared memory holds
  int parts;   // blocks that share an utterance's frames (ranks of a cluster, or chunks)
  int cr;      // partial column sums of a block
  int pvec;    // the parameters' vectors of V start at multiples of their size
  u32 by_tw, by_rs, by_dv;  // divisors' reciprocals (quot)
};
// x / d by the reciprocal ceil(2^32 / d) (0: d is 1): exact for x d < 2^32
__host__ __device__ __forceinline__ u32 reciprocal(u32 d) { return d > 1 ? (u32)(((1ull << 32) + d - 1) / d) : 0u; }
__device__ __forceinline__ int quot(int x, u32 rec) { return rec ? (int)__umulhi((u32)x, rec) : x; }

// ---------------------------------------------------------------- vectors

// V elements as one access, and as pairs (the second of a single one is 0).
template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
  typedef uint4 type;
};
template <>
struct Raw<8> {
  typedef uint2 type;
};
template <>
struct Raw<4> {
  typedef u32 type;
};
template <>
struct Raw<2> {
  typedef u16 type;
};
template <class T, int V>
struct Vec {
  static constexpr int bytes = V * (int)sizeof(T), P = (V + 1) / 2;
  typename Raw<bytes>::type q;
  __device__ __forceinline__ u32 word(int i) const {
    if constexpr (bytes == 16)
      return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
    else if constexpr (bytes == 8)
      return i == 0 ? q.x : q.y;
    else
      return (u32)q;
  }
  __device__ __forceinline__ void get(u64 (&v)[P]) const {
    if constexpr (V == 1 && sizeof(T) == 2) {
      v[0] = pair(Elem<T>::to(*reinterpret_cast<const T*>(&q)), 0.f);
    } else if constexpr (V == 1) {
      v[0] = pair(__uint_as_float(q), 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if constexpr (sizeof(T) == 4)
          v[i] = pair(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
        else
          v[i] = Elem<T>::unpack(word(i));
      }
    }
  }
  __device__ __forceinline__ void put(const u64 (&v)[P]) {
    if constexpr (V == 1) {
      float x, y;
      unpair(x, y, v[0]);
      const T e = Elem<T>::from(x);
      q = *reinterpret_cast<const decltype(q)*>(&e);
    } else {
      u32 w[4];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float x, y;
        unpair(x, y, v[i]);
        if constexpr (sizeof(T) == 4) {
          w[2 * i] = __float_as_uint(x);
          w[2 * i + 1] = __float_as_uint(y);
        } else {
          w[i] = Elem<T>::pack(x, y);
        }
      }
      if constexpr (bytes == 16)
        q = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (bytes == 8)
        q = make_uint2(w[0], w[1]);
      else
        q = w[0];
    }
  }
  __device__ __forceinline__ void zero() {
    if constexpr (bytes == 16)
      q = make_uint4(0, 0, 0, 0);
    else if constexpr (bytes == 8)
      q = make_uint2(0, 0);
    else
      q = 0;
  }
  __device__ __forceinline__ void load(const T* p) { q = *reinterpret_cast<const decltype(q)*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(q)*>(p) = q; }
  __device__ __forceinline__ void load_shared(u32 at) {
    if constexpr (bytes == 16)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                   : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                   : "r"(at)
                   : "memory");
    else if constexpr (bytes == 8)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(q.x), "=r"(q.y) : "r"(at) : "memory");
    else if constexpr (bytes == 4)
      asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(q) : "r"(at) : "memory");
    else
      asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(q) : "r"(at) : "memory");
  }
  __device__ __forceinline__ void store_shared(u32 at) const {
    if constexpr (bytes == 2) asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(at), "h"(q) : "memory");
  }
};
// n rows of a vector into shared memory, each `pitch` bytes on; they are there for
// this thread after cp_wait_all.  (There is no asynchronous copy of two bytes.)
template <class T, int V>
__device__ __forceinline__ void fetch_rows(u32 to, u32 pitch, const T* from, long long step, int n) {
  typedef Vec<T, V> W;
  if constexpr (W::bytes == 2) {
    for (int k = 0; k < n; k += 8) {
      W w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < n) w[i].load(from + i * step);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < n) w[i].store_shared(to + i * pitch);
      to += 8 * pitch;
      from += 8 * step;
    }
  } else {
#pragma unroll 4
    for (int k = 0; k < n; ++k, to += pitch, from += step) {
      if constexpr (W::bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(to), "l"(from), "n"(W::bytes) : "memory");
    }
  }
}
// the sum of a vector's elements
template <int V>
__device__ __forceinline__ float lanes(const u64 (&v)[(V + 1) / 2]) {
  if constexpr (V == 1) {
    float x, y;
    unpair(x, y, v[0]);
    return x;
  } else {
    u64 s = v[0];
#pragma unroll
    for (int i = 1; i < V / 2; ++i) s = add2(s, v[i]);
    return pair_sum(s);
  }
}

// ---------------------------------------------------------------- statistics

// Count, mean and sum of squared distances from it; joined without a difference of
// large sums (Chan, Golub, LeVeque).
struct Moments {
  float n, mean, m2;
  __device__ __forceinline__ void join(const Moments& o) {
    const float tot = n + o.n, share = tot > 0.f ? __fdividef(o.n, tot) : 0.f, d = o.mean - mean;
    mean = fmaf(d, share, mean);
    m2 += fmaf(d * d, n * share, o.m2);
    n = tot;
  }
  __device__ __forceinline__ float rstd(float eps) const { return rsqrtf(m2 / n + eps); }
};
struct Two {
  float a, b;
  __device__ __forceinline__ void join(const Two& o) {
    a += o.a;
    b += o.b;
  }
};
template <class S>
__device__ __forceinline__ S shuffled(const S& s, int mask) {
  constexpr int n = sizeof(S) / 4;
  S r;
#pragma unroll
  for (int i = 0; i < n; ++i)
    reinterpret_cast<float*>(&r)[i] = __shfl_xor_sync(0xffffffffu, reinterpret_cast<const float*>(&s)[i], mask);
  return r;
}
template <class S>
__device__ __forceinline__ void warp_join(S& s) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) s.join(shuffled(s, m));
}

// ---------------------------------------------------------------- places

__device__ __forceinline__ int frames_of(const GnArgs& a, int b) {
  if (!a.lengths) return a.T;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

struct Place {
  int part;            // of the utterance's frames
  int g0, groups;      // the slab's groups
  int piece;           // ... or which piece of its one group
  int c0, wv;          // its first channel, its vectors
  int cv, ty;          // the thread's vector, and its first row
  bool on;             // the thread has a vector
  template <int V>
  __device__ __forceinline__ void set(const GnArgs& a, int slab, int part_) {
    part = part_;
    if (a.pieces > 1) {
      const int dv = a.D / V;
      g0 = slab / a.pieces;
      piece = slab - g0 * a.pieces;
      groups = 1;
      c0 = g0 * a.D + piece * a.tw * V;
      wv = dv - piece * a.tw < a.tw ? dv - piece * a.tw : a.tw;
    } else {
      g0 = slab * a.gs;
      piece = 0;
      groups = a.G - g0 < a.gs ? a.G - g0 : a.gs;
      c0 = g0 * a.D;
      wv = groups == a.gs ? a.tw : groups * (a.D / V);
    }
    ty = quot(threadIdx.x, a.by_tw);
    cv = threadIdx.x - ty * a.tw;
    on = ty < a.rs && cv < wv;
  }
  // group of the thread's vector in the slab
  template <int V>
  __device__ __forceinline__ int group(const GnArgs& a) const {
    return a.pieces > 1 || !on ? 0 : quot(cv, a.by_dv);
  }
};
// The frames of a part: the thread's first, and how many it has.
struct Rows {
  int first, n;
  __device__ __forceinline__ Rows(const GnArgs& a, const Place& p, int len) {
    const int each = a.parts > 1 ? (len + a.parts - 1) / a.parts : len, from = p.part * each;
    const int left = (from + each < len ? each : len - from) - p.ty;
    first = from + p.ty;
    n = p.on && left > 0 ? quot(left + a.rs - 1, a.by_rs) : 0;
  }
};

// A thread's elements of a parameter (`none` without it).
template <int V>
__device__ __forceinline__ void param_of(u64 (&w)[(V + 1) / 2], const void* p, int type, bool vec, int c, bool on, float none) {
  constexpr int P = (V + 1) / 2;
#pragma unroll
  for (int i = 0; i < P; ++i) w[i] = pair(none, none);
  if (!p || !on) return;
  if (vec && V > 1) {
    if (type == CTCPB_F32) {
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = reinterpret_cast<const u64*>((const float*)p + c)[i];
    } else {
      u32 q[P];
#pragma unroll
      for (int i = 0; i < P; ++i) q[i] = reinterpret_cast<const u32*>((const u16*)p + c)[i];
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = type == CTCPB_BF16 ? Elem<__nv_bfloat16>::unpack(q[i]) : Elem<__half>::unpack(q[i]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    w[i] = pair(load_elem(p, type, c + 2 * i), 2 * i + 1 < V ? load_elem(p, type, c + 2 * i + 1) : none);
}
template <int V>
__device__ __forceinline__ void params_of(const GnArgs& a, int c, bool on, u64 (&w)[(V + 1) / 2], u64 (&b)[(V + 1) / 2]) {
  param_of<V>(w, a.weight, a.ptype, a.pvec, c, on, 1.f);
  param_of<V>(b, a.bias, a.ptype, a.pvec, c, on, 0.f);
}

// y is 0 in the frames behind the last (the parts take them in turn).
template <class T, int V>
__device__ __forceinline__ void zero_rows(const GnArgs& a, const Place& p, T* y, int len) {
  if (!p.on) return;
  Vec<T, V> z;
  z.zero();
  const int step = a.parts * a.rs;
  int r = len + p.part * a.rs + p.ty;
  T* to = y + r * a.y_t + p.cv * V;
  const long long y_step = step * a.y_t;
  for (; r < a.T; r += step, to += y_step) z.store(to);
}

// ---------------------------------------------------------------- the activation

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// h / (1 + e^-h)
__device__ __forceinline__ u64 silu2(u64 h) {
  float x, y;
  unpair(x, y, mul2(h, pair(-kLog2e, -kLog2e)));
  unpair(x, y, add2(pair(ex2(x), ex2(y)), pair(1.f, 1.f)));
  return mul2(h, pair(rcp(x), rcp(y)));
}
// Its slope s (1 + h (1 - s)), s = 1 / (1 + e^-h)
__device__ __forceinline__ u64 silu_slope2(u64 h) {
  float x, y;
  unpair(x, y, mul2(h, pair(-kLog2e, -kLog2e)));
  const u64 one = pair(1.f, 1.f);
  unpair(x, y, add2(pair(ex2(x), ex2(y)), one));
  const u64 s = pair(rcp(x), rcp(y));
  return mul2(s, fma2(h, fma2(s, pair(-1.f, -1.f), one), one));
}
__device__ __forceinline__ float relu(float x) { return x > 0.f ? x : x != x ? x : 0.f; }

// act((x - mean) w + b)
template <int P>
__device__ __forceinline__ void activate(u64 (&v)[P], u64 nm, const u64 (&w)[P], const u64 (&b)[P], int act) {
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = fma2(add2(v[i], nm), w[i], b[i]);
  if (act == CTCPB_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = silu2(v[i]);
  } else if (act == CTCPB_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float x, y;
      unpair(x, y, v[i]);
      v[i] = pair(relu(x), relu(y));
    }
  }
}
// x -> x - mean, dy -> dh (wr: the weight times rstd)
template <int P>
__device__ __forceinline__ void before(u64 (&x)[P], u64 (&d)[P], u64 nm, const u64 (&wr)[P], const u64 (&b)[P], int act) {
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = add2(x[i], nm);
  if (act == CTCPB_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < P; ++i) d[i] = mul2(d[i], silu_slope2(fma2(x[i], wr[i], b[i])));
  } else if (act == CTCPB_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float h, k, p, q;
      unpair(h, k, fma2(x[i], wr[i], b[i]));
      unpair(p, q, d[i]);
      d[i] = pair(h > 0.f ? p : 0.f, k > 0.f ? q : 0.f);
    }
  }
}
// A thread's sums of an utterance, of dh (x - mean) and dh, as the group's of dh w and
// dh w xh (the first times rstd, which dx has as a factor).
template <int V>
__device__ __forceinline__ Two thread_sums(const u64 (&sw)[(V + 1) / 2], const u64 (&sb)[(V + 1) / 2],
                                           const u64 (&wr)[(V + 1) / 2]) {
  constexpr int P = (V + 1) / 2;
  u64 a[P], b[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    a[i] = mul2(sb[i], wr[i]);
    b[i] = mul2(sw[i], wr[i]);
  }
  return Two{lanes<V>(a), lanes<V>(b)};
}
// dx = dh wr + (x - mean) m1 + m0, from the group's sums above: m0 = -rstd mean(dh w),
// m1 = -rstd^2 mean(dh w xh)
__device__ __forceinline__ void factors(const GnArgs& a, const Two& t, int len, float rstd, u64& m0, u64& m1) {
  const float inv = len > 0 ? __fdividef(1.f, (float)len * (float)a.D) : 0.f;
  const float c0 = -t.a * inv, c1 = -t.b * inv * rstd * rstd;
  m0 = pair(c0, c0);
  m1 = pair(c1, c1);
}

// ---------------------------------------------------------------- sums over a block

// The threads' `s` by group of the slab, a warp for each; lane 0 of it has the sum
// and calls done(group, sum).
template <class S, int V, class F>
__device__ __forceinline__ void by_group(const GnArgs& a, const Place& p, const S& s, S* each, F done) {
  each[threadIdx.x] = s;
  __syncthreads();
  const int dv = a.pieces > 1 ? p.wv : a.D / V, lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < p.groups; g += blockDim.x >> 5) {
    S t{};
    for (int e = lane; e < dv * a.rs; e += 32) {
      const int ty = a.pieces > 1 ? e / dv : quot(e, a.by_dv);
      t.join(each[ty * a.tw + g * dv + e - ty * dv]);
    }
    warp_join(t);
    if (lane == 0) done(g, t);
  }
}

// The threads' column sums of an utterance (of dh (x - mean), times rstd, and dh) into
// `red` [cr][2][tw * V]: a warp's threads of one column first, where its columns repeat.
// A thread's place there is its own.
template <int V>
__device__ __forceinline__ void add_columns(const GnArgs& a, const Place& p, u64 (&sw)[(V + 1) / 2], u64 (&sb)[(V + 1) / 2],
                                            float rstd, float* red, bool more) {
  constexpr int P = (V + 1) / 2;
  const int width = a.tw * V;
  const bool by_warp = a.cr < a.rs;
#pragma unroll
  for (int i = 0; i < P; ++i) sw[i] = mul2(sw[i], pair(rstd, rstd));
  if (by_warp)
    for (int m = a.tw; m < 32; m <<= 1) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        sw[i] = add2(sw[i], __shfl_xor_sync(0xffffffffu, sw[i], m));
        sb[i] = add2(sb[i], __shfl_xor_sync(0xffffffffu, sb[i], m));
      }
    }
  const int at = by_warp ? threadIdx.x >> 5 : p.ty;
  if (by_warp ? (int)(threadIdx.x & 31) < a.tw : p.ty < a.rs) {
    float* const o = red + 2 * at * width + p.cv * V;
    if constexpr (V == 1) {
      float x, y, none;
      unpair(x, none, sw[0]);
      unpair(y, none, sb[0]);
      o[0] = more ? o[0] + x : x;
      o[width] = more ? o[width] + y : y;
    } else {
      u64* const ow = reinterpret_cast<u64*>(o);
      u64* const ob = reinterpret_cast<u64*>(o + width);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        ow[i] = more ? add2(ow[i], sw[i]) : sw[i];
        ob[i] = more ? add2(ob[i], sb[i]) : sb[i];
      }
    }
  }
}
// ... and from there, after a barrier, into a.cols, in order.
template <int V>
__device__ __forceinline__ void column_sums(const GnArgs& a, const Place& p, const float* red, long long row) {
  const int width = a.tw * V;
  float* const to = a.cols + row * 2 * a.C + p.c0;
  for (int e = threadIdx.x; e < 2 * width; e += blockDim.x) {
    const int second = e >= width, c = e - second * width;
    if (c >= p.wv * V) continue;
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < a.cr; ++k) s += red[2 * k * width + e];
    to[second * (long long)a.C + c] = s;
  }
}

// ---------------------------------------------------------------- geometry

struct GnShape {
  int v;  // elements of an access
  int threads, gs, pieces, slabs, tw, rs, slots, parts, cr, by;
  bool split;   // two launches; else the slab stays in shared memory
  size_t smem;
};
cudaError_t gn_split(int type, bool bwd, GnArgs& a, const GnShape& s, cudaStream_t st);

template <class T, class F>
cudaError_t gn_each_vec(int v, F f) {
  if constexpr (sizeof(T) == 2) {
    if (v == 8) return f(Vec<T, 8>(), std::integral_constant<int, 8>());
  }
  if (v == 4) return f(Vec<T, 4>(), std::integral_constant<int, 4>());
  if (v == 2) return f(Vec<T, 2>(), std::integral_constant<int, 2>());
  return f(Vec<T, 1>(), std::integral_constant<int, 1>());
}

}  // namespace ctcpb
