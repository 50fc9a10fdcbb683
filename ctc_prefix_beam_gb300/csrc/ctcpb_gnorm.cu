// Group norm with an activation over channels-last frames, and its backward pass
// (ctcpb_group_norm, ctcpb_group_norm_backward).
//
//   xh = (x - mean) r,  h = xh w + b,  y = act(h),   r = 1 / sqrt(var + eps)
//   dh = dy act'(h),  t = dh w,  dx = r (t - mean(t) - xh mean(t xh))
//   dw = sum_{b,t} dh xh,  db = sum_{b,t} dh
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and writes
// dx.  A group's statistics need all of an utterance's frames before the first
// output, so a block takes a slab, some whole groups' channels of one utterance,
// and keeps it in shared memory between the two passes; where a slab is too long
// for a block, or there are too few of them, a cluster of blocks shares its frames
// and exchanges the statistics.  A thread copies into shared memory just what it
// will read itself.  What no cluster holds is read twice.
#include "ctcpb_head.cuh"

namespace ctcpb {
namespace {

constexpr int kGnThreads = 512;          // of a block at most
constexpr int kGnRanks = 8;              // blocks that share a slab at most
constexpr int kGnSmem = 200 * 1024;      // what a block keeps of a slab at most
constexpr int kGnSmemShare = 72 * 1024;  // ... and where more blocks can share it: three on an SM
constexpr int kGnPart = 4096;            // blocks of a backward launch that hold column sums
constexpr long long kGnPartSize = 1 << 22;  // ... and their columns

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
  float* part;  // [slots][2][C]
  // geometry
  int gs;      // groups of a slab
  int tw;      // vectors of a row that the block takes at once
  int tiles;   // ... and how often (more than once only where a slab is one group)
  int rs;      // rows that the block takes at once
  int slots;   // rows of a thread that shared memory holds
  int ranks;
};

// V elements as one access.
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
  static constexpr int bytes = V * (int)sizeof(T);
  typename Raw<bytes>::type q;
  __device__ __forceinline__ void get(float (&v)[V]) const {
    const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Elem<T>::to(e[i]);
  }
  __device__ __forceinline__ void put(const float (&v)[V]) {
    T* e = reinterpret_cast<T*>(&q);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = Elem<T>::from(v[i]);
  }
  __device__ __forceinline__ void load(const T* p) { q = *reinterpret_cast<const decltype(q)*>(p); }
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
  }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(q)*>(p) = q; }
};
template <int BYTES>
__device__ __forceinline__ void copy_async(u32 dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// Count, mean and sum of squared distances from it; joined without a difference of
// large sums (Chan, Golub, LeVeque).
struct Moments {
  float n, mean, m2;
  __device__ __forceinline__ void join(const Moments& o) {
    const float tot = n + o.n, share = tot > 0.f ? o.n / tot : 0.f, d = o.mean - mean;
    mean = fmaf(d, share, mean);
    m2 += fmaf(d * d, n * share, o.m2);
    n = tot;
  }
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

__device__ __forceinline__ int frames_of(const GnArgs& a, int b) {
  if (!a.lengths) return a.T;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// What a block works on.
struct Place {
  int slab, rank, groups, c0, wv;  // groups and vectors of this slab, its first channel
  int cv, ty;
  bool on;  // the thread has a vector
};
template <int V>
__device__ __forceinline__ Place place_of(const GnArgs& a) {
  Place p;
  p.slab = blockIdx.x / a.ranks;
  p.rank = blockIdx.x - p.slab * a.ranks;
  p.groups = a.G - p.slab * a.gs < a.gs ? a.G - p.slab * a.gs : a.gs;
  p.c0 = p.slab * a.gs * a.D;
  p.wv = p.groups * (a.D / V);
  p.ty = threadIdx.x / a.tw;
  p.cv = threadIdx.x - p.ty * a.tw;
  p.on = p.ty < a.rs;
  return p;
}

// The sums `s` of all threads by group (in `own`, [groups]), then over the blocks
// of the slab (in `all`).  A warp per group; blocks in order.
template <class S, int V>
__device__ __forceinline__ void group_sums(const GnArgs& a, const Place& p, const S& s, S* each, S* own, S* all) {
  each[threadIdx.x] = s;
  __syncthreads();
  const int dv = a.tiles > 1 ? a.tw : a.D / V, lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < p.groups; g += blockDim.x >> 5) {
    S t{};
    for (int e = lane; e < dv * a.rs; e += 32) {
      const int ty = e / dv;
      t.join(each[ty * a.tw + g * dv + e - ty * dv]);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) t.join(shuffled(t, m));
    if (lane == 0) (a.ranks > 1 ? own : all)[g] = t;
  }
  if (a.ranks > 1) {
    cluster_sync();
    constexpr int n = sizeof(S) / 4;
    for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
      S t{};
      for (int r = 0; r < a.ranks; ++r) {
        S o;
        const u32 at = cluster_addr(saddr(own + g), r);
#pragma unroll
        for (int i = 0; i < n; ++i)
          asm volatile("ld.shared::cluster.f32 %0, [%1];\n"
                       : "=f"(reinterpret_cast<float*>(&o)[i])
                       : "r"(at + 4 * i)
                       : "memory");
        t.join(o);
      }
      all[g] = t;
    }
    // every block has read before any writes `own` again or leaves
    asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
  }
  __syncthreads();
}
__device__ __forceinline__ void group_sums_done(const GnArgs& a) {
  if (a.ranks > 1) asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
}

// Rows of a rank: [first, end).
__device__ __forceinline__ void rows_of(const GnArgs& a, const Place& p, int len, long long& first, long long& end) {
  first = (u32)len * (u32)p.rank / (u32)a.ranks;  // len <= 2^24
  end = (u32)len * (u32)(p.rank + 1) / (u32)a.ranks;
}

__device__ __forceinline__ float sigmoid(float h) { return __fdividef(1.f, 1.f + ex2(-kLog2e * h)); }

template <class T, int V>
__device__ __forceinline__ void zero_rows(const GnArgs& a, const Place& p, T* yb, int len) {
  Vec<T, V> z;
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
  z.put(v);
  if (!p.on) return;
  for (int tile = 0; tile < a.tiles; ++tile) {
    const int at = tile * a.tw + p.cv;
    if (at >= p.wv) break;
    for (long long r = len + p.rank * a.rs + p.ty; r < a.T; r += a.ranks * a.rs) z.store(yb + r * a.y_t + at * V);
  }
}

template <int V>
__device__ __forceinline__ void params_of(const GnArgs& a, int c, float (&w)[V], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = a.weight ? load_elem(a.weight, a.ptype, c + i) : 1.f;
    b[i] = a.bias ? load_elem(a.bias, a.ptype, c + i) : 0.f;
  }
}

// RES: the slab stays in shared memory.
template <class T, int V, bool RES>
__global__ void __launch_bounds__(kGnThreads) k_gn(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int kRows = 4;
  Moments* const each = reinterpret_cast<Moments*>(smem);
  Moments* const own = each + blockDim.x;
  Moments* const all = own + a.gs;
  const u32 keep = (saddr(all + a.gs) + 15u & ~15u) + threadIdx.x * W::bytes;
  const u32 pitch = blockDim.x * W::bytes;
  pdl_wait();
  pdl_next();
  const Place p = place_of<V>(a);
  const int dv = a.D / V;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int len = frames_of(a, b);
    long long first, end;
    rows_of(a, p, len, first, end);
    const T* const xb = (const T*)a.x + (long long)b * a.x_b + p.c0;
    T* const yb = (T*)a.y + (long long)b * a.y_b + p.c0;
    first += p.ty;
    const int n = first < end ? ((int)(end - first) + a.rs - 1) / a.rs : 0;  // rows of this thread
    const long long x_step = a.rs * a.x_t, y_step = a.rs * a.y_t;
    // row k of the thread's vector `at` of a tile
    auto fetch = [&](W& v, int tile, int at, int k) {
      if constexpr (RES)
        v.load_shared(keep + (tile * a.slots + k) * pitch);
      else
        v.load(xb + first * a.x_t + at * V + k * x_step);
    };
    if constexpr (RES) {
      if (p.on)
        for (int tile = 0; tile < a.tiles; ++tile) {
          const int at = tile * a.tw + p.cv;
          u32 to = keep + tile * a.slots * pitch;
          const T* from = xb + first * a.x_t + at * V;
          if (at < p.wv)
            for (int k = 0; k < n; ++k, to += pitch, from += x_step) copy_async<W::bytes>(to, from);
        }
      cp_wait_all();
    }
    Moments m{0.f, 0.f, 0.f};
    if (p.on)
      for (int tile = 0; tile < a.tiles; ++tile) {
        const int at = tile * a.tw + p.cv;
        if (at >= p.wv) break;
        for (int k0 = 0; k0 < n; k0 += kRows) {
          W raw[kRows];
          float v[kRows][V];
          const int here = n - k0 < kRows ? n - k0 : kRows;
#pragma unroll
          for (int k = 0; k < kRows; ++k)
            if (k < here) fetch(raw[k], tile, at, k0 + k);
          float s = 0.f, q = 0.f;
#pragma unroll
          for (int k = 0; k < kRows; ++k)
            if (k < here) {
              raw[k].get(v[k]);
#pragma unroll
              for (int i = 0; i < V; ++i) s += v[k][i];
            }
          const float cnt = (float)(here * V), mean = s / cnt;
#pragma unroll
          for (int k = 0; k < kRows; ++k)
            if (k < here) {
#pragma unroll
              for (int i = 0; i < V; ++i) q = fmaf(v[k][i] - mean, v[k][i] - mean, q);
            }
          m.join(Moments{cnt, mean, q});
        }
      }
    group_sums<Moments, V>(a, p, m, each, own, all);
    if (a.mean && p.rank == 0)
      for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
        const long long o = (long long)b * a.G + p.slab * a.gs + g;
        a.mean[o] = all[g].mean;
        a.rstd[o] = len > 0 ? rsqrtf(all[g].m2 / all[g].n + a.eps) : 0.f;
      }
    if (p.on)
      for (int tile = 0; tile < a.tiles; ++tile) {
        const int at = tile * a.tw + p.cv;
        if (at >= p.wv) break;
        const Moments t = all[at / dv];
        const float rstd = rsqrtf(t.m2 / t.n + a.eps), mean = t.mean;
        float w[V], bias[V];
        params_of<V>(a, p.c0 + at * V, w, bias);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] *= rstd;
        T* to = yb + first * a.y_t + at * V;
#pragma unroll 4
        for (int k = 0; k < n; ++k, to += y_step) {
          W raw;
          float v[V];
          fetch(raw, tile, at, k);
          raw.get(v);
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = fmaf(v[i] - mean, w[i], bias[i]);
          if (a.act == CTCPB_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= sigmoid(v[i]);
          } else if (a.act == CTCPB_ACT_RELU) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = v[i] > 0.f ? v[i] : v[i] != v[i] ? v[i] : 0.f;
          }
          raw.put(v);
          raw.store(to);
        }
      }
    zero_rows<T, V>(a, p, yb, len);
    group_sums_done(a);
    __syncthreads();
  }
}

template <class T, int V, bool RES>
__global__ void __launch_bounds__(kGnThreads) k_gn_bwd(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  Two* const each = reinterpret_cast<Two*>(smem);
  Two* const own = each + blockDim.x;
  Two* const all = own + a.gs;
  const u32 keep = (saddr(all + a.gs) + 15u & ~15u) + threadIdx.x * W::bytes;
  const u32 pitch = blockDim.x * W::bytes, second = a.tiles * a.slots * pitch;  // dy lies behind x
  pdl_wait();
  pdl_next();
  const Place p = place_of<V>(a);
  const int dv = a.D / V;
  float* const part = a.part ? a.part + (long long)(blockIdx.y * a.ranks + p.rank) * 2 * a.C + p.c0 : nullptr;
  float tw[V], tb[V];  // column sums (one tile)
#pragma unroll
  for (int i = 0; i < V; ++i) tw[i] = tb[i] = 0.f;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int len = frames_of(a, b);
    long long first, end;
    rows_of(a, p, len, first, end);
    const T* const xb = (const T*)a.x + (long long)b * a.x_b + p.c0;
    const T* const db = (const T*)a.dy + (long long)b * a.dy_b + p.c0;
    T* const yb = (T*)a.y + (long long)b * a.y_b + p.c0;
    first += p.ty;
    const int n = first < end ? ((int)(end - first) + a.rs - 1) / a.rs : 0;
    const long long x_step = a.rs * a.x_t, d_step = a.rs * a.dy_t, y_step = a.rs * a.y_t;
    auto fetch = [&](float (&x)[V], float (&d)[V], int tile, int at, int k) {
      W v, u;
      if constexpr (RES) {
        const u32 from = keep + (tile * a.slots + k) * pitch;
        v.load_shared(from);
        u.load_shared(from + second);
      } else {
        v.load(xb + first * a.x_t + at * V + k * x_step);
        u.load(db + first * a.dy_t + at * V + k * d_step);
      }
      v.get(x);
      u.get(d);
    };
    if constexpr (RES) {
      if (p.on)
        for (int tile = 0; tile < a.tiles; ++tile) {
          const int at = tile * a.tw + p.cv;
          u32 to = keep + tile * a.slots * pitch;
          const T *px = xb + first * a.x_t + at * V, *pd = db + first * a.dy_t + at * V;
          if (at < p.wv)
            for (int k = 0; k < n; ++k, to += pitch, px += x_step, pd += d_step) {
              copy_async<W::bytes>(to, px);
              copy_async<W::bytes>(to + second, pd);
            }
        }
      cp_wait_all();
    }
    // xh into x, the gradient before the activation into d
    auto before = [&](float (&x)[V], float (&d)[V], const float (&w)[V], const float (&bias)[V], float mean, float rstd) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = (x[i] - mean) * rstd;
      if (a.act == CTCPB_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float h = fmaf(x[i], w[i], bias[i]), s = sigmoid(h);
          d[i] *= s * fmaf(h, 1.f - s, 1.f);
        }
      } else if (a.act == CTCPB_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = fmaf(x[i], w[i], bias[i]) > 0.f ? d[i] : 0.f;
      }
    };
    Two m{0.f, 0.f};
    if (p.on)
      for (int tile = 0; tile < a.tiles; ++tile) {
        const int at = tile * a.tw + p.cv;
        if (at >= p.wv) break;
        const long long o = (long long)b * a.G + p.slab * a.gs + at / dv;
        const float mean = a.mean[o], rstd = a.rstd[o];
        float w[V], bias[V], sw[V], sb[V];
        params_of<V>(a, p.c0 + at * V, w, bias);
#pragma unroll
        for (int i = 0; i < V; ++i) sw[i] = sb[i] = 0.f;
#pragma unroll 2
        for (int k = 0; k < n; ++k) {
          float x[V], d[V];
          fetch(x, d, tile, at, k);
          before(x, d, w, bias, mean, rstd);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            sw[i] = fmaf(d[i], x[i], sw[i]);
            sb[i] += d[i];
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          m.a = fmaf(sb[i], w[i], m.a);
          m.b = fmaf(sw[i], w[i], m.b);
          if (a.tiles == 1) {
            tw[i] += sw[i];
            tb[i] += sb[i];
          } else if (part) {  // the thread alone has these columns
            float* const q = part + at * V + i;
            const bool begun = b != (int)blockIdx.y;
            q[0] = begun ? q[0] + sw[i] : sw[i];
            q[a.C] = begun ? q[a.C] + sb[i] : sb[i];
          }
        }
      }
    if (a.y) {
      group_sums<Two, V>(a, p, m, each, own, all);
      const float inv = len > 0 ? 1.f / ((float)len * (float)a.D) : 0.f;
      if (p.on)
        for (int tile = 0; tile < a.tiles; ++tile) {
          const int at = tile * a.tw + p.cv;
          if (at >= p.wv) break;
          const long long o = (long long)b * a.G + p.slab * a.gs + at / dv;
          const float mean = a.mean[o], rstd = a.rstd[o];
          const Two t = all[at / dv];
          const float m0 = t.a * inv, m1 = t.b * inv;
          float w[V], bias[V];
          params_of<V>(a, p.c0 + at * V, w, bias);
          T* to = yb + first * a.y_t + at * V;
#pragma unroll 2
          for (int k = 0; k < n; ++k, to += y_step) {
            float x[V], d[V];
            fetch(x, d, tile, at, k);
            before(x, d, w, bias, mean, rstd);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = rstd * fmaf(-x[i], m1, fmaf(d[i], w[i], -m0));
            W out;
            out.put(d);
            out.store(to);
          }
        }
      zero_rows<T, V>(a, p, yb, len);
      group_sums_done(a);
      __syncthreads();
    }
  }
  if (!part || a.tiles > 1) return;
  // column sums over the threads that share them, in order (the slab's memory is free now)
  float* const cols = reinterpret_cast<float*>(smem);  // [rs][2][tw * V]
  const int width = a.tw * V;
  __syncthreads();
  if (p.on)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      cols[(2 * p.ty) * width + p.cv * V + i] = tw[i];
      cols[(2 * p.ty + 1) * width + p.cv * V + i] = tb[i];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * width; e += blockDim.x) {
    const int c = e < width ? e : e - width;
    if (c >= p.wv * V) continue;
    float s = 0.f;
    for (int k = 0; k < a.rs; ++k) s += cols[2 * k * width + e];
    part[(e < width ? 0 : a.C) + c] = s;
  }
}

// dw and db: the blocks' sums, in order (32 slices of them, then the slices).
__global__ void __launch_bounds__(1024) k_gn_cols(const float* __restrict__ part, int rows, int C, int ptype, void* dw,
                                                  void* db) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, each = (rows + 31) / 32;
  float s = 0.f;
  if (c < 2 * C) {
    const int first = warp * each, end = first + each < rows ? first + each : rows;
#pragma unroll 8
    for (int k = first; k < end; ++k) s += part[(long long)k * 2 * C + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  s = red[lane][warp];  // a warp per column
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  const int cc = blockIdx.x * 32 + warp;
  if (lane == 0 && cc < 2 * C) {
    if (cc < C) {
      if (dw) store_elem(dw, ptype, cc, s);
    } else if (db) {
      store_elem(db, ptype, cc - C, s);
    }
  }
}

struct GnShape {
  int v;  // elements of an access
  int threads, gs, tw, tiles, rs, slots, ranks, slabs, by;
  bool res;
  size_t smem;
};
// Elements of one access: a group's channels and every row start at its multiples.
int gn_vec(int type, int D, uintptr_t at, long long strides) {
  const int e = type == CTCPB_F32 ? 4 : 2;
  int v = 16 / e;
  while (v > 1 && (D % v != 0 || (at | (uintptr_t)(strides * e)) % (v * e) != 0)) v /= 2;
  return v;
}
int up32(long long n) { return (int)((n + 31) / 32 * 32); }

GnShape gn_shape(int type, int v, int B, int T, int C, int G, bool bwd) {
  GnShape s{};
  const int e = type == CTCPB_F32 ? 4 : 2, D = C / G, dv = D / v;
  s.v = v;
  // 128 bytes of a row, more where there are too few rows to fill a warp
  s.gs = 128 / (D * e) > 1 ? 128 / (D * e) : 1;
  while (s.gs < G && (long long)s.gs * dv * T < 32) s.gs *= 2;
  if (s.gs > G) s.gs = G;
  s.slabs = (G + s.gs - 1) / s.gs;
  const int wv = s.gs * dv;
  s.threads = wv > 256 ? up32(wv) : up32((long long)wv * T < 256 ? (long long)wv * T : 256);
  if (s.threads > kGnThreads) s.threads = kGnThreads;
  if (s.threads < 32) s.threads = 32;
  s.tw = wv < s.threads ? wv : s.threads;
  s.tiles = (wv + s.tw - 1) / s.tw;
  s.rs = s.threads / s.tw;
  const size_t stat = align_up((size_t)(s.threads + 2 * s.gs) * (bwd ? sizeof(Two) : sizeof(Moments)), 16);
  auto slab = [&](int ranks) {
    s.slots = ((T + ranks - 1) / ranks + s.rs - 1) / s.rs;
    return (size_t)s.slots * s.tiles * s.threads * v * e * (bwd ? 2 : 1);
  };
  s.ranks = 1;
  while (s.ranks < kGnRanks && T > 2 * s.ranks * s.rs &&
         (slab(s.ranks) > (size_t)kGnSmemShare || (long long)B * s.slabs * s.ranks < 304))
    s.ranks *= 2;
  s.smem = slab(s.ranks);
  s.res = v * e >= 4 && s.smem <= (size_t)kGnSmem;
  s.smem = stat + (s.res ? s.smem : 0);
  if (bwd && s.tiles == 1) {
    const size_t cols = (size_t)s.rs * 2 * s.tw * v * 4;
    if (s.smem < cols) s.smem = cols;
  }
  long long by = B;
  if (bwd) {  // column sums of so many blocks at most
    long long cap = kGnPart / ((long long)s.slabs * s.ranks), room = kGnPartSize / C / s.ranks;
    if (cap > room) cap = room;
    if (by > cap) by = cap > 1 ? cap : 1;
  }
  s.by = (int)(by < 65535 ? by : 65535);
  return s;
}

template <class T, int V>
cudaError_t gn_run(bool bwd, GnArgs& a, const GnShape& s, cudaStream_t st) {
  a.gs = s.gs;
  a.tw = s.tw;
  a.tiles = s.tiles;
  a.rs = s.rs;
  a.slots = s.slots;
  a.ranks = s.ranks;
  const dim3 grid(s.slabs * s.ranks, s.by);
  auto go = [&](auto kern, cudaError_t e) {
    return e != cudaSuccess ? e : launch(kern, grid, s.threads, s.smem, st, s.ranks, a);
  };
  if constexpr (V * sizeof(T) >= 4) {
    if (s.res) {
      constexpr auto f = k_gn<T, V, true>, g = k_gn_bwd<T, V, true>;
      return bwd ? go(g, smem_optin<g>(s.smem)) : go(f, smem_optin<f>(s.smem));
    }
  }
  constexpr auto f = k_gn<T, V, false>, g = k_gn_bwd<T, V, false>;
  return bwd ? go(g, smem_optin<g>(s.smem)) : go(f, smem_optin<f>(s.smem));
}
template <class T>
cudaError_t gn_run_v(bool bwd, GnArgs& a, const GnShape& s, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (s.v == 8) return gn_run<T, 8>(bwd, a, s, st);
  }
  if (s.v == 4) return gn_run<T, 4>(bwd, a, s, st);
  if (s.v == 2) return gn_run<T, 2>(bwd, a, s, st);
  return gn_run<T, 1>(bwd, a, s, st);
}
cudaError_t gn_run_t(int type, bool bwd, GnArgs& a, const GnShape& s, cudaStream_t st) {
  if (type == CTCPB_F32) return gn_run_v<float>(bwd, a, s, st);
  if (type == CTCPB_BF16) return gn_run_v<__nv_bfloat16>(bwd, a, s, st);
  return gn_run_v<__half>(bwd, a, s, st);
}

int gn_check(int type, int ptype, int act, int B, int T, int C, int G) {
  if (type != CTCPB_F32 && type != CTCPB_BF16 && type != CTCPB_F16) return CTCPB_EINVAL;
  if (ptype != type && ptype != CTCPB_F32) return CTCPB_EINVAL;
  if (act < CTCPB_ACT_NONE || act > CTCPB_ACT_SILU) return CTCPB_EINVAL;
  if (B < 0 || T < 0 || (long long)B * T > kHeadMaxRows || B > kHeadMaxRows || T > kHeadMaxRows || C < 1 ||
      C > kHeadMaxWidth || G < 1 || C % G)
    return CTCPB_EINVAL;
  return CTCPB_OK;
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" {

int ctcpb_group_norm(int type, int param_type, const void* x, int64_t x_stride_b, int64_t x_stride_t,
                     const void* weight, const void* bias, const int32_t* lengths, float eps, int activation, int B,
                     int T, int C, int G, void* y, int64_t y_stride_b, int64_t y_stride_t, float* mean, float* rstd,
                     ctcpb_stream_t stream) {
  int rc = gn_check(type, weight || bias ? param_type : type, activation, B, T, C, G);
  if (rc) return rc;
  if (!(eps >= 0.f)) return CTCPB_EINVAL;
  if ((mean == nullptr) != (rstd == nullptr)) return CTCPB_ENULL;
  if (B == 0 || (T == 0 && !mean)) return CTCPB_OK;
  if (T > 0 && (x_stride_t < C || y_stride_t < C || x_stride_b < 0 || y_stride_b < 0)) return CTCPB_EINVAL;
  if (T > 0 && (!x || !y)) return CTCPB_ENULL;
  GnArgs a{};
  a.x = x;
  a.y = y;
  a.x_b = x_stride_b;
  a.x_t = x_stride_t;
  a.y_b = y_stride_b;
  a.y_t = y_stride_t;
  a.weight = weight;
  a.bias = bias;
  a.ptype = param_type;
  a.lengths = lengths;
  a.B = B;
  a.T = T;
  a.C = C;
  a.G = G;
  a.D = C / G;
  a.eps = eps;
  a.act = activation;
  a.mean = mean;
  a.rstd = rstd;
  const int v = gn_vec(type, a.D, (uintptr_t)x | (uintptr_t)y, x_stride_b | x_stride_t | y_stride_b | y_stride_t);
  const GnShape s = gn_shape(type, v, B, T, C, G, false);
  return gn_run_t(type, false, a, s, (cudaStream_t)stream) == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
}

int ctcpb_group_norm_workspace_size(int B, int T, int C, int G, size_t* bytes) {
  int rc = gn_check(CTCPB_F32, CTCPB_F32, CTCPB_ACT_NONE, B, T, C, G);
  if (rc) return rc;
  if (!bytes) return CTCPB_ENULL;
  long long rows = kGnPartSize / C < kGnPart ? kGnPartSize / C : kGnPart;
  if (rows < kGnRanks) rows = kGnRanks;
  if (rows > (long long)B * kGnRanks) rows = (long long)B * kGnRanks;
  *bytes = align_up((size_t)(rows > 0 ? rows : 1) * 2 * C * 4, 256);
  return CTCPB_OK;
}

int ctcpb_group_norm_backward(int type, int param_type, const void* dy, int64_t dy_stride_b, int64_t dy_stride_t,
                              const void* x, int64_t x_stride_b, int64_t x_stride_t, const void* weight,
                              const void* bias, const int32_t* lengths, const float* mean, const float* rstd,
                              int activation, int B, int T, int C, int G, void* dx, int64_t dx_stride_b,
                              int64_t dx_stride_t, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                              ctcpb_stream_t stream) {
  const bool cols = dweight || dbias;
  int rc = gn_check(type, weight || bias || cols ? param_type : type, activation, B, T, C, G);
  if (rc) return rc;
  if (!dx && !cols) return CTCPB_OK;
  const bool any = B > 0 && T > 0;
  if (any && (x_stride_t < C || dy_stride_t < C || x_stride_b < 0 || dy_stride_b < 0 ||
              (dx && (dx_stride_t < C || dx_stride_b < 0))))
    return CTCPB_EINVAL;
  if (any && (!dy || !x || !mean || !rstd)) return CTCPB_ENULL;
  if (cols) {
    size_t need = 0;
    if ((rc = ctcpb_group_norm_workspace_size(B, T, C, G, &need))) return rc;
    if (!ws) return CTCPB_ENULL;
    if (((uintptr_t)ws & 255u) != 0) return CTCPB_EALIGN;
    if (ws_bytes < need) return CTCPB_ESIZE;
  }
  cudaStream_t st = (cudaStream_t)stream;
  int rows = 0;
  if (any) {
    GnArgs a{};
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.x_b = x_stride_b;
    a.x_t = x_stride_t;
    a.dy_b = dy_stride_b;
    a.dy_t = dy_stride_t;
    a.y_b = dx ? dx_stride_b : 0;
    a.y_t = dx ? dx_stride_t : 0;
    a.weight = weight;
    a.bias = bias;
    a.ptype = param_type;
    a.lengths = lengths;
    a.B = B;
    a.T = T;
    a.C = C;
    a.G = G;
    a.D = C / G;
    a.act = activation;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = cols ? (float*)ws : nullptr;
    const int v = gn_vec(type, a.D, (uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx,
                         x_stride_b | x_stride_t | dy_stride_b | dy_stride_t | a.y_b | a.y_t);
    const GnShape s = gn_shape(type, v, B, T, C, G, true);
    rows = s.by * s.ranks;
    if (gn_run_t(type, true, a, s, st) != cudaSuccess) return CTCPB_ECUDA;
  }
  if (cols && launch(k_gn_cols, (2 * C + 31) / 32, 1024, 0, st, 1, (const float*)ws, rows, C, param_type, dweight, dbias) !=
                  cudaSuccess)
    return CTCPB_ECUDA;
  return CTCPB_OK;
}

}  // extern "C"
