// Group norm in two launches, where no cluster's shared memory holds an utterance's
// frames of some whole groups, or too few blocks would work: the utterances' frames
// are dealt to as many blocks as fill the GPU, first for the groups' sums of each
// block's frames, then, every block adding up its groups' over all of them, for the
// outputs.  x (and dy) are read twice, the second time from L2 where they fit: 2 x 20000
// x 512 float16 23 us (3.6 TB/s of x read and y written once; 12 us would be HBM's).
#include <type_traits>

#include "ctcpb_gnorm.cuh"

namespace ctcpb {
namespace {

constexpr int kAhead = 8;  // rows that a thread has on their way

// The second launches begin before the first is done: what they read besides its sums
// was there before the first began, since that had waited for it when it let them begin
// (pdl_wait, then pdl_next).

// The group's sums over the parts of the frames, in order (a warp for each group).
template <class S>
__device__ __forceinline__ void over_parts(const GnArgs& a, const Place& p, int b, S* all) {
  const S* const g = reinterpret_cast<const S*>(a.group) + (long long)b * a.parts * a.G * a.pieces;
  const int lane = threadIdx.x & 31, n = a.parts * a.pieces;
  for (int k = threadIdx.x >> 5; k < p.groups; k += blockDim.x >> 5) {
    S t{};
    for (int e = lane; e < n; e += 32) {
      const int part = e / a.pieces;
      t.join(g[((long long)part * a.G + p.g0 + k) * a.pieces + e - part * a.pieces]);
    }
    warp_join(t);
    if (lane == 0) all[k] = t;
  }
  __syncthreads();
}
template <class S>
__device__ __forceinline__ S* group_slot(const GnArgs& a, const Place& p, int b) {
  return reinterpret_cast<S*>(a.group) + (((long long)b * a.parts + p.part) * a.G + p.g0) * a.pieces + p.piece;
}

template <class T, int V>
__global__ void __launch_bounds__(kGnThreads, 2) k_gn_stats(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int P = W::P;
  Moments* const each = reinterpret_cast<Moments*>(smem);
  Place p;
  p.set<V>(a, blockIdx.x, blockIdx.y);
  pdl_wait();
  pdl_next();
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const Rows rows(a, p, frames_of(a, b));
    const T* x = (const T*)a.x + (long long)b * a.x_b + p.c0 + rows.first * a.x_t + p.cv * V;
    const long long step = a.rs * a.x_t;
    Moments m{0.f, 0.f, 0.f};
    for (int k = 0; k < rows.n; k += kAhead, x += kAhead * step) {
      W raw[kAhead];
      const int here = rows.n - k < kAhead ? rows.n - k : kAhead;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < here) raw[i].load(x + i * step);
      u64 s[P], q[P];
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] = q[i] = 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < here) {
          u64 v[P];
          raw[i].get(v);
#pragma unroll
          for (int j = 0; j < P; ++j) s[j] = add2(s[j], v[j]);
        }
      const float n = (float)(here * V), mean = __fdividef(lanes<V>(s), n);
      const u64 nm = pair(-mean, -mean);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < here) {
          u64 v[P];
          raw[i].get(v);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            v[j] = add2(v[j], nm);
            q[j] = fma2(v[j], v[j], q[j]);
          }
        }
      m.join(Moments{n, mean, lanes<V>(q)});
    }
    by_group<Moments, V>(a, p, m, each, [&](int g, const Moments& t) { group_slot<Moments>(a, p, b)[g * a.pieces] = t; });
    __syncthreads();
  }
}

template <class T, int V>
__global__ void __launch_bounds__(kGnThreads, 2) k_gn_apply(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int P = W::P, U = 4;
  Moments* const all = reinterpret_cast<Moments*>(smem);
  Place p;
  p.set<V>(a, blockIdx.x, blockIdx.y);
  u64 w[P], bias[P];
  params_of<V>(a, p.c0 + p.cv * V, p.on, w, bias);
  const long long step = a.rs * a.x_t, y_step = a.rs * a.y_t;
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const int len = frames_of(a, b);
    const Rows rows(a, p, len);
    const T* x = (const T*)a.x + (long long)b * a.x_b + p.c0 + rows.first * a.x_t + p.cv * V;
    T* const y = (T*)a.y + (long long)b * a.y_b + p.c0;
    W raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < rows.n) raw[i].load(x + i * step);
    if (b == (int)blockIdx.z) {
      pdl_wait();
      pdl_next();
    }
    over_parts<Moments>(a, p, b, all);
    if (a.mean && p.part == 0 && p.piece == 0)
      for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
        const long long o = (long long)b * a.G + p.g0 + g;
        a.mean[o] = all[g].mean;
        a.rstd[o] = len > 0 ? all[g].rstd(a.eps) : 0.f;
      }
    const Moments t = all[p.group<V>(a)];
    const float rstd = t.rstd(a.eps);
    const u64 nm = pair(-t.mean, -t.mean);
    u64 wr[P];
#pragma unroll
    for (int i = 0; i < P; ++i) wr[i] = mul2(w[i], pair(rstd, rstd));
    T* to = y + rows.first * a.y_t + p.cv * V;
    for (int k = 0; k < rows.n; k += U, to += U * y_step) {
      W now[U];
      x += U * step;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        now[i] = raw[i];
        if (k + U + i < rows.n) raw[i].load(x + i * step);
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (k + i < rows.n) {
          u64 v[P];
          now[i].get(v);
          activate(v, nm, wr, bias, a.act);
          now[i].put(v);
          now[i].store(to + i * y_step);
        }
    }
    zero_rows<T, V>(a, p, y, len);
    __syncthreads();
  }
}

template <class T, int V>
__global__ void __launch_bounds__(kGnThreads, 1) k_gn_bwd_sums(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int P = W::P, U = 4;
  Two* const each = reinterpret_cast<Two*>(smem);
  float* const red = reinterpret_cast<float*>(each + blockDim.x);
  Place p;
  p.set<V>(a, blockIdx.x, blockIdx.y);
  pdl_wait();
  pdl_next();
  u64 w[P], bias[P];
  params_of<V>(a, p.c0 + p.cv * V, p.on, w, bias);
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const Rows rows(a, p, frames_of(a, b));
    const T* x = (const T*)a.x + (long long)b * a.x_b + p.c0 + rows.first * a.x_t + p.cv * V;
    const T* dy = (const T*)a.dy + (long long)b * a.dy_b + p.c0 + rows.first * a.dy_t + p.cv * V;
    const long long step = a.rs * a.x_t, d_step = a.rs * a.dy_t, o = (long long)b * a.G + p.g0 + p.group<V>(a);
    const float mean = a.mean[o], rstd = a.rstd[o];
    const u64 nm = pair(-mean, -mean);
    u64 wr[P], sw[P], sb[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      wr[i] = mul2(w[i], pair(rstd, rstd));
      sw[i] = sb[i] = 0;
    }
    for (int k = 0; k < rows.n; k += U, x += U * step, dy += U * d_step) {
      W raw[U], raw_d[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (k + i < rows.n) {
          raw[i].load(x + i * step);
          raw_d[i].load(dy + i * d_step);
        }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (k + i < rows.n) {
          u64 v[P], d[P];
          raw[i].get(v);
          raw_d[i].get(d);
          before(v, d, nm, wr, bias, a.act);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            sw[j] = fma2(d[j], v[j], sw[j]);
            sb[j] = add2(sb[j], d[j]);
          }
        }
    }
    const Two m = thread_sums<V>(sw, sb, wr);
    if (a.cols) add_columns<V>(a, p, sw, sb, rstd, red, b != (int)blockIdx.z);
    if (a.y) by_group<Two, V>(a, p, m, each, [&](int g, const Two& t) { group_slot<Two>(a, p, b)[g * a.pieces] = t; });
    __syncthreads();
  }
  if (a.cols) column_sums<V>(a, p, red, (long long)blockIdx.z * a.parts + p.part);
}

template <class T, int V>
__global__ void __launch_bounds__(kGnThreads, 1) k_gn_bwd_apply(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int P = W::P, U = 4;
  Two* const all = reinterpret_cast<Two*>(smem);
  Place p;
  p.set<V>(a, blockIdx.x, blockIdx.y);
  u64 w[P], bias[P];
  params_of<V>(a, p.c0 + p.cv * V, p.on, w, bias);
  const long long step = a.rs * a.x_t, d_step = a.rs * a.dy_t, y_step = a.rs * a.y_t;
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const int len = frames_of(a, b);
    const Rows rows(a, p, len);
    const T* x = (const T*)a.x + (long long)b * a.x_b + p.c0 + rows.first * a.x_t + p.cv * V;
    const T* dy = (const T*)a.dy + (long long)b * a.dy_b + p.c0 + rows.first * a.dy_t + p.cv * V;
    T* const y = (T*)a.y + (long long)b * a.y_b + p.c0;
    const long long o = (long long)b * a.G + p.g0 + p.group<V>(a);
    W raw[U], raw_d[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < rows.n) {
        raw[i].load(x + i * step);
        raw_d[i].load(dy + i * d_step);
      }
    const float mean = a.mean[o], rstd = a.rstd[o];
    const u64 nm = pair(-mean, -mean);
    u64 wr[P], m0, m1;
#pragma unroll
    for (int i = 0; i < P; ++i) wr[i] = mul2(w[i], pair(rstd, rstd));
    if (b == (int)blockIdx.z) {
      pdl_wait();
      pdl_next();
    }
    over_parts<Two>(a, p, b, all);
    factors(a, all[p.group<V>(a)], len, rstd, m0, m1);
    T* to = y + rows.first * a.y_t + p.cv * V;
    for (int k = 0; k < rows.n; k += U, to += U * y_step) {
      W now[U], now_d[U];
      x += U * step;
      dy += U * d_step;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        now[i] = raw[i];
        now_d[i] = raw_d[i];
        if (k + U + i < rows.n) {
          raw[i].load(x + i * step);
          raw_d[i].load(dy + i * d_step);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (k + i < rows.n) {
          u64 v[P], d[P];
          now[i].get(v);
          now_d[i].get(d);
          before(v, d, nm, wr, bias, a.act);
#pragma unroll
          for (int j = 0; j < P; ++j) d[j] = fma2(d[j], wr[j], fma2(v[j], m1, m0));
          now[i].put(d);
          now[i].store(to + i * y_step);
        }
    }
    zero_rows<T, V>(a, p, y, len);
    __syncthreads();
  }
}

template <class T>
cudaError_t split(bool bwd, const GnArgs& a, const GnShape& s, cudaStream_t st) {
  return gn_each_vec<T>(s.v, [&](auto, auto vc) {
    constexpr int V = decltype(vc)::value;
    const dim3 grid(s.slabs, s.parts, s.by);
    cudaError_t e = launch(bwd ? k_gn_bwd_sums<T, V> : k_gn_stats<T, V>, grid, s.threads, s.smem, st, 1, a);
    if (e == cudaSuccess && a.y)
      e = launch(bwd ? k_gn_bwd_apply<T, V> : k_gn_apply<T, V>, dim3(s.slabs, s.parts, a.B < 65535 ? a.B : 65535), s.threads,
                 s.smem, st, 1, a);
    return e;
  });
}

}  // namespace

cudaError_t gn_split(int type, bool bwd, GnArgs& a, const GnShape& s, cudaStream_t st) {
  if (type == CTCPB_F32) return split<float>(bwd, a, s, st);
  if (type == CTCPB_BF16) return split<__nv_bfloat16>(bwd, a, s, st);
  return split<__half>(bwd, a, s, st);
}

}  // namespace ctcpb
