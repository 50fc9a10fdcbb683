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
// will read itself.  What no cluster holds, or too few blocks would work on, takes
// two launches (ctcpb_gnorm_split.cu).
//
// 128 utterances of up to 500 frames (375 on average) of 1024 channels, bfloat16, SiLU:
// forward 49 us (4.7 TB/s of x read and y written, padding and all), backward 96 (3.4),
// its column sums 5.  What bounds it is the work between a block's loads and its stores:
// with three to six blocks an SM the issue slots are 52 to 62% busy, HBM some 45%.
#include <type_traits>

#include "ctcpb_gnorm.cuh"

namespace ctcpb {
namespace {

constexpr int kGnRanks = 16;             // blocks that share a slab at most
constexpr int kGnSmem = 80 * 1024;       // what a block has of shared memory at most
constexpr int kGnSmemShare = 72 * 1024;  // ... and keeps of a slab, where more can share it: three on an SM
constexpr int kGnPart = 4096;            // blocks of a backward launch that hold column sums
constexpr long long kGnPartSize = 1 << 22;  // ... and their columns

// The slab's sums over the blocks of the cluster, in order: `own` -> `all`.
template <class S>
__device__ __forceinline__ void over_cluster(const GnArgs& a, const Place& p, S* own, S* all) {
  if (a.parts > 1) {
    __syncwarp();  // the barrier takes whole warps
    cluster_sync();
    constexpr int n = sizeof(S) / 4;
    for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
      S t{};
      for (int r = 0; r < a.parts; ++r) {
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
    // every block has read before any writes `own` again or leaves (over_cluster_done)
    asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
  }
  __syncthreads();
}
__device__ __forceinline__ void over_cluster_done(const GnArgs& a) {
  if (a.parts > 1) asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
}

template <class T, int V>
__global__ void __launch_bounds__(kGnThreads, 2) k_gn(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int P = W::P;
  Moments* const each = reinterpret_cast<Moments*>(smem);
  Moments* const own = each + blockDim.x;
  Moments* const all = own + a.gs;
  const u32 keep = (saddr(all + a.gs) + 15u & ~15u) + threadIdx.x * W::bytes;
  const u32 pitch = blockDim.x * W::bytes;
  Place p;
  p.set<V>(a, blockIdx.x / (u32)a.parts, blockIdx.x % (u32)a.parts);
  pdl_wait();
  pdl_next();
  u64 w[P], bias[P];
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int len = frames_of(a, b);
    const Rows rows(a, p, len);
    const T* const x = (const T*)a.x + (long long)b * a.x_b + p.c0;
    T* const y = (T*)a.y + (long long)b * a.y_b + p.c0;
    fetch_rows<T, V>(keep, pitch, x + rows.first * a.x_t + p.cv * V, a.rs * a.x_t, rows.n);
    params_of<V>(a, p.c0 + p.cv * V, p.on, w, bias);
    cp_wait_all();
    u64 s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = 0;
#pragma unroll 4
    for (int k = 0; k < rows.n; ++k) {
      W raw;
      u64 v[P];
      raw.load_shared(keep + k * pitch);
      raw.get(v);
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] = add2(s[i], v[i]);
    }
    Moments m{(float)(rows.n * V), 0.f, 0.f};
    if (rows.n > 0) m.mean = lanes<V>(s) / m.n;
    u64 nm = pair(-m.mean, -m.mean);
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = 0;
#pragma unroll 4
    for (int k = 0; k < rows.n; ++k) {
      W raw;
      u64 v[P];
      raw.load_shared(keep + k * pitch);
      raw.get(v);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v[i] = add2(v[i], nm);
        s[i] = fma2(v[i], v[i], s[i]);
      }
    }
    m.m2 = lanes<V>(s);
    by_group<Moments, V>(a, p, m, each, [&](int g, const Moments& t) { (a.parts > 1 ? own : all)[g] = t; });
    over_cluster(a, p, own, all);
    if (a.mean && p.part == 0)
      for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
        const long long o = (long long)b * a.G + p.g0 + g;
        a.mean[o] = all[g].mean;
        a.rstd[o] = len > 0 ? all[g].rstd(a.eps) : 0.f;
      }
    const Moments t = all[p.group<V>(a)];
    const float rstd = t.rstd(a.eps);
    nm = pair(-t.mean, -t.mean);
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = mul2(w[i], pair(rstd, rstd));
    const long long step = a.rs * a.y_t;
    T* to = y + rows.first * a.y_t + p.cv * V;
#pragma unroll 2
    for (int k = 0; k < rows.n; ++k, to += step) {
      W raw;
      u64 v[P];
      raw.load_shared(keep + k * pitch);
      raw.get(v);
      activate(v, nm, w, bias, a.act);
      raw.put(v);
      raw.store(to);
    }
    zero_rows<T, V>(a, p, y, len);
    over_cluster_done(a);
    __syncthreads();
  }
}

template <class T, int V>
__global__ void __launch_bounds__(kGnThreads, 2) k_gn_bwd(const GnArgs a) {
  extern __shared__ __align__(16) char smem[];
  typedef Vec<T, V> W;
  constexpr int P = W::P;
  Two* const each = reinterpret_cast<Two*>(smem);
  Two* const own = each + blockDim.x;
  Two* const all = own + a.gs;
  float* const red = reinterpret_cast<float*>(all + a.gs);
  const u32 keep = (saddr(red + 2 * a.cr * a.tw * V) + 15u & ~15u) + threadIdx.x * W::bytes;
  const u32 pitch = blockDim.x * W::bytes, second = a.slots * pitch;  // dy lies behind x
  Place p;
  p.set<V>(a, blockIdx.x / (u32)a.parts, blockIdx.x % (u32)a.parts);
  pdl_wait();
  pdl_next();
  u64 w[P], bias[P];
  params_of<V>(a, p.c0 + p.cv * V, p.on, w, bias);
  const int group = p.g0 + p.group<V>(a);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int len = frames_of(a, b);
    const Rows rows(a, p, len);
    const T* const x = (const T*)a.x + (long long)b * a.x_b + p.c0;
    const T* const dy = (const T*)a.dy + (long long)b * a.dy_b + p.c0;
    fetch_rows<T, V>(keep, pitch, x + rows.first * a.x_t + p.cv * V, a.rs * a.x_t, rows.n);
    fetch_rows<T, V>(keep + second, pitch, dy + rows.first * a.dy_t + p.cv * V, a.rs * a.dy_t, rows.n);
    const long long o = (long long)b * a.G + group;
    const float mean = a.mean[o], rstd = a.rstd[o];
    const u64 nm = pair(-mean, -mean);
    u64 wr[P], sw[P], sb[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      wr[i] = mul2(w[i], pair(rstd, rstd));
      sw[i] = sb[i] = 0;
    }
    cp_wait_all();
#pragma unroll 2
    for (int k = 0; k < rows.n; ++k) {
      W raw;
      u64 v[P], d[P];
      raw.load_shared(keep + k * pitch);
      raw.get(v);
      raw.load_shared(keep + second + k * pitch);
      raw.get(d);
      before(v, d, nm, wr, bias, a.act);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        sw[i] = fma2(d[i], v[i], sw[i]);
        sb[i] = add2(sb[i], d[i]);
      }
    }
    const Two m = thread_sums<V>(sw, sb, wr);
    if (a.cols) add_columns<V>(a, p, sw, sb, rstd, red, b != (int)blockIdx.y);
    if (a.y) {
      T* const y = (T*)a.y + (long long)b * a.y_b + p.c0;
      by_group<Two, V>(a, p, m, each, [&](int g, const Two& t) { (a.parts > 1 ? own : all)[g] = t; });
      over_cluster(a, p, own, all);
      u64 m0, m1;
      factors(a, all[p.group<V>(a)], len, rstd, m0, m1);
      const long long step = a.rs * a.y_t;
      T* to = y + rows.first * a.y_t + p.cv * V;
#pragma unroll 2
      for (int k = 0; k < rows.n; ++k, to += step) {
        W raw;
        u64 v[P], d[P];
        raw.load_shared(keep + k * pitch);
        raw.get(v);
        raw.load_shared(keep + second + k * pitch);
        raw.get(d);
        before(v, d, nm, wr, bias, a.act);
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = fma2(d[i], wr[i], fma2(v[i], m1, m0));
        raw.put(d);
        raw.store(to);
      }
      zero_rows<T, V>(a, p, y, len);
      over_cluster_done(a);
    }
    __syncthreads();
  }
  if (a.cols) column_sums<V>(a, p, red, (long long)blockIdx.y * a.parts + p.part);
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

// Elements of one access: a group's channels and every row start at its multiples.
int gn_vec(int type, int D, uintptr_t at, long long strides) {
  const int e = type == CTCPB_F32 ? 4 : 2;
  int v = 16 / e;
  while (v > 1 && (D % v != 0 || (at | (uintptr_t)(strides * e)) % (v * e) != 0)) v /= 2;
  return v;
}
int up32(long long n) { return (int)((n + 31) / 32 * 32); }

// Slabs of `bytes` of a row, at least a group, and as many of their rows at a time as
// `threads` take.
void gn_slabs(GnShape& s, int e, int T, int C, int G, int bytes, int threads) {
  const int D = C / G, dv = D / s.v;
  s.gs = bytes / (D * e) > 1 ? bytes / (D * e) : 1;
  while (s.gs < G && (long long)s.gs * dv * T < 32) s.gs *= 2;  // more where there are too few rows to fill a warp
  if (s.gs > G) s.gs = G;
  s.pieces = s.gs * dv > kGnThreads ? (dv + kGnThreads - 1) / kGnThreads : 1;
  s.tw = s.pieces > 1 ? (dv + s.pieces - 1) / s.pieces : s.gs * dv;
  s.slabs = s.pieces > 1 ? G * s.pieces : (G + s.gs - 1) / s.gs;
  s.threads = s.tw > threads ? up32(s.tw) : up32((long long)s.tw * T < threads ? (long long)s.tw * T : threads);
  if (s.threads < 32) s.threads = 32;
  s.rs = s.threads / s.tw;
  s.cr = 32 % s.tw == 0 && s.rs * s.tw == s.threads ? s.threads / 32 : s.rs;
}
size_t gn_sums(const GnShape& s, bool bwd) {  // shared memory but for the slab
  return align_up((size_t)(s.threads + 2 * s.gs) * (bwd ? sizeof(Two) : sizeof(Moments)) +
                      (bwd ? (size_t)s.cr * 2 * s.tw * s.v * 4 : 0), 16);
}

GnShape gn_shape(int type, int v, int B, int T, int C, int G, bool bwd) {
  GnShape s{};
  const int e = type == CTCPB_F32 ? 4 : 2;
  s.v = v;
  // slabs of 64 bytes of a row, so that a block keeps more frames of one (32 x 500 x 512: 11.6 us with 128
  // bytes, 10.8 with 64; forward and backward of 128 x 500 x 1024: 157 and 150); the forward pass has
  // blocks of 128 threads where there are many, whose start is then divided by twice the rows (50 us, 63
  // with 256; where there are few, 12.4 us instead of 10.8)
  gn_slabs(s, e, T, C, G, 64, 256);
  if (!bwd && (long long)B * s.slabs >= 152 * 8) gn_slabs(s, e, T, C, G, 64, 128);
  auto slab = [&](int ranks) {
    s.slots = ((T + ranks - 1) / ranks + s.rs - 1) / s.rs;
    return (size_t)s.slots * s.threads * v * e * (bwd ? 2 : 1);
  };
  s.parts = 1;
  while (s.parts < kGnRanks && T > 2 * s.parts * s.rs &&
         (slab(s.parts) > (size_t)kGnSmemShare || (long long)B * s.slabs * s.parts < 152))
    s.parts *= 2;
  s.smem = gn_sums(s, bwd) + slab(s.parts);
  s.split = s.pieces > 1 || s.smem > (size_t)kGnSmem;
  if (s.split) {
    // rows of 256 bytes (2 x 20000 x 512 float16: 27 us with 128, 23 with 256, 24 with 512, whose groups'
    // sums are of more parts), so many chunks of frames that the blocks just fill the SMs (29 us with
    // two thirds of it), eight of a thread's rows in each at least
    gn_slabs(s, e, T, C, G, 256, 256);
    const long long most = ((long long)T + 8 * s.rs - 1) / (8 * s.rs);
    long long parts = (152 * 3 + (long long)B * s.slabs - 1) / ((long long)B * s.slabs);
    if (parts > most) parts = most;
    s.parts = (int)(parts > 1 ? parts : 1);
    s.smem = gn_sums(s, bwd);
  }
  long long by = B;
  if (bwd) {  // column sums of so many blocks at most
    long long cap = kGnPart / ((long long)s.slabs * s.parts), room = kGnPartSize / C / s.parts;
    if (cap > room) cap = room;
    if (by > cap) by = cap > 1 ? cap : 1;
  }
  s.by = (int)(by < 65535 ? by : 65535);
  return s;
}
// Workspace: the column sums, then the groups' sums of a split call.
struct GnLayout {
  size_t o_group, total;
};
GnLayout gn_layout(const GnShape& s, int B, int C, int G, bool bwd) {
  GnLayout l{};
  l.o_group = bwd ? align_up((size_t)s.by * s.parts * 2 * C * 4, 256) : 0;
  l.total = l.o_group + (s.split ? align_up((size_t)B * s.parts * G * s.pieces * (bwd ? sizeof(Two) : sizeof(Moments)), 256) : 0);
  return l;
}

template <class T>
cudaError_t gn_whole(bool bwd, const GnArgs& a, const GnShape& s, cudaStream_t st) {
  return gn_each_vec<T>(s.v, [&](auto, auto vc) {
    constexpr int V = decltype(vc)::value;
    constexpr auto f = k_gn<T, V>, g = k_gn_bwd<T, V>;
    cudaError_t e = bwd ? smem_optin<g>(s.smem) : smem_optin<f>(s.smem);
    if (e == cudaSuccess && s.parts > 8)
      e = cudaFuncSetAttribute(bwd ? (const void*)g : (const void*)f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e != cudaSuccess ? e : launch(bwd ? g : f, dim3(s.slabs * s.parts, s.by), s.threads, s.smem, st, s.parts, a);
  });
}
cudaError_t gn_run(int type, bool bwd, GnArgs& a, const GnShape& s, cudaStream_t st) {
  a.gs = s.gs;
  a.pieces = s.pieces;
  a.tw = s.tw;
  a.rs = s.rs;
  a.slots = s.slots;
  a.parts = s.parts;
  a.cr = s.cr;
  a.by_tw = reciprocal(s.tw);
  a.by_rs = reciprocal(s.rs);
  a.by_dv = reciprocal(a.D / s.v);
  const int e = a.ptype == CTCPB_F32 ? 4 : 2;
  a.pvec = (((uintptr_t)a.weight | (uintptr_t)a.bias) & (s.v * e < 8 ? s.v * e - 1 : 7)) == 0;
  if (s.split) return gn_split(type, bwd, a, s, st);
  if (type == CTCPB_F32) return gn_whole<float>(bwd, a, s, st);
  if (type == CTCPB_BF16) return gn_whole<__nv_bfloat16>(bwd, a, s, st);
  return gn_whole<__half>(bwd, a, s, st);
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

// The most that any alignment of a call's tensors needs.
size_t gn_need(int type, int B, int T, int C, int G, bool bwd) {
  size_t most = 0;
  if (B > 0)
    for (int v = gn_vec(type, C / G, 0, 0); v >= 1; v /= 2) {
      const size_t n = gn_layout(gn_shape(type, v, B, T, C, G, bwd), B, C, G, bwd).total;
      if (n > most) most = n;
    }
  return most;
}
// What this call needs, at most gn_need.
int gn_workspace(GnArgs& a, const GnShape& s, bool bwd, void* ws, size_t ws_bytes) {
  const GnLayout l = gn_layout(s, a.B, a.C, a.G, bwd);
  if (l.total == 0) return CTCPB_OK;
  if (!ws) return CTCPB_ENULL;
  if (((uintptr_t)ws & 255u) != 0) return CTCPB_EALIGN;
  if (ws_bytes < l.total) return CTCPB_ESIZE;
  a.cols = bwd ? (float*)ws : nullptr;
  a.group = (float*)((char*)ws + l.o_group);
  return CTCPB_OK;
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" {

int ctcpb_group_norm(int type, int param_type, const void* x, int64_t x_stride_b, int64_t x_stride_t,
                     const void* weight, const void* bias, const int32_t* lengths, float eps, int activation, int B,
                     int T, int C, int G, void* y, int64_t y_stride_b, int64_t y_stride_t, float* mean, float* rstd,
                     void* ws, size_t ws_bytes, ctcpb_stream_t stream) {
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
  if ((rc = gn_workspace(a, s, false, ws, ws_bytes))) return rc;
  return gn_run(type, false, a, s, (cudaStream_t)stream) == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
}

int ctcpb_group_norm_workspace_size(int type, int B, int T, int C, int G, int backward, size_t* bytes) {
  int rc = gn_check(type, type, CTCPB_ACT_NONE, B, T, C, G);
  if (rc) return rc;
  if (backward != 0 && backward != 1) return CTCPB_EINVAL;
  if (!bytes) return CTCPB_ENULL;
  *bytes = gn_need(type, B, T, C, G, backward);
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
    const int v = gn_vec(type, a.D, (uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx,
                         x_stride_b | x_stride_t | dy_stride_b | dy_stride_t | a.y_b | a.y_t);
    const GnShape s = gn_shape(type, v, B, T, C, G, true);
    if ((rc = gn_workspace(a, s, true, ws, ws_bytes))) return rc;
    if (!cols) a.cols = nullptr;
    rows = s.by * s.parts;
    if (gn_run(type, true, a, s, st) != cudaSuccess) return CTCPB_ECUDA;
  }
  if (cols && launch(k_gn_cols, (2 * C + 31) / 32, 1024, 0, st, 1, (const float*)ws, rows, C, param_type, dweight, dbias) !=
                  cudaSuccess)
    return CTCPB_ECUDA;
  return CTCPB_OK;
}

}  // extern "C"
