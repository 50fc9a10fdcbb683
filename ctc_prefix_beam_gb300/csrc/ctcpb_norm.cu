// Layer norm and its backward pass (ctcpb_layer_norm, ctcpb_layer_norm_backward).
//
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  t = dy w
//   dx = rstd (t - mean(t) - xh mean(t xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and
// writes dx.  A row is held in registers, 16 elements a thread, by the fewest
// warps that hold it; the next row's loads are in flight while one is worked
// on.  The sums over rows for dw and db stay in the registers of the threads
// that own the columns, so they cost no traffic until a block's last row.
#include "ctcpb_head.cuh"

namespace ctcpb {
namespace {

constexpr int kPer = 16;        // elements of a row a thread holds
constexpr int kLnBlocks = 304;  // two blocks an SM; also the number of partial column sums

struct NormArgs {
  const void* x;
  long long ldx;
  const void* dy;
  long long lddy;
  const void* weight;
  const void* bias;
  int ptype;
  float eps;
  long long N;
  int H;
  int wpr;  // warps of a row
  void* y;  // or dx
  long long ldy;
  float* mean;
  float* rstd;
  float* part;  // [blocks][2][H]
};

// A thread's 16 elements of a row as they are in memory: whole 16-byte pieces
// (VEC), or single elements.
template <class T, bool VEC>
struct Piece {
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, C = kPer / V;
  union {
    uint4 q[VEC ? C : 1];
    T e[kPer];
  };
  __device__ __forceinline__ Piece() {}
  __device__ __forceinline__ void load(const T* row, int t, int tpr, int H, bool live) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = (i * tpr + t) * V;
      if constexpr (VEC)
        q[i] = live && at < H ? *reinterpret_cast<const uint4*>(row + at) : make_uint4(0, 0, 0, 0);
      else
        e[i] = live && at < H ? row[at] : Elem<T>::from(0.f);
    }
  }
  __device__ __forceinline__ void get(float (&v)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = Elem<T>::to(e[i]);
  }
  __device__ __forceinline__ void put(const float (&v)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = Elem<T>::from(v[i]);
  }
  __device__ __forceinline__ void store(T* row, int t, int tpr, int H) const {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = (i * tpr + t) * V;
      if (at < H) {
        if constexpr (VEC)
          *reinterpret_cast<uint4*>(row + at) = q[i];
        else
          row[at] = e[i];
      }
    }
  }
  // column of element i
  static __device__ __forceinline__ int col(int i, int t, int tpr) { return ((i / V) * tpr + t) * V + i % V; }
};

// Sums over the threads of a row (wpr warps; every thread of the block calls).
template <bool MULTI>
__device__ __forceinline__ float2 row_sum(float2 v, int wpr, float2* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, s);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, s);
  }
  if constexpr (MULTI) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
    const int w0 = warp / wpr * wpr;
    for (int w = 0; w < wpr; ++w) {
      v.x += red[w0 + w].x;
      v.y += red[w0 + w].y;
    }
  }
  return v;
}

template <class T, bool VEC, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 512 : 256) k_ln(const NormArgs a) {
  __shared__ float2 red[2][32];  // two buffers: a row's second sum may be written while its first is read
  const int wpr = MULTI ? a.wpr : 1, tpr = wpr * 32;
  const int per = (int)blockDim.x / tpr;  // rows a block works on at once
  const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
  using P = Piece<T, VEC>;
  float w[kPer], b[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = P::col(i, t, tpr);
    w[i] = c < a.H && a.weight ? load_elem(a.weight, a.ptype, c) : 1.f;
    b[i] = c < a.H && a.bias ? load_elem(a.bias, a.ptype, c) : 0.f;
  }
  const float inv = 1.f / (float)a.H;
  const long long step = (long long)gridDim.x * per;
  P next;
  long long r = (long long)blockIdx.x * per + g;
  next.load((const T*)a.x + r * a.ldx, t, tpr, a.H, r < a.N);
  for (long long r0 = (long long)blockIdx.x * per; r0 < a.N; r0 += step, r += step) {
    float v[kPer];
    next.get(v);
    const bool live = r < a.N;
    next.load((const T*)a.x + (r + step) * a.ldx, t, tpr, a.H, r + step < a.N);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s += v[i];
    const float mean = row_sum<MULTI>(make_float2(s, 0.f), wpr, red[0]).x * inv;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] -= mean;
      ss = P::col(i, t, tpr) < a.H ? __fmaf_rn(v[i], v[i], ss) : ss;
    }
    const float var = row_sum<MULTI>(make_float2(ss, 0.f), wpr, red[1]).x * inv;
    const float rstd = rsqrtf(var + a.eps);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = __fmaf_rn(v[i] * rstd, w[i], b[i]);
    if (live) {
      P out;
      out.put(v);
      out.store((T*)a.y + r * a.ldy, t, tpr, a.H);
      if (t == 0 && a.mean) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
      }
    }
  }
}

template <class T, bool VEC, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 512 : 256) k_ln_bwd(const NormArgs a) {
  extern __shared__ float col_sums[];  // [2][H]
  __shared__ float2 red[2][32];
  const int wpr = MULTI ? a.wpr : 1, tpr = wpr * 32;
  const int per = (int)blockDim.x / tpr;
  const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
  using P = Piece<T, VEC>;
  float w[kPer], dw[kPer], db[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = P::col(i, t, tpr);
    w[i] = c < a.H && a.weight ? load_elem(a.weight, a.ptype, c) : 1.f;
    dw[i] = db[i] = 0.f;
  }
  const float inv = 1.f / (float)a.H;
  const long long step = (long long)gridDim.x * per;
  P nx, ny;
  float nmean = 0.f, nrstd = 0.f;
  long long r = (long long)blockIdx.x * per + g;
  int par = 0;
  auto fetch = [&](long long row) {
    const bool live = row < a.N;
    nx.load((const T*)a.x + row * a.ldx, t, tpr, a.H, live);
    ny.load((const T*)a.dy + row * a.lddy, t, tpr, a.H, live);
    nmean = live ? a.mean[row] : 0.f;
    nrstd = live ? a.rstd[row] : 0.f;
  };
  fetch(r);
  for (long long r0 = (long long)blockIdx.x * per; r0 < a.N; r0 += step, r += step) {
    float xh[kPer], d[kPer];
    nx.get(xh);
    ny.get(d);
    const float mean = nmean, rstd = nrstd;
    const bool live = r < a.N;
    fetch(r + step);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // a column past H has d = 0, so it adds nothing
      xh[i] = (xh[i] - mean) * rstd;
      db[i] += d[i];
      dw[i] = __fmaf_rn(d[i], xh[i], dw[i]);
      d[i] *= w[i];
      s0 += d[i];
      s1 = __fmaf_rn(d[i], xh[i], s1);
    }
    const float2 s = row_sum<MULTI>(make_float2(s0, s1), wpr, red[par]);
    par ^= 1;
    if (live && a.y) {
      const float m0 = s.x * inv, m1 = s.y * inv;
#pragma unroll
      for (int i = 0; i < kPer; ++i) d[i] = rstd * (d[i] - m0 - xh[i] * m1);
      P out;
      out.put(d);
      out.store((T*)a.y + r * a.ldy, t, tpr, a.H);
    }
  }
  if (!a.part) return;
  // the block's rows are dealt to its groups: their sums, in order
  for (int k = 0; k < per; ++k) {
    if (g == k) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int c = P::col(i, t, tpr);
        if (c < a.H) {
          col_sums[c] = k ? col_sums[c] + dw[i] : dw[i];
          col_sums[a.H + c] = k ? col_sums[a.H + c] + db[i] : db[i];
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * a.H; c += blockDim.x) a.part[(long long)blockIdx.x * 2 * a.H + c] = col_sums[c];
}

// dw and db: the blocks' sums, in order (8 slices of the blocks, then the slices).
__global__ void __launch_bounds__(256) k_ln_cols(const float* __restrict__ part, int blocks, int H, int ptype, void* dw,
                                                 void* db) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * H)
    for (int j = warp; j < blocks; j += 8) s += part[(long long)j * 2 * H + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * H) {
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    if (c < H) {
      if (dw) store_elem(dw, ptype, c, s);
    } else if (db) {
      store_elem(db, ptype, c - H, s);
    }
  }
}

struct Shape {
  int wpr, threads, blocks;
};
Shape shape_of(long long N, int H) {
  Shape s{1, 256, 0};
  while (s.wpr * 32 * kPer < H) s.wpr *= 2;
  if (s.wpr > 8) s.threads = s.wpr * 32;
  const int per = s.threads / 32 / s.wpr;
  const long long b = (N + per - 1) / per;
  s.blocks = (int)(b < kLnBlocks ? b : kLnBlocks);
  return s;
}

bool vec_ok(int type, const void* p, long long ld) {
  const int v = type == CTCPB_F32 ? 4 : 8;
  return ((uintptr_t)p & 15) == 0 && ld % v == 0;
}

template <class T, bool VEC, bool MULTI>
cudaError_t run_t(bool bwd, const NormArgs& a, const Shape& s, cudaStream_t st) {
  if (bwd) {
    const size_t smem = a.part ? (size_t)2 * a.H * 4 : 0;
    constexpr auto kern = k_ln_bwd<T, VEC, MULTI>;
    if (smem > 48 * 1024) {
      cudaError_t e = smem_optin<kern>(smem);
      if (e != cudaSuccess) return e;
    }
    kern<<<s.blocks, s.threads, smem, st>>>(a);
  } else {
    k_ln<T, VEC, MULTI><<<s.blocks, s.threads, 0, st>>>(a);
  }
  return cudaGetLastError();
}
template <class T>
cudaError_t run(bool bwd, bool vec, const NormArgs& a, const Shape& s, cudaStream_t st) {
  if (a.wpr == 1) return vec ? run_t<T, true, false>(bwd, a, s, st) : run_t<T, false, false>(bwd, a, s, st);
  return vec ? run_t<T, true, true>(bwd, a, s, st) : run_t<T, false, true>(bwd, a, s, st);
}
cudaError_t run(int type, bool bwd, bool vec, const NormArgs& a, const Shape& s, cudaStream_t st) {
  if (type == CTCPB_F32) return run<float>(bwd, vec, a, s, st);
  if (type == CTCPB_BF16) return run<__nv_bfloat16>(bwd, vec, a, s, st);
  return run<__half>(bwd, vec, a, s, st);
}

int check(int type, int ptype, long long N, int H) {
  if (type != CTCPB_F32 && type != CTCPB_BF16 && type != CTCPB_F16) return CTCPB_EINVAL;
  if (ptype != type && ptype != CTCPB_F32) return CTCPB_EINVAL;
  if (N < 0 || N > kHeadMaxRows || H < 1 || H > kHeadMaxWidth) return CTCPB_EINVAL;
  return CTCPB_OK;
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" {

int ctcpb_layer_norm(int type, int param_type, const void* x, int64_t ldx, const void* weight, const void* bias,
                     float eps, int64_t N, int H, void* y, int64_t ldy, float* mean, float* rstd,
                     ctcpb_stream_t stream) {
  int rc = check(type, weight || bias ? param_type : type, N, H);
  if (rc) return rc;
  if (!(eps >= 0.f)) return CTCPB_EINVAL;
  if (N == 0) return CTCPB_OK;
  if (ldx < H || ldy < H) return CTCPB_EINVAL;
  if (!x || !y || (mean == nullptr) != (rstd == nullptr)) return CTCPB_ENULL;
  const Shape s = shape_of(N, H);
  NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.ptype = param_type;
  a.eps = eps;
  a.N = N;
  a.H = H;
  a.wpr = s.wpr;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  const bool vec = H % (type == CTCPB_F32 ? 4 : 8) == 0 && vec_ok(type, x, ldx) && vec_ok(type, y, ldy);
  return run(type, false, vec, a, s, (cudaStream_t)stream) == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
}

int ctcpb_layer_norm_workspace_size(int64_t N, int H, size_t* bytes) {
  int rc = check(CTCPB_F32, CTCPB_F32, N, H);
  if (rc) return rc;
  if (!bytes) return CTCPB_ENULL;
  const Shape s = shape_of(N, H);
  *bytes = align_up((size_t)(s.blocks > 0 ? s.blocks : 1) * 2 * H * 4, 256);
  return CTCPB_OK;
}

int ctcpb_layer_norm_backward(int type, int param_type, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                              const void* weight, const float* mean, const float* rstd, int64_t N, int H, void* dx,
                              int64_t lddx, void* dweight, void* dbias, void* ws, size_t ws_bytes,
                              ctcpb_stream_t stream) {
  int rc = check(type, weight || dweight || dbias ? param_type : type, N, H);
  if (rc) return rc;
  if (!dx && !dweight && !dbias) return CTCPB_OK;
  if (N > 0 && (ldx < H || lddy < H || (dx && lddx < H))) return CTCPB_EINVAL;
  if (N > 0 && (!dy || !x || !mean || !rstd)) return CTCPB_ENULL;
  const bool cols = dweight || dbias;
  if (cols) {
    size_t need = 0;
    if ((rc = ctcpb_layer_norm_workspace_size(N, H, &need))) return rc;
    if (!ws) return CTCPB_ENULL;
    if (((uintptr_t)ws & 255u) != 0) return CTCPB_EALIGN;
    if (ws_bytes < need) return CTCPB_ESIZE;
  }
  const Shape s = shape_of(N, H);
  cudaStream_t st = (cudaStream_t)stream;
  if (N > 0) {
    NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.dy = dy;
    a.lddy = lddy;
    a.weight = weight;
    a.ptype = param_type;
    a.N = N;
    a.H = H;
    a.wpr = s.wpr;
    a.y = dx;
    a.ldy = lddx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = cols ? (float*)ws : nullptr;
    const bool vec = H % (type == CTCPB_F32 ? 4 : 8) == 0 && vec_ok(type, x, ldx) && vec_ok(type, dy, lddy) &&
                     (!dx || vec_ok(type, dx, lddx));
    if (run(type, true, vec, a, s, st) != cudaSuccess) return CTCPB_ECUDA;
  }
  if (cols) {
    k_ln_cols<<<(2 * H + 31) / 32, 256, 0, st>>>((const float*)ws, N > 0 ? s.blocks : 0, H, param_type, dweight, dbias);
    if (cudaGetLastError() != cudaSuccess) return CTCPB_ECUDA;
  }
  return CTCPB_OK;
}

}  // extern "C"
