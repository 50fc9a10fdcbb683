// Layer norm and its backward pass (ctcpb_layer_norm, ctcpb_layer_norm_backward).
//
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  t = dy w
//   dx = rstd (t - mean(t) - xh mean(t xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and
// writes dx.  A row is worked on by the fewest warps that hold it, 8 to 32
// elements a thread, in pairs (one instruction for two); the next rows are on
// their way into shared memory meanwhile, each thread copying just what it will
// read itself, so a row costs no barrier but the sums' own.  The sums over rows
// for dw and db stay in the registers of the threads that own the columns, so
// they cost no traffic until a block's last row.  64000 rows of 1024 in
// bfloat16: forward 42 us (6.2 TB/s), backward 68 us (5.8 TB/s) and 5 us for
// its column sums.
#include "ctcpb_head.cuh"

namespace ctcpb {
namespace {

constexpr int kLnBlocks = 456;  // three blocks an SM; also the number of partial column sums

__host__ __device__ constexpr int threads_of(int wpr) { return wpr > 8 ? wpr * 32 : 256; }  // of a block

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
  void* y;  // or dx
  long long ldy;
  float* mean;
  float* rstd;
  float* part;  // [blocks][2][H]
};

// A thread's E elements of a row as E / 2 pairs: C pieces of V elements, piece i
// at column (i * tpr + t) * V.  VEC: pieces are 16 bytes; else single elements.
template <class T, bool VEC, int E, int WPR>
struct Piece {
  static constexpr int tpr = 32 * WPR;  // threads of a row
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, C = E / V;
  // column of element i
  static __device__ __forceinline__ int col(int i, int t) { return ((i / V) * tpr + t) * V + i % V; }
  static __device__ __forceinline__ bool live(int i, int t, int H) { return (i * tpr + t) * V < H; }

  static __device__ __forceinline__ void unpack(uint4 q, u64* v) {  // one piece (VEC)
    if constexpr (sizeof(T) == 4) {
      v[0] = pair(__uint_as_float(q.x), __uint_as_float(q.y));
      v[1] = pair(__uint_as_float(q.z), __uint_as_float(q.w));
    } else {
      v[0] = Elem<T>::unpack(q.x);
      v[1] = Elem<T>::unpack(q.y);
      v[2] = Elem<T>::unpack(q.z);
      v[3] = Elem<T>::unpack(q.w);
    }
  }
  static __device__ __forceinline__ u32 pack(u64 v) {
    float x, y;
    unpair(x, y, v);
    return Elem<T>::pack(x, y);
  }
  static __device__ __forceinline__ void store(T* row, const u64 (&v)[E / 2], int t, int H) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (!live(i, t, H)) continue;
      T* const o = row + (i * tpr + t) * V;
      if constexpr (!VEC) {
        float x, y;
        unpair(x, y, v[i / 2]);
        *o = Elem<T>::from(i & 1 ? y : x);
      } else if constexpr (sizeof(T) == 4) {
        float4 f;
        unpair(f.x, f.y, v[2 * i]);
        unpair(f.z, f.w, v[2 * i + 1]);
        *reinterpret_cast<float4*>(o) = f;
      } else {
        *reinterpret_cast<uint4*>(o) = make_uint4(pack(v[4 * i]), pack(v[4 * i + 1]), pack(v[4 * i + 2]), pack(v[4 * i + 3]));
      }
    }
  }
};

// A thread's elements of a parameter vector (`none` where there is none).
template <class P, int E>
__device__ __forceinline__ void load_params(u64 (&v)[E / 2], const void* p, int type, int t, int H, float none) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const int c0 = P::col(2 * i, t), c1 = P::col(2 * i + 1, t);
    v[i] = pair(c0 < H && p ? load_elem(p, type, c0) : none, c1 < H && p ? load_elem(p, type, c1) : none);
  }
}

// The rows ahead of the one worked on, for NA arrays: kDepth rows in shared
// memory (VEC: 16-byte asynchronous copies), or one in registers.
template <class T, bool VEC, int E, int WPR, int NA>
struct Ahead {
  using P = Piece<T, VEC, E, WPR>;
  static constexpr int tpr = P::tpr;
  static constexpr int kDepth = VEC ? (NA * sizeof(T) * E > 64 ? 3 : 4) : 1;
  static constexpr int kStage = NA * P::C;  // 16-byte pieces of a thread
  T reg[VEC ? 1 : NA * E];
  // the ring, [depth][stage][threads]: the distances of its pieces and rows
  static constexpr u32 piece = threads_of(WPR) * 16, row_bytes = kStage * piece;
  u32 put_at, get_at, ring;
  __device__ __forceinline__ void init(char* smem) {
    put_at = get_at = ring = saddr(smem) + threadIdx.x * 16;
  }
  __device__ __forceinline__ void fetch(const T* const (&rows)[NA], int t, int H, bool row) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < P::C; ++i)
        if (row && P::live(i, t, H)) {
#pragma unroll
          for (int n = 0; n < NA; ++n)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(put_at + (n * P::C + i) * piece),
                         "l"(rows[n] + (i * tpr + t) * P::V)
                         : "memory");
        }
      cp_commit();
      put_at += row_bytes;
      if (put_at == ring + kDepth * row_bytes) put_at = ring;
    } else {
#pragma unroll
      for (int n = 0; n < NA; ++n)
#pragma unroll
        for (int i = 0; i < E; ++i)
          reg[n * E + i] = row && P::live(i, t, H) ? rows[n][i * tpr + t] : Elem<T>::from(0.f);
    }
  }
  // the oldest row fetched, zeros past its end (the caller keeps kDepth rows in flight)
  __device__ __forceinline__ void take(u64 (&v)[NA][E / 2], int t, int H) {
    if constexpr (VEC) {
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth - 1) : "memory");
#pragma unroll
      for (int i = 0; i < P::C; ++i) {
        const bool in = P::live(i, t, H);
#pragma unroll
        for (int n = 0; n < NA; ++n) {
          uint4 q = make_uint4(0, 0, 0, 0);
          if (in)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                         : "r"(get_at + (n * P::C + i) * piece)
                         : "memory");
          P::unpack(q, v[n] + i * (P::V / 2));
        }
      }
      get_at += row_bytes;
      if (get_at == ring + kDepth * row_bytes) get_at = ring;
    } else {
#pragma unroll
      for (int n = 0; n < NA; ++n)
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
          v[n][i] = pair(Elem<T>::to(reg[n * E + 2 * i]), Elem<T>::to(reg[n * E + 2 * i + 1]));
    }
  }
  static constexpr size_t bytes = VEC ? (size_t)kDepth * row_bytes : 0;
};

// Sums over the threads of a row (its wpr warps meet at a barrier of their own).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5, g = warp / WPR;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    asm volatile("bar.sync %0, %1;\n" ::"r"(1 + g), "n"(WPR * 32) : "memory");
    v = 0.f;
    #pragma unroll
    for (int w = 0; w < WPR; ++w) v += red[g * WPR + w];
  }
  return v;
}
template <int WPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, s);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, s);
  }
  if constexpr (WPR > 1) {
    const int warp = threadIdx.x >> 5, g = warp / WPR;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    asm volatile("bar.sync %0, %1;\n" ::"r"(1 + g), "n"(WPR * 32) : "memory");
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      v.x += red[g * WPR + w].x;
      v.y += red[g * WPR + w].y;
    }
  }
  return v;
}

template <class T, bool VEC, int WPR, int E>
__global__ void __launch_bounds__(threads_of(WPR), WPR <= 8 && VEC ? 2 : 1) k_ln(const NormArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2][32];  // two buffers: a row's second sum may be written while its first is read
  constexpr int tpr = 32 * WPR, per = threads_of(WPR) / tpr;  // rows a block works on at once
  const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
  using P = Piece<T, VEC, E, WPR>;
  using A = Ahead<T, VEC, E, WPR, 1>;
  pdl_wait();
  pdl_next();
  const long long step = (long long)gridDim.x * per, r0 = (long long)blockIdx.x * per + g;
  const long long jump_x = step * a.ldx, jump_y = step * a.ldy;
  A ahead;
  ahead.init(smem);
  const T* px = (const T*)a.x + r0 * a.ldx;  // the next row to fetch
  long long rx = r0;
  auto fetch = [&]() {
    const T* const rows[1] = {px};
    ahead.fetch(rows, t, a.H, rx < a.N);
    px += jump_x;
    rx += step;
  };
#pragma unroll
  for (int i = 0; i < A::kDepth; ++i) fetch();
  u64 w[E / 2], b[E / 2];
  load_params<P, E>(w, a.weight, a.ptype, t, a.H, 1.f);
  load_params<P, E>(b, a.bias, a.ptype, t, a.H, 0.f);
  const float inv = 1.f / (float)a.H;
  T* py = (T*)a.y + r0 * a.ldy;
  for (long long r = r0; r < a.N; r += step) {
    u64 va[1][E / 2];
    ahead.take(va, t, a.H);
    u64(&v)[E / 2] = va[0];
    fetch();
    u64 s = v[0], s1 = v[1];
#pragma unroll
    for (int i = 2; i < E / 2; i += 2) {
      s = add2(s, v[i]);
      s1 = add2(s1, v[i + 1]);
    }
    const float mean = row_sum<WPR>(pair_sum(add2(s, s1)), red[0]) * inv;
    const u64 nm = pair(-mean, -mean);
    s = s1 = 0;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[i] = add2(v[i], nm);
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < P::C; ++i)
        if (P::live(i, t, a.H)) {  // a piece is in the row or past its end
#pragma unroll
          for (int k = 0; k < P::V / 2; k += 2) {
            const u64 v0 = v[i * (P::V / 2) + k], v1 = v[i * (P::V / 2) + k + 1];
            s = fma2(v0, v0, s);
            s1 = fma2(v1, v1, s1);
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        float x, y;
        unpair(x, y, v[i]);
        const u64 d = pair(P::live(2 * i, t, a.H) ? x : 0.f, P::live(2 * i + 1, t, a.H) ? y : 0.f);
        s = fma2(d, d, s);
      }
    }
    const float var = row_sum<WPR>(pair_sum(add2(s, s1)), red[1]) * inv;
    const float rstd = rsqrtf(var + a.eps);
    const u64 rr = pair(rstd, rstd);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[i] = fma2(mul2(v[i], rr), w[i], b[i]);
    P::store(py, v, t, a.H);
    py += jump_y;
    if (t == 0 && a.mean) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
  cp_wait_all();
}

template <class T, bool VEC, int WPR, int E>
__global__ void __launch_bounds__(threads_of(WPR), WPR > 8 || !VEC ? 1 : E == 8 ? 3 : 2) k_ln_bwd(const NormArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float2 red[2][32];
  constexpr int tpr = 32 * WPR, per = threads_of(WPR) / tpr;
  const int g = threadIdx.x / tpr, t = threadIdx.x % tpr;
  using P = Piece<T, VEC, E, WPR>;
  using A = Ahead<T, VEC, E, WPR, 2>;
  pdl_wait();
  pdl_next();
  const long long step = (long long)gridDim.x * per, r0 = (long long)blockIdx.x * per + g;
  const long long jump_x = step * a.ldx, jump_y = step * a.ldy;
  A ahead;
  ahead.init(smem);
  const T *px = (const T*)a.x + r0 * a.ldx, *pd = (const T*)a.dy + r0 * a.lddy;
  const long long jump_d = step * a.lddy;
  long long rx = r0;
  auto fetch = [&]() {
    const T* const rows[2] = {px, pd};
    ahead.fetch(rows, t, a.H, rx < a.N);
    px += jump_x;
    pd += jump_d;
    rx += step;
  };
#pragma unroll
  for (int i = 0; i < A::kDepth; ++i) fetch();
  u64 w[E / 2], dw[E / 2], db[E / 2];
  load_params<P, E>(w, a.weight, a.ptype, t, a.H, 1.f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dw[i] = db[i] = 0;
  const float inv = 1.f / (float)a.H;
  const float *pm = a.mean + r0, *pr = a.rstd + r0;  // of the row after the one worked on
  float nmean = r0 < a.N ? *pm : 0.f, nrstd = r0 < a.N ? *pr : 0.f;
  int par = 0;
  T* py = (T*)a.y + r0 * a.ldy;
  for (long long r = r0; r < a.N; r += step) {
    u64 v[2][E / 2];
    ahead.take(v, t, a.H);
    u64(&xh)[E / 2] = v[0];
    u64(&d)[E / 2] = v[1];
    const u64 nm = pair(-nmean, -nmean), rr = pair(nrstd, nrstd);
    pm += step;
    pr += step;
    if (r + step < a.N) {
      nmean = *pm;
      nrstd = *pr;
    }
    fetch();
    u64 s0 = 0, s1 = 0;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      // a column past H has d = 0, so it adds nothing
      xh[i] = mul2(add2(xh[i], nm), rr);
      db[i] = add2(db[i], d[i]);
      dw[i] = fma2(d[i], xh[i], dw[i]);
      d[i] = mul2(d[i], w[i]);
      s0 = add2(s0, d[i]);
      s1 = fma2(d[i], xh[i], s1);
    }
    const float2 s = row_sum<WPR>(make_float2(pair_sum(s0), pair_sum(s1)), red[par]);
    par ^= 1;
    if (a.y) {
      const u64 m0 = pair(-s.x * inv, -s.x * inv), m1 = pair(-s.y * inv, -s.y * inv);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) d[i] = mul2(rr, fma2(xh[i], m1, add2(d[i], m0)));
      P::store(py, d, t, a.H);
      py += jump_y;
    }
  }
  cp_wait_all();
  if (!a.part) return;
  // the block's rows are dealt to its groups: their sums, in order (the ring's memory is free now)
  float* const col_sums = reinterpret_cast<float*>(smem);  // [2][H]
  __syncthreads();
  for (int k = 0; k < per; ++k) {
    if (g == k) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        float x[2], y[2];
        unpair(x[0], x[1], dw[i]);
        unpair(y[0], y[1], db[i]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = P::col(2 * i + e, t);
          if (c < a.H) {
            col_sums[c] = k ? col_sums[c] + x[e] : x[e];
            col_sums[a.H + c] = k ? col_sums[a.H + c] + y[e] : y[e];
          }
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * a.H; c += blockDim.x) a.part[(long long)blockIdx.x * 2 * a.H + c] = col_sums[c];
}

// dw and db: the blocks' sums, in order (32 slices of the blocks, all of a
// slice's loads in flight, then the slices).
__global__ void __launch_bounds__(1024) k_ln_cols(const float* __restrict__ part, int blocks, int H, int ptype, void* dw,
                                                  void* db) {
  constexpr int kEach = (kLnBlocks + 31) / 32;
  __shared__ float red[32][33];
  pdl_wait();
  pdl_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * H) {
    float p[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) p[k] = warp * kEach + k < blocks ? part[(long long)(warp * kEach + k) * 2 * H + c] : 0.f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) s += p[k];
  }
  red[warp][lane] = s;
  __syncthreads();
  s = red[lane][warp];  // a warp per column
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  const int cc = blockIdx.x * 32 + warp;
  if (lane == 0 && cc < 2 * H) {
    if (cc < H) {
      if (dw) store_elem(dw, ptype, cc, s);
    } else if (db) {
      store_elem(db, ptype, cc - H, s);
    }
  }
}

// Elements of a row a thread holds.  Forward, 32 where 16 would take a second
// warp and 32 do not: the sums then need no barrier (64000 rows of 1024: 48 us
// with 16, 42 with 32).  Backward its registers also hold the weights and both
// column sums: 8 let three blocks share an SM (76 us with 16, 69 with 8), as
// long as eight warps hold the row.
int per_thread(int H, bool vec, bool bwd) { return bwd ? (H <= 2048 ? 8 : 16) : vec && H > 512 && H <= 1024 ? 32 : 16; }

struct Shape {
  int wpr, threads, blocks;
};
Shape shape_of(long long N, int H, bool vec, bool bwd) {
  Shape s{1, 256, 0};
  const int each = per_thread(H, vec, bwd);
  while (s.wpr * 32 * each < H) s.wpr *= 2;
  s.threads = threads_of(s.wpr);
  const int per = s.threads / 32 / s.wpr, most = bwd && vec && each == 8 ? kLnBlocks : kLnBlocks / 3 * 2;
  const long long b = (N + per - 1) / per;
  s.blocks = (int)(b < most ? b : most);
  return s;
}

bool vec_ok(int type, const void* p, long long ld) {
  const int v = type == CTCPB_F32 ? 4 : 8;
  return ((uintptr_t)p & 15) == 0 && ld % v == 0;
}

template <class T, bool VEC, int WPR, int E>
cudaError_t run_fwd(const NormArgs& a, const Shape& s, cudaStream_t st) {
  constexpr auto kern = k_ln<T, VEC, WPR, E>;
  constexpr size_t smem = Ahead<T, VEC, E, WPR, 1>::bytes;
  cudaError_t e = smem_optin<kern>(smem);
  return e != cudaSuccess ? e : launch(kern, s.blocks, s.threads, smem, st, 1, a);
}
template <class T, bool VEC, int WPR, int E>
cudaError_t run_bwd(const NormArgs& a, const Shape& s, cudaStream_t st) {
  const size_t sums = a.part ? (size_t)2 * a.H * 4 : 0, ring = Ahead<T, VEC, E, WPR, 2>::bytes;
  const size_t smem = sums > ring ? sums : ring;
  constexpr auto kern = k_ln_bwd<T, VEC, WPR, E>;
  cudaError_t e = smem_optin<kern>(smem);
  return e != cudaSuccess ? e : launch(kern, s.blocks, s.threads, smem, st, 1, a);
}
template <class T, bool VEC, int WPR>
cudaError_t run_t(bool bwd, const NormArgs& a, const Shape& s, cudaStream_t st) {
  if (!bwd) {
    if constexpr (VEC && WPR == 1) {
      if (per_thread(a.H, true, false) == 32) return run_fwd<T, VEC, WPR, 32>(a, s, st);
    }
    return run_fwd<T, VEC, WPR, 16>(a, s, st);
  }
  if constexpr (WPR >= 8) {
    if (per_thread(a.H, VEC, true) == 16) return run_bwd<T, VEC, WPR, 16>(a, s, st);
  }
  if constexpr (WPR <= 8) return run_bwd<T, VEC, WPR, 8>(a, s, st);
  return cudaErrorInvalidValue;  // no width leads here
}
template <class T, bool VEC>
cudaError_t run_w(bool bwd, const NormArgs& a, const Shape& s, cudaStream_t st) {
  switch (s.wpr) {
    case 1: return run_t<T, VEC, 1>(bwd, a, s, st);
    case 2: return run_t<T, VEC, 2>(bwd, a, s, st);
    case 4: return run_t<T, VEC, 4>(bwd, a, s, st);
    case 8: return run_t<T, VEC, 8>(bwd, a, s, st);
    default: return run_t<T, VEC, 16>(bwd, a, s, st);
  }
}
template <class T>
cudaError_t run(bool bwd, bool vec, const NormArgs& a, const Shape& s, cudaStream_t st) {
  return vec ? run_w<T, true>(bwd, a, s, st) : run_w<T, false>(bwd, a, s, st);
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
  NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.ptype = param_type;
  a.eps = eps;
  a.N = N;
  a.H = H;
  const bool vec = H % (type == CTCPB_F32 ? 4 : 8) == 0 && vec_ok(type, x, ldx) && vec_ok(type, y, ldy);
  const Shape s = shape_of(N, H, vec, false);
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  return run(type, false, vec, a, s, (cudaStream_t)stream) == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
}

int ctcpb_layer_norm_workspace_size(int64_t N, int H, size_t* bytes) {
  int rc = check(CTCPB_F32, CTCPB_F32, N, H);
  if (rc) return rc;
  if (!bytes) return CTCPB_ENULL;
  const Shape s = shape_of(N, H, true, true);  // the most blocks of either kind
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
  const bool vec = H % (type == CTCPB_F32 ? 4 : 8) == 0 && vec_ok(type, x, ldx) && vec_ok(type, dy, lddy) &&
                   (!dx || vec_ok(type, dx, lddx));
  const Shape s = shape_of(N, H, vec, true);
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
      a.y = dx;
    a.ldy = lddx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = cols ? (float*)ws : nullptr;
    if (run(type, true, vec, a, s, st) != cudaSuccess) return CTCPB_ECUDA;
  }
  if (cols) {
    if (launch(k_ln_cols, (2 * H + 31) / 32, 1024, 0, st, 1, (const float*)ws, N > 0 ? s.blocks : 0, H, param_type, dweight,
               dbias) != cudaSuccess)
      return CTCPB_ECUDA;
  }
  return CTCPB_OK;
}

}  // extern "C"
