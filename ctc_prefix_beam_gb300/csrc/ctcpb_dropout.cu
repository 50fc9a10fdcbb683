// Dropout from a counter-based generator (ctcpb_dropout).
//
//   y = residual + x [u(i) >= k] 65536 / (65536 - k),   u(i) 16 bits of Philox4x32-10
//
// The mask is a function of the element's index, the seed and the offset, so the
// backward pass makes it again and nothing is stored.  A thread makes one block
// of the generator for the eight elements it moves: 16 bits an element, because
// 32 would make the generator's integer work longer than the memory's.  Bound by HBM
// with a residual (64000 x 1024 bfloat16: 56 us, 7.0 TB/s), without one about equally
// by the generator's multiplications (43 us, 6.1 TB/s).  What brought it there: keys in
// uniform registers, halves compared at the top of their words, and one address for rows
// that lie end to end (57 us before that one).
#include "ctcpb_head.cuh"

namespace ctcpb {
namespace {

constexpr int kDropThreads = 256;

struct DropArgs {
  const void* x;
  const void* res;
  void* y;
  long long ldx, ldr, ldy;
  long long n, H;       // elements, and of a row
  u32 bound;            // k at the top of a word
  int none;             // k is 65536: nothing is kept
  float scale;
  const long long* rng;
};

// The four words of block `ctr` of Philox4x32 with 10 rounds: in a round the
// outer words are multiplied, the products' high halves mixed with the inner
// words and the key, and the key moves on by a constant.
__device__ __forceinline__ uint4 philox(uint4 ctr, u32 k0, u32 k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const u64 a = (u64)ctr.x * 0xD2511F53u, b = (u64)ctr.z * 0xCD9E8D57u;
    ctr = make_uint4((u32)(b >> 32) ^ ctr.y ^ k0, (u32)b, (u32)(a >> 32) ^ ctr.w ^ k1, (u32)a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return ctr;
}

// The same in all threads of a warp, and known to be: it and what follows from it
// alone, the ten keys, is in uniform registers, made once.
__device__ __forceinline__ u32 uniform(u32 v) { return __reduce_or_sync(0xffffffffu, v); }
struct Draw {
  u32 k0, k1, o0, o1;
  __device__ __forceinline__ explicit Draw(const long long* rng) {
    const u64 seed = (u64)rng[0], off = (u64)rng[1];
    k0 = uniform((u32)seed);
    k1 = uniform((u32)(seed >> 32));
    o0 = uniform((u32)off);
    o1 = uniform((u32)(off >> 32));
  }
  __device__ __forceinline__ uint4 of(long long q) const {
    return philox(make_uint4((u32)q, (u32)((u64)q >> 32), o0, o1), k0, k1);
  }
};
// Whether element j of a block is kept: its half, at the top of a word, against the
// bound there.
__device__ __forceinline__ bool kept(const uint4& w, int j, u32 bound) {
  const u32 v = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return (j & 1 ? v : v * 65536u) >= bound;
}

// Eight elements as 16-byte vectors.
template <class T>
struct Oct {
  static constexpr int Q = sizeof(T) == 4 ? 2 : 1;
  uint4 q[Q];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < Q; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < Q; ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < Q; ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const u32 w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[Q - 1].x, q[Q - 1].y, q[Q - 1].z, q[Q - 1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else if (i % 2 == 0) {
        unpair(v[i], v[i + 1], Elem<T>::unpack(w[i / 2]));
      }
    }
  }
  __device__ __forceinline__ void put(const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
      q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      q[0] = make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]),
                        Elem<T>::pack(v[6], v[7]));
    }
  }
};

// Octet q, for any strides and alignment, or of fewer elements.
template <class T, bool RES>
__device__ __forceinline__ void drop_any(const DropArgs& a, const Draw& draw, long long q) {
  const uint4 w = draw.of(q);
  const long long i0 = q * 8;
  long long r = i0 < a.H ? 0 : i0 / a.H, c = i0 - r * a.H;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i0 + j < a.n) {
      float p = kept(w, j, a.bound) && !a.none ? Elem<T>::to(((const T*)a.x)[r * a.ldx + c]) * a.scale : 0.f;
      if (RES) p = Elem<T>::to(((const T*)a.res)[r * a.ldr + c]) + p;
      ((T*)a.y)[r * a.ldy + c] = Elem<T>::from(p);
      if (++c == a.H) {
        c = 0;
        ++r;
      }
    }
  }
}
// Octets on 16-byte boundaries: FLAT: one after the other; else in rows of whole ones.
// A thread takes U of them, so far apart that a warp's are together.
template <class T, bool RES, bool FLAT, int U, int MINB>
__global__ void __launch_bounds__(kDropThreads, MINB) k_dropout(const DropArgs a) {
  pdl_wait();
  pdl_next();
  const Draw draw(a.rng);
  const long long octs = a.n / 8, step = (long long)gridDim.x * (U * kDropThreads);
  for (long long q0 = (long long)blockIdx.x * (U * kDropThreads) + threadIdx.x; q0 < octs; q0 += step) {
    Oct<T> x[U], res[RES ? U : 1];
    T* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long q = q0 + u * kDropThreads;
      if (U > 1 && q >= octs) break;
      const long long i = q * 8, r = FLAT || i < a.H ? 0 : i / a.H, c = i - r * a.H;
      x[u].load((const T*)a.x + (FLAT ? i : r * a.ldx + c));
      if constexpr (RES) res[u].load((const T*)a.res + (FLAT ? i : r * a.ldr + c));
      to[u] = (T*)a.y + (FLAT ? i : r * a.ldy + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long q = q0 + u * kDropThreads;
      if (U > 1 && q >= octs) break;
      const uint4 w = draw.of(q);
      if (a.none) x[u].clear();
      float v[8], s[8];
      x[u].get(v);
      if constexpr (RES) res[u].get(s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = kept(w, j, a.bound) ? v[j] * a.scale : 0.f;
        if constexpr (RES) v[j] = s[j] + v[j];
      }
      x[u].put(v);
      x[u].store(to[u]);
    }
  }
  if (a.n % 8 && blockIdx.x == 0 && threadIdx.x == 0) drop_any<T, RES>(a, draw, octs);
}

template <class T, bool RES>
__global__ void __launch_bounds__(kDropThreads) k_dropout_any(const DropArgs a) {
  pdl_wait();
  pdl_next();
  const Draw draw(a.rng);
  const long long octs = (a.n + 7) / 8;
  for (long long q = (long long)blockIdx.x * kDropThreads + threadIdx.x; q < octs; q += (long long)gridDim.x * kDropThreads)
    drop_any<T, RES>(a, draw, q);
}

template <class T, bool RES>
cudaError_t run_drop(const DropArgs& a, bool vec, cudaStream_t s) {
  const long long b = (a.n + 8 * kDropThreads - 1) / (8 * kDropThreads), most = 152 * 64;
  const int grid = (int)(b < most ? b : most);
  if (!vec) return launch(k_dropout_any<T, RES>, grid, kDropThreads, 0, s, 1, a);
  // Two octets a thread where an octet is one load and store (65.5 M elements: 43 us, 47 with one); with
  // a residual or float32 the loads are twice as many already (56 us; float32 14 and 18 us for 8.2 M).
  constexpr int U = RES || sizeof(T) == 4 ? 1 : 2, MINB = U == 1 ? 8 : 6;
  return a.H == a.n ? launch(k_dropout<T, RES, true, U, MINB>, grid, kDropThreads, 0, s, 1, a)
                    : launch(k_dropout<T, RES, false, U, MINB>, grid, kDropThreads, 0, s, 1, a);
}
template <class T>
cudaError_t run_drop(const DropArgs& a, bool vec, cudaStream_t s) {
  return a.res ? run_drop<T, true>(a, vec, s) : run_drop<T, false>(a, vec, s);
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" int ctcpb_dropout(int type, const void* x, int64_t ldx, const void* residual, int64_t ldr, double p,
                             const int64_t* rng, int64_t N, int H, void* y, int64_t ldy, ctcpb_stream_t stream) {
  if (type != CTCPB_F32 && type != CTCPB_BF16 && type != CTCPB_F16) return CTCPB_EINVAL;
  if (N < 0 || N > kHeadMaxRows || H < 1 || H > kHeadMaxWidth || !(p >= 0. && p <= 1.)) return CTCPB_EINVAL;
  if (N == 0) return CTCPB_OK;
  if (ldx < H || ldy < H || (residual && ldr < H)) return CTCPB_EINVAL;
  if (!x || !y || !rng) return CTCPB_ENULL;
  DropArgs a{};
  a.x = x;
  a.res = residual;
  a.y = y;
  a.n = N * H;
  const bool flat = N == 1 || (ldx == H && ldy == H && (!residual || ldr == H));
  a.H = flat ? a.n : H;  // rows end to end are one
  a.ldx = ldx;
  a.ldr = residual ? ldr : H;
  a.ldy = ldy;
  const u32 k = (u32)__builtin_llrint(p * 65536.);
  a.none = k >= 65536u;
  a.bound = a.none ? 0u : k << 16;
  a.scale = a.none ? 0.f : (float)(65536. / (65536. - k));
  a.rng = (const long long*)rng;
  const int e = type == CTCPB_F32 ? 4 : 2;
  const bool aligned = (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)y) & 15u) == 0;
  const bool octs = H % 8 == 0 && ((ldx | a.ldr | ldy) * e) % 16 == 0;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t err = type == CTCPB_F32    ? run_drop<float>(a, aligned && (flat || octs), s)
                    : type == CTCPB_BF16 ? run_drop<__nv_bfloat16>(a, aligned && (flat || octs), s)
                                         : run_drop<__half>(a, aligned && (flat || octs), s);
  return err == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
}
