// Dropout from a counter-based generator (ctcpb_dropout).
//
//   y = residual + x [u(i) >= k] 65536 / (65536 - k),   u(i) 16 bits of Philox4x32-10
//
// The mask is a function of the element's index, the seed and the offset, so the
// backward pass makes it again and nothing is stored.  A thread makes one block
// of the generator for the eight elements it moves: 16 bits an element, because
// 32 would make the generator's integer work as long as the memory's.
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
  u32 cut;
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

struct Draw {
  u32 k0, k1, o0, o1;
  __device__ __forceinline__ explicit Draw(const long long* rng) {
    const u64 seed = (u64)rng[0], off = (u64)rng[1];
    k0 = (u32)seed;
    k1 = (u32)(seed >> 32);
    o0 = (u32)off;
    o1 = (u32)(off >> 32);
  }
  __device__ __forceinline__ uint4 of(long long q) const {
    return philox(make_uint4((u32)q, (u32)((u64)q >> 32), o0, o1), k0, k1);
  }
};
__device__ __forceinline__ u32 half_of(const uint4& w, int j) {
  const u32 v = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return j & 1 ? v >> 16 : v & 0xffffu;
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

// VEC: rows end to end (or of whole octets), all on 16-byte boundaries.
template <class T, bool VEC, bool RES>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const DropArgs a) {
  pdl_wait();
  pdl_next();
  const Draw draw(a.rng);
  const long long octs = (a.n + 7) / 8;
  for (long long q = (long long)blockIdx.x * kDropThreads + threadIdx.x; q < octs; q += (long long)gridDim.x * kDropThreads) {
    const long long i0 = q * 8;
    const long long r = i0 < a.H ? 0 : i0 / a.H, c = i0 - r * a.H;
    if (VEC && i0 + 8 <= a.n) {
      Oct<T> x, res;
      x.load((const T*)a.x + r * a.ldx + c);
      if (RES) res.load((const T*)a.res + r * a.ldr + c);
      const uint4 w = draw.of(q);
      float v[8], s[8];
      x.get(v);
      if (RES) res.get(s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = half_of(w, j) >= a.cut ? v[j] * a.scale : 0.f;
        v[j] = RES ? s[j] + p : p;
      }
      x.put(v);
      x.store((T*)a.y + r * a.ldy + c);
      continue;
    }
    const uint4 w = draw.of(q);
    long long rr = r, cc = c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j < a.n) {
        float p = half_of(w, j) >= a.cut ? Elem<T>::to(((const T*)a.x)[rr * a.ldx + cc]) * a.scale : 0.f;
        if (RES) p = Elem<T>::to(((const T*)a.res)[rr * a.ldr + cc]) + p;
        ((T*)a.y)[rr * a.ldy + cc] = Elem<T>::from(p);
        if (++cc == a.H) {
          cc = 0;
          ++rr;
        }
      }
    }
  }
}

template <class T>
cudaError_t run_drop(const DropArgs& a, bool vec, cudaStream_t s) {
  const long long blocks = (a.n + 8 * kDropThreads - 1) / (8 * kDropThreads), most = 152 * 64;
  const int grid = (int)(blocks < most ? blocks : most);
  if (vec) return a.res ? launch(k_dropout<T, true, true>, grid, kDropThreads, 0, s, 1, a)
                        : launch(k_dropout<T, true, false>, grid, kDropThreads, 0, s, 1, a);
  return a.res ? launch(k_dropout<T, false, true>, grid, kDropThreads, 0, s, 1, a)
               : launch(k_dropout<T, false, false>, grid, kDropThreads, 0, s, 1, a);
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
  a.cut = (u32)__builtin_llrint(p * 65536.);
  a.scale = a.cut < 65536u ? (float)(65536. / (65536. - a.cut)) : 0.f;
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
