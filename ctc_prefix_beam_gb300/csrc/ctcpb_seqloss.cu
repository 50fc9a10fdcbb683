// Losses of the decoder's own N-best lists, with their gradients: the clipped
// policy loss with a KL term, and the preference loss of pairs
// (ctcpb_policy_loss, ctcpb_preference_loss).
//
//   d = old - nll, ratio = e^d, u = nll - ref
//   token loss = -(A + A q) + kl (e^u - 1 - u),  q = e^d - 1, held at the border's
//   R = sum (ref - nll),  z = beta (R_c - R_r) - margin,  log(1 + e^-z)
//
// Each input is read once, the gradient written in the same pass.  The gradient's
// factor needs the number of tokens, sequences or pairs first: every block counts
// the lengths (or pairs) itself, up to kCountHere of them, else a launch before does.
// Small calls are one launch of one cluster, whose blocks add up their sums through
// shared memory; larger ones leave them to a launch after, which starts meanwhile.
//
// 4096 sequences of up to 1024 tokens (3.1 M), with a reference and an advantage each:
// 23 us, bound by instructions (170 a token, two exponentials and the sums' errors; HBM
// would take 10); 1024 lists of 4 x 1000 tokens 10 us (HBM 4.4; a block's chain: the
// pair, its lengths, its rows, the gradient).
//
// A list's advantages sum to about nothing, so the policy loss is a small rest of
// large terms: A and A q are added apart, as pairs of float32 (value and error), and
// e^x - 1 comes without its cancellation.  So are the sums R, whose difference counts.
// (Pairs of float32, not float64: this machine has two float64 lanes an SM for 128 of
// float32, and one conversion and addition a token would take as long as its memory.)
#include <cmath>

#include "ctcpb_head.cuh"

namespace ctcpb {
namespace {

constexpr int kLossThreads = 256;  // of a block of the policy loss
constexpr int kPairThreads = 128;  // ... of the preference loss
constexpr int kLossBlocks = 152 * 8;
constexpr int kWarpList = 256;     // tokens up to which a list is a warp's, not a block's
constexpr int kOneBlocks = 8;      // of a call that is one cluster
constexpr int kCountHere = 8192;   // lengths or pairs that every block counts itself
constexpr int kCountBlocks = 128;  // blocks of the launch that counts more
constexpr long long kMaxSeqs = 1 << 24, kMaxTokens = 1 << 24, kMaxCall = (1ll << 32) - 1;

// What a call's lengths or pairs come to.
struct Ctl {
  long long items;  // tokens, or pairs
  double factor;    // of the sum of the losses (means: 1 over how many)
  float grad;       // of the gradients: the loss's, times the factor (REDUCE_NONE: 1)
  u32 bad;          // an index past the end
};
struct LossLayout {
  size_t o_ctl, o_counts, o_part, total;
};
LossLayout loss_layout() {
  LossLayout l{};
  l.o_ctl = sizeof(Header);
  l.o_counts = l.o_ctl + 256;
  l.o_part = l.o_counts + kCountBlocks * sizeof(longlong2);
  l.total = align_up(l.o_part + (size_t)kLossBlocks * 3 * sizeof(float2), 256);
  return l;
}

// x / d for any x < 2^32 (Granlund and Montgomery: a multiplication by the
// divisor's reciprocal to 33 bits).
struct Divisor {
  u32 d, m, s1, s2;
  explicit Divisor(u32 d_ = 1) : d(d_) {
    int l = 0;
    while ((1ull << l) < d) ++l;
    m = (u32)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    s1 = l < 1 ? l : 1;
    s2 = l > 1 ? l - 1 : 0;
  }
  __device__ __forceinline__ u32 operator()(u32 x) const {
    const u32 t = __umulhi(m, x);
    return (t + ((x - t) >> s1)) >> s2;
  }
};

// A sum as value and error: what each addition rounds off is kept.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float s = hi + v, t = s - hi;
    lo += (hi - (s - t)) + (v - t);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum2& v) {
    add(v.hi);
    lo += v.lo;
  }
  // times a factor given as value and error
  __device__ __forceinline__ Sum2 times(float f, float f_lo) const {
    Sum2 r;
    r.hi = hi * f;
    r.lo = fmaf(hi, f, -r.hi) + fmaf(lo, f, hi * f_lo);
    return r;
  }
  // an infinite sum's error is not a number
  __device__ __forceinline__ double value() const { return isfinite(hi) ? (double)hi + (double)lo : (double)hi; }
  __device__ __forceinline__ Sum2 other(int lane_mask) const {
    Sum2 r;
    r.hi = __shfl_xor_sync(0xffffffffu, hi, lane_mask);
    r.lo = __shfl_xor_sync(0xffffffffu, lo, lane_mask);
    return r;
  }
  __device__ __forceinline__ void warp_sum() {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) add(other(s));
  }
};
// Two such sums side by side.
struct Sum2x2 {
  u64 hi = 0, lo = 0;
  __device__ __forceinline__ void add(u64 v) {
    const u64 minus = pair(-1.f, -1.f), s = add2(hi, v), t = fma2(hi, minus, s);  // (products by -1 are exact)
    lo = add2(lo, add2(fma2(fma2(t, minus, s), minus, hi), fma2(t, minus, v)));
    hi = s;
  }
  __device__ __forceinline__ void into(Sum2& s) const {
    Sum2 a, b;
    unpair(a.hi, b.hi, hi);
    unpair(a.lo, b.lo, lo);
    s.add(a);
    s.add(b);
  }
};
// a - b as value and error
__device__ __forceinline__ void add_difference(Sum2& s, float a, float b) {
  const float d = a - b, t = d - a;
  s.add(d);
  s.lo += (a - (d - t)) - (b + t);
}

// e^x - 1 and e^x - 1 - x.  With n the integer next to x / ln 2 and r = x - n ln 2 (in
// two steps, Cody and Waite), e^x = 2^n (1 + r + c), c = r^2 (1/2! + r/3! + ...) by its
// Taylor series (the first term left out is 9e-8 of c at most, at |r| = ln 2 / 2).  Next
// to 0, where n = 0, nothing cancels: e^x - 1 - x is c.  Above 88.37 the exponential is
// infinite.  (One value at a time: the constants are immediates then.  In pairs they
// would take two registers each, and were loaded again for every token.)
struct ExpLess {
  float x, r, c, s, less;
  __device__ __forceinline__ explicit ExpLess(float v) {
    x = v > 88.37f ? 89.f : v;
    float y;  // (NaN stays NaN)
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-87.f));
    const float t = fmaf(y, 1.4426950408889634f, 12582912.f), n = t - 12582912.f;  // n is in t's lowest bits
    r = fmaf(n, 2.12194440e-4f, fmaf(n, -0.693359375f, y));
    c = fmaf(1.f / 5040.f, r, 1.f / 720.f);
    c = fmaf(c, r, 1.f / 120.f);
    c = fmaf(c, r, 1.f / 24.f);
    c = fmaf(c, r, 1.f / 6.f);
    c = fmaf(c, r, 0.5f);
    c = c * (r * r);
    s = __int_as_float((__float_as_int(t) << 23) + 0x3f800000);
    less = s - 1.f;
  }
  __device__ __forceinline__ float one() const { return fmaf(s, r + c, less); }
  __device__ __forceinline__ float two() const { return fmaf(s, c, fmaf(s, r, less) - x); }
};

__device__ __forceinline__ long long length_of(const int* lengths, long long s, long long L) {
  if (!lengths) return L;
  const long long n = lengths[s];
  return n < 0 ? 0 : n > L ? L : n;
}

// A list's pair: (chosen, rejected), or false where it takes no part.
__device__ __forceinline__ bool pair_of(const int* chosen, const int* rejected, long long b, int N, int& c, int& r) {
  c = chosen[b];
  r = rejected[b];
  return c >= 0 && r >= 0 && c < N && r < N;
}

// ---------------------------------------------------------------- counts

// What a call counts: tokens and sequences that have some, or pairs.
struct Counted {
  const int *lengths, *chosen, *rejected;
  long long n, L;  // lengths, or lists
  int N, reduction;
  const float* grad;
  const longlong2* counts;  // ... or what the blocks of a launch before counted of them
};
// A block's count, of every `step`-th from `first` on for its first thread; thread 0 has it.
__device__ __forceinline__ longlong2 count(const Counted& a, long long first, long long step, long long (*red)[2]) {
  long long v[2] = {0, 0};
#pragma unroll 8
  for (long long i = first + threadIdx.x; i < (a.counts ? kCountBlocks : a.n); i += step) {
    if (a.counts) {
      v[0] += a.counts[i].x;
      v[1] += a.counts[i].y;
    } else if (a.chosen) {
      int c, r;
      v[0] += pair_of(a.chosen, a.rejected, i, a.N, c, r);
      v[1] += c >= a.N || r >= a.N;
    } else {
      const long long l = length_of(a.lengths, i, a.L);
      v[0] += l;
      v[1] += l > 0;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], s);
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5][0] = v[0];
    red[threadIdx.x >> 5][1] = v[1];
  }
  __syncthreads();
  v[0] = v[1] = 0;
  if (threadIdx.x == 0)
    for (u32 w = 0; w < blockDim.x >> 5; ++w) {
      v[0] += red[w][0];
      v[1] += red[w][1];
    }
  return make_longlong2(v[0], v[1]);
}
__device__ __forceinline__ Ctl ctl_of(const Counted& a, const longlong2& v) {
  const bool mean = a.reduction == CTCPB_REDUCE_MEAN || a.reduction == CTCPB_REDUCE_SEQUENCE_MEAN;
  const double of = (double)(a.reduction == CTCPB_REDUCE_SEQUENCE_MEAN ? v.y : v.x);
  Ctl c;
  c.items = v.x;
  c.factor = mean ? 1. / of : 1.;
  c.grad = a.reduction == CTCPB_REDUCE_NONE || !a.grad ? 1.f : mean ? (float)((double)*a.grad / of) : *a.grad;
  c.bad = a.chosen && v.y ? 1u : 0u;
  return c;
}
__global__ void __launch_bounds__(1024) k_count(const Counted a, longlong2* counts) {
  __shared__ long long red[32][2];
  pdl_wait();
  pdl_next();
  const longlong2 v = count(a, (long long)blockIdx.x * blockDim.x, (long long)gridDim.x * blockDim.x, red);
  if (threadIdx.x == 0) counts[blockIdx.x] = v;
}

// ---------------------------------------------------------------- the end of a call

// How a launch's blocks come by the counts and leave their sums.
struct Ends {
  Counted counted;
  int one;        // the launch is one cluster (else sums go to part, for k_loss_end)
  Ctl* ctl;
  float2* part;   // [blocks][3]
  u32* status;    // (may be null in a call of one cluster)
  float *loss, *stats;
};
struct Shared {
  long long count[32][2];
  float2 warp[32][3];
  float2 block[3];
  Ctl ctl;
};
__device__ __forceinline__ void begin(const Ends& a, Shared& sh) {
  const longlong2 v = count(a.counted, 0, blockDim.x, sh.count);
  if (threadIdx.x == 0) {
    sh.ctl = ctl_of(a.counted, v);
    if (blockIdx.x == 0 && !a.one) *a.ctl = sh.ctl;  // for the launch after
  }
  if (threadIdx.x == 0 && blockIdx.x == 0 && a.status) *a.status = sh.ctl.bad ? CTCPB_DEV_TARGET : 0u;
  __syncthreads();
}
// A block's sums, in a fixed order (in sh.block once a barrier has passed).
template <int N>
__device__ __forceinline__ void block_sums(Sum2 (&v)[N], Shared& sh) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i].warp_sum();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sh.warp[warp][i] = make_float2(v[i].hi, v[i].lo);
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Sum2 s;
      if (lane < (int)(blockDim.x >> 5)) {
        s.hi = sh.warp[lane][i].x;
        s.lo = sh.warp[lane][i].y;
      }
      s.warp_sum();
      if (lane == 0) sh.block[i] = make_float2(s.hi, s.lo);
    }
  }
}
// The results.  Over no tokens or pairs a mean's factor is infinite: not a number.
__device__ __forceinline__ void results(const Ends& a, const Ctl& ctl, const Sum2 (&s)[3]) {
  if (a.loss) *a.loss = (float)(s[0].value() * ctl.factor);
  if (a.stats) {
    a.stats[0] = (float)(s[1].value() / (double)ctl.items);
    a.stats[1] = (float)(s[2].value() / (double)ctl.items);
  }
}
template <int N>
__device__ __forceinline__ void end(const Ends& a, Sum2 (&v)[N], Shared& sh) {
  block_sums<N>(v, sh);
  if (!a.one) {
    if (threadIdx.x == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) a.part[(size_t)blockIdx.x * 3 + i] = sh.block[i];
    return;
  }
  __syncwarp();  // the barrier takes whole warps
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    Sum2 s[3];
    for (u32 r = 0; r < gridDim.x; ++r)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Sum2 q;
        const u32 at = cluster_addr(saddr(&sh.block[i]), r);
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(q.hi), "=f"(q.lo) : "r"(at) : "memory");
        s[i].add(q);
      }
    results(a, sh.ctl, s);
  }
  __syncwarp();
  cluster_sync();  // no block leaves before its sums are read
}
// The blocks' sums, in order.
template <int N>
__global__ void __launch_bounds__(256) k_loss_end(const Ends a, int blocks) {
  __shared__ Shared sh;
  pdl_wait();
  pdl_next();
  Sum2 v[3];
  for (int b = threadIdx.x; b < blocks; b += blockDim.x)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 p = a.part[(size_t)b * 3 + i];
      Sum2 q;
      q.hi = p.x;
      q.lo = p.y;
      v[i].add(q);
    }
  block_sums<3>(v, sh);
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i].hi = sh.block[i].x;
    v[i].lo = sh.block[i].y;
  }
  results(a, *a.ctl, v);
}

// ---------------------------------------------------------------- the policy loss

struct PolicyArgs {
  const float *nll, *old, *ref, *adv;
  long long ld_nll, ld_old, ld_ref, ld_adv;
  const int* lengths;
  long long S, L;
  double high, low;  // borders of d: log(1 + clip_high), log(1 - clip_low)
  float fhigh, flow, qhigh, qlow;
  float kl;
  int reduction;
  const float* grad;
  float *loss, *dnll;  // the loss of each token (REDUCE_NONE)
  Divisor pieces;      // vectors of a row
  int dense;           // the rows of all inputs lie end to end
  u32 work;            // vectors of all rows
  Ends ends;
};

// One token.  A ratio past the border is held there and counts no more.  Returns the
// loss but for its -A.
__device__ __forceinline__ float token(const PolicyArgs& a, float nll, float old, float ref, float A, float& kl, float& held,
                                       float& slope) {
  const float d = old - nll;
  float q = ExpLess(d).one();
  const bool up = A > 0.f;
  const float side = __int_as_float(__float_as_int(d) ^ (__float_as_int(A) & 0x80000000)) - (up ? a.fhigh : -a.flow);
  bool hold = side > 0.f && A != 0.f;
  // d is rounded, which keeps its order with a rounded border: only where the two
  // are equal does it take the exact difference
  if (side == 0.f && A != 0.f) {
    const double exact = (double)old - (double)nll;
    hold = up ? exact > a.high : exact < a.low;
  }
  if (A == 0.f) q = 0.f;  // a token without an advantage adds nothing, whatever its ratio overflows to
  slope = hold ? 0.f : fmaf(A, q, A);
  if (hold) q = up ? a.qhigh : a.qlow;
  float rest = -A * q;
  if (a.ref) {
    const ExpLess e(nll - ref);
    const float k = e.two();
    kl += k;
    rest = fmaf(a.kl, k, rest);
    slope = fmaf(a.kl, e.one(), slope);
  }
  held += hold ? 1.f : 0.f;
  return rest;
}

// A thread's tokens: four of a row, or one.
template <int V>
struct Tokens {
  float nll[V], old[V], ref[V], adv[V], up[V];
  static __device__ __forceinline__ void get(float (&v)[V], const float* p) {
    if constexpr (V == 4) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      v[0] = __ldcs(p);
    }
  }
  // (a vector may reach behind the length, not behind the row)
  __device__ __forceinline__ void load(const PolicyArgs& a, bool none, u64 x, u32 s, u32 t) {
    const u64 flat = x * V;  // rows end to end
    get(nll, a.nll + (a.dense ? flat : s * a.ld_nll + t));
    get(old, a.old + (a.dense ? flat : s * a.ld_old + t));
    if (a.ref) get(ref, a.ref + (a.dense ? flat : s * a.ld_ref + t));
    if (a.ld_adv)
      get(adv, a.adv + (a.dense ? flat : s * a.ld_adv + t));
    else
      adv[0] = a.adv[s];
    if (none && a.grad) get(up, a.grad + flat);
  }
};
// Where a thread's tokens are: the row, the first, how many of its length.
struct At {
  u32 s, t, len;
  __device__ __forceinline__ void set(const PolicyArgs& a, u64 x, int V) {
    len = t = s = 0;
    if (x < a.work) {
      s = a.pieces((u32)x);
      t = ((u32)x - s * a.pieces.d) * V;
      const int n = a.lengths ? a.lengths[s] : (int)a.L;
      len = n < 0 ? 0 : n < (int)a.L ? n : (u32)a.L;
    }
  }
  __device__ __forceinline__ int live(int V) const { return len <= t ? 0 : len - t >= (u32)V ? V : (int)(len - t); }
};

template <bool VEC>
__global__ void __launch_bounds__(kLossThreads, 3) k_policy(const PolicyArgs a) {
  __shared__ Shared sh;
  constexpr int V = VEC ? 4 : 1;
  pdl_wait();
  pdl_next();
  const bool none = a.reduction == CTCPB_REDUCE_NONE, by_len = a.reduction == CTCPB_REDUCE_SEQUENCE_MEAN;
  // the next tokens are on their way while these are worked on, the lengths after them too
  const u64 step = (u64)gridDim.x * kLossThreads;
  u64 x = (u64)blockIdx.x * kLossThreads + threadIdx.x;
  At at, next;
  Tokens<V> ahead;
  at.set(a, x, V);
  if (at.live(V)) ahead.load(a, none, x, at.s, at.t);
  next.set(a, x + step, V);
  begin(a.ends, sh);
  const float g = sh.ctl.grad;
  Sum2 sums[3];
  float held = 0.f;  // (whole numbers below 2^24)
  for (; x < a.work; x += step) {
    Tokens<V> k = ahead;
    const At now = at;
    at = next;
    if (at.live(V)) ahead.load(a, none, x + step, at.s, at.t);
    next.set(a, x + 2 * step, V);
    const int live = now.live(V);
    float slope[V], each[V];
    if (live) {
      if (!a.ld_adv) {
#pragma unroll
        for (int i = 1; i < V; ++i) k.adv[i] = k.adv[0];
      }
      if (V > 1 && live < V) {  // a token that is not there has no advantage, and the same score three times
#pragma unroll
        for (int i = 1; i < V; ++i)
          if (i >= live) k.nll[i] = k.old[i] = k.ref[i] = k.adv[i] = 0.f;
      }
      // 1 / len, and what its rounding took off (len <= 2^24 is exact)
      const float len = (float)now.len, wt = by_len ? 1.f / len : 1.f;
      const float gw = g * wt;
      float more = 0.f, kl = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float rest = token(a, k.nll[i], k.old[i], k.ref[i], k.adv[i], kl, held, slope[i]);
        more += rest;
        each[i] = rest - k.adv[i];
        slope[i] *= none ? (a.grad && i < live ? k.up[i] : 1.f) : gw;
      }
      if (V > 1 && live < V) {
#pragma unroll
        for (int i = 1; i < V; ++i)
          if (i >= live) slope[i] = each[i] = 0.f;
      }
      Sum2 loss;
      loss.hi = more;
      sums[1].add(kl);
      if constexpr (V == 4) {
        Sum2x2 advs;
        advs.hi = pair(-k.adv[0], -k.adv[1]);
        advs.add(pair(-k.adv[2], -k.adv[3]));
        advs.into(loss);
      } else {
        loss.add(-k.adv[0]);
      }
      sums[0].add(by_len ? loss.times(wt, fmaf(-wt, len, 1.f) * wt) : loss);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) slope[i] = each[i] = 0.f;
    }
    const u64 o = x * V;
    if constexpr (VEC) {
      if (a.dnll) __stcs(reinterpret_cast<float4*>(a.dnll + o), make_float4(slope[0], slope[1], slope[2], slope[3]));
      if (a.loss) __stcs(reinterpret_cast<float4*>(a.loss + o), make_float4(each[0], each[1], each[2], each[3]));
    } else {
      if (a.dnll) a.dnll[o] = slope[0];
      if (a.loss) a.loss[o] = each[0];
    }
  }
  sums[2].add(held);
  end<3>(a.ends, sums, sh);
}

// ---------------------------------------------------------------- the preference loss

struct PairArgs {
  const float *nll, *ref;
  long long ld_nll, ld_ref;
  const int *chosen, *rejected, *lengths;
  long long B, L;
  int N;
  float beta, margin, smooth;
  int average, reduction;
  const float* grad;
  float *loss, *margins, *dnll;  // the loss of each list (REDUCE_NONE)
  Ends ends;
};

// A row's values from `from` on: v in the first `len`, 0 behind.
template <bool VEC, int GT>
__device__ __forceinline__ void write_row(float* row, long long L, long long len, float v, int t0) {
  constexpr int V = VEC ? 4 : 1;
  for (long long t = (long long)t0 * V; t < L; t += GT * V) {
    if constexpr (VEC)
      __stcs(reinterpret_cast<float4*>(row + t),
             make_float4(t < len ? v : 0.f, t + 1 < len ? v : 0.f, t + 2 < len ? v : 0.f, t + 3 < len ? v : 0.f));
    else
      row[t] = t < len ? v : 0.f;
  }
}

// A list is worked on by GT threads (a warp, or the block): both rows' sums, the
// pair's loss, then the two rows' gradients; the other rows' zeros while the sums'
// values are on their way.
// (Eight blocks an SM: 1024 lists are one wave, 12.7 us; with 80 registers a thread 16.6.)
template <bool VEC, int GT>
__global__ void __launch_bounds__(kPairThreads, 8) k_preference(const PairArgs a) {
  __shared__ Shared sh;
  __shared__ float2 rowsum[2][GT / 32];
  __shared__ float slopes[kPairThreads / GT];
  constexpr int V = VEC ? 4 : 1, per = kPairThreads / GT, U = 4;
  pdl_wait();
  pdl_next();
  begin(a.ends, sh);
  const int t0 = threadIdx.x % GT, g = threadIdx.x / GT;
  const bool none = a.reduction == CTCPB_REDUCE_NONE;
  const float scale = sh.ctl.grad * a.beta;
  Sum2 sums[1];
  const long long groups = (a.B + per - 1) / per;
  for (long long w = blockIdx.x; w < groups; w += gridDim.x) {
    const long long b = w * per + g;
    if (b >= a.B) continue;  // (a whole warp; never a part of the block where it meets)
    int c, r;
    const bool pair = pair_of(a.chosen, a.rejected, b, a.N, c, r), both = pair && c != r;
    const long long lc = pair ? length_of(a.lengths, b * a.N + c, a.L) : 0;
    const long long lr = pair ? length_of(a.lengths, b * a.N + r, a.L) : 0;
    float* const out = a.dnll ? a.dnll + b * a.N * a.L : nullptr;
    if (out) {
#pragma unroll 1
      for (int n = 0; n < a.N; ++n)
        if (!both || (n != c && n != r)) write_row<VEC, GT>(out + n * a.L, a.L, 0, 0.f, t0);
    }
    Sum2 R[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long row = b * a.N + (k ? r : c), len = both ? (k ? lr : lc) : 0;
      const float *const pn = a.nll + row * a.ld_nll, *const pf = a.ref + row * a.ld_ref;
      for (long long t = (long long)t0 * V; t < len; t += U * GT * V) {
        float n[U][V], f[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const long long at = t + i * GT * V;
#pragma unroll
          for (int j = 0; j < V; ++j) f[i][j] = 0.f;
          if (at < len) {
            Tokens<V>::get(n[i], pn + at);
            if (a.ref) Tokens<V>::get(f[i], pf + at);
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (t + i * GT * V + j < len) add_difference(R[k], f[i][j], n[i][j]);
      }
      R[k].warp_sum();
    }
    if constexpr (GT > 32) {
      if ((threadIdx.x & 31) == 0) {
        rowsum[0][threadIdx.x >> 5] = make_float2(R[0].hi, R[0].lo);
        rowsum[1][threadIdx.x >> 5] = make_float2(R[1].hi, R[1].lo);
      }
      __syncthreads();
    }
    if (t0 == 0) {
      double z = 0.;
      if (both) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (GT > 32) {
            R[k] = Sum2();
            for (int i = 0; i < GT / 32; ++i) {
              Sum2 q;
              q.hi = rowsum[k][i].x;
              q.lo = rowsum[k][i].y;
              R[k].add(q);
            }
          }
        }
        double p = R[0].value(), q = R[1].value();
        if (a.average) {
          p /= lc > 0 ? (double)lc : 1.;
          q /= lr > 0 ? (double)lr : 1.;
        }
        z = (double)a.beta * (p - q);
      }
      const float m = pair ? (float)(z - (double)a.margin) : 0.f;
      const float e = expf(-fabsf(m)), tail = log1pf(e);
      const float up = (m >= 0.f ? 1.f : e) / (1.f + e), dn = (m >= 0.f ? e : 1.f) / (1.f + e);  // of m and -m
      const float loss = pair ? (1.f - a.smooth) * (fmaxf(-m, 0.f) + tail) + a.smooth * (fmaxf(m, 0.f) + tail) : 0.f;
      if (a.loss) a.loss[b] = loss;
      if (a.margins) a.margins[b] = m;
      sums[0].add(loss);
      slopes[g] = a.smooth * up - (1.f - a.smooth) * dn;
    }
    if constexpr (GT > 32)
      __syncthreads();
    else
      __syncwarp();
    if (out && both) {
      const float dz = slopes[g] * (none ? a.beta * a.grad[b] : scale);
      write_row<VEC, GT>(out + c * a.L, a.L, lc, -dz / (a.average && lc > 0 ? (float)lc : 1.f), t0);
      write_row<VEC, GT>(out + r * a.L, a.L, lr, dz / (a.average && lr > 0 ? (float)lr : 1.f), t0);
    }
    // (the next list's first meeting comes after its sums, so slopes may be written again then)
    if constexpr (GT == 32) __syncwarp();
  }
  end<1>(a.ends, sums, sh);
}

bool on16(const void* p, long long ld) { return ((uintptr_t)p & 15u) == 0 && ld % 4 == 0; }

// Small calls are one cluster, where its blocks are not much longer at them than a
// second launch is (3 us of the host's): 320 x 40 tokens 8.4 us on the GPU, in two
// launches 7.6; 320 x 200 are 13.9 and 8.1.  Lists: 32 x 10 x 40 7.5 and 8.2, 64 x 10 x
// 40 11.2 and 7.8; of more tokens, a block each: 8 x 4 x 1000 6.9 and 7.5, 16: 9.9 and 7.2.
bool one_policy(long long S, long long L) { return S <= kCountHere && S * L <= 16384; }
bool one_preference(long long B, int N, long long L) { return B <= (L > kWarpList ? 8 : 32) && B * N * L <= 65536; }

// The launches of a call around its main one, `run(blocks, cluster)`.
template <int N, class F>
int loss_call(Ends& e, bool one, int blocks, void* ws, cudaStream_t s, F run) {
  const LossLayout l = loss_layout();
  e.one = one;
  e.ctl = (Ctl*)((char*)ws + l.o_ctl);
  e.part = (float2*)((char*)ws + l.o_part);
  e.status = ws ? &((Header*)ws)->status : nullptr;
  if (one) {
    if (blocks > kOneBlocks) blocks = kOneBlocks;
    while (blocks & (blocks - 1)) ++blocks;  // clusters of a power of two
    return run(blocks, blocks) == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
  }
  if (e.counted.n > kCountHere) {
    longlong2* const counts = (longlong2*)((char*)ws + l.o_counts);
    if (launch(k_count, kCountBlocks, 1024, 0, s, 1, e.counted, counts) != cudaSuccess) return CTCPB_ECUDA;
    e.counted.counts = counts;
  }
  if (run(blocks, 1) != cudaSuccess) return CTCPB_ECUDA;
  if ((e.loss || e.stats) && launch(k_loss_end<N>, 1, 256, 0, s, 1, e, blocks) != cudaSuccess) return CTCPB_ECUDA;
  return CTCPB_OK;
}

int check_loss_ws(const void* ws, size_t ws_bytes, bool one) {
  if (!ws) return one ? CTCPB_OK : CTCPB_ENULL;
  if (((uintptr_t)ws & 255u) != 0) return CTCPB_EALIGN;
  return ws_bytes < (one ? sizeof(Header) : loss_layout().total) ? CTCPB_ESIZE : CTCPB_OK;
}
int check_policy(long long S, long long L) {
  return S < 0 || S > kMaxSeqs || L < 0 || L > kMaxTokens || (L > 0 && S > kMaxCall / L) ? CTCPB_EINVAL : CTCPB_OK;
}
int check_lists(long long B, int N, long long L) {
  return B < 0 || N < 1 || N > kMaxSeqs || B > kMaxSeqs / N || L < 0 || L > kMaxTokens ? CTCPB_EINVAL : CTCPB_OK;
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" {

int ctcpb_policy_loss_workspace_size(int64_t S, int64_t L, size_t* bytes) {
  if (int rc = check_policy(S, L)) return rc;
  if (!bytes) return CTCPB_ENULL;
  *bytes = one_policy(S, L) ? sizeof(Header) : loss_layout().total;
  return CTCPB_OK;
}

int ctcpb_policy_loss(const float* nll, int64_t ld_nll, const float* old_nll, int64_t ld_old, const float* ref_nll,
                      int64_t ld_ref, const float* advantages, int64_t ld_advantages, const int32_t* lengths,
                      int64_t S, int64_t L, double clip_low, double clip_high, float kl_weight, int reduction,
                      const float* grad, float* loss, float* stats, float* dnll, void* ws, size_t ws_bytes,
                      ctcpb_stream_t stream) {
  if (int rc = check_policy(S, L)) return rc;
  if (reduction < CTCPB_REDUCE_NONE || reduction > CTCPB_REDUCE_SEQUENCE_MEAN) return CTCPB_EINVAL;
  if (!(clip_low >= 0.) || std::isinf(clip_low) || !(clip_high >= 0.) || !std::isfinite(kl_weight)) return CTCPB_EINVAL;
  const bool any = S > 0 && L > 0, one = one_policy(S, L);
  if (any && (ld_nll < L || ld_old < L || (ref_nll && ld_ref < L) || (ld_advantages != 0 && ld_advantages < L)))
    return CTCPB_EINVAL;
  if (any && (!nll || !old_nll || !advantages)) return CTCPB_ENULL;
  if (any && dnll && !grad) return CTCPB_ENULL;
  if (int rc = check_loss_ws(ws, ws_bytes, one)) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  PolicyArgs a{};
  a.nll = nll;
  a.old = old_nll;
  a.ref = ref_nll;
  a.adv = advantages;
  a.ld_nll = ld_nll;
  a.ld_old = ld_old;
  a.ld_ref = ld_ref;
  a.ld_adv = ld_advantages;
  a.lengths = lengths;
  a.S = any ? S : 0;
  a.L = L;
  a.high = std::log1p(clip_high);
  a.low = clip_low < 1. ? std::log1p(-clip_low) : -INFINITY;
  a.fhigh = (float)a.high;
  a.flow = (float)a.low;
  a.qhigh = (float)clip_high;
  a.qlow = (float)-clip_low;
  a.kl = kl_weight;
  a.reduction = reduction;
  a.grad = grad;
  const bool none = reduction == CTCPB_REDUCE_NONE;
  a.loss = none ? loss : nullptr;
  a.dnll = dnll;
  const bool vec = L % 4 == 0 && on16(nll, ld_nll) && on16(old_nll, ld_old) && on16(ref_nll, ref_nll ? ld_ref : 0) &&
                   (ld_advantages == 0 || on16(advantages, ld_advantages)) && on16(dnll, 0) &&
                   (!none || (on16(loss, 0) && on16(grad, 0)));
  const long long pieces = vec ? L / 4 : L;
  a.pieces = Divisor(any ? (u32)pieces : 1u);
  a.work = any ? (u32)(S * pieces) : 0u;
  a.dense = ld_nll == L && ld_old == L && (!ref_nll || ld_ref == L) && (ld_advantages == 0 || ld_advantages == L);
  a.ends.counted = Counted{lengths, nullptr, nullptr, a.S, L, 0, reduction, grad, nullptr};
  a.ends.loss = none ? nullptr : loss;
  a.ends.stats = stats;
  const long long blocks = ((long long)a.work + kLossThreads - 1) / kLossThreads;
  const int most = 152 * (vec ? 3 : 4);
  return loss_call<3>(a.ends, one, blocks < 1 ? 1 : blocks < most ? (int)blocks : most, ws, s, [&](int n, int cluster) {
    return vec ? launch(k_policy<true>, n, kLossThreads, 0, s, cluster, a)
               : launch(k_policy<false>, n, kLossThreads, 0, s, cluster, a);
  });
}

int ctcpb_preference_loss_workspace_size(int64_t B, int N, int64_t L, size_t* bytes) {
  if (int rc = check_lists(B, N, L)) return rc;
  if (!bytes) return CTCPB_ENULL;
  *bytes = one_preference(B, N, L) ? sizeof(Header) : loss_layout().total;
  return CTCPB_OK;
}

int ctcpb_preference_loss(const float* nll, int64_t ld_nll, const float* ref_nll, int64_t ld_ref,
                          const int32_t* chosen, const int32_t* rejected, const int32_t* lengths, int64_t B, int N,
                          int64_t L, float beta, float margin, float label_smoothing, int average, int reduction,
                          const float* grad, float* loss, float* margins, float* dnll, void* ws, size_t ws_bytes,
                          ctcpb_stream_t stream) {
  if (int rc = check_lists(B, N, L)) return rc;
  if (reduction < CTCPB_REDUCE_NONE || reduction > CTCPB_REDUCE_SUM || (average != 0 && average != 1)) return CTCPB_EINVAL;
  if (!std::isfinite(beta) || !std::isfinite(margin) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
    return CTCPB_EINVAL;
  const bool one = one_preference(B, N, L);
  if (B > 0 && L > 0 && (ld_nll < L || (ref_nll && ld_ref < L))) return CTCPB_EINVAL;
  if (B > 0 && (!chosen || !rejected || (L > 0 && !nll))) return CTCPB_ENULL;
  if (B > 0 && L > 0 && dnll && !grad) return CTCPB_ENULL;
  if (int rc = check_loss_ws(ws, ws_bytes, one)) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  PairArgs a{};
  a.nll = nll;
  a.ref = ref_nll;
  a.ld_nll = ld_nll;
  a.ld_ref = ld_ref;
  a.chosen = chosen;
  a.rejected = rejected;
  a.lengths = lengths;
  a.B = B;
  a.L = L;
  a.N = N;
  a.beta = beta;
  a.margin = margin;
  a.smooth = label_smoothing;
  a.average = average;
  a.reduction = reduction;
  a.grad = grad;
  const bool none = reduction == CTCPB_REDUCE_NONE;
  a.loss = none ? loss : nullptr;
  a.margins = margins;
  a.dnll = L > 0 ? dnll : nullptr;
  a.ends.counted = Counted{nullptr, chosen, rejected, B, 0, N, reduction, grad, nullptr};
  a.ends.loss = none ? nullptr : loss;
  const bool vec = L % 4 == 0 && on16(nll, ld_nll) && on16(ref_nll, ref_nll ? ld_ref : 0) && on16(dnll, 0);
  const bool wide = L > kWarpList;
  const long long per = wide ? 1 : kPairThreads / 32, blocks = (B + per - 1) / per;
  return loss_call<1>(a.ends, one, blocks < 1 ? 1 : blocks < kLossBlocks ? (int)blocks : kLossBlocks, ws, s,
                      [&](int n, int cluster) {
                        if (vec)
                          return wide ? launch(k_preference<true, kPairThreads>, n, kPairThreads, 0, s, cluster, a)
                                      : launch(k_preference<true, 32>, n, kPairThreads, 0, s, cluster, a);
                        return wide ? launch(k_preference<false, kPairThreads>, n, kPairThreads, 0, s, cluster, a)
                                    : launch(k_preference<false, 32>, n, kPairThreads, 0, s, cluster, a);
                      });
}

}  // extern "C"
