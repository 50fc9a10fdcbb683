// Losses of the decoder's own N-best lists, with their gradients: the clipped
// policy loss with a KL term, and the preference loss of pairs
// (ctcpb_policy_loss, ctcpb_preference_loss).
//
//   d = old - nll, ratio = e^d, u = nll - ref
//   token loss = -(A + A q) + kl (e^u - 1 - u),  q = e^d - 1, held at the border's
//   R = sum (ref - nll),  z = beta (R_c - R_r) - margin,  log(1 + e^-z)
//
// Bound by HBM where lists are long, by the launches where they are short: each
// input is read once, the gradient written in the same pass.  What the gradient's
// factor needs first (the number of tokens, sequences or pairs) is a launch before.
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

constexpr int kLossThreads = 256;
constexpr int kLossBlocks = 152 * 8;
constexpr long long kMaxSeqs = 1 << 24, kMaxTokens = 1 << 24;

// What a launch before the main one finds.
struct Ctl {
  long long items;  // tokens, or pairs
  double factor;    // of the sum of the losses (means: 1 over how many)
  float grad;       // of the gradients: the loss's, times the factor (REDUCE_NONE: 1)
  u32 ticket;
};
struct LossLayout {
  size_t o_ctl, o_part, total;
};
LossLayout loss_layout() {
  LossLayout l{};
  l.o_ctl = sizeof(Header);
  l.o_part = l.o_ctl + 256;
  l.total = align_up(l.o_part + (size_t)kLossBlocks * 3 * sizeof(float2), 256);
  return l;
}

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
// a - b as value and error
__device__ __forceinline__ void add_difference(Sum2& s, float a, float b) {
  const float d = a - b, t = d - a;
  s.add(d);
  s.lo += (a - (d - t)) - (b + t);
}

// e^x - 1 and e^x - 1 - x.  Near 0 the second is x^2 (1/2! + x/3! + ...), the first
// that and x: neither loses digits.  Elsewhere the exponential, less 1.
__device__ __forceinline__ void exp_less(float x, float& e1, float& e2) {
  if (fabsf(x) < 0.5f) {  // the next term is 2e-9 of the sum
    float p = 1.f / 362880.f;
    p = fmaf(p, x, 1.f / 40320.f);
    p = fmaf(p, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    e2 = p * x * x;
    e1 = e2 + x;
  } else {
    e1 = expf(x) - 1.f;
    e2 = isinf(e1) ? e1 : e1 - x;
  }
}

// Sums over a block, in a fixed order; thread 0 has them.
template <int N>
__device__ __forceinline__ void block_sums(Sum2 (&v)[N], float2 (*red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i].warp_sum();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
    for (int i = 0; i < N; ++i) red[warp][i] = make_float2(v[i].hi, v[i].lo);
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = Sum2();
      if (lane < (int)(blockDim.x >> 5)) {
        v[i].hi = red[lane][i].x;
        v[i].lo = red[lane][i].y;
      }
      v[i].warp_sum();
    }
  }
}
__device__ __forceinline__ void block_counts(long long (&v)[2], long long (*red)[2]) {
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
}
__device__ __forceinline__ void set_ctl(Ctl* ctl, long long items, long long of, int reduction, const float* grad) {
  const bool mean = reduction == CTCPB_REDUCE_MEAN || reduction == CTCPB_REDUCE_SEQUENCE_MEAN;
  ctl->items = items;
  ctl->factor = mean ? 1. / (double)of : 1.;
  ctl->grad = reduction == CTCPB_REDUCE_NONE || !grad ? 1.f : mean ? (float)((double)*grad / (double)of) : *grad;
  ctl->ticket = 0;
}

__device__ __forceinline__ long long length_of(const int* lengths, long long s, long long L) {
  if (!lengths) return L;
  const long long n = lengths[s];
  return n < 0 ? 0 : n > L ? L : n;
}

// ---------------------------------------------------------------- counts

// Tokens and sequences that have some.
__global__ void __launch_bounds__(1024) k_count_tokens(const int* lengths, long long S, long long L, int reduction,
                                                       const float* grad, Ctl* ctl, u32* status) {
  __shared__ long long red[32][2];
  pdl_wait();
  pdl_next();
  long long v[2] = {0, 0};
  for (long long s = threadIdx.x; s < S; s += blockDim.x) {
    const long long l = length_of(lengths, s, L);
    v[0] += l;
    v[1] += l > 0;
  }
  block_counts(v, red);
  if (threadIdx.x == 0) {
    set_ctl(ctl, v[0], reduction == CTCPB_REDUCE_SEQUENCE_MEAN ? v[1] : v[0], reduction, grad);
    *status = 0;
  }
}

// A list's pair: (chosen, rejected), or false where it takes no part.
__device__ __forceinline__ bool pair_of(const int* chosen, const int* rejected, long long b, int N, int& c, int& r) {
  c = chosen[b];
  r = rejected[b];
  return c >= 0 && r >= 0 && c < N && r < N;
}
__global__ void __launch_bounds__(1024) k_count_pairs(const int* chosen, const int* rejected, long long B, int N,
                                                      int reduction, const float* grad, Ctl* ctl, u32* status) {
  __shared__ long long red[32][2];
  pdl_wait();
  pdl_next();
  long long v[2] = {0, 0};  // pairs, and lists with an index past the end
  for (long long b = threadIdx.x; b < B; b += blockDim.x) {
    int c, r;
    v[0] += pair_of(chosen, rejected, b, N, c, r);
    v[1] += c >= N || r >= N;
  }
  block_counts(v, red);
  if (threadIdx.x == 0) {
    set_ctl(ctl, v[0], v[0], reduction, grad);
    *status = v[1] ? CTCPB_DEV_TARGET : 0u;
  }
}

// ---------------------------------------------------------------- the end of a call

// A block's sums go to its place; the block that comes last adds all of them in
// order.  Returns whether this is that block (its thread 0 has the totals).
template <int N>
__device__ __forceinline__ bool last_block(Sum2 (&v)[N], float2* part, u32* ticket, float2 (*red)[N]) {
  __shared__ u32 last;
  block_sums<N>(v, red);
  if (threadIdx.x == 0) {
    for (int i = 0; i < N; ++i) part[(size_t)blockIdx.x * N + i] = make_float2(v[i].hi, v[i].lo);
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return false;
  __threadfence();
  for (int i = 0; i < N; ++i) v[i] = Sum2();
  for (u32 b = threadIdx.x; b < gridDim.x; b += blockDim.x)
    for (int i = 0; i < N; ++i) {
      const float2 p = __ldcg(part + (size_t)b * N + i);
      Sum2 q;
      q.hi = p.x;
      q.lo = p.y;
      v[i].add(q);
    }
  block_sums<N>(v, red);
  return true;
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
  float *loss, *stats, *dnll;
  Ctl* ctl;
  float2* part;
  int tx;            // threads of a row (a power of two)
  long long chunks;  // pieces of a row
};

// One token.  `hold`: the ratio is past the border and counts no more.
__device__ __forceinline__ void token(const PolicyArgs& a, float nll, float old, float ref, float A, Sum2& loss, float& kl,
                                      float& held, float& slope, float& each) {
  const float d = old - nll;
  float q, k;
  exp_less(d, q, k);
  bool hold = false;
  // d is rounded, which keeps its order with a rounded border: only where the two
  // are equal does it take the exact difference
  if (A > 0.f)
    hold = d > a.fhigh || (d == a.fhigh && (double)old - (double)nll > a.high);
  else if (A < 0.f)
    hold = d < a.flow || (d == a.flow && (double)old - (double)nll < a.low);
  else if (A == 0.f)
    q = 0.f;  // a token without an advantage adds nothing, whatever its ratio overflows to
  slope = hold ? 0.f : fmaf(A, q, A);
  if (hold) q = A > 0.f ? a.qhigh : a.qlow;
  float more = -A * q;
  if (a.ref) {
    float e;
    exp_less(nll - ref, e, k);
    kl += k;
    more = fmaf(a.kl, k, more);
    slope = fmaf(a.kl, e, slope);
  }
  loss.add(-A);
  loss.add(more);
  held += hold ? 1.f : 0.f;
  each = more - A;
}

template <bool VEC>
__global__ void __launch_bounds__(kLossThreads) k_policy(const PolicyArgs a) {
  __shared__ float2 red[32][3];
  constexpr int V = VEC ? 4 : 1;
  pdl_wait();
  pdl_next();
  const int tx = threadIdx.x & (a.tx - 1), ty = threadIdx.x / a.tx, rows = kLossThreads / a.tx;
  const bool none = a.reduction == CTCPB_REDUCE_NONE, by_len = a.reduction == CTCPB_REDUCE_SEQUENCE_MEAN;
  const float g = a.ctl->grad;
  Sum2 sums[3];
  const long long groups = (a.S + rows - 1) / rows, work = groups * a.chunks;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const long long group = a.chunks == 1 ? w : w / a.chunks, s = group * rows + ty;
    const long long t = ((w - group * a.chunks) * a.tx + tx) * V;
    if (s >= a.S || t >= a.L) continue;
    const long long len = length_of(a.lengths, s, a.L);
    // 1 / len, and what its rounding took off (len <= 2^24 is exact)
    const float wt = by_len && len > 0 ? 1.f / (float)len : 1.f;
    const float wt_lo = by_len && len > 0 ? fmaf(-wt, (float)len, 1.f) * wt : 0.f;
    const float gw = g * wt;
    float nll[V], old[V], ref[V], adv[V], up[V], slope[V], each[V];
    const long long at = s * a.L + t;
    const int live = len - t >= V ? V : len > t ? (int)(len - t) : 0;
    if (live) {
      // (a vector may reach behind the length, not behind the row)
      if constexpr (VEC) {
        auto get = [](float (&v)[4], const float* p) {
          const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        };
        get(nll, a.nll + s * a.ld_nll + t);
        get(old, a.old + s * a.ld_old + t);
        if (a.ref) get(ref, a.ref + s * a.ld_ref + t);
        if (a.ld_adv) get(adv, a.adv + s * a.ld_adv + t);
        if (none && a.grad) get(up, a.grad + at);
      } else {
        nll[0] = a.nll[s * a.ld_nll + t];
        old[0] = a.old[s * a.ld_old + t];
        if (a.ref) ref[0] = a.ref[s * a.ld_ref + t];
        if (a.ld_adv) adv[0] = a.adv[s * a.ld_adv + t];
        if (none && a.grad) up[0] = a.grad[at];
      }
    }
    const float row_adv = a.ld_adv == 0 && live ? a.adv[s] : 0.f;
    Sum2 loss;
    float kl = 0.f, held = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      slope[i] = each[i] = 0.f;
      if (i < live) {
        token(a, nll[i], old[i], a.ref ? ref[i] : 0.f, a.ld_adv ? adv[i] : row_adv, loss, kl, held, slope[i], each[i]);
        slope[i] *= none ? (a.grad ? up[i] : 1.f) : gw;
      }
    }
    if (live) {
      sums[0].add(by_len ? loss.times(wt, wt_lo) : loss);
      sums[1].add(kl);
      sums[2].add(held);
    }
    if constexpr (VEC) {
      if (a.dnll) __stcs(reinterpret_cast<float4*>(a.dnll + at), make_float4(slope[0], slope[1], slope[2], slope[3]));
      if (none && a.loss) __stcs(reinterpret_cast<float4*>(a.loss + at), make_float4(each[0], each[1], each[2], each[3]));
    } else {
      if (a.dnll) a.dnll[at] = slope[0];
      if (none && a.loss) a.loss[at] = each[0];
    }
  }
  if (!last_block<3>(sums, a.part, &a.ctl->ticket, red) || threadIdx.x != 0) return;
  // over no tokens the factor is infinite and the means are not numbers
  const double tokens = (double)a.ctl->items;
  if (!none && a.loss) *a.loss = (float)(sums[0].value() * a.ctl->factor);
  if (a.stats) {
    a.stats[0] = (float)(sums[1].value() / tokens);
    a.stats[1] = (float)(sums[2].value() / tokens);
  }
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
  float *loss, *margins, *dnll;
  Ctl* ctl;
  float2* part;
};

// A list is worked on by GT threads (a warp, or the block): both rows' sums, the
// pair's loss, then the gradients of all its hypotheses.
template <bool VEC, int GT>
__global__ void __launch_bounds__(kLossThreads) k_preference(const PairArgs a) {
  __shared__ float2 red[32][1];
  __shared__ float2 rowsum[2][GT / 32];
  __shared__ float slopes[kLossThreads / GT];
  constexpr int V = VEC ? 4 : 1, per = kLossThreads / GT;
  pdl_wait();
  pdl_next();
  const int t0 = threadIdx.x % GT, g = threadIdx.x / GT;
  const bool none = a.reduction == CTCPB_REDUCE_NONE;
  const float scale = a.ctl->grad * a.beta;
  Sum2 sums[1];
  const long long groups = (a.B + per - 1) / per;
  for (long long w = blockIdx.x; w < groups; w += gridDim.x) {
    const long long b = w * per + g;
    if (b >= a.B) continue;  // (a whole warp; never a part of the block where it meets)
    int c, r;
    const bool pair = pair_of(a.chosen, a.rejected, b, a.N, c, r);
    const long long lc = pair ? length_of(a.lengths, b * a.N + c, a.L) : 0;
    const long long lr = pair ? length_of(a.lengths, b * a.N + r, a.L) : 0;
    Sum2 R[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long row = b * a.N + (k ? r : c), len = k ? lr : lc;
      const float *const pn = a.nll + row * a.ld_nll, *const pf = a.ref + row * a.ld_ref;
      for (long long t = (long long)t0 * V; t < len; t += GT * V) {
        if constexpr (VEC) {
          const float4 n = *reinterpret_cast<const float4*>(pn + t);
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
          if (a.ref) f = *reinterpret_cast<const float4*>(pf + t);
          add_difference(R[k], f.x, n.x);
          if (t + 1 < len) add_difference(R[k], f.y, n.y);
          if (t + 2 < len) add_difference(R[k], f.z, n.z);
          if (t + 3 < len) add_difference(R[k], f.w, n.w);
        } else {
          add_difference(R[k], a.ref ? pf[t] : 0.f, pn[t]);
        }
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
      if (c != r) {
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
      if (none && a.loss) a.loss[b] = loss;
      if (a.margins) a.margins[b] = m;
      sums[0].add(loss);
      slopes[g] = a.smooth * up - (1.f - a.smooth) * dn;
    }
    if constexpr (GT > 32)
      __syncthreads();
    else
      __syncwarp();
    if (a.dnll) {
      const float dz = pair && c != r ? slopes[g] * (none ? a.beta * a.grad[b] : scale) : 0.f;
      const float gc = -dz / (a.average && lc > 0 ? (float)lc : 1.f), gr = dz / (a.average && lr > 0 ? (float)lr : 1.f);
      float* const out = a.dnll + b * a.N * a.L;
      for (int n = 0; n < a.N; ++n) {
        const bool is = pair && c != r && (n == c || n == r);
        const float v = n == c ? gc : gr;
        const long long len = is ? (n == c ? lc : lr) : 0;
        for (long long t = (long long)t0 * V; t < a.L; t += GT * V) {
          float* const p = out + n * a.L + t;
          if constexpr (VEC)
            *reinterpret_cast<float4*>(p) =
                make_float4(t < len ? v : 0.f, t + 1 < len ? v : 0.f, t + 2 < len ? v : 0.f, t + 3 < len ? v : 0.f);
          else
            *p = t < len ? v : 0.f;
        }
      }
    }
    // (the next list's first meeting comes after its sums, so slopes may be written again then)
    if constexpr (GT == 32) __syncwarp();
  }
  if (!last_block<1>(sums, a.part, &a.ctl->ticket, red) || threadIdx.x != 0) return;
  if (!none && a.loss) *a.loss = (float)(sums[0].value() * a.ctl->factor);
}

bool on16(const void* p, long long ld) { return ((uintptr_t)p & 15u) == 0 && ld % 4 == 0; }

int check_loss_ws(const void* ws, size_t ws_bytes) {
  if (!ws) return CTCPB_ENULL;
  if (((uintptr_t)ws & 255u) != 0) return CTCPB_EALIGN;
  return ws_bytes < loss_layout().total ? CTCPB_ESIZE : CTCPB_OK;
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" {

int ctcpb_policy_loss_workspace_size(int64_t S, int64_t L, size_t* bytes) {
  if (S < 0 || S > kMaxSeqs || L < 0 || L > kMaxTokens) return CTCPB_EINVAL;
  if (!bytes) return CTCPB_ENULL;
  *bytes = loss_layout().total;
  return CTCPB_OK;
}

int ctcpb_policy_loss(const float* nll, int64_t ld_nll, const float* old_nll, int64_t ld_old, const float* ref_nll,
                      int64_t ld_ref, const float* advantages, int64_t ld_advantages, const int32_t* lengths,
                      int64_t S, int64_t L, double clip_low, double clip_high, float kl_weight, int reduction,
                      const float* grad, float* loss, float* stats, float* dnll, void* ws, size_t ws_bytes,
                      ctcpb_stream_t stream) {
  if (S < 0 || S > kMaxSeqs || L < 0 || L > kMaxTokens) return CTCPB_EINVAL;
  if (reduction < CTCPB_REDUCE_NONE || reduction > CTCPB_REDUCE_SEQUENCE_MEAN) return CTCPB_EINVAL;
  if (!(clip_low >= 0.) || std::isinf(clip_low) || !(clip_high >= 0.) || !std::isfinite(kl_weight)) return CTCPB_EINVAL;
  const bool any = S > 0 && L > 0;
  if (any && (ld_nll < L || ld_old < L || (ref_nll && ld_ref < L) || (ld_advantages != 0 && ld_advantages < L)))
    return CTCPB_EINVAL;
  if (any && (!nll || !old_nll || !advantages)) return CTCPB_ENULL;
  if (any && dnll && !grad) return CTCPB_ENULL;
  if (int rc = check_loss_ws(ws, ws_bytes)) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  const LossLayout l = loss_layout();
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
  a.loss = loss;
  a.stats = stats;
  a.dnll = dnll;
  a.ctl = (Ctl*)((char*)ws + l.o_ctl);
  a.part = (float2*)((char*)ws + l.o_part);
  const bool none = reduction == CTCPB_REDUCE_NONE;
  const bool vec = L % 4 == 0 && on16(nll, ld_nll) && on16(old_nll, ld_old) && on16(ref_nll, ref_nll ? ld_ref : 0) &&
                   (ld_advantages == 0 || on16(advantages, ld_advantages)) && on16(dnll, 0) &&
                   (!none || (on16(loss, 0) && on16(grad, 0)));
  const long long pieces = vec ? L / 4 : L;
  a.tx = 1;
  while (a.tx < kLossThreads && a.tx < pieces) a.tx *= 2;
  a.chunks = pieces > 0 ? (pieces + a.tx - 1) / a.tx : 1;
  const long long rows = kLossThreads / a.tx, work = any ? (S + rows - 1) / rows * a.chunks : 0;
  const int grid = work < 1 ? 1 : work < kLossBlocks ? (int)work : kLossBlocks;
  if (launch(k_count_tokens, 1, 1024, 0, s, 1, lengths, a.S, a.L, reduction, grad, a.ctl, &((Header*)ws)->status) !=
      cudaSuccess)
    return CTCPB_ECUDA;
  if ((vec ? launch(k_policy<true>, grid, kLossThreads, 0, s, 1, a) : launch(k_policy<false>, grid, kLossThreads, 0, s, 1, a)) !=
      cudaSuccess)
    return CTCPB_ECUDA;
  return CTCPB_OK;
}

int ctcpb_preference_loss_workspace_size(int64_t B, int N, int64_t L, size_t* bytes) {
  if (B < 0 || N < 1 || N > kMaxSeqs || B > kMaxSeqs / N || L < 0 || L > kMaxTokens) return CTCPB_EINVAL;
  if (!bytes) return CTCPB_ENULL;
  *bytes = loss_layout().total;
  return CTCPB_OK;
}

int ctcpb_preference_loss(const float* nll, int64_t ld_nll, const float* ref_nll, int64_t ld_ref,
                          const int32_t* chosen, const int32_t* rejected, const int32_t* lengths, int64_t B, int N,
                          int64_t L, float beta, float margin, float label_smoothing, int average, int reduction,
                          const float* grad, float* loss, float* margins, float* dnll, void* ws, size_t ws_bytes,
                          ctcpb_stream_t stream) {
  if (B < 0 || N < 1 || N > kMaxSeqs || B > kMaxSeqs / N || L < 0 || L > kMaxTokens) return CTCPB_EINVAL;
  if (reduction < CTCPB_REDUCE_NONE || reduction > CTCPB_REDUCE_SUM || (average != 0 && average != 1)) return CTCPB_EINVAL;
  if (!std::isfinite(beta) || !std::isfinite(margin) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
    return CTCPB_EINVAL;
  if (B > 0 && L > 0 && (ld_nll < L || (ref_nll && ld_ref < L))) return CTCPB_EINVAL;
  if (B > 0 && (!chosen || !rejected || (L > 0 && !nll))) return CTCPB_ENULL;
  if (B > 0 && L > 0 && dnll && !grad) return CTCPB_ENULL;
  if (int rc = check_loss_ws(ws, ws_bytes)) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  const LossLayout l = loss_layout();
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
  a.loss = loss;
  a.margins = margins;
  a.dnll = L > 0 ? dnll : nullptr;
  a.ctl = (Ctl*)((char*)ws + l.o_ctl);
  a.part = (float2*)((char*)ws + l.o_part);
  const bool vec = L % 4 == 0 && on16(nll, ld_nll) && on16(ref_nll, ref_nll ? ld_ref : 0) && on16(dnll, 0);
  const bool wide = L > 256;
  const long long per = wide ? 1 : kLossThreads / 32, work = (B + per - 1) / per;
  const int grid = work < 1 ? 1 : work < kLossBlocks ? (int)work : kLossBlocks;
  if (launch(k_count_pairs, 1, 1024, 0, s, 1, chosen, rejected, a.B, N, reduction, grad, a.ctl, &((Header*)ws)->status) !=
      cudaSuccess)
    return CTCPB_ECUDA;
  const cudaError_t e = vec ? (wide ? launch(k_preference<true, kLossThreads>, grid, kLossThreads, 0, s, 1, a)
                                    : launch(k_preference<true, 32>, grid, kLossThreads, 0, s, 1, a))
                            : (wide ? launch(k_preference<false, kLossThreads>, grid, kLossThreads, 0, s, 1, a)
                                    : launch(k_preference<false, 32>, grid, kLossThreads, 0, s, 1, a));
  return e == cudaSuccess ? CTCPB_OK : CTCPB_ECUDA;
}

}  // extern "C"
