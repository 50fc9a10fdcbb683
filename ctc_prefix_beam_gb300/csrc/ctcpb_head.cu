// The label head's products: log-probabilities log_softmax(x w^T + b) for the
// decoder, and softmax cross entropy over the same product with its gradients
// (ctcpb_log_probs, ctcpb_cross_entropy, ctcpb_cross_entropy_backward).
//
// All three rest on one matrix kernel, k_gemm, with an epilogue for each use:
//
//   z = x w^T + b                        [rows, V], never stored as such
//   kStats    per row and column tile (max z, sum exp(z - max)), z[target]
//   kLogp     z - lse, float32           the decoder's log_prob, as (z - max z) - log(sum)
//   kBand     both at once: a band of rows stays in the tensor memory of the
//             blocks that share it until its lse is known
//   kDlogits  d = (exp(z - lse) - [c = target]) r   16 bits, a piece of V
//   kProduct  dx += d w  and  dw = d^T x  (kDx, kDw: one of them)
//
// Sums, maxima and exponentials are float32; d is rounded to the operands' 16
// bits because the products that read it take no other: each of its entries
// moves by half a unit at most, as the rounded gradients themselves do.  In small
// calls (terms_of) what the rounding took off is a second term of the products.
#include <atomic>
#include <mutex>

#include "ctcpb_head.cuh"

namespace ctcpb {
namespace {

enum Mode { kStats = 0, kLogp = 1, kDlogits = 2, kProduct = 3, kBand = 4, kDx = 5, kDw = 6 };
__host__ __device__ constexpr bool is_product(int mode) { return mode == kProduct || mode == kDx || mode == kDw; }

constexpr int kEpiWarps = 16;      // 4 for each quarter of a tile's 256 columns
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kMaxStages = 8;
constexpr int kTileBytes = 163840;  // operand tiles
constexpr int kStageBuf = 4096;     // per epilogue warp: 32 rows of 128 bytes
constexpr int kEpiBytes = kEpiWarps * (kStageBuf + 32 * 4);  // ... and 32 biases
constexpr int kCtlBytes = 512;      // barriers, the tensor-memory address, the give-up flag
constexpr int kSmem = kTileBytes + kEpiBytes + kCtlBytes;
constexpr u32 kTmemCols = 512;
constexpr int kSplitDepth = 8;      // slices of 64 below which a tile is never split along K

// Partial (max, sum) pairs a row has for each column tile: one for each 64 columns.
__host__ __device__ constexpr int part_slots(int bn) { return (bn + 63) / 64; }

struct GemmArgs {
  const int* rows_dev;  // number of rows, on the device (null: `rows`)
  int rows;             // ... or its bound
  int M, N, K;          // output rows and columns, depth; the row count replaces M (K in d^T x)
  int bn;               // columns of a tile
  int none;             // 1: this gradient is not wanted, 2: not of this launch
  int stages;
  int group;            // row tiles that share a sweep over the columns
  int col0;             // first vocabulary entry of the piece
  int lo_at;            // columns from d to its second term (0: it has one)
  // logits
  const void* bias;
  int bias_type;
  const int* tgt;
  const float* lse;
  const float* rs;      // per-row factor of d
  int per_row;          // ... which differs from row to row
  float one_r, log2_r;  // ... or is this, and its log2
  float factor;         // of the accumulator: what truncation lost (kBand: times log2(e))
  const float2* norm;   // kLogp: a row's max z and -log of its sum
  float* zt;
  float2* part;
  long long part_ld;
  float* dbp;           // column sums of d per 32 rows [4 * row tiles][ldo]
  // output
  void* out;
  long long ldo;
  int vec;              // rows of `out` start on 16-byte boundaries
  int tiled;            // ... and tiled copies may write them (map_o)
  const float* scale;
  const int* rowmap;
  float* slots;         // partial tiles of the split wave
  float* acc;           // running sum over the pieces (null: one piece)
  int first, last;      // of the pieces
  u32* status;
  int reset_status;
  // kBand
  int members, bands;   // workers that share a row tile; row tiles worked on at once
};

// What a launch works on: one product, or dx and dw.  The maps are of the
// operands and of the output, where tiled copies write it.
template <int MODE>
struct Params {
  static constexpr int kProblems = is_product(MODE) ? 2 : 1;
  CUtensorMap a[kProblems], b[kProblems], o;
  GemmArgs g[kProblems];
};

// ---------------------------------------------------------------- tiles and their split

// A worker (block or pair) takes whole tiles in waves.  dx and dw may be one
// launch: the tiles of the second follow those of the first.  What is left of
// either, less than a wave, would leave workers idle: it is laid end to end and
// cut along K into equal shares.  A share begins or ends inside a tile at most
// once each; its sums there go to slots 2w (the part it begins with) and 2w + 1,
// and k_finish adds a tile's parts in order.
struct Seg {
  int p, m, n, tile, k0, k1, slot;  // problem; slot -1: the whole depth
};
template <int P>
struct Sched {
  int mt[P], nt[P], ks[P], group[P], dp[P], rem[P];
  bool off[P];                  // not wanted: its tiles are passed over (the others' split stays what it is)
  int w, G, t, u, u1, nw;
  int part, odd;                // a share's slices: part + 1 for the first `odd` workers, then part
  int members, band, bands;     // kBand: this worker's column tile is w % members; the next row tile, and the step
  __device__ int share(int i) const { return part * i + (i < odd ? i : odd); }  // the first slice of worker i's share
  __device__ int worker_of(int slice) const {
    const int big = odd * (part + 1);
    return slice < big ? slice / (part + 1) : odd + (slice - big) / part;
  }
  __device__ void init(const GemmArgs (&g)[P], int cg, int worker, int workers) {
    G = workers;
    w = worker;
    int slices = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const GemmArgs& a = g[i];
      off[i] = a.none != 0;
      dp[i] = rem[i] = 0;
      mt[i] = nt[i] = ks[i] = group[i] = 1;
      if (a.none == 2) continue;
      const int rows = a.rows_dev ? *a.rows_dev : a.rows;
      const bool rows_k = a.M > 0;  // M given: the rows are the depth
      const int M = rows_k ? a.M : rows, K = rows_k ? rows : a.K;
      mt[i] = M > 0 ? (M + 128 * cg - 1) / (128 * cg) : 1;
      nt[i] = (a.N + a.bn - 1) / a.bn;
      ks[i] = K > 0 ? (K + 63) / 64 : 1;
      group[i] = a.group < mt[i] ? a.group : mt[i];
      const int tiles = mt[i] * nt[i];
      if (P > 1 && ks[i] >= kSplitDepth) {
        rem[i] = tiles % G;
        if (5 * rem[i] > 4 * G) rem[i] = 0;  // a nearly full wave: joining would cost more than it gives
      }
      if (P > 1 && a.lo_at) ks[i] *= 2;  // both terms of d, one after the other
      dp[i] = tiles - rem[i];
      slices += rem[i] * ks[i];
    }
    nw = slices / 4;  // at least 4 slices of K a share
    if (nw > G) nw = G;
    if (nw < 1) nw = 1;
    part = slices / nw;
    odd = slices - part * nw;
    t = w;
    u = w < nw ? share(w) : 0;
    u1 = w < nw ? share(w + 1) : 0;
    members = g[0].members;
    if (members > 0) {
      bands = g[0].bands;
      band = w < members * bands ? w / members : mt[0];
    }
  }
  // kBand: every other band, from the second on if `turn`
  __device__ void take_turns(int turn) {
    band += turn * bands;
    bands *= 2;
  }
  __device__ void place(int i, int tile, Seg& s) const {
    const int per = group[i] * nt[i], g = tile / per, in = tile - g * per;
    const int gs = mt[i] - g * group[i] < group[i] ? mt[i] - g * group[i] : group[i];
    s.p = i;
    s.tile = tile;
    s.n = in / gs;
    s.m = g * group[i] + in - s.n * gs;
  }
  // the first slice of problem i's tile r of those that are cut
  __device__ int slice_of(int i, int r) const { return (i ? rem[0] * ks[0] : 0) + r * ks[i]; }
  // next() for who needs the depth alone: one problem's tiles all have the same
  __device__ bool next_depth(Seg& s) {
    if (P > 1 || members > 0) return next(s);
    s.k0 = 0;
    s.k1 = ks[0];
    const bool more = t < dp[0];
    t += G;
    return more;
  }
  __device__ bool next(Seg& s) {
    s.slot = -1;
    s.k0 = 0;
    if (P == 1 && members > 0) {
      if (band >= mt[0]) return false;
      s.p = s.tile = 0;
      s.m = band;
      s.n = w % members;
      s.k1 = ks[0];
      band += bands;
      return true;
    }
    const int whole = P > 1 ? dp[0] + dp[P - 1] : dp[0];
    while (t < whole) {
      const int i = P > 1 && t >= dp[0] ? 1 : 0, tile = i ? t - dp[0] : t;
      t += G;
      if (off[i ? P - 1 : 0]) continue;
      if (i)
        place(P - 1, tile, s);
      else
        place(0, tile, s);
      s.k1 = i ? ks[P - 1] : ks[0];
      return true;
    }
    while (u < u1) {
      const int i = P > 1 && u >= rem[0] * ks[0] ? 1 : 0;
      const int at = i ? u - rem[0] * ks[0] : u, depth = i ? ks[P - 1] : ks[0], r = at / depth;
      const int begin = u;
      s.k0 = at - r * depth;
      s.k1 = s.k0 + (u1 - u) < depth ? s.k0 + (u1 - u) : depth;
      u += s.k1 - s.k0;
      if (off[i ? P - 1 : 0]) continue;
      if (i)
        place(P - 1, dp[P - 1] + r, s);
      else
        place(0, dp[0] + r, s);
      if (s.k0 > 0 || s.k1 < depth) s.slot = 2 * w + (begin == share(w) ? 0 : 1);
      return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------- writing rows through shared memory
//
// A thread holds 32 columns of its own row.  The warp puts 128 bytes of each row
// into a 4 KB buffer, its 16-byte chunks permuted by row & 7: neither side has
// bank conflicts, and a tiled copy with the 128-byte swizzle reads it as it is.
// Such a copy writes whole lines without a thread's help (log-probabilities of
// 16000 frames: 91 us with the warps' own 64-byte stores); rows that it cannot
// take are written by the warp, a row's 128 bytes side by side.

__device__ __forceinline__ u32 stage_at(int row, int chunk) { return (u32)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

template <class T>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]),
                    Elem<T>::pack(v[6], v[7]));
}
__device__ __forceinline__ void stage_f32(char* buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(buf + stage_at(lane, c)) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
// 32 columns of a thread's own row as two 16-bit terms, the rounded value and what
// that took off, written by the thread itself (small calls only).
template <class T>
__device__ __forceinline__ void store_terms(T* hi, T* lo, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    u32 h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[8 * c + 2 * i], y = v[8 * c + 2 * i + 1];
      float hx, hy;
      h[i] = Elem<T>::pack(x, y);
      unpair(hx, hy, Elem<T>::unpack(h[i]));
      l[i] = Elem<T>::pack(x - hx, y - hy);
    }
    reinterpret_cast<uint4*>(hi)[c] = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4*>(lo)[c] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}
template <class T>
__device__ __forceinline__ void stage_16(char* buf, int lane, const float (&v)[32], int half) {
#pragma unroll
  for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(buf + stage_at(lane, 4 * half + c)) = pack8<T>(v + 8 * c);
}
// Write the buffer's rows (128 / sizeof(E) columns from c0 on, those below
// `cols`) to the output; orow is this lane's output row, -1 for none.
template <class E>
__device__ __forceinline__ void flush_rows(const char* buf, int lane, E* out, long long ldo, int orow, int c0, int cols,
                                           bool vec) {
  constexpr int per = 16 / (int)sizeof(E);  // elements of a chunk
  __syncwarp();
  if (vec) {
    const int c = lane & 7, col = c0 + c * per;
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int row = it * 4 + (lane >> 3);
      const int r = __shfl_sync(0xffffffffu, orow, row);
      const uint4 p = *reinterpret_cast<const uint4*>(buf + stage_at(row, c));
      if (r >= 0 && col < cols) {
        E* const o = out + (long long)r * ldo + col;
        if (col + per <= cols) {
          *reinterpret_cast<uint4*>(o) = p;
        } else {
          const E* e = reinterpret_cast<const E*>(&p);
#pragma unroll
          for (int i = 0; i < per; ++i)
            if (col + i < cols) o[i] = e[i];
        }
      }
    }
  } else {
#pragma unroll 4
    for (int row = 0; row < 32; ++row) {
      const int r = __shfl_sync(0xffffffffu, orow, row);
#pragma unroll
      for (int c = lane; c < 8 * per; c += 32) {
        const E e = *reinterpret_cast<const E*>(buf + stage_at(row, c / per) + (c % per) * (int)sizeof(E));
        if (r >= 0 && c0 + c < cols) out[(long long)r * ldo + c0 + c] = e;
      }
    }
  }
  __syncwarp();
}

// Sum of column l over the warp's rows, in lane l: at each halving a lane
// hands over the half of the columns that its partner keeps (31 exchanges).
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, s);
    }
  }
  return v[0];
}

// ---------------------------------------------------------------- log-probabilities in one pass
//
// The members of a band (blocks, or pairs of blocks) hold its logits in tensor
// memory, a column tile each.  A member publishes each row's (max, sum), waits
// for the others', and writes z - lse: the product is made once and the output
// written once.  The next band's product runs meanwhile into the other half of
// tensor memory.  A published pair is one 64-bit store over a mark that no pair
// can be, so that it is its own flag: whoever needs it reads until it is there
// (with a counter, its fence and two barriers an exchange took 6600 cycles,
// 12200 a band).  Every member must be resident (a cooperative launch); the wait
// for the others is bounded.  A wait that gives up makes every later one return
// at once, so that the warps go through the same barriers to the end.
//
// 16000 x 5000 x 512: 110 us, 2.9 TB/s written (two passes: 145).  A round of 256
// rows takes 9000 cycles: sums 2900, exchange 3000 to 4000, writes 5000 (the SM
// sends some 25 bytes a cycle), under each other only as far as the two sets go.

constexpr int kBandTile = kTileBytes - 2 * 512 * 8;  // operand tiles; the rest holds the rows' sums
constexpr int kSetWarps = kEpiWarps / 2;             // of the two sets, one for each half of tensor memory
constexpr int kPairSpins = 1 << 20;                  // of about 0.5 us
constexpr u64 kNoPair = ~0ull;                       // two NaNs that no arithmetic makes

__device__ __forceinline__ void set_sync(int set) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(1 + set), "n"(32 * kSetWarps) : "memory");
}
// (max, sum) pairs into one: the maxima first, so that the exponentials do not wait for one another
template <int K>
__device__ __forceinline__ float2 join_sums(const float2 (&p)[K]) {
  float m = p[0].x;
#pragma unroll
  for (int k = 1; k < K; ++k) m = fmaxf(m, p[k].x);
  const float mm = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) s = __fmaf_rn(p[k].y, ex2(p[k].x - mm), s);
  return make_float2(m, s);
}

template <int CG, class W>
__device__ void band_epilogue(const GemmArgs& a, Sched<1> sc, char* smem, u32 tmem, u32 s_tfull, u32 s_tempty, u32 rank,
                              const CUtensorMap* map_o, volatile u32* dead, W& wait) {
  // two sets of eight warps take the bands in turn: one's waits and copies are
  // under the other's arithmetic.  A warp has 32 rows and half the columns.
  const int warp = (int)threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int set = (warp - 4) / kSetWarps, half = ((warp - 4) >> 2) & 1, q = warp & 3, u = half * 128;
  char* const buf = smem + kTileBytes + (warp - 4) * kStageBuf;
  float* const bias_s = reinterpret_cast<float*>(smem + kTileBytes + kEpiWarps * kStageBuf) + set * 256;  // the member's
  float2* const own = reinterpret_cast<float2*>(smem + kBandTile) + set * 512;  // [2][128]: the halves' sums
  float2* const all = own + 256;                                                // [2][128]: half the members' each
  const int r128 = q * 32 + lane, G = a.members;
  const u32 tfull = s_tfull + 8 * set, tempty = (CG == 2 ? cluster_addr(s_tempty, 0) : s_tempty) + 8 * set;
  const u32 d = tmem + 256u * set + ((u32)(q * 32) << 16);
  sc.take_turns(set);
  Seg sg;
  bool first = true;
  int n0 = 0, end = 0, lim = 0;  // the member's columns: the first, how many, how many up to the last label
  u32 ph = 0;
  while (sc.next(sg)) {
    if (first) {  // the member's biases; a column past the vocabulary gets -inf
      n0 = sg.n * a.bn;
      lim = a.N - n0;
      end = a.bn < lim ? a.bn : lim;
      const int c = (int)threadIdx.x - 128 - set * 256;
      bias_s[c] = c < end ? (a.bias ? load_elem(a.bias, a.bias_type, n0 + c) * kLog2e : 0.f) : -INFINITY;
      set_sync(set);
      first = false;
    }
    __all_sync(0xffffffffu, wait(tfull, ph));
    ph ^= 1;
    tc_fence_after();
    // 1. the sums of the warp's columns, of the tile's (z to base 2 here, so that exp takes no product)
    float bm = -INFINITY, bs = 0.f;
#pragma unroll 1
    for (int c0 = u; c0 < end && c0 < u + 128; c0 += 32) {
      float v[32];
      tmem_load32(v, d + c0);
      tmem_wait(v);
      const float4* b4 = reinterpret_cast<const float4*>(bias_s + c0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = b4[i];
        fma2(v[4 * i], v[4 * i + 1], a.factor, b.x, b.y);
        fma2(v[4 * i + 2], v[4 * i + 3], a.factor, b.z, b.w);
      }
      // a tile's width is a multiple of 16 columns: the rest of a chunk is other memory
      if (c0 + 32 > a.bn) {
#pragma unroll
        for (int i = 16; i < 32; ++i) v[i] = -INFINITY;
      }
      float m4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m4[i] = fmaxf(v[i], v[i + 4]);
#pragma unroll
      for (int i = 8; i < 32; i += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], fmaxf(v[i + k], v[i + k + 4]));
      }
      const float mn = fmaxf(fmaxf(bm, fmaxf(m4[0], m4[1])), fmaxf(m4[2], m4[3]));
      const float mm = mn == -INFINITY ? 0.f : mn;
      float s[4] = {bs * ex2(bm - mm), 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        add2(v[i], v[i + 1], -mm);
        add2(v[i + 2], v[i + 3], -mm);
        add2(s[0], s[1], ex2(v[i]), ex2(v[i + 1]));
        add2(s[2], s[3], ex2(v[i + 2]), ex2(v[i + 3]));
      }
      bm = mn;
      bs = (s[0] + s[1]) + (s[2] + s[3]);
    }
    own[half * 128 + r128] = make_float2(bm, bs);
    set_sync(set);
    const float2 mine[2] = {own[r128], own[128 + r128]};
    float2 sum = join_sums(mine);
    if (G > 1) {
      // 2. publish the member's, read all of them as they come, half the members each
      u64* const part = reinterpret_cast<u64*>(a.part) + ((long long)sg.m * CG + rank) * G * 128 + r128;
      if (half == 0)
        asm volatile("st.relaxed.gpu.global.u64 [%0], %1;\n" ::"l"(part + (long long)sg.n * 128), "l"(pair(sum.x, sum.y))
                     : "memory");
      sum = make_float2(-INFINITY, 0.f);
      for (int i = half; i < G; i += 16) {
        u64 p[8];
        int spin = 0;
        bool there;
        do {
          there = true;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            p[k] = pair(-INFINITY, 0.f);
            if (i + 2 * k < G)
              asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];\n"
                           : "=l"(p[k])
                           : "l"(part + (long long)(i + 2 * k) * 128)
                           : "memory");
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) there = there && p[k] != kNoPair;
        } while (!there && ++spin < kPairSpins && !*dead);
        if (!there) *dead = 1;
        float2 f[9];
#pragma unroll
        for (int k = 0; k < 8; ++k) unpair(f[k].x, f[k].y, p[k]);
        f[8] = sum;
        sum = join_sums(f);
      }
      all[half * 128 + r128] = sum;
    }
    set_sync(set);  // (with one member: its sums have been read)
    if (G > 1) {
      const float2 both[2] = {all[r128], all[128 + r128]};
      sum = join_sums(both);
    }
    // 3. z - lse as (z - m) - log(sum), so that nothing grows with |z|
    const float ls = -log2f(sum.y) * kLn2;
    const int row0 = (sg.m * CG + (int)rank) * 128 + q * 32, row = row0 + lane;
#pragma unroll 1
    for (int c0 = u; c0 < end && c0 < u + 128; c0 += 32) {
      float v[32];
      tmem_load32(v, d + c0);
      if (a.tiled) {  // the last copy out of the buffer has read it
        if (lane == 0) tma_store_wait();
        __syncwarp();
      }
      tmem_wait(v);
      const float4* b4 = reinterpret_cast<const float4*>(bias_s + c0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = b4[i];
        fma2(v[4 * i], v[4 * i + 1], a.factor, b.x, b.y);
        fma2(v[4 * i + 2], v[4 * i + 3], a.factor, b.z, b.w);
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        add2(v[i], v[i + 1], -sum.x);
        fma2(v[i], v[i + 1], kLn2, ls, ls);
      }
      stage_f32(buf, lane, v);
      // a tiled copy writes 32 columns, and cuts a row off at 16 bytes only
      if (a.tiled && c0 + 32 <= a.bn && (a.N % 4 == 0 || c0 + 32 <= lim)) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && row0 < a.rows) tma_store(map_o, n0 + c0, row0, saddr(buf));
      } else {
        flush_rows<float>(buf, lane, (float*)a.out, a.ldo, row < a.rows ? row : -1, n0 + c0, n0 + end, a.vec);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(tempty);
  }
  if (a.tiled && lane == 0) tma_store_done();
  __syncwarp();
}

// Mark n pairs of pairs as not there, in a launch before the one that exchanges
// them: no member then reads what an earlier call left, and the members need not
// meet first, a wait that would have no limit (128 x 5000 x 512, both launches:
// 13.8 us a call, 14.4 with a meeting; 512 x 5000 x 512: 15.6 and 14.5).
__global__ void __launch_bounds__(256) k_marks(uint4* pairs, long long n) {
  pdl_wait();
  pdl_next();
  static_assert(kNoPair == ~0ull, "the mark is all ones");
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256)
    pairs[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// ---------------------------------------------------------------- the matrix kernel

// Persistent, one block (or pair of blocks, on a tile of 256 x 256) per SM.  One
// thread feeds 128-byte swizzled operand tiles by tiled copies through a ring,
// one warp issues tcgen05 matrix instructions into tensor memory, sixteen warps run
// the epilogue of the tile before meanwhile (two accumulators of 256 columns).
// Shared memory: the ring, the epilogue warps' buffers, the barriers.
//
// Bound by the tensor cores where K is long: kStats on 12800 x 32000 x 1024 runs
// alone in 406 us, 2.06 PFLOP/s, the tensor pipe active 94% of the time; back to
// back the power limit lowers the clock (465 us).  With K = 512 the epilogue's
// warps run all the time and keep the warp that issues from its slots: a step of 64
// takes 750 cycles then instead of 512 (12000 x 5000 x 512: kStats 42.7 us, 1.44
// PFLOP/s, the pipe active 64%; kDlogits 53 us, whose epilogue also sums the columns
// and writes 120 MB).  dx and dw, 89 us, take some 757 cycles a step: its copies take
// 544 (an SM takes in 60 bytes a cycle) and nothing makes up a late one, and the cut
// tiles of dw read d from HBM again (381 MB, 262 would do); bringing d into L2 ahead
// takes from the same rate (109 us and more), and with d in L2 a step is no shorter.
//
// TWO (kDlogits, kProduct): d has two terms.
template <int MODE, class T, int CG, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) k_gemm(const __grid_constant__ Params<MODE> prm) {
  constexpr int P = Params<MODE>::kProblems;
  constexpr bool BMN = is_product(MODE);  // the second operand has its rows along K
  auto problem = [](const Seg& g) { return MODE == kDx || P == 1 ? 0 : MODE == kDw ? 1 : g.p; };
  const GemmArgs& a = prm.g[0];           // (what both products share)
  const CUtensorMap& map_o = prm.o;
  extern __shared__ __align__(1024) char smem[];
  char* const ctl = smem + kTileBytes + kEpiBytes;
  const u32 s_tiles = saddr(smem);
  const u32 s_full = saddr(ctl), s_empty = s_full + 8 * kMaxStages, s_tfull = s_empty + 8 * kMaxStages,
            s_tempty = s_tfull + 16, s_tptr = s_tempty + 16;
  volatile u32* const tmem_ptr = reinterpret_cast<volatile u32*>(ctl + (s_tptr - s_full));
  volatile u32* const dead = tmem_ptr + 1;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const u32 rank = CG == 2 ? cluster_rank() : 0;
  const int worker = (int)blockIdx.x / CG, workers = (int)gridDim.x / CG;
  const int bnb = a.bn / CG;  // columns of B this block loads
  const u32 stage_bytes = 16384u + (u32)bnb * 128u;

  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      tma_prefetch_map(&prm.a[i]);
      tma_prefetch_map(&prm.b[i]);
    }
    if ((MODE == kLogp || MODE == kDlogits || MODE == kBand) && a.tiled) tma_prefetch_map(&map_o);
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init_n(s_full + 8 * i, 1);
      mbar_init_n(s_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_n(s_tfull + 8 * i, 1);
      mbar_init_n(s_tempty + 8 * i, (MODE == kBand ? kSetWarps : kEpiWarps) * CG);
    }
    *dead = 0;
    mbar_init_fence();
    fence_proxy_async();
  }
  if (warp == 2) tmem_alloc<CG>(s_tptr, kTmemCols);
  tc_fence_before();
  if (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const u32 tmem = *tmem_ptr;
  pdl_wait();
  pdl_next();
  if (a.reset_status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;

  // bounded wait; false once any wait of the block has given up
  auto wait = [&](u32 bar, u32 parity) -> bool {
    if (mbar_test_at(bar, parity)) return true;
    for (long long i = 0; i < kWaitSpins && !*dead; ++i)
      if (mbar_test_at(bar, parity)) return true;
    *dead = 1;
    return false;
  };

  Sched<P> sc;
  sc.init(prm.g, CG, worker, workers);
  Seg sg;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {  // ---- operand tiles
      int st = 0;
      u32 ph = 1;
      const u32 full0 = CG == 2 ? cluster_addr(s_full, 0) : s_full;
      while (ok && sc.next(sg)) {
        const int m0 = (sg.m * CG + (int)rank) * 128, n0 = sg.n * a.bn + (int)rank * bnb, col0 = prm.g[problem(sg)].col0;
        const CUtensorMap *map_a = &prm.a[problem(sg)], *map_b = &prm.b[problem(sg)];
        const bool amn = problem(sg) == 1;  // d^T: its columns are the rows, and contiguous
        const int each = (problem(sg) ? sc.ks[P - 1] : sc.ks[0]) / 2;  // TWO: slices of a term
        for (int j = sg.k0; j < sg.k1; ++j) {
          const bool lo = is_product(MODE) && TWO && j >= each;
          const int k = lo ? j - each : j, term = lo ? a.lo_at : 0;
          if (!(ok = wait(s_empty + 8 * st, ph))) break;
          const u32 at = s_tiles + (u32)st * stage_bytes, bt = at + 16384u, bar = full0 + 8 * st;
          if (rank == 0) mbar_expect(s_full + 8 * st, stage_bytes * CG);
          if (!amn) {
            tma_load<CG>(at, map_a, term + k * 64, m0, bar);
          } else {
            tma_load<CG>(at, map_a, term + m0, k * 64, bar);
            tma_load<CG>(at + 8192u, map_a, term + m0 + 64, k * 64, bar);
          }
          if constexpr (!BMN) {
            tma_load<CG>(bt, map_b, k * 64, col0 + n0, bar);
          } else {
            for (int c = 0; c < bnb; c += 64) tma_load<CG>(bt + (u32)c * 128u, map_b, n0 + c, col0 + k * 64, bar);
          }
          if (++st == a.stages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {  // ---- matrix instructions
      const u32 one = lane == 0;
      int st = 0, as = 0;
      u32 ph = 0, aph = 1;
      constexpr u64 kStepB = BMN ? 2048 >> 4 : 32 >> 4;
      // The epilogue's warps take most of the issue slots, and the queue in front of
      // the tensor cores is short, so a slice's instructions are few: the warp runs
      // this as one, a lane issues (12000 x 5000 x 512: kStats 42.4 us, 45.4 with a
      // lane alone in here), and a stage's descriptors are the first stage's with its
      // offset added (the address, in the lowest 14 bits, stays below 256 KB).
      const u64 desc_b = smem_desc(s_tiles + 16384u, BMN ? 8192 : 16);
      const u32 stage = stage_bytes >> 4;
      bool more = sc.next_depth(sg);
      while (more) {
        if (!(ok = __all_sync(0xffffffffu, wait(s_tempty + 8 * as, aph)))) break;
        tc_fence_after();
        const u32 d = tmem + 256u * as;
        const int slices = sg.k1 - sg.k0;
        const bool amn = problem(sg) == 1;
        const u32 idesc = mma_idesc(Elem<T>::kFormat, amn, BMN, 128 * CG, a.bn);
        const u64 step_a = amn ? 2048 >> 4 : 32 >> 4, desc_a = smem_desc(s_tiles, amn ? 8192 : 16);
        for (int k = 0; k < slices; ++k) {
          if (!(ok = __all_sync(0xffffffffu, wait(s_full + 8 * st, ph)))) break;
          tc_fence_after();
          const u64 da = desc_a + (u32)st * stage, db = desc_b + (u32)st * stage;
          mma_f16<CG>(d, da, db, idesc, k > 0, one);
#pragma unroll
          for (int i = 1; i < 4; ++i) mma_f16<CG>(d, da + i * step_a, db + i * kStepB, idesc, true, one);
          mma_commit<CG>(s_empty + 8 * st, one);
          if (++st == a.stages) {
            st = 0;
            ph ^= 1;
          }
          if (k == 0) more = sc.next_depth(sg);  // found while the tensor cores are busy
        }
        if (!ok) break;
        mma_commit<CG>(s_tfull + 8 * as, one);
        if (++as == 2) {
          as = 0;
          aph ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (MODE == kBand && warp >= 4) {
    if constexpr (MODE == kBand) band_epilogue<CG>(a, sc, smem, tmem, s_tfull, s_tempty, rank, &map_o, dead, wait);
  } else if (MODE != kBand && warp >= 4) {  // ---- epilogue: a warp's 32 rows and 64 columns of a tile
    const int q = warp & 3, u = ((warp - 4) >> 2) * 64;
    char* const buf = smem + kTileBytes + (warp - 4) * kStageBuf;
    float* const bias_s = reinterpret_cast<float*>(smem + kTileBytes + kEpiWarps * kStageBuf) + (warp - 4) * 32;
    const u32 tempty0 = CG == 2 ? cluster_addr(s_tempty, 0) : s_tempty;
    const int rows = a.rows_dev ? *a.rows_dev : a.rows;
    const bool store_tiled = (MODE == kLogp || MODE == kDlogits) && a.tiled;
    // what a tile's rows and columns bring, read while the tile before it is worked on
    struct Given {
      float bias[2], lse, rs;
      int tgt, orow;
    };
    auto read = [&](const Seg& g) {
      Given w{{0.f, 0.f}, 0.f, 0.f, -1, -1};
      const int row = (g.m * CG + (int)rank) * 128 + q * 32 + lane, n0 = g.n * a.bn;
      const int mrows = problem(g) == 1 ? prm.g[P - 1].M : rows;
      if (row < mrows) w.orow = row;
      if constexpr (is_product(MODE)) {
        const int* const rowmap = prm.g[problem(g)].rowmap;
        if (rowmap && row < mrows) w.orow = rowmap[row];
      } else {
        // a column past the vocabulary gets -inf, so that its exponential is 0
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = n0 + u + 32 * i + lane;
          w.bias[i] = u < a.bn && col < a.N ? (a.bias ? load_elem(a.bias, a.bias_type, (long long)a.col0 + col) : 0.f) : -INFINITY;
        }
        if (row < mrows) {
          if (MODE != kLogp && a.tgt) w.tgt = a.tgt[row];
          if (MODE == kLogp) {
            const float2 norm = a.norm[row];
            w.rs = norm.x;
            w.lse = norm.y;
          }
          if (MODE == kDlogits) {
            w.lse = a.lse[row];
            w.rs = a.rs[row];
          }
        }
      }
      return w;
    };
    int as = 0;
    u32 aph = 0;
    bool more = sc.next(sg);
    Given w = more ? read(sg) : Given{};
    while (more) {
      const GemmArgs& a = prm.g[problem(sg)];
      const int mrows = rows;  // (of the logits; a product's rows are in orow)
      const int mtile = sg.m * CG + (int)rank;
      const int row0 = mtile * 128 + q * 32, row = row0 + lane, n0 = sg.n * a.bn;
      // the columns that this tile writes end here (kDlogits fills its piece's width)
      const int lim = MODE == kDlogits ? (int)a.ldo - n0 : a.N - n0;
      const bool busy = u < a.bn && u < lim;
      const int tile = sg.tile, slot = sg.slot, stat = sg.n * part_slots(a.bn) + u / 64;
      float bm = -INFINITY, bs = 0.f;  // running max and sum of the row
      const int orow = w.orow, tgt = w.tgt - a.col0 - n0;  // (no target: below every column)
      const float rs = w.rs;
      const float lse = w.lse, bq[2] = {w.bias[0], w.bias[1]};
      if (!(ok = __all_sync(0xffffffffu, wait(s_tfull + 8 * as, aph)))) break;
      tc_fence_after();
      more = sc.next(sg);
      if (more) w = read(sg);
      const u32 d = tmem + 256u * as + ((u32)(q * 32) << 16);
      if (store_tiled) {  // the last copy out of the buffer has read it
        if (lane == 0) tma_store_wait();
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c0 = u + 32 * j;
        if (!busy || c0 >= lim) break;
        float v[32];
        if (c0 < a.bn) {
          tmem_load32(v, d + c0);
          if constexpr (!is_product(MODE)) {
            bias_s[lane] = bq[j];
            __syncwarp();
          }
          tmem_wait(v);
        } else {  // kDlogits, a tile of 32 columns: zeros fill the piece
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        if constexpr (!is_product(MODE)) {
          // z, the same bits in every use: z - max z and z - lse are exact where they are small
          if (c0 < a.bn) {
            const float4* b4 = reinterpret_cast<const float4*>(bias_s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 b = b4[i];
              fma2(v[4 * i], v[4 * i + 1], a.factor, b.x, b.y);
              fma2(v[4 * i + 2], v[4 * i + 3], a.factor, b.z, b.w);
            }
          }
        }
        if constexpr (MODE == kStats) {
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(v[i], v[i + 4]);
#pragma unroll
          for (int i = 8; i < 32; i += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], fmaxf(v[i + k], v[i + k + 4]));
          }
          const float mn = fmaxf(fmaxf(bm, fmaxf(m4[0], m4[1])), fmaxf(m4[2], m4[3]));
          const float mm = mn == -INFINITY ? 0.f : mn;
          const int tr = tgt - c0;
          if (__any_sync(0xffffffffu, (u32)tr < 32u)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (tr == i) a.zt[row] = v[i];
          }
          float s[4] = {bs * ex2((bm - mm) * kLog2e), 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            add2(v[i], v[i + 1], -mm);
            add2(v[i + 2], v[i + 3], -mm);
            mul2(v[i], v[i + 1], kLog2e);
            mul2(v[i + 2], v[i + 3], kLog2e);
            add2(s[0], s[1], ex2(v[i]), ex2(v[i + 1]));
            add2(s[2], s[3], ex2(v[i + 2]), ex2(v[i + 3]));
          }
          bm = mn;
          bs = (s[0] + s[1]) + (s[2] + s[3]);
        } else if constexpr (MODE == kLogp) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            add2(v[i], v[i + 1], -rs);
            add2(v[i], v[i + 1], lse);
          }
          if (store_tiled && j) {
            if (lane == 0) tma_store_wait();
            __syncwarp();
          }
          stage_f32(buf, lane, v);
          // a tiled copy cuts a row off at 16 bytes only
          if (store_tiled && (a.N % 4 == 0 || c0 + 32 <= lim)) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && row0 < mrows) tma_store(&map_o, n0 + c0, row0, saddr(buf));
          } else {
            flush_rows<float>(buf, lane, (float*)a.out, a.ldo, orow, n0 + c0, a.N, a.vec);
          }
        } else if constexpr (MODE == kDlogits) {
          if (c0 < a.bn) {
            const float lr = a.per_row ? 0.f : a.log2_r;  // d = exp(z - lse) r: a factor r that all rows share is in the exponent
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              add2(v[i], v[i + 1], -lse);
              fma2(v[i], v[i + 1], kLog2e, lr, lr);
              v[i] = ex2(v[i]);
              v[i + 1] = ex2(v[i + 1]);
            }
            const int tr = tgt - c0;
            if (__any_sync(0xffffffffu, (u32)tr < 32u)) {
              const float one = a.per_row ? 1.f : a.one_r;
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] -= tr == i ? one : 0.f;
            }
            if (a.per_row) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= rs;
            }
            if (__any_sync(0xffffffffu, row >= mrows)) {  // rows past the last one are exact zeros (their z may hold anything)
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = row < mrows ? v[i] : 0.f;
            }
          }
          if constexpr (TWO) {
            T* const o = (T*)a.out + (long long)row * (2 * a.ldo) + n0 + c0;
            store_terms<T>(o, o + a.lo_at, v);
          } else {
            stage_16<T>(buf, lane, v, j);
          }
          if (a.dbp) {
            const float cs = column_sums(v, lane);
            if (c0 + lane < lim) a.dbp[((long long)mtile * 4 + q) * a.ldo + n0 + c0 + lane] = cs;
          }
        } else {
          const long long at = (long long)c0 * 128 + q * 32 + lane, size = 128ll * a.bn;
          if (slot >= 0) {  // a share of the depth: to its slot, a column's rows side by side
            float* o = a.slots + ((long long)slot * CG + rank) * size + at;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i * 128] = v[i];
          } else {
            if (a.acc) {
              float* o = a.acc + ((long long)tile * CG + rank) * size + at;
              if (!a.first) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += o[i * 128];
              }
              if (!a.last) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i * 128] = v[i];
              }
            }
            if (a.last) {
              const float f = *a.scale;
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= f;
              stage_16<T>(buf, lane, v, j);
            }
          }
        }
        __syncwarp();
      }
      if constexpr (MODE == kStats)
        if (u < a.bn && row < mrows) a.part[(long long)stat * a.part_ld + row] = make_float2(bm, bs);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * as);
      if (++as == 2) {
        as = 0;
        aph ^= 1;
      }
      // 64 columns of 16 bits are a buffer's worth
      if constexpr (MODE == kDlogits) {
        if (busy && !TWO) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) tma_store(&map_o, n0 + u, row0, saddr(buf));
        }
      }
      if constexpr (is_product(MODE)) {
        if (busy && slot < 0 && a.last) flush_rows<T>(buf, lane, (T*)a.out, a.ldo, orow, n0 + u, a.N, a.vec);
      }
    }
    if (store_tiled && lane == 0) tma_store_done();
    __syncwarp();
  }
  __syncthreads();
  if (*dead) {
    // a wait gave up: let the copies and matrix instructions in flight land
    // before the memory goes to another block
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
    if (threadIdx.x == 0) atomicOr(a.status, CTCPB_DEV_TIMEOUT);
  }
  tc_fence_before();
  if (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc<CG>(tmem, kTmemCols);
}

// ---------------------------------------------------------------- what is left after the products

// The parts of a tile that was cut, added in the order of K, and the tile's
// output written: a block per 32 rows and 64 columns, 8 columns a warp (16
// bytes of each row), two parts' loads in flight.
template <class T>
__device__ void join_tile(const GemmArgs& a, const Sched<2>& sc, int i, int cg, int r, int unit, char* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = sc.slice_of(i, r), hi = lo + sc.ks[i];
  const int w = sc.worker_of(lo);
  if (sc.share(w) <= lo && sc.share(w + 1) >= hi) return;  // one share: written by the matrix kernel
  Seg sg;
  sc.place(i, sc.dp[i] + r, sg);
  const int q = unit & 3, rank = (unit >> 2) % cg, u = (unit >> 2) / cg * 64;
  const int n0 = sg.n * a.bn;
  if (n0 + u >= a.N) return;
  const int rows = a.rows_dev ? *a.rows_dev : a.rows;
  const int mrows = a.M > 0 ? a.M : rows;
  const int c0 = u + 8 * warp;  // bn is a multiple of 64
  const long long at = (long long)c0 * 128 + q * 32 + lane, tile = 128ll * a.bn;
  // the output rows (four a warp) and the scale, on their way with the shares
  const int rr = warp * 4 + (lane >> 3);
  const int mine = (sg.m * cg + rank) * 128 + q * 32 + rr;
  const int orow = mine < mrows ? (a.rowmap ? a.rowmap[mine] : mine) : -1;
  const float f = a.last ? *a.scale : 0.f;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  auto slot_of = [&](int x) { return a.slots + ((2ll * x + (sc.share(x) >= lo ? 0 : 1)) * cg + rank) * tile + at; };
  for (int x = w; x < sc.nw && sc.share(x) < hi; x += 2) {
    const bool two = x + 1 < sc.nw && sc.share(x + 1) < hi;
    const float *o = slot_of(x), *p = two ? slot_of(x + 1) : o;
    float e[8], f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = o[i * 128];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = two ? p[i * 128] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (v[i] + e[i]) + f[i];
  }
  if (a.acc) {
    float* o = a.acc + ((long long)sg.tile * cg + rank) * tile + at;
    if (!a.first) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += o[i * 128];
    }
    if (!a.last) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i * 128] = v[i];
    }
  }
  if (!a.last) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  *reinterpret_cast<uint4*>(buf + stage_at(lane, warp)) = pack8<T>(v);
  __syncthreads();
  if (orow < 0) return;
  T* const out = (T*)a.out + (long long)orow * a.ldo;
  if (a.vec) {
    const int col = n0 + u + (lane & 7) * 8;
    const uint4 p = *reinterpret_cast<const uint4*>(buf + stage_at(rr, lane & 7));
    if (col + 8 <= a.N) {
      *reinterpret_cast<uint4*>(out + col) = p;
    } else {
      const T* e = reinterpret_cast<const T*>(&p);
      for (int i = 0; i < 8; ++i)
        if (col + i < a.N) out[col + i] = e[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // 8 lanes a row, neighbouring columns
      const int c = (lane & 7) + 8 * i;
      const T e = *reinterpret_cast<const T*>(buf + stage_at(rr, c >> 3) + (c & 7) * 2);
      if (n0 + u + c < a.N) out[n0 + u + c] = e;
    }
  }
}

struct FinishArgs {
  GemmArgs g[2][2];              // what each launch of the products worked on
  int runs, cg, workers, units;  // launches (0: nothing to join), units of a tile
  // db of a piece: the column sums of d over the row tiles
  const float* dbp;
  long long ld;
  const int* rows_dev;
  int per, cols, col0, type, bias_units;
  const float* scale;
  void* db;
};

// One launch for what the products of a piece leave: db (a block per 32
// columns, 8 slices of the rows, eight loads of a slice in flight) and the
// joins of dx and dw.  How many tiles were cut is known here only, so the
// blocks go through the units.  Bound by latency: some 45 MB, 21 us for 12000 x
// 5000 x 512.
template <class T>
__global__ void __launch_bounds__(256, 5) k_finish(const FinishArgs f) {
  __shared__ __align__(16) char buf[kStageBuf];
  pdl_wait();
  pdl_next();
  Sched<2> sc[2];
  int joins[2][2] = {{0, 0}, {0, 0}}, total = f.bias_units;
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (r < f.runs) {
      sc[r].init(f.g[r], f.cg, 0, f.workers);
#pragma unroll
      for (int i = 0; i < 2; ++i) total += joins[r][i] = sc[r].off[i] ? 0 : sc[r].rem[i] * f.units;
    }
  for (int b = blockIdx.x; b < total; b += gridDim.x) {
    if (b < f.bias_units) {
      float(*red)[32] = reinterpret_cast<float(*)[32]>(buf);
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      const int c = b * 32 + lane;
      int n = (*f.rows_dev + 128 * f.per - 1) / (128 * f.per);
      n = (n < 1 ? 1 : n) * 4 * f.per;
      float s = 0.f;
      if (c < f.cols)
        for (int j = warp; j < n; j += 64) {
          float p[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) p[k] = j + 8 * k < n ? f.dbp[(long long)(j + 8 * k) * f.ld + c] : 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) s += p[k];
        }
      red[warp][lane] = s;
      __syncthreads();
      if (warp == 0 && c < f.cols) {
        for (int w = 1; w < 8; ++w) s += red[w][lane];
        store_elem(f.db, f.type, (long long)f.col0 + c, s * *f.scale);
      }
    } else {
      int k = b - f.bias_units;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (k >= 0 && k < joins[r][i]) join_tile<T>(f.g[r][i], sc[r], i, f.cg, k / f.units, k % f.units, buf);
          k -= joins[r][i];
        }
    }
    __syncthreads();  // the buffer is used again
  }
}

// ---------------------------------------------------------------- rows

// Copy H 16-bit elements of a row by a warp, zero up to ld; `vec`: both sides
// on 16-byte boundaries and H a multiple of 8.
__device__ __forceinline__ void copy_row(const u16* __restrict__ in, u16* __restrict__ out, int H, int ld, bool vec,
                                         int lane) {
  if (vec) {
    const uint4* const i4 = reinterpret_cast<const uint4*>(in);
    uint4* const o4 = reinterpret_cast<uint4*>(out);
    const int n = H >> 3;
    for (int c = lane; c < n; c += 128) {
      uint4 p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + 32 * k < n) p[k] = i4[c + 32 * k];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + 32 * k < n) o4[c + 32 * k] = p[k];
    }
  } else {
    for (int c = lane; c < ld; c += 256) {
      u16 p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = c + 32 * k < H ? in[c + 32 * k] : (u16)0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + 32 * k < ld) out[c + 32 * k] = p[k];
    }
  }
}

// Rows of 16-bit elements to rows of ldo elements, zero from H on.
__global__ void __launch_bounds__(256) k_copy_rows(const u16* __restrict__ in, long long ldi, u16* __restrict__ out,
                                                   int ldo, long long n, int H) {
  pdl_wait();
  pdl_next();
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < n; r += (long long)gridDim.x * 8)
    copy_row(in + r * ldi, out + r * ldo, H, ldo, false, threadIdx.x & 31);
}

struct RowArgs {
  const int* targets;
  int N, V, H, ignore;
  const u16* x;
  long long ldx;
  int vec;             // x's rows are whole 16-byte pieces on 16-byte boundaries
  u16* xg;
  int ldg;
  int* rowmap;
  int* tgt;
  int* nv;             // out: number of rows kept
  u32* status;
  u32* ticket;
  // forward
  float* loss;         // per-row losses (reduction none) or null
  float* lse;
  // backward
  int type, reduction;
  const float* grad;
  const float* lse_in;
  float* lse_c;
  float* rs;
  float* scale;
  u16* dx;
  long long lddx;
  int dx_vec;
};

constexpr int kRowBlocks = 512;  // blocks of k_rows at most

__device__ __forceinline__ int block_sum(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) s += red[i];
  __syncthreads();
  return s;
}

// Keep the rows that have a target, in order, side by side: an ignored row
// costs no product, and whatever it holds (padding may be NaN) never meets a
// sum.  Each block counts the kept rows before its own by reading the targets,
// so one launch does it; `per` rows a block keep the blocks, and so the
// targets read, in proportion to N.  The rows up to the next multiple of 64,
// the depth that the last step of d^T x reads, are zeros.  Bound by latency:
// 16000 rows of 512, a quarter ignored, 12 us (28 MB).
__global__ void __launch_bounds__(256) k_rows(const RowArgs a, int per) {
  __shared__ int red[8];
  __shared__ float fred[8];
  __shared__ int src[256];
  pdl_wait();
  pdl_next();
  const int base = blockIdx.x * per, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int end = base + per < a.N ? base + per : a.N;
  const bool last = blockIdx.x == gridDim.x - 1;
  auto kept = [&](int t) { return t >= 0 && t < a.V && t != a.ignore; };
  const int t_first = base + (int)threadIdx.x < end ? a.targets[base + (int)threadIdx.x] : a.ignore;
  int before = 0, bad = 0;
  auto count = [&](int t) {
    const bool in = kept(t);
    before += in;
    bad |= !in && t != a.ignore;
  };
  int done = 0;  // `base` is a multiple of 16
  if (((uintptr_t)a.targets & 15) == 0) {
    const int4* const t4 = reinterpret_cast<const int4*>(a.targets);
    for (int i = threadIdx.x; i < base / 4; i += 256 * 8) {
      int4 t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = i + 256 * k < base / 4 ? t4[i + 256 * k] : make_int4(a.ignore, a.ignore, a.ignore, a.ignore);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        count(t[k].x);
        count(t[k].y);
        count(t[k].z);
        count(t[k].w);
      }
    }
    done = base;
  }
  for (int i = done + threadIdx.x; i < base; i += 256 * 8) {
    int t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = i + 256 * k < base ? a.targets[i + 256 * k] : a.ignore;
#pragma unroll
    for (int k = 0; k < 8; ++k) count(t[k]);
  }
  before = block_sum(before, red);
  // the largest finite |grad| of the rows that are kept (float16 only): d is scaled
  // by it to stay in range.  An ignored row's gradient is not asked for, and one that
  // is not finite must not take the others' with it.
  float gmax = 1.f;
  if (a.grad && a.reduction == CTCPB_REDUCE_NONE && a.type == CTCPB_F16) {
    float g = 0.f;
    for (int i = threadIdx.x; i < a.N; i += 256) {
      const float v = fabsf(a.grad[i]);
      if (kept(a.targets[i]) && v < INFINITY) g = fmaxf(g, v);
    }
    for (int s = 16; s > 0; s >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, s));
    if (lane == 0) fred[warp] = g;
    __syncthreads();
    for (int i = 0; i < 8; ++i) g = fmaxf(g, fred[i]);
    gmax = g > 0.f ? g : 1.f;
  }
  const float up = a.type == CTCPB_F16 ? 32768.f : 1.f;  // float16: |d| <= 1 is stored as |d| 2^15
  for (int r0 = base; r0 < end; r0 += 256) {  // 256 rows at a time
    const int row = r0 + (int)threadIdx.x;
    const int t = r0 == base ? t_first : row < end ? a.targets[row] : a.ignore;
    const bool in = kept(t);
    bad |= !in && t != a.ignore;
    const u32 m = __ballot_sync(0xffffffffu, in);
    if (lane == 0) red[warp] = __popc(m);
    __syncthreads();
    int off = 0, count = 0;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) off += red[i];
      count += red[i];
    }
    if (row < end) {
      // a kept row's place, an ignored row's complement
      src[threadIdx.x] = in ? before + off + __popc(m & ((1u << lane) - 1)) : -1;
      if (in) {
        const int to = src[threadIdx.x];
        a.rowmap[to] = row;
        a.tgt[to] = t;
        if (a.grad) {
          a.lse_c[to] = a.lse_in[row];
          a.rs[to] = a.reduction == CTCPB_REDUCE_NONE ? a.grad[row] / gmax * up : up;
        }
      } else {
        if (a.loss) a.loss[row] = 0.f;
        if (a.lse) a.lse[row] = 0.f;
      }
    }
    __syncthreads();
    const int n = end - r0 < 256 ? end - r0 : 256;
    for (int i = warp; i < n; i += 8) {
      const int to = src[i];
      if (to >= 0) {
        copy_row(a.x + (long long)(r0 + i) * a.ldx, a.xg + (long long)to * a.ldg, a.H, a.ldg, a.vec, lane);
      } else if (a.dx) {  // an ignored row has no gradient
        u16* d = a.dx + (long long)(r0 + i) * a.lddx;
        if (a.dx_vec)
          for (int c = lane; c < a.H / 8; c += 32) reinterpret_cast<uint4*>(d)[c] = make_uint4(0, 0, 0, 0);
        else
          for (int c = lane; c < a.H; c += 32) d[c] = 0;
      }
    }
    before += count;
    __syncthreads();
  }
  if (last) {
    const int nv = before;  // every kept row
    const long long z0 = (long long)nv * a.ldg / 8, z1 = (long long)(nv > 0 ? (nv + 63) / 64 * 64 : 64) * a.ldg / 8;
    for (long long i = z0 + threadIdx.x; i < z1; i += 256) reinterpret_cast<uint4*>(a.xg)[i] = make_uint4(0, 0, 0, 0);
    bad = block_sum(bad, red);
    if (threadIdx.x == 0) {
      *a.nv = nv;
      *a.status = bad ? CTCPB_DEV_TARGET : 0u;
      *a.ticket = 0;
      if (a.grad)
        *a.scale = (a.reduction == CTCPB_REDUCE_NONE
                        ? gmax
                        : a.grad[0] / (a.reduction == CTCPB_REDUCE_MEAN ? (float)(nv > 0 ? nv : 1) : 1.f)) /
                   up;
    }
  }
}

struct CombineArgs {
  const int* rows_dev;
  int rows;
  const float2* part;
  long long part_ld;
  int slots;
  float* lse;            // [row]
  float2* norm;          // or, for log-probabilities: m and -log(sum)
  const int* rowmap;     // null: the rows themselves, no loss
  const float* zt;
  float* loss;
  int reduction;
  float* sums;           // per block
  u32* ticket;
};

// lse = m + log(sum_j s_j exp(m_j - m)) over a row's tiles, and the losses,
// (m - z[target]) + log(sum): a block per 32 rows, 16 slices of
// the tiles, eight of a slice's loads in flight.  12000 rows of 80 pairs: 12 us,
// half of it the mean's chain of block sums.
constexpr int kSlices = 16;
__global__ void __launch_bounds__(32 * kSlices) k_combine(const CombineArgs a) {
  __shared__ float2 red[kSlices][32];
  __shared__ bool fin;
  pdl_wait();
  pdl_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = a.rows_dev ? *a.rows_dev : a.rows;
  const int i = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.f, zt = 0.f;
  int row = i;
  if (i < rows) {
    if (warp == 0 && a.rowmap) {
      row = a.rowmap[i];
      zt = a.zt[i];
    }
    for (int j = warp; j < a.slots; j += 8 * kSlices) {
      float2 p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        p[k] = j + k * kSlices < a.slots ? a.part[(long long)(j + k * kSlices) * a.part_ld + i]
                                         : make_float2(-INFINITY, 0.f);
      float mn = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) mn = fmaxf(mn, p[k].x);
      const float mm = mn == -INFINITY ? 0.f : mn;
      s *= ex2((m - mm) * kLog2e);
#pragma unroll
      for (int k = 0; k < 8; ++k) s = __fmaf_rn(p[k].y, ex2((p[k].x - mm) * kLog2e), s);
      m = mn;
    }
  }
  red[warp][lane] = make_float2(m, s);
  __syncthreads();
  float loss = 0.f;
  if (warp == 0 && i < rows) {
    for (int w = 1; w < kSlices; ++w) m = fmaxf(m, red[w][lane].x);
    const float mm = m == -INFINITY ? 0.f : m;
    s = 0.f;
    for (int w = 0; w < kSlices; ++w) s = __fmaf_rn(red[w][lane].y, ex2((red[w][lane].x - mm) * kLog2e), s);
    const float l = log2f(s) * kLn2;
    if (a.rowmap) {
      a.lse[row] = mm + l;
      loss = (m - zt) + l;  // the target's distance to the largest first: it is exact where it is small
      if (a.reduction == CTCPB_REDUCE_NONE) a.loss[row] = loss;
    } else {
      a.norm[row] = make_float2(m, -l);
    }
  }
  if (!a.rowmap || a.reduction == CTCPB_REDUCE_NONE) return;
  // the sum of the losses: each block's in a fixed order, then the blocks' by the last one
  if (warp == 0) {
    for (int k = 16; k > 0; k >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, k);
    if (lane == 0) {
      a.sums[blockIdx.x] = loss;
      __threadfence();
      fin = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!fin) return;
  __threadfence();
  __shared__ double dred[kSlices];
  double d = 0.0;
  for (int k = threadIdx.x; k < (int)gridDim.x; k += 32 * kSlices) d += (double)((volatile float*)a.sums)[k];
  for (int k = 16; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
  if (lane == 0) dred[warp] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kSlices; ++k) d += dred[k];
    *a.loss = (float)(a.reduction == CTCPB_REDUCE_MEAN ? d / (double)rows : d);
    *a.ticket = 0;
  }
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// An [outer, inner] matrix, rows of ld elements, in boxes of 128 bytes x box_outer.
bool make_map(CUtensorMap* m, int type, const void* base, long long inner, long long outer, long long ld, int box_outer) {
  const int size = type == CTCPB_F32 ? 4 : 2;
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * size};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_outer}, es[2] = {1, 1};
  const CUtensorMapDataType dt = type == CTCPB_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : type == CTCPB_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(m, dt, 2,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
Params<MODE> as_mode(const Params<kProduct>& p) {
  return {{p.a[0], p.a[1]}, {p.b[0], p.b[1]}, p.o, {p.g[0], p.g[1]}};
}
template <int MODE, class T, int CG, bool TWO>
cudaError_t launch_gemm_t(const Params<MODE>& prm, int blocks, cudaStream_t s) {
  constexpr auto kern = k_gemm<MODE, T, CG, TWO>;
  cudaError_t e = smem_optin<kern>(kSmem);
  if (e != cudaSuccess) return e;
  return launch_as(MODE == kBand, kern, dim3(blocks), kThreads, kSmem, s, CG, prm);
}
template <int MODE, bool TWO = false>
cudaError_t launch_gemm(int type, int cg, const Params<MODE>& prm, int blocks, cudaStream_t s) {
  if (cg == 2)
    return type == CTCPB_BF16 ? launch_gemm_t<MODE, __nv_bfloat16, 2, TWO>(prm, blocks, s)
                              : launch_gemm_t<MODE, __half, 2, TWO>(prm, blocks, s);
  return type == CTCPB_BF16 ? launch_gemm_t<MODE, __nv_bfloat16, 1, TWO>(prm, blocks, s)
                            : launch_gemm_t<MODE, __half, 1, TWO>(prm, blocks, s);
}
template <int MODE, bool TWO = false>
cudaError_t launch_gemm(int type, int cg, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                        const GemmArgs& a, int blocks, cudaStream_t s) {
  Params<MODE> prm;
  prm.a[0] = ma;
  prm.b[0] = mb;
  prm.o = mo;
  prm.g[0] = a;
  return launch_gemm<MODE, TWO>(type, cg, prm, blocks, s);
}

constexpr int kWorkers = 152;  // SMs; the split wave's slots are sized by it

int sm_count() {
  static std::atomic<int> known[128];  // by device
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return kWorkers;
  if (dev < 128 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return kWorkers;
  if (n > kWorkers) n = kWorkers;
  if (dev < 128) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

long long up_to(long long x, long long a) { return (x + a - 1) / a * a; }

// Columns of a tile of the logits: as wide as leaves no SM idle (128 x 5000 x
// 512 in two passes: kStats 9 us on 79 blocks of 64 columns).
int logits_bn(long long rows, int V) {
  const long long mt = (rows + 127) / 128;
  for (int bn = 256; bn > 64; bn >>= 1)
    if (V > bn / 2 && mt * ((V + bn - 1) / bn) >= kWorkers) return bn;
  return V > 32 ? 64 : 32;
}
int product_bn(int N) { return N > 128 ? 256 : N > 64 ? 128 : 64; }
// Two SMs on one tile of 256 x 256: each holds half of either operand, so a
// step moves 32 KB an SM for the work of 48 KB.  Against single SMs, 8192 x
// 65536 x 2048 with its gradients 6.21 -> 5.78 ms, 12800 x 32000 x 1024 568 ->
// 549 us; rows that fill half a pair's tile stay with single SMs.
int pair_of(long long rows, int bn) { return bn == 256 && rows > 128 ? 2 : 1; }
int stages_of(int bn, int cg, int bytes = kTileBytes) {
  const int n = bytes / (16384 + bn / cg * 128);
  return n < kMaxStages ? n : kMaxStages;
}
// Row tiles whose operand rows fit in half of L2 sweep the columns together.
int group_of(int K, int cg) {
  const long long g = (48ll << 20) / ((long long)128 * cg * K * 2);
  return g < 1 ? 1 : g > (1 << 20) ? 1 << 20 : (int)g;
}

// The tensor cores truncate the float32 accumulator at every K = 16 step, so
// a sum ends short of its value.  How far depends on the operands.  In units of
// 2^-24 of the value, a step, measured for K = 512 to 8192:
//   dense, of either sign    bfloat16 0.23 to 0.27, float16 0.28 to 0.36
//   one label far ahead      bfloat16 0.28, float16 0.42 to 0.69
//   sparse (5%)              bfloat16 0.02, float16 0.12
//   one-hot, small integers  0 (every partial sum is exact)
//   all of one sign          bfloat16 0.5 to 1.2, float16 1.4 to 1.75
// The factor that scales the accumulator anyway puts 0.26 back, the mean of what
// a layer norm's features lose (the mean loss at K = 2048 was 2.4e-6 off without).
// Its price: exact sums come out that much too large, 5e-7 of the value at K = 512
// and 8e-6 at 8192, as the others would come out too small without it.
constexpr double kLog2ed = 1.4426950408889634;
float factor_of(int K, double f) { return (float)(f * (1.0 + 0.26 * ((K + 15) / 16) * (1.0 / 16777216.0))); }

bool rows_aligned(const void* p, long long ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }
// Rows that tiled copies may read: they fill what lies past H only from the next 16 bytes on.
bool rows_tiled(const void* p, long long ld, int H) { return rows_aligned(p, ld) && H % 8 == 0; }

cudaError_t copy_rows(const void* in, long long ldi, void* out, int ldo, long long n, int H, cudaStream_t s) {
  const long long b = (n + 7) / 8;
  return launch(k_copy_rows, (unsigned)(b < 4864 ? b : 4864), 256, 0, s, 1, (const u16*)in, (long long)ldi, (u16*)out, ldo, n, H);
}

int check_types(int type, int param_type) {
  if (type != CTCPB_BF16 && type != CTCPB_F16) return CTCPB_EINVAL;
  if (param_type != type && param_type != CTCPB_F32) return CTCPB_EINVAL;
  return CTCPB_OK;
}
int check_dims(long long N, int V, int H) {
  if (N < 0 || N > kHeadMaxRows || V < 1 || V > kMaxV || H < 1 || H > kHeadMaxWidth) return CTCPB_EINVAL;
  return CTCPB_OK;
}
int check_ws(const void* p, size_t have, size_t need) {
  if (!p) return CTCPB_ENULL;
  if (((uintptr_t)p & 255u) != 0) return CTCPB_EALIGN;
  if (have < need) return CTCPB_ESIZE;
  return CTCPB_OK;
}

#define TRY(x)                                 \
  do {                                         \
    if ((x) != cudaSuccess) return CTCPB_ECUDA; \
  } while (0)

struct Taker {
  size_t off = sizeof(Header);
  size_t take(size_t bytes) {
    const size_t at = align_up(off, 1024);
    off = at + bytes;
    return at;
  }
};

// How a call is made in one pass: `members` workers share a row tile (a band),
// `bands` of them at once; members == 0: more columns than tensor memory holds.
// The tile's width is the one whose rounds cost least: a round takes a time
// that grows with the width, and one that does not (the members' exchange, about
// as long as 128 columns, and the reading of a sum from each member).
struct BandPlan {
  int cg, bn, members, bands;
};
BandPlan band_plan(long long N, int V) {
  BandPlan best{N > 128 ? 2 : 1, 0, 0, 0};
  const int W = kWorkers / best.cg;
  const long long mt = (N + 128 * best.cg - 1) / (128 * best.cg);
  long long cost = 0;
  for (int bn = 32; bn <= 256; bn += 16) {
    const int G = (V + bn - 1) / bn;
    if (G > W) continue;
    const int bands = (int)(W / G < mt ? W / G : mt);
    const long long c = (mt + bands - 1) / bands * (bn + (G > 1 ? 128 + G : 0));
    if (best.members == 0 || c < cost) {
      best.bn = bn;
      best.members = G;
      best.bands = bands;
      cost = c;
    }
  }
  return best;
}

struct LogpLayout {
  BandPlan band;
  int bn, nt, Hp;
  long long Np;
  size_t o_part, o_norm, o_x, o_w, total;
};
LogpLayout logp_layout(long long N, int V, int H) {
  LogpLayout l{};
  l.band = band_plan(N, V);
  l.bn = logits_bn(N, V);
  l.nt = (V + l.bn - 1) / l.bn;
  l.Hp = (int)up_to(H, 8);
  l.Np = up_to(N > 0 ? N : 1, 256);
  const size_t two = (size_t)l.nt * part_slots(l.bn), one = (size_t)l.band.members;
  Taker t;
  l.o_part = t.take((two > one ? two : one) * l.Np * 8);
  l.o_norm = t.take((size_t)l.Np * 8);
  l.o_x = t.take((size_t)N * l.Hp * 2);  // rows that no tiled copy can read are laid out here
  l.o_w = t.take((size_t)V * l.Hp * 2);
  l.total = align_up(t.off, 256);
  return l;
}

// Terms of d.  One 16-bit term puts the error of dx at 1.43 times the one that its
// rounding has anyway where few labels carry a row's sum (1.25 for V >= 5000), and at
// up to 1.7 in small calls, where no number of rows averages it out.  Two terms, the
// rounded value and what that took off, have no part in it and double the products'
// depth.  Two in calls whose products are no longer than their launch (backward, of
// a graph: 50 x 32 x 64 15.7 -> 16.7 us, 50 x 2000 x 64 23.8 -> 25.3, 1000 x 60 x 60
// 22.8 -> 26.1); beyond, 4000 rows of 8 labels and 512 features would go from 38 to 49.
int terms_of(long long Np, int V, int H) { return Np <= 1024 && Np * V * up_to(H, 64) <= 1ll << 25 ? 2 : 1; }

struct CeLayout {
  int bn, nt, Hp, pieces, piece, pbn, terms;
  long long Np;
  size_t o_ctl, o_map, o_tgt, o_xg, o_w;
  size_t o_part, o_zt, o_sums;
  size_t o_lse, o_rs, o_d, o_dbp, o_slots[2], o_acc, total;
};
CeLayout ce_layout(long long N, int V, int H, bool backward) {
  CeLayout l{};
  l.Hp = (int)up_to(H, 8);
  l.Np = up_to(N > 0 ? N : 1, 256);
  Taker t;
  l.o_ctl = t.take(256);
  l.o_map = t.take((size_t)l.Np * 4);
  l.o_tgt = t.take((size_t)l.Np * 4);
  l.o_xg = t.take((size_t)l.Np * l.Hp * 2);
  l.o_w = t.take((size_t)V * l.Hp * 2);
  l.bn = logits_bn(N, V);
  if (!backward) {
    l.nt = (V + l.bn - 1) / l.bn;
    l.o_part = t.take((size_t)l.nt * part_slots(l.bn) * l.Np * 8);
    l.o_zt = t.take((size_t)l.Np * 4);
    l.o_sums = t.take((size_t)(l.Np / 32) * 4);
  } else {
    // pieces of the vocabulary whose d takes at most 256 MB (but 256 labels at least), of equal width
    const long long most = (256ll << 20) / (l.Np * 2) / 256 * 256;
    const long long Vp = up_to(V, 256);
    l.pieces = (int)((Vp + (most > 256 ? most : 256) - 1) / (most > 256 ? most : 256));
    l.piece = (int)up_to((V + l.pieces - 1) / l.pieces, 256);
    if (l.pieces == 1) l.piece = (int)up_to(V, 64);
    l.pieces = (V + l.piece - 1) / l.piece;
    l.terms = l.pieces == 1 ? terms_of(l.Np, V, H) : 1;
    l.pbn = product_bn(H);
    const long long mt = l.Np / 128, nt = (H + l.pbn - 1) / l.pbn;
    l.o_lse = t.take((size_t)l.Np * 4);
    l.o_rs = t.take((size_t)l.Np * 4);
    l.o_d = t.take((size_t)l.Np * l.piece * 2 * l.terms);
    l.o_dbp = t.take((size_t)mt * 4 * l.piece * 4);
    for (auto& o : l.o_slots) o = t.take((size_t)2 * kWorkers * 128 * l.pbn * 4);
    l.o_acc = t.take(l.pieces > 1 ? (size_t)mt * nt * 128 * l.pbn * 4 : 0);
  }
  l.total = align_up(t.off, 256);
  return l;
}

}  // namespace
}  // namespace ctcpb

using namespace ctcpb;

extern "C" {

int ctcpb_log_probs_workspace_size(int type, int64_t N, int V, int H, size_t* bytes) {
  int rc = check_types(type, type);
  if (rc || (rc = check_dims(N, V, H))) return rc;
  if (!bytes) return CTCPB_ENULL;
  *bytes = logp_layout(N, V, H).total;
  return CTCPB_OK;
}

int ctcpb_log_probs(int type, int bias_type, const void* x, int64_t ldx, const void* weight, int64_t ldw,
                    const void* bias, int64_t N, int V, int H, float* out, int64_t ldo, void* ws, size_t ws_bytes,
                    ctcpb_stream_t stream) {
  int rc = check_types(type, bias ? bias_type : type);
  if (rc || (rc = check_dims(N, V, H))) return rc;
  if (N == 0) return CTCPB_OK;
  if (ldx < H || ldw < H || ldo < V) return CTCPB_EINVAL;
  if (!x || !weight || !out) return CTCPB_ENULL;
  const LogpLayout l = logp_layout(N, V, H);
  if ((rc = check_ws(ws, ws_bytes, l.total))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  char* b = (char*)ws;
  if (!rows_tiled(x, ldx, H)) {
    TRY(copy_rows(x, ldx, b + l.o_x, l.Hp, N, H, s));
    x = b + l.o_x;
    ldx = l.Hp;
  }
  if (!rows_tiled(weight, ldw, H)) {
    TRY(copy_rows(weight, ldw, b + l.o_w, l.Hp, V, H, s));
    weight = b + l.o_w;
    ldw = l.Hp;
  }
  CUtensorMap ma, mb, mo = {};
  GemmArgs a{};
  a.rows = (int)N;
  a.N = V;
  a.K = H;
  a.bias = bias;
  a.bias_type = bias_type;
  a.part = (float2*)(b + l.o_part);
  a.out = out;
  a.ldo = ldo;
  a.vec = ((uintptr_t)out & 15) == 0 && ldo % 4 == 0;
  a.tiled = a.vec && make_map(&mo, CTCPB_F32, out, V, N, ldo, 32);
  a.status = &((Header*)ws)->status;
  if (!make_map(&ma, type, x, l.Hp, N, ldx, 128)) return CTCPB_ECUDA;
  const int sms = sm_count();
  const BandPlan& p = l.band;
  if (p.members > 0 && sms == kWorkers) {
    if (!make_map(&mb, type, weight, l.Hp, V, ldw, p.bn / p.cg)) return CTCPB_ECUDA;
    a.bn = p.bn;
    a.stages = stages_of(p.bn, p.cg, kBandTile);
    a.factor = factor_of(H, kLog2ed);
    a.members = p.members;
    a.bands = p.bands;
    a.reset_status = 1;
    if (p.members > 1) {
      const long long n = up_to(N, 128 * p.cg) * p.members / 2, blocks = (n + 255) / 256;
      TRY(launch(k_marks, (unsigned)(blocks < 4 * kWorkers ? blocks : 4 * kWorkers), 256, 0, s, 1, (uint4*)a.part, n));
    }
    const cudaError_t e = launch_gemm<kBand>(type, p.cg, ma, mb, mo, a, p.cg * p.members * p.bands, s);
    if (e == cudaSuccess) return CTCPB_OK;
    if (e != cudaErrorCooperativeLaunchTooLarge && e != cudaErrorNotSupported) return CTCPB_ECUDA;
    (void)cudaGetLastError();  // the blocks cannot all be resident here: two passes
    a.members = 0;
    a.reset_status = 0;
  }
  const int cg = pair_of(N, l.bn);
  if (!make_map(&mb, type, weight, l.Hp, V, ldw, l.bn / cg)) return CTCPB_ECUDA;
  a.bn = l.bn;
  a.stages = stages_of(l.bn, cg);
  a.group = group_of(H, cg);
  a.part_ld = l.Np;
  a.factor = factor_of(H, 1.0);
  a.norm = (const float2*)(b + l.o_norm);
  a.reset_status = 1;
  const long long tiles = (N + 128 * cg - 1) / (128 * cg) * l.nt;
  const int blocks = cg * (int)(tiles < sms / cg ? tiles : sms / cg);
  TRY((launch_gemm<kStats>(type, cg, ma, mb, ma, a, blocks, s)));
  a.reset_status = 0;
  CombineArgs c{};
  c.rows = (int)N;
  c.part = a.part;
  c.part_ld = l.Np;
  c.slots = part_slots(l.bn) * l.nt;
  c.norm = (float2*)(b + l.o_norm);
  TRY(launch(k_combine, (unsigned)((N + 31) / 32), 32 * kSlices, 0, s, 1, c));
  a.group = 1;  // neighbours write neighbouring columns
  TRY((launch_gemm<kLogp>(type, cg, ma, mb, mo, a, blocks, s)));
  return CTCPB_OK;
}

int ctcpb_cross_entropy_workspace_size(int type, int64_t N, int V, int H, int backward, size_t* bytes) {
  int rc = check_types(type, type);
  if (rc || (rc = check_dims(N, V, H))) return rc;
  if (backward != 0 && backward != 1) return CTCPB_EINVAL;
  if (!bytes) return CTCPB_ENULL;
  *bytes = ce_layout(N, V, H, backward != 0).total;
  return CTCPB_OK;
}

}  // extern "C"

namespace {

// The checks and the row kernel that both directions share.
int ce_rows(int type, const void* x, int64_t ldx, const int32_t* targets, int64_t N, int V, int H, int32_t ignore_index,
            int reduction, const CeLayout& l, char* b, RowArgs& r, cudaStream_t s) {
  r.targets = targets;
  r.N = (int)N;
  r.V = V;
  r.H = H;
  r.ignore = ignore_index;
  r.x = (const u16*)x;
  r.ldx = ldx;
  r.vec = rows_tiled(x, ldx, H);
  r.xg = (u16*)(b + l.o_xg);
  r.ldg = l.Hp;
  r.rowmap = (int*)(b + l.o_map);
  r.tgt = (int*)(b + l.o_tgt);
  r.nv = (int*)(b + l.o_ctl);
  r.scale = (float*)(b + l.o_ctl + 4);
  r.ticket = (u32*)(b + l.o_ctl + 8);
  r.status = &((Header*)b)->status;
  r.type = type;
  r.reduction = reduction;
  r.dx_vec = r.dx && rows_aligned(r.dx, r.lddx) && H % 8 == 0;
  long long per = up_to((N + kRowBlocks - 1) / kRowBlocks, 16);
  if (per < 16) per = 16;
  const long long blocks = N > 0 ? (N + per - 1) / per : 1;
  TRY(launch(k_rows, (unsigned)blocks, 256, 0, s, 1, r, (int)per));
  return CTCPB_OK;
}

}  // namespace

extern "C" {

int ctcpb_cross_entropy(int type, int bias_type, const void* x, int64_t ldx, const void* weight, int64_t ldw,
                        const void* bias, const int32_t* targets, int64_t N, int V, int H, int32_t ignore_index,
                        int reduction, float* loss, float* lse, void* ws, size_t ws_bytes, ctcpb_stream_t stream) {
  int rc = check_types(type, bias ? bias_type : type);
  if (rc || (rc = check_dims(N, V, H))) return rc;
  if (reduction < CTCPB_REDUCE_NONE || reduction > CTCPB_REDUCE_SUM) return CTCPB_EINVAL;
  if (N == 0 && reduction == CTCPB_REDUCE_NONE) return CTCPB_OK;
  if (N > 0 && (ldx < H || ldw < H)) return CTCPB_EINVAL;
  if (!weight || !loss || (N > 0 && (!x || !targets || !lse))) return CTCPB_ENULL;
  const CeLayout l = ce_layout(N, V, H, false);
  if ((rc = check_ws(ws, ws_bytes, l.total))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  char* b = (char*)ws;
  RowArgs r{};
  if (reduction == CTCPB_REDUCE_NONE) r.loss = loss;
  r.lse = lse;
  if ((rc = ce_rows(type, x, ldx, targets, N, V, H, ignore_index, reduction, l, b, r, s))) return rc;
  if (!rows_tiled(weight, ldw, H)) {
    TRY(copy_rows(weight, ldw, b + l.o_w, l.Hp, V, H, s));
    weight = b + l.o_w;
    ldw = l.Hp;
  }
  const int cg = pair_of(N, l.bn);
  CUtensorMap ma, mb;
  if (!make_map(&ma, type, r.xg, l.Hp, l.Np, l.Hp, 128) || !make_map(&mb, type, weight, l.Hp, V, ldw, l.bn / cg))
    return CTCPB_ECUDA;
  GemmArgs a{};
  a.rows_dev = r.nv;
  a.rows = (int)N;
  a.N = V;
  a.K = H;
  a.bn = l.bn;
  a.stages = stages_of(l.bn, cg);
  a.group = group_of(H, cg);
  a.bias = bias;
  a.bias_type = bias_type;
  a.tgt = r.tgt;
  a.factor = factor_of(H, 1.0);
  a.zt = (float*)(b + l.o_zt);
  a.part = (float2*)(b + l.o_part);
  a.part_ld = l.Np;
  a.status = r.status;
  const long long tiles = l.Np / (128 * cg) * l.nt;
  const int sms = sm_count();
  TRY((launch_gemm<kStats>(type, cg, ma, mb, ma, a, cg * (int)(tiles < sms / cg ? tiles : sms / cg), s)));
  CombineArgs c{};
  c.rows_dev = r.nv;
  c.part = a.part;
  c.part_ld = l.Np;
  c.slots = part_slots(l.bn) * l.nt;
  c.lse = lse;
  c.rowmap = r.rowmap;
  c.zt = a.zt;
  c.loss = loss;
  c.reduction = reduction;
  c.sums = (float*)(b + l.o_sums);
  c.ticket = r.ticket;
  TRY(launch(k_combine, (unsigned)(l.Np / 32), 32 * kSlices, 0, s, 1, c));
  return CTCPB_OK;
}

int ctcpb_cross_entropy_backward(int type, int bias_type, const float* grad, const void* x, int64_t ldx,
                                 const void* weight, int64_t ldw, const void* bias, const int32_t* targets,
                                 const float* lse, int64_t N, int V, int H, int32_t ignore_index, int reduction,
                                 void* dx, int64_t lddx, void* dweight, int64_t lddw, void* dbias, void* ws,
                                 size_t ws_bytes, ctcpb_stream_t stream) {
  int rc = check_types(type, bias || dbias ? bias_type : type);
  if (rc || (rc = check_dims(N, V, H))) return rc;
  if (reduction < CTCPB_REDUCE_NONE || reduction > CTCPB_REDUCE_SUM) return CTCPB_EINVAL;
  if (!dx && !dweight && !dbias) return CTCPB_OK;
  if ((N > 0 && (ldx < H || (dx && lddx < H))) || ldw < H || (dweight && lddw < H)) return CTCPB_EINVAL;
  if (!weight || (N > 0 && (!x || !targets || !lse || !grad)) || (reduction != CTCPB_REDUCE_NONE && !grad))
    return CTCPB_ENULL;
  const CeLayout l = ce_layout(N, V, H, true);
  if ((rc = check_ws(ws, ws_bytes, l.total))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  char* b = (char*)ws;
  RowArgs r{};
  // with no rows and no reduction there is no gradient to read: the scale does not matter, nothing is summed
  r.grad = grad ? grad : (const float*)(b + l.o_ctl + 16);
  r.lse_in = lse;
  r.lse_c = (float*)(b + l.o_lse);
  r.rs = (float*)(b + l.o_rs);
  r.dx = (u16*)dx;
  r.lddx = lddx;
  if ((rc = ce_rows(type, x, ldx, targets, N, V, H, ignore_index, reduction, l, b, r, s))) return rc;
  if (!rows_tiled(weight, ldw, H)) {
    TRY(copy_rows(weight, ldw, b + l.o_w, l.Hp, V, H, s));
    weight = b + l.o_w;
    ldw = l.Hp;
  }
  const int cg = pair_of(N, l.bn), sms = sm_count();
  const int ldd = l.piece * l.terms, lo_at = l.terms > 1 ? l.piece : 0;  // d's rows: a term behind the other
  for (int p = 0; p < l.pieces; ++p) {
    const int v0 = p * l.piece, cols = V - v0 < l.piece ? V - v0 : l.piece;
    CUtensorMap ma, mb, mo;
    // d
    if (!make_map(&ma, type, r.xg, l.Hp, l.Np, l.Hp, 128) || !make_map(&mb, type, weight, l.Hp, V, ldw, l.bn / cg) ||
        !make_map(&mo, type, b + l.o_d, ldd, l.Np, ldd, 32))
      return CTCPB_ECUDA;
    GemmArgs a{};
    a.rows_dev = r.nv;
    a.rows = (int)N;
    a.N = cols;
    a.K = H;
    a.bn = l.bn;
    a.stages = stages_of(l.bn, cg);
    a.group = group_of(H, cg);
    a.col0 = v0;
    a.bias = bias;
    a.bias_type = bias_type;
    a.tgt = r.tgt;
    a.lse = r.lse_c;
    a.rs = r.rs;
    a.per_row = reduction == CTCPB_REDUCE_NONE;
    a.log2_r = type == CTCPB_F16 ? 15.f : 0.f;  // see k_rows
    a.one_r = type == CTCPB_F16 ? 32768.f : 1.f;
    a.factor = factor_of(H, 1.0);
    a.out = b + l.o_d;
    a.ldo = l.piece;
    a.lo_at = lo_at;
    a.tiled = 1;
    a.dbp = dbias ? (float*)(b + l.o_dbp) : nullptr;
    a.status = r.status;
    long long tiles = l.Np / (128 * cg) * ((cols + l.bn - 1) / l.bn);
    const int blocks_d = cg * (int)(tiles < sms / cg ? tiles : sms / cg);
    TRY(lo_at ? (launch_gemm<kDlogits, true>(type, cg, ma, mb, mo, a, blocks_d, s))
              : (launch_gemm<kDlogits>(type, cg, ma, mb, mo, a, blocks_d, s)));
    FinishArgs f{};
    long long left = 0;
    if (dbias) {
      f.dbp = a.dbp;
      f.ld = l.piece;
      f.rows_dev = r.nv;
      f.per = cg;
      f.cols = cols;
      f.col0 = v0;
      f.type = bias_type;
      left = f.bias_units = (cols + 31) / 32;
      f.scale = r.scale;
      f.db = dbias;
    }
    if ((dx && N > 0) || dweight) {
      // pairs where either product fills their tiles
      const int cgp = pair_of(N > cols ? N : cols, l.pbn), workers = sms / cgp;
      Params<kProduct> prm{};
      GemmArgs g{};
      g.rows_dev = r.nv;
      g.rows = (int)N;
      g.N = H;
      g.stages = stages_of(l.pbn, cgp);
      g.scale = r.scale;
      g.slots = (float*)(b + l.o_slots[0]);
      g.status = r.status;
      g.bn = l.pbn;
      g.lo_at = lo_at;
      prm.g[0] = prm.g[1] = g;
      {  // dx (+)= d w[piece]
        GemmArgs& q = prm.g[0];
        q.none = !(dx && N > 0);
        q.K = cols;
        q.group = group_of(l.piece, cgp);
        q.col0 = v0;
        q.out = dx;
        q.ldo = lddx;
        q.vec = rows_aligned(dx, lddx);
        q.rowmap = r.rowmap;
        q.acc = l.pieces > 1 ? (float*)(b + l.o_acc) : nullptr;
        q.first = p == 0;
        q.last = p == l.pieces - 1;
        if (!make_map(&prm.a[0], type, b + l.o_d, ldd, l.Np, ldd, 128) ||
            !make_map(&prm.b[0], type, weight, l.Hp, V, ldw, 64))
          return CTCPB_ECUDA;
      }
      {  // dw[piece] = d^T x
        GemmArgs& q = prm.g[1];
        q.none = !dweight;
        q.M = cols;
        q.group = 8;
        q.out = dweight ? (u16*)dweight + (long long)v0 * lddw : nullptr;
        q.ldo = lddw;
        q.vec = rows_aligned(q.out, lddw);
        q.first = q.last = 1;
        if (!make_map(&prm.a[1], type, b + l.o_d, ldd, l.Np, ldd, 64) ||
            !make_map(&prm.b[1], type, r.xg, l.Hp, l.Np, l.Hp, 64))
          return CTCPB_ECUDA;
      }
      prm.o = prm.a[0];  // (not used)
      // One launch where the tiles are few waves: one tail instead of two
      // (12000 x 5000 x 512: 93 us apart, 88 together).  With more, each its own:
      // the waves of either share what they read (8192 x 65536 x 2048 with all
      // its gradients: 5.27 ms apart, 5.50 together).
      const long long mt = (N > 0 ? N : 1), nt = (H + l.pbn - 1) / l.pbn, rows = 128 * cgp;
      const bool apart = !lo_at && ((mt + rows - 1) / rows + (cols + rows - 1) / rows) * nt > 4ll * workers;
      f.runs = 0;
      for (int run = 0; run < (apart ? 2 : 1); ++run) {
        Params<kProduct> q = prm;
        if (apart) {
          if (q.g[run].none) continue;
          q.g[1 - run].none = 2;
          q.g[run].slots = (float*)(b + l.o_slots[run]);
        }
        TRY(lo_at      ? (launch_gemm<kProduct, true>(type, cgp, q, workers * cgp, s))
            : !apart   ? launch_gemm<kProduct>(type, cgp, q, workers * cgp, s)
            : run == 0 ? launch_gemm<kDx>(type, cgp, as_mode<kDx>(q), workers * cgp, s)
                       : launch_gemm<kDw>(type, cgp, as_mode<kDw>(q), workers * cgp, s));
        f.g[f.runs][0] = q.g[0];
        f.g[f.runs][1] = q.g[1];
        ++f.runs;
      }
      // shares to join: none if neither depth (on the device, for d^T x) can be cut
      if (cols > 64 * (kSplitDepth - 1) || N > 64 * (kSplitDepth - 1)) {
        f.cg = cgp;
        f.workers = workers;
        f.units = cgp * 4 * ((l.pbn + 63) / 64);
        left += 2ll * workers * f.units;
      } else {
        f.runs = 0;
      }
    }
    const unsigned most = 10u * kWorkers, blocks = left < most ? (unsigned)left : most;
    if (left > 0)
      TRY(type == CTCPB_BF16 ? launch(k_finish<__nv_bfloat16>, blocks, 256, 0, s, 1, f)
                             : launch(k_finish<__half>, blocks, 256, 0, s, 1, f));
  }
  return CTCPB_OK;
}

}  // extern "C"
