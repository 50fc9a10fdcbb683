// Tensor-core building blocks of the label head's kernels: tiled bulk copies
// (tensor maps), tcgen05 matrix instructions on tiles in shared memory with
// accumulators in tensor memory, and the element types they take.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ctcpb_async.cuh"

namespace ctcpb {

// ---------------------------------------------------------------- pairs

// Two float32 operations in one instruction, on a pair of values.
__device__ __forceinline__ u64 pair(float x, float y) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(float& x, float& y, u64 r) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r)); }
__device__ __forceinline__ float pair_sum(u64 r) {
  float x, y;
  unpair(x, y, r);
  return x + y;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// (x, y) = (x, y) * f + (bx, by)
__device__ __forceinline__ void fma2(float& x, float& y, float f, float bx, float by) {
  unpair(x, y, fma2(pair(x, y), pair(f, f), pair(bx, by)));
}
__device__ __forceinline__ void add2(float& x, float& y, float bx, float by) {
  unpair(x, y, add2(pair(x, y), pair(bx, by)));
}
__device__ __forceinline__ void add2(float& x, float& y, float b) { add2(x, y, b, b); }
__device__ __forceinline__ void mul2(float& x, float& y, float f) { unpair(x, y, mul2(pair(x, y), pair(f, f))); }

// ---------------------------------------------------------------- element types

template <class T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr u32 kFormat = 1;  // operand format code of a 16-bit matrix instruction
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ u64 unpack(u32 q) {
    return pair(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
  }
  static __device__ __forceinline__ u32 pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const u32*>(&v);
  }
};
template <>
struct Elem<__half> {
  static constexpr u32 kFormat = 0;
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ u64 unpack(u32 q) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q));
    return pair(f.x, f.y);
  }
  static __device__ __forceinline__ u32 pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const u32*>(&v);
  }
};

// Element i of an array whose type is known at run time (the small parameter
// vectors, which may be float32 beside 16-bit activations).
__device__ __forceinline__ float load_elem(const void* p, int type, long long i) {
  if (type == CTCPB_F32) return ((const float*)p)[i];
  if (type == CTCPB_BF16) return __bfloat162float(((const __nv_bfloat16*)p)[i]);
  return __half2float(((const __half*)p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, int type, long long i, float v) {
  if (type == CTCPB_F32)
    ((float*)p)[i] = v;
  else if (type == CTCPB_BF16)
    ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
  else
    ((__half*)p)[i] = __float2half_rn(v);
}

// 2^x by the hardware's instruction (its relative error, 2 ulp, is far below
// what the sums and the rounding to 16 bits add)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Programmatic launches: wait for the launch before this one on the stream to
// be done, its writes visible; let the next one's blocks begin their set-up.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// ---------------------------------------------------------------- barriers

__device__ __forceinline__ void mbar_init_n(u32 bar, u32 count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(u32 bar, u32 bytes) {
  asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n" ::"r"(bar), "r"(bytes)
               : "memory");
}
// arrive on a barrier of any block of the cluster
__device__ __forceinline__ void mbar_arrive_cluster(u32 bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_test_at(u32 bar, u32 parity) {
  u32 ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// the address, in the cluster's window, of block `rank`'s copy of a shared-memory address
__device__ __forceinline__ u32 cluster_addr(u32 addr, u32 rank) {
  u32 r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ u32 cluster_rank() {
  u32 r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// ---------------------------------------------------------------- tiled copies

// Copy the box at (x, y) of a tensor map into shared memory; x * element size
// must be a multiple of 16 bytes.  With CG = 2 the barrier may be the pair's
// other block's.
template <int CG>
__device__ __forceinline__ void tma_load(u32 dst, const CUtensorMap* map, int x, int y, u32 bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n" ::"r"(
            dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];\n" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// Copy a box from shared memory to (x, y) of a tensor map (what lies outside
// the tensor is dropped); one group a thread at a time, whose memory may be
// written again once tma_store_wait has returned.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, u32 src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(x), "r"(y),
               "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------- tcgen05

template <int CG>
__device__ __forceinline__ void tmem_alloc(u32 smem_dst, u32 cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_dst), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_dst), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(u32 tmem, u32 cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols));
}
// D (+)= A B on one K = 16 slice of 16-bit operands in shared memory.  The whole warp
// calls with the same operands, and the lane with `one` set issues: operands that
// are the warp's need no move to where the instruction takes them from.
template <int CG>
__device__ __forceinline__ void mma_f16(u32 d, u64 a, u64 b, u32 idesc, bool add, u32 one) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((u32)add), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((u32)add), "r"(one)
        : "memory");
}
// arrive on a barrier (in both blocks of a pair) once the matrix instructions issued so far are done
template <int CG>
__device__ __forceinline__ void mma_commit(u32 bar, u32 one) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
            bar),
        "h"((unsigned short)3), "r"(one)
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

// 32 columns of the warp's 32 tensor-memory lanes: thread l gets lane l's
__device__ __forceinline__ void tmem_load32(float (&v)[32], u32 addr) {
  u32* r = reinterpret_cast<u32*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// ... which are there once this has returned (the values go through it, so no
// use of them can move before it)
__device__ __forceinline__ void tmem_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// Shared-memory operand descriptor of a tile in the 128-byte swizzle (its
// 8 x 128-byte groups 1024-byte aligned), as the tiled copies write it.
//   K contiguous  (rows of 64 elements of K): 8-row groups 1024 bytes apart;
//                 the next K = 16 slice is 32 bytes on.
//   M/N contiguous (blocks of 64 elements of M or N, a row per k): the next
//                 8 k are 1024 bytes on, the next block of 64 is `block`
//                 bytes on; the next K = 16 slice is 2048 bytes on.
__device__ __forceinline__ u64 smem_desc(u32 addr, u32 lead_bytes) {
  return (u64)((addr >> 4) & 0x3fffu) | ((u64)(lead_bytes >> 4) << 16) | ((u64)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
// Instruction descriptor: float32 accumulator, 16-bit operands of one format,
// which operand is M/N contiguous, N and M.
__host__ __device__ constexpr u32 mma_idesc(u32 format, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | (format << 7) | (format << 10) | ((u32)a_mn << 15) | ((u32)b_mn << 16) | ((u32)(n >> 3) << 17) |
         ((u32)(m >> 4) << 24);
}

}  // namespace ctcpb
