// adapter_mma.cuh - what the adapters' tcgen05 kernels share: asynchronous copies to
// swizzled places, descriptors and products of 16-bit operands.
#pragma once

#include "adapter_common.cuh"

namespace moe {

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
// An arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Sixteen bytes of a row that starts anywhere: the aligned words around them, to be
// put in order once they have arrived.  (Words that hold an element of the row are
// read, others not.)
struct Loose {
  uint32_t w[5];
  __device__ __forceinline__ static bool odd(const void* at) { return ((uintptr_t)at & 2) != 0; }
  // `left` elements of the row from `at` on
  __device__ __forceinline__ void load(const void* at, int left, bool on) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>((uintptr_t)at & ~(uintptr_t)3);
    const int o = odd(at);
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = on && 2 * j - o < min(left, 8) ? p[j] : 0u;
  }
  __device__ __forceinline__ uint4 chunk(bool odd, int left) const {
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = odd ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
      if (2 * j + 1 >= left) r[j] = 2 * j < left ? r[j] & 0xffffu : 0u;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};
__device__ __forceinline__ void put16(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Writes to shared memory that this thread made, or waited for, before later
// accesses of the tensor cores: to its own CTA's memory, or any in the cluster.  (A
// fence also waits for the thread's own copies in flight: the thread that issues
// the products issues no copies, or every stage would cost their whole latency.)
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_async_cluster() { asm volatile("fence.proxy.async;" ::: "memory"); }

// D[tmem] (+)= A B, both operands 16-bit in shared memory.
__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// A CTA's waits, bounded: after one that runs out, further ones end at once, and whoever
// waited in vain does no more of what it waited for.
struct Waits {
  volatile int* gave_up;
  uint64_t most;  // nanoseconds
  __device__ __forceinline__ Waits(volatile int* flag, int silent) : gave_up(flag), most(silent ? 1000000 : 2000000000) {}
  __device__ __forceinline__ bool alone(uint64_t* bar, int parity) const {  // (one lane)
    if (mbar_try_wait(bar, (uint32_t)parity)) return true;
    if (!*gave_up && mbar_wait_bounded(bar, (uint32_t)parity, gave_up, most)) return true;
    *gave_up = 1;
    return false;
  }
  __device__ __forceinline__ bool warp(uint64_t* bar, int parity) const {  // (the same for all lanes)
    return __all_sync(0xffffffffu, alone(bar, parity));
  }
  // After a wait that ran out, by all threads: copies and products on their way end
  // before what they use is given back or serves something else.  `issuer`: the
  // thread that issues the products; `last`: a barrier of one arrival.
  __device__ __forceinline__ void settle(uint64_t* last, int parity, bool issuer) const {
    copy_wait_all();
    if (issuer) {
      tc_commit(last);
      mbar_wait_bounded(last, (uint32_t)parity, nullptr, 1000000000ull);
    }
    __syncthreads();
  }
};

// Threads of the tcgen05 kernels: eight warps that copy and one whose first lane
// issues the products.
constexpr int TENSOR_THREADS = ADAPTER_THREADS + 32;

// M 128, FP32 sums; a_rows, b_rows: the operand's contraction runs across its
// rows.
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc_f16(int N, bool a_rows, bool b_rows) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_rows << 15) | ((uint32_t)b_rows << 16) |
         ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}
// Descriptor of an operand whose contraction runs across rows of 128 bytes, with
// the 128-byte swizzle: panels of 64 columns `panel` bytes apart, in a panel
// eight rows every 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t saddr, uint32_t panel = 1024) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 16-byte chunk c of a row of 128 bytes lies at chunk c ^ (row % 8).
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
  return (uint32_t)row * 128 + (uint32_t)((chunk ^ (row & 7)) << 4);
}

}  // namespace moe
