// Element access shared by the streaming kernels: fp32 or bf16 in memory, fp32 in registers.
#pragma once
#include <atomic>

#include "common.cuh"

namespace va {

__device__ __forceinline__ float elem_f(float x) { return x; }
__device__ __forceinline__ float elem_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T elem_of(float x);
template <> __device__ __forceinline__ float elem_of<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 elem_of<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements as they lie in memory, aligned to their size (at most 16 bytes).
template <class T, int N> struct alignas(sizeof(T) * N) Pack {
  static_assert(sizeof(T) * N <= 16 && (N & (N - 1)) == 0, "one access of at most 16 bytes");
  T e[N];
  __device__ __forceinline__ float operator[](int i) const { return elem_f(e[i]); }
  __device__ __forceinline__ void set(int i, float x) { e[i] = elem_of<T>(x); }
};

namespace elem_detail {
template <int BYTES> struct Word;
template <> struct Word<2> { using type = unsigned short; };
template <> struct Word<4> { using type = unsigned int; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };
}  // namespace elem_detail

template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  using Wd = typename elem_detail::Word<sizeof(T) * N>::type;
  Pack<T, N> r;
  *reinterpret_cast<Wd*>(&r) = *reinterpret_cast<const Wd*>(p);
  return r;
}
template <class T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& v) {
  using Wd = typename elem_detail::Word<sizeof(T) * N>::type;
  *reinterpret_cast<Wd*>(p) = *reinterpret_cast<const Wd*>(&v);
}
template <class T, int N>
__device__ __forceinline__ void store_pack_cs(T* p, const Pack<T, N>& v) {
  using Wd = typename elem_detail::Word<sizeof(T) * N>::type;
  __stcs(reinterpret_cast<Wd*>(p), *reinterpret_cast<const Wd*>(&v));
}

// Asynchronous copies of 16 bytes to shared memory, in groups of the thread's own.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// SMs of the current device (a device's number is asked for once).
inline int device_sms() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  sms = sms > 0 ? sms : 1;
  if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

}  // namespace va
