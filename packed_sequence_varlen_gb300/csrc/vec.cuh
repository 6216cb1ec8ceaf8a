// Small vectors of fp32 in registers with packed arithmetic.
#pragma once
#include "elem.cuh"

namespace va {

// V numbers at a time, two an instruction; each result is rounded by itself, whatever the code around it.
template <int V> struct Vec {
  static_assert(V % 2 == 0, "pairs");
  float e[V];
  __device__ __forceinline__ float& operator[](int i) { return e[i]; }
  __device__ __forceinline__ const float& operator[](int i) const { return e[i]; }
};
template <int V>
__device__ __forceinline__ Vec<V> fill(float x) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = x;
  return r;
}
template <class T, int V>
__device__ __forceinline__ Vec<V> wide_of(const Pack<T, V>& p) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = p[i];
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> add(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
        " add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"  // (.rn: never folded into a product)
        : "=f"(r[i]), "=f"(r[i + 1])
        : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> fma(const Vec<V>& a, const Vec<V>& b, const Vec<V>& c) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; i += 2) ffma2(r[i], r[i + 1], a[i], a[i + 1], b[i], b[i + 1], c[i], c[i + 1]);
  return r;
}
// (a product as a fused one with -0 added: it is never fused with a sum that follows)
template <int V>
__device__ __forceinline__ Vec<V> mul(const Vec<V>& a, const Vec<V>& b) {
  return fma(a, b, fill<V>(-0.f));
}
template <class T, int V>
__device__ __forceinline__ Pack<T, V> narrow(const Vec<V>& v) {
  Pack<T, V> r;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) reinterpret_cast<uint32_t*>(&r)[i / 2] = pack_bf16(v[i], v[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.set(i, v[i]);
  }
  return r;
}

}  // namespace va
