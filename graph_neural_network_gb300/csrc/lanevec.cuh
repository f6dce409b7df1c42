// Lane vectors of kE elements of a feature row, for kernels whose Shape counts
// rows in such vectors instead of 16-byte ones.
#pragma once

#include "device.cuh"

namespace gnn {

// kE elements of a row of T, as loaded.
template <typename T, int kE>
struct RawT {
  uint4 v[kE * int(sizeof(T)) / 16];
};

template <typename T, int kE>
__device__ __forceinline__ RawT<T, kE> ldT(const void* p, int64_t node, const Shape& s,
                                           const Lane<1>& L, bool ok) {
  RawT<T, kE> r;
  constexpr int n = kE * int(sizeof(T)) / 16;
  const char* at = reinterpret_cast<const char*>(p) + (node * s.rv + L.q[0]) * (kE * sizeof(T));
#pragma unroll
  for (int k = 0; k < n; ++k) r.v[k] = ok ? ld16(at + 16 * k) : make_uint4(0, 0, 0, 0);
  return r;
}

template <typename T, int kE>
__device__ __forceinline__ void widenT(const RawT<T, kE>& r, float (&x)[kE]) {
  constexpr int V = VecOf<T>::n;
#pragma unroll
  for (int k = 0; k < kE / V; ++k) unpack<T>(r.v[k], *reinterpret_cast<float(*)[V]>(x + V * k));
}

template <typename T, int kE>
__device__ __forceinline__ void storeT(void* p, int64_t node, const Shape& s, const Lane<1>& L,
                                       const float (&x)[kE]) {
  constexpr int V = VecOf<T>::n;
  char* at = reinterpret_cast<char*>(p) + (node * s.rv + L.q[0]) * (kE * sizeof(T));
#pragma unroll
  for (int k = 0; k < kE / V; ++k)
    st16(at + 16 * k, pack<T>(*reinterpret_cast<const float(*)[V]>(x + V * k)));
}

// Dot product with a vector held for many edges: bfloat16 stays packed on both
// sides (every product is exact in float32), float32 is widened already.
template <typename T, int kE>
struct HeldT {
  float x[kE];
  __device__ __forceinline__ void set(const RawT<T, kE>& r) { widenT<T, kE>(r, x); }
  __device__ __forceinline__ float dot_with(const RawT<T, kE>& r) const {
    float y[kE];
    widenT<T, kE>(r, y);
    return dot<kE>(y, x);
  }
};
template <int kE>
struct HeldT<__nv_bfloat16, kE> {
  RawT<__nv_bfloat16, kE> x;
  __device__ __forceinline__ void set(const RawT<__nv_bfloat16, kE>& r) { x = r; }
  __device__ __forceinline__ float dot_with(const RawT<__nv_bfloat16, kE>& r) const {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(&x);
    const uint32_t* b = reinterpret_cast<const uint32_t*>(&r);
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int w = 0; w < kE / 2; ++w)
      asm("{\n .reg .b16 al, ah, bl, bh;\n mov.b32 {al, ah}, %2;\n mov.b32 {bl, bh}, %3;\n"
          " fma.rn.f32.bf16 %0, al, bl, %0;\n fma.rn.f32.bf16 %1, ah, bh, %1;\n}"
          : "+f"(d0), "+f"(d1)
          : "r"(a[w]), "r"(b[w]));
    return d0 + d1;
  }
};

// The geometry of rows of s in vectors of e elements (a power of two dividing D).
inline Shape lane_shape(const Shape& s, int e) {
  Shape w = s;
  w.hv = s.D / e;
  w.rv = s.H * w.hv;
  w.nv = 1;
  w.hv_log2 = 0;
  while ((1 << w.hv_log2) < w.hv) ++w.hv_log2;
  w.lpr_log2 = 0;
  while ((1 << w.lpr_log2) < w.rv) ++w.lpr_log2;
  w.lpr = 1 << w.lpr_log2;
  return w;
}

}  // namespace gnn
