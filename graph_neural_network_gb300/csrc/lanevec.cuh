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

// This lane's part of the rows of a tensor: kBytes at a fixed place of every row.
// (A lane beyond the row's vectors reads the first one, for nothing.)
template <int kBytes>
struct LanePlace {
  uint32_t off, stride;
  __device__ __forceinline__ LanePlace(const Shape& s, const Lane<1>& L)
      : off(L.ok[0] ? uint32_t(L.q[0]) * kBytes : 0u), stride(uint32_t(s.rv) * kBytes) {}
  // the same place of another tensor's row
  __device__ __forceinline__ const char* of(const void* p, int node) const {
    return static_cast<const char*>(p) + (uint64_t(uint32_t(node)) * stride + off);
  }
};
// ... of one tensor that is gathered.
template <int kBytes>
struct LaneRows {
  const char* base;
  uint32_t stride;
  __device__ __forceinline__ LaneRows(const void* p, const LanePlace<kBytes>& at)
      : base(static_cast<const char*>(p) + at.off), stride(at.stride) {}
  __device__ __forceinline__ const char* at(int node) const {
    return base + uint64_t(uint32_t(node)) * stride;
  }
};

// (Vectors of 32 bytes or more: one load per 32, from 32-byte boundaries.)
template <typename T, int kE>
__device__ __forceinline__ RawT<T, kE> ldT(const char* at) {
  RawT<T, kE> r;
  constexpr int n = kE * int(sizeof(T)) / 16;
  if constexpr (n % 2 == 0) {
#pragma unroll
    for (int k = 0; k < n; k += 2) {
      const RawV<32> t = ldv<32>(at + 16 * k);
      r.v[k] = t.a;
      r.v[k + 1] = t.b;
    }
  } else {
#pragma unroll
    for (int k = 0; k < n; ++k) r.v[k] = ld16(at + 16 * k);
  }
  return r;
}

template <typename T, int kE>
__device__ __forceinline__ void widenT(const RawT<T, kE>& r, float (&x)[kE]) {
  constexpr int V = VecOf<T>::n;
#pragma unroll
  for (int k = 0; k < kE / V; ++k) unpack<T>(r.v[k], *reinterpret_cast<float(*)[V]>(x + V * k));
}

template <typename T, int kE>
__device__ __forceinline__ void storeT(char* at, const float (&x)[kE]) {
  constexpr int V = VecOf<T>::n;
#pragma unroll
  for (int k = 0; k < kE / V; ++k)
    st16(at + 16 * k, pack<T>(*reinterpret_cast<const float(*)[V]>(x + V * k)));
}

// Dot product of two lane vectors: bfloat16 stays packed on both sides (every
// product is exact in float32), float32 as it is.
template <int kE>
__device__ __forceinline__ float dotT(const RawT<float, kE>& a, const RawT<float, kE>& b) {
  float x[kE], y[kE];
  widenT<float, kE>(a, x);
  widenT<float, kE>(b, y);
  return dot<kE>(x, y);
}
template <int kE>
__device__ __forceinline__ float dotT(const RawT<__nv_bfloat16, kE>& p,
                                      const RawT<__nv_bfloat16, kE>& q) {
  const uint32_t* a = reinterpret_cast<const uint32_t*>(&p);
  const uint32_t* b = reinterpret_cast<const uint32_t*>(&q);
  float d0 = 0.f, d1 = 0.f;
#pragma unroll
  for (int w = 0; w < kE / 2; ++w)
    asm("{\n .reg .b16 al, ah, bl, bh;\n mov.b32 {al, ah}, %2;\n mov.b32 {bl, bh}, %3;\n"
        " fma.rn.f32.bf16 %0, al, bl, %0;\n fma.rn.f32.bf16 %1, ah, bh, %1;\n}"
        : "+f"(d0), "+f"(d1)
        : "r"(a[w]), "r"(b[w]));
  return d0 + d1;
}

// A lane vector of a node's own row kept in shared memory, in 16-byte parts of the
// lane's own (512 bytes apart, one lane's next to the other's): copied there
// asynchronously, so that the change of nodes waits for nothing, and no
// registers between its uses.
template <typename T, int kE>
struct HeldT {
  static constexpr int kParts = kE * int(sizeof(T)) / 16;
  static constexpr int kBytes = 512 * kParts;  // of a warp
  uint32_t at;
  __device__ __forceinline__ void place(const unsigned char* warp, int lane) {
    at = uint32_t(__cvta_generic_to_shared(warp)) + 16 * lane;
  }
  __device__ __forceinline__ void fetch(const char* from) {
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(at + 512 * k),
                   "l"(from + 16 * k)
                   : "memory");
  }
  // values computed by this lane
  __device__ __forceinline__ void put(const float (&x)[kE]) {
    constexpr int V = VecOf<T>::n;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const uint4 v = pack<T>(*reinterpret_cast<const float(*)[V]>(x + V * k));
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 512 * k), "r"(v.x),
                   "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    }
  }
  // after held_ready() or put()
  __device__ __forceinline__ RawT<T, kE> get() const {
    RawT<T, kE> r;
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.v[k].x), "=r"(r.v[k].y), "=r"(r.v[k].z), "=r"(r.v[k].w)
                   : "r"(at + 512 * k)
                   : "memory");
    return r;
  }
};

// Waits for this lane's copies.
__device__ __forceinline__ void held_ready() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// P = f (P - d Q)
template <int kE>
__device__ __forceinline__ void minus_scaled(float (&P)[kE], const float (&Q)[kE], float d, float f) {
  scale<kE>(P, f);
  axpy<kE>(P, -f * d, Q);
}

// 1 / x to within an ulp of float32 (x a sum of weights: from 2^-126 to 2^31).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

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
