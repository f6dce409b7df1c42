// Activation checkpoints in 8 bits: for every head vector x of a row,
//   s = max(max |x| / 127, 2^-126),  x8 = x / s rounded to the nearest integer
// (ties to even), standing for x8 * s; a vector of zeros has x8 = 0 and
// any s.  A vector with an infinity or NaN keeps s = NaN and x8 = 0, so it reads
// back as NaN.
//
// x8 is the exact rounding of the real quotient x / s, not of its float32
// approximation: the product with an approximate reciprocal, rounded to a whole
// number by the addition of 1.5 * 2^23, gives a candidate at most one step off; the
// residue r = x - x8 s is exact in one fused multiply-add (r is a multiple of a
// power of two at most 24 bits below it), and comparing it with s / 2 settles
// the border.  Only a residue of half a scale or more, about one vector in ten
// thousand, takes the branch that corrects the candidate.
//
// Bound: HBM, s bytes read and 1 + 4 / D written per element, if the arithmetic
// stays below about eight instructions an element: hence the candidate and its
// residue two elements an instruction, and one branch a vector.  One thread per
// 16-byte vector (two of them in flight), the head's maximum over its aligned
// group of lanes by shuffles; rows are contiguous, so the tensor is one stream.
// 1M x 128 bfloat16, three tensors: 197 us, 6.3 TB/s (288 us with a division and a
// rounding per element).
#include "device.cuh"

namespace gnn {
namespace {

struct Pack8Args {
  int64_t vecs;   // 16-byte vectors of one tensor
  int hv_log2;    // vectors of a head vector
  const void* x[kPack8Max];
  int8_t* x8[kPack8Max];
  float* s[kPack8Max];
};

constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number

// Magnitude bits (infinities and NaN above all numbers) of the largest element.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const uint4& r);
template <>
__device__ __forceinline__ uint32_t top_bits<float>(const uint4& r) {
  return max(max(r.x & 0x7fffffffu, r.y & 0x7fffffffu), max(r.z & 0x7fffffffu, r.w & 0x7fffffffu));
}
template <>
__device__ __forceinline__ uint32_t top_bits<__nv_bfloat16>(const uint4& r) {
  // two at a time: a maximum that keeps NaN
  const auto two = [](uint32_t a, uint32_t b) {
    const __nv_bfloat162 x = __hmax2_nan(__habs2(*reinterpret_cast<__nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&x);
  };
  const uint32_t m = two(two(r.x, r.y), two(r.z, r.w));
  return max(m << 16, m & 0xffff0000u);
}

// max(top / 127, 2^-126).  The quotient is correctly rounded (Markstein 1990,
// "Computation of elementary functions on the IBM RISC System/6000": with c the
// rounded reciprocal and q within one step, q + (a - b q) c rounds to a / b);
// quotients below 2^-126, where the residue is not exact, give way to the bound.
__device__ __forceinline__ float scale_of(float top) {
  const float c = 0.007874015748031496f;
  const float q = __fmul_rn(top, c);
  return fmaxf(__fmaf_rn(__fmaf_rn(-127.f, q, top), c, q), 1.17549435e-38f);
}

// Candidates t[k] (whole numbers plus kWhole) for the quotients x / s, and the
// largest residue.
template <int V>
__device__ __forceinline__ float candidates(const float (&x)[V], float s, float inv,
                                            float (&t)[V], float (&r)[V]) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < V; c += 2) {
    t[c] = t[c + 1] = kWhole;
    fma2(t[c], t[c + 1], x[c], x[c + 1], inv, inv);
    float q0, q1;
    add2(q0, q1, t[c], t[c + 1], -kWhole, -kWhole);
    r[c] = x[c];
    r[c + 1] = x[c + 1];
    fma2(r[c], r[c + 1], q0, q1, -s, -s);
    most = fmaxf(most, fmaxf(fabsf(r[c]), fabsf(r[c + 1])));
  }
  return most;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pack8_rows(const __grid_constant__ Pack8Args A) {
  constexpr int V = VecOf<T>::n;
  constexpr int U = 2;
  const void* x = A.x[blockIdx.y];
  int8_t* x8 = A.x8[blockIdx.y];
  float* scales = A.s[blockIdx.y];
  const int lanes = (1 << A.hv_log2) - 1;
  for (int64_t v0 = int64_t(blockIdx.x) * (U * kThreads); v0 < A.vecs;
       v0 += int64_t(gridDim.x) * (U * kThreads)) {
    uint4 raw[U];
    uint32_t top[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kThreads + threadIdx.x;
      raw[u] = v < A.vecs ? ld16(reinterpret_cast<const char*>(x) + 16 * v)
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) top[u] = top_bits<T>(raw[u]);
    for (int o = 1; o <= lanes; o <<= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) top[u] = max(top[u], __shfl_xor_sync(kFull, top[u], o));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kThreads + threadIdx.x;
      const bool finite = top[u] < 0x7f800000u;
      const float s = scale_of(__uint_as_float(top[u]));
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      float e[V], t[V], r[V];
      unpack<T>(raw[u], e);
      const float half = 0.5f * s;
      if (candidates<V>(e, s, inv, t, r) >= half) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float a = fabsf(r[c]);
          if (a > half || (a == half && (__float_as_uint(t[c]) & 1)))
            t[c] += r[c] > 0.f ? 1.f : -1.f;
        }
      }
      // the low byte of whole + kWhole is the whole number's
      uint32_t w[V / 4];
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        const uint32_t a = __byte_perm(__float_as_uint(t[4 * c]), __float_as_uint(t[4 * c + 1]), 0x0040);
        const uint32_t b = __byte_perm(__float_as_uint(t[4 * c + 2]), __float_as_uint(t[4 * c + 3]), 0x0040);
        w[c] = finite ? __byte_perm(a, b, 0x5410) : 0u;
      }
      if (v >= A.vecs) continue;
      if constexpr (V == 8)
        reinterpret_cast<uint2*>(x8)[v] = make_uint2(w[0], w[1]);
      else
        reinterpret_cast<uint32_t*>(x8)[v] = w[0];
      if ((int(v) & lanes) == 0)
        scales[v >> A.hv_log2] = finite ? s : __int_as_float(0x7fc00000);
    }
  }
}

// One thread per kE elements (16 bytes of T, or 8 where a bfloat16 head has
// only four elements).
template <typename T, int kE>
__global__ void __launch_bounds__(kThreads)
    unpack8_rows(const int8_t* x8, const float* s, int64_t vecs, int hv_log2, void* x) {
  for (int64_t v = int64_t(blockIdx.x) * kThreads + threadIdx.x; v < vecs;
       v += int64_t(gridDim.x) * kThreads) {
    uint32_t w[kE / 4];
    if constexpr (kE == 8) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(x8) + v);
      w[0] = t.x;
      w[1] = t.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(x8) + v);
    }
    const float sc = __ldg(s + (v >> hv_log2));
    float e[kE];
#pragma unroll
    for (int c4 = 0; c4 < kE / 4; ++c4) widen8(w[c4], &e[4 * c4]);
    scale<kE>(e, sc);
    if constexpr (kE == VecOf<T>::n)
      st16(reinterpret_cast<char*>(x) + 16 * v, pack<T>(e));
    else
      reinterpret_cast<uint2*>(x)[v] = make_uint2(bf2(e[0], e[1]), bf2(e[2], e[3]));
  }
}

unsigned stream_blocks(int64_t vecs, int sm_count) {
  const int64_t want = (vecs + kThreads - 1) / kThreads, cap = int64_t(sm_count) * 32;
  return unsigned(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_pack8(int count, int64_t vecs, int hv_log2, gnn_dtype dt, const void* const* x,
                         int8_t* const* x8, float* const* s, int sm_count, cudaStream_t st) {
  Pack8Args A{};
  A.vecs = vecs;
  A.hv_log2 = hv_log2;
  for (int k = 0; k < count; ++k) {
    A.x[k] = x[k];
    A.x8[k] = x8[k];
    A.s[k] = s[k];
  }
  const dim3 grid(stream_blocks((vecs + 1) / 2, sm_count), unsigned(count));
  if (dt == GNN_F32)
    pack8_rows<float><<<grid, kThreads, 0, st>>>(A);
  else
    pack8_rows<__nv_bfloat16><<<grid, kThreads, 0, st>>>(A);
  return cudaGetLastError();
}

cudaError_t launch_unpack8(const int8_t* x8, const float* s, int64_t n, int H, int D,
                           gnn_dtype dt, void* x, int sm_count, cudaStream_t st) {
  const int e = dt == GNN_F32 || D < 8 ? 4 : 8;
  const int64_t vecs = n * H * (D / e);
  int hv_log2 = 0;
  while ((e << hv_log2) < D) ++hv_log2;
  const unsigned grid = stream_blocks(vecs, sm_count);
  if (dt == GNN_F32)
    unpack8_rows<float, 4><<<grid, kThreads, 0, st>>>(x8, s, vecs, hv_log2, x);
  else if (e == 8)
    unpack8_rows<__nv_bfloat16, 8><<<grid, kThreads, 0, st>>>(x8, s, vecs, hv_log2, x);
  else
    unpack8_rows<__nv_bfloat16, 4><<<grid, kThreads, 0, st>>>(x8, s, vecs, hv_log2, x);
  return cudaGetLastError();
}

}  // namespace gnn
