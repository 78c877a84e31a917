// rows_io.cuh - rows of bf16, fp16 or fp32 in registers as fp32, for the operators around the products.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"
#include "grouped.h"

namespace moe {

constexpr int CHUNK = 8;   // elements of a 16-byte word of 16-bit values, the unit of aligned rows

__device__ __forceinline__ float one_value(const void* p, long long i, int dtype) {
  if (dtype == GT_FP32) return __ldcs(static_cast<const float*>(p) + i);
  const uint16_t b = __ldcs(static_cast<const uint16_t*>(p) + i);
  return dtype == GT_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ void put_value(void* p, long long i, int dtype, float v) {
  if (dtype == GT_FP32) static_cast<float*>(p)[i] = v;
  else if (dtype == GT_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}
__device__ __forceinline__ float2 two_16(uint32_t w, int dtype) {
  if (dtype == GT_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack_16(float lo, float hi, int dtype) {
  if (dtype == GT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float round_to(float v, int dtype) {
  return dtype == GT_FP32 ? v : dtype == GT_BF16 ? __bfloat162float(__float2bfloat16_rn(v)) : __half2float(__float2half_rn(v));
}

// A thread's values of a row.  Aligned rows: chunks tid + i * stride, 8 elements each; others: elements tid + j * stride.
// Values past the row are `past`.
template <int NC, bool VEC>
__device__ __forceinline__ int element_of(int j, int tid, int stride) {
  return VEC ? (tid + (j / CHUNK) * stride) * CHUNK + j % CHUNK : tid + j * stride;
}

template <int NC, bool VEC>
__device__ __forceinline__ void load_row(const void* row, int dtype, int H, int tid, int stride, float (&v)[NC * CHUNK],
                                         float past = 0.f) {
  if (!VEC) {
    // the loads of a type stand together, as a branch around each would run them one after another
    auto all = [&](auto one) {
#pragma unroll
      for (int j = 0; j < NC * CHUNK; ++j) {
        const int e = tid + j * stride;
        v[j] = e < H ? one(e) : past;
      }
    };
    if (dtype == GT_FP32) all([&](int e) { return __ldcs(static_cast<const float*>(row) + e); });
    else if (dtype == GT_BF16) all([&](int e) { return bf16_bits_to_float(__ldcs(static_cast<const uint16_t*>(row) + e)); });
    else all([&](int e) { return __half2float(__ushort_as_half(__ldcs(static_cast<const uint16_t*>(row) + e))); });
    return;
  }
  const int n = H / CHUNK;
  if (dtype == GT_FP32) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tid + i * stride;
      float4 a = make_float4(past, past, past, past), b = a;
      if (c < n) {
        a = __ldcs(static_cast<const float4*>(row) + 2 * c);
        b = __ldcs(static_cast<const float4*>(row) + 2 * c + 1);
      }
      float* d = v + i * CHUNK;
      d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
    }
    return;
  }
  uint4 raw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tid + i * stride;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (c < n) raw[i] = __ldcs(static_cast<const uint4*>(row) + c);
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    const bool in = tid + i * stride < n;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = two_16(w[q], dtype);
      v[i * CHUNK + 2 * q] = in ? f.x : past;
      v[i * CHUNK + 2 * q + 1] = in ? f.y : past;
    }
  }
}

template <int NC, bool VEC>
__device__ __forceinline__ void store_row(void* row, int dtype, int H, int tid, int stride, const float (&v)[NC * CHUNK]) {
  if (!VEC) {
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) {
      const int e = tid + j * stride;
      if (e < H) put_value(row, e, dtype, v[j]);
    }
    return;
  }
  const int n = H / CHUNK;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tid + i * stride;
    const float* s = v + i * CHUNK;
    if (c >= n) break;
    if (dtype == GT_FP32) {
      static_cast<float4*>(row)[2 * c] = make_float4(s[0], s[1], s[2], s[3]);
      static_cast<float4*>(row)[2 * c + 1] = make_float4(s[4], s[5], s[6], s[7]);
    } else {
      static_cast<uint4*>(row)[c] = make_uint4(pack_16(s[0], s[1], dtype), pack_16(s[2], s[3], dtype), pack_16(s[4], s[5], dtype),
                                               pack_16(s[6], s[7], dtype));
    }
  }
}

// y / scale rounded to nearest, inv = 1 / scale: the product's remainder added (Markstein, IBM J. Res. Dev. 34, 1990).  With the
// product alone quotients that lie on a border between two e4m3 numbers go either way, which is common for 16-bit rows: 1 value in
// 700, and an error of 3.8e-3 instead of 1.7e-3 in a bf16 product that reads them.
__device__ __forceinline__ float quotient(float y, float scale, float inv) {
  const float q = y * inv;
  return fmaf(fmaf(-q, scale, y), inv, q);
}
// e4m3, to nearest, at most 448 (NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
template <int NC, bool VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int H, int tid, int stride, const float (&v)[NC * CHUNK], float scale) {
  const float inv = 1.f / scale;
  auto q = [&](float y) { return quotient(y, scale, inv); };
  if (!VEC) {
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) {
      const int e = tid + j * stride;
      if (e < H) row[e] = (uint8_t)e4m3_pair(q(v[j]), 0.f);
    }
    return;
  }
  const int n = H / CHUNK;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tid + i * stride;
    const float* s = v + i * CHUNK;
    if (c >= n) break;
    reinterpret_cast<uint2*>(row)[c] =
        make_uint2(e4m3_pair(q(s[0]), q(s[1])) | e4m3_pair(q(s[2]), q(s[3])) << 16,
                   e4m3_pair(q(s[4]), q(s[5])) | e4m3_pair(q(s[6]), q(s[7])) << 16);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

}  // namespace moe
