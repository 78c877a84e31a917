// rows_io.cuh - rows of bf16, fp16 or fp32 in registers as fp32, for the operators around the products.
#pragma once
#include "common.cuh"
#include "grouped.h"

namespace moe {

constexpr int CHUNK = 8;   // elements of a 16-byte word of 16-bit values, the unit of aligned rows

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
// Values past the row are 0.
template <int NC, bool VEC>
__device__ __forceinline__ int element_of(int j, int tid, int stride) {
  return VEC ? (tid + (j / CHUNK) * stride) * CHUNK + j % CHUNK : tid + j * stride;
}

template <int NC, bool VEC>
__device__ __forceinline__ void load_row(const void* row, int dtype, int H, int tid, int stride, float (&v)[NC * CHUNK]) {
  if (!VEC) {
    // the loads of a type stand together, as a branch around each would run them one after another
    auto all = [&](auto one) {
#pragma unroll
      for (int j = 0; j < NC * CHUNK; ++j) {
        const int e = tid + j * stride;
        v[j] = e < H ? one(e) : 0.f;
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
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
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
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = two_16(w[q], dtype);
      v[i * CHUNK + 2 * q] = f.x;
      v[i * CHUNK + 2 * q + 1] = f.y;
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

// Word c of a row at `off` elements, as it lies: 8 elements (VEC) or one.  Predicated, not branched around, so that the loads of
// several rows are in flight together.
template <bool VEC, int TYPE>
struct Word {
  static constexpr int N = VEC ? CHUNK : 1, REGS = VEC ? (TYPE == GT_FP32 ? 8 : 4) : 1;
  uint32_t r[REGS];
  __device__ __forceinline__ void load(const void* p, long long off, int c, bool in) {
    const char* s = static_cast<const char*>(p) + (off + (long long)c * N) * (TYPE == GT_FP32 ? 4 : 2);
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < REGS; q += 4)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
            " @p ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
            : "=&r"(r[q]), "=&r"(r[q + 1]), "=&r"(r[q + 2]), "=&r"(r[q + 3])
            : "l"(s + 4 * q), "r"((uint32_t)in)
            : "memory");
    } else if constexpr (TYPE == GT_FP32) {
      asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, 0;\n @p ld.global.cs.u32 %0, [%1];\n}\n"
                   : "=&r"(r[0])
                   : "l"(s), "r"((uint32_t)in)
                   : "memory");
    } else {
      uint16_t h;
      asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u16 %0, 0;\n @p ld.global.cs.u16 %0, [%1];\n}\n"
                   : "=&h"(h)
                   : "l"(s), "r"((uint32_t)in)
                   : "memory");
      r[0] = h;
    }
  }
  __device__ __forceinline__ void store(void* p, int c) const {   // (VEC)
    uint4* d = reinterpret_cast<uint4*>(static_cast<char*>(p) + (long long)c * REGS * 4);
#pragma unroll
    for (int q = 0; q < REGS; q += 4) d[q / 4] = make_uint4(r[q], r[q + 1], r[q + 2], r[q + 3]);
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {   // (VEC) rounded to the type
#pragma unroll
    for (int i = 0; i < REGS; ++i) r[i] = TYPE == GT_FP32 ? __float_as_uint(v[i]) : pack_16(v[2 * i % N], v[(2 * i + 1) % N], TYPE);
  }
  // the largest magnitude, two at a time (16 bits, VEC); NaN is passed over, as by fmaxf
  __device__ __forceinline__ float largest() const {
    auto pair = [&](auto two) {
      using P = decltype(two);
      auto at = [&](int q) { return __habs2(*reinterpret_cast<const P*>(&r[q])); };
      return __hmax2(__hmax2(at(0), at(1 % REGS)), __hmax2(at(2 % REGS), at(3 % REGS)));
    };
    if constexpr (TYPE == GT_BF16) {
      const float2 f = __bfloat1622float2(pair(__nv_bfloat162()));
      return fmaxf(f.x, f.y);
    } else {
      const float2 f = __half22float2(pair(__half2()));
      return fmaxf(f.x, f.y);
    }
  }
  __device__ __forceinline__ float get(int i) const {   // i: a constant once unrolled
    if (TYPE == GT_FP32) return __uint_as_float(r[i]);
    const float2 f = two_16(r[i / 2], TYPE);
    return i % 2 ? f.y : f.x;
  }
};
// y / scale rounded to nearest, inv = 1 / scale: the product's remainder added (Markstein, IBM J. Res. Dev. 34, 1990).  With the
// product alone quotients that lie on a border between two e4m3 numbers go either way, which is common for 16-bit rows: 1 value in
// 700, and an error of 3.8e-3 instead of 1.7e-3 in a bf16 product that reads them.
// An infinite scale has no remainder: finite values are 0, infinite ones NaN.
struct Divisor {
  float inv, scale, back;
  __device__ __forceinline__ explicit Divisor(float s) : inv(1.f / s), scale(s < INFINITY ? s : 0.f), back(s < INFINITY ? inv : 0.f) {}
  __device__ __forceinline__ float operator()(float y) const {
    const float q = y * inv;
    return fmaf(fmaf(-q, scale, y), back, q);
  }
};
// e4m3, to nearest, at most 448 (NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3_four(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint2 e4m3_chunk(const float* s, const Divisor& by) {
  return make_uint2(e4m3_four(by(s[0]), by(s[1]), by(s[2]), by(s[3])), e4m3_four(by(s[4]), by(s[5]), by(s[6]), by(s[7])));
}
// (element by element)
template <int NC>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int H, int tid, int stride, const float (&v)[NC * CHUNK], float scale) {
  const Divisor q(scale);
#pragma unroll
  for (int j = 0; j < NC * CHUNK; ++j) {
    const int e = tid + j * stride;
    if (e < H) row[e] = (uint8_t)e4m3_four(q(v[j]), 0.f, 0.f, 0.f);
  }
}

// 8 elements of a type known at run time, from read-only or shared memory
template <bool SHARED>
__device__ __forceinline__ void chunk_of(const void* p, int c, int type, float (&v)[CHUNK]) {
  auto word = [&](int i) { return SHARED ? static_cast<const uint4*>(p)[i] : __ldg(static_cast<const uint4*>(p) + i); };
  if (type == GT_FP32) {
    const uint4 a = word(2 * c), b = word(2 * c + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    const uint4 a = word(c);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) {
      const float2 f = two_16(w[i / 2], type);
      v[i] = i % 2 ? f.y : f.x;
    }
  }
}
__device__ __forceinline__ void put_chunk(void* p, int c, int type, const float (&v)[CHUNK]) {
  if (type == GT_FP32) {
    static_cast<float4*>(p)[2 * c] = make_float4(v[0], v[1], v[2], v[3]);
    static_cast<float4*>(p)[2 * c + 1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    static_cast<uint4*>(p)[c] =
        make_uint4(pack_16(v[0], v[1], type), pack_16(v[2], v[3], type), pack_16(v[4], v[5], type), pack_16(v[6], v[7], type));
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
