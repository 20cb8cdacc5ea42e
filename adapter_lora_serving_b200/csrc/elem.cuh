// Element types of the routed layer's tensors (bf16, fp16, fp32): loads and
// stores of eight consecutive elements and single conversions.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace lora {

LORA_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
LORA_DEV float to_f32(__half v) { return __half2float(v); }
LORA_DEV float to_f32(float v) { return v; }

template <typename T>
LORA_DEV T from_f32(float v);
template <>
LORA_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
LORA_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
LORA_DEV float from_f32<float>(float v) { return v; }

LORA_DEV uint32_t pack2(__nv_bfloat16, float lo, float hi) { return pack_bf16x2(lo, hi); }
LORA_DEV uint32_t pack2(__half, float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
LORA_DEV float2 unpack2(__nv_bfloat16, uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }
LORA_DEV float2 unpack2(__half, uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// pack2 where a template also names it for fp32 (and never calls it there).
template <typename T>
LORA_DEV uint32_t pack2_any(T t, float lo, float hi) { return pack2(t, lo, hi); }
LORA_DEV uint32_t pack2_any(float, float lo, float) { return __float_as_uint(lo); }

// 16 bytes, or zeros where `valid` is false: one predicated load without a branch,
// so that several stay in flight.
LORA_DEV uint4 load16_if(const void* p, bool valid) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(valid ? 1 : 0));
  return v;
}

// Eight consecutive elements as raw words (16-byte accesses; two for fp32).
template <typename T>
struct Raw8 {
  uint4 v;
  LORA_DEV void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
  LORA_DEV void load_if(const T* p, bool valid) { v = load16_if(p, valid); }
  LORA_DEV void store(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
  LORA_DEV void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack2(T(), w[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  LORA_DEV void set(const float (&f)[8]) {
    v = make_uint4(pack2(T(), f[0], f[1]), pack2(T(), f[2], f[3]), pack2(T(), f[4], f[5]),
                   pack2(T(), f[6], f[7]));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  LORA_DEV void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  LORA_DEV void load_if(const float* p, bool valid) {
    const uint4 u = load16_if(p, valid), w = load16_if(p + 4, valid);
    a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    b = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
  }
  LORA_DEV void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  LORA_DEV void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  LORA_DEV void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

}  // namespace lora
