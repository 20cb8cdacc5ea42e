// MXFP4 quantisation: 32 consecutive values of a row share a power of two,
//   scale = 2^e,  e = max(floor(log2(max |v|)) - 2, -127)   (stored as e + 127),
//   code  = round-to-nearest-even of v / 2^e to {0, .5, 1, 1.5, 2, 3, 4, 6},
// magnitudes above 6 becoming 6 (the OCP Microscaling formats, E2M1 elements
// and E8M0 scales).  v / 2^e is exact in fp32, so the codes are those of exact
// arithmetic.  A block that holds a NaN or an infinity has no scale: byte 255
// (NaN) and codes 0, and the caller's flag is raised.
//
// Memory bound: a value is read once (bf16: 2 bytes) and half a byte and 1/32
// byte written; a thread owns eight consecutive values (one 16-byte load), four
// threads a block, four such pieces in flight per thread.
#include "elem.cuh"
#include "experts.h"

namespace lora {

namespace {

constexpr int kQThreads = 256;
constexpr int kQPieces = 4;

// Eight values, already divided by the block's scale, as eight 4-bit codes, the
// first in the low bits.  (Four conversions packed by one mov.b32 of .b8
// registers came out wrong here, so each byte is widened on its own.)
LORA_DEV uint32_t pack_e2m1(const float (&v)[8]) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(t)
        : "f"(v[2 * i]), "f"(v[2 * i + 1]));
    r |= t << (8 * i);
  }
  return r;
}

__device__ __noinline__ double silu_mul_double(float g, float u) {
  return (double)g / (1.0 + exp(-(double)g)) * (double)u;
}

// silu(g) * u rounded once to T.  The fp32 value is within 2^-21 of it (expf,
// a sum, a division and a product) unless the exponential is near its overflow
// or the result near underflow; where moving it by 2^-20 changes what it rounds
// to, it is computed again in 64 bits.
template <typename T>
LORA_DEV T silu_mul(float g, float u) {
  const float e = expf(-g);
  const float a = g / (1.0f + e) * u;
  const T lo = from_f32<T>(a * (1.0f - 0x1p-20f)), hi = from_f32<T>(a * (1.0f + 0x1p-20f));
  if (to_f32(lo) == to_f32(hi) && e < 0x1p100f && fabsf(a) > 0x1p-100f) return lo;
  const double d = silu_mul_double(g, u);
  // double -> fp32 -> T would round twice: fold what the first step drops into
  // the last bit (round to odd), below every rounding border of T
  const float f = (float)d;
  const double back = (double)f;
  if (back == d || !(fabs(d) < (double)INFINITY)) return from_f32<T>(f);
  uint32_t b = __float_as_uint(f);
  if (fabs(back) > fabs(d)) b -= 1u;   // towards zero
  return from_f32<T>(__uint_as_float(b | 1u));
}
template <>
LORA_DEV float silu_mul<float>(float g, float u) { return (float)silu_mul_double(g, u); }

template <typename T, bool kSilu>
__global__ void __launch_bounds__(kQThreads) mx_quant_kernel(const MxQuantParams p) {
  const int cols = p.F >> 3;   // pieces per row, a multiple of four
  const int rows = p.row_count != nullptr ? min(max(__ldg(p.row_count), 0), p.rows) : p.rows;
  const long long n = (long long)rows * cols;
  const T* x = reinterpret_cast<const T*>(p.x);
  const int pitch = kSilu ? 2 * p.F : p.F;
  const int lane = threadIdx.x & 31;
  bool bad_row = false, bad_val = false;
  for (long long i0 = (long long)blockIdx.x * kQThreads * kQPieces; i0 < n;
       i0 += (long long)gridDim.x * kQThreads * kQPieces) {
    Raw8<T> v[kQPieces], w[kSilu ? kQPieces : 1];
    bool live[kQPieces];
    int row[kQPieces], col[kQPieces];
#pragma unroll
    for (int q = 0; q < kQPieces; ++q) {
      const long long i = i0 + q * kQThreads + threadIdx.x;
      live[q] = i < n;
      row[q] = 0;
      col[q] = 0;
      if (live[q]) {
        row[q] = (int)(i / cols);
        col[q] = (int)(i - (long long)row[q] * cols) * 8;
        int src = row[q];
        if (p.row_index != nullptr) src = __ldg(p.row_index + row[q]);
        if (src < 0 || src >= p.x_rows) {
          bad_row = true;
          live[q] = false;
        } else {
          v[q].load(x + (size_t)src * pitch + col[q]);
          if (kSilu) w[q].load(x + (size_t)src * pitch + p.F + col[q]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kQPieces; ++q) {
      float f[8];
      uint32_t top = 0;
      if (live[q]) {
        v[q].get(f);
        if (kSilu) {
          float u[8];
          w[q].get(u);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = to_f32(silu_mul<T>(f[k], u[k]));
          v[q].set(f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(f[k]) & 0x7fffffffu);
      }
      // the four threads of a block are neighbours and live or dead together
      __syncwarp();
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (!live[q]) continue;
      const bool finite = top < 0x7f800000u;
      const uint32_t ex = top >> 23;                       // biased exponent, 0 if subnormal
      const uint32_t scale = finite ? (ex > 2u ? ex - 2u : 0u) : 255u;
      // 2^-(scale - 127): a normal number for every scale a finite block has
      const float inv = finite ? __uint_as_float((254u - scale) << 23) : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= inv;
      uint32_t codes = pack_e2m1(f);
      if (!finite) {
        codes = 0;
        bad_val = true;
      }
      const size_t at = (size_t)row[q] * p.F + col[q];
      *reinterpret_cast<uint32_t*>(p.codes + (at >> 1)) = codes;
      if ((lane & 3) == 0) p.scales[at >> 5] = (uint8_t)scale;
      if (p.rows_out != nullptr) v[q].store(reinterpret_cast<T*>(p.rows_out) + at);
    }
  }
  if (p.flags != nullptr) {
    const uint32_t bits = (bad_row ? LORA_FLAG_BAD_ROW : 0u) | (bad_val ? LORA_FLAG_NONFINITE : 0u);
    raise_flag(p.flags, bits);
  }
}

// value = E2M1(code) * 2^(scale - 127), rounded to T (exact in bf16 and fp32).
LORA_DEV float e2m1(uint32_t code) {
  // exponent and fraction bits as an fp32 with exponent field 0..3: its value is
  // the element's times 2^-126 (a subnormal for the element's own subnormal)
  const float m = __uint_as_float((code & 7u) << 22) * 0x1p126f;
  return (code & 8u) ? -m : m;
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mx_dequant_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, T* __restrict__ out,
    long long pieces) {
  const long long stride = (long long)gridDim.x * kQThreads;
  for (long long i0 = (long long)blockIdx.x * kQThreads + threadIdx.x; i0 < pieces;
       i0 += stride * kQPieces) {
    uint32_t c[kQPieces], s[kQPieces];
#pragma unroll
    for (int q = 0; q < kQPieces; ++q) {
      const long long i = i0 + q * stride;
      c[q] = i < pieces ? __ldg(reinterpret_cast<const uint32_t*>(codes) + i) : 0u;
      s[q] = i < pieces ? __ldg(scales + (i >> 2)) : 0u;
    }
#pragma unroll
    for (int q = 0; q < kQPieces; ++q) {
      const long long i = i0 + q * stride;
      if (i >= pieces) break;
      // 2^(s - 127): subnormal for s = 0, NaN for s = 255
      const float scale = s[q] == 255u ? __uint_as_float(0x7fc00000u)
                          : s[q] == 0u ? 0x1p-127f : __uint_as_float(s[q] << 23);
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = e2m1(c[q] >> (4 * k)) * scale;
      Raw8<T> o;
      o.set(f);
      o.store(out + i * 8);
    }
  }
}

int grid_for(long long n, int per_block) {
  // enough blocks to fill the device a few times over; the rest strides
  const long long b = (n + per_block - 1) / per_block;
  return (int)(b < 148 * 16 ? (b > 0 ? b : 1) : 148 * 16);
}

template <typename T>
cudaError_t quant_typed(const MxQuantParams& p, int act, cudaStream_t stream) {
  const int grid = grid_for((long long)p.rows * (p.F >> 3), kQThreads * kQPieces);
  if (act == LORA_ACT_SILU_MUL) mx_quant_kernel<T, true><<<grid, kQThreads, 0, stream>>>(p);
  else mx_quant_kernel<T, false><<<grid, kQThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequant_typed(const uint8_t* codes, const uint8_t* scales, void* out, int rows, int F,
                          cudaStream_t stream) {
  const long long n = (long long)rows * (F >> 3);
  mx_dequant_kernel<T><<<grid_for(n, kQThreads * kQPieces), kQThreads, 0, stream>>>(
      codes, scales, reinterpret_cast<T*>(out), n);
  return cudaGetLastError();
}

}  // namespace

cudaError_t mx_quant_launch(const MxQuantParams& p, int type, int act, cudaStream_t stream) {
  if (type == LORA_TYPE_BF16) return quant_typed<__nv_bfloat16>(p, act, stream);
  if (type == LORA_TYPE_F16) return quant_typed<__half>(p, act, stream);
  return quant_typed<float>(p, act, stream);
}

cudaError_t mx_dequant_launch(const uint8_t* codes, const uint8_t* scales, void* out, int rows,
                              int F, int type, cudaStream_t stream) {
  if (type == LORA_TYPE_BF16) return dequant_typed<__nv_bfloat16>(codes, scales, out, rows, F, stream);
  if (type == LORA_TYPE_F16) return dequant_typed<__half>(codes, scales, out, rows, F, stream);
  return dequant_typed<float>(codes, scales, out, rows, F, stream);
}

}  // namespace lora
