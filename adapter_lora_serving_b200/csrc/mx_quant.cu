// MXFP4 quantisation: 32 consecutive values of a row share a power of two,
//   scale = 2^e,  e = max(floor(log2(max |v|)) - 2, -127)   (stored as e + 127),
//   code  = round-to-nearest-even of v / 2^e to {0, .5, 1, 1.5, 2, 3, 4, 6},
// magnitudes above 6 becoming 6 (the OCP Microscaling formats, E2M1 elements
// and E8M0 scales).  v / 2^e is exact in fp32, so the codes are those of exact
// arithmetic.  A block that holds a NaN or an infinity has no scale: byte 255
// (NaN) and codes 0, and the caller's flag is raised.
//
// Memory bound: a value is read once (bf16: 2 bytes) and half a byte and 1/32
// byte written.  16384 x 4096 bf16 take 29.0 us, 26.0 being the bytes at the copy
// rate; 2048 rows of 2048 gathered to 16384, kept in bf16 too, 18.8 of 14.3; after
// SwiGLU (16384 x 768, the activation kept) 23.2 of 12.6, bound by the exponentials and
// the check of each rounding; in f16, where eight times as many values go to 64 bits,
// 29.1; in fp32, where all do, 45.7 of 24.1.
#include <type_traits>

#include "elem.cuh"
#include "experts.h"

namespace lora {

namespace {

constexpr int kQThreads = 256;
constexpr int kQPieces = 4;   // dequantisation: pieces of eight values in flight a thread

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

// Largest magnitude of eight values, as ordered bits, and those bits as fp32's.
// 16-bit types compare two at a time.
template <typename T>
struct Top {
  static LORA_DEV uint32_t of(const Raw8<T>& r) {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(r.v.x & k, r.v.y & k), __vmaxu2(r.v.z & k, r.v.w & k));
    return max(m & 0xffffu, m >> 16);
  }
  static LORA_DEV uint32_t as_f32(uint32_t m) {
    return __float_as_uint(unpack2(T(), m).x);
  }
};
template <>
struct Top<float> {
  static LORA_DEV uint32_t of(const Raw8<float>& r) {
    float f[8];
    r.get(f);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(f[k]) & 0x7fffffffu);
    return m;
  }
  static LORA_DEV uint32_t as_f32(uint32_t m) { return m; }
};

// silu(g) * u rounded once to T.  In fp32 (expf, a sum, a fast quotient, a product)
// it is within 8 ulps; where that lets it fall on either side of a rounding border
// of T (the middle of the bits that T drops), or the exponential or the result is
// near the end of fp32's range, or T is subnormal, it is computed again in 64 bits.
// Returns whether it is decided, in *out.
template <typename T>
LORA_DEV bool silu_mul_fast(float g, float u, float* out) {
  constexpr bool kBf16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
  constexpr uint32_t kDropped = kBf16 ? 0xffffu : 0x1fffu, kMiddle = kBf16 ? 0x8000u : 0x1000u;
  const float e = expf(-g);
  const float a = __fdividef(g, 1.0f + e) * u;
  *out = a;
  const bool clear = ((__float_as_uint(a) - kMiddle + 16u) & kDropped) > 32u;
  return clear && e < 0x1p100f && fabsf(a) > (kBf16 ? 0x1p-100f : 0x1p-14f) && fabsf(a) < 0x1p126f;
}
template <>
LORA_DEV bool silu_mul_fast<float>(float, float, float*) { return false; }

// The same from 64 bits: double -> fp32 -> T would round twice, so what the first
// step drops is folded into the last bit (round to odd), below T's borders.
template <typename T>
__device__ __noinline__ float silu_mul_exact(float g, float u) {
  const double d = (double)g / (1.0 + exp(-(double)g)) * (double)u;
  const float f = (float)d;
  const double back = (double)f;
  if (sizeof(T) == 4 || back == d || !(fabs(d) < (double)INFINITY)) return f;
  uint32_t b = __float_as_uint(f);
  if (fabs(back) > fabs(d)) b -= 1u;   // towards zero
  return __uint_as_float(b | 1u);
}

// What a thread takes at once: 16 values of a 16-bit type (two of them per block,
// less to do per value besides the conversions, which bound the kernel: 39 us with
// eight for 16384 x 4096 bf16), eight of fp32; and how many such pieces are in
// flight.
template <typename T>
struct Piece {
  static constexpr int kVals = sizeof(T) == 2 ? 16 : 8;
  template <bool kSilu>
  static constexpr int count() { return kSilu ? 1 : 2; }
};

// i / d for i < 2^31 by a multiplication (d >= 1): the high word of i * m, shifted.
struct Divisor {
  uint32_t d, m, shift;
  __host__ explicit Divisor(uint32_t div) : d(div), m(0), shift(0) {
    // shift = ceil(log2 d), m = ceil(2^(31 + shift) / d): exact for 31-bit i
    while ((1ull << shift) < div) ++shift;
    m = (uint32_t)(((1ull << (31 + shift)) + div - 1) / div);
  }
  LORA_DEV uint32_t operator()(uint32_t i) const {
    return (uint32_t)(((uint64_t)i * m) >> 31 >> shift);
  }
};

template <typename T, bool kSilu>
__global__ void __launch_bounds__(kQThreads)
mx_quant_kernel(const __grid_constant__ MxQuantParams p, const Divisor by_cols, int first_row) {
  constexpr int kVals = Piece<T>::kVals, kRaw = kVals / 8;
  constexpr int kPieces = Piece<T>::template count<kSilu>();
  // rows [first_row, first_row + the launch's); fewer than 2^31 pieces
  const int total = p.row_count != nullptr ? min(max(__ldg(p.row_count), 0), p.rows) : p.rows;
  const uint32_t cols = by_cols.d;   // pieces per row: whole blocks
  const uint32_t rows = (uint32_t)min(max(total - first_row, 0), (int)(0x7fffffffu / cols));
  const uint32_t n = rows * cols;
  const T* x = reinterpret_cast<const T*>(p.x);
  const size_t pitch = kSilu ? 2 * (size_t)p.F : (size_t)p.F;
  const int lane = threadIdx.x & 31;
  bool bad_row = false, bad_val = false;
  const uint32_t step = gridDim.x * (kQThreads * kPieces);
  for (uint32_t i0 = blockIdx.x * (kQThreads * kPieces); i0 < n; i0 += step) {
    Raw8<T> v[kPieces][kRaw], w[kSilu ? kPieces : 1][kRaw];
    bool live[kPieces];
    size_t at[kPieces];
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const uint32_t i = i0 + q * kQThreads + threadIdx.x;
      live[q] = i < n;
      at[q] = 0;
      if (live[q]) {
        const uint32_t r = by_cols(i);
        const uint32_t c = (i - r * cols) * kVals;
        const int row = first_row + (int)r;
        int src = row;
        if (p.row_index != nullptr) src = __ldg(p.row_index + row);
        at[q] = (size_t)row * p.F + c;
        if (src < 0 || src >= p.x_rows) {
          bad_row = true;
          live[q] = false;
        } else {
          const T* from = x + (size_t)src * pitch + c;
#pragma unroll
          for (int h = 0; h < kRaw; ++h) {
            v[q][h].load(from + 8 * h);
            if (kSilu) w[q][h].load(from + p.F + 8 * h);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      uint32_t top = 0;
      if (live[q]) {
#pragma unroll
        for (int h = 0; h < kRaw; ++h) {
          if (kSilu) {
            float g[8], u[8], a[8];
            v[q][h].get(g);
            w[q][h].get(u);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (!silu_mul_fast<T>(g[k], u[k], &a[k])) a[k] = silu_mul_exact<T>(g[k], u[k]);
            v[q][h].set(a);
          }
          top = max(top, Top<T>::of(v[q][h]));
        }
      }
      // the threads of a block are neighbours and live or dead together
      __syncwarp();
#pragma unroll
      for (int o = 1; o < 32 / kVals; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (live[q]) {
        const uint32_t bits = Top<T>::as_f32(top);
        const bool finite = bits < 0x7f800000u;
        const uint32_t ex = bits >> 23;                      // biased exponent, 0 if subnormal
        const uint32_t scale = finite ? (ex > 2u ? ex - 2u : 0u) : 255u;
        // 2^-(scale - 127): a normal number for every scale a finite block has
        const float inv = finite ? __uint_as_float((254u - scale) << 23) : 0.0f;
        uint32_t codes[kRaw];
#pragma unroll
        for (int h = 0; h < kRaw; ++h) {
          float f[8];
          v[q][h].get(f);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= inv;
          codes[h] = pack_e2m1(f);
          if (!finite) codes[h] = 0;
        }
        bad_val |= !finite;
        uint8_t* to = p.codes + (at[q] >> 1);
        if (kRaw == 2) *reinterpret_cast<uint2*>(to) = make_uint2(codes[0], codes[kRaw - 1]);
        else *reinterpret_cast<uint32_t*>(to) = codes[0];
        if ((lane & (32 / kVals - 1)) == 0) p.scales[at[q] >> 5] = (uint8_t)scale;
        if (p.rows_out != nullptr) {
#pragma unroll
          for (int h = 0; h < kRaw; ++h)
            v[q][h].store(reinterpret_cast<T*>(p.rows_out) + at[q] + 8 * h);
        }
      }
    }
  }
  if (p.flags != nullptr) {
    const uint32_t bits = (bad_row ? LORA_FLAG_BAD_ROW : 0u) | (bad_val ? LORA_FLAG_NONFINITE : 0u);
    raise_flag(p.flags, bits);
  }
}

// value = E2M1(code) * 2^(scale - 127), rounded to T (exact in bf16 and fp32).
// Memory bound: 31.2 us for 16384 x 4096 to bf16, of 26.0 at the copy rate.
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
  constexpr int kVals = Piece<T>::kVals;
  const Divisor by_cols((uint32_t)p.F / kVals);
  const int most = (int)(0x7fffffffu / by_cols.d);   // rows of one launch
  for (long long first = 0; first < p.rows; first += most) {
    const long long rows = p.rows - first < most ? p.rows - first : most;
    const bool silu = act == LORA_ACT_SILU_MUL;
    const int grid = grid_for(rows * by_cols.d, kQThreads * (silu ? Piece<T>::template count<true>()
                                                                  : Piece<T>::template count<false>()));
    if (silu)
      mx_quant_kernel<T, true><<<grid, kQThreads, 0, stream>>>(p, by_cols, (int)first);
    else
      mx_quant_kernel<T, false><<<grid, kQThreads, 0, stream>>>(p, by_cols, (int)first);
  }
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
