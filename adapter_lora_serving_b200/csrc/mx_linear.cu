// Products of MXFP4 rows with MXFP4 weights on the block-scaled tensor cores:
//   y[r, n] = sum_k x[r, k] w[e(r), n, k],
// both operands 4-bit elements with a power-of-two scale per 32 of k, fp32 sums
// in tensor memory, one rounding to y's type.  One weight (a base projection),
// or one per expert with the rows sorted by expert (the base grouped product of
// a routed layer, whose output the expert fold adds to).
//
// D[128 features, BN rows] = W X^T: the weight is the M operand, so that the
// row tile (N) can follow the number of rows an expert has, 16 to 128, while
// every fetched weight tile is full.
//
// Warps: 0 loads element tiles by tensor TMA (128-byte swizzled, K-major, 256
// elements of k a stage); 2 and 3 bring the scales of the weight and x rows into
// the order the tensor core reads (32 lanes x 4 words: row 32 j + l in word j of
// lane l, a word being the scales of 128 elements); 1 copies those to tensor
// memory (tcgen05.cp) and issues the MMAs (kind::mxf4, 64 elements of k each);
// 4 to 7 drain the accumulator (two of them, so that a tile drains while the
// next one runs).
// With few tiles a cluster of `splits` CTAs shares one tile, each over its part
// of k, and the partial sums are added through distributed shared memory in
// rank order (the result does not depend on timing).
//
// Every wait is bounded; on a timeout the CTA raises LORA_FLAG_TIMEOUT, stops
// issuing, lets its copies land, frees its tensor memory and exits.
//
// Sources: spark_model/lora/expert_apply.rs, module text (the base grouped GEMM
// writes the sorted rows the fold adds to); mstar.model.components.linear
// (FusedColumnLinear, the base projection under the linear delta).
#include <cudaTypedefs.h>

#include <mutex>

#include "elem.cuh"
#include "experts.h"
#include "tcgen05.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kM = 128;               // features per tile
constexpr int kK = 256;               // elements of k per stage
constexpr int kATile = kM * kK / 2;   // 16 KB
constexpr int kSfAtom = 512;          // scales of 128 rows x 128 elements
constexpr int kAhead = 4;             // stages of scales fetched ahead
constexpr int kHeader = 6144;         // barriers, scan scratch and the experts' tile prefix (1025 ints)

template <int BN>
struct Cfg {
  static constexpr int kBTile = BN * kK / 2;
  static constexpr int kSfBytes = 4 * kSfAtom;   // two atoms of each operand
  static constexpr int kStage = kATile + kBTile + kSfBytes;
  static constexpr int kStages = BN >= 128 ? 6 : BN >= 64 ? 8 : 9;
  static constexpr int kSmem = 1024 + kHeader + kStages * kStage;   // 1024: alignment slack
  // two accumulators, then two sets of scales (8 columns each of W and of X)
  static constexpr int kCols = 2 * BN + 32 <= 64 ? 64 : 2 * BN + 32 <= 128 ? 128 : 2 * BN + 32 <= 256 ? 256 : 512;
};

struct Params {
  MxLinearParams q;
  int ftiles;       // feature tiles of a weight
  int splits;       // CTAs per tile (the cluster size)
  int kstages;      // stages of the whole k
  int per_split;    // stages of a CTA's part
};

LORA_DEV uint32_t up1024(uint32_t v) { return (v + 1023u) & ~1023u; }

// Wait that also gives up when another role of the CTA has.
LORA_DEV bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop, uint32_t* flags) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *stop = 1;
      raise_flag(flags, LORA_FLAG_TIMEOUT);
      return false;
    }
  }
  return true;
}
LORA_DEV bool warp_wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop,
                                uint32_t* flags) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_or_stop(bar, parity, stop, flags) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Instruction descriptor of kind::mxf4: both operands E2M1 (1) and K-major,
// scales UE8M0, 64 elements of k; `half` picks the lower or upper two bytes of
// the scale words.
LORA_DEV uint32_t mxf4_idesc(int N, uint32_t half) {
  return ((half * 2u) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(kM >> 7) << 27) | ((half * 2u) << 29);
}

LORA_DEV void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 rows of 16 bytes from shared memory to four columns of tensor memory, the
// same in each quarter of the lanes.
LORA_DEV void copy_scales(uint32_t taddr, uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1u << 16;          // leading byte offset (one 16-byte column: unused)
  d |= (uint64_t)(128u >> 4) << 32; // eight rows of 16 bytes to the next eight
  d |= (uint64_t)1u << 46;          // descriptor version; no swizzle
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// A tile: `rows` rows of x from row0 on times the 128 weight rows from wrow on.
struct Tile {
  int row0, rows, f0;
  int wrow;
};

struct Plan {
  const int* prefix;    // [experts + 1] tiles before each expert
  const int* offsets;
  int tiles;
};

template <int BN>
LORA_DEV Tile tile_of(const Params& p, const Plan& plan, int u) {
  Tile t;
  int e = 0, lo = 0, hi = p.q.rows;
  if (plan.offsets != nullptr) {
    e = find_segment(plan.prefix, p.q.experts, u);
    lo = plan.offsets[e];
    hi = plan.offsets[e + 1];
    u -= plan.prefix[e];
  }
  const int rt = (hi - lo + BN - 1) / BN;   // row tiles run fastest: they share the weight tile
  const int f = u / rt;
  t.row0 = lo + (u - f * rt) * BN;
  t.rows = min(BN, hi - t.row0);
  t.f0 = f * kM;
  t.wrow = e * p.q.N + t.f0;
  return t;
}

// Eight scale bytes (256 elements of k) of a row as two words, zero past the end.
LORA_DEV uint2 load_scales(const uint8_t* base, long long row, long long rows, int per_row, int at) {
  uint2 v = make_uint2(0u, 0u);
  if (row >= rows || at >= per_row) return v;
  const uint8_t* s = base + row * per_row + at;
  if ((per_row & 7) == 0) return __ldg(reinterpret_cast<const uint2*>(s));
  const int n = min(8, per_row - at);
  if ((per_row & 3) == 0) {
    v.x = __ldg(reinterpret_cast<const uint32_t*>(s));
    if (n > 4) v.y = __ldg(reinterpret_cast<const uint32_t*>(s) + 1);
    return v;
  }
  for (int i = 0; i < n; ++i) {
    const uint32_t b = __ldg(s + i);
    if (i < 4) v.x |= b << (8 * i);
    else v.y |= b << (8 * (i - 4));
  }
  return v;
}

template <int BN, typename OT>
__global__ void __launch_bounds__(kThreads, 1)
mx_linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                 const Params p) {
  typedef Cfg<BN> C;
  constexpr int kS = C::kStages;
  extern __shared__ uint8_t mx_smem[];
  uint8_t* base = mx_smem + (up1024(smem_u32(mx_smem)) - smem_u32(mx_smem));
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* empty = full + kS;
  uint64_t* accfull = empty + kS;
  uint64_t* accempty = accfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 512);
  volatile int* stop = reinterpret_cast<volatile int*>(base + 516);
  int* scratch = reinterpret_cast<int*>(base + 576);
  int* prefix = reinterpret_cast<int*>(base + 1024);   // up to 1025 ints
  uint8_t* ring = base + kHeader;
  auto a_tile = [&](int s) { return ring + s * C::kStage; };
  auto b_tile = [&](int s) { return ring + s * C::kStage + kATile; };
  auto sf_tile = [&](int s) { return ring + s * C::kStage + kATile + C::kBTile; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = p.splits;
  const int part = splits > 1 ? (int)cluster_ctarank() : 0;
  const int first_unit = (int)blockIdx.x / splits;
  const int unit_step = (int)gridDim.x / splits;
  const int ks0 = part * p.per_split;
  const int kst = min(p.kstages - ks0, p.per_split);   // >= 1

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&full[i], 3);    // the producer and the two scale warps
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], 4);
    }
    *stop = 0;
    fence_mbar_init();
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  Plan plan;
  plan.prefix = prefix;
  plan.offsets = p.q.expert_offsets;
  if (plan.offsets == nullptr) {
    plan.tiles = ((p.q.rows + BN - 1) / BN) * p.ftiles;
  } else {
    int carry = 0;
    uint32_t bad = 0;
    if (threadIdx.x == 0) prefix[0] = 0;
    for (int e0 = 0; e0 < p.q.experts; e0 += kThreads) {
      const int e = e0 + threadIdx.x;
      int cnt = 0;
      if (e < p.q.experts) {
        const int lo = plan.offsets[e], hi = plan.offsets[e + 1];
        if (lo < 0 || hi > p.q.rows || hi < lo) bad |= LORA_FLAG_BAD_OFFSETS;
        else cnt = (hi - lo + BN - 1) / BN * p.ftiles;
      }
      int tot;
      const int inc = block_inclusive_scan<kThreads>(cnt, scratch, &tot);
      if (e < p.q.experts) prefix[e + 1] = carry + inc;
      carry += tot;
    }
    if (blockIdx.x == 0) raise_flag(p.q.flags, bad);
    plan.tiles = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.tiles > first_unit ? (plan.tiles - first_unit - 1) / unit_step + 1 : 0;
  const int total = units * kst;    // stages this CTA runs

  // ---- roles; `g` counts stages over all units, so rings and phases run on ----
  if (warp == 0) {
    if (lane == 0) {
      int g = 0;
      for (int i = 0; i < units && !*stop; ++i) {
        const Tile t = tile_of<BN>(p, plan, first_unit + i * unit_step);
        for (int k = 0; k < kst; ++k, ++g) {
          const int s = g % kS;
          if (g >= kS && !wait_or_stop(&empty[s], (uint32_t)((g / kS - 1) & 1), stop, p.q.flags)) break;
          mbar_arrive_expect_tx(&full[s], kATile + C::kBTile);
          tma_load_2d(a_tile(s), &map_w, (ks0 + k) * (kK / 2), t.wrow, &full[s]);
          tma_load_2d(b_tile(s), &map_x, (ks0 + k) * (kK / 2), t.row0, &full[s]);
        }
      }
    }
  } else if (warp == 1) {
    int g = 0;
    for (int i = 0; i < units; ++i) {
      const int acc = i & 1;
      if (i >= 2 && !warp_wait_or_stop(&accempty[acc], (uint32_t)((i / 2 - 1) & 1), stop, p.q.flags)) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * BN);
      bool ok = true;
      for (int k = 0; k < kst; ++k, ++g) {
        const int s = g % kS;
        if (!(ok = warp_wait_or_stop(&full[s], (uint32_t)((g / kS) & 1), stop, p.q.flags))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sf = tmem + (uint32_t)(2 * BN + (g & 1) * 16);
          const uint32_t ssf = smem_u32(sf_tile(s));
          const int steps = min(4, (p.q.K - (ks0 + k) * kK + 63) / 64);
          for (int c = 0; c < 2; ++c) {
            copy_scales(sf + 4 * c, ssf + c * kSfAtom);
            copy_scales(sf + 8 + 4 * c, ssf + (2 + c) * kSfAtom);
          }
          const uint32_t sa = smem_u32(a_tile(s)), sb = smem_u32(b_tile(s));
          for (int j = 0; j < steps; ++j)
            mma_mxf4(d, smem_desc_kmajor(sa + j * 32, 128), smem_desc_kmajor(sb + j * 32, 128),
                     mxf4_idesc(BN, (uint32_t)(j & 1)), sf + 4 * (j >> 1), sf + 8 + 4 * (j >> 1),
                     (k > 0 || j > 0) ? 1u : 0u);
          mma_commit(&empty[s]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) mma_commit(&accfull[acc]);
      __syncwarp();
    }
  } else if (warp < 4) {
    // scales: warp 2 the weight's 128 rows, warp 3 the BN rows of x.  Lane l has
    // rows l, l + 32, l + 64, l + 96 of the tile.
    const bool of_w = warp == 2;
    const uint8_t* src = of_w ? p.q.w_scales : p.q.x_scales;
    const long long nrows = of_w ? (long long)max(p.q.experts, 1) * p.q.N : p.q.rows;
    const int per_row = p.q.K / 32;
    const int nj = of_w ? 4 : (BN + 31) / 32;
    uint2 buf[kAhead][4];
    int li = 0, lk = 0;   // next stage to fetch
    long long row = 0;
    auto fetch = [&](uint2 (&v)[4]) {
      if (li < units) {
        if (lk == 0) {
          const Tile t = tile_of<BN>(p, plan, first_unit + li * unit_step);
          row = (of_w ? t.wrow : t.row0) + lane;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nj) v[j] = load_scales(src, row + 32 * j, nrows, per_row, (ks0 + lk) * (kK / 32));
        if (++lk == kst) {
          lk = 0;
          ++li;
        }
      }
    };
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) buf[q][j] = make_uint2(0u, 0u);
      fetch(buf[q]);
    }
    bool ok = true;
    for (int g0 = 0; g0 < total && ok; g0 += kAhead) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int g = g0 + q;
        if (g < total && ok) {
          const int s = g % kS;
          if (g >= kS)
            ok = warp_wait_or_stop(&empty[s], (uint32_t)((g / kS - 1) & 1), stop, p.q.flags);
          if (ok) {
            uint8_t* dst = sf_tile(s) + (of_w ? 0 : 2 * kSfAtom) + lane * 16;
            *reinterpret_cast<uint4*>(dst) = make_uint4(buf[q][0].x, buf[q][1].x, buf[q][2].x, buf[q][3].x);
            *reinterpret_cast<uint4*>(dst + kSfAtom) =
                make_uint4(buf[q][0].y, buf[q][1].y, buf[q][2].y, buf[q][3].y);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
            fetch(buf[q]);
          }
        }
      }
    }
  } else if (splits == 1) {
    // epilogue: lane = feature, column = row of x
    const int quarter = warp & 3;
    OT* y = reinterpret_cast<OT*>(p.q.y);
    for (int i = 0; i < units; ++i) {
      const Tile t = tile_of<BN>(p, plan, first_unit + i * unit_step);
      const int acc = i & 1;
      if (!warp_wait_or_stop(&accfull[acc], (uint32_t)((i / 2) & 1), stop, p.q.flags)) break;
      tc_fence_after();
      const int f = t.f0 + quarter * 32 + lane;
      const bool f_ok = f < p.q.N;
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32) {
        if (c0 < t.rows) {   // warp-uniform
          float v[32];
          tmem_ld_32x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * BN + c0), v);
          if (f_ok) {
            OT* o = y + (size_t)(t.row0 + c0) * p.q.N + f;
#pragma unroll
            for (int n = 0; n < 32; ++n)
              if (c0 + n < t.rows) o[(size_t)n * p.q.N] = from_f32<OT>(v[n]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty[acc]);
    }
  }

  __syncwarp();
  if (*stop) {
    // given up: let copies and MMAs that are still under way land first
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Tensor map over `rows` rows of `bytes` bytes, box 128 bytes x box_rows.
cudaError_t make_map(CUtensorMap* map, const void* ptr, uint64_t bytes, uint64_t rows,
                     uint32_t box_rows, const char** why) {
  auto fn = encode_fn();
  if (fn == nullptr) {
    *why = "cuTensorMapEncodeTiled is not available";
    return cudaErrorNotSupported;
  }
  const cuuint64_t dims[2] = {bytes, rows};
  const cuuint64_t strides[1] = {bytes};
  const cuuint32_t box[2] = {kK / 2, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *why = "cuTensorMapEncodeTiled rejected the tensor";
    return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

struct DevInfo {
  int sms = 0;
};
std::mutex g_mu;
DevInfo g_dev[64];

cudaError_t dev_sms(int* dev, int* sms) {
  cudaError_t err = cudaGetDevice(dev);
  if (err != cudaSuccess) return err;
  if (*dev < 0 || *dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& d = g_dev[*dev];
  if (d.sms == 0) {
    err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, *dev);
    if (err != cudaSuccess) return err;
  }
  *sms = d.sms;
  return cudaSuccess;
}

template <int BN, typename OT>
cudaError_t launch(const MxLinearParams& q, cudaStream_t stream, const char** why) {
  typedef Cfg<BN> C;
  int dev = 0, sms = 0;
  cudaError_t err = dev_sms(&dev, &sms);
  if (err != cudaSuccess) return err;
  static bool attr[64];
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!attr[dev]) {
      err = cudaFuncSetAttribute(mx_linear_kernel<BN, OT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (err != cudaSuccess) return err;
      attr[dev] = true;
    }
  }
  const int experts = q.expert_offsets != nullptr ? q.experts : 1;
  CUtensorMap map_w, map_x;
  err = make_map(&map_w, q.w_codes, (uint64_t)q.K / 2, (uint64_t)experts * q.N, kM, why);
  if (err != cudaSuccess) return err;
  err = make_map(&map_x, q.x_codes, (uint64_t)q.K / 2, (uint64_t)q.rows, BN, why);
  if (err != cudaSuccess) return err;
  Params p = {};
  p.q = q;
  p.ftiles = (q.N + kM - 1) / kM;
  p.splits = 1;
  p.kstages = (q.K + kK - 1) / kK;
  p.per_split = p.kstages;
  // tiles there can be: every expert's last one may be partial
  const long long bound =
      ((long long)(q.rows + BN - 1) / BN + (experts > 1 ? min(experts, q.rows) : 0)) * p.ftiles;
  const int grid = (int)min((long long)sms, bound);
  mx_linear_kernel<BN, OT><<<grid, kThreads, C::kSmem, stream>>>(map_w, map_x, p);
  return cudaGetLastError();
}

template <typename OT>
cudaError_t launch_typed(const MxLinearParams& q, cudaStream_t stream, const char** why) {
  const int experts = q.expert_offsets != nullptr ? q.experts : 1;
  const long long mean = ((long long)q.rows + experts - 1) / experts;
  if (mean <= 16) return launch<16, OT>(q, stream, why);
  if (mean <= 32) return launch<32, OT>(q, stream, why);
  if (mean <= 64) return launch<64, OT>(q, stream, why);
  return launch<128, OT>(q, stream, why);
}

}  // namespace

cudaError_t mx_linear_launch(const MxLinearParams& q, int type, cudaStream_t stream,
                             const char** why) {
  if (type == LORA_TYPE_BF16) return launch_typed<__nv_bfloat16>(q, stream, why);
  if (type == LORA_TYPE_F16) return launch_typed<__half>(q, stream, why);
  return launch_typed<float>(q, stream, why);
}

}  // namespace lora
