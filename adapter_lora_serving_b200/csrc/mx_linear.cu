// Products of MXFP4 rows with MXFP4 weights on the block-scaled tensor cores:
//   y[r, n] = sum_k x[r, k] w[e(r), n, k],
// both operands 4-bit elements with a power-of-two scale per 32 of k, fp32 sums
// in tensor memory, one rounding to y's type.  One weight (a base projection),
// or one per expert with the rows sorted by expert (the base grouped product of
// a routed layer, whose output the expert fold adds to).
//
// D[128 features, BN rows] = W X^T: the weight is the M operand, so that the row
// tile (N, 16 to 256) can follow the number of rows an expert has while every
// fetched weight tile is full; a tile that an expert's end cuts short computes its
// rows in 32s.
//
// Warps: one loads element tiles by tensor TMA (128-byte swizzled, K-major, 256
// elements of k a stage); one the raw scales (512 elements of k a block: 16 bytes a
// row, by TMA, or by asynchronous copies where the rows' pitch is no multiple of
// 16); two put those in the order the tensor core reads (32 lanes x 4 words: row
// 32 j + l in word j of lane l, a word being the scales of 128 elements); one thread
// copies them to tensor memory (tcgen05.cp) and issues the MMAs (kind::mxf4, 64
// elements of k each); four or eight warps drain the accumulator (two of them up to
// 128 rows, so that a tile drains while the next one runs), turn it with stmatrix
// and store 16 bytes of features a lane.  The issuing thread's work per stage is
// what the first version of this kernel spent its time on (a stage of 128 x 128
// took 1270 cycles, 270 being the tensor core's): its descriptors are additions to
// precomputed words.
//
// What bounds it.  Few rows: the weight's bytes (32 tokens x 8 of 128 experts, 2048
// by 1536: 166 MB in 31.2 us, 5.3 TB/s with start and end; one row of 4096 by 28672:
// 14.7 us, 9.6 being its 62.5 MB at the copy rate).  Where there are fewer tiles
// than SMs a cluster of `splits` CTAs shares a tile, each over its part of k, and
// the partial sums are added through distributed shared memory in rank order (the
// result does not depend on timing): 128 rows of 14336 by 4096 take 13.4 us instead
// of 18.4.  Many rows: a 128 x 256 tile of one CTA is bound by shared memory (12 KB
// read and 12 written per MMA of 135 cycles); two CTAs on one tile of 256 x 256
// (below) take 8 and 8: 8192 rows of 4096 by 28672 in 358 us (5.4 PFLOP/s; 408 with
// one CTA a tile), or 421 us where it runs long enough to meet the power limit.
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

constexpr int kM = 128;               // features per tile
constexpr int kK = 256;               // elements of k per stage of element tiles
constexpr int kATile = kM * kK / 2;   // 16 KB
constexpr int kBlockK = 512;          // elements of k per block of scales (16 bytes a row)
constexpr int kSfAtom = 512;          // scales of 128 rows x 128 elements
constexpr int kTurn = 1024;            // an epilogue warp's 16 rows x 32 features of 16 bits
constexpr int kHeader = 6144;         // barriers, scan scratch and the experts' tile prefix (1025 ints)
constexpr int kOffsets = 4608;        // a copy of the experts' offsets (1025 ints)

template <int BN>
struct Cfg {
  static constexpr int kBTile = BN * kK / 2;
  static constexpr int kStage = kATile + kBTile;
  static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 6 : BN >= 64 ? 8 : BN >= 32 ? 9 : 8;
  static constexpr int kSfSlots = BN >= 64 ? 3 : 5;   // blocks of scales in flight
  // the experts' offsets in shared memory, where there is room: a tile is looked up
  // by every role, from global memory in about a thousand cycles
  static constexpr bool kOwnOffsets = BN <= 128;
  static constexpr int kAtoms = BN > 128 ? 2 : 1;             // of x, per 128 elements of k
  // a slot: raw rows of 16 bytes, or (up to 128 rows) of the 20 around 16 unaligned
  // ones, W's then X's; put in order in place
  static constexpr int kSfX0 = BN > 128 ? 4 * kSfAtom : kM * 20;
  static constexpr int kSfSlot = BN > 128 ? 12 * kSfAtom : 2 * kM * 20;
  static constexpr int kAcc = BN > 128 ? 1 : 2;               // accumulators
  static constexpr int kSfCols = 16 + 16 * kAtoms;            // tensor memory columns of a block of scales
  static constexpr int kUsed = kAcc * BN + 2 * kSfCols;
  static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static constexpr int kEpiWarps = BN >= 64 ? 8 : 4;
  static constexpr int kWarpCols = BN >= 64 ? BN / 2 : 32;    // columns an epilogue warp drains
  static constexpr int kThreads = 160 + 32 * kEpiWarps;       // and the scales' producer
  static constexpr int kSmem = 1024 + kHeader + kStages * kStage + kSfSlots * kSfSlot +
                               kEpiWarps * kTurn + (kOwnOffsets ? kOffsets : 0);   // 1024: alignment slack
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

enum ScaleCopy { kByTma = 0, kBy8 = 8, kBy4 = 4, kAround = 1 };

struct Params {
  MxLinearParams q;
  int ftiles;       // feature tiles of a weight
  int most;         // tiles that offsets which do not overlap can make
  int splits;       // CTAs per tile (the cluster size)
  int blocks;       // 512-element blocks of the whole k
  int per_split;    // blocks of a CTA's part
  int scale_copy;   // how scales come: by TMA, by asynchronous copies of 8 or 4 bytes, or of the
                    // words around them
};

LORA_DEV uint32_t up1024(uint32_t v) { return (v + 1023u) & ~1023u; }

// Phase test with a long suspension of the waiting thread (20 us at most; a dozen
// warps wait most of the time, and their polling costs power, that is clock: 34.7
// us against 34.1 for 32 x 8 rows of 128 experts).  CLUSTER: for arrivals of
// another CTA, with what its shared memory held before them (the fence is for shared
// memory alone: an acquire at cluster scope drops the L1 cache with every wait).
template <bool CLUSTER>
LORA_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "fence.acquire.sync_restrict::shared::cluster.cluster;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
  return ok != 0;
}

// Wait that also gives up when another role of the CTA has.  The clock is looked
// at only now and then.
template <bool CLUSTER = false>
LORA_DEV bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop, uint32_t* flags) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_test<CLUSTER>(bar, parity); ++i) {
    if (*stop) return false;
    if ((i & 15u) == 0u) {
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *stop = 1;
        raise_flag(flags, LORA_FLAG_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}

// The same for a whole warp, whose lanes go on or give up together: collective
// instructions follow, and one lane can see its time run out when another does not.
// (Most waits end in their first test: 2048 x 8 rows of 768 by 2048 43.3 us, 43.8 with
// the vote behind the loop alone, 43.1 without one.)
template <bool CLUSTER = false>
LORA_DEV bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* stop, uint32_t* flags) {
  if (__all_sync(0xffffffffu, mbar_test<CLUSTER>(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_or_stop<CLUSTER>(bar, parity, stop, flags));
}

// The same barrier of the cluster's first CTA, and an arrival there.
LORA_DEV uint32_t at_first(const uint64_t* bar) { return dsmem_addr(bar, 0); }
// For what this CTA's warp wrote to its shared memory (RELEASE), or for accesses to
// tensor memory, which the tcgen05 fences around an arrival and its wait order.  The
// release is for shared memory alone: one of all memory takes over a microsecond, 488
// us for 8192 x 4096 x 28672 with one for every block of scales, 361 as here.
template <bool RELEASE>
LORA_DEV void arrive_at_first(const uint64_t* bar) {
  if (RELEASE) asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(at_first(bar))
               : "memory");
}
// A ring position and the parity of its current round.
struct Ring {
  int s = 0;
  uint32_t round = 0;
  template <int N>
  LORA_DEV void next() {
    if (++s == N) {
      s = 0;
      round ^= 1u;
    }
  }
};

// A tile: `rows` rows of x from row0 on times the 128 weight rows from wrow on.
struct Tile {
  int row0, rows, f0;
  int wrow;
};

// Instruction descriptor of kind::mxf4: both operands E2M1 (1) and K-major,
// scales UE8M0, 64 elements of k, M x N.  `half` picks the lower or upper two bytes
// of the scale words.
LORA_DEV uint32_t mxf4_idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}
constexpr uint32_t mxf4_half(int half) { return ((uint32_t)half << 5) | ((uint32_t)half << 30); }

// Columns that a tile's MMAs compute: its rows in 32s (a tile that an expert's end
// cuts short costs as much less).
LORA_DEV int columns_of(const Tile& t, int most) { return min(most, (t.rows + 31) & ~31); }

// Shared-memory matrix descriptors: the low word holds the address / 16 (and the
// unused leading offset), the high word is a constant.
constexpr uint32_t kDescTile = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kDescScale = (128u >> 4) | (1u << 14);               // 8 rows of 16 bytes, no swizzle
LORA_DEV uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }

LORA_DEV void mma_mxf4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa,
                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %7};\n\t"
      "mov.b64 b, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescTile)
      : "memory");
}

// 32 rows of 16 bytes from shared memory to four columns of tensor memory, the
// same in each quarter of the lanes.
LORA_DEV void copy_scales(uint32_t taddr, uint32_t lo) {
  asm volatile(
      "{\n\t.reg .b64 d;\n\t"
      "mov.b64 d, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
      "r"(lo), "r"(kDescScale)
      : "memory");
}

// One lane of the (converged) warp.
LORA_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

struct Plan {
  const int* prefix;    // [experts + 1] tiles before each expert
  const int* offsets;
  int tiles;
};

// Tiles of BN rows before each expert (the whole CTA; __syncthreads follows).
template <int BN, int THREADS>
LORA_DEV Plan make_plan(const Params& p, int* prefix, int* scratch, int* own_offsets = nullptr) {
  Plan plan = {prefix, p.q.expert_offsets, 0};
  if (plan.offsets == nullptr) {
    plan.tiles = ((p.q.rows + BN - 1) / BN) * p.ftiles;
    return plan;
  }
  uint32_t bad = 0;
  if (threadIdx.x == 0) prefix[0] = 0;
  for (int e0 = 0; e0 < p.q.experts; e0 += THREADS) {
    const int e = e0 + (int)threadIdx.x;
    int cnt = 0;
    if (e < p.q.experts) {
      const int lo = plan.offsets[e], hi = plan.offsets[e + 1];
      if (own_offsets != nullptr) {
        own_offsets[e] = lo;
        if (e + 1 == p.q.experts) own_offsets[e + 1] = hi;
      }
      if (lo < 0 || hi > p.q.rows || hi < lo) bad |= LORA_FLAG_BAD_OFFSETS;
      else cnt = (hi - lo + BN - 1) / BN * p.ftiles;
    }
    int tot;
    const int inc = block_inclusive_scan<THREADS>(cnt, scratch, &tot);
    if (e < p.q.experts) prefix[e + 1] = plan.tiles + inc;
    plan.tiles += tot;
  }
  if (__syncthreads_or(bad != 0)) {
    // Offsets that go back can make blocks overlap, and more tiles than there is
    // room for: counted again one by one, leaving out experts beyond that.
    if (threadIdx.x == 0) {
      int tiles = 0;
      for (int e = 0; e < p.q.experts; ++e) {
        const int lo = plan.offsets[e], hi = plan.offsets[e + 1];
        if (lo >= 0 && hi <= p.q.rows && hi >= lo) {
          const long long cnt = (long long)((hi - lo + BN - 1) / BN) * p.ftiles;
          if (tiles + cnt <= p.most) tiles += (int)cnt;
        }
        prefix[e + 1] = tiles;
      }
    }
    __syncthreads();
    plan.tiles = prefix[p.q.experts];
  }
  if (blockIdx.x == 0) raise_flag(p.q.flags, bad);
  if (own_offsets != nullptr) plan.offsets = own_offsets;   // (after the barriers above)
  return plan;
}

template <int BN, int FEATURES = kM>
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
  const int f = rt == 1 ? u : u / rt;
  t.row0 = lo + (u - f * rt) * BN;
  t.rows = min(BN, hi - t.row0);
  t.f0 = f * FEATURES;
  t.wrow = e * p.q.N + t.f0;
  return t;
}

// Rows' scale bytes in the order the tensor core reads, into a slot (the whole warp):
// lane l has rows l, l + 32, l + 64, l + 96 of an atom (v[atom][j]); word c of row
// 32 j + l becomes word j of lane l of atom c.  Visible to tcgen05.cp on return.
template <int ATOMS>
LORA_DEV void write_ordered(uint8_t* slot, const uint4 (&v)[ATOMS][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < ATOMS; ++h) {
    uint8_t* dst = slot + h * kSfAtom + lane * 16;
    constexpr int kStep = ATOMS * kSfAtom;
    *reinterpret_cast<uint4*>(dst) = make_uint4(v[h][0].x, v[h][1].x, v[h][2].x, v[h][3].x);
    *reinterpret_cast<uint4*>(dst + kStep) = make_uint4(v[h][0].y, v[h][1].y, v[h][2].y, v[h][3].y);
    *reinterpret_cast<uint4*>(dst + 2 * kStep) =
        make_uint4(v[h][0].z, v[h][1].z, v[h][2].z, v[h][3].z);
    *reinterpret_cast<uint4*>(dst + 3 * kStep) =
        make_uint4(v[h][0].w, v[h][1].w, v[h][2].w, v[h][3].w);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Raw scales of a tile put in order, in place, block after block.  (Rows past the
// tile's are whatever the slot held: their products are not stored.)
template <int ATOMS, int SLOTS, bool PAIR = false>
LORA_DEV void order_scales(uint8_t* ring, int slot_bytes, uint64_t* raw, uint64_t* ready,
                           volatile int* stop, uint32_t* flags, int total) {
  const int lane = threadIdx.x & 31;
  Ring b;
  for (int n = 0; n < total; ++n) {
    uint8_t* slot = ring + b.s * slot_bytes;
    if (!warp_wait(&raw[b.s], b.round, stop, flags)) break;
    uint4 v[ATOMS][4];
#pragma unroll
    for (int h = 0; h < ATOMS; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[h][j] = *reinterpret_cast<const uint4*>(slot + (h * 128 + j * 32 + lane) * 16);
    __syncwarp();
    write_ordered<ATOMS>(slot, v);
    if (lane == 0) {
      if (PAIR) arrive_at_first<true>(&ready[b.s]);
      else mbar_arrive(&ready[b.s]);
    }
    b.next<SLOTS>();
  }
}

// ROWS rows' 16 scale bytes from byte `at` of row row0 on into a slot (the whole
// warp), zeros past a row's end and past the last row: copies of N bytes that land
// later (arriving on `raw`, 32 arrivals), for row pitches that are multiples of N.
template <int N, int ROWS>
LORA_DEV void copy_scale_rows(uint8_t* slot, const uint8_t* src, long long row0, long long nrows,
                              int per_row, int at, uint64_t* raw) {
  const int lane = threadIdx.x & 31;
  const int rows = (int)min((long long)ROWS, nrows - row0);
  const int bytes = per_row - at;
  const uint8_t* s = src + (row0 + lane) * per_row + at;
  uint32_t to = smem_u32(slot + lane * 16);
#pragma unroll
  for (int r = 0; r < ROWS; r += 32) {
    const bool valid = r + lane < rows;
    if (ROWS >= 32 || lane < ROWS) {
#pragma unroll
      for (int o = 0; o < 16; o += N) {
        const bool some = valid && o < bytes;
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to + o),
                     "l"(some ? s + o : src), "n"(N), "r"(some ? N : 0)
                     : "memory");
      }
    }
    s += 32 * per_row;
    to += 32 * 16;
  }
  cp_async_arrive_noinc(raw);
}

// The same for any pitch: the five aligned words around a row's 16 bytes, to rows of
// 20.  Nothing past `end`, the array's, is read.
template <int ROWS>
LORA_DEV void copy_scale_words(uint8_t* slot, const uint8_t* src, const uint8_t* end, long long row0,
                               long long nrows, int per_row, int at, uint64_t* raw) {
  const int lane = threadIdx.x & 31;
  const int rows = (int)min((long long)ROWS, nrows - row0);
  const uint8_t* s = src + (row0 + lane) * per_row + at;
  uint32_t to = smem_u32(slot + lane * 20);
#pragma unroll
  for (int r = 0; r < ROWS; r += 32) {
    const bool valid = r + lane < rows;
    if (ROWS >= 32 || lane < ROWS) {
      const uint8_t* first = s - (reinterpret_cast<uintptr_t>(s) & 3u);
      const bool inside = valid && end - first >= 20;
#pragma unroll
      for (int o = 0; o < 20; o += 4) {
        int n = inside ? 4 : 0;
        if (valid && !inside) n = (int)max(0LL, min(4LL, (long long)(end - first) - o));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + o),
                     "l"(n > 0 ? first + o : src), "r"(n)
                     : "memory");
      }
    }
    s += 32 * per_row;
    to += 32 * 20;
  }
  cp_async_arrive_noinc(raw);
}

// order_scales for those: the words are shifted into place, and what is past a row's
// end cleared.
template <int ROWS, int SLOTS, typename RowOf>
LORA_DEV void order_scale_words(uint8_t* ring, int slot_bytes, uint64_t* raw, uint64_t* ready,
                                volatile int* stop, uint32_t* flags, int units, int blocks,
                                int block0, RowOf row_of, const uint8_t* src, int per_row) {
  const int lane = threadIdx.x & 31;
  Ring b;
  bool ok = true;
  for (int i = 0; i < units && ok; ++i) {
    const long long row = (long long)row_of(i) + lane;
    for (int k = 0; k < blocks; ++k) {
      const int at = (block0 + k) * (kBlockK / 32);
      uint8_t* slot = ring + b.s * slot_bytes;
      if (!(ok = warp_wait(&raw[b.s], b.round, stop, flags))) break;
      uint4 v[1][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[0][j] = make_uint4(0u, 0u, 0u, 0u);
        if (j * 32 + lane < ROWS) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(slot + (j * 32 + lane) * 20);
          const uint32_t shift =
              (uint32_t)((reinterpret_cast<uintptr_t>(src) + (row + j * 32) * per_row + at) & 3) * 8u;
          uint32_t x[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[c] = __funnelshift_r(w[c], w[c + 1], shift);
            const int keep = per_row - at - 4 * c;   // bytes of this word that are the row's
            if (keep < 4) x[c] &= keep <= 0 ? 0u : (1u << (8 * keep)) - 1u;
          }
          v[0][j] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      __syncwarp();
      write_ordered<1>(slot, v);
      if (lane == 0) mbar_arrive(&ready[b.s]);
      b.next<SLOTS>();
    }
  }
}

// 16 lanes x 32 columns of fp32 from tensor memory in the layout of a matrix
// fragment: of each 8 columns the thread gets lanes l / 4 and l / 4 + 8, columns
// 2 (l % 4) and the next.  Packed in pairs of columns: out[2 c8 + half].
template <typename OT>
LORA_DEV void tmem_ld_fragments(uint32_t taddr, uint32_t (&out)[8]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i)
    out[i] = pack2_any(OT(), __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

LORA_DEV void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// A warp's 32 features x 32 columns (lo: features 0..15, hi: 16..31, as above)
// to y, `rows` of the columns being rows of y.  Turned in shared memory, 16 rows
// at a time, to 64 bytes of features a row (16-byte chunks swizzled by the row),
// then stored 16 bytes a lane.
template <typename OT>
LORA_DEV void store_fragments(OT* y, int N, int f0, int rows, uint8_t* turn, const uint32_t (&lo)[8],
                              const uint32_t (&hi)[8]) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(turn);
  // stmatrix: lanes 8 i .. 8 i + 7 address the rows of matrix i: features 8 i..
  const int r8 = lane & 7, q = lane >> 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (16 * h >= rows) break;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * c + r8;
      const int i = 2 * (2 * h + c);
      stmatrix_x4_trans(base + row * 64 + ((q ^ ((row >> 1) & 3)) << 4), lo[i], lo[i + 1], hi[i],
                        hi[i + 1]);
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * c + (lane >> 2), ch = lane & 3;
      const uint4 v =
          *reinterpret_cast<const uint4*>(turn + row * 64 + ((ch ^ ((row >> 1) & 3)) << 4));
      if (16 * h + row < rows && f0 + ch * 8 < N)
        *reinterpret_cast<uint4*>(y + (size_t)(16 * h + row) * N + f0 + ch * 8) = v;
    }
  }
}

template <int BN, typename OT>
__global__ void __launch_bounds__(Cfg<BN>::kThreads, 1)
mx_linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_ws,
                 const __grid_constant__ CUtensorMap map_xs, const Params p) {
  typedef Cfg<BN> C;
  constexpr int kS = C::kStages;
  extern __shared__ uint8_t mx_smem[];
  uint8_t* base = mx_smem + (up1024(smem_u32(mx_smem)) - smem_u32(mx_smem));
  uint64_t* full = reinterpret_cast<uint64_t*>(base);
  uint64_t* empty = full + kS;
  uint64_t* sf_raw = empty + kS;                // a block of scales has landed (by TMA):
                                                // the weight's, then x's
  uint64_t* sf_full = sf_raw + 2 * C::kSfSlots;    // ... is in order
  uint64_t* sf_empty = sf_full + C::kSfSlots;  // ... is in tensor memory
  uint64_t* accfull = sf_empty + C::kSfSlots;
  uint64_t* accempty = accfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 512);
  volatile int* stop = reinterpret_cast<volatile int*>(base + 516);
  int* scratch = reinterpret_cast<int*>(base + 576);
  int* prefix = reinterpret_cast<int*>(base + 1024);   // up to 1025 ints
  uint8_t* ring = base + kHeader;
  uint8_t* sf_ring = ring + kS * C::kStage;
  uint8_t* turn = sf_ring + C::kSfSlots * C::kSfSlot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = p.splits;
  const int part = splits > 1 ? (int)cluster_ctarank() : 0;
  const int first_unit = (int)blockIdx.x / splits;
  const int unit_step = (int)gridDim.x / splits;
  const int block0 = part * p.per_split;
  const int blocks = min(p.blocks - block0, p.per_split);                  // >= 1
  const int k0 = block0 * kBlockK;
  const int kcount = min(p.q.K - k0, blocks * kBlockK);                    // this CTA's part of k
  const int stages = (kcount + kK - 1) / kK;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kSfSlots; ++i) {
      // by TMA one arrival, else one of each copying lane
      mbar_init(&sf_raw[i], p.scale_copy == kByTma ? 1 : 32);
      mbar_init(&sf_raw[C::kSfSlots + i], p.scale_copy == kByTma ? 1 : 32);
      mbar_init(&sf_full[i], 2);    // the two scale warps
      mbar_init(&sf_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], C::kEpiWarps);
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
  const Plan plan = make_plan<BN, C::kThreads>(
      p, prefix, scratch,
      C::kOwnOffsets ? reinterpret_cast<int*>(turn + C::kEpiWarps * kTurn) : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.tiles > first_unit ? (plan.tiles - first_unit - 1) / unit_step + 1 : 0;

  if (warp == 0) {
    // ---- element tiles ----
    if (elect_one()) {
      Ring r;
      for (int i = 0; i < units && !*stop; ++i) {
        const Tile t = tile_of<BN>(p, plan, first_unit + i * unit_step);
        for (int k = 0; k < stages; ++k) {
          if (!wait_or_stop(&empty[r.s], r.round ^ 1u, stop, p.q.flags)) break;
          uint8_t* slot = ring + r.s * C::kStage;
          const int at = (k0 + k * kK) / 2;
          mbar_arrive_expect_tx(&full[r.s], C::kStage);
          tma_load_2d(slot, &map_w, at, t.wrow, &full[r.s]);
          tma_load_2d(slot + kATile, &map_x, at, t.row0, &full[r.s]);
          r.next<kS>();
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMAs: one thread ----
    if (elect_one()) {
      Ring r, b, acc;
      const uint32_t ring_lo = desc_lo(smem_u32(ring)), sf_lo = desc_lo(smem_u32(sf_ring));
      bool ok = true;
      uint32_t idesc = mxf4_idesc(kM, BN);
      auto shape = [&](int i) {
        if (BN > 32 && i < units)
          idesc = mxf4_idesc(kM, columns_of(tile_of<BN>(p, plan, first_unit + i * unit_step), BN));
      };
      shape(0);
      for (int i = 0; i < units && ok; ++i) {
        if (!(ok = wait_or_stop(&accempty[acc.s], acc.round ^ 1u, stop, p.q.flags))) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc.s * BN);
        uint32_t sf = 0;
        for (int k = 0; k < stages; ++k) {
          if ((k & 1) == 0) {
            if (!(ok = wait_or_stop(&sf_full[b.s], b.round, stop, p.q.flags))) break;
            tc_fence_after();
            // the two blocks of scales in tensor memory take turns with the MMAs
            // in issue order: copies and MMAs of one thread run in order
            sf = tmem + (uint32_t)(C::kAcc * BN + (k & 2 ? C::kSfCols : 0));
            const uint32_t lo = sf_lo + (uint32_t)b.s * (C::kSfSlot >> 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              copy_scales(sf + 4 * c, lo + c * (kSfAtom >> 4));
#pragma unroll
              for (int h = 0; h < C::kAtoms; ++h)
                copy_scales(sf + 16 + 4 * (C::kAtoms * c + h),
                            lo + (C::kSfX0 >> 4) + (C::kAtoms * c + h) * (kSfAtom >> 4));
            }
            mma_commit(&sf_empty[b.s]);
            b.next<C::kSfSlots>();
          }
          if (!(ok = wait_or_stop(&full[r.s], r.round, stop, p.q.flags))) break;
          tc_fence_after();
          const uint32_t a_lo = ring_lo + (uint32_t)r.s * (C::kStage >> 4);
          const uint32_t b_lo = a_lo + (kATile >> 4);
          const uint32_t sfk = sf + (k & 1 ? 8u : 0u), sfx = sf + 16u + (k & 1 ? 8u * C::kAtoms : 0u);
          const int left = kcount - k * kK;   // elements of k from this stage on
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j == 0 || left > 64 * j)
              mma_mxf4(d, a_lo + 2 * j, b_lo + 2 * j, idesc | mxf4_half(j & 1), sfk + 4 * (j >> 1),
                       sfx + 4 * C::kAtoms * (j >> 1), (k | j) != 0 ? 1u : 0u);
          mma_commit(&empty[r.s]);
          r.next<kS>();
        }
        if (!ok) break;
        mma_commit(&accfull[acc.s]);
        acc.next<C::kAcc>();
        shape(i + 1);   // while the MMAs run
      }
    }
  } else if (warp < 4) {
    // ---- scales into the tensor core's order: warp 2 the weight's 128 rows, warp
    // 3 those of x.  Lane l has rows l, l + 32, l + 64, l + 96 of an atom; a row's
    // 16 bytes are one word for each of four atoms. ----
    if (BN <= 128 && p.scale_copy == kAround) {
      if (warp == 2)
        order_scale_words<kM, C::kSfSlots>(
            sf_ring, C::kSfSlot, sf_raw, sf_full, stop, p.q.flags, units, blocks, block0,
            [&](int i) { return tile_of<BN>(p, plan, first_unit + i * unit_step).wrow; },
            p.q.w_scales, p.q.K / 32);
      else
        order_scale_words<BN, C::kSfSlots>(
            sf_ring + C::kSfX0, C::kSfSlot, sf_raw + C::kSfSlots, sf_full, stop, p.q.flags, units,
            blocks, block0,
            [&](int i) { return tile_of<BN>(p, plan, first_unit + i * unit_step).row0; },
            p.q.x_scales, p.q.K / 32);
    } else if (warp == 2) {
      order_scales<1, C::kSfSlots>(sf_ring, C::kSfSlot, sf_raw, sf_full, stop, p.q.flags,
                                   units * blocks);
    } else {
      order_scales<C::kAtoms, C::kSfSlots>(sf_ring + C::kSfX0, C::kSfSlot, sf_raw + C::kSfSlots,
                                           sf_full, stop, p.q.flags, units * blocks);
    }
  } else if (warp == 4 + C::kEpiWarps) {
    // ---- raw scales ----
    const bool by_tma = p.scale_copy == kByTma;
    const int per_row = p.q.K / 32;
    const long long w_rows = (long long)p.q.experts * p.q.N;
    if (!by_tma || elect_one()) {
      Ring b;
      bool ok = true;
      for (int i = 0; i < units && ok; ++i) {
        const Tile t = tile_of<BN>(p, plan, first_unit + i * unit_step);
        for (int k = 0; k < blocks; ++k) {
          if (!(ok = wait_or_stop(&sf_empty[b.s], b.round ^ 1u, stop, p.q.flags))) break;
          uint8_t* w = sf_ring + b.s * C::kSfSlot;
          uint8_t* x = w + C::kSfX0;
          uint64_t *raw_w = &sf_raw[b.s], *raw_x = &sf_raw[C::kSfSlots + b.s];
          const int at = k0 / 32 + k * (kBlockK / 32);
          if (by_tma) {
            mbar_arrive_expect_tx(raw_w, kM * 16);
            tma_load_2d(w, &map_ws, at, t.wrow, raw_w);
            mbar_arrive_expect_tx(raw_x, BN * 16);
            tma_load_2d(x, &map_xs, at, t.row0, raw_x);
          } else if (p.scale_copy == kBy8) {
            copy_scale_rows<8, kM>(w, p.q.w_scales, t.wrow, w_rows, per_row, at, raw_w);
            copy_scale_rows<8, BN>(x, p.q.x_scales, t.row0, p.q.rows, per_row, at, raw_x);
          } else if (p.scale_copy == kBy4) {
            copy_scale_rows<4, kM>(w, p.q.w_scales, t.wrow, w_rows, per_row, at, raw_w);
            copy_scale_rows<4, BN>(x, p.q.x_scales, t.row0, p.q.rows, per_row, at, raw_x);
          } else if (BN <= 128) {
            copy_scale_words<kM>(w, p.q.w_scales, p.q.w_scales + w_rows * per_row, t.wrow, w_rows,
                                 per_row, at, raw_w);
            copy_scale_words<BN>(x, p.q.x_scales, p.q.x_scales + (long long)p.q.rows * per_row,
                                 t.row0, p.q.rows, per_row, at, raw_x);
          }
          b.next<C::kSfSlots>();
        }
      }
      // copies of a warp that gave up land before it leaves
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---- epilogue: lane = feature, column = row of x ----
    const int quarter = warp & 3;
    const int c_first = ((warp - 4) >> 2) * C::kWarpCols;
    OT* y = reinterpret_cast<OT*>(p.q.y);
    Ring acc;
    for (int i = 0; i < units; ++i) {
      const Tile t = tile_of<BN>(p, plan, first_unit + i * unit_step);
      if (!warp_wait(&accfull[acc.s], acc.round, stop, p.q.flags)) break;
      __syncwarp();
      tc_fence_after();
      const int f = t.f0 + quarter * 32 + lane;
      const bool f_ok = f < p.q.N;
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc.s * BN + c_first);
      if (splits > 1) {
        // partial sums to shared memory, [column][feature]: the ring is idle, this
        // being the CTA's only tile and its MMAs done
        float* part_sums = reinterpret_cast<float*>(ring) + (size_t)c_first * kM + quarter * 32 + lane;
#pragma unroll
        for (int c = 0; c < C::kWarpCols / 32; ++c)
          if (c_first + c * 32 < t.rows) {   // warp-uniform
            float v[32];
            tmem_ld_32x32(src + c * 32, v);
#pragma unroll
            for (int n = 0; n < 32; ++n)
              if (c_first + c * 32 + n < BN) part_sums[(c * 32 + n) * kM] = v[n];
          }
        tc_fence_before();
        break;
      }
      if (sizeof(OT) == 2) {
        // all of it into registers first, so that the accumulator is free early
        uint32_t lo[C::kWarpCols / 32][8], hi[C::kWarpCols / 32][8];
#pragma unroll
        for (int c = 0; c < C::kWarpCols / 32; ++c)
          if (c_first + c * 32 < t.rows) {   // warp-uniform
            tmem_ld_fragments<OT>(src + c * 32, lo[c]);
            tmem_ld_fragments<OT>(src + (16u << 16) + c * 32, hi[c]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&accempty[acc.s]);
#pragma unroll
        for (int c = 0; c < C::kWarpCols / 32; ++c) {
          const int c0 = c_first + c * 32;
          if (c0 < t.rows)
            store_fragments(y + (size_t)(t.row0 + c0) * p.q.N, p.q.N, t.f0 + quarter * 32,
                            t.rows - c0, turn + (warp - 4) * kTurn, lo[c], hi[c]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < C::kWarpCols / 32; ++c) {
          const int c0 = c_first + c * 32;
          if (c0 < t.rows) {
            float v[32];
            tmem_ld_32x32(src + c * 32, v);
            if (f_ok) {
              float* o = reinterpret_cast<float*>(p.q.y) + (size_t)(t.row0 + c0) * p.q.N + f;
#pragma unroll
              for (int n = 0; n < 32; ++n)
                if (c0 + n < t.rows) o[(size_t)n * p.q.N] = v[n];
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&accempty[acc.s]);
      }
      acc.next<C::kAcc>();
    }
  }

  __syncwarp();
  if (splits > 1) {
    // Sum over the cluster in rank order; each CTA finishes its share of the rows.
    // Every CTA of the cluster has the same tile, so all of them are here.
    cluster_sync();
    if (units > 0) {
      const Tile t = tile_of<BN>(p, plan, first_unit);
      const int share = (t.rows + splits - 1) / splits;
      const int c1 = min(t.rows, (part + 1) * share);
      const int f = lane * 4;
      for (int c = part * share + warp; c < c1; c += C::kThreads / 32) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < splits; ++s) {
          const float4 v = dsmem_ld_f32x4(dsmem_addr(ring + (c * kM + f) * 4, (uint32_t)s));
          sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
        }
        if (t.f0 + f < p.q.N) {   // N is a multiple of 8
          OT* o = reinterpret_cast<OT*>(p.q.y) + (size_t)(t.row0 + c) * p.q.N + t.f0 + f;
          if (sizeof(OT) == 2)
            *reinterpret_cast<uint2*>(o) =
                make_uint2(pack2_any(OT(), sum.x, sum.y), pack2_any(OT(), sum.z, sum.w));
          else
            *reinterpret_cast<float4*>(o) = sum;
        }
      }
    }
    cluster_sync();   // no CTA leaves while its sums are read
  }
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

// ---------------------------------------------------------------------------
// Two CTAs on one tile of 256 features x 256 (or 128) rows (cta_group::2), for
// products of many rows.  Each CTA holds 128 features of the weight and 128 of the rows, and
// the tensor cores of both read them from both: 8 KB of shared memory per MMA and
// SM instead of the 12 that a 128 x 256 tile of one CTA reads, and as much less to
// fetch, which is what bounds that tile (a stage takes 795 cycles there, 540 being
// the tensor core's).  Each CTA brings its own element tiles, the scales of its
// features and those of all rows; the first CTA issues the MMAs and the copies of
// scales (they run in both), waiting on barriers on which both arrive, and its
// commits arrive in both.
// ---------------------------------------------------------------------------

template <int ROWS>
struct PairCfg {
  static constexpr int kRows = ROWS;
  static constexpr int kBTile = ROWS / 2 * kK / 2;
  static constexpr int kStage = kATile + kBTile;             // 128 features and half of the rows
  static constexpr int kStages = ROWS == 256 ? 6 : 8;
  static constexpr int kAtoms = ROWS / 128;
  static constexpr int kSfSlot = (4 + 4 * kAtoms) * kSfAtom; // per 512 of k: of W, of all of X
  static constexpr int kSfSlots = ROWS == 256 ? 3 : 4;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 160 + 32 * kEpiWarps;
  static constexpr int kSmem = 1024 + kHeader + kStages * kStage + kSfSlots * kSfSlot + kEpiWarps * kTurn;
  static constexpr int kAcc = 256 / ROWS;                    // accumulators: 256 columns in all
  static constexpr int kSfCols = 16 + 16 * kAtoms;           // two sets behind them
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

LORA_DEV void mma_mxf4_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa,
                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %7};\n\t"
      "mov.b64 b, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
      "[%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescTile)
      : "memory");
}
LORA_DEV void copy_scales_pair(uint32_t taddr, uint32_t lo) {
  asm volatile(
      "{\n\t.reg .b64 d;\n\t"
      "mov.b64 d, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
      "r"(lo), "r"(kDescScale)
      : "memory");
}
// Arrives on `bar` of both CTAs once what this thread issued so far is done.
LORA_DEV void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// A tile into this CTA's memory, counted on a barrier of the pair's first.
LORA_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

template <int ROWS, typename OT>
__global__ void __launch_bounds__(PairCfg<ROWS>::kThreads, 1)
mx_linear_pair_kernel(const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_ws,
                      const __grid_constant__ CUtensorMap map_xs, const Params p) {
  typedef PairCfg<ROWS> C;
  constexpr int kS = C::kStages, kSl = C::kSfSlots;
  extern __shared__ uint8_t mx_smem[];
  uint8_t* base = mx_smem + (up1024(smem_u32(mx_smem)) - smem_u32(mx_smem));
  uint64_t* full = reinterpret_cast<uint64_t*>(base);   // (the first CTA's are used)
  uint64_t* empty = full + kS;
  uint64_t* sf_raw = empty + kS;
  uint64_t* sf_full = sf_raw + 2 * kSl;                  // (the first CTA's)
  uint64_t* sf_empty = sf_full + kSl;
  uint64_t* accfull = sf_empty + kSl;
  uint64_t* accempty = accfull + C::kAcc;                // (the first CTA's)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + 512);
  volatile int* stop = reinterpret_cast<volatile int*>(base + 516);
  int* scratch = reinterpret_cast<int*>(base + 576);
  int* prefix = reinterpret_cast<int*>(base + 1024);
  uint8_t* ring = base + kHeader;
  uint8_t* sf_ring = ring + kS * C::kStage;
  uint8_t* turn = sf_ring + kSl * C::kSfSlot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int first_unit = (int)blockIdx.x / 2, unit_step = (int)gridDim.x / 2;
  const int stages = (p.q.K + kK - 1) / kK, blocks = p.blocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kSl; ++i) {
      mbar_init(&sf_raw[i], 1);
      mbar_init(&sf_raw[kSl + i], 1);
      mbar_init(&sf_full[i], 4);                // two scale warps of each CTA
      mbar_init(&sf_empty[i], 1);
    }
    for (int i = 0; i < C::kAcc; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], 2 * C::kEpiWarps);
    }
    *stop = 0;
    fence_mbar_init();
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
    prefetch_tensormap(&map_ws);
    prefetch_tensormap(&map_xs);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const Plan plan = make_plan<C::kRows, C::kThreads>(p, prefix, scratch);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the barriers of both CTAs are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.tiles > first_unit ? (plan.tiles - first_unit - 1) / unit_step + 1 : 0;
  // this CTA's share of a unit: 128 of its features
  auto unit = [&](int i) {
    Tile t = tile_of<C::kRows, 2 * kM>(p, plan, first_unit + i * unit_step);
    t.f0 += rank * kM;
    t.wrow += rank * kM;
    return t;
  };

  if (warp == 0) {
    if (elect_one()) {
      Ring r;
      for (int i = 0; i < units && !*stop; ++i) {
        const Tile t = unit(i);
        // the MMAs' columns are split between the CTAs
        const int x_row = t.row0 + rank * (columns_of(t, ROWS) / 2);
        for (int k = 0; k < stages; ++k) {
          if (!wait_or_stop<true>(&empty[r.s], r.round ^ 1u, stop, p.q.flags)) break;
          uint8_t* slot = ring + r.s * C::kStage;
          const uint32_t bar = at_first(&full[r.s]);
          if (rank == 0) mbar_arrive_expect_tx(&full[r.s], 2 * C::kStage);
          tma_load_2d_pair(slot, &map_w, k * (kK / 2), t.wrow, bar);
          tma_load_2d_pair(slot + kATile, &map_x, k * (kK / 2), x_row, bar);
          r.next<kS>();
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      Ring r, b, acc;
      const uint32_t ring_lo = desc_lo(smem_u32(ring)), sf_lo = desc_lo(smem_u32(sf_ring));
      bool ok = true;
      uint32_t idesc = 0;
      auto shape = [&](int i) {
        if (i < units) idesc = mxf4_idesc(2 * kM, columns_of(unit(i), ROWS));
      };
      shape(0);
      for (int i = 0; i < units && ok; ++i) {
        if (!(ok = wait_or_stop<true>(&accempty[acc.s], acc.round ^ 1u, stop, p.q.flags))) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc.s * ROWS);
        uint32_t sf = 0;
        for (int k = 0; k < stages; ++k) {
          if ((k & 1) == 0) {
            if (!(ok = wait_or_stop<true>(&sf_full[b.s], b.round, stop, p.q.flags))) break;
            tc_fence_after();
            sf = tmem + (uint32_t)(256 + (k & 2 ? C::kSfCols : 0));
            const uint32_t lo = sf_lo + (uint32_t)b.s * (C::kSfSlot >> 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              copy_scales_pair(sf + 4 * c, lo + c * (kSfAtom >> 4));
#pragma unroll
              for (int h = 0; h < C::kAtoms; ++h)
                copy_scales_pair(sf + 16 + 4 * (C::kAtoms * c + h),
                                 lo + (4 + C::kAtoms * c + h) * (kSfAtom >> 4));
            }
            commit_pair(&sf_empty[b.s]);
            b.next<kSl>();
          }
          if (!(ok = wait_or_stop<true>(&full[r.s], r.round, stop, p.q.flags))) break;
          tc_fence_after();
          const uint32_t a_lo = ring_lo + (uint32_t)r.s * (C::kStage >> 4);
          const uint32_t b_lo = a_lo + (kATile >> 4);
          const uint32_t sfk = sf + (k & 1 ? 8u : 0u), sfx = sf + 16u + (k & 1 ? 8u * C::kAtoms : 0u);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_mxf4_pair(d, a_lo + 2 * j, b_lo + 2 * j, idesc | mxf4_half(j & 1),
                          sfk + 4 * (j >> 1), sfx + 4 * C::kAtoms * (j >> 1), (k | j) != 0 ? 1u : 0u);
          commit_pair(&empty[r.s]);
          r.next<kS>();
        }
        if (!ok) break;
        commit_pair(&accfull[acc.s]);
        acc.next<C::kAcc>();
        shape(i + 1);   // while the MMAs run
      }
    }
  } else if (warp == 2) {
    order_scales<1, kSl, true>(sf_ring, C::kSfSlot, sf_raw, sf_full, stop, p.q.flags, units * blocks);
  } else if (warp == 3) {
    order_scales<C::kAtoms, kSl, true>(sf_ring + 4 * kSfAtom, C::kSfSlot, sf_raw + kSl, sf_full, stop,
                               p.q.flags, units * blocks);
  } else if (warp == 4 + C::kEpiWarps) {
    if (elect_one()) {
      Ring b;
      bool ok = true;
      for (int i = 0; i < units && ok; ++i) {
        const Tile t = unit(i);
        for (int k = 0; k < blocks; ++k) {
          if (!(ok = wait_or_stop<true>(&sf_empty[b.s], b.round ^ 1u, stop, p.q.flags))) break;
          uint8_t* slot = sf_ring + b.s * C::kSfSlot;
          mbar_arrive_expect_tx(&sf_raw[b.s], kM * 16);
          tma_load_2d(slot, &map_ws, k * (kBlockK / 32), t.wrow, &sf_raw[b.s]);
          mbar_arrive_expect_tx(&sf_raw[kSl + b.s], C::kRows * 16);
          tma_load_2d(slot + 4 * kSfAtom, &map_xs, k * (kBlockK / 32), t.row0, &sf_raw[kSl + b.s]);
          b.next<kSl>();
        }
      }
    }
  } else {
    const int quarter = warp & 3;
    const int c_first = ((warp - 4) >> 2) * (C::kRows / 2);
    OT* y = reinterpret_cast<OT*>(p.q.y);
    Ring acc;
    for (int i = 0; i < units; ++i, acc.next<C::kAcc>()) {
      const Tile t = unit(i);
      if (!warp_wait<true>(&accfull[acc.s], acc.round, stop, p.q.flags)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc.s * ROWS + c_first);
      const int f = t.f0 + quarter * 32;
      constexpr int kParts = C::kRows / 2 / 32;
      if (sizeof(OT) == 2) {
        uint32_t lo[kParts][8], hi[kParts][8];
#pragma unroll
        for (int c = 0; c < kParts; ++c)
          if (c_first + c * 32 < t.rows) {   // warp-uniform
            tmem_ld_fragments<OT>(src + c * 32, lo[c]);
            tmem_ld_fragments<OT>(src + (16u << 16) + c * 32, hi[c]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at_first<false>(&accempty[acc.s]);
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          const int c0 = c_first + c * 32;
          if (c0 < t.rows)
            store_fragments(y + (size_t)(t.row0 + c0) * p.q.N, p.q.N, f, t.rows - c0,
                            turn + (warp - 4) * kTurn, lo[c], hi[c]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          const int c0 = c_first + c * 32;
          if (c0 < t.rows) {
            float v[32];
            tmem_ld_32x32(src + c * 32, v);
            if (f + lane < p.q.N) {
              float* o = reinterpret_cast<float*>(p.q.y) + (size_t)(t.row0 + c0) * p.q.N + f + lane;
#pragma unroll
              for (int n = 0; n < 32; ++n)
                if (c0 + n < t.rows) o[(size_t)n * p.q.N] = v[n];
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at_first<false>(&accempty[acc.s]);
      }
    }
  }

  __syncwarp();
  if (*stop) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the other reads its memory or arrives there
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
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

// Tensor map over `rows` rows of `bytes` bytes, box box_bytes x box_rows.
cudaError_t make_map(CUtensorMap* map, const void* ptr, uint64_t bytes, uint64_t rows,
                     uint32_t box_bytes, uint32_t box_rows, const char** why) {
  auto fn = encode_fn();
  if (fn == nullptr) {
    *why = "cuTensorMapEncodeTiled is not available";
    return cudaErrorNotSupported;
  }
  const cuuint64_t dims[2] = {bytes, rows};
  const cuuint64_t strides[1] = {bytes};
  const cuuint32_t box[2] = {box_bytes, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
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

// Tiles there can be: every expert's last one may be partial.
long long tile_bound(const MxLinearParams& q, int BN) {
  const long long ftiles = (q.N + kM - 1) / kM;
  if (q.expert_offsets == nullptr) return ((long long)q.rows + BN - 1) / BN * ftiles;
  return ((long long)q.rows / BN + min(q.experts, q.rows)) * ftiles;
}

template <int BN, typename OT>
cudaError_t launch(const MxLinearParams& q, int splits, cudaStream_t stream, const char** why) {
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
  const uint64_t w_rows = (uint64_t)experts * q.N, x_rows = (uint64_t)q.rows;
  CUtensorMap map_w, map_x, map_ws = {}, map_xs = {};
  err = make_map(&map_w, q.w_codes, (uint64_t)q.K / 2, w_rows, kK / 2, kM, why);
  if (err != cudaSuccess) return err;
  err = make_map(&map_x, q.x_codes, (uint64_t)q.K / 2, x_rows, kK / 2, BN, why);
  if (err != cudaSuccess) return err;
  Params p = {};
  p.q = q;
  p.ftiles = (q.N + kM - 1) / kM;
  p.blocks = (q.K + kBlockK - 1) / kBlockK;
  p.per_split = (p.blocks + splits - 1) / splits;
  p.most = (int)tile_bound(q, BN);
  p.splits = (p.blocks + p.per_split - 1) / p.per_split;   // every CTA has a part
  p.scale_copy = q.K % kBlockK == 0 ? kByTma : q.K % 256 == 0 ? kBy8 : q.K % 128 == 0 ? kBy4 : kAround;
  if (p.scale_copy == kByTma) {
    err = make_map(&map_ws, q.w_scales, (uint64_t)q.K / 32, w_rows, kBlockK / 32, kM, why);
    if (err != cudaSuccess) return err;
    err = make_map(&map_xs, q.x_scales, (uint64_t)q.K / 32, x_rows, kBlockK / 32, BN, why);
    if (err != cudaSuccess) return err;
  }
  const long long tiles = tile_bound(q, BN);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  // a cluster for each tile, or one CTA per SM over all tiles
  cfg.gridDim = dim3((unsigned)(p.splits > 1 ? tiles * p.splits : min((long long)sms, tiles)), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = (unsigned)p.splits;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, mx_linear_kernel<BN, OT>, map_w, map_x, map_ws, map_xs, p);
}

// Tiles of the pair kernel there can be.
long long pair_bound(const MxLinearParams& q, int rows) {
  const long long ftiles = (q.N + 2 * kM - 1) / (2 * kM);
  if (q.expert_offsets == nullptr) return ((long long)q.rows + rows - 1) / rows * ftiles;
  return ((long long)q.rows / rows + min(q.experts, q.rows)) * ftiles;
}

template <int ROWS, typename OT>
cudaError_t launch_pair(const MxLinearParams& q, int sms, cudaStream_t stream, const char** why) {
  typedef PairCfg<ROWS> C;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  static bool attr[64];
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!attr[dev]) {
      err = cudaFuncSetAttribute(mx_linear_pair_kernel<ROWS, OT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (err != cudaSuccess) return err;
      attr[dev] = true;
    }
  }
  const uint64_t w_rows = (uint64_t)(q.expert_offsets != nullptr ? q.experts : 1) * q.N;
  CUtensorMap map_w, map_x, map_ws, map_xs;
  err = make_map(&map_w, q.w_codes, (uint64_t)q.K / 2, w_rows, kK / 2, kM, why);
  if (err == cudaSuccess)
    err = make_map(&map_x, q.x_codes, (uint64_t)q.K / 2, (uint64_t)q.rows, kK / 2, C::kRows / 2, why);
  if (err == cudaSuccess)
    err = make_map(&map_ws, q.w_scales, (uint64_t)q.K / 32, w_rows, kBlockK / 32, kM, why);
  if (err == cudaSuccess)
    err = make_map(&map_xs, q.x_scales, (uint64_t)q.K / 32, (uint64_t)q.rows, kBlockK / 32, C::kRows, why);
  if (err != cudaSuccess) return err;
  Params p = {};
  p.q = q;
  p.ftiles = (q.N + 2 * kM - 1) / (2 * kM);
  p.splits = 1;
  p.most = (int)pair_bound(q, ROWS);
  p.blocks = p.per_split = q.K / kBlockK;
  p.scale_copy = kByTma;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  cfg.gridDim = dim3((unsigned)(2 * min((long long)sms / 2, pair_bound(q, ROWS))), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 2;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mx_linear_pair_kernel<ROWS, OT>, map_w, map_x, map_ws, map_xs, p);
}

// Clusters of `size` CTAs (one to an SM) that run at once: fewer than SMs / size,
// for a cluster stays within a group of SMs (45 of three on 148 SMs).
int clusters_at_once(int dev, int size) {
  static int known[64][9];
  std::lock_guard<std::mutex> lk(g_mu);
  int& n = known[dev][size];
  if (n == 0) {
    typedef Cfg<128> C;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)size, 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int got = 0;
    if (cudaFuncSetAttribute(mx_linear_kernel<128, __nv_bfloat16>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&got, mx_linear_kernel<128, __nv_bfloat16>, &cfg) != cudaSuccess)
      got = 0;
    n = got > 0 ? got : -1;
  }
  return n;
}

// Which tile, and how many CTAs to a tile.  The smallest row tile that holds the
// rows an expert has on average; and where the tiles do not fill the SMs, as many
// CTAs to each as do (a cluster of at most eight, each with at least one block of k).
// With one weight and more than 128 rows both larger tiles are weighed by what a CTA
// then has to do: a stage costs what its bytes take at 60 a cycle, and a tile an
// epilogue (cycles, fitted to 8192 and 2048 rows of 4096 by 28672 and 6144).
struct Shape {
  int rows, splits;
};
Shape choose(const MxLinearParams& q, int dev, int sms) {
  const int experts = q.expert_offsets != nullptr ? min(q.experts, q.rows) : 1;
  const long long mean = ((long long)q.rows + experts - 1) / experts;
  const int blocks = (q.K + kBlockK - 1) / kBlockK;
  auto splits_for = [&](long long tiles) {
    // as many as let every tile's cluster run at once
    int s = (int)min((long long)sms / (tiles > 0 ? tiles : 1), (long long)min(8, blocks));
    while (s > 1 && clusters_at_once(dev, s) < tiles) --s;
    return max(1, s);
  };
  // (with few k a tile's epilogue weighs more, and experts have ragged numbers of rows:
  // a tile that holds half as many rows again as the mean, 8 to 128 experts of 256 to
  // 1024 by 1024 to 4096.  128 of 768 by 4096, a mean of 14, 30 and 60 rows: 40, 45 and
  // 50 us, 56, 58 and 65 by the mean; 8 of 512 by 4096, a mean of 20 and 40: 6.6 and
  // 7.3, 7.7 and 8.7 by twice the mean)
  const long long fit = q.K <= 1024 && experts > 1 ? mean + mean / 2 : mean;
  Shape best = {fit <= 16 ? 16 : fit <= 32 ? 32 : fit <= 64 ? 64 : 128, 1};
  best.splits = splits_for(tile_bound(q, best.rows));
  if (mean <= 128 || q.K % 128 != 0) return best;   // (256 rows: no room for unaligned scales)
  if (q.expert_offsets != nullptr) return {256, splits_for(tile_bound(q, 256))};
  double least = 0;
  for (int bn = 128; bn <= 256; bn += 128) {
    const long long tiles = tile_bound(q, bn);
    const int splits = splits_for(tiles);
    const long long rounds = splits > 1 ? 1 : (tiles + sms - 1) / sms;
    const double stages = 2.0 * ((blocks + splits - 1) / splits);
    const double cost = rounds * (stages * (kATile + bn * kK / 2) / 60.0 + 8.0 * bn) +
                        (splits > 1 ? 1500.0 + 10.0 * bn : 0.0);
    if (bn == 128 || cost < least) {
      least = cost;
      best = {bn, splits};
    }
  }
  return best;
}

template <typename OT>
cudaError_t launch_typed(const MxLinearParams& q, cudaStream_t stream, const char** why) {
  int dev = 0, sms = 0;
  const cudaError_t err = dev_sms(&dev, &sms);
  if (err != cudaSuccess) return err;
  const Shape s = choose(q, dev, sms);
  if (s.splits == 1 && q.K % kBlockK == 0) {
    if (s.rows == 256 && pair_bound(q, 256) >= sms / 2)
      return launch_pair<256, OT>(q, sms, stream, why);
    if (s.rows == 128 && pair_bound(q, 128) >= sms / 2)
      return launch_pair<128, OT>(q, sms, stream, why);
  }
  switch (s.rows) {
    case 16: return launch<16, OT>(q, s.splits, stream, why);
    case 32: return launch<32, OT>(q, s.splits, stream, why);
    case 64: return launch<64, OT>(q, s.splits, stream, why);
    case 128: return launch<128, OT>(q, s.splits, stream, why);
    default: return launch<256, OT>(q, s.splits, stream, why);
  }
}

}  // namespace

cudaError_t mx_linear_launch(const MxLinearParams& q, int type, cudaStream_t stream,
                             const char** why) {
  if (type == LORA_TYPE_BF16) return launch_typed<__nv_bfloat16>(q, stream, why);
  if (type == LORA_TYPE_F16) return launch_typed<__half>(q, stream, why);
  return launch_typed<float>(q, stream, why);
}

}  // namespace lora
