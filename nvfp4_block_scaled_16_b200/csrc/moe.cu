// moe.cu -- a mixture-of-experts layer for a few tokens, and its router.
//
//   nvfp4_moe_route        the top-k experts of every token and their weights
//   nvfp4_moe_few_tokens   out[i] = sum_j w_ij * Wd[e_ij] (silu(Wg[e_ij] x_i) * (Wu[e_ij] x_i))
//
// The layer's time is the reading of the chosen experts' NVFP4 weights, so every weight byte goes
// once from HBM to shared memory (TMA) and from there straight into tcgen05.mma: the 128 weight
// rows of a tile are the MMA's M side and the few activations its N side.  The activations are not
// quantized to FP4 but written as a sum of FP4 numbers, so the block-scaled FP4 MMA computes with
// them at about bf16 precision and no weight is ever unpacked:
//
//   Slices.  A 16-value block of an activation chunk with largest magnitude m becomes
//     x = F * 2^s * (d0 + d1/4 + d2/32 + d3/256) + r,   every d an e2m1 value,
//   F a power of two for the whole chunk (256 values of x, 128 of h), 2^s >= m/(6F) the smallest
//   power of two, d0 the e2m1 rounding of x/(F*2^s), d1 of four times what is left, d2 and d3 of eight times
//   what is left after that (rounding leaves at most 1, then at most 1/2: 4*1 and 8*1/2 are within e2m1).
//   The block scales 2^s, 2^(s-2), 2^(s-5), 2^(s-8) are exact in ue4m3.  |r| <= F*2^s/512, and F*2^s < m/3:
//   at most m/1536, a third of the half step 2^-9 that bf16 has at m.  s is at least -1 (2^(s-8) is the smallest
//   ue4m3 value), so a block more than 2^9 below the largest value M of its chunk is held to M/786432 instead.
//   Four slices are four MMA columns; their sum is taken when the accumulator is read.
//
// A segment is up to 16 (token, slot) pairs of one expert: 16, 32 or 64 MMA columns.  Three launches:
//   moe_prepare_kernel      groups the slots by expert, writes x as slices in the shared-memory
//                           layout (one contiguous block per segment and 256 values of K);
//   moe_kernel<false>       gate and up tiles, SiLU * up in fp32, h written as slices (rounded
//                           to nothing coarser on the way);
//   moe_kernel<true>        down tiles, weighted sum over the slots of a token, bf16 output.
// Both GEMM kernels give every CTA the same number of (128-row tile, 256-value K stage) units; a tile whose units
// fall to several CTAs is finished by the last of them, which adds the partial sums in CTA
// order, so results do not depend on timing.
//
// Sources (page title, section): flashinfer PR #1774 (masked per-expert operands, silu_and_mul);
// NVIDIA/Fuser PR #5737 (routed experts NVFP4InferenceGroupedSwiGLU, f16a_nvfp4weight_scaled_mm: bf16
// activation, NVFP4 weight).  The router and the few-token form are this library's own.
#include <cuda_bf16.h>

#include "common.cuh"
#include "nvfp4_math.cuh"
#include "tc_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopk = 16;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxTopk;
constexpr int kMoeMaxExperts = 1024;
constexpr int kSegSlots = 16;                    // (token, slot) pairs of a segment
constexpr int kSlices = 4;
constexpr int kSfBlockBytes = 4 * 512;           // scales of one K stage (4 chunks)
constexpr int kRowsBytes = kSegSlots * kSlices * 128;   // at most 64 rows of 256 FP4 values
constexpr int kTileBytes = 128 * 128;            // 128 weight rows x 256 FP4 values
constexpr int kMoeThreads = 64 + 256;            // producer, MMA issuer, 8 epilogue warps

struct Segment {
  int32_t expert, first, count, offset;          // offset: bytes per K stage of all segments before it
};

__host__ __device__ inline int segment_columns(int count) { return count <= 4 ? 16 : (count <= 8 ? 32 : 64); }

// Byte offsets of the caller's workspace.
struct MoeLayout {
  int64_t segments, pos_slot, count_up, count_down, f_x, f_h, b_x, b_h, part_up, part_down, bytes;
  int64_t b_units;                               // bound of a K stage's bytes over all segments
  int32_t max_segments;
};

constexpr int kMoeMaxCtas = 192;

MoeLayout moe_layout(int64_t t, int64_t topk, int64_t E, int64_t n, int64_t k) {
  const int64_t S = t * topk;
  const int64_t hit = S < E ? S : E;
  const int64_t segs = hit + S / kSegSlots < S ? hit + S / kSegSlots : S;
  const int64_t ks1 = (k + 255) / 256, ks2 = (n + 255) / 256;
  // columns of all segments: at most 64 each, and 16 + 8 * count each
  const int64_t cols = 64 * segs < 16 * segs + 8 * S ? 64 * segs : 16 * segs + 8 * S;
  MoeLayout L;
  L.max_segments = static_cast<int32_t>(segs);
  L.b_units = segs * kSfBlockBytes + cols * 128;
  int64_t at = 256;                              // the header: number of segments
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  L.segments = take(segs * static_cast<int64_t>(sizeof(Segment)));
  L.pos_slot = take(S * 4);
  L.count_up = take(segs * ((n + 127) / 128) * 4);
  L.count_down = take((k + 127) / 128 * 4);
  L.f_x = take(segs * ks1 * kSegSlots * 4);
  L.f_h = take(segs * 2 * ks2 * kSegSlots * 4);
  L.b_x = take(L.b_units * ks1);
  L.b_h = take(L.b_units * ks2);
  L.part_up = take(static_cast<int64_t>(kMoeMaxCtas) * 2 * 2 * kSegSlots * 128 * 4);
  L.part_down = take(static_cast<int64_t>(kMoeMaxCtas) * 2 * t * 128 * 4);
  L.bytes = at;
  return L;
}

struct MoeParams {
  const uint16_t* x;            // [t, k] bf16
  const int32_t* ids;           // [t * topk]
  const float* weights;         // [t * topk]
  const uint8_t *sf0, *sf1;     // gate and up scales, or down scales (sf0)
  const float *amax0, *amax1;   // gate and up amax [E]; amax of down in amax_down
  const float* amax_down;
  __nv_bfloat16* out;           // [t, k]
  int* status;
  int32_t* nseg;
  Segment* segments;
  int32_t* pos_slot;
  uint32_t *count_up, *count_down;
  float *f_x, *f_h;
  uint8_t *b_x, *b_h;
  float *part_up, *part_down;
  int64_t sf_stride;            // nvfp4_scale_bytes of one expert's matrix (this phase)
  int64_t b_units;              // extents for the debug build's index checks
  int32_t max_segments;
  int32_t t, topk, experts, n, k;
};

// ---- slices -------------------------------------------------------------------------------------

// z minus the e2m1 value of code i of q.  The code's three magnitude bits on top of an fp32's mantissa and
// the end of its exponent are that value times 2^-126 (a subnormal one included).
__device__ __forceinline__ float minus_e2m1(float z, uint32_t q, int i) {
  const uint32_t bits = i < 6 ? q << (22 - 4 * (i < 6 ? i : 0)) : q >> (4 * (i < 6 ? 6 : i) - 22);
  const uint32_t sign = i < 7 ? q << (28 - 4 * i) : q;
  return fmaf(__uint_as_float((bits & 0x01c00000u) | (sign & 0x80000000u)), -0x1p126f, z);
}

struct Slices {
  uint32_t q[kSlices];          // eight codes of each slice
  uint32_t sf;                  // scale codes of the block's four slices, slice 0 in the low byte
  float factor;                 // F of the chunk (NaN when the chunk holds an infinity or NaN)
};

// ue4m3 code of 2^e, -9 <= e <= 8.
__device__ __forceinline__ uint32_t ue4m3_pow2(int e) {
  return e >= -6 ? static_cast<uint32_t>(e + 7) << 3 : 1u << (e + 9);
}

// smallest e with 6 * 2^e >= m, from the bits of m >= 0
__device__ __forceinline__ int block_exponent(uint32_t bits) {
  return static_cast<int>(bits >> 23) - 129 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
}

// Slices of the chunk held by kLanes consecutive lanes, eight values each (two lanes a block).
// Every lane of the warp calls it.  The exponent of the chunk is kept above -100 so that F and
// 1/F are normal numbers: values below 2^-120 lose their last bits, absolutely below 2^-117.
template <int kLanes>
__device__ __forceinline__ Slices slice8(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  const uint32_t mb = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  uint32_t mc = mb;
#pragma unroll
  for (int o = 2; o < kLanes; o <<= 1) mc = max(mc, __shfl_xor_sync(0xffffffffu, mc, o));
  const bool finite = mc < 0x7f800000u;          // infinities and NaN compare above every finite magnitude
  const int ec = finite ? max(block_exponent(mc), -100) : 0;
  const int sb = finite ? max(block_exponent(mb) - ec + 8, -1) : 0;
  const float down = pow2_int(8 - ec);
  const float up = finite ? pow2_int(-sb) : 0.0f;
  Slices s;
  s.factor = finite ? pow2_int(ec - 8) : __uint_as_float(0x7fffffffu);
  s.sf = ue4m3_pow2(sb) | (ue4m3_pow2(sb - 2) << 8) | (ue4m3_pow2(sb - 5) << 16) | (ue4m3_pow2(sb - 8) << 24);
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = finite ? (v[i] * down) * up : 0.0f;
#pragma unroll
  for (int l = 0; l < kSlices; ++l) {
    s.q[l] = e2m1x8(z);
    if (l + 1 < kSlices) {
      const float next = l == 0 ? 4.0f : 8.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = minus_e2m1(z[i], s.q[l], i) * next;
    }
  }
  return s;
}

// Writes the slices of eight values at K position k8 * 8 (k8 < 32) of a stage block: scale chunk
// bytes first, then the 128-byte rows of the MMA's N operand with the 128-byte swizzle.
__device__ __forceinline__ void store_slices(uint8_t* block, int slot, int k8, const Slices& s, const uint8_t* base,
                                             uint64_t extent, int* status) {
#pragma unroll
  for (int l = 0; l < kSlices; ++l) {
    const int r = slot * kSlices + l;
    uint8_t* row = block + kSfBlockBytes + r * 128 + (((k8 >> 2) ^ (r & 7)) << 4) + (k8 & 3) * 4;
    if (index_ok(static_cast<uint64_t>(row - base) + 3, extent, status)) *reinterpret_cast<uint32_t*>(row) = s.q[l];
    if ((k8 & 1) == 0) {
      uint8_t* sf = block + (k8 >> 3) * 512 + (r & 31) * 16 + (r >> 5) * 4 + ((k8 >> 1) & 3);
      if (index_ok(static_cast<uint64_t>(sf - base), extent, status)) *sf = static_cast<uint8_t>(s.sf >> (8 * l));
    }
  }
}

// ---- grouping and the slices of x -----------------------------------------------------------------

__global__ void __launch_bounds__(256) moe_prepare_kernel(const MoeParams p) {
  __shared__ int ids[kMoeMaxSlots];
  __shared__ int rank[kMoeMaxSlots];
  __shared__ int count[kMoeMaxExperts];          // slots of the expert
  __shared__ int first[kMoeMaxExperts];          // its first position, segment and offset
  __shared__ int seg0[kMoeMaxExperts];
  __shared__ int off0[kMoeMaxExperts];
  const int S = p.t * p.topk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  for (int i = tid; i < S; i += 256) {
    const int e = p.ids[i];
    ids[i] = e >= 0 && e < p.experts ? e : -1;
  }
  for (int e = tid; e < p.experts; e += 256) count[e] = 0;
  // the tile counters of the two GEMM kernels
  const int ups = p.max_segments * ((p.n + 127) / 128), downs = (p.k + 127) / 128;
  for (int i = blockIdx.x * 256 + tid; i < ups + downs; i += gridDim.x * 256) {
    if (i < ups) p.count_up[i] = 0;
    else p.count_down[i - ups] = 0;
  }
  __syncthreads();
  if (warp == 0) {
    // a slot's rank among the slots of its expert, in slot order
    for (int i0 = 0; i0 < S; i0 += 32) {
      const int e = i0 + lane < S ? ids[i0 + lane] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int old = e >= 0 ? count[e] : 0;
      __syncwarp();
      if (e >= 0) {
        rank[i0 + lane] = old + before;
        if (before == 0) count[e] = old + __popc(same);
      }
      __syncwarp();
    }
    int pos = 0, seg = 0, off = 0;               // running totals over the experts
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int c = e0 + lane < p.experts ? count[e0 + lane] : 0;
      const int full = c / kSegSlots, rest = c % kSegSlots;
      int a = c, b = full + (rest ? 1 : 0);
      int o = full * (kSfBlockBytes + 64 * 128) + (rest ? kSfBlockBytes + segment_columns(rest) * 128 : 0);
      const int a1 = a, b1 = b, o1 = o;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int ta = __shfl_up_sync(0xffffffffu, a, d), tb = __shfl_up_sync(0xffffffffu, b, d),
                  to = __shfl_up_sync(0xffffffffu, o, d);
        if (lane >= d) a += ta, b += tb, o += to;
      }
      if (e0 + lane < p.experts) {
        first[e0 + lane] = pos + a - a1;
        seg0[e0 + lane] = seg + b - b1;
        off0[e0 + lane] = off + o - o1;
      }
      pos += __shfl_sync(0xffffffffu, a, 31);
      seg += __shfl_sync(0xffffffffu, b, 31);
      off += __shfl_sync(0xffffffffu, o, 31);
    }
    if (blockIdx.x == 0 && lane == 0) *p.nseg = seg;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = tid; e < p.experts; e += 256) {
      for (int j = 0; j * kSegSlots < count[e]; ++j) {
        Segment s;
        s.expert = e;
        s.first = first[e] + j * kSegSlots;
        s.count = min(count[e] - j * kSegSlots, kSegSlots);
        s.offset = off0[e] + j * (kSfBlockBytes + 64 * 128);
        if (index_ok(seg0[e] + j, p.max_segments, p.status)) p.segments[seg0[e] + j] = s;
      }
    }
    for (int i = tid; i < S; i += 256) {
      if (ids[i] >= 0 && index_ok(first[ids[i]] + rank[i], S, p.status)) p.pos_slot[first[ids[i]] + rank[i]] = i;
    }
  }
  // one warp per (slot, 256 values of x): eight values a lane
  const int ks1 = (p.k + 255) / 256;
  for (int item = blockIdx.x * 8 + warp; item < S * ks1; item += gridDim.x * 8) {
    const int i = item / ks1, ks = item - i * ks1;
    const int e = ids[i];
    if (e < 0) continue;
    const int j = rank[i] / kSegSlots, slot = rank[i] % kSegSlots;
    const int cols = segment_columns(min(count[e] - j * kSegSlots, kSegSlots));
    const int64_t off = off0[e] + j * (kSfBlockBytes + 64 * 128);
    const int c = ks * 256 + lane * 8;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    const int64_t src = static_cast<int64_t>(i / p.topk) * p.k + c;
    if (c < p.k && index_ok(src + 7, static_cast<uint64_t>(p.t) * p.k, p.status))
      raw = __ldg(reinterpret_cast<const uint4*>(p.x + src));
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[2 * q] = bf16_lo(w[q]), v[2 * q + 1] = bf16_hi(w[q]);
    const Slices s = slice8<32>(v);
    uint8_t* block = p.b_x + off * ks1 + static_cast<int64_t>(ks) * (kSfBlockBytes + cols * 128);
    store_slices(block, slot, lane, s, p.b_x, static_cast<uint64_t>(p.b_units) * ks1, p.status);
    const int f = ((seg0[e] + j) * ks1 + ks) * kSegSlots + slot;
    if (lane == 0 && index_ok(f, static_cast<uint64_t>(p.max_segments) * ks1 * kSegSlots, p.status)) p.f_x[f] = s.factor;
  }
}

// ---- the GEMM kernels --------------------------------------------------------------------------------

struct MoeMaps {
  CUtensorMap w0, w1;           // gate and up, or down (w0)
};

// The factors F of a stage travel with its loads into a ring of their own, because the epilogue reads them after the MMAs
// have given the stage's slot back: the load of unit i + 8 waits for the MMAs of unit i + 8 - kStages (i + 3 or later), and
// those for the epilogue's release of the accumulator that unit i + 1 used.
constexpr int kFactorRing = 8;
constexpr int kFactorBytes = 2 * kSegSlots * 4;

template <bool kDown>
struct MoeSmem {
  static constexpr int kStages = kDown ? 5 : 4;
  static constexpr int kTiles = kDown ? 1 : 2;
  static constexpr int kBAt = kTiles * kTileBytes;               // the activations' block: scales, then rows
  static constexpr int kSfaAt = kBAt + kSfBlockBytes + kRowsBytes;
  static constexpr int kStageBytes = kSfaAt + kTiles * kSfBlockBytes;
  // after the ring: up: sums of gate and up [2][16][128] fp32; down: the CTA's sums for every token,
  // one copy per half of K stages [2][t][128] fp32
  static constexpr int kSumBytes = kDown ? 2 * kMoeMaxTokens * 128 * 4 : 2 * kSegSlots * 128 * 4;
  static constexpr int kBytes = kStages * kStageBytes + kSumBytes + kFactorRing * kFactorBytes + 256 + 1024;
  static_assert(kStageBytes % 1024 == 0 && kBytes <= 227 * 1024, "shared memory layout");
};

struct __align__(8) MoeControl {
  uint64_t full[5], empty[5];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int32_t abort;
  int32_t last;
};
static_assert(sizeof(MoeControl) <= 256, "control block");

constexpr uint32_t kMoeTmemCols = 512;
constexpr uint32_t kMoeSfCol = 256;              // scales after two accumulator buffers of 2 x 64 columns

// This CTA's range of units, and what finishing a shared tile needs.
struct MoeSplit {
  int64_t units, begin, end;
  int upt;                                       // units per tile
  int ctas;
  __device__ __forceinline__ MoeSplit(int64_t tiles, int upt_) : units(tiles * upt_), upt(upt_) {
    ctas = static_cast<int>(units < gridDim.x ? units : gridDim.x);
    const int c = blockIdx.x;
    begin = c < ctas ? start(c) : 0;
    end = c < ctas ? start(c + 1) : 0;
  }
  __device__ __forceinline__ int64_t start(int c) const { return c * units / ctas; }
  __device__ __forceinline__ int cta_of(int64_t u) const { return static_cast<int>(((u + 1) * ctas - 1) / units); }
};

// Walks a CTA's units: the tile, its segment, row tile and K stage.
template <bool kDown>
struct MoeWalk {
  int tile, in, sg, ks, rt;
  int stages, row_tiles, upt;
  __device__ __forceinline__ MoeWalk(const MoeSplit& s, int stages_, int row_tiles_)
      : stages(stages_), row_tiles(row_tiles_), upt(s.upt) {
    tile = s.units ? static_cast<int>(s.begin / upt) : 0;
    in = s.units ? static_cast<int>(s.begin - static_cast<int64_t>(tile) * upt) : 0;
    sg = kDown ? in / stages : tile / row_tiles;
    ks = kDown ? in - sg * stages : in;
    rt = kDown ? tile : tile - sg * row_tiles;
  }
  __device__ __forceinline__ void next() {
    ++in;
    ++ks;
    if (kDown && ks == stages) {
      ks = 0;
      ++sg;
    }
    if (in == upt) {
      in = ks = 0;
      ++tile;
      ++rt;
      if (kDown) {
        sg = 0;
      } else if (rt == row_tiles) {
        rt = 0;
        ++sg;
      }
    }
  }
};

// The segment of the current unit, with the one after it already on its way.
struct SegmentCursor {
  const Segment* table;
  Segment now, next;
  int nseg, at;
  __device__ __forceinline__ SegmentCursor(const Segment* t, int n, int sg) : table(t), now{}, next{}, nseg(n), at(sg) {
    if (n == 0) return;
    now = table[sg];
    next = table[sg + 1 < n ? sg + 1 : 0];
  }
  // true when sg begins a segment other than the last one asked for
  __device__ __forceinline__ bool move(int sg) {
    if (sg == at) return false;
    at = sg;
    now = next;
    next = table[sg + 1 < nseg ? sg + 1 : 0];
    return true;
  }
};

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <bool kDown>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_kernel(const __grid_constant__ MoeMaps maps, const MoeParams p) {
  using L = MoeSmem<kDown>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sums = reinterpret_cast<float*>(smem + L::kStages * L::kStageBytes);
  float* factors = sums + L::kSumBytes / 4;
  MoeControl& ctl = *reinterpret_cast<MoeControl*>(factors + kFactorRing * kFactorBytes / 4);
  volatile int32_t* abort = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.acc_full[b], 1);
      mbar_init(&ctl.acc_empty[b], 8);
    }
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem_base)),
                 "r"(kMoeTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  const int nseg = *p.nseg;
  const int kdim = kDown ? p.n : p.k;            // the contraction
  const int stages = (kdim + 255) / 256;
  const int row_tiles = ((kDown ? p.k : p.n) + 127) / 128;
  const int groups = kdim / 64;
  const uint8_t* blocks = kDown ? p.b_h : p.b_x;
  // up: tiles are (segment, 128 rows of gate and up); down: 128 rows of the output over all segments
  const MoeSplit split(kDown ? row_tiles : static_cast<int64_t>(nseg) * row_tiles, kDown ? nseg * stages : stages);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (elect_one()) {
      prefetch_map(&maps.w0);
      if constexpr (!kDown) prefetch_map(&maps.w1);
    }
    __syncwarp();
    uint32_t slot = 0, phase = 0, i = 0;
    bool wrapped = false;
    MoeWalk<kDown> w(split, stages, row_tiles);
    SegmentCursor cursor(p.segments, nseg, w.sg);
    for (int64_t u = split.begin; u < split.end; ++u, ++i, w.next()) {
      const int sg = w.sg, ks = w.ks, rt = w.rt;
      cursor.move(sg);
      const Segment& seg = cursor.now;
      if (wrapped && !mbar_wait_fast(&ctl.empty[slot], phase, abort, p.status)) break;
      if (elect_one()) {
        uint8_t* st = smem + slot * L::kStageBytes;
        uint64_t* full = &ctl.full[slot];
        const uint32_t sf_bytes = static_cast<uint32_t>(min(4, groups - 4 * ks)) * 512u;
        const uint32_t b_bytes = kSfBlockBytes + segment_columns(seg.count) * 128;
        const int64_t sf_at = seg.expert * p.sf_stride + (static_cast<int64_t>(rt) * groups + 4 * ks) * 512;
        constexpr uint32_t f_bytes = kDown ? kFactorBytes : kFactorBytes / 2;
        mbar_arrive_expect_tx(full, L::kTiles * (kTileBytes + sf_bytes) + b_bytes + f_bytes);
        tma_load_3d_cta(st, &maps.w0, full, ks * 128, rt * 128, seg.expert);
        if constexpr (!kDown) tma_load_3d_cta(st + kTileBytes, &maps.w1, full, ks * 128, rt * 128, seg.expert);
        bulk_load_cta(st + L::kBAt, blocks + static_cast<int64_t>(seg.offset) * stages + static_cast<int64_t>(ks) * b_bytes,
                      b_bytes, full);
        bulk_load_cta(factors + (i % kFactorRing) * (kFactorBytes / 4),
                      (kDown ? p.f_h : p.f_x) + (static_cast<int64_t>(sg) * stages + ks) * (f_bytes / 4), f_bytes, full);
        bulk_load_cta(st + L::kSfaAt, p.sf0 + sf_at, sf_bytes, full);
        if constexpr (!kDown) bulk_load_cta(st + L::kSfaAt + kSfBlockBytes, p.sf1 + sf_at, sf_bytes, full);
      }
      __syncwarp();
      if (++slot == L::kStages) {
        slot = 0;
        if (wrapped) phase ^= 1u;
        wrapped = true;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t smem0 = smem_u32(smem);
    uint32_t slot = 0, phase = 0, i = 0;
    MoeWalk<kDown> w(split, stages, row_tiles);
    SegmentCursor cursor(p.segments, nseg, w.sg);
    for (int64_t u = split.begin; u < split.end; ++u, ++i, w.next()) {
      const int ks = w.ks;
      cursor.move(w.sg);
      const int columns = segment_columns(cursor.now.count);
      const uint32_t b = i & 1u;
      if (i >= 2 && !mbar_wait_fast(&ctl.acc_empty[b], ((i >> 1) - 1u) & 1u, abort, p.status)) break;
      if (!mbar_wait_fast(&ctl.full[slot], phase, abort, p.status)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t st = smem0 + slot * L::kStageBytes;
        const uint32_t idesc = idesc_fp4_cta(static_cast<uint32_t>(columns));
        const uint64_t a0 = operand_desc(st), a1 = operand_desc(st + kTileBytes);
        const uint64_t b0 = operand_desc(st + L::kBAt + kSfBlockBytes);
        const uint64_t sfa = sf_chunk_desc(st + L::kSfaAt), sfb = sf_chunk_desc(st + L::kBAt);
        const uint32_t acc = tmem + b * 128u;
        const int steps = min(4, groups - 4 * ks);
        for (int j = 0; j < steps; ++j) {
          const uint32_t col = tmem + kMoeSfCol + 12u * j;
          tc_copy_sf_cta(col, sfa + 32 * j);
          if constexpr (!kDown) tc_copy_sf_cta(col + 4, sfa + (kSfBlockBytes >> 4) + 32 * j);
          tc_copy_sf_cta(col + 8, sfb + 32 * j);
          if constexpr (kDown) {
            // K values [0, 128) of the stage into one accumulator, [128, 256) into the other: h has a factor for each
            mma_fp4_cta(acc + (j >> 1) * 64u, a0 + 2 * j, b0 + 2 * j, idesc, col, col + 8, j & 1);
          } else {
            mma_fp4_cta(acc, a0 + 2 * j, b0 + 2 * j, idesc, col, col + 8, j > 0);
            mma_fp4_cta(acc + 64u, a1 + 2 * j, b0 + 2 * j, idesc, col + 4, col + 8, j > 0);
          }
        }
        mma_commit_cta(&ctl.empty[slot]);
        mma_commit_cta(&ctl.acc_full[b]);
      }
      __syncwarp();
      if (++slot == L::kStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    // Eight warps, two per TMEM lane quarter: half 0 reads the first accumulator of a stage (gate, or K values
    // [0, 128)), half 1 the second (up, or [128, 256)).  A thread owns one weight row and adds, per slot, its four
    // slices times the chunk's factor into fp32 registers.  Once a wait has given up the loops
    // run on without waiting, so that every barrier below still meets all eight warps.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;
    const int tid = threadIdx.x - 64;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    float acc[kSegSlots];
#pragma unroll
    for (int s = 0; s < kSegSlots; ++s) acc[s] = 0.0f;
    if (kDown && nseg == 0) {
      // no token has an expert: the output is zero
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + tid; i < static_cast<int64_t>(p.t) * p.k / 8;
           i += static_cast<int64_t>(gridDim.x) * 256)
        reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (kDown) {
      for (int i = 0; i < p.t; ++i) sums[(half * p.t + i) * 128 + row] = 0.0f;
    }
    uint32_t i = 0;
    MoeWalk<kDown> w(split, stages, row_tiles);
    SegmentCursor cursor(p.segments, nseg, w.sg);
    // what the end of a segment or tile needs is loaded when the segment begins
    int token = 0;                               // down: token of slot lane % 16
    float sg0 = 0.0f, su = 0.0f, sd = 0.0f;      // up: global scales; sd with the routing weight of slot tid / 16
    auto begin_segment = [&]() {
      const Segment& seg = cursor.now;
      if constexpr (kDown) {
        token = (lane & 15) < seg.count ? p.pos_slot[seg.first + (lane & 15)] / p.topk : 0;
      } else {
        sg0 = p.amax0[seg.expert] * (1.0f / 2688.0f);
        su = p.amax1[seg.expert] * (1.0f / 2688.0f);
        sd = (tid >> 4) < seg.count ? p.weights[p.pos_slot[seg.first + (tid >> 4)]] * (p.amax_down[seg.expert] * (1.0f / 2688.0f))
                                    : 0.0f;
      }
    };
    if (split.begin < split.end) begin_segment();
    for (int64_t u = split.begin; u < split.end; ++u, ++i, w.next()) {
      const int tile = w.tile, sg = w.sg, ks = w.ks;
      if (cursor.move(sg)) begin_segment();
      const Segment& seg = cursor.now;
      const float* f = factors + (i % kFactorRing) * (kFactorBytes / 4) + (kDown ? half * kSegSlots : 0);
      const uint32_t b = i & 1u;
      if (ok) ok = mbar_wait_fast(&ctl.acc_full[b], (i >> 1) & 1u, abort, p.status);
      tc_fence_after();
      const uint32_t at = tmem + b * 128u + half * 64u + lane_base;
      uint32_t v[64];
      if (!kDown || half == 0 || groups - 4 * ks > 2) {
        if (seg.count <= 4) {
          tmem_load_16(at, v);
          tmem_wait_ld<16>(v);
        } else if (seg.count <= 8) {
          tmem_load_32(at, v);
          tmem_wait_ld<32>(v);
        } else {
          tmem_load_64(at, v);
          tmem_wait_ld<64>(v);
        }
#pragma unroll
        for (int s = 0; s < kSegSlots; ++s) {
          if (s < seg.count) {
            const float sum = (__uint_as_float(v[4 * s]) + __uint_as_float(v[4 * s + 1])) +
                              (__uint_as_float(v[4 * s + 2]) + __uint_as_float(v[4 * s + 3]));
            acc[s] = fmaf(f[s], sum, acc[s]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.acc_empty[b]);

      const bool tile_end = u + 1 == split.end || w.in + 1 == split.upt;
      if constexpr (kDown) {
        if (ks + 1 == stages || tile_end) {
          // the segment's rows for its tokens; this thread alone adds to (half, token, row)
#pragma unroll
          for (int s = 0; s < kSegSlots; ++s) {
            if (s < seg.count) {
              const int i_tok = __shfl_sync(0xffffffffu, token, s);
              sums[(half * p.t + i_tok) * 128 + row] += acc[s];
            }
            acc[s] = 0.0f;
          }
        }
      }
      if (!tile_end) continue;

      const int64_t tile0 = static_cast<int64_t>(tile) * split.upt;
      const int c0 = split.cta_of(tile0), c1 = split.cta_of(tile0 + split.upt - 1);
      // CTA c keeps its partial sums at place 2c for the first tile of its range, 2c + 1 for its last: every CTA after c0
      // begins inside this tile, c0 may have begun before it
      const int first_place = 2 * c0 + (split.start(c0) < tile0 ? 1 : 0);
      const int width = kDown ? p.t * 128 : seg.count * 128;       // fp32 values of one half
      if constexpr (!kDown) {
#pragma unroll
        for (int s = 0; s < kSegSlots; ++s) {
          if (s < seg.count) sums[(half * seg.count + s) * 128 + row] = acc[s];
          acc[s] = 0.0f;
        }
      }
      epilogue_sync();
      bool finish = true;
      if (c0 != c1) {
        // shared with other CTAs: leave the partial sums, and the last CTA to do so adds them up
        float* parts = kDown ? p.part_down : p.part_up;
        const int64_t stride = kDown ? static_cast<int64_t>(p.t) * 128 : 2 * kSegSlots * 128;
        const int n_out = kDown ? width : 2 * width;
        float* mine_out = parts + (static_cast<int>(blockIdx.x) == c0 ? first_place : 2 * static_cast<int>(blockIdx.x)) * stride;
        for (int j = tid * 4; j < n_out; j += 1024) {
          float4 a = *reinterpret_cast<const float4*>(sums + j);
          if constexpr (kDown) {
            const float4 c = *reinterpret_cast<const float4*>(sums + width + j);
            a = make_float4(a.x + c.x, a.y + c.y, a.z + c.z, a.w + c.w);
          }
          __stcg(reinterpret_cast<float4*>(mine_out + j), a);
        }
        __threadfence();
        epilogue_sync();
        if (tid == 0)
          ctl.last = atomicAdd((kDown ? p.count_down : p.count_up) + tile, 1u) == static_cast<uint32_t>(c1 - c0);
        epilogue_sync();
        finish = ctl.last != 0;
        if (finish) {
          __threadfence();
          for (int j = tid * 4; j < n_out; j += 1024) {
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              const float4 b4 = __ldcg(reinterpret_cast<const float4*>(parts + (c == c0 ? first_place : 2 * c) * stride + j));
              a = make_float4(a.x + b4.x, a.y + b4.y, a.z + b4.z, a.w + b4.w);
            }
            *reinterpret_cast<float4*>(sums + j) = a;
            if constexpr (kDown) *reinterpret_cast<float4*>(sums + width + j) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
          epilogue_sync();
        }
      }
      if (finish) {
        if constexpr (kDown) {
          for (int j = tid; j < p.t * 64; j += 256) {
            const int token = j >> 6, r = (j & 63) * 2;
            const int col = tile * 128 + r;
            const float* s0 = sums + token * 128 + r;
            const int64_t o = static_cast<int64_t>(token) * p.k + col;
            if (col < p.k && index_ok(o + 1, static_cast<uint64_t>(p.t) * p.k, p.status))
              *reinterpret_cast<uint32_t*>(p.out + o) = pack_bf16x2(s0[0] + s0[width], s0[1] + s0[width + 1]);
          }
        } else {
          // sixteen lanes a slot, eight rows a lane: h = silu(g) * u in fp32, written as slices; F carries the
          // routing weight and the down projection's global scale
          const int s = tid >> 4, l16 = tid & 15;
          const int rt = w.rt;
          const bool valid = s < seg.count;
          float h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float g = valid ? sums[s * 128 + l16 * 8 + e] * sg0 : 0.0f;
            const float up = valid ? sums[width + s * 128 + l16 * 8 + e] * su : 0.0f;
            h[e] = g / (1.0f + expf(-g)) * up;
          }
          const Slices sl = slice8<16>(h);
          const int hs = (p.n + 255) / 256;                // K stages of the down projection
          if (valid && rt * 128 + l16 * 8 < p.n) {
            uint8_t* block = p.b_h + static_cast<int64_t>(seg.offset) * hs +
                             static_cast<int64_t>(rt >> 1) * (kSfBlockBytes + segment_columns(seg.count) * 128);
            store_slices(block, s, (rt & 1) * 16 + l16, sl, p.b_h, static_cast<uint64_t>(p.b_units) * hs, p.status);
            if (l16 == 0) {
              const int fo = (sg * 2 * hs + rt) * kSegSlots + s;
              if (index_ok(fo, static_cast<uint64_t>(p.max_segments) * 2 * hs * kSegSlots, p.status))
                p.f_h[fo] = sl.factor * sd;
            }
          }
        }
      }
      epilogue_sync();                           // the sums are free again
      if constexpr (kDown) {
        for (int j = 0; j < p.t; ++j) sums[(half * p.t + j) * 128 + row] = 0.0f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort) {
    const uint64_t t0 = global_ns();             // bounded time for copies and MMAs in flight to drain
    while (global_ns() - t0 < 2000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kMoeTmemCols) : "memory");
  }
}

// ---- the router --------------------------------------------------------------------------------------

// One warp a token; a lane holds kPer consecutive logits as order-preserving keys (0: masked).
// topk times the warp takes the largest key (one redux), the lowest lane that holds it and that lane's first such
// logit, so equal logits go to the lowest index; only that lane looks its keys through again.
template <int kPer, typename T>
__global__ void __launch_bounds__(256) moe_route_kernel(const T* logits, int t, int experts, int topk, int weighting,
                                                        int32_t* ids, float* weights, int* status) {
  const int token = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  if (token >= t) return;
  uint32_t key[kPer];
  const int64_t row = static_cast<int64_t>(token) * experts;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * kPer + j;
    float x = __uint_as_float(0xff800000u);
    if (e < experts && index_ok(row + e, static_cast<uint64_t>(t) * experts, status)) {
      if constexpr (sizeof(T) == 2) x = __uint_as_float(static_cast<uint32_t>(logits[row + e]) << 16);
      else x = logits[row + e];
    }
    const uint32_t b = __float_as_uint(fminf(x, 3.402823466e38f) + 0.0f);     // -0 equals 0; +inf counts as FLT_MAX
    key[j] = x > __uint_as_float(0xff800000u) ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;   // NaN: masked
  }
  auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k); };
  uint32_t best = 0;
  int at = 0;
  auto look = [&]() {
    best = key[0];
    at = 0;
#pragma unroll
    for (int j = 1; j < kPer; ++j)
      if (key[j] > best) best = key[j], at = j;
  };
  look();
  const uint32_t top_key = __reduce_max_sync(0xffffffffu, best);
  const float top = value(top_key);
  float total = 0.0f;
  if (weighting == NVFP4_ROUTE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (key[j]) total += expf(value(key[j]) - top);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  uint32_t my_key = 0;
  int my_id = -1;
  for (int r = 0; r < topk; ++r) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0) break;                           // only masked logits are left
    const int owner = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
    const int id = __shfl_sync(0xffffffffu, lane * kPer + at, owner);
    if (lane == r) my_key = m, my_id = id;
    if (lane == owner) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j == at) key[j] = 0;
      look();
    }
  }
  const float logit = value(my_key);
  float w = 0.0f;
  if (my_id >= 0) w = weighting == NVFP4_ROUTE_SIGMOID ? 1.0f / (1.0f + expf(-logit)) : expf(logit - top);
  if (weighting == NVFP4_ROUTE_SOFTMAX_SELECTED) {
    total = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (weighting != NVFP4_ROUTE_SIGMOID && my_id >= 0) w = w / total;
  const int64_t o = static_cast<int64_t>(token) * topk + lane;
  if (lane < topk && index_ok(o, static_cast<uint64_t>(t) * topk, status)) {
    ids[o] = my_id;
    weights[o] = w;
  }
}

// ---- host side ----------------------------------------------------------------------------------------

template <typename T>
int run_route(const void* logits, int t, int experts, int topk, int weighting, int32_t* ids, float* weights, int* status,
              cudaStream_t stream) {
  const dim3 grid((t + 7) / 8), block(256);
  const T* x = static_cast<const T*>(logits);
  const int per = (experts + 31) / 32;
  if (per <= 1) return launch_kernel(moe_route_kernel<1, T>, grid, block, 0, stream, x, t, experts, topk, weighting, ids, weights, status);
  if (per <= 2) return launch_kernel(moe_route_kernel<2, T>, grid, block, 0, stream, x, t, experts, topk, weighting, ids, weights, status);
  if (per <= 4) return launch_kernel(moe_route_kernel<4, T>, grid, block, 0, stream, x, t, experts, topk, weighting, ids, weights, status);
  if (per <= 8) return launch_kernel(moe_route_kernel<8, T>, grid, block, 0, stream, x, t, experts, topk, weighting, ids, weights, status);
  if (per <= 16) return launch_kernel(moe_route_kernel<16, T>, grid, block, 0, stream, x, t, experts, topk, weighting, ids, weights, status);
  return launch_kernel(moe_route_kernel<32, T>, grid, block, 0, stream, x, t, experts, topk, weighting, ids, weights, status);
}

// Packed FP4 weights [experts, rows, k/2], boxes of 128 bytes x 128 rows, 128-byte swizzle.
int make_weight_map(CUtensorMap* map, const uint8_t* base, int64_t experts, int64_t rows, int64_t k) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (!encode) return NVFP4_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k / 2), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(experts)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(k / 2), static_cast<cuuint64_t>(rows * (k / 2))};
  const cuuint32_t box[3] = {128, 128, 1}, one[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NVFP4_OK : NVFP4_ERR_INVALID_ARGUMENT;
}

template <bool kDown>
int run_moe(const MoeMaps& maps, const MoeParams& p, const DeviceInfo& info, cudaStream_t stream) {
  auto kernel = moe_kernel<kDown>;
  constexpr int kSmem = MoeSmem<kDown>::kBytes;
  int ready = 0;
  const int st = kernel_setup(reinterpret_cast<const void*>(kernel), info.device, [&](int* v) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
      cudaGetLastError();
      return static_cast<int>(NVFP4_ERR_CUDA);
    }
    *v = 1;
    return static_cast<int>(NVFP4_OK);
  }, &ready);
  if (st != NVFP4_OK) return st;
  const int grid = info.sm_count < kMoeMaxCtas ? info.sm_count : kMoeMaxCtas;
  return launch_kernel(kernel, dim3(grid), dim3(kMoeThreads), kSmem, stream, maps, p);
}

bool moe_shape_ok(int64_t t, int64_t topk, int64_t E, int64_t n, int64_t k) {
  return t >= 0 && t <= kMoeMaxTokens && topk > 0 && topk <= kMoeMaxTopk && E > 0 && E <= kMoeMaxExperts && n > 0 && k > 0 &&
         n % 64 == 0 && k % 64 == 0 && n <= (1 << 20) && k <= (1 << 20);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_moe_route(const void* logits, int logits_bf16, int64_t t, int64_t E, int64_t topk, int weighting, int32_t* ids_out,
                    float* weights_out, nvfp4_stream_t stream) {
  if (t < 0 || t > (1 << 28) || E <= 0 || E > kMoeMaxExperts || topk <= 0 || topk > 32 || topk > E || weighting < 0 || weighting > 2)
    return NVFP4_ERR_INVALID_ARGUMENT;
  if (t == 0) return NVFP4_OK;
  if (!logits || !ids_out || !weights_out || !aligned(logits, logits_bf16 ? 2 : 4) || !aligned(ids_out, 4) ||
      !aligned(weights_out, 4))
    return NVFP4_ERR_INVALID_ARGUMENT;
  DeviceInfo info;
  const int st = current_device(&info);
  if (st != NVFP4_OK) return st;
  const int ti = static_cast<int>(t), e = static_cast<int>(E), kk = static_cast<int>(topk);
  return logits_bf16 ? run_route<uint16_t>(logits, ti, e, kk, weighting, ids_out, weights_out, info.status, stream)
                     : run_route<float>(logits, ti, e, kk, weighting, ids_out, weights_out, info.status, stream);
}

int64_t nvfp4_moe_few_tokens_workspace(int64_t t, int64_t topk, int64_t E, int64_t n, int64_t k) {
  if (!moe_shape_ok(t, topk, E, n, k)) return -1;
  return moe_layout(t, topk, E, n, k).bytes;
}

int nvfp4_moe_few_tokens(const void* x_bf16, const int32_t* ids, const float* weights, const uint8_t* w_gate,
                         const uint8_t* w_up, const uint8_t* w_down, const uint8_t* w_gate_sf, const uint8_t* w_up_sf,
                         const uint8_t* w_down_sf, const float* gate_amax, const float* up_amax, const float* down_amax,
                         void* out_bf16, void* workspace, int64_t workspace_bytes, int64_t t, int64_t topk, int64_t E,
                         int64_t n, int64_t k, nvfp4_stream_t stream) {
  if (!moe_shape_ok(t, topk, E, n, k)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (t == 0) return NVFP4_OK;
  const void* required[] = {x_bf16, w_gate, w_up, w_down, w_gate_sf, w_up_sf, w_down_sf, out_bf16, workspace};
  for (const void* q : required)
    if (!q || !aligned(q, 16)) return NVFP4_ERR_INVALID_ARGUMENT;
  const void* words[] = {ids, weights, gate_amax, up_amax, down_amax};
  for (const void* q : words)
    if (!q || !aligned(q, 4)) return NVFP4_ERR_INVALID_ARGUMENT;
  const MoeLayout L = moe_layout(t, topk, E, n, k);
  if (workspace_bytes < L.bytes) return NVFP4_ERR_INVALID_ARGUMENT;
  DeviceInfo info;
  int st = current_device(&info);
  if (st != NVFP4_OK) return st;
  MoeMaps up, down;
  memset(&up, 0, sizeof(up));
  memset(&down, 0, sizeof(down));
  if ((st = make_weight_map(&up.w0, w_gate, E, n, k)) != NVFP4_OK) return st;
  if ((st = make_weight_map(&up.w1, w_up, E, n, k)) != NVFP4_OK) return st;
  if ((st = make_weight_map(&down.w0, w_down, E, k, n)) != NVFP4_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeParams p;
  memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.ids = ids;
  p.weights = weights;
  p.sf0 = w_gate_sf;
  p.sf1 = w_up_sf;
  p.amax0 = gate_amax;
  p.amax1 = up_amax;
  p.amax_down = down_amax;
  p.out = static_cast<__nv_bfloat16*>(out_bf16);
  p.status = info.status;
  p.nseg = reinterpret_cast<int32_t*>(ws);
  p.segments = reinterpret_cast<Segment*>(ws + L.segments);
  p.pos_slot = reinterpret_cast<int32_t*>(ws + L.pos_slot);
  p.count_up = reinterpret_cast<uint32_t*>(ws + L.count_up);
  p.count_down = reinterpret_cast<uint32_t*>(ws + L.count_down);
  p.f_x = reinterpret_cast<float*>(ws + L.f_x);
  p.f_h = reinterpret_cast<float*>(ws + L.f_h);
  p.b_x = ws + L.b_x;
  p.b_h = ws + L.b_h;
  p.part_up = reinterpret_cast<float*>(ws + L.part_up);
  p.part_down = reinterpret_cast<float*>(ws + L.part_down);
  p.sf_stride = nvfp4_scale_bytes(n, k);
  p.b_units = L.b_units;
  p.max_segments = L.max_segments;
  p.t = static_cast<int32_t>(t);
  p.topk = static_cast<int32_t>(topk);
  p.experts = static_cast<int32_t>(E);
  p.n = static_cast<int32_t>(n);
  p.k = static_cast<int32_t>(k);
  const int64_t items = (t * topk * ((k + 255) / 256) + 7) / 8;
  const int grid = static_cast<int>(items < 2 * info.sm_count ? items : 2 * info.sm_count);
  if ((st = launch_kernel(moe_prepare_kernel, dim3(grid), dim3(256), 0, stream, p)) != NVFP4_OK) return st;
  if ((st = run_moe<false>(up, p, info, stream)) != NVFP4_OK) return st;
  p.sf0 = w_down_sf;
  p.sf_stride = nvfp4_scale_bytes(k, n);
  return run_moe<true>(down, p, info, stream);
}

}  // extern "C"
