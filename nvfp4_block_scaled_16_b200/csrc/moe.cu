// moe.cu -- a mixture-of-experts layer for a few tokens.
//
//   nvfp4_moe_few_tokens   out[i] = sum_j w_ij * Wd[e_ij] (silu(Wg[e_ij] x_i) * (Wu[e_ij] x_i))
//
// The layer's time is the reading of the chosen experts' NVFP4 weights, so every weight byte goes
// once from HBM to shared memory (TMA) and from there straight into tcgen05.mma: the 128 weight
// rows of a tile are the MMA's M side and the few activations its N side.  The activations are not
// quantized to FP4 but written as a sum of FP4 numbers, so the block-scaled FP4 MMA computes with
// them and no weight is ever unpacked.  A block's largest values are held better than bf16 would hold them, values far below
// them worse (the bounds follow):
//
//   Slices.  A 16-value block of an activation chunk with largest magnitude m becomes
//     x = F * 2^s * (d0 + d1/4 + d2/32 + d3/256) + r,   every d an e2m1 value,
//   F a power of two for the whole chunk (256 values of x, 128 of h), 2^s >= m/(6F) the smallest
//   power of two, d0 the e2m1 rounding of x/(F*2^s), d1 of four times what is left, d2 and d3 of eight times
//   what is left after that (rounding leaves at most 1, then at most 1/2: 4*1 and 8*1/2 are within e2m1).
//   The block scales 2^s, 2^(s-2), 2^(s-5), 2^(s-8) are exact in ue4m3.  |r| <= F*2^s/512, and F*2^s < m/3:
//   at most m/1536, a third of bf16's half step at m (2^-9 to 2^-8 of it).  s is at least -1 (2^(s-8) is the smallest
//   ue4m3 value), so a block more than 2^9 below the largest value M of its chunk is held to M/786432 instead.
//   Four slices are four MMA columns; their sum is taken when the accumulator is read.
//
// A segment is up to 16 (token, slot) pairs of one expert: 16, 32 or 64 MMA columns.  The kernels:
//   moe_slice_kernel  x as slices, in the shared-memory layout: one contiguous block per segment and 256 values of K
//                     (one token: left out, moe_up_kernel makes them).
//   moe_up_kernel     gate and up tiles (128 rows of each), SiLU * up in fp32, h written as slices.  Its CTAs start beside
//                     moe_slice_kernel's, group the slots by expert themselves and have weights on their way
//                     when the slices are ready.  Clusters of one to four CTAs share a tile by K.
//   moe_down_kernel   down tiles, weighted by the routing weights.  Every CTA takes the same number of (tile, 256 values
//                     of K) units; a tile that falls to several CTAs is finished by the last of them.
//                     With more than kMoeLastCtaTokens tokens it writes every slot's result instead, and
//   moe_combine_kernel  adds those of each token.
// Partial sums are added in CTA order everywhere, so results do not depend on timing.
//
// Each kernel starts beside the end of the one before it: moe_up_kernel and moe_down_kernel read only the call's inputs until that one's results are
// needed, and group the slots themselves rather than wait for a list.
//
// Measured, back to back on new weights (HBM copies at 6.53 TB/s): 8 tokens, 16 experts 8192 x 5120, about 9 of them used, 637 MB:
// 106 us (6.0 TB/s); 64 tokens, 64 experts 1408 x 2048, topk 6, 311 MB: 71 us (4.4 TB/s; gate and up stream at 6.5, the rest
// is the kernels' starts and ends); one token, 128 experts 768 x 2048, topk 8, 21 MB: 18.2 us, all starts and ends.
//
// Sources (page title, section): flashinfer PR #1774 (masked per-expert operands, silu_and_mul);
// NVIDIA/Fuser PR #5737 (routed experts NVFP4InferenceGroupedSwiGLU, f16a_nvfp4weight_scaled_mm: bf16
// activation, NVFP4 weight).  The few-token form is this library's own.
#include <cmath>
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
constexpr int kMoeMaxCtas = 192;
constexpr int kMoeLastCtaTokens = 8;
// Up to so many tokens moe_up_kernel makes the slices of x itself, for each of its tiles anew: a launch less.  Back to back in graphs
// and called one by one from Python, us, against moe_slice_kernel: 1 token, 128 experts 768 x 2048, topk 8: 18.2 and 19.2 against
// 18.5 and 21.2; 1 token, 16 experts 8192 x 5120, topk 2: 40.2 and 40.5 against 39.8 and 40.9; 2 tokens of each: 24.7 and 24.7
// against 24.0 and 25.6, 58.3 and 58.4 against 56.0 and 56.3; 8 tokens of the latter: 129 against 105.
constexpr int kMoeConvertTokens = 1;

struct Segment {
  int32_t expert, first, count, offset;          // offset: kBlockUnit bytes per K stage of all segments before it
};

constexpr int kBlockUnit = 2048;
__host__ __device__ inline int segment_columns(int count) { return count <= 4 ? 16 : (count <= 8 ? 32 : 64); }
// bytes of a segment's block of one K stage: scale chunks, then the rows of its columns
__host__ __device__ inline int block_bytes(int count) { return kSfBlockBytes + segment_columns(count) * 128; }

// Byte offsets of the caller's workspace: what one kernel leaves for the next, and partial sums.
struct MoeLayout {
  int64_t segments, slot_pos, count, f_x, f_h, b_x, b_h, part, rest, bytes;
  int64_t b_units;                               // bound of a K stage's bytes over all segments
  int32_t max_segments;
};

MoeLayout moe_layout(int64_t t, int64_t topk, int64_t E, int64_t n, int64_t k) {
  const int64_t S = t * topk;
  const int64_t hit = S < E ? S : E;
  const int64_t segs = hit + S / kSegSlots < S ? hit + S / kSegSlots : S;
  const int64_t ks1 = (k + 255) / 256, ks = (n + 255) / 256;
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
  L.slot_pos = take(S * 4);
  L.count = take((k + 127) / 128 * 4);
  L.f_x = take(segs * ks1 * kSegSlots * 4);
  L.f_h = take(segs * 2 * ks * kSegSlots * 4);
  L.b_x = take(L.b_units * ks1);
  L.b_h = take(L.b_units * ks);
  // few tokens: sums of every token for the tiles that CTAs share; else every slot's result, and what CTAs add to those
  // that another one began
  L.part = take(t <= kMoeLastCtaTokens ? static_cast<int64_t>(kMoeMaxCtas) * 2 * t * 128 * 4 : S * k * 4);
  L.rest = take(t <= kMoeLastCtaTokens ? 0 : static_cast<int64_t>(kMoeMaxCtas) * kSegSlots * 128 * 4);
  L.bytes = at;
  return L;
}

struct MoeParams {
  const uint16_t* x;            // [t, k] bf16
  const int32_t* ids;           // [t * topk]
  const float* weights;         // [t * topk]
  const uint8_t *gate_sf, *up_sf, *down_sf;
  const float *gate_amax, *up_amax, *down_amax;
  __nv_bfloat16* out;           // [t, k]
  int* status;
  int32_t* nseg;
  Segment* segments;
  uint32_t* slot_pos;           // of each slot: position (low 16 bits) and segment, or kNoPosition
  uint32_t* count;              // down: CTAs that left their sums of a tile
  float *f_x, *f_h;             // F of x [segment][stage][16]; F of h with routing weight and global scale [segment][2 * stage][16]
  uint8_t *b_x, *b_h;           // slices of x and h: one block per segment and K stage
  float *part, *rest;
  int64_t up_stride, down_stride;   // nvfp4_scale_bytes of one expert's matrix
  int64_t b_units;              // extents of b_x and b_h per K stage, for the debug build's index checks
  int32_t max_segments;
  int32_t t, topk, experts, n, k;
  int32_t down_ctas;            // grid of moe_down_kernel
  int32_t down_early;           // it loads weights before moe_up_kernel is done
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

// Writes the slices of eight values at K position k8 * 8 (k8 < 32) of a stage block of `columns` rows: scale chunk
// bytes first, then the 128-byte rows of the MMA's N operand with the 128-byte swizzle.  Slice l of a slot is row
// l * columns / 4 + slot, so that the accumulator columns of neighbouring slots are neighbours.
__device__ __forceinline__ void put_slices(uint8_t* block, int columns, int slot, int k8, const Slices& s) {
#pragma unroll
  for (int l = 0; l < kSlices; ++l) {
    const int r = l * (columns >> 2) + slot;
    *reinterpret_cast<uint32_t*>(block + kSfBlockBytes + r * 128 + (((k8 >> 2) ^ (r & 7)) << 4) + (k8 & 3) * 4) = s.q[l];
    if ((k8 & 1) == 0)
      block[(k8 >> 3) * 512 + (r & 31) * 16 + (r >> 5) * 4 + ((k8 >> 1) & 3)] = static_cast<uint8_t>(s.sf >> (8 * l));
  }
}

// ---- grouping -----------------------------------------------------------------------------------

// The slots are sorted by expert, in slot order within an expert, and each expert's cut into segments.
struct Grouping {
  uint32_t* count;                               // [experts] slots of the expert
  uint16_t *seg0, *off0;                         // [experts] its first segment and that one's offset
  uint16_t* id;                                  // [slots] expert of the slot, or kNoExpert
  __device__ __forceinline__ Grouping(uint8_t* at, int experts)
      : count(reinterpret_cast<uint32_t*>(at)), seg0(reinterpret_cast<uint16_t*>(at + 4 * experts)), off0(seg0 + experts),
        id(off0 + experts) {}
};
__host__ __device__ constexpr int grouping_bytes(int experts, int slots) { return 8 * experts + 2 * slots; }
constexpr uint32_t kNoExpert = 0xffffu, kNoPosition = 0xffffffffu;

// Number of segments of an expert with c slots, and their kBlockUnits per K stage.
__device__ __forceinline__ int segments_of(int c) { return (c + kSegSlots - 1) / kSegSlots; }
__device__ __forceinline__ int units_of(int c) {
  const int rest = c % kSegSlots;
  return c / kSegSlots * (block_bytes(kSegSlots) / kBlockUnit) + (rest ? block_bytes(rest) / kBlockUnit : 0);
}

// With id and count filled: seg0 and off0, the experts' first positions when `first` is given, and the number of segments.
// Called by one warp; a lane takes a run of experts.
__device__ __forceinline__ int place_experts(int experts, const Grouping& g, uint16_t* first) {
  const int lane = threadIdx.x & 31, per = (experts + 31) / 32;
  const int e0 = min(lane * per, experts), e1 = min(e0 + per, experts);
  int pos = 0, seg = 0, off = 0;
  for (int e = e0; e < e1; ++e) {
    const int c = static_cast<int>(g.count[e]);
    pos += c, seg += segments_of(c), off += units_of(c);
  }
  const int pos1 = pos, seg1 = seg, off1 = off;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, pos, d), b = __shfl_up_sync(0xffffffffu, seg, d),
              o = __shfl_up_sync(0xffffffffu, off, d);
    if (lane >= d) pos += a, seg += b, off += o;
  }
  const int total = __shfl_sync(0xffffffffu, seg, 31);
  pos -= pos1, seg -= seg1, off -= off1;
  for (int e = e0; e < e1; ++e) {
    const int c = static_cast<int>(g.count[e]);
    if (first) first[e] = static_cast<uint16_t>(pos);
    g.seg0[e] = static_cast<uint16_t>(seg);
    g.off0[e] = static_cast<uint16_t>(off);
    pos += c, seg += segments_of(c), off += units_of(c);
  }
  return total;
}

// The segments in shared memory: expert (10 bits), count (5 bits), first position (from bit 16); offset.  Of each position its
// routing weight (kWeights) or token (kTokens).
template <bool kWeights_, bool kTokens_>
struct SegmentTable {
  static constexpr bool kWeights = kWeights_, kTokens = kTokens_;
  int32_t* nseg;
  uint2* seg;
  float* weight;
  uint16_t* token;
  __device__ __forceinline__ SegmentTable(uint8_t* at, int slots)
      : nseg(reinterpret_cast<int32_t*>(at)), seg(reinterpret_cast<uint2*>(at + 16)), weight(reinterpret_cast<float*>(seg + slots)),
        token(kWeights ? reinterpret_cast<uint16_t*>(weight + slots) : reinterpret_cast<uint16_t*>(seg + slots)) {}
};
// with what follows on a 16-byte boundary
__host__ __device__ constexpr int table_bytes(int slots, int per_position) { return 16 + (slots * (8 + per_position) + 15) / 16 * 16; }
__device__ __forceinline__ Segment unpack_segment(uint2 v) {
  Segment s;
  s.expert = static_cast<int32_t>(v.x & 1023u);
  s.count = static_cast<int32_t>((v.x >> 10) & 31u);
  s.first = static_cast<int32_t>(v.x >> 16);
  s.offset = static_cast<int32_t>(v.y);
  return s;
}

// A slot's rank among its expert's is the number of bits below its own in the expert's mask of slots.
constexpr int kTableScratch = grouping_bytes(kMoeMaxExperts, kMoeMaxSlots) + 2 * kMoeMaxExperts + 4 * kMoeMaxSlots +
                              4 * kMoeMaxExperts * (kMoeMaxSlots / 32);

__device__ __forceinline__ uint2 table_entry(uint32_t expert, int count, int first, int offset) {
  return make_uint2(expert | (static_cast<uint32_t>(count) << 10) | (static_cast<uint32_t>(first) << 16),
                    static_cast<uint32_t>(offset));
}

// Up to 32 slots one warp sorts: a slot's position is the number of smaller (expert, slot) pairs, and the segments follow from
// ballots over the sorted experts.  Nothing depends on the number of experts.
template <class Table>
__device__ __forceinline__ void build_small_table(const MoeParams& p, const Table& table, uint32_t* slot_pos) {
  const int S = p.t * p.topk, lane = threadIdx.x & 31;
  uint32_t key = kNoPosition;                    // expert * 32 + slot; larger than all of those without an expert
  float weight = 0.0f;
  if (lane < S) {
    const int e = p.ids[lane];
    if constexpr (Table::kWeights) weight = p.weights[lane];
    if (e >= 0 && e < p.experts) key = static_cast<uint32_t>(e * 32 + lane);
  }
  const bool valid = key != kNoPosition;
  int at = 0;                                    // among the slots with an expert
#pragma unroll 4
  for (int j = 0; j < S; ++j) at += __shfl_sync(0xffffffffu, key, j) < key;
  const uint32_t same = __match_any_sync(0xffffffffu, key >> 5);
  const int r = __popc(same & ((1u << lane) - 1u)), count = min(__popc(same) - r, kSegSlots);
  const bool begins = valid && r % kSegSlots == 0;
  // bits at the positions where segments begin, and where those of 32 and 64 columns do
  const uint32_t bit = begins ? 1u << at : 0u;
  const uint32_t all = __reduce_or_sync(0xffffffffu, bit),
                 mid = __reduce_or_sync(0xffffffffu, segment_columns(count) == 32 ? bit : 0u),
                 wide = __reduce_or_sync(0xffffffffu, segment_columns(count) == 64 ? bit : 0u);
  if (valid) {
    const uint32_t below = (1u << at) - 1u;
    if (begins)
      table.seg[__popc(all & below)] =
          table_entry(key >> 5, count, at,
                      __popc(all & below) * (block_bytes(1) / kBlockUnit) +
                          __popc(mid & below) * ((block_bytes(8) - block_bytes(1)) / kBlockUnit) +
                          __popc(wide & below) * ((block_bytes(kSegSlots) - block_bytes(1)) / kBlockUnit));
    if constexpr (Table::kTokens) table.token[at] = static_cast<uint16_t>(lane / p.topk);
    if constexpr (Table::kWeights) table.weight[at] = weight;
  }
  // the segment of a slot is the last that begins at or before it
  if (slot_pos && lane < S && index_ok(lane, S, p.status))
    slot_pos[lane] = valid ? static_cast<uint32_t>(at) | (static_cast<uint32_t>(__popc(all & ((2u << at) - 1u)) - 1) << 16)
                           : kNoPosition;
  if (lane == 0) *table.nseg = __popc(all);
}

// Each kernel makes its own table, from the call's ids; slot_pos, where it is given, gets MoeParams::slot_pos.
template <class Table>
__device__ __forceinline__ void build_table(const MoeParams& p, uint8_t* scratch, const Table& table, uint32_t* slot_pos) {
  const int S = p.t * p.topk, words = (S + 31) / 32;
  const int tid = threadIdx.x, threads = blockDim.x;
  if (S <= 32) {
    if (tid < 32) build_small_table(p, table, slot_pos);
    __syncthreads();
    return;
  }
  uint32_t* const mask = reinterpret_cast<uint32_t*>(scratch);             // [experts][words]
  float* const weight = reinterpret_cast<float*>(mask + p.experts * words);
  const Grouping g(reinterpret_cast<uint8_t*>(weight + S), p.experts);
  uint16_t* const first = g.id + S;
  for (int i = tid; i < S; i += threads) {
    const int e = p.ids[i];
    if constexpr (Table::kWeights) weight[i] = p.weights[i];
    g.id[i] = static_cast<uint16_t>(e >= 0 && e < p.experts ? static_cast<uint32_t>(e) : kNoExpert);
  }
  for (int e = tid; e < p.experts; e += threads) g.count[e] = 0;
  for (int i = tid; i < p.experts * words; i += threads) mask[i] = 0;
  __syncthreads();
  for (int i = tid; i < S; i += threads) {
    const uint32_t e = g.id[i];
    if (e == kNoExpert) continue;
    atomicAdd(&g.count[e], 1u);
    atomicOr(&mask[e * words + (i >> 5)], 1u << (i & 31));
  }
  __syncthreads();
  if (tid < 32) {
    const int n = place_experts(p.experts, g, first);
    if (tid == 0) *table.nseg = n;
  }
  __syncthreads();
  for (int i = tid; i < S; i += threads) {
    const uint32_t e = g.id[i];
    uint32_t place = kNoPosition;
    if (e != kNoExpert) {
      const uint32_t* m = mask + e * words;
      int r = __popc(m[i >> 5] & ((1u << (i & 31)) - 1u));
      for (int j = 0; j < (i >> 5); ++j) r += __popc(m[j]);
      const int at = first[e] + r;
      if constexpr (Table::kTokens) table.token[at] = static_cast<uint16_t>(i / p.topk);
      if constexpr (Table::kWeights) table.weight[at] = weight[i];
      place = static_cast<uint32_t>(at) | (static_cast<uint32_t>(g.seg0[e] + r / kSegSlots) << 16);
      if (r % kSegSlots == 0) {                  // the segment's first slot writes its entry
        const int j = r / kSegSlots, count = min(static_cast<int>(g.count[e]) - r, kSegSlots);
        table.seg[g.seg0[e] + j] = table_entry(e, count, at, g.off0[e] + j * (block_bytes(kSegSlots) / kBlockUnit));
      }
    }
    if (slot_pos && index_ok(i, S, p.status)) slot_pos[i] = place;
  }
  __syncthreads();
}

// ---- the slices of x ----------------------------------------------------------------------------------

// One warp per (token, 256 values of K, part of the token's slots), eight values a lane.  The kernel after it may start
// as soon as every CTA is past the wait: it reads the call's inputs, which are complete then, and waits for this kernel before
// it reads the slices.
__global__ void __launch_bounds__(256) moe_slice_kernel(const MoeParams p, int parts) {
  extern __shared__ uint8_t smem_raw[];
  const Grouping g(smem_raw, p.experts);
  const int S = p.t * p.topk, lane = threadIdx.x & 31, ks1 = (p.k + 255) / 256, items = p.t * ks1 * parts;
  int item = blockIdx.x * 8 + (threadIdx.x >> 5);
  int token, ks, part;
  auto locate = [&]() {
    token = item / (ks1 * parts);
    ks = item / parts - token * ks1;
    part = item % parts;
  };
  auto load = [&]() {
    const int c = ks * 256 + lane * 8;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    const int64_t src = static_cast<int64_t>(token) * p.k + c;
    if (c < p.k && index_ok(src + 7, static_cast<uint64_t>(p.t) * p.k, p.status))
      raw = __ldg(reinterpret_cast<const uint4*>(p.x + src));
    return raw;
  };
  auto slices = [&](const uint4& raw) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[2 * q] = bf16_lo(w[q]), x[2 * q + 1] = bf16_hi(w[q]);
    return slice8<32>(x);
  };
  locate();
  for (int e = threadIdx.x; e < p.experts; e += 256) g.count[e] = 0;
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  Slices s;
  // The first pass, on zeros, brings the code into the instruction cache while the kernel before this one ends (7 tokens, 5 experts
  // 192 x 320: 14.7 against 15.0 us; behind a kernel that lets this one start only at its end it costs 0.6 us).
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass) {
      pdl_wait();
      pdl_launch_dependents();
      if (item < items) raw = load();
      for (int i = threadIdx.x; i < S; i += 256) {
        const int e = p.ids[i];
        const bool valid = e >= 0 && e < p.experts;
        g.id[i] = static_cast<uint16_t>(valid ? static_cast<uint32_t>(e) : kNoExpert);
        if (valid) atomicAdd(&g.count[e], 1u);
      }
    }
    __syncthreads();
    // one warp places the experts while the others are at their first slices
    if (threadIdx.x < 32) place_experts(p.experts, g, nullptr);
    s = slices(raw);
    __syncthreads();
  }
  while (item < items) {
    for (int i = token * p.topk + part; i < (token + 1) * p.topk; i += parts) {
      const uint32_t e = g.id[i];
      if (e == kNoExpert) continue;
      int r = 0;                                 // the slot's rank among its expert's
#pragma unroll 4
      for (int q = 0; q < i; q += 32) r += __popc(__ballot_sync(0xffffffffu, q + lane < i && g.id[q + lane] == e));
      const int j = r / kSegSlots, slot = r % kSegSlots;
      const int bytes = block_bytes(min(static_cast<int>(g.count[e]) - j * kSegSlots, kSegSlots));
      const int64_t at = static_cast<int64_t>(g.off0[e] + j * (block_bytes(kSegSlots) / kBlockUnit)) * kBlockUnit * ks1 +
                         static_cast<int64_t>(ks) * bytes;
      if (index_ok(at + bytes - 1, static_cast<uint64_t>(p.b_units) * ks1, p.status)) put_slices(p.b_x + at, (bytes - kSfBlockBytes) / 128, slot, lane, s);
      const int f = ((g.seg0[e] + j) * ks1 + ks) * kSegSlots + slot;
      if (lane == 0 && index_ok(f, static_cast<uint64_t>(p.max_segments) * ks1 * kSegSlots, p.status)) p.f_x[f] = s.factor;
    }
    item += gridDim.x * 8;
    if (item < items) {
      locate();
      s = slices(load());
    }
  }
}

// ---- reading an accumulator --------------------------------------------------------------------------

__device__ __forceinline__ uint64_t pack_bits(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// acc[s] += f[s] * (sum of the four slices' columns of slot s) for kQ slots, two slots an instruction.
template <int kQ>
__device__ __forceinline__ void add_slots(uint32_t taddr, const float* f, uint64_t* acc) {
  uint32_t v[4 * kQ];
  if constexpr (kQ == 4) tmem_load_16(taddr, v);
  if constexpr (kQ == 8) tmem_load_32(taddr, v);
  if constexpr (kQ == 16) tmem_load_64(taddr, v);
  tmem_wait_ld<4 * kQ>(v);
#pragma unroll
  for (int s = 0; s < kQ; s += 2) {
    const uint64_t sum = add2(add2(pack_bits(v[s], v[s + 1]), pack_bits(v[kQ + s], v[kQ + s + 1])),
                              add2(pack_bits(v[2 * kQ + s], v[2 * kQ + s + 1]), pack_bits(v[3 * kQ + s], v[3 * kQ + s + 1])));
    acc[s / 2] = fma2(*reinterpret_cast<const uint64_t*>(f + s), sum, acc[s / 2]);
  }
}
__device__ __forceinline__ void add_slots(int count, uint32_t taddr, const float* f, uint64_t* acc) {
  if (count <= 4) add_slots<4>(taddr, f, acc);
  else if (count <= 8) add_slots<8>(taddr, f, acc);
  else add_slots<16>(taddr, f, acc);
}
__device__ __forceinline__ float acc_slot(const uint64_t* acc, int s) {
  float lo, hi;
  unpack2(acc[s / 2], lo, hi);
  return s & 1 ? hi : lo;
}

// ---- the down kernel's units ---------------------------------------------------------------------------

// Units (128-row tile, segment, K stage), in that order, cut into equal ranges, one per CTA; fewer than 2^31 of them.
struct DownSplit {
  int units, upt, ctas, q, r;                    // units per tile; the first r CTAs take q + 1 units, the others q
  __device__ __forceinline__ DownSplit(int tiles, int upt_, int max_ctas) : units(tiles * upt_), upt(upt_) {
    ctas = min(units, max_ctas);
    q = ctas ? units / ctas : 0;
    r = ctas ? units - q * ctas : 0;
  }
  __device__ __forceinline__ int start(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int cta_of(int u) const { return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q; }
};
struct DownWalk {
  int u, end, tile, in, sg, ks;
  int stages, upt;
  __device__ __forceinline__ DownWalk(const DownSplit& s, int stages_) : stages(stages_), upt(s.upt) {
    const int c = blockIdx.x;
    u = c < s.ctas ? s.start(c) : 0;
    end = c < s.ctas ? s.start(c + 1) : 0;
    tile = upt ? u / upt : 0;
    in = u - tile * upt;
    sg = in / stages;
    ks = in - sg * stages;
  }
  __device__ __forceinline__ bool valid() const { return u < end; }
  __device__ __forceinline__ bool tile_end() const { return u + 1 == end || in + 1 == upt; }
  __device__ __forceinline__ void next() {
    ++u;
    if (++ks == stages) {
      ks = 0;
      ++sg;
    }
    if (++in == upt) {
      in = sg = ks = 0;
      ++tile;
    }
  }
};

// ---- gate and up ------------------------------------------------------------------------------------

struct MoeMaps {
  CUtensorMap gate, up, down;
};

constexpr uint32_t kMoeTmemCols = 512;
// Accumulator buffers of 2 x 64 columns, then the scales.  A unit's way from the first MMA through the commit, the epilogue's reads and
// back to the MMA issuer takes about 1.2 us whatever its width, so with two buffers a unit took 0.6 us or more.
constexpr uint32_t kAccBuffers = 3;
constexpr uint32_t kMoeSfCol = 128 * kAccBuffers;
static_assert(kMoeSfCol + 48 <= kMoeTmemCols, "tensor memory");

// Warps: 0 weight loads, 1 MMA issuer, 2-5 epilogue, 6-10 finishers, 11 activation loads; with kConvert 6-8 finishers, 9-11 converters.
constexpr int kUpThreads = 384;
constexpr int kUpStages = 4;
constexpr int kUpConverters = 3;
constexpr int kUpFinishers = 5;                  // two slots at a time each.  4: 1 us slower with 64 tokens; 8: fewer registers, 0.7 us slower
__host__ __device__ constexpr int up_finishers(bool convert) { return convert ? kUpFinishers + 1 - kUpConverters : kUpFinishers; }
static_assert(64 + 128 + 32 * kUpFinishers + 32 == kUpThreads, "warp roles");
constexpr int kUpBAt = 2 * kTileBytes;                         // x's block: scales, then rows
constexpr int kUpSfaAt = kUpBAt + kSfBlockBytes + kRowsBytes;
constexpr int kUpStageBytes = kUpSfaAt + 2 * kSfBlockBytes;    // 46 KB
constexpr int kUpSumBytes = 2 * kSegSlots * 128 * 4;           // the tile's gate and up sums [2][16][128] fp32
// The factors F of a stage go to a ring of their own, because the epilogue reads them after the MMAs have given the
// stage's slot back: the load (or conversion) of unit i + 8 waits for the MMAs of unit i + 8 - stages (i + 3 or later), and those for the
// epilogue's release of the accumulator that unit i or a later one used.
constexpr int kFactorRing = 8;

struct __align__(8) UpControl {
  uint64_t full[kUpStages], empty[kUpStages];
  uint64_t acc_full[kAccBuffers], acc_empty[kAccBuffers];
  uint64_t sums_full, sums_empty;
  uint32_t tmem_base;
  int32_t abort;
};

__host__ __device__ constexpr int up_smem(int slots) {
  return kUpStages * kUpStageBytes + kUpSumBytes + kFactorRing * kSegSlots * 4 + table_bytes(slots, 6) +
         static_cast<int>(sizeof(UpControl)) + 1024;
}
static_assert(kUpStageBytes % 1024 == 0 && up_smem(kMoeMaxSlots) <= 227 * 1024, "shared memory layout");
static_assert(kTableScratch <= kUpStages * kUpStageBytes, "the grouping's scratch lies in the ring");

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Arrives on the barrier at the same place of every CTA of the cluster (the lane of that rank does).  A cluster of one stays with
// the CTA's scope: an arrival that releases to the cluster waits 1 to 5 us for the SM's memory traffic when that is heavy.
__device__ __forceinline__ void arrive_cluster_wide(uint64_t* bar, int lane, int ctas) {
  if (ctas == 1) {
    if (lane == 0) mbar_arrive(bar);
  } else if (lane < ctas) {
    mbar_arrive_cluster(map_to_rank(bar, static_cast<uint32_t>(lane)));
  }
  __syncwarp();
}

// A cluster's tiles (its own, then every clusters-th) and this CTA's K stages of each.
struct UpWalk {
  int tile, sg, rt, ks;
  int tiles, step, row_tiles, k0, k1;
  __device__ __forceinline__ UpWalk(int nseg, int row_tiles_, int stages, int rank, int ctas)
      : tiles(nseg * row_tiles_), row_tiles(row_tiles_) {
    step = static_cast<int>(gridDim.x) / ctas;
    tile = static_cast<int>(blockIdx.x) / ctas;
    k0 = rank * stages / ctas;
    k1 = (rank + 1) * stages / ctas;
    ks = k0;
    locate();
  }
  __device__ __forceinline__ void locate() {
    sg = tile / row_tiles;
    rt = tile - sg * row_tiles;
  }
  __device__ __forceinline__ bool valid() const { return tile < tiles; }
  __device__ __forceinline__ bool last() const { return ks + 1 == k1; }
  __device__ __forceinline__ void next() {
    if (++ks == k1) {
      ks = k0;
      tile += step;
      locate();
    }
  }
};

// Eight values of a lane as slices of slot s of a stage's block; the chunk's factor.  Not inlined, so that a first call on zeros brings the
// code into the instruction cache.
__device__ __noinline__ float convert_slot(uint4 raw, uint8_t* block, int columns, int s) {
  const int lane = threadIdx.x & 31;
  const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) x[2 * q] = bf16_lo(v[q]), x[2 * q + 1] = bf16_hi(v[q]);
  const Slices sl = slice8<32>(x);
  put_slices(block, columns, s, lane, sl);
  return sl.factor;
}

template <bool kConvert>
__global__ void __launch_bounds__(kUpThreads, 1) moe_up_kernel(const __grid_constant__ MoeMaps maps, const MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sums = reinterpret_cast<float*>(smem + kUpStages * kUpStageBytes);
  float* factors = sums + kUpSumBytes / 4;
  uint8_t* const table_at = reinterpret_cast<uint8_t*>(factors + kFactorRing * kSegSlots);
  const SegmentTable<true, kConvert> table(table_at, p.t * p.topk);
  UpControl& ctl = *reinterpret_cast<UpControl*>(table_at + table_bytes(p.t * p.topk, 6));
  volatile int32_t* abort = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_ctas());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kUpStages; ++s) {
      mbar_init(&ctl.full[s], 2);                // both load warps; a converter
      mbar_init(&ctl.empty[s], 1);
    }
    for (uint32_t b = 0; b < kAccBuffers; ++b) {
      mbar_init(&ctl.acc_full[b], 1);
      mbar_init(&ctl.acc_empty[b], 4);
    }
    mbar_init(&ctl.sums_full, 4 * ctas);         // the epilogue (finisher) warps of every CTA of the cluster
    mbar_init(&ctl.sums_empty, up_finishers(kConvert) * ctas);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem_base)),
                 "r"(kMoeTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && elect_one()) {
    prefetch_map(&maps.gate);
    prefetch_map(&maps.up);
  }
  __syncwarp();
  if (ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // peers signal this CTA's barriers
  if constexpr (kConvert) {
    if (warp >= 6 + up_finishers(true)) convert_slot(make_uint4(0u, 0u, 0u, 0u), reinterpret_cast<uint8_t*>(sums), 16, warp & 3);
    pdl_wait();                                  // the call's first kernel
  }
  pdl_launch_dependents();
  // of the call's inputs alone: see moe_slice_kernel
  build_table(p, smem, table, blockIdx.x == 0 && p.t > kMoeLastCtaTokens ? p.slot_pos : nullptr);
  fence_async_smem();                            // the ring's loads overwrite the grouping's scratch
  tc_fence_before();
  __syncthreads();
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;

  const int nseg = *table.nseg;
  const int stages = (p.k + 255) / 256, groups = p.k / 64;
  const int row_tiles = (p.n + 127) / 128;
  UpWalk w(nseg, row_tiles, stages, rank, ctas);
  if (blockIdx.x == 0) {
    // what the kernels after it read
    if (p.t > kMoeLastCtaTokens) {
      if (threadIdx.x == 0) *p.nseg = nseg;
      for (int i = threadIdx.x; i < nseg; i += kUpThreads)
        if (index_ok(i, p.max_segments, p.status)) p.segments[i] = unpack_segment(table.seg[i]);
    }
    for (int i = threadIdx.x; i < (p.k + 127) / 128; i += kUpThreads) p.count[i] = 0;
  }

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer: weights and their scales
    uint32_t slot = 0, phase = 0;
    bool wrapped = false;
    for (; w.valid(); w.next()) {
      const int expert = static_cast<int>(table.seg[w.sg].x & 1023u);
      if (wrapped && !mbar_wait_fast(&ctl.empty[slot], phase, abort, p.status)) break;
      if (elect_one()) {
        uint8_t* st = smem + slot * kUpStageBytes;
        uint64_t* full = &ctl.full[slot];
        const uint32_t sf_bytes = static_cast<uint32_t>(min(4, groups - 4 * w.ks)) * 512u;
        const int64_t sf_at = expert * p.up_stride + (static_cast<int64_t>(w.rt) * groups + 4 * w.ks) * 512;
        mbar_arrive_expect_tx(full, 2 * (kTileBytes + sf_bytes));
        tma_load_3d_cta(st, &maps.gate, full, w.ks * 128, w.rt * 128, expert);
        tma_load_3d_cta(st + kTileBytes, &maps.up, full, w.ks * 128, w.rt * 128, expert);
        bulk_load_cta(st + kUpSfaAt, p.gate_sf + sf_at, sf_bytes, full);
        bulk_load_cta(st + kUpSfaAt + kSfBlockBytes, p.up_sf + sf_at, sf_bytes, full);
      }
      __syncwarp();
      if (++slot == kUpStages) {
        slot = 0;
        if (wrapped) phase ^= 1u;
        wrapped = true;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t smem0 = smem_u32(smem);
    uint32_t slot = 0, phase = 0, i = 0;
    for (; w.valid(); w.next(), ++i) {
      const uint32_t idesc = idesc_fp4_cta(static_cast<uint32_t>(segment_columns(static_cast<int>((table.seg[w.sg].x >> 10) & 31u))));
      const uint32_t b = i % kAccBuffers;
      if (i >= kAccBuffers && !mbar_wait_fast(&ctl.acc_empty[b], (i / kAccBuffers - 1u) & 1u, abort, p.status)) break;
      if (!mbar_wait_fast(&ctl.full[slot], phase, abort, p.status)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t st = smem0 + slot * kUpStageBytes;
        const uint64_t a0 = operand_desc(st), a1 = operand_desc(st + kTileBytes);
        const uint64_t b0 = operand_desc(st + kUpBAt + kSfBlockBytes);
        const uint64_t sfa = sf_chunk_desc(st + kUpSfaAt), sfb = sf_chunk_desc(st + kUpBAt);
        const uint32_t acc = tmem + b * 128u;
        const int steps = min(4, groups - 4 * w.ks);
        auto step = [&](int j) {
          const uint32_t col = tmem + kMoeSfCol + 12u * j;
          tc_copy_sf_cta(col, sfa + 32 * j);
          tc_copy_sf_cta(col + 4, sfa + (kSfBlockBytes >> 4) + 32 * j);
          tc_copy_sf_cta(col + 8, sfb + 32 * j);
          mma_fp4_cta(acc, a0 + 2 * j, b0 + 2 * j, idesc, col, col + 8, j > 0);
          mma_fp4_cta(acc + 64u, a1 + 2 * j, b0 + 2 * j, idesc, col + 4, col + 8, j > 0);
        };
        if (steps == 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) step(j);
        } else {
#pragma unroll 1
          for (int j = 0; j < steps; ++j) step(j);
        }
        mma_commit_cta(&ctl.empty[slot]);
        mma_commit_cta(&ctl.acc_full[b]);
      }
      __syncwarp();
      if (++slot == kUpStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------------ epilogue
    // One warp per TMEM lane quarter; a thread owns one row of gate and of up and adds, per slot, its four slices times the chunk's factor
    // into fp32 registers.  At the tile's end the sums go to shared memory for the converters of the cluster.
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint64_t acc[2][kSegSlots / 2];
#pragma unroll
    for (int j = 0; j < kSegSlots / 2; ++j) acc[0][j] = acc[1][j] = 0;
    uint32_t i = 0, tiles_done = 0;
    // The first pass runs on whatever lies in tensor memory and is thrown away: it brings the code into the instruction cache
    // while the first loads are under way.
    bool dry = true;
    while (w.valid()) {
      const int count = static_cast<int>((table.seg[w.sg].x >> 10) & 31u);
      const float* f = factors + (i % kFactorRing) * kSegSlots;
      const uint32_t b = i % kAccBuffers;
      if (!dry && !mbar_wait_fast(&ctl.acc_full[b], (i / kAccBuffers) & 1u, abort, p.status)) break;
      tc_fence_after();
      add_slots(count, tmem + b * 128u + lane_base, f, acc[0]);
      add_slots(count, tmem + b * 128u + 64u + lane_base, f, acc[1]);
      if (dry) {
        dry = false;
#pragma unroll
        for (int j = 0; j < kSegSlots / 2; ++j) acc[0][j] = acc[1][j] = 0;
        continue;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.acc_empty[b]);
      if (w.last()) {
        if (tiles_done > 0 && !mbar_wait_fast(&ctl.sums_empty, (tiles_done - 1) & 1u, abort, p.status)) break;
#pragma unroll
        for (int s = 0; s < kSegSlots; ++s) {
          if (s < count) {
            sums[s * 128 + row] = acc_slot(acc[0], s);
            sums[(kSegSlots + s) * 128 + row] = acc_slot(acc[1], s);
          }
        }
#pragma unroll
        for (int j = 0; j < kSegSlots / 2; ++j) acc[0][j] = acc[1][j] = 0;
        __syncwarp();
        arrive_cluster_wide(&ctl.sums_full, lane, ctas);
        ++tiles_done;
      }
      w.next();
      ++i;
    }
  } else if (kConvert && warp >= 6 + up_finishers(kConvert)) {
    // ------------------------------------------------------------------ converters
    // The slices of a stage's slots, eight values a lane; the warps take stages in turn, and ask for the next slot's values first.
    auto load = [&](const UpWalk& at, int s) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (!at.valid()) return raw;
      const Segment seg = unpack_segment(table.seg[at.sg]);
      const int c = at.ks * 256 + lane * 8;
      if (c >= p.k) return raw;
      const int64_t src = static_cast<int64_t>(table.token[seg.first + s]) * p.k + c;
      if (index_ok(src + 7, static_cast<uint64_t>(p.t) * p.k, p.status)) raw = __ldg(reinterpret_cast<const uint4*>(p.x + src));
      return raw;
    };
    auto advance = [&](UpWalk& at, int n) {
      for (int q = 0; q < n && at.valid(); ++q) at.next();
    };
    uint32_t i = static_cast<uint32_t>(warp - 6 - up_finishers(kConvert));
    advance(w, static_cast<int>(i));
    uint4 raw = load(w, 0);
    while (w.valid()) {
      const int count = static_cast<int>((table.seg[w.sg].x >> 10) & 31u);
      UpWalk after = w;
      advance(after, kUpConverters);
      const uint32_t slot = i % kUpStages;
      if (i >= kUpStages && !mbar_wait_fast(&ctl.empty[slot], (i / kUpStages - 1u) & 1u, abort, p.status)) break;
      uint8_t* block = smem + slot * kUpStageBytes + kUpBAt;
      for (int s = 0; s < count; ++s) {
        const uint4 next = s + 1 < count ? load(w, s + 1) : load(after, 0);
        const float f = convert_slot(raw, block, segment_columns(count), s);
        if (lane == 0) factors[(i % kFactorRing) * kSegSlots + s] = f;
        raw = next;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.full[slot]);
      w = after;
      i += kUpConverters;
    }
  } else if (!kConvert && warp == 6 + up_finishers(kConvert)) {
    // ------------------------------------------------------------------ TMA producer: slices of x and their factors
    pdl_wait();
    uint32_t slot = 0, phase = 0, i = 0;
    bool wrapped = false;
    for (; w.valid(); w.next(), ++i) {
      const Segment seg = unpack_segment(table.seg[w.sg]);
      if (wrapped && !mbar_wait_fast(&ctl.empty[slot], phase, abort, p.status)) break;
      if (elect_one()) {
        uint64_t* full = &ctl.full[slot];
        const uint32_t bytes = static_cast<uint32_t>(block_bytes(seg.count));
        mbar_arrive_expect_tx(full, bytes + kSegSlots * 4);
        bulk_load_cta(smem + slot * kUpStageBytes + kUpBAt,
                      p.b_x + static_cast<int64_t>(seg.offset) * kBlockUnit * stages + static_cast<int64_t>(w.ks) * bytes, bytes, full);
        bulk_load_cta(factors + (i % kFactorRing) * kSegSlots, p.f_x + (static_cast<int64_t>(w.sg) * stages + w.ks) * kSegSlots,
                      kSegSlots * 4, full);
      }
      __syncwarp();
      if (++slot == kUpStages) {
        slot = 0;
        if (wrapped) phase ^= 1u;
        wrapped = true;
      }
    }
  } else {
    // ------------------------------------------------------------------ finishers
    // h of each tile: sixteen lanes a slot, eight rows a lane; the cluster's CTAs take every ctas-th slot.
    const int fw = warp - 6, l16 = lane & 15;
    const int hs = (p.n + 255) / 256;            // K stages of the down projection
    uint32_t n = 0;
    bool dry = true;                             // as in the epilogue
    while (w.valid()) {
      const Segment seg = unpack_segment(table.seg[w.sg]);
      const float sg = p.gate_amax[seg.expert] * (1.0f / 2688.0f), su = p.up_amax[seg.expert] * (1.0f / 2688.0f);
      const float sd = p.down_amax[seg.expert] * (1.0f / 2688.0f);
      if (!dry && !mbar_wait_fast(&ctl.sums_full, n & 1u, abort, p.status)) break;
#pragma unroll 1
      for (int s0 = rank + ctas * 2 * fw; dry || s0 < seg.count; s0 += ctas * 2 * up_finishers(kConvert)) {
        const int s = s0 + ctas * (lane >> 4);
        // Rows of the tile beyond n count as zero before the chunk's largest magnitude is taken: their codes are loaded as zeros, but
        // their scales are the caller's padding, where a NaN may stand.
        const bool valid = !dry && s < seg.count && w.rt * 128 + l16 * 8 < p.n;
        float g[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.0f;
        if (valid) {
          const uint32_t off = static_cast<uint32_t>((s * 128 + l16 * 8) * 4);
#pragma unroll 1
          for (int q = 0; q < ctas; ++q) {
            const uint32_t at = map_to_rank(sums, static_cast<uint32_t>(q)) + off;
            const float4 g0 = ld_cluster_v4(at), g1 = ld_cluster_v4(at + 16);
            const float4 u0 = ld_cluster_v4(at + kSegSlots * 512), u1 = ld_cluster_v4(at + kSegSlots * 512 + 16);
            g[0] += g0.x, g[1] += g0.y, g[2] += g0.z, g[3] += g0.w, g[4] += g1.x, g[5] += g1.y, g[6] += g1.z, g[7] += g1.w;
            u[0] += u0.x, u[1] += u0.y, u[2] += u0.z, u[3] += u0.w, u[4] += u1.x, u[5] += u1.y, u[6] += u1.z, u[7] += u1.w;
          }
        }
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gate = g[e] * sg;
          h[e] = gate / (1.0f + expf(-gate)) * (u[e] * su);
        }
        const Slices sl = slice8<16>(h);
        if (valid) {
          const int bytes = block_bytes(seg.count);
          const int64_t at = static_cast<int64_t>(seg.offset) * kBlockUnit * hs + static_cast<int64_t>(w.rt >> 1) * bytes;
          if (index_ok(at + bytes - 1, static_cast<uint64_t>(p.b_units) * hs, p.status))
            put_slices(p.b_h + at, segment_columns(seg.count), s, (w.rt & 1) * 16 + l16, sl);
          const int fo = (w.sg * 2 * hs + w.rt) * kSegSlots + s;
          if (l16 == 0 && index_ok(fo, static_cast<uint64_t>(p.max_segments) * 2 * hs * kSegSlots, p.status))
            p.f_h[fo] = sl.factor * (table.weight[seg.first + s] * sd);
        }
        if (dry) break;
      }
      __syncwarp();
      if (!dry) arrive_cluster_wide(&ctl.sums_empty, lane, ctas);
      if (dry) {
        dry = false;
        continue;
      }
      w.tile += w.step;
      w.locate();
      ++n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort) {
    const uint64_t t0 = global_ns();             // bounded time for copies and MMAs in flight to drain
    while (global_ns() - t0 < 2000000ull) {
    }
  }
  if (ctas > 1) cluster_sync();                  // no CTA leaves while a peer may read its sums or signal it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kMoeTmemCols) : "memory");
  }
}

// ---- down -------------------------------------------------------------------------------------------

// Warps: 0 weight loads, 1 MMA issuer, 2-5 epilogue, 6 activation loads.
constexpr int kDownThreads = 64 + 128 + 32;
constexpr int kDownMaxStages = 7;
constexpr int kDownBAt = kTileBytes;                           // h's block: scales, then rows
constexpr int kDownSfaAt = kDownBAt + kSfBlockBytes + kRowsBytes;
constexpr int kDownStageBytes = kDownSfaAt + kSfBlockBytes;    // 28 KB
constexpr int kDownFactorBytes = 2 * kSegSlots * 4;
// Here a factor ring of 8 would be overwritten early: with 7 stages the load of unit i + 8 waits for the MMAs of unit i + 1 only.
constexpr int kDownFactorRing = 16;

struct __align__(8) DownControl {
  uint64_t full[kDownMaxStages], empty[kDownMaxStages];
  uint64_t acc_full[kAccBuffers], acc_empty[kAccBuffers];
  uint32_t tmem_base;
  int32_t abort;
  int32_t last;
};
static_assert(kDownStageBytes % 1024 == 0, "operand tiles are 1 KB aligned");
// A stage's 16 KB of weights are held for about 2 us: 6 of them (96 KB per SM) just cover HBM's latency at full rate.
__host__ __device__ constexpr int down_sum_rows(int t) { return t <= kMoeLastCtaTokens ? t + 1 : 0; }
__host__ __device__ constexpr int down_rest_bytes(int t, int slots) {
  return down_sum_rows(t) * 512 + kDownFactorRing * kDownFactorBytes +
         table_bytes(slots, t <= kMoeLastCtaTokens ? 2 : 0) + static_cast<int>(sizeof(DownControl)) + 1024;
}
__host__ __device__ constexpr int down_ring_stages(int t, int slots) {
  return (227 * 1024 - down_rest_bytes(t, slots)) / kDownStageBytes < kDownMaxStages
             ? (227 * 1024 - down_rest_bytes(t, slots)) / kDownStageBytes
             : kDownMaxStages;
}
__host__ __device__ constexpr int down_smem(int t, int slots) {
  return down_ring_stages(t, slots) * kDownStageBytes + down_rest_bytes(t, slots);
}
static_assert(down_ring_stages(kMoeLastCtaTokens, kMoeLastCtaTokens * kMoeMaxTopk) == kDownMaxStages &&
                  down_ring_stages(kMoeMaxTokens, kMoeMaxSlots) == kDownMaxStages &&
                  down_smem(kMoeMaxTokens, kMoeMaxSlots) <= 227 * 1024,
              "shared memory layout");
static_assert(kTableScratch <= kDownMaxStages * kDownStageBytes, "the grouping's scratch lies in the ring");

// The CTAs that share a tile.  CTA c leaves its partial sums at place 2c for the first tile of its range and 2c + 1 for its last:
// every CTA after c0 begins inside the tile, c0 may have begun before it.
struct TileShare {
  int c0, c1, first_place;
  __device__ __forceinline__ TileShare(const DownSplit& s, int tile) {
    const int u0 = tile * s.upt;
    c0 = s.cta_of(u0);
    c1 = s.cta_of(u0 + s.upt - 1);
    first_place = 2 * c0 + (s.start(c0) < u0 ? 1 : 0);
  }
  __device__ __forceinline__ int place(int c) const { return c == c0 ? first_place : 2 * c; }
};

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// kCombine: a thread writes every slot's result (or what it adds to one that another CTA began) for moe_combine_kernel, which leaves
// no shared sums to wait for (64 tokens, 64 experts 1408 x 2048: the layer 77.3 against 78.4 us).  Otherwise the CTA adds up its tokens in shared
// memory, and the last CTA of a tile finishes it: one launch less, which is what counts with few tokens.
template <bool kCombine>
__global__ void __launch_bounds__(kDownThreads, 1) moe_down_kernel(const __grid_constant__ MoeMaps maps, const MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sums = reinterpret_cast<float*>(smem + kDownMaxStages * kDownStageBytes);
  float* factors = sums + down_sum_rows(p.t) * 128;
  uint8_t* const table_at = reinterpret_cast<uint8_t*>(factors + kDownFactorRing * kDownFactorBytes / 4);
  const SegmentTable<false, !kCombine> table(table_at, p.t * p.topk);
  DownControl& ctl = *reinterpret_cast<DownControl*>(table_at + table_bytes(p.t * p.topk, kCombine ? 0 : 2));
  volatile int32_t* abort = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kDownMaxStages; ++s) {
      mbar_init(&ctl.full[s], 2);                // both load warps
      mbar_init(&ctl.empty[s], 1);
    }
    for (uint32_t b = 0; b < kAccBuffers; ++b) {
      mbar_init(&ctl.acc_full[b], 1);
      mbar_init(&ctl.acc_empty[b], 4);
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
  if (warp == 0 && elect_one()) prefetch_map(&maps.down);
  __syncwarp();
  // A CTA starts when one of moe_up_kernel's leaves its SM.  It groups the slots itself (of the call's inputs, as that kernel did)
  // and has its first weights on their way while the other CTAs of that kernel finish.
  build_table(p, smem, table, nullptr);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  if (warp != 0 || !p.down_early) pdl_wait();
  if (warp == 1) pdl_launch_dependents();        // after the wait: moe_combine_kernel reads moe_up_kernel's results as it starts

  const int nseg = *table.nseg;
  const int stages = (p.n + 255) / 256, groups = p.n / 64;
  const DownSplit split((p.k + 127) / 128, nseg * stages, gridDim.x);
  DownWalk w(split, stages);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer: weights and their scales
    uint32_t slot = 0, phase = 0;
    bool wrapped = false;
    for (; w.valid(); w.next()) {
      const int expert = static_cast<int>(table.seg[w.sg].x & 1023u);
      if (wrapped && !mbar_wait_fast(&ctl.empty[slot], phase, abort, p.status)) break;
      if (elect_one()) {
        uint8_t* st = smem + slot * kDownStageBytes;
        uint64_t* full = &ctl.full[slot];
        const uint32_t sf_bytes = static_cast<uint32_t>(min(4, groups - 4 * w.ks)) * 512u;
        mbar_arrive_expect_tx(full, kTileBytes + sf_bytes);
        tma_load_3d_cta(st, &maps.down, full, w.ks * 128, w.tile * 128, expert);
        bulk_load_cta(st + kDownSfaAt, p.down_sf + expert * p.down_stride + (static_cast<int64_t>(w.tile) * groups + 4 * w.ks) * 512,
                      sf_bytes, full);
      }
      __syncwarp();
      if (++slot == kDownMaxStages) {
        if (!wrapped) pdl_wait();                // from here on a slot is free when h has been used
        slot = 0;
        if (wrapped) phase ^= 1u;
        wrapped = true;
      }
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------------ TMA producer: slices of h and their factors
    uint32_t slot = 0, phase = 0, i = 0;
    bool wrapped = false;
    for (; w.valid(); w.next(), ++i) {
      const Segment seg = unpack_segment(table.seg[w.sg]);
      if (wrapped && !mbar_wait_fast(&ctl.empty[slot], phase, abort, p.status)) break;
      if (elect_one()) {
        uint64_t* full = &ctl.full[slot];
        const uint32_t bytes = static_cast<uint32_t>(block_bytes(seg.count));
        mbar_arrive_expect_tx(full, bytes + kDownFactorBytes);
        bulk_load_cta(smem + slot * kDownStageBytes + kDownBAt,
                      p.b_h + static_cast<int64_t>(seg.offset) * kBlockUnit * stages + static_cast<int64_t>(w.ks) * bytes, bytes, full);
        bulk_load_cta(factors + (i % kDownFactorRing) * (kDownFactorBytes / 4),
                      p.f_h + (static_cast<int64_t>(w.sg) * stages + w.ks) * (kDownFactorBytes / 4), kDownFactorBytes, full);
      }
      __syncwarp();
      if (++slot == kDownMaxStages) {
        slot = 0;
        if (wrapped) phase ^= 1u;
        wrapped = true;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t smem0 = smem_u32(smem);
    uint32_t slot = 0, phase = 0, i = 0;
    for (; w.valid(); w.next(), ++i) {
      const uint32_t idesc = idesc_fp4_cta(static_cast<uint32_t>(segment_columns(static_cast<int>((table.seg[w.sg].x >> 10) & 31u))));
      const uint32_t b = i % kAccBuffers;
      if (i >= kAccBuffers && !mbar_wait_fast(&ctl.acc_empty[b], (i / kAccBuffers - 1u) & 1u, abort, p.status)) break;
      if (!mbar_wait_fast(&ctl.full[slot], phase, abort, p.status)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t st = smem0 + slot * kDownStageBytes;
        const uint64_t a0 = operand_desc(st), b0 = operand_desc(st + kDownBAt + kSfBlockBytes);
        const uint64_t sfa = sf_chunk_desc(st + kDownSfaAt), sfb = sf_chunk_desc(st + kDownBAt);
        const uint32_t acc = tmem + b * 128u;
        const int steps = min(4, groups - 4 * w.ks);
        auto step = [&](int j) {
          const uint32_t col = tmem + kMoeSfCol + 8u * j;
          tc_copy_sf_cta(col, sfa + 32 * j);
          tc_copy_sf_cta(col + 4, sfb + 32 * j);
          // K values [0, 128) of the stage into one accumulator, [128, 256) into the other: h has a factor for each
          mma_fp4_cta(acc + (j >> 1) * 64u, a0 + 2 * j, b0 + 2 * j, idesc, col, col + 4, j & 1);
        };
        if (steps == 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) step(j);
        } else {
#pragma unroll 1
          for (int j = 0; j < steps; ++j) step(j);
        }
        mma_commit_cta(&ctl.empty[slot]);
        mma_commit_cta(&ctl.acc_full[b]);
      }
      __syncwarp();
      if (++slot == kDownMaxStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    // One warp per TMEM lane quarter; a thread owns one output row and adds, per slot, the slices of the stage's K values [0, 128) and
    // [128, 256), each times its chunk's factor, into fp32 registers, and at a segment's end those to the tokens'
    // sums.  Once a wait has given up the loops run on without waiting, so that every barrier below still meets all
    // four warps.
    const int row = (warp & 3) * 32 + lane;
    const int tid = threadIdx.x - 64;
    const int width = p.t * 128;                 // fp32 sums
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* my_sums = sums + row;
    bool ok = true;
    uint64_t acc[kSegSlots / 2];
#pragma unroll
    for (int j = 0; j < kSegSlots / 2; ++j) acc[j] = 0;
    if (!kCombine && nseg == 0) {
      // no token has an expert: the output is zero
      for (int64_t j = static_cast<int64_t>(blockIdx.x) * 128 + tid; j < static_cast<int64_t>(p.t) * p.k / 8;
           j += static_cast<int64_t>(gridDim.x) * 128)
        reinterpret_cast<uint4*>(p.out)[j] = make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (!kCombine)
      for (int j = 0; j < p.t; ++j) my_sums[j * 128] = 0.0f;
    bool began = w.ks == 0;                      // this CTA has the segment's first K stage
    uint32_t i = 0;
    bool dry = true;                             // the first pass only warms the instruction cache, as in moe_up_kernel
    while (w.valid()) {
      const Segment seg = unpack_segment(table.seg[w.sg]);
      const int count = seg.count;
      const float* f = factors + (i % kDownFactorRing) * (kDownFactorBytes / 4);
      const uint32_t b = i % kAccBuffers;
      if (ok && !dry) ok = mbar_wait_fast(&ctl.acc_full[b], (i / kAccBuffers) & 1u, abort, p.status);
      tc_fence_after();
      add_slots(count, tmem + b * 128u + lane_base, f, acc);
      if (groups - 4 * w.ks > 2)                 // the stage has K values beyond 128
        add_slots(count, tmem + b * 128u + 64u + lane_base, f + kSegSlots, acc);
      if (dry) {
        dry = false;
#pragma unroll
        for (int j = 0; j < kSegSlots / 2; ++j) acc[j] = 0;
        continue;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.acc_empty[b]);

      const bool tile_end = w.tile_end();
      if (kCombine && (w.ks + 1 == stages || tile_end)) {
        const int col = w.tile * 128 + row;
        float* dst = began ? p.part + static_cast<int64_t>(seg.first) * p.k + col
                           : p.rest + (static_cast<int64_t>(blockIdx.x) * kSegSlots) * 128 + row;
        const int64_t step = began ? p.k : 128;
#pragma unroll
        for (int s0 = 0; s0 < kSegSlots; s0 += 4) {
          if (s0 >= count) break;
#pragma unroll
          for (int s = s0; s < s0 + 4; ++s, dst += step) {
            const bool inside = index_ok(static_cast<uint64_t>(dst - (began ? p.part : p.rest)),
                                         began ? static_cast<uint64_t>(p.t) * p.topk * p.k
                                               : static_cast<uint64_t>(kMoeMaxCtas) * kSegSlots * 128,
                                         s < count && col < p.k ? p.status : nullptr);
            if (s < count && col < p.k && inside) __stcg(dst, acc_slot(acc, s));
          }
        }
#pragma unroll
        for (int j = 0; j < kSegSlots / 2; ++j) acc[j] = 0;
        began = true;
      }
      if (!kCombine && (w.ks + 1 == stages || tile_end)) {
        // the segment's sums for its tokens; this thread alone adds to (token, row).  Four at a time, without branches
        // (unused slots add to row p.t): a token's slots of one expert are neighbours and are added up first, so that four
        // sums can be read before any is written.
        const int token = (lane & 15) < count ? table.token[seg.first + (lane & 15)] : p.t;   // of slot lane % 16
#pragma unroll
        for (int s0 = 0; s0 < kSegSlots; s0 += 4) {
          if (s0 >= count) break;
          float add[4], old[4];
          int at[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            at[s] = __shfl_sync(0xffffffffu, token, s0 + s) * 128;
            add[s] = acc_slot(acc, s0 + s);
            if (s > 0) {
              const bool same = at[s] == at[s - 1];
              add[s] += same ? add[s - 1] : 0.0f;
              at[s - 1] = same ? p.t * 128 : at[s - 1];
            }
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) old[s] = my_sums[at[s]];
#pragma unroll
          for (int s = 0; s < 4; ++s) my_sums[at[s]] = old[s] + add[s];
        }
#pragma unroll
        for (int j = 0; j < kSegSlots / 2; ++j) acc[j] = 0;
      }
      if (kCombine || !tile_end) {
        w.next();
        ++i;
        continue;
      }
      const TileShare share(split, w.tile);
      epilogue_sync();
      bool finish = true;
      if (share.c0 != share.c1) {
        float* mine = p.part + static_cast<int64_t>(share.place(blockIdx.x)) * width;
        for (int j = tid * 4; j < width; j += 512)
          __stcg(reinterpret_cast<float4*>(mine + j), *reinterpret_cast<const float4*>(sums + j));
        __threadfence();
        epilogue_sync();
        if (tid == 0) ctl.last = atomicAdd(p.count + w.tile, 1u) == static_cast<uint32_t>(share.c1 - share.c0);
        epilogue_sync();
        finish = ctl.last != 0;
        if (finish) {
          __threadfence();
          for (int j = tid * 4; j < width; j += 512) {
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int c = share.c0; c <= share.c1; ++c) {
              const float4 b4 = __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(share.place(c)) * width + j));
              a = make_float4(a.x + b4.x, a.y + b4.y, a.z + b4.z, a.w + b4.w);
            }
            *reinterpret_cast<float4*>(sums + j) = a;
          }
          epilogue_sync();
        }
      }
      if (finish) {
        for (int j = tid; j < p.t * 64; j += 128) {
          const int tok = j >> 6, r = (j & 63) * 2, col = w.tile * 128 + r;
          const float* s0 = sums + tok * 128 + r;
          const int64_t o = static_cast<int64_t>(tok) * p.k + col;
          if (col < p.k && index_ok(o + 1, static_cast<uint64_t>(p.t) * p.k, p.status))
            *reinterpret_cast<uint32_t*>(p.out + o) = pack_bf16x2(s0[0], s0[1]);
        }
      }
      epilogue_sync();                           // the sums are free again
      w.next();
      ++i;
      if (w.valid())
        for (int j = 0; j < p.t; ++j) my_sums[j * 128] = 0.0f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kMoeTmemCols) : "memory");
  }
}

// Adds the results of a token's slots, in a fixed order, four columns a thread.  What moe_up_kernel left (complete when this kernel
// starts: see moe_down_kernel) is read beside that kernel's last tiles, past L1.
__global__ void __launch_bounds__(256) moe_combine_kernel(const MoeParams p) {
  __shared__ int2 joined[kMoeMaxCtas];           // the tile's CTAs after c0, the one that begins it: a segment that each joined, its first position
  pdl_launch_dependents();
  const int nseg = __ldcg(p.nseg);
  const int tile = blockIdx.x;
  const int j = (blockIdx.y * 256 + threadIdx.x) * 4;
  const int tok = j >> 7, in = j & 127, col = tile * 128 + in;
  constexpr int kBatch = 8;                      // slots whose results are asked for together
  uint32_t v[kBatch];
  auto places = [&](int i0) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = tok * p.topk + i0 + q;
      v[q] = tok < p.t && i0 + q < p.topk && index_ok(i, p.t * p.topk, p.status) ? __ldcg(p.slot_pos + i) : kNoPosition;
    }
  };
  places(0);
  int c0 = 0, parts = 0;
  if (nseg) {
    const int stages = (p.n + 255) / 256;
    const DownSplit split((p.k + 127) / 128, nseg * stages, p.down_ctas);
    const int u0 = tile * split.upt;
    c0 = split.cta_of(u0);
    parts = split.cta_of(u0 + split.upt - 1) - c0;
    if (threadIdx.x < parts) {
      const int in_tile = split.start(c0 + 1 + static_cast<int>(threadIdx.x)) - u0, sg = in_tile / stages;
      const bool joins = in_tile != sg * stages;
      joined[threadIdx.x] = make_int2(joins ? sg : -1, joins ? __ldcg(&p.segments[sg].first) : 0);
    }
  }
  __syncthreads();
  pdl_wait();
  if (tok >= p.t || col >= p.k) return;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = 0; i0 < p.topk; i0 += kBatch) {
    if (i0 > 0) places(i0);
    float4 b[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      b[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (v[q] != kNoPosition) b[q] = __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(v[q] & 0xffffu) * p.k + col));
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) a = make_float4(a.x + b[q].x, a.y + b[q].y, a.z + b[q].z, a.w + b[q].w);
    for (int c = 0; c < parts; ++c) {
      const int2 from = joined[c];
      if (from.x < 0) continue;
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (v[q] == kNoPosition || static_cast<int>(v[q] >> 16) != from.x) continue;
        const int s = static_cast<int>(v[q] & 0xffffu) - from.y;
        const float4 r = __ldcg(reinterpret_cast<const float4*>(p.rest + (static_cast<int64_t>(c0 + 1 + c) * kSegSlots + s) * 128 + in));
        a = make_float4(a.x + r.x, a.y + r.y, a.z + r.z, a.w + r.w);
      }
    }
  }
  const int64_t o = static_cast<int64_t>(tok) * p.k + col;
  if (index_ok(o + 3, static_cast<uint64_t>(p.t) * p.k, p.status))
    *reinterpret_cast<uint2*>(p.out + o) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

// ---- host side ----------------------------------------------------------------------------------------

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

// CTAs of a cluster of moe_up_kernel, 1 to kUpMaxCluster.
constexpr int kUpMaxCluster = 4;

// A CTA per tile is best where there are tiles enough: a cluster's CTAs wait for one another at every tile (clusters of 2 instead:
// 64 tokens, 64 experts 1408 x 2048 87 against 71 us, the wide experts 119 against 112).  With few tiles clusters share them by K.
// One cluster of 1 to 4 CTAs per tile: the size for which the busiest cluster's K stages per CTA, with two stages' time
// for each tile that a cluster has to gather, are fewest.  `fits` has the number of clusters that run at once for each
// size; the number of segments is known on the device only, so the expected one is taken.
int up_cluster(int64_t S, int64_t E, int64_t row_tiles, int64_t stages, const int* fits) {
  // (1 - 1/E)^S: an expert without slots
  const double miss = std::pow(1.0 - 1.0 / static_cast<double>(E), static_cast<double>(S));
  const double segs = static_cast<double>(E) * (1.0 - miss);
  const int64_t tiles = static_cast<int64_t>(segs + 0.5 < 1.0 ? 1.0 : segs + 0.5) * row_tiles;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kUpMaxCluster && s <= stages; ++s) {
    if (fits[s - 1] <= 0) continue;
    const int64_t cost = (tiles + fits[s - 1] - 1) / fits[s - 1] * ((stages + s - 1) / s + (s > 1 ? 2 : 0));
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

template <bool kConvert>
int run_up(const MoeMaps& maps, MoeParams& p, const DeviceInfo& info, cudaStream_t stream) {
  auto kernel = moe_up_kernel<kConvert>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kUpThreads);
  cfg.dynamicSmemBytes = up_smem(p.t * p.topk);
  cfg.attrs = attr;
  int packed = 0;                                // clusters that fit, 8 bits for each size
  const int st = kernel_setup(reinterpret_cast<const void*>(kernel), info.device, [&](int* v) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, up_smem(kMoeMaxSlots)) != cudaSuccess) {
      cudaGetLastError();
      return static_cast<int>(NVFP4_ERR_CUDA);
    }
    uint32_t bits = 0;
    for (int s = 1; s <= kUpMaxCluster; ++s) {
      attr[0].val.clusterDim.x = static_cast<unsigned>(s);
      cfg.gridDim = dim3(static_cast<unsigned>(info.sm_count / s * s));
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      bits |= static_cast<uint32_t>(n < 255 ? n : 255) << (8 * (s - 1));
    }
    *v = static_cast<int>(bits);
    return static_cast<int>(NVFP4_OK);
  }, &packed);
  if (st != NVFP4_OK) return st;
  int fits[kUpMaxCluster];
  for (int s = 0; s < kUpMaxCluster; ++s) fits[s] = static_cast<int>((static_cast<uint32_t>(packed) >> (8 * s)) & 255u);
  if (fits[0] <= 0) return NVFP4_ERR_CUDA;
  const int64_t row_tiles = (p.n + 127) / 128;
  const int s = up_cluster(static_cast<int64_t>(p.t) * p.topk, p.experts, row_tiles, (p.k + 255) / 256, fits);
  const int64_t most = static_cast<int64_t>(p.max_segments) * row_tiles;     // tiles
  const int64_t clusters = most < fits[s - 1] ? most : fits[s - 1];
  attr[0].val.clusterDim.x = static_cast<unsigned>(s);
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * s));
  // Where this kernel leaves SMs free, CTAs of the next one run beside it from its start, and their loads would only compete
  // with its own (one token, when the slices had a kernel of their own: 20.2 against 20.0 us); otherwise they fill its end (8 tokens
  // of the wide experts: 108 against 110 us).
  p.down_early = clusters == fits[s - 1];
  cfg.stream = stream;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  return NVFP4_OK;
}

template <bool kCombine>
int run_down(const MoeMaps& maps, const MoeParams& p, const DeviceInfo& info, cudaStream_t stream) {
  auto kernel = moe_down_kernel<kCombine>;
  int ready = 0;
  int st = kernel_setup(reinterpret_cast<const void*>(kernel), info.device, [&](int* v) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) {
      cudaGetLastError();
      return static_cast<int>(NVFP4_ERR_CUDA);
    }
    *v = 1;
    return static_cast<int>(NVFP4_OK);
  }, &ready);
  if (st != NVFP4_OK) return st;
  const int grid = p.down_ctas;
  st = launch_kernel(kernel, dim3(grid), dim3(kDownThreads), down_smem(p.t, p.t * p.topk), stream, maps, p);
  if (st != NVFP4_OK || !kCombine) return st;
  return launch_kernel(moe_combine_kernel, dim3((p.k + 127) / 128, (p.t * 32 + 255) / 256), dim3(256), 0, stream, p);
}

bool moe_shape_ok(int64_t t, int64_t topk, int64_t E, int64_t n, int64_t k) {
  return t >= 0 && t <= kMoeMaxTokens && topk > 0 && topk <= kMoeMaxTopk && E > 0 && E <= kMoeMaxExperts && n > 0 && k > 0 &&
         n % 64 == 0 && k % 64 == 0 && n <= (1 << 17) && k <= (1 << 17);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

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
  MoeMaps maps;
  if ((st = make_weight_map(&maps.gate, w_gate, E, n, k)) != NVFP4_OK) return st;
  if ((st = make_weight_map(&maps.up, w_up, E, n, k)) != NVFP4_OK) return st;
  if ((st = make_weight_map(&maps.down, w_down, E, k, n)) != NVFP4_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeParams p;
  memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.ids = ids;
  p.weights = weights;
  p.gate_sf = w_gate_sf;
  p.up_sf = w_up_sf;
  p.down_sf = w_down_sf;
  p.gate_amax = gate_amax;
  p.up_amax = up_amax;
  p.down_amax = down_amax;
  p.out = static_cast<__nv_bfloat16*>(out_bf16);
  p.status = info.status;
  p.nseg = reinterpret_cast<int32_t*>(ws);
  p.segments = reinterpret_cast<Segment*>(ws + L.segments);
  p.count = reinterpret_cast<uint32_t*>(ws + L.count);
  p.f_x = reinterpret_cast<float*>(ws + L.f_x);
  p.f_h = reinterpret_cast<float*>(ws + L.f_h);
  p.b_x = ws + L.b_x;
  p.b_h = ws + L.b_h;
  p.slot_pos = reinterpret_cast<uint32_t*>(ws + L.slot_pos);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.rest = reinterpret_cast<float*>(ws + L.rest);
  p.up_stride = nvfp4_scale_bytes(n, k);
  p.down_stride = nvfp4_scale_bytes(k, n);
  p.b_units = L.b_units;
  p.max_segments = L.max_segments;
  p.t = static_cast<int32_t>(t);
  p.topk = static_cast<int32_t>(topk);
  p.experts = static_cast<int32_t>(E);
  p.n = static_cast<int32_t>(n);
  p.k = static_cast<int32_t>(k);
  p.down_ctas = info.sm_count < kMoeMaxCtas ? info.sm_count : kMoeMaxCtas;
  if (t <= kMoeConvertTokens) {
    if ((st = run_up<true>(maps, p, info, stream)) != NVFP4_OK) return st;
    return run_down<false>(maps, p, info, stream);
  }
  // a token's slots in as many parts as one CTA per SM has warps for
  const int64_t chunks = t * ((k + 255) / 256), want = 8 * info.sm_count / chunks;
  const int parts = static_cast<int>(want < 1 ? 1 : (want < topk ? want : topk));
  const int64_t items = (chunks * parts + 7) / 8;
  const int grid = static_cast<int>(items < info.sm_count ? items : info.sm_count);
  const int slice_smem = grouping_bytes(p.experts, p.t * p.topk);
  if ((st = launch_kernel(moe_slice_kernel, dim3(grid), dim3(256), slice_smem, stream, p, parts)) != NVFP4_OK) return st;
  if ((st = run_up<false>(maps, p, info, stream)) != NVFP4_OK) return st;
  return t > kMoeLastCtaTokens ? run_down<true>(maps, p, info, stream) : run_down<false>(maps, p, info, stream);
}

}  // extern "C"
