// lora.cu -- low-rank adapters of many requests beside a shared NVFP4 projection.
//
//   nvfp4_lora_down_batched   d[i] = bf16(x[i] @ w[adapter[i]]^T)
//   nvfp4_gemm_lora_batched   out[i] = bf16(alpha * a[i] @ b^T + d[i] @ l1[adapter[i]]^T [+ bias])
//
// Every row names its adapter.  Both products are matrix products only among rows of the same adapter, so
// a tile of rows takes one MMA pass per adapter that occurs in it (rows of one request are usually
// adjacent: one to three adapters a tile) and each row keeps the pass of its own adapter:
//   lora_down_tiles_kernel   128 rows of x against the occurring adapters' w side by side (as many as fit
//                            256 accumulator columns), tcgen05 bf16 MMA, K split over a cluster of 4 CTAs
//                            whose partial sums meet through distributed shared memory; a row reads only
//                            its adapter's columns.  x is read once.
//   lora_down_mixed_kernel   tiles of many adapters, one row at a time like the next one.
//   lora_down_rows_kernel    the same for few rows, where reading the adapters is the whole time: one CTA per row and 8 of
//                            its rank's values, so that rows x ranks spread over the GPU.
//   gemm_lora_rows_kernel    few rows of small rank: projection and low-rank products in one launch.
//   lora_spread_kernel       for each 256-row output tile the list of its adapters and, per adapter, d / alpha with other
//                            adapters' rows zeroed; the GEMM adds one bf16 MMA per listed adapter to its FP4
//                            accumulator (gemm.cu) and out is written once.  It also looks for values that these MMAs
//                            cannot take; the rows concerned get their low-rank term in the GEMM's epilogue.
//
// Measured, back to back (HBM copies at 6.53 TB/s): lora_down_tiles_kernel, 4096 rows of 5120, 8 adapters of rank 64, 45 MB:
// 15.6 us (2.9 TB/s; it streams at 6.7 for 6 us, start and the sum over the cluster take the rest); lora_down_rows_kernel,
// 48 rows of 5120, 40 adapters of rank 16, 4.7 MB: 3.5 us; gemm_lora_rows_kernel, 1 x 5120 x 5120, rank 16, 15 MB: 6.7 us and
// 48 x 7168 x 5120, 40 adapters, 27 MB: 11.5 us; the GEMM with lora_spread_kernel, 2011 x 8192 x 5120, 12 adapters of rank 32: 45 us
// (nvfp4_gemm alone 39: the second launch and the wait for it 3, loads of the low-rank stages 2, their MMAs 1; with every row finished
// in the epilogue 195).
//
// Sources (page title, section): flashinfer docs mm_nvfp4_svdquant (the single low-rank pair that these calls extend to
// one pair per row).
#include <cuda_bf16.h>

#include "common.cuh"
#include "nvfp4_math.cuh"
#include "tc_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kLoraMaxRank = 256;
constexpr int kLoraMaxAdapters = 65536;

// ---- the distinct adapters of kRows rows ---------------------------------------------------------------

template <int kRows>
struct __align__(16) AdapterList {
  int32_t id[kRows];            // adapter of the row (-1: none)
  int16_t first[kRows];         // first rows of the distinct adapters, in order
  int16_t at[kRows];            // the place of the row's adapter among them (-1: none)
  int32_t warp_count[kRows / 32];
  int32_t count;
  __device__ __forceinline__ int32_t adapter(int place) const { return id[first[place]]; }
};

// Fills `a` for rows [row0, row0 + kRows) with threads [0, kRows); every thread of the CTA calls it.
template <int kRows>
__device__ __forceinline__ void list_adapters(AdapterList<kRows>& a, const int32_t* adapter, int row0, int m, int adapters,
                                              int* status) {
  const int t = threadIdx.x, lane = t & 31;
  if (t < kRows) {
    int id = -1;
    if (row0 + t < m && index_ok(row0 + t, m, status)) id = adapter[row0 + t];
    a.id[t] = id >= 0 && id < adapters ? id : -1;
  }
  __syncthreads();
  bool first = false;
  int same = t;
  uint32_t firsts = 0;
  if (t < kRows) {
    // the first row of this adapter: within the warp, else in an earlier warp's rows (read four at a time)
    const int id = a.id[t];
    same = (t & ~31) + __ffs(__match_any_sync(0xffffffffu, id)) - 1;
    const int4* ids = reinterpret_cast<const int4*>(a.id);
#pragma unroll 4
    for (int j = (t >> 5) * 8 - 1; j >= 0; --j) {
      const int4 v = ids[j];
      same = v.w == id ? 4 * j + 3 : same;
      same = v.z == id ? 4 * j + 2 : same;
      same = v.y == id ? 4 * j + 1 : same;
      same = v.x == id ? 4 * j : same;
    }
    first = id >= 0 && same == t;
    firsts = __ballot_sync(0xffffffffu, first);
    if (lane == 0) a.warp_count[t >> 5] = __popc(firsts);
  }
  __syncthreads();
  if (t < kRows) {
    int base = 0;
    for (int w = 0; w < (t >> 5); ++w) base += a.warp_count[w];
    const int place = base + __popc(firsts & ((1u << lane) - 1u));
    if (first) {
      a.first[place] = static_cast<int16_t>(t);
      a.at[t] = static_cast<int16_t>(place);
    }
    if (t == kRows - 1) a.count = base + __popc(firsts);
  }
  __syncthreads();
  if (t < kRows && !first) a.at[t] = a.id[t] < 0 ? int16_t(-1) : a.at[same];
  __syncthreads();
}

// ---- lora down, tiles of 128 rows -------------------------------------------------------------------------

constexpr int kLdSplit = 4;
constexpr int kLdXBytes = 128 * 128;                 // 128 rows x 64 bf16
constexpr int kLdColumns = 256;                      // most accumulator columns of a pass: adapters x rank
// A stage is 128 values of K of x and of as many rows of w as the tile's adapters have, 64, 128 or 256 at a time: 48, 64 or 96 KB,
// so that the ring holds 4, 3 or 2 stages.  With stages of 64 values the MMA issuer's waits and commits were the bound (4096 rows of 5120:
// 16.0 us).
constexpr int kLdRingBytes = 192 * 1024;
constexpr int kLdMaxStages = 4;
constexpr int kLdThreads = 192;                      // producer, MMA issuer, four drain warps

struct __align__(16) LdControl {
  uint64_t full[kLdMaxStages], empty[kLdMaxStages], acc_full;
  uint32_t tmem_base;
  int32_t abort;
  AdapterList<128> rows;
};
constexpr int kLdSmem = kLdRingBytes + static_cast<int>(sizeof(LdControl)) + 1024;
static_assert(kLdSmem <= 227 * 1024, "shared memory layout exceeds the per-block limit");
static_assert(128 * kLoraMaxRank * 4 <= kLdRingBytes, "the partial sums reuse the ring");

struct LdMaps {
  CUtensorMap x, w;
};

struct LoraDownParams {
  const int32_t* adapter;
  __nv_bfloat16* d;
  int* status;
  int32_t m, k, r, adapters;
  int32_t max_passes;           // tiles that would take more are left to lora_down_mixed_kernel
};

// Accumulator columns of an adapter, columns of a pass over a tile with `count` adapters, and the passes it takes.
__host__ __device__ inline int ld_columns(int r) { return (r + 15) / 16 * 16; }
__host__ __device__ inline int ld_pass_columns(int r, int count) {
  const int want = count * ld_columns(r);
  return want <= 64 ? 64 : (want <= 128 ? 128 : kLdColumns);
}
__host__ __device__ inline int ld_passes(int r, int count) {
  if (count == 0) return 0;
  const int per = ld_pass_columns(r, count) / ld_columns(r);
  return (count + per - 1) / per;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __cluster_dims__(kLdSplit, 1, 1) __launch_bounds__(kLdThreads, 1)
    lora_down_tiles_kernel(const __grid_constant__ LdMaps maps, const LoraDownParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LdControl& ctl = *reinterpret_cast<LdControl*>(smem + kLdRingBytes);
  volatile int32_t* abort = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int row0 = blockIdx.y * 128;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kLdMaxStages; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    mbar_init(&ctl.acc_full, 1);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem_base)),
                 "r"(static_cast<uint32_t>(kLdColumns))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  pdl_wait();
  pdl_launch_dependents();       // in this order: lora_down_mixed_kernel reads the call's inputs as it starts
  list_adapters(ctl.rows, p.adapter, row0, p.m, p.adapters, p.status);

  const int chunks = (p.k + 127) / 128;                          // what lies beyond k is loaded as zeros
  const int nch = (chunks - rank + kLdSplit - 1) / kLdSplit;     // this CTA's chunks: rank, rank + 4, ...
  const int cols = ld_columns(p.r);
  const int pass_cols = ld_pass_columns(p.r, ctl.rows.count);
  const int per = pass_cols / cols;                              // adapters of a pass
  const int half_bytes = kLdXBytes + pass_cols * 128;            // 64 values of K
  const int stage_bytes = 2 * half_bytes;
  const uint32_t ring = static_cast<uint32_t>(min(kLdRingBytes / stage_bytes, kLdMaxStages));
  const int all = ld_passes(p.r, ctl.rows.count), passes = all <= p.max_passes ? all : 0;
  float* partial = reinterpret_cast<float*>(smem);
  uint32_t s = 0, phase = 0;                                     // the ring goes on over all passes
  bool wrapped = false;                                          // (producer)
  for (int pass = 0; pass < passes; ++pass) {
    const int first = pass * per, here = min(per, ctl.rows.count - first);
    if (warp == 0) {
      for (int c = 0; c < nch; ++c) {
        if (wrapped && !mbar_wait_fast(&ctl.empty[s], phase, abort, p.status)) break;
        if (elect_one()) {
          uint8_t* st = smem + s * stage_bytes;
          mbar_arrive_expect_tx(&ctl.full[s], static_cast<uint32_t>(2 * (kLdXBytes + here * cols * 128)));
          for (int h = 0; h < 2; ++h, st += half_bytes) {
            const int k0 = (rank + c * kLdSplit) * 128 + h * 64;
            tma_load_2d_cta(st, &maps.x, &ctl.full[s], k0, row0);
            for (int j = 0; j < here; ++j)
              tma_load_3d_cta(st + kLdXBytes + j * cols * 128, &maps.w, &ctl.full[s], k0, 0, ctl.rows.adapter(first + j));
          }
        }
        __syncwarp();
        if (++s == ring) {
          s = 0;
          if (wrapped) phase ^= 1u;
          wrapped = true;
        }
      }
    } else if (warp == 1) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(cols >> 3) << 17) | ((128u >> 4) << 24);
      bool ok = true;
      for (int c = 0; c < nch; ++c) {
        if (!(ok = mbar_wait_fast(&ctl.full[s], phase, abort, p.status))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t st = smem_u32(smem) + s * stage_bytes;
          const uint64_t a0 = operand_desc(st), a1 = operand_desc(st + half_bytes);
          for (int j = 0; j < here; ++j) {
            const uint64_t b0 = operand_desc(st + kLdXBytes + j * cols * 128);
            const uint64_t b1 = operand_desc(st + half_bytes + kLdXBytes + j * cols * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_bf16_cta(tmem + j * cols, a0 + 2 * q, b0 + 2 * q, idesc, c > 0 || q > 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_bf16_cta(tmem + j * cols, a1 + 2 * q, b1 + 2 * q, idesc, true);
          }
          mma_commit_cta(&ctl.empty[s]);
        }
        __syncwarp();
        if (++s == ring) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (ok && nch > 0 && elect_one()) mma_commit_cta(&ctl.acc_full);
      __syncwarp();
    } else {
      // the row's own adapter's columns, column-major: partial[column][row]
      const int row = (warp & 3) * 32 + lane;
      const int mine = ctl.rows.at[row] - first;
      const bool in_pass = ctl.rows.at[row] >= 0 && mine >= 0 && mine < here;
      const bool ready = nch > 0 && mbar_wait(&ctl.acc_full, pass & 1, abort, p.status);
      tc_fence_after();
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      for (int j = 0; j < here; ++j) {
        if (!__any_sync(0xffffffffu, in_pass && mine == j)) continue;
        for (int c0 = 0; c0 < cols; c0 += 16) {
          uint32_t v[16];
          if (nch > 0) {
            tmem_load_16(tmem + j * cols + c0 + lane_base, v);
            tmem_wait_ld<16>(v);
          }
          if (in_pass && mine == j) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c0 + e < p.r) partial[(c0 + e) * 128 + row] = ready ? __uint_as_float(v[e]) : 0.0f;
          }
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    cluster_sync();          // the partial sums of all four CTAs are in their shared memory
    // CTA c adds up rows [32c, 32c + 32) of the tile: a lane per row, the warps share the columns by eights
    {
      const int row = rank * 32 + lane;
      const int mine = ctl.rows.at[row] - first;
      if (ctl.rows.at[row] >= 0 && mine >= 0 && mine < here && !*abort) {
        uint32_t peer[kLdSplit];
#pragma unroll
        for (int q = 0; q < kLdSplit; ++q) peer[q] = map_to_rank(partial, static_cast<uint32_t>(q));
        for (int c0 = warp * 8; c0 < p.r; c0 += 8 * (kLdThreads / 32)) {
          float sum[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t off = static_cast<uint32_t>(((c0 + e) * 128 + row) * 4);
            sum[e] = 0.0f;
#pragma unroll
            for (int q = 0; q < kLdSplit; ++q) sum[e] += ld_cluster_f32(peer[q] + off);
          }
          const int64_t o = static_cast<int64_t>(row0 + row) * p.r + c0;
          if (index_ok(o + 7, static_cast<uint64_t>(p.m) * p.r, p.status))
            *reinterpret_cast<uint4*>(p.d + o) = make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]),
                                                            pack_bf16x2(sum[4], sum[5]), pack_bf16x2(sum[6], sum[7]));
        }
      }
    }
    fence_async_smem();      // the next pass loads over the partial sums
    cluster_sync();
  }
  // rows without an adapter
  {
    const int row = rank * 32 + lane;
    if (row0 + row < p.m && ctl.rows.at[row] < 0) {
      for (int c0 = warp * 8; c0 < p.r; c0 += 8 * (kLdThreads / 32)) {
        const int64_t o = static_cast<int64_t>(row0 + row) * p.r + c0;
        if (index_ok(o + 7, static_cast<uint64_t>(p.m) * p.r, p.status))
          *reinterpret_cast<uint4*>(p.d + o) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  if (*abort) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(kLdColumns))
                 : "memory");
  }
}

// ---- lora down, few rows -------------------------------------------------------------------------------------

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// d[row][c0 .. c0 + 8) of a row with adapter `id` (-1: zeros): the CTA's threads share K, a thread multiplies eight values of x with eight
// rows of w, two products an instruction.
__device__ __forceinline__ void lora_down_row(const uint16_t* x, const uint16_t* w, const LoraDownParams& p, int row, int id, int c0,
                                              float (&part)[8][8]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0;
  if (id >= 0) {
    const uint16_t* xr = x + static_cast<int64_t>(row) * p.k;
    const uint16_t* wr = w + (static_cast<int64_t>(id) * p.r + c0) * p.k;
    for (int k0 = threadIdx.x * 8; k0 < p.k; k0 += 2048) {
      if (!index_ok((static_cast<uint64_t>(id) * p.r + c0 + 7) * p.k + k0 + 7, static_cast<uint64_t>(p.adapters) * p.r * p.k,
                    p.status) ||
          !index_ok(static_cast<uint64_t>(row) * p.k + k0 + 7, static_cast<uint64_t>(p.m) * p.k, p.status))
        break;
      const uint4 xv = __ldg(reinterpret_cast<const uint4*>(xr + k0));
      uint4 wv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) wv[j] = __ldg(reinterpret_cast<const uint4*>(wr + static_cast<int64_t>(j) * p.k + k0));
      const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
      uint64_t x2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x2[e] = pack2(bf16_lo(xs[e]), bf16_hi(xs[e]));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t ws[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j] = fma_f32x2(x2[e], pack2(bf16_lo(ws[e]), bf16_hi(ws[e])), acc[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float lo, hi;
    unpack2(acc[j], lo, hi);
    float sum = lo + hi;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp][j] = sum;
  }
  __syncthreads();
  if (threadIdx.x < 8) {
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) sum += part[q][threadIdx.x];
    const int64_t o = static_cast<int64_t>(row) * p.r + c0 + threadIdx.x;
    if (index_ok(o, static_cast<uint64_t>(p.m) * p.r, p.status)) p.d[o] = __float2bfloat16_rn(sum);
  }
}

// One CTA per (row, 8 rank values).  Its time is the reading of w from L2 (about 16 TB/s at 1024 rows of rank 64); giving a CTA four rows
// of one adapter, so that they share w, was 10 to 15 % faster on sorted rows and up to 60 % slower on mixed ones.
__global__ void __launch_bounds__(256) lora_down_rows_kernel(const uint16_t* x, const uint16_t* w, const LoraDownParams p) {
  __shared__ float part[8][8];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x;
  int id = index_ok(row, p.m, p.status) ? p.adapter[row] : -1;
  if (id >= p.adapters) id = -1;
  lora_down_row(x, w, p, row, id, blockIdx.y * 8, part);
}

// The rows of the tiles that lora_down_tiles_kernel leaves out, the same way, beside that kernel; the CTAs of blockIdx.y share a tile.
__global__ void __launch_bounds__(256) lora_down_mixed_kernel(const uint16_t* x, const uint16_t* w, const LoraDownParams p) {
  __shared__ float part[8][8];
  __shared__ AdapterList<128> rows;
  pdl_launch_dependents();
  const int row0 = blockIdx.x * 128;
  list_adapters(rows, p.adapter, row0, p.m, p.adapters, p.status);
  if (ld_passes(p.r, rows.count) > p.max_passes) {
    const int groups = p.r / 8;
    for (int i = blockIdx.y; i < min(128, p.m - row0) * groups; i += gridDim.y) {
      const int row = i / groups, id = rows.id[row];
      if (id < 0) continue;      // that kernel writes its zeros
      lora_down_row(x, w, p, row0 + row, id, (i - row * groups) * 8, part);
      __syncthreads();           // part is free again
    }
  }
  pdl_wait();                    // this kernel ends after that one
}

// ---- the projection of few rows ------------------------------------------------------------------------------------

// Up to 128 rows: the 128-row tiles of the weight b are the MMA's M side and the rows of a its N side (16 to 128 columns), so that
// every SM streams weights: a tile belongs to a cluster of one to four CTAs that share its K stages.  While the weights come in, the
// epilogue warps compute the low-rank products of the CTA's share of the rows from l1 (each l1 row is needed by one tile
// only); then the CTAs' sums meet through distributed shared memory and every CTA writes its share of the rows.
constexpr int kGrMaxRows = 128;
constexpr int kGrMaxStages = 8;
constexpr int kGrEpiWarps = 16;
constexpr int kGrThreads = 64 + 32 * kGrEpiWarps;   // TMA producer, MMA issuer, epilogue warps
constexpr int kGrMaxCluster = 4;
constexpr uint32_t kGrTmemCols = 256;            // 128 accumulator columns, then 4 x 8 of scales

struct __align__(8) GrControl {
  uint64_t full[kGrMaxStages], empty[kGrMaxStages], acc_full;
  uint32_t tmem_base;
  int32_t abort;
};

__host__ __device__ constexpr int gr_columns(int m) { return m <= 16 ? 16 : (m <= 32 ? 32 : (m <= 64 ? 64 : 128)); }
// a stage: 128 weight rows and `columns` rows of a, 256 FP4 values each, and their scales (4 chunks each)
__host__ __device__ constexpr int gr_stage_bytes(int columns) { return 128 * 128 + columns * 128 + 2 * 2048; }
__host__ __device__ constexpr int gr_rest_bytes(int m) { return gr_columns(m) * 512 + static_cast<int>(sizeof(GrControl)) + 1024; }
__host__ __device__ constexpr int gr_stages(int m) {
  return (227 * 1024 - gr_rest_bytes(m)) / gr_stage_bytes(gr_columns(m)) < kGrMaxStages
             ? (227 * 1024 - gr_rest_bytes(m)) / gr_stage_bytes(gr_columns(m))
             : kGrMaxStages;
}
__host__ __device__ constexpr int gr_smem(int m) { return gr_stages(m) * gr_stage_bytes(gr_columns(m)) + gr_rest_bytes(m); }
static_assert(gr_stages(kGrMaxRows) >= 4 && gr_stage_bytes(16) % 1024 == 0, "shared memory layout");

struct GrMaps {
  CUtensorMap a, b;
};

struct GrParams {
  const uint8_t *a_sf, *b_sf;
  const float* alpha;
  const uint16_t *d, *l1, *bias;
  const int32_t* adapter;
  __nv_bfloat16* out;
  int* status;
  int32_t m, n, k, r, adapters;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__global__ void __launch_bounds__(kGrThreads, 1) gemm_lora_rows_kernel(const __grid_constant__ GrMaps maps, const GrParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int columns = gr_columns(p.m), ring = gr_stages(p.m), stage_bytes = gr_stage_bytes(columns);
  float* sums = reinterpret_cast<float*>(smem + ring * stage_bytes);           // [columns][128]
  GrControl& ctl = *reinterpret_cast<GrControl*>(sums + columns * 128);
  volatile int32_t* abort = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    mbar_init(&ctl.acc_full, 1);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem_base)),
                 "r"(kGrTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && elect_one()) {
    prefetch_map(&maps.a);
    prefetch_map(&maps.b);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  const int stages = (p.k + 255) / 256, groups = p.k / 64, tiles = (p.n + 127) / 128;
  const int k0 = rank * stages / ctas, k1 = (rank + 1) * stages / ctas;       // this CTA's K stages of every tile
  uint32_t n_tile = 0, s = 0, phase = 0;        // the ring goes on over all tiles
  bool wrapped = false;                          // (producer)
  for (int tile = static_cast<int>(blockIdx.x) / ctas; tile < tiles; tile += static_cast<int>(gridDim.x) / ctas, ++n_tile) {
    if (warp == 0) {
      for (int ks = k0; ks < k1; ++ks) {
        if (wrapped && !mbar_wait_fast(&ctl.empty[s], phase, abort, p.status)) break;
        if (elect_one()) {
          uint8_t* st = smem + s * stage_bytes;
          const uint32_t sf_bytes = static_cast<uint32_t>(min(4, groups - 4 * ks)) * 512u;
          mbar_arrive_expect_tx(&ctl.full[s], 128 * 128 + columns * 128 + 2 * sf_bytes);
          tma_load_2d_cta(st, &maps.b, &ctl.full[s], ks * 128, tile * 128);
          tma_load_2d_cta(st + 128 * 128, &maps.a, &ctl.full[s], ks * 128, 0);
          bulk_load_cta(st + 128 * 128 + columns * 128, p.b_sf + (static_cast<int64_t>(tile) * groups + 4 * ks) * 512, sf_bytes,
                        &ctl.full[s]);
          bulk_load_cta(st + 128 * 128 + columns * 128 + 2048, p.a_sf + static_cast<int64_t>(ks) * 2048, sf_bytes, &ctl.full[s]);
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(ring)) {
          s = 0;
          if (wrapped) phase ^= 1u;
          wrapped = true;
        }
      }
    } else if (warp == 1) {
      const uint32_t idesc = idesc_fp4_cta(static_cast<uint32_t>(columns));
      bool ok = true;
      for (int ks = k0; ks < k1; ++ks) {
        if (!(ok = mbar_wait_fast(&ctl.full[s], phase, abort, p.status))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t st = smem_u32(smem) + s * stage_bytes;
          const uint64_t a0 = operand_desc(st), b0 = operand_desc(st + 128 * 128);
          const uint64_t sfa = sf_chunk_desc(st + 128 * 128 + columns * 128), sfb = sf_chunk_desc(st + 128 * 128 + columns * 128 + 2048);
          auto step = [&](int j) {
            const uint32_t col = tmem + 128u + 8u * j;
            tc_copy_sf_cta(col, sfa + 32 * j);
            tc_copy_sf_cta(col + 4, sfb + 32 * j);
            mma_fp4_cta(tmem, a0 + 2 * j, b0 + 2 * j, idesc, col, col + 4, ks > k0 || j > 0);
          };
          const int steps = min(4, groups - 4 * ks);
          if (steps == 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) step(j);
          } else {
#pragma unroll 1
            for (int j = 0; j < steps; ++j) step(j);
          }
          mma_commit_cta(&ctl.empty[s]);
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(ring)) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (ok && elect_one()) mma_commit_cta(&ctl.acc_full);
      __syncwarp();
    } else {
      // a thread owns a weight row; the four warps of each TMEM lane quarter share the columns (rows of a)
      const int row = (warp & 3) * 32 + lane, part = (warp - 2) >> 2;
      const int g_row = tile * 128 + row;
      // low-rank products of rows rank, rank + ctas, ... of a for this thread's weight row, four at a time, the parts taking turns
      constexpr int kBatch = 4;
      int next[kBatch];                          // adapters of the next four rows, asked for before these rows' l1 is used
      auto ask = [&](int ib) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int i = ib + q * ctas;
          next[q] = i < p.m && index_ok(i, p.m, p.status) ? __ldg(p.adapter + i) : -1;
        }
      };
      ask(rank + ctas * kBatch * part);
      for (int ib = rank + ctas * kBatch * part; ib < p.m; ib += 4 * ctas * kBatch) {
        float acc[kBatch];
        const uint16_t* src[kBatch];
        bool any = false;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int ad = next[q];
          const bool has = ad >= 0 && ad < p.adapters && g_row < p.n;
          acc[q] = 0.0f;
          src[q] = has ? p.l1 + (static_cast<int64_t>(ad) * p.n + g_row) * p.r : nullptr;
          any = any || has;
        }
        ask(ib + 4 * ctas * kBatch);
        if (any) {
          for (int c0 = 0; c0 < p.r; c0 += 32) {
            uint4 w[kBatch][4];                  // 32 values of each row of l1
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                w[q][e] = make_uint4(0u, 0u, 0u, 0u);
                const int c = c0 + 8 * e;
                if (src[q] && c < p.r &&
                    index_ok(static_cast<uint64_t>(src[q] - p.l1) + c + 7, static_cast<uint64_t>(p.adapters) * p.n * p.r, p.status))
                  w[q][e] = __ldg(reinterpret_cast<const uint4*>(src[q] + c));
              }
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
              const uint16_t* x = p.d + static_cast<int64_t>(ib + q * ctas) * p.r;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int c = c0 + 8 * e;
                if (src[q] && c < p.r) acc[q] = dot8(w[q][e], __ldg(reinterpret_cast<const uint4*>(x + c)), acc[q]);
              }
            }
          }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
          if (ib + q * ctas < p.m) sums[(ib + q * ctas) * 128 + row] = acc[q];
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kGrEpiWarps) : "memory");
      const float alpha = __ldg(p.alpha);
      const bool ready = mbar_wait(&ctl.acc_full, n_tile & 1u, abort, p.status);
      tc_fence_after();
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      for (int c0 = 8 * part; c0 < columns; c0 += 32) {
        uint32_t v[8];
        tmem_load_8(tmem + static_cast<uint32_t>(c0) + lane_base, v);
        int own = (c0 + ctas - rank) % ctas;     // 0: a row of this CTA's share, which has its low-rank product already
        tmem_wait_ld<8>(v);
        float old[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) old[e] = sums[(c0 + e) * 128 + row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float base = own == 0 ? old[e] : 0.0f;
          if (ready) sums[(c0 + e) * 128 + row] = fmaf(alpha, __uint_as_float(v[e]), base);
          own = own + 1 == ctas ? 0 : own + 1;
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    // rows rank, rank + ctas, ... of a: the CTAs' sums in CTA order, bias, four output columns a lane
    if (!*abort) {
      for (int i = rank + ctas * warp; i < p.m; i += ctas * (kGrThreads / 32)) {
        const int col = tile * 128 + lane * 4;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int q = 0; q < ctas; ++q) {
          const float4 b = ld_cluster_f4(map_to_rank(sums + i * 128 + lane * 4, static_cast<uint32_t>(q)));
          a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        }
        if (p.bias && col < p.n && index_ok(col + 3, p.n, p.status)) {
          const uint2 bb = __ldg(reinterpret_cast<const uint2*>(p.bias + col));
          a.x += bf16_lo(bb.x), a.y += bf16_hi(bb.x), a.z += bf16_lo(bb.y), a.w += bf16_hi(bb.y);
        }
        const int64_t o = static_cast<int64_t>(i) * p.n + col;
        if (col < p.n && index_ok(o + 3, static_cast<uint64_t>(p.m) * p.n, p.status))
          *reinterpret_cast<uint2*>(p.out + o) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      }
    }
    __syncwarp();
    if (ctas > 1) cluster_sync();                // the sums are free again
    else __syncthreads();
  }
  if (*abort) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kGrTmemCols) : "memory");
  }
}

// ---- the GEMM's low-rank operand ---------------------------------------------------------------------------------

struct SpreadParams {
  const uint16_t* d;            // [m, r]
  const uint16_t* l1;           // [adapters, n, r]
  const int32_t* adapter;
  const float* alpha;
  int32_t *count, *list;
  int32_t* rows;                // [m]
  uint8_t* unfit;               // [adapters][kCheckParts]
  uint16_t* spread;             // [tiles][max][256][r]
  int* status;
  int32_t m, n, r, adapters, max;
  int32_t tiles, slices;        // the first tiles * slices CTAs spread, the others check
};

// d / alpha is rounded to bf16 once more (relative 2^-8 of each value): the MMA adds it to the FP4 accumulator, which the
// epilogue multiplies by alpha.  Rows with a value for which that does not work go to the GEMM's epilogue instead, which adds their
// product of d and l1 in fp32 (odd in p.rows; zeros here): every row with an adapter where 1 / alpha is not finite (alpha 0 or below
// 2^-128) or alpha above 2^32 (below that only a d under 2^-94 loses bits to bf16's subnormal range, and at most 2^-102), else
// those with a d / alpha above 2^64, infinities and NaN among them.
constexpr float kSpreadLimit = 0x1p64f, kAlphaLimit = 0x1p32f;
// A tile's MMA with an adapter multiplies the rows of the others by zero, so an infinity or NaN in one l1 would reach them all.
// Adapters with such a value, or one above 2^50 (2^64 * 2^50 * 256 is within fp32), are unfit for it: the GEMM loads zeros in their
// place, and their rows too go to its epilogue.  Looking for such values reads the l1 of every used adapter once (the GEMM reads
// them again, from L2 where they fit), beside the GEMM's first FP4 stages.
constexpr uint32_t kAbove = (0x7fffu - ((127 + 50) << 7)) * 0x10001u;   // added to two magnitudes, sets the top bits of those above 2^50
constexpr int kCheckParts = 16;                  // CTAs that share an adapter's l1; a byte each

struct __align__(16) SpreadShared {
  AdapterList<256> rows;
  uint32_t beyond[8];           // a bit for each row of the tile: a value above the limit
};
struct __align__(16) CheckShared {
  uint16_t mine[256];           // adapters that this CTA looks at
  uint32_t bad[8];              // a bit for each of them
  int32_t warp_count[8];
};                              // then a word of bits for every 32 adapters (used), and how many used ones come before each word
// With less than 2.9 KB a CTA of this kernel leaves room for one of the GEMM's beside it.
int spread_smem(int64_t adapters) {
  const int64_t check = sizeof(CheckShared) + (adapters + 31) / 32 * 6;
  return static_cast<int>(check > static_cast<int64_t>(sizeof(SpreadShared)) ? check : sizeof(SpreadShared));
}

__device__ __forceinline__ void spread_rows(const SpreadParams& p, SpreadShared& sh, int tile, int slice) {
  AdapterList<256>& rows = sh.rows;
  const int row0 = tile * 256;
  if (threadIdx.x < 8) sh.beyond[threadIdx.x] = 0;
  const float alpha = *p.alpha;
  list_adapters(rows, p.adapter, row0, p.m, p.adapters, p.status);
  const float inv = __fdiv_rn(1.0f, alpha);
  const int count = fabsf(inv) <= 3.402823466e38f && fabsf(alpha) <= kAlphaLimit ? rows.count : 0;
  if (slice == 0) {
    if (threadIdx.x == 0 && index_ok(tile, p.tiles, p.status)) p.count[tile] = count;
    for (int j = threadIdx.x; j < count; j += 256)
      if (index_ok(j, p.max, p.status)) p.list[static_cast<int64_t>(tile) * p.max + j] = rows.adapter(j);
  }
  const int words = p.r / 8, valid = min(256, p.m - row0);
  // this thread's row, if the CTA spreads its adapter (or none)
  const int my_at = rows.at[threadIdx.x];
  const bool mine = static_cast<int>(threadIdx.x) < valid && max(my_at, 0) % p.slices == slice &&
                    index_ok(row0 + threadIdx.x, p.m, p.status);
  if (mine) p.rows[row0 + threadIdx.x] = my_at >= 0 ? 2 * rows.id[threadIdx.x] + (my_at >= count) : -1;
  bool any_beyond = false;
  const uint64_t extent = static_cast<uint64_t>(p.tiles) * p.max * 256 * p.r;
  for (int j = slice; j < count; j += p.slices) {
    uint16_t* dst = p.spread + (static_cast<int64_t>(tile) * p.max + j) * 256 * p.r;
    for (int i = threadIdx.x; i < valid * words; i += 256) {
      const int row = i / words, c = (i - row * words) * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      const int64_t src = static_cast<int64_t>(row0 + row) * p.r + c;
      if (rows.at[row] == j && index_ok(src + 7, static_cast<uint64_t>(p.m) * p.r, p.status)) {
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p.d + src));
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        bool fits = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = bf16_lo(w[e]) * inv, hi = bf16_hi(w[e]) * inv;
          fits = fits && fabsf(lo) <= kSpreadLimit && fabsf(hi) <= kSpreadLimit;
          w[e] = pack_bf16x2(lo, hi);
        }
        if (!fits) {
          atomicOr(&sh.beyond[row >> 5], 1u << (row & 31));
          any_beyond = true;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (index_ok((static_cast<uint64_t>(tile) * p.max + j) * 256 * p.r + row * p.r + c + 7, extent, p.status))
        *reinterpret_cast<uint4*>(dst + row * p.r + c) = v;
    }
  }
  if (__syncthreads_or(any_beyond) && mine && my_at >= 0 && (sh.beyond[threadIdx.x >> 5] >> (threadIdx.x & 31) & 1u)) {
    p.rows[row0 + threadIdx.x] = 2 * rows.id[threadIdx.x] + 1;
    const int64_t dst = ((static_cast<int64_t>(tile) * p.max + my_at) * 256 + threadIdx.x) * p.r;
    for (int c = 0; c < p.r; c += 8)
      if (index_ok(dst + c + 7, extent, p.status)) *reinterpret_cast<uint4*>(p.spread + dst + c) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// CTA `block` of `blocks` (a multiple of kCheckParts) looks at one part of l1 of every blocks / kCheckParts-th used adapter.
__device__ __forceinline__ void check_adapters(const SpreadParams& p, CheckShared& sh, int block, int blocks) {
  constexpr int kDepth = 4;      // 8: no faster
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, words = (p.adapters + 31) / 32;
  uint32_t* const used = reinterpret_cast<uint32_t*>(&sh + 1);
  uint16_t* const before = reinterpret_cast<uint16_t*>(used + words);
  for (int w = t; w < words; w += 256) used[w] = 0;
  __syncthreads();
#pragma unroll 8
  for (int i = t; i < p.m; i += 256) {
    const int id = index_ok(i, p.m, p.status) ? p.adapter[i] : -1;
    if (id >= 0 && id < p.adapters && !(*const_cast<volatile uint32_t*>(used + (id >> 5)) >> (id & 31) & 1u))
      atomicOr(used + (id >> 5), 1u << (id & 31));
  }
  __syncthreads();
  const int per = (words + 255) / 256, w0 = min(t * per, words), w1 = min(w0 + per, words);
  int sum = 0;
  for (int w = w0; w < w1; ++w) sum += __popc(used[w]);
  const int here = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) sh.warp_count[warp] = sum;
  __syncthreads();
  sum -= here;
  int total = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (q < warp) sum += sh.warp_count[q];
    total += sh.warp_count[q];
  }
  for (int w = w0; w < w1; ++w) {
    before[w] = static_cast<uint16_t>(sum);
    sum += __popc(used[w]);
  }
  const int part = block % kCheckParts, group = block / kCheckParts, groups = blocks / kCheckParts;
  const int all_mine = (total - group + groups - 1) / groups;      // used adapters group, group + groups, ... in ascending order
  const int64_t vectors = static_cast<int64_t>(p.n) * p.r / 8, v0 = vectors * part / kCheckParts, v1 = vectors * (part + 1) / kCheckParts;
  for (int first = 0; first < all_mine; first += 256) {
    const int mine = min(256, all_mine - first);
    if (t < 8) sh.bad[t] = 0;
    __syncthreads();
    for (int w = warp; w < words; w += 8) {
      const uint32_t bits = used[w];
      if (!(bits >> lane & 1u)) continue;
      const int at = before[w] + __popc(bits & ((1u << lane) - 1u)), place = at / groups - first;
      if (at % groups == group && place >= 0 && place < 256) sh.mine[place] = static_cast<uint16_t>(32 * w + lane);
    }
    __syncthreads();
    for (int j = 0; j < mine; ++j) {
      const int64_t base = sh.mine[j] * vectors;
      const uint4* src = reinterpret_cast<const uint4*>(p.l1) + base;
      uint32_t above = 0;
      for (int64_t i = v0; i < v1; i += kDepth * 256) {
        uint4 v[kDepth];
#pragma unroll
        for (int q = 0; q < kDepth; ++q) {
          const int64_t at_v = min(i + q * 256 + t, v1 - 1);     // beyond the end: the last vector again
          v[q] = make_uint4(0u, 0u, 0u, 0u);
          if (index_ok(base + at_v, static_cast<uint64_t>(p.adapters) * vectors, p.status)) v[q] = __ldg(src + at_v);
        }
#pragma unroll
        for (int q = 0; q < kDepth; ++q) {
          above |= ((v[q].x & 0x7fff7fffu) + kAbove) | ((v[q].y & 0x7fff7fffu) + kAbove) | ((v[q].z & 0x7fff7fffu) + kAbove) |
                   ((v[q].w & 0x7fff7fffu) + kAbove);
        }
      }
      if (above & 0x80008000u) atomicOr(&sh.bad[j >> 5], 1u << (j & 31));
    }
    __syncthreads();
    if (t < mine) {
      const int64_t o = static_cast<int64_t>(sh.mine[t]) * kCheckParts + part;
      if (index_ok(o, static_cast<uint64_t>(p.adapters) * kCheckParts, p.status))
        p.unfit[o] = static_cast<uint8_t>(sh.bad[t >> 5] >> (t & 31) & 1u);
    }
    __syncthreads();             // the list is free again
  }
}

__global__ void __launch_bounds__(256) lora_spread_kernel(const SpreadParams p) {
  extern __shared__ __align__(16) uint8_t spread_smem_raw[];
  pdl_wait();
  pdl_launch_dependents();       // in this order: see nvfp4_gemm_kernel, whose FP4 stages run beside this kernel
  const int block = blockIdx.x, spreading = p.tiles * p.slices;
  if (block < spreading)
    spread_rows(p, *reinterpret_cast<SpreadShared*>(spread_smem_raw), block % p.tiles, block / p.tiles);
  else
    check_adapters(p, *reinterpret_cast<CheckShared*>(spread_smem_raw), block - spreading, static_cast<int>(gridDim.x) - spreading);
}

// ---- host side -----------------------------------------------------------------------------------------------------

int make_lora_map(CUtensorMap* map, const void* base, uint32_t dims_n, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (!encode) return NVFP4_ERR_CUDA;
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims_n, const_cast<void*>(base), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NVFP4_OK : NVFP4_ERR_INVALID_ARGUMENT;
}

// Rows times rank up to which lora_down_rows_kernel is taken.  Measured, us with k = 5120, that kernel against the tiles: m 128,
// r 64: 8 against 12 for rows of 2 adapters one after the other and 186 for 40 adapters row by row; m 256: 13 against 15 and
// 179; m 512: 23 against 15 and 186.  Which of the two the rows are is not known on the host.
constexpr int64_t kLdRowsWork = 32768;
// Above that, tiles that take more passes than rows times rank / kLdMixedWork go to lora_down_mixed_kernel, whose time grows with the
// rows where a pass takes 17 us for any number of them (k = 5120, 40 adapters of rank 64 row by row: m 1024, 10 passes: 60 against 166 us;
// m 2048: 111 against 169; m 4096: 212 against 174; 10 adapters, m 1024, 3 passes: 56 against 47).  Its launch, which costs 3 us where no
// tile needs it, is left out where `adapters` rules such tiles out.
constexpr int64_t kLdMixedWork = 20480;

bool lora_rank_ok(int64_t r, int64_t adapters) {
  return r > 0 && r <= kLoraMaxRank && r % 8 == 0 && adapters > 0 && adapters <= kLoraMaxAdapters;
}

constexpr int64_t kMaxRows = 65535 * int64_t(128);

// Adapters that a 256-row tile can have at most.
int64_t lora_tile_adapters(int64_t adapters, int64_t m) {
  const int64_t rows = m < 256 ? m : 256;
  return adapters < rows ? adapters : rows;
}

struct LoraLayout {
  int64_t count, list, rows, unfit, spread, bytes;
};

LoraLayout lora_layout(int64_t m, int64_t r, int64_t adapters) {
  const int64_t tiles = (m + 255) / 256, most = lora_tile_adapters(adapters, m);
  LoraLayout L;
  L.count = 0;
  L.list = (tiles * 4 + 255) / 256 * 256;
  L.rows = L.list + (tiles * most * 4 + 255) / 256 * 256;
  L.unfit = L.rows + tiles * 256 * 4;
  L.spread = L.unfit + (adapters * kCheckParts + 255) / 256 * 256;
  L.bytes = L.spread + tiles * most * 256 * r * 2;
  return L;
}

// gemm_lora_rows_kernel is taken for few rows with little low-rank work, which there runs on the CUDA cores.  Measured, us with
// n = 5120, k = 5120, on new inputs, against the GEMM with lora_spread_kernel: m 1, r 16: 7 against 13; m 48, r 16, 40 adapters: 9
// against 24; m 128, r 16, 40 adapters: 15 against 30; m 16, r 128, 8 adapters: 19 against 20; m 64, r 64: 28 against 27 (40 adapters)
// and 24 against 15 (2 adapters); at n = 16384 m 128, r 16: 29 against 42.
constexpr int64_t kGrMaxWork = 2048;             // m * r
bool gemm_lora_few_rows(int64_t m, int64_t r) { return m <= kGrMaxRows && m * r <= kGrMaxWork; }

// Packed FP4 matrix [rows, k/2], boxes of 128 bytes x box_rows, 128-byte swizzle.
int make_fp4_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int64_t k, uint32_t box_rows) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (!encode) return NVFP4_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k / 2), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(k / 2)};
  const cuuint32_t box[2] = {128, box_rows}, one[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NVFP4_OK : NVFP4_ERR_INVALID_ARGUMENT;
}

int run_gemm_rows(const uint8_t* a, const uint8_t* b, const GrParams& p, const DeviceInfo& info, cudaStream_t stream) {
  GrMaps maps;
  int st;
  if ((st = make_fp4_map(&maps.a, a, p.m, p.k, static_cast<uint32_t>(gr_columns(p.m)))) != NVFP4_OK) return st;
  if ((st = make_fp4_map(&maps.b, b, p.n, p.k, 128)) != NVFP4_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kGrThreads);
  cfg.attrs = attr;
  int packed = 0;                                // clusters that fit, 8 bits for each size
  st = kernel_setup(reinterpret_cast<const void*>(gemm_lora_rows_kernel), info.device, [&](int* v) {
    if (cudaFuncSetAttribute(gemm_lora_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) {
      cudaGetLastError();
      return static_cast<int>(NVFP4_ERR_CUDA);
    }
    uint32_t bits = 0;
    for (int s = 1; s <= kGrMaxCluster; ++s) {
      attr[0].val.clusterDim.x = static_cast<unsigned>(s);
      cfg.gridDim = dim3(static_cast<unsigned>(info.sm_count / s * s));
      cfg.dynamicSmemBytes = 227 * 1024;         // one CTA per SM for every m
      cfg.numAttrs = 1;
      int c = 0;
      if (cudaOccupancyMaxActiveClusters(&c, gemm_lora_rows_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        c = 0;
      }
      bits |= static_cast<uint32_t>(c < 255 ? c : 255) << (8 * (s - 1));
    }
    *v = static_cast<int>(bits);
    return static_cast<int>(NVFP4_OK);
  }, &packed);
  if (st != NVFP4_OK) return st;
  // the cluster size for which the busiest cluster's K stages per CTA, and two stages' time for each tile gathered from
  // several CTAs, are fewest
  const int tiles = (p.n + 127) / 128, stages = (p.k + 255) / 256;
  int best = 0, clusters = 0;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kGrMaxCluster && s <= stages; ++s) {
    const int fit = static_cast<int>((static_cast<uint32_t>(packed) >> (8 * (s - 1))) & 255u);
    if (fit <= 0) continue;
    const int64_t cost = static_cast<int64_t>((tiles + fit - 1) / fit) * ((stages + s - 1) / s + (s > 1 ? 2 : 0));
    if (cost < least) {
      least = cost;
      best = s;
      clusters = tiles < fit ? tiles : fit;
    }
  }
  if (best == 0) return NVFP4_ERR_CUDA;
  attr[0].val.clusterDim.x = static_cast<unsigned>(best);
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * best));
  cfg.dynamicSmemBytes = static_cast<size_t>(gr_smem(p.m));
  cfg.stream = stream;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, gemm_lora_rows_kernel, maps, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  return NVFP4_OK;
}

bool gemm_lora_shape_ok(int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  return m >= 0 && m <= kMaxRows && n >= 0 && n % 8 == 0 && n <= (1 << 29) && k > 0 && k % 64 == 0 && k <= (1 << 30) &&
         lora_rank_ok(r, adapters) && (m + 255) / 256 * lora_tile_adapters(adapters, m) * 256 < (int64_t(1) << 31);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_lora_down_batched(const void* x_bf16, int64_t m, int64_t k, const void* w_bf16, int64_t r, int64_t adapters,
                            const int32_t* adapter, void* d_bf16, nvfp4_stream_t stream) {
  if (m < 0 || m > kMaxRows || k <= 0 || k % 64 != 0 || k > (1 << 30) || !lora_rank_ok(r, adapters)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (m == 0) return NVFP4_OK;
  if (!x_bf16 || !w_bf16 || !adapter || !d_bf16 || !aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(adapter, 4) ||
      !aligned(d_bf16, 16))
    return NVFP4_ERR_INVALID_ARGUMENT;
  DeviceInfo info;
  int st = current_device(&info);
  if (st != NVFP4_OK) return st;
  LoraDownParams p;
  p.adapter = adapter;
  p.d = static_cast<__nv_bfloat16*>(d_bf16);
  p.status = info.status;
  p.m = static_cast<int32_t>(m);
  p.k = static_cast<int32_t>(k);
  p.r = static_cast<int32_t>(r);
  p.adapters = static_cast<int32_t>(adapters);
  p.max_passes = INT32_MAX;
  const uint16_t* x16 = static_cast<const uint16_t*>(x_bf16);
  const uint16_t* w16 = static_cast<const uint16_t*>(w_bf16);
  if (m * r <= kLdRowsWork)
    return launch_kernel(lora_down_rows_kernel, dim3(static_cast<unsigned>(m), static_cast<unsigned>(r / 8)), dim3(256), 0, stream,
                         x16, w16, p);
  LdMaps maps;
  memset(&maps, 0, sizeof(maps));
  const cuuint64_t xd[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(m)}, xs[1] = {static_cast<cuuint64_t>(k * 2)};
  const cuuint32_t xb[2] = {64, 128};
  if ((st = make_lora_map(&maps.x, x_bf16, 2, xd, xs, xb)) != NVFP4_OK) return st;
  const cuuint64_t wd[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(r), static_cast<cuuint64_t>(adapters)};
  const cuuint64_t wst[2] = {static_cast<cuuint64_t>(k * 2), static_cast<cuuint64_t>(k * r * 2)};
  const cuuint32_t wb[3] = {64, static_cast<cuuint32_t>((r + 15) / 16 * 16), 1};
  if ((st = make_lora_map(&maps.w, w_bf16, 3, wd, wst, wb)) != NVFP4_OK) return st;
  int ready = 0;
  st = kernel_setup(reinterpret_cast<const void*>(lora_down_tiles_kernel), info.device, [&](int* v) {
    if (cudaFuncSetAttribute(lora_down_tiles_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLdSmem) != cudaSuccess) {
      cudaGetLastError();
      return static_cast<int>(NVFP4_ERR_CUDA);
    }
    *v = 1;
    return static_cast<int>(NVFP4_OK);
  }, &ready);
  if (st != NVFP4_OK) return st;
  const int64_t tiles = (m + 127) / 128, passes = m * r / kLdMixedWork > 1 ? m * r / kLdMixedWork : 1;
  const bool mixed = ld_passes(p.r, static_cast<int>(adapters < 128 ? adapters : 128)) > passes;
  if (mixed) p.max_passes = static_cast<int32_t>(passes);
  st = launch_kernel(lora_down_tiles_kernel, dim3(kLdSplit, static_cast<unsigned>(tiles)), dim3(kLdThreads), kLdSmem, stream, maps, p);
  if (st != NVFP4_OK || !mixed) return st;
  const int64_t want = (8 * info.sm_count + tiles - 1) / tiles;      // about eight CTAs per SM over all tiles
  const unsigned slices = static_cast<unsigned>(want < 128 * (r / 8) ? want : 128 * (r / 8));
  return launch_kernel(lora_down_mixed_kernel, dim3(static_cast<unsigned>(tiles), slices), dim3(256), 0, stream, x16, w16, p);
}

int64_t nvfp4_gemm_lora_batched_workspace(int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  if (!gemm_lora_shape_ok(m, n, k, r, adapters)) return -1;
  return gemm_lora_few_rows(m, r) ? 0 : lora_layout(m, r, adapters).bytes;
}

int nvfp4_gemm_lora_batched(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf, const float* alpha,
                            const void* d_bf16, const void* l1_bf16, int64_t r, int64_t adapters, const int32_t* adapter,
                            const void* bias_bf16, void* out_bf16, void* workspace, int64_t workspace_bytes, int64_t m, int64_t n,
                            int64_t k, nvfp4_stream_t stream) {
  if (!gemm_lora_shape_ok(m, n, k, r, adapters)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (m == 0 || n == 0) return NVFP4_OK;
  const bool few = gemm_lora_few_rows(m, r);
  if (!few && !workspace) return NVFP4_ERR_INVALID_ARGUMENT;
  const void* required[] = {a, b, a_sf, b_sf, d_bf16, l1_bf16, out_bf16, few ? a : workspace};
  for (const void* q : required)
    if (!q || !aligned(q, 16)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (!alpha || !aligned(alpha, 4) || !adapter || !aligned(adapter, 4) || (bias_bf16 && !aligned(bias_bf16, 16)))
    return NVFP4_ERR_INVALID_ARGUMENT;
  const LoraLayout L = lora_layout(m, r, adapters);
  if (!few && workspace_bytes < L.bytes) return NVFP4_ERR_INVALID_ARGUMENT;
  const int64_t tiles = (m + 255) / 256, most = lora_tile_adapters(adapters, m);
  DeviceInfo info;
  int st = current_device(&info);
  if (st != NVFP4_OK) return st;
  if (few) {
    GrParams g;
    g.a_sf = a_sf;
    g.b_sf = b_sf;
    g.alpha = alpha;
    g.d = static_cast<const uint16_t*>(d_bf16);
    g.l1 = static_cast<const uint16_t*>(l1_bf16);
    g.bias = static_cast<const uint16_t*>(bias_bf16);
    g.adapter = adapter;
    g.out = static_cast<__nv_bfloat16*>(out_bf16);
    g.status = info.status;
    g.m = static_cast<int32_t>(m);
    g.n = static_cast<int32_t>(n);
    g.k = static_cast<int32_t>(k);
    g.r = static_cast<int32_t>(r);
    g.adapters = static_cast<int32_t>(adapters);
    return run_gemm_rows(a, b, g, info, stream);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SpreadParams p;
  p.d = static_cast<const uint16_t*>(d_bf16);
  p.adapter = adapter;
  p.alpha = alpha;
  p.count = reinterpret_cast<int32_t*>(ws + L.count);
  p.list = reinterpret_cast<int32_t*>(ws + L.list);
  p.l1 = static_cast<const uint16_t*>(l1_bf16);
  p.rows = reinterpret_cast<int32_t*>(ws + L.rows);
  p.unfit = ws + L.unfit;
  p.spread = reinterpret_cast<uint16_t*>(ws + L.spread);
  p.status = info.status;
  p.m = static_cast<int32_t>(m);
  p.r = static_cast<int32_t>(r);
  p.adapters = static_cast<int32_t>(adapters);
  p.max = static_cast<int32_t>(most);
  p.n = static_cast<int32_t>(n);
  // CTAs that spread: about one for three SMs over all tiles.  With two per SM, those left without an adapter delayed the GEMM's CTAs
  // (2011x8192x5120 r32: 46.8 us against 45.0).
  const int64_t want = (info.sm_count / 3 + tiles - 1) / tiles;
  p.tiles = static_cast<int32_t>(tiles);
  p.slices = static_cast<int32_t>(want < 1 ? 1 : (want < most ? want : most));
  // CTAs that check l1: up to two per SM, or four where there may be more than 64 MB of it.  2048x8192x128 r128, 48 adapters (101 MB):
  // 62.7 us with four, 77.7 with two; 256x8192x5120 r16, 48 adapters (13 MB): 38.7 and 36.0; one: 102 and 35.8, but 64x5120x5120
  // r64, 40 adapters (26 MB) 29.7 against 27.2 with two.
  const int64_t used = adapters < m ? adapters : m, most_checks = info.sm_count * (used * n * r * 2 > (int64_t(64) << 20) ? 4 : 2);
  const int64_t groups = most_checks / kCheckParts < 1 ? 1 : most_checks / kCheckParts;
  const int64_t checks = kCheckParts * (used < groups ? used : groups);
  if ((st = launch_kernel(lora_spread_kernel, dim3(static_cast<unsigned>(tiles * p.slices + checks)), dim3(256),
                          static_cast<size_t>(spread_smem(adapters)), stream, p)) != NVFP4_OK)
    return st;
  return gemm_batched_lowrank(a, b, a_sf, b_sf, alpha, p.spread, p.count, p.list, most, p.rows, p.unfit, d_bf16, l1_bf16, adapters, r,
                              bias_bf16, out_bf16, m, n, k, stream);
}

}  // extern "C"
