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
//   lora_down_rows_kernel    the same for few rows, where reading the adapters is the whole time: one CTA per row and 8 of
//                            its rank's values, so that rows x ranks spread over the GPU.
//   lora_spread_kernel       for each 256-row output tile the list of its adapters and, per adapter, d / alpha with other
//                            adapters' rows zeroed; the GEMM adds one bf16 MMA per listed adapter to its FP4
//                            accumulator (gemm.cu) and out is written once.
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
struct AdapterList {
  int32_t id[kRows];            // adapter of the row (-1: none)
  int32_t list[kRows];          // distinct adapters in order of their first row
  int32_t at[kRows];            // the row's place in list (-1: none)
  int32_t warp_count[kRows / 32];
  int32_t count;
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
    const int id = a.id[t];
    for (int j = 0; j < kRows; ++j)
      if (j < same && a.id[j] == id) same = j;       // the first row of this adapter
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
      a.list[place] = a.id[t];
      a.at[t] = place;
    }
    if (t == kRows - 1) a.count = base + __popc(firsts);
  }
  __syncthreads();
  if (t < kRows && !first) a.at[t] = a.id[t] < 0 ? -1 : a.at[same];
  __syncthreads();
}

// ---- lora down, tiles of 128 rows -------------------------------------------------------------------------

constexpr int kLdSplit = 4;
constexpr int kLdStages = 4;
constexpr int kLdXBytes = 128 * 128;                 // 128 rows x 64 bf16
constexpr int kLdColumns = 256;                      // accumulator columns: adapters of a pass x rank
constexpr int kLdStageBytes = kLdXBytes + kLdColumns * 128;
constexpr int kLdThreads = 192;                      // producer, MMA issuer, four drain warps

struct __align__(8) LdControl {
  uint64_t full[kLdStages], empty[kLdStages], acc_full;
  uint32_t tmem_base;
  int32_t abort;
  AdapterList<128> rows;
};
constexpr int kLdSmem = kLdStages * kLdStageBytes + static_cast<int>(sizeof(LdControl)) + 1024;
static_assert(kLdSmem <= 227 * 1024, "shared memory layout exceeds the per-block limit");
static_assert(128 * kLoraMaxRank * 4 <= kLdStages * kLdStageBytes, "the partial sums reuse the ring");

struct LdMaps {
  CUtensorMap x, w;
};

struct LoraDownParams {
  const int32_t* adapter;
  __nv_bfloat16* d;
  int* status;
  int32_t m, k, r, adapters;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __cluster_dims__(kLdSplit, 1, 1) __launch_bounds__(kLdThreads, 1)
    lora_down_tiles_kernel(const __grid_constant__ LdMaps maps, const LoraDownParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LdControl& ctl = *reinterpret_cast<LdControl*>(smem + kLdStages * kLdStageBytes);
  volatile int32_t* abort = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int row0 = blockIdx.y * 128;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kLdStages; ++s) {
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
  pdl_launch_dependents();
  pdl_wait();
  list_adapters(ctl.rows, p.adapter, row0, p.m, p.adapters, p.status);

  const int chunks = p.k / 64;
  const int nch = (chunks - rank + kLdSplit - 1) / kLdSplit;     // this CTA's chunks: rank, rank + 4, ...
  const int cols = (p.r + 15) / 16 * 16;                         // accumulator columns of an adapter
  const int per = kLdColumns / cols;                             // adapters of a pass
  const int passes = (ctl.rows.count + per - 1) / per;
  float* partial = reinterpret_cast<float*>(smem);
  uint32_t it = 0;                                               // stages so far, over all passes
  for (int pass = 0; pass < passes; ++pass) {
    const int first = pass * per, here = min(per, ctl.rows.count - first);
    if (warp == 0) {
      uint32_t i = it;
      for (int c = 0; c < nch; ++c, ++i) {
        const uint32_t s = i % kLdStages;
        if (i >= kLdStages && !mbar_wait_fast(&ctl.empty[s], (i / kLdStages - 1) & 1u, abort, p.status)) break;
        if (elect_one()) {
          uint8_t* st = smem + s * kLdStageBytes;
          const int k0 = (rank + c * kLdSplit) * 64;
          mbar_arrive_expect_tx(&ctl.full[s], static_cast<uint32_t>(kLdXBytes + here * cols * 128));
          tma_load_2d_cta(st, &maps.x, &ctl.full[s], k0, row0);
          for (int j = 0; j < here; ++j)
            tma_load_3d_cta(st + kLdXBytes + j * cols * 128, &maps.w, &ctl.full[s], k0, 0, ctl.rows.list[first + j]);
        }
        __syncwarp();
      }
    } else if (warp == 1) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(cols >> 3) << 17) | ((128u >> 4) << 24);
      uint32_t i = it;
      bool ok = true;
      for (int c = 0; c < nch; ++c, ++i) {
        const uint32_t s = i % kLdStages;
        if (!(ok = mbar_wait_fast(&ctl.full[s], (i / kLdStages) & 1u, abort, p.status))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t st = smem_u32(smem) + s * kLdStageBytes;
          const uint64_t a0 = operand_desc(st);
          for (int j = 0; j < here; ++j) {
            const uint64_t b0 = operand_desc(st + kLdXBytes + j * cols * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_bf16_cta(tmem + j * cols, a0 + 2 * q, b0 + 2 * q, idesc, c > 0 || q > 0);
          }
          mma_commit_cta(&ctl.empty[s]);
        }
        __syncwarp();
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
    it += nch;
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

// One CTA per (row, 8 rank values): the warps share K, a lane multiplies 8 values of x with 8 rows of w.
__global__ void __launch_bounds__(256) lora_down_rows_kernel(const uint16_t* x, const uint16_t* w, const LoraDownParams p) {
  __shared__ float part[8][8];
  const int row = blockIdx.x, c0 = blockIdx.y * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  int id = index_ok(row, p.m, p.status) ? p.adapter[row] : -1;
  if (id >= p.adapters) id = -1;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
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
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t ws[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[j] = fmaf(bf16_lo(xs[e]), bf16_lo(ws[e]), acc[j]);
          acc[j] = fmaf(bf16_hi(xs[e]), bf16_hi(ws[e]), acc[j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (lane == 0) part[warp][j] = acc[j];
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

// ---- the GEMM's low-rank operand ---------------------------------------------------------------------------------

struct SpreadParams {
  const uint16_t* d;            // [m, r]
  const int32_t* adapter;
  const float* alpha;
  int32_t *count, *list;
  uint16_t* spread;             // [tiles][max][256][r]
  int* status;
  int32_t m, r, adapters, max;
};

// d / alpha is rounded to bf16 once more (relative 2^-9 of the low-rank term): the MMA adds it to the FP4 accumulator, which the
// epilogue multiplies by alpha.
__global__ void __launch_bounds__(256) lora_spread_kernel(const SpreadParams p) {
  __shared__ AdapterList<256> rows;
  const int tile = blockIdx.x, row0 = tile * 256;
  pdl_launch_dependents();
  pdl_wait();
  list_adapters(rows, p.adapter, row0, p.m, p.adapters, p.status);
  if (blockIdx.y == 0) {
    if (threadIdx.x == 0 && index_ok(tile, gridDim.x, p.status)) p.count[tile] = rows.count;
    for (int j = threadIdx.x; j < rows.count; j += 256)
      if (index_ok(j, p.max, p.status)) p.list[static_cast<int64_t>(tile) * p.max + j] = rows.list[j];
  }
  const float inv = __fdiv_rn(1.0f, *p.alpha);
  const int words = p.r / 8, valid = min(256, p.m - row0);
  for (int j = blockIdx.y; j < rows.count; j += gridDim.y) {
    uint16_t* dst = p.spread + (static_cast<int64_t>(tile) * p.max + j) * 256 * p.r;
    for (int i = threadIdx.x; i < valid * words; i += 256) {
      const int row = i / words, c = (i - row * words) * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      const int64_t src = static_cast<int64_t>(row0 + row) * p.r + c;
      if (rows.at[row] == j && index_ok(src + 7, static_cast<uint64_t>(p.m) * p.r, p.status)) {
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p.d + src));
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(bf16_lo(w[e]) * inv, bf16_hi(w[e]) * inv);
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (index_ok((static_cast<uint64_t>(tile) * p.max + j) * 256 * p.r + row * p.r + c + 7,
                   static_cast<uint64_t>(gridDim.x) * p.max * 256 * p.r, p.status))
        *reinterpret_cast<uint4*>(dst + row * p.r + c) = v;
    }
  }
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
  int64_t count, list, spread, bytes;
};

LoraLayout lora_layout(int64_t m, int64_t r, int64_t adapters) {
  const int64_t tiles = (m + 255) / 256, most = lora_tile_adapters(adapters, m);
  LoraLayout L;
  L.count = 0;
  L.list = (tiles * 4 + 255) / 256 * 256;
  L.spread = L.list + (tiles * most * 4 + 255) / 256 * 256;
  L.bytes = L.spread + tiles * most * 256 * r * 2;
  return L;
}

bool gemm_lora_shape_ok(int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  return m >= 0 && m <= kMaxRows && n >= 0 && n % 8 == 0 && n <= (1 << 29) && k > 0 && k % 64 == 0 && k <= (1 << 30) &&
         lora_rank_ok(r, adapters);
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
  if (m <= 128)
    return launch_kernel(lora_down_rows_kernel, dim3(static_cast<unsigned>(m), static_cast<unsigned>(r / 8)), dim3(256), 0, stream,
                         static_cast<const uint16_t*>(x_bf16), static_cast<const uint16_t*>(w_bf16), p);
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
  return launch_kernel(lora_down_tiles_kernel, dim3(kLdSplit, static_cast<unsigned>((m + 127) / 128)), dim3(kLdThreads), kLdSmem,
                       stream, maps, p);
}

int64_t nvfp4_gemm_lora_batched_workspace(int64_t m, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  if (!gemm_lora_shape_ok(m, n, k, r, adapters)) return -1;
  return lora_layout(m, r, adapters).bytes;
}

int nvfp4_gemm_lora_batched(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf, const float* alpha,
                            const void* d_bf16, const void* l1_bf16, int64_t r, int64_t adapters, const int32_t* adapter,
                            const void* bias_bf16, void* out_bf16, void* workspace, int64_t workspace_bytes, int64_t m, int64_t n,
                            int64_t k, nvfp4_stream_t stream) {
  if (!gemm_lora_shape_ok(m, n, k, r, adapters)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (m == 0 || n == 0) return NVFP4_OK;
  const void* required[] = {a, b, a_sf, b_sf, d_bf16, l1_bf16, out_bf16, workspace};
  for (const void* q : required)
    if (!q || !aligned(q, 16)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (!alpha || !aligned(alpha, 4) || !adapter || !aligned(adapter, 4) || (bias_bf16 && !aligned(bias_bf16, 16)))
    return NVFP4_ERR_INVALID_ARGUMENT;
  const LoraLayout L = lora_layout(m, r, adapters);
  if (workspace_bytes < L.bytes) return NVFP4_ERR_INVALID_ARGUMENT;
  const int64_t tiles = (m + 255) / 256, most = lora_tile_adapters(adapters, m);
  if (tiles * most * 256 >= (int64_t(1) << 31)) return NVFP4_ERR_INVALID_ARGUMENT;
  DeviceInfo info;
  int st = current_device(&info);
  if (st != NVFP4_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SpreadParams p;
  p.d = static_cast<const uint16_t*>(d_bf16);
  p.adapter = adapter;
  p.alpha = alpha;
  p.count = reinterpret_cast<int32_t*>(ws + L.count);
  p.list = reinterpret_cast<int32_t*>(ws + L.list);
  p.spread = reinterpret_cast<uint16_t*>(ws + L.spread);
  p.status = info.status;
  p.m = static_cast<int32_t>(m);
  p.r = static_cast<int32_t>(r);
  p.adapters = static_cast<int32_t>(adapters);
  p.max = static_cast<int32_t>(most);
  const int64_t want = (2 * info.sm_count + tiles - 1) / tiles;      // about two CTAs per SM over all tiles
  const unsigned slices = static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most));
  if ((st = launch_kernel(lora_spread_kernel, dim3(static_cast<unsigned>(tiles), slices), dim3(256), 0, stream, p)) != NVFP4_OK)
    return st;
  return gemm_batched_lowrank(a, b, a_sf, b_sf, alpha, p.spread, p.count, p.list, most, l1_bf16, adapters, r, bias_bf16, out_bf16,
                              m, n, k, stream);
}

}  // extern "C"
