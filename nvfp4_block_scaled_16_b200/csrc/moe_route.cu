// moe_route.cu -- the router of a mixture-of-experts layer.
//
//   nvfp4_moe_route   ids, weights = the topk largest logits of every token and their softmax or sigmoid
//
// The chosen ids depend on comparisons of the logits alone, so they are exact; the weights are fp32.  This entry point is the
// library's own: the pages' masked batches begin after the routing.
#include "common.cuh"

namespace nvfp4 {
namespace {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;                // a lane of the token's warp keeps each choice

// ---- the router --------------------------------------------------------------------------------------

// A decode step's call is a launch, one load and topk dependent rounds (32 tokens of 128 fp32 logits, topk 8: 2.8 us); many tokens
// are bound by the issue of those rounds, not by memory (8192 tokens of 256 bf16 logits, topk 8, 4.7 MB: 9.4 us).
// One warp a token; a lane holds kPer consecutive logits as order-preserving keys (0: masked).
// topk times the warp takes the largest key (one redux), the lowest lane that holds it and that lane's first such
// logit, so equal logits go to the lowest index.
template <int kPer, typename T>
__global__ void __launch_bounds__(256) moe_route_kernel(const T* logits, int t, int experts, int topk, int weighting,
                                                        int32_t* ids, float* weights, int* status) {
  const int token = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  if (token >= t) return;
  uint32_t key[kPer];
  const int64_t row = static_cast<int64_t>(token) * experts;
  // 16 bytes a load where every row begins on such a boundary and no group of that size reaches beyond it (32 tokens of 128 fp32
  // logits, before the sort below: 3.3 us against 3.5 one by one)
  constexpr int kGroup = 16 / sizeof(T);
  constexpr bool kGroups = kPer % kGroup == 0;
  const bool wide = kGroups && experts % kGroup == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  T v[kPer] = {};
  if (wide) {
    if constexpr (kGroups) {
#pragma unroll
      for (int j = 0; j < kPer; j += kGroup) {
        const int e = lane * kPer + j;
        if (e < experts && index_ok(row + e + kGroup - 1, static_cast<uint64_t>(t) * experts, status)) {
          const uint4 raw = __ldg(reinterpret_cast<const uint4*>(logits + row + e));
          memcpy(v + j, &raw, 16);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane * kPer + j;
      if (e < experts && index_ok(row + e, static_cast<uint64_t>(t) * experts, status)) v[j] = logits[row + e];
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    float x = __uint_as_float(0xff800000u);
    if (lane * kPer + j < experts) {
      if constexpr (sizeof(T) == 2) x = __uint_as_float(static_cast<uint32_t>(v[j]) << 16);
      else x = v[j];
    }
    const uint32_t b = __float_as_uint(fminf(x, 3.402823466e38f) + 0.0f);     // -0 equals 0; +inf counts as FLT_MAX
    key[j] = x > __uint_as_float(0xff800000u) ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;   // NaN: masked
  }
  auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k); };
  // Up to 8 logits a lane sorts them once (by adjacent exchanges, so that equal ones keep their order) and then takes from the
  // front; more are looked through again after each choice, which with 8 took 10.3 us where sorting takes 9.4 (8192 tokens) and with 4 3.3
  // against 2.8 (32 tokens).  Sorting 16 would cost about 500 instructions, what topk 8 saves.
  constexpr bool kSorted = kPer <= 8;
  int index[kSorted ? kPer : 1];
  if constexpr (kSorted) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) index[j] = j;
#pragma unroll
    for (int pass = 0; pass < kPer; ++pass) {
#pragma unroll
      for (int j = pass & 1; j + 1 < kPer; j += 2) {
        const bool swap = key[j] < key[j + 1];
        const uint32_t k0 = key[j];
        const int i0 = index[j];
        key[j] = swap ? key[j + 1] : k0, index[j] = swap ? index[j + 1] : i0;
        key[j + 1] = swap ? k0 : key[j + 1], index[j + 1] = swap ? i0 : index[j + 1];
      }
    }
  }
  uint32_t best = 0;
  int at = 0;
  auto look = [&]() {
    best = key[0];
    at = 0;
    if constexpr (kSorted) {
      at = index[0];
    } else {
#pragma unroll
      for (int j = 1; j < kPer; ++j)
        if (key[j] > best) best = key[j], at = j;
    }
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
      if constexpr (kSorted) {
#pragma unroll
        for (int j = 0; j + 1 < kPer; ++j) key[j] = key[j + 1], index[j] = index[j + 1];
        key[kPer - 1] = 0;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j == at) key[j] = 0;
      }
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

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_moe_route(const void* logits, int logits_bf16, int64_t t, int64_t E, int64_t topk, int weighting, int32_t* ids_out,
                    float* weights_out, nvfp4_stream_t stream) {
  if (t < 0 || t > (1 << 28) || E <= 0 || E > kRouteMaxExperts || topk <= 0 || topk > kRouteMaxTopk || topk > E || weighting < 0 || weighting > 2)
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

}  // extern "C"
