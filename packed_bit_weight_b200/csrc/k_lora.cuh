// k_lora.cuh -- low-rank adapters of many requests beside a shared projection:
// y[i] = fp16(base[i] + s_a B_a (A_a x[i])) for the adapter a of row i, A_a
// [rank][k] and B_a [n][rank] ("1bit.gg zyphra": the graph form base +
// B*(A*x)).
#pragma once
#include "k_rows.cuh"

namespace qmm {

constexpr int kLoraMaxRank = 256;

struct LoraArgs {
  const uint16_t* a;       // [L] stacks of [R][k], a_stride bytes apart
  const uint16_t* b;       // [L] stacks of [n][R], b_stride bytes apart
  const float* scales;     // [L]
  const int32_t* ranks;    // [L] rows of A (columns of B) in use, or null: all R
  int64_t a_stride, b_stride;
  int L, R, n, k, m;
  const int32_t* ids;      // [m]
  const uint16_t* x;
  const uint16_t* base;    // [m][n]; may be y
  uint16_t* y;
  float* h;                // workspace [m][R]
};

// Rank in use of adapter a (bad values are reported and clamped).
__device__ __forceinline__ int lora_rank(const LoraArgs& p, int a) {
  if (!p.ranks) return p.R;
  const int r = p.ranks[a];
  const int c = min(max(r, 0), p.R);
  if (c != r) raise_error(ERR_BAD_EXPERT);
  return c;
}

// One warp per (row, rank index): h[i][r] = sum_k A_a[r][k] x[i][k] in fp32.
__global__ void __launch_bounds__(256) lora_shrink_simple_kernel(const LoraArgs p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t i = w / p.R;
  const int r = (int)(w - i * p.R);
  if (i >= p.m) return;
  const int a = p.ids[i];
  if (a < 0 || a >= p.L) {
    if (a != -1) raise_error(ERR_BAD_EXPERT);
    return;
  }
  float s = 0.f;
  if (r < lora_rank(p, a)) {
    const uint4* ap = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p.a) + a * p.a_stride) +
                      (int64_t)r * (p.k / 8);
    const uint4* xp = reinterpret_cast<const uint4*>(p.x) + i * (p.k / 8);
    for (int j = lane; j < p.k / 8; j += 32) {
      const uint4 u = ap[j], v = xp[j];
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const float2 f = f16x2_to_f32x2(uw[q]), g = f16x2_to_f32x2(vw[q]);
        s = fmaf(f.x, g.x, s);
        s = fmaf(f.y, g.y, s);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  }
  if (lane == 0) p.h[i * p.R + r] = s;
}

// One thread per output.
__global__ void __launch_bounds__(256) lora_expand_simple_kernel(const LoraArgs p) {
  pdl_enter();
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t i = q / p.n;
  const int c = (int)(q - i * p.n);
  if (i >= p.m) return;
  const int a = p.ids[i];
  if (a < 0 || a >= p.L) {
    p.y[q] = p.base[q];
    return;
  }
  const int rank = lora_rank(p, a);
  const uint16_t* bp = reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(p.b) + a * p.b_stride) +
                       (int64_t)c * p.R;
  float s = 0.f;
  for (int r = 0; r < rank; r++) s = fmaf(p.h[i * p.R + r], __half2float(__ushort_as_half(bp[r])), s);
  p.y[q] = f32_to_f16_bits(fmaf(p.scales[a], s, __half2float(__ushort_as_half(p.base[q]))));
}

}  // namespace qmm
