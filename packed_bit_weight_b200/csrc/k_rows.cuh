// k_rows.cuh -- rows grouped by an index: the stable sort of (token, slot)
// pairs by expert with its inverse, the token rows laid out in that order,
// the rows brought back with their routing weights, and the gradients of both
// ("Mark-Experimental-V3-8B", section "Mixture-of-Experts (MoE)": top-4 of 32
// experts per token, y = ... + sum_i g_i F_i(x)).
//
// All of it moves bytes: the bound is HBM (or L2, for a window that fits it)
// for long inputs and the launch for short ones.
#pragma once
#include "qmm_dev.cuh"

namespace qmm {

constexpr int kRowsMaxBins = 1024;   // experts (or adapters) of one sort, one more for rows without
constexpr int kRowsSortWarps = 16;   // warps per CTA of the sort
constexpr int kRowsSortThreads = kRowsSortWarps * 32;

// Rows [start, end) of group g when the caller supplies the offsets: clamped
// into the P rows there are, so that bad offsets are reported, not followed.
__device__ __forceinline__ int group_range(const int32_t* __restrict__ offsets, int g, int P, int& start) {
  const int a = offsets[g], b = offsets[g + 1];
  const int ca = min(max(a, 0), P), cb = min(max(b, ca), P);
  if (ca != a || cb != b) raise_error(ERR_BAD_EXPERT);
  start = ca;
  return cb - ca;
}

// SiLU(z) = z / (1 + e^-z) by the fast exponential and division, in both
// kernels of the SwiGLU product over sorted rows: off by 2 + 1.2 |z| and 2 fp32
// steps, far below half an fp16 step of the result it is rounded to (|z| of 80,
// where that is 2^-16 of the value, gives 0 in fp16).  (With the copies and the
// decode left out, gate and up of 8,192 pairs took 147 us with expf and the IEEE
// division, one epilogue warp per scheduler, and 78 us with these.)
__device__ __forceinline__ float silu_fast(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

__device__ __forceinline__ int ld_dsmem_s32(const int* local, uint32_t r) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(r));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// Stable counting sort of pair indices by ids[p], with its inverse.
//
// One thread-block cluster (1 to 8 CTAs) does the whole sort, so it is one
// launch and needs no workspace.  Every warp of the cluster owns one
// contiguous run of pairs, which makes the order stable: it counts its ids
// (lanes of equal id find each other with warp votes, so no atomics), the
// CTA scans its warps' counts, the CTAs exchange their totals through
// distributed shared memory, and a second walk over the same run writes each
// pair's place.  ids outside [0, E) take no place; -1 says so on purpose
// (padding, a request without an adapter), anything else raises the error.
// With `rest` they are kept instead, as the last bin E - 1.
//
// RowTiles: the groups cut into tiles of at most T rows (equal ones of whole
// 16-row steps), listed in group order, for kernels that give each tile a CTA.
// ---------------------------------------------------------------------------
// The lanes that hold the same valid id: one vote per bit of the ids (a match
// over the warp costs a round per distinct id: the sort of 65,536 pairs over
// 128 experts took 22 us with it, so 16).
__device__ __forceinline__ unsigned same_id(int e, bool valid, int bits) {
  unsigned m = __ballot_sync(0xFFFFFFFFu, valid);
  for (int b = 0; b < bits; b++) {
    const bool on = (e >> b) & 1;
    const unsigned v = __ballot_sync(0xFFFFFFFFu, on);
    m &= on ? v : ~v;
  }
  return m;
}

struct RowTile {  // rows perm[start] .. perm[start + count - 1] of group g
  int g, start, count, pad;
};
struct RowTiles {
  RowTile* list;   // null: none wanted
  int32_t* num;
  int T;
  int skip_last;   // the last bin gets no tiles
};

__host__ __device__ constexpr int route_rows_smem(int E) { return (kRowsSortWarps + 3) * E * 4; }

__global__ void __launch_bounds__(kRowsSortThreads, 1)
    route_rows_kernel(const int32_t* __restrict__ ids, int P, int E, int rest, int32_t* __restrict__ offsets,
                      int32_t* __restrict__ perm, int32_t* __restrict__ row_of, const RowTiles tiles) {
  extern __shared__ int smem_rows[];
  int* cnt = smem_rows;                      // [warp][E]: counts, then the warp's next place within its expert
  int* total = cnt + kRowsSortWarps * E;     // [E] this CTA's pairs per expert (read by the other CTAs)
  int* grand = total + E;                    // [E] all pairs per expert, then their exclusive scan
  int* before = grand + E;                   // [E] pairs of earlier CTAs per expert
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_nctarank(), c = (int)cluster_ctarank();
  const unsigned lt = (1u << lane) - 1u;
  asm volatile("griddepcontrol.launch_dependents;" :::);  // (a plain launch itself: everything before it is done)
  for (int i = tid; i < kRowsSortWarps * E; i += kRowsSortThreads) cnt[i] = 0;
  __syncthreads();
  const int steps = (P + C * kRowsSortThreads - 1) / (C * kRowsSortThreads);  // 32-pair steps per warp
  const int64_t p0 = (int64_t)(c * kRowsSortWarps + warp) * steps * 32;
  int* mine = cnt + warp * E;
  const int bits = 32 - __clz(E - 1 | 1);
  bool bad = false;
  auto id_at = [&](int i) {  // this lane's id of step i (read four steps ahead of its use below)
    const int64_t p = p0 + i * 32 + lane;
    return i < steps && p < P ? ids[p] : -1;
  };
  int ahead[4];
#pragma unroll
  for (int j = 0; j < 4; j++) ahead[j] = id_at(j);
#pragma unroll 4
  for (int i = 0; i < steps; i++) {
    const int64_t p = p0 + i * 32 + lane;
    int e = ahead[i & 3];
    ahead[i & 3] = id_at(i + 4);
    bool valid = e >= 0 && e < E - rest;
    bad |= !valid && e != -1;
    if (rest && !valid && p < P) { e = E - 1; valid = true; }
    const unsigned peers = same_id(e, valid, bits);
    if (valid && (peers & lt) == 0) mine[e] += __popc(peers);
    __syncwarp();
  }
  if (bad) raise_error(ERR_BAD_EXPERT);
  __syncthreads();
  for (int e = tid; e < E; e += kRowsSortThreads) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kRowsSortWarps; w++) {
      const int v = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += v;
    }
    total[e] = run;
  }
  __syncwarp();  // (a cluster barrier is warp-wide; the lanes have walked different numbers of experts)
  cluster_sync();
  for (int e = tid; e < E; e += kRowsSortThreads) {
    int all = 0, b = 0;
    for (int r = 0; r < C; r++) {
      const int v = ld_dsmem_s32(total + e, (uint32_t)r);
      if (r == c) b = all;
      all += v;
    }
    grand[e] = all;
    before[e] = b;
  }
  __syncwarp();
  cluster_sync();  // (also: no CTA leaves while another still reads its totals)
  if (warp == 0) {  // exclusive scan over the experts, and over their tiles
    const bool want = tiles.list && c == 0;
    int run = 0, trun = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int v = e < E ? grand[e] : 0;
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      if (e < E) {
        grand[e] = run + s - v;
        if (c == 0) offsets[e] = run + s - v;
      }
      run += __shfl_sync(0xFFFFFFFFu, s, 31);
      if (want) {
        const int t = (tiles.skip_last && e == E - 1) ? 0 : (v + tiles.T - 1) / tiles.T;
        int ts = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, ts, o);
          if (lane >= o) ts += u;
        }
        const int per = t ? (((v + t - 1) / t) + 15) & ~15 : 0;
        for (int j = 0; j < t; j++) {
          RowTile tile;
          tile.g = e;
          tile.count = max(0, min(per, v - j * per));
          tile.pad = 0;
          tile.start = grand[e] + j * per;
          tiles.list[trun + ts - t + j] = tile;
        }
        trun += __shfl_sync(0xFFFFFFFFu, ts, 31);
      }
    }
    if (lane == 0 && c == 0) {
      offsets[E] = run;
      if (want) *tiles.num = trun;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; j++) ahead[j] = id_at(j);
#pragma unroll 4
  for (int i = 0; i < steps; i++) {
    const int64_t p = p0 + i * 32 + lane;
    int e = ahead[i & 3];
    ahead[i & 3] = id_at(i + 4);
    bool valid = e >= 0 && e < E - rest;
    if (rest && !valid && p < P) { e = E - 1; valid = true; }
    const unsigned peers = same_id(e, valid, bits);
    int place = -1;
    if (valid) place = grand[e] + before[e] + mine[e] + __popc(peers & lt);
    __syncwarp();
    if (valid && (peers & lt) == 0) mine[e] += __popc(peers);
    __syncwarp();
    if (valid) perm[place] = (int32_t)p;
    if (p < P && row_of) row_of[p] = place;
  }
}

// ---------------------------------------------------------------------------
// Row movement.  A row is d fp16 values = d/8 chunks of 16 bytes; a warp owns
// (token, 32 * U chunks).  Row numbers outside [0, P) (pairs without an
// expert) are skipped.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void pdl_enter() {
  // wait for the kernel before this one, and only then let the next one start:
  // a kernel that reads ahead of its own wait stays ordered behind this one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
}

// xs[row_of[t][s]] = x[t]: every token row is read once and stored topk times.
template <int U>
__global__ void __launch_bounds__(256) permute_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ row_of,
                                                      int64_t t, int topk, int d8, int segs, int P,
                                                      uint4* __restrict__ xs) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t tok = w / segs;
  if (tok >= t) return;
  const int j0 = (int)(w - tok * segs) * (32 * U) + lane;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; u++)
    if (j0 + 32 * u < d8) v[u] = x[tok * d8 + j0 + 32 * u];
  for (int s = 0; s < topk; s++) {
    const int r = row_of[tok * topk + s];
    if (r < 0 || r >= P) continue;
#pragma unroll
    for (int u = 0; u < U; u++)
      if (j0 + 32 * u < d8) xs[(int64_t)r * d8 + j0 + 32 * u] = v[u];
  }
}

__device__ __forceinline__ void fma8(float (&acc)[8], float g, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 f = f16x2_to_f32x2(w[i]);
    acc[2 * i] = fmaf(g, f.x, acc[2 * i]);
    acc[2 * i + 1] = fmaf(g, f.y, acc[2 * i + 1]);
  }
}

// out[t] = fp16(sum_s g[t][s] ys[row_of[t][s]]), fp32 in slot order; g = 1
// where gw is null (the gradient of permute).
template <int U>
__global__ void __launch_bounds__(256) unpermute_kernel(const uint4* __restrict__ ys, const int32_t* __restrict__ row_of,
                                                        const float* __restrict__ gw, int64_t t, int topk, int d8,
                                                        int segs, int P, uint4* __restrict__ out) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t tok = w / segs;
  if (tok >= t) return;
  const int j0 = (int)(w - tok * segs) * (32 * U) + lane;
  float acc[U][8];
#pragma unroll
  for (int u = 0; u < U; u++)
#pragma unroll
    for (int i = 0; i < 8; i++) acc[u][i] = 0.f;
#pragma unroll 2
  for (int s = 0; s < topk; s++) {
    const int r = row_of[tok * topk + s];
    if (r < 0 || r >= P) continue;
    const float g = gw ? gw[tok * topk + s] : 1.0f;
#pragma unroll
    for (int u = 0; u < U; u++)
      if (j0 + 32 * u < d8) fma8(acc[u], g, ys[(int64_t)r * d8 + j0 + 32 * u]);
  }
#pragma unroll
  for (int u = 0; u < U; u++)
    if (j0 + 32 * u < d8)
      out[tok * d8 + j0 + 32 * u] =
          make_uint4(f32x2_to_f16x2(acc[u][0], acc[u][1]), f32x2_to_f16x2(acc[u][2], acc[u][3]),
                     f32x2_to_f16x2(acc[u][4], acc[u][5]), f32x2_to_f16x2(acc[u][6], acc[u][7]));
}

// Gradient of unpermute, a warp per pair p = (t, s) with row r = row_of[p]:
// dys[r] = fp16(g[p] dout[t]), dg[p] = sum_j ys[r][j] dout[t][j] (lanes' fp32
// sums joined in a fixed order).  The pairs of a token are neighbouring warps,
// so dout comes from L1 after its first reader.
__global__ void __launch_bounds__(256) unpermute_backward_kernel(
    const uint4* __restrict__ dout, const uint4* __restrict__ ys, const int32_t* __restrict__ row_of,
    const float* __restrict__ gw, int64_t pairs, int topk, int d8, uint4* __restrict__ dys, float* __restrict__ dg) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t p = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (p >= pairs) return;
  const int r = row_of[p];
  if (r < 0 || r >= pairs) {
    if (lane == 0) dg[p] = 0.f;
    return;
  }
  const float g = gw ? gw[p] : 1.0f;
  const uint4* dp = dout + (p / topk) * d8;
  const uint4* yp = ys + (int64_t)r * d8;
  uint4* op = dys + (int64_t)r * d8;
  float sum = 0.f;
#pragma unroll 4
  for (int j = lane; j < d8; j += 32) {
    const uint4 a = dp[j], b = yp[j];
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 da = f16x2_to_f32x2(aw[i]), yb = f16x2_to_f32x2(bw[i]);
      o[i] = f32x2_to_f16x2(g * da.x, g * da.y);
      sum = fmaf(da.x, yb.x, sum);
      sum = fmaf(da.y, yb.y, sum);
    }
    op[j] = make_uint4(o[0], o[1], o[2], o[3]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) dg[p] = sum;
}

}  // namespace qmm
