// k_lora.cuh -- low-rank adapters of many requests beside a shared projection:
// y[i] = fp16(base[i] + s_a B_a (A_a x[i])) for the adapter a of row i, A_a
// [rank][k] and B_a [n][rank] ("1bit.gg zyphra": the graph form base +
// B*(A*x)).
//
// A few rows (decode): one launch, a thread-block cluster per row and part of
// n (lora_token_kernel).  More rows: the rows are sorted by adapter into tiles
// (the sort of k_rows.cuh), the middle products A x are taken per tile with the
// cluster's CTAs and warps sharing k (lora_shrink_kernel), and B and base are
// streamed once per tile (lora_expand_kernel; lora_expand_tc_kernel for long
// inputs).  The bound is bytes: A and B of the adapters in use, x, base and y.
// The products are small beside them (rank times two operations a value), so
// legacy MMAs keep up except at 512 rows and more of ranks above 32.
#pragma once
#include "k_ggemm.cuh"
#include "k_rows.cuh"

namespace qmm {

constexpr int kLoraMaxRank = 256;
constexpr int kLoraCluster = 8;    // CTAs that share a row; at most so many share a tile's k
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;

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
  // workspace
  int32_t* offsets;        // [L + 2]
  int32_t* perm;           // [m]
  RowTile* tiles;          // g: the adapter, L for rows without one
  int32_t* num_tiles;
  float* h;                // [m][R] in the order of perm
};

// Rank in use of adapter a (bad values are reported and clamped).
__device__ __forceinline__ int lora_rank(const LoraArgs& p, int a) {
  if (!p.ranks) return p.R;
  const int r = p.ranks[a];
  const int c = min(max(r, 0), p.R);
  if (c != r) raise_error(ERR_BAD_EXPERT);
  return c;
}

__device__ __forceinline__ const uint16_t* lora_a(const LoraArgs& p, int a) {
  return reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(p.a) + a * p.a_stride);
}
__device__ __forceinline__ const uint16_t* lora_b(const LoraArgs& p, int a) {
  return reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(p.b) + a * p.b_stride);
}

__device__ __forceinline__ float dot8(const uint4& u, const uint4& v, float s) {
  const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const float2 f = f16x2_to_f32x2(uw[q]), g = f16x2_to_f32x2(vw[q]);
    s = fmaf(f.x, g.x, s);
    s = fmaf(f.y, g.y, s);
  }
  return s;
}
__device__ __forceinline__ float dot8f(const uint4& u, const float (&h)[8], float s) {
  const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const float2 f = f16x2_to_f32x2(uw[q]);
    s = fmaf(f.x, h[2 * q], s);
    s = fmaf(f.y, h[2 * q + 1], s);
  }
  return s;
}

// Bad ids and ranks of a pool without products (rank 0 or k = 0, where y = base
// is a copy) are reported all the same.
__global__ void __launch_bounds__(256) lora_check_kernel(const LoraArgs p) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.m; i += (int64_t)gridDim.x * 256) {
    const int a = p.ids[i];
    if (a >= 0 && a < p.L) lora_rank(p, a);
    else if (a != -1) raise_error(ERR_BAD_EXPERT);
  }
}

// Elements of an 8-value piece that lie at or past `left` set to zero (what a
// rank leaves out is never used, whatever it holds).
__device__ __forceinline__ uint4 mask8(uint4 v, int left) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; q++) {
    if (2 * q >= left) w[q] = 0u;
    else if (2 * q + 1 >= left) w[q] &= 0xFFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// y[c0 .. c1) = base[c0 .. c1) (not overlapping) by `threads` threads; vec:
// both are 16-byte aligned at multiples of 8 columns, and c0 is one.
__device__ __forceinline__ void copy_span(uint16_t* __restrict__ y, const uint16_t* __restrict__ base, int c0, int c1,
                                          bool vec, int t, int threads) {
  int c = c0;
  if (vec) {
#pragma unroll 4
    for (int i = c0 + 8 * t; i + 8 <= c1; i += 8 * threads)
      *reinterpret_cast<uint4*>(y + i) = *reinterpret_cast<const uint4*>(base + i);
    c = c0 + ((c1 - c0) & ~7);
  }
#pragma unroll 4
  for (int i = c + t; i < c1; i += threads) y[i] = base[i];
}

// ---------------------------------------------------------------------------
// Decode: a cluster of 8 CTAs per (row, part of n).  CTA q multiplies R/8 rows
// of A with x (every warp an eighth of k, the partial sums joined in warp
// order), the CTAs read each other's values through distributed shared memory,
// and each goes on with its own rows of B: rank/8 lanes a row (rounded up to a
// power of two), 16 bytes each, the first of them loaded before the exchange.
// At one row all of it is latency: a launch, two dependent reads (the id, then
// A), a cluster barrier.
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kLoraCluster, 1, 1) __launch_bounds__(kLoraThreads, 2)
    lora_token_kernel(const LoraArgs p, int parts) {
  __shared__ float red[kLoraWarps][kLoraMaxRank / kLoraCluster];
  __shared__ float mine[kLoraMaxRank / kLoraCluster];
  __shared__ float h[kLoraMaxRank];
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int q = (int)cluster_ctarank();
  const int cl = blockIdx.x / kLoraCluster;
  const int i = cl / parts, part = cl - i * parts;
  const int64_t row = i;
  // this CTA's outputs
  const int slices = parts * kLoraCluster, slice = part * kLoraCluster + q;
  const int per = ((p.n + slices - 1) / slices + 7) & ~7;
  const int c0 = min(slice * per, p.n), c1 = min(c0 + per, p.n);
  const int a = p.ids[i];
  if (a < 0 || a >= p.L) {  // the whole cluster
    if (a != -1) raise_error(ERR_BAD_EXPERT);
    if (p.base != p.y)
      copy_span(p.y + row * p.n, p.base + row * p.n, c0, c1, (p.n & 7) == 0, tid, kLoraThreads);
    return;
  }
  const int rank = lora_rank(p, a);
  const float scale = p.scales[a];
  const int R = p.R, k8 = p.k >> 3;
  // expand geometry: lpr lanes per row of B, 32 / lpr rows per warp and step
  int lpr = 1;
  while (lpr * 8 < R) lpr *= 2;
  const int sub = lane & (lpr - 1), rows = 32 / lpr, r0 = sub * 8;
  const uint16_t* B = lora_b(p, a);
  constexpr int kPre = 4;  // steps loaded ahead
  uint4 pre[kPre];
  uint16_t pre_base[kPre];
  auto b_row = [&](int c) {
    return (c < c1 && r0 < rank) ? *reinterpret_cast<const uint4*>(B + (int64_t)c * R + r0)
                                 : make_uint4(0u, 0u, 0u, 0u);
  };
  const int cw = c0 + warp * rows + lane / lpr;  // this lane's first row of B
#pragma unroll
  for (int u = 0; u < kPre; u++) {
    const int c = cw + u * rows * kLoraWarps;
    pre[u] = b_row(c);
    pre_base[u] = c < c1 ? p.base[row * p.n + c] : (uint16_t)0;
  }

  // ---- h rows q Rc .. q Rc + Rc - 1 ----
  const int Rc = R / kLoraCluster;
  const uint4* xp = reinterpret_cast<const uint4*>(p.x) + row * k8;
  const uint4* A = reinterpret_cast<const uint4*>(lora_a(p, a));
  for (int b = 0; b < Rc; b += 8) {
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; j++) acc[j] = 0.f;
#pragma unroll 2
    for (int c = tid; c < k8; c += kLoraThreads) {
      const uint4 xv = xp[c];
      uint4 w[8];  // (all loads before the first use)
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int r = q * Rc + b + j;
        w[j] = (b + j < Rc && r < rank) ? A[(int64_t)r * k8 + c] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (b + j < Rc && q * Rc + b + j < rank) acc[j] = dot8(w[j], xv, acc[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (b + j >= Rc) break;
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
      if (lane == 0) red[warp][b + j] = acc[j];
    }
  }
  __syncthreads();
  if (tid < Rc) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; w++) s += red[w][tid];
    mine[tid] = s;
  }
  __syncwarp();
  cluster_sync();
  if (tid < R) h[tid] = ld_dsmem_f32(&mine[tid % Rc], (uint32_t)(tid / Rc));
  __syncwarp();
  cluster_sync();  // (no CTA leaves while another reads its values; h is complete here too)

  // ---- this CTA's rows of B ----
  float hv[8];
#pragma unroll
  for (int j = 0; j < 8; j++) hv[j] = r0 + j < R ? h[min(r0 + j, kLoraMaxRank - 1)] : 0.f;
  for (int c = cw; c - lane / lpr < c1;) {
    // the next step's pieces are loaded before this one's outputs are stored
    // (y may be base, so no load moves up past a store by itself)
    uint4 next[kPre];
    uint16_t next_base[kPre];
    const int cn = c + kPre * rows * kLoraWarps;
#pragma unroll
    for (int u = 0; u < kPre; u++) {
      const int cc = cn + u * rows * kLoraWarps;
      next[u] = b_row(cc);
      next_base[u] = cc < c1 ? p.base[row * p.n + cc] : (uint16_t)0;
    }
    float s[kPre];
#pragma unroll
    for (int u = 0; u < kPre; u++) s[u] = dot8f((rank & 7) ? mask8(pre[u], rank - r0) : pre[u], hv, 0.f);
    for (int o = lpr >> 1; o; o >>= 1)
#pragma unroll
      for (int u = 0; u < kPre; u++) s[u] += __shfl_xor_sync(0xFFFFFFFFu, s[u], o);
#pragma unroll
    for (int u = 0; u < kPre; u++) {
      const int cc = c + u * rows * kLoraWarps;
      if (sub == 0 && cc < c1)
        p.y[row * p.n + cc] = f32_to_f16_bits(fmaf(scale, s[u], __half2float(__ushort_as_half(pre_base[u]))));
      pre[u] = next[u];
      pre_base[u] = next_base[u];
    }
    c += kPre * rows * kLoraWarps;
  }
}

// ---------------------------------------------------------------------------
// Middle products of a tile: h[row][r] = sum_k A[r][k] x[row][k], fp32, 64
// ranks per CTA (blockIdx.y).  The CTAs of a cluster each take a share of k,
// in blocks of 256: the block's piece of A arrives by cp.async in one of two
// buffers (rows 576 bytes apart: the fragment reads of 8 rows hit every bank
// group once) while the block before is multiplied, x comes straight from
// global memory, each row read by one warp.  The 8 warps are mw groups of 16
// rows times 8/mw shares of the block's eight 32-wide chunks.  MMA m16n8k16
// with the rows as M and the ranks as N; the k order inside a chunk is chosen
// so that a lane's 16 bytes of a row are its fragment words.  Partial sums
// meet in shared memory, then across the cluster, each in a fixed order.
// (With A read from global memory by every warp the loads of 8 rows' lines per
// instruction took 38 us for 2,048 rows of rank 128 and k = 4096, so 26.)
// ---------------------------------------------------------------------------
constexpr int kShrinkK = 256;                       // k per block
constexpr int kShrinkRow = kShrinkK * 2 + 64;       // bytes between rows of A in a buffer
constexpr int kShrinkBuf = 64 * kShrinkRow;
constexpr int kShrinkSmem = 2 * kShrinkBuf;         // (the partial sums, 32 KB, take the first buffer's place)

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool on) {
  const uint32_t bytes = on ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__global__ void __launch_bounds__(kLoraThreads, 2) lora_shrink_kernel(const LoraArgs p) {
  extern __shared__ __align__(16) uint8_t smem_shrink[];
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane >> 2, tig = lane & 3;
  const int q = (int)cluster_ctarank(), cs = (int)cluster_nctarank(), t = blockIdx.x / cs;
  const RowTile tile = p.tiles[t];  // (the list has room for every CTA's tile)
  if (t >= *p.num_tiles) return;    // the whole cluster
  if (tile.g >= p.L || tile.count <= 0) return;
  const int rank = lora_rank(p, tile.g), R = p.R, rb = blockIdx.y * 64;
  int mw = 1;
  while (mw * 16 < tile.count) mw *= 2;
  const int kw = kLoraWarps / mw;
  const int mg = warp % mw, ks = warp / mw;
  const int blocks = (p.k + kShrinkK - 1) / kShrinkK;
  const int bl0 = blocks * q / cs, bl1 = blocks * (q + 1) / cs;
  const uint16_t* A = lora_a(p, tile.g);
  const uint32_t sm = smem_addr(smem_shrink);
  const int arow = tid >> 5, acol = tid & 31;  // 8 rows of 32 pieces per pass
  auto stage = [&](int bl) {
    const uint32_t dst = sm + (bl & 1) * kShrinkBuf + arow * kShrinkRow + acol * 16;
    const int kk = bl * kShrinkK + acol * 8;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int r = rb + arow + 8 * i;
      const bool on = r < rank && kk < p.k;  // (k % 8 == 0: a piece is inside or outside)
      cp_async16_zfill(dst + i * 8 * kShrinkRow, on ? A + (int64_t)r * p.k + kk : A, on);
    }
    cp_commit_g();
  };
  if (bl0 < bl1) stage(bl0);
  const int row0 = mg * 16 + grp, row1 = row0 + 8;
  const uint16_t* x0 = p.x + (int64_t)p.perm[tile.start + (row0 < tile.count ? row0 : 0)] * p.k;
  const uint16_t* x1 = p.x + (int64_t)p.perm[tile.start + (row1 < tile.count ? row1 : 0)] * p.k;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; j++)
#pragma unroll
    for (int c = 0; c < 4; c++) acc[j][c] = 0.f;
  for (int bl = bl0; bl < bl1; bl++) {
    if (bl + 1 < bl1) stage(bl + 1);
    else cp_commit_g();  // (an empty group keeps the count)
    uint4 u[8][2];  // this warp's chunks of the block
#pragma unroll
    for (int c = 0; c < 8; c++) {
      const int kk = bl * kShrinkK + (ks * mw + c) * 32 + tig * 8;
      const bool in = c < mw && kk < p.k;
      u[c][0] = in ? *reinterpret_cast<const uint4*>(x0 + kk) : zero;
      u[c][1] = in ? *reinterpret_cast<const uint4*>(x1 + kk) : zero;
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const uint32_t src = sm + (bl & 1) * kShrinkBuf + grp * kShrinkRow + tig * 16 + ks * mw * 64;
#pragma unroll
    for (int c = 0; c < 8; c++) {
      if (c >= mw) break;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint4 w = lds128(src + c * 64 + 8 * j * kShrinkRow);
        mma_16816(acc[j], u[c][0].x, u[c][1].x, u[c][0].y, u[c][1].y, w.x, w.y);
        mma_16816(acc[j], u[c][0].z, u[c][1].z, u[c][0].w, u[c][1].w, w.z, w.w);
      }
    }
    __syncthreads();  // the buffer may be filled again
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // partial sums [ks][row][64]
  float* sh = reinterpret_cast<float*>(smem_shrink);
  float* mine = sh + (ks * mw * 16) * 64;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int c = 8 * j + 2 * tig;
    *reinterpret_cast<float2*>(mine + row0 * 64 + c) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(mine + row1 * 64 + c) = make_float2(acc[j][2], acc[j][3]);
  }
  __syncthreads();
  const int cells = mw * 16 * 64;
  if (kw > 1)
    for (int i = tid; i < cells; i += kLoraThreads) {
      float s = sh[i];
      for (int j = 1; j < kw; j++) s += sh[j * cells + i];
      sh[i] = s;
    }
  __syncthreads();
  cluster_sync();
  // this CTA joins its share of the tile's cells
  const int width = min(64, R - rb);
  for (int i = q * kLoraThreads + tid; i < tile.count * 64; i += cs * kLoraThreads) {
    const int r = i & 63;
    if (r >= width) continue;
    float s = 0.f;
#pragma unroll 8
    for (int c = 0; c < cs; c++) s += ld_dsmem_f32(sh + i, (uint32_t)c);
    // (0 past the rank, where the staged zeros times an infinity or NaN in x are NaN)
    p.h[(int64_t)(tile.start + (i >> 6)) * R + rb + r] = rb + r < rank ? s : 0.f;
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while its partial sums are read
}

// ---------------------------------------------------------------------------
// y = base + s B h for a tile's rows and a range of columns.  MMA m16n8k16
// with the rows as M and 8 columns of y (rows of B) as N.  B goes from global
// memory into fragments (a lane's 16 bytes of a row of B, as above) and stays
// there for all of the tile's rows; a warp's four n-tiles are interleaved so
// that a lane's columns are 8 neighbours, one 16-byte piece of base and y.
//
// The middle product is held as two fp16 halves, h = 2^e (hi + 2^-12 lo): each
// row is scaled by a power of two that brings its largest finite value to
// [2^14, 2^15), hi is the rounded value and lo 2^12 times the rounded rest.  hi
// is off by half a step, 2^-12 of a value of 2^-14 and more (2^-25 below), and lo
// by 2^-12 of that rest or 2^-25, so a value of 2^-15 and more (2^-29 of the
// row's largest) keeps 22 bits, at twice the MMAs of one fp16, which the stream
// of base and y hides.  (With lo not scaled up its smallest step, 2^-24, took
// bits from 2^-18 of the largest down.)  The products of lo come first, their
// sum is multiplied by 2^-12, exactly, and the products of hi are added.  A row
// with a smaller value in it (about one in 10^6 rows of rank 128 and normal
// values) is taken by lora_row_fp32, and so is one whose scale and power of two
// together leave fp32.
// ---------------------------------------------------------------------------
// Scale of a row of h held 32 values per register across the warp: f1 f2 =
// 2^(14 - e) for the largest finite |value| in [2^e, 2^(e+1)) (two factors, so
// that neither leaves fp32), back = 2^(e - 14).
template <int N>
__device__ __forceinline__ void h_scale(const float (&v)[N], float& f1, float& f2, float& back) {
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < N; c++) {
    const float f = fabsf(v[c]);
    if (f <= 3.4028235e38f) top = fmaxf(top, f);  // (finite)
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  const int sh = top > 0.f ? min(14 - e, 126) : 0;
  f1 = __uint_as_float((uint32_t)(127 + (sh >> 1)) << 23);
  f2 = __uint_as_float((uint32_t)(127 + (sh - (sh >> 1))) << 23);
  back = __uint_as_float((uint32_t)(127 - sh) << 23);
}
// x = hi + 2^-12 lo as fp16 halves; an infinite or NaN hi has lo = 0.
constexpr int kLoraLoBits = 12;
__device__ __forceinline__ void h_split(float x, uint16_t& hi, uint16_t& lo) {
  const __half h = __float2half_rn(x);
  const float back = __half2float(h);
  hi = __half_as_ushort(h);
  lo = fabsf(back) <= 65504.f ? __half_as_ushort(__float2half_rn((x - back) * (float)(1 << kLoraLoBits))) : (uint16_t)0;
}
// A scaled value that the halves hold in fewer than 22 bits.
__device__ __forceinline__ bool h_small(float x) { return x != 0.f && fabsf(x) < 0x1p-15f; }
// scale * back, or NaN for a row that is left for lora_row_fp32, as its outputs
// then show: here one whose factor alone is infinite.
__device__ __forceinline__ float h_factor(float scale, float back) {
  const float f = scale * back;
  return fabsf(f) > 3.4028235e38f && fabsf(scale) <= 3.4028235e38f ? __uint_as_float(0x7FC00000u) : f;
}

// True if one of 8 fp16 values is an infinity or NaN (0 times it is NaN).
__device__ __forceinline__ bool nonfinite8(const uint4& v) {
  uint32_t acc;
  asm("{\n .reg .b32 t;\n mul.rn.f16x2 t, %1, %5;\n fma.rn.f16x2 t, %2, %5, t;\n fma.rn.f16x2 t, %3, %5, t;\n"
      " fma.rn.f16x2 %0, %4, %5, t;\n}"
      : "=r"(acc)
      : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(0u));
  return (acc & 0x7FFF7FFFu) != 0u;
}

// 8 columns of a row of which the first `left` exist, value by value (rows that
// do not start on 16 bytes).
__device__ __forceinline__ uint4 load8(const uint16_t* p, int left) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (i < left) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(uint16_t* p, const uint4& v, int left) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (i < left) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// Columns c0 .. c1 - 1 of one row by one warp, in fp32 alone: y[c] =
// fp16(base[c] + scale sum_r h[r] B[c][r]).  The products of two fp16 halves
// give NaN where B holds an infinity (inf * hi + inf * lo, with lo 0 or of the
// other sign), so outputs that come out infinite or NaN are not stored and are
// taken again here, and so are rows with a value that the halves hold in too few
// bits.  Rare, so it reads h and B from global memory.
__device__ __noinline__ void lora_row_fp32(uint16_t* y, const uint16_t* base, const float* h, const uint16_t* B, int R,
                                           int rank, float scale, int c0, int c1) {
  for (int c = c0 + (threadIdx.x & 31); c < c1; c += 32) {
    float s = 0.f;
    for (int r = 0; r < rank; r += 8) {
      const float4 h0 = *reinterpret_cast<const float4*>(h + r), h1 = *reinterpret_cast<const float4*>(h + r + 4);
      const float hv[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
      s = dot8f(mask8(*reinterpret_cast<const uint4*>(B + (int64_t)c * R + r), rank - r), hv, s);
    }
    y[c] = f32_to_f16_bits(fmaf(scale, s, __half2float(__ushort_as_half(base[c]))));
  }
}

// CTAs per SM: what the registers of B's fragments (16 KC a thread) leave
constexpr int lora_expand_ctas(int KC) { return KC <= 4 ? 2 : 1; }

// KC: 32-wide chunks of the rank, R <= 32 KC.  VEC: rows of y are whole 16-byte
// pieces (n % 8 == 0).
template <int KC, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, lora_expand_ctas(KC)) lora_expand_kernel(const LoraArgs p) {
  extern __shared__ __align__(16) uint4 frag[];  // [row group][chunk][step][hi, lo][lane] fragments of h
  __shared__ int64_t yoff[128];  // rows of base and y, in elements
  __shared__ float factor[128];  // s 2^e of each row
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane >> 2, tig = lane & 3;
  // The work is num tiles x nch pieces of 256 columns (32 a warp), tiles
  // outer; every CTA takes an equal run of it, which is mostly one tile's (the
  // number of tiles is known only here).
  const int num = *p.num_tiles, n = p.n, R = p.R;
  const int nch = (n + 255) / 256;
  const int64_t units = (int64_t)num * nch;
  const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
  int run = 0;
  for (int64_t u = units * blockIdx.x / gridDim.x; u < u1; u += run) {
    const int t = (int)(u / nch), first = (int)(u - (int64_t)t * nch);
    run = (int)min((int64_t)(nch - first), u1 - u);
    const RowTile tile = p.tiles[t];
    const int c0 = first * 256, c1 = min((first + run) * 256, n);
    if (tile.count <= 0) continue;
    __syncthreads();  // (the last item's rows and fragments are no longer read)
    for (int i = tid; i < tile.count; i += kLoraThreads) yoff[i] = (int64_t)p.perm[tile.start + i] * n;
    if (tile.g >= p.L) {  // rows without an adapter
      __syncthreads();
      for (int i = warp; i < tile.count; i += kLoraWarps) {
        const int64_t at = yoff[i];
        copy_span(p.y + at, p.base + at, c0, c1, VEC, lane, 32);
      }
      continue;
    }
    const int rank = lora_rank(p, tile.g);
    const float scale = p.scales[tile.g];
    const int groups = (tile.count + 15) >> 4;
    // fragments of h: kAtOnce rows per warp at a time
    constexpr int kAtOnce = KC <= 4 ? 4 : 2;
    for (int i0 = warp * kAtOnce; i0 < groups * 16; i0 += kLoraWarps * kAtOnce) {
      float v[kAtOnce][KC];
#pragma unroll
      for (int r = 0; r < kAtOnce; r++)
#pragma unroll
        for (int c = 0; c < KC; c++)
          v[r][c] = (i0 + r < tile.count && 32 * c + lane < R) ? p.h[(int64_t)(tile.start + i0 + r) * R + 32 * c + lane]
                                                               : 0.f;
      unsigned few = 0;  // rows with a value of this lane that is too small
#pragma unroll
      for (int r = 0; r < kAtOnce; r++) {
        const int i = i0 + r;
        float f1, f2, back;
        h_scale<KC>(v[r], f1, f2, back);
        if (lane == 0) factor[i] = h_factor(scale, back);
        // column r = 32 c + 8 t + 4 s + 2 w + b of row i: word (row half) + 2 w of
        // lane (i % 8, t), step s of chunk c, half b
        const int t = lane >> 3, s = (lane >> 2) & 1, w = (lane >> 1) & 1, b = lane & 1;
        const int word = ((i >> 3) & 1) + 2 * w, to = ((i & 7) << 2) | t;
#pragma unroll
        for (int c = 0; c < KC; c++) {
          uint16_t hi, lo;
          h_split(v[r][c] * f1 * f2, hi, lo);
          if (h_small(v[r][c] * f1 * f2)) few |= 1u << r;
          uint16_t* f = reinterpret_cast<uint16_t*>(frag + ((((i >> 4) * KC + c) * 2 + s) * 2) * 32 + to);
          f[word * 2 + b] = hi;
          f[32 * 8 + word * 2 + b] = lo;
        }
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < kAtOnce; r++)
        if (few >> r & 1u) factor[i0 + r] = __uint_as_float(0x7FC00000u);
    }
    __syncthreads();
    const uint16_t* B = lora_b(p, tile.g);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int nb = c0 + warp * 32; nb < c1; nb += kLoraWarps * 32) {
      uint4 w[4][KC];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int col = nb + 8 * (grp >> 1) + 2 * j + (grp & 1);
#pragma unroll
        for (int c = 0; c < KC; c++) {
          const int r = 32 * c + 8 * tig;
          w[j][c] = (col < n && r < rank) ? *reinterpret_cast<const uint4*>(B + (int64_t)col * R + r) : zero;
        }
      }
      // the next columns' rows of B on their way into L2 meanwhile
      const int ncol = nb + kLoraWarps * 32 + lane;
      if (ncol < c1)
        for (int r = 0; r < rank; r += 64)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(B + (int64_t)ncol * R + r));
      const int col = nb + 8 * tig;  // this lane's 8 columns
      // base, kAhead row groups ahead of its use (loads stay behind the stores
      // they follow: y may be base)
      constexpr int kAhead = KC == 1 ? 3 : KC <= 4 ? 2 : 1;  // (KC 2 and 4 meet tiles of two groups only)
      uint4 ahead[kAhead][2];
      auto load_base = [&](int g, uint4 (&v)[2]) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int i = g * 16 + grp + 8 * h;
          v[h] = (VEC && i < tile.count && col < c1)
                     ? *reinterpret_cast<const uint4*>(p.base + yoff[i] + col)
                     : zero;
        }
      };
#pragma unroll
      for (int d = 0; d < kAhead; d++) load_base(d, ahead[d]);
      if (rank & 7) {  // (after the loads: a use between them would make each wait for the last)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
          for (int c = 0; c < KC; c++) w[j][c] = mask8(w[j][c], rank - (32 * c + 8 * tig));
      }
      unsigned redo = 0;  // this lane's pieces taken again in fp32: bits 2g, 2g + 1 for its two rows of group g
      for (int g0 = 0; g0 < groups; g0 += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; d++) {
          const int g = g0 + d;
          if (g >= groups) break;
          const int i0 = g * 16 + grp, i1 = i0 + 8;
          const bool ok0 = i0 < tile.count, ok1 = i1 < tile.count;
          const int64_t at0 = yoff[ok0 ? i0 : 0] + col, at1 = yoff[ok1 ? i1 : 0] + col;
          uint4 b0 = ahead[d][0], b1 = ahead[d][1];
          load_base(g + kAhead, ahead[d]);
          float acc[4][4];
#pragma unroll
          for (int j = 0; j < 4; j++)
#pragma unroll
            for (int c = 0; c < 4; c++) acc[j][c] = 0.f;
#pragma unroll
          for (int half = 1; half >= 0; half--) {  // lo, then hi
#pragma unroll
            for (int c = 0; c < KC; c++) {
              if (32 * c >= rank) break;
#pragma unroll
              for (int s = 0; s < 2; s++) {
                const uint4 hv = frag[((((g * KC + c) * 2 + s) * 2) + half) * 32 + lane];
#pragma unroll
                for (int j = 0; j < 4; j++)
                  mma_16816(acc[j], hv.x, hv.y, hv.z, hv.w, s ? w[j][c].z : w[j][c].x, s ? w[j][c].w : w[j][c].y);
              }
            }
            if (half) {
#pragma unroll
              for (int j = 0; j < 4; j++)
#pragma unroll
                for (int c = 0; c < 4; c++) acc[j][c] *= 1.0f / (1 << kLoraLoBits);
            }
          }
          // acc[j][0..1]: row i0, columns col + 2j, + 1; acc[j][2..3]: row i1
          const float q0 = factor[i0], q1 = factor[i1];
          if (!VEC) {
            if (ok0) b0 = load8(p.base + at0, c1 - col);
            if (ok1) b1 = load8(p.base + at1, c1 - col);
          }
          const uint32_t bw0[4] = {b0.x, b0.y, b0.z, b0.w}, bw1[4] = {b1.x, b1.y, b1.z, b1.w};
          uint32_t o0[4], o1[4];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const float2 f0 = f16x2_to_f32x2(bw0[j]), f1 = f16x2_to_f32x2(bw1[j]);
            o0[j] = f32x2_to_f16x2(fmaf(acc[j][0], q0, f0.x), fmaf(acc[j][1], q0, f0.y));
            o1[j] = f32x2_to_f16x2(fmaf(acc[j][2], q1, f1.x), fmaf(acc[j][3], q1, f1.y));
          }
          const uint4 v0 = make_uint4(o0[0], o0[1], o0[2], o0[3]), v1 = make_uint4(o1[0], o1[1], o1[2], o1[3]);
          // a piece that is infinite or NaN somewhere is left for lora_row_fp32
          const bool on0 = ok0 && col < c1, on1 = ok1 && col < c1;
          const bool bad0 = on0 && nonfinite8(v0), bad1 = on1 && nonfinite8(v1);
          redo |= (bad0 ? 1u : 0u) << (2 * g) | (bad1 ? 2u : 0u) << (2 * g);
          if (on0 && !bad0) {
            if (VEC) *reinterpret_cast<uint4*>(p.y + at0) = v0;
            else store8(p.y + at0, v0, c1 - col);
          }
          if (on1 && !bad1) {
            if (VEC) *reinterpret_cast<uint4*>(p.y + at1) = v1;
            else store8(p.y + at1, v1, c1 - col);
          }
        }
      }
      for (unsigned todo = __ballot_sync(0xFFFFFFFFu, redo != 0); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, cf = nb + 8 * (from & 3);
        for (unsigned m = __shfl_sync(0xFFFFFFFFu, redo, from); m; m &= m - 1) {
          const int bit = __ffs(m) - 1, i = (bit >> 1) * 16 + (bit & 1) * 8 + (from >> 2);
          lora_row_fp32(p.y + yoff[i], p.base + yoff[i], p.h + (int64_t)(tile.start + i) * R, B, R, rank, scale, cf,
                        min(cf + 8, c1));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The same for long inputs (tiles of up to 128 rows, R <= 128) on
// 5th-generation tensor cores.  The tile's rows are M, 128 columns of y (rows of
// B, brought by TMA into 128-byte-swizzled stages) are N, and K runs over the
// rank twice, for the two halves of h, against the same stage of B.  A lane of
// the epilogue then holds a row's neighbouring columns, 32 bytes a load and
// store (with the columns as M it held a column, and the lanes had to exchange:
// 75 us against 49 for 2,048 rows of rank 64 and 18,560 columns).  The legacy
// MMAs of lora_expand_kernel take 34 us of tensor time alone at rank 128 and
// their fragments as much again (89 us in all); here the products take 9 us (52
// in all, 37 of them the hand-overs between the roles: what is left when base
// and y are neither loaded nor stored).
//
// Roles (one CTA per SM, an equal run of (tile, 128 columns) units each):
//   warp 0       B by TMA, kLtStages deep
//   warp 1       tcgen05.mma issue; owns tensor memory (4 accumulators of 128
//                columns)
//   warps 2-3    zero what a rank that is not a multiple of 16 leaves of its
//                last 16 columns in each stage (it may hold anything)
//   warps 4-19   write a tile's h into shared memory when the tile changes;
//                epilogue: four groups of four warps take the units in turn,
//                with base loaded before the wait for the products
// Every wait is bounded, as in the GEMMs.
// ---------------------------------------------------------------------------
constexpr int kLtStages = 3, kLtGroups = 4, kLtEpi = kLtGroups * 4 * 32, kLtThreads = 4 * 32 + kLtEpi;
constexpr int kLtHalf = 128 * 128;               // bytes of 128 rows x 64 k
__host__ __device__ constexpr int lora_tc_smem(int KB) {
  return 1024 + 2 * KB * kLtHalf + kLtStages * KB * kLtHalf + 256;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Ranks whose last k16 step is not all of their own columns.
__device__ __forceinline__ bool lora_partial(int rank) { return (rank & 15) != 0 || rank == 0; }

// 32 bytes a lane (32-byte aligned).
__device__ __forceinline__ void ld256(uint32_t (&w)[8], const void* p) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st256(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// D = A B + 2^-BITS D
template <int BITS>
__device__ __forceinline__ void umma_f16_scaled_d(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, 1, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p, %4;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(BITS)
      : "memory");
}

// All lanes of the warp here, before a warp-wide instruction; orders no memory.
// (Predicated loads and stores instead, as st128_if, took 92 us where this takes
// 85 for 2,048 rows of rank 128.)
__device__ __forceinline__ void warp_converge() { asm volatile("bar.warp.sync 0xffffffff;"); }

template <int KB>  // 64-wide k blocks: R <= 64 KB
__global__ void __launch_bounds__(kLtThreads, 1)
    lora_expand_tc_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ LoraArgs p) {
  extern __shared__ uint8_t smem_lt[];
  __shared__ int64_t yoff[2][128];
  __shared__ float factor[2][128];
  __shared__ volatile int s_abort;
  const uint32_t base = (smem_addr(smem_lt) + 1023u) & ~1023u;
  const uint32_t h_s = base, b_s = h_s + 2 * KB * kLtHalf, bars = b_s + kLtStages * KB * kLtHalf;
  const uint32_t full = bars, fixd = full + 8 * kLtStages, empty = fixd + 8 * kLtStages, accf = empty + 8 * kLtStages,
                 acce = accf + 32, hfree = acce + 32, hfull = hfree + 8, done_bar = hfull + 8, tmem_slot = done_bar + 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < kLtStages; s++) {
      mbar_init(full + 8 * s, 1);
      mbar_init(fixd + 8 * s, 2);
      mbar_init(empty + 8 * s, 1);
    }
    for (int a = 0; a < 4; a++) {
      mbar_init(accf + 8 * a, 1);
      mbar_init(acce + 8 * a, 4);
    }
    mbar_init(hfree, kLtEpi / 32);
    mbar_init(hfull, kLtEpi / 32);
    mbar_init(done_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_enter();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
  const int num = *p.num_tiles, n = p.n, R = p.R;
  const int nch = (n + 127) >> 7;
  const int64_t units = (int64_t)num * nch;
  const int64_t u0 = units * blockIdx.x / gridDim.x;
  const int my_units = (int)(units * (blockIdx.x + 1) / gridDim.x - u0);
  const int t0 = (int)(u0 / nch), ch0 = (int)(u0 - (int64_t)t0 * nch);  // the first unit's tile and columns
  // (units of rows without an adapter are copied by the epilogue warps alone)

  if (warp == 0) {
    // ------------------------------- B -------------------------------------
    if (lane == 0) {
      prefetch_tmap(&tm_b);
      uint32_t c = 0, issued = 0;  // stages filled
      const bool withhold = (g_test_flags & kTestWithholdXTiles) != 0;  // test switch: issue nothing
      RowTile tile = {};
      for (int u = 0, t = t0, ch = ch0; u < my_units && !withhold; u++, ch++) {
        if (ch == nch) { ch = 0; t++; }
        if (u == 0 || ch == 0) tile = p.tiles[t];
        if (tile.g >= p.L || tile.count <= 0) continue;
        const uint32_t s = c % kLtStages;
        if (!gg_wait(empty + 8 * s, ((c / kLtStages) & 1u) ^ 1u)) { s_abort = 1; break; }
        mbar_arrive_expect_tx(full + 8 * s, KB * kLtHalf);
        for (int b = 0; b < KB; b++)
          tma_load_3d(b_s + (s * KB + b) * kLtHalf, &tm_b, b * 64, ch * 128, tile.g, full + 8 * s);
        c++;
        issued = c;
      }
      for (uint32_t s = 0; s < kLtStages && s < issued; s++) {  // drain our copies
        const uint32_t last = issued - 1 - ((issued - 1 - s) % kLtStages);
        gg_wait(full + 8 * s, (last / kLtStages) & 1u);
      }
    }
  } else if (warp == 1) {
    // ---------------------------- MMA issuer ------------------------------
    const bool leader = elect_one();
    uint32_t c = 0, tiles = 0;
    int k16 = 0;
    RowTile tile = {};
    const uint32_t idesc = umma_idesc_f16(128);
    for (int u = 0, t = t0, ch = ch0; u < my_units; u++, ch++) {
      if (ch == nch) { ch = 0; t++; }
      const bool fresh = u == 0 || ch == 0;  // a new tile
      if (fresh) tile = p.tiles[t];
      if (tile.g >= p.L || tile.count <= 0) continue;
      bool ok = true;
      if (fresh) {
        const int rank = (int)warp_uniform((uint32_t)lora_rank(p, tile.g));
        k16 = max((rank + 15) >> 4, 1);  // (rank 0: one step of zeros)
        ok = gg_wait(hfull, tiles++ & 1u);
      }
      const uint32_t s = c % kLtStages, a = c & 3u;
      // (both barriers for every stage: neither may get a phase ahead of its other waiter)
      ok = ok && gg_wait(acce + 8 * a, ((c >> 2) & 1u) ^ 1u) && gg_wait(full + 8 * s, (c / kLtStages) & 1u) &&
           gg_wait(fixd + 8 * s, (c / kLtStages) & 1u);
      if (!__all_sync(0xFFFFFFFFu, ok)) { s_abort = 1; break; }
      tc_fence_after();
      const uint32_t d = warp_uniform(tmem) + 128u * a;
      if (leader) {
        for (int kk = 0; kk < k16; kk++) {
          const uint32_t blk = (uint32_t)(kk >> 2) * kLtHalf;
          const uint64_t db = umma_desc_k128(b_s + s * KB * kLtHalf + blk) + (uint64_t)(2 * (kk & 3));
          const uint64_t dh = umma_desc_k128(h_s + blk) + (uint64_t)(2 * (kk & 3));
          umma_f16(d, dh + (uint64_t)(KB * kLtHalf / 16), db, idesc, kk != 0);
        }
        for (int kk = 0; kk < k16; kk++) {
          const uint32_t blk = (uint32_t)(kk >> 2) * kLtHalf;
          const uint64_t db = umma_desc_k128(b_s + s * KB * kLtHalf + blk) + (uint64_t)(2 * (kk & 3));
          const uint64_t dh = umma_desc_k128(h_s + blk) + (uint64_t)(2 * (kk & 3));
          if (kk == 0) umma_f16_scaled_d<kLoraLoBits>(d, dh, db, idesc);
          else umma_f16(d, dh, db, idesc, 1);
        }
        umma_commit(empty + 8 * s);
        umma_commit(accf + 8 * a);
      }
      __syncwarp();
      c++;
    }
    if (leader) umma_commit(done_bar);
  } else if (warp < 4) {
    // ----------------------- ranks inside a k16 step ------------------------
    uint32_t c = 0;
    int rank = 0;
    RowTile tile = {};
    for (int u = 0, t = t0, ch = ch0; u < my_units; u++, ch++) {
      if (ch == nch) { ch = 0; t++; }
      if (u == 0 || ch == 0) {
        tile = p.tiles[t];
        if (tile.g < p.L) rank = lora_rank(p, tile.g);
      }
      if (tile.g >= p.L || tile.count <= 0) continue;
      const uint32_t s = c % kLtStages;
      const bool ok = gg_wait(full + 8 * s, (c / kLtStages) & 1u);
      if (!__all_sync(0xFFFFFFFFu, ok)) { s_abort = 1; break; }
      if (lora_partial(rank)) {
        const int top = max((rank + 15) & ~15, 16);
        for (int r = (warp - 2) * 64 + lane; r < (warp - 1) * 64; r += 32)
          for (int k = rank; k < top; k++) {
          const uint32_t at = b_s + (s * KB + (k >> 6)) * kLtHalf + r * 128 + ((((k & 63) >> 3) ^ (r & 7)) << 4) +
                              (k & 7) * 2;
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)0) : "memory");
        }
        fence_proxy_async_shared();
      }
      warp_arrive(fixd + 8 * s, lane);
      c++;
    }
  } else {
    // -------------------------- h and epilogue ------------------------------
    const int ew = warp - 4, q = warp & 3, grp = ew >> 2;
    const bool vec = (n & 7) == 0;
    // whole 32-byte sectors a lane where rows and buffers allow it
    const bool wide = (n & 15) == 0 &&
                      ((reinterpret_cast<uintptr_t>(p.base) | reinterpret_cast<uintptr_t>(p.y)) & 31) == 0;
    const int row = 32 * q + lane;  // of the tile: a TMEM lane
    uint32_t c = 0, tiles = 0;
    int tb = 0;
    RowTile tile = {};
    float scale = 0.f;
    bool ok = true;
    for (int u = 0, t = t0, ch = ch0; u < my_units && ok; u++, ch++) {
      if (ch == nch) { ch = 0; t++; }
      const bool fresh = u == 0 || ch == 0;  // a new tile
      if (fresh) tile = p.tiles[t];
      if (tile.count <= 0) continue;
      if (tile.g >= p.L) {  // rows without an adapter
        const int c0 = ch * 128, c1 = min(c0 + 128, n);
        for (int i = ew; i < tile.count; i += kLtEpi / 32) {
          const int64_t at = (int64_t)p.perm[tile.start + i] * n;
          copy_span(p.y + at, p.base + at, c0, c1, vec, lane, 32);
        }
        continue;
      }
      if (fresh) {
        // once every epilogue warp is here, all units of the last one
        // have been multiplied (each has waited for that tile's last unit)
        warp_arrive(hfree, lane);
        ok = gg_wait(hfree, tiles & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) { s_abort = 1; break; }
        tb ^= 1;
        scale = p.scales[tile.g];
        for (int i = tid - 128; i < tile.count; i += kLtEpi) yoff[tb][i] = (int64_t)p.perm[tile.start + i] * n;
        for (int i0 = ew * 4; i0 < 128; i0 += kLtEpi / 8) {
          float v[4][2 * KB];
#pragma unroll
          for (int r = 0; r < 4; r++)
#pragma unroll
            for (int b = 0; b < 2 * KB; b++)
              v[r][b] = (i0 + r < tile.count && 32 * b + lane < R)
                            ? p.h[(int64_t)(tile.start + i0 + r) * R + 32 * b + lane]
                            : 0.f;
          unsigned few = 0;  // rows with a value of this lane that is too small
#pragma unroll
          for (int r = 0; r < 4; r++) {
            float f1, f2, back;
            h_scale<2 * KB>(v[r], f1, f2, back);
            const int i = i0 + r;
            if (lane == 0) factor[tb][i] = h_factor(scale, back);
#pragma unroll
            for (int b = 0; b < 2 * KB; b++) {
              uint16_t hi, lo;
              h_split(v[r][b] * f1 * f2, hi, lo);
              if (h_small(v[r][b] * f1 * f2)) few |= 1u << r;
              const int k = 32 * b + lane;
              const uint32_t at = h_s + (k >> 6) * kLtHalf + i * 128 + ((((k & 63) >> 3) ^ (i & 7)) << 4) + (k & 7) * 2;
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(hi) : "memory");
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + KB * kLtHalf), "h"(lo) : "memory");
            }
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < 4; r++)
            if (few >> r & 1u) factor[tb][i0 + r] = __uint_as_float(0x7FC00000u);
        }
        fence_proxy_async_shared();
        warp_arrive(hfull, lane);
        ok = gg_wait(hfull, tiles++ & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) { s_abort = 1; break; }
      }
      if ((int)(c % kLtGroups) == grp) {
        const uint32_t a = c & 3u;
        const int c0 = ch * 128, left = n - c0;  // columns from here on
        const bool live = row < tile.count;
        const uint16_t* bp = p.base + yoff[tb][live ? row : 0] + c0;
        uint16_t* yp = p.y + yoff[tb][live ? row : 0] + c0;
        const float f = factor[tb][row];
        // base, 64 columns ahead of its use (the first before the products are
        // waited for)
        uint32_t bv[2][16];
        auto load_base = [&](int j, uint32_t(&to)[16]) {
#pragma unroll
          for (int i = 0; i < 2; i++) {
            uint32_t(&w)[8] = *reinterpret_cast<uint32_t(*)[8]>(&to[8 * i]);
            const int col = 32 * j + 16 * i;
            if (live && wide && col < left) {
              ld256(w, bp + col);
            } else if (live && vec && col < left) {
              const uint4 v0 = *reinterpret_cast<const uint4*>(bp + col);
              const uint4 v1 =
                  col + 8 < left ? *reinterpret_cast<const uint4*>(bp + col + 8) : make_uint4(0u, 0u, 0u, 0u);
              w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w; w[4] = v1.x; w[5] = v1.y; w[6] = v1.z; w[7] = v1.w;
            } else {
#pragma unroll
              for (int x = 0; x < 8; x++) w[x] = 0u;
            }
          }
        };
        load_base(0, bv[0]);
        load_base(1, bv[1]);
        ok = gg_wait(accf + 8 * a, (c >> 2) & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) { s_abort = 1; break; }
        tc_fence_after();
        if (32 * q < tile.count) {
          unsigned redo = 0;  // this row's pieces of 16 columns that are infinite or NaN somewhere, for lora_row_fp32
#pragma unroll
          for (int j = 0; j < 4; j++) {
            uint32_t r[32];
            warp_converge();  // (the stores before are not the whole warp's)
            tmem_ld32(tmem + 128u * a + 32u * j + ((uint32_t)(32 * q) << 16), r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const int col = 32 * j + 16 * i;
              if (!vec && live) {
                uint32_t(&w)[8] = *reinterpret_cast<uint32_t(*)[8]>(&bv[j & 1][8 * i]);
                const uint4 v0 = load8(bp + col, left - col), v1 = load8(bp + col + 8, left - col - 8);
                w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w; w[4] = v1.x; w[5] = v1.y; w[6] = v1.z; w[7] = v1.w;
              }
              uint32_t o[8];
#pragma unroll
              for (int x = 0; x < 8; x++) {
                const float2 b = f16x2_to_f32x2(bv[j & 1][8 * i + x]);
                o[x] = f32x2_to_f16x2(fmaf(__uint_as_float(r[16 * i + 2 * x]), f, b.x),
                                      fmaf(__uint_as_float(r[16 * i + 2 * x + 1]), f, b.y));
              }
              const uint4 v0 = make_uint4(o[0], o[1], o[2], o[3]), v1 = make_uint4(o[4], o[5], o[6], o[7]);
              const bool on = live && col < left;
              const bool bad = on && (nonfinite8(v0) || nonfinite8(v1));
              if (on && !bad) {
                if (wide) {
                  st256(yp + col, o);
                } else if (vec) {
                  *reinterpret_cast<uint4*>(yp + col) = v0;
                  if (col + 8 < left) *reinterpret_cast<uint4*>(yp + col + 8) = v1;
                } else {
                  store8(yp + col, v0, left - col);
                  store8(yp + col + 8, v1, left - col - 8);
                }
              }
              redo |= (bad ? 1u : 0u) << (2 * j + i);
            }
            if (j + 2 < 4) load_base(j + 2, bv[j & 1]);
          }
          for (unsigned todo = __ballot_sync(0xFFFFFFFFu, redo != 0); todo; todo &= todo - 1) {
            const int from = __ffs(todo) - 1, i = 32 * q + from;
            for (unsigned m = __shfl_sync(0xFFFFFFFFu, redo, from); m; m &= m - 1) {
              const int cf = c0 + 16 * (__ffs(m) - 1);
              lora_row_fp32(p.y + yoff[tb][i], p.base + yoff[tb][i], p.h + (int64_t)(tile.start + i) * R,
                            lora_b(p, tile.g), R, lora_rank(p, tile.g), scale, cf, min(cf + 16, n));
            }
          }
        }
        tc_fence_before();
        warp_arrive(acce + 8 * a, lane);
      } else if (u + 1 == my_units || ch + 1 == nch) {
        // the tile's last unit is another group's: wait for its products too,
        // so that h may be written again
        ok = gg_wait(accf + 8 * (c & 3u), (c >> 2) & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) { s_abort = 1; break; }
      }
      c++;
    }
  }

  // teardown: no MMA of ours may still be using tensor memory
  if (warp == 1 && lane == 0) gg_wait(done_bar, 0);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace qmm
