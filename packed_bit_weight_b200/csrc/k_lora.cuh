// k_lora.cuh -- low-rank adapters of many requests beside a shared projection:
// y[i] = fp16(base[i] + s_a B_a (A_a x[i])) for the adapter a of row i, A_a
// [rank][k] and B_a [n][rank] ("1bit.gg zyphra": the graph form base +
// B*(A*x)).
//
// A few rows (decode): one launch, a thread-block cluster per row and part of
// n (lora_token_kernel).  More rows: the rows are sorted by adapter into tiles
// (the sort of k_rows.cuh), the middle products A x are taken per tile with the
// cluster's CTAs and warps sharing k (lora_shrink_kernel), and B and base are
// streamed once per tile (lora_expand_kernel).  The bound is bytes: A and B of
// the adapters in use, x, base and y; the products are rank / (bytes) small,
// so legacy MMAs straight from global memory, without staging, keep up.
#pragma once
#include "k_gemm.cuh"
#include "k_gemv.cuh"
#include "k_rows.cuh"

namespace qmm {

constexpr int kLoraMaxRank = 256;
constexpr int kLoraCluster = 8;    // CTAs that share a row (or a tile)
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
// instruction took 38 us for 2,048 rows of rank 128 and k = 4096.)
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
    p.h[(int64_t)(tile.start + (i >> 6)) * R + rb + r] = s;
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
// The middle product is held as two fp16 halves, h = 2^e (hi + lo): each row
// is scaled by a power of two that brings its largest finite value to
// [2^14, 2^15), hi is the rounded value and lo the rounded rest, so h keeps 22
// bits (off by 2^-22 where one fp16 would be off by 2^-12) at twice the MMAs,
// which the stream of base and y hides.
// ---------------------------------------------------------------------------
// CTAs per SM: what the registers of B's fragments (16 KC a thread) leave
constexpr int lora_expand_ctas(int KC) { return KC <= 4 ? 2 : 1; }

template <int KC>  // 32-wide chunks of the rank: R <= 32 KC
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
      copy_span(p.y + at, p.base + at, c0, c1, (n & 7) == 0, lane, 32);
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
#pragma unroll
    for (int r = 0; r < kAtOnce; r++) {
    const int i = i0 + r;
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < KC; c++) {
      const float f = fabsf(v[r][c]);
      if (f <= 3.4028235e38f) top = fmaxf(top, f);  // (finite)
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    // top in [2^e, 2^(e+1)): scaled by 2^(14 - e), in two factors so that neither leaves fp32
    const int e = (int)(__float_as_uint(top) >> 23) - 127;
    const int sh = top > 0.f ? min(14 - e, 126) : 0;
    const float f1 = __uint_as_float((uint32_t)(127 + (sh >> 1)) << 23);
    const float f2 = __uint_as_float((uint32_t)(127 + (sh - (sh >> 1))) << 23);
    if (lane == 0) factor[i] = scale * __uint_as_float((uint32_t)(127 - sh) << 23);
    // column r = 32 c + 8 t + 4 s + 2 w + b of row i: word (row half) + 2 w of lane (i % 8, t), step s of chunk c, half b
    const int t = lane >> 3, s = (lane >> 2) & 1, w = (lane >> 1) & 1, b = lane & 1;
    const int word = ((i >> 3) & 1) + 2 * w, to = ((i & 7) << 2) | t;
#pragma unroll
    for (int c = 0; c < KC; c++) {
      const float x = v[r][c] * f1 * f2;
      const __half hi = __float2half_rn(x);
      const float back = __half2float(hi);
      const bool finite = fabsf(back) <= 65504.f;
      const __half lo = finite ? __float2half_rn(x - back) : __float2half_rn(0.f);
      __half* f = reinterpret_cast<__half*>(frag + ((((i >> 4) * KC + c) * 2 + s) * 2) * 32 + to);
      f[word * 2 + b] = hi;
      f[32 * 8 + word * 2 + b] = lo;
    }
    }
  }
  __syncthreads();
  const uint16_t* B = lora_b(p, tile.g);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const bool vec = (n & 7) == 0;
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
    constexpr int kAhead = KC <= 4 ? 3 : 1;
    uint4 ahead[kAhead][2];
    auto load_base = [&](int g, uint4 (&v)[2]) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int i = g * 16 + grp + 8 * h;
        v[h] = (vec && i < tile.count && col < c1)
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
    for (int g0 = 0; g0 < groups; g0 += kAhead) {
#pragma unroll
    for (int d = 0; d < kAhead; d++) {
      const int g = g0 + d;
      if (g >= groups) break;
      const int i0 = g * 16 + grp, i1 = i0 + 8;
      const bool ok0 = i0 < tile.count, ok1 = i1 < tile.count;
      const int64_t at0 = yoff[ok0 ? i0 : 0] + col, at1 = yoff[ok1 ? i1 : 0] + col;
      const uint4 b0 = ahead[d][0], b1 = ahead[d][1];
      load_base(g + kAhead, ahead[d]);
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) acc[j][c] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; c++) {
        if (32 * c >= rank) break;
#pragma unroll
        for (int s = 0; s < 2; s++) {
          const uint4* f = frag + (((g * KC + c) * 2 + s) * 2) * 32 + lane;
          const uint4 hi = f[0], lo = f[32];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t v0 = s ? w[j][c].z : w[j][c].x, v1 = s ? w[j][c].w : w[j][c].y;
            mma_16816(acc[j], hi.x, hi.y, hi.z, hi.w, v0, v1);
            mma_16816(acc[j], lo.x, lo.y, lo.z, lo.w, v0, v1);
          }
        }
      }
      // acc[j][0..1]: row i0, columns col + 2j, + 1; acc[j][2..3]: row i1
      const float q0 = factor[i0], q1 = factor[i1];
      if (vec) {
        const uint32_t bw0[4] = {b0.x, b0.y, b0.z, b0.w}, bw1[4] = {b1.x, b1.y, b1.z, b1.w};
        uint32_t o0[4], o1[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float2 f0 = f16x2_to_f32x2(bw0[j]), f1 = f16x2_to_f32x2(bw1[j]);
          o0[j] = f32x2_to_f16x2(fmaf(acc[j][0], q0, f0.x), fmaf(acc[j][1], q0, f0.y));
          o1[j] = f32x2_to_f16x2(fmaf(acc[j][2], q1, f1.x), fmaf(acc[j][3], q1, f1.y));
        }
        if (ok0 && col < c1) *reinterpret_cast<uint4*>(p.y + at0) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
        if (ok1 && col < c1) *reinterpret_cast<uint4*>(p.y + at1) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
          for (int b = 0; b < 2; b++) {
            if (col + 2 * j + b >= c1) continue;
            if (ok0) {
              const int64_t at = at0 + 2 * j + b;
              p.y[at] = f32_to_f16_bits(fmaf(acc[j][b], q0, __half2float(__ushort_as_half(p.base[at]))));
            }
            if (ok1) {
              const int64_t at = at1 + 2 * j + b;
              p.y[at] = f32_to_f16_bits(fmaf(acc[j][b + 2], q1, __half2float(__ushort_as_half(p.base[at]))));
            }
          }
      }
    }
    }
  }
  }
}

}  // namespace qmm
