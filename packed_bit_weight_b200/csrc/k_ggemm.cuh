// k_ggemm.cuh -- the experts' products over rows sorted by expert, on
// 5th-generation tensor cores ("Mark-Experimental-V3-8B", section
// "Mixture-of-Experts (MoE)").
//
// ys[r] = W_e xs[r] for the rows r of expert e.  A tile is 128 weight rows of
// one expert times up to 256 of its rows; D^T = W X^T, so the decoded weights
// are the A operand and live in TENSOR MEMORY (a decode thread owns a weight
// row = a TMEM lane, and stores its decoded pairs as consecutive columns),
// the X rows are the B operand in shared memory, and N is the number of rows
// rounded up to 16.  With both operands in shared memory a 256 x 128 tile
// reads 64 KB, writes 48 KB and looks 4,096 pairs up per 64-wide k step, about
// 1,100 cycles of the 128-byte port for 512 cycles of MMA; with the weights
// in TMEM the port carries X once in and once out and the lookups, ~650.
// On B200, 32 IQ4_NL experts over 8,192 rows: gate and up (896 x 2560 each)
// 116 to 122 us, 620 to 650 TFLOP/s, from box to box; down (2560 x 896) 66 to
// 69 us; gate and up in FP4-G16, E4M3 and MXFP4 110, 107 and 110 us where IQ4_NL
// takes 119.  What bounds it: the decode's
// latency (434 ns per step at 16 rows, 262 with the lookups left out, 208 with
// copies and X left out too; the MMAs of 256 rows are 260), and 5 rounds of
// tiles where 4.5 would do.
//
// Roles per CTA (persistent, one per SM, 24 warps):
//   warp 0       X rows by TMA (64-row boxes, 128-byte swizzle), kGgStages deep
//   warp 1       tcgen05.mma issue; owns the tensor memory
//   warps 2-3    packed weights by cp.async, chunks of 256 k, kGgSlots deep
//   warps 4-19   weight decode: four groups of four warps, group j has step j
//                of each chunk.  A step's chain (wait, read, look up, multiply,
//                wait, tcgen05.st, arrive) is latency, ~1,000 cycles of it, and
//                only more warps hide it
//   warps 20-23  epilogue: tcgen05.ld, fp16, store
// Tensor memory: kGgStages x 32 columns of weights and three accumulators of
// 128 columns.  A tile of more than 128 rows takes the middle one and, in
// turn, the first or the last, which are one run of columns (one MMA of N up
// to 256 per k16 step); the epilogue drains the middle one first, so the next
// tile waits for half of this one's stores.  Smaller tiles take the first and
// the last in turn.
//
// SWI: the tile's 128 weight rows are 64 rows of gate and of up, 16 + 16 in
// each warp's 32 lanes, so that SiLU(gate) * up needs one shuffle per pair of
// tokens and nothing leaves the SM in between.
//
// Every wait is bounded; on a timeout the kernel raises the error word, lets
// its own copies and MMAs finish, frees its tensor memory and returns.
#pragma once
#include "k_gemm.cuh"
#include "k_iq4t.cuh"
#include "k_rows.cuh"

namespace qmm {

constexpr int kGgStages = kGemmChunkSteps;        // stage = a step's place in its chunk
constexpr int kGgSlots = 3;                       // packed chunks of 256 k in flight
constexpr int kGgRows = 128;                      // weight rows per tile
constexpr int kGgTok = 256;                       // rows of X per tile at most
constexpr int kGgXBytes = kGgTok * kGemmBK * 2;   // 32 KB per stage
constexpr int kGgMaxExperts = 256;
constexpr int kGgCopyWarps = 2, kGgGroups = 4, kGgDecodeWarps = 4 * kGgGroups;
constexpr int kGgThreads = (2 + kGgCopyWarps + kGgDecodeWarps + 4) * 32;
constexpr int kGgCodes = kGgRows * 128;           // FP4 slot: codes [128][128 B] (unit u of row r at u ^ (r & 7))
constexpr int kGgSlotFp4 = kGgCodes + kGgRows * 32;   // then scales [128][32 B]
// IQ4_NL slot: [128 rows][144 B] (9 units: 16-byte reads of 8 rows hit 8 bank groups)
constexpr int kGgSlotIq4 = kGgRows * 144;
constexpr uint32_t kGgAccCol = 0, kGgACol = 384;  // TMEM columns: 3 x 128 accumulators, 4 x 32 weights

struct GgArgs {
  const uint8_t* data[2];    // stacks: [0] (gate), [1] up
  const uint8_t* scales[2];
  int64_t dstride[2], sstride[2];
  float g[2];
  const int32_t* offsets;
  uint16_t* y;
  int E, P, n, k;
};

__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait whose first polls touch nothing but the barrier (its time limit is
// a global load and a timer read, which a wait of a few hundred cycles should
// not pay for).
__device__ __forceinline__ bool gg_wait(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; i++)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity);
}

// gg_wait of a whole warp, with one answer for all its lanes: on the fast path
// none, a lane at a time only if one runs out of polls.
__device__ __forceinline__ bool gg_wait_warp(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; i++)
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
}

// Predicated stores: where a warp-wide instruction (tcgen05.ld) follows, the
// lanes must not part for their stores.  (Joining them again by a barrier takes
// 2 to 3 % of the grouped product: it holds the next load behind the stores.)
__device__ __forceinline__ void st128_if(bool on, void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n @p st.global.v4.b32 [%1], {%2,%3,%4,%5};\n}" ::"r"(
                   (uint32_t)on),
               "l"(p), "r"(a), "r"(b), "r"(c), "r"(d));
}
__device__ __forceinline__ void st16_if(bool on, void* p, uint32_t v) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n @p st.global.b16 [%1], %2;\n}" ::"r"((uint32_t)on), "l"(p),
               "h"((unsigned short)v));
}

// One arrival for a whole warp, once all its lanes are done (128 threads
// arriving on one barrier one after another took longer than a k step).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// True in one lane of the warp.  tcgen05.mma issued under it costs ~9 cycles,
// under lane == 0 ~46 (the compiler cannot see that one lane is left).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}

// A value that is the same in every lane, as the compiler can see it.
__device__ __forceinline__ uint32_t warp_uniform(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }

// Shared memory (from a 1,024-byte boundary): X stages, packed slots, the
// IQ4_NL pair table (32 copies, one per bank), barriers.
template <int FMT>
struct GgSmem {
  static constexpr uint32_t kSlot = FMT == 1 ? kGgSlotIq4 : kGgSlotFp4;
  static constexpr uint32_t kX = 0, kP = kGgStages * kGgXBytes, kLut = kP + kGgSlots * kSlot,
                            kBars = kLut + (FMT == 1 ? (uint32_t)kIqLutBytes : 0u),
                            kBytes = kBars + 8 * (2 * kGgStages + 2 * 3 + 1 + 2 * kGgSlots) + 16;
  static constexpr size_t total() { return 1024 + kBytes; }
};

// A tile's place: weight rows from n0 of expert e, rows m0 .. m0 + cnt - 1.
struct GgTile {
  int e, m0, cnt, n0;
};

// Step J (64 k) of tile row `row` from its packed chunk: 32 words of two
// weights in k order, the exact decoded fp16 weights (E4M3: without the global
// scale).  Rows past n decode to zeros.
template <int FMT, int J>
__device__ __forceinline__ void gg_decode(uint32_t src, int row, bool valid, uint32_t lut_lane, uint32_t (&o)[32]) {
  if (FMT == 1) {
    // two blocks: 36 bytes from byte 36 J of the row, in its units 2J .. 2J+2
    uint32_t uw[12];
#pragma unroll
    for (int u = 0; u < 3; u++) {
      const uint4 v = lds128(src + row * 144 + (2 * J + u) * 16);
      uw[4 * u] = v.x; uw[4 * u + 1] = v.y; uw[4 * u + 2] = v.z; uw[4 * u + 3] = v.w;
    }
    const uint32_t da = __byte_perm(uw[J], 0u, valid ? 0x1010u : 0x4444u);
    const uint32_t db = __byte_perm(uw[J + 4], 0u, valid ? 0x3232u : 0x4444u);
#pragma unroll
    for (int i = 0; i < 8; i++) {  // index words: 4 of each block
      const uint32_t q = i < 4 ? __funnelshift_r(uw[J + i], uw[J + i + 1], 16) : uw[J + 1 + i];
      const uint32_t d = i < 4 ? da : db;
      uint32_t w[4];  // byte b: weights (4i + b, 4i + b + 16) of the block
#pragma unroll
      for (int b = 0; b < 4; b++) w[b] = hmul2(lds32(lut_addr(q, b, lut_lane)), d);
      const int at = (i >> 2) * 16 + (i & 3) * 2;
      o[at] = __byte_perm(w[0], w[1], 0x5410);
      o[at + 1] = __byte_perm(w[2], w[3], 0x5410);
      o[at + 8] = __byte_perm(w[0], w[1], 0x7632);
      o[at + 9] = __byte_perm(w[2], w[3], 0x7632);
    }
  } else {
    uint32_t q[8];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const uint4 v = lds128(src + row * 128 + (((2 * J + u) ^ (row & 7)) << 4));
      q[4 * u] = v.x; q[4 * u + 1] = v.y; q[4 * u + 2] = v.z; q[4 * u + 3] = v.w;
    }
    uint32_t f1[4], f2[4];  // per 16 k: the scale, and for wide E8M0 scales a first factor
    bool two = false;
    if (FMT == 2) {
      const uint2 sv = lds64(src + kGgCodes + row * 32 + (((J >> 1) ^ ((row >> 2) & 1)) << 4) + (J & 1) * 8);
      f1[0] = bcast_lo(sv.x); f1[1] = bcast_hi(sv.x); f1[2] = bcast_lo(sv.y); f1[3] = bcast_hi(sv.y);
    } else if (FMT == 3) {
      const uint32_t sw = lds32(src + kGgCodes + row * 32 + J * 4);
      const uint32_t e01 = e4m3x2_to_f16x2(sw & 0xFFFFu), e23 = e4m3x2_to_f16x2(sw >> 16);
      f1[0] = bcast_lo(e01); f1[1] = bcast_hi(e01); f1[2] = bcast_lo(e23); f1[3] = bcast_hi(e23);
    } else {
      const uint32_t sw = lds32(src + kGgCodes + row * 32 + (J >> 1) * 4) >> ((J & 1) * 16);
      const uint32_t b0 = sw & 0xFFu, b1 = (sw >> 8) & 0xFFu;
      two = !(e8m0_f16_ok(b0) && e8m0_f16_ok(b1));
      e8m0_f16_factors(b0, f2[0], f1[0]);
      e8m0_f16_factors(b1, f2[2], f1[2]);
      f1[1] = f1[0]; f1[3] = f1[2]; f2[1] = f2[0]; f2[3] = f2[2];
    }
    if (!valid) f1[0] = f1[1] = f1[2] = f1[3] = 0u;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      uint32_t w4[4];
      e2m1x8_to_f16x2(q[i], w4);
      if (FMT == 4 && two) {
#pragma unroll
        for (int v = 0; v < 4; v++) w4[v] = hmul2(w4[v], f2[i >> 1]);
      }
#pragma unroll
      for (int v = 0; v < 4; v++) o[4 * i + v] = hmul2(w4[v], f1[i >> 1]);
    }
    if (FMT == 4 && two && !valid) {  // (an infinite first product times 0)
#pragma unroll
      for (int i = 0; i < 32; i++) o[i] = 0u;
    }
  }
}

// Store 32 rows of a warp's columns.  p[i] holds two columns of one row, its
// number's bits by exchange: bit 0 of the lane has been exchanged for the
// lowest bit of i.  Two more steps (lane bits 1 and 2) leave 8 columns, 4 words,
// of NR rows.  NR = 4: 32 columns, rows numbered 8i + (lane & 1) + (lane & 2) +
// (lane & 4); NR = 2: 16 columns, rows 2 (8i + ...) + (lane >> 4).
template <int NR>
__device__ __forceinline__ void gg_store(const uint32_t (&p)[4 * NR], int lane, int left, uint16_t* y, int n, int col0,
                                         bool vec) {
  uint32_t q2[2 * NR][2];  // 4 columns
#pragma unroll
  for (int i = 0; i < 2 * NR; i++) {
    const bool hi = lane & 2;
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, hi ? p[2 * i] : p[2 * i + 1], 2);
    q2[i][0] = hi ? got : p[2 * i];
    q2[i][1] = hi ? p[2 * i + 1] : got;
  }
  uint32_t q4[NR][4];  // 8 columns
#pragma unroll
  for (int i = 0; i < NR; i++) {
    const bool hi = lane & 4;
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, hi ? q2[2 * i][w] : q2[2 * i + 1][w], 4);
      q4[i][w] = hi ? got : q2[2 * i][w];
      q4[i][2 + w] = hi ? q2[2 * i + 1][w] : got;
    }
  }
  const int col = col0 + (NR == 4 ? (lane & 24) : (lane & 8));
#pragma unroll
  for (int i = 0; i < NR; i++) {
    const int r8 = 8 * i + (lane & 7);
    const int row = NR == 4 ? r8 : 2 * r8 + (lane >> 4);
    uint16_t* yp = y + (int64_t)row * n + col;
    if (vec) {
      st128_if(row < left && col < n, yp, q4[i][0], q4[i][1], q4[i][2], q4[i][3]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; c++) st16_if(row < left && col + c < n, yp + c, q4[i][c >> 1] >> (16 * (c & 1)));
    }
  }
}

template <int FMT, bool SWI>
__global__ void __launch_bounds__(kGgThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ GgArgs a) {
  using SM = GgSmem<FMT>;
  constexpr int kOutRows = SWI ? kGgRows / 2 : kGgRows;  // outputs per tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ volatile int s_abort;
  __shared__ int s_cum[kGgMaxExperts + 1];   // row tiles before expert e
  __shared__ int s_start[kGgMaxExperts], s_cnt[kGgMaxExperts];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t x_s = base + SM::kX, p_s = base + SM::kP, lut_s = base + SM::kLut, bars = base + SM::kBars;
  const uint32_t full = bars, empty = full + 8 * kGgStages, accf = empty + 8 * kGgStages, acce = accf + 24,
                 done_bar = acce + 24, cfull = done_bar + 8, cempty = cfull + 8 * kGgSlots,
                 tmem_slot = cempty + 8 * kGgSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = a.n, k = a.k;

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kGgStages; s++) {
      mbar_init(full + 8 * s, 1 + 4);  // the X copies and the four warps of a decode group
      mbar_init(empty + 8 * s, 1);       // MMA commit
    }
    for (int h = 0; h < 3; h++) {
      mbar_init(accf + 8 * h, 1);
      mbar_init(acce + 8 * h, 4);
    }
    mbar_init(done_bar, 1);
    for (int c = 0; c < kGgSlots; c++) {
      mbar_init(cfull + 8 * c, kGgCopyWarps * 32);  // every copying thread's copies landed
      mbar_init(cempty + 8 * c, kGgDecodeWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (FMT == 1) {
    const uint4* src = reinterpret_cast<const uint4*>(&g_iq_pair_table);
    for (int i = threadIdx.x; i < kIqLutBytes / 16; i += kGgThreads) {
      const uint4 v = src[i];
      sts128(lut_s + 16u * i, v.x, v.y, v.z, v.w);
    }
  }
  for (int e = threadIdx.x; e < a.E; e += kGgThreads) {
    int start;
    s_cnt[e] = group_range(a.offsets, e, a.P, start);
    s_start[e] = start;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {  // row tiles before each expert
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int v = e0 + lane < a.E ? (s_cnt[e0 + lane] + kGgTok - 1) / kGgTok : 0;
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      if (e0 + lane < a.E) s_cum[e0 + lane] = run + s - v;
      run += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) s_cum[a.E] = run;
  }
  __syncthreads();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
  const int n_tiles = (n + kOutRows - 1) / kOutRows;
  const int tiles = s_cum[a.E] * n_tiles;
  const int G = (int)gridDim.x;
  const int my_tiles = (tiles - (int)blockIdx.x + G - 1) / G;  // (0 for CTAs past the last tile)
  const int ksteps = k / kGemmBK;
  const int nck = (ksteps + kGemmChunkSteps - 1) / kGemmChunkSteps;  // chunks per tile (the last may be half)
  const int nfull = ksteps / kGemmChunkSteps;
  // A step's stage is its place in its chunk, so that a stage always belongs to
  // one decode group (half chunks leave stages 2 and 3 out): the how-manieth
  // use of its stage step ks of the li-th tile is.
  auto stage_use = [&](int li, int ks) { return (uint32_t)(li * ((ks & 3) < 2 ? nck : nfull) + (ks >> 2)); };

  auto tile_at = [&](int li) {
    const int tile = (int)blockIdx.x + li * G;
    const int mt = tile / n_tiles;
    int lo = 0, hi = a.E;  // the last e with s_cum[e] <= mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid] <= mt) lo = mid;
      else hi = mid;
    }
    GgTile t;
    t.e = lo;
    t.n0 = (tile - mt * n_tiles) * kOutRows;
    // an expert's rows in equal tiles (whole 16-row steps), not full ones and a remainder
    const int rows = s_cnt[lo], parts = s_cum[lo + 1] - s_cum[lo];
    const int per = (((rows + parts - 1) / parts) + 15) & ~15;
    const int off = (mt - s_cum[lo]) * per;
    t.m0 = s_start[lo] + off;
    t.cnt = min(per, rows - off);
    return t;
  };

  if (warp == 0) {
    // ------------------------------ X rows ---------------------------------
    if (lane == 0) {
      prefetch_tmap(&tm_x);
      uint32_t any = 0, par = 0;  // per stage: copies issued, parity of the last use
      const int tissue = (g_test_flags & kTestWithholdXTiles) ? 0 : my_tiles;  // test switch: issue nothing
      for (int li = 0; li < tissue && !s_abort; li++) {
        const GgTile t = tile_at(li);
        const int boxes = (t.cnt + 63) >> 6;
        for (int ks = 0; ks < ksteps; ks++) {
          const uint32_t s = ks & 3, use = stage_use(li, ks);
          if (!gg_wait(empty + 8 * s, (use & 1u) ^ 1u)) { s_abort = 1; break; }
          mbar_arrive_expect_tx(full + 8 * s, (uint32_t)boxes * 64u * 128u);
          for (int b = 0; b < boxes; b++)
            tma_load_2d(x_s + s * kGgXBytes + b * 64 * 128, &tm_x, ks * kGemmBK, t.m0 + 64 * b, full + 8 * s);
          any |= 1u << s;
          par = (par & ~(1u << s)) | ((use & 1u) << s);
        }
      }
      for (uint32_t s = 0; s < kGgStages; s++)  // drain our copies
        if (any >> s & 1u) gg_wait(full + 8 * s, par >> s & 1u);
    }
  } else if (warp == 1) {
    // ---------------------------- MMA issuer ------------------------------
    // The whole warp walks the loop and one lane issues: with everything an MMA
    // names computed alike in all lanes (warp_uniform: a warp reduction, whose
    // result is a uniform register) no operand has to be moved there per MMA.
    const uint32_t d0 = warp_uniform(tmem) + kGgAccCol, a0 = warp_uniform(tmem) + kGgACol;
    const uint32_t xb = warp_uniform(x_s), fb = warp_uniform(full), eb = warp_uniform(empty);
    const bool leader = elect_one();
    uint32_t used[3] = {0, 0, 0};  // tiles so far per accumulator
    for (int li = 0; li < my_tiles; li++) {
      const int cnt = (int)warp_uniform((uint32_t)tile_at(li).cnt);
      const int own = (li & 1) ? 2 : 0;  // the accumulator that is not shared with the next tile
      const bool big = cnt > 128;
      bool ok = !s_abort && gg_wait(acce + 8 * own, (used[own == 0 ? 0 : 2] & 1u) ^ 1u);
      if (big) ok = ok && gg_wait(acce + 8, (used[1] & 1u) ^ 1u);
      if (!__all_sync(0xFFFFFFFFu, ok)) { s_abort = 1; break; }
      if (own == 0) used[0]++;
      else used[2]++;
      if (big) used[1]++;
      tc_fence_after();
      const uint32_t d = d0 + (own == 0 ? 0u : big ? 128u : 256u);
      const uint32_t idesc = umma_idesc_f16((cnt + 15) & ~15);
      for (int ks = 0; ks < ksteps; ks++) {
        const uint32_t s = ks & 3;
        ok = gg_wait(fb + 8 * s, stage_use(li, ks) & 1u);
        if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; s_abort = 1; break; }
        tc_fence_after();
        const uint64_t db = umma_desc_k128(xb + s * kGgXBytes);
        const uint32_t wa = a0 + 32u * s;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kGemmBK / 16; kk++)
            umma_f16_ta(d, wa + 8u * kk, db + (uint64_t)(2 * kk), idesc, (ks | kk) != 0);
          umma_commit(eb + 8 * s);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (leader) {
        umma_commit(accf + 8 * own);
        if (big) umma_commit(accf + 8);
      }
      __syncwarp();
    }
    if (leader) umma_commit(done_bar);  // every MMA we issued has completed when this arrives
  } else if (warp < 2 + kGgCopyWarps) {
    // --------------------------- packed weights ----------------------------
    // Warp cw copies the tile's rows 64 cw .. 64 cw + 63.  IQ4_NL rows are
    // copied in units of 8 bytes (a row of k % 256 = 128 starts on 8), 18 a
    // chunk: 16 lanes take the first 16 of a row, and the rest follow by twos;
    // FP4 rows in 8 units of 16 bytes.  Rows past n copy row n - 1.
    const int cw = warp - 2;
    const int rowb = FMT == 1 ? (k >> 5) * 18 : k >> 1;
    constexpr int kScaleHalf = FMT == 2 ? 16 : FMT == 3 ? 8 : 4;  // scale bytes of 128 k
    const int srow = (k >> 7) * kScaleHalf;
    constexpr int kPer = FMT == 1 ? 2 : 4, kLanes = 32 / kPer;  // rows per instruction, lanes per row
    const int lr = lane / kLanes, u = lane % kLanes;
    // tile row 64 cw + i (i < 64, its low part may depend on the lane) as a
    // weight row; its stack with SWI is (i >> 4) & 1
    auto wrow = [&](int n0, int i) {
      return min(SWI ? n0 + 32 * cw + ((i >> 5) << 4) + (i & 15) : n0 + 64 * cw + i, n - 1);
    };
    int ck = 0;  // chunks so far
    bool ok = true;
    for (int li = 0; li < my_tiles && ok; li++) {
      const GgTile g = tile_at(li);
      const uint8_t* b0 = a.data[0] + g.e * a.dstride[0];
      const uint8_t* b1 = SWI ? a.data[1] + g.e * a.dstride[1] : b0;
      const uint8_t* s0 = FMT != 1 ? a.scales[0] + g.e * a.sstride[0] : nullptr;
      const uint8_t* s1 = FMT != 1 && SWI ? a.scales[1] + g.e * a.sstride[1] : s0;
      for (int cc = 0; cc < nck; cc++, ck++) {
        const int slot = ck % kGgSlots;
        ok = gg_wait(cempty + 8 * slot, ((uint32_t)(ck / kGgSlots) & 1u) ^ 1u);
        if (!ok) break;
        const bool whole = k - cc * 256 >= 256;  // 256 k, else the last 128
        const uint32_t dst = p_s + slot * SM::kSlot + (uint32_t)(cw * 64) * (FMT == 1 ? 144u : 128u);
        const int off = cc * (FMT == 1 ? 144 : 128);
        // blocks of 16 rows, one stack each
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const uint8_t* src = ((q & 1) ? b1 : b0) + off;
          if (FMT == 1) {
            if (whole || u < 9) {
#pragma unroll
              for (int i = 0; i < 8; i++)
                cp_async8_g(dst + (16 * q + 2 * i + lr) * 144 + u * 8,
                            src + (int64_t)wrow(g.n0, 16 * q + 2 * i + lr) * rowb + u * 8);
            }
            if (whole)
              cp_async8_g(dst + (16 * q + (lane >> 1)) * 144 + 128 + (lane & 1) * 8,
                          src + (int64_t)wrow(g.n0, 16 * q + (lane >> 1)) * rowb + 128 + (lane & 1) * 8);
          } else {
            if (whole || u < 4) {
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int r = 16 * q + 4 * i + lr;
                cp_async16_g(dst + r * 128 + ((u ^ (r & 7)) << 4), src + (int64_t)wrow(g.n0, r) * rowb + u * 16);
              }
            }
            const int h = lane & 1;  // scales: two halves of 128 k a row
            if (whole || h == 0) {
              const int r = 16 * q + (lane >> 1);
              const uint8_t* sp = ((q & 1) ? s1 : s0) + (int64_t)wrow(g.n0, r) * srow + (cc * 2 + h) * kScaleHalf;
              const uint32_t sd = p_s + slot * SM::kSlot + kGgCodes + (cw * 64 + r) * 32;
              if (FMT == 2) cp_async16_g(sd + ((h ^ ((r >> 2) & 1)) << 4), sp);
              else if (FMT == 3) cp_async8_g(sd + h * 8, sp);
              else cp_async4_g(sd + h * 4, sp);
            }
          }
        }
        cp_async_mbar_arrive_noinc(cfull + 8 * slot);
      }
    }
    if (!ok) s_abort = 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < 2 + kGgCopyWarps + kGgDecodeWarps) {
    // --------------------------- weight decode -----------------------------
    const int group = (warp - 2 - kGgCopyWarps) >> 2;  // its step of every chunk
    const int row = ((warp & 3) << 5) | lane;  // tile row = TMEM lane (a warp reaches lanes 32 (warp % 4) .. + 31)
    const uint32_t lane_tm = tmem + kGgACol + ((uint32_t)((warp & 3) * 32) << 16);
    int ck = 0;  // chunks so far
    bool ok = true;
    for (int li = 0; li < my_tiles && ok; li++) {
      const int n0 = tile_at(li).n0;
      const bool valid = (SWI ? n0 + ((row >> 5) << 4) + (row & 15) : n0 + row) < n;
      for (int cc = 0; cc < nck; cc++, ck++) {
        const int slot = ck % kGgSlots;
        ok = gg_wait_warp(cfull + 8 * slot, (uint32_t)(ck / kGgSlots) & 1u);
        if (!ok) break;
        const int steps = min(kGemmChunkSteps, ksteps - cc * kGemmChunkSteps);
        if (group < steps) {
          const uint32_t src = p_s + slot * SM::kSlot;
          uint32_t o[32];  // the step's 64 weights of this row, two per word, k order
          const uint32_t lut_lane = lut_s + 4u * (uint32_t)lane;
          if (group == 0) gg_decode<FMT, 0>(src, row, valid, lut_lane, o);
          else if (group == 1) gg_decode<FMT, 1>(src, row, valid, lut_lane, o);
          else if (group == 2) gg_decode<FMT, 2>(src, row, valid, lut_lane, o);
          else gg_decode<FMT, 3>(src, row, valid, lut_lane, o);
          const int s = group;
          ok = gg_wait(empty + 8 * s, (stage_use(li, cc * kGemmChunkSteps + group) & 1u) ^ 1u);
          ok = __all_sync(0xFFFFFFFFu, ok);  // (the stores are warp-wide)
          if (!ok) break;
          tc_fence_after();
          tmem_st32(lane_tm + 32u * (uint32_t)s, o);
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(full + 8 * s, lane);
        }
        warp_arrive(cempty + 8 * slot, lane);
      }
    }
    if (!ok) s_abort = 1;
  } else {
    // ------------------------------ epilogue ------------------------------
    // A lane holds one output column of 32 rows; lanes exchange (3 butterfly
    // steps) until each holds 8 columns of 4 rows (SWI: of 2), which is one
    // 16-byte store a row where the rows of y are 16-byte aligned.
    const int q = warp & 3;  // TMEM lanes 32q ..
    const float g0 = (FMT == 3) ? a.g[0] : 1.0f, g1 = (FMT == 3) ? a.g[1] : 1.0f;
    const bool vec = (n & 7) == 0;
    uint32_t used[3] = {0, 0, 0};
    for (int li = 0; li < my_tiles; li++) {
      const GgTile t = tile_at(li);
      const int own = (li & 1) ? 2 : 0;
      const bool big = t.cnt > 128;
      const int col0 = SWI ? t.n0 + 16 * q : t.n0 + 32 * q;  // this warp's first output column
      bool ok = true;
      for (int h = 0; h < (big ? 2 : 1); h++) {
        const int acc = (big && h == 0) ? 1 : own;             // the middle accumulator first
        const int first = (big && (acc == 1) == (own == 0)) ? 128 : 0;  // the tile's row in its column 0
        const uint32_t turn = acc == 0 ? used[0]++ : acc == 1 ? used[1]++ : used[2]++;
        ok = gg_wait(accf + 8 * acc, turn & 1u);
        if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
        tc_fence_after();
        const int c = min(128, t.cnt - first);
        for (int j = 0; j < c; j += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + kGgAccCol + 128u * acc + (uint32_t)j + ((uint32_t)(32 * q) << 16), r);
          tmem_ld_wait();
          const int64_t m = t.m0 + first + j;
          const int left = c - j;
          if (!SWI) {
            uint32_t p[16];  // after the exchange over lane bit 0: columns (lane & ~1, + 1) of row 2i + (lane & 1)
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const bool odd = lane & 1;
              const float mine = __uint_as_float(odd ? r[2 * i + 1] : r[2 * i]) * g0;
              const float other =
                  __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, odd ? r[2 * i] : r[2 * i + 1], 1)) * g0;
              p[i] = odd ? f32x2_to_f16x2(other, mine) : f32x2_to_f16x2(mine, other);
            }
            gg_store<4>(p, lane, left, a.y + m * n, n, col0, vec);
          } else {
            const bool up = (lane & 16) != 0;  // lanes 0-15 hold gate rows, 16-31 the same rows of up
            float v[16];  // row 2i + (lane >> 4) of column lane & 15
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? r[2 * i] : r[2 * i + 1], 16);
              const float zg = __uint_as_float(up ? got : r[2 * i]) * g0;
              const float zu = __uint_as_float(up ? r[2 * i + 1] : got) * g1;
              v[i] = silu_fast(zg) * zu;
            }
            uint32_t p[8];  // columns (lane & 14, + 1) of row 2 (2i + (lane & 1)) + (lane >> 4)
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const bool odd = lane & 1;
              const float mine = odd ? v[2 * i + 1] : v[2 * i];
              const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[2 * i] : v[2 * i + 1], 1);
              p[i] = odd ? f32x2_to_f16x2(other, mine) : f32x2_to_f16x2(mine, other);
            }
            gg_store<2>(p, lane, left, a.y + m * n, n, col0, vec);
          }
        }
        tc_fence_before();
        warp_arrive(acce + 8 * acc, lane);
      }
      if (!ok) { s_abort = 1; break; }
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
