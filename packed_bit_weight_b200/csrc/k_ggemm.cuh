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
//
// Roles per CTA (persistent, one per SM):
//   warp 0       X rows by TMA (64-row boxes, 128-byte swizzle), kGgStages deep
//   warp 1       tcgen05.mma issue; owns the tensor memory
//   warps 2-9    weight decode: packed chunks of 256 k arrive by cp.async in a
//                ring, warps 2-5 decode the even 64-wide steps, 6-9 the odd
//                ones (a thread then has two steps' time for one step's chain
//                of wait, decode, tcgen05.st, fence, arrive)
//   warps 10-13  epilogue: tcgen05.ld, fp16, store
// Tensor memory: kGgStages x 32 columns of weights and three accumulators of
// 128 columns; a tile takes one accumulator per 128 rows, so the next tile
// starts while the last one or two are still being stored.
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

constexpr int kGgStages = 4;
constexpr int kGgSlots = 3;                       // packed chunks of 256 k in flight
constexpr int kGgRows = 128;                      // weight rows per tile
constexpr int kGgTok = 256;                       // rows of X per tile at most
constexpr int kGgXBytes = kGgTok * kGemmBK * 2;   // 32 KB per stage
constexpr int kGgMaxExperts = 256;
constexpr int kGgThreads = (2 + kGemmDecodeWarps + 4) * 32;
constexpr int kGgCodes = kGgRows * 128;           // FP4 slot: codes [128][128 B] (unit u of row r at u ^ (r & 7))
constexpr int kGgSlotFp4 = kGgCodes + kGgRows * 32;   // then scales [128][32 B]
constexpr int kGgSlotIq4 = 9 * kGgRows * 16;      // IQ4_NL slot: [9 units][128 rows][16 B]
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
      mbar_init(full + 8 * s, 1 + 128);  // the X copies and one decode group
      mbar_init(empty + 8 * s, 1);       // MMA commit
    }
    for (int h = 0; h < 3; h++) {
      mbar_init(accf + 8 * h, 1);
      mbar_init(acce + 8 * h, 128);
    }
    mbar_init(done_bar, 1);
    for (int c = 0; c < kGgSlots; c++) {
      mbar_init(cfull + 8 * c, kGemmDecodeThreads);
      mbar_init(cempty + 8 * c, kGemmDecodeThreads);
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
      int gs = 0, issued = 0;
      const int tissue = (g_test_flags & kTestWithholdXTiles) ? 0 : my_tiles;  // test switch: issue nothing
      for (int li = 0; li < tissue && !s_abort; li++) {
        const GgTile t = tile_at(li);
        const int boxes = (t.cnt + 63) >> 6;
        for (int ks = 0; ks < ksteps; ks++, gs++) {
          const int s = gs % kGgStages;
          if (s_abort || !mbar_wait(empty + 8 * s, ((uint32_t)(gs / kGgStages) & 1u) ^ 1u)) { s_abort = 1; break; }
          mbar_arrive_expect_tx(full + 8 * s, (uint32_t)boxes * 64u * 128u);
          for (int b = 0; b < boxes; b++)
            tma_load_2d(x_s + s * kGgXBytes + b * 64 * 128, &tm_x, ks * kGemmBK, t.m0 + 64 * b, full + 8 * s);
          issued = gs + 1;
        }
      }
      for (int s = 0; s < kGgStages && s < issued; s++) {  // drain our copies
        const int last = issued - 1 - ((issued - 1 - s) % kGgStages);
        mbar_wait(full + 8 * s, (uint32_t)(last / kGgStages) & 1u);
      }
    }
  } else if (warp == 1) {
    // ---------------------------- MMA issuer ------------------------------
    if (lane == 0) {
      int gs = 0, hc = 0;  // k steps, accumulators so far
      for (int li = 0; li < my_tiles && !s_abort; li++) {
        const GgTile t = tile_at(li);
        const int halves = t.cnt > 128 ? 2 : 1;
        bool ok = true;
        for (int h = 0; h < halves; h++)
          ok = ok && mbar_wait(acce + 8 * ((hc + h) % 3), ((uint32_t)((hc + h) / 3) & 1u) ^ 1u);
        if (!ok) { s_abort = 1; break; }
        tc_fence_after();
        uint32_t d[2], idesc[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          d[h] = tmem + kGgAccCol + 128u * (uint32_t)((hc + h) % 3);
          const int c = min(128, t.cnt - 128 * h);
          idesc[h] = umma_idesc_f16((c + 15) & ~15);
        }
        for (int ks = 0; ks < ksteps; ks++, gs++) {
          const int s = gs % kGgStages;
          if (s_abort || !mbar_wait(full + 8 * s, (uint32_t)(gs / kGgStages) & 1u)) { s_abort = 1; ok = false; break; }
          tc_fence_after();
          const uint64_t db = umma_desc_k128(x_s + s * kGgXBytes);
          const uint32_t wa = tmem + kGgACol + 32u * (uint32_t)s;
#pragma unroll
          for (int h = 0; h < 2; h++) {
            if (h < halves) {
#pragma unroll
              for (int kk = 0; kk < kGemmBK / 16; kk++)
                umma_f16_ta(d[h], wa + 8u * kk, db + (uint64_t)(h * (128 * 128 / 16) + 2 * kk), idesc[h], (ks | kk) != 0);
            }
          }
          umma_commit(empty + 8 * s);
        }
        if (!ok) break;
        for (int h = 0; h < halves; h++) umma_commit(accf + 8 * ((hc + h) % 3));
        hc += halves;
      }
      umma_commit(done_bar);  // every MMA we issued has completed when this arrives
    }
  } else if (warp < 2 + kGemmDecodeWarps) {
    // --------------------------- weight decode -----------------------------
    const int t = threadIdx.x - 64;
    const int group = t >> 7;                 // decodes the steps of this parity
    const int row = ((warp & 3) << 5) | lane; // tile row = TMEM lane (a warp reaches lanes 32 (warp % 4) .. + 31)
    const int nck = (ksteps + kGemmChunkSteps - 1) / kGemmChunkSteps;  // chunks per tile (the last may be half)
    const int total_ck = my_tiles * nck;
    // source row of tile row r: the stack and the weight row (clamped to n-1)
    auto row_of = [&](const GgTile& g, int r, int& which) {
      int w = g.n0 + r;
      which = 0;
      if (SWI) {
        which = (r >> 4) & 1;
        w = g.n0 + ((r >> 5) << 4) + (r & 15);
      }
      return w;
    };
    GgTile gi = {}, gd = {};  // the tiles of the chunk being copied and of the one being decoded
    auto issue_chunk = [&](int c) -> bool {
      const int slot = c % kGgSlots;
      if (!mbar_wait(cempty + 8 * slot, ((uint32_t)(c / kGgSlots) & 1u) ^ 1u)) return false;
      if (c % nck == 0) gi = tile_at(c / nck);
      const GgTile& g = gi;
      const int kc = (c % nck) * (kGemmChunkSteps * kGemmBK);
      const bool whole = k - kc >= kGemmChunkSteps * kGemmBK;  // 256 k, else 128
      const uint32_t dst = p_s + slot * SM::kSlot;
      if (FMT == 1) {  // 18-byte blocks: 144 (72) bytes a row; rows start on 8 bytes at least
        const int64_t rowb = (int64_t)(k >> 5) * 18;
        const int64_t off = (int64_t)(kc >> 5) * 18;
        if ((k & 255) == 0) {
#pragma unroll
          for (int i = 0; i < (9 * kGgRows + kGemmDecodeThreads - 1) / kGemmDecodeThreads; i++) {
            const int pc = i * kGemmDecodeThreads + t;
            if (pc >= 9 * kGgRows) break;
            const int r = pc / 9, u = pc - r * 9;
            int which;
            const int64_t w = min(row_of(g, r, which), n - 1);
            cp_async16_g(dst + u * (kGgRows * 16) + r * 16, a.data[which] + g.e * a.dstride[which] + w * rowb + off + u * 16);
          }
        } else {
          const int units = whole ? 18 : 9;  // of 8 bytes
          for (int pc = t; pc < units * kGgRows; pc += kGemmDecodeThreads) {
            const int r = pc / units, u = pc - r * units;
            int which;
            const int64_t w = min(row_of(g, r, which), n - 1);
            cp_async8_g(dst + (u >> 1) * (kGgRows * 16) + r * 16 + (u & 1) * 8,
                        a.data[which] + g.e * a.dstride[which] + w * rowb + off + u * 8);
          }
        }
      } else {
        const int units = whole ? 8 : 4, sh = whole ? 3 : 2;  // codes: 16-byte units of a row
        for (int pc = t; pc < units * kGgRows; pc += kGemmDecodeThreads) {
          const int r = pc >> sh, u = pc & (units - 1);
          int which;
          const int64_t w = min(row_of(g, r, which), n - 1);
          cp_async16_g(dst + r * 128 + ((u ^ (r & 7)) << 4),
                       a.data[which] + g.e * a.dstride[which] + w * (int64_t)(k >> 1) + (kc >> 1) + u * 16);
        }
        // scales: two halves of 128 k a row, of 16 (fp16), 8 (E4M3) or 4 bytes (E8M0)
        const int r = t >> 1, h = t & 1;
        if (whole || h == 0) {
          int which;
          const int64_t w = min(row_of(g, r, which), n - 1);
          const uint8_t* sp = a.scales[which] + g.e * a.sstride[which];
          const uint32_t sd = dst + kGgCodes + r * 32;
          if (FMT == 2)
            cp_async16_g(sd + ((h ^ ((r >> 2) & 1)) << 4), sp + (w * (int64_t)(k >> 4) + (kc >> 4)) * 2 + h * 16);
          else if (FMT == 3)
            cp_async8_g(sd + h * 8, sp + w * (int64_t)(k >> 4) + (kc >> 4) + h * 8);
          else
            cp_async4_g(sd + h * 4, sp + w * (int64_t)(k >> 5) + (kc >> 5) + h * 4);
        }
      }
      cp_async_mbar_arrive_noinc(cfull + 8 * slot);
      return true;
    };
    bool stop = false;
    for (int c = 0; c < kGgSlots - 1 && c < total_ck && !stop; c++) stop = !issue_chunk(c);
    int step0 = 0;  // global step number of the chunk's first step
    for (int c = 0; c < total_ck && !stop; c++) {
      if (c + kGgSlots - 1 < total_ck && !issue_chunk(c + kGgSlots - 1)) { s_abort = 1; break; }
      const int slot = c % kGgSlots;
      if (s_abort || !mbar_wait(cfull + 8 * slot, (uint32_t)(c / kGgSlots) & 1u)) { s_abort = 1; break; }
      if (c % nck == 0) gd = tile_at(c / nck);
      int which;
      const bool valid = row_of(gd, row, which) < n;
      const int steps = min(kGemmChunkSteps, ksteps - (c % nck) * kGemmChunkSteps);
      const uint32_t src = p_s + slot * SM::kSlot;
#pragma unroll
      for (int j = 0; j < kGemmChunkSteps; j++) {
        if (j >= steps) break;
        const int gs = step0 + j;
        if ((gs & 1) != group) continue;
        uint32_t o[32];  // the step's 64 weights of this row, two per word, k order
        if (FMT == 1) {
          // two blocks: 36 bytes from byte 36j of the row, in its units 2j .. 2j+2
          uint32_t uw[12];
#pragma unroll
          for (int u = 0; u < 3; u++) {
            const uint4 v = lds128(src + (2 * j + u) * (kGgRows * 16) + row * 16);
            uw[4 * u] = v.x; uw[4 * u + 1] = v.y; uw[4 * u + 2] = v.z; uw[4 * u + 3] = v.w;
          }
          uint32_t w[9];
#pragma unroll
          for (int i = 0; i < 9; i++) w[i] = uw[i + j];  // (j is a constant: the loop is unrolled)
          uint32_t qa[4], qb[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            qa[i] = __funnelshift_r(w[i], w[i + 1], 16);
            qb[i] = w[5 + i];
          }
          uint32_t da = w[0] & 0xFFFFu, db = w[4] >> 16;
          da = valid ? (da | (da << 16)) : 0u;
          db = valid ? (db | (db << 16)) : 0u;
          const uint32_t lut_lane = lut_s + 4u * (uint32_t)lane;
          uint32_t oa[16], ob[16];
          iq4_block_chunks<7>(qa, da, lut_lane, oa);
          iq4_block_chunks<7>(qb, db, lut_lane, ob);
#pragma unroll
          for (int i = 0; i < 16; i++) { o[i] = oa[i]; o[16 + i] = ob[i]; }
        } else {
          uint32_t q[8];
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const uint4 v = lds128(src + row * 128 + (((2 * j + u) ^ (row & 7)) << 4));
            q[4 * u] = v.x; q[4 * u + 1] = v.y; q[4 * u + 2] = v.z; q[4 * u + 3] = v.w;
          }
          uint32_t f1[4], f2[4];  // per 16 k: the scale, and for wide E8M0 scales a second factor
          bool two = false;
          if (FMT == 2) {
            const uint2 sv = lds64(src + kGgCodes + row * 32 + (((j >> 1) ^ ((row >> 2) & 1)) << 4) + (j & 1) * 8);
            f1[0] = bcast_lo(sv.x); f1[1] = bcast_hi(sv.x); f1[2] = bcast_lo(sv.y); f1[3] = bcast_hi(sv.y);
          } else if (FMT == 3) {
            const uint32_t sw = lds32(src + kGgCodes + row * 32 + j * 4);
            const uint32_t e01 = e4m3x2_to_f16x2(sw & 0xFFFFu), e23 = e4m3x2_to_f16x2(sw >> 16);
            f1[0] = bcast_lo(e01); f1[1] = bcast_hi(e01); f1[2] = bcast_lo(e23); f1[3] = bcast_hi(e23);
          } else {
            const uint32_t sw = lds32(src + kGgCodes + row * 32 + (j >> 1) * 4) >> ((j & 1) * 16);
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
        const int s = gs % kGgStages;
        const bool ok = !s_abort && mbar_wait(empty + 8 * s, ((uint32_t)(gs / kGgStages) & 1u) ^ 1u);
        if (!__all_sync(0xFFFFFFFFu, ok)) { s_abort = 1; stop = true; break; }  // (the stores are warp-wide)
        tc_fence_after();
        tmem_st32(tmem + kGgACol + 32u * (uint32_t)s + ((uint32_t)((warp & 3) * 32) << 16), o);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(full + 8 * s);
      }
      step0 += steps;
      mbar_arrive(cempty + 8 * slot);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------ epilogue ------------------------------
    const int q = warp & 3;  // TMEM lanes 32q ..
    const float g0 = (FMT == 3) ? a.g[0] : 1.0f, g1 = (FMT == 3) ? a.g[1] : 1.0f;
    int hc = 0;
    for (int li = 0; li < my_tiles; li++) {
      const GgTile t = tile_at(li);
      const int halves = t.cnt > 128 ? 2 : 1;
      const int col = SWI ? t.n0 + 16 * q + (lane & 15) : t.n0 + 32 * q + lane;  // this lane's output column
      bool ok = true;
      for (int h = 0; h < halves; h++, hc++) {
        const int acc = hc % 3;
        ok = !s_abort && mbar_wait(accf + 8 * acc, (uint32_t)(hc / 3) & 1u);
        if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
        tc_fence_after();
        const int c = min(128, t.cnt - 128 * h);
        for (int j = 0; j < c; j += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + kGgAccCol + 128u * acc + (uint32_t)j + ((uint32_t)(32 * q) << 16), r);
          tmem_ld_wait();
          const int64_t m = t.m0 + 128 * h + j;
          uint16_t* yp = a.y + m * n + col;
          const int left = c - j;
          if (!SWI) {
#pragma unroll
            for (int i = 0; i < 32; i++)
              if (i < left && col < n) yp[(int64_t)i * n] = f32_to_f16_bits(__uint_as_float(r[i]) * g0);
          } else {
            const bool up = (lane & 16) != 0;  // lanes 0-15 hold gate rows, 16-31 the same rows of up
#pragma unroll
            for (int i = 0; i < 32; i += 2) {  // gate lanes take token i, up lanes token i + 1
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? r[i] : r[i + 1], 16);
              const float zg = __uint_as_float(up ? got : r[i]) * g0, zu = __uint_as_float(up ? r[i + 1] : got) * g1;
              const int tok = i + (up ? 1 : 0);
              if (tok < left && col < n) yp[(int64_t)tok * n] = f32_to_f16_bits(zg / (1.0f + expf(-zg)) * zu);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(acce + 8 * acc);
      }
      if (!ok) { s_abort = 1; break; }
    }
  }

  // teardown: no MMA of ours may still be using tensor memory
  if (warp == 1 && lane == 0) mbar_wait(done_bar, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace qmm
