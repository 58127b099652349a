// mx_gemm16.cu -- GEMM on BF16 / FP16 operands for sm_100a, dense (batched),
// grouped along M with ragged groups, and grouped along K with ragged groups.
//
// Two kernels compute the same thing (mx_gemm16.cuh):
//
//  g16_pair_kernel  two CTAs of a cluster share a 256 x 256 tile of D
//    (tcgen05.mma cta_group::2, 128 rows of A and of B in each CTA's shared
//    memory), persistent, the accumulator double-buffered in TMEM so that the
//    epilogue of one tile runs beside the MMAs of the next.
//      warp 0      TMA producer (both CTAs): 64 elements of K per stage
//      warp 1      MMA issuer (leader), K = 16 per instruction
//      warps 2-9   epilogue: two warps per TMEM lane quarter, 128 columns each
//                  (linear and poly: warps 2-17, four per quarter, 64 columns each)
//      warp 10     ragged K only (both CTAs): clears the rows of the stage that
//                  lie behind the group's last token before the MMAs read them
//    (Times here and below: captured graphs on a card that has rested.  A call outside a
//    graph adds the host's part to small ones, loops of seconds the power limit to large ones.)
//    Bound by the tensor cores: 8192x4096x4096 in 178 us (1550 TFLOP/s; in loops of
//    seconds the card's power holds it to 1310, as it does the library product);
//    with GELU and the pre-activation the tensor pipe is active 82 % of the time.
//    Where K is short the epilogue bounds it: 16384x4096x256 46 us plain, 52 with bias,
//    80 with bias and GELU, 81 with bias and residual.
//    Sums longer than an accumulator may take (kSumWhole) have a form of their own
//    (kEpiLong; the small kernel's LONG), which adds the parts in registers (there: in
//    TMEM): 2048x2048x32768 182 us against 181 in one accumulator, 64x2112x65536 64 against
//    63, the 16-bit weight gradient of 65536 rows over 32 experts (7168x2048) equal.
//
//  g16_small_kernel  one CTA per 128 x 128 tile, K split over a cluster of 1, 2,
//    4 or 8 CTAs whose partial sums meet in distributed shared memory (in a
//    fixed order), two CTAs to an SM.  For products that would leave most SMs
//    idle in 256 x 256 tiles, where the operands' bytes bound the time: 512 rows
//    over 32 experts of 4096x7168 read 1.88 GB in 305 us, 6170 GB/s, what a copy of as
//    many bytes takes (called with inputs not in L2: 344 us, 5480).  The smallest are bound by latency: of a lone 128x128x64
//    tile's 3.8 us (plain) 2.1 are the launch's and 1.0 the operands' and the MMAs';
//    64x2112x7168 by 4 takes 12.6 us, its bytes 4.8.
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "mx_gemm16.cuh"
#include "mx_launch.h"

namespace mxk {

// ======================================================================= CTA-pair kernel

// Epilogue warps: the arithmetic of the linear and poly epilogues (an activation is
// some 20 instructions a value) wants four to a scheduler; plain and sum keep 8 with
// more registers.  One more warp clears rows (ragged K, plain and sum only).
__host__ __device__ constexpr int p16_epi_warps(int epi) { return epi == kEpiLinear || epi == kEpiPoly ? 16 : 8; }
__host__ __device__ constexpr int p16_threads(int epi) {
  return 32 * (2 + p16_epi_warps(epi) + (p16_epi_warps(epi) == 16 ? 0 : 1));
}
constexpr int kP16TM = 256, kP16TN = 256;
constexpr int kP16K = 64;     // elements of K per stage
// K of one accumulator (FP32 results show what it truncates long before 16-bit ones do)
__host__ __device__ constexpr int p16_part(int epi, int kn) {
  return epi == kEpiSum ? 512 : epi == kEpiLong && kn > kSumWhole ? kSumPart : kn;
}

// 16 epilogue warps take a stage's place for their staging tiles, where the
// residual's (or C's) rows wait for the sum (five stages cost about 1 % of a long
// product).
template <int EPI>
struct P16Layout {
  static constexpr int STAGES = p16_epi_warps(EPI) == 16 ? 5 : 6;
  static constexpr int WARPS = p16_epi_warps(EPI);
  static constexpr int OP_BYTES = 128 * 128;        // 16 KB: one operand's half tile of a stage
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + STAGES * OP_BYTES;
  static constexpr int OFF_STG = OFF_B + STAGES * OP_BYTES;
  static constexpr int STG_BYTES = 32 * 128;        // a staging tile: 32 rows of 128 bytes
  static constexpr int OFF_BAR = OFF_STG + WARPS * STG_BYTES;
  // full, empty, tail landed, tail cleared per stage; accumulator full and empty
  // (2 each); drain; residual landed per epilogue warp
  static constexpr int NUM_BARS = 4 * STAGES + 5 + WARPS;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_TAB = OFF_MISC + 16;
  static constexpr int BYTES = OFF_TAB + (kMaxGroups / kTabStep + 1) * 4;
  static constexpr int ALLOC = BYTES + 1024;
  static_assert(OFF_STG % 1024 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(ALLOC <= 232448, "shared memory budget");
};

template <int EPI>
__global__ void __launch_bounds__(p16_threads(EPI), 1)
    g16_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_d, const __grid_constant__ CUtensorMap tmap_z,
                    const __grid_constant__ CUtensorMap tmap_r, const G16Args args) {
  using L = P16Layout<EPI>;
  constexpr int S = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x) >> 1;
  const int npairs = static_cast<int>(gridDim.x) >> 1;
  const bool ragged_k = args.mode == kRaggedK;

  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile uint32_t* tmem_slot = misc + 0;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + L::OFF_TAB);

  auto full_bar = [&](int s) { return sbase + L::OFF_BAR + 8u * s; };
  auto empty_bar = [&](int s) { return sbase + L::OFF_BAR + 8u * (S + s); };
  auto tail_bar = [&](int s) { return sbase + L::OFF_BAR + 8u * (2 * S + s); };
  auto ready_bar = [&](int s) { return sbase + L::OFF_BAR + 8u * (3 * S + s); };
  auto accf_bar = [&](int b) { return sbase + L::OFF_BAR + 8u * (4 * S + b); };
  auto acce_bar = [&](int b) { return sbase + L::OFF_BAR + 8u * (4 * S + 2 + b); };
  const uint32_t drain_bar = sbase + L::OFF_BAR + 8u * (4 * S + 4);
  auto res_bar = [&](int w) { return sbase + L::OFF_BAR + 8u * (4 * S + 5 + w); };
  // ragged K: does a stage with `left` of the group's K end inside an MMA's 16,
  // so that the rows behind it have to be cleared?  Such a stage lands on each
  // CTA's own tail barrier, its warp 10 clears the rows and arrives on the
  // leader's ready barrier; every other stage goes straight to the MMA issuer.
  auto needs_clearing = [&](int left) { return ragged_k && left < kP16K && (left & 15) != 0; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);   // one arrival that announces the bytes
      mbar_init(empty_bar(s), 1);  // the leader's commit, multicast to both CTAs
      mbar_init(tail_bar(s), 1);
      mbar_init(ready_bar(s), 2);  // one arrival from each CTA's warp 10, on the leader
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * L::WARPS);  // one lane of each epilogue warp of both CTAs, on the leader
    }
    mbar_init(drain_bar, 1);
    for (int w = 0; w < L::WARPS; ++w) mbar_init(res_bar(w), 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    prefetch_tmap(&tmap_d);
  }
  pdl_launch_dependents();
  pdl_wait_prior();

  int bad = 0;
  if (args.mode != kBatched) {
    bad = g16_offsets_bad(args, args.mode == kRaggedM ? args.m : args.k);
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0 && rank == 0) report(args.status, 0x1);
    if (args.mode == kRaggedM && warp == 0) g16_prefix<kP16TM>(args, tab, bad, &misc[2]);
  }
  __syncthreads();
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish_pair();
  }
  // barriers initialised and TMEM allocated in BOTH CTAs before any cross-CTA traffic
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = bad                      ? 0
                    : args.mode == kRaggedM ? static_cast<int>(misc[2])
                                            : args.groups * g16_tiles_per_entry(args);

  if (warp == 0) {
    if (elect_one()) {
      // ===== TMA producer.  Both CTAs' loads complete on the leader's full
      // barrier, or (needs_clearing) on the CTA's own tail barrier.
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, uint32_t dst, uint32_t bar, int mn_major, int wide, int mn, int k, int z) {
        if (!mn_major) {
          tma_load_3d_pair(dst, map, bar, k, mn, z);
        } else if (wide) {
          tma_load_4d_pair(dst, map, bar, 0, k, mn / 64, z);
        } else {
          tma_load_3d_pair(dst, map, bar, mn, k, z);
          tma_load_3d_pair(dst + 8192, map, bar, mn + 64, k, z);
        }
      };
      for (int t = pair; t < total && ok; t += npairs) {
        const G16Tile tl = g16_decode<kP16TM>(args, tab, t);
        const int a_mn0 = tl.row0 + 128 * static_cast<int>(rank);
        const int b_mn0 = tl.nb * kP16TN + 128 * static_cast<int>(rank);
        const int a_z = args.mode == kBatched ? tl.group : 0;
        const int b_z = args.b_per_group ? tl.group : 0;
        int k0, kn;
        g16_k_range(args, tl.group, k0, kn);
        for (int kk = 0; kk < kn; kk += kP16K) {
          if (!wait16<false>(empty_bar(stage), phase ^ 1u, abort_flag, args.wait_ns)) { ok = false; break; }
          uint32_t bar = map_to_rank(full_bar(stage), 0);
          if (needs_clearing(kn - kk)) {
            bar = map_to_rank(tail_bar(stage), rank);
            mbar_arrive_expect_tx(tail_bar(stage), 2 * L::OP_BYTES);
            if (rank == 0) mbar_arrive(full_bar(stage));  // a phase that nobody waits for
          } else if (rank == 0) {
            mbar_arrive_expect_tx(full_bar(stage), 4 * L::OP_BYTES);
          }
          load(&tmap_a, sbase + L::OFF_A + stage * L::OP_BYTES, bar, args.a_mn, args.a_wide, a_mn0, k0 + kk, a_z);
          load(&tmap_b, sbase + L::OFF_B + stage * L::OP_BYTES, bar, args.b_mn, args.b_wide, b_mn0, k0 + kk, b_z);
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // loads already in flight land during the teardown's linger
        report(args.status, 0x4);
        *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ===== MMA issuer: up to 4 pair MMAs of K = 16 per stage.  Accumulator
      // buffer `it & 1` takes a tile's sum, or (kEpiSum, kEpiLong) that of a part of its K.
      const uint32_t idesc = idesc_f16(kP16TM, kP16TN, args.op_fp16, args.a_mn, args.b_mn);
      const uint64_t da0 = args.a_mn ? desc_mnmajor_sw128(sbase + L::OFF_A, 8192) : desc_kmajor_sw128(sbase + L::OFF_A);
      const uint64_t db0 = args.b_mn ? desc_mnmajor_sw128(sbase + L::OFF_B, 8192) : desc_kmajor_sw128(sbase + L::OFF_B);
      const uint64_t da_step = args.a_mn ? 128 : 2, db_step = args.b_mn ? 128 : 2;  // 16 of K, in 16-byte units
      int stage = 0;
      uint32_t phase = 0, tail_phase = 0;  // tail_phase: a bit per stage
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        int k0, kn;
        g16_k_range(args, g16_decode<kP16TM>(args, tab, t).group, k0, kn);
        if (kn == 0) continue;  // the epilogue writes zeros by itself
        int kk = 0;
        do {
          const uint32_t buf = it & 1u;
          if (!wait16<true>(acce_bar(buf), ((it >> 1) & 1u) ^ 1u, abort_flag, args.wait_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t acc = tmem_base + buf * kP16TN;
          const int part = p16_part(EPI, kn);
          const int k_end = kn - kk > part ? kk + part : kn;
          uint32_t accumulate = 0;
          for (; kk < k_end; kk += kP16K) {
            if (needs_clearing(kn - kk)) {
              ok = wait16<true>(ready_bar(stage), (tail_phase >> stage) & 1u, abort_flag, args.wait_ns);
              tail_phase ^= 1u << stage;
            } else {
              ok = wait16<false>(full_bar(stage), phase, abort_flag, args.wait_ns);
            }
            if (!ok) break;
            const uint64_t da = da0 + static_cast<uint64_t>(stage * (L::OP_BYTES >> 4));
            const uint64_t db = db0 + static_cast<uint64_t>(stage * (L::OP_BYTES >> 4));
            // what is behind K's end is zeros or not this group's: left out
            const int steps = kn - kk >= kP16K ? 4 : (kn - kk + 15) >> 4;
            if (steps == 4) {
              tc_mma_pair_f16(acc, da, db, idesc, accumulate);
              tc_mma_pair_f16(acc, da + da_step, db + db_step, idesc, 1);
              tc_mma_pair_f16(acc, da + 2 * da_step, db + 2 * db_step, idesc, 1);
              tc_mma_pair_f16(acc, da + 3 * da_step, db + 3 * db_step, idesc, 1);
            } else {
              for (int s = 0; s < steps; ++s) tc_mma_pair_f16(acc, da + s * da_step, db + s * db_step, idesc, s | accumulate);
            }
            accumulate = 1;
            tc_commit_pair_multicast(empty_bar(stage), 0x3);
            if (++stage == S) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          tc_commit_pair_multicast(accf_bar(buf), 0x3);
          ++it;
        } while (kk < kn);
      }
      if (!ok) {
        report(args.status, 0x4);
        *abort_flag = 1;
      }
      // every pair MMA issued must finish before either CTA frees its TMEM
      tc_commit_pair_multicast(drain_bar, 0x1);
      wait16<false>(drain_bar, 0, nullptr, 100000000ull);
    }
  } else if (warp == 2 + L::WARPS) {
    if (ragged_k) {
      // ===== the K rows behind a group's last token belong to the next group:
      // cleared up to the end of the MMAs' last step of 16 in both operands, so
      // that whatever they hold (infinities included) adds nothing
      uint32_t next = 0, tail_phase = 0;  // stage of the next tile's first; a phase bit per stage
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        int k0, kn;
        g16_k_range(args, g16_decode<kP16TM>(args, tab, t).group, k0, kn);
        if (kn == 0) continue;
        const uint32_t stages = static_cast<uint32_t>((kn + kP16K - 1) / kP16K);
        const uint32_t stage = (next + stages - 1) % S;
        next = (next + stages) % S;
        const int left = kn - (static_cast<int>(stages) - 1) * kP16K;
        if (!needs_clearing(left)) continue;
        ok = wait16<false>(tail_bar(stage), (tail_phase >> stage) & 1u, abort_flag, args.wait_ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
        tail_phase ^= 1u << stage;
        const int rows = 16 - (left & 15);
        // 4 tiles (A's and B's two chunks of 64 columns) x rows x 8 pieces of 16 bytes
        for (int i = lane; i < 4 * rows * 8; i += 32) {
          const int piece = i & 7, row = (i >> 3) % rows, tile = (i >> 3) / rows;
          const uint32_t at = sbase + (tile < 2 ? L::OFF_A : L::OFF_B) + stage * L::OP_BYTES + (tile & 1) * 8192 +
                              (left + row) * 128 + piece * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(ready_bar(stage), 0));
      }
      if (!ok && lane == 0) {
        report(args.status, 0x4);
        *abort_flag = 1;
      }
    }
  } else {
    // ===== epilogue: rows of the warp's TMEM lane quarter, one half of the columns
    const int ew = warp - 2;
    const int quarter = warp & 3;
    const int half = ew >> 2;  // which of the column groups
    const uint32_t stg = sbase + L::OFF_STG + ew * L::STG_BYTES;
    uint32_t res_phase = 0;
    bool zeros = false;  // the staging tile holds zeros
    const int h = args.out_type == 1;
    uint32_t it = 0;
    bool ok = true;
    // 32 words of each of the warp's rows through its staging tile (128-byte
    // swizzle); the store before must have read it
    auto send = [&](const CUtensorMap* map, int x, int y, int z) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(map, stg, x, y, z);
        bulk_commit_group();
      }
    };
    auto put = [&](const CUtensorMap* map, const uint32_t* w, int x, int y, int z) {
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t off = lane * 128 + ((j ^ (lane & 7)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + off), "r"(w[4 * j]), "r"(w[4 * j + 1]),
                     "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
      }
      send(map, x, y, z);
    };
    // the accumulator's next buffer is full; false (on every lane) if the wait ran out
    auto wait_full = [&]() -> bool {
      // (a part of a long sum is there before 32 attempts have failed)
      const bool got = wait16<false, EPI == kEpiLong ? 2 : 32>(accf_bar(it & 1u), (it >> 1) & 1u, abort_flag, args.wait_ns);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) {
          report(args.status, 0x4);
          *abort_flag = 1;
        }
        return false;
      }
      tc_fence_after();
      return true;
    };
    // this warp has read the buffer
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(acce_bar(it & 1u), 0));
      ++it;
    };
    for (int t = pair; t < total && ok; t += npairs) {
      const G16Tile tl = g16_decode<kP16TM>(args, tab, t);
      int k0, kn;
      g16_k_range(args, tl.group, k0, kn);
      const int row_w = tl.row0 + 128 * static_cast<int>(rank) + 32 * quarter;  // the warp's first row
      const int row = row_w + lane;
      constexpr int WCOLS = 1024 / L::WARPS;                                    // columns of a warp
      const int col_w = tl.nb * kP16TN + half * WCOLS;                          // and column
      const bool valid = row < tl.rows_end;
      const bool mine = row_w < tl.rows_end && col_w < args.n;  // anything to store
      // TMA clips rows behind the tensor's last but not behind a group's
      const bool tma = args.mode != kRaggedM || row_w + 32 <= tl.rows_end;
      const int z_out = args.mode == kRaggedM ? 0 : tl.group;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * WCOLS;
      if constexpr (EPI == kEpiPlain || EPI == kEpiSum || EPI == kEpiLong) {
        if (kn == 0) {  // a group without tokens: zeros from the staging tile, no accumulator
          if (mine) {
            if (!zeros) {
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stg + j * 512 + lane * 16), "r"(0) : "memory");
              fence_proxy_async_smem();
              __syncwarp();
              zeros = true;
            }
            if (lane == 0) {
              constexpr int COLS = EPI == kEpiSum ? 32 : 64;
              for (int c = 0; c < WCOLS && col_w + c < args.n; c += COLS) tma_store_3d(&tmap_d, stg, col_w + c, row_w, z_out);
              bulk_commit_group();
            }
          }
          continue;
        }
        zeros = false;
      }
      // one accumulator has the whole sum: 64 columns at a time
      auto plain = [&]() {
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          const int col0 = col_w + c;
          if (!mine || col0 >= args.n) {
            if (c == 64) release();
            continue;
          }
          float v[64];
          __syncwarp();  // TMEM loads are the whole warp's
          {
            uint32_t raw[2][32];
            tc_ld_32x32b_x32(t_row + (it & 1u) * kP16TN + c, raw[0]);
            tc_ld_32x32b_x32(t_row + (it & 1u) * kP16TN + c + 32, raw[1]);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(raw[j / 32][j % 32]);
          }
          if (c == 64) release();
          if (tma) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = pack16(v[2 * j], v[2 * j + 1], h);
            put(&tmap_d, w, col0, row_w, z_out);
          } else if (valid) {
            g16_store_row<64>(args, args.d, v, tl.group, row, col0, args.n);
          }
        }
      };
      const int part = p16_part(EPI, kn);
      if (EPI == kEpiLong && part >= kn && args.epi == kEpiPlain) {  // a short group among long ones
        ok = wait_full();
        if (!ok) break;
        plain();
        continue;
      }
      if constexpr (EPI == kEpiSum || EPI == kEpiLong) {
        // long sums: the tensor core's accumulator truncates, so each part of K goes
        // into one of its own, and these are added here, rounded
        float sum[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
        for (int kk = 0; kk < kn; kk += part) {
          ok = wait_full();
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t raw[16];
            tc_ld_32x32b_x16(t_row + (it & 1u) * kP16TN + c * 16, raw);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c * 16 + j] += __uint_as_float(raw[j]);
          }
          release();
        }
        if (!ok) break;
        if constexpr (EPI == kEpiSum) {
          if (mine) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (col_w + c * 32 < args.n)
                put(&tmap_d, reinterpret_cast<const uint32_t*>(sum) + c * 32, col_w + c * 32, row_w, z_out);
          }
        } else if (mine && args.epi == kEpiPlain && tma) {
#pragma unroll
          for (int c = 0; c < 128; c += 64) {
            if (col_w + c < args.n) {
              uint32_t w[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) w[j] = pack16(sum[c + 2 * j], sum[c + 2 * j + 1], h);
              put(&tmap_d, w, col_w + c, row_w, z_out);
            }
          }
        } else if (mine) {
          // the other epilogues, 32 columns at a time by plain loads and stores: next to
          // a long sum they are nothing
          const float scale = args.epi == kEpiPoly ? g16_scale(args, tl.group) : 1.0f;
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            const int col0 = col_w + c;
            if (col0 < args.n) {
              float v[32];
              uint4 res[4], low[4];
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = sum[c + j];
              g16_load_res<32>(args, args.res, tl.group, row, col0, args.n, valid, res);
              if (args.epi == kEpiLinear) {
                if (args.bias != nullptr) {
                  uint32_t bias2 = 0;
                  if (lane < 16 && col0 + 2 * lane < args.n)
                    bias2 = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(args.bias) + col0) + lane);
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    const float2 b = unpack16(__shfl_sync(0xFFFFFFFFu, bias2, j), args.op_fp16);
                    v[2 * j] += b.x;
                    v[2 * j + 1] += b.y;
                  }
                }
                if (args.z != nullptr && valid) g16_store_row<32>(args, args.z, v, tl.group, row, col0, args.n);
                g16_activate<32>(args, v, res);
              } else if (args.epi == kEpiPoly) {
                g16_load_res<32>(args, args.res_lo, tl.group, row, col0, args.n, valid, low);
                g16_epilogue<kEpiPoly, 32>(args, v, res, low, nullptr, tl.group, row, col0, scale);
                if (args.sym && tl.mb != tl.nb) g16_store_mirror<32>(args, v, tl.group, row, col0, args.n, valid);
              }
              if (valid) g16_store_row<32>(args, args.d, v, tl.group, row, col0, args.n);
              if (args.epi == kEpiPoly && args.z != nullptr && valid) {
                g16_remainder<32>(args, v);
                g16_store_row<32>(args, args.z, v, tl.group, row, col0, args.n);
              }
            }
          }
        }
      } else if constexpr (EPI == kEpiPlain) {
        ok = wait_full();
        if (!ok) break;
        plain();
      } else {
        // 64 columns a warp, 32 at a time.  The rows of the residual or C come into the
        // staging tile by TMA, while the MMAs run if they can, and the result takes
        // their place.
        const bool has_res = args.res != nullptr && mine;
        auto tile_free = [&]() {  // the last store has read the staging tile
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        };
        auto fetch_res = [&]() {
          if (lane == 0) {
            bulk_wait_group_read<0>();
            mbar_arrive_expect_tx(res_bar(ew), L::STG_BYTES);
            tma_load_3d(stg, &tmap_r, res_bar(ew), col_w, row_w, tl.group);
          }
        };
        auto wait_res = [&]() -> bool {
          const bool got = wait16<false>(res_bar(ew), res_phase, abort_flag, args.wait_ns);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            if (lane == 0) {
              report(args.status, 0x4);
              *abort_flag = 1;
            }
            return false;
          }
          res_phase ^= 1u;
          return true;
        };
        // 32 columns from `c` of the warp's 64: the accumulator, and this lane's row of the tile
        auto acc32 = [&](int c, float (&v)[32]) {
          uint32_t raw[32];
          __syncwarp();  // TMEM loads are the whole warp's
          tc_ld_32x32b_x32(t_row + (it & 1u) * kP16TN + c, raw);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
        };
        auto at8 = [&](int c) { return stg + lane * 128 + (((c / 8) ^ (lane & 7)) << 4); };
        auto staged32 = [&](int c, uint4 (&w)[4]) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[q].x), "=r"(w[q].y), "=r"(w[q].z), "=r"(w[q].w)
                         : "r"(at8(c + q * 8))
                         : "memory");
        };
        auto stage32 = [&](int c, const uint4 (&w)[4]) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at8(c + q * 8)), "r"(w[q].x), "r"(w[q].y),
                         "r"(w[q].z), "r"(w[q].w)
                         : "memory");
        };
        auto pack32 = [&](const float (&v)[32], uint4 (&w)[4]) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = make_uint4(pack16(v[8 * q], v[8 * q + 1], h), pack16(v[8 * q + 2], v[8 * q + 3], h),
                              pack16(v[8 * q + 4], v[8 * q + 5], h), pack16(v[8 * q + 6], v[8 * q + 7], h));
        };
        if constexpr (EPI == kEpiLinear) {
          // the bias of the warp's 64 columns, two a lane, fetched while the MMAs run
          uint32_t bias2 = 0;
          if (args.bias != nullptr && col_w + 2 * lane < args.n)
            bias2 = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(args.bias) + col_w) + lane);
          auto pre32 = [&](int c, float (&v)[32]) {  // the pre-activation
            acc32(c, v);
            if (args.bias != nullptr) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 b = unpack16(__shfl_sync(0xFFFFFFFFu, bias2, c / 2 + j), args.op_fp16);
                v[2 * j] += b.x;
                v[2 * j + 1] += b.y;
              }
            }
          };
          if (has_res && args.z == nullptr) fetch_res();
          ok = wait_full();
          if (!ok) break;
          if (mine && args.z != nullptr) {
            // a pre-activation that is wanted takes a pass of its own over the
            // accumulator, so that one staging tile does
            tile_free();
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
              float v[32];
              uint4 w[4];
              pre32(c, v);
              pack32(v, w);
              stage32(c, w);
            }
            send(&tmap_z, col_w, row_w, 0);
            if (has_res) fetch_res();
          }
          if (has_res) {
            ok = wait_res();
            if (!ok) break;
          } else {
            tile_free();
          }
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            if (mine) {
              float v[32];
              uint4 w[4];
              pre32(c, v);
              if (c == 32) release();
              if (has_res) staged32(c, w);
              g16_activate<32>(args, v, w);
              pack32(v, w);
              stage32(c, w);
            } else if (c == 32) {
              release();
            }
          }
          if (mine) send(&tmap_d, col_w, row_w, 0);
        } else {
          if (has_res) fetch_res();
          ok = wait_full();
          if (!ok) break;
          if (has_res) {
            ok = wait_res();
            if (!ok) break;
          } else {
            tile_free();
          }
          const float scale = g16_scale(args, tl.group);
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            if (mine) {
              uint4 res[4], low[4];
              g16_load_res<32>(args, args.res_lo, tl.group, row, col_w + c, args.n, valid, low);
              float v[32];
              acc32(c, v);
              if (c == 32) release();
              if (has_res) staged32(c, res);
              g16_epilogue<EPI, 32>(args, v, res, low, nullptr, tl.group, row, col_w + c, scale);
              if (args.sym && tl.mb != tl.nb)
                g16_store_mirror<32>(args, v, tl.group, row, col_w + c, args.n, valid);
              if (args.z != nullptr) {
                // the low half of D, through the staging tile before D itself: a store has
                // 64 bytes each of eight rows (16 of each of 32: 4 x 1536 x 1536 428 us, so 415)
                uint4 l[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  uint32_t u[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float a0 = v[8 * q + 2 * j], a1 = v[8 * q + 2 * j + 1];
                    const float2 r2 = unpack16(pack16(a0, a1, 1), 1);
                    u[j] = pack16(a0 - r2.x, a1 - r2.y, 1);
                  }
                  l[q] = make_uint4(u[0], u[1], u[2], u[3]);
                }
                stage32(c, l);
                __syncwarp();
                const int col = col_w + c + (lane & 3) * 8;
                uint16_t* to = static_cast<uint16_t*>(args.z) + tl.group * args.d_batch + col;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int rr = i * 8 + (lane >> 2);
                  if (row_w + rr < tl.rows_end && col < args.n) {
                    uint4 q;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                                 : "r"(stg + rr * 128 + (((c / 8 + (lane & 3)) ^ (rr & 7)) << 4))
                                 : "memory");
                    *reinterpret_cast<uint4*>(to + (row_w + rr) * args.d_ld) = q;
                  }
                }
                __syncwarp();
              }
              uint4 w[4];
              pack32(v, w);
              stage32(c, w);
            } else if (c == 32) {
              release();
            }
          }
          if (mine) send(&tmap_d, col_w, row_w, tl.group);
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();
  }

  // neither CTA may leave while its peer can still signal its barriers, read
  // its shared memory or write its TMEM; a CTA that gave up lingers first
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (threadIdx.x == 0 && *abort_flag) linger_after_abort();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ======================================================================= one-CTA split-K kernel

// Producer, MMA and the epilogue's warps: eight, so that a whole or half tile's
// columns are shared by two to a lane quarter (128x128x64 5.7 -> 4.6 us); four where a
// CTA finishes a quarter or less.
__host__ __device__ constexpr int s16_threads(int splits) { return splits <= 2 ? 320 : 192; }
constexpr int kS16T = 128;        // tile rows and columns
// (With three stages, and so 96 registers, the linear epilogue spills 8 bytes and the poly one
// 64, LONG ones 84 to 260; of the pair kernel poly spills 16, kEpiLong 270.)
constexpr int kS16K = 64;

// STAGES: 3 where two CTAs share an SM, 6 where a CTA has one to itself (the
// operands of as many K chunks in flight either way).
template <int STAGES>
struct S16Layout {
  static constexpr int STG_BYTES = 32 * 64;  // a staging tile of an epilogue warp: 32 rows of 32 columns
  static constexpr int OFF_STG = 65536;      // behind the partial sums
  static constexpr int OP_BYTES = 128 * 128;  // 16 KB
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + STAGES * OP_BYTES;
  static constexpr int OFF_BAR = OFF_B + STAGES * OP_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 3;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_TAB = (OFF_MISC + 16 + 15) / 16 * 16;
  static constexpr int OFF_BIAS = (OFF_TAB + (kMaxGroups / kTabStep + 1) * 4 + 15) / 16 * 16;
  static constexpr int BYTES = OFF_BIAS + 128 * 4;
  static constexpr int ALLOC = BYTES + 1024;
  // partial sums of the other CTAs (at most 7 slices of 16 columns x 128 rows,
  // or 1 of 64) take the operand ring's place once the MMAs are done
  static_assert(7 * 16 * 128 * 4 <= OFF_STG && OFF_STG + 8 * STG_BYTES <= OFF_BAR, "reduction buffer and staging tiles");
  static_assert((STAGES <= 3 ? 2 : 1) * ALLOC <= 232448, "shared memory budget");
};

// One CTA's part of a product: `cta` counts from the product's first CTA.  LONG: its
// sum goes through the accumulator in parts of kSumPart, which the epilogue's warps
// add up in TMEM columns behind it (64x2112x65536: 2 % of the time).
template <int EPI, int STAGES, bool LONG>
__device__ __forceinline__ void g16_small_cta(const CUtensorMap* tmap_a, const CUtensorMap* tmap_b, const G16Args& args,
                                              const int cta) {
  using L = S16Layout<STAGES>;
  constexpr int S = STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int splits = args.splits;
  const int tile = cta / splits;
  const int part = cta - tile * splits;  // also the rank in the cluster

  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile uint32_t* tmem_slot = misc + 0;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + L::OFF_TAB);
  float* bias = reinterpret_cast<float*>(smem + L::OFF_BIAS);
  auto full_bar = [&](int s) { return sbase + L::OFF_BAR + 8u * s; };
  auto empty_bar = [&](int s) { return sbase + L::OFF_BAR + 8u * (S + s); };
  const uint32_t acc_bar = sbase + L::OFF_BAR + 8u * (2 * S);
  const uint32_t added_bar = acc_bar + 8, drain_bar = acc_bar + 16;  // LONG
  constexpr int kTmem = LONG ? 2 * kS16T : kS16T;  // of two CTAs to an SM: no more than TMEM's 512, so neither waits
  constexpr int kPart = kSumPart / kS16K;  // chunks of an accumulator

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(acc_bar, 1);
    if constexpr (LONG) {
      mbar_init(added_bar, (s16_threads(splits) - 64) / 32);  // one lane of each epilogue warp
      mbar_init(drain_bar, 1);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(tmap_a);
    prefetch_tmap(tmap_b);
  }
  pdl_launch_dependents();
  pdl_wait_prior();

  int total;
  if (args.mode == kRaggedM) {
    const int bad = __syncthreads_or(g16_offsets_bad(args, args.m));
    if (bad && threadIdx.x == 0 && cta == 0) report(args.status, 0x1);
    if (warp == 0) g16_prefix<kS16T>(args, tab, bad, &misc[2]);
    __syncthreads();
    total = static_cast<int>(misc[2]);
  } else {
    total = args.groups * g16_tiles_per_entry(args);
  }
  if (tile >= total) return;  // the whole cluster has this tile (the grid covers the most tiles there can be)

  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const G16Tile tl = g16_decode<kS16T>(args, tab, tile);
  const int chunks = (args.k + kS16K - 1) / kS16K;
  const int c_begin = static_cast<int>(static_cast<int64_t>(chunks) * part / splits);
  const int c_end = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / splits);

  if (warp == 0) {
    if (elect_one()) {
      // ===== TMA producer.  A K-major A comes in boxes of 32 rows, and only
      // those with rows of the tile; the other rows of the tile are whatever the
      // shared memory holds and feed accumulator rows that are never stored.
      const int left = tl.rows_end - tl.row0;
      const int a_boxes = args.a_mn ? 2 : ((left < kS16T ? left : kS16T) + 31) / 32;
      const int a_z = args.mode == kBatched ? tl.group : 0;
      const int b_z = args.b_per_group ? tl.group : 0;
      const int col0 = tl.nb * kS16T;
      const uint32_t bytes = (args.a_mn ? L::OP_BYTES : a_boxes * 4096) + L::OP_BYTES;
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int c = c_begin; c < c_end; ++c) {
        if (!wait16<false>(empty_bar(s), phase ^ 1u, abort_flag, args.wait_ns)) { ok = false; break; }
        mbar_arrive_expect_tx(full_bar(s), bytes);
        const uint32_t sa = sbase + L::OFF_A + s * L::OP_BYTES;
        const uint32_t sb = sbase + L::OFF_B + s * L::OP_BYTES;
        const int kk = c * kS16K;
        if (!args.b_mn) {
          tma_load_3d(sb, tmap_b, full_bar(s), kk, col0, b_z);
        } else if (args.b_wide) {
          tma_load_4d(sb, tmap_b, full_bar(s), 0, kk, col0 / 64, b_z);
        } else {
          tma_load_3d(sb, tmap_b, full_bar(s), col0, kk, b_z);
          tma_load_3d(sb + 8192, tmap_b, full_bar(s), col0 + 64, kk, b_z);
        }
        if (!args.a_mn) {
          for (int b = 0; b < a_boxes; ++b) tma_load_3d(sa + b * 4096, tmap_a, full_bar(s), kk, tl.row0 + b * 32, a_z);
        } else if (args.a_wide) {
          tma_load_4d(sa, tmap_a, full_bar(s), 0, kk, tl.row0 / 64, a_z);
        } else {
          tma_load_3d(sa, tmap_a, full_bar(s), tl.row0, kk, a_z);
          tma_load_3d(sa + 8192, tmap_a, full_bar(s), tl.row0 + 64, kk, a_z);
        }
        if (++s == S) { s = 0; phase ^= 1u; }
      }
      if (!ok) {
        report(args.status, 0x4);
        *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_f16(kS16T, kS16T, args.op_fp16, args.a_mn, args.b_mn);
      const uint64_t da0 = args.a_mn ? desc_mnmajor_sw128(sbase + L::OFF_A, 8192) : desc_kmajor_sw128(sbase + L::OFF_A);
      const uint64_t db0 = args.b_mn ? desc_mnmajor_sw128(sbase + L::OFF_B, 8192) : desc_kmajor_sw128(sbase + L::OFF_B);
      const uint64_t da_step = args.a_mn ? 128 : 2, db_step = args.b_mn ? 128 : 2;  // 16 of K, in 16-byte units
      int s = 0;
      uint32_t phase = 0, added = 0;
      bool ok = true;
      for (int c = c_begin; c < c_end; ++c) {
        const int i = LONG ? (c - c_begin) % kPart : c - c_begin;
        if constexpr (LONG) {
          if (i == 0 && c != c_begin) {  // the accumulator starts anew
            tc_commit(acc_bar);
            if (!wait16<false>(added_bar, added, abort_flag, args.wait_ns)) { ok = false; break; }
            added ^= 1u;
            tc_fence_after();
          }
        }
        if (!wait16<false>(full_bar(s), phase, abort_flag, args.wait_ns)) { ok = false; break; }
        const uint64_t da = da0 + static_cast<uint64_t>(s * (L::OP_BYTES >> 4));
        const uint64_t db = db0 + static_cast<uint64_t>(s * (L::OP_BYTES >> 4));
        const int left = args.k - c * kS16K;
        const int steps = left >= kS16K ? 4 : (left + 15) >> 4;  // zeros behind K's end are left out
        if (steps == 4) {
          tc_mma_f16(tmem_base, da, db, idesc, i != 0 ? 1u : 0u);
          tc_mma_f16(tmem_base, da + da_step, db + db_step, idesc, 1);
          tc_mma_f16(tmem_base, da + 2 * da_step, db + 2 * db_step, idesc, 1);
          tc_mma_f16(tmem_base, da + 3 * da_step, db + 3 * db_step, idesc, 1);
        } else {
          for (int q = 0; q < steps; ++q) tc_mma_f16(tmem_base, da + q * da_step, db + q * db_step, idesc, (i | q) != 0 ? 1u : 0u);
        }
        tc_commit(empty_bar(s));
        if (++s == S) { s = 0; phase ^= 1u; }
      }
      if (!ok) {
        report(args.status, 0x4);
        *abort_flag = 1;
      }
      tc_commit(acc_bar);
      // on every path, so that nothing is in flight when TMEM is freed
      if constexpr (LONG) tc_commit(drain_bar);
      wait16<false>(LONG ? drain_bar : acc_bar, 0, nullptr, 100000000ull);
    }
    __syncwarp();
  }
  if (warp < 2) {
    if (splits > 1) {  // the epilogue warps' exchange of partial sums
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ===== epilogue: a warp has the rows of a TMEM lane quarter and some of the columns
    const int ew = warp - 2, grp = ew >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const int row_w = tl.row0 + quarter * 32;  // the warp's first row
    const int row = row_w + lane;
    const bool valid = row < tl.rows_end;
    const int width = kS16T / splits;          // columns of the tile this CTA finishes
    const int grps = splits <= 2 ? 2 : 1;      // warps of a quarter
    const int wcols = width / grps;            // columns of this warp
    const int wc = grp * wcols;
    const int col_w = tl.nb * kS16T + part * width + wc;
    const int col_end = col_w + wcols < args.n ? col_w + wcols : args.n;
    // what the epilogue reads comes while the operands do: C and the residual into
    // registers, the bias as FP32 into shared memory
    uint4 res[2][4];
    if constexpr (EPI == kEpiLinear) {
      const int j = threadIdx.x - 64, col = tl.nb * kS16T + part * width + j;
      if (args.bias != nullptr && j < width && col < args.n)
        bias[j] = unpack16(__ldg(static_cast<const uint16_t*>(args.bias) + col), args.op_fp16).x;
      named_barrier_sync(1, s16_threads(splits) - 64);
    }
    if constexpr (EPI != kEpiPlain) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        g16_load_res<32>(args, args.res, tl.group, row, col_w + c * 32, col_end, valid, res[c]);
    }
    const float scale = EPI == kEpiPoly ? g16_scale(args, tl.group) : 1.0f;
    // 32 columns of this thread's row of the sum (16 where a CTA has no more)
    const uint32_t t_sum = LONG ? t_row + kS16T : t_row;
    const int unit = width < 32 ? 16 : 32;
    auto columns = [&](int col_t, bool whole, uint32_t (&raw)[32]) {
      __syncwarp();  // TMEM loads are the whole warp's
      if (whole) {
        tc_ld_32x32b_x32(t_sum + col_t, raw);
      } else {
        uint32_t r16[16];
        tc_ld_32x32b_x16(t_sum + col_t, r16);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          raw[j] = r16[j];
          raw[16 + j] = 0;
        }
      }
      tc_wait_ld();
    };
    // 32 columns of the warp's rows to global memory through a
    // tile in shared memory, so that a store has 64 bytes each of eight rows (16 of
    // each of 32 took 1 us of a tile's 5.7)
    const uint32_t stg = sbase + L::OFF_STG + ew * L::STG_BYTES;
    auto store = [&](void* out, const float (&v)[32], int col0) {
      const int h = args.out_type == 1;
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* f = v + q * 8;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)),
                     "r"(pack16(f[0], f[1], h)), "r"(pack16(f[2], f[3], h)), "r"(pack16(f[4], f[5], h)),
                     "r"(pack16(f[6], f[7], h))
                     : "memory");
      }
      __syncwarp();
      const int q = lane & 3, col = col0 + q * 8;
      uint16_t* to = static_cast<uint16_t*>(out) + tl.group * args.d_batch + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = i * 8 + (lane >> 2);
        if (row_w + rr < tl.rows_end && col < col_end) {
          uint4 w;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                       : "r"(stg + rr * 64 + ((q ^ ((rr >> 1) & 3)) << 4))
                       : "memory");
          *reinterpret_cast<uint4*>(to + (row_w + rr) * args.d_ld) = w;
        }
      }
    };
    const int parts = LONG ? (c_end - c_begin + kPart - 1) / kPart : 1;
    bool got = true;
    for (int p = 0; p < parts && got; ++p) {
      got = wait16<false, LONG ? 2 : 32>(acc_bar, p & 1, abort_flag, args.wait_ns);
      got = __all_sync(0xFFFFFFFFu, got);
      if (!got && lane == 0) {
        report(args.status, 0x4);
        *abort_flag = 1;
      }
      tc_fence_after();
      if constexpr (LONG) {
        const int span = kS16T / grps;  // columns that this warp adds
        for (int c = grp * span; c < (grp + 1) * span && got; c += 32) {
          uint32_t acc[32], sum[32];
          __syncwarp();
          tc_ld_32x32b_x32(t_row + c, acc);
          if (p != 0) {
            tc_ld_32x32b_x32(t_sum + c, sum);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[j] = __float_as_uint(__uint_as_float(acc[j]) + __uint_as_float(sum[j]));
          }
          tc_wait_ld();
          tc_st_32x32b_x32(t_sum + c, acc);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (got && lane == 0 && p + 1 < parts) mbar_arrive(added_bar);
      }
    }
    if constexpr (LONG) {  // a row's warps read what the others have added
      named_barrier_sync(1, s16_threads(splits) - 64);
      tc_fence_after();
    }
    const bool rows_here = got && row_w < tl.rows_end;
    if (splits > 1) {
      // every CTA's MMAs have read their operands: the rings can take partial sums
      cluster_sync();
      if (rows_here) {
        const int per = width / unit;  // units of an owner's columns, shared by the warps of a quarter
#pragma unroll 1
        for (int u = grp; u < (splits - 1) * per; u += grps) {
          const int o = 1 + u / per, c = (u % per) * unit;
          const int owner = (part + o) % splits;
          const int slot = part < owner ? part : part - 1;
          // [slot][quad of columns][row] of float4: a warp's 32 rows are 512 bytes
          const uint32_t dst = map_to_rank(sbase, owner) + static_cast<uint32_t>(((slot * width + c) / 4 * kS16T + r) * 16);
          uint32_t raw[32];
          columns(owner * width + c, unit == 32, raw);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j * 4 < unit)
              st_cluster_v4(dst + j * kS16T * 16, raw[4 * j], raw[4 * j + 1], raw[4 * j + 2], raw[4 * j + 3]);
        }
      }
      cluster_sync();
    }
#pragma unroll 1
    for (int ci = 0; ci < 2 && rows_here; ++ci) {
      const int c = wc + ci * 32;  // of the CTA's columns
      const int col0 = col_w + ci * 32;
      if (col0 >= col_end) break;
      uint4 low[4];
      if constexpr (EPI == kEpiPoly) g16_load_res<32>(args, args.res_lo, tl.group, row, col0, col_end, valid, low);
      uint32_t raw[32];
      columns(part * width + c, wcols >= 32, raw);
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
#pragma unroll 1
      for (int slot = 0; slot < splits - 1; ++slot) {
        const float4* src = reinterpret_cast<const float4*>(smem) + (slot * width + c) / 4 * kS16T + r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j * 4 < wcols) {
            const float4 f = src[j * kS16T];
            v[4 * j] += f.x;
            v[4 * j + 1] += f.y;
            v[4 * j + 2] += f.z;
            v[4 * j + 3] += f.w;
          }
        }
      }
      g16_epilogue<EPI, 32>(args, v, res[0], low, bias + c, tl.group, row, col0, scale);
      if constexpr (EPI == kEpiLinear) {
        if (args.z != nullptr) store(args.z, v, col0);
        g16_activate<32>(args, v, res[0]);
      }
      if constexpr (EPI == kEpiPoly) {
        if (args.sym && tl.mb != tl.nb) g16_store_mirror<32>(args, v, tl.group, row, col0, col_end, valid);
      }
      store(args.d, v, col0);
      if constexpr (EPI == kEpiPoly) {
        if (args.z != nullptr) {
          g16_remainder<32>(args, v);
          store(args.z, v, col0);
        }
      }
      if constexpr (EPI != kEpiPlain) {
#pragma unroll
        for (int q = 0; q < 4; ++q) res[0][q] = res[1][q];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) linger_after_abort();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmem);
  }
}

template <int EPI, int STAGES, bool LONG>
__global__ void __launch_bounds__(s16_threads(1), STAGES <= 3 ? 2 : 1)
    g16_small_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ G16Args args) {
  g16_small_cta<EPI, STAGES, LONG>(&tmap_a, &tmap_b, args, static_cast<int>(blockIdx.x));
}

// Two independent products of plain epilogue in one launch, the first's CTAs
// before the second's, K split alike (a layer's two gradients: neither fills the
// GPU, and the second's launch costs as much as its work).
struct G16Two {
  G16Args first, second;
  int first_ctas;
};

template <int STAGES>
__global__ void __launch_bounds__(s16_threads(1), STAGES <= 3 ? 2 : 1)
    g16_two_kernel(const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap b1,
                   const __grid_constant__ CUtensorMap a2, const __grid_constant__ CUtensorMap b2,
                   const __grid_constant__ G16Two two) {
  const int cta = static_cast<int>(blockIdx.x);
  const bool second = cta >= two.first_ctas;
  g16_small_cta<kEpiPlain, STAGES, false>(second ? &a2 : &a1, second ? &b2 : &b1, second ? two.second : two.first,
                                   second ? cta - two.first_ctas : cta);
}

// ======================================================================= host

// 16-bit operand [depth, rows, cols] (cols contiguous, rows `ld` elements
// apart) read in boxes of box_rows x 64 elements, 128-byte swizzle.
static bool make_tmap16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t depth, int64_t ld,
                        int64_t batch, int box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(depth)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(batch * 2)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MN-major operand whose rows are whole groups of 64 elements, viewed as
// [depth, cols / 64, rows, 64]: one box of two groups brings 128 of MN by 64 of
// K, the groups 8 KB apart as the MMA's descriptor wants them.  (With a part
// group at the end it would read behind the tensor's last row: two plain boxes then.)
static bool make_tmap16_wide(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t depth, int64_t ld,
                             int64_t batch) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64),
                              static_cast<cuuint64_t>(depth)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld * 2), 128, static_cast<cuuint64_t>(batch * 2)};
  const cuuint32_t box[4] = {64, 64, 2, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One operand's map: K-major [rows, k] in boxes of box_rows, or MN-major [k, mn].
static bool make_operand16(CUtensorMap* m, const void* base, int mn_major, int wide, int64_t mn, int64_t k, int64_t depth,
                           int64_t ld, int64_t batch, int box_rows) {
  if (!mn_major) return make_tmap16(m, base, k, mn, depth, ld, batch, box_rows);
  return wide ? make_tmap16_wide(m, base, mn, k, depth, ld, batch) : make_tmap16(m, base, mn, k, depth, ld, batch, 64);
}

// D (or z): boxes of 32 rows x 128 bytes, 128-byte swizzle (the epilogue's staging tiles).
static bool make_tmap_out16(CUtensorMap* m, void* base, int64_t cols, int64_t rows, int64_t depth, int64_t ld,
                            int64_t batch, bool fp32) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const int size = fp32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(depth)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * size), static_cast<cuuint64_t>(batch * size)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, base, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The shared-memory attribute belongs to a kernel on a device: set once for each.
constexpr int kMaxDevices = 64;
template <typename K>
static cudaError_t allow_smem(K kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

static cudaLaunchConfig_t g16_config(int64_t ctas, int threads, int smem, int cluster, cudaStream_t stream,
                                     cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int EPI>
static cudaError_t launch_pair16(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td,
                                 const CUtensorMap& tz, const CUtensorMap& tr, const G16Args& a, int64_t tiles,
                                 int num_sms, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = allow_smem(g16_pair_kernel<EPI>, P16Layout<EPI>::ALLOC, done);
  if (e != cudaSuccess) return e;
  const int64_t most = num_sms / 2;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      g16_config(2 * (tiles < most ? tiles : most), p16_threads(EPI), P16Layout<EPI>::ALLOC, 2, stream, attr);
  return cudaLaunchKernelEx(&cfg, g16_pair_kernel<EPI>, ta, tb, td, tz, tr, a);
}

// Clusters of `splits` CTAs that the GPU holds at once with one CTA to an SM
// (a cluster stays inside a GPC, so fewer than SMs / splits).
static int64_t lone_clusters(int splits, int num_sms) {
  static std::atomic<int> known[kMaxDevices][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return 0;
  int v = known[dev][splits].load(std::memory_order_relaxed);
  if (v == 0) {
    static std::atomic<bool> done[kMaxDevices];
    if (allow_smem(g16_small_kernel<kEpiPlain, 6, false>, S16Layout<6>::ALLOC, done) != cudaSuccess) return 0;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = g16_config(splits, s16_threads(splits), S16Layout<6>::ALLOC, splits, nullptr, attr);
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&v, g16_small_kernel<kEpiPlain, 6, false>, &cfg) != cudaSuccess || v <= 0) {
      cudaGetLastError();
      v = num_sms / splits / 2;
    }
    known[dev][splits].store(v, std::memory_order_relaxed);
  }
  return v;
}

template <int EPI, int STAGES, bool LONG>
static cudaError_t launch_small16s(const CUtensorMap& ta, const CUtensorMap& tb, const G16Args& a, int64_t tiles,
                                   cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = allow_smem(g16_small_kernel<EPI, STAGES, LONG>, S16Layout<STAGES>::ALLOC, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      g16_config(tiles * a.splits, s16_threads(a.splits), S16Layout<STAGES>::ALLOC, a.splits, stream, attr);
  return cudaLaunchKernelEx(&cfg, g16_small_kernel<EPI, STAGES, LONG>, ta, tb, a);
}

// Is a CTA's share of the sum too long for one accumulator?
static bool small_long(int64_t k, int splits) {
  const int64_t chunks = (k + kS16K - 1) / kS16K;
  return (chunks + splits - 1) / splits > kSumWhole / kS16K;
}

template <int EPI>
static cudaError_t launch_small16(const CUtensorMap& ta, const CUtensorMap& tb, const G16Args& a, int64_t tiles,
                                  int num_sms, cudaStream_t stream) {
  const bool lone = tiles <= lone_clusters(a.splits, num_sms);
  if (small_long(a.k, a.splits))
    return lone ? launch_small16s<EPI, 6, true>(ta, tb, a, tiles, stream) : launch_small16s<EPI, 3, true>(ta, tb, a, tiles, stream);
  return lone ? launch_small16s<EPI, 6, false>(ta, tb, a, tiles, stream) : launch_small16s<EPI, 3, false>(ta, tb, a, tiles, stream);
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which kernel, and how many CTAs share a tile's K: the one whose estimated time
// (in us, fitted to measured launches) is less.
//   pair kernel: 7 us for launch, first operands and last epilogue, and 0.31 us per
//     K chunk of 64 for each round of tiles (1024x1024x1024 12 us estimated, 11.4
//     measured; 1037x7168x2048 26.8, 28.1; 64x2112x7168 41.7, 38.5).
//   small kernel: 3.6 us with a plain epilogue, the exchange of partial sums, and per
//     K chunk of a CTA 0.27 us where all clusters have SMs to themselves (six stages);
//     else 2.6 us more, 0.3 us a chunk, or 0.4 us where there are more CTAs than SMs, and
//     2.5 us for every further round (256x256x256 whole: 4.7 estimated, 4.8 measured;
//     64x2112x7168 by 4: 13.2, 12.6; by 2: 20.4, 18.7; 128x4224x4096 by 4, 33 clusters
//     that fit: 9.9, 11.1; 128x4352x4096, 34 that do not: 13.0, 12.9; 1037x7168x2048
//     whole: 34.3, 34.2).
struct G16Tiles {
  double pair, small;  // 256 x 256 and 128 x 128 tiles to do
  int64_t chunks;      // of 64 of K
};

static G16Tiles count_tiles(const Gemm16& p) {
  const double np = static_cast<double>(ceil_div(p.n, kP16TN)), ns = static_cast<double>(ceil_div(p.n, kS16T));
  G16Tiles c;
  c.chunks = ceil_div(p.k, kS16K);
  if (p.mode == kRaggedM) {
    // the groups' sizes are on the device: the mean size, with half a tile more for each group's end
    const double groups = static_cast<double>(p.m < p.groups ? p.m : p.groups), rows = static_cast<double>(p.m) / groups;
    c.pair = groups * std::fmax(1.0, rows / kP16TM + 0.5) * np;
    c.small = groups * std::fmax(1.0, rows / kS16T + 0.5) * ns;
  } else {
    const double entries = static_cast<double>(p.groups);
    const double mp = static_cast<double>(ceil_div(p.m, kP16TM)), ms = static_cast<double>(ceil_div(p.m, kS16T));
    c.pair = entries * (p.sym ? mp * (mp + 1) / 2 : mp * np);
    c.small = entries * (p.sym ? ms * (ms + 1) / 2 : ms * ns);
  }
  return c;
}

// What an epilogue adds to the last tile, in us.
static double epilogue_cost(const Gemm16& p) {
  if (p.epi == kEpiPoly) return 3.5;
  return p.epi == kEpiLinear ? (p.act != 0 ? 1.8 : 0.8) : 0.0;
}

static double pair_cost(const G16Tiles& c, double epilogue, int num_sms) {
  return 7.0 + epilogue + 0.31 * std::ceil(c.pair / (num_sms / 2)) * static_cast<double>(c.chunks);
}

// The small kernel's cost on `tiles` tiles, the longest of `chunks`, and the best
// split, at most one CTA per chunk of the product with the fewest.
static double small_cost(double tiles, int64_t chunks, int64_t fewest, double epilogue, int num_sms, int* splits) {
  double best = 1e30;
  *splits = 1;
  for (int s = 1; s <= 8; s *= 2) {
    if (s > fewest || (s > 1 && tiles * s > num_sms)) break;  // (128x5120x4096, 40 tiles: by 2 14.5, by 4 14.9, by 8 22.6)
    const double each = static_cast<double>(ceil_div(chunks, s));
    const double exchange = s == 1 ? 0.0 : s == 2 ? 1.65 : s == 4 ? 2.0 : 3.0;
    const double rounds = std::ceil(tiles * s / (2.0 * num_sms));
    double cost = 3.6 + exchange + (s == 1 ? epilogue : 0.5 * epilogue);  // a warp has 64 columns, else 32 or less
    if (tiles <= static_cast<double>(lone_clusters(s, num_sms)))
      cost += 0.27 * each;
    else
      cost += 2.6 + (tiles * s <= num_sms ? 0.3 * each : 0.4 * each * rounds) + 2.5 * (rounds - 1.0);
    if (cost < best) {
      best = cost;
      *splits = s;
    }
  }
  return best;
}

static bool small_can(const Gemm16& p) {
  return p.mode != kRaggedK && p.out_type != 2;  // it neither clears rows behind a group nor sums in parts
}

struct G16Choice {
  bool small;
  int splits;
};

// MX_GEMM16_CONFIG forces a kernel for tests and tuning: 0 the pair kernel, 1, 2, 4
// or 8 the small one with that many CTAs (at most one per K chunk) a tile.  -1: not set.
static int forced_config() {
  const char* v = std::getenv("MX_GEMM16_CONFIG");
  if (v == nullptr || v[0] == 0 || v[1] != 0) return -1;
  const int n = v[0] - '0';
  return n == 0 || n == 1 || n == 2 || n == 4 || n == 8 ? n : -1;
}

static G16Choice choose(const Gemm16& p, int num_sms) {
  G16Choice c = {false, 1};
  const int forced = forced_config();
  if (forced >= 0) {
    if (forced == 0 || !small_can(p)) return c;
    c.small = true;
    for (c.splits = forced; c.splits > ceil_div(p.k, kS16K); c.splits /= 2) {
    }
    return c;
  }
  if (!small_can(p)) return c;
  const G16Tiles tiles = count_tiles(p);
  c.small = small_cost(tiles.small, tiles.chunks, tiles.chunks, epilogue_cost(p), num_sms, &c.splits) < pair_cost(tiles, epilogue_cost(p), num_sms);
  return c;
}

// Arguments and operand maps of a product on the chosen kernel; *tiles is the most there can be.
static cudaError_t prepare16(const Gemm16& p, const G16Choice& c, G16Args* args, CUtensorMap* ta, CUtensorMap* tb,
                             int64_t* tiles) {
  const int tm = c.small ? kS16T : kP16TM, tn = c.small ? kS16T : kP16TN;
  G16Args& a = *args;
  a = {};
  a.bias = p.bias;
  a.res = p.res;
  a.res_lo = p.res_lo;
  a.d = p.d;
  a.z = p.z;
  a.group_offsets = p.group_offsets;
  a.scale = p.scale;
  a.status = p.status;
  a.wait_ns = wait_limit_ns();
  a.d_ld = p.d_ld;
  a.d_batch = p.mode == kRaggedM ? 0 : p.d_batch;  // ragged M: one D, its rows numbered through
  a.res_ld = p.res_ld;
  a.res_batch = p.res_batch;
  a.alpha = p.alpha;
  a.beta = p.beta;
  a.diag = p.diag;
  a.scale_pow = p.scale_pow;
  a.m = static_cast<int>(p.m);
  a.n = static_cast<int>(p.n);
  a.k = static_cast<int>(p.k);
  a.m_tiles = static_cast<int>(ceil_div(p.m, tm));
  a.n_tiles = static_cast<int>(ceil_div(p.n, tn));
  a.groups = static_cast<int>(p.groups);
  a.mode = p.mode;
  a.a_mn = p.a_mn;
  a.b_mn = p.b_mn;
  a.a_wide = p.a_mn && p.m % 64 == 0;
  a.b_wide = p.b_mn && p.n % 64 == 0;
  a.b_per_group = p.mode != kRaggedK;
  a.op_fp16 = p.op_fp16;
  a.out_type = p.out_type;
  a.epi = p.epi;
  a.act = p.act;
  a.sym = p.sym;
  a.splits = c.splits;

  // (ragged M: every group adds at most one part tile a column)
  *tiles = p.mode == kRaggedM ? (p.m / tm + p.groups) * a.n_tiles
                              : p.groups * (p.sym ? static_cast<int64_t>(a.m_tiles) * (a.m_tiles + 1) / 2
                                                  : static_cast<int64_t>(a.m_tiles) * a.n_tiles);
  if (*tiles * c.splits > 0x3FFFFFFFll) return cudaErrorInvalidValue;  // tile numbers are 32-bit
  const int64_t a_depth = p.mode == kBatched ? p.groups : 1;
  const int64_t b_depth = a.b_per_group ? p.groups : 1;
  if (!make_operand16(ta, p.a, p.a_mn, a.a_wide, p.m, p.k, a_depth, p.a_ld, p.a_batch, c.small ? 32 : 128) ||
      !make_operand16(tb, p.b, p.b_mn, a.b_wide, p.n, p.k, b_depth, p.b_ld, p.b_batch, 128))
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

cudaError_t launch_gemm16(const Gemm16& p, int num_sms, cudaStream_t stream) {
  const G16Choice c = choose(p, num_sms);
  G16Args a;
  CUtensorMap ta, tb, td = {}, tz = {}, tr = {};
  int64_t tiles = 0;
  const cudaError_t e = prepare16(p, c, &a, &ta, &tb, &tiles);
  if (e != cudaSuccess) return e;
  if (c.small) {
    if (p.epi == kEpiLinear) return launch_small16<kEpiLinear>(ta, tb, a, tiles, num_sms, stream);
    if (p.epi == kEpiPoly) return launch_small16<kEpiPoly>(ta, tb, a, tiles, num_sms, stream);
    return launch_small16<kEpiPlain>(ta, tb, a, tiles, num_sms, stream);
  }
  const int64_t d_depth = p.mode == kRaggedM ? 1 : p.groups;
  if (!make_tmap_out16(&td, p.d, p.n, p.m, d_depth, p.d_ld, p.d_batch, p.out_type == 2)) return cudaErrorInvalidValue;
  if (p.z && p.epi == kEpiLinear && !make_tmap_out16(&tz, p.z, p.n, p.m, d_depth, p.d_ld, p.d_batch, false))
    return cudaErrorInvalidValue;
  if (p.res && !make_tmap_out16(&tr, const_cast<void*>(p.res), p.n, p.m, p.groups, p.res_ld, p.res_batch, false))
    return cudaErrorInvalidValue;
  // (ragged K: one group may have all rows)
  if (p.out_type != 2 && p.k > kSumWhole) return launch_pair16<kEpiLong>(ta, tb, td, tz, tr, a, tiles, num_sms, stream);
  if (p.out_type == 2) return launch_pair16<kEpiSum>(ta, tb, td, tz, tr, a, tiles, num_sms, stream);
  if (p.epi == kEpiLinear) return launch_pair16<kEpiLinear>(ta, tb, td, tz, tr, a, tiles, num_sms, stream);
  if (p.epi == kEpiPoly) return launch_pair16<kEpiPoly>(ta, tb, td, tz, tr, a, tiles, num_sms, stream);
  return launch_pair16<kEpiPlain>(ta, tb, td, tz, tr, a, tiles, num_sms, stream);
}

// Two products of plain epilogue, neither of which the other reads: one launch
// where the small kernel does both sooner than two.
cudaError_t launch_gemm16_two(const Gemm16& p, const Gemm16& q, int num_sms, cudaStream_t stream) {
  const G16Tiles tp = count_tiles(p), tq = count_tiles(q);
  int sp = 1, sq = 1, s = 1;
  const double apart = std::fmin(small_cost(tp.small, tp.chunks, tp.chunks, epilogue_cost(p), num_sms, &sp), pair_cost(tp, epilogue_cost(p), num_sms)) +
                       std::fmin(small_cost(tq.small, tq.chunks, tq.chunks, epilogue_cost(q), num_sms, &sq), pair_cost(tq, epilogue_cost(q), num_sms));
  const int64_t longest = tp.chunks > tq.chunks ? tp.chunks : tq.chunks, fewest = tp.chunks < tq.chunks ? tp.chunks : tq.chunks;
  const bool together = p.mode == kBatched && q.mode == kBatched && p.epi == kEpiPlain && q.epi == kEpiPlain && small_can(p) &&
                        small_can(q) && forced_config() < 0 &&
                        small_cost(tp.small + tq.small, longest, fewest, epilogue_cost(p), num_sms, &s) < apart &&
                        !small_long(p.k, s) && !small_long(q.k, s);
  if (!together) {
    const cudaError_t e = launch_gemm16(p, num_sms, stream);
    return e != cudaSuccess ? e : launch_gemm16(q, num_sms, stream);
  }
  const G16Choice c = {true, s};
  G16Two two = {};
  CUtensorMap a1, b1, a2, b2;
  int64_t t1 = 0, t2 = 0;
  cudaError_t e = prepare16(p, c, &two.first, &a1, &b1, &t1);
  if (e == cudaSuccess) e = prepare16(q, c, &two.second, &a2, &b2, &t2);
  if (e != cudaSuccess) return e;
  two.first_ctas = static_cast<int>(t1 * s);
  const bool lone = t1 + t2 <= lone_clusters(s, num_sms);
  static std::atomic<bool> done3[kMaxDevices], done6[kMaxDevices];
  e = lone ? allow_smem(g16_two_kernel<6>, S16Layout<6>::ALLOC, done6) : allow_smem(g16_two_kernel<3>, S16Layout<3>::ALLOC, done3);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      g16_config((t1 + t2) * s, s16_threads(s), lone ? S16Layout<6>::ALLOC : S16Layout<3>::ALLOC, s, stream, attr);
  return lone ? cudaLaunchKernelEx(&cfg, g16_two_kernel<6>, a1, b1, a2, b2, two)
              : cudaLaunchKernelEx(&cfg, g16_two_kernel<3>, a1, b1, a2, b2, two);
}

}  // namespace mxk
