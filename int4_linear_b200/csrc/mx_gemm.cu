// Block-scaled product of microscaled 4-bit operands on the tensor cores
// (tcgen05.mma kind::mxf4 / kind::mxf4nvf4 .block_scale), and the linear layer.
//
//   y[m][n] = fp16(g_x g_w sum_b s_x[m][b] s_w[n][b] sum_{k in b} x[m][k] w[n][k])
//
// The weights are the row operand (tensor-memory lanes), the tokens the N
// operand (BN = 16..256 columns), so that few tokens still fill the lanes. One CTA per SM:
// warp 0 brings stages of 256 values along K (128 bytes per row: one swizzle
// row) and their scales, which lie in memory as the 512-byte tiles that
// tcgen05.cp spreads over tensor memory; a thread each of warps 2 and 3 issues these copies (6 or 12
// per stage at 256 tokens, each holding its thread for 45 cycles: in the MMA thread's way they cost a
// third of the rate, from one thread 13 % of NVFP4's), one of warp 1 the four MMAs of a stage; warps
// 4-7 drain finished tiles. Every stage has its own scale columns, so the stage's barriers guard both.
//
// More than 64 tokens run on CTA pairs (PAIR): 256 weight rows per tile, each CTA
// holding its 128 rows, half of the tokens' rows and the scales of all of them; the even CTA's
// thread issues for both. A stage's copies of both CTAs complete on the even CTA's barrier, and its
// commits reach both.
//
// Work: whole tiles dealt to the CTAs in turn, or, for up to 64 tokens where that leaves SMs idle for
// longer than a join takes, equal contiguous parts of the (tile, stage) sequence; the CTA that arrives
// last at a divided tile adds the float32 parts in the CTAs' order.
//
// Bounds (2 M N K operations at four times the bf16 rate, 6.6 PFLOP/s, or the weights' bytes at 6.55 TB/s), with the
// quantizer before it: 16 x 57344 x 8192 (M x N x K) 43.3 us, 6.1 TB/s; 2048 x 28672 x 4096 102 us in MXFP4, 110 us
// in NVFP4, 4.7 and 4.4 PFLOP/s: there the power limit holds the clock at 1.5-1.6 GHz, and the tensor pipe is active in
// 65 % of its cycles (what idles it in the others has not been found); a single token's 6144 x 4096
// takes 8.6 us, nearly all of it launch, first loads, and the way out.
#include <cuda_fp16.h>

#include <algorithm>

#include "fq_device.cuh"
#include "fq_host.h"
#include "mx.cuh"

namespace fq {

size_t sync_block_bytes();

namespace {

constexpr int kStageK = 256;                    // values along K per stage
constexpr int kRowB = kStageK / 2;              // 128 bytes per row
constexpr int kTileN = 128;                     // weight rows per tile
constexpr int kMxGemmThreads = 256;
constexpr int kStoreRows = 16;                  // tokens per output block
constexpr int kJoinParts = 4;                   // parts of a divided tile read at once
constexpr int kStoreBytes = kStoreRows * 32 * 2;  // one warp's 16 x 32 outputs

struct MxGemmParams {
  const float *gx, *gw;
  int M, N, K;
  int mt, tiles, ks;       // token tiles, tiles, stages per tile
  int full;                // tiles taken whole; each one after these as two halves of its tokens (256 on pairs only)
  int split;               // 1: equal parts of the (tile, stage) sequence
  float* part;             // [2 * CTAs][BN][128]
  unsigned* count;
  unsigned* err;
};

template <int FMT, int BN, bool PAIR>
struct MxCfg {
  static constexpr int SB = FMT == FQ_NVFP4 ? 4 : 2;      // scale tiles along K per stage
  static constexpr int NBT = (BN + 127) / 128;            // scale tiles along the tokens
  static constexpr int BROWS = PAIR ? BN / 2 : BN;        // tokens' rows in this CTA
  static constexpr int A_BYTES = kTileN * kRowB, B_BYTES = BROWS * kRowB;
  static constexpr int SA_BYTES = SB * kMxTileBytes, SX_BYTES = SB * NBT * kMxTileBytes;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SX_BYTES;
  static constexpr int AB = BN <= 128 ? 2 : 1;            // accumulators
  static constexpr int ACC = BN < 32 ? 32 : BN;           // columns of one
  static constexpr int SF0 = AB * ACC;                    // first scale column
  static constexpr int SFA = SB * 4, SFX = SB * 4 * NBT;  // scale columns per stage
  static constexpr int OUT = 8 * kStoreBytes;             // two output blocks per epilogue warp
  static constexpr int BUDGET = 227 * 1024 - 1024 - OUT - 512;
  static constexpr int S0 = BUDGET / STAGE;
  static constexpr int S1 = (512 - SF0) / (SFA + SFX);
  static constexpr int S = S0 < S1 ? (S0 < 12 ? S0 : 12) : (S1 < 12 ? S1 : 12);
  // B's tile must start on a swizzle atom: A and B first, scales behind them
  static constexpr int OFF_SA = S * (A_BYTES + B_BYTES);
  static constexpr int OFF_OUT = OFF_SA + S * (SA_BYTES + SX_BYTES);
  static constexpr int OFF_BAR = OFF_OUT + OUT;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static_assert((A_BYTES + B_BYTES) % 1024 == 0 && A_BYTES % 1024 == 0 && SA_BYTES % 512 == 0, "operand layout");
  static_assert(SF0 + S * (SFA + SFX) <= 512, "tensor memory");
  static_assert(SMEM <= 227 * 1024 && (3 * S + 5) * 8 + 8 <= 512, "shared memory");
};

// 32 rows of 16 bytes (8-row groups 128 bytes apart, no swizzle) -> 4 columns of 32
// lanes, repeated in each quarter of the lanes; PAIR: in both CTAs.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(128u >> 4) << 32) | (uint64_t(1) << 46);
}
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of kind::mxf4 / mxf4nvf4: A = B = E2M1 K-major, M = m, N = n,
// scale type E8M0 or E4M3, scale byte (0 or 2) of both operands' 32-bit columns.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_mx(int m, int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | ((FMT == FQ_MXFP4 ? 1u : 0u) << 23) |
         (uint32_t(m >> 4) << 24) | (sf << 29);
}

template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
#define FQ_MX_MMA(GROUP, KIND)                                                                                   \
  asm volatile(                                                                                                  \
      "{\n\t.reg .pred p;\n\t"                                                                                  \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                                \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),          \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                              \
      : "memory")
  if (FMT == FQ_MXFP4) {
    if (PAIR)
      FQ_MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else
      FQ_MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
  } else {
    if (PAIR)
      FQ_MX_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else
      FQ_MX_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  }
#undef FQ_MX_MMA
}

// Tile load into this CTA's shared memory; PAIR: completing on the even CTA's barrier (`bar` is then a
// shared::cluster address).
template <bool PAIR>
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, uint64_t pol) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(pol)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, "
        "%4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(pol)
        : "memory");
}

__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// shared::cluster address of `p`'s counterpart in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// 16 lanes x 32 (x4) or 16 (x2) columns as 8-column blocks b: r[4 b + 2 h + e] is lane t / 4 + 8 h, column
// 8 b + 2 (t % 4) + e of thread t, the fragment that stmatrix stores.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Four 8 x 8 blocks of fp16 stored transposed; lane l gives the address of row l % 8 of block l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// Wait for a barrier's phase.  The thread sleeps in the instruction (up to the hint, 1 ms) instead of asking
// again and again: polling threads get in the way of the ones that issue copies and MMAs (64 quick
// tries per wait cost 20 % of the rate).  false after kWaitLimitNs.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
  constexpr uint32_t kHintNs = 1000000;
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    if (CLUSTER)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "r"(kHintNs)
          : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "r"(kHintNs)
          : "memory");
    if (ok) return true;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0)
      t0 = now;
    else if (now - t0 > kWaitLimitNs)
      return false;
  }
}

// wait_phase by a whole warp, which leaves it together.
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait_phase(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_phase<CLUSTER>(bar, parity));
}

// True on one lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A stage of the ring and its phase.
struct MxStage {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int S) {
    if (++s == S) {
      s = 0;
      phase ^= 1u;
    }
  }
};

// This CTA's segments: (tile, half of its tokens or -1, stages [k0, k1)), the same sequence for every role.
struct MxWalk {
  long long u, u1;
  int ks, step, split, full, mt, M;
  int tile, half, k0, k1;
  __device__ __forceinline__ MxWalk(const MxGemmParams& p, int cta, int ctas)
      : ks(p.ks), step(ctas), split(p.split), full(p.full), mt(p.mt), M(p.M), half(-1) {
    const long long total = static_cast<long long>(p.tiles) * p.ks;
    if (split) {
      u = total * cta / ctas;
      u1 = total * (cta + 1) / ctas;
    } else {
      u = cta;
      u1 = 2ll * p.tiles - full;
    }
  }
  __device__ __forceinline__ bool next() {
    while (u < u1) {
      if (split) {
        tile = int(u / ks);
        k0 = int(u % ks);
        k1 = int(min(static_cast<long long>(ks), k0 + (u1 - u)));
        u += k1 - k0;
        return true;
      }
      const long long rest = u - full;
      tile = int(rest < 0 ? u : full + (rest >> 1));
      half = rest < 0 ? -1 : int(rest & 1);
      k0 = 0;
      k1 = ks;
      u += step;
      if (half == 1 && tile % mt * 256 + 128 >= M) continue;  // no tokens there
      return true;
    }
    return false;
  }
};

template <int FMT, int BN, bool PAIR>
__global__ void __launch_bounds__(kMxGemmThreads, 1)
    mx_gemm_kernel(const MxGemmParams p, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSw,
                   const __grid_constant__ CUtensorMap tmSx, const __grid_constant__ CUtensorMap tmY) {
  using C = MxCfg<FMT, BN, PAIR>;
  constexpr int S = C::S;
  constexpr bool HALVES = PAIR && BN == 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + S;
  uint64_t* sf_full = empty + S;       // scales in tensor memory
  uint64_t* acc_full = sf_full + S;    // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2]
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  int* join = reinterpret_cast<int*>(done + 1) + 1;
  // The issuing warps run their loops as whole warps, one elected lane sending the instructions: addresses and
  // descriptors then stay in uniform registers, which the instructions take (from divergent code every operand
  // is moved there first).
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], PAIR ? 8 : 4);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_launch_dependents();
  if (warp != 0) pdl_wait();  // the producer prefetches first

  MxWalk walk(p, unit, units);
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    if (leader) {
      prefetch_tensormap(&tmW);
      prefetch_tensormap(&tmX);
      prefetch_tensormap(&tmSw);
      prefetch_tensormap(&tmSx);
    }
    const uint64_t pol_w = BN <= 64 ? policy_evict_first() : policy_evict_normal();  // few tokens: read once
    const uint64_t pol_x = policy_evict_last();  // the tokens are read by every CTA
    // The first stages' weights into L2 (where a running kernel's writes go as well) while the tokens are being
    // quantized: 42.5 -> 40.4 us for 16 x 57344 x 8192; two or four rings' worth made 777 x 5000 x 4224 slower.
    {
      MxWalk w = walk;
      int ahead = 0;
      while (ahead < S && w.next())
        for (int k = w.k0; k < w.k1 && ahead < S; ++k, ++ahead)
          if (leader) {
            const int nt = w.tile / p.mt * (PAIR ? 2 : 1) + int(rank);
            prefetch_tile(&tmW, k * kRowB, nt * kTileN);
            prefetch_tile(&tmSw, k * C::SB * 64, nt);
          }
    }
    pdl_wait();
    const uint32_t bar0 = PAIR ? cluster_addr(full, 0) : smem_u32(full);
    MxStage st;
    int sent = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const int nt = walk.tile / p.mt * (PAIR ? 2 : 1) + int(rank), mt = walk.tile % p.mt;  // 128 rows, BN tokens
      // of a half tile each CTA holds 64 rows (the box brings 64 more), and the half's scales come first
      const bool half = HALVES && walk.half >= 0;
      const int yw = nt * kTileN, yx = mt * BN + (half ? walk.half * 128 + int(rank) * 64 : int(rank) * C::BROWS);
      const int ysx = mt * BN / kMxTileRows + (half ? walk.half : 0);
      for (int k = walk.k0; k < walk.k1; ++k, st.next(S)) {
        if (!warp_wait_phase<false>(&empty[st.s], st.phase ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t bar = bar0 + 8u * st.s;
        uint8_t* ab = smem + st.s * (C::A_BYTES + C::B_BYTES);
        uint8_t* sf = smem + C::OFF_SA + st.s * (C::SA_BYTES + C::SX_BYTES);
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(&full[st.s], C::STAGE * (PAIR ? 2 : 1));
          load_tile<PAIR>(ab, &tmW, bar, k * kRowB, yw, pol_w);
          load_tile<PAIR>(ab + C::A_BYTES, &tmX, bar, k * kRowB, yx, pol_x);
          // scale tiles, 64 words of 8 bytes each; what lies past the last one reads as 0
          load_tile<PAIR>(sf, &tmSw, bar, k * C::SB * 64, nt, pol_w);
#pragma unroll
          for (int j = 0; j < C::NBT; ++j)
            load_tile<PAIR>(sf + C::SA_BYTES * (1 + j), &tmSx, bar, k * C::SB * 64, ysx + j, pol_x);
        }
        sent = min(sent + 1, S);
      }
    }
    // Before the CTA may leave, every copy has landed and the products' arrival for it, which a pair's even CTA
    // sends to both, has come: the last `sent` stages, oldest first.
    for (int i = 0; ok && i < sent; ++i) {
      const int back = sent - i, s = st.s - back < 0 ? st.s - back + S : st.s - back;
      ok = warp_wait_phase<false>(&empty[s], st.s - back < 0 ? st.phase ^ 1 : st.phase);
    }
    if (!ok && leader) record_error(p.err, kErrTimeoutProducer);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (rank == 0) {
      const bool leader = elect_one();
      auto commit = [&](uint64_t* bar) {
        if (PAIR)
          mma_commit_pair(bar, 3);
        else
          mma_commit(bar);
      };
      constexpr uint32_t kStep16 = (C::A_BYTES + C::B_BYTES) >> 4;  // a stage in the descriptors' 16-byte units
      const uint64_t a_desc = sdesc_k128_sw128(smem_u32(smem)), b_desc = sdesc_k128_sw128(smem_u32(smem) + C::A_BYTES);
      constexpr int kRows = PAIR ? 256 : 128, kHalf = HALVES ? 128 : BN;
      const bool tail = p.K % kStageK != 0;  // 128 values in the last stage
      MxStage st;
      int seg = 0;
      bool ok = true;
      while (ok && walk.next()) {
        const int buf = seg % C::AB;
        if (!warp_wait_phase<PAIR>(&acc_empty[buf], ((seg / C::AB) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(buf * C::ACC);
        const bool half_tile = HALVES && walk.half >= 0;
        const uint32_t i0 = half_tile ? idesc_mx<FMT>(kRows, kHalf, 0) : idesc_mx<FMT>(kRows, BN, 0);
        const uint32_t i2 = half_tile ? idesc_mx<FMT>(kRows, kHalf, 2) : idesc_mx<FMT>(kRows, BN, 2);
        for (int k = walk.k0; k < walk.k1; ++k, st.next(S)) {
          // the operands, then the scales, which came after them
          if (!warp_wait_phase<false>(&full[st.s], st.phase) || !warp_wait_phase<false>(&sf_full[st.s], st.phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a_desc + uint32_t(st.s) * kStep16, bd = b_desc + uint32_t(st.s) * kStep16;
          const uint32_t ta = tmem + uint32_t(C::SF0 + st.s * (C::SFA + C::SFX)), tx = ta + uint32_t(C::SFA);
          const bool half = tail && k + 1 == p.ks;
          if (leader) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (q >= 2 && half) break;
              const int b = FMT == FQ_NVFP4 ? q : q / 2;
              mma_mx<FMT, PAIR>(d, ad + 2 * q, bd + 2 * q, FMT == FQ_MXFP4 && (q & 1) ? i2 : i0, ta + 4 * b,
                                tx + 4 * b * C::NBT, q > 0 ? 1u : uint32_t(k > walk.k0));
            }
            commit(&empty[st.s]);
          }
        }
        if (leader) commit(&acc_full[buf]);
        ++seg;
      }
      // nothing issued may still run when tensor memory is freed
      if (leader) commit(done);
      ok = warp_wait_phase<false>(done, 0) && ok;
      if (!ok && leader) record_error(p.err, kErrTimeoutMma);
    } else if (!warp_wait_phase<false>(done, 0) && lane == 0) {
      // the odd CTA stays until the products, which read its shared and tensor memory, are done and their
      // last arrival has come here too
      record_error(p.err, kErrTimeoutMma);
    }
  } else if (warp == 2 || warp == 3) {
    // ------------------------------------------------------------ scales to tensor memory, every other tile each
    if (rank == 0) {
      const bool leader = elect_one();
      const uint64_t sf_desc = sdesc_scales(smem_u32(smem + C::OFF_SA));
      constexpr uint32_t kStep16 = (C::SA_BYTES + C::SX_BYTES) >> 4, kTile16 = kMxTileBytes >> 4;
      const bool tail = p.K % kStageK != 0;
      MxStage st;
      int sent = 0;
      bool ok = true;
      while (ok && walk.next()) {
        for (int k = walk.k0; k < walk.k1; ++k, st.next(S)) {
          if (!warp_wait_phase<false>(&full[st.s], st.phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t sd = sf_desc + uint32_t(st.s) * kStep16;
          const uint32_t ta = tmem + uint32_t(C::SF0 + st.s * (C::SFA + C::SFX)), tx = ta + uint32_t(C::SFA);
          const bool half = tail && k + 1 == p.ks;
          if (leader) {
#pragma unroll
            for (int b0 = 0; b0 < C::SB; b0 += 2) {
              if (b0 >= C::SB / 2 && half && C::SB > 2) break;
              if (half && C::SB == 2 && warp == 3) break;
              const int b = b0 + (warp & 1);
              copy_scales<PAIR>(ta + 4 * b, sd + b * kTile16);
#pragma unroll
              for (int j = 0; j < C::NBT; ++j)
                copy_scales<PAIR>(tx + 4 * (b * C::NBT + j), sd + (C::SB * (1 + j) + b) * kTile16);
            }
            if (PAIR)
              mma_commit_pair(&sf_full[st.s], 1);
            else
              mma_commit(&sf_full[st.s]);
          }
          sent = min(sent + 1, S);
        }
      }
      // every copy sent has been made before tensor memory is freed
      for (int i = 0; ok && i < sent; ++i) {
        const int back = sent - i, s = st.s - back < 0 ? st.s - back + S : st.s - back;
        ok = warp_wait_phase<false>(&sf_full[s], st.s - back < 0 ? st.phase ^ 1 : st.phase);
      }
      if (!ok && leader) record_error(p.err, kErrTimeoutUnpack);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ finished tiles
    const int w = warp & 3;  // lanes 32 w .. 32 w + 31: weight rows of the tile
    const uint32_t lanes = uint32_t(32 * w) << 16;
    uint8_t* out = smem + C::OFF_OUT + w * 2 * kStoreBytes;
    const float g = (p.gx ? *p.gx : 1.0f) * (p.gw ? *p.gw : 1.0f);
    int seg = 0, stored = 0;
    bool bad = false;
    // 16 tokens (columns col0..) of this warp's 32 rows: a block of 16 token rows of 64 bytes in shared
    // memory (64-byte swizzle, which keeps the 8 rows of a stored block in different banks), out by one
    // copy.  h[4 hf + 2 b + r]: rows 16 hf + 8 r + lane / 4, tokens 8 b + 2 (lane % 4), + 1
    const int mrow = lane & 7, mblk = lane >> 3;
    auto emit = [&](int nt, int mt, int col0, const uint32_t* h) {
      const int x = nt * kTileN + 32 * w, y = mt * BN + col0;
      if (x >= p.N || y >= p.M) return;
      const uint32_t blk = smem_u32(out) + (stored & 1) * kStoreBytes;
      if (lane == 0) bulk_wait_group_read<1>();
      __syncwarp();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int row = 8 * b + mrow;
        stmatrix_x4_trans(blk + row * 64 + ((mblk ^ ((row >> 1) & 3)) << 4), h[2 * b], h[2 * b + 1], h[4 + 2 * b],
                          h[4 + 2 * b + 1]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&tmY, out + (stored & 1) * kStoreBytes, x, y);
        bulk_commit_group();
      }
      ++stored;
    };
    auto pack = [&](uint32_t a, uint32_t b) {  // MXFP4 has no tensor scales
      const float2 v = make_float2(__uint_as_float(a), __uint_as_float(b));
      const float2 s = FMT == FQ_NVFP4 ? fmul2(v, make_float2(g, g)) : v;
      const __half2 r = __floats2half2_rn(s.x, s.y);
      return *reinterpret_cast<const uint32_t*>(&r);
    };
    // CH columns of this warp's lanes: v[16 hf + 4 b + ...] (CH = 32) or v[8 hf + 4 b + ...] (CH = 16)
    constexpr int CH = BN < 32 ? 16 : 32;  // columns per tensor-memory load
    constexpr int FR = CH / 2;             // fragment words per half of the lanes
    auto load_columns = [&](uint32_t addr, uint32_t* v) {
      if (CH == 32) {
        tmem_ld_16x256b_x4(addr, v);
        tmem_ld_16x256b_x4(addr + (16u << 16), v + FR);
      } else {
        tmem_ld_16x256b_x2(addr, v);
        tmem_ld_16x256b_x2(addr + (16u << 16), v + FR);
      }
    };
    while (walk.next()) {
      const int nt = walk.tile / p.mt * (PAIR ? 2 : 1) + int(rank), mt = walk.tile % p.mt;
      const int buf = seg % C::AB;
      const uint32_t d = tmem + uint32_t(buf * C::ACC) + lanes;
      auto release = [&]() {  // the accumulator goes back
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_cluster(&acc_empty[buf], 0);
          else
            mbar_arrive(&acc_empty[buf]);
        }
      };
      if (!bad && !__all_sync(0xffffffffu, lane != 0 || wait_phase<false>(&acc_full[buf], (seg / C::AB) & 1))) {
        if (lane == 0) record_error(p.err, kErrTimeoutEpilogue);
        bad = true;
      }
      tc_fence_after();
      ++seg;
      if (walk.k0 == 0 && walk.k1 == p.ks) {
        uint32_t h[BN / 2];  // 8 words per 16 tokens
        uint32_t v[2][2 * FR];
        load_columns(d, v[0]);
#pragma unroll
        for (int c = 0; c < BN; c += CH) {
          tmem_wait_ld();
          if (c + CH < BN) load_columns(d + c + CH, v[(c / CH + 1) & 1]);  // under way while this one is packed
          const uint32_t* f = v[(c / CH) & 1];
#pragma unroll
          for (int q = 0; q < CH / 16; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int at = FR * (j >> 2) + 8 * q + 4 * ((j >> 1) & 1) + 2 * (j & 1);
              h[c / 2 + 8 * q + j] = pack(f[at], f[at + 1]);
            }
        }
        release();  // before the outputs are on their way
        if (!bad) {
#pragma unroll
          for (int c = 0; c < BN; c += kStoreRows) {
            if (HALVES && c == 128 && walk.half >= 0) break;  // a half tile's columns end here
            emit(nt, mt, (HALVES && walk.half > 0 ? 128 : 0) + c, h + c / 2);
          }
        }
        continue;
      }
      // a part of a tile: float32 sums to this CTA's slot, as the lanes hold them: [warp][16 tokens][4][32 lanes][4]
      const long long total = static_cast<long long>(p.tiles) * p.ks, t0 = static_cast<long long>(walk.tile) * p.ks;
      const int G = units;
      const int c_first = int(((t0 + 1) * G - 1) / total);
      const int parts = int(((t0 + p.ks) * G - 1) / total) - c_first + 1;
      const size_t slot_floats = size_t(BN) * kTileN;
      const int cols = min(BN, p.M - mt * BN);
      const size_t mine = size_t(w) * BN * 32 + lane * 4;
      float* dst = p.part + (2 * size_t(blockIdx.x) + (walk.k0 == 0 ? 1 : 0)) * slot_floats + mine;
#pragma unroll
      for (int c = 0; c < BN; c += CH) {
        uint32_t v[2 * FR];
        load_columns(d + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < CH / 16; ++q)
          if (c + 16 * q < cols) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const uint32_t* f = v + FR * (j >> 3) + 8 * q + (j & 7);
              *reinterpret_cast<uint4*>(dst + (c + 16 * q + j) * 32) = make_uint4(f[0], f[1], f[2], f[3]);
            }
          }
      }
      release();
      __threadfence();
      named_barrier(1, 128);
      if (threadIdx.x == 128) *join = atomicInc(&p.count[c_first], unsigned(parts - 1)) == unsigned(parts - 1);
      named_barrier(1, 128);
      if (*join && !bad) {
        __threadfence();
        for (int c = 0; c < cols; c += kStoreRows) {
          float acc[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] = 0.f;
          for (int i = 0; i < parts; i += kJoinParts) {
            float4 v[kJoinParts][4];  // all under way at once: the join waits for memory
#pragma unroll
            for (int u = 0; u < kJoinParts; ++u)
              if (i + u < parts) {
                const float* src = p.part + (2 * size_t(c_first + i + u) + (i + u == 0)) * slot_floats + mine + c * 32;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[u][j] = __ldcg(reinterpret_cast<const float4*>(src + j * 128));
              }
#pragma unroll
            for (int u = 0; u < kJoinParts; ++u)
              if (i + u < parts) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  acc[4 * j] += v[u][j].x;
                  acc[4 * j + 1] += v[u][j].y;
                  acc[4 * j + 2] += v[u][j].z;
                  acc[4 * j + 3] += v[u][j].w;
                }
              }
          }
          uint32_t hh[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) hh[j] = pack(__float_as_uint(acc[2 * j]), __float_as_uint(acc[2 * j + 1]));
          emit(nt, mt, c, hh);
        }
      }
      named_barrier(1, 128);  // join is read before the next tile's flag
    }
    if (lane == 0) bulk_wait_group<0>();
  }
  __syncwarp();
  tc_fence_before();
  // a pair: neither CTA leaves while the other's threads may still signal it (what its tensor core sends and
  // reads has been waited for above)
  if (PAIR)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// Tokens per tile, tiles and whether K is divided, from the sizes alone.  Measured, quantizer included, us:
//  - pairs or single CTAs (tiles of 128 tokens): 128 x 8192 x 28672 (M x N x K) 38.1 / 39.2,
//    128 x 57344 x 8192 51.7 / 54.2, 256 x 4096 x 4096 10.5 / 20.2, 2048 x 28672 x 4096 102 / 137;
//    for 100 x 57344 x 2048 in NVFP4 17.7 / 17.0;
//  - tiles of 128 or 256 tokens on pairs: 256 x 4096 x 4096 10.5 / 12.4, 777 x 5000 x 4224 19.4 / 23.8,
//    1024 x 6144 x 4096 22.0 / 20.9, 2048 x 28672 x 4096 124 / 102: a tile of 256 takes 20 / 11 of one of 128;
//  - a last round of tiles of 256 that leaves at least half of the pairs idle, whole or as halves of 128 tokens:
//    1024 x 6144 x 4096 22.2 / 20.0, 4096 x 4096 x 4096 47.1 / 42, 2048 x 28672 x 4096 102 / 102 (bound by power);
//  - divided or not: a stage of a lone tile takes 0.28 us and the join of a tile what 12 + BN / 4 stages take (the
//    parts' way through memory, and their count on one CTA).  8 x 6144 x 4096 9.4 / 8.3, 8 x 28672 x 4096 14.4 / 13.9,
//    8 x 57344 x 8192 40.1 / 42.4, 8 x 4096 x 14336 11.9 / 19.1, 64 x 6144 x 4096 13.0 / 9.4, 64 x 8192 x 28672
//    27.1 / 37.8.
struct MxPlan {
  int bn, mt, tiles, full, ks, split, grid, sms;
  bool pair;
};

MxPlan mx_plan(int M, int N, int K) {
  MxPlan q;
  const int sms = q.sms = sm_count();
  q.ks = (K + kStageK - 1) / kStageK;
  q.pair = M > 64;
  const int workers = q.pair ? sms / 2 : sms;
  int rest = 0;
  const int nt = (N + (q.pair ? 255 : 127)) / (q.pair ? 256 : 128);
  if (!q.pair) {
    q.bn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  } else {
    const long long t128 = static_cast<long long>(nt) * ((M + 127) / 128), t256 = static_cast<long long>(nt) * ((M + 255) / 256);
    const long long w128 = (t128 + workers - 1) / workers, last = t256 % workers;
    const bool halves = last > 0 && 2 * last <= workers;
    const long long w256 = 20 * (t256 / workers) + (last == 0 ? 0 : halves ? 11 : 20);
    q.bn = w128 * 11 <= w256 ? 128 : 256;
    if (q.bn == 256 && halves) rest = int(last);
  }
  q.mt = (M + q.bn - 1) / q.bn;
  q.tiles = nt * q.mt;
  q.full = q.tiles - rest;
  const long long units = static_cast<long long>(q.tiles) * q.ks, waves = (q.tiles + workers - 1) / workers;
  q.split = !q.pair && waves * q.ks > (units + workers - 1) / workers + 12 + q.bn / 4;
  q.grid = int(std::min<long long>(workers, q.split ? units : q.tiles + rest)) * (q.pair ? 2 : 1);
  return q;
}

template <int FMT, int BN, bool PAIR>
fq_status launch_mx(const MxGemmParams& p, const CUtensorMap (&m)[5], int grid, cudaStream_t stream) {
  using C = MxCfg<FMT, BN, PAIR>;
  auto kern = mx_gemm_kernel<FMT, BN, PAIR>;
  static std::atomic<uint64_t> allowed{0};
  if (!allow_smem(kern, C::SMEM, allowed))
    return fail(FQ_ERR_CUDA, "cannot reserve %d bytes of shared memory", C::SMEM);
  if (PAIR)
    launch_pdl_cluster(kern, dim3(grid), dim3(kMxGemmThreads), C::SMEM, stream, 2, p, m[0], m[1], m[2], m[3], m[4]);
  else
    launch_pdl(kern, dim3(grid), dim3(kMxGemmThreads), C::SMEM, stream, p, m[0], m[1], m[2], m[3], m[4]);
  return check_launch("mx_gemm_kernel");
}

template <int FMT>
fq_status launch_mx_bn(const MxPlan& q, const MxGemmParams& p, const CUtensorMap (&m)[5], cudaStream_t stream) {
  if (q.pair)
    return q.bn == 128 ? launch_mx<FMT, 128, true>(p, m, q.grid, stream) : launch_mx<FMT, 256, true>(p, m, q.grid, stream);
  switch (q.bn) {
    case 16: return launch_mx<FMT, 16, false>(p, m, q.grid, stream);
    case 32: return launch_mx<FMT, 32, false>(p, m, q.grid, stream);
    default: return launch_mx<FMT, 64, false>(p, m, q.grid, stream);
  }
}

constexpr int kMaxRows = 1 << 30;

bool mx_sizes_ok(int M, int N, int K, fq_mx_format fmt) {
  return M >= 1 && M <= kMaxRows && N >= 8 && N <= kMaxRows && N % 8 == 0 && K >= kGroup && K <= kMaxK && K % kGroup == 0 &&
         (fmt == FQ_MXFP4 || fmt == FQ_NVFP4);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

size_t mx_gemm_workspace(const MxPlan& q) {
  if (q.pair) return 0;
  // whether or not K is divided, so that the caller need not know
  const long long ctas = std::min<long long>(q.sms, static_cast<long long>(q.tiles) * q.ks);
  return sync_block_bytes() + size_t(2) * ctas * q.bn * kTileN * sizeof(float);
}

// The linear layer's workspace: the product's part, the tokens' codes, their scales.
struct MxLinearLayout {
  size_t codes, scales, bytes;
  MxLinearLayout(const MxPlan& q, int M, int K, fq_mx_format fmt) {
    codes = up256(std::max(sync_block_bytes(), mx_gemm_workspace(q)));
    scales = codes + up256(size_t(M) * (K / 2));
    bytes = scales + fq_mx_scale_bytes(M, K, fmt);
  }
};

// The product by a plan of its sizes, all arguments but Xq's and Sx's checked.
fq_status mx_gemm(const MxPlan& q, const uint8_t* Xq, const uint8_t* Sx, const float* g_x, const uint8_t* Wq,
                  const uint8_t* Sw, const float* g_w, int M, int N, int K, fq_mx_format fmt, uint16_t* Y,
                  void* workspace, void* stream) {
  FQ_CHECK_ARG(static_cast<long long>((N + 127) / 128) * q.mt < (1ll << 31), "M = %d and N = %d: too many tiles", M, N);
  unsigned* err = device_error_word();
  if (!err) return fail(FQ_ERR_CUDA, "device error word unavailable");
  // weights, tokens, their scales (rows of 128-row tiles, 8-byte words), outputs
  CUtensorMap m[5];
  const int sb = fmt == FQ_NVFP4 ? 4 : 2;
  const uint64_t sw = uint64_t(K / mx_block(fmt) / kMxTileBlocks) * (kMxTileBytes / 8);
  fq_status st = make_tmap_2d(&m[0], Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, K / 2, N, K / 2, kRowB, kTileN,
                              CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == FQ_OK)
    st = make_tmap_2d(&m[1], Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, K / 2, M, K / 2, kRowB,
                      q.pair ? q.bn / 2 : q.bn, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == FQ_OK)
    st = make_tmap_2d(&m[2], Sw, CU_TENSOR_MAP_DATA_TYPE_INT64, sw, (N + 127) / 128, sw * 8, sb * 64, 1);
  if (st == FQ_OK)
    st = make_tmap_2d(&m[3], Sx, CU_TENSOR_MAP_DATA_TYPE_INT64, sw, (M + 127) / 128, sw * 8, sb * 64, 1);
  if (st == FQ_OK)
    st = make_tmap_2d(&m[4], Y, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, N, M, size_t(N) * 2, 32, kStoreRows,
                      CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != FQ_OK) return st;
  MxGemmParams p{};
  p.gx = g_x;
  p.gw = g_w;
  p.M = M;
  p.N = N;
  p.K = K;
  p.mt = q.mt;
  p.tiles = q.tiles;
  p.full = q.full;
  p.ks = q.ks;
  p.split = q.split;
  p.count = static_cast<unsigned*>(workspace) + kJoinCounters;
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sync_block_bytes());
  p.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fmt == FQ_MXFP4 ? launch_mx_bn<FQ_MXFP4>(q, p, m, s) : launch_mx_bn<FQ_NVFP4>(q, p, m, s);
}

}  // namespace
}  // namespace fq

extern "C" {

size_t fq_mx_gemm_workspace_size(int M, int N, int K, fq_mx_format fmt) {
  return fq::mx_sizes_ok(M, N, K, fmt) ? fq::mx_gemm_workspace(fq::mx_plan(M, N, K)) : 0;
}

size_t fq_mx_linear_workspace_size(int M, int N, int K, fq_mx_format fmt) {
  return fq::mx_sizes_ok(M, N, K, fmt) ? fq::MxLinearLayout(fq::mx_plan(M, N, K), M, K, fmt).bytes : 0;
}

fq_status fq_mx_gemm(const uint8_t* Xq, const uint8_t* Sx, const float* g_x, const uint8_t* Wq, const uint8_t* Sw,
                     const float* g_w, int M, int N, int K, fq_mx_format fmt, uint16_t* Y, void* workspace,
                     size_t ws_bytes, void* stream) {
  fq::clear_error();
  if (fmt != FQ_MXFP4 && fmt != FQ_NVFP4)
    return fq::fail(FQ_ERR_UNSUPPORTED, "format %d is not provided", int(fmt));
  FQ_CHECK_ARG(fq::mx_sizes_ok(M, N, K, fmt),
               "sizes M = %d, N = %d, K = %d: M and N in [1, 2^30], N a multiple of 8, K one of 128 in [128, %d]", M, N, K,
               fq::kMaxK);
  for (const void* q : {static_cast<const void*>(Xq), static_cast<const void*>(Sx), static_cast<const void*>(Wq),
                        static_cast<const void*>(Sw), static_cast<const void*>(Y)})
    FQ_CHECK_ARG(q && fq::aligned(q, 16), "Xq, Sx, Wq, Sw and Y must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(fq::aligned(g_x, 4) && fq::aligned(g_w, 4), "g_x and g_w must be 4-byte aligned");
  FQ_CHECK_ARG(fmt == FQ_NVFP4 || (!g_x && !g_w), "FQ_MXFP4 has no tensor scales: g_x and g_w must be NULL");
  const fq::MxPlan q = fq::mx_plan(M, N, K);
  const size_t need = fq::mx_gemm_workspace(q);
  if (need && (!workspace || ws_bytes < need || !fq::aligned(workspace, 256)))
    return fq::fail(FQ_ERR_INVALID, "workspace of %zu bytes (256-byte aligned) required, got %zu", need, ws_bytes);
  return fq::mx_gemm(q, Xq, Sx, g_x, Wq, Sw, g_w, M, N, K, fmt, Y, workspace, stream);
}

fq_status fq_mx_linear(const uint16_t* X, long long ldx, int M, int K, fq_mx_format fmt, const float* g_x,
                       const uint8_t* Wq, const uint8_t* Sw, const float* g_w, int N, uint16_t* Y, void* workspace,
                       size_t ws_bytes, void* stream) {
  fq::clear_error();
  if (fmt != FQ_MXFP4 && fmt != FQ_NVFP4)
    return fq::fail(FQ_ERR_UNSUPPORTED, "format %d is not provided", int(fmt));
  FQ_CHECK_ARG(fq::mx_sizes_ok(M, N, K, fmt),
               "sizes M = %d, N = %d, K = %d: M and N in [1, 2^30], N a multiple of 8, K one of 128 in [128, %d]", M, N, K,
               fq::kMaxK);
  // everything the second launch checks, before the first
  FQ_CHECK_ARG(Wq && Sw && Y && fq::aligned(Wq, 16) && fq::aligned(Sw, 16) && fq::aligned(Y, 16),
               "Wq, Sw and Y must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(fq::aligned(g_x, 4) && fq::aligned(g_w, 4), "g_x and g_w must be 4-byte aligned");
  FQ_CHECK_ARG(fmt == FQ_NVFP4 || (!g_x && !g_w), "FQ_MXFP4 has no tensor scales: g_x and g_w must be NULL");
  const fq::MxPlan q = fq::mx_plan(M, N, K);
  const fq::MxLinearLayout at(q, M, K, fmt);
  if (!workspace || ws_bytes < at.bytes || !fq::aligned(workspace, 256))
    return fq::fail(FQ_ERR_INVALID, "workspace of %zu bytes (256-byte aligned) required, got %zu", at.bytes, ws_bytes);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const fq_status st = fq_mx_quant(X, ldx, M, K, fmt, g_x, base + at.codes, base + at.scales, stream);
  if (st != FQ_OK) return st;
  return fq::mx_gemm(q, base + at.codes, base + at.scales, g_x, Wq, Sw, g_w, M, N, K, fmt, Y, base, stream);
}

}  // extern "C"
