// Gradient of the grouped expert MLP on Blackwell tensor cores (bf16
// operands, fp32 accumulation in tensor memory).
//
// MMOE: Modernizing Diffusion Transformers with Efficient Expert Design,
// "MoE++ expert layer": heavy experts are standard MLPs; "shared experts":
// one dense expert is always active. With U = X W1^T, H = act(U):
//   dH = dY W2, dU = dH act'(U), dX = dU W1, dW2 = dY^T H, dW1 = dU^T X.
//
// Five products of 2 rows d h FLOPs (10 and 5 with SwiGLU's 2h) in three
// launches, each a persistent stream of 256 x 256 tiles over CTA pairs
// (tcgen05.mma.cta_group::2, M = 256), bound by the tensor cores for large
// groups and by the weights' bytes for small ones:
//   act_grad   U and dH of a tile in one go. Both have K = d and the same
//              output tile, so the tile keeps two 256-column accumulators
//              (all 512 columns of tensor memory) and neither U nor act'(U)
//              is written to memory or rounded: while the dH product runs,
//              the epilogue turns U into H (stored) and act'(U), which it
//              holds in fp32 registers; when dH is done it stores the
//              product. The next tile's U overlaps that second half. (At
//              the 168 registers that ten warps can have it spills 120
//              bytes a thread, 180 for SwiGLU.)
//   dX         rows ragged, K = hidden width, two accumulators in turn.
//   dW         both weight gradients (K = the group's rows) in one launch;
//              small groups' dX and dW side by side in one.
// DiT-MoE-XL (8 experts that share 16384 rows, two shared experts of 8192
// each, 1152 x 4608, 1.74 TFLOP): 525-548 + 222-247 + 540-562 us launched
// apart (1270-1325, 1410-1565 and 1240-1290 TFLOP/s of a 1660 burst peak),
// 1.63-1.70 ms back to back under the power limit (1393 TFLOP/s sustained
// peak). 64 SwiGLU experts that share 256 rows, 2048 x 1024: 145-154 + 77-82 +
// 183-185 us for 805 MB read, 537 MB read and 805 MB written; a plain read of
// 805 MB takes 147 us, a plain fill 208.
//
// Operands are stored with K contiguous (x, dy, dU as rows of the output;
// W1 in U) or with the other dimension contiguous (W2 in dH, W1 in dX, and
// both sides of dW); the latter are MN-major tiles of tcgen05: a TMA box is
// 64 columns by 64 K rows, one 128-byte swizzled row per K.
//
// Ragged K: a group's last K block holds rows of the next group (or of
// nothing, with any bit pattern in it), which must count as zero on both
// sides, or a NaN there would spread. In the MN-major box a K row is one
// 128-byte row, so a warp of its own waits for that block's copies, clears
// the rows past the group's end up to the MMA's next 16, and only then hands
// the block over. It is the first block of a tile, so the wait overlaps the
// tile before. Only these blocks need a signal from the peer CTA (a release
// arrival on every block's barrier held both launches to half their rate: dX
// 587 us against 251, dW 1208 against 565 on DiT-MoE-XL's experts).
// Every wait is bounded: on expiry the kernel flags MOE_DEV_TIMEOUT, lets
// its copies and MMAs in flight finish, frees tensor memory and returns.
#include <string.h>

#include <type_traits>

#include "backward.h"
#include "chained.cuh"
#include "gemm_sched.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int BMP = 256;                       // rows of a pair's tile
constexpr int BN = 256;                        // columns of a tile
constexpr int kEpiWarps = 8;                   // two per TMEM lane quadrant
constexpr int kThreads = 64 + 32 * kEpiWarps;  // producer warp, MMA warp, epilogue warps
constexpr int kTailWarp = 2 + kEpiWarps;       // dW: clears the K blocks that end a group
constexpr int STAGES = 6;
constexpr uint32_t A_BYTES = BM * BK * 2;      // one CTA's half of A and of B
constexpr uint32_t B_BYTES = (BN / 2) * BK * 2;
constexpr uint32_t kStgBytes = 32 * 32 * 2;    // an epilogue warp's staging tile of 32 columns
constexpr size_t smem_bytes(uint32_t staging) {
  return 1024 + (size_t)STAGES * (A_BYTES + B_BYTES) + (size_t)kEpiWarps * staging;
}
constexpr uint32_t kBox = 64 * 64 * 2;         // an MN-major box: 64 columns by 64 K rows

// MN-major operand, 128-byte swizzle: 64-column blocks kBox apart (leading
// offset), 8-row K groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(kBox >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
constexpr uint64_t kStepK = 2;     // descriptor units of 16 K elements, K contiguous: 32 bytes
constexpr uint64_t kStepMn = 128;  // ... 16 K rows of 128 bytes
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;  // instruction descriptor: MN-major A, B

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// 32 fp32 columns of this lane's row, rounded, as row `lane` of the warp's
// 32 x 32 staging tile in the TMA 64-byte swizzle.
__device__ __forceinline__ void stage_row(const float (&v)[32], uint32_t stg, int lane) {
  const uint32_t row = stg + (uint32_t)lane * 64u, sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h2 = __floats2bfloat162_rn(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t *>(&h2);
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((uint32_t)q ^ sw) << 4)), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
}
// 64 columns, as row `lane` of a 32 x 64 tile in the TMA 128-byte swizzle.
__device__ __forceinline__ void stage_row(const float (&v)[2][32], uint32_t stg, int lane) {
  const uint32_t row = stg + (uint32_t)lane * 128u, sw = (uint32_t)(lane & 7);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h2 = __floats2bfloat162_rn(v[q >> 2][8 * (q & 3) + 2 * i], v[q >> 2][8 * (q & 3) + 2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t *>(&h2);
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((uint32_t)q ^ sw) << 4)), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
}
// The staging tile may be written: the warp's last store has read it.
__device__ __forceinline__ void stage_begin(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}
// 32 columns of one row, in units of 8, those below `n` (a multiple of 8).
__device__ __forceinline__ void store_row(__nv_bfloat16 *o, const float (&v)[32], int n) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (8 * q < n) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = v[8 * q + i];
      store8(o + 8 * q, f);
    }
}

// 64 consecutive fp32 columns of this thread's TMEM lane, both loads in flight.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[2][32]) {
  uint32_t r[2][32];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3]), "=r"(r[h][4]), "=r"(r[h][5]), "=r"(r[h][6]),
          "=r"(r[h][7]), "=r"(r[h][8]), "=r"(r[h][9]), "=r"(r[h][10]), "=r"(r[h][11]), "=r"(r[h][12]),
          "=r"(r[h][13]), "=r"(r[h][14]), "=r"(r[h][15]), "=r"(r[h][16]), "=r"(r[h][17]), "=r"(r[h][18]),
          "=r"(r[h][19]), "=r"(r[h][20]), "=r"(r[h][21]), "=r"(r[h][22]), "=r"(r[h][23]), "=r"(r[h][24]),
          "=r"(r[h][25]), "=r"(r[h][26]), "=r"(r[h][27]), "=r"(r[h][28]), "=r"(r[h][29]), "=r"(r[h][30]),
          "=r"(r[h][31])
        : "r"(taddr + 32 * h));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 32; ++i) v[h][i] = __uint_as_float(r[h][i]);
}

// H = GELU(u) and GELU'(u) of two values. With Q = 1 - Phi(|u|) =
// 0.5 P(t) exp(-u^2/2) (Abramowitz & Stegun 7.1.26, as in gelu_erf_x2; the
// error in Phi is below 1e-7) the exponential serves both:
//   H = max(u, 0) - |u| Q,  H' = Phi(u) + u exp(-u^2/2) / sqrt(2 pi)
__device__ __forceinline__ void gelu_and_grad_x2(float &v0, float &v1, float &g0, float &g1) {
  const uint64_t ax = f2_pack(fabsf(v0), fabsf(v1)), v = f2_pack(v0, v1);
  float d0, d1;
  f2_unpack(f2_fma(ax, f2_splat(0.23164189f), f2_splat(1.0f)), d0, d1);
  const uint64_t t = f2_pack(rcp_approx(d0), rcp_approx(d1));
  uint64_t q = f2_fma(f2_splat(0.5307027145f), t, f2_splat(-0.7265760135f));
  q = f2_fma(q, t, f2_splat(0.7107068705f));
  q = f2_fma(q, t, f2_splat(-0.142248368f));
  q = f2_fma(q, t, f2_splat(0.127414796f));
  float s0, s1;
  f2_unpack(f2_mul(f2_mul(v, v), f2_splat(-0.72134752044f)), s0, s1);
  const uint64_t e = f2_pack(ex2_approx(s0), ex2_approx(s1));
  q = f2_mul(f2_mul(q, t), e);  // 1 - Phi(|u|)
  float q0, q1;
  f2_unpack(q, q0, q1);
  const uint64_t phi = f2_pack(v0 < 0.f ? q0 : 1.0f - q0, v1 < 0.f ? q1 : 1.0f - q1);
  f2_unpack(f2_fma(f2_mul(v, f2_splat(0.3989422804f)), e, phi), g0, g1);
  const float m0 = fmaxf(v0, 0.f), m1 = fmaxf(v1, 0.f);
  f2_unpack(f2_fma(f2_mul(ax, f2_splat(-1.0f)), q, f2_pack(m0, m1)), v0, v1);
}

// ---------------------------------------------------------------- act_grad
struct ActGradProb {
  const int32_t *offsets;
  int n_groups, h, h1;  // h1: rows of W1 per group (2h when gated)
  int64_t rows;
  __nv_bfloat16 *H, *dU;
  int tma_out;
};
struct ActGradParams {
  int n_probs, d;
  ActGradProb pr[2];
  int32_t *status;
};
struct ActGradMaps {
  CUtensorMap x[2], dy[2], w1[2], w2[2], H[2], dU[2];
};

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
act_grad_kernel(const __grid_constant__ ActGradMaps tm, const __grid_constant__ ActGradParams p) {
  constexpr int HC = GATED ? BN / 2 : BN;            // hidden columns per tile
  constexpr uint32_t B2_BYTES = (HC / 2) * BK * 2;   // one CTA's half of W2's columns
  constexpr uint32_t IDESC_U = idesc_bf16_f32(BMP, BN), IDESC_D = idesc_bf16_f32(BMP, HC) | kMajorB;
  constexpr int NC = HC / 64;                        // 32-column chunks per epilogue warp

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * STAGES + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ Sched sched;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = (int)cluster_id_x(), npairs = (int)nclusters_x();
  chain_next();
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sA = smem_u32(base), sB = sA + STAGES * A_BYTES, sO = sB + STAGES * B_BYTES;
  const uint32_t full0 = smem_u32(&bars[0]), empty0 = smem_u32(&bars[STAGES]);
  const uint32_t tfull0 = smem_u32(&bars[2 * STAGES]), tempty0 = smem_u32(&bars[2 * STAGES + 2]);
  const uint32_t drain = smem_u32(&bars[2 * STAGES + 4]);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {  // accumulator 0: U, 1: dH
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 2) {
    int run = 0, ne = 0;
    for (int pi = 0; pi < p.n_probs; ++pi)
      sched_add(sched, pi, p.pr[pi].offsets, p.pr[pi].n_groups, p.pr[pi].rows, BMP, (p.pr[pi].h + HC - 1) / HC,
                p.status, run, ne);
    sched_close(sched, p.n_probs, run, ne);
  }
  chain_wait();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int nkb = (p.d + BK - 1) / BK;
  TileSeq seq;
  seq.init(sched, nkb, nkb, p.n_probs, pair, npairs);
  const uint32_t leader_full0 = mapa_shared(full0, 0), leader_tempty0 = mapa_shared(tempty0, 0);

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer (both CTAs): U's K blocks, then dH's
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    for (int t = seq.next(); ok && t >= 0; t = seq.next()) {
      const int e = find_entry(sched, t), pi = sched.prob[e], g = sched.group[e];
      const ActGradProb &pr = p.pr[pi];
      const int ntn = (pr.h + HC - 1) / HC, local = t - sched.tile_start[e];
      const int mt = local / ntn, n0 = (local - mt * ntn) * HC;
      const int a_row = sched.row0[e] + mt * BMP + (int)rank * BM;
      // Rank r's half of U's columns: 128 more hidden columns, or (gated) the up rows of the same ones.
      const int w1_row = g * pr.h1 + n0 + (int)rank * (GATED ? pr.h : BN / 2);
      const int w2_col = n0 + (int)rank * (HC / 2);
      for (int kb = 0; ok && kb < 2 * nkb; ++kb) {
        const bool second = kb >= nkb;
        const int k0 = (second ? kb - nkb : kb) * BK;
        if (!mbar_wait_cluster(empty0 + 8 * stage, phase ^ 1u, &abort_flag, p.status)) { ok = false; break; }
        if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * (A_BYTES + (second ? B2_BYTES : B_BYTES)));
        const uint32_t fb = leader_full0 + 8 * stage, dA = sA + stage * A_BYTES, dB = sB + stage * B_BYTES;
        if (!second) {
          tma_load_2d_pair(dA, &tm.x[pi], k0, a_row, fb);
          tma_load_2d_pair(dB, &tm.w1[pi], k0, w1_row, fb);
        } else {
          tma_load_2d_pair(dA, &tm.dy[pi], k0, a_row, fb);
#pragma unroll
          for (int b = 0; b < HC / 128; ++b)
            tma_load_3d_pair(dB + b * kBox, &tm.w2[pi], w2_col + 64 * b, k0, g, fb);
        }
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (leader)  // the leader's full barriers count both CTAs' copies
      for (int s = 0; s < STAGES; ++s)
        if (armed & (1u << s))
          mbar_wait_cluster(full0 + 8 * s, (armed_parity >> s) & 1u, &abort_flag, p.status, false);
  } else if (warp == 1 && lane == 0) {
    if (leader) {
      // ---------------- MMA issuer (leader only)
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = seq.next(); ok && t >= 0; t = seq.next()) {
        for (int a = 0; ok && a < 2; ++a) {
          if (!mbar_wait_cluster(tempty0 + 8 * a, acc_phase ^ 1u, &abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait_cluster(full0 + 8 * stage, phase, &abort_flag, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint64_t adesc = smem_desc_sw128(sA + stage * A_BYTES);
            if (a == 0) {
              const uint64_t bdesc = smem_desc_sw128(sB + stage * B_BYTES);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                tc_mma_pair(tmem_base, adesc + kStepK * kk, bdesc + kStepK * kk, IDESC_U, (kb | kk) != 0 ? 1u : 0u);
            } else {
              const uint64_t bdesc = smem_desc_mn(sB + stage * B_BYTES);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                tc_mma_pair(tmem_base + BN, adesc + kStepK * kk, bdesc + kStepMn * kk, IDESC_D,
                            (kb | kk) != 0 ? 1u : 0u);
            }
            tc_commit_pair(empty0 + 8 * stage, 0x3);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (ok) tc_commit_pair(tfull0 + 8 * a, 0x3);
        }
        acc_phase ^= 1u;
      }
      tc_commit_pair(drain, 0x3);
    }
    // Every MMA that reads this CTA's shared memory or writes its TMEM has
    // completed once the leader's last commit lands here.
    mbar_wait_cluster(drain, 0, &abort_flag, p.status, false);
  } else if (warp >= 2) {
    // ---------------- epilogue (both CTAs, own TMEM rows)
    const int quad = warp & 3, c_lo = ((warp - 2) / 4) * (HC / 2);
    const uint32_t stg = sO + (uint32_t)(warp - 2) * kStgBytes;
    uint32_t acc_phase = 0;
    for (int t = seq.next(); t >= 0; t = seq.next()) {
      const int e = find_entry(sched, t), pi = sched.prob[e];
      const ActGradProb &pr = p.pr[pi];
      const int ntn = (pr.h + HC - 1) / HC, local = t - sched.tile_start[e];
      const int mt = local / ntn, n0 = (local - mt * ntn) * HC;
      const int wrow0 = sched.row0[e] + mt * BMP + (int)rank * BM + quad * 32, row = wrow0 + lane;
      const bool valid = row < sched.row_end[e];
      const bool rows_tma = pr.tma_out && wrow0 + 32 <= sched.row_end[e];
      const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16);
      bool ready = mbar_wait_cluster(tfull0, acc_phase, &abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ready)) break;
      tc_fence_after();
      float g1[NC][32], g2[GATED ? NC : 1][32];  // act'(U) of this lane's row; gated: the factors of dg and du
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        const int c = c_lo + 32 * q, n = pr.h - (n0 + c);  // columns left of the hidden width
        float v[32];
        tmem_ld32(taddr + c, v);
        if (GATED) {
          float u[32];
          tmem_ld32(taddr + BN / 2 + c, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a = v[i], sg = rcp_approx(1.0f + ex2_approx(-1.4426950409f * a)), s = a * sg;
            g1[q][i] = u[i] * fmaf(sg, 1.0f - s, s);  // u silu'(a), silu' = sg + s (1 - sg) = sg (1 - s) + s
            g2[q][i] = s;
            v[i] = s * u[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 2) gelu_and_grad_x2(v[i], v[i + 1], g1[q][i], g1[q][i + 1]);
        }
        if (rows_tma && n >= 32) {
          stage_begin(lane);
          stage_row(v, stg, lane);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm.H[pi], n0 + c, wrow0, stg);
            bulk_commit();
          }
        } else if (valid) {
          store_row(pr.H + (size_t)row * pr.h + n0 + c, v, n);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty0);
      ready = mbar_wait_cluster(tfull0 + 8, acc_phase, &abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ready)) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        const int c = c_lo + 32 * q, n = pr.h - (n0 + c);
        float v[32];
        tmem_ld32(taddr + BN + c, v);
#pragma unroll
        for (int part = 0; part < (GATED ? 2 : 1); ++part) {
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = v[i] * (part ? g2[GATED ? q : 0][i] : g1[q][i]);
          const int oc = part * pr.h + n0 + c;
          if (rows_tma && n >= 32) {
            stage_begin(lane);
            stage_row(o, stg, lane);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tm.dU[pi], oc, wrow0, stg);
              bulk_commit();
            }
          } else if (valid) {
            store_row(pr.dU + (size_t)row * pr.h1 + oc, o, n);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8);
      acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_all();  // every tile store has landed before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
}

// ------------------------------------------------------------- dX and dW
// One product per problem, D = A . B with 256 x 256 tiles (the last columns
// of a problem as a 256 x 128 tile when 128 are enough):
//   RAGGED_K false (dX): D[rows, N] = A[rows, K] B_g[K, N], A K-major
//   RAGGED_K true  (dW): D_g[M, N] = sum over the group's rows A[r, M] B[r, N],
//                        A MN-major; an empty group's tiles are zero
// B is MN-major in both.
struct GemmProb {
  const int32_t *offsets;
  int n_groups;
  int64_t rows;
  int M, N, K;   // M: dW; K: dX
  __nv_bfloat16 *out;
  int tma_out;
  int tile_end;  // dW: tiles of the problems up to this one
};
constexpr int kMaxProbs = 4;
struct GemmParams {
  int n_probs;
  GemmProb pr[kMaxProbs];
  int32_t *status;
};
struct GemmMaps {
  CUtensorMap a[kMaxProbs], b[kMaxProbs], o[kMaxProbs];
};

// dX and dW side by side: the first x_pairs pairs run dX.
struct BothMaps {
  GemmMaps x, w;
};
struct BothParams {
  GemmParams x, w;
  int x_pairs;
};

struct Tile {
  int pi, g, m0, n0, nw;  // m0: dX's first row, dW's first output row; nw: columns of the MMA
  int lo, hi;             // the group's rows (dX: row_end in hi)
  int nkb;
};

// The order of a pair's tiles: dX from the table of row tiles, dW counted
// off problem by problem, group by group, columns fastest.
template <bool RAGGED_K> struct Tiles;
template <> struct Tiles<false> {
  TileSeq seq;
  const Sched *s;
  __device__ void init(const Sched *sched, const GemmParams &p, int id, int n) {
    s = sched;
    seq.init(*s, (p.pr[0].K + BK - 1) / BK, (p.pr[1].K + BK - 1) / BK, p.n_probs, id, n);
  }
  __device__ bool next(const GemmParams &p, Tile &o) {
    const int t = seq.next();
    if (t < 0) return false;
    const int e = find_entry(*s, t);
    o.pi = s->prob[e];
    o.g = s->group[e];
    const GemmProb &pr = p.pr[o.pi];
    const int ntn = (pr.N + BN - 1) / BN, local = t - s->tile_start[e], mt = local / ntn;
    o.m0 = s->row0[e] + mt * BMP;
    o.hi = s->row_end[e];
    o.n0 = (local - mt * ntn) * BN;
    o.nw = pr.N - o.n0 <= BN / 2 ? BN / 2 : BN;
    o.nkb = (pr.K + BK - 1) / BK;
    return true;
  }
};
template <> struct Tiles<true> {
  int t, step;
  const int *rows;  // the groups' row offsets in shared memory
  __device__ void init(const int *offsets, const GemmParams &, int id, int n) { t = id; step = n; rows = offsets; }
  __device__ bool next(const GemmParams &p, Tile &o) {
    int pi = 0, first = 0;
    while (pi < p.n_probs && t >= p.pr[pi].tile_end) first = p.pr[pi++].tile_end;
    if (pi == p.n_probs) return false;
    const GemmProb &pr = p.pr[pi];
    const int ntn = (pr.N + BN - 1) / BN, per = ntn * ((pr.M + BMP - 1) / BMP), local = t - first;
    o.pi = pi;
    o.g = local / per;
    const int r = local - o.g * per;
    o.m0 = (r / ntn) * BMP;
    o.n0 = (r % ntn) * BN;
    o.nw = pr.N - o.n0 <= BN / 2 ? BN / 2 : BN;
    o.lo = pr.offsets ? rows[o.g] : 0;
    o.hi = pr.offsets ? rows[o.g + 1] : (int)pr.rows;
    check_group_rows(o.lo, o.hi, pr.rows, p.status);
    o.nkb = (o.hi - o.lo + BK - 1) / BK;
    t += step;
    return true;
  }
};

// An epilogue warp's staging tile. dW's tiles of small groups are little
// more than their stores, which go out as whole 128-byte lines (64 columns);
// dX's tile table takes that space.
constexpr uint32_t staging_bytes(bool ragged_k) { return ragged_k ? 2 * kStgBytes : kStgBytes; }

// One CTA's part of pair `id` of `n`.
template <bool RAGGED_K>
__device__ __forceinline__ void pair_gemm(const GemmMaps &tm, const GemmParams &p, int id, int n) {
  constexpr uint32_t IDESC0 = kMajorB | (RAGGED_K ? kMajorA : 0u);
  constexpr uint32_t IDESC_W = idesc_bf16_f32(BMP, BN) | IDESC0, IDESC_N = idesc_bf16_f32(BMP, BN / 2) | IDESC0;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[4 * STAGES + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  // dX: the table of row tiles; dW: the routed groups' row offsets.
  // dX's table lies behind its staging tiles.
  struct Offsets { int at[kMaxLayerExperts + 1]; };
  __shared__ Offsets offsets;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sA = smem_u32(base), sB = sA + STAGES * A_BYTES, sO = sB + STAGES * B_BYTES;
  Sched &sched = *reinterpret_cast<Sched *>(base + STAGES * (A_BYTES + B_BYTES) + kEpiWarps * kStgBytes);
  const uint32_t full0 = smem_u32(&bars[0]), empty0 = smem_u32(&bars[STAGES]);
  const uint32_t tfull0 = smem_u32(&bars[2 * STAGES]), tempty0 = smem_u32(&bars[2 * STAGES + 2]);
  const uint32_t drain = smem_u32(&bars[2 * STAGES + 4]), tail0 = smem_u32(&bars[2 * STAGES + 5]);
  // The peer's word that its part of a stage's tail block is ready, one per
  // stage: the peer may be a ring ahead of the leader, never more.
  const uint32_t peer_tail0 = smem_u32(&bars[3 * STAGES + 5]), leader_peer_tail0 = mapa_shared(peer_tail0, 0);

  chain_next();
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(tail0 + 8 * s, 1);
      mbar_init(peer_tail0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 2) {
    if constexpr (RAGGED_K) {
      // Every problem with offsets has the routed experts' ones.
      for (int pi = 0; pi < p.n_probs; ++pi)
        if (p.pr[pi].offsets)
          for (int g = lane; g <= p.pr[pi].n_groups; g += 32) offsets.at[g] = p.pr[pi].offsets[g];
    } else {
      int run = 0, ne = 0;
      for (int pi = 0; pi < p.n_probs; ++pi)
        sched_add(sched, pi, p.pr[pi].offsets, p.pr[pi].n_groups, p.pr[pi].rows, BMP, (p.pr[pi].N + BN - 1) / BN,
                  p.status, run, ne);
      sched_close(sched, p.n_probs, run, ne);
    }
  }
  // H and dU are there; some of their rows were written by plain stores, and
  // the TMA reads them.
  chain_wait();
  asm volatile("fence.proxy.async;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  Tiles<RAGGED_K> tiles;  // the same in both CTAs of the pair
  if constexpr (RAGGED_K) tiles.init(offsets.at, p, id, n);
  else tiles.init(&sched, p, id, n);
  const uint32_t leader_full0 = mapa_shared(full0, 0), leader_tempty0 = mapa_shared(tempty0, 0);
  Tile t;

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer (both CTAs). A tail block goes to the
    // CTA's own barrier of its stage; the tail warp clears it and hands it over.
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0, tail_phase = 0, tail_armed = 0;
    bool ok = true;
    while (ok && tiles.next(p, t)) {
      const CUtensorMap *mA = &tm.a[t.pi], *mB = &tm.b[t.pi];
      const int bx = t.n0 + (int)rank * (t.nw / 2), nb = t.nw / 128;  // this CTA's columns of B, in boxes
      const int am = t.m0 + (int)rank * BM;
      const uint32_t mine = A_BYTES + (uint32_t)nb * kBox;
      for (int i = 0; i < t.nkb; ++i) {
        const int kb = RAGGED_K ? t.nkb - 1 - i : i;  // a tail block first
        if (!mbar_wait_cluster(empty0 + 8 * stage, phase ^ 1u, &abort_flag, p.status)) { ok = false; break; }
        const uint32_t dA = sA + stage * A_BYTES, dB = sB + stage * B_BYTES, fb = leader_full0 + 8 * stage;
        if (RAGGED_K && t.lo + kb * BK + BK > t.hi) {
          const int row = t.lo + kb * BK;
          const uint32_t tb = tail0 + 8 * stage;
          mbar_arrive_expect_tx(tb, mine);
          tma_load_2d(dA, mA, am, row, tb);
          tma_load_2d(dA + kBox, mA, am + 64, row, tb);
          for (int b = 0; b < nb; ++b) tma_load_2d(dB + b * kBox, mB, bx + 64 * b, row, tb);
          tail_armed |= 1u << stage;  // the parity of this use
          tail_phase ^= 1u << stage;
        } else {
          if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * mine);
          if (RAGGED_K) {
            const int row = t.lo + kb * BK;
            tma_load_2d_pair(dA, mA, am, row, fb);
            tma_load_2d_pair(dA + kBox, mA, am + 64, row, fb);
            for (int b = 0; b < nb; ++b) tma_load_2d_pair(dB + b * kBox, mB, bx + 64 * b, row, fb);
          } else {
            tma_load_2d_pair(dA, mA, kb * BK, am, fb);
            for (int b = 0; b < nb; ++b) tma_load_3d_pair(dB + b * kBox, mB, bx + 64 * b, kb * BK, t.g, fb);
          }
        }
        // The stage's last use, of either kind: its full barrier goes no further.
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    // Let every copy land before the CTA can exit: the leader's full barriers
    // count both CTAs' copies, a tail's barrier its own CTA's.
    for (int s = 0; s < STAGES; ++s) {
      if (leader && (armed & (1u << s)))
        mbar_wait_cluster(full0 + 8 * s, (armed_parity >> s) & 1u, &abort_flag, p.status, false);
      if (tail_armed & (1u << s)) mbar_wait(tail0 + 8 * s, ((tail_phase >> s) & 1u) ^ 1u, &abort_flag, p.status, false);
    }
  } else if (RAGGED_K && warp == kTailWarp) {
    // ---------------- tail warp (both CTAs): the ring stages of tail blocks, in order
    int stage = 0;
    uint32_t tail_phase = 0;  // a bit per stage
    bool ok = true;
    while (ok && tiles.next(p, t)) {
      const int rows = (t.hi - t.lo) % BK;
      if (rows) {
        ok = __all_sync(0xffffffffu, mbar_wait(tail0 + 8 * stage, (tail_phase >> stage) & 1u, &abort_flag, p.status));
        if (!ok) break;
        // The MMA takes the block's rows in steps of 16: clear up to the next one.
        const uint32_t lo = (uint32_t)rows * 128u, hi = (uint32_t)((rows + 15) & ~15) * 128u;
        for (int b = 0; b < 2 + t.nw / 128; ++b) {
          const uint32_t box = b < 2 ? sA + stage * A_BYTES + b * kBox : sB + stage * B_BYTES + (b - 2) * kBox;
          for (uint32_t o = lo + lane * 16u; o < hi; o += 512u)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(box + o), "r"(0) : "memory");
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (!leader) {
            mbar_arrive_cluster(leader_peer_tail0 + 8 * stage);
          } else {
            ok = mbar_wait_cluster(peer_tail0 + 8 * stage, (tail_phase >> stage) & 1u, &abort_flag, p.status);
            mbar_arrive_cluster(leader_full0 + 8 * stage);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        tail_phase ^= 1u << stage;
      }
      stage = (stage + t.nkb) % STAGES;
    }
  } else if (warp == 1 && lane == 0) {
    if (leader) {
      // ---------------- MMA issuer (leader only)
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok && tiles.next(p, t)) {
        if (t.nkb == 0) continue;  // an empty group: the epilogue stores zeros
        if (!mbar_wait_cluster(tempty0 + 8 * acc, acc_phase ^ 1u, &abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
        const uint32_t idesc = t.nw == BN ? IDESC_W : IDESC_N;
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!mbar_wait_cluster(full0 + 8 * stage, phase, &abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint64_t adesc = RAGGED_K ? smem_desc_mn(sA + stage * A_BYTES) : smem_desc_sw128(sA + stage * A_BYTES);
          const uint64_t bdesc = smem_desc_mn(sB + stage * B_BYTES);
          // A tail block (the tile's first) ends at the last 16 rows that hold any of the group's.
          const int tail_rows = RAGGED_K && kb == 0 ? (t.hi - t.lo) % BK : 0;
          const int steps = tail_rows ? (tail_rows + 15) / 16 : BK / 16;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            if (kk < steps)
              tc_mma_pair(d_tmem, adesc + (RAGGED_K ? kStepMn : kStepK) * kk, bdesc + kStepMn * kk, idesc,
                          (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair(empty0 + 8 * stage, 0x3);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(tfull0 + 8 * acc, 0x3);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      tc_commit_pair(drain, 0x3);
    }
    mbar_wait_cluster(drain, 0, &abort_flag, p.status, false);
  } else if (warp >= 2 && warp < kTailWarp) {
    // ---------------- epilogue (both CTAs, own TMEM rows)
    const int quad = warp & 3;
    const uint32_t stg = sO + (uint32_t)(warp - 2) * staging_bytes(RAGGED_K);
    int acc = 0;
    uint32_t acc_phase = 0;
    while (tiles.next(p, t)) {
      const GemmProb &pr = p.pr[t.pi];
      const int wrow0 = t.m0 + (int)rank * BM + quad * 32, row = wrow0 + lane;
      const int half = t.nw / 2, c_lo = ((warp - 2) / 4) * half;
      if (t.nkb > 0) {
        const bool ready = mbar_wait_cluster(tfull0 + 8 * acc, acc_phase, &abort_flag, p.status);
        if (!__all_sync(0xffffffffu, ready)) break;
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * BN);
      auto release = [&] {  // the accumulator may be overwritten
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8 * acc);
      };
      if (RAGGED_K) {
        // The accumulator goes into registers and is handed back before the
        // stores: small groups' tiles are little else, and MMA, epilogue and
        // the two signals between them would otherwise take turns. dW's rows
        // end with its tensor, where the TMA store clips them.
        float v[2][2][32];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (t.nkb > 0 && 64 * k < half) {
            tmem_ld64(taddr + c_lo + 64 * k, v[k]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[k][0][i] = v[k][1][i] = 0.f;
          }
        }
        if (t.nkb > 0) release();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = t.n0 + c_lo + 64 * k;
          if (64 * k < half && col < pr.N && wrow0 < pr.M) {
            stage_begin(lane);
            stage_row(v[k], stg, lane);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tm.o[t.pi], col, wrow0, t.g, stg);
              bulk_commit();
            }
          }
        }
      } else {
        // dX's groups end inside the tensor: a block of rows reaching past a
        // group's last one is stored lane by lane.
        const bool tma = pr.tma_out && wrow0 + 32 <= t.hi;
#pragma unroll 1
        for (int c = c_lo; c < c_lo + half; c += 32) {
          const int col = t.n0 + c;
          if (col >= pr.N) break;
          float v[32];
          tmem_ld32(taddr + c, v);
          if (tma) {
            stage_begin(lane);
            stage_row(v, stg, lane);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tm.o[t.pi], col, wrow0, stg);
              bulk_commit();
            }
          } else if (row < t.hi) {
            store_row(pr.out + (size_t)row * pr.N + col, v, pr.N - col);
          }
        }
      }
      if (t.nkb > 0) {
        if (!RAGGED_K) release();
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
    }
    if (lane == 0) bulk_wait_all();  // every tile store has landed before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
}

template <bool RAGGED_K>
__global__ void __launch_bounds__(kThreads + (RAGGED_K ? 32 : 0), 1)
mlp_bwd_pair_kernel(const __grid_constant__ GemmMaps tm, const __grid_constant__ GemmParams p) {
  pair_gemm<RAGGED_K>(tm, p, (int)cluster_id_x(), (int)nclusters_x());
}

__global__ void __launch_bounds__(kThreads + 32, 1)
mlp_bwd_both_kernel(const __grid_constant__ BothMaps tm, const __grid_constant__ BothParams p) {
  const int id = (int)cluster_id_x(), n = (int)nclusters_x();
  const int nx = p.x_pairs < n ? p.x_pairs : n - 1;  // a pair for dW at least
  if (id < nx) pair_gemm<false>(tm.x, p.x, id, nx);
  else pair_gemm<true>(tm.w, p.w, id - nx, n - nx);
}

// ------------------------------------------------------------ host side
typedef CUresult (*TensorMapEncoder)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                     const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                     CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                     CUtensorMapFloatOOBfill);
// The driver's tensor-map encoder, looked up once (a function-local static is
// initialised once, safely under concurrent first calls); null if the driver
// does not provide it.
TensorMapEncoder tensor_map_encoder() {
  static const TensorMapEncoder fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<TensorMapEncoder>(ptr);
    return static_cast<TensorMapEncoder>(nullptr);
  }();
  return fn;
}

// bf16 tensor [z, rows, cols] (z = 0: 2-D), box {bx, by}, swizzled by the
// box's row: 128 bytes (64 columns) or 64 (32 columns).
bool make_map(CUtensorMap *m, const void *ptr, int64_t cols, int64_t rows, int64_t z, int bx, int by, bool store) {
  const bool narrow = bx == 32;
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const int rank = z > 0 ? 3 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)(rows > 0 ? rows : 1), (cuuint64_t)z};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * 2 * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            store ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool operand_k(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols) {  // K contiguous, 128 rows a box
  return make_map(m, ptr, cols, rows, 0, BK, BM, false);
}
bool operand_mn(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t z) {
  return make_map(m, ptr, cols, rows, z, 64, 64, false);
}
bool stored(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols) {
  return make_map(m, ptr, cols, rows, 0, 32, 32, true);
}
bool stored_grouped(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t z) {
  return make_map(m, ptr, cols, rows, z, 64, 32, true);
}

// `chained`: whether an earlier launch of this call precedes it; true from then on.
template <auto kern, int threads, uint32_t staging, int min_clusters = 1, typename Maps, typename Params>
int launch_pairs(const Maps &maps, const Params &params, int64_t max_tiles, cudaStream_t stream, bool &chained) {
  if (max_tiles == 0) return MOE_OK;
  MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(staging)));
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem_bytes(staging);
  cfg.stream = stream;
  cfg.gridDim = dim3(2 * (unsigned)(num_sms() / 2));
  // Co-resident CTA pairs, asked once per kernel (a function-local static is
  // initialised once, safely under concurrent first calls).
  static const int max_clusters = [&] {
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
    return n;
  }();
  int clusters = max_clusters;
  if (clusters < min_clusters) return MOE_ERR_UNSUPPORTED;
  if (max_tiles < clusters) clusters = (int)max_tiles;
  cfg.gridDim = dim3(2 * (unsigned)clusters);
  if (chained) cfg.numAttrs = 2;
  chained = true;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, maps, params));
  return last_launch_status();
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Row tiles at most, whatever the groups' sizes, and as many as groups of
// about the same size have.
inline int64_t row_tiles(const MlpBwdProblem &q) { return div_up(q.rows, BMP) + (q.offsets ? q.n_groups : 0); }
inline int64_t likely_row_tiles(const MlpBwdProblem &q) {
  if (!q.offsets) return div_up(q.rows, BMP);
  const int64_t few = q.rows < q.n_groups ? q.rows : q.n_groups, many = div_up(q.rows, BMP) + q.n_groups / 2;
  return few > many ? few : many;
}
constexpr int64_t kMaxTiles = 0x7fffffff;

// dX and dW do not depend on each other. In turn, a dX of few tiles leaves
// pairs idle, a small group's dX only reads and its dW only writes, and there
// is a launch more. Side by side in one launch they fill each other's gaps,
// but the pairs are split once, so a few long tiles may fit worse. The rule
// predicts both sides' times in K blocks of a tile; a tile's stores take as
// long as about 6. With groups of up to 384 rows dW is all stores, in many
// small tiles: always side by side. Otherwise it has to gain a sixteenth.
// In turn -> side by side: 64 SwiGLU experts 2048 x 1024, 512 tokens 638 -> 606
// us, 32 tokens 468 -> 465; 32 of 2048 x 768, 1024 tokens 294 -> 273; 19
// experts 1152 x 3200, 64 tokens 190 -> 173; two experts 64 x 64 30 -> 21.
// Where it is refused: one expert 512 x 4096, 9000 tokens 208 -> 233. 117
// sizes, 96 of them random, take 0.87 of the time in the mean; the one worse
// by more than drift was 64 experts 256 x 8192, 116 tokens, 544 -> 568.
constexpr int64_t kStoreBlocks = 6;
struct SideCost {
  int64_t tiles = 0, blocks = 0;  // blocks: in K blocks of a tile
  void add(int64_t t, int64_t kb) { tiles += t; blocks += t * (kb < kStoreBlocks ? kStoreBlocks : kb); }
  int64_t span(int64_t pairs) const { return div_up(tiles, pairs) * blocks / tiles; }
};

// The pairs that run dX so that both sides end soonest; 0 for one after the other.
int split_pairs(const SideCost &x_most, const SideCost &x_likely, const SideCost &w) {
  int64_t n = num_sms() / 2;
  // One tile more than pairs is a second chain of loads: as many as there can
  // be if those fit, else as many as there likely are.
  const SideCost &x = x_most.tiles <= n ? x_most : x_likely;
  if (x.tiles == 0 || w.tiles == 0) return 0;
  if (n > x.tiles + w.tiles) n = x.tiles + w.tiles;
  int64_t best = INT64_MAX;
  int pairs = 0;
  for (int64_t k = 1; k < n && k <= x.tiles; ++k) {
    const int64_t a = x.span(k), b = w.span(n - k), both = a > b ? a : b;
    if (both < best) { best = both; pairs = (int)k; }
  }
  const bool stores = w.blocks == w.tiles * kStoreBlocks;
  return stores || best * 16 <= (x.span(n) + w.span(n)) * 15 ? pairs : 0;
}

// Problems i of `q` with rows, in one launch (all gated or none).
int run_act_grad(const MlpBwdProblem *q, int n, bool gated, int32_t *status, cudaStream_t stream, bool &chained) {
  ActGradMaps maps;
  ActGradParams pd;
  memset(&maps, 0, sizeof(maps));
  memset(&pd, 0, sizeof(pd));
  pd.status = status;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    const MlpBwdProblem &s = q[i];
    if (s.rows == 0 || (s.gated != 0) != gated) continue;
    const int k = pd.n_probs++, h1 = gated ? 2 * s.h : s.h;
    pd.d = s.d;
    ActGradProb &o = pd.pr[k];
    o.offsets = s.offsets; o.n_groups = s.n_groups; o.h = s.h; o.h1 = h1; o.rows = s.rows;
    o.H = static_cast<__nv_bfloat16 *>(s.H); o.dU = static_cast<__nv_bfloat16 *>(s.dU);
    if (!operand_k(&maps.x[k], s.x, s.rows, s.d) || !operand_k(&maps.dy[k], s.dy, s.rows, s.d) ||
        !operand_k(&maps.w1[k], s.W1, (int64_t)s.n_groups * h1, s.d) ||
        !operand_mn(&maps.w2[k], s.W2, s.d, s.h, s.n_groups))
      return MOE_ERR_CUDA;
    o.tma_out = stored(&maps.H[k], s.H, s.rows, s.h) && stored(&maps.dU[k], s.dU, s.rows, h1);
    tiles += row_tiles(s) * div_up(s.h, gated ? BN / 2 : BN);
  }
  if (tiles > kMaxTiles) return MOE_ERR_UNSUPPORTED;
  return gated ? launch_pairs<act_grad_kernel<true>, kThreads, kStgBytes>(maps, pd, tiles, stream, chained)
               : launch_pairs<act_grad_kernel<false>, kThreads, kStgBytes>(maps, pd, tiles, stream, chained);
}

}  // namespace

int launch_mlp_bwd_bf16(const MlpBwdProblem *q, int n, int32_t *status, cudaStream_t stream) {
  bool chained = false;
  int st = run_act_grad(q, n, false, status, stream, chained);
  if (st == MOE_OK) st = run_act_grad(q, n, true, status, stream, chained);
  if (st != MOE_OK) return st;
  BothMaps maps;
  BothParams pd;
  memset(&maps, 0, sizeof(maps));
  memset(&pd, 0, sizeof(pd));
  pd.x.status = pd.w.status = status;
  int64_t x_tiles = 0, w_tiles = 0;
  SideCost x_most, x_likely, w_side;
  for (int i = 0; i < n; ++i) {  // dX = dU W1
    const MlpBwdProblem &s = q[i];
    if (!s.dx || s.rows == 0) continue;
    const int k = pd.x.n_probs++, h1 = s.gated ? 2 * s.h : s.h;
    GemmProb &o = pd.x.pr[k];
    o.offsets = s.offsets; o.n_groups = s.n_groups; o.rows = s.rows; o.N = s.d; o.K = h1;
    o.out = static_cast<__nv_bfloat16 *>(s.dx);
    if (!operand_k(&maps.x.a[k], s.dU, s.rows, h1) || !operand_mn(&maps.x.b[k], s.W1, h1, s.d, s.n_groups))
      return MOE_ERR_CUDA;
    o.tma_out = stored(&maps.x.o[k], s.dx, s.rows, s.d);
    x_tiles += row_tiles(s) * div_up(s.d, BN);
    x_most.add(row_tiles(s) * div_up(s.d, BN), div_up(h1, BK));
    x_likely.add(likely_row_tiles(s) * div_up(s.d, BN), div_up(h1, BK));
  }
  if (x_tiles > kMaxTiles) return MOE_ERR_UNSUPPORTED;
  for (int i = n - 1; i >= 0; --i)   // the shared expert's long K first
    for (int which = 0; which < 2; ++which) {
      const MlpBwdProblem &s = q[i];
      void *out = which ? s.dW1 : s.dW2;
      if (!out) continue;
      const int k = pd.w.n_probs++, h1 = s.gated ? 2 * s.h : s.h;
      GemmProb &o = pd.w.pr[k];
      o.offsets = s.offsets; o.n_groups = s.n_groups; o.rows = s.rows;
      o.M = which ? h1 : s.d;  // dW1 = dU^T X, dW2 = dY^T H
      o.N = which ? s.d : s.h;
      o.out = static_cast<__nv_bfloat16 *>(out);
      const void *A = which ? s.dU : s.dy, *B = which ? s.x : s.H;
      if (s.rows > 0 && (!operand_mn(&maps.w.a[k], A, s.rows, o.M, 0) || !operand_mn(&maps.w.b[k], B, s.rows, o.N, 0)))
        return MOE_ERR_CUDA;
      if (!stored_grouped(&maps.w.o[k], out, o.M, o.N, s.n_groups)) return MOE_ERR_CUDA;
      const int64_t tiles = s.n_groups * div_up(o.M, BMP) * div_up(o.N, BN), kb = div_up(s.rows, (int64_t)s.n_groups * BK);
      w_tiles += tiles;
      w_side.add(tiles, kb);
      if (w_tiles > kMaxTiles) return MOE_ERR_UNSUPPORTED;
      o.tile_end = (int)w_tiles;
    }
  pd.x_pairs = split_pairs(x_most, x_likely, w_side);
  if (pd.x_pairs > 0)
    return launch_pairs<mlp_bwd_both_kernel, kThreads + 32, staging_bytes(true), 2>(maps, pd, x_tiles + w_tiles, stream,
                                                                                  chained);
  if ((st = launch_pairs<mlp_bwd_pair_kernel<false>, kThreads, staging_bytes(true)>(maps.x, pd.x, x_tiles, stream,
                                                                                      chained)) != MOE_OK)
    return st;
  return launch_pairs<mlp_bwd_pair_kernel<true>, kThreads + 32, staging_bytes(true)>(maps.w, pd.w, w_tiles, stream,
                                                                                     chained);
}

}  // namespace moe
