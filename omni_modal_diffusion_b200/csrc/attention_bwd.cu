// Backward pass of the non-causal attention of the packed sequence on tcgen05
// tensor cores.  With S = Q K^T, c = 1 / sqrt(128), P = exp(c S - lse) row by
// row (lse: the forward call's log-sum-exp) and delta = rowsum(dO (.) O):
//   dV = P^T dO,  dP = dO V^T,  dS = P (.) (dP - delta),
//   dQ = c dS K,  dK = c dS^T Q.
// The probabilities are recomputed, never stored.
//
// Two passes instead of one: a CTA owns a query tile and walks the keys (dQ), or
// a key tile and walks the queries (dK, dV).  S and dP are taken twice, but each
// result then lives in one CTA's TMEM: no fp32 dQ in memory, no atomics (the
// same call gives the same bits), and P and dS go from the registers that
// computed them to TMEM as the next product's A operand.
//
// delta cannot be had from O alone: O is bf16, and a row whose delta is off by e
// has e P_ij in every dS_ij, so e times the mean key in dQ, where dS K itself
// lets everything that the keys share drop out.  (Unit-variance keys and values
// with an offset of the same size in each channel: dQ off by 3.5e-2 of its
// 2-norm at 1,024 tokens, 8e-2 at 4,096; offsets of 4: 0.76.)  The rows of dS
// sum to 0 with the delta of P and dP themselves, so the query tiles start from
// delta(O), take rho = rowsum(dS) in fp32 and, beside dS K, P K, and end with
//   dQ = c (dS K - rho P K),  delta = delta(O) + rho,
// the second for the key tiles, which come after.  rho is some 2^-8 of dS's
// terms, so the rounding of P in P K does not matter.  That makes eight tile
// products of the five that the formulas have, and two launches that follow one
// another.
//
// Measured: 56 heads of 7,904 tokens 5.5 ms, 4 heads of 32,160 tokens 6.2 ms:
// 814 and 855 TFLOP/s counting five products, 1,300 and 1,370 of the eight done,
// at the power limit.  (With delta from O alone, seven products in one launch:
// 4.9 and 5.4 ms; 64 tokens, 4 heads: 14 us, so 22.)
//
// P and dS are rounded to bf16 for their products (half a step, relative 2^-8 at
// most, each, as the forward pass rounds P); sums, exponentials and the
// subtraction are fp32.
//
// Valid rows end inside a tile: the tensor maps stop at token L, TMA reads
// zeros past it (whatever the padding rows hold), and masked queries have
// lse = +inf (P = 0).  Masked keys are set to P = 0 in the last key tile that a
// query tile walks; in a key tile they are rows of their own, zeroed as they are
// stored.
#include "h3_internal.cuh"
#include "ptx.cuh"

namespace h3 {

namespace attn_bwd {
using attn_detail::HALF_BYTES;
using attn_detail::TILE;
using attn_detail::TILE_BYTES;
using attn_split::tmem_st16;

// Warp 0 TMA, warp 1 MMA, warps 2-17 elementwise: lane quarter w % 4, 32 of the
// tile's 128 columns
constexpr int THREADS = 18 * 32;
constexpr int CWARPS = 16;

struct BwdMaps {
  CUtensorMap q, k, v;  // [H][L][128] (row stride 128, head stride L_pad * 128)
  CUtensorMap d;        // dO, token-major [L][H * 128]
};

__device__ __forceinline__ void load_head_tile(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int row, int h) {
  tma_load_3d(dst, m, bar, 0, row, h);
  tma_load_3d(dst + HALF_BYTES, m, bar, 64, row, h);
}
__device__ __forceinline__ void load_token_tile(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int row, int h) {
  tma_load_2d(dst, m, bar, h * 128, row);
  tma_load_2d(dst + HALF_BYTES, m, bar, h * 128 + 64, row);
}

// D = A B^T over d = 128, both K-major 128 x 128 tiles
__device__ __forceinline__ void mma_abt(uint32_t d_tmem, uint64_t ad, uint64_t bd) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint64_t off = (uint64_t)(((kk >> 2) * HALF_BYTES + (kk & 3) * 32) >> 4);
    umma_bf16(d_tmem, ad + off, bd + off, idesc, kk != 0 ? 1u : 0u);
  }
}
// D (+)= A B over 128 rows of B: A packed bf16 in TMEM, columns of 32-wide group
// g at a_tmem + 32 g .. + 16; B a 128 x 128 tile taken MN-major
__device__ __forceinline__ void mma_tmem_ab(uint32_t d_tmem, uint32_t a_tmem, uint64_t bd, bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, true);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    umma_bf16_tmem_a(d_tmem, a_tmem + (kk >> 1) * 32 + (kk & 1) * 8, bd + (uint64_t)((kk * 2048) >> 4), idesc,
                     (accumulate || kk != 0) ? 1u : 0u);
}

// 2^(s c + b) for a pair of scores, in place
__device__ __forceinline__ void exp2_pair(float* s, uint64_t c2, uint64_t b2) {
  float x0, x1;
  f2_unpack(f2_fma(f2_pack(s[0], s[1]), c2, b2), x0, x1);
  s[0] = ex2_approx(x0);
  s[1] = ex2_approx(x1);
}

// 16 lanes x 32 consecutive 32-bit columns: thread t receives rows t / 4
// (r[4i], r[4i + 1]) and t / 4 + 8 (r[4i + 2], r[4i + 3]) of columns 8i + 2 (t % 4)
// and the next, i < 4.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 lanes x 16 consecutive 32-bit columns: thread t gives rows t / 4 (r[2i])
// and t / 4 + 8 (r[2i + 1]) of column 4i + t % 4: the bf16 pairs of the values
// that tmem_ld_16x256b_x4 gave it.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 columns of one row of an fp32 accumulator, scaled, as bf16
__device__ __forceinline__ void store_cols32(uint32_t taddr, float scale, bf16* dst) {
  float v[32];
  tmem_ld32(taddr, reinterpret_cast<uint32_t*>(v));
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 32; j += 8)
    *reinterpret_cast<uint4*>(dst + j) =
        make_uint4(pack_bf16x2(v[j] * scale, v[j + 1] * scale), pack_bf16x2(v[j + 2] * scale, v[j + 3] * scale),
                   pack_bf16x2(v[j + 4] * scale, v[j + 5] * scale), pack_bf16x2(v[j + 6] * scale, v[j + 7] * scale));
}
__device__ __forceinline__ void zero_cols32(bf16* dst) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) *reinterpret_cast<uint4*>(dst + j) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------ dK, dV
// TMEM: S^T [0, 128), dP^T [128, 256) with P^T and dS^T (bf16, half a column
// each) over it, dV, dK.  S^T(i) is free as soon as it is in registers, so the
// next one is taken while its exponentials run, and the tensor core's turn is
//   dV(i) dK(i) dP^T(i + 1) S^T(i + 2)
// where dV waits for P^T(i), which is stored the moment dP^T(i) has been read,
// while S^T(i + 1), already issued, runs; dK for dS^T(i); and S^T(i + 2) for
// S^T(i + 1) to be in registers.
struct KvLayout {
  static constexpr int QS = 3;  // Q stages: Q(i + 2) for S^T(i + 2) is loaded while dK(i) still reads Q(i)
  static constexpr int K = 0, V = TILE_BYTES, Q = 2 * TILE_BYTES, D = Q + QS * TILE_BYTES;  // dO: two stages
  static constexpr int STAT = D + 2 * TILE_BYTES;  // [2][-lse log2 e, -delta][128]
  static constexpr int BAR = STAT + 2 * 2 * 128 * 4;
  static constexpr int BYTES = BAR + 256;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

struct BwdArgs {
  const bf16 *o, *d;  // [L_pad][H * 128]
  const float* lse;   // [H][L_pad]
  // Row statistics [H][L_pad], which the query tiles leave for the key tiles:
  // -lse log2(e) (-inf past L: P = 0) and -delta (0 past L)
  float *nlse2, *ndelta;
  int H, L, L_pad;
  float scale, scale_log2;
  bf16 *dq, *dk, *dv;
};

__device__ __forceinline__ void key_tile(const BwdMaps& maps, const BwdArgs& p, int tile, int h, uint8_t* smem) {
  const float *nlse2 = p.nlse2, *ndelta = p.ndelta;
  const int L = p.L, L_pad = p.L_pad;
  const float scale = p.scale, scale_log2 = p.scale_log2;
  bf16 *dk = p.dk, *dv = p.dv;
  using Y = KvLayout;
  constexpr int QS = Y::QS;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Y::BAR);
  uint64_t* kv_full = bars + 0;
  uint64_t* q_full = bars + 1;    // [3]
  uint64_t* q_empty = bars + 4;   // [3] after dK of the tile
  uint64_t* d_full = bars + 7;    // [2]
  uint64_t* d_empty = bars + 9;   // [2] after dV of the tile
  uint64_t* st_full = bars + 11;  // [2] the rows' statistics
  uint64_t* st_empty = bars + 13; // [2] read by every elementwise warp
  uint64_t* s_full = bars + 15;
  uint64_t* s_read = bars + 16;   // S^T in registers
  uint64_t* dp_full = bars + 17;
  uint64_t* p_ready = bars + 18;
  uint64_t* ds_ready = bars + 19;
  uint64_t* acc_full = bars + 20;
  uint64_t* drain = bars + 21;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 22);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int key0 = tile * TILE;
  const int n_q = (L + TILE - 1) / TILE;
  if (key0 >= L) {  // a tile of padding rows
    for (int i = threadIdx.x; i < TILE * 16; i += THREADS) {
      const long at = ((long)h * L_pad + key0 + (i >> 4)) * 16 + (i & 15);
      reinterpret_cast<uint4*>(dk)[at] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(dv)[at] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&d_full[s], 1);
      mbar_init(&d_empty[s], 1);
      mbar_init(&st_full[s], 1);
      mbar_init(&st_empty[s], CWARPS);
    }
    mbar_init(s_full, 1);
    mbar_init(s_read, CWARPS);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, CWARPS);
    mbar_init(ds_ready, CWARPS);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.d);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * TILE_BYTES);
      load_head_tile(smem + Y::K, &maps.k, kv_full, key0, h);
      load_head_tile(smem + Y::V, &maps.v, kv_full, key0, h);
      long long q_issued = 0, st_issued = 0, d_issued = 0;
      for (int i = 0; i < n_q; ++i) {
        const int sq = i % QS, st = i & 1;
        const uint32_t ph = ((i >> 1) & 1) ^ 1;
        if (!mbar_wait(&q_empty[sq], ((i / QS) & 1) ^ 1)) break;
        mbar_arrive_expect_tx(&q_full[sq], TILE_BYTES);
        load_head_tile(smem + Y::Q + sq * TILE_BYTES, &maps.q, &q_full[sq], i * TILE, h);
        ++q_issued;
        if (!mbar_wait(&d_empty[st], ph)) break;
        mbar_arrive_expect_tx(&d_full[st], TILE_BYTES);
        load_token_tile(smem + Y::D + st * TILE_BYTES, &maps.d, &d_full[st], i * TILE, h);
        ++d_issued;
        if (!mbar_wait(&st_empty[st], ph)) break;
        mbar_arrive_expect_tx(&st_full[st], 2 * 128 * 4);
        const long at = (long)h * L_pad + i * TILE;
        bulk_load(smem + Y::STAT + st * 1024, nlse2 + at, 512, &st_full[st]);
        bulk_load(smem + Y::STAT + st * 1024 + 512, ndelta + at, 512, &st_full[st]);
        ++st_issued;
      }
      mbar_wait(kv_full, 0);
      drain_loads(q_full, QS, q_issued);
      drain_loads(d_full, 2, d_issued);
      drain_loads(st_full, 2, st_issued);
    }
  } else if (warp == 1) {
    const uint64_t kd = sdesc_sw128(smem_u32(smem + Y::K), 16, 1024);
    const uint64_t vd = sdesc_sw128(smem_u32(smem + Y::V), 16, 1024);
    const uint64_t qd = sdesc_sw128(smem_u32(smem + Y::Q), 16, 1024);
    const uint64_t dd = sdesc_sw128(smem_u32(smem + Y::D), 16, 1024);
    const uint64_t qd_mn = sdesc_sw128(smem_u32(smem + Y::Q), HALF_BYTES, 1024);
    const uint64_t dd_mn = sdesc_sw128(smem_u32(smem + Y::D), HALF_BYTES, 1024);
    constexpr uint64_t ST = TILE_BYTES >> 4;
    auto issue_s = [&](int i) {
      if (!mbar_wait_warp(&q_full[i % QS], (i / QS) & 1)) return false;
      if (i > 0 && !mbar_wait_warp(s_read, (i - 1) & 1)) return false;
      tc_fence_after();
      mma_abt(tmem, kd, qd + (uint64_t)(i % QS) * ST);
      umma_commit(s_full);
      return true;
    };
    auto issue_dp = [&](int i) {
      if (!mbar_wait_warp(&d_full[i & 1], (i >> 1) & 1)) return false;
      tc_fence_after();
      mma_abt(tmem + 128, vd, dd + (uint64_t)(i & 1) * ST);
      umma_commit(dp_full);
      return true;
    };
    bool ok = mbar_wait_warp(kv_full, 0) && issue_s(0) && issue_dp(0) && (n_q < 2 || issue_s(1));
    for (int i = 0; i < n_q && ok; ++i) {
      if (!mbar_wait_warp(p_ready, i & 1)) { ok = false; break; }
      tc_fence_after();
      mma_tmem_ab(tmem + 256, tmem + 128, dd_mn + (uint64_t)(i & 1) * ST, i != 0);
      umma_commit(&d_empty[i & 1]);
      if (!mbar_wait_warp(ds_ready, i & 1)) { ok = false; break; }
      tc_fence_after();
      mma_tmem_ab(tmem + 384, tmem + 128 + 16, qd_mn + (uint64_t)(i % QS) * ST, i != 0);
      umma_commit(&q_empty[i % QS]);
      ok = (i + 1 >= n_q || issue_dp(i + 1)) && (i + 2 >= n_q || issue_s(i + 2));
    }
    umma_commit(acc_full);
    drain_mmas(drain);
  } else {
    const int qw = warp & 3, g = (warp - 2) >> 2;  // TMEM lane quarter, 32-column group
    const int r = qw * 32 + lane;                  // key row of the tile (epilogue)
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    const uint32_t tS = tmem + lanes + g * 32, tP = tS + 128;
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    bool ok = true;
    // The statistics belong to the columns (queries).  With one key row per
    // thread a warp would read 32 + 32 of them for every thread, 1,024 clocks
    // of the shared-memory pipe per tile (measured: 14% of the kernel); in the
    // 16-lane layout a thread holds four rows of eight columns and reads 8 + 8.
    for (int i = 0; i < n_q; ++i) {
      const float2* st = reinterpret_cast<const float2*>(smem + Y::STAT + (i & 1) * 1024) + g * 16 + (lane & 3);
      ok = mbar_wait_warp(&st_full[i & 1], (i >> 1) & 1) && mbar_wait_warp(s_full, i & 1);
      if (!ok) break;
      tc_fence_after();
      float pr[2][16];
      uint32_t pk[2][8];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        tmem_ld_16x256b_x4(tS + ((uint32_t)(hh * 16) << 16), reinterpret_cast<uint32_t*>(pr[hh]));
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_read);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 nl = st[c * 4];
        const uint64_t nl2 = f2_pack(nl.x, nl.y);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          exp2_pair(pr[hh] + c * 4, sc2, nl2);
          exp2_pair(pr[hh] + c * 4 + 2, sc2, nl2);
          pk[hh][c * 2] = pack_bf16x2(pr[hh][c * 4], pr[hh][c * 4 + 1]);
          pk[hh][c * 2 + 1] = pack_bf16x2(pr[hh][c * 4 + 2], pr[hh][c * 4 + 3]);
        }
      }
      ok = mbar_wait_warp(dp_full, i & 1);
      if (!ok) break;
      tc_fence_after();
      float dp[2][16];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        tmem_ld_16x256b_x4(tP + ((uint32_t)(hh * 16) << 16), reinterpret_cast<uint32_t*>(dp[hh]));
      tmem_wait_ld();
      // the warp's own 32 columns of dP^T are read: P^T over the first 16
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) tmem_st_16x128b_x4(tP + ((uint32_t)(hh * 16) << 16), pk[hh]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 nd = st[64 + c * 4];
        const uint64_t nd2 = f2_pack(nd.x, nd.y);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int j = c * 4 + e;
            float a, b;
            f2_unpack(f2_mul(f2_pack(pr[hh][j], pr[hh][j + 1]), f2_add(f2_pack(dp[hh][j], dp[hh][j + 1]), nd2)), a, b);
            pk[hh][c * 2 + e / 2] = pack_bf16x2(a, b);
          }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) tmem_st_16x128b_x4(tP + 16 + ((uint32_t)(hh * 16) << 16), pk[hh]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_ready);
        mbar_arrive(&st_empty[i & 1]);
      }
    }
    ok = ok && mbar_wait_warp(acc_full, 0);
    if (ok) {
      tc_fence_after();
      // group 0, 1: the halves of dV; 2, 3: of dK
      bf16* dst = (g < 2 ? dv : dk) + ((long)h * L_pad + key0 + r) * 128 + (g & 1) * 64;
      const uint32_t src = tmem + lanes + 256 + g * 64;
      const float sc = g < 2 ? 1.0f : scale;
      const bool valid = key0 + r < L;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        store_cols32(src + c * 32, sc, dst + c * 32);
        if (!valid) zero_cols32(dst + c * 32);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------ dQ
// The same pipeline on a query tile: TMEM S(j) [0, 128), dP(j) [128, 256) with P
// and dS (bf16) over it, the running dS K [256, 384) and P K [384, 512).  Both
// read K(j) and P(j) or dS(j):
//   PK(j) dSK(j) dP(j + 1) S(j + 2)
// with the waits of the key tiles.  K has three stages, as Q has there.
struct QLayout {
  static constexpr int KS = 3, VS = 2;
  static constexpr int Q = 0, D = TILE_BYTES, K = 2 * TILE_BYTES, V = K + KS * TILE_BYTES;
  static constexpr int SUM = V + VS * TILE_BYTES;  // [4 column groups][128 rows] sums of do o, then of dS
  static constexpr int BAR = SUM + 4 * 128 * 4;
  static constexpr int BYTES = BAR + 256;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void query_tile(const BwdMaps& maps, const BwdArgs& p, int tile, int h, uint8_t* smem) {
  const int L = p.L, L_pad = p.L_pad, H = p.H;
  const float scale = p.scale, scale_log2 = p.scale_log2;
  bf16* dq = p.dq;
  using Y = QLayout;
  constexpr int KS = Y::KS, VS = Y::VS;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Y::BAR);
  uint64_t* qd_full = bars + 0;
  uint64_t* k_full = bars + 1;       // [KS]
  uint64_t* k_empty = k_full + KS;   // [KS] after dS K of the tile
  uint64_t* v_full = k_empty + KS;   // [VS]
  uint64_t* v_empty = v_full + VS;   // [VS] after dP of the tile
  uint64_t* s_full = v_empty + VS;
  uint64_t* s_read = s_full + 1;     // S in registers
  uint64_t* dp_full = s_full + 2;
  uint64_t* p_ready = s_full + 3;
  uint64_t* ds_ready = s_full + 4;
  uint64_t* acc_full = s_full + 5;
  uint64_t* drain = s_full + 6;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 7);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row0 = tile * TILE;
  const int n_k = (L + TILE - 1) / TILE;
  if (row0 >= L) {  // a tile of padding rows
    for (int i = threadIdx.x; i < TILE * 16; i += THREADS)
      reinterpret_cast<uint4*>(dq)[((long)h * L_pad + row0 + (i >> 4)) * 16 + (i & 15)] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(qd_full, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_read, CWARPS);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, CWARPS);
    mbar_init(ds_ready, CWARPS);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      mbar_arrive_expect_tx(qd_full, 2 * TILE_BYTES);
      load_head_tile(smem + Y::Q, &maps.q, qd_full, row0, h);
      load_token_tile(smem + Y::D, &maps.d, qd_full, row0, h);
      long long k_issued = 0, v_issued = 0;
      for (int j = 0; j < n_k; ++j) {
        const int sk = j % KS, sv = j % VS;
        if (!mbar_wait(&k_empty[sk], ((j / KS) & 1) ^ 1)) break;
        mbar_arrive_expect_tx(&k_full[sk], TILE_BYTES);
        load_head_tile(smem + Y::K + sk * TILE_BYTES, &maps.k, &k_full[sk], j * TILE, h);
        ++k_issued;
        if (!mbar_wait(&v_empty[sv], ((j / VS) & 1) ^ 1)) break;
        mbar_arrive_expect_tx(&v_full[sv], TILE_BYTES);
        load_head_tile(smem + Y::V + sv * TILE_BYTES, &maps.v, &v_full[sv], j * TILE, h);
        ++v_issued;
      }
      mbar_wait(qd_full, 0);
      drain_loads(k_full, KS, k_issued);
      drain_loads(v_full, VS, v_issued);
    }
  } else if (warp == 1) {
    const uint64_t qd = sdesc_sw128(smem_u32(smem + Y::Q), 16, 1024);
    const uint64_t dd = sdesc_sw128(smem_u32(smem + Y::D), 16, 1024);
    const uint64_t kd = sdesc_sw128(smem_u32(smem + Y::K), 16, 1024);
    const uint64_t vd = sdesc_sw128(smem_u32(smem + Y::V), 16, 1024);
    const uint64_t kd_mn = sdesc_sw128(smem_u32(smem + Y::K), HALF_BYTES, 1024);
    constexpr uint64_t ST = TILE_BYTES >> 4;
    auto issue_s = [&](int j) {
      if (!mbar_wait_warp(&k_full[j % KS], (j / KS) & 1)) return false;
      if (j > 0 && !mbar_wait_warp(s_read, (j - 1) & 1)) return false;
      tc_fence_after();
      mma_abt(tmem, qd, kd + (uint64_t)(j % KS) * ST);
      umma_commit(s_full);
      return true;
    };
    auto issue_dp = [&](int j) {
      if (!mbar_wait_warp(&v_full[j % VS], (j / VS) & 1)) return false;
      tc_fence_after();
      mma_abt(tmem + 128, dd, vd + (uint64_t)(j % VS) * ST);
      umma_commit(dp_full);
      umma_commit(&v_empty[j % VS]);
      return true;
    };
    bool ok = mbar_wait_warp(qd_full, 0) && issue_s(0) && issue_dp(0) && (n_k < 2 || issue_s(1));
    for (int j = 0; j < n_k && ok; ++j) {
      if (!mbar_wait_warp(p_ready, j & 1)) { ok = false; break; }
      tc_fence_after();
      mma_tmem_ab(tmem + 384, tmem + 128, kd_mn + (uint64_t)(j % KS) * ST, j != 0);
      if (!mbar_wait_warp(ds_ready, j & 1)) { ok = false; break; }
      tc_fence_after();
      mma_tmem_ab(tmem + 256, tmem + 128 + 16, kd_mn + (uint64_t)(j % KS) * ST, j != 0);
      umma_commit(&k_empty[j % KS]);
      ok = (j + 1 >= n_k || issue_dp(j + 1)) && (j + 2 >= n_k || issue_s(j + 2));
    }
    umma_commit(acc_full);
    drain_mmas(drain);
  } else {
    const int qw = warp & 3, g = (warp - 2) >> 2;
    const int r = qw * 32 + lane;  // query row of the tile
    const uint32_t lanes = (uint32_t)(qw * 32) << 16;
    const uint32_t tS = tmem + lanes + g * 32, tP = tS + 128;
    const long at = (long)h * L_pad + row0 + r;
    const bool in = row0 + r < L;
    float* sums = reinterpret_cast<float*>(smem + Y::SUM) + r;
    // a sum over the row's four warps, added in the same order by each
    auto row_sum = [&](float part) {
      sums[g * 128] = part;
      named_barrier_sync(1, CWARPS * 32);
      return (sums[0] + sums[128]) + (sums[256] + sums[384]);
    };
    const float nl = in ? -p.lse[at] * 1.4426950408889634f : -INFINITY;
    float nd = 0.f;
    if (in) {
      const long col = (long)(row0 + r) * H * 128 + h * 128 + g * 32;
      const uint4 *po = reinterpret_cast<const uint4*>(p.o + col), *pd = reinterpret_cast<const uint4*>(p.d + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = __ldg(po + i), w = __ldg(pd + i);
        const __nv_bfloat162 *pu = reinterpret_cast<const __nv_bfloat162*>(&u),
                             *pw = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = __bfloat1622float2(pu[e]), y = __bfloat1622float2(pw[e]);
          nd = fmaf(-x.x, y.x, nd);
          nd = fmaf(-x.y, y.y, nd);
        }
      }
    }
    nd = row_sum(nd);
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
    uint64_t ds_sum = 0ull;  // of this warp's columns of the row, as they are before their rounding
    bool ok = true;
    for (int j = 0; j < n_k; ++j) {
      ok = mbar_wait_warp(s_full, j & 1);
      if (!ok) break;
      tc_fence_after();
      float pr[32], dp[32];
      uint32_t pk[16];
      tmem_ld32(tS, reinterpret_cast<uint32_t*>(pr));
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_read);
#pragma unroll
      for (int c = 0; c < 32; c += 2) exp2_pair(pr + c, sc2, nl2);
      const int valid = L - j * TILE - g * 32;
      if (valid < 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c >= valid) pr[c] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < 32; c += 2) pk[c / 2] = pack_bf16x2(pr[c], pr[c + 1]);
      ok = mbar_wait_warp(dp_full, j & 1);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(tP, reinterpret_cast<uint32_t*>(dp));
      tmem_wait_ld();
      // the warp's own 32 columns of dP are read: P over the first 16
      tmem_st16(tP, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const uint64_t ds = f2_mul(f2_pack(pr[c], pr[c + 1]), f2_add(f2_pack(dp[c], dp[c + 1]), nd2));
        ds_sum = f2_add(ds_sum, ds);
        float a, b;
        f2_unpack(ds, a, b);
        pk[c / 2] = pack_bf16x2(a, b);
      }
      tmem_st16(tP + 16, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);
    }
    // (every warp has left the sums above before the first tile's dS K)
    float s0, s1;
    f2_unpack(ds_sum, s0, s1);
    const float rest = row_sum(s0 + s1);
    ok = ok && mbar_wait_warp(acc_full, 0);
    if (ok) {
      tc_fence_after();
      bf16* dst = dq + at * 128 + g * 32;
      float a[32], b[32];
      tmem_ld32(tmem + lanes + 256 + g * 32, reinterpret_cast<uint32_t*>(a));
      tmem_ld32(tmem + lanes + 384 + g * 32, reinterpret_cast<uint32_t*>(b));
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; ++c) a[c] = fmaf(-rest, b[c], a[c]) * scale;
#pragma unroll
      for (int c = 0; c < 32; c += 8)
        *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack_bf16x2(a[c], a[c + 1]), pack_bf16x2(a[c + 2], a[c + 3]),
                                                        pack_bf16x2(a[c + 4], a[c + 5]), pack_bf16x2(a[c + 6], a[c + 7]));
      if (!in) zero_cols32(dst);
      if (g == 0) {
        p.nlse2[at] = nl;
        p.ndelta[at] = in ? nd - rest : 0.f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A CTA a tile: KEYS the key tiles, else the query tiles, which go first and
// leave the deltas that the key tiles read.
template <bool KEYS>
__global__ void __launch_bounds__(THREADS, 1)
    attention_bwd_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs p, int n) {
  // seven tiles leave no room to align the base by hand: the swizzled tiles
  // need 1 KB alignment, which the declaration asks for and this check holds
  extern __shared__ __align__(1024) uint8_t smem_bwd[];
  chain_wait();
  if (smem_u32(smem_bwd) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(&g_h3_device_error, 0, 1);
    return;
  }
  if constexpr (KEYS)
    key_tile(maps, p, blockIdx.x % n, blockIdx.x / n, smem_bwd);
  else
    query_tile(maps, p, blockIdx.x % n, blockIdx.x / n, smem_bwd);
}

// [H][L_pad][128] heads as 64 x 128-row boxes whose rows end at L
bool make_tmap_heads(CUtensorMap* map, const void* base, int H, int L, int L_pad) {
  gemm_detail::EncodeTiledFn fn = gemm_detail::encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[3] = {128, (cuuint64_t)L, (cuuint64_t)H};
  cuuint64_t gstride[2] = {256, (cuuint64_t)L_pad * 256};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn_bwd

// ws: nlse2 and ndelta, [H][L_pad] fp32 each
cudaError_t launch_attention_bwd(const bf16* q, const bf16* k, const bf16* v, const bf16* o, const float* lse,
                                 const bf16* d, int H, int L, int L_pad, float scale, float scale_log2, bf16* dq,
                                 bf16* dk, bf16* dv, float* ws, cudaStream_t stream) {
  using namespace attn_bwd;
  static unsigned long long done[2] = {0, 0};
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(attention_bwd_kernel<false>), QLayout::BYTES, &done[0]);
  if (e != cudaSuccess) return e;
  e = ensure_smem_attr(reinterpret_cast<const void*>(attention_bwd_kernel<true>), KvLayout::BYTES, &done[1]);
  if (e != cudaSuccess) return e;
  BwdMaps maps;
  if (!make_tmap_heads(&maps.q, q, H, L, L_pad) || !make_tmap_heads(&maps.k, k, H, L, L_pad) ||
      !make_tmap_heads(&maps.v, v, H, L, L_pad) || !make_tmap_bf16(&maps.d, d, L, 128L * H, 128L * H, 128))
    return cudaErrorInvalidValue;
  const int n = L_pad / attn_detail::TILE;
  const BwdArgs args{o, d, lse, ws, ws + (size_t)H * L_pad, H, L, L_pad, scale, scale_log2, dq, dk, dv};
  e = launch_chained(attention_bwd_kernel<false>, dim3(n * H), THREADS, QLayout::BYTES, stream, maps, args, n);
  if (e != cudaSuccess) return e;
  return launch_chained(attention_bwd_kernel<true>, dim3(n * H), THREADS, KvLayout::BYTES, stream, maps, args, n);
}

}  // namespace h3
