// tcgen05 GEMMs of the block's backward pass, all on CTA pairs (cta_group::2,
// 256 x 256 output tiles over two SMs, fp32 accumulators in TMEM):
//
//   DGRAD   out[t][n] = sum_k A[t][k] B[k][n]: the gradient of a linear's input.
//           B is the forward weight [out, in] read with its rows as the
//           contraction, so no transposed copy of a weight exists: its tiles
//           enter shared memory as they lie (64 columns x 64 rows per TMA box)
//           and the MMA takes them MN-major.
//   WGRAD   out[j][n] = sum_t A[t][j] B[t][n]: the gradient of a weight; both
//           operands MN-major, the contraction over the tokens.
//   GATED   WGRAD for a linear behind a modality gate (y = gate_m (.) (B W^T)):
//           one accumulator per modality range, G_m = sum_{t in m} A^T B, then
//             dW[j][n]    = sum_m gate_m[j] G_m[j][n]
//             dgate_m[j]  = sum_n W[j][n] G_m[j][n]
//           (the second is sum_t dx[t][j] (B W^T)[t][j] with the order of the
//           sums exchanged), so the gate's gradient needs neither the branch
//           output nor another product, and a gate of 0 loses nothing.
//   QKNORM  x = A W_qk^T (the q, k projection again), and in the epilogue the
//           backward pass of RoPE and of the per-head RMSNorm.
//   FFN     gate, up = A Wgu^T and dh = dY Wd in one K loop, and in the epilogue
//           h = SiLU(g) u and the gradients of g and u.
//
// A segment, a ragged length and the padding rows end inside a tile: the tensor
// maps stop at the last valid token, and TMA reads zeros past it.
#include "h3_internal.cuh"
#include "ptx.cuh"

namespace h3 {

namespace gemm_bwd {
using gemm_detail::tile_coords;

enum Kind : int { DGRAD = 0, WGRAD = 1, GATED = 2, QKNORM = 3, FFN = 4 };

struct Maps {
  CUtensorMap a[3], b[3];  // per segment (GATED), else index 0; FFN: a[1], b[1] are dY and Wd
  CUtensorMap w;           // GATED: W, 128-row boxes
};

struct Params {
  int M, N, K;  // output rows and columns; contraction length (unused by WGRAD, GATED)
  int m_tiles, n_tiles, group_m;
  // The contraction in `splits` equal runs of k blocks, each a unit of work of
  // its own that writes an fp32 partial, part [splits][M][N]; 1: none
  int splits;
  float* part;
  int rows;           // valid token rows
  int seg_rows[3];    // WGRAD: [0] = rows; GATED: tokens of each modality
  bf16* out;          // DGRAD, WGRAD, GATED (may be null): [M][ldo]
  long ldo;
  // GATED
  const float* mod;   // [3][6][D]
  int gate_slot, D;
  int gate_grad;      // whether the gate's gradient is wanted
  float* gate_part;   // [3][splits * 4 n_tiles][M] column-quarter partials of the gate's gradient
  // FFN
  bf16* h;            // [.][F]
  bf16* dgu;          // [.][2F]
  int F;
  // QKNORM
  const bf16* dq;     // [H][L_pad][128], gradients of the rotated q and k
  const bf16* dk;
  const bf16* qn_w;
  const bf16* kn_w;
  const float* pos;   // [L_pad][3]
  int L_pad, I, rope_t, rope_h, rope_w;
  float theta, eps_qk;
  float* w_part;      // [CTAs][2][128] partials of the norm weights' gradients
};

constexpr int BK = 64;
constexpr int OPERAND = 128 * BK * 2;  // one 128 x 64 operand tile of a CTA, 16 KB
template <int KIND>
struct Cfg {
  static constexpr bool FFN_ = KIND == FFN;
  static constexpr int STAGES = FFN_ || KIND == GATED ? 4 : 6;
  // FFN: xm, dY (16 KB each), gate or up rows of Wgu (16 KB), 64 columns of Wd (8 KB)
  static constexpr int STAGE = FFN_ ? 3 * OPERAND + OPERAND / 2 : 2 * OPERAND;
  static constexpr int ACCS = FFN_ ? 1 : 2;  // TMEM accumulators: 256 + 128 columns, or 2 x 256
  // Warp 0 TMA, warp 1 MMA, then EW epilogue warps: EW / 4 of each TMEM lane
  // quarter, sharing the tile's columns.  Sixteen hide the latency of the
  // TMEM and global accesses of one tile; QKNORM needs a head's 128 columns in
  // one warp and has eight.
  static constexpr int EW = KIND == QKNORM ? 8 : 16;
  // GATED: one more warp loads the tile of W that the gate's gradient needs
  static constexpr int THREADS = (2 + EW + (KIND == GATED ? 1 : 0)) * 32;
  static constexpr int WTILE = KIND == GATED ? 4 * OPERAND : 0;  // 128 rows x 256 columns
  static constexpr int MISC = 768;
  static constexpr int NORM = KIND == QKNORM ? 8 * 2 * 128 * 4 : 0;  // [epilogue warp][q, k][128]
  static constexpr int BYTES = STAGES * STAGE + WTILE + 1024 + MISC + NORM;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void ld_chunk(uint32_t taddr, float* v) {
  tmem_ld32(taddr, reinterpret_cast<uint32_t*>(v));
}
// 32 lanes x 16 consecutive 32-bit columns
__device__ __forceinline__ void ld_chunk16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st_v4(uint32_t* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 8 words of row m (lane = m % 32): 16 bf16 or 8 fp32 columns; ld in words.
// Lanes 2i and 2i + 1 exchange halves so that each store instruction writes
// whole 32-byte sectors: first the even rows', then the odd rows'.
// Warp-collective.
__device__ __forceinline__ void store8w(uint32_t* dst, long ld, int m, int M, const uint32_t* w) {
  const bool odd = (threadIdx.x & 1) != 0;
  uint32_t t[4], e[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = __shfl_xor_sync(0xffffffffu, odd ? w[i] : w[4 + i], 1);
    e[i] = odd ? t[i] : w[i];
    o[i] = odd ? w[4 + i] : t[i];
  }
  // the lane's place in the even and in the odd row of its pair
  uint32_t* pe = dst + (odd ? 4 - ld : 0L);
  uint32_t* po = dst + (odd ? 4L : ld);
  if ((m & ~1) < M) st_v4(pe, e[0], e[1], e[2], e[3]);
  if ((m | 1) < M) st_v4(po, o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store16(bf16* dst, long ld, int m, int M, const uint32_t* w) {
  store8w(reinterpret_cast<uint32_t*>(dst), ld / 2, m, M, w);
}
// the warp's columns [n0, n0 + COLS) of one split's fp32 partial [M][N]
template <int COLS>
__device__ __forceinline__ void store_part(float* part, int N, int n0, int m, int M, const float* v) {
#pragma unroll
  for (int c = 0; c < COLS; c += 8)
    if (n0 + c < N)
      store8w(reinterpret_cast<uint32_t*>(part + (long)m * N + n0 + c), N, m, M, reinterpret_cast<const uint32_t*>(v + c));
}
template <int N>
__device__ __forceinline__ void pack_row(const float* v, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N; i += 2) w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
}
__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(b[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

// One 32-column chunk of d(rotated q or k) of a token and head, turned back by
// the token's angles: (a, b) = (d0 cos + d1 sin, d1 cos - d0 sin), the
// transpose of the forward rotation.
__device__ __forceinline__ void unrotate32(const bf16* d, bool valid, const float* p3, const float* freq,
                                           const uint8_t* axis, int c, float* t) {
  if (!valid) {
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = 0.f;
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; j += 8) unpack8(__ldg(reinterpret_cast<const uint4*>(d + c * 32 + j)), t + j);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int ip = c * 16 + i, ax = axis[ip];
    const float pa = ax == 0 ? p3[0] : (ax == 1 ? p3[1] : p3[2]);
    float sn, cs;
    gemm_detail::rope_sincos(pa * freq[ip], &sn, &cs);
    const float a = t[2 * i], b = t[2 * i + 1];
    t[2 * i] = a * cs + b * sn;
    t[2 * i + 1] = b * cs - a * sn;
  }
}

// RMSNorm backward of one head row: x raw (TMEM), xhat = x inv, dh = t (.) w,
// dx = inv (dh - xhat mean(dh xhat)); with s = sum dh x, mean(dh xhat) =
// s inv / 128.  Two passes over the row's four chunks; sum_t t xhat, the
// gradient of w, goes to wacc[128] of this warp.
template <typename Release>
__device__ __forceinline__ void epi_qknorm(const Params& p, uint32_t tb, int m, int n, const float* freq,
                                           const uint8_t* axis, float* wacc2, Release release) {
  const int lane = threadIdx.x & 31;
  const int part = n / p.I, hd = (n % p.I) / 128;
  const bool valid = m < p.rows;
  const bf16* d = (part == 0 ? p.dq : p.dk) + ((long)hd * p.L_pad + (valid ? m : 0)) * 128;
  const bf16* w = part == 0 ? p.qn_w : p.kn_w;
  float* wacc = wacc2 + part * 128;
  float p3[3] = {0.f, 0.f, 0.f};
  if (valid) {
    p3[0] = p.pos[(long)m * 3];
    p3[1] = p.pos[(long)m * 3 + 1];
    p3[2] = p.pos[(long)m * 3 + 2];
  }
  float ss = 0.f, s = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float x[32], t[32];
    ld_chunk(tb + c * 32, x);
    unrotate32(d, valid, p3, freq, axis, c, t);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      float wv[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(w + c * 32 + j)), wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(x[j + i], x[j + i], ss);
        s = fmaf(t[j + i] * wv[i], x[j + i], s);
      }
    }
  }
  const float inv = rsqrtf(ss * (1.0f / 128.0f) + p.eps_qk);
  const float mean = s * inv * (1.0f / 128.0f);
  uint32_t out[64];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x[32], t[32];
    ld_chunk(tb + c * 32, x);
    unrotate32(d, valid, p3, freq, axis, c, t);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      float wv[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(w + c * 32 + j)), wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[j + i] * inv;
        x[j + i] = inv * (t[j + i] * wv[i] - xh * mean);
        t[j + i] *= xh;
      }
    }
    pack_row<32>(x, out + c * 16);
    // sum over the warp's 32 rows: lane l ends with column l of the chunk
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float send = up ? t[i] : t[i + o], keep = up ? t[i + o] : t[i];
        t[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
    wacc[c * 32 + lane] += t[0];
  }
  release();
  bf16* dst = p.out + (long)m * p.ldo + n;
#pragma unroll
  for (int c = 0; c < 8; ++c) store16(dst + c * 16, p.ldo, m, p.rows, out + c * 8);
}

// h = SiLU(g) u, du = dh SiLU(g), dg = dh u sig(g) (1 + g (1 - sig(g))) for 32 of
// the tile's 128 hidden columns; accumulator columns [0, 128) g, [128, 256) u,
// [256, 384) dh
template <typename Release>
__device__ __forceinline__ void epi_ffn(const Params& p, uint32_t tb, int m, int nt, int sub, Release release) {
  uint32_t hw[16], gw[16], uw[16];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float g[16], u[16], dh[16];
    const uint32_t t0 = tb + sub * 32 + c * 16;
    ld_chunk16(t0, g);
    ld_chunk16(t0 + 128, u);
    ld_chunk16(t0 + 256, dh);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float sig = __fdividef(1.0f, 1.0f + __expf(-g[j]));
      const float act = g[j] * sig;
      const float dact = sig + act * (1.0f - sig);
      const float d = dh[j];
      dh[j] = act * u[j];      // h
      g[j] = d * u[j] * dact;  // dg
      u[j] = d * act;          // du
    }
    pack_row<16>(dh, hw + c * 8);
    pack_row<16>(g, gw + c * 8);
    pack_row<16>(u, uw + c * 8);
  }
  release();
  bf16* hrow = p.h + (long)m * p.F + (long)nt * 128 + sub * 32;
  bf16* grow = p.dgu + (long)m * 2 * p.F + (long)nt * 128 + sub * 32;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    store16(hrow + c * 16, p.F, m, p.rows, hw + c * 8);
    store16(grow + c * 16, 2L * p.F, m, p.rows, gw + c * 8);
    store16(grow + p.F + c * 16, 2L * p.F, m, p.rows, uw + c * 8);
  }
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<KIND>::THREADS, 1)
    gemm_bwd_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = Cfg<KIND>;
  constexpr int STAGES = C::STAGES, STAGE = C::STAGE, EW = C::EW;
  constexpr int COLS = 1024 / EW;  // output columns of an epilogue warp (FFN: 32)
  constexpr bool A_MN = KIND == WGRAD || KIND == GATED;
  constexpr bool B_MN = KIND != QKNORM && KIND != FFN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sW = smem + STAGES * STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE + C::WTILE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* w_full = drain + 1;   // GATED: W of the tile
  uint64_t* w_empty = drain + 2;  // GATED: read by every epilogue warp of this CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 3);
  float* freq = reinterpret_cast<float*>(tmem_slot + 4);
  uint8_t* axis = reinterpret_cast<uint8_t*>(freq + 64);
  float* wacc = reinterpret_cast<float*>(smem + STAGES * STAGE + C::WTILE + C::MISC);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);   // the leader's producer arrives (+ both CTAs' bytes)
      mbar_init(&empty[s], 1);  // the leader's MMA commit, delivered to both CTAs
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);    // the leader's commit, delivered to both CTAs
      mbar_init(&tempty[a], 2 * EW);  // the epilogue warps of both CTAs (leader's copy used)
    }
    mbar_init(drain, 1);
    mbar_init(w_full, 1);
    mbar_init(w_empty, EW);
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if constexpr (KIND == QKNORM) {
    if (threadIdx.x >= 64 && threadIdx.x < 128) {  // rotation frequency and axis of each pair, as the forward call's
      const int i = threadIdx.x - 64;
      const int pt = p.rope_t / 2, ph = p.rope_h / 2;
      int ax, i_sec, d_sec;
      if (i < pt) { ax = 0; i_sec = i; d_sec = p.rope_t; }
      else if (i < pt + ph) { ax = 1; i_sec = i - pt; d_sec = p.rope_h; }
      else { ax = 2; i_sec = i - pt - ph; d_sec = p.rope_w; }
      freq[i] = powf(p.theta, -2.0f * (float)i_sec / (float)d_sec);
      axis[i] = (uint8_t)ax;
    }
    for (int i = threadIdx.x; i < 8 * 2 * 128; i += C::THREADS) wacc[i] = 0.f;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  chain_wait();

  const int num_tiles = p.m_tiles * p.n_tiles;
  const int num_units = num_tiles * p.splits;
  constexpr int SEGS = KIND == GATED ? 3 : 1;
  auto seg_kb = [&](int sg) {
    return (KIND == WGRAD || KIND == GATED) ? (p.seg_rows[sg] + BK - 1) / BK : p.K / BK;
  };
  int kb_total = 0;
  for (int sg = 0; sg < SEGS; ++sg) kb_total += seg_kb(sg);
  const int kb_split = (kb_total + p.splits - 1) / p.splits;
  // k blocks [lo, hi) of segment sg in split sp, the segments' blocks counted
  // one after another
  auto seg_range = [&](int sp, int sg, int& lo, int& hi) {
    int before = 0;
    for (int i = 0; i < sg; ++i) before += seg_kb(i);
    const int n = seg_kb(sg);
    lo = min(n, max(0, sp * kb_split - before));
    hi = max(lo, min(n, (sp + 1) * kb_split - before));
  };

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t leader_full0 = mapa_shared(smem_u32(&full[0]), 0);
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = pair; u < num_units && ok; u += n_pairs) {
        int mt, nt;
        const int sp = u / num_tiles;
        tile_coords(u - sp * num_tiles, p.m_tiles, p.n_tiles, p.group_m, mt, nt);
        const int a0 = mt * 256 + (int)rank * 128;  // this CTA's A rows (or MN-major columns)
        const int b0 = nt * (KIND == FFN ? 128 : 256) + (int)rank * (KIND == FFN ? p.F : 128);
        for (int sg = 0; sg < SEGS && ok; ++sg) {
          int lo, hi;
          seg_range(sp, sg, lo, hi);
          for (int kb = lo; kb < hi; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1)) { ok = false; break; }
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * STAGE);
            const uint32_t fb = leader_full0 + stage * 8;
            uint8_t* sA = smem + stage * STAGE;
            uint8_t* sB = sA + OPERAND;
            if constexpr (A_MN) {
              tma_load_2d_pair(sA, &maps.a[sg], fb, a0, kb * BK);
              tma_load_2d_pair(sA + OPERAND / 2, &maps.a[sg], fb, a0 + 64, kb * BK);
            } else {
              tma_load_2d_pair(sA, &maps.a[0], fb, kb * BK, a0);
            }
            if constexpr (B_MN) {
              tma_load_2d_pair(sB, &maps.b[sg], fb, b0, kb * BK);
              tma_load_2d_pair(sB + OPERAND / 2, &maps.b[sg], fb, b0 + 64, kb * BK);
            } else {
              tma_load_2d_pair(sB, &maps.b[0], fb, kb * BK, b0);
            }
            if constexpr (KIND == FFN) {
              tma_load_2d_pair(sA + 2 * OPERAND, &maps.a[1], fb, kb * BK, a0);
              tma_load_2d_pair(sA + 3 * OPERAND, &maps.b[1], fb, nt * 128 + (int)rank * 64, kb * BK);
            }
            ++issued;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
        }
      }
      // the leader's full barriers count both CTAs' bytes: the leader waits
      // for both, the peer CTA is held by the cluster barrier below
      if (leader) drain_loads(full, STAGES, issued);
    }
  } else if (warp == 1) {
    if (leader) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256, B_MN) | (A_MN ? 1u << 15 : 0u);
      constexpr uint32_t idesc_dh = idesc_bf16_f32(256, 128, true);
      // MN-major operands: 64-column blocks 8 KB apart, 8-row groups 1 KB
      // apart, 16 rows (2 KB) per MMA; K-major: 32 bytes per MMA
      const uint64_t a_desc0 = sdesc_sw128(smem_u32(smem), A_MN ? OPERAND / 2 : 16, 1024);
      const uint64_t b_desc0 = sdesc_sw128(smem_u32(smem + OPERAND), B_MN ? OPERAND / 2 : 16, 1024);
      const uint64_t a2_desc0 = sdesc_sw128(smem_u32(smem + 2 * OPERAND), 16, 1024);
      const uint64_t b2_desc0 = sdesc_sw128(smem_u32(smem + 3 * OPERAND), OPERAND / 2, 1024);
      constexpr uint64_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int u = pair; u < num_units && ok; u += n_pairs) {
        for (int sg = 0; sg < SEGS && ok; ++sg) {
          int lo, hi;
          seg_range(u / num_tiles, sg, lo, hi);
          if (lo == hi) continue;
          if (!mbar_wait_warp(&tempty[acc], acc_phase ^ 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * 256);
          for (int kb = lo; kb < hi; ++kb) {
            if (!mbar_wait_warp(&full[stage], phase)) { ok = false; break; }
            tc_fence_after();
            const uint64_t off = (uint64_t)((stage * STAGE) >> 4);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              umma_bf16_pair(d_tmem, a_desc0 + off + kk * A_STEP, b_desc0 + off + kk * B_STEP, idesc,
                             (kb != lo || kk != 0) ? 1u : 0u);
            if constexpr (KIND == FFN) {
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                umma_bf16_pair(d_tmem + 256, a2_desc0 + off + kk * 2, b2_desc0 + off + kk * 128, idesc_dh,
                               (kb != lo || kk != 0) ? 1u : 0u);
            }
            umma_commit_pair(&empty[stage]);
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
          umma_commit_pair(&tfull[acc]);
          if (++acc == C::ACCS) { acc = 0; acc_phase ^= 1; }
        }
      }
      umma_commit_pair(drain);
      mbar_wait(drain, 0);
    }
  } else if (warp >= 2 + EW) {  // GATED: the tiles of W
    if (lane == 0 && p.gate_grad) {
      int n = 0;
      for (int u = pair; u < num_units; u += n_pairs, ++n) {
        int mt, nt;
        tile_coords(u % num_tiles, p.m_tiles, p.n_tiles, p.group_m, mt, nt);
        if (!mbar_wait(w_empty, (n & 1) ^ 1)) break;
        mbar_arrive_expect_tx(w_full, C::WTILE);
        for (int c = 0; c < 4; ++c)
          tma_load_2d(sW + c * OPERAND, &maps.w, w_full, nt * 256 + c * 64, mt * 256 + (int)rank * 128);
      }
      if (n > 0) mbar_wait(w_full, (n - 1) & 1);
    }
  } else {
    const int q = warp & 3;           // TMEM lane quarter
    const int sub = (warp - 2) >> 2;  // which share of the tile's columns
    const int row_in_tile = q * 32 + lane;
    const uint32_t tempty_leader = mapa_shared(smem_u32(&tempty[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    auto wait_full = [&]() {
      ok = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase));
      tc_fence_after();
      return ok;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + acc * 8);
      if (++acc == C::ACCS) { acc = 0; acc_phase ^= 1; }
    };
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    int n_tile = 0;
    for (int u = pair; u < num_units; u += n_pairs) {
      int mt, nt;
      const int sp = u / num_tiles;
      tile_coords(u - sp * num_tiles, p.m_tiles, p.n_tiles, p.group_m, mt, nt);
      float* part = p.part + (long)sp * p.M * p.N;
      const int m = mt * 256 + (int)rank * 128 + row_in_tile;
      const int n0 = nt * 256 + sub * COLS;
      if constexpr (KIND == GATED) {
        // the warp's 64 output columns of this row stay in registers while the
        // modalities' accumulators come by; W's 64 columns (one swizzled box)
        // are in shared memory
        float sum[COLS];
#pragma unroll
        for (int j = 0; j < COLS; ++j) sum[j] = 0.f;
        const bool in = m < p.M;
        const uint8_t* wrow = sW + sub * OPERAND + row_in_tile * 128;
        if (p.gate_grad) {
          ok = mbar_wait_warp(w_full, n_tile & 1);
          if (!ok) break;
        }
#pragma unroll 1
        for (int sg = 0; sg < 3; ++sg) {
          if (p.seg_rows[sg] == 0) continue;
          float* gp = p.gate_part + ((long)(sg * p.splits + sp) * 4 * p.n_tiles + nt * 4 + sub) * p.M + m;
          int lo, hi;
          seg_range(sp, sg, lo, hi);
          if (lo == hi) {  // none of this modality in this split
            if (p.gate_grad && in) *gp = 0.f;
            continue;
          }
          const float gate = in ? __ldg(p.mod + (long)(sg * 6 + p.gate_slot) * p.D + m) : 0.f;
          if (!wait_full()) break;
          const uint32_t tb = tmem_base + lane_off + (uint32_t)(acc * 256 + sub * COLS);
          float dot = 0.f;
#pragma unroll
          for (int c = 0; c < COLS; c += 16) {
            float v[16];
            ld_chunk16(tb + c, v);
            tmem_wait_ld();
            if (p.gate_grad) {
#pragma unroll
              for (int j = 0; j < 16; j += 8) {
                float wv[8];
                unpack8(*reinterpret_cast<const uint4*>(wrow + ((((c + j) >> 3) ^ (row_in_tile & 7)) << 4)), wv);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(wv[i], v[j + i], dot);
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c + j] = fmaf(gate, v[j], sum[c + j]);
          }
          release();
          if (p.gate_grad && in) *gp = dot;
        }
        if (!ok) break;
        if (p.gate_grad) {
          __syncwarp();
          if (lane == 0) mbar_arrive(w_empty);
        }
        if (p.out != nullptr && p.splits > 1) {
          store_part<COLS>(part, p.N, n0, m, p.M, sum);
        } else if (p.out != nullptr) {
#pragma unroll
          for (int c = 0; c < COLS; c += 16) {
            uint32_t w[8];
            pack_row<16>(sum + c, w);
            if (n0 + c < p.N) store16(p.out + (long)m * p.ldo + n0 + c, p.ldo, m, p.M, w);
          }
        }
      } else {
        int lo, hi;
        seg_range(sp, 0, lo, hi);
        if (lo < hi && !wait_full()) break;
        const uint32_t tb = tmem_base + lane_off + (uint32_t)(acc * 256);
        // the accumulator is handed back before the tile's stores
        if constexpr (KIND == FFN) {
          epi_ffn(p, tb, m, nt, sub, release);
        } else if constexpr (KIND == QKNORM) {
          epi_qknorm(p, tb + sub * COLS, m, n0, freq, axis, wacc + (warp - 2) * 256, release);
        } else if (p.splits > 1) {
          float v[COLS];
          if (lo < hi) {
#pragma unroll
            for (int c = 0; c < COLS; c += 32) ld_chunk(tb + sub * COLS + c, v + c);
            tmem_wait_ld();
            release();
          } else {
#pragma unroll
            for (int c = 0; c < COLS; ++c) v[c] = 0.f;
          }
          store_part<COLS>(part, p.N, n0, m, p.M, v);
        } else {
          uint32_t w[COLS / 2];
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            float v[32];
            ld_chunk(tb + sub * COLS + c, v);
            tmem_wait_ld();
            pack_row<32>(v, w + c / 2);
          }
          release();
#pragma unroll
          for (int c = 0; c < COLS; c += 16)
            if (n0 + c < p.N) store16(p.out + (long)m * p.ldo + n0 + c, p.ldo, m, p.M, w + c / 2);
        }
      }
      ++n_tile;
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (KIND == QKNORM) {
    if (threadIdx.x < 256) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += wacc[w * 256 + threadIdx.x];
      p.w_part[(long)blockIdx.x * 256 + threadIdx.x] = s;
    }
  }
  cluster_sync();  // no MMA of the pair is in flight and no remote arrival pending
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

int max_cta_pairs() {
  const int n = num_sms() / 2;
  return n < 128 ? n : 128;
}

// Splitting the contraction of a product with few output tiles.  In units of
// one k block's MMAs (about 0.3 us): the longest pair's blocks, and for more
// than one split a kernel (4 us) and the partials through memory.  Measured
// at 5,376 x 28,672 over 512 rows (42 tiles for 74 pairs): see the case in the
// launchers below.
constexpr size_t SPLIT_BYTES = 48u << 20;  // of the partials, at most
int plan_splits(int M, int N, int num_kb) {
  const int tiles = (M + 255) / 256 * ((N + 255) / 256), pairs = max_cta_pairs();
  if (tiles >= 2 * pairs) return 1;
  int best = 1;
  double best_t = (double)((tiles + pairs - 1) / pairs) * num_kb;
  for (int s = 2; s <= 32 && s * 2 <= num_kb && (size_t)s * M * N * 4 <= SPLIT_BYTES; ++s) {
    const double t = (double)((tiles * s + pairs - 1) / pairs) * ((num_kb + s - 1) / s) + 14.0 +
                     (double)s * M * N * 8 / 1.8e6;
    if (t < best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}
size_t split_bytes(int M, int N, int num_kb) {
  const int s = plan_splits(M, N, num_kb);
  return s > 1 ? (size_t)s * M * N * 4 : 0;
}

template <int KIND>
cudaError_t launch(const Maps& maps, Params p, cudaStream_t stream) {
  static unsigned long long attr_done = 0;
  const void* fn = reinterpret_cast<const void*>(gemm_bwd_kernel<KIND>);
  cudaError_t e = ensure_smem_attr(fn, Cfg<KIND>::BYTES, &attr_done);
  if (e != cudaSuccess) return e;
  p.m_tiles = (p.M + 255) / 256;
  p.n_tiles = (p.N + (KIND == FFN ? 127 : 255)) / (KIND == FFN ? 128 : 256);
  // bands of eight row tiles: a wave of 74 tiles is then about 8 x 9, whose
  // operands (17 panels) are the fewest a wave can read
  p.group_m = p.m_tiles < 8 ? p.m_tiles : 8;
  if (p.splits < 1) p.splits = 1;
  const int units = p.m_tiles * p.n_tiles * p.splits;
  const int max_pairs = max_cta_pairs();
  const int pairs = units < max_pairs ? units : max_pairs;
  return launch_chained(gemm_bwd_kernel<KIND>, dim3(2 * pairs), Cfg<KIND>::THREADS, Cfg<KIND>::BYTES, stream, maps, p);
}

// the sum of a split product's partials
cudaError_t finish(const Params& p, cudaStream_t stream) {
  static const int none[3] = {0, 0, 0};
  return launch_finish_gated(nullptr, 0, none, 0, 0, nullptr, p.part, p.splits, (long)p.M * p.N, p.out, stream);
}

// K-major operand: rows x cols, 128-row boxes; MN-major: 64-row boxes
bool map_k(CUtensorMap* m, const void* base, long rows, long cols, long ld) {
  return make_tmap_bf16(m, base, rows, cols, ld, 128);
}
bool map_mn(CUtensorMap* m, const void* base, long rows, long cols, long ld) {
  return make_tmap_bf16(m, base, rows, cols, ld, 64);
}

}  // namespace gemm_bwd

// out [out_rows][N] = A [rows][K] B [K][N] for token rows (rows past `rows`: 0)
// (part: split_bytes(out_rows, N, K / 64) of scratch)
cudaError_t launch_dgrad(const bf16* A, const bf16* B, int rows, int out_rows, int N, int K, bf16* out, float* part,
                         cudaStream_t stream) {
  using namespace gemm_bwd;
  Maps maps;
  Params p;
  memset(&maps, 0, sizeof(maps));
  memset(&p, 0, sizeof(p));
  if (!map_k(&maps.a[0], A, rows, K, K) || !map_mn(&maps.b[0], B, K, N, N)) return cudaErrorInvalidValue;
  p.M = out_rows;
  p.N = N;
  p.K = K;
  p.rows = rows;
  p.out = out;
  p.ldo = N;
  p.splits = plan_splits(out_rows, N, K / gemm_bwd::BK);
  p.part = part;
  const cudaError_t e = launch<DGRAD>(maps, p, stream);
  return e != cudaSuccess ? e : finish(p, stream);
}

// out [M][N] = A [rows][M]^T B [rows][N] (part: split_bytes(M, N, L_pad / 64))
cudaError_t launch_wgrad(const bf16* A, const bf16* B, int rows, int L_pad, int M, int N, bf16* out, float* part,
                         cudaStream_t stream) {
  using namespace gemm_bwd;
  Maps maps;
  Params p;
  memset(&maps, 0, sizeof(maps));
  memset(&p, 0, sizeof(p));
  if (!map_mn(&maps.a[0], A, rows, M, M) || !map_mn(&maps.b[0], B, rows, N, N)) return cudaErrorInvalidValue;
  p.M = M;
  p.N = N;
  p.rows = p.seg_rows[0] = rows;
  p.out = out;
  p.ldo = N;
  p.splits = plan_splits(M, N, L_pad / gemm_bwd::BK);
  p.part = part;
  const cudaError_t e = launch<WGRAD>(maps, p, stream);
  return e != cudaSuccess ? e : finish(p, stream);
}

// Partials of the gate's gradient for each modality
int gate_parts(int M, int N, int L_pad) {
  return 4 * ((N + 255) / 256) * gemm_bwd::plan_splits(M, N, L_pad / gemm_bwd::BK);
}


// dW [M][N] = sum_m gate_m (.) A_m^T B_m over the modality ranges (out; null: no
// weight gradient), and the gate's gradient into its slot of dmod (null: none)
// by way of gate_part [3][gate_parts][M]; W: the weight behind the gate
// (part: split_bytes(M, N, L_pad / 64))
cudaError_t launch_wgrad_gated(const bf16* A, const bf16* B, const int* start, const int* count, int L_pad, int M, int N,
                               const float* mod, int gate_slot, const bf16* W, bf16* out, bf16* dmod, float* gate_part,
                               float* part, cudaStream_t stream) {
  using namespace gemm_bwd;
  Maps maps;
  Params p;
  memset(&maps, 0, sizeof(maps));
  memset(&p, 0, sizeof(p));
  for (int m = 0; m < 3; ++m) {
    p.seg_rows[m] = count[m];
    if (count[m] == 0) continue;
    if (!map_mn(&maps.a[m], A + (long)start[m] * M, count[m], M, M) ||
        !map_mn(&maps.b[m], B + (long)start[m] * N, count[m], N, N))
      return cudaErrorInvalidValue;
  }
  p.M = M;
  p.N = N;
  p.out = out;
  p.ldo = N;
  p.mod = mod;
  p.gate_slot = gate_slot;
  p.D = M;
  p.gate_grad = dmod != nullptr;
  if (p.gate_grad && !map_k(&maps.w, W, M, N, N)) return cudaErrorInvalidValue;
  p.gate_part = gate_part;
  p.splits = plan_splits(M, N, L_pad / gemm_bwd::BK);
  p.part = part;
  const cudaError_t e = launch<GATED>(maps, p, stream);
  if (e != cudaSuccess) return e;
  return launch_finish_gated(gate_part, gate_parts(M, N, L_pad), count, M, gate_slot, dmod, part, p.splits, (long)M * N,
                             out, stream);
}

// h [rows][F] and dgu [rows][2F] from xm, dy [rows][D], Wgu [2F][D], Wd [D][F]
cudaError_t launch_ffn_bwd(const bf16* xm, const bf16* dy, const bf16* Wgu, const bf16* Wd, int rows, int D, int F,
                           bf16* h, bf16* dgu, cudaStream_t stream) {
  using namespace gemm_bwd;
  Maps maps;
  Params p;
  memset(&maps, 0, sizeof(maps));
  memset(&p, 0, sizeof(p));
  if (!map_k(&maps.a[0], xm, rows, D, D) || !map_k(&maps.a[1], dy, rows, D, D) || !map_k(&maps.b[0], Wgu, 2 * F, D, D) ||
      !map_mn(&maps.b[1], Wd, D, F, F))
    return cudaErrorInvalidValue;
  p.M = rows;
  p.N = F;
  p.K = D;
  p.rows = rows;
  p.F = F;
  p.h = h;
  p.dgu = dgu;
  return launch<FFN>(maps, p, stream);
}

constexpr int QKNORM_PARTS = 256;  // CTAs of the QKNORM kernel, at most

// dqkv[:, 0 : 2I] (row stride 3I) and the norm weights' partials w_part
// [*n_parts][2][128], from xm [rows][D] and the q, k rows of Wqkv
cudaError_t launch_qknorm_bwd(const bf16* xm, const bf16* Wqkv, const bf16* dq, const bf16* dk, const bf16* qn_w,
                              const bf16* kn_w, const float* pos, int rows, int L_pad, int D, int I, const int* rope,
                              float theta, float eps, bf16* dqkv, float* w_part, int* n_parts, cudaStream_t stream) {
  using namespace gemm_bwd;
  Maps maps;
  Params p;
  memset(&maps, 0, sizeof(maps));
  memset(&p, 0, sizeof(p));
  if (!map_k(&maps.a[0], xm, rows, D, D) || !map_k(&maps.b[0], Wqkv, 2 * I, D, D)) return cudaErrorInvalidValue;
  p.M = rows;
  p.N = 2 * I;
  p.K = D;
  p.rows = rows;
  p.out = dqkv;
  p.ldo = 3L * I;
  p.dq = dq;
  p.dk = dk;
  p.qn_w = qn_w;
  p.kn_w = kn_w;
  p.pos = pos;
  p.L_pad = L_pad;
  p.I = I;
  p.rope_t = rope[0];
  p.rope_h = rope[1];
  p.rope_w = rope[2];
  p.theta = theta;
  p.eps_qk = eps;
  p.w_part = w_part;
  const int tiles = (rows + 255) / 256 * ((2 * I + 255) / 256);
  const int max_pairs = max_cta_pairs();
  *n_parts = 2 * (tiles < max_pairs ? tiles : max_pairs);
  return launch<QKNORM>(maps, p, stream);
}

}  // namespace h3
