// tcgen05 GEMMs of the block's backward pass, all on CTA pairs (cta_group::2,
// 256 x 256 output tiles over two SMs, fp32 accumulators in TMEM):
//
//   PRODUCTS  up to three independent products; short ones in one persistent
//           launch, the tiles of one after those of another (one tail instead
//           of three, and small ones side by side):
//     input gradient   out[t][n] = sum_k A[t][k] B[k][n].  B is the forward
//           weight [out, in] read with its rows as the contraction, so no
//           transposed copy of a weight exists: its tiles enter shared memory
//           as they lie (64 columns x 64 rows per TMA box) and the MMA takes
//           them MN-major.
//     weight gradient  out[j][n] = sum_t A[t][j] B[t][n]: both operands
//           MN-major, the contraction over the tokens.
//     gated weight gradient, for a linear behind a modality gate
//           (y = gate_m (.) (B W^T)): one accumulator per modality range, G_m =
//           sum_{t in m} A^T B, then
//             dW[j][n]    = sum_m gate_m[j] G_m[j][n]
//             dgate_m[j]  = sum_n W[j][n] G_m[j][n]
//           (the second is sum_t dx[t][j] (B W^T)[t][j] with the order of the
//           sums exchanged), so the gate's gradient needs neither the branch
//           output nor another product, and a gate of 0 loses nothing.
//   QKNORM    x = A W_qk^T (the q, k projection again), and in the epilogue the
//           backward pass of RoPE and of the per-head RMSNorm.
//   FFN       gate, up = A Wgu^T and dh = dY Wd in one K loop, and in the
//           epilogue h = SiLU(g) u and the gradients of g and u.
//
// Tensor cores bound all three where contractions are long.  Tensor pipe active
// while an SM has tiles, at 2,048 tokens of width 5,376 (56 heads, F 14,336):
// QKNORM 86% (235 us), FFN 89% (676 us), input and weight gradients 95-97%.  A
// gated weight gradient over short modality ranges has an epilogue for each
// range (59% there, 29 k blocks the longest), and over 512 tokens (8 k blocks a
// tile) its stores and the tiles of W bound it.  Long calls run against the power limit: 1,250-1,300 TFLOP/s
// sustained.
//
// A segment, a ragged length and the padding rows end inside a tile: the tensor
// maps stop at the last valid token, and TMA reads zeros past it.
#include "h3_internal.cuh"
#include "ptx.cuh"

namespace h3 {

namespace gemm_bwd {
using gemm_detail::tile_coords;

enum Kind : int { PRODUCTS = 0, QKNORM = 1, FFN = 2 };

constexpr int MAX_PRODUCTS = 3;
struct Maps {
  // QKNORM: A, B; FFN: xm, Wgu, dY, Wd; PRODUCTS: of each product A and B of
  // every segment, then W if gated (input and weight gradients 2 each, gated 7)
  CUtensorMap m[11];
};

struct Product {
  int map0;           // its first tensor map
  int a_mn;           // A MN-major (weight gradients) or K-major
  int gated, segs;    // gated: three segments, else one
  int M, N;           // output rows and columns
  int m_tiles, n_tiles, group_m;
  int kb[3];          // k blocks of each segment
  // The contraction in `splits` equal runs of k blocks, each a unit of work of
  // its own that writes an fp32 partial, part [splits][M][N]; 1: none
  int splits, units;
  int per;            // k blocks of a split
  float* part;
  bf16* out;          // [M][N]; null (gated only): not wanted
};

struct Params {
  int n_products, units, n_maps;
  int catch_up;       // units after the first product's for the pairs that its last turn leaves out
  Product pr[MAX_PRODUCTS];
  // the gated product
  const float* mod;   // [3][6][D], D = its M
  int gate_slot;
  int gate_grad;      // whether the gate's gradient is wanted
  float* gate_part;   // [3][splits * 4 n_tiles][M] column-quarter partials of it
  int rows;           // QKNORM, FFN: valid token rows
  // FFN
  bf16* h;            // [.][F]
  bf16* dgu;          // [.][2F]
  int F;
  // QKNORM
  bf16* dqkv;         // [.][3I]
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
  static constexpr int STAGES = KIND == FFN ? 4 : (KIND == QKNORM ? 6 : 5);
  // FFN: xm, dY (16 KB each), gate or up rows of Wgu (16 KB), 64 columns of Wd (8 KB)
  static constexpr int STAGE = KIND == FFN ? 3 * OPERAND + OPERAND / 2 : 2 * OPERAND;
  static constexpr int ACCS = KIND == FFN ? 1 : 2;  // TMEM accumulators: 256 + 128 columns, or 2 x 256
  // Warp 0 TMA, warp 1 MMA, then EW epilogue warps: EW / 4 of each TMEM lane
  // quarter, sharing the tile's columns.  Sixteen hide the latency of the
  // TMEM and global accesses of one tile.
  static constexpr int EW = 16;
  // PRODUCTS: one more warp loads the tile of W that a gate's gradient needs.
  // (Five stages beside its 64 KB: 2-4% faster than four for the gated product,
  // 1% slower than six for a long input gradient.)
  static constexpr int THREADS = (2 + EW + (KIND == PRODUCTS ? 1 : 0)) * 32;
  static constexpr int WTILE = KIND == PRODUCTS ? 4 * OPERAND : 0;  // 128 rows x 256 columns
  static constexpr int MISC = 768;
  // QKNORM: [epilogue warp][q, k][32] sums, and two floats of each row, head and
  // warp for the exchange between a row's four warps, for two tiles in turn (a
  // warp that writes one has passed the other's barrier, so all have read it)
  static constexpr int NORM = KIND == QKNORM ? EW * 64 * 4 + 2 * EW * 2 * 32 * 8 : 0;
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
// 32 lanes x 8 consecutive 32-bit columns
__device__ __forceinline__ void ld_chunk8(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// (L1::no_allocate: what is left of L1 beside the stages serves the loads; 9%
// of a weight gradient over 64 tokens, which is bound by its stores)
__device__ __forceinline__ void st_v4(uint32_t* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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
template <int N>
__device__ __forceinline__ void pack_row(const float* v, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N; i += 2) w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
}
// The warp's columns [n0, n0 + COLS) of the output as bf16, or of one split's
// partial as fp32
template <int COLS>
__device__ __forceinline__ void store_tile(const Product& pr, int sp, int n0, int m, const float* v) {
  const int M = pr.M, N = pr.N;
  if (pr.splits > 1) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(pr.part + ((long)sp * M + m) * N + n0);
#pragma unroll
    for (int c = 0; c < COLS; c += 8)
      if (n0 + c < N) store8w(dst + c, N, m, M, reinterpret_cast<const uint32_t*>(v + c));
  } else {
    bf16* dst = pr.out + (long)m * N + n0;
#pragma unroll
    for (int c = 0; c < COLS; c += 16) {
      uint32_t w[8];
      pack_row<16>(v + c, w);
      if (n0 + c < N) store16(dst + c, N, m, M, w);
    }
  }
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

__device__ __forceinline__ void unpack16(const bf16* w, float* f) {
  unpack8(__ldg(reinterpret_cast<const uint4*>(w)), f);
  unpack8(__ldg(reinterpret_cast<const uint4*>(w + 8)), f + 8);
}

// RoPE and RMSNorm backward of the tile's two heads at one token.  With d the
// gradient of the rotated head, t = d turned back by the token's angles
// ((a, b) = (d0 cos + d1 sin, d1 cos - d0 sin), the transpose of the forward
// rotation), x the head before its norm (TMEM), xhat = x inv, dh = t (.) w:
//   dx = inv (dh - xhat mean(dh xhat));  with s = sum dh x, mean = s inv / 128
// and the gradient of w is sum_t t xhat.
// Four warps share a token's heads, 32 columns of both each, so that an angle's
// sine and cosine serve both heads; two passes, with the sums of x^2 and dh x
// exchanged between the four after the first (xch[4 warps][2 heads][32 lanes]
// of this tile; `bar` at phase `parity`).  wacc[q, k][32] of this warp takes the
// sums over its rows.  Loops that are not unrolled: unrolled, the code was some
// 80 KB and the first tile of a small call spent most of its time fetching it.
// False: a wait gave up.
template <typename Wait, typename Release>
__device__ __forceinline__ bool epi_qknorm(const Params& p, uint32_t tb, int m, int n0, int I, int sub,
                                           const float* freq, const uint8_t* axis, float* wacc, float2* xch,
                                           uint64_t* bar, uint32_t parity, Wait wait, Release release) {
  const int lane = threadIdx.x & 31;
  const bool valid = m < p.rows;
  const bf16 *d[2], *w[2];
  int part[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + h * 128, hd = (n % I) / 128;
    part[h] = n / I;
    d[h] = (part[h] == 0 ? p.dq : p.dk) + ((long)hd * p.L_pad + (valid ? m : 0)) * 128 + sub * 32;
    // into L2 while the accumulator is awaited
    asm volatile("prefetch.global.L2 [%0];" ::"l"(d[h]));
    w[h] = (part[h] == 0 ? p.qn_w : p.kn_w) + sub * 32;
  }
  tb += sub * 32;
  float p3[3] = {0.f, 0.f, 0.f};
  if (valid) {
    p3[0] = p.pos[(long)m * 3];
    p3[1] = p.pos[(long)m * 3 + 1];
    p3[2] = p.pos[(long)m * 3 + 2];
  }
  // sine and cosine of the 8 pairs of columns [16 c, 16 c + 16) of the warp's 32
  auto angles = [&](int c, float* cs, float* sn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ip = sub * 16 + c * 8 + i, ax = axis[ip];
      const float pa = ax == 0 ? p3[0] : (ax == 1 ? p3[1] : p3[2]);
      gemm_detail::rope_sincos(pa * freq[ip], &sn[i], &cs[i]);
    }
  };
  auto turn_back = [&](const bf16* src, const float* cs, const float* sn, float* t) {
    uint4 u = make_uint4(0, 0, 0, 0), v = u;
    if (valid) {
      u = __ldg(reinterpret_cast<const uint4*>(src));
      v = __ldg(reinterpret_cast<const uint4*>(src + 8));
    }
    unpack8(u, t);
    unpack8(v, t + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = t[2 * i], b = t[2 * i + 1];
      t[2 * i] = a * cs[i] + b * sn[i];
      t[2 * i + 1] = b * cs[i] - a * sn[i];
    }
  };
  if (!wait()) return false;
  float ss[2] = {0.f, 0.f}, s[2] = {0.f, 0.f};
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float cs[8], sn[8];
    angles(c, cs, sn);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[16], t[16], wv[16];
      ld_chunk16(tb + h * 128 + c * 16, x);
      turn_back(d[h] + c * 16, cs, sn, t);
      unpack16(w[h] + c * 16, wv);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        ss[h] = fmaf(x[j], x[j], ss[h]);
        s[h] = fmaf(t[j] * wv[j], x[j], s[h]);
      }
    }
  }
  xch[(sub * 2) * 32 + lane] = make_float2(ss[0], s[0]);
  xch[(sub * 2 + 1) * 32 + lane] = make_float2(ss[1], s[1]);
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  if (!mbar_wait_warp(bar, parity)) return false;
  float inv[2], mean[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // added in the same order by all four
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = xch[(k * 2 + h) * 32 + lane];
      a += v.x;
      b += v.y;
    }
    inv[h] = rsqrtf(a * (1.0f / 128.0f) + p.eps_qk);
    mean[h] = b * inv[h] * (1.0f / 128.0f);
  }
  bf16* dst = p.dqkv + (long)m * 3 * p.I + n0 + sub * 32;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float cs[8], sn[8];
    angles(c, cs, sn);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[16], t[16], wv[16];
      ld_chunk16(tb + h * 128 + c * 16, x);
      turn_back(d[h] + c * 16, cs, sn, t);
      unpack16(w[h] + c * 16, wv);
      tmem_wait_ld();
      if (c == 1 && h == 1) release();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float xh = x[j] * inv[h];
        x[j] = inv[h] * (t[j] * wv[j] - xh * mean[h]);
        t[j] *= xh;
      }
      uint32_t out[8];
      pack_row<16>(x, out);
      store16(dst + h * 128 + c * 16, 3L * p.I, m, p.rows, out);
      // sum over the warp's 32 rows: lanes 2l and 2l + 1 end with column l
#pragma unroll
      for (int o = 16; o > 1; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o / 2; ++i) {
          const float send = up ? t[i] : t[i + o / 2], keep = up ? t[i + o / 2] : t[i];
          t[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      t[0] += __shfl_xor_sync(0xffffffffu, t[0], 1);
      if ((lane & 1) == 0) wacc[part[h] * 32 + c * 16 + (lane >> 1)] += t[0];
    }
  }
  return true;
}

// h = SiLU(g) u, du = dh SiLU(g), dg = dh u sig(g) (1 + g (1 - sig(g))) for 32 of
// the tile's 128 hidden columns; accumulator columns [0, 128) g, [128, 256) u,
// [256, 384) dh.  h, dg and du are rounded to bf16 (half a step, 2^-8 at most),
// as operands of the products that follow; with the gradient's own operand and
// the result that makes 2.9e-3 of a result's 2-norm, 1.7e-3 of it the result's
// rounding.  A second bf16 for what each loses would cost a quarter more time.
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

// A unit of work: split sp of tile (mt, nt) of product pr
struct Unit {
  int product, sp, mt, nt;
};
template <int KIND>
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  Unit w;
  w.product = 0;
  if constexpr (KIND == PRODUCTS)
    while (u >= p.pr[w.product].units) u -= p.pr[w.product++].units;
  const Product& pr = p.pr[w.product];
  const int tiles = pr.m_tiles * pr.n_tiles;
  w.sp = u / tiles;
  tile_coords(u - w.sp * tiles, pr.m_tiles, pr.n_tiles, pr.group_m, w.mt, w.nt);
  return w;
}
// The pair's unit after u (its first: after pair - n_pairs): the first
// product's in turns of all pairs, then the catch_up units in turns of the
// pairs without one in its last, partial turn, then the rest in turns of all,
// those pairs first.
template <int KIND>
__device__ __forceinline__ int next_unit(const Params& p, int u, int pair, int n_pairs) {
  if constexpr (KIND != PRODUCTS) return u + n_pairs;
  const int n0 = p.pr[0].units, end = n0 + p.catch_up, rem = n0 % n_pairs;
  if (u < n0) {
    u += n_pairs;
    if (u < n0) return u;
    u = pair < rem ? end : n0 + pair - rem;
  } else if (u < end) {
    u += n_pairs - rem;
  } else {
    return u + n_pairs;
  }
  return u < end ? u : end + n_pairs - 1 - pair;
}
// k blocks [lo, hi) of segment sg in split sp, the segments' blocks counted one
// after another
__device__ __forceinline__ void seg_range(const Product& pr, int sp, int sg, int& lo, int& hi) {
  const int before = sg == 0 ? 0 : (sg == 1 ? pr.kb[0] : pr.kb[0] + pr.kb[1]);
  const int per = pr.per, n = pr.kb[sg];
  lo = min(n, max(0, sp * per - before));
  hi = max(lo, min(n, (sp + 1) * per - before));
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<KIND>::THREADS, 1)
    gemm_bwd_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = Cfg<KIND>;
  constexpr int STAGES = C::STAGES, STAGE = C::STAGE, EW = C::EW;
  constexpr int COLS = 1024 / EW;  // output columns of an epilogue warp (FFN: 32)
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sW = smem + STAGES * STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE + C::WTILE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* w_full = drain + 1;   // PRODUCTS: W of the tile
  uint64_t* w_empty = drain + 2;  // PRODUCTS: read by every epilogue warp of this CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 3);
  float* freq = reinterpret_cast<float*>(tmem_slot + 4);
  uint8_t* axis = reinterpret_cast<uint8_t*>(freq + 64);
  uint64_t* xbar = reinterpret_cast<uint64_t*>(axis + 64);  // QKNORM: [4] the four warps of a lane quarter
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
      mbar_init(&tfull[a], 1);         // the leader's commit, delivered to both CTAs
      mbar_init(&tempty[a], 2 * EW);   // the epilogue warps of both CTAs (leader's copy used)
    }
    mbar_init(drain, 1);
    mbar_init(w_full, 1);
    mbar_init(w_empty, EW);
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], 4);
    fence_mbar_init();
    for (int i = 0; i < p.n_maps; ++i) tma_prefetch_desc(&maps.m[i]);
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
    for (int i = threadIdx.x; i < EW * 64; i += C::THREADS) wacc[i] = 0.f;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  chain_wait();

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t leader_full0 = mapa_shared(smem_u32(&full[0]), 0);
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = next_unit<KIND>(p, pair - n_pairs, pair, n_pairs); u < p.units && ok;
           u = next_unit<KIND>(p, u, pair, n_pairs)) {
        // One thread feeds the tile: everything its loop needs is in registers
        // before it (a parameter indexed by the product costs the whole kernel
        // 7% when it is read again for every load).
        const Unit w = unit_of<KIND>(p, u);
        const Product& pr = p.pr[w.product];  // 0 but for PRODUCTS
        const int a0 = w.mt * 256 + (int)rank * 128;  // this CTA's A rows (or MN-major columns)
        const int b0 = w.nt * (KIND == FFN ? 128 : 256) + (int)rank * (KIND == FFN ? p.F : 128);
        const int d0 = w.nt * 128 + (int)rank * 64;
        const int segs = pr.segs, map0 = pr.map0;
        const bool a_mn = KIND == PRODUCTS && pr.a_mn;
        for (int sg = 0; sg < segs && ok; ++sg) {
          const CUtensorMap* ma = &maps.m[map0 + sg];
          const CUtensorMap* mb = &maps.m[map0 + segs + sg];
          int lo, hi;
          seg_range(pr, w.sp, sg, lo, hi);
          auto feed = [&](auto a_tag) {
            constexpr bool A_MN = decltype(a_tag)::value;
            for (int kb = lo; kb < hi; ++kb) {
              if (!mbar_wait(&empty[stage], phase ^ 1)) { ok = false; break; }
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * STAGE);
              const uint32_t fb = leader_full0 + stage * 8;
              uint8_t* sA = smem + stage * STAGE;
              uint8_t* sB = sA + OPERAND;
              if constexpr (A_MN) {
                tma_load_3d_pair(sA, ma, fb, 0, kb * BK, a0 / 64);
              } else {
                tma_load_2d_pair(sA, ma, fb, kb * BK, a0);
              }
              if constexpr (KIND == PRODUCTS) {
                tma_load_3d_pair(sB, mb, fb, 0, kb * BK, b0 / 64);
              } else {
                tma_load_2d_pair(sB, mb, fb, kb * BK, b0);
              }
              if constexpr (KIND == FFN) {
                tma_load_2d_pair(sA + 2 * OPERAND, &maps.m[2], fb, kb * BK, a0);
                tma_load_3d_pair(sA + 3 * OPERAND, &maps.m[3], fb, 0, kb * BK, d0 / 64);
              }
              ++issued;
              if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
          };
          if (a_mn)
            feed(std::true_type{});
          else
            feed(std::false_type{});
        }
      }
      // the leader's full barriers count both CTAs' bytes: the leader waits
      // for both, the peer CTA is held by the cluster barrier below
      if (leader) drain_loads(full, STAGES, issued);
    }
  } else if (warp == 1) {
    if (leader) {
      // MN-major operands: 64-column blocks 8 KB apart, 8-row groups 1 KB
      // apart, 16 rows (2 KB) per MMA; K-major: 32 bytes per MMA
      constexpr bool B_MN = KIND == PRODUCTS;
      const uint64_t b_desc0 = sdesc_sw128(smem_u32(smem + OPERAND), B_MN ? OPERAND / 2 : 16, 1024);
      const uint64_t a2_desc0 = sdesc_sw128(smem_u32(smem + 2 * OPERAND), 16, 1024);
      const uint64_t b2_desc0 = sdesc_sw128(smem_u32(smem + 3 * OPERAND), OPERAND / 2, 1024);
      constexpr uint32_t idesc_dh = idesc_bf16_f32(256, 128, true);
      constexpr uint64_t B_STEP = B_MN ? 128 : 2;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int u = next_unit<KIND>(p, pair - n_pairs, pair, n_pairs); u < p.units && ok;
           u = next_unit<KIND>(p, u, pair, n_pairs)) {
        const Unit w = unit_of<KIND>(p, u);
        const Product& pr = p.pr[w.product];
        // the MMAs' descriptors are constants but for the start address: one
        // loop for each majorness of A
        auto contract = [&](auto a_tag, int sg) {
          constexpr bool A_MN = decltype(a_tag)::value;
          constexpr uint32_t idesc = idesc_bf16_f32(256, 256, B_MN) | (A_MN ? 1u << 15 : 0u);
          constexpr uint64_t A_STEP = A_MN ? 128 : 2;
          const uint64_t a_desc0 = sdesc_sw128(smem_u32(smem), A_MN ? OPERAND / 2 : 16, 1024);
          int lo, hi;
          seg_range(pr, w.sp, sg, lo, hi);
          if (lo == hi) return true;
          if (!mbar_wait_warp(&tempty[acc], acc_phase ^ 1)) return false;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * 256);
          for (int kb = lo; kb < hi; ++kb) {
            if (!mbar_wait_warp(&full[stage], phase)) return false;
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
          return true;
        };
        for (int sg = 0; sg < pr.segs && ok; ++sg) {
          if (KIND == PRODUCTS && pr.a_mn)
            ok = contract(std::true_type{}, sg);
          else
            ok = contract(std::false_type{}, sg);
        }
      }
      umma_commit_pair(drain);
      mbar_wait(drain, 0);
    }
  } else if (warp >= 2 + EW) {  // PRODUCTS: the gated product's tiles of W
    if (lane == 0 && p.gate_grad) {
      int n = 0;
      for (int u = next_unit<KIND>(p, pair - n_pairs, pair, n_pairs); u < p.units;
         u = next_unit<KIND>(p, u, pair, n_pairs)) {
        const Unit w = unit_of<KIND>(p, u);
        const Product& pr = p.pr[w.product];
        if (!pr.gated) continue;
        if (!mbar_wait(w_empty, (n & 1) ^ 1)) break;
        mbar_arrive_expect_tx(w_full, C::WTILE);
        tma_load_3d(sW, &maps.m[pr.map0 + 6], w_full, 0, w.mt * 256 + (int)rank * 128, w.nt * 4);
        ++n;
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
    int n_w = 0;
    for (int u = next_unit<KIND>(p, pair - n_pairs, pair, n_pairs); u < p.units;
         u = next_unit<KIND>(p, u, pair, n_pairs)) {
      const Unit w = unit_of<KIND>(p, u);
      const Product& pr = p.pr[w.product];
      const int m = w.mt * 256 + (int)rank * 128 + row_in_tile;
      const int n0 = w.nt * 256 + sub * COLS;
      if constexpr (KIND == FFN) {
        if (!wait_full()) break;
        epi_ffn(p, tmem_base + lane_off + (uint32_t)(acc * 256), m, w.nt, sub, release);
      } else if constexpr (KIND == QKNORM) {
        float2* xch = reinterpret_cast<float2*>(wacc + EW * 64) + ((n_w & 1) * 4 + q) * 4 * 2 * 32;
        ok = epi_qknorm(p, tmem_base + lane_off + (uint32_t)(acc * 256), m, w.nt * 256, pr.N / 2, sub, freq, axis,
                        wacc + (warp - 2) * 64, xch, &xbar[q], n_w & 1, wait_full, release);
        if (!ok) break;
        ++n_w;
      } else if (pr.gated) {
        // the warp's 64 output columns of this row stay in registers while the
        // modalities' accumulators come by; W's 64 columns (one swizzled box)
        // are in shared memory
        float sum[COLS];
#pragma unroll
        for (int j = 0; j < COLS; ++j) sum[j] = 0.f;
        const bool in = m < pr.M;
        const uint8_t* wrow = sW + sub * OPERAND + row_in_tile * 128;
        if (p.gate_grad) {
          ok = mbar_wait_warp(w_full, n_w & 1);
          if (!ok) break;
        }
#pragma unroll 1
        for (int sg = 0; sg < 3; ++sg) {
          if (pr.kb[sg] == 0) continue;
          float* gp = p.gate_part + ((long)(sg * pr.splits + w.sp) * 4 * pr.n_tiles + w.nt * 4 + sub) * pr.M + m;
          int lo, hi;
          seg_range(pr, w.sp, sg, lo, hi);
          if (lo == hi) {  // none of this modality in this split
            if (p.gate_grad && in) *gp = 0.f;
            continue;
          }
          const float gate = in ? __ldg(p.mod + (long)(sg * 6 + p.gate_slot) * pr.M + m) : 0.f;
          if (!wait_full()) break;
          const uint32_t tb = tmem_base + lane_off + (uint32_t)(acc * 256 + sub * COLS);
          // eight columns at a time, with a few words of spills (36 bytes stored, 28
          // loaded); with 16 more of the sums spill (out-projection at 512 tokens
          // 87.6 us, so 85.7; at 2,048 tokens 262 and 258)
          float dot = 0.f;
#pragma unroll
          for (int c = 0; c < COLS; c += 8) {
            float v[8];
            ld_chunk8(tb + c, v);
            tmem_wait_ld();
            if (p.gate_grad) {
              float wv[8];
              unpack8(*reinterpret_cast<const uint4*>(wrow + (((c >> 3) ^ (row_in_tile & 7)) << 4)), wv);
#pragma unroll
              for (int i = 0; i < 8; ++i) dot = fmaf(wv[i], v[i], dot);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[c + j] = fmaf(gate, v[j], sum[c + j]);
          }
          release();
          if (p.gate_grad && in) *gp = dot;
        }
        if (!ok) break;
        if (p.gate_grad) {
          ++n_w;
          __syncwarp();
          if (lane == 0) mbar_arrive(w_empty);
        }
        if (pr.out != nullptr) store_tile<COLS>(pr, w.sp, n0, m, sum);
      } else {
        int lo, hi;
        seg_range(pr, w.sp, 0, lo, hi);
        float v[COLS];
        if (lo < hi) {
          if (!wait_full()) break;
          const uint32_t tb = tmem_base + lane_off + (uint32_t)(acc * 256 + sub * COLS);
#pragma unroll
          for (int c = 0; c < COLS; c += 32) ld_chunk(tb + c, v + c);
          tmem_wait_ld();
          release();  // before the stores
        } else {
#pragma unroll
          for (int c = 0; c < COLS; ++c) v[c] = 0.f;
        }
        store_tile<COLS>(pr, w.sp, n0, m, v);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (KIND == QKNORM) {
    if (threadIdx.x < 256) {  // column c of q or k: the warps that hold it, one a lane quarter
      const int part = threadIdx.x >> 7, c = threadIdx.x & 127;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) s += wacc[((c >> 5) * 4 + k) * 64 + part * 32 + (c & 31)];
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
// than one split a kernel (4 us) and the partials through memory.  Measured:
// 512 rows of 28,672 x 5,376 (42 tiles for 74 pairs) 212 -> 148 us in three
// splits; 320 x 1,792 over 32,160 rows (14 tiles) 224 -> 59 us in five.
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
  return s > 1 ? ((size_t)s * M * N * 4 + 255) / 256 * 256 : 0;
}

// K-major operand: rows x cols in 128-row boxes
bool map_k(CUtensorMap* m, const void* base, long rows, long cols, long ld) {
  return make_tmap_bf16(m, base, rows, cols, ld, 128);
}
// MN-major operand: its columns (a multiple of 64) as blocks of 64, the
// outermost dimension, so that one load of `blocks` of them fills an operand,
// each block's rows together as the swizzled layout wants them (3% fewer SM
// cycles over the backward calls than a load for each block).
bool map_mn(CUtensorMap* m, const void* base, long rows, long cols, int box_rows, int blocks) {
  gemm_detail::EncodeTiledFn fn = gemm_detail::encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64};
  cuuint64_t gstride[2] = {(cuuint64_t)cols * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void set_tiles(Product& pr, int M, int N, int n_step) {
  pr.M = M;
  pr.N = N;
  pr.m_tiles = (M + 255) / 256;
  pr.n_tiles = (N + n_step - 1) / n_step;
  // bands of eight row tiles: a wave of 74 tiles is then about 8 x 9, whose
  // operands (17 panels) are the fewest a wave can read (measured at 32,160
  // tokens: four or twelve rows 3-8% slower)
  pr.group_m = pr.m_tiles < 8 ? pr.m_tiles : 8;
}

// What the pairs that the first product's last turn leaves out do meanwhile, in
// units of the products after it.  A unit takes its k blocks' time, or where
// they are few its epilogue's (24 k blocks with a gate, 12 without).  Measured
// with and without: out-projection at full width, 512 tokens (56 units of 84 k
// blocks, then 588 of 8) 87.8 and 90.8 us, 352 tokens 105.8 and 111.9, 2,048
// tokens 263 and 269.  (Costs of 16 and 40 for 24: 87.8 and 91.6, 113.7 and 112.8.)
int catch_up_units(const Params& p, int pairs) {
  auto cost = [&](const Product& pr) {
    const int kb = (pr.kb[0] + pr.kb[1] + pr.kb[2] + pr.splits - 1) / pr.splits, least = pr.gated ? 24 : 12;
    return kb > least ? kb : least;
  };
  const int rem = p.pr[0].units % pairs, light = pairs - rem;
  if (p.n_products < 2 || rem == 0) return 0;
  int spare = cost(p.pr[0]), rounds = 0, rest = 0;
  for (int i = 1; i < p.n_products; ++i) rest += p.pr[i].units;
  for (int i = 1; i < p.n_products; ++i) {
    const int c = cost(p.pr[i]), all = (p.pr[i].units + light - 1) / light;
    const int n = all < spare / c ? all : spare / c;
    rounds += n;
    spare -= n * c;
    if (n < all) break;
  }
  return rounds * light < rest ? rounds * light : rest;
}

template <int KIND>
cudaError_t launch(const Maps& maps, Params& p, cudaStream_t stream) {
  static unsigned long long attr_done = 0;
  const void* fn = reinterpret_cast<const void*>(gemm_bwd_kernel<KIND>);
  cudaError_t e = ensure_smem_attr(fn, Cfg<KIND>::BYTES, &attr_done);
  if (e != cudaSuccess) return e;
  p.units = 0;
  for (int i = 0; i < p.n_products; ++i) {
    Product& pr = p.pr[i];
    pr.units = pr.m_tiles * pr.n_tiles * pr.splits;
    pr.per = (pr.kb[0] + pr.kb[1] + pr.kb[2] + pr.splits - 1) / pr.splits;
    p.units += pr.units;
  }
  const int max_pairs = max_cta_pairs();
  const int pairs = p.units < max_pairs ? p.units : max_pairs;
  p.catch_up = catch_up_units(p, pairs);
  return launch_chained(gemm_bwd_kernel<KIND>, dim3(2 * pairs), Cfg<KIND>::THREADS, Cfg<KIND>::BYTES, stream, maps, p);
}

}  // namespace gemm_bwd

// Partials of the gate's gradient for each modality
int gate_parts(int M, int N, int L_pad) {
  return 4 * ((N + 255) / 256) * gemm_bwd::plan_splits(M, N, L_pad / gemm_bwd::BK);
}

// The products that end a backward call: added one by one, then launched
// together.  Partials of split products take their parts of `split` one after
// another (split_bytes each, 256-byte aligned).
struct Products {
  gemm_bwd::Maps maps;
  gemm_bwd::Params p;
  FinishArgs fin;
  uint8_t* split;
  int n_maps = 0;
  bool good = true;

  explicit Products(float* split_ws) : split(reinterpret_cast<uint8_t*>(split_ws)) {
    memset(&maps, 0, sizeof(maps));
    memset(&p, 0, sizeof(p));
    memset(&fin, 0, sizeof(fin));
  }
  gemm_bwd::Product& add(int M, int N, int segs, int splits, bf16* out) {
    gemm_bwd::Product& pr = p.pr[p.n_products++];
    pr.map0 = n_maps;
    pr.segs = segs;
    gemm_bwd::set_tiles(pr, M, N, 256);
    pr.splits = splits;
    pr.out = out;
    if (splits > 1) {
      pr.part = reinterpret_cast<float*>(split);
      split += ((size_t)splits * M * N * 4 + 255) / 256 * 256;
      if (out != nullptr) fin.sum[fin.n_sums++] = {pr.part, out, (long)M * N, splits};
    }
    return pr;
  }
  // out [out_rows][N] = A [rows][K] B [K][N] (token rows past `rows`: 0)
  void input_gradient(const bf16* A, const bf16* B, int rows, int out_rows, int N, int K, bf16* out) {
    using namespace gemm_bwd;
    Product& pr = add(out_rows, N, 1, plan_splits(out_rows, N, K / gemm_bwd::BK), out);
    pr.kb[0] = K / gemm_bwd::BK;
    good = good && map_k(&maps.m[n_maps], A, rows, K, K) && map_mn(&maps.m[n_maps + 1], B, K, N, gemm_bwd::BK, 2);
    n_maps += 2;
  }
  // out [M][N] = A [rows][M]^T B [rows][N]
  void weight_gradient(const bf16* A, const bf16* B, int rows, int L_pad, int M, int N, bf16* out) {
    using namespace gemm_bwd;
    Product& pr = add(M, N, 1, plan_splits(M, N, L_pad / gemm_bwd::BK), out);
    pr.a_mn = 1;
    pr.kb[0] = (rows + gemm_bwd::BK - 1) / gemm_bwd::BK;
    good = good && map_mn(&maps.m[n_maps], A, rows, M, gemm_bwd::BK, 2) &&
           map_mn(&maps.m[n_maps + 1], B, rows, N, gemm_bwd::BK, 2);
    n_maps += 2;
  }
  // dW [M][N] = sum_m gate_m (.) A_m^T B_m over the modality ranges (null: not
  // wanted), and the gate's gradient into its slot of dmod (null: not wanted)
  // by way of gate_part [3][gate_parts][M]; W: the weight behind the gate
  void gated_weight_gradient(const bf16* A, const bf16* B, const int* start, const int* count, int L_pad, int M, int N,
                             const float* mod, int slot, const bf16* W, bf16* dW, bf16* dmod, float* gate_part) {
    using namespace gemm_bwd;
    Product& pr = add(M, N, 3, plan_splits(M, N, L_pad / gemm_bwd::BK), dW);
    pr.a_mn = pr.gated = 1;
    for (int m = 0; m < 3; ++m) {
      pr.kb[m] = (count[m] + gemm_bwd::BK - 1) / gemm_bwd::BK;
      if (count[m] == 0) continue;
      good = good && map_mn(&maps.m[n_maps + m], A + (long)start[m] * M, count[m], M, gemm_bwd::BK, 2) &&
             map_mn(&maps.m[n_maps + 3 + m], B + (long)start[m] * N, count[m], N, gemm_bwd::BK, 2);
    }
    good = good && map_mn(&maps.m[n_maps + 6], W, M, N, 128, 4);
    n_maps += 7;
    p.mod = mod;
    p.gate_slot = slot;
    p.gate_grad = dmod != nullptr;
    p.gate_part = gate_part;
    if (dmod != nullptr) {
      const int n = gate_parts(M, N, L_pad);
      for (int m = 0; m < 3; ++m) {
        fin.reduce.begin[m] = m * n;
        fin.reduce.end[m] = count[m] > 0 ? (m + 1) * n : m * n;  // no tokens: 0
        fin.reduce.out[m] = dmod + (long)(m * 6 + slot) * M;
      }
      fin.n_reduce = 3;
      fin.reduce_part = gate_part;
      fin.reduce_stride = M;
      fin.reduce_cols = M;
    }
  }
  // One launch for all products, or one for each: pairs that begin a product
  // together walk it in step, so that a wave's shared panels are read from
  // HBM once; those that run on into the next product while others finish the
  // last lose that (QKV at 7,904 tokens: 6.1 against 4.7 GB read, and under
  // the power cap 4.02 against 3.86 ms; out-projection at 32,160 tokens 4.53
  // against 4.10 ms).  Short products gain more from the one tail and launch
  // (out-projection at 4,096 tokens 532 against 567 us, 1,024 x 1,024 x 1,024
  // 20 against 30 us).  The two meet near 2,000 k blocks for each pair.
  bool together() const {
    long blocks = 0;
    for (int i = 0; i < p.n_products; ++i)
      blocks += (long)p.pr[i].m_tiles * p.pr[i].n_tiles * (p.pr[i].kb[0] + p.pr[i].kb[1] + p.pr[i].kb[2]);
    return blocks < 2000L * gemm_bwd::max_cta_pairs();
  }
  cudaError_t run(cudaStream_t stream) {
    if (!good) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (together()) {
      p.n_maps = n_maps;
      e = gemm_bwd::launch<gemm_bwd::PRODUCTS>(maps, p, stream);
    } else {
      for (int i = 0; i < p.n_products && e == cudaSuccess; ++i) {
        gemm_bwd::Params one = p;
        gemm_bwd::Maps m;
        memset(&m, 0, sizeof(m));
        one.pr[0] = p.pr[i];
        one.n_products = 1;
        one.n_maps = 2 * p.pr[i].segs + p.pr[i].gated;
        memcpy(m.m, maps.m + p.pr[i].map0, one.n_maps * sizeof(CUtensorMap));
        one.pr[0].map0 = 0;
        one.gate_grad = p.gate_grad && p.pr[i].gated;
        e = gemm_bwd::launch<gemm_bwd::PRODUCTS>(m, one, stream);
      }
    }
    return e != cudaSuccess ? e : launch_finish(fin, stream);
  }
};

// h [rows][F] and dgu [rows][2F] from xm, dy [rows][D], Wgu [2F][D], Wd [D][F]
cudaError_t launch_ffn_bwd(const bf16* xm, const bf16* dy, const bf16* Wgu, const bf16* Wd, int rows, int D, int F,
                           bf16* h, bf16* dgu, cudaStream_t stream) {
  using namespace gemm_bwd;
  Maps maps;
  Params p;
  memset(&maps, 0, sizeof(maps));
  memset(&p, 0, sizeof(p));
  if (!map_k(&maps.m[0], xm, rows, D, D) || !map_k(&maps.m[1], Wgu, 2 * F, D, D) ||
      !map_k(&maps.m[2], dy, rows, D, D) || !map_mn(&maps.m[3], Wd, D, F, gemm_bwd::BK, 1))
    return cudaErrorInvalidValue;
  p.n_products = 1;
  Product& pr = p.pr[0];
  p.n_maps = 4;
  set_tiles(pr, rows, F, 128);
  pr.segs = pr.splits = 1;
  pr.kb[0] = D / gemm_bwd::BK;
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
  if (!map_k(&maps.m[0], xm, rows, D, D) || !map_k(&maps.m[1], Wqkv, 2 * I, D, D)) return cudaErrorInvalidValue;
  p.n_products = 1;
  Product& pr = p.pr[0];
  p.n_maps = 2;
  set_tiles(pr, rows, 2 * I, 256);
  pr.segs = pr.splits = 1;
  pr.kb[0] = D / gemm_bwd::BK;
  p.rows = rows;
  p.dqkv = dqkv;
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
  const int tiles = pr.m_tiles * pr.n_tiles, max_pairs = max_cta_pairs();
  *n_parts = 2 * (tiles < max_pairs ? tiles : max_pairs);
  return launch<QKNORM>(maps, p, stream);
}

}  // namespace h3
