// Memory-bound kernels of the block's backward pass: the AdaLN norm's
// gradient, the bf16 copies of a residual gradient that the backward GEMMs
// read, the token-major copy of dv, and the reductions that finish
// per-CTA partial sums in a fixed order (no atomics: the same call gives the
// same bits).
#include "h3_internal.cuh"
#include "ptx.cuh"

namespace h3 {

namespace bwd_detail {
using ew_detail::RangeArgs;
using ew_detail::range_of;

// ------------------------------------------------------------ AdaLN backward
// y = xhat (1 + scale_m) + shift_m, xhat = (x - mu) rstd.  With dh = dy (1 +
// scale_m):
//   dx       = dres + rstd (dh - mean(dh) - xhat mean(dh xhat))
//   dshift_m = sum_{rows of m} dy,   dscale_m = sum_{rows of m} dy xhat
// The statistics are recomputed from x (4 bytes of the 14 an element moves).
// A CTA takes a run of rows of one modality; its rows come through a ring of
// shared-memory stages by bulk copies (x, dy and dres of a row, 10 D bytes),
// so that HBM is never idle while a row waits for its two reductions, and its
// columns' two sums stay in registers, leaving as one partial row per CTA.
// HBM bounds it: 32,160 rows of 5,376 (2.42 GB) in 433 us with the reduction of
// the partials, 5.6 TB/s.
constexpr int AB_MAX_THREADS = 512;
constexpr int AB_STAGES = 4;
constexpr int AB_SMEM = 216 * 1024;  // per SM, for the stages of its CTAs

struct AdalnPlan {
  int vpt;       // float4 columns of a thread
  int threads;   // of a CTA, up to 512
  int per_sm;    // CTAs per SM: one row's reductions hide behind another's arithmetic
  int stages;
  int ctas;      // partial rows, at most
};
static AdalnPlan adaln_plan(int D) {
  AdalnPlan p;
  const int nv = D / 4;
  if (nv <= 128) {
    // narrow rows: one warp a row, no barrier in its reductions, and as many
    // of them as fit with four stages and 1.5 KB each (26,857 rows of 256,
    // the second launch included: 51 us with a CTA of 64 threads a row, 27 us so)
    p.vpt = (nv + 31) / 32;
    p.threads = 32;
    p.stages = AB_STAGES;
    const int fit = 225 * 1024 / (AB_STAGES * 10 * D + 1536);
    p.per_sm = fit < 16 ? fit : 16;
    p.ctas = 148 * p.per_sm;
    return p;
  }
  p.vpt = (nv + AB_MAX_THREADS - 1) / AB_MAX_THREADS;
  p.threads = ((nv + p.vpt - 1) / p.vpt + 31) / 32 * 32;
  p.per_sm = 1024 / p.threads;
  if (p.per_sm > 8) p.per_sm = 8;
  while (p.per_sm > 1 && AB_SMEM / p.per_sm < 20 * D) --p.per_sm;  // two stages at least: 20 D <= 160 KB
  const int fit = AB_SMEM / p.per_sm / (10 * D);
  p.stages = fit < AB_STAGES ? fit : AB_STAGES;
  p.ctas = 148 * p.per_sm;
  return p;
}

struct Chunks {
  int first[4];   // CTAs [first[m], first[m + 1]) take modality m's rows
  int rows;       // rows per CTA
};

// N sums over the CTA at once; `red` holds N x 16 floats and is free again
// after the next barrier
template <int N>
__device__ __forceinline__ void block_sums(float* v, float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int w = threadIdx.x / 32, l = threadIdx.x % 32, nw = blockDim.x / 32;
  if (nw == 1) {
    __syncwarp();
    return;
  }
  if (l == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 16 + w] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = l < nw ? red[i * 16 + l] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    v[i] = __shfl_sync(0xffffffffu, t, 0);
  }
}

// a pair of bf16 as a packed pair of fp32
__device__ __forceinline__ uint64_t f2_of_bf16(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float f2_sum(uint64_t a, uint64_t b) {
  float x, y;
  f2_unpack(f2_add(a, b), x, y);
  return x + y;
}

// VPT: float4 columns per thread (D <= 4 VPT threads); arithmetic on packed
// pairs of fp32
template <int VPT>
__global__ void __launch_bounds__(AB_MAX_THREADS, VPT <= 3 ? 2 : 1) adaln_bwd_kernel(
    const float* __restrict__ x, const float* __restrict__ mod, int branch, const bf16* __restrict__ dy,
    const float* dres, float* dx, RangeArgs rg, Chunks ch, int L, int L_pad, int D, float eps, int stages,
    float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t smem_ab[];
  __shared__ float red[2][3 * 16];
  __shared__ uint64_t full[AB_STAGES];
  const int nv = D / 4, T = blockDim.x;
  const int n_chunks = ch.first[3];
  chain_wait();
  if ((int)blockIdx.x >= n_chunks) {  // padding rows
    for (long row = L + blockIdx.x - n_chunks; row < L_pad; row += gridDim.x - n_chunks)
      for (int i = threadIdx.x; i < nv; i += T)
        reinterpret_cast<float4*>(dx + row * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  const int m = (int)blockIdx.x >= ch.first[2] ? 2 : ((int)blockIdx.x >= ch.first[1] ? 1 : 0);
  const int off = ((int)blockIdx.x - ch.first[m]) * ch.rows;
  const long row0 = rg.start[m] + off;
  const int n_rows = min(rg.count[m] - off, ch.rows);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t stage_bytes = 10u * D;
  // row i's x | dres | dy into stage i % stages
  auto load_row = [&](int i) {
    const int st = i % stages;
    uint8_t* dst = smem_ab + st * stage_bytes;
    mbar_arrive_expect_tx(&full[st], stage_bytes);
    bulk_load(dst, x + (row0 + i) * D, 4u * D, &full[st]);
    bulk_load(dst + 4u * D, dres + (row0 + i) * D, 4u * D, &full[st]);
    bulk_load(dst + 8u * D, dy + (row0 + i) * D, 2u * D, &full[st]);
  };
  int issued = 0;  // thread 0's
  if (threadIdx.x == 0)
    while (issued < stages - 1 && issued < n_rows) load_row(issued++);
  const float4* scale = reinterpret_cast<const float4*>(mod + (long)(m * 6 + 3 * branch + 1) * D);
  uint64_t a_shift[VPT][2], a_scale[VPT][2], sc[VPT][2];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = threadIdx.x + k * T;
    const float4 t = i < nv ? __ldg(scale + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    sc[k][0] = f2_pack(1.f + t.x, 1.f + t.y);
    sc[k][1] = f2_pack(1.f + t.z, 1.f + t.w);
#pragma unroll
    for (int j = 0; j < 2; ++j) a_shift[k][j] = a_scale[k][j] = 0ull;
  }
  bool ok = true;
  for (int r = 0; r < n_rows && ok; ++r) {
    const int st = r % stages;
    const ulonglong2* xr = reinterpret_cast<const ulonglong2*>(smem_ab + st * stage_bytes);
    const ulonglong2* rr = xr + nv;
    const uint2* yr = reinterpret_cast<const uint2*>(rr + nv);
    ok = mbar_wait(&full[st], (r / stages) & 1);
    uint64_t v[VPT][2];
    float s1[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = threadIdx.x + k * T;
      v[k][0] = v[k][1] = 0ull;
      if (i < nv) {
        const ulonglong2 t = xr[i];
        v[k][0] = t.x;
        v[k][1] = t.y;
      }
      s1[0] += f2_sum(v[k][0], v[k][1]);
    }
    block_sums<1>(s1, red[0]);
    // every thread has left row r - 1, whose stage takes row r + stages - 1
    if (threadIdx.x == 0 && r + stages - 1 < n_rows) load_row(issued++);
    const float mu = s1[0] / (float)D;  // divided as the forward call divides: a constant row has xhat = 0
    const uint64_t nmu = f2_pack(-mu, -mu);
    uint64_t q[3] = {0ull, 0ull, 0ull};  // sum (x - mu)^2, sum dh, sum dh (x - mu)
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = threadIdx.x + k * T;
      if (i < nv) {
        const uint2 g = yr[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[k][j] = f2_add(v[k][j], nmu);
          const uint64_t h = f2_mul(f2_of_bf16(j == 0 ? g.x : g.y), sc[k][j]);
          q[0] = f2_fma(v[k][j], v[k][j], q[0]);
          q[1] = f2_add(q[1], h);
          q[2] = f2_fma(h, v[k][j], q[2]);
        }
      }
    }
    float s3[3] = {f2_sum(q[0], 0ull), f2_sum(q[1], 0ull), f2_sum(q[2], 0ull)};
    block_sums<3>(s3, red[1]);
    const float rstd = rsqrtf(s3[0] / (float)D + eps);
    const float mean_h = s3[1] / (float)D, mean_hx = s3[2] / (float)D * rstd;  // mean(dh), mean(dh xhat)
    const uint64_t rs = f2_pack(rstd, rstd), nmh = f2_pack(-mean_h, -mean_h), nmx = f2_pack(-mean_hx, -mean_hx);
    float4* out = reinterpret_cast<float4*>(dx + (row0 + r) * D);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = threadIdx.x + k * T;
      if (i < nv) {
        const uint2 g2 = yr[i];
        const ulonglong2 res = rr[i];
        uint64_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t g = f2_of_bf16(j == 0 ? g2.x : g2.y), xh = f2_mul(v[k][j], rs);
          a_shift[k][j] = f2_add(a_shift[k][j], g);
          a_scale[k][j] = f2_fma(g, xh, a_scale[k][j]);
          o[j] = f2_fma(f2_fma(xh, nmx, f2_fma(g, sc[k][j], nmh)), rs, j == 0 ? res.x : res.y);
        }
        float4 w;
        f2_unpack(o[0], w.x, w.y);
        f2_unpack(o[1], w.z, w.w);
        __stcs(out + i, w);
      }
    }
  }
  if (threadIdx.x == 0 && !ok) drain_loads(full, stages, issued);  // after a wait that gave up
  ulonglong2* p0 = reinterpret_cast<ulonglong2*>(part + (long)blockIdx.x * 2 * D);
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = threadIdx.x + k * T;
    if (i < nv) {
      p0[i] = make_ulonglong2(a_shift[k][0], a_shift[k][1]);
      p0[nv + i] = make_ulonglong2(a_scale[k][0], a_scale[k][1]);
    }
  }
}

// ------------------------------------------------------------ partial sums
// out[m][c] = bf16(sum of part[p * stride + m * offset + c] over p in [begin[m],
// end[m])), c < cols, for the blockIdx.y-th m.  A CTA takes 32 columns; its W
// warps take every W-th partial, eight at a time, and their sums are added in
// order.
struct Parts {
  int begin[3], end[3];
  bf16* out[3];  // null: not wanted
};
template <int W>
__device__ __forceinline__ void reduce_parts(const float* __restrict__ part, const Parts& pp, int m, long stride,
                                             long offset, int cols, int block, float (*acc)[32]) {
  const int c = block * 32 + (threadIdx.x & 31), w = threadIdx.x / 32;
  part += m * offset + c;
  float s = 0.f;
  if (c < cols && pp.out[m] != nullptr) {
    int p = pp.begin[m] + w;
    const int end = pp.end[m];
    for (; p + 7 * W < end; p += 8 * W) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = part[(p + k * W) * stride];
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; p < end; p += W) s += part[p * stride];
  }
  acc[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0 && c < cols && pp.out[m] != nullptr) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) t += acc[k][threadIdx.x];
    pp.out[m][c] = __float2bfloat16_rn(t);
  }
}
template <int W>
__global__ void __launch_bounds__(W * 32) reduce_parts_kernel(const float* __restrict__ part,
                                                              const __grid_constant__ Parts pp, long stride,
                                                              long offset, int cols) {
  __shared__ float acc[W][32];
  chain_wait();
  reduce_parts<W>(part, pp, blockIdx.y, stride, offset, cols, blockIdx.x, acc);
}

// What is left after the products of a backward call: the sums of the split
// ones, out [n] = bf16(sum over part [splits][n]) (n a multiple of 8), and one
// reduction of partials (a gate's or the norm weights' gradients)
struct SplitSum {
  const float* part;
  bf16* out;
  long n;
  int splits;
};
struct FinishArgs {
  int n_sums, n_reduce;
  SplitSum sum[3];
  int first[4];  // CTAs [first[i], first[i + 1]) take sum i, the rest the reduction
  Parts reduce;
  const float* reduce_part;
  long reduce_stride, reduce_offset;
  int reduce_cols, reduce_ctas;
};
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishArgs f) {
  __shared__ float acc[8][32];
  chain_wait();
  const int b = blockIdx.x;
  if (b >= f.first[f.n_sums]) {
    const int r = b - f.first[f.n_sums];
    reduce_parts<8>(f.reduce_part, f.reduce, r / f.reduce_ctas, f.reduce_stride, f.reduce_offset, f.reduce_cols,
                 r % f.reduce_ctas, acc);
    return;
  }
  int k = 0;
  while (b >= f.first[k + 1]) ++k;
  const SplitSum& j = f.sum[k];
  const long step = (f.first[k + 1] - f.first[k]) * 2048L;
  for (long i = ((b - f.first[k]) * 256L + threadIdx.x) * 8; i < j.n; i += step) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    for (int s = 0; s < j.splits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(j.part + s * j.n + i);
      const float4 u = __ldcs(src), v = __ldcs(src + 1);
      x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
      y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    *reinterpret_cast<uint4*>(j.out + i) =
        make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  }
}

// ------------------------------------------------------------ residual gradient
// The bf16 operands of a gated linear's backward GEMMs from the fp32 residual
// gradient: plain = bf16(dx) (weight and gate gradients) and gated =
// bf16(gate_m (.) dx) (input gradient), each rounded once, by half a step (2^-8)
// at most, as the tensor cores' operand.  Valid rows only; either may be null.
// 32,160 rows of 5,376 in 0.25 ms (HBM).
__global__ void __launch_bounds__(256) gate_cast_kernel(const float* __restrict__ dx, const float* __restrict__ mod,
                                                        int gate_slot, RangeArgs rg, int L, int D,
                                                        bf16* __restrict__ plain, bf16* __restrict__ gated) {
  const int n8 = D / 8;
  const long total = (long)L * n8;
  chain_wait();
  for (long i = blockIdx.x * 256L + threadIdx.x; i < total; i += gridDim.x * 256L) {
    const int row = (int)(i / n8), c = (int)(i - (long)row * n8);
    const float4* src = reinterpret_cast<const float4*>(dx + (long)row * D) + 2 * c;
    const float4 a = __ldcs(src), b = __ldcs(src + 1);
    if (plain)
      reinterpret_cast<uint4*>(plain)[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w),
                                                      pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
    if (gated) {
      const int m = range_of(row, rg.start, rg.count);
      const float4* g = reinterpret_cast<const float4*>(mod + (long)(m * 6 + gate_slot) * D) + 2 * c;
      const float4 ga = __ldg(g), gb = __ldg(g + 1);
      reinterpret_cast<uint4*>(gated)[i] =
          make_uint4(pack_bf16x2(a.x * ga.x, a.y * ga.y), pack_bf16x2(a.z * ga.z, a.w * ga.w),
                     pack_bf16x2(b.x * gb.x, b.y * gb.y), pack_bf16x2(b.z * gb.z, b.w * gb.w));
    }
  }
}

// dv [H][L_pad][128] -> columns [2I, 3I) of the token-major dqkv [L][3I]
__global__ void __launch_bounds__(256) dv_rows_kernel(const bf16* __restrict__ dv, int H, int L, int L_pad,
                                                      bf16* __restrict__ dqkv) {
  const int per_row = H * 16;  // 16-byte pieces
  const long total = (long)L * per_row;
  chain_wait();
  for (long i = blockIdx.x * 256L + threadIdx.x; i < total; i += gridDim.x * 256L) {
    const int row = (int)(i / per_row), c = (int)(i - (long)row * per_row);
    const int h = c >> 4, j = c & 15;
    reinterpret_cast<uint4*>(dqkv)[(long)row * 3 * per_row + 2 * per_row + c] =
        __ldcs(reinterpret_cast<const uint4*>(dv) + ((long)h * L_pad + row) * 16 + j);
  }
}

}  // namespace bwd_detail
using namespace bwd_detail;

int adaln_bwd_parts(int D) { return adaln_plan(D).ctas; }

cudaError_t launch_adaln_bwd(const float* x, const float* mod, int branch, const bf16* dy, const float* dres, float* dx,
                             const int* rstart, const int* rcount, int L, int L_pad, int D, float eps, float* part,
                             bf16* dmod, cudaStream_t stream) {
  const AdalnPlan plan = adaln_plan(D);
  RangeArgs rg;
  Chunks ch;
  // as few rows per CTA as let the three modalities' CTAs, whose last ones may
  // be short, run in one wave
  ch.rows = (L + plan.ctas - 1) / plan.ctas;
  if (plan.threads == 32 && L > 1024 && ch.rows < 4) ch.rows = 4;  // fewer partials than a warp a row would leave
  for (;; ++ch.rows) {
    ch.first[0] = 0;
    for (int m = 0; m < 3; ++m) ch.first[m + 1] = ch.first[m] + (rcount[m] + ch.rows - 1) / ch.rows;
    if (ch.first[3] <= plan.ctas) break;
  }
  for (int m = 0; m < 3; ++m) {
    rg.start[m] = rstart[m];
    rg.count[m] = rcount[m];
  }
  const int pad = L_pad - L < plan.ctas ? L_pad - L : plan.ctas;
  const int grid = ch.first[3] + pad;
  const int bytes = plan.stages * 10 * D;
  static unsigned long long attr_done[4] = {0, 0, 0, 0};
  cudaError_t e = cudaSuccess;
#define H3_ADALN_BWD(V)                                                                                              \
  case V: {                                                                                                          \
    cudaError_t ea = ensure_smem_attr(reinterpret_cast<const void*>(adaln_bwd_kernel<V>), AB_SMEM, &attr_done[V - 1]); \
    if (ea != cudaSuccess) return ea;                                                                                \
    e = launch_chained(adaln_bwd_kernel<V>, dim3(grid), plan.threads, bytes, stream, x, mod, branch, dy, dres, dx, rg, \
                       ch, L, L_pad, D, eps, plan.stages, part);                                                     \
    break;                                                                                                           \
  }
  switch (plan.vpt) {
    H3_ADALN_BWD(1)
    H3_ADALN_BWD(2)
    H3_ADALN_BWD(3)
    H3_ADALN_BWD(4)
    default: return cudaErrorInvalidValue;
  }
#undef H3_ADALN_BWD
  if (e != cudaSuccess || dmod == nullptr) return e;
  // the branch's shift and scale rows are neighbours in [3][6][D], as their
  // partials are
  Parts pp;
  for (int m = 0; m < 3; ++m) {
    pp.begin[m] = ch.first[m];
    pp.end[m] = ch.first[m + 1];
    pp.out[m] = dmod + (long)(m * 6 + 3 * branch) * D;
  }
  const dim3 grid_r((2 * D + 31) / 32, 3);
  // eight warps a CTA, or 32 where they would walk more than 32 partials each
  // (2,368 partials of 512 columns: 12 us with eight, 5 us with 32)
  if (ch.first[3] > 256)
    return launch_chained(reduce_parts_kernel<32>, grid_r, 1024, 0, stream, part, pp, 2L * D, 0L, 2 * D);
  return launch_chained(reduce_parts_kernel<8>, grid_r, 256, 0, stream, part, pp, 2L * D, 0L, 2 * D);
}

// One launch for all of it (none if nothing is left)
cudaError_t launch_finish(FinishArgs f, cudaStream_t stream) {
  int ctas = 0;
  for (int i = 0; i < f.n_sums; ++i) {
    const long blocks = (f.sum[i].n / 8 + 255) / 256, most = (long)num_sms() * 8;
    f.first[i] = ctas;
    ctas += (int)(blocks < most ? blocks : most);
  }
  f.first[f.n_sums] = ctas;
  if (f.n_reduce > 0) {
    f.reduce_ctas = (f.reduce_cols + 31) / 32;
    ctas += f.n_reduce * f.reduce_ctas;
  }
  return ctas > 0 ? launch_chained(finish_kernel, dim3(ctas), 256, 0, stream, f) : cudaSuccess;
}

static int stream_grid(long items) {
  long blocks = (items + 255) / 256;
  const long most = (long)num_sms() * 16;
  return (int)(blocks > most ? most : (blocks < 1 ? 1 : blocks));
}

cudaError_t launch_gate_cast(const float* dx, const float* mod, int gate_slot, const int* rstart, const int* rcount,
                             int L, int D, bf16* plain, bf16* gated, cudaStream_t stream) {
  RangeArgs rg;
  for (int m = 0; m < 3; ++m) {
    rg.start[m] = rstart[m];
    rg.count[m] = rcount[m];
  }
  return launch_chained(gate_cast_kernel, dim3(stream_grid((long)L * D / 8)), 256, 0, stream, dx, mod, gate_slot, rg, L,
                        D, plain, gated);
}

cudaError_t launch_dv_rows(const bf16* dv, int H, int L, int L_pad, bf16* dqkv, cudaStream_t stream) {
  return launch_chained(dv_rows_kernel, dim3(stream_grid((long)L * H * 16)), 256, 0, stream, dv, H, L, L_pad, dqkv);
}

}  // namespace h3
