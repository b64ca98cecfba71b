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
// A CTA takes a run of rows of one modality and keeps its columns' two sums
// in registers; they leave as one partial row per CTA.
constexpr int AB_THREADS = 256;

struct Chunks {
  int first[4];   // CTAs [first[m], first[m + 1]) take modality m's rows
  int rows[3];    // rows per CTA of modality m
};

// N sums over the CTA at once; `red` holds N x 8 floats and is free again
// after the call's last barrier plus the next call's first
template <int N>
__device__ __forceinline__ void block_sums(float* v, float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  if (l == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 8 + w] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < AB_THREADS / 32; ++k) t += red[i * 8 + k];
    v[i] = t;
  }
}

// VPT: float4 columns per thread (D <= 1024 VPT)
template <int VPT>
__global__ void __launch_bounds__(AB_THREADS) adaln_bwd_kernel(
    const float* __restrict__ x, const float* __restrict__ mod, int branch, const bf16* __restrict__ dy,
    const float* dres, float* dx, RangeArgs rg, Chunks ch, int L, int L_pad, int D, float eps,
    float* __restrict__ part) {
  __shared__ float red[2][3 * 8];
  const int nv = D / 4;
  const int n_chunks = ch.first[3];
  if ((int)blockIdx.x >= n_chunks) {  // padding rows
    for (long row = L + blockIdx.x - n_chunks; row < L_pad; row += gridDim.x - n_chunks)
      for (int i = threadIdx.x; i < nv; i += AB_THREADS)
        reinterpret_cast<float4*>(dx + row * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  const int m = (int)blockIdx.x >= ch.first[2] ? 2 : ((int)blockIdx.x >= ch.first[1] ? 1 : 0);
  const int off = ((int)blockIdx.x - ch.first[m]) * ch.rows[m];
  const int row_end = rg.start[m] + min(rg.count[m], off + ch.rows[m]);
  const float4* scale = reinterpret_cast<const float4*>(mod + (long)(m * 6 + 3 * branch + 1) * D);
  float4 a_shift[VPT], a_scale[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) a_shift[k] = a_scale[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (long row = rg.start[m] + off; row < row_end; ++row) {
    const float4* xr = reinterpret_cast<const float4*>(x + row * D);
    const uint2* yr = reinterpret_cast<const uint2*>(dy + row * D);
    const float4* rr = reinterpret_cast<const float4*>(dres + row * D);
    float4 v[VPT];
    uint2 g[VPT];
    float s1[1] = {0.f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = threadIdx.x + k * AB_THREADS;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      g[k] = make_uint2(0, 0);
      if (i < nv) {
        v[k] = __ldcs(xr + i);
        g[k] = __ldcs(yr + i);
        s1[0] += (v[k].x + v[k].y) + (v[k].z + v[k].w);
      }
    }
    block_sums<1>(s1, red[0]);
    const float mu = s1[0] / (float)D;  // divided as the forward call divides: a constant row has xhat = 0
    float s3[3] = {0.f, 0.f, 0.f};  // sum (x - mu)^2, sum dh, sum dh (x - mu)
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = threadIdx.x + k * AB_THREADS;
      if (i < nv) {
        v[k].x -= mu;
        v[k].y -= mu;
        v[k].z -= mu;
        v[k].w -= mu;
        const float4 sc = __ldg(scale + i);
        const float2 g0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&g[k].x));
        const float2 g1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&g[k].y));
        const float h0 = g0.x * (1.f + sc.x), h1 = g0.y * (1.f + sc.y), h2 = g1.x * (1.f + sc.z),
                    h3 = g1.y * (1.f + sc.w);
        s3[0] += (v[k].x * v[k].x + v[k].y * v[k].y) + (v[k].z * v[k].z + v[k].w * v[k].w);
        s3[1] += (h0 + h1) + (h2 + h3);
        s3[2] += (h0 * v[k].x + h1 * v[k].y) + (h2 * v[k].z + h3 * v[k].w);
      }
    }
    block_sums<3>(s3, red[1]);
    const float rstd = rsqrtf(s3[0] / (float)D + eps);
    const float mean_h = s3[1] / (float)D, mean_hx = s3[2] / (float)D * rstd;  // mean(dh), mean(dh xhat)
    float4* out = reinterpret_cast<float4*>(dx + row * D);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = threadIdx.x + k * AB_THREADS;
      if (i < nv) {
        const float4 sc = __ldg(scale + i);
        const float4 r = __ldcs(rr + i);
        const float2 g0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&g[k].x));
        const float2 g1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&g[k].y));
        const float4 xh = make_float4(v[k].x * rstd, v[k].y * rstd, v[k].z * rstd, v[k].w * rstd);
        a_shift[k].x += g0.x;
        a_shift[k].y += g0.y;
        a_shift[k].z += g1.x;
        a_shift[k].w += g1.y;
        a_scale[k].x = fmaf(g0.x, xh.x, a_scale[k].x);
        a_scale[k].y = fmaf(g0.y, xh.y, a_scale[k].y);
        a_scale[k].z = fmaf(g1.x, xh.z, a_scale[k].z);
        a_scale[k].w = fmaf(g1.y, xh.w, a_scale[k].w);
        float4 o;
        o.x = fmaf(rstd, g0.x * (1.f + sc.x) - mean_h - xh.x * mean_hx, r.x);
        o.y = fmaf(rstd, g0.y * (1.f + sc.y) - mean_h - xh.y * mean_hx, r.y);
        o.z = fmaf(rstd, g1.x * (1.f + sc.z) - mean_h - xh.z * mean_hx, r.z);
        o.w = fmaf(rstd, g1.y * (1.f + sc.w) - mean_h - xh.w * mean_hx, r.w);
        __stcs(out + i, o);
      }
    }
  }
  float4* p0 = reinterpret_cast<float4*>(part + (long)blockIdx.x * 2 * D);
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = threadIdx.x + k * AB_THREADS;
    if (i < nv) {
      p0[i] = a_shift[k];
      p0[nv + i] = a_scale[k];
    }
  }
}

// ------------------------------------------------------------ partial sums
// out[m * out_stride + c] = bf16(sum of part[p * stride + c] over p in
// [begin[m], end[m])), c < cols.  A CTA takes 32
// columns; its eight warps take every eighth partial and their sums are added
// in order.
struct Parts {
  int begin[3], end[3];
};
__global__ void __launch_bounds__(256) reduce_parts_kernel(const float* __restrict__ part, Parts pp, long stride,
                                                           int cols, bf16* __restrict__ out, long out_stride) {
  __shared__ float acc[8][32];
  const int m = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x / 32;
  float s = 0.f;
  if (c < cols) {
    int p = pp.begin[m] + w;
    const int end = pp.end[m];
    for (; p + 24 < end; p += 32) {
      const float a = part[p * stride + c], b = part[(p + 8) * stride + c], d = part[(p + 16) * stride + c],
                  e = part[(p + 24) * stride + c];
      s += (a + b) + (d + e);
    }
    for (; p < end; p += 8) s += part[p * stride + c];
  }
  acc[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += acc[k][threadIdx.x];
    out[m * out_stride + c] = __float2bfloat16_rn(t);
  }
}

// ------------------------------------------------------------ residual gradient
// The bf16 operands of a gated linear's backward GEMMs from the fp32 residual
// gradient: plain = bf16(dx) (weight and gate gradients) and gated =
// bf16(gate_m (.) dx) (input gradient).  Valid rows only; either may be null.
__global__ void __launch_bounds__(256) gate_cast_kernel(const float* __restrict__ dx, const float* __restrict__ mod,
                                                        int gate_slot, RangeArgs rg, int L, int D,
                                                        bf16* __restrict__ plain, bf16* __restrict__ gated) {
  const int n8 = D / 8;
  const long total = (long)L * n8;
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
  for (long i = blockIdx.x * 256L + threadIdx.x; i < total; i += gridDim.x * 256L) {
    const int row = (int)(i / per_row), c = (int)(i - (long)row * per_row);
    const int h = c >> 4, j = c & 15;
    reinterpret_cast<uint4*>(dqkv)[(long)row * 3 * per_row + 2 * per_row + c] =
        __ldcs(reinterpret_cast<const uint4*>(dv) + ((long)h * L_pad + row) * 16 + j);
  }
}

}  // namespace bwd_detail
using namespace bwd_detail;

// CTAs that the AdaLN backward pass spreads the valid rows over: two per SM.
// Each modality's last one may be short, so up to two more partial rows.
constexpr int ADALN_BWD_CTAS = 296;
constexpr int ADALN_BWD_PARTS = ADALN_BWD_CTAS + 2;

cudaError_t launch_adaln_bwd(const float* x, const float* mod, int branch, const bf16* dy, const float* dres, float* dx,
                             const int* rstart, const int* rcount, int L, int L_pad, int D, float eps, float* part,
                             bf16* dmod, cudaStream_t stream) {
  RangeArgs rg;
  Chunks ch;
  const int per_cta = (L + ADALN_BWD_CTAS - 1) / ADALN_BWD_CTAS;
  int n = 0;
  for (int m = 0; m < 3; ++m) {
    rg.start[m] = rstart[m];
    rg.count[m] = rcount[m];
    ch.first[m] = n;
    ch.rows[m] = per_cta;
    n += (rcount[m] + per_cta - 1) / per_cta;
  }
  ch.first[3] = n;
  const int pad = L_pad - L < ADALN_BWD_CTAS ? L_pad - L : ADALN_BWD_CTAS;
  const int grid = n + pad;
#define H3_ADALN_BWD(V)                                                                                              \
  case V:                                                                                                            \
    adaln_bwd_kernel<V><<<grid, AB_THREADS, 0, stream>>>(x, mod, branch, dy, dres, dx, rg, ch, L, L_pad, D, eps, part); \
    break;
  switch ((D + 1023) / 1024) {
    H3_ADALN_BWD(1)
    H3_ADALN_BWD(2)
    H3_ADALN_BWD(3)
    H3_ADALN_BWD(4)
    H3_ADALN_BWD(5)
    H3_ADALN_BWD(6)
    H3_ADALN_BWD(7)
    H3_ADALN_BWD(8)
    default: return cudaErrorInvalidValue;
  }
#undef H3_ADALN_BWD
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || dmod == nullptr) return e;
  // the branch's shift and scale rows are neighbours in [3][6][D], as their
  // partials are
  Parts pp;
  for (int m = 0; m < 3; ++m) {
    pp.begin[m] = ch.first[m];
    pp.end[m] = ch.first[m + 1];
  }
  reduce_parts_kernel<<<dim3((2 * D + 31) / 32, 3), 256, 0, stream>>>(part, pp, 2L * D, 2 * D,
                                                                      dmod + (long)3 * branch * D, 6L * D);
  return cudaGetLastError();
}

// dmod[m][gate_slot][:] from part [3][n_parts][D] (modalities without tokens: 0)
cudaError_t launch_gate_reduce(const float* part, int n_parts, const int* rcount, int D, int gate_slot, bf16* dmod,
                               cudaStream_t stream) {
  Parts pp;
  for (int m = 0; m < 3; ++m) {
    pp.begin[m] = m * n_parts;
    pp.end[m] = rcount[m] > 0 ? (m + 1) * n_parts : m * n_parts;
  }
  reduce_parts_kernel<<<dim3((D + 31) / 32, 3), 256, 0, stream>>>(part, pp, D, D, dmod + (long)gate_slot * D, 6L * D);
  return cudaGetLastError();
}

// dqn_w, dkn_w [128] from part [n_parts][2][128]
cudaError_t launch_norm_weight_reduce(const float* part, int n_parts, bf16* dqn_w, bf16* dkn_w, cudaStream_t stream) {
  Parts pp;
  memset(&pp, 0, sizeof(pp));
  pp.end[0] = n_parts;
  if (dqn_w) reduce_parts_kernel<<<dim3(4, 1), 256, 0, stream>>>(part, pp, 256, 128, dqn_w, 0);
  if (dkn_w) reduce_parts_kernel<<<dim3(4, 1), 256, 0, stream>>>(part + 128, pp, 256, 128, dkn_w, 0);
  return cudaGetLastError();
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
  gate_cast_kernel<<<stream_grid((long)L * D / 8), 256, 0, stream>>>(dx, mod, gate_slot, rg, L, D, plain, gated);
  return cudaGetLastError();
}

cudaError_t launch_dv_rows(const bf16* dv, int H, int L, int L_pad, bf16* dqkv, cudaStream_t stream) {
  dv_rows_kernel<<<stream_grid((long)L * H * 16), 256, 0, stream>>>(dv, H, L, L_pad, dqkv);
  return cudaGetLastError();
}

}  // namespace h3
