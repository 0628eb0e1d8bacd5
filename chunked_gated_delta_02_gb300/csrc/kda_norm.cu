// Norms of a layer: the heads' output norm with its gate, and the norms around the residual
// addition with its gate and scale.
//
//   norm_gate:  y = x rms(x) w act(gate),            act = sigmoid or SiLU, rows of D values
//   add_norm:   z = x [rms(x) w_post] [sigmoid(gate)];  h = residual + s z;  y = h rms(h) w
//   rms(x) = 1 / sqrt(mean(x^2) + eps)
//
// Everything between the loads and the stores is fp32: y comes from the unrounded h, and each
// output is rounded once. Bound: every value is read and written once and costs a few operations,
// so memory bandwidth bounds large calls and launch and load latency small ones. A row lies in the
// registers of TPR threads (a part of a warp, or a CTA), 16 bytes per load, so the statistics need
// no second read; all loads of a row are issued before the first reduction.
//
// Measured on one GB300 (copy bandwidth 6.78 TB/s): norm_gate of 16384 x 32 rows of 128 values 62 us, 96% of that
// bandwidth; add_norm of 16384 rows of 4096 values, fp32 residual and all parts, 138 us, 100%; bf16 residual,
// addition and norm alone, 82 us, 96%. With a bf16 residual and all parts, rows of other lengths get less: 6000 of
// 5120 values 57.5 us, 79%; 4000 of 7168 52.3, 81%; 3068 of 5120 31.6, 73%.
//
// Launches overlap the end of the kernel ahead in the stream: in a graph of calls on eight rows norm_gate takes
// 1.6 us instead of 1.9, add_norm 2.35 instead of 2.7.
//
// Rows that do not fit the 16-byte path (D not a multiple of 8, an unaligned base or stride, or
// more than 16384 values) take a CTA per row with element-wise loads and the row in shared memory. Loads of 2 and 4
// bytes and, for short rows, idle threads between two block barriers bound them far above the bytes: add_norm, fp32
// residual and all parts, 16384 rows of 1023 values 77.3 us, 45% of the copy bandwidth, of 100 values 30.4 us, 11%;
// norm_gate 59.7 us, 25%, and 23.5 us, 6%.
#include <cmath>
#include <cstring>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_host.cuh"

namespace kda {

struct NormGateArgs {
  const __nv_bfloat16 *x, *gate;
  const float *weight;
  __nv_bfloat16 *y;
  int rows, inner;                 // rows in all, rows per outer index
  long long xs[2], gs[2];          // strides in elements: outer, inner
  int D;
  float eps;
  int silu;
};

struct AddNormArgs {
  const __nv_bfloat16 *x, *gate;   // gate may be null
  const void *residual;
  const float *weight, *post, *scale_vec;   // each may be null
  __nv_bfloat16 *y;
  void *h;
  long long xs, rs, gs;            // row strides in elements
  float scale, eps;
  int D;
  int ahead;                       // rows between the one a thread group has and the one it prefetches
};

__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(const float *src, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(src)), b = __ldg(reinterpret_cast<const float4 *>(src) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Sum over the TPR threads of a row: part of a warp, or the CTA (blockDim.x == TPR). The two sums
// of one row use different halves of `part`, so one barrier each is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float *part) {
#pragma unroll
  for (int m = 1; m < (TPR < 32 ? TPR : 32); m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) s += part[w];
  }
  return s;
}

// U rows per thread group (16-byte chunk c * TPR + t of a row in thread t), so that enough loads
// are in flight for short rows.
template <int TPR, int C, int U>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_gate_kernel(const NormGateArgs a) {
  __shared__ float part[TPR > 32 ? TPR / 32 : 1];
  pdl_wait();
  const int t = threadIdx.x % TPR;
  const int groups = blockDim.x / TPR;
  const int chunks = a.D / 8;
  const float inv_d = 1.0f / (float)a.D;
  const unsigned row0 = blockIdx.x * (groups * U) + threadIdx.x / TPR;   // rows < 2^31: no overflow
  uint4 xr[U][C], gr[U][C];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned row = row0 + u * groups;
    if (row >= (unsigned)a.rows) continue;
    unsigned i = row, j = 0;
    if (a.inner > 1) {   // 32-bit: a 64-bit division costs more than the rest of the row
      i = row / (unsigned)a.inner;
      j = row % (unsigned)a.inner;
    }
    const uint4 *x = reinterpret_cast<const uint4 *>(a.x + i * a.xs[0] + j * a.xs[1]);
    const uint4 *g = reinterpret_cast<const uint4 *>(a.gate + i * a.gs[0] + j * a.gs[1]);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * TPR + t < chunks) {
        xr[u][c] = __ldcs(x + c * TPR + t);
        gr[u][c] = __ldcs(g + c * TPR + t);
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned row = row0 + u * groups;
    const bool live = row < (unsigned)a.rows;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live && c * TPR + t < chunks) {
        float x[8];
        unpack8(xr[u][c], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
      }
    s = row_sum<TPR>(s, part);
    const float r = rsqrtf(fmaf(s, inv_d, a.eps));
    if (!live) continue;
    uint4 *y = reinterpret_cast<uint4 *>(a.y + (long long)row * a.D);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * TPR + t < chunks) {
        float x[8], g[8], w[8];
        unpack8(xr[u][c], x);
        unpack8(gr[u][c], g);
        if (a.weight) load8(a.weight + (c * TPR + t) * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float act = sigmoid_fast(g[e]);
          x[e] *= r * (a.silu ? g[e] * act : act);
          if (a.weight) x[e] *= w[e];
        }
        __stcs(y + c * TPR + t, pack8(x));
      }
  }
}

// Threads per SM the registers are fitted to, and bytes of input by which each row is prefetched into L2 before
// a CTA has it. A thread has fewer bytes of a bf16 residual in flight than of an fp32 one, too few for the
// whole bandwidth; from L2 they come sooner. Measured without and with prefetching (microseconds, 152 SMs; 6 MB gains
// less, 9 to 15 MB about the same): bf16 residual, 16384 rows of 4096 values 92 and 82, all parts 115 and 109;
// 10744 rows of 2880, all parts, 58 and 51; 4096 rows of 8192, all parts, 73 and 60; fp32 residual, 16384 rows of
// 4096, all parts, 137 and 138, 2048 rows of 16384 103 and 81. Two chunks per thread, bf16: 1280 threads 92, 1024 97.
template <int TPR, int C, typename RT>
constexpr int kAddNormThreads = C == 1 ? 1536 : C == 2 ? (sizeof(RT) == 2 ? 1280 : 1024) : TPR <= 384 ? 768 : 512;
constexpr double kAddNormAheadBytes = 15e6;
template <int TPR>
constexpr int kNormBlock = TPR > 32 ? TPR : 256;

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int TPR, int C, typename RT>
__global__ void __launch_bounds__(kNormBlock<TPR>, kAddNormThreads<TPR, C, RT> / kNormBlock<TPR>)
add_norm_kernel(const AddNormArgs a, long long rows) {
  __shared__ float part[2][TPR > 32 ? TPR / 32 : 1];
  pdl_wait();
  const int t = threadIdx.x % TPR;
  const int chunks = a.D / 8;
  const float inv_d = 1.0f / (float)a.D;
  const long long row = (long long)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
  const bool live = row < rows;
  uint4 xr[C], gr[C];
  float h[C][8];
  const uint4 *x = reinterpret_cast<const uint4 *>(a.x + row * a.xs);
  const uint4 *g = reinterpret_cast<const uint4 *>(a.gate + row * a.gs);
  const RT *res = static_cast<const RT *>(a.residual) + row * a.rs;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = c * TPR + t;
    if (live && k < chunks) {
      xr[c] = __ldcs(x + k);
      if (a.gate) gr[c] = __ldcs(g + k);
      if constexpr (sizeof(RT) == 4) {
        const float4 lo = __ldcs(reinterpret_cast<const float4 *>(res) + 2 * k);
        const float4 hi = __ldcs(reinterpret_cast<const float4 *>(res) + 2 * k + 1);
        h[c][0] = lo.x; h[c][1] = lo.y; h[c][2] = lo.z; h[c][3] = lo.w;
        h[c][4] = hi.x; h[c][5] = hi.y; h[c][6] = hi.z; h[c][7] = hi.w;
      } else {
        unpack8(__ldcs(reinterpret_cast<const uint4 *>(res) + k), h[c]);
      }
    }
  }
  if (row + a.ahead < rows) {
    const long long later = row + a.ahead;
    const char *xp = reinterpret_cast<const char *>(a.x + later * a.xs);
    const char *gp = reinterpret_cast<const char *>(a.gate + later * a.gs);
    const char *rp = reinterpret_cast<const char *>(static_cast<const RT *>(a.residual) + later * a.rs);
    for (int k = t; k < a.D / 64; k += TPR) {
      prefetch_l2(xp + k * 128);
      if (a.gate) prefetch_l2(gp + k * 128);
    }
    for (int k = t; k < a.D / (128 / (int)sizeof(RT)); k += TPR) prefetch_l2(rp + k * 128);
  }
  float r_post = 1.f;
  if (a.post) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live && c * TPR + t < chunks) {
        float v[8];
        unpack8(xr[c], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
      }
    r_post = rsqrtf(fmaf(row_sum<TPR>(s, part[0]), inv_d, a.eps));
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = c * TPR + t;
    if (live && k < chunks) {
      float z[8], f[8];
      unpack8(xr[c], z);
      if (a.post) {
        load8(a.post + k * 8, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= r_post * f[e];
      }
      if (a.gate) {
        unpack8(gr[c], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= sigmoid_fast(f[e]);
      }
      if (a.scale_vec) {
        load8(a.scale_vec + k * 8, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = fmaf(f[e], z[e], h[c][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = fmaf(a.scale, z[e], h[c][e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(h[c][e], h[c][e], s);
      RT *out = static_cast<RT *>(a.h) + row * a.D;
      if constexpr (sizeof(RT) == 4) {
        __stcs(reinterpret_cast<float4 *>(out) + 2 * k, make_float4(h[c][0], h[c][1], h[c][2], h[c][3]));
        __stcs(reinterpret_cast<float4 *>(out) + 2 * k + 1, make_float4(h[c][4], h[c][5], h[c][6], h[c][7]));
      } else {
        __stcs(reinterpret_cast<uint4 *>(out) + k, pack8(h[c]));
      }
    }
  }
  const float r = rsqrtf(fmaf(row_sum<TPR>(s, part[1]), inv_d, a.eps));
  if (!live) return;
  uint4 *y = reinterpret_cast<uint4 *>(a.y + row * a.D);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = c * TPR + t;
    if (k < chunks) {
      float f[8];
      if (a.weight) load8(a.weight + k * 8, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c][e] *= a.weight ? r * f[e] : r;
      __stcs(y + k, pack8(h[c]));
    }
  }
}

// ---- any D, alignment and stride: one CTA per row, the row's fp32 values in shared memory
constexpr int kAnyThreads = 256;
constexpr int kAnyMaxD = 32768;   // 128 KiB of shared memory

__global__ void __launch_bounds__(kAnyThreads) norm_gate_any_kernel(const NormGateArgs a) {
  extern __shared__ float row_buf[];
  __shared__ float part[kAnyThreads / 32];
  pdl_wait();
  const long long row = blockIdx.x;
  const unsigned i = blockIdx.x / (unsigned)a.inner, j = blockIdx.x % (unsigned)a.inner;
  const __nv_bfloat16 *x = a.x + i * a.xs[0] + j * a.xs[1], *g = a.gate + i * a.gs[0] + j * a.gs[1];
  float s = 0.f;
  for (int k = threadIdx.x; k < a.D; k += kAnyThreads) {
    const float v = __bfloat162float(x[k]);
    row_buf[k] = v;
    s = fmaf(v, v, s);
  }
  const float r = rsqrtf(fmaf(row_sum<kAnyThreads>(s, part), 1.0f / (float)a.D, a.eps));
  for (int k = threadIdx.x; k < a.D; k += kAnyThreads) {
    const float gv = __bfloat162float(g[k]), act = sigmoid_fast(gv);
    float v = row_buf[k] * (r * (a.silu ? gv * act : act));
    if (a.weight) v *= a.weight[k];
    a.y[row * a.D + k] = __float2bfloat16_rn(v);
  }
}

template <typename RT>
__global__ void __launch_bounds__(kAnyThreads) add_norm_any_kernel(const AddNormArgs a) {
  extern __shared__ float row_buf[];
  __shared__ float part[2][kAnyThreads / 32];
  pdl_wait();
  const long long row = blockIdx.x;
  const __nv_bfloat16 *x = a.x + row * a.xs, *g = a.gate ? a.gate + row * a.gs : nullptr;
  const RT *res = static_cast<const RT *>(a.residual) + row * a.rs;
  const float inv_d = 1.0f / (float)a.D;
  float s = 0.f;
  for (int k = threadIdx.x; k < a.D; k += kAnyThreads) {
    const float v = __bfloat162float(x[k]);
    row_buf[k] = v;
    s = fmaf(v, v, s);
  }
  const float r_post = a.post ? rsqrtf(fmaf(row_sum<kAnyThreads>(s, part[0]), inv_d, a.eps)) : 1.f;
  s = 0.f;
  for (int k = threadIdx.x; k < a.D; k += kAnyThreads) {   // each thread reads back what it wrote
    float z = row_buf[k];
    if (a.post) z *= r_post * a.post[k];
    if (g) z *= sigmoid_fast(__bfloat162float(g[k]));
    const float h = fmaf(a.scale_vec ? a.scale_vec[k] : a.scale, z, (float)res[k]);
    row_buf[k] = h;
    s = fmaf(h, h, s);
    static_cast<RT *>(a.h)[row * a.D + k] = (RT)h;
  }
  const float r = rsqrtf(fmaf(row_sum<kAnyThreads>(s, part[1]), inv_d, a.eps));
  for (int k = threadIdx.x; k < a.D; k += kAnyThreads)
    a.y[row * a.D + k] = __float2bfloat16_rn(row_buf[k] * (a.weight ? r * a.weight[k] : r));
}

static cudaError_t any_smem_limit(const void *kernel, PerDeviceOnce &once) {
  return once([&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAnyMaxD * 4);
  });
}

// Threads per row and 16-byte chunks per thread of a row of D values: one chunk up to 2048 values, two up to
// 6144, four beyond, and as few idle threads as multiples of 64 allow. (add_norm on one GB300, microseconds:
// 16384 rows of 2048 bf16 values, without gate and post norm, 46.7 with one chunk, 49.8 with two; 16384 of 4096, fp32
// residual, all parts, 136 with two, 152 with one; 8000 of 6144, bf16 residual, all parts, 77.5 with two, 84.2 with
// four; 4096 of 8192 59.1 and 57.3; 10744 of 2880 64 with 192 threads, 72 with 256.)
struct RowShape { int tpr, c; };
static RowShape row_shape(int D) {
  const int n = D / 8;
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  const int c = n <= 256 ? 1 : n <= 768 ? 2 : 4;
  return {(n + 64 * c - 1) / (64 * c) * 64, c};
}

template <int TPR, int C>
static cudaError_t launch_norm_gate(const NormGateArgs &a, cudaStream_t s, int sms) {
  constexpr int kThreads = kNormBlock<TPR>, kGroups = kThreads / TPR;
  if constexpr (TPR <= 32) {
    // Four rows per group only when that still leaves 24 CTAs per SM. Four and one, microseconds: 524288 rows of 128
    // values 63.4 and 66.2 (two: 65.7), of 64 values 31.7 and 33.5; 131072 strided rows of 128 20.8 and 18.9; 196608
    // rows of 64 15.4 and 14.8.
    if (a.rows >= sms * 24 * kGroups * 4)
      return launch_kernel(norm_gate_kernel<TPR, C, 4>, dim3(((unsigned)a.rows + kGroups * 4 - 1) / (kGroups * 4)),
                           dim3(kThreads), 0, s, true, a);
  }
  return launch_kernel(norm_gate_kernel<TPR, C, 1>, dim3(((unsigned)a.rows + kGroups - 1) / kGroups),
                       dim3(kThreads), 0, s, true, a);
}

template <int TPR, int C, typename RT>
static cudaError_t launch_add_norm(AddNormArgs a, long long rows, cudaStream_t s) {
  constexpr int kThreads = kNormBlock<TPR>, kGroups = kThreads / TPR;
  a.ahead = (int)(kAddNormAheadBytes / (a.D * (2.0 + sizeof(RT) + (a.gate ? 2 : 0))));
  return launch_kernel(add_norm_kernel<TPR, C, RT>, dim3((unsigned)((rows + kGroups - 1) / kGroups)), dim3(kThreads),
                       0, s, true, a, rows);
}

template <typename RT>
static cudaError_t launch_add_norm_rows(const AddNormArgs &a, long long rows, bool vec, cudaStream_t s) {
  if (!vec) {
    static PerDeviceOnce once;
    const cudaError_t e = any_smem_limit(reinterpret_cast<const void *>(add_norm_any_kernel<RT>), once);
    if (e != cudaSuccess) return e;
    return launch_kernel(add_norm_any_kernel<RT>, dim3((unsigned)rows), dim3(kAnyThreads), (size_t)a.D * 4, s, true, a);
  }
  const RowShape r = row_shape(a.D);
  switch (r.tpr * 8 + r.c) {
    case 8 * 8 + 1: return launch_add_norm<8, 1, RT>(a, rows, s);
    case 16 * 8 + 1: return launch_add_norm<16, 1, RT>(a, rows, s);
    case 32 * 8 + 1: return launch_add_norm<32, 1, RT>(a, rows, s);
    case 64 * 8 + 1: return launch_add_norm<64, 1, RT>(a, rows, s);
    case 128 * 8 + 1: return launch_add_norm<128, 1, RT>(a, rows, s);
    case 192 * 8 + 1: return launch_add_norm<192, 1, RT>(a, rows, s);
    case 256 * 8 + 1: return launch_add_norm<256, 1, RT>(a, rows, s);
    case 192 * 8 + 2: return launch_add_norm<192, 2, RT>(a, rows, s);
    case 256 * 8 + 2: return launch_add_norm<256, 2, RT>(a, rows, s);
    case 320 * 8 + 2: return launch_add_norm<320, 2, RT>(a, rows, s);
    case 384 * 8 + 2: return launch_add_norm<384, 2, RT>(a, rows, s);
    case 256 * 8 + 4: return launch_add_norm<256, 4, RT>(a, rows, s);
    case 320 * 8 + 4: return launch_add_norm<320, 4, RT>(a, rows, s);
    case 384 * 8 + 4: return launch_add_norm<384, 4, RT>(a, rows, s);
    case 448 * 8 + 4: return launch_add_norm<448, 4, RT>(a, rows, s);
    default: return launch_add_norm<512, 4, RT>(a, rows, s);
  }
}

static cudaError_t launch_norm_gate_rows(const NormGateArgs &a, bool vec, cudaStream_t s) {
  if (!vec) {
    static PerDeviceOnce once;
    const cudaError_t e = any_smem_limit(reinterpret_cast<const void *>(norm_gate_any_kernel), once);
    if (e != cudaSuccess) return e;
    return launch_kernel(norm_gate_any_kernel, dim3((unsigned)a.rows), dim3(kAnyThreads), (size_t)a.D * 4, s, true, a);
  }
  const int sms = device_sm_count();
  const RowShape r = row_shape(a.D);
  switch (r.tpr * 8 + r.c) {
    case 8 * 8 + 1: return launch_norm_gate<8, 1>(a, s, sms);
    case 16 * 8 + 1: return launch_norm_gate<16, 1>(a, s, sms);
    case 32 * 8 + 1: return launch_norm_gate<32, 1>(a, s, sms);
    case 64 * 8 + 1: return launch_norm_gate<64, 1>(a, s, sms);
    case 128 * 8 + 1: return launch_norm_gate<128, 1>(a, s, sms);
    case 192 * 8 + 1: return launch_norm_gate<192, 1>(a, s, sms);
    case 256 * 8 + 1: return launch_norm_gate<256, 1>(a, s, sms);
    case 192 * 8 + 2: return launch_norm_gate<192, 2>(a, s, sms);
    case 256 * 8 + 2: return launch_norm_gate<256, 2>(a, s, sms);
    case 320 * 8 + 2: return launch_norm_gate<320, 2>(a, s, sms);
    case 384 * 8 + 2: return launch_norm_gate<384, 2>(a, s, sms);
    case 256 * 8 + 4: return launch_norm_gate<256, 4>(a, s, sms);
    case 320 * 8 + 4: return launch_norm_gate<320, 4>(a, s, sms);
    case 384 * 8 + 4: return launch_norm_gate<384, 4>(a, s, sms);
    case 448 * 8 + 4: return launch_norm_gate<448, 4>(a, s, sms);
    default: return launch_norm_gate<512, 4>(a, s, sms);
  }
}

static bool all_multiples_of_8(const int64_t *s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] % 8 != 0) return false;
  return true;
}

}  // namespace kda

extern "C" {

kda_status_t kda_norm_gate(const void *x, const void *gate, const float *weight, float eps, int64_t outer,
                           int64_t inner, int D, const int64_t *strides, uint32_t flags, void *y,
                           kda_stream_t stream) {
  using namespace kda;
  if ((flags & ~KDA_NORM_SILU) || outer < 0 || inner < 1 || D < 1) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return KDA_ERR_INVALID_ARG;
  if (outer > 0 && (!x || !gate || !y)) return KDA_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(gate, 2) || !aligned(y, 2) || (weight && !aligned(weight, 4))) return KDA_ERR_INVALID_ARG;
  if (D > kAnyMaxD || (double)outer * (double)inner > 2147483647.0) return KDA_ERR_UNSUPPORTED;
  if (outer == 0) return KDA_OK;
  const int64_t contiguous[4] = {inner * D, D, inner * D, D};
  const int64_t *st = strides ? strides : contiguous;
  NormGateArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = static_cast<const __nv_bfloat16 *>(x);
  a.gate = static_cast<const __nv_bfloat16 *>(gate);
  a.weight = weight;
  a.y = static_cast<__nv_bfloat16 *>(y);
  a.rows = (int)(outer * inner);
  a.inner = (int)inner;
  a.xs[0] = st[0]; a.xs[1] = st[1];
  a.gs[0] = st[2]; a.gs[1] = st[3];
  a.D = D;
  a.eps = eps;
  a.silu = (flags & KDA_NORM_SILU) ? 1 : 0;
  const bool vec = D % 8 == 0 && D <= 16384 && all_multiples_of_8(st, 4) && aligned(x, 16) && aligned(gate, 16) &&
                   aligned(y, 16) && aligned(weight, 16);
  NvtxRange r("kda norm gate");
  return launch_norm_gate_rows(a, vec, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_add_norm(const void *x, const void *residual, const void *gate, const float *post_weight,
                          const float *weight, const float *scale_vec, float scale, float eps, int64_t rows, int D,
                          const int64_t *strides, uint32_t flags, void *y, void *h, kda_stream_t stream) {
  using namespace kda;
  if ((flags & ~KDA_NORM_RESIDUAL_F32) || rows < 0 || D < 1) return KDA_ERR_INVALID_ARG;
  const bool f32 = flags & KDA_NORM_RESIDUAL_F32;
  const size_t rsize = f32 ? 4 : 2;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !residual || !y || !h)) return KDA_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(gate, 2) || !aligned(y, 2) || !aligned(residual, rsize) || !aligned(h, rsize) ||
      !aligned(weight, 4) || !aligned(post_weight, 4) || !aligned(scale_vec, 4))
    return KDA_ERR_INVALID_ARG;
  if (D > kAnyMaxD || rows > 2147483647ll) return KDA_ERR_UNSUPPORTED;
  if (rows == 0) return KDA_OK;
  const int64_t contiguous[3] = {D, D, D};
  const int64_t *st = strides ? strides : contiguous;
  AddNormArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = static_cast<const __nv_bfloat16 *>(x);
  a.gate = static_cast<const __nv_bfloat16 *>(gate);
  a.residual = residual;
  a.weight = weight;
  a.post = post_weight;
  a.scale_vec = scale_vec;
  a.y = static_cast<__nv_bfloat16 *>(y);
  a.h = h;
  a.xs = st[0];
  a.rs = st[1];
  a.gs = gate ? st[2] : 0;
  a.scale = scale;
  a.eps = eps;
  a.D = D;
  const bool vec = D % 8 == 0 && D <= 16384 && all_multiples_of_8(st, gate ? 3 : 2) && aligned(x, 16) &&
                   aligned(gate, 16) && aligned(residual, 16) && aligned(y, 16) && aligned(h, 16) &&
                   aligned(weight, 16) && aligned(post_weight, 16) && aligned(scale_vec, 16);
  NvtxRange r("kda add norm");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return (f32 ? launch_add_norm_rows<float>(a, rows, vec, s) : launch_add_norm_rows<__nv_bfloat16>(a, rows, vec, s)) ==
                 cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

}  // extern "C"
