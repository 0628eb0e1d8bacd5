// Single-token recurrences over a pool of states (decoding): one token of the KDA recurrence, or
// of linear attention with one decay per head, for each of N requests.
//
// Per request n and head h, with the state S (K x V) of pool row state_indices[n]:
//   KDA:               s = Diag(alpha) S;  u = beta (v - s^T khat);  S' = s + khat u^T
//   linear attention:  S' = exp(a) S + k v^T
//   o = scale S'^T q   (KDA: qhat; alpha, khat, qhat and beta as in kda_fwd)
//
// For KDA the output needs no second pass over S': o = scale (s^T qhat + (qhat . khat) u), so both
// products s^T khat and s^T qhat are formed in one sweep and S' is written from registers.
//
// Bound: the state is read and written once, 128 KiB per request and head at K = V = 128 in fp32, against
// about 1 KiB of token data and 7 K V operations: memory bandwidth. A CTA of 128 threads takes a 16 KiB
// tile of one state (8 KiB of bf16 at K = 64). It issues the token's loads together with that of the row
// index, all loads of the tile as soon as the index is there, and only then computes anything: the gate,
// the norms and the block reduction run while the tile is in flight. Small batches (N H < SM count) still
// give V / 32 CTAs per fp32 state.
//
// Measured for 200 requests of 32 heads, K = V = 128, microseconds and the share of the copy bandwidth of
// 6.78 TB/s: fp32 KDA 124.8 (100%) and, [K, V] layout, 126.6 (99%), linear attention 124.0 (100%); bf16 KDA
// 70.0 (90%) and 78.1 (81%). With the token's loads after the tile's, fp32 [K, V] took 137 and four
// requests 7.2 us instead of 6.0. Where bf16 states leave bandwidth unused, it is the fixed work per CTA:
// 400 requests at K = V = 64 take 45.8 us (70%), and halving the tile at K = 128 made 90 us of 72.
#include <cmath>
#include <cstring>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_host.cuh"

namespace kda {

constexpr int kStepThreads = 128;
constexpr int kStepWarps = kStepThreads / 32;

struct StepArgs {
  const __nv_bfloat16 *q, *k, *v;
  const void *g;               // KDA: bf16 gate; linear attention: fp32 log decay per token, or per head
  const void *beta;            // KDA: logits, bf16 or fp32
  const float *A_log, *dt_bias;
  void *state;                 // [num_states, H, V, K] or [num_states, H, K, V]
  const int32_t *idx;          // [N] pool rows, or null: row n
  __nv_bfloat16 *o;            // [N, H, V]
  int *dev_status;
  long long num_states;
  long long qs[2], ks[2], vs[2], gs[2], bs[2];   // strides in elements: request, head
  float lb, scale;
  int N, H, group, V;          // group: value heads per query / key head
  uint32_t flags;
};

// 16 bytes of state, 4 fp32 or 8 bf16 values, as pairs for the packed fp32 instructions.
template <typename ST> struct StateVec;
template <> struct StateVec<float> {
  static constexpr int n = 4;
  __device__ static __forceinline__ void unpack(const uint4 &r, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    x[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  __device__ static __forceinline__ uint4 pack(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
  }
};
template <> struct StateVec<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static __forceinline__ void unpack(const uint4 &r, float2 (&x)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  // the one rounding of a bf16 state per token, to nearest even
  __device__ static __forceinline__ uint4 pack(const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int N>
__device__ __forceinline__ void load_shared(const float *src, float2 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 f = *reinterpret_cast<const float4 *>(src + 2 * i);
    x[i] = make_float2(f.x, f.y);
    x[i + 1] = make_float2(f.z, f.w);
  }
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// Tile of one CTA: R rows x CB columns of the stored matrix, CB along the contiguous dimension.
//   [V, K] layout: rows are value columns v, a row holds all K channels (CB = K);
//   [K, V] layout: rows are all K channels, CB value columns (128 bytes).
// 8 lanes cover 128 bytes of a row at a time, a warp 4 rows, the CTA 16 rows per pass. A bf16 row of KDA at
// K = 128 is covered by 16 lanes at once: 8 would hold the three factors of 16 channels each, which leaves
// registers for four CTAs per SM (72.6 us; 16 lanes and seven CTAs 69.5 us, 16 lanes and four 72.5).
template <bool KDA, int K, typename ST, bool KV>
struct StepTile {
  static constexpr int vec = StateVec<ST>::n;
  static constexpr int lanes = (KDA && !KV && K == 128 && vec == 8) ? 16 : 8;         // of a row
  static constexpr int span = lanes * vec;                               // values that they load at a time
  static constexpr int cols = KV ? span : K;
  static constexpr int per_row = cols / span;                            // 16-byte loads per lane and row
  static constexpr int rows = KV ? K : (per_row == 4 ? 32 : 64);
  static constexpr int pass_rows = kStepThreads / lanes;
  static constexpr int passes = rows / pass_rows;
  static constexpr int slice = KV ? cols : rows;                         // value columns per CTA
};

// CTAs per SM the registers are fitted to: six keep 96 KiB of loads in flight, as much as an fp32 state
// needs (124.4 us of 125.0). bf16 states have twice the values per byte to work on, and more or fewer CTAs
// pay, as long as nothing spills (microseconds at 200 requests of 32 heads, K = 64: 400, V = 64): linear
// attention at K = 64 ten, 35.5 (six 37.6, twelve 37.4); KDA at K = 64 six, 45.8 (five 49.1, seven 46.1),
// at K = 128 seven, 70.0 (six 70.7, eight 74.5), and in the [K, V] layout, where it spills from five on,
// four, 78.1 (five 81.2, seven 95.8).
template <bool KDA, int K, typename ST, bool KV>
constexpr int kStepCtas = sizeof(ST) == 4 ? 6 : KDA ? (K == 64 ? 6 : KV ? 4 : 7) : K == 64 ? 10 : 6;

template <bool KDA, int K, typename ST, bool KV>
__global__ void __launch_bounds__(kStepThreads, kStepCtas<KDA, K, ST, KV>) step_kernel(const StepArgs a) {
  using T = StepTile<KDA, K, ST, KV>;
  using Vec = StateVec<ST>;
  constexpr int kVec = T::vec;
  __shared__ __align__(16) float s_q[K], s_k[K], s_a[K], s_v[T::slice];
  __shared__ float s_part[3][kStepWarps];
  __shared__ __align__(16) float s_red[KV ? 2 : 1][KV ? kStepWarps : 1][T::slice];   // [K, V] layout: sums over the warps

  pdl_wait();   // launched to overlap the kernel ahead (see launch_step_t)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slices = a.V / T::slice;
  const int v0 = (int)(blockIdx.x % slices) * T::slice;
  const int nh = (int)(blockIdx.x / slices);
  const int n = nh / a.H, h = nh % a.H;
  __nv_bfloat16 *o = a.o + (long long)nh * a.V + v0;
  const long long row = a.idx ? (long long)a.idx[n] : (long long)n;

  // ---- token data, on its way while the row index is (and converted only later: a use would wait for it):
  // channel tid of q, k and the gate; value column tid of the slice
  __nv_bfloat16 q_raw = {}, k_raw = {}, v_raw = {}, g_raw = {}, beta_raw = {};
  float beta = 0.f, log_decay = 0.f, dt = 0.f, A_log = 0.f;
  if (tid < K) {
    const int hk = h / a.group;
    q_raw = a.q[n * a.qs[0] + hk * a.qs[1] + tid];
    k_raw = a.k[n * a.ks[0] + hk * a.ks[1] + tid];
    if constexpr (KDA) {
      const bool per_head = a.flags & kGatePerHead;
      g_raw = static_cast<const __nv_bfloat16 *>(a.g)[n * a.gs[0] + h * a.gs[1] + (per_head ? 0 : tid)];
      if (a.dt_bias) dt = a.dt_bias[per_head ? h : h * K + tid];
    }
  }
  if (tid < T::slice) v_raw = a.v[n * a.vs[0] + h * a.vs[1] + v0 + tid];
  if constexpr (KDA) {
    A_log = a.A_log[h];
    const long long bi = n * a.bs[0] + h * a.bs[1];
    if (a.flags & kBetaF32) beta = static_cast<const float *>(a.beta)[bi];
    else beta_raw = static_cast<const __nv_bfloat16 *>(a.beta)[bi];
  } else {
    log_decay = static_cast<const float *>(a.g)[(a.flags & kLaTokenDecay) ? n * a.gs[0] + h * a.gs[1] : h];
  }
  if (row < 0 || row >= a.num_states) {   // a padding entry, or an index outside the pool: no state is touched
    if (row >= a.num_states && tid == 0) atomicExch(a.dev_status, kDevBadStateIndex);
    if (tid < T::slice) o[tid] = __float2bfloat16_rn(0.f);
    return;
  }
  const int c = lane % T::lanes, r = tid / T::lanes;
  ST *tile = static_cast<ST *>(a.state) + (row * a.H + h) * (long long)K * a.V + (KV ? v0 : (long long)v0 * K);
  const long long ld = KV ? a.V : K;

  // ---- all of the tile's loads first
  uint4 raw[T::passes][T::per_row];
#pragma unroll
  for (int p = 0; p < T::passes; ++p)
#pragma unroll
    for (int j = 0; j < T::per_row; ++j)
      raw[p][j] = __ldcs(reinterpret_cast<const uint4 *>(tile + (p * T::pass_rows + r) * ld + j * T::span + c * kVec));

  float sums[3] = {0.f, 0.f, 0.f};   // |q|^2, |k|^2, q . k
  if (tid < K) {
    const float qv = __bfloat162float(q_raw), kv = __bfloat162float(k_raw);
    s_q[tid] = qv;
    s_k[tid] = kv;
    if constexpr (KDA) {
      s_a[tid] = ex2_approx(log2_decay(__bfloat162float(g_raw), dt, ex2_approx(A_log * kLog2e), a.lb * kLog2e));
      sums[0] = qv * qv;
      sums[1] = kv * kv;
      sums[2] = qv * kv;
    }
  }
  if (tid < T::slice) s_v[tid] = __bfloat162float(v_raw);
  const float decay = KDA ? 1.f : ex2_approx(log_decay * kLog2e);
  if constexpr (KDA) {
    beta = sigmoid_fast((a.flags & kBetaF32) ? beta : __bfloat162float(beta_raw));
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      sums[i] = warp_sum(sums[i]);
      if (lane == 0) s_part[i][warp] = sums[i];
    }
  }
  __syncthreads();
  float rq = 1.f, rk = 1.f, qk = 0.f;   // norm factors of q and k, and qhat . khat
  if constexpr (KDA) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      sums[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kStepWarps; ++w) sums[i] += s_part[i][w];
    }
    rq = rsqrtf(sums[0] + kNormEps);
    rk = rsqrtf(sums[1] + kNormEps);
    qk = sums[2] * rq * rk;
  }

  constexpr int kPairs = kVec / 2;
  if constexpr (!KV) {
    // Rows are value columns: the products over k are sums over a lane's values and 8 lanes. A
    // lane's channels are the same in every row, so their factors stay in registers: read per row,
    // they would take more shared-memory time than the state takes from memory.
    float2 kk[T::per_row][kPairs], qq[T::per_row][kPairs], aa[KDA ? T::per_row : 1][kPairs];
#pragma unroll
    for (int j = 0; j < T::per_row; ++j) {
      load_shared(s_k + j * T::span + c * kVec, kk[j]);
      load_shared(s_q + j * T::span + c * kVec, qq[j]);
      if constexpr (KDA) load_shared(s_a + j * T::span + c * kVec, aa[j]);
    }
#pragma unroll
    for (int p = 0; p < T::passes; ++p) {
      const int vi = p * T::pass_rows + r;
      const float vv = s_v[vi];
      float2 x[T::per_row][kPairs];
      float2 d1 = splat(0.f), d2 = splat(0.f);
#pragma unroll
      for (int j = 0; j < T::per_row; ++j) {
        Vec::unpack(raw[p][j], x[j]);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          if constexpr (KDA) {
            x[j][e] = __fmul2_rn(aa[j][e], x[j][e]);
            d1 = __ffma2_rn(kk[j][e], x[j][e], d1);
          } else {
            x[j][e] = __ffma2_rn(splat(decay), x[j][e], __fmul2_rn(kk[j][e], splat(vv)));
          }
          d2 = __ffma2_rn(qq[j][e], x[j][e], d2);
        }
      }
      float s1 = d1.x + d1.y, s2 = d2.x + d2.y;
#pragma unroll
      for (int m = 1; m < T::lanes; m <<= 1) {
        if constexpr (KDA) s1 += __shfl_xor_sync(0xffffffffu, s1, m);
        s2 += __shfl_xor_sync(0xffffffffu, s2, m);
      }
      if constexpr (KDA) {
        const float u = beta * (vv - rk * s1);
        s2 = fmaf(qk, u, rq * s2);
        const float2 ku = splat(rk * u);
#pragma unroll
        for (int j = 0; j < T::per_row; ++j)
#pragma unroll
          for (int e = 0; e < kPairs; ++e) x[j][e] = __ffma2_rn(ku, kk[j][e], x[j][e]);
      }
#pragma unroll
      for (int j = 0; j < T::per_row; ++j)
        __stcs(reinterpret_cast<uint4 *>(tile + vi * ld + j * T::span + c * kVec), Vec::pack(x[j]));
      if (c == 0) o[vi] = __float2bfloat16_rn(a.scale * s2);
    }
  } else {
    // Rows are channels k: the products over k are sums over a lane's rows, 4 lanes and the warps.
    float2 d1[kPairs], d2[kPairs], vv[kPairs];
    load_shared(s_v + c * kVec, vv);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) d1[e] = d2[e] = splat(0.f);
#pragma unroll
    for (int p = 0; p < T::passes; ++p) {
      const int k = p * T::pass_rows + r;
      const float2 kk = splat(s_k[k]), qq = splat(s_q[k]);
      float2 x[kPairs];
      Vec::unpack(raw[p][0], x);
      if constexpr (KDA) {
        const float2 aa = splat(s_a[k]);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const float2 t = __fmul2_rn(aa, x[e]);
          d1[e] = __ffma2_rn(kk, t, d1[e]);
          d2[e] = __ffma2_rn(qq, t, d2[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          x[e] = __ffma2_rn(splat(decay), x[e], __fmul2_rn(kk, vv[e]));
          d2[e] = __ffma2_rn(qq, x[e], d2[e]);
        }
        __stcs(reinterpret_cast<uint4 *>(tile + k * ld + c * kVec), Vec::pack(x));
      }
    }
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
#pragma unroll
      for (int m = 8; m < 32; m <<= 1) {
        if constexpr (KDA) {
          d1[e].x += __shfl_xor_sync(0xffffffffu, d1[e].x, m);
          d1[e].y += __shfl_xor_sync(0xffffffffu, d1[e].y, m);
        }
        d2[e].x += __shfl_xor_sync(0xffffffffu, d2[e].x, m);
        d2[e].y += __shfl_xor_sync(0xffffffffu, d2[e].y, m);
      }
      if (lane < 8) {
        *reinterpret_cast<float2 *>(&s_red[0][warp][c * kVec + 2 * e]) = d2[e];
        if constexpr (KDA) *reinterpret_cast<float2 *>(&s_red[1][warp][c * kVec + 2 * e]) = d1[e];
      }
    }
    __syncthreads();
    if constexpr (KDA) {
      float2 u[kPairs];   // rk u of this lane's columns
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        float2 t = splat(0.f);
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w)
          t = __fadd2_rn(t, *reinterpret_cast<const float2 *>(&s_red[1][w][c * kVec + 2 * e]));
        u[e] = __fmul2_rn(splat(beta * rk), __ffma2_rn(splat(-rk), t, vv[e]));
      }
#pragma unroll
      for (int p = 0; p < T::passes; ++p) {
        const int k = p * T::pass_rows + r;
        const float2 kk = splat(s_k[k]), aa = splat(s_a[k]);
        float2 x[kPairs];
        Vec::unpack(raw[p][0], x);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) x[e] = __ffma2_rn(kk, u[e], __fmul2_rn(aa, x[e]));
        __stcs(reinterpret_cast<uint4 *>(tile + k * ld + c * kVec), Vec::pack(x));
      }
    }
    if (tid < T::slice) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int w = 0; w < kStepWarps; ++w) {
        s2 += s_red[0][w][tid];
        if constexpr (KDA) s1 += s_red[1][w][tid];
      }
      if constexpr (KDA) s2 = fmaf(qk, beta * (s_v[tid] - rk * s1), rq * s2);
      o[tid] = __float2bfloat16_rn(a.scale * s2);
    }
  }
}

template <bool KDA, int K, typename ST, bool KV>
static cudaError_t launch_step_t(const StepArgs &a, cudaStream_t stream) {
  // The launch overlaps the end of the kernel ahead in the stream, whichever that is: in a graph of such calls
  // one request of 32 heads takes 1.6 us instead of 2.1 (linear attention), four take 3.3 instead of 3.8 (KDA).
  const long long grid = (long long)a.N * a.H * (a.V / StepTile<KDA, K, ST, KV>::slice);
  return launch_kernel(step_kernel<KDA, K, ST, KV>, dim3((unsigned)grid), dim3(kStepThreads), 0, stream, true, a);
}

template <bool KDA>
static cudaError_t launch_step(const StepArgs &a, int K, cudaStream_t stream) {
  const bool bf16 = a.flags & kStateBf16, kv = a.flags & kStateKV;
  if (K == 64) {
    if (bf16) return kv ? launch_step_t<KDA, 64, __nv_bfloat16, true>(a, stream) : launch_step_t<KDA, 64, __nv_bfloat16, false>(a, stream);
    return kv ? launch_step_t<KDA, 64, float, true>(a, stream) : launch_step_t<KDA, 64, float, false>(a, stream);
  }
  if (bf16) return kv ? launch_step_t<KDA, 128, __nv_bfloat16, true>(a, stream) : launch_step_t<KDA, 128, __nv_bfloat16, false>(a, stream);
  return kv ? launch_step_t<KDA, 128, float, true>(a, stream) : launch_step_t<KDA, 128, float, false>(a, stream);
}

// Checks and fields that both recurrences share.
static kda_status_t fill_step(StepArgs &a, const void *q, const void *k, const void *v, const void *g, float scale,
                              void *state, const int32_t *idx, int N, int Hk, int H, int K, int V,
                              long long num_states, const kda_step_strides_t *st, uint32_t flags, void *o,
                              bool gate_per_channel) {
  if (N < 0 || H < 1 || Hk < 1 || K < 1 || V < 1 || num_states < 0 || H % Hk != 0) return KDA_ERR_INVALID_ARG;
  if ((N > 0 && (!q || !k || !v || !g || !o)) || (num_states > 0 && !state)) return KDA_ERR_INVALID_ARG;
  if ((K != 64 && K != 128) || (V != 64 && V != 128)) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (!idx && num_states < N) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(o, 2) || !aligned(state, 16) ||
      (idx && !aligned(idx, 4)))
    return KDA_ERR_INVALID_ARG;
  if ((double)N * H * (V / 32) > 2147483647.0 || (double)num_states * H * K * V > 9.0e15) return KDA_ERR_UNSUPPORTED;
  std::memset(&a, 0, sizeof a);
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.g = g;
  a.scale = scale;
  a.state = state;
  a.idx = idx;
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.num_states = num_states;
  a.N = N;
  a.H = H;
  a.group = H / Hk;
  a.V = V;
  a.flags = flags;
  auto set = [&](long long (&dst)[2], const int64_t *src, long long request, long long head) {
    dst[0] = src ? src[0] : request;
    dst[1] = src ? src[1] : head;
  };
  const long long gw = gate_per_channel ? K : 1;
  set(a.qs, st ? st->q : nullptr, (long long)Hk * K, K);
  set(a.ks, st ? st->k : nullptr, (long long)Hk * K, K);
  set(a.vs, st ? st->v : nullptr, (long long)H * V, V);
  set(a.gs, st ? st->g : nullptr, (long long)H * gw, gw);
  set(a.bs, st ? st->beta : nullptr, H, 1);
  return KDA_OK;
}

static kda_status_t run_step(bool is_kda, StepArgs &a, int K, kda_stream_t stream) {
  if (a.N == 0) return KDA_OK;
  a.dev_status = device_status_address();
  if (!a.dev_status) return KDA_ERR_CUDA;
  NvtxRange r(is_kda ? "kda step" : "kda la step");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return (is_kda ? launch_step<true>(a, K, s) : launch_step<false>(a, K, s)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda

extern "C" {

kda_status_t kda_step(const void *q, const void *k, const void *v, const void *g, const void *beta,
                      const float *A_log, const float *dt_bias, float lower_bound, float scale, void *state,
                      const int32_t *state_indices, int N, int H, int K, int V, int64_t num_states,
                      const kda_step_strides_t *strides, uint32_t flags, void *o, kda_stream_t stream) {
  using namespace kda;
  if (flags & ~(kGatePerHead | kBetaF32 | kStateBf16 | kStateKV)) return KDA_ERR_INVALID_ARG;
  const bool per_head = flags & kGatePerHead;
  StepArgs a;
  const kda_status_t st = fill_step(a, q, k, v, g, scale, state, state_indices, N, H, H, K, V, num_states, strides,
                                    flags, o, !per_head);
  if (st != KDA_OK) return st;
  if (!A_log || (N > 0 && !beta)) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(lower_bound) || lower_bound < -5.0f || lower_bound > 0.0f) return KDA_ERR_INVALID_ARG;
  if (!aligned(g, 2) || !aligned(beta, (flags & kBetaF32) ? 4 : 2) || !aligned(A_log, 4) ||
      (dt_bias && !aligned(dt_bias, 4)))
    return KDA_ERR_INVALID_ARG;
  a.beta = beta;
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.lb = lower_bound;
  return run_step(true, a, K, stream);
}

kda_status_t kda_la_step(const void *q, const void *k, const void *v, const float *log_decay, float scale,
                         void *state, const int32_t *state_indices, int N, int Hk, int H, int K, int V,
                         int64_t num_states, const kda_step_strides_t *strides, uint32_t flags, void *o,
                         kda_stream_t stream) {
  using namespace kda;
  if (flags & ~(kLaTokenDecay | kStateBf16 | kStateKV)) return KDA_ERR_INVALID_ARG;
  StepArgs a;
  const kda_status_t st = fill_step(a, q, k, v, log_decay, scale, state, state_indices, N, Hk, H, K, V, num_states,
                                    strides, flags, o, false);
  if (st != KDA_OK) return st;
  if (!aligned(log_decay, 4)) return KDA_ERR_INVALID_ARG;
  return run_step(false, a, K, stream);
}

}  // extern "C"
