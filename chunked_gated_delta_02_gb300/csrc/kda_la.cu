// Linear attention with one decay per head, chunked form, on the 5th-generation tensor cores
// (tcgen05, accumulators in tensor memory).
//
// Per sequence and head, for tokens t in order (S is K x V, a_t <= 0 the log decay):
//   S_t = exp(a_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// With chunks of C = 128 tokens and G_i the sum of the log decays of the chunk up to token i:
//   o_i = scale (sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j + exp(G_i) S^T q_i)
//   S   = exp(G_C) S + sum_j exp(G_C - G_j) k_j v_j^T
// as four products per chunk:
//   M1: scores = Q K^T               C x C,  both operands in shared memory
//   M2: O      = Q S                 C x V,  S in bf16
//   M3: O     += P V                 C x V,  P the masked scores times exp(G_i - G_j - R_i), in bf16
//   M4: D^T    = V'^T K              V x K,  V' = v_j exp(G_C - G_j) as a sum of three bf16 terms
//   o_i = scale exp(R_i) O_i,  S^T = exp(G_C) S^T + D^T in fp32, in registers for the whole sequence
//
// R_i = max(G_i, -64 ln 2) takes the row's decay out of P, so that M2 and M3 can add into one
// accumulator and an element of P costs one factor of its column, exp(-G_j). Where the decay of a
// chunk goes below 2^-64, G_i - G_j - R_i stays within (-inf, 64 ln 2] and is formed pairwise; rows
// that far down take 2^-64 Q S instead of less, which is below the rounding of anything else. Positive
// log decays may lead back up: with m_i the least G_j of j <= i, G_i - G_j - R_i would reach -m_i where
// G_i > -64 ln 2, and R_i is raised to G_i - m_i - 96 ln 2. Such rows take exp(G_i - m_i) 2^-96 Q S, at
// most 2^-32 Q S for growths up to 2^64, where token argmin m counts 2^96 times as much.
//
// What is rounded: q, k and v are exact (bf16 inputs). P and the copy of S that M2 reads are bf16,
// like the output they go to: each adds about as much error as the rounding of o itself. The state
// is fp32 and has to stay fp32-accurate over a whole sequence, so its only rounded operand, V', is
// split into three bf16 terms, which hold all 24 bits: with two the state's error against fp64 was
// 2.7e-6, more than ten times that of fp32 arithmetic.
//
// A CTA takes (sequence segment, head) items, all V columns at once, so that q, k and v are read
// once; it is persistent over items (one CTA per SM: two stages of q, k and v and S fill the
// shared memory). Warp roles, coupled by mbarriers only:
//   warps 0-3    P, in place of the scores in tensor memory (A operand of M3)
//   warps 4-7    V', transposed from the v tile into tensor memory (A operand of M4), 32 tokens at
//                a time into two buffers in turn
//   warps 8-15   the state, and the scaled output in bf16
//   warp 16      loads (TMA, 128-byte swizzle) and the chunk's decay factors
//   warp 17      issues M1, M2 and M3;  warp 18  issues M4
//   warp 19      stores the output tile, which the state warps leave in the chunk's v buffer
// V' as the tensor-memory operand makes D^T come out with one value column per lane, the layout in
// which a thread can update its part of S^T and write it as rows of M2's operand without transposing.
//
// Bound: a chunk of one head moves 128 KiB at K = V = 128, 2.9 us of an SM's share of the measured
// bandwidth, against 48 tensor-core steps of 64 clocks, 1.6 us: memory bandwidth, where every SM has work.
// Measured: 4 x 4096 tokens of 64 heads 188 us, 5.7 TB/s, 85% of the copy bandwidth. Alone on its SM a
// chunk takes 2.75 us, whatever the other SMs do, and few sequences and heads are bound by that: scores ->
// P -> O -> next scores and D -> S -> O -> next D are two loops of about 5200 clocks, of which the products
// take 3100. What keeps them short: V' and P in separate warps; q, k and v released on their own; a state's
// update or a chunk's output, whichever product is done first; o stored by the copy engine (by the state
// warps it took 1400 clocks of their time from shared memory and 2700 from registers).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/kda.h"
#include "kda_host.cuh"
#include "kda_la.cuh"
#include "umma.cuh"

namespace kda {

constexpr int kLaThreads = 640;
// Registers per thread by warpgroup; a block is launched with 96 for each of its threads, and the
// state warps' increase is what the others give back: 2 x 32 = 8 + 8 + 48.
constexpr int kLaRegsOperands = 88, kLaRegsState = 128, kLaRegsIssue = 48;
static_assert(2 * kLaRegsOperands + 2 * kLaRegsState + kLaRegsIssue <= 5 * 96, "registers at launch");
constexpr uint32_t kLaTmemCols = 512;
constexpr unsigned kLaWaitLimit = 4000000000u;   // ~2 s of SM clocks per wait
// The smallest log2 decay of a token: 2^-126 is the smallest normal fp32 number, so that a decay of
// zero (log decay -inf) drops the state without an inf - inf in the sums.
constexpr float kLaMinLog2 = -126.0f;
// Row decays below 2^-64 stay in P (see above): 2^64 leaves the scores and values as much range again.
constexpr float kLaRowLog2 = -64.0f;
constexpr float kLaMostLog2 = 96.0f;   // the largest G_i - G_j - R_i

// Decay factors of one chunk.
struct LaGate {
  // G_i, the log2 decay from the chunk's start through token i; in a weak chunk, whose decay stays
  // above 2^-64, the factor 2^-G_i itself
  float G[kLaChunk];
  float cf[kLaChunk];   // decay from token j to the end of its 32-token block; 0 past the sequence
  float bf[4];          // decay from the end of 32-token block c to the chunk's end
  float gamma;          // decay of the whole chunk
  int weak;             // 1: weak; 0: not; -1: not, and some token's log decay is positive
  float pad[2];
};

// G_i - R_i of a chunk that is not weak.
__device__ __forceinline__ float la_row_shift(const LaGate &g, int row, int weak) {
  float x = fminf(g.G[row] - kLaRowLog2, 0.f);
  if (weak < 0) {
    float least = 0.f;
#pragma unroll 1
    for (int j = 0; j <= row; ++j) least = fminf(least, g.G[j]);
    x = fminf(x, least + kLaMostLog2);
  }
  return x;
}

struct LaMisc {
  // per stage: q and k loaded, consumed; v loaded, consumed; decay factors written (consumed with q and
  // k); v rows past the sequence cleared; V' formed; output tile written over v
  uint64_t full[3], empty[3], full_v[3], empty_v[3], gate[3], v_rdy[3], v_read[3], o_st[3];
  uint64_t p_raw, p_rdy, s_free, o_done, o_free, s_rdy;   // one phase per chunk
  uint64_t vp_rdy[4], vp_free[4];                   // per V' buffer: 32 tokens ready, read
  uint64_t d_rdy[2], d_free[2];                     // per D buffer: ready, read
  uint64_t state_sync;                              // the state warps among themselves
  uint64_t bar_exit;
  uint32_t tmem_slot;
  int err;
  // this CTA's place among the others; its one item past the whole rounds, if it has one; the first chunk of
  // item cta - 1, and the end of item cta, that it does
  int cta, extra, cut0, cut1;
};

template <int K, int V, bool AGG>
struct LaLayout {
  static constexpr uint32_t panel = kLaChunk * 128;   // 128 tokens x 64 columns
  static constexpr uint32_t k_off = AGG ? 0 : (K / 64) * panel;
  static constexpr uint32_t v_off = k_off + (K / 64) * panel;
  static constexpr uint32_t stage = v_off + (V / 64) * panel;
  static constexpr int stages = (AGG || K + V == 128) ? 3 : 2;
  static constexpr uint32_t s_off = stages * stage;                 // S^T rows v, bf16, K-major panels
  static constexpr uint32_t s_panel = V * 128;
  static constexpr uint32_t gate = s_off + (AGG ? 0 : (K / 64) * s_panel);
  static constexpr uint32_t misc = gate + stages * (uint32_t)sizeof(LaGate);
  static constexpr uint32_t bytes = misc + (uint32_t)sizeof(LaMisc);
  static_assert(bytes <= 232448, "shared memory of one CTA");
};

// Tensor memory columns.
constexpr uint32_t kTmP = 0;      // scores, 128 fp32; P takes the first 64 (bf16 pairs)
constexpr uint32_t kTmVp = 128;   // V'^T: two buffers of 32 tokens, three terms of 16 columns each
constexpr uint32_t kTmVpBuf = 48;
constexpr uint32_t kTmO = 256;    // O, V columns
constexpr uint32_t kTmD = 384;    // D^T, K columns
// Without scores and O, V' has a buffer for every 32 tokens of a chunk, and D^T two.
constexpr uint32_t kTmVpAgg = 0, kTmDAgg = 256;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&x);
}

__device__ __forceinline__ LaItem la_item(const LaProblem &p, int idx) {
  LaItem it;
  if (p.cu) {
    it = p.items[idx];
  } else {
    const int s = idx / p.n_seg, g = idx % p.n_seg;
    it.seq = s;
    it.b = s;
    it.t0 = g * p.seg_chunks * kLaChunk;
    it.len = max(0, min(p.T - it.t0, p.seg_chunks * kLaChunk));
    it.slot = idx;
    it.seg = g;
    it.n_seg = p.n_seg;
    it.part = 0;
  }
  return it;
}

// S^T rows v0 + lane of (sequence s, head h), columns [k0, k0 + N), between a warp's registers and the
// caller's state in any type and layout, by way of `buf`: 32 rows of K / 4 fp32 values of shared memory
// that the warp has to itself. From there every access covers whole 64- or 128-byte pieces of memory,
// and only one loop, not one per register and variant, has the memory side's code.
template <int K, int V, int N, bool STORE>
__device__ __forceinline__ void la_state_move(const LaProblem &p, int s, int h, int v0, int k0, float (&S)[N],
                                              float *buf) {
  constexpr int kCols = K / 4, kChunks = kCols / 4;   // 16-byte chunk c of row r lies at chunk c ^ (r % kChunks)
  const int lane = threadIdx.x & 31;
  const long long base = ((long long)s * p.H + h) * K * V;
  const bool bf16 = p.flags & kStateBf16, kv = p.flags & kStateKV;
  float4 *mine = reinterpret_cast<float4 *>(buf) + lane * kChunks;
#pragma unroll
  for (int r = 0; r < N; r += kCols) {
    if (STORE) {
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        mine[j ^ (lane & (kChunks - 1))] = make_float4(S[r + 4 * j], S[r + 4 * j + 1], S[r + 4 * j + 2], S[r + 4 * j + 3]);
      __syncwarp();
    }
    // Step i moves four consecutive values per lane: columns of a row, or rows of a column ([K, V] layout).
#pragma unroll (STORE ? 2 : 8)
    for (int i = 0; i < kChunks; ++i) {
      const int row = kv ? 4 * (lane & 7) : (i * 32 + lane) / kChunks;
      const int col = kv ? 4 * i + (lane >> 3) : 4 * (lane % kChunks);
      const int at = row * kCols + (((col >> 2) ^ (row & (kChunks - 1))) << 2) + (col & 3);
      // the places of four rows of one column
      const int at1 = (row + 1) * kCols + (((col >> 2) ^ ((row + 1) & (kChunks - 1))) << 2) + (col & 3);
      const int at2 = (row + 2) * kCols + (((col >> 2) ^ ((row + 2) & (kChunks - 1))) << 2) + (col & 3);
      const int at3 = (row + 3) * kCols + (((col >> 2) ^ ((row + 3) & (kChunks - 1))) << 2) + (col & 3);
      const long long g = base + (kv ? (k0 + r + col) * V + v0 + row : (v0 + row) * K + k0 + r + col);
      if (STORE) {
        const float4 f = kv ? make_float4(buf[at], buf[at1], buf[at2], buf[at3]) : *reinterpret_cast<const float4 *>(buf + at);
        if (bf16) *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.final_state) + g) = make_uint2(pack_bf16(f.x, f.y), pack_bf16(f.z, f.w));
        else *reinterpret_cast<float4 *>(static_cast<float *>(p.final_state) + g) = f;
      } else {
        float4 f;
        if (bf16) {
          const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.init) + g);
          f = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                          __uint_as_float(u.y & 0xFFFF0000u));
        } else {
          f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.init) + g);
        }
        if (kv) {
          buf[at] = f.x; buf[at1] = f.y; buf[at2] = f.z; buf[at3] = f.w;
        } else {
          *reinterpret_cast<float4 *>(buf + at) = f;
        }
      }
    }
    __syncwarp();
    if (!STORE) {
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const float4 f = mine[j ^ (lane & (kChunks - 1))];
        S[r + 4 * j] = f.x; S[r + 4 * j + 1] = f.y; S[r + 4 * j + 2] = f.z; S[r + 4 * j + 3] = f.w;
      }
      __syncwarp();
    }
  }
}

// Segment states: float4 j of thread (half, v) at [j][half V + v], so that warps read and write
// 512 contiguous bytes. Column k = half K / 2 + 4 j + e.
template <int K, int V>
__device__ __forceinline__ long long la_seg_index(int half, int v, int j) {
  return ((long long)j * (2 * V) + half * V + v) * 4;
}

// AGG: only the state that each segment adds, started from zero (segments before the last of their
// sequence). Otherwise everything, from the segment's start state. SHARE: CTAs share items (below); a
// kernel of its own, because in the one for short items what it adds cost 1 us per item.
template <int K, int V, bool AGG, bool SHARE>
__global__ void __launch_bounds__(kLaThreads, 1)
la_kernel(const LaProblem p, const __grid_constant__ LaMaps maps) {
  using Lay = LaLayout<K, V, AGG>;
  constexpr int kStages = Lay::stages;
  extern __shared__ __align__(1024) unsigned char sm[];
  LaMisc &ms = *reinterpret_cast<LaMisc *>(sm + Lay::misc);
  LaGate *gates = reinterpret_cast<LaGate *>(sm + Lay::gate);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sbase = umma::smem_u32(sm);
  pdl_wait();   // the schedule, the segment states, or whatever kernel is ahead: every launch overlaps its end
  if (p.flag && *p.flag != kDevOk) return;
  if (sbase & 1023u) {   // the operand layouts need it; never the case for a kernel without static shared memory
    if (tid == 0) atomicExch(p.dev_status, kDevWaitTimeout);
    return;
  }
  const int total = (p.cu ? p.counts[AGG ? 1 : 0] : p.N * p.n_seg) * p.H;   // below 2^31 (kda_la_fwd)
  if (total == 0) return;

  // With R whole rounds of G CTAs and x more items, a CTA's even share is R + x / G items. CTA
  // c begins with the first chunks of item c, goes on with items c + G, c + 2 G, ..., one of the x more where
  // c x / G passes a whole number, and ends with the chunks of item c - 1 that CTA c - 1 left: where that one
  // stopped makes all shares even. A state is thus handed over long after it was formed, and only by a CTA
  // that started earlier: places are given in the order of starts.
  if (SHARE && tid == 32) {
    const int cta = atomicAdd(p.started, 1), G = gridDim.x, x = total % G;
    const int e0 = (cta * x + G - 1) / G, e1 = ((cta + 1) * x + G - 1) / G;   // of the x, before and through this CTA
    int cut[2];
    for (int i = 0; i < 2; ++i) {
      const int n = p.seg_chunks, left = (int)((long long)n * ((i ? e1 : e0) * G - (cta + i) * x) / G);
      cut[i] = left < 2 ? n : n - left < 2 ? 0 : n - left;   // (handing over costs about a chunk's time)
    }
    ms.cta = cta;
    ms.extra = e1 > e0 ? total - x + e0 : -1;
    ms.cut0 = cut[0];
    ms.cut1 = cut[1];
  }
  if (warp == 0) {
    umma::tmem_alloc(&ms.tmem_slot, kLaTmemCols);
    umma::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      umma::mbar_init(&ms.full[s], 1);
      umma::mbar_init(&ms.full_v[s], 1);
      umma::mbar_init(&ms.gate[s], 1);
      umma::mbar_init(&ms.v_rdy[s], 4);
      umma::mbar_init(&ms.empty[s], AGG ? 1 + 8 : 2 + 4 + 8);   // M4, M2, P and state warps
      umma::mbar_init(&ms.empty_v[s], AGG ? 8 : 1);             // V' warps; the output's store
      umma::mbar_init(&ms.v_read[s], 4);
      umma::mbar_init(&ms.o_st[s], 8);
    }
    for (int b = 0; b < 4; ++b) {
      umma::mbar_init(&ms.vp_rdy[b], 4);
      umma::mbar_init(&ms.vp_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      umma::mbar_init(&ms.d_rdy[b], 1);
      umma::mbar_init(&ms.d_free[b], 8);
    }
    umma::mbar_init(&ms.p_raw, 1);
    umma::mbar_init(&ms.p_rdy, 4);
    umma::mbar_init(&ms.s_free, 1);
    umma::mbar_init(&ms.o_done, 1);
    umma::mbar_init(&ms.o_free, 8);
    umma::mbar_init(&ms.state_sync, 8);
    umma::mbar_init(&ms.s_rdy, 8);
    umma::mbar_init(&ms.bar_exit, 2);
    umma::mbar_fence_init();
    ms.err = 0;
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = ms.tmem_slot;
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const int row = (warp & 3) * 32 + lane;   // this thread's tensor memory lane

  // Bounded wait of one thread; it ends early once any wait of the CTA has given up.
  auto wait1 = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (umma::mbar_try_wait(bar, parity)) return true;
    const unsigned t0 = (unsigned)clock();
    while (!umma::mbar_try_wait(bar, parity)) {
      if (*(volatile int *)&ms.err) return false;
      if ((unsigned)clock() - t0 > kLaWaitLimit) {
        *(volatile int *)&ms.err = 1;
        return false;
      }
    }
    return true;
  };
  // The same for a whole warp, with one answer.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    const bool ok = __all_sync(0xffffffffu, wait1(bar, parity));
    umma::fence_after_sync();
    return ok;
  };
  // One arrival for the warp after its tensor memory or shared memory accesses.
  auto arrive = [&](uint64_t *bar) {
    umma::fence_before_sync();
    __syncwarp();
    if (lane == 0) umma::mbar_arrive(bar);
  };
  // f(item, head, n): every chunk of this CTA's items, n counting them over all items; begin(item,
  // head, chunks) and end(item, head, chunks) around them. All stop at the first false.
  auto for_chunks = [&](auto &&begin, auto &&chunk, auto &&end) {
    // Rounds of one item per CTA: neighbouring heads at the same time, whose tokens are neighbours in memory.
    // Where none are shared, the items come longest first, and every other round goes backwards, to even
    // out what the CTAs get.
    int n = 0;
    const int ctas = gridDim.x, cta = SHARE ? ms.cta : (int)blockIdx.x, rounds = total / ctas;
    for (int i = 0; i <= rounds + SHARE; ++i) {
      int w = i * ctas + ((i & 1) && !SHARE ? ctas - 1 - cta : cta);
      if (SHARE && i >= rounds) w = i == rounds ? ms.extra : cta - 1;
      if (w < 0 || w >= total) continue;
      LaItem it = la_item(p, w / p.H);
      const int h = w % p.H;
      if (AGG && it.seg == it.n_seg - 1) continue;
      if constexpr (SHARE) {
        if (i == 0 && it.len > ms.cut1 * kLaChunk) {
          it.len = ms.cut1 * kLaChunk;
          it.part = kLaToOther;
        }
        if (i > rounds) {
          const int done = ms.cut0 * kLaChunk;
          it.t0 += done;
          it.len -= done;
          it.part = done ? kLaFromOther : 0;
        }
        if (it.len <= 0) continue;
      }
      const int nch = (it.len + kLaChunk - 1) / kLaChunk;
      if (!begin(it, h, nch)) return;
      for (int c = 0; c < nch; ++c, ++n)
        if (!chunk(it, h, c, nch, n)) return;
      if (!end(it, h, nch)) return;
    }
  };
  auto nothing = [](const LaItem &, int, int) { return true; };

  if (warp >= 16) umma::regs_dec<kLaRegsIssue>();
  if (warp == 16) {
    // ======================= loads and decay factors =======================
    const int hq_group = p.H / p.Hk;
    const bool per_token = p.flags & kLaTokenDecay;
    int issued = 0, issued_v = 0;
    // Lane l: tokens 4 l .. 4 l + 3; lanes 8 c .. 8 c + 7 are 32-token block c. The decays of a chunk are
    // loaded while the one before is in use. A full chunk's factors of a head without decays per token are
    // those of any other: they stay in their stage (held: that head, by stage).
    float next[4] = {0.f, 0.f, 0.f, 0.f};
    int held[3] = {-1, -1, -1};
    const char *init = static_cast<const char *>(p.init);
    const int state_bytes = K * V * ((p.flags & kStateBf16) ? 2 : 4);
    auto load_decays = [&](const LaItem &it, int h, int c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = c * kLaChunk + 4 * lane + e;
        if (i < it.len)
          next[e] = per_token ? p.decay[it.b * p.ds[0] + (long long)(it.t0 + i) * p.ds[1] + h * p.ds[2]] : p.decay[h];
      }
    };
    for_chunks([&](const LaItem &it, int h, int nch) {
      if (nch > 0) load_decays(it, h, 0);
      // The state that the state warps need when they get to this item, some chunks from now. (64 x 512 tokens of
      // 64 heads, without and with: fp32 states 486 and 480 us, bf16 502 and 485, bf16 [K, V] 587 and 500.)
      if (!AGG && init && it.n_seg == 1 && umma::elect_one())
        umma::prefetch_l2_bulk(init + (long long)(it.seq * p.H + h) * state_bytes, state_bytes);
      return true;
    }, [&](const LaItem &it, int h, int c, int nch, int n) {
      const int st = n % kStages;
      const uint32_t ph = (uint32_t)((n / kStages) & 1);
      if (n >= kStages && !wait(&ms.empty[st], ph ^ 1u)) return false;
      const int t0 = it.t0 + c * kLaChunk, L = min(kLaChunk, it.len - c * kLaChunk);
      if (umma::elect_one()) {
        unsigned char *dst = sm + st * Lay::stage;
        umma::mbar_arrive_expect_tx(&ms.full[st], Lay::v_off);
        const int hq = h / hq_group;
        if constexpr (!AGG)
          for (int x = 0; x < K / 64; ++x) umma::tma_load_4d(dst + x * Lay::panel, &maps.q, x * 64, hq, t0, it.b, &ms.full[st]);
        for (int x = 0; x < K / 64; ++x) umma::tma_load_4d(dst + Lay::k_off + x * Lay::panel, &maps.k, x * 64, hq, t0, it.b, &ms.full[st]);
      }
      issued = n + 1;
      if (n >= kStages && !wait(&ms.empty_v[st], ph ^ 1u)) return false;
      if (umma::elect_one()) {
        umma::mbar_arrive_expect_tx(&ms.full_v[st], Lay::stage - Lay::v_off);
        for (int x = 0; x < V / 64; ++x)
          umma::tma_load_4d(sm + st * Lay::stage + Lay::v_off + x * Lay::panel, &maps.v, x * 64, h, t0, it.b, &ms.full_v[st]);
      }
      issued_v = n + 1;
      const int here = st == 0 ? held[0] : st == 1 ? held[1] : held[2];
      if (per_token || L < kLaChunk || here != h) {
        float a[4], pre[4], suf[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = next[e] * kLog2e;
          a[e] = 4 * lane + e >= L ? 0.f : x < kLaMinLog2 ? kLaMinLog2 : x;   // NaN stays
        }
        if (c + 1 < nch) load_decays(it, h, c + 1);
        pre[0] = a[0];
        suf[3] = 0.f;
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          pre[e] = pre[e - 1] + a[e];
          suf[3 - e] = suf[4 - e] + a[4 - e];
        }
        float incl = pre[3];   // sums through this lane
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const float y = __shfl_up_sync(0xffffffffu, incl, m);
          if (lane >= m) incl += y;
        }
        float before = __shfl_up_sync(0xffffffffu, incl, 1);
        if (lane == 0) before = 0.f;
        // sums over the later lanes of the block, formed from the block's end so that small sums
        // near the end keep their precision
        float after = pre[3];
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, after, m);
          if ((lane & 7) + m < 8) after += y;
        }
        const float block = __shfl_sync(0xffffffffu, after, lane & 24);   // the block's total
        const float later = __shfl_down_sync(0xffffffffu, after, 1);
        const float tail = (lane & 7) == 7 ? 0.f : later;
        LaGate &g = gates[st];
        // The least of the sums is the last one, unless a log decay is positive.
        float least = __shfl_sync(0xffffffffu, incl, 31);
        const bool rises = __any_sync(0xffffffffu, fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) > 0.f);
        if (rises) {
          least = before + fminf(fminf(pre[0], pre[1]), fminf(pre[2], pre[3]));
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, m));
        }
        const bool weak = least >= kLaRowLog2;
        float G[4], cf[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          G[e] = weak ? ex2_approx(-(before + pre[e])) : before + pre[e];
          cf[e] = 4 * lane + e < L ? ex2_approx(suf[e] + tail) : 0.f;
        }
        *reinterpret_cast<float4 *>(&g.G[4 * lane]) = make_float4(G[0], G[1], G[2], G[3]);
        *reinterpret_cast<float4 *>(&g.cf[4 * lane]) = make_float4(cf[0], cf[1], cf[2], cf[3]);
        const float b1 = __shfl_sync(0xffffffffu, block, 8), b2 = __shfl_sync(0xffffffffu, block, 16),
                    b3 = __shfl_sync(0xffffffffu, block, 24), b0 = __shfl_sync(0xffffffffu, block, 0);
        if (lane == 0) {
          g.bf[0] = ex2_approx(b1 + b2 + b3);
          g.bf[1] = ex2_approx(b2 + b3);
          g.bf[2] = ex2_approx(b3);
          g.bf[3] = 1.f;
          g.gamma = ex2_approx(b0 + b1 + b2 + b3);
          g.weak = weak ? 1 : rises ? -1 : 0;
        }
        __syncwarp();
        const int keep = per_token || L < kLaChunk ? -1 : h;
        if (st == 0) held[0] = keep;
        else if (st == 1) held[1] = keep;
        else held[2] = keep;
      }
      if (lane == 0) umma::mbar_arrive(&ms.gate[st]);
      return true;
    }, nothing);
    // after a timeout: wait (bounded) for the copies in flight
    if (lane == 0 && *(volatile int *)&ms.err) {
      for (int n = max(0, issued - kStages); n < issued; ++n)
        umma::mbar_wait_bounded(&ms.full[n % kStages], (uint32_t)((n / kStages) & 1), kLaWaitLimit);
      for (int n = max(0, issued_v - kStages); n < issued_v; ++n)
        umma::mbar_wait_bounded(&ms.full_v[n % kStages], (uint32_t)((n / kStages) & 1), kLaWaitLimit);
    }
  } else if (warp == 17) {
    // ======================= M1, M2, M3 =======================
    if constexpr (!AGG) {
      constexpr uint32_t id1 = umma::idesc_bf16(128, 128, 0, 0), id2 = umma::idesc_bf16(128, V, 0, 0);
      constexpr uint32_t id3 = umma::idesc_bf16(128, V, 0, 1);
      const uint64_t bs = umma::sdesc_sw128(sbase + Lay::s_off, 16, 1024);
      for_chunks(nothing, [&](const LaItem &, int, int, int, int n) {
        const int st = n % kStages;
        const uint32_t ph = (uint32_t)(n & 1), sph = (uint32_t)((n / kStages) & 1), q0 = sbase + st * Lay::stage;
        const uint64_t aq = umma::sdesc_sw128(q0, 16, 1024), bk = umma::sdesc_sw128(q0 + Lay::k_off, 16, 1024);
        const uint64_t bv = umma::sdesc_sw128(q0 + Lay::v_off, Lay::panel, 1024);
        if (!wait(&ms.full[st], sph)) return false;
        // M1: scores = Q K^T (the scores of the chunk before were last read by its M3, ahead of this in order)
        if (umma::elect_one()) {
#pragma unroll 1
          for (int x = 0; x < K / 64; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              umma::mma_f16_ss(tmem + kTmP, umma::desc_add(aq, x * Lay::panel + y * 32),
                               umma::desc_add(bk, x * Lay::panel + y * 32), id1, x + y > 0);
          umma::commit(&ms.p_raw);
        }
        // M2: O = Q S
        if (!wait(&ms.s_rdy, ph)) return false;
        if (n > 0 && !wait(&ms.o_free, ph ^ 1u)) return false;
        if (umma::elect_one()) {
#pragma unroll 1
          for (int x = 0; x < K / 64; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              umma::mma_f16_ss(tmem + kTmO, umma::desc_add(aq, x * Lay::panel + y * 32),
                               umma::desc_add(bs, x * Lay::s_panel + y * 32), id2, x + y > 0);
          umma::commit(&ms.s_free);
          umma::commit(&ms.empty[st]);
        }
        // M3: O += P V; v_rdy: rows of the v tile past the sequence have been cleared
        if (!wait(&ms.v_rdy[st], sph) || !wait(&ms.p_rdy, ph)) return false;
        if (umma::elect_one()) {
#pragma unroll 1
          for (int x = 0; x < 8; x += 4)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              umma::mma_f16_ts(tmem + kTmO, tmem + kTmP + (x + y) * 8, umma::desc_add(bv, (x + y) * 2048), id3, 1);
          umma::commit(&ms.o_done);
        }
        __syncwarp();
        return true;
      }, nothing);
    }
    if (umma::elect_one()) umma::commit(&ms.bar_exit);   // arrives once this thread's products are done
  } else if (warp == 18) {
    // ======================= M4: D^T = V'^T K =======================
    constexpr uint32_t id4 = umma::idesc_bf16(128, K, 0, 1);
    for_chunks(nothing, [&](const LaItem &, int, int, int, int n) {
      const int st = n % kStages;
      const uint64_t kt = umma::sdesc_sw128(sbase + st * Lay::stage + Lay::k_off, Lay::panel, 1024);
      if (!wait(&ms.full[st], (uint32_t)((n / kStages) & 1))) return false;
      const int di = AGG ? n & 1 : 0;
      const uint32_t dph = (uint32_t)((AGG ? n >> 1 : n) & 1), tD = tmem + (AGG ? kTmDAgg + di * 128 : kTmD);
      if (n >= (AGG ? 2 : 1) && !wait(&ms.d_free[di], dph ^ 1u)) return false;
#pragma unroll (AGG ? 4 : 1)
      for (int b = 0; b < 4; ++b) {   // 32 tokens: two steps of 16, three terms
        const int buf = AGG ? b : b & 1;   // of two buffers, each has two phases per chunk
        if (!wait(&ms.vp_rdy[buf], (uint32_t)(AGG ? n & 1 : b >> 1))) return false;
        if (umma::elect_one()) {
#pragma unroll
          for (int x = 0; x < 6; ++x)
            umma::mma_f16_ts(tD, tmem + (AGG ? kTmVpAgg : kTmVp) + buf * kTmVpBuf + x * 8,
                             umma::desc_add(kt, (2 * b + (x & 1)) * 2048), id4, b > 0 || x > 0);
          umma::commit(&ms.vp_free[buf]);
          if (b == 3) {
            umma::commit(&ms.d_rdy[di]);
            umma::commit(&ms.empty[st]);
          }
        }
        __syncwarp();
      }
      return true;
    }, nothing);
    if (umma::elect_one()) umma::commit(&ms.bar_exit);
  } else if (warp == 19) {
    // ======================= output =======================
    if constexpr (!AGG) {
      for_chunks(nothing, [&](const LaItem &it, int h, int c, int, int n) {
        const int st = n % kStages;
        if (!wait(&ms.o_st[st], (uint32_t)((n / kStages) & 1))) return false;
        const unsigned char *tile = sm + st * Lay::stage + Lay::v_off;
        const int t0 = it.t0 + c * kLaChunk, L = min(kLaChunk, it.len - c * kLaChunk);
        if (L == kLaChunk || !p.cu) {   // a partial chunk of an unpacked sequence ends at T, where the map ends
          if (umma::elect_one()) {
#pragma unroll
            for (int x = 0; x < V / 64; ++x) umma::tma_store_4d(&maps.o, tile + x * Lay::panel, x * 64, h, t0, it.b);
            umma::bulk_commit();
            umma::bulk_wait_read();
          }
        } else {                        // the rows after it are the next packed sequence's
          __nv_bfloat16 *dst = p.o + (((long long)it.b * p.T + t0) * p.H + h) * V;
#pragma unroll 4
          for (int x = lane; x < L * (V / 8); x += 32) {
            const int i = x / (V / 8), j = x % (V / 8);
            *reinterpret_cast<uint4 *>(dst + (long long)i * p.H * V + j * 8) =
                *reinterpret_cast<const uint4 *>(tile + (j >> 3) * Lay::panel + umma::sw128_chunk(i, j & 7));
          }
        }
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&ms.empty_v[st]);
        return true;
      }, nothing);
    }
  } else if (warp < 8) {
    // ======================= P and V' =======================
    umma::regs_dec<kLaRegsOperands>();
    const int wg = warp >> 2, quad = warp & 3;
    const bool has_ch = quad * 32 < V;   // V' lanes are value columns
    // 8 x 8 blocks of the v tile, transposed: matrix i of a load is channels 8 (i % 2), tokens 8 (i / 2) of
    // 16 channels x 16 tokens; lane l names token l % 8 of matrix l / 8
    const int ch0 = quad * 32 + ((lane >> 3) & 1) * 8;
    const uint32_t v_src = (uint32_t)((ch0 >> 6) * Lay::panel + ((lane >> 4) * 8 + (lane & 7)) * 128);
    // Without P to form, both warpgroups take every other 32 tokens of V'.
    const int b_first = AGG ? wg : 0, b_step = AGG ? 2 : 1;
    // The roles' loops stay rolled: each warp runs alone on its scheduler in its role, and code that does
    // not repeat is fetched at every step (fully unrolled, P and V' took twice as long).
    if (AGG || wg == 1) for_chunks(nothing, [&](const LaItem &it, int, int c, int, int n) {
      const int st = n % kStages;
      const uint32_t sph = (uint32_t)((n / kStages) & 1);
      if (!wait(&ms.full_v[st], sph) || !wait(&ms.gate[st], sph)) return false;
      unsigned char *kt = sm + st * Lay::stage + Lay::k_off, *vt = sm + st * Lay::stage + Lay::v_off;
      const int L = min(kLaChunk, it.len - c * kLaChunk);
      if (L < kLaChunk) {
        // k and v rows past the sequence hold the next packed sequence: their factors are zero, but
        // zero times an inf or NaN there would not be. This warpgroup clears them; what it reads
        // below of v before that is masked.
        if (!wait(&ms.full[st], sph)) return false;
        for (int x = tid & 127; x < (kLaChunk - L) * 8; x += 128) {
          const uint32_t off = (uint32_t)(L * 128 + x * 16);
#pragma unroll
          for (int y = 0; y < K / 64; ++y) *reinterpret_cast<uint4 *>(kt + y * Lay::panel + off) = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int y = 0; y < V / 64; ++y) *reinterpret_cast<uint4 *>(vt + y * Lay::panel + off) = make_uint4(0, 0, 0, 0);
        }
        umma::fence_proxy_async_smem();
      }
      if constexpr (!AGG) arrive(&ms.v_rdy[st]);
      const LaGate &g = gates[st];
#pragma unroll 1
      for (int b = b_first; b < 4; b += b_step) {
        const int buf = AGG ? b : b & 1;
        // M4 has read the buffer's last content, of the chunk before or of block b - 2
        auto buffer_free = [&] {
          return AGG ? n == 0 || wait(&ms.vp_free[buf], (uint32_t)((n - 1) & 1))
                     : (n == 0 && b < 2) || wait(&ms.vp_free[buf], (uint32_t)((b >> 1) ^ 1));
        };
        uint32_t t0[16], t1[16], t2[16];
        if (has_ch) {
          uint32_t raw[16];
          const uint32_t src = umma::smem_u32(vt) + v_src + (uint32_t)(32 * b * 128);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              umma::ldmatrix_x4_trans(src + 16 * i * 128 + (uint32_t)(((((ch0 & 63) >> 3) + 2 * hh) ^ (lane & 7)) << 4),
                                      raw[8 * hh + 4 * i], raw[8 * hh + 4 * i + 1], raw[8 * hh + 4 * i + 2], raw[8 * hh + 4 * i + 3]);
          if (L < kLaChunk) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int t = 32 * b + 8 * ((r >> 1) & 3) + 2 * (lane & 3);
              raw[r] &= t + 1 < L ? 0xFFFFFFFFu : t < L ? 0xFFFFu : 0u;
            }
          }
          const float bf = g.bf[b];
          const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float2 w = __fmul2_rn(*reinterpret_cast<const float2 *>(&g.cf[32 * b + 8 * m + 2 * (lane & 3)]), make_float2(bf, bf));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 8 * (e >> 1) + 2 * m + (e & 1);
              float2 x = __fmul2_rn(make_float2(__uint_as_float(raw[r] << 16), __uint_as_float(raw[r] & 0xFFFF0000u)), w);
              t0[r] = pack_bf16(x.x, x.y);
              x = __ffma2_rn(make_float2(__uint_as_float(t0[r] << 16), __uint_as_float(t0[r] & 0xFFFF0000u)), minus, x);
              t1[r] = pack_bf16(x.x, x.y);
              x = __ffma2_rn(make_float2(__uint_as_float(t1[r] << 16), __uint_as_float(t1[r] & 0xFFFF0000u)), minus, x);
              t2[r] = pack_bf16(x.x, x.y);
            }
          }
        }
        if (!buffer_free()) return false;
        if (has_ch) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t dst = tmem + (AGG ? kTmVpAgg : kTmVp) + buf * kTmVpBuf + lane_base + ((uint32_t)(hh * 16) << 16);
            umma::tmem_st_16x128b_x4(dst, t0 + 8 * hh);
            umma::tmem_st_16x128b_x4(dst + 16, t1 + 8 * hh);
            umma::tmem_st_16x128b_x4(dst + 32, t2 + 8 * hh);
          }
          umma::tmem_st_wait();
        }
        if (b + b_step >= 4) arrive(AGG ? &ms.empty_v[st] : &ms.v_read[st]);
        arrive(&ms.vp_rdy[buf]);
      }
      return true;
    }, nothing);
    if (!AGG && wg == 0) for_chunks(nothing, [&](const LaItem &, int, int, int, int n) {
      const int st = n % kStages;
      if (!wait(&ms.gate[st], (uint32_t)((n / kStages) & 1))) return false;
      const LaGate &g = gates[st];
      const int mode = g.weak;
      const bool weak = mode > 0;
      const float Gr = weak ? 0.f : la_row_shift(g, row, mode);   // G_i - R_i
      if (!wait(&ms.p_raw, (uint32_t)(n & 1))) return false;
      // block c of P goes to columns 16 c .. of the scores, block c / 2 of them: read by then
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
        if (c <= quad) {
          float x[32];
          umma::tmem_ld32(tmem + kTmP + lane_base + c * 32, x);
          umma::tmem_ld_wait();
          if (weak) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 w = *reinterpret_cast<const float4 *>(&g.G[32 * c + j]);
              const float2 a = __fmul2_rn(make_float2(x[j], x[j + 1]), make_float2(w.x, w.y));
              const float2 b = __fmul2_rn(make_float2(x[j + 2], x[j + 3]), make_float2(w.z, w.w));
              x[j] = a.x; x[j + 1] = a.y; x[j + 2] = b.x; x[j + 3] = b.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] *= ex2_approx(Gr - g.G[32 * c + j]);
          }
          if (c == quad) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = j <= lane ? x[j] : 0.f;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
        }
        umma::tmem_st16(tmem + kTmP + lane_base + c * 16, pk);
      }
      umma::tmem_st_wait();
      arrive(&ms.p_rdy);
      arrive(&ms.empty[st]);
      return true;
    }, nothing);
  } else if (warp < 16) {
    // ======================= state and output =======================
    umma::regs_inc<kLaRegsState>();
    constexpr int KH = K / 2, VH = V / 2;      // this warpgroup's columns of S^T and of O
    const int half = (warp - 8) >> 2;
    const bool has_v = (warp & 3) * 32 < V;    // lanes are value columns of S^T, token rows of O
    float S[KH];
    float seg_decay = 1.f;
    uint32_t sync_phase = 0;
    auto sync_state = [&] {
      arrive(&ms.state_sync);
      const bool ok = wait(&ms.state_sync, sync_phase);
      sync_phase ^= 1u;
      return ok;
    };
    auto copy_s = [&] {                        // bf16 copy of S^T, the operand of M2
      if (has_v) {
#pragma unroll
        for (int j = 0; j < KH; j += 8) {
          const int k = half * KH + j;
          *reinterpret_cast<uint4 *>(sm + Lay::s_off + (k >> 6) * Lay::s_panel + umma::sw128_chunk(row, (k & 63) >> 3)) =
              make_uint4(pack_bf16(S[j], S[j + 1]), pack_bf16(S[j + 2], S[j + 3]), pack_bf16(S[j + 4], S[j + 5]),
                         pack_bf16(S[j + 6], S[j + 7]));
        }
      }
      umma::fence_proxy_async_smem();
      arrive(&ms.s_rdy);
    };
    // this warp's part of the copy's buffer, for the states' way to and from memory between items
    float *patch = reinterpret_cast<float *>(sm + Lay::s_off) + (half * (V / 32) + (warp & 3)) * (32 * (K / 4));
    auto seg_block = [&](int slot, int h) { return p.seg_state + ((long long)slot * p.H + h) * (K * V); };
    // A state on its way from one CTA to the next, and this warp's flag for it
    auto hand_block = [&](int cta) { return p.hand + (long long)cta * (K * V); };
    auto hand_flag = [&](int cta) { return p.hand_there + cta * 8 + (warp - 8); };
    auto hand_wait = [&](int cta) {
      bool ok = true;
      if (lane == 0) {
        const unsigned t0 = (unsigned)clock();
        while (ok && !umma::ld_acquire(hand_flag(cta))) {
          if ((unsigned)clock() - t0 > kLaWaitLimit) *(volatile int *)&ms.err = 1;
          ok = !*(volatile int *)&ms.err;
        }
      }
      __syncwarp();   // the vote orders no memory: the other lanes' reads of the state come after the flag's by this
      return (bool)__all_sync(0xffffffffu, ok);
    };
    for_chunks(
        [&](const LaItem &it, int h, int nch) {
          // Only a sequence in one piece reads p.init here, and writes final_state after it: they may be one
          // buffer, and between the segments of a sequence, on different CTAs, nothing else orders the two.
          const bool other = SHARE && (it.part & kLaFromOther), first = it.seg == 0 && !other;
          if (AGG || (first && !p.init) || !has_v) {
#pragma unroll
            for (int j = 0; j < KH; ++j) S[j] = 0.f;
          } else if (first && it.n_seg == 1) {
            la_state_move<K, V, KH, false>(p, it.seq, h, (warp & 3) * 32, half * KH, S, patch);
          } else {
            if (other && !hand_wait(ms.cta - 1)) return false;
            const float *src = other ? hand_block(ms.cta - 1) : seg_block(first ? it.slot + it.n_seg - 1 : it.slot - 1, h);
#pragma unroll
            for (int j = 0; j < KH / 4; ++j) {
              const float4 f = __ldcg(reinterpret_cast<const float4 *>(src + la_seg_index<K, V>(half, row, j)));
              S[4 * j] = f.x; S[4 * j + 1] = f.y; S[4 * j + 2] = f.z; S[4 * j + 3] = f.w;
            }
          }
          seg_decay = 1.f;
          if constexpr (!AGG) {
            if (!sync_state()) return false;   // the states have left the copy's buffer, M2 has read it (s_free)
            if (nch > 0) copy_s();
          }
          return true;
        },
        [&](const LaItem &it, int h, int c, int nch, int n) {
          const int st = (int)(n % kStages);
          const uint32_t ph = (uint32_t)(n & 1);
          if (!wait(&ms.gate[st], (uint32_t)((n / kStages) & 1))) return false;
          const float gamma = gates[st].gamma;
          float f = 0.f;   // scale exp(R_i) of this thread's token row
          if constexpr (!AGG) {
            const float G = gates[st].G[row];
            const int weak = gates[st].weak;
            f = p.scale * (weak > 0 ? rcp_approx(G) : ex2_approx(G - la_row_shift(gates[st], row, weak)));
          }
          arrive(&ms.empty[st]);   // the factors have been read
          auto new_state = [&] {   // S^T = gamma S^T + D^T
            const int di = AGG ? n & 1 : 0;
            if (!wait(&ms.d_rdy[di], (uint32_t)((AGG ? n >> 1 : n) & 1))) return false;
            if (has_v) {
#pragma unroll
              for (int x = 0; x < KH; x += 32) {
                float y[32];
                umma::tmem_ld32(tmem + (AGG ? kTmDAgg + di * 128 : kTmD) + lane_base + half * KH + x, y);
                umma::tmem_ld_wait();
                if (x + 32 >= KH) arrive(&ms.d_free[di]);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  const float2 a = __ffma2_rn(make_float2(gamma, gamma), make_float2(S[x + j], S[x + j + 1]), make_float2(y[j], y[j + 1]));
                  S[x + j] = a.x;
                  S[x + j + 1] = a.y;
                }
              }
            } else {
              arrive(&ms.d_free[di]);
            }
            if constexpr (AGG) seg_decay *= gamma;
            if (AGG) return true;
            if (!wait(&ms.s_free, ph)) return false;   // M2 has read the copy
            if (c + 1 < nch) copy_s();
            return true;
          };
          auto output = [&] {      // o = f O in bf16, over the chunk's v, which M3 and the V' warps have read
            if (!wait(&ms.o_done, ph) || !wait(&ms.v_read[st], (uint32_t)((n / kStages) & 1))) return false;
            unsigned char *tile = sm + st * Lay::stage + Lay::v_off;
#pragma unroll 1
            for (int x = 0; x < VH; x += 32) {
              float y[32];
              umma::tmem_ld32(tmem + kTmO + lane_base + half * VH + x, y);
              umma::tmem_ld_wait();
              if (x + 32 >= VH) arrive(&ms.o_free);
              const int col = half * VH + x;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t pk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 a = __fmul2_rn(make_float2(y[8 * j + 2 * e], y[8 * j + 2 * e + 1]), make_float2(f, f));
                  pk[e] = pack_bf16(a.x, a.y);
                }
                *reinterpret_cast<uint4 *>(tile + (col >> 6) * Lay::panel + umma::sw128_chunk(row, ((col & 63) >> 3) + j)) =
                    make_uint4(pk[0], pk[1], pk[2], pk[3]);
              }
            }
            umma::fence_proxy_async_smem();
            arrive(&ms.o_st[st]);
            return true;
          };
          if constexpr (AGG) return new_state();
          // whichever product is done first; rolled, so that each part is one piece of code
          const bool state_first = __all_sync(0xffffffffu, umma::mbar_test(&ms.d_rdy[0], ph));
#pragma unroll 1
          for (int part = 0; part < 2; ++part)
            if (!((part == 0) == state_first ? new_state() : output())) return false;
          return true;
        },
        [&](const LaItem &it, int h, int) {
          if (!has_v) return true;
          if (AGG || (SHARE && (it.part & kLaToOther))) {
            float *dst = AGG ? seg_block(it.slot, h) : hand_block(ms.cta);
#pragma unroll
            for (int j = 0; j < KH / 4; ++j)
              *reinterpret_cast<float4 *>(dst + la_seg_index<K, V>(half, row, j)) =
                  make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
            if constexpr (AGG) {
              if (tid == 8 * 32) p.seg_decay[(long long)it.slot * p.H + h] = seg_decay;
            } else {
              __threadfence();
              __syncwarp();
              if (lane == 0) umma::st_release(hand_flag(ms.cta), 1);
            }
          } else if (it.seg == it.n_seg - 1 && p.final_state) {
            la_state_move<K, V, KH, true>(p, it.seq, h, (warp & 3) * 32, half * KH, S, patch);
          }
          return true;
        });
  }

  // no product of this CTA may be in flight past this point
  if (warp == 17 || warp == 18) umma::mbar_wait_bounded(&ms.bar_exit, 0, kLaWaitLimit);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (tid == 0 && ms.err) atomicExch(p.dev_status, kDevWaitTimeout);
  if (warp == 0) umma::tmem_dealloc(tmem, kLaTmemCols);
}

// Start states of the segments: chains, over the segments of a sequence, what each segment adds.
// One thread per four state values; segment g's block is read and then holds the start of g + 1, and the
// last segment's block, which adds to none, the start of the first: the initial state in fp32. Bound by
// latency: 6.8 us for nine segments of 16 heads at K = V = 128 (8 MB read), with eight loads of a thread in
// flight; a launch of it with nothing to combine takes 4 us.
template <int K, int V>
__global__ void __launch_bounds__(256) la_combine_kernel(const LaProblem p) {
  pdl_wait();
  if (p.flag && *p.flag != kDevOk) return;
  const int h = blockIdx.x % p.H;
  int s = blockIdx.x / p.H;
  if (p.cu) {
    if (s >= p.counts[2]) return;
    s = p.multi[s];
  }
  const int slot0 = p.cu ? p.slot0[s] : s * p.n_seg;
  const int n = p.cu ? p.slot0[s + 1] - slot0 : p.n_seg;
  const int x = blockIdx.y * 256 + threadIdx.x;             // float4 index of the block
  const int j = x / (2 * V), half = (x / V) & 1, v = x % V;
  float S[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.init) {
    const long long base = ((long long)s * p.H + h) * (K * V);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = half * (K / 2) + 4 * j + e;
      const long long i = base + ((p.flags & kStateKV) ? k * V + v : v * K + k);
      S[e] = (p.flags & kStateBf16) ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.init)[i])
                                    : static_cast<const float *>(p.init)[i];
    }
    reinterpret_cast<float4 *>(p.seg_state + ((long long)(slot0 + n - 1) * p.H + h) * (K * V))[x] =
        make_float4(S[0], S[1], S[2], S[3]);
  }
  constexpr int kAhead = 8;   // blocks whose loads are in flight together
  for (int g0 = 0; g0 + 1 < n; g0 += kAhead) {
    float4 f[kAhead];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (g0 + i + 1 < n) {
        const long long block = (long long)(slot0 + g0 + i) * p.H + h;
        f[i] = reinterpret_cast<const float4 *>(p.seg_state + block * (K * V))[x];
        d[i] = p.seg_decay[block];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (g0 + i + 1 < n) {
        S[0] = fmaf(d[i], S[0], f[i].x);
        S[1] = fmaf(d[i], S[1], f[i].y);
        S[2] = fmaf(d[i], S[2], f[i].z);
        S[3] = fmaf(d[i], S[3], f[i].w);
        reinterpret_cast<float4 *>(p.seg_state + ((long long)(slot0 + g0 + i) * p.H + h) * (K * V))[x] =
            make_float4(S[0], S[1], S[2], S[3]);
      }
    }
  }
}

// Clears the flags of the states handed over and the count of started CTAs.
__global__ void __launch_bounds__(256) la_clear_kernel(int32_t *flags, int n) {
  pdl_launch_dependents();
  pdl_wait();
  for (int i = threadIdx.x; i < n; i += 256) flags[i] = 0;
}

// Varlen schedule: checks cu_seqlens, cuts the sequences into segments of seg_chunks chunks and lists
// them: first the segments whose states are formed ahead (all but the last of a sequence, equally
// long), then the others, longest first (counting sort; very long ones share bins, which only makes
// the order approximate). Also lists the sequences of more than one segment. One CTA, bound by latency: 6.5
// us for 16 sequences, 7.3 for 512, of which the kernel behind it hides its own launch and set-up.
constexpr int kLaSchedThreads = 1024, kLaSchedBins = 2048;

// Exclusive sum over the CTA's threads, and the total; `part` holds 33 ints.
__device__ __forceinline__ int block_exclusive_sum(int x, int *part, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += y;
  }
  __syncthreads();
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int t = part[lane], ti = t;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ti, m);
      if (lane >= m) ti += y;
    }
    part[lane] = ti - t;
    if (lane == 31) part[32] = ti;
  }
  __syncthreads();
  total = part[32];
  return part[warp] + incl - x;
}

__global__ void __launch_bounds__(kLaSchedThreads) la_schedule_kernel(const LaProblem p) {
  __shared__ int s_part[33];
  __shared__ int s_bins[kLaSchedBins];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, N = p.N;
  const int32_t *cu = p.cu;
  bool bad = tid == 0 && (cu[0] != 0 || cu[N] != p.T);
  for (int i = tid; i < N; i += kLaSchedThreads) bad |= cu[i + 1] < cu[i];
  for (int b = tid; b < kLaSchedBins; b += kLaSchedThreads) s_bins[b] = 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      *p.flag = kDevBadCuSeqlens;
      atomicExch(p.dev_status, kDevBadCuSeqlens);
    }
    return;
  }
  if (tid == 0) *p.flag = kDevOk;
  const int seg_len = p.seg_chunks * kLaChunk;
  auto put = [&](int pos, int seq, int t0, int len, int g, int n, int slot0) {
    LaItem it;
    it.seq = seq;
    it.b = 0;
    it.seg = g;
    it.n_seg = n;
    it.slot = slot0 + g;
    it.t0 = g ? t0 + g * seg_len : t0;
    it.len = g < n - 1 ? seg_len : len - (it.t0 - t0);
    it.part = 0;
    p.items[pos] = it;
  };
  const int longest = min(p.seg_chunks, (p.T + kLaChunk - 1) / kLaChunk);
  const int per_bin = longest / kLaSchedBins + 1;   // chunk counts per bin; bins in descending order
  auto bin_of = [&](int chunks) { return (longest - chunks) / per_bin; };
  // how many segments are formed ahead, how many sequences have any
  int ahead = 0, multi = 0;
  for (int base = 0; base < N; base += kLaSchedThreads) {
    const int i = base + tid;
    int n = 1, t0 = 0, len = 0;
    if (i < N) {
      t0 = cu[i];
      len = cu[i + 1] - t0;
      const int nc = (len + kLaChunk - 1) / kLaChunk;
      n = max(1, (nc + p.seg_chunks - 1) / p.seg_chunks);
      atomicAdd(&s_bins[bin_of(nc - (n - 1) * p.seg_chunks)], 1);
    }
    int more, many;
    const int before = ahead + block_exclusive_sum(n - 1, s_part, more);
    const int rank = multi + block_exclusive_sum(n > 1, s_part, many);
    if (i < N) p.slot0[i] = before + rank;   // the sequences before that have slots have one more than are formed ahead
    if (n > 1) p.multi[rank] = i;
    for (int g = 0; g < n - 1; ++g) put(before + g, i, t0, len, g, n, before + rank);
    ahead += more;
    multi += many;
  }
  if (tid == 0) {
    p.slot0[N] = ahead + multi;
    p.counts[0] = N + ahead;
    p.counts[1] = ahead;
    p.counts[2] = multi;
  }
  // start positions of the bins, two per thread, after the segments formed ahead
  __syncthreads();
  const int x0 = s_bins[2 * tid], x1 = s_bins[2 * tid + 1];
  int total;
  const int at = ahead + block_exclusive_sum(x0 + x1, s_part, total);
  s_bins[2 * tid] = at;
  s_bins[2 * tid + 1] = at + x0;
  __syncthreads();
  for (int i = tid; i < N; i += kLaSchedThreads) {
    const int t0 = cu[i], len = cu[i + 1] - t0;
    const int nc = (len + kLaChunk - 1) / kLaChunk, n = max(1, (nc + p.seg_chunks - 1) / p.seg_chunks);
    put(atomicAdd(&s_bins[bin_of(nc - (n - 1) * p.seg_chunks)], 1), i, t0, len, n - 1, n, p.slot0[i]);
  }
}

// ---------------------------------------------------------------------------------- host

// How a call is cut: chunks per segment, segments per sequence (fixed length), and how many items and
// segment states the workspace holds.
struct LaPlan {
  int seg_chunks, n_seg;
  long long items;     // segments of all sequences: at most so many
  long long slots;     // segments of the sequences of more than one: at most so many
  bool segments;       // whether any sequence may have more than one segment
  long long multi;     // how many may
  int shared;          // CTAs of a call that may hand a state over, or 0
};

// CTAs share items where one of them would else have more than this many chunks over its share. Measured on
// 152 SMs with K = V = 128, shared and whole items: 256 items of 8 chunks, 2.5 over, 70 and 66 us; 160
// items of 4, 3.8 over, 37.5 and 39.6; 256 of 16, 5 over, 108 and 111; 256 of 32, 10 over, 187 and 199; 192
// of 128, 94 over, 518 and 754.
constexpr int kLaShareChunks = 3;

// Time model of a call, in microseconds: rounds of items of `chunks` chunks each per CTA, in the kernel
// that does everything and in the one that forms the segments' states. The constants were measured at K = V
// = 128: 512 chunks in a row take 1407 us, and the segments of 65536 tokens of 16 heads, 57 chunks per CTA,
// 88 us; an item adds 2 us, the second pass with its combine 12. A chunk takes at least its bytes' share of
// the memory bandwidth. The number of segments it chooses is within 4% of the best of 24 that were tried
// for each of 22 shapes (but 6% for 3 x 4096 tokens of 24 heads).
constexpr double kLaChunkUs = 2.75, kLaAggChunkUs = 1.6, kLaItemUs = 2.0, kLaPassUs = 12.0, kLaBytesPerUs = 6.5e6;

static double la_pass_us(long long items, int chunks, int sms, double chunk_us, double chunk_bytes, bool share) {
  if (items == 0) return 0.0;
  double rounds = (double)((items + sms - 1) / sms);
  if (share && (rounds - (double)items / sms) * chunks > kLaShareChunks)
    rounds = std::max(1.0, (double)items / sms + (double)kLaShareChunks / chunks);
  const double mem_us = chunk_bytes * (double)std::min(items, (long long)sms) / kLaBytesPerUs;
  return rounds * (chunks * std::max(chunk_us, mem_us) + kLaItemUs);
}

// Chunks per segment of `chains` (sequence, head) pairs of nc chunks each: few chains leave SMs idle,
// and cutting them into segments costs a pass over k and v. share: whether CTAs may share items.
static int la_segment_chunks(long long chains, int nc, int K, int V, int sms, bool share) {
  const double bytes = kLaChunk * 2.0 * (2 * K + 2 * V), agg_bytes = kLaChunk * 2.0 * (K + V);
  int best = nc;
  double best_us = la_pass_us(chains, nc, sms, kLaChunkUs, bytes, share);
  for (int n = 2; n <= 512 && n <= nc; ++n) {
    const int seg = (nc + n - 1) / n, m = (nc + seg - 1) / seg;
    const double us = la_pass_us(chains * m, seg, sms, kLaChunkUs, bytes, share) +
                      la_pass_us(chains * (m - 1), seg, sms, kLaAggChunkUs, agg_bytes, false) + kLaPassUs;
    if (us < 0.95 * best_us) {
      best_us = us;
      best = seg;
    }
  }
  return best;
}

static LaPlan la_plan(int T, int H, int K, int V, int N, bool varlen) {
  LaPlan r = {};
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const int nc = std::max(1, (int)(((long long)T + kLaChunk - 1) / kLaChunk));
  if (!varlen) {
    r.seg_chunks = la_segment_chunks((long long)N * H, nc, K, V, sms, true);
    r.n_seg = (nc + r.seg_chunks - 1) / r.seg_chunks;
    r.segments = r.n_seg > 1;
    r.items = r.slots = (long long)N * r.n_seg;
    r.multi = N;
    const long long items = r.items * H, rounds = (items + sms - 1) / sms;
    if (items > sms && (rounds - (double)items / sms) * r.seg_chunks > kLaShareChunks) r.shared = sms;
    return r;
  }
  // The lengths are on the device: segments as for equal lengths, and never longer than what an SM has
  // to do on average, so that one long sequence among short ones does not hold up the call.
  const int nc_mean = std::max(1, (int)(((long long)T / std::max(N, 1) + kLaChunk - 1) / kLaChunk));
  const int share = (int)std::min((double)nc, std::ceil((nc + 0.5 * N) * (double)H / sms));
  r.seg_chunks = la_segment_chunks((long long)N * H, nc_mean, K, V, sms, false);
  if (r.seg_chunks >= nc_mean) r.seg_chunks = std::max(nc_mean, std::max(share, 8));
  r.n_seg = 1;
  // Each segment but a sequence's last is full, and has a token behind it.
  const long long ahead = std::max(T - 1, 0) / ((long long)r.seg_chunks * kLaChunk);
  r.multi = std::min((long long)N, ahead);
  r.segments = r.multi > 0;
  r.items = N + ahead;
  r.slots = r.multi + ahead;
  return r;
}

struct LaScratch {
  size_t flag, counts, slot0, multi, items, decay, state, hand, there, total;
};
static LaScratch la_scratch(const LaPlan &pl, int H, int K, int V, int N, bool varlen) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  LaScratch s = {};
  size_t off = 0;
  if (varlen) {
    s.flag = off;
    s.counts = off + 4;
    off = up(off + 16);
    s.slot0 = off;
    off = up(off + 4 * ((size_t)N + 1));
    s.multi = off;
    off = up(off + 4 * (size_t)pl.multi);
    s.items = off;
    off = up(off + sizeof(LaItem) * (size_t)pl.items);
  }
  if (pl.segments) {
    s.decay = off;
    off = up(off + 4 * (size_t)pl.slots * H);
    s.state = off;
    off = up(off + 4 * (size_t)pl.slots * H * K * V);
  }
  if (pl.shared) {
    s.there = off;   // and after the flags the count of started CTAs
    off = up(off + 4 * (8 * (size_t)pl.shared + 1));
    s.hand = off;
    off = up(off + 4 * (size_t)pl.shared * K * V);
  }
  s.total = off;
  return s;
}

template <int K, int V, bool AGG, bool SHARE = false>
static cudaError_t launch_la_t(const LaProblem &p, const LaMaps &maps, long long items, cudaStream_t stream) {
  static PerDeviceOnce attr;
  constexpr int smem = (int)LaLayout<K, V, AGG>::bytes;
  cudaError_t e = attr([&](int) {
    return cudaFuncSetAttribute(la_kernel<K, V, AGG, SHARE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  const long long grid = std::min(items * p.H, (long long)(sms > 0 ? sms : 1));
  return launch_kernel(la_kernel<K, V, AGG, SHARE>, dim3((unsigned)grid), dim3(kLaThreads), smem, stream, true, p, maps);
}

template <int K, int V>
static cudaError_t launch_la(const LaProblem &p, const LaMaps &maps, const LaPlan &pl, cudaStream_t s) {
  // Every launch overlaps the end of the kernel ahead, the first one the caller's: 128 tokens of two heads take
  // 7.2 us from one call to the next instead of 10.2.
  if (p.cu) {
    const cudaError_t e = launch_kernel(la_schedule_kernel, dim3(1), dim3(kLaSchedThreads), 0, s, true, p);
    if (e != cudaSuccess) return e;
  }
  if (pl.shared) {
    const cudaError_t e = launch_kernel(la_clear_kernel, dim3(1), dim3(256), 0, s, true, p.hand_there, 8 * pl.shared + 1);
    if (e != cudaSuccess) return e;
  }
  if (pl.segments) {
    cudaError_t e = launch_la_t<K, V, true>(p, maps, pl.items, s);
    if (e == cudaSuccess)
      e = launch_kernel(la_combine_kernel<K, V>, dim3((unsigned)(pl.multi * p.H), K * V / 1024), dim3(256), 0, s, true, p);
    if (e != cudaSuccess) return e;
  }
  return pl.shared ? launch_la_t<K, V, false, true>(p, maps, pl.items, s)
                   : launch_la_t<K, V, false>(p, maps, pl.items, s);
}

static bool la_sizes_ok(int B, int T, int Hk, int H, int K, int V, int N) {
  return B >= 1 && T >= 0 && Hk >= 1 && H >= 1 && H % Hk == 0 && K >= 1 && V >= 1 && N >= 0;
}

}  // namespace kda

extern "C" {

size_t kda_la_workspace_size(int B, int T, int H, int K, int V, int num_seqs, int varlen) {
  using namespace kda;
  if (!la_sizes_ok(B, T, 1, H, K, V, num_seqs)) return 0;
  return la_scratch(la_plan(T, H, K, V, num_seqs, varlen != 0), H, K, V, num_seqs, varlen != 0).total;
}

kda_status_t kda_la_fwd(const void *q, const void *k, const void *v, const float *log_decay, float scale,
                        const void *initial_state, void *final_state, const int32_t *cu_seqlens, int B, int T, int Hk,
                        int H, int K, int V, int num_seqs, const kda_la_strides_t *strides, uint32_t flags, void *o,
                        void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  using namespace kda;
  if (flags & ~(kLaTokenDecay | kStateBf16 | kStateKV)) return KDA_ERR_INVALID_ARG;
  if (!la_sizes_ok(B, T, Hk, H, K, V, num_seqs)) return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k || !v || !log_decay || !o)) return KDA_ERR_INVALID_ARG;
  if ((K != 64 && K != 128) || (V != 64 && V != 128)) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if (cu_seqlens ? (B != 1 || !aligned(cu_seqlens, 4)) : num_seqs != B) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(log_decay, 4) ||
      !aligned(initial_state, 16) || !aligned(final_state, 16))
    return KDA_ERR_INVALID_ARG;
  const int64_t contiguous[3][3] = {{(int64_t)T * Hk * K, (int64_t)Hk * K, K},
                                    {(int64_t)T * H * V, (int64_t)H * V, V},
                                    {(int64_t)T * H, H, 1}};
  const int64_t *sq = strides ? strides->q : contiguous[0], *sk = strides ? strides->k : contiguous[0];
  const int64_t *sv = strides ? strides->v : contiguous[1], *sd = strides ? strides->log_decay : contiguous[2];
  const int64_t extent[3] = {B, T, 0};
  for (int i = 0; i < 3; ++i) {
    const int64_t *s3[3] = {sq, sk, sv};
    for (int x = 0; x < 3; ++x) {
      const int64_t n = i < 2 ? extent[i] : (x == 2 ? H : Hk);
      if (n > 1 && (s3[x][i] <= 0 || s3[x][i] % 8 != 0 || s3[x][i] >= (int64_t)1 << 39)) return KDA_ERR_INVALID_ARG;
    }
  }
  // Token positions, and work items a little past their number, are counted in 32 bits.
  if ((double)B * T * H * std::max(K, V) > 9.0e15 || T > 2147480000) return KDA_ERR_UNSUPPORTED;
  const bool varlen = cu_seqlens != nullptr;
  const LaPlan pl = la_plan(T, H, K, V, num_seqs, varlen);
  if ((double)(pl.items + (varlen ? num_seqs : 0)) * H > 2.0e9) return KDA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return KDA_OK;
  const LaScratch L = la_scratch(pl, H, K, V, num_seqs, varlen);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *ws = workspace;
  if (L.total > 0) {
    if (workspace) {
      if (workspace_bytes < L.total || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    } else if (cudaMallocAsync(&ws, L.total, s) != cudaSuccess) {
      cudaGetLastError();
      return KDA_ERR_WORKSPACE;
    }
  }
  LaProblem p;
  std::memset(&p, 0, sizeof p);
  char *base = static_cast<char *>(ws);
  p.decay = log_decay;
  for (int i = 0; i < 3; ++i) p.ds[i] = sd[i];
  p.init = initial_state;
  p.final_state = final_state;
  p.cu = cu_seqlens;
  p.o = static_cast<__nv_bfloat16 *>(o);
  if (varlen) {
    p.flag = reinterpret_cast<int32_t *>(base + L.flag);
    p.counts = reinterpret_cast<int32_t *>(base + L.counts);
    p.multi = reinterpret_cast<int32_t *>(base + L.multi);
    p.slot0 = reinterpret_cast<int32_t *>(base + L.slot0);
    p.items = reinterpret_cast<LaItem *>(base + L.items);
  }
  if (pl.segments) {
    p.seg_decay = reinterpret_cast<float *>(base + L.decay);
    p.seg_state = reinterpret_cast<float *>(base + L.state);
  }
  if (pl.shared) {
    p.hand = reinterpret_cast<float *>(base + L.hand);
    p.hand_there = reinterpret_cast<int32_t *>(base + L.there);
    p.started = p.hand_there + 8 * pl.shared;
  }
  p.scale = scale;
  p.B = B; p.T = T; p.Hk = Hk; p.H = H; p.N = num_seqs;
  p.seg_chunks = pl.seg_chunks;
  p.n_seg = pl.n_seg;
  p.flags = flags;
  p.dev_status = device_status_address();
  kda_status_t st = p.dev_status ? KDA_OK : KDA_ERR_CUDA;
  LaMaps maps;
  std::memset(&maps, 0, sizeof maps);
  if (st == KDA_OK && T > 0) {
    auto encode = [&](CUtensorMap *m, const void *ptr, int D, int heads, const int64_t *e) {
      const long long bytes[3] = {(long long)e[2] * 2, (long long)e[1] * 2, (long long)e[0] * 2};
      return encode_swizzled_token_map(m, ptr, D, heads, T, B, bytes, kLaChunk);
    };
    if (!encode(&maps.q, q, K, Hk, sq) || !encode(&maps.k, k, K, Hk, sk) || !encode(&maps.v, v, V, H, sv) ||
        !encode(&maps.o, o, V, H, contiguous[1]))
      st = KDA_ERR_CUDA;
  }
  if (st == KDA_OK) {
    NvtxRange r("kda la forward");
    const cudaError_t e = K == 128 ? (V == 128 ? launch_la<128, 128>(p, maps, pl, s) : launch_la<128, 64>(p, maps, pl, s))
                                   : (V == 128 ? launch_la<64, 128>(p, maps, pl, s) : launch_la<64, 64>(p, maps, pl, s));
    if (e != cudaSuccess) st = KDA_ERR_CUDA;
  }
  if (L.total > 0 && !workspace) cudaFreeAsync(ws, s);
  return st;
}

}  // extern "C"
