// router_loss.hip -- the router's training step next to its gating: the
// load-balance loss with its per-expert counts, and the gradients of the loss
// and of the gating weights on the router logits.
//
// With m_t = 1 for the tokens that count (token_mask), N = sum m_t,
// c_e = the counted pairs routed to expert e, p_te = softmax(logits[t])_e,
// P_e = sum_t m_t p_te / N and f_e = c_e / (N k):
//   loss = coef * E * sum_e f_e P_e           (= coef under an even load)
//   d loss / d logits[t][i] = m_t coef E / N * p_ti (f_i - sum_e f_e p_te)
// f is a count and carries no gradient.  The gradient uses f_e - 1/E in the
// place of f_e: sum_e p_te = 1, so both are the same, and the difference,
// formed from the integer c_e E - N k, does not cancel in fp32 when the load
// is nearly even.  The gating weights w_j of the selected experts give
//   renormalised : d logits[id_j] = w_j (g_j - S),  S = sum_i w_i g_i
//   plain softmax: d logits[e] = [e = id_j] w_j g_j - p_te S.
//
// Both directions are one pass over [T,E] fp32 rows and bound by HBM for
// large batches (131072 x 256 in a training step: loss 43 us, without its
// arithmetic 38, since the step's last gradient is still being written back; its
// gradient 42 us, 6.4 TB/s; 65536 x 256, a third of it padding, both gradients
// with plain softmax 26 us, 4.6 TB/s), by launch latency for small ones (16 x 64:
// 3.8 and 2.5 us of kernel under 7 us of host work per call; 4096 x 256: 6.5, 4.2
// and 5.4 us in three dependent launches for 4 MB).  Blocks of 1024 threads take
// 64 rows at a time there, so 4096 rows fill 64 of the 256 CUs.  L = 16 lanes hold a row of
// up to 256 logits (four rows per wave), each lane NC runs of 4 values, so the
// row reductions stay inside the 16-lane rows that DPP moves reach at full
// rate; longer rows take 32 or 64 lanes rather than more registers per lane
// (16 lanes of 64 values held one wave per SIMD: 1024 experts at 2.3 TB/s).
// No sum depends on scheduling: blocks write partial sums that one block adds in
// block order, and the counts are integers.
#include "moe_common.h"

namespace moe {

constexpr int kLossThreads = 1024;
constexpr int kGradThreads = 256;

// Sum / maximum over the L lanes of a logits row; every lane gets it.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  if (L >= 32) v += __shfl_xor(v, 16);
  if (L >= 64) v += __shfl_xor(v, 32);
  return v;
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  if (L >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  if (L >= 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}

// Orders a wave's LDS accesses: its earlier writes are seen by its lanes.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Value q = 4c + i of lane l is expert (c * L + l) * 4 + i when E is a
// multiple of 4 (16-byte loads), else (4c + i) * L + l.
template <int L, bool VEC>
__device__ __forceinline__ int expert_of(int c, int i, int l) {
  return VEC ? (c * L + l) * 4 + i : (4 * c + i) * L + l;
}

template <int L, int NC, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l,
                                         float (&v)[4 * NC], float fill) {
#pragma unroll
  for (int c = 0; c < NC; c++) {
    if (VEC) {
      const int e = expert_of<L, true>(c, 0, l);
      f32x4 r = {fill, fill, fill, fill};
      if (e < E) r = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; i++) v[4 * c + i] = r[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int e = expert_of<L, false>(c, i, l);
        v[4 * c + i] = e < E ? row[e] : fill;
      }
    }
  }
}

// e^x for x <= 0 within about 2 steps: 2^y with y = fl(x log2 e), corrected by
// the part of x log2 e that y lost (7 instructions; the library's expf takes
// about twice as many, most of them for overflow and subnormal results, which
// a softmax does not need: results below 2^-126 become 0).
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596299e-8f, kLn2 = 0.693147182f;
  x = fmaxf(x, -128.0f);  // keeps the correction finite for -inf
  const float y = x * kLog2e;
  const float lost = fmaf(x, kLog2eLo, fmaf(x, kLog2e, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e, lost * kLn2, e);
}

// Softmax of a row in place; NaN reads as -inf (as the gating reads it), a row
// of -inf only becomes all zero, and a row with +inf all NaN.
template <int L, int N>
__device__ __forceinline__ void softmax_row(float (&v)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < N; q++) {
    v[q] = v[q] == v[q] ? v[q] : -INFINITY;
    m = fmaxf(m, v[q]);
  }
  m = row_max<L>(m);
  if (m == -INFINITY) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < N; q++) {
    v[q] = exp_neg(v[q] - m);
    s += v[q];
  }
  s = row_sum<L>(s);
  const float inv = s > 0.f ? 1.0f / s : m == INFINITY ? NAN : 0.f;
#pragma unroll
  for (int q = 0; q < N; q++) v[q] *= inv;
}

__device__ __forceinline__ bool row_live(const uint8_t* mask, long r, long end) {
  return r < end && (!mask || mask[r]);
}

// Writes expert e's count and mean probability from its sums over all tokens;
// returns the block's sum of count * probability (valid in thread 0).  Thread
// i holds expert e (none where e >= E); red: one double per wave.
__device__ __forceinline__ double finish_experts(double sum_p, int sum_c, int n, int e, int E,
                                                 int32_t* counts, float* probs, double* red) {
  const double p = n > 0 ? sum_p / n : 0.0;
  double part = 0.0;
  if (e < E) {
    counts[e] = sum_c;
    probs[e] = (float)p;
    part = sum_c * p;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) part += __shfl_xor(part, o);
  if (lane_id() == 0) red[threadIdx.x / kWave] = part;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < (int)blockDim.x / kWave; w++) part += red[w];
  return part;
}

__device__ __forceinline__ void finish_loss(double sum_cp, int n, int E, int k, float coef,
                                            float* loss, int32_t* token_count) {
  *loss = n > 0 ? (float)((double)coef * E * sum_cp / ((double)n * k)) : 0.f;
  *token_count = n;
}

// Block b sums the probabilities and counts of rows [b rows, (b + 1) rows)
// into row b of part_p and part_c (e4 values each) and part_n[b]; a single
// block writes the outputs itself.
template <int L, int NC, bool VEC>
__global__ __launch_bounds__(kLossThreads) void balance_loss_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, int rows, float coef,
    float* __restrict__ part_p, int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
    LossTicket* __restrict__ ticket, float* __restrict__ loss, int32_t* __restrict__ counts,
    float* __restrict__ probs, int32_t* __restrict__ token_count) {
  constexpr int N = 4 * NC, THREADS = kLossThreads, NW = THREADS / kWave;
  constexpr int E_MAX = N * L, STEP = THREADS / L;
  __shared__ float wsum[NW][E_MAX];
  __shared__ int hist[E_MAX];
  __shared__ double red[NW];
  __shared__ int n_live;
  const int t = threadIdx.x, l = t % L, w = t / kWave;
  const long lo = (long)blockIdx.x * rows, hi = min((long)T, lo + rows);
  for (int e = t; e < E; e += THREADS) hist[e] = 0;
  if (t == 0) n_live = 0;

  // rows r, r + STEP, ...: the next row is on its way while one is summed
  // (two buffers in turn: a copy would wait for the load), and the mask byte
  // of the one after it
  float acc[N], v[N], w2[N];
#pragma unroll
  for (int q = 0; q < N; q++) acc[q] = 0.f;
  const long f0 = lo * k + t;
  const int id0 = f0 < hi * k && (!mask || mask[f0 / k]) ? ids[f0] : -1;
  long r = lo + t / L;
  int live = 0;
  bool on = row_live(mask, r, hi), on1 = row_live(mask, r + STEP, hi);
  if (on) load_row<L, NC, VEC>(logits + (size_t)r * E, E, l, v, -INFINITY);
  __syncthreads();
  if ((unsigned)id0 < (unsigned)E) atomicAdd(&hist[id0], 1);
  for (long f = f0 + THREADS; f < hi * k; f += THREADS) {
    const int e = ids[f];
    if ((unsigned)e < (unsigned)E && (!mask || mask[f / k])) atomicAdd(&hist[e], 1);
  }
  auto round = [&](float(&cur)[N], float(&next)[N]) {
    const bool on2 = row_live(mask, r + 2 * STEP, hi);
    if (on1) load_row<L, NC, VEC>(logits + (size_t)(r + STEP) * E, E, l, next, -INFINITY);
    if (on) {
      softmax_row<L>(cur);
#pragma unroll
      for (int q = 0; q < N; q++) acc[q] += cur[q];
      live++;
    }
    on = on1;
    on1 = on2;
    r += STEP;
  };
  while (r < hi) {
    round(v, w2);
    round(w2, v);  // past the last row: nothing is on
  }
  if (l == 0 && live) atomicAdd(&n_live, live);
  // the wave's rows, then the waves in order
#pragma unroll
  for (int q = 0; q < N; q++) {
    if (L <= 16) acc[q] += __shfl_xor(acc[q], 16);
    if (L <= 32) acc[q] += __shfl_xor(acc[q], 32);
  }
  if (lane_id() < L) {
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) wsum[w][expert_of<L, VEC>(c, i, l)] = acc[4 * c + i];
  }
  __syncthreads();
  const int e4 = (E + 3) & ~3;
  const bool single = gridDim.x == 1;
  for (int e = t; e < (single ? E : e4); e += THREADS) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < NW; q++) s += wsum[q][e];
    if (single) {
      wsum[0][e] = s;  // this thread's expert
    } else {
      part_p[(size_t)blockIdx.x * e4 + e] = s;
      part_c[(size_t)blockIdx.x * e4 + e] = e < E ? hist[e] : 0;
    }
  }
  if (!single) {
    if (t == 0) {
      part_n[blockIdx.x] = n_live;
      if (blockIdx.x == 0) ticket->done = 0;  // for the launch after this one
    }
    return;
  }
  const double cp = finish_experts(t < E ? wsum[0][t] : 0.0, t < E ? hist[t] : 0, n_live, t, E,
                                   counts, probs, red);
  if (t == 0) finish_loss(cp, n_live, E, k, coef, loss, token_count);
}

// Adds the partial sums of n_parts blocks, FE experts a block: thread (s, q)
// those of experts 4q .. 4q+3 from blocks s, s + S, ... in order (16-byte
// loads, a few in flight at once), then the S slices in order.  With several
// blocks the last one to end adds their shares of the loss, in block order.
// One block for 256 experts' sums of up to 128 parts: the ticket's fence costs
// 0.9 us of 5 (64 parts 5.0 -> 4.2 us; 256 parts 7.2 -> 9 us); beyond that 128
// experts a block (one block for all read 1024 experts' 2 MB in 20 us).  Up to 64 experts
// take twice the slices (256 parts of 61: 5.1 -> 4.7 us).
template <int FE>
__global__ __launch_bounds__(1024) void balance_finish_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
    const int32_t* __restrict__ part_n, LossTicket* ticket, int n_parts, int E, int k, float coef,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ probs,
    int32_t* __restrict__ token_count) {
  constexpr int Q = FE / 4, S = 1024 / Q;
  __shared__ __attribute__((aligned(16))) double sp[S][FE];
  __shared__ __attribute__((aligned(16))) int sc[S][FE];
  __shared__ double red[16];
  __shared__ int live[16];
  const int t = threadIdx.x, q = t % Q, s = t / Q, e0 = blockIdx.x * FE;
  const int e4 = (E + 3) & ~3;
  int n = t < n_parts ? part_n[t] : 0;  // n_parts <= 1024
  double p[4] = {0, 0, 0, 0};
  int c[4] = {0, 0, 0, 0};
  if (e0 + 4 * q < E) {
#pragma unroll 4
    for (int b = s; b < n_parts; b += S) {
      const size_t o = (size_t)b * e4 + e0 + 4 * q;
      const f32x4 pv = *reinterpret_cast<const f32x4*>(part_p + o);
      const i32x4 cv = *reinterpret_cast<const i32x4*>(part_c + o);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        p[i] += pv[i];
        c[i] += cv[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    sp[s][4 * q + i] = p[i];
    sc[s][4 * q + i] = c[i];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  if (lane_id() == 0) live[t / kWave] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < 16; w++) n += live[w];
  double tp = 0.0;
  int tc = 0;
  if (t < FE) {
#pragma unroll 8
    for (int x = 0; x < S; x++) {
      tp += sp[x][t];
      tc += sc[x][t];
    }
  }
  double cp = finish_experts(tp, tc, n, t < FE ? e0 + t : E, E, counts, probs, red);
  if (t > 0) return;
  if (gridDim.x > 1) {
    ticket->share[blockIdx.x] = cp;
    __threadfence();
    if (atomicAdd(&ticket->done, 1) != (int)gridDim.x - 1) return;
    __threadfence();
    cp = 0.0;
    for (int b = 0; b < (int)gridDim.x; b++)
      cp += __hip_atomic_load(&ticket->share[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  finish_loss(cp, n, E, k, coef, loss, token_count);
}

// Gradient rows.  SOFT: the row's softmax is needed (the balance term, or the
// plain-softmax gating term); GATE: the gating term is added (ids, weights
// and grad_weights given).  The balance term is added when grad_loss is.
// A selected expert's term reaches the lane that owns the expert through the
// row's LDS copy: the lane of slot j adds the terms of every slot naming the
// same expert in slot order, and the first of those slots writes the sum.
// A row with NaN weights is one that the gating found no finite maximum in: its
// terms are 0 if it holds no +inf, else its gradient is NaN.  Where the softmax
// is not formed, such a row's logits are looked at for that alone.
template <int L, int NC, bool VEC, bool SOFT, bool GATE>
__global__ __launch_bounds__(kGradThreads) void router_grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, const float* __restrict__ grad_weights,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ token_count, const float* __restrict__ grad_loss, float coef,
    int renorm, int T, int E, int k, float* __restrict__ grad) {
  constexpr int N = 4 * NC, E_MAX = N * L, ROWS = kGradThreads / L, PER_WAVE = kWave / L;
  __shared__ __attribute__((aligned(16))) float sel[GATE ? ROWS : 1][GATE ? E_MAX : 4];
  const int t = threadIdx.x, l = t % L, g = t / L;
  const long step = (long)gridDim.x * ROWS;
  long r = (long)blockIdx.x * ROWS + g;
  // the first row is on its way while the counts are turned into d
  float v[N], v2[N];
  bool on = row_live(mask, r, T);
  if (SOFT && on) load_row<L, NC, VEC>(logits + (size_t)r * E, E, l, v, -INFINITY);
  float d[N];
  float scale = 0.f;
  if (SOFT && grad_loss) {
    const int n = *token_count;
    const double nk = (double)n * k, inv = n > 0 ? 1.0 / (nk * E) : 0.0;
    scale = n > 0 ? (float)((double)coef * E * *grad_loss / n) : 0.f;
#pragma unroll
    for (int c = 0; c < NC; c++) {
      i32x4 cv = {0, 0, 0, 0};
      if (VEC) {
        const int e = expert_of<L, true>(c, 0, l);
        if (e < E) cv = *reinterpret_cast<const i32x4*>(counts + e);
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int e = expert_of<L, false>(c, i, l);
          if (e < E) cv[i] = counts[e];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) d[4 * c + i] = (float)(((double)cv[i] * E - nk) * inv);
    }
  } else {
#pragma unroll
    for (int q = 0; q < N; q++) d[q] = 0.f;
  }
  if (GATE) {
#pragma unroll
    for (int q = 0; q < N; q++) sel[g][q * L + l] = 0.f;
    wave_lds_fence();
  }
  // a wave's rows take the same number of rounds: the LDS copy needs
  // fences inside the wave only
  auto round = [&](float(&v)[N], float(&next)[N]) {
    const bool on1 = row_live(mask, r + step, T);
    if (SOFT && on1) load_row<L, NC, VEC>(logits + (size_t)(r + step) * E, E, l, next, -INFINITY);
    float S = 0.f;
    int id = -1;
    bool lost = false;  // !SOFT: the row's gradient is NaN
    if (GATE) {
      float wg = 0.f, wj = 0.f;
      bool nan_w = false;
      if (on && l < k) {
        const size_t f = (size_t)r * k + l;
        id = ids[f];
        wj = weights[f];
        const float gj = grad_weights[f];
        nan_w = wj != wj;
        wj = nan_w ? 0.f : wj;
        wg = wj * gj;
        if ((unsigned)id >= (unsigned)E) {
          id = -1;
          wj = wg = 0.f;
        }
      }
      if (!SOFT && __any(nan_w && logits)) {  // the same way for the whole wave
        float m = -INFINITY;
        if (on)
          for (int e = l; e < E; e += L) m = fmaxf(m, logits[(size_t)r * E + e]);
        m = row_max<L>(m);
        lost = row_max<L>(nan_w ? 1.f : 0.f) > 0.f && m == INFINITY;
      }
      S = row_sum<L>(wg);
      const float term = renorm ? wg - wj * S : wg;
      float sum = 0.f;
      bool first = id >= 0;
      for (int j = 0; j < k; j++) {
        const int idj = __shfl(id, j, L);
        const float tj = __shfl(term, j, L);
        if (idj == id) {
          sum += tj;
          if (j < l) first = false;
        }
      }
      if (first) sel[g][id] = sum;
      wave_lds_fence();
    }
    if (on) {
      if (SOFT) {
        softmax_row<L>(v);
        float dp = 0.f;
#pragma unroll
        for (int q = 0; q < N; q++) dp = fmaf(d[q], v[q], dp);
        dp = row_sum<L>(dp);
        const float s0 = GATE && !renorm ? S : 0.f;
#pragma unroll
        for (int q = 0; q < N; q++) v[q] *= scale * (d[q] - dp) - s0;
      }
      if (GATE) {
#pragma unroll
        for (int c = 0; c < NC; c++) {
          if (VEC) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(&sel[g][expert_of<L, true>(c, 0, l)]);
#pragma unroll
            for (int i = 0; i < 4; i++) v[4 * c + i] = (SOFT ? v[4 * c + i] : 0.f) + a[i];
          } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
              v[4 * c + i] = (SOFT ? v[4 * c + i] : 0.f) + sel[g][expert_of<L, false>(c, i, l)];
          }
        }
        if (!SOFT && lost) {
#pragma unroll
          for (int q = 0; q < N; q++) v[q] = NAN;
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < N; q++) v[q] = 0.f;
    }
    if (r < T) {
      float* out = grad + (size_t)r * E;
#pragma unroll
      for (int c = 0; c < NC; c++) {
        if (VEC) {
          const int e = expert_of<L, true>(c, 0, l);
          if (e < E)
            *reinterpret_cast<f32x4*>(out + e) =
                f32x4{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int e = expert_of<L, false>(c, i, l);
            if (e < E) out[e] = v[4 * c + i];
          }
        }
      }
    }
    if (GATE) {
      wave_lds_fence();  // the row's reads are done
      if (id >= 0) sel[g][id] = 0.f;
      wave_lds_fence();
    }
    on = on1;
    r += step;
  };
  while (r - g % PER_WAVE < T) {  // the next row is on its way while one is worked on
    round(v, v2);
    round(v2, v);  // past the last row: nothing is read or written
  }
}

inline int row_lanes(int E) { return E <= 256 ? 16 : E <= 512 ? 32 : 64; }

// Blocks of the loss kernel: as many rows as a block takes at once, at most
// one block per CU; one block up to twice that many rows, which saves the
// finishing launch.
int balance_loss_blocks(int T, int E) {
  const long rows = kLossThreads / row_lanes(E), b = (T + rows - 1) / rows;
  return b <= 2 ? 1 : (b > 256 ? 256 : (int)b);
}

#define MOE_BY_EXPERTS_AS(CALL, VEC_)    \
  do {                                   \
    if (E <= 64) CALL(16, 1, VEC_);      \
    else if (E <= 128) CALL(16, 2, VEC_); \
    else if (E <= 256) CALL(16, 4, VEC_); \
    else if (E <= 512) CALL(32, 4, VEC_); \
    else CALL(64, 4, VEC_);              \
  } while (0)
#define MOE_BY_EXPERTS(CALL)            \
  do {                                  \
    if (E % 4 == 0)                     \
      MOE_BY_EXPERTS_AS(CALL, true);    \
    else                                \
      MOE_BY_EXPERTS_AS(CALL, false);   \
  } while (0)

hipError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T,
                               int E, int k, float coef, float* loss, int32_t* counts,
                               float* probs, int32_t* token_count, float* part_p, int32_t* part_c,
                               int32_t* part_n, LossTicket* ticket, hipStream_t st) {
  const int nb = balance_loss_blocks(T, E), rows = (int)(((long)T + nb - 1) / nb);
#define MOE_LOSS(L_, NC_, VEC_)                                                                \
  balance_loss_kernel<L_, NC_, VEC_><<<nb, kLossThreads, 0, st>>>(                             \
      logits, ids, mask, T, E, k, rows, coef, part_p, part_c, part_n, ticket, loss, counts,    \
      probs, token_count)
  MOE_BY_EXPERTS(MOE_LOSS);
#undef MOE_LOSS
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || nb == 1) return err;
#define MOE_FINISH(FE_, BLOCKS_)                                                              \
  balance_finish_kernel<FE_><<<BLOCKS_, 1024, 0, st>>>(part_p, part_c, part_n, ticket, nb, E, \
                                                       k, coef, loss, counts, probs, token_count)
  if (E <= 64)
    MOE_FINISH(64, 1);
  else if (E > 128 && E <= 256 && nb <= 128)
    MOE_FINISH(256, 1);
  else
    MOE_FINISH(128, (E + 127) / 128);
#undef MOE_FINISH
  return hipGetLastError();
}

hipError_t launch_router_grad(const float* logits, const int32_t* ids, const float* weights,
                              const float* grad_weights, const uint8_t* mask,
                              const int32_t* counts, const int32_t* token_count,
                              const float* grad_loss, float coef, int renorm, int T, int E, int k,
                              float* grad, hipStream_t st) {
  const bool gate = ids != nullptr, soft = grad_loss || !renorm;
  const int rows = kGradThreads / row_lanes(E);  // of a block at a time
  long nb = ((long)T + rows - 1) / rows;
  if (nb > 2048) nb = 2048;
#define MOE_GRAD_AS(L_, NC_, VEC_, SOFT_, GATE_)                                                 \
  router_grad_kernel<L_, NC_, VEC_, SOFT_, GATE_><<<(int)nb, kGradThreads, 0, st>>>(               \
      logits, ids, weights, grad_weights, mask, counts, token_count, grad_loss, coef, renorm, T, \
      E, k, grad)
#define MOE_GRAD(L_, NC_, VEC_)                      \
  do {                                               \
    if (!gate) MOE_GRAD_AS(L_, NC_, VEC_, true, false);  \
    else if (soft) MOE_GRAD_AS(L_, NC_, VEC_, true, true); \
    else MOE_GRAD_AS(L_, NC_, VEC_, false, true);        \
  } while (0)
  MOE_BY_EXPERTS(MOE_GRAD);
#undef MOE_GRAD
#undef MOE_GRAD_AS
  return hipGetLastError();
}

}  // namespace moe
