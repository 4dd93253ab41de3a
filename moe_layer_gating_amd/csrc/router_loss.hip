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
// large batches, by launch latency for small ones.  16 lanes hold a row
// (four rows per wave), each NC runs of 4 values, so the row reductions stay
// inside the 16-lane rows that DPP moves reach at full rate.  No sum depends
// on scheduling: blocks write partial sums that one block adds in block
// order, and the counts are integers.
#include "moe_common.h"

namespace moe {

constexpr int kRowLanes = 16;  // lanes per logits row (k <= 16: a lane per slot too)
constexpr int kLossThreads = 512;
constexpr int kGradThreads = 256;

// Sum / maximum over the 16 lanes of a DPP row; every lane gets it.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  return v;
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  return v;
}

// Value q = 4c + i of lane l is expert (c * 16 + l) * 4 + i when E is a
// multiple of 4 (16-byte loads), else (4c + i) * 16 + l.
template <bool VEC>
__device__ __forceinline__ int expert_of(int c, int i, int l) {
  return VEC ? (c * kRowLanes + l) * 4 + i : (4 * c + i) * kRowLanes + l;
}

template <int NC, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l,
                                         float (&v)[4 * NC], float fill) {
#pragma unroll
  for (int c = 0; c < NC; c++) {
    if (VEC) {
      const int e = expert_of<true>(c, 0, l);
      f32x4 r = {fill, fill, fill, fill};
      if (e < E) r = *reinterpret_cast<const f32x4*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; i++) v[4 * c + i] = r[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int e = expert_of<false>(c, i, l);
        v[4 * c + i] = e < E ? row[e] : fill;
      }
    }
  }
}

// Softmax of a row in place; NaN reads as -inf (as the gating reads it), and
// a row without a finite logit becomes all zero.
template <int N>
__device__ __forceinline__ void softmax_row(float (&v)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < N; q++) {
    v[q] = v[q] == v[q] ? v[q] : -INFINITY;
    m = fmaxf(m, v[q]);
  }
  m = row_max(m);
  if (m == -INFINITY) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < N; q++) {
    v[q] = expf(v[q] - m);
    s += v[q];
  }
  s = row_sum(s);
  const float inv = s > 0.f ? 1.0f / s : 0.f;
#pragma unroll
  for (int q = 0; q < N; q++) v[q] *= inv;
}

// Turns the sums over all tokens into the outputs; called by every thread of
// one block.  sum_p / sum_c: E sums in LDS.  red: one double per wave.
__device__ void finish_loss(const double* sum_p, const int* sum_c, int n, int E, int k, float coef,
                            float* loss, int32_t* counts, float* probs, int32_t* token_count,
                            double* red) {
  const double inv_n = n > 0 ? 1.0 / n : 0.0;
  double part = 0.0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const double p = sum_p[e] * inv_n;
    counts[e] = sum_c[e];
    probs[e] = (float)p;
    part += sum_c[e] * p;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) part += __shfl_xor(part, o);
  if (lane_id() == 0) red[threadIdx.x / kWave] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < (int)blockDim.x / kWave; w++) s += red[w];
    *loss = (float)((double)coef * E * s * inv_n / k);
    *token_count = n;
  }
}

// Block b sums the probabilities and counts of rows [b rows, (b + 1) rows)
// into part_p[b], part_c[b], part_n[b]; a single block writes the outputs.
template <int NC, bool VEC>
__global__ __launch_bounds__(kLossThreads) void balance_loss_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, int rows, float coef,
    float* __restrict__ part_p, int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ probs,
    int32_t* __restrict__ token_count) {
  constexpr int N = 4 * NC, NW = kLossThreads / kWave, E_MAX = N * kRowLanes;
  __shared__ float wsum[NW][E_MAX];
  __shared__ int hist[E_MAX];
  __shared__ double total[E_MAX];
  __shared__ double red[NW];
  __shared__ int n_live;
  const int t = threadIdx.x, l = t % kRowLanes, w = t / kWave;
  const int lo = blockIdx.x * rows, hi = min(T, lo + rows);
  for (int e = t; e < E; e += kLossThreads) hist[e] = 0;
  if (t == 0) n_live = 0;
  __syncthreads();

  float acc[N];
#pragma unroll
  for (int q = 0; q < N; q++) acc[q] = 0.f;
  int live = 0;
  for (int r = lo + t / kRowLanes; r < hi; r += kLossThreads / kRowLanes) {
    if (mask && !mask[r]) continue;  // the same for the row's 16 lanes
    float v[N];
    load_row<NC, VEC>(logits + (size_t)r * E, E, l, v, -INFINITY);
    softmax_row(v);
#pragma unroll
    for (int q = 0; q < N; q++) acc[q] += v[q];
    live++;
  }
  for (size_t f = (size_t)lo * k + t; f < (size_t)hi * k; f += kLossThreads) {
    const int e = ids[f];
    if ((unsigned)e < (unsigned)E && (!mask || mask[f / k])) atomicAdd(&hist[e], 1);
  }
  if (l == 0 && live) atomicAdd(&n_live, live);
  // the wave's four rows, then the waves in order
#pragma unroll
  for (int q = 0; q < N; q++) {
    acc[q] += __shfl_xor(acc[q], 16);
    acc[q] += __shfl_xor(acc[q], 32);
  }
  if (lane_id() < kRowLanes) {
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) wsum[w][expert_of<VEC>(c, i, l)] = acc[4 * c + i];
  }
  __syncthreads();
  const bool single = gridDim.x == 1;
  for (int e = t; e < E; e += kLossThreads) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < NW; q++) s += wsum[q][e];
    if (single) {
      total[e] = s;
    } else {
      part_p[(size_t)blockIdx.x * E + e] = s;
      part_c[(size_t)blockIdx.x * E + e] = hist[e];
    }
  }
  if (!single) {
    if (t == 0) part_n[blockIdx.x] = n_live;
    return;
  }
  __syncthreads();
  finish_loss(total, hist, n_live, E, k, coef, loss, counts, probs, token_count, red);
}

// One block adds the partial sums of n_parts blocks, in block order inside
// each of the S = 1024 / E_pad slices and then slice by slice.
__global__ __launch_bounds__(1024) void balance_finish_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
    const int32_t* __restrict__ part_n, int n_parts, int E, int e_pad, int k, float coef,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ probs,
    int32_t* __restrict__ token_count) {
  __shared__ double sp[1024];
  __shared__ int sc[1024];
  __shared__ double red[16];
  __shared__ int n_live;
  const int t = threadIdx.x, e = t % e_pad, s = t / e_pad, S = 1024 / e_pad;
  if (t == 0) n_live = 0;
  __syncthreads();
  double p = 0.0;
  int c = 0;
  if (e < E) {
#pragma unroll 8
    for (int b = s; b < n_parts; b += S) {
      p += part_p[(size_t)b * E + e];
      c += part_c[(size_t)b * E + e];
    }
  }
  sp[t] = p;
  sc[t] = c;
  for (int b = t; b < n_parts; b += 1024) atomicAdd(&n_live, part_n[b]);
  __syncthreads();
  if (t < e_pad) {
    for (int q = 1; q < S; q++) {
      p += sp[q * e_pad + t];
      c += sc[q * e_pad + t];
    }
    sp[t] = p;
    sc[t] = c;
  }
  __syncthreads();
  finish_loss(sp, sc, n_live, E, k, coef, loss, counts, probs, token_count, red);
}

// Gradient rows.  SOFT: the row's softmax is needed (the balance term, or the
// plain-softmax gating term); GATE: the gating term is added (ids, weights
// and grad_weights given).  The balance term is added when grad_loss is.
// A selected expert's term reaches the lane that owns the expert through the
// row's LDS copy: the lane of slot j adds the terms of every slot naming the
// same expert in slot order, and the first of those slots writes the sum.
template <int NC, bool VEC, bool SOFT, bool GATE>
__global__ __launch_bounds__(kGradThreads) void router_grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, const float* __restrict__ grad_weights,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ token_count, const float* __restrict__ grad_loss, float coef,
    int renorm, int T, int E, int k, float* __restrict__ grad) {
  constexpr int N = 4 * NC, E_MAX = N * kRowLanes, ROWS = kGradThreads / kRowLanes;
  __shared__ float sel[GATE ? ROWS : 1][GATE ? E_MAX : 1];
  const int t = threadIdx.x, l = t % kRowLanes, g = t / kRowLanes;
  float d[N];
  float scale = 0.f;
  if (SOFT && grad_loss) {
    const int n = *token_count;
    const double nk = (double)n * k, inv = n > 0 ? 1.0 / (nk * E) : 0.0;
    scale = n > 0 ? (float)((double)coef * E * *grad_loss / n) : 0.f;
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int e = expert_of<VEC>(c, i, l);
        d[4 * c + i] = e < E ? (float)(((double)counts[e] * E - nk) * inv) : 0.f;
      }
  } else {
#pragma unroll
    for (int q = 0; q < N; q++) d[q] = 0.f;
  }
  if (GATE) {
    for (int e = l; e < E_MAX; e += kRowLanes) sel[g][e] = 0.f;
    __syncthreads();
  }
  // every thread takes the same number of rounds (the block's rows may run out)
  for (int r0 = blockIdx.x * ROWS; r0 < T; r0 += gridDim.x * ROWS) {
    const int r = r0 + g;
    const bool live = r < T && (!mask || mask[r]);
    float v[N];
#pragma unroll
    for (int q = 0; q < N; q++) v[q] = 0.f;
    float S = 0.f;
    int id = -1;
    if (GATE) {
      float wg = 0.f, wj = 0.f;
      if (live && l < k) {
        const size_t f = (size_t)r * k + l;
        id = ids[f];
        wj = weights[f];
        wj = wj == wj ? wj : 0.f;  // the gating of a row without a finite logit
        if ((unsigned)id >= (unsigned)E) {
          id = -1;
          wj = 0.f;
        }
        wg = wj * grad_weights[f];
        if (id < 0) wg = 0.f;
      }
      S = row_sum(wg);
      const float term = renorm ? wg - wj * S : wg;
      float sum = 0.f;
      bool first = id >= 0;
      for (int j = 0; j < k; j++) {
        const int idj = __shfl(id, j, kRowLanes);
        const float tj = __shfl(term, j, kRowLanes);
        if (idj == id) {
          sum += tj;
          if (j < l) first = false;
        }
      }
      if (first) sel[g][id] = sum;
      __syncthreads();
    }
    if (live) {
      if (SOFT) {
        load_row<NC, VEC>(logits + (size_t)r * E, E, l, v, -INFINITY);
        softmax_row(v);
        float dp = 0.f;
#pragma unroll
        for (int q = 0; q < N; q++) dp = fmaf(d[q], v[q], dp);
        dp = row_sum(dp);
        const float s0 = GATE && !renorm ? S : 0.f;
#pragma unroll
        for (int q = 0; q < N; q++) v[q] *= scale * (d[q] - dp) - s0;
      }
      if (GATE) {
#pragma unroll
        for (int c = 0; c < NC; c++)
#pragma unroll
          for (int i = 0; i < 4; i++) v[4 * c + i] += sel[g][expert_of<VEC>(c, i, l)];
      }
    }
    if (r < T) {
      float* out = grad + (size_t)r * E;
#pragma unroll
      for (int c = 0; c < NC; c++) {
        if (VEC) {
          const int e = expert_of<true>(c, 0, l);
          if (e < E)
            *reinterpret_cast<f32x4*>(out + e) =
                f32x4{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int e = expert_of<false>(c, i, l);
            if (e < E) out[e] = v[4 * c + i];
          }
        }
      }
    }
    if (GATE) {
      __syncthreads();  // the row's reads are done
      if (id >= 0) sel[g][id] = 0.f;
      __syncthreads();
    }
  }
}

// Blocks of the loss kernel: at least 64 rows each (the finishing block reads
// E sums per block), at most one per CU.
int balance_loss_blocks(int T) {
  const int b = (T + 63) / 64;
  return T <= 128 ? 1 : (b > 256 ? 256 : b);
}

#define MOE_BY_EXPERTS(CALL)                                              \
  do {                                                                    \
    if (E % 4 == 0) {                                                     \
      if (E <= 64) CALL(1, true);                                         \
      else if (E <= 128) CALL(2, true);                                   \
      else if (E <= 256) CALL(4, true);                                   \
      else if (E <= 512) CALL(8, true);                                   \
      else CALL(16, true);                                                \
    } else {                                                              \
      if (E <= 64) CALL(1, false);                                        \
      else if (E <= 128) CALL(2, false);                                  \
      else if (E <= 256) CALL(4, false);                                  \
      else if (E <= 512) CALL(8, false);                                  \
      else CALL(16, false);                                               \
    }                                                                     \
  } while (0)

hipError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T,
                               int E, int k, float coef, float* loss, int32_t* counts,
                               float* probs, int32_t* token_count, float* part_p, int32_t* part_c,
                               int32_t* part_n, hipStream_t st) {
  const int nb = balance_loss_blocks(T), rows = (T + nb - 1) / nb;
#define MOE_LOSS(NC_, VEC_)                                                                    \
  balance_loss_kernel<NC_, VEC_><<<nb, kLossThreads, 0, st>>>(                                 \
      logits, ids, mask, T, E, k, rows, coef, part_p, part_c, part_n, loss, counts, probs,     \
      token_count)
  MOE_BY_EXPERTS(MOE_LOSS);
#undef MOE_LOSS
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || nb == 1) return err;
  int e_pad = 1;
  while (e_pad < E) e_pad *= 2;
  balance_finish_kernel<<<1, 1024, 0, st>>>(part_p, part_c, part_n, nb, E, e_pad, k, coef, loss,
                                            counts, probs, token_count);
  return hipGetLastError();
}

hipError_t launch_router_grad(const float* logits, const int32_t* ids, const float* weights,
                              const float* grad_weights, const uint8_t* mask,
                              const int32_t* counts, const int32_t* token_count,
                              const float* grad_loss, float coef, int renorm, int T, int E, int k,
                              float* grad, hipStream_t st) {
  const bool gate = ids != nullptr, soft = grad_loss || !renorm;
  long nb = ((long)T + kGradThreads / kRowLanes - 1) / (kGradThreads / kRowLanes);
  if (nb > 2048) nb = 2048;
#define MOE_GRAD_AS(NC_, VEC_, SOFT_, GATE_)                                                    \
  router_grad_kernel<NC_, VEC_, SOFT_, GATE_><<<(int)nb, kGradThreads, 0, st>>>(                \
      logits, ids, weights, grad_weights, mask, counts, token_count, grad_loss, coef, renorm, T, \
      E, k, grad)
#define MOE_GRAD(NC_, VEC_)                          \
  do {                                               \
    if (!gate) MOE_GRAD_AS(NC_, VEC_, true, false);  \
    else if (soft) MOE_GRAD_AS(NC_, VEC_, true, true); \
    else MOE_GRAD_AS(NC_, VEC_, false, true);        \
  } while (0)
  MOE_BY_EXPERTS(MOE_GRAD);
#undef MOE_GRAD
#undef MOE_GRAD_AS
  return hipGetLastError();
}

}  // namespace moe
