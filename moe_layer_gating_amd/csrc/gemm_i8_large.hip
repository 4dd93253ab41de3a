// gemm_i8_large.hip -- grouped int8 expert products for 8 or more pairs per
// expert: acc[p][n] = sum_k q_a[p][k] q_w[e][n][k] in 32-bit integers (exact:
// 128 * 127 * K < 2^31), scaled by fl32(s_a[p] * s_w[e][n]) in the epilogue.
//
// A block of 4 waves owns 256 weight rows (128 in the small form) and a tile of
// up to 256 sorted positions (64) of one expert, weights on the MFMA row side.
// Both operands go straight from memory into LDS (global_load_lds, 16 bytes a
// lane), 128 bytes of K of every row a stage, in two or three stage buffers.
//
// Why this shape.  v_mfma_i32_32x32x32_i8 takes 32 cycles for 64 bytes of
// fragments per lane pair, so LDS has to deliver fragments and take the loads
// besides: per stage of 256 x 256 the waves read (128 + 128) rows each as 2 x 2
// waves of 128 x 128 (1024 cycles of LDS at 128 B a cycle), the loads write 64
// KB (512), against 2048 cycles of MFMA.  With weights in registers and 32 rows
// a wave, as in the FP8 tiles, LDS alone needs 1.6 times the MFMA time.  The
// 256 accumulators a lane leave one wave per SIMD, so the main loop hides its
// own latencies: every instruction is placed by hand, the next K step's
// fragments are read under this step's MFMAs, and the one barrier of a stage
// sits a K step before its end, with 16 MFMAs still to issue behind it.
//
// Measured (the kernel alone, mean of 24 calls on two sets of operands, the
// fastest in brackets): 8 experts of 2048 pairs, 28672 x 4096 gate/up (3.85 Tops)
// 1.84 ms (1.75), 2.09 Pop/s; a square library product of the same type (16384 x
// 16384 x 8192) reaches 2.13 Pop/s on one such card: bound by the matrix units at
// the clock the power limit leaves.  4096 tokens on 256 experts (H 7168, I 2048):
// gate/up 1.66 ms (1.62), down 1.03 ms (1.01), bound by the memory system: 7.5
// and 3.8 GB of weights (1.19 and 0.60 ms at 6.3 TB/s) become 9.9 and 4.9 GB into
// the L2s, since each XCD reads a tile's rows, and the down projection writes
// 0.94 GB.  The register-ring tiles of gemm_tiles.hip, given int8 operands, took
// 2.55 ms for the first and 1.88 ms for the second gate/up.
#include <type_traits>

#include "moe_common.h"

namespace moe {

typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kLargeK = 128;  // codes of K per stage

// LDS slot of 16-byte chunk c of stage row r: c ^ swz_l(r).  A load's lanes
// write 8 rows in order (lane l takes row l / 8 and, as source, the chunk that
// belongs at slot l % 8); 8 consecutive rows at one chunk fall in 8 slots.
__device__ __forceinline__ int swz_l(int r) { return (r ^ (r >> 3)) & 7; }

__device__ __forceinline__ void dma16(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)src,
      (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// s_waitcnt with only vmcnt limited, to N / only lgkmcnt limited, to 0
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt has six bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xc07f); }

// Main loop of a block of 4 waves on ROWS weight rows and NPOS positions: each
// of the WR x WC waves accumulates RT x CT tiles of 32 x 32.  A stage is 128
// bytes of K of every row, loaded straight into one of NBUF LDS buffers
// (weights, then tokens).  ap: this lane's source of each weight load; tokens()
// gives those of the token loads, called once the first weights are on their
// way (it may wait for the rows' token numbers).
template <int ROWS, int NPOS, int NBUF, int WR, int WC, int RT, int CT, typename Tokens>
__device__ __forceinline__ void large_loop(const char* (&ap)[ROWS / 32], Tokens&& tokens,
                                           int n_stages, char* __restrict__ b0, char* __restrict__ b1,
                                           char* __restrict__ b2, i32x16 (&acc)[RT][CT]) {
  static_assert(NBUF == 2 || NBUF == 3, "buffers");
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r32 = lane & 31, hi = lane >> 5;
  const int wr = w / WC, wc = w % WC;
  constexpr int NA = ROWS / 32, NB = NPOS / 32, NL = NA + NB, kABytes = ROWS * kLargeK;
  const char* bp[NB];
  // the q-th of a stage's loads; the next one reads inc bytes further
  auto load = [&](char* buf, int q, int inc) {
    if (q < NA) {
      dma16(ap[q], buf + (w * NA + q) * 1024);
      ap[q] += inc;
    } else if (q < NL) {
      dma16(bp[q - NA], buf + kABytes + (w * NB + q - NA) * 1024);
      bp[q - NA] += inc;
    }
  };
  // K step kk of tile i: chunk 2 kk + lane / 32 of row 32 i + r32, kept at
  // slot chunk ^ swz(row); swz(row + 32 i) = swz(row) ^ 4 (i % 2), so every
  // address is one of four (kk ^ 2 (i % 2)) plus a constant
  const int rowa = wr * RT * 32 + r32, rowb = wc * CT * 32 + r32;
  const int la = rowa * kLargeK + ((hi ^ swz_l(rowa)) << 4);
  const int lb = kABytes + rowb * kLargeK + ((hi ^ swz_l(rowb)) << 4);
  i32x4 fa[2][RT], fb[2][CT];
  auto read = [&](const char* buf, int kk, int q, i32x4(&a)[RT], i32x4(&b)[CT]) {
    const int i = q < RT ? q : q - RT, sw = (kk ^ (2 * (i & 1))) << 5;
    if (q < RT)
      a[i] = *reinterpret_cast<const i32x4*>(buf + (la ^ sw) + i * 4096);
    else
      b[i] = *reinterpret_cast<const i32x4*>(buf + (lb ^ sw) + i * 4096);
  };
  auto mma = [&](int q, const i32x4(&a)[RT], const i32x4(&b)[CT]) {
    const int i = q / CT, j = q % CT;
    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
  };
  const int last = n_stages - 1;
  // stage by stage: the waits below count the loads issued after a stage's
  // (others in between only make them stricter)
#pragma unroll
  for (int n = 0; n < NBUF; n++) {
#pragma unroll
    for (int q = 0; q < NL; q++) {
      if (n == 0 && q == NA) tokens(bp);
      load(n == 0 ? b0 : n == 1 ? b1 : b2, q, last > n ? kLargeK : 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_vm<(NBUF - 1) * NL>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int q = 0; q < RT + CT; q++) read(b0, 0, q, fa[0], fb[0]);
  // Stage s in cur; s + 1 .. s + NBUF - 1 are in the other buffers or on their
  // way.  The barrier before the last K step finds every wave done reading
  // cur, which takes stage s + NBUF, and stage s + 1 landed.  (The order of the
  // instructions is fixed: each MFMA is followed by what can be issued in its
  // shadow, a fragment read and a load.  Past the last stage the loads repeat
  // it, so that the wait counts stay.)
  constexpr int M = RT * CT, R = RT + CT, S3 = M > R ? M : R, S4 = S3 > NL ? S3 : NL;
  auto stage = [&](char* cur, char* nxt, int s) {
#pragma unroll
    for (int kk = 0; kk < 3; kk++) {
#pragma unroll
      for (int q = 0; q < S3; q++) {
        if (q < M) mma(q, fa[kk & 1], fb[kk & 1]);
        if (q < R) read(cur, kk + 1, q, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_lgkm0();
    wait_vm<(NBUF - 2) * NL>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    const int inc = s + NBUF < last ? kLargeK : 0;
#pragma unroll
    for (int q = 0; q < S4; q++) {
      if (q < M) mma(q, fa[1], fb[1]);
      if (q < R) read(nxt, 0, q, fa[0], fb[0]);
      load(cur, q, inc);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int s = 0;
  if constexpr (NBUF == 2) {
    for (; s + 2 <= n_stages; s += 2) {
      stage(b0, b1, s);
      stage(b1, b0, s + 1);
    }
    if (s < n_stages) stage(b0, b1, s);
  } else {
    for (; s + 3 <= n_stages; s += 3) {
      stage(b0, b1, s);
      stage(b1, b2, s + 1);
      stage(b2, b0, s + 2);
    }
    if (s < n_stages) stage(b0, b1, s);
    if (s + 1 < n_stages) stage(b1, b2, s + 1);
  }
  // the last loads into LDS land, and every wave is done with its fragments:
  // LDS is free for the epilogue
  wait_lgkm0();
  wait_vm<0>();
  __builtin_amdgcn_s_barrier();
}

// Waves and their tiles, LDS stages.  256 positions: 2 x 2 waves of 128 x 128
// (the fewest fragment bytes per MFMA; 256 accumulators leave one wave per
// SIMD); fewer: a wave per quarter of the rows.
template <int ROWS, int NPOS>
struct LargeShape {
  static constexpr int NBUF = 3, WR = 4, WC = 1, RT = ROWS / 128, CT = NPOS / 32;
  static constexpr int STAGE = (ROWS + NPOS) * kLargeK;
};
template <>
struct LargeShape<256, 256> {
  static constexpr int NBUF = 2, WR = 2, WC = 2, RT = 4, CT = 4;
  static constexpr int STAGE = 512 * kLargeK;
};

// LDS: NBUF stage buffers of (ROWS + NPOS) rows of 128 bytes (the kernel's
// widest tiles decide their size), then the block's channel and row scales.
// The epilogue lays the output tile over the stage buffers, a row of 16-byte
// chunks per position with chunk c of row p at slot c ^ (p mod the row's
// chunks), and stores whole lines.
template <int ROWS, int BM>
struct LargeLds {
  static constexpr int N = BM < 256 ? BM : 128;
  char buf[LargeShape<ROWS, N>::NBUF * LargeShape<ROWS, N>::STAGE];
  float ws[ROWS], as[BM];
};

// bf16 of two floats (round to nearest even), the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Rows p < mt of CH chunks each from LDS to out, `pitch` bytes apart.
template <int CH>
__device__ __forceinline__ void store_rows(const char* buf, int mt, char* out, size_t pitch) {
  for (int i = threadIdx.x; i < mt * CH; i += 256) {
    const int p = i / CH, c = i % CH;
    *reinterpret_cast<uint4*>(out + p * pitch + c * 16) =
        *reinterpret_cast<const uint4*>(buf + p * CH * 16 + ((c ^ (p & (CH - 1))) << 4));
  }
}

template <int ROWS, int NPOS, int BM>
__device__ __forceinline__ void w13_large_tile(const char* b, const char* w13,
                                               const float* w13_scale, const int32_t* sorted_ids,
                                               const Tile& tl, int nb, int H, int I, int k,
                                               const float* xs, uint16_t* h,
                                               LargeLds<ROWS, BM>& L) {
  typedef LargeShape<ROWS, NPOS> S;
  const int t = threadIdx.x, lane = lane_id(), w = t / kWave;
  constexpr int NA = ROWS / 32, F = ROWS / 2;  // weight loads of a lane, features
  const char* ap[NA];
#pragma unroll
  for (int i = 0; i < NA; i++) {
    const int r = (w * NA + i) * 8 + (lane >> 3);
    const int f = nb * F + (r >> 1);
    const int row = (r & 1) ? I + f : f;
    ap[i] = w13 + ((size_t)tl.e * 2 * I + row) * H + (((lane & 7) ^ swz_l(r)) << 4);
  }
  int id[NPOS / 32], as_id = 0;
#pragma unroll
  for (int i = 0; i < NPOS / 32; i++)
    id[i] = sorted_ids[tl.p0 + min((w * (NPOS / 32) + i) * 8 + (lane >> 3), tl.mt - 1)];
  if (t < NPOS) as_id = sorted_ids[tl.p0 + min(t, tl.mt - 1)];
  float as_t = 0.f;
  auto tokens = [&](const char*(&bp)[NPOS / 32]) {
#pragma unroll
    for (int i = 0; i < NPOS / 32; i++) {
      const int r = (w * (NPOS / 32) + i) * 8 + (lane >> 3);
      bp[i] = b + (size_t)(id[i] / k) * H + (((lane & 7) ^ swz_l(r)) << 4);
    }
    if (t < NPOS) as_t = xs[as_id / k];
  };
  float ws_t = 0.f;
  if (t < ROWS) ws_t = w13_scale[(size_t)tl.e * 2 * I + (t & 1 ? I : 0) + nb * F + (t >> 1)];
  i32x16 acc[S::RT][S::CT];
#pragma unroll
  for (int i = 0; i < S::RT; i++)
#pragma unroll
    for (int j = 0; j < S::CT; j++)
#pragma unroll
      for (int q = 0; q < 16; q++) acc[i][j][q] = 0;
  static_assert(NPOS <= BM && S::NBUF * S::STAGE <= (int)sizeof(L.buf), "stage buffers");
  large_loop<ROWS, NPOS, S::NBUF, S::WR, S::WC, S::RT, S::CT>(
      ap, tokens, H / kLargeK, L.buf, L.buf + S::STAGE, L.buf + 2 * S::STAGE, acc);
  const int wr = w / S::WC, wc = w % S::WC, r32 = lane & 31, hi = lane >> 5;
  if (t < ROWS) L.ws[t] = ws_t;
  if (t < NPOS) L.as[t] = as_t;
  __syncthreads();
  float sx[S::CT];
#pragma unroll
  for (int j = 0; j < S::CT; j++) sx[j] = L.as[(wc * S::CT + j) * 32 + r32];
#pragma unroll
  for (int i = 0; i < S::RT; i++)
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int r = (wr * S::RT + i) * 32 + q * 8 + hi * 4;  // rows r .. r + 3: g u g u
      const f32x4 ws = *reinterpret_cast<const f32x4*>(&L.ws[r]);
#pragma unroll
      for (int j = 0; j < S::CT; j++) {
        // 2^x and the reciprocal of the hardware, a few fp32 steps off: h rounds
        // to bf16, 2^16 times coarser, right after; past -g = 126 ln 2 it may be 0
        float hv[2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const float g = (float)acc[i][j][4 * q + 2 * u] * (sx[j] * ws[2 * u]);
          const float up = (float)acc[i][j][4 * q + 2 * u + 1] * (sx[j] * ws[2 * u + 1]);
          const float e = __builtin_amdgcn_exp2f(g * -1.44269502f);
          hv[u] = g * __builtin_amdgcn_rcpf(1.0f + e) * up;
        }
        const int p = (wc * S::CT + j) * 32 + r32;
        *reinterpret_cast<uint32_t*>(L.buf + p * (2 * F) + (((r >> 4) ^ (p & (F / 8 - 1))) << 4) +
                                     (r & 15)) = pack_bf16(hv[0], hv[1]);
      }
    }
  __syncthreads();
  store_rows<F / 8>(L.buf, tl.mt, reinterpret_cast<char*>(h + (size_t)tl.p0 * I + nb * F),
                 (size_t)I * 2);
}

template <int ROWS, int NPOS, int BM>
__device__ __forceinline__ void w2_large_tile(const char* b, const char* w2, const float* w2_scale,
                                              const Tile& tl, int nb, int H, int I,
                                              const float* hs, float* y, LargeLds<ROWS, BM>& L) {
  typedef LargeShape<ROWS, NPOS> S;
  const int t = threadIdx.x, lane = lane_id(), w = t / kWave;
  constexpr int NA = ROWS / 32;
  const char* ap[NA];
#pragma unroll
  for (int i = 0; i < NA; i++) {
    const int r = (w * NA + i) * 8 + (lane >> 3);
    const int row = min(nb * ROWS + r, H - 1);
    ap[i] = w2 + ((size_t)tl.e * H + row) * I + (((lane & 7) ^ swz_l(r)) << 4);
  }
  auto tokens = [&](const char*(&bp)[NPOS / 32]) {
#pragma unroll
    for (int i = 0; i < NPOS / 32; i++) {
      const int r = (w * (NPOS / 32) + i) * 8 + (lane >> 3);
      bp[i] = b + (size_t)(tl.p0 + min(r, tl.mt - 1)) * I + (((lane & 7) ^ swz_l(r)) << 4);
    }
  };
  float ws_t = 0.f;
  if (t < ROWS) ws_t = w2_scale[(size_t)tl.e * H + min(nb * ROWS + t, H - 1)];
  float as_t = 0.f;
  if (t < NPOS) as_t = hs[tl.p0 + min(t, tl.mt - 1)];
  i32x16 acc[S::RT][S::CT];
#pragma unroll
  for (int i = 0; i < S::RT; i++)
#pragma unroll
    for (int j = 0; j < S::CT; j++)
#pragma unroll
      for (int q = 0; q < 16; q++) acc[i][j][q] = 0;
  static_assert(NPOS <= BM && S::NBUF * S::STAGE <= (int)sizeof(L.buf), "stage buffers");
  large_loop<ROWS, NPOS, S::NBUF, S::WR, S::WC, S::RT, S::CT>(
      ap, tokens, I / kLargeK, L.buf, L.buf + S::STAGE, L.buf + 2 * S::STAGE, acc);
  const int wr = w / S::WC, wc = w % S::WC, r32 = lane & 31, hi = lane >> 5;
  if (t < ROWS) L.ws[t] = ws_t;
  if (t < NPOS) L.as[t] = as_t;
  __syncthreads();
  float sh[S::CT];
#pragma unroll
  for (int j = 0; j < S::CT; j++) sh[j] = L.as[(wc * S::CT + j) * 32 + r32];
  // a position's row in LDS holds 512 bytes: 128 channels, 256 in two passes
  // (half of each wave's row tiles)
  constexpr int ES = 4, PASSES = ROWS * ES > 512 ? 2 : 1, RP = S::RT / PASSES;
  constexpr int ROWB = ROWS * ES / PASSES, CH = ROWB / 16;
#pragma unroll
  for (int pass = 0; pass < PASSES; pass++) {
    if (pass) __syncthreads();
#pragma unroll
    for (int i = 0; i < RP; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int r = (wr * S::RT + pass * RP + i) * 32 + q * 8 + hi * 4;
        const int o = ((wr * RP + i) * 32 + q * 8 + hi * 4) * ES;  // byte in the LDS row
        const f32x4 ws = *reinterpret_cast<const f32x4*>(&L.ws[r]);
#pragma unroll
        for (int j = 0; j < S::CT; j++) {
          float v[4];
#pragma unroll
          for (int u = 0; u < 4; u++)
            v[u] = (float)acc[pass * RP + i][j][4 * q + u] * (ws[u] * sh[j]);
          const int p = (wc * S::CT + j) * 32 + r32;
          *reinterpret_cast<f32x4*>(L.buf + p * ROWB + (((o >> 4) ^ (p & (CH - 1))) << 4)) =
              f32x4{v[0], v[1], v[2], v[3]};
        }
      }
    __syncthreads();
    // segments of RP * 32 channels per wave row
    constexpr int SEG = RP * 32 * ES / 16;  // chunks
    for (int i = t; i < tl.mt * CH; i += 256) {
      const int p = i / CH, c = i % CH;
      const int ch = nb * ROWS + (c / SEG * S::RT + pass * RP) * 32 + c % SEG * 16 / ES;
      if (ch < H)
        *reinterpret_cast<f32x4*>(y + (size_t)(tl.p0 + p) * H + ch) =
            *reinterpret_cast<const f32x4*>(L.buf + p * ROWB + ((c ^ (p & (CH - 1))) << 4));
    }
  }
}

// Block -> (tile, row block).  In order of the list, row block by row block
// (a tile's blocks are dealt over the XCDs, so that each L2 holds a share of
// the expert's weights for the expert's next tile); the 64-position tiles, of
// experts that mostly have one, are dealt to the XCDs in contiguous eighths
// instead, which reads a tile's rows into one L2.  Measured when it was
// chosen, list order against eighths: 4096 tokens on 256 experts 2.81 / 2.86 ms
// a layer (y in bf16 then), 8 experts of 2048 pairs 1.89 / 2.32 ms, down
// projection of 32 pairs per expert 0.688 / 0.667 ms.
template <int BM>
__device__ __forceinline__ bool large_work(const Tile* tiles, const int32_t* num_tiles, int n_blk,
                                           Tile* tl, int* nb) {
  if constexpr (BM == 64) {
    const int n = *num_tiles, x = blockIdx.x % 8, s = blockIdx.x / 8;
    const int tile = (int)((long)x * n / 8) + s / n_blk;
    *nb = s % n_blk;
    if (tile >= (int)((long)(x + 1) * n / 8)) return false;
    *tl = tiles[tile];
    return true;
  } else {
    const int tile = blockIdx.x / n_blk;  // below the list's capacity
    *nb = blockIdx.x - tile * n_blk;
    *tl = tiles[tile];  // beside the count, not after it
    return tile < *num_tiles;
  }
}

// The narrowest main loop that holds a tile of mt positions.
template <int BM, typename F>
__device__ __forceinline__ void by_width(int mt, F&& run) {
  if constexpr (BM == 256)
    if (mt > 128) return run(std::integral_constant<int, 256>{});
  if constexpr (BM >= 128)
    if (mt > 64) return run(std::integral_constant<int, 128>{});
  if (mt > 32) return run(std::integral_constant<int, 64>{});
  run(std::integral_constant<int, 32>{});
}

// BM = 64 (experts of few dozen pairs, bound by their weights' stream): 128
// rows, so that two blocks fit a CU and one streams while the other starts or
// ends; else 256 rows.
template <int BM>
constexpr int large_rows() {
  return BM == 64 ? 128 : 256;
}

template <int BM>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(BM == 64 ? 2 : 1, BM == 64 ? 2 : 1))) void w13_large_i8(
    const char* __restrict__ b, const char* __restrict__ w13, const float* __restrict__ w13_scale,
    const int32_t* __restrict__ sorted_ids, const Tile* __restrict__ tiles,
    const int32_t* __restrict__ num_tiles, int H, int I, int k, const float* __restrict__ xs,
    uint16_t* __restrict__ h) {
  constexpr int ROWS = large_rows<BM>();
  __shared__ __attribute__((aligned(16))) LargeLds<ROWS, BM> L;
  Tile tl;
  int nb;
  if (!large_work<BM>(tiles, num_tiles, 2 * I / ROWS, &tl, &nb)) return;
  by_width<BM>(tl.mt, [&](auto n) {
    w13_large_tile<ROWS, n.value, BM>(b, w13, w13_scale, sorted_ids, tl, nb, H, I, k, xs, h, L);
  });
}

template <int BM>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(BM == 64 ? 2 : 1, BM == 64 ? 2 : 1))) void w2_large_i8(
    const char* __restrict__ b, const char* __restrict__ w2, const float* __restrict__ w2_scale,
    const Tile* __restrict__ tiles, const int32_t* __restrict__ num_tiles, int H, int I,
    const float* __restrict__ hs, float* __restrict__ y) {
  constexpr int ROWS = large_rows<BM>();
  __shared__ __attribute__((aligned(16))) LargeLds<ROWS, BM> L;
  Tile tl;
  int nb;
  if (!large_work<BM>(tiles, num_tiles, (H + ROWS - 1) / ROWS, &tl, &nb)) return;
  by_width<BM>(tl.mt, [&](auto n) {
    w2_large_tile<ROWS, n.value, BM>(b, w2, w2_scale, tl, nb, H, I, hs, y, L);
  });
}

static long large_grid(int bm, long max_tiles, long channels) {
  const int rows = bm == 64 ? large_rows<64>() : large_rows<256>();
  return (bm == 64 ? (max_tiles + 7) / 8 * 8 : max_tiles) * ((channels + rows - 1) / rows);
}

hipError_t launch_w13_large_i8(int bm, const void* b, const void* w13, const float* w13_scale,
                               const int32_t* sorted_ids, const Tile* tiles,
                               const int32_t* num_tiles, int max_tiles, int H, int I, int k,
                               const float* xs, void* h, hipEvent_t e0, hipEvent_t e1,
                               hipStream_t st) {
  launch_on(bm == 64 ? w13_large_i8<64> : w13_large_i8<256>,
            dim3(large_grid(bm, max_tiles, 2L * I)), dim3(256), st, e0, e1, reinterpret_cast<const char*>(b),
            reinterpret_cast<const char*>(w13), w13_scale, sorted_ids, tiles, num_tiles, H, I, k,
            xs, reinterpret_cast<uint16_t*>(h));
  return hipGetLastError();
}

hipError_t launch_w2_large_i8(int bm, const void* b, const void* w2, const float* w2_scale,
                              const Tile* tiles, const int32_t* num_tiles, int max_tiles, int H,
                              int I, const float* hs, float* y, hipEvent_t e0, hipEvent_t e1,
                              hipStream_t st) {
  launch_on(bm == 64 ? w2_large_i8<64> : w2_large_i8<256>, dim3(large_grid(bm, max_tiles, H)),
            dim3(256), st, e0, e1, reinterpret_cast<const char*>(b),
            reinterpret_cast<const char*>(w2), w2_scale, tiles, num_tiles, H, I, hs, y);
  return hipGetLastError();
}

}  // namespace moe
