// Backward of the chunked gated delta rule (notation of kda_gdr.cuh; the prep pass and the state
// pass have run again and left S at every chunk's start and U in the workspace).
//
// Per chunk, with dO~ = scale dO, dS' the adjoint of the chunk's last state and X the gradient of
// the right-hand side beta R of (I + A) U = beta R:
//     dU = P^T dO~ + E (K dS'),   X = T^T dU,   dV = beta X
//     dS = G_C dS' + Q^T (G dO~) - K^T (G beta X)
// is the reverse state pass: the chunks of a sequence from the last to the first, with dS^T in
// registers exactly as the forward carries S^T (a warp owns 16 value channels).  It leaves dS' and
// X in the workspace, and the local pass, one CTA per (chunk, key head), computes for the key
// head's value heads in turn
//     dP = dO~ U^T,  dA = -X U^T,  W = dP D,  M = dA beta D (strictly lower)
//     dQ = G dO~ S^T + W K
//     dK = W^T Q + E U dS'^T - G beta X S^T + (M + M^T) K
//     dbeta_r = X_r.R_r + sum_i dA_ri D_ri k_r.k_i,   X_r.R_r = X_r.V_r - G_r (X S^T)_r.k_r
//     dgamma = row sums - column sums of (W Q K^T + M K K^T) + q.(G dO~ S^T) - G beta k.(X S^T) - e,
//              e = k.(E U dS'^T), and for the last token + sum e + G_C <dS', S>
//     dg = reverse cumulative sum of dgamma inside the chunk
// (each decay factor's gradient times the factor itself, so nothing is divided by a decay).
// dQ and dK of a key head's value heads are summed in registers in a fixed order.
//
// Per value head and chunk at D = 128 the reverse pass is 504 MMAs per 16 value channels, the local
// pass about 1000 per warp (8 warps); a chunk of the local pass reads 270 KB.  The local pass keeps S and dS' as split
// fp16 rows in shared memory (128 KB) with K, Q, U and dO or X, one persistent CTA per SM.
// Bounds: the reverse pass a chain's latency, 5.6 us a chunk (64 chains of 32 chunks on 128 SMs: 180 us);
// the local pass the latency of its steps with two warps per SM quarter (the tensor pipe is busy 34% of the
// time, 30% of the issue slots), 27 us a chunk and SM: 2048 chunks 371 us, 629 MB.  16 warps per CTA took
// 15% longer; one scale for all of W or M and of S or dS' instead of one per row would save 4%.
#include "kda_gdr.cuh"
#include "kda_tcgen05.cuh"

namespace kda {
namespace {
using namespace gdr;

// ---- reverse state pass ------------------------------------------------------------------
// It reads the prep pass's records alone, so it is launched behind the forward's start (whose CTAs
// wait for the prep pass before they let it go) and runs beside it on the SMs that are free; only its
// end waits for the forward's, on which the local pass counts.  One after the other / beside one
// another: 4096 tokens and 8 heads 750 / 523 us, ragged sequences of 1875 tokens and 8 heads 240 / 183.

// The form of whole heads: eight warps per CTA, 16 value channels each.
template <int D> struct ReverseSmem {
  static constexpr int NW = D / 16;
  static constexpr int kLd = 16 * NW + 4;  // row stride of the dO tile: no bank conflicts
  static constexpr uint32_t kK = 0, kQ = kQRows;
  static constexpr uint32_t kScales = kq_tile_bytes(D);
  static constexpr uint32_t kTp = kq_bytes(D);
  static constexpr uint32_t kDo = kTp + kTpBytes;  // [64][kLd] fp32
  static constexpr uint32_t kStage = kDo + C * kLd * 4;
  static constexpr uint32_t kBytes = 2 * kStage;
};

template <typename Tin, int D>
__global__ void __launch_bounds__(2 * D, 1)
gdr_reverse_kernel(const float *__restrict__ d_o, const float *d_sN, const int32_t *__restrict__ cu,
                   float scale, int N, int T, int HK, int HV, uint8_t *__restrict__ ws, Layout lay,
                   Tin *__restrict__ dv, float *d_s0, int *status) {
  using Sm = ReverseSmem<D>;
  constexpr int NW = Sm::NW, NT = D / 8, KK = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % HV, hk = h / (HV / HK);
  int n = blockIdx.x / HV;
  if (gridDim.x > 148 && cu && N <= kRanked) n = sequence_of_place(cu, N, T, n, status);
  const size_t nh = (size_t)n * HV + h;
  int bos, eos;
  seq_bounds(cu, n, T, status, bos, eos);
  const int chunks = (eos - bos + C - 1) / C;
  const long long slot0 = first_slot(bos, n);
  if (!in_range(status, slot0 + chunks, slots(N, T) + 1)) {
    wait_for_previous_kernel();
    return;
  }
  const int row = warp * 16 + lane / 4;  // this lane's value channels: row, row + 8
  const int col = 2 * (lane & 3);

  auto load = [&](int c) {
    const uint32_t st = sbase + (c & 1) * Sm::kStage;
    const long long slot = slot0 + c;
    cp_block(st, ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D), kq_bytes(D));
    cp_block(st + Sm::kTp, ws + lay.tp + (size_t)(slot * HV + h) * kTpBytes, kTpBytes);
    constexpr int kPieces = 4 * NW;
    const int t0 = bos + c * C, len = min(C, eos - t0);
    for (int i = threadIdx.x; i < C * kPieces; i += NW * 32) {
      const int r = i / kPieces, p = i % kPieces;
      cp16(st + Sm::kDo + (r * Sm::kLd + 4 * p) * 4,
           d_o + ((size_t)(t0 + min(r, len - 1)) * HV + h) * D + 4 * p, r < len);
    }
  };
  if (chunks > 0) load(chunks - 1);
  cp_commit();

  float s[NT][4];  // dS^T
  zero(s);
  if (d_sN) {
    const float *p = d_sN + (nh * D + row) * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float2 a = *reinterpret_cast<const float2 *>(p + 8 * i);
      const float2 b = *reinterpret_cast<const float2 *>(p + 8 * D + 8 * i);
      s[i][0] = a.x; s[i][1] = a.y; s[i][2] = b.x; s[i][3] = b.y;
    }
  }

  for (int c = chunks - 1; c >= 0; --c) {
    if (c > 0) load(c - 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    const uint32_t st = sbase + (c & 1) * Sm::kStage;
    const uint8_t *stp = smem + (c & 1) * Sm::kStage;
    const float2 kqs = *reinterpret_cast<const float2 *>(stp + Sm::kScales);
    const float *vec = reinterpret_cast<const float *>(stp + Sm::kTp + kVec);
    const int t0 = bos + c * C, len = min(C, eos - t0);
    const size_t rec = (size_t)(slot0 + c) * HV + h;

    {
      float *p = reinterpret_cast<float *>(ws + lay.dstate) + rec * D * D + row;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(8 * i + col + (e & 1)) * D + 8 * (e >> 1)] = s[i][e];
    }
    // (K dS')^T.
    float du[8][4];
    zero(du);
    Scale a0, a1;
    row_scales(s, a0, a1);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(s, kk, a0, a1, hi, lo);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t b[4];
        load_b<kKq>(b, st + Sm::kK, 16 * np, 16 * kk);
        mma(du[2 * np], hi, b[0], b[1]);
        mma(du[2 * np + 1], hi, b[2], b[3]);
        mma(du[2 * np], lo, b[0], b[1]);
        mma(du[2 * np + 1], lo, b[2], b[3]);
      }
    }
    // dO~^T of the warp's channels, and (P^T dO~)^T: P's rows are the sum's index, so their
    // scales go to the other operand.
    float x[8][4], t[8][4];
    const float *dop = reinterpret_cast<const float *>(stp + Sm::kDo) + warp * 16 + lane / 4;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[i][e] = scale * dop[(8 * i + col + (e & 1)) * Sm::kLd + 8 * (e >> 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = *reinterpret_cast<const float2 *>(vec + kVecP * C + 8 * i + col);
      t[i][0] = x[i][0] * p.x;
      t[i][1] = x[i][1] * p.y;
      t[i][2] = x[i][2] * p.x;
      t[i][3] = x[i][3] * p.y;
    }
    float pd[8][4];
    zero(pd);
    Scale r0, r1;
    row_scales(t, r0, r1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(t, kk, r0, r1, hi, lo);
#pragma unroll
      for (int np = 0; np <= kk; ++np) {
        uint32_t b[4], bl[4];
        load_bt(b, st + Sm::kTp + kP_HI, 16 * np, 16 * kk);
        load_bt(bl, st + Sm::kTp + kP_LO, 16 * np, 16 * kk);
        mma(pd[2 * np], hi, b[0], b[1]);
        mma(pd[2 * np + 1], hi, b[2], b[3]);
        mma(pd[2 * np], lo, b[0], b[1]);
        mma(pd[2 * np + 1], lo, b[2], b[3]);
        mma(pd[2 * np], hi, bl[0], bl[1]);
        mma(pd[2 * np + 1], hi, bl[2], bl[3]);
      }
    }
    // dU^T, its tokens scaled for T's rows.
    {
      const float f0 = a0.s * kqs.x, f1 = a1.s * kqs.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 e = *reinterpret_cast<const float2 *>(vec + kVecE * C + 8 * i + col);
        const float2 tt = *reinterpret_cast<const float2 *>(vec + kVecT * C + 8 * i + col);
        du[i][0] = tt.x * (e.x * (f0 * du[i][0]) + r0.s * pd[i][0]);
        du[i][1] = tt.y * (e.y * (f0 * du[i][1]) + r0.s * pd[i][1]);
        du[i][2] = tt.x * (e.x * (f1 * du[i][2]) + r1.s * pd[i][2]);
        du[i][3] = tt.y * (e.y * (f1 * du[i][3]) + r1.s * pd[i][3]);
      }
    }
    // X^T = (T^T dU)^T, in t.
    zero(t);
    row_scales(du, r0, r1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(du, kk, r0, r1, hi, lo);
#pragma unroll
      for (int np = 0; np <= kk; ++np) {
        uint32_t b[4], bl[4];
        load_bt(b, st + Sm::kTp + kT_HI, 16 * np, 16 * kk);
        load_bt(bl, st + Sm::kTp + kT_LO, 16 * np, 16 * kk);
        mma(t[2 * np], hi, b[0], b[1]);
        mma(t[2 * np + 1], hi, b[2], b[3]);
        mma(t[2 * np], lo, b[0], b[1]);
        mma(t[2 * np + 1], lo, b[2], b[3]);
        mma(t[2 * np], hi, bl[0], bl[1]);
        mma(t[2 * np + 1], hi, bl[2], bl[3]);
      }
    }
    {
      float *xp = reinterpret_cast<float *>(ws + lay.x) + rec * C * D + row;
      Tin *vp = dv + ((size_t)t0 * HV + h) * D + row;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 bt = *reinterpret_cast<const float2 *>(vec + kVecBeta * C + 8 * i + col);
        const float2 g = *reinterpret_cast<const float2 *>(vec + kVecG * C + 8 * i + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 8 * i + col + (e & 1);
          const float xx = (e >> 1 ? r1.s : r0.s) * t[i][e];
          xp[tok * D + 8 * (e >> 1)] = xx;
          const float dr = xx * (e & 1 ? bt.y : bt.x);
          if (tok < len) vp[(size_t)tok * HV * D + 8 * (e >> 1)] = from_f32<Tin>(dr);
          const float gg = e & 1 ? g.y : g.x;
          t[i][e] = gg * dr;    // G beta X
          x[i][e] *= gg;        // G dO~
        }
      }
    }
    // dS^T = G_C dS'^T + (G dO~)^T Q - (G beta X)^T K.
    Scale q0, q1;
    row_scales(x, q0, q1);
    row_scales(t, r0, r1);
    uint32_t qh[4][4], ql[4][4], kh[4][4], kl[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      split_a(x, kk, q0, q1, qh[kk], ql[kk]);
      split_a(t, kk, r0, r1, kh[kk], kl[kk]);
    }
    const float gl = vec[kVecG * C + C - 1];
    const float wq0 = q0.s * kqs.y, wq1 = q1.s * kqs.y, wk0 = -r0.s * kqs.x, wk1 = -r1.s * kqs.x;
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) {
      float aq[2][4], ak[2][4];
      zero(aq);
      zero(ak);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t b[4];
        load_bt<kKq>(b, st + Sm::kQ, 16 * j, 16 * kk);
        mma(aq[0], qh[kk], b[0], b[1]);
        mma(aq[1], qh[kk], b[2], b[3]);
        mma(aq[0], ql[kk], b[0], b[1]);
        mma(aq[1], ql[kk], b[2], b[3]);
        load_bt<kKq>(b, st + Sm::kK, 16 * j, 16 * kk);
        mma(ak[0], kh[kk], b[0], b[1]);
        mma(ak[1], kh[kk], b[2], b[3]);
        mma(ak[0], kl[kk], b[0], b[1]);
        mma(ak[1], kl[kk], b[2], b[3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float(&y)[4] = s[2 * j + i];
        y[0] = fmaf(gl, y[0], fmaf(wq0, aq[i][0], wk0 * ak[i][0]));
        y[1] = fmaf(gl, y[1], fmaf(wq0, aq[i][1], wk0 * ak[i][1]));
        y[2] = fmaf(gl, y[2], fmaf(wq1, aq[i][2], wk1 * ak[i][2]));
        y[3] = fmaf(gl, y[3], fmaf(wq1, aq[i][3], wk1 * ak[i][3]));
      }
    }
    __syncthreads();
  }
  cp_wait<0>();
  if (d_s0) {
    float *p = d_s0 + (nh * D + row) * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2 *>(p + 8 * i) = make_float2(s[i][0], s[i][1]);
      *reinterpret_cast<float2 *>(p + 8 * D + 8 * i) = make_float2(s[i][2], s[i][3]);
    }
  }
  wait_for_previous_kernel();  // this one's end is the forward's too
}

// The form of 64 value channels per CTA: warps 0-3 carry the chain, and warps 4-7 compute, one chunk ahead
// of them, what does not depend on dS': (P^T dO~)^T and ((G dO~)^T Q).  A lane of warp w + 4 holds the
// elements that the same lane of warp w adds, so they pass through shared memory lane by lane.  The
// chain is 316 of the 504 MMAs: 5.6 us a chunk, 6.9 with all of them on four warps (4 x 2048 tokens, 16
// heads: 749 -> 716 us).
template <int D> struct PairSmem {
  static constexpr int kLd = 64 + 4;                            // row stride of the dO tile
  static constexpr uint32_t kTile = (uint32_t)C * D * 2;         // K or Q
  static constexpr uint32_t kTri = 2 * kTriBytes;                // T or P, hi and lo
  static constexpr uint32_t kVecBytes = gdr::kVecs * C * 4;
  // the chain's stages: K, scales, T, vectors; the others': Q, scales, P, vectors, dO
  static constexpr uint32_t kScales = kTile, kTp = kScales + 128, kVecs = kTp + kTri, kDo = kVecs + kVecBytes;
  static constexpr uint32_t kChain = kDo, kSide = kDo + C * kLd * 4;
  static constexpr uint32_t kSides = 2 * kChain;
  static constexpr uint32_t kGiven = kSides + 2 * kSide;         // [4 warps][8 + D / 8][32] float4
  static constexpr uint32_t kBytes = kGiven + 4 * (8 + D / 8) * 32 * 16;
};

__device__ __forceinline__ void half_barrier(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}

template <typename Tin, int D>
__global__ void __launch_bounds__(256, 1)
gdr_reverse_pair_kernel(const float *__restrict__ d_o, const float *d_sN, const int32_t *__restrict__ cu,
                        float scale, int N, int T, int HK, int HV, uint8_t *__restrict__ ws, Layout lay,
                        Tin *__restrict__ dv, float *d_s0, int *status) {
  using Sm = PairSmem<D>;
  constexpr int NT = D / 8, KK = D / 16, kParts = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5, half = threadIdx.x >> 7;
  const int part = blockIdx.x % kParts, nh = blockIdx.x / kParts;
  const int n = nh / HV, h = nh % HV, hk = h / (HV / HK);
  int bos, eos;
  seq_bounds(cu, n, T, status, bos, eos);
  const int chunks = (eos - bos + C - 1) / C;
  const long long slot0 = first_slot(bos, n);
  if (!in_range(status, slot0 + chunks, slots(N, T) + 1)) {
    wait_for_previous_kernel();
    return;
  }
  const int row = (part * 4 + warp) * 16 + lane / 4;  // this lane's value channels: row, row + 8
  const int col = 2 * (lane & 3);
  float4 *given = reinterpret_cast<float4 *>(smem + Sm::kGiven) + warp * (8 + NT) * 32 + lane;

  auto copy = [&](uint32_t dst, const uint8_t *src, uint32_t bytes) {
    for (uint32_t i = tid * 16; i < bytes; i += 128 * 16) cp16(dst + i, src + i);
  };
  // Chunk c's stage of this half.
  const uint32_t stages = sbase + (half ? Sm::kSides : 0), stage_bytes = half ? Sm::kSide : Sm::kChain;
  auto load = [&](int c) {
    const uint32_t st = stages + (c & 1) * stage_bytes;
    const long long slot = slot0 + c;
    const uint8_t *kq = ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D);
    const uint8_t *tp = ws + lay.tp + (size_t)(slot * HV + h) * kTpBytes;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) copy(st + i * kQRows, kq + (2 * i + half) * kQRows, kQRows);
    copy(st + Sm::kScales, kq + kq_tile_bytes(D), 16);
    copy(st + Sm::kTp, tp + (half ? kP_HI : kT_HI), Sm::kTri);
    copy(st + Sm::kVecs, tp + kVec, Sm::kVecBytes);
    if (half == 0) return;
    const int t0 = bos + c * C, len = min(C, eos - t0);
    for (int i = tid; i < C * 16; i += 128) {
      const int r = i / 16, p = i % 16;
      cp16(st + Sm::kDo + (r * Sm::kLd + 4 * p) * 4,
           d_o + ((size_t)(t0 + min(r, len - 1)) * HV + h) * D + part * 64 + 4 * p, r < len);
    }
  };
  if (chunks > 0) load(chunks - 1);
  cp_commit();

  // Lower triangular products (X^T lower)^T: the tile's rows are the sum's index.
  auto triangular = [&](float (&out)[8][4], const float (&x)[8][4], uint32_t tile, Scale &r0, Scale &r1) {
    zero(out);
    row_scales(x, r0, r1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(x, kk, r0, r1, hi, lo);
#pragma unroll
      for (int np = 0; np <= kk; ++np) {
        uint32_t b[4], bl[4];
        load_bt(b, tile, 16 * np, 16 * kk);
        load_bt(bl, tile + kTriBytes, 16 * np, 16 * kk);
        mma(out[2 * np], hi, b[0], b[1]);
        mma(out[2 * np + 1], hi, b[2], b[3]);
        mma(out[2 * np], lo, b[0], b[1]);
        mma(out[2 * np + 1], lo, b[2], b[3]);
        mma(out[2 * np], hi, bl[0], bl[1]);
        mma(out[2 * np + 1], hi, bl[2], bl[3]);
      }
    }
  };

  if (half) {
    for (int c = chunks - 1; c >= -1; --c) {
      float pd[8][4], qd[NT][4];
      if (c >= 0) {
        if (c > 0) load(c - 1);
        cp_commit();
        cp_wait<1>();
        half_barrier(1);
        const uint32_t st = stages + (c & 1) * stage_bytes;
        const uint8_t *stp = smem + (st - sbase);
        const float qs = *reinterpret_cast<const float *>(stp + Sm::kScales + 4);
        const float *vec = reinterpret_cast<const float *>(stp + Sm::kVecs);
        const float *dop = reinterpret_cast<const float *>(stp + Sm::kDo) + warp * 16 + lane / 4;
        // dO~^T of the warp's channels, and (P^T dO~)^T: P's scales go to the other operand.
        float x[8][4], t[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 p = *reinterpret_cast<const float2 *>(vec + kVecP * C + 8 * i + col);
          const float2 g = *reinterpret_cast<const float2 *>(vec + kVecG * C + 8 * i + col);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = scale * dop[(8 * i + col + (e & 1)) * Sm::kLd + 8 * (e >> 1)];
            t[i][e] = (e & 1 ? p.y : p.x) * d;
            x[i][e] = (e & 1 ? g.y : g.x) * d;  // G dO~
          }
        }
        Scale r0, r1;
        triangular(pd, t, st + Sm::kTp, r0, r1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pd[i][0] *= r0.s; pd[i][1] *= r0.s; pd[i][2] *= r1.s; pd[i][3] *= r1.s;
        }
        row_scales(x, r0, r1);
        uint32_t hi[4][4], lo[4][4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) split_a(x, kk, r0, r1, hi[kk], lo[kk]);
        const float w0 = r0.s * qs, w1 = r1.s * qs;
        zero(qd);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint32_t b[4];
            load_bt(b, st, 16 * j, 16 * kk);
            mma(qd[2 * j], hi[kk], b[0], b[1]);
            mma(qd[2 * j + 1], hi[kk], b[2], b[3]);
            mma(qd[2 * j], lo[kk], b[0], b[1]);
            mma(qd[2 * j + 1], lo[kk], b[2], b[3]);
          }
#pragma unroll
          for (int i = 2 * j; i < 2 * j + 2; ++i) {
            qd[i][0] *= w0; qd[i][1] *= w0; qd[i][2] *= w1; qd[i][3] *= w1;
          }
        }
      }
      __syncthreads();  // the chain has taken what was given for the chunk before
      if (c >= 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) given[i * 32] = make_float4(pd[i][0], pd[i][1], pd[i][2], pd[i][3]);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          given[(8 + i) * 32] = make_float4(qd[i][0], qd[i][1], qd[i][2], qd[i][3]);
      }
      __syncthreads();
    }
    cp_wait<0>();
    wait_for_previous_kernel();
    return;
  }

  float s[NT][4];  // dS^T
  zero(s);
  if (d_sN) {
    const float *p = d_sN + ((size_t)nh * D + row) * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float2 a = *reinterpret_cast<const float2 *>(p + 8 * i);
      const float2 b = *reinterpret_cast<const float2 *>(p + 8 * D + 8 * i);
      s[i][0] = a.x; s[i][1] = a.y; s[i][2] = b.x; s[i][3] = b.y;
    }
  }
  __syncthreads();
  __syncthreads();
  for (int c = chunks - 1; c >= 0; --c) {
    if (c > 0) load(c - 1);
    cp_commit();
    cp_wait<1>();
    half_barrier(0);
    const uint32_t st = stages + (c & 1) * stage_bytes;
    const uint8_t *stp = smem + (st - sbase);
    const float ks = *reinterpret_cast<const float *>(stp + Sm::kScales);
    const float *vec = reinterpret_cast<const float *>(stp + Sm::kVecs);
    const int t0 = bos + c * C, len = min(C, eos - t0);
    const size_t rec = (size_t)(slot0 + c) * HV + h;
    {
      float *p = reinterpret_cast<float *>(ws + lay.dstate) + rec * D * D + row;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(8 * i + col + (e & 1)) * D + 8 * (e >> 1)] = s[i][e];
    }
    // (K dS')^T.
    float du[8][4];
    zero(du);
    Scale a0, a1, r0, r1;
    row_scales(s, a0, a1);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(s, kk, a0, a1, hi, lo);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t b[4];
        load_b(b, st, 16 * np, 16 * kk);
        mma(du[2 * np], hi, b[0], b[1]);
        mma(du[2 * np + 1], hi, b[2], b[3]);
        mma(du[2 * np], lo, b[0], b[1]);
        mma(du[2 * np + 1], lo, b[2], b[3]);
      }
    }
    // dU^T, its tokens scaled for T's rows.
    {
      const float f0 = a0.s * ks, f1 = a1.s * ks;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 e = *reinterpret_cast<const float2 *>(vec + kVecE * C + 8 * i + col);
        const float2 tt = *reinterpret_cast<const float2 *>(vec + kVecT * C + 8 * i + col);
        const float4 pd = given[i * 32];
        du[i][0] = tt.x * (e.x * (f0 * du[i][0]) + pd.x);
        du[i][1] = tt.y * (e.y * (f0 * du[i][1]) + pd.y);
        du[i][2] = tt.x * (e.x * (f1 * du[i][2]) + pd.z);
        du[i][3] = tt.y * (e.y * (f1 * du[i][3]) + pd.w);
      }
    }
    // X^T = (T^T dU)^T.
    float t[8][4];
    triangular(t, du, st + Sm::kTp, r0, r1);
    {
      float *xp = reinterpret_cast<float *>(ws + lay.x) + rec * C * D + row;
      Tin *vp = dv + ((size_t)t0 * HV + h) * D + row;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 bt = *reinterpret_cast<const float2 *>(vec + kVecBeta * C + 8 * i + col);
        const float2 g = *reinterpret_cast<const float2 *>(vec + kVecG * C + 8 * i + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 8 * i + col + (e & 1);
          const float xx = (e >> 1 ? r1.s : r0.s) * t[i][e];
          xp[tok * D + 8 * (e >> 1)] = xx;
          const float dr = xx * (e & 1 ? bt.y : bt.x);
          if (tok < len) vp[(size_t)tok * HV * D + 8 * (e >> 1)] = from_f32<Tin>(dr);
          t[i][e] = (e & 1 ? g.y : g.x) * dr;  // G beta X
        }
      }
    }
    // dS^T = G_C dS'^T + (G dO~)^T Q - (G beta X)^T K.
    row_scales(t, r0, r1);
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) split_a(t, kk, r0, r1, hi[kk], lo[kk]);
    const float gl = vec[kVecG * C + C - 1];
    const float w0 = -r0.s * ks, w1 = -r1.s * ks;
#pragma unroll
    for (int j = 0; j < NT / 4; ++j) {
      float acc[4][4];
      zero(acc);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int np = 0; np < 2; ++np) {
          uint32_t b[4];
          load_bt(b, st, 32 * j + 16 * np, 16 * kk);
          mma(acc[2 * np], hi[kk], b[0], b[1]);
          mma(acc[2 * np + 1], hi[kk], b[2], b[3]);
          mma(acc[2 * np], lo[kk], b[0], b[1]);
          mma(acc[2 * np + 1], lo[kk], b[2], b[3]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float(&y)[4] = s[4 * j + i];
        const float4 qd = given[(8 + 4 * j + i) * 32];
        y[0] = fmaf(gl, y[0], fmaf(w0, acc[i][0], qd.x));
        y[1] = fmaf(gl, y[1], fmaf(w0, acc[i][1], qd.y));
        y[2] = fmaf(gl, y[2], fmaf(w1, acc[i][2], qd.z));
        y[3] = fmaf(gl, y[3], fmaf(w1, acc[i][3], qd.w));
      }
    }
    __syncthreads();
    __syncthreads();
  }
  cp_wait<0>();
  if (d_s0) {
    float *p = d_s0 + ((size_t)nh * D + row) * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2 *>(p + 8 * i) = make_float2(s[i][0], s[i][1]);
      *reinterpret_cast<float2 *>(p + 8 * D + 8 * i) = make_float2(s[i][2], s[i][3]);
    }
  }
  wait_for_previous_kernel();
}

// ---- local pass --------------------------------------------------------------------------

constexpr int kLocalThreads = 256;

__device__ __forceinline__ uint32_t times2(uint32_t x, __half2 f) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x), f);
  return *reinterpret_cast<const uint32_t *>(&y);
}

template <int D> struct LocalSmem {
  static constexpr uint32_t kK = 0, kQ = kQRows;
  static constexpr uint32_t kS = kq_tile_bytes(D);   // S, D rows (key channels)
  static constexpr uint32_t kD = kS + D * D * 4;     // dS'
  static constexpr uint32_t kU = kD + D * D * 4;     // U, 64 rows; later W hi, lo, M hi, lo
  static constexpr uint32_t kUBytes = C * D * 4 > 4 * kTriBytes ? C * D * 4 : 4 * kTriBytes;
  static constexpr uint32_t kA = kU + kUBytes;       // dO, then X, 64 rows; later the sums
  static constexpr uint32_t kSmall = kA + C * D * 4;
  struct Sums {                        // in kA
    float rows[2][C];                  // per half: what dgamma takes per row
    float cols[4][C];                  // per row block: column sums
    float tail[2][C], zk[2][C], db[2][C];
    float cross[8];
    float row_max[2][2][C];            // of W and M, per half
    float most[8][2];                  // and per warp
    float scale[2][C + 1];             // of W's and M's rows, and the largest
    alignas(4) __half rel[2][C];       // the rows' over the largest
  };
  static_assert(sizeof(Sums) <= C * D * 4, "the sums fit where X was");
  struct Small {
    alignas(16) float scales[2][D];      // of the rows (key channels) of S and of dS'
    alignas(16) float2 gamma[C];
    float beta[C], us[C], as[C], xv[C];  // us, as: scales of U's and of dO's or X's rows
    alignas(16) float kq[4];             // the tile's two scales
    uint64_t states, rest;               // S and dS' have landed; U (and K and Q) have
  };
  static constexpr uint32_t kBytes = kSmall + sizeof(Small);
};

// One step of a reduction that folds 2 n values a lane to n: a lane keeps the lower or the upper half, by
// its bit `off`, each the larger of its own and the other lane's.
template <int n> __device__ __forceinline__ void fold_max(float *x, int off) {
  const bool upper = threadIdx.x & off;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[i + n], off);
    x[i] = fmaxf(upper ? x[i + n] : x[i], other);
  }
}
__device__ __forceinline__ float max_abs4(const float4 &x, float m) {
  return fmaxf(fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
}

// Sum over the eight lanes that share accumulator columns.
__device__ __forceinline__ float col_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// fp16 pair at (row, column col of 8-column block c8) of the K and Q tile.
__device__ __forceinline__ float2 tile_pair(const uint8_t *tile, int row, int c8, int col) {
  const uint32_t u = *reinterpret_cast<const uint32_t *>(tile + tile_off<kKq>(row, c8) + 2 * col);
  return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// Persistent: a CTA takes every gridDim.x-th (chunk, key head).  S and dS' of the next (chunk,
// head) are fetched as soon as this one's have been used, behind the products that are left.
// A warp splits its rows of S and of dS' in their places (row_off; whole rows, so no block barrier), each
// row with its own power of two, and sums their products on the way.  `rows` is a multiple of four accesses
// of 128 / D rows.
template <int D>
__device__ __forceinline__ float split_states_in_place(uint8_t *s, uint8_t *ds, int row0, int rows,
                                                       float (*scales)[D]) {
  constexpr int LR = D / 4, RP = 32 / LR;  // lanes per row, rows per warp access
  const int lane = threadIdx.x & 31, rl = lane / LR, cl = lane % LR;
  float cross = 0.f;
#pragma unroll 1
  for (int i = 0; i < rows; i += 4 * RP) {
    float4 x[2][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = (row0 + i + k * RP + rl) * 4 * D + 16 * cl;
      x[0][k] = *reinterpret_cast<const float4 *>(s + at);
      x[1][k] = *reinterpret_cast<const float4 *>(ds + at);
    }
    // The rows' largest: folded to one row of one matrix per lane, and exchanged.
    float big[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) big[k] = max_abs4(x[k >> 2][k & 3], 0.f);
    fold_max<4>(big, LR / 2);
    fold_max<2>(big, LR / 4);
    fold_max<1>(big, LR / 8);
#pragma unroll
    for (int off = LR / 16; off > 0; off >>= 1) big[0] = fmaxf(big[0], __shfl_xor_sync(0xffffffffu, big[0], off));
    const Scale mine = scale_of(big[0]);
    if (cl % (LR / 8) == 0) {
      const int j = cl / (LR / 8);
      scales[j >> 2][row0 + i + (j & 3) * RP + rl] = mine.s;
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 &a = x[0][k], &b = x[1][k];
      cross += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
      const uint32_t o = row_off<D>(row0 + i + k * RP + rl, cl >> 1) + 8 * (cl & 1);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const float4 &y = x[which][k];
        const float inv = __shfl_sync(0xffffffffu, mine.inv, rl * LR + (4 * which + k) * (LR / 8));
        uint8_t *to = (which ? ds : s) + o;
        uint2 hi, lo;
        split2(y.x, y.y, inv, hi.x, lo.x);
        split2(y.z, y.w, inv, hi.y, lo.y);
        *reinterpret_cast<uint2 *>(to) = hi;
        *reinterpret_cast<uint2 *>(to + 2 * D) = lo;
      }
    }
    __syncwarp();
  }
  return cross;
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kLocalThreads, 1)
gdr_local_kernel(const Tin *__restrict__ v, const float *__restrict__ g,
                 const float *__restrict__ beta, const float *__restrict__ d_o,
                 const int32_t *__restrict__ cu, float scale, int N, int T, int HK, int HV,
                 const uint8_t *__restrict__ ws, Layout lay, Tin *__restrict__ dq,
                 Tin *__restrict__ dk, float *__restrict__ dg, float *__restrict__ dbeta,
                 int *status) {
  using Sm = LocalSmem<D>;
  constexpr int KK = D / 16;       // k-steps over the head dimension
  constexpr int NH = D / 16;       // 8-column blocks of a warp's half of the key channels
  constexpr int LR = D / 4;        // lanes per row of an fp32 matrix
  constexpr int RP = 32 / LR;      // rows per warp access
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  typename Sm::Small &sm = *reinterpret_cast<typename Sm::Small *>(smem + Sm::kSmall);
  typename Sm::Sums &sums = *reinterpret_cast<typename Sm::Sums *>(smem + Sm::kA);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = warp & 3, half = warp >> 2;       // token rows 16 m .., half of the columns
  const int r0 = 16 * m + lane / 4, r1 = r0 + 8, col = 2 * (lane & 3);
  const int rl = lane / LR, cl = lane % LR;       // row and quad of a lane in a warp access
  const int group = HV / HK;
  const long long items = slots(N, T) * HK;

  // The next item at or after `item` whose slot has a chunk; `items` if there is none.
  int bos = 0, eos = 0, c = 0, n = 0;
  auto next_item = [&](long long item) {
    while (item < items &&
           !(chunk_of_slot(cu, N, T, item / HK, status, n, bos, eos, c) &&
             in_range(status, item / HK, slots(N, T))))
      item += gridDim.x;
    return item;
  };
  // One thread: S and dS' of a (chunk, head), 4 D^2 bytes each as the state passes left them.
  auto fetch_states = [&](long long item, int j) {
    const size_t rec = (size_t)(item / HK) * HV + item % HK * group + j;
    tc::mbar_arrive_expect_tx(&sm.states, 2 * D * D * 4);
    tc::bulk_load(smem + Sm::kS, ws + lay.state + rec * D * D * 4, D * D * 4, &sm.states);
    tc::bulk_load(smem + Sm::kD, ws + lay.dstate + rec * D * D * 4, D * D * 4, &sm.states);
  };
  // A warp's 8 of 64 rows, held in registers, with a scale per row.
  constexpr int kHeld = 8 / RP;
  auto store_rows = [&](const float4 (&x)[kHeld], uint32_t base, float *scales) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int row = 8 * warp + k * RP + rl;
      float big = max_abs4(x[k], 0.f);
#pragma unroll
      for (int off = LR / 2; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
      const Scale s = scale_of(big);
      uint2 hi, lo;
      split2(x[k].x, x[k].y, s.inv, hi.x, lo.x);
      split2(x[k].z, x[k].w, s.inv, hi.y, lo.y);
      const uint32_t o = base + row_off<D>(row, cl >> 1) + 8 * (cl & 1);
      *reinterpret_cast<uint2 *>(smem + o) = hi;
      *reinterpret_cast<uint2 *>(smem + o + 2 * D) = lo;
      if (cl == 0) scales[row] = s.s;
    }
  };
  // The same for rows that lie in their place as fp32.
  auto split_own = [&](uint32_t base, float *scales) {
    float4 x[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      x[k] = *reinterpret_cast<const float4 *>(smem + base + (8 * warp + k * RP + rl) * 4 * D + 16 * cl);
    __syncwarp();
    store_rows(x, base, scales);
  };

  // A (chunk, head)'s g (warp 7) or beta (warp 6), an item ahead like its states.
  float small[2];
  auto fetch_small = [&](int t0, int len, int h) {
    if (warp == 7) {
      const float *g0 = g + (size_t)t0 * HV + h;
      small[0] = load_g(g0, HV, 2 * lane, len);
      small[1] = load_g(g0, HV, 2 * lane + 1, len);
    } else if (warp == 6) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        small[i] = lane + 32 * i < len ? __ldg(beta + (size_t)(t0 + lane + 32 * i) * HV + h) : 0.f;
    }
  };
  if (tid == 0) {
    tc::mbar_init(&sm.states, 1);
    tc::mbar_init(&sm.rest, 1);
    tc::fence_mbar_init();
  }
  __syncthreads();
  uint32_t par = 0;  // of both barriers: one phase each per (chunk, head)
  long long item = next_item(blockIdx.x);
  if (tid == 0 && item < items) fetch_states(item, 0);
  if (item < items) fetch_small(bos + c * C, min(C, eos - bos - c * C), (int)(item % HK) * group);
  while (item < items) {
    const long long slot = item / HK;
    const int hk = (int)(item % HK);
    const int t0 = bos + c * C, len = min(C, eos - t0);
    float aq[NH][4], ak[NH][4];  // dQ, dK: rows r0, r1; columns 8 (half NH + i) + col
    zero(aq);
    zero(ak);
    long long following = items;
    for (int j = 0; j < group; ++j) {
      const int h = hk * group + j;
      const size_t rec = (size_t)(slot * HV + h);
      const float *Ug = reinterpret_cast<const float *>(ws + lay.u) + rec * C * D;
      const float *Xg = reinterpret_cast<const float *>(ws + lay.x) + rec * C * D;
      const float *Og = d_o + ((size_t)t0 * HV + h) * D;
      // U (with the first head K and Q) and dO on their way behind S and dS'.
      if (tid == 0) {
        const uint8_t *kq = ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D);
        tc::mbar_arrive_expect_tx(&sm.rest, C * D * 4 + (j == 0 ? kq_tile_bytes(D) + 16 : 0));
        tc::bulk_load(smem + Sm::kU, Ug, C * D * 4, &sm.rest);
        if (j == 0) {
          tc::bulk_load(smem, kq, kq_tile_bytes(D), &sm.rest);
          tc::bulk_load(sm.kq, kq + kq_tile_bytes(D), 16, &sm.rest);
        }
      }
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int row = 8 * warp + k * RP + rl;
        cp16(sb + Sm::kA + row * 4 * D + 16 * cl, Og + (size_t)min(row, len - 1) * HV * D + 4 * cl, row < len);
      }
      cp_commit();
      if (warp == 7) {
        gamma_of(small[0], small[1], sm.gamma);
      } else if (warp == 6) {
        sm.beta[lane] = small[0];
        sm.beta[lane + 32] = small[1];
      }
      // S and dS', a power of two per key channel, and <dS', S>.
      if (!tc::wait_all(&sm.states, par, status)) {
        if (tid == 0) {  // what is in flight lands before the CTA's memory goes
          tc::drain(&sm.states);
          tc::drain(&sm.rest);
        }
        cp_wait<0>();
        __syncthreads();
        return;
      }
      constexpr int kRows = D / 8;  // of each matrix per warp
      float cross = split_states_in_place<D>(smem + Sm::kS, smem + Sm::kD, kRows * warp, kRows, sm.scales);
      cp_wait<0>();  // this thread's part of its own warp's rows of dO
      __syncwarp();
      split_own(Sm::kA, sm.as);
      if (!tc::wait_all(&sm.rest, par, status)) {
        if (tid == 0) tc::drain(&sm.rest);
        __syncthreads();
        return;
      }
      split_own(Sm::kU, sm.us);
      __syncthreads();
      par ^= 1;
      // X and V, on their way behind the first products.
      float4 x[kHeld];
      uint2 vx[kHeld];
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int row = 8 * warp + k * RP + rl;
        x[k] = __ldg(reinterpret_cast<const float4 *>(Xg + row * D) + cl);
        vx[k] = make_uint2(0u, 0u);
        if (row < len)
          vx[k] = __ldg(reinterpret_cast<const uint2 *>(v + ((size_t)(t0 + row) * HV + h) * D) + cl);
      }
      const float ks = sm.kq[0], qs = sm.kq[1];

      float dp[4][4], da[4][4];  // rows r0, r1; columns 32 half + 8 i + col
      // z = (a matrix of 64 rows) (a matrix of key channels)^T, this warp's rows and columns, and
      // with_u: y = the same 64 rows times U^T, in the blocks that reach below the diagonal.
      auto rows_times = [&](uint32_t a, uint32_t b, float (&z)[NH][4], float (&y)[4][4], bool with_u) {
        zero(z);
        if (with_u) zero(y);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          uint32_t hi[4], lo[4];
          load_rows_a<D>(hi, sb + a, 16 * m, 16 * kk, false);
          load_rows_a<D>(lo, sb + a, 16 * m, 16 * kk, true);
#pragma unroll
          for (int np = 0; np < NH / 2; ++np) {
            uint32_t bh[4], bl[4];
            load_rows_b<D>(bh, sb + b, half * (D / 2) + 16 * np, 16 * kk, false);
            load_rows_b<D>(bl, sb + b, half * (D / 2) + 16 * np, 16 * kk, true);
            mma(z[2 * np], hi, bh[0], bh[1]);
            mma(z[2 * np + 1], hi, bh[2], bh[3]);
            mma(z[2 * np], lo, bh[0], bh[1]);
            mma(z[2 * np + 1], lo, bh[2], bh[3]);
            mma(z[2 * np], hi, bl[0], bl[1]);
            mma(z[2 * np + 1], hi, bl[2], bl[3]);
          }
          if (!with_u) continue;
#pragma unroll
          for (int np = 0; np < 2; ++np) {
            if (2 * half + np > m) break;
            uint32_t bh[4], bl[4];
            load_rows_b<D>(bh, sb + Sm::kU, 32 * half + 16 * np, 16 * kk, false);
            load_rows_b<D>(bl, sb + Sm::kU, 32 * half + 16 * np, 16 * kk, true);
            mma(y[2 * np], hi, bh[0], bh[1]);
            mma(y[2 * np + 1], hi, bh[2], bh[3]);
            mma(y[2 * np], lo, bh[0], bh[1]);
            mma(y[2 * np + 1], lo, bh[2], bh[3]);
            mma(y[2 * np], hi, bl[0], bl[1]);
            mma(y[2 * np + 1], hi, bl[2], bl[3]);
          }
        }
      };
      auto scale_y = [&](float (&y)[4][4], float f0, float f1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = *reinterpret_cast<const float2 *>(sm.us + 32 * half + 8 * i + col);
          y[i][0] *= f0 * u.x; y[i][1] *= f0 * u.y;
          y[i][2] *= f1 * u.x; y[i][3] *= f1 * u.y;
        }
      };
      // z's rows times f0, f1 and its columns times their key channels' scales.
      auto scale_z = [&](float (&z)[NH][4], int which, float f0, float f1) {
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          const float2 s = *reinterpret_cast<const float2 *>(sm.scales[which] + half * (D / 2) + 8 * i + col);
          z[i][0] *= f0 * s.x; z[i][1] *= f0 * s.y;
          z[i][2] *= f1 * s.x; z[i][3] *= f1 * s.y;
        }
      };
      // Row dots of z with the rows of a tile (keys or queries), summed over this warp's columns.
      auto row_dots = [&](const float (&z)[NH][4], uint32_t tile, float f, float &d0, float &d1) {
        d0 = d1 = 0.f;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          const float2 a = tile_pair(smem + tile, r0, half * NH + i, col);
          const float2 b = tile_pair(smem + tile, r1, half * NH + i, col);
          d0 += z[i][0] * a.x + z[i][1] * a.y;
          d1 += z[i][2] * b.x + z[i][3] * b.y;
        }
        d0 = f * quad_sum(d0);
        d1 = f * quad_sum(d1);
      };
      float z[NH][4];
      float rg0, rg1, zk0, zk1, tl0, tl1;
      const float2 gr[2] = {sm.gamma[r0], sm.gamma[r1]};
      const float g0 = ex2_approx(gr[0].x + gr[0].y), g1 = ex2_approx(gr[1].x + gr[1].y);
      const float b0 = sm.beta[r0], b1 = sm.beta[r1];
      {  // dO~ S^T and dO~ U^T
        rows_times(Sm::kA, Sm::kS, z, dp, true);
        const float f0 = scale * sm.as[r0], f1 = scale * sm.as[r1];
        scale_y(dp, f0, f1);
        scale_z(z, 0, g0 * f0, g1 * f1);
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) aq[i][e] += z[i][e];
        row_dots(z, Sm::kQ, qs, rg0, rg1);
      }
      __syncthreads();
      // X's rows, and X_r . V_r on the way.
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int row = 8 * warp + k * RP + rl;
        const Tin *vp = reinterpret_cast<const Tin *>(&vx[k]);
        float d = x[k].x * to_f32(vp[0]) + x[k].y * to_f32(vp[1]) + x[k].z * to_f32(vp[2]) +
                  x[k].w * to_f32(vp[3]);
#pragma unroll
        for (int off = LR / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        if (cl == 0) sm.xv[row] = d;
      }
      store_rows(x, Sm::kA, sm.as);
      __syncthreads();
      {  // X S^T and X U^T
        rows_times(Sm::kA, Sm::kS, z, da, true);
        const float f0 = sm.as[r0], f1 = sm.as[r1];
        scale_y(da, f0, f1);
        scale_z(z, 0, f0, f1);
        row_dots(z, Sm::kK, ks, zk0, zk1);
        const float k0 = g0 * b0, k1 = g1 * b1;
        rg0 -= k0 * zk0;
        rg1 -= k1 * zk1;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          ak[i][0] -= k0 * z[i][0]; ak[i][1] -= k0 * z[i][1];
          ak[i][2] -= k1 * z[i][2]; ak[i][3] -= k1 * z[i][3];
        }
      }
      {  // E U dS'^T
        rows_times(Sm::kU, Sm::kD, z, da, false);
        const float2 gl = sm.gamma[C - 1];
        scale_z(z, 1, sm.us[r0] * decay_between(gl, gr[0]), sm.us[r1] * decay_between(gl, gr[1]));
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) ak[i][e] += z[i][e];
        row_dots(z, Sm::kK, ks, tl0, tl1);
      }
      // W, M and their sums over rows and columns; Q K^T and K K^T again, from the tiles.  A token's
      // own term decays by nothing: it stays out of the sums, where it would be added and taken
      // away again, next to which the others may be small.
      float row_w[2] = {0.f, 0.f}, row_m[2] = {0.f, 0.f}, cs[4][2], nb[2] = {0.f, 0.f};
      {
        float qk[4][4], kk2[4][4];
        zero(qk);
        zero(kk2);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          uint32_t a[4], aa[4];
          load_a<kKq>(a, sb + Sm::kQ, 16 * m, 16 * kk);
          load_a<kKq>(aa, sb + Sm::kK, 16 * m, 16 * kk);
#pragma unroll
          for (int np = 0; np < 2; ++np) {
            if (2 * half + np > m) break;
            uint32_t b[4];
            load_b<kKq>(b, sb + Sm::kK, 32 * half + 16 * np, 16 * kk);
            mma(qk[2 * np], a, b[0], b[1]);
            mma(qk[2 * np + 1], a, b[2], b[3]);
            mma(kk2[2 * np], aa, b[0], b[1]);
            mma(kk2[2 * np + 1], aa, b[2], b[3]);
          }
        }
        float rows[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cs[i][0] = cs[i][1] = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e >> 1 ? r1 : r0, cc = 32 * half + 8 * i + col + (e & 1);
            const float dec = cc <= r ? decay_between(gr[e >> 1], sm.gamma[cc]) : 0.f;
            const float w = cc <= r ? dp[i][e] * dec : 0.f;
            const float m0 = cc < r ? -da[i][e] * dec : 0.f;  // dA D
            const float mk = m0 * (ks * ks * kk2[i][e]);
            const float b = e >> 1 ? b1 : b0;
            const float t = cc < r ? w * (qs * ks * qk[i][e]) + b * mk : 0.f;
            nb[e >> 1] += mk;
            rows[e >> 1] += t;
            cs[i][e & 1] += t;
            dp[i][e] = w;
            da[i][e] = b * m0;
            row_w[e >> 1] = fmaxf(row_w[e >> 1], fabsf(w));
            row_m[e >> 1] = fmaxf(row_m[e >> 1], fabsf(da[i][e]));
          }
          cs[i][0] = col_sum(cs[i][0]);
          cs[i][1] = col_sum(cs[i][1]);
        }
        rg0 += quad_sum(rows[0]);
        rg1 += quad_sum(rows[1]);
        nb[0] = quad_sum(nb[0]);
        nb[1] = quad_sum(nb[1]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) cross += __shfl_xor_sync(0xffffffffu, cross, off);
      float most[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row_w[e] = quad_max(row_w[e]);
        row_m[e] = quad_max(row_m[e]);
      }
      most[0] = fmaxf(row_w[0], row_w[1]);
      most[1] = fmaxf(row_m[0], row_m[1]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        most[0] = fmaxf(most[0], __shfl_xor_sync(0xffffffffu, most[0], off));
        most[1] = fmaxf(most[1], __shfl_xor_sync(0xffffffffu, most[1], off));
      }
      tc::fence_async_smem();  // the split rows were ordinary writes; the copies below are not
      __syncthreads();         // S, dS', U, X have been read
      if (lane < 2) sums.most[warp][lane] = lane ? most[1] : most[0];
      if ((lane & 3) == 0) {
        sums.row_max[0][half][r0] = row_w[0];
        sums.row_max[0][half][r1] = row_w[1];
        sums.row_max[1][half][r0] = row_m[0];
        sums.row_max[1][half][r1] = row_m[1];
      }
      if (j + 1 < group) {
        if (tid == 0) fetch_states(item, j + 1);
        fetch_small(t0, len, h + 1);
      } else {
        following = next_item(item + gridDim.x);  // bos, eos and c are the next item's from here on
        if (tid == 0 && following < items) fetch_states(following, 0);
        if (following < items)
          fetch_small(bos + c * C, min(C, eos - bos - c * C), (int)(following % HK) * group);
      }
      __syncthreads();
      // W and M, a power of two per row: a token's W K and M K are as exact for themselves where other
      // tokens' rows are larger by many powers of two.  In W^T Q and M^T K, where the rows are summed
      // over, they go to the operand as fp16 factors, exact down to 2^-24 of the largest row's value.
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float(&y)[4][4] = which ? da : dp;
        Scale s[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[e] = scale_of(fmaxf(sums.row_max[which][0][e ? r1 : r0], sums.row_max[which][1][e ? r1 : r0]));
        }
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = fmaxf(all, sums.most[i][which]);
        const Scale sa = scale_of(all);
        if (tid == 0) sums.scale[which][C] = sa.s;
        if (half == 0 && (lane & 3) == 0) {
          sums.scale[which][r0] = s[0].s;
          sums.scale[which][r1] = s[1].s;
          sums.rel[which][r0] = __float2half_rn(s[0].s * sa.inv);
          sums.rel[which][r1] = __float2half_rn(s[1].s * sa.inv);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (2 * half + (i >> 1) > m) break;  // nothing above the 16 x 16 diagonal blocks is read
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t hi, lo;
            split2(y[i][2 * e], y[i][2 * e + 1], s[e].inv, hi, lo);
            uint8_t *to = smem + Sm::kU + 2 * which * kTriBytes + tile_off(e ? r1 : r0, 4 * half + i) + 2 * col;
            *reinterpret_cast<uint32_t *>(to) = hi;
            *reinterpret_cast<uint32_t *>(to + kTriBytes) = lo;
          }
        }
      }
      if (lane < 4)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) sums.cols[m][32 * half + 8 * i + col + e] = cs[i][e];
      if ((lane & 3) == 0) {
        sums.rows[half][r0] = rg0;
        sums.rows[half][r1] = rg1;
        sums.zk[half][r0] = zk0;
        sums.zk[half][r1] = zk1;
        sums.tail[half][r0] = tl0;
        sums.tail[half][r1] = tl1;
        sums.db[half][r0] = nb[0];
        sums.db[half][r1] = nb[1];
      }
      if (lane == 0) sums.cross[warp] = cross;
      __syncthreads();

      auto times = [&](int which, bool transposed, uint32_t tile, float f, float (&out)[NH][4]) {
        zero(z);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (transposed ? kk < m : kk > m) continue;
          uint32_t hi[4], lo[4];
          const uint32_t plane = sb + Sm::kU + 2 * which * kTriBytes;
          if (transposed) {
            load_at(hi, plane, 16 * m, 16 * kk);
            load_at(lo, plane + kTriBytes, 16 * m, 16 * kk);
            const __half2 ra = *reinterpret_cast<const __half2 *>(&sums.rel[which][16 * kk + col]);
            const __half2 rb = *reinterpret_cast<const __half2 *>(&sums.rel[which][16 * kk + 8 + col]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hi[i] = times2(hi[i], i < 2 ? ra : rb);
              lo[i] = times2(lo[i], i < 2 ? ra : rb);
            }
          } else {
            load_a(hi, plane, 16 * m, 16 * kk);
            load_a(lo, plane + kTriBytes, 16 * m, 16 * kk);
          }
#pragma unroll
          for (int np = 0; np < NH / 2; ++np) {
            uint32_t b[4];
            load_bt<kKq>(b, tile, half * (D / 2) + 16 * np, 16 * kk);
            mma(z[2 * np], hi, b[0], b[1]);
            mma(z[2 * np + 1], hi, b[2], b[3]);
            mma(z[2 * np], lo, b[0], b[1]);
            mma(z[2 * np + 1], lo, b[2], b[3]);
          }
        }
        const float f0 = f * sums.scale[which][transposed ? C : r0];
        const float f1 = f * sums.scale[which][transposed ? C : r1];
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) out[i][e] = fmaf(e >> 1 ? f1 : f0, z[i][e], out[i][e]);
      };
      times(0, false, sb + Sm::kK, ks, aq);
      times(0, true, sb + Sm::kQ, qs, ak);
      times(1, false, sb + Sm::kK, ks, ak);
      times(1, true, sb + Sm::kK, ks, ak);

      if (warp == 0) {  // dg and dbeta of tokens 2 lane, 2 lane + 1
        double d[2], e = 0.0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * lane + i;
          const float2 gm = sm.gamma[r];
          // M's contribution to dbeta has beta left out, so that it holds for beta = 0 too.
          const float b = sm.xv[r] - ex2_approx(gm.x + gm.y) * (sums.zk[0][r] + sums.zk[1][r]) +
                          sums.db[0][r] + sums.db[1][r];
          if (r < len) dbeta[(size_t)(t0 + r) * HV + h] = b;
          const double et = (double)sums.tail[0][r] + sums.tail[1][r];
          d[i] = (double)sums.rows[0][r] + sums.rows[1][r] - et -
                 ((double)sums.cols[0][r] + sums.cols[1][r] + sums.cols[2][r] + sums.cols[3][r]);
          e += et;
        }
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sums.cross[i];
        const float2 gl = sm.gamma[C - 1];
        // The last token's share is in every sum from a token to the end.
        double s = d[0] + d[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const double o = __shfl_down_sync(0xffffffffu, s, off);
          e += __shfl_xor_sync(0xffffffffu, e, off);
          if (lane + off < 32) s += o;
        }
        s += e + (double)(ex2_approx(gl.x + gl.y) * t);
        if (2 * lane < len) dg[(size_t)(t0 + 2 * lane) * HV + h] = (float)s;
        if (2 * lane + 1 < len) dg[(size_t)(t0 + 2 * lane + 1) * HV + h] = (float)(s - d[0]);
      }
      tc::fence_async_smem();
      __syncthreads();  // gamma, the sums, W and M (and K and Q, after the last head) have been read
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = e ? r1 : r0;
      if (r >= len) continue;
      const size_t at = ((size_t)(t0 + r) * HK + hk) * D + half * (D / 2) + col;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        Tin o[2] = {from_f32<Tin>(aq[i][2 * e]), from_f32<Tin>(aq[i][2 * e + 1])};
        *reinterpret_cast<uint32_t *>(dq + at + 8 * i) = *reinterpret_cast<const uint32_t *>(o);
        o[0] = from_f32<Tin>(ak[i][2 * e]);
        o[1] = from_f32<Tin>(ak[i][2 * e + 1]);
        *reinterpret_cast<uint32_t *>(dk + at + 8 * i) = *reinterpret_cast<const uint32_t *>(o);
      }
    }
    item = following;
  }
}

template <typename Tin, int D>
cudaError_t launch_reverse(const int32_t *cu, float scale, int N, int T, int HK, int HV, void *ws,
                           const Layout &lay, const float *d_o, const float *d_sN, void *dv, float *d_s0,
                           int *status, cudaStream_t s) {
  // Two CTAs of 64 value channels per head as long as all of them run at once (5.6 us a chunk), else whole
  // heads (10.4 us; the two halves on one SM in turn 11.2), as the forward (kda_gdr_state.cu).
  const bool whole = D == 128 && (long long)N * HV * 2 > 148;
  void (*kern)(const float *, const float *, const int32_t *, float, int, int, int, int, uint8_t *, Layout,
               Tin *, float *, int *) = gdr_reverse_pair_kernel<Tin, D>;
  int bytes = (int)PairSmem<D>::kBytes;
  cudaError_t e = cudaSuccess;
  long long ctas = (long long)N * HV * (D / 64);
  if constexpr (D == 128)
    if (whole) {
      kern = gdr_reverse_kernel<Tin, D>;
      bytes = (int)ReverseSmem<D>::kBytes;
      ctas = (long long)N * HV;
      e = allow_smem<(int)ReverseSmem<D>::kBytes>(kern);
    }
  if (!whole) e = allow_smem<(int)PairSmem<D>::kBytes>(kern);
  if (ctas >= (1LL << 31)) return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return launch_behind(kern, dim3((unsigned)ctas), 256, bytes, s, d_o, d_sN, cu, scale, N, T, HK, HV,
                       static_cast<uint8_t *>(ws), lay, static_cast<Tin *>(dv),
                       d_s0, status);
}

template <typename Tin, int D>
cudaError_t launch_typed(const void *v, const float *g, const float *beta, const int32_t *cu,
                         float scale, int N, int T, int HK, int HV, void *ws, const Layout &lay,
                         const float *d_o, const float *d_sN, void *dq, void *dk, void *dv, float *dg, float *dbeta,
                         float *d_s0, int *status, cudaStream_t s) {
  cudaError_t e = launch_reverse<Tin, D>(cu, scale, N, T, HK, HV, ws, lay, d_o, d_sN, dv, d_s0, status, s);
  if (e != cudaSuccess) return e;
  auto kern = gdr_local_kernel<Tin, D>;
  constexpr int bytes = (int)LocalSmem<D>::kBytes;
  e = allow_smem<bytes>(kern);
  if (e != cudaSuccess) return e;
  const long long items = slots(N, T) * HK;
  const unsigned ctas = (unsigned)(items < 148 ? items : 148);  // one per SM
  kern<<<ctas, kLocalThreads, bytes, s>>>(
      static_cast<const Tin *>(v), g, beta, d_o, cu, scale, N, T, HK, HV,
      static_cast<const uint8_t *>(ws), lay, static_cast<Tin *>(dq),
      static_cast<Tin *>(dk), dg, dbeta, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_bwd(const void *v, const float *g, const float *beta, const int32_t *cu,
                           float scale, int N, int T, int HK, int HV, int D, kda_dtype dt, void *ws,
                           const Layout &lay, const float *d_o, const float *d_sN, void *dq, void *dk, void *dv,
                           float *dg, float *dbeta, float *d_s0, int *status, cudaStream_t s) {
  const bool bf = dt == KDA_BF16;
  if (D == 128)
    return bf ? launch_typed<__nv_bfloat16, 128>(v, g, beta, cu, scale, N, T, HK, HV, ws, lay, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s)
              : launch_typed<__half, 128>(v, g, beta, cu, scale, N, T, HK, HV, ws, lay, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s);
  if (D == 64)
    return bf ? launch_typed<__nv_bfloat16, 64>(v, g, beta, cu, scale, N, T, HK, HV, ws, lay, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s)
              : launch_typed<__half, 64>(v, g, beta, cu, scale, N, T, HK, HV, ws, lay, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s);
  return cudaErrorInvalidValue;
}

}  // namespace kda
