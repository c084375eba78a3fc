// State pass of the chunked gated delta rule (kda_gdr.cuh): the chunks of a sequence in order.
//
// The rows of S^T (one per value channel) need nothing from one another, so a warp owns 16 of
// them as the accumulators of its MMAs and carries them through all chunks of its (sequence,
// value head) without a word to another warp.  Everything is computed transposed, with the value
// channels as the MMAs' rows, because an accumulator of one product is then, split in two fp16
// terms in registers, the A operand of the next:
//     (K S)^T = S^T K^T            B: the K tile, read along its rows
//     (Q S)^T = S^T Q^T
//     R^T = beta (V^T - G (K S)^T)
//     U^T = R^T T^T                B: the T tiles (blocks above the diagonal skipped)
//     O^T = scale (G (Q S)^T + U^T P^T)
//     S^T = G_C S^T + (E U)^T K    B: the K tile, read across (ldmatrix.trans)
// The records and the V tile of the next chunk arrive by cp.async while this one is computed;
// the CTA's two barriers per chunk only guard the two buffers.
//
// D = 128: 504 MMAs (16 x 8 x 16) per warp and chunk, one warp per SM quarter, 64 value channels per
// CTA.  mma.sync runs at 9 cycles per MMA and SM quarter (527 TFLOP/s measured over the GPU), 2.4 us a
// chunk; bound by the chain's latency, 4.9 us a chunk with the read-out and 3.9 without (64 chains of
// 32 chunks, split over 128 SMs: 125 us).  A whole head on eight warps of one CTA took 7.7.
//
// For more heads than that, and for segments, D = 128 runs on tcgen05 (kda_gdr_state_tc.cu), which
// takes the same time for a whole head on one SM.
#include <type_traits>

#include "kda_gdr.cuh"

namespace kda {
namespace {
using namespace gdr;

// A stage: K (and Q), T (and P), the chunk's vectors, V.  The backward's forward needs no Q and no P.
template <int D, int NW, int kRole> struct StateSmem {
  static constexpr bool kAll = kRole != kKeep;
  static constexpr int kRows = kAll ? kKq : C;                 // rows of the K (and Q) tile
  static constexpr uint32_t kScales = (uint32_t)kRows * D * 2;
  static constexpr uint32_t kTp = kScales + 128;               // T hi, lo (P hi, lo)
  static constexpr uint32_t kVecs = kTp + (kAll ? 4 : 2) * kTriBytes;
  static constexpr uint32_t kV = kVecs + gdr::kVecs * C * 4;   // [64][16 NW] 16-bit, swizzled
  static constexpr uint32_t kStage = kV + C * 32 * NW;
  static constexpr uint32_t kBytes = 2 * kStage;
};

// Value channels of a scan's CTA, and its shared memory: two stages of a segment's M and of those
// channels of its B, and the halves of E that its warps exchange.
constexpr int kScanRows = 32;
template <int D> struct ScanSmem {
  static constexpr int kLd = D + 8;                            // floats per row of B and E
  static constexpr uint32_t kRows = kScanRows * kLd * 4;
  static constexpr uint32_t kB = map_bytes(D);
  static constexpr uint32_t kStage = kB + kRows;
  static constexpr uint32_t kE = 2 * kStage;
  static constexpr uint32_t kBytes = kE + kRows;
};

// Byte offset of the 16-byte piece p of token row `row` of a V tile 16 NW channels wide.
template <int NW> __device__ __forceinline__ uint32_t v_off(int row, int p) {
  return (uint32_t)(row * (32 * NW) + ((p ^ (row & 7)) << 4));
}

__device__ __forceinline__ float2 widen2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 widen2(uint32_t u, __half) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

template <typename Tin, int D, int NW, int kRole>
__global__ void __launch_bounds__(NW * 32, 1)
gdr_state_kernel(const Tin *__restrict__ v, const float *s0, const int32_t *__restrict__ cu,
                 float scale, int N, int T, int HK, int HV, uint8_t *__restrict__ ws, Layout lay,
                 float *__restrict__ o, float *sN, int *status) {
  using Sm = StateSmem<D, NW, kRole>;
  constexpr int NT = D / 8, KK = D / 16;
  constexpr int kParts = D / (16 * NW);  // CTAs per head
  extern __shared__ __align__(128) uint8_t smem[];
  wait_for_previous_kernel();  // before any way out: what comes next takes this one's end for the last one's
  if (kRole == kKeep) next_kernel_may_start();  // the reverse pass only needs what is there by now
  const uint32_t sbase = smem_addr(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = blockIdx.x;
  const int part = b % kParts;
  b /= kParts;
  Part pt;
  if (!part_of<kRole, D == 64>(b, cu, N, T, HV, lay, status, pt)) return;
  const int h = pt.h, hk = h / (HV / HK), bos = pt.bos, eos = pt.eos, first = pt.first, end = pt.end;
  const long long slot0 = pt.slot - first;
  const int ch0 = (part * NW + warp) * 16;     // the warp's first value channel
  const int row = ch0 + lane / 4;              // and this lane's rows: row, row + 8
  const int col = 2 * (lane & 3);

  auto load = [&](int c) {
    const uint32_t st = sbase + (c & 1) * Sm::kStage;
    const long long slot = slot0 + c;
    const uint8_t *kq = ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D);
    const uint8_t *tp = ws + lay.tp + (size_t)(slot * HV + h) * kTpBytes;
    if constexpr (Sm::kAll) {
      cp_block(st, kq, kq_bytes(D));
      cp_block(st + Sm::kTp, tp, kTpBytes);
    } else {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) cp_block(st + i * kQRows, kq + i * 2 * kQRows, kQRows);
      cp_block(st + Sm::kScales, kq + kq_tile_bytes(D), 16);
      cp_block(st + Sm::kTp, tp + kT_HI, 2 * kTriBytes);
      cp_block(st + Sm::kVecs, tp + kVec, gdr::kVecs * C * 4);
    }
    constexpr int kPieces = 2 * NW;
    const int t0 = bos + c * C, len = min(C, eos - t0);
    for (int i = threadIdx.x; i < C * kPieces; i += NW * 32) {
      const int r = i / kPieces, p = i % kPieces;
      cp16(st + Sm::kV + v_off<NW>(r, p),
           v + ((size_t)(t0 + min(r, len - 1)) * HV + h) * D + part * NW * 16 + p * 8, r < len);
    }
  };
  if (first < end) load(first);
  cp_commit();

  float s[NT][4];
  zero(s);
  auto store = [&](float *to) {
    float *p = to + (size_t)row * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2 *>(p + 8 * i) = make_float2(s[i][0], s[i][1]);
      *reinterpret_cast<float2 *>(p + 8 * D + 8 * i) = make_float2(s[i][2], s[i][3]);
    }
  };
  const float *from = first_state<kRole>(pt, s0, ws, lay, HV, D);
  if (kRole == kMap && pt.kind == 1) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = row + 8 * (e >> 1) == 8 * i + col + (e & 1) ? 1.f : 0.f;
  } else if (from) {
    const float *p = from + (size_t)row * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float2 a = *reinterpret_cast<const float2 *>(p + 8 * i);
      const float2 b = *reinterpret_cast<const float2 *>(p + 8 * D + 8 * i);
      s[i][0] = a.x; s[i][1] = a.y; s[i][2] = b.x; s[i][3] = b.y;
    }
    if (kRole == kMap) store(reinterpret_cast<float *>(ws + lay.seg_e) + pt.seg * D * D);
  }

  for (int c = first; c < end; ++c) {
    if (c + 1 < end) load(c + 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    const uint32_t st = sbase + (c & 1) * Sm::kStage;
    const uint8_t *stp = smem + (c & 1) * Sm::kStage;
    const float2 kqs = *reinterpret_cast<const float2 *>(stp + Sm::kScales);
    const float *vec = reinterpret_cast<const float *>(stp + Sm::kVecs);
    const int t0 = bos + c * C, len = min(C, eos - t0);

    if constexpr (kRole == kKeep) {
      float *p = reinterpret_cast<float *>(ws + lay.state) + ((size_t)(slot0 + c) * HV + h) * D * D + row;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(8 * i + col + (e & 1)) * D + 8 * (e >> 1)] = s[i][e];
    }

    // (K S)^T and (Q S)^T.
    float ks[8][4], qs[8][4];
    zero(ks);
    zero(qs);
    Scale a0, a1;
    row_scales(s, a0, a1);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(s, kk, a0, a1, hi, lo);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t b[4];
        load_b<Sm::kRows>(b, st, 16 * np, 16 * kk);
        mma(ks[2 * np], hi, b[0], b[1]);
        mma(ks[2 * np + 1], hi, b[2], b[3]);
        mma(ks[2 * np], lo, b[0], b[1]);
        mma(ks[2 * np + 1], lo, b[2], b[3]);
        if constexpr (kRole == kOut) {
          load_b<kKq>(b, st + kQRows, 16 * np, 16 * kk);
          mma(qs[2 * np], hi, b[0], b[1]);
          mma(qs[2 * np + 1], hi, b[2], b[3]);
          mma(qs[2 * np], lo, b[0], b[1]);
          mma(qs[2 * np + 1], lo, b[2], b[3]);
        }
      }
    }
    // R^T = beta (V^T - G (K S)^T), in ks.
    {
      const float f0 = a0.s * kqs.x, f1 = a1.s * kqs.x;
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t b[4];
        const int m = lane >> 3, r = 16 * np + (m >> 1) * 8 + (lane & 7);
        ldsm4t(b, st + Sm::kV + v_off<NW>(r, 2 * warp + (m & 1)));
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // 8-token blocks 2 np + e
          const int i = 2 * np + e;
          const float2 g = *reinterpret_cast<const float2 *>(vec + kVecG * C + 8 * i + col);
          const float2 bt = *reinterpret_cast<const float2 *>(vec + kVecBeta * C + 8 * i + col);
          float2 v0 = widen2(b[2 * e], Tin{}), v1 = widen2(b[2 * e + 1], Tin{});
          if (kRole == kMap && pt.kind == 1) v0 = v1 = make_float2(0.f, 0.f);
          ks[i][0] = bt.x * (v0.x - g.x * (f0 * ks[i][0]));
          ks[i][1] = bt.y * (v0.y - g.y * (f0 * ks[i][1]));
          ks[i][2] = bt.x * (v1.x - g.x * (f1 * ks[i][2]));
          ks[i][3] = bt.y * (v1.y - g.y * (f1 * ks[i][3]));
        }
      }
    }
    // U^T = R^T T^T.
    float u[8][4];
    zero(u);
    Scale r0, r1;
    row_scales(ks, r0, r1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      split_a(ks, kk, r0, r1, hi, lo);
#pragma unroll
      for (int np = kk; np < 4; ++np) {
        uint32_t b[4], bl[4];
        load_b(b, st + Sm::kTp + kT_HI, 16 * np, 16 * kk);
        load_b(bl, st + Sm::kTp + kT_LO, 16 * np, 16 * kk);
        mma(u[2 * np], hi, b[0], b[1]);
        mma(u[2 * np + 1], hi, b[2], b[3]);
        mma(u[2 * np], lo, b[0], b[1]);
        mma(u[2 * np + 1], lo, b[2], b[3]);
        mma(u[2 * np], hi, bl[0], bl[1]);
        mma(u[2 * np + 1], hi, bl[2], bl[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = *reinterpret_cast<const float2 *>(vec + kVecT * C + 8 * i + col);
      u[i][0] *= r0.s * t.x;
      u[i][1] *= r0.s * t.y;
      u[i][2] *= r1.s * t.x;
      u[i][3] *= r1.s * t.y;
    }
    if constexpr (kRole == kKeep) {
      float *p = reinterpret_cast<float *>(ws + lay.u) + ((size_t)(slot0 + c) * HV + h) * C * D + row;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(8 * i + col + (e & 1)) * D + 8 * (e >> 1)] = u[i][e];
    }
    if constexpr (kRole == kOut) {
      // O^T = scale (G (Q S)^T + U^T P^T).
      float pu[8][4];
      zero(pu);
      row_scales(u, r0, r1);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t hi[4], lo[4];
        split_a(u, kk, r0, r1, hi, lo);
#pragma unroll
        for (int np = kk; np < 4; ++np) {
          uint32_t b[4], bl[4];
          load_b(b, st + Sm::kTp + kP_HI, 16 * np, 16 * kk);
          load_b(bl, st + Sm::kTp + kP_LO, 16 * np, 16 * kk);
          mma(pu[2 * np], hi, b[0], b[1]);
          mma(pu[2 * np + 1], hi, b[2], b[3]);
          mma(pu[2 * np], lo, b[0], b[1]);
          mma(pu[2 * np + 1], lo, b[2], b[3]);
          mma(pu[2 * np], hi, bl[0], bl[1]);
          mma(pu[2 * np + 1], hi, bl[2], bl[3]);
        }
      }
      float *op = o + ((size_t)t0 * HV + h) * D + row;
      const float q0 = a0.s * kqs.y, q1 = a1.s * kqs.y;
      auto out = [&](int i, auto whole) {
        const float2 g = *reinterpret_cast<const float2 *>(vec + kVecG * C + 8 * i + col);
        const float2 p = *reinterpret_cast<const float2 *>(vec + kVecP * C + 8 * i + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 8 * i + col + (e & 1);
          const float gg = e & 1 ? g.y : g.x, pp = e & 1 ? p.y : p.x;
          const float x = gg * ((e >> 1 ? q1 : q0) * qs[i][e]) + (e >> 1 ? r1.s : r0.s) * pp * pu[i][e];
          if (decltype(whole)::value || t < len) __stcs(op + (size_t)t * HV * D + 8 * (e >> 1), scale * x);
        }
      };
      if (len == C) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out(i, std::true_type{});
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) out(i, std::false_type{});
      }
    }
    // S^T = G_C S^T + (E U)^T K.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 e = *reinterpret_cast<const float2 *>(vec + kVecE * C + 8 * i + col);
      u[i][0] *= e.x;
      u[i][1] *= e.y;
      u[i][2] *= e.x;
      u[i][3] *= e.y;
    }
    row_scales(u, r0, r1);
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) split_a(u, kk, r0, r1, hi[kk], lo[kk]);
    const float gl = vec[kVecG * C + C - 1];
    const float w0 = r0.s * kqs.x, w1 = r1.s * kqs.x;
#pragma unroll
    for (int j = 0; j < NT / 4; ++j) {
      float acc[4][4];
      zero(acc);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int np = 0; np < 2; ++np) {
          uint32_t b[4];
          load_bt<Sm::kRows>(b, st, 32 * j + 16 * np, 16 * kk);
          mma(acc[2 * np], hi[kk], b[0], b[1]);
          mma(acc[2 * np + 1], hi[kk], b[2], b[3]);
          mma(acc[2 * np], lo[kk], b[0], b[1]);
          mma(acc[2 * np + 1], lo[kk], b[2], b[3]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float(&x)[4] = s[4 * j + i];
        x[0] = fmaf(gl, x[0], w0 * acc[i][0]);
        x[1] = fmaf(gl, x[1], w0 * acc[i][1]);
        x[2] = fmaf(gl, x[2], w1 * acc[i][2]);
        x[3] = fmaf(gl, x[3], w1 * acc[i][3]);
      }
    }
    __syncthreads();  // the other buffer is free for the chunk after next
  }
  cp_wait<0>();
  if (kRole != kKeep) next_kernel_may_start();

  if (kRole == kMap && pt.kind == 1) {
    uint8_t *m = ws + lay.seg_m + pt.seg * map_bytes(D);
    Scale r0, r1;
    row_scales(s, r0, r1);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, lo;
        split2(s[i][2 * e], s[i][2 * e + 1], e ? r1.inv : r0.inv, hi, lo);
        uint8_t *to = m + row_off<D>(row + 8 * e, i) + 2 * col;
        *reinterpret_cast<uint32_t *>(to) = hi;
        *reinterpret_cast<uint32_t *>(to + 2 * D) = lo;
      }
    if ((lane & 3) == 0) {
      float *scales = reinterpret_cast<float *>(m + D * D * 4);
      scales[row] = r0.s;
      scales[row + 8] = r1.s;
    }
  } else if (kRole == kMap) {
    store(reinterpret_cast<float *>(ws + lay.seg_b) + pt.seg * D * D);
  } else if (pt.is_last && sN) {
    store(sN + ((size_t)pt.n * HV + h) * D * D);
  }
}

// First states of the segments: E_1 = B_0 and E_g+1 = M_g E_g + B_g, 32 value channels per CTA.
// E^T is the A operand of its own next step, as S^T in the pass above.  Four warps: 16 value channels
// times half the key channels of the result each, and the halves are exchanged after every step.  M
// comes split, row by row; its rows' scales go to E's columns.
// Bound: a step's chain, 192 MMAs a warp, about 2 us at D = 128 (64 value channels and whole rows per warp:
// 3.2; all 128 channels with M split here: 6).
template <int D>
__global__ void __launch_bounds__(128, 1)
gdr_scan_kernel(const int32_t *__restrict__ cu, int N, int T, int HV, uint8_t *__restrict__ ws,
                Layout lay, int *status) {
  using Sm = ScanSmem<D>;
  constexpr int NH = D / 16, KH = D / 32, kParts = D / kScanRows;  // 8-column blocks, k-steps of a half
  extern __shared__ __align__(128) uint8_t smem[];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % kParts, nh = blockIdx.x / kParts;
  const int n = nh / HV, h = nh % HV, L = lay.seg_chunks;
  int bos, eos;
  seq_bounds(cu, n, T, status, bos, eos);
  const int G = ((eos - bos + C - 1) / C + L - 1) / L;
  const long long slot0 = bos / (C * L) + n;
  if (G < 2 || !in_range(status, slot0 + G, segment_slots(N, T, L) + 1)) return;
  const int rl = 16 * (warp & 1) + lane / 4;                      // rows rl, rl + 8 of the CTA's
  const int mine = (warp >> 1) * (D / 2), his = D / 2 - mine;      // first columns of the two halves
  const int col = 2 * (lane & 3);
  auto state_of = [&](size_t area, int g) {
    return reinterpret_cast<float *>(ws + area) +
           (((size_t)(slot0 + g) * HV + h) * D + kScanRows * part) * D;
  };
  auto fetch = [&](int g) {
    const uint32_t st = smem_addr(smem) + (g & 1) * Sm::kStage;
    cp_block(st, ws + lay.seg_m + ((size_t)(slot0 + g) * HV + h) * map_bytes(D), map_bytes(D));
    const float *b = state_of(lay.seg_b, g);
    for (int i = threadIdx.x; i < kScanRows * D / 4; i += 128) {
      const int r = i / (D / 4), p = i % (D / 4);
      cp16(st + Sm::kB + (r * Sm::kLd + 4 * p) * 4, b + r * D + 4 * p);
    }
  };
  if (G > 2) fetch(1);
  cp_commit();
  float e[2][NH][4];  // this warp's half, the other warp's
  auto load = [&](float(&x)[NH][4], const float *p, int ld) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const float2 a = *reinterpret_cast<const float2 *>(p + 8 * i);
      const float2 b = *reinterpret_cast<const float2 *>(p + 8 * ld + 8 * i);
      x[i][0] = a.x; x[i][1] = a.y; x[i][2] = b.x; x[i][3] = b.y;
    }
  };
  auto store = [&](float *p, int ld) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      *reinterpret_cast<float2 *>(p + 8 * i) = make_float2(e[0][i][0], e[0][i][1]);
      *reinterpret_cast<float2 *>(p + 8 * ld + 8 * i) = make_float2(e[0][i][2], e[0][i][3]);
    }
  };
  load(e[0], state_of(lay.seg_b, 0) + rl * D + mine + col, D);
  load(e[1], state_of(lay.seg_b, 0) + rl * D + his + col, D);
  for (int g = 1;; ++g) {
    store(state_of(lay.seg_e, g) + rl * D + mine + col, D);
    if (g + 1 >= G) break;
    if (g + 2 < G) fetch(g + 1);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    const uint8_t *st = smem + (g & 1) * Sm::kStage;
    const uint32_t mat = smem_addr(st);
    const float *scales = reinterpret_cast<const float *>(st + D * D * 4) + col;
    float big0 = 0.f, big1 = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        float(&x)[4] = e[half][i];
        const float2 f = *reinterpret_cast<const float2 *>(scales + (half ? his : mine) + 8 * i);
        x[0] *= f.x; x[1] *= f.y; x[2] *= f.x; x[3] *= f.y;
        big0 = fmaxf(big0, fmaxf(fabsf(x[0]), fabsf(x[1])));
        big1 = fmaxf(big1, fmaxf(fabsf(x[2]), fabsf(x[3])));
      }
    const Scale a0 = scale_of(quad_max(big0)), a1 = scale_of(quad_max(big1));
    float acc[NH][4];
    zero(acc);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int kk = 0; kk < KH; ++kk) {
        uint32_t hi[4], lo[4];
        split_a(e[half], kk, a0, a1, hi, lo);
        const int k0 = (half ? his : mine) + 16 * kk;
#pragma unroll
        for (int np = 0; np < NH / 2; ++np) {
          uint32_t b[4], bl[4];
          load_rows_bt<D>(b, mat, mine + 16 * np, k0, false);
          load_rows_bt<D>(bl, mat, mine + 16 * np, k0, true);
          mma(acc[2 * np], hi, b[0], b[1]);
          mma(acc[2 * np + 1], hi, b[2], b[3]);
          mma(acc[2 * np], lo, b[0], b[1]);
          mma(acc[2 * np + 1], lo, b[2], b[3]);
          mma(acc[2 * np], hi, bl[0], bl[1]);
          mma(acc[2 * np + 1], hi, bl[2], bl[3]);
        }
      }
    load(e[0], reinterpret_cast<const float *>(st + Sm::kB) + rl * Sm::kLd + mine + col, Sm::kLd);
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      float(&x)[4] = e[0][i];
      x[0] = fmaf(a0.s, acc[i][0], x[0]);
      x[1] = fmaf(a0.s, acc[i][1], x[1]);
      x[2] = fmaf(a1.s, acc[i][2], x[2]);
      x[3] = fmaf(a1.s, acc[i][3], x[3]);
    }
    float *all = reinterpret_cast<float *>(smem + Sm::kE) + rl * Sm::kLd + col;
    store(all + mine, Sm::kLd);
    __syncthreads();  // also: the matrix has been read, the next fetch may take its place
    load(e[1], all + his, Sm::kLd);
  }
  cp_wait<0>();
}

template <typename Tin, int D, int NW, int kRole>
cudaError_t launch_role(const void *v, const float *s0, const int32_t *cu, float scale, int N, int T,
                        int HK, int HV, void *ws, const Layout &lay, float *o, float *sN, int *status,
                        cudaStream_t s) {
  auto kern = gdr_state_kernel<Tin, D, NW, kRole>;
  const long long units = kRole != kKeep && lay.seg_chunks ? segment_slots(N, T, lay.seg_chunks) : N;
  const long long ctas = units * HV * (D / (16 * NW)) * (kRole == kMap ? 2 : 1);
  if (ctas >= (1LL << 31)) return cudaErrorInvalidValue;
  constexpr int kBytes = (int)StateSmem<D, NW, kRole>::kBytes;
  const int bytes = chain_smem(kBytes, ctas);
  const cudaError_t e = allow_smem<chain_smem(kBytes, 1)>(kern);  // the most that any launch asks for
  if (e != cudaSuccess) return e;
  return launch_behind(kern, dim3((unsigned)ctas), NW * 32, bytes, s, static_cast<const Tin *>(v), s0,
                       cu, scale, N, T, HK, HV, static_cast<uint8_t *>(ws), lay, o, sN, status);
}

template <typename Tin, int D>
cudaError_t launch_d(const void *v, const float *s0, const int32_t *cu, float scale, int N, int T,
                     int HK, int HV, void *ws, const Layout &lay, bool bwd, float *o, float *sN,
                     int *status, cudaStream_t s) {
  // D = 128: two CTAs of four warps per head, one per SM, if they all run at once, or else, and for
  // segments, which fill the SMs by themselves, the tcgen05 form with one CTA per head.  Microseconds a
  // chunk, here and there: with the read-out 4.9 and 5.3, kept for the backward 3.9 and 6.3, maps 4.1 and 4.2.
  const bool tensor_memory = D == 128 && (lay.seg_chunks || (long long)N * HV * 2 > 148);
  const kda_dtype dt = std::is_same<Tin, __half>::value ? KDA_F16 : KDA_BF16;
  if (bwd)
    return tensor_memory
               ? launch_gdr_state_tc(v, s0, cu, scale, N, T, HK, HV, dt, ws, lay, kKeep, o, sN, status, s)
               : launch_role<Tin, D, 4, kKeep>(v, s0, cu, scale, N, T, HK, HV, ws, lay, o, sN, status, s);
  if (lay.seg_chunks) {
    cudaError_t e;
    if constexpr (D == 128)
      e = launch_gdr_state_tc(v, s0, cu, scale, N, T, HK, HV, dt, ws, lay, kMap, o, sN, status, s);
    else
      e = launch_role<Tin, D, 4, kMap>(v, s0, cu, scale, N, T, HK, HV, ws, lay, o, sN, status, s);
    if (e != cudaSuccess) return e;
    auto scan = gdr_scan_kernel<D>;
    constexpr int bytes = (int)ScanSmem<D>::kBytes;
    e = allow_smem<bytes>(scan);
    if (e != cudaSuccess) return e;
    e = launch_behind(scan, dim3((unsigned)(N * HV * (D / kScanRows))), 128, bytes, s, cu, N, T, HV,
                      static_cast<uint8_t *>(ws), lay, status);
    if (e != cudaSuccess) return e;
  }
  return tensor_memory
             ? launch_gdr_state_tc(v, s0, cu, scale, N, T, HK, HV, dt, ws, lay, kOut, o, sN, status, s)
             : launch_role<Tin, D, 4, kOut>(v, s0, cu, scale, N, T, HK, HV, ws, lay, o, sN, status, s);
}

}  // namespace

cudaError_t launch_gdr_state(const void *v, const float *s0, const int32_t *cu, float scale, int N,
                             int T, int HK, int HV, int D, kda_dtype dt, void *ws, const Layout &lay,
                             bool bwd, float *o, float *sN, int *status, cudaStream_t s) {
  if (dt == KDA_BF16)
    return D == 64 ? launch_d<__nv_bfloat16, 64>(v, s0, cu, scale, N, T, HK, HV, ws, lay, bwd, o, sN, status, s)
                   : launch_d<__nv_bfloat16, 128>(v, s0, cu, scale, N, T, HK, HV, ws, lay, bwd, o, sN, status, s);
  return D == 64 ? launch_d<__half, 64>(v, s0, cu, scale, N, T, HK, HV, ws, lay, bwd, o, sN, status, s)
                 : launch_d<__half, 128>(v, s0, cu, scale, N, T, HK, HV, ws, lay, bwd, o, sN, status, s);
}

}  // namespace kda
