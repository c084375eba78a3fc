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
// Per value head and chunk at D = 128 the reverse pass is 504 MMAs per warp (8 warps), the local
// pass about 1000; both are bound by the mma.sync rate as the forward is.  The local pass keeps
// S and dS' as split fp16 planes in shared memory (128 KB) with K, Q and U, one CTA per SM.
#include "kda_gdr.cuh"

namespace kda {
namespace {
using namespace gdr;

// ---- reverse state pass ------------------------------------------------------------------

template <int D, int NW> struct ReverseSmem {
  static constexpr int kLd = 16 * NW + 4;  // row stride of the dO tile: no bank conflicts
  static constexpr uint32_t kK = 0, kQ = kQRows;
  static constexpr uint32_t kScales = kq_tile_bytes(D);
  static constexpr uint32_t kTp = kq_bytes(D);
  static constexpr uint32_t kDo = kTp + kTpBytes;  // [64][kLd] fp32
  static constexpr uint32_t kStage = kDo + C * kLd * 4;
  static constexpr uint32_t kBytes = 2 * kStage;
};

template <typename Tin, int D, int NW>
__global__ void __launch_bounds__(NW * 32, 1)
gdr_reverse_kernel(const float *__restrict__ d_o, const float *d_sN, const int32_t *__restrict__ cu,
                   float scale, int N, int T, int HK, int HV, uint8_t *__restrict__ ws, Layout lay,
                   Tin *__restrict__ dv, float *d_s0, int *status) {
  using Sm = ReverseSmem<D, NW>;
  constexpr int NT = D / 8, KK = D / 16, kParts = D / (16 * NW);
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % kParts, nh = blockIdx.x / kParts;
  const int n = nh / HV, h = nh % HV, hk = h / (HV / HK);
  int bos, eos;
  seq_bounds(cu, n, T, status, bos, eos);
  const int chunks = (eos - bos + C - 1) / C;
  const long long slot0 = first_slot(bos, n);
  if (!in_range(status, slot0 + chunks, slots(N, T) + 1)) return;
  const int row = (part * NW + warp) * 16 + lane / 4;  // this lane's value channels: row, row + 8
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
           d_o + ((size_t)(t0 + min(r, len - 1)) * HV + h) * D + part * NW * 16 + 4 * p, r < len);
    }
  };
  if (chunks > 0) load(chunks - 1);
  cp_commit();

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
    float *p = d_s0 + ((size_t)nh * D + row) * D + col;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2 *>(p + 8 * i) = make_float2(s[i][0], s[i][1]);
      *reinterpret_cast<float2 *>(p + 8 * D + 8 * i) = make_float2(s[i][2], s[i][3]);
    }
  }
}

// ---- local pass --------------------------------------------------------------------------

constexpr int kLocalThreads = 256;

template <int D> struct LocalSmem {
  static constexpr uint32_t kK = 0, kQ = kQRows;
  static constexpr uint32_t kSHi = kq_tile_bytes(D), kSLo = kSHi + D * D * 2;
  static constexpr uint32_t kDHi = kSLo + D * D * 2, kDLo = kDHi + D * D * 2;
  static constexpr uint32_t kU = kDLo + D * D * 2;          // U hi, lo; later W hi, lo, M hi, lo
  static constexpr uint32_t kULo = kU + C * D * 2;
  static constexpr uint32_t kUBytes = C * D * 4 > 4 * kTriBytes ? C * D * 4 : 4 * kTriBytes;
  static constexpr uint32_t kSmall = kU + kUBytes;
  struct Small {
    alignas(16) float2 gamma[C];
    float G[C], E[C], beta[C], us[C];  // us: scale of U's rows
    float rows[2][C];                  // per half: sums that dgamma and dbeta take per row
    float cols[4][C];                  // per row block: column sums
    float tail[2][C], zk[2][C], db[2][C], xv[C];
    float red[8][4];
    float kq[2];
  };
  static constexpr uint32_t kBytes = kSmall + sizeof(Small);
};

// The largest over the block of each of two values (one barrier pair).
__device__ __forceinline__ float2 block_max2(float a, float b, float (*red)[4]) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5][0] = a;
    red[threadIdx.x >> 5][1] = b;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a = fmaxf(a, red[i][0]);
    b = fmaxf(b, red[i][1]);
  }
  return make_float2(a, b);
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
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  typename Sm::Small &sm = *reinterpret_cast<typename Sm::Small *>(smem + Sm::kSmall);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = warp & 3, half = warp >> 2;       // token rows 16 m .., half of the columns
  const int hk = blockIdx.x % HK;
  const long long slot = blockIdx.x / HK;
  int n, bos, eos, c;
  if (!chunk_of_slot(cu, N, T, slot, status, n, bos, eos, c)) return;
  if (!in_range(status, slot, slots(N, T))) return;
  const int t0 = bos + c * C, len = min(C, eos - t0);
  const int r0 = 16 * m + lane / 4, r1 = r0 + 8, col = 2 * (lane & 3);

  {
    const uint8_t *kq = ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D);
    cp_block(sb, kq, kq_tile_bytes(D));
    cp_commit();
    if (tid == 0) {
      const float2 f = *reinterpret_cast<const float2 *>(kq + kq_tile_bytes(D));
      sm.kq[0] = f.x;
      sm.kq[1] = f.y;
    }
  }
  float aq[NH][4], ak[NH][4];  // dQ, dK: rows r0, r1; columns 8 (half NH + i) + col
  zero(aq);
  zero(ak);
  const int group = HV / HK;
  for (int j = 0; j < group; ++j) {
    const int h = hk * group + j;
    const size_t rec = (size_t)(slot * HV + h);
    const float *Sg = reinterpret_cast<const float *>(ws + lay.state) + rec * D * D;
    const float *Dg = reinterpret_cast<const float *>(ws + lay.dstate) + rec * D * D;
    const float *Ug = reinterpret_cast<const float *>(ws + lay.u) + rec * C * D;
    const float *Xg = reinterpret_cast<const float *>(ws + lay.x) + rec * C * D;
    const float *vec = reinterpret_cast<const float *>(ws + lay.tp + rec * kTpBytes + kVec);
    __syncthreads();  // the previous head has been read
    if (tid < C) {
      sm.G[tid] = vec[kVecG * C + tid];
      sm.E[tid] = vec[kVecE * C + tid];
      sm.beta[tid] = vec[kVecBeta * C + tid];
    }
    if (warp == 7) {
      const float *g0 = g + (size_t)t0 * HV + h;
      gamma_of(load_g(g0, HV, 2 * lane, len), load_g(g0, HV, 2 * lane + 1, len), sm.gamma);
    }
    // S and dS' as planes with one power of two per matrix; <dS', S> from the planes' values.
    Scale ss, ds;
    float cross = 0.f;
    {
      constexpr int kQuads = D * D / 4 / kLocalThreads;
      float4 a[kQuads];
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        a[i] = __ldg(reinterpret_cast<const float4 *>(Sg) + tid + i * kLocalThreads);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(a[i].x), fabsf(a[i].y)), fmaxf(fabsf(a[i].z), fabsf(a[i].w))));
      }
      ss = scale_of(block_max2(big, 0.f, sm.red).x);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int e = 4 * (tid + i * kLocalThreads), r = e / D, cc = e % D;
        uint2 hi, lo;
        split2(a[i].x, a[i].y, ss.inv, hi.x, lo.x);
        split2(a[i].z, a[i].w, ss.inv, hi.y, lo.y);
        const uint32_t at = tile_off<D>(r, cc >> 3) + 2 * (cc & 7);
        *reinterpret_cast<uint2 *>(smem + Sm::kSHi + at) = hi;
        *reinterpret_cast<uint2 *>(smem + Sm::kSLo + at) = lo;
      }
      big = 0.f;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        a[i] = __ldg(reinterpret_cast<const float4 *>(Dg) + tid + i * kLocalThreads);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(a[i].x), fabsf(a[i].y)), fmaxf(fabsf(a[i].z), fabsf(a[i].w))));
      }
      ds = scale_of(block_max2(big, 0.f, sm.red).x);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int e = 4 * (tid + i * kLocalThreads), r = e / D, cc = e % D;
        const uint32_t at = tile_off<D>(r, cc >> 3) + 2 * (cc & 7);
        const uint2 sh = *reinterpret_cast<const uint2 *>(smem + Sm::kSHi + at);
        const uint2 sl = *reinterpret_cast<const uint2 *>(smem + Sm::kSLo + at);
        const float2 h0 = __half22float2(*reinterpret_cast<const __half2 *>(&sh.x));
        const float2 h1 = __half22float2(*reinterpret_cast<const __half2 *>(&sh.y));
        const float2 l0 = __half22float2(*reinterpret_cast<const __half2 *>(&sl.x));
        const float2 l1 = __half22float2(*reinterpret_cast<const __half2 *>(&sl.y));
        cross = fmaf(a[i].x, h0.x + l0.x, cross);
        cross = fmaf(a[i].y, h0.y + l0.y, cross);
        cross = fmaf(a[i].z, h1.x + l1.x, cross);
        cross = fmaf(a[i].w, h1.y + l1.y, cross);
        uint2 hi, lo;
        split2(a[i].x, a[i].y, ds.inv, hi.x, lo.x);
        split2(a[i].z, a[i].w, ds.inv, hi.y, lo.y);
        *reinterpret_cast<uint2 *>(smem + Sm::kDHi + at) = hi;
        *reinterpret_cast<uint2 *>(smem + Sm::kDLo + at) = lo;
      }
    }
    {  // U: four threads per token row, a power of two per row
      const int r = tid >> 2, part = tid & 3;
      constexpr int kQuads = D / 16;
      float4 a[kQuads];
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        a[i] = __ldg(reinterpret_cast<const float4 *>(Ug + r * D) + part + 4 * i);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(a[i].x), fabsf(a[i].y)), fmaxf(fabsf(a[i].z), fabsf(a[i].w))));
      }
      const Scale us = scale_of(quad_max(big));
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int cc = 4 * (part + 4 * i);
        uint2 hi, lo;
        split2(a[i].x, a[i].y, us.inv, hi.x, lo.x);
        split2(a[i].z, a[i].w, us.inv, hi.y, lo.y);
        const uint32_t at = tile_off(r, cc >> 3) + 2 * (cc & 7);
        *reinterpret_cast<uint2 *>(smem + Sm::kU + at) = hi;
        *reinterpret_cast<uint2 *>(smem + Sm::kULo + at) = lo;
      }
      if (part == 0) sm.us[r] = us.s;
    }
    cp_wait<0>();
    __syncthreads();
    const float ks = sm.kq[0], qs = sm.kq[1];

    float dp[4][4], da[4][4];  // rows r0, r1; columns 32 half + 8 i + col
    // A = dO~ or X (rows of this warp's tokens): z = A S^T, dp or da = A U^T.
    auto rows_times = [&](const float *a0p, const float *a1p, bool ok0, bool ok1, float f,
                          float (&z)[NH][4], float (&y)[4][4], float *dot, const Tin *v0, const Tin *v1) {
      float a[2 * KK][4];  // columns 8 i + col of rows r0 (0, 1) and r1 (2, 3)
#pragma unroll
      for (int i = 0; i < 2 * KK; ++i) {
        float2 p = make_float2(0.f, 0.f), q = p;
        if (ok0) p = *reinterpret_cast<const float2 *>(a0p + 8 * i + col);
        if (ok1) q = *reinterpret_cast<const float2 *>(a1p + 8 * i + col);
        a[i][0] = f * p.x; a[i][1] = f * p.y; a[i][2] = f * q.x; a[i][3] = f * q.y;
      }
      if (dot != nullptr) {  // X_r . V_r
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * KK; ++i) {
          if (ok0) d0 += a[i][0] * to_f32(v0[8 * i + col]) + a[i][1] * to_f32(v0[8 * i + col + 1]);
          if (ok1) d1 += a[i][2] * to_f32(v1[8 * i + col]) + a[i][3] * to_f32(v1[8 * i + col + 1]);
        }
        d0 = quad_sum(d0);
        d1 = quad_sum(d1);
        if ((lane & 3) == 0) {
          dot[r0] = d0;
          dot[r1] = d1;
        }
      }
      Scale s0, s1;
      row_scales(a, s0, s1);
      zero(z);
      zero(y);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        uint32_t hi[4], lo[4];
        split_a(a, kk, s0, s1, hi, lo);
#pragma unroll
        for (int np = 0; np < NH / 2; ++np) {
          uint32_t b[4], bl[4];
          load_b<D>(b, sb + Sm::kSHi, half * (D / 2) + 16 * np, 16 * kk);
          load_b<D>(bl, sb + Sm::kSLo, half * (D / 2) + 16 * np, 16 * kk);
          mma(z[2 * np], hi, b[0], b[1]);
          mma(z[2 * np + 1], hi, b[2], b[3]);
          mma(z[2 * np], lo, b[0], b[1]);
          mma(z[2 * np + 1], lo, b[2], b[3]);
          mma(z[2 * np], hi, bl[0], bl[1]);
          mma(z[2 * np + 1], hi, bl[2], bl[3]);
        }
#pragma unroll
        for (int np = 0; np < 2; ++np) {
          if (2 * half + np > m) break;
          uint32_t b[4], bl[4];
          load_b(b, sb + Sm::kU, 32 * half + 16 * np, 16 * kk);
          load_b(bl, sb + Sm::kULo, 32 * half + 16 * np, 16 * kk);
          mma(y[2 * np], hi, b[0], b[1]);
          mma(y[2 * np + 1], hi, b[2], b[3]);
          mma(y[2 * np], lo, b[0], b[1]);
          mma(y[2 * np + 1], lo, b[2], b[3]);
          mma(y[2 * np], hi, bl[0], bl[1]);
          mma(y[2 * np + 1], hi, bl[2], bl[3]);
        }
      }
      const float f0 = s0.s * ss.s, f1 = s1.s * ss.s;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        z[i][0] *= f0; z[i][1] *= f0; z[i][2] *= f1; z[i][3] *= f1;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = *reinterpret_cast<const float2 *>(sm.us + 32 * half + 8 * i + col);
        y[i][0] *= s0.s * u.x; y[i][1] *= s0.s * u.y;
        y[i][2] *= s1.s * u.x; y[i][3] *= s1.s * u.y;
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
    float rg0, rg1;  // what dgamma takes per row
    float z[NH][4];
    const float g0 = sm.G[r0], g1 = sm.G[r1], b0 = sm.beta[r0], b1 = sm.beta[r1];
    {
      const float *p = d_o + ((size_t)t0 * HV + h) * D;
      rows_times(p + (size_t)r0 * HV * D, p + (size_t)r1 * HV * D, r0 < len, r1 < len, scale, z, dp,
                 nullptr, nullptr, nullptr);
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        z[i][0] *= g0; z[i][1] *= g0; z[i][2] *= g1; z[i][3] *= g1;
#pragma unroll
        for (int e = 0; e < 4; ++e) aq[i][e] += z[i][e];
      }
      row_dots(z, Sm::kQ, qs, rg0, rg1);
    }
    {
      const Tin *vp = v + ((size_t)t0 * HV + h) * D;
      rows_times(Xg + r0 * D, Xg + r1 * D, r0 < len, r1 < len, 1.f, z, da, half == 0 ? sm.xv : nullptr,
                 vp + (size_t)r0 * HV * D, vp + (size_t)r1 * HV * D);
      float d0, d1;
      row_dots(z, Sm::kK, ks, d0, d1);
      if ((lane & 3) == 0) {
        sm.zk[half][r0] = d0;
        sm.zk[half][r1] = d1;
      }
      const float f0 = g0 * b0, f1 = g1 * b1;
      rg0 -= f0 * d0;
      rg1 -= f1 * d1;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        ak[i][0] -= f0 * z[i][0]; ak[i][1] -= f0 * z[i][1];
        ak[i][2] -= f1 * z[i][2]; ak[i][3] -= f1 * z[i][3];
      }
    }
    {  // E U dS'^T
      zero(z);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        uint32_t hi[4], lo[4];
        load_a(hi, sb + Sm::kU, 16 * m, 16 * kk);
        load_a(lo, sb + Sm::kULo, 16 * m, 16 * kk);
#pragma unroll
        for (int np = 0; np < NH / 2; ++np) {
          uint32_t b[4], bl[4];
          load_b<D>(b, sb + Sm::kDHi, half * (D / 2) + 16 * np, 16 * kk);
          load_b<D>(bl, sb + Sm::kDLo, half * (D / 2) + 16 * np, 16 * kk);
          mma(z[2 * np], hi, b[0], b[1]);
          mma(z[2 * np + 1], hi, b[2], b[3]);
          mma(z[2 * np], lo, b[0], b[1]);
          mma(z[2 * np + 1], lo, b[2], b[3]);
          mma(z[2 * np], hi, bl[0], bl[1]);
          mma(z[2 * np + 1], hi, bl[2], bl[3]);
        }
      }
      const float f0 = sm.us[r0] * ds.s * sm.E[r0], f1 = sm.us[r1] * ds.s * sm.E[r1];
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        z[i][0] *= f0; z[i][1] *= f0; z[i][2] *= f1; z[i][3] *= f1;
#pragma unroll
        for (int e = 0; e < 4; ++e) ak[i][e] += z[i][e];
      }
      float d0, d1;
      row_dots(z, Sm::kK, ks, d0, d1);
      if ((lane & 3) == 0) {
        sm.tail[half][r0] = d0;
        sm.tail[half][r1] = d1;
      }
    }
    // W, M and their sums over rows and columns; Q K^T and K K^T again, from the tiles.  A token's
    // own term decays by nothing: it stays out of the sums, where it would be added and taken
    // away again, next to which the others may be small.
    float bigw = 0.f, bigm = 0.f;
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
      const float2 gr[2] = {sm.gamma[r0], sm.gamma[r1]};
      float nb[2] = {0.f, 0.f}, rows[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float cs[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1 ? r1 : r0, cc = 32 * half + 8 * i + col + (e & 1);
          const float dec = cc <= r ? decay_between(gr[e >> 1], sm.gamma[cc]) : 0.f;
          const float w = cc <= r ? dp[i][e] * dec : 0.f;
          const float m0 = cc < r ? -da[i][e] * dec : 0.f;  // dA D
          const float mk = m0 * (ks * ks * kk2[i][e]);
          const float b = e >> 1 ? b1 : b0;
          const float x = cc < r ? w * (qs * ks * qk[i][e]) + b * mk : 0.f;
          nb[e >> 1] += mk;
          rows[e >> 1] += x;
          cs[e & 1] += x;
          dp[i][e] = w;
          da[i][e] = b * m0;
          bigw = fmaxf(bigw, fabsf(w));
          bigm = fmaxf(bigm, fabsf(da[i][e]));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float t = col_sum(cs[e]);
          if (lane < 4) sm.cols[m][32 * half + 8 * i + col + e] = t;
        }
      }
      rg0 += quad_sum(rows[0]);
      rg1 += quad_sum(rows[1]);
      nb[0] = quad_sum(nb[0]);
      nb[1] = quad_sum(nb[1]);
      if ((lane & 3) == 0) {
        sm.rows[half][r0] = rg0;
        sm.rows[half][r1] = rg1;
        sm.db[half][r0] = nb[0];
        sm.db[half][r1] = nb[1];
      }
    }
    const float2 big = block_max2(bigw, bigm, sm.red);  // also: U has been read
    const Scale sw = scale_of(big.x), sn = scale_of(big.y);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = tile_off(e ? r1 : r0, 4 * half + i) + 2 * col;
        uint32_t hi, lo;
        split2(dp[i][2 * e], dp[i][2 * e + 1], sw.inv, hi, lo);
        *reinterpret_cast<uint32_t *>(smem + Sm::kU + at) = hi;
        *reinterpret_cast<uint32_t *>(smem + Sm::kU + kTriBytes + at) = lo;
        split2(da[i][2 * e], da[i][2 * e + 1], sn.inv, hi, lo);
        *reinterpret_cast<uint32_t *>(smem + Sm::kU + 2 * kTriBytes + at) = hi;
        *reinterpret_cast<uint32_t *>(smem + Sm::kU + 3 * kTriBytes + at) = lo;
      }
    // <dS', S>, summed in a fixed order
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cross += __shfl_xor_sync(0xffffffffu, cross, off);
    if (lane == 0) sm.red[warp][2] = cross;
    __syncthreads();

    auto times = [&](uint32_t plane, bool transposed, uint32_t tile, float f, float (&out)[NH][4]) {
      zero(z);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (transposed ? kk < m : kk > m) continue;
        uint32_t hi[4], lo[4];
        if (transposed) {
          load_at(hi, plane, 16 * m, 16 * kk);
          load_at(lo, plane + kTriBytes, 16 * m, 16 * kk);
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
#pragma unroll
      for (int i = 0; i < NH; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][e] = fmaf(f, z[i][e], out[i][e]);
    };
    times(sb + Sm::kU, false, sb + Sm::kK, sw.s * ks, aq);
    times(sb + Sm::kU, true, sb + Sm::kQ, sw.s * qs, ak);
    times(sb + Sm::kU + 2 * kTriBytes, false, sb + Sm::kK, sn.s * ks, ak);
    times(sb + Sm::kU + 2 * kTriBytes, true, sb + Sm::kK, sn.s * ks, ak);

    if (warp == 0) {  // dg and dbeta of tokens 2 lane, 2 lane + 1
      double d[2], e = 0.0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        // M's contribution to dbeta has beta left out, so that it holds for beta = 0 too.
        const float b = sm.xv[r] - sm.G[r] * (sm.zk[0][r] + sm.zk[1][r]) + sm.db[0][r] + sm.db[1][r];
        if (r < len) dbeta[(size_t)(t0 + r) * HV + h] = b;
        const double et = (double)sm.tail[0][r] + sm.tail[1][r];
        d[i] = (double)sm.rows[0][r] + sm.rows[1][r] - et -
               ((double)sm.cols[0][r] + sm.cols[1][r] + sm.cols[2][r] + sm.cols[3][r]);
        e += et;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x += sm.red[i][2];
      if (lane == 31) d[1] += e + (double)(sm.G[C - 1] * (x * ss.s));
      double s = d[0] + d[1];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_down_sync(0xffffffffu, s, off);
        if (lane + off < 32) s += o;
      }
      if (2 * lane < len) dg[(size_t)(t0 + 2 * lane) * HV + h] = (float)s;
      if (2 * lane + 1 < len) dg[(size_t)(t0 + 2 * lane + 1) * HV + h] = (float)(s - d[0]);
    }
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
}

template <typename Tin, int D, int NW>
cudaError_t launch_reverse(const int32_t *cu, float scale, int N, int T, int HK, int HV, void *ws,
                           const float *d_o, const float *d_sN, void *dv, float *d_s0, int *status,
                           cudaStream_t s) {
  auto kern = gdr_reverse_kernel<Tin, D, NW>;
  const int bytes = (int)ReverseSmem<D, NW>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)N * HV * (D / (16 * NW));
  if (ctas >= (1LL << 31)) return cudaErrorInvalidValue;
  kern<<<(unsigned)ctas, NW * 32, bytes, s>>>(d_o, d_sN, cu, scale, N, T, HK, HV,
                                              static_cast<uint8_t *>(ws),
                                              layout(N, T, HK, HV, D, true), static_cast<Tin *>(dv),
                                              d_s0, status);
  return cudaGetLastError();
}

template <typename Tin, int D>
cudaError_t launch_typed(const void *v, const float *g, const float *beta, const int32_t *cu,
                         float scale, int N, int T, int HK, int HV, void *ws, const float *d_o,
                         const float *d_sN, void *dq, void *dk, void *dv, float *dg, float *dbeta,
                         float *d_s0, int *status, cudaStream_t s) {
  cudaError_t e;
  // The split of a head over CTAs is the forward's (kda_gdr_state.cu).
  if (D == 64 || (long long)N * HV * 2 <= 148)
    e = launch_reverse<Tin, D, 4>(cu, scale, N, T, HK, HV, ws, d_o, d_sN, dv, d_s0, status, s);
  else
    e = launch_reverse<Tin, D, D == 64 ? 4 : 8>(cu, scale, N, T, HK, HV, ws, d_o, d_sN, dv, d_s0,
                                                status, s);
  if (e != cudaSuccess) return e;
  auto kern = gdr_local_kernel<Tin, D>;
  const int bytes = (int)LocalSmem<D>::kBytes;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long ctas = slots(N, T) * HK;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidValue;
  kern<<<(unsigned)ctas, kLocalThreads, bytes, s>>>(
      static_cast<const Tin *>(v), g, beta, d_o, cu, scale, N, T, HK, HV,
      static_cast<const uint8_t *>(ws), layout(N, T, HK, HV, D, true), static_cast<Tin *>(dq),
      static_cast<Tin *>(dk), dg, dbeta, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_bwd(const void *v, const float *g, const float *beta, const int32_t *cu,
                           float scale, int N, int T, int HK, int HV, int D, kda_dtype dt, void *ws,
                           const float *d_o, const float *d_sN, void *dq, void *dk, void *dv,
                           float *dg, float *dbeta, float *d_s0, int *status, cudaStream_t s) {
  const bool bf = dt == KDA_BF16;
  if (D == 128)
    return bf ? launch_typed<__nv_bfloat16, 128>(v, g, beta, cu, scale, N, T, HK, HV, ws, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s)
              : launch_typed<__half, 128>(v, g, beta, cu, scale, N, T, HK, HV, ws, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s);
  if (D == 64)
    return bf ? launch_typed<__nv_bfloat16, 64>(v, g, beta, cu, scale, N, T, HK, HV, ws, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s)
              : launch_typed<__half, 64>(v, g, beta, cu, scale, N, T, HK, HV, ws, d_o, d_sN, dq, dk, dv, dg, dbeta, d_s0, status, s);
  return cudaErrorInvalidValue;
}

}  // namespace kda
