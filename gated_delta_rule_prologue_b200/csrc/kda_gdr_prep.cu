// Prep pass of the chunked gated delta rule (kda_gdr.cuh): everything of a chunk that no state
// enters, for all chunks at once.  One CTA of four warps per (chunk, value head), 16 token rows
// each: Q K^T, then P; K K^T, then A and T = (I + A)^-1, all out as split fp16 tiles.  The value
// heads of a key head repeat its two products (a tenth of the work) and share their input in L2;
// the first of them writes the KQ record.
//
// T by blocks of 16: the inverses D_i of the diagonal blocks by forward substitution in fp32 (one
// column per lane, a block per warp), then, with warp j owning block column j,
//     T_ij = -D_i (A_ij T_jj + ... + A_i,i-1 T_i-1,j),  i = j + 1 .. 3
// on the tensor cores with split operands.  The products run transposed, T_ij^T = -(sum of
// T_kj^T A_ik^T) D_i^T, because an accumulator then is the next product's A operand as it stands;
// A and D are B operands read along their rows from shared memory.  Block substitution adds
// nothing to the error of the element-wise one, and nothing is divided.
//
// Bound: the latency of one item's steps; four CTAs per SM (128 registers, 47 KB) hide one
// another's: 41% of the issue slots, 53% of the shared-memory wavefronts, and no one stall reason
// above a fifth.  Bytes per item: 2 x 64 x D x 2 in, 33 KB out, and the KQ record once per key head.
// D = 128, 29 920 items, two value heads per key head: 811 us, 1.79 GB, 2.2 TB/s.  Three, five or six
// CTAs per SM: 6, 0 and 10% longer.
#include <type_traits>

#include "kda_gdr.cuh"

namespace kda {
namespace {
using namespace gdr;

constexpr int kThreads = 128;
constexpr int kLdD = 17;

template <int D> struct PrepSmem {
  union {
    uint8_t tiles[2 * C * D * 2];    // K and Q, until their products are in registers
    struct {
      uint8_t a[2 * kTriBytes];      // A hi, A lo (64 x 64 tiles); then T hi, T lo
    } m;
  };
  uint8_t d[4][2][512];              // D_i hi, lo: 16 rows x 32 bytes, pieces swapped in odd row quads
  float diag[4][16][kLdD];           // A's diagonal blocks, then D_i, in fp32
  alignas(16) float2 gamma[4][C];    // a copy per warp
  float beta[4][C];
  float before[4][C];                // per warp: decay from token i to the end of the block before its rows
  float sa[C], sd[4];                // scales of A's rows and of the D_i
  float tmax[4][C];                  // per block column, the largest of T's rows
  float largest[2][4];
};

// The largest magnitude of eight bf16 values, in both halves' running maxima.
__device__ __forceinline__ __nv_bfloat162 max_abs(__nv_bfloat162 m, const uint4 &u) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(h[i]));
  return m;
}
// Eight bf16 values of a tile, scaled by a power of two and rounded to fp16 (exact for values of
// at least 2^-14 of the tile's largest, off by 2^-25 of it below).
__device__ __forceinline__ uint4 to_f16(const uint4 &u, float inv) {
  float2 f[4];
  widen_pairs(u, f, __nv_bfloat16{});
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], make_float2(inv, inv));
  return pack_pairs(f, __half{});
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads, 4)
gdr_prep_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const float *__restrict__ g,
                const float *__restrict__ beta, const int32_t *__restrict__ cu, int N, int T, int HK,
                int HV, uint8_t *__restrict__ ws, Layout lay, int *status) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrepSmem<D> &sm = *reinterpret_cast<PrepSmem<D> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % HV, hk = h / (HV / HK);
  const long long slot = blockIdx.x / HV;
  int n, bos, eos, c;
  if (!chunk_of_slot(cu, N, T, slot, status, n, bos, eos, c)) return;
  if (!in_range(status, slot, slots(N, T))) return;
  const int t0 = bos + c * C, len = min(C, eos - t0);

  // The tiles, zeros behind the sequence's end: in registers until their scale is known (fp16
  // inputs are used as they are).  g and beta are on their way meanwhile.
  constexpr int kPieces = D / 8;                       // 16-byte pieces per row
  constexpr int kEach = C * kPieces / kThreads;        // pieces of each tile per thread
  const float *g0 = g + (size_t)t0 * HV + h;
  const float *beta0 = beta + (size_t)t0 * HV + h;
  uint4 x[2][kEach];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = tid + i * kThreads, row = e / kPieces;
      x[which][i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < len)
        x[which][i] = __ldg(reinterpret_cast<const uint4 *>((which ? q : k) +
                                                            ((size_t)(t0 + row) * HK + hk) * D) +
                            e % kPieces);
    }
  const float ga = load_g(g0, HV, 2 * lane, len), gb = load_g(g0, HV, 2 * lane + 1, len);
  const float ba = lane < len ? __ldg(beta0 + (size_t)lane * HV) : 0.f;  // tokens lane, lane + 32
  const float bb = lane + 32 < len ? __ldg(beta0 + (size_t)(lane + 32) * HV) : 0.f;
  const uint32_t tiles = smem_addr(sm.tiles);
  float ks = 1.f, qs = 1.f;
  if constexpr (std::is_same<Tin, __nv_bfloat16>::value) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
      for (int i = 0; i < kEach; ++i) m = max_abs(m, x[which][i]);
      float big = fmaxf(__low2float(m), __high2float(m));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
      if (lane == 0) sm.largest[which][warp] = big;
    }
    __syncthreads();
    float big[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      big[0] = fmaxf(big[0], sm.largest[0][i]);
      big[1] = fmaxf(big[1], sm.largest[1][i]);
    }
    const Scale sk = scale_of(big[0]), sq = scale_of(big[1]);
    ks = sk.s;
    qs = sq.s;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      x[0][i] = to_f16(x[0][i], sk.inv);
      x[1][i] = to_f16(x[1][i], sq.inv);
    }
  }
  uint8_t *kq = ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D);
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = tid + i * kThreads;
      const uint32_t o = which * kQRows + tile_off<kKq>(e / kPieces, e % kPieces);
      *reinterpret_cast<uint4 *>(sm.tiles + o) = x[which][i];
      if (h % (HV / HK) == 0) *reinterpret_cast<uint4 *>(kq + o) = x[which][i];
    }
  if (tid == 0 && h % (HV / HK) == 0) *reinterpret_cast<float2 *>(kq + kq_tile_bytes(D)) = make_float2(ks, qs);
  __syncthreads();

  const uint32_t at_a = smem_addr(sm.m.a);
  const int w4 = warp;
  const int r0 = 16 * w4 + lane / 4, r1 = r0 + 8, col = 2 * (lane & 3);
  const int last = 2 * w4 + 1;  // the warp's last 8-column block that reaches below the diagonal
  uint8_t *tp = ws + lay.tp + (size_t)(slot * HV + h) * kTpBytes;
  float *vec = reinterpret_cast<float *>(tp + kVec);
  float2 *gamma = sm.gamma[warp];
  gamma_of(ga, gb, gamma);
  sm.beta[w4][lane] = ba;
  sm.beta[w4][lane + 32] = bb;
  __syncwarp();

  // A row's decay since token i < 16 w4 is the decay from i to the end of the block before the
  // warp's rows times that from there on: no factor is above 1, and one exponential per row and
  // column does for all of them.
  const float2 gr[2] = {gamma[r0], gamma[r1]};
  const float2 gs = gamma[max(16 * w4 - 1, 0)];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < 16 * w4) sm.before[w4][lane + 32 * i] = decay_between(gs, gamma[lane + 32 * i]);
  __syncwarp();
  const float from0 = decay_between(gr[0], gs), from1 = decay_between(gr[1], gs);

  // Rows 16 w4 .. of Q K^T D (own = 1: with the diagonal) or beta K K^T D (own = 0: without).
  float x4[8][4];
  auto product = [&](uint32_t rows, float unit, float b0, float b1, int own) {
    zero(x4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
      load_a<kKq>(a, tiles + rows, 16 * w4, 16 * kk);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np > w4) break;
        uint32_t b[4];
        load_b<kKq>(b, tiles, 16 * np, 16 * kk);
        mma(x4[2 * np], a, b[0], b[1]);
        mma(x4[2 * np + 1], a, b[2], b[3]);
      }
    }
    b0 *= unit;
    b1 *= unit;
    const float f0 = b0 * from0, f1 = b1 * from1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i > last) break;
      float(&y)[4] = x4[i];
      if (i < 2 * w4) {
        const float2 d = *reinterpret_cast<const float2 *>(sm.before[w4] + 8 * i + col);
        y[0] = f0 * y[0] * d.x;
        y[1] = f0 * y[1] * d.y;
        y[2] = f1 * y[2] * d.x;
        y[3] = f1 * y[3] * d.y;
        continue;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int cc = 8 * i + col + e;
        const float2 gc = gamma[cc];
        y[e] = cc < r0 + own ? b0 * decay_between(gr[0], gc) * y[e] : 0.f;
        y[e + 2] = cc < r1 + own ? b1 * decay_between(gr[1], gc) * y[e + 2] : 0.f;
      }
    }
  };

  product(kQRows, ks * qs, 1.f, 1.f, 1);
  {
    Scale s0, s1;
    row_scales(x4, s0, s1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i > last) break;  // nothing above the 16 x 16 diagonal blocks is ever read
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, lo;
        split2(x4[i][2 * e], x4[i][2 * e + 1], e ? s1.inv : s0.inv, hi, lo);
        const uint32_t o = tile_off(r0 + 8 * e, i) + 2 * col;
        *reinterpret_cast<uint32_t *>(tp + kP_HI + o) = hi;
        *reinterpret_cast<uint32_t *>(tp + kP_LO + o) = lo;
      }
    }
    if ((lane & 3) == 0) {
      vec[kVecP * C + r0] = s0.s;
      vec[kVecP * C + r1] = s1.s;
    }
    const int t = 16 * w4 + (lane & 15);
    if (lane < 16) {
      vec[kVecG * C + t] = ex2_approx(gamma[t].x + gamma[t].y);
      vec[kVecBeta * C + t] = sm.beta[w4][t];
    } else {
      vec[kVecE * C + t] = decay_between(gamma[C - 1], gamma[t]);
    }
  }

  // A's rows of this warp as planes, its diagonal block in fp32 too.
  product(0, ks * ks, sm.beta[w4][r0], sm.beta[w4][r1], 0);
  __syncthreads();  // the tiles have been read: the planes lie over them
  {
    Scale s0, s1;
    row_scales(x4, s0, s1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i > last) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, lo;
        split2(x4[i][2 * e], x4[i][2 * e + 1], e ? s1.inv : s0.inv, hi, lo);
        const uint32_t o = tile_off(r0 + 8 * e, i) + 2 * col;
        *reinterpret_cast<uint32_t *>(sm.m.a + o) = hi;
        *reinterpret_cast<uint32_t *>(sm.m.a + kTriBytes + o) = lo;
        if (i >= last - 1) {
          float *d = &sm.diag[w4][lane / 4 + 8 * e][8 * (i - last + 1) + col];
          d[0] = x4[i][2 * e];
          d[1] = x4[i][2 * e + 1];
        }
      }
    }
    if ((lane & 3) == 0) {
      sm.sa[r0] = s0.s;
      sm.sa[r1] = s1.s;
    }
  }
  __syncwarp();
  // D_i of this warp's block: lane = column (lanes 16-31 repeat 0-15).
  {
    const int cc = lane & 15;
    float x[16], big = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float t = r == cc ? 1.f : 0.f, t2 = 0.f;
#pragma unroll
      for (int i = 0; i < r; ++i) {  // two sums: half the chain
        float &s = i & 1 ? t2 : t;
        s = fmaf(-sm.diag[w4][r][i], x[i], s);
      }
      x[r] = t + t2;
      big = fmaxf(big, fabsf(x[r]));
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    const Scale sd = scale_of(big);
    __syncwarp();
    if (lane < 16) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        sm.diag[w4][r][cc] = x[r];
        const float v = x[r] * sd.inv;
        const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
        const int o = r * 32 + (((cc >> 3) ^ ((r >> 2) & 1)) << 4) + 2 * (cc & 7);
        *reinterpret_cast<__half *>(&sm.d[w4][0][o]) = hi;
        *reinterpret_cast<__half *>(&sm.d[w4][1][o]) = lo;
      }
    }
    if (lane == 0) sm.sd[w4] = sd.s;
  }
  __syncthreads();
  // Block column w4 of T, transposed: tt[i] has rows c = 16 w4 + lane/4 (+8), columns r = 16 i ..
  // T_kj is split once and enters the sums of all i > k; only the sum that T_k+1,j waits for is
  // on the path to the next step.
  float tt[4][2][4], sum[4][2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    zero(tt[i]);
    zero(sum[i]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < w4) continue;
    if (k == w4) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int f = 0; f < 4; ++f)
          tt[k][e][f] = sm.diag[w4][8 * e + col + (f & 1)][lane / 4 + 8 * (f >> 1)];
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 s = *reinterpret_cast<const float2 *>(sm.sa + 16 * k + 8 * e + col);
        sum[k][e][0] *= s.x; sum[k][e][1] *= s.y; sum[k][e][2] *= s.x; sum[k][e][3] *= s.y;
      }
      Scale t0s, t1s;
      row_scales(sum[k], t0s, t1s);
      uint32_t hi[4], lo[4], b[4], bl[4];
      const int m = lane >> 3, r = (m >> 1) * 8 + (lane & 7);
      const uint32_t o = r * 32 + (((m & 1) ^ ((r >> 2) & 1)) << 4);
      ldsm4(b, smem_addr(sm.d[k][0]) + o);
      ldsm4(bl, smem_addr(sm.d[k][1]) + o);
      split_a(sum[k], 0, t0s, t1s, hi, lo);
      float y[2][4], y2[2][4];  // two chains of MMAs
      mma0(y[0], hi, b[0], b[1]);
      mma0(y[1], hi, b[2], b[3]);
      mma0(y2[0], lo, b[0], b[1]);
      mma0(y2[1], lo, b[2], b[3]);
      mma(y2[0], hi, bl[0], bl[1]);
      mma(y2[1], hi, bl[2], bl[3]);
      const float f0 = -sm.sd[k] * t0s.s, f1 = -sm.sd[k] * t1s.s;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int f = 0; f < 4; ++f) tt[k][e][f] = (f >> 1 ? f1 : f0) * (y[e][f] + y2[e][f]);
    }
    if (k == 3) continue;
    Scale t0s, t1s;
    row_scales(tt[k], t0s, t1s);
    uint32_t hi[4], lo[4];
    split_a(tt[k], 0, t0s, t1s, hi, lo);
#pragma unroll
    for (int i = k + 1; i < 4; ++i) {
      uint32_t b[4], bl[4];
      load_b(b, at_a, 16 * i, 16 * k);
      load_b(bl, at_a + kTriBytes, 16 * i, 16 * k);
      float y[2][4], y2[2][4];
      mma0(y[0], hi, b[0], b[1]);
      mma0(y[1], hi, b[2], b[3]);
      mma0(y2[0], lo, b[0], b[1]);
      mma0(y2[1], lo, b[2], b[3]);
      mma(y2[0], hi, bl[0], bl[1]);
      mma(y2[1], hi, bl[2], bl[3]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int f = 0; f < 4; ++f)
          sum[i][e][f] = fmaf(f >> 1 ? t1s.s : t0s.s, y[e][f] + y2[e][f], sum[i][e][f]);
    }
  }
  next_kernel_may_start();
  // Scales of T's rows (its columns are spread over the warps).
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w4) continue;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        float v = fmaxf(fabsf(tt[i][e][f]), fabsf(tt[i][e][f + 2]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        if (lane < 4) sm.tmax[w4][16 * i + 8 * e + col + f] = v;
      }
  }
  __syncthreads();  // also: A's planes have been read
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w4) continue;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float inv[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int r = 16 * i + 8 * e + col + f;
        float v = sm.tmax[0][r];
#pragma unroll
        for (int jj = 1; jj < 4; ++jj)
          if (jj <= i) v = fmaxf(v, sm.tmax[jj][r]);
        const Scale s = scale_of(v);
        inv[f] = s.inv;
        if (i == w4 && lane < 4) vec[kVecT * C + r] = s.s;
      }
      split2(tt[i][e][0] * inv[0], tt[i][e][1] * inv[1], 1.f, hi[2 * e], lo[2 * e]);
      split2(tt[i][e][2] * inv[0], tt[i][e][3] * inv[1], 1.f, hi[2 * e + 1], lo[2 * e + 1]);
    }
    const int m = lane >> 3;
    const uint32_t o = tile_off(16 * i + (m >> 1) * 8 + (lane & 7), 2 * w4 + (m & 1));
    stsm4t(at_a + o, hi[0], hi[1], hi[2], hi[3]);
    stsm4t(at_a + kTriBytes + o, lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();
  for (int i = tid; i < 2 * kTriBytes / 16; i += 128)
    *reinterpret_cast<uint4 *>(tp + kT_HI + i * 16) = *reinterpret_cast<const uint4 *>(sm.m.a + i * 16);
}

template <typename Tin, int D>
cudaError_t launch_typed(const void *q, const void *k, const float *g, const float *beta,
                         const int32_t *cu, int N, int T, int HK, int HV, void *ws,
                         const Layout &lay, int *status, cudaStream_t s) {
  auto kern = gdr_prep_kernel<Tin, D>;
  constexpr int bytes = (int)sizeof(PrepSmem<D>);
  const cudaError_t e = allow_smem<bytes>(kern);
  if (e != cudaSuccess) return e;
  const long long ctas = slots(N, T) * HV;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidValue;
  kern<<<(unsigned)ctas, kThreads, bytes, s>>>(
      static_cast<const Tin *>(q), static_cast<const Tin *>(k), g, beta, cu, N, T, HK, HV,
      static_cast<uint8_t *>(ws), lay, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_prep(const void *q, const void *k, const float *g, const float *beta,
                            const int32_t *cu, int N, int T, int HK, int HV, int D, kda_dtype dt,
                            void *ws, const Layout &lay, int *status, cudaStream_t s) {
  const bool bf = dt == KDA_BF16;
  if (D == 128)
    return bf ? launch_typed<__nv_bfloat16, 128>(q, k, g, beta, cu, N, T, HK, HV, ws, lay, status, s)
              : launch_typed<__half, 128>(q, k, g, beta, cu, N, T, HK, HV, ws, lay, status, s);
  if (D == 64)
    return bf ? launch_typed<__nv_bfloat16, 64>(q, k, g, beta, cu, N, T, HK, HV, ws, lay, status, s)
              : launch_typed<__half, 64>(q, k, g, beta, cu, N, T, HK, HV, ws, lay, status, s);
  return cudaErrorInvalidValue;
}

}  // namespace kda
