// Prep pass of the chunked gated delta rule (kda_gdr.cuh): everything of a chunk that no state
// enters, for all chunks at once.  One CTA per (chunk, key head): the products K K^T and Q K^T
// are shared by the key head's value heads and stay in registers; per value head the decay
// matrix, P, A and T = (I + A)^-1 follow and go out as split fp16 tiles.
//
// T: the inverses of the four 16 x 16 diagonal blocks by forward substitution (one column per
// thread), then [[X, 0], [-Y A21 X, Y]] from blocks X, Y of 16 to 32 and from 32 to 64, in fp32
// on the CUDA cores.  The substitution's error is that of fp32; nothing is divided.
//
// Bound: the CTA's chain of barriers (products, substitution, four small products); several CTAs
// per SM hide one another's.  Bytes: 2 x 64 x D in and out per key head, 33 KB out per value head.
#include <type_traits>

#include "kda_gdr.cuh"

namespace kda {
namespace {
using namespace gdr;

constexpr int kThreads = 256;
constexpr int kLd = C + 1;      // row stride of the fp32 matrices
constexpr int kLdM = 33;

template <int D> struct PrepSmem {
  union {
    uint8_t tiles[2 * C * D * 2];        // K, Q (until the products are in registers)
    struct {
      float A[C][kLd], T[C][kLd], M[32][kLdM];
    } m;
  };
  double gamma[C];
  float beta[C];
  float largest[2][8];
};

// Eight 16-bit values of a tile, scaled by a power of two and rounded to fp16 (exact for bf16
// values of at least 2^-14 of the tile's largest, off by 2^-25 of it below).
__device__ __forceinline__ uint4 to_f16(const uint4 &u, float inv, __nv_bfloat16) {
  float2 f[4];
  widen_pairs(u, f, __nv_bfloat16{});
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], make_float2(inv, inv));
  return pack_pairs(f, __half{});
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads, 3)
gdr_prep_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const float *__restrict__ g,
                const float *__restrict__ beta, const int32_t *__restrict__ cu, int N, int T, int HK,
                int HV, uint8_t *__restrict__ ws, Layout lay, int *status) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrepSmem<D> &sm = *reinterpret_cast<PrepSmem<D> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x % HK;
  const long long slot = blockIdx.x / HK;
  int n, bos, eos, c;
  if (!chunk_of_slot(cu, N, T, slot, status, n, bos, eos, c)) return;
  if (!in_range(status, slot, slots(N, T))) return;
  const int t0 = bos + c * C, len = min(C, eos - t0);

  // The tiles as they are, zeros behind the sequence's end.
  constexpr int kPieces = D / 8;  // 16-byte pieces per row
  const uint32_t tiles = smem_addr(sm.tiles);
  for (int i = tid; i < 2 * C * kPieces; i += kThreads) {
    const int which = i / (C * kPieces), row = i / kPieces % C, c8 = i % kPieces;
    const Tin *src = (which ? q : k) + ((size_t)(t0 + min(row, len - 1)) * HK + hk) * D + c8 * 8;
    cp16(tiles + which * kq_tile_bytes(D) + tile_off(row, c8), src, row < len);
  }
  cp_commit();
  cp_wait<0>();
  __syncthreads();

  // Scales: fp16 inputs are used as they are.
  float ks = 1.f, qs = 1.f;
  uint8_t *kq = ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D);
  if constexpr (std::is_same<Tin, __nv_bfloat16>::value) {
    float big[2] = {0.f, 0.f};
#pragma unroll
    for (int which = 0; which < 2; ++which)
      for (int i = tid; i < C * kPieces; i += kThreads) {
        float2 f[4];
        widen_pairs(*reinterpret_cast<const uint4 *>(sm.tiles + which * kq_tile_bytes(D) + i * 16), f,
                    __nv_bfloat16{});
#pragma unroll
        for (int e = 0; e < 4; ++e) big[which] = fmaxf(big[which], fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
      }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        big[which] = fmaxf(big[which], __shfl_xor_sync(0xffffffffu, big[which], off));
      if (lane == 0) sm.largest[which][warp] = big[which];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      big[0] = fmaxf(big[0], sm.largest[0][i]);
      big[1] = fmaxf(big[1], sm.largest[1][i]);
    }
    const Scale sk = scale_of(big[0]), sq = scale_of(big[1]);
    ks = sk.s;
    qs = sq.s;
#pragma unroll
    for (int which = 0; which < 2; ++which)
      for (int i = tid; i < C * kPieces; i += kThreads) {
        uint4 *p = reinterpret_cast<uint4 *>(sm.tiles + which * kq_tile_bytes(D) + i * 16);
        const uint4 h = to_f16(*p, which ? sq.inv : sk.inv, __nv_bfloat16{});
        *p = h;
        *reinterpret_cast<uint4 *>(kq + which * kq_tile_bytes(D) + i * 16) = h;
      }
    __syncthreads();
  } else {
    for (int i = tid; i < 2 * C * kPieces; i += kThreads)
      *reinterpret_cast<uint4 *>(kq + i * 16) = *reinterpret_cast<const uint4 *>(sm.tiles + i * 16);
  }
  if (tid == 0) *reinterpret_cast<float2 *>(kq + 2 * kq_tile_bytes(D)) = make_float2(ks, qs);

  // Warps 0-3: rows 16 w of K K^T; warps 4-7: of Q K^T.  Blocks above the diagonal are not needed.
  const int w4 = warp & 3;
  const bool is_q = warp >= 4;
  float acc[8][4];
  zero(acc);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    uint32_t a[4];
    load_a(a, tiles + (is_q ? kq_tile_bytes(D) : 0), 16 * w4, 16 * kk);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np > w4) break;
      uint32_t b[4];
      load_b(b, tiles, 16 * np, 16 * kk);
      mma(acc[2 * np], a, b[0], b[1]);
      mma(acc[2 * np + 1], a, b[2], b[3]);
    }
  }
  const float unit = is_q ? ks * qs : ks * ks;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] *= unit;

  const int r0 = 16 * w4 + lane / 4, col = 2 * (lane & 3);
  const int group = HV / HK;
  for (int j = 0; j < group; ++j) {
    const int h = hk * group + j;
    __syncthreads();  // the tiles, or the previous head's matrices, have been read
    if (warp == 0) {  // gamma: tokens 2 lane, 2 lane + 1
      const int ta = 2 * lane, tb = ta + 1;
      const size_t at = (size_t)(t0 + ta) * HV + h;
      const float ga = ta < len ? floor_g(__ldg(g + at)) : 0.f;
      const float gb = tb < len ? floor_g(__ldg(g + at + HV)) : 0.f;
      double s = (double)ga + gb;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
      }
      sm.gamma[tb] = s;
      sm.gamma[ta] = s - gb;
    } else if (warp == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        sm.beta[t] = t < len ? __ldg(beta + (size_t)(t0 + t) * HV + h) : 0.f;
      }
    }
    __syncthreads();
    uint8_t *tp = ws + lay.tp + (size_t)(slot * HV + h) * kTpBytes;
    float *vec = reinterpret_cast<float *>(tp + kVec);
    const double gr[2] = {sm.gamma[r0], sm.gamma[r0 + 8]};
    if (!is_q) {
      const float br[2] = {sm.beta[r0], sm.beta[r0 + 8]};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 8 * (e >> 1), cc = 8 * i + col + (e & 1);
          sm.m.A[r][cc] = cc < r ? br[e >> 1] * expf((float)(gr[e >> 1] - sm.gamma[cc])) * acc[i][e] : 0.f;
        }
    } else {
      float p[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 8 * (e >> 1), cc = 8 * i + col + (e & 1);
          p[i][e] = cc <= r ? expf((float)(gr[e >> 1] - sm.gamma[cc])) * acc[i][e] : 0.f;
        }
      Scale s0, s1;
      row_scales(p, s0, s1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t hi, lo;
          split2(p[i][2 * e], p[i][2 * e + 1], e ? s1.inv : s0.inv, hi, lo);
          const uint32_t at = tile_off(r0 + 8 * e, i) + 2 * col;
          *reinterpret_cast<uint32_t *>(tp + kP_HI + at) = hi;
          *reinterpret_cast<uint32_t *>(tp + kP_LO + at) = lo;
        }
      if ((lane & 3) == 0) {
        vec[kVecP * C + r0] = s0.s;
        vec[kVecP * C + r0 + 8] = s1.s;
      }
    }
    if (tid < C) {
      const double last = sm.gamma[C - 1];
      vec[kVecG * C + tid] = expf((float)sm.gamma[tid]);
      vec[kVecE * C + tid] = expf((float)(last - sm.gamma[tid]));
      vec[kVecBeta * C + tid] = sm.beta[tid];
    }
    __syncthreads();

    // T.  Diagonal blocks: thread = (block, column).
    if (tid < C) {
      const int b = tid & ~15, cc = tid & 15;
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float t = r == cc ? 1.f : 0.f;
#pragma unroll
        for (int i = 0; i < r; ++i) t = fmaf(-sm.m.A[b + r][b + i], x[i], t);
        x[r] = t;
        sm.m.T[b + r][b + cc] = t;
      }
    }
    __syncthreads();
    // 16 -> 32: block rows 16..31 of each half, M = A21 X, then -Y M.
    {
      const int half = tid >> 7, r = (tid >> 3) & 15, c2 = 2 * (tid & 7), o = 32 * half;
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = sm.m.A[o + 16 + r][o + i];
        m0 = fmaf(a, sm.m.T[o + i][o + c2], m0);
        m1 = fmaf(a, sm.m.T[o + i][o + c2 + 1], m1);
      }
      sm.m.M[16 * half + r][c2] = m0;
      sm.m.M[16 * half + r][c2 + 1] = m1;
      __syncthreads();
      m0 = m1 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y = sm.m.T[o + 16 + r][o + 16 + i];
        m0 = fmaf(y, sm.m.M[16 * half + i][c2], m0);
        m1 = fmaf(y, sm.m.M[16 * half + i][c2 + 1], m1);
      }
      sm.m.T[o + 16 + r][o + c2] = -m0;
      sm.m.T[o + 16 + r][o + c2 + 1] = -m1;
      sm.m.T[o + r][o + 16 + c2] = 0.f;      // above the diagonal
      sm.m.T[o + r][o + 16 + c2 + 1] = 0.f;
    }
    __syncthreads();
    // 32 -> 64.
    {
      const int r = tid >> 3, c4 = 4 * (tid & 7);
      float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const float a = sm.m.A[32 + r][i];
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = fmaf(a, sm.m.T[i][c4 + e], m[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sm.m.M[r][c4 + e] = m[e];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = 0.f;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const float y = sm.m.T[32 + r][32 + i];
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = fmaf(y, sm.m.M[i][c4 + e], m[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sm.m.T[32 + r][c4 + e] = -m[e];
    }
    __syncthreads();
    // Rows out: four threads per row, 16 columns each; nothing above the 16 x 16 diagonal blocks
    // is ever read.
    {
      const int r = tid >> 2, b = tid & 3;
      float x[16], big = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = b <= r / 16 ? sm.m.T[r][16 * b + e] : 0.f;
        big = fmaxf(big, fabsf(x[e]));
      }
      const Scale s = scale_of(quad_max(big));
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) split2(x[2 * e], x[2 * e + 1], s.inv, hi[e], lo[e]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = tile_off(r, 2 * b + e);
        *reinterpret_cast<uint4 *>(tp + kT_HI + at) =
            make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
        *reinterpret_cast<uint4 *>(tp + kT_LO + at) =
            make_uint4(lo[4 * e], lo[4 * e + 1], lo[4 * e + 2], lo[4 * e + 3]);
      }
      if (b == 0) vec[kVecT * C + r] = s.s;
    }
  }
}

template <typename Tin, int D>
cudaError_t launch_typed(const void *q, const void *k, const float *g, const float *beta,
                         const int32_t *cu, int N, int T, int HK, int HV, void *ws, bool bwd,
                         int *status, cudaStream_t s) {
  auto kern = gdr_prep_kernel<Tin, D>;
  const int bytes = (int)sizeof(PrepSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long ctas = slots(N, T) * HK;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidValue;
  kern<<<(unsigned)ctas, kThreads, bytes, s>>>(
      static_cast<const Tin *>(q), static_cast<const Tin *>(k), g, beta, cu, N, T, HK, HV,
      static_cast<uint8_t *>(ws), layout(N, T, HK, HV, D, bwd), status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_prep(const void *q, const void *k, const float *g, const float *beta,
                            const int32_t *cu, int N, int T, int HK, int HV, int D, kda_dtype dt,
                            void *ws, bool bwd, int *status, cudaStream_t s) {
  const bool bf = dt == KDA_BF16;
  if (D == 128)
    return bf ? launch_typed<__nv_bfloat16, 128>(q, k, g, beta, cu, N, T, HK, HV, ws, bwd, status, s)
              : launch_typed<__half, 128>(q, k, g, beta, cu, N, T, HK, HV, ws, bwd, status, s);
  if (D == 64)
    return bf ? launch_typed<__nv_bfloat16, 64>(q, k, g, beta, cu, N, T, HK, HV, ws, bwd, status, s)
              : launch_typed<__half, 64>(q, k, g, beta, cu, N, T, HK, HV, ws, bwd, status, s);
  return cudaErrorInvalidValue;
}

}  // namespace kda
