// Gated delta rule with one decay per head and token, token by token.
//
// Per value head h with state S (D x D, stored value-major: row j holds S[:, j]), key head
// h / (HV / HK), a = exp(g_t):
//     S' = a S;  e = v_t - S'^T k_t;  S = S' + beta_t k_t e^T;  o_t = scale S^T q_t
// The rows j of the stored state are independent of one another given k_t, q_t:
//     p_j = <S'_j, k>,  r_j = <S'_j, q>,  be_j = beta (v_j - p_j)
//     S_j = S'_j + be_j k,  o_j = scale (r_j + be_j <k, q>)
// so a warp owns whole rows and keeps them in registers for all tokens of its sequence:
// the state is read and written once per call, whatever the number of tokens.  D/16 lanes
// share a row with 16 values each (four float4 accesses that together cover 128 contiguous
// bytes per row), so a dot product ends in log2(D/16) shuffles, and a warp's shuffles serve
// 512/D rows at once.  No shared memory and no barrier: k and q come through L1.
//
// Bound: one token per sequence is HBM-bound on the state (8 D^2 bytes per head); many
// tokens are bound by the latency of one token's step (two dot products and the update).  D = 128:
// one token each for 24 576 heads 472 us, 3.26 GB, 6.9 TB/s; one to five tokens each for 1024 heads 29 us
// of 21 for the states' bytes (fewer rows per warp, and so more warps: 35); 8 heads 2.9 us.
// Head split: with few (sequence, head) pairs a head's rows are spread over four CTAs, so
// that its 64 KiB come through four SMs instead of one.
#include "kda_common.cuh"

namespace kda {
namespace {

template <int D> struct RecShape {
  static constexpr int kPerLane = D >= 32 ? 16 : 8;   // state values of a row per lane
  static constexpr int kLanes = D / kPerLane;         // lanes per row
  static constexpr int kRows = 32 / kLanes;           // rows per warp access
  static constexpr int kWarps = D / kRows < 8 ? D / kRows : 8;
  static constexpr int kGroups = D / (kRows * kWarps);  // row groups per warp, whole head per CTA
};

// Four consecutive elements as stored.
template <typename T> struct Raw4 { uint2 u; };
template <> struct Raw4<float> { float4 u; };
__device__ __forceinline__ void widen4(const Raw4<float> &r, float *f) {
  f[0] = r.u.x; f[1] = r.u.y; f[2] = r.u.z; f[3] = r.u.w;
}
__device__ __forceinline__ void widen4(const Raw4<__nv_bfloat16> &r, float *f) {
  f[0] = __uint_as_float(r.u.x << 16); f[1] = __uint_as_float(r.u.x & 0xffff0000u);
  f[2] = __uint_as_float(r.u.y << 16); f[3] = __uint_as_float(r.u.y & 0xffff0000u);
}
__device__ __forceinline__ void widen4(const Raw4<__half> &r, float *f) {
  const __half2 *h = reinterpret_cast<const __half2 *>(&r.u);
  const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// What one token brings to a lane.
template <typename Tin, int D, int G> struct Token {
  Raw4<Tin> k[RecShape<D>::kPerLane / 4], q[RecShape<D>::kPerLane / 4];
  Tin v[G];
  float g, beta;
};

template <typename Tin, int D, int G>
__global__ void __launch_bounds__(RecShape<D>::kWarps * 32, G >= 4 && sizeof(Tin) == 2 ? 2 : 1)
gdr_recurrent_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k,
                     const Tin *__restrict__ v, const float *__restrict__ g,
                     const float *__restrict__ beta, float scale, const float *s0,
                     const int32_t *__restrict__ cu, bool one_token, int T, int HK, int HV,
                     float *__restrict__ o, float *sN, int *status) {
  using Sh = RecShape<D>;
  constexpr int P = Sh::kPerLane, L = Sh::kLanes, R = Sh::kRows;
  constexpr int kSplit = Sh::kGroups / G;  // CTAs per head
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % L, rsub = lane / L;
  const int part = blockIdx.x % kSplit;
  const int nh = blockIdx.x / kSplit;
  const int n = nh / HV, h = nh % HV, hk = h / (HV / HK);
  int bos = n, eos = n + 1;
  if (!one_token) seq_bounds(cu, n, T, status, bos, eos);
  if (!in_range(status, eos, (long long)T + 1)) return;
  const int row0 = (part * Sh::kWarps + warp) * G * R + rsub;  // this lane's first row

  auto load = [&](int t) {
    Token<Tin, D, G> x;
    const size_t kb = ((size_t)t * HK + hk) * D + 4 * sub, hb = (size_t)t * HV + h;
#pragma unroll
    for (int i = 0; i < P / 4; ++i) {
      x.k[i].u = __ldg(reinterpret_cast<const decltype(x.k[i].u) *>(k + kb + 4 * L * i));
      x.q[i].u = __ldg(reinterpret_cast<const decltype(x.q[i].u) *>(q + kb + 4 * L * i));
    }
#pragma unroll
    for (int i = 0; i < G; ++i) x.v[i] = v[hb * D + row0 + i * R];
    x.g = __ldg(g + hb);
    x.beta = __ldg(beta + hb);
    return x;
  };

  Token<Tin, D, G> tok;
  if (bos < eos) tok = load(bos);
  const size_t base = (size_t)nh * D * D;
  float s[G][P];
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int c = 0; c < P / 4; ++c) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0)
        x = __ldcs(reinterpret_cast<const float4 *>(s0 + base + (size_t)(row0 + i * R) * D + 4 * sub +
                                                    4 * L * c));
      s[i][4 * c] = x.x; s[i][4 * c + 1] = x.y; s[i][4 * c + 2] = x.z; s[i][4 * c + 3] = x.w;
    }

  for (int t = bos; t < eos; ++t) {
    float kf[P], qf[P], vf[G];
#pragma unroll
    for (int c = 0; c < P / 4; ++c) {
      widen4(tok.k[c], kf + 4 * c);
      widen4(tok.q[c], qf + 4 * c);
    }
#pragma unroll
    for (int i = 0; i < G; ++i) vf[i] = to_f32(tok.v[i]);
    const float a = expf(tok.g), b = tok.beta;
    if (t + 1 < eos) tok = load(t + 1);
    float kq = 0.f;
#pragma unroll
    for (int c = 0; c < P; ++c) kq = fmaf(kf[c], qf[c], kq);
    float pk[G], pq[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      pk[i] = pq[i] = 0.f;
#pragma unroll
      for (int c = 0; c < P; ++c) {
        s[i][c] *= a;
        pk[i] = fmaf(s[i][c], kf[c], pk[i]);
        pq[i] = fmaf(s[i][c], qf[c], pq[i]);
      }
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) {
      kq += __shfl_xor_sync(0xffffffffu, kq, off);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        pk[i] += __shfl_xor_sync(0xffffffffu, pk[i], off);
        pq[i] += __shfl_xor_sync(0xffffffffu, pq[i], off);
      }
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float be = b * (vf[i] - pk[i]);
#pragma unroll
      for (int c = 0; c < P; ++c) s[i][c] = fmaf(be, kf[c], s[i][c]);
      if (sub == 0) o[((size_t)t * HV + h) * D + row0 + i * R] = scale * fmaf(be, kq, pq[i]);
    }
  }

  if (sN) {
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int c = 0; c < P / 4; ++c)
        __stcs(reinterpret_cast<float4 *>(sN + base + (size_t)(row0 + i * R) * D + 4 * sub +
                                          4 * L * c),
               make_float4(s[i][4 * c], s[i][4 * c + 1], s[i][4 * c + 2], s[i][4 * c + 3]));
  }
}

// The CTAs below which a head's rows are split: two whole-head CTAs fit an SM, and with
// fewer than that many heads a split leaves no SM with less to do.
constexpr long long kSplitBelow = 2 * 148;

template <typename Tin, int D>
cudaError_t launch_typed(const void *q, const void *k, const void *v, const float *g,
                         const float *beta, float scale, const float *s0, const int32_t *cu,
                         bool one_token, int N, int T, int HK, int HV, float *o, float *sN,
                         int *status, cudaStream_t s) {
  using Sh = RecShape<D>;
  const long long heads = (long long)N * HV;
  auto go = [&](auto kern, int split) {
    if (heads * split >= (1LL << 31)) return cudaErrorInvalidValue;
    kern<<<(unsigned)(heads * split), Sh::kWarps * 32, 0, s>>>(
        static_cast<const Tin *>(q), static_cast<const Tin *>(k), static_cast<const Tin *>(v), g,
        beta, scale, s0, cu, one_token, T, HK, HV, o, sN, status);
    return cudaGetLastError();
  };
  if constexpr (Sh::kGroups > 1) {
    if (heads < kSplitBelow) return go(gdr_recurrent_kernel<Tin, D, 1>, Sh::kGroups);
  }
  return go(gdr_recurrent_kernel<Tin, D, Sh::kGroups>, 1);
}

template <typename Tin>
cudaError_t launch_d(int D, const void *q, const void *k, const void *v, const float *g,
                     const float *beta, float scale, const float *s0, const int32_t *cu,
                     bool one_token, int N, int T, int HK, int HV, float *o, float *sN,
                     int *status, cudaStream_t s) {
  switch (D) {
    case 16: return launch_typed<Tin, 16>(q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
    case 32: return launch_typed<Tin, 32>(q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
    case 64: return launch_typed<Tin, 64>(q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
    case 128: return launch_typed<Tin, 128>(q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_gdr_recurrent(const void *q, const void *k, const void *v, const float *g,
                                 const float *beta, float scale, const float *s0,
                                 const int32_t *cu, bool one_token, int N, int T, int HK, int HV,
                                 int D, kda_dtype dt, float *o, float *sN, int *status,
                                 cudaStream_t s) {
  if (dt == KDA_BF16)
    return launch_d<__nv_bfloat16>(D, q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
  if (dt == KDA_F16)
    return launch_d<__half>(D, q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
  return launch_d<float>(D, q, k, v, g, beta, scale, s0, cu, one_token, N, T, HK, HV, o, sN, status, s);
}

}  // namespace kda
