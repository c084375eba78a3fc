// Backward of the output epilogue out = o r * weight * sigmoid(gate), r = 1/sqrt(mean o^2 + eps)
// (kda_epilogue.cu).  With u = o r, s = sigmoid(gate), d = dL/dout and dn = d s weight:
//     d_o      = r (dn - u mean(dn u))
//     d_gate   = d u weight s (1 - s)
//     d_weight = sum over rows of d s u
// HBM-bound: D/4 lanes own one (token, head) row as in the forward, two rows per lane group
// in flight; the two row sums (o^2, then dn u) are xor shuffles inside the row's lanes.
// s (1 - s) is e / (1 + e)^2 with e = exp(-|gate|), so neither end of the sigmoid cancels.
// d_weight: each thread sums its four channels over the rows of its grid-stride walk, the
// CTA adds its threads' sums in a fixed order and writes one row of the workspace; a second
// kernel adds the CTAs' rows in a fixed order.  The grid depends on the sizes alone and no
// atomics are used, so repeated calls give the same bits.
// Bytes per row: 8 D (o, d_o) + 3 D sizeof(dt) (gate, d_out, d_gate).  8192 tokens, 32 heads of 128 in
// bf16: 82 us, 470 MB, 5.7 TB/s (77 us and 6.1 TB/s of it this kernel, the rest the weights' second).
#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsInFlight = 2;
constexpr int kMaxCtas = 148 * 4;  // one wave (64 registers: four CTAs per SM)

template <typename T> struct Quad { uint2 u; };
template <> struct Quad<float> { float4 u; };
template <typename T> __device__ __forceinline__ void unpack(const Quad<T> &r, float (&f)[4]) {
  const T *h = reinterpret_cast<const T *>(&r.u);
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = to_f32(h[e]);
}
template <typename T> __device__ __forceinline__ Quad<T> pack(const float (&f)[4]) {
  Quad<T> r;
  T *h = reinterpret_cast<T *>(&r.u);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = from_f32<T>(f[e]);
  return r;
}

template <typename Tg, int D>
__global__ void __launch_bounds__(kThreads)
epilogue_bwd_kernel(const float *__restrict__ o, const Tg *__restrict__ gate,
                    const float *__restrict__ weight, float eps, const Tg *__restrict__ d_out,
                    long long rows, float *__restrict__ d_o, Tg *__restrict__ d_gate,
                    float *__restrict__ partial) {
  constexpr int LPR = D / 4, RPW = 32 / LPR;
  __shared__ float sums[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR, d0 = 4 * sub;
  const long long nwarps = (long long)gridDim.x * kWarps;
  const float4 w4 = __ldg(reinterpret_cast<const float4 *>(weight + d0));
  const float w[4] = {w4.x, w4.y, w4.z, w4.w};
  float dw[4] = {0.f, 0.f, 0.f, 0.f};
  // A warp's first row decides its loop, so that all lanes make the same trips.
  for (long long wrow = ((long long)blockIdx.x * kWarps + warp) * RPW; wrow < rows;
       wrow += nwarps * RPW * kRowsInFlight) {
    float4 x4[kRowsInFlight];
    Quad<Tg> z4[kRowsInFlight], g4[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const long long row = wrow + (long long)i * nwarps * RPW + lane / LPR;
      const size_t at = (size_t)(row < rows ? row : 0) * D + d0;
      x4[i] = __ldcs(reinterpret_cast<const float4 *>(o + at));
      z4[i] = *reinterpret_cast<const Quad<Tg> *>(gate + at);
      g4[i] = *reinterpret_cast<const Quad<Tg> *>(d_out + at);
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const long long row = wrow + (long long)i * nwarps * RPW + lane / LPR;
      const bool on = row < rows;
      const float x[4] = {x4[i].x, x4[i].y, x4[i].z, x4[i].w};
      float z[4], d[4], dn[4];
      unpack<Tg>(z4[i], z);
      unpack<Tg>(g4[i], d);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = rsqrtf(ss * (1.f / D) + eps);
      float dz[4], u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ex = __expf(-fabsf(z[e])), p = __fdividef(1.f, 1.f + ex);
        const float s = z[e] >= 0.f ? p : ex * p;
        u[e] = x[e] * r;
        const float ds = d[e] * s;
        dn[e] = ds * w[e];
        dot = fmaf(dn[e], u[e], dot);
        dz[e] = d[e] * u[e] * w[e] * (ex * p * p);
        if (on) dw[e] = fmaf(ds, u[e], dw[e]);
      }
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      dot *= 1.f / D;
      if (on) {
        const size_t at = (size_t)row * D + d0;
        __stcs(reinterpret_cast<float4 *>(d_o + at),
               make_float4(r * (dn[0] - u[0] * dot), r * (dn[1] - u[1] * dot),
                           r * (dn[2] - u[2] * dot), r * (dn[3] - u[3] * dot)));
        *reinterpret_cast<Quad<Tg> *>(d_gate + at) = pack<Tg>(dz);
      }
    }
  }
  next_kernel_may_start();
  if (partial == nullptr) return;
  // The warp's rows share channels: lanes LPR apart; then the warps, in order.
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int off = 16; off >= LPR; off >>= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], off);
  if (lane < LPR)
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][d0 + e] = dw[e];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += sums[i][c];
    partial[(size_t)blockIdx.x * D + c] = t;
  }
}

// d_weight[c] = sum of the CTAs' rows: eight channels per CTA, 32 slices of the rows each summed
// in order, then the slices in order (fp64: a few hundred values per channel).
template <int D>
__global__ void __launch_bounds__(256)
epilogue_bwd_weight_kernel(const float *__restrict__ partial, int n, float *__restrict__ d_weight) {
  wait_for_previous_kernel();
  __shared__ double part[32][8];
  const int c = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const float *p = partial + 8 * blockIdx.x + c;
  double t = 0.0;
#pragma unroll 4
  for (int i = slice; i < n; i += 32) t += (double)__ldg(p + (size_t)i * D);
  part[slice][c] = t;
  __syncthreads();
  if (slice == 0) {
    for (int i = 1; i < 32; ++i) t += part[i][c];
    d_weight[8 * blockIdx.x + c] = (float)t;
  }
}

int ctas_of(long long rows, int D) {
  const long long per_cta = (long long)kWarps * (128 / D) * kRowsInFlight;
  // A few trips of one CTA take less than the second kernel's launch.
  if (rows <= 4 * per_cta) return rows > 0 ? 1 : 0;
  const long long want = (rows + per_cta - 1) / per_cta;
  return (int)(want < kMaxCtas ? want : kMaxCtas);
}

template <typename Tg, int D>
cudaError_t launch_typed(const float *o, const void *gate, const float *weight, float eps,
                         const void *d_out, long long rows, float *d_o, void *d_gate,
                         float *d_weight, float *ws, cudaStream_t s) {
  const int ctas = ctas_of(rows, D);
  // One CTA's row is the sum itself; no rows give a sum of none.
  float *partial = d_weight == nullptr ? nullptr : (ctas == 1 ? d_weight : ws);
  if (ctas > 0)
    epilogue_bwd_kernel<Tg, D><<<ctas, kThreads, 0, s>>>(
        o, static_cast<const Tg *>(gate), weight, eps, static_cast<const Tg *>(d_out), rows, d_o,
        static_cast<Tg *>(d_gate), partial);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || d_weight == nullptr || ctas == 1) return e;
  return launch_behind(epilogue_bwd_weight_kernel<D>, dim3(D / 8), 256, 0, s, (const float *)ws, ctas,
                       d_weight);
}

template <typename Tg>
cudaError_t launch_d(int D, const float *o, const void *gate, const float *weight, float eps,
                     const void *d_out, long long rows, float *d_o, void *d_gate, float *d_weight,
                     float *ws, cudaStream_t s) {
  switch (D) {
    case 16: return launch_typed<Tg, 16>(o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, ws, s);
    case 32: return launch_typed<Tg, 32>(o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, ws, s);
    case 64: return launch_typed<Tg, 64>(o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, ws, s);
    case 128: return launch_typed<Tg, 128>(o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, ws, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

size_t epilogue_bwd_workspace_bytes(long long rows, int D) {
  const int ctas = ctas_of(rows, D);
  return ctas > 1 ? (size_t)ctas * D * sizeof(float) : 0;
}

cudaError_t launch_epilogue_bwd(const float *o, const void *gate, const float *weight, float eps,
                                const void *d_out, long long rows, int D, kda_dtype dt, float *d_o,
                                void *d_gate, float *d_weight, void *ws, cudaStream_t s) {
  float *w = static_cast<float *>(ws);
  if (dt == KDA_BF16)
    return launch_d<__nv_bfloat16>(D, o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, w, s);
  if (dt == KDA_F16)
    return launch_d<__half>(D, o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, w, s);
  return launch_d<float>(D, o, gate, weight, eps, d_out, rows, d_o, d_gate, d_weight, w, s);
}

}  // namespace kda
