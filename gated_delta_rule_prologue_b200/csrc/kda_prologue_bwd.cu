// Backward of the prologue (kda_prologue.cu).  Per channel and token, with x the sequence's
// inputs behind its three rows of history:
//     c_t = sum_j w_j x_{t-3+j};  y = c s, s = sigmoid(c);  q, k: n = y r, r = (sum y^2 + 1e-6)^-1/2
//     dy   = r (dn - n <n, dn>) for q and k (the head's D channels), dn for v
//     dc_t = dy s (1 + c (1 - s))
//     dx_t = sum_j w_j dc_{t+3-j}   (zero past the sequence's end)
//     dw_j = sum_t dc_t x_{t-3+j}
// and the history's gradient is dx at the three places before the sequence.
//
// One thread owns four channels of one (part, head) segment and walks a tile of consecutive
// tokens of one sequence at a time: three inputs and three dc behind it live in registers, so
// x, dn and dx are touched once.  dx_{t-3} is complete when dc_t is known, so a tile walks three
// tokens past its end (their dc is recomputed by the next tile; nothing is exchanged).  The two
// sums of the norm are xor shuffles over the D/4 lanes of a head, for two tokens at a time.  The
// next kAhead tokens' rows are on their way while the current ones are used.
//
// dw: a thread sums its channels' four taps over the tile in fp32 and writes them to the
// workspace, [tile][channel][tap]; a second kernel adds the tiles in a fixed order (fp64).  The
// tile length depends on the sizes alone and no atomics are used, so repeated calls give the
// same bits.
//
// Bytes: x + dx + dn (6 per channel and token for 16-bit types), plus 3 halo rows per tile served by
// L2.  8192 tokens, 32 heads of 128 in bf16: 158 us with the weights' second kernel, 604 MB, 3.8 TB/s.
// Bound by latency with the four warps per scheduler that 128 registers leave: 54% of the issue slots, 43%
// of DRAM; a warp issues every 6.8 cycles (fixed latencies 1.5, loads 1.0, math pipe 0.9, shuffles 0.8).
// 168 us with looks at the stretch's ends in every step.  The rows fetched to shared memory instead,
// eight or twelve tokens ahead, no register spilled: 164 and 161 us.
#include <type_traits>

#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // tokens whose rows are on their way (a multiple of two)

template <typename T> struct Quad { uint2 u; };
template <> struct Quad<float> { float4 u; };
__device__ __forceinline__ void unpack(const Quad<float> &r, float2 (&f)[2]) {
  f[0] = make_float2(r.u.x, r.u.y);
  f[1] = make_float2(r.u.z, r.u.w);
}
__device__ __forceinline__ void unpack(const Quad<__nv_bfloat16> &r, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(r.u.x << 16), __uint_as_float(r.u.x & 0xffff0000u));
  f[1] = make_float2(__uint_as_float(r.u.y << 16), __uint_as_float(r.u.y & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Quad<__half> &r, float2 (&f)[2]) {
  const __half2 *h = reinterpret_cast<const __half2 *>(&r.u);
  f[0] = __half22float2(h[0]);
  f[1] = __half22float2(h[1]);
}
template <typename T> __device__ __forceinline__ Quad<T> pack(const float2 (&f)[2]) {
  Quad<T> r;
  T *h = reinterpret_cast<T *>(&r.u);
  h[0] = from_f32<T>(f[0].x); h[1] = from_f32<T>(f[0].y);
  h[2] = from_f32<T>(f[1].x); h[3] = from_f32<T>(f[1].y);
  return r;
}
template <typename T> __device__ __forceinline__ Quad<T> zero_quad() {
  Quad<T> r;
  memset(&r, 0, sizeof(r));
  return r;
}
template <typename T> __device__ __forceinline__ Quad<T> load_quad(const T *p) {
  Quad<T> r;
  r.u = __ldg(reinterpret_cast<const decltype(r.u) *>(p));
  return r;
}

// r and m of two tokens (dy = r g + m y) from the lanes' parts of sum y^2 and of <y, g>: the four
// sums over a head's G lanes are folded into one another (each lane ends up with one sum of one
// token), a lane finishes its token's r and m, and the tokens' values are exchanged: nine shuffles
// for G = 32 where four separate reductions take twenty.
template <int G>
__device__ __forceinline__ void norm_pair(const float2 (&ss)[2], const float2 (&dot)[2], bool norm,
                                          float (&r)[2], float (&m)[2]) {
  const int lane = threadIdx.x & 31;
  const bool second = lane & (G / 2), is_dot = lane & (G / 4);
  const float s0 = ss[0].x + ss[0].y, s1 = ss[1].x + ss[1].y;
  const float d0 = dot[0].x + dot[0].y, d1 = dot[1].x + dot[1].y;
  const float s = (second ? s1 : s0) + __shfl_xor_sync(0xffffffffu, second ? s0 : s1, G / 2);
  const float d = (second ? d1 : d0) + __shfl_xor_sync(0xffffffffu, second ? d0 : d1, G / 2);
  float v = (is_dot ? d : s) + __shfl_xor_sync(0xffffffffu, is_dot ? s : d, G / 4);
#pragma unroll
  for (int off = G / 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const float o = __shfl_xor_sync(0xffffffffu, v, G / 4);
  float rr = rsqrtf((is_dot ? o : v) + 1e-6f);
  float mm = -rr * rr * rr * (is_dot ? v : o);
  if (!norm) {
    rr = 1.f;
    mm = 0.f;
  }
  const float ro = __shfl_xor_sync(0xffffffffu, rr, G / 2), mo = __shfl_xor_sync(0xffffffffu, mm, G / 2);
  r[0] = second ? ro : rr;
  r[1] = second ? rr : ro;
  m[0] = second ? mo : mm;
  m[1] = second ? mm : mo;
}

template <typename Tin, typename Tg, int D>
__global__ void __launch_bounds__(kThreads, 2)
prologue_bwd_kernel(const Tin *__restrict__ x, const float *__restrict__ w,
                    const Tin *__restrict__ cache_in, const int32_t *__restrict__ cu, int N, int T,
                    int H, const Tg *__restrict__ dq, const Tg *__restrict__ dk,
                    const Tg *__restrict__ dv, int tile, Tin *__restrict__ dx,
                    Tin *__restrict__ d_cache, float *__restrict__ partial, int *status) {
  constexpr int G = D / 4;  // lanes per head segment
  const int HD = H * D, Cn = 3 * HD;
  const int c0 = (blockIdx.x * kThreads + threadIdx.x) * 4;
  const bool active = c0 < Cn, all_active = __all_sync(0xffffffffu, active);
  const int p = active ? c0 / HD : 0;
  const Tg *dn_base = p == 0 ? dq : (p == 1 ? dk : dv);
  const int cg = active ? c0 % HD : 0;  // the channel within q, k or v
  const bool norm = p < 2;
  const bool norm_warp = __any_sync(0xffffffffu, norm);  // a warp of v's channels has no sums to make

  // The history of a sequence without tokens reaches no output.
  if (blockIdx.y == 0 && d_cache != nullptr && active) {
    for (int n = 0; n < N; ++n) {
      const int a = cu ? cu[n] : 0, b = cu ? cu[n + 1] : T;
      if (a != b) continue;
      for (int r = 0; r < 3; ++r)
        *reinterpret_cast<Quad<Tin> *>(d_cache + ((size_t)n * 3 + r) * Cn + c0) = zero_quad<Tin>();
    }
  }
  const int t0 = blockIdx.y * tile;
  const int t_end = min(t0 + tile, T);
  if (cu != nullptr && (cu[0] != 0 || cu[N] != T)) {
    report(status, KDA_ERR_DEVICE_BOUNDS);
    return;
  }

  float2 wt[4][2], dw[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) dw[j][i] = wt[j][i] = make_float2(0.f, 0.f);
  if (active) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(w + (size_t)(c0 + 2 * i) * 4));
      const float4 b = __ldg(reinterpret_cast<const float4 *>(w + (size_t)(c0 + 2 * i + 1) * 4));
      wt[0][i] = make_float2(a.x, b.x);
      wt[1][i] = make_float2(a.y, b.y);
      wt[2][i] = make_float2(a.z, b.z);
      wt[3][i] = make_float2(a.w, b.w);
    }
  }

  int n = t0 < t_end ? seq_of_token(cu, N, t0) : 0;
  if (!in_range(status, n, N)) return;
  for (int ta = t0; ta < t_end;) {  // the tile's stretch of one sequence after another
    int bos, eos;
    seq_bounds(cu, n, T, status, bos, eos);
    if (ta >= eos) {
      if (++n >= N) break;
      continue;
    }
    const int tb = min(t_end, eos);         // this stretch is [ta, tb)
    const int last = min(tb + 3, eos);      // and the tokens after it whose dc reach it
    float2 xh[3][2], ch[3][2];              // x and dc of the three tokens behind
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int t = ta - 3 + j;
      Quad<Tin> r = zero_quad<Tin>();
      if (active && t >= bos) {
        if (in_range(status, t, T)) r = load_quad(x + (size_t)t * Cn + c0);
      } else if (active && cache_in != nullptr && in_range(status, 3 - (bos - t), 3)) {
        r = load_quad(cache_in + ((size_t)n * 3 + (3 - (bos - t))) * Cn + c0);
      }
      unpack(r, xh[j]);
      ch[j][0] = ch[j][1] = make_float2(0.f, 0.f);
    }
    Quad<Tin> xr[kAhead];
    Quad<Tg> gr[kAhead];
    auto fetch = [&](int t, Quad<Tin> &a, Quad<Tg> &b) {
      const bool ok = active && t < last && in_range(status, t, T);
      a = ok ? load_quad(x + (size_t)t * Cn + c0) : zero_quad<Tin>();
      b = ok ? load_quad(dn_base + (size_t)t * HD + cg) : zero_quad<Tg>();
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(ta + i, xr[i], gr[i]);
    // kAhead tokens; whole: neither they nor the ones fetched for them need a look at the stretch's ends.
    auto group = [&](int tt, auto whole) {
      constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
      for (int i = 0; i < kAhead; i += 2) {
        const int t = tt + i;  // tokens t and t + 1
        float2 xf[2][2], g[2][2], s[2][2], y[2][2], ss[2], dot[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          unpack(xr[i + k], xf[k]);
          unpack(gr[i + k], g[k]);
          if constexpr (kWhole) {
            if (in_range(status, t + k + kAhead, T)) {
              xr[i + k] = load_quad(x + (size_t)(t + k + kAhead) * Cn + c0);
              gr[i + k] = load_quad(dn_base + (size_t)(t + k + kAhead) * HD + cg);
            }
          } else {
            fetch(t + k + kAhead, xr[i + k], gr[i + k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ss[k] = dot[k] = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2 a = __fmul2_rn(wt[0][e], xh[k][e]);
            a = __ffma2_rn(wt[1][e], xh[k + 1][e], a);
            a = __ffma2_rn(wt[2][e], k ? xf[0][e] : xh[2][e], a);
            const float2 c = __ffma2_rn(wt[3][e], xf[k][e], a);
            s[k][e] = __fmul2_rn(c, make_float2(-1.4426950408889634f, -1.4426950408889634f));
            s[k][e].x = ex2_approx(s[k][e].x);
            s[k][e].y = ex2_approx(s[k][e].y);
            s[k][e] = __fadd2_rn(s[k][e], make_float2(1.f, 1.f));
            s[k][e].x = rcp_approx(s[k][e].x);
            s[k][e].y = rcp_approx(s[k][e].y);
            y[k][e] = __fmul2_rn(c, s[k][e]);
            ss[k] = __ffma2_rn(y[k][e], y[k][e], ss[k]);
            dot[k] = __ffma2_rn(y[k][e], g[k][e], dot[k]);
          }
        }
        float r[2] = {1.f, 1.f}, m[2] = {0.f, 0.f};  // dy = r g + m y
        if (norm_warp) norm_pair<G>(ss, dot, norm, r, m);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool in_seq = kWhole || t + k < last, own = kWhole || t + k < tb;
          float2 dc[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2 dy = __fmul2_rn(make_float2(r[k], r[k]), g[k][e]);
            dy = __ffma2_rn(make_float2(m[k], m[k]), y[k][e], dy);
            // s (1 + c (1 - s)) = s + y (1 - s)
            const float2 om = __fadd2_rn(make_float2(1.f, 1.f), make_float2(-s[k][e].x, -s[k][e].y));
            dc[e] = __fmul2_rn(dy, __ffma2_rn(y[k][e], om, s[k][e]));
            if (!in_seq) dc[e] = make_float2(0.f, 0.f);
          }
          if (own) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              dw[0][e] = __ffma2_rn(dc[e], xh[0][e], dw[0][e]);
              dw[1][e] = __ffma2_rn(dc[e], xh[1][e], dw[1][e]);
              dw[2][e] = __ffma2_rn(dc[e], xh[2][e], dw[2][e]);
              dw[3][e] = __ffma2_rn(dc[e], xf[k][e], dw[3][e]);
            }
          }
          const int td = t + k - 3;  // dx_{t-3} is complete
          if (kWhole || (active && td < tb && (td >= ta || (d_cache != nullptr && ta == bos)))) {
            float2 d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              d[e] = __fmul2_rn(wt[3][e], ch[0][e]);
              d[e] = __ffma2_rn(wt[2][e], ch[1][e], d[e]);
              d[e] = __ffma2_rn(wt[1][e], ch[2][e], d[e]);
              d[e] = __ffma2_rn(wt[0][e], dc[e], d[e]);
            }
            Tin *to = kWhole || td >= ta ? dx + (size_t)td * Cn + c0
                               : d_cache + ((size_t)n * 3 + (td - bos + 3)) * Cn + c0;
            *reinterpret_cast<Quad<Tin> *>(to) = pack<Tin>(d);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            xh[0][e] = xh[1][e]; xh[1][e] = xh[2][e]; xh[2][e] = xf[k][e];
            ch[0][e] = ch[1][e]; ch[1][e] = ch[2][e]; ch[2][e] = dc[e];
          }
        }
      }
    };
    for (int tt = ta; tt < tb + 3; tt += kAhead) {
      if (all_active && tt >= ta + 3 && tt + 2 * kAhead <= tb)
        group(tt, std::true_type{});
      else
        group(tt, std::false_type{});
    }
    ta = tb;
  }
  next_kernel_may_start();
  if (partial != nullptr && active) {
    float4 *to = reinterpret_cast<float4 *>(partial) + (size_t)blockIdx.y * Cn + c0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      to[2 * i] = make_float4(dw[0][i].x, dw[1][i].x, dw[2][i].x, dw[3][i].x);
      to[2 * i + 1] = make_float4(dw[0][i].y, dw[1][i].y, dw[2][i].y, dw[3][i].y);
    }
  }
}

// dw[channel] = sum of the tiles' rows: eight slices of the tiles per channel, each in order,
// then the slices in order.
__global__ void __launch_bounds__(256)
prologue_bwd_weight_kernel(const float4 *__restrict__ partial, int tiles, int Cn,
                           float4 *__restrict__ dw) {
  wait_for_previous_kernel();
  __shared__ double4 part[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  double4 t = {0.0, 0.0, 0.0, 0.0};
  if (c < Cn)
    for (int i = slice; i < tiles; i += 8) {
      const float4 v = __ldg(partial + (size_t)i * Cn + c);
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
  part[slice][threadIdx.x & 31] = t;
  __syncthreads();
  if (slice == 0 && c < Cn) {
    for (int i = 1; i < 8; ++i) {
      const double4 v = part[i][threadIdx.x];
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    dw[c] = make_float4((float)t.x, (float)t.y, (float)t.z, (float)t.w);
  }
}

int channel_blocks(int Cn) { return (Cn / 4 + kThreads - 1) / kThreads; }

// Tokens per tile: as many tiles as fill two CTAs per SM once, a multiple of four tokens each, up
// to 512 (then more waves).  A tile costs about 16 tokens beside its own (three halo tokens, filling
// the pipeline, a row of dw written and read), so one wave of long tiles beats several of short
// ones: 8192 tokens x 96 heads of 128 in 344-token tiles take 168 us, in 64-token tiles (5.2 waves)
// 182.
int tile_of(int T, int Cn) {
  const long long blocks = channel_blocks(Cn), slots = 2 * 148;
  const long long wave = blocks < slots ? slots / blocks : 1;
  long long tile = (T + wave - 1) / wave;
  if (tile > 512) {
    const long long waves = (tile + 511) / 512;
    tile = (T + wave * waves - 1) / (wave * waves);
  }
  tile = tile < 4 ? 4 : (tile + 3) / 4 * 4;
  while ((T + tile - 1) / tile > 65535) tile *= 2;  // the grid's second dimension
  return (int)tile;
}

template <typename Tin, typename Tg, int D>
cudaError_t launch_typed(const void *x, const float *w, const void *cache_in, const int32_t *cu,
                         int N, int T, int H, const void *dq, const void *dk, const void *dv,
                         void *dx, float *dw, void *d_cache, void *ws, int *status,
                         cudaStream_t s) {
  const int Cn = 3 * H * D, tile = tile_of(T, Cn), tiles = T > 0 ? (T + tile - 1) / tile : 1;
  // One tile's row is the sum itself.
  float *partial = dw == nullptr ? nullptr : (tiles == 1 ? dw : static_cast<float *>(ws));
  prologue_bwd_kernel<Tin, Tg, D><<<dim3(channel_blocks(Cn), tiles), kThreads, 0, s>>>(
      static_cast<const Tin *>(x), w, static_cast<const Tin *>(cache_in), cu, N, T, H,
      static_cast<const Tg *>(dq), static_cast<const Tg *>(dk), static_cast<const Tg *>(dv), tile,
      static_cast<Tin *>(dx), static_cast<Tin *>(d_cache), partial, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (dw != nullptr && tiles > 1)
    return launch_behind(prologue_bwd_weight_kernel, dim3((Cn + 31) / 32), 256, 0, s,
                         static_cast<const float4 *>(ws), tiles, Cn, reinterpret_cast<float4 *>(dw));
  return cudaGetLastError();
}

template <typename Tin, typename Tg>
cudaError_t launch_d(int D, const void *x, const float *w, const void *ci, const int32_t *cu, int N,
                     int T, int H, const void *dq, const void *dk, const void *dv, void *dx,
                     float *dw, void *dc, void *ws, int *status, cudaStream_t s) {
  switch (D) {
    case 16: return launch_typed<Tin, Tg, 16>(x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
    case 32: return launch_typed<Tin, Tg, 32>(x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
    case 64: return launch_typed<Tin, Tg, 64>(x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
    case 128: return launch_typed<Tin, Tg, 128>(x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
    default: return cudaErrorInvalidValue;
  }
}

template <typename Tin>
cudaError_t launch_grad(kda_dtype gdt, int D, const void *x, const float *w, const void *ci,
                        const int32_t *cu, int N, int T, int H, const void *dq, const void *dk,
                        const void *dv, void *dx, float *dw, void *dc, void *ws, int *status,
                        cudaStream_t s) {
  switch (gdt) {
    case KDA_BF16:
      return launch_d<Tin, __nv_bfloat16>(D, x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
    case KDA_F16:
      return launch_d<Tin, __half>(D, x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
    default:
      return launch_d<Tin, float>(D, x, w, ci, cu, N, T, H, dq, dk, dv, dx, dw, dc, ws, status, s);
  }
}

}  // namespace

size_t prologue_bwd_workspace_bytes(int T, int H, int D) {
  if (T <= 0) return 0;
  const int Cn = 3 * H * D, tile = tile_of(T, Cn), tiles = (T + tile - 1) / tile;
  return tiles > 1 ? (size_t)tiles * Cn * 16 : 0;
}

cudaError_t launch_prologue_bwd(const void *x, const float *w, const void *cache_in,
                                const int32_t *cu, int N, int T, int H, int D, kda_dtype dt,
                                kda_dtype gdt, const void *dq, const void *dk, const void *dv,
                                void *dx, float *dw, void *d_cache, void *ws, int *status,
                                cudaStream_t s) {
  switch (dt) {
    case KDA_BF16:
      return launch_grad<__nv_bfloat16>(gdt, D, x, w, cache_in, cu, N, T, H, dq, dk, dv, dx, dw, d_cache, ws, status, s);
    case KDA_F16:
      return launch_grad<__half>(gdt, D, x, w, cache_in, cu, N, T, H, dq, dk, dv, dx, dw, d_cache, ws, status, s);
    default:
      return launch_grad<float>(gdt, D, x, w, cache_in, cu, N, T, H, dq, dk, dv, dx, dw, d_cache, ws, status, s);
  }
}

}  // namespace kda
