// State pass of the chunked gated delta rule (kda_gdr.cuh) for D = 128 on tcgen05: one CTA per
// (sequence, value head) carries the head's S^T, 128 value channels as the 128 TMEM lanes.
//
// As in the mma.sync form (kda_gdr_state.cu) everything is computed transposed, and a product's
// result becomes the next product's A operand: here it is read from TMEM, split in two fp16 terms
// and written back to TMEM, where tcgen05.mma takes A from; the B operands are the records' tiles
// in shared memory as they stand ([K; Q] along its rows for K S and Q S in one product of 128
// columns, K across, as an MN-major operand, for the state update, T and P along their rows).
//
// Roles (twelve warps, 168 registers a thread):
//   warps 0-7   the chain: R = beta (V - G K S) -> TMEM; W = E U -> TMEM; S = G_C S + W K, kept in
//               fp32 registers, and its split -> TMEM for the next chunk.  Two threads share a
//               value channel (half the tokens, half the key channels each) and exchange the
//               largest value for the row's scale; a thread of warp 0 issues the chain's MMAs
//   warps 8-11  the read-out, off the chain: Q S into registers, U -> TMEM for P U, then
//               O = scale (G Q S + P U); a thread of warp 8 issues P U and the copies of the
//               records and of V
// Hand-over is by mbarriers in both directions (no block barrier inside the loop); every wait is
// bounded, and a wait that ran out ends the loop of the warp that saw it, after which the others'
// waits run out too.  A wait names a parity, so no barrier may complete its next phase before every
// warp that waits for this one has seen it: a stage's two barriers hold one another (what is loaded
// next waits for `empty`), s_ready is waited for by the read-out only where q_read holds the chain
// until then, and the chain's first warp sees u_ready of the last chunk before it arrives at r_ready.
//
// Triangular T and P: the k-step of tokens 16 k .. only reaches token columns from 16 k on, so its
// MMA is 64 - 16 k columns wide.
//
// Bound: the latency of a chunk's chain (three MMA groups, each followed by a TMEM read, a split
// and a TMEM write), 5.3 us with the read-out, of which the MMAs are about 2; one CTA per SM (all 512
// TMEM columns).  Ten prompts, 59566 tokens, 32 heads: 1.39 ms, the chain of the longest (256 chunks);
// the chunks of all would take 1.0 ms on 148 SMs.  Four warps instead of eight on the chain: 514 us
// where eight take 342.
#include <type_traits>

#include "kda_gdr.cuh"
#include "kda_tcgen05.cuh"

namespace kda {
namespace {
using namespace gdr;

constexpr int D = 128;
constexpr int kChainWarps = 8, kOutWarps = 4;
constexpr int kThreads = 32 * (kChainWarps + kOutWarps);

// TMEM columns.
constexpr uint32_t TM_ACC = 0;    // (K S)^T, then (Q S)^T (64 fp32 each); then W K (128)
constexpr uint32_t TM_U = 128;    // U^T
constexpr uint32_t TM_PU = 192;   // (P U)^T
constexpr uint32_t TM_UP = 256;   // U hi, lo (32 columns each: 64 fp16)
constexpr uint32_t TM_S = 320;    // S^T hi, lo (64 columns each)
constexpr uint32_t TM_W = 448;    // R hi, lo (32 columns each); then W hi, lo

// Shared memory of a stage (1024-byte aligned tiles).
constexpr uint32_t kStKq = 0, kStScales = kq_tile_bytes(D);
constexpr uint32_t kStTp = 33792;
constexpr uint32_t kStV = kStTp + 34816;
constexpr uint32_t kStage = kStV + C * D * 2;
static_assert(kq_bytes(D) <= kStTp && kTpBytes <= 34816 && kStage % 1024 == 0, "stage plan");

struct Small {
  uint64_t full[2], empty[2], s_ready, r_ready, w_ready, q_read, u_ready, out_done, d_s, d_u, d_acc, d_pu;
  uint64_t met[4][3];                 // per 32 value channels: the two warps' largest S, R, W
  uint32_t tmem;
  int dead;
  float most[4][3][2][32];
  float s_scale[2][128], r_scale[2][128];
};
constexpr uint32_t kSmem = 2 * kStage + sizeof(Small) + 1024;

__device__ __forceinline__ void arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// One arrival per warp, after its lanes' TMEM accesses.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  tc::tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// D (+)= A B for one k-step of 16: A fp16 in TMEM (two per column), B in shared memory.  The whole
// warp comes here and one lane issues, so that the operands stay in uniform registers.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          tc::smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}

// Two fp16 terms of 32 values of a row, to TMEM columns hi and lo.
__device__ __forceinline__ void store_split(const float *x, float inv, uint32_t hi, uint32_t lo) {
  uint32_t h[16], l[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) split2(x[2 * i], x[2 * i + 1], inv, h[i], l[i]);
  tmem_st16(hi, h);
  tmem_st16(lo, l);
}
__device__ __forceinline__ float max_abs32(const float *x, float m) {
  float a = m, b = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    a = fmaxf(a, fabsf(x[i]));
    b = fmaxf(b, fabsf(x[i + 1]));
  }
  return fmaxf(a, b);
}

// A bounded wait of a whole warp; a wait that ran out is recorded and seen by every role.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Small &sm, int *status) {
  if (__all_sync(0xffffffffu, tc::mbar_wait(bar, parity))) {
    tc::tc_fence_after();
    return true;
  }
  report(status, KDA_ERR_DEVICE_TIMEOUT);
  *static_cast<volatile int *>(&sm.dead) = 1;
  return false;
}

bool make_v_map(CUtensorMap *m, const void *v, kda_dtype dt, int HV, int T) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)HV * D, (cuuint64_t)T};
  cuuint64_t strides[1] = {(cuuint64_t)HV * D * 2};
  cuuint32_t box[2] = {D, C};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, dt == KDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             2, const_cast<void *>(v), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Tin, int kRole>
__global__ void __launch_bounds__(kThreads, 1)
gdr_state_tc_kernel(const __grid_constant__ CUtensorMap tm_v, const float *s0,
                    const int32_t *__restrict__ cu, float scale, int N, int T, int HK, int HV,
                    uint8_t *__restrict__ ws, Layout lay, float *__restrict__ o, float *sN,
                    int *status) {
  extern __shared__ uint8_t smem_raw[];
  wait_for_previous_kernel();
  if (kRole == kKeep) next_kernel_may_start();  // the reverse pass only needs what is there by now
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  Small &sm = *reinterpret_cast<Small *>(smem + 2 * kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Part pt;
  if (!part_of<kRole, true>(blockIdx.x, cu, N, T, HV, lay, status, pt)) return;
  const int h = pt.h, hk = h / (HV / HK);
  const int bos = pt.bos + pt.first * C, eos = pt.eos, chunks = pt.end - pt.first;  // of this part
  const long long slot0 = pt.slot;
  const size_t nh = (size_t)pt.n * HV + h;
  const bool identity = kRole == kMap && pt.kind == 1;  // M: from the identity, without values

  if (chunks == 0) {  // the state comes back as it was
    if (sN)
      for (int i = tid; i < D * D / 4; i += kThreads)
        reinterpret_cast<float4 *>(sN + nh * D * D)[i] =
            s0 ? reinterpret_cast<const float4 *>(s0 + nh * D * D)[i]
               : make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  if (warp == 0) {
    tc::tmem_alloc(&sm.tmem, 512);
    if (lane == 0) {
      tc::mbar_init(&sm.full[0], 1);
      tc::mbar_init(&sm.full[1], 1);
      tc::mbar_init(&sm.empty[0], kChainWarps);
      tc::mbar_init(&sm.empty[1], kChainWarps);
      tc::mbar_init(&sm.s_ready, kChainWarps);
      tc::mbar_init(&sm.r_ready, kChainWarps);
      tc::mbar_init(&sm.w_ready, kChainWarps);
      tc::mbar_init(&sm.q_read, kOutWarps);
      tc::mbar_init(&sm.u_ready, kOutWarps);
      tc::mbar_init(&sm.out_done, kOutWarps);
      tc::mbar_init(&sm.d_s, 1);
      tc::mbar_init(&sm.d_u, 1);
      tc::mbar_init(&sm.d_acc, 1);
      tc::mbar_init(&sm.d_pu, 1);
      for (int i = 0; i < 12; ++i) tc::mbar_init(&sm.met[0][0] + i, 2);
      tc::fence_mbar_init();
      sm.dead = 0;
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = sm.tmem;
  const uint32_t sbase = tc::smem_u32(smem);
  const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);  // this warp's TMEM lanes
  const int row = 32 * (warp & 3) + lane;                        // and this thread's value channel
  bool ok = true;
  const uint32_t leader = elect_one();

  // A 64-column operand (two terms) times a lower triangular tile (two terms): k-step ks from
  // column 16 ks on, where the tile's rows 16 ks .. are (16 rows of 128 bytes on).
  // A descriptor's address field counts 16 bytes, so a tile's further k-steps are additions.
  auto mma_triangular = [&](uint32_t d, uint32_t a, uint64_t hi) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const uint32_t id = tc::idesc_fp16(128, 64 - 16 * ks, false, false);
      const uint64_t bh = hi + ks * ((2048 + 32) >> 4), bl = bh + (kTriBytes >> 4);
      mma_ts(leader, d + 16 * ks, a + 8 * ks, bh, id, ks > 0);
      mma_ts(leader, d + 16 * ks, a + 32 + 8 * ks, bh, id, 1);
      mma_ts(leader, d + 16 * ks, a + 8 * ks, bl, id, 1);
    }
  };

  if (warp < kChainWarps) {
    const int half = warp >> 2;
    // The larger of the two threads' values of a row (which: 0 S, 1 R, 2 W; one phase per chunk).
    auto meet = [&](int which, float x, uint32_t parity) {
      uint64_t *bar = &sm.met[warp & 3][which];
      float(*most)[32] = sm.most[warp & 3][which];
      most[half][lane] = x;
      __syncwarp();
      if (lane == 0) arrive(bar);
      ok = wait(bar, parity, sm, status);
      return fmaxf(x, most[half ^ 1][lane]);
    };
    float s[D / 2];  // key channels 64 half ..
    const size_t at = (size_t)row * D + half * 64;
    auto store = [&](float *to) {
      float4 *p = reinterpret_cast<float4 *>(to + at);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        p[i] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    };
    const float *from = first_state<kRole>(pt, s0, ws, lay, HV, D);
    if (from && !identity) {
      const float4 *p = reinterpret_cast<const float4 *>(from + at);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float4 x = p[i];
        s[4 * i] = x.x; s[4 * i + 1] = x.y; s[4 * i + 2] = x.z; s[4 * i + 3] = x.w;
      }
      if (kRole == kMap) store(reinterpret_cast<float *>(ws + lay.seg_e) + pt.seg * D * D);
    } else {
#pragma unroll
      for (int i = 0; i < D / 2; ++i) s[i] = identity && row == 64 * half + i ? 1.f : 0.f;
    }
    for (int c = 0; c < chunks; ++c) {
      const uint32_t par = c & 1;
      uint8_t *st = smem + par * kStage;
      const uint32_t st32 = sbase + par * kStage;
      const float *vec = reinterpret_cast<const float *>(st + kStTp + kVec);
      const Tin *vt = reinterpret_cast<const Tin *>(st + kStV) + (32 * half) * D + row;
      const int len = min(C, eos - bos - c * C) - 32 * half;  // tokens of this half
      // S's operand for this chunk.
      const float sbig = meet(0, max_abs32(s + 32, max_abs32(s, 0.f)), par);
      if (!ok) break;
      const Scale ss = scale_of(sbig);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        store_split(s + 32 * i, ss.inv, tl + TM_S + 32 * half + 16 * i, tl + TM_S + 64 + 32 * half + 16 * i);
      if (half == 0) sm.s_scale[par][row] = ss.s;
      tmem_wait_st();
      warp_arrive(&sm.s_ready);
      if constexpr (kRole == kKeep) {
        float *p = reinterpret_cast<float *>(ws + lay.state) +
                   (((size_t)(slot0 + c) * HV + h) * D + half * 64) * D + row;
#pragma unroll
        for (int i = 0; i < D / 2; ++i) __stcs(p + i * D, s[i]);
      }
      if (!(ok = wait(&sm.full[par], (c >> 1) & 1, sm, status))) break;
      if (warp == 0) {
        if (!(ok = wait(&sm.s_ready, par, sm, status))) break;
        constexpr uint32_t id = tc::idesc_fp16(128, kRole == kOut ? 128 : 64, false, false);
        const uint64_t b0 = tc::sdesc(st32 + kStKq, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t b = b0 + (((ks >> 2) * kKq * 128 + (ks & 3) * 32) >> 4);
          mma_ts(leader, tm + TM_ACC, tm + TM_S + 8 * ks, b, id, ks > 0);
          mma_ts(leader, tm + TM_ACC, tm + TM_S + 64 + 8 * ks, b, id, 1);
        }
        commit(leader, &sm.d_s);
      }
      const float ks = *reinterpret_cast<const float *>(st + kStScales);
      const float gl = vec[kVecG * C + C - 1];
      if (len < 32 && !identity) {  // other sequences' rows: this thread alone reads this column
        for (int t = max(len, 0); t < 32; ++t) const_cast<Tin *>(vt)[t * D] = from_f32<Tin>(0.f);
      }
      float x[32];
      {
        const float f = -ss.s * ks;
        float bb[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) bb[i] = identity ? 0.f : to_f32(vt[i * D]);  // on their way while the MMAs run
        if (!(ok = wait(&sm.d_s, par, sm, status))) break;
        tc::tmem_ld32(tl + TM_ACC + 32 * half, x);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 g = *reinterpret_cast<const float4 *>(vec + kVecG * C + 32 * half + i);
          const float4 bt = *reinterpret_cast<const float4 *>(vec + kVecBeta * C + 32 * half + i);
          x[i] = bt.x * fmaf(g.x * f, x[i], bb[i]);
          x[i + 1] = bt.y * fmaf(g.y * f, x[i + 1], bb[i + 1]);
          x[i + 2] = bt.z * fmaf(g.z * f, x[i + 2], bb[i + 2]);
          x[i + 3] = bt.w * fmaf(g.w * f, x[i + 3], bb[i + 3]);
        }
      }
      const float rbig = meet(1, max_abs32(x, 0.f), par);
      if (!ok) break;
      const Scale rs = scale_of(rbig);
      store_split(x, rs.inv, tl + TM_W + 16 * half, tl + TM_W + 32 + 16 * half);
      if (half == 0) sm.r_scale[par][row] = rs.s;
      tmem_wait_st();
      // The last chunk's U has been read; and no warp of the read-out is left behind that chunk's r_ready.
      if (warp == 0 && kRole != kMap && c > 0 && !(ok = wait(&sm.u_ready, par ^ 1, sm, status))) break;
      warp_arrive(&sm.r_ready);
      if (warp == 0) {
        if (!(ok = wait(&sm.r_ready, par, sm, status))) break;
        mma_triangular(tm + TM_U, tm + TM_W, tc::sdesc(st32 + kStTp + kT_HI, 16, 1024));
        commit(leader, &sm.d_u);
      }
      if (!(ok = wait(&sm.d_u, par, sm, status))) break;
      tc::tmem_ld32(tl + TM_U + 32 * half, x);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 e = *reinterpret_cast<const float4 *>(vec + kVecE * C + 32 * half + i);
        const float4 tt = *reinterpret_cast<const float4 *>(vec + kVecT * C + 32 * half + i);
        x[i] *= (rs.s * tt.x) * e.x;
        x[i + 1] *= (rs.s * tt.y) * e.y;
        x[i + 2] *= (rs.s * tt.z) * e.z;
        x[i + 3] *= (rs.s * tt.w) * e.w;
      }
      const float wbig = meet(2, max_abs32(x, 0.f), par);
      if (!ok) break;
      const Scale wsc = scale_of(wbig);
      store_split(x, wsc.inv, tl + TM_W + 16 * half, tl + TM_W + 32 + 16 * half);
      tmem_wait_st();
      warp_arrive(&sm.w_ready);
      if (warp == 0) {
        if (!(ok = wait(&sm.w_ready, par, sm, status))) break;
        // the accumulator lies over Q S
        if (kRole == kOut && !(ok = wait(&sm.q_read, par, sm, status))) break;
        constexpr uint32_t id = tc::idesc_fp16(128, 128, false, true);
        const uint64_t b0 = tc::sdesc(st32 + kStKq, kKq * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t b = b0 + ((kk * 2048) >> 4);
          mma_ts(leader, tm + TM_ACC, tm + TM_W + 8 * kk, b, id, kk > 0);
          mma_ts(leader, tm + TM_ACC, tm + TM_W + 32 + 8 * kk, b, id, 1);
        }
        commit(leader, &sm.d_acc);
      }
      if (!(ok = wait(&sm.d_acc, par, sm, status))) break;
      warp_arrive(&sm.empty[par]);
      const float f = wsc.s * ks;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        tc::tmem_ld32(tl + TM_ACC + 64 * half + 32 * b, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[32 * b + i] = fmaf(gl, s[32 * b + i], f * x[i]);
      }
    }
    if (kRole == kOut && ok && pt.is_last && sN) store(sN + nh * D * D);
    if (kRole == kMap && ok && !identity) store(reinterpret_cast<float *>(ws + lay.seg_b) + pt.seg * D * D);
    if (identity && ok) {
      const float big = meet(0, max_abs32(s + 32, max_abs32(s, 0.f)), chunks & 1);
      const Scale sc = scale_of(big);
      uint8_t *m = ws + lay.seg_m + pt.seg * map_bytes(D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 hi, lo;
        split2(s[8 * i], s[8 * i + 1], sc.inv, hi.x, lo.x);
        split2(s[8 * i + 2], s[8 * i + 3], sc.inv, hi.y, lo.y);
        split2(s[8 * i + 4], s[8 * i + 5], sc.inv, hi.z, lo.z);
        split2(s[8 * i + 6], s[8 * i + 7], sc.inv, hi.w, lo.w);
        uint8_t *to = m + row_off<D>(row, 8 * half + i);
        *reinterpret_cast<uint4 *>(to) = hi;
        *reinterpret_cast<uint4 *>(to + 2 * D) = lo;
      }
      if (half == 0) reinterpret_cast<float *>(m + D * D * 4)[row] = sc.s;
    }
  } else {
    auto load = [&](int c) {
      uint8_t *st = smem + (c & 1) * kStage;
      const long long slot = slot0 + c;
      uint64_t *bar = &sm.full[c & 1];
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bar, kq_bytes(D) + kTpBytes + (identity ? 0 : C * D * 2));
        tc::bulk_load(st, ws + lay.kq + (size_t)(slot * HK + hk) * kq_bytes(D), kq_bytes(D), bar);
        tc::bulk_load(st + kStTp, ws + lay.tp + (size_t)(slot * HV + h) * kTpBytes, kTpBytes, bar);
        if (!identity) tc::tma_load_2d(st + kStV, &tm_v, bar, h * D, bos + c * C);
      }
    };
    if (warp == kChainWarps) {
      load(0);
      if (chunks > 1) load(1);
    }
    for (int c = 0; c < chunks; ++c) {
      const uint32_t par = c & 1;
      const uint8_t *st = smem + par * kStage;
      const float *vec = reinterpret_cast<const float *>(st + kStTp + kVec);
      const int t0 = bos + c * C, len = min(C, eos - t0);
      if constexpr (kRole == kMap) {  // nothing to read out: a stage is free when the chain has left it
        if (warp > kChainWarps) break;
        if (c > 0 && c + 1 < chunks) {
          if (!(ok = wait(&sm.empty[par ^ 1], ((c - 1) >> 1) & 1, sm, status))) break;
          load(c + 1);
        }
        continue;
      }
      if (!(ok = wait(&sm.full[par], (c >> 1) & 1, sm, status))) break;
      if (kRole == kOut && !(ok = wait(&sm.s_ready, par, sm, status))) break;
      // Chunk c - 1's read-out is done, and the chain has left its stage.
      if (warp == kChainWarps && c > 0) {
        if (!(ok = wait(&sm.out_done, par ^ 1, sm, status))) break;
        if (c + 1 < chunks) {
          if (!(ok = wait(&sm.empty[par ^ 1], ((c - 1) >> 1) & 1, sm, status))) break;
          load(c + 1);
        }
      }
      float q[kRole == kOut ? C : 1];
      if constexpr (kRole == kOut) {
        const float qf = sm.s_scale[par][row] * *reinterpret_cast<const float *>(st + kStScales + 4);
        if (!(ok = wait(&sm.d_s, par, sm, status))) break;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x[32];
          tc::tmem_ld32(tl + TM_ACC + 64 + 32 * b, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) q[32 * b + i] = qf * x[i];
        }
        warp_arrive(&sm.q_read);
      }
      if (!(ok = wait(&sm.r_ready, par, sm, status))) break;
      const float rf = sm.r_scale[par][row];
      if (!(ok = wait(&sm.d_u, par, sm, status))) break;
      // U, twice read: once for its scale.
      auto load_u = [&](int b, float (&x)[32]) {
        tc::tmem_ld32(tl + TM_U + 32 * b, x);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 tt = *reinterpret_cast<const float4 *>(vec + kVecT * C + 32 * b + i);
          x[i] *= rf * tt.x;
          x[i + 1] *= rf * tt.y;
          x[i + 2] *= rf * tt.z;
          x[i + 3] *= rf * tt.w;
        }
      };
      if constexpr (kRole == kKeep) {
        float *p = reinterpret_cast<float *>(ws + lay.u) + ((size_t)(slot0 + c) * HV + h) * C * D + row;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x[32];
          load_u(b, x);
          if (b == 1) warp_arrive(&sm.u_ready);
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcs(p + (32 * b + i) * D, x[i]);
        }
      } else {
        float x[32];
        load_u(0, x);
        float big = max_abs32(x, 0.f);
        load_u(1, x);
        big = max_abs32(x, big);
        const Scale us = scale_of(big);
        store_split(x, us.inv, tl + TM_UP + 16, tl + TM_UP + 48);
        load_u(0, x);
        store_split(x, us.inv, tl + TM_UP, tl + TM_UP + 32);
        tmem_wait_st();
        warp_arrive(&sm.u_ready);
        if (warp == kChainWarps) {
          if (!(ok = wait(&sm.u_ready, par, sm, status))) break;
          mma_triangular(tm + TM_PU, tm + TM_UP, tc::sdesc(sbase + par * kStage + kStTp + kP_HI, 16, 1024));
          commit(leader, &sm.d_pu);
        }
        if (!(ok = wait(&sm.d_pu, par, sm, status))) break;
        float *op = o + ((size_t)t0 * HV + h) * D + row;
        const size_t stride = (size_t)HV * D;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          tc::tmem_ld32(tl + TM_PU + 32 * b, x);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const int t = 32 * b + i;
            const float4 g = *reinterpret_cast<const float4 *>(vec + kVecG * C + t);
            const float4 p = *reinterpret_cast<const float4 *>(vec + kVecP * C + t);
            x[i] = scale * fmaf(g.x, q[t], us.s * p.x * x[i]);
            x[i + 1] = scale * fmaf(g.y, q[t + 1], us.s * p.y * x[i + 1]);
            x[i + 2] = scale * fmaf(g.z, q[t + 2], us.s * p.z * x[i + 2]);
            x[i + 3] = scale * fmaf(g.w, q[t + 3], us.s * p.w * x[i + 3]);
          }
          if (len == C) {
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcs(op + (32 * b + i) * stride, x[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * b + i < len) __stcs(op + (32 * b + i) * stride, x[i]);
          }
        }
      }
      warp_arrive(&sm.out_done);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (sm.dead) {  // let what is in flight land before the CTA's memory goes
    if (tid == 0) {
      tc::drain(&sm.full[0]);
      tc::drain(&sm.full[1]);
      tc::drain(&sm.d_s);
      tc::drain(&sm.d_u);
      tc::drain(&sm.d_acc);
      tc::drain(&sm.d_pu);
    }
    __syncthreads();
  }
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tm, 512);
}

template <typename Tin, int kRole>
cudaError_t launch_typed(const void *v, const float *s0, const int32_t *cu, float scale, int N, int T,
                         int HK, int HV, kda_dtype dt, void *ws, const Layout &lay, float *o, float *sN,
                         int *status, cudaStream_t s) {
  auto kern = gdr_state_tc_kernel<Tin, kRole>;
  const cudaError_t e = allow_smem<(int)kSmem>(kern);
  if (e != cudaSuccess) return e;
  const long long units = lay.seg_chunks ? segment_slots(N, T, lay.seg_chunks) : N;
  const long long ctas = units * HV * (kRole == kMap ? 2 : 1);
  CUtensorMap tm;
  if (ctas >= (1LL << 31) || !make_v_map(&tm, v, dt, HV, T)) return cudaErrorInvalidValue;
  return launch_behind(kern, dim3((unsigned)ctas), kThreads, kSmem, s, tm, s0, cu, scale, N, T, HK, HV,
                       static_cast<uint8_t *>(ws), lay, o, sN, status);
}

template <typename Tin, typename... Args> cudaError_t launch_for(Role role, const Args &...args) {
  return role == kOut    ? launch_typed<Tin, kOut>(args...)
         : role == kKeep ? launch_typed<Tin, kKeep>(args...)
                         : launch_typed<Tin, kMap>(args...);
}

}  // namespace

cudaError_t launch_gdr_state_tc(const void *v, const float *s0, const int32_t *cu, float scale, int N,
                                int T, int HK, int HV, kda_dtype dt, void *ws, const Layout &lay, Role role,
                                float *o, float *sN, int *status, cudaStream_t s) {
  return dt == KDA_BF16
             ? launch_for<__nv_bfloat16>(role, v, s0, cu, scale, N, T, HK, HV, dt, ws, lay, o, sN, status, s)
             : launch_for<__half>(role, v, s0, cu, scale, N, T, HK, HV, dt, ws, lay, o, sN, status, s);
}

}  // namespace kda
