// Chunked gated delta rule with one decay per head and token: shared parts of the prep pass
// (kda_gdr_prep.cu), the state pass (kda_gdr_state.cu) and the backward (kda_gdr_bwd.cu).
//
// Mathematics, per value head with key head h / (HV / HK), chunks of C = 64 tokens, entry state
// S (D x D, key-first), gamma_r the inclusive sum of g inside the chunk, G_r = exp(gamma_r),
// D_ri = exp(gamma_r - gamma_i) for i <= r, E_r = exp(gamma_C - gamma_r):
//     A  = strictly lower (beta_r D_ri k_r.k_i),   T = (I + A)^-1,   P = lower (D_ri q_r.k_i)
//     U  = T (beta (V - G K S)),   O = scale (G Q S + P U),   S' = G_C S + K^T (E U)
// Every decay factor is exp of a difference that is never positive when g is not, so no factor
// leaves the fp32 range, whatever the decay; gamma is summed in fp64, so a token that all but
// erases the state (g down to -256, where exp is 0 in fp32; smaller g counts as -256) leaves the
// differences behind it exact.
//
// Arithmetic.  Products run on the tensor cores with fp32 sums.  The keys and queries are exact
// in fp16 (one power of two per 64-token tile keeps bf16 inputs of any size in range); every
// other operand (state, U, T, P, gradients) is split in two fp16 terms, x 2^-e = hi + lo, with a
// power of two per row that puts the row's largest value in [1, 2): 22 significant bits below that,
// so a product's errors are those of fp32 arithmetic on rows whose values are all as large as their
// largest, and no value of the fp32 range overflows.  A row is a token over the chunk's tokens (T, P, and
// the local pass's W and M); in the state passes a value channel over the key channels or over the
// chunk's 64 tokens; in the local pass a token over the channels (dO, X, U) and a key channel over the
// value channels (S, dS').  A product of a split operand with an exact one takes two MMAs, of two split
// ones three (hi hi, hi lo, lo hi).
//
// Workspace: records of the chunks.  Chunk c of sequence n, whose first token is bos, has slot
// bos / 64 + n + c (strictly increasing from chunk to chunk, so no index pass is needed; T / 64 +
// N + 1 slots).
//   KQ record (slot, key head):   one tile of 128 rows (K's tokens, then Q's) x D fp16: 64-column
//                                 blocks of 128 rows x 128 bytes with the 16-byte pieces
//                                 XOR-swizzled by the row; {2^eK, 2^eQ} as two floats
//   TP record (slot, value head): T hi, T lo, P hi, P lo: 64 x 64 fp16 tiles, same layout, rows
//                                 scaled; then fp32 [64]: G, E, 2^eT, 2^eP, beta
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace gdr {

constexpr int C = 64;

// Tile layout: byte offset of the 16-byte piece c8 (columns 8 c8 ..) of a row of a tile of R rows.
template <int R = C> __host__ __device__ constexpr uint32_t tile_off(int row, int c8) {
  return (uint32_t)((c8 >> 3) * (R * 128) + row * 128 + (((c8 & 7) ^ (row & 7)) << 4));
}

constexpr uint32_t kTriBytes = C * C * 2;  // one 64 x 64 fp16 tile
constexpr uint32_t kT_HI = 0, kT_LO = kTriBytes, kP_HI = 2 * kTriBytes, kP_LO = 3 * kTriBytes;
constexpr uint32_t kVec = 4 * kTriBytes;
enum { kVecG = 0, kVecE = 1, kVecT = 2, kVecP = 3, kVecBeta = 4, kVecs = 5 };
constexpr uint32_t kTpBytes = kVec + kVecs * C * 4;
constexpr int kKq = 2 * C;               // rows of the K and Q tile
constexpr uint32_t kQRows = C * 128;     // byte offset of Q's first row in each column block
__host__ __device__ constexpr uint32_t kq_tile_bytes(int D) { return (uint32_t)kKq * D * 2; }
__host__ __device__ constexpr uint32_t kq_bytes(int D) { return kq_tile_bytes(D) + 128; }

__host__ __device__ inline long long slots(int N, int T) { return (long long)T / C + N + 1; }
__host__ __device__ inline long long first_slot(int bos, int n) { return bos / C + n; }

// Segments of the forward's state pass.  The chunks' effect on the state is affine, S -> M S + B, and
// with few (sequence, head) pairs most SMs would wait for a long sequence's chain of chunks.  Then
// sequences are cut into segments of L chunks: a map pass finds every segment's B (from a zero or the
// initial state) and M (its effect on the identity), a scan composes the segments' first states,
// and the read-out pass runs all segments at once.  Segment g of sequence n has slot
// bos / (64 L) + n + g, as chunks have theirs.
__host__ __device__ inline long long segment_slots(int N, int T, int L) {
  return (long long)T / ((long long)C * L) + N + 1;
}
// Chunks per segment (0: whole sequences), by a model of B200 measurements for sequences of about
// T / N tokens, one CTA per (segment, head) and SM.  Microseconds for D = 128 (64): a chunk 4.9 (3.5)
// of whole sequences, 4.2 (2.2) of a map, 5.3 (3.5) of a segment's read-out, a wave of either 3 more,
// a step of the scan 2 (0.9), the two more launches 13 (4).  Cutting has to save a tenth.  `room`: the
// segments whose maps and states the workspace can hold (segment_slots times heads).
inline int segment_chunks(int N, int T, int HV, int D, long long room) {
  const long long ctas = (long long)N * HV;
  if (N < 1 || T < 1 || ctas > 148) return 0;
  const bool d128 = D == 128;
  const double whole = d128 ? 4.9 : 3.5, map = d128 ? 4.2 : 2.2, read = d128 ? 5.3 : 3.5;
  const double step = d128 ? 2.0 : 0.9, more = d128 ? 13.0 : 4.0;
  const long long n = (((long long)T + N - 1) / N + C - 1) / C;
  double best = 0.9 * whole * (double)n;
  int len = 0;
  for (long long G = 2; G <= n / 2 && G <= 64; ++G) {
    const long long L = (n + G - 1) / G, Gs = (n + L - 1) / L;
    if (Gs < 2 || segment_slots(N, T, (int)L) * HV > room) continue;
    const long long maps = ctas * (2 * Gs - 3), reads = ctas * Gs;
    const double t = (double)((maps + 147) / 148) * (L * map + 3.0) +
                     (double)((reads + 147) / 148) * (L * read + 3.0) + step * (double)(Gs - 2) + more;
    if (t < best) {
      best = t;
      len = (int)L;
    }
  }
  return len;
}
// M of a segment as the scan takes it: D rows of D fp16 hi and D fp16 lo (row_off), then the rows'
// scales.  Row i has M's column i: the effect on the i-th unit vector.
__host__ __device__ constexpr uint32_t map_bytes(int D) { return (uint32_t)D * D * 4 + D * 4; }

// Shared memory of a launch of `ctas` chains of chunks: so much that two never share an SM while there
// are SMs for all.  A chain is bound by its own latency, and two on an SM hold one another up: the CTAs
// of a launch behind a kernel that is still ending are set up wherever there is room first (backward of
// 4 x 2048 tokens, 16 heads: 753 us so, 813 us with the SMs shared).
constexpr int chain_smem(int bytes, long long ctas) {
  constexpr int kMoreThanHalf = 116 * 1024;
  return ctas <= 148 && bytes < kMoreThanHalf ? kMoreThanHalf : bytes;
}

// Byte offsets in the workspace.
struct Layout {
  size_t kq, tp;                 // records
  size_t state, dstate, u, x;    // backward: per chunk fp32 S and dS' (key-major: [key][value channel]),
                                 // U and X [64][D]
  int seg_chunks;                // forward: chunks per segment, or 0
  size_t seg_m, seg_b, seg_e;    // and per segment M (map_bytes), fp32 B and first state, like a state
  size_t bytes;
};
// The layout that a workspace of `given` bytes has: the fastest of those that fit, down to the records
// alone, whose bytes grow with N and T (what the fastest takes does not: few long sequences are cut, many
// are not).  Without `given`, the fastest.  `bytes` says what it takes.
inline Layout layout(int N, int T, int HK, int HV, int D, bool bwd, size_t given = SIZE_MAX) {
  const size_t n = (size_t)slots(N, T);
  Layout l;
  l.kq = 0;
  l.tp = l.kq + n * HK * kq_bytes(D);
  l.state = l.tp + n * HV * kTpBytes;
  const size_t sq = n * HV * (size_t)D * D * 4, rows = n * HV * (size_t)C * D * 4;
  l.dstate = l.state + (bwd ? sq : 0);
  l.u = l.dstate + (bwd ? sq : 0);
  l.x = l.u + (bwd ? rows : 0);
  l.seg_m = l.x + (bwd ? rows : 0);
  const size_t seg1 = (size_t)D * D * 4;
  const size_t room = given > l.seg_m ? (given - l.seg_m) / (map_bytes(D) + 2 * seg1) : 0;
  l.seg_chunks = bwd ? 0 : segment_chunks(N, T, HV, D, (long long)room);
  const size_t segs = l.seg_chunks ? (size_t)segment_slots(N, T, l.seg_chunks) * HV : 0;
  const size_t seg = segs * seg1;
  l.seg_b = l.seg_m + segs * map_bytes(D);
  l.seg_e = l.seg_b + seg;
  l.bytes = l.seg_e + seg;
  return l;
}

// The log-decay as the chunked form takes it (NaN stays NaN).
__device__ __forceinline__ float floor_g(float g) { return g < -256.f ? -256.f : g; }

// gamma of a chunk's tokens in base-2 units (gamma / ln 2), as two floats each (their sum in fp64,
// split), by one warp whose lane holds g of tokens 2 lane and 2 lane + 1 (0 behind the end).
__device__ __forceinline__ void gamma_of(float ga, float gb, float2 *gamma) {
  const int lane = threadIdx.x & 31;
  const double b = gb;
  double s = ga + b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += o;
  }
  constexpr double kLog2e = 1.4426950408889634074;
  const double a = (s - b) * kLog2e;
  s *= kLog2e;
  const float ah = (float)a, sh = (float)s;
  *reinterpret_cast<float4 *>(gamma + 2 * lane) =
      make_float4(ah, (float)(a - ah), sh, (float)(s - sh));
}
// exp(gamma_r - gamma_i): the difference of the two sums is off by 2^-24 of itself, the
// approximate base-2 exponential by a few 2^-23.
__device__ __forceinline__ float decay_between(float2 r, float2 i) {
  return ex2_approx((r.x - i.x) + (r.y - i.y));
}
// g of a token of the chunk at g0 (its head's first value, `stride` apart).
__device__ __forceinline__ float load_g(const float *g0, size_t stride, int t, int len) {
  return t < len ? floor_g(__ldg(g0 + t * stride)) : 0.f;
}

// Sequence of a slot and the slot's place in it, for slots of `span` tokens (a chunk, or a segment).
__device__ __forceinline__ long long place_of_slot(const int32_t *cu, int N, int T, long long slot,
                                                   int span, int *status, int &n, int &bos, int &eos) {
  int lo = 0, hi = N - 1;
  n = 0;
  if (cu) {
    while (lo <= hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] / span + mid <= slot) {
        n = mid;
        lo = mid + 1;
      } else {
        hi = mid - 1;
      }
    }
  }
  seq_bounds(cu, n, T, status, bos, eos);
  return slot - (bos / span + n);
}
// Sequence and chunk of a slot; false for a slot that no chunk has.
__device__ __forceinline__ bool chunk_of_slot(const int32_t *cu, int N, int T, long long slot,
                                              int *status, int &n, int &bos, int &eos, int &c) {
  const long long cc = place_of_slot(cu, N, T, slot, C, status, n, bos, eos);
  if (cc < 0 || cc * C >= eos - bos) return false;
  c = (int)cc;
  return true;
}

// Sequence of a chain by its place in the launch, the longest first (equal lengths by index): for
// launches whose chains do not all run at once, so that no long chain starts when the others end, and
// of up to kRanked sequences.  Ten packed prompts of 512 to 16384 tokens, 32 heads: 2255 -> 2165 us; 0.5 us
// more per CTA.  By all threads of a block; not inlined, for the callers' registers.
constexpr int kRanked = 64;
[[maybe_unused]] static __device__ __noinline__ int sequence_of_place(const int32_t *cu, int N, int T,
                                                                      int place, int *status) {
  __shared__ int length[kRanked], found;
  const int i = threadIdx.x;
  int mine = 0;
  if (i < N) {
    int bos, eos;
    seq_bounds(cu, i, T, status, bos, eos);
    length[i] = mine = eos - bos;
  }
  __syncthreads();
  if (i < N) {
    int before = 0;
    for (int j = 0; j < N; ++j) before += length[j] > mine || (length[j] == mine && j < i);
    if (before == place) found = i;
  }
  __syncthreads();
  return found;
}

// What a launch of the state pass is for.
enum Role {
  kOut,   // the read-out and the last states; of segments from the scan's states, if sequences are cut
  kKeep,  // the backward's forward: S at the start of every chunk and U go to the workspace
  kMap    // a segment's B (kind 0) or M (kind 1); not of a sequence's last segment, nor M of its first
};
// The chunks of a CTA of the state pass: first .. end - 1 of sequence n.
struct Part {
  int n, h, kind, bos, eos, first, end;
  bool is_last;        // the sequence's last chunk is among them
  size_t seg;          // the segment's (slot, head), if sequences are cut
  long long slot;      // of the first chunk
};
// Part b (segments, or whole sequences, times heads; times two for maps); false: nothing to do.
template <int kRole, bool kRanks>
__device__ __forceinline__ bool part_of(int b, const int32_t *cu, int N, int T, int HV, const Layout &lay,
                                        int *status, Part &p) {
  p.kind = kRole == kMap ? b & 1 : 0;
  if (kRole == kMap) b >>= 1;
  p.h = b % HV;
  p.n = b / HV;
  p.first = 0;
  p.seg = 0;
  const int L = kRole == kKeep ? 0 : lay.seg_chunks;
  if (L == 0) {
    if (kRanks && gridDim.x > 148 && cu && N <= kRanked) p.n = sequence_of_place(cu, N, T, p.n, status);
    seq_bounds(cu, p.n, T, status, p.bos, p.eos);
    p.end = (p.eos - p.bos + C - 1) / C;
  } else {
    const long long slot = p.n;
    const long long g = place_of_slot(cu, N, T, slot, C * L, status, p.n, p.bos, p.eos);
    p.end = (p.eos - p.bos + C - 1) / C;
    if (g < 0 || (g > 0 && g * L >= p.end) || !in_range(status, slot, segment_slots(N, T, L))) return false;
    p.first = (int)g * L;
    if (kRole == kMap && (p.first + L >= p.end || (p.kind == 1 && g == 0))) return false;
    p.end = min(p.end, p.first + L);
    p.seg = (size_t)slot * HV + p.h;
  }
  p.is_last = p.end * C >= p.eos - p.bos;
  p.slot = first_slot(p.bos, p.n) + p.first;
  return in_range(status, p.slot + (p.end - p.first), slots(N, T) + 1);
}
// Where a part's first state comes from (null: zero; a map of kind 1 starts from the identity).  The
// read-out of a cut sequence starts from the workspace alone, its first segment too: the last
// segment may be writing sN, which may be s0, by then.
template <int kRole>
__device__ __forceinline__ const float *first_state(const Part &p, const float *s0, const uint8_t *ws,
                                                    const Layout &lay, int HV, int D) {
  if (kRole == kOut && (p.first > 0 || (s0 && !p.is_last)))
    return reinterpret_cast<const float *>(ws + lay.seg_e) + p.seg * D * D;
  return s0 && p.first == 0 ? s0 + ((size_t)p.n * HV + p.h) * D * D : nullptr;
}

// ---------------------------------------------------------------------------
// Warp-level pieces
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes global -> shared, zeros when !ok (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok = true) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// `bytes` (a multiple of 16) by all threads of the block.
__device__ __forceinline__ void cp_block(uint32_t dst, const uint8_t *src, uint32_t bytes) {
  for (uint32_t i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16) cp16(dst + i, src + i);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// c += a b: a 16 x 16 (rows lane/4, +8), b 16 x 8, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = a b, without the eight moves that clear c.
__device__ __forceinline__ void mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Four 8 x 8 blocks of accumulator layout, written transposed (a lane gives a row's address).
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
// Two 8-column blocks (n0 .. n0 + 15) of a B operand for the 16 k-values from k0 on.
// Rows of the tile are B's columns (n), 16-byte pieces its k: r = {b0, b1, b0', b1'}.
template <int R = C>
__device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t tile, int n0, int k0) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4(r, tile + tile_off<R>(n0 + (m >> 1) * 8 + (lane & 7), (k0 >> 3) + (m & 1)));
}
// Rows of the tile are B's k.
template <int R = C>
__device__ __forceinline__ void load_bt(uint32_t (&r)[4], uint32_t tile, int n0, int k0) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4t(r, tile + tile_off<R>(k0 + (m & 1) * 8 + (lane & 7), (n0 >> 3) + (m >> 1)));
}
// A operand (16 rows from m0, 16 k from k0): rows of the tile are A's rows.
template <int R = C>
__device__ __forceinline__ void load_a(uint32_t (&r)[4], uint32_t tile, int m0, int k0) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4(r, tile + tile_off<R>(m0 + (m & 1) * 8 + (lane & 7), (k0 >> 3) + (m >> 1)));
}
// Rows of the tile are A's k (the transposed tile is the operand).
__device__ __forceinline__ void load_at(uint32_t (&r)[4], uint32_t tile, int m0, int k0) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4t(r, tile + tile_off(k0 + (m >> 1) * 8 + (lane & 7), (m0 >> 3) + (m & 1)));
}

// Power of two s with x / s in [1, 2) for x = the largest magnitude of a row (any s for 0), and
// its inverse.  Exponents are kept in the range where both are normal numbers.
struct Scale {
  float s, inv;
};
__device__ __forceinline__ Scale scale_of(float largest) {
  int e = (int)(__float_as_uint(largest) >> 23) & 255;
  e = min(max(e, 1), 253);
  return {__uint_as_float((uint32_t)e << 23), __uint_as_float((uint32_t)(254 - e) << 23)};
}
// The largest of the four lanes that share accumulator rows.
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// (x, y) inv = hi + lo, each term rounded to fp16 (nearest): the first keeps 11 bits, the second
// the next 11, so the pair is off by at most 2^-23 of the value (2^-25 absolute near zero).
__device__ __forceinline__ void split2(float x, float y, float inv, uint32_t &hi, uint32_t &lo) {
  const float2 v = __fmul2_rn(make_float2(x, y), make_float2(inv, inv));
  const __half2 h = __floats2half2_rn(v.x, v.y);
  const float2 f = __half22float2(h);
  const float2 r = __fadd2_rn(v, make_float2(-f.x, -f.y));
  const __half2 l = __floats2half2_rn(r.x, r.y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Row scales of an accumulator of NT 8-column blocks (rows lane/4 and lane/4 + 8).
template <int NT> __device__ __forceinline__ void row_scales(const float (&c)[NT][4], Scale &r0, Scale &r1) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    a = fmaxf(a, fmaxf(fabsf(c[i][0]), fabsf(c[i][1])));
    b = fmaxf(b, fmaxf(fabsf(c[i][2]), fabsf(c[i][3])));
  }
  r0 = scale_of(quad_max(a));
  r1 = scale_of(quad_max(b));
}
// The A operand of k-step kk (columns 16 kk ..) from an accumulator, as two fp16 terms.
template <int NT>
__device__ __forceinline__ void split_a(const float (&c)[NT][4], int kk, const Scale &r0, const Scale &r1,
                                        uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(c[2 * kk][0], c[2 * kk][1], r0.inv, hi[0], lo[0]);
  split2(c[2 * kk][2], c[2 * kk][3], r1.inv, hi[1], lo[1]);
  split2(c[2 * kk + 1][0], c[2 * kk + 1][1], r0.inv, hi[2], lo[2]);
  split2(c[2 * kk + 1][2], c[2 * kk + 1][3], r1.inv, hi[3], lo[3]);
}

template <int NT> __device__ __forceinline__ void zero(float (&c)[NT][4]) {
#pragma unroll
  for (int i = 0; i < NT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
}

// A matrix of fp32 rows of D values becomes, in its place, one of split rows: per row D fp16 hi,
// then D fp16 lo (4 D bytes as before), the 16-byte pieces of each XOR-swizzled by the row, so that
// ldmatrix reads eight rows without bank conflicts.
template <int D> __device__ __forceinline__ uint32_t row_off(int row, int c8) {
  return (uint32_t)(row * 4 * D + ((c8 ^ (row & 7)) << 4));
}
// B operand whose columns (n) are rows n0 .. n0 + 15; lo: the second term.
template <int D>
__device__ __forceinline__ void load_rows_b(uint32_t (&r)[4], uint32_t base, int n0, int k0, bool lo) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4(r, base + row_off<D>(n0 + (m >> 1) * 8 + (lane & 7), (k0 >> 3) + (m & 1)) + (lo ? 2 * D : 0));
}
// A operand of rows m0 .. m0 + 15.
template <int D>
__device__ __forceinline__ void load_rows_a(uint32_t (&r)[4], uint32_t base, int m0, int k0, bool lo) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4(r, base + row_off<D>(m0 + (m & 1) * 8 + (lane & 7), (k0 >> 3) + (m >> 1)) + (lo ? 2 * D : 0));
}

// B operand whose k are rows k0 .. k0 + 15.
template <int D>
__device__ __forceinline__ void load_rows_bt(uint32_t (&r)[4], uint32_t base, int n0, int k0, bool lo) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  ldsm4t(r, base + row_off<D>(k0 + (m & 1) * 8 + (lane & 7), (n0 >> 3) + (m >> 1)) + (lo ? 2 * D : 0));
}
}  // namespace gdr

// Host side (kda_gdr_*.cu), called by kda_api.cu with one layout for all of a call; the *_tc form is launch_gdr_state's for D = 128.
cudaError_t launch_gdr_state_tc(const void *v, const float *s0, const int32_t *cu, float scale, int N,
                                int T, int HK, int HV, kda_dtype dt, void *ws, const gdr::Layout &lay,
                                gdr::Role role, float *o, float *sN, int *status, cudaStream_t s);
cudaError_t launch_gdr_prep(const void *q, const void *k, const float *g, const float *beta,
                            const int32_t *cu, int N, int T, int HK, int HV, int D, kda_dtype dt,
                            void *ws, const gdr::Layout &lay, int *status, cudaStream_t s);
cudaError_t launch_gdr_state(const void *v, const float *s0, const int32_t *cu, float scale, int N,
                             int T, int HK, int HV, int D, kda_dtype dt, void *ws,
                             const gdr::Layout &lay, bool bwd, float *o, float *sN, int *status,
                             cudaStream_t s);
cudaError_t launch_gdr_bwd(const void *v, const float *g, const float *beta, const int32_t *cu,
                           float scale, int N, int T, int HK, int HV, int D, kda_dtype dt, void *ws,
                           const gdr::Layout &lay, const float *d_o, const float *d_sN, void *dq, void *dk, void *dv,
                           float *dg, float *dbeta, float *d_s0, int *status, cudaStream_t s);
}  // namespace kda
