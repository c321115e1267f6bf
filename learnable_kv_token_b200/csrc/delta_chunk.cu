// Gated delta rule over prompts, in chunks of 64 tokens on tensor cores
// (formulas and precision: delta_chunk.cuh).  Two launches: everything that
// depends on no state, for all chunks at once, then the chain of states.
#include "delta_chunk.cuh"

namespace lte {
namespace delta {

// ------------------------------------------------------------------- prepare
// One CTA of four warps per (head, chunk).  K K^T and Q K^T by warp MMAs (warp
// w: token rows 16 w .. + 15, only the tiles on and below the diagonal); then
// X = (I + M)^{-1} in fp32: the four 16 x 16 diagonal blocks by forward
// substitution (a thread per column), joined in pairs twice by
//   [A 0; C B]^{-1} = [A' 0; -B' C A' B'].
// Forward substitution keeps X accurate where a series in powers of M would
// not (equal keys make M's powers grow; X itself stays bounded).
constexpr int kPrepThreads = 128;
constexpr int kXs = 68;                                   // row stride of M and X in floats

__device__ __forceinline__ float ex2_approx(float x) {     // relative error about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x = hi + lo in TF32 (11 bits each); the tensor core drops the lower bits of lo
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// c (16 x 8 NT) = sign A (16 x 8 KS) B (8 KS x 8 NT), row stride kXs: three TF32
// products per step keep about 21 bits
template <int NT, int KS>
__device__ __forceinline__ void mma_tf32x3(float (&c)[NT][4], const float* A, const float* B, float sign, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      split_tf32(sign * A[(g + 8 * (e & 1)) * kXs + 8 * k + t + 4 * (e >> 1)], ah[e], al[e]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) split_tf32(B[(8 * k + t + 4 * e) * kXs + 8 * n + g], bh[e], bl[e]);
      mma_tf32(c[n], ah, bh);
      mma_tf32(c[n], ah, bl);
      mma_tf32(c[n], al, bh);
    }
  }
}
__device__ __forceinline__ void store_c(float* p, const float* c, int lane) {
  float* q = p + (lane >> 2) * kXs + (lane & 3) * 2;
  *reinterpret_cast<float2*>(q) = make_float2(c[0], c[1]);
  *reinterpret_cast<float2*>(q + 8 * kXs) = make_float2(c[2], c[3]);
}

template <int DK, bool A_LO>
__global__ void __launch_bounds__(kPrepThreads, 5)
delta_prepare_kernel(const ChunkArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(16) float2 G2[L];                  // log2(e) G as a float pair
  __shared__ __align__(16) float bs[L];
  const int u = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
  const int b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = (lane & 3) * 2;
  const int len = seq_len(a.lens, b, a.T), t0 = c * L;
  if (t0 >= len) return;
  const uint32_t s0 = smem_u32(sm), sK = s0, sQ = s0 + L * DK * 2;
  load_rows<DK, kPrepThreads>(sK, a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, t0, len);
  load_rows<DK, kPrepThreads>(sQ, a.q + b * a.qs.b + hk * a.qs.h, a.qs.t, t0, len);
  cp_async_commit();
  uint8_t* rec = a.rec + (long long)blockIdx.x * rec_bytes(A_LO);
  float* scal = reinterpret_cast<float*>(rec + (A_LO ? 4 : 3) * kImg);
  if (warp == 0) {
    // running sums of the gates in 64 bits: after a gate that forgets
    // everything, differences of later sums keep their digits
    double x0 = 0, x1 = 0;
    float b0 = 0x1p-60f, b1 = 0x1p-60f;
    const long long gi = ((long long)b * a.T + t0 + 2 * lane) * a.H + h;
    if (t0 + 2 * lane < len) {
      const float x = a.g[gi];
      x0 = x < -104.f ? -104.f : x;                       // e^-104 is 0 in fp32
      b0 = live_beta(a.beta[gi]);
    }
    if (t0 + 2 * lane + 1 < len) {
      const float x = a.g[gi + a.H];
      x1 = x < -104.f ? -104.f : x;
      b1 = live_beta(a.beta[gi + a.H]);
    }
    double sum = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const double last = __shfl_sync(0xffffffffu, sum, 31);
    const double G0 = sum - x1, G1 = sum;
    constexpr double kLog2e = 1.4426950408889634;
    const float h0 = (float)(G0 * kLog2e), h1 = (float)(G1 * kLog2e);
    G2[2 * lane] = make_float2(h0, (float)(G0 * kLog2e - h0));
    G2[2 * lane + 1] = make_float2(h1, (float)(G1 * kLog2e - h1));
    bs[2 * lane] = b0;
    bs[2 * lane + 1] = b1;
    float2* out = reinterpret_cast<float2*>(scal) + lane;
    out[kEG * 32] = make_float2(expf((float)G0), expf((float)G1));
    out[kLam * 32] = make_float2(expf((float)(last - G0)), expf((float)(last - G1)));
    out[kBeta * 32] = make_float2(b0, b1);
    out[kGhi * 32] = make_float2((float)G0, (float)G1);
    out[kGlo * 32] = make_float2((float)(G0 - (float)G0), (float)(G1 - (float)G1));
  }
  cp_async_wait<0>();
  __syncthreads();
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t ak[4], aq[4];
    const uint32_t ra = swz<DK>(16 * warp + ldt_row(lane), 2 * ks + ldt_col(lane));
    ldsm_x4(sK + ra, ak[0], ak[1], ak[2], ak[3]);
    ldsm_x4(sQ + ra, aq[0], aq[1], aq[2], aq[3]);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      if (np <= warp) {
        uint32_t x[4];
        ldsm_x4(sK + swz<DK>(16 * np + ldn_row(lane), 2 * ks + ldn_col(lane)), x[0], x[1], x[2], x[3]);
        mma_bf16(kk[2 * np], ak, x[0], x[1]);
        mma_bf16(kk[2 * np + 1], ak, x[2], x[3]);
        mma_bf16(qk[2 * np], aq, x[0], x[1]);
        mma_bf16(qk[2 * np + 1], aq, x[2], x[3]);
      }
    }
  }
  __syncthreads();                                        // K and Q have been read
  float* M = reinterpret_cast<float*>(sm);
  float* X = M + L * kXs;
  uint8_t* img = reinterpret_cast<uint8_t*>(X);           // A's image, before X is formed
  const int ta = 16 * warp + g;
  const float2 Ga = G2[ta], Gb = G2[ta + 8];
  const float ba = bs[ta], bb = bs[ta + 8];
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int s = 8 * n + t2;
    const bool below = n <= 2 * warp + 1;                   // else nothing of this tile is at or below the diagonal
    const float4 Gs = *reinterpret_cast<const float4*>(&G2[s]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = ta + 8 * r;
      const uint32_t off = t * 128 + ((n ^ (t & 7)) << 4) + t2 * 2;
      uint32_t hi = 0, lo = 0;
      if (below) {
        const float2 Gt = r ? Gb : Ga;
        const float bt = r ? bb : ba;
        const float d0 = s <= t ? ex2_approx((Gt.x - Gs.x) + (Gt.y - Gs.y)) : 0.f;
        const float d1 = s + 1 <= t ? ex2_approx((Gt.x - Gs.z) + (Gt.y - Gs.w)) : 0.f;
        *reinterpret_cast<float2*>(&M[t * kXs + s]) =
            make_float2(s < t ? bt * (d0 * kk[n][2 * r]) : 0.f, s + 1 < t ? bt * (d1 * kk[n][2 * r + 1]) : 0.f);
        split2(a.scale * (d0 * qk[n][2 * r]), a.scale * (d1 * qk[n][2 * r + 1]), hi, lo);
      }
      *reinterpret_cast<uint32_t*>(img + off) = hi;
      if (A_LO) *reinterpret_cast<uint32_t*>(img + kImg + off) = lo;
    }
  }
  __syncthreads();
  for (int i = tid; i < (A_LO ? 2 : 1) * kImg / 16; i += kPrepThreads)
    reinterpret_cast<uint4*>(rec + 2 * kImg)[i] = reinterpret_cast<const uint4*>(img)[i];
  __syncthreads();
  // the diagonal blocks: warp d, a lane per column; rows of M by broadcast
  if (lane < 16) {
    const int d = 16 * warp;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; k += 4) {
        const float4 m = *reinterpret_cast<const float4*>(&M[(d + i) * kXs + d + k]);
        s = fmaf(-m.x, x[k], s);
        if (k + 1 < i) s = fmaf(-m.y, x[k + 1], s);
        if (k + 2 < i) s = fmaf(-m.z, x[k + 2], s);
        if (k + 3 < i) s = fmaf(-m.w, x[k + 3], s);
      }
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) X[(d + i) * kXs + d + lane] = x[i];
  }
  __syncthreads();
  // pairs of 16 (warp: pair and half of its columns), then the pair of 32 (warp:
  // half of its rows and of its columns): W = C A' goes to the block above M's
  // diagonal, which is not used otherwise; then -B' W
  {
    const int c0 = 32 * (warp >> 1), r0 = c0 + 16, n0 = 8 * (warp & 1);
    float w[1][4] = {};
    mma_tf32x3<1, 2>(w, &M[r0 * kXs + c0], &X[c0 * kXs + c0 + n0], 1.f, lane);
    store_c(&M[c0 * kXs + r0 + n0], w[0], lane);
    __syncthreads();
    float y[1][4] = {};
    mma_tf32x3<1, 2>(y, &X[r0 * kXs + r0], &M[c0 * kXs + r0 + n0], -1.f, lane);
    store_c(&X[r0 * kXs + c0 + n0], y[0], lane);
    const float zero[4] = {};
    store_c(&X[c0 * kXs + r0 + n0], zero, lane);           // above the diagonal of the pair
  }
  __syncthreads();
  {
    const int m0 = 16 * (warp >> 1), n0 = 16 * (warp & 1);
    float w[2][4] = {};
    mma_tf32x3<2, 4>(w, &M[(32 + m0) * kXs], &X[n0], 1.f, lane);
    store_c(&M[m0 * kXs + 32 + n0], w[0], lane);
    store_c(&M[m0 * kXs + 40 + n0], w[1], lane);
    __syncthreads();
    float y[2][4] = {};
    mma_tf32x3<2, 4>(y, &X[(32 + m0) * kXs + 32], &M[32 + n0], -1.f, lane);
    store_c(&X[(32 + m0) * kXs + n0], y[0], lane);
    store_c(&X[(32 + m0) * kXs + n0 + 8], y[1], lane);
  }
  __syncthreads();
  // T = X diag(b) below the diagonal, as hi and lo (its diagonal is b itself)
  for (int i = tid; i < L * 8; i += kPrepThreads) {
    const int t = i >> 3, cc = i & 7;
    uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
    if (8 * cc < t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = 8 * cc + 4 * e;
        const float4 x = *reinterpret_cast<const float4*>(&X[t * kXs + s]);
        const float4 bb = *reinterpret_cast<const float4*>(&bs[s]);
        split2(s < t ? x.x * bb.x : 0.f, s + 1 < t ? x.y * bb.y : 0.f, hi[2 * e], lo[2 * e]);
        split2(s + 2 < t ? x.z * bb.z : 0.f, s + 3 < t ? x.w * bb.w : 0.f, hi[2 * e + 1], lo[2 * e + 1]);
      }
    }
    const uint32_t off = t * 128 + ((cc ^ (t & 7)) << 4);
    *reinterpret_cast<uint4*>(rec + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(rec + kImg + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// --------------------------------------------------------------------- chain
// W warps per CTA, each with 16 value channels (rows of S) of one head and no
// word exchanged between them: rows of S evolve apart.  All products are kept
// transposed, value channels as the MMA's rows, so that each result is, in the
// registers it is in, the A operand of the next:
//   P^T = S K^T -> R^T = V^T - P^T diag(e^G) -> U^T = R^T T^T
//   -> S = e^{G_L} S + (U diag(e^{G_L - G}))^T K,  O^T = scale (S Q^T) diag(e^G) + U^T A^T
// and the chain of a chunk has no shared-memory round trip and no barrier.
// Shared memory holds the chunk's K, Q, V and record, loaded one chunk ahead by
// cp.async.
template <int DK, int W, bool OUT>
struct ChainSmem {
  static constexpr int kRec = OUT ? 3 * kImg : 2 * kImg;
  static constexpr int kK = 0, kQ = L * DK * 2, kV = kQ + (OUT ? L * DK * 2 : 0), kR = kV + L * 32 * W;
  static constexpr int kS = kR + kRec, kStage = kS + kScal;
  static constexpr int kO = 2 * kStage, kTotal = kO + (OUT ? W * L * 32 : 0);
};

template <int DK, int W, bool OUT>
__global__ void __launch_bounds__(W * 32)
delta_chain_kernel(const ChunkArgs a) {
  using SM = ChainSmem<DK, W, OUT>;
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int kThr = W * 32;
  const int slices = a.dv / (16 * W);
  const int u = blockIdx.x / slices, slice = blockIdx.x % slices;
  const int b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = (lane & 3) * 2;
  const int len = seq_len(a.lens, b, a.T), n_chunks = (len + L - 1) / L;
  const int row = (slice * W + warp) * 16 + g;             // value channels row, row + 8
  const uint32_t s0 = smem_u32(sm);
  const __nv_bfloat16* kp = a.k + b * a.ks.b + hk * a.ks.h;
  const __nv_bfloat16* qp = a.q + b * a.qs.b + hk * a.qs.h;
  const __nv_bfloat16* vp = a.v + b * a.vs.b + h * a.vs.h + slice * W * 16;
  __nv_bfloat16* op = a.o + b * a.os.b + h * a.os.h + (slice * W + warp) * 16;
  constexpr int kRecBytes = rec_bytes(!OUT);               // the gradients' record also has A's lo
  const uint8_t* recs = a.rec + (long long)u * a.chunks * kRecBytes;
  auto load = [&](int c) {
    const uint32_t d = s0 + (c & 1) * SM::kStage;
    const int t0 = c * L;
    const uint8_t* r = recs + (long long)c * kRecBytes;
    load_rows<DK, kThr>(d + SM::kK, kp, a.ks.t, t0, len);
    if (OUT) load_rows<DK, kThr>(d + SM::kQ, qp, a.qs.t, t0, len);
    for (int i = tid; i < L * 2 * W; i += kThr) {
      const int t = i / (2 * W), cc = i % (2 * W);
      const bool ok = t0 + t < len;
      cp_async16(d + SM::kV + swz_cols<W>(t, cc), vp + (long long)(ok ? t0 + t : t0) * a.vs.t + cc * 8, ok);
    }
    load_linear<SM::kRec, kThr>(d + SM::kR, r);
    load_linear<kScal, kThr>(d + SM::kS, r + (OUT ? 3 : 4) * kImg);
    cp_async_commit();
  };
  if (n_chunks > 0) load(0);
  float S[DK / 8][4];
  const long long srow = ((long long)u * a.dv + row) * DK + t2;
#pragma unroll
  for (int j = 0; j < DK / 8; ++j) {
    float2 x = make_float2(0.f, 0.f), y = x;
    if (a.s_in != nullptr) {
      x = *reinterpret_cast<const float2*>(a.s_in + srow + 8 * j);
      y = *reinterpret_cast<const float2*>(a.s_in + srow + 8 * DK + 8 * j);
    }
    S[j][0] = x.x; S[j][1] = x.y; S[j][2] = y.x; S[j][3] = y.y;
  }
  for (int c = 0; c < n_chunks; ++c) {
    cp_async_wait<0>();
    __syncthreads();                                       // chunk c has landed; chunk c - 1 has been read
    if (c + 1 < n_chunks) load(c + 1);
    const uint32_t d = s0 + (c & 1) * SM::kStage;
    const float* scal = reinterpret_cast<const float*>(sm + (c & 1) * SM::kStage + SM::kS);
    const float* eG = scal + kEG * L;
    const float* lam = scal + kLam * L;
    const long long img = (long long)u * a.chunks + c;
    // ---- P^T = S K^T (S as hi + lo); S Q^T (S as hi) beside it
    float P[8][4], O[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) P[n][e] = O[n][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t hi[4], lo[4];
      split_a(S[2 * ks], S[2 * ks + 1], hi, lo);
      if (!OUT) {
        uint32_t* im = a.s0 + img * a.dv * DK;             // two planes of dv * DK / 2 words
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const long long w = block_word((slice * W + warp) * 2 + (e & 1), 2 * ks + (e >> 1), DK / 8, lane);
          im[w] = hi[e];
          im[(long long)a.dv * DK / 2 + w] = lo[e];
        }
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t x[4];
        const uint32_t off = swz<DK>(16 * np + ldn_row(lane), 2 * ks + ldn_col(lane));
        ldsm_x4(d + SM::kK + off, x[0], x[1], x[2], x[3]);
        mma_bf16(P[2 * np], hi, x[0], x[1]);
        mma_bf16(P[2 * np + 1], hi, x[2], x[3]);
        mma_bf16(P[2 * np], lo, x[0], x[1]);
        mma_bf16(P[2 * np + 1], lo, x[2], x[3]);
        if (OUT) {
          ldsm_x4(d + SM::kQ + off, x[0], x[1], x[2], x[3]);
          mma_bf16(O[2 * np], hi, x[0], x[1]);
          mma_bf16(O[2 * np + 1], hi, x[2], x[3]);
        }
      }
    }
    // ---- R^T = V^T - P^T diag(e^G), as hi + lo
    uint32_t rh[4][4], rl[4][4];
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t x[4];                                       // (tokens 0-7 | 8-15) x (channels 0-7 | 8-15)
      ldsm_x4_t(d + SM::kV + swz_cols<W>(16 * np + ldn_row(lane), 2 * warp + ldn_col(lane)), x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* p = P[2 * np + i];
        const float2 e = *reinterpret_cast<const float2*>(eG + 16 * np + 8 * i + t2);
        p[0] = fmaf(-e.x, p[0], bf_lo(x[2 * i]));
        p[1] = fmaf(-e.y, p[1], bf_hi(x[2 * i]));
        p[2] = fmaf(-e.x, p[2], bf_lo(x[2 * i + 1]));
        p[3] = fmaf(-e.y, p[3], bf_hi(x[2 * i + 1]));
      }
      split_a(P[2 * np], P[2 * np + 1], rh[np], rl[np]);
    }
    // ---- U^T = R^T T^T: the diagonal b in fp32, hi hi + lo hi + hi lo below it
    float U[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 bt = *reinterpret_cast<const float2*>(scal + kBeta * L + 8 * n + t2);
      U[n][0] = bt.x * P[n][0]; U[n][1] = bt.y * P[n][1];
      U[n][2] = bt.x * P[n][2]; U[n][3] = bt.y * P[n][3];
    }
#pragma unroll
    for (int np = 0; np < 4; ++np) {
#pragma unroll
      for (int ks = 0; ks <= np; ++ks) {
        uint32_t x[4];
        const uint32_t off = swz<64>(16 * np + ldn_row(lane), 2 * ks + ldn_col(lane));
        ldsm_x4(d + SM::kR + off, x[0], x[1], x[2], x[3]);
        mma_bf16(U[2 * np], rh[ks], x[0], x[1]);
        mma_bf16(U[2 * np + 1], rh[ks], x[2], x[3]);
        mma_bf16(U[2 * np], rl[ks], x[0], x[1]);
        mma_bf16(U[2 * np + 1], rl[ks], x[2], x[3]);
        ldsm_x4(d + SM::kR + kImg + off, x[0], x[1], x[2], x[3]);
        mma_bf16(U[2 * np], rh[ks], x[0], x[1]);
        mma_bf16(U[2 * np + 1], rh[ks], x[2], x[3]);
      }
    }
    if (!OUT) {
      uint32_t* im = a.u + img * a.dv * L;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t hi[4], lo[4];
        split_a(U[2 * ks], U[2 * ks + 1], hi, lo);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const long long w = block_word((slice * W + warp) * 2 + (e & 1), 2 * ks + (e >> 1), L / 8, lane);
          im[w] = hi[e];
          im[(long long)a.dv * L / 2 + w] = lo[e];
        }
      }
    }
    // ---- O^T = scale (S Q^T) diag(e^G) + U^T A^T (U as hi + lo), rounded once, token rows out
    if (OUT) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 e = *reinterpret_cast<const float2*>(eG + 8 * n + t2);
        O[n][0] *= a.scale * e.x;
        O[n][1] *= a.scale * e.y;
        O[n][2] *= a.scale * e.x;
        O[n][3] *= a.scale * e.y;
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t hi[4], lo[4];
        split_a(U[2 * ks], U[2 * ks + 1], hi, lo);
#pragma unroll
        for (int np = ks; np < 4; ++np) {
          uint32_t x[4];
          ldsm_x4(d + SM::kR + 2 * kImg + swz<64>(16 * np + ldn_row(lane), 2 * ks + ldn_col(lane)), x[0], x[1], x[2],
                  x[3]);
          mma_bf16(O[2 * np], hi, x[0], x[1]);
          mma_bf16(O[2 * np + 1], hi, x[2], x[3]);
          mma_bf16(O[2 * np], lo, x[0], x[1]);
          mma_bf16(O[2 * np + 1], lo, x[2], x[3]);
        }
      }
      const uint32_t so = s0 + SM::kO + warp * (L * 32);   // this warp's [64][16]
      __syncwarp();
#pragma unroll
      for (int np = 0; np < 4; ++np)
        stsm_x4_t(so + swz_cols<1>(16 * np + ldn_row(lane), ldn_col(lane)), pack_bf16(O[2 * np][0], O[2 * np][1]),
                  pack_bf16(O[2 * np][2], O[2 * np][3]), pack_bf16(O[2 * np + 1][0], O[2 * np + 1][1]),
                  pack_bf16(O[2 * np + 1][2], O[2 * np + 1][3]));
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * i + (lane >> 1), cc = lane & 1;
        if (c * L + t < len)
          *reinterpret_cast<uint4*>(op + (long long)(c * L + t) * a.os.t + cc * 8) =
              *reinterpret_cast<const uint4*>(sm + SM::kO + warp * (L * 32) + swz_cols<1>(t, cc));
      }
    }
    // ---- S = e^{G_L} S + (U diag(e^{G_L - G}))^T K
    const float el = eG[L - 1];
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] *= el;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = *reinterpret_cast<const float2*>(lam + 16 * ks + 8 * i + t2);
        float* x = U[2 * ks + i];
        x[0] *= f.x; x[1] *= f.y; x[2] *= f.x; x[3] *= f.y;
      }
      split_a(U[2 * ks], U[2 * ks + 1], hi, lo);
#pragma unroll
      for (int j = 0; j < DK / 16; ++j) {
        uint32_t x[4];
        ldsm_x4_t(d + SM::kK + swz<DK>(16 * ks + ldt_row(lane), 2 * j + ldt_col(lane)), x[0], x[1], x[2], x[3]);
        mma_bf16(S[2 * j], hi, x[0], x[1]);
        mma_bf16(S[2 * j + 1], hi, x[2], x[3]);
        mma_bf16(S[2 * j], lo, x[0], x[1]);
        mma_bf16(S[2 * j + 1], lo, x[2], x[3]);
      }
    }
  }
  if (a.s_out != nullptr) {
#pragma unroll
    for (int j = 0; j < DK / 8; ++j) {
      *reinterpret_cast<float2*>(a.s_out + srow + 8 * j) = make_float2(S[j][0], S[j][1]);
      *reinterpret_cast<float2*>(a.s_out + srow + 8 * DK + 8 * j) = make_float2(S[j][2], S[j][3]);
    }
  }
}

template <int DK, bool A_LO>
cudaError_t launch_prepare(const ChunkArgs& a, int B, cudaStream_t stream) {
  constexpr int smem = 2 * L * kXs * 4 > 2 * L * DK * 2 ? 2 * L * kXs * 4 : 2 * L * DK * 2;
  cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel<DK, A_LO>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  delta_prepare_kernel<DK, A_LO><<<(unsigned)(B * a.H) * a.chunks, kPrepThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t prepare(const ChunkArgs& a, int B, int dk, bool a_lo, cudaStream_t stream) {
  if (dk == 128) return a_lo ? launch_prepare<128, true>(a, B, stream) : launch_prepare<128, false>(a, B, stream);
  return a_lo ? launch_prepare<64, true>(a, B, stream) : launch_prepare<64, false>(a, B, stream);
}

template <int DK, int W, bool OUT>
cudaError_t launch_chain(const ChunkArgs& a, int B, cudaStream_t stream) {
  constexpr int smem = ChainSmem<DK, W, OUT>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(delta_chain_kernel<DK, W, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  delta_chain_kernel<DK, W, OUT><<<(unsigned)(B * a.H) * (a.dv / (16 * W)), W * 32, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int DK, bool OUT>
cudaError_t chain(const ChunkArgs& a, int B, cudaStream_t stream) {
  // few heads: fewer warps per CTA, so that the slices of a head's value channels spread over the SMs
  const long long strips = (long long)B * a.H * (a.dv / 16);
  if (strips >= 8 * 96 && a.dv == 128) return launch_chain<DK, 8, OUT>(a, B, stream);
  if (strips >= 4 * 148) return launch_chain<DK, 4, OUT>(a, B, stream);
  if (strips >= 2 * 148) return launch_chain<DK, 2, OUT>(a, B, stream);
  return launch_chain<DK, 1, OUT>(a, B, stream);
}

cudaError_t forward_chain(const ChunkArgs& a, int B, int dk, cudaStream_t stream) {
  bool done = false;
  const cudaError_t e = forward_chain_tc(a, B, dk, stream, &done);
  if (done) return e;
  const bool out = a.s0 == nullptr;
  if (dk == 128) return out ? chain<128, true>(a, B, stream) : chain<128, false>(a, B, stream);
  return out ? chain<64, true>(a, B, stream) : chain<64, false>(a, B, stream);
}

}  // namespace delta

bool delta_chunked(const lte_gdr_dims* d) { return d->dtype == LTE_BF16 && d->T > delta::kFewTokens; }

namespace {
// workspace: records, then the segments' maps and states
struct PrefillLayout {
  int chunks, segs;
  size_t n, x, s, total;
  explicit PrefillLayout(const lte_gdr_dims* d) {
    const size_t units = (size_t)d->B * d->H, state = (size_t)d->dv * d->dk * 4;
    chunks = (d->T + delta::L - 1) / delta::L;
    segs = delta::chain_segments((long long)units, chunks);
    size_t at = units * chunks * delta::rec_bytes(false);
    auto take = [&](size_t bytes) { const size_t r = (at + 255) & ~(size_t)255; at = r + bytes; return r; };
    n = take(segs > 1 ? units * (segs - 1) * state : 0);
    x = take(segs > 1 ? units * (segs - 2) * d->dk * d->dk * 4 : 0);
    s = take(segs > 1 ? units * segs * state : 0);
    total = at;
  }
};
}  // namespace

size_t delta_prefill_bytes(const lte_gdr_dims* d) { return delta_chunked(d) ? PrefillLayout(d).total : 0; }

cudaError_t delta_prefill(const DeltaArgs& a, cudaStream_t stream) {
  const lte_gdr_dims* d = a.d;
  if (!delta_chunked(d)) return delta_recurrent(a, stream);
  const PrefillLayout w(d);
  uint8_t* ws = (uint8_t*)a.scratch;
  delta::ChunkArgs c{};
  c.q = (const __nv_bfloat16*)a.q; c.k = (const __nv_bfloat16*)a.k; c.v = (const __nv_bfloat16*)a.v;
  c.qs = a.qs; c.ks = a.ks; c.vs = a.vs; c.os = a.os;
  c.g = a.g; c.beta = a.beta; c.lens = a.lens; c.s_in = a.s_in; c.s_out = a.s_out;
  c.o = (__nv_bfloat16*)a.o; c.rec = ws;
  c.T = d->T; c.H = d->H; c.Hk = d->Hk; c.dv = d->dv; c.chunks = w.chunks;
  c.scale = d->scale;
  c.segs = w.segs; c.seg_chunks = (w.chunks + w.segs - 1) / w.segs;
  c.seg_n = (float*)(ws + w.n); c.seg_x = (float*)(ws + w.x); c.seg_s = (float*)(ws + w.s);
  cudaError_t e = delta::prepare(c, d->B, d->dk, false, stream);
  return e != cudaSuccess ? e : delta::forward_chain(c, d->B, d->dk, stream);
}

}  // namespace lte
