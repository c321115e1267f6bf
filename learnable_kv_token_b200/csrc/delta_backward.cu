// Gradients of the gated delta rule, in chunks of 64 tokens on tensor cores.
//
// With the notation of delta_chunk.cuh, dS the gradient of the state behind the
// chunk, u, U and T as in the forward pass:
//   dU  = A^T dO + diag(e^{G_L - G}) K dS^T
//   F   = T^T dU             (F_t = b_t y_t, y_t the full gradient of u_t)
//   dV  = F
//   dS_0 = e^{G_L} dS + scale (diag(e^G) dO)^T Q - (diag(e^G) F)^T K
//   dQ  = scale diag(e^G) dO S_0 + W K,      W_ts = scale e^{G_t - G_s} dO_t.U_s (s <= t)
//   dK  = diag(e^{G_L - G}) U dS - diag(e^G) F S_0 + W^T Q + (Z + Z^T) K,
//                                            Z_ts = -e^{G_t - G_s} F_t.U_s (s < t)
//   db_t = y_t.u_t / b_t
//   dg_t = q_t.dq_t - v_t.dv_t + dg_{t+1}    (dg_t = <S_{t-1}, its gradient>; what
//          is read from t on is linear in S_{t-1} and the v together, and
//          linear in q), which within a chunk runs from dg_first = <dS_0, S_0>:
//          no difference of long sums.
// Launches: the per-chunk systems (delta_prepare.cu), the forward chain with S_0
// and U of every chunk to the workspace (delta_chain_tc.cu), the backward chain
// with dS, F and dV (delta_back_tc.cu), then all chunks at once for dQ, dK, dg and
// db (here).  The sums over value channels and over the heads that
// share a key run in a fixed order: no atomics.
#include "delta_chunk.cuh"

namespace lte {
namespace delta {

// -------------------------------------------------------------- all chunks
// One CTA of eight warps per (batch, key head, chunk): warp (m, half) has token
// rows 16 m .. + 15 and one half of the columns of every product.  The value
// heads that share the key head follow one another; dQ and dK stay in
// registers over them and are rounded once.
template <int DK, int DV>
struct GradSmem {
  static constexpr int kK = 0, kQ = kK + L * DK * 2, kD = kQ + L * DK * 2, kU = kD + L * DV * 2;
  static constexpr int kF = kU + 2 * DV * L * 2, kS = kF + DV * L * 2, kG = kS + 2 * DV * DK * 2;
  static constexpr int kW = kG + DV * DK * 2, kZ = kW + 2 * kImg, kC = kZ + kImg;
  static constexpr int kR = kC + kScal, kTotal = kR + 2 * L * 4;
};

template <int DK, int DV>
__global__ void __launch_bounds__(256, 1)
delta_grad_kernel(const GradArgs ga) {
  using SM = GradSmem<DK, DV>;
  static_assert(SM::kTotal <= 227 * 1024, "shared memory");
  const ChunkArgs& a = ga.f;
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int NP = DK / 32;                              // column pairs of 16 per warp in dQ, dK
  const int c = blockIdx.x % a.chunks, bh = blockIdx.x / a.chunks, b = bh / a.Hk, hk = bh % a.Hk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = (lane & 3) * 2;
  const int m = warp & 3, half = warp >> 2, rep = a.H / a.Hk;
  const int len = seq_len(a.lens, b, a.T), t0 = c * L;
  if (t0 >= len) return;
  const uint32_t s0 = smem_u32(sm);
  const int l7 = lane & 7, i0 = (lane >> 3) & 1, i1 = lane >> 4;
  // operands from 8 x 8 blocks: [k][n] as B (both 8-row halves of k, two n-tiles); [k][m] as A
  auto blk = [](uint32_t base, int rb, int cb, int cbs, int r) { return base + (uint32_t)((rb * cbs + cb) * 128 + r * 16); };
  load_rows<DK, 256>(s0 + SM::kK, a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, t0, len);
  load_rows<DK, 256>(s0 + SM::kQ, a.q + b * a.qs.b + hk * a.qs.h, a.qs.t, t0, len);
  float dQ[2 * NP][4], dK[2 * NP][4];
#pragma unroll
  for (int n = 0; n < 2 * NP; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dQ[n][e] = dK[n][e] = 0.f;
  const float* scal = reinterpret_cast<const float*>(sm + SM::kC);
  float* qdq = reinterpret_cast<float*>(sm + SM::kR);
  const int ta = 16 * m + g, tb = ta + 8;                  // this thread's token rows
  for (int r = 0; r < rep; ++r) {
    const int h = hk * rep + r;
    const long long img = ((long long)b * a.H + h) * a.chunks + c;
    if (r > 0) __syncthreads();                            // the head before has been read
    load_rows<DV, 256>(s0 + SM::kD, ga.dO + b * ga.dos.b + h * ga.dos.h, ga.dos.t, t0, len);
    load_linear<2 * DV * L * 2, 256>(s0 + SM::kU, reinterpret_cast<const uint8_t*>(a.u) + img * (2 * DV * L * 2));
    load_linear<DV * L * 2, 256>(s0 + SM::kF, reinterpret_cast<const uint8_t*>(ga.fimg) + img * (DV * L * 2));
    load_linear<kScal, 256>(s0 + SM::kC, a.rec + img * rec_bytes(true) + 4 * kImg);
    cp_async_commit();
    load_linear<2 * DV * DK * 2, 256>(s0 + SM::kS, reinterpret_cast<const uint8_t*>(a.s0) + img * (2 * DV * DK * 2));
    load_linear<DV * DK * 2, 256>(s0 + SM::kG, reinterpret_cast<const uint8_t*>(ga.ds) + img * (DV * DK * 2));
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    // ---- dO U^T (U as hi + lo) and F U^T, columns 32 half .. + 31, on and below the diagonal
    {
      float X[4][4], Y[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) X[n][e] = Y[n][e] = 0.f;
      if (2 * half <= m) {
#pragma unroll
        for (int ks = 0; ks < DV / 16; ++ks) {
          uint32_t ad[4], af[4];
          ldsm_x4(s0 + SM::kD + swz<DV>(16 * m + ldt_row(lane), 2 * ks + ldt_col(lane)), ad[0], ad[1], ad[2], ad[3]);
          ldsm_x4_t(blk(s0 + SM::kF, 2 * ks + i1, 2 * m + i0, L / 8, l7), af[0], af[1], af[2], af[3]);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int np = 2 * half + p;
            if (np <= m) {
              uint32_t x[4];
              ldsm_x4_t(blk(s0 + SM::kU, 2 * ks + i0, 2 * np + i1, L / 8, l7), x[0], x[1], x[2], x[3]);
              mma_bf16(X[2 * p], ad, x[0], x[1]);
              mma_bf16(X[2 * p + 1], ad, x[2], x[3]);
              mma_bf16(Y[2 * p], af, x[0], x[1]);
              mma_bf16(Y[2 * p + 1], af, x[2], x[3]);
              ldsm_x4_t(blk(s0 + SM::kU + DV * L * 2, 2 * ks + i0, 2 * np + i1, L / 8, l7), x[0], x[1], x[2], x[3]);
              mma_bf16(X[2 * p], ad, x[0], x[1]);
              mma_bf16(X[2 * p + 1], ad, x[2], x[3]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int s = 32 * half + 8 * n + t2;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = i ? tb : ta;
            float w[2], z[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float d = s + e <= t ? expf((scal[kGhi * L + t] - scal[kGhi * L + s + e]) +
                                                (scal[kGlo * L + t] - scal[kGlo * L + s + e]))
                                         : 0.f;
              w[e] = s + e <= t ? a.scale * d * X[n][2 * i + e] : 0.f;
              z[e] = s + e < t ? -d * Y[n][2 * i + e] : 0.f;
            }
            uint32_t hi, lo;
            split2(w[0], w[1], hi, lo);
            const uint32_t off = swz<64>(t, s >> 3) + t2 * 2;
            *reinterpret_cast<uint32_t*>(sm + SM::kW + off) = hi;
            *reinterpret_cast<uint32_t*>(sm + SM::kW + kImg + off) = lo;
            *reinterpret_cast<uint32_t*>(sm + SM::kZ + off) = pack_bf16(z[0], z[1]);
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    const float ea = scal[kEG * L + ta], eb = scal[kEG * L + tb];
    float acc[2 * NP][4];
    // ---- dQ of this head: scale e^G dO S_0 + W K, and q.dq per token
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DV / 16; ++ks) {
      uint32_t ad[4];
      ldsm_x4(s0 + SM::kD + swz<DV>(16 * m + ldt_row(lane), 2 * ks + ldt_col(lane)), ad[0], ad[1], ad[2], ad[3]);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t x[4];
        const int cb = 2 * (half * NP + p) + i1;
        ldsm_x4_t(blk(s0 + SM::kS, 2 * ks + i0, cb, DK / 8, l7), x[0], x[1], x[2], x[3]);
        mma_bf16(acc[2 * p], ad, x[0], x[1]);
        mma_bf16(acc[2 * p + 1], ad, x[2], x[3]);
        ldsm_x4_t(blk(s0 + SM::kS + DV * DK * 2, 2 * ks + i0, cb, DK / 8, l7), x[0], x[1], x[2], x[3]);
        mma_bf16(acc[2 * p], ad, x[0], x[1]);
        mma_bf16(acc[2 * p + 1], ad, x[2], x[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n) {
      acc[n][0] *= a.scale * ea; acc[n][1] *= a.scale * ea;
      acc[n][2] *= a.scale * eb; acc[n][3] *= a.scale * eb;
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks <= m) {
        uint32_t wh[4], wl[4];
        const uint32_t off = swz<64>(16 * m + ldt_row(lane), 2 * ks + ldt_col(lane));
        ldsm_x4(s0 + SM::kW + off, wh[0], wh[1], wh[2], wh[3]);
        ldsm_x4(s0 + SM::kW + kImg + off, wl[0], wl[1], wl[2], wl[3]);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint32_t x[4];
          ldsm_x4_t(s0 + SM::kK + swz<DK>(16 * ks + ldt_row(lane), 2 * (half * NP + p) + ldt_col(lane)), x[0], x[1],
                    x[2], x[3]);
          mma_bf16(acc[2 * p], wh, x[0], x[1]);
          mma_bf16(acc[2 * p + 1], wh, x[2], x[3]);
          mma_bf16(acc[2 * p], wl, x[0], x[1]);
          mma_bf16(acc[2 * p + 1], wl, x[2], x[3]);
        }
      }
    }
    {
      float da = 0.f, dbb = 0.f;
#pragma unroll
      for (int n = 0; n < 2 * NP; ++n) {
        const int cc = half * 2 * NP + n;
        const uint32_t qa = *reinterpret_cast<const uint32_t*>(sm + SM::kQ + swz<DK>(ta, cc) + t2 * 2);
        const uint32_t qb = *reinterpret_cast<const uint32_t*>(sm + SM::kQ + swz<DK>(tb, cc) + t2 * 2);
        da = fmaf(acc[n][0], bf_lo(qa), fmaf(acc[n][1], bf_hi(qa), da));
        dbb = fmaf(acc[n][2], bf_lo(qb), fmaf(acc[n][3], bf_hi(qb), dbb));
#pragma unroll
        for (int e = 0; e < 4; ++e) dQ[n][e] += acc[n][e];
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        da += __shfl_xor_sync(0xffffffffu, da, o);
        dbb += __shfl_xor_sync(0xffffffffu, dbb, o);
      }
      if ((lane & 3) == 0) {
        qdq[half * L + ta] = da;
        qdq[half * L + tb] = dbb;
      }
    }
    // ---- dK of this head; rows are the tokens s
    const float la = scal[kLam * L + ta], lb = scal[kLam * L + tb];
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DV / 16; ++ks) {                 // U dS
      uint32_t au[4];
      ldsm_x4_t(blk(s0 + SM::kU, 2 * ks + i1, 2 * m + i0, L / 8, l7), au[0], au[1], au[2], au[3]);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t x[4];
        ldsm_x4_t(blk(s0 + SM::kG, 2 * ks + i0, 2 * (half * NP + p) + i1, DK / 8, l7), x[0], x[1], x[2], x[3]);
        mma_bf16(acc[2 * p], au, x[0], x[1]);
        mma_bf16(acc[2 * p + 1], au, x[2], x[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n) {
      dK[n][0] = fmaf(la, acc[n][0], dK[n][0]); dK[n][1] = fmaf(la, acc[n][1], dK[n][1]);
      dK[n][2] = fmaf(lb, acc[n][2], dK[n][2]); dK[n][3] = fmaf(lb, acc[n][3], dK[n][3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    }
#pragma unroll
    for (int ks = 0; ks < DV / 16; ++ks) {                 // F S_0
      uint32_t af[4];
      ldsm_x4_t(blk(s0 + SM::kF, 2 * ks + i1, 2 * m + i0, L / 8, l7), af[0], af[1], af[2], af[3]);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t x[4];
        ldsm_x4_t(blk(s0 + SM::kS, 2 * ks + i0, 2 * (half * NP + p) + i1, DK / 8, l7), x[0], x[1], x[2], x[3]);
        mma_bf16(acc[2 * p], af, x[0], x[1]);
        mma_bf16(acc[2 * p + 1], af, x[2], x[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n) {
      dK[n][0] = fmaf(-ea, acc[n][0], dK[n][0]); dK[n][1] = fmaf(-ea, acc[n][1], dK[n][1]);
      dK[n][2] = fmaf(-eb, acc[n][2], dK[n][2]); dK[n][3] = fmaf(-eb, acc[n][3], dK[n][3]);
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t z[4], w[4], y[4];
      if (ks <= m) ldsm_x4(s0 + SM::kZ + swz<64>(16 * m + ldt_row(lane), 2 * ks + ldt_col(lane)), z[0], z[1], z[2], z[3]);
      if (ks >= m) {
        const uint32_t off = swz<64>(16 * ks + ldn_row(lane), 2 * m + ldn_col(lane));
        ldsm_x4_t(s0 + SM::kW + off, w[0], w[1], w[2], w[3]);
        ldsm_x4_t(s0 + SM::kZ + off, y[0], y[1], y[2], y[3]);
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t x[4];
        const uint32_t off = swz<DK>(16 * ks + ldt_row(lane), 2 * (half * NP + p) + ldt_col(lane));
        ldsm_x4_t(s0 + SM::kK + off, x[0], x[1], x[2], x[3]);
        if (ks <= m) {                                     // Z K
          mma_bf16(dK[2 * p], z, x[0], x[1]);
          mma_bf16(dK[2 * p + 1], z, x[2], x[3]);
        }
        if (ks >= m) {                                     // Z^T K + W^T Q
          mma_bf16(dK[2 * p], y, x[0], x[1]);
          mma_bf16(dK[2 * p + 1], y, x[2], x[3]);
          ldsm_x4_t(s0 + SM::kQ + off, x[0], x[1], x[2], x[3]);
          mma_bf16(dK[2 * p], w, x[0], x[1]);
          mma_bf16(dK[2 * p + 1], w, x[2], x[3]);
        }
      }
    }
    __syncthreads();                                       // q.dq of both halves
    // ---- gates: db_t = u.y / b, dg_t = <dS_0, S_0> - sum_{t' < t} (q.dq - v.dv)
    if (warp == 0) {
      constexpr int strips = DV / 16;
      const float* xp = ga.x + img * strips * (2 * L) + 2 * lane;
      double in = 0.0;
      float x[2] = {0.f, 0.f}, vf[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < strips; ++i) {
        in += (double)ga.inner[img * strips + i];
        const float2 p = *reinterpret_cast<const float2*>(xp + i * 2 * L);
        const float2 q = *reinterpret_cast<const float2*>(xp + i * 2 * L + L);
        x[0] += p.x;
        x[1] += p.y;
        vf[0] += q.x;
        vf[1] += q.y;
      }
      const double y0 = (double)(qdq[2 * lane] + qdq[L + 2 * lane]) - vf[0];
      const double y1 = (double)(qdq[2 * lane + 1] + qdq[L + 2 * lane + 1]) - vf[1];
      double sum = y0 + y1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const double first = in - (sum - y1 - y0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = t0 + 2 * lane + i;
        if (t < len) {
          const long long gi = ((long long)b * a.T + t) * a.H + h;
          ga.dg[gi] = (float)(i ? first - y0 : first);
          ga.db[gi] = x[i] / scal[kBeta * L + 2 * lane + i];
        }
      }
    }
  }
  // ---- dQ, dK as bf16 token rows, through the K and Q tiles
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 2 * NP; ++n) {
    const int cc = half * 2 * NP + n;
    *reinterpret_cast<uint32_t*>(sm + SM::kQ + swz<DK>(ta, cc) + t2 * 2) = pack_bf16(dQ[n][0], dQ[n][1]);
    *reinterpret_cast<uint32_t*>(sm + SM::kQ + swz<DK>(tb, cc) + t2 * 2) = pack_bf16(dQ[n][2], dQ[n][3]);
    *reinterpret_cast<uint32_t*>(sm + SM::kK + swz<DK>(ta, cc) + t2 * 2) = pack_bf16(dK[n][0], dK[n][1]);
    *reinterpret_cast<uint32_t*>(sm + SM::kK + swz<DK>(tb, cc) + t2 * 2) = pack_bf16(dK[n][2], dK[n][3]);
  }
  __syncthreads();
  for (int i = tid; i < L * (DK / 8); i += 256) {
    const int t = i / (DK / 8), cc = i % (DK / 8);
    if (t0 + t < len) {
      const long long o = (((long long)b * a.T + t0 + t) * a.Hk + hk) * DK + cc * 8;
      *reinterpret_cast<uint4*>(ga.dq + o) = *reinterpret_cast<const uint4*>(sm + SM::kQ + swz<DK>(t, cc));
      *reinterpret_cast<uint4*>(ga.dk + o) = *reinterpret_cast<const uint4*>(sm + SM::kK + swz<DK>(t, cc));
    }
  }
}

template <int DK, int DV>
cudaError_t grad(const GradArgs& a, int B, cudaStream_t stream) {
  constexpr int smem = GradSmem<DK, DV>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(delta_grad_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  delta_grad_kernel<DK, DV><<<(unsigned)(B * a.f.Hk) * a.f.chunks, 256, smem, stream>>>(a);
  return cudaGetLastError();
}

// workspace: records, then the images and partial sums, each rounded up to 256 bytes
struct BackwardLayout {
  size_t rec, s0, u, f, ds, x, inner, total;
  explicit BackwardLayout(const lte_gdr_dims* d) {
    const size_t n = (size_t)d->B * d->H * ((d->T + L - 1) / L), dv = d->dv, dk = d->dk;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += (bytes + 255) & ~(size_t)255; return r; };
    rec = take(n * rec_bytes(true));
    s0 = take(n * dv * dk * 4);
    u = take(n * dv * L * 4);
    f = take(n * dv * L * 2);
    ds = take(n * dv * dk * 2);
    x = take(n * (dv / 16) * 2 * L * 4);
    inner = take(n * (dv / 16) * 4);
    total = at;
  }
};

}  // namespace delta

size_t delta_backward_bytes(const lte_gdr_dims* d) { return delta::BackwardLayout(d).total; }

cudaError_t delta_backward(const DeltaArgs& a, const DeltaGradArgs& ga, cudaStream_t stream) {
  const lte_gdr_dims* d = a.d;
  const delta::BackwardLayout w(d);
  uint8_t* ws = (uint8_t*)a.scratch;
  delta::GradArgs n{};
  delta::ChunkArgs& c = n.f;
  c.q = (const __nv_bfloat16*)a.q; c.k = (const __nv_bfloat16*)a.k; c.v = (const __nv_bfloat16*)a.v;
  c.qs = a.qs; c.ks = a.ks; c.vs = a.vs; c.g = a.g; c.beta = a.beta; c.lens = a.lens; c.s_in = a.s_in;
  c.rec = ws + w.rec; c.s0 = (uint32_t*)(ws + w.s0); c.u = (uint32_t*)(ws + w.u);
  c.T = d->T; c.H = d->H; c.Hk = d->Hk; c.dv = d->dv; c.chunks = (d->T + delta::L - 1) / delta::L;
  c.scale = d->scale; c.segs = 1; c.seg_chunks = c.chunks;
  n.dO = (const __nv_bfloat16*)ga.dO; n.dos = ga.dos; n.ds_out = ga.ds_out; n.ds_in = ga.ds_in;
  n.dq = (__nv_bfloat16*)ga.dq; n.dk = (__nv_bfloat16*)ga.dk; n.dv = (__nv_bfloat16*)ga.dv;
  n.dg = ga.dg; n.db = ga.db; n.ds = (uint32_t*)(ws + w.ds); n.fimg = (uint32_t*)(ws + w.f);
  n.x = (float*)(ws + w.x); n.inner = (float*)(ws + w.inner);
  cudaError_t e = delta::prepare(c, d->B, d->dk, true, stream);
  if (e == cudaSuccess) e = delta::forward_chain(c, d->B, d->dk, stream);
  if (e == cudaSuccess) e = delta::back_chain(n, d->B, d->dk, stream);
  if (e != cudaSuccess) return e;
  if (d->dk == 128)
    return d->dv == 128 ? delta::grad<128, 128>(n, d->B, stream) : delta::grad<128, 64>(n, d->B, stream);
  return d->dv == 128 ? delta::grad<64, 128>(n, d->B, stream) : delta::grad<64, 64>(n, d->B, stream);
}

}  // namespace lte
