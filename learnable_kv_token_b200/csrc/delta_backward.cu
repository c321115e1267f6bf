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
#include "delta_chain_tc.cuh"

namespace lte {
namespace delta {

// -------------------------------------------------------------- all chunks
// Persistent CTAs of sixteen warps, one per SM, over (batch, key head, chunk): warp
// (m, q) has token rows 16 m .. + 15 and a quarter of the columns of every product
// (warp MMAs: the operands are small, all in shared memory, and each result's rows
// are scaled, summed or masked before its next use).  The value channels come in
// halves, two buffers deep: the next half, of the next head or chunk too, loads
// while this one is in use (images by bulk copies, token rows by cp.async).  The value heads that share a key head follow
// one another; dQ and dK stay in registers over them and are rounded once.
// 224 KB read per chunk and head, 176 of them images: 8 x 4096 tokens x 16 heads of
// 128 channels in 545 us, 3.4 TB/s (572 for 4 key heads, each shared by four).  Of 19000 cycles per chunk 7200 are warp MMAs;
// the rest is phases between barriers with sixteen warps to an SM.
// What feeds dQ, and through q.dQ the gates, takes pairs (U, S_0, W).  What feeds dK
// alone takes one bf16 of each: F and dS, which no pair of is kept, U and S_0 beside
// them, W transposed, Z.  dK comes out 2.9e-3 off in the 2-norm, 1.7e-3 of it its own
// rounding; with the pairs that are here (U, S_0, W) 2.3e-3, in 645 us for 545.
constexpr int kGradThreads = 512;
constexpr int kHV = 64;                                    // value channels of a half

template <int DK>
struct GradSmem {
  static constexpr int kD = 0, kU = kD + L * kHV * 2, kF = kU + 2 * kHV * L * 2, kS = kF + kHV * L * 2;
  static constexpr int kG = kS + 2 * kHV * DK * 2, kStage = kG + kHV * DK * 2;
  static constexpr int kK = 2 * kStage, kQ = kK + L * DK * 2, kW = kQ + L * DK * 2, kZ = kW + 2 * kImg;
  static constexpr int kR = kZ + kImg, kC = kR + 4 * L * 4;
  // a head's scalars and its partial sums of u.y, v.dv and <dS_0, S_0> (up to 8 strips)
  static constexpr int kX = kC + kScal, kI = kX + 8 * 2 * L * 4, kBar = kI + 32, kTotal = kBar + 32;
};

// SHARED: several value heads to a key head, whose dQ and dK are kept in registers
// beside the products of the next one
template <int DK, int DV, bool SHARED>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_kernel(const GradArgs ga, int items) {
  using SM = GradSmem<DK>;
  static_assert(SM::kTotal <= 227 * 1024, "shared memory");
  const ChunkArgs& a = ga.f;
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int NP = DK / 64, NH = DV / kHV;               // column pairs of 16 per warp in dQ, dK; halves
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = (lane & 3) * 2;
  // (m differs among the warps of a scheduler: work on and below the diagonal grows with it)
  const int q = warp >> 2, m = (warp + q) & 3, rep = SHARED ? a.H / a.Hk : 1;
  const uint32_t s0 = smem_u32(sm);
  const int l7 = lane & 7, i0 = (lane >> 3) & 1, i1 = lane >> 4;
  // operands from 8 x 8 blocks: [k][n] as B (both 8-row halves of k, two n-tiles); [k][m] as A
  auto blk = [](uint32_t base, int rb, int cb, int cbs, int r) { return base + (uint32_t)((rb * cbs + cb) * 128 + r * 16); };
  auto len_of = [&](int it) { return seq_len(a.lens, it / a.chunks / a.Hk, a.T); };
  auto next = [&](int it) {                                // the next chunk that has tokens
    for (it += gridDim.x; it < items && (it % a.chunks) * L >= len_of(it); it += gridDim.x) {
    }
    return it;
  };
  auto load_half = [&](int it, int r, int hv, uint32_t n) {   // the CTA's n-th
    const int c = it % a.chunks, bh = it / a.chunks, b = bh / a.Hk, h = (bh % a.Hk) * rep + r;
    const long long img = ((long long)b * a.H + h) * a.chunks + c;
    const uint32_t buf = n & 1, d = s0 + buf * SM::kStage;
    load_rows<kHV, kGradThreads>(d + SM::kD, ga.dO + b * ga.dos.b + h * ga.dos.h + hv * kHV, ga.dos.t, c * L, len_of(it));
    if (tid != 0 || (int)n == a.withhold) return;
    const uint32_t bar = s0 + SM::kBar + 8 * buf;
    chaintc::mbar_expect_tx(bar, SM::kStage - SM::kU);
    const uint8_t* us = reinterpret_cast<const uint8_t*>(a.u) + img * (2 * DV * L * 2) + hv * (kHV * L * 2);
    const uint8_t* ss = reinterpret_cast<const uint8_t*>(a.s0) + img * (2 * DV * DK * 2) + hv * (kHV * DK * 2);
    chaintc::bulk_load(d + SM::kU, us, kHV * L * 2, bar);
    chaintc::bulk_load(d + SM::kU + kHV * L * 2, us + DV * L * 2, kHV * L * 2, bar);
    chaintc::bulk_load(d + SM::kF, reinterpret_cast<const uint8_t*>(ga.fimg) + img * (DV * L * 2) + hv * (kHV * L * 2), kHV * L * 2, bar);
    chaintc::bulk_load(d + SM::kS, ss, kHV * DK * 2, bar);
    chaintc::bulk_load(d + SM::kS + kHV * DK * 2, ss + DV * DK * 2, kHV * DK * 2, bar);
    chaintc::bulk_load(d + SM::kG, reinterpret_cast<const uint8_t*>(ga.ds) + img * (DV * DK * 2) + hv * (kHV * DK * 2), kHV * DK * 2, bar);
  };
  float* qdq = reinterpret_cast<float*>(sm + SM::kR);
  const int ta = 16 * m + g, tb = ta + 8;                  // this thread's token rows
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + SM::kBar + 16);
  if (tid == 0) {
    chaintc::mbar_init(s0 + SM::kBar, 1);
    chaintc::mbar_init(s0 + SM::kBar + 8, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint32_t halves = 0;                                     // halves waited for; buffer = halves mod 2
  bool ok = true;
  int it = next((int)blockIdx.x - (int)gridDim.x);
  if (it < items) load_half(it, 0, 0, 0);
  cp_async_commit();
  while (it < items) {
    const int c = it % a.chunks, bh = it / a.chunks, b = bh / a.Hk, hk = bh % a.Hk, t0 = c * L;
    const int len = len_of(it), it1 = next(it);
    float dQ[2 * NP][4], dK[2 * NP][4];
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dQ[n][e] = dK[n][e] = 0.f;
#pragma unroll 1
    for (int r = 0; r < rep; ++r) {
      const int h = hk * rep + r;
      const long long img = ((long long)b * a.H + h) * a.chunks + c;
      float X[2][4], Y[2][4], QI[2 * NP][4], US[2 * NP][4], FS[2 * NP][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int n = 0; n < 2; ++n) X[n][e] = Y[n][e] = 0.f;
#pragma unroll
        for (int n = 0; n < 2 * NP; ++n) QI[n][e] = US[n][e] = FS[n][e] = 0.f;
      }
#pragma unroll 1
      for (int hv = 0; hv < NH; ++hv) {
        const int buf = halves & 1;
        cp_async_wait<0>();
        ok = chaintc::mbar_wait(s0 + SM::kBar + 8 * buf, (halves >> 1) & 1, a.wait_ns, abort_flag);
        ++halves;
        // this half has landed; the one before has been read
        if (!(ok = __syncthreads_and(ok))) break;
        if (r == 0 && hv == 0) {                           // (and so have the chunk before's K and Q)
          load_rows<DK, kGradThreads>(s0 + SM::kK, a.k + b * a.ks.b + hk * a.ks.h, a.ks.t, t0, len);
          load_rows<DK, kGradThreads>(s0 + SM::kQ, a.q + b * a.qs.b + hk * a.qs.h, a.qs.t, t0, len);
        }
        if (hv == 0) {                                     // the head's small things, used behind its last half
          load_linear<kScal, kGradThreads>(s0 + SM::kC, a.rec + img * rec_bytes(true) + 4 * kImg);
          load_linear<(DV / 16) * 2 * L * 4, kGradThreads>(s0 + SM::kX, reinterpret_cast<const uint8_t*>(ga.x) + img * ((DV / 16) * 2 * L * 4));
          load_linear<(DV / 16) * 4, kGradThreads>(s0 + SM::kI, reinterpret_cast<const uint8_t*>(ga.inner) + img * ((DV / 16) * 4));
          if (NH == 1) cp_async_commit();
        }
        if (hv + 1 < NH) load_half(it, r, hv + 1, halves);
        else if (r + 1 < rep) load_half(it, r + 1, 0, halves);
        else if (it1 < items) load_half(it1, 0, 0, halves);
        cp_async_commit();
        const uint32_t d = s0 + buf * SM::kStage;
#pragma unroll
        for (int ks = 0; ks < kHV / 16; ++ks) {
          uint32_t ad[4], af[4], au[4];
          ldsm_x4(d + SM::kD + swz<kHV>(16 * m + ldt_row(lane), 2 * ks + ldt_col(lane)), ad[0], ad[1], ad[2], ad[3]);
          ldsm_x4_t(blk(d + SM::kF, 2 * ks + i1, 2 * m + i0, L / 8, l7), af[0], af[1], af[2], af[3]);
          ldsm_x4_t(blk(d + SM::kU, 2 * ks + i1, 2 * m + i0, L / 8, l7), au[0], au[1], au[2], au[3]);
          if (q <= m) {                                    // dO U^T (U as hi + lo), F U^T: columns 16 q .. + 15
            uint32_t x[4];
            ldsm_x4_t(blk(d + SM::kU, 2 * ks + i0, 2 * q + i1, L / 8, l7), x[0], x[1], x[2], x[3]);
            mma_bf16(X[0], ad, x[0], x[1]);
            mma_bf16(X[1], ad, x[2], x[3]);
            mma_bf16(Y[0], af, x[0], x[1]);
            mma_bf16(Y[1], af, x[2], x[3]);
            ldsm_x4_t(blk(d + SM::kU + kHV * L * 2, 2 * ks + i0, 2 * q + i1, L / 8, l7), x[0], x[1], x[2], x[3]);
            mma_bf16(X[0], ad, x[0], x[1]);
            mma_bf16(X[1], ad, x[2], x[3]);
          }
#pragma unroll
          for (int p = 0; p < NP; ++p) {                   // dO S_0 (hi + lo), F S_0, U dS
            uint32_t x[4];
            const int cb = 2 * (q * NP + p) + i1;
            ldsm_x4_t(blk(d + SM::kS, 2 * ks + i0, cb, DK / 8, l7), x[0], x[1], x[2], x[3]);
            mma_bf16(QI[2 * p], ad, x[0], x[1]);
            mma_bf16(QI[2 * p + 1], ad, x[2], x[3]);
            mma_bf16(FS[2 * p], af, x[0], x[1]);
            mma_bf16(FS[2 * p + 1], af, x[2], x[3]);
            ldsm_x4_t(blk(d + SM::kS + kHV * DK * 2, 2 * ks + i0, cb, DK / 8, l7), x[0], x[1], x[2], x[3]);
            mma_bf16(QI[2 * p], ad, x[0], x[1]);
            mma_bf16(QI[2 * p + 1], ad, x[2], x[3]);
            ldsm_x4_t(blk(d + SM::kG, 2 * ks + i0, cb, DK / 8, l7), x[0], x[1], x[2], x[3]);
            mma_bf16(US[2 * p], au, x[0], x[1]);
            mma_bf16(US[2 * p + 1], au, x[2], x[3]);
          }
        }
      }
      if (!ok) break;
      const float* scal = reinterpret_cast<const float*>(sm + SM::kC);
      if (NH == 1) {                                       // K, Q and the small things (else: waited for with the second half)
        cp_async_wait<1>();
        __syncthreads();
      }
      // ---- W and Z from dO U^T and F U^T
      if (q <= m) {
        const float ha = scal[kGhi * L + ta], oa = scal[kGlo * L + ta], hb = scal[kGhi * L + tb], ob = scal[kGlo * L + tb];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int s = 16 * q + 8 * n + t2;
          const float2 hs = *reinterpret_cast<const float2*>(scal + kGhi * L + s);
          const float2 os = *reinterpret_cast<const float2*>(scal + kGlo * L + s);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = i ? tb : ta;
            const float gh = i ? hb : ha, go = i ? ob : oa;
            const float d0 = s <= t ? expf((gh - hs.x) + (go - os.x)) : 0.f;
            const float d1 = s + 1 <= t ? expf((gh - hs.y) + (go - os.y)) : 0.f;
            uint32_t hi, lo;
            split2(a.scale * d0 * X[n][2 * i], a.scale * d1 * X[n][2 * i + 1], hi, lo);
            const uint32_t off = swz<64>(t, s >> 3) + t2 * 2;
            *reinterpret_cast<uint32_t*>(sm + SM::kW + off) = hi;
            *reinterpret_cast<uint32_t*>(sm + SM::kW + kImg + off) = lo;
            *reinterpret_cast<uint32_t*>(sm + SM::kZ + off) =
                pack_bf16(s < t ? -d0 * Y[n][2 * i] : 0.f, s + 1 < t ? -d1 * Y[n][2 * i + 1] : 0.f);
          }
        }
      }
      __syncthreads();
      // ---- dQ of this head: scale e^G dO S_0 + W K, and q.dq per token
      const float ea = scal[kEG * L + ta], eb = scal[kEG * L + tb], la = scal[kLam * L + ta], lb = scal[kLam * L + tb];
#pragma unroll
      for (int n = 0; n < 2 * NP; ++n) {
        QI[n][0] *= a.scale * ea; QI[n][1] *= a.scale * ea;
        QI[n][2] *= a.scale * eb; QI[n][3] *= a.scale * eb;
        dK[n][0] += la * US[n][0] - ea * FS[n][0]; dK[n][1] += la * US[n][1] - ea * FS[n][1];
        dK[n][2] += lb * US[n][2] - eb * FS[n][2]; dK[n][3] += lb * US[n][3] - eb * FS[n][3];
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t wh[4], wl[4], z[4], w[4], y[4];
        if (ks <= m) {
          const uint32_t off = swz<64>(16 * m + ldt_row(lane), 2 * ks + ldt_col(lane));
          ldsm_x4(s0 + SM::kW + off, wh[0], wh[1], wh[2], wh[3]);
          ldsm_x4(s0 + SM::kW + kImg + off, wl[0], wl[1], wl[2], wl[3]);
          ldsm_x4(s0 + SM::kZ + off, z[0], z[1], z[2], z[3]);
        }
        if (ks >= m) {
          const uint32_t off = swz<64>(16 * ks + ldn_row(lane), 2 * m + ldn_col(lane));
          ldsm_x4_t(s0 + SM::kW + off, w[0], w[1], w[2], w[3]);
          ldsm_x4_t(s0 + SM::kZ + off, y[0], y[1], y[2], y[3]);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          uint32_t x[4];
          const uint32_t off = swz<DK>(16 * ks + ldt_row(lane), 2 * (q * NP + p) + ldt_col(lane));
          ldsm_x4_t(s0 + SM::kK + off, x[0], x[1], x[2], x[3]);
          if (ks <= m) {                                   // W K; Z K
            mma_bf16(QI[2 * p], wh, x[0], x[1]);
            mma_bf16(QI[2 * p + 1], wh, x[2], x[3]);
            mma_bf16(QI[2 * p], wl, x[0], x[1]);
            mma_bf16(QI[2 * p + 1], wl, x[2], x[3]);
            mma_bf16(dK[2 * p], z, x[0], x[1]);
            mma_bf16(dK[2 * p + 1], z, x[2], x[3]);
          }
          if (ks >= m) {                                   // Z^T K; W^T Q
            mma_bf16(dK[2 * p], y, x[0], x[1]);
            mma_bf16(dK[2 * p + 1], y, x[2], x[3]);
            ldsm_x4_t(s0 + SM::kQ + off, x[0], x[1], x[2], x[3]);
            mma_bf16(dK[2 * p], w, x[0], x[1]);
            mma_bf16(dK[2 * p + 1], w, x[2], x[3]);
          }
        }
      }
      {
        float da = 0.f, dbb = 0.f;
#pragma unroll
        for (int n = 0; n < 2 * NP; ++n) {
          const int cc = q * 2 * NP + n;
          const uint32_t qa = *reinterpret_cast<const uint32_t*>(sm + SM::kQ + swz<DK>(ta, cc) + t2 * 2);
          const uint32_t qb = *reinterpret_cast<const uint32_t*>(sm + SM::kQ + swz<DK>(tb, cc) + t2 * 2);
          da = fmaf(QI[n][0], bf_lo(qa), fmaf(QI[n][1], bf_hi(qa), da));
          dbb = fmaf(QI[n][2], bf_lo(qb), fmaf(QI[n][3], bf_hi(qb), dbb));
#pragma unroll
          for (int e = 0; e < 4; ++e) dQ[n][e] += QI[n][e];
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          da += __shfl_xor_sync(0xffffffffu, da, o);
          dbb += __shfl_xor_sync(0xffffffffu, dbb, o);
        }
        if ((lane & 3) == 0) {
          qdq[q * L + ta] = da;
          qdq[q * L + tb] = dbb;
        }
      }
      __syncthreads();                                     // q.dq of all quarters; W and Z have been read
      // ---- gates: db_t = u.y / b, dg_t = <dS_0, S_0> - sum_{t' < t} (q.dq - v.dv)
      if (warp == 15) {                                    // (the warps with q > m have less to do before)
        constexpr int strips = DV / 16;
        const float* xp = reinterpret_cast<const float*>(sm + SM::kX) + 2 * lane;
        const float* inner = reinterpret_cast<const float*>(sm + SM::kI);
        double in = 0.0;
        float x[2] = {0.f, 0.f}, vf[2] = {0.f, 0.f}, qd[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < strips; ++i) {
          in += (double)inner[i];
          const float2 p = *reinterpret_cast<const float2*>(xp + i * 2 * L);
          const float2 w = *reinterpret_cast<const float2*>(xp + i * 2 * L + L);
          x[0] += p.x;
          x[1] += p.y;
          vf[0] += w.x;
          vf[1] += w.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qd[0] += qdq[i * L + 2 * lane];
          qd[1] += qdq[i * L + 2 * lane + 1];
        }
        const double y0 = (double)qd[0] - vf[0], y1 = (double)qd[1] - vf[1];
        double sum = y0 + y1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        const double first = in - (sum - y1 - y0);
        // nothing passes a gate whose exponential is zero (-104 in the sums), and no gradient: not the
        // rounding of a difference that should vanish
        const float2 gh = *reinterpret_cast<const float2*>(scal + kGhi * L + 2 * lane);
        const float2 go = *reinterpret_cast<const float2*>(scal + kGlo * L + 2 * lane);
        const float ph = __shfl_up_sync(0xffffffffu, gh.y, 1), po = __shfl_up_sync(0xffffffffu, go.y, 1);
        const bool shut[2] = {(gh.x - (lane ? ph : 0.f)) + (go.x - (lane ? po : 0.f)) < -103.99f,
                              (gh.y - gh.x) + (go.y - go.x) < -103.99f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = t0 + 2 * lane + i;
          if (t < len) {
            const long long gi = ((long long)b * a.T + t) * a.H + h;
            ga.dg[gi] = shut[i] ? 0.f : (float)(i ? first - y0 : first);
            ga.db[gi] = x[i] / scal[kBeta * L + 2 * lane + i];
          }
        }
      }
    }
    if (!ok) break;
    // ---- dQ, dK as bf16 token rows, through the K and Q tiles (all warps are past them)
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n) {
      const int cc = q * 2 * NP + n;
      *reinterpret_cast<uint32_t*>(sm + SM::kQ + swz<DK>(ta, cc) + t2 * 2) = pack_bf16(dQ[n][0], dQ[n][1]);
      *reinterpret_cast<uint32_t*>(sm + SM::kQ + swz<DK>(tb, cc) + t2 * 2) = pack_bf16(dQ[n][2], dQ[n][3]);
      *reinterpret_cast<uint32_t*>(sm + SM::kK + swz<DK>(ta, cc) + t2 * 2) = pack_bf16(dK[n][0], dK[n][1]);
      *reinterpret_cast<uint32_t*>(sm + SM::kK + swz<DK>(tb, cc) + t2 * 2) = pack_bf16(dK[n][2], dK[n][3]);
    }
    __syncthreads();
    for (int i = tid; i < L * (DK / 8); i += kGradThreads) {
      const int t = i / (DK / 8), cc = i % (DK / 8);
      if (t0 + t < len) {
        const long long o = (((long long)b * a.T + t0 + t) * a.Hk + hk) * DK + cc * 8;
        *reinterpret_cast<uint4*>(ga.dq + o) = *reinterpret_cast<const uint4*>(sm + SM::kQ + swz<DK>(t, cc));
        *reinterpret_cast<uint4*>(ga.dk + o) = *reinterpret_cast<const uint4*>(sm + SM::kK + swz<DK>(t, cc));
      }
    }
    it = it1;
  }
  cp_async_wait<0>();
  if (!ok) {                                               // a copy did not land: NaN in all that is not done
    if (tid == 0 && (int)halves - 1 != a.withhold) chaintc::mbar_drain(s0 + SM::kBar + 8 * ((halves - 1) & 1), ((halves - 1) >> 1) & 1);
    for (; it < items; it = next(it)) {
      const int bh = it / a.chunks, b = bh / a.Hk, hk = bh % a.Hk, t0 = (it % a.chunks) * L, n = min(len_of(it) - t0, L);
      const long long row = (long long)b * a.T + t0;
      chaintc::nan_rows<DK>(ga.dq + (row * a.Hk + hk) * DK, (long long)a.Hk * DK, n, tid, kGradThreads);
      chaintc::nan_rows<DK>(ga.dk + (row * a.Hk + hk) * DK, (long long)a.Hk * DK, n, tid, kGradThreads);
      for (int i = tid; i < n * rep; i += kGradThreads)
        ga.dg[(row + i / rep) * a.H + hk * rep + i % rep] = ga.db[(row + i / rep) * a.H + hk * rep + i % rep] =
            __int_as_float(0x7fffffff);
    }
    __syncthreads();
  }
}

template <int DK, int DV, bool SHARED>
cudaError_t grad_as(const GradArgs& args, int B, cudaStream_t stream) {
  GradArgs a = args;
  set_waits(a.f, LTE_GDR_LAUNCH_PASS);
  constexpr int smem = GradSmem<DK>::kTotal;
  const int items = B * a.f.Hk * a.f.chunks;
  const cudaError_t e = cudaFuncSetAttribute(delta_grad_kernel<DK, DV, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // (not launch_after: the wait costs this kernel two more spilled registers, 570 us for 550)
  delta_grad_kernel<DK, DV, SHARED><<<items < 148 ? items : 148, kGradThreads, smem, stream>>>(a, items);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t grad(const GradArgs& a, int B, cudaStream_t stream) {
  return a.f.H == a.f.Hk ? grad_as<DK, DV, false>(a, B, stream) : grad_as<DK, DV, true>(a, B, stream);
}

// Segments of a sequence for both chains, by an estimate in us as in the forward pass
// (chain_segments): a chunk takes 2.6 forwards, 2.5 for dS alone and from 5.3 to 7.7
// backwards, the more CTAs run.  Both chains and all that segments add, 16 heads of
// 16384 tokens: 2153 us in one piece, 661 in six, 640 in eight, 817 in twelve; 2 heads
// of 4096: 518, 154 in eight, 142 in twelve; one head of 1536: 206, 91 in six.
int grad_segments(long long units, int chunks, long long join_ctas) {
  auto waves = [](long long ctas) { return (double)((ctas + 147) / 148); };
  auto chunk = [](long long ctas) { return 7.9 + 2.4 * (ctas < 148 ? ctas : 148) / 148; };    // forwards and backwards
  int best = 1;
  double least = 0.95 * waves(units) * (chunk(units) * chunks + 14);
  for (int g = 3; g <= 64 && g * 2 <= chunks; ++g) {
    const int per = (chunks + g - 1) / g;
    const double t = waves(units * (2 * g - 3)) * (2.3 * per + 6) + waves(units * (g - 1)) * (2.5 * per + 6) +
                     waves(units * g) * (chunk(units * g) * per + 14) + 3.2 * (g - 1) * waves(join_ctas) + 20;
    if (t < least) {
      least = t;
      best = g;
    }
  }
  return best;
}

// workspace: records, then the images and partial sums, each rounded up to 256 bytes
struct BackwardLayout {
  size_t rec, s0, u, f, ds, x, inner, hand, turn, seg_n, seg_x, seg_xt, seg_s, total;
  int segs, pieces;
  explicit BackwardLayout(const lte_gdr_dims* d) {
    const size_t units = (size_t)d->B * d->H, n = units * ((d->T + L - 1) / L), dv = d->dv, dk = d->dk;
    const int chunks = (d->T + L - 1) / L;
    segs = grad_segments((long long)units, chunks, (long long)(units * dv * dk / 1024));
    // (a chunk takes both chains 10 us together: a CTA's start and end cost less of one)
    pieces = segs > 1 ? 1 : chain_pieces((long long)units, chunks, 1.5, 2);
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += (bytes + 255) & ~(size_t)255; return r; };
    rec = take(n * rec_bytes(true));
    s0 = take(n * dv * dk * 4);
    u = take(n * dv * L * 4);
    f = take(n * dv * L * 2);
    ds = take(n * dv * dk * 2);
    x = take(n * (dv / 16) * 2 * L * 4);
    inner = take(n * (dv / 16) * 4);
    hand = take(pieces > 1 ? units * dv * dk * 4 : 0);
    turn = take(pieces > 1 ? piece_bytes(units) : 0);
    seg_n = take(segs > 1 ? units * (segs - 1) * dv * dk * 4 : 0);
    seg_x = take(segs > 1 ? units * (segs - 2) * dk * dk * 4 : 0);
    seg_xt = take(segs > 1 ? units * (segs - 2) * dk * dk * 4 : 0);
    seg_s = take(segs > 1 ? units * segs * dv * dk * 4 : 0);
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
  c.scale = d->scale; c.segs = w.segs; c.pieces = w.pieces; c.seg_chunks = (c.chunks + w.segs * w.pieces - 1) / (w.segs * w.pieces);
  c.a_lo = true; c.seg_n = (float*)(ws + w.seg_n); c.seg_x = (float*)(ws + w.seg_x);
  c.seg_xt = (float*)(ws + w.seg_xt); c.seg_s = (float*)(ws + w.seg_s);
  if (w.pieces > 1) c.s_out = n.hand = (float*)(ws + w.hand);
  c.turn = (int*)(ws + w.turn); c.done = c.turn + 2;
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
