// The backward chain of the gated delta rule on 5th-generation tensor cores
// (formulas: delta_backward.cu; layout and pipeline as in delta_chain_tc.cu).
//
// One CTA per (batch, value head) walks the chunks from the last to the first
// with dS in TMEM, lane = value channel:
//   X   = dO^T A                                   SS, A as hi + lo (columns s <= t)
//   P   = dS K^T                                   TS, dS as hi + lo
//   dU  = P diag(e^{G_L - G}) + X                  by threads; hi + lo over P
//   F   = dU T                                     TS; + b dU by threads; -e^G F as hi + lo over F
//   dS  = e^{G_L} dS + (scale e^G dO)^T Q - (e^G F)^T K     TS
// (all transposed: rows are value channels, columns tokens or key channels).
// Columns: dS (DK), dS hi, lo (DK / 2 each), P or dU (64), F (64), X, then F as
// fp32 (64), dO^T, then scale e^G dO^T as hi + lo (64).
//
// Warps 0-7 keep the chain.  8-11 scale dO, write the image of dS and take <dS, S>;
// 12-15 write dV and the image of F and take the sums over value channels u.F / b
// and v.F per token (the sums are what the gates' gradients need).  16 loads; 17
// issues the MMAs.
// The products of dO with Q run while the chain warps turn F, so the chain of a
// chunk is P -> dU -> F -> dS as in the forward pass.  Sequences of more heads than
// SMs are cut into pieces as there; dS goes from one to the next by `hand`.  Long
// sequences of few heads are cut into segments as there: dS goes back through a
// segment by the transpose of its X, so a first pass finds the chains from zero,
// the join carries them, and a second pass runs every segment from its dS.  64 chunks of 128 heads of
// 128 channels (one wave): 490 us, 7.6 us a chunk; 160 KB of images and dV
// per chunk beside 97 KB of inputs (2.1 GB, 4.3 TB/s) make memory latency the bound.
#include <math.h>

#include "delta_chain_tc.cuh"

namespace lte {
namespace delta {
namespace backtc {

using namespace chaintc;

constexpr int kThreads = 640;
// registers of a thread: warps 0-3, 4-7 (chain), 8-11 (dO, <dS, S>), 12-15 (F, dV), 16-19 (the rest)
constexpr int kChainRegs = 112, kStateRegs = 120, kValueRegs = 88, kRestRegs = 48;
static_assert(2 * kChainRegs + kStateRegs + kValueRegs + kRestRegs <= kThreads / 128 * launch_regs(kThreads), "registers");
// a stage: K, Q, dO, V (two halves each), the record's T hi, T lo, A hi, A lo, scalars
constexpr uint32_t kK = 0, kQ = 2 * kHalf, kD = 4 * kHalf, kV = 6 * kHalf, kR = 8 * kHalf;
constexpr uint32_t kScalOff = kR + 4 * kImg;
constexpr uint32_t kStage = (kScalOff + kGradScal + 1023) / 1024 * 1024;
// then the identity and the last 32 of 128 key channels of a state (128 rows, hi and lo)
constexpr uint32_t kIdent = 2 * kStage, kState = kIdent + kImg, kBars = kState + 2 * 128 * 64, kSmem = kBars + 256;
static_assert(kSmem <= 227 * 1024, "shared memory");

enum : int { bFull = 0, bEmpty = 2, bTail = 4, bSr = 5, bX = 7, bP = 8, bUr = 9, bF = 10, bFr = 11, bFx = 12, bXf = 13,
             bDr = 14, bS = 15, bSread = 17, bD = 18, bSt = 19, bStFree = 20, bDrain = 21, kBarCount = 22 };
constexpr uint32_t kColS = 0, kColP = 256, kColF = 320, kColX = 384, kColD = 448;

// z[j] summed over the warp's lanes; lane j gets the sum of z[j].  At each step
// a lane keeps half of its values and adds its partner's copy of them.
template <int N>
__device__ __forceinline__ void fold(float (&z)[32], int lane) {
  const bool upper = (lane & N) != 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float send = upper ? z[j] : z[j + N], keep = upper ? z[j + N] : z[j];
    z[j] = keep + __shfl_xor_sync(0xffffffffu, send, N);
  }
}
__device__ __forceinline__ float lane_sums(float (&z)[32], int lane) {
  fold<16>(z, lane);
  fold<8>(z, lane);
  fold<4>(z, lane);
  fold<2>(z, lane);
  fold<1>(z, lane);
  return z[0];
}
__device__ __forceinline__ float dot8(const uint4& h, const uint4& l, const float* x, float s) {
  const uint32_t a[4] = {h.x, h.y, h.z, h.w}, b[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s = fmaf(x[2 * e], bf_lo(a[e]) + bf_lo(b[e]), s);
    s = fmaf(x[2 * e + 1], bf_hi(a[e]) + bf_hi(b[e]), s);
  }
  return s;
}

// read once: not kept in what is left of the L1 cache
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// a unit whole, in pieces, in segments, or segments' chains of dS alone
enum : int { kWhole = 0, kPieces = 1, kSegments = 2, kSegState = 3 };

template <int DK, int DV, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
delta_back_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_dv, const GradArgs ga) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const ChunkArgs& a = ga.f;
  constexpr uint32_t kColSh = DK, kColSl = DK + DK / 2;
  constexpr int kHK = DK / 64, kHV = DV / 64, kStrips = DV / 16;
  constexpr bool PIECES = KIND == kPieces, STATE = KIND == kSegState, SEG = KIND == kSegments || STATE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t s0 = sa(sm), bars = s0 + kBars;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kBars + 8 * kBarCount);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kBars + 8 * kBarCount + 8);
  volatile int* ticket = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* flight = ticket + 1;                           // chunks and states requested; MMAs issued
  auto bar = [&](int i) { return bars + 8 * i; };

  if (tid == 0) {
    for (int i = 0; i < kBarCount; ++i) {
      const bool chain = i == bSr || i == bSr + 1 || i == bUr || i == bFr || i == bFx;     // 8 chain warps
      const bool out = i == bDr || i == bXf || i == bSread || i == bStFree;                                // one output group
      mbar_init(bar(i), i == bEmpty || i == bEmpty + 1 ? 17 : chain ? 8 : out ? 4 : 1);
    }
    *abort_flag = 0;
    if (PIECES) {
      after_previous();
      *ticket = atomicAdd(a.turn + 1, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  write_identity(sm + kIdent, kThreads);
  fence_proxy_async();
  if (warp == 17) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  after_previous();
  const uint32_t tmem = *tmem_slot;
  // the unit, and its chunks cb .. cb + n - 1 (pieces from the last to the first; dS alone of segments 1 on)
  const int units = PIECES ? gridDim.x / a.pieces : 1, per = STATE ? a.segs - 1 : SEG ? a.segs : 1;
  const int u = PIECES ? *ticket % units : (int)blockIdx.x / per;
  const int piece = PIECES ? *ticket / units : 0, seg = SEG ? (int)blockIdx.x % per + STATE : 0;
  const int cb = PIECES ? (a.pieces - 1 - piece) * a.seg_chunks : seg * a.seg_chunks;
  const int b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  const int len = seq_len(a.lens, b, a.T);
  const int n = PIECES || SEG ? min(max((len + L - 1) / L - cb, 0), a.seg_chunks) : (len + L - 1) / L;
  bool ok = true;

  if (warp >= 16) regs_dec<kRestRegs>();
  if (warp == 16) {
    // ================================================================ loads
    const uint8_t* recs = a.rec + (long long)u * a.chunks * rec_bytes(true);
    const int n_load = (unsigned)a.withhold < (unsigned)n ? a.withhold : n;
    int loaded = 0, states = 0;
    for (int i = 0; i < n_load; ++i) {
      const int s = i & 1, c = cb + n - 1 - i;
      if (i >= 2 && !(ok = wwait(bar(bEmpty + s), ((i >> 1) - 1) & 1, a.wait_ns, abort_flag))) break;
      const uint32_t d = s0 + s * kStage;
      const bool tail = c * L + L > len;                       // the first one to come
      const uint32_t fb = tail ? bar(bTail) : bar(bFull + s);
      if (elect_one()) {
        mbar_expect_tx(fb, (2 * kHK + (STATE ? 1 : 2) * kHV) * kHalf + 4 * kImg + kGradScal);
        for (int j = 0; j < kHK; ++j) {
          tma_load_4d(d + kK + j * kHalf, &tm_k, fb, 64 * j, hk, c * L, b);
          tma_load_4d(d + kQ + j * kHalf, &tm_q, fb, 64 * j, hk, c * L, b);
        }
        for (int j = 0; j < kHV; ++j) {
          tma_load_4d(d + kD + j * kHalf, &tm_d, fb, 64 * j, h, c * L, b);
          if (!STATE) tma_load_4d(d + kV + j * kHalf, &tm_v, fb, 64 * j, h, c * L, b);
        }
        bulk_load(d + kR, recs + (long long)c * rec_bytes(true), 4 * kImg + kGradScal, fb);
      }
      if (!STATE) {                                            // the images that the output warps read: to L2, a piece per lane
        const long long img = (long long)u * a.chunks + c;
        prefetch_l2(reinterpret_cast<const uint8_t*>(a.u + img * DV * L) + lane * (DV * L / 8), DV * L / 8);
        prefetch_l2(reinterpret_cast<const uint8_t*>(a.s0 + img * DV * DK) + lane * (DV * DK / 8), DV * DK / 8);
      }
      ++loaded;
      if (DK == 128 && !STATE && i > 0) {                      // the state of the chunk behind, key channels 96 on
        if (i > 1 && !(ok = wwait(bar(bStFree), i & 1, a.wait_ns, abort_flag))) break;
        if (lane == 0) mbar_expect_tx(bar(bSt), DV / 8 * 2 * 512);
        __syncwarp();
        const int rb = lane & 15, p = lane >> 4;               // a lane per eight rows of hi or lo
        if (rb < DV / 8)
          bulk_load(s0 + kState + p * (128 * 64) + rb * 512,
                    reinterpret_cast<const uint8_t*>(a.s0) + ((long long)u * a.chunks + c + 1) * (DV * DK * 4) + p * (DV * DK * 2) +
                        rb * (DK / 8) * 128 + 12 * 128, 512, bar(bSt));
        ++states;
      }
      if (tail) {
        if (!(ok = wwait(fb, 0, a.wait_ns, abort_flag))) break;
        const int r0 = len - c * L;
        uint8_t* st = sm + s * kStage;
        for (int j = 0; j < kHK; ++j) {
          zero_rows(st + kK + j * kHalf, r0, lane);
          zero_rows(st + kQ + j * kHalf, r0, lane);
        }
        for (int j = 0; j < kHV; ++j) {
          zero_rows(st + kD + j * kHalf, r0, lane);
          if (!STATE) zero_rows(st + kV + j * kHalf, r0, lane);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bFull + s));
      }
    }
    if (lane == 0) {
      flight[kFlightLoads] = loaded;
      flight[kFlightStates] = states;
    }
  } else if (warp == 17) {
    // ================================================================= MMAs
    const uint32_t id_tok = idesc2(128, L, false, false), id_dt = idesc2(128, L, true, false);
    const uint32_t id_s = idesc2(128, 64, false, true);
    const uint64_t ident = sdesc(s0 + kIdent, 16, 1024);
    int issued = 0;
    for (int i = 0; i < n; ++i) {
      const int s = i & 1, ph = i & 1;
      const uint32_t d = s0 + s * kStage;
      if (!(ok = wwait(bar(bFull + s), (i >> 1) & 1, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      issued = 1;
      const uint64_t dk = sdesc(d + kK, 16, 1024), dd = sdesc(d + kD, kHalf, 1024), dt = sdesc(d + kR, kHalf, 1024);
#pragma unroll
      for (int p = 0; p < 2; ++p) {                            // P = dS K^T, by halves of dS's columns
        if (ok) ok = wwait(bar(bSr + p), ph, a.wait_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < DK / 16; ++j) {
            const int ks = p * (DK / 32) + j / 2;
            mma_f16_ts(tmem + kColP, tmem + (j & 1 ? kColSl : kColSh) + 8 * ks, dk + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                       id_tok, p + j > 0);
          }
          if (p == 1) mma_commit(bar(bP));
        }
      }
      if (!ok) break;
      // (X's columns still hold the F of the chunk before until its sums have been taken)
      if (!STATE && i > 0 && !(ok = wwait(bar(bXf), (i - 1) & 1, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {                                       // X = dO^T A, and dO^T
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = L / 16 - 1; ks >= 0; --ks)
            mma_f16(tmem + kColX, dd + ((ks * 2048) >> 4), dt + (((2 + p) * kImg + ks * 2048) >> 4),
                    idesc2(128, 16 * (ks + 1), true, true), !(p == 0 && ks == L / 16 - 1));
        mma_commit(bar(bX));
#pragma unroll
        for (int ks = 0; ks < L / 16; ++ks)
          mma_f16(tmem + kColD, dd + ((ks * 2048) >> 4), ident + ((ks * 32) >> 4), id_dt, ks > 0);
        mma_commit(bar(bD));
      }
      if (!(ok = wwait(bar(bUr), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {                                       // F = dU T, columns s < 16 (ks + 1)
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int ks = L / 16 - 1; ks >= 0; --ks)
            mma_f16_ts(tmem + kColF, tmem + kColP + pair_col(ks, p == 1), dt + (((p == 2 ? kImg : 0) + ks * 2048) >> 4),
                       idesc2(128, 16 * (ks + 1), false, true), !(p == 0 && ks == L / 16 - 1));
        mma_commit(bar(bF));
      }
      if (!(ok = wwait(bar(bDr), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {                                       // dS += (scale e^G dO)^T Q
#pragma unroll
        for (int m = 0; m < kHK; ++m)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < L / 16; ++ks)
              mma_f16_ts(tmem + kColS + 64 * m, tmem + kColD + pair_col(ks, p),
                         sdesc(d + kQ + m * kHalf, kHalf, 1024) + ((ks * 2048) >> 4), id_s, 1u);
      }
      if (!(ok = wwait(bar(bFr), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {                                       // dS -= (e^G F)^T K, by halves of its columns
#pragma unroll
        for (int m = 0; m < kHK; ++m) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < L / 16; ++ks)
              mma_f16_ts(tmem + kColS + 64 * m, tmem + kColF + pair_col(ks, p),
                         sdesc(d + kK + m * kHalf, kHalf, 1024) + ((ks * 2048) >> 4), id_s, 1u);
          mma_commit(bar(bS + m));
        }
        if (kHK == 1) mma_commit(bar(bS + 1));
        if (i + 2 < n) mma_commit(bar(bEmpty + s));            // the stage is loaded once more
      }
    }
    if (lane == 0) flight[kFlightMma] = issued;
  } else if (warp < 8) {
    // ========================================================== chain warps
    regs_inc<kChainRegs>();
    constexpr int QC = DK / 4;
    const int row = (warp & 3) * 32 + lane, hc = warp >> 2;
    const uint32_t la = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const long long srow = ((long long)u * DV + (row < DV ? row : 0)) * DK;
    auto arrive = [&](int j) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(j));
    };
    {                                                          // the gradient behind, while the last chunk loads
      const bool later = PIECES && n > 0 && (cb + n) * L < len;
      if (later) ok = piece_ready(a.done + units + u, piece, a.wait_ns, abort_flag);
      const float* src = later ? ga.hand + srow : STATE && seg < a.segs - 1 ? nullptr : ga.ds_out;
      if (SEG && !STATE) src = a.seg_s + ((long long)u * a.segs + a.segs - 1 - seg) * DV * DK + (row < DV ? row : 0) * DK;
      else if (!later && src != nullptr) src += srow;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c0 = QC * (2 * p + hc);
        uint32_t r[QC];
#pragma unroll
        for (int e = 0; e < QC / 4; ++e) {
          const float4 v = src != nullptr && row < DV ? __ldcg(reinterpret_cast<const float4*>(src + c0 + 4 * e))
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
          r[4 * e] = __float_as_uint(v.x);
          r[4 * e + 1] = __float_as_uint(v.y);
          r[4 * e + 2] = __float_as_uint(v.z);
          r[4 * e + 3] = __float_as_uint(v.w);
        }
        tm_st(la + kColS + c0, r);
      }
      tmem_wait_st();
    }
    for (int i = 0; ok && i < n; ++i) {
      const int s = i & 1, ph = i & 1;
      if (!(ok = wwait(bar(bFull + s), (i >> 1) & 1, a.wait_ns, abort_flag))) break;
      const float* scal = reinterpret_cast<const float*>(sm + s * kStage + kScalOff);
      // ---- dS as bf16 hi and lo (columns QC (2 p + hc) .. + QC - 1)
      if (!STATE && i > 0 && !(ok = wwait(bar(bSread), (i - 1) & 1, a.wait_ns, abort_flag))) break;
      const float el = scal[kEG * L + L - 1];
      const uint64_t el2 = f2(el, el);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c0 = QC * (2 * p + hc);
        uint64_t S[QC / 2];
        if (i > 0 && ok) ok = wwait(bar(bS + p), (i - 1) & 1, a.wait_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        {
          uint32_t r[QC];
          tm_ld(la + kColS + c0, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < QC / 2; ++e) S[e] = pair_of(r + 2 * e);
        }
        {
          uint32_t hi[QC / 2], lo[QC / 2];
          split_pairs(S, hi, lo);
          tm_st(la + kColSh + c0 / 2, hi);
          tm_st(la + kColSl + c0 / 2, lo);
        }
        arrive(bSr + p);
        // e^{G_L} dS for this chunk's update (published with dU)
        uint32_t r[QC];
#pragma unroll
        for (int e = 0; e < QC / 2; ++e) {
          float x, y;
          unf2(mul2(S[e], el2), x, y);
          r[2 * e] = __float_as_uint(x);
          r[2 * e + 1] = __float_as_uint(y);
        }
        tm_st(la + kColS + c0, r);
      }
      if (!ok) break;
      // ---- dU = P diag(e^{G_L - G}) + X, tokens 32 hc .. + 31
      uint64_t U[16];
      if (!(ok = wwait(bar(bX), ph, a.wait_ns, abort_flag) && wwait(bar(bP), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {                          // 16 columns at a time
          uint32_t x[16], v[16];
          tmem_ld16(la + kColP + 32 * hc + 16 * q, x);
          tmem_ld16(la + kColX + 32 * hc + 16 * q, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 g = *reinterpret_cast<const float4*>(scal + kLam * L + 32 * hc + 16 * q + 4 * e);
            U[8 * q + 2 * e] = fma2(f2(g.x, g.y), pair_of(x + 4 * e), pair_of(v + 4 * e));
            U[8 * q + 2 * e + 1] = fma2(f2(g.z, g.w), pair_of(x + 4 * e + 2), pair_of(v + 4 * e + 2));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) split_pair(U[8 * q + e], hi[8 * q + e], lo[8 * q + e]);
        }
        tmem_st16(la + kColP + 32 * hc, hi);
        tmem_st16(la + kColP + 32 * hc + 16, lo);
      }
      arrive(bUr);
      // ---- F = dU T + b dU; first -e^G F as hi and lo, then F itself
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 g = *reinterpret_cast<const float4*>(scal + kBeta * L + 32 * hc + 4 * e);
        U[2 * e] = mul2(U[2 * e], f2(g.x, g.y));
        U[2 * e + 1] = mul2(U[2 * e + 1], f2(g.z, g.w));
      }
      if (!(ok = wwait(bar(bF), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      {
        uint32_t hi[16], lo[16];
        const uint64_t one = f2(1.f, 1.f);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t x[16];
          tmem_ld16(la + kColF + 32 * hc + 16 * q, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 g = *reinterpret_cast<const float4*>(scal + kEG * L + 32 * hc + 16 * q + 4 * e);
            const int f = 8 * q + 2 * e;
            U[f] = fma2(pair_of(x + 4 * e), one, U[f]);
            U[f + 1] = fma2(pair_of(x + 4 * e + 2), one, U[f + 1]);
            split_pair(mul2(U[f], f2(-g.x, -g.y)), hi[f], lo[f]);
            split_pair(mul2(U[f + 1], f2(-g.z, -g.w)), hi[f + 1], lo[f + 1]);
          }
        }
        tmem_st16(la + kColF + 32 * hc, hi);
        tmem_st16(la + kColF + 32 * hc + 16, lo);
        arrive(bFr);
        if (lane == 0) mbar_arrive(bar(bEmpty + s));           // the scalars have been read
        if (STATE) continue;
        uint32_t x[32];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float y, z;
          unf2(U[e], y, z);
          x[2 * e] = __float_as_uint(y);
          x[2 * e + 1] = __float_as_uint(z);
        }
        tmem_st32(la + kColX + 32 * hc, x);
        arrive(bFx);
      }
    }
    if (ok && n > 0) {
      ok = wwait(bar(bS), (n - 1) & 1, a.wait_ns, abort_flag) && wwait(bar(bS + 1), (n - 1) & 1, a.wait_ns, abort_flag);
      tc_fence_after();
    }
    float* dst = cb == 0 ? ga.ds_in : PIECES && n > 0 ? ga.hand : nullptr;
    if (STATE) dst = a.seg_n + ((long long)u * (a.segs - 1) + a.segs - 1 - seg) * DV * DK + (row < DV ? row : 0) * DK;
    else if (dst != nullptr) dst += srow;
    if (dst != nullptr) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c0 = QC * (2 * p + hc);
        uint32_t r[QC];
        tm_ld(la + kColS + c0, r);
        tmem_wait_ld();
        if (row < DV) {
#pragma unroll
          for (int e = 0; e < QC / 4; ++e) {
            float4 v = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                   __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
            if (!ok) v = make_float4(NAN, NAN, NAN, NAN);
            *reinterpret_cast<float4*>(dst + c0 + 4 * e) = v;
          }
        }
      }
      if (PIECES && cb > 0) piece_done(a.done + units + u, piece, ok, 2, 256);
    }
  } else if (warp < 16) {
    // ================================================= the two output groups
    const int quad = warp & 3, row = quad * 32 + lane;
    const bool mine = quad * 32 < DV;                          // a warp of value channels that exist
    const int rb = row >> 3, r7 = row & 7;
    const uint32_t la = tmem + ((uint32_t)(quad * 32) << 16);
    // this row's 16 bytes in column block 0 of the images of S_0, dS, U and F
    const int at_s = rb * (DK / 8) * 128 + r7 * 16, at_t = rb * (L / 8) * 128 + r7 * 16;
    const uint8_t* s_img = reinterpret_cast<const uint8_t*>(a.s0) + (long long)u * a.chunks * (DV * DK * 4) + at_s;
    if (warp < 12) {
      regs_inc<kStateRegs>();
      // ---- scale e^G dO, the image of dS, <dS, S>
      uint8_t* d_img = reinterpret_cast<uint8_t*>(ga.ds) + (long long)u * a.chunks * (DV * DK * 2) + at_s;
      constexpr int kAhead = 4, kPieces = DK == 128 ? 6 : DK / 16;   // (the others come to shared memory)
      auto put_inner = [&](int c, float s) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0 && mine) {                               // (the warp's second strip of 16: nothing)
          float* p = ga.inner + ((long long)u * a.chunks + c) * kStrips + 2 * quad;
          p[0] = s;
          p[1] = 0.f;
        }
      };
      for (int i = 0; i < n; ++i) {
        const int s = i & 1, ph = i & 1, c = cb + n - 1 - i;
        if (!(ok = wwait(bar(bFull + s), (i >> 1) & 1, a.wait_ns, abort_flag))) break;
        const float* scal = reinterpret_cast<const float*>(sm + s * kStage + kScalOff);
        // the state of the chunk behind, hi and lo, 16 key channels at a time, asked for
        // kAhead pieces ahead of their use: as much in flight as registers hold
        uint4 st[kAhead + 1][4];
        const bool inner = !STATE && mine && i > 0;
        auto fetch_state = [&](int j) {
          const uint8_t* p = s_img + (long long)(c + 1) * (DV * DK * 4) + j * 256;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            st[j % (kAhead + 1)][e] = load_once(p + e * 128);
            st[j % (kAhead + 1)][2 + e] = load_once(p + DV * DK * 2 + e * 128);
          }
        };
        if (inner)
#pragma unroll
          for (int j = 0; j < kAhead; ++j) fetch_state(j);
        // scale e^G dO^T as hi and lo
        if (!(ok = wwait(bar(bD), ph, a.wait_ns, abort_flag))) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {                        // 16 columns at a time
            uint32_t r[16];
            tmem_ld16(la + kColD + 32 * j + 16 * q, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 g = *reinterpret_cast<const float4*>(scal + kEG * L + 32 * j + 16 * q + 4 * e);
              split_pair(mul2(pair_of(r + 4 * e), f2(a.scale * g.x, a.scale * g.y)), hi[8 * q + 2 * e], lo[8 * q + 2 * e]);
              split_pair(mul2(pair_of(r + 4 * e + 2), f2(a.scale * g.z, a.scale * g.w)), hi[8 * q + 2 * e + 1], lo[8 * q + 2 * e + 1]);
            }
          }
          tmem_st16(la + kColD + 32 * j, hi);
          tmem_st16(la + kColD + 32 * j + 16, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bDr));
          mbar_arrive(bar(bEmpty + s));
        }
        if (STATE) continue;
        // dS: its image (hi), and <dS, S_0> with the state of the chunk behind
        if (!(ok = wwait(bar(bSr), ph, a.wait_ns, abort_flag) && wwait(bar(bSr + 1), ph, a.wait_ns, abort_flag))) break;
        tc_fence_after();
        float in = 0.f;
        uint8_t* im = d_img + (long long)c * (DV * DK * 2);
#pragma unroll
        for (int j = 0; j < DK / 16; ++j) {                    // 16 key channels: 8 words each of hi and lo
          uint32_t hi[8], lo[8];
          if (inner && j + kAhead < kPieces) fetch_state(j + kAhead);
          tm_ld(la + kColSh + 8 * j, hi);
          tm_ld(la + kColSl + 8 * j, lo);
          tmem_wait_ld();
          if (j == DK / 16 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bSread));
          }
          if (mine) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(im + (2 * j + e) * 128) = make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
          }
          if (j == kPieces && i > 0 && ok) ok = wwait(bar(bSt), (i - 1) & 1, a.wait_ns, abort_flag);
          if (inner) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x[8];
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                x[2 * f] = bf_lo(hi[4 * e + f]) + bf_lo(lo[4 * e + f]);
                x[2 * f + 1] = bf_hi(hi[4 * e + f]) + bf_hi(lo[4 * e + f]);
              }
              if (j < kPieces) {
                in = dot8(st[j % (kAhead + 1)][e], st[j % (kAhead + 1)][2 + e], x, in);
              } else {
                const uint8_t* p = sm + kState + rb * 512 + (2 * (j - kPieces) + e) * 128 + r7 * 16;
                in = dot8(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 128 * 64), x, in);
              }
            }
          }
        }
        if (DK == 128 && i > 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bStFree));
        }
        if (!ok) break;
        if (i > 0) put_inner(c + 1, in);
      }
      // the gradient of the (piece's) initial state with that state
      if (!STATE && ok && n > 0 && wwait(bar(bS), (n - 1) & 1, a.wait_ns, abort_flag) &&
          wwait(bar(bS + 1), (n - 1) & 1, a.wait_ns, abort_flag)) {
        tc_fence_after();
        float in = 0.f;
#pragma unroll
        for (int j = 0; j < DK / 16; ++j) {
          uint32_t r[16];
          tmem_ld16(la + kColS + 16 * j, r);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x[8];
#pragma unroll
              for (int f = 0; f < 8; ++f) x[f] = __uint_as_float(r[8 * e + f]);
              if (cb > 0)                                      // as the next chunk of the piece would see it
#pragma unroll
                for (int f = 0; f < 8; f += 2) {
                  uint32_t hi, lo;
                  split_pair(f2(x[f], x[f + 1]), hi, lo);
                  x[f] = bf_lo(hi) + bf_lo(lo);
                  x[f + 1] = bf_hi(hi) + bf_hi(lo);
                }
              const uint8_t* p = s_img + (long long)cb * (DV * DK * 4) + (2 * j + e) * 128;
              in = dot8(load_once(p), load_once(p + DV * DK * 2), x, in);
            }
          }
        }
        put_inner(cb, in);
      }
    } else {
      regs_dec<kValueRegs>();
      // ---- F: image, dV, u.F / b and v.F per token
      const uint8_t* u_img = reinterpret_cast<const uint8_t*>(a.u) + (long long)u * a.chunks * (DV * L * 4) + at_t;
      uint8_t* f_img = reinterpret_cast<uint8_t*>(ga.fimg) + (long long)u * a.chunks * (DV * L * 2) + at_t;
      __nv_bfloat16* dvp = ga.dv + ((long long)b * a.T * a.H + h) * DV;
      const uint32_t colv = (uint32_t)(row >> 6) * kHalf + (row & 7) * 2;
      const int cv = (row & 63) >> 3;
      for (int i = 0; i < n; ++i) {
        const int s = i & 1, ph = i & 1, c = cb + n - 1 - i;
        const long long img = (long long)u * a.chunks + c;
        // (a warp whose wait gave up still meets the others at the vote below)
        ok = wwait(bar(bFull + s), (i >> 1) & 1, a.wait_ns, abort_flag);
        if (STATE) {
          if (!ok) break;
          if (lane == 0) mbar_arrive(bar(bEmpty + s));
          continue;
        }
        const float* scal = reinterpret_cast<const float*>(sm + s * kStage + kScalOff);
        uint4 uw[2][4];
        auto fetch_u = [&](int j) {                            // 16 tokens, hi and lo
          const uint8_t* p = u_img + (long long)c * (DV * L * 4) + j * 256;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uw[j & 1][e] = load_once(p + e * 128);
            uw[j & 1][2 + e] = load_once(p + DV * L * 2 + e * 128);
          }
        };
        if (mine) fetch_u(0);
        ok = ok && wwait(bar(bFx), ph, a.wait_ns, abort_flag);
        tc_fence_after();
        if (!(ok = bar_and(1, 128, ok))) break;
        uint8_t* im = f_img + (long long)c * (DV * L * 2);
        float* xp = ga.x + (img * kStrips + 2 * quad) * (2 * L);
#pragma unroll
        for (int j = 0; j < 4; ++j) {                          // 16 tokens
          uint32_t F[16];
          if (mine && j < 3) fetch_u(j + 1);
          tmem_ld16(la + kColX + 16 * j, F);
          tmem_wait_ld();
          if (j == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bXf));
          }
          if (mine) {
            float z[32];                                       // 16 products with u, 16 with v
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 h4 = uw[j & 1][e], l4 = uw[j & 1][2 + e];
              const uint32_t wh[4] = {h4.x, h4.y, h4.z, h4.w}, wl[4] = {l4.x, l4.y, l4.z, l4.w};
              uint32_t w[4];
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const int k = 8 * e + 2 * f, t = 16 * j + k;
                const float f0 = __uint_as_float(F[k]), f1 = __uint_as_float(F[k + 1]);
                const uint32_t a0 = colv + t * 128 + ((cv ^ (t & 7)) << 4), a1 = colv + (t + 1) * 128 + ((cv ^ ((t + 1) & 7)) << 4);
                const uint32_t v0 = *reinterpret_cast<const uint16_t*>(sm + s * kStage + kV + a0);
                const uint32_t v1 = *reinterpret_cast<const uint16_t*>(sm + s * kStage + kV + a1);
                const float2 ib = *reinterpret_cast<const float2*>(scal + kInvB * L + t);
                z[k] = (f0 * ib.x) * (bf_lo(wh[f]) + bf_lo(wl[f]));
                z[k + 1] = (f1 * ib.y) * (bf_hi(wh[f]) + bf_hi(wl[f]));
                z[16 + k] = f0 * bf_lo(v0);
                z[17 + k] = f1 * bf_lo(v1);
                w[f] = pack_bf16(f0, f1);
                // dV takes V's place (each thread its own channel), from where it is stored
                *reinterpret_cast<uint16_t*>(sm + s * kStage + kV + a0) = (uint16_t)(w[f] & 0xffff);
                *reinterpret_cast<uint16_t*>(sm + s * kStage + kV + a1) = (uint16_t)(w[f] >> 16);
              }
              *reinterpret_cast<uint4*>(im + (2 * j + e) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            const float sum = lane_sums(z, lane);              // lanes 0-15: u.F / b, 16-31: v.F of token lane mod 16
            const int t = 16 * j + (lane & 15);
            xp[(lane >> 4) * L + t] = sum;
            xp[2 * L + (lane >> 4) * L + t] = 0.f;             // the warp's second strip of 16
          }
        }
        const int nt = len - c * L;
        if (nt >= L) {
          fence_proxy_async();
          bar_sync(1, 128);
          if (tid == 384) {
            for (int j = 0; j < kHV; ++j) tma_store_4d(&tm_dv, s0 + s * kStage + kV + j * kHalf, 64 * j, h, c * L, b);
            bulk_commit();
            bulk_wait_read();
          }
        } else {
          bar_sync(1, 128);
          for (int j = tid - 384; j < nt * (DV / 8); j += 128) {
            const int t = j / (DV / 8), cc = j % (DV / 8);
            *reinterpret_cast<uint4*>(dvp + (long long)(c * L + t) * a.H * DV + cc * 8) =
                *reinterpret_cast<const uint4*>(sm + s * kStage + kV + (cc >> 3) * kHalf + t * 128 + (((cc & 7) ^ (t & 7)) << 4));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bEmpty + s));           // V, dV and the scalars have been read
      }
    }
  }
  if (tid == 384) bulk_wait_read();                            // output stores have left shared memory
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {                                           // a wait gave up: as in the forward chain
    const int id = PIECES ? *ticket : block_again(), units = PIECES ? gridDim.x / a.pieces : 1;
    const int per = STATE ? a.segs - 1 : SEG ? a.segs : 1, u = PIECES ? id % units : id / per;
    const int cb = PIECES ? (a.pieces - 1 - id / units) * a.seg_chunks : SEG ? (id % per + STATE) * a.seg_chunks : 0;
    const int b = u / a.H, h = u % a.H, len = seq_len(a.lens, b, a.T);
    const int n = PIECES || SEG ? min(max((len + L - 1) / L - cb, 0), a.seg_chunks) : (len + L - 1) / L;
    if (warp == 17 && flight[kFlightMma]) {
      if (elect_one()) mma_commit(bar(bDrain));
      __syncwarp();
      mbar_drain(bar(bDrain), 0);
    }
    if (warp == 16) {
      for (int m = flight[kFlightLoads], i = max(m - 2, 0); i < m; ++i)
        if ((cb + n - 1 - i) * L + L <= len) mbar_drain(bar(bFull + (i & 1)), (i >> 1) & 1);
        else mbar_drain(bar(bTail), 0);
      if (flight[kFlightStates] > 0) mbar_drain(bar(bSt), (flight[kFlightStates] - 1) & 1);
    }
    if (tid == 384) bulk_wait_all();
    __syncthreads();
    if (!STATE) {
      const long long t0 = (long long)cb * L;
      nan_rows<DV>(ga.dv + ((b * (long long)a.T + t0) * a.H + h) * DV, (long long)a.H * DV, min(len - cb * L, n * L), tid, kThreads);
      nan_records(a.rec + ((long long)u * a.chunks + cb) * rec_bytes(true), n, kThreads);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 17)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int DK, int DV, int KIND>
cudaError_t launch_as(const CUtensorMap* m, const GradArgs& args, int B, cudaStream_t stream) {
  GradArgs a = args;
  set_waits(a.f, KIND == kSegState ? LTE_GDR_LAUNCH_BACK_SEGMENTS : LTE_GDR_LAUNCH_BACK);
  const int per = KIND == kSegState ? a.f.segs - 1 : a.f.segs * a.f.pieces;
  return launch_after(delta_back_tc_kernel<DK, DV, KIND>, (unsigned)(B * a.f.H * per), kThreads, kSmem, stream, m[0], m[1], m[2],
                      m[3], m[4], a);
}
template <int DK, int DV>
cudaError_t launch(const CUtensorMap* m, const GradArgs& a, int B, cudaStream_t stream) {
  if (a.f.segs > 1) {
    cudaError_t e = launch_as<DK, DV, kSegState>(m, a, B, stream);
    if (e == cudaSuccess) e = join_states(a.f, a.ds_out, true, B, DK, stream);
    return e == cudaSuccess ? launch_as<DK, DV, kSegments>(m, a, B, stream) : e;
  }
  return a.f.pieces > 1 ? launch_as<DK, DV, kPieces>(m, a, B, stream) : launch_as<DK, DV, kWhole>(m, a, B, stream);
}

}  // namespace backtc

cudaError_t back_chain(const GradArgs& g, int B, int dk, cudaStream_t stream) {
  using namespace backtc;
  const ChunkArgs& a = g.f;
  CUtensorMap m[5];
  const Strides4 out{(long long)a.T * a.H * a.dv, (long long)a.H * a.dv, a.dv};
  if (!map_of(&m[0], a.q, dk, a.Hk, a.T, B, a.qs) || !map_of(&m[1], a.k, dk, a.Hk, a.T, B, a.ks) ||
      !map_of(&m[2], g.dO, a.dv, a.H, a.T, B, g.dos) || !map_of(&m[3], a.v, a.dv, a.H, a.T, B, a.vs) ||
      !map_of(&m[4], g.dv, a.dv, a.H, a.T, B, out))
    return cudaErrorNotSupported;
  if (dk == 128) return a.dv == 128 ? launch<128, 128>(m, g, B, stream) : launch<128, 64>(m, g, B, stream);
  return a.dv == 128 ? launch<64, 128>(m, g, B, stream) : launch<64, 64>(m, g, B, stream);
}

}  // namespace delta
}  // namespace lte
