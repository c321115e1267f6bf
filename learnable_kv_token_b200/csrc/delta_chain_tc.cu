// The forward chain of states of the gated delta rule on 5th-generation tensor
// cores (formulas and precision: delta_chunk.cuh).
//
// One CTA per (batch, value head) walks the chunks.  The state lives in TMEM,
// lane = value channel, for the whole sequence, and every product is kept
// transposed (value channels = the MMA's 128 rows), so each result is turned
// into the A operand of the next where it lies:
//   P^T = S K^T            TS, S as bf16 hi + lo
//   R^T = V^T - P^T diag(e^G)         by threads; hi + lo over P's columns
//   U^T = R^T T^T          TS; + b R^T by threads
//   S   = e^{G_L} S + (U diag(e^{G_L - G}))^T K     TS, hi + lo over U's columns
//   O^T = scale S Q^T diag(e^G) + U^T A^T           TS, beside the chain
// V^T comes to TMEM as fp32 by one product with an identity.  Columns: S (DK),
// S hi, S lo (DK / 2 each), P or R (64), V or U (64), U hi, U lo (32 each), O (64).
//
// Warps: 0-7 turn S, R and U (two threads per value channel, each with half of
// the columns: chain warps); 8-11 finish O (or, for the gradients, write the
// images of S and U); 12 loads (TMA for K, Q and V, bulk copies for the record;
// two stages); 13 issues the MMAs.
// What bounds a chunk is the chain P -> R -> U -> S, so everything else is kept
// off it: a pass publishes what the next product needs before it does the rest
// (e^{G_L} S, U for O); S comes and goes in two halves of its columns, so a pass
// over one half runs beside the product on the other; products with T and A
// leave out the columns above the diagonal.  64 chunks of 512 heads of 128
// channels: 672 us (seven waves of half sequences; 660 without A's lo), 4400 cycles a chunk, 1300 of
// them products; 3.0 GB moved, 4.5 TB/s, which two stages of loads cover.
//
// Long sequences of few heads are cut into segments of chunks, one CTA each.  A
// row of S goes through a segment by an affine map s -> s X + n that is the same
// X for every row, so a first pass finds, for all segments at once, n (the chain
// from a zero state) and X (the chain from the identity with no values); a small
// kernel carries the states from segment to segment, and a second pass runs every
// segment from its state for O.  Twice the work on many times the SMs.
//
// With more heads than SMs, sequences are cut into pieces that follow one another,
// one CTA each, so that the last wave of CTAs is short.  A piece starts from the
// state that the one before left in s_out.  CTAs draw their pieces in order, all
// first ones before all second ones: what a CTA waits for was drawn before by one
// that is running or done, so the wait ends, and as a rule is over already.
//
// Rows of the last chunk behind the sequence's length are set to zero in shared
// memory before use, so what lies there (NaN, another sequence) does not enter.
// Every wait is bounded; what a CTA that gives up has not finished is NaN: its state (or
// n, X), its rows of o, or, for the gradients, its chunks' records, and with them all
// that is made of those.
#include <math.h>

#include "delta_chain_tc.cuh"

namespace lte {
namespace delta {
namespace chaintc {

constexpr int kThreads = 512;
// registers of a thread: warps 0-3, 4-7 (chain), 8-11 (O), 12-15 (the rest)
constexpr int kChainRegs = 144, kOutRegs = 144, kRestRegs = 80;
static_assert(2 * kChainRegs + kOutRegs + kRestRegs <= kThreads / 128 * launch_regs(kThreads), "registers");
// a stage: K, Q, V (two halves each), then T hi, T lo, A, scalars as in the record
constexpr uint32_t kK = 0, kQ = 2 * kHalf, kV = 4 * kHalf, kR = 6 * kHalf;
constexpr uint32_t kScalOff = kR + 3 * kImg;
constexpr uint32_t kStage = (kScalOff + kScal + 1023) / 1024 * 1024;
// then the identity and a chunk of O as token rows (two halves)
constexpr uint32_t kIdent = 2 * kStage, kOut = kIdent + kImg, kBars = kOut + 2 * kHalf, kSmem = kBars + 256;
static_assert(kSmem <= 227 * 1024, "shared memory");

// mbarriers; those without [] complete once per chunk
enum : int { bFull = 0, bEmpty = 2, bTail = 4, bSr = 5, bP = 7, bRr = 8, bU = 9, bUr = 10, bUh = 11, bS = 12, bQS = 14,
             bOs = 15, bO = 16, bOf = 17, bSread = 18, bUread = 19, bDrain = 20, kBarCount = 21 };
// columns; R and the scaled U lie over P and U (pair_col)
constexpr uint32_t kColS = 0, kColPR = 256, kColVU = 320, kColUH = 384, kColUL = 416, kColO = 448;

// what a chain leaves besides the state
enum : int { kImages = 0, kO = 1, kStateOnly = 2 };

template <int DK, int DV, int KIND, bool PIECES>
__global__ void __launch_bounds__(kThreads, 1)
delta_chain_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                      const ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  constexpr uint32_t kColSh = DK, kColSl = DK + DK / 2;
  constexpr int kHK = DK / 64, kHV = DV / 64;                // 64-channel halves
  constexpr bool OUT = KIND == kO;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t s0 = sa(sm), bars = s0 + kBars;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kBars + 8 * kBarCount);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kBars + 8 * kBarCount + 8);
  volatile int* ticket = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* flight = ticket + 1;                         // chunks requested; MMAs issued
  auto bar = [&](int i) { return bars + 8 * i; };
  const bool a_lo = KIND == kImages || (KIND == kStateOnly && a.a_lo);      // the records hold A's lo

  if (tid == 0) {
    for (int i = 0; i < kBarCount; ++i) {
      const bool chain = i == bSr || i == bSr + 1 || i == bRr || i == bUr || i == bUh;      // 8 chain warps
      const bool out = i == bOs || i == bOf || i == bSread || i == bUread;                  // 4 output warps
      mbar_init(bar(i), i == bEmpty || i == bEmpty + 1 ? 13 : chain ? 8 : out ? 4 : 1);
    }
    *abort_flag = 0;
    if (PIECES) {
      after_previous();
      *ticket = atomicAdd(a.turn, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  write_identity(sm + kIdent, kThreads);
  fence_proxy_async();
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  after_previous();
  const uint32_t tmem = *tmem_slot;
  // the unit's segment: for kStateOnly first n of segments 0 .. G - 2, then X of 1 .. G - 2;
  // or its piece, all first pieces before all second ones
  auto unit_of = [&](int i, int& u, int& seg) {
    const int per = KIND == kStateOnly ? 2 * a.segs - 3 : a.segs;
    const int units = PIECES ? gridDim.x / a.pieces : 1;
    u = PIECES ? i % units : i / per;
    seg = PIECES ? i / units : i % per;
    const bool hom = KIND == kStateOnly && seg >= a.segs - 1;
    if (hom) seg -= a.segs - 2;
    return hom;
  };
  auto unit_seg = [&](int& u, int& seg) { return unit_of(PIECES ? *ticket : (int)blockIdx.x, u, seg); };
  int u, seg;
  const bool hom = unit_seg(u, seg);
  const int b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  // chunks cb .. cb + n_chunks - 1 of the sequence; `len` tokens from chunk cb on
  const int cb = seg * a.seg_chunks;
  const int len = max(seq_len(a.lens, b, a.T) - cb * L, 0);
  const int n_chunks = min((len + L - 1) / L, a.seg_chunks);
  bool ok = true;

  if (warp >= 12) regs_dec<kRestRegs>();
  if (warp == 12) {
    // ================================================================ loads
    const uint8_t* recs = a.rec + ((long long)u * a.chunks + cb) * rec_bytes(a_lo);
    const int n_load = (unsigned)a.withhold < (unsigned)n_chunks ? a.withhold : n_chunks;
    int loaded = 0;
    for (int c = 0; c < n_load; ++c) {
      const int s = c & 1;
      if (c >= 2 && !(ok = wwait(bar(bEmpty + s), ((c >> 1) - 1) & 1, a.wait_ns, abort_flag))) break;
      const uint32_t d = s0 + s * kStage;
      const bool tail = c * L + L > len;
      const uint32_t fb = tail ? bar(bTail) : bar(bFull + s);
      if (elect_one()) {
        const uint8_t* r = recs + (long long)c * rec_bytes(a_lo);
        mbar_expect_tx(fb, (OUT ? 2 * kHK + kHV : kHK + kHV) * kHalf + (OUT ? 3 : 2) * kImg + kScal);
        for (int i = 0; i < kHK; ++i) {
          tma_load_4d(d + kK + i * kHalf, &tm_k, fb, 64 * i, hk, (cb + c) * L, b);
          if (OUT) tma_load_4d(d + kQ + i * kHalf, &tm_q, fb, 64 * i, hk, (cb + c) * L, b);
        }
        for (int i = 0; i < kHV; ++i) tma_load_4d(d + kV + i * kHalf, &tm_v, fb, 64 * i, h, (cb + c) * L, b);
        if (OUT) {
          bulk_load(d + kR, r, 3 * kImg + kScal, fb);
        } else {
          bulk_load(d + kR, r, 2 * kImg, fb);
          bulk_load(d + kScalOff, r + (a_lo ? 4 : 3) * kImg, kScal, fb);
        }
      }
      ++loaded;
      if (tail) {                                            // the last chunk: zeros behind the sequence
        if (!(ok = wwait(fb, 0, a.wait_ns, abort_flag))) break;
        const int r0 = len - c * L;
        for (int j = 0; j < kHK; ++j) zero_rows(sm + s * kStage + kK + j * kHalf, r0, lane);
        for (int j = 0; j < kHV; ++j) zero_rows(sm + s * kStage + kV + j * kHalf, r0, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bFull + s));
      }
    }
    if (lane == 0) flight[kFlightLoads] = loaded;
  } else if (warp == 13) {
    // ================================================================= MMAs
    const uint32_t id_tok = idesc2(128, L, false, false);      // N = tokens, B [n][k]
    const uint32_t id_vt = idesc2(128, L, true, false);        // V^T from [token][channel]
    const uint32_t id_s = idesc2(128, 64, false, true);        // N = 64 key channels, B [k][n]
    const uint64_t ident = sdesc(s0 + kIdent, 16, 1024);
    int issued = 0;
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c & 1, ph = c & 1;
      const uint32_t d = s0 + s * kStage;
      if (!(ok = wwait(bar(bFull + s), (c >> 1) & 1, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      issued = 1;
      const uint64_t dk = sdesc(d + kK, 16, 1024), dq = sdesc(d + kQ, 16, 1024), dt = sdesc(d + kR, 16, 1024);
      if (elect_one()) {                                       // V^T
        const uint64_t dv = sdesc(d + kV, kHalf, 1024);
#pragma unroll
        for (int ks = 0; ks < L / 16; ++ks)
          mma_f16(tmem + kColVU, dv + ((ks * 2048) >> 4), ident + ((ks * 32) >> 4), id_vt, ks > 0);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {                            // P^T = S K^T, by halves of S's columns
        if (ok) ok = wwait(bar(bSr + p), ph, a.wait_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < DK / 16; ++i) {
            const int ks = p * (DK / 32) + i / 2;
            mma_f16_ts(tmem + kColPR, tmem + (i & 1 ? kColSl : kColSh) + 8 * ks, dk + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                       id_tok, p + i > 0);
          }
          if (p == 1) mma_commit(bar(bP));
        }
      }
      if (!ok) break;
      if (OUT) {                                               // S Q^T
        if (c > 0 && !(ok = wwait(bar(bOf), (c - 1) & 1, a.wait_ns, abort_flag))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
              mma_f16_ts(tmem + kColO, tmem + (p ? kColSl : kColSh) + 8 * ks, dq + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                         id_tok, p + ks > 0);
          mma_commit(bar(bQS));
        }
      }
      if (!(ok = wwait(bar(bRr), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {                                       // U^T = R^T T^T: columns t >= 16 ks
#pragma unroll
        for (int p = 0; p < 3; ++p)                            // hi hi, lo hi, hi lo
#pragma unroll
          for (int ks = 0; ks < L / 16; ++ks)
            mma_f16_ts(tmem + kColVU + 16 * ks, tmem + kColPR + pair_col(ks, p == 1),
                       dt + (((p == 2 ? kImg : 0) + ks * (16 * 128 + 32)) >> 4), idesc2(128, L - 16 * ks, false, false),
                       p + ks > 0);
        mma_commit(bar(bU));
      }
      if (!(ok = wwait(bar(bUr), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {                                       // S += (U diag(e^{G_L - G}))^T K, by halves of its columns
        constexpr int kN = DK == 128 ? 2 : 1;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const uint64_t dkn = sdesc(d + kK + n * kHalf, kHalf, 1024);
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < L / 16; ++ks)
              mma_f16_ts(tmem + kColS + 64 * n, tmem + kColVU + pair_col(ks, p), dkn + ((ks * 2048) >> 4), id_s, 1u);
          mma_commit(bar(bS + n));
        }
        if (kN == 1) mma_commit(bar(bS + 1));
      }
      if (OUT) {                                               // O^T += U^T A^T, columns t >= 16 ks
        if (!(ok = wwait(bar(bUh), ph, a.wait_ns, abort_flag))) break;
        if (!(ok = wwait(bar(bOs), ph, a.wait_ns, abort_flag))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < L / 16; ++ks)
              mma_f16_ts(tmem + kColO + 16 * ks, tmem + (p ? kColUL : kColUH) + 8 * ks,
                         dt + ((2 * kImg + ks * (16 * 128 + 32)) >> 4), idesc2(128, L - 16 * ks, false, false), 1u);
          // U hi with A's lo, from where prepare put its columns of blocks
#pragma unroll
          for (int ks = 1; ks < L / 16; ++ks)
            mma_f16_ts(tmem + kColO + 16 * ks, tmem + kColUH + 8 * ks, dt + ((2 * kImg + (4 - ks) * 32) >> 4),
                       idesc2(128, L - 16 * ks, false, false), 1u);
          mma_f16_ts(tmem + kColO, tmem + kColUH, dt + ((kImg + 2 * 32) >> 4), idesc2(128, 16, false, false), 1u);
          mma_f16_ts(tmem + kColO + 16, tmem + kColUH, dt + ((kImg + 3 * 32) >> 4), idesc2(128, L - 16, false, false), 1u);
          mma_commit(bar(bO));
        }
      }
      if (c + 2 < n_chunks && elect_one()) mma_commit(bar(bEmpty + s));   // the stage is loaded once more
    }
    if (lane == 0) flight[kFlightMma] = issued;
  } else if (warp < 8) {
    // ========================================================== chain warps
    regs_inc<kChainRegs>();
    constexpr int QC = DK / 4;                                 // S columns per thread and half
    const int row = (warp & 3) * 32 + lane, hc = warp >> 2;    // value channel = TMEM lane; which columns
    const uint32_t la = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int rows = hom ? DK : DV;
    {                                                          // the state, while the first chunk loads
      const bool joined = KIND != kStateOnly && a.segs > 1;            // (s_out may be s_in: that was read by the join)
      const float* src = joined ? a.seg_s + seg * DV * DK : seg == 0 ? a.s_in : PIECES ? a.s_out : nullptr;
      if (PIECES && seg > 0 && n_chunks > 0) ok = piece_ready(a.done + u, seg, a.wait_ns, abort_flag);
      if (src != nullptr) src += (long long)u * (joined ? a.segs : 1) * DV * DK + row * DK;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c0 = QC * (2 * p + hc);
        uint32_t r[QC];
#pragma unroll
        for (int e = 0; e < QC / 4; ++e) {
          const int col = c0 + 4 * e;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (hom) v = make_float4(col == row, col + 1 == row, col + 2 == row, col + 3 == row);
          else if (src != nullptr && row < DV) v = __ldcg(reinterpret_cast<const float4*>(src + col));
          r[4 * e] = __float_as_uint(v.x);
          r[4 * e + 1] = __float_as_uint(v.y);
          r[4 * e + 2] = __float_as_uint(v.z);
          r[4 * e + 3] = __float_as_uint(v.w);
        }
        tm_st(la + kColS + c0, r);
      }
      tmem_wait_st();
    }
    auto arrive = [&](int i) {                                 // this warp's TMEM writes are done
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    for (int c = 0; ok && c < n_chunks; ++c) {
      const int s = c & 1, ph = c & 1;
      if (!(ok = wwait(bar(bFull + s), (c >> 1) & 1, a.wait_ns, abort_flag))) break;
      const float* scal = reinterpret_cast<const float*>(sm + s * kStage + kScalOff);
      // ---- the state as bf16 hi and lo (columns QC (2 p + hc) .. + QC - 1)
      if (KIND == kImages && c > 0 && !(ok = wwait(bar(bSread), (c - 1) & 1, a.wait_ns, abort_flag))) break;
      uint64_t S[2][QC / 2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c0 = QC * (2 * p + hc);
        if (c > 0 && ok) ok = wwait(bar(bS + p), (c - 1) & 1, a.wait_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[QC];
        tm_ld(la + kColS + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < QC / 2; ++e) S[p][e] = pair_of(r + 2 * e);
        uint32_t hi[QC / 2], lo[QC / 2];
        split_pairs(S[p], hi, lo);
        tm_st(la + kColSh + c0 / 2, hi);
        tm_st(la + kColSl + c0 / 2, lo);
        arrive(bSr + p);
      }
      if (!ok) break;
      // ---- e^{G_L} S for this chunk's update (published with R)
      {
        const float el = scal[kEG * L + L - 1];
        const uint64_t el2 = f2(el, el);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t r[QC];
#pragma unroll
          for (int e = 0; e < QC / 2; ++e) {
            float x, y;
            unf2(mul2(S[p][e], el2), x, y);
            r[2 * e] = __float_as_uint(x);
            r[2 * e + 1] = __float_as_uint(y);
          }
          tm_st(la + kColS + QC * (2 * p + hc), r);
        }
      }
      // ---- R^T = V^T - P^T diag(e^G), tokens 32 hc .. + 31
      uint64_t gm[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 g = *reinterpret_cast<const float4*>(scal + kEG * L + 32 * hc + 4 * e);
        gm[2 * e] = f2(-g.x, -g.y);
        gm[2 * e + 1] = f2(-g.z, -g.w);
      }
      if (!(ok = wwait(bar(bP), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      uint64_t R[16];
      {
        uint32_t x[32], v[32], hi[16], lo[16];
        tmem_ld32(la + kColPR + 32 * hc, x);
        tmem_ld32(la + kColVU + 32 * hc, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          R[e] = KIND == kStateOnly && hom ? mul2(gm[e], pair_of(x + 2 * e)) : fma2(gm[e], pair_of(x + 2 * e), pair_of(v + 2 * e));
        split_pairs(R, hi, lo);
        tmem_st16(la + kColPR + 32 * hc, hi);
        tmem_st16(la + kColPR + 32 * hc + 16, lo);
      }
      arrive(bRr);
      // ---- U = T R + b R; first U diag(e^{G_L - G}) as hi and lo, then U
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 g = *reinterpret_cast<const float4*>(scal + kBeta * L + 32 * hc + 4 * e);
        R[2 * e] = mul2(R[2 * e], f2(g.x, g.y));
        R[2 * e + 1] = mul2(R[2 * e + 1], f2(g.z, g.w));
        const float4 l = *reinterpret_cast<const float4*>(scal + kLam * L + 32 * hc + 4 * e);
        gm[2 * e] = f2(l.x, l.y);
        gm[2 * e + 1] = f2(l.z, l.w);
      }
      if (lane == 0) mbar_arrive(bar(bEmpty + s));             // the scalars have been read
      if (!(ok = wwait(bar(bU), ph, a.wait_ns, abort_flag))) break;
      tc_fence_after();
      {
        uint32_t x[32], hi[16], lo[16];
        tmem_ld32(la + kColVU + 32 * hc, x);
        tmem_wait_ld();
        const uint64_t one = f2(1.f, 1.f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          R[e] = fma2(pair_of(x + 2 * e), one, R[e]);
          gm[e] = mul2(R[e], gm[e]);
        }
        split_pairs(gm, hi, lo);
        tmem_st16(la + kColVU + 32 * hc, hi);
        tmem_st16(la + kColVU + 32 * hc + 16, lo);
        arrive(bUr);
        if (KIND == kStateOnly) continue;
        split_pairs(R, hi, lo);
        if (KIND == kImages && c > 0 && !(ok = wwait(bar(bUread), (c - 1) & 1, a.wait_ns, abort_flag))) break;
        tmem_st16(la + kColUH + 16 * hc, hi);
        tmem_st16(la + kColUL + 16 * hc, lo);
        arrive(bUh);
      }
    }
    if (ok && n_chunks > 0) {
      ok = wwait(bar(bS), (n_chunks - 1) & 1, a.wait_ns, abort_flag) && wwait(bar(bS + 1), (n_chunks - 1) & 1, a.wait_ns, abort_flag);
      tc_fence_after();
    }
    int ul, segl;
    unit_seg(ul, segl);
    float* dst = KIND == kStateOnly ? (hom ? a.seg_x + ((long long)ul * (a.segs - 2) + segl - 1) * DK * DK
                                           : a.seg_n + ((long long)ul * (a.segs - 1) + segl) * DV * DK)
                 : a.s_out != nullptr && (PIECES ? segl == 0 || n_chunks > 0 : segl == a.segs - 1)
                     ? a.s_out + (long long)ul * DV * DK : nullptr;
    if (dst != nullptr) {
      dst += row * DK;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c0 = QC * (2 * p + hc);
        uint32_t r[QC];
        tm_ld(la + kColS + c0, r);
        tmem_wait_ld();
        if (row < rows) {
#pragma unroll
          for (int e = 0; e < QC / 4; ++e) {
            float4 v = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                   __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
            if (!ok) v = make_float4(NAN, NAN, NAN, NAN);
            *reinterpret_cast<float4*>(dst + c0 + 4 * e) = v;
            if (KIND == kStateOnly && hom && a.seg_xt != nullptr) {
              float* t = a.seg_xt + ((long long)ul * (a.segs - 2) + segl - 1) * DK * DK + (c0 + 4 * e) * DK + row;
              t[0] = v.x;
              t[DK] = v.y;
              t[2 * DK] = v.z;
              t[3 * DK] = v.w;
            }
          }
        }
      }
      if (PIECES && !piece_done(a.done + ul, segl, ok, 2, 256) && row < rows)
        for (int i = 0; i < DK / 8; ++i)
          *reinterpret_cast<float4*>(dst + QC * 2 * hc + 4 * i) = make_float4(NAN, NAN, NAN, NAN);
    }
  } else if (warp < 12) {
    // ==================================================== O, or the images
    regs_inc<kOutRegs>();
    const int quad = warp - 8, row = quad * 32 + lane;
    const uint32_t la = tmem + ((uint32_t)(quad * 32) << 16);
    int c = 0;
    for (; c < n_chunks; ++c) {
      const int s = c & 1, ph = c & 1;
      ok = wwait(bar(bFull + s), (c >> 1) & 1, a.wait_ns, abort_flag);
      if (!OUT && !ok) break;                                  // (O: the warps meet at the vote below)
      const float* scal = reinterpret_cast<const float*>(sm + s * kStage + kScalOff);
      const long long img = KIND == kImages ? (long long)u * a.chunks + cb + c : 0;
      if (KIND == kStateOnly) {
        if (lane == 0) mbar_arrive(bar(bEmpty + s));
      } else if (OUT) {
        ok = ok && wwait(bar(bQS), ph, a.wait_ns, abort_flag);
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t r[32];
          tmem_ld32(la + kColO + 32 * j, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(scal + kEG * L + 32 * j + e);
            r[e] = __float_as_uint(__uint_as_float(r[e]) * (a.scale * g.x));
            r[e + 1] = __float_as_uint(__uint_as_float(r[e + 1]) * (a.scale * g.y));
            r[e + 2] = __float_as_uint(__uint_as_float(r[e + 2]) * (a.scale * g.z));
            r[e + 3] = __float_as_uint(__uint_as_float(r[e + 3]) * (a.scale * g.w));
          }
          tmem_st32(la + kColO + 32 * j, r);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bEmpty + s));
          mbar_arrive(bar(bOs));
        }
        ok = ok && wwait(bar(bO), ph, a.wait_ns, abort_flag);
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(la + kColO, r[0]);
        tmem_ld32(la + kColO + 32, r[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bOf));
        // token rows in shared memory, then one TMA store per half; the last
        // chunk's rows behind the sequence are not written
        if (tid == 256) bulk_wait_read();                      // the chunk before has left the buffer
        if (!(ok = bar_and(1, 128, ok))) break;
        if (row < DV) {
          const uint32_t col = (uint32_t)(row >> 6) * kHalf + (row & 7) * 2;
          const int cc = (row & 63) >> 3;
#pragma unroll
          for (int t = 0; t < L; ++t)
            *reinterpret_cast<__nv_bfloat16*>(sm + kOut + col + t * 128 + ((cc ^ (t & 7)) << 4)) =
                __float2bfloat16_rn(__uint_as_float(r[t >> 5][t & 31]));
        }
        const int n = len - c * L;
        if (n >= L) {
          fence_proxy_async();
          bar_sync(1, 128);
          if (tid == 256) {
            int u, seg;                                        // (not kept in registers over the chunks)
            unit_seg(u, seg);
            const int b = u / a.H, h = u % a.H, cb = seg * a.seg_chunks;
            for (int i = 0; i < kHV; ++i) tma_store_4d(&tm_o, s0 + kOut + i * kHalf, 64 * i, h, (cb + c) * L, b);
            bulk_commit();
          }
        } else {
          bar_sync(1, 128);
          int u, seg;
          unit_seg(u, seg);
          const int cb = seg * a.seg_chunks;
          __nv_bfloat16* op = a.o + (u / a.H) * a.os.b + (u % a.H) * a.os.h;
          for (int i = tid - 256; i < n * (DV / 8); i += 128) {
            const int t = i / (DV / 8), cc = i % (DV / 8);
            *reinterpret_cast<uint4*>(op + (long long)((cb + c) * L + t) * a.os.t + cc * 8) =
                *reinterpret_cast<const uint4*>(sm + kOut + (cc >> 3) * kHalf + t * 128 + (((cc & 7) ^ (t & 7)) << 4));
          }
        }
      } else {
        if (lane == 0) mbar_arrive(bar(bEmpty + s));
        if (!(ok = wwait(bar(bSr), ph, a.wait_ns, abort_flag) && wwait(bar(bSr + 1), ph, a.wait_ns, abort_flag))) break;
        tc_fence_after();
        // images in 8 x 8 blocks: a row's 16 bytes of each column block
        const int rb = row >> 3, r7 = row & 7;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint8_t* im = reinterpret_cast<uint8_t*>(a.s0 + img * a.dv * DK + (long long)p * (DV * DK / 2));
#pragma unroll
          for (int j = 0; j < DK / 64; ++j) {
            uint32_t r[32];
            tmem_ld32(la + (p ? kColSl : kColSh) + 32 * j, r);
            tmem_wait_ld();
            if (row < DV)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(im + ((long long)rb * (DK / 8) + 8 * j + e) * 128 + r7 * 16) =
                    make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bSread));
        if (!(ok = wwait(bar(bUh), ph, a.wait_ns, abort_flag))) break;
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(la + kColUH, r[0]);
        tmem_ld32(la + kColUL, r[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bUread));
        if (row < DV)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint8_t* im = reinterpret_cast<uint8_t*>(a.u + img * a.dv * L + (long long)p * (DV * L / 2));
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(im + ((long long)rb * (L / 8) + e) * 128 + r7 * 16) =
                  make_uint4(r[p][4 * e], r[p][4 * e + 1], r[p][4 * e + 2], r[p][4 * e + 3]);
          }
      }
    }
    if (OUT && !ok) {                                          // the rows from this chunk on
      int u, seg;
      unit_seg(u, seg);
      const int first = (seg * a.seg_chunks + c) * L, rows = min((seg + 1) * a.seg_chunks * L, seq_len(a.lens, u / a.H, a.T)) - first;
      nan_rows<DV>(a.o + (u / a.H) * a.os.b + (u % a.H) * a.os.h + (long long)first * a.os.t, a.os.t, rows, tid - 256, 128);
    }
  }
  if (OUT && tid == 256) bulk_wait_read();                     // output stores have left shared memory
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {                                           // a wait gave up (every warp is past its last one)
    int u, seg;
    unit_of(PIECES ? *ticket : block_again(), u, seg);
    const int cb = seg * a.seg_chunks, len = max(seq_len(a.lens, u / a.H, a.T) - cb * L, 0);
    const int n_chunks = min((len + L - 1) / L, a.seg_chunks);
    // MMAs and copies in flight end before the memory that they use goes
    if (warp == 13 && flight[kFlightMma]) {
      if (elect_one()) mma_commit(bar(bDrain));
      __syncwarp();
      mbar_drain(bar(bDrain), 0);
    }
    if (warp == 12)
      for (int n = flight[kFlightLoads], i = max(n - 2, 0); i < n; ++i)
        if (i * L + L <= len) mbar_drain(bar(bFull + (i & 1)), (i >> 1) & 1);
        else mbar_drain(bar(bTail), 0);
    __syncthreads();
    // (the maps' n and X, every state and the rows of o are NaN by the warps that did not finish them)
    if (KIND == kImages) nan_records(a.rec + ((long long)u * a.chunks + cb) * rec_bytes(true), n_chunks, kThreads);
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 13)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// The states that the segments start from: S_0 as given, S_1 = n_0, S_{g+1} = S_g
// X_g + n_g, in fp32 (the gradients: from the last segment to the first, with X
// transposed).  Rows do not mix, so a CTA takes 1024 entries of a unit's state; each
// of its eight warps takes an eighth of the sum over k for all of them, eight rows
// and four columns to a lane, so that what shared memory gives is used 32 times.
// The next segment's X comes in by cp.async meanwhile.  1.6 us a segment of 128 x
// 128 for up to 148 CTAs (9 units); 12.6 for eight segments.
template <int DK>
__global__ void __launch_bounds__(256)
delta_join_kernel(const ChunkArgs a, const float* given, const float* xs, bool reverse) {
  constexpr int ROWS = 1024 / DK, KW = DK / 8;                 // k of a warp
  extern __shared__ __align__(128) float jsm[];                // two X, the rows of S by k, the warps' sums
  float* S = jsm + 2 * DK * DK;
  float* part = S + DK * ROWS;
  const int slices = a.dv / ROWS, u = blockIdx.x / slices, r0 = (blockIdx.x % slices) * ROWS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cl = 4 * (lane % (DK / 4)), rl = 8 * (lane / (DK / 4));        // sums: this lane's columns and rows
  const int col = threadIdx.x % DK, row = 4 * (threadIdx.x / DK);          // results: four rows of a column
  auto fetch = [&](int g) {                                    // X of segment g
    if (g >= 1 && g + 1 < a.segs) {
      const float* x = xs + ((long long)u * (a.segs - 2) + (reverse ? a.segs - 2 - g : g - 1)) * DK * DK;
      const uint32_t d = smem_u32(jsm + (g & 1) * DK * DK);
#pragma unroll
      for (int i = 0; i < DK * DK / 4 / 256; ++i)
        cp_async16(d + (i * 256 + threadIdx.x) * 16, x + (i * 256 + threadIdx.x) * 4, true);
    }
    cp_async_commit();
  };
  after_previous();
  fetch(1);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    a.seg_s[((long long)u * a.segs * a.dv + r0 + row + r) * DK + col] =
        given == nullptr ? 0.f : given[((long long)u * a.dv + r0 + row + r) * DK + col];
  for (int g = 0; g + 1 < a.segs; ++g) {
    float y[4];
    const float* n = a.seg_n + (((long long)u * (a.segs - 1) + g) * a.dv + r0 + row) * DK + col;
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = n[r * DK];
    if (g > 0) {
      fetch(g + 1);
      cp_async_wait<1>();
      __syncthreads();                                         // X of g has landed; S is complete
      const float* x = jsm + (g & 1) * DK * DK + cl;
      uint64_t acc[4][4];                                      // [row pair][column]
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[p][c] = 0;
#pragma unroll 4
      for (int k = warp * KW; k < warp * KW + KW; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(x + k * DK);
        const ulonglong2 s0 = *reinterpret_cast<const ulonglong2*>(S + k * ROWS + rl);
        const ulonglong2 s1 = *reinterpret_cast<const ulonglong2*>(S + k * ROWS + rl + 4);
        const uint64_t s[4] = {s0.x, s0.y, s1.x, s1.y};
        const float vc[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint64_t vv = f2(vc[c], vc[c]);
#pragma unroll
          for (int p = 0; p < 4; ++p) acc[p][c] = fma2(s[p], vv, acc[p][c]);
        }
      }
      float* w = part + warp * (ROWS * DK) + rl * DK + cl;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float4 e, o;
        unf2(acc[p][0], e.x, o.x);
        unf2(acc[p][1], e.y, o.y);
        unf2(acc[p][2], e.z, o.z);
        unf2(acc[p][3], e.w, o.w);
        *reinterpret_cast<float4*>(w + 2 * p * DK) = e;
        *reinterpret_cast<float4*>(w + (2 * p + 1) * DK) = o;
      }
      __syncthreads();                                         // sums are complete; S and X of g have been read
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] += part[i * (ROWS * DK) + (row + r) * DK + col];
    }
    float* out = a.seg_s + (((long long)u * a.segs + g + 1) * a.dv + r0 + row) * DK + col;
#pragma unroll
    for (int r = 0; r < 4; ++r) out[r * DK] = y[r];
    *reinterpret_cast<float4*>(&S[col * ROWS + row]) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

template <int DK>
cudaError_t join_as(const ChunkArgs& a, const float* given, bool reverse, int B, cudaStream_t stream) {
  constexpr int smem = (2 * DK * DK + 9 * 1024) * 4;
  const float* x = reverse ? a.seg_xt : a.seg_x;
  return launch_after(delta_join_kernel<DK>, (unsigned)(B * a.H * (a.dv * DK / 1024)), 256, smem, stream, a, given, x, reverse);
}

template <int DK, int DV, int KIND, bool PIECES = false>
cudaError_t launch(const CUtensorMap* m, const ChunkArgs& args, int B, cudaStream_t stream) {
  ChunkArgs a = args;
  set_waits(a, KIND == kStateOnly ? LTE_GDR_LAUNCH_SEGMENTS : LTE_GDR_LAUNCH_CHAIN);
  const int per = KIND == kStateOnly ? 2 * a.segs - 3 : a.segs;
  return launch_after(delta_chain_tc_kernel<DK, DV, KIND, PIECES>, (unsigned)(B * a.H * per * a.pieces), kThreads, kSmem, stream,
                      m[0], m[1], m[2], m[3], a);
}
template <int DK, int DV>
cudaError_t run(const CUtensorMap* m, const ChunkArgs& a, int B, cudaStream_t stream) {
  if (a.segs > 1) {
    cudaError_t e = launch<DK, DV, kStateOnly>(m, a, B, stream);
    if (e == cudaSuccess) e = join_states(a, a.s_in, false, B, DK, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.s0 != nullptr)
    return a.pieces > 1 ? launch<DK, DV, kImages, true>(m, a, B, stream) : launch<DK, DV, kImages>(m, a, B, stream);
  return a.pieces > 1 ? launch<DK, DV, kO, true>(m, a, B, stream) : launch<DK, DV, kO>(m, a, B, stream);
}

}  // namespace chaintc

cudaError_t join_states(const ChunkArgs& a, const float* given, bool reverse, int B, int dk, cudaStream_t stream) {
  return dk == 128 ? chaintc::join_as<128>(a, given, reverse, B, stream) : chaintc::join_as<64>(a, given, reverse, B, stream);
}

cudaError_t forward_chain(const ChunkArgs& a, int B, int dk, cudaStream_t stream) {
  CUtensorMap m[4];
  if (!chaintc::map_of(&m[0], a.q, dk, a.Hk, a.T, B, a.qs) || !chaintc::map_of(&m[1], a.k, dk, a.Hk, a.T, B, a.ks) ||
      !chaintc::map_of(&m[2], a.v, a.dv, a.H, a.T, B, a.vs) ||
      (a.s0 == nullptr && !chaintc::map_of(&m[3], a.o, a.dv, a.H, a.T, B, a.os)))
    return cudaErrorNotSupported;
  if (dk == 128) return a.dv == 128 ? chaintc::run<128, 128>(m, a, B, stream) : chaintc::run<128, 64>(m, a, B, stream);
  return a.dv == 128 ? chaintc::run<64, 128>(m, a, B, stream) : chaintc::run<64, 64>(m, a, B, stream);
}

// Pieces of the sequences, in chunk steps: units over 148 come in waves, and the
// last wave is the shorter the shorter its CTAs.  Forwards a step is 2.6 us, and a
// CTA costs three more, or four and a half with a state to hand over.  64 chunks:
// 512 heads 690 us whole, 653 in two pieces, 702 in three; 160 heads 339, 275, 258,
// and 259 in four.  16 chunks of 512 heads: 193 whole, 220 in two.
int chain_pieces(long long units, int chunks, double whole, double cut) {
  int best = 1;
  double least = (double)((units + 147) / 148) * (chunks + whole);
  for (int p = 2; p <= (units > 148 ? 8 : 1) && p <= chunks; ++p) {
    const double t = (double)((units * p + 147) / 148) * ((chunks + p - 1) / p + cut);
    if (t < 0.98 * least) {
      least = t;
      best = p;
    }
  }
  return best;
}

// Segments of a sequence, by an estimate in us: a wave of CTAs is 148, a chunk takes
// 2.3 us for the maps and 2.6 for O, a CTA 6 beside its chunks, a segment 1.6 in the
// join, the two more launches 6.  One sequence of 16384 tokens: 16 heads 650 us in
// one piece, 238 in six (104 + 16 + 119), 271 in eight (two waves of maps); of 4096
// tokens: 2 heads 171 us in one, 65 in eight, 60 in twelve.
int chain_segments(long long units, int chunks, long long join_ctas) {
  auto waves = [](long long ctas) { return (double)((ctas + 147) / 148); };
  int best = 1;
  double least = 0.95 * waves(units) * (2.6 * chunks + 6);
  for (int g = 3; g <= 64 && g * 2 <= chunks; ++g) {
    const int per = (chunks + g - 1) / g;
    const double t = waves(units * (2 * g - 3)) * (2.3 * per + 6) + waves(units * g) * (2.6 * per + 6) +
                     1.6 * (g - 1) * waves(join_ctas) + 6;
    if (t < least) {
      least = t;
      best = g;
    }
  }
  return best;
}

}  // namespace delta
}  // namespace lte
