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
// Warps: 0-3 turn S, R and U (a thread per value channel, chain warps); 4-7
// finish O (or, for the gradients, write the images of S and U); 8 loads (TMA
// for K, Q and V, bulk copies for the record; two stages); 9 issues the MMAs.
// What bounds a chunk is the chain P -> R -> U -> S: about 1400 cycles of MMAs
// and, between them, the chain warps' passes over 256 values per thread.
//
// Rows of the last chunk behind the sequence's length are set to zero in shared
// memory before use, so what lies there (NaN, another sequence) does not enter.
// Every mbarrier wait is bounded; a CTA that gives up writes NaN to its state.
#include <math.h>

#include "delta_chunk.cuh"
#include "tc_ptx.cuh"

namespace lte {
namespace delta {
namespace chaintc {

using namespace tc;

constexpr int kThreads = 320;
constexpr uint32_t kHalf = L * 128;                          // [64 tokens][64 channels] bf16, 128B-swizzled
// a stage: K, Q, V (two halves each), then T hi, T lo, A, scalars as in the record
constexpr uint32_t kK = 0, kQ = 2 * kHalf, kV = 4 * kHalf, kR = 6 * kHalf;
constexpr uint32_t kScalOff = kR + 3 * kImg;
constexpr uint32_t kStage = (kScalOff + kScal + 1023) / 1024 * 1024;
constexpr uint32_t kIdent = 2 * kStage, kBars = kIdent + kImg, kSmem = kBars + 256;
static_assert(kSmem <= 227 * 1024, "shared memory");

// mbarriers; those without [] complete once per chunk
enum : int { bFull = 0, bEmpty = 2, bTail = 4, bSr = 5, bP = 6, bRr = 7, bU = 8, bUr = 9, bS = 10, bQS = 11, bOs = 12,
             bO = 13, bOf = 14, bSread = 15, bUread = 16, bDrain = 17, kBarCount = 18 };
constexpr uint32_t kColS = 0, kColPR = 256, kColVU = 320, kColUH = 384, kColUL = 416, kColO = 448;

__device__ __forceinline__ uint32_t idesc2(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// 16 pairs of values -> bf16 hi and lo words
__device__ __forceinline__ void split32(const float (&x)[32], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) split2(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
}
__device__ __forceinline__ void as_float(const uint32_t (&r)[32], float (&x)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r[e]);
}

template <int DK, int DV, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
delta_chain_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  constexpr uint32_t kColSh = DK, kColSl = DK + DK / 2;
  constexpr int kHK = DK / 64, kHV = DV / 64;                // 64-channel halves
  const int u = blockIdx.x, b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t s0 = sa(sm), bars = s0 + kBars;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kBars + 8 * kBarCount);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kBars + 8 * kBarCount + 8);
  auto bar = [&](int i) { return bars + 8 * i; };
  const int len = seq_len(a.lens, b, a.T), n_chunks = (len + L - 1) / L;
  constexpr int kRecBytes = rec_bytes(!OUT);

  if (tid == 0) {
    for (int i = 0; i < kBarCount; ++i) {
      const bool warps4 = i == bSr || i == bRr || i == bUr || i == bOs || i == bOf || i == bSread || i == bUread;
      mbar_init(bar(i), i == bEmpty || i == bEmpty + 1 ? 9 : warps4 ? 4 : 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the identity, [n][k] bf16
  for (int i = tid; i < L * 8; i += kThreads) {
    const int n = i >> 3, cc = i & 7;
    uint32_t w[4] = {0, 0, 0, 0};
    if (cc == n >> 3) w[(n & 7) >> 1] = (n & 1) ? 0x3f800000u : 0x00003f80u;
    *reinterpret_cast<uint4*>(sm + kIdent + n * 128 + ((cc ^ (n & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  fence_proxy_async();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  int loaded = 0;                                            // chunks requested (producer)
  bool issued = false;                                       // MMAs issued (MMA warp)

  if (warp == 8) {
    // ================================================================ loads
    const uint8_t* recs = a.rec + (long long)u * a.chunks * kRecBytes;
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c & 1;
      if (c >= 2 && !(ok = wwait(bar(bEmpty + s), ((c >> 1) - 1) & 1, abort_flag, nullptr, 0))) break;
      const uint32_t d = s0 + s * kStage;
      const bool tail = c * L + L > len;
      const uint32_t fb = tail ? bar(bTail) : bar(bFull + s);
      if (elect_one()) {
        const uint8_t* r = recs + (long long)c * kRecBytes;
        mbar_expect_tx(fb, (OUT ? 2 * kHK + kHV : kHK + kHV) * kHalf + (OUT ? 3 : 2) * kImg + kScal);
        for (int i = 0; i < kHK; ++i) {
          tma_load_4d(d + kK + i * kHalf, &tm_k, fb, 64 * i, hk, c * L, b);
          if (OUT) tma_load_4d(d + kQ + i * kHalf, &tm_q, fb, 64 * i, hk, c * L, b);
        }
        for (int i = 0; i < kHV; ++i) tma_load_4d(d + kV + i * kHalf, &tm_v, fb, 64 * i, h, c * L, b);
        if (OUT) {
          bulk_load(d + kR, r, 3 * kImg + kScal, fb);
        } else {
          bulk_load(d + kR, r, 2 * kImg, fb);
          bulk_load(d + kScalOff, r + 4 * kImg, kScal, fb);
        }
      }
      ++loaded;
      if (tail) {                                            // the last chunk: zeros behind the sequence
        if (!(ok = wwait(fb, 0, abort_flag, nullptr, 0))) break;
        const int r0 = len - c * L;
        for (int i = lane; i < (L - r0) * 8; i += 32) {
          const uint32_t off = (uint32_t)(r0 * 128 + i * 16);
          for (int j = 0; j < kHK; ++j) *reinterpret_cast<uint4*>(sm + s * kStage + kK + j * kHalf + off) = make_uint4(0, 0, 0, 0);
          for (int j = 0; j < kHV; ++j) *reinterpret_cast<uint4*>(sm + s * kStage + kV + j * kHalf + off) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bFull + s));
      }
    }
  } else if (warp == 9) {
    // ================================================================= MMAs
    const uint32_t id_tok = idesc2(128, L, false, false);      // N = tokens, B [n][k]
    const uint32_t id_vt = idesc2(128, L, true, false);        // V^T from [token][channel]
    const uint32_t id_s = idesc2(128, DK, false, true);        // N = key channels, B [k][n]
    const uint64_t ident = sdesc(s0 + kIdent, 16, 1024);
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c & 1, ph = c & 1;
      const uint32_t d = s0 + s * kStage;
      if (!(ok = wwait(bar(bFull + s), (c >> 1) & 1, abort_flag, nullptr, 0))) break;
      tc_fence_after();
      issued = true;
      const uint64_t dk = sdesc(d + kK, 16, 1024), dq = sdesc(d + kQ, 16, 1024), dt = sdesc(d + kR, 16, 1024);
      if (elect_one()) {                                       // V^T
        const uint64_t dv = sdesc(d + kV, kHalf, 1024);
#pragma unroll
        for (int ks = 0; ks < L / 16; ++ks)
          mma_f16(tmem + kColVU, dv + ((ks * 2048) >> 4), ident + ((ks * 32) >> 4), id_vt, ks > 0);
      }
      if (!(ok = wwait(bar(bSr), ph, abort_flag, nullptr, 0))) break;
      tc_fence_after();
      if (elect_one()) {                                       // P^T = S K^T
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_f16_ts(tmem + kColPR, tmem + (p ? kColSl : kColSh) + 8 * ks, dk + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                       id_tok, p + ks > 0);
        mma_commit(bar(bP));
      }
      if (OUT) {                                               // S Q^T
        if (c > 0 && !(ok = wwait(bar(bOf), (c - 1) & 1, abort_flag, nullptr, 0))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_f16_ts(tmem + kColO, tmem + kColSh + 8 * ks, dq + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4), id_tok, ks > 0);
          mma_commit(bar(bQS));
        }
      }
      if (!(ok = wwait(bar(bRr), ph, abort_flag, nullptr, 0))) break;
      tc_fence_after();
      if (elect_one()) {                                       // U^T = R^T T^T
#pragma unroll
        for (int p = 0; p < 3; ++p)                            // hi hi, lo hi, hi lo
#pragma unroll
          for (int ks = 0; ks < L / 16; ++ks)
            mma_f16_ts(tmem + kColVU, tmem + kColPR + (p == 1 ? 32 : 0) + 8 * ks,
                       dt + (((p == 2 ? kImg : 0) + ks * 32) >> 4), id_tok, p + ks > 0);
        mma_commit(bar(bU));
      }
      if (!(ok = wwait(bar(bUr), ph, abort_flag, nullptr, 0))) break;
      tc_fence_after();
      if (elect_one()) {                                       // S += (U diag(e^{G_L - G}))^T K
        const uint64_t dkn = sdesc(d + kK, kHalf, 1024);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < L / 16; ++ks)
            mma_f16_ts(tmem + kColS, tmem + kColVU + 32 * p + 8 * ks, dkn + ((ks * 2048) >> 4), id_s, 1u);
        mma_commit(bar(bS));
      }
      if (OUT) {                                               // O^T += U^T A^T
        if (!(ok = wwait(bar(bOs), ph, abort_flag, nullptr, 0))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < L / 16; ++ks)
              mma_f16_ts(tmem + kColO, tmem + (p ? kColUL : kColUH) + 8 * ks, dt + ((2 * kImg + ks * 32) >> 4), id_tok, 1u);
          mma_commit(bar(bO));
        }
      }
      if (c + 2 < n_chunks && elect_one()) mma_commit(bar(bEmpty + s));   // the stage is loaded once more
    }
    if (!ok && issued) {                                       // MMAs in flight end before exit
      __syncwarp();
      if (elect_one()) mma_commit(bar(bDrain));
      __syncwarp();
      mbar_drain(bar(bDrain), 0);
    }
  } else if (warp < 4) {
    // ========================================================== chain warps
    const int row = warp * 32 + lane;                          // value channel = TMEM lane
    const uint32_t la = tmem + ((uint32_t)(warp * 32) << 16);
    const long long srow = ((long long)u * DV + (row < DV ? row : 0)) * DK;
    auto scal_of = [&](int c) { return reinterpret_cast<const float*>(sm + (c & 1) * kStage + kScalOff); };
    auto arrive = [&](int i) {                                 // this warp's TMEM writes are done
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c & 1, ph = c & 1;
      if (!(ok = wwait(bar(bFull + s), (c >> 1) & 1, abort_flag, nullptr, 0))) break;
      const float* scal = scal_of(c);
      // ---- the state: bf16 hi and lo, and e^{G_L} S for this chunk's update
      if (c > 0) {
        if (!(ok = wwait(bar(bS), (c - 1) & 1, abort_flag, nullptr, 0))) break;
        if (!OUT && !(ok = wwait(bar(bSread), (c - 1) & 1, abort_flag, nullptr, 0))) break;
        tc_fence_after();
      }
      const float el = scal[kEG * L + L - 1];
#pragma unroll
      for (int j = 0; j < DK / 32; ++j) {
        float x[32];
        uint32_t r[32], hi[16], lo[16];
        if (c > 0) {
          tmem_ld32(la + kColS + 32 * j, r);
          tmem_wait_ld();
          as_float(r, x);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.s_in != nullptr && row < DV) v = reinterpret_cast<const float4*>(a.s_in + srow + 32 * j)[e];
            x[4 * e] = v.x; x[4 * e + 1] = v.y; x[4 * e + 2] = v.z; x[4 * e + 3] = v.w;
          }
        }
        split32(x, hi, lo);
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(x[e] * el);
        tmem_st16(la + kColSh + 16 * j, hi);
        tmem_st16(la + kColSl + 16 * j, lo);
        tmem_st32(la + kColS + 32 * j, r);
      }
      arrive(bSr);
      // ---- R^T = V^T - P^T diag(e^G)
      if (!(ok = wwait(bar(bP), ph, abort_flag, nullptr, 0))) break;
      tc_fence_after();
      float R[2][32];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t p[32], v[32], hi[16], lo[16];
        tmem_ld32(la + kColPR + 32 * j, p);
        tmem_ld32(la + kColVU + 32 * j, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 g = *reinterpret_cast<const float4*>(scal + kEG * L + 32 * j + e);
          R[j][e] = fmaf(-g.x, __uint_as_float(p[e]), __uint_as_float(v[e]));
          R[j][e + 1] = fmaf(-g.y, __uint_as_float(p[e + 1]), __uint_as_float(v[e + 1]));
          R[j][e + 2] = fmaf(-g.z, __uint_as_float(p[e + 2]), __uint_as_float(v[e + 2]));
          R[j][e + 3] = fmaf(-g.w, __uint_as_float(p[e + 3]), __uint_as_float(v[e + 3]));
        }
        split32(R[j], hi, lo);
        // hi over columns 0-31 of P's region, lo over 32-63: both halves of P are read first
        if (j == 0) {
          uint32_t p1[32], v1[32];
          tmem_ld32(la + kColPR + 32, p1);
          tmem_ld32(la + kColVU + 32, v1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(scal + kEG * L + 32 + e);
            R[1][e] = fmaf(-g.x, __uint_as_float(p1[e]), __uint_as_float(v1[e]));
            R[1][e + 1] = fmaf(-g.y, __uint_as_float(p1[e + 1]), __uint_as_float(v1[e + 1]));
            R[1][e + 2] = fmaf(-g.z, __uint_as_float(p1[e + 2]), __uint_as_float(v1[e + 2]));
            R[1][e + 3] = fmaf(-g.w, __uint_as_float(p1[e + 3]), __uint_as_float(v1[e + 3]));
          }
          tmem_st16(la + kColPR, hi);
          tmem_st16(la + kColPR + 32, lo);
          split32(R[1], hi, lo);
          tmem_st16(la + kColPR + 16, hi);
          tmem_st16(la + kColPR + 48, lo);
          break;
        }
      }
      arrive(bRr);
      // ---- U = T R + b R; U and U diag(e^{G_L - G}) as hi and lo
      if (!(ok = wwait(bar(bU), ph, abort_flag, nullptr, 0))) break;
      if (!OUT && c > 0 && !(ok = wwait(bar(bUread), (c - 1) & 1, abort_flag, nullptr, 0))) break;
      tc_fence_after();
      {
        uint32_t r0[32], r1[32];
        tmem_ld32(la + kColVU, r0);
        tmem_ld32(la + kColVU + 32, r1);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x[32];
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(scal + kBeta * L + 32 * j + e);
            const uint32_t* r = j ? r1 : r0;
            x[e] = fmaf(g.x, R[j][e], __uint_as_float(r[e]));
            x[e + 1] = fmaf(g.y, R[j][e + 1], __uint_as_float(r[e + 1]));
            x[e + 2] = fmaf(g.z, R[j][e + 2], __uint_as_float(r[e + 2]));
            x[e + 3] = fmaf(g.w, R[j][e + 3], __uint_as_float(r[e + 3]));
          }
          split32(x, hi, lo);
          tmem_st16(la + kColUH + 16 * j, hi);
          tmem_st16(la + kColUL + 16 * j, lo);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(scal + kLam * L + 32 * j + e);
            x[e] *= g.x; x[e + 1] *= g.y; x[e + 2] *= g.z; x[e + 3] *= g.w;
          }
          split32(x, hi, lo);
          tmem_st16(la + kColVU + 16 * j, hi);
          tmem_st16(la + kColVU + 32 + 16 * j, lo);
        }
      }
      arrive(bUr);
      if (lane == 0) mbar_arrive(bar(bEmpty + s));
    }
    if (ok && n_chunks > 0) {
      ok = wwait(bar(bS), (n_chunks - 1) & 1, abort_flag, nullptr, 0);
      tc_fence_after();
    }
    if (a.s_out != nullptr) {
#pragma unroll
      for (int j = 0; j < DK / 32; ++j) {
        uint32_t r[32];
        tmem_ld32(la + kColS + 32 * j, r);
        tmem_wait_ld();
        if (row < DV) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 v = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                   __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
            if (n_chunks == 0)
              v = a.s_in == nullptr ? make_float4(0.f, 0.f, 0.f, 0.f)
                                    : reinterpret_cast<const float4*>(a.s_in + srow + 32 * j)[e];
            if (!ok) v = make_float4(NAN, NAN, NAN, NAN);
            reinterpret_cast<float4*>(a.s_out + srow + 32 * j)[e] = v;
          }
        }
      }
    }
  } else {
    // ==================================================== O, or the images
    const int quad = warp - 4, row = quad * 32 + lane;
    const uint32_t la = tmem + ((uint32_t)(quad * 32) << 16);
    __nv_bfloat16* op = a.o + b * a.os.b + h * a.os.h + row;
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c & 1, ph = c & 1;
      if (!(ok = wwait(bar(bFull + s), (c >> 1) & 1, abort_flag, nullptr, 0))) break;
      const float* scal = reinterpret_cast<const float*>(sm + s * kStage + kScalOff);
      const long long img = (long long)u * a.chunks + c;
      if (OUT) {
        if (!(ok = wwait(bar(bQS), ph, abort_flag, nullptr, 0))) break;
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
        if (!(ok = wwait(bar(bO), ph, abort_flag, nullptr, 0))) break;
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(la + kColO, r[0]);
        tmem_ld32(la + kColO + 32, r[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bOf));
        if (row < DV) {                                        // a warp writes 64 bytes of each token's row
          const int n = min(L, len - c * L);
          __nv_bfloat16* o = op + (long long)c * L * a.os.t;
#pragma unroll
          for (int t = 0; t < L; ++t)
            if (t < n) o[(long long)t * a.os.t] = __float2bfloat16_rn(__uint_as_float(r[t >> 5][t & 31]));
        }
      } else {
        if (lane == 0) mbar_arrive(bar(bEmpty + s));
        if (!(ok = wwait(bar(bSr), ph, abort_flag, nullptr, 0))) break;
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
        if (!(ok = wwait(bar(bUr), ph, abort_flag, nullptr, 0))) break;
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
  }
  // copies in flight land before exit (only after a wait gave up)
  if (warp == 8 && *abort_flag) {
    for (int i = loaded - 2 > 0 ? loaded - 2 : 0; i < loaded; ++i)
      if (i * L + L <= len) mbar_drain(bar(bFull + (i & 1)), (i >> 1) & 1);
      else mbar_drain(bar(bTail), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// [channels, heads, T, B] with the tensor's strides; boxes of 64 tokens x 64 channels
inline bool map_of(CUtensorMap* m, const void* p, int D, int heads, int T, int B, Strides4 s) {
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  // the stride of an extent of 1 is never used, and need not be valid
  const cuuint64_t sb[3] = {(cuuint64_t)(heads > 1 ? s.h : D) * 2, (cuuint64_t)(T > 1 ? s.t : D) * 2,
                            (cuuint64_t)(B > 1 ? s.b : D) * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)L, 1};
  return tc::encode(m, p, 4, dims, sb, box);
}

template <int DK, int DV, bool OUT>
cudaError_t launch(const CUtensorMap* m, const ChunkArgs& a, int B, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(delta_chain_tc_kernel<DK, DV, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  delta_chain_tc_kernel<DK, DV, OUT><<<(unsigned)(B * a.H), kThreads, kSmem, stream>>>(m[0], m[1], m[2], a);
  return cudaGetLastError();
}
template <bool OUT>
cudaError_t dispatch(const CUtensorMap* m, const ChunkArgs& a, int B, int dk, cudaStream_t stream) {
  if (dk == 128) return a.dv == 128 ? launch<128, 128, OUT>(m, a, B, stream) : launch<128, 64, OUT>(m, a, B, stream);
  return a.dv == 128 ? launch<64, 128, OUT>(m, a, B, stream) : launch<64, 64, OUT>(m, a, B, stream);
}

}  // namespace chaintc

cudaError_t forward_chain_tc(const ChunkArgs& a, int B, int dk, cudaStream_t stream, bool* done) {
  CUtensorMap m[3];
  *done = chaintc::map_of(&m[0], a.q, dk, a.Hk, a.T, B, a.qs) && chaintc::map_of(&m[1], a.k, dk, a.Hk, a.T, B, a.ks) &&
          chaintc::map_of(&m[2], a.v, a.dv, a.H, a.T, B, a.vs);
  if (!*done) return cudaSuccess;
  return a.s0 == nullptr ? chaintc::dispatch<true>(m, a, B, dk, stream) : chaintc::dispatch<false>(m, a, B, dk, stream);
}

}  // namespace delta
}  // namespace lte
