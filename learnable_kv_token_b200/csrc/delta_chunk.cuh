// The chunk form of the gated delta rule and what its kernels share.
//
// Within a chunk of L = 64 tokens, with G_t = sum_{i<=t} g_i from its first
// token on and S_0 the state before it, the corrections u_t = b_t (v_t - a_t
// S_{t-1} k_t) solve a unit lower triangular system:
//   (I + M) U = diag(b) R,   M_ts = b_t e^{G_t - G_s} k_t.k_s  (s < t),
//   R = V - diag(e^G) K S_0^T,
// so with T = (I + M)^{-1} diag(b):
//   U   = T R
//   O   = scale diag(e^G) Q S_0^T + A U,  A_ts = scale e^{G_t - G_s} q_t.k_s  (s <= t)
//   S_L = e^{G_L} S_0 + U^T diag(e^{G_L - G}) K.
// T and A depend on no state: one launch computes them for every chunk at
// once (delta_prepare.cu).  Every exponent is a difference taken forwards
// in time, so with g <= 0 no factor exceeds 1, whatever the decay.
//
// Precision.  q, k, v and their gradients are bf16, exact as operands.  Where a
// state or a correction is an operand of a product that feeds a state, it goes in as
// a bf16 pair hi + lo (two products; relative error about 2^-18 in the mean); T's
// product leaves out lo lo, of the same size.  States and their gradients come out
// 3.4e-6 to 4.1e-6 off in the 2-norm, gates' gradients 5e-6 to 7e-6, where fp32
// products give 4e-7 and 9e-7.  Nearly all of a state's share is U's split (2.8e-6 of
// 3.1e-6 with S, R, T and U split in 64-bit arithmetic on the host; a third part of
// each leaves 1e-7).  Third parts would be half as many products again on the chain
// that bounds these kernels, and their columns do not fit the backward chain's TMEM,
// which pairs fill.  What feeds bf16 outputs alone takes fewer bits where that is
// measurably cheaper (delta_backward.cu); O takes A and U as pairs.
#pragma once

#include "lte_common.cuh"
#include "lte_internal.h"
#include "mma_sync.cuh"

namespace lte {
namespace delta {

constexpr int L = 64;

// Per-chunk record in the workspace: T below its diagonal as hi and lo (the
// diagonal is b; T's rows act on R mostly through it, so it stays in fp32 and
// the bf16 pairs' error falls on the rest), A as hi and lo, each a [64][64] bf16
// image in the swizzled order in which it lies in shared memory (A's lo has one for
// the gradients only; for the prompt it lies in blocks of A's and T lo's that are not
// used, delta_prepare.cu), then five rows of 64 floats, and a sixth for the gradients.
constexpr int kImg = L * L * 2;
constexpr int kScal = 5 * L * 4;
constexpr int kEG = 0, kLam = 1, kBeta = 2, kGhi = 3, kGlo = 4;   // e^G, e^{G_L - G}, b, G as a float pair
constexpr int kInvB = 5;                                          // 1 / b
constexpr int kGradScal = kScal + L * 4;
__host__ __device__ constexpr int rec_bytes(bool a_lo) { return a_lo ? 4 * kImg + kGradScal : 3 * kImg + kScal; }

// A correction of b = 0 is exactly zero.  The gradients carry it as u = 2^-60 e
// instead, far below what fp32 sums beside it can see, so that e = u / b always
// exists (the gradient of b is y.e); the prompt takes b as it is, so that a token
// of b = 0 writes nothing at all.  F = b y is as small, so it is divided by b before it
// meets u: a product of both would be 2^-120 y e, and gradients of 1e-6 would
// leave the range of fp32's digits.
__device__ __forceinline__ float live_beta(float b) { return fabsf(b) < 0x1p-60f ? 0x1p-60f : b; }

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// (x0, x1) as bf16 pairs: hi rounded to nearest, lo the rounded remainder
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  lo = pack_bf16(x0 - bf_lo(hi), x1 - bf_hi(hi));
}

// B operand pair from [n][k] rows: n-tiles n0, n0 + 8 of k-step at 16-byte piece c
__device__ __forceinline__ int ldn_row(int lane) { return (lane & 7) + ((lane >> 4) & 1) * 8; }
__device__ __forceinline__ int ldn_col(int lane) { return (lane >> 3) & 1; }
// B operand pair from [k][n] rows (transposed load): k-step rows, n-tiles at pieces c, c + 1
__device__ __forceinline__ int ldt_row(int lane) { return (lane & 7) + ((lane >> 3) & 1) * 8; }
__device__ __forceinline__ int ldt_col(int lane) { return (lane >> 4) & 1; }

// rows [t0, t0 + 64) of a [T][D] tensor (row stride `ts`) -> a swizzled tile,
// zeros from row `len` on
template <int D, int THREADS>
__device__ __forceinline__ void load_rows(uint32_t dst, const __nv_bfloat16* src, long long ts, int t0, int len) {
#pragma unroll
  for (int i = threadIdx.x; i < L * (D / 8); i += THREADS) {
    const int r = i / (D / 8), c = i % (D / 8);
    const bool ok = t0 + r < len;
    cp_async16(dst + swz<D>(r, c), src + (long long)(ok ? t0 + r : t0) * ts + c * 8, ok);
  }
}
template <int BYTES, int THREADS>
__device__ __forceinline__ void load_linear(uint32_t dst, const uint8_t* src) {
  for (int i = threadIdx.x; i < BYTES / 16; i += THREADS) cp_async16(dst + i * 16, src + i * 16, true);
}

// 16-byte multiples of contiguous memory on their way to L2
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int T) {
  return lens == nullptr ? T : min(max(lens[b], 0), T);
}

struct ChunkArgs {
  const __nv_bfloat16 *q, *k, *v;
  Strides4 qs, ks, vs, os;
  const float *g, *beta;
  const int32_t* lens;
  const float* s_in;
  float* s_out;
  __nv_bfloat16* o;
  uint8_t* rec;          // [units][chunks] records
  // For the gradients, per chunk: images of S_0 (hi, lo) and U (hi, lo), [rows][cols] bf16
  // in blocks of 8 x 8 (128 bytes: row g at 16 g), rows = value channels.  A thread that
  // has a row stores 16 bytes per block, eight threads a block; ldmatrix reads blocks
  // without bank conflicts.
  uint32_t *s0, *u;
  int T, H, Hk, dv, chunks;
  float scale;
  // segments (segs = 1: the sequence in one piece): chunks of each, n [units][segs - 1][dv][dk],
  // X [units][segs - 2][dk][dk], states [units][segs][dv][dk], each in the chain's order
  // (backward: n of the last segment first); for the gradients X transposed too, and the
  // records hold A's lo
  int segs, seg_chunks;
  bool a_lo;
  // or pieces that follow one another (pieces = 1: one; seg_chunks: chunks of each): the
  // next piece's number and, per unit, its pieces that are done, each for the forward and
  // the backward chain (prepare sets all to zero)
  int pieces, *turn, *done;
  float *seg_n, *seg_x, *seg_xt, *seg_s;
  unsigned wait_ns;      // the launch's waits give up after this
  int withhold;          // the chunk, in the order in which a CTA takes them, whose loads are left out; -1
};

struct GradArgs {
  ChunkArgs f;
  const __nv_bfloat16* dO;
  Strides4 dos;
  const float* ds_out;       // gradient of the final state (NULL = zeros)
  float* ds_in;              // gradient of the initial state (nullable)
  __nv_bfloat16 *dq, *dk, *dv;
  float *dg, *db;
  uint32_t *ds, *fimg;       // images of dS (hi) and F (hi) per chunk, laid out as S_0's and U's
  float* hand;               // [units][dv][dk]: dS between pieces (forward: S, as s_out)
  float *x, *inner;          // per chunk and strip of 16 value channels: u.y and v.dv per token; <dS_0, S_0>
};

// Sets wait_ns and withhold of a launch (LTE_GDR_LAUNCH_*): one second and none, but for lte_gdr_withhold
void set_waits(ChunkArgs& a, int launch);

// Each returns cudaErrorNotSupported, without a launch, for tensors whose strides
// TMA does not take.
// delta_prepare.cu: the records of all chunks (with A's lo for the gradients)
cudaError_t prepare(const ChunkArgs& a, int B, int dk, bool a_lo, cudaStream_t stream);
// delta_chain_tc.cu: the chain of states with O; with s0 and u, writes their images instead of O
cudaError_t forward_chain(const ChunkArgs& a, int B, int dk, cudaStream_t stream);
// join_ctas: of the join of all units (units dv dk / 1024)
int chain_segments(long long units, int chunks, long long join_ctas);
// the states that the segments start from (seg_s), by n, X and the one given; reverse: the gradients, by X transposed
cudaError_t join_states(const ChunkArgs& a, const float* given, bool reverse, int B, int dk, cudaStream_t stream);
// `whole`, `cut`: what a CTA costs beside its chunks, in chunk steps, without and with a state to hand over
int chain_pieces(long long units, int chunks, double whole, double cut);
inline size_t piece_bytes(size_t units) { return (2 + 2 * units) * 4; }   // turn, then done
// delta_back_tc.cu: the backward chain
cudaError_t back_chain(const GradArgs& a, int B, int dk, cudaStream_t stream);

}  // namespace delta
}  // namespace lte
