// The part of the gated delta rule's chunk form that depends on no state, for
// every chunk at once (formulas: delta_chunk.cuh): T = (I + M)^{-1} diag(b) below
// its diagonal and A, and the chunk's scalars.
//
// One CTA of four warps per (head, chunk), six to an SM.  K and Q come by TMA as
// 128 stacked rows; one tcgen05 product with K gives K K^T (TMEM lanes 0-63) and
// Q K^T (64-127), so warps 0-1 have a row of M per thread and warps 2-3 a row of
// A.  X = (I + M)^{-1} in fp32, in place of M: the four 16 x 16 diagonal blocks by
// forward substitution (a lane per column), joined in pairs twice by
//   [A 0; C B]^{-1} = [A' 0; -B' C A' B'],
// the products as three TF32 warp MMAs.  Decays are powers of two by the approximate
// exponential (2 units in the last place, as expf) of float pairs.  Forward substitution keeps X accurate
// where a series in powers of M would not (equal keys make M's powers grow; X
// itself stays bounded).  A and T leave as images by bulk copies.
// The launch moves 57 KB per chunk (q, k in; T, A, scalars out): 1.87 GB for 32 x
// 4096 tokens x 16 heads in 425 us, 4.4 TB/s (409 without A's lo).  Beside that traffic it is bound by
// instruction issue (55 % busy) and by the barriers between its steps; loops over
// columns are not unrolled because six CTAs in different steps miss the instruction
// cache otherwise (29 us more).
#include <math.h>

#include "delta_chain_tc.cuh"

namespace lte {
namespace delta {
namespace prep {

using namespace chaintc;

constexpr int kPrepThreads = 128;
constexpr int kXs = 68;                                   // row stride of M and X in floats
// shared memory: the K and Q halves, then M over them and the images behind it
constexpr uint32_t kImages = 17 * 1024, kSmem = kImages + 2 * kImg;
static_assert(L * kXs * 4 <= kImages, "M");

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
// c (16 x 8 NT) = A (16 x 8 KS) B (8 KS x 8 NT), row stride kXs: three TF32
// products per step keep about 21 bits
template <int NT, int KS>
__device__ __forceinline__ void mma_tf32x3(float (&c)[NT][4], const float* A, const float* B, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll 2
  for (int k = 0; k < KS; ++k) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      split_tf32(A[(g + 8 * (e & 1)) * kXs + 8 * k + t + 4 * (e >> 1)], ah[e], al[e]);
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
__device__ __forceinline__ void store_c(float* p, const float* c, int lane, float sign = 1.f) {
  float* q = p + (lane >> 2) * kXs + (lane & 3) * 2;
  *reinterpret_cast<float2*>(q) = make_float2(sign * c[0], sign * c[1]);
  *reinterpret_cast<float2*>(q + 8 * kXs) = make_float2(sign * c[2], sign * c[3]);
}


// The prompt's record has no image for A's lo: products leave out the 16 x 16 blocks
// above the diagonal, and there it lies, a column of blocks of it under one another for
// the chain's operands.  Column j >= 1 in A's image from row 0 of column 4 - j on; of
// column 0, which no column has room for, the block on the diagonal in T lo's image
// (the second buffer) in column 2, the others there in column 3.  (Offset of token row t,
// in bytes, and its first 16-byte piece.)
__device__ __forceinline__ uint32_t alo_at(int t, int j) {
  return j > 0 ? (t - 16 * j) * 128 : kImg + (t < 16 ? t : t - 16) * 128;
}
__device__ __forceinline__ int alo_col(int t, int j) { return j > 0 ? 2 * (4 - j) : t < 16 ? 4 : 6; }

template <int DK, bool A_LO>
__global__ void __launch_bounds__(kPrepThreads, 6)
delta_prepare_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ __align__(16) float2 G2[L];                  // log2(e) G as a float pair
  __shared__ __align__(16) float bs[L];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  constexpr int kHK = DK / 64;
  const int u = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
  const int b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = seq_len(a.lens, b, a.T), t0 = c * L;
  if (gridDim.x <= 6 * 74) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.pieces > 1 && c == 0 && tid == 0) {
    a.done[u] = a.done[gridDim.x / a.chunks + u] = 0;
    if (u == 0) a.turn[0] = a.turn[1] = 0;
  }
  if (t0 >= len) return;
  const uint32_t s0 = sa(sm), bar_in = sa(&bars[0]), bar_mma = sa(&bars[1]);
  uint8_t* rec = a.rec + (long long)blockIdx.x * rec_bytes(A_LO);
  float* scal = reinterpret_cast<float*>(rec + (A_LO ? 4 : 3) * kImg);
  if (tid == 0) {
    mbar_init(bar_in, 1);
    mbar_init(bar_mma, 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (c != a.withhold) mbar_expect_tx(bar_in, 2 * kHK * kHalf);
    for (int i = 0; i < (c != a.withhold ? kHK : 0); ++i) {                       // half i: 64 rows of K, then 64 of Q
      tma_load_4d(s0 + 2 * i * kHalf, &tm_k, bar_in, 64 * i, hk, t0, b);
      tma_load_4d(s0 + (2 * i + 1) * kHalf, &tm_q, bar_in, 64 * i, hk, t0, b);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&tmem_slot)), "r"(64u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 3) {
    // running sums of the gates in 64 bits: after a gate that forgets
    // everything, differences of later sums keep their digits
    double x0 = 0, x1 = 0;
    float b0 = 0x1p-60f, b1 = 0x1p-60f;
    const long long gi = ((long long)b * a.T + t0 + 2 * lane) * a.H + h;
    if (t0 + 2 * lane < len) {
      const float x = a.g[gi];
      x0 = x < -104.f ? -104.f : x;                       // e^-104 is 0 in fp32
      b0 = A_LO ? live_beta(a.beta[gi]) : a.beta[gi];
    }
    if (t0 + 2 * lane + 1 < len) {
      const float x = a.g[gi + a.H];
      x1 = x < -104.f ? -104.f : x;
      b1 = A_LO ? live_beta(a.beta[gi + a.H]) : a.beta[gi + a.H];
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
    if (A_LO) out[kInvB * 32] = make_float2(1.f / b0, 1.f / b1);
    out[kGhi * 32] = make_float2((float)G0, (float)G1);
    out[kGlo * 32] = make_float2((float)(G0 - (float)G0), (float)(G1 - (float)G1));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true, issued = false;
  if (t0 + L > len) {                                     // rows behind the sequence are not data
    ok = mbar_wait(bar_in, 0, a.wait_ns, &abort_flag);
    const int r0 = len - t0;
    for (int i = warp; i < 2 * kHK; i += 4) zero_rows(sm + i * kHalf, r0, lane);
    fence_proxy_async();
    ok = __syncthreads_and(ok);
  }
  if (warp == 0) {                                        // [K; Q] K^T
    ok = ok && wwait(bar_in, 0, a.wait_ns, &abort_flag);
    tc_fence_after();
    issued = ok;
    if (ok && elect_one()) {
      const uint64_t d = sdesc(s0, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        const uint64_t x = d + (((ks >> 2) * 2 * kHalf + (ks & 3) * 32) >> 4);
        mma_f16(tmem, x, x, idesc2(128, L, false, false), ks > 0);
      }
      mma_commit(bar_mma);
    }
  }
  ok = ok && mbar_wait(bar_mma, 0, a.wait_ns, &abort_flag);
  // all or none: also, every thread is past the product before its operands are overwritten
  ok = __syncthreads_and(ok);
  if (ok) {
    tc_fence_after();
    float* M = reinterpret_cast<float*>(sm);
    uint8_t* img = sm + kImages;
    {
      const int t = tid & 63, far = warp & 1;             // rows 32 .. 63 reach columns 32 .. 63
      const uint32_t la = tmem + ((uint32_t)(warp * 32) << 16);
      const float2 Gt = G2[t];
      const bool keys = warp < 2;
      const float f = keys ? bs[t] : a.scale;
      const int last = keys ? t - 1 : t;                  // M is strictly below the diagonal
      const uint64_t gh = f2(Gt.x, Gt.x), gl = f2(Gt.y, Gt.y), ff = f2(f, f), minus = f2(-1.f, -1.f);
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {                       // 16 columns (not unrolled: six CTAs share the instruction cache)
        float y[16];
        if (j < 2 || far) {
          uint32_t r[16];
          tmem_ld16(la + 16 * j, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            // G2 holds two columns as (hi, lo, hi, lo): gathered as pairs of hi and of lo
            const float4 Gs = *reinterpret_cast<const float4*>(&G2[16 * j + e]);
            const uint64_t d = fma2(f2(Gs.x, Gs.z), minus, gh), dl = fma2(f2(Gs.y, Gs.w), minus, gl);
            float d0, d1;
            unf2(fma2(dl, f2(1.f, 1.f), d), d0, d1);
            unf2(mul2(mul2(pair_of(r + e), ff), f2(ex2(d0), ex2(d1))), y[e], y[e + 1]);
          }
          if (j >= 2 * far) {                             // a block on the diagonal of this warp's rows
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = 16 * j + e <= last ? y[e] : 0.f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = 0.f;
        }
        if (keys) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(&M[t * kXs + 16 * j + e]) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        } else {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(y[2 * e], y[2 * e + 1], hi[e], lo[e]);
          // lo: an image of its own, or in blocks above the diagonal (alo_at; t & 7 is the place's as well)
          const uint32_t at = A_LO ? kImg + t * 128 : alo_at(t, j);
          const int cl = A_LO ? 2 * j : alo_col(t, j);
          if (A_LO || j <= t >> 4) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              *reinterpret_cast<uint4*>(img + t * 128 + (((2 * j + e) ^ (t & 7)) << 4)) =
                  make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
              *reinterpret_cast<uint4*>(img + at + (((cl + e) ^ (t & 7)) << 4)) =
                  make_uint4(lo[4 * e], lo[4 * e + 1], lo[4 * e + 2], lo[4 * e + 3]);
            }
          }
        }
      }
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == 127) {
      bulk_store(rec + 2 * kImg, s0 + kImages, (A_LO ? 2 : 1) * kImg);
      bulk_commit();
    }
    // the diagonal blocks: warp d, a lane per column; rows of M by broadcast
    {
      const int d = 16 * warp, col = lane & 15;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == col ? 1.f : 0.f;
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
      __syncwarp();
      if (lane < 16)
#pragma unroll
        for (int i = 0; i < 16; ++i) M[(d + i) * kXs + d + lane] = x[i];
    }
    __syncthreads();
    // pairs of 16 (warp: pair and half of its columns), then the pair of 32 (warp:
    // half of its rows and of its columns): W = C A' goes to the block above the
    // diagonal, which is not used otherwise; then -B' W in the place of C
    {
      const int c0 = 32 * (warp >> 1), r0 = c0 + 16, n0 = 8 * (warp & 1);
      float w[1][4] = {};
      mma_tf32x3<1, 2>(w, &M[r0 * kXs + c0], &M[c0 * kXs + c0 + n0], lane);
      store_c(&M[c0 * kXs + r0 + n0], w[0], lane);
      __syncthreads();
      float y[1][4] = {};
      mma_tf32x3<1, 2>(y, &M[r0 * kXs + r0], &M[c0 * kXs + r0 + n0], lane);
      __syncthreads();                                    // W has been read
      store_c(&M[r0 * kXs + c0 + n0], y[0], lane, -1.f);
      const float zero[4] = {};
      store_c(&M[c0 * kXs + r0 + n0], zero, lane);        // above the diagonal of the pair
    }
    __syncthreads();
    {
      const int m0 = 16 * (warp >> 1), n0 = 16 * (warp & 1);
      float w[2][4] = {};
      mma_tf32x3<2, 4>(w, &M[(32 + m0) * kXs], &M[n0], lane);
      store_c(&M[m0 * kXs + 32 + n0], w[0], lane);
      store_c(&M[m0 * kXs + 40 + n0], w[1], lane);
      __syncthreads();
      float y[2][4] = {};
      mma_tf32x3<2, 4>(y, &M[(32 + m0) * kXs + 32], &M[32 + n0], lane);
      store_c(&M[(32 + m0) * kXs + n0], y[0], lane, -1.f); // C was read before W was complete
      store_c(&M[(32 + m0) * kXs + n0 + 8], y[1], lane, -1.f);
    }
    if (tid == 127) bulk_wait_read();                     // A's image has left
    __syncthreads();
    // T = X diag(b) below the diagonal, as hi and lo (its diagonal is b itself)
#pragma unroll 1
    for (int it = 0; it < L * 8 / kPrepThreads; ++it) {
      const int i = it * kPrepThreads + tid, t = i >> 3, cc = i & 7;
      if (!A_LO && cc >> 1 > t >> 4) continue;            // a block above the diagonal: A's lo, or nothing that is read
      uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
      if (8 * cc < t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int s = 8 * cc + 4 * e;
          const float4 x = *reinterpret_cast<const float4*>(&M[t * kXs + s]);
          const float4 bb = *reinterpret_cast<const float4*>(&bs[s]);
          split2(s < t ? x.x * bb.x : 0.f, s + 1 < t ? x.y * bb.y : 0.f, hi[2 * e], lo[2 * e]);
          split2(s + 2 < t ? x.z * bb.z : 0.f, s + 3 < t ? x.w * bb.w : 0.f, hi[2 * e + 1], lo[2 * e + 1]);
        }
      }
      const uint32_t off = t * 128 + ((cc ^ (t & 7)) << 4);
      *reinterpret_cast<uint4*>(img + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(img + kImg + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_proxy_async();
    __syncthreads();
    if (tid == 127) {
      bulk_store(rec, s0 + kImages, 2 * kImg);
      bulk_commit();
      bulk_wait_all();
    }
  } else {
    // a wait gave up: the chunk's scalars turn everything behind them into NaN; the
    // product and the copies in flight end before the memory that they use goes
    for (int i = tid; i < (A_LO ? kGradScal : kScal) / 4; i += kPrepThreads) scal[i] = NAN;
    if (tid == 0 && c != a.withhold) mbar_drain(bar_in, 0);
    if (issued) mbar_drain(bar_mma, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(64u) : "memory");
}

template <int DK, bool A_LO>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const ChunkArgs& a, int B, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel<DK, A_LO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  delta_prepare_kernel<DK, A_LO><<<(unsigned)(B * a.H) * a.chunks, kPrepThreads, kSmem, stream>>>(mq, mk, a);
  return cudaGetLastError();
}

}  // namespace prep

cudaError_t prepare(const ChunkArgs& args, int B, int dk, bool a_lo, cudaStream_t stream) {
  ChunkArgs a = args;
  set_waits(a, LTE_GDR_LAUNCH_PREPARE);
  CUtensorMap q, k;
  if (!chaintc::map_of(&q, a.q, dk, a.Hk, a.T, B, a.qs) || !chaintc::map_of(&k, a.k, dk, a.Hk, a.T, B, a.ks))
    return cudaErrorNotSupported;
  if (dk == 128) return a_lo ? prep::launch<128, true>(q, k, a, B, stream) : prep::launch<128, false>(q, k, a, B, stream);
  return a_lo ? prep::launch<64, true>(q, k, a, B, stream) : prep::launch<64, false>(q, k, a, B, stream);
}

}  // namespace delta
}  // namespace lte
