// The gated delta rule, the linear layer whose state forgets by key:
//   S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,  a_t = e^{g_t},
//   o_t = scale S_t q_t                                     (S: dv x dk, fp32),
// which is, row by row of S, S_t = a_t S_{t-1} + u_t k_t^T with
//   u_t = b_t (v_t - a_t S_{t-1} k_t).
// The rows of S (value channels) do not depend on one another.
//
// This file holds the forms that walk the tokens one by one: the decode step
// and the recurrent kernel (fp32 inputs, and prompts of few tokens, where a
// chunk of 64 would be mostly empty).  Prompts in bf16 run in chunks on tensor
// cores (delta_chunk.cu).
#include "lte_common.cuh"
#include "lte_internal.h"

namespace lte {
namespace delta {

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16);
  v[1] = __uint_as_float(a.x & 0xffff0000u);
  v[2] = __uint_as_float(a.y << 16);
  v[3] = __uint_as_float(a.y & 0xffff0000u);
}

// ------------------------------------------------------------------ recurrent
// 8 lanes hold one row of S in registers (lane l: channels 4 l + 32 j .. + 3),
// 16 rows per CTA of 128 threads; blocks of kTok tokens of q, k and v are
// staged in shared memory as fp32.  Bound by the latency of a token's two sums:
// 0.34 us a token for up to 148 CTAs (18 heads of 128 value channels), 0.5 for 512,
// 3.1 for 4096.
constexpr int kTok = 16, kRecRows = 16;

struct RecArgs {
  const void *q, *k, *v;
  Strides4 qs, ks, vs, os;
  const float *g, *beta;
  const int32_t* lens;
  const float* s_in;
  float* s_out;
  void* o;
  int T, H, Hk, dv;
  float scale;
};

template <typename T, int DK>
__global__ void __launch_bounds__(128) delta_recurrent_kernel(const RecArgs a) {
  __shared__ __align__(16) float qs[kTok][DK], ks[kTok][DK];
  __shared__ float vs[kTok][kRecRows], as[kTok], bs[kTok];
  constexpr int J = DK / 32;
  const int slices = a.dv / kRecRows;
  const int u = blockIdx.x / slices, slice = blockIdx.x % slices;
  const int b = u / a.H, h = u % a.H, hk = h / (a.H / a.Hk);
  const int tid = threadIdx.x, l = tid & 7, row = tid >> 3;
  const int len = a.lens == nullptr ? a.T : min(max(a.lens[b], 0), a.T);
  const long long srow = ((long long)u * a.dv + slice * kRecRows + row) * DK;
  float S[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (a.s_in != nullptr) load4(a.s_in + srow + 4 * l + 32 * j, S[j]);
    else S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
  }
  const T* q = (const T*)a.q + b * a.qs.b + hk * a.qs.h;
  const T* k = (const T*)a.k + b * a.ks.b + hk * a.ks.h;
  const T* v = (const T*)a.v + b * a.vs.b + h * a.vs.h + slice * kRecRows;
  T* o = (T*)a.o + b * a.os.b + h * a.os.h + slice * kRecRows + row;
  for (int t0 = 0; t0 < len; t0 += kTok) {
    const int n = min(kTok, len - t0);
    __syncthreads();
    for (int i = tid; i < n * (DK / 4); i += 128) {
      const int t = i / (DK / 4), c = (i % (DK / 4)) * 4;
      float x[4];
      load4(q + (t0 + t) * a.qs.t + c, x);
      *reinterpret_cast<float4*>(&qs[t][c]) = make_float4(x[0], x[1], x[2], x[3]);
      load4(k + (t0 + t) * a.ks.t + c, x);
      *reinterpret_cast<float4*>(&ks[t][c]) = make_float4(x[0], x[1], x[2], x[3]);
    }
    for (int i = tid; i < n * kRecRows; i += 128)
      vs[i / kRecRows][i % kRecRows] = to_f32(v[(long long)(t0 + i / kRecRows) * a.vs.t + i % kRecRows]);
    if (tid < n) {
      const long long gi = ((long long)b * a.T + t0 + tid) * a.H + h;
      as[tid] = expf(a.g[gi]);
      bs[tid] = a.beta[gi];
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      float kk[J][4], sk = 0.f, sq = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        load4(&ks[t][4 * l + 32 * j], kk[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sk = fmaf(S[j][e], kk[j][e], sk);
      }
#pragma unroll
      for (int x = 4; x >= 1; x >>= 1) sk += __shfl_xor_sync(0xffffffffu, sk, x);
      const float ut = bs[t] * (vs[t][row] - as[t] * sk);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float qq[4];
        load4(&qs[t][4 * l + 32 * j], qq);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[j][e] = fmaf(S[j][e], as[t], ut * kk[j][e]);
          sq = fmaf(S[j][e], qq[e], sq);
        }
      }
#pragma unroll
      for (int x = 4; x >= 1; x >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, x);
      if (l == 0) o[(long long)(t0 + t) * a.os.t] = from_f32<T>(a.scale * sq);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
    *reinterpret_cast<float4*>(a.s_out + srow + 4 * l + 32 * j) = make_float4(S[j][0], S[j][1], S[j][2], S[j][3]);
}

// --------------------------------------------------------------------- decode
// One token: the state is read once and written once, 16 bytes per lane (the
// only traffic that counts: 8 dv dk bytes per head).  A warp takes kRows rows;
// their loads are all issued first, then the two dot products of each row
// (S k and S q) are summed over the lanes together.  With S q and k.q known,
//   o = scale (a S q + u (k.q)),
// so the output needs no second pass over the new state.  8.9 us for 512 states
// of 128 x 128 in fp32: 67 MB, the measured copy bandwidth or above (part of a
// state that was written last may still be in L2).
template <typename T, int DK, int ROWS>
__global__ void __launch_bounds__(128)
delta_step_kernel(int H, int Hk, int dv, float scale, const T* __restrict__ q, const T* __restrict__ k,
                  const T* __restrict__ v, const float* __restrict__ g, const float* __restrict__ beta,
                  T* __restrict__ o, float* __restrict__ state) {
  constexpr int LPR = DK / 4;                           // lanes of a row
  constexpr int PER = 32 / LPR;                         // rows side by side in a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int cpu = dv / (4 * ROWS * PER);                // CTAs per (batch, head)
  const int u = blockIdx.x / cpu;
  const int row0 = ((blockIdx.x % cpu) * 4 + warp) * ROWS * PER + sub;
  // the previous kernel in the stream may write this step's inputs or be the
  // previous step on this state; see the gated linear layer's step
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = u / H, h = u % H, hk = h / (H / Hk);
  float* st = state + ((long long)u * dv + row0) * DK + l * 4;
  float S[ROWS][4];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) load4(st + (long long)r * PER * DK, S[r]);
  float q4[4], k4[4];
  load4(q + ((long long)b * Hk + hk) * DK + l * 4, q4);
  load4(k + ((long long)b * Hk + hk) * DK + l * 4, k4);
  const float at = expf(g[u]), bt = beta[u];
  float kq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) kq = fmaf(k4[e], q4[e], kq);
#pragma unroll
  for (int x = LPR / 2; x >= 1; x >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, x);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const long long row = (long long)u * dv + row0 + r * PER;
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sk = fmaf(S[r][e], k4[e], sk);
      sq = fmaf(S[r][e], q4[e], sq);
    }
#pragma unroll
    for (int x = LPR / 2; x >= 1; x >>= 1) {
      sk += __shfl_xor_sync(0xffffffffu, sk, x);
      sq += __shfl_xor_sync(0xffffffffu, sq, x);
    }
    const float ut = bt * (to_f32(v[row]) - at * sk);
    *reinterpret_cast<float4*>(st + (long long)r * PER * DK) =
        make_float4(fmaf(at, S[r][0], ut * k4[0]), fmaf(at, S[r][1], ut * k4[1]),
                    fmaf(at, S[r][2], ut * k4[2]), fmaf(at, S[r][3], ut * k4[3]));
    if (l == 0) o[row] = from_f32<T>(scale * fmaf(at, sq, ut * kq));
  }
}

// -------------------------------------------------------------------- padding
// The rows behind a sequence are one stretch of each contiguous tensor: 16 bytes a
// thread, single words at its unaligned ends.  Bound by the writes: 537 MB (all of 32
// x 4096 rows) in 88 us, 6.1 TB/s; half of them 46.  (Zeroing the whole tensors
// first costs what is not padding too, and a launch for each.)
struct PadArgs {
  const int32_t* lens;
  char* x[8];
  long long row[8];
  int B, T;
};

__global__ void __launch_bounds__(256) delta_zero_padding_kernel(const PadArgs a) {
  char* x = a.x[blockIdx.y];
  const long long row = a.row[blockIdx.y];
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    const int len = min(max(a.lens[b], 0), a.T);
    char* p = x + ((long long)b * a.T + len) * row;
    const long long bytes = (a.T - len) * row;
    const long long head = min((long long)(-reinterpret_cast<intptr_t>(p) & 15), bytes), body = (bytes - head) / 16;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < body; i += gridDim.x * 256ll)
      *reinterpret_cast<uint4*>(p + head + i * 16) = make_uint4(0, 0, 0, 0);
    if (blockIdx.x == 0 && threadIdx.x < 8) {                  // up to three words before and behind
      const long long at = threadIdx.x < 4 ? threadIdx.x * 4 : head + body * 16 + (threadIdx.x - 4) * 4;
      if (at < (threadIdx.x < 4 ? head : bytes)) *reinterpret_cast<uint32_t*>(p + at) = 0;
    }
  }
}

template <typename T, int DK>
cudaError_t step(const lte_gdr_dims* d, const void* q, const void* k, const void* v, const float* g,
                 const float* beta, void* o, float* state, cudaStream_t stream) {
  constexpr int ROWS = 8, PER = 32 / (DK / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(d->B * d->H) * (d->dv / (4 * ROWS * PER)));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, delta_step_kernel<T, DK, ROWS>, d->H, d->Hk, d->dv, d->scale,
                            (const T*)q, (const T*)k, (const T*)v, g, beta, (T*)o, state);
}

}  // namespace delta

cudaError_t delta_recurrent(const DeltaArgs& a, cudaStream_t stream) {
  const lte_gdr_dims* d = a.d;
  delta::RecArgs r{a.q, a.k, a.v, a.qs, a.ks, a.vs, a.os, a.g, a.beta, a.lens, a.s_in, a.s_out, a.o,
                   d->T, d->H, d->Hk, d->dv, d->scale};
  const unsigned grid = (unsigned)(d->B * d->H) * (d->dv / delta::kRecRows);
  if (d->dtype == LTE_BF16) {
    if (d->dk == 128) delta::delta_recurrent_kernel<__nv_bfloat16, 128><<<grid, 128, 0, stream>>>(r);
    else delta::delta_recurrent_kernel<__nv_bfloat16, 64><<<grid, 128, 0, stream>>>(r);
  } else {
    if (d->dk == 128) delta::delta_recurrent_kernel<float, 128><<<grid, 128, 0, stream>>>(r);
    else delta::delta_recurrent_kernel<float, 64><<<grid, 128, 0, stream>>>(r);
  }
  return cudaGetLastError();
}

cudaError_t delta_zero_padding(int B, int T, const int32_t* lens, int n, void* const* x, const int64_t* row_bytes,
                               cudaStream_t stream) {
  delta::PadArgs a{};
  a.lens = lens; a.B = B; a.T = T;
  long long most = 0;
  for (int i = 0; i < n; ++i) {
    a.x[i] = (char*)x[i];
    a.row[i] = row_bytes[i];
    most = most > row_bytes[i] ? most : row_bytes[i];
  }
  // blocks for a stretch of T rows at 16 KB each, about eight to an SM over all stretches
  const int z = B < 65535 ? B : 65535;
  const long long need = (T * most + 16383) / 16384, fair = 8 * 148 / ((long long)z * n) + 1;
  const dim3 grid((unsigned)(need < fair ? need : fair), n, z);
  delta::delta_zero_padding_kernel<<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t delta_step(const lte_gdr_dims* d, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, void* o, float* state, cudaStream_t stream) {
  if (d->dtype == LTE_BF16)
    return d->dk == 128 ? delta::step<__nv_bfloat16, 128>(d, q, k, v, g, beta, o, state, stream)
                        : delta::step<__nv_bfloat16, 64>(d, q, k, v, g, beta, o, state, stream);
  return d->dk == 128 ? delta::step<float, 128>(d, q, k, v, g, beta, o, state, stream)
                      : delta::step<float, 64>(d, q, k, v, g, beta, o, state, stream);
}

}  // namespace lte
