// Norms of queries and keys per head with the position rotation in the same
// pass, and their gradients.
//
// Row x of D channels (one token, one head), weight w, c = 1/D (RMS) or 1 (L2):
//   r = (c sum x^2 + eps)^(-1/2),  n = x r w,  y = rotation of n by the row's
//   position (channel pairs (i, i + R/2) or (2i, 2i + 1), i < R/2).
// Gradient, with dn the rotation back of dy (the rotation is orthogonal):
//   dx = r w dn - x c r^3 <w dn, x>,   dw = sum over rows of dn x r.
//
// Both are bound by memory: every row is read once and written once.  D / 8
// lanes hold a row, 8 channels (16 bytes of bf16) each; the sums and the
// partner channels of the (i, i + R/2) pairs go by shuffles.  A group of lanes
// takes several rows of the same token, so its cosines and sines (more bytes
// than a bf16 row) are read once, and the rows' loads are in flight together.
#include "lte_common.cuh"
#include "lte_internal.h"

namespace lte {
namespace qkn {

constexpr int kThreads = 256;

struct Args {
  const void *x[2];            // q, k
  const void *dy[2];           // gradients of the outputs (backward)
  void* y[2];                  // outputs: q', k' or dq, dk
  Strides4 xs[2], ds[2];       // strides of x, dy
  const float* w[2];
  const int32_t* pos;          // [B,T] or NULL (position t)
  const float* table;          // [n_pos][R]
  float* part;                 // [blocks][2][D] partial weight gradients
  long long tokens;            // B * T
  int T, H[2], n_pos, rot, norm, inter;   // norm: 0 none, 1 on
  float c, eps;
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
template <int LPR>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The rotation's factors for one lane's 8 channels: cos and sin of the pair of
// each channel, sin negated on the pair's first member (y = x cos + partner sin).
// A position outside the table gives NaN, which reaches the output.
struct Turn {
  float c[8], s[8];
  int src;                     // lane that holds the partner channels ((i, i + R/2) pairs)
};
template <int LPR>
__device__ __forceinline__ void load_turn(const Args& a, int lg, long long token, float dir, Turn& t) {
  const int lane = threadIdx.x & 31, e0 = lg * 8, R = a.rot;
  t.src = lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.f;
    t.s[i] = 0.f;
  }
  if (e0 >= R) return;
  const int p = a.pos != nullptr ? a.pos[token] : (int)(token % a.T);
  const bool ok = p >= 0 && p < a.n_pos;
  const float* row = a.table + (long long)(ok ? p : 0) * R;
  const float bad = __int_as_float(0x7fc00000);
  if (a.inter) {
    const float4 c4 = *reinterpret_cast<const float4*>(row + e0 / 2);
    const float4 s4 = *reinterpret_cast<const float4*>(row + R / 2 + e0 / 2);
    const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.c[2 * i] = t.c[2 * i + 1] = ok ? cc[i] : bad;
      t.s[2 * i] = -dir * ss[i];
      t.s[2 * i + 1] = dir * ss[i];
    }
  } else {
    const bool first = e0 < R / 2;
    const int i0 = first ? e0 : e0 - R / 2;
    t.src = first ? lane + R / 16 : lane - R / 16;
    load8(row + i0, t.c);
    load8(row + R / 2 + i0, t.s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] = ok ? t.c[i] : bad;
      t.s[i] *= first ? -dir : dir;
    }
  }
}
__device__ __forceinline__ void turn8(const Turn& t, bool inter, float (&v)[8]) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = inter ? v[i ^ 1] : __shfl_sync(0xffffffffu, v[i], t.src);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], t.c[i], o[i] * t.s[i]);
}

// rows [RPG part, RPG part + RPG) of a token's Hq + Hkv rows per group of lanes
template <typename T, int D, int RPG>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const Args a) {
  constexpr int LPR = D / 8, kGroups = kThreads / LPR;
  const int lg = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int heads = a.H[0] + a.H[1], parts = (heads + RPG - 1) / RPG;
  const long long gi = (long long)blockIdx.x * kGroups + grp;
  long long token = gi / parts;
  const int row0 = (int)(gi % parts) * RPG;
  const bool live = token < a.tokens;
  if (!live) token = 0;
  const long long b = token / a.T, t = token % a.T;
  float x[RPG][8];
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int row = row0 + i, which = row >= a.H[0], h = which ? row - a.H[0] : row;
    if (live && row < heads)
      load8((const T*)a.x[which] + b * a.xs[which].b + t * a.xs[which].t + h * a.xs[which].h + lg * 8, x[i]);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
  }
  Turn turn;
  load_turn<LPR>(a, lg, token, 1.f, turn);
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int row = row0 + i, which = row >= a.H[0], h = which ? row - a.H[0] : row;
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
      const float r = rsqrtf(fmaf(a.c, row_sum<LPR>(ss), a.eps));
      const float* w = a.w[which];
      if (w != nullptr) {
        float w8[8];
        load8(w + lg * 8, w8);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= r * w8[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= r;
      }
    }
    if (a.rot) turn8(turn, a.inter, x[i]);
    if (live && row < heads)
      store8((T*)a.y[which] + ((b * a.T + t) * a.H[which] + h) * D + lg * 8, x[i]);
  }
}

// Gradients: the blocks walk the groups; a lane sums its channels' weight
// gradients over all its rows in fp32 and the block's lanes add theirs in a
// fixed order, so the result does not change from run to run.
template <typename T, typename TG, int D, int RPG>
__global__ void __launch_bounds__(kThreads) qk_norm_backward_kernel(const Args a) {
  constexpr int LPR = D / 8, kGroups = kThreads / LPR;
  __shared__ float red[kGroups][2 * D];
  const int lg = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int heads = a.H[0] + a.H[1], parts = (heads + RPG - 1) / RPG;
  const long long total = a.tokens * parts, step = (long long)gridDim.x * kGroups;
  float dw[2][8], w8[2][8];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[n][e] = 0.f;
      w8[n][e] = 1.f;
    }
    if (a.norm && a.w[n] != nullptr) load8(a.w[n] + lg * 8, w8[n]);
  }
  for (long long g0 = (long long)blockIdx.x * kGroups; g0 < total; g0 += step) {
    const long long gi = g0 + grp;
    long long token = gi / parts;
    const int row0 = (int)(gi % parts) * RPG;
    const bool live = gi < total;
    if (!live) token = 0;
    const long long b = token / a.T, t = token % a.T;
    float x[RPG][8], dn[RPG][8];
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
      const int row = row0 + i, which = row >= a.H[0], h = which ? row - a.H[0] : row;
      if (live && row < heads) {
        load8((const TG*)a.dy[which] + b * a.ds[which].b + t * a.ds[which].t + h * a.ds[which].h + lg * 8, dn[i]);
        load8((const T*)a.x[which] + b * a.xs[which].b + t * a.xs[which].t + h * a.xs[which].h + lg * 8, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = dn[i][e] = 0.f;
      }
    }
    Turn turn;
    load_turn<LPR>(a, lg, token, -1.f, turn);
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
      const int row = row0 + i, which = row >= a.H[0], h = which ? row - a.H[0] : row;
      const bool on = live && row < heads;
      if (a.rot) turn8(turn, a.inter, dn[i]);
      if (a.norm) {
        float ss = 0.f, in = 0.f, z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[e] = dn[i][e] * (which ? w8[1][e] : w8[0][e]);
          ss = fmaf(x[i][e], x[i][e], ss);
          in = fmaf(z[e], x[i][e], in);
        }
        const float r = rsqrtf(fmaf(a.c, row_sum<LPR>(ss), a.eps));
        const float m = a.c * r * r * r * row_sum<LPR>(in);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = on ? dn[i][e] * x[i][e] * r : 0.f;
          dw[0][e] += which ? 0.f : d;
          dw[1][e] += which ? d : 0.f;
          dn[i][e] = fmaf(r, z[e], -m * x[i][e]);
        }
      }
      if (on) store8((T*)a.y[which] + ((b * a.T + t) * a.H[which] + h) * D + lg * 8, dn[i]);
    }
  }
  if (a.part == nullptr) return;
#pragma unroll
  for (int n = 0; n < 2; ++n) store8(&red[grp][n * D + lg * 8], dw[n]);
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s += red[g][i];
    a.part[(long long)blockIdx.x * 2 * D + i] = s;
  }
}

// dw[i] = sum over the blocks' partials, 32 columns per CTA, in a fixed order
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* __restrict__ part, int blocks, int D,
                                                          float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  float s = 0.f;
  for (int b = row; b < blocks; b += 32) s += part[(long long)b * 2 * D + col];
  red[row][threadIdx.x & 31] = s;
  __syncthreads();
  if (row == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    float* out = col < D ? dwq : dwk;
    if (out != nullptr) out[col < D ? col : col - D] = s;
  }
}

constexpr int kRows = 4;                 // rows of one token per group of lanes
constexpr int kBackwardBlocks = 148 * 6; // resident CTAs of the gradient kernel on 148 SMs

template <typename T, int D>
cudaError_t forward(const Args& a, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const int heads = a.H[0] + a.H[1];
  // few tokens (a decode step): one row per group, so that the rows spread over the SMs
  const bool few = a.tokens * heads <= 148LL * kGroups * kRows;
  const int parts = few ? heads : (heads + kRows - 1) / kRows;
  const unsigned grid = (unsigned)((a.tokens * parts + kGroups - 1) / kGroups);
  if (few) qk_norm_kernel<T, D, 1><<<grid, kThreads, 0, stream>>>(a);
  else qk_norm_kernel<T, D, kRows><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

inline int backward_blocks(long long tokens, int heads, int D) {
  const int groups = kThreads / (D / 8);
  const long long need = (tokens * ((heads + kRows - 1) / kRows) + groups - 1) / groups;
  return (int)(need < kBackwardBlocks ? need : kBackwardBlocks);
}

template <typename T, typename TG, int D>
cudaError_t backward(const Args& a, float* dwq, float* dwk, cudaStream_t stream) {
  const int blocks = backward_blocks(a.tokens, a.H[0] + a.H[1], D);
  qk_norm_backward_kernel<T, TG, D, kRows><<<blocks, kThreads, 0, stream>>>(a);
  if (a.part != nullptr) qk_norm_dw_kernel<<<2 * D / 32, 1024, 0, stream>>>(a.part, blocks, D, dwq, dwk);
  return cudaGetLastError();
}

Args args_of(const QkNormArgs& n) {
  Args a{};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = n.x[i];
    a.dy[i] = n.dy[i];
    a.y[i] = n.y[i];
    a.xs[i] = n.xs[i];
    a.ds[i] = n.ds[i];
    a.w[i] = n.w[i];
    a.H[i] = n.H[i];
  }
  a.pos = n.pos;
  a.table = n.table;
  a.part = (n.dwq != nullptr || n.dwk != nullptr) ? n.part : nullptr;
  a.tokens = (long long)n.B * n.T;
  a.T = n.T;
  a.n_pos = n.n_pos;
  a.rot = n.rot;
  a.inter = n.inter;
  a.norm = n.kind != LTE_NORM_NONE;
  a.c = n.kind == LTE_NORM_RMS ? 1.0f / n.D : 1.0f;
  a.eps = n.eps;
  return a;
}

}  // namespace qkn

size_t qk_norm_backward_bytes(int B, int T, int Hq, int Hkv, int D) {
  return (size_t)qkn::backward_blocks((long long)B * T, Hq + Hkv, D) * 2 * D * sizeof(float);
}

cudaError_t qk_norm(const QkNormArgs& n, cudaStream_t stream) {
  const qkn::Args a = qkn::args_of(n);
  if (n.dtype == LTE_BF16)
    return n.D == 128 ? qkn::forward<__nv_bfloat16, 128>(a, stream) : qkn::forward<__nv_bfloat16, 64>(a, stream);
  return n.D == 128 ? qkn::forward<float, 128>(a, stream) : qkn::forward<float, 64>(a, stream);
}

cudaError_t qk_norm_backward(const QkNormArgs& n, cudaStream_t stream) {
  const qkn::Args a = qkn::args_of(n);
  if (n.dtype == LTE_F32)
    return n.D == 128 ? qkn::backward<float, float, 128>(a, n.dwq, n.dwk, stream)
                      : qkn::backward<float, float, 64>(a, n.dwq, n.dwk, stream);
  if (n.grad_dtype == LTE_F32)
    return n.D == 128 ? qkn::backward<__nv_bfloat16, float, 128>(a, n.dwq, n.dwk, stream)
                      : qkn::backward<__nv_bfloat16, float, 64>(a, n.dwq, n.dwk, stream);
  return n.D == 128 ? qkn::backward<__nv_bfloat16, __nv_bfloat16, 128>(a, n.dwq, n.dwk, stream)
                    : qkn::backward<__nv_bfloat16, __nv_bfloat16, 64>(a, n.dwq, n.dwk, stream);
}

}  // namespace lte
