// Norms of queries and keys per head with the position rotation in the same
// pass, and their gradients.
//
// Row x of D channels (one token, one head), weight w, c = 1/D (RMS) or 1 (L2):
//   r = (c sum x^2 + eps)^(-1/2),  n = x r w,  y = rotation of n by the row's
//   position (channel pairs (i, i + R/2) or (2i, 2i + 1), i < R/2).
// Gradient, with dn the rotation back of dy (the rotation is orthogonal) and z = x r:
//   dx = r (w dn - z c r <w dn, x>),   dw = sum over rows of dn z.
//
// Both are bound by memory: every row is read once and written once.  D / 8
// lanes hold a row, two groups of 4 channels each, chosen so that both members
// of every pair are in one lane: channels 4 l and R/2 + 4 l on for the (i, i + R/2)
// pairs, 8 l and 8 l + 4 on otherwise.  Only the sums go by shuffles (with the
// partners fetched by shuffles too, waits for them were 30 to 44 % of all stalls:
// 277 us instead of 213 for 32 x 4096 tokens of 20 heads).  A group of lanes takes
// several rows of the same token, so its cosines and sines (as many bytes as a
// bf16 row) are read once, and the rows' loads are in flight together.
#include "lte_common.cuh"
#include "lte_internal.h"

namespace lte {
namespace qkn {

constexpr int kThreads = 256;

struct Args {
  const void *x[2];            // q, k
  const void *dy[2];           // gradients of the outputs (backward)
  void* y[2];                  // outputs: q', k' or dq, dk
  Strides4 xs[2];              // strides of x
  const float* w[2];
  const int32_t* pos;          // [B,T] or NULL (position t)
  const float* table;          // [n_pos][R]
  float* part;                 // [blocks][D] partial weight gradients
  long long tokens;            // B * T
  int T, H[2], n_pos, rot, norm, inter;   // norm: 0 none, 1 on
  float c, eps;
};

// a lane's 8 channels: 4 from channel a0 on, 4 from a1 on
struct Cols {
  int a0, a1;
};
__device__ __forceinline__ void load8(const float* p, Cols c, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p + c.a0), b = *reinterpret_cast<const float4*>(p + c.a1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// as they lie in memory: rows in flight take 4 registers in bf16, 8 in fp32
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, Cols c) {
    a = *reinterpret_cast<const float4*>(p + c.a0);
    b = *reinterpret_cast<const float4*>(p + c.a1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, Cols c) {
    a = *reinterpret_cast<const uint2*>(p + c.a0);
    b = *reinterpret_cast<const uint2*>(p + c.a1);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, Cols c, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p + c.a0) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + c.a1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, Cols c, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint2*>(p + c.a0) = make_uint2(u[0], u[1]);
  *reinterpret_cast<uint2*>(p + c.a1) = make_uint2(u[2], u[3]);
}
template <int LPR>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// lane lg of a row: its channels
__device__ __forceinline__ Cols cols_of(const Args& a, int lg) {
  if (!a.inter && 8 * lg < a.rot) return Cols{4 * lg, a.rot / 2 + 4 * lg};
  return Cols{8 * lg, 8 * lg + 4};
}
// The rotation's factors for one lane's four pairs.  Lanes behind R turn by nothing;
// a position outside the table gives NaN, which reaches the output.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ void load_turn(const Args& a, int lg, unsigned token, int pos, float dir, Turn& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.c[i] = 1.f;
    t.s[i] = 0.f;
  }
  if (8 * lg >= a.rot) return;
  const int p = a.pos != nullptr ? a.pos[token] : pos;
  const bool ok = p >= 0 && p < a.n_pos;
  const float* row = a.table + (long long)(ok ? p : 0) * a.rot + 4 * lg;
  const float4 c4 = *reinterpret_cast<const float4*>(row), s4 = *reinterpret_cast<const float4*>(row + a.rot / 2);
  const float bad = __int_as_float(0x7fc00000);
  t.c[0] = ok ? c4.x : bad; t.c[1] = ok ? c4.y : bad; t.c[2] = ok ? c4.z : bad; t.c[3] = ok ? c4.w : bad;
  t.s[0] = dir * s4.x; t.s[1] = dir * s4.y; t.s[2] = dir * s4.z; t.s[3] = dir * s4.w;
}
__device__ __forceinline__ void turn8(const Turn& t, bool inter, float (&v)[8]) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = inter ? v[2 * i] : v[i], y = inter ? v[2 * i + 1] : v[i + 4];
    const float p = fmaf(x, t.c[i], -y * t.s[i]), q = fmaf(y, t.c[i], x * t.s[i]);
    o[i] = p;
    o[i + 4] = q;
  }
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = o[i];
      v[2 * i + 1] = o[i + 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = o[i];
  }
}

// A group of lanes takes rows [h0, h0 + rows) of one token's queries or keys.
// The group index is 32 bits (host check), so its divisions are short.
struct Group {
  long long b, t;
  unsigned token;
  int h0, rows;
};
template <int RPG>
__device__ __forceinline__ Group group_of(const Args& a, unsigned gi, int which, unsigned parts, unsigned part0) {
  Group g;
  g.token = gi / parts;
  const int part = (int)(gi - g.token * parts) - (int)part0;
  g.h0 = part * RPG;
  g.rows = min(RPG, a.H[which] - g.h0);
  g.b = g.token / (unsigned)a.T;
  g.t = g.token - (unsigned)g.b * (unsigned)a.T;
  return g;
}

template <typename T, int D, int RPG>
__global__ void __launch_bounds__(kThreads, 5) qk_norm_kernel(const Args a) {
  constexpr int LPR = D / 8, kGroups = kThreads / LPR;
  const int lg = threadIdx.x % LPR;
  const unsigned partsq = (a.H[0] + RPG - 1) / RPG, parts = partsq + (a.H[1] + RPG - 1) / RPG;
  unsigned gi = blockIdx.x * (unsigned)kGroups + threadIdx.x / LPR;
  const bool live = gi < (unsigned)a.tokens * parts;
  if (!live) gi = 0;                                       // the lanes stay for the shuffles
  const int which = gi % parts >= partsq;
  const Group g = group_of<RPG>(a, gi, which, parts, which ? partsq : 0);
  const T* x = (const T*)a.x[which] + g.b * a.xs[which].b + g.t * a.xs[which].t + g.h0 * a.xs[which].h;
  T* y = (T*)a.y[which] + ((long long)g.token * a.H[which] + g.h0) * D;
  const Cols cols = cols_of(a, lg);
  Raw8<T> raw[RPG];
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    if (i < g.rows) raw[i].load(x + i * a.xs[which].h, cols);
    else raw[i].zero();
  }
  Turn turn;
  load_turn(a, lg, g.token, (int)g.t, 1.f, turn);
  float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (a.norm && a.w[which] != nullptr) load8(a.w[which], cols, w);
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    float v[8];
    raw[i].get(v);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
      const float r = rsqrtf(fmaf(a.c, row_sum<LPR>(ss), a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= r * w[e];
    }
    if (a.rot) turn8(turn, a.inter, v);
    if (live && i < g.rows) store8(y + i * D, cols, v);
  }
}

// Gradients: a block takes groups of queries or groups of keys only (blocks
// [0, blocks_q) and the rest), so a lane holds one set of weight gradients: its
// channels' sums over all its rows, in fp32.  The block's lanes are added in a
// fixed order, and so are the blocks, so the result repeats bit by bit.
template <typename T, typename TG, int D, int RPG>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_backward_kernel(const Args a, int blocks_q) {
  constexpr int LPR = D / 8, kGroups = kThreads / LPR;
  __shared__ float red[kGroups][D];
  const int lg = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int which = (int)blockIdx.x >= blocks_q;
  const unsigned block = which ? blockIdx.x - blocks_q : blockIdx.x, blocks = which ? gridDim.x - blocks_q : blocks_q;
  const unsigned parts = (a.H[which] + RPG - 1) / RPG, total = (unsigned)a.tokens * parts;
  const Cols cols = cols_of(a, lg);
  float dw[8], w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    dw[e] = 0.f;
    w[e] = 1.f;
  }
  if (a.norm && a.w[which] != nullptr) load8(a.w[which], cols, w);
  for (unsigned g0 = block * kGroups; g0 < total; g0 += blocks * kGroups) {
    const bool live = g0 + grp < total;
    const Group g = group_of<RPG>(a, live ? g0 + grp : 0, which, parts, 0);
    const T* xp = (const T*)a.x[which] + g.b * a.xs[which].b + g.t * a.xs[which].t + g.h0 * a.xs[which].h;
    const long long at = ((long long)g.token * a.H[which] + g.h0) * D;
    const TG* dp = (const TG*)a.dy[which] + at;
    Raw8<T> rx[RPG];
    Raw8<TG> rd[RPG];
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
      if (live && i < g.rows) {
        rd[i].load(dp + i * D, cols);
        rx[i].load(xp + i * a.xs[which].h, cols);
      } else {                                             // zeros add nothing to the weight gradients
        rd[i].zero();
        rx[i].zero();
      }
    }
    Turn turn;
    load_turn(a, lg, g.token, (int)g.t, -1.f, turn);
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
      const bool on = live && i < g.rows;
      float dn[8];
      rd[i].get(dn);
      if (a.rot) turn8(turn, a.inter, dn);
      if (a.norm) {
        float ss = 0.f, in = 0.f, v[8];
        rx[i].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(v[e], v[e], ss);
          in = fmaf(dn[e] * w[e], v[e], in);
        }
        const float r = rsqrtf(fmaf(a.c, row_sum<LPR>(ss), a.eps));
        // x r is bounded; r^3 is not (eps below 1e-25, rows of zeros): the sum takes one r, x another
        const float m = a.c * (r * row_sum<LPR>(in));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = v[e] * r;
          dw[e] += on ? dn[e] * z : 0.f;
          dn[e] = r * fmaf(w[e], dn[e], -m * z);
        }
      }
      if (on) store8((T*)a.y[which] + at + i * D, cols, dn);
    }
  }
  if (a.part == nullptr) return;
  store8(&red[grp][0], cols, dw);
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s += red[g][threadIdx.x];
    a.part[(long long)blockIdx.x * D + threadIdx.x] = s;
  }
}

// dw[i] = sum over the blocks' partials (rows [0, blocks_q) for the queries'
// weight, the others for the keys'), 32 columns per CTA, in a fixed order
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* __restrict__ part, int blocks_q, int blocks,
                                                          int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int which = blockIdx.x >= D / 32, lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int col = (which ? blockIdx.x - D / 32 : blockIdx.x) * 32 + lane;
  float s = 0.f;
  for (int b = (which ? blocks_q : 0) + row; b < (which ? blocks : blocks_q); b += 32) s += part[(long long)b * D + col];
  red[row][lane] = s;
  __syncthreads();
  if (row == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    float* out = which ? dwk : dwq;
    if (out != nullptr) out[col] = s;
  }
}

// rows of one token per group of lanes: what 64 registers hold without spills
template <typename T> constexpr int kRows = sizeof(T) == 2 ? 4 : 2;
constexpr int kBackRows = 2;             // (gradients: two rows of x and dy in flight)
constexpr int kBackBlocks = 148 * 3;     // resident CTAs of the gradient kernel on 148 SMs

template <typename T, int D>
cudaError_t forward(const Args& a, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8), kRpg = kRows<T>;
  // few tokens (a decode step): one row per group, so that the rows spread over the SMs
  const bool few = a.tokens * (a.H[0] + a.H[1]) <= 148LL * kGroups * kRpg;
  const int rpg = few ? 1 : kRpg;
  const long long groups = a.tokens * ((a.H[0] + rpg - 1) / rpg + (a.H[1] + rpg - 1) / rpg);
  const unsigned grid = (unsigned)((groups + kGroups - 1) / kGroups);
  if (few) qk_norm_kernel<T, D, 1><<<grid, kThreads, 0, stream>>>(a);
  else qk_norm_kernel<T, D, kRpg><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// blocks for the queries and for the keys, in proportion to their groups
inline void backward_blocks(long long tokens, int Hq, int Hkv, int D, int* bq, int* bk) {
  const int per = kThreads / (D / 8);
  const long long gq = tokens * ((Hq + kBackRows - 1) / kBackRows), gk = tokens * ((Hkv + kBackRows - 1) / kBackRows);
  const long long nq = (gq + per - 1) / per, nk = (gk + per - 1) / per;
  const long long q = nq * kBackBlocks / (nq + nk);
  *bq = (int)(nq + nk <= kBackBlocks ? nq : (q < 1 ? 1 : q));
  *bk = (int)(nq + nk <= kBackBlocks ? nk : (kBackBlocks - *bq < 1 ? 1 : kBackBlocks - *bq));
}

template <typename T, typename TG, int D>
cudaError_t backward(const Args& a, float* dwq, float* dwk, cudaStream_t stream) {
  int bq, bk;
  backward_blocks(a.tokens, a.H[0], a.H[1], D, &bq, &bk);
  qk_norm_backward_kernel<T, TG, D, kBackRows><<<bq + bk, kThreads, 0, stream>>>(a, bq);
  if (a.part != nullptr) qk_norm_dw_kernel<<<2 * D / 32, 1024, 0, stream>>>(a.part, bq, bq + bk, D, dwq, dwk);
  return cudaGetLastError();
}

Args args_of(const QkNormArgs& n) {
  Args a{};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = n.x[i];
    a.dy[i] = n.dy[i];
    a.y[i] = n.y[i];
    a.xs[i] = n.xs[i];
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
  int bq, bk;
  qkn::backward_blocks((long long)B * T, Hq, Hkv, D, &bq, &bk);
  return (size_t)(bq + bk) * D * sizeof(float);
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
