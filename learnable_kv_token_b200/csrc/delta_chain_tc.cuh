// What the tcgen05 chains of the gated delta rule share.
#pragma once

#include "delta_chunk.cuh"
#include "tc_ptx.cuh"

namespace lte {
namespace delta {
namespace chaintc {

using namespace tc;

constexpr uint32_t kHalf = L * 128;                          // [64 tokens][64 channels] bf16, 128B-swizzled
// columns of a bf16 operand that lies as hi (16) and lo (16) over each 32 fp32 columns it was made from
__device__ __forceinline__ uint32_t pair_col(int ks, int lo) { return 32 * (ks >> 1) + 16 * lo + 8 * (ks & 1); }
__device__ __forceinline__ uint32_t idesc2(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// Registers go from the warps that load and issue to those that compute.  (With
// nearly all of the L1 cache as shared memory, a spilled register costs a trip to
// L2.)  All four warps of a group call these.  What the groups hold together after
// them must not exceed what the launch allocated, or regs_inc would wait for good:
// each kernel checks its own groups against launch_regs, a thread's share of the SM's
// 65536 registers in steps of 8.
constexpr int launch_regs(int threads) { return 65536 / threads / 8 * 8; }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// two fp32 values in one register pair
__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t r, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// a pair -> bf16 hi and lo words (as split2)
__device__ __forceinline__ void split_pair(uint64_t x, uint32_t& hi, uint32_t& lo) {
  float x0, x1;
  unf2(x, x0, x1);
  hi = pack_bf16(x0, x1);
  unf2(fma2(f2(bf_lo(hi), bf_hi(hi)), f2(-1.f, -1.f), x), x0, x1);
  lo = pack_bf16(x0, x1);
}
template <int N>
__device__ __forceinline__ void split_pairs(const uint64_t (&x)[N], uint32_t (&hi)[N], uint32_t (&lo)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) split_pair(x[e], hi[e], lo[e]);
}
// columns of this warp's lanes <-> registers, by count
__device__ __forceinline__ void tm_ld(uint32_t t, uint32_t (&r)[32]) { tmem_ld32(t, r); }
__device__ __forceinline__ void tm_ld(uint32_t t, uint32_t (&r)[16]) { tmem_ld16(t, r); }
__device__ __forceinline__ void tm_ld(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void tm_st(uint32_t t, const uint32_t (&r)[32]) { tmem_st32(t, r); }
__device__ __forceinline__ void tm_st(uint32_t t, const uint32_t (&r)[16]) { tmem_st16(t, r); }
__device__ __forceinline__ void tm_st(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint64_t pair_of(const uint32_t* r) { return f2(__uint_as_float(r[0]), __uint_as_float(r[1])); }

// the identity [n][k] bf16 in shared memory (all threads of the CTA)
__device__ __forceinline__ void write_identity(uint8_t* p, int threads) {
  for (int i = threadIdx.x; i < L * 8; i += threads) {
    const int n = i >> 3, cc = i & 7;
    uint32_t w[4] = {0, 0, 0, 0};
    if (cc == n >> 3) w[(n & 7) >> 1] = (n & 1) ? 0x3f800000u : 0x00003f80u;
    *reinterpret_cast<uint4*>(p + n * 128 + ((cc ^ (n & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// zeros in rows [r0, 64) of a half (the lanes of one warp)
__device__ __forceinline__ void zero_rows(uint8_t* half, int r0, int lane) {
  for (int i = lane; i < (L - r0) * 8; i += 32) *reinterpret_cast<uint4*>(half + r0 * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// A call's launches follow one another programmatically: a kernel sets up while the
// one before ends, and waits for its results here (which also waits, by induction,
// for all before it).  Where the grid leaves half of the SMs free, the next kernel's
// CTAs come at once, else when this one's have gone: 3 x 777 tokens of 8 heads, gradients,
// 126 -> 113 us; 512 tokens of 4 heads 36 -> 33; long calls as before.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (gridDim.x <= 74) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The delta rule's waits: for at most `limit` ns, then the CTA gives up (*abort_flag)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned limit, volatile int* abort_flag) {
  return mbar_wait_bounded(bar, parity, limit, abort_flag, nullptr, 0);
}
__device__ __forceinline__ bool wwait(uint32_t bar, uint32_t parity, unsigned limit, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit, abort_flag));
}
// What a CTA that gave up marks, so that nothing it left as it was is taken for a result:
// NaN in `rows` token rows, and in the scalars of `chunks` records, which turns all that
// the later launches make of those chunks into NaN.
// (The block's number is read anew there, and what is in flight is counted in shared
// memory: nothing for this end is kept in registers over the chunks.)
__device__ __forceinline__ int block_again() {
  int i;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(i));
  return i;
}
enum : int { kFlightLoads = 0, kFlightStates = 1, kFlightMma = 2 };
template <int COLS>
__device__ __forceinline__ void nan_rows(__nv_bfloat16* p, long long stride, int rows, int thread, int threads) {
  for (int i = thread; i < rows * (COLS / 8); i += threads)
    *reinterpret_cast<uint4*>(p + (i / (COLS / 8)) * stride + i % (COLS / 8) * 8) =
        make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
}
__device__ __forceinline__ void nan_records(uint8_t* rec, int chunks, int threads) {
  for (int c = 0; c < chunks; ++c)
    for (int i = threadIdx.x; i < kGradScal / 4; i += threads)
      reinterpret_cast<uint32_t*>(rec + (long long)c * rec_bytes(true) + 4 * kImg)[i] = 0x7fffffffu;
}

// Pieces of a sequence (chain_pieces): the number of a unit's pieces that are done, or
// kPieceFailed once one of them has given up: those behind it give up too, and a piece
// before it that was only slow must not leave its state where NaN belongs.
constexpr int kPieceFailed = 1 << 30;
// Every lane of a warp waits (half as long as the waits behind this one may take),
// so each has acquired what was written before the number.
__device__ __forceinline__ bool piece_ready(const int* done, int want, unsigned limit, volatile int* abort_flag) {
  const unsigned long long t0 = gtime();
  int v;
  do {
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
  } while (v < want && *abort_flag == 0 && gtime() - t0 < limit / 2);
  const bool ok = v >= want && v < kPieceFailed;
  if (!ok) *abort_flag = 1;
  return __all_sync(0xffffffffu, ok);
}
// By the warps that wrote the state (`threads` threads, all of which get here), `ok` where
// it is as it should be.  False: the unit's state has to become NaN.  (Whoever comes
// second to the counter sees the other, and writes after it: a piece that fails sets the
// counter before its NaN, one that is done has written its state before it looks.)
__device__ __forceinline__ bool piece_done(int* done, int seg, bool ok, int id, int threads) {
  __threadfence();
  ok = bar_and(id, threads, ok);
  bool stands = true;
  if (threadIdx.x == 0) {
    stands = atomicMax(done, ok ? seg + 1 : kPieceFailed) < kPieceFailed && ok;
    __threadfence();
  }
  return bar_and(id, threads, stands);
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

}  // namespace chaintc
}  // namespace delta
}  // namespace lte
