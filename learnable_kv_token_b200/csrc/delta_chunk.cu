// Gated delta rule over prompts, in chunks of 64 tokens on tensor cores
// (formulas and precision: delta_chunk.cuh): which form a call takes, its
// workspace and its launches.  Everything that depends on no state, for all
// chunks at once (delta_prepare.cu), then the chain of states (delta_chain_tc.cu).
#include <atomic>

#include "delta_chunk.cuh"
#include "tc_ptx.cuh"

namespace lte {

// Few tokens run token by token: a chunk costs its two launches (16 us, 49 for 512
// heads) however empty it is, a token 0.34 us while its CTAs (one per 16 value
// channels of a head) find an SM each, 0.5 at 512 of them, 3.1 at 4096.  Measured
// crossings: 40 tokens for 4 heads of 128 channels, 28 for 64, 15 for 512.
bool delta_chunked(const lte_gdr_dims* d) {
  const long long strips = (long long)d->B * d->H * (d->dv / 16);
  return d->dtype == LTE_BF16 && d->T > (strips <= 148 ? 40 : strips <= 512 ? 28 : 15);
}

namespace {
std::atomic<int> g_withheld{0}, g_chunk{0};
std::atomic<unsigned> g_limit_ns{0};
}  // namespace
void delta_withhold(int launches, int chunk, unsigned limit_ns) {
  g_chunk = chunk;
  g_limit_ns = limit_ns;
  g_withheld = launches;
}
void delta::set_waits(ChunkArgs& a, int launch) {
  const bool on = g_withheld & launch;
  a.wait_ns = on ? g_limit_ns.load() : (unsigned)tc::kWaitNs;
  a.withhold = on ? g_chunk.load() : -1;
}

namespace {
// workspace: records, then the segments' maps and states, then the pieces' counters
struct PrefillLayout {
  int chunks, segs, pieces;
  size_t n, x, s, turn, total;
  explicit PrefillLayout(const lte_gdr_dims* d) {
    const size_t units = (size_t)d->B * d->H, state = (size_t)d->dv * d->dk * 4;
    chunks = (d->T + delta::L - 1) / delta::L;
    segs = delta::chain_segments((long long)units, chunks, (long long)units * d->dv * d->dk / 1024);
    pieces = segs > 1 ? 1 : delta::chain_pieces((long long)units, chunks, 3, 4.5);
    size_t at = units * chunks * delta::rec_bytes(false);
    auto take = [&](size_t bytes) { const size_t r = (at + 255) & ~(size_t)255; at = r + bytes; return r; };
    n = take(segs > 1 ? units * (segs - 1) * state : 0);
    x = take(segs > 1 ? units * (segs - 2) * d->dk * d->dk * 4 : 0);
    s = take(segs > 1 ? units * segs * state : 0);
    turn = take(pieces > 1 ? delta::piece_bytes(units) : 0);
    total = at;
  }
};
}  // namespace

size_t delta_prefill_bytes(const lte_gdr_dims* d) { return delta_chunked(d) ? PrefillLayout(d).total : 0; }

cudaError_t delta_prefill(const DeltaArgs& a, cudaStream_t stream) {
  const lte_gdr_dims* d = a.d;
  if (!delta_chunked(d)) return delta_recurrent(a, stream);
  const PrefillLayout w(d);
  uint8_t* ws = (uint8_t*)a.scratch;
  delta::ChunkArgs c{};
  c.q = (const __nv_bfloat16*)a.q; c.k = (const __nv_bfloat16*)a.k; c.v = (const __nv_bfloat16*)a.v;
  c.qs = a.qs; c.ks = a.ks; c.vs = a.vs; c.os = a.os;
  c.g = a.g; c.beta = a.beta; c.lens = a.lens; c.s_in = a.s_in; c.s_out = a.s_out;
  c.o = (__nv_bfloat16*)a.o; c.rec = ws;
  c.T = d->T; c.H = d->H; c.Hk = d->Hk; c.dv = d->dv; c.chunks = w.chunks;
  c.scale = d->scale;
  c.segs = w.segs; c.pieces = w.pieces; c.seg_chunks = (w.chunks + w.segs * w.pieces - 1) / (w.segs * w.pieces);
  c.turn = (int*)(ws + w.turn); c.done = c.turn + 2;
  c.seg_n = (float*)(ws + w.n); c.seg_x = (float*)(ws + w.x); c.seg_s = (float*)(ws + w.s);
  cudaError_t e = delta::prepare(c, d->B, d->dk, false, stream);
  if (e == cudaSuccess) e = delta::forward_chain(c, d->B, d->dk, stream);
  // strides that TMA does not take: token by token (whatever ran is written again)
  return e == cudaErrorNotSupported ? delta_recurrent(a, stream) : e;
}

}  // namespace lte
