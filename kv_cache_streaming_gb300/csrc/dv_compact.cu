// dv_kv_compact: cache rows moved towards the front of their range, in place.
//
// A pure copy: row s + i <- row keep[i] >= s + i, for K and V of every layer
// and head.  A row's 16-byte chunks move independently, so the unit of work is
// a warp with a slice of a (layer, K|V, sequence, head)'s chunks.  The warp
// walks the destinations upwards in steps of as many rows as fill 16 chunks a
// lane, and reads a whole step before it writes it.  In place this is safe:
// later steps read rows at or past their own destinations, which earlier steps
// have not written.  Bound by memory: on the x-interleaved K side a lane per
// row (a step's destinations are contiguous runs per chunk row), on the V side
// a row's chunks side by side.  An accepted path of a few rows is bound by the
// 16-byte K accesses, each a 32-byte sector of its own.
// Measured: a window of 300 to 509 rows moved down in 24 layers x 8 sequences x
// 25 heads of 64 (1.07 GB) 185 us, 5.8 TB/s; accepted paths of 4 to 8 rows in 8 layers
// x 8 x 40 heads of 128 (15 MB asked for, 22 MB of sectors) 6.3 us.
#include "dv_ops.h"

namespace dv {
namespace {

constexpr int kCompactThreads = 256;
constexpr int kCells = 16;  // 16-byte chunks in flight per lane; 4 where the longest range needs no more

template <int MAXB>
struct CompactParams {
  uint4* k;
  uint4* v;
  const int32_t* keep;
  int64_t layer_chunks;
  int64_t units;  // warps of work
  int32_t l0, H, C, S;
  int32_t slice, slices;  // chunks of a warp, slices of a row
  SeqTable<MAXB> seq;
};

template <int U, int MAXB>
__global__ __launch_bounds__(kCompactThreads) void compact_kernel(
    const __grid_constant__ CompactParams<MAXB> p) {
  ops_pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kCompactThreads / 32) + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  // unit = ((layer * 2 + kv) * batch + b) * H * slices + h * slices + slice
  const int per_seq = p.H * p.slices;
  const int64_t lkvb = unit / per_seq;
  const int hs = (int)(unit - lkvb * per_seq);
  const int h = hs / p.slices, c0 = (hs - h * p.slices) * p.slice;
  const int64_t lkv = lkvb / p.seq.batch;
  const int b = (int)(lkvb - lkv * p.seq.batch);
  const bool is_k = (lkv & 1) == 0;
  const int s = p.seq.start[b], t0 = p.seq.pre[b], n = p.seq.pre[b + 1] - t0;
  const int cw = min(p.slice, p.C - c0);
  uint4* base = (is_k ? p.k : p.v) + (p.l0 + (lkv >> 1)) * p.layer_chunks +
                ((int64_t)b * p.H + h) * p.C * p.S;
  const int step = U * 32 / cw;
  for (int i0 = 0; i0 < n; i0 += step) {
    const int m = min(step, n - i0);  // rows of this step
    const int cells = m * cw;
    // K: a lane per row, then the next chunk; V: a row's chunks side by side.  The
    // quotient by a multiplication (j and the divisor are at most 512).
    const uint32_t inner = is_k ? m : cw, inv = ((1u << 20) + inner - 1) / inner;
    uint4 x[U];
    int64_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = u * 32 + lane;
      to[u] = -1;
      if (j < (uint32_t)cells) {
        const int outer = (int)((j * inv) >> 20), rest = (int)(j - outer * inner);
        const int i = is_k ? rest : outer, c = c0 + (is_k ? outer : rest);
        const int dst = s + i0 + i, src = __ldg(p.keep + t0 + i0 + i);
        if (src > dst && src < p.S) {  // an entry outside this leaves its row alone
          const int64_t row = is_k ? (int64_t)c * p.S : c, pitch = is_k ? 1 : p.C;
          x[u] = base[row + src * pitch];
          to[u] = row + dst * pitch;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) base[to[u]] = x[u];
    __syncwarp();
  }
}

template <int MAXB>
cudaError_t launch_compact(const Plan& p, const int32_t* keep, cudaStream_t stream) {
  CompactParams<MAXB> kp;
  kp.k = static_cast<uint4*>(p.k);
  kp.v = static_cast<uint4*>(p.v);
  kp.keep = keep;
  kp.layer_chunks = p.layer_chunks;
  kp.l0 = p.l0;
  kp.H = p.H;
  kp.C = p.C;
  kp.S = p.S;
  fill_table(p, &kp.seq);
  // A row's chunks stay with one warp (V rows are then contiguous runs), 16 at
  // most; few and long ranges are cut finer, down to a 32-byte sector, until
  // 16 warps an SM have work.
  const int64_t rows = 2 * (int64_t)(p.l1 - p.l0) * p.B * p.H;
  int slice = p.C < 16 ? p.C : 16;
  while (slice > 2 && (int64_t)p.max_len * slice > kCells * 32 &&
         rows * ((p.C + slice - 1) / slice) < 152 * 16)
    slice = (slice + 1) / 2;
  kp.slice = slice;
  kp.slices = (p.C + slice - 1) / slice;
  kp.units = rows * kp.slices;
  const int64_t ctas = (kp.units + kCompactThreads / 32 - 1) / (kCompactThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  // Few rows (an accepted path): a quarter of the registers, so that more warps are resident
  // (paths of 4 to 8 rows in 8 layers x 8 x 40 heads of 128: 6.3 us, 9.4 with 16 cells a lane).
  if ((int64_t)p.max_len * slice <= 4 * 32)
    return ops_launch(compact_kernel<4, MAXB>, dim3((unsigned)ctas), kCompactThreads, 0, stream,
                      kp);
  return ops_launch(compact_kernel<kCells, MAXB>, dim3((unsigned)ctas), kCompactThreads, 0, stream,
                    kp);
}

}  // namespace
}  // namespace dv

extern "C" dv_status dv_kv_compact(const dv_cache* cache, int32_t l0, int32_t l1,
                                   const int32_t* seq_start, const int32_t* seq_end,
                                   const int32_t* keep, int64_t count, dv_stream stream) {
  dv::Trace trace("dv_kv_compact");
  dv::Plan p;
  dv_status st = dv::plan_ranges(cache, l0, l1, seq_start, seq_end, &p);
  if (st != DV_OK) return st;
  if (count != p.tokens)
    return dv::fail(DV_ERR_INVALID_ARG, "keep holds %lld entries, the ranges %lld",
                    (long long)count, (long long)p.tokens);
  if (p.bytes == 0) return DV_OK;
  if ((int64_t)p.H * p.C > INT32_MAX / 2 || 2 * (int64_t)(l1 - l0) * p.B * p.H > INT32_MAX)
    return dv::fail(DV_ERR_UNSUPPORTED, "%d layers, %d sequences, %d heads of %d chunks", l1 - l0,
                    p.B, p.H, p.C);
  if (dv::overlaps_layers(p, keep, (size_t)p.tokens * 4))
    return dv::fail(DV_ERR_INVALID_ARG, "keep overlaps a layer that the call moves rows of");
  if ((st = dv::resolve_layers(&p)) != DV_OK) return st;
  void* dev = nullptr;
  if ((st = dv::resolve_words(keep, (size_t)p.tokens * 4, 4, "keep", &dev)) != DV_OK) return st;
  const int32_t* kd = static_cast<const int32_t*>(dev);
  const cudaError_t err = p.B <= dv::kSmallBatch
                              ? dv::launch_compact<dv::kSmallBatch>(p, kd, stream)
                              : dv::launch_compact<dv::kMaxBatch>(p, kd, stream);
  return err == cudaSuccess ? DV_OK : dv::cuda_fail(err, "compact launch");
}
