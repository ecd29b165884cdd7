// dv_kv_evict: of each (layer, sequence, key head) the rows that received most weight stay,
// beside the first and the last ones, and are moved together in place.
//
// One kernel, a CTA or a cluster of them for a (layer, sequence, key head): it finds the rows,
// then copies them, so that some CTAs' search runs under others' copies.
//
// The search: of the candidates, the rows between the first and the last ones, those with the
// `need` largest weights.  A weight's bits, turned so that they order as the numbers do, are
// looked at 11 at a time from the top: a histogram of the candidates that agree with the border
// so far says which value the next 11 bits of the border have and how many of the candidates at
// it still fit; it ends early when all of them do.  Each kept row's place is the number of kept
// ones before it, those above the border and of those at it the first that fit.  The weights
// are read once and stay in shared memory; in a cluster each CTA takes a run of the rows, and
// the histograms and counts are added through distributed shared memory.  Weights that are more
// than a cluster's shared memory holds (409600) one CTA reads again in each pass.
//
// The copy: row i <- row keep[i] >= i, of K and V.  A CTA takes slices of the rows' 16-byte
// chunks and walks the destinations upwards; a step's reads come before its writes, and later
// steps read rows past what earlier ones have written.
//
// Bound by memory, and on K by the rate of DRAM accesses: in the x-interleaved layout a kept row's
// chunk is 16 bytes between others that go, of which a miss fetches 64.  Measured, calls in a
// loop: the rows of 8 sequences x 40 heads of 128 halved in 8 layers (1.79 GB asked for) 344 us (like
// rows of 1-, 2- and 4-byte elements 199, 338, 648); two contexts of 110000 rows cut to a tenth, 8 heads of 128, 4
// layers (0.86 GB asked for, 1.2 GB of DRAM traffic, 12.5 million K chunks) 340 to 345 us; two of
// 450000 rows, beyond shared memory, cut to 20000, 2 heads of 64, 0.92 ms; in a replayed graph, 8
// sequences x 25 heads brought from 433 to 400 rows 14.2 us (17 in a loop, the host's call).  Tried
// and slower: the search a launch of its own (413, 654, 16.4 us); K chunks by whole lines (436 us on
// the long contexts); the weights read again from the caches in each pass, four CTAs of 256
// threads an SM (437, 401, 24 us).
#include <algorithm>

#include "dv_ops.h"

namespace dv {
namespace {

constexpr int kEvictThreads = 512;  // two CTAs an SM
constexpr int kWarps = kEvictThreads / 32;
constexpr int kCells = 8;           // 16-byte chunks in flight per thread
constexpr int kBins = 2048;         // of 11 bits of a key
constexpr int kMaxCluster = 8;      // CTAs of a unit
constexpr int kHeld = 24 * 1024;    // weights of a CTA in shared memory, where two fit an SM
constexpr int kMostHeld = 50 * 1024;
constexpr int kLeastRun = 512;      // rows of a CTA below which a unit has no more of them

template <int MAXB>
struct EvictTable {
  int32_t batch;
  int32_t rows[MAXB];     // rows in use
  int32_t pre[MAXB + 1];  // kept rows of the sequences before
};

template <int MAXB>
struct EvictParams {
  uint4* k;
  uint4* v;
  const float* mass;
  float* mass_out;  // may be mass
  int32_t* keep;    // [layer][H][T]
  int64_t layer_chunks;
  int32_t l0, H, C, S, sinks, recent;
  int32_t ctas;           // of a unit
  int32_t slice, slices;  // chunks that a CTA copies at a time, slices of a row
  EvictTable<MAXB> seq;
};

// A weight's place in the order: NaN above all numbers, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return ~0u;
  return u ^ ((u >> 31) ? ~0u : 0x80000000u);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word (four words) at the same place in another CTA's shared memory.
__device__ __forceinline__ uint32_t remote_word(const uint32_t* mine, int rank) {
  uint32_t addr, x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(addr)
               : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint4 remote_words(const uint32_t* mine, int rank) {
  uint32_t addr;
  uint4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(addr)
               : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

// A 16-byte load whose miss fetches 64 bytes from memory: of K's chunk rows a few scattered
// chunks are read.
__device__ __forceinline__ uint4 load_sparse(const uint4* src) {
  uint4 x;
  asm volatile("ld.global.cg.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(src)
               : "memory");
  return x;
}

// HELD: the weights are in shared memory (else they are more than a cluster's holds: one CTA
// of it searches, and reads them from memory each time).
template <int MAXB, bool HELD>
__global__ __launch_bounds__(kEvictThreads, 2) void evict_kernel(
    const __grid_constant__ EvictParams<MAXB> p) {
  extern __shared__ float held[];
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ uint32_t border[3];  // the bits found, how many at them fit, how many there are
  __shared__ uint32_t sums[kWarps];
  __shared__ uint2 totals[2][kWarps];
  __shared__ uint32_t counts[2];  // of this CTA: rows above the border and at it
  ops_pdl_enter();
  const int ctas = p.ctas, rank = (int)(blockIdx.x % ctas), unit = blockIdx.x / ctas;
  const int B = p.seq.batch, b = unit % B, lh = unit / B;
  const int l = lh / p.H, h = lh - l * p.H;
  const int n = p.seq.rows[b], m = p.seq.pre[b + 1] - p.seq.pre[b];
  const int64_t at = (((int64_t)l * B + b) * p.H + h) * p.S;
  const float* const mass = p.mass + at;
  float* const out = p.mass_out + at;
  int32_t* const keep = p.keep + (int64_t)lh * p.seq.pre[B] + p.seq.pre[b];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const auto sync = [&]() {  // of the CTAs that search
    if (HELD && ctas > 1) cluster_sync(); else __syncthreads();
  };
  // this CTA's rows [lo, hi)
  const int run = HELD || n == m ? (n + ctas - 1) / ctas : n;
  const int lo = min(rank * run, n), hi = min(lo + run, n);
  if (n == m) {  // (the same for every CTA of the cluster)
    for (int i = lo + tid; i < hi; i += kEvictThreads) keep[i] = i;
    if (out == mass) return;
#pragma unroll 1
    for (int i0 = lo + tid; i0 < hi; i0 += kEvictThreads * kCells) {
      float x[kCells];
#pragma unroll
      for (int u = 0; u < kCells; ++u)
        x[u] = i0 + u * kEvictThreads < hi ? mass[i0 + u * kEvictThreads] : 0.f;
#pragma unroll
      for (int u = 0; u < kCells; ++u)
        if (i0 + u * kEvictThreads < hi) out[i0 + u * kEvictThreads] = x[u];
    }
    return;
  }
  if (HELD) {
#pragma unroll 8
    for (int i = lo + tid; i < hi; i += kEvictThreads) held[i - lo] = mass[i];
    __syncthreads();
  }
  const auto weight = [&](int i) { return HELD ? held[i - lo] : mass[i]; };

  const bool listed = ctas == 1 && m <= kBins;  // the list is kept in place of the histogram too
  if (HELD || rank == 0) {
    // ---- the border ----
    const int c0 = p.sinks, c1 = n - p.recent;
    uint32_t need = m - p.sinks - p.recent, bits = 0, mask = 0;
    bool fit = false;  // all of those at the border
    if (need == 0) {
      bits = mask = ~0u;
    } else {
#pragma unroll 1
      for (int shift = 21;; shift = shift == 21 ? 10 : 0) {  // 11, 11 and the last 10 bits
        const uint32_t field = shift == 0 ? 1023u : 2047u;
#pragma unroll
        for (int i = tid; i < kBins; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int i = max(lo, c0) + tid; i < min(hi, c1); i += kEvictThreads) {
          const uint32_t key = order_key(weight(i));
          if ((key & mask) == bits) atomicAdd(&hist[key >> shift & field], 1u);
        }
        sync();
        // four bins a thread, the largest first
        const uint32_t* const bins = &hist[kBins - 4 - 4 * tid];
        uint4 four = make_uint4(0, 0, 0, 0);
        if (HELD && ctas > 1) {
          uint4 of[kMaxCluster];
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            of[r] = r < ctas ? remote_words(bins, r) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            four = make_uint4(four.x + of[r].x, four.y + of[r].y, four.z + of[r].z, four.w + of[r].w);
        } else {
          four = *reinterpret_cast<const uint4*>(bins);
        }
        const uint32_t mine[4] = {four.w, four.z, four.y, four.x};
        const uint32_t sum = (four.x + four.y) + (four.z + four.w);
        uint32_t before = sum;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const uint32_t x = __shfl_up_sync(~0u, before, d);
          if (lane >= d) before += x;
        }
        if (lane == 31) sums[warp] = before;
        sync();  // (the histograms have been read)
        before -= sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) before += w < warp ? sums[w] : 0;
        if (before < need && need <= before + sum) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (before < need && need <= before + mine[e]) {
              border[0] = kBins - 1 - 4 * tid - e;
              border[1] = need - before;
              border[2] = mine[e];
            }
            before += mine[e];
          }
        }
        __syncthreads();
        bits |= border[0] << shift;
        mask |= field << shift;
        need = border[1];
        fit = border[2] == need;
        if (shift == 0 || fit) break;
      }
    }

    // ---- places: kept rows before each one ----
    const auto side = [&](int i, int end, float x, bool* above, bool* level) {
      const uint32_t key = order_key(x) & mask;
      const bool candidate = i >= c0 && i < c1;
      *above = i < end && (!candidate || key > bits || (fit && key == bits));
      *level = !fit && i < end && candidate && key == bits;
    };
    const uint32_t lower = (1u << lane) - 1;
    if constexpr (HELD) {
      // a warp's rows [w0, w1)
      const int part = ((run + kWarps - 1) / kWarps + 31) & ~31;
      const int w0 = min(lo + warp * part, hi), w1 = min(w0 + part, hi);
      uint32_t a = 0, e = 0;
#pragma unroll 4
      for (int i0 = w0; i0 < w1; i0 += 32) {
        bool up, eq;
        side(i0 + lane, w1, i0 + lane < w1 ? weight(i0 + lane) : 0.f, &up, &eq);
        a += up;
        e += eq;
      }
      a = __reduce_add_sync(~0u, a);
      e = __reduce_add_sync(~0u, e);
      if (lane == 0) totals[0][warp] = make_uint2(a, e);
      __syncthreads();
      a = e = 0;
      uint32_t all_a = 0, all_e = 0;
      for (int w = 0; w < kWarps; ++w) {
        const uint2 t = totals[0][w];
        if (w < warp) {
          a += t.x;
          e += t.y;
        }
        all_a += t.x;
        all_e += t.y;
      }
      if (ctas > 1) {
        if (tid == 0) {
          counts[0] = all_a;
          counts[1] = all_e;
        }
        cluster_sync();
#pragma unroll
        for (int r = 0; r < kMaxCluster - 1; ++r) {
          a += r < rank ? remote_word(&counts[0], r) : 0;
          e += r < rank ? remote_word(&counts[1], r) : 0;
        }
      }
      // (every weight has been read from memory: they may be overwritten)
#pragma unroll 2
      for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const float x = i < w1 ? weight(i) : 0.f;
        bool up, eq;
        side(i, w1, x, &up, &eq);
        const uint32_t ups = __ballot_sync(~0u, up);
        uint32_t to = a + __popc(ups & lower);
        if (!fit) {
          const uint32_t eqs = __ballot_sync(~0u, eq), at_i = e + __popc(eqs & lower);
          to += min(at_i, need);
          up |= eq && at_i < need;
          e += __popc(eqs);
        }
        if (up) {
          keep[to] = i;
          if (listed) hist[to] = i;
          out[to] = x;
        }
        a += __popc(ups);
      }
    } else {
      // in order of rows, so that none is overwritten before it is read
      uint32_t above = 0, level = 0;
      for (int base = 0, turn = 0; base < n; base += kEvictThreads, turn ^= 1) {
        const int i = base + tid;
        const float x = i < n ? mass[i] : 0.f;
        bool up, eq;
        side(i, n, x, &up, &eq);
        const uint32_t ups = __ballot_sync(~0u, up), eqs = __ballot_sync(~0u, eq);
        if (lane == 0) totals[turn][warp] = make_uint2(__popc(ups), __popc(eqs));
        __syncthreads();
        uint32_t a = above, e = level;
        for (int w = 0; w < kWarps; ++w) {
          const uint2 t = totals[turn][w];
          if (w < warp) {
            a += t.x;
            e += t.y;
          }
          above += t.x;
          level += t.y;
        }
        a += __popc(ups & lower);
        e += __popc(eqs & lower);
        if (up || (eq && e < need)) {
          const uint32_t to = a + (fit ? 0 : min(e, need));
          keep[to] = i;
          if (listed) hist[to] = i;
          out[to] = x;
        }
      }
      __syncthreads();
    }
    for (int i = max(m, lo) + tid; i < hi; i += kEvictThreads) out[i] = 0.f;
  }
  // the list is complete (and no CTA leaves while others read its counts)
  if (ctas > 1) cluster_sync(); else __syncthreads();

  // ---- the copy ----
#pragma unroll 1
  for (int part = rank; part < 2 * p.slices; part += ctas) {
    const bool is_k = part < p.slices;
    const int c0 = (is_k ? part : part - p.slices) * p.slice, cw = min(p.slice, p.C - c0);
    uint4* const base = (is_k ? p.k : p.v) + (p.l0 + l) * p.layer_chunks +
                        ((int64_t)b * p.H + h) * p.C * p.S;
    const int step = kEvictThreads * kCells / cw;
#pragma unroll 1
    for (int i0 = 0; i0 < m; i0 += step) {
      const int rows = min(step, m - i0), cells = rows * cw;
      // K: a thread per row, then the next chunk; V: a row's chunks side by side.  The quotient
      // by a multiplication (exact: the cells and the divisor are at most 2^12).
      const uint32_t inner = is_k ? rows : cw, inv = (uint32_t)(((1ull << 32) + inner - 1) / inner);
      uint4 y[kCells];
      int64_t to[kCells];
#pragma unroll
      for (int u = 0; u < kCells; ++u) {
        const uint32_t j = u * kEvictThreads + tid;
        to[u] = -1;
        if (j < (uint32_t)cells) {
          const int outer = inner == 1 ? (int)j : (int)__umulhi(j, inv), rest = (int)(j - outer * inner);
          const int dst = i0 + (is_k ? rest : outer), c = c0 + (is_k ? outer : rest);
          const int src = listed ? (int)hist[dst] : keep[dst];
          if (src > dst) {
            const int64_t row = is_k ? (int64_t)c * p.S : c, pitch = is_k ? 1 : p.C;
            y[u] = is_k ? load_sparse(base + row + src) : base[row + src * pitch];
            to[u] = row + dst * pitch;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCells; ++u)
        if (to[u] >= 0) base[to[u]] = y[u];
    }
  }
}

template <int MAXB>
void fill_table(const Plan& p, EvictTable<MAXB>* t) {  // the plan's ranges: [kept, rows)
  t->batch = p.B;
  t->pre[0] = 0;
  for (int b = 0; b < p.B; ++b) {
    t->rows[b] = p.seq_start[b] + p.seq_len[b];
    t->pre[b + 1] = t->pre[b] + p.seq_start[b];
  }
}

template <int MAXB, bool HELD>
cudaError_t launch_kernel(const EvictParams<MAXB>& kp, int64_t units, size_t smem,
                          cudaStream_t stream) {
  void (*const kernel)(EvictParams<MAXB>) = evict_kernel<MAXB, HELD>;
  cudaError_t err = cudaSuccess;
  if (HELD)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostHeld * 4);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * kp.ctas));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)kp.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kp.ctas > 1 ? 2 : 1;
  err = cudaLaunchKernelEx(&cfg, kernel, kp);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int MAXB>
cudaError_t launch_evict(const Plan& p, int32_t sinks, int32_t recent, const float* mass,
                         float* mass_out, int32_t* keep, cudaStream_t stream) {
  EvictParams<MAXB> kp;
  kp.k = static_cast<uint4*>(p.k);
  kp.v = static_cast<uint4*>(p.v);
  kp.mass = mass;
  kp.mass_out = mass_out;
  kp.keep = keep;
  kp.layer_chunks = p.layer_chunks;
  kp.l0 = p.l0;
  kp.H = p.H;
  kp.C = p.C;
  kp.S = p.S;
  kp.sinks = sinks;
  kp.recent = recent;
  fill_table(p, &kp.seq);
  // As many CTAs a unit as hold its weights, and where there are few units as fill the SMs
  // with runs of kLeastRun rows.  Sequences that keep all have no say in the first: one of 131072
  // rows beside 31 brought from 2000 to 1000, 8 heads of 64, 39 us (53 with a mass_out of its
  // own); with clusters as for its rows, 170.
  const int64_t units = (int64_t)(p.l1 - p.l0) * p.H * p.B;
  int32_t most = 0, longest = 0;  // rows of a unit that searches; of one that moves weights
  for (int b = 0; b < p.B; ++b) {
    if (p.seq_len[b] > 0) most = std::max(most, kp.seq.rows[b]);
    if (p.seq_len[b] > 0 || mass_out != mass) longest = std::max(longest, kp.seq.rows[b]);
  }
  const int64_t places = 2 * sm_count();  // two CTAs an SM
  int ctas = 1;
  while (ctas < kMaxCluster && (most > ctas * kHeld || (longest > ctas * kLeastRun &&
                                                        units * ctas * 2 <= places)))
    ctas *= 2;
  kp.ctas = ctas;
  const int64_t run = ((int64_t)most + ctas - 1) / ctas;
  const bool held = run <= kMostHeld;
  // Slices of K and of V, 32 to 256 bytes of a row each (16 where it has no more), which a unit's
  // CTAs take in turn, K's first.  With heads of 128 each of 8 CTAs gets one of K and one of V;
  // with heads of 64, 4 slices of each, half of them copy K alone and half V (two contexts of
  // 110000 cut to 12000, 8 heads, 4 layers: 211 us).
  int slices = std::max((p.C + 15) / 16, kp.ctas);
  kp.slice = std::max((p.C + slices - 1) / slices, std::min(2, p.C));
  kp.slices = (p.C + kp.slice - 1) / kp.slice;
  return held ? launch_kernel<MAXB, true>(kp, units, (size_t)run * 4, stream)
              : launch_kernel<MAXB, false>(kp, units, 0, stream);
}

}  // namespace
}  // namespace dv

extern "C" dv_status dv_kv_evict(const dv_cache* cache, int32_t l0, int32_t l1,
                                 const int32_t* rows, const int32_t* kept, int32_t sinks,
                                 int32_t recent, const float* mass, float* mass_out, int32_t* keep,
                                 int64_t count, dv_stream stream) {
  dv::Trace trace("dv_kv_evict");
  dv::Plan p;  // of the rows that go, in number: [kept, rows)
  dv_status st = dv::check_max_seq(cache);
  if (st == DV_OK) st = dv::plan_ranges(cache, l0, l1, kept, rows, &p);
  if (st != DV_OK) return st;
  if (sinks < 0 || recent < 0)
    return dv::fail(DV_ERR_INVALID_ARG, "%d first and %d last rows", sinks, recent);
  int64_t total = 0, used = 0;
  for (int b = 0; b < p.B; ++b) {
    if (p.seq_len[b] > 0 && (int64_t)sinks + recent > p.seq_start[b])
      return dv::fail(DV_ERR_INVALID_ARG,
                      "sequence %d keeps %d rows, fewer than the %d first and %d last", b,
                      p.seq_start[b], sinks, recent);
    total += p.seq_start[b];
    used += (int64_t)p.seq_start[b] + p.seq_len[b];
  }
  const int64_t heads = (int64_t)(l1 - l0) * p.H;
  if (heads > INT32_MAX / p.B || heads * p.B > INT32_MAX / (2 * std::max(dv::kMaxCluster, (p.C + 1) / 2)) ||
      total > INT32_MAX)
    return dv::fail(DV_ERR_UNSUPPORTED, "%d layers, %d sequences, %d heads of %d chunks, %lld rows",
                    l1 - l0, p.B, p.H, p.C, (long long)total);
  if (count != heads * total)
    return dv::fail(DV_ERR_INVALID_ARG, "keep holds %lld entries, not %lld", (long long)count,
                    (long long)(heads * total));
  if (heads == 0 || used == 0) return DV_OK;
  const size_t nm = (size_t)heads * p.B * p.S * 4, nk = (size_t)count * 4;
  if (mass_out != mass && dv::overlap(mass_out, nm, mass, nm))
    return dv::fail(DV_ERR_INVALID_ARG, "mass_out overlaps mass and is not the same");
  if (dv::overlap(keep, nk, mass, nm) || dv::overlap(keep, nk, mass_out, nm))
    return dv::fail(DV_ERR_INVALID_ARG, "keep overlaps the weights");
  if (dv::overlaps_layers(p, keep, nk) || dv::overlaps_layers(p, mass, nm) ||
      dv::overlaps_layers(p, mass_out, nm))
    return dv::fail(DV_ERR_INVALID_ARG, "keep or the weights overlap a layer that the call moves rows of");
  if ((st = dv::resolve_layers(&p)) != DV_OK) return st;
  void *m = nullptr, *o = nullptr, *k = nullptr;
  if ((st = dv::resolve_words(mass, nm, 4, "mass", &m)) != DV_OK) return st;
  if ((st = dv::resolve_words(mass_out, nm, 4, "mass_out", &o)) != DV_OK) return st;
  if (nk > 0 && (st = dv::resolve_words(keep, nk, 4, "keep", &k)) != DV_OK) return st;
  const cudaError_t err =
      p.B <= dv::kSmallBatch
          ? dv::launch_evict<dv::kSmallBatch>(p, sinks, recent, static_cast<const float*>(m),
                                              static_cast<float*>(o), static_cast<int32_t*>(k),
                                              stream)
          : dv::launch_evict<dv::kMaxBatch>(p, sinks, recent, static_cast<const float*>(m),
                                            static_cast<float*>(o), static_cast<int32_t*>(k),
                                            stream);
  return err == cudaSuccess ? DV_OK : dv::cuda_fail(err, "evict launch");
}
