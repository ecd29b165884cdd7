// dv_kv_evict: of each (layer, sequence, key head) the rows that received most weight stay,
// beside the first and the last ones, and are moved together in place.
//
// select_kernel finds a unit's rows: of the candidates, the rows between the first and the
// last ones, those with the `need` largest weights.  A weight's bits, turned so that they order
// as the numbers do, are looked at 8 at a time from the top: a histogram of the candidates that
// agree with the border so far says which value the next 8 bits of the border have and how
// many of the candidates at it still fit.  Then one pass in order of rows gives each kept row
// its place (the kept ones before it: those above the border, and of those at it the first that
// fit) and moves the weights.
//
// move_kernel is a pure copy of K and V rows, row i <- row keep[i] >= i.  A CTA takes a slice of
// the 16-byte chunks of a (layer, K|V, sequence, key head)'s rows and walks the destinations
// upwards; a step's reads come before its writes, and later steps read rows past what earlier
// ones have written.  Bound by memory.
#include "dv_ops.h"

namespace dv {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveCells = 8;  // 16-byte chunks in flight per thread

template <int MAXB>
struct EvictTable {
  int32_t batch;
  int32_t rows[MAXB];     // rows in use
  int32_t pre[MAXB + 1];  // kept rows of the sequences before
};

template <int MAXB>
struct SelectParams {
  const float* mass;
  float* mass_out;  // may be mass
  int32_t* keep;    // [layer][H][T]
  int32_t H, S, sinks, recent;
  EvictTable<MAXB> seq;
};

// A weight's place in the order: NaN above all numbers, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return ~0u;
  return u ^ ((u >> 31) ? ~0u : 0x80000000u);
}

template <int MAXB>
__global__ __launch_bounds__(kSelectThreads) void select_kernel(
    const __grid_constant__ SelectParams<MAXB> p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t border[3];  // the bits found, how many at them fit, how many there are
  __shared__ uint2 totals[2][kSelectWarps];
  ops_pdl_enter();
  const int B = p.seq.batch, b = blockIdx.x % B, lh = blockIdx.x / B;
  const int l = lh / p.H, h = lh - l * p.H;
  const int n = p.seq.rows[b], m = p.seq.pre[b + 1] - p.seq.pre[b];
  const int64_t at = (((int64_t)l * B + b) * p.H + h) * p.S;
  const float* const mass = p.mass + at;
  float* const out = p.mass_out + at;
  int32_t* const keep = p.keep + (int64_t)lh * p.seq.pre[B] + p.seq.pre[b];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (n == m) {
    for (int i = tid; i < n; i += kSelectThreads) {
      keep[i] = i;
      out[i] = mass[i];
    }
    return;
  }
  const int c0 = p.sinks, c1 = n - p.recent;
  uint32_t need = m - p.sinks - p.recent, bits = 0, mask = 0;
  if (need == 0) {
    bits = mask = ~0u;
  } else {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = c0 + tid; i < c1; i += kSelectThreads) {
        const uint32_t key = order_key(mass[i]);
        if ((key & mask) == bits) atomicAdd(&hist[key >> shift & 255], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // a lane's eight values, the largest first
        uint32_t mine[8], sum = 0;
        for (int e = 0; e < 8; ++e) sum += mine[e] = hist[255 - 8 * lane - e];
        uint32_t before = sum;
        for (int d = 1; d < 32; d *= 2) {
          const uint32_t x = __shfl_up_sync(~0u, before, d);
          if (lane >= d) before += x;
        }
        before -= sum;
        for (int e = 0; e < 8; ++e) {
          if (before < need && need <= before + mine[e]) {
            border[0] = 255 - 8 * lane - e;
            border[1] = need - before;
            border[2] = mine[e];
          }
          before += mine[e];
        }
      }
      __syncthreads();
      bits |= border[0] << shift;
      mask |= 255u << shift;
      need = border[1];
      if (border[2] == need) break;  // all of them fit
    }
  }
  // Places: kept rows before this one.
  uint32_t above = 0, level = 0;  // above the border (or first, or last), and at it, so far
  for (int base = 0, turn = 0; base < n; base += kSelectThreads, turn ^= 1) {
    const int i = base + tid;
    const float x = i < n ? mass[i] : 0.f;
    const uint32_t key = order_key(x) & mask;
    const bool candidate = i >= c0 && i < c1;
    const bool hi = i < n && (!candidate || key > bits), eq = candidate && key == bits;
    const uint32_t his = __ballot_sync(~0u, hi), eqs = __ballot_sync(~0u, eq);
    if (lane == 0) totals[turn][warp] = make_uint2(__popc(his), __popc(eqs));
    __syncthreads();
    uint32_t a = above, e = level;
    for (int w = 0; w < kSelectWarps; ++w) {
      const uint2 t = totals[turn][w];
      if (w < warp) {
        a += t.x;
        e += t.y;
      }
      above += t.x;
      level += t.y;
    }
    a += __popc(his & ((1u << lane) - 1));
    e += __popc(eqs & ((1u << lane) - 1));
    if (hi || (eq && e < need)) {
      const uint32_t to = a + min(e, need);
      keep[to] = i;
      out[to] = x;
    }
  }
  __syncthreads();
  for (int i = m + tid; i < n; i += kSelectThreads) out[i] = 0.f;
}

template <int MAXB>
struct MoveParams {
  uint4* k;
  uint4* v;
  const int32_t* keep;
  int64_t layer_chunks;
  int32_t l0, H, C, S;
  int32_t slice, slices;  // chunks of a CTA, slices of a row
  EvictTable<MAXB> seq;
};

template <int MAXB>
__global__ __launch_bounds__(kMoveThreads) void move_kernel(
    const __grid_constant__ MoveParams<MAXB> p) {
  ops_pdl_enter();
  // block = (((layer * 2 + kv) * batch + b) * H + h) * slices + slice
  int64_t x = blockIdx.x;
  const int slice = (int)(x % p.slices);
  x /= p.slices;
  const int h = (int)(x % p.H);
  x /= p.H;
  const int b = (int)(x % p.seq.batch);
  x /= p.seq.batch;
  const bool is_k = (x & 1) == 0;
  const int l = (int)(x >> 1);
  const int n = p.seq.rows[b], m = p.seq.pre[b + 1] - p.seq.pre[b];
  if (n == m) return;
  const int c0 = slice * p.slice, cw = min(p.slice, p.C - c0);
  uint4* const base = (is_k ? p.k : p.v) + (p.l0 + l) * p.layer_chunks +
                      ((int64_t)b * p.H + h) * p.C * p.S;
  const int32_t* const keep =
      p.keep + ((int64_t)l * p.H + h) * p.seq.pre[p.seq.batch] + p.seq.pre[b];
  const int step = kMoveThreads * kMoveCells / cw;
  for (int i0 = 0; i0 < m; i0 += step) {
    const int rows = min(step, m - i0), cells = rows * cw;
    uint4 y[kMoveCells];
    int64_t to[kMoveCells];
#pragma unroll
    for (int u = 0; u < kMoveCells; ++u) {
      const int j = u * kMoveThreads + threadIdx.x;
      to[u] = -1;
      if (j < cells) {
        // K: a thread per row, then the next chunk; V: a row's chunks side by side
        const int outer = is_k ? j / rows : j / cw, inner = j - outer * (is_k ? rows : cw);
        const int dst = i0 + (is_k ? inner : outer), c = c0 + (is_k ? outer : inner);
        const int src = keep[dst];
        if (src > dst) {
          const int64_t row = is_k ? (int64_t)c * p.S : c, pitch = is_k ? 1 : p.C;
          y[u] = base[row + src * pitch];
          to[u] = row + dst * pitch;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveCells; ++u)
      if (to[u] >= 0) base[to[u]] = y[u];
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

template <int MAXB>
cudaError_t launch_evict(const Plan& p, int32_t sinks, int32_t recent, const float* mass,
                         float* mass_out, int32_t* keep, cudaStream_t stream) {
  SelectParams<MAXB> sp;
  sp.mass = mass;
  sp.mass_out = mass_out;
  sp.keep = keep;
  sp.H = p.H;
  sp.S = p.S;
  sp.sinks = sinks;
  sp.recent = recent;
  fill_table(p, &sp.seq);
  const int64_t units = (int64_t)(p.l1 - p.l0) * p.H * p.B;
  cudaError_t err = ops_launch(select_kernel<MAXB>, dim3((unsigned)units), kSelectThreads, 0,
                               stream, sp);
  if (err != cudaSuccess || p.tokens == 0) return err;  // no row goes: none is moved
  MoveParams<MAXB> mp;
  mp.k = static_cast<uint4*>(p.k);
  mp.v = static_cast<uint4*>(p.v);
  mp.keep = keep;
  mp.layer_chunks = p.layer_chunks;
  mp.l0 = p.l0;
  mp.H = p.H;
  mp.C = p.C;
  mp.S = p.S;
  mp.seq = sp.seq;
  int slice = p.C < 16 ? p.C : 16;
  while (slice > 2 && 2 * units * ((p.C + slice - 1) / slice) < 152 * 6) slice = (slice + 1) / 2;
  mp.slice = slice;
  mp.slices = (p.C + slice - 1) / slice;
  return ops_launch(move_kernel<MAXB>, dim3((unsigned)(2 * units * mp.slices)), kMoveThreads, 0,
                    stream, mp);
}

}  // namespace
}  // namespace dv

extern "C" dv_status dv_kv_evict(const dv_cache* cache, int32_t l0, int32_t l1,
                                 const int32_t* rows, const int32_t* kept, int32_t sinks,
                                 int32_t recent, const float* mass, float* mass_out, int32_t* keep,
                                 int64_t count, dv_stream stream) {
  dv::Trace trace("dv_kv_evict");
  dv::Plan p;  // of the rows that go, in number: [kept, rows)
  dv_status st = dv::plan_ranges(cache, l0, l1, kept, rows, &p);
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
  if (heads > INT32_MAX / p.B || heads * p.B > INT32_MAX / (2 * ((p.C + 1) / 2)) ||
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
