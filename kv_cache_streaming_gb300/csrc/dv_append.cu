// dv_rope_init and dv_kv_append: rotary positions for the new tokens' queries
// and keys, and their keys and values written to the cache's rows.
//
// Pair i of a head turns by the angle position * f_i:
//   (x, y) -> m (x cos - y sin, x sin + y cos).
// f_i is held in turns per position as a 64-bit binary fraction, so that
// position * f_i mod 1 is one integer product, exact at any position; the top
// 32 bits of it, as a signed fraction of half a turn, go to sincospi.  (A
// float product would round an angle near 10^6 by up to 0.03 rad.)
//
// Memory bound: every value is read once and written once (the half layout's
// partner chunk comes from L1).  Two kernels:
//  * append_tile_kernel: a warp covers 4 consecutive cache rows x 8 chunks of
//    16 bytes, and walks over heads with its lanes' cosines and sines in
//    registers.  On the token-major side that is 128 contiguous bytes a token, on
//    the x-interleaved K side 64 a chunk row: whole 32-byte sectors on both, with
//    no transpose through shared memory.  Row groups start at multiples of 4, so
//    a range's edges alone leave lanes idle.  (451 MB of ragged prompts, 40 heads of
//    128: 72 us, 6.3 TB/s; as 8 rows x 4 chunks 87 us, as 16 x 2 94 us.)
//  * append_token_kernel: decode steps and short trees, a CTA per token and
//    slice of its chunks, the angles' table in shared memory.
#include <type_traits>

#include "dv_ops.h"

namespace dv {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kTileRows = 4;    // cache rows of a warp in the tile kernel
constexpr int kTileChunks = 8;  // and 16-byte chunks of them
// Ranges of fewer tokens than this on average go to the token kernel: the
// tile kernel's lanes are tied to 4 rows, so shorter ranges leave most idle (32 ranges
// of 1 / 3 tokens, 40 heads of 128: 5.4 / 5.9 us there, 2.7 / 4.6 in the token kernel).  By the
// call's tokens the crossover lies higher: 8 to 17 tokens a range there (7.4 and 6.9
// at 8; 12.2 and 12.6 at 17; 31.3 and 35.2 at 64), past 64 with 4 ranges (6.8 and 6.7).
constexpr int kTileMinMean = 4;

template <int MAXB>
struct AppendParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint4* kc;  // K and V of the layer
  uint4* vc;
  const int32_t* positions;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int32_t Hq, H, D, C, S;
  int32_t rot, half;  // rot 0: nothing is rotated; half = rot / 2
  float factor;
  uint64_t turn[DV_MAX_ROT / 2];
  SeqTable<MAXB> seq;
  int32_t group_pre[MAXB + 1];  // tile kernel: row groups before the sequence
};

__device__ __forceinline__ float2 cos_sin(uint64_t turn, int32_t pos, float factor) {
  const int64_t a = (int64_t)((uint64_t)(int64_t)pos * turn);
  // the angle in half turns, in [-1, 1): rounded to 24 bits, at most 2^-25 off
  const float x = (float)(int32_t)(a >> 32) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * factor, s * factor);
}

// How pairs lie in a head's 16-byte chunks.
enum Pairs {
  kNeighbours,  // interleaved: both of a pair in one word
  kHalves,      // the other half's chunk: rot / 2 a multiple of 8
  kAcross       // the other half, at any element
};

// The partners of the 8 elements of chunk c of a head's row x (kHalves, kAcross).
template <Pairs W, typename P>
__device__ __forceinline__ uint4 partner(const P& p, const uint16_t* row, int c) {
  const int d0 = c * 8;
  if constexpr (W == kHalves) {
    return __ldg(reinterpret_cast<const uint4*>(row) +
                 (d0 < p.half ? c + (p.half >> 3) : c - (p.half >> 3)));
  } else {
    uint16_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = d0 + i;
      y[i] = d >= p.rot ? (uint16_t)0 : __ldg(row + (d < p.half ? d + p.half : d - p.half));
    }
    return make_uint4(y[0] | (uint32_t)y[1] << 16, y[2] | (uint32_t)y[3] << 16,
                      y[4] | (uint32_t)y[5] << 16, y[6] | (uint32_t)y[7] << 16);
  }
}

// A chunk's cosines and sines: of its 4 pairs (kNeighbours), or of its 8
// elements with the sign that the partner's sine takes (the first of a pair
// loses y sin, the second gains x sin).
template <Pairs W>
struct Angles {
  static constexpr int N = W == kNeighbours ? 4 : 8;
  float c[N], s[N];
  // `of(f)`: cosine and sine of frequency f; the first n elements rotate
  template <typename P, typename F>
  __device__ __forceinline__ void fill(const P& p, int chunk, int n, F&& of) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = W == kNeighbours ? 2 * i : i, d = chunk * 8 + e;
      c[i] = 1.f;
      s[i] = 0.f;
      if (e < n) {
        const float2 w = of(W == kNeighbours ? d >> 1 : d < p.half ? d : d - p.half);
        c[i] = w.x;
        s[i] = W != kNeighbours && d < p.half ? -w.y : w.y;
      }
    }
  }
};

// 8 elements turned, rounded once; the first n rotate, the others keep their bits.
template <typename T, Pairs W>
__device__ __forceinline__ uint4 rotate(uint4 x, uint4 y, const Angles<W>& a, int n) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = Pack2<T>::unpack(xs[i]);
    uint32_t w;
    if (W == kNeighbours) {
      w = Pack2<T>::pack(fmaf(-u.y, a.s[i], u.x * a.c[i]), fmaf(u.x, a.s[i], u.y * a.c[i]));
      r[i] = 2 * i < n ? w : xs[i];
    } else {
      const float2 v = Pack2<T>::unpack(ys[i]);
      w = Pack2<T>::pack(fmaf(v.x, a.s[2 * i], u.x * a.c[2 * i]),
                         fmaf(v.y, a.s[2 * i + 1], u.y * a.c[2 * i + 1]));
      r[i] = 2 * i + 1 < n ? w : 2 * i < n ? (w & 0xffffu) | (xs[i] & 0xffff0000u) : xs[i];
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// 1024 threads an SM: with the 87 registers the compiler would take, half of
// them kept too few loads in flight (ragged prompts at 2.7 TB/s).
template <typename T, Pairs W, int MAXB>
__global__ __launch_bounds__(kAppendThreads, 8) void append_tile_kernel(
    const __grid_constant__ AppendParams<MAXB> p) {
  ops_pdl_enter();
  const int lane = threadIdx.x & 31;
  const int gid = blockIdx.y * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int parts = (p.C + kTileChunks - 1) / kTileChunks;  // of a head's row
  const int step = (gridDim.y * (kAppendThreads / 32)) / parts;  // warps over the heads
  const int part = gid % parts, h0 = gid / parts;
  if (h0 >= step) return;
  const int b = find_span(p.group_pre, p.seq.batch, blockIdx.x);
  const int s = p.seq.start[b];
  const int row = (s / kTileRows + (blockIdx.x - p.group_pre[b])) * kTileRows + (lane & (kTileRows - 1));
  const int c = part * kTileChunks + lane / kTileRows;
  const int n = p.seq.pre[b + 1] - p.seq.pre[b];
  if (row < s || row >= s + n || c >= p.C) return;
  const int64_t tok = p.seq.pre[b] + (row - s);

  const int nrot = min(8, max(0, p.rot - c * 8));  // rotated elements of the chunk
  Angles<W> ang;
  if (nrot > 0) {
    const int32_t pos = p.positions ? p.positions[tok] : row;
    ang.fill(p, c, nrot, [&](int f) { return cos_sin(p.turn[f], pos, p.factor); });
  }
  // `put(chunk of head h)` for the warp's heads, U of them in flight.
  const auto turned = [&](const uint16_t* base, int heads, auto&& put) {
    constexpr int U = W == kNeighbours ? 4 : 3;
#pragma unroll 1
    for (int h = h0; h < heads; h += U * step) {
      uint4 x[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * step < heads) {
          const uint16_t* r = base + (h + u * step) * p.D;
          x[u] = __ldg(reinterpret_cast<const uint4*>(r) + c);
          y[u] = W == kNeighbours ? x[u] : partner<W>(p, r, c);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * step < heads) put(h + u * step, rotate<T, W>(x[u], y[u], ang, nrot));
    }
  };
  const auto copied = [&](const uint16_t* base, int heads, auto&& put) {
    constexpr int U = 6;
#pragma unroll 1
    for (int h = h0; h < heads; h += U * step) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * step < heads)
          x[u] = __ldg(reinterpret_cast<const uint4*>(base + (h + u * step) * p.D) + c);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * step < heads) put(h + u * step, x[u]);
    }
  };
  uint4* const qo = reinterpret_cast<uint4*>(p.q_out + tok * p.q_out_stride) + c;
  uint4* const kc = p.kc + ((int64_t)b * p.H * p.C + c) * p.S + row;
  uint4* const vc = p.vc + ((int64_t)b * p.H * p.S + row) * p.C + c;
  const auto put_q = [&](int h, uint4 x) { qo[h * p.C] = x; };
  const auto put_k = [&](int h, uint4 x) { kc[(int64_t)h * p.C * p.S] = x; };
  if (nrot > 0) {
    turned(p.q + tok * p.q_stride, p.Hq, put_q);
    turned(p.k + tok * p.k_stride, p.H, put_k);
  } else {
    copied(p.q + tok * p.q_stride, p.Hq, put_q);
    copied(p.k + tok * p.k_stride, p.H, put_k);
  }
  copied(p.v + tok * p.v_stride, p.H,
         [&](int h, uint4 x) { vc[(int64_t)h * p.S * p.C] = x; });
}

template <typename T, Pairs W, int MAXB>
__global__ __launch_bounds__(kAppendThreads) void append_token_kernel(
    const __grid_constant__ AppendParams<MAXB> p) {
  __shared__ float2 table[DV_MAX_ROT / 2];
  ops_pdl_enter();
  const int64_t tok = blockIdx.x;
  const int b = find_span(p.seq.pre, p.seq.batch, blockIdx.x);
  const int row = p.seq.start[b] + (blockIdx.x - p.seq.pre[b]);
  const int32_t pos = p.positions ? p.positions[tok] : row;
  for (int i = threadIdx.x; i < p.half; i += kAppendThreads)
    table[i] = cos_sin(p.turn[i], pos, p.factor);
  __syncthreads();
  const int total = (p.Hq + 2 * p.H) * p.C;
  for (int i = blockIdx.y * kAppendThreads + threadIdx.x; i < total;
       i += gridDim.y * kAppendThreads) {
    const int g = i / p.C, c = i - g * p.C;
    const int kind = g < p.Hq ? 0 : g < p.Hq + p.H ? 1 : 2;
    const int h = kind == 0 ? g : kind == 1 ? g - p.Hq : g - p.Hq - p.H;
    const uint16_t* r = (kind == 0   ? p.q + tok * p.q_stride
                         : kind == 1 ? p.k + tok * p.k_stride
                                     : p.v + tok * p.v_stride) +
                        (int64_t)h * p.D;
    uint4 x = __ldg(reinterpret_cast<const uint4*>(r) + c);
    const int nrot = min(8, max(0, p.rot - c * 8));
    if (kind != 2 && nrot > 0) {
      Angles<W> ang;
      ang.fill(p, c, nrot, [&](int f) { return table[f]; });
      x = rotate<T, W>(x, W == kNeighbours ? x : partner<W>(p, r, c), ang, nrot);
    }
    const int64_t head = (int64_t)b * p.H + h;
    if (kind == 0)
      reinterpret_cast<uint4*>(p.q_out + tok * p.q_out_stride + (int64_t)h * p.D)[c] = x;
    else if (kind == 1)
      p.kc[(head * p.C + c) * p.S + row] = x;
    else
      p.vc[(head * p.S + row) * p.C + c] = x;
  }
}

template <typename T, Pairs W, int MAXB>
cudaError_t launch_append(const Plan& p, const dv_new_tokens& t, cudaStream_t stream) {
  AppendParams<MAXB> kp;
  kp.q = static_cast<const uint16_t*>(t.q);
  kp.k = static_cast<const uint16_t*>(t.k);
  kp.v = static_cast<const uint16_t*>(t.v);
  kp.q_out = static_cast<uint16_t*>(t.q_out);
  kp.kc = static_cast<uint4*>(p.k) + p.l0 * p.layer_chunks;
  kp.vc = static_cast<uint4*>(p.v) + p.l0 * p.layer_chunks;
  kp.positions = t.positions;
  kp.q_stride = t.q_stride;
  kp.k_stride = t.k_stride;
  kp.v_stride = t.v_stride;
  kp.q_out_stride = t.q_out_stride;
  kp.Hq = t.q_heads;
  kp.H = p.H;
  kp.D = p.D;
  kp.C = p.C;
  kp.S = p.S;
  kp.rot = t.rope ? t.rope->rot_dim : 0;
  kp.half = kp.rot / 2;
  kp.factor = t.rope ? t.rope->value_factor : 1.f;
  for (int i = 0; i < kp.half; ++i) kp.turn[i] = t.rope->turn[i];
  fill_table(p, &kp.seq);
  constexpr int kWarps = kAppendThreads / 32;
  const int heads = t.q_heads + 2 * p.H;
  if (p.tokens < (int64_t)kTileMinMean * p.active) {
    const int slices = (int)(((int64_t)heads * p.C + kAppendThreads - 1) / kAppendThreads);
    // one chunk a thread while the grid is small, more once it fills the GPU
    const int fit = (int)((int64_t)152 * 64 / p.tokens);
    const int y = slices < fit ? slices : fit > 1 ? fit : 1;
    return ops_launch(append_token_kernel<T, W, MAXB>, dim3((unsigned)p.tokens, y < 65535 ? y : 65535),
                      kAppendThreads, 0, stream, kp);
  }
  int64_t groups = 0;
  for (int b = 0; b < p.B; ++b) {
    kp.group_pre[b] = (int32_t)groups;
    const int64_t s = p.seq_start[b], e = s + p.seq_len[b];
    if (e > s) groups += (e + kTileRows - 1) / kTileRows - s / kTileRows;
  }
  kp.group_pre[p.B] = (int32_t)groups;
  // Warps over the heads: 4 heads to a warp, about what it has in flight at once (ragged
  // prompts, 40 heads of 128: 72 us; 89 at 2 heads, 76 at 6, 74 at 8).
  const int parts = (p.C + kTileChunks - 1) / kTileChunks;
  const int most_heads = t.q_heads > p.H ? t.q_heads : p.H;
  const int64_t warps = (int64_t)parts * ((most_heads + 3) / 4);
  int64_t y = (warps + kWarps - 1) / kWarps;
  if (y > 65535) y = 65535;
  return ops_launch(append_tile_kernel<T, W, MAXB>, dim3((unsigned)groups, (unsigned)y),
                    kAppendThreads, 0, stream, kp);
}

}  // namespace
}  // namespace dv

using dv::fail;

extern "C" dv_status dv_rope_init(dv_rope* rope, int32_t rot_dim, int32_t interleaved, double base,
                                  int32_t scaling, double factor, int32_t original_max) {
  if (!rope) return fail(DV_ERR_INVALID_ARG, "rope is NULL");
  if (rot_dim < 2 || rot_dim > DV_MAX_ROT || rot_dim % 2 != 0)
    return fail(DV_ERR_INVALID_ARG, "rot_dim %d is not an even number in [2,%d]", rot_dim,
                DV_MAX_ROT);
  if (interleaved != 0 && interleaved != 1)
    return fail(DV_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", interleaved);
  if (!(base > 1.0) || !std::isfinite(base))
    return fail(DV_ERR_INVALID_ARG, "base must be finite and above 1 (got %g)", base);
  if (scaling < DV_ROPE_NONE || scaling > DV_ROPE_PARTS)
    return fail(DV_ERR_INVALID_ARG, "unknown scaling %d", scaling);
  if (scaling != DV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(DV_ERR_INVALID_ARG, "factor must be finite and at least 1 (got %g)", factor);
  if (scaling == DV_ROPE_NTK && rot_dim <= 2)
    return fail(DV_ERR_INVALID_ARG, "DV_ROPE_NTK needs rot_dim above 2");
  if (scaling == DV_ROPE_PARTS && original_max <= 0)
    return fail(DV_ERR_INVALID_ARG, "DV_ROPE_PARTS needs original_max (got %d)", original_max);
  const double two_pi = 6.283185307179586476925;
  if (scaling == DV_ROPE_NTK) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  rope->rot_dim = rot_dim;
  rope->interleaved = interleaved;
  rope->value_factor = scaling == DV_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  rope->reserved = 0;
  for (int i = 0; i < DV_MAX_ROT / 2; ++i) {
    if (i >= rot_dim / 2) {
      rope->turn[i] = 0;
      continue;
    }
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == DV_ROPE_LINEAR) f /= factor;
    if (scaling == DV_ROPE_PARTS) {
      const double g = ((double)original_max * f / two_pi - 1.0) / 31.0;
      const double w = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = w * f + (1.0 - w) * f / factor;
    }
    rope->turn[i] = (uint64_t)std::ldexp(f / two_pi, 64);  // f <= 1: below 0.16 of 2^64
  }
  return DV_OK;
}

extern "C" dv_status dv_kv_append(const dv_cache* cache, int32_t layer, const int32_t* seq_start,
                                  const int32_t* seq_end, const dv_new_tokens* tokens,
                                  dv_stream stream) {
  dv::Trace trace("dv_kv_append");
  if (!tokens) return fail(DV_ERR_INVALID_ARG, "tokens is NULL");
  dv::Plan p;
  dv_status st = dv::plan_layer(cache, layer, seq_start, seq_end, tokens->dtype, &p);
  if (st != DV_OK) return st;
  dv_new_tokens t = *tokens;
  if (t.q_heads < 0 || (int64_t)t.q_heads * p.D > INT32_MAX / 2)
    return fail(DV_ERR_INVALID_ARG, "q_heads is %d", t.q_heads);
  if ((int64_t)p.H * p.D > 1 << 23)  // the tile kernel's grid has a warp for each 64 of a head's
    return fail(DV_ERR_UNSUPPORTED, "%d heads of %d elements", p.H, p.D);
  if (t.rope) {
    if (t.rope->rot_dim < 2 || t.rope->rot_dim > DV_MAX_ROT || t.rope->rot_dim % 2 != 0 ||
        t.rope->rot_dim > p.D)
      return fail(DV_ERR_INVALID_ARG, "rot_dim %d does not fit head_dim %d", t.rope->rot_dim, p.D);
    if (t.rope->interleaved != 0 && t.rope->interleaved != 1)
      return fail(DV_ERR_INVALID_ARG, "rope.interleaved is %d", t.rope->interleaved);
    if (!std::isfinite(t.rope->value_factor))
      return fail(DV_ERR_INVALID_ARG, "rope.value_factor is %g", (double)t.rope->value_factor);
  }
  if (t.tokens != p.tokens)
    return fail(DV_ERR_INVALID_ARG, "the buffers hold %lld tokens, the ranges %lld",
                (long long)t.tokens, (long long)p.tokens);
  if (p.tokens == 0) return DV_OK;
  // What the call writes (q_out and the layer) shares no bytes with what it reads.
  size_t nk = 0, nv = 0, nq = 0, no = 0;
  const size_t np = (size_t)p.tokens * 4;
  if ((st = dv::span_rows(p, p.H, t.k_stride, "k", &nk)) != DV_OK) return st;
  if ((st = dv::span_rows(p, p.H, t.v_stride, "v", &nv)) != DV_OK) return st;
  if (t.q_heads > 0) {
    if ((st = dv::span_rows(p, t.q_heads, t.q_stride, "q", &nq)) != DV_OK) return st;
    if ((st = dv::span_rows(p, t.q_heads, t.q_out_stride, "q_out", &no)) != DV_OK) return st;
    if (dv::overlap(t.q_out, no, t.q, nq) || dv::overlap(t.q_out, no, t.k, nk) ||
        dv::overlap(t.q_out, no, t.v, nv) || dv::overlap(t.q_out, no, t.positions, np))
      return fail(DV_ERR_INVALID_ARG, "q_out overlaps q, k, v or positions");
    if (dv::overlaps_layers(p, t.q_out, no) || dv::overlaps_layers(p, t.q, nq))
      return fail(DV_ERR_INVALID_ARG, "q or q_out overlaps the cache's layer");
  }
  if (dv::overlaps_layers(p, t.k, nk) || dv::overlaps_layers(p, t.v, nv) ||
      dv::overlaps_layers(p, t.positions, np))
    return fail(DV_ERR_INVALID_ARG, "k, v or positions overlaps the cache's layer");
  if ((st = dv::resolve_layers(&p)) != DV_OK) return st;
  void* dev = nullptr;
  if ((st = dv::resolve_words(t.k, nk, 16, "k", &dev)) != DV_OK) return st;
  t.k = dev;
  if ((st = dv::resolve_words(t.v, nv, 16, "v", &dev)) != DV_OK) return st;
  t.v = dev;
  if (t.q_heads > 0) {
    if ((st = dv::resolve_words(t.q, nq, 16, "q", &dev)) != DV_OK) return st;
    t.q = dev;
    if ((st = dv::resolve_words(t.q_out, no, 16, "q_out", &dev)) != DV_OK) return st;
    t.q_out = dev;
  }
  if (t.positions) {
    if ((st = dv::resolve_words(t.positions, np, 4, "positions", &dev)) != DV_OK) return st;
    t.positions = static_cast<const int32_t*>(dev);
  }
  const auto launch = [&](auto elem) {
    using T = decltype(elem);
    const auto batch = [&](auto pairs) {
      constexpr dv::Pairs W = decltype(pairs)::value;
      return p.B <= dv::kSmallBatch ? dv::launch_append<T, W, dv::kSmallBatch>(p, t, stream)
                                    : dv::launch_append<T, W, dv::kMaxBatch>(p, t, stream);
    };
    if (t.rope && t.rope->interleaved)
      return batch(std::integral_constant<dv::Pairs, dv::kNeighbours>());
    if (!t.rope || t.rope->rot_dim % 16 == 0)
      return batch(std::integral_constant<dv::Pairs, dv::kHalves>());
    return batch(std::integral_constant<dv::Pairs, dv::kAcross>());
  };
  const cudaError_t err = t.dtype == DV_DTYPE_FP16 ? launch(__half()) : launch(__nv_bfloat16());
  return err == cudaSuccess ? DV_OK : dv::cuda_fail(err, "append launch");
}
