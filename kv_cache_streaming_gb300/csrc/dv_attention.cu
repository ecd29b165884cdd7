// dv_prompt_attention and dv_tree_attention: attention of new tokens over the
// cache, by a kernel that is right for every case before it is fast: a warp
// per (token, query head) walks the attended rows 32 at a time, a lane per key
// for the scores, a lane per value element for the sums, with the running
// maximum and sum of the softmax.
#include "dv_ops.h"

namespace dv {
namespace {

template <int MAXB>
struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  const uint4* k;
  const uint16_t* v;
  const uint64_t* tree;
  int64_t q_stride, out_stride;
  int32_t Hq, H, G, D, C, S;
  float scale;
  int32_t use_tree;
  SeqTable<MAXB> seq;
};

template <typename T, int MAXB>
__global__ __launch_bounds__(128) void attention_simple(
    const __grid_constant__ AttnParams<MAXB> p) {
  __shared__ float qs[4][128];
  ops_pdl_enter();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int tok = blockIdx.x, hq = blockIdx.y * 4 + w;
  if (hq >= p.Hq) return;
  const int b = find_span(p.seq.pre, p.seq.batch, tok);
  const int i = tok - p.seq.pre[b], n = p.seq.pre[b + 1] - p.seq.pre[b], s = p.seq.start[b];
  const int h = hq / p.G;
  uint64_t bits = p.use_tree && p.tree ? p.tree[tok] : 0;
  const auto seen = [&](int row) {
    if (row < s) return true;
    if (row >= s + n) return false;
    return p.tree ? ((bits >> (row - s)) & 1) != 0 : row <= s + i;
  };
  const uint16_t* q = p.q + (int64_t)tok * p.q_stride + (int64_t)hq * p.D;
  for (int d = lane * 2; d < p.D; d += 64) {
    const float2 f = Pack2<T>::unpack(*reinterpret_cast<const uint32_t*>(q + d));
    qs[w][d] = f.x;
    qs[w][d + 1] = f.y;
  }
  __syncwarp();
  const int64_t head = (int64_t)b * p.H + h;
  const uint4* kh = p.k + head * p.C * p.S;
  const uint16_t* vh = p.v + head * p.S * p.D;
  float m = -INFINITY, l = 0.f, o[4] = {};
  for (int r0 = 0; r0 < s + n; r0 += 32) {
    const int row = r0 + lane;
    float x = -INFINITY;
    if (row < s + n && seen(row)) {
      float a = 0.f;
      for (int c = 0; c < p.C; ++c) {
        const uint4 u = kh[(int64_t)c * p.S + row];
        const uint32_t us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Pack2<T>::unpack(us[e]);
          a += f.x * qs[w][c * 8 + 2 * e] + f.y * qs[w][c * 8 + 2 * e + 1];
        }
      }
      x = a * p.scale;
    }
    float mx = x;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = __expf(m - base), e = __expf(x - base);
    float sum = e;
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
    l = l * f + sum;
    for (int k = 0; k < 4; ++k) o[k] *= f;
    m = mn;
    for (int j = 0; j < 32; ++j) {
      if (r0 + j >= s + n || !seen(r0 + j)) continue;
      const float pj = __shfl_sync(~0u, e, j);
      const uint16_t* vr = vh + (int64_t)(r0 + j) * p.D;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k * 64 + lane * 2 < p.D) {
          const float2 f2 =
              Pack2<T>::unpack(*reinterpret_cast<const uint32_t*>(vr + k * 64 + lane * 2));
          o[2 * k] += pj * f2.x;
          o[2 * k + 1] += pj * f2.y;
        }
    }
  }
  uint16_t* out = p.out + (int64_t)tok * p.out_stride + (int64_t)hq * p.D;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k * 64 + lane * 2 < p.D)
      *reinterpret_cast<uint32_t*>(out + k * 64 + lane * 2) =
          Pack2<T>::pack(o[2 * k] * inv, o[2 * k + 1] * inv);
}

template <typename T, int MAXB>
cudaError_t launch_attention(const Plan& p, const dv_queries& q, const uint64_t* tree,
                             cudaStream_t stream) {
  AttnParams<MAXB> kp;
  kp.q = static_cast<const uint16_t*>(q.q);
  kp.out = static_cast<uint16_t*>(q.out);
  kp.k = static_cast<const uint4*>(p.k) + p.l0 * p.layer_chunks;
  kp.v = reinterpret_cast<const uint16_t*>(static_cast<const uint4*>(p.v) + p.l0 * p.layer_chunks);
  kp.tree = tree;
  kp.use_tree = tree != nullptr;
  kp.q_stride = q.q_stride;
  kp.out_stride = q.out_stride;
  kp.Hq = q.q_heads;
  kp.H = p.H;
  kp.G = q.q_heads / p.H;
  kp.D = p.D;
  kp.C = p.C;
  kp.S = p.S;
  kp.scale = q.scale;
  fill_table(p, &kp.seq);
  return ops_launch(attention_simple<T, MAXB>, dim3((unsigned)p.tokens, (q.q_heads + 3) / 4), 128,
                    0, stream, kp);
}

dv_status check_heads(const dv_cache* cache, const Plan& p, int32_t q_heads) {
  if (cache->elem_bytes != 2)
    return fail(DV_ERR_UNSUPPORTED, "attention needs 2-byte elements (elem_bytes %d)",
                cache->elem_bytes);
  if (p.D > 128) return fail(DV_ERR_UNSUPPORTED, "attention needs head_dim <= 128 (got %d)", p.D);
  if (q_heads <= 0 || q_heads % p.H != 0)
    return fail(DV_ERR_INVALID_ARG, "q_heads %d is not a multiple of num_heads %d", q_heads, p.H);
  if (q_heads / p.H > DV_MAX_GROUP)
    return fail(DV_ERR_UNSUPPORTED, "%d query heads share a key head, more than %d", q_heads / p.H,
                DV_MAX_GROUP);
  return DV_OK;
}

dv_status attention(const dv_cache* cache, int32_t layer, const int32_t* s, const int32_t* e,
                    const dv_queries* queries, bool is_tree, const uint64_t* tree, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  if (!queries) return fail(DV_ERR_INVALID_ARG, "queries is NULL");
  Plan p;
  dv_status st = plan_layer(cache, layer, s, e, queries->dtype, &p);
  if (st != DV_OK) return st;
  dv_queries q = *queries;
  if ((st = check_heads(cache, p, q.q_heads)) != DV_OK) return st;
  if (!(q.scale > 0.f) || !std::isfinite(q.scale))
    return fail(DV_ERR_INVALID_ARG, "scale must be finite and positive (got %g)", (double)q.scale);
  if (is_tree && p.max_len > DV_MAX_TREE)
    return fail(DV_ERR_UNSUPPORTED, "%d drafted tokens of a sequence, more than %d", p.max_len,
                DV_MAX_TREE);
  if (p.tokens == 0) return DV_OK;
  if ((st = resolve_cache(cache, &p)) != DV_OK) return st;
  void* dev = nullptr;
  size_t nq = 0, no = 0;
  if ((st = resolve_rows(p, q.q, q.q_heads, q.q_stride, "q", &dev, &nq)) != DV_OK) return st;
  q.q = dev;
  if ((st = resolve_rows(p, q.out, q.q_heads, q.out_stride, "out", &dev, &no)) != DV_OK) return st;
  q.out = dev;
  if (overlap(q.out, no, q.q, nq)) return fail(DV_ERR_INVALID_ARG, "out overlaps q");
  if (tree) {
    if ((st = resolve_words(tree, (size_t)p.tokens * 8, 8, "tree", &dev)) != DV_OK) return st;
    tree = static_cast<const uint64_t*>(dev);
  }
  cudaError_t err;
  const bool small = p.B <= kSmallBatch;
  if (q.dtype == DV_DTYPE_FP16)
    err = small ? launch_attention<__half, kSmallBatch>(p, q, tree, stream)
                : launch_attention<__half, kMaxBatch>(p, q, tree, stream);
  else
    err = small ? launch_attention<__nv_bfloat16, kSmallBatch>(p, q, tree, stream)
                : launch_attention<__nv_bfloat16, kMaxBatch>(p, q, tree, stream);
  return err == cudaSuccess ? DV_OK : cuda_fail(err, "attention launch");
}

}  // namespace
}  // namespace dv

extern "C" dv_status dv_attention_workspace(const dv_cache* cache, const int32_t* seq_start,
                                            const int32_t* seq_end, int32_t q_heads,
                                            size_t* bytes) {
  if (!bytes) return dv::fail(DV_ERR_INVALID_ARG, "bytes is NULL");
  dv::Plan p;
  dv_status st = dv::plan_ranges(cache, 0, 1, seq_start, seq_end, &p);
  if (st != DV_OK) return st;
  if ((st = dv::check_heads(cache, p, q_heads)) != DV_OK) return st;
  *bytes = 0;
  return DV_OK;
}

extern "C" dv_status dv_prompt_attention(const dv_cache* cache, int32_t layer,
                                         const int32_t* seq_start, const int32_t* seq_end,
                                         const dv_queries* queries, void* workspace,
                                         size_t workspace_bytes, dv_stream stream) {
  dv::Trace trace("dv_prompt_attention");
  return dv::attention(cache, layer, seq_start, seq_end, queries, false, nullptr, workspace,
                       workspace_bytes, stream);
}

extern "C" dv_status dv_tree_attention(const dv_cache* cache, int32_t layer,
                                       const int32_t* seq_start, const int32_t* seq_end,
                                       const dv_queries* queries, const uint64_t* tree,
                                       void* workspace, size_t workspace_bytes, dv_stream stream) {
  dv::Trace trace("dv_tree_attention");
  return dv::attention(cache, layer, seq_start, seq_end, queries, true, tree, workspace,
                       workspace_bytes, stream);
}
