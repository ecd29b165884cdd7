// dv_prompt_attention and dv_tree_attention (the kernel: dv_attention.cuh), the
// workspace of an attention call, and the report of waits that gave up.
#include <atomic>
#include <mutex>
#include <vector>

#include "dv_attention.cuh"

namespace dv {
namespace {

std::atomic<uint32_t> g_tries{kSpinLimit};

}  // namespace

cudaError_t plain_waits(void** address) { return waits_address(address); }
uint32_t attention_tries() { return g_tries.load(std::memory_order_relaxed); }

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
  if (p.tokens == 0) return DV_OK;
  const int group = q_heads / p.H;
  dv::Extra tree;
  tree.is_tree = true;
  // (a window takes no more tiles, and so no more CTAs)
  const size_t a = dv::schedule<dv::kPlain>(p, group, {}, nullptr).bytes;
  const size_t b =
      p.max_len <= DV_MAX_TREE ? dv::schedule<dv::kPlain>(p, group, tree, nullptr).bytes : 0;
  *bytes = a > b ? a : b;
  return DV_OK;
}

extern "C" dv_status dv_debug_attention_tries(int32_t tries) {
  if (tries > (int32_t)dv::kSpinLimit)
    return dv::fail(DV_ERR_INVALID_ARG, "%d tries are more than %u", tries, dv::kSpinLimit);
  dv::g_tries.store(tries < 0 ? dv::kSpinLimit : (uint32_t)tries, std::memory_order_relaxed);
  return DV_OK;
}

namespace {

// The count of waits that gave up as a stream's last check found it; streams without an entry
// have found none.
struct Checked {
  unsigned long long context, stream, count;
};

// Whether `count` is news to the stream; remembers it.
bool count_is_new(unsigned long long context, unsigned long long stream, unsigned long long count) {
  static std::mutex mu;
  static std::vector<Checked> checked;
  if (count == 0) return false;
  std::lock_guard<std::mutex> lock(mu);
  for (Checked& c : checked)
    if (c.context == context && c.stream == stream) {
      const bool news = c.count != count;
      c.count = count;
      return news;
    }
  try {
    checked.push_back({context, stream, count});
  } catch (...) {  // reported again by the next check
  }
  return true;
}

}  // namespace

extern "C" dv_status dv_attention_check(dv_stream stream) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t err = cudaStreamIsCapturing(stream, &capture);
  if (err == cudaSuccess && capture != cudaStreamCaptureStatusNone)
    return dv::fail(DV_ERR_INVALID_ARG, "dv_attention_check waits for its stream, which is being "
                    "captured into a graph");
  // one count for each form's translation unit, where the form has been launched (a fetch takes
  // 9 us, a form's first one 2 ms)
  using Counter = cudaError_t (*)(void**);
  constexpr Counter counters[] = {dv::plain_waits, dv::window_waits, dv::scored_waits};
  constexpr int n = sizeof(counters) / sizeof(counters[0]);
  unsigned long long id = 0, context = 0, counts[n] = {}, count = 0;
  if (err == cudaSuccess) err = cudaStreamGetId(stream, &id);
  for (int i = 0; i < n && err == cudaSuccess; ++i) {
    void* counter = nullptr;
    err = counters[i](&counter);
    if (err == cudaSuccess && counter)
      err = cudaMemcpyAsync(&counts[i], counter, sizeof(counts[i]), cudaMemcpyDeviceToHost, stream);
  }
  if (err == cudaSuccess) err = cudaStreamSynchronize(stream);
  if (err != cudaSuccess) return dv::cuda_fail(err, "reading the attention kernels' count");
  for (const unsigned long long c : counts) count += c;
  dv::context_id(&context);
  if (count_is_new(context, id, count))
    return dv::fail(DV_ERR_TIMEOUT, "an attention kernel gave up a wait; its output is not valid");
  return DV_OK;
}

extern "C" dv_status dv_prompt_attention(const dv_cache* cache, int32_t layer,
                                         const int32_t* seq_start, const int32_t* seq_end,
                                         const dv_queries* queries, void* workspace,
                                         size_t workspace_bytes, dv_stream stream) {
  dv::Trace trace("dv_prompt_attention");
  return dv::attention<dv::kPlain>(cache, layer, seq_start, seq_end, queries, {}, workspace,
                                   workspace_bytes, stream);
}

extern "C" dv_status dv_tree_attention(const dv_cache* cache, int32_t layer,
                                       const int32_t* seq_start, const int32_t* seq_end,
                                       const dv_queries* queries, const uint64_t* tree,
                                       void* workspace, size_t workspace_bytes, dv_stream stream) {
  dv::Trace trace("dv_tree_attention");
  dv::Extra x;
  x.is_tree = true;
  x.tree = tree;
  return dv::attention<dv::kPlain>(cache, layer, seq_start, seq_end, queries, x, workspace,
                                   workspace_bytes, stream);
}
