// dv_window_attention: causal attention in which a token attends the last rows up to its own
// and a few first ones (the kernel: dv_attention.cuh, form kWindow).  Of a tree, whose new rows
// are not its tokens' places one after the other, the window ends at the token's depth; no
// new row is outside it, as it is at least as long as a tree may be.
#include "dv_attention.cuh"

namespace dv {

cudaError_t window_waits(void** address) { return waits_address(address); }

}  // namespace dv

extern "C" dv_status dv_window_attention(const dv_cache* cache, int32_t layer,
                                         const int32_t* seq_start, const int32_t* seq_end,
                                         const dv_queries* queries, int32_t window, int32_t sinks,
                                         const uint64_t* tree, void* workspace, size_t workspace_bytes,
                                         dv_stream stream) {
  dv::Trace trace("dv_window_attention");
  if (!cache) return dv::fail(DV_ERR_INVALID_ARG, "cache is NULL");
  if (window < 1 || sinks < 0)
    return dv::fail(DV_ERR_INVALID_ARG, "a window of %d rows and %d first ones", window, sinks);
  if (tree && window < DV_MAX_TREE)
    return dv::fail(DV_ERR_UNSUPPORTED, "a window of %d rows with a tree, fewer than %d", window,
                    DV_MAX_TREE);
  const dv_status st = dv::check_max_seq(cache);
  if (st != DV_OK) return st;
  dv::Extra x;  // (more rows than there are: all of them)
  x.window = window < cache->max_seq ? window : cache->max_seq;
  x.sinks = sinks < cache->max_seq ? sinks : cache->max_seq;
  x.is_tree = tree != nullptr;
  x.tree = tree;
  return dv::attention<dv::kWindow>(cache, layer, seq_start, seq_end, queries, x, workspace,
                                    workspace_bytes, stream);
}
