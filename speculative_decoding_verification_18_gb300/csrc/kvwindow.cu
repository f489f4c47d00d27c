// Attention over the paged cache through a sliding window, the first slots always visible
// (include/specverify_kv.h): the attention's kernels with the slots between the two left out.

#include "kvattention.cuh"

extern "C" sv_status spec_kv_attention_window(
    const sv_kv_cache* cache, const void* q, const sv_strides* q_strides, sv_dtype dtype,
    const int32_t* kv_len, const int32_t* num_new, const int32_t* tree_parents, float scale,
    int window, int sinks, int B, int N, int q_heads, void* out, void* ws, size_t ws_bytes,
    uint32_t* status, cudaStream_t stream) {
    return svkv::attend<true>(cache, q, q_strides, dtype, kv_len, num_new, tree_parents, scale,
                              window, sinks, B, N, q_heads, out, ws, ws_bytes, status, stream);
}
