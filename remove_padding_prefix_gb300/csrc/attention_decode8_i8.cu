// Single-token attention over a paged cache of 8-bit codes: int8, and the call for both (the kernel: attention_decode8.cuh).
#include "attention_decode8.cuh"

namespace rpp {

cudaError_t launch_attention_decode8_e4m3(const void* params, cudaStream_t stream);   // attention_decode8_e4m3.cu

size_t attention_decode8_ws_bytes(int n, int nh, int nkv, int d) {
  return line_ws_bytes(n, nh, nkv, d, decode8_warps(nh / nkv, d));
}

cudaError_t launch_attention_decode8(const KvDims& d, const KvState& c, const Kv8Scales& q8, int layer, const void* q,
                                     rpp_dtype dtype, int q_stride, const int32_t* slots, int n, int nh, float scale,
                                     void* out, void* ws, int32_t* err, cudaStream_t stream) {
  const size_t heads = static_cast<size_t>(d.pages) * 2 * d.kv_heads * layer;
  Decode8Params p{};
  p.d = d;
  p.pool = static_cast<const uint8_t*>(c.pool) + heads * d.page_size * d.head_dim;
  p.scales = q8.scales + heads * (d.page_size >> q8.shift);
  p.shift = q8.shift;
  p.bf16 = dtype == RPP_BF16;
  p.head_bytes = static_cast<long long>(d.page_size) * d.head_dim;
  p.v_bytes = d.kv_heads * p.head_bytes;
  p.page_bytes = 2 * p.v_bytes;
  p.head_scales = d.page_size >> q8.shift;
  p.v_scales = d.kv_heads * p.head_scales;
  p.page_scales = 2 * p.v_scales;
  p.table = c.table;
  p.lens = c.lens;
  p.q = q;
  p.q_stride = q_stride;
  p.slots = slots;
  p.n = n;
  p.nh = nh;
  p.group = nh / d.kv_heads;
  p.parts = (p.group + kRows - 1) / kRows;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  line_ws_bind(&p, ws, decode8_warps(p.group, d.head_dim));
  p.err = err;
  return q8.i8 ? launch_codes<true>(p, stream) : launch_attention_decode8_e4m3(&p, stream);
}

}  // namespace rpp
