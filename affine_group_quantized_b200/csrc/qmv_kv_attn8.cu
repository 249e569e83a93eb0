// qmv_kv_attn8.cu -- kv_attention's kernels for 8-bit codes.
#include "qmv_kv_attn.cuh"

namespace qmvc {

size_t attn_workspace_8(const CacheView &c, int batch, int num_q_heads, bool weights, int sms) {
  return attn_workspace_bits<8>(c, batch, num_q_heads, weights, sms);
}
cudaError_t attn_launch_8(const AttnArgs &a, const Device &dev) { return attn_launch_bits<8>(a, dev); }

}  // namespace qmvc
