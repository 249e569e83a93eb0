// qmv_kv_attn4.cu -- kv_attention's kernels for 4-bit codes.
#include "qmv_kv_attn.cuh"

namespace qmvc {

size_t attn_workspace_4(const CacheView &c, int batch, int num_q_heads, bool weights, int sms) {
  return attn_workspace_bits<4>(c, batch, num_q_heads, weights, sms);
}
cudaError_t attn_launch_4(const AttnArgs &a, const Device &dev) { return attn_launch_bits<4>(a, dev); }

}  // namespace qmvc
