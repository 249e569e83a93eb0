// qmv_kv_attn16.cu -- kv_attention's kernels for bf16 rows.
#include "qmv_kv_attn.cuh"

namespace qmvc {

size_t attn_workspace_16(const CacheView &c, int batch, int num_q_heads, bool weights, int sms) {
  return attn_workspace_bits<16>(c, batch, num_q_heads, weights, sms);
}
cudaError_t attn_launch_16(const AttnArgs &a, const Device &dev) { return attn_launch_bits<16>(a, dev); }

}  // namespace qmvc
