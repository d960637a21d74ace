// kv_attention_128.cu -- the attention kernels for few rows with heads of up to 128 values.
#include "kv_attention.cuh"

namespace qk {
namespace kv {
cudaError_t launch_few_128(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev) {
    return launch_few_dp<128>(p, nb, hl, st, num_sms, dev);
}
}  // namespace kv
}  // namespace qk
