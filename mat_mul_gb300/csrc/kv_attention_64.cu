// kv_attention_64.cu -- the attention kernels for few rows with heads of up to 64 values.
#include "kv_attention.cuh"

namespace qk {
namespace kv {
cudaError_t launch_few_64(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev) {
    return launch_few_dp<64>(p, nb, hl, st, num_sms, dev);
}
}  // namespace kv
}  // namespace qk
