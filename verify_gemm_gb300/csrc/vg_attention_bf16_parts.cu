// vg_attention_bf16_parts.cu -- the same for the parts of a prefix attention.
#include "vg_attention.cuh"

namespace vg {
namespace attn {
const Variants kPartsBf16 = VG_ATTENTION_VARIANTS(kBf16, true);
}  // namespace attn
}  // namespace vg
