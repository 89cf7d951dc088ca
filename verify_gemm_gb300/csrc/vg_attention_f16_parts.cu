// vg_attention_f16_parts.cu -- the same for the parts of a prefix attention.
#include "vg_attention.cuh"

namespace vg {
namespace attn {
const Variants kPartsF16 = VG_ATTENTION_VARIANTS(kF16, true);
}  // namespace attn
}  // namespace vg
