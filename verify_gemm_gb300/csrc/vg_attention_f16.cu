// vg_attention_f16.cu -- the attention kernel over caches of this type.
#include "vg_attention.cuh"

namespace vg {
namespace attn {
const Variants kVariantsF16 = VG_ATTENTION_VARIANTS(kF16);
}  // namespace attn
}  // namespace vg
