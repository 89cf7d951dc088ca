// vg_attention_bf16.cu -- the attention kernel over caches of this type.
#include "vg_attention.cuh"

namespace vg {
namespace attn {
const Variants kVariantsBf16 = VG_ATTENTION_VARIANTS(kBf16, false);
}  // namespace attn
}  // namespace vg
