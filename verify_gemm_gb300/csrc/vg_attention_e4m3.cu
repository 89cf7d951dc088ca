// vg_attention_e4m3.cu -- the attention kernel over caches of this type.
#include "vg_attention.cuh"

namespace vg {
namespace attn {
const Variants kVariantsE4M3 = VG_ATTENTION_VARIANTS(kE4M3, false);
}  // namespace attn
}  // namespace vg
