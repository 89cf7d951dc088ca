// vg_attention_e4m3_parts.cu -- the same for the parts of a prefix attention.
#include "vg_attention.cuh"

namespace vg {
namespace attn {
const Variants kPartsE4M3 = VG_ATTENTION_VARIANTS(kE4M3, true);
}  // namespace attn
}  // namespace vg
