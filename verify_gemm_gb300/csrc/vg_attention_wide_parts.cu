// vg_attention_wide_parts.cu -- the tcgen05 attention kernel for the parts of a prefix attention.
#include "vg_attention_wide.cuh"

namespace vg {
namespace attn {
const WideVariants kWideParts = {VG_WIDE(kBf16, true), VG_WIDE(kF16, true), VG_WIDE(kE4M3, true)};
}  // namespace attn
}  // namespace vg
