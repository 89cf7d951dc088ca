// vg_attention_wide.cu -- the tcgen05 attention kernel with its variants.
#include "vg_attention_wide.cuh"

namespace vg {
namespace attn {
const WideVariants kWide = {VG_WIDE(kBf16, false), VG_WIDE(kF16, false), VG_WIDE(kE4M3, false)};
}  // namespace attn
}  // namespace vg
