// vg_attention_wide.cu -- the tcgen05 attention kernel over 16-bit caches.
#include "vg_attention_wide.cuh"

namespace vg {
namespace attn {
const WideVariants kWide = {
    {{wide_variant<kBf16, 1, 1>(), wide_variant<kBf16, 1, 2>()},
     {wide_variant<kBf16, 2, 1>(), wide_variant<kBf16, 2, 2>()}},
    {{wide_variant<kF16, 1, 1>(), wide_variant<kF16, 1, 2>()},
     {wide_variant<kF16, 2, 1>(), wide_variant<kF16, 2, 2>()}}};
}  // namespace attn
}  // namespace vg
