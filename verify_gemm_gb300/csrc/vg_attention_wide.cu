// vg_attention_wide.cu -- the tcgen05 attention kernel with its variants.
#include "vg_attention_wide.cuh"

namespace vg {
namespace attn {
#define VG_WIDE(T)                                      \
  {{wide_variant<T, 1, 1>(), wide_variant<T, 1, 2>()},  \
   {wide_variant<T, 2, 1>(), wide_variant<T, 2, 2>()}}
const WideVariants kWide = {VG_WIDE(kBf16), VG_WIDE(kF16), VG_WIDE(kE4M3)};
}  // namespace attn
}  // namespace vg
