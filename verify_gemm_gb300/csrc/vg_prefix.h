// vg_prefix.h -- the launch that joins a shared prefix's results to the sequences' own.
#pragma once

#include "vg_attention.cuh"

namespace vg {
namespace attn {

// The partial results of the prefix's launch: `partial` floats each, [column / 4][row][4] (wide) or in
// fragment order, then (m, l) of each row at `state`.
struct PrefixJoin {
  int wide, e4m3, rows, columns, partial, state, grid, sms;
  float lift;                       // of the weights, log2
};

cudaError_t launch_prefix_join(const AttnParams &own, const AttnParams &first, const PrefixJoin &j, cudaStream_t st);

}  // namespace attn
}  // namespace vg
