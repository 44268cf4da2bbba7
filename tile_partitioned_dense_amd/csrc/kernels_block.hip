// kernels_block.hip -- instances of the E4M3 products with block scales for
// one configuration, selected with -DTG_BLOCK_CONFIG=<index into kBlockConfigs>.
#include "block_launch.hpp"

#ifndef TG_BLOCK_CONFIG
#error "TG_BLOCK_CONFIG must name a configuration index"
#endif

namespace tg {

template <int CFG, bool EXPERTS, bool OB>
const void* block_fn() {
  constexpr BlockConfig c = kBlockConfigs[CFG];
  if constexpr (!OB && c.bm * c.bn / (c.wm * c.wn) > 96 * 64) return nullptr;  // (not planned for fp32)
  else if constexpr (c.tile)
    return reinterpret_cast<const void*>(&block_tile_kernel<c.bm, c.bn, c.wm, c.wn, EXPERTS, !OB>);
  else return reinterpret_cast<const void*>(
      &block_gemm_kernel<c.bm, c.bn, c.wm, c.wn, c.ks, c.sb, c.stages, EXPERTS, OB>);
}

template <int CFG>
hipError_t launch_block(const BlockArgs& a, bool experts, bool out_bf16, int64_t grid, hipStream_t stream) {
  constexpr BlockConfig c = kBlockConfigs[CFG];
  const void* fn = experts ? (out_bf16 ? block_fn<CFG, true, true>() : block_fn<CFG, true, false>())
                           : (out_bf16 ? block_fn<CFG, false, true>() : block_fn<CFG, false, false>());
  if (!fn) return hipErrorInvalidDeviceFunction;
  return launch_raw(fn, dim3((unsigned)grid), dim3(c.wm * c.wn * c.ks * 64), a, stream);
}

template hipError_t launch_block<TG_BLOCK_CONFIG>(const BlockArgs&, bool, bool, int64_t, hipStream_t);

}  // namespace tg
