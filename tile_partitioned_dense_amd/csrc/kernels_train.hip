// kernels_train.hip -- instances of the tile and stream kernels with the
// stores of train_epilogue.hpp, one per translation unit:
// -DTG_TRAIN_KERNEL=<index into kTrainKernels>.
#include "train_launch.hpp"

#ifndef TG_TRAIN_KERNEL
#error "TG_TRAIN_KERNEL must name a training kernel"
#endif

namespace tg {

template <int ID>
const void* train_fn(int& threads) {
  constexpr TrainKernel k = kTrainKernels.k[ID];
  constexpr int kind = k.store == kStoreStats      ? kEpiStats
                       : k.store == kStoreXentGrad ? kEpiXentGrad
                       : k.store == kStoreGluGrad  ? kEpiGluGrad
                       : k.store == kStoreGlu      ? kEpiGlu
                                                   : kEpiPartial;
  constexpr int epi = k.gate >= 0 ? with_gate(kind, k.gate) : kind;
  if constexpr (k.tile >= kNumTrainTiles) {
    constexpr TrainStream c = kTrainStreams[k.tile - kNumTrainTiles];
    threads = c.bn / 32 * c.ks * 64;
    return reinterpret_cast<const void*>(&stream_gemm_kernel<c.bm, c.bn, c.sb, c.stages, c.ks, k.bf16, false, epi>);
  } else {
    constexpr TrainTile t = kTrainTiles[k.tile];
    threads = t.wm * t.wn * 64;
    if constexpr (t.bm == 256)
      return reinterpret_cast<const void*>(&tile64_gemm_kernel<t.bm, t.bn, t.wm, t.wn, k.bcol, k.bf16, false, epi>);
    else
      return reinterpret_cast<const void*>(
          &tile16_gemm_kernel<t.bm, t.bn, t.wm, t.wn, 4, k.bcol, k.bf16, false, epi>);
  }
}

template <int ID>
hipError_t launch_train(const TrainArgs& a, int64_t grid, hipStream_t stream) {
  int threads = 0;
  const void* fn = train_fn<ID>(threads);
  return launch_raw(fn, dim3((unsigned)grid), dim3(threads), a, stream);
}

template hipError_t launch_train<TG_TRAIN_KERNEL>(const TrainArgs&, int64_t, hipStream_t);

}  // namespace tg
