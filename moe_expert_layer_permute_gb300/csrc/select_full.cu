// select_full.cu - routing by scores: the forward for rows in fours that fill every lane.
#include "select_fwd.cuh"

namespace moe {

template cudaError_t select_kind<kSelFull>(cudaStream_t st, const SelectArgs& a, int W, int V, int num_sms);

}  // namespace moe
