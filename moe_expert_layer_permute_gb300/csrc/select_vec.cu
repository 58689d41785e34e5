// select_vec.cu - routing by scores: the forward for rows in fours.
#include "select_fwd.cuh"

namespace moe {

template cudaError_t select_kind<kSelVec>(cudaStream_t st, const SelectArgs& a, int W, int V, int num_sms);

}  // namespace moe
