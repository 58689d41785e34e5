// select_odd.cu - routing by scores: the forward for rows whose groups are no multiple of four values.
#include "select_fwd.cuh"

namespace moe {

template cudaError_t select_kind<kSelOdd>(cudaStream_t st, const SelectArgs& a, int W, int V, int num_sms);

}  // namespace moe
