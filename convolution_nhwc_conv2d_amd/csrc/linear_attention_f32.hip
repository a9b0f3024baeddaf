// Linear attention's chunk kernels for f32.
#include "linear_attention_launch.hpp"

namespace cnhwc {
namespace seq {

template hipError_t launch_passes<CNHWC_F32>(Passes<CNHWC_F32>&, int, LaGeo, const Cut&, int64_t, char*, hipStream_t);
template hipError_t launch_decay<CNHWC_F32>(DecayPass<CNHWC_F32>&, LaGeo, const Cut&, int64_t, char*, float*, hipStream_t);

}  // namespace seq
}  // namespace cnhwc
