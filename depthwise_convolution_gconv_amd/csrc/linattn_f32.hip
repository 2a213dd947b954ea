// linattn_f32.hip -- the chunked pass of linear attention over fp32 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walk_f32(const LinWalk &p, bool full)
{
    return full ? run_walk<float, float, true>(p) : run_walk<float, float, false>(p);
}

}  // namespace gconv
