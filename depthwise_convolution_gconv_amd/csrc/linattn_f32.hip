// linattn_f32.hip -- the chunked pass of linear attention over fp32 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walks_f32(const LinWalks &all, bool full)
{
    return full ? run_walks<float, true>(all) : run_walks<float, false>(all);
}

}  // namespace gconv
