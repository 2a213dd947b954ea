// linattn_f16.hip -- the chunked pass of linear attention over fp16 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walks_f16(const LinWalks &all, bool full)
{
    return full ? run_walks<_Float16, true>(all) : run_walks<_Float16, false>(all);
}

}  // namespace gconv
