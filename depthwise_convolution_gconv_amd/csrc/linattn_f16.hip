// linattn_f16.hip -- the chunked pass of linear attention over fp16 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walks_f16(const LinWalks &all, bool full)
{
    return full ? run_walks<_Float16, true>(all) : run_walks<_Float16, false>(all);
}
int lin_held_f16(int64_t Da, int64_t Dc) { return held_walks<_Float16>(Da, Dc, DT_F16); }

}  // namespace gconv
