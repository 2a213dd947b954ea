// linattn_f32.hip -- the chunked pass of linear attention over fp32 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walks_f32(const LinWalks &all, bool full)
{
    return full ? run_walks<float, true>(all) : run_walks<float, false>(all);
}
int lin_held_f32(int64_t Da, int64_t Dc) { return held_walks<float>(Da, Dc, DT_F32); }

}  // namespace gconv
