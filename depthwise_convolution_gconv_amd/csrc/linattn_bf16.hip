// linattn_bf16.hip -- the chunked pass of linear attention over bf16 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walks_bf16(const LinWalks &all, bool full)
{
    return full ? run_walks<__bf16, true>(all) : run_walks<__bf16, false>(all);
}
int lin_held_bf16(int64_t Da, int64_t Dc) { return held_walks<__bf16>(Da, Dc, DT_BF16); }

}  // namespace gconv
