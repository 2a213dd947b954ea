// linattn_bf16.hip -- the chunked pass of linear attention over bf16 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walk_bf16(const LinWalk &p, bool full)
{
    if (!full) return run_walk<__bf16, __bf16, false>(p);
    return p.out_f32 ? run_walk<__bf16, float, true>(p) : run_walk<__bf16, __bf16, true>(p);
}

}  // namespace gconv
