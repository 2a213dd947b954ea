// linattn_f16.hip -- the chunked pass of linear attention over fp16 tensors.
#include "linattn_walk.hpp"

namespace gconv {

hipError_t run_lin_walk_f16(const LinWalk &p, bool full)
{
    if (!full) return run_walk<_Float16, _Float16, false>(p);
    return p.out_f32 ? run_walk<_Float16, float, true>(p) : run_walk<_Float16, _Float16, true>(p);
}

}  // namespace gconv
