// Which kernels a call takes, as the library decides it (csrc/ffn_plan.hpp).
// Compiled by tests/test_ffn_plan_cpu.py.
#include "../../sparse_hashed_gram_amd/csrc/ffn_plan.hpp"

using namespace ffn_plan;

// fwd: few, wide, hidden shape, rows shape, parts; bwd: wide, merged, hidden
// shape, rows shape, parts, dW shape, parts
extern "C" void model_plan(int64_t T, int64_t F, int32_t *fwd, int32_t *bwd)
{
    const Fwd f = plan_fwd(T, F);
    const int32_t a[] = {f.few, f.wide, f.hidden.shape, f.rows.shape, f.rows.parts};
    for (int i = 0; i < 5; ++i)
        fwd[i] = a[i];
    const Bwd b = plan_bwd(T, F);
    const int32_t c[] = {b.wide, b.merged, b.hidden.shape, b.rows.shape, b.rows.parts, b.dw.shape, b.dw.parts};
    for (int i = 0; i < 7; ++i)
        bwd[i] = c[i];
}
