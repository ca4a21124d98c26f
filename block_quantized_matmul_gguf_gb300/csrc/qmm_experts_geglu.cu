// qmm_experts_geglu.cu -- the streaming form's GeGLU kernels (qmm_experts.cuh).
#include "qmm_experts.cuh"

namespace qmm {

cudaError_t launch_experts_geglu(const ExpertsGeglu &a, cudaStream_t stream, const LaunchCtx &ctx) {
    if (a.workspace && experts_tiles_pay(a.plan, a.x, a.x_stride, a.x_bf16 && a.h_bf16, a.n, a.k, true))
        return launch_experts_tile_geglu(a, stream, ctx);
    experts::StreamParams p = {};
    p.plan = a.plan;
    p.w[0] = a.wg;
    p.w[1] = a.wu;
    p.x = a.x;
    p.x_stride = a.x_stride;
    p.x_bf16 = a.x_bf16;
    p.out = a.h;
    p.out_stride = a.h_stride;
    p.out_bf16 = a.h_bf16;
    p.n = a.n;
    p.k = a.k;
    p.ctx = ctx;
    return experts::launch_form<true>(p, stream);
}

}  // namespace qmm
