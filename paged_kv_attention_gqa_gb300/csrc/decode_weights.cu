// Instances of the decode kernel that also store their logits (DECODE_WEIGHTS plans), in their own
// translation unit.
#include "decode_kernel.cuh"
#include "evict.h"

namespace pkv {

cudaError_t launch_decode_weights(const Shape &s, const Plan &p, const WeightsPlan &wp, const CUtensorMap &tm, void *ws,
                                  const void *q, void *kv_layer, void *out, float *lse, cudaStream_t st) {
    if (p.dec_ctas == 0) return cudaSuccess;
    dev::DecodeArgs a;
    if (!decode_args(s, p, ws, q, kv_layer, out, lse, nullptr, nullptr, a)) return cudaErrorInvalidValue;
    a.logits = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + wp.off_logits);
    a.logit_stride = wp.logit_stride;
    const int warps = a.heads + a.producers;
    const size_t smem = decode_smem_bytes(s);
    const dim3 grid(p.dec_ctas, s.dec_head_groups());
    cudaError_t e = cudaErrorInvalidValue;
    const int g = s.group();
#define PKV_DECW(DD, GG)                                                                        \
    if (s.head_dim == DD && g == GG)                                                             \
        e = s.page_size < 16 ? launch_decode_t<DD, GG, true, true>(tm, a, grid, warps, smem, st) \
                             : launch_decode_t<DD, GG, false, true>(tm, a, grid, warps, smem, st);
    PKV_FOR_EACH_HEAD_DIM_AND_GROUP(PKV_DECW)
#undef PKV_DECW
    return e == cudaSuccess ? launch_decode_merge(s, p, ws, a, st) : e;
}

}  // namespace pkv
