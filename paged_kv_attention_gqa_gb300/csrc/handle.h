// The handle behind the C ABI and the host helpers that its entry points share (pkv_api.cu,
// latent_api.cu): NVTX ranges, plan staging, tensor-map encoding.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <string>
#include <vector>

#include "../../include/pkv.h"
#include "evict.h"
#include "plan.h"

// Page-locked staging ring (PinnedIndexRing: depth 2; a set is rewritten only after
// the copy out of it has completed, fenced by an event recorded after that copy).
struct PkvStaging {
    void *pinned[2] = {nullptr, nullptr};
    size_t pinned_bytes[2] = {0, 0};
    cudaEvent_t fence[2] = {nullptr, nullptr};
    bool fence_live[2] = {false, false};
    int ring_at = 0;
    // Copy `nbytes` of a plan image to `workspace` on `st`; `what` names the failing call.
    cudaError_t copy(const void *image, size_t nbytes, void *workspace, cudaStream_t st, const char **what);
    void release();  // waits for the copies still queued
};

struct pkv_handle_s {
    pkv::Shape shape{};
    std::string err;
    pkv::Plan plan;
    // the image buffer of the previous plan, handed to the next one so that building its
    // image reuses memory already mapped (the staged plan keeps no image)
    std::vector<uint8_t> spare_image;
    pkv::WeightsPlan weights;  // the score arrays of DECODE_WEIGHTS / WEIGHTS plans
    pkv::EvictPlan evict;      // EVICT plans
    void *planned_ws = nullptr;
    PkvStaging staging;
    // side stream + fork/join events of the mixed step's concurrent passes
    cudaStream_t side = nullptr;
    cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
    // last encoded tensor maps (re-encoded when the layer pointer changes)
    const void *tm_dec_ptr = nullptr, *tm_pf_ptr = nullptr, *tm_q_ptr = nullptr;
    int tm_q_rows = -1;
    CUtensorMap tm_dec{}, tm_pf{}, tm_q{};
    bool nvtx = false;  // one NVTX range per call (pkv_config.enable_nvtx)
};

// The NVTX range of one call on a handle with enable_nvtx set: opened here, closed when
// the call returns.
struct NvtxCall {
    bool on;
    NvtxCall(bool enabled, const char *name) : on(enabled) {
        if (on) nvtxRangePushA(name);
    }
    NvtxCall(const pkv_handle_s *h, const char *name) : NvtxCall(h && h->nvtx, name) {}
    ~NvtxCall() {
        if (on) nvtxRangePop();
    }
};

namespace pkv {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // nullptr when the driver lacks it
}
