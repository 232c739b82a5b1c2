// The handle behind gemm_handle_t and the host helpers its entry points share (not
// installed).
#pragma once

#include <cstddef>
#include <new>

#include "internal.h"

struct gemm_ctx {
    int device = 0;
    int num_sms = 0;
    int* d_status = nullptr;  // device status word written by kernels with bounded waits
    float* workspace = nullptr;
    size_t workspace_bytes = 0;
    unsigned long long* tc_counters = nullptr;  // last-wave split counters of the tensor-core GEMM
    size_t tc_counters_bytes = 0;
    unsigned tc_seq = 0;  // tag of the last split tensor-core launch
    unsigned long long* f32_counters = nullptr;  // K-slice counters of the persistent fp32 GEMM
    size_t f32_counters_bytes = 0;
    unsigned f32_seq = 0;  // tag of the last split persistent fp32 launch
    void* host_stage = nullptr;  // gemm_run_host(_batch) device copies of A, B and C
    size_t host_stage_bytes = 0;
    float* product = nullptr;  // fp32 product for the generalised epilogue of fp32 inputs
    size_t product_bytes = 0;
    int opt_f32_kernel = 0;
    int opt_split_k = 0;
    int opt_tc_chunk = 0;  // tensor-core accumulation chunk in 64-wide k-blocks (0 = default)
    int opt_tc_pair = 0;   // tensor-core tile: 0 choose, 1 single CTA, 2 CTA pair
    int opt_test_stall = 0;  // test hook: kernels with bounded waits let one wait run out
    int opt_test_stall_pair = 0;  // and of the linear layers' only this CTA pair (from 1; 0: all)
    int opt_conv_stack = 0;  // tensor-core convolution: output positions stacked along N (0 = choose)
    int opt_conv_split = 0;  // tensor-core convolution: 0 choose, 1 one CTA pair per tile, 2 two pairs
    uint64_t wait_limit_ns = 2000000000ull;
    // linear layers and routing: partial tiles of K slices, dZ, pieces of column sums, the
    // router's counts per block; these grow by grow_buffer below
    float* lin_partials = nullptr;
    size_t lin_partials_bytes = 0;
    void* lin_dz = nullptr;
    size_t lin_dz_bytes = 0;
    void* lin_sums = nullptr;
    size_t lin_sums_bytes = 0;
    void* route_counts = nullptr;
    size_t route_counts_bytes = 0;
    void* layer = nullptr;  // moe_layer: the picks' rows between and after the two products
    size_t layer_bytes = 0;
    void* adapt = nullptr;  // adapters: the rows' narrow products and the row tiles' lists
    size_t adapt_bytes = 0;
    // arrival counters, zero after every launch: linear_counters(num_sms) of the products, then
    // the router's, then kLayerCounters of moe_layer.  Made with the handle, so that they never move
    unsigned* lin_counters = nullptr;
    bool captured = false;    // a graph holds addresses of the buffers that grow
    struct KeptBuffer {
        void* p;
        KeptBuffer* next;
    };
    KeptBuffer* kept = nullptr;  // outgrown buffers that a graph may hold
    int64_t launches = 0;  // kernels launched through this handle
    // gemm_run_host pipeline: copy-in and copy-out streams and their events
    cudaStream_t s_in = nullptr, s_out = nullptr;
    static constexpr int kMaxChunks = 8;
    cudaEvent_t ev_start = nullptr, ev_done = nullptr;
    cudaEvent_t ev_a[kMaxChunks] = {}, ev_c[kMaxChunks] = {};
};

namespace gemm_gb300 {


class DeviceGuard {
  public:
    explicit DeviceGuard(int dev) : ok_(false), prev_(-1)
    {
        if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
        ok_ = (prev_ == dev) || (cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceGuard()
    {
        if (prev_ >= 0) cudaSetDevice(prev_);
    }
    bool ok() const { return ok_; }

  private:
    bool ok_;
    int prev_;
};

inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA; }

// Grow a device buffer to at least `bytes` (contents are not kept).
inline int ensure_buffer(void** buf, size_t* have, size_t bytes)
{
    if (*have >= bytes && *buf) return GEMM_OK;
    if (*buf) {
        cudaFree(*buf);  // implicit device synchronisation: no kernel still uses it
        *buf = nullptr;
        *have = 0;
    }
    size_t want = bytes < 256 ? 256 : bytes;
    if (cudaMalloc(buf, want) != cudaSuccess) {
        *buf = nullptr;
        (void)cudaGetLastError();  // an allocation failure is not sticky: keep it out of later launch checks
        return GEMM_ERR_CUDA;
    }
    *have = want;
    return GEMM_OK;
}

// The same for a buffer whose address calls captured in CUDA graphs may hold.  Under capture
// the buffer must be large enough: the call is refused, with the capture and the buffer as they
// were.  Once any call was captured, an outgrown buffer is kept until the handle is destroyed:
// the graph's replays go on using it.
inline int grow_buffer(gemm_ctx* h, void** buf, size_t* have, size_t bytes, cudaStream_t s)
{
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &st) != cudaSuccess) {
        (void)cudaGetLastError();  // (the legacy stream, while another one captures: its launch will say so)
        st = cudaStreamCaptureStatusNone;
    }
    const bool capturing = st != cudaStreamCaptureStatusNone;
    const bool enough = *buf && *have >= bytes;
    if (capturing && !enough) {
        glog("a captured call needs %zu bytes of workspace, %zu are there: run one such call before the capture", bytes,
             *have);
        return GEMM_ERR_CUDA;
    }
    if (capturing) h->captured = true;
    if (enough) return GEMM_OK;
    if (*buf && h->captured) {
        gemm_ctx::KeptBuffer* k = new (std::nothrow) gemm_ctx::KeptBuffer{*buf, h->kept};
        if (!k) return GEMM_ERR_CUDA;
        h->kept = k;
        *buf = nullptr;
        *have = 0;
    }
    return ensure_buffer(buf, have, bytes);
}

const char* dtype_name(int d);

}  // namespace gemm_gb300
