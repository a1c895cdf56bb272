// ssd_block.cuh -- the operators around the scan (short causal convolution,
// selective scan, norms): what their host side (ssd_block_api.cu) hands to the
// kernels. Internal, not part of the C ABI.
#pragma once

#include "ssd_common.cuh"

namespace ssd {

// Sizes are validated on the host: batch * seqlen < 2^31, channels <= 2^20.
struct ConvArgs {
    int batch, seqlen, channels, width, nseq;
    int64_t xs_b, xs_t;  // strides of x, in elements
    int c1, c2;          // first channel of out1 / out2 (= channels when unused)
    int silu;
    const void* x;
    const float* weight;
    const float* bias;
    const void* init;  // ssd_causal_conv: initial windows; ssd_conv_step: the window state
    const int32_t* seq_idx;
    void* out[3];
    void* final_states;  // ssd_conv_step: the window state
};

struct SelectiveArgs {
    int batch, seqlen, channels, dstate, ngroups, nseq;
    int64_t us_b, us_t, ds_b, ds_t, zs_b, zs_t, bs_b, bs_t, cs_b, cs_t;
    int softplus;
    const void *u, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias;
    const float* init;  // ssd_selective_step: the state, read and written
    const int32_t* seq_idx;
    void* y;
    float* final_states;
};

enum NormMode { kNormPlain = 0, kNormGateFirst = 1, kNormGateLast = 2, kNormAdd = 3 };

struct NormArgs {
    int batch, seqlen, channels, ngroups;
    int64_t xs_b, xs_t, zs_b, zs_t;
    float eps, alpha;
    NormMode mode;
    const void* x;
    const void* z;  // the gate, or the residual
    const float* weight;
    const float* scale;
    void* out;
    void* residual_out;
};

cudaError_t launch_causal_conv(const ConvArgs& a, ssd_dtype dt, cudaStream_t st);
cudaError_t launch_conv_step(const ConvArgs& a, ssd_dtype dt, cudaStream_t st);
cudaError_t launch_selective_scan(const SelectiveArgs& a, ssd_dtype dt, cudaStream_t st);
cudaError_t launch_selective_step(const SelectiveArgs& a, ssd_dtype dt, cudaStream_t st);
cudaError_t launch_row_norm(const NormArgs& a, ssd_dtype dt, ssd_dtype residual_dt, cudaStream_t st);

// V consecutive elements, moved as one access of 2, 4, 8 or 16 bytes (or as several of 16).
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T v[V];
};

// silu(v) = v / (1 + exp(-v)). For fp32 outputs with the full-precision
// exponential and division; for bf16 outputs with the hardware's fast forms,
// whose error (a few 2^-22) disappears in the output's rounding (2^-9).
template <typename T>
__device__ __forceinline__ float silu_for(float v);
template <>
__device__ __forceinline__ float silu_for<float>(float v) {
    return v / (1.f + expf(-v));
}
template <>
__device__ __forceinline__ float silu_for<__nv_bfloat16>(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return v * r;
}

// Largest number of channels per access (16-byte, 4-byte or one element) that
// every address and every stride (in elements) allows.
struct VectorRule {
    uint64_t bits = 0;  // OR of all byte offsets that must be multiples of the access
    size_t e;
    explicit VectorRule(size_t elem) : e(elem) {}
    VectorRule& address(const void* p) {
        bits |= reinterpret_cast<uintptr_t>(p);
        return *this;
    }
    VectorRule& elements(int64_t n) {
        bits |= (uint64_t)n * e;
        return *this;
    }
    bool multiple_of(unsigned bytes) const { return (bits & (bytes - 1)) == 0; }
};

}  // namespace ssd
