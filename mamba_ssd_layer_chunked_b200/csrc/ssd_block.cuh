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

// V fp32 values from and to their packed form, bf16 pairs converted together.
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& p, float (&f)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&p.v[e]));
            f[e] = v.x, f[e + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = to_f32(p.v[e]);
    }
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&f)[V]) {
    Pack<T, V> p;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2)
            *reinterpret_cast<__nv_bfloat162*>(&p.v[e]) = __floats2bfloat162_rn(f[e], f[e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) p.v[e] = from_f32<T>(f[e]);
    }
    return p;
}

__device__ __forceinline__ float exp2_approx(float x) {  // hardware 2^x, error about 2^-22; denormal results are 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {  // hardware 1 / x, error about 2^-23; 0 for x >= 2^126
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// silu(v) = v / (1 + exp(-v)). For fp32 outputs with the full-precision
// exponential (the rounding of v log2 e alone is a relative error of |v| 2^-24);
// for bf16 outputs with the hardware's, whose errors disappear in the output's
// rounding (2^-8).
template <typename T>
__device__ __forceinline__ float silu_for(float v) {
    return v * rcp_approx(1.f + (sizeof(T) == 4 ? expf(-v) : exp2_approx(-kLog2e * v)));
}
template <typename T>
__device__ __forceinline__ float2 silu_for(float2 v) {
    if constexpr (sizeof(T) == 4) return make_float2(silu_for<T>(v.x), silu_for<T>(v.y));
    const float2 x = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(exp2_approx(x.x), exp2_approx(x.y)), make_float2(1.f, 1.f));
    return __fmul2_rn(v, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}

// Asynchronous copy of `bytes` bytes (2, 4, ... kBytes) to shared memory, zeros behind them.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(src), "r"(bytes), "n"(kBytes)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
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
