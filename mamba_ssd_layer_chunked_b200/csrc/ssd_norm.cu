// ssd_norm.cu -- the norms of a block, each with what a block does around it:
// the gated norm after the mixer and the norm before a block with its residual
// sum.
//
//   gated:  v = x silu(z), out = w v / sqrt(mean_group v^2 + eps)   (or the gate after the norm)
//   add:    r = residual + alpha scale x, out = w r / sqrt(mean r^2 + eps), r returned
//
// Source: "Mamba-2" (awesome.papernotes.org), design 3: the extra norm before
// the output projection, after the gate of the Mamba block (ai.tomabc.com).
//
// Bound by bytes: every operand once. A CTA holds one row's group in registers
// (up to 32 channels per thread), so the sum of squares and the scaled output
// need one read. Sums: fp32 per thread, then a fixed tree over the CTA.

#include "ssd_block.cuh"

namespace ssd {

namespace {

constexpr int kNormMaxThreads = 1024;

// The CTA's sum of v in a fixed order (same result on every thread).
__device__ __forceinline__ float cta_sum(float v) {
    __shared__ float part[32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x / 32;
    if (warps == 1) return v;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = (int)(threadIdx.x % 32) < warps ? part[threadIdx.x % 32] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v *= silu(z)
template <typename T, int V>
__device__ __forceinline__ void gate(float (&v)[V], const float (&z)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 s = silu_for<T>(make_float2(z[e], z[e + 1]));
            v[e] *= s.x, v[e + 1] *= s.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= silu_for<T>(z[e]);
    }
}

// One CTA per (row, group); thread i takes the group's vectors i, i + threads, ...
// (NV of them at most). R: type of the residual (mode add).
template <typename T, typename R, int V, int NV, int kMode>
__global__ void __launch_bounds__(kNormMaxThreads) row_norm_kernel(const NormArgs a, int group, int nvec) {
    const int row = blockIdx.x / a.ngroups, g = blockIdx.x % a.ngroups;
    const int b = row / a.seqlen, t = row - b * a.seqlen;
    const int c0 = g * group;
    const T* x = static_cast<const T*>(a.x) + b * a.xs_b + t * a.xs_t + c0;
    const T* z = static_cast<const T*>(a.z) + b * a.zs_b + t * a.zs_t + c0;
    const R* res = static_cast<const R*>(a.z) + b * a.zs_b + t * a.zs_t;
    const int64_t o = (int64_t)row * a.channels + c0;
    Pack<T, V> xv[NV], zv[kMode == kNormGateFirst || kMode == kNormGateLast ? NV : 1];
    Pack<R, V> rv[kMode == kNormAdd ? NV : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nvec) break;
        xv[k] = reinterpret_cast<const Pack<T, V>*>(x)[i];
        if constexpr (kMode == kNormGateFirst || kMode == kNormGateLast)
            zv[k] = reinterpret_cast<const Pack<T, V>*>(z)[i];
        if constexpr (kMode == kNormAdd) {
            if (a.z) rv[k] = reinterpret_cast<const Pack<R, V>*>(res)[i];
        }
    }
    float v[NV][V], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nvec) break;
        unpack(xv[k], v[k]);
        if constexpr (kMode == kNormGateFirst) {
            float zf[V];
            unpack(zv[k], zf);
            gate<T>(v[k], zf);
        }
        if constexpr (kMode == kNormAdd) {
            float rf[V];
            if (a.z) unpack(rv[k], rf);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[k][e] *= a.scale ? a.alpha * a.scale[i * V + e] : a.alpha;
                if (a.z) v[k][e] += rf[e];
            }
            reinterpret_cast<Pack<R, V>*>(static_cast<R*>(a.residual_out) + o)[i] = pack<R, V>(v[k]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(v[k][e], v[k][e], ss);
    }
    const float inv = 1.f / sqrtf(cta_sum(ss) / (float)group + a.eps);
    T* out = static_cast<T*>(a.out) + o;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i >= nvec) break;
        const Pack<float, V> w = reinterpret_cast<const Pack<float, V>*>(a.weight + c0)[i];
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] *= inv * w.v[e];
        if constexpr (kMode == kNormGateLast) {
            float zf[V];
            unpack(zv[k], zf);
            gate<T>(v[k], zf);
        }
        reinterpret_cast<Pack<T, V>*>(out)[i] = pack<T, V>(v[k]);
    }
}

template <typename T, typename R, int V, int NV, int kMode>
cudaError_t run(const NormArgs& a, int group, int nvec, cudaStream_t st) {
    const int threads = ((nvec + NV - 1) / NV + 31) / 32 * 32;
    const unsigned grid = (unsigned)((int64_t)a.batch * a.seqlen * a.ngroups);
    row_norm_kernel<T, R, V, NV, kMode><<<grid, threads, 0, st>>>(a, group, nvec);
    return cudaGetLastError();
}

// Vectors per thread. Fewer threads with more bytes each keep more rows in flight
// per SM across the CTA's one synchronisation. Rows of 5120 bf16 (640 vectors,
// 16384 rows): gated 123 us with 1 vector per thread, 92 with 2, 84 with 4 (93 % of
// the copy bandwidth). Rows of 2560 (320 vectors) with an fp32 residual: 81 us with
// 1 or 2, 92 with 4, whose wider rows cost occupancy. Rows of odd length go element by
// element: 5001 bf16 per row 164 us with 8 per thread, 283 with 32.
template <typename T, typename R, int V, int kMode>
cudaError_t by_count(const NormArgs& a, int group, cudaStream_t st) {
    const int nvec = group / V;
    if constexpr (V > 1) {
        if (nvec <= 256) return run<T, R, V, 1, kMode>(a, group, nvec, st);
        if (nvec <= 512) return run<T, R, V, 2, kMode>(a, group, nvec, st);
        if (V == 8 || nvec <= 2048) return run<T, R, V, 4, kMode>(a, group, nvec, st);
        return run<T, R, V, 32 / V, kMode>(a, group, nvec, st);
    } else {
        if (nvec <= 2048) return run<T, R, V, 4, kMode>(a, group, nvec, st);
        if (nvec <= 8 * kNormMaxThreads) return run<T, R, V, 8, kMode>(a, group, nvec, st);
        return run<T, R, V, 32, kMode>(a, group, nvec, st);
    }
}

template <typename T, typename R, int kMode>
cudaError_t by_access(const NormArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int group = a.channels / a.ngroups;
    // the residual and the parameters may be wider than x: then V of them are two accesses
    VectorRule r(sizeof(T)), q(sizeof(R)), w(sizeof(float));
    r.address(a.x).address(a.out).elements(a.xs_b).elements(a.xs_t).elements(group);
    q.elements(group);
    if (a.z) q.address(a.z).elements(a.zs_b).elements(a.zs_t);
    if (kMode == kNormAdd) q.address(a.residual_out);
    w.address(a.weight);
    const bool vec = r.multiple_of(16) && q.multiple_of(sizeof(Pack<R, V>) < 16 ? sizeof(Pack<R, V>) : 16) && w.multiple_of(16);
    return vec ? by_count<T, R, V, kMode>(a, group, st) : by_count<T, R, 1, kMode>(a, group, st);
}

template <typename T>
cudaError_t by_mode(const NormArgs& a, ssd_dtype residual_dt, cudaStream_t st) {
    switch (a.mode) {
        case kNormPlain: return by_access<T, T, kNormPlain>(a, st);
        case kNormGateFirst: return by_access<T, T, kNormGateFirst>(a, st);
        case kNormGateLast: return by_access<T, T, kNormGateLast>(a, st);
        default:
            return residual_dt == SSD_DTYPE_F32 ? by_access<T, float, kNormAdd>(a, st)
                                                : by_access<T, T, kNormAdd>(a, st);
    }
}

}  // namespace

cudaError_t launch_row_norm(const NormArgs& a, ssd_dtype dt, ssd_dtype residual_dt, cudaStream_t st) {
    return dt == SSD_DTYPE_F32 ? by_mode<float>(a, residual_dt, st) : by_mode<__nv_bfloat16>(a, residual_dt, st);
}

}  // namespace ssd
