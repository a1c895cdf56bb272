// ssd_selective.cu -- the selective scan with a decay per channel and state, for
// prompts (packed sequences, initial and final states) and for single tokens.
//
//   delta = softplus(dt + bias),  h[n] <- exp(delta A[n]) h[n] + delta u B[n]
//   y = (sum_n C[n] h[n] + D u) silu(z)
//
// Source: "Mamba" (ai.tomabc.com): the selective SSM of the block pseudocode,
// discretised with delta. Every (channel, state) decays at its own rate, so the
// chunked matrix form of the scalar-decay scan does not exist here: the work is
// one exponential and three multiply-adds per (token, channel, state).
//
// Prompts: a CTA owns 32 channels of one row and walks its tokens. Lane =
// channel; a warp holds S of the N states of its 32 channels in registers, so
// B and C are warp-uniform (broadcast from shared memory) and no shuffles are
// needed. Tokens are staged 32 at a time: delta and delta u are computed once
// per (token, channel) and shared by the warps; the warps' partial read-outs
// meet in shared memory, where the gate is applied.

#include "ssd_block.cuh"

namespace ssd {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTok = 32;  // tokens per staged tile (one bit each of the start mask)

// 2^x, the hardware approximation (denormal results flushed to 0)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float softplus(float z) { return z > 20.f ? z : log1pf(expf(z)); }

// S states per warp, NW = ceil(N / S) warps
template <typename T, int S>
__global__ void selective_scan_kernel(const SelectiveArgs a, int blocks_per_group) {
    extern __shared__ float4 smem4[];
    const int NW = blockDim.x / 32, w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int Np = NW * S, N = a.dstate;
    float* sm_delta = reinterpret_cast<float*>(smem4);  // [kTok][32]
    float* sm_du = sm_delta + kTok * 32;                // [kTok][32]
    float* sm_B = sm_du + kTok * 32;                    // [kTok][Np]
    float* sm_C = sm_B + kTok * Np;                     // [kTok][Np]
    float* sm_y = sm_C + kTok * Np;                     // [NW][kTok][32]
    int* sm_id = reinterpret_cast<int*>(sm_y + NW * kTok * 32);  // [kTok]

    const int per = a.channels / a.ngroups;
    const int b = blockIdx.x / (a.ngroups * blocks_per_group);
    const int gb = blockIdx.x % (a.ngroups * blocks_per_group);
    const int g = gb / blocks_per_group;
    const int cg = (gb % blocks_per_group) * 32 + lane;  // channel within the group
    const bool live = cg < per;
    const int c = g * per + (live ? cg : per - 1);
    const int64_t row0 = (int64_t)b * a.seqlen;
    const T* u = static_cast<const T*>(a.u) + b * a.us_b + c;
    const T* dt = static_cast<const T*>(a.dt) + b * a.ds_b + c;
    const T* z = static_cast<const T*>(a.z) + b * a.zs_b + c;
    const T* B = static_cast<const T*>(a.B) + b * a.bs_b + g * N;
    const T* C = static_cast<const T*>(a.C) + b * a.cs_b + g * N;
    T* y = static_cast<T*>(a.y) + row0 * a.channels + c;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    const float D = a.D ? a.D[c] : 0.f;

    float A2[S], h[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int n = w * S + j;
        A2[j] = n < N ? a.A[(int64_t)c * N + n] * kLog2e : 0.f;
        h[j] = 0.f;
    }
    const auto state_at = [&](int s, int n) { return (((int64_t)b * a.nseq + s) * N + n) * a.channels + c; };
    // ids that do not occur keep their initial state
    const auto keep = [&](int lo, int hi) {
        if (!a.final_states || !live) return;
        for (int s = lo; s < hi; ++s)
#pragma unroll
            for (int j = 0; j < S; ++j) {
                const int n = w * S + j;
                if (n < N) a.final_states[state_at(s, n)] = a.init ? a.init[state_at(s, n)] : 0.f;
            }
    };
    const auto finish = [&](int s) {  // the state after a sequence's last token
        if (!a.final_states || !live) return;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int n = w * S + j;
            if (n < N) a.final_states[state_at(s, n)] = h[j];
        }
    };
    int cur = -1;  // the sequence that h belongs to
    const auto enter = [&](int s) {
        if (cur >= 0) finish(cur);
        keep(cur + 1, s);
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int n = w * S + j;
            h[j] = a.init && n < N ? a.init[state_at(s, n)] : 0.f;
        }
        cur = s;
    };

    for (int t0 = 0; t0 < a.seqlen; t0 += kTok) {
        const int nt = min(kTok, a.seqlen - t0);
        for (int t = w; t < nt; t += NW) {
            float d = to_f32(dt[(t0 + t) * a.ds_t]) + bias;
            if (a.softplus) d = softplus(d);
            sm_delta[t * 32 + lane] = d;
            sm_du[t * 32 + lane] = d * to_f32(u[(t0 + t) * a.us_t]);
        }
        for (int i = threadIdx.x; i < nt * Np; i += blockDim.x) {
            const int t = i / Np, n = i - t * Np;
            sm_B[i] = n < N ? to_f32(B[(t0 + t) * a.bs_t + n]) : 0.f;
            sm_C[i] = n < N ? to_f32(C[(t0 + t) * a.cs_t + n]) : 0.f;
        }
        if (w == 0) sm_id[lane] = seq_at(a.seq_idx, row0, min(t0 + lane, a.seqlen - 1), a.nseq);
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            if (sm_id[t] != cur) enter(sm_id[t]);
            const float d = sm_delta[t * 32 + lane], du = sm_du[t * 32 + lane];
            float acc = 0.f;
#pragma unroll
            for (int j = 0; j < S; ++j) {
                const float e = exp2_fast(d * A2[j]);
                h[j] = fmaf(e, h[j], du * sm_B[t * Np + w * S + j]);
                acc = fmaf(sm_C[t * Np + w * S + j], h[j], acc);
            }
            sm_y[(w * kTok + t) * 32 + lane] = acc;
        }
        __syncthreads();
        for (int t = w; t < nt; t += NW) {
            float v = D * to_f32(u[(t0 + t) * a.us_t]);
            for (int k = 0; k < NW; ++k) v += sm_y[(k * kTok + t) * 32 + lane];
            if (a.z) v *= silu_for<T>(to_f32(z[(t0 + t) * a.zs_t]));
            if (live) y[(int64_t)(t0 + t) * a.channels] = from_f32<T>(v);
        }
    }
    finish(cur);
    keep(cur + 1, a.nseq);
}

constexpr int kStepThreads = 128;

// One thread per (row, channel): its N states in and out, in batches of 16.
template <typename T>
__global__ void __launch_bounds__(kStepThreads) selective_step_kernel(const SelectiveArgs a, int blocks) {
    const int b = blockIdx.x / blocks;
    const int c = (blockIdx.x % blocks) * kStepThreads + threadIdx.x;
    if (c >= a.channels) return;
    const int N = a.dstate, g = c / (a.channels / a.ngroups);
    const float uf = to_f32(static_cast<const T*>(a.u)[b * a.us_b + c]);
    float d = to_f32(static_cast<const T*>(a.dt)[b * a.ds_b + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
    if (a.softplus) d = softplus(d);
    const float du = d * uf;
    const T* B = static_cast<const T*>(a.B) + b * a.bs_b + g * N;
    const T* C = static_cast<const T*>(a.C) + b * a.cs_b + g * N;
    float* h = a.final_states + (int64_t)b * N * a.channels + c;
    const float* A = a.A + (int64_t)c * N;
    float y = a.D ? a.D[c] * uf : 0.f;
    for (int n0 = 0; n0 < N; n0 += 16) {
        float hv[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (n0 + j < N) hv[j] = h[(int64_t)(n0 + j) * a.channels];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (n0 + j < N) {
                const float e = exp2_fast(d * (A[n0 + j] * kLog2e));
                const float v = fmaf(e, hv[j], du * to_f32(B[n0 + j]));
                h[(int64_t)(n0 + j) * a.channels] = v;
                y = fmaf(to_f32(C[n0 + j]), v, y);
            }
    }
    if (a.z) y *= silu_for<T>(to_f32(static_cast<const T*>(a.z)[b * a.zs_b + c]));
    static_cast<T*>(a.y)[(int64_t)b * a.channels + c] = from_f32<T>(y);
}

template <typename T, int S>
cudaError_t run_scan(const SelectiveArgs& a, cudaStream_t st) {
    const int NW = (a.dstate + S - 1) / S;
    const int per = a.channels / a.ngroups, bpg = (per + 31) / 32;
    const size_t smem = (size_t)(2 * kTok * 32 + 2 * kTok * NW * S + NW * kTok * 32 + kTok) * sizeof(float);
    static_assert(2 * kTok * 32 + 2 * kTok * 256 + 16 * kTok * 32 + kTok <= 227 * 256, "fits one SM");
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute((const void*)selective_scan_kernel<T, S>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    selective_scan_kernel<T, S><<<(unsigned)((int64_t)a.batch * a.ngroups * bpg), NW * 32, smem, st>>>(a, bpg);
    return cudaGetLastError();
}

template <typename T>
cudaError_t scan_by_states(const SelectiveArgs& a, cudaStream_t st) {
    return a.dstate <= 64 ? run_scan<T, 4>(a, st) : run_scan<T, 16>(a, st);
}

}  // namespace

cudaError_t launch_selective_scan(const SelectiveArgs& a, ssd_dtype dt, cudaStream_t st) {
    return dt == SSD_DTYPE_F32 ? scan_by_states<float>(a, st) : scan_by_states<__nv_bfloat16>(a, st);
}

cudaError_t launch_selective_step(const SelectiveArgs& a, ssd_dtype dt, cudaStream_t st) {
    const int blocks = (a.channels + kStepThreads - 1) / kStepThreads;
    const unsigned grid = (unsigned)((int64_t)a.batch * blocks);
    if (dt == SSD_DTYPE_F32)
        selective_step_kernel<float><<<grid, kStepThreads, 0, st>>>(a, blocks);
    else
        selective_step_kernel<__nv_bfloat16><<<grid, kStepThreads, 0, st>>>(a, blocks);
    return cudaGetLastError();
}

}  // namespace ssd
