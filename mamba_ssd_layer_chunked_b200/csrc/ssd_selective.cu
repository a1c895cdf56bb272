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
// Prompts: a warp owns a few channels of one row, LN lanes per channel with S
// states each in registers, and a CTA's K warps take consecutive slices of
// kSlice tokens, so that the exponentials of K * kSlice tokens are formed at
// once although the recurrence is sequential. Over a slice the recurrence is
// affine, h_end = P h_start + E: each warp forms its a = exp(delta A) (kept in
// registers), E and P, the warps exchange (E, P) once per tile through shared
// memory, each chains the slices before its own, and walks its slice again from
// the true state, with the kept a, for the read-out. Every exponential is formed
// once. Bound by the special-function unit (one exponential per (token,
// channel, state)), then by the issue rate.

#include "ssd_block.cuh"

namespace ssd {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSlice = 8;       // tokens per warp and tile
constexpr int kPairStride = 20; // floats between channels' (delta, delta u) rows: 16 used, conflict-free

// 2^x, the hardware approximation (denormal results flushed to 0)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softplus(z) = max(z, 0) + log(1 + e), e = exp(-|z|) in [0, 1]. The logarithm
// as 2 atanh(r), r = e / (2 + e) <= 1/3, by its power series: the first term left
// out is r^17 / 17 < 5e-10 of r, and small e keep their relative accuracy, which
// log(1 + e) taken directly would lose.
__device__ __forceinline__ float softplus(float z) {
    const float e = exp2_fast(-kLog2e * fabsf(z));
    const float r = __fdividef(e, 2.f + e), q = r * r;
    float s = 1.f / 15.f;
    s = fmaf(s, q, 1.f / 13.f);
    s = fmaf(s, q, 1.f / 11.f);
    s = fmaf(s, q, 1.f / 9.f);
    s = fmaf(s, q, 1.f / 7.f);
    s = fmaf(s, q, 1.f / 5.f);
    s = fmaf(s, q, 1.f / 3.f);
    s = fmaf(s, q, 1.f);
    return fmaf(2.f * r, s, fmaxf(z, 0.f));
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Lane = state slice * CPW + channel, CPW = 32 / LN channels per warp; a lane
// holds states [ns * S, ns * S + S) of its channel. For loading inputs and
// storing outputs a lane owns kSlice / LN tokens of its channel (one, shared by
// LN / kSlice lanes, where LN > kSlice): those whose read-out it ends up with.
template <typename T, int S, int LN, int K, bool kSeq>
__global__ void __launch_bounds__(32 * K, K == 4 ? 5 : 1) selective_scan_kernel(const SelectiveArgs a,
                                                                                int units_per_group) {
    constexpr int CPW = 32 / LN, NP = S * LN, S2 = S / 2;
    constexpr int TPL = LN < kSlice ? kSlice / LN : 1;       // tokens owned by a lane
    constexpr int SHARE = LN > kSlice ? LN / kSlice : 1;     // lanes that own the same token
    constexpr int VEC = 16 / (int)sizeof(T);                 // B, C elements per 16-byte load
    constexpr int NV = kSlice * 2 * NP / VEC / 32;           // such loads per lane and slice
    constexpr bool kAhead = NV >= 1 && NV <= 2;              // load a tile ahead, in registers
    extern __shared__ float4 smem4[];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int ch = lane % CPW, ns = lane / CPW, N = a.dstate;
    float* sm_pair = reinterpret_cast<float*>(smem4) + w * (CPW * kPairStride);
    float* sm_bc = reinterpret_cast<float*>(smem4) + K * (CPW * kPairStride) + w * (kSlice * 2 * NP);
    // [2 buffers][K][E, P][S / 4][32] float4
    float4* sm_ep = smem4 + K * (CPW * kPairStride + kSlice * 2 * NP) / 4;

    const int per = a.channels / a.ngroups;
    const int unit = blockIdx.x % units_per_group, bg = blockIdx.x / units_per_group;
    const int g = bg % a.ngroups, b = bg / a.ngroups;
    const bool live = unit * CPW + ch < per;
    const int c = g * per + (live ? unit * CPW + ch : per - 1);
    const int64_t row0 = (int64_t)b * a.seqlen;
    const int own = ns * kSlice / LN;  // first token of the slice that this lane owns
    const bool owner = live && ns % SHARE == 0;
    const T* u = static_cast<const T*>(a.u) + b * a.us_b + c;
    const T* dt = static_cast<const T*>(a.dt) + b * a.ds_b + c;
    const T* z = static_cast<const T*>(a.z) + b * a.zs_b + c;
    const T* B = static_cast<const T*>(a.B) + b * a.bs_b + g * N;
    const T* C = static_cast<const T*>(a.C) + b * a.cs_b + g * N;
    T* y = static_cast<T*>(a.y) + row0 * a.channels + c;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    const float D = a.D ? a.D[c] : 0.f;

    float2 A2[S2];
#pragma unroll
    for (int j = 0; j < S2; ++j) {
        const int n = ns * S + 2 * j;
        A2[j].x = n < N ? a.A[(int64_t)c * N + n] * kLog2e : 0.f;
        A2[j].y = n + 1 < N ? a.A[(int64_t)c * N + n + 1] * kLog2e : 0.f;
    }
    const auto state_at = [&](int s, int n) { return (((int64_t)b * a.nseq + s) * N + n) * a.channels + c; };
    const auto init_state = [&](float2(&h)[S2], int s) {
#pragma unroll
        for (int j = 0; j < S2; ++j) {
            const int n = ns * S + 2 * j;
            h[j].x = a.init && n < N ? a.init[state_at(s, n)] : 0.f;
            h[j].y = a.init && n + 1 < N ? a.init[state_at(s, n + 1)] : 0.f;
        }
    };
    const auto write_state = [&](const float2(&h)[S2], int s) {
        if (!a.final_states || !live) return;
#pragma unroll
        for (int j = 0; j < S2; ++j) {
            const int n = ns * S + 2 * j;
            if (n < N) a.final_states[state_at(s, n)] = h[j].x;
            if (n + 1 < N) a.final_states[state_at(s, n + 1)] = h[j].y;
        }
    };
    // ids that do not occur keep their initial state
    const auto keep = [&](int lo, int hi) {
        for (int s = lo; s < hi; ++s) {
            float2 h[S2];
            init_state(h, s);
            write_state(h, s);
        }
    };

    // the lane's raw inputs of one slice
    T ru[TPL], rd[TPL], rz[TPL];
    const auto load_tokens = [&](int tw) {
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            const int t = tw + own + i;
            ru[i] = rd[i] = rz[i] = from_f32<T>(0.f);
            if (t < a.seqlen) {
                ru[i] = u[t * a.us_t];
                rd[i] = dt[t * a.ds_t];
                if (a.z) rz[i] = z[t * a.zs_t];
            }
        }
    };
    uint4 rbc[kAhead ? NV : 1];
    // vector i of the slice's B and C: token, which of the two, first state
    const auto bc_vector = [&](int tw, int i) {
        constexpr int PT = NV >= 1 ? 2 * NP / VEC : 1;  // vectors per token
        const int v = lane + 32 * i, tok = v / PT, r = v % PT, n = (r % (PT / 2 > 0 ? PT / 2 : 1)) * VEC;
        const int t = tw + tok;
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (n < N && t < a.seqlen)
            raw = *reinterpret_cast<const uint4*>((r < PT / 2 ? B + t * a.bs_t : C + t * a.cs_t) + n);
        return raw;
    };
    const auto put_bc = [&](const uint4& raw, int i) {  // vectors lie in shared memory in their order
        const T* e = reinterpret_cast<const T*>(&raw);
        float* dst = sm_bc + (lane + 32 * i) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; k += 4)
            *reinterpret_cast<float4*>(dst + k) =
                make_float4(to_f32(e[k]), to_f32(e[k + 1]), to_f32(e[k + 2]), to_f32(e[k + 3]));
    };
    const auto load_bc = [&](int tw) {
        if constexpr (kAhead) {
            if (a.bc_vectors) {
#pragma unroll
                for (int i = 0; i < NV; ++i) rbc[i] = bc_vector(tw, i);
            }
        }
    };

    float2 h0[S2];  // the state before the tile, the same in every warp
    init_state(h0, 0);
    if (kSeq) {
#pragma unroll
        for (int j = 0; j < S2; ++j) h0[j] = both(0.f);
    }
    load_tokens(w * kSlice);
    load_bc(w * kSlice);
    int buf = 0;
    for (int t0 = 0; t0 < a.seqlen; t0 += K * kSlice, buf ^= 1) {
        const int tw = t0 + w * kSlice;
        // ---- this slice's inputs: (delta, delta u), B, C to shared memory ----
        __syncwarp();
        float skip[TPL], gate[TPL];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            const float uf = to_f32(ru[i]);
            float d = to_f32(rd[i]) + bias;
            if (a.softplus) d = softplus(d);
            if (tw + own + i >= a.seqlen) d = 0.f;  // past the end: a = 1 and no input
            skip[i] = D * uf;
            gate[i] = a.z ? silu_for<T>(to_f32(rz[i])) : 1.f;
            *reinterpret_cast<float2*>(sm_pair + ch * kPairStride + 2 * (own + i)) = make_float2(d, d * uf);
        }
        bool staged = false;
        if constexpr (NV >= 1) {
            if (a.bc_vectors) {
                staged = true;
#pragma unroll
                for (int i = 0; i < NV; ++i) put_bc(kAhead ? rbc[kAhead ? i : 0] : bc_vector(tw, i), i);
            }
        }
        if (!staged) {
            for (int i = lane; i < kSlice * 2 * NP; i += 32) {
                const int tok = i / (2 * NP), r = i % (2 * NP), n = r % NP, t = tw + tok;
                float v = 0.f;
                if (n < N && t < a.seqlen) v = to_f32(r < NP ? B[t * a.bs_t + n] : C[t * a.cs_t + n]);
                sm_bc[i] = v;
            }
        }
        // sequences that start in this slice: lane i < kSlice looks at token tw + i
        unsigned starts = 0u;
        int id = 0, id_before = -1;
        if (kSeq) {
            const int t = min(tw + lane % kSlice, a.seqlen - 1);
            id = seq_at(a.seq_idx, row0, t, a.nseq);
            if (t > 0) id_before = seq_at(a.seq_idx, row0, t - 1, a.nseq);
            starts = __ballot_sync(0xffffffffu, lane < kSlice && tw + lane < a.seqlen && (t == 0 || id != id_before));
        }
        __syncwarp();
        load_tokens(tw + K * kSlice);
        load_bc(tw + K * kSlice);
        // ---- the slice from zero: a (kept), end state E, product P ----
        float2 av[kSlice][S2], E[S2], P[S2];
#pragma unroll
        for (int j = 0; j < S2; ++j) E[j] = both(0.f), P[j] = both(1.f);
#pragma unroll
        for (int t = 0; t < kSlice; ++t) {
            const float2 dd = *reinterpret_cast<const float2*>(sm_pair + ch * kPairStride + 2 * t);
            const float2* Bt = reinterpret_cast<const float2*>(sm_bc + t * 2 * NP + ns * S);
            if (kSeq && (starts >> t & 1u)) {
                init_state(E, __shfl_sync(0xffffffffu, id, t));
#pragma unroll
                for (int j = 0; j < S2; ++j) P[j] = both(0.f);
            }
#pragma unroll
            for (int j = 0; j < S2; ++j) {
                const float2 x = __fmul2_rn(both(dd.x), A2[j]);
                av[t][j] = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                E[j] = __ffma2_rn(av[t][j], E[j], __fmul2_rn(both(dd.y), Bt[j]));
                P[j] = __fmul2_rn(P[j], av[t][j]);
            }
        }
        // ---- chain the slices: the state before this one, and before the next tile ----
        float4* ep = sm_ep + (buf * K * 2) * (S / 4) * 32 + lane;
#pragma unroll
        for (int j = 0; j < S / 4; ++j) {
            ep[((w * 2 + 0) * (S / 4) + j) * 32] = make_float4(E[2 * j].x, E[2 * j].y, E[2 * j + 1].x, E[2 * j + 1].y);
            ep[((w * 2 + 1) * (S / 4) + j) * 32] = make_float4(P[2 * j].x, P[2 * j].y, P[2 * j + 1].x, P[2 * j + 1].y);
        }
        __syncthreads();
        float2 h[S2];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k == w) {
#pragma unroll
                for (int j = 0; j < S2; ++j) h[j] = h0[j];
            }
#pragma unroll
            for (int j = 0; j < S / 4; ++j) {
                const float4 e = ep[((k * 2 + 0) * (S / 4) + j) * 32], p = ep[((k * 2 + 1) * (S / 4) + j) * 32];
                h0[2 * j] = __ffma2_rn(make_float2(p.x, p.y), h0[2 * j], make_float2(e.x, e.y));
                h0[2 * j + 1] = __ffma2_rn(make_float2(p.z, p.w), h0[2 * j + 1], make_float2(e.z, e.w));
            }
        }
        // ---- the slice from its true state, and the read-out ----
        float acc[kSlice];
#pragma unroll
        for (int t = 0; t < kSlice; ++t) {
            const float du = sm_pair[ch * kPairStride + 2 * t + 1];
            const float2* Bt = reinterpret_cast<const float2*>(sm_bc + t * 2 * NP + ns * S);
            const float2* Ct = reinterpret_cast<const float2*>(sm_bc + t * 2 * NP + NP + ns * S);
            if (kSeq && (starts >> t & 1u)) {
                const int s = __shfl_sync(0xffffffffu, id, t), p = __shfl_sync(0xffffffffu, id_before, t);
                if (p >= 0) write_state(h, p);
                keep(p + 1, s);
                init_state(h, s);
            }
            float2 r = both(0.f);
#pragma unroll
            for (int j = 0; j < S2; ++j) {
                h[j] = __ffma2_rn(av[t][j], h[j], __fmul2_rn(both(du), Bt[j]));
                r = __ffma2_rn(Ct[j], h[j], r);
            }
            acc[t] = r.x + r.y;
        }
        if (a.final_states && tw < a.seqlen && tw + kSlice >= a.seqlen) {  // this slice has the last token
            const int s = kSeq ? __shfl_sync(0xffffffffu, id, a.seqlen - 1 - tw) : 0;
            write_state(h, s);
            keep(s + 1, a.nseq);
        }
        // ---- sum over the channel's lanes; each ends with the tokens it owns ----
#pragma unroll
        for (int m = LN / 2, n = kSlice; m >= 1; m /= 2) {
            if (n > 1) {  // keep the half of the tokens that the lane's side owns
                n /= 2;
                const bool up = ns & m;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float give = up ? acc[i] : acc[i + n], stay = up ? acc[i + n] : acc[i];
                    acc[i] = stay + __shfl_xor_sync(0xffffffffu, give, m * CPW);
                }
            } else {
                acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], m * CPW);
            }
        }
        if (owner) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const int t = tw + own + i;
                if (t < a.seqlen) y[(int64_t)t * a.channels] = from_f32<T>((acc[i] + skip[i]) * gate[i]);
            }
        }
    }
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

template <typename T, int S, int LN, int K>
cudaError_t run_scan(const SelectiveArgs& a, cudaStream_t st) {
    constexpr int CPW = 32 / LN, NP = S * LN;
    constexpr int smem = (K * (CPW * kPairStride + kSlice * 2 * NP) + 2 * K * 2 * S * 32) * (int)sizeof(float);
    static_assert(smem <= 227 * 1024, "fits one SM");
    const int per = a.channels / a.ngroups, units = (per + CPW - 1) / CPW;
    const unsigned grid = (unsigned)((int64_t)a.batch * a.ngroups * units);
    const auto kernel = a.seq_idx ? selective_scan_kernel<T, S, LN, K, true> : selective_scan_kernel<T, S, LN, K, false>;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, 32 * K, smem, st>>>(a, units);
    return cudaGetLastError();
}

template <typename T, int S, int LN>
cudaError_t scan_by_slices(const SelectiveArgs& a, cudaStream_t st) {
    const int64_t units = (int64_t)a.batch * a.ngroups * ((a.channels / a.ngroups + 32 / LN - 1) / (32 / LN));
    // 16 warps per CTA where the CTAs do not fill the GPU's SMs twice, else 4
    if constexpr (S * LN <= 128) {
        if (units < 2 * 148 && a.seqlen > 4 * kSlice) return run_scan<T, S, LN, 16>(a, st);
    }
    return run_scan<T, S, LN, 4>(a, st);
}

template <typename T>
cudaError_t scan_by_states(SelectiveArgs a, cudaStream_t st) {
    VectorRule r(sizeof(T));
    r.address(a.B).address(a.C).elements(a.bs_b).elements(a.bs_t).elements(a.cs_b).elements(a.cs_t).elements(a.dstate);
    a.bc_vectors = r.multiple_of(16);
    if (a.dstate <= 8) return scan_by_slices<T, 4, 2>(a, st);
    if (a.dstate <= 16) return scan_by_slices<T, 4, 4>(a, st);
    if (a.dstate <= 32) return scan_by_slices<T, 4, 8>(a, st);
    if (a.dstate <= 64) return scan_by_slices<T, 4, 16>(a, st);
    if (a.dstate <= 128) return scan_by_slices<T, 4, 32>(a, st);
    return scan_by_slices<T, 8, 32>(a, st);
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
