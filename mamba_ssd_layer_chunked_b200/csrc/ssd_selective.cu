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
// affine in the state before it: with the local state (from zero) l_t and the
// decay p_t since the slice's start, h_t = l_t + p_t h_start, so
//   y_t = C_t . l_t + (C_t p_t) . h_start.
// Each warp walks its slice once, keeping C_t p_t in registers, the warps
// exchange (l_end, p_end) once per tile through shared memory, each chains the
// slices before its own, and adds the second term. Every exponential is formed
// once. Bound by the special-function unit (one exponential per (token,
// channel, state)) and the issue rate together.

#include "ssd_block.cuh"

namespace ssd {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSlice = 8;       // tokens per warp and tile

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
__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }

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

constexpr int kStages = 3;  // slices of raw inputs in shared memory: two in flight behind the current one

// Layout of the scan's shared memory and its copies, for S states per lane, LN
// lanes per channel, K warps.
template <typename T, int S, int LN, int K>
struct ScanShape {
    static constexpr int CPW = 32 / LN;                                // channels per warp
    static constexpr int NP = S * LN;                                  // states, padded
    static constexpr int E = (int)sizeof(T);
    static constexpr int TPL = LN < kSlice ? kSlice / LN : 1;          // tokens owned by a lane
    static constexpr int SHARE = LN > kSlice ? LN / kSlice : 1;        // lanes that own the same token
    static constexpr int ROW = CPW * E;                                // bytes of a token's channels
    static constexpr int TB = ROW < 16 ? ROW : 16;                     // bytes per copy of u, dt, z
    static constexpr int TR = (3 * kSlice * ROW / TB + 31) / 32;       // such copies per lane and slice
    static constexpr int BV = 16 / E;                                  // B, C elements per copy
    static constexpr int BR = kSlice * 2 * NP / BV / 32;               // such copies per lane and slice
    static constexpr bool kCanCopy = TB >= 4 && NP >= BV && BR >= 1 && BR <= 4;
    static constexpr int PAIR = CPW * (kSlice * 4 + 4);                // floats: (delta, delta, du, du) per token
    static constexpr int BC = kSlice * 2 * NP;                         // floats: B and C of the slice
    static constexpr int RAW = 3 * kSlice * ROW + BC * E;              // bytes of a raw stage
    static constexpr int smem(bool copies) {
        return K * (PAIR + BC) * 4 + 2 * K * 2 * S * 32 * 4 + (copies ? K * kStages * RAW : 0);
    }
};

// Lane = state slice * CPW + channel; a lane holds states [ns * S, ns * S + S) of
// its channel. A lane owns the kSlice / LN tokens of its channel (one, shared by
// LN / kSlice lanes, where LN > kSlice) whose read-out it ends up with: it
// prepares their inputs and stores their outputs.
// kCopy: all rows allow the asynchronous copies of ScanShape; else element loads.
template <typename T, int S, int LN, int K, bool kSeq, bool kCopy>
__global__ void __launch_bounds__(32 * K, K == 4 ? 5 : 1) selective_scan_kernel(const SelectiveArgs a,
                                                                                int units_per_group) {
    using Sh = ScanShape<T, S, LN, K>;
    constexpr int CPW = Sh::CPW, NP = Sh::NP, S2 = S / 2, S4 = S / 4, TPL = Sh::TPL;
    constexpr int PROW = kSlice * 4 + 4;
    extern __shared__ float4 smem4[];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int ch = lane % CPW, ns = lane / CPW, N = a.dstate;
    float* sm_pair = reinterpret_cast<float*>(smem4) + w * Sh::PAIR;
    float* sm_bc = reinterpret_cast<float*>(smem4) + K * Sh::PAIR + w * Sh::BC;
    float4* sm_ep = smem4 + K * (Sh::PAIR + Sh::BC) / 4;  // [2 buffers][K][E, P][S / 4][32]
    char* sm_raw = reinterpret_cast<char*>(sm_ep + 2 * K * 2 * S4 * 32) + w * (kStages * Sh::RAW);

    const int per = a.channels / a.ngroups;
    const int unit = blockIdx.x % units_per_group, bg = blockIdx.x / units_per_group;
    const int g = bg % a.ngroups, b = bg / a.ngroups;
    const bool live = unit * CPW + ch < per;
    const int c = g * per + (live ? unit * CPW + ch : per - 1);
    const int64_t row0 = (int64_t)b * a.seqlen;
    const int own = ns * kSlice / LN;  // first token of the slice that this lane owns
    const bool owner = live && ns % Sh::SHARE == 0;
    const T* u = static_cast<const T*>(a.u) + b * a.us_b;
    const T* dt = static_cast<const T*>(a.dt) + b * a.ds_b;
    const T* z = static_cast<const T*>(a.z) + b * a.zs_b;
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
        if (!live) return;
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

    // ---- inputs, ahead of their use: copies into shared memory, or registers ----
    const T* tsrc[kCopy ? Sh::TR : 1];
    int64_t tstep[kCopy ? Sh::TR : 1];
    int tbytes[kCopy ? Sh::TR : 1];
    const T* bsrc[kCopy ? Sh::BR : 1];
    int64_t bstep[kCopy ? Sh::BR : 1];
    T ru[kCopy ? 1 : TPL], rd[kCopy ? 1 : TPL], rz[kCopy ? 1 : TPL];
    if constexpr (kCopy) {
#pragma unroll
        for (int i = 0; i < Sh::TR; ++i) {  // copy v: array (u, dt, z), token, part of the token's channels
            constexpr int PT = Sh::ROW / Sh::TB;
            const int v = lane + 32 * i, arr = v / (kSlice * PT), tok = v / PT % kSlice, part = v % PT;
            const int cg = unit * CPW + part * (Sh::TB / Sh::E);
            const int64_t step = arr == 0 ? a.us_t : arr == 1 ? a.ds_t : a.zs_t;
            tstep[i] = step * (K * kSlice);
            tsrc[i] = (arr == 0 ? u : arr == 1 ? dt : z) + (w * kSlice + tok) * step + (g * per + min(cg, per - 1));
            tbytes[i] = min(Sh::TB, max(0, per - cg) * Sh::E);
            if (arr == 2 && !a.z) tbytes[i] = 0, tsrc[i] = u;  // no gate: zeros
            if (arr > 2) tbytes[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < Sh::BR; ++i) {  // copy v: token, B or C, states
            constexpr int PT = 2 * NP / Sh::BV;
            const int v = lane + 32 * i, tok = v / PT, r = v % PT, n = r % (PT / 2) * Sh::BV;
            const int64_t step = r < PT / 2 ? a.bs_t : a.cs_t;
            bstep[i] = n < N ? step * (K * kSlice) : -1;
            bsrc[i] = (r < PT / 2 ? B : C) + (w * kSlice + tok) * step + (n < N ? n : 0);
        }
    }
    const auto fetch = [&](int tw, int stage) {  // the slice that starts at token tw
        if constexpr (kCopy) {
            char* dst = sm_raw + stage * Sh::RAW;
#pragma unroll
            for (int i = 0; i < Sh::TR; ++i) {
                const int v = lane + 32 * i, tok = v / (Sh::ROW / Sh::TB) % kSlice;
                if (tbytes[i] >= 0) {
                    const bool in = tw + tok < a.seqlen;
                    copy_async<Sh::TB>(dst + v * Sh::TB, in ? tsrc[i] : u, in ? tbytes[i] : 0);
                    tsrc[i] += tstep[i];
                }
            }
#pragma unroll
            for (int i = 0; i < Sh::BR; ++i) {
                const int v = lane + 32 * i, tok = v / (2 * NP / Sh::BV);
                const bool in = tw + tok < a.seqlen && bstep[i] >= 0;
                copy_async<16>(dst + 3 * kSlice * Sh::ROW + v * 16, in ? bsrc[i] : B, in ? 16 : 0);
                bsrc[i] += bstep[i];
            }
            copy_commit();
        } else {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const int t = tw + own + i;
                ru[i] = rd[i] = rz[i] = from_f32<T>(0.f);
                if (t < a.seqlen) {
                    ru[i] = u[t * a.us_t + c];
                    rd[i] = dt[t * a.ds_t + c];
                    if (a.z) rz[i] = z[t * a.zs_t + c];
                }
            }
        }
    };

    float2 h0[S2];  // the state before the tile, the same in every warp
    if (kSeq) {
#pragma unroll
        for (int j = 0; j < S2; ++j) h0[j] = both(0.f);
    } else {
        init_state(h0, 0);
    }
    fetch(w * kSlice, 0);
    if (kCopy) fetch((K + w) * kSlice, 1);
    int buf = 0, stage = 0;
    for (int t0 = 0; t0 < a.seqlen; t0 += K * kSlice, buf ^= 1) {
        const int tw = t0 + w * kSlice;
        // ---- this slice's (delta, delta u), B and C, in fp32 ----
        if (kCopy) copy_wait<1>();
        __syncwarp();
        const char* raw = sm_raw + stage * Sh::RAW;
        float skip[TPL], gate[TPL];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            float uf, d, zf;
            if constexpr (kCopy) {
                const T* e = reinterpret_cast<const T*>(raw) + (own + i) * CPW + ch;
                uf = to_f32(e[0]), d = to_f32(e[kSlice * CPW]), zf = to_f32(e[2 * kSlice * CPW]);
            } else {
                uf = to_f32(ru[i]), d = to_f32(rd[i]), zf = to_f32(rz[i]);
            }
            d += bias;
            if (a.softplus) d = softplus(d);
            if (tw + own + i >= a.seqlen) d = 0.f;  // past the end: a = 1 and no input
            skip[i] = D * uf;
            gate[i] = a.z ? silu_for<T>(zf) : 1.f;
            const float du = d * uf;
            *reinterpret_cast<float4*>(sm_pair + ch * PROW + 4 * (own + i)) = make_float4(d, d, du, du);
        }
        if constexpr (kCopy) {
#pragma unroll
            for (int i = 0; i < Sh::BR; ++i) {
                const int v = lane + 32 * i;
                const Pack<T, Sh::BV> e = *reinterpret_cast<const Pack<T, Sh::BV>*>(raw + 3 * kSlice * Sh::ROW + v * 16);
#pragma unroll
                for (int k = 0; k < Sh::BV; k += 4)
                    *reinterpret_cast<float4*>(sm_bc + v * Sh::BV + k) = make_float4(
                        to_f32(e.v[k]), to_f32(e.v[k + 1]), to_f32(e.v[k + 2]), to_f32(e.v[k + 3]));
            }
        } else {
            for (int i = lane; i < Sh::BC; i += 32) {
                const int tok = i / (2 * NP), r = i % (2 * NP), n = r % NP, t = tw + tok;
                float v = 0.f;
                if (n < N && t < a.seqlen) v = to_f32(r < NP ? B[t * a.bs_t + n] : C[t * a.cs_t + n]);
                sm_bc[i] = v;
            }
        }
        if (kCopy) {
            fetch(tw + 2 * K * kSlice, stage == 0 ? 2 : stage - 1);
            stage = stage == kStages - 1 ? 0 : stage + 1;
        } else {
            fetch(tw + K * kSlice, 0);
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
        // ---- the slice from zero: local state l, decay p, C l, and C p (kept) ----
        float2 l[S2], p[S2], cp[kSlice][S2], acc[kSlice];
#pragma unroll
        for (int j = 0; j < S2; ++j) l[j] = both(0.f), p[j] = both(1.f);
#pragma unroll
        for (int t = 0; t < kSlice; ++t) {
            const float4 dd = *reinterpret_cast<const float4*>(sm_pair + ch * PROW + 4 * t);
            const float4* Bt = reinterpret_cast<const float4*>(sm_bc + t * 2 * NP + ns * S);
            const float4* Ct = reinterpret_cast<const float4*>(sm_bc + t * 2 * NP + NP + ns * S);
            if (kSeq && (starts >> t & 1u)) {
                init_state(l, __shfl_sync(0xffffffffu, id, t));
#pragma unroll
                for (int j = 0; j < S2; ++j) p[j] = both(0.f);
            }
            acc[t] = both(0.f);
#pragma unroll
            for (int j = 0; j < S2; ++j) {
                const float2 x = __fmul2_rn(lo2(dd), A2[j]);
                const float2 av = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                const float2 Bj = j % 2 ? hi2(Bt[j / 2]) : lo2(Bt[j / 2]), Cj = j % 2 ? hi2(Ct[j / 2]) : lo2(Ct[j / 2]);
                l[j] = __ffma2_rn(av, l[j], __fmul2_rn(hi2(dd), Bj));
                p[j] = __fmul2_rn(p[j], av);
                acc[t] = __ffma2_rn(Cj, l[j], acc[t]);
                cp[t][j] = __fmul2_rn(Cj, p[j]);
            }
        }
        // ---- chain the slices: the state before this one, and before the next tile ----
        float4* ep = sm_ep + (buf * K * 2) * S4 * 32 + lane;
#pragma unroll
        for (int j = 0; j < S4; ++j) {
            ep[((w * 2 + 0) * S4 + j) * 32] = make_float4(l[2 * j].x, l[2 * j].y, l[2 * j + 1].x, l[2 * j + 1].y);
            ep[((w * 2 + 1) * S4 + j) * 32] = make_float4(p[2 * j].x, p[2 * j].y, p[2 * j + 1].x, p[2 * j + 1].y);
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
            for (int j = 0; j < S4; ++j) {
                const float4 e = ep[((k * 2 + 0) * S4 + j) * 32], q = ep[((k * 2 + 1) * S4 + j) * 32];
                h0[2 * j] = __ffma2_rn(lo2(q), h0[2 * j], lo2(e));
                h0[2 * j + 1] = __ffma2_rn(hi2(q), h0[2 * j + 1], hi2(e));
            }
        }
        // ---- the read-out of the state before the slice ----
        float out[kSlice];
#pragma unroll
        for (int t = 0; t < kSlice; ++t) {
#pragma unroll
            for (int j = 0; j < S2; ++j) acc[t] = __ffma2_rn(cp[t][j], h[j], acc[t]);
            out[t] = acc[t].x + acc[t].y;
        }
        // ---- final states: of sequences that end inside the slice, and of the row's last ----
        if (a.final_states) {
            const bool last = tw < a.seqlen && tw + kSlice >= a.seqlen;
            if (last) {
#pragma unroll
                for (int j = 0; j < S2; ++j) l[j] = __ffma2_rn(p[j], h[j], l[j]);
                const int s = kSeq ? __shfl_sync(0xffffffffu, id, a.seqlen - 1 - tw) : 0;
                write_state(l, s);
                keep(s + 1, a.nseq);
            }
            if (kSeq && starts) {  // rare: walk the slice again from its true state
                for (int t = 0; t < kSlice; ++t) {
                    if (starts >> t & 1u) {
                        const int s = __shfl_sync(0xffffffffu, id, t), before = __shfl_sync(0xffffffffu, id_before, t);
                        if (before >= 0) write_state(h, before);
                        keep(before + 1, s);
                        init_state(h, s);
                    }
                    const float4 dd = *reinterpret_cast<const float4*>(sm_pair + ch * PROW + 4 * t);
#pragma unroll
                    for (int j = 0; j < S2; ++j) {
                        const float2 Bj = *reinterpret_cast<const float2*>(sm_bc + t * 2 * NP + ns * S + 2 * j);
                        const float2 x = __fmul2_rn(lo2(dd), A2[j]);
                        h[j] = __ffma2_rn(make_float2(exp2_fast(x.x), exp2_fast(x.y)), h[j], __fmul2_rn(hi2(dd), Bj));
                    }
                }
            }
        }
        // ---- sum over the channel's lanes; each ends with the tokens it owns ----
#pragma unroll
        for (int m = LN / 2, n = kSlice; m >= 1; m /= 2) {
            if (n > 1) {  // keep the half of the tokens that the lane's side owns
                n /= 2;
                const bool up = ns & m;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float give = up ? out[i] : out[i + n], stay = up ? out[i + n] : out[i];
                    out[i] = stay + __shfl_xor_sync(0xffffffffu, give, m * CPW);
                }
            } else {
                out[0] += __shfl_xor_sync(0xffffffffu, out[0], m * CPW);
            }
        }
        if (owner) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const int t = tw + own + i;
                if (t < a.seqlen) y[(int64_t)t * a.channels] = from_f32<T>((out[i] + skip[i]) * gate[i]);
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

template <typename T, int S, int LN, int K, bool kSeq, bool kCopy>
cudaError_t start_scan(const SelectiveArgs& a, cudaStream_t st) {
    using Sh = ScanShape<T, S, LN, K>;
    constexpr int smem = Sh::smem(kCopy);
    static_assert(smem <= 227 * 1024, "fits one SM");
    const int per = a.channels / a.ngroups, units = (per + Sh::CPW - 1) / Sh::CPW;
    const unsigned grid = (unsigned)((int64_t)a.batch * a.ngroups * units);
    const auto kernel = selective_scan_kernel<T, S, LN, K, kSeq, kCopy>;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, 32 * K, smem, st>>>(a, units);
    return cudaGetLastError();
}

template <typename T, int S, int LN, int K>
cudaError_t run_scan(const SelectiveArgs& a, cudaStream_t st) {
    using Sh = ScanShape<T, S, LN, K>;
    if constexpr (Sh::kCanCopy) {
        VectorRule tok(sizeof(T)), bc(sizeof(T));
        tok.address(a.u).address(a.dt).elements(a.us_b).elements(a.us_t).elements(a.ds_b).elements(a.ds_t);
        if (a.z) tok.address(a.z).elements(a.zs_b).elements(a.zs_t);
        tok.elements(a.channels / a.ngroups);
        bc.address(a.B).address(a.C).elements(a.bs_b).elements(a.bs_t).elements(a.cs_b).elements(a.cs_t);
        bc.elements(a.dstate);
        if (tok.multiple_of(Sh::TB) && bc.multiple_of(16))
            return a.seq_idx ? start_scan<T, S, LN, K, true, true>(a, st) : start_scan<T, S, LN, K, false, true>(a, st);
    }
    return a.seq_idx ? start_scan<T, S, LN, K, true, false>(a, st) : start_scan<T, S, LN, K, false, false>(a, st);
}

template <typename T, int S, int LN>
cudaError_t scan_by_slices(const SelectiveArgs& a, cudaStream_t st) {
    const int64_t units = (int64_t)a.batch * a.ngroups * ((a.channels / a.ngroups + 32 / LN - 1) / (32 / LN));
    // 16 warps per CTA where the CTAs do not fill the GPU's SMs twice, else 4
    if constexpr (S * LN <= 64) {
        if (units < 2 * 148 && a.seqlen > 4 * kSlice) return run_scan<T, S, LN, 16>(a, st);
    }
    return run_scan<T, S, LN, 4>(a, st);
}

template <typename T>
cudaError_t scan_by_states(const SelectiveArgs& a, cudaStream_t st) {
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
