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
// Prompts: a warp owns a few channels of one row, LN lanes per CH channels with
// S states of each in registers. The exponentials do not depend on the state, so
// a CTA's K warps take consecutive slices of L tokens in turn: each forms
// a = exp(delta A) and v = delta u B of its slice in registers, waits for the
// state that the warp before it leaves in shared memory (a named barrier between
// the two), runs the L dependent multiply-adds, hands the state on, and reads
// out. The chain is short beside the rest, so the warps work side by side
// although the recurrence is sequential. Every exponential is formed once.
//
// Measured at b 1 x T 4096 x 5120 channels, N 16, bf16: 207 us (b 4: 711).
// Per slice of a warp (8 channels x 8 tokens x 16 states) it issues 355 instructions,
// 40 of them special-function, and 117 shared-memory wavefronts: 89, 80 and 117
// cycles of an SM, against about 155 that a slice takes in steady state: shared memory
// is the busiest, and 16 warps per SM (limited by the 64 registers that a and v
// take) do not cover its latency. The special functions alone would take 90 us,
// those of the states 72. The 640 units of 8 channels are 5 on 48 SMs and 4 on the
// others: the rules below ask whether the SMs are filled once, not how full the last
// turn is. Packed rows issue 427 instructions and 125 wavefronts per slice: 278 us
// with 16 sequences. Stack for spilled registers at 16 states, copied rows: none in
// bf16, 40 bytes in fp32 (packed: 16 and 8); the most without copies at 256 states,
// 216 bytes. Ways that measured slower: one slice per warp from zero, its end state
// and decay exchanged by all warps (293 us: every element costs two more
// multiplies); two channels per lane and slices of 4 at N 16 (245); 4 to 7, 9 or 10
// warps per CTA (231 to 320).

#include <atomic>
#include <cfloat>
#include <type_traits>

#include "ssd_block.cuh"

namespace ssd {

namespace {

// exp(x) for x <= 0 with its relative accuracy: the rounding of p = x log2 e alone
// would be an error of |x| 2^-24 in 2^p, 64 half steps at x = -85. fp32: the full
// exponential (7 fp32 sequences in 5003 x 1536: 2.0e-7 off 64 bits, 3.8e-7
// with the other form, 125 us against 124). bf16, whose inputs carry more error than
// that: the rounding put back to first order, 2^p (1 + x - p ln 2) with ln 2 in two
// parts (bf16 prompt of the header: 207 us, 211 with expf).
template <typename T>
__device__ __forceinline__ float exp_for(float x) {
    if constexpr (sizeof(T) == 4) return expf(x);
    x = fmaxf(x, -128.f);  // 2^p is 0 there
    const float p = x * kLog2e, d = fmaf(p, 1.9046543e-9f, fmaf(p, -0.69314718f, x)), e = exp2_approx(p);
    return fmaf(e, d, e);
}

// softplus(z) = max(z, 0) + log(1 + e), e = exp(-|z|) in [0, 1]. The logarithm
// as 2 atanh(r), r = e / (2 + e) <= 1/3, by its power series: the first term left
// out is r^17 / 17 < 1.4e-9 of r, and small e keep their relative accuracy, which
// log(1 + e) taken directly would lose. NaN comes through the last term.
template <typename T>
__device__ __forceinline__ float softplus(float z) {
    const float e = exp_for<T>(-fabsf(z));
    const float r = e * rcp_approx(2.f + e), q = r * r;
    float s = 1.f / 15.f;
    s = fmaf(s, q, 1.f / 13.f);
    s = fmaf(s, q, 1.f / 11.f);
    s = fmaf(s, q, 1.f / 9.f);
    s = fmaf(s, q, 1.f / 7.f);
    s = fmaf(s, q, 1.f / 5.f);
    s = fmaf(s, q, 1.f / 3.f);
    s = fmaf(s, q, 1.f);
    return fmaf(2.f * r, s, z < 0.f ? 0.f : z);
}

// A rate of -infinity (a state without memory) as the lowest finite one: its decay is 0 at every step size
// that is not 0 all the same, and 1, not NaN, at the tokens behind a row's end, whose step size is 0.
__device__ __forceinline__ float finite_rate(float A2) { return A2 < -FLT_MAX ? -FLT_MAX : A2; }

constexpr int kStages = 3;  // slices of raw inputs in shared memory: two in flight behind the current one

// CH channels and S states of each per lane, LN lanes per channel, slices of L
// tokens, K warps.
template <typename T, int CH_, int S_, int LN_, int L_, int K_>
struct ScanShape {
    static constexpr int CH = CH_, S = S_, LN = LN_, L = L_, K = K_;
    static constexpr int COLS = 32 / LN;                       // lanes side by side in channels
    static constexpr int CPW = COLS * CH;                      // channels per warp
    static constexpr int NP = S * LN;                          // states, padded
    static constexpr int E = (int)sizeof(T);
    static constexpr int OUTS = CH * L;                        // (token, channel) sums a lane takes part in
    static constexpr int OWN = LN < OUTS ? OUTS / LN : 1;      // of those, the ones it ends up with
    static constexpr int SHARE = LN > OUTS ? LN / OUTS : 1;    // lanes that end up with the same one
    static constexpr int ROW = CPW * E;                        // bytes of a token's channels
    static constexpr int TB = ROW < 16 ? ROW : 16;             // bytes per copy of u, dt, z
    static constexpr int TR = (3 * L * ROW / TB + 31) / 32;    // such copies per lane and slice
    static constexpr int BV = 16 / E;                          // B, C elements per copy
    static constexpr int BN = L * 2 * NP / BV;                 // such copies per slice
    static constexpr int BR = (BN + 31) / 32;                  // and per lane
    static constexpr bool kCanCopy = TB >= 4 && NP >= BV && BR <= 8;
    static constexpr int PAIR = L * CPW * 2;                   // floats: (delta, delta u) per token and channel
    static constexpr int BC = L * 2 * NP;                      // floats: B and C of the slice
    static constexpr int NB = BC / 32;                         // of those, a lane's share
    static constexpr int STATE = CH * S * 32;                  // floats: a state handed on
    static constexpr int TOKENS = (3 * L * ROW + 15) / 16 * 16; // bytes of u, dt, z in a raw stage
    static constexpr int RAW = TOKENS + BC * E;                // bytes of a raw stage
    static_assert(PAIR % 4 == 0 && BC % 4 == 0 && STATE % 4 == 0 && BC * E % 16 == 0, "16-byte parts");
    static constexpr int smem(bool copies) { return K * (PAIR + BC + STATE) * 4 + (copies ? K * kStages * RAW : 0); }
};

// Lane = state slice * COLS + column; a lane holds states [ns * S, ns * S + S) of
// the CH channels of its column. Of the OUTS sums over states that the LN lanes of
// a column form together (token-major, its CH channels within a token) a lane
// ends up with OWN; those (token, channel) are also the ones whose inputs it
// prepares. kCopy: all rows allow the asynchronous copies of ScanShape.
template <typename T, typename Sh, int kMinCtas, bool kSeq, bool kCopy>
__global__ void __launch_bounds__(32 * Sh::K, kMinCtas) selective_scan_kernel(const SelectiveArgs a,
                                                                              int units_per_group) {
    constexpr int CH = Sh::CH, S = Sh::S, L = Sh::L, K = Sh::K, COLS = Sh::COLS, CPW = Sh::CPW, NP = Sh::NP;
    constexpr int S2 = S / 2, OWN = Sh::OWN;
    // bf16 B and C of many states are read where the copies put them: every lane of a column converts its own,
    // but shared memory moves half the bytes and no staged fp32 copy is written (N 64: 199 -> 173 us, N 128: 256 ->
    // 188 us per 5120 channels and 1024, 512 tokens; N 16 the other way, 209 -> 224 us for 4096 tokens).
    constexpr bool kRawBC = kCopy && sizeof(T) == 2 && NP >= 32;
    extern __shared__ float4 smem4[];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int col = lane % COLS, ns = lane / COLS, N = a.dstate;
    constexpr int kWarpBytes = (Sh::PAIR + Sh::BC + Sh::STATE) * 4 + (kCopy ? kStages * Sh::RAW : 0);
    char* mine4 = reinterpret_cast<char*>(smem4) + w * kWarpBytes;  // the warp's part
    float* sm_pair = reinterpret_cast<float*>(mine4);
    float* sm_bc = sm_pair + Sh::PAIR;
    float4* sm_state = reinterpret_cast<float4*>(sm_bc + Sh::BC) + lane;  // [CH * S / 4][32]
    float4* sm_next = reinterpret_cast<float4*>(
        reinterpret_cast<char*>(sm_state) + (w == K - 1 ? -(K - 1) * kWarpBytes : kWarpBytes));
    char* sm_raw = reinterpret_cast<char*>(sm_bc + Sh::BC + Sh::STATE);

    const int per = a.channels / a.ngroups;
    const int unit = blockIdx.x % units_per_group, bg = blockIdx.x / units_per_group;
    const int g = bg % a.ngroups, b = bg / a.ngroups;
    const int cg0 = unit * CPW;  // the warp's first channel within the group
    const int64_t row0 = (int64_t)b * a.seqlen;
    const T* u = static_cast<const T*>(a.u) + b * a.us_b + g * per;
    const T* dt = static_cast<const T*>(a.dt) + b * a.ds_b + g * per;
    const T* z = static_cast<const T*>(a.z) + b * a.zs_b + g * per;
    const T* B = static_cast<const T*>(a.B) + b * a.bs_b + g * N;
    const T* C = static_cast<const T*>(a.C) + b * a.cs_b + g * N;

    // the lane's own (token, channel) pairs: tok(i), and cg(i) within the group
    const int first = ns * Sh::OUTS / Sh::LN;
    const auto tok = [&](int i) { return (first + i) / CH; };
    const auto cl = [&](int i) { return col * CH + (first + i) % CH; };  // within the warp's channels
    float bias[OWN], D[OWN];
    bool mine[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int cg = min(cg0 + cl(i), per - 1), c = g * per + cg;
        mine[i] = cg0 + cl(i) < per && ns % Sh::SHARE == 0;
        bias[i] = a.dt_bias ? a.dt_bias[c] : 0.f;
        D[i] = a.D ? a.D[c] : 0.f;
    }
    // the lane's states: channel m, states ns * S + 2 j, + 1
    float2 A2[CH][S2];
#pragma unroll
    for (int m = 0; m < CH; ++m)
#pragma unroll
        for (int j = 0; j < S2; ++j) {
            const int n = ns * S + 2 * j;
            const int64_t r = (int64_t)(g * per + min(cg0 + col * CH + m, per - 1)) * N;
            A2[m][j].x = n < N ? finite_rate(a.A[r + n] * kLog2e) : 0.f;
            A2[m][j].y = n + 1 < N ? finite_rate(a.A[r + n + 1] * kLog2e) : 0.f;
        }
    using State = float2[CH][S2];
    const auto init_state = [&](State& h, int s) {
#pragma unroll
        for (int m = 0; m < CH; ++m) {
            const int cg = min(cg0 + col * CH + m, per - 1);
#pragma unroll
            for (int j = 0; j < S2; ++j) {
                const int n = ns * S + 2 * j;
                const int64_t o = (((int64_t)b * a.nseq + s) * N + n) * a.channels + g * per + cg;
                h[m][j].x = a.init && n < N ? a.init[o] : 0.f;
                h[m][j].y = a.init && n + 1 < N ? a.init[o + a.channels] : 0.f;
            }
        }
    };
    const auto write_state = [&](const State& h, int s) {
#pragma unroll
        for (int m = 0; m < CH; ++m) {
            const int cg = cg0 + col * CH + m;
#pragma unroll
            for (int j = 0; j < S2; ++j) {
                const int n = ns * S + 2 * j;
                const int64_t o = (((int64_t)b * a.nseq + s) * N + n) * a.channels + g * per + cg;
                if (cg < per && n < N) a.final_states[o] = h[m][j].x;
                if (cg < per && n + 1 < N) a.final_states[o + a.channels] = h[m][j].y;
            }
        }
    };
    // ids that do not occur keep their initial state
    const auto keep = [&](int lo, int hi) {
        for (int s = lo; s < hi; ++s) {
            State h;
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
    int bbytes[kCopy ? Sh::BR : 1];
    T ru[kCopy ? 1 : OWN], rd[kCopy ? 1 : OWN], rz[kCopy ? 1 : OWN];
    T rbc[kCopy ? 1 : Sh::NB];
    // element lane + 32 i of the slice's B and C
    const auto bc_element = [&](int tw, int i, auto full) {
        const int v = lane + 32 * i, r = v % (2 * NP), n = r % NP, t = tw + v / (2 * NP);
        T e = from_f32<T>(0.f);
        if (n < N && (full || t < a.seqlen)) e = r < NP ? B[t * a.bs_t + n] : C[t * a.cs_t + n];
        return e;
    };
    if constexpr (kCopy) {
        constexpr int PT = Sh::ROW / Sh::TB, PB = 2 * NP / Sh::BV;
#pragma unroll
        for (int i = 0; i < Sh::TR; ++i) {  // copy v: array (u, dt, z), token, part of the token's channels
            const int v = lane + 32 * i, arr = v / (L * PT), t = v / PT % L, part = v % PT;
            // per is a multiple of a part, so a part lies in the group or behind it. Those behind it (in the last
            // unit) copy no bytes, but their source has to be as aligned as any: the group's first channel.
            const int cg = cg0 + part * (Sh::TB / Sh::E);
            const int64_t step = arr == 0 ? a.us_t : arr == 1 ? a.ds_t : a.zs_t;
            tstep[i] = step * (K * L);
            tsrc[i] = (arr == 0 ? u : arr == 1 ? dt : z) + (w * L + t) * step + (cg < per ? cg : 0);
            tbytes[i] = cg < per ? Sh::TB : 0;
            if (arr == 2 && !a.z) tbytes[i] = 0, tsrc[i] = u, tstep[i] = 0;  // no gate: zeros
            if (arr > 2) tbytes[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < Sh::BR; ++i) {  // copy v: token, B or C, states
            const int v = lane + 32 * i, t = v / PB, r = v % PB, n = r % (PB / 2) * Sh::BV;
            const int64_t step = r < PB / 2 ? a.bs_t : a.cs_t;
            bstep[i] = step * (K * L);
            bbytes[i] = n < N ? 16 : 0;
            bsrc[i] = (r < PB / 2 ? B : C) + (w * L + t) * step + (n < N ? n : 0);
        }
    }
    // the slice that starts at token tw; full: it lies inside the row
    const auto fetch = [&](int tw, int stage, auto full) {
        if constexpr (kCopy) {
            char* dst = sm_raw + stage + lane * Sh::TB;
            char* dst_bc = sm_raw + stage + Sh::TOKENS + lane * 16;
#pragma unroll
            for (int i = 0; i < Sh::TR; ++i) {
                const int t = (lane + 32 * i) / (Sh::ROW / Sh::TB) % L;
                if (tbytes[i] >= 0) {
                    const bool in = full || tw + t < a.seqlen;
                    copy_async<Sh::TB>(dst + i * 32 * Sh::TB, in ? tsrc[i] : u, in ? tbytes[i] : 0);
                    tsrc[i] += tstep[i];
                }
            }
#pragma unroll
            for (int i = 0; i < Sh::BR; ++i) {
                const int t = (lane + 32 * i) / (2 * NP / Sh::BV);
                if (Sh::BN % 32 == 0 || lane + 32 * i < Sh::BN) {
                    const bool in = full || tw + t < a.seqlen;
                    copy_async<16>(dst_bc + i * 512, in ? bsrc[i] : B, in ? bbytes[i] : 0);
                    bsrc[i] += bstep[i];
                }
            }
            copy_commit();
        } else {
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                const int t = tw + tok(i), cg = min(cg0 + cl(i), per - 1);
                ru[i] = rd[i] = rz[i] = from_f32<T>(0.f);
                if (full || t < a.seqlen) {
                    ru[i] = u[t * a.us_t + cg];
                    rd[i] = dt[t * a.ds_t + cg];
                    if (a.z) rz[i] = z[t * a.zs_t + cg];
                }
            }
#pragma unroll
            for (int i = 0; i < Sh::NB; ++i) rbc[i] = bc_element(tw, i, full);
        }
    };

    // hand a state on to the next warp
    const int next = w == K - 1 ? 0 : w + 1;
    const auto put_state = [&](const State& h) {
#pragma unroll
        for (int i = 0; i < CH * S / 4; ++i) {
            const float2 lo = h[4 * i / S][4 * i % S / 2], hi = h[4 * i / S][4 * i % S / 2 + 1];
            sm_next[i * 32] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
        __syncwarp();  // the warp arrives as one
        asm volatile("bar.arrive %0, 64;" ::"r"(next) : "memory");
    };
    fetch(w * L, 0, std::false_type());
    if (kCopy) fetch((K + w) * L, Sh::RAW, std::false_type());
    int stage = 0;  // byte offset of the current raw stage
    T* y = static_cast<T*>(a.y) + (row0 + w * L + tok(0)) * a.channels + g * per + cg0 + cl(0);
    if (w == K - 1) {  // the state before the row, for warp 0's first slice
        State h;
        init_state(h, 0);
        put_state(h);
    }
    // What a slice is prepared to, carried from one turn of the loop to the next: the compiler then cannot
    // move the exponentials behind the wait for the state, where they would delay every warp of the CTA.
    float2 av[L][CH][S2], hv[L][CH][S2];  // a and v
    float skip[OWN], gate[OWN];
    [[maybe_unused]] const char* bc_raw = sm_raw;  // the slice's B and C as copied
    // the lane's states of token t's B (which = 0) or C (1)
    const auto load_bc = [&](int t, int which, float (&f)[S]) {
        const int i = t * 2 * NP + which * NP + ns * S;
        if constexpr (kRawBC)
            unpack(*reinterpret_cast<const Pack<T, S>*>(bc_raw + i * Sh::E), f);
        else
            unpack(*reinterpret_cast<const Pack<float, S>*>(sm_bc + i), f);
    };
    unsigned starts = 0u;  // sequences that start in the slice: bit t for token t
    int id = 0, id_before = 0;
    // The ids around the next slice: lane i <= L has that of its token i - 1 (as loaded: a use would wait).
    int next_id = 0, id_token = w * L - 1 + min(lane, L);
    const auto load_ids = [&]() {
        if (id_token >= 0 && id_token < a.seqlen) next_id = a.seq_idx[row0 + id_token];
        id_token += K * L;
    };
    // The slice that starts at token tw. full: it, and the slice fetched meanwhile, lie inside the row, and
    // it is not the row's last one.
    const auto prepare = [&](int tw, auto full) {
        const bool past_end = !full && tw + L > a.seqlen;
        // ---- this slice's (delta, delta u), B and C, in fp32 ----
        if (kCopy) copy_wait<1>();
        __syncwarp();
        [[maybe_unused]] const char* raw = sm_raw + stage;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            float uf, d, zf;
            if constexpr (kCopy) {
                const T* e = reinterpret_cast<const T*>(raw) + tok(i) * CPW + cl(i);
                uf = to_f32(e[0]), d = to_f32(e[L * CPW]), zf = to_f32(e[2 * L * CPW]);
            } else {
                uf = to_f32(ru[i]), d = to_f32(rd[i]), zf = to_f32(rz[i]);
            }
            d += bias[i];
            if (a.softplus) d = softplus<T>(d);
            if (past_end && tw + tok(i) >= a.seqlen) d = 0.f;  // a = 1 and no input
            skip[i] = D[i] * uf;
            gate[i] = a.z ? silu_for<T>(zf) : 1.f;
            *reinterpret_cast<float2*>(sm_pair + (tok(i) * CPW + cl(i)) * 2) = make_float2(d, d * uf);
        }
        bc_raw = raw + Sh::TOKENS;
        if constexpr (kCopy) {
#pragma unroll
            for (int i = 0; i < (kRawBC ? 0 : Sh::BR); ++i) {
                const int v = lane + 32 * i;
                if (Sh::BN % 32 == 0 || v < Sh::BN) {
                    const Pack<T, Sh::BV> e =
                        *reinterpret_cast<const Pack<T, Sh::BV>*>(raw + Sh::TOKENS + v * 16);
#pragma unroll
                    for (int k = 0; k < Sh::BV; k += 4)
                        *reinterpret_cast<float4*>(sm_bc + v * Sh::BV + k) = make_float4(
                            to_f32(e.v[k]), to_f32(e.v[k + 1]), to_f32(e.v[k + 2]), to_f32(e.v[k + 3]));
                }
            }
            fetch(tw + 2 * K * L, stage == 0 ? 2 * Sh::RAW : stage - Sh::RAW, full);
            stage = stage == (kStages - 1) * Sh::RAW ? 0 : stage + Sh::RAW;
        } else {
#pragma unroll
            for (int i = 0; i < Sh::NB; ++i) sm_bc[lane + 32 * i] = to_f32(rbc[i]);
            fetch(tw + K * L, 0, full);
        }
        if (kSeq) {  // lane i looks at token tw + i, and at the one before it
            id_before = min(max(next_id, 0), a.nseq - 1);
            id = __shfl_down_sync(0xffffffffu, id_before, 1);
            const bool first = tw + lane == 0 || id != id_before;
            starts = __ballot_sync(0xffffffffu, first && lane < L && (full || tw + lane < a.seqlen));
            load_ids();
        }
        __syncwarp();
        // ---- a and v of the slice ----
#pragma unroll
        for (int t = 0; t < L; ++t) {
            const Pack<float, 2 * CH> d = *reinterpret_cast<const Pack<float, 2 * CH>*>(
                sm_pair + (t * CPW + col * CH) * 2);  // delta, delta u of each channel
            float Bt[S];
            load_bc(t, 0, Bt);
#pragma unroll
            for (int j = 0; j < S2; ++j) {
#pragma unroll
                for (int m = 0; m < CH; ++m) {
                    av[t][m][j] = make_float2(exp2_approx(d.v[2 * m] * A2[m][j].x), exp2_approx(d.v[2 * m] * A2[m][j].y));
                    hv[t][m][j] = make_float2(d.v[2 * m + 1] * Bt[2 * j], d.v[2 * m + 1] * Bt[2 * j + 1]);
                }
            }
        }
    };
    // The recurrence through the prepared slice, and its read-out.
    const auto finish = [&](int tw, auto full) {
        const bool past_end = !full && tw + L > a.seqlen;
        // ---- the recurrence: the state from the slice before, through this one, to the next ----
        State h;
        asm volatile("bar.sync %0, 64;" ::"r"(w) : "memory");  // with the arrival of the warp before
#pragma unroll
        for (int i = 0; i < CH * S / 4; ++i) {
            const float4 q = sm_state[i * 32];
            h[4 * i / S][4 * i % S / 2] = make_float2(q.x, q.y);
            h[4 * i / S][4 * i % S / 2 + 1] = make_float2(q.z, q.w);
        }
        const auto advance = [&](int t) {
#pragma unroll
            for (int m = 0; m < CH; ++m)
#pragma unroll
                for (int j = 0; j < S2; ++j) h[m][j] = hv[t][m][j] = __ffma2_rn(av[t][m][j], h[m][j], hv[t][m][j]);
        };
        if (!kSeq || starts == 0u) {  // a branch per token here would delay every warp of the CTA
#pragma unroll
            for (int t = 0; t < L; ++t) advance(t);
        } else {
#pragma unroll
            for (int t = 0; t < L; ++t) {
                if (starts >> t & 1u) {
                    const int s = __shfl_sync(0xffffffffu, id, t), before = __shfl_sync(0xffffffffu, id_before, t);
                    if (a.final_states) {
                        if (tw + t > 0) write_state(h, before);
                        keep(tw + t > 0 ? before + 1 : 0, s);
                    }
                    init_state(h, s);
                }
                advance(t);
            }
        }
        if (full || w < K - 1 || tw + L < a.seqlen) put_state(h);  // the row's last tile ends the chain
        if (!full && a.final_states && tw < a.seqlen && tw + L >= a.seqlen) {  // this slice has the row's last token
            const int s = kSeq ? __shfl_sync(0xffffffffu, id, a.seqlen - 1 - tw) : 0;
            write_state(h, s);
            keep(s + 1, a.nseq);
        }
        // ---- read-out, summed over a column's lanes; each ends with the sums it owns ----
        float out[Sh::OUTS];
#pragma unroll
        for (int t = 0; t < L; ++t) {
            float Ct[S];
            load_bc(t, 1, Ct);
            float2 acc[CH];
#pragma unroll
            for (int j = 0; j < S2; ++j) {
                const float2 Cj = make_float2(Ct[2 * j], Ct[2 * j + 1]);
#pragma unroll
                for (int m = 0; m < CH; ++m)
                    acc[m] = j == 0 ? __fmul2_rn(Cj, hv[t][m][j]) : __ffma2_rn(Cj, hv[t][m][j], acc[m]);
            }
#pragma unroll
            for (int m = 0; m < CH; ++m) out[t * CH + m] = acc[m].x + acc[m].y;
        }
#pragma unroll
        for (int k = Sh::LN / 2, n = Sh::OUTS; k >= 1; k /= 2) {
            if (n > 1) {  // keep the half of the sums that the lane's side owns
                n /= 2;
                const bool up = ns & k;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float give = up ? out[i] : out[i + n], stay = up ? out[i + n] : out[i];
                    out[i] = stay + __shfl_xor_sync(0xffffffffu, give, k * COLS);
                }
            } else {
                out[0] += __shfl_xor_sync(0xffffffffu, out[0], k * COLS);
            }
        }
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            if (!mine[i] || (past_end && tw + tok(i) >= a.seqlen)) continue;
            y[(int64_t)(tok(i) - tok(0)) * a.channels + (cl(i) - cl(0))] = from_f32<T>((out[i] + skip[i]) * gate[i]);
        }
        y += (int64_t)(K * L) * a.channels;
    };
    const int tiles = (a.seqlen + K * L - 1) / (K * L);
    const int first_token = w * L, step = K * L;
    // whole: the tiles whose fetches, two tiles ahead at most, lie inside the row
    const int whole = max(0, min(a.seqlen / step - 2, tiles - 1));
    if (kSeq) load_ids();
    prepare(first_token, std::false_type());
    int tile = 0;
    for (; tile + 1 < whole; ++tile) {
        finish(first_token + tile * step, std::true_type());
        prepare(first_token + (tile + 1) * step, std::true_type());
    }
    for (; tile < tiles; ++tile) {
        finish(first_token + tile * step, std::false_type());
        if (tile + 1 < tiles) prepare(first_token + (tile + 1) * step, std::false_type());
    }
}

constexpr int kStepThreads = 128;
constexpr int kStepStates = 16;  // states of a thread in flight per row

// One token: a thread takes one channel of a batch row, kStepStates states at a
// time; a CTA's channels lie in one group, whose B and C rows it keeps in shared
// memory. 64 rows x 5120 channels x 16 states take 12.4 us in a graph of steps on
// different states (3.6 TB/s; the bytes' time is 7 us), 256 rows 42 (4.2 TB/s), and 3 rows x
// 1536 channels 2.3; a call from Python takes 15 to 16 us whatever the size up to 64 rows. Bound by the
// latency of the state's loads: 2560 CTAs at 5 per SM are 3.5 turns, 27 % of the warps are
// resident and the issue slots are used at 39 %. Two rows per thread took longer (29 us cold against 25).
// kVec: A's rows allow 16-byte loads; kWhole: N is a multiple of kStepStates.
// Offsets within a row's state (at most 2^20 x 256 floats, 1 GB) are 32 bits from a
// CTA-wide base: with 64-bit addresses per access their arithmetic was most of
// the kernel's instructions.
template <typename T, bool kVec, bool kWhole>
__global__ void __launch_bounds__(kStepThreads, 5) selective_step_kernel(const SelectiveArgs a, int blocks_per_group) {
    __shared__ float4 sm_b[kStepStates / 4], sm_c[kStepStates / 4];
    const int N = a.dstate, per = a.channels / a.ngroups;
    const int bg = blockIdx.x / blocks_per_group, b = bg / a.ngroups, g = bg % a.ngroups;
    const int cg = (blockIdx.x % blocks_per_group) * kStepThreads + threadIdx.x;
    const bool live = cg < per;
    const int c = g * per + min(cg, per - 1);
    const T* B = static_cast<const T*>(a.B) + b * a.bs_b + g * N;
    const T* C = static_cast<const T*>(a.C) + b * a.cs_b + g * N;
    char* hb = reinterpret_cast<char*>(a.final_states + (int64_t)b * N * a.channels);
    const uint32_t step = 4u * (uint32_t)a.channels;
    uint32_t off = 4u * (uint32_t)c;
    const auto in = [&](int n) { return kWhole || n < N; };
    float d = 0.f, du = 0.f, y = 0.f, zf = 0.f;
    for (int n0 = 0; n0 < N; n0 += kStepStates) {
        float hv[kStepStates], A2[kStepStates];
#pragma unroll
        for (int j = 0; j < kStepStates; ++j)
            if (in(n0 + j)) hv[j] = __ldcs(reinterpret_cast<const float*>(hb + (off + j * step)));
        const char* Ab = reinterpret_cast<const char*>(a.A);
        const uint32_t aoff = 4u * ((uint32_t)c * (uint32_t)N + (uint32_t)n0);
#pragma unroll
        for (int j = 0; j < kStepStates; j += kVec ? 4 : 1) {
            using Q = Pack<float, kVec ? 4 : 1>;
            if (in(n0 + j)) *reinterpret_cast<Q*>(A2 + j) = *reinterpret_cast<const Q*>(Ab + (aoff + 4u * j));
        }
        if (n0 == 0) {
            const float uf = to_f32(static_cast<const T*>(a.u)[b * a.us_b + c]);
            d = to_f32(static_cast<const T*>(a.dt)[b * a.ds_b + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
            if (a.z) zf = to_f32(static_cast<const T*>(a.z)[b * a.zs_b + c]);
            y = a.D ? a.D[c] * uf : 0.f;
            if (a.softplus) d = softplus<T>(d);
            du = d * uf;
            d *= kLog2e;
        } else {
            __syncthreads();  // the states before are done with B and C
        }
        if (threadIdx.x < kStepStates) {
            const int n = n0 + threadIdx.x;
            reinterpret_cast<float*>(sm_b)[threadIdx.x] = n < N ? to_f32(B[n]) : 0.f;
            reinterpret_cast<float*>(sm_c)[threadIdx.x] = n < N ? to_f32(C[n]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kStepStates / 4; ++q) {
            const float4 Bq = sm_b[q], Cq = sm_c[q];
            const float Bv[4] = {Bq.x, Bq.y, Bq.z, Bq.w}, Cv[4] = {Cq.x, Cq.y, Cq.z, Cq.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = 4 * q + k;
                if (in(n0 + j)) {
                    const float v = fmaf(exp2_approx(d * A2[j]), hv[j], du * Bv[k]);
                    if (live) __stcs(reinterpret_cast<float*>(hb + (off + j * step)), v);
                    y = fmaf(Cv[k], v, y);
                }
            }
        }
        off += kStepStates * step;
    }
    if (live)
        static_cast<T*>(a.y)[(int64_t)b * a.channels + c] = from_f32<T>(a.z ? y * silu_for<T>(zf) : y);
}

template <typename T>
cudaError_t run_step(const SelectiveArgs& a, cudaStream_t st) {
    const int per = a.channels / a.ngroups, bpg = (per + kStepThreads - 1) / kStepThreads;
    const bool vec = VectorRule(4).address(a.A).elements(a.dstate).multiple_of(16);
    const unsigned grid = (unsigned)((int64_t)a.batch * a.ngroups * bpg);
    const auto kernel = a.dstate % kStepStates == 0 ? (vec ? selective_step_kernel<T, true, true> : selective_step_kernel<T, false, true>)
                                                    : (vec ? selective_step_kernel<T, true, false> : selective_step_kernel<T, false, false>);
    kernel<<<grid, kStepThreads, 0, st>>>(a, bpg);
    return cudaGetLastError();
}

template <typename T, typename Sh, int kMinCtas, bool kSeq, bool kCopy>
cudaError_t start_scan(const SelectiveArgs& a, cudaStream_t st) {
    constexpr int smem = Sh::smem(kCopy);
    static_assert(smem <= 227 * 1024, "fits one SM");
    const int per = a.channels / a.ngroups, units = (per + Sh::CPW - 1) / Sh::CPW;
    const unsigned grid = (unsigned)((int64_t)a.batch * a.ngroups * units);
    const auto kernel = selective_scan_kernel<T, Sh, kMinCtas, kSeq, kCopy>;
    if (smem > 48 * 1024) {  // once per device (a race only repeats it)
        static std::atomic<uint64_t> set{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (!bit || !(set.load(std::memory_order_acquire) & bit)) {
            e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            set.fetch_or(bit, std::memory_order_release);
        }
    }
    kernel<<<grid, 32 * Sh::K, smem, st>>>(a, units);
    return cudaGetLastError();
}

template <typename T, typename Sh, int kMinCtas>
cudaError_t run_scan(const SelectiveArgs& a, cudaStream_t st) {
    if constexpr (Sh::kCanCopy) {
        VectorRule tok(sizeof(T)), bc(sizeof(T));
        tok.address(a.u).address(a.dt).elements(a.us_b).elements(a.us_t).elements(a.ds_b).elements(a.ds_t);
        if (a.z) tok.address(a.z).elements(a.zs_b).elements(a.zs_t);
        tok.elements(a.channels / a.ngroups);
        bc.address(a.B).address(a.C).elements(a.bs_b).elements(a.bs_t).elements(a.cs_b).elements(a.cs_t);
        bc.elements(a.dstate);
        if (tok.multiple_of(Sh::TB) && bc.multiple_of(16))
            return a.seq_idx ? start_scan<T, Sh, kMinCtas, true, true>(a, st)
                             : start_scan<T, Sh, kMinCtas, false, true>(a, st);
    }
    return a.seq_idx ? start_scan<T, Sh, kMinCtas, true, false>(a, st)
                     : start_scan<T, Sh, kMinCtas, false, false>(a, st);
}

// LN lanes hold a channel's states. Up to 32 states: one channel per lane, 8 tokens
// per slice; two CTAs of 8 warps per SM, or one of 16 while there are no more CTAs
// than SMs. More states: two channels per lane, which halves the reads of B and C
// (N 64, 1024 tokens x 5120 channels: 202 us against 287), and slices of 4.
template <typename T, int LN>
cudaError_t scan_by_size(const SelectiveArgs& a, cudaStream_t st) {
    constexpr int kChannels = 32 / LN * (LN <= 8 ? 1 : 2);  // per CTA
    const int64_t per = a.channels / a.ngroups;
    const int64_t ctas = (int64_t)a.batch * a.ngroups * ((per + kChannels - 1) / kChannels);
    if constexpr (LN <= 8) {
        if (ctas <= 148) return run_scan<T, ScanShape<T, 1, 4, LN, 8, 16>, 1>(a, st);
        return run_scan<T, ScanShape<T, 1, 4, LN, 8, 8>, 2>(a, st);
    } else {
        if (ctas <= 2 * 148) return run_scan<T, ScanShape<T, 2, 4, LN, 4, 8>, 2>(a, st);
        return run_scan<T, ScanShape<T, 2, 4, LN, 4, 4>, 4>(a, st);
    }
}

template <typename T>
cudaError_t scan_by_states(const SelectiveArgs& a, cudaStream_t st) {
    if (a.dstate <= 8) return scan_by_size<T, 2>(a, st);
    if (a.dstate <= 16) return scan_by_size<T, 4>(a, st);
    if (a.dstate <= 32) return scan_by_size<T, 8>(a, st);
    if (a.dstate <= 64) return scan_by_size<T, 16>(a, st);
    if (a.dstate <= 128) return scan_by_size<T, 32>(a, st);
    return run_scan<T, ScanShape<T, 2, 8, 32, 2, 8>, 2>(a, st);
}

}  // namespace

cudaError_t launch_selective_scan(const SelectiveArgs& a, ssd_dtype dt, cudaStream_t st) {
    return dt == SSD_DTYPE_F32 ? scan_by_states<float>(a, st) : scan_by_states<__nv_bfloat16>(a, st);
}

cudaError_t launch_selective_step(const SelectiveArgs& a, ssd_dtype dt, cudaStream_t st) {
    return dt == SSD_DTYPE_F32 ? run_step<float>(a, st) : run_step<__nv_bfloat16>(a, st);
}

}  // namespace ssd
