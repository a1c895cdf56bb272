// ssd_conv.cu -- the short causal convolution in front of the scan, for prompts
// (packed sequences, initial and final windows) and for single tokens.
//
//   y[t, c] = act(bias[c] + sum_k weight[c, k] in[t - (W - 1) + k, c])
//
// Source: "Mamba" (ai.tomabc.com): conv1d and SiLU of the block pseudocode. Each
// channel has its own W <= 4 taps, so there is no matrix product in it: 2 W + 5
// operations per element against 2 elements moved. Both kernels are bound by
// the bytes of x and y.
//
// Prompts: a thread owns V channels (16 bytes of a token's row) and walks a tile
// of tokens in batches of kConvBatch with the last W - 1 inputs in registers, so x
// is read once, plus W - 1 tokens per tile. A batch that lies in one sequence is
// computed channel pair by channel pair (packed fp32 pairs), its outputs replacing
// its inputs in the registers; other batches go token by token. Inputs are copied
// ahead into the thread's own slots of shared memory: a register ring of the same
// depth spilled at the 128 registers that 16 warps per SM allow. Measured at b 4 x
// T 4096 x 5376 channels, bf16, W 4: 71 us on the device (5.0 TB/s of x and y), 100 us without
// the copies ahead, 114 us with the window in fp32 registers and scalar taps. Left
// to the bytes' time (55 us): the taps' and first inputs' latency at each tile's
// start, and two special-function operations per element for the silu (39 us).

#include "ssd_block.cuh"

namespace ssd {

namespace {

constexpr int kConvThreads = 128;
constexpr int kConvBatch = 4;  // tokens computed together
constexpr int kConvAhead = 3;  // batches in flight, where a thread moves 16 bytes per token

// Where a thread's channels go: address of row 0 and the row's length.
template <typename T>
struct ConvOut {
    T* p;
    int row;
    __device__ __forceinline__ ConvOut(const ConvArgs& a, int c) {
        if (c < a.c1)
            p = static_cast<T*>(a.out[0]) + c, row = a.c1;
        else if (c < a.c2)
            p = static_cast<T*>(a.out[1]) + (c - a.c1), row = a.c2 - a.c1;
        else
            p = static_cast<T*>(a.out[2]) + (c - a.c2), row = a.channels - a.c2;
    }
};

// One or two channels side by side, in fp32.
template <int G>
struct Lanes;
template <>
struct Lanes<1> {
    using F = float;
    static __device__ __forceinline__ F fma(F a, F b, F c) { return fmaf(a, b, c); }
    template <typename T>
    static __device__ __forceinline__ F load(const T* p) {
        return to_f32(*p);
    }
    template <typename T>
    static __device__ __forceinline__ void store(T* p, F v) {
        *p = from_f32<T>(v);
    }
};
template <>
struct Lanes<2> {
    using F = float2;
    static __device__ __forceinline__ F fma(F a, F b, F c) { return __ffma2_rn(a, b, c); }
    static __device__ __forceinline__ F load(const float* p) { return make_float2(p[0], p[1]); }
    static __device__ __forceinline__ F load(const __nv_bfloat16* p) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
    }
    static __device__ __forceinline__ void store(float* p, F v) { p[0] = v.x, p[1] = v.y; }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, F v) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
    }
};

// The taps and bias of V channels, in groups of G.
template <int V, int W>
struct Taps {
    static constexpr int G = V % 2 == 0 ? 2 : 1;
    using L = Lanes<G>;
    using F = typename L::F;
    F w[V / G][W], bias[V / G];
    __device__ __forceinline__ void load(const ConvArgs& a, int c) {
        constexpr int Q = G == 2 && V * W % 4 == 0 ? 4 : 1;  // G = 2: the launcher checked the 16-byte alignment
        float raw[V * W];
        const auto* src = reinterpret_cast<const Pack<float, Q>*>(a.weight + (int64_t)c * W);
#pragma unroll
        for (int i = 0; i < V * W / Q; ++i) {
            const Pack<float, Q> v = src[i];
#pragma unroll
            for (int k = 0; k < Q; ++k) raw[i * Q + k] = v.v[k];
        }
#pragma unroll
        for (int e = 0; e < V / G; ++e) {
            float b[G];
#pragma unroll
            for (int i = 0; i < G; ++i) b[i] = a.bias ? __ldg(a.bias + c + e * G + i) : 0.f;
            bias[e] = L::load(b);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                float t[G];
#pragma unroll
                for (int i = 0; i < G; ++i) t[i] = raw[(e * G + i) * W + k];
                w[e][k] = L::load(t);
            }
        }
    }
    // act(bias + taps . in[0 .. W-1]) of channel group e
    template <typename T>
    __device__ __forceinline__ F apply(int e, const F* in, int silu) const {
        F acc = bias[e];
#pragma unroll
        for (int k = 0; k < W; ++k) acc = L::fma(w[e][k], in[k], acc);
        return silu ? silu_for<T>(acc) : acc;
    }
    // all channels of one token; in[W-1] is the token itself
    template <typename T>
    __device__ __forceinline__ Pack<T, V> token(const Pack<T, V> (&in)[W], int silu) const {
        Pack<T, V> y;
#pragma unroll
        for (int e = 0; e < V / G; ++e) {
            F f[W];
#pragma unroll
            for (int k = 0; k < W; ++k) f[k] = L::load(&in[k].v[e * G]);
            L::store(&y.v[e * G], apply<T>(e, f, silu));
        }
        return y;
    }
};

// kSeq: sequence ids are given (else one sequence per row, id 0).
template <typename T, int V, int W, bool kSeq>
__global__ void __launch_bounds__(kConvThreads, V >= 4 ? 4 : 1)
    causal_conv_kernel(const ConvArgs a, int ncv, int ntiles, int tile, int64_t nthreads) {
    using P = Pack<T, V>;
    using L = typename Taps<V, W>::L;
    constexpr int G = Taps<V, W>::G;
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    if (i >= nthreads) return;
    int cv, tl, b;  // channel vector (fastest), tile, batch row
    if (nthreads <= UINT32_MAX) {  // a 64-bit division costs several times a 32-bit one
        const uint32_t r = (uint32_t)i / (uint32_t)ncv;
        cv = (int)((uint32_t)i - r * (uint32_t)ncv);
        b = (int)(r / (uint32_t)ntiles);
        tl = (int)(r - (uint32_t)b * (uint32_t)ntiles);
    } else {
        const int64_t r = i / ncv;
        cv = (int)(i - r * ncv);
        b = (int)(r / ntiles);
        tl = (int)(r - (int64_t)b * ntiles);
    }
    const int c = cv * V, T_ = a.seqlen;
    const int t0 = tl * tile, t1 = min(T_, t0 + tile);
    const T* x = static_cast<const T*>(a.x) + b * a.xs_b + c;
    const int64_t row0 = (int64_t)b * T_;
    const auto id_at = [&](int t) { return seq_at(kSeq ? a.seq_idx : nullptr, row0, t, a.nseq); };
    const auto input = [&](int t) { return *reinterpret_cast<const P*>(x + (int64_t)t * a.xs_t); };
    // windows of sequence s: entry j (0 = oldest)
    const auto entry = [&](int s, int j) { return (((int64_t)b * a.nseq + s) * (W - 1) + j) * a.channels + c; };
    const auto init_entry = [&](int s, int j) {
        P p;
#pragma unroll
        for (int e = 0; e < V; ++e) p.v[e] = from_f32<T>(0.f);
        if (a.init) p = *reinterpret_cast<const P*>(static_cast<const T*>(a.init) + entry(s, j));
        return p;
    };
    const auto put_entry = [&](int s, int j, const P& p) {
        *reinterpret_cast<P*>(static_cast<T*>(a.final_states) + entry(s, j)) = p;
    };
    // ids that do not occur keep their initial window
    const auto keep = [&](int lo, int hi) {
        if (!a.final_states) return;
        for (int s = lo; s < hi; ++s)
            for (int j = 0; j < W - 1; ++j) put_entry(s, j, init_entry(s, j));
    };
    // the W - 1 inputs before token t of sequence s: tokens of s, and the initial window before those
    const auto window = [&](int t, int s, P* win) {
        int have = 0;
#pragma unroll
        for (int j = 1; j < W; ++j)
            if (have == j - 1 && t - j >= 0 && id_at(t - j) == s) have = j;
#pragma unroll
        for (int j = 1; j < W; ++j) win[W - 1 - j] = j <= have ? input(t - j) : init_entry(s, W - 1 - (j - have));
        if (have == 0) keep(t > 0 ? id_at(t - 1) + 1 : 0, s);  // t is its sequence's first token
    };
    Taps<V, W> taps;
    taps.load(a, c);
    const ConvOut<T> out(a, c);
    T* y = out.p + (row0 + t0) * out.row;
    P win[W - 1];
    int s = id_at(t0);
    window(t0, s, win);
    bool have_window = true;
    // 16-byte inputs are copied ahead into shared memory, each thread's into its own slots
    constexpr bool kRing = sizeof(P) == 16;
    __shared__ P ring[kRing ? kConvAhead * kConvBatch : 1][kRing ? kConvThreads : 1];
    const T* ahead = x + (int64_t)t0 * a.xs_t;
    const auto copy_batch = [&](int tb, int slot) {
#pragma unroll
        for (int j = 0; j < kConvBatch; ++j) {
            if (tb + j < t1) copy_async<16>(&ring[slot + j][threadIdx.x], ahead, 16);
            ahead += a.xs_t;
        }
        copy_commit();
    };
    if constexpr (kRing) {
#pragma unroll
        for (int k = 0; k < kConvAhead; ++k) copy_batch(t0 + k * kConvBatch, k * kConvBatch);
    }
    int slot = 0;
    for (int tb = t0; tb < t1; tb += kConvBatch) {
        bool whole = tb + kConvBatch <= t1, ends = tb + kConvBatch == T_;
        if (kSeq && whole) {
            if (!have_window || id_at(tb) != s) {
                s = id_at(tb);
                window(tb, s, win);
                have_window = true;
            }
            // ids do not decrease along a row, but out-of-contract ones must not mix windows either
            for (int j = 1; j < kConvBatch; ++j) whole &= id_at(tb + j) == s;
            ends |= tb + kConvBatch < T_ && id_at(tb + kConvBatch) != s;
        }
        if (whole) {
            P xs[kConvBatch];
            if constexpr (kRing) {
                copy_wait<kConvAhead - 1>();
#pragma unroll
                for (int j = 0; j < kConvBatch; ++j) xs[j] = ring[slot + j][threadIdx.x];
            } else {
#pragma unroll
                for (int j = 0; j < kConvBatch; ++j) xs[j] = input(tb + j);
            }
#pragma unroll
            for (int e = 0; e < V / G; ++e) {
                typename L::F f[W - 1 + kConvBatch];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) f[k] = L::load(&win[k].v[e * G]);
#pragma unroll
                for (int j = 0; j < kConvBatch; ++j) f[W - 1 + j] = L::load(&xs[j].v[e * G]);
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
#pragma unroll
                    for (int q = 0; q < G; ++q) win[k].v[e * G + q] = xs[kConvBatch - (W - 1) + k].v[e * G + q];
#pragma unroll
                for (int j = 0; j < kConvBatch; ++j)
                    L::store(&xs[j].v[e * G], taps.template apply<T>(e, f + j, a.silu));
            }
#pragma unroll
            for (int j = 0; j < kConvBatch; ++j) {
                *reinterpret_cast<P*>(y) = xs[j];
                y += out.row;
            }
            if (ends && a.final_states) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) put_entry(s, k, win[k]);
                if (tb + kConvBatch == T_) keep(s + 1, a.nseq);
            }
        } else {
            have_window = false;
#pragma unroll 1
            for (int t = tb; t < min(tb + kConvBatch, t1); ++t) {
                P in[W];
                s = id_at(t);
                window(t, s, in);
                in[W - 1] = input(t);
                *reinterpret_cast<P*>(y) = taps.template token<T>(in, a.silu);
                y += out.row;
                if (a.final_states && (t == T_ - 1 || id_at(t + 1) != s)) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) put_entry(s, k, in[k + 1]);
                    if (t == T_ - 1) keep(s + 1, a.nseq);
                }
            }
            // The batch's own copies were not read, but have to land before its slots are copied into again:
            // copies are not ordered among each other.
            if constexpr (kRing) copy_wait<kConvAhead - 1>();
        }
        if constexpr (kRing) {
            copy_batch(tb + kConvAhead * kConvBatch, slot);
            slot = slot == (kConvAhead - 1) * kConvBatch ? 0 : slot + kConvBatch;
        }
    }
}

// One thread per V channels of a batch row: window and token in, window and y out.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvArgs a, int ncv, int64_t nthreads) {
    using P = Pack<T, V>;
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    if (i >= nthreads) return;
    const int64_t b = nthreads <= UINT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)ncv) : i / ncv;
    const int c = (int)(i - b * ncv) * V;
    const P x = *reinterpret_cast<const P*>(static_cast<const T*>(a.x) + b * a.xs_b + c);
    T* state = static_cast<T*>(a.final_states) + b * (W - 1) * a.channels + c;
    P raw[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) raw[k] = *reinterpret_cast<const P*>(state + (int64_t)k * a.channels);
    Taps<V, W> taps;
    taps.load(a, c);
    P in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k] = raw[k];
    in[W - 1] = x;
    const ConvOut<T> out(a, c);
    *reinterpret_cast<P*>(out.p + b * out.row) = taps.template token<T>(in, a.silu);
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) *reinterpret_cast<P*>(state + (int64_t)k * a.channels) = raw[k + 1];
    *reinterpret_cast<P*>(state + (int64_t)(W - 2) * a.channels) = x;
}

// bytes per access that every row, window and output of the problem allows
template <typename T>
int conv_access(const ConvArgs& a, bool step) {
    VectorRule r(sizeof(T));
    r.address(a.x).address(a.init).address(a.final_states).address(a.out[0]).address(a.out[1]).address(a.out[2]);
    r.elements(a.channels).elements(a.c1).elements(a.c2).elements(a.xs_b);
    if (!step) r.elements(a.xs_t);
    if (!VectorRule(4).address(a.weight).multiple_of(16)) return (int)sizeof(T);  // taps are loaded 16 bytes at a time
    return r.multiple_of(16) ? 16 : (r.multiple_of(4) ? 4 : (int)sizeof(T));
}

template <typename T, int V, int W>
cudaError_t run_conv(const ConvArgs& a, cudaStream_t st) {
    const int ncv = a.channels / V;
    // Tokens per thread: 32, where 3 extra inputs per tile hardly count, or fewer while the threads
    // would not fill the SMs (4 CTAs each).
    int tile = 32;
    while (tile > kConvBatch && (int64_t)a.batch * ((a.seqlen + tile - 1) / tile) * ncv < 148 * 4 * kConvThreads)
        tile /= 2;
    const int ntiles = (a.seqlen + tile - 1) / tile;
    const int64_t n = (int64_t)a.batch * ntiles * ncv;
    const unsigned grid = (unsigned)((n + kConvThreads - 1) / kConvThreads);
    if (a.seq_idx)
        causal_conv_kernel<T, V, W, true><<<grid, kConvThreads, 0, st>>>(a, ncv, ntiles, tile, n);
    else
        causal_conv_kernel<T, V, W, false><<<grid, kConvThreads, 0, st>>>(a, ncv, ntiles, tile, n);
    return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t run_step(const ConvArgs& a, cudaStream_t st) {
    const int ncv = a.channels / V;
    const int64_t n = (int64_t)a.batch * ncv;
    const unsigned grid = (unsigned)((n + kConvThreads - 1) / kConvThreads);
    conv_step_kernel<T, V, W><<<grid, kConvThreads, 0, st>>>(a, ncv, n);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t by_width(const ConvArgs& a, bool step, cudaStream_t st) {
    switch (a.width) {
        case 2: return step ? run_step<T, V, 2>(a, st) : run_conv<T, V, 2>(a, st);
        case 3: return step ? run_step<T, V, 3>(a, st) : run_conv<T, V, 3>(a, st);
        default: return step ? run_step<T, V, 4>(a, st) : run_conv<T, V, 4>(a, st);
    }
}

cudaError_t by_access(const ConvArgs& a, ssd_dtype dt, bool step, cudaStream_t st) {
    if (dt == SSD_DTYPE_F32)
        return conv_access<float>(a, step) == 16 ? by_width<float, 4>(a, step, st) : by_width<float, 1>(a, step, st);
    switch (conv_access<__nv_bfloat16>(a, step)) {
        case 16: return by_width<__nv_bfloat16, 8>(a, step, st);
        case 4: return by_width<__nv_bfloat16, 2>(a, step, st);
        default: return by_width<__nv_bfloat16, 1>(a, step, st);
    }
}

}  // namespace

cudaError_t launch_causal_conv(const ConvArgs& a, ssd_dtype dt, cudaStream_t st) { return by_access(a, dt, false, st); }

cudaError_t launch_conv_step(const ConvArgs& a, ssd_dtype dt, cudaStream_t st) { return by_access(a, dt, true, st); }

}  // namespace ssd
