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
// of tokens with the last W - 1 inputs in registers, so x is read once, plus
// W - 1 tokens per tile.

#include "ssd_block.cuh"

namespace ssd {

namespace {

constexpr int kConvThreads = 128;
constexpr int kConvBatch = 8;  // tokens whose loads are in flight together

template <typename T, int V>
__device__ __forceinline__ T* conv_out(const ConvArgs& a, int64_t row, int c) {
    if (c < a.c1) return static_cast<T*>(a.out[0]) + row * a.c1 + c;
    if (c < a.c2) return static_cast<T*>(a.out[1]) + row * (a.c2 - a.c1) + (c - a.c1);
    return static_cast<T*>(a.out[2]) + row * (a.channels - a.c2) + (c - a.c2);
}

template <int V, int W>
struct Taps {
    float w[V][W];
    float bias[V];
    __device__ __forceinline__ void load(const ConvArgs& a, int c) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[e][k] = __ldg(a.weight + (int64_t)(c + e) * W + k);
            bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
        }
    }
};

// out = act(bias + taps . (win[0 .. W-2], x)), one rounding at the end
template <typename T, int V, int W>
__device__ __forceinline__ Pack<T, V> conv_token(const Taps<V, W>& taps, const Pack<T, V> (&win)[W - 1],
                                                 const Pack<T, V>& x, int silu) {
    Pack<T, V> y;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float acc = taps.bias[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) acc = fmaf(taps.w[e][k], to_f32(win[k].v[e]), acc);
        acc = fmaf(taps.w[e][W - 1], to_f32(x.v[e]), acc);
        y.v[e] = from_f32<T>(silu ? silu_for<T>(acc) : acc);
    }
    return y;
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zero_pack() {
    Pack<T, V> p;
#pragma unroll
    for (int e = 0; e < V; ++e) p.v[e] = from_f32<T>(0.f);
    return p;
}

// kSeq: sequence ids are given (else one sequence per row, id 0)
template <typename T, int V, int W, bool kSeq>
__global__ void __launch_bounds__(kConvThreads) causal_conv_kernel(const ConvArgs a, int ncv, int ntiles, int tile,
                                                                   int64_t nthreads) {
    using P = Pack<T, V>;
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
    const int32_t* ids = kSeq ? a.seq_idx : nullptr;
    // window w of sequence s: entry j (0 = oldest) at [j]
    const auto window = [&](const void* base, int s, int j) {
        return reinterpret_cast<P*>(const_cast<T*>(static_cast<const T*>(base)) +
                                    (((int64_t)b * a.nseq + s) * (W - 1) + j) * a.channels + c);
    };
    const auto init_entry = [&](int s, int j) { return a.init ? *window(a.init, s, j) : zero_pack<T, V>(); };
    // ids that do not occur keep their initial window
    const auto keep = [&](int lo, int hi) {
        if (!a.final_states) return;
        for (int s = lo; s < hi; ++s)
            for (int j = 0; j < W - 1; ++j) *window(a.final_states, s, j) = init_entry(s, j);
    };
    Taps<V, W> taps;
    taps.load(a, c);
    P win[W - 1];
    int s = seq_at(ids, row0, t0, a.nseq);
    {  // the window before token t0: inputs of its sequence, and the initial window before those
        int have = 0;
#pragma unroll
        for (int j = 1; j < W; ++j)
            if (have == j - 1 && t0 - j >= 0 && seq_at(ids, row0, t0 - j, a.nseq) == s) have = j;
#pragma unroll
        for (int j = 1; j < W; ++j)  // j tokens back
            win[W - 1 - j] = j <= have ? *reinterpret_cast<const P*>(x + (int64_t)(t0 - j) * a.xs_t)
                                       : init_entry(s, W - 1 - (j - have));
        if (have == 0) {
            const int before = t0 > 0 ? seq_at(ids, row0, t0 - 1, a.nseq) : -1;
            if (s != before) keep(before + 1, s);
        }
    }
    for (int tb = t0; tb < t1; tb += kConvBatch) {
        P xs[kConvBatch];
        int id[kConvBatch + 1];
#pragma unroll
        for (int j = 0; j < kConvBatch; ++j)
            if (tb + j < t1) xs[j] = *reinterpret_cast<const P*>(x + (int64_t)(tb + j) * a.xs_t);
        if (kSeq) {
#pragma unroll
            for (int j = 0; j <= kConvBatch; ++j) id[j] = tb + j < T_ ? seq_at(ids, row0, tb + j, a.nseq) : -1;
        }
#pragma unroll
        for (int j = 0; j < kConvBatch; ++j) {
            const int t = tb + j;
            if (t >= t1) break;
            if (kSeq && t > t0 && id[j] != s) {  // a sequence starts here (at t0: the prologue did it)
                keep(s + 1, id[j]);
                s = id[j];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[k] = init_entry(s, k);
            }
            *reinterpret_cast<P*>(conv_out<T, V>(a, row0 + t, c)) = conv_token<T, V, W>(taps, win, xs[j], a.silu);
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) win[k] = win[k + 1];
            win[W - 2] = xs[j];
            const bool ends = t == T_ - 1 || (kSeq && id[j + 1] != s);
            if (ends && a.final_states) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) *window(a.final_states, s, k) = win[k];
                if (t == T_ - 1) keep(s + 1, a.nseq);
            }
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
    P win[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) win[k] = *reinterpret_cast<const P*>(state + (int64_t)k * a.channels);
    Taps<V, W> taps;
    taps.load(a, c);
    *reinterpret_cast<P*>(conv_out<T, V>(a, b, c)) = conv_token<T, V, W>(taps, win, x, a.silu);
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) *reinterpret_cast<P*>(state + (int64_t)k * a.channels) = win[k + 1];
    *reinterpret_cast<P*>(state + (int64_t)(W - 2) * a.channels) = x;
}

// bytes per access that every row, window and output of the problem allows
template <typename T>
int conv_access(const ConvArgs& a, bool step) {
    VectorRule r(sizeof(T));
    r.address(a.x).address(a.init).address(a.final_states).address(a.out[0]).address(a.out[1]).address(a.out[2]);
    r.elements(a.channels).elements(a.c1).elements(a.c2).elements(a.xs_b);
    if (!step) r.elements(a.xs_t);
    return r.multiple_of(16) ? 16 : (r.multiple_of(4) ? 4 : (int)sizeof(T));
}

template <typename T, int V, int W>
cudaError_t run_conv(const ConvArgs& a, cudaStream_t st) {
    const int ncv = a.channels / V;
    const int tile = 32;
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
