// ssd_block_api.cu -- host side of the operators around the scan: argument
// validation and launch. Nothing here allocates, synchronises or reads device
// memory.

#include <cmath>

#include "ssd_block.cuh"
#include "ssd_host.cuh"

namespace {

using ssd::check_device;
using ssd::cuda_status;
using ssd::TraceRange;

constexpr int64_t kMaxChannels = 1 << 20;
constexpr int64_t kMaxSeqs = 1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

size_t elem_size(ssd_dtype t) { return t == SSD_DTYPE_F32 ? 4 : 2; }

bool known_dtype(ssd_dtype t) { return t == SSD_DTYPE_F32 || t == SSD_DTYPE_BF16; }

bool aligned_to(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// The bytes of memory from a tensor's first to its last element.
struct Span {
    uintptr_t lo, hi;  // hi exclusive; lo == hi for an absent tensor
};

Span dense(const void* p, int64_t n, size_t e) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + (uintptr_t)n * e : a};
}

Span strided(const void* p, int64_t batch, int64_t tokens, const int64_t* stride, int64_t channels, size_t e) {
    if (!p) return {0, 0};  // an absent tensor's strides are not read
    return dense(p, (batch - 1) * stride[0] + (tokens - 1) * stride[1] + channels, e);
}

bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// No output (the first n_out spans) overlaps another output or an input.
template <size_t M>
bool apart(const Span (&s)[M], int n_out) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < (int)M; ++j)
            if (overlap(s[i], s[j])) return false;
    return true;
}

// INVALID for a negative stride, UNSUPPORTED for one whose extent could pass 62 bits
ssd_status check_strides(const int64_t* s, int n, int64_t batch, int64_t tokens) {
    const int64_t count[2] = {batch, tokens};
    for (int i = 0; i < n; ++i) {
        if (s[i] < 0) return SSD_ERR_INVALID_ARG;
        if (s[i] > kMaxStride || (double)s[i] * (double)count[i] > 1e18) return SSD_ERR_UNSUPPORTED;
    }
    return SSD_OK;
}

ssd_status check_sizes(int64_t batch, int64_t seqlen, int64_t channels) {
    if (batch < 1 || seqlen < 1 || channels < 1) return SSD_ERR_INVALID_ARG;
    // token indices and a few tiles beyond the last one stay in 32 bits
    if (batch > INT32_MAX || seqlen > (1 << 30) || batch * seqlen > INT32_MAX || channels > kMaxChannels)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Strides a single token does not have count as 0 (they are never used).
struct Strides {
    int64_t s[2];
    Strides(const int64_t* p, bool step) : s{p[0], step ? 0 : p[1]} {}
};

ssd_status check_conv(const ssd_conv_problem* p, bool step) {
    if (!p) return SSD_ERR_INVALID_ARG;
    ssd_status s = check_sizes(p->batch, step ? 1 : p->seqlen, p->channels);
    if (s != SSD_OK) return s;
    if (!known_dtype(p->dtype) || (p->act != SSD_ACT_NONE && p->act != SSD_ACT_SILU)) return SSD_ERR_INVALID_ARG;
    if (p->width < 1 || (!step && p->nseq < 1)) return SSD_ERR_INVALID_ARG;
    const int64_t* q = p->split;
    if (q[0] < 1 || q[1] < 0 || q[2] < 0 || (q[1] == 0 && q[2] != 0) || q[0] > p->channels || q[1] > p->channels ||
        q[2] > p->channels || q[0] + q[1] + q[2] != p->channels)
        return SSD_ERR_INVALID_ARG;
    if (p->width < 2 || p->width > 4) return SSD_ERR_UNSUPPORTED;
    if (!step && p->nseq > kMaxSeqs) return SSD_ERR_UNSUPPORTED;
    return check_strides(p->x_stride, step ? 1 : 2, p->batch, p->seqlen);
}

// The arguments both convolution entry points share; `window` is the state of
// the step, and the initial windows of the prompt form.
ssd::ConvArgs conv_args(const ssd_conv_problem* p, bool step, const void* x, const float* weight, const float* bias,
                        const void* init, const int32_t* seq_idx, void* const* out, void* final_states) {
    ssd::ConvArgs a;
    a.batch = (int)p->batch;
    a.seqlen = step ? 1 : (int)p->seqlen;
    a.channels = (int)p->channels;
    a.width = (int)p->width;
    a.nseq = step ? 1 : (int)p->nseq;
    a.xs_b = p->x_stride[0];
    a.xs_t = step ? 0 : p->x_stride[1];
    a.c1 = (int)p->split[0];
    a.c2 = (int)(p->split[0] + p->split[1]);
    a.silu = p->act == SSD_ACT_SILU;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.init = init;
    a.seq_idx = seq_idx;
    for (int i = 0; i < 3; ++i) a.out[i] = p->split[i] ? out[i] : nullptr;
    a.final_states = final_states;
    return a;
}

ssd_status run_conv(const ssd_conv_problem* p, bool step, const void* x, const float* weight, const float* bias,
                    const void* init, const int32_t* seq_idx, void* const* out, void* final_states, void* stream) {
    ssd_status s = check_conv(p, step);
    if (s != SSD_OK) return s;
    if (!step && !seq_idx && p->nseq != 1) return SSD_ERR_INVALID_ARG;
    if (!x || !weight || (step && !final_states)) return SSD_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if ((p->split[i] != 0) != (out[i] != nullptr)) return SSD_ERR_INVALID_ARG;
    const size_t e = elem_size(p->dtype);
    for (const void* q : {x, init, (const void*)final_states, (const void*)out[0], (const void*)out[1],
                          (const void*)out[2]})
        if (!aligned_to(q, e)) return SSD_ERR_INVALID_ARG;
    for (const void* q : {(const void*)weight, (const void*)bias, (const void*)seq_idx})
        if (!aligned_to(q, 4)) return SSD_ERR_INVALID_ARG;
    const int64_t T = step ? 1 : p->seqlen, rows = p->batch * T;
    const int64_t windows = p->batch * (step ? 1 : p->nseq) * (p->width - 1) * p->channels;
    const Strides xs(p->x_stride, step);
    const Span spans[] = {dense(out[0], rows * p->split[0], e),
                          dense(out[1], rows * p->split[1], e),
                          dense(out[2], rows * p->split[2], e),
                          dense(final_states, windows, e),
                          strided(x, p->batch, T, xs.s, p->channels, e),
                          dense(weight, p->channels * p->width, 4),
                          dense(bias, p->channels, 4),
                          dense(seq_idx, rows, 4),
                          dense(step ? nullptr : init, windows, e)};
    if (!apart(spans, 4)) return SSD_ERR_INVALID_ARG;
    // one thread per channel and token at most: the grid stays below 2^31 blocks of 128
    if ((double)rows * (double)p->channels > 128.0 * INT32_MAX) return SSD_ERR_UNSUPPORTED;
    if ((s = check_device()) != SSD_OK) return s;
    const ssd::ConvArgs a = conv_args(p, step, x, weight, bias, init, seq_idx, out, final_states);
    cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(step ? ssd::launch_conv_step(a, p->dtype, st) : ssd::launch_causal_conv(a, p->dtype, st));
}

ssd_status check_selective(const ssd_selective_problem* p, bool step) {
    if (!p) return SSD_ERR_INVALID_ARG;
    ssd_status s = check_sizes(p->batch, step ? 1 : p->seqlen, p->channels);
    if (s == SSD_ERR_INVALID_ARG) return s;
    if (p->dstate < 1 || p->ngroups < 1 || p->channels % p->ngroups != 0 || !known_dtype(p->dtype) ||
        (!step && p->nseq < 1))
        return SSD_ERR_INVALID_ARG;
    if (s != SSD_OK) return s;
    if (p->dstate > 256 || (!step && p->nseq > kMaxSeqs)) return SSD_ERR_UNSUPPORTED;
    if (p->batch * p->channels > INT32_MAX) return SSD_ERR_UNSUPPORTED;  // CTAs: at most one per channel
    return SSD_OK;
}

ssd_status run_selective(const ssd_selective_problem* p, bool step, const void* u, const void* dt, const float* A,
                         const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                         const float* init, const int32_t* seq_idx, void* y, float* final_states, void* stream) {
    ssd_status s = check_selective(p, step);
    if (s != SSD_OK) return s;
    for (const int64_t* q : {p->u_stride, p->dt_stride, z ? p->z_stride : p->u_stride, p->B_stride, p->C_stride})
        if ((s = check_strides(q, step ? 1 : 2, p->batch, p->seqlen)) != SSD_OK) return s;
    if (!step && !seq_idx && p->nseq != 1) return SSD_ERR_INVALID_ARG;
    if (!u || !dt || !A || !B || !C || !y || (step && !final_states)) return SSD_ERR_INVALID_ARG;
    const size_t e = elem_size(p->dtype);
    for (const void* q : {u, dt, B, C, z, (const void*)y})
        if (!aligned_to(q, e)) return SSD_ERR_INVALID_ARG;
    for (const void* q : {(const void*)A, (const void*)D, (const void*)dt_bias, (const void*)init,
                          (const void*)seq_idx, (const void*)final_states})
        if (!aligned_to(q, 4)) return SSD_ERR_INVALID_ARG;
    const int64_t T = step ? 1 : p->seqlen, rows = p->batch * T, n = p->channels;
    const int64_t states = p->batch * (step ? 1 : p->nseq) * p->dstate * n, GN = p->ngroups * p->dstate;
    const Strides us(p->u_stride, step), ds(p->dt_stride, step), zs(z ? p->z_stride : p->u_stride, step), bs(p->B_stride, step),
        cs(p->C_stride, step);
    const Span spans[] = {dense(y, rows * n, e),
                          dense(final_states, states, 4),
                          strided(u, p->batch, T, us.s, n, e),
                          strided(dt, p->batch, T, ds.s, n, e),
                          strided(z, p->batch, T, zs.s, n, e),
                          strided(B, p->batch, T, bs.s, GN, e),
                          strided(C, p->batch, T, cs.s, GN, e),
                          dense(A, n * p->dstate, 4),
                          dense(D, n, 4),
                          dense(dt_bias, n, 4),
                          dense(init, states, 4),
                          dense(seq_idx, rows, 4)};
    if (!apart(spans, 2)) return SSD_ERR_INVALID_ARG;
    if ((s = check_device()) != SSD_OK) return s;
    ssd::SelectiveArgs a;
    a.batch = (int)p->batch;
    a.seqlen = (int)T;
    a.channels = (int)n;
    a.dstate = (int)p->dstate;
    a.ngroups = (int)p->ngroups;
    a.nseq = step ? 1 : (int)p->nseq;
    a.us_b = us.s[0], a.us_t = us.s[1];
    a.ds_b = ds.s[0], a.ds_t = ds.s[1];
    a.zs_b = zs.s[0], a.zs_t = zs.s[1];
    a.bs_b = bs.s[0], a.bs_t = bs.s[1];
    a.cs_b = cs.s[0], a.cs_t = cs.s[1];
    a.softplus = p->dt_softplus != 0;
    a.u = u, a.dt = dt, a.B = B, a.C = C, a.z = z;
    a.A = A, a.D = D, a.dt_bias = dt_bias;
    a.init = init;
    a.seq_idx = seq_idx;
    a.y = y;
    a.final_states = final_states;
    cudaStream_t st = (cudaStream_t)stream;
    return cuda_status(step ? ssd::launch_selective_step(a, p->dtype, st)
                            : ssd::launch_selective_scan(a, p->dtype, st));
}

ssd_status check_norm(const ssd_norm_problem* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    ssd_status s = check_sizes(p->batch, p->seqlen, p->channels);
    if (s == SSD_ERR_INVALID_ARG) return s;
    if (p->ngroups < 1 || p->channels % p->ngroups != 0 || !known_dtype(p->dtype) || !(p->eps >= 0.f) ||
        std::isinf(p->eps))
        return SSD_ERR_INVALID_ARG;
    if (s != SSD_OK) return s;
    if (p->channels / p->ngroups > 32768) return SSD_ERR_UNSUPPORTED;
    if (p->batch * p->seqlen * p->ngroups > INT32_MAX) return SSD_ERR_UNSUPPORTED;  // CTAs
    if ((s = check_strides(p->x_stride, 2, p->batch, p->seqlen)) != SSD_OK) return s;
    return SSD_OK;
}

ssd::NormArgs norm_args(const ssd_norm_problem* p, ssd::NormMode mode, const void* x, const void* z,
                        const float* weight, const float* scale, void* out, void* residual_out) {
    ssd::NormArgs a;
    a.batch = (int)p->batch;
    a.seqlen = (int)p->seqlen;
    a.channels = (int)p->channels;
    a.ngroups = (int)p->ngroups;
    a.xs_b = p->x_stride[0], a.xs_t = p->x_stride[1];
    a.zs_b = z ? p->z_stride[0] : 0, a.zs_t = z ? p->z_stride[1] : 0;
    a.eps = p->eps;
    a.alpha = p->alpha;
    a.mode = mode;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.scale = scale;
    a.out = out;
    a.residual_out = residual_out;
    return a;
}

}  // namespace

extern "C" {

ssd_status ssd_causal_conv(const ssd_conv_problem* p, const void* x, const float* weight, const float* bias,
                           const void* init_states, const int32_t* seq_idx, void* out0, void* out1, void* out2,
                           void* final_states, void* stream) {
    TraceRange trace("ssd_causal_conv");
    void* const out[3] = {out0, out1, out2};
    return run_conv(p, false, x, weight, bias, init_states, seq_idx, out, final_states, stream);
}

ssd_status ssd_conv_step(const ssd_conv_problem* p, const void* x, const float* weight, const float* bias,
                         void* state, void* out0, void* out1, void* out2, void* stream) {
    TraceRange trace("ssd_conv_step");
    void* const out[3] = {out0, out1, out2};
    return run_conv(p, true, x, weight, bias, nullptr, nullptr, out, state, stream);
}

ssd_status ssd_selective_scan(const ssd_selective_problem* p, const void* u, const void* dt, const float* A,
                              const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                              const float* init_states, const int32_t* seq_idx, void* y, float* final_states,
                              void* stream) {
    TraceRange trace("ssd_selective_scan");
    return run_selective(p, false, u, dt, A, B, C, D, z, dt_bias, init_states, seq_idx, y, final_states, stream);
}

ssd_status ssd_selective_step(const ssd_selective_problem* p, const void* u, const void* dt, const float* A,
                              const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                              float* state, void* y, void* stream) {
    TraceRange trace("ssd_selective_step");
    return run_selective(p, true, u, dt, A, B, C, D, z, dt_bias, nullptr, nullptr, y, state, stream);
}

ssd_status ssd_gated_norm(const ssd_norm_problem* p, const void* x, const void* z, const float* weight, void* out,
                          void* stream) {
    TraceRange trace("ssd_gated_norm");
    ssd_status s = check_norm(p);
    if (s != SSD_OK) return s;
    if (z && (s = check_strides(p->z_stride, 2, p->batch, p->seqlen)) != SSD_OK) return s;
    if (!x || !weight || !out) return SSD_ERR_INVALID_ARG;
    const size_t e = elem_size(p->dtype);
    if (!aligned_to(x, e) || !aligned_to(z, e) || !aligned_to(out, e) || !aligned_to(weight, 4))
        return SSD_ERR_INVALID_ARG;
    const Span spans[] = {dense(out, p->batch * p->seqlen * p->channels, e),
                          strided(x, p->batch, p->seqlen, p->x_stride, p->channels, e),
                          strided(z, p->batch, p->seqlen, p->z_stride, p->channels, e),
                          dense(weight, p->channels, 4)};
    if (!apart(spans, 1)) return SSD_ERR_INVALID_ARG;
    if ((s = check_device()) != SSD_OK) return s;
    const ssd::NormMode mode = !z ? ssd::kNormPlain : (p->gate_first ? ssd::kNormGateFirst : ssd::kNormGateLast);
    return cuda_status(ssd::launch_row_norm(norm_args(p, mode, x, z, weight, nullptr, out, nullptr), p->dtype,
                                            p->dtype, (cudaStream_t)stream));
}

ssd_status ssd_add_norm(const ssd_norm_problem* p, const void* x, const void* residual, const float* weight,
                        const float* scale, void* out, void* residual_out, void* stream) {
    TraceRange trace("ssd_add_norm");
    ssd_status s = check_norm(p);
    if (s != SSD_OK) return s;
    if (residual && (s = check_strides(p->z_stride, 2, p->batch, p->seqlen)) != SSD_OK) return s;
    if (p->ngroups != 1 || (p->residual_dtype != SSD_DTYPE_F32 && p->residual_dtype != p->dtype))
        return SSD_ERR_INVALID_ARG;
    if (!x || !weight || !out || !residual_out) return SSD_ERR_INVALID_ARG;
    const size_t e = elem_size(p->dtype), r = elem_size(p->residual_dtype);
    if (!aligned_to(x, e) || !aligned_to(out, e) || !aligned_to(residual, r) || !aligned_to(residual_out, r) ||
        !aligned_to(weight, 4) || !aligned_to(scale, 4))
        return SSD_ERR_INVALID_ARG;
    const int64_t n = p->batch * p->seqlen * p->channels;
    // in place: each thread reads the residual's elements before it writes them
    const bool in_place = residual && residual == residual_out &&
                          (p->seqlen == 1 || p->z_stride[1] == p->channels) &&
                          (p->batch == 1 || p->z_stride[0] == p->seqlen * p->channels);
    const Span spans[] = {dense(out, n, e),
                          dense(residual_out, n, r),
                          strided(x, p->batch, p->seqlen, p->x_stride, p->channels, e),
                          in_place ? Span{0, 0}
                                   : strided(residual, p->batch, p->seqlen, p->z_stride, p->channels, r),
                          dense(weight, p->channels, 4),
                          dense(scale, p->channels, 4)};
    if (!apart(spans, 2)) return SSD_ERR_INVALID_ARG;
    if ((s = check_device()) != SSD_OK) return s;
    return cuda_status(ssd::launch_row_norm(norm_args(p, ssd::kNormAdd, x, residual, weight, scale, out, residual_out),
                                            p->dtype, p->residual_dtype, (cudaStream_t)stream));
}

}  // extern "C"
