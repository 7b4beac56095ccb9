// Rotary positions and group norm (declared in include/fedavg.h): argument checks, workspace,
// launches.
#include "strided.hpp"

#include "group_norm.cuh"
#include "rotary.cuh"

namespace {

// ----------------------------------------------------------------- rotary positions
fa_status rotary_impl(fa_work* w, const fa_rotary_args& p, cudaStream_t s) {
    if (p.flags & ~(FA_ROTARY_INTERLEAVED | FA_ROTARY_INVERSE)) return fail(w, FA_ERR_ARG, "unknown flag");
    if (!dtype_ok(p.dtype)) return fail(w, FA_ERR_DTYPE, "dtype");
    if (!std::isfinite(p.scale)) return fail(w, FA_ERR_ARG, "scale not finite");
    if (p.rotary_dim < 2 || p.rotary_dim % 2 || p.rotary_dim > FA_ROTARY_MAX_DIM || p.rotary_dim > p.head_dim)
        return fail(w, FA_ERR_RANGE, "rotary_dim is not an even number from 2 to FA_ROTARY_MAX_DIM and head_dim");
    if (p.head_dim > 65536 || p.q.heads > 65536 || p.k.heads > 65536)
        return fail(w, FA_ERR_RANGE, "head_dim or heads above 65536");
    if (p.batch >= kMaxSize || p.seq >= kMaxSize || (p.batch && p.seq >= (kMaxSize + p.batch - 1) / p.batch))
        return fail(w, FA_ERR_RANGE, "2^31 tokens or more");
    if (!p.turns) return fail(w, FA_ERR_ARG, "turns is NULL");
    if (!p.position && (p.first < 0 || p.first >> 62)) return fail(w, FA_ERR_RANGE, "first out of range");
    const uint64_t tokens = p.batch * p.seq;
    if (tokens == 0 || p.q.heads + p.k.heads == 0) return FA_OK;
    const uint64_t size = size_of(p.dtype);
    const fa_rotary_part* part[2] = {&p.q, &p.k};
    const char* const name[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    Grid in[2], out[2];
    bool inplace[2] = {true, true};
    for (int i = 0; i < 2; ++i) {
        const fa_rotary_part& t = *part[i];
        if (t.heads == 0) continue;
        in[i] = Grid(t.x, p.head_dim, size, {{p.batch, t.batch_stride}, {p.seq, t.token_stride}, {t.heads, t.head_stride}});
        out[i] = Grid(t.out, p.head_dim, size,
                      {{p.batch, t.out_batch_stride}, {p.seq, t.out_token_stride}, {t.heads, t.out_head_stride}});
        fa_status r = check_grid(w, in[i], name[i][0]);
        if (r == FA_OK) r = check_out(w, out[i], name[i][1]);
        if (r != FA_OK) return r;
        inplace[i] = in[i].same(out[i]);
    }
    fa_status r = p.position ? check_mat(w, p.position, 1, tokens, tokens, FA_F32, "position") : FA_OK;
    if (r != FA_OK) return r;
    const Extent position{p.position, 1, tokens, tokens, 4};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (!(i == j && inplace[i]) && overlap(out[i].extent(), in[j].extent()))
                return fail(w, FA_ERR_ARG, "an output overlaps q or k without being it");
    if (overlap(out[0].extent(), out[1].extent())) return fail(w, FA_ERR_ARG, "q_out overlaps k_out");
    if (overlap(out[0].extent(), position) || overlap(out[1].extent(), position))
        return fail(w, FA_ERR_ARG, "an output overlaps position");
    fa::RotaryArgs a{};
    for (int i = 0; i < 2; ++i) {
        const fa_rotary_part& t = *part[i];
        // strides of single elements are not used: zero, so that they do not spoil the alignment
        const auto used = [](uint64_t extent, uint64_t stride) { return extent > 1 ? stride : 0; };
        if (t.heads)
            a.part[i] = {t.x, t.out, used(p.batch, t.batch_stride), used(p.seq, t.token_stride), used(t.heads, t.head_stride),
                         used(p.batch, t.out_batch_stride), used(p.seq, t.out_token_stride), used(t.heads, t.out_head_stride),
                         t.heads};
    }
    a.position = p.position;
    a.first = p.first;
    a.err = w->err_dev;
    a.tokens = static_cast<uint32_t>(tokens);
    a.seq = static_cast<uint32_t>(p.seq);
    a.head_dim = p.head_dim;
    a.rotary_dim = p.rotary_dim;
    a.dtype = code_of(p.dtype);
    a.scale = static_cast<float>(p.scale);
    a.interleaved = p.flags & FA_ROTARY_INTERLEAVED;
    a.inverse = p.flags & FA_ROTARY_INVERSE;
    a.copy = p.rotary_dim < p.head_dim && !(inplace[0] && inplace[1]);
    std::memcpy(a.turns, p.turns, p.rotary_dim / 2 * sizeof(uint64_t));
    const bool cap = capturing(s);
    r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    ChainOut chain(w, s, cap);
    return chain.end(launched(w, fa::launch_rotary(a, static_cast<uint32_t>(w->tc.sms), s), "rotary positions"));
}

// ----------------------------------------------------------------- group norm
template <typename Args>
fa_status check_norm(fa_work* w, const Args& p) {
    if (p.flags) return fail(w, FA_ERR_ARG, "unknown flag");
    if (!dtype_ok(p.dtype) || !dtype_ok(p.dtype_param)) return fail(w, FA_ERR_DTYPE, "dtype");
    if (p.act < FA_ACT_NONE || p.act > FA_ACT_SILU) return fail(w, FA_ERR_ARG, "unknown activation");
    if (p.n >= kMaxSize || p.positions >= kMaxSize) return fail(w, FA_ERR_RANGE, "a size of 2^31 or more");
    if (p.channels < 1 || p.channels > FA_NORM_MAX_CHANNELS) return fail(w, FA_ERR_RANGE, "channels out of range");
    if (p.groups < 1 || p.channels % p.groups) return fail(w, FA_ERR_RANGE, "channels is not a multiple of groups");
    return FA_OK;
}

// Positions ld apart, samples step apart (0: one after the other).  A stride out of range stays so.
uint64_t sample_step(uint64_t positions, uint64_t ld, uint64_t step) {
    return step ? step : ld >> 40 ? ld : std::min<unsigned __int128>(static_cast<unsigned __int128>(positions) * ld, ~0ull);
}

template <typename Args>
Grid norm_grid(const Args& p, const void* t, uint64_t ld, uint64_t step) {
    return Grid(t, p.channels, size_of(p.dtype), {{p.n, sample_step(p.positions, ld, step)}, {p.positions, ld}});
}

template <typename Args>
fa::NormTensor norm_tensor(const Args& p, const void* t, uint64_t ld, uint64_t step) {
    return {t, p.positions > 1 ? ld : 0, p.n > 1 ? sample_step(p.positions, ld, step) : 0};
}

template <typename Args>
void norm_sizes(fa::NormArgs& a, const Args& p, unsigned int* err) {
    a.n = static_cast<uint32_t>(p.n);
    a.positions = static_cast<uint32_t>(p.positions);
    a.channels = static_cast<uint32_t>(p.channels);
    a.groups = static_cast<uint32_t>(p.groups);
    a.dtype = code_of(p.dtype);
    a.param_dtype = code_of(p.dtype_param);
    a.act = p.act;
    a.err = err;
    a.counters = err + kNormCounters;
    a.gamma = p.gamma;
    a.beta = p.beta;
}

fa_status norm_impl(fa_work* w, const fa_group_norm_args& p, cudaStream_t s) {
    fa_status r = check_norm(w, p);
    if (r != FA_OK) return r;
    if (!(p.eps >= 0.0) || !std::isfinite(p.eps)) return fail(w, FA_ERR_ARG, "eps is negative or not finite");
    if (p.n == 0 || p.positions == 0) return FA_OK;
    const uint64_t stats = p.n * p.groups, C = p.channels, sp = size_of(p.dtype_param);
    const Grid x = norm_grid(p, p.x, p.ldx, p.step_x), y = norm_grid(p, p.y, p.ldy, p.step_y);
    r = check_grid(w, x, "x");
    if (r == FA_OK) r = check_out(w, y, "y");
    if (r == FA_OK && p.gamma) r = check_mat(w, p.gamma, 1, C, C, p.dtype_param, "gamma");
    if (r == FA_OK && p.beta) r = check_mat(w, p.beta, 1, C, C, p.dtype_param, "beta");
    if (r == FA_OK && p.mean) r = check_mat(w, p.mean, 1, stats, stats, FA_F32, "mean");
    if (r == FA_OK && p.rstd) r = check_mat(w, p.rstd, 1, stats, stats, FA_F32, "rstd");
    if (r != FA_OK) return r;
    const Extent out[] = {y.extent(), {p.mean, 1, stats, stats, 4}, {p.rstd, 1, stats, stats, 4}};
    const Extent in[] = {x.extent(), {p.gamma, 1, C, C, sp}, {p.beta, 1, C, C, sp}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j)
            if (!(i == 0 && j == 0 && x.same(y)) && overlap(out[i], in[j]))
                return fail(w, FA_ERR_ARG, "an output overlaps another tensor of the call");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(w, FA_ERR_ARG, "an output overlaps another tensor of the call");
    }
    fa::NormArgs a{};
    norm_sizes(a, p, w->err_dev);
    a.x = norm_tensor(p, p.x, p.ldx, p.step_x);
    a.out = norm_tensor(p, p.y, p.ldy, p.step_y);
    a.mean_out = p.mean;
    a.rstd_out = p.rstd;
    a.eps = static_cast<float>(p.eps);
    const uint32_t sms = static_cast<uint32_t>(w->tc.sms);
    const bool one = fa::plan_norm_one(a, false, sms);
    if (!one) fa::plan_norm(a, false, sms);
    const bool cap = capturing(s);
    Carve need{nullptr}, c{nullptr};
    const auto carve = [&](Carve& from) {
        a.stat = static_cast<float4*>(from.take(stats * a.chunks * sizeof(float4)));
    };
    carve(need);
    r = ensure_ws(w, need.used, cap);
    if (r == FA_OK) r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    c.base = w->ws;
    carve(c);
    ChainOut chain(w, s, cap);
    unsigned launches = one;
    const cudaError_t e = one ? fa::launch_norm_one(a, false, s) : fa::launch_norm(a, s, &launches);
    w->stats.kernel_launches += launches;
    return chain.end(e == cudaSuccess ? FA_OK : cuda_fail(w, e, "group norm"));
}

fa_status norm_backward_impl(fa_work* w, const fa_group_norm_backward_args& p, cudaStream_t s) {
    fa_status r = check_norm(w, p);
    if (r != FA_OK) return r;
    const uint64_t stats = p.n * p.groups, C = p.channels, sp = size_of(p.dtype_param);
    const bool any = p.n && p.positions;
    const Grid x = norm_grid(p, any ? p.x : nullptr, p.ldx, p.step_x), d = norm_grid(p, any ? p.dout : nullptr, p.ldd, p.step_d),
               dx = norm_grid(p, any ? p.dx : nullptr, p.lddx, p.step_dx);
    if (any) {
        r = check_grid(w, x, "x");
        if (r == FA_OK) r = check_grid(w, d, "dout");
        if (r == FA_OK) r = check_out(w, dx, "dx");
        if (r == FA_OK && p.gamma) r = check_mat(w, p.gamma, 1, C, C, p.dtype_param, "gamma");
        if (r == FA_OK && p.beta) r = check_mat(w, p.beta, 1, C, C, p.dtype_param, "beta");
        if (r == FA_OK) r = check_mat(w, p.mean, 1, stats, stats, FA_F32, "mean");
        if (r == FA_OK) r = check_mat(w, p.rstd, 1, stats, stats, FA_F32, "rstd");
    }
    if (r == FA_OK && p.d_gamma) r = check_mat(w, p.d_gamma, 1, C, C, p.dtype_param, "d_gamma");
    if (r == FA_OK && p.d_beta) r = check_mat(w, p.d_beta, 1, C, C, p.dtype_param, "d_beta");
    if (r != FA_OK) return r;
    const Extent out[] = {dx.extent(), {p.d_gamma, 1, C, C, sp}, {p.d_beta, 1, C, C, sp}};
    const Extent in[] = {x.extent(), d.extent(), {p.gamma, 1, C, C, sp}, {p.beta, 1, C, C, sp},
                         {any ? p.mean : nullptr, 1, stats, stats, 4}, {any ? p.rstd : nullptr, 1, stats, stats, 4}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 6; ++j)
            if (!(i == 0 && ((j == 0 && dx.same(x)) || (j == 1 && dx.same(d)))) && overlap(out[i], in[j]))
                return fail(w, FA_ERR_ARG, "an output overlaps another tensor of the call");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(w, FA_ERR_ARG, "an output overlaps another tensor of the call");
    }
    if (!any && !p.d_gamma && !p.d_beta) return FA_OK;
    fa::NormArgs a{};
    norm_sizes(a, p, w->err_dev);
    a.x = norm_tensor(p, p.x, p.ldx, p.step_x);
    a.dout = norm_tensor(p, p.dout, p.ldd, p.step_d);
    a.out = norm_tensor(p, p.dx, p.lddx, p.step_dx);
    a.mean = p.mean;
    a.rstd = p.rstd;
    a.d_gamma = p.d_gamma;
    a.d_beta = p.d_beta;
    const bool cap = capturing(s), params = p.d_gamma || p.d_beta;
    const uint32_t sms = static_cast<uint32_t>(w->tc.sms);
    bool one = false;
    uint32_t rows = 0;                   // of the parameters' partial sums
    Carve need{nullptr}, c{nullptr};
    const auto carve = [&](Carve& from) {
        a.part = static_cast<float2*>(from.take(stats * a.chunks * sizeof(float2)));
        a.cpart = params ? static_cast<float2*>(from.take(rows * C * sizeof(float2))) : nullptr;
    };
    if (any) {
        one = fa::plan_norm_one(a, true, sms);
        if (!one) fa::plan_norm(a, true, sms);
        rows = static_cast<uint32_t>(one ? a.across * a.chunks : fa::norm_rows(a) * a.chunks);
        carve(need);
    }
    r = ensure_ws(w, need.used, cap);
    if (r == FA_OK) r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    c.base = w->ws;
    if (any) carve(c);
    ChainOut chain(w, s, cap);
    unsigned launches = one;
    cudaError_t e = !any ? cudaSuccess : one ? fa::launch_norm_one(a, true, s) : fa::launch_norm_backward(a, s, &launches);
    if (e == cudaSuccess && params) {
        e = fa::launch_norm_param(a, rows, s);
        ++launches;
    }
    w->stats.kernel_launches += launches;
    return chain.end(e == cudaSuccess ? FA_OK : cuda_fail(w, e, "group norm gradient"));
}

}  // namespace

extern "C" {

fa_status fa_rotary_turns(uint32_t rotary_dim, double base, int32_t scaling, double factor, double context, double low,
                          double high, uint64_t* turns) {
    if (!turns || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > FA_ROTARY_MAX_DIM) return FA_ERR_ARG;
    if (!(base >= 1.0) || !std::isfinite(base)) return FA_ERR_ARG;
    if (scaling < FA_ROTARY_PLAIN || scaling > FA_ROTARY_BANDED) return FA_ERR_ARG;
    if (scaling != FA_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return FA_ERR_ARG;
    if (scaling == FA_ROTARY_BANDED && (!(context > 0.0) || !std::isfinite(context) || !(low >= 0.0) || !(high > low) || !std::isfinite(high)))
        return FA_ERR_ARG;
    constexpr double kTwoPi = 6.283185307179586476925;
    const double r = rotary_dim;
    if (scaling == FA_ROTARY_BASE && rotary_dim > 2) base *= std::pow(factor, r / (r - 2.0));
    if (!std::isfinite(base)) return FA_ERR_ARG;
    for (uint32_t i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        if (scaling == FA_ROTARY_LINEAR) f /= factor;
        if (scaling == FA_ROTARY_BANDED) {
            const double keep = std::min(1.0, std::max(0.0, (context * f / kTwoPi - low) / (high - low)));
            f *= keep + (1.0 - keep) / factor;
        }
        turns[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / kTwoPi, 64)));     // below 0.16 of 2^64
    }
    return FA_OK;
}

fa_status fa_rotary(fa_work* w, const fa_rotary_args* args, void* stream) {
    return enter("fa_rotary", w, args,
                 [&](const fa_rotary_args& p) { return rotary_impl(w, p, static_cast<cudaStream_t>(stream)); });
}

fa_status fa_group_norm(fa_work* w, const fa_group_norm_args* args, void* stream) {
    return enter("fa_group_norm", w, args,
                 [&](const fa_group_norm_args& p) { return norm_impl(w, p, static_cast<cudaStream_t>(stream)); });
}

fa_status fa_group_norm_backward(fa_work* w, const fa_group_norm_backward_args* args, void* stream) {
    return enter("fa_group_norm_backward", w, args, [&](const fa_group_norm_backward_args& p) {
        return norm_backward_impl(w, p, static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
