// Orthogonalised weight steps (declared in include/fedavg.h): argument checks, the order of the
// Newton-Schulz products, their scales, workspace, launches.
#include "strided.hpp"

namespace {

// The largest |a x + b x^3 + c x^5| for x from 0 to `most`.
double most_of(double a, double b, double c, double most) {
    const auto f = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
    double top = f(most);
    const auto at = [&](double y) {              // y = x^2 of an extremum
        if (y > 0.0 && y < most * most) top = std::max(top, f(std::sqrt(y)));
    };
    if (c != 0.0) {
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        at(-a / (3.0 * b));
    }
    return top;
}

// The power of two by which a matrix whose elements are below `bound` is held in fp16: below 2^15,
// with a factor of two to spare.
int shift_of(double bound) { return static_cast<int>(std::floor(std::log2(30000.0 / std::max(bound, 1e-6)))); }

// A matrix of the iteration: where it is, and its scale.
struct Held {
    const fa::OrthoBuf* buf = nullptr;
    double bound = 0.0;
    int shift = 0;
    void set(const fa::OrthoBuf* b, double top) {
        buf = b;
        bound = top;
        shift = shift_of(top);
    }
};

struct Sizes {
    uint32_t rows, cols, m, n;       // m: the short side
    bool wide;
};

constexpr double kMostSingular = 4.0;
constexpr int kSquares = 7;          // m x m matrices of the longest segment

// The steps in segments: of one, which are the iteration as it stands, or (joined) of up to three.
// Within a longer one everything is a polynomial in A = X X^T: with P_j = b A_j + c A_j^2, the product of
// the (a + P_j) is kept as q + Q, A_{j+1} = (a + P_j)^2 A_j, and X is read by two products in all instead
// of two per step.  An error in A grows with the square of what X's own does (12 per step), so after
// three steps A is formed anew: simulated in fp64 with fp16 pairs, 5 steps in one segment are off by up to
// 2.7e-5 on an update with a few strong directions, 3 + 2 by 1.1e-6, 1 + 1 + 1 + 1 + 1 by 1.4e-6.
std::vector<uint32_t> segments(uint32_t steps, bool joined) {
    const uint32_t parts = joined ? (steps + 2) / 3 : steps;
    std::vector<uint32_t> s;
    for (uint32_t left = steps, n = parts; n > 0; --n) {
        s.push_back((left + n - 1) / n);
        left -= s.back();
    }
    return s;
}

struct Run {
    Sizes z;
    uint32_t chunk;
    bool bf16;                       // of the result
    double a, b, c;
    fa::OrthoBuf x[2], sq[kSquares];
    std::vector<fa::OrthoProduct> list;

    void product(const Held& P, bool pk, const Held& Q, bool qk, uint32_t k, const Held& out, bool symmetric, double c1,
                      const Held* e1, double c2, const Held* e2, double c3) {
        fa::OrthoProduct p{};
        p.P = P.buf;
        p.Q = Q.buf;
        p.out = out.buf;
        p.e1 = e1 ? e1->buf : nullptr;
        p.e2 = e2 ? e2->buf : nullptr;
        p.p_kmajor = pk;
        p.q_kmajor = qk;
        p.symmetric = symmetric;
        p.k = k;
        p.chunk = chunk;
        // from true values to held ones
        p.c1 = static_cast<float>(std::ldexp(c1, out.shift - P.shift - Q.shift));
        p.c2 = e1 ? static_cast<float>(std::ldexp(c2, out.shift - e1->shift)) : 0.0f;
        p.c3 = e2 ? static_cast<float>(std::ldexp(c3, out.shift - e2->shift)) : 0.0f;
        list.push_back(p);
    }

    // The whole list of products; where X is then.
    Held products(const std::vector<uint32_t>& parts, const std::vector<double>& top) {
        list.clear();
        Held X;
        X.set(&x[0], 1.0);
        uint32_t steps = 0;
        for (uint32_t n : parts) {
            steps += n;
            segment(n, X, top[steps]);
        }
        return X;
    }

    // `steps` steps from X, which is replaced; `next` bounds its singular values then.
    void segment(uint32_t steps, Held& X, double next) {
        int used = 0;
        const auto square = [&](double bound) {
            Held h;
            h.set(&sq[used++ % kSquares], bound);
            return h;
        };
        Held A = square(X.bound * X.bound), Q, P;
        product(X, z.wide, X, z.wide, z.n, A, true, 1.0, nullptr, 0, nullptr, 0);
        double q = 1.0, top = X.bound;
        for (uint32_t j = 0; j < steps; ++j) {
            const double vertex = c != 0.0 ? -b / (2.0 * c) : -1.0, most = top * top;
            double bound = std::fabs(most * (b + c * most));
            if (vertex > 0.0 && vertex < most) bound = std::max(bound, std::fabs(vertex * (b + c * vertex)));
            P = square(bound);
            product(A, true, A, true, z.m, P, true, c, &A, b, nullptr, 0);
            if (j == 0) {
                Q = P;
                q = a;
            } else {
                Held N = square(P.bound * Q.bound + std::fabs(a) * Q.bound + std::fabs(q) * P.bound);
                product(P, true, Q, true, z.m, N, true, 1.0, &Q, a, &P, q);
                Q = N;
                q *= a;
            }
            if (j + 1 < steps) {
                Held R = square(A.bound * (std::fabs(a) + P.bound));
                product(A, true, P, true, z.m, R, true, 1.0, &A, a, nullptr, 0);
                top = most_of(a, b, c, top);
                Held N = square(top * top);
                product(R, true, P, true, z.m, N, true, 1.0, &R, a, nullptr, 0);
                A = N;
            }
        }
        Held N;
        N.set(X.buf == &x[0] ? &x[1] : &x[0], next);
        if (z.wide)
            product(Q, true, X, false, z.m, N, false, 1.0, &X, q, nullptr, 0);
        else
            product(X, true, Q, true, z.m, N, false, 1.0, &X, q, nullptr, 0);
        X = N;
    }
};

fa_status ortho_impl(fa_work* w, const fa_orthogonalise_args& p, cudaStream_t s) {
    if (p.flags & ~FA_ORTHO_NESTEROV) return fail(w, FA_ERR_ARG, "unknown flag");
    if (!dtype_ok(p.dtype_in) || !dtype_ok(p.dtype_out)) return fail(w, FA_ERR_DTYPE, "dtype");
    for (double v : {p.mu, p.alpha, p.beta, p.a, p.b, p.c})
        if (!std::isfinite(v) || std::fabs(v) > 1e30) return fail(w, FA_ERR_ARG, "a factor is not finite, or above 1e30");
    if (!(p.eps >= 1e-30) || !(p.eps <= 1e30)) return fail(w, FA_ERR_ARG, "eps is not from 1e-30 to 1e30");
    if (p.steps > FA_ORTHO_MAX_STEPS) return fail(w, FA_ERR_RANGE, "more than 32 steps");
    if (p.count >= kMaxSize || p.rows >= 1u << 24 || p.cols >= 1u << 24 || p.rows * p.cols > 1ull << 32 ||
        std::min(p.rows, p.cols) > 1u << 15)
        return fail(w, FA_ERR_RANGE, "a size out of range");
    std::vector<double> top(p.steps + 1, 1.0);
    for (uint32_t i = 0; i < p.steps; ++i) {
        top[i + 1] = most_of(p.a, p.b, p.c, top[i]);
        if (!(top[i + 1] <= kMostSingular)) return fail(w, FA_ERR_RANGE, "coefficients by which singular values may grow beyond 4");
    }
    if (p.count == 0 || p.rows == 0 || p.cols == 0) return FA_OK;
    const void* res = p.beta != 0.0 ? p.residual : nullptr;
    const auto step = [&](uint64_t ld, uint64_t given) { return given ? given : ld >> 40 ? ld : p.rows * ld; };
    const auto grid = [&](const void* t, int32_t dt, uint64_t ld, uint64_t given) {
        return Grid(t, p.cols, size_of(dt), {{p.count, step(ld, given)}, {p.rows, ld}});
    };
    const Grid u = grid(p.update, p.dtype_in, p.ldu, p.step_u), m = grid(p.momentum, FA_F32, p.ldm, p.step_m),
               mo = grid(p.momentum_out, FA_F32, p.ldmo, p.step_mo), rs = grid(res, p.dtype_out, p.ldr, p.step_r),
               o = grid(p.out, p.dtype_out, p.ldo, p.step_o);
    fa_status r = check_grid(w, u, "update");
    if (r == FA_OK && p.momentum) r = check_grid(w, m, "momentum");
    if (r == FA_OK && p.momentum_out) r = check_out(w, mo, "momentum_out");
    if (r == FA_OK && res) r = check_grid(w, rs, "residual");
    if (r == FA_OK) r = check_out(w, o, "out");
    if (r != FA_OK) return r;
    const Extent eu = u.extent(), em = m.extent(), emo = mo.extent(), er = rs.extent(), eo = o.extent();
    if (overlap(emo, eu) || overlap(emo, er) || overlap(emo, eo) || (!mo.same(m) && overlap(emo, em)) || overlap(eo, em) ||
        (!o.same(rs) && overlap(eo, er)) || (!o.same(u) && overlap(eo, eu)))
        return fail(w, FA_ERR_ARG, "an output overlaps another tensor of the call");

    const uint32_t rows = static_cast<uint32_t>(p.rows), cols = static_cast<uint32_t>(p.cols);
    const Sizes z{rows, cols, std::min(rows, cols), std::max(rows, cols), rows <= cols};
    const bool small = fa::ortho_small_fits(p.count, rows, cols);
    Run run{};
    run.z = z;
    run.bf16 = p.dtype_out == FA_BF16;
    // blocks that the tensor cores' truncating sum takes before it is emptied.  bf16 results round more than
    // 16 cost; fp32 ones lose half a digit at small sizes with 4, where emptying is cheap (1024 x 1024 190
    // us, with 4 187), 4096 x 4096 takes 2.86 ms with 4 and 2.76 with 16.
    run.chunk = run.bf16 ? 16 : z.m <= 512 ? 1 : z.m <= 1024 ? 2 : 4;
    run.a = p.a;
    run.b = p.b;
    run.c = p.c;
    for (fa::OrthoBuf& b : run.x) {
        b.rows = rows;
        b.cols = cols;
        b.ld = (cols + 7ull) / 8 * 8;
    }
    for (fa::OrthoBuf& b : run.sq) {
        b.rows = b.cols = z.m;
        b.ld = (z.m + 7ull) / 8 * 8;
    }
    // Towards a bf16 result steps are joined where that takes less time, by the products' cost model: 11008 x
    // 4096 4.17 ms joined, 5.92 as they stand; 700 x 4100 246 and 277 us, 900 x 1120 220 and 184.  (Where both are
    // near it may err: 4 of 1000 x 1300 are joined, 488 us, and take 471 as they stand.)
    // (fp32 results were 2 to 5 times further off when joined.)
    std::vector<uint32_t> parts = segments(p.steps, false);
    if (!small && run.bf16) {
        const auto cost = [&](const std::vector<uint32_t>& of) {
            run.products(of, top);
            return fa::ortho_cost(run.list.data(), static_cast<uint32_t>(run.list.size()),
                                  static_cast<uint32_t>(std::min<uint64_t>(p.count, 1024)), static_cast<uint32_t>(w->tc.sms));
        };
        const std::vector<uint32_t> joined = segments(p.steps, true);
        if (joined.size() < parts.size() && cost(joined) < cost(parts)) parts = joined;
    }
    uint32_t longest = 0;
    for (uint32_t v : parts) longest = std::max(longest, v);
    // A segment of one holds A and P, longer ones up to seven squares.
    const int squares = longest == 0 ? 0 : longest == 1 ? 2 : kSquares;
    const uint64_t ldx = run.x[0].ld, ldm = run.sq[0].ld;
    const uint64_t each = 4 * ((longest ? 2 : 1) * rows * ldx + squares * z.m * ldm);
    // Matrices at one time: what fits 1 GiB of workspace, one at least.
    const uint32_t group = static_cast<uint32_t>(
        small ? std::min<uint64_t>(p.count, 1u << 20) : std::min<uint64_t>({p.count, std::max<uint64_t>(1, (1ull << 30) / each), 32768}));
    const bool cap = capturing(s);
    float3* part = nullptr;
    uint32_t* done = nullptr;
    const uint32_t blocks = fa::ortho_blocks(group, rows, cols, static_cast<uint32_t>(w->tc.sms));
    const auto carve = [&](Carve& c) {
        for (int i = 0; i < (longest ? 2 : 1); ++i) {
            run.x[i].p = static_cast<uint16_t*>(c.take(4ull * group * rows * ldx));
        }
        for (int i = 0; i < squares; ++i) {
            run.sq[i].p = static_cast<uint16_t*>(c.take(4ull * group * z.m * ldm));
        }
        part = static_cast<float3*>(c.take(sizeof(float3) * group * blocks));
        done = static_cast<uint32_t*>(c.take(sizeof(uint32_t) * group));
    };
    Carve need{nullptr}, c{nullptr};
    if (!small) {
        carve(need);
        FW_CUDA(w, fa::prepare_ortho(&w->ortho));
    }
    r = ensure_ws(w, need.used, cap);
    if (r == FA_OK) r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    if (!small) {
        c.base = w->ws;
        carve(c);
        for (int i = 0; i < (longest ? 2 : 1); ++i) FW_CUDA(w, fa::map_ortho(&run.x[i], group));
        for (int i = 0; i < squares; ++i) FW_CUDA(w, fa::map_ortho(&run.sq[i], group));
    }
    fa::OrthoEnds e{};
    const auto mat = [&](const void* t, int32_t dt, uint64_t ld, uint64_t given) {
        return fa::OrthoMat{t, rows > 1 ? ld : 0, p.count > 1 ? step(ld, given) : 0, code_of(dt)};
    };
    e.update = mat(p.update, p.dtype_in, p.ldu, p.step_u);
    e.momentum = mat(p.momentum, FA_F32, p.ldm, p.step_m);
    e.momentum_out = mat(p.momentum_out, FA_F32, p.ldmo, p.step_mo);
    e.residual = mat(res, p.dtype_out, p.ldr, p.step_r);
    e.out = mat(p.out, p.dtype_out, p.ldo, p.step_o);
    e.rows = rows;
    e.cols = cols;
    e.blocks = blocks;
    e.part = part;
    e.done = done;
    e.ld = ldx;
    e.eps = p.eps;
    e.mu = static_cast<float>(p.mu);
    e.beta = static_cast<float>(p.beta);
    e.nesterov = p.flags & FA_ORTHO_NESTEROV;
    ChainOut chain(w, s, cap);
    for (uint64_t first = 0; first < p.count && r == FA_OK; first += group) {
        e.items = static_cast<uint32_t>(std::min<uint64_t>(group, p.count - first));
        if (small) {
            const fa::OrthoSmall steps{p.steps, p.dtype_out == FA_BF16 ? (p.steps + 2) / 3 : p.steps, static_cast<float>(p.a), static_cast<float>(p.b), static_cast<float>(p.c)};
            e.alpha = static_cast<float>(p.alpha);
            r = launched(w, fa::launch_ortho_small(e, steps, s), "weight step");
        } else {
            e.x = run.x[0].p;
            e.shift = shift_of(1.0);
            r = launched(w, fa::launch_ortho_norm(e, s), "update's norm");
            if (r == FA_OK) r = launched(w, fa::launch_ortho_scale(e, s), "update's scale");
            const Held X = run.products(parts, top);
            uint32_t counted = 0;
            const size_t all = run.list.size();
            for (size_t at = 0; r == FA_OK && at < all; at += fa::kOrthoOps) {
                const cudaError_t ce = fa::launch_ortho_products(
                    run.list.data() + at, static_cast<uint32_t>(std::min<size_t>(fa::kOrthoOps, all - at)), e.items, done, &counted,
                    w->ortho, w->err_dev, (w->flags & FA_TEST_WAIT_EXPIRES) != 0, s, &w->stats.kernel_launches);
                if (ce != cudaSuccess) r = cuda_fail(w, ce, "orthogonalisation");
            }
            e.x = X.buf->p;
            e.alpha = static_cast<float>(std::ldexp(p.alpha, -X.shift));
            if (r == FA_OK) r = launched(w, fa::launch_ortho_finish(e, s), "weight step");
        }
        for (fa::OrthoMat* t : {&e.update, &e.momentum, &e.momentum_out, &e.residual, &e.out})
            if (t->p) t->p = static_cast<const uint8_t*>(t->p) + group * t->step * (t->dtype ? 2 : 4);
    }
    return chain.end(r);
}

}  // namespace

extern "C" fa_status fa_orthogonalise(fa_work* w, const fa_orthogonalise_args* args, void* stream) {
    return enter("fa_orthogonalise", w, args,
                 [&](const fa_orthogonalise_args& p) { return ortho_impl(w, p, static_cast<cudaStream_t>(stream)); });
}
