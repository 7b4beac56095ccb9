// Work handles and the products and distillation of server-side training (declared in
// include/fedavg.h): the handle's life, argument checks, launches.
#include "work.hpp"

#include "distill.cuh"

namespace {

// ----------------------------------------------------------------- products
// Too little work to fill a tensor-core tile: a thread or warp per output, where no sum is longer
// than `most`.  In a CUDA graph 40 x 40 x 40 takes 1.9 us so, 4.7 (bf16) and 9.2 (fp32) on the
// tensor cores; 256 x 256 x 8, the limit of the work, 4.3 and 4.4; 4 x 10 x 256 bf16 2.5 and
// 3.1, but 8 x 8 x 1000 bf16 6.9 and 4.0, fp32 6.7 and 8.2.
bool use_tiny(uint64_t m, uint64_t n, uint64_t k, uint64_t longest, uint64_t most) {
    return k == 0 || (m * n * k <= (1ull << 16) && longest <= most);
}

bool tma_ready(const fa::ProdOperand& o) {
    return o.dtype == 1 && reinterpret_cast<uintptr_t>(o.p) % 16 == 0 && o.ld % 8 == 0 && o.ld < (1ull << 36);
}

// The operand as the tensor-core kernel reads it: as it is, or to be laid out in the workspace
// by `jobs`.  x: its extent beside the summed one.
fa::TcOperand lay_out(const fa::ProdOperand& o, uint32_t x, uint32_t k, Carve* c, fa::SplitJob* jobs, int* n) {
    if (tma_ready(o)) return {o.p, o.ld, 0, 1, o.kmajor};
    const uint32_t rows = o.kmajor ? x : k, cols = o.kmajor ? k : x, planes = o.dtype ? 1 : 3;
    const uint64_t ldd = (cols + 7ull) / 8 * 8;
    void* dst = c->take(ldd * rows * planes * 2);
    jobs[(*n)++] = {o.p, o.ld, o.dtype, rows, cols, planes, dst, ldd};
    return {dst, ldd, ldd * rows, planes, o.kmajor};
}

// Tile configuration and split of the summed index: the least time by a model in
// microseconds, fitted to sweeps of every configuration over 35 shapes on GB300.  A launch
// takes 4, a tile 1 to 2 beside its blocks of 64 terms, the exchange of a split 1.5.  A block
// takes the largest of its latency, its MMA time, and its operand bytes at the 112 GB/s that
// L2 gives each SM when all of them load.  The choice was within 15 % of the best configuration
// in 34 of the 35 shapes.
void choose(fa::TcProduct* p, const fa::TcShape& shape) {
    const auto up = [](uint64_t a, uint64_t b) { return (a + b - 1) / b; };
    const uint64_t kb = up(p->k, 64), n_sm = static_cast<uint64_t>(shape.sms);
    const uint32_t planes = p->a.planes + p->b.planes, products = planes == 6 ? 6 : planes == 4 ? 3 : 1;
    p->drain = p->e.out_dtype == 0;
    double best = 1e300;
    const auto consider = [&](int cfg, uint64_t tiles, uint32_t ctas, double kbytes, double latency, double mma,
                              double per_tile, uint32_t splits) {
        const uint64_t room = std::max(1, shape.split_ctas[splits]);      // larger clusters leave SMs of a GPC unused
        const uint64_t all = tiles * splits * ctas, active = std::min(all, room);
        const double load = kbytes * 1.024 * planes / 2 / 112 * static_cast<double>(active) / static_cast<double>(n_sm);
        const double block = std::max(std::max(latency, load), mma * products);
        // a split's clusters do one tile each: a further wave starts anew
        const double start = splits > 1 ? 4.0 : 0.0, waves = static_cast<double>(up(all, room));
        const double cost = waves * (static_cast<double>(up(kb, splits)) * block + per_tile + start) - start +
                            (splits > 1 ? 1.5 : 0.0);
        if (cost < best) {
            best = cost;
            p->cfg = cfg;
            p->splits = splits;
        }
    };
    const uint64_t m128 = up(p->m, 128), m256 = up(p->m, 256), n64 = up(p->n, 64), n128 = up(p->n, 128), n256 = up(p->n, 256);
    // few tokens: in the MMA's columns
    if (p->m <= 64 && (p->a.kmajor || p->m > 32)) {
        const int cfg = p->m <= 16 ? fa::kTcSwap16 : p->m <= 32 ? fa::kTcSwap32 : fa::kTcSwap64;
        const double kbytes = p->m <= 16 ? 18 : p->m <= 32 ? 20 : 24;
        for (uint32_t s = 1; s <= 8 && kb >= s; ++s) consider(cfg, n128, 1, kbytes, 0.15, 0.13, p->m > 32 ? 1.5 : 1.0, s);
        if (p->m <= 32) return;
    }
    // planes need TMEM and shared memory beside 256 columns
    if (planes == 2) consider(fa::kTcPair256, m256 * n256, 2, 32, 0.30, 0.30, 1.8, 1);
    consider(fa::kTcPair128, m256 * n128, 2, 24, 0.165, 0.16, 1.6, 1);
    for (uint32_t s = 1; s <= 8 && kb >= s; ++s) {
        consider(fa::kTc128, m128 * n128, 1, 32, 0.185, 0.165, 1.6, s);
        consider(fa::kTc64, m128 * n64, 1, 24, 0.16, 0.13, 1.5, s);
    }
}

// Few rows that the tensor cores could only take after a pass over the weights (fp32 ones into
// three planes, 16 bytes moved per weight instead of 4; bf16 ones of an odd stride into an
// aligned copy): read as they are on the FP32 units.  Against 4096 x 4096 fp32 weights: 16
// rows 23.5 us (tensor cores with their pass 46), 32 rows 46 (48), 64 rows 90 (50).  Against
// 4097 x 4095 bf16 ones: stored [n, k] 1 row 8.1 us (20.5), 8 rows 16.3 (20.7); stored [k, n]
// 1 row 13.8 (20.9), 4 rows 17.4 (21.1), 8 rows 25.8 (21.3).
bool use_thin(const fa::ProdArgs& q) {
    if (!q.a.kmajor || q.a.dtype != q.b.dtype) return false;
    // With b stored [k, n] a warp walks down its share of the rows, eight loads in flight, for
    // every eight rows of a: 1.3 ns per row of b, or b's bytes at some 3.3 TB/s where that is
    // more.  The tensor cores with their pass over fp32 weights (16 bytes moved for each) take
    // some 9 us, 1.2 ns per row, and those bytes at 6.5 TB/s: measured 10 rows by 21360 x 88
    // 56.5 us (thin) and 40.3, 8 rows by 20000 x 2000 66.5 and 122.9, 16 by 4096 x 4096 28.8
    // and 50.7.
    if (!q.b.kmajor && q.b.dtype == 0) {
        const double groups = (q.m + 7) / 8, k = q.k, kn = static_cast<double>(q.k) * q.n;
        if (groups * std::max(0.0013 * k, kn * 4 / 3.3e6) > 9 + 0.0012 * k + kn * 16 / 6.5e6) return false;
    }
    return q.b.dtype == 0 ? q.m <= (q.b.kmajor ? 24 : 16) : q.m <= (q.b.kmajor ? 8 : 4) && !tma_ready(q.b);
}

// A product by the kernel that suits its size.  run == false only adds up the workspace.
fa_status do_product(fa_work* w, const fa::ProdArgs& q, const fa::TcOperand* ready_a, const fa::TcOperand* ready_b, Carve* c,
                     bool run, cudaStream_t s, const char* what) {
    fa::TcProduct t{};
    t.m = q.m;
    t.n = q.n;
    t.k = q.k;
    t.e = q.e;
    if (!ready_a && !ready_b && use_thin(q)) return run ? launched(w, fa::launch_product_thin(q, s), what) : FA_OK;
    fa::SplitJob jobs[2];
    int n = 0;
    t.a = ready_a ? *ready_a : lay_out(q.a, q.m, q.k, c, jobs, &n);
    t.b = ready_b ? *ready_b : lay_out(q.b, q.n, q.k, c, jobs, &n);
    if (!run) return FA_OK;
    if (n > 0) {
        const fa_status r = launched(w, fa::launch_split(jobs, n, s), "operand layout");
        if (r != FA_OK) return r;
    }
    choose(&t, w->tc);
    return launched(w, fa::launch_product_tc(t, w->tc, w->err_dev, (w->flags & FA_TEST_WAIT_EXPIRES) != 0, s), what);
}

fa_status product_impl(fa_work* w, const fa_product_args& p, cudaStream_t s) {
    if (p.flags & ~(FA_TRANS_A | FA_TRANS_B)) return fail(w, FA_ERR_ARG, "unknown flag");
    if (!dtype_ok(p.dtype_in) || !dtype_ok(p.dtype_out)) return fail(w, FA_ERR_DTYPE, "dtype");
    if (p.act < FA_ACT_NONE || p.act > FA_ACT_SILU) return fail(w, FA_ERR_ARG, "unknown activation");
    if (!std::isfinite(p.alpha) || !std::isfinite(p.beta)) return fail(w, FA_ERR_ARG, "alpha or beta not finite");
    if (p.m >= kMaxSize || p.n >= kMaxSize || p.k >= kMaxSize)
        return fail(w, FA_ERR_RANGE, "a size of 2^31 or more");
    if (p.m == 0 || p.n == 0) return FA_OK;
    const bool ta = p.flags & FA_TRANS_A, tb = p.flags & FA_TRANS_B;
    const uint64_t ar = ta ? p.k : p.m, aw = ta ? p.m : p.k, br = tb ? p.n : p.k, bw = tb ? p.k : p.n;
    const uint64_t si = size_of(p.dtype_in), so = size_of(p.dtype_out);
    const void* res = p.beta != 0.0 ? p.residual : nullptr;
    fa_status r = check_mat(w, p.a, ar, aw, p.lda, p.dtype_in, "a");
    if (r == FA_OK) r = check_mat(w, p.b, br, bw, p.ldb, p.dtype_in, "b");
    if (r == FA_OK) r = check_mat(w, p.out, p.m, p.n, p.ldo, p.dtype_out, "out");
    if (r == FA_OK && p.bias) r = check_mat(w, p.bias, 1, p.n, p.n, p.dtype_in, "bias");
    if (r == FA_OK && res) r = check_mat(w, res, p.m, p.n, p.ldr, p.dtype_out, "residual");
    if (r == FA_OK && p.pre) r = check_mat(w, p.pre, p.m, p.n, p.ldo, p.dtype_out, "pre");
    if (r != FA_OK) return r;
    const Extent out{p.out, p.m, p.n, p.ldo, so}, pre{p.pre, p.m, p.n, p.ldo, so}, residual{res, p.m, p.n, p.ldr, so};
    const Extent in[] = {{p.a, ar, aw, p.lda, si}, {p.b, br, bw, p.ldb, si}, {p.bias, 1, p.n, p.n, si}};
    for (const Extent& e : in)
        if (overlap(out, e) || overlap(pre, e)) return fail(w, FA_ERR_ARG, "an output overlaps a, b or bias");
    if (overlap(out, pre)) return fail(w, FA_ERR_ARG, "out overlaps pre");
    if (overlap(pre, residual)) return fail(w, FA_ERR_ARG, "pre overlaps residual");
    if (!(res == p.out && p.ldr == p.ldo) && overlap(out, residual))
        return fail(w, FA_ERR_ARG, "out overlaps residual without being it");
    const bool cap = capturing(s);
    fa::ProdArgs q{};
    q.m = static_cast<uint32_t>(p.m);
    q.n = static_cast<uint32_t>(p.n);
    q.k = static_cast<uint32_t>(p.k);
    q.a = {p.a, p.lda, code_of(p.dtype_in), !ta};
    q.b = {p.b, p.ldb, code_of(p.dtype_in), tb};
    q.e = {static_cast<float>(p.alpha), static_cast<float>(p.beta), p.bias, res, p.out, p.pre, p.ldr, p.ldo,
           code_of(p.dtype_in), code_of(p.dtype_out), p.act};
    // a few long sums of fp32 operands have more lanes in the thin kernel (8 x 8 x 1000: 2.3 us
    // against 6.7, 4 x 10 x 256: 1.7 against 2.4)
    const bool tiny = use_tiny(p.m, p.n, p.k, p.k, p.dtype_in == FA_F32 ? 1024 : 256) && !(p.k > 128 && tb && p.dtype_in == FA_F32 && use_thin(q));
    Carve need{nullptr};
    if (!tiny) do_product(w, q, nullptr, nullptr, &need, false, s, "product");
    r = ensure_ws(w, need.used, cap);
    if (r == FA_OK) r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    ChainOut chain(w, s, cap);
    Carve c{w->ws};
    return chain.end(tiny ? launched(w, fa::launch_product_tiny(q, s), "product")
                          : do_product(w, q, nullptr, nullptr, &c, true, s, "product"));
}

// Rows per block of the activation's gradient: the number with the least work in the last of the
// turns that four blocks per SM take, a block's start and end costing as much as some 8 rows.
// In a CUDA graph both gradients of 8192 x 1024 x 512 bf16 with gelu and bias: 48.4 us, always 32
// rows 52.5; of 2056 x 4096 x 1024 53.2 and 55; of 777 x 4096 x 256 fp32 51.8 and 55.2.
uint32_t grad_rows(uint32_t m, uint32_t n, uint32_t sms) {
    const uint64_t across = (n + 255) / 256;
    uint64_t best = ~0ull;
    uint32_t rows = 8;
    for (uint32_t r = 8; r <= 128; r += 8) {
        const uint64_t blocks = across * ((m + r - 1ull) / r), turns = (blocks + 4 * sms - 1) / (4 * sms);
        if (turns * (r + 8) < best) {
            best = turns * (r + 8);
            rows = r;
        }
    }
    return rows;
}

fa_status backward_impl(fa_work* w, const fa_product_backward_args& p, cudaStream_t s) {
    if (p.flags & ~(FA_TRANS_A | FA_TRANS_B)) return fail(w, FA_ERR_ARG, "unknown flag");
    if (!dtype_ok(p.dtype_in) || !dtype_ok(p.dtype_dout) || !dtype_ok(p.dtype_grad))
        return fail(w, FA_ERR_DTYPE, "dtype");
    if (p.act < FA_ACT_NONE || p.act > FA_ACT_SILU) return fail(w, FA_ERR_ARG, "unknown activation");
    if (!std::isfinite(p.alpha)) return fail(w, FA_ERR_ARG, "alpha not finite");
    if (p.m >= kMaxSize || p.n >= kMaxSize || p.k >= kMaxSize)
        return fail(w, FA_ERR_RANGE, "a size of 2^31 or more");
    const bool ta = p.flags & FA_TRANS_A, tb = p.flags & FA_TRANS_B;
    const bool act = p.act != FA_ACT_NONE;
    const uint64_t ar = ta ? p.k : p.m, aw = ta ? p.m : p.k, br = tb ? p.n : p.k, bw = tb ? p.k : p.n;
    const uint64_t si = size_of(p.dtype_in), sd = size_of(p.dtype_dout), sg = size_of(p.dtype_grad);
    fa_status r = check_mat(w, p.dout, p.m, p.n, p.ldd, p.dtype_dout, "dout");
    if (r == FA_OK && act) r = check_mat(w, p.pre, p.m, p.n, p.ldp, p.dtype_dout, "pre");
    if (r == FA_OK && p.d_b) r = check_mat(w, p.a, ar, aw, p.lda, p.dtype_in, "a");
    if (r == FA_OK && p.d_a) r = check_mat(w, p.b, br, bw, p.ldb, p.dtype_in, "b");
    if (r == FA_OK && p.d_a) r = check_mat(w, p.d_a, ar, aw, p.ldda, p.dtype_grad, "d_a");
    if (r == FA_OK && p.d_b) r = check_mat(w, p.d_b, br, bw, p.lddb, p.dtype_grad, "d_b");
    if (r == FA_OK && p.d_bias) r = check_mat(w, p.d_bias, 1, p.n, p.n, p.dtype_grad, "d_bias");
    if (r != FA_OK) return r;
    const Extent t[] = {{p.d_a, ar, aw, p.ldda, sg}, {p.d_b, br, bw, p.lddb, sg}, {p.d_bias, 1, p.n, p.n, sg},
                        {p.d_b ? p.a : nullptr, ar, aw, p.lda, si}, {p.d_a ? p.b : nullptr, br, bw, p.ldb, si},
                        {p.dout, p.m, p.n, p.ldd, sd}, {act ? p.pre : nullptr, p.m, p.n, p.ldp, sd}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (overlap(t[i], t[j])) return fail(w, FA_ERR_ARG, "a gradient overlaps another tensor of the call");
    const bool want_a = p.d_a && p.m && p.k, want_b = p.d_b && p.n && p.k, want_bias = p.d_bias && p.n;
    if (!want_a && !want_b && !want_bias) return FA_OK;
    const uint32_t m = static_cast<uint32_t>(p.m), n = static_cast<uint32_t>(p.n), k = static_cast<uint32_t>(p.k);
    const uint32_t rows = grad_rows(m, n, static_cast<uint32_t>(w->tc.sms)), blocks = (m + rows - 1) / rows;
    const int it = code_of(p.dtype_in), dt = code_of(p.dtype_dout), gt = code_of(p.dtype_grad);
    // dZ is dout itself, or is written to the workspace: in fp32 for the tiny kernel and for few
    // fp32 rows, else as bf16 planes.  few: the gradient of a is for the thin kernels (see
    // use_thin), which take dZ as it lies; both gradients of 1 x 1024 x 4096 fp32 then take 19.0
    // us (28.5 on the tensor cores), of 8 x 4096 x 1024 26.9 (30.8), of 16 x 4096 x 4096 85.0
    // (86.2), of 1 x 10387 x 9180 bf16 160 (201), of 4 x 4097 x 4095 bf16 54.6 (55.0)
    const bool tiny = use_tiny(p.m, p.n, p.k, p.m * p.n * p.k ? std::max({p.m, p.n, p.k}) : 0, 1024);
    const bool few = !tiny && (it == 0 ? p.m <= 16
                                       : gt == 1 && p.m <= 4 && want_a && (act || dt == it) &&
                                             !tma_ready({p.b, p.ldb, it, !tb}));
    const bool products = want_a || want_b;
    const fa::ProdOperand d_in{p.dout, p.ldd, dt, true};
    const bool write_dz = products && m && n && (act || (!tiny && !few && !tma_ready(d_in)));
    const int planes = tiny || (few && it == 0) ? 0 : (gt == 0 && (act || dt == 0)) ? 3 : 1;
    const uint64_t ldz = planes == 0 ? p.n : (p.n + 7) / 8 * 8;
    const bool cap = capturing(s);
    // two passes over the same steps: the first adds up the workspace
    const auto pass = [&](Carve& c, bool run) {
        void* dz = write_dz ? c.take(p.m * ldz * (planes ? 2 * planes : 4)) : nullptr;
        float* part = want_bias ? static_cast<float*>(c.take(blocks * p.n * 4)) : nullptr;
        if (run && (write_dz || want_bias) && m && n) {
            const fa::ActGradArgs g{m, n, rows, p.dout, act ? p.pre : nullptr, p.ldd, p.ldp, dt, p.act, dz, ldz, planes, part};
            r = launched(w, fa::launch_act_grad(g, s), "activation gradient");
        }
        if (run && r == FA_OK && want_bias)
            r = launched(w, fa::launch_col_sum(part, blocks, n, p.d_bias, gt, s), "bias gradient");
        const fa::ProdOperand z = write_dz ? fa::ProdOperand{dz, ldz, planes ? 1 : 0, true} : d_in;
        fa::ProdOperand z_n = z;         // x = n (sum over m); z: x = m (sum over n)
        z_n.kmajor = false;
        const uint32_t zp = write_dz && planes ? planes : 1;
        const fa::TcOperand tz{z.p, z.ld, p.m * ldz, zp, true}, tz_n{z.p, z.ld, p.m * ldz, zp, false};
        fa::ProdEpilogue e{};
        e.alpha = static_cast<float>(p.alpha);
        e.out_dtype = gt;
        const uint64_t mark = c.used;
        if (r == FA_OK && want_a) {
            const fa::ProdOperand b{p.b, p.ldb, it, !tb};      // x = k, sum over n
            e.out = p.d_a;
            e.ldo = p.ldda;
            const fa::ProdArgs q = ta ? fa::ProdArgs{k, m, n, b, z, e} : fa::ProdArgs{m, k, n, z, b, e};
            if (tiny || n == 0)
                r = run ? launched(w, fa::launch_product_tiny(q, s), "gradient of a") : FA_OK;
            else
                r = do_product(w, q, ta || few ? nullptr : &tz, ta && !few ? &tz : nullptr, &c, run, s, "gradient of a");
        }
        const uint64_t after_a = c.used;
        c.used = mark;                    // the second product's operand may take the first's place
        if (r == FA_OK && want_b) {
            const fa::ProdOperand a{p.a, p.lda, it, ta};       // x = k, sum over m
            e.out = p.d_b;
            e.ldo = p.lddb;
            const fa::ProdArgs q = tb ? fa::ProdArgs{n, k, m, z_n, a, e} : fa::ProdArgs{k, n, m, a, z_n, e};
            if (tiny || m == 0)
                r = run ? launched(w, fa::launch_product_tiny(q, s), "gradient of b") : FA_OK;
            else
                r = do_product(w, q, tb && !few ? &tz_n : nullptr, tb || few ? nullptr : &tz_n, &c, run, s, "gradient of b");
        }
        c.used = std::max(c.used, after_a);
    };
    Carve need{nullptr}, c{nullptr};
    pass(need, false);
    if (r == FA_OK) r = ensure_ws(w, need.used, cap);
    if (r == FA_OK) r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    ChainOut chain(w, s, cap);
    c.base = w->ws;
    pass(c, true);
    return chain.end(r);
}

fa_status distill_impl(fa_work* w, const fa_distill_args& p, bool grad, cudaStream_t s) {
    if (!dtype_ok(p.dtype) || !dtype_ok(p.dtype_value)) return fail(w, FA_ERR_DTYPE, "dtype");
    if (p.n_clients < 1 || p.n_clients > FA_DISTILL_MAX_CLIENTS || p.clients == nullptr)
        return fail(w, FA_ERR_ARG, "1 to 16 clients are needed");
    if (!(p.temperature >= FA_DISTILL_MIN_TEMPERATURE && p.temperature <= FA_DISTILL_MAX_TEMPERATURE))
        return fail(w, FA_ERR_ARG, "temperature out of range");
    if (p.rows >= kMaxSize || p.vocab >= kMaxSize || p.vocab == 0)
        return fail(w, FA_ERR_RANGE, "rows or vocab out of range");
    fa::DistillArgs a{};
    uint64_t entries = 0;
    double heaviest = 0.0, total = 0.0;
    for (uint32_t j = 0; j < p.n_clients; ++j) {
        const fa_distill_client& c = p.clients[j];
        if (c.topk < 1 || c.topk > FA_DISTILL_MAX_TOPK) return fail(w, FA_ERR_RANGE, "topk out of range");
        if (!std::isfinite(c.weight) || c.weight < 0.0 || c.weight > 16777216.0)
            return fail(w, FA_ERR_WEIGHT, "client weight");
        entries += c.topk;
        heaviest = std::max(heaviest, c.weight);
    }
    if (entries > FA_DISTILL_MAX_TOPK) return fail(w, FA_ERR_RANGE, "more than 2048 list places per row");
    if (p.rows == 0) return FA_OK;
    // The kernels' fp32 weights: only their ratios matter, so the largest is moved to 2^99 by a power
    // of two (exact).  Those that fall below fp32's normal numbers, 2^-225 of the largest, count as 0.
    double weight[FA_DISTILL_MAX_CLIENTS];
    const int shift = heaviest > 0.0 ? 99 - std::ilogb(heaviest) : 0;
    for (uint32_t j = 0; j < p.n_clients; ++j) {
        weight[j] = std::ldexp(p.clients[j].weight, shift);
        if (weight[j] < std::numeric_limits<float>::min()) weight[j] = 0.0;
        total += weight[j];
    }
    for (uint32_t j = 0; j < p.n_clients; ++j)
        a.light |= weight[j] > 0.0 && weight[j] * fa::kLightest < total * (1.0 + 1e-6);   // (1e-6: fp32 in the kernel)
    fa_status r = check_mat(w, p.logits, p.rows, p.vocab, p.ld, p.dtype, "logits");
    for (uint32_t j = 0; r == FA_OK && j < p.n_clients; ++j) {
        const fa_distill_client& c = p.clients[j];
        r = check_mat(w, c.index, p.rows, c.topk, c.topk, FA_F32, "index");
        if (r == FA_OK) r = check_mat(w, c.value, p.rows, c.topk, c.topk, p.dtype_value, "value");
        a.client[j] = {c.index, c.value, c.topk, static_cast<float>(weight[j]),
                       total > 0.0 ? static_cast<float>(weight[j] / total) : 0.0f};
    }
    if (r == FA_OK && p.row_weight) r = check_mat(w, p.row_weight, 1, p.rows, p.rows, FA_F32, "row_weight");
    if (r == FA_OK && (p.loss || !grad)) r = check_mat(w, p.loss, 1, p.rows, p.rows, FA_F32, "loss");
    if (r == FA_OK && p.lse) r = check_mat(w, p.lse, 1, p.rows, p.rows, FA_F32, "lse");
    if (r == FA_OK && grad) r = check_mat(w, p.grad, p.rows, p.vocab, p.ldg, p.dtype, "grad");
    if (r != FA_OK) return r;
    const uint64_t sz = size_of(p.dtype);
    const bool inplace = grad && p.grad == p.logits && p.ldg == p.ld;
    const auto vector = [&](const void* v) { return Extent{v, 1, p.rows, p.rows, 4}; };
    const Extent out[] = {vector(p.loss), vector(grad ? nullptr : p.lse), {grad ? p.grad : nullptr, p.rows, p.vocab, p.ldg, sz}};
    const Extent logits{p.logits, p.rows, p.vocab, p.ld, sz};
    for (int i = 0; i < 3; ++i) {
        bool bad = (!(i == 2 && inplace) && overlap(out[i], logits)) || overlap(out[i], vector(p.row_weight)) ||
                   (grad && overlap(out[i], vector(p.lse)));
        for (uint32_t j = 0; !bad && j < p.n_clients; ++j) {
            const uint64_t k = p.clients[j].topk;
            bad = overlap(out[i], {p.clients[j].index, p.rows, k, k, 4}) ||
                  overlap(out[i], {p.clients[j].value, p.rows, k, k, size_of(p.dtype_value)});
        }
        for (int k = 0; !bad && k < i; ++k) bad = overlap(out[i], out[k]);
        if (bad) return fail(w, FA_ERR_ARG, "an output overlaps another tensor of the call");
    }
    const bool cap = capturing(s);
    r = chain_in(w, s, cap);
    if (r != FA_OK) return r;
    a.logits = p.logits;
    a.grad = grad ? p.grad : nullptr;
    a.row_weight = p.row_weight;
    a.loss = p.loss;
    a.lse_in = grad ? p.lse : nullptr;
    a.lse_out = grad ? nullptr : p.lse;
    a.err = w->err_dev;
    a.sms = static_cast<uint32_t>(w->tc.sms);
    a.test_expire = (w->flags & FA_TEST_WAIT_EXPIRES) != 0;
    a.ld = p.ld;
    a.ldg = p.ldg;
    a.rows = static_cast<uint32_t>(p.rows);
    a.vocab = static_cast<uint32_t>(p.vocab);
    a.nclients = p.n_clients;
    a.temperature = static_cast<float>(p.temperature);
    a.inv_t = static_cast<float>(1.0 / p.temperature);
    a.total = static_cast<float>(total);
    a.dtype = code_of(p.dtype);
    a.value_dtype = code_of(p.dtype_value);
    ChainOut chain(w, s, cap);
    return chain.end(launched(w, fa::launch_distill(a, s), grad ? "distillation gradient" : "distillation loss"));
}

void free_work(fa_work* w) {
    if (w->ws) cudaFree(w->ws);
    for (void* p : w->retired) cudaFree(p);
    if (w->chain) cudaEventDestroy(w->chain);
    if (w->err_ev) cudaEventDestroy(w->err_ev);
    if (w->err_stream) cudaStreamDestroy(w->err_stream);
    if (w->err_host) cudaFreeHost(w->err_host);
    if (w->err_dev) cudaFree(w->err_dev);
    delete w;
}

fa_status sync_impl(fa_work* w) {
    if (w->chain_valid) {
        const fa_status r = wait_event(w, w->chain, "fa_work_sync");
        if (r != FA_OK) return r;
    }
    *w->err_host = 0;
    FW_CUDA(w, cudaMemcpyAsync(w->err_host, w->err_dev, sizeof(unsigned int), cudaMemcpyDeviceToHost, w->err_stream));
    FW_CUDA(w, cudaMemsetAsync(w->err_dev, 0, sizeof(unsigned int), w->err_stream));
    FW_CUDA(w, cudaEventRecord(w->err_ev, w->err_stream));
    const fa_status r = wait_event(w, w->err_ev, "fa_work_sync (error word)");
    if (r != FA_OK) return r;
    if (*w->err_host & fa::kErrWaitTimeout)
        return fail(w, FA_ERR_INTERNAL, "a device-side wait gave up (bounded mbarrier wait): outputs are invalid");
    if (*w->err_host & fa::kErrListIndex)
        return fail(w, FA_ERR_RANGE, "a client's list named a vocabulary entry >= vocab (left out)");
    return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_work_open(const fa_work_opts* opts, fa_work** out) {
    if (out == nullptr) return FA_ERR_ARG;
    *out = nullptr;
    fa_work_opts o{};
    if (opts) {
        if (opts->size < sizeof(uint32_t) * 2) return FA_ERR_ARG;
        std::memcpy(&o, opts, std::min<size_t>(opts->size, sizeof o));
    }
    if (o.flags & ~FA_TEST_WAIT_EXPIRES) return FA_ERR_ARG;
    if (o.workspace_bytes >> 40) return FA_ERR_ARG;
    fa_work* w = new (std::nothrow) fa_work;
    if (!w) return FA_ERR_NOMEM;
    if (o.timeout_ms) w->timeout_ms = o.timeout_ms;
    w->flags = o.flags;
    cudaError_t ce = cudaGetDevice(&w->device);
    if (ce == cudaSuccess) ce = fa::prepare_distill();
    if (ce == cudaSuccess) ce = fa::prepare_product_tc(&w->tc);
    if (ce == cudaSuccess) ce = cudaMalloc(reinterpret_cast<void**>(&w->err_dev), kErrBytes);
    if (ce == cudaSuccess) ce = cudaEventCreateWithFlags(&w->chain, cudaEventDisableTiming);
    if (ce == cudaSuccess) ce = cudaEventCreateWithFlags(&w->err_ev, cudaEventDisableTiming);
    if (ce == cudaSuccess) ce = cudaStreamCreateWithFlags(&w->err_stream, cudaStreamNonBlocking);
    // zero before any caller's stream can set it: a memset does not wait for its own end
    if (ce == cudaSuccess) ce = cudaMemsetAsync(w->err_dev, 0, kErrBytes, w->err_stream);
    if (ce == cudaSuccess) ce = cudaStreamSynchronize(w->err_stream);
    if (ce == cudaSuccess)
        ce = cudaHostAlloc(reinterpret_cast<void**>(&w->err_host), sizeof(unsigned int), cudaHostAllocDefault);
    if (ce == cudaSuccess && o.workspace_bytes) {
        const uint64_t bytes = (o.workspace_bytes + (1ull << 21) - 1) >> 21 << 21;
        ce = cudaMalloc(reinterpret_cast<void**>(&w->ws), bytes);
        if (ce == cudaSuccess) w->ws_bytes = w->stats.workspace_bytes = bytes;
    }
    if (ce != cudaSuccess) {
        cudaGetLastError();
        free_work(w);
        return ce == cudaErrorMemoryAllocation ? FA_ERR_NOMEM : FA_ERR_CUDA;
    }
    *out = w;
    return FA_OK;
}

fa_status fa_work_close(fa_work* w) {
    if (!w) return FA_OK;
    return guarded([&]() -> fa_status {
        DeviceGuard dg(w->device);
        {
            std::lock_guard<std::mutex> lk(w->mu);
            if (w->chain_valid) {
                const fa_status r = wait_event(w, w->chain, "fa_work_close");
                if (r == FA_ERR_TIMEOUT) return r;
            }
        }
        free_work(w);
        return FA_OK;
    });
}

fa_status fa_work_sync(fa_work* w) {
    if (!w) return FA_ERR_ARG;
    return guarded([&] {
        std::lock_guard<std::mutex> lk(w->mu);
        DeviceGuard dg(w->device);
        w->err.clear();
        return sync_impl(w);
    });
}

fa_status fa_work_get_stats(fa_work* w, fa_work_stats* out) {
    if (!w || !out) return FA_ERR_ARG;
    std::lock_guard<std::mutex> lk(w->mu);
    *out = w->stats;
    return FA_OK;
}

const char* fa_work_last_error(const fa_work* w) { return w ? w->err.c_str() : ""; }

fa_status fa_product(fa_work* w, const fa_product_args* args, void* stream) {
    return enter("fa_product", w, args,
                 [&](const fa_product_args& p) { return product_impl(w, p, static_cast<cudaStream_t>(stream)); });
}

fa_status fa_product_backward(fa_work* w, const fa_product_backward_args* args, void* stream) {
    return enter("fa_product_backward", w, args, [&](const fa_product_backward_args& p) {
        return backward_impl(w, p, static_cast<cudaStream_t>(stream));
    });
}

fa_status fa_distill_loss(fa_work* w, const fa_distill_args* args, void* stream) {
    return enter("fa_distill_loss", w, args, [&](const fa_distill_args& p) {
        return distill_impl(w, p, false, static_cast<cudaStream_t>(stream));
    });
}

fa_status fa_distill_grad(fa_work* w, const fa_distill_args* args, void* stream) {
    return enter("fa_distill_grad", w, args, [&](const fa_distill_args& p) {
        return distill_impl(w, p, true, static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
