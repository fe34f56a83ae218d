// C entries of the state-space operators (include/pn.h): argument checks on
// the host, then launches on the caller's stream.  Nothing here allocates
// device memory or waits.

#include <algorithm>
#include <cmath>

#include "pn_seq_check.hpp"
#include "pn_ssm.hpp"

namespace {

using namespace pn;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 64;
constexpr int64_t kMaxSlots = int64_t(1) << 31;

bool misaligned(std::initializer_list<const void*> ps, int64_t bytes) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % bytes) return true;
    return false;
}

// Whether an output overlaps an input, or another output.
int check_overlaps(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& r : ins)
            if (overlap(*o, r)) return fail(PN_EINVAL, "an output overlaps an input");
        for (auto q = outs.begin(); q != o; ++q)
            if (overlap(*o, *q)) return fail(PN_EINVAL, "two outputs overlap");
    }
    return PN_OK;
}

int check_workspace(const void* ws, int64_t bytes, size_t need) {
    if (need == 0) return PN_OK;
    if (!ws || bytes < 0 || static_cast<size_t>(bytes) < need) return fail(PN_EWORKSPACE, "a workspace of %zu bytes is needed", need);
    if (reinterpret_cast<uintptr_t>(ws) % kAlign) return fail(PN_EWORKSPACE, "workspace must be 256-byte aligned");
    return PN_OK;
}

// Never kAlign, which says that none is needed.
size_t padded(size_t n) { return n == 0 ? 0 : std::max(align_up(n), 2 * kAlign); }

Range range3(const pn_tokens& x, int64_t B, int64_t T, int64_t D, int64_t elem) {
    return x.p ? range(pn_tokens{x.p, x.sb, x.st, 0}, B, T, 1, D, elem) : Range{0, 0};
}

// Tokens without heads, whose stride of heads is any number.
int check_rows(const pn_tokens& x, const char* name, int64_t elem) {
    return check_tokens(pn_tokens{x.p, x.sb, x.st, 0}, name, elem);
}

int check_types(int64_t dtype, int64_t B, int64_t T, int64_t D) {
    if (dtype < PN_F32 || dtype > PN_F16) return fail(PN_EINVAL, "unknown storage type %lld", (long long)dtype);
    if (B < 0 || T < 0 || D < 0) return fail(PN_EINVAL, "negative size");
    if (T > kMaxTokens || D > kMaxBlocks || !small_product({B, T}, kMaxBlocks) ||
        !small_product({B, std::max<int64_t>(T, 1), D}, int64_t(1) << 38))
        return fail(PN_EUNSUPPORTED, "size too large");
    return PN_OK;
}

// ---------------------------------------------------------------- short convolution

int check_conv_sizes(int64_t dtype, int64_t B, int64_t T, int64_t D, int64_t W, int64_t activation) {
    PN_TRY(check_types(dtype, B, T, D));
    if (W < 1 || W > 8) return fail(PN_EUNSUPPORTED, "1 .. 8 taps are supported");
    if (activation < 0 || activation > 1) return fail(PN_EINVAL, "activation must be 0 or 1");
    return PN_OK;
}

int check_conv(const pn_conv_args* p, bool backward) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_conv_args& a = *p;
    PN_TRY(check_conv_sizes(a.dtype, a.B, a.T, a.D, a.W, a.activation));
    if (a.D == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype), taps = 4 * a.D * a.W, state = e * a.B * (a.W - 1) * a.D;
    if (!a.weight) return fail(PN_EINVAL, "weight is NULL");
    if (backward && (!a.dweight || (a.bias && !a.dbias))) return fail(PN_EINVAL, "an output is NULL");
    if (misaligned({a.weight, a.bias, a.lengths, a.dweight, a.dbias}, 4)) return fail(PN_EINVAL, "a 4-byte array is not aligned");
    if (misaligned({a.initial_state, a.y, a.final_state, a.d_final_state, a.dx, a.d_initial_state}, e))
        return fail(PN_EINVAL, "an array is not aligned to its type");
    const bool tokens = a.B > 0 && a.T > 0;
    if (tokens) {
        PN_TRY(check_rows(a.x, "x", e));
        if (backward) PN_TRY(check_rows(a.dy, "dy", e));
        if (backward ? !a.dx : !a.y) return fail(PN_EINVAL, "an output is NULL");
    }
    const Range x = range3(a.x, a.B, a.T, a.D, e), w = range(a.weight, taps), bias = range(a.bias, 4 * a.D);
    const Range n = range(a.lengths, 4 * a.B), s0 = range(a.initial_state, state);
    if (!backward)
        return check_overlaps({range(a.y, e * a.B * a.T * a.D), range(a.final_state, state)}, {x, w, bias, n, s0});
    const size_t need = tokens ? padded(conv_workspace(a)) : 0;
    PN_TRY(check_workspace(a.workspace, a.workspace_bytes, need));
    return check_overlaps({range(a.dx, e * a.B * a.T * a.D), range(a.dweight, taps), range(a.bias ? a.dbias : nullptr, 4 * a.D),
                           range(a.d_initial_state, state), range(need ? a.workspace : nullptr, static_cast<int64_t>(need))},
                          {x, w, bias, n, s0, range3(a.dy, a.B, a.T, a.D, e), range(a.d_final_state, state)});
}

// ---------------------------------------------------------------- selective scan

int check_ssm_sizes(int64_t dtype, int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int64_t softplus) {
    PN_TRY(check_types(dtype, B, T, D));
    if (D > int64_t(1) << 24) return fail(PN_EUNSUPPORTED, "size too large");
    if (N < 1 || N > 128) return fail(PN_EUNSUPPORTED, "1 .. 128 states per channel are supported");
    if (G < 1 || (D > 0 && (G > D || D % G))) return fail(PN_EINVAL, "D must be a multiple of G >= 1");
    if (softplus < 0 || softplus > 1) return fail(PN_EINVAL, "softplus must be 0 or 1");
    if (!small_product({std::max<int64_t>(B, 1), std::max<int64_t>(T, 1), G, 2 * N}, int64_t(1) << 38) ||
        !small_product({std::max<int64_t>(B, 1), D, N}, int64_t(1) << 38))
        return fail(PN_EUNSUPPORTED, "size too large");
    return PN_OK;
}

// Offsets within a tile of the scan are 32 bits wide.
constexpr int64_t kMaxScanStride = int64_t(1) << 26;

int check_ssm(const pn_ssm_args* p, bool backward) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_ssm_args& a = *p;
    PN_TRY(check_ssm_sizes(a.dtype, a.B, a.T, a.D, a.N, a.G, a.softplus));
    if (a.D == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype), state = 4 * a.B * a.D * a.N, rows = a.B * a.T;
    if (!a.A) return fail(PN_EINVAL, "A is NULL");
    if (backward && (!a.dA || (a.skip && !a.dskip) || (a.dt_bias && !a.ddt_bias))) return fail(PN_EINVAL, "an output is NULL");
    if (misaligned({a.A, a.skip, a.dt_bias, a.lengths, a.initial_state, a.final_state, a.d_final_state, a.dA, a.dskip, a.ddt_bias,
                    a.d_initial_state}, 4))
        return fail(PN_EINVAL, "a 4-byte array is not aligned");
    if (misaligned({a.y, a.dx, a.ddt, a.dgate, a.db, a.dc}, e)) return fail(PN_EINVAL, "an output is not aligned to its type");
    if (rows > 0) {
        PN_TRY(check_rows(a.x, "x", e));
        PN_TRY(check_rows(a.dt, "dt", e));
        PN_TRY(check_tokens(a.b, "b", e));
        PN_TRY(check_tokens(a.c, "c", e));
        if (a.gate.p) PN_TRY(check_rows(a.gate, "gate", e));
        if (backward) PN_TRY(check_rows(a.dy, "dy", e));
        if (backward ? !a.dx || !a.ddt || !a.db || !a.dc || (a.gate.p && !a.dgate) : !a.y)
            return fail(PN_EINVAL, "an output is NULL");
    }
    if (a.T > 1)
        for (const pn_tokens* t : {&a.x, &a.dt, &a.gate, &a.b, &a.c, &a.dy})
            if (t->p && (backward || t != &a.dy) && t->st > kMaxScanStride)
                return fail(PN_EUNSUPPORTED, "token strides of up to 2^26 elements are supported");
    const Range none{0, 0};
    const Range x = range3(a.x, a.B, a.T, a.D, e), dt = range3(a.dt, a.B, a.T, a.D, e), z = range3(a.gate, a.B, a.T, a.D, e);
    const Range b = range(a.b, a.B, a.T, a.G, a.N, e), c = range(a.c, a.B, a.T, a.G, a.N, e);
    const Range A = range(a.A, 4 * a.D * a.N), skip = range(a.skip, 4 * a.D), bias = range(a.dt_bias, 4 * a.D);
    const Range n = range(a.lengths, 4 * a.B), s0 = range(a.initial_state, state);
    size_t need = 0;
    if (a.B > 0) {
        const SsmPlan plan = plan_ssm(a, backward);
        if (!ssm_fits(a, plan)) return fail(PN_EUNSUPPORTED, "too many sequences and channels for one launch");
        need = padded(sizeof(float) * static_cast<size_t>(plan.total));
    }
    PN_TRY(check_workspace(a.workspace, a.workspace_bytes, need));
    const Range ws = need ? range(a.workspace, static_cast<int64_t>(need)) : none;
    if (!backward)
        return check_overlaps({range(a.y, e * rows * a.D), range(a.final_state, state), ws}, {x, dt, z, b, c, A, skip, bias, n, s0});
    return check_overlaps({range(a.dx, e * rows * a.D), range(a.ddt, e * rows * a.D), range(a.gate.p ? a.dgate : nullptr, e * rows * a.D),
                           range(a.db, e * rows * a.G * a.N), range(a.dc, e * rows * a.G * a.N), range(a.dA, 4 * a.D * a.N),
                           range(a.skip ? a.dskip : nullptr, 4 * a.D), range(a.dt_bias ? a.ddt_bias : nullptr, 4 * a.D),
                           range(a.d_initial_state, state), ws},
                          {x, dt, z, b, c, A, skip, bias, n, s0, range3(a.dy, a.B, a.T, a.D, e), range(a.d_final_state, state)});
}

// The token stride of one token is any number, and is left out.
pn_ssm_args one_token(pn_ssm_args a) {
    if (a.T <= 1)
        for (pn_tokens* t : {&a.x, &a.dt, &a.gate, &a.b, &a.c, &a.dy}) t->st = 0;
    return a;
}

// ---------------------------------------------------------------- norms around a block

int check_norm_sizes(const pn_block_norm_args& a) {
    PN_TRY(check_types(a.dtype, a.B, a.T, a.D));
    if (a.residual_dtype != PN_F32 && a.residual_dtype != a.dtype)
        return fail(PN_EINVAL, "the residual has the storage type or float32");
    if (a.D < 1 || a.D > 8192) return fail(PN_EUNSUPPORTED, "1 .. 8192 channels are supported");
    if (!(a.eps >= 0.0 && std::isfinite(a.eps))) return fail(PN_EINVAL, "eps must be finite and >= 0");
    return PN_OK;
}

int check_norm(const pn_block_norm_args* p, bool backward) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_block_norm_args& a = *p;
    PN_TRY(check_norm_sizes(a));
    const int64_t e = elem_bytes(a.dtype), er = elem_bytes(a.residual_dtype), n = a.B * a.T * a.D;
    if (misaligned({a.weight, a.post_weight, a.scale, a.dweight, a.dpost_weight, a.dscale}, 4))
        return fail(PN_EINVAL, "a float array is not aligned");
    if (backward && ((a.weight && !a.dweight) || (a.post_weight && !a.dpost_weight) || (a.scale && !a.dscale)))
        return fail(PN_EINVAL, "an output is NULL");
    if (n > 0) {
        PN_TRY(check_rows(a.x, "x", e));
        if (a.gate.p) PN_TRY(check_rows(a.gate, "gate", e));
        if (a.residual.p) PN_TRY(check_rows(a.residual, "residual", er));
        if (!backward) {
            if (!a.s || (a.weight && !a.y)) return fail(PN_EINVAL, "an output is NULL");
        } else {
            if (a.weight) PN_TRY(check_rows(a.dy, "dy", e));
            if (a.ds.p) PN_TRY(check_rows(a.ds, "ds", er));
            if (!a.dx || (a.gate.p && !a.dgate)) return fail(PN_EINVAL, "an output is NULL");
        }
        if (misaligned({a.y, a.dx, a.dgate}, e) || misaligned({a.s, a.dresidual}, er))
            return fail(PN_EINVAL, "an output is not aligned to its type");
    }
    const Range x = range3(a.x, a.B, a.T, a.D, e), z = range3(a.gate, a.B, a.T, a.D, e);
    const Range w = range(a.weight, 4 * a.D), pw = range(a.post_weight, 4 * a.D), sc = range(a.scale, 4 * a.D);
    const Range res = range3(a.residual, a.B, a.T, a.D, er);
    if (!backward)
        return check_overlaps({range(a.weight ? a.y : nullptr, e * n), range(a.s, er * n)},
                              {x, z, w, pw, sc, res});
    const size_t need = n > 0 ? padded(block_norm_workspace(a)) : 0;
    PN_TRY(check_workspace(a.workspace, a.workspace_bytes, need));
    return check_overlaps({range(a.dx, e * n), range(a.gate.p ? a.dgate : nullptr, e * n), range(a.dresidual, er * n),
                           range(a.weight ? a.dweight : nullptr, 4 * a.D), range(a.post_weight ? a.dpost_weight : nullptr, 4 * a.D),
                           range(a.scale ? a.dscale : nullptr, 4 * a.D), need ? range(a.workspace, static_cast<int64_t>(need)) : Range{0, 0}},
                          {x, z, w, pw, sc, res, a.weight ? range3(a.dy, a.B, a.T, a.D, e) : Range{0, 0},
                           range3(a.ds, a.B, a.T, a.D, er)});
}

int zeros(float* p, int64_t n, hipStream_t st) { return p ? launched(launch_fill(p, n, st)) : PN_OK; }

}  // namespace

extern "C" {

int pn_short_conv(const pn_conv_args* a) {
    PN_TRY(check_conv(a, false));
    if (a->B == 0 || a->D == 0) return PN_OK;
    return launched(launch_conv(*a, static_cast<hipStream_t>(a->stream)));
}

int pn_short_conv_backward(const pn_conv_args* a) {
    PN_TRY(check_conv(a, true));
    if (a->D == 0) return PN_OK;
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    if (a->B == 0 || a->T == 0) {                        // no token: sums over nothing, and the state is the initial one
        PN_TRY(zeros(a->dweight, a->D * a->W, st));
        PN_TRY(zeros(a->bias ? a->dbias : nullptr, a->D, st));
        if (a->B == 0 || !a->d_initial_state || a->W == 1) return PN_OK;
        return launched(launch_conv_state(*a, st));
    }
    return launched(launch_conv_backward(*a, st));
}

size_t pn_short_conv_workspace_bytes(const pn_conv_args* a) {
    clear_error();
    if (!a) {
        fail(PN_EINVAL, "the arguments are NULL");
        return 0;
    }
    if (check_conv_sizes(a->dtype, a->B, a->T, a->D, a->W, a->activation) != PN_OK) return 0;
    if (a->B == 0 || a->T == 0 || a->D == 0) return kAlign;
    return padded(conv_workspace(*a));
}

int pn_short_conv_step(const pn_conv_step_args* p) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_conv_step_args& a = *p;
    PN_TRY(check_conv_sizes(a.dtype, a.B, 1, a.D, a.W, a.activation));
    if (a.n_slots < 0 || a.n_slots > kMaxSlots) return fail(PN_EINVAL, "n_slots out of range");
    if (!small_product({std::max<int64_t>(a.n_slots, 1), a.D, a.W}, int64_t(1) << 45)) return fail(PN_EUNSUPPORTED, "size too large");
    if (a.B == 0 || a.D == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype);
    PN_TRY(check_rows(a.x, "x", e));
    if (!a.weight || !a.y) return fail(PN_EINVAL, "weight or y is NULL");
    if (!a.state && a.n_slots > 0 && a.W > 1) return fail(PN_EINVAL, "state is NULL");
    if (!a.slots && a.n_slots < a.B) return fail(PN_EINVAL, "fewer slots than sequences");
    if (misaligned({a.weight, a.bias, a.slots}, 4) || misaligned({a.state, a.y}, e))
        return fail(PN_EINVAL, "an array is not aligned to its type");
    PN_TRY(check_overlaps({range(a.y, e * a.B * a.D), range(a.state, e * a.n_slots * (a.W - 1) * a.D)},
                          {range3(a.x, a.B, 1, a.D, e), range(a.weight, 4 * a.D * a.W), range(a.bias, 4 * a.D), range(a.slots, 4 * a.B)}));
    return launched(launch_conv_step(a, static_cast<hipStream_t>(a.stream)));
}

size_t pn_ssm_scan_workspace_bytes(const pn_ssm_args* a, int32_t backward) {
    clear_error();
    if (!a) {
        fail(PN_EINVAL, "the arguments are NULL");
        return 0;
    }
    if (check_ssm_sizes(a->dtype, a->B, a->T, a->D, a->N, a->G, a->softplus) != PN_OK) return 0;
    if (a->B == 0 || a->D == 0) return kAlign;
    const SsmPlan p = plan_ssm(*a, backward != 0);
    if (!ssm_fits(*a, p)) {
        fail(PN_EUNSUPPORTED, "too many sequences and channels for one launch");
        return 0;
    }
    return p.total > 0 ? padded(sizeof(float) * static_cast<size_t>(p.total)) : kAlign;
}

int pn_ssm_scan(const pn_ssm_args* p) {
    PN_TRY(check_ssm(p, false));
    if (p->B == 0 || p->D == 0) return PN_OK;
    const pn_ssm_args a = one_token(*p);
    return launched(launch_ssm(a, plan_ssm(a, false), static_cast<hipStream_t>(a.stream)));
}

int pn_ssm_scan_backward(const pn_ssm_args* p) {
    PN_TRY(check_ssm(p, true));
    if (p->D == 0) return PN_OK;
    const pn_ssm_args a = one_token(*p);
    hipStream_t st = static_cast<hipStream_t>(a.stream);
    if (a.B == 0) {                                      // sums over nothing
        PN_TRY(zeros(a.dA, a.D * a.N, st));
        PN_TRY(zeros(a.skip ? a.dskip : nullptr, a.D, st));
        return zeros(a.dt_bias ? a.ddt_bias : nullptr, a.D, st);
    }
    return launched(launch_ssm_backward(a, plan_ssm(a, true), st));
}

int pn_ssm_step(const pn_ssm_step_args* p) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_ssm_step_args& a = *p;
    PN_TRY(check_ssm_sizes(a.dtype, a.B, 1, a.D, a.N, a.G, a.softplus));
    if (a.n_slots < 0 || a.n_slots > kMaxSlots) return fail(PN_EINVAL, "n_slots out of range");
    if (!small_product({std::max<int64_t>(a.n_slots, 1), std::max<int64_t>(a.D, 1), a.N}, int64_t(1) << 45) ||
        !small_product({a.B, a.D}, kMaxBlocks))
        return fail(PN_EUNSUPPORTED, "size too large");
    if (a.B == 0 || a.D == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype);
    PN_TRY(check_rows(a.x, "x", e));
    PN_TRY(check_rows(a.dt, "dt", e));
    PN_TRY(check_tokens(a.b, "b", e));
    PN_TRY(check_tokens(a.c, "c", e));
    if (a.gate.p) PN_TRY(check_rows(a.gate, "gate", e));
    if (!a.A || !a.y) return fail(PN_EINVAL, "A or y is NULL");
    if (!a.state && a.n_slots > 0) return fail(PN_EINVAL, "state is NULL");
    if (!a.slots && a.n_slots < a.B) return fail(PN_EINVAL, "fewer slots than sequences");
    if (misaligned({a.A, a.skip, a.dt_bias, a.state, a.slots}, 4) || misaligned({a.y}, e))
        return fail(PN_EINVAL, "an array is not aligned to its type");
    PN_TRY(check_overlaps({range(a.y, e * a.B * a.D), range(a.state, 4 * a.n_slots * a.D * a.N)},
                          {range3(a.x, a.B, 1, a.D, e), range3(a.dt, a.B, 1, a.D, e), range3(a.gate, a.B, 1, a.D, e),
                           range(a.b, a.B, 1, a.G, a.N, e), range(a.c, a.B, 1, a.G, a.N, e), range(a.A, 4 * a.D * a.N),
                           range(a.skip, 4 * a.D), range(a.dt_bias, 4 * a.D), range(a.slots, 4 * a.B)}));
    return launched(launch_ssm_step(a, static_cast<hipStream_t>(a.stream)));
}

int pn_block_norm(const pn_block_norm_args* a) {
    PN_TRY(check_norm(a, false));
    if (a->B == 0 || a->T == 0) return PN_OK;
    return launched(launch_block_norm(*a, static_cast<hipStream_t>(a->stream)));
}

size_t pn_block_norm_workspace_bytes(const pn_block_norm_args* a) {
    clear_error();
    if (!a) {
        fail(PN_EINVAL, "the arguments are NULL");
        return 0;
    }
    if (check_norm_sizes(*a) != PN_OK) return 0;
    if (a->B == 0 || a->T == 0) return kAlign;
    const size_t n = padded(block_norm_workspace(*a));
    return n > 0 ? n : kAlign;
}

int pn_block_norm_backward(const pn_block_norm_args* a) {
    PN_TRY(check_norm(a, true));
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    if (a->B == 0 || a->T == 0) {                        // sums over nothing
        PN_TRY(zeros(a->weight ? a->dweight : nullptr, a->D, st));
        PN_TRY(zeros(a->post_weight ? a->dpost_weight : nullptr, a->D, st));
        return zeros(a->scale ? a->dscale : nullptr, a->D, st);
    }
    return launched(launch_block_norm_backward(*a, st));
}

}  // extern "C"
