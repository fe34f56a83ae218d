// C entries of the sequence-layer operators (include/pn.h): argument checks
// on the host, then launches on the caller's stream.  Nothing here allocates
// device memory or waits.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "pn_seq.hpp"

namespace {

using namespace pn;

constexpr int64_t kMaxBlocks = (int64_t(1) << 31) - 1;
constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

int fail(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_error(code, buf);
}

int launched(hipError_t e) {
    return e == hipSuccess ? PN_OK : fail(PN_EHIP, "launch failed: %s", hipGetErrorString(e));
}

int64_t elem_bytes(int64_t dtype) { return dtype == PN_F32 ? 4 : 2; }

// The bytes an array may touch.
struct Range {
    uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return p && bytes > 0 ? Range{a, a + static_cast<uintptr_t>(bytes)} : Range{0, 0};
}
Range range(const pn_tokens& x, int64_t B, int64_t T, int64_t heads, int64_t D, int64_t elem) {
    if (B <= 0 || T <= 0 || heads <= 0) return Range{0, 0};
    return range(x.p, elem * ((B - 1) * x.sb + (T - 1) * x.st + (heads - 1) * x.sh + D));
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Products of sizes in int64 without overflow.
bool small_product(std::initializer_list<int64_t> v, int64_t limit) {
    int64_t p = 1;
    for (int64_t x : v) {
        if (x == 0) return true;
        if (p > limit / x) return false;
        p *= x;
    }
    return p <= limit;
}

constexpr int64_t kMaxStride = int64_t(1) << 40;
int check_tokens(const pn_tokens& x, const char* name, int64_t elem) {
    if (!x.p) return fail(PN_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(x.p) % elem) return fail(PN_EINVAL, "%s is not aligned to its type", name);
    for (int64_t s : {x.sb, x.st, x.sh})
        if (s < 0 || s > kMaxStride) return fail(PN_EINVAL, "a stride of %s is out of range", name);
    return PN_OK;
}

#define PN_TRY(call)                      \
    do {                                  \
        const int rc_ = (call);           \
        if (rc_ != PN_OK) return rc_;     \
    } while (0)

// Never kAlign, which says that none is needed.
size_t norm_workspace(const pn_rotary_args& a) { return std::max(align_up(rotary_backward_workspace(a)), 2 * kAlign); }

int check_rotary_sizes(const pn_rotary_args& a, bool norm) {
    if (a.dtype < PN_F32 || a.dtype > PN_F16) return fail(PN_EINVAL, "unknown storage type %lld", (long long)a.dtype);
    if (a.B < 0 || a.T < 0 || a.hq < 0 || a.hk < 0) return fail(PN_EINVAL, "negative size");
    if (a.D < 1 || a.D > 256) return fail(PN_EUNSUPPORTED, "channels per head must lie in 1 .. 256");
    if (a.R < 0 || a.R > a.D || a.R % 2) return fail(PN_EINVAL, "the rotated channels must be even and within the head");
    if (a.interleaved < 0 || a.interleaved > 1 || a.inverse < 0 || a.inverse > 1)
        return fail(PN_EINVAL, "interleaved and inverse must be 0 or 1");
    if (a.hk > 0 && a.hq == 0) return fail(PN_EINVAL, "k without q");
    if (norm && !(a.eps >= 0.0 && std::isfinite(a.eps))) return fail(PN_EINVAL, "eps must be finite and >= 0");
    if (norm && ((a.qw_sh != 0 && a.qw_sh != a.D) || (a.kw_sh != 0 && a.kw_sh != a.D)))
        return fail(PN_EINVAL, "the stride of a weight's heads must be 0 or D");
    if (!small_product({a.B, a.T, a.hq + a.hk}, kMaxBlocks)) return fail(PN_EUNSUPPORTED, "size too large");
    return PN_OK;
}

int check_rotary(const pn_rotary_args* p, bool norm, bool backward) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_rotary_args& a = *p;
    PN_TRY(check_rotary_sizes(a, norm));
    if (a.B == 0 || a.T == 0 || a.hq == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype);
    PN_TRY(check_tokens(a.q, "q", e));
    if (a.hk) PN_TRY(check_tokens(a.k, "k", e));
    if (!a.q_out || (a.hk && !a.k_out)) return fail(PN_EINVAL, "an output is NULL");
    if (reinterpret_cast<uintptr_t>(a.q_out) % e || reinterpret_cast<uintptr_t>(a.k_out) % e)
        return fail(PN_EINVAL, "an output is not aligned to its type");
    if (a.R > 0) {
        if (!a.table) return fail(PN_EINVAL, "table is NULL");
        if (a.n_pos < 0 || !small_product({a.n_pos, a.R}, int64_t(1) << 40)) return fail(PN_EINVAL, "n_pos out of range");
    }
    if (a.positions) {                                   // read whatever R is
        if (a.pos64 < 0 || a.pos64 > 1) return fail(PN_EINVAL, "pos64 must be 0 or 1");
        if (a.pos_sb < 0 || a.pos_st < 0 || a.pos_sb > kMaxStride || a.pos_st > kMaxStride)
            return fail(PN_EINVAL, "a stride of positions is out of range");
        if (reinterpret_cast<uintptr_t>(a.positions) % (a.pos64 ? 8 : 4))
            return fail(PN_EINVAL, "positions are not aligned to their type");
    }
    if ((reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.qw) |
         reinterpret_cast<uintptr_t>(a.kw) | reinterpret_cast<uintptr_t>(a.dqw) |
         reinterpret_cast<uintptr_t>(a.dkw)) % 4)
        return fail(PN_EINVAL, "a float array is not aligned");
    if (backward) {
        PN_TRY(check_tokens(a.dq, "dq", e));
        if (a.hk) PN_TRY(check_tokens(a.dk, "dk", e));
    }
    const Range qi = range(a.q, a.B, a.T, a.hq, a.D, e), ki = range(a.k, a.B, a.T, a.hk, a.D, e);
    const Range qo = range(a.q_out, e * a.B * a.T * a.hq * a.D), ko = range(a.k_out, e * a.B * a.T * a.hk * a.D);
    // in place: the output is its own input, laid out alike
    auto in_place = [&](const pn_tokens& x, const void* out, int64_t heads) {
        return !backward && x.p == out && (heads == 1 || x.sh == a.D) && (a.T == 1 || x.st == heads * a.D) &&
               (a.B == 1 || x.sb == a.T * heads * a.D);
    };
    bool bad = overlap(qo, ko) || overlap(qo, ki) || overlap(ko, qi);
    bad = bad || (overlap(qo, qi) && !in_place(a.q, a.q_out, a.hq));
    bad = bad || (a.hk && overlap(ko, ki) && !in_place(a.k, a.k_out, a.hk));
    const Range aux[4] = {range(a.table, a.R > 0 ? 4 * a.n_pos * a.R : 0),
                          range(a.positions, a.positions ? (a.pos64 ? 8 : 4) * ((a.B - 1) * a.pos_sb + (a.T - 1) * a.pos_st + 1) : 0),
                          range(norm ? a.qw : nullptr, 4 * (a.qw_sh ? a.hq * a.D : a.D)),
                          range(norm ? a.kw : nullptr, 4 * (a.kw_sh ? a.hk * a.D : a.D))};
    for (const Range& r : aux) bad = bad || overlap(qo, r) || overlap(ko, r);
    if (backward) {
        const Range dqi = range(a.dq, a.B, a.T, a.hq, a.D, e), dki = range(a.dk, a.B, a.T, a.hk, a.D, e);
        const Range w[2] = {range(a.dqw, 4 * (a.qw_sh ? a.hq * a.D : a.D)), range(a.dkw, 4 * (a.kw_sh ? a.hk * a.D : a.D))};
        for (const Range& o : {qo, ko, w[0], w[1]}) bad = bad || overlap(o, dqi) || overlap(o, dki);
        for (const Range& o : w) {
            bad = bad || overlap(o, qi) || overlap(o, ki) || overlap(o, qo) || overlap(o, ko);
            for (const Range& r : aux) bad = bad || overlap(o, r);
        }
        bad = bad || overlap(w[0], w[1]);
        const Range ws = range(a.workspace, static_cast<int64_t>(norm_workspace(a)));
        for (const Range& r : {qi, ki, dqi, dki, qo, ko, w[0], w[1], aux[0], aux[1], aux[2], aux[3]}) bad = bad || overlap(ws, r);
    }
    if (bad) return fail(PN_EINVAL, "an output overlaps an input or another output");
    return PN_OK;
}

int check_linattn_sizes(int64_t dtype, int64_t B, int64_t T, int64_t H, int64_t HK, int64_t dk, int64_t dv,
                        double scale) {
    if (dtype < PN_F32 || dtype > PN_F16) return fail(PN_EINVAL, "unknown storage type %lld", (long long)dtype);
    if (B < 0 || T < 0 || H < 0) return fail(PN_EINVAL, "negative size");
    if (H > 0 && (HK < 1 || H % HK)) return fail(PN_EINVAL, "H must be a multiple of HK >= 1");
    if (dk < 1 || dv < 1 || dk > 256 || dv > 256) return fail(PN_EUNSUPPORTED, "channels per head must lie in 1 .. 256");
    if (!std::isfinite(scale)) return fail(PN_EINVAL, "scale must be finite");
    if (T >= (int64_t(1) << 31) - 64 || !small_product({B, H}, int64_t(1) << 24) || !small_product({B, T, H}, kMaxBlocks))
        return fail(PN_EUNSUPPORTED, "size too large");
    return PN_OK;
}

// The token stride of one token is any number, and is left out: over reversed
// time the kernel steps back over the tokens that a chunk lacks.
LaOperand operand(const pn_tokens& x, int64_t T, int div) { return LaOperand{x.p, x.sb, T > 1 ? x.st : 0, x.sh, div}; }

// The operators of a call and the regions of its workspace.
struct LinattnPlan {
    LaArgs la{};
    size_t off_dk = 0, off_dv = 0, off_carry = 0, total = 0;   // float32 dk, dv of each head (where shared), carries
};
LinattnPlan plan_linattn(const pn_linattn_args& a, bool backward) {
    LinattnPlan p;
    LaArgs& g = p.la;
    g.dtype = static_cast<int32_t>(a.dtype);
    g.B = static_cast<int32_t>(a.B);
    g.H = static_cast<int32_t>(a.H);
    g.T = a.T;
    g.log_decay = a.log_decay;
    g.lengths = a.lengths;
    const int share = static_cast<int>(a.H / a.HK);
    const int32_t dk = static_cast<int32_t>(a.dk), dv = static_cast<int32_t>(a.dv);
    const float scale = static_cast<float>(a.scale);
    char* ws = static_cast<char*>(a.workspace);
    if (!backward) {
        LaOp& f = g.op[0];
        f.q = operand(a.q, a.T, 1);
        f.k = operand(a.k, a.T, share);
        f.v = operand(a.v, a.T, share);
        f.o = a.o;
        f.DK = dk;
        f.DV = dv;
        f.inter = scale;
        f.ws = 1.0f;
        f.s_in = a.initial_state;
        f.s_k = dv;
        f.s_v = 1;
        f.s_out = a.final_state;
        f.exact = a.final_state != nullptr;
        g.n_ops = 1;
    } else {
        if (share > 1) {
            p.total = align_up(sizeof(float) * static_cast<size_t>(a.B * a.T * a.H) * dk);
            p.off_dv = p.total;
            p.total += align_up(sizeof(float) * static_cast<size_t>(a.B * a.T * a.H) * dv);
        }
        // dq: the state S again, transposed
        LaOp& q = g.op[0];
        q.q = operand(a.do_, a.T, 1);
        q.k = operand(a.v, a.T, share);
        q.v = operand(a.k, a.T, share);
        q.o = a.dq;
        q.DK = dv;
        q.DV = dk;
        q.inter = scale;
        q.ws = 1.0f;
        q.s_in = a.initial_state;
        q.s_k = 1;
        q.s_v = dv;
        // dv: the state's gradient R, backwards in time
        LaOp& v = g.op[1];
        v.q = operand(a.k, a.T, share);
        v.k = operand(a.q, a.T, 1);
        v.v = operand(a.do_, a.T, 1);
        v.o = share > 1 ? static_cast<void*>(ws + p.off_dv) : a.dv_;
        v.o_f32 = share > 1;
        v.reverse = 1;
        v.DK = dk;
        v.DV = dv;
        v.inter = 1.0f;
        v.ws = scale;
        v.s_in = a.d_final_state;
        v.s_k = dv;
        v.s_v = 1;
        v.s_out = a.d_initial_state;
        v.exact = a.d_initial_state != nullptr;
        v.carry_from = 1;
        // dk: R again, transposed
        LaOp& k = g.op[2];
        k.q = operand(a.v, a.T, share);
        k.k = operand(a.do_, a.T, 1);
        k.v = operand(a.q, a.T, 1);
        k.o = share > 1 ? static_cast<void*>(ws + p.off_dk) : a.dk_;
        k.o_f32 = share > 1;
        k.reverse = 1;
        k.DK = dv;
        k.DV = dk;
        k.inter = 1.0f;
        k.ws = scale;
        k.s_in = a.d_final_state;
        k.s_k = 1;
        k.s_v = dv;
        k.carry_from = 1;
        g.n_ops = 3;
    }
    p.off_carry = p.total;
    p.total += align_up(linattn_workspace(g));
    if (p.total > 0) p.total = std::max(p.total, 2 * kAlign);
    return p;
}

int check_linattn(const pn_linattn_args* p, bool backward) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_linattn_args& a = *p;
    PN_TRY(check_linattn_sizes(a.dtype, a.B, a.T, a.H, a.HK, a.dk, a.dv, a.scale));
    if (a.B == 0 || a.H == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype), ns = 4 * a.B * a.H * a.dk * a.dv;
    if (!a.log_decay) return fail(PN_EINVAL, "log_decay is NULL");
    if (a.T > 0) {
        PN_TRY(check_tokens(a.q, "q", e));
        PN_TRY(check_tokens(a.k, "k", e));
        PN_TRY(check_tokens(a.v, "v", e));
        if (backward) PN_TRY(check_tokens(a.do_, "do", e));
        if (backward ? !a.dq || !a.dk_ || !a.dv_ : !a.o) return fail(PN_EINVAL, "an output is NULL");
    }
    const void* f32s[] = {a.log_decay, a.lengths, a.initial_state, a.final_state, a.d_final_state, a.d_initial_state};
    for (const void* f : f32s)
        if (reinterpret_cast<uintptr_t>(f) % 4) return fail(PN_EINVAL, "a 4-byte array is not aligned");
    const void* outs_e[] = {a.o, a.dq, a.dk_, a.dv_};
    for (const void* f : outs_e)
        if (reinterpret_cast<uintptr_t>(f) % e) return fail(PN_EINVAL, "an output is not aligned to its type");
    const Range in[] = {range(a.q, a.B, a.T, a.H, a.dk, e),     range(a.k, a.B, a.T, a.HK, a.dk, e),
                        range(a.v, a.B, a.T, a.HK, a.dv, e),    range(a.log_decay, 4 * a.H),
                        range(a.lengths, 4 * a.B),              range(a.initial_state, ns),
                        backward ? range(a.do_, a.B, a.T, a.H, a.dv, e) : Range{0, 0},
                        backward ? range(a.d_final_state, ns) : Range{0, 0}};
    Range out[5] = {};
    if (backward) {
        out[0] = range(a.dq, e * a.B * a.T * a.H * a.dk);
        out[1] = range(a.dk_, e * a.B * a.T * a.HK * a.dk);
        out[2] = range(a.dv_, e * a.B * a.T * a.HK * a.dv);
        out[3] = range(a.d_initial_state, ns);
    } else {
        out[0] = range(a.o, e * a.B * a.T * a.H * a.dv);
        out[1] = range(a.final_state, ns);
    }
    const LinattnPlan plan = plan_linattn(a, backward);
    if (!linattn_fits(plan.la)) return fail(PN_EUNSUPPORTED, "too many sequences and heads for one launch");
    const size_t need = plan.total;
    if (need > 0) {
        if (!a.workspace || a.workspace_bytes < 0 || static_cast<size_t>(a.workspace_bytes) < need)
            return fail(PN_EWORKSPACE, "a workspace of %zu bytes is needed", need);
        if (reinterpret_cast<uintptr_t>(a.workspace) % kAlign)
            return fail(PN_EWORKSPACE, "workspace must be 256-byte aligned");
        out[4] = range(a.workspace, static_cast<int64_t>(need));
    }
    for (int i = 0; i < 5; ++i) {
        for (const Range& r : in)
            if (overlap(out[i], r)) return fail(PN_EINVAL, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(PN_EINVAL, "two outputs overlap");
    }
    return PN_OK;
}

}  // namespace

extern "C" {

int pn_rotary_table(const double* freq, int64_t n_freq, int64_t n_pos, double magnitude, float* table, void* stream) {
    clear_error();
    if (!freq) return fail(PN_EINVAL, "freq is NULL");
    if (n_freq < 1 || n_freq > 128) return fail(PN_EUNSUPPORTED, "1 .. 128 frequencies are supported");
    if (n_pos < 0 || !small_product({n_pos, n_freq}, int64_t(1) << 38)) return fail(PN_EINVAL, "n_pos out of range");
    for (int64_t i = 0; i < n_freq; ++i)
        if (!std::isfinite(freq[i])) return fail(PN_EINVAL, "a frequency is not finite");
    if (!std::isfinite(magnitude)) return fail(PN_EINVAL, "magnitude must be finite");
    if (n_pos == 0) return PN_OK;
    if (!table || reinterpret_cast<uintptr_t>(table) % 4) return fail(PN_EINVAL, "table is NULL or not aligned");
    return launched(launch_rotary_table(freq, static_cast<int>(n_freq), n_pos, magnitude, table,
                                        static_cast<hipStream_t>(stream)));
}

int pn_rotary(const pn_rotary_args* a) {
    PN_TRY(check_rotary(a, false, false));
    if (a->B == 0 || a->T == 0 || a->hq == 0) return PN_OK;
    return launched(launch_rotary(*a, kRotate, static_cast<hipStream_t>(a->stream)));
}

int pn_qk_norm_rotary(const pn_rotary_args* a) {
    PN_TRY(check_rotary(a, true, false));
    if (a->B == 0 || a->T == 0 || a->hq == 0) return PN_OK;
    pn_rotary_args f = *a;
    f.inverse = 0;
    return launched(launch_rotary(f, kNormRotate, static_cast<hipStream_t>(a->stream)));
}

size_t pn_qk_norm_rotary_workspace_bytes(const pn_rotary_args* a) {
    clear_error();
    if (!a) {
        fail(PN_EINVAL, "the arguments are NULL");
        return 0;
    }
    if (check_rotary_sizes(*a, true) != PN_OK) return 0;
    if (a->B == 0 || a->T == 0 || a->hq == 0) return kAlign;
    return norm_workspace(*a);
}

int pn_qk_norm_rotary_backward(const pn_rotary_args* a) {
    PN_TRY(check_rotary(a, true, true));
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    const bool empty = a->B == 0 || a->T == 0 || a->hq == 0;
    if (!empty) {
        const size_t need = norm_workspace(*a);
        if (!a->workspace || a->workspace_bytes < 0 || static_cast<size_t>(a->workspace_bytes) < need)
            return fail(PN_EWORKSPACE, "a workspace of %zu bytes is needed", need);
        if (reinterpret_cast<uintptr_t>(a->workspace) % kAlign)
            return fail(PN_EWORKSPACE, "workspace must be 256-byte aligned");
    }
    // no token, or k without heads: the weights' gradients are sums over nothing
    for (int k = 0; k < 2; ++k) {
        float* d = k ? a->dkw : a->dqw;
        const int64_t heads = k ? a->hk : a->hq;
        if (!d || !(k ? a->kw : a->qw) || !(empty || heads == 0)) continue;
        PN_TRY(launched(launch_fill(d, ((k ? a->kw_sh : a->qw_sh) ? heads : 1) * a->D, st)));
    }
    if (empty) return PN_OK;
    return launched(launch_rotary_backward(*a, st));
}

size_t pn_linear_attention_workspace_bytes(const pn_linattn_args* a, int32_t backward) {
    clear_error();
    if (!a) {
        fail(PN_EINVAL, "the arguments are NULL");
        return 0;
    }
    if (check_linattn_sizes(a->dtype, a->B, a->T, a->H, a->HK, a->dk, a->dv, a->scale) != PN_OK) return 0;
    if (a->B == 0 || a->H == 0) return kAlign;
    const LinattnPlan plan = plan_linattn(*a, backward != 0);
    if (!linattn_fits(plan.la)) {
        fail(PN_EUNSUPPORTED, "too many sequences and heads for one launch");
        return 0;
    }
    return plan.total > 0 ? plan.total : kAlign;
}

int pn_linear_attention(const pn_linattn_args* a) {
    PN_TRY(check_linattn(a, false));
    if (a->B == 0 || a->H == 0) return PN_OK;
    const LinattnPlan p = plan_linattn(*a, false);
    return launched(launch_linattn(p.la, static_cast<char*>(a->workspace) + p.off_carry, static_cast<hipStream_t>(a->stream)));
}

int pn_linear_attention_backward(const pn_linattn_args* a) {
    PN_TRY(check_linattn(a, true));
    if (a->B == 0 || a->H == 0) return PN_OK;
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    const LinattnPlan p = plan_linattn(*a, true);
    char* ws = static_cast<char*>(a->workspace);
    PN_TRY(launched(launch_linattn(p.la, ws + p.off_carry, st)));
    const int share = static_cast<int>(a->H / a->HK);
    if (share > 1 && a->T > 0) {
        const int64_t rows = a->B * a->T * a->HK;
        PN_TRY(launched(launch_group_sum(reinterpret_cast<float*>(ws + p.off_dk), a->dk_, p.la.dtype, rows, share,
                                         static_cast<int>(a->dk), st)));
        PN_TRY(launched(launch_group_sum(reinterpret_cast<float*>(ws + p.off_dv), a->dv_, p.la.dtype, rows, share,
                                         static_cast<int>(a->dv), st)));
    }
    return PN_OK;
}

int pn_linear_attention_step(const pn_linattn_step_args* p) {
    clear_error();
    if (!p) return fail(PN_EINVAL, "the arguments are NULL");
    const pn_linattn_step_args& a = *p;
    PN_TRY(check_linattn_sizes(a.dtype, a.B, 1, a.H, a.HK, a.dk, a.dv, a.scale));
    if (a.B * a.H * 256 >= int64_t(1) << 32) return fail(PN_EUNSUPPORTED, "too many sequences and heads for one launch");
    if (a.n_slots < 0 || a.n_slots > (int64_t(1) << 31)) return fail(PN_EINVAL, "n_slots out of range");
    if (a.B == 0 || a.H == 0) return PN_OK;
    const int64_t e = elem_bytes(a.dtype);
    PN_TRY(check_tokens(a.q, "q", e));
    PN_TRY(check_tokens(a.k, "k", e));
    PN_TRY(check_tokens(a.v, "v", e));
    if (!a.log_decay || !a.o) return fail(PN_EINVAL, "log_decay or o is NULL");
    if (!a.state && a.n_slots > 0) return fail(PN_EINVAL, "state is NULL");
    if (!a.slots && a.n_slots < a.B) return fail(PN_EINVAL, "fewer slots than sequences");
    if ((reinterpret_cast<uintptr_t>(a.log_decay) | reinterpret_cast<uintptr_t>(a.state) |
         reinterpret_cast<uintptr_t>(a.slots)) % 4 || reinterpret_cast<uintptr_t>(a.o) % e)
        return fail(PN_EINVAL, "an array is not aligned to its type");
    const Range in[] = {range(a.q, a.B, 1, a.H, a.dk, e), range(a.k, a.B, 1, a.HK, a.dk, e),
                        range(a.v, a.B, 1, a.HK, a.dv, e), range(a.log_decay, 4 * a.H), range(a.slots, 4 * a.B)};
    const Range o = range(a.o, e * a.B * a.H * a.dv), s = range(a.state, 4 * a.n_slots * a.H * a.dk * a.dv);
    for (const Range& r : in)
        if (overlap(o, r) || overlap(s, r)) return fail(PN_EINVAL, "an output overlaps an input");
    if (overlap(o, s)) return fail(PN_EINVAL, "two outputs overlap");
    return launched(launch_linattn_step(a, static_cast<hipStream_t>(a.stream)));
}

}  // extern "C"
