// C-ABI entry points of the selective state space scan, the short causal
// convolution, the group norm, linear attention and the layer norm: argument
// validation (before any HIP call) and dispatch to the kernel launchers.  See
// include/ssm.h, include/shortconv.h, include/groupnorm.h, include/linattn.h and
// include/layernorm.h for the contracts.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/layernorm.h"
#include "../../include/linattn.h"
#include "../../include/wkv7.h"
#include "layernorm.h"
#include "linattn/linattn_internal.h"
#include "seq_internal.h"
#include "wkv7_host.h"

namespace {

using namespace wkv7;

constexpr int64_t kMaxElems = int64_t(1) << 46;   // 64-bit offsets in bytes stay far from their end
constexpr int64_t kMaxItems = int64_t(1) << 30;   // workgroups of a launch, rows of a batch

// The arrays of one call, in the order they were named.
struct Arrays {
    struct Item {
        Span s;
        bool written;
    } it[28];
    int n = 0;

    // `need`: a NULL is an error where the array has bytes.  An optional array may be NULL.
    int add(const void* p, int64_t bytes, const char* name, bool need, bool written) {
        if (bytes > 0 && need && !p) return fail(WKV7_EINVAL, "%s is NULL", name);
        if (p && !aligned16(p)) return fail(WKV7_EINVAL, "%s is not 16-byte aligned", name);
        it[n++] = {{p, bytes, name}, written};
        return WKV7_OK;
    }
    // An optional array of int32 (its own alignment is checked with the descriptor).
    void index(const int32_t* p, int64_t count, const char* name) {
        if (p) it[n++] = {{p, count * 4, name}, false};
    }
    // Every written array shares no byte with another; with `in_place`, state_out may be state_in itself
    // (or another named pair the same).
    int disjoint(bool in_place = false, const char* moved = "state_out", const char* from = "state_in") const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < n; ++j) {
                if (i == j || !it[i].written || (it[j].written && j < i)) continue;
                const Span &x = it[i].s, &y = it[j].s;
                if (in_place && x.p == y.p && !std::strcmp(x.name, moved) && !std::strcmp(y.name, from)) continue;
                if (overlap(x.p, x.bytes, y.p, y.bytes)) return fail(WKV7_EINVAL, "%s overlaps %s", x.name, y.name);
            }
        return WKV7_OK;
    }
    int workspace(const void* ws, int64_t given, int64_t need) {
        if (need <= 0) return WKV7_OK;
        if (!ws) return fail(WKV7_EINVAL, "workspace is NULL (%lld bytes needed)", (long long)need);
        if (given < need)
            return fail(WKV7_EINVAL, "workspace has %lld bytes, %lld needed", (long long)given, (long long)need);
        return add(ws, need, "workspace", true, true);
    }
};

#define WKV7_TRY(call)           \
    do {                         \
        const int rc_ = (call);  \
        if (rc_) return rc_;     \
    } while (0)

int check_dtypes(int in, int y) {
    if (in != WKV7_F32 && in != WKV7_BF16) return fail(WKV7_EINVAL, "in_dtype %d unknown", in);
    if (y != WKV7_F32 && y != WKV7_BF16) return fail(WKV7_EINVAL, "y_dtype %d unknown", y);
    return WKV7_OK;
}
int check_lengths(const int32_t* lengths, bool allowed) {
    if (lengths && !allowed) return fail(WKV7_EINVAL, "lengths must be NULL for a step");
    if (reinterpret_cast<uintptr_t>(lengths) & 3u) return fail(WKV7_EINVAL, "lengths is not 4-byte aligned");
    return WKV7_OK;
}
int check_index(const int32_t* index, int B, int S) {
    if (reinterpret_cast<uintptr_t>(index) & 3u) return fail(WKV7_EINVAL, "state_index is not 4-byte aligned");
    if (S < 0) return fail(WKV7_EINVAL, "negative size (S=%d)", S);
    if (!index && S < B) return fail(WKV7_EINVAL, "S=%d states for B=%d rows without a state_index", S, B);
    return WKV7_OK;
}
int64_t esize(bool bf16) { return bf16 ? 2 : 4; }

int check_threads(int64_t threads) {
    if (threads >> 32) return fail(WKV7_EUNSUPPORTED, "the call needs %lld threads in one launch; less than 2^32 are supported", (long long)threads);
    return WKV7_OK;
}

// ---------------------------------------------------------------- scan

int ssm_desc_check(const ssm_desc* d, bool step, SsmParams* p) {
    if (!d) return fail(WKV7_EINVAL, "desc is NULL");
    if (d->B < 0 || d->T < 0 || d->C < 0 || d->G < 0)
        return fail(WKV7_EINVAL, "negative size (B=%d T=%d C=%d G=%d)", d->B, d->T, d->C, d->G);
    if (d->N <= 0) return fail(WKV7_EINVAL, "N must be positive (got %d)", d->N);
    if (d->N > 64) return fail(WKV7_EUNSUPPORTED, "N=%d; up to 64 states are supported", d->N);
    const int G = d->G ? d->G : 1;
    if (d->C % G) return fail(WKV7_EINVAL, "C=%d is not a multiple of G=%d", d->C, G);
    WKV7_TRY(check_dtypes(d->in_dtype, d->y_dtype));
    if (d->dt_softplus != 0 && d->dt_softplus != 1) return fail(WKV7_EINVAL, "dt_softplus must be 0 or 1 (got %d)", d->dt_softplus);
    if (d->reserved != 0) return fail(WKV7_EINVAL, "reserved must be 0 (got %d)", d->reserved);
    WKV7_TRY(check_lengths(d->lengths, !step));
    if (step && d->T != 1) return fail(WKV7_EINVAL, "ssm_step needs T == 1 (got %d)", d->T);
    const int64_t bt = int64_t(d->B) * d->T, bc = int64_t(d->B) * d->C;
    if (bt > kMaxElems / 64 / (d->C ? d->C : 1) || bc > kMaxItems || (step && int64_t(d->S) * d->C > kMaxElems / 64) ||
        d->T > INT32_MAX - 4096)
        return fail(WKV7_EUNSUPPORTED, "B=%d, T=%d, C=%d or S=%d too large", d->B, d->T, d->C, d->S);
    // Offsets within 128 rows are 32-bit.
    if (d->C >= (1 << 22) || int64_t(G) * d->N >= (1 << 22)) return fail(WKV7_EUNSUPPORTED, "C=%d or G*N=%lld too large", d->C, (long long)(int64_t(G) * d->N));
    if (bt > (int64_t(1) << 38) / (int64_t(G) * d->N)) return fail(WKV7_EUNSUPPORTED, "B*T*G*N too large");
    *p = SsmParams{};
    p->B = d->B; p->T = d->T; p->C = d->C; p->N = d->N; p->G = G; p->S = d->S;
    p->in_bf16 = d->in_dtype == WKV7_BF16; p->y_bf16 = d->y_dtype == WKV7_BF16; p->softplus = d->dt_softplus;
    p->lengths = d->lengths;
    p->nck = int((int64_t(d->T) + SSM_CHECKPOINT_TOKENS - 1) / SSM_CHECKPOINT_TOKENS);
    return WKV7_OK;
}
// The inputs of the three directions.
int ssm_inputs(const SsmParams& p, Arrays& a) {
    const int64_t e = esize(p.in_bf16), row = int64_t(p.B) * p.T * p.C, vec = int64_t(p.B) * p.T * p.G * p.N;
    const bool some = row > 0;
    WKV7_TRY(a.add(p.x, row * e, "x", true, false));
    WKV7_TRY(a.add(p.dt, row * e, "dt", true, false));
    WKV7_TRY(a.add(p.A, int64_t(p.C) * p.N * 4, "A", true, false));
    WKV7_TRY(a.add(p.Bm, some ? vec * e : 0, "Bm", true, false));
    WKV7_TRY(a.add(p.Cm, some ? vec * e : 0, "Cm", true, false));
    WKV7_TRY(a.add(p.D, int64_t(p.C) * 4, "D", false, false));
    WKV7_TRY(a.add(p.dt_bias, int64_t(p.C) * 4, "dt_bias", false, false));
    WKV7_TRY(a.add(p.z, row * e, "z", false, false));
    a.index(p.lengths, p.B, "lengths");
    return WKV7_OK;
}
int64_t ssm_ck_bytes(const SsmParams& p) { return int64_t(p.B) * p.nck * p.C * p.N * 4; }

// ---------------------------------------------------------------- convolution

int conv_desc_check(const shortconv_desc* d, bool step, ConvParams* p) {
    if (!d) return fail(WKV7_EINVAL, "desc is NULL");
    if (d->B < 0 || d->T < 0 || d->C < 0) return fail(WKV7_EINVAL, "negative size (B=%d T=%d C=%d)", d->B, d->T, d->C);
    if (d->K <= 0) return fail(WKV7_EINVAL, "K must be positive (got %d)", d->K);
    if (d->K < 2 || d->K > 4) return fail(WKV7_EUNSUPPORTED, "K=%d; 2, 3 and 4 taps are supported", d->K);
    WKV7_TRY(check_dtypes(d->in_dtype, d->y_dtype));
    if (d->act != SHORTCONV_NONE && d->act != SHORTCONV_SILU) return fail(WKV7_EINVAL, "act %d unknown", d->act);
    WKV7_TRY(check_lengths(d->lengths, !step));
    if (step && d->T != 1) return fail(WKV7_EINVAL, "shortconv_step needs T == 1 (got %d)", d->T);
    const int64_t bt = int64_t(d->B) * d->T, bc = int64_t(d->B) * d->C;
    // Threads and workgroups: at most one per 8 tokens of a channel.
    if (bt > kMaxElems / 64 / (d->C ? d->C : 1) || (bt / 8 + d->B) * d->C / 64 > kMaxItems || bc > kMaxItems ||
        (step && int64_t(d->S) * d->C > kMaxElems / 64) || d->T > INT32_MAX - 4096)
        return fail(WKV7_EUNSUPPORTED, "B=%d, T=%d, C=%d or S=%d too large", d->B, d->T, d->C, d->S);
    *p = ConvParams{};
    p->B = d->B; p->T = d->T; p->C = d->C; p->K = d->K; p->S = d->S;
    p->in_bf16 = d->in_dtype == WKV7_BF16; p->y_bf16 = d->y_dtype == WKV7_BF16; p->silu = d->act == SHORTCONV_SILU;
    p->lengths = d->lengths;
    return WKV7_OK;
}
int conv_inputs(const ConvParams& p, Arrays& a) {
    const int64_t row = int64_t(p.B) * p.T * p.C;
    WKV7_TRY(a.add(p.x, row * esize(p.in_bf16), "x", true, false));
    WKV7_TRY(a.add(p.w, int64_t(p.C) * p.K * 4, "w", row > 0, false));
    WKV7_TRY(a.add(p.bias, int64_t(p.C) * 4, "bias", false, false));
    a.index(p.lengths, p.B, "lengths");
    return WKV7_OK;
}

// ---------------------------------------------------------------- norm

int norm_desc_check(const groupnorm_desc* d, NormParams* p) {
    if (!d) return fail(WKV7_EINVAL, "desc is NULL");
    if (d->B < 0 || d->T < 0 || d->C < 0) return fail(WKV7_EINVAL, "negative size (B=%d T=%d C=%d)", d->B, d->T, d->C);
    if (d->G <= 0) return fail(WKV7_EINVAL, "G must be positive (got %d)", d->G);
    if (d->C % d->G) return fail(WKV7_EINVAL, "C=%d is not a multiple of G=%d", d->C, d->G);
    WKV7_TRY(check_dtypes(d->in_dtype, d->y_dtype));
    if (d->act != GROUPNORM_NONE && d->act != GROUPNORM_SILU) return fail(WKV7_EINVAL, "act %d unknown", d->act);
    if (!std::isfinite(d->eps) || d->eps <= 0.f) return fail(WKV7_EINVAL, "eps must be positive and finite");
    WKV7_TRY(check_lengths(d->lengths, true));
    const int64_t bt = int64_t(d->B) * d->T, n = bt / 64 + d->B;
    if (bt > kMaxElems / 64 / (d->C ? d->C : 1) || n * (d->C / 256 + 1) > kMaxItems || int64_t(d->B) * d->G > kMaxItems ||
        d->T > INT32_MAX - 4096)
        return fail(WKV7_EUNSUPPORTED, "B=%d, T=%d or C=%d too large", d->B, d->T, d->C);
    *p = NormParams{};
    p->B = d->B; p->T = d->T; p->C = d->C; p->G = d->G;
    p->in_bf16 = d->in_dtype == WKV7_BF16; p->y_bf16 = d->y_dtype == WKV7_BF16; p->silu = d->act == GROUPNORM_SILU;
    p->eps = d->eps; p->lengths = d->lengths;
    return WKV7_OK;
}
int norm_inputs(const NormParams& p, Arrays& a) {
    const int64_t row = int64_t(p.B) * p.T * p.C;
    WKV7_TRY(a.add(p.x, row * esize(p.in_bf16), "x", true, false));
    WKV7_TRY(a.add(p.weight, int64_t(p.C) * 4, "weight", false, false));
    WKV7_TRY(a.add(p.bias, int64_t(p.C) * 4, "bias", false, false));
    WKV7_TRY(a.add(p.gate, row * esize(p.in_bf16), "gate", false, false));
    a.index(p.lengths, p.B, "lengths");
    return WKV7_OK;
}

// ---------------------------------------------------------------- linear attention

int linattn_desc_check(const linattn_desc* d, bool step, LinAttnParams* p) {
    if (!d) return fail(WKV7_EINVAL, "desc is NULL");
    if (d->B < 0 || d->T < 0 || d->H < 0 || d->Hq < 0 || d->Hk < 0 || d->Hv < 0)
        return fail(WKV7_EINVAL, "negative size (B=%d T=%d H=%d Hq=%d Hk=%d Hv=%d)", d->B, d->T, d->H, d->Hq, d->Hk, d->Hv);
    if (d->Dk <= 0 || d->Dv <= 0) return fail(WKV7_EINVAL, "Dk and Dv must be positive (got %d and %d)", d->Dk, d->Dv);
    if (d->Dk > 128 || d->Dv > 128) return fail(WKV7_EUNSUPPORTED, "Dk=%d, Dv=%d; up to 128 are supported", d->Dk, d->Dv);
    const int Hq = d->Hq ? d->Hq : d->H, Hk = d->Hk ? d->Hk : d->H, Hv = d->Hv ? d->Hv : d->H;
    if (d->H ? d->H % Hq || d->H % Hk || d->H % Hv : Hq || Hk || Hv)
        return fail(WKV7_EINVAL, "Hq=%d, Hk=%d and Hv=%d must divide H=%d", Hq, Hk, Hv, d->H);
    WKV7_TRY(check_dtypes(d->in_dtype, d->y_dtype));
    if (d->g_per_token != 0 && d->g_per_token != 1) return fail(WKV7_EINVAL, "g_per_token must be 0 or 1 (got %d)", d->g_per_token);
    if (!std::isfinite(d->scale)) return fail(WKV7_EINVAL, "scale must be finite");
    if (d->reserved != 0) return fail(WKV7_EINVAL, "reserved must be 0 (got %d)", d->reserved);
    WKV7_TRY(check_lengths(d->lengths, !step));
    if (step && d->T != 1) return fail(WKV7_EINVAL, "linattn_step needs T == 1 (got %d)", d->T);
    // Offsets within 64 rows are 32-bit.
    if (d->H > (1 << 14)) return fail(WKV7_EUNSUPPORTED, "H=%d; up to 16384 heads are supported", d->H);
    const int64_t bt = int64_t(d->B) * d->T, state = int64_t(d->H) * d->Dk * d->Dv;
    if (bt > kMaxElems / 128 / (d->H ? d->H : 1) || int64_t(d->B) * d->H > kMaxItems || (state && d->B > kMaxElems / state) ||
        (step && state && d->S > kMaxElems / state) || d->T > INT32_MAX - 4096)
        return fail(WKV7_EUNSUPPORTED, "B=%d, T=%d, H=%d or S=%d too large", d->B, d->T, d->H, d->S);
    *p = LinAttnParams{};
    p->B = d->B; p->T = d->T; p->H = d->H; p->Hq = Hq; p->Hk = Hk; p->Hv = Hv; p->Dk = d->Dk; p->Dv = d->Dv; p->S = d->S;
    p->in_bf16 = d->in_dtype == WKV7_BF16; p->y_bf16 = d->y_dtype == WKV7_BF16; p->g_per_token = d->g_per_token;
    p->scale = d->scale; p->lengths = d->lengths;
    return WKV7_OK;
}
int64_t linattn_rows(const LinAttnParams& p) { return int64_t(p.B) * p.T; }
int64_t linattn_state_bytes(const LinAttnParams& p) { return int64_t(p.B) * p.H * p.Dk * p.Dv * 4; }
int64_t linattn_g_bytes(const LinAttnParams& p) { return (p.g_per_token ? linattn_rows(p) : 1) * p.H * 4; }
int linattn_inputs(const LinAttnParams& p, Arrays& a) {
    const int64_t e = esize(p.in_bf16), rows = linattn_rows(p);
    WKV7_TRY(a.add(p.q, rows * p.Hq * p.Dk * e, "q", true, false));
    WKV7_TRY(a.add(p.k, rows * p.Hk * p.Dk * e, "k", true, false));
    WKV7_TRY(a.add(p.v, rows * p.Hv * p.Dv * e, "v", true, false));
    WKV7_TRY(a.add(p.g, linattn_g_bytes(p), "g", rows > 0, false));
    a.index(p.lengths, p.B, "lengths");
    return WKV7_OK;
}

// ---------------------------------------------------------------- layer norm

int layernorm_desc_check(const layernorm_desc* d, LayerNormParams* p) {
    if (!d) return fail(WKV7_EINVAL, "desc is NULL");
    if (d->B < 0 || d->T < 0 || d->C < 0) return fail(WKV7_EINVAL, "negative size (B=%d T=%d C=%d)", d->B, d->T, d->C);
    if (d->x_dtype != WKV7_F32 && d->x_dtype != WKV7_BF16) return fail(WKV7_EINVAL, "x_dtype %d unknown", d->x_dtype);
    if (d->h_dtype != WKV7_F32 && d->h_dtype != WKV7_BF16) return fail(WKV7_EINVAL, "h_dtype %d unknown", d->h_dtype);
    if (d->y_dtype != WKV7_F32 && d->y_dtype != WKV7_BF16) return fail(WKV7_EINVAL, "y_dtype %d unknown", d->y_dtype);
    if (!std::isfinite(d->eps) || d->eps <= 0.f) return fail(WKV7_EINVAL, "eps must be positive and finite");
    if (d->reserved != 0) return fail(WKV7_EINVAL, "reserved must be 0 (got %d)", d->reserved);
    WKV7_TRY(check_lengths(d->lengths, true));
    if (int64_t(d->B) * d->T > kMaxElems / 64 / (d->C ? d->C : 1) || d->C >= (1 << 24))
        return fail(WKV7_EUNSUPPORTED, "B=%d, T=%d or C=%d too large", d->B, d->T, d->C);
    *p = LayerNormParams{};
    p->B = d->B; p->T = d->T; p->C = d->C;
    p->x_bf16 = d->x_dtype == WKV7_BF16; p->h_bf16 = d->h_dtype == WKV7_BF16; p->y_bf16 = d->y_dtype == WKV7_BF16;
    p->eps = d->eps; p->lengths = d->lengths;
    return WKV7_OK;
}

hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int64_t ssm_checkpoint_bytes(const ssm_desc* desc) {
    g_last_error[0] = '\0';
    SsmParams p;
    const int rc = ssm_desc_check(desc, false, &p);
    return rc ? -rc : ssm_ck_bytes(p);
}

int ssm_forward(const ssm_desc* desc, const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                const float* D, const float* dt_bias, const void* z, const float* state_in, void* y, float* state_out,
                float* checkpoints, void* stream) {
    g_last_error[0] = '\0';
    SsmParams p;
    WKV7_TRY(ssm_desc_check(desc, false, &p));
    p.x = x; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.D = D; p.dt_bias = dt_bias; p.z = z;
    p.s0 = state_in; p.y = y; p.s1 = state_out; p.ck = checkpoints;
    Arrays a;
    const int64_t st = int64_t(p.B) * p.C * p.N * 4;
    WKV7_TRY(ssm_inputs(p, a));
    WKV7_TRY(a.add(state_in, st, "state_in", false, false));
    WKV7_TRY(a.add(y, int64_t(p.B) * p.T * p.C * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.add(state_out, st, "state_out", false, true));
    WKV7_TRY(a.add(checkpoints, ssm_ck_bytes(p), "checkpoints", false, true));
    WKV7_TRY(a.disjoint(true));
    if (int64_t(p.B) * p.C == 0 || (p.T == 0 && !state_out)) return WKV7_OK;
    WKV7_TRY(check_threads(ssm_forward_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_ssm_forward(p, stream_of(stream)), "ssm");
}

int ssm_step(const ssm_desc* desc, const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
             const float* D, const float* dt_bias, const void* z, float* state, const int32_t* state_index, void* y,
             void* stream) {
    g_last_error[0] = '\0';
    SsmParams p;
    WKV7_TRY(ssm_desc_check(desc, true, &p));
    WKV7_TRY(check_index(state_index, p.B, p.S));
    p.x = x; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.D = D; p.dt_bias = dt_bias; p.z = z;
    p.s0 = state; p.s1 = state; p.index = state_index; p.y = y;
    Arrays a;
    WKV7_TRY(ssm_inputs(p, a));
    a.index(state_index, p.B, "state_index");
    WKV7_TRY(a.add(state, int64_t(p.B) * p.C == 0 ? 0 : int64_t(p.S) * p.C * p.N * 4, "state", true, true));
    WKV7_TRY(a.add(y, int64_t(p.B) * p.C * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.disjoint());
    if (int64_t(p.B) * p.C == 0) return WKV7_OK;
    WKV7_TRY(check_threads(ssm_step_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_ssm_step(p, stream_of(stream)), "ssm step");
}

int64_t ssm_backward_workspace_bytes(const ssm_desc* desc, int without_checkpoints) {
    g_last_error[0] = '\0';
    SsmParams p;
    const int rc = ssm_desc_check(desc, false, &p);
    return rc ? -rc : ssm_backward_workspace(p, without_checkpoints != 0);
}

int ssm_backward(const ssm_desc* desc, const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                 const float* D, const float* dt_bias, const void* z, const float* state_in, const void* dy,
                 const float* dstate_out, const float* checkpoints, void* dx, void* ddt, float* dA, void* dBm, void* dCm,
                 float* dD, float* ddt_bias, void* dz, float* dstate_in, void* workspace, int64_t workspace_bytes,
                 void* stream) {
    g_last_error[0] = '\0';
    SsmParams p;
    WKV7_TRY(ssm_desc_check(desc, false, &p));
    p.x = x; p.dt = dt; p.A = A; p.Bm = Bm; p.Cm = Cm; p.D = D; p.dt_bias = dt_bias; p.z = z;
    p.s0 = state_in; p.dy = dy; p.ds1 = dstate_out; p.ck = const_cast<float*>(checkpoints);
    p.dx = dx; p.ddt = ddt; p.dA = dA; p.dBm = dBm; p.dCm = dCm; p.dD = dD; p.dbias = ddt_bias; p.dz = dz;
    p.ds0 = dstate_in; p.ws = workspace;
    Arrays a;
    const int64_t e = esize(p.in_bf16), row = int64_t(p.B) * p.T * p.C, st = int64_t(p.B) * p.C * p.N * 4;
    const int64_t vec = int64_t(p.B) * p.T * p.G * p.N * e;   // there without channels too
    WKV7_TRY(ssm_inputs(p, a));
    WKV7_TRY(a.add(state_in, st, "state_in", false, false));
    WKV7_TRY(a.add(dy, row * esize(p.y_bf16), "dy", true, false));
    WKV7_TRY(a.add(dstate_out, st, "dstate_out", false, false));
    WKV7_TRY(a.add(checkpoints, ssm_ck_bytes(p), "checkpoints", false, false));
    if (row > 0 && z && !dz) return fail(WKV7_EINVAL, "dz is NULL but z is given");
    if (row > 0 && !z && dz) return fail(WKV7_EINVAL, "dz is given but z is NULL");
    if (p.C > 0 && D && !dD) return fail(WKV7_EINVAL, "dD is NULL but D is given");
    if (p.C > 0 && dt_bias && !ddt_bias) return fail(WKV7_EINVAL, "ddt_bias is NULL but dt_bias is given");
    WKV7_TRY(a.add(dx, row * e, "dx", true, true));
    WKV7_TRY(a.add(ddt, row * e, "ddt", true, true));
    WKV7_TRY(a.add(dA, int64_t(p.C) * p.N * 4, "dA", true, true));
    WKV7_TRY(a.add(dBm, vec, "dBm", true, true));
    WKV7_TRY(a.add(dCm, vec, "dCm", true, true));
    WKV7_TRY(a.add(dD, int64_t(p.C) * 4, "dD", false, true));
    WKV7_TRY(a.add(ddt_bias, int64_t(p.C) * 4, "ddt_bias", false, true));
    WKV7_TRY(a.add(dz, row * e, "dz", false, true));
    WKV7_TRY(a.add(dstate_in, st, "dstate_in", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, ssm_backward_workspace(p, !checkpoints)));
    WKV7_TRY(a.disjoint());
    if (p.C == 0 && vec == 0) return WKV7_OK;
    WKV7_TRY(check_threads(ssm_backward_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_ssm_backward(p, stream_of(stream)), "ssm backward");
}

int shortconv_forward(const shortconv_desc* desc, const void* x, const float* w, const float* bias, const void* state_in,
                      void* y, void* state_out, void* stream) {
    g_last_error[0] = '\0';
    ConvParams p;
    WKV7_TRY(conv_desc_check(desc, false, &p));
    p.x = x; p.w = w; p.bias = bias; p.s0 = state_in; p.y = y; p.s1 = state_out;
    Arrays a;
    const int64_t st = int64_t(p.B) * (p.K - 1) * p.C * esize(p.in_bf16);
    WKV7_TRY(conv_inputs(p, a));
    WKV7_TRY(a.add(state_in, st, "state_in", false, false));
    WKV7_TRY(a.add(y, int64_t(p.B) * p.T * p.C * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.add(state_out, st, "state_out", false, true));
    WKV7_TRY(a.disjoint(true));
    if (int64_t(p.B) * p.C == 0) return WKV7_OK;
    WKV7_TRY(check_threads(shortconv_forward_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_shortconv_forward(p, stream_of(stream)), "shortconv");
}

int shortconv_step(const shortconv_desc* desc, const void* x, const float* w, const float* bias, void* state,
                   const int32_t* state_index, void* y, void* stream) {
    g_last_error[0] = '\0';
    ConvParams p;
    WKV7_TRY(conv_desc_check(desc, true, &p));
    WKV7_TRY(check_index(state_index, p.B, p.S));
    p.x = x; p.w = w; p.bias = bias; p.s0 = state; p.s1 = state; p.index = state_index; p.y = y;
    Arrays a;
    WKV7_TRY(conv_inputs(p, a));
    a.index(state_index, p.B, "state_index");
    WKV7_TRY(a.add(state, int64_t(p.B) * p.C == 0 ? 0 : int64_t(p.S) * (p.K - 1) * p.C * esize(p.in_bf16), "state", true, true));
    WKV7_TRY(a.add(y, int64_t(p.B) * p.C * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.disjoint());
    if (int64_t(p.B) * p.C == 0) return WKV7_OK;
    WKV7_TRY(check_threads(shortconv_step_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_shortconv_step(p, stream_of(stream)), "shortconv step");
}

int64_t shortconv_backward_workspace_bytes(const shortconv_desc* desc) {
    g_last_error[0] = '\0';
    ConvParams p;
    const int rc = conv_desc_check(desc, false, &p);
    return rc ? -rc : shortconv_backward_workspace(p);
}

int shortconv_backward(const shortconv_desc* desc, const void* x, const float* w, const float* bias, const void* state_in,
                       const void* dy, const float* dstate_out, void* dx, float* dw, float* dbias, float* dstate_in,
                       void* workspace, int64_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    ConvParams p;
    WKV7_TRY(conv_desc_check(desc, false, &p));
    p.x = x; p.w = w; p.bias = bias; p.s0 = state_in; p.dy = dy; p.ds1 = dstate_out;
    p.dx = dx; p.dw = dw; p.dbias = dbias; p.ds0 = dstate_in; p.ws = workspace;
    Arrays a;
    const int64_t row = int64_t(p.B) * p.T * p.C, st = int64_t(p.B) * (p.K - 1) * p.C;
    WKV7_TRY(conv_inputs(p, a));
    WKV7_TRY(a.add(state_in, st * esize(p.in_bf16), "state_in", false, false));
    WKV7_TRY(a.add(dy, row * esize(p.y_bf16), "dy", true, false));
    WKV7_TRY(a.add(dstate_out, st * 4, "dstate_out", false, false));
    if (p.C > 0 && bias && !dbias) return fail(WKV7_EINVAL, "dbias is NULL but bias is given");
    WKV7_TRY(a.add(dx, row * esize(p.in_bf16), "dx", true, true));
    WKV7_TRY(a.add(dw, int64_t(p.C) * p.K * 4, "dw", true, true));
    WKV7_TRY(a.add(dbias, int64_t(p.C) * 4, "dbias", false, true));
    WKV7_TRY(a.add(dstate_in, st * 4, "dstate_in", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, shortconv_backward_workspace(p)));
    WKV7_TRY(a.disjoint());
    if (p.C == 0) return WKV7_OK;
    WKV7_TRY(check_threads(shortconv_backward_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_shortconv_backward(p, stream_of(stream)), "shortconv backward");
}

int64_t groupnorm_workspace_bytes(const groupnorm_desc* desc) {
    g_last_error[0] = '\0';
    NormParams p;
    const int rc = norm_desc_check(desc, &p);
    return rc ? -rc : groupnorm_workspace(p);
}

int groupnorm_forward(const groupnorm_desc* desc, const void* x, const float* weight, const float* bias, const void* gate,
                      void* y, float* mean, float* rstd, void* workspace, int64_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    NormParams p;
    WKV7_TRY(norm_desc_check(desc, &p));
    p.x = x; p.weight = weight; p.bias = bias; p.gate = gate; p.y = y; p.mean = mean; p.rstd = rstd; p.ws = workspace;
    Arrays a;
    const int64_t st = int64_t(p.B) * p.G * 4;
    WKV7_TRY(norm_inputs(p, a));
    if (!mean != !rstd) return fail(WKV7_EINVAL, "mean and rstd go together: one of them is NULL");
    WKV7_TRY(a.add(y, int64_t(p.B) * p.T * p.C * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.add(mean, st, "mean", false, true));
    WKV7_TRY(a.add(rstd, st, "rstd", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, groupnorm_workspace(p)));
    WKV7_TRY(a.disjoint());
    if (p.B == 0 || (int64_t(p.T) * p.C == 0 && !mean)) return WKV7_OK;
    WKV7_TRY(check_threads(groupnorm_threads(p, false)));
    WKV7_TRY(check_device());
    return finish_launch(launch_groupnorm_forward(p, stream_of(stream)), "groupnorm");
}

int64_t groupnorm_backward_workspace_bytes(const groupnorm_desc* desc) {
    g_last_error[0] = '\0';
    NormParams p;
    const int rc = norm_desc_check(desc, &p);
    return rc ? -rc : groupnorm_backward_workspace(p);
}

int groupnorm_backward(const groupnorm_desc* desc, const void* x, const float* weight, const float* bias, const void* gate,
                       const void* dy, const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                       void* dgate, void* workspace, int64_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    NormParams p;
    WKV7_TRY(norm_desc_check(desc, &p));
    p.x = x; p.weight = weight; p.bias = bias; p.gate = gate; p.dy = dy;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dx = dx; p.dweight = dweight; p.dbias = dbias; p.dgate = dgate; p.ws = workspace;
    Arrays a;
    const int64_t row = int64_t(p.B) * p.T * p.C, e = esize(p.in_bf16), st = row > 0 ? int64_t(p.B) * p.G * 4 : 0;
    WKV7_TRY(norm_inputs(p, a));
    WKV7_TRY(a.add(dy, row * esize(p.y_bf16), "dy", true, false));
    WKV7_TRY(a.add(mean, st, "mean", true, false));
    WKV7_TRY(a.add(rstd, st, "rstd", true, false));
    if (p.C > 0 && weight && !dweight) return fail(WKV7_EINVAL, "dweight is NULL but weight is given");
    if (p.C > 0 && bias && !dbias) return fail(WKV7_EINVAL, "dbias is NULL but bias is given");
    if (row > 0 && !gate != !dgate) return fail(WKV7_EINVAL, "gate and dgate go together: one of them is NULL");
    WKV7_TRY(a.add(dx, row * e, "dx", true, true));
    WKV7_TRY(a.add(dweight, int64_t(p.C) * 4, "dweight", false, true));
    WKV7_TRY(a.add(dbias, int64_t(p.C) * 4, "dbias", false, true));
    WKV7_TRY(a.add(dgate, row * e, "dgate", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, groupnorm_backward_workspace(p)));
    WKV7_TRY(a.disjoint());
    if (p.C == 0) return WKV7_OK;
    WKV7_TRY(check_threads(groupnorm_threads(p, true)));
    WKV7_TRY(check_device());
    return finish_launch(launch_groupnorm_backward(p, stream_of(stream)), "groupnorm backward");
}

int64_t linattn_workspace_bytes(const linattn_desc* desc) {
    g_last_error[0] = '\0';
    LinAttnParams p;
    const int rc = linattn_desc_check(desc, false, &p);
    return rc ? -rc : linattn_forward_workspace(p);
}

int linattn_forward(const linattn_desc* desc, const void* q, const void* k, const void* v, const float* g,
                    const float* state_in, void* y, float* state_out, void* workspace, int64_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    LinAttnParams p;
    WKV7_TRY(linattn_desc_check(desc, false, &p));
    p.q = q; p.k = k; p.v = v; p.g = g; p.s0 = state_in; p.y = y; p.s1 = state_out; p.ws = workspace;
    Arrays a;
    WKV7_TRY(linattn_inputs(p, a));
    WKV7_TRY(a.add(state_in, linattn_state_bytes(p), "state_in", false, false));
    WKV7_TRY(a.add(y, linattn_rows(p) * p.H * p.Dv * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.add(state_out, linattn_state_bytes(p), "state_out", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, linattn_forward_workspace(p)));
    WKV7_TRY(a.disjoint(true));
    if (int64_t(p.B) * p.H == 0 || (p.T == 0 && !state_out)) return WKV7_OK;
    WKV7_TRY(check_threads(linattn_forward_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_linattn_forward(p, stream_of(stream)), "linattn");
}

int linattn_step(const linattn_desc* desc, const void* q, const void* k, const void* v, const float* g, float* state,
                 const int32_t* state_index, void* y, void* stream) {
    g_last_error[0] = '\0';
    LinAttnParams p;
    WKV7_TRY(linattn_desc_check(desc, true, &p));
    WKV7_TRY(check_index(state_index, p.B, p.S));
    p.q = q; p.k = k; p.v = v; p.g = g; p.s1 = state; p.index = state_index; p.y = y;
    Arrays a;
    const bool some = int64_t(p.B) * p.H > 0;
    WKV7_TRY(linattn_inputs(p, a));
    a.index(state_index, p.B, "state_index");
    WKV7_TRY(a.add(state, some ? int64_t(p.S) * p.H * p.Dk * p.Dv * 4 : 0, "state", true, true));
    WKV7_TRY(a.add(y, linattn_rows(p) * p.H * p.Dv * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.disjoint());
    if (!some) return WKV7_OK;
    WKV7_TRY(check_threads(linattn_step_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_linattn_step(p, stream_of(stream)), "linattn step");
}

int64_t linattn_backward_workspace_bytes(const linattn_desc* desc) {
    g_last_error[0] = '\0';
    LinAttnParams p;
    const int rc = linattn_desc_check(desc, false, &p);
    return rc ? -rc : linattn_backward_workspace(p);
}

int linattn_backward(const linattn_desc* desc, const void* q, const void* k, const void* v, const float* g,
                     const float* state_in, const void* dy, const float* dstate_out, void* dq, void* dk, void* dv, float* dg,
                     float* dstate_in, void* workspace, int64_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    LinAttnParams p;
    WKV7_TRY(linattn_desc_check(desc, false, &p));
    p.q = q; p.k = k; p.v = v; p.g = g; p.s0 = state_in; p.dy = dy; p.ds1 = dstate_out;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.ds0 = dstate_in; p.ws = workspace;
    Arrays a;
    const int64_t e = esize(p.in_bf16), rows = linattn_rows(p);
    WKV7_TRY(linattn_inputs(p, a));
    WKV7_TRY(a.add(state_in, linattn_state_bytes(p), "state_in", false, false));
    WKV7_TRY(a.add(dy, rows * p.H * p.Dv * esize(p.y_bf16), "dy", true, false));
    WKV7_TRY(a.add(dstate_out, linattn_state_bytes(p), "dstate_out", false, false));
    WKV7_TRY(a.add(dq, rows * p.Hq * p.Dk * e, "dq", true, true));
    WKV7_TRY(a.add(dk, rows * p.Hk * p.Dk * e, "dk", true, true));
    WKV7_TRY(a.add(dv, rows * p.Hv * p.Dv * e, "dv", true, true));
    WKV7_TRY(a.add(dg, linattn_g_bytes(p), "dg", false, true));
    WKV7_TRY(a.add(dstate_in, linattn_state_bytes(p), "dstate_in", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, linattn_backward_workspace(p)));
    WKV7_TRY(a.disjoint());
    if (p.H == 0) return WKV7_OK;
    WKV7_TRY(check_threads(linattn_backward_threads(p)));
    WKV7_TRY(check_device());
    return finish_launch(launch_linattn_backward(p, stream_of(stream)), "linattn backward");
}

int layernorm_forward(const layernorm_desc* desc, const void* x, const void* residual, const float* weight, const float* bias,
                      void* h, void* y, float* mean, float* rstd, void* stream) {
    g_last_error[0] = '\0';
    LayerNormParams p;
    WKV7_TRY(layernorm_desc_check(desc, &p));
    p.x = x; p.res = residual; p.weight = weight; p.bias = bias; p.h = h; p.y = y; p.mean = mean; p.rstd = rstd;
    Arrays a;
    const int64_t rows = int64_t(p.B) * p.T, n = rows * p.C;
    if (n > 0 && !residual != !h) return fail(WKV7_EINVAL, "residual and h go together: one of them is NULL");
    if (!residual && p.x_bf16 != p.h_bf16) return fail(WKV7_EINVAL, "h_dtype differs from x_dtype without a residual");
    if (!mean != !rstd) return fail(WKV7_EINVAL, "mean and rstd go together: one of them is NULL");
    WKV7_TRY(a.add(x, n * esize(p.x_bf16), "x", true, false));
    WKV7_TRY(a.add(residual, n * esize(p.h_bf16), "residual", false, false));
    WKV7_TRY(a.add(weight, int64_t(p.C) * 4, "weight", false, false));
    WKV7_TRY(a.add(bias, int64_t(p.C) * 4, "bias", false, false));
    a.index(p.lengths, p.B, "lengths");
    WKV7_TRY(a.add(h, n * esize(p.h_bf16), "h", false, true));
    WKV7_TRY(a.add(y, n * esize(p.y_bf16), "y", true, true));
    WKV7_TRY(a.add(mean, rows * 4, "mean", false, true));
    WKV7_TRY(a.add(rstd, rows * 4, "rstd", false, true));
    WKV7_TRY(a.disjoint(true, "h", "residual"));
    if (rows == 0 || (p.C == 0 && !mean)) return WKV7_OK;
    WKV7_TRY(check_threads(layernorm_threads(p, false)));
    WKV7_TRY(check_device());
    return finish_launch(launch_layernorm_forward(p, stream_of(stream)), "layernorm");
}

int64_t layernorm_backward_workspace_bytes(const layernorm_desc* desc) {
    g_last_error[0] = '\0';
    LayerNormParams p;
    const int rc = layernorm_desc_check(desc, &p);
    return rc ? -rc : layernorm_backward_workspace(p);
}

int layernorm_backward(const layernorm_desc* desc, const void* h, const float* weight, const float* bias, const void* dy,
                       const void* dh, const float* mean, const float* rstd, void* dresidual, void* dx, float* dweight,
                       float* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    LayerNormParams p;
    WKV7_TRY(layernorm_desc_check(desc, &p));
    p.h = const_cast<void*>(h); p.weight = weight; p.bias = bias; p.dy = dy; p.dh = dh;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dres = dresidual; p.dx = dx; p.dweight = dweight; p.dbias = dbias; p.ws = workspace;
    Arrays a;
    const int64_t rows = int64_t(p.B) * p.T, n = rows * p.C;
    if (p.C > 0 && weight && !dweight) return fail(WKV7_EINVAL, "dweight is NULL but weight is given");
    if (p.C > 0 && bias && !dbias) return fail(WKV7_EINVAL, "dbias is NULL but bias is given");
    WKV7_TRY(a.add(h, n * esize(p.h_bf16), "h", true, false));
    WKV7_TRY(a.add(weight, int64_t(p.C) * 4, "weight", false, false));
    WKV7_TRY(a.add(bias, int64_t(p.C) * 4, "bias", false, false));
    a.index(p.lengths, p.B, "lengths");
    WKV7_TRY(a.add(dy, n * esize(p.y_bf16), "dy", true, false));
    WKV7_TRY(a.add(dh, n * esize(p.h_bf16), "dh", false, false));
    WKV7_TRY(a.add(mean, n > 0 ? rows * 4 : 0, "mean", true, false));
    WKV7_TRY(a.add(rstd, n > 0 ? rows * 4 : 0, "rstd", true, false));
    WKV7_TRY(a.add(dresidual, n * esize(p.h_bf16), "dresidual", true, true));
    WKV7_TRY(a.add(dx, n * esize(p.x_bf16), "dx", false, true));
    WKV7_TRY(a.add(dweight, int64_t(p.C) * 4, "dweight", false, true));
    WKV7_TRY(a.add(dbias, int64_t(p.C) * 4, "dbias", false, true));
    WKV7_TRY(a.workspace(workspace, workspace_bytes, layernorm_backward_workspace(p)));
    WKV7_TRY(a.disjoint(true, "dresidual", "dh"));
    if (p.C == 0) return WKV7_OK;
    WKV7_TRY(check_threads(layernorm_threads(p, true)));
    WKV7_TRY(check_device());
    return finish_launch(launch_layernorm_backward(p, stream_of(stream)), "layernorm backward");
}

}  // extern "C"
