// gdn_abi.hip -- the extern "C" entry points of libgdn (declared in
// include/gdn.h): argument validation on the host, then one launch on the
// caller's stream.  Nothing is allocated, nothing is synchronised.
//
// Every check happens before any launch, because a device fault takes the
// whole context down with it (the pages report exactly that failure mode:
// atlas PR #297, commit message on the illegal-address crash that poisoned
// the CUDA context).
#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv_internal.h"
#include "gdn_window_internal.h"

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return code;
}

int ok()
{
    g_err[0] = '\0';
    return GDN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(Span a, Span b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

int launch_status(hipError_t e, const char* what)
{
    if (e != hipSuccess) return fail(GDN_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

size_t elem_size(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

bool valid_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }

#define REQUIRE(cond, code, ...)          \
    do {                                  \
        if (!(cond)) return fail(code, __VA_ARGS__); \
    } while (0)

// shared checks of the GDN shapes (verify and prefill)
int check_gdn_shape(const char* fn, int B, int K, int Hk, int Hv, int dk, int dv, int in_dtype, int o_dtype,
                    float eps)
{
    REQUIRE(B >= 0, GDN_EINVAL, "%s: B = %d < 0", fn, B);
    REQUIRE(K >= 1, GDN_EINVAL, "%s: token count %d < 1", fn, K);
    REQUIRE(Hk >= 1 && Hv >= 1, GDN_EINVAL, "%s: Hk = %d, Hv = %d must be >= 1", fn, Hk, Hv);
    REQUIRE(Hv % Hk == 0, GDN_EINVAL, "%s: Hv = %d is not a multiple of Hk = %d", fn, Hv, Hk);
    REQUIRE(dk >= 1 && dv >= 1, GDN_EINVAL, "%s: dk = %d, dv = %d must be >= 1", fn, dk, dv);
    REQUIRE(dk == 32 || dk == 64 || dk == 128, GDN_EUNSUPPORTED, "%s: dk = %d not in {32, 64, 128}", fn, dk);
    REQUIRE(dv % 8 == 0, GDN_EUNSUPPORTED, "%s: dv = %d is not a multiple of 8", fn, dv);
    REQUIRE(valid_dtype(in_dtype) && valid_dtype(o_dtype), GDN_EINVAL, "%s: bad dtype code (%d, %d)", fn,
            in_dtype, o_dtype);
    REQUIRE(eps >= 0.0f, GDN_EINVAL, "%s: l2_eps < 0", fn);
    return GDN_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// shared checks of the cache's geometry; fills g
int check_kv(const char* fn, int planes, int n_pages, int Hkv, int page, int D, int dtype, gdn::KvGeom& g)
{
    REQUIRE(valid_dtype(dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, dtype);
    REQUIRE(planes >= 1 && n_pages >= 1 && Hkv >= 1, GDN_EINVAL, "%s: planes = %d, n_pages = %d, Hkv = %d must be >= 1",
            fn, planes, n_pages, Hkv);
    REQUIRE(page >= 1, GDN_EINVAL, "%s: page = %d < 1", fn, page);
    REQUIRE(D == 64 || D == 128 || D == 256, GDN_EUNSUPPORTED, "%s: D = %d not in {64, 128, 256}", fn, D);
    REQUIRE(page >= 16 && page <= 1024 && (page & (page - 1)) == 0, GDN_EUNSUPPORTED,
            "%s: page = %d is not a power of two in 16..1024", fn, page);
    REQUIRE(n_pages <= gdn::kKvPagesMax, GDN_EUNSUPPORTED, "%s: n_pages = %d > %d", fn, n_pages, gdn::kKvPagesMax);
    REQUIRE(Hkv <= 1024, GDN_EUNSUPPORTED, "%s: Hkv = %d > 1024", fn, Hkv);
    REQUIRE((long long)Hkv * page * D <= (1 << 28), GDN_EUNSUPPORTED, "%s: a page of %d x %d x %d passes 2^28 elements",
            fn, Hkv, page, D);
    REQUIRE(planes <= 65535, GDN_EUNSUPPORTED, "%s: planes = %d > 65535", fn, planes);
    // (a token's 16-byte pieces in all planes are counted in 32 bits)
    REQUIRE((long long)planes * Hkv * D * (int)elem_size(dtype) <= 1LL << 33, GDN_EUNSUPPORTED,
            "%s: a token of %d planes x %d x %d passes 2^33 bytes", fn, planes, Hkv, D);
    g.planes = planes;
    g.n_pages = n_pages;
    g.Hkv = Hkv;
    g.page_log2 = 0;
    while ((1 << g.page_log2) < page) ++g.page_log2;
    g.row_bytes = D * (int)elem_size(dtype);
    return GDN_OK;
}

// outputs that overlap one another or an input; a pair of null spans never does
bool any_overlap(const Span* outs, int n_out, const Span* ins, int n_in)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

Span ints(const int32_t* p, size_t n) { return Span{p, p ? n * 4 : 0}; }

}  // namespace

extern "C" {

int gdn_version(void) { return GDN_VERSION; }

const char* gdn_last_error(void) { return g_err; }

int gdn_debug_clamped_accepts(long long* count, int reset)
{
    const char* fn = "gdn_debug_clamped_accepts";
#ifdef GDN_DEBUG
    REQUIRE(count, GDN_EINVAL, "%s: null count", fn);
    // one counter per translation unit that clamps accept lengths
    hipError_t (*const readers[])(unsigned long long*, bool) = {
        gdn::clamped_accepts_rollback,          gdn::clamped_accepts_conv,
        gdn::clamped_accepts_step,              gdn::clamped_accepts_verify_bf16_bf16,
        gdn::clamped_accepts_verify_bf16_f32,   gdn::clamped_accepts_verify_f32_bf16,
        gdn::clamped_accepts_verify_f32_f32};
    unsigned long long total = 0;
    for (auto rd : readers) {
        unsigned long long n = 0;
        const hipError_t e = rd(&n, reset != 0);
        if (e != hipSuccess) return fail(GDN_EHIP, "%s: %s", fn, hipGetErrorString(e));
        total += n;
    }
    *count = (long long)total;
    return ok();
#else
    (void)count;
    (void)reset;
    return fail(GDN_EUNSUPPORTED, "%s: counted only in the debug build (libgdn_debug.so)", fn);
#endif
}

int gdn_conv_step(const void* x, const float* w, void* hist, void* y, void* win_out, int B, int T, int C, int W,
                  int io_dtype, void* stream)
{
    return gdn_conv_step_ex(x, w, hist, y, win_out, nullptr, B, T, C, W, io_dtype, stream);
}

int gdn_conv_step_ex(const void* x, const float* w, void* hist, void* y, void* win_out, const int32_t* lens, int B,
                     int T, int C, int W, int io_dtype, void* stream)
{
    const char* fn = "gdn_conv_step";
    REQUIRE(B >= 0, GDN_EINVAL, "%s: B = %d < 0", fn, B);
    REQUIRE(T >= 1, GDN_EINVAL, "%s: T = %d < 1", fn, T);
    REQUIRE(C >= 1, GDN_EINVAL, "%s: C = %d < 1", fn, C);
    REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
    REQUIRE(valid_dtype(io_dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, io_dtype);
    REQUIRE((long long)B * T * C < (1LL << 40), GDN_EUNSUPPORTED, "%s: problem too large", fn);
    if (B == 0) return ok();
    REQUIRE(x && w && hist && y, GDN_EINVAL, "%s: null pointer (x, w, hist and y are required)", fn);
    REQUIRE(aligned16(x) && aligned16(w) && aligned16(hist) && aligned16(y) && (!win_out || aligned16(win_out)),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(!lens || ((uintptr_t)lens & 3) == 0, GDN_EINVAL, "%s: lens must be 4-byte aligned", fn);
    const size_t es = elem_size(io_dtype);
    const Span sx{x, (size_t)B * T * C * es}, sw{w, (size_t)C * W * 4}, sh{hist, (size_t)B * (W - 1) * C * es},
        sy{y, (size_t)B * T * C * es}, swin{win_out, win_out ? (size_t)B * (W - 1 + T) * C * es : 0};
    REQUIRE(!overlap(sy, sx) && !overlap(sy, sw) && !overlap(sy, sh), GDN_EINVAL, "%s: y overlaps an input", fn);
    REQUIRE(!overlap(swin, sx) && !overlap(swin, sw) && !overlap(swin, sh) && !overlap(swin, sy), GDN_EINVAL,
            "%s: win_out overlaps another buffer", fn);
    REQUIRE(!overlap(sh, sx) && !overlap(sh, sw), GDN_EINVAL, "%s: hist overlaps x or w", fn);
    REQUIRE(T <= 65535 * 16, GDN_EUNSUPPORTED, "%s: T = %d too large", fn, T);
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d too large", fn, B);
    REQUIRE(!overlap(sh, Span{lens, lens ? (size_t)B * 4 : 0}) && !overlap(sy, Span{lens, lens ? (size_t)B * 4 : 0}) &&
                !overlap(swin, Span{lens, lens ? (size_t)B * 4 : 0}),
            GDN_EINVAL, "%s: an output overlaps lens", fn);
    gdn::ConvArgs a{x, w, hist, y, win_out, B, T, C, W, lens};
    return launch_status(gdn::launch_conv_step(a, io_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_verify(const void* qkv, const void* beta_raw, const void* alpha, const float* dt_bias, const float* A_log,
               const float* S_in, float* S_out, float* H, void* o, int B, int K, int Hk, int Hv, int dk, int dv,
               int in_dtype, int o_dtype, float l2_eps, void* stream)
{
    return gdn_verify_ex(qkv, beta_raw, alpha, Hv, dt_bias, A_log, S_in, S_out, H, o, nullptr, B, K, Hk, Hv, dk, dv,
                         in_dtype, o_dtype, l2_eps, stream);
}

int gdn_verify_ex(const void* qkv, const void* beta_raw, const void* alpha, int gate_stride, const float* dt_bias,
                  const float* A_log, const float* S_in, float* S_out, float* H, void* o, const int32_t* lens, int B,
                  int K, int Hk, int Hv, int dk, int dv, int in_dtype, int o_dtype, float l2_eps, void* stream)
{
    const char* fn = "gdn_verify";
    int rc = check_gdn_shape(fn, B, K, Hk, Hv, dk, dv, in_dtype, o_dtype, l2_eps);
    if (rc) return rc;
    REQUIRE(K <= gdn::kVerifyMax, GDN_EUNSUPPORTED, "%s: K = %d > %d", fn, K, gdn::kVerifyMax);
    REQUIRE(B <= 65535 && Hv <= 65535, GDN_EUNSUPPORTED, "%s: B or Hv too large", fn);
    REQUIRE((dt_bias == nullptr) == (A_log == nullptr), GDN_EINVAL,
            "%s: dt_bias and A_log must be both given (raw gates) or both NULL (activated gates)", fn);
    if (B == 0) return ok();
    REQUIRE(qkv && beta_raw && alpha && S_in && S_out && o, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(gate_stride >= Hv, GDN_EINVAL, "%s: gate_stride = %d < Hv = %d", fn, gate_stride, Hv);
    const size_t ie = elem_size(in_dtype), oe = elem_size(o_dtype);
    REQUIRE(aligned16(qkv) && aligned16(S_in) && aligned16(S_out) && aligned16(o) && (!H || aligned16(H)) &&
                (!dt_bias || (aligned16(dt_bias) && aligned16(A_log))),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)beta_raw % ie) == 0 && ((uintptr_t)alpha % ie) == 0 && (!lens || ((uintptr_t)lens & 3) == 0),
            GDN_EINVAL, "%s: gate or lens pointers not aligned to their element size", fn);
    const size_t C = (size_t)2 * Hk * dk + (size_t)Hv * dv;
    const size_t SD = (size_t)B * Hv * dv * dk * 4;
    const size_t gspan = ((size_t)B * K - 1) * gate_stride + Hv;   // elements from the first to the last gate
    const Span sq{qkv, (size_t)B * K * C * ie}, sb{beta_raw, gspan * ie}, sa{alpha, gspan * ie},
        ssi{S_in, SD}, sso{S_out, SD},
        sH{H, H ? (size_t)B * (K - 1) * Hv * dv * dk * 4 : 0}, so{o, (size_t)B * K * Hv * dv * oe},
        sdt{dt_bias, dt_bias ? (size_t)Hv * 4 : 0}, sal{A_log, A_log ? (size_t)Hv * 4 : 0};
    REQUIRE(!(overlap(sso, ssi) && S_out != S_in), GDN_EINVAL, "%s: S_out partially overlaps S_in", fn);
    const Span sl{lens, lens ? (size_t)B * 4 : 0};
    const Span ins[] = {sq, sb, sa, sdt, sal, sl};
    for (const Span& s : ins) {
        REQUIRE(!overlap(sso, s), GDN_EINVAL, "%s: S_out overlaps an input", fn);
        REQUIRE(!overlap(sH, s) && !overlap(so, s), GDN_EINVAL, "%s: H or o overlaps an input", fn);
    }
    REQUIRE(!overlap(sH, ssi) && !overlap(sH, sso) && !overlap(so, ssi) && !overlap(so, sso) && !overlap(so, sH),
            GDN_EINVAL, "%s: H, o and the state buffers must not overlap", fn);
    gdn::VerifyArgs a{qkv, beta_raw, alpha, dt_bias, A_log, S_in, S_out, H, o, B, K, Hk, Hv, dk, dv, l2_eps, lens,
                      gate_stride};
    return launch_status(gdn::launch_verify(a, in_dtype == GDN_BF16, o_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_rollback(const int32_t* accept, int K, const float* S_in, const float* H, float* S_out, void* hist,
                 const void* win, int B, int Hv, int dv, int dk, int C, int W, int io_dtype, void* stream)
{
    return gdn_rollback_ex(accept, nullptr, K, S_in, H, S_out, hist, win, B, Hv, dv, dk, C, W, io_dtype, stream);
}

int gdn_rollback_ex(const int32_t* accept, const int32_t* lens, int K, const float* S_in, const float* H,
                    float* S_out, void* hist, const void* win, int B, int Hv, int dv, int dk, int C, int W,
                    int io_dtype, void* stream)
{
    const char* fn = "gdn_rollback";
    REQUIRE(B >= 0, GDN_EINVAL, "%s: B = %d < 0", fn, B);
    REQUIRE(K >= 1, GDN_EINVAL, "%s: K = %d < 1", fn, K);
    REQUIRE(Hv >= 1 && dv >= 1 && dk >= 1, GDN_EINVAL, "%s: bad state shape", fn);
    REQUIRE(((long long)Hv * dv * dk) % 4 == 0, GDN_EUNSUPPORTED, "%s: Hv*dv*dk must be a multiple of 4", fn);
    REQUIRE((hist == nullptr) == (win == nullptr), GDN_EINVAL, "%s: hist and win must be both given or both NULL",
            fn);
    if (hist) {
        REQUIRE(C >= 1, GDN_EINVAL, "%s: C = %d < 1", fn, C);
        REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
        REQUIRE(valid_dtype(io_dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, io_dtype);
    }
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d too large", fn, B);
    if (B == 0) return ok();
    REQUIRE(accept && S_in && S_out, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(H || K == 1, GDN_EINVAL, "%s: H is required when K > 1", fn);
    REQUIRE(S_in != S_out, GDN_EINVAL, "%s: S_out must not be S_in (the pre-window state is needed)", fn);
    REQUIRE(aligned16(S_in) && aligned16(S_out) && (!H || aligned16(H)) && aligned16(accept) &&
                (!hist || (aligned16(hist) && aligned16(win))),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    const size_t st = (size_t)Hv * dv * dk * 4;
    const Span ssi{S_in, B * st}, sso{S_out, B * st}, sH{H, H ? (size_t)B * (K - 1) * st : 0};
    REQUIRE(!overlap(sso, ssi) && !overlap(sso, sH), GDN_EINVAL, "%s: S_out overlaps S_in or H", fn);
    REQUIRE(!lens || ((uintptr_t)lens & 3) == 0, GDN_EINVAL, "%s: lens must be 4-byte aligned", fn);
    REQUIRE(!overlap(sso, Span{lens, lens ? (size_t)B * 4 : 0}), GDN_EINVAL, "%s: S_out overlaps lens", fn);
    if (hist) {
        const size_t es = elem_size(io_dtype);
        const Span sh{hist, (size_t)B * (W - 1) * C * es}, sw{win, (size_t)B * (W - 1 + K) * C * es};
        REQUIRE(!overlap(sh, sw) && !overlap(sh, sso) && !overlap(sh, ssi) && !overlap(sh, sH), GDN_EINVAL,
                "%s: hist overlaps another buffer", fn);
    }
    gdn::RollbackArgs a{accept, S_in, H, S_out, hist, win, B, K, (long long)Hv * dv * dk, C, W,
                        (int)elem_size(io_dtype), lens};
    return launch_status(gdn::launch_rollback(a, (hipStream_t)stream), fn);
}

int gdn_replay(const int32_t* accept, const void* qkv, const void* beta_raw, const void* alpha, int gate_stride,
               const float* dt_bias, const float* A_log, const float* S_ckpt, float* S_out, void* hist,
               const void* win, int B, int K, int Hk, int Hv, int dk, int dv, int W, int in_dtype, float l2_eps,
               void* stream)
{
    const char* fn = "gdn_replay";
    int rc = check_gdn_shape(fn, B, K, Hk, Hv, dk, dv, in_dtype, GDN_F32, l2_eps);
    if (rc) return rc;
    REQUIRE(K <= gdn::kVerifyMax, GDN_EUNSUPPORTED, "%s: K = %d > %d", fn, K, gdn::kVerifyMax);
    REQUIRE(B <= 65535 && Hv <= 65535, GDN_EUNSUPPORTED, "%s: B or Hv too large", fn);
    REQUIRE((dt_bias == nullptr) == (A_log == nullptr), GDN_EINVAL,
            "%s: dt_bias and A_log must be both given (raw gates) or both NULL (activated gates)", fn);
    REQUIRE((hist == nullptr) == (win == nullptr), GDN_EINVAL, "%s: hist and win must be both given or both NULL",
            fn);
    if (hist) REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
    if (B == 0) return ok();
    REQUIRE(accept && qkv && beta_raw && alpha && S_ckpt && S_out, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(S_ckpt != S_out, GDN_EINVAL, "%s: S_out must not be the checkpoint", fn);
    REQUIRE(gate_stride >= Hv, GDN_EINVAL, "%s: gate_stride = %d < Hv = %d", fn, gate_stride, Hv);
    const size_t ie = elem_size(in_dtype);
    REQUIRE(aligned16(accept) && aligned16(qkv) && aligned16(S_ckpt) && aligned16(S_out) &&
                (!dt_bias || (aligned16(dt_bias) && aligned16(A_log))) && (!hist || (aligned16(hist) && aligned16(win))),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)beta_raw % ie) == 0 && ((uintptr_t)alpha % ie) == 0, GDN_EINVAL,
            "%s: gate pointers not aligned to their element size", fn);
    const size_t C = (size_t)2 * Hk * dk + (size_t)Hv * dv;
    const size_t SD = (size_t)B * Hv * dv * dk * 4;
    const size_t gspan = ((size_t)B * K - 1) * gate_stride + Hv;
    const Span sq{qkv, (size_t)B * K * C * ie}, sb{beta_raw, gspan * ie}, sa{alpha, gspan * ie}, sc{S_ckpt, SD},
        sso{S_out, SD}, sacc{accept, (size_t)B * 4}, sdt{dt_bias, dt_bias ? (size_t)Hv * 4 : 0},
        sal{A_log, A_log ? (size_t)Hv * 4 : 0}, sh{hist, hist ? (size_t)B * (W - 1) * C * ie : 0},
        sw{win, win ? (size_t)B * (W - 1 + K) * C * ie : 0};
    const Span ins[] = {sq, sb, sa, sc, sacc, sdt, sal, sw};
    for (const Span& s : ins)
        REQUIRE(!overlap(sso, s) && !overlap(sh, s), GDN_EINVAL, "%s: an output overlaps an input", fn);
    REQUIRE(!overlap(sso, sh), GDN_EINVAL, "%s: S_out overlaps hist", fn);
    gdn::VerifyArgs a{qkv, beta_raw, alpha, dt_bias, A_log, S_ckpt, S_out, nullptr, nullptr, B, K, Hk, Hv, dk, dv,
                      l2_eps, nullptr, gate_stride, accept};
    rc = launch_status(gdn::launch_verify(a, in_dtype == GDN_BF16, false, (hipStream_t)stream), fn);
    if (rc || !hist) return rc;
    // the conv history of the accepted prefix: the rollback's conv rows only
    gdn::RollbackArgs r{accept, S_ckpt, nullptr, S_out, hist, win, B, K, 0, (int)C, W, (int)ie};
    return launch_status(gdn::launch_rollback(r, (hipStream_t)stream), fn);
}

int gdn_rollback_conv_step(const int32_t* accept, int K_prev, const float* S_in, const float* H, float* S_out,
                           const void* win_prev, const void* x, const float* w, void* hist, void* y, void* win,
                           int B, int Hv, int dv, int dk, int T, int C, int W, int io_dtype, void* stream)
{
    const char* fn = "gdn_rollback_conv_step";
    REQUIRE(B >= 0, GDN_EINVAL, "%s: B = %d < 0", fn, B);
    REQUIRE(K_prev >= 1, GDN_EINVAL, "%s: K_prev = %d < 1", fn, K_prev);
    REQUIRE(T >= 1, GDN_EINVAL, "%s: T = %d < 1", fn, T);
    REQUIRE(C >= 1, GDN_EINVAL, "%s: C = %d < 1", fn, C);
    REQUIRE(Hv >= 1 && dv >= 1 && dk >= 1, GDN_EINVAL, "%s: bad state shape", fn);
    REQUIRE(((long long)Hv * dv * dk) % 4 == 0, GDN_EUNSUPPORTED, "%s: Hv*dv*dk must be a multiple of 4", fn);
    REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
    REQUIRE(valid_dtype(io_dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, io_dtype);
    REQUIRE((long long)B * (T + K_prev) * C < (1LL << 40), GDN_EUNSUPPORTED, "%s: problem too large", fn);
    REQUIRE(T <= 65535 * 16, GDN_EUNSUPPORTED, "%s: T = %d too large", fn, T);
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d too large", fn, B);
    if (B == 0) return ok();
    REQUIRE(accept && S_in && S_out && win_prev && x && w && hist && y && win, GDN_EINVAL,
            "%s: null pointer (only H may be NULL, and only when K_prev == 1)", fn);
    REQUIRE(H || K_prev == 1, GDN_EINVAL, "%s: H is required when K_prev > 1", fn);
    REQUIRE(S_in != S_out, GDN_EINVAL, "%s: S_out must not be S_in (the pre-window state is needed)", fn);
    REQUIRE(aligned16(accept) && aligned16(S_in) && aligned16(S_out) && (!H || aligned16(H)) && aligned16(win_prev) &&
                aligned16(x) && aligned16(w) && aligned16(hist) && aligned16(y) && aligned16(win),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    const size_t st = (size_t)Hv * dv * dk * 4, es = elem_size(io_dtype);
    const Span ssi{S_in, B * st}, sso{S_out, B * st}, sH{H, H ? (size_t)B * (K_prev - 1) * st : 0},
        swp{win_prev, (size_t)B * (W - 1 + K_prev) * C * es}, sx{x, (size_t)B * T * C * es},
        sw{w, (size_t)C * W * 4}, sh{hist, (size_t)B * (W - 1) * C * es}, sy{y, (size_t)B * T * C * es},
        swin{win, (size_t)B * (W - 1 + T) * C * es}, sacc{accept, (size_t)B * 4};
    const Span ins[] = {ssi, sH, swp, sx, sw, sacc};
    const Span outs[] = {sso, sh, sy, swin};
    for (const Span& o : outs)
        for (const Span& i : ins) REQUIRE(!overlap(o, i), GDN_EINVAL, "%s: an output overlaps an input", fn);
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            REQUIRE(!overlap(outs[i], outs[j]), GDN_EINVAL, "%s: two outputs overlap", fn);
    gdn::RollConvArgs a{accept, K_prev, S_in, H, S_out, (long long)Hv * dv * dk, win_prev, x, w, hist, y, win,
                        B, T, C, W};
    return launch_status(gdn::launch_rollback_conv(a, io_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_prefill_chunked(const void* qkv, const void* beta_raw, const void* alpha, const float* dt_bias,
                        const float* A_log, const float* S_in, float* S_out, void* o, int B, int T, int chunk,
                        int Hk, int Hv, int dk, int dv, int in_dtype, int o_dtype, float l2_eps, void* stream)
{
    const char* fn = "gdn_prefill_chunked";
    int rc = check_gdn_shape(fn, B, T, Hk, Hv, dk, dv, in_dtype, o_dtype, l2_eps);
    if (rc) return rc;
    REQUIRE(chunk == 16 || chunk == 32 || chunk == 64, GDN_EUNSUPPORTED, "%s: chunk = %d not in {16, 32, 64}", fn,
            chunk);
    REQUIRE(B <= 65535 && Hv <= 65535, GDN_EUNSUPPORTED, "%s: B or Hv too large", fn);
    REQUIRE((dt_bias == nullptr) == (A_log == nullptr), GDN_EINVAL,
            "%s: dt_bias and A_log must be both given or both NULL", fn);
    if (B == 0) return ok();
    REQUIRE(qkv && beta_raw && alpha && S_in && S_out && o, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(qkv) && aligned16(beta_raw) && aligned16(alpha) && aligned16(S_in) && aligned16(S_out) &&
                aligned16(o) && (!dt_bias || (aligned16(dt_bias) && aligned16(A_log))),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    const size_t ie = elem_size(in_dtype), oe = elem_size(o_dtype);
    const size_t C = (size_t)2 * Hk * dk + (size_t)Hv * dv;
    const size_t SD = (size_t)B * Hv * dv * dk * 4;
    const Span sq{qkv, (size_t)B * T * C * ie}, sb{beta_raw, (size_t)B * T * Hv * ie},
        sa{alpha, (size_t)B * T * Hv * ie}, ssi{S_in, SD}, sso{S_out, SD}, so{o, (size_t)B * T * Hv * dv * oe};
    REQUIRE(!(overlap(sso, ssi) && S_out != S_in), GDN_EINVAL, "%s: S_out partially overlaps S_in", fn);
    const Span ins[] = {sq, sb, sa};
    for (const Span& s : ins)
        REQUIRE(!overlap(sso, s) && !overlap(so, s), GDN_EINVAL, "%s: an output overlaps an input", fn);
    REQUIRE(!overlap(so, ssi) && !overlap(so, sso), GDN_EINVAL, "%s: o overlaps the state", fn);
    gdn::PrefillArgs a{qkv, beta_raw, alpha, dt_bias, A_log, S_in, S_out, o, B, T, chunk, Hk, Hv, dk, dv, l2_eps};
    return launch_status(gdn::launch_prefill(a, in_dtype == GDN_BF16, o_dtype == GDN_BF16, (hipStream_t)stream),
                         fn);
}

int gdn_verify_step(const int32_t* accept_prev, int K_prev, const float* S_prev_ckpt, const float* H_prev,
                    const float* S_prev_out, const void* win_prev, const float* S_in, const void* hist, const void* x,
                    const float* w, const void* beta_raw, const void* alpha, int gate_stride, const float* dt_bias,
                    const float* A_log, float* S_ckpt, float* S_out, float* H, void* o, void* y, void* win, int B,
                    int K, int Hk, int Hv, int dk, int dv, int W, int in_dtype, int o_dtype, float l2_eps,
                    void* stream)
{
    const char* fn = "gdn_verify_step";
    int rc = check_gdn_shape(fn, B, K, Hk, Hv, dk, dv, in_dtype, o_dtype, l2_eps);
    if (rc) return rc;
    REQUIRE(K <= gdn::kVerifyMax, GDN_EUNSUPPORTED, "%s: K = %d > %d", fn, K, gdn::kVerifyMax);
    REQUIRE(W == 4, GDN_EUNSUPPORTED, "%s: W = %d (the fused step takes conv width 4)", fn, W);
    REQUIRE(B <= 65535 && Hv <= 65535, GDN_EUNSUPPORTED, "%s: B or Hv too large", fn);
    REQUIRE((dt_bias == nullptr) == (A_log == nullptr), GDN_EINVAL,
            "%s: dt_bias and A_log must be both given (raw gates) or both NULL (activated gates)", fn);
    if (accept_prev)
        REQUIRE(K_prev >= 1 && K_prev <= gdn::kVerifyMax, GDN_EINVAL, "%s: K_prev = %d not in 1..%d", fn, K_prev,
                gdn::kVerifyMax);
    if (B == 0) return ok();
    REQUIRE(x && w && beta_raw && alpha && S_out && o, GDN_EINVAL, "%s: null pointer", fn);
    if (accept_prev) {
        REQUIRE(S_prev_ckpt && S_prev_out && win_prev && (H_prev || K_prev == 1), GDN_EINVAL,
                "%s: the previous window needs S_prev_ckpt, S_prev_out, win_prev and (K_prev > 1) H_prev", fn);
    } else {
        REQUIRE(S_in && hist, GDN_EINVAL, "%s: the first window needs S_in and hist", fn);
    }
    REQUIRE(gate_stride >= Hv, GDN_EINVAL, "%s: gate_stride = %d < Hv = %d", fn, gate_stride, Hv);
    const size_t ie = elem_size(in_dtype), oe = elem_size(o_dtype);
    auto a16 = [](const void* q) { return q == nullptr || aligned16(q); };
    REQUIRE(a16(x) && a16(w) && a16(S_prev_ckpt) && a16(H_prev) && a16(S_prev_out) && a16(win_prev) && a16(S_in) &&
                a16(hist) && a16(dt_bias) && a16(A_log) && a16(S_ckpt) && a16(S_out) && a16(H) && a16(o) && a16(y) &&
                a16(win),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)beta_raw % ie) == 0 && ((uintptr_t)alpha % ie) == 0 && ((uintptr_t)accept_prev & 3) == 0,
            GDN_EINVAL, "%s: gate or accept pointers not aligned to their element size", fn);
    const size_t C = (size_t)2 * Hk * dk + (size_t)Hv * dv;
    const size_t st = (size_t)Hv * dv * dk * 4;
    const size_t gspan = ((size_t)B * K - 1) * gate_stride + Hv;
    const Span ins[] = {Span{x, (size_t)B * K * C * ie},
                        Span{w, C * 4 * 4},
                        Span{beta_raw, gspan * ie},
                        Span{alpha, gspan * ie},
                        Span{dt_bias, dt_bias ? (size_t)Hv * 4 : 0},
                        Span{A_log, A_log ? (size_t)Hv * 4 : 0},
                        Span{accept_prev, accept_prev ? (size_t)B * 4 : 0},
                        Span{accept_prev ? S_prev_ckpt : nullptr, B * st},
                        Span{accept_prev ? H_prev : nullptr, H_prev ? (size_t)B * (K_prev - 1) * st : 0},
                        Span{accept_prev ? S_prev_out : nullptr, B * st},
                        Span{accept_prev ? win_prev : nullptr, (size_t)B * (W - 1 + K_prev) * C * ie},
                        Span{accept_prev ? nullptr : S_in, B * st},
                        Span{accept_prev ? nullptr : hist, (size_t)B * (W - 1) * C * ie}};
    const Span outs[] = {Span{S_ckpt, B * st}, Span{S_out, B * st}, Span{H, H ? (size_t)B * (K - 1) * st : 0},
                         Span{o, (size_t)B * K * Hv * dv * oe}, Span{y, (size_t)B * K * C * ie},
                         Span{win, (size_t)B * (W - 1 + K) * C * ie}};
    for (const Span& q : outs)
        for (const Span& i : ins) REQUIRE(!overlap(q, i), GDN_EINVAL, "%s: an output overlaps an input", fn);
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 6; ++j) REQUIRE(!overlap(outs[i], outs[j]), GDN_EINVAL, "%s: two outputs overlap", fn);
    gdn::VerifyArgs a{x, beta_raw, alpha, dt_bias, A_log, accept_prev ? nullptr : S_in, S_out, H, o, B, K, Hk, Hv,
                      dk, dv, l2_eps, nullptr, gate_stride};
    a.x = x;
    a.w = w;
    a.hsrc = accept_prev ? win_prev : hist;
    a.hrows = accept_prev ? W - 1 + K_prev : W - 1;
    a.acc_prev = accept_prev;
    a.Kp = accept_prev ? K_prev : 0;
    a.Sp_ckpt = S_prev_ckpt;
    a.Sp_H = H_prev;
    a.Sp_out = S_prev_out;
    a.S_ckpt = S_ckpt;
    a.y = y;
    a.win = win;
    return launch_status(gdn::launch_step(a, in_dtype == GDN_BF16, o_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_conv_tree(const void* x, const float* w, const void* hist, const int32_t* parent, void* y, int B, int N,
                  int C, int W, int io_dtype, void* stream)
{
    const char* fn = "gdn_conv_tree";
    REQUIRE(B >= 0, GDN_EINVAL, "%s: B = %d < 0", fn, B);
    REQUIRE(N >= 1, GDN_EINVAL, "%s: N = %d < 1", fn, N);
    REQUIRE(N <= gdn::kTreeMax, GDN_EUNSUPPORTED, "%s: N = %d > %d", fn, N, gdn::kTreeMax);
    REQUIRE(C >= 1, GDN_EINVAL, "%s: C = %d < 1", fn, C);
    REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
    REQUIRE(valid_dtype(io_dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, io_dtype);
    REQUIRE((long long)B * N * C < (1LL << 40), GDN_EUNSUPPORTED, "%s: problem too large", fn);
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d too large", fn, B);
    if (B == 0) return ok();
    REQUIRE(x && w && hist && parent && y, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(x) && aligned16(w) && aligned16(hist) && aligned16(y), GDN_EINVAL,
            "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)parent & 3) == 0, GDN_EINVAL, "%s: parent must be 4-byte aligned", fn);
    const size_t es = elem_size(io_dtype);
    const Span sy{y, (size_t)B * N * C * es};
    const Span ins[] = {Span{x, (size_t)B * N * C * es}, Span{w, (size_t)C * W * 4},
                        Span{hist, (size_t)B * (W - 1) * C * es}, Span{parent, (size_t)B * N * 4}};
    for (const Span& s : ins) REQUIRE(!overlap(sy, s), GDN_EINVAL, "%s: y overlaps an input", fn);
    gdn::ConvTreeArgs a{x, w, hist, parent, y, B, N, C, W};
    return launch_status(gdn::launch_conv_tree(a, io_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_verify_tree(const void* qkv, const void* beta_raw, const void* alpha, int gate_stride, const float* dt_bias,
                    const float* A_log, const int32_t* parent, const float* S_in, float* H, void* o, int B, int N,
                    int Hk, int Hv, int dk, int dv, int in_dtype, int o_dtype, float l2_eps, void* stream)
{
    const char* fn = "gdn_verify_tree";
    int rc = check_gdn_shape(fn, B, N, Hk, Hv, dk, dv, in_dtype, o_dtype, l2_eps);
    if (rc) return rc;
    REQUIRE(N <= gdn::kTreeMax, GDN_EUNSUPPORTED, "%s: N = %d > %d", fn, N, gdn::kTreeMax);
    REQUIRE(B <= 65535 && Hv <= 65535, GDN_EUNSUPPORTED, "%s: B or Hv too large", fn);
    REQUIRE((dt_bias == nullptr) == (A_log == nullptr), GDN_EINVAL,
            "%s: dt_bias and A_log must be both given (raw gates) or both NULL (activated gates)", fn);
    if (B == 0) return ok();
    REQUIRE(qkv && beta_raw && alpha && parent && S_in && H && o, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(gate_stride >= Hv, GDN_EINVAL, "%s: gate_stride = %d < Hv = %d", fn, gate_stride, Hv);
    const size_t ie = elem_size(in_dtype), oe = elem_size(o_dtype);
    REQUIRE(aligned16(qkv) && aligned16(S_in) && aligned16(H) && aligned16(o) &&
                (!dt_bias || (aligned16(dt_bias) && aligned16(A_log))),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)beta_raw % ie) == 0 && ((uintptr_t)alpha % ie) == 0 && ((uintptr_t)parent & 3) == 0,
            GDN_EINVAL, "%s: gate or parent pointers not aligned to their element size", fn);
    const size_t C = (size_t)2 * Hk * dk + (size_t)Hv * dv;
    const size_t st = (size_t)Hv * dv * dk * 4;
    const size_t gspan = ((size_t)B * N - 1) * gate_stride + Hv;
    const Span sH{H, (size_t)B * N * st}, so{o, (size_t)B * N * Hv * dv * oe};
    const Span ins[] = {Span{qkv, (size_t)B * N * C * ie}, Span{beta_raw, gspan * ie}, Span{alpha, gspan * ie},
                        Span{dt_bias, dt_bias ? (size_t)Hv * 4 : 0}, Span{A_log, A_log ? (size_t)Hv * 4 : 0},
                        Span{parent, (size_t)B * N * 4}, Span{S_in, B * st}};
    for (const Span& s : ins)
        REQUIRE(!overlap(sH, s) && !overlap(so, s), GDN_EINVAL, "%s: H or o overlaps an input", fn);
    REQUIRE(!overlap(sH, so), GDN_EINVAL, "%s: H and o overlap", fn);
    gdn::VerifyArgs a{qkv, beta_raw, alpha, dt_bias, A_log, S_in, nullptr, H, o, B, N, Hk, Hv, dk, dv, l2_eps,
                      nullptr, gate_stride, nullptr, parent};
    return launch_status(gdn::launch_verify(a, in_dtype == GDN_BF16, o_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_rollback_tree(const int32_t* node, const int32_t* parent, int N, const float* S_in, const float* H,
                      float* S_out, const void* x, void* hist, int B, int Hv, int dv, int dk, int C, int W,
                      int io_dtype, void* stream)
{
    const char* fn = "gdn_rollback_tree";
    REQUIRE(B >= 0, GDN_EINVAL, "%s: B = %d < 0", fn, B);
    REQUIRE(N >= 1, GDN_EINVAL, "%s: N = %d < 1", fn, N);
    REQUIRE(N <= gdn::kTreeMax, GDN_EUNSUPPORTED, "%s: N = %d > %d", fn, N, gdn::kTreeMax);
    REQUIRE(Hv >= 1 && dv >= 1 && dk >= 1, GDN_EINVAL, "%s: bad state shape", fn);
    REQUIRE(((long long)Hv * dv * dk) % 4 == 0, GDN_EUNSUPPORTED, "%s: Hv*dv*dk must be a multiple of 4", fn);
    REQUIRE((hist == nullptr) == (x == nullptr), GDN_EINVAL, "%s: x and hist must be both given or both NULL", fn);
    if (hist) {
        REQUIRE(C >= 1, GDN_EINVAL, "%s: C = %d < 1", fn, C);
        REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
        REQUIRE(valid_dtype(io_dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, io_dtype);
    }
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d too large", fn, B);
    if (B == 0) return ok();
    REQUIRE(node && parent && S_in && H && S_out, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(S_in != S_out, GDN_EINVAL, "%s: S_out must not be S_in", fn);
    REQUIRE(aligned16(S_in) && aligned16(S_out) && aligned16(H) && (!hist || (aligned16(hist) && aligned16(x))),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)node & 3) == 0 && ((uintptr_t)parent & 3) == 0, GDN_EINVAL,
            "%s: node and parent must be 4-byte aligned", fn);
    const size_t st = (size_t)Hv * dv * dk * 4;
    const Span sso{S_out, B * st}, sh{hist, hist ? (size_t)B * (W - 1) * C * elem_size(io_dtype) : 0};
    const Span ins[] = {Span{S_in, B * st}, Span{H, (size_t)B * N * st}, Span{node, (size_t)B * 4},
                        Span{parent, (size_t)B * N * 4},
                        Span{x, x ? (size_t)B * N * C * elem_size(io_dtype) : 0}};
    for (const Span& s : ins)
        REQUIRE(!overlap(sso, s) && !overlap(sh, s), GDN_EINVAL, "%s: an output overlaps an input", fn);
    REQUIRE(!overlap(sso, sh), GDN_EINVAL, "%s: S_out overlaps hist", fn);
    gdn::TreeRollbackArgs a{node, parent, S_in, H, S_out, (long long)Hv * dv * dk, x, hist, B, N, C, W,
                            (int)elem_size(io_dtype)};
    return launch_status(gdn::launch_tree_rollback(a, (hipStream_t)stream), fn);
}

int gdn_verify_tree_step(const int32_t* node_prev, int N_prev, const int32_t* parent_prev, const float* S_prev_ckpt,
                         const float* H_prev, const void* x_prev, const void* hist_prev, const void* x, const float* w,
                         const int32_t* parent, const void* beta_raw, const void* alpha, int gate_stride,
                         const float* dt_bias, const float* A_log, float* S_ckpt, float* H, void* o, void* y,
                         void* hist_out, int B, int N, int Hk, int Hv, int dk, int dv, int W, int in_dtype,
                         int o_dtype, float l2_eps, void* stream)
{
    const char* fn = "gdn_verify_tree_step";
    int rc = check_gdn_shape(fn, B, N, Hk, Hv, dk, dv, in_dtype, o_dtype, l2_eps);
    if (rc) return rc;
    REQUIRE(N <= gdn::kTreeMax, GDN_EUNSUPPORTED, "%s: N = %d > %d", fn, N, gdn::kTreeMax);
    REQUIRE(W >= 2 && W <= 8, GDN_EUNSUPPORTED, "%s: W = %d not in 2..8", fn, W);
    REQUIRE(B <= 65535 && Hv <= 65535, GDN_EUNSUPPORTED, "%s: B or Hv too large", fn);
    REQUIRE((dt_bias == nullptr) == (A_log == nullptr), GDN_EINVAL,
            "%s: dt_bias and A_log must be both given (raw gates) or both NULL (activated gates)", fn);
    if (node_prev)
        REQUIRE(N_prev >= 1 && N_prev <= gdn::kTreeMax, GDN_EINVAL, "%s: N_prev = %d not in 1..%d", fn, N_prev,
                gdn::kTreeMax);
    if (B == 0) return ok();
    REQUIRE(S_prev_ckpt && hist_prev && x && w && parent && beta_raw && alpha && H && o && y, GDN_EINVAL,
            "%s: null pointer", fn);
    if (node_prev)
        REQUIRE(parent_prev && H_prev && x_prev, GDN_EINVAL,
                "%s: a previous tree needs parent_prev, H_prev and x_prev", fn);
    REQUIRE(gate_stride >= Hv, GDN_EINVAL, "%s: gate_stride = %d < Hv = %d", fn, gate_stride, Hv);
    const size_t ie = elem_size(in_dtype), oe = elem_size(o_dtype);
    auto a16 = [](const void* q) { return q == nullptr || aligned16(q); };
    REQUIRE(a16(S_prev_ckpt) && a16(H_prev) && a16(x_prev) && a16(hist_prev) && a16(x) && a16(w) && a16(dt_bias) &&
                a16(A_log) && a16(S_ckpt) && a16(H) && a16(o) && a16(y) && a16(hist_out),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(((uintptr_t)beta_raw % ie) == 0 && ((uintptr_t)alpha % ie) == 0 && ((uintptr_t)parent & 3) == 0 &&
                ((uintptr_t)node_prev & 3) == 0 && ((uintptr_t)parent_prev & 3) == 0,
            GDN_EINVAL, "%s: gate, node or parent pointers not aligned to their element size", fn);
    const size_t C = (size_t)2 * Hk * dk + (size_t)Hv * dv;
    const size_t st = (size_t)Hv * dv * dk * 4;
    const size_t gspan = ((size_t)B * N - 1) * gate_stride + Hv;
    const size_t hrows = (size_t)B * (W - 1) * C * ie;
    const Span ins[] = {Span{node_prev, node_prev ? (size_t)B * 4 : 0},
                        Span{node_prev ? parent_prev : nullptr, node_prev ? (size_t)B * N_prev * 4 : 0},
                        Span{S_prev_ckpt, B * st},
                        Span{node_prev ? H_prev : nullptr, node_prev ? (size_t)B * N_prev * st : 0},
                        Span{node_prev ? x_prev : nullptr, node_prev ? (size_t)B * N_prev * C * ie : 0},
                        Span{hist_prev, hrows},
                        Span{x, (size_t)B * N * C * ie},
                        Span{w, C * W * 4},
                        Span{parent, (size_t)B * N * 4},
                        Span{beta_raw, gspan * ie},
                        Span{alpha, gspan * ie},
                        Span{dt_bias, dt_bias ? (size_t)Hv * 4 : 0},
                        Span{A_log, A_log ? (size_t)Hv * 4 : 0}};
    const Span outs[] = {Span{S_ckpt, B * st}, Span{H, (size_t)B * N * st}, Span{o, (size_t)B * N * Hv * dv * oe},
                         Span{y, (size_t)B * N * C * ie}, Span{hist_out, hist_out ? hrows : 0}};
    for (const Span& q : outs)
        for (const Span& i : ins) REQUIRE(!overlap(q, i), GDN_EINVAL, "%s: an output overlaps an input", fn);
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j) REQUIRE(!overlap(outs[i], outs[j]), GDN_EINVAL, "%s: two outputs overlap", fn);
    // 1. the conv of every node, its history the previous tree's accepted path (then hist_prev)
    gdn::ConvTreeArgs c{x, w, hist_prev, parent, y, B, N, (int)C, W};
    c.node_prev = node_prev;
    c.parent_prev = parent_prev;
    c.x_prev = x_prev;
    c.N_prev = node_prev ? N_prev : 0;
    c.hist_out = hist_out;
    rc = launch_status(gdn::launch_conv_tree(c, in_dtype == GDN_BF16, (hipStream_t)stream), fn);
    if (rc) return rc;
    // 2. the tree verify from the start state the accepted node picks, written out as the checkpoint
    gdn::VerifyArgs a{y, beta_raw, alpha, dt_bias, A_log, S_prev_ckpt, nullptr, H, o, B, N, Hk, Hv, dk, dv, l2_eps,
                      nullptr, gate_stride, nullptr, parent};
    a.acc_prev = node_prev;
    a.Kp = node_prev ? N_prev : 0;
    a.Sp_ckpt = S_prev_ckpt;
    a.Sp_H = H_prev;
    a.S_ckpt = S_ckpt;
    a.pick = true;
    return launch_status(gdn::launch_verify(a, in_dtype == GDN_BF16, o_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_kv_reserve(const int32_t* lens, const int32_t* add, int32_t* table, int32_t* ref, int32_t* granted, int B,
                   int P, int n_pages, int page, void* stream)
{
    const char* fn = "gdn_kv_reserve";
    gdn::KvGeom g;
    int rc = check_kv(fn, 1, n_pages, 1, page, 64, GDN_F32, g);
    if (rc) return rc;
    REQUIRE(B >= 0 && P >= 1, GDN_EINVAL, "%s: B = %d, P = %d", fn, B, P);
    REQUIRE(B <= 65536, GDN_EUNSUPPORTED, "%s: B = %d > 65536", fn, B);
    if (B == 0) return ok();
    REQUIRE(lens && add && table && ref && granted, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned4(lens) && aligned4(add) && aligned4(table) && aligned4(ref) && aligned4(granted), GDN_EINVAL,
            "%s: pointers must be 4-byte aligned", fn);
    const Span outs[] = {ints(table, (size_t)B * P), ints(ref, n_pages), ints(granted, B)};
    const Span ins[] = {ints(lens, B), ints(add, B)};
    REQUIRE(!any_overlap(outs, 3, ins, 2), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    const gdn::KvReserveArgs a{lens, add, table, ref, granted, B, P, n_pages, g.page_log2};
    return launch_status(gdn::launch_kv_reserve(a, (hipStream_t)stream), fn);
}

int gdn_kv_append(const void* k, const void* v, long long kv_stride, void* k_pages, void* v_pages,
                  const int32_t* lens, const int32_t* count, const int32_t* table, int B, int K, int Hkv, int D,
                  int page, int n_pages, int P, int dtype, void* stream)
{
    const char* fn = "gdn_kv_append";
    gdn::KvGeom g;
    int rc = check_kv(fn, 1, n_pages, Hkv, page, D, dtype, g);
    if (rc) return rc;
    REQUIRE(B >= 0 && K >= 1 && P >= 1, GDN_EINVAL, "%s: B = %d, K = %d, P = %d", fn, B, K, P);
    REQUIRE(B <= 65535 && K <= 65536, GDN_EUNSUPPORTED, "%s: B = %d or K = %d too large", fn, B, K);
    REQUIRE((long long)K * Hkv * D * (int)elem_size(dtype) <= 1LL << 33, GDN_EUNSUPPORTED,
            "%s: a window of %d x %d x %d passes 2^33 bytes", fn, K, Hkv, D);
    if (B == 0) return ok();
    REQUIRE(k && v && k_pages && v_pages && lens && table, GDN_EINVAL, "%s: null pointer", fn);
    const size_t es = elem_size(dtype), token = (size_t)Hkv * D;
    REQUIRE(kv_stride >= (long long)token && kv_stride < (1LL << 40) && kv_stride * es % 16 == 0, GDN_EINVAL,
            "%s: kv_stride = %lld is below Hkv*D or no multiple of 16 bytes", fn, kv_stride);
    REQUIRE(aligned16(k) && aligned16(v) && aligned16(k_pages) && aligned16(v_pages), GDN_EINVAL,
            "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(aligned4(lens) && aligned4(count) && aligned4(table), GDN_EINVAL, "%s: lens, count and table must be "
            "4-byte aligned", fn);
    const size_t in = (((size_t)B * K - 1) * kv_stride + token) * es, plane = (size_t)n_pages * g.page_bytes();
    const Span outs[] = {Span{k_pages, plane}, Span{v_pages, plane}};
    const Span ins[] = {Span{k, in}, Span{v, in}, ints(lens, B), ints(count, B), ints(table, (size_t)B * P)};
    REQUIRE(!any_overlap(outs, 2, ins, 5), GDN_EINVAL, "%s: a plane overlaps another buffer", fn);
    const gdn::KvAppendArgs a{k, v, (size_t)kv_stride * es, k_pages, v_pages, lens, count, table, B, K, P, g};
    return launch_status(gdn::launch_kv_append(a, (hipStream_t)stream), fn);
}

int gdn_kv_rollback_tree(const int32_t* node, const int32_t* parent, const int32_t* lens, const int32_t* count,
                         int32_t* table, int32_t* ref, void* pool, int32_t* lens_out, int B, int N, int P, int planes,
                         int n_pages, int Hkv, int page, int D, int dtype, void* stream)
{
    const char* fn = "gdn_kv_rollback_tree";
    gdn::KvGeom g;
    int rc = check_kv(fn, planes, n_pages, Hkv, page, D, dtype, g);
    if (rc) return rc;
    REQUIRE(B >= 0 && N >= 1 && P >= 1, GDN_EINVAL, "%s: B = %d, N = %d, P = %d", fn, B, N, P);
    REQUIRE(N <= gdn::kKvWindowMax, GDN_EUNSUPPORTED, "%s: N = %d > %d", fn, N, gdn::kKvWindowMax);
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d too large", fn, B);
    if (B == 0) return ok();
    REQUIRE(node && lens && table && ref && pool && lens_out, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(pool), GDN_EINVAL, "%s: pool must be 16-byte aligned", fn);
    REQUIRE(aligned4(node) && aligned4(parent) && aligned4(lens) && aligned4(count) && aligned4(table) &&
                aligned4(ref) && aligned4(lens_out),
            GDN_EINVAL, "%s: int32 pointers must be 4-byte aligned", fn);
    const Span outs[] = {ints(table, (size_t)B * P), ints(ref, n_pages), ints(lens_out, B),
                         Span{pool, (size_t)planes * n_pages * g.page_bytes()}};
    const Span ins[] = {ints(node, B), ints(parent, (size_t)B * N), ints(count, B),
                        ints(lens == lens_out ? nullptr : lens, B)};
    REQUIRE(!any_overlap(outs, 4, ins, 4), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    const Span len_in[] = {ints(lens, B)};
    const Span rest[] = {outs[0], outs[1], outs[3]};
    for (const Span& o : rest) REQUIRE(!overlap(o, len_in[0]), GDN_EINVAL, "%s: an output overlaps lens", fn);
    const gdn::KvRollbackArgs a{node, parent, lens, count, table, ref, pool, lens_out, B, N, P, g};
    return launch_status(gdn::launch_kv_rollback(a, (hipStream_t)stream), fn);
}

int gdn_kv_free(const int32_t* rows, int32_t* lens, int32_t* table, int32_t* ref, int n, int B, int P, int n_pages,
                void* stream)
{
    const char* fn = "gdn_kv_free";
    gdn::KvGeom g;
    int rc = check_kv(fn, 1, n_pages, 1, 16, 64, GDN_F32, g);
    if (rc) return rc;
    REQUIRE(n >= 0 && B >= 0 && P >= 1, GDN_EINVAL, "%s: n = %d, B = %d, P = %d", fn, n, B, P);
    REQUIRE(n <= 1 << 20, GDN_EUNSUPPORTED, "%s: n = %d > 2^20", fn, n);
    if (n == 0 || B == 0) return ok();
    REQUIRE(rows && lens && table && ref, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned4(rows) && aligned4(lens) && aligned4(table) && aligned4(ref), GDN_EINVAL,
            "%s: pointers must be 4-byte aligned", fn);
    const Span outs[] = {ints(lens, B), ints(table, (size_t)B * P), ints(ref, n_pages)};
    const Span ins[] = {ints(rows, n)};
    REQUIRE(!any_overlap(outs, 3, ins, 1), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    return launch_status(gdn::launch_kv_free(rows, lens, table, ref, n, B, P, n_pages, (hipStream_t)stream), fn);
}

int gdn_kv_fork(const int32_t* src, const int32_t* dst, int32_t* lens, int32_t* table, int32_t* ref, void* pool,
                int32_t* granted, int n, int B, int P, int planes, int n_pages, int Hkv, int page, int D, int dtype,
                void* stream)
{
    const char* fn = "gdn_kv_fork";
    gdn::KvGeom g;
    int rc = check_kv(fn, planes, n_pages, Hkv, page, D, dtype, g);
    if (rc) return rc;
    REQUIRE(n >= 0 && B >= 0 && P >= 1, GDN_EINVAL, "%s: n = %d, B = %d, P = %d", fn, n, B, P);
    REQUIRE(n <= gdn::kKvForkMax, GDN_EUNSUPPORTED, "%s: n = %d > %d", fn, n, gdn::kKvForkMax);
    if (n == 0) return ok();
    REQUIRE(B >= 1, GDN_EINVAL, "%s: %d forks of no rows", fn, n);
    REQUIRE(src && dst && lens && table && ref && pool && granted, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(pool), GDN_EINVAL, "%s: pool must be 16-byte aligned", fn);
    REQUIRE(aligned4(src) && aligned4(dst) && aligned4(lens) && aligned4(table) && aligned4(ref) && aligned4(granted),
            GDN_EINVAL, "%s: int32 pointers must be 4-byte aligned", fn);
    const Span outs[] = {ints(lens, B), ints(table, (size_t)B * P), ints(ref, n_pages), ints(granted, n),
                         Span{pool, (size_t)planes * n_pages * g.page_bytes()}};
    const Span ins[] = {ints(src, n), ints(dst, n)};
    REQUIRE(!any_overlap(outs, 5, ins, 2), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    const gdn::KvForkArgs a{src, dst, lens, table, ref, pool, granted, n, B, P, g};
    return launch_status(gdn::launch_kv_fork(a, (hipStream_t)stream), fn);
}

int gdn_kv_compact_workspace(int n_pages, size_t* bytes)
{
    const char* fn = "gdn_kv_compact_workspace";
    gdn::KvGeom g;
    int rc = check_kv(fn, 1, n_pages, 1, 16, 64, GDN_F32, g);
    if (rc) return rc;
    REQUIRE(bytes, GDN_EINVAL, "%s: null bytes", fn);
    *bytes = gdn::kv_compact_words(n_pages) * 4;
    return ok();
}

int gdn_kv_compact(const int32_t* table, const int32_t* ref, void* pool, int32_t* table_out, int32_t* ref_out,
                   void* workspace, size_t workspace_bytes, long long entries, int planes, int n_pages, int Hkv,
                   int page, int D, int dtype, void* stream)
{
    const char* fn = "gdn_kv_compact";
    gdn::KvGeom g;
    int rc = check_kv(fn, planes, n_pages, Hkv, page, D, dtype, g);
    if (rc) return rc;
    REQUIRE(entries >= 0 && entries < (1LL << 40), GDN_EINVAL, "%s: entries = %lld", fn, entries);
    REQUIRE(ref && pool && ref_out && workspace && (entries == 0 || (table && table_out)), GDN_EINVAL,
            "%s: null pointer", fn);
    REQUIRE(aligned16(pool) && aligned16(workspace), GDN_EINVAL, "%s: pool and workspace must be 16-byte aligned", fn);
    REQUIRE(aligned4(table) && aligned4(ref) && aligned4(table_out) && aligned4(ref_out), GDN_EINVAL,
            "%s: int32 pointers must be 4-byte aligned", fn);
    const size_t need = gdn::kv_compact_words(n_pages) * 4;
    REQUIRE(workspace_bytes >= need, GDN_EINVAL, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
    const Span outs[] = {ints(table_out, entries), ints(ref_out, n_pages), Span{workspace, need},
                         Span{pool, (size_t)planes * n_pages * g.page_bytes()}};
    const Span ins[] = {ints(table, entries), ints(ref, n_pages)};
    REQUIRE(!any_overlap(outs, 4, ins, 2), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    const gdn::KvCompactArgs a{table, ref, pool, table_out, ref_out, static_cast<int32_t*>(workspace), entries, g};
    return launch_status(gdn::launch_kv_compact(a, (hipStream_t)stream), fn);
}

int gdn_kv_copy(const int32_t* src, const int32_t* dst, void* pool, int n, int planes, int n_pages, int Hkv, int page,
                int D, int dtype, void* stream)
{
    const char* fn = "gdn_kv_copy";
    gdn::KvGeom g;
    int rc = check_kv(fn, planes, n_pages, Hkv, page, D, dtype, g);
    if (rc) return rc;
    REQUIRE(n >= 0, GDN_EINVAL, "%s: n = %d < 0", fn, n);
    REQUIRE(gdn::kv_copy_countable(n, g), GDN_EUNSUPPORTED, "%s: %d pages in %d planes are too many pieces", fn, n, planes);
    if (n == 0) return ok();
    REQUIRE(src && dst && pool, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(pool) && aligned4(src) && aligned4(dst), GDN_EINVAL,
            "%s: pool must be 16-byte, src and dst 4-byte aligned", fn);
    const Span outs[] = {Span{pool, (size_t)planes * n_pages * g.page_bytes()}};
    const Span ins[] = {ints(src, n), ints(dst, n)};
    REQUIRE(!any_overlap(outs, 1, ins, 2), GDN_EINVAL, "%s: the pool overlaps src or dst", fn);
    return launch_status(gdn::launch_kv_copy(src, dst, pool, n, g, (hipStream_t)stream), fn);
}

static int check_attn(const char* fn, int B, int K, int Hq, int Hkv, int D, int page, int P, int prefix_len, int dtype,
                      int n_pages, gdn::KvGeom& g)
{
    int rc = check_kv(fn, 1, n_pages, Hkv, page, D, dtype, g);
    if (rc) return rc;
    REQUIRE(B >= 0 && K >= 1 && P >= 1, GDN_EINVAL, "%s: B = %d, K = %d, P = %d", fn, B, K, P);
    REQUIRE(Hq >= 1 && Hq % Hkv == 0, GDN_EINVAL, "%s: Hq = %d is not a multiple of Hkv = %d", fn, Hq, Hkv);
    REQUIRE(prefix_len >= 0 && prefix_len % page == 0 && prefix_len / page <= P, GDN_EINVAL,
            "%s: prefix_len = %d is no multiple of page = %d within %d slots", fn, prefix_len, page, P);
    REQUIRE(K <= gdn::kKvWindowMax, GDN_EUNSUPPORTED, "%s: K = %d > %d", fn, K, gdn::kKvWindowMax);
    REQUIRE(B <= gdn::kAttnBatchMax, GDN_EUNSUPPORTED, "%s: B = %d > %d", fn, B, gdn::kAttnBatchMax);
    REQUIRE(Hq <= 1024, GDN_EUNSUPPORTED, "%s: Hq = %d > 1024", fn, Hq);
    REQUIRE((long long)P * page <= (1LL << 30), GDN_EUNSUPPORTED, "%s: %d slots of %d tokens pass 2^30", fn, P, page);
    return GDN_OK;
}

int gdn_attn_workspace(int B, int K, int Hq, int Hkv, int D, int page, int P, int prefix_len, int dtype, size_t* bytes)
{
    const char* fn = "gdn_attn_workspace";
    gdn::KvGeom g;
    int rc = check_attn(fn, B, K, Hq, Hkv, D, page, P, prefix_len, dtype, 1, g);
    if (rc) return rc;
    REQUIRE(bytes, GDN_EINVAL, "%s: null bytes", fn);
    const size_t need = gdn::attn_work_bytes(B, K, Hq, Hkv, D, g.page_log2, P, prefix_len, dtype == GDN_BF16);
    REQUIRE(need > 0, GDN_EUNSUPPORTED, "%s: %d tables of %d slots pass 2^31 units of work", fn, B, P);
    *bytes = need;
    return ok();
}

int gdn_attn_verify(const void* q, long long q_stride, const void* k_pages, const void* v_pages, const int32_t* lens,
                    const int32_t* count, const int32_t* parent, const int32_t* table, void* o, float* lse,
                    void* workspace, size_t workspace_bytes, int B, int K, int Hq, int Hkv, int D, int page,
                    int n_pages, int P, int prefix_len, float scale, int dtype, void* stream)
{
    const char* fn = "gdn_attn_verify";
    gdn::KvGeom g;
    int rc = check_attn(fn, B, K, Hq, Hkv, D, page, P, prefix_len, dtype, n_pages, g);
    if (rc) return rc;
    REQUIRE(scale - scale == 0.0f, GDN_EINVAL, "%s: scale is not finite", fn);
    if (B == 0) return ok();
    REQUIRE(q && k_pages && v_pages && lens && table && o && workspace, GDN_EINVAL, "%s: null pointer", fn);
    const size_t es = elem_size(dtype), token = (size_t)Hq * D;
    REQUIRE(q_stride >= (long long)token && q_stride < (1LL << 40) && q_stride * es % 16 == 0, GDN_EINVAL,
            "%s: q_stride = %lld is below Hq*D or no multiple of 16 bytes", fn, q_stride);
    REQUIRE(aligned16(q) && aligned16(k_pages) && aligned16(v_pages) && aligned16(o) && aligned16(workspace),
            GDN_EINVAL, "%s: pointers must be 16-byte aligned", fn);
    REQUIRE(aligned4(lens) && aligned4(count) && aligned4(parent) && aligned4(table) && aligned4(lse), GDN_EINVAL,
            "%s: lens, count, parent, table and lse must be 4-byte aligned", fn);
    const bool bf16 = dtype == GDN_BF16;
    const size_t need = gdn::attn_work_bytes(B, K, Hq, Hkv, D, g.page_log2, P, prefix_len, bf16);
    REQUIRE(need > 0, GDN_EUNSUPPORTED, "%s: %d tables of %d slots pass 2^31 units of work", fn, B, P);
    REQUIRE(workspace_bytes >= need, GDN_EINVAL, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
    const size_t plane = (size_t)n_pages * g.page_bytes(), rows = (size_t)B * K;
    const Span outs[] = {Span{o, rows * token * es}, Span{lse, lse ? rows * Hq * 4 : 0}, Span{workspace, need}};
    const Span ins[] = {Span{q, ((rows - 1) * q_stride + token) * es}, Span{k_pages, plane}, Span{v_pages, plane},
                        ints(lens, B), ints(count, B), ints(parent, rows), ints(table, (size_t)B * P)};
    REQUIRE(!any_overlap(outs, 3, ins, 7), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    const gdn::AttnArgs a{q, (size_t)q_stride, k_pages, v_pages, lens, count, parent, table, o, lse, workspace,
                          B, K, Hq, Hkv, D, g.page_log2, n_pages, P, prefix_len, scale, 0, 0, {}};
    return launch_status(gdn::launch_attn(a, bf16, (hipStream_t)stream), fn);
}

}  // extern "C"

namespace {

// Where x [B][K][H][D] lies: strides in elements from one sequence, token and head to the next (NULL: dense), as bytes
// in `step` (0 where there is no next), and the bytes from its first to its last element in `bytes`.  An output's rows
// must not meet one another (`apart`).
int check_heads(const char* fn, const char* what, const long long* strides, int B, int K, int H, int D, size_t es,
                bool apart, long long step[3], size_t& bytes)
{
    const long long n[3] = {B, K, H};
    const long long dense[3] = {(long long)K * H * D, (long long)H * D, D};
    const long long row = (long long)D * (long long)es;
    long long last = 0;
    for (int i = 0; i < 3; ++i) {
        const long long s = strides ? strides[i] : dense[i];
        step[i] = 0;
        if (n[i] <= 1) continue;
        REQUIRE(s >= 0 && s < (1LL << 40) && s * (long long)es % 16 == 0, GDN_EINVAL,
                "%s: a stride of %s (%lld) is below 0, too large or no multiple of 16 bytes", fn, what, s);
        step[i] = s * (long long)es;
        REQUIRE(step[i] == 0 || n[i] - 1 <= (1LL << 46) / step[i], GDN_EUNSUPPORTED, "%s: %s passes 2^46 bytes", fn, what);
        last += (n[i] - 1) * step[i];
    }
    if (apart) {
        // from the smallest step on, each has to pass what the smaller ones reach
        bool done[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
        long long reach = row;
        for (int k = 0; k < 3; ++k) {
            int m = -1;
            for (int i = 0; i < 3; ++i)
                if (!done[i] && (m < 0 || step[i] < step[m])) m = i;
            if (m < 0) break;
            REQUIRE(step[m] >= reach, GDN_EINVAL, "%s: rows of %s overlap", fn, what);
            reach += (n[m] - 1) * step[m];
            done[m] = true;
        }
    }
    bytes = (size_t)(last + row);
    return GDN_OK;
}

// what the three rotary calls share
int check_rope(const char* fn, int B, int K, int D, const int32_t* parent, const double* freqs, int rot, int layout,
               float mscale, float eps, int dtype, bool may_rest)
{
    REQUIRE(valid_dtype(dtype), GDN_EINVAL, "%s: bad dtype code %d", fn, dtype);
    REQUIRE(B >= 0 && K >= 1 && D >= 1, GDN_EINVAL, "%s: B = %d, K = %d, D = %d", fn, B, K, D);
    REQUIRE(layout == GDN_ROPE_HALVES || layout == GDN_ROPE_INTERLEAVED, GDN_EINVAL, "%s: bad layout code %d", fn, layout);
    REQUIRE(rot >= 0 && rot % 2 == 0 && rot <= D, GDN_EINVAL, "%s: rot = %d is odd or outside 0..D = %d", fn, rot, D);
    REQUIRE(rot > 0 || may_rest, GDN_EINVAL, "%s: rot = 0 leaves nothing to do", fn);
    REQUIRE(mscale - mscale == 0.0f, GDN_EINVAL, "%s: mscale is not finite", fn);
    REQUIRE(eps >= 0.0f && eps - eps == 0.0f, GDN_EINVAL, "%s: eps is below 0 or not finite", fn);
    REQUIRE(D % 16 == 0 && D <= gdn::kRopeHeadMax, GDN_EUNSUPPORTED, "%s: D = %d is no multiple of 16 up to %d", fn, D,
            gdn::kRopeHeadMax);
    REQUIRE(B <= 65535 && K <= 65536 && (long long)B * K < (1LL << 31), GDN_EUNSUPPORTED, "%s: B = %d, K = %d too large",
            fn, B, K);
    REQUIRE(!parent || K <= gdn::kKvWindowMax, GDN_EUNSUPPORTED, "%s: a tree of K = %d > %d nodes", fn, K,
            gdn::kKvWindowMax);
    REQUIRE(rot == 0 || freqs || B == 0, GDN_EINVAL, "%s: null freqs", fn);
    REQUIRE((reinterpret_cast<uintptr_t>(freqs) & 7u) == 0, GDN_EINVAL, "%s: freqs must be 8-byte aligned", fn);
    return GDN_OK;
}

bool heads_in_range(int H) { return H >= 1 && H <= 1024; }

}  // namespace

extern "C" {

int gdn_rope_freqs(int rot, double base, int scaling, double factor, double low, double high, double original,
                   double* freqs, float* mscale)
{
    const char* fn = "gdn_rope_freqs";
    REQUIRE(rot >= 2 && rot % 2 == 0, GDN_EINVAL, "%s: rot = %d is odd or below 2", fn, rot);
    REQUIRE(rot <= gdn::kRopeHeadMax, GDN_EUNSUPPORTED, "%s: rot = %d > %d", fn, rot, gdn::kRopeHeadMax);
    REQUIRE(std::isfinite(base) && base > 1.0, GDN_EINVAL, "%s: base = %g is not above 1", fn, base);
    REQUIRE(scaling >= GDN_ROPE_PLAIN && scaling <= GDN_ROPE_YARN_ROUNDED, GDN_EINVAL, "%s: bad scaling code %d", fn, scaling);
    REQUIRE(freqs && mscale, GDN_EINVAL, "%s: null pointer", fn);
    if (scaling != GDN_ROPE_PLAIN)
        REQUIRE(std::isfinite(factor) && factor >= 1.0, GDN_EINVAL, "%s: factor = %g is below 1", fn, factor);
    if (scaling == GDN_ROPE_NTK) REQUIRE(rot > 2, GDN_EINVAL, "%s: one pair has no base to enlarge", fn);
    if (scaling >= GDN_ROPE_BANDS)
        REQUIRE(std::isfinite(original) && original > 0.0 && low > 0.0 && high > low && std::isfinite(high), GDN_EINVAL,
                "%s: original = %g, low = %g, high = %g", fn, original, low, high);
    if (scaling == GDN_ROPE_YARN)   // (its logarithm divides)
        REQUIRE(high / low > 1.0 && std::isfinite(high / low), GDN_EUNSUPPORTED, "%s: high / low = %g", fn, high / low);
    const double two_pi = 6.283185307179586476925;
    if (scaling == GDN_ROPE_NTK) {
        base *= std::pow(factor, (double)rot / (rot - 2));
        REQUIRE(std::isfinite(base), GDN_EUNSUPPORTED, "%s: the enlarged base passes 64 bits", fn);
    }
    // the pair that turns n times over the original context, as a number between the pairs
    auto pair_of = [&](double n) { return rot * std::log(original / (n * two_pi)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == GDN_ROPE_YARN_ROUNDED) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        const double turns = original * f / two_pi;   // over the original context
        // how much of the frequency is kept, the rest being divided by the factor
        double keep = scaling == GDN_ROPE_LINEAR ? 0.0 : 1.0;
        if (scaling == GDN_ROPE_BANDS) keep = (turns - low) / (high - low);
        // (the pair's index is linear in the logarithm of its turns)
        if (scaling == GDN_ROPE_YARN) keep = std::log(turns / low) / std::log(high / low);
        if (scaling == GDN_ROPE_YARN_ROUNDED) keep = i <= first ? 1.0 : i >= last ? 0.0 : (last - i) / (last - first);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        freqs[i] = keep == 1.0 ? f : keep * f + (1.0 - keep) * f / factor;
    }
    *mscale = scaling >= GDN_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return ok();
}

int gdn_rope(const void* x, const long long* x_strides, void* y, const long long* y_strides, const int32_t* pos,
             const int32_t* lens, const int32_t* parent, const int32_t* count, const double* freqs, int rot, int layout,
             float mscale, int B, int K, int H, int D, int dtype, void* stream)
{
    const char* fn = "gdn_rope";
    int rc = check_rope(fn, B, K, D, parent, freqs, rot, layout, mscale, 0.0f, dtype, false);
    if (rc) return rc;
    REQUIRE(H >= 1, GDN_EINVAL, "%s: H = %d < 1", fn, H);
    REQUIRE(heads_in_range(H), GDN_EUNSUPPORTED, "%s: H = %d > 1024", fn, H);
    if (B == 0) return ok();
    REQUIRE(x && y, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(x) && aligned16(y), GDN_EINVAL, "%s: x and y must be 16-byte aligned", fn);
    REQUIRE(aligned4(pos) && aligned4(lens) && aligned4(parent) && aligned4(count), GDN_EINVAL,
            "%s: int32 pointers must be 4-byte aligned", fn);
    const size_t es = elem_size(dtype), tokens = (size_t)B * K;
    gdn::RopeArgs a{};
    gdn::RopePart& q = a.part[0];
    size_t in, out;
    if ((rc = check_heads(fn, "x", x_strides, B, K, H, D, es, false, q.xs, in))) return rc;
    if ((rc = check_heads(fn, "y", y_strides, B, K, H, D, es, true, q.ys, out))) return rc;
    const bool in_place = x == y && memcmp(q.xs, q.ys, sizeof(q.xs)) == 0;
    const Span outs[] = {Span{y, out}};
    const Span ins[] = {Span{in_place ? nullptr : x, in}, ints(pos, tokens), ints(lens, B), ints(parent, tokens),
                        ints(count, B), Span{freqs, (size_t)rot / 2 * 8}};
    REQUIRE(!any_overlap(outs, 1, ins, 6), GDN_EINVAL, "%s: y overlaps an input", fn);
    q.x = x, q.y = y, q.H = H, q.turned = 1;
    a.pos = pos, a.lens = lens, a.parent = parent, a.count = count, a.freqs = freqs;
    a.rot = rot, a.mscale = mscale, a.B = B, a.K = K, a.D = D;
    return launch_status(gdn::launch_rope(a, dtype == GDN_BF16, layout == GDN_ROPE_INTERLEAVED, (hipStream_t)stream), fn);
}

int gdn_qk_norm_rope(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                     const float* wq, const float* wk, float eps, void* q_out, void* k_out, const int32_t* pos,
                     const int32_t* lens, const int32_t* parent, const int32_t* count, const double* freqs, int rot,
                     int layout, float mscale, int B, int K, int Hq, int Hk, int D, int dtype, void* stream)
{
    const char* fn = "gdn_qk_norm_rope";
    int rc = check_rope(fn, B, K, D, parent, freqs, rot, layout, mscale, eps, dtype, true);
    if (rc) return rc;
    REQUIRE(Hq >= 1 && Hk >= 1, GDN_EINVAL, "%s: Hq = %d, Hk = %d must be >= 1", fn, Hq, Hk);
    REQUIRE(heads_in_range(Hq) && heads_in_range(Hk), GDN_EUNSUPPORTED, "%s: Hq = %d or Hk = %d > 1024", fn, Hq, Hk);
    if (B == 0) return ok();
    REQUIRE(q && k && wq && wk && q_out && k_out, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned16(q) && aligned16(k) && aligned16(q_out) && aligned16(k_out), GDN_EINVAL,
            "%s: q, k, q_out and k_out must be 16-byte aligned", fn);
    REQUIRE(aligned4(wq) && aligned4(wk) && aligned4(pos) && aligned4(lens) && aligned4(parent) && aligned4(count),
            GDN_EINVAL, "%s: weights and int32 pointers must be 4-byte aligned", fn);
    const size_t es = elem_size(dtype), tokens = (size_t)B * K;
    gdn::RopeArgs a{};
    const void* x[2] = {q, k};
    void* y[2] = {q_out, k_out};
    const long long* strides[2] = {q_strides, k_strides};
    const float* w[2] = {wq, wk};
    const int H[2] = {Hq, Hk};
    const char* name[2] = {"q", "k"};
    size_t in[2], out[2];
    bool in_place[2];
    for (int i = 0; i < 2; ++i) {
        gdn::RopePart& p = a.part[i];
        if ((rc = check_heads(fn, name[i], strides[i], B, K, H[i], D, es, false, p.xs, in[i]))) return rc;
        if ((rc = check_heads(fn, name[i], nullptr, B, K, H[i], D, es, true, p.ys, out[i]))) return rc;
        p.x = x[i], p.y = y[i], p.w = w[i], p.H = H[i], p.turned = 1;
        in_place[i] = x[i] == y[i] && memcmp(p.xs, p.ys, sizeof(p.xs)) == 0;
    }
    // a dense q may be q_out, a dense k k_out; nothing else may be shared
    const Span spans[] = {Span{q, in[0]}, Span{k, in[1]}};
    const Span outs[] = {Span{q_out, out[0]}, Span{k_out, out[1]}};
    const Span ins[] = {ints(pos, tokens), ints(lens, B), ints(parent, tokens), ints(count, B), Span{wq, (size_t)D * 4},
                        Span{wk, (size_t)D * 4}, Span{freqs, (size_t)rot / 2 * 8}};
    REQUIRE(!any_overlap(outs, 2, ins, 7), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            REQUIRE((i == j && in_place[i]) || !overlap(outs[i], spans[j]), GDN_EINVAL, "%s: %s_out overlaps %s", fn,
                    name[i], name[j]);
    a.pos = pos, a.lens = lens, a.parent = parent, a.count = count, a.freqs = freqs;
    a.rot = rot, a.mscale = mscale, a.eps = eps, a.B = B, a.K = K, a.D = D;
    return launch_status(gdn::launch_rope(a, dtype == GDN_BF16, layout == GDN_ROPE_INTERLEAVED, (hipStream_t)stream), fn);
}

int gdn_kv_append_rope(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                       const void* v, const long long* v_strides, const float* wq, const float* wk, float eps,
                       void* q_out, void* k_pages, void* v_pages, const int32_t* pos, const int32_t* lens,
                       const int32_t* parent, const int32_t* count, const int32_t* table, const double* freqs, int rot,
                       int layout, float mscale, int B, int K, int Hq, int Hkv, int D, int page, int n_pages, int P,
                       int dtype, void* stream)
{
    const char* fn = "gdn_kv_append_rope";
    gdn::RopeArgs a{};
    int rc = check_kv(fn, 1, n_pages, Hkv, page, D, dtype, a.g);
    if (rc) return rc;
    if ((rc = check_rope(fn, B, K, D, parent, freqs, rot, layout, mscale, eps, dtype, true))) return rc;
    REQUIRE(P >= 1, GDN_EINVAL, "%s: P = %d < 1", fn, P);
    REQUIRE(Hq >= 0, GDN_EINVAL, "%s: Hq = %d < 0", fn, Hq);
    REQUIRE(Hq <= 1024, GDN_EUNSUPPORTED, "%s: Hq = %d > 1024", fn, Hq);
    if (B == 0) return ok();
    REQUIRE(k && v && k_pages && v_pages && lens && table, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE((q != nullptr) == (Hq > 0) && (q_out != nullptr) == (Hq > 0), GDN_EINVAL,
            "%s: q and q_out are both given (Hq heads) or both NULL (Hq = 0)", fn);
    REQUIRE(!wq || Hq > 0, GDN_EINVAL, "%s: wq without q", fn);
    REQUIRE(aligned16(q) && aligned16(k) && aligned16(v) && aligned16(q_out) && aligned16(k_pages) && aligned16(v_pages),
            GDN_EINVAL, "%s: q, k, v, q_out and the planes must be 16-byte aligned", fn);
    REQUIRE(aligned4(wq) && aligned4(wk) && aligned4(pos) && aligned4(lens) && aligned4(parent) && aligned4(count) &&
                aligned4(table),
            GDN_EINVAL, "%s: weights and int32 pointers must be 4-byte aligned", fn);
    const size_t es = elem_size(dtype), tokens = (size_t)B * K, plane = (size_t)n_pages * a.g.page_bytes();
    gdn::RopePart &pq = a.part[0], &pk = a.part[1], &pv = a.part[2];
    size_t in_q = 0, in_k, in_v, out_q = 0;
    if (Hq > 0) {
        if ((rc = check_heads(fn, "q", q_strides, B, K, Hq, D, es, false, pq.xs, in_q))) return rc;
        if ((rc = check_heads(fn, "q_out", nullptr, B, K, Hq, D, es, true, pq.ys, out_q))) return rc;
    }
    if ((rc = check_heads(fn, "k", k_strides, B, K, Hkv, D, es, false, pk.xs, in_k))) return rc;
    if ((rc = check_heads(fn, "v", v_strides, B, K, Hkv, D, es, false, pv.xs, in_v))) return rc;
    pq.x = q, pq.y = q_out, pq.w = wq, pq.H = Hq, pq.turned = 1;
    pk.x = k, pk.y = k_pages, pk.w = wk, pk.H = Hkv, pk.turned = 1, pk.paged = 1;
    pv.x = v, pv.y = v_pages, pv.H = Hkv, pv.paged = 1;
    const bool in_place = q == q_out && memcmp(pq.xs, pq.ys, sizeof(pq.xs)) == 0;
    const Span sq{q, in_q}, so{q_out, out_q};
    const Span outs[] = {so, Span{k_pages, plane}, Span{v_pages, plane}};
    const Span ins[] = {Span{k, in_k}, Span{v, in_v}, ints(pos, tokens), ints(lens, B), ints(parent, tokens),
                        ints(count, B), ints(table, (size_t)B * P), Span{wq, (size_t)D * 4}, Span{wk, (size_t)D * 4},
                        Span{freqs, (size_t)rot / 2 * 8}};
    REQUIRE(!any_overlap(outs, 3, ins, 10), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    REQUIRE(!overlap(outs[1], sq) && !overlap(outs[2], sq) && (in_place || !overlap(so, sq)), GDN_EINVAL,
            "%s: an output overlaps q", fn);
    a.pos = pos, a.lens = lens, a.parent = parent, a.count = count, a.table = table, a.freqs = freqs;
    a.rot = rot, a.mscale = mscale, a.eps = eps, a.B = B, a.K = K, a.D = D, a.P = P;
    return launch_status(gdn::launch_rope(a, dtype == GDN_BF16, layout == GDN_ROPE_INTERLEAVED, (hipStream_t)stream), fn);
}

static int check_logits(const char* fn, int B, int K, int V)
{
    REQUIRE(B >= 0 && K >= 1 && V >= 1, GDN_EINVAL, "%s: B = %d, K = %d, V = %d", fn, B, K, V);
    REQUIRE(B <= 65535, GDN_EUNSUPPORTED, "%s: B = %d > 65535", fn, B);
    REQUIRE(K <= gdn::kKvWindowMax, GDN_EUNSUPPORTED, "%s: K = %d > %d", fn, K, gdn::kKvWindowMax);
    REQUIRE(V <= 1 << 24, GDN_EUNSUPPORTED, "%s: V = %d > 2^24", fn, V);
    return GDN_OK;
}

int gdn_logits_workspace(int B, int K, int V, size_t* bytes)
{
    const char* fn = "gdn_logits_workspace";
    int rc = check_logits(fn, B, K, V);
    if (rc) return rc;
    REQUIRE(bytes, GDN_EINVAL, "%s: null bytes", fn);
    *bytes = (size_t)B * K * gdn::logits_slices(V) * 8;
    return ok();
}

int gdn_logits_adjust(const void* logits, long long logits_stride, void* out, long long out_stride, int32_t* best,
                      const int32_t* history, const int32_t* history_lens, const int32_t* history_start, int capacity,
                      const int32_t* tokens, const int32_t* parent, const int32_t* count, const float* params,
                      const int32_t* bias_ids, const float* bias_values, int n_bias, const uint32_t* mask,
                      const float* noise, void* workspace, size_t workspace_bytes, int B, int K, int V, int dtype,
                      int out_dtype, void* stream)
{
    const char* fn = "gdn_logits_adjust";
    int rc = check_logits(fn, B, K, V);
    if (rc) return rc;
    REQUIRE(valid_dtype(dtype) && valid_dtype(out_dtype), GDN_EINVAL, "%s: bad dtype code (%d, %d)", fn, dtype, out_dtype);
    REQUIRE(n_bias >= 0 && n_bias <= 1 << 20, GDN_EINVAL, "%s: n_bias = %d is not in 0..2^20", fn, n_bias);
    if (B == 0) return ok();
    REQUIRE(logits && (out || best), GDN_EINVAL, "%s: null logits, or neither out nor best", fn);
    const size_t es = elem_size(dtype), oe = elem_size(out_dtype), rows = (size_t)B * K;
    REQUIRE(logits_stride >= V && logits_stride < (1LL << 40), GDN_EINVAL, "%s: logits_stride = %lld < V = %d", fn,
            logits_stride, V);
    if (out)
        REQUIRE(out_stride >= V && out_stride < (1LL << 40), GDN_EINVAL, "%s: out_stride = %lld < V = %d", fn, out_stride, V);
    REQUIRE(aligned16(logits) && aligned16(out) && aligned16(noise) && aligned16(workspace), GDN_EINVAL,
            "%s: logits, out, noise and workspace must be 16-byte aligned", fn);
    REQUIRE(aligned4(best) && aligned4(history) && aligned4(history_lens) && aligned4(history_start) &&
                aligned4(tokens) && aligned4(parent) && aligned4(count) && aligned4(params) && aligned4(bias_ids) &&
                aligned4(bias_values) && aligned4(mask),
            GDN_EINVAL, "%s: int32 and float pointers must be 4-byte aligned", fn);
    if (history) {
        REQUIRE(history_lens, GDN_EINVAL, "%s: history without history_lens", fn);
        REQUIRE(capacity >= 1 && capacity <= 1 << 29, GDN_EINVAL, "%s: capacity = %d is not in 1..2^29", fn, capacity);
    }
    REQUIRE(n_bias == 0 || (bias_ids && bias_values), GDN_EINVAL, "%s: biases without bias_ids or bias_values", fn);
    REQUIRE(!noise || best, GDN_EINVAL, "%s: noise is for finding best", fn);
    size_t need = 0;
    if (best) {
        need = rows * gdn::logits_slices(V) * 8;
        REQUIRE(workspace && workspace_bytes >= need, GDN_EINVAL, "%s: workspace of %zu bytes, %zu needed", fn,
                workspace ? workspace_bytes : (size_t)0, need);
    }
    const bool in_place = logits == out && dtype == out_dtype && logits_stride == out_stride;
    const Span sx{logits, ((rows - 1) * logits_stride + V) * es};
    const Span outs[] = {Span{out, out ? ((rows - 1) * out_stride + V) * oe : 0}, ints(best, rows),
                         Span{best ? workspace : nullptr, need}};
    const Span ins[] = {ints(history, history ? (size_t)B * capacity : 0), ints(history_lens, B), ints(history_start, B),
                        ints(tokens, rows), ints(parent, rows), ints(count, B), Span{params, (size_t)B * 16},
                        ints(n_bias ? bias_ids : nullptr, (size_t)B * n_bias),
                        Span{n_bias ? bias_values : nullptr, (size_t)B * n_bias * 4},
                        Span{mask, rows * (((size_t)V + 31) / 32) * 4}, Span{noise, rows * V * 4}};
    REQUIRE(!any_overlap(outs, 3, ins, 11), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    REQUIRE(!overlap(outs[1], sx) && !overlap(outs[2], sx) && (in_place || !overlap(outs[0], sx)), GDN_EINVAL,
            "%s: an output overlaps logits", fn);
    gdn::LogitsArgs a{};
    a.x = logits, a.out = out, a.x_stride = (size_t)logits_stride, a.out_stride = out ? (size_t)out_stride : 0;
    a.best = best, a.history = history, a.history_lens = history_lens, a.history_start = history_start;
    a.tokens = tokens, a.parent = parent, a.count = count, a.params = params, a.bias_ids = bias_ids;
    a.bias_values = bias_values, a.mask = mask, a.noise = noise, a.work = static_cast<unsigned long long*>(workspace);
    a.B = B, a.K = K, a.V = V, a.capacity = capacity, a.n_bias = n_bias;
    return launch_status(gdn::launch_logits(a, dtype == GDN_BF16, out_dtype == GDN_BF16, (hipStream_t)stream), fn);
}

int gdn_accept_tree(const int32_t* target, const int32_t* tokens, const int32_t* parent, const int32_t* count,
                    const int32_t* root, int32_t* node, int32_t* next, int32_t* history, const int32_t* lens,
                    int32_t* lens_out, int capacity, int B, int K, void* stream)
{
    const char* fn = "gdn_accept_tree";
    REQUIRE(B >= 0 && K >= 1, GDN_EINVAL, "%s: B = %d, K = %d", fn, B, K);
    REQUIRE(K <= gdn::kKvWindowMax, GDN_EUNSUPPORTED, "%s: K = %d > %d", fn, K, gdn::kKvWindowMax);
    REQUIRE(B <= 1 << 20, GDN_EUNSUPPORTED, "%s: B = %d > 2^20", fn, B);
    if (B == 0) return ok();
    REQUIRE(target && tokens && node && next, GDN_EINVAL, "%s: null pointer", fn);
    REQUIRE((history != nullptr) == (lens != nullptr) && (history != nullptr) == (lens_out != nullptr), GDN_EINVAL,
            "%s: history, lens and lens_out are all given or all NULL", fn);
    if (history)
        REQUIRE(capacity >= 1 && capacity <= 1 << 29, GDN_EINVAL, "%s: capacity = %d is not in 1..2^29", fn, capacity);
    REQUIRE(aligned4(target) && aligned4(tokens) && aligned4(parent) && aligned4(count) && aligned4(root) &&
                aligned4(node) && aligned4(next) && aligned4(history) && aligned4(lens) && aligned4(lens_out),
            GDN_EINVAL, "%s: pointers must be 4-byte aligned", fn);
    const size_t n = (size_t)B * K;
    const Span outs[] = {ints(node, B), ints(next, B), ints(history, history ? (size_t)B * capacity : 0),
                         ints(lens_out, B)};
    const Span ins[] = {ints(target, n), ints(tokens, n), ints(parent, n), ints(count, B), ints(root, B),
                        ints(lens == lens_out ? nullptr : lens, B)};
    REQUIRE(!any_overlap(outs, 4, ins, 6), GDN_EINVAL, "%s: an output overlaps another buffer", fn);
    const gdn::AcceptArgs a{target, tokens, parent, count, root, node, next, history, lens, lens_out, B, K, capacity};
    return launch_status(gdn::launch_accept(a, (hipStream_t)stream), fn);
}

}  // extern "C"
