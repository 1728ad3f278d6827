// C ABI of the packed-int4 GEMM library: host-side validation, then launches.
// Nothing is launched and nothing is written unless every check passes.
#include "qgemm.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <set>
#include <string>

#include "qg_kv4.h"
#include "qg_launch.h"

namespace {

thread_local char g_err[512] = "";

int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return status;
}

int ok()
{
    g_err[0] = '\0';
    return QG_OK;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// gfx950 check of the current device; cached per device id.
int check_device()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return fail(QG_ERR_DEVICE, "no HIP device is current");
    if (!qg_device_supported(dev))
        return fail(QG_ERR_DEVICE, "device %d is not a gfx950 GPU", dev);
    return QG_OK;
}

// QG_DEBUG_SYNC: the library built with it set (libqgemm_debugsync.so, for
// race checks) also waits for each call's kernels and reports a failed kernel
// as that call's error; it must not be used under stream capture.
#ifndef QG_DEBUG_SYNC
#define QG_DEBUG_SYNC 0
#endif

int launch_status(hipError_t e, const char *what, hipStream_t st)
{
    if (e != hipSuccess)
        return fail(QG_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
    if (QG_DEBUG_SYNC) {
        e = hipStreamSynchronize(st);
        if (e != hipSuccess)
            return fail(QG_ERR_LAUNCH, "%s: kernel failed: %s", what, hipGetErrorString(e));
    }
    return ok();
}

// With QGEMM_LOG set (and not "0"): one stderr line for the first successful
// launch of each distinct call description, as the pages' integration logs its
// first dispatch ("Marlin INT4 on Ada - how it works", "End-to-end result on
// RTX 4090").
bool log_enabled()
{
    static const bool on = [] {
        const char *e = getenv("QGEMM_LOG");
        return e && *e && strcmp(e, "0") != 0;
    }();
    return on;
}

void log_first(const char *fmt, ...)
{
    if (!log_enabled()) return;
    char line[320];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(line, sizeof(line), fmt, ap);
    va_end(ap);
    static std::mutex mu;
    static std::set<std::string> seen;
    std::lock_guard<std::mutex> lk(mu);
    if (seen.insert(line).second) fprintf(stderr, "[qgemm] first dispatch ok: %s\n", line);
}

// The kernels address a tile's activation rows and a scale row with 32-bit
// byte offsets: K < 2^22 and ceil(K/g) * N * 2 < 2^31 keep every one in
// range (far beyond any layer; larger shapes are refused, not miscomputed).
int check_offsets(const char *what, int N, int K, int g)
{
    const long long groups = (K + (long long)g - 1) / g;
    if (K >= (1 << 22) || groups * N * 2 >= (1ll << 31))
        return fail(QG_ERR_UNSUPPORTED, "%s: K=%d, N=%d too large for 32-bit offsets", what, K, N);
    return QG_OK;
}

// Shape rules shared by every GEMM-like entry point.  Normalises the per-column
// sentinel -1 to K.
int check_shape(const char *what, int M, int N, int K, int *g)
{
    if (M < 1 || N < 1 || K < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: M, N, K must be >= 1 (got %d, %d, %d)", what, M, N, K);
    if (K % 128 != 0 || N % 128 != 0)
        return fail(QG_ERR_UNSUPPORTED, "%s: K and N must be multiples of 128 (got K=%d N=%d)",
                    what, K, N);
    if (*g == -1) *g = K;
    if (*g < 1 || K % *g != 0)
        return fail(QG_ERR_INVALID_ARG, "%s: group_size %d does not divide K=%d", what, *g, K);
    if (*g != K && *g % 128 != 0 && *g != 64 && *g != 32)
        return fail(QG_ERR_UNSUPPORTED,
                    "%s: group_size %d unsupported (must be 32, 64, a multiple of 128, K, or -1)",
                    what, *g);
    if ((long long)M * K > (1ll << 40) || (long long)K * N > (1ll << 40))
        return fail(QG_ERR_UNSUPPORTED, "%s: shape too large", what);
    return check_offsets(what, N, K, *g);
}

// Shape rules of the entry points that take tails (pack_int4_weights,
// qgemm_w4a16): K and N any positive size; group_size 32, 64, a multiple of
// 128 (the last group may be partial), K, or -1 (normalised to K).
int check_shape_tail(const char *what, int M, int N, int K, int *g)
{
    if (M < 1 || N < 1 || K < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: M, N, K must be >= 1 (got %d, %d, %d)", what, M, N, K);
    if (*g == -1) *g = K;
    if (*g < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: group_size %d", what, *g);
    if (*g != K && *g % 128 != 0 && *g != 64 && *g != 32) {
        if (K % *g != 0)
            return fail(QG_ERR_INVALID_ARG, "%s: group_size %d does not divide K=%d", what, *g, K);
        return fail(QG_ERR_UNSUPPORTED,
                    "%s: group_size %d unsupported (must be 32, 64, a multiple of 128, K, or -1)",
                    what, *g);
    }
    if (K > (1 << 28) || N > (1 << 28) || (long long)M * K > (1ll << 40) ||
        (long long)K * N > (1ll << 40))
        return fail(QG_ERR_UNSUPPORTED, "%s: shape too large", what);
    return check_offsets(what, N, K, *g);
}

size_t corr_ws_bytes(int M, int K, int g) { return (size_t)M * (size_t)(K / g) * sizeof(float); }

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// W4A16 workspace: [counters][decode partial sums][correction a_sum when
// separate].  The counter region is always first, whatever the call, so a
// workspace shared by different shapes never has group sums or partials
// written over a counter.
size_t w4a16_gemm_ws_bytes(int M, int N, int K, int g, bool separate)
{
    const size_t gemm = qg::w4a16_workspace_bytes(M, N, K, g);
    if (gemm) return gemm;
    return separate ? qg::W4A16_WS_COUNTER_BYTES : 0;
}

size_t w4a16_ws_bytes(int M, int N, int K, int g, bool separate)
{
    const size_t gemm = w4a16_gemm_ws_bytes(M, N, K, g, separate);
    if (!separate) return gemm;
    return align256(gemm) + corr_ws_bytes(M, K, g);
}

// Host checks of a W4A16 call shared by qgemm_w4a16 and qgemm_w4a16_noalloc:
// shape, pointers, alignment and flags; fills the group size, the path and
// the scratch bytes the call needs.
struct W4A16Call {
    int g;
    bool separate, tail;
    size_t need;
};

int w4a16_check(const char *what, const uint16_t *A, const uint32_t *w_packed,
                const uint16_t *scale, const uint16_t *delta, const uint16_t *C, int M, int N,
                int K, int group_size, unsigned flags, W4A16Call *call)
{
    int g = group_size;
    int rc = check_shape_tail(what, M, N, K, &g);
    if (rc) return rc;
    if (!A || !w_packed || !scale || !C)
        return fail(QG_ERR_INVALID_ARG, "%s: NULL A/w_packed/scale/C", what);
    if (!aligned(A, 16) || !aligned(w_packed, 16) || !aligned(scale, 2) || !aligned(C, 2) ||
        (delta && !aligned(delta, 2)))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    if (flags & ~QG_CORR_SEPARATE)
        return fail(QG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
    call->g = g;
    call->separate = (flags & QG_CORR_SEPARATE) && delta;
    call->tail = qg::is_tail_shape(N, K, g);
    if (call->tail && call->separate)
        return fail(QG_ERR_UNSUPPORTED, "%s: QG_CORR_SEPARATE needs K, N multiples of 128", what);
    call->need = call->tail ? qg::tail_workspace_bytes(M, N, K, g)
                            : w4a16_ws_bytes(M, N, K, g, call->separate);
    return QG_OK;
}

// The launches of a checked W4A16 call; `workspace` holds call.need bytes.
int w4a16_launch(const char *what, const W4A16Call &call, const uint16_t *A,
                 const uint32_t *w_packed, const uint16_t *scale, const uint16_t *delta,
                 uint16_t *C, int M, int N, int K, void *workspace, hipStream_t st)
{
    const int g = call.g;
    int rc;
    if (call.tail) {
        rc = launch_status(qg::launch_w4a16_tail(A, w_packed, scale, delta, C, M, N, K, g, true,
                                                 workspace, st),
                           what, st);
    } else {
        const size_t gemm_ws = w4a16_gemm_ws_bytes(M, N, K, g, call.separate);
        hipError_t e = qg::launch_w4a16(A, w_packed, scale, delta, C, M, N, K, g, !call.separate,
                                        qg::w4a16_workspace_bytes(M, N, K, g) ? workspace : nullptr, st);
        if (e == hipSuccess && call.separate)
            e = qg::launch_group_sum_correction(A, delta, C, M, N, K, g,
                                                (float *)((char *)workspace + align256(gemm_ws)), st);
        rc = launch_status(e, what, st);
    }
    if (rc == QG_OK && log_enabled()) {
        int Kp = K, Np = N, gp = g;
        if (call.tail) qg::padded_shape(K, N, g, &Kp, &Np, &gp);
        char kern[160];
        qg::describe_w4a16(M, Np, Kp, gp, delta && !call.separate, false, kern, sizeof(kern));
        log_first("%s M=%d N=%d K=%d gs=%d %s: %s%s%s", what, M, N, K, g,
                  delta ? (call.separate ? "asymmetric (separate correction)" : "asymmetric")
                        : "symmetric",
                  call.tail ? "padded shape, " : "", kern,
                  call.separate ? " + group sums + correction" : "");
    }
    return rc;
}

// Shape rules of the fp8 GEMM: rows of whole 16-byte chunks, and the kernels'
// 32-bit offsets within a tile's rows and within one expert's scales.
int check_fp8_shape(const char *what, int M, int N, int K)
{
    if (M < 0 || N < 1 || K < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: M >= 0, N >= 1, K >= 1 needed (got %d, %d, %d)", what, M, N, K);
    if (K % 16 != 0)
        return fail(QG_ERR_UNSUPPORTED, "%s: K must be a multiple of 16 (got %d)", what, K);
    const long long KB = (K + 127ll) / 128, NB = (N + 127ll) / 128;
    if (K >= (1 << 22) || KB * NB >= (1ll << 29) || (long long)M + N > 0x7FFFFF00ll ||
        (long long)M * K > (1ll << 46))
        return fail(QG_ERR_UNSUPPORTED, "%s: M=%d, N=%d, K=%d too large", what, M, N, K);
    return QG_OK;
}

// Threads of one launch's grid along x: a 32-bit count.
constexpr long long MAX_GRID_THREADS = 0xFFFFFFFFll;

int check_dtype16(const char *what, int dtype)
{
    if (dtype != QG_DTYPE_F16 && dtype != QG_DTYPE_BF16)
        return fail(QG_ERR_INVALID_ARG, "%s: dtype %d is neither QG_DTYPE_F16 nor QG_DTYPE_BF16", what, dtype);
    return QG_OK;
}

int check_sort_shape(const char *what, int T, int topk, int E)
{
    if (T < 0 || topk < 1 || E < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: T >= 0, topk >= 1, E >= 1 needed (got %d, %d, %d)", what, T, topk, E);
    if (E > 1024 || (long long)T * topk >= (1ll << 30))
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, topk=%d, E=%d too large", what, T, topk, E);
    return QG_OK;
}

// Cache and batch of the kv4 calls; *c and *s as the kernels take them.
int check_kv4(const char *what, const void *k, const void *v, const void *k_sz, const void *v_sz, int pages, int heads,
              int page_size, int D, int g, const int32_t *off, const int32_t *lens, const int32_t *table, int B,
              int max_pages, int T, qg::Kv4Cache *c, qg::Kv4Batch *s)
{
    if (pages < 1 || heads < 1 || max_pages < 1 || B < 0 || T < 0)
        return fail(QG_ERR_INVALID_ARG, "%s: num_pages=%d, heads=%d, max_pages=%d, B=%d, T=%d", what, pages, heads,
                    max_pages, B, T);
    if (D != 64 && D != 128 && D != 256)
        return fail(QG_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256 (got %d)", what, D);
    if ((g != 32 && g != 64 && g != 128) || g > D)
        return fail(QG_ERR_UNSUPPORTED, "%s: group must be 32, 64 or 128 and at most head_dim=%d (got %d)", what, D, g);
    if (page_size < 32 || page_size > 1024 || (page_size & (page_size - 1)))
        return fail(QG_ERR_UNSUPPORTED, "%s: page_size must be a power of two from 32 to 1024 (got %d)", what, page_size);
    if (heads > 4096 || (long long)max_pages * page_size > (1ll << 30) || T >= (1 << 28) || B >= (1 << 28) ||
        (long long)pages * heads > 0x7FFFFFFFll)
        return fail(QG_ERR_UNSUPPORTED, "%s: heads=%d, max_pages=%d, num_pages=%d, T=%d, B=%d too large", what, heads,
                    max_pages, pages, T, B);
    if (!off && T != B)
        return fail(QG_ERR_INVALID_ARG, "%s: T=%d rows of B=%d sequences need seq_offsets", what, T, B);
    if (T > 0 && B > 0) {
        if (!k || !v || !k_sz || !v_sz) return fail(QG_ERR_INVALID_ARG, "%s: NULL cache", what);
        if (!lens || !table) return fail(QG_ERR_INVALID_ARG, "%s: NULL kv_lens/page_table", what);
        if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_sz, 16) || !aligned(v_sz, 16) || !aligned(lens, 4) ||
            !aligned(table, 4) || (off && !aligned(off, 4)))
            return fail(QG_ERR_INVALID_ARG, "%s: misaligned cache, lengths, offsets or page table", what);
    }
    *c = qg::Kv4Cache{(uint32_t *)k, (uint32_t *)v, (uint32_t *)k_sz, (uint32_t *)v_sz, pages, heads,
                      __builtin_ctz((unsigned)page_size), D, g};
    *s = qg::Kv4Batch{off, lens, table, B, max_pages, T};
    return QG_OK;
}

// Rows of `heads` heads of D channels, ld elements apart.
int check_kv4_rows(const char *what, const char *name, const void *p, int ld, int heads, int D)
{
    if (!p) return fail(QG_ERR_INVALID_ARG, "%s: NULL %s", what, name);
    if (!aligned(p, 16)) return fail(QG_ERR_INVALID_ARG, "%s: misaligned %s", what, name);
    if (ld % 8 || ld < (long long)heads * D)
        return fail(QG_ERR_INVALID_ARG, "%s: rows of %s %d elements apart (a multiple of 8, at least %lld)", what, name,
                    ld, (long long)heads * D);
    return QG_OK;
}

int check_attend_shape(const char *what, int T, int max_new, int B, int q_heads, int heads, int window, int sinks)
{
    if (max_new < 1 || window < 0 || sinks < 0)
        return fail(QG_ERR_INVALID_ARG, "%s: max_new=%d, window=%d, sinks=%d", what, max_new, window, sinks);
    if (heads < 1 || q_heads < 1 || q_heads % heads)
        return fail(QG_ERR_INVALID_ARG, "%s: %d query heads over %d key/value heads", what, q_heads, heads);
    if ((long long)T * q_heads >= (1ll << 30) || (long long)B * q_heads >= (1ll << 30))
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, B=%d, q_heads=%d too large", what, T, B, q_heads);
    return QG_OK;
}

// Window and sinks past every token are none and all.
int capped(int n) { return n < (1 << 30) ? n : 1 << 30; }

int check_lora_shape(const char *what, int T, int L, int K, int N, int R)
{
    if (T < 0 || L < 1 || K < 1 || N < 1 || R < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: T >= 0, L, K, N, R >= 1 needed (got %d, %d, %d, %d, %d)", what, T, L, K, N, R);
    if (K % 8 || N % 8 || R % 8)
        return fail(QG_ERR_UNSUPPORTED, "%s: K, N, R must be multiples of 8 (got %d, %d, %d)", what, K, N, R);
    if (L > 65535 || R > 512 || K > (1 << 24) || N > (1 << 24) || T >= (1 << 24))
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, L=%d, K=%d, N=%d, R=%d too large", what, T, L, K, N, R);
    return QG_OK;
}

} // namespace

extern "C" {

int qg_padded_shape(int K, int N, int group_size, int *K_padded, int *N_padded, int *groups)
{
    int g = group_size;
    int rc = check_shape_tail("qg_padded_shape", 1, N, K, &g);
    if (rc) return rc;
    int Kp, Np, gp;
    qg::padded_shape(K, N, g, &Kp, &Np, &gp);
    if (K_padded) *K_padded = Kp;
    if (N_padded) *N_padded = Np;
    if (groups) *groups = Kp / gp;
    return ok();
}

int qg_device_supported(int device)
{
    int n = 0;
    if (hipGetDeviceCount(&n) != hipSuccess || device < 0 || device >= n) return 0;
    static std::mutex mu;
    static int cache[64];
    static bool cached[64];
    if (device < 64) {
        std::lock_guard<std::mutex> lk(mu);
        if (cached[device]) return cache[device];
    }
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, device) != hipSuccess) return 0;
    int yes = strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : 0;
    if (device < 64) {
        std::lock_guard<std::mutex> lk(mu);
        cache[device] = yes;
        cached[device] = true;
    }
    return yes;
}

const char *qg_status_string(int status)
{
    switch (status) {
    case QG_OK: return "ok";
    case QG_ERR_INVALID_ARG: return "invalid argument";
    case QG_ERR_UNSUPPORTED: return "unsupported shape or group size";
    case QG_ERR_WORKSPACE: return "workspace missing or too small";
    case QG_ERR_DEVICE: return "no supported (gfx950) device";
    case QG_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
    }
}

const char *qg_last_error(void) { return g_err; }

size_t qg_workspace_bytes(int op, int M, int N, int K, int group_size, int num_experts,
                          unsigned flags)
{
    int g = group_size;
    switch (op) {
    case QG_OP_W4A16:
        if (check_shape_tail("qg_workspace_bytes", M, N, K, &g) != QG_OK) return (size_t)-1;
        if (qg::is_tail_shape(N, K, g)) {
            if (flags & QG_CORR_SEPARATE) {
                fail(QG_ERR_UNSUPPORTED, "qg_workspace_bytes: QG_CORR_SEPARATE needs K, N multiples of 128");
                return (size_t)-1;
            }
            return qg::tail_workspace_bytes(M, N, K, g);
        }
        return w4a16_ws_bytes(M, N, K, g, (flags & QG_CORR_SEPARATE) != 0);
    case QG_OP_W4A16_SWIGLU:
        if (check_shape("qg_workspace_bytes", M, N, K, &g) != QG_OK) return (size_t)-1;
        if (N > 0x3FFFFFFF) return (size_t)-1;
        return qg::swiglu_workspace_bytes(M, N, K, g);
    case QG_OP_GROUP_SUM_CORRECTION:
        if (check_shape("qg_workspace_bytes", M, N, K, &g) != QG_OK) return (size_t)-1;
        return corr_ws_bytes(M, K, g);
    case QG_OP_W4A8:
        if (check_shape_tail("qg_workspace_bytes", M < 1 ? 1 : M, N, K, &g) != QG_OK) return (size_t)-1;
        return qg::is_tail_shape(N, K, g) ? qg::w4a8_tail_workspace_bytes(M < 1 ? 1 : M, N, K, g) : 0;
    case QG_OP_FP8:
        if (check_fp8_shape("qg_workspace_bytes", M, N, K) != QG_OK) return (size_t)-1;
        return 0;
    case QG_OP_MOE_SORT:
        if (check_sort_shape("qg_workspace_bytes", M, N, num_experts) != QG_OK) return (size_t)-1;
        return qg::moe_sort_workspace_bytes(M, N, num_experts);
    case QG_OP_LORA:
        if (check_lora_shape("qg_workspace_bytes", M, num_experts, K, N, group_size) != QG_OK) return (size_t)-1;
        return M == 0 ? 0 : qg::lora_plan(M, num_experts, K, N, group_size).bytes;
    case QG_OP_PACK:
        if (check_shape("qg_workspace_bytes", M < 1 ? 1 : M, N, K, &g) != QG_OK) return (size_t)-1;
        return 0;
    default:
        fail(QG_ERR_INVALID_ARG, "qg_workspace_bytes: unknown op %d", op);
        return (size_t)-1;
    }
}

int pack_int4_weights(const uint8_t *q, const uint16_t *scale, const uint16_t *zero, int K,
                      int N, int group_size, unsigned flags, uint32_t *w_packed,
                      uint16_t *scale_out, uint16_t *delta_out, void *stream)
{
    int g = group_size;
    int rc = check_shape_tail("pack_int4_weights", 1, N, K, &g);
    if (rc) return rc;
    if (!q || !scale || !w_packed || !scale_out)
        return fail(QG_ERR_INVALID_ARG, "pack_int4_weights: NULL q/scale/w_packed/scale_out");
    if (zero && !delta_out)
        return fail(QG_ERR_INVALID_ARG, "pack_int4_weights: delta_out is required with zero");
    if (!aligned(w_packed, 16) || !aligned(scale, 2) || !aligned(scale_out, 2) ||
        (zero && !aligned(zero, 2)) || (delta_out && !aligned(delta_out, 2)))
        return fail(QG_ERR_INVALID_ARG, "pack_int4_weights: misaligned pointer");
    if (flags & ~QG_PACK_FOLD_NEG_SCALES)
        return fail(QG_ERR_INVALID_ARG, "pack_int4_weights: unknown flags 0x%x", flags);
    if ((const void *)scale_out == (const void *)scale) {
        int Kp, Np, gp;
        qg::padded_shape(K, N, g, &Kp, &Np, &gp);
        if (Np != N || Kp / gp != (K + g - 1) / g)
            return fail(QG_ERR_INVALID_ARG,
                        "pack_int4_weights: scale_out may alias scale only when the padded "
                        "shape adds no columns and no groups");
    }
    if ((rc = check_device())) return rc;
    hipError_t e = qg::launch_pack(q, scale, zero, K, N, g, (flags & QG_PACK_FOLD_NEG_SCALES) != 0,
                                   w_packed, scale_out, zero ? delta_out : nullptr,
                                   (hipStream_t)stream);
    rc = launch_status(e, "pack_int4_weights", (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("pack_int4_weights K=%d N=%d gs=%d %s%s", K, N, g, zero ? "asymmetric" : "symmetric",
                  (flags & QG_PACK_FOLD_NEG_SCALES) ? ", negative scales folded" : "");
    return rc;
}

int qgemm_w4a16(const uint16_t *A, const uint32_t *w_packed, const uint16_t *scale,
                const uint16_t *delta, uint16_t *C, int M, int N, int K, int group_size,
                unsigned flags, void *workspace, size_t workspace_bytes, void *stream)
{
    W4A16Call call;
    int rc = w4a16_check("qgemm_w4a16", A, w_packed, scale, delta, C, M, N, K, group_size, flags,
                         &call);
    if (rc) return rc;
    if (call.need > 0) {
        if (!workspace || workspace_bytes < call.need)
            return fail(QG_ERR_WORKSPACE, "qgemm_w4a16: workspace of %zu bytes needed, got %zu",
                        call.need, workspace ? workspace_bytes : (size_t)0);
        if (!aligned(workspace, 256))
            return fail(QG_ERR_INVALID_ARG, "qgemm_w4a16: workspace must be 256-byte aligned");
    }
    if ((rc = check_device())) return rc;
    return w4a16_launch("qgemm_w4a16", call, A, w_packed, scale, delta, C, M, N, K, workspace,
                        (hipStream_t)stream);
}

int qgemm_w4a16_noalloc(const uint16_t *A, const uint32_t *w_packed, const uint16_t *scale,
                        const uint16_t *delta, uint16_t *C, int M, int N, int K, int group_size,
                        unsigned flags, void *stream)
{
    W4A16Call call;
    int rc = w4a16_check("qgemm_w4a16_noalloc", A, w_packed, scale, delta, C, M, N, K, group_size,
                         flags, &call);
    if (rc) return rc;
    if (call.need > QG_NOALLOC_SCRATCH_BYTES)
        return fail(QG_ERR_WORKSPACE,
                    "qgemm_w4a16_noalloc: this call needs %zu bytes of scratch, more than the "
                    "library's static scratch of %zu bytes (use qgemm_w4a16 with a workspace)",
                    call.need, (size_t)QG_NOALLOC_SCRATCH_BYTES);
    if ((rc = check_device())) return rc;
    void *ws = nullptr;
    if (call.need > 0) {
        hipError_t e = qg::noalloc_scratch((hipStream_t)stream, &ws);
        if (e != hipSuccess)
            return fail(QG_ERR_LAUNCH, "qgemm_w4a16_noalloc: static scratch unavailable: %s",
                        hipGetErrorString(e));
    }
    return w4a16_launch("qgemm_w4a16_noalloc", call, A, w_packed, scale, delta, C, M, N, K, ws,
                        (hipStream_t)stream);
}

int qgemm_w4a16_swiglu(const uint16_t *A, const uint32_t *w_packed, const uint16_t *scale,
                       const uint16_t *delta, uint16_t *H, int M, int N, int K, int group_size,
                       unsigned flags, void *workspace, size_t workspace_bytes, void *stream)
{
    int g = group_size;
    int rc = check_shape("qgemm_w4a16_swiglu", M, N, K, &g);
    if (rc) return rc;
    if (N > 0x3FFFFFFF || (size_t)K * 2 * (size_t)N / 8 > 0x7FFFFFFFull * 16)
        return fail(QG_ERR_UNSUPPORTED, "qgemm_w4a16_swiglu: shape too large");
    if ((rc = check_offsets("qgemm_w4a16_swiglu", 2 * N, K, g))) return rc;   // the pair's width
    if (!A || !w_packed || !scale || !H)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a16_swiglu: NULL A/w_packed/scale/H");
    if (!aligned(A, 16) || !aligned(w_packed, 16) || !aligned(scale, 2) || !aligned(H, 16) ||
        (delta && !aligned(delta, 2)))
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a16_swiglu: misaligned pointer");
    if (flags != 0)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a16_swiglu: unknown flags 0x%x", flags);
    const size_t need = qg::swiglu_workspace_bytes(M, N, K, g);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(QG_ERR_WORKSPACE, "qgemm_w4a16_swiglu: workspace of %zu bytes needed, got %zu",
                        need, workspace ? workspace_bytes : (size_t)0);
        if (!aligned(workspace, 256))
            return fail(QG_ERR_INVALID_ARG, "qgemm_w4a16_swiglu: workspace must be 256-byte aligned");
    }
    if ((rc = check_device())) return rc;
    hipError_t e = qg::launch_w4a16_swiglu(A, w_packed, scale, delta, H, M, N, K, g,
                                           need ? workspace : nullptr, (hipStream_t)stream);
    rc = launch_status(e, "qgemm_w4a16_swiglu", (hipStream_t)stream);
    if (rc == QG_OK && log_enabled()) {
        char kern[160];
        qg::describe_w4a16(M, N, K, g, delta != nullptr, true, kern, sizeof(kern));
        log_first("qgemm_w4a16_swiglu M=%d N=%d (pair %d) K=%d gs=%d %s: %s", M, N, 2 * N, K, g,
                  delta ? "asymmetric" : "symmetric", kern);
    }
    return rc;
}

int group_sum_correction(const uint16_t *A, const uint16_t *delta, uint16_t *C, int M, int N,
                         int K, int group_size, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    int g = group_size;
    int rc = check_shape("group_sum_correction", M, N, K, &g);
    if (rc) return rc;
    if (!A || !delta || !C)
        return fail(QG_ERR_INVALID_ARG, "group_sum_correction: NULL A/delta/C");
    if (!aligned(A, 2) || !aligned(delta, 2) || !aligned(C, 2))
        return fail(QG_ERR_INVALID_ARG, "group_sum_correction: misaligned pointer");
    size_t need = corr_ws_bytes(M, K, g);
    if (!workspace || workspace_bytes < need)
        return fail(QG_ERR_WORKSPACE, "group_sum_correction: workspace of %zu bytes needed, got %zu",
                    need, workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, 4))
        return fail(QG_ERR_INVALID_ARG, "group_sum_correction: misaligned workspace");
    if ((rc = check_device())) return rc;
    hipError_t e = qg::launch_group_sum_correction(A, delta, C, M, N, K, g, (float *)workspace,
                                                   (hipStream_t)stream);
    rc = launch_status(e, "group_sum_correction", (hipStream_t)stream);
    if (rc == QG_OK) log_first("group_sum_correction M=%d N=%d K=%d gs=%d", M, N, K, g);
    return rc;
}

int qgemm_w4a8(const int8_t *A_q, const float *a_scale, const uint32_t *w_packed,
               const uint16_t *w_scale, const uint16_t *w_delta,
               const int32_t *expert_offsets, int num_experts,
               int M_total, int max_rows_per_expert, int N, int K, int group_size, uint16_t *C,
               int32_t *acc_debug, void *workspace, size_t workspace_bytes, unsigned flags,
               void *stream)
{
    int g = group_size;
    int rc = check_shape_tail("qgemm_w4a8", M_total, N, K, &g);
    if (rc) return rc;
    const bool tail = qg::is_tail_shape(N, K, g);
    if (!A_q || !a_scale || !w_packed || !w_scale || !C)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: NULL A_q/a_scale/w_packed/w_scale/C");
    if (num_experts < 1 || num_experts > 65535)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: num_experts %d out of range", num_experts);
    if (!expert_offsets && num_experts != 1)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: expert_offsets is required when E > 1");
    if (max_rows_per_expert < 1)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: max_rows_per_expert must be >= 1");
    if (!expert_offsets && max_rows_per_expert < M_total)
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: max_rows_per_expert < M_total with one expert");
    if (K > 131072)
        return fail(QG_ERR_UNSUPPORTED, "qgemm_w4a8: K > 131072 would overflow int32 accumulators");
    if (!aligned(A_q, 8) || !aligned(a_scale, 4) || !aligned(w_packed, 16) ||
        !aligned(w_scale, 2) || (w_delta && !aligned(w_delta, 2)) || !aligned(C, 2) ||
        (acc_debug && !aligned(acc_debug, 4)) ||
        (expert_offsets && !aligned(expert_offsets, 4)))
        return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: misaligned pointer");
    if (flags != 0) return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: unknown flags 0x%x", flags);
    if (tail) {
        if (acc_debug)
            return fail(QG_ERR_UNSUPPORTED, "qgemm_w4a8: acc_debug needs K, N multiples of 128");
        const size_t need = qg::w4a8_tail_workspace_bytes(M_total, N, K, g);
        if (!workspace || workspace_bytes < need)
            return fail(QG_ERR_WORKSPACE, "qgemm_w4a8: workspace of %zu bytes needed, got %zu", need,
                        workspace ? workspace_bytes : (size_t)0);
        if (!aligned(workspace, 256))
            return fail(QG_ERR_INVALID_ARG, "qgemm_w4a8: workspace must be 256-byte aligned");
    }
    if ((rc = check_device())) return rc;
    int max_rows = max_rows_per_expert > M_total ? M_total : max_rows_per_expert;
    const hipError_t e =
        tail ? qg::launch_w4a8_tail(A_q, a_scale, w_packed, w_scale, w_delta, expert_offsets,
                                    num_experts, M_total, max_rows, N, K, g, C, workspace,
                                    (hipStream_t)stream)
             : qg::launch_w4a8(A_q, a_scale, w_packed, w_scale, w_delta, expert_offsets, num_experts,
                               M_total, max_rows, N, K, g, C, acc_debug, (hipStream_t)stream);
    rc = launch_status(e, "qgemm_w4a8", (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("qgemm_w4a8 experts=%d M_total=%d max_rows=%d N=%d K=%d gs=%d %s%s%s", num_experts,
                  M_total, max_rows_per_expert, N, K, g, w_delta ? "zero-points" : "symmetric",
                  tail ? ", padded shape" : "", acc_debug ? ", acc_debug" : "");
    return rc;
}

int quantize_rows_int8(const uint16_t *A, int M, int K, int8_t *A_q, float *a_scale,
                       void *stream)
{
    if (!A || !A_q || !a_scale)
        return fail(QG_ERR_INVALID_ARG, "quantize_rows_int8: NULL A/A_q/a_scale");
    if (M < 1 || K < 1)
        return fail(QG_ERR_INVALID_ARG, "quantize_rows_int8: M and K must be >= 1 (got %d, %d)", M, K);
    if (K % 8)
        return fail(QG_ERR_UNSUPPORTED, "quantize_rows_int8: K must be a multiple of 8 (got %d)", K);
    if (!aligned(A, 16) || !aligned(A_q, 8) || !aligned(a_scale, 4))
        return fail(QG_ERR_INVALID_ARG, "quantize_rows_int8: misaligned pointer");
    int rc = check_device();
    if (rc) return rc;
    hipError_t e = qg::launch_quantize_rows_int8(A, M, K, A_q, a_scale, (hipStream_t)stream);
    rc = launch_status(e, "quantize_rows_int8", (hipStream_t)stream);
    if (rc == QG_OK) log_first("quantize_rows_int8 M=%d K=%d", M, K);
    return rc;
}

int quantize_rows_fp8(const void *A, int dtype, int M, int K, unsigned flags, uint8_t *A_q,
                      float *a_scale, void *stream)
{
    const char *const what = "quantize_rows_fp8";
    int rc = check_dtype16(what, dtype);
    if (rc) return rc;
    if (M < 0 || K < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: M >= 0 and K >= 1 needed (got %d, %d)", what, M, K);
    if (K % 16) return fail(QG_ERR_UNSUPPORTED, "%s: K must be a multiple of 16 (got %d)", what, K);
    if (M * ((K + 127ll) / 128) * 16 > MAX_GRID_THREADS - 256)
        return fail(QG_ERR_UNSUPPORTED, "%s: M=%d, K=%d too large", what, M, K);
    if (flags & ~QG_QUANT_SWIGLU) return fail(QG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
    if (M == 0) return ok();
    if (!A || !A_q || !a_scale) return fail(QG_ERR_INVALID_ARG, "%s: NULL A/A_q/a_scale", what);
    if (!aligned(A, 16) || !aligned(A_q, 16) || !aligned(a_scale, 4))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    if ((rc = check_device())) return rc;
    const bool swiglu = (flags & QG_QUANT_SWIGLU) != 0;
    rc = launch_status(qg::launch_quantize_rows_fp8(A, dtype, M, K, swiglu, A_q, a_scale, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("%s M=%d K=%d %s%s", what, M, K, dtype == QG_DTYPE_BF16 ? "bf16" : "fp16",
                  swiglu ? ", SwiGLU pair" : "");
    return rc;
}

int qgemm_fp8(const uint8_t *A_q, const float *a_scale, const int32_t *a_rows, int M_a,
              const uint8_t *W, const float *w_scale, const int32_t *expert_offsets,
              int num_experts, int M_total, int N, int K, int dtype, void *C, void *workspace,
              size_t workspace_bytes, unsigned flags, void *stream)
{
    const char *const what = "qgemm_fp8";
    (void)workspace;
    (void)workspace_bytes;
    int rc = check_fp8_shape(what, M_total, N, K);
    if (rc) return rc;
    if ((rc = check_dtype16(what, dtype))) return rc;
    if (num_experts < 1 || num_experts > 65535)
        return fail(QG_ERR_INVALID_ARG, "%s: num_experts %d out of range", what, num_experts);
    if (!expert_offsets && num_experts != 1)
        return fail(QG_ERR_INVALID_ARG, "%s: expert_offsets is required when E > 1", what);
    if (flags != 0) return fail(QG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
    if (M_total == 0) return ok();
    if (M_a < 0 || (!a_rows && M_a != M_total))
        return fail(QG_ERR_INVALID_ARG, "%s: M_a %d with M_total %d and %s a_rows", what, M_a, M_total,
                    a_rows ? "an" : "no");
    if (M_a == 0) return fail(QG_ERR_INVALID_ARG, "%s: a_rows needs at least one row of A", what);
    if (!A_q || !a_scale || !W || !w_scale || !C)
        return fail(QG_ERR_INVALID_ARG, "%s: NULL A_q/a_scale/W/w_scale/C", what);
    if (!aligned(A_q, 16) || !aligned(a_scale, 4) || !aligned(W, 16) || !aligned(w_scale, 4) ||
        !aligned(C, 2) || (a_rows && !aligned(a_rows, 4)) || (expert_offsets && !aligned(expert_offsets, 4)))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    if (a_rows && (long long)M_a * K > (1ll << 32) - (1ll << 23))
        return fail(QG_ERR_UNSUPPORTED, "%s: a_rows with M_a * K = %lld bytes of codes (32-bit offsets)", what,
                    (long long)M_a * K);
    if (qg::fp8_threads(expert_offsets != nullptr, num_experts, M_total, N, K) > MAX_GRID_THREADS)
        return fail(QG_ERR_UNSUPPORTED, "%s: M_total=%d, N=%d, E=%d too large for one launch", what, M_total, N,
                    num_experts);
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_fp8(A_q, a_scale, a_rows, M_a, W, w_scale, expert_offsets, num_experts,
                                      M_total, N, K, dtype, C, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK && log_enabled()) {
        char kern[160];
        qg::describe_fp8(expert_offsets != nullptr, num_experts, M_total, N, K, kern, sizeof(kern));
        log_first("%s experts=%d M_total=%d N=%d K=%d %s%s: %s", what, num_experts, M_total, N, K,
                  dtype == QG_DTYPE_BF16 ? "bf16" : "fp16", a_rows ? ", rows by index" : "", kern);
    }
    return rc;
}

int moe_route(const void *logits, int dtype, const float *bias, int T, int E, int topk,
              int n_group, int topk_group, float scaling, unsigned flags, int32_t *ids,
              float *weights, void *stream)
{
    const char *const what = "moe_route";
    if (dtype != QG_DTYPE_F32 && dtype != QG_DTYPE_F16 && dtype != QG_DTYPE_BF16)
        return fail(QG_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
    if (T < 0 || E < 1 || topk < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: T >= 0, E >= 1, topk >= 1 needed (got %d, %d, %d)", what, T, E, topk);
    if (E > 1024 || topk > 64 || n_group > 64)
        return fail(QG_ERR_UNSUPPORTED, "%s: E=%d, topk=%d, n_group=%d (at most 1024, 64, 64)", what, E, topk, n_group);
    if (T > MAX_GRID_THREADS / 64 - 4) return fail(QG_ERR_UNSUPPORTED, "%s: T=%d too large for one launch", what, T);
    if (n_group < 1 || E % n_group || topk_group < 1 || topk_group > n_group)
        return fail(QG_ERR_INVALID_ARG, "%s: %d of %d groups of E=%d experts", what, topk_group, n_group, E);
    if (topk > topk_group * (E / n_group))
        return fail(QG_ERR_INVALID_ARG, "%s: topk=%d of %d experts that can be chosen", what, topk,
                    topk_group * (E / n_group));
    if (flags & ~(QG_ROUTE_SIGMOID | QG_ROUTE_RENORMALIZE | QG_ROUTE_GROUP_TOP2))
        return fail(QG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
    if (T == 0) return ok();
    if (!logits || !ids || !weights) return fail(QG_ERR_INVALID_ARG, "%s: NULL logits/ids/weights", what);
    if (!aligned(logits, dtype == QG_DTYPE_F32 ? 4 : 2) || (bias && !aligned(bias, 4)) || !aligned(ids, 4) ||
        !aligned(weights, 4))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    int rc = check_device();
    if (rc) return rc;
    rc = launch_status(qg::launch_moe_route(logits, dtype, bias, T, E, topk, n_group, topk_group, scaling, flags,
                                            ids, weights, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("%s T=%d E=%d topk=%d groups=%d/%d %s%s", what, T, E, topk, topk_group, n_group,
                  (flags & QG_ROUTE_SIGMOID) ? "sigmoid" : "softmax", bias ? ", bias" : "");
    return rc;
}

int moe_sort_rows(const int32_t *ids, int T, int topk, int num_experts, int32_t *expert_offsets,
                  int32_t *row_token, int32_t *slot_row, void *workspace, size_t workspace_bytes,
                  void *stream)
{
    const char *const what = "moe_sort_rows";
    int rc = check_sort_shape(what, T, topk, num_experts);
    if (rc) return rc;
    if (!expert_offsets || (T > 0 && (!ids || !row_token || !slot_row)))
        return fail(QG_ERR_INVALID_ARG, "%s: NULL ids/expert_offsets/row_token/slot_row", what);
    if (!aligned(ids, 4) || !aligned(expert_offsets, 4) || !aligned(row_token, 4) || !aligned(slot_row, 4))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    const size_t need = qg::moe_sort_workspace_bytes(T, topk, num_experts);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(QG_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, got %zu", what, need,
                        workspace ? workspace_bytes : (size_t)0);
        if (!aligned(workspace, 256))
            return fail(QG_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", what);
    }
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_moe_sort(ids, T, topk, num_experts, expert_offsets, row_token, slot_row,
                                           need ? workspace : nullptr, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK) log_first("%s T=%d topk=%d E=%d", what, T, topk, num_experts);
    return rc;
}

int moe_combine_rows(const void *Y, int dtype, const int32_t *slot_row, const float *weights,
                     int T, int topk, int M_rows, int N, void *out, void *stream)
{
    const char *const what = "moe_combine_rows";
    int rc = check_dtype16(what, dtype);
    if (rc) return rc;
    if (T < 0 || topk < 1 || M_rows < 0 || N < 1)
        return fail(QG_ERR_INVALID_ARG, "%s: T=%d, topk=%d, M_rows=%d, N=%d", what, T, topk, M_rows, N);
    if (topk > 64 || (long long)T * topk >= (1ll << 30) || N > (1 << 28))
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, topk=%d, N=%d too large", what, T, topk, N);
    if (T == 0) return ok();
    if ((M_rows > 0 && !Y) || !slot_row || !weights || !out)
        return fail(QG_ERR_INVALID_ARG, "%s: NULL Y/slot_row/weights/out", what);
    if (!aligned(Y, 2) || !aligned(slot_row, 4) || !aligned(weights, 4) || !aligned(out, 2))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_moe_combine(Y, dtype, slot_row, weights, T, topk, M_rows, N, out,
                                              (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK) log_first("%s T=%d topk=%d N=%d", what, T, topk, N);
    return rc;
}

int kv4_append(const void *k, const void *v, const void *q, int dtype, int T, int ld_k, int ld_v, int ld_q, int q_heads,
               const int32_t *seq_offsets, const int32_t *kv_lens, const int32_t *page_table, int B, int max_pages,
               const int32_t *positions, const float *cos_sin, int rot_dim, int max_pos, unsigned flags,
               uint32_t *cache_k, uint32_t *cache_v, uint16_t *cache_k_sz, uint16_t *cache_v_sz, int num_pages,
               int heads, int page_size, int head_dim, int group, void *q_out, void *stream)
{
    const char *const what = "kv4_append";
    qg::Kv4Cache c;
    qg::Kv4Batch s;
    int rc = check_kv4(what, cache_k, cache_v, cache_k_sz, cache_v_sz, num_pages, heads, page_size, head_dim, group,
                       seq_offsets, kv_lens, page_table, B, max_pages, T, &c, &s);
    if (rc) return rc;
    if ((rc = check_dtype16(what, dtype))) return rc;
    if (flags & ~QG_KV4_INTERLEAVED) return fail(QG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
        return fail(QG_ERR_UNSUPPORTED, "%s: rot_dim must be a multiple of 16, at most head_dim=%d (got %d)", what,
                    head_dim, rot_dim);
    if (rot_dim > 0 && (!cos_sin || max_pos < 1 || !aligned(cos_sin, 16)))
        return fail(QG_ERR_INVALID_ARG, "%s: rot_dim=%d without angles (16-byte aligned, max_pos >= 1)", what, rot_dim);
    // (a grid has 65535 in y: four query heads each, behind the keys and values of 4096)
    if (q && (q_heads < 1 || q_heads > (1 << 17)))
        return fail(QG_ERR_INVALID_ARG, "%s: q_heads=%d out of range", what, q_heads);
    if (T == 0 || B == 0) return ok();
    if ((rc = check_kv4_rows(what, "k", k, ld_k, heads, head_dim))) return rc;
    if ((rc = check_kv4_rows(what, "v", v, ld_v, heads, head_dim))) return rc;
    if (q && (rc = check_kv4_rows(what, "q", q, ld_q, q_heads, head_dim))) return rc;
    if (q && (!q_out || !aligned(q_out, 16))) return fail(QG_ERR_INVALID_ARG, "%s: NULL or misaligned q_out", what);
    if (positions && !aligned(positions, 4)) return fail(QG_ERR_INVALID_ARG, "%s: misaligned positions", what);
    if (qg::kv4_blocks_bound(T, B) * 256 > MAX_GRID_THREADS)
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, B=%d too large for one launch", what, T, B);
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_kv4_append(c, s, k, v, q, ld_k, ld_v, ld_q, q_heads, dtype, positions, cos_sin, rot_dim,
                                             max_pos, (flags & QG_KV4_INTERLEAVED) != 0, q_out, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("%s T=%d B=%d heads=%d head_dim=%d group=%d page_size=%d rot_dim=%d%s %s%s", what, T, B, heads, head_dim,
                  group, page_size, rot_dim, (flags & QG_KV4_INTERLEAVED) ? " interleaved" : "",
                  dtype == QG_DTYPE_BF16 ? "bf16" : "fp16", q ? ", queries" : "");
    return rc;
}

int kv4_read(const uint32_t *cache_k, const uint32_t *cache_v, const uint16_t *cache_k_sz, const uint16_t *cache_v_sz,
             int num_pages, int heads, int page_size, int head_dim, int group, const int32_t *seq_offsets,
             const int32_t *kv_lens, const int32_t *page_table, int B, int max_pages, int T, int dtype, void *k_out,
             void *v_out, void *stream)
{
    const char *const what = "kv4_read";
    qg::Kv4Cache c;
    qg::Kv4Batch s;
    int rc = check_kv4(what, cache_k, cache_v, cache_k_sz, cache_v_sz, num_pages, heads, page_size, head_dim, group,
                       seq_offsets, kv_lens, page_table, B, max_pages, T, &c, &s);
    if (rc) return rc;
    if (dtype != QG_DTYPE_F32 && dtype != QG_DTYPE_F16 && dtype != QG_DTYPE_BF16)
        return fail(QG_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
    if (T == 0 || B == 0) return ok();
    if (!k_out || !v_out) return fail(QG_ERR_INVALID_ARG, "%s: NULL k_out/v_out", what);
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    if (qg::kv4_blocks_bound(T, B) * 256 > MAX_GRID_THREADS)
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, B=%d too large for one launch", what, T, B);
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_kv4_read(c, s, dtype, k_out, v_out, (hipStream_t)stream), what, (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("%s T=%d B=%d heads=%d head_dim=%d group=%d page_size=%d", what, T, B, heads, head_dim, group, page_size);
    return rc;
}

size_t kv4_attend_workspace_bytes(int T, int max_new, int B, int q_heads, int heads, int head_dim, int max_pages,
                                  int page_size, int window, int sinks)
{
    const char *const what = "kv4_attend_workspace_bytes";
    if (T < 0 || B < 0 || max_pages < 1 || page_size < 1 || head_dim < 1 ||
        (long long)max_pages * page_size > (1ll << 30)) {
        fail(QG_ERR_INVALID_ARG, "%s: T=%d, B=%d, head_dim=%d, max_pages=%d, page_size=%d", what, T, B, head_dim,
             max_pages, page_size);
        return (size_t)-1;
    }
    if (check_attend_shape(what, T, max_new, B, q_heads, heads, window, sinks) != QG_OK) return (size_t)-1;
    if (T == 0 || B == 0) return 0;
    return qg::kv4_attend_plan(T, max_new, B, q_heads, heads, head_dim, max_pages * page_size, capped(window),
                               capped(sinks)).bytes;
}

int kv4_attend(const void *q, int dtype, int T, int ld_q, int q_heads, int max_new, const int32_t *seq_offsets,
               const int32_t *kv_lens, const int32_t *page_table, int B, int max_pages, const uint32_t *cache_k,
               const uint32_t *cache_v, const uint16_t *cache_k_sz, const uint16_t *cache_v_sz, int num_pages, int heads,
               int page_size, int head_dim, int group, float scale, int window, int sinks, void *out, void *workspace,
               size_t workspace_bytes, unsigned flags, void *stream)
{
    const char *const what = "kv4_attend";
    qg::Kv4Cache c;
    qg::Kv4Batch s;
    int rc = check_kv4(what, cache_k, cache_v, cache_k_sz, cache_v_sz, num_pages, heads, page_size, head_dim, group,
                       seq_offsets, kv_lens, page_table, B, max_pages, T, &c, &s);
    if (rc) return rc;
    if ((rc = check_dtype16(what, dtype))) return rc;
    if ((rc = check_attend_shape(what, T, max_new, B, q_heads, heads, window, sinks))) return rc;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(QG_ERR_INVALID_ARG, "%s: scale must be finite and > 0", what);
    if (flags != 0) return fail(QG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
    if (T == 0 || B == 0) return ok();
    if ((rc = check_kv4_rows(what, "q", q, ld_q, q_heads, head_dim))) return rc;
    if (!out || !aligned(out, 16)) return fail(QG_ERR_INVALID_ARG, "%s: NULL or misaligned out", what);
    const qg::Kv4AttendPlan plan = qg::kv4_attend_plan(T, max_new, B, q_heads, heads, head_dim, max_pages * page_size,
                                                       capped(window), capped(sinks));
    if (plan.workgroups * (plan.shared == 8 ? 512 : 256) > MAX_GRID_THREADS)
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d, B=%d, q_heads=%d too large for one launch", what, T, B, q_heads);
    if (plan.bytes > 0) {
        if (!workspace || workspace_bytes < plan.bytes)
            return fail(QG_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, got %zu", what, plan.bytes,
                        workspace ? workspace_bytes : (size_t)0);
        if (!aligned(workspace, 256))
            return fail(QG_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", what);
    }
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_kv4_attend(plan, c, s, q, ld_q, q_heads, dtype, scale, capped(window), capped(sinks),
                                             out, plan.bytes ? workspace : nullptr, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("%s T=%d B=%d max_new=%d heads=%d/%d head_dim=%d group=%d page_size=%d window=%d sinks=%d %s: %d rows a "
                  "wave, %d parts", what, T, B, max_new, q_heads, heads, head_dim, group, page_size, window, sinks,
                  dtype == QG_DTYPE_BF16 ? "bf16" : "fp16", plan.rows, plan.splits);
    return rc;
}

int lora_add(const void *X, const void *A, const void *B, const float *scaling, const int32_t *adapter_offsets,
             const int32_t *row_token, const int32_t *slot_row, int L, int T, int K, int N, int R, int dtype, void *Y,
             void *workspace, size_t workspace_bytes, void *stream)
{
    const char *const what = "lora_add";
    int rc = check_dtype16(what, dtype);
    if (rc) return rc;
    if ((rc = check_lora_shape(what, T, L, K, N, R))) return rc;
    if (T == 0) return ok();
    if (!X || !A || !B || !Y || !adapter_offsets || !row_token || !slot_row)
        return fail(QG_ERR_INVALID_ARG, "%s: NULL X/A/B/Y/adapter_offsets/row_token/slot_row", what);
    if (!aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(Y, 16) || (scaling && !aligned(scaling, 4)) ||
        !aligned(adapter_offsets, 4) || !aligned(row_token, 4) || !aligned(slot_row, 4))
        return fail(QG_ERR_INVALID_ARG, "%s: misaligned pointer", what);
    const qg::LoraPlan plan = qg::lora_plan(T, L, K, N, R);
    if (plan.tiles * plan.ranges * 256 > MAX_GRID_THREADS || plan.narrow * 256 > MAX_GRID_THREADS ||
        (long long)T * ((R + 63) / 64) * 8 > MAX_GRID_THREADS - 256)
        return fail(QG_ERR_UNSUPPORTED, "%s: T=%d too large for one launch", what, T);
    if (!workspace || workspace_bytes < plan.bytes)
        return fail(QG_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, got %zu", what, plan.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, 256)) return fail(QG_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", what);
    if ((rc = check_device())) return rc;
    rc = launch_status(qg::launch_lora(plan, X, A, B, scaling, adapter_offsets, row_token, slot_row, L, T, K, N, R, dtype,
                                       Y, workspace, (hipStream_t)stream),
                       what, (hipStream_t)stream);
    if (rc == QG_OK)
        log_first("%s T=%d L=%d K=%d N=%d R=%d %s: narrow product in %d-row tiles and %d parts of K, wide one in %d-row tiles", what, T,
                  L, K, N, R, dtype == QG_DTYPE_BF16 ? "bf16" : "fp16", plan.narrow_rows, plan.splits, plan.tall ? 128 : 16);
    return rc;
}

} // extern "C"
