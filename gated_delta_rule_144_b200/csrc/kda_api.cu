// C ABI of libkda.so: argument validation, path selection and the device error word.
// Declarations and the contract of every entry point are in include/kda.h.

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "kda.h"

#include "kda_bwd.cuh"
#include "kda_internal.cuh"
#include "kda_linear.cuh"
#include "kda_pages.cuh"
#include "kda_scan.cuh"
#include "kda_tree.cuh"

namespace {

// What the kernels store is what kda_get_device_error returns.
static_assert((int)kda::DEV_OK == KDA_OK && (int)kda::DEV_TIMEOUT == KDA_ERR_TIMEOUT &&
                  (int)kda::DEV_BAD_SEQLENS == KDA_ERR_BAD_SEQLENS &&
                  (int)kda::DEV_RANGE == KDA_ERR_RANGE &&
                  (int)kda::DEV_BAD_INDEX == KDA_ERR_BAD_INDEX, "device error codes");

// Sticky device error word (one per device context; see kda_get_device_error).
__device__ unsigned g_device_error = 0;

thread_local char t_last_error[512] = "";

kda_status_t fail(kda_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_last_error, sizeof(t_last_error), fmt, ap);
    va_end(ap);
    return st;
}

kda_status_t cuda_fail(cudaError_t e, const char* what) {
    return fail(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;
unsigned* g_err_addr[kMaxDevices] = {};
std::mutex g_err_mu;

// Device address of the error word on the current device (looked up once per device).
kda_status_t device_error_word(unsigned** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(KDA_ERR_UNSUPPORTED, "device %d", dev);
    std::lock_guard<std::mutex> lock(g_err_mu);
    if (!g_err_addr[dev]) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_device_error);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(error word)");
        g_err_addr[dev] = static_cast<unsigned*>(p);
    }
    *out = g_err_addr[dev];
    return KDA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

kda_status_t check_ptr(const void* p, const char* name, bool required) {
    if (!p) return required ? fail(KDA_ERR_INVALID_ARG, "%s is NULL", name) : KDA_OK;
    if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return KDA_OK;
}

enum class Path { kPerToken, kChunk64 };

kda_status_t check_fwd_desc(const kda_fwd_desc_t* d, bool has_cu, Path* path) {
    if (!d) return fail(KDA_ERR_INVALID_ARG, "desc is NULL");
    if (d->B < 1 || d->T < 0 || d->H < 1 || d->dk < 1 || d->dv < 1 || d->num_seqs < 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%d T=%d H=%d dk=%d dv=%d N=%d", d->B, d->T,
                    d->H, d->dk, d->dv, d->num_seqs);
    if (d->dtype != KDA_F32 && d->dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)d->dtype);
    if (has_cu) {
        if (d->B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1");
    } else if (d->num_seqs != d->B) {
        return fail(KDA_ERR_INVALID_ARG, "num_seqs (%d) must equal B (%d) without cu_seqlens",
                    d->num_seqs, d->B);
    }
    if ((int64_t)d->B * d->T * d->H > (int64_t)1 << 40)
        return fail(KDA_ERR_INVALID_ARG, "problem too large");
    const bool tc_shape =
        d->dtype == KDA_BF16 && d->dk == 128 && d->dv == 128 && kda::chunk64_available();
    switch (d->chunk_size) {
        case KDA_CHUNK_AUTO:
            *path = tc_shape ? Path::kChunk64 : Path::kPerToken;
            break;
        case KDA_CHUNK_PER_TOKEN:
            *path = Path::kPerToken;
            break;
        case KDA_CHUNK_64:
            if (d->dtype == KDA_F32) {
                *path = Path::kPerToken;  // fp32 inputs always take the exact path
                break;
            }
            if (!tc_shape)
                return fail(KDA_ERR_UNSUPPORTED,
                            "chunk_size 64 needs bf16 with dk = dv = 128 (and the chunked kernel)");
            *path = Path::kChunk64;
            break;
        default:
            if (d->dtype == KDA_F32 && d->chunk_size > 0) {
                *path = Path::kPerToken;
                break;
            }
            return fail(KDA_ERR_UNSUPPORTED, "chunk_size %d", d->chunk_size);
    }
    if (*path == Path::kPerToken && (d->dk > 256 || d->dv > 256))
        return fail(KDA_ERR_UNSUPPORTED, "per-token path supports dk, dv <= 256");
    return KDA_OK;
}

}  // namespace

namespace kda {
void set_last_error(const char* msg) {
    snprintf(t_last_error, sizeof(t_last_error), "%s", msg);
}
}  // namespace kda

extern "C" {

int kda_version(void) { return 100; }

const char* kda_last_error(void) { return t_last_error; }

const char* kda_status_string(kda_status_t s) {
    switch (s) {
        case KDA_OK: return "ok";
        case KDA_ERR_INVALID_ARG: return "invalid argument";
        case KDA_ERR_UNSUPPORTED: return "unsupported configuration";
        case KDA_ERR_CUDA: return "CUDA runtime error";
        case KDA_ERR_TIMEOUT: return "device pipeline wait timed out";
        case KDA_ERR_BAD_SEQLENS: return "malformed cu_seqlens";
        case KDA_ERR_RANGE: return "decay out of range (reserved; no longer raised)";
        case KDA_ERR_BAD_INDEX: return "tree parent, path row or state page out of range";
    }
    return "unknown status";
}

// Segments of at least 32 chunks, at most 12, and one segment up to 64 chunks. Measured on one
// B200 (L2 flushed before each call): the long-context workload (1024 chunks per sequence, 64
// chains) takes 3.84, 3.89, 3.63, 3.71, 3.65 ms at 1, 4, 8, 12, 16 segments; the single-sequence
// one (64 chunks, 16 chains) 0.154, 0.178, 0.170, 0.168 ms at 1, 2, 3, 4: the next segment's
// intra-chunk launch takes the SMs before a short state pass can start, so a short chain gains no
// overlap and pays the side stream's joins.
// KDA_SPLIT_SEGMENTS (1-16, read per call) overrides the count, capped at the chunk count; the
// result is the same whatever the count (the state crosses segments in fp32).
static int split_segments(int ncT) {
    int s = ncT <= 64 ? 1 : ncT / 32;
    if (s > 12) s = 12;
    if (const char* env = std::getenv("KDA_SPLIT_SEGMENTS")) {
        const int v = std::atoi(env);
        if (v >= 1) s = v;
    }
    if (s > kda::kMaxSegments) s = kda::kMaxSegments;
    return s > ncT ? (ncT > 0 ? ncT : 1) : s;
}

// Two-level state pass for equal-length sequences with few chains (the sequential chunk chain,
// one SM per chain, would leave most SMs idle): P segments of m chunks, P >= 3, or 1 for the
// plain pass. Phases (one SM per unit): the state pass of segment 0 from h0 (with its outputs),
// beside the transition maps A_p and zero-start states B_p of segments 1 .. P-2 (2 (P-2) units per
// chain, no outputs); then S_{p+1} = A_p S_p + B_p in fp32 (P - 2 steps of a 128 x 128 x 128
// product per chain); then segments 1 .. P-1 at once from their initial states. P minimises a
// cost model in units of one chunk of the state pass (about 1.6 us on B200): the intra-chunk
// kernel (about 3.7 units of SM time per record, all SMs), then the phases, each ceil(units /
// 148) waves of m chunks, plus 2.5 units per combine step and 4 for the launches; the plain pass is
// intra-chunk kernel + chain (one segment) or the larger of the two (chunk segments overlapping).
// The two-level pass is used when it models at least 15 % faster. Measured on one B200 (L2
// flushed, ms per call at P = plain, 3, 4, 5, 6, 7, 8, 10): 1 x 4096 tokens x 16 heads 0.158,
// 0.147, 0.133, 0.129, 0.127, 0.144, 0.139, 0.141 (the model picks 6); 1 x 16384 x 16 0.543,
// 0.440, 0.381, 0.354, 0.336, 0.373, 0.359, 0.354 (picks 6); 1 x 8192 x 8 0.260, 0.205, 0.176,
// 0.162, 0.155, 0.150, 0.145, 0.143 (picks 10). KDA_SCAN_SEGMENTS (read per
// call) overrides: 0 or 1 = the plain pass, 3 .. 32 = that many segments (capped by the chunks).
static int scan_segments(int ncT, long long chains) {
    if (ncT < 3 || chains <= 0 || chains > 148) return 1;
    auto effective = [&](int P) {   // segments of ceil(ncT / P) chunks, none empty
        const int m = (ncT + P - 1) / P;
        return (ncT + m - 1) / m;
    };
    if (const char* env = std::getenv("KDA_SCAN_SEGMENTS")) {
        int v = std::atoi(env);
        if (v < 3) return 1;
        if (v > kda::kMaxScanSegments) v = kda::kMaxScanSegments;
        if (v > ncT) v = ncT;
        v = effective(v);
        return v >= 3 ? v : 1;
    }
    const double sms = 148.0, ch = (double)chains;
    const double intra = (double)ncT * ch * 3.7 / sms;
    const int S = split_segments(ncT);
    const double plain = S == 1 ? intra + ncT
                                : std::max(intra * sms / (sms - std::min(ch, 74.0)), (double)ncT);
    double best = 0.85 * plain;
    int bestP = 1;
    for (int P = 3; P <= std::min(ncT, kda::kMaxScanSegments); ++P) {
        if (effective(P) != P) continue;
        const int m = (ncT + P - 1) / P;
        const double w1 = std::ceil((2.0 * (P - 2) + 1.0) * ch / sms);
        const double w3 = std::ceil((P - 1.0) * ch / sms);
        const double cost = intra + (w1 + w3) * m + 2.5 * (P - 2) + 4.0;
        if (cost < best) best = cost, bestP = P;
    }
    return bestP;
}

int kda_fwd_algorithm(const kda_fwd_desc_t* desc, int has_cu_seqlens) {
    Path path;
    const kda_status_t st = check_fwd_desc(desc, has_cu_seqlens != 0, &path);
    if (st != KDA_OK) return -(int)st;
    return path == Path::kChunk64 ? KDA_CHUNK_64 : KDA_CHUNK_PER_TOKEN;
}

int kda_fwd_split_segments(const kda_fwd_desc_t* desc, int has_cu_seqlens) {
    Path path;
    const kda_status_t st = check_fwd_desc(desc, has_cu_seqlens != 0, &path);
    if (st != KDA_OK) return -(int)st;
    if (path != Path::kChunk64 || has_cu_seqlens || desc->T <= 0) return 1;
    const int ncT = (desc->T + 63) / 64;
    if (scan_segments(ncT, (long long)desc->num_seqs * desc->H) >= 3) return 1;
    return split_segments(ncT);
}

int kda_fwd_scan_segments(const kda_fwd_desc_t* desc, int has_cu_seqlens) {
    Path path;
    const kda_status_t st = check_fwd_desc(desc, has_cu_seqlens != 0, &path);
    if (st != KDA_OK) return -(int)st;
    if (path != Path::kChunk64 || has_cu_seqlens || desc->T <= 0) return 1;
    return scan_segments((desc->T + 63) / 64, (long long)desc->num_seqs * desc->H);
}

// Packed documents on the chunked path are scheduled longest first; the permutation lives in the
// caller's workspace (one int32 per document). Nothing else needs scratch.
static size_t order_bytes(const kda_fwd_desc_t* d, Path path) {
    const bool packed = d->B == 1 && d->num_seqs >= 2;  // without cu_seqlens num_seqs == B
    if (path != Path::kChunk64 || !packed || d->num_seqs > kda::kMaxOrderedDocs) return 0;
    return ((size_t)d->num_seqs * sizeof(int32_t) + 255) / 256 * 256;
}

// Workspace of the split chunked path (intra-chunk kernel + state pass), 256-byte aligned parts.
struct SplitLayout {
    size_t order, map, counters, state, decay, wq, ke, ut, aq, total;
    size_t maps, total_pscan;   // two-level state pass: its states, and the workspace it needs
    long long G;
    int ncT;
    int P;                      // segments of the two-level state pass (1: the plain pass)
    bool has_order;
};

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// packed: the call passes cu_seqlens (records are indexed floor(t0 / 64) + document + chunk).
static bool split_layout(const kda_fwd_desc_t* d, Path path, bool packed, SplitLayout* L) {
    if (path != Path::kChunk64 || d->T <= 0 || d->num_seqs <= 0) return false;
    L->ncT = (d->T + 63) / 64;
    L->G = packed ? (long long)L->ncT + d->num_seqs : (long long)d->B * L->ncT;
    const long long R = L->G * d->H;
    if (R * 128 > 0x7fffffffLL) return false;   // TMA row coordinates are 32-bit
    L->has_order = packed && d->num_seqs >= 2 && d->num_seqs <= kda::kMaxOrderedDocs;
    size_t off = 0;
    L->order = off; off += L->has_order ? up256((size_t)d->num_seqs * 4) : 0;
    L->map = off;   off += packed ? up256((size_t)L->G * 4) : 0;
    L->counters = off; off += up256((size_t)kda::kMaxSegments * 8);
    // state between chunk segments (equal-length sequences): N x H fp32 128 x 128
    L->state = off; off += packed ? 0 : (size_t)d->num_seqs * d->H * 65536;
    L->decay = off; off += up256((size_t)R * 512);
    L->wq = off;    off += (size_t)R * 32768;
    L->ke = off;    off += (size_t)R * 16384;
    L->ut = off;    off += (size_t)R * 16384;
    L->aq = off;    off += (size_t)R * 8192;
    L->total = off;
    // two-level state pass: A_p and B_p of segments 1 .. P-2, then the initial states of
    // segments 1 .. P-1, each N x H fp32 128 x 128
    L->P = packed ? 1 : scan_segments(L->ncT, (long long)d->num_seqs * d->H);
    L->maps = off;
    if (L->P >= 3) off += (size_t)(3 * L->P - 5) * d->num_seqs * d->H * 65536;
    L->total_pscan = off;
    return true;
}

size_t kda_fwd_workspace_size(const kda_fwd_desc_t* desc) {
    Path path;
    const bool maybe_packed = desc && desc->B == 1;
    if (!desc || check_fwd_desc(desc, maybe_packed && desc->num_seqs >= 2, &path) != KDA_OK)
        return 0;
    t_last_error[0] = 0;
    SplitLayout L;
    // B == 1 may come with cu_seqlens: size for the packed record numbering (one record more
    // per document than a single sequence needs), or for the two-level state pass without them
    if (split_layout(desc, path, maybe_packed, &L)) {
        size_t t = L.total_pscan;
        SplitLayout U;
        if (maybe_packed && split_layout(desc, path, false, &U)) t = std::max(t, U.total_pscan);
        return t;
    }
    return order_bytes(desc, path);
}

size_t kda_fwd_workspace_size_min(const kda_fwd_desc_t* desc) {
    Path path;
    if (!desc || check_fwd_desc(desc, desc->B == 1 && desc->num_seqs >= 2, &path) != KDA_OK)
        return 0;
    t_last_error[0] = 0;
    return order_bytes(desc, path);
}

// Chunk segments of the split path for equal-length sequences with ncT chunks each: the state
// pass of segment s (one CTA per chain, so at most N x H SMs) runs on a side stream while the
// intra-chunk kernel works on segment s + 1 with the other SMs. Short sequences run in one.
// Side stream (highest priority, so that its state-pass CTAs take SMs first when both kernels are
// ready) and events, one set per host thread and device: concurrent calls from several host
// threads never share events.
struct SideStream {
    cudaStream_t aux = nullptr;
    cudaEvent_t join = nullptr;
    cudaEvent_t seg[kda::kMaxSegments] = {};
};
static thread_local SideStream t_side[kMaxDevices];

static cudaError_t side_stream(SideStream** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    SideStream& ss = t_side[dev];
    if (!ss.aux) {
        int least = 0, greatest = 0;
        if ((e = cudaDeviceGetStreamPriorityRange(&least, &greatest)) != cudaSuccess) return e;
        cudaStream_t aux;
        if ((e = cudaStreamCreateWithPriority(&aux, cudaStreamNonBlocking, greatest)) !=
            cudaSuccess)
            return e;
        if ((e = cudaEventCreateWithFlags(&ss.join, cudaEventDisableTiming)) != cudaSuccess)
            return e;
        for (int i = 0; i < kda::kMaxSegments; ++i)
            if ((e = cudaEventCreateWithFlags(&ss.seg[i], cudaEventDisableTiming)) != cudaSuccess)
                return e;
        ss.aux = aux;
    }
    *out = &ss;
    return cudaSuccess;
}

// kda_fwd with an optional gated RMSNorm epilogue (norm == nullptr: none).
static kda_status_t fwd_impl(const kda_fwd_desc_t* d, const void* q, const void* k,
                             const void* v, const float* log_g, const void* beta,
                             const float* h0, const int32_t* cu_seqlens, void* o, float* hT,
                             void* workspace, size_t workspace_bytes,
                             const kda_out_norm_t* norm, kda_stream_t stream) {
    t_last_error[0] = 0;
    Path path;
    kda_status_t st = check_fwd_desc(d, cu_seqlens != nullptr, &path);
    if (st != KDA_OK) return st;
    const bool tokens = (int64_t)d->B * d->T > 0;
    const bool has_units = d->num_seqs > 0;
    if ((st = check_ptr(q, "q", tokens)) || (st = check_ptr(k, "k", tokens)) ||
        (st = check_ptr(v, "v", tokens)) || (st = check_ptr(log_g, "log_g", tokens)) ||
        (st = check_ptr(beta, "beta", false)) || (st = check_ptr(o, "o", tokens)) ||
        (st = check_ptr(h0, "h0", false)) || (st = check_ptr(hT, "hT", false)) ||
        (st = check_ptr(cu_seqlens, "cu_seqlens", false)))
        return st;
    if (tokens && !beta) return fail(KDA_ERR_INVALID_ARG, "beta is NULL");
    if (norm) {
        if ((st = check_ptr(norm->gate, "norm gate", tokens)) ||
            (st = check_ptr(norm->weight, "norm weight", tokens)))
            return st;
        if (!(norm->eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "norm eps must be >= 0");
    }
    SplitLayout L;
    const bool split = tokens && split_layout(d, path, cu_seqlens != nullptr, &L) && workspace &&
                       aligned16(workspace) && workspace_bytes >= L.total;
    // the two-level state pass when the plan has one and the workspace holds its states
    const bool pscan = split && !cu_seqlens && L.P >= 3 && workspace_bytes >= L.total_pscan;
    const size_t need_ws = (cu_seqlens && !split) ? order_bytes(d, path) : 0;
    if (need_ws > 0 && (workspace_bytes < need_ws || !workspace || !aligned16(workspace)))
        return fail(KDA_ERR_INVALID_ARG,
                    "workspace must be a 16-byte aligned device buffer of %zu bytes "
                    "(kda_fwd_workspace_size)", need_ws);
    if (!has_units) return KDA_OK;

    kda::FwdParams p{};
    p.q = q; p.k = k; p.v = v; p.log_g = log_g; p.beta = beta; p.h0 = h0;
    p.cu_seqlens = cu_seqlens; p.o = o; p.hT = hT;
    p.B = d->B; p.T = d->T; p.H = d->H; p.dk = d->dk; p.dv = d->dv; p.N = d->num_seqs;
    p.bf16 = d->dtype == KDA_BF16;
    p.doc_order = nullptr;
    if ((st = device_error_word(&p.err)) != KDA_OK) return st;
    // the epilogue: on the split path the state pass's epilogue warps apply it to the fp32 o as
    // they store it; the other paths run it as one bandwidth-bound pass over o afterwards
    auto norm_after = [&]() -> cudaError_t {
        if (!norm || !tokens) return cudaSuccess;
        return kda::launch_out_norm_gated(o, norm->gate, norm->weight, norm->eps, o,
                                          (long long)d->B * d->T * d->H, d->dv, p.bf16,
                                          reinterpret_cast<cudaStream_t>(stream));
    };
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (split) {
        uint8_t* w = static_cast<uint8_t*>(workspace);
        kda::SplitWorkspace ws;
        ws.wq = reinterpret_cast<__nv_bfloat16*>(w + L.wq);
        ws.ke = reinterpret_cast<__nv_bfloat16*>(w + L.ke);
        ws.ut = reinterpret_cast<__nv_bfloat16*>(w + L.ut);
        ws.aq = reinterpret_cast<__nv_bfloat16*>(w + L.aq);
        ws.decay = reinterpret_cast<float*>(w + L.decay);
        ws.map = cu_seqlens ? reinterpret_cast<int32_t*>(w + L.map) : nullptr;
        ws.counters = reinterpret_cast<unsigned long long*>(w + L.counters);
        ws.state = cu_seqlens ? nullptr : reinterpret_cast<float*>(w + L.state);
        ws.G = L.G;
        ws.ncT = L.ncT;
        p.split = &ws;
        if (L.has_order) {
            int32_t* order = reinterpret_cast<int32_t*>(w + L.order);
            e = kda::launch_doc_order(cu_seqlens, d->num_seqs, order, s);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd document scheduling");
            p.doc_order = order;
        }
        if (cu_seqlens) {
            e = kda::launch_chunk_map(cu_seqlens, d->num_seqs, d->T, L.G, ws.map, p.err, s);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd chunk map");
        }
        kda::ScanNorm sn{};
        const kda::ScanNorm* snp = nullptr;
        if (norm) {
            sn.gate = norm->gate;
            sn.weight = norm->weight;
            sn.eps = norm->eps;
            snp = &sn;
        }
        const int S = cu_seqlens || pscan ? 1 : split_segments(L.ncT);
        e = cudaMemsetAsync(ws.counters, 0, sizeof(unsigned long long) * S, s);
        if (e != cudaSuccess) return cuda_fail(e, "kda_fwd workspace counters");
        if (pscan) {
            // intra-chunk kernel over every chunk; then segment 0 (side stream) beside the maps
            // of segments 1 .. P-2 (caller's stream); the segments' initial states; then
            // segments 1 .. P-1 at once
            const int P = L.P, m = (L.ncT + P - 1) / P;
            const size_t states = (size_t)d->num_seqs * d->H * 16384;   // floats per state set
            float* maps = reinterpret_cast<float*>(w + L.maps);         // A: [P-2], B: [P-2]
            float* sinit = maps + 2 * (size_t)(P - 2) * states;          // [P-1]
            SideStream* ss = nullptr;
            if ((e = side_stream(&ss)) != cudaSuccess) return cuda_fail(e, "kda_fwd side stream");
            e = kda::launch_chunk64_intra(p, 0, L.ncT, ws.counters, s);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd intra-chunk launch");
            const kda::ScanSegment seg0{0, m, h0, sinit};
            const kda::ScanSegment mid{0, 0, nullptr, maps};
            kda::ScanSplit mid_split;
            mid_split.seg_m = m;
            mid_split.seg_p0 = 1;
            mid_split.seg_count = P - 2;
            mid_split.groups = 2;
            mid_split.nseg = P;
            mid_split.ident = true;
            mid_split.no_out = true;
            const kda::ScanSegment rest{0, 0, sinit, hT};
            kda::ScanSplit rest_split;
            rest_split.seg_m = m;
            rest_split.seg_p0 = 1;
            rest_split.seg_count = P - 1;
            rest_split.nseg = P;
            rest_split.hT_last = true;
            cudaError_t first = cudaSuccess;
            if ((first = cudaEventRecord(ss->seg[0], s)) == cudaSuccess &&
                (first = cudaStreamWaitEvent(ss->aux, ss->seg[0], 0)) == cudaSuccess &&
                (first = kda::launch_chunk_scan(p, seg0, ss->aux, snp)) == cudaSuccess)
                first = kda::launch_chunk_scan_split(p, mid, mid_split, s);
            // join even after a failed launch, so that nothing is left pending on the side stream
            e = cudaEventRecord(ss->join, ss->aux);
            if (e == cudaSuccess) e = cudaStreamWaitEvent(s, ss->join, 0);
            if (first != cudaSuccess) return cuda_fail(first, "kda_fwd state-pass launch");
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd side stream join");
            e = kda::launch_scan_combine(maps, maps + (size_t)(P - 2) * states, sinit,
                                         d->num_seqs * d->H, P - 2, s);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd segment-state launch");
            e = kda::launch_chunk_scan_split(p, rest, rest_split, s, snp);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd state-pass launch");
        } else if (S == 1) {
            e = kda::launch_chunk64_intra(p, 0, L.ncT, ws.counters, s);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd intra-chunk launch");
            e = kda::launch_chunk_scan(p, kda::ScanSegment{0, L.ncT, h0, hT}, s, snp);
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd state-pass launch");
        } else {
            // intra(0) intra(1) ... on the caller's stream; state(i) on the side stream after
            // intra(i) and state(i - 1); the caller's stream then waits for the last state pass
            SideStream* ss = nullptr;
            if ((e = side_stream(&ss)) != cudaSuccess) return cuda_fail(e, "kda_fwd side stream");
            cudaError_t first = cudaSuccess;
            for (int i = 0; i < S && first == cudaSuccess; ++i) {
                const int cb = (int)((long long)L.ncT * i / S);
                const int ce = (int)((long long)L.ncT * (i + 1) / S);
                const kda::ScanSegment seg{cb, ce, i == 0 ? h0 : ws.state,
                                           i == S - 1 ? hT : ws.state};
                if ((e = kda::launch_chunk64_intra(p, cb, ce - cb, ws.counters + i, s)) !=
                        cudaSuccess ||
                    (e = cudaEventRecord(ss->seg[i], s)) != cudaSuccess ||
                    (e = cudaStreamWaitEvent(ss->aux, ss->seg[i], 0)) != cudaSuccess ||
                    (e = kda::launch_chunk_scan(p, seg, ss->aux, snp)) != cudaSuccess)
                    first = e;
            }
            // join even after a failed launch, so that nothing is left pending on the side stream
            e = cudaEventRecord(ss->join, ss->aux);
            if (e == cudaSuccess) e = cudaStreamWaitEvent(s, ss->join, 0);
            if (first != cudaSuccess) return cuda_fail(first, "kda_fwd split launch");
            if (e != cudaSuccess) return cuda_fail(e, "kda_fwd side stream join");
        }
        return KDA_OK;
    }
    if (need_ws > 0 && tokens) {
        int32_t* order = static_cast<int32_t*>(workspace);
        e = kda::launch_doc_order(cu_seqlens, d->num_seqs, order, s);
        if (e != cudaSuccess) return cuda_fail(e, "kda_fwd document scheduling");
        p.doc_order = order;
    }
    e = path == Path::kChunk64 ? kda::launch_chunk64(p, s) : kda::launch_recurrent(p, s);
    if (e != cudaSuccess) return cuda_fail(e, "kda_fwd launch");
    e = norm_after();
    if (e != cudaSuccess) return cuda_fail(e, "kda_fwd output norm launch");
    return KDA_OK;
}

kda_status_t kda_fwd(const kda_fwd_desc_t* d, const void* q, const void* k, const void* v,
                     const float* log_g, const void* beta, const float* h0,
                     const int32_t* cu_seqlens, void* o, float* hT, void* workspace,
                     size_t workspace_bytes, kda_stream_t stream) {
    return fwd_impl(d, q, k, v, log_g, beta, h0, cu_seqlens, o, hT, workspace, workspace_bytes,
                    nullptr, stream);
}

kda_status_t kda_fwd_normed(const kda_fwd_desc_t* d, const void* q, const void* k,
                            const void* v, const float* log_g, const void* beta,
                            const float* h0, const int32_t* cu_seqlens,
                            const kda_out_norm_t* norm, void* y, float* hT, void* workspace,
                            size_t workspace_bytes, kda_stream_t stream) {
    if (!norm) {
        t_last_error[0] = 0;
        return fail(KDA_ERR_INVALID_ARG, "norm is NULL");
    }
    if (d && d->dv > 256) {
        t_last_error[0] = 0;
        return fail(KDA_ERR_UNSUPPORTED, "the output norm supports dv <= 256");
    }
    return fwd_impl(d, q, k, v, log_g, beta, h0, cu_seqlens, y, hT, workspace, workspace_bytes,
                    norm, stream);
}

static kda_status_t check_bwd_desc(const kda_fwd_desc_t* d, bool has_cu) {
    Path path;
    kda_status_t st = check_fwd_desc(d, has_cu, &path);
    if (st != KDA_OK) return st;
    if (d->dk != 128 || d->dv != 128)
        return fail(KDA_ERR_UNSUPPORTED, "kda_bwd supports dk = dv = 128 (got %d, %d)", d->dk,
                    d->dv);
    return KDA_OK;
}

size_t kda_bwd_workspace_size(const kda_fwd_desc_t* desc) {
    if (!desc || check_bwd_desc(desc, desc->B == 1 && desc->num_seqs >= 2) != KDA_OK) return 0;
    t_last_error[0] = 0;
    if (desc->T <= 0 || desc->num_seqs <= 0) return 0;
    return kda::bwd_workspace_bytes((long long)desc->num_seqs * desc->H, desc->T);
}

kda_status_t kda_bwd(const kda_fwd_desc_t* d, const void* q, const void* k, const void* v,
                     const float* log_g, const void* beta, const float* h0,
                     const int32_t* cu_seqlens, const void* dout, const float* dhT, float* dq,
                     float* dk, float* dv, float* dlog_g, float* dbeta, float* dh0,
                     void* workspace, size_t workspace_bytes, kda_stream_t stream) {
    t_last_error[0] = 0;
    kda_status_t st = check_bwd_desc(d, cu_seqlens != nullptr);
    if (st != KDA_OK) return st;
    const bool tokens = (int64_t)d->B * d->T > 0;
    if ((st = check_ptr(q, "q", tokens)) || (st = check_ptr(k, "k", tokens)) ||
        (st = check_ptr(v, "v", tokens)) || (st = check_ptr(log_g, "log_g", tokens)) ||
        (st = check_ptr(beta, "beta", false)) || (st = check_ptr(dout, "do", tokens)) ||
        (st = check_ptr(dq, "dq", tokens)) || (st = check_ptr(dk, "dk", tokens)) ||
        (st = check_ptr(dv, "dv", tokens)) || (st = check_ptr(dlog_g, "dlog_g", tokens)) ||
        (st = check_ptr(dbeta, "dbeta", false)) || (st = check_ptr(h0, "h0", false)) ||
        (st = check_ptr(dhT, "dhT", false)) || (st = check_ptr(dh0, "dh0", false)) ||
        (st = check_ptr(cu_seqlens, "cu_seqlens", false)))
        return st;
    if (tokens && (!beta || !dbeta)) return fail(KDA_ERR_INVALID_ARG, "beta or dbeta is NULL");
    const long long chains = (long long)d->num_seqs * d->H;
    const size_t need = (tokens && chains > 0) ? kda::bwd_workspace_bytes(chains, d->T) : 0;
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return fail(KDA_ERR_INVALID_ARG,
                    "workspace must be a 16-byte aligned device buffer of %zu bytes "
                    "(kda_bwd_workspace_size)", need);
    if (chains == 0) return KDA_OK;
    if (!tokens) {   // no tokens: dh0 = dhT (or zero)
        if (!dh0) return KDA_OK;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        const size_t bytes = (size_t)chains * 128 * 128 * sizeof(float);
        cudaError_t e = dhT ? cudaMemcpyAsync(dh0, dhT, bytes, cudaMemcpyDeviceToDevice, s)
                            : cudaMemsetAsync(dh0, 0, bytes, s);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_bwd dh0");
    }
    kda::BwdParams p{};
    p.q = q; p.k = k; p.v = v; p.beta = beta; p.dout = dout; p.log_g = log_g; p.h0 = h0;
    p.dhT = dhT; p.cu_seqlens = cu_seqlens; p.dq = dq; p.dk = dk; p.dv = dv; p.dlog_g = dlog_g;
    p.dbeta = dbeta; p.dh0 = dh0; p.workspace = workspace;
    p.T = d->T; p.H = d->H; p.N = d->num_seqs;
    p.bf16 = d->dtype == KDA_BF16;
    if ((st = device_error_word(&p.err)) != KDA_OK) return st;
    cudaError_t e = kda::launch_bwd(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_bwd launch");
    return KDA_OK;
}

kda_status_t kda_out_norm_gated(long long vectors, int dv, kda_dtype_t dtype, const void* x,
                                const void* gate, const float* weight, float eps, void* y,
                                kda_stream_t stream) {
    t_last_error[0] = 0;
    if (vectors < 0 || dv < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes vectors=%lld dv=%d",
                                           vectors, dv);
    if (dv > 256) return fail(KDA_ERR_UNSUPPORTED, "the output norm supports dv <= 256");
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be >= 0");
    kda_status_t st;
    const bool any = vectors > 0;
    if ((st = check_ptr(x, "x", any)) || (st = check_ptr(gate, "gate", any)) ||
        (st = check_ptr(weight, "weight", any)) || (st = check_ptr(y, "y", any)))
        return st;
    if (!any) return KDA_OK;
    cudaError_t e = kda::launch_out_norm_gated(x, gate, weight, eps, y, vectors, dv,
                                               dtype == KDA_BF16,
                                               reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_out_norm_gated launch");
    return KDA_OK;
}

kda_status_t kda_short_conv(int B, int T, int C, int W, kda_dtype_t dtype, const void* x,
                            const float* weight, const int32_t* cu_seqlens, int num_seqs,
                            kda_activation_t act, int norm_group, float eps, void* y,
                            kda_stream_t stream) {
    t_last_error[0] = 0;
    if (B < 1 || T < 0 || C < 1 || num_seqs < 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%d T=%d C=%d N=%d", B, T, C, num_seqs);
    if (W < 1 || W > 8) return fail(KDA_ERR_UNSUPPORTED, "kernel width %d (1..8)", W);
    if (C % 4) return fail(KDA_ERR_UNSUPPORTED, "C = %d is not a multiple of 4", C);
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (act != KDA_ACT_NONE && act != KDA_ACT_SILU)
        return fail(KDA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    if (norm_group != 0 && (norm_group < 4 || norm_group > 128 ||
                            (norm_group & (norm_group - 1)) || C % norm_group))
        return fail(KDA_ERR_UNSUPPORTED,
                    "norm_group %d (0, or a power of two from 4 to 128 dividing C)", norm_group);
    if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be >= 0");
    if (cu_seqlens && B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1");
    if (cu_seqlens && num_seqs < 1)
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens needs num_seqs >= 1");
    if ((int64_t)B * T * C > (int64_t)1 << 40) return fail(KDA_ERR_INVALID_ARG, "problem too large");
    kda_status_t st;
    const bool any = (int64_t)B * T > 0;
    if ((st = check_ptr(x, "x", any)) || (st = check_ptr(weight, "weight", any)) ||
        (st = check_ptr(y, "y", any)) || (st = check_ptr(cu_seqlens, "cu_seqlens", false)))
        return st;
    if (!any) return KDA_OK;
    const size_t esz = dtype == KDA_BF16 ? 2 : 4;
    const uintptr_t xb = reinterpret_cast<uintptr_t>(x), yb = reinterpret_cast<uintptr_t>(y);
    const size_t bytes = (size_t)B * T * C * esz;
    if (xb < yb + bytes && yb < xb + bytes)
        return fail(KDA_ERR_INVALID_ARG, "y overlaps x (the window reads earlier rows of x)");
    unsigned* err = nullptr;
    if ((st = device_error_word(&err)) != KDA_OK) return st;
    cudaError_t e = kda::launch_short_conv(x, weight, cu_seqlens, num_seqs, y, B, T, C, W,
                                           dtype == KDA_BF16, (int)act, norm_group, eps, err,
                                           reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_short_conv launch");
    return KDA_OK;
}

kda_status_t kda_decode_step(int N, int H, int dk, int dv, kda_dtype_t dtype, const void* q,
                             const void* k, const void* v, const float* log_g, const void* beta,
                             float* S_inout, void* o, kda_stream_t stream) {
    t_last_error[0] = 0;
    if (N < 0 || H < 1 || dk < 1 || dv < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d H=%d dk=%d dv=%d", N, H, dk, dv);
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (dk > 256 || dv > 256) return fail(KDA_ERR_UNSUPPORTED, "decode supports dk, dv <= 256");
    kda_status_t st;
    const bool any = N > 0;
    if ((st = check_ptr(q, "q", any)) || (st = check_ptr(k, "k", any)) ||
        (st = check_ptr(v, "v", any)) || (st = check_ptr(log_g, "log_g", any)) ||
        (st = check_ptr(beta, "beta", any)) || (st = check_ptr(S_inout, "S_inout", any)) ||
        (st = check_ptr(o, "o", any)))
        return st;
    if (!any) return KDA_OK;
    unsigned* err = nullptr;
    if ((st = device_error_word(&err)) != KDA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dk == 128 && dv == 128) {
        kda::DecodeParams p{q, k, v, log_g, beta, S_inout, o, N, H, dk, dv,
                            dtype == KDA_BF16, err};
        e = kda::launch_decode_d128(p, s);
    } else {
        // general sizes: the per-token walk over one token, state read from and written to S
        kda::FwdParams p{};
        p.q = q; p.k = k; p.v = v; p.log_g = log_g; p.beta = beta; p.h0 = S_inout;
        p.cu_seqlens = nullptr; p.o = o; p.hT = S_inout;
        p.B = N; p.T = 1; p.H = H; p.dk = dk; p.dv = dv; p.N = N;
        p.bf16 = dtype == KDA_BF16;
        p.err = err;
        e = kda::launch_recurrent(p, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "kda_decode_step launch");
    return KDA_OK;
}

kda_status_t kda_decode_tokens(int N, int H, int T, int dk, int dv, kda_dtype_t dtype,
                               const void* q, const void* k, const void* v, const float* log_g,
                               const void* beta, float* S_inout, void* o, kda_stream_t stream) {
    t_last_error[0] = 0;
    if (N < 0 || H < 1 || T < 0 || dk < 1 || dv < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d H=%d T=%d dk=%d dv=%d", N, H, T, dk,
                    dv);
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (dk > 256 || dv > 256) return fail(KDA_ERR_UNSUPPORTED, "decode supports dk, dv <= 256");
    if ((int64_t)N * T * H > (int64_t)1 << 40) return fail(KDA_ERR_INVALID_ARG, "problem too large");
    kda_status_t st;
    const bool any = N > 0 && T > 0;
    if ((st = check_ptr(q, "q", any)) || (st = check_ptr(k, "k", any)) ||
        (st = check_ptr(v, "v", any)) || (st = check_ptr(log_g, "log_g", any)) ||
        (st = check_ptr(beta, "beta", any)) || (st = check_ptr(S_inout, "S_inout", any)) ||
        (st = check_ptr(o, "o", any)))
        return st;
    if (!any) return KDA_OK;
    unsigned* err = nullptr;
    if ((st = device_error_word(&err)) != KDA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dk == 128 && dv == 128) {
        kda::DecodeParams p{q, k, v, log_g, beta, S_inout, o, N, H, dk, dv,
                            dtype == KDA_BF16, err};
        e = kda::launch_decode_tokens_d128(p, T, s);
    } else {
        // general sizes: the per-token walk over N sequences of T tokens, state in place
        kda::FwdParams p{};
        p.q = q; p.k = k; p.v = v; p.log_g = log_g; p.beta = beta; p.h0 = S_inout;
        p.cu_seqlens = nullptr; p.o = o; p.hT = S_inout;
        p.B = N; p.T = T; p.H = H; p.dk = dk; p.dv = dv; p.N = N;
        p.bf16 = dtype == KDA_BF16;
        p.err = err;
        e = kda::launch_recurrent(p, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "kda_decode_tokens launch");
    return KDA_OK;
}

// ------------------------------------------------------------------ linear attention

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

struct Span {
    const void* at;
    size_t bytes;
    const char* name;
};

// No output overlaps an input or another output: the first `outputs` of `spans` are outputs.
static kda_status_t check_apart(std::initializer_list<Span> spans, size_t outputs) {
    for (const Span *a = spans.begin(); a < spans.begin() + outputs; ++a)
        for (const Span* b = a + 1; b < spans.end(); ++b)
            if (overlap(a->at, a->bytes, b->at, b->bytes))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", a->name, b->name);
    return KDA_OK;
}

static kda_status_t check_linear_desc(const kda_linear_desc_t* d, bool has_cu) {
    if (!d) return fail(KDA_ERR_INVALID_ARG, "desc is NULL");
    if (d->B < 1 || d->T < 0 || d->H < 1 || d->Hk < 1 || d->dk < 1 || d->dv < 1 || d->num_seqs < 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%d T=%d H=%d Hk=%d dk=%d dv=%d N=%d", d->B,
                    d->T, d->H, d->Hk, d->dk, d->dv, d->num_seqs);
    if (d->H % d->Hk)
        return fail(KDA_ERR_INVALID_ARG, "H = %d is not a multiple of Hk = %d", d->H, d->Hk);
    if (d->dtype != KDA_F32 && d->dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)d->dtype);
    if (d->gate != KDA_GATE_TOKEN && d->gate != KDA_GATE_HEAD)
        return fail(KDA_ERR_INVALID_ARG, "unknown gate %d", (int)d->gate);
    if (d->dk > 256 || d->dv > 256)
        return fail(KDA_ERR_UNSUPPORTED, "linear attention supports dk, dv <= 256");
    if (has_cu) {
        if (d->B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1");
        if (d->num_seqs == 0 && d->T > 0)
            return fail(KDA_ERR_INVALID_ARG, "%d tokens but no documents", d->T);
    } else if (d->num_seqs != d->B) {
        return fail(KDA_ERR_INVALID_ARG, "num_seqs (%d) must equal B (%d) without cu_seqlens",
                    d->num_seqs, d->B);
    }
    // (a row or a segment's first one, up to T and a segment's length behind it, is held in an int)
    if ((int64_t)d->B * d->T * d->H > (int64_t)1 << 40 || (int64_t)d->B * d->T > 1 << 30 ||
        (int64_t)d->num_seqs * d->H > 0x7fffffffLL)
        return fail(KDA_ERR_INVALID_ARG, "problem too large");
    return KDA_OK;
}

// Whether the chunked kernel runs. A CTA of it takes about 9 us for a sequence of up to one chunk,
// one at a time per SM; the walk takes shorter, many sequences faster: 1000 sequences x 16 heads of
// 16, 32, 64 tokens 1016, 1736, 3192 us against 2698, 2687, 2636; 8 x 16 heads of 4 and 16 tokens
// 17 and 37 against 26 us.
static bool linear_chunked(const kda_linear_desc_t* d) {
    if (!kda::linear_chunk_takes(d->dtype == KDA_BF16, d->dk, d->dv)) return false;
    const int64_t tokens = (int64_t)d->B * d->T, n = d->num_seqs;
    const bool many = n * d->H * ((d->dv + 63) / 64) >= 512;
    return tokens > 4 * n && (tokens > 32 * n || !many);
}

// Tokens per segment of the per-token walk (0: whole sequences). The walk has one warp per 16 value
// columns of a (segment, head) (8 above dk = 128); segments are cut so that about 4096 warps (7 per
// scheduler) share the work: one fp32 prompt of 4096 tokens x 16 heads takes 301 us, 346 with 2048
// and 314 with 8192. Below 64 tokens a segment's states cost more than it gains (4 x 1000 tokens x 4
// heads of 64 x 64 56 us at 64, 62 at 32), but for a short prompt (100 tokens x 16 heads: 52 us at
// 64, 41 at 32 when it was chosen, 32 now).
static int linear_walk_segment(const kda_linear_desc_t* d) {
    const int nc = d->dk <= 128 ? 16 : 8;
    const int64_t groups = (int64_t)d->H * ((d->dv + nc - 1) / nc);
    const int64_t want = ((int64_t)d->B * d->T * groups / 4096 + 31) / 32 * 32;
    const int L = (int)std::max<int64_t>(d->T <= 256 ? 32 : 64, want);
    if (d->num_seqs * groups >= 2048) return 0;
    return d->T > L ? L : 0;
}

// Tokens per segment of the chunked kernel (0: whole sequences), whose CTAs take one (segment,
// head, 64 value columns) each, one per SM. Equal lengths: the count of segments with the least
// modelled time, in units of one chunk with outputs (about 2 us): waves of m such chunks, and
// before them the states of all segments but the last at 0.4 of a chunk each, 3 units per CTA's
// start and end, 1 for the further launch. Packed documents, whose lengths the host does not see,
// are cut only where one takes much more than an SM's even share of all chunks (the CTAs take the
// longest first, so shorter ones pack well).
static int linear_chunk_segment(const kda_linear_desc_t* d, bool packed) {
    const int n = (d->T + kda::kLinearChunk - 1) / kda::kLinearChunk;
    const double units = (double)d->H * ((d->dv + 63) / 64), sms = 148.0;
    if (packed && d->num_seqs > 1) {
        const int m = std::max(8, (int)std::ceil(1.25 * n * units / sms));
        return n > m ? m * kda::kLinearChunk : 0;
    }
    const double all = units * d->num_seqs;
    double best = std::ceil(all / sms) * (n + 3.0);
    int m_best = 0;
    for (int m = 1; m < n; ++m) {
        const int P = (n + m - 1) / m;
        if (P > 64) continue;
        const double cost = std::ceil(all * (P - 1) / sms) * (0.4 * m + 3.0) +
                            std::ceil(all * P / sms) * (m + 3.0) + 1.0;
        if (cost < best) best = cost, m_best = m;
    }
    return m_best * kda::kLinearChunk;
}

// Segments up to which the chunked kernel's CTAs chain their own initial state.
constexpr int kChainedSegments = 12;

static int linear_segment(const kda_linear_desc_t* d, bool packed) {
    if (d->num_seqs > 1024 || d->H > 65535) return 0;   // enough sequences to fill the GPU
    return linear_chunked(d) ? linear_chunk_segment(d, packed) : linear_walk_segment(d);
}

struct LinearLayout {
    int seg_tokens, slots;
    size_t decay, total;
};

static LinearLayout linear_layout(const kda_linear_desc_t* d, bool packed) {
    LinearLayout L{linear_segment(d, packed), d->num_seqs, 0, 0};
    if (L.seg_tokens == 0) return L;
    const int segs = (d->T + L.seg_tokens - 1) / L.seg_tokens;
    L.slots = packed ? d->T / L.seg_tokens + d->num_seqs : d->num_seqs * segs;
    L.decay = up256((size_t)L.slots * d->H * d->dk * d->dv * sizeof(float));
    L.total = L.decay + up256((size_t)L.slots * d->H * sizeof(float));
    return L;
}

size_t kda_linear_fwd_workspace_size(const kda_linear_desc_t* desc) {
    if (check_linear_desc(desc, desc && desc->B == 1) != KDA_OK) return 0;
    t_last_error[0] = 0;
    // B == 1 may come with cu_seqlens, with other segments and one slot more per document
    const size_t whole = desc->num_seqs == desc->B ? linear_layout(desc, false).total : 0;
    return desc->B == 1 ? std::max(whole, linear_layout(desc, true).total) : whole;
}

static kda::LinearParams linear_params(const kda_linear_desc_t* d) {
    kda::LinearParams p{};
    p.B = d->B; p.T = d->T; p.H = d->H; p.Hk = d->Hk; p.dk = d->dk; p.dv = d->dv;
    p.N = d->num_seqs;
    p.bf16 = d->dtype == KDA_BF16;
    p.gate_head = d->gate == KDA_GATE_HEAD;
    p.slots = d->num_seqs;
    return p;
}

kda_status_t kda_linear_fwd(const kda_linear_desc_t* d, const void* q, const void* k,
                            const void* v, const float* log_g, const float* h0,
                            const int32_t* cu_seqlens, void* o, float* hT, void* workspace,
                            size_t workspace_bytes, kda_stream_t stream) {
    t_last_error[0] = 0;
    kda_status_t st = check_linear_desc(d, cu_seqlens != nullptr);
    if (st != KDA_OK) return st;
    const bool tokens = (int64_t)d->B * d->T > 0;
    if ((st = check_ptr(q, "q", tokens)) || (st = check_ptr(k, "k", tokens)) ||
        (st = check_ptr(v, "v", tokens)) || (st = check_ptr(log_g, "log_g", tokens)) ||
        (st = check_ptr(h0, "h0", false)) || (st = check_ptr(hT, "hT", false)) ||
        (st = check_ptr(o, "o", tokens)) || (st = check_ptr(cu_seqlens, "cu_seqlens", false)))
        return st;
    const size_t esz = d->dtype == KDA_BF16 ? 2 : 4, rows = (size_t)d->B * d->T;
    const size_t qk_bytes = rows * d->Hk * d->dk * esz, v_bytes = rows * d->H * d->dv * esz;
    const size_t h_bytes = (size_t)d->num_seqs * d->H * d->dk * d->dv * sizeof(float);
    const LinearLayout L = linear_layout(d, cu_seqlens != nullptr);
    if (L.total > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < L.total))
        return fail(KDA_ERR_INVALID_ARG,
                    "workspace must be a 16-byte aligned device buffer of %zu bytes "
                    "(kda_linear_fwd_workspace_size)", L.total);
    const size_t gates = d->gate == KDA_GATE_HEAD ? d->H : rows * d->H;
    if ((st = check_apart({{o, v_bytes, "o"}, {hT, h_bytes, "hT"},
                          {L.total > 0 ? workspace : nullptr, L.total, "the workspace"},
                          {q, qk_bytes, "q"}, {k, qk_bytes, "k"}, {v, v_bytes, "v"},
                          {log_g, gates * 4, "log_g"}, {h0, h_bytes, "h0"},
                          {cu_seqlens, ((size_t)d->num_seqs + 1) * 4, "cu_seqlens"}}, 3)) !=
        KDA_OK)
        return st;
    if (d->num_seqs == 0) return KDA_OK;
    kda::LinearParams p = linear_params(d);
    p.q = q; p.k = k; p.v = v; p.log_g = log_g; p.h0 = h0; p.cu_seqlens = cu_seqlens;
    p.o = o; p.hT = hT;
    if ((st = device_error_word(&p.err)) != KDA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    auto pass = [&](kda::LinearPass which) {
        return linear_chunked(d) && tokens ? kda::launch_linear_chunk(p, which, s)
                                           : kda::launch_linear_walk(p, which, s);
    };
    if (L.seg_tokens == 0) {
        e = pass(kda::LinearPass::kWhole);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_linear_fwd launch");
    }
    p.seg_tokens = L.seg_tokens;
    // Packed sequences little longer than a segment stay whole: the states before a second segment
    // cost more than it gains (three of 56 chunks, 32 heads, segments of 46: 166 us, 204 cut).
    p.whole_tokens = cu_seqlens && linear_chunked(d) ? L.seg_tokens / 5 * 8 : L.seg_tokens;
    p.slots = L.slots;
    p.seg_state = static_cast<float*>(workspace);
    p.seg_decay = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.decay);
    const bool chunked = linear_chunked(d);
    if (cu_seqlens && !chunked && (e = kda::launch_linear_check(p, s)) != cudaSuccess)
        return cuda_fail(e, "kda_linear_fwd cu_seqlens check");
    if ((e = pass(kda::LinearPass::kStates)) != cudaSuccess)
        return cuda_fail(e, "kda_linear_fwd launch");
    p.seg_ready = !chunked || d->T > kChainedSegments * L.seg_tokens;
    if ((p.seg_ready && (e = kda::launch_linear_combine(p, s)) != cudaSuccess) ||
        (e = pass(kda::LinearPass::kOutputs)) != cudaSuccess)
        return cuda_fail(e, "kda_linear_fwd launch");
    return KDA_OK;
}

kda_status_t kda_linear_decode(int N, int T, int H, int Hk, int dk, int dv, kda_dtype_t dtype,
                               kda_gate_t gate, const void* q, const void* k, const void* v,
                               const float* log_g, float* S_inout, void* o, kda_stream_t stream) {
    t_last_error[0] = 0;
    if (N < 0) return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d", N);
    // N sequences of T tokens; N = 0 is checked like N = 1
    const kda_linear_desc_t d{std::max(N, 1), T, H, Hk, dk, dv, std::max(N, 1), dtype, gate};
    kda_status_t st = check_linear_desc(&d, false);
    if (st != KDA_OK) return st;
    const bool any = N > 0 && T > 0;
    if ((st = check_ptr(q, "q", any)) || (st = check_ptr(k, "k", any)) ||
        (st = check_ptr(v, "v", any)) || (st = check_ptr(log_g, "log_g", any)) ||
        (st = check_ptr(S_inout, "S_inout", any)) || (st = check_ptr(o, "o", any)))
        return st;
    if (!any) return KDA_OK;
    const size_t esz = dtype == KDA_BF16 ? 2 : 4, rows = (size_t)N * T;
    const size_t qk_bytes = rows * Hk * dk * esz, v_bytes = rows * H * dv * esz;
    const size_t s_bytes = (size_t)N * H * dk * dv * sizeof(float);
    const size_t gates = gate == KDA_GATE_HEAD ? H : rows * H;
    if ((st = check_apart({{S_inout, s_bytes, "S_inout"}, {o, v_bytes, "o"}, {q, qk_bytes, "q"},
                          {k, qk_bytes, "k"}, {v, v_bytes, "v"}, {log_g, gates * 4, "log_g"}}, 2)) !=
        KDA_OK)
        return st;
    kda::LinearParams p = linear_params(&d);
    p.q = q; p.k = k; p.v = v; p.log_g = log_g; p.o = o;
    p.h0 = p.hT = S_inout;   // each thread writes what it alone has read
    if ((st = device_error_word(&p.err)) != KDA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = kda::linear_decode_takes(T, dk, dv)
                              ? kda::launch_linear_decode(p, s)
                              : kda::launch_linear_walk(p, kda::LinearPass::kWhole, s);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_linear_decode launch");
}

// ------------------------------------------------------------------ trees of drafted tokens

static kda_status_t check_tree_sizes(int N, int H, int T, kda_dtype_t dtype) {
    if (N < 0 || H < 1 || T < 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d H=%d T=%d", N, H, T);
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    // (a TMA row coordinate counts 128 state rows per sequence and head)
    if ((int64_t)N * H * 128 > 0x7fffffffLL || (int64_t)N * T * H > (int64_t)1 << 40)
        return fail(KDA_ERR_INVALID_ARG, "problem too large");
    return KDA_OK;
}

kda_status_t kda_decode_tree(int N, int H, int T, kda_dtype_t dtype, const void* q, const void* k,
                             const void* v, const float* log_g, const void* beta,
                             const int32_t* parents, const float* S, void* o, int clear_absent,
                             kda_stream_t stream) {
    t_last_error[0] = 0;
    kda_status_t st = check_tree_sizes(N, H, T, dtype);
    if (st != KDA_OK) return st;
    if (T > KDA_TREE_MAX_NODES)
        return fail(KDA_ERR_UNSUPPORTED, "%d nodes (at most %d)", T, KDA_TREE_MAX_NODES);
    const bool any = N > 0 && T > 0;
    if ((st = check_ptr(q, "q", any)) || (st = check_ptr(k, "k", any)) ||
        (st = check_ptr(v, "v", any)) || (st = check_ptr(log_g, "log_g", any)) ||
        (st = check_ptr(beta, "beta", any)) || (st = check_ptr(parents, "parents", any)) ||
        (st = check_ptr(S, "S", any)) || (st = check_ptr(o, "o", any)))
        return st;
    if (!any) return KDA_OK;
    const size_t rows = (size_t)N * T * H, x = rows * 128 * (dtype == KDA_BF16 ? 2 : 4);
    if ((st = check_apart({{o, x, "o"}, {q, x, "q"}, {k, x, "k"}, {v, x, "v"},
                          {log_g, rows * 512, "log_g"}, {beta, x / 128, "beta"},
                          {parents, (size_t)N * T * 4, "parents"},
                          {S, (size_t)N * H * 65536, "S"}}, 1)) !=
        KDA_OK)
        return st;
    kda::TreeParams p{q, k, v, log_g, beta, parents, const_cast<float*>(S), o, N, H, T, 0,
                      dtype == KDA_BF16, nullptr, clear_absent != 0};
    if ((st = device_error_word(&p.err)) != KDA_OK) return st;
    const cudaError_t e = kda::launch_decode_tree(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_decode_tree launch");
}

kda_status_t kda_commit_path(int N, int H, int T, int A, kda_dtype_t dtype, const void* k,
                             const void* v, const float* log_g, const void* beta,
                             const int32_t* path, float* S_inout, kda_stream_t stream) {
    t_last_error[0] = 0;
    kda_status_t st = check_tree_sizes(N, H, T, dtype);
    if (st != KDA_OK) return st;
    if (A < 0) return fail(KDA_ERR_INVALID_ARG, "bad sizes A=%d", A);
    const bool any = N > 0 && A > 0, read = any && T > 0;   // (T = 0: no path may name a row)
    if ((st = check_ptr(k, "k", read)) || (st = check_ptr(v, "v", read)) ||
        (st = check_ptr(log_g, "log_g", read)) || (st = check_ptr(beta, "beta", read)) ||
        (st = check_ptr(path, "path", any)) || (st = check_ptr(S_inout, "S_inout", any)))
        return st;
    if (!any) return KDA_OK;
    const size_t rows = (size_t)N * T * H, x = rows * 128 * (dtype == KDA_BF16 ? 2 : 4);
    if ((st = check_apart({{S_inout, (size_t)N * H * 65536, "S_inout"}, {k, x, "k"}, {v, x, "v"},
                          {log_g, rows * 512, "log_g"}, {beta, x / 128, "beta"},
                          {path, (size_t)N * A * 4, "path"}}, 1)) !=
        KDA_OK)
        return st;
    kda::TreeParams p{nullptr, k, v, log_g, beta, path, S_inout, nullptr, N, H, T, A,
                      dtype == KDA_BF16, nullptr, false};
    if ((st = device_error_word(&p.err)) != KDA_OK) return st;
    const cudaError_t e = kda::launch_commit_path(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_commit_path launch");
}

// ------------------------------------------------------------------ pages of states

kda_status_t kda_state_copy(void* pool, int layers, int pages, long long page_bytes,
                            const int32_t* src, const int32_t* dst, int n, kda_stream_t stream) {
    t_last_error[0] = 0;
    if (layers < 0 || pages < 0 || n < 0 || page_bytes < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes layers=%d pages=%d page_bytes=%lld n=%d",
                    layers, pages, page_bytes, n);
    if (page_bytes % 16)
        return fail(KDA_ERR_UNSUPPORTED, "page_bytes %lld is not a multiple of 16", page_bytes);
    kda_status_t st;
    const bool any = layers > 0 && n > 0;
    if ((st = check_ptr(pool, "pool", any && pages > 0)) || (st = check_ptr(src, "src", any)) ||
        (st = check_ptr(dst, "dst", any)))
        return st;
    if (!any) return KDA_OK;
    const size_t bytes = (size_t)layers * pages * page_bytes, list = (size_t)n * 4;
    if (overlap(pool, bytes, src, list) || overlap(pool, bytes, dst, list))
        return fail(KDA_ERR_INVALID_ARG, "the pool overlaps src or dst");
    unsigned* err = nullptr;
    if ((st = device_error_word(&err)) != KDA_OK) return st;
    const cudaError_t e = kda::launch_page_copy(pool, src, dst, n, layers, pages, page_bytes, err,
                                                reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_state_copy launch");
}

kda_status_t kda_get_device_error(kda_stream_t stream) {
    t_last_error[0] = 0;
    unsigned* err = nullptr;
    kda_status_t st = device_error_word(&err);
    if (st != KDA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    unsigned host = 0;
    cudaError_t e = cudaMemcpyAsync(&host, err, sizeof(host), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
    if (host != 0) {
        const unsigned zero = 0;
        e = cudaMemcpyAsync(err, &zero, sizeof(zero), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return cuda_fail(e, "clearing the device error word");
        return fail(static_cast<kda_status_t>(host), "device reported: %s",
                    kda_status_string(static_cast<kda_status_t>(host)));
    }
    return KDA_OK;
}

}  // extern "C"
