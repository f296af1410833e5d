// Linear attention with a scalar decay for each head, on CUDA cores: the per-token walk and the
// kernel that chains segments.
//
// The walk follows the recurrence token by token,
//     S <- g S + k v^T,   o = S^T q,   g = exp(log_g),
// everything in fp32. It serves fp32 inputs and the sizes the tensor-core kernel does not take.
//
// Work split. Column j of S meets only column j of v, so one warp owns kNC value columns of one
// (segment, head), with the dk rows spread over the lanes (lane l holds rows l, l + 32, ...). Per
// token a lane does 2 fp32 operations per state element and one for the read-out; the read-out's
// sum over the rows halves its columns at each butterfly step (4 + 2 + 1 + 1 + 1 shuffles for 8
// columns). Bound: fp32 issue.

#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kNC = 8;             // value columns per warp
constexpr int kWarpsPerBlock = 4;

// Sum of x[i] over the warp's lanes; lane l returns the sum of column l / 4.
__device__ __forceinline__ float reduce8(const float (&x)[kNC], int lane) {
    float y[4], z[2], w;
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float keep = b4 ? x[4 + i] : x[i], give = b4 ? x[i] : x[4 + i];
        y[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = b3 ? y[2 + i] : y[i], give = b3 ? y[i] : y[2 + i];
        z[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    w = (b2 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, b2 ? z[0] : z[1], 4);
    w += __shfl_xor_sync(0xffffffffu, w, 2);
    w += __shfl_xor_sync(0xffffffffu, w, 1);
    return w;
}

template <typename Tin, int RPL>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
linear_walk_kernel(const LinearParams p, const LinearPass pass, const int col_groups) {
    const Tin* __restrict__ q = static_cast<const Tin*>(p.q);
    const Tin* __restrict__ k = static_cast<const Tin*>(p.k);
    const Tin* __restrict__ v = static_cast<const Tin*>(p.v);
    Tin* __restrict__ o = static_cast<Tin*>(p.o);
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
    if (warp >= (int64_t)p.slots * p.H * col_groups) return;
    const int cg = (int)(warp % col_groups);
    const int h = (int)(warp / col_groups % p.H);
    const int g = (int)(warp / col_groups / p.H);
    LinearSlot sl;
    if (!linear_slot(p, g, &sl)) return;
    const bool states = pass == LinearPass::kStates;
    if (states && sl.last) return;

    const int dk = p.dk, dv = p.dv, j0 = cg * kNC;
    const int hk = h / (p.H / p.Hk);
    const size_t unit = (size_t)dk * dv;
    const float* init = nullptr;
    if (!states)
        init = sl.seg > 0 ? p.seg_state + ((size_t)g * p.H + h) * unit
                          : (p.h0 ? p.h0 + ((size_t)sl.n * p.H + h) * unit : nullptr);
    float S[RPL][kNC];
#pragma unroll
    for (int r = 0; r < RPL; ++r) {
        const int c = lane + 32 * r;
#pragma unroll
        for (int i = 0; i < kNC; ++i)
            S[r][i] = (init && c < dk && j0 + i < dv) ? init[(size_t)c * dv + j0 + i] : 0.f;
    }

    float kr[RPL], qr[RPL], vr[kNC], lg = 0.f;
    auto fetch = [&](int64_t t, float* kk, float* qq, float* vv, float& ll) {
        const int64_t qk = (t * p.Hk + hk) * (int64_t)dk;
        const int64_t vo = (t * p.H + h) * (int64_t)dv;
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            const int c = lane + 32 * r;
            kk[r] = c < dk ? load_elem(k, qk + c) : 0.f;
            qq[r] = c < dk && !states ? load_elem(q, qk + c) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kNC; ++i) vv[i] = (j0 + i < dv) ? load_elem(v, vo + j0 + i) : 0.f;
        ll = p.log_g[p.gate_head ? h : t * p.H + h];
    };
    if (sl.begin < sl.end) fetch(sl.begin, kr, qr, vr, lg);
    float total = 0.f;

    for (int64_t t = sl.begin; t < sl.end; ++t) {
        float kn[RPL], qn[RPL], vn[kNC], ln = 0.f;
        if (t + 1 < sl.end) fetch(t + 1, kn, qn, vn, ln);
        const float gt = expf(lg);
        total += lg;
        float acc[kNC];
#pragma unroll
        for (int i = 0; i < kNC; ++i) acc[i] = 0.f;
#pragma unroll
        for (int r = 0; r < RPL; ++r)
#pragma unroll
            for (int i = 0; i < kNC; ++i) {
                S[r][i] = fmaf(kr[r], vr[i], gt * S[r][i]);
                acc[i] = fmaf(qr[r], S[r][i], acc[i]);
            }
        if (!states) {
            const float oi = reduce8(acc, lane);
            const int j = j0 + (lane >> 2);
            if ((lane & 3) == 0 && j < dv) store_elem(o, (t * p.H + h) * (int64_t)dv + j, oi);
        }
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            kr[r] = kn[r];
            qr[r] = qn[r];
        }
#pragma unroll
        for (int i = 0; i < kNC; ++i) vr[i] = vn[i];
        lg = ln;
    }

    float* out = states ? p.seg_state + ((size_t)g * p.H + h) * unit
                        : (sl.last && p.hT ? p.hT + ((size_t)sl.n * p.H + h) * unit : nullptr);
    if (out) {
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            const int c = lane + 32 * r;
            if (c >= dk) continue;
#pragma unroll
            for (int i = 0; i < kNC; ++i)
                if (j0 + i < dv) out[(size_t)c * dv + j0 + i] = S[r][i];
        }
    }
    if (states && cg == 0 && lane == 0) p.seg_decay[(size_t)g * p.H + h] = expf(total);
}

// The state before segment s of a sequence is d_{s-1} (state before s - 1) + B_{s-1}; the B of a
// slot gives way to its initial state. One thread per state element; the loads of kAhead segments
// do not wait for the chain.
__global__ void __launch_bounds__(256)
linear_combine_kernel(const LinearParams p) {
    constexpr int kAhead = 8;
    const int unit = p.dk * p.dv;
    const int e = blockIdx.x * 256 + threadIdx.x;
    const int n = blockIdx.z, h = blockIdx.y;
    const int L = p.seg_tokens;
    long long len = p.T, first;
    if (p.cu_seqlens) {
        const long long t0 = p.cu_seqlens[n], t1 = p.cu_seqlens[n + 1];
        if (t0 < 0 || t1 < t0 || t1 > p.T) return;   // recorded by the other launches
        len = t1 - t0;
        first = t0 / L + n;
    } else {
        first = (long long)n * max(1, (p.T + L - 1) / L);
    }
    const int segs = (int)((len + L - 1) / L);
    if (segs < 2 || e >= unit) return;
    float S = p.h0 ? p.h0[((size_t)n * p.H + h) * unit + e] : 0.f;
    float* st = p.seg_state + ((size_t)first * p.H + h) * unit + e;
    const float* dc = p.seg_decay + (size_t)first * p.H + h;
    const size_t step = (size_t)p.H * unit;
    float carry = st[0];
    for (int s0 = 0; s0 + 1 < segs; s0 += kAhead) {   // reads B of s0 .. s0 + kAhead first
        float b[kAhead], d[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s0 + i + 1 < segs) {
                b[i] = i == 0 ? carry : st[(size_t)(s0 + i) * step];
                d[i] = dc[(size_t)(s0 + i) * p.H];
            }
        if (s0 + kAhead + 1 < segs) carry = st[(size_t)(s0 + kAhead) * step];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s0 + i + 1 < segs) {
                S = fmaf(d[i], S, b[i]);
                st[(size_t)(s0 + i + 1) * step] = S;
            }
    }
}

__global__ void linear_check_kernel(const int32_t* __restrict__ cu, int N, int T, unsigned* err) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i > N) return;
    const int c = cu[i];
    if ((i == 0 && c != 0) || (i == N && c != T) || (i < N && cu[i + 1] < c))
        set_device_error(err, DEV_BAD_SEQLENS);
}

template <typename Tin, int RPL>
cudaError_t launch_walk_typed(const LinearParams& p, LinearPass pass, cudaStream_t stream) {
    const int col_groups = (p.dv + kNC - 1) / kNC;
    const int64_t warps = (int64_t)p.slots * p.H * col_groups;
    const int64_t blocks = (warps + kWarpsPerBlock - 1) / kWarpsPerBlock;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    linear_walk_kernel<Tin, RPL>
        <<<(unsigned)blocks, kWarpsPerBlock * 32, 0, stream>>>(p, pass, col_groups);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_walk_rpl(const LinearParams& p, LinearPass pass, cudaStream_t stream) {
    if (p.dk <= 32) return launch_walk_typed<Tin, 1>(p, pass, stream);
    if (p.dk <= 64) return launch_walk_typed<Tin, 2>(p, pass, stream);
    if (p.dk <= 128) return launch_walk_typed<Tin, 4>(p, pass, stream);
    return launch_walk_typed<Tin, 8>(p, pass, stream);
}

}  // namespace

cudaError_t launch_linear_walk(const LinearParams& p, LinearPass pass, cudaStream_t stream) {
    return p.bf16 ? launch_walk_rpl<__nv_bfloat16>(p, pass, stream)
                  : launch_walk_rpl<float>(p, pass, stream);
}

cudaError_t launch_linear_combine(const LinearParams& p, cudaStream_t stream) {
    if (p.N > 65535 || p.H > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((p.dk * p.dv + 255) / 256, p.H, p.N);
    linear_combine_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_linear_check(const LinearParams& p, cudaStream_t stream) {
    linear_check_kernel<<<p.N / 256 + 1, 256, 0, stream>>>(p.cu_seqlens, p.N, p.T, p.err);
    return cudaGetLastError();
}

}  // namespace kda
