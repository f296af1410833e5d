// Linear attention for one or a few tokens of many sequences, the state in place.
//
// One 256-thread block per (sequence, head) holds the whole state in registers between one
// streaming read and one streaming write: thread (r, c) has columns 4 c .. 4 c + 3 of rows r, r + R,
// r + 2 R, ... (R = 256 / (dv / 4) row groups), so a row's dv columns are consecutive lanes. Per
// token S <- g S + k v^T needs nothing from other threads; the read-out S^T q is summed over a
// thread's rows in registers and over the row groups in shared memory. Up to kGroup tokens' q, k
// and gates are staged at once. Bound: HBM (the state read once and written once, whatever T).
//
// Against one warp per 8 columns (the walk, 32-byte pieces of rows): 256 sequences x 32 heads x
// 128 x 128, one bf16 token, 170 us (0.97 of the measured copy rate) against 1024.

#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 8;       // tokens staged at once
constexpr int kMaxRows = 16;    // state rows per thread

__device__ __forceinline__ float4 load4(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// NR: rows per thread (dk <= NR * row groups).
template <typename Tin, int NR>
__global__ void __launch_bounds__(kThreads, 2)
linear_decode_kernel(const __grid_constant__ LinearParams p, float* S) {
    extern __shared__ __align__(16) float sm[];   // q, k [kGroup][dk]; sums [2][R][dv]
    __shared__ float s_g[kGroup];
    const int tid = threadIdx.x, dk = p.dk, dv = p.dv, T = p.T;
    const int cols = dv / 4, R = kThreads / cols;
    const int r0 = tid / cols, c = 4 * (tid % cols);
    const bool mine = r0 < R;
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
    float *s_q = sm, *s_k = s_q + kGroup * dk, *s_o = s_k + kGroup * dk;
    const Tin* q = static_cast<const Tin*>(p.q);
    const Tin* k = static_cast<const Tin*>(p.k);
    const Tin* v = static_cast<const Tin*>(p.v);
    Tin* o = static_cast<Tin*>(p.o);

    float* at = S + (size_t)blockIdx.x * dk * dv + (size_t)r0 * dv + c;
    const size_t step = (size_t)R * dv;
    float4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        if (mine && r0 + i * R < dk) s[i] = __ldcs(reinterpret_cast<const float4*>(at + i * step));

    for (int t0 = 0; t0 < T; t0 += kGroup) {
        const int m = min(kGroup, T - t0);
        for (int i = tid; i < m * dk; i += kThreads) {
            const int t = i / dk, e = i - t * dk;
            const int64_t x = (((int64_t)n * T + t0 + t) * p.Hk + hk) * dk + e;
            s_q[i] = load_elem(q, x);
            s_k[i] = load_elem(k, x);
        }
        if (tid < m)
            s_g[tid] = expf(p.log_g[p.gate_head ? h : ((int64_t)n * T + t0 + tid) * p.H + h]);
        __syncthreads();
        for (int t = 0; t < m; ++t) {
            const int64_t row = (((int64_t)n * T + t0 + t) * p.H + h) * dv;
            float* sum = s_o + (t & 1) * R * dv;
            if (mine) {
                const float4 x = load4(v + row + c);
                const float g = s_g[t];
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int r = r0 + i * R;
                    if (r < dk) {
                        const float kr = s_k[t * dk + r], qr = s_q[t * dk + r];
                        s[i].x = fmaf(kr, x.x, g * s[i].x), s[i].y = fmaf(kr, x.y, g * s[i].y);
                        s[i].z = fmaf(kr, x.z, g * s[i].z), s[i].w = fmaf(kr, x.w, g * s[i].w);
                        y.x = fmaf(qr, s[i].x, y.x), y.y = fmaf(qr, s[i].y, y.y);
                        y.z = fmaf(qr, s[i].z, y.z), y.w = fmaf(qr, s[i].w, y.w);
                        if (t0 + t + 1 == T)
                            __stcs(reinterpret_cast<float4*>(at + i * step), s[i]);
                    }
                }
                *reinterpret_cast<float4*>(sum + r0 * dv + c) = y;
            }
            __syncthreads();
            if (tid < dv) {
                float y = 0.f;
                for (int r = 0; r < R; ++r) y += sum[r * dv + tid];
                store_elem(o, row + tid, y);
            }
        }
        __syncthreads();
    }
}

template <typename Tin, int NR>
cudaError_t launch(const LinearParams& p, cudaStream_t stream) {
    const int R = kThreads / (p.dv / 4);
    const size_t bytes = (size_t)(2 * kGroup * p.dk + 2 * R * p.dv) * sizeof(float);
    linear_decode_kernel<Tin, NR>
        <<<(unsigned)(p.N * p.H), kThreads, bytes, stream>>>(p, p.hT);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_rows(const LinearParams& p, cudaStream_t stream) {
    const int R = kThreads / (p.dv / 4), rows = (p.dk + R - 1) / R;
    if (rows <= 4) return launch<Tin, 4>(p, stream);
    if (rows <= 8) return launch<Tin, 8>(p, stream);
    return launch<Tin, kMaxRows>(p, stream);
}

}  // namespace

// A thread's rows fit its registers, and columns come in fours. T above 64 goes to the walk, whose
// tokens cost no block-wide barrier.
bool linear_decode_takes(int T, int dk, int dv) {
    return T <= 64 && dv % 4 == 0 && dk <= kMaxRows * (kThreads / (dv / 4));
}

cudaError_t launch_linear_decode(const LinearParams& p, cudaStream_t stream) {
    return p.bf16 ? launch_rows<__nv_bfloat16>(p, stream) : launch_rows<float>(p, stream);
}

}  // namespace kda
