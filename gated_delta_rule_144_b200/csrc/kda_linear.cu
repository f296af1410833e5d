// Linear attention with a scalar decay for each head, on CUDA cores: the per-token walk and the
// kernel that chains segments.
//
// The walk follows the recurrence token by token,
//     S <- g S + k v^T,   o = S^T q,   g = exp(log_g),
// everything in fp32. It serves fp32 inputs and the sizes the tensor-core kernel does not take.
//
// Work split. Column j of S meets only column j of v, so one warp owns NC value columns of one
// (segment, head), with the dk rows spread over the lanes (lane l holds rows l, l + 32, ...); four
// warps form a block. The block stages kTokens tokens' rows in shared memory while it works on the
// kTokens before them: a token's arithmetic is shorter than a load's time. The state pairs its
// columns, so that one two-lane instruction works on both. The read-out's sum over the rows halves
// its columns at each butterfly step (8 + 4 + 2 + 1 + 1 shuffles for 16 columns). A segment's own
// contribution (no read-out) is taken from its last token back, with the product of the gates
// behind as a running factor of k: one multiply-add per element instead of two. Bound: issue.
// (With the next token's rows fetched into registers instead, a token took a load's time: one
// prompt of 4096 tokens x 16 heads in fp32 782 us; now 297 to 301.)

#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kWarpsPerBlock = 4, kBlock = 32 * kWarpsPerBlock;
constexpr int kTokens = 16;   // staged at once

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Sum of x[i] over the warp's lanes; lane l returns the sum of column l / (32 / NC).
template <int NC>
__device__ __forceinline__ float reduce_columns(float (&x)[NC], int lane) {
    int off = 16;
#pragma unroll
    for (int n = NC / 2; n > 0; n /= 2, off /= 2) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i)
            x[i] = (up ? x[n + i] : x[i]) +
                   __shfl_xor_sync(0xffffffffu, up ? x[i] : x[n + i], off);
    }
    float y = x[0];
#pragma unroll
    for (; off > 0; off /= 2) y += __shfl_xor_sync(0xffffffffu, y, off);
    return y;
}

__device__ __forceinline__ float2 pair_at(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 pair_at(const __nv_bfloat16* p) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

template <typename Tin, int RPL, int NC>
struct WalkSmem {
    static constexpr int kRow = 32 * RPL, kCols = NC * kWarpsPerBlock;
    Tin q[2][kTokens][kRow], k[2][kTokens][kRow], v[2][kTokens][kCols];
    float g[2][kTokens];
};

// kEvery: dk is all of the 32 RPL rows. Else the lanes without a row take no part in a token's
// products (with k = q = 0 there an infinite v would give 0 x inf = NaN to every output), which
// costs 7 to 18 % (one fp32 prompt of 4096 tokens x 16 heads 317 us, 296 without the test).
template <typename Tin, int RPL, int NC, bool kStates, bool kEvery>
__global__ void __launch_bounds__(kBlock)
linear_walk_kernel(const __grid_constant__ LinearParams p, const int col_groups) {
    using Smem = WalkSmem<Tin, RPL, NC>;
    extern __shared__ __align__(16) uint8_t raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const Tin* __restrict__ q = static_cast<const Tin*>(p.q);
    const Tin* __restrict__ k = static_cast<const Tin*>(p.k);
    const Tin* __restrict__ v = static_cast<const Tin*>(p.v);
    Tin* __restrict__ o = static_cast<Tin*>(p.o);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cg = blockIdx.x % col_groups;
    const int h = blockIdx.x / col_groups % p.H, g = blockIdx.x / col_groups / p.H;
    LinearSlot sl;
    if (!linear_slot(p, g, &sl)) return;
    if (kStates && sl.last) return;

    const int dk = p.dk, dv = p.dv;
    const int b0 = cg * Smem::kCols, bcols = min(Smem::kCols, dv - b0);   // the block's columns
    const int j0 = b0 + warp * NC, cols = max(0, min(NC, dv - j0));       // the warp's
    const bool whole = cols == NC && dv % 4 == 0;   // (16-byte pieces of state rows)
    const int hk = h / (p.H / p.Hk);
    const size_t unit = (size_t)dk * dv;
    const float* init = nullptr;
    if (!kStates)
        init = sl.seg > 0 ? p.seg_state + ((size_t)g * p.H + h) * unit
                          : (p.h0 ? p.h0 + ((size_t)sl.n * p.H + h) * unit : nullptr);
    float2 S[RPL][NC / 2];
#pragma unroll
    for (int r = 0; r < RPL; ++r) {
        const int c = lane + 32 * r;
        const float* at = init + (size_t)c * dv + j0;
        if (whole && init && c < dk) {
#pragma unroll
            for (int i = 0; i < NC / 2; i += 2) {
                const float4 x = *reinterpret_cast<const float4*>(at + 2 * i);
                S[r][i] = make_float2(x.x, x.y);
                S[r][i + 1] = make_float2(x.z, x.w);
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < NC / 2; ++i)
            S[r][i] = make_float2(init && c < dk && 2 * i < cols ? at[2 * i] : 0.f,
                                  init && c < dk && 2 * i + 1 < cols ? at[2 * i + 1] : 0.f);
    }

    // rows of tokens [t0, t0 + m) into buffer b: in 16-byte pieces where every row starts and ends
    // on one
    const bool pieces = dk * sizeof(Tin) % 16 == 0 && dv * sizeof(Tin) % 16 == 0;
    auto rows = [&](Tin* to, int ld, const Tin* from, int64_t stride, int width, int m) {
        if (pieces) {
            constexpr int kEl = 16 / sizeof(Tin);
            const int per = width / kEl;
            for (int i = tid; i < m * per; i += kBlock) {
                const int t = i / per, e = (i - t * per) * kEl;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(to + t * ld + e)),
                             "l"(from + t * stride + e)
                             : "memory");
            }
        } else {
            for (int i = tid; i < m * width; i += kBlock) {
                const int t = i / width, e = i - t * width;
                to[t * ld + e] = from[t * stride + e];
            }
        }
    };
    auto stage = [&](int b, int64_t t0, int m) {
        rows(sm.k[b][0], Smem::kRow, k + (t0 * p.Hk + hk) * dk, (int64_t)p.Hk * dk, dk, m);
        if (!kStates)
            rows(sm.q[b][0], Smem::kRow, q + (t0 * p.Hk + hk) * dk, (int64_t)p.Hk * dk, dk, m);
        rows(sm.v[b][0], Smem::kCols, v + (t0 * p.H + h) * dv + b0, (int64_t)p.H * dv, bcols, m);
        if (tid < m) sm.g[b][tid] = expf(p.log_g[p.gate_head ? h : (t0 + tid) * p.H + h]);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // blocks of tokens in order, or (kStates) from the last back
    const int64_t n = sl.end - sl.begin;
    const int nblocks = (int)((n + kTokens - 1) / kTokens);
    auto first = [&](int i) {
        return sl.begin + (int64_t)(kStates ? nblocks - 1 - i : i) * kTokens;
    };
    auto count = [&](int i) { return (int)min((long long)kTokens, (long long)(sl.end - first(i))); };
    if (nblocks > 0) stage(0, first(0), count(0));
    float behind = 1.f;   // kStates: the product of the gates behind the token

#pragma unroll 1
    for (int i = 0; i < nblocks; ++i) {
        const int b = i & 1, m = count(i);
        const int64_t t0 = first(i);
        if (i + 1 < nblocks) stage(b ^ 1, first(i + 1), count(i + 1));
        if (i + 1 < nblocks) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
#pragma unroll 2
        for (int x = 0; x < m; ++x) {
            const int t = kStates ? m - 1 - x : x;
            const float gt = sm.g[b][t];
            float2 vr[NC / 2];
#pragma unroll
            for (int e = 0; e < NC / 2; ++e) vr[e] = pair_at(&sm.v[b][t][warp * NC + 2 * e]);
            if (kStates) {
#pragma unroll
                for (int r = 0; r < RPL; ++r) {
                    const float kb = behind * load_elem(sm.k[b][t], lane + 32 * r);
                    const float2 k2 = make_float2(kb, kb);
#pragma unroll
                    for (int e = 0; e < NC / 2; ++e) S[r][e] = fma2(k2, vr[e], S[r][e]);
                }
                behind *= gt;
                continue;
            }
            const float2 g2 = make_float2(gt, gt);
            float2 acc[NC / 2];
#pragma unroll
            for (int e = 0; e < NC / 2; ++e) acc[e] = make_float2(0.f, 0.f);
#pragma unroll
            for (int r = 0; r < RPL; ++r) {
                const int c = lane + 32 * r;
                if (!kEvery && c >= dk) continue;
                const float kr = load_elem(sm.k[b][t], c), qr = load_elem(sm.q[b][t], c);
                const float2 k2 = make_float2(kr, kr), q2 = make_float2(qr, qr);
#pragma unroll
                for (int e = 0; e < NC / 2; ++e) {
                    S[r][e] = fma2(k2, vr[e], mul2(g2, S[r][e]));
                    acc[e] = fma2(q2, S[r][e], acc[e]);
                }
            }
            float y[NC];
#pragma unroll
            for (int e = 0; e < NC / 2; ++e) y[2 * e] = acc[e].x, y[2 * e + 1] = acc[e].y;
            const float sum = reduce_columns<NC>(y, lane);
            constexpr int kLanes = 32 / NC;   // per column
            const int j = lane / kLanes;
            if (lane % kLanes == 0 && j < cols)
                store_elem(o, ((t0 + t) * p.H + h) * (int64_t)dv + j0 + j, sum);
        }
        __syncthreads();
    }

    float* out = kStates ? p.seg_state + ((size_t)g * p.H + h) * unit
                         : (sl.last && p.hT ? p.hT + ((size_t)sl.n * p.H + h) * unit : nullptr);
    if (out) {
#pragma unroll
        for (int r = 0; r < RPL; ++r) {
            const int c = lane + 32 * r;
            if (c >= dk) continue;
            float* to = out + (size_t)c * dv + j0;
            if (whole) {
#pragma unroll
                for (int i = 0; i < NC / 2; i += 2)
                    *reinterpret_cast<float4*>(to + 2 * i) =
                        make_float4(S[r][i].x, S[r][i].y, S[r][i + 1].x, S[r][i + 1].y);
                continue;
            }
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                if (2 * i < cols) to[2 * i] = S[r][i].x;
                if (2 * i + 1 < cols) to[2 * i + 1] = S[r][i].y;
            }
        }
    }
    if (kStates && cg == 0 && tid == 0) p.seg_decay[(size_t)g * p.H + h] = behind;
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
    const int segs = len <= p.whole_tokens ? 1 : (int)((len + L - 1) / L);
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

PerDevice g_walk_setup[2][4][3];   // by type, rows per lane and form

template <typename Tin, int RPL, int NC, bool kStates, bool kEvery>
cudaError_t launch_walk_typed(const LinearParams& p, PerDevice& setup, cudaStream_t stream) {
    using Smem = WalkSmem<Tin, RPL, NC>;
    const cudaError_t e = setup.run([](int) {
        return cudaFuncSetAttribute(linear_walk_kernel<Tin, RPL, NC, kStates, kEvery>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(Smem));
    });
    if (e != cudaSuccess) return e;
    const int col_groups = (p.dv + Smem::kCols - 1) / Smem::kCols;
    const int64_t blocks = (int64_t)p.slots * p.H * col_groups;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    linear_walk_kernel<Tin, RPL, NC, kStates, kEvery>
        <<<(unsigned)blocks, kBlock, sizeof(Smem), stream>>>(p, col_groups);
    return cudaGetLastError();
}

template <typename Tin, int RPL, int NC>
cudaError_t launch_walk_pass(const LinearParams& p, LinearPass pass, int rows,
                             cudaStream_t stream) {
    PerDevice(&setup)[3] = g_walk_setup[p.bf16][rows];
    if (pass == LinearPass::kStates)   // (rows behind dk are not stored)
        return launch_walk_typed<Tin, RPL, NC, true, true>(p, setup[0], stream);
    return p.dk == 32 * RPL ? launch_walk_typed<Tin, RPL, NC, false, true>(p, setup[1], stream)
                            : launch_walk_typed<Tin, RPL, NC, false, false>(p, setup[2], stream);
}

template <typename Tin>
cudaError_t launch_walk_rpl(const LinearParams& p, LinearPass pass, cudaStream_t stream) {
    if (p.dk <= 32) return launch_walk_pass<Tin, 1, 16>(p, pass, 0, stream);
    if (p.dk <= 64) return launch_walk_pass<Tin, 2, 16>(p, pass, 1, stream);
    if (p.dk <= 128) return launch_walk_pass<Tin, 4, 16>(p, pass, 2, stream);
    return launch_walk_pass<Tin, 8, 8>(p, pass, 3, stream);   // (the same registers of state)
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
