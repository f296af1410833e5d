// A tree of drafted tokens against a decode state (dk = dv = 128), and the commit of its accepted
// path.
//
// Every node i of the tree has the gated delta rule's state after its own path from the root. With
// d_ij the product, per key channel, of the gates of the nodes from i up to but not including its
// ancestor j, and d_i the product over i's whole path,
//     u_i = beta_i (v_i - (k_i d_i)^T S - sum_{j above i} (k_i . d_ij k_j) u_j)
//     o_i = (q_i d_i)^T S + sum_{j above i, and i} (q_i . d_ij k_j) u_j
// so the state is read once, whatever the number of nodes, and only u (one row of 128 values per
// node) follows the tree's order. A path's rows are a tree without branches, and the state after
// its last row e is diag(d_e) S + sum_j (d_ej k_j) u_j^T.
//
// One 256-thread block per (sequence, head); two blocks fit an SM. Phases:
//   load     warp w issues the loads of value columns [16 w, 16 w + 16) of S straight into the
//            registers that the products below read (64 per thread, all in flight at once); the
//            rows of k and the gates go to shared memory.
//   walk     a warp per node i walks i's ancestors with d_ij in registers (4 channels per lane):
//            only products of gates <= 1 appear, so no gate, -inf included, is out of range. It
//            leaves the two scalars per pair and the rows k_i d_i, q_i d_i.
//   product  [k d; q d] S on the tensor cores (warp-level tf32 products: 16 x 8 x 8). The tree of
//            bf16 rows uses one tf32 product (its operands lose at most 2^-11, below the bf16
//            output's 2^-8); fp32 rows, and the commit, whose state stays fp32, split both
//            operands into a tf32 part and a tf32 remainder and sum three products (2^-21).
//   solve    a thread per value column substitutes forward through the nodes, 16 at a time in
//            registers, and writes o.
//   update   (commit) S = d_e S + sum_j (d_ej k_j) u_j^T in the same registers, then stored.
// Bound: HBM (64 KiB of state per block, twice for the commit).

#include "kda_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

using sm100::mma_tf32_16x8x8;

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kFrag = 132;   // floats per (16 rows, 8 channels) block of the left operand, padded:
                             // consecutive blocks start four banks apart
constexpr int kXs = 144;     // floats per row of the products: two rows' 16-byte stores per
                             // quarter warp fall in different banks
constexpr int kPh = 36;      // floats per row phase of the update's keys, padded

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ uint32_t tf32_rn(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}

// Sums of a and b over the warp, in every lane.
__device__ __forceinline__ void warp_sum2(float& a, float& b, int lane) {
    const bool up = lane & 16;
    float x = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const float y = __shfl_xor_sync(0xffffffffu, x, 16);
    a = up ? y : x;
    b = up ? x : y;
}

// Row m of the left operand, channels 4 lane .. 4 lane + 3, into fragment order (rows g, g + 8 and
// channels t, t + 4 of lane 4 g + t).
__device__ __forceinline__ void store_frag(float* frag, int m, int lane, float4 x) {
    const int r = m & 15;
    float* p = frag + ((m >> 4) * 16 + (lane >> 1)) * kFrag + (r & 7) * 16 + (r >> 3) +
               2 * (lane & 1);
    p[0] = x.x;
    p[4] = x.y;
    p[8] = x.z;
    p[12] = x.w;
}

// S columns [16 warp, +16): this thread's rows 8 s + t and 8 s + t + 4 at [2 s] and [2 s + 1],
// columns 2 g and 2 g + 1 (the first and second 8-column tile of the product).
__device__ __forceinline__ void load_state(float2 (&s)[32], const float* S, int warp, int lane) {
    const float* p = S + (size_t)(lane & 3) * kD + 16 * warp + 2 * (lane >> 2);
#pragma unroll
    for (int i = 0; i < 32; ++i)
        s[i] = __ldcs(reinterpret_cast<const float2*>(p + (size_t)(4 * i) * kD));
}

// Rows [16 mt, +16) of the product with S into x (stride kXs).
template <bool kSplit>
__device__ __forceinline__ void product(const float2 (&s)[32], const float* frag, float* x, int mt,
                                        int warp, int lane) {
    float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 16; ++ks) {
        const float4 f = *reinterpret_cast<const float4*>(frag + (mt * 16 + ks) * kFrag + 4 * lane);
        const uint32_t ah[4] = {tf32_rn(f.x), tf32_rn(f.y), tf32_rn(f.z), tf32_rn(f.w)};
        const float2 p = s[2 * ks], q = s[2 * ks + 1];
        const uint32_t b0[2] = {tf32_rn(p.x), tf32_rn(q.x)}, b1[2] = {tf32_rn(p.y), tf32_rn(q.y)};
        if (kSplit) {
            const uint32_t al[4] = {tf32_rn(f.x - __uint_as_float(ah[0])),
                                    tf32_rn(f.y - __uint_as_float(ah[1])),
                                    tf32_rn(f.z - __uint_as_float(ah[2])),
                                    tf32_rn(f.w - __uint_as_float(ah[3]))};
            const uint32_t l0[2] = {tf32_rn(p.x - __uint_as_float(b0[0])),
                                    tf32_rn(q.x - __uint_as_float(b0[1]))};
            const uint32_t l1[2] = {tf32_rn(p.y - __uint_as_float(b1[0])),
                                    tf32_rn(q.y - __uint_as_float(b1[1]))};
            mma_tf32_16x8x8(a0, al, b0);
            mma_tf32_16x8x8(a1, al, b1);
            mma_tf32_16x8x8(a0, ah, l0);
            mma_tf32_16x8x8(a1, ah, l1);
        }
        mma_tf32_16x8x8(a0, ah, b0);
        mma_tf32_16x8x8(a1, ah, b1);
    }
    float* p = x + (size_t)(16 * mt + (lane >> 2)) * kXs + 16 * warp + 4 * (lane & 3);
    *reinterpret_cast<float4*>(p) = make_float4(a0[0], a1[0], a0[1], a1[1]);
    *reinterpret_cast<float4*>(p + 8 * kXs) = make_float4(a0[2], a1[2], a0[3], a1[3]);
}

// Shared memory of the tree, in floats, for Tp = 16 ceil(T / 16) nodes: the left operand; then k
// and the gates, whose place the products take; then the two matrices of pairs.
struct TreeSmem {
    int frag, rows, pairs, total;
    __host__ __device__ explicit TreeSmem(int Tp) {
        frag = 0;
        rows = frag + 2 * Tp * kFrag;                 // 2 Tp / 16 row blocks of 16 channel blocks
        const int in = 2 * Tp * kD, out = 2 * Tp * kXs;
        pairs = rows + (in > out ? in : out);
        total = pairs + 2 * Tp * Tp;
    }
};

// Two blocks per SM for bf16 rows; the split products of fp32 rows need the registers of one.
template <typename Tin>
__global__ void __launch_bounds__(kThreads, sizeof(Tin) == 2 ? 2 : 1)
decode_tree_kernel(const TreeParams p) {
    extern __shared__ __align__(16) float sm[];
    __shared__ int s_par[kMaxTreeNodes];
    __shared__ float s_beta[kMaxTreeNodes];
    __shared__ unsigned long long s_above[kMaxTreeNodes];   // the ancestors of each node
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, n = unit / p.H, h = unit % p.H;
    const int T = p.T, Tp = (T + 15) & ~15;
    const TreeSmem L(Tp);
    float *frag = sm + L.frag, *s_k = sm + L.rows, *s_g = s_k + Tp * kD, *x = sm + L.rows;
    float *akk = sm + L.pairs, *aqk = akk + Tp * Tp;
    const Tin* q = static_cast<const Tin*>(p.q);
    const Tin* k = static_cast<const Tin*>(p.k);
    const Tin* v = static_cast<const Tin*>(p.v);
    auto row = [&](int i) { return (((size_t)n * T + i) * p.H + h) * kD; };

    float2 s[32];
    load_state(s, p.S + (size_t)unit * kD * kD, warp, lane);

    if (tid == 0) s_bad = 0;
    if (tid < kMaxTreeNodes) {
        const int par = tid < T ? p.nodes[(size_t)n * T + tid] : -2;
        s_par[tid] = par;
        s_beta[tid] = par == -2 ? 0.f
                                : load_elem(static_cast<const Tin*>(p.beta),
                                            ((int64_t)n * T + tid) * p.H + h);
    }
    for (int i = tid; i < T * (kD / 4); i += kThreads) {
        const int r = i >> 5, c = 4 * (i & 31);
        const float4 g = load4(p.log_g + row(r) + c);
        *reinterpret_cast<float4*>(s_k + r * kD + c) = load4(k + row(r) + c);
        *reinterpret_cast<float4*>(s_g + r * kD + c) =
            make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w));
    }
    for (int i = tid; i < 2 * Tp * Tp / 4; i += kThreads)
        *reinterpret_cast<float4*>(akk + 4 * i) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    if (tid < T) {   // -2: no node; else the root or an earlier node that is there
        const int par = s_par[tid];
        if (par < -2 || par >= tid || (par >= 0 && s_par[par] == -2)) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {
        if (tid == 0) set_device_error(p.err, DEV_BAD_INDEX);
        return;
    }

    for (int i = warp; i < Tp; i += kWarps) {
        float4 ki = make_float4(0.f, 0.f, 0.f, 0.f), qi = ki, d = ki;
        unsigned long long above = 0;
        if (s_par[i] != -2) {
            ki = *reinterpret_cast<const float4*>(s_k + i * kD + 4 * lane);
            qi = load4(q + row(i) + 4 * lane);
            float qk = dot4(qi, ki), none = 0.f;
            warp_sum2(qk, none, lane);
            if (lane == 0) aqk[i * Tp + i] = qk;
            d = *reinterpret_cast<const float4*>(s_g + i * kD + 4 * lane);
            for (int j = s_par[i]; j >= 0; j = s_par[j]) {
                const float4 kj =
                    mul4(d, *reinterpret_cast<const float4*>(s_k + j * kD + 4 * lane));
                float a = dot4(ki, kj), b = dot4(qi, kj);
                warp_sum2(a, b, lane);
                if (lane == 0) akk[i * Tp + j] = a, aqk[i * Tp + j] = b;
                above |= 1ull << j;
                d = mul4(d, *reinterpret_cast<const float4*>(s_g + j * kD + 4 * lane));
            }
        }
        if (lane == 0) s_above[i] = above;
        store_frag(frag, i, lane, mul4(ki, d));
        store_frag(frag, Tp + i, lane, mul4(qi, d));
    }
    __syncthreads();

    for (int mt = 0; mt < 2 * Tp / 16; ++mt)
        product<sizeof(Tin) == 4>(s, frag, x, mt, warp, lane);
    __syncthreads();

    if (tid < kD) {   // a column's rows are read and written by its own thread alone
        Tin* o = static_cast<Tin*>(p.o);
        // The pairs of other branches have coefficient 0. An infinite or NaN u would turn that
        // into NaN, so such a u enters the sums as 0, and `bad` has its node: what is below it
        // in the tree becomes NaN, what is beside it does not.
        unsigned long long bad = 0;
        for (int b = 0; b < Tp; b += 16) {
            float u[16], vi[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                vi[i] = s_par[b + i] != -2 ? load_elem(v, row(b + i) + tid) : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float *ak = akk + (b + i) * Tp, *aq = aqk + (b + i) * Tp;
                float r = vi[i] - x[(b + i) * kXs + tid], y = x[(Tp + b + i) * kXs + tid];
                for (int j = 0; j < b; j += 4) {
                    const float4 a = load4(ak + j), c = load4(aq + j);
                    const float u0 = x[j * kXs + tid], u1 = x[(j + 1) * kXs + tid],
                                u2 = x[(j + 2) * kXs + tid], u3 = x[(j + 3) * kXs + tid];
                    r -= fmaf(a.x, u0, fmaf(a.y, u1, fmaf(a.z, u2, a.w * u3)));
                    y += fmaf(c.x, u0, fmaf(c.y, u1, fmaf(c.z, u2, c.w * u3)));
                }
#pragma unroll
                for (int j = 0; j < i; ++j) {
                    r = fmaf(-ak[b + j], u[j], r);
                    y = fmaf(aq[b + j], u[j], y);
                }
                if (bad & s_above[b + i]) r = y = __int_as_float(0x7fc00000);
                u[i] = s_beta[b + i] * r;
                y = fmaf(aq[b + i], u[i], y);
                if (!(fabsf(u[i]) <= 3.402823466e38f)) {
                    u[i] = 0.f;
                    bad |= 1ull << (b + i);
                }
                x[(b + i) * kXs + tid] = u[i];
                if (s_par[b + i] != -2) store_elem(o, row(b + i) + tid, y);
            }
        }
    }
}

constexpr int kGroup = 16;   // rows of a path taken at once

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 2)
commit_path_kernel(const TreeParams p) {
    __shared__ __align__(16) float frag[16 * kFrag];
    __shared__ __align__(16) float s_rows[2 * kGroup * kXs];   // k and the gates, then k S
    __shared__ __align__(16) float s_ke[kGroup][4 * kPh];      // d_ej k_j by row phase
    __shared__ __align__(16) float s_end[4 * kPh];             // d_e by row phase
    __shared__ __align__(16) float akk[kGroup * kGroup];
    __shared__ float s_beta[kGroup];
    __shared__ int s_row[kGroup];
    __shared__ int s_len, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, n = unit / p.H, h = unit % p.H;
    const int32_t* path = p.nodes + (size_t)n * p.A;
    float *s_k = s_rows, *s_g = s_rows + kGroup * kD, *x = s_rows;
    const Tin* k = static_cast<const Tin*>(p.k);
    const Tin* v = static_cast<const Tin*>(p.v);
    auto row = [&](int i) { return (((size_t)n * p.T + i) * p.H + h) * kD; };

    if (tid == 0) s_len = p.A, s_bad = 0;
    __syncthreads();
    for (int i = tid; i < p.A; i += kThreads) {   // the path ends at its first negative entry
        const int r = path[i];
        if (r < 0) atomicMin(&s_len, i);
    }
    __syncthreads();
    const int len = s_len;
    for (int i = tid; i < len; i += kThreads)
        if (path[i] >= p.T) s_bad = 1;
    __syncthreads();
    if (s_bad) {
        if (tid == 0) set_device_error(p.err, DEV_BAD_INDEX);
        return;
    }
    if (len == 0) return;

    float2 s[32];
    float* S = p.S + (size_t)unit * kD * kD;
    load_state(s, S, warp, lane);

    for (int a0 = 0; a0 < len; a0 += kGroup) {
        const int m = min(kGroup, len - a0);
        if (tid < kGroup) {
            const int r = tid < m ? path[a0 + tid] : 0;
            s_row[tid] = r;
            s_beta[tid] =
                tid < m ? load_elem(static_cast<const Tin*>(p.beta),
                                    ((int64_t)n * p.T + r) * p.H + h)
                        : 0.f;
        }
        akk[tid] = 0.f;
        __syncthreads();
        for (int i = tid; i < m * (kD / 4); i += kThreads) {
            const int r = i >> 5, c = 4 * (i & 31);
            const size_t at = row(s_row[r]) + c;
            const float4 g = load4(p.log_g + at);
            *reinterpret_cast<float4*>(s_k + r * kD + c) = load4(k + at);
            *reinterpret_cast<float4*>(s_g + r * kD + c) =
                make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w));
        }
        __syncthreads();

        for (int i = warp; i < kGroup; i += kWarps) {
            float4 ki = make_float4(0.f, 0.f, 0.f, 0.f), d = ki;
            if (i < m) {
                // channel c sits at row phase c % 4, place 2 (c / 8) + (c / 4) % 2 = c / 4
                const bool end = i == m - 1;
                ki = *reinterpret_cast<const float4*>(s_k + i * kD + 4 * lane);
                d = make_float4(1.f, 1.f, 1.f, 1.f);
                for (int j = i; j >= 0; --j) {
                    const float4 kj =
                        mul4(d, *reinterpret_cast<const float4*>(s_k + j * kD + 4 * lane));
                    if (end) {
                        s_ke[j][lane] = kj.x;
                        s_ke[j][kPh + lane] = kj.y;
                        s_ke[j][2 * kPh + lane] = kj.z;
                        s_ke[j][3 * kPh + lane] = kj.w;
                    }
                    if (j < i) {
                        float a = dot4(ki, kj), none = 0.f;
                        warp_sum2(a, none, lane);
                        if (lane == 0) akk[i * kGroup + j] = a;
                    }
                    d = mul4(d, *reinterpret_cast<const float4*>(s_g + j * kD + 4 * lane));
                }
                if (end) {
                    s_end[lane] = d.x;
                    s_end[kPh + lane] = d.y;
                    s_end[2 * kPh + lane] = d.z;
                    s_end[3 * kPh + lane] = d.w;
                }
            }
            store_frag(frag, i, lane, mul4(ki, d));
        }
        __syncthreads();

        product<true>(s, frag, x, 0, warp, lane);
        __syncthreads();

        if (tid < kD) {
            float u[kGroup], vi[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                vi[i] = i < m ? load_elem(v, row(s_row[i]) + tid) : 0.f;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                float r = vi[i] - x[i * kXs + tid];
#pragma unroll
                for (int j = 0; j < i; ++j) r = fmaf(-akk[i * kGroup + j], u[j], r);
                u[i] = s_beta[i] * r;
                x[i * kXs + tid] = u[i];
            }
        }
        __syncthreads();

        const int t = lane & 3, col = 16 * warp + 2 * (lane >> 2);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 d = load4(s_end + t * kPh + i);
            s[i].x *= d.x, s[i].y *= d.x;
            s[i + 1].x *= d.y, s[i + 1].y *= d.y;
            s[i + 2].x *= d.z, s[i + 2].y *= d.z;
            s[i + 3].x *= d.w, s[i + 3].y *= d.w;
        }
        for (int j = 0; j < m; ++j) {
            const float2 u = *reinterpret_cast<const float2*>(x + j * kXs + col);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 c = load4(&s_ke[j][t * kPh + i]);
                s[i].x = fmaf(c.x, u.x, s[i].x), s[i].y = fmaf(c.x, u.y, s[i].y);
                s[i + 1].x = fmaf(c.y, u.x, s[i + 1].x), s[i + 1].y = fmaf(c.y, u.y, s[i + 1].y);
                s[i + 2].x = fmaf(c.z, u.x, s[i + 2].x), s[i + 2].y = fmaf(c.z, u.y, s[i + 2].y);
                s[i + 3].x = fmaf(c.w, u.x, s[i + 3].x), s[i + 3].y = fmaf(c.w, u.y, s[i + 3].y);
            }
        }
        __syncthreads();   // the next group's rows take the place of these
    }

    float* out = S + (size_t)(lane & 3) * kD + 16 * warp + 2 * (lane >> 2);
#pragma unroll
    for (int i = 0; i < 32; ++i)
        __stcs(reinterpret_cast<float2*>(out + (size_t)(4 * i) * kD), s[i]);
}

PerDevice g_tree_setup;

template <typename Tin>
cudaError_t launch_tree_typed(const TreeParams& p, cudaStream_t stream) {
    const int bytes = TreeSmem((p.T + 15) & ~15).total * (int)sizeof(float);
    decode_tree_kernel<Tin><<<(unsigned)(p.N * p.H), kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream) {
    const cudaError_t e = g_tree_setup.run([](int) {
        const int most = TreeSmem(kMaxTreeNodes).total * (int)sizeof(float);
        const cudaError_t a = cudaFuncSetAttribute(
            decode_tree_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (a != cudaSuccess) return a;
        return cudaFuncSetAttribute(decode_tree_kernel<__nv_bfloat16>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    if (e != cudaSuccess) return e;
    return p.bf16 ? launch_tree_typed<__nv_bfloat16>(p, stream)
                  : launch_tree_typed<float>(p, stream);
}

cudaError_t launch_commit_path(const TreeParams& p, cudaStream_t stream) {
    const unsigned blocks = (unsigned)(p.N * p.H);
    if (p.bf16) commit_path_kernel<__nv_bfloat16><<<blocks, kThreads, 0, stream>>>(p);
    else commit_path_kernel<float><<<blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
