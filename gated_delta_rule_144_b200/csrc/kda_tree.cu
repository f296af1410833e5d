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
// The tree: one block of 256 threads per (sequence, head) up to 32 nodes, 512 above; two blocks per SM
// up to 16 nodes, one above (the shared memory of 17 to 32 nodes is 126 KB: 128 sequences x 32 heads
// of 16 bf16 nodes 109 us, of 18 to 24 nodes 289). Phases:
//   load     S by TMA into shared memory, under way until the product; the rows of k and the
//            gates.
//   paths    d_i of every node, one after another: a thread per channel, no barrier between them.
//   pairs    d_ij = d_i / d_j, so all pairs are one product [k d; q d] (k / d)^T on the tensor
//            cores, of which the tree keeps its own. Where some d is below 1e-20 (a gate of -inf
//            included) the quotient leaves the range: then a warp per node walks the node's
//            ancestors with d_ij in registers, where only products of gates <= 1 appear. One such
//            channel of one node sends the whole (sequence, head) there. With gates of
//            -softplus(N(2, 1)) that is 10 % of chains of 16 nodes and nearly all of 18 or more:
//            128 sequences x 32 heads, chains of 18 nodes 567 us against 289, one sequence's chain
//            of 61 nodes 78 us against 18.5 of a bushy tree.
//   product  [k d; q d] S on the tensor cores (warp-level tf32 products: 16 x 8 x 8). The tree of
//            bf16 rows uses one tf32 product: its operands, rounded to nearest, lose at most 2^-11
//            each, below the bf16 output's 2^-8 (S and k / d cut off instead lose 2^-10, always
//            towards zero, and save 2 of 109 us). fp32 rows split both operands into a tf32 part
//            and a tf32 remainder and sum three products (2^-21).
//   solve    a thread per value column and block of 16 nodes substitutes forward in registers:
//            each u, once known, leaves all later rows' sums, so that a step waits for one
//            product only; then the blocks behind take the block's u from shared memory, and the
//            threads that wait add it to their read-outs.
// Bound: the phases' latency, two blocks per SM beside each other; HBM (64 KiB of state per block) in
// the limit. 128 sequences x 32 heads, 16 bf16 nodes: 109 us (0.52 of the measured copy rate), a
// block's cycles 3400 until rows and gates are there, 950 paths, 1100 quotients and fragments, 3900
// products (a tf32 product takes 18 to 20 cycles of a scheduler), 1300 solve, 2200 read-outs (counted
// when it took 105). One sequence of 61 nodes and 32 heads: 18.5 us. Before: read-outs
// within the substitution and v loaded by the solve's threads 136 and 26.6 us; path products in
// rounds that double the stretch covered 125 and 22.

#include <algorithm>

#include "kda_sm100.cuh"
#include "kda_tma.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kD = 128;
// Threads of a tree's block: one per value column and block of nodes in the solve, 8 warps at least.
constexpr int tree_threads(int nb) { return nb > 2 ? 512 : 256; }
constexpr int kB = 16;       // nodes per block of the solve
// Floats per row, so that a fragment's rows fall in different banks: of the products (16 apart: two
// rows of 16 columns), of k (8 apart: four rows of 8), and between nodes of the pairs.
constexpr int kLd = kD + 16, kLk = kD + 8, kPad = 4;
constexpr float kSteep = 1e-20f;   // a path product below this, or a quotient above the other,
constexpr float kLarge = 1e30f;    // takes the direct walk
constexpr uint32_t kStateBytes = kD * kD * 4;
constexpr long long kWaitCycles = 1ll << 31;   // about one second

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
// Four elements as they are in memory, and their values.
template <typename Tin>
struct Raw4 {
    using type = float4;
};
template <>
struct Raw4<__nv_bfloat16> {
    using type = uint2;
};
__device__ __forceinline__ float4 widen(float4 x) { return x; }
__device__ __forceinline__ float4 widen(uint2 u) {
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

__device__ __forceinline__ float round_tf32(float x) { return __uint_as_float(tf32_rn(x)); }

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Sum of x[i] over the warp's lanes; lane l returns the sum of x[l / 4].
__device__ __forceinline__ float warp_sum8(const float (&x)[8], int lane) {
    float y[4], z[2], w;
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = (b4 ? x[4 + i] : x[i]) + __shfl_xor_sync(0xffffffffu, b4 ? x[i] : x[4 + i], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        z[i] = (b3 ? y[2 + i] : y[i]) + __shfl_xor_sync(0xffffffffu, b3 ? y[i] : y[2 + i], 8);
    w = (b2 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, b2 ? z[0] : z[1], 4);
    w += __shfl_xor_sync(0xffffffffu, w, 2);
    w += __shfl_xor_sync(0xffffffffu, w, 1);
    return w;
}

// Row r (of 16) of a tile of the left operand, channels 4 lane .. 4 lane + 3, into fragment order:
// per 8 channels 128 floats, lane 4 g + t's four values (rows g, g + 8, channels 2 t, 2 t + 1)
// together, the lanes' places permuted by the channel block so that the blocks' stores fall in
// different banks. (A product's step sums over 8 channels in any order; with these pairs the rows of
// S that four lanes read are 0, 2, 4, 6, whose swizzled pieces are in different banks.)
template <bool kRound>   // to tf32, for the plain product
__device__ __forceinline__ void store_frag(float* tile, int r, int lane, float4 x) {
    if (kRound)
        x = make_float4(round_tf32(x.x), round_tf32(x.y), round_tf32(x.z), round_tf32(x.w));
    const int ks = lane >> 1, l0 = (r & 7) * 4 + 2 * (lane & 1);
    float* p = tile + ks * 128 + 2 * (r >> 3);
    *reinterpret_cast<float2*>(p + 4 * (l0 ^ (ks & 7))) = make_float2(x.x, x.y);
    *reinterpret_cast<float2*>(p + 4 * ((l0 + 1) ^ (ks & 7))) = make_float2(x.z, x.w);
}
__device__ __forceinline__ float4 load_frag(const float* tile, int ks, int lane) {
    const float4 x = load4(tile + ks * 128 + 4 * (lane ^ (ks & 7)));
    return make_float4(x.x, x.z, x.y, x.w);   // (rows g, g + 8 of the first channel, of the second)
}

// acc += one 16-row tile (fragments a) times 16 columns of the state (this lane's rows 2 t and
// 2 t + 1 of 8, columns 2 g and 2 g + 1: one per 8-column product).
// Without kSplit both operands are tf32 values already (2^-11 of an element at most, to nearest).
template <bool kSplit>
__device__ __forceinline__ void mma_step(float (&c0)[4], float (&c1)[4], float4 f, float2 p,
                                         float2 q) {
    if (!kSplit) {
        const uint32_t a[4] = {__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z),
                               __float_as_uint(f.w)};
        const uint32_t b0[2] = {__float_as_uint(p.x), __float_as_uint(q.x)};
        const uint32_t b1[2] = {__float_as_uint(p.y), __float_as_uint(q.y)};
        mma_tf32_16x8x8(c0, a, b0);
        mma_tf32_16x8x8(c1, a, b1);
        return;
    }
    const uint32_t ah[4] = {tf32_rn(f.x), tf32_rn(f.y), tf32_rn(f.z), tf32_rn(f.w)};
    const uint32_t b0[2] = {tf32_rn(p.x), tf32_rn(q.x)}, b1[2] = {tf32_rn(p.y), tf32_rn(q.y)};
    const uint32_t al[4] = {
        tf32_rn(f.x - __uint_as_float(ah[0])), tf32_rn(f.y - __uint_as_float(ah[1])),
        tf32_rn(f.z - __uint_as_float(ah[2])), tf32_rn(f.w - __uint_as_float(ah[3]))};
    const uint32_t l0[2] = {tf32_rn(p.x - __uint_as_float(b0[0])),
                            tf32_rn(q.x - __uint_as_float(b0[1]))};
    const uint32_t l1[2] = {tf32_rn(p.y - __uint_as_float(b1[0])),
                            tf32_rn(q.y - __uint_as_float(b1[1]))};
    mma_tf32_16x8x8(c0, al, b0);
    mma_tf32_16x8x8(c1, al, b1);
    mma_tf32_16x8x8(c0, ah, l0);
    mma_tf32_16x8x8(c1, ah, l1);
    mma_tf32_16x8x8(c0, ah, b0);
    mma_tf32_16x8x8(c1, ah, b1);
}
// One 8-column product.
template <bool kSplit>
__device__ __forceinline__ void mma_step(float (&c)[4], float4 f, float p, float q) {
    if (!kSplit) {
        const uint32_t a[4] = {__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z),
                               __float_as_uint(f.w)};
        const uint32_t b[2] = {__float_as_uint(p), __float_as_uint(q)};
        mma_tf32_16x8x8(c, a, b);
        return;
    }
    const uint32_t ah[4] = {tf32_rn(f.x), tf32_rn(f.y), tf32_rn(f.z), tf32_rn(f.w)};
    const uint32_t b[2] = {tf32_rn(p), tf32_rn(q)};
    const uint32_t al[4] = {
        tf32_rn(f.x - __uint_as_float(ah[0])), tf32_rn(f.y - __uint_as_float(ah[1])),
        tf32_rn(f.z - __uint_as_float(ah[2])), tf32_rn(f.w - __uint_as_float(ah[3]))};
    const uint32_t l[2] = {tf32_rn(p - __uint_as_float(b[0])), tf32_rn(q - __uint_as_float(b[1]))};
    mma_tf32_16x8x8(c, al, b);
    mma_tf32_16x8x8(c, ah, l);
    mma_tf32_16x8x8(c, ah, b);
}

// Offset of state element (r, c) in shared memory: four 32-column panels as TMA lays them out with
// the 128-byte swizzle (16-byte pieces permuted by row mod 8).
__device__ __forceinline__ int state_at(int r, int c) {
    return (c >> 5) * (kD * 32) + r * 32 + ((((c & 31) >> 2) ^ (r & 7)) << 2) + (c & 3);
}
// A tile's product to rows 0 .. 15 of x, columns cols .. cols + 15.
__device__ __forceinline__ void store_tile(float* x, int cols, int lane, const float (&c0)[4],
                                           const float (&c1)[4]) {
    float* p = x + (lane >> 2) * kLd + cols + 4 * (lane & 3);
    *reinterpret_cast<float4*>(p) = make_float4(c0[0], c1[0], c0[1], c1[1]);
    *reinterpret_cast<float4*>(p + 8 * kLd) = make_float4(c0[2], c1[2], c0[3], c1[3]);
}

// NB: blocks of 16 nodes.
template <typename Tin, int NB>
struct TreeSmem {
    static constexpr int kN = kB * NB;
    // S, then the products: rows i of k d S, rows kN + i of q d S
    float state[2 * kN * kLd > kD * kD ? 2 * kN * kLd : kD * kD];
    // the gates, then path products; then the left operand; then u, [node][column]
    float frag[2 * kN * kD];
    float k[kN * kLk];                   // k, then k / (path product)
    static constexpr int kP = kN + kPad;
    float akk[kN * kP], aqk[kN * kP];    // [j][i]: pairs of node i and j above it (and j = i)
    unsigned long long bad[kD];          // by column: nodes whose u is infinite or NaN
    unsigned long long above[kN];        // the nodes above each node
    alignas(16) int par[kN];
    float beta[kN];
    unsigned long long bar;
    int bad_tree;
};

// Pairs of a tree with steep gates: a warp per node walks the node's ancestors with the product of
// the gates between in registers, every factor <= 1. The gates come from global memory again.
template <typename Tin, int NB>
__device__ __noinline__ void direct_pairs(TreeSmem<Tin, NB>& sm, const TreeParams& p, int n, int h,
                                          int warp, int lane) {
    using Smem = TreeSmem<Tin, NB>;
    constexpr int kN = kB * NB, kWarps = tree_threads(NB) / 32;
    for (int i = (int)threadIdx.x; i < kN * Smem::kP / 2; i += 32 * kWarps)   // both matrices
        *reinterpret_cast<float4*>(sm.akk + 4 * i) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    const Tin* q = static_cast<const Tin*>(p.q);
    for (int i = warp; i < kN; i += kWarps) {
        if (sm.par[i] == -2) continue;
        auto at = [&](int j) { return (((size_t)n * p.T + j) * p.H + h) * kD + 4 * lane; };
        const float4 ki = load4(sm.k + i * kLk + 4 * lane), qi = load4(q + at(i));
        float4 d = make_float4(1.f, 1.f, 1.f, 1.f);
        for (int j = i; j >= 0; j = sm.par[j]) {
            const float4 kj = mul4(d, load4(sm.k + j * kLk + 4 * lane));
            const float x[8] = {dot4(ki, kj), dot4(qi, kj), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const float sum = warp_sum8(x, lane);
            if (lane == 0 && j != i) sm.akk[j * Smem::kP + i] = sum;
            if (lane == 4) sm.aqk[j * Smem::kP + i] = sum;
            const float4 g = load4(p.log_g + at(j));
            d = mul4(d, make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w)));
        }
    }
}

template <typename Tin, int NB>
__global__ void __launch_bounds__(tree_threads(NB), NB == 1 && sizeof(Tin) == 2 ? 2 : 1)
decode_tree_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeParams p) {
    using Smem = TreeSmem<Tin, NB>;
    constexpr int kN = Smem::kN, kP = Smem::kP, kThreads = tree_threads(NB), kWarps = kThreads / 32;
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, n = unit / p.H, h = unit % p.H, T = p.T;
    const int width = kD / gridDim.y, c0 = width * blockIdx.y;   // this block's value columns
    float* s_d = sm.frag;   // the gates, then the products over each node's path
    const Tin* q = static_cast<const Tin*>(p.q);
    const Tin* k = static_cast<const Tin*>(p.k);
    const Tin* v = static_cast<const Tin*>(p.v);
    const size_t first = ((size_t)n * T * p.H + h) * kD, stride = (size_t)p.H * kD;   // of rows
    const uint32_t bar = smem_u32(&sm.bar);

    // this thread's pieces: node piece / 32, four channels; absent nodes hold k = q = 0, gate 1
    constexpr int kMine = kN * 32 / kThreads;
    const int col = tid & (kD - 1), blk = tid >> 7;   // the solve's column and group of nodes
    const bool mine = col >= c0 && col < c0 + width;
    float4 qd[kMine], kd[kMine];
    // half of the warps take the products with S, kCols columns each, and take v from the sums of
    // the rows k d: bf16 rows before the products, whose accumulation cuts sums off at 2^-23 of their
    // size, fp32 rows after them
    constexpr int kCols = kD / (kWarps / 2), kN8 = kCols / 16;   // columns, pairs of 8 of them
    const int cols = kCols * warp;
    const bool own = cols >= c0 && cols < c0 + width;
    using Raw = typename Raw4<Tin>::type;
    Raw vr[NB][kN8][2];
    {   // all loads that wait for nothing, at once; rows of absent nodes are dropped afterwards
        float4 g[kMine];
        int par[kMine];
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int r = min(m * kWarps + warp, T - 1);
            const size_t at = first + r * stride + 4 * lane;
            kd[m] = load4(k + at);
            qd[m] = load4(q + at);
            g[m] = load4(p.log_g + at);
            par[m] = p.nodes[(size_t)n * T + r];
        }
        if (warp < kWarps / 2) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < kN8; ++e)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = kB * b + (lane >> 2) + 8 * x;
                        vr[b][e][x] = Raw{};
                        if (r < T && own)
                            vr[b][e][x] = *reinterpret_cast<const Raw*>(
                                v + first + r * stride + cols + 16 * e + 4 * (lane & 3));
                    }
        }
        const int node = tid - kThreads / 2, own = min(max(node, 0), T - 1);
        int parent = p.nodes[(size_t)n * T + own];
        const Tin beta = static_cast<const Tin*>(p.beta)[((int64_t)n * T + own) * p.H + h];
        if (tid == kThreads - 32) {   // behind the rows, which are needed first
            mbar_init(bar, 1);
            fence_mbar_init();
            mbar_arrive_expect_tx(bar, kD * 4 * width);
            for (int c = c0; c < c0 + width; c += 32)
                tma_load_2d(smem_u32(sm.state + c * kD), &map, bar, c, unit * kD);
            sm.bad_tree = 0;
        }
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int r = m * kWarps + warp;
            if (r >= T || par[m] == -2) {
                kd[m] = qd[m] = make_float4(0.f, 0.f, 0.f, 0.f);
                g[m] = make_float4(1.f, 1.f, 1.f, 1.f);
            } else {
                g[m] = make_float4(expf(g[m].x), expf(g[m].y), expf(g[m].z), expf(g[m].w));
            }
            *reinterpret_cast<float4*>(s_d + r * kD + 4 * lane) = g[m];
            *reinterpret_cast<float4*>(sm.k + r * kLk + 4 * lane) = kd[m];
        }
        if (node >= 0 && node < kN) {
            if (node >= T) parent = -2;
            sm.par[node] = parent;
            sm.beta[node] = parent == -2 ? 0.f : load_elem(&beta, 0);
        }
    }
    __syncthreads();
    if (tid < T) {   // -2: no node; else the root or an earlier node that is there
        const int par = sm.par[tid];
        if (par < -2 || par >= tid || (par >= 0 && sm.par[par] == -2)) sm.bad_tree = 1;
    }
    __syncthreads();
    if (sm.bad_tree) {   // (the copy lands before its shared memory goes away)
        if (tid == kThreads - 32) {
            set_device_error(p.err, DEV_BAD_INDEX);
            mbar_wait(bar, 0, kWaitCycles);
        }
        for (int i = tid; p.clear && i < T * width; i += kThreads)
            store_elem(static_cast<Tin*>(p.o), first + i / width * stride + c0 + i % width, 0.f);
        return;
    }

    // paths, in the nodes' order, four at a time: a thread per channel multiplies each node's gate by
    // its parent's product, which it has in a register or wrote itself, so nothing waits for another
    // thread; another warp gathers the nodes above each node, reaching twice as far each round
    bool steep = false;
    if (tid < kD) {
        int4 next = *reinterpret_cast<const int4*>(sm.par);
        float ng[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) ng[e] = s_d[e * kD + tid];
#pragma unroll 1
        for (int i = 0; i < kN; i += 4) {
            const int j[4] = {next.x, next.y, next.z, next.w};
            float x[4], d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[e] = ng[e];
                x[e] = j[e] >= 0 && j[e] < i ? s_d[j[e] * kD + tid] : 1.f;
            }
            const int i2 = min(i + 4, kN - 4);
            next = *reinterpret_cast<const int4*>(sm.par + i2);
#pragma unroll
            for (int e = 0; e < 4; ++e) ng[e] = s_d[(i2 + e) * kD + tid];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int m = 0; m < e; ++m) x[e] = j[e] == i + m ? d[m] : x[e];
                d[e] *= x[e];
                s_d[(i + e) * kD + tid] = d[e];
            }
        }
    } else if (warp == kD / 32) {
        constexpr int kPer = kN > 32 ? 2 : 1;   // nodes per lane: lane, lane + 32
        int j[kPer];
        unsigned long long x[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            j[e] = lane + 32 * e < kN ? sm.par[lane + 32 * e] : -1;
            x[e] = j[e] >= 0 ? 1ull << j[e] : 0;
        }
        auto of = [&](const auto& y, int i) {   // node i's
            const auto lo = __shfl_sync(0xffffffffu, y[0], i & 31);
            if (kPer == 1) return lo;
            const auto hi = __shfl_sync(0xffffffffu, y[kPer - 1], i & 31);
            return i < 32 ? lo : hi;
        };
        while (__any_sync(0xffffffffu, j[0] >= 0 || j[kPer - 1] >= 0)) {
            int far[kPer];
            unsigned long long more[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) far[e] = of(j, j[e]), more[e] = of(x, j[e]);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                x[e] |= j[e] >= 0 ? more[e] : 0;
                j[e] = j[e] >= 0 ? far[e] : -1;
            }
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (lane + 32 * e < kN) sm.above[lane + 32 * e] = x[e];
    }
    __syncthreads();
    const float* path = s_d;
    const unsigned long long* s_above = sm.above;
    // the left operand's rows k d and q d; k / d for the pairs
    float4 over[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const float4 d = load4(path + (m * kWarps + warp) * kD + 4 * lane), x = kd[m];
        over[m] = make_float4(__fdividef(x.x, d.x), __fdividef(x.y, d.y), __fdividef(x.z, d.z),
                              __fdividef(x.w, d.w));   // (2 units in the last place, d is not steep)
        kd[m] = mul4(x, d);
        qd[m] = mul4(qd[m], d);
        auto size = [](float4 a) { return (fabsf(a.x) + fabsf(a.y)) + (fabsf(a.z) + fabsf(a.w)); };
        steep |= !(fminf(d.x, d.y) >= kSteep && fminf(d.z, d.w) >= kSteep && size(d) <= 4.f);
        // (a k that is infinite or NaN itself spoils its node's pairs only, either way)
        steep |= size(x) <= kLarge && !(size(over[m]) <= kLarge);
    }
    steep = __syncthreads_or(steep);
    if (!steep) {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            float4 x = over[m];
            if (sizeof(Tin) == 2)
                x = make_float4(round_tf32(x.x), round_tf32(x.y), round_tf32(x.z), round_tf32(x.w));
            *reinterpret_cast<float4*>(sm.k + (m * kWarps + warp) * kLk + 4 * lane) = x;
        }
        __syncthreads();
    } else {
        direct_pairs<Tin, NB>(sm, p, n, h, warp, lane);
        __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int i = m * kWarps + warp;
        store_frag<sizeof(Tin) == 2>(sm.frag + (i >> 4) * 2048, i & 15, lane, kd[m]);
        store_frag<sizeof(Tin) == 2>(sm.frag + (NB + (i >> 4)) * 2048, i & 15, lane, qd[m]);
    }
    __syncthreads();
    const bool ok = mbar_wait(bar, 0, kWaitCycles);
    if (!ok) set_device_error(p.err, DEV_TIMEOUT);
    if (__syncthreads_or(!ok)) return;

    // the products with S (all 2 NB tiles of a warp's columns, so that S is read once) beside the pairs
    if (warp < kWarps / 2 && own) {
        int at0[kN8], at1[kN8];
#pragma unroll
        for (int e = 0; e < kN8; ++e) {
            at0[e] = state_at(2 * (lane & 3), cols + 16 * e + 2 * (lane >> 2));
            at1[e] = state_at(2 * (lane & 3) + 1, cols + 16 * e + 2 * (lane >> 2));
        }
        float a0[2 * NB][kN8][4], a1[2 * NB][kN8][4];
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
            for (int e = 0; e < kN8; ++e)
#pragma unroll
                for (int x = 0; x < 4; ++x) a0[b][e][x] = a1[b][e][x] = 0.f;
        auto less_v = [&] {   // (a tile's four columns as store_tile has them)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < kN8; ++e)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float4 y = widen(vr[b][e][x]);
                        a0[b][e][2 * x] -= y.x, a1[b][e][2 * x] -= y.y;
                        a0[b][e][2 * x + 1] -= y.z, a1[b][e][2 * x + 1] -= y.w;
                    }
        };
        if (sizeof(Tin) == 2) less_v();
#pragma unroll 2
        for (int ks = 0; ks < 16; ++ks) {
            float2 s0[kN8], s1[kN8];
#pragma unroll
            for (int e = 0; e < kN8; ++e) {
                s0[e] = *reinterpret_cast<const float2*>(sm.state + at0[e] + ks * 256);
                s1[e] = *reinterpret_cast<const float2*>(sm.state + at1[e] + ks * 256);
                if (sizeof(Tin) == 2) {
                    s0[e] = make_float2(round_tf32(s0[e].x), round_tf32(s0[e].y));
                    s1[e] = make_float2(round_tf32(s1[e].x), round_tf32(s1[e].y));
                }
            }
#pragma unroll
            for (int b = 0; b < 2 * NB; ++b) {
                const float4 f = load_frag(sm.frag + b * 2048, ks, lane);
#pragma unroll
                for (int e = 0; e < kN8; ++e)
                    mma_step<sizeof(Tin) == 4>(a0[b][e], a1[b][e], f, s0[e], s1[e]);
            }
        }
        if (sizeof(Tin) == 4) less_v();
        bar_sync(1, 32 * width / kCols);   // S has been read
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
            for (int e = 0; e < kN8; ++e)
                store_tile(sm.state + kB * b * kLd, cols + 16 * e, lane, a0[b][e], a1[b][e]);
    } else if (!steep) {
        // tiles (16 rows of k d or q d, block b) x (8 nodes of the blocks up to b)
        const int workers = kWarps - width / kCols, before = c0 / kCols;
        constexpr int kTiles = NB * (NB + 1);   // of k d; as many of q d
#pragma unroll 1
        for (int tile = warp < kWarps / 2 && warp < before ? warp : warp - width / kCols;
             tile < 2 * kTiles; tile += workers) {
            const int half = tile / kTiles;
            int nt = tile % kTiles, blk = 0;
            while (nt >= 2 * (blk + 1)) nt -= 2 * ++blk;
            float c[2][4] = {};   // sums of even and odd steps
            const float* b = sm.k + (8 * nt + (lane >> 2)) * kLk + 2 * (lane & 3);
            const float* a = sm.frag + (half * NB + blk) * 2048;
#pragma unroll 8
            for (int ks = 0; ks < 16; ++ks) {
                const float2 y = *reinterpret_cast<const float2*>(b + 8 * ks);
                mma_step<sizeof(Tin) == 4>(c[ks & 1], load_frag(a, ks, lane), y.x, y.y);
            }
            float* to = half ? sm.aqk : sm.akk;
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // rows g, g + 8; nodes 2 t, 2 t + 1
                const int i = 16 * blk + (lane >> 2) + 8 * (e >> 1);
                const int j = 8 * nt + 2 * (lane & 3) + (e & 1);
                const bool pair = (s_above[i] >> j & 1) || (half && i == j);
                to[j * kP + i] = pair ? c[0][e] + c[1][e] : 0.f;
            }
        }
    }
    __syncthreads();

    // The substitution for u: group b of 128 threads, one per column, solves block b in registers
    // while the others add the block before to their read-outs; then the groups behind take its u.
    float* s_u = sm.frag;
    float r[kB];
    if (blk < NB && mine) {
#pragma unroll
        for (int i = 0; i < kB; ++i)
            r[i] = sm.par[kB * blk + i] != -2
                       ? -sm.state[(kB * blk + i) * kLd + col] : 0.f;
    }
    // r less what node `at`'s u adds to the rows e of block `to`, first <= e
    auto spread = [&](int at, int to, float u, int first) {
        const float* ak = sm.akk + at * kP + kB * to;
#pragma unroll
        for (int i4 = 0; i4 < kB; i4 += 4) {
            if (i4 + 3 < first) continue;
            const float4 a = load4(ak + i4);
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i4 + e >= first) r[i4 + e] = fmaf(-av[e], u, r[i4 + e]);
        }
    };
    // the thread's read-outs, rows y0 .. y0 + kY - 1: y plus what block b's u adds to them
    constexpr int kY = kThreads == kD * NB ? kB : kN * kD / kThreads;
    const int y0 = kY * blk;
    float y[kY];
    if (mine) {
#pragma unroll
        for (int i = 0; i < kY; ++i) y[i] = sm.state[(kN + y0 + i) * kLd + col];
    }
    auto read_out = [&](int b) {
        const float *u = s_u + kB * b * kD + col, *aq = sm.aqk + kB * b * kP + y0;
#pragma unroll 4
        for (int j = 0; j < kB; ++j) {
            const float x = u[j * kD];
#pragma unroll
            for (int i = 0; i < kY; i += 4) {
                const float4 c = load4(aq + j * kP + i);
                y[i] = fmaf(c.x, x, y[i]), y[i + 1] = fmaf(c.y, x, y[i + 1]);
                y[i + 2] = fmaf(c.z, x, y[i + 2]), y[i + 3] = fmaf(c.w, x, y[i + 3]);
            }
        }
    };
    int done = 0;   // blocks in the read-outs
#pragma unroll 1
    for (int b = 0; b < NB && mine; ++b) {
        if (blk == b) {
            unsigned long long bad = b > 0 ? sm.bad[col] : 0;
            float finite = 0.f;
            float* rs = sm.state + kB * b * kLd + col;   // r as it is, in the product's place
#pragma unroll
            for (int j = 0; j < kB; ++j) rs[j * kLd] = r[j];
            float u[kB];   // (stored at the end, so that no load waits for a store)
#pragma unroll
            for (int j = 0; j < kB; ++j) u[j] = sm.beta[kB * b + j];
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                u[j] *= r[j];
                finite = fmaf(u[j], 0.f, finite);
                spread(kB * b + j, b, u[j], j + 1);
            }
#pragma unroll
            for (int j = 0; j < kB; ++j) s_u[(kB * b + j) * kD + col] = u[j];
            if (bad != 0 || finite != 0.f) {
                // The pairs of other branches have coefficient 0. An infinite or NaN u turned that
                // into NaN: again, with such a u entering the sums as 0. What is below its node in
                // the tree becomes NaN, what is beside it does not.
#pragma unroll 1
                for (int j = 0; j < kB; ++j) {
                    const int at = kB * b + j;
                    const float* ak = sm.akk + at * kP + kB * b;
                    float u = sm.beta[at] * rs[j * kLd];
                    if (bad & s_above[at] || !(fabsf(u) <= 3.402823466e38f)) {
                        u = 0.f;
                        bad |= 1ull << at;
                    }
                    s_u[at * kD + col] = u;
#pragma unroll 1
                    for (int e = j + 1; e < kB; ++e) rs[e * kLd] = fmaf(-ak[e], u, rs[e * kLd]);
                }
            }
            sm.bad[col] = bad;
        } else if (done < b && done <= blk) {   // (one block at a time: no longer than the solve)
            read_out(done++);
        }
        bar_sync(1, NB == 1 ? 2 * width : NB * width);
        if (blk > b && blk < NB) {
#pragma unroll 4
            for (int j = 0; j < kB; ++j) spread(kB * b + j, blk, s_u[(kB * b + j) * kD + col], 0);
        }
    }
    if (!mine) return;
#pragma unroll 1
    while (done <= min(blk, NB - 1)) read_out(done++);
    Tin* o = static_cast<Tin*>(p.o) + first + y0 * stride + col;
    const unsigned long long bad = sm.bad[col];
#pragma unroll
    for (int i = 0; i < kY; ++i, o += stride) {
        if (sm.par[y0 + i] != -2)
            store_elem(o, 0, bad >> (y0 + i) & 1 ? __int_as_float(0x7fc00000) : y[i]);
        else if (p.clear && y0 + i < T)
            store_elem(o, 0, 0.f);
    }
}

// The commit. Two blocks per SM walk the (sequence, head) units: four warps work on one unit's state
// in registers while a fifth brings the next unit's state and first rows into shared memory by bulk
// copies. Rows are taken four at a time: thread c holds channel c of the rows (their products of
// gates are its own running products), then, as (row phase, four columns), 32 rows of the state:
// k d S, the substitution for u in registers, and S = d_e S + sum_j (d_ej k_j) u_j^T, each one pass
// over the registers. (Tensor-core products of 16-row tiles, split for fp32, take more instructions
// up to about 9 rows: 567 us against 280 then.) Bound: HBM (the state read and written). 256
// sequences x 32 heads, paths of up to 6 of 16 bf16 rows: 192 to 202 us, 0.85 to 0.89 of the measured
// copy rate; when it was built 192, 211 with only four rows brought ahead, 280 without the loader
// warp; 199 with a path's last one or two rows taken as two instead of four.
constexpr int kRows = 4;
constexpr int kStaged = 8;   // rows of a path that the loader brings
constexpr int kPathWorkers = 128, kPathThreads = kPathWorkers + 32;
template <typename Tin>
struct PathSmem {
    float state[kD * kD];           // the next unit's state
    Tin k[2][kStaged][kD], v[2][kStaged][kD];   // first rows of this unit and the next
    float g[2][kStaged][kD], beta[2][kStaged];
    float4 kd[kD], ke[kD];          // [channel][row]: k_j d_j, d_ej k_j
    float end[kD];                  // d_e
    float pairs[4][8];              // per warp: pair sums
    int unit[2], len[2];            // (unit at the end of the walk: -1)
    unsigned long long full[2], ready[2], free;
};

template <typename Tin>
__global__ void __launch_bounds__(kPathThreads, 2)
commit_path_kernel(const TreeParams p, const int units) {
    extern __shared__ __align__(16) uint8_t raw[];
    PathSmem<Tin>& sm = *reinterpret_cast<PathSmem<Tin>*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tin* k = static_cast<const Tin*>(p.k);
    const Tin* v = static_cast<const Tin*>(p.v);
    const uint32_t full = smem_u32(sm.full), ready = smem_u32(sm.ready),
                   free = smem_u32(&sm.free);
    if (tid == 0) {
        mbar_init(full, 1);
        mbar_init(full + 8, 1);
        mbar_init(ready, 1);
        mbar_init(ready + 8, 1);
        mbar_init(free, kPathWorkers);
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kPathWorkers / 32) {   // ------------------------------------------------ loader
        int it = 0;
        bool ok = true;
        for (int unit = blockIdx.x; unit < units && ok; unit += gridDim.x) {
            // the path's length: up to its first negative entry; nothing is done where it leaves
            // the rows
            const int n = unit / p.H, h = unit % p.H;
            const int32_t* path = p.nodes + (size_t)n * p.A;
            int len = p.A, first = -1;
            bool bad = false;
            for (int i0 = 0; i0 < len; i0 += 32) {
                const int r = i0 + lane < p.A ? path[i0 + lane] : -1;
                const unsigned stop = __ballot_sync(0xffffffffu, r < 0);
                const int here = stop ? __ffs(stop) - 1 : 32;
                bad |= lane < here && r >= p.T;
                if (i0 == 0) first = r;
                if (stop) len = i0 + here;
            }
            if (__any_sync(0xffffffffu, bad)) {
                if (lane == 0) set_device_error(p.err, DEV_BAD_INDEX);
                continue;
            }
            if (len == 0) continue;
            // the workers have the previous state in registers, and are done with this buffer's
            // rows
            const int b = it & 1, m = min(len, kStaged);
            if (it > 0) ok = __all_sync(0xffffffffu, mbar_wait(free, (it - 1) & 1, kWaitCycles));
            if (!ok) {   // (nothing of this CTA is in flight)
                if (lane == 0) {
                    sm.unit[b] = -1;
                    mbar_arrive(ready + 8 * b);
                }
                break;
            }
            const uint32_t bar = full + 8 * b;
            if (lane < kStaged)
                sm.beta[b][lane] = lane < m ? load_elem(static_cast<const Tin*>(p.beta),
                                                        ((int64_t)n * p.T + first) * p.H + h)
                                            : 0.f;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, kStateBytes + m * kD * (2 * sizeof(Tin) + 4));
                for (int i = 0; i < 4; ++i)
                    bulk_load(smem_u32(sm.state) + i * (kStateBytes / 4),
                              p.S + (size_t)unit * kD * kD + i * (kD * kD / 4), kStateBytes / 4,
                              bar);
            }
            __syncwarp();
            if (lane < m) {
                const size_t at = (((size_t)n * p.T + first) * p.H + h) * kD;
                bulk_load(smem_u32(sm.k[b][lane]), k + at, kD * sizeof(Tin), bar);
                bulk_load(smem_u32(sm.v[b][lane]), v + at, kD * sizeof(Tin), bar);
                bulk_load(smem_u32(sm.g[b][lane]), p.log_g + at, kD * 4, bar);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(bar, (it >> 1) & 1, kWaitCycles));
            if (lane == 0) {
                sm.unit[b] = ok ? unit : -1;
                sm.len[b] = len;
                mbar_arrive(ready + 8 * b);
            }
            __syncwarp();
            ++it;
        }
        if (!ok) {
            if (lane == 0) set_device_error(p.err, DEV_TIMEOUT);
            return;
        }
        // (the buffer of two units ago: free once the unit before is in registers)
        if (it > 0 && !__all_sync(0xffffffffu, mbar_wait(free, (it - 1) & 1, kWaitCycles)) &&
            lane == 0)
            set_device_error(p.err, DEV_TIMEOUT);
        if (lane == 0) {
            sm.unit[it & 1] = -1;
            mbar_arrive(ready + 8 * (it & 1));
        }
        return;
    }

    // ------------------------------------------------------------------------------ workers
    const int phase = lane >> 3, col = 32 * warp + 4 * (lane & 7);
    for (int it = 0;; ++it) {
        const int b = it & 1;
        // the loader arrives within two of its own bounds, whether the copies landed or not, so
        // that the four warps always take the same way here (the look at `full` orders the copies
        // before this thread's reads)
        if (!mbar_wait(ready + 8 * b, (it >> 1) & 1, 8 * kWaitCycles)) return;
        mbar_try_wait(full + 8 * b, (it >> 1) & 1);
        const int unit = sm.unit[b], len = sm.len[b];
        if (unit < 0) return;
        const int n = unit / p.H, h = unit % p.H;
        const int32_t* path = p.nodes + (size_t)n * p.A;
        auto row = [&](int a) { return (((size_t)n * p.T + path[a]) * p.H + h) * kD; };
        float4 s[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = load4(sm.state + (phase + 4 * i) * kD + col);
        mbar_arrive(free);

        for (int a0 = 0; a0 < len; a0 += kRows) {
            float kk[kRows], gg[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                kk[j] = 0.f;
                gg[j] = 1.f;
                if (a0 + j >= len) continue;
                if (a0 < kStaged) {
                    kk[j] = load_elem(sm.k[b][a0 + j], tid);
                    gg[j] = expf(sm.g[b][a0 + j][tid]);
                } else {
                    const size_t at = row(a0 + j) + tid;
                    kk[j] = load_elem(k, at);
                    gg[j] = expf(p.log_g[at]);
                }
            }
            // channel tid: products of gates up to each row, from behind each row, between rows
            const float p0 = gg[0], p1 = p0 * gg[1], p2 = p1 * gg[2], p3 = p2 * gg[3];
            const float q2 = gg[3], q1 = gg[2] * q2, q0 = gg[1] * q1;
            bar_sync(1, kPathWorkers);   // everyone has read the rows before these
            sm.kd[tid] = make_float4(kk[0] * p0, kk[1] * p1, kk[2] * p2, kk[3] * p3);
            sm.ke[tid] = make_float4(kk[0] * q0, kk[1] * q1, kk[2] * q2, kk[3]);
            sm.end[tid] = p3;
            {   // pairs (1,0) (2,0) (2,1) (3,0) (3,1) (3,2)
                const float g12 = gg[1] * gg[2], g23 = gg[2] * gg[3];
                const float x[8] = {kk[1] * gg[1] * kk[0], kk[2] * g12 * kk[0], kk[2] * gg[2] * kk[1],
                                    kk[3] * (g12 * gg[3]) * kk[0], kk[3] * g23 * kk[1],
                                    kk[3] * gg[3] * kk[2], 0.f, 0.f};
                const float sum = warp_sum8(x, lane);
                if ((lane & 3) == 0) sm.pairs[warp][lane >> 2] = sum;
            }
            bar_sync(1, kPathWorkers);
            float4 y[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j) y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float4 c = sm.kd[phase + 4 * i];
                const float cj[kRows] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    y[j].x = fmaf(cj[j], s[i].x, y[j].x), y[j].y = fmaf(cj[j], s[i].y, y[j].y);
                    y[j].z = fmaf(cj[j], s[i].z, y[j].z), y[j].w = fmaf(cj[j], s[i].w, y[j].w);
                }
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j)
#pragma unroll
                for (int off = 8; off <= 16; off <<= 1) {
                    y[j].x += __shfl_xor_sync(0xffffffffu, y[j].x, off);
                    y[j].y += __shfl_xor_sync(0xffffffffu, y[j].y, off);
                    y[j].z += __shfl_xor_sync(0xffffffffu, y[j].z, off);
                    y[j].w += __shfl_xor_sync(0xffffffffu, y[j].w, off);
                }
            // u_j = beta_j (v_j - k_j d_j S - sum_{l<j} pair(j, l) u_l), in place of y
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
                if (a0 + j < len)
                    r = a0 < kStaged ? load4(sm.v[b][a0 + j] + col) : load4(v + row(a0 + j) + col);
                r = make_float4(r.x - y[j].x, r.y - y[j].y, r.z - y[j].z, r.w - y[j].w);
#pragma unroll
                for (int l = 0; l < j; ++l) {
                    const int e = j * (j - 1) / 2 + l;
                    const float a = -((sm.pairs[0][e] + sm.pairs[1][e]) +
                                      (sm.pairs[2][e] + sm.pairs[3][e]));
                    r.x = fmaf(a, y[l].x, r.x), r.y = fmaf(a, y[l].y, r.y);
                    r.z = fmaf(a, y[l].z, r.z), r.w = fmaf(a, y[l].w, r.w);
                }
                const float beta =
                    a0 < kStaged ? sm.beta[b][a0 + j]
                    : a0 + j < len ? load_elem(static_cast<const Tin*>(p.beta), row(a0 + j) / kD)
                                   : 0.f;
                y[j] = make_float4(beta * r.x, beta * r.y, beta * r.z, beta * r.w);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float4 c = sm.ke[phase + 4 * i];
                const float d = sm.end[phase + 4 * i];
                s[i].x *= d, s[i].y *= d, s[i].z *= d, s[i].w *= d;
                const float cj[kRows] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    s[i].x = fmaf(cj[j], y[j].x, s[i].x), s[i].y = fmaf(cj[j], y[j].y, s[i].y);
                    s[i].z = fmaf(cj[j], y[j].z, s[i].z), s[i].w = fmaf(cj[j], y[j].w, s[i].w);
                }
            }
        }
        float* out = p.S + (size_t)unit * kD * kD + phase * kD + col;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            __stcs(reinterpret_cast<float4*>(out + 4 * i * kD), s[i]);
    }
}

PerDevice g_setup;
int g_sms[PerDevice::kMax];   // written once per device, under g_setup

template <typename Tin, int NB>
cudaError_t set_tree() {
    return cudaFuncSetAttribute(decode_tree_kernel<Tin, NB>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(TreeSmem<Tin, NB>));
}

cudaError_t set_up(int dev) {
    cudaError_t e = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if ((e = set_tree<float, 1>()) != cudaSuccess || (e = set_tree<float, 2>()) != cudaSuccess ||
        (e = set_tree<float, 4>()) != cudaSuccess ||
        (e = set_tree<__nv_bfloat16, 1>()) != cudaSuccess ||
        (e = set_tree<__nv_bfloat16, 2>()) != cudaSuccess ||
        (e = set_tree<__nv_bfloat16, 4>()) != cudaSuccess)
        return e;
    if ((e = cudaFuncSetAttribute(commit_path_kernel<float>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)sizeof(PathSmem<float>))) != cudaSuccess)
        return e;
    return cudaFuncSetAttribute(commit_path_kernel<__nv_bfloat16>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(PathSmem<__nv_bfloat16>));
}

template <typename Tin, int NB>
cudaError_t launch_tree(const TreeParams& p, int sms, cudaStream_t stream) {
    CUtensorMap map;
    const cudaError_t e = make_map_2d(&map, p.S, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                                      (unsigned long long)p.N * p.H * kD, kD, 32, kD,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    // two blocks per unit, half of the value columns each, where SMs are to spare (32 units, 61 nodes:
    // 16.9 us against 20.3 with one, 30 nodes 9.95 / 10.4, 12 nodes 6.06 / 6.43)
    const dim3 grid((unsigned)(p.N * p.H), p.N * p.H * 2 <= sms ? 2 : 1);
    decode_tree_kernel<Tin, NB>
        <<<grid, tree_threads(NB), sizeof(TreeSmem<Tin, NB>), stream>>>(map, p);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_tree_nodes(const TreeParams& p, int sms, cudaStream_t stream) {
    if (p.T <= 16) return launch_tree<Tin, 1>(p, sms, stream);
    if (p.T <= 32) return launch_tree<Tin, 2>(p, sms, stream);
    return launch_tree<Tin, 4>(p, sms, stream);
}

}  // namespace

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream) {
    int dev = 0;
    const cudaError_t e = g_setup.run(set_up, &dev);
    if (e != cudaSuccess) return e;
    return p.bf16 ? launch_tree_nodes<__nv_bfloat16>(p, g_sms[dev], stream)
                  : launch_tree_nodes<float>(p, g_sms[dev], stream);
}

cudaError_t launch_commit_path(const TreeParams& p, cudaStream_t stream) {
    int dev = 0;
    const cudaError_t e = g_setup.run(set_up, &dev);
    if (e != cudaSuccess) return e;
    const int units = p.N * p.H;
    const unsigned blocks = (unsigned)std::min(units, 2 * g_sms[dev]);
    if (p.bf16)
        commit_path_kernel<__nv_bfloat16>
            <<<blocks, kPathThreads, sizeof(PathSmem<__nv_bfloat16>), stream>>>(p, units);
    else
        commit_path_kernel<float>
            <<<blocks, kPathThreads, sizeof(PathSmem<float>), stream>>>(p, units);
    return cudaGetLastError();
}

}  // namespace kda
