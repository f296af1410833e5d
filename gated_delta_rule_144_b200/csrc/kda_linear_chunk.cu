// Linear attention with a scalar decay for each head, in chunks of 128 tokens on the tensor cores
// (bf16, dk <= 128, dk and dv multiples of 8).
//
// With G_i the sum of the log gates of a chunk's rows 0 .. i, S the state before the chunk and E
// the sum over all its rows,
//     o_i = e^{G_i} (q_i S) + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j
//     S  <- e^E S + sum_j k_j (e^{E - G_j} v_j)^T
// One CTA owns 64 value columns of one (segment, head) and walks its chunks in order. The products
// that follow from q, k and v alone do not wait for the state, which is one multiply-add per
// element, so the walk is bound by the data's way into the SM, not by a chain.
//
// What keeps which precision.
//   - The state stays fp32 in registers. What a chunk adds to it, K^T (decayed V), must not lose
//     what fp32 holds, so the decayed v is split into three bf16 terms (8 bits each, 2^-25 left)
//     and the three products are summed in fp32. The product runs once with N = 192, the three
//     terms side by side.
//   - q S reads the state rounded to bf16, and the decayed scores are rounded to bf16: each 2^-9
//     of a term at most, as the output's own rounding, on disjoint parts of the output.
//   - Decays are products of gates <= 1: a pair of rows in different 32-row blocks takes
//     (suffix of j's block) (blocks between) (prefix of i's block), so no exponential grows
//     and none is taken of a difference of large sums; inside a block G_i - G_j is a
//     difference of sums over at most 32 rows. Gates below -110 count as -110, whose
//     exponential is 0 in fp32 like that of anything below.
//
// Roles (15 warps), which meet through mbarriers only:
//   warps 0-3   scores: P = Q K^T out of TMEM, times the decays, rounded to bf16 into TMEM, where
//               P V takes its left operand (row i is TMEM lane i; a warp is a 32-row block)
//   warps 4-7   state: lane i holds row i of S, 64 columns in registers; adds a chunk's three
//               partial products and writes S as bf16 to shared memory for the next Q S
//   warps 8-11  values: the three terms of the decayed V to shared memory; the chunk's output
//               o = P V + e^G (Q S) out of TMEM to global memory
//   warp 12     loader: q, k, v by TMA, two stages. It clears the rows of k and v behind a
//               sequence's end (they are another's), so that nothing of them enters a product
//   warp 13     issues every tcgen05.mma
//   warp 14     gates: block-wise prefix and suffix sums, a chunk ahead
// TMEM: P 128 columns, bf16 P 64, P V 64, Q S 64, three state terms 192: all 512. Shared memory:
// 2 x 80 KiB of stages, 48 KiB of decayed V, 16 KiB of bf16 state.
// Every wait is bounded; on expiry the CTA records KDA_ERR_TIMEOUT, drains its copies and
// products, frees TMEM and exits.

#include <cuda.h>

#include <cstdlib>

#include "kda_linear.cuh"
#include "kda_sm100.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kC = 128;                 // tokens per chunk
constexpr int kNV = 64;                 // value columns per CTA
constexpr int kThreads = 15 * 32;
constexpr int kLoadWarp = 12, kMmaWarp = 13;   // the last warp is the gates'

constexpr uint32_t kPanel = 16384;      // 128 rows x 128 bytes, 128-byte swizzle
constexpr uint32_t ST_Q = 0, ST_K = 2 * kPanel, ST_V = 4 * kPanel, kStage = 5 * kPanel;
constexpr uint32_t OFF_VH = 2 * kStage;             // three terms of the decayed V
constexpr uint32_t OFF_SB = OFF_VH + 3 * kPanel;    // bf16 state
constexpr uint32_t OFF_GATE = OFF_SB + kPanel;      // per stage: loc[128], suf[128], tot[4]
constexpr uint32_t kGateBytes = (2 * kC + 4) * 4;
constexpr uint32_t OFF_BAR = OFF_GATE + 2 * kGateBytes;
constexpr uint32_t OFF_MISC = OFF_BAR + 18 * 8;     // TMEM address, abort flag
constexpr uint32_t kSmem = OFF_MISC + 16;
static_assert(kSmem <= 232448, "shared memory");
static_assert(OFF_BAR % 8 == 0 && OFF_GATE % 16 == 0 && kGateBytes % 16 == 0, "alignment");

constexpr uint32_t TM_P = 0, TM_PB = 128, TM_O1 = 192, TM_O2 = 256, TM_KV = 320;
constexpr int kTmemCols = 512;

struct ChunkArgs {
    LinearParams p;
    int tiles;              // 64-column tiles of dv
    long long budget;       // cycles a wait may take
    int debug_stall;
};

struct ChunkMaps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_bf(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// kOut: outputs (kWhole, kOutputs); else the states of segments (kStates).
template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
linear_chunk_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkArgs args) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const LinearParams& p = args.p;
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = blockIdx.x % args.tiles;
    const int h = blockIdx.x / args.tiles % p.H, g = blockIdx.x / args.tiles / p.H;
    const int hk = h / (p.H / p.Hk);
    LinearSlot sl;
    if (!linear_slot(p, g, &sl)) return;
    if (!kOut && sl.last) return;
    const int nchunks = (int)((sl.end - sl.begin + kC - 1) / kC);
    const int j0 = tile * kNV;

    // barriers: each role's waits on one count the chunks (two of a kind: one per stage)
    uint32_t nb = sb + OFF_BAR;
    const uint32_t b_full = nb, b_empty = nb + 16, b_gfull = nb + 32, b_gempty = nb + 48,
                   b_p = nb + 64, b_pb = nb + 72, b_vh = nb + 80, b_kv = nb + 88,
                   b_kvfree = nb + 96, b_s = nb + 104, b_sfree = nb + 112, b_o = nb + 120,
                   b_ofree = nb + 128, b_tail = nb + 136;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(sm + OFF_MISC);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
            mbar_init(b_gfull + 8 * i, 1);
            mbar_init(b_gempty + 8 * i, kOut ? 12 : 8);   // one per reading warp
        }
        mbar_init(b_p, 1);
        mbar_init(b_pb, 128);
        mbar_init(b_vh, 128);
        mbar_init(b_kv, 1);
        mbar_init(b_kvfree, 128);
        mbar_init(b_s, 128);
        mbar_init(b_sfree, 1);
        mbar_init(b_o, 1);
        mbar_init(b_ofree, 128);
        mbar_init(b_tail, 1);
        fence_mbar_init();
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_s), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_s;
    const uint32_t lq = (uint32_t)(32 * (warp & 3)) << 16;   // this warp's TMEM lane quarter
    const int row = tid & 127;                               // TMEM lane in warps 0-11

    // every lane waits; a warp goes on together or not at all
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool ok = mbar_wait(bar, parity & 1u, args.budget);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (lane == 0) set_device_error(p.err, DEV_TIMEOUT);
        return false;
    };
    auto rows_of = [&](int c) { return (int)min((long long)kC, sl.end - sl.begin - (long long)c * kC); };
    auto gates = [&](int c) {
        return reinterpret_cast<float*>(sm + OFF_GATE + (c & 1) * kGateBytes);
    };

    if (warp < 4) {
        // ============================================================ scores
        if (kOut) {
            for (int c = 0; c < nchunks; ++c) {
                if (!wait(b_gfull + 8 * (c & 1), c >> 1)) break;
                const float* gt = gates(c);
                const float loc = gt[row];
                float f[4];   // what the suffix of block b lacks to reach this row
                f[3] = 1.f;
                const float pre = expf(loc);
#pragma unroll
                for (int b = 0; b < 3; ++b) {
                    float between = 0.f;
#pragma unroll
                    for (int m = 1; m < 3; ++m)
                        if (m > b && m < warp) between += gt[2 * kC + m];
                    f[b] = pre * expf(between);
                }
                if (!wait(b_p, c)) break;
                // the bf16 scores are free once the previous chunk's P V is done
                if (c > 0 && !wait(b_o, c - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t pk[16];
                    if (b > warp) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = 0u;
                    } else {
                        float x[32];
                        tmem_ld32(tbase + lq + TM_P + 32 * b, x);
                        tmem_ld_wait();
                        const float* at = gt + 32 * b + (b < warp ? kC : 0);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(at + i);
                            const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[i + e] = b < warp ? x[i + e] * (f[b] * z[e])
                                           : i + e <= lane ? x[i + e] * __expf(loc - z[e])
                                                           : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = pack2(x[2 * i], x[2 * i + 1]);
                    }
                    tmem_st16u(tbase + lq + TM_PB + 16 * b, pk);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(b_pb);
                __syncwarp();
                if (lane == 0) mbar_arrive(b_gempty + 8 * (c & 1));
            }
        }
    } else if (warp < 8) {
        // ============================================================ state
        const size_t unit = (size_t)p.dk * p.dv;
        const size_t at = (size_t)row * p.dv + j0;
        const float* init = nullptr;
        if (kOut)
            init = sl.seg > 0 ? p.seg_state + ((size_t)g * p.H + h) * unit
                              : (p.h0 ? p.h0 + ((size_t)sl.n * p.H + h) * unit : nullptr);
        float S[kNV];
#pragma unroll
        for (int i = 0; i < kNV; i += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (init && row < p.dk && j0 + i < p.dv)
                x = *reinterpret_cast<const float4*>(init + at + i);
            S[i] = x.x, S[i + 1] = x.y, S[i + 2] = x.z, S[i + 3] = x.w;
        }
        auto publish = [&] {   // bf16 S, row `row`
            uint8_t* to = sm + OFF_SB + row * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(to + ((i ^ (row & 7)) << 4)) =
                    make_uint4(pack2(S[8 * i], S[8 * i + 1]), pack2(S[8 * i + 2], S[8 * i + 3]),
                               pack2(S[8 * i + 4], S[8 * i + 5]), pack2(S[8 * i + 6], S[8 * i + 7]));
            fence_proxy_async();
            mbar_arrive(b_s);
        };
        if (kOut && nchunks > 0) publish();
        float decay = 0.f;   // log of the product over the walk (states only)
        int c = 0;
        for (; c < nchunks; ++c) {
            if (!wait(b_gfull + 8 * (c & 1), c >> 1)) break;
            const float4 tot = *reinterpret_cast<const float4*>(gates(c) + 2 * kC);
            const float sum = (tot.x + tot.y) + (tot.z + tot.w);
            const float e = expf(sum);
            decay += sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gempty + 8 * (c & 1));
            if (!wait(b_kv, c)) break;
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[32], y[32];
                // the smallest terms first
                tmem_ld32(tbase + lq + TM_KV + 128 + 32 * half, x);
                tmem_ld32(tbase + lq + TM_KV + 64 + 32 * half, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] += y[i];
                tmem_ld32(tbase + lq + TM_KV + 32 * half, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    S[32 * half + i] = fmaf(e, S[32 * half + i], x[i] + y[i]);
            }
            tc_fence_before();
            mbar_arrive(b_kvfree);
            if (kOut && c + 1 < nchunks) {
                if (!wait(b_sfree, c)) break;
                publish();
            }
        }
        float* out = kOut ? (sl.last && p.hT ? p.hT + ((size_t)sl.n * p.H + h) * unit : nullptr)
                          : p.seg_state + ((size_t)g * p.H + h) * unit;
        if (out && c == nchunks && row < p.dk) {
#pragma unroll
            for (int i = 0; i < kNV; i += 4)
                if (j0 + i < p.dv)
                    *reinterpret_cast<float4*>(out + at + i) =
                        make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        }
        if (!kOut && tile == 0 && row == 0) p.seg_decay[(size_t)g * p.H + h] = expf(decay);
    } else if (warp < 12) {
        // ============================================================ values and outputs
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o);
        auto store = [&](int c, float er) -> bool {
            if (!wait(b_o, c)) return false;
            tc_fence_after();
            const bool mine = row < rows_of(c);
            __nv_bfloat16* to =
                o + ((sl.begin + (long long)c * kC + row) * p.H + h) * (long long)p.dv + j0;
            uint32_t pk[32];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[32], y[32];
                tmem_ld32(tbase + lq + TM_O1 + 32 * half, x);
                tmem_ld32(tbase + lq + TM_O2 + 32 * half, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    pk[16 * half + i] = pack2(fmaf(er, y[2 * i], x[2 * i]),
                                              fmaf(er, y[2 * i + 1], x[2 * i + 1]));
            }
            tc_fence_before();
            mbar_arrive(b_ofree);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (mine && j0 + 8 * i < p.dv)
                    *reinterpret_cast<uint4*>(to + 8 * i) =
                        make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
            return true;
        };
        float er_last = 0.f;
        bool ok = true;
        for (int c = 0; c < nchunks; ++c) {
            ok = wait(b_gfull + 8 * (c & 1), c >> 1) && wait(b_full + 8 * (c & 1), c >> 1);
            if (!ok) break;
            const float* gt = gates(c);
            const int block = row >> 5;
            float before = 0.f, behind = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float t = gt[2 * kC + m];
                if (m < block) before += t;
                if (m > block) behind += t;
            }
            const float er = expf(before) * expf(gt[row]);
            const float ek = expf(behind) * gt[kC + row];
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gempty + 8 * (c & 1));
            // the decayed V is free once the previous chunk's product is done
            ok = c == 0 || wait(b_kv, c - 1);
            if (!ok) break;
            const uint8_t* v = sm + (c & 1) * kStage + ST_V + row * 128;
            uint8_t* vh = sm + OFF_VH + row * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t ch = (uint32_t)(i ^ (row & 7)) << 4;
                const uint4 u = *reinterpret_cast<const uint4*>(v + ch);
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                uint32_t t[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a = ek * lo_bf(in[e]), b = ek * hi_bf(in[e]);
#pragma unroll
                    for (int m = 0; m < 3; ++m) {
                        t[m][e] = pack2(a, b);
                        a -= lo_bf(t[m][e]);
                        b -= hi_bf(t[m][e]);
                    }
                }
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    *reinterpret_cast<uint4*>(vh + m * kPanel + ch) =
                        make_uint4(t[m][0], t[m][1], t[m][2], t[m][3]);
            }
            fence_proxy_async();
            mbar_arrive(b_vh);
            if (kOut && c > 0 && !(ok = store(c - 1, er_last))) break;
            er_last = er;
        }
        if (kOut && ok && nchunks > 0) store(nchunks - 1, er_last);
    } else if (warp == kLoadWarp) {
        // ============================================================ loader
        const uint32_t bytes = (kOut ? 5u : 3u) * kPanel;
        for (int c = 0; c < nchunks; ++c) {
            const int s = c & 1;
            if (args.debug_stall && !wait(b_tail, 0)) break;
            if (c >= 2 && !wait(b_empty + 8 * s, (c >> 1) - 1)) break;
            const int valid = rows_of(c);
            const uint32_t st = sb + s * kStage, bar = valid < kC ? b_tail : b_full + 8 * s;
            if (lane == 0) {
                const int t = (int)(sl.begin + (long long)c * kC);
                mbar_arrive_expect_tx(bar, bytes);
                tma_load_3d(st + ST_K, &maps.k, bar, 0, hk, t);
                tma_load_3d(st + ST_K + kPanel, &maps.k, bar, 64, hk, t);
                tma_load_3d(st + ST_V, &maps.v, bar, j0, h, t);
                if (kOut) {
                    tma_load_3d(st + ST_Q, &maps.q, bar, 0, hk, t);
                    tma_load_3d(st + ST_Q + kPanel, &maps.q, bar, 64, hk, t);
                }
            }
            __syncwarp();
            if (valid < kC) {   // a sequence's last chunk
                if (!wait(b_tail, 0)) break;
                uint8_t* at = sm + s * kStage + ST_K;   // k's two panels, then v's
                const int vecs = (kC - valid) * 8;      // 16-byte pieces per panel
                for (int m = 0; m < 3; ++m)
                    for (int i = lane; i < vecs; i += 32)
                        *reinterpret_cast<uint4*>(at + m * kPanel + valid * 128 + i * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_full + 8 * s);
            }
        }
        // copies in flight land before the shared memory goes away (bounded; a completed phase
        // returns at once)
        for (int c = max(0, nchunks - 2); c < nchunks; ++c)
            mbar_wait(rows_of(c) < kC ? b_tail : b_full + 8 * (c & 1),
                      rows_of(c) < kC ? 0u : (uint32_t)((c >> 1) & 1), args.budget);
    } else if (warp == kMmaWarp) {
        // ============================================================ products
        const uint64_t dK = sw128_desc(0, 16, 1024);          // K-major
        const uint64_t dM = sw128_desc(0, kPanel, 1024);      // MN-major, 128-row panels
        const uint32_t id_qk = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, kNV, 0, 1),
                       id_kv = idesc_bf16(128, 3 * kNV, 1, 1);
        auto scores = [&](int c) -> bool {
            if (!wait(b_full + 8 * (c & 1), c >> 1)) return false;
            tc_fence_after();
            const uint32_t st = sb + (c & 1) * kStage;
#pragma unroll
            for (int s = 0; s < 8; ++s)
                umma_f16_warp(tbase + TM_P,
                              desc_at(dK, st + ST_Q + (s >> 2) * kPanel + (s & 3) * 32),
                              desc_at(dK, st + ST_K + (s >> 2) * kPanel + (s & 3) * 32), id_qk,
                              s > 0);
            umma_commit_warp(b_p);
            return true;
        };
        int done = 0;   // chunks whose products were all issued
        if (!kOut || nchunks == 0 || scores(0)) {
            for (int c = 0; c < nchunks; ++c) {
                const uint32_t st = sb + (c & 1) * kStage;
                if (!wait(b_vh, c)) break;
                if (c > 0 && !wait(b_kvfree, c - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    umma_f16_warp(tbase + TM_KV, desc_at(dM, st + ST_K + 2048 * s),
                                  desc_at(dM, sb + OFF_VH + 2048 * s), id_kv, s > 0);
                umma_commit_warp(b_kv);
                if (kOut) {
                    if (!wait(b_s, c)) break;
                    if (c > 0 && !wait(b_ofree, c - 1)) break;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        umma_f16_warp(tbase + TM_O2,
                                      desc_at(dK, st + ST_Q + (s >> 2) * kPanel + (s & 3) * 32),
                                      desc_at(dM, sb + OFF_SB + 2048 * s), id_o, s > 0);
                    umma_commit_warp(b_sfree);
                    if (!wait(b_pb, c)) break;
                    tc_fence_after();
                    if (c + 1 < nchunks && !scores(c + 1)) break;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        umma_f16_ts_warp(tbase + TM_O1, tbase + TM_PB + 8 * s,
                                         desc_at(dM, st + ST_V + 2048 * s), id_o, s > 0);
                    umma_commit_warp(b_o);
                }
                umma_commit_warp(b_empty + 8 * (c & 1));
                done = c + 1;
            }
        }
        // every product issued is finished before TMEM and the shared memory go away: the last
        // commit, and on the way out after an expired wait one more for what was issued since
        if (done == nchunks) {
            if (nchunks > 0) mbar_wait(b_empty + 8 * ((nchunks - 1) & 1),
                                       (uint32_t)(((nchunks - 1) >> 1) & 1), args.budget);
        } else {
            umma_commit_warp(b_empty + 8 * (done & 1));
            mbar_wait(b_empty + 8 * (done & 1), (uint32_t)((done >> 1) & 1), args.budget);
        }
    } else {
        // ============================================================ gates
        float x[4], nx[4];
        auto fetch = [&](int c, float (&to)[4]) {
            const int valid = c < nchunks ? rows_of(c) : 0;
            const long long t = sl.begin + (long long)c * kC + 4 * lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = 0.f;
                if (4 * lane + e < valid) y = p.log_g[p.gate_head ? h : (t + e) * p.H + h];
                to[e] = y < -110.f ? -110.f : y;
            }
        };
        fetch(0, x);
        for (int c = 0; c < nchunks; ++c) {
            fetch(c + 1, nx);
            if (c >= 2 && !wait(b_gempty + 8 * (c & 1), (c >> 1) - 1)) break;
            float* gt = gates(c);
            // inclusive prefix and exclusive suffix sums in the lane's 32-row block (8 lanes)
            const float a1 = x[0] + x[1], a2 = a1 + x[2], all = a2 + x[3];
            float up = all, down = all;
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, up, off, 8);
                const float d = __shfl_down_sync(0xffffffffu, down, off, 8);
                if ((lane & 7) >= off) up += u;
                if ((lane & 7) + off < 8) down += d;
            }
            float pre = __shfl_up_sync(0xffffffffu, up, 1, 8);
            float suf = __shfl_down_sync(0xffffffffu, down, 1, 8);
            if ((lane & 7) == 0) pre = 0.f;
            if ((lane & 7) == 7) suf = 0.f;
            *reinterpret_cast<float4*>(gt + 4 * lane) =
                make_float4(pre + x[0], pre + a1, pre + a2, pre + all);
            const float s2 = suf + x[3], s1 = s2 + x[2], s0 = s1 + x[1];
            *reinterpret_cast<float4*>(gt + kC + 4 * lane) =
                make_float4(expf(s0), expf(s1), expf(s2), expf(suf));
            if ((lane & 7) == 0) gt[2 * kC + (lane >> 3)] = down;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gfull + 8 * (c & 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = nx[e];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, kTmemCols);
}

long long wait_budget() {
    static const long long budget = [] {
        const char* s = std::getenv("KDA_DEBUG_WAIT_CYCLES");
        const long long v = s && *s ? std::atoll(s) : 0;
        return v > 0 ? v : 1ll << 31;   // about one second of SM clock
    }();
    return budget;
}

int debug_stall() {
    static const int v = [] {
        const char* s = std::getenv("KDA_DEBUG_STALL_WAIT");
        return s && *s && *s != '0' ? 1 : 0;
    }();
    return v;
}

PerDevice g_setup;

}  // namespace

bool linear_chunk_takes(bool bf16, int dk, int dv) {
    return bf16 && dk <= 128 && dk % 8 == 0 && dv % 8 == 0;
}

cudaError_t launch_linear_chunk(const LinearParams& p, LinearPass pass, cudaStream_t stream) {
    cudaError_t e = g_setup.run([](int) {
        const cudaError_t a = cudaFuncSetAttribute(
            linear_chunk_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (a != cudaSuccess) return a;
        return cudaFuncSetAttribute(linear_chunk_kernel<false>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess) return e;
    ChunkArgs a{p, (p.dv + kNV - 1) / kNV, wait_budget(), debug_stall()};
    const long long blocks = (long long)p.slots * p.H * a.tiles;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    ChunkMaps m;
    const unsigned long long rows = (unsigned long long)p.B * p.T;
    auto map = [&](CUtensorMap* t, const void* base, int heads, int cols) {
        return make_map_3d_box(t, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, heads, cols, 64,
                               kC, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if ((e = map(&m.q, p.q, p.Hk, p.dk)) != cudaSuccess ||
        (e = map(&m.k, p.k, p.Hk, p.dk)) != cudaSuccess ||
        (e = map(&m.v, p.v, p.H, p.dv)) != cudaSuccess)
        return e;
    if (pass == LinearPass::kStates)
        linear_chunk_kernel<false><<<(unsigned)blocks, kThreads, kSmem, stream>>>(m, a);
    else
        linear_chunk_kernel<true><<<(unsigned)blocks, kThreads, kSmem, stream>>>(m, a);
    return cudaGetLastError();
}

}  // namespace kda
