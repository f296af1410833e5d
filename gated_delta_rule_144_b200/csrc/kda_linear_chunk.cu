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
//     what fp32 holds, so the decayed v is split into three bf16 terms (8 bits each, 2^-25 left).
//     The products of the first and of the two small terms are summed apart and meet in fp32.
//   - q S reads the state rounded to bf16, and the decayed scores are rounded to bf16: each 2^-9
//     of a term at most, as the output's own rounding, on disjoint parts of the output.
//   - Gate sums are held in powers of two. Decays are products of gates <= 1: a pair of rows in
//     different 32-row blocks takes (suffix of j's block) (blocks between) (prefix of i's block),
//     so no exponential grows and none is taken of a difference of large sums; inside a block
//     G_i - G_j is a difference of sums over at most 32 rows. Gates below -110 count as -110, whose
//     exponential is 0 in fp32 like that of anything below.
//
// Roles (16 warps), which meet through mbarriers only:
//   warps 0-3   scores: P = Q K^T out of TMEM, times the decays, rounded to bf16 into TMEM, where
//               P V takes its left operand (row i is TMEM lane i; a warp is a 32-row block); then
//               the chunk before's output, o = P V + e^G (Q S), out of TMEM, staged in shared
//               memory and stored by TMA (a sequence's last, partial chunk row by row)
//   warps 4-7   state: lane i holds row i of S, 64 columns in registers; adds a chunk's
//               partial products and writes S as bf16 to shared memory for the next Q S
//   warps 8-11  values: the three terms of the decayed V to shared memory, 32 rows at a time in
//               two buffers, so that one is written while the other is multiplied (without
//               outputs warps 0-3 take half of them, in four buffers)
//   warp 12     loader: q, k, v by TMA, two stages. It clears the rows of k and v behind a
//               sequence's end (they are another's), so that nothing of them enters a product
//   warp 13     issues the state's products, warp 14 the scores', Q S and P V
//   warp 15     gates: block-wise prefix and suffix sums, a chunk ahead
// The loops over pieces of a tile are mostly not unrolled: every role runs its code once per
// chunk, all at the same time, and the kernel is bound by instruction fetch where their sum
// outgrows the cache (132 KB of code ran a chunk in 7.2 us, the same loops rolled up, 77 KB, in
// 3.3 us).
// Bound: shared memory. A chunk of a CTA takes about 3690 cycles, of which about 3375 move operands,
// decayed V, state and output through it. 2 x 65536 tokens x 32 heads x 128 x 128 take 1.36 to 1.37
// ms in a long run (0.48 of the measured copy rate), where the power limit holds the clock down, and
// 1.08 to 1.27 in the first tens of calls; eight packed documents of 28937 tokens, 32 heads of 64
// columns 168 us (150 as a replayed graph); one prompt of 4096 tokens x 16 heads 49 us (47). Not kept,
// on the first of these, a few calls at a time: tiles fetched
// into L2 two chunks ahead 1.15 (against 1.10), one product of 192 columns for all terms 1.36
// (1.15), the last quarter of the values by the state warps 1.30 (1.15), outputs stored by each warp
// for itself 1.23 (1.14).
// TMEM: P 128 columns, bf16 P 64, P V 64, Q S 2 x 64, the state's terms 2 x 64: all 512. Shared
// memory: 2 x 80 KiB of stages, 24 KiB of decayed V, 16 KiB of bf16 state, 16 KiB of output.
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
constexpr int kThreads = 16 * 32;
constexpr int kLoadWarp = 12, kStateMma = 13, kOutMma = 14;   // the last warp is the gates'

constexpr uint32_t kPanel = 16384;      // 128 rows x 128 bytes, 128-byte swizzle
constexpr uint32_t ST_Q = 0, ST_K = 2 * kPanel, ST_V = 4 * kPanel, kStage = 5 * kPanel;
constexpr uint32_t kQuarter = kPanel / 4;           // 32 rows of one term of the decayed V
constexpr uint32_t kVH = 3 * kQuarter;
constexpr uint32_t OFF_VH = 2 * kStage;             // two buffers of 32 rows of the three terms (four
                                                    // without outputs: also what follows)
constexpr uint32_t OFF_SB = OFF_VH + 2 * kVH;       // bf16 state
constexpr uint32_t OFF_OUT = OFF_SB + kPanel;       // output on its way to global memory
constexpr uint32_t OFF_GATE = OFF_OUT + kPanel;      // per stage: loc[128], suf[128], tot[4]
constexpr uint32_t kGateBytes = (2 * kC + 4) * 4;
// A CTA's search for its slot runs in the gates' area, which plain stores alone write: a plain store
// to a stage would need a proxy fence before the TMA copies there.
constexpr uint32_t OFF_FIND = OFF_GATE;
constexpr uint32_t OFF_BAR = OFF_GATE + 2 * kGateBytes;
constexpr uint32_t OFF_MISC = OFF_BAR + 34 * 8;     // TMEM address, abort flag
constexpr uint32_t kSmem = OFF_MISC + 16;
static_assert(kSmem <= 232448, "shared memory");
static_assert(OFF_BAR % 8 == 0 && OFF_GATE % 16 == 0 && kGateBytes % 16 == 0, "alignment");

constexpr uint32_t TM_P = 0, TM_PB = 128, TM_O1 = 192, TM_O2 = 256 /* two */, TM_KV = 384;
constexpr int kTmemCols = 512;

struct ChunkArgs {
    LinearParams p;
    int tiles;              // 64-column tiles of dv
    uint32_t budget;        // cycles a wait may take
    int debug_stall;
};

struct ChunkMaps {
    CUtensorMap q, k, v, o;
};

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_bf(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// 2^x, at most 2 units in the last place off.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// mbar_wait in few instructions: a first test, then suspending ones until `budget` cycles passed.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint32_t budget) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 t0, t1;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u32 t0, %%clock;\n\t"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n\t"
        "@p bra DONE;\n\t"
        "mov.u32 t1, %%clock;\n\t"
        "sub.u32 t1, t1, t0;\n\t"
        "setp.le.u32 q, t1, %3;\n\t"
        "@q bra AGAIN;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(budget), "r"(1000000u)
        : "memory");
    return ok != 0;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ void mul2(float& a, float& b, float f) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(a), "+f"(b) : "f"(f));
}
__device__ __forceinline__ void sub2(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 x, y, m;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mov.b64 m, {%4, %4};\n\tfma.rn.f32x2 x, y, m, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b) : "f"(c), "f"(d), "f"(-1.f));
}
__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t count, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"((uint32_t)pred), "r"(id), "r"(count) : "memory");
    return r != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// What a CTA works on: segment `seg` of sequence n (rows [begin, end)), its place among the slots.
struct ChunkSlot {
    int n, seg, slot;
    long long begin, end;
    bool last;
};
constexpr int kSorted = 128;    // packed slots up to which CTAs take them longest first (a CTA ranks
                                // all of them: 32 comparisons per thread)
constexpr int kScanned = 1024;  // packed sequences up to which every CTA reads all offsets
constexpr int kFindInts = kSorted > kThreads / 32 + 2 ? kSorted : kThreads / 32 + 2;
static_assert(OFF_FIND >= OFF_OUT + kPanel && OFF_FIND + 4 * kFindInts <= OFF_BAR,
              "the search's words lie behind everything that TMA reads or writes");

// The CTA's g-th slot, found by the whole block (kStates: the g-th segment that is not its sequence's
// last); `tmp` is kFindInts ints of shared memory. Equal lengths: first segments first (they wait for
// nothing). Packed: longest first up to kSorted slots, so that no long one starts last. Every CTA
// reads all offsets, and a malformed cu_seqlens makes each of them report it and stop; above
// kScanned sequences, which are never cut into segments, each checks its own, and some CTA meets
// what is malformed. False: nothing to do.
template <bool kStates>
__device__ __forceinline__ bool chunk_slot(const LinearParams& p, int g, int tid, int* tmp,
                                           ChunkSlot* s) {
    const int L = p.seg_tokens;
    if (!p.cu_seqlens) {
        const int segs = L > 0 ? max(1, (p.T + L - 1) / L) : 1;
        s->seg = g / p.N;
        s->n = g % p.N;
        s->slot = s->n * segs + s->seg;
        const long long t0 = (long long)s->n * p.T;
        s->begin = t0 + (long long)s->seg * L;
        s->end = L > 0 ? min(t0 + p.T, s->begin + L) : t0 + p.T;
        s->last = s->seg == segs - 1;
        return true;
    }
    const int32_t* __restrict__ cu = p.cu_seqlens;
    bool bad = false;
    if (p.N > kScanned) {
        const int c0 = cu[g], c1 = cu[g + 1];
        if (c0 < 0 || c1 < c0 || c1 > p.T || (g == 0 && c0 != 0) || (g == p.N - 1 && c1 != p.T)) {
            if (tid == 0) set_device_error(p.err, DEV_BAD_SEQLENS);
            return false;
        }
        *s = ChunkSlot{g, 0, g, c0, c1, true};
        return true;
    }
    for (int i = tid; i <= p.N; i += kThreads) {
        const int c = cu[i];
        bad |= (i == 0 && c != 0) || (i == p.N && c != p.T) || (i < p.N && cu[i + 1] < c);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) set_device_error(p.err, DEV_BAD_SEQLENS);
        return false;
    }
    // slot of (n, segment 0): floor(cu[n] / L) + n, or n; rows of slot i of sequence n
    auto first = [&](int n) { return L > 0 ? cu[n] / L + n : n; };
    auto rows = [&](int n, int slot) {
        const int len = cu[n + 1] - cu[n], at = L > 0 ? (slot - first(n)) * L : 0;
        if (L <= 0 || len <= p.whole_tokens) return at == 0 ? len : -1;
        return at < len ? min(len - at, L) : -1;
    };
    if (kStates) {   // counts of such segments, summed over the sequences before each
        const int lane = tid & 31, warp = tid >> 5;
        int base = 0;
        for (int i0 = 0; i0 < p.N; i0 += kThreads) {
            const int n = i0 + tid, len = n < p.N ? cu[n + 1] - cu[n] : 0;
            const int mine = len <= p.whole_tokens ? 0 : (len - 1) / L;
            int sum = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += x;
            }
            if (lane == 31) tmp[warp] = sum;
            __syncthreads();
            int all = 0, before = base;
            for (int w = 0; w < kThreads / 32; ++w) {
                before += w < warp ? tmp[w] : 0;
                all += tmp[w];
            }
            before += sum - mine;
            if (g >= before && g < before + mine)
                tmp[kThreads / 32] = n, tmp[kThreads / 32 + 1] = g - before;
            base += all;
            __syncthreads();
        }
        if (g >= base) return false;
        s->n = tmp[kThreads / 32];
        s->seg = tmp[kThreads / 32 + 1];
        s->slot = first(s->n) + s->seg;
        s->begin = cu[s->n] + (long long)s->seg * L;
        s->end = s->begin + L;
        s->last = false;
        return true;
    }
    int slot = g;
    if (p.slots <= kSorted) {
        for (int i = tid; i < p.slots; i += kThreads) tmp[i] = -1;   // (slots that nothing uses)
        __syncthreads();
        for (int n = tid; n < p.N; n += kThreads)
            for (int i = first(n); i < p.slots; ++i) {
                const int r = rows(n, i);
                if (r < 0) break;
                tmp[i] = r;
                if (L <= 0) break;
            }
        __syncthreads();
        int mine = -1;   // the slot with g slots before it
        for (int i = tid; i < p.slots; i += kThreads) {
            const int r = tmp[i];
            int before = 0;
            for (int j = 0; j < p.slots; ++j) {
                const int x = tmp[j];
                before += x > r || (x == r && j < i);
            }
            if (before == g) mine = i;
        }
        __syncthreads();
        if (mine >= 0) tmp[0] = mine;
        __syncthreads();
        slot = tmp[0];
    }
    int below = 0;   // sequences whose first slot is not behind this one
    for (int i0 = 0; i0 < p.N; i0 += kThreads)
        below += __syncthreads_count(i0 + tid < p.N && first(i0 + tid) <= slot);
    const int n = below - 1, r = rows(n, slot);
    if (r < 0) return false;
    s->n = n;
    s->slot = slot;
    s->seg = slot - first(n);
    s->begin = cu[n] + (long long)s->seg * L;
    s->end = s->begin + r;
    s->last = s->end == cu[n + 1];
    return true;
}

// Row `row` of the state before the CTA's segment, N columns from `col`: h0, and on top of it the
// states of the segments before, or their sum from a launch of its own (seg_ready).
template <int N>
__device__ __forceinline__ void initial_state(const LinearParams& p, const ChunkSlot& sl, int h,
                                              int row, int col, float (&S)[N]) {
    const size_t unit = (size_t)p.dk * p.dv, at = (size_t)row * p.dv + col;
    auto add = [&](const float* from, float f) {   // S <- f S + what is at `from`
        if (row >= p.dk) return;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            if (col + i >= p.dv) continue;
            const float4 x = *reinterpret_cast<const float4*>(from + at + i);
            S[i] = fmaf(f, S[i], x.x), S[i + 1] = fmaf(f, S[i + 1], x.y);
            S[i + 2] = fmaf(f, S[i + 2], x.z), S[i + 3] = fmaf(f, S[i + 3], x.w);
        }
    };
    const bool ready = p.seg_ready && sl.seg > 0;
    if (sl.seg > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 1
    for (int i = ready ? 0 : sl.seg; i >= 0; --i) {
        const size_t from = (size_t)(sl.slot - i) * p.H + h;
        const bool start = i == sl.seg && !ready;
        if (start && !p.h0) continue;
        add(start ? p.h0 + ((size_t)sl.n * p.H + h) * unit
                  : p.seg_state + (ready ? from : from - p.H) * unit,
            start || ready ? 0.f : p.seg_decay[from - p.H]);
    }
}

// In P V a value that is not finite also meets the zero scores of the rows before its own, and
// 0 x NaN is NaN. The block computes the outputs of those rows (the rest of the chunk before the
// first such value of a column) again, walking the segment token by token from its initial state.
// Thread (row, group) holds 16 columns of a state row; `sm`: 64 + 4 * 64 words.
__device__ __forceinline__ void repair_rows(const LinearParams& p, const ChunkSlot& sl, int h,
                                            int j0, int tid, void* sm) {
    int* first = static_cast<int*>(sm);                      // by column: its first such token
    float(*sums)[kNV] = reinterpret_cast<float(*)[kNV]>(first + kNV);   // by warp of a group
    const int len = (int)(sl.end - sl.begin), cols = min(kNV, p.dv - j0);
    const long long vs = (long long)p.H * p.dv, ks = (long long)p.Hk * p.dk;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + sl.begin * vs +
                             (long long)h * p.dv + j0;
    const long long k0 = sl.begin * ks + (long long)(h / (p.H / p.Hk)) * p.dk;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + k0;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + k0;
    if (tid < kNV) first[tid] = len;
    __syncthreads();
    if (tid % kNV < cols)
#pragma unroll 1
        for (int t = tid / kNV; t < len; t += kThreads / kNV)
            if (!isfinite(__bfloat162float(v[t * vs + tid % kNV]))) {
                atomicMin(first + tid % kNV, t);
                break;
            }
    __syncthreads();
    int end = 0;   // tokens to walk
    for (int i = 0; i < cols; ++i)
        if (first[i] < len && first[i] % kC) end = max(end, first[i]);
    const int row = tid % kC, col = tid / kC * 16, lane = tid & 31;
    float S[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) S[i] = 0.f;
    if (end > 0) initial_state(p, sl, h, row, j0 + col, S);
#pragma unroll 1
    for (int t = 0; t < end; ++t) {
        const float g = expf(p.log_g[p.gate_head ? h : (sl.begin + t) * p.H + h]);
        const float kr = row < p.dk ? __bfloat162float(k[t * ks + row]) : 0.f;
        const float qr = row < p.dk ? __bfloat162float(q[t * ks + row]) : 0.f;
        bool any = false;   // whether a column's output is due
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            S[i] = fmaf(kr, col + i < cols ? __bfloat162float(v[t * vs + col + i]) : 0.f, g * S[i]);
            any |= t < first[col + i] && t >= first[col + i] / kC * kC;
        }
        if (!__syncthreads_or(any)) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = qr * S[i];
#pragma unroll
            for (int off = 16; off > 0; off /= 2) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (lane == 0) sums[row / 32][col + i] = x;
        }
        __syncthreads();
        if (tid < cols && t < first[tid] && t >= first[tid] / kC * kC && first[tid] < len)
            static_cast<__nv_bfloat16*>(p.o)[((sl.begin + t) * p.H + h) * p.dv + j0 + tid] =
                __float2bfloat16_rn((sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]));
    }
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
    ChunkSlot sl;
    if (!chunk_slot<!kOut>(p, g, tid, reinterpret_cast<int*>(sm + OFF_FIND), &sl)) return;
    // the outputs' launch may start now; what it reads of this one it waits for
    if (!kOut) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int nchunks = (int)((sl.end - sl.begin + kC - 1) / kC);
    const int j0 = tile * kNV;
    constexpr int kBufs = kOut ? 2 : 4;

    // barriers: each counts the chunks (pairs: one per stage or parity; b_vh: one per
    // buffer)
    const uint32_t nb = sb + OFF_BAR;
    const uint32_t b_full = nb, b_qkfree = nb + 16, b_vfree = nb + 32, b_gfull = nb + 48,
                   b_gfree = nb + 64, b_vh = nb + 208, b_vhfree = nb + 240, b_kv = nb + 80,
                   b_kvfree = nb + 96, b_p = nb + 120, b_pb = nb + 128, b_s = nb + 136,
                   b_sfree = nb + 144, b_o = nb + 152, b_ofree = nb + 160, b_tail = nb + 168,
                   b_vfull = nb + 176;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(sm + OFF_MISC);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_full + 8 * i, 1);                 // q, k
            mbar_init(b_vfull + 8 * i, 1);
            mbar_init(b_qkfree + 8 * i, kOut ? 2 : 1);    // both issuing warps have read
            mbar_init(b_vfree + 8 * i, 1);
            mbar_init(b_gfull + 8 * i, 1);
            mbar_init(b_gfree + 8 * i, 12);               // one per reading warp
            mbar_init(b_kv + 8 * i, 1);
            mbar_init(b_kvfree + 8 * i, 128);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(b_vh + 8 * i, 128);
            mbar_init(b_vhfree + 8 * i, 1);
        }
        mbar_init(b_p, 1);
        mbar_init(b_pb, 128);
        mbar_init(b_s, 128);
        mbar_init(b_sfree, 1);
        mbar_init(b_o, 1);
        mbar_init(b_ofree, 128);
        mbar_init(b_tail, 1);
        fence_mbar_init();
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
        if (kOut) prefetch_tmap(&maps.o);
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
    bool failed = false;
    bool spoilt = false;   // the state at the end is not finite
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool ok = __all_sync(0xffffffffu, wait_phase(bar, parity & 1u, args.budget));
        failed = !ok;
        return ok;
    };
    auto rows_of = [&](int c) { return (int)min((long long)kC, sl.end - sl.begin - (long long)c * kC); };
    auto gates = [&](int c) {
        return reinterpret_cast<float*>(sm + OFF_GATE + (c & 1) * kGateBytes);
    };
    // a chunk's state terms in TMEM: alternating places where nothing else needs them
    auto kv_at = [&](int c) { return tbase + (kOut || !(c & 1) ? TM_KV : 0u); };

    // The values' role: the decayed V of the 32-row quarters q0, q0 + kStep, ...: lane r takes row r,
    // the warp 16 of the columns.
    constexpr int kStep = kOut ? 1 : 2;
    auto values = [&](int q0) {
        const int v0 = 2 * (warp & 3);   // first 16-byte piece
#pragma unroll 1
        for (int c = 0; c < nchunks; ++c) {
            if (!wait(b_gfull + 8 * (c & 1), c >> 1)) break;
            const float* gt = gates(c);
            float ek[4], behind = 1.f;
#pragma unroll
            for (int q = 3; q >= 0; --q) {
                ek[q] = behind * gt[kC + 32 * q + lane];
                behind *= ex2(gt[2 * kC + q]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gfree + 8 * (c & 1));
            if (!wait(b_vfull + 8 * (c & 1), c >> 1)) break;
            const uint8_t* v = sm + (c & 1) * kStage + ST_V + lane * 128;
            bool ok = true;
#pragma unroll 1
            for (int q = q0; q < 4; q += kStep) {
                // a buffer's use u follows the product that read use u - 1
                const int b = q & (kBufs - 1), u = kOut ? 2 * c + (q >> 1) : c;
                ok = u == 0 || wait(b_vhfree + 8 * b, u - 1);
                if (!ok) break;
                uint8_t* vh = sm + OFF_VH + b * kVH + lane * 128;
                const float f = q < 2 ? (q == 0 ? ek[0] : ek[1]) : (q == 2 ? ek[2] : ek[3]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t ch = (uint32_t)((v0 + i) ^ (lane & 7)) << 4;
                    const uint4 x = *reinterpret_cast<const uint4*>(v + q * kQuarter + ch);
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                    uint32_t t[3][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a = lo_bf(in[e]), b = hi_bf(in[e]);
                        mul2(a, b, f);
#pragma unroll
                        for (int m = 0; m < 3; ++m) {
                            t[m][e] = pack2(a, b);
                            if (m < 2) sub2(a, b, lo_bf(t[m][e]), hi_bf(t[m][e]));
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        *reinterpret_cast<uint4*>(vh + m * kQuarter + ch) =
                            make_uint4(t[m][0], t[m][1], t[m][2], t[m][3]);
                }
                fence_proxy_async();
                mbar_arrive(b_vh + 8 * b);
            }
            if (!ok) break;
        }
    };

    if (warp < 4) {
        // ============================================================ scores
        if (!kOut) values(0);
        // chunk c's scores, then, while chunk c + 1's are multiplied, chunk c - 1's output
        const uint32_t pb = tbase + lq + TM_PB;
        float er_last = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; kOut && nchunks > 0 && c <= nchunks; ++c) {
            float er = 0.f;
            if (c < nchunks) ok = ok && wait(b_gfull + 8 * (c & 1), c >> 1) && wait(b_p, c);
            // P V of the chunk before is done: its bf16 scores' columns are free and its output
            // is there
            if (c > 0) ok = ok && wait(b_o, c - 1);
            tc_fence_after();
            if (ok && c < nchunks) {
                const float* gt = gates(c);
                const float loc = gt[row], pre = ex2(loc);
                // the blocks before this row's: what the suffix of block b lacks to reach the row
                float between = 1.f;
#pragma unroll 1
                for (int b = warp - 1; b >= 0; --b) {
                    float x[32];
                    tmem_ld32(tbase + lq + TM_P + 32 * b, x);
                    const float f = pre * between;
                    between *= ex2(gt[2 * kC + b]);
                    const float* at = gt + kC + 32 * b;
                    uint32_t pk[16];
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 y = *reinterpret_cast<const float4*>(at + i);
                        pk[i / 2] = pack2(x[i] * (f * y.x), x[i + 1] * (f * y.y));
                        pk[i / 2 + 1] = pack2(x[i + 2] * (f * y.z), x[i + 3] * (f * y.w));
                    }
                    tmem_st16u(pb + 16 * b, pk);
                }
                er = pre * between;
                {   // the row's own block
                    float x[32];
                    tmem_ld32(tbase + lq + TM_P + 32 * warp, x);
                    const float* at = gt + 32 * warp;
                    uint32_t pk[16];
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 y = *reinterpret_cast<const float4*>(at + i);
                        const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[i + e] = i + e <= lane ? x[i + e] * ex2(loc - z[e]) : 0.f;
                        pk[i / 2] = pack2(x[i], x[i + 1]);
                        pk[i / 2 + 1] = pack2(x[i + 2], x[i + 3]);
                    }
                    tmem_st16u(pb + 16 * warp, pk);
                }
                if (c == 0) {   // the blocks behind stay zero: no later chunk writes them
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = 0u;
#pragma unroll 1
                    for (int b = warp + 1; b < 4; ++b) tmem_st16u(pb + 16 * b, pk);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(b_pb);
                __syncwarp();
                if (lane == 0) mbar_arrive(b_gfree + 8 * (c & 1));
            }
            if (c > 0) {   // o = P V + e^G (Q S) of chunk c - 1, staged in shared memory
                if (tid == 0) bulk_wait_read_all();   // the previous output has left it
                // (the four warps go on together: one whose wait expired comes here too)
                if (bar_or(1, 128, !ok)) break;
                uint8_t* to = sm + OFF_OUT + row * 128;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float x[32], y[32];
                    tmem_ld32(tbase + lq + TM_O1 + 32 * hf, x);
                    tmem_ld32(tbase + lq + TM_O2 + 64 * ((c - 1) & 1) + 32 * hf, y);
                    tmem_ld_wait();
                    if (hf == 1) {
                        tc_fence_before();
                        mbar_arrive(b_ofree);
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = pack2(fmaf(er_last, y[2 * i], x[2 * i]),
                                      fmaf(er_last, y[2 * i + 1], x[2 * i + 1]));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(to + (((4 * hf + i) ^ (row & 7)) << 4)) =
                            make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                }
                const int valid = rows_of(c - 1);
                const long long t = sl.begin + (long long)(c - 1) * kC;
                if (valid == kC) {
                    fence_proxy_async();
                    bar_sync(1, 128);
                    if (tid == 0) {
                        tma_store_3d(&maps.o, sb + OFF_OUT, j0, h, (int)t);
                        bulk_commit();
                    }
                } else if (row < valid) {   // not the rows behind the sequence's end
                    __nv_bfloat16* g = static_cast<__nv_bfloat16*>(p.o) +
                                       ((t + row) * p.H + h) * (long long)p.dv + j0;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i)
                        if (j0 + 8 * i < p.dv)
                            *reinterpret_cast<uint4*>(g + 8 * i) =
                                *reinterpret_cast<const uint4*>(to + ((i ^ (row & 7)) << 4));
                }
            }
            er_last = er;
        }
        if (kOut && tid == 0) bulk_wait_read_all();
    } else if (warp < 8) {
        // ============================================================ state
        const size_t unit = (size_t)p.dk * p.dv;
        const size_t at = (size_t)row * p.dv + j0;
        float S[kNV];
#pragma unroll
        for (int i = 0; i < kNV; ++i) S[i] = 0.f;
        if (kOut) initial_state(p, sl, h, row, j0, S);
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
#pragma unroll 1
        for (; c < nchunks; ++c) {
            if (!wait(b_gfull + 8 * (c & 1), c >> 1)) break;
            const float4 tot = *reinterpret_cast<const float4*>(gates(c) + 2 * kC);
            const float sum = (tot.x + tot.y) + (tot.z + tot.w);
            const float e = exp2f(sum);
            decay += sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gfree + 8 * (c & 1));
            if (!wait(b_kv + 8 * (c & 1), c >> 1)) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[16], y[16];
                tmem_ld16(kv_at(c) + lq + 16 * q, x);
                tmem_ld16(kv_at(c) + lq + 64 + 16 * q, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    S[16 * q + i] = fmaf(e, S[16 * q + i], x[i] + y[i]);
            }
            tc_fence_before();
            mbar_arrive(b_kvfree + 8 * (c & 1));
            if (kOut && c + 1 < nchunks) {
                if (!wait(b_sfree, c)) break;
                publish();
            }
        }
        float zero = 0.f;
#pragma unroll
        for (int i = 0; kOut && i < kNV; ++i) zero = fmaf(0.f, S[i], zero);
        spoilt = zero != 0.f && !failed;
        float* out = kOut ? (sl.last && p.hT ? p.hT + ((size_t)sl.n * p.H + h) * unit : nullptr)
                          : p.seg_state + ((size_t)sl.slot * p.H + h) * unit;
        if (out && !failed && row < p.dk) {
#pragma unroll
            for (int i = 0; i < kNV; i += 4)
                if (j0 + i < p.dv)
                    *reinterpret_cast<float4*>(out + at + i) =
                        make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        }
        if (!kOut && tile == 0 && row == 0) p.seg_decay[(size_t)sl.slot * p.H + h] = exp2f(decay);
    } else if (warp < 12) {
        // ============================================================ values
        values(kOut ? 0 : 1);
    } else if (warp == kLoadWarp) {
        // ============================================================ loader
        // Loads of a chunk follow its stage's release, a chunk before their use. (Fetching the tiles
        // into L2 two chunks before that as well: 1.15 ms against 1.10 on the long-context case.)
        constexpr int kBoxes = kOut ? 4 : 2;   // k's two panels, then q's
        auto place = [&](int m) { return m < 2 ? ST_K + m * kPanel : ST_Q + (m - 2) * kPanel; };
#pragma unroll 1
        for (int c = 0; c < nchunks; ++c) {
            const int s = c & 1;
            if (args.debug_stall && !wait(b_tail, 0)) break;
            if (c >= 2 && !wait(b_qkfree + 8 * s, (c >> 1) - 1)) break;
            const int valid = rows_of(c);
            const int t = (int)(sl.begin + (long long)c * kC);
            const uint32_t st = sb + s * kStage;
            if (lane == 0) {
                const uint32_t bar = valid < kC ? b_tail : b_full + 8 * s;
                mbar_arrive_expect_tx(bar, (kBoxes + (valid < kC ? 1 : 0)) * kPanel);
#pragma unroll 1
                for (int m = 0; m < kBoxes; ++m)
                    tma_load_3d(st + place(m), m < 2 ? &maps.k : &maps.q, bar, 64 * (m & 1), hk, t);
            }
            __syncwarp();
            if (c >= 2 && !wait(b_vfree + 8 * s, (c >> 1) - 1)) break;
            if (lane == 0) {
                const uint32_t bar = valid < kC ? b_tail : b_vfull + 8 * s;
                if (valid == kC) mbar_arrive_expect_tx(bar, kPanel);
                tma_load_3d(st + ST_V, &maps.v, bar, j0, h, t);
            }
            __syncwarp();
            if (valid < kC) {   // a sequence's last chunk
                if (!wait(b_tail, 0)) break;
                uint8_t* at = sm + s * kStage + ST_K;   // k's two panels, then v's
                const int vecs = (kC - valid) * 8;      // 16-byte pieces per panel
#pragma unroll 1
                for (int m = 0; m < 3; ++m)
#pragma unroll 1
                    for (int i = lane; i < vecs; i += 32)
                        *reinterpret_cast<uint4*>(at + m * kPanel + valid * 128 + i * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(b_full + 8 * s);
                    mbar_arrive(b_vfull + 8 * s);
                }
            }
        }
        // copies in flight land before the shared memory goes away (bounded; a completed phase
        // returns at once)
#pragma unroll 1
        for (int c = max(0, nchunks - 2); c < nchunks; ++c) {
            const uint32_t par = (uint32_t)((c >> 1) & 1);
            if (rows_of(c) < kC) {
                wait_phase(b_tail, 0u, args.budget);
            } else {
                wait_phase(b_full + 8 * (c & 1), par, args.budget);
                wait_phase(b_vfull + 8 * (c & 1), par, args.budget);
            }
        }
    } else if (warp == kStateMma) {
        // ============================================================ the state's products
        const uint64_t dM = sw128_desc(0, kPanel, 1024);         // MN-major, 128-row panels
        const uint64_t dV = sw128_desc(0, kQuarter, 1024);       // MN-major, 32-row panels
        const uint32_t id2 = idesc_bf16(128, 2 * kNV, 1, 1), id1 = idesc_bf16(128, kNV, 1, 1);
        int c = 0;
        bool ok = true;
#pragma unroll 1
        for (; c < nchunks; ++c) {
            uint32_t k = sb + (c & 1) * kStage + ST_K;
            // (kOut: one place for the terms, free once chunk c - 1's were read; else c - 2's)
            const int before = c - (kOut ? 1 : 2);
            ok = wait(b_full + 8 * (c & 1), c >> 1) &&
                 (before < 0 || wait(b_kvfree + 8 * (before & 1), before >> 1));
            const uint32_t kv = kv_at(c);
#pragma unroll 1
            for (int q = 0; ok && q < 4; ++q) {
                const int b = q & (kBufs - 1);
                ok = wait(b_vh + 8 * b, kOut ? 2 * c + (q >> 1) : c);
                if (!ok) break;
                tc_fence_after();
                uint32_t v = sb + OFF_VH + b * kVH;
                // the first two terms side by side, then the third onto the second's sum
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    umma_f16_warp(kv, desc_at(dM, k), desc_at(dV, v), id2, q > 0 || s > 0);
                    umma_f16_warp(kv + kNV, desc_at(dM, k), desc_at(dV, v + 2 * kQuarter),
                                  id1, 1);
                    k += 2048;
                    v += 2048;
                }
                umma_commit_warp(b_vhfree + 8 * b);
            }
            if (!ok) break;
            umma_commit_warp(b_kv + 8 * (c & 1));
            umma_commit_warp(b_qkfree + 8 * (c & 1));
            if (!kOut) umma_commit_warp(b_vfree + 8 * (c & 1));
        }
        // every product issued is finished before TMEM and the shared memory go away: the last
        // chunk's, or, on the way out after an expired wait, what this last commit covers
        if (c < nchunks) umma_commit_warp(b_kv + 8 * (c & 1));
        if (nchunks > 0) {
            const int last = min(c, nchunks - 1);
            wait_phase(b_kv + 8 * (last & 1), (uint32_t)((last >> 1) & 1), args.budget);
        }
    } else if (warp == kOutMma) {
        // ============================================================ scores, Q S and P V
        const uint64_t dK = sw128_desc(0, 16, 1024);          // K-major
        const uint64_t dM = sw128_desc(0, kPanel, 1024);      // MN-major, 128-row panels
        const uint32_t id_qk = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, kNV, 0, 1);
        // iteration c issues chunk c's Q S, which frees its q and k; then, as soon as the score
        // warps have read chunk c's scores, chunk c + 1's; then chunk c's P V
        int c = kOut && nchunks > 0 ? -1 : nchunks;
#pragma unroll 1
        for (; c < nchunks; ++c) {
            const uint32_t st = sb + (c & 1) * kStage, sn = sb + ((c + 1) & 1) * kStage;
            if (c >= 0) {
                if (!wait(b_s, c)) break;
                tc_fence_after();   // (its columns of O2 are free: P V of c - 1 went after their reader)
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    umma_f16_warp(tbase + TM_O2 + 64 * (c & 1),
                                  desc_at(dK, st + ST_Q + (s >> 2) * kPanel + (s & 3) * 32),
                                  desc_at(dM, sb + OFF_SB + 2048 * s), id_o, s > 0);
                umma_commit_warp(b_sfree);
                umma_commit_warp(b_qkfree + 8 * (c & 1));
                if (!wait(b_pb, c)) break;
            }
            if (c + 1 < nchunks) {
                if (!wait(b_full + 8 * ((c + 1) & 1), (c + 1) >> 1)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    umma_f16_warp(tbase + TM_P,
                                  desc_at(dK, sn + ST_Q + (s >> 2) * kPanel + (s & 3) * 32),
                                  desc_at(dK, sn + ST_K + (s >> 2) * kPanel + (s & 3) * 32), id_qk,
                                  s > 0);
                umma_commit_warp(b_p);
            }
            if (c < 0) continue;
            if (c > 0 && !wait(b_ofree, c - 1)) break;
            if (!wait(b_vfull + 8 * (c & 1), c >> 1)) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 8; ++s)
                umma_f16_ts_warp(tbase + TM_O1, tbase + TM_PB + 8 * s,
                                 desc_at(dM, st + ST_V + 2048 * s), id_o, s > 0);
            umma_commit_warp(b_vfree + 8 * (c & 1));
            umma_commit_warp(b_o);
        }
        if (kOut && nchunks > 0) {
            if (c < nchunks) umma_commit_warp(b_o);
            wait_phase(b_o, (uint32_t)(max(0, min(c, nchunks - 1)) & 1), args.budget);
        }
    } else {
        // ============================================================ gates
        float x[4], nx[4] = {0.f, 0.f, 0.f, 0.f};
        auto fetch = [&](int c, float (&to)[4]) {
            const int valid = c < nchunks ? rows_of(c) : 0;
            const long long t = sl.begin + (long long)c * kC + 4 * lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = 0.f;
                if (4 * lane + e < valid) y = p.log_g[p.gate_head ? h : (t + e) * p.H + h];
                to[e] = 1.4426950408889634f * (y < -110.f ? -110.f : y);   // in powers of two
            }
        };
#pragma unroll 1
        for (int c = -1; c < nchunks; ++c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = nx[e];
            fetch(c + 1, nx);
            if (c < 0) continue;
            if (c >= 2 && !wait(b_gfree + 8 * (c & 1), (c >> 1) - 1)) break;
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
                make_float4(ex2(s0), ex2(s1), ex2(s2), ex2(suf));
            if ((lane & 7) == 0) gt[2 * kC + (lane >> 3)] = down;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gfull + 8 * (c & 1));
        }
    }
    if (failed && lane == 0) set_device_error(p.err, DEV_TIMEOUT);
    // (this launch does not end before the one that it may have overtaken)
    if (kOut && warp == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    // (a value that is not finite leaves a state that is not, whatever follows it)
    const bool again = __syncthreads_or(spoilt);
    if (warp == 0) tmem_dealloc(tbase, kTmemCols);
    if (kOut && again) {
        if (tid == 0) bulk_wait_all();   // the outputs' stores have landed
        repair_rows(p, sl, h, j0, tid, sm);
    }
}

uint32_t wait_budget() {
    static const uint32_t budget = [] {
        const char* s = std::getenv("KDA_DEBUG_WAIT_CYCLES");
        const long long v = s && *s ? std::atoll(s) : 0;
        return v > 0 && v < 1ll << 31 ? (uint32_t)v : 1u << 31;   // about one second of SM clock
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
    // (there are at most slots - N segments that are not a sequence's last)
    const long long slots = pass == LinearPass::kStates ? p.slots - p.N : p.slots;
    const long long blocks = slots * p.H * a.tiles;
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
        (e = map(&m.v, p.v, p.H, p.dv)) != cudaSuccess ||
        (e = map(&m.o, p.o, p.H, p.dv)) != cudaSuccess)
        return e;
    if (pass == LinearPass::kStates) {
        linear_chunk_kernel<false><<<(unsigned)blocks, kThreads, kSmem, stream>>>(m, a);
        return cudaGetLastError();
    }
    // Outputs right behind the states' launch start beside it, on the SMs that it leaves free.
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = pass == LinearPass::kOutputs && !p.seg_ready ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, linear_chunk_kernel<true>, m, a);
}

}  // namespace kda
