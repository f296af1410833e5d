// Linear attention with a scalar decay for each head: parameters and launchers.
//
//   S <- exp(log_g) S + k v^T,   o = S^T q
//
// The map from a stretch of tokens' initial to its final state is S -> d S + B (d the product of
// its gates, B its final state from S = 0), so a long sequence is cut into segments of seg_tokens
// tokens: one launch computes B and d of every segment but a sequence's last, a small kernel
// chains the segments' initial states, and a second launch computes every segment's outputs.
#pragma once

#include "kda_internal.cuh"

namespace kda {

struct LinearParams {
    const void* q;              // [B, T, Hk, dk]
    const void* k;
    const void* v;              // [B, T, H, dv]
    const float* log_g;         // [B, T, H], or [H] with gate_head
    const float* h0;            // nullable; [N, H, dk, dv]
    const int32_t* cu_seqlens;  // nullable (device)
    void* o;                    // [B, T, H, dv]
    float* hT;                  // nullable
    int B, T, H, Hk, dk, dv, N;
    bool bf16, gate_head;
    unsigned* err;
    // segments (seg_tokens > 0): slot g holds segment s of sequence n, g = n segs + s for
    // equal-length sequences, else floor(cu[n] / seg_tokens) + n + s (strictly increasing over
    // (n, s), so slots never collide and g < slots = floor(T / seg_tokens) + N)
    int seg_tokens;
    int whole_tokens;           // packed, chunked: sequences up to this long are one segment
    int slots;                  // slots per head (N without segments)
    float* seg_state;           // [slots, H, dk, dv]: B, then the segment's initial state
    float* seg_decay;           // [slots, H]
    bool seg_ready;             // chunked outputs: seg_state has been chained by launch_linear_combine
};

enum class LinearPass {
    kWhole,       // whole sequences: h0 -> o, hT
    kStates,      // segments but the last: B and d
    kOutputs      // segments from their initial states: o, and hT from the last
};

// One slot's stretch of tokens.
struct LinearSlot {
    int n, seg;
    long long begin, end;   // rows of the flat token axis
    bool last;              // the sequence's last segment
};

// False where the slot is unused, or where cu_seqlens is malformed around it (which sets the
// error word). Every bound that comes from cu_seqlens is checked here, so a malformed one never
// leads outside the tensors.
__device__ __forceinline__ bool linear_slot(const LinearParams& p, int g, LinearSlot* s) {
    const int L = p.seg_tokens;
    long long t0, t1;
    if (!p.cu_seqlens) {
        const int segs = L > 0 ? max(1, (p.T + L - 1) / L) : 1;
        s->n = g / segs;
        s->seg = g % segs;
        if (s->n >= p.N) return false;
        t0 = (long long)s->n * p.T;
        t1 = t0 + p.T;
    } else {
        int n = g;
        if (L > 0) {   // the last n with floor(cu[n] / L) + n <= g
            int lo = 0, hi = p.N - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.cu_seqlens[mid] / L + mid <= g) lo = mid;
                else hi = mid - 1;
            }
            n = lo;
        }
        if (n >= p.N) return false;
        t0 = p.cu_seqlens[n];
        t1 = p.cu_seqlens[n + 1];
        const bool bad_ends = (n == 0 && t0 != 0) || (n == p.N - 1 && t1 != p.T);
        if (t1 < t0 || t0 < 0 || t1 > p.T || bad_ends) {
            set_device_error(p.err, DEV_BAD_SEQLENS);
            return false;
        }
        s->n = n;
        s->seg = L > 0 ? g - (int)(t0 / L) - n : 0;
    }
    if (L <= 0) {
        s->begin = t0;
        s->end = t1;
        s->last = true;
        return true;
    }
    const long long b = t0 + (long long)s->seg * L;
    if (s->seg < 0 || (s->seg > 0 && b >= t1)) return false;
    s->begin = b;
    s->end = min(t1, b + L);
    s->last = b + L >= t1;
    return true;
}

// CUDA-core walk, token by token in fp32: any dtype, dk, dv <= 256.
cudaError_t launch_linear_walk(const LinearParams& p, LinearPass pass, cudaStream_t stream);
// Chunks of 128 tokens on the tensor cores; seg_tokens a multiple of 128.
constexpr int kLinearChunk = 128;
bool linear_chunk_takes(bool bf16, int dk, int dv);
cudaError_t launch_linear_chunk(const LinearParams& p, LinearPass pass, cudaStream_t stream);
// A few tokens of whole sequences in place (state at hT): registers hold the state.
bool linear_decode_takes(int T, int dk, int dv);
cudaError_t launch_linear_decode(const LinearParams& p, cudaStream_t stream);
// Chains the segments' initial states: seg_state[n, s] <- state before segment s >= 1.
cudaError_t launch_linear_combine(const LinearParams& p, cudaStream_t stream);
// Sets the error word where cu_seqlens does not rise from 0 to T (segmented launches may not
// visit every sequence of a malformed one).
cudaError_t launch_linear_check(const LinearParams& p, cudaStream_t stream);

}  // namespace kda
