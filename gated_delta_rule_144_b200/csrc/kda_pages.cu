// Pages of a pool of states copied in place: page dst[i] <- page src[i], or zeros, in every layer.
//
// The pool is [layers][pages][page_bytes]; a fork copies one page to several, a compaction moves
// pages from the pool's tail into holes, a new sequence's page is cleared. Bound: HBM (one read
// and one write per moved page; the reads of a forked page after the first come from L2).
//
// A block copies one piece of one pair's page, 16 bytes per thread and load, eight loads in
// flight. All blocks run at once, so a page may not be both read and written, nor written twice:
// each block checks its own pair against the whole list (8 bytes per pair from L2, small beside
// its piece) and leaves a pair in conflict, or out of range, as it is, recording the error.
// 595 MB of moves and clears of 2 MiB pages take 96 us (0.95 of the measured copy rate), 8192 pairs of
// 128 KiB 333 us (0.98); 20000 pairs of 16 KiB, where the list outweighs the page, 309 us (0.32).

#include "kda_pages.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;

__global__ void __launch_bounds__(kThreads)
page_copy_kernel(uint4* pool, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                 int n, int pages, long long page_vecs, long long piece_vecs, int pieces,
                 unsigned* err) {
    const long long b = blockIdx.x;
    const int piece = (int)(b % pieces);
    const int i = (int)(b / pieces % n);
    const long long layer = b / pieces / n;
    const int s = src[i], d = dst[i];
    if (d == -1) return;
    bool bad = s < -1 || s >= pages || d < 0 || d >= pages;
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const int dj = dst[j], sj = src[j];
        if (j != i && dj != -1) bad |= dj == d || sj == d || (s >= 0 && dj == s);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_device_error(err, DEV_BAD_INDEX);
        return;
    }
    if (s == d) return;
    uint4* to = pool + (layer * pages + d) * page_vecs;
    const uint4* from = pool + (layer * pages + (s < 0 ? 0 : s)) * page_vecs;
    const long long end = min(page_vecs, (piece + 1) * piece_vecs);
    for (long long v = piece * piece_vecs + threadIdx.x; v < end; v += kThreads * kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long at = v + u * kThreads;
            x[u] = s >= 0 && at < end ? from[at] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long at = v + u * kThreads;
            if (at < end) __stcs(to + at, x[u]);
        }
    }
}

}  // namespace

cudaError_t launch_page_copy(void* pool, const int32_t* src, const int32_t* dst, int n, int layers,
                             int pages, long long page_bytes, unsigned* err, cudaStream_t stream) {
    const long long vecs = page_bytes / 16;
    // 32 KiB pieces (one pass of the block's loads); larger ones where there are blocks to spare
    long long piece = kThreads * kUnroll;
    const long long total = (long long)n * layers * ((vecs + piece - 1) / piece);
    if (total > 148 * 32) piece *= 4;
    const long long pieces = (vecs + piece - 1) / piece, blocks = pieces * n * layers;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    page_copy_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(
        static_cast<uint4*>(pool), src, dst, n, pages, vecs, piece, (int)pieces, err);
    return cudaGetLastError();
}

}  // namespace kda
