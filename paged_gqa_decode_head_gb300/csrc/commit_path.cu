// commit_path.cu -- kv_cache_commit_path: the accepted path of a drafted tree
// moves behind the prefix, in every layer and KV head, in one launch.
//
// Slot base + path[i] goes to slot base + i. The path is strictly increasing,
// so path[i] >= i: a destination i is a source only of entries before i. Rows
// are taken in ascending chunks, each chunk read into registers by the whole
// block before any of it is written, so no row is overwritten before it was
// read, without scratch memory.
//
// The entries that move are the path's end: once path[i] > i it stays so.
//
// Bound: latency. A step moves a few KB per sequence and layer; what a call
// costs is its launch and a chain of four trips to memory (lengths, path, table
// entries, rows). So one launch covers all layers, and a block owns all heads
// of a (sequence, layer), whose first three trips they share, or one head where
// there are too few blocks.
#include "common.cuh"
#include "launch.h"

namespace pgqa {
namespace {

__device__ unsigned g_flags_commit_path;

constexpr int kCommitThreads = 256;
constexpr int kLanesPerRow = kRowBytes / 16;               // 16
constexpr int kRowsAtOnce = kCommitThreads / kLanesPerRow; // 16 rows per unit
constexpr int kUnits = 4;                                  // units in registers at a time
constexpr int kMaxDrafted = 64;

struct CommitParams {
    uint16_t *k_caches[PGQA_MAX_COMMIT_LAYERS], *v_caches[PGQA_MAX_COMMIT_LAYERS];
    const int32_t *block_tables[PGQA_MAX_COMMIT_LAYERS];
    const int32_t *context_lens, *draft_lens, *path, *path_lens;
    int32_t *context_lens_out;
    int M, A, Hkv, heads, log2_page, max_pages, num_pages; // heads: per block
};

__global__ void __launch_bounds__(kCommitThreads) commit_path_kernel(const __grid_constant__ CommitParams p)
{
    // The next kernel may read tables, lengths and cache rows before it waits for
    // this one (the decode kernels do, rows by bulk copies): no early launch of it
    // here, and every write is performed before its thread ends, rows for such reads too.
    grid_dependency_wait();
    __shared__ long long from[kMaxDrafted], to[kMaxDrafted]; // cache rows of KV head 0, -1: page outside the pool
    const int tid = threadIdx.x;
    const int h0 = blockIdx.x * p.heads, b = blockIdx.y, layer = blockIdx.z;
    const bool reports = h0 == 0 && layer == 0; // this block writes the sequence's length and flags
    const int T = p.context_lens[b];
    const int n = p.draft_lens ? p.draft_lens[b] : p.M;
    const int a = p.path_lens[b];
    if (n < 0 || n > p.M || T < n || T > (p.max_pages << p.log2_page)) {
        if (reports && tid == 0) {
            p.context_lens_out[b] = T;
            atomicOr(&g_flags_commit_path, PGQA_DEVERR_BAD_CONTEXT);
            __threadfence();
        }
        return;
    }
    // the whole path is checked before anything moves
    bool bad = a < 0 || a > p.A;
    bool moves = false, page_missing = false;
    if (!bad && tid < a) { // a <= A <= 64
        const int32_t *path = p.path + static_cast<size_t>(b) * p.A;
        const int e = path[tid];
        bad = e >= n || e < 0 || (tid > 0 && path[tid - 1] >= e);
        moves = e != tid;
        if (!bad && moves) {
            const int32_t *table = p.block_tables[layer] + static_cast<size_t>(b) * p.max_pages;
            const int P = 1 << p.log2_page;
            const auto cell = [&](int slot) -> long long {
                const int phys = table[slot >> p.log2_page];
                if (phys < 0 || phys >= p.num_pages)
                    return -1;
                return ((static_cast<long long>(phys) * p.Hkv) << p.log2_page) + (slot & (P - 1));
            };
            from[tid] = cell(T - n + e);
            to[tid] = cell(T - n + tid);
            page_missing = from[tid] < 0 || to[tid] < 0;
        }
    }
    bad = __syncthreads_or(bad);
    if (reports && tid == 0) {
        p.context_lens_out[b] = T - n + (bad ? 0 : a);
        if (bad)
            atomicOr(&g_flags_commit_path, PGQA_DEVERR_BAD_PATH);
        __threadfence();
    }
    if (bad)
        return;
    if (page_missing)
        atomicOr(&g_flags_commit_path, PGQA_DEVERR_BAD_PAGE);
    const int moved = __syncthreads_count(moves); // the path's last entries
    const int lane = tid % kLanesPerRow, group = tid / kLanesPerRow;
    const int heads = min(p.heads, p.Hkv - h0);
    const int per_entry = 2 * heads, items = moved * per_entry; // item: entry, then head, then K or V
    for (int first = 0; first < items; first += kRowsAtOnce * kUnits) {
        uint4 row[kUnits];
        uint16_t *dst[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int item = first + u * kRowsAtOnce + group;
            dst[u] = nullptr;
            if (item < items) {
                const int i = item / per_entry, e = a - moved + i, rest = item - i * per_entry;
                if (from[e] >= 0 && to[e] >= 0) {
                    uint16_t *cache = rest & 1 ? p.v_caches[layer] : p.k_caches[layer];
                    const long long head = static_cast<long long>(h0 + (rest >> 1)) << p.log2_page;
                    row[u] = reinterpret_cast<const uint4 *>(cache + (from[e] + head) * kHeadDim)[lane];
                    dst[u] = cache + (to[e] + head) * kHeadDim;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            if (dst[u])
                reinterpret_cast<uint4 *>(dst[u])[lane] = row[u];
        __syncthreads();
    }
    __threadfence();
    fence_proxy_async_global();
}

} // namespace

cudaError_t launch_commit_path(const CommitPathArgs &a, cudaStream_t stream)
{
    CommitParams p{};
    for (int l = 0; l < a.n_layers; ++l) {
        p.k_caches[l] = a.k_caches[l];
        p.v_caches[l] = a.v_caches[l];
        p.block_tables[l] = a.block_tables[l];
    }
    p.context_lens = a.context_lens;
    p.draft_lens = a.draft_lens;
    p.path = a.path;
    p.path_lens = a.path_lens;
    p.context_lens_out = a.context_lens_out;
    p.M = a.M;
    p.A = a.A;
    p.Hkv = a.Hkv;
    p.log2_page = __builtin_ctz(static_cast<unsigned>(a.page_size));
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    // One block per (sequence, layer), or per head while these do not give each
    // SM a block.
    p.heads = static_cast<long long>(a.B) * a.n_layers >= a.sm_count ? a.Hkv : 1;
    return launch_pdl(commit_path_kernel,
                      dim3(static_cast<unsigned>((a.Hkv + p.heads - 1) / p.heads), static_cast<unsigned>(a.B),
                           static_cast<unsigned>(a.n_layers)),
                      dim3(kCommitThreads), 0, stream, p);
}

cudaError_t read_flags_commit_path(unsigned *flags, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_flags_commit_path, sizeof(unsigned));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_flags_commit_path, &zero, sizeof(unsigned));
    }
    return err;
}

} // namespace pgqa
