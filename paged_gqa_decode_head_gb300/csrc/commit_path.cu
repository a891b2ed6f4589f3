// commit_path.cu -- kv_cache_commit_path: the accepted path of a drafted tree
// moves behind the prefix, in every layer and KV head, in one launch.
//
// Slot base + path[i] goes to slot base + i. The path is strictly increasing,
// so path[i] >= i: a destination i is a source only of entries before i. Rows
// are taken in ascending chunks, each chunk read into registers by the whole
// block before any of it is written, so no row is overwritten before it was
// read, without scratch memory.
//
// Bound: latency. A step moves a few KB per sequence and layer; what a call
// costs is its launch and one dependent chain of loads (lengths, path, table
// entry, row). So one launch covers all layers, a block owns one (layer,
// sequence, head), and its 16-lane groups move a 256-byte row each.
#include "common.cuh"
#include "launch.h"

namespace pgqa {
namespace {

__device__ unsigned g_flags_commit_path;

constexpr int kCommitThreads = 128;
constexpr int kLanesPerRow = kRowBytes / 16;                       // 16
constexpr int kRowsAtOnce = kCommitThreads / kLanesPerRow;         // 8 rows, K or V, per unit
constexpr int kUnits = 4;                                          // units in registers per chunk
constexpr int kChunkEntries = kRowsAtOnce * kUnits / 2;            // path entries per chunk (K and V)

struct CommitParams {
    uint16_t *k_caches[PGQA_MAX_COMMIT_LAYERS], *v_caches[PGQA_MAX_COMMIT_LAYERS];
    const int32_t *block_tables[PGQA_MAX_COMMIT_LAYERS];
    const int32_t *context_lens, *draft_lens, *path, *path_lens;
    int32_t *context_lens_out;
    int M, A, Hkv, log2_page, max_pages, num_pages;
};

__global__ void __launch_bounds__(kCommitThreads) commit_path_kernel(const __grid_constant__ CommitParams p)
{
    allow_dependent_launch();
    grid_dependency_wait();
    const int tid = threadIdx.x;
    const int h = blockIdx.x, b = blockIdx.y, layer = blockIdx.z;
    const bool reports = h == 0 && layer == 0; // this block writes the sequence's length and flags
    const int T = p.context_lens[b];
    const int n = p.draft_lens ? p.draft_lens[b] : p.M;
    const int a = p.path_lens[b];
    if (n < 0 || n > p.M || T < n || T > (p.max_pages << p.log2_page)) {
        if (reports && tid == 0) {
            p.context_lens_out[b] = T;
            atomicOr(&g_flags_commit_path, PGQA_DEVERR_BAD_CONTEXT);
        }
        return;
    }
    // the whole path is checked before anything moves
    bool bad = a < 0 || a > p.A;
    const int32_t *path = p.path + static_cast<size_t>(b) * p.A;
    if (!bad && tid < a) // a <= A <= 64
        bad = path[tid] >= n || path[tid] < 0 || (tid > 0 && path[tid - 1] >= path[tid]);
    bad = __syncthreads_or(bad);
    if (reports && tid == 0) {
        p.context_lens_out[b] = T - n + (bad ? 0 : a);
        if (bad)
            atomicOr(&g_flags_commit_path, PGQA_DEVERR_BAD_PATH);
    }
    if (bad)
        return;
    const int32_t *table = p.block_tables[layer] + static_cast<size_t>(b) * p.max_pages;
    const int P = 1 << p.log2_page;
    const int lane = tid % kLanesPerRow, group = tid / kLanesPerRow;
    // offset of slot's row in a cache, or -1 (page outside the pool)
    const auto row_of = [&](int slot) -> long long {
        const int phys = table[slot >> p.log2_page];
        if (phys < 0 || phys >= p.num_pages)
            return -1;
        return ((static_cast<long long>(phys) * p.Hkv + h) * P + (slot & (P - 1))) * kHeadDim;
    };
    for (int first = 0; first < a; first += kChunkEntries) {
        uint4 row[kUnits];
        uint16_t *dst[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int item = u * kRowsAtOnce + group; // entry within the chunk, then K or V
            const int e = first + (item >> 1);
            uint16_t *cache = item & 1 ? p.v_caches[layer] : p.k_caches[layer];
            dst[u] = nullptr;
            if (e < a && path[e] != e) {
                const long long from = row_of(T - n + path[e]), to = row_of(T - n + e);
                if (from >= 0 && to >= 0) {
                    row[u] = reinterpret_cast<const uint4 *>(cache + from)[lane];
                    dst[u] = cache + to;
                } else if (lane == 0) {
                    atomicOr(&g_flags_commit_path, PGQA_DEVERR_BAD_PAGE);
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
    return launch_pdl(commit_path_kernel,
                      dim3(static_cast<unsigned>(a.Hkv), static_cast<unsigned>(a.B), static_cast<unsigned>(a.n_layers)),
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
