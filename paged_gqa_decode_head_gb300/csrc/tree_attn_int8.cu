// tree_attn_int8.cu -- decode_attn_paged_tree_int8: attention of a tree of
// drafted tokens over the paged INT8 cache.
//
// First form: one warp per query row, keys 32 at a time, scores and the running
// softmax in fp64 where the bias needs it.
#include "common.cuh"
#include "launch.h"

#include <cmath>

namespace pgqa {
namespace {

__device__ unsigned g_flags_tree_int8;

struct Params8 {
    TreeAttnInt8Args a;
    int log2_page, g;
};

__global__ void __launch_bounds__(128) tree_rows_kernel(const __grid_constant__ Params8 p)
{
    grid_dependency_wait();
    allow_dependent_launch();
    const TreeAttnInt8Args &a = p.a;
    __shared__ float qs[4][kHeadDim];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r = blockIdx.x * 4ll + warp;
    if (r >= static_cast<long long>(a.B) * a.M * a.Hq)
        return;
    const int hq = static_cast<int>(r % a.Hq), i = static_cast<int>(r / a.Hq % a.M), b = static_cast<int>(r / a.Hq / a.M);
    const int h = hq / p.g;
    const int T = a.context_lens[b], n = a.draft_lens ? a.draft_lens[b] : a.M;
    const bool good = n >= 0 && n <= a.M && T >= n && T <= (a.max_pages << p.log2_page);
    if (!good && lane == 0)
        atomicOr(&g_flags_tree_int8, PGQA_DEVERR_BAD_CONTEXT);
    if (good && i >= n)
        return;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    double m = -INFINITY, l = 0.0;
    if (good) {
        for (int d = lane; d < kHeadDim; d += 32)
            qs[warp][d] = __uint_as_float(static_cast<uint32_t>(a.q[r * kHeadDim + d]) << 16);
        __syncwarp();
        const uint64_t mask = a.tree_mask[static_cast<size_t>(b) * a.M + i];
        const int prefix = T - n;
        for (int k0 = 0; k0 < T; k0 += 32) {
            const int key = k0 + lane;
            double y = -INFINITY;
            size_t row = 0;
            bool seen = key < T && (key < prefix || (mask >> (key - prefix) & 1u));
            if (key < T) {
                const int phys = a.block_table[static_cast<size_t>(b) * a.max_pages + (key >> p.log2_page)];
                if (phys < 0 || phys >= a.num_pages) {
                    seen = false;
                    atomicOr(&g_flags_tree_int8, PGQA_DEVERR_BAD_PAGE);
                } else {
                    row = ((static_cast<size_t>(phys) * a.Hkv + h) << p.log2_page) + (key & ((1 << p.log2_page) - 1));
                }
            }
            if (seen) {
                float dot = 0.f;
                for (int d = 0; d < kHeadDim; ++d)
                    dot = fmaf(static_cast<float>(a.k_cache8[row * kHeadDim + d]), qs[warp][d], dot);
                y = static_cast<double>(dot) * a.k_scale[row] * a.scale;
                if (a.softcap > 0.f)
                    y = a.softcap * tanh(y / a.softcap);
                if (a.slopes) {
                    const int32_t *pos = a.positions + static_cast<size_t>(b) * a.M;
                    const long long at = key < prefix ? key : pos[key - prefix];
                    y += static_cast<double>(a.slopes[hq]) * static_cast<double>(at - pos[i]);
                }
            }
            double top = fmax(m, y);
            for (int off = 16; off > 0; off >>= 1)
                top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            if (top == -INFINITY)
                continue;
            const double f = m == -INFINITY ? 0.0 : exp(m - top);
            const double w = seen ? exp(y - top) : 0.0;
            m = top;
            l *= f;
            for (int e = 0; e < 4; ++e)
                acc[e] *= static_cast<float>(f);
            double sum = w;
            for (int off = 16; off > 0; off >>= 1)
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            l += sum;
            const float wv = seen ? static_cast<float>(w * a.v_scale[row]) : 0.f;
            for (int j = 0; j < 32; ++j) {
                const float pj = __shfl_sync(0xFFFFFFFFu, wv, j);
                const size_t rj = __shfl_sync(0xFFFFFFFFu, row, j);
                if (__shfl_sync(0xFFFFFFFFu, seen, j))
                    for (int e = 0; e < 4; ++e)
                        acc[e] = fmaf(pj, static_cast<float>(a.v_cache8[rj * kHeadDim + lane + 32 * e]), acc[e]);
            }
        }
    }
    const float inv = l == 0.0 ? 0.f : static_cast<float>(1.0 / l);
    for (int e = 0; e < 4; ++e) {
        const float o = acc[e] * inv;
        if (a.out_f32)
            a.out_f32[r * kHeadDim + lane + 32 * e] = o;
        if (a.out_bf16)
            a.out_bf16[r * kHeadDim + lane + 32 * e] = f32_to_bf16_bits(o);
    }
}

} // namespace

size_t tree_attn_int8_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_tree_attn_int8(const TreeAttnInt8Args &a, cudaStream_t stream)
{
    const Params8 p{a, __builtin_ctz(static_cast<unsigned>(a.page_size)), a.Hq / a.Hkv};
    const long long rows = static_cast<long long>(a.B) * a.M * a.Hq;
    return launch_pdl(tree_rows_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, p);
}

cudaError_t read_flags_tree_attn_int8(unsigned *flags, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_flags_tree_int8, sizeof(unsigned));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_flags_tree_int8, &zero, sizeof(unsigned));
    }
    return err;
}

} // namespace pgqa
