// tree_attn.cu -- decode_attn_paged_tree: attention of a tree of drafted
// tokens over the paged cache, with an optional tanh cap and distance bias.
//
// One warp per query row (sequence, drafted token, head) walks the keys with
// an online softmax; lane l holds dims 4l .. 4l+3. Every row reads the cache
// by itself.
#include "common.cuh"
#include "launch.h"

namespace pgqa {
namespace {

__device__ unsigned g_flags_tree;

struct TreeParams {
    const uint16_t *q, *k, *v;
    const int32_t *block_table, *context_lens;
    const uint64_t *tree_mask;
    const int32_t *positions, *draft_lens;
    const float *slopes;
    int M, Hq, Hkv, log2_page, max_pages, num_pages;
    float scale, softcap;
    float *out_f32;
    uint16_t *out_bf16;
};

__device__ __forceinline__ float4 load4(const uint16_t *row)
{
    const uint2 u = reinterpret_cast<const uint2 *>(row)[threadIdx.x & 31];
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

__global__ void __launch_bounds__(32) tree_rows_kernel(const TreeParams p)
{
    allow_dependent_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x;
    const int h = blockIdx.x % p.Hq, i = blockIdx.x / p.Hq, b = blockIdx.y;
    const int T = p.context_lens[b], n = p.draft_lens ? p.draft_lens[b] : p.M;
    const bool valid = n >= 0 && n <= p.M && T >= n && T <= (p.max_pages << p.log2_page);
    if (valid && i >= n)
        return;
    const size_t row = (static_cast<size_t>(b) * p.M + i) * p.Hq + h;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    if (valid) {
        const float4 q = load4(p.q + row * kHeadDim);
        const int prefix = T - n;
        const uint64_t mask = p.tree_mask[static_cast<size_t>(b) * p.M + i];
        const int kvh = h / (p.Hq / p.Hkv);
        const int pos_i = p.positions ? p.positions[static_cast<size_t>(b) * p.M + i] : 0;
        for (int j = 0; j < T; ++j) {
            if (j >= prefix && !(mask >> (j - prefix) & 1))
                continue;
            const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + (j >> p.log2_page)];
            if (phys < 0 || phys >= p.num_pages) {
                if (lane == 0)
                    atomicOr(&g_flags_tree, PGQA_DEVERR_BAD_PAGE);
                continue;
            }
            const size_t cell =
                (((static_cast<size_t>(phys) * p.Hkv + kvh) << p.log2_page) + (j & ((1 << p.log2_page) - 1))) * kHeadDim;
            const float4 k = load4(p.k + cell);
            float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
            x *= p.scale;
            if (p.softcap > 0.f)
                x = p.softcap * tanhf(x / p.softcap);
            if (p.slopes) {
                const int pos_j = j < prefix ? j : p.positions[static_cast<size_t>(b) * p.M + j - prefix];
                x = fmaf(p.slopes[h], static_cast<float>(pos_j - pos_i), x);
            }
            const float m_new = fmaxf(m, x);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            const float keep = exp2f((m - ref) * kLog2e), w = exp2f((x - ref) * kLog2e);
            const float4 v = load4(p.v + cell);
            acc.x = fmaf(w, v.x, acc.x * keep);
            acc.y = fmaf(w, v.y, acc.y * keep);
            acc.z = fmaf(w, v.z, acc.z * keep);
            acc.w = fmaf(w, v.w, acc.w * keep);
            l = fmaf(l, keep, w);
            m = m_new;
        }
    } else if (i == 0 && h == 0 && lane == 0) {
        atomicOr(&g_flags_tree, PGQA_DEVERR_BAD_CONTEXT);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const float4 r = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (p.out_f32)
        reinterpret_cast<float4 *>(p.out_f32 + row * kHeadDim)[lane] = r;
    if (p.out_bf16)
        reinterpret_cast<uint2 *>(p.out_bf16 + row * kHeadDim)[lane] =
            make_uint2(pack_bf16x2(r.x, r.y), pack_bf16x2(r.z, r.w));
}

} // namespace

size_t tree_attn_workspace_bytes(int B, int M, int Hq, int Hkv, int page_size, int max_pages, int sm_count)
{
    (void)B, (void)M, (void)Hq, (void)Hkv, (void)page_size, (void)max_pages, (void)sm_count;
    return 0;
}

cudaError_t launch_tree_attn(const TreeAttnArgs &a, cudaStream_t stream)
{
    const TreeParams p{a.q, a.k_cache, a.v_cache, a.block_table, a.context_lens, a.tree_mask, a.positions,
                       a.draft_lens, a.slopes, a.M, a.Hq, a.Hkv, __builtin_ctz(static_cast<unsigned>(a.page_size)),
                       a.max_pages, a.num_pages, a.scale, a.softcap, a.out_f32, a.out_bf16};
    return launch_pdl(tree_rows_kernel, dim3(static_cast<unsigned>(a.M * a.Hq), static_cast<unsigned>(a.B)), dim3(32),
                      0, stream, p);
}

cudaError_t read_flags_tree_attn(unsigned *flags, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_flags_tree, sizeof(unsigned));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_flags_tree, &zero, sizeof(unsigned));
    }
    return err;
}

} // namespace pgqa
