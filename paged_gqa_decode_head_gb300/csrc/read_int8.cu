// read_int8.cu -- kv_cache_read_int8: rows of the paged INT8 cache read back as
// bf16, for attention of prompt chunks, for moving a sequence elsewhere, or for
// inspection.
//
// Row i of sequence b is slot first_b + i, as far as it lies below T_b:
//   out = bf16(code * s), one rounding of the exact product's fp32 value.
//
// Bound: memory, 132 bytes read and 256 written per (slot, KV head) of K and of
// V. Eight lanes take a row (16 codes each, two 16-byte stores), a warp four
// rows at a time; rows in the output's order, so that the writes, two thirds of the
// traffic, are contiguous over the whole block. Measured: 19387 slots of 8 heads in 8 ragged
// sequences 22.8 us, 5.3 TB/s (four rows of a thread in flight: 28.1 us, with half the warps).
#include "common.cuh"
#include "launch.h"

namespace pgqa {
namespace {

__device__ unsigned g_flags_read_int8;

constexpr int kReadThreads = 256;
constexpr int kReadLanes = 8;                               // lanes of a row
constexpr int kReadRows = kReadThreads / kReadLanes;        // rows of a block's pass

struct ReadParams {
    const int8_t *k_cache8, *v_cache8;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *context_lens, *first;
    uint16_t *k_out, *v_out;
    int N, Hkv, log2_page, max_pages, num_pages;
    int slots; // of a block
};

__global__ void __launch_bounds__(kReadThreads) read_int8_kernel(const __grid_constant__ ReadParams p)
{
    // What is read may come from the kernel before this one; nothing that this
    // one writes is read before a wait by any kernel here, caches apart, which it
    // does not write.
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.y, i0 = blockIdx.x * p.slots;
    const int T = p.context_lens[b], first = p.first ? p.first[b] : 0;
    if (T < 0 || T > (p.max_pages << p.log2_page) || first < 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            atomicOr(&g_flags_read_int8, PGQA_DEVERR_BAD_CONTEXT);
        return;
    }
    const long long behind = static_cast<long long>(T) - first - i0; // rows that exist from i0 on
    const int live = static_cast<int>(min(behind, static_cast<long long>(min(p.slots, p.N - i0))));
    if (live <= 0)
        return;
    const int lane8 = threadIdx.x % kReadLanes;
    const int rows = 2 * live * p.Hkv; // all of K, then all of V, each [slot][head]
    for (int r = threadIdx.x / kReadLanes; r < rows; r += kReadRows) {
        const bool is_v = r >= live * p.Hkv;
        const int in = is_v ? r - live * p.Hkv : r;
        const int i = in / p.Hkv, h = in - i * p.Hkv;
        const int slot = first + i0 + i;
        const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + (slot >> p.log2_page)];
        if (phys < 0 || phys >= p.num_pages) {
            atomicOr(&g_flags_read_int8, PGQA_DEVERR_BAD_PAGE);
            continue;
        }
        const size_t row = ((static_cast<size_t>(phys) * p.Hkv + h) << p.log2_page) + (slot & ((1 << p.log2_page) - 1));
        const uint4 codes = *reinterpret_cast<const uint4 *>((is_v ? p.v_cache8 : p.k_cache8) + row * kHeadDim + 16 * lane8);
        const float s = (is_v ? p.v_scale : p.k_scale)[row];
        const uint32_t words[4] = {codes.x, codes.y, codes.z, codes.w};
        uint32_t out[8];
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float lo = static_cast<float>(static_cast<int8_t>(words[w] >> (16 * half)));
                const float hi = static_cast<float>(static_cast<int8_t>(words[w] >> (16 * half + 8)));
                out[2 * w + half] = pack_bf16x2(lo * s, hi * s);
            }
        uint4 *dst = reinterpret_cast<uint4 *>((is_v ? p.v_out : p.k_out) +
                                               ((static_cast<size_t>(b) * p.N + i0 + i) * p.Hkv + h) * kHeadDim + 16 * lane8);
        dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
        dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

} // namespace

cudaError_t launch_read_int8(const ReadInt8Args &a, cudaStream_t stream)
{
    ReadParams p{a.k_cache8, a.v_cache8, a.k_scale, a.v_scale, a.block_table, a.context_lens, a.first, a.k_out, a.v_out,
                 a.N, a.Hkv, __builtin_ctz(static_cast<unsigned>(a.page_size)), a.max_pages, a.num_pages, 0};
    // a block takes slots of some 128 rows
    p.slots = 64 / a.Hkv > 0 ? 64 / a.Hkv : 1;
    return launch_pdl(read_int8_kernel, dim3(static_cast<unsigned>((a.N + p.slots - 1) / p.slots), static_cast<unsigned>(a.B)),
                      dim3(kReadThreads), 0, stream, p);
}

cudaError_t read_flags_read_int8(unsigned *flags, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_flags_read_int8, sizeof(unsigned));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_flags_read_int8, &zero, sizeof(unsigned));
    }
    return err;
}

} // namespace pgqa
