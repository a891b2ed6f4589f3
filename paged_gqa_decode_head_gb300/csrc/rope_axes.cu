// rope_axes.cu -- qk_norm_rope_append_axes: per-head Q/K RMSNorm, rotary
// positions with several axes, and the paged K/V append of M tokens per
// sequence (drafted trees, image and video patches, prompts).
//
// For token i with positions p_0 .. p_(A-1) and pair r (dims r and r + 64):
//   xhat = x * gamma / sqrt(mean(x^2) + eps)
//   phi_r = p_(axis(r)) * theta^(-2r/128)
//   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi)
// The angle is taken modulo one turn in 64-bit fixed point: w_r = frac(omega_r
// / 2 pi) * 2^64, and the low 64 bits of p * w_r are the fraction of a turn,
// exactly for that w_r and any int32 p. This GPU's fp64 rate is a small
// fraction of its integer rate; one 64-bit integer product replaces the fp64
// product and reduction.
//
// Bound: memory, (2 Hq + 4 Hkv) * 256 bytes a token, read and written once. The
// single-token prologue (prologue.cu) recomputes the angles for every head; at
// prompt lengths that would cost more than the copy, so here a block owns one
// to three tokens of a sequence, forms their rotations once in shared memory, and
// its 16 groups of 8 lanes walk the tokens' Hq + 2 Hkv rows with 16-byte loads
// and stores, two rows of a group on their way at a time (lane s of a group
// holds dims 8s .. 8s+7 and 64 + 8s .. 64 + 8s + 7, so a pair's two halves are in
// one lane). Measured (32 query, 8 KV heads): 32768 tokens 128 us, 6.3 TB/s, 93 % of
// the measured copy bandwidth; 19658 tokens in 8 ragged sequences of up to 4096 80 us,
// 6.0 TB/s; 4095 tokens of 16 + 8 heads 13.9 us, 4.8 TB/s (the start and end of its
// blocks); 1 or 16 tokens 3.4 us, a launch and three trips to memory.
#include "common.cuh"
#include "launch.h"

#include <cmath>

namespace pgqa {
namespace {

__device__ unsigned g_flags_rope_axes;

constexpr int kPairs = kHeadDim / 2;
constexpr int kRopeThreads = 128;
constexpr int kRopeBlocksPerSm = 9;                        // 56 registers a thread
constexpr int kRowLanes = 8;                               // lanes that hold one head row
constexpr int kRowsPerPass = kRopeThreads / kRowLanes;     // head rows a block handles at once
constexpr int kInFlight = 2;                               // rows a group of lanes has on their way

struct RopeAxesParams {
    uint64_t turn[kPairs];  // frac(omega_r / 2 pi) * 2^64
    uint64_t axis_bits[2];  // axis of pair r: two bits at 2 (r % 32) of word r / 32
    const uint16_t *q, *k, *v, *gamma_q, *gamma_k;
    const int32_t *positions, *context_lens, *new_lens, *block_table;
    uint16_t *k_cache, *v_cache, *q_out;
    int M, Hq, Hkv, n_axes, log2_page, max_pages, num_pages;
    int blocks_per_seq;
    float eps;
};

// x -> the row's element j of lo (dims 8s + j) or hi (64 + 8s + j)
__device__ __forceinline__ uint4 pack8(const float *f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// kTokens consecutive tokens of one sequence per block.
template <int kTokens>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) rope_axes_kernel(const __grid_constant__ RopeAxesParams p)
{
    // Everything this kernel reads may come from the kernel before it, and
    // what it writes may still be read there: wait before touching memory. The
    // next kernel may read cache rows before it waits for this one (the decode
    // kernels do, up to a length of their own and through a table of their own):
    // no early launch of it, not behind a single token's row either, and every
    // write is performed before its thread ends, also for reads by bulk copies.
    grid_dependency_wait();
    const int tid = threadIdx.x;
    const int b = blockIdx.x / p.blocks_per_seq, i0 = (blockIdx.x - b * p.blocks_per_seq) * kTokens;
    const int n = p.new_lens ? p.new_lens[b] : p.M;
    const int T = p.context_lens[b];
    if (n < 0 || n > p.M || T < n || T > (p.max_pages << p.log2_page)) {
        if (i0 == 0 && tid == 0)
            atomicOr(&g_flags_rope_axes, PGQA_DEVERR_BAD_CONTEXT);
        return;
    }
    const int live = min(n - i0, kTokens);
    if (live <= 0)
        return;
    const size_t tok0 = static_cast<size_t>(b) * p.M + i0;
    const int lane8 = tid & (kRowLanes - 1);
    const int rows = p.Hq + 2 * p.Hkv; // of a token: Q heads, K heads, V heads
    const size_t P = size_t{1} << p.log2_page;

    // The block's rows, token by token; this thread's group takes every 16th.
    struct At {
        int t, row;
    };
    const auto step = [&](At &at) {
        at.row += kRowsPerPass;
        while (at.row >= rows)
            at.row -= rows, ++at.t;
    };
    const auto load = [&](const At &at, uint4 &lo, uint4 &hi) {
        const size_t tok = tok0 + at.t;
        const uint16_t *src;
        if (at.row < p.Hq)
            src = p.q + (tok * p.Hq + at.row) * kHeadDim;
        else if (at.row < p.Hq + p.Hkv)
            src = p.k + (tok * p.Hkv + at.row - p.Hq) * kHeadDim;
        else
            src = p.v + (tok * p.Hkv + at.row - p.Hq - p.Hkv) * kHeadDim;
        lo = *reinterpret_cast<const uint4 *>(src + 8 * lane8);
        hi = *reinterpret_cast<const uint4 *>(src + kPairs + 8 * lane8);
    };
    At at{0, tid / kRowLanes};
    while (at.row >= rows)
        at.row -= rows, ++at.t;
    At ahead = at;
    uint4 lo[kInFlight], hi[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
        if (ahead.t < live)
            load(ahead, lo[k], hi[k]);
        step(ahead);
    }

    __shared__ __align__(16) float rot_cos[kTokens][kPairs], rot_sin[kTokens][kPairs];
    __shared__ long long cells[kTokens]; // cache row of the token's slot in KV head 0, -1: page outside the pool
    for (int r = tid; r < live * kPairs; r += kRopeThreads) {
        const int t = r / kPairs, pair = r % kPairs;
        const int axis = static_cast<int>(p.axis_bits[pair >> 5] >> (2 * (pair & 31))) & 3;
        const int pos = p.positions[(tok0 + t) * p.n_axes + axis];
        const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.turn[pair];
        // the upper 32 bits as a signed part of a turn, in half turns
        const float half_turns = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f;
        sincospif(half_turns, &rot_sin[t][pair], &rot_cos[t][pair]);
    }
    if (tid < live) {
        const int slot = T - n + i0 + tid;
        const int phys = p.block_table[static_cast<size_t>(b) * p.max_pages + (slot >> p.log2_page)];
        const bool in_pool = phys >= 0 && phys < p.num_pages;
        cells[tid] = in_pool ? static_cast<long long>(phys) * p.Hkv * P + (slot & (P - 1)) : -1;
        if (!in_pool)
            atomicOr(&g_flags_rope_axes, PGQA_DEVERR_BAD_PAGE);
    }
    __syncthreads();

    const int passes = (live * rows + kRowsPerPass - 1) / kRowsPerPass;
    for (int pass = 0; pass < passes; pass += kInFlight) {
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const bool here = at.t < live; // (a row group may be past the last row)
            const bool is_q = at.row < p.Hq, is_v = at.row >= p.Hq + p.Hkv;
            const int t = here ? at.t : 0;
            const uint4 in_lo = lo[k], in_hi = hi[k];
            float a[8], c[8];
            unpack8(in_lo, a);
            unpack8(in_hi, c);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = fmaf(a[j], a[j], fmaf(c[j], c[j], ss));
#pragma unroll
            for (int off = kRowLanes / 2; off > 0; off >>= 1)
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
            if (ahead.t < live)
                load(ahead, lo[k], hi[k]);
            step(ahead);
            const long long cell = cells[t];
            if (here && (is_q || cell >= 0)) {
                uint4 out_lo = in_lo, out_hi = in_hi; // V rows go through bit for bit
                if (!is_v) {
                    const float inv_rms = rsqrtf(fmaf(ss, 1.0f / kHeadDim, p.eps));
                    const uint16_t *gamma = is_q ? p.gamma_q : p.gamma_k;
                    float ga[8], gc[8];
                    unpack8(*reinterpret_cast<const uint4 *>(gamma + 8 * lane8), ga);
                    unpack8(*reinterpret_cast<const uint4 *>(gamma + kPairs + 8 * lane8), gc);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float cs = rot_cos[t][8 * lane8 + j], sn = rot_sin[t][8 * lane8 + j];
                        const float x = a[j] * inv_rms * ga[j], y = c[j] * inv_rms * gc[j];
                        a[j] = fmaf(x, cs, -(y * sn));
                        c[j] = fmaf(y, cs, x * sn);
                    }
                    out_lo = pack8(a);
                    out_hi = pack8(c);
                }
                uint16_t *dst;
                if (is_q)
                    dst = p.q_out + ((tok0 + t) * p.Hq + at.row) * kHeadDim;
                else if (!is_v)
                    dst = p.k_cache + (cell + (at.row - p.Hq) * P) * kHeadDim;
                else
                    dst = p.v_cache + (cell + (at.row - p.Hq - p.Hkv) * P) * kHeadDim;
                *reinterpret_cast<uint4 *>(dst + 8 * lane8) = out_lo;
                *reinterpret_cast<uint4 *>(dst + kPairs + 8 * lane8) = out_hi;
            }
            step(at);
        }
    }
    __threadfence(); // performed before the thread ends, and so before the next kernel starts
    fence_proxy_async_global();
}

} // namespace

cudaError_t launch_rope_axes(const RopeAxesArgs &a, cudaStream_t stream)
{
    // 64 powers cost more than a launch, and a model has one theta: the thread
    // keeps the table of the last one.
    static thread_local double table_theta = 0.0; // no valid theta
    static thread_local uint64_t table[kPairs];
    if (table_theta != a.rope_theta) {
        for (int r = 0; r < kPairs; ++r) {
            const double turns = std::pow(a.rope_theta, -2.0 * r / kHeadDim) / 6.283185307179586476925;
            table[r] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
        }
        table_theta = a.rope_theta;
    }
    RopeAxesParams p{};
    for (int r = 0; r < kPairs; ++r) {
        p.turn[r] = table[r];
        p.axis_bits[r >> 5] |= static_cast<uint64_t>(a.axis_of_pair[r] & 3) << (2 * (r & 31));
    }
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.gamma_q = a.gamma_q;
    p.gamma_k = a.gamma_k;
    p.positions = a.positions;
    p.context_lens = a.context_lens;
    p.new_lens = a.new_lens;
    p.block_table = a.block_table;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.q_out = a.q_out;
    p.M = a.M;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.n_axes = a.n_axes;
    p.log2_page = __builtin_ctz(static_cast<unsigned>(a.page_size));
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.eps = a.eps;
    // One token per block as long as all blocks run at once, then two, then three:
    // a block that had to wait for another's end costs more than the longer blocks,
    // which share the trips to lengths and tables. Tokens of 16 + 8 heads with one, two
    // and three per block: 16 3.4, 4.4, 5.4 us; 1100 6.6, 7.1, 8.1 us; 1500 9.9, 7.9, 8.7
    // us; 2700 12.9, 10.2, 10.9 us; 3192 15.6, 14.4, 11.8 us; 4095 18.1, 16.0, 13.9 us (four:
    // 15). Past that, three of up to 32 rows (16384: 57.1, 48.7, 47.0 us) and two of more
    // (32 + 8 heads: 8192 41.8, 36.0, 36.4 us; 19658 in 8 ragged sequences 96.8, 80.2, 81.3
    // us; 32768 144.6, 127.8, 128.0 us).
    const long long at_once = static_cast<long long>(kRopeBlocksPerSm) * (a.sm_count > 0 ? a.sm_count : 1);
    const long long per_block = (static_cast<long long>(a.B) * a.M + at_once - 1) / at_once;
    const int tokens = per_block <= 3 ? static_cast<int>(per_block) : a.Hq + 2 * a.Hkv <= 32 ? 3 : 2;
    const auto kernel = tokens == 1 ? rope_axes_kernel<1> : tokens == 2 ? rope_axes_kernel<2> : rope_axes_kernel<3>;
    p.blocks_per_seq = (a.M + tokens - 1) / tokens;
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(p.blocks_per_seq));
    return launch_pdl(kernel, grid, dim3(kRopeThreads), 0, stream, p);
}

cudaError_t read_flags_rope_axes(unsigned *flags, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_flags_rope_axes, sizeof(unsigned));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_flags_rope_axes, &zero, sizeof(unsigned));
    }
    return err;
}

} // namespace pgqa
