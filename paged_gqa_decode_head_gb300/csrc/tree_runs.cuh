// tree_runs.cuh -- what the tree attention's kernels (bf16 and INT8 caches) share:
// the division of all tiles of 128 keys into equal runs, one per CTA, the walk
// through a run, and the join of the pieces of a (sequence, KV head) that several
// CTAs worked on.
//
// The kernels' parameter structs (P below) hold B, M, Hq, Hkv, log2_page, max_pages,
// context_lens, draft_lens, g, tile_tokens, row_groups, rec_rows, ctas, unit_base,
// rec_m, rec_l, rec_acc, out_f32 and out_bf16; their shared memory (S) holds start_b,
// start_h, start_tile, start_T, start_n, units and scan.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pgqa {
namespace {

constexpr int kTileKeys = 128;
constexpr int kMergeThreads = 128;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A bounded wait by a whole warp, with one answer for all its lanes. The limit
// is counted in SM clocks (some 200 ms): reading %globaltimer between two tries
// takes about as long as a tile's scores.
constexpr long long kWaitLimitClocks = 400ll * 1000 * 1000;
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    bool there = mbar_try_wait(bar, parity);
    if (!there) {
        const long long start = clock64();
        do
            there = mbar_try_wait(bar, parity);
        while (!there && clock64() - start < kWaitLimitClocks);
    }
    return __all_sync(0xFFFFFFFFu, there);
}

// Sequence b's length and drafted tokens; false if they make no sense.
template <typename P>
__device__ __forceinline__ bool sequence(const P &p, int b, int &T, int &n)
{
    T = p.context_lens[b];
    n = p.draft_lens ? p.draft_lens[b] : p.M;
    return n >= 0 && n <= p.M && T >= n && T <= (p.max_pages << p.log2_page);
}
template <typename P>
__device__ __forceinline__ int tiles_of(const P &p, int b, int &T, int &n)
{
    return sequence(p, b, T, n) && n > 0 ? (T - 1) / kTileKeys + 1 : 0;
}

// CTA c's run of the `total` tiles: [first, first + result). Equal parts, the
// first total % ctas CTAs one more; with fewer tiles than CTAs the first take
// one each, so every CTA between a (sequence, head)'s first and last has a
// piece of it.
template <typename P>
__device__ __forceinline__ int run_of(const P &p, int total, int c, int &first)
{
    const int part = total / p.ctas, more = total - part * p.ctas;
    first = c * part + min(c, more);
    return part + (c < more ? 1 : 0);
}
// The CTA whose run holds tile u.
template <typename P>
__device__ __forceinline__ int cta_of(const P &p, int total, int u)
{
    const int part = total / p.ctas, more = total - part * p.ctas;
    const int head = more * (part + 1); // tiles of the CTAs with one more
    return u < head ? u / (part + 1) : more + (u - head) / part;
}

// Walks a CTA's run of tiles, segment by segment (the tiles of one (sequence,
// KV head)).
struct Segments {
    int b, h, tile, left;      // next tile, tiles left in the run
    int T, n, tiles;           // sequence b
    int seg_tile0, seg_tile1;  // current segment
    template <typename S>
    __device__ explicit Segments(const S &s)
        : b(s.start_b), h(s.start_h), tile(s.start_tile), left(s.units), T(s.start_T), n(s.start_n),
          tiles((s.start_T - 1) / kTileKeys + 1)
    {
    }
    template <typename P>
    __device__ bool next(const P &p)
    {
        if (left <= 0)
            return false;
        if (tile >= tiles) {
            tile = 0;
            if (++h == p.Hkv) {
                h = 0;
                do {
                    if (++b >= p.B)
                        return false;
                    tiles = tiles_of(p, b, T, n);
                } while (tiles == 0);
            }
        }
        seg_tile0 = tile;
        seg_tile1 = min(tiles, tile + left);
        left -= seg_tile1 - tile;
        tile = seg_tile1;
        return true;
    }
};

// Finds CTA `cta`'s run, by the whole block; the caller synchronises it afterwards.
template <int kThreads, typename P, typename S> __device__ __forceinline__ void plan_run(const P &p, S &s, int cta)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // This CTA's run of tiles: thread t sums the tiles of sequences [t per, (t + 1) per).
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int mine = 0, T, n;
    for (int b = b0; b < b1; ++b)
        mine += tiles_of(p, b, T, n) * p.Hkv;
    int before = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, off);
        if (lane >= off)
            before += v;
    }
    if (lane == 31)
        s.scan[warp] = before;
    before -= mine;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp)
            before += s.scan[w];
        total += s.scan[w];
    }
    int u0;
    const int units = run_of(p, total, cta, u0);
    if (tid == 0)
        s.units = units;
    if (mine > 0 && u0 >= before && u0 < before + mine) {
        int b = b0, at = before, tiles = mine / p.Hkv; // of one head of sequence b
        if (per > 1)
            for (; at + (tiles = tiles_of(p, b, T, n)) * p.Hkv <= u0; ++b)
                at += tiles * p.Hkv;
        s.start_b = b;
        s.start_h = (u0 - at) / tiles;
        s.start_tile = u0 - at - s.start_h * tiles;
        s.start_T = T;
        s.start_n = n;
    }
    if (blockIdx.x == 0) { // for the merge
        if (per == 1) {
            if (b0 < b1)
                p.unit_base[b0] = before;
        } else {
            int at = before;
            for (int b = b0; b < b1; ++b) {
                p.unit_base[b] = at;
                at += tiles_of(p, b, T, n) * p.Hkv;
            }
        }
        if (tid == 0)
            p.unit_base[p.B] = total;
    }
}

// a - b as a float for any two int32 (by halves: the difference of 64-bit
// integers would go through this GPU's slow 64-bit conversion).
__device__ __forceinline__ float distance(int a, int b)
{
    return fmaf(2.f, static_cast<float>((a >> 1) - (b >> 1)), static_cast<float>((a & 1) - (b & 1)));
}

// The cap c tanh(u), u = scale x / c. For |u| <= 1 the polynomial u P(u^2), whose
// error is relative to the value (degree 6 in u^2, fitted to tanh(u) / u on [0, 1]:
// 5e-8; 3 units of 2^-24 evaluated in fp32), and which takes no turn of the
// special-function unit; only scores past their cap take c - 2 c / (1 + e^2|u|),
// whose error is relative to 2 c / (1 + e^2|u|).
constexpr int kTanhTerms = 7;
constexpr double kTanh[kTanhTerms] = {0.9999999502432662,   -0.33332839158678823, 0.13325204110108205,
                                      -0.053457030406905304, 0.020289981289038105, -0.006203379388692019,
                                      0.0010410225990803521};

// Joins the pieces of every (sequence, KV head) that several CTAs worked on:
//   top = max m_k, out = sum acc_k 2^(m_k - top) / sum l_k 2^(m_k - top).
// A row belongs to kParts warps; warp w takes pieces w, w + kParts, .. in order
// (each with all its loads in flight at once), and the sums are added in order.
// What bounds it is latency: two trips to memory after the lengths. Rows of
// sequences whose lengths make no sense become zeros here.
template <int kParts, typename P>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ P p)
{
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ float4 sums[kMergeThreads];
    __shared__ float sum_l[kMergeThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kParts;
    const int r = blockIdx.x * (kMergeThreads / 32 / kParts) + warp / kParts;
    const int h = blockIdx.y, b = blockIdx.z;
    const int token = r / p.g;
    int T, n;
    const int base = p.unit_base[b], total = p.unit_base[p.B];
    const bool good = sequence(p, b, T, n);
    const int tiles = (T - 1) / kTileKeys + 1;
    int c0 = 0, c1 = 0;
    if (good && n > 0) {
        c0 = cta_of(p, total, base + h * tiles);
        c1 = cta_of(p, total, base + (h + 1) * tiles - 1);
    }
    if (good && c0 == c1) // nothing to join (the same for the whole block)
        return;
    const bool live = r < p.M * p.g && (!good || token < n);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (good && live) {
        const int row_tile = token / p.tile_tokens, rg = row_tile / P::kTilesPerRecord;
        const int rec_row = row_tile % P::kTilesPerRecord * P::kRowsPerTile + r - row_tile * p.tile_tokens * p.g;
        // piece k is CTA c0 + k's: its last segment for the first piece, its first for the others
        const auto record = [&](int k) {
            return (static_cast<size_t>(c0 + k) * p.row_groups + rg) * 2 * p.rec_rows + (k == 0 ? p.rec_rows : 0) + rec_row;
        };
        const int pieces = c1 - c0 + 1;
        constexpr int kFlight = 8; // this warp's pieces in flight
        for (int first = 0; first < pieces; first += kFlight * kParts) {
            float4 v[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int k = first + kParts * i + part;
                if (k < pieces)
                    v[i] = reinterpret_cast<const float4 *>(p.rec_acc + record(k) * kHeadDim)[lane];
            }
            // the reference over all pieces, the same in all of the row's warps
            float top = -INFINITY;
            for (int k = lane; k < pieces; k += 32) {
                const float m = p.rec_m[record(k)], piece_l = p.rec_l[record(k)];
                top = piece_l == 0.f ? top : fmaxf(top, m);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            const int mine = first + kParts * lane + part; // lane i holds piece i of this warp
            float w = 0.f, piece_l = 0.f;
            if (lane < kFlight && mine < pieces) {
                piece_l = p.rec_l[record(mine)];
                w = piece_l == 0.f ? 0.f : ex2(p.rec_m[record(mine)] - top);
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const float wi = __shfl_sync(0xFFFFFFFFu, w, i), li = __shfl_sync(0xFFFFFFFFu, piece_l, i);
                if (li != 0.f) { // a piece without a visible key counts for nothing
                    l = fmaf(li, wi, l);
                    acc.x = fmaf(v[i].x, wi, acc.x);
                    acc.y = fmaf(v[i].y, wi, acc.y);
                    acc.z = fmaf(v[i].z, wi, acc.z);
                    acc.w = fmaf(v[i].w, wi, acc.w);
                }
            }
        }
    }
    if (!good && r == 0 && h == 0 && threadIdx.x == 0)
        P::raise(PGQA_DEVERR_BAD_CONTEXT);
    sums[threadIdx.x] = acc;
    if (lane == 0)
        sum_l[warp] = l;
    __syncthreads();
    if (!live || part != 0)
        return;
    for (int i = 1; i < kParts; ++i) {
        const float4 v = sums[threadIdx.x + 32 * i];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        l += sum_l[warp + i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    const size_t out_row = (static_cast<size_t>(b) * p.M + token) * p.Hq + h * p.g + r % p.g;
    if (p.out_f32)
        reinterpret_cast<float4 *>(p.out_f32 + out_row * kHeadDim)[lane] = acc;
    if (p.out_bf16)
        reinterpret_cast<uint2 *>(p.out_bf16 + out_row * kHeadDim)[lane] =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

template <typename P> cudaError_t launch_tree_merge(const P &p, int ctas, cudaStream_t stream)
{
    // Four warps a row where a (sequence, head) is cut into many pieces, one where
    // there are few pieces each or many rows (four times the blocks). With four and
    // one, g = 2 unless said, pieces being CTAs per head: 19 pieces, 128 to 2048 rows in all
    // (M = 8 to 32, g = 8 at last): 21.1 and 25.2, 16.9 and 23.5, 25.5 and 31.1 us; 9.5
    // pieces, 1024, 2048 and 4096 rows: 22.0 and 24.5, 21.7 and 22.3, 37.7 and 32.2; 6.3
    // pieces, 768 and 1536: 20.3 and 20.7, 27.1 and 25.9; 4.75 pieces, 1024 and 2048: 26.4
    // and 27.2, 30.7 and 28.6; 3.2 pieces, 144, 384 and 1536: 30.4 and 30.3, 24.8 and 24.5,
    // 26.8 and 25.0; 1.2 pieces, 32768 (g = 8): 153 and 102. (With the bf16 kernel; the INT8 one
    // shares the rule.)
    const long long heads = static_cast<long long>(p.B) * p.Hkv, rows_in_all = static_cast<long long>(p.B) * p.M * p.Hq;
    const int parts = ctas >= 4 * heads && rows_in_all * heads <= 220ll * ctas ? 4 : 1;
    const int per_block = kMergeThreads / 32 / parts;
    const dim3 grid(static_cast<unsigned>((p.M * p.g + per_block - 1) / per_block), static_cast<unsigned>(p.Hkv),
                    static_cast<unsigned>(p.B));
    return launch_pdl(parts == 4 ? tree_merge_kernel<4, P> : tree_merge_kernel<1, P>, grid, dim3(kMergeThreads), 0, stream, p);
}

} // namespace
} // namespace pgqa
