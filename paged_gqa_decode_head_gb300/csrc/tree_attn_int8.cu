// tree_attn_int8.cu -- decode_attn_paged_tree_int8: attention of a tree of
// drafted tokens over the paged INT8 cache, with an optional tanh cap and
// distance bias.
//
// Mathematics. As decode_attn_paged_tree (tree_attn.cu): x = scale Q K^T, capped
// and biased, softmax over the keys that a row sees, O = P V, in tiles of 128 keys
// with a running reference m and sum l per row. A key's K row is ks * code, its V
// row vs * code: the codes enter the products exactly, as fp16, and the scales
// multiply what stands for that key, the scores (ks) and the weights (vs).
//
// Layout. The keys are the M = 128 rows of both products and the query rows (drafted
// token, head) their N columns: S^T = K Q^T, O^T = V^T P^T. So
//   - a softmax thread owns a key: its two scales are two registers, and the work
//     grows with the rows that there are (8, 16, 32 or 64 columns), not with a tile of 128;
//   - K^T's operand comes from tensor memory, lane = key, written there by the thread
//     that converted the key's codes; V's and P's lie in shared memory, dims and rows
//     contiguous;
//   - the maximum over the keys is not needed in a tile: a thread only asks whether one
//     of its terms 2^x vs rises more than 8 (base 2) above the row's reference. If one does
//     in any of the 128 threads, the references move and l and O are rescaled. The tiles of
//     a run are taken from its end, so that under a distance bias, whose usual sign favours
//     the nearest keys, the first ones bring the maximum.
// Sums l stay in the threads, one per row, until a segment's end.
//
// Queries enter their product as fp16. bf16's range is far larger, so a row is divided by a
// unit 2^(16 k) to a largest element in [2^-4, 2^12): its elements are exact down to 2^-13 of
// the largest at least, and off by 2^-21 of the largest below. k is 0 for rows whose largest
// lies there, as normalised queries' does; where all rows of a CTA have one k, the unit
// multiplies the keys' scales, and only rows of very different sizes take a factor per score.
//
// Rounding. P vs enters its product as an fp16 pair hi + lo (22 bits), two columns of
// one product. A row's reference r belongs to what goes in there, not to its scores: the
// largest term 2^(x - r) |vs| that the row has met lies in [2^6, 2^15), so that the pair does
// not overflow, and what half its smallest step, 2^-25, takes from a term is at most 2^-31 of
// the row's largest, whatever the V scales of keys that other rows see or that hardly weigh.
// Sums l take the same 2^(x - r): up to 2^95 for keys whose V is next to nothing (a V scale
// counts as 2^-80 at least), which fp32 holds for 2^30 keys. V scales are in units of F, a
// power of two which brings the largest in the first tile, of the keys that all rows see, to
// [8, 16), so that their own size does not matter; one above 2^60 makes F smaller. S, O, m and
// l are fp32; for fp32 outputs O moves out of the tensor core every kSpan tiles, as in
// tree_attn.cu.
//
// Bound. The cache is read once: 264 bytes per (key, KV head), 33 KB a tile of K and V, some
// 1440 clocks of an SM's share of the memory. Measured: 64 sequences of 16384 keys and 8 heads
// at 8 rows 389 us, 5.7 TB/s, 0.84 of the measured copy bandwidth (pages of 64; of 16, whose
// 16 boxes a tile one thread issues in some 1300 clocks, 419 us); at 32 rows 487 us, 4.5 TB/s,
// the two softmax warpgroups' work (2300 clocks a tile: one key's rows a thread in sequence,
// and code that the instruction caches do not hold); 512 rows per KV head, 16384 keys, 8
// sequences 610 us, 451 TFLOP/s; 64 rows 122 us. Rows of very different sizes, whose scores are
// scaled one by one: at 32 rows 549 us, 512 rows 730 us.
//
// Pairs. Where a (sequence, KV head) has more than 64 rows a CTA has two groups of them, one
// for each stream, which both take every tile: its codes are widened once for 128 rows (512
// rows: 707 us with a CTA per group of 64, 596 us in pairs, before rows had units and V
// scales a share in the references).
//
// CTA: one per SM, five warpgroups (four at 64 rows, whose softmax wants the registers)
// around tensor memory and rings of three (two) tiles of K's and V's codes. Two streams take
// alternate tiles of the CTA's run:
//   warps 0-3, 4-7    one softmax warpgroup per stream: S -> P -> shared memory;
//   warps 8-11        widen K's codes to fp16 into tensor memory, for both streams;
//   warps 12-15       widen V's into shared memory (at 64 rows warps 8-11 do);
// and four warps alone:
//   the first         requests codes (TMA, a box per page of a tile);
//   the second        prepares the next segment's queries, masks and slopes;
//   the other two     issue one stream's products each, S and O += P V, as their operands
//                     come.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "tensor_map.h"
#include "tree_runs.cuh"

#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>

namespace pgqa {
namespace {

__device__ unsigned g_flags_tree_int8;

constexpr int kCodeBytes = kTileKeys * kHeadDim; // 16 KB of K or V codes
constexpr float kTop = 7.f;   // a row's largest term, in base 2, when its reference is set
constexpr float kRise = 8.f;  // its rise that moves the reference
constexpr float kLeastScale = -80.f, kMostScale = 60.f;   // V scales in units of F, in base 2
constexpr float kLeastVf = 0x1p-80f, kMostTerm = 0x1p15f; // 2^kLeastScale, 2^(kTop + kRise)
constexpr int kSpan = 16;     // a stream's tiles between two moves of O out of the tensor core (fp32 outputs)
constexpr int kMaxRows = 64;  // query rows of a row group

// TMEM columns of stream s, + 256 s: S^T (64), K (64, two fp16 each), O^T (128).
constexpr uint32_t kColS = 0, kColK = 64, kColO = 128, kStreamColumns = 256;

struct TreeInt8Params {
    static constexpr int kTilesPerRecord = 1, kRowsPerTile = kMaxRows;
    static __device__ void raise(unsigned flag) { atomicOr(&g_flags_tree_int8, flag); }
    const uint16_t *q;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *context_lens;
    const uint64_t *tree_mask;
    const int32_t *positions, *draft_lens;
    const float *slopes;
    int B, M, Hq, Hkv, log2_page, max_pages, num_pages;
    int g;             // query heads per KV head
    int tile_tokens;   // drafted tokens of a row group (g * tile_tokens <= 64 rows)
    int row_groups;    // that share a run of tiles
    int rec_rows;      // rows of a partial record
    int ctas;          // runs of tiles
    float c;               // plain scores: y = c ks S, c = scale log2 e
    float cap_u, cap_out;  // capped: y = cap_out tanh(cap_u ks S)
    float tanh_c[7];       // cap_out times the polynomial's coefficients
    float *out_f32;
    uint16_t *out_bf16;
    int32_t *unit_base;    // [B + 1] first tile number of each sequence, total
    float *rec_m, *rec_l;  // [2 * ctas * row_groups][rec_rows]
    float *rec_acc;        // [2 * ctas * row_groups][rec_rows][128]
    float *sums;           // [2 * grid][rows][128]: O of earlier spans; null: bf16 outputs only
};

// kRows: query rows of a CTA. Up to 64 both streams have all of them and take the tiles in
// turn. 128: a pair of row groups, 64 rows for each stream, which both take every tile.
template <int kRows> struct Shape {
    static constexpr bool kPair = kRows == 128;
    static constexpr int kOwn = kPair ? 64 : kRows;               // rows of a stream: the softmax's columns
    static constexpr int kSets = kPair ? 2 : 1, kTurns = kPair ? 1 : 2; // sets of rows; a stream's tiles are every kTurns-th
    static constexpr int kScoreColumns = kOwn < 16 ? 16 : kOwn;   // of S^T = K Q^T
    static constexpr int kOutColumns = kOwn == 64 ? 128 : 64;     // of O^T: hi, then lo
    static constexpr int kLo = kOutColumns / 2;                   // lo's first column
    static constexpr int kRing = kOwn == 64 ? 2 : 3;              // slots of K's codes
    static constexpr int kRingV = kPair ? 1 : kRing;              // and of V's
    static constexpr int kQueries = kOwn == 64 ? 1 : 2;           // segments whose queries are kept
    // Warps: softmax from 0, widening from 8 (K's and V's apart, or both), then four alone.
    static constexpr bool kApart = kOwn < 64;
    static constexpr int kThreads = kApart ? 640 : 512;
    static constexpr int kCodeWarp = kThreads / 32 - 4, kQueryWarp = kCodeWarp + 1, kMmaWarp = kCodeWarp + 2; // and + 3
    // Registers move to the softmax, within those of the launch: 96 or 128 a thread.
    static constexpr int kMost = kApart ? 128 : 176, kLeast = kApart ? 72 : 80;
    static_assert(256 * kMost + (kThreads - 256) * kLeast <= kThreads * (kApart ? 96 : 128), "registers of the launch");
};

template <int kRows> struct __align__(1024) TreeInt8Smem {
    using Sh = Shape<kRows>;
    unsigned char codes[Sh::kRing + Sh::kRingV][kCodeBytes]; // K's, V's
    unsigned char v16[2][kTileKeys * kRowBytes];
    unsigned char p16[2][kTileKeys * Sh::kOutColumns * 2];
    unsigned char q16[Sh::kQueries][Sh::kSets][Sh::kScoreColumns * kRowBytes];
    // what a segment's rows bring, for two segments in turn
    uint64_t sees[2][Sh::kSets][64]; // drafted token j: the rows that see it
    float slope_up[2][Sh::kSets][Sh::kOwn], slope_down[2][Sh::kSets][Sh::kOwn]; // slopes (base 2), split by sign
    int anchor[2][Sh::kSets][Sh::kOwn];
    // what the rows' queries were divided by twice; 0: each row by its own
    // (behind the rows' own: scale log2 e, or scale / cap)
    float q_root[2][Sh::kSets], q_roots[2][Sh::kSets][Sh::kOwn + 1];
    int by_sign[2][Sh::kSets]; // every row's anchor is the prefix's end, or its first key for a falling slope
    // a stream's rows
    float neg_m[2][Sh::kOwn]; // minus the reference
    float f_l[2][Sh::kOwn], f_o[2][Sh::kOwn], g_sums[2][Sh::kOwn];
    float warp_part[2][4][Sh::kOwn], warp_common[2][4], warp_vs[2][4];
    float m_end[2][Sh::kOwn], l_end[2][Sh::kOwn], inv_f[2];
    float weight[2][2][Sh::kOwn]; // by the stream that writes; of stream 0's and 1's O
    uint32_t warp_over[2][4];
    uint64_t code_full[Sh::kRing + Sh::kRingV], code_empty[Sh::kRing + Sh::kRingV];
    uint64_t q_full[Sh::kQueries], q_empty[Sh::kQueries];
    uint64_t rows_full[2], rows_empty[2];
    uint64_t k_ready[2], v_ready[2]; // a tile's codes are widened, in two places in turn
    uint64_t k_free[2], v_free[2];   // pairs: both streams' products have read them
    uint64_t s_full[2], s_read[2], p_ready[2], o_done[2], drain[2];
    uint32_t tmem_base;
    int start_b, start_h, start_tile, start_T, start_n, units; // this CTA's run
    int scan[Sh::kThreads / 32];
};
template <int kRows> constexpr int kInt8Smem = sizeof(TreeInt8Smem<kRows>);
static_assert(kInt8Smem<32> <= 232448 && kInt8Smem<64> <= 232448 && kInt8Smem<128> <= 232448, "one CTA's shared memory");

__device__ __forceinline__ void stream_sync(int stream)
{
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + stream) : "memory");
}
__device__ __forceinline__ bool stream_any(int stream, bool x)
{
    uint32_t y;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %2, 0;\n\tbarrier.cta.red.or.pred b, %1, 128, a;\n\t"
                 "selp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(y)
                 : "r"(1 + stream), "r"(x ? 1u : 0u)
                 : "memory");
    return y != 0;
}
__device__ __forceinline__ void both_streams_sync() { asm volatile("barrier.cta.sync 3, 256;" ::: "memory"); }

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Whether the phase with the given parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}

// As tmem_ld16, 8 columns.
__device__ __forceinline__ void tmem_ld8(float *r, uint32_t addr)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld8(float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float *r)
{
    const uint32_t *u = reinterpret_cast<const uint32_t *>(r);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// Instruction descriptor of kind::f16 with fp16 A and B, fp32 D, M = 128 (tcgen05.cuh);
// A "MN-major" (its M dimension contiguous) in bit 15.
__host__ __device__ constexpr uint32_t tc_idesc_f16(uint32_t n, bool mn_major)
{
    return (1u << 4) | ((mn_major ? 3u : 0u) << 15) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// The fp16 pair (22 bits) of two floats.
__device__ __forceinline__ void split_f16(f32x2 w, uint32_t &hi, uint32_t &lo)
{
    float a, b, ra, rb;
    w.get(a, b);
    hi = pack_f16x2(a, b);
    fma2(f32x2(f16_lo(hi), f16_hi(hi)), f32x2(-1.f, -1.f), w).get(ra, rb);
    lo = pack_f16x2(ra, rb);
}

// Sums over a warp's lanes of N values: lane i / (32 / N) gets that of value i (N <= 32).
template <int N> __device__ __forceinline__ float sum_lanes(float *x)
{
    const int lane = threadIdx.x & 31;
    int off = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, off /= 2) {
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = upper ? x[i + n] : x[i], give = upper ? x[i] : x[i + n];
            x[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, off);
        }
    }
    for (; off >= 1; off /= 2)
        x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], off);
    return x[0];
}

// ---------------------------------------------------------------- codes
template <int kRows>
__device__ bool fetch_codes(const TreeInt8Params &p, TreeInt8Smem<kRows> &s, const CUtensorMap *mk, const CUtensorMap *mv)
{
    using Sh = Shape<kRows>;
    const int lane = threadIdx.x & 31;
    const int P = 1 << p.log2_page;
    const int box_keys = min(P, kTileKeys);
    const int boxes = kTileKeys / box_keys; // pages of a tile
    const int outside = static_cast<int>(static_cast<long long>(p.num_pages) * p.Hkv << p.log2_page);
    // one row group reads the cache once; of several, running side by side, the
    // first leaves it in L2 for the others
    const uint64_t policy = p.row_groups <= Sh::kSets ? l2_evict_first_policy() : l2_evict_normal_policy();
    bool ok = true;
    const bool leader = elect_one();
    int unit = 0; // K's requested; V's are one behind, as they are widened
    int v_row = 0;
    const auto request = [&](int is_v, int u, int row) { // one tile's codes
        const int ring = is_v ? Sh::kRingV : Sh::kRing, slot = (is_v ? Sh::kRing : 0) + u % ring;
        ok = ok && warp_wait(&s.code_empty[slot], ((u / ring) & 1) ^ 1);
        if (!ok)
            return;
        uint64_t *full = &s.code_full[slot];
        int rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rows[i] = __shfl_sync(0xFFFFFFFFu, row, i);
        // One thread issues all boxes: a lane each would take its turn with all of a request's
        // latency, 66 clocks (of some 1400 in which the memory brings a tile).
        if (leader) {
            mbar_arrive_expect_tx(full, kCodeBytes);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < boxes) // a box outside the tensor arrives as zeros
                    tma_load_2d(s.codes[slot] + i * box_keys * kHeadDim, is_v ? mv : mk, 0, rows[i], full, policy);
        }
        __syncwarp();
    };
    Segments seg(s);
    while (ok && seg.next(p)) {
        const int32_t *table = p.block_table + static_cast<size_t>(seg.b) * p.max_pages;
        const auto entry = [&](int tile) {
            const int key = tile * kTileKeys + lane * box_keys;
            return lane < boxes && key < seg.T ? table[key >> p.log2_page] : 0;
        };
        int phys_next = entry(seg.seg_tile1 - 1);
        for (int tile = seg.seg_tile1 - 1; ok && tile >= seg.seg_tile0; --tile) {
            const int phys = phys_next;
            if (tile > seg.seg_tile0)
                phys_next = entry(tile - 1);
            const int key = tile * kTileKeys + lane * box_keys;
            const bool needed = lane < boxes && key < seg.T;
            const bool in_pool = phys >= 0 && phys < p.num_pages;
            const bool here = needed && in_pool;
            if (needed && !in_pool)
                atomicOr(&g_flags_tree_int8, PGQA_DEVERR_BAD_PAGE);
            const int row = here ? ((phys * p.Hkv + seg.h) << p.log2_page) + (key & (P - 1)) : outside;
            request(0, unit, row);
            if (!ok)
                break;
            if (unit > 0)
                request(1, unit - 1, v_row);
            v_row = row;
            ++unit;
        }
    }
    if (unit > 0)
        request(1, unit - 1, v_row);
    // Nothing may still be on its way into shared memory when the CTA ends: a slot's last
    // load each. (After a wait that ran out the last K's may have no V.)
    const int last_v = ok ? unit : unit - 1;
    for (int u = max(0, unit - Sh::kRing); u < unit; ++u)
        ok = warp_wait(&s.code_full[u % Sh::kRing], (u / Sh::kRing) & 1) && ok;
    for (int u = max(0, last_v - Sh::kRingV); u < last_v; ++u)
        ok = warp_wait(&s.code_full[Sh::kRing + u % Sh::kRingV], (u / Sh::kRingV) & 1) && ok;
    return ok;
}

// ---------------------------------------------------------------- queries and masks
// The square root of a row's unit 2^(16 k): the unit itself may lie past fp32's range.
__device__ __forceinline__ float root_of_unit(int k)
{
    return __uint_as_float(static_cast<uint32_t>(127 + 8 * k) << 23);
}

// The larger of two pairs' elements each, by size (their signs are of no use).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight bf16 elements divided by root twice (exact but for what falls below bf16's smallest).
__device__ __forceinline__ uint4 divided_twice(uint4 x, float root)
{
    const uint32_t inv = (254u << 7) - (__float_as_uint(root) >> 16), pair = inv << 16 | inv; // 1 / root
    const auto times = [pair](uint32_t v) {
        uint32_t r;
        asm("{\n\t.reg .b32 t;\n\tmul.rn.bf16x2 t, %1, %2;\n\tmul.rn.bf16x2 %0, t, %2;\n\t}"
            : "=r"(r)
            : "r"(v), "r"(pair));
        return r;
    };
    return make_uint4(times(x.x), times(x.y), times(x.z), times(x.w));
}

template <int kScore, int kRows>
__device__ bool fetch_rows(const TreeInt8Params &p, TreeInt8Smem<kRows> &s, int rg)
{
    using Sh = Shape<kRows>;
    const int lane = threadIdx.x & 31;
    const int rows = p.tile_tokens * p.g;
    bool ok = true;
    Segments seg(s);
    for (int index = 0; ok && seg.next(p); ++index) {
        const int buf = index & 1, qbuf = index % Sh::kQueries;
        const int n = seg.n, prefix = seg.T - n;
        ok = warp_wait(&s.rows_empty[buf], ((index >> 1) & 1) ^ 1);
        if (!ok)
            break;
#pragma unroll 1
        for (int set = 0; set < Sh::kSets; ++set) {
            const int token0 = (rg + set) * p.tile_tokens;
            const auto live = [&](int row) { return row < rows && token0 + row / p.g < n; };
            // masks by row become rows by drafted token
            const uint64_t *masks = p.tree_mask + static_cast<size_t>(seg.b) * p.M + token0;
            const uint64_t m0 = live(lane) ? masks[lane / p.g] : 0, m1 = live(lane + 32) ? masks[(lane + 32) / p.g] : 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const uint32_t lo = __ballot_sync(0xFFFFFFFFu, (m0 >> j) & 1u);
                const uint32_t hi = Sh::kOwn > 32 ? __ballot_sync(0xFFFFFFFFu, (m1 >> j) & 1u) : 0u;
                if (lane == (j & 31))
                    s.sees[buf][set][j] = static_cast<uint64_t>(hi) << 32 | lo;
            }
            if constexpr ((kScore & 2) != 0) {
                // A row's own position is a constant of its scores and cancels in the softmax: the
                // bias is taken relative to a key that it favours, as in tree_attn.cu.
                const int32_t *at = p.positions + static_cast<size_t>(seg.b) * p.M;
                const int pos_lo = lane < n ? at[lane] : 0, pos_hi = lane + 32 < n ? at[lane + 32] : 0;
                const auto near = [&](int j, int pos) {
                    return j >= n || static_cast<uint32_t>(pos) - static_cast<uint32_t>(prefix) + 64u < 128u;
                };
                bool by_sign = near(lane, pos_lo) && near(lane + 32, pos_hi);
                float slope[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = lane + 32 * i;
                    slope[i] = live(row) ? p.slopes[seg.h * p.g + row % p.g] * kLog2e : 0.f;
                    by_sign = by_sign && fabsf(slope[i]) <= 2.f;
                }
                by_sign = __all_sync(0xFFFFFFFFu, by_sign);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool falls = slope[i] < 0.f;
                    int anchor = falls ? 0 : prefix;
                    if (!by_sign) {
                        if (prefix == 0)
                            anchor = falls ? INT_MAX : INT_MIN;
                        const uint64_t mask = i ? m1 : m0;
#pragma unroll 1
                        for (int j = 0; j < n; ++j) {
                            const int pos = __shfl_sync(0xFFFFFFFFu, j < 32 ? pos_lo : pos_hi, j & 31);
                            if (mask >> j & 1u)
                                anchor = falls ? min(anchor, pos) : max(anchor, pos);
                        }
                    }
                    if (lane + 32 * i < Sh::kOwn) {
                        s.slope_up[buf][set][lane + 32 * i] = fmaxf(slope[i], 0.f);
                        s.slope_down[buf][set][lane + 32 * i] = fminf(slope[i], 0.f);
                        s.anchor[buf][set][lane + 32 * i] = anchor;
                    }
                }
                if (lane == 0)
                    s.by_sign[buf][set] = by_sign;
            }
        }
        // Every row's unit, from its largest element. A row has a few lanes, whose loads are on
        // their way together (and bring it near for its conversion).
        constexpr int kLanes = Sh::kOwn < 32 ? 32 / Sh::kOwn : 1;
#pragma unroll 1
        for (int set = 0; set < Sh::kSets; ++set) {
            const int token0 = (rg + set) * p.tile_tokens;
            int least = INT_MAX, most = INT_MIN; // k of the set's rows
#pragma unroll 1
            for (int row = lane / kLanes; row < Sh::kOwn; row += 32) {
                uint32_t pairs = 0; // the largest elements so far
                if (row < rows && token0 + row / p.g < n) {
                    const uint4 *from = reinterpret_cast<const uint4 *>(
                        p.q + ((static_cast<size_t>(seg.b) * p.M + token0 + row / p.g) * p.Hq + seg.h * p.g + row % p.g) *
                                  kHeadDim) + lane % kLanes;
#pragma unroll 8
                    for (int i = 0; i < 16 / kLanes; ++i) {
                        const uint4 x = from[i * kLanes];
                        pairs = larger(larger(larger(larger(pairs, x.x), x.y), x.z), x.w);
                    }
                }
                uint32_t top = max(pairs & 0x7FFFu, pairs >> 16 & 0x7FFFu); // ordered as the sizes
#pragma unroll
                for (int off = kLanes / 2; off >= 1; off /= 2)
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
                // 2^e <= the largest < 2^(e + 1), e = (top >> 7) - 127: k = floor((e + 4) / 16), -8 .. 8
                const int k = top ? (static_cast<int>(top >> 7) - 123) >> 4 : 0;
                if (top) // zeros fit any unit
                    least = min(least, k), most = max(most, k);
                s.q_roots[buf][set][row] = root_of_unit(k);
            }
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            if (lane == 0) {
                s.q_root[buf][set] = most > least ? 0.f : root_of_unit(most < least ? 0 : least);
                s.q_roots[buf][set][Sh::kOwn] = kScore & 1 ? p.cap_u : p.c;
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.rows_full[buf]);
        ok = warp_wait(&s.q_empty[qbuf], ((index / Sh::kQueries) & 1) ^ 1);
        if (!ok)
            break;
        // Q as the K-major operand: two halves of 64 dims, swizzled 8-row atoms; rows that
        // do not exist are zeros
        const int part = lane & 15, half = part >> 3;
        constexpr int kFlight = Sh::kScoreColumns / 2 < 8 ? Sh::kScoreColumns / 2 : 8;
#pragma unroll 1
        for (int at = 0; at < Sh::kSets * Sh::kScoreColumns; at += 2 * kFlight) {
            const int set = at / Sh::kScoreColumns, r0 = at % Sh::kScoreColumns;
            const int token0 = (rg + set) * p.tile_tokens;
            const auto live = [&](int row) { return row < rows && token0 + row / p.g < n; };
            uint4 x[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int row = r0 + 2 * i + (lane >> 4);
                x[i] = make_uint4(0, 0, 0, 0);
                if (live(row))
                    x[i] = reinterpret_cast<const uint4 *>(
                        p.q + ((static_cast<size_t>(seg.b) * p.M + token0 + row / p.g) * p.Hq + seg.h * p.g + row % p.g) *
                                  kHeadDim)[part];
            }
            if (__builtin_expect(s.q_root[buf][set] != 1.f, 0)) {
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const int row = r0 + 2 * i + (lane >> 4);
                    if (row < Sh::kOwn)
                        x[i] = divided_twice(x[i], s.q_roots[buf][set][row]);
                }
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int row = r0 + 2 * i + (lane >> 4);
                const auto convert = [](uint32_t pair) { return pack_f16x2(bf16_lo(pair), bf16_hi(pair)); };
                *reinterpret_cast<uint4 *>(s.q16[qbuf][set] + half * (Sh::kScoreColumns * 128) + row * 128 +
                                           (((part & 7) ^ (row & 7)) << 4)) =
                    make_uint4(convert(x[i].x), convert(x[i].y), convert(x[i].z), convert(x[i].w));
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.q_full[qbuf]);
    }
    return ok;
}

// ---------------------------------------------------------------- a stream
// 16 codes of a row -> 16 fp16, as two times 16 bytes.
__device__ __forceinline__ void widen_codes(const uint4 &codes, uint32_t *out)
{
    const uint32_t words[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t biased = words[i] ^ 0x80808080u;
        out[2 * i] = biased8x2_to_f16x2(biased, 0x100u);
        out[2 * i + 1] = biased8x2_to_f16x2(biased, 0x302u);
    }
}

// Both streams' codes, widened tile by tile: a thread has a key. Where one warpgroup has K and
// V, V follows one tile behind, as K's product and softmax come before V is wanted.
template <int kRows, bool kHasK, bool kHasV> __device__ bool widen(const TreeInt8Params &p, TreeInt8Smem<kRows> &s)
{
    using Sh = Shape<kRows>;
    constexpr int kRing = Sh::kRing, kRingV = Sh::kRingV;
    uint64_t *k_free = Sh::kPair ? s.k_free : s.s_full, *v_free = Sh::kPair ? s.v_free : s.o_done;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int key_row = warp * 32 + lane;
    bool ok = true;
    // A row's chunks of 16 codes, four at a time: the loops are small enough to stay in the
    // scheduler's own instruction cache.
    const auto load4 = [&](const unsigned char *codes, int c0, uint4 *row) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            row[c] = *reinterpret_cast<const uint4 *>(codes + key_row * kHeadDim + (((c0 + c) ^ (key_row & 7)) << 4));
    };
    for (int unit = kHasK ? 0 : 1; unit < s.units + kHasV; ++unit) {
        uint4 row[4];
        if (kHasK && unit < s.units) {
            const int stream = unit & 1, step = unit >> 1, slot = unit % kRing;
            const uint32_t tmem_k = s.tmem_base + (static_cast<uint32_t>(warp * 32) << 16) + stream * kStreamColumns + kColK;
            ok = ok && warp_wait(&s.code_full[slot], (unit / kRing) & 1);
            // the last K of the stream is read
            if (step > 0)
                ok = ok && warp_wait(&k_free[stream], (step - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; c += 4) {
                load4(s.codes[slot], c, row);
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    uint32_t w[16];
                    widen_codes(row[i], w);
                    widen_codes(row[i + 1], w + 8);
                    tmem_st16(tmem_k + 8 * (c + i), reinterpret_cast<const float *>(w));
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.code_empty[slot]);
                mbar_arrive(&s.k_ready[stream]);
            }
        }
        if (kHasV && unit > 0) {
            const int last = unit - 1, stream = last & 1, step = last >> 1, slot = kRing + last % kRingV;
            ok = ok && warp_wait(&s.code_full[slot], (last / kRingV) & 1);
            // the last tile's product with V is through with the buffer
            if (step > 0)
                ok = ok && warp_wait(&v_free[stream], (step - 1) & 1);
            unsigned char *v_row = s.v16[stream] + (key_row >> 3) * 2048 + (key_row & 7) * 128;
#pragma unroll 1
            for (int c = 0; c < 8; c += 4) { // half a row of fp16
                load4(s.codes[slot], c, row);
                unsigned char *half = v_row + c * 256;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[8];
                    widen_codes(row[i], w);
                    *reinterpret_cast<uint4 *>(half + ((2 * i ^ (key_row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(half + ((2 * i + 1 ^ (key_row & 7)) << 4)) =
                        make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.code_empty[slot]);
                mbar_arrive(&s.v_ready[stream]);
            }
        }
    }
    return ok;
}

// ---------------------------------------------------------------- matrix products
template <int kRows> __device__ bool multiply(const TreeInt8Params &p, TreeInt8Smem<kRows> &s, int stream)
{
    using Sh = Shape<kRows>;
    const bool leader = elect_one(); // issues every product and commit
    const uint32_t tmem = warp_uniform(s.tmem_base + stream * kStreamColumns);
    const uint32_t idesc_s = tc_idesc_f16(Sh::kScoreColumns, false);
    const uint32_t idesc_o = tc_idesc_f16(Sh::kOutColumns, true);
    // where tile `step` of this stream is widened to, and how often that was filled before
    const auto place = [&](int step) { return Sh::kPair ? step & 1 : stream; };
    const auto filled = [&](int step) { return Sh::kPair ? step >> 1 : step; };
    const uint32_t va0 = warp_uniform(tc_desc_low(smem_addr(s.v16[0]), 1024));
    const uint32_t va1 = warp_uniform(tc_desc_low(smem_addr(s.v16[1]), 1024));
    const uint32_t pa = warp_uniform(tc_desc_low(smem_addr(s.p16[stream]), 1024));
    constexpr int kStepP = Sh::kOwn == 64 ? 4096 : 2048; // 16 keys of P
    bool ok = true;
    const auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && warp_wait(bar, parity); };
    const auto passed = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)); };
    Segments seg(s);
    int unit0 = 0, step = 0;
    bool keep = false;    // the last tile's product adds to O
    bool pending = false; // the last tile's product is not issued yet
    for (int index = 0; ok && seg.next(p); ++index) {
        const int qbuf = index % Sh::kQueries, tiles = seg.seg_tile1 - seg.seg_tile0;
        const int first = Sh::kPair ? 0 : (unit0 ^ stream) & 1;
        wait(&s.q_full[qbuf], (index / Sh::kQueries) & 1);
        const uint32_t qa = warp_uniform(tc_desc_low(smem_addr(s.q16[qbuf][Sh::kPair ? stream : 0]), 16));
        if (first >= tiles && leader)
            mbar_arrive(&s.q_empty[qbuf]);
        // The last tile's product with V is left to the turn of the next one's scores. Where the
        // segment has no tile for this stream it is made at once: its end must come before the
        // rows of the segment after this. So is that of the run's last tile.
        const int end = first >= tiles || seg.left <= 0 ? tiles + Sh::kTurns : tiles;
        for (int i = first; ok && i < end; i += Sh::kTurns) {
            bool scores = i < tiles; // to be issued
            const long long start = clock64();
            while (ok && (scores || pending)) {
                if (scores && passed(&s.k_ready[place(step)], filled(step) & 1) &&
                    (step == 0 || passed(&s.s_read[stream], (step - 1) & 1))) {
                    tc_fence_after();
                    const uint32_t tmem_k = warp_uniform(s.tmem_base + place(step) * kStreamColumns + kColK);
                    if (leader) { // S^T = K Q^T
#pragma unroll
                        for (int k = 0; k < kHeadDim / 16; ++k) // 64 dims a half, 32 bytes a step
                            tc_mma_ts(tmem + kColS, tmem_k + 8 * k,
                                      qa + (k >> 2) * (Sh::kScoreColumns * 128 / 16) + (k & 3) * 2, tc_desc_high(1024),
                                      idesc_s, k > 0);
                        tc_commit(&s.s_full[stream]);
                        if (Sh::kPair)
                            tc_commit(&s.k_free[step & 1]);
                        if (i + Sh::kTurns >= tiles)
                            tc_commit(&s.q_empty[qbuf]);
                    }
                    __syncwarp();
                    scores = false;
                }
                if (pending && passed(&s.p_ready[stream], (step - 1) & 1) &&
                    passed(&s.v_ready[place(step - 1)], filled(step - 1) & 1)) {
                    tc_fence_after();
                    const uint32_t va = warp_uniform(place(step - 1) ? va1 : va0);
                    if (leader) { // O^T (+)= V^T P^T
#pragma unroll
                        for (int k = 0; k < kTileKeys / 16; ++k)
                            tc_mma_ss(tmem + kColO, va + k * (4096 / 16), tc_desc_high(2048), pa + k * (kStepP / 16),
                                      tc_desc_high(kStepP / 2), idesc_o, k > 0 || keep);
                        tc_commit(&s.o_done[stream]);
                        if (Sh::kPair)
                            tc_commit(&s.v_free[(step - 1) & 1]);
                    }
                    __syncwarp();
                    pending = false;
                }
                ok = __all_sync(0xFFFFFFFFu, clock64() - start < kWaitLimitClocks);
            }
            if (i < tiles) {
                keep = i > first && !(p.sums && (i - first) / Sh::kTurns % kSpan == 0);
                pending = true;
                ++step;
            }
        }
        unit0 += tiles;
    }
    // no product may still be running when the CTA ends
    if (leader)
        tc_commit(&s.drain[stream]);
    return warp_wait(&s.drain[stream], 0) && ok;
}

// ---------------------------------------------------------------- softmax
// Eight scores of this thread's key, from S to base 2 without the reference; kScore bit 0:
// capped, bit 1: biased; plain ones are left as S (the caller has the factor). j: the first
// one's row.
template <int kScore, int kRows>
__device__ __forceinline__ void form_scores(const TreeInt8Params &p, const TreeInt8Smem<kRows> &s, float *x, int j,
                                            float factor, int buf, int set, float up, float down, int pos)
{
    if constexpr ((kScore & 1) != 0) {
        float u[8], over = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const f32x2 v = mul2(f32x2(x[k], x[k + 1]), f32x2(factor, factor)), t = mul2(v, v);
            float t0, t1;
            t.get(t0, t1);
            over = max3(over, t0, t1);
            f32x2 y(p.tanh_c[kTanhTerms - 1], p.tanh_c[kTanhTerms - 1]);
#pragma unroll
            for (int i = kTanhTerms - 2; i >= 0; --i)
                y = fma2(y, t, f32x2(p.tanh_c[i], p.tanh_c[i]));
            v.get(u[k], u[k + 1]);
            mul2(v, y).get(x[k], x[k + 1]);
        }
        if (__any_sync(0xFFFFFFFFu, over > 1.f)) { // scores past their cap
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float size = fabsf(u[k]), rest = rcp(1.f + ex2(size * (2.f * kLog2e)));
                const float y = copysignf(fmaf(-2.f * p.cap_out, rest, p.cap_out), u[k]);
                x[k] = size > 1.f ? y : x[k];
            }
        }
    }
    if constexpr ((kScore & 2) != 0) {
        if constexpr ((kScore & 1) == 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] *= factor;
        }
        const float *slope_up = s.slope_up[buf][set] + j, *slope_down = s.slope_down[buf][set] + j;
        if (s.by_sign[buf][set]) {
#pragma unroll
            for (int k = 0; k < 8; k += 2)
                fma2(f32x2(slope_up[k], slope_up[k + 1]), f32x2(up, up),
                     fma2(f32x2(slope_down[k], slope_down[k + 1]), f32x2(down, down), f32x2(x[k], x[k + 1])))
                    .get(x[k], x[k + 1]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = fmaf(slope_up[k] + slope_down[k], distance(pos, s.anchor[buf][set][j + k]), x[k]);
        }
    }
}

// A key's scores in place, each by its K scale, the call's factor and its row's unit, in an order
// in which no partial product is past fp32's range before the score itself is (a call, as it is
// rarely made and its code would take registers and instruction cache from the loop around it).
__device__ __noinline__ void apply_units(uint32_t tmem_s, float ks, const float *roots, int n)
{
    const float plain = roots[n];
#pragma unroll 1
    for (int j = 0; j < n; j += 8) {
        float y[8];
        tmem_ld8(y, tmem_s + j);
        tmem_wait_ld8(y);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = y[k] * ks * roots[j + k] * plain * roots[j + k];
        tmem_st8(tmem_s + j, y);
    }
    tmem_wait_st();
}

template <int kScore, int kRows> __device__ bool soften(const TreeInt8Params &p, TreeInt8Smem<kRows> &s, int rg, int stream)
{
    using Sh = Shape<kRows>;
    constexpr int kOwn = Sh::kOwn, kTurns = Sh::kTurns;
    constexpr int kGroups = kOwn / 8; // rows are taken eight at a time
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int key_row = warp * 32 + lane; // of a tile; of O^T: the dim
    const int set = Sh::kPair ? stream : 0; // of the segment's rows
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tmem_s = s.tmem_base + lanes + stream * kStreamColumns + kColS;
    const uint32_t tmem_o = s.tmem_base + lanes + stream * kStreamColumns + kColO;
    // A wait that ran out ends no loop: all of a stream's warps meet at its barriers, and
    // do so to the end, without further waits.
    bool ok = true;
    const auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && warp_wait(bar, parity); };
    float *sums = p.sums ? p.sums + static_cast<size_t>(2 * blockIdx.x + stream) * kOwn * kHeadDim + key_row : nullptr;
    // what the threads of one stream share by row
    float *neg_m = s.neg_m[stream], *f_l = s.f_l[stream], *f_o = s.f_o[stream], *g_sums = s.g_sums[stream];
    float (*warp_part)[kOwn] = s.warp_part[stream];

    Segments seg(s);
    int unit0 = 0; // the segment's first tile in the run
    int step = 0;  // this stream's tiles so far
    for (int index = 0; seg.next(p); ++index) {
        const int buf = index & 1;
        const int tiles = seg.seg_tile1 - seg.seg_tile0;
        const int prefix = seg.T - seg.n;
        if (key_row < kOwn) {
            neg_m[key_row] = INFINITY; // nothing seen yet
            g_sums[key_row] = 1.f;
        }
        stream_sync(stream);
        float l[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            l[j] = 0.f;
        float f = 0.f;                 // F; 0 until a row sees a key
        bool summed = false;           // `sums` holds earlier spans
        bool large = false;            // a reference beyond 65536
        const int first = Sh::kPair ? 0 : (unit0 ^ stream) & 1;
        // This thread's key's scales come a tile ahead of their use, its page two.
        const int32_t *table = p.block_table + static_cast<size_t>(seg.b) * p.max_pages;
        const int first_key = seg.seg_tile0 * kTileKeys + key_row;
        int next_key = (seg.seg_tile1 - 1 - first) * kTileKeys + key_row;
        float next_ks = 0.f, next_vs = 0.f;
        bool next_valid = false;
        int next_page = next_key >= first_key && next_key < seg.T ? table[next_key >> p.log2_page] : -1;
        const auto load_scales = [&] { // of next_key, whose page next_page is
            next_valid = static_cast<unsigned>(next_page) < static_cast<unsigned>(p.num_pages);
            const int row = ((next_page * p.Hkv + seg.h) << p.log2_page) + (next_key & ((1 << p.log2_page) - 1));
            next_ks = next_vs = 0.f;
            if (next_valid)
                next_ks = p.k_scale[row], next_vs = p.v_scale[row];
            next_key -= kTurns * kTileKeys;
            next_page = next_key >= first_key ? table[next_key >> p.log2_page] : -1;
        };
        load_scales();
        wait(&s.rows_full[buf], (index >> 1) & 1);
        // scale log2 e, or scale / cap, in the unit of the rows' queries, where they have one and
        // the product keeps well within fp32's range; 0: row by row
        const float root = s.q_root[buf][set], in_unit = (kScore & 1 ? p.cap_u : p.c) * root * root;
        const float by = root == 1.f || (fabsf(in_unit) > 0x1p-100f && fabsf(in_unit) < 0x1p100f) ? in_unit : 0.f;
        for (int i = first; i < tiles; i += kTurns, ++step) {
            const int key0 = (seg.seg_tile1 - 1 - i) * kTileKeys, key = key0 + key_row;
            float factor = next_ks * (by == 0.f ? 1.f : by), vs = next_vs; // a score is S times the factor
            const bool valid = next_valid;
            load_scales();
            wait(&s.s_full[stream], step & 1);
            tc_fence_after();
            // ---- the rows that see this key
            uint32_t sees_lo = 0xFFFFFFFFu, sees_hi = 0xFFFFFFFFu;
            const bool fix = __any_sync(0xFFFFFFFFu, key >= prefix || !valid);
            if (fix) {
                const uint64_t sees = !valid ? 0 : key < prefix ? ~0ull : s.sees[buf][set][key - prefix];
                sees_lo = static_cast<uint32_t>(sees), sees_hi = static_cast<uint32_t>(sees >> 32);
                if (!sees)
                    factor = vs = 0.f; // may hold anything
            }
            const auto seen = [&](int j) { return (j < 32 ? sees_lo : sees_hi) >> (j & 31); };
            if (__builtin_expect(by == 0.f, 0)) {
                apply_units(tmem_s, factor, s.q_roots[buf][set], kOwn);
                factor = 1.f;
            }
            // Capped and biased scores are formed in place, in a loop small enough for the
            // instruction cache.
            if constexpr (kScore != 0) {
                int pos = key;
                float up = 0.f, down = 0.f;
                if constexpr ((kScore & 2) != 0) {
                    if (key >= prefix && key < seg.T)
                        pos = p.positions[static_cast<size_t>(seg.b) * p.M + key - prefix];
                    up = distance(pos, prefix), down = distance(pos, 0);
                }
                float y[2][8];
                tmem_ld8(y[0], tmem_s);
                const auto group = [&](int j, float *now, float *next) {
                    tmem_wait_ld8(now);
                    if (j + 8 < kOwn)
                        tmem_ld8(next, tmem_s + j + 8);
                    form_scores<kScore, kRows>(p, s, now, j, factor, buf, set, up, down, pos);
                    tmem_st8(tmem_s + j, now);
                };
#pragma unroll 1
                for (int j = 0; j < kOwn; j += 16) {
                    group(j, y[0], y[1]);
                    if (j + 8 < kOwn)
                        group(j + 8, y[1], y[0]);
                }
                tmem_wait_st();
            }
            const float mul = kScore ? 1.f : factor;
            const auto number = [&] { return fabsf(vs) <= FLT_MAX; };
            float vf = number() ? vs * f : 0.f;
            const auto size_of = [](float v) { // |v| < 2^size
                return fmaxf(static_cast<float>(static_cast<int>(__float_as_uint(v) >> 23 & 0xFFu) - 126), kLeastScale);
            };
            bool there = step == 0; // the last tile's product with V is done
            const bool span = sums && i > first && (i - first) / kTurns % kSpan == 0;
            float x[kOwn];
            // Once more after the references moved (which settles it; the limit is for no case known).
#pragma unroll 1
            for (int turn = 0;; ++turn) {
                if constexpr (kOwn == 8) {
                    tmem_ld8(x, tmem_s);
                    tmem_wait_ld8(x);
                } else {
#pragma unroll
                    for (int j = 0; j < kOwn; j += 16)
                        tmem_ld16(x + j, tmem_s + j);
#pragma unroll
                    for (int j = 0; j < kOwn; j += 16)
                        tmem_wait_ld16(x + j);
                }
                // For references so large that their rounding matters the scores are rounded
                // as they were, before the difference (a packed product and sum would be fused).
                if (kScore == 0 && large) {
#pragma unroll
                    for (int j = 0; j < kOwn; ++j)
                        x[j] = __fadd_rn(__fmul_rn(x[j], mul), neg_m[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < kOwn; j += 2)
                        fma2(f32x2(x[j], x[j + 1]), f32x2(mul, mul), f32x2(neg_m[j], neg_m[j + 1])).get(x[j], x[j + 1]);
                }
                if (fix) {
#pragma unroll
                    for (int j = 0; j < kOwn; ++j)
                        x[j] = seen(j) & 1u ? x[j] : -INFINITY;
                }
                float tops[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float *y = x + 8 * g;
                    tops[g] = fmaxf(max3(max3(y[0], y[1], y[2]), y[3], y[4]), max3(y[5], y[6], y[7]));
                }
                float top = tops[0];
#pragma unroll
                for (int g = 1; g < kGroups; ++g)
                    top = fmaxf(top, tops[g]);
                if (!stream_any(stream, ex2(top) * fmaxf(fabsf(vf), kLeastVf) > kMostTerm) || turn == 4)
                    break;
                // ---- references move in the groups that need it; F may too
                if (!there)
                    wait(&s.o_done[stream], (step - 1) & 1);
                there = true;
                tc_fence_after();
                constexpr uint32_t kNewUnit = 1u << 31;
                float size = size_of(vf);
                uint32_t over = f == 0.f || size > kMostScale ? kNewUnit : 0u;
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    over |= tops[g] + size > kTop + kRise ? 1u << g : 0u;
                over = __reduce_or_sync(0xFFFFFFFFu, over);
                if (lane == 0)
                    s.warp_over[stream][warp] = over;
                stream_sync(stream);
                const uint32_t *o4 = s.warp_over[stream];
                over = o4[0] | o4[1] | o4[2] | o4[3];
                int moved = 0;     // F's exponent
                bool with = false; // references and sums move along with it
                if (over & kNewUnit) {
                    over &= ~kNewUnit;
                    const float vs_size = number() ? fabsf(vs) : 0.f;
                    const int own = min(p.tile_tokens, seg.n - rg * p.tile_tokens) * p.g; // rows, may be negative
                    const uint64_t sees = static_cast<uint64_t>(sees_hi) << 32 | sees_lo;
                    const bool common = own <= 0 || ~sees << (64 - own) == 0; // all rows see this key
                    const float warp_common = warp_max(common ? vs_size : 0.f), warp_vs = warp_max(vs_size);
                    if (lane == 0)
                        s.warp_common[stream][warp] = warp_common, s.warp_vs[stream][warp] = warp_vs;
                    stream_sync(stream);
                    const auto largest = [](const float *v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); };
                    const float common_vs = largest(s.warp_common[stream]), all_vs = largest(s.warp_vs[stream]);
                    const int of_common = __float_as_uint(common_vs) >> 23; // exponents
                    const int of_all = __float_as_uint(all_vs) >> 23;
                    // At first F brings the largest that all rows see to [8, 16); or, where there is
                    // none, the largest of all to 2^50, as others' may be far smaller.
                    const int to = common_vs > 0.f ? 130 - of_common : all_vs > 0.f ? 177 - of_all : 40;
                    const int was = f == 0.f ? to : static_cast<int>(__float_as_uint(f) >> 23) - 127;
                    const int e = max(-126, min(min(was, 126), static_cast<int>(kMostScale) + 126 - of_all));
                    moved = f == 0.f ? 0 : e - was;
                    f = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                    vf = number() ? vs * f : 0.f;
                    size = size_of(vf);
                    if (moved != 0) {
                        // A smaller F changes references and sums along with it, and no term; unless
                        // sums are so large that they would overflow.
                        const float limit = ex2(static_cast<float>(120 + moved));
                        bool large_sum = false;
#pragma unroll
                        for (int j = 0; j < kOwn; ++j)
                            large_sum = large_sum || l[j] > limit;
                        with = !stream_any(stream, large_sum);
                    }
                }
#pragma unroll 1
                for (uint32_t rest = over; rest; rest &= rest - 1) {
                    const int j = 8 * (__ffs(rest) - 1);
                    float y[8];
                    tmem_ld8(y, tmem_s + j);
                    tmem_wait_ld8(y);
                    const uint32_t bits = seen(j);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // (rounded up: however large the score, no term is past its range)
                        const float mine = __fadd_ru(__fmul_rn(y[k], mul), size - kTop);
                        const float most = warp_max(bits >> k & 1u ? mine : -INFINITY);
                        if (lane == k)
                            warp_part[warp][j + k] = most;
                    }
                }
                stream_sync(stream);
                bool far = false;
                if (key_row < kOwn) {
                    const float last = -neg_m[key_row];
                    float m = with ? __fadd_ru(last, static_cast<float>(moved)) : last;
                    if (over >> (key_row >> 3) & 1u) {
                        const float most = fmaxf(fmaxf(warp_part[0][key_row], warp_part[1][key_row]),
                                                 fmaxf(warp_part[2][key_row], warp_part[3][key_row]));
                        // any rise, as the group is at it: fewer rows come back for another
                        m = most > m ? most : m;
                    }
                    const float fm = last == m ? 1.f : last == -INFINITY ? 0.f : ex2(last - m);
                    const float fv = ex2(static_cast<float>(moved));
                    neg_m[key_row] = -m;
                    far = fabsf(m) > 65536.f && m > -INFINITY;
                    f_l[key_row] = fm;
                    f_o[key_row] = fm * fv;
                    g_sums[key_row] *= fm * fv;
                }
                large = stream_any(stream, far);
#pragma unroll
                for (int j = 0; j < kOwn; ++j)
                    l[j] *= f_l[j];
                if (i > first) {
#pragma unroll 1
                    for (uint32_t rest = moved == 0 ? over : (1u << kGroups) - 1u; rest; rest &= rest - 1) {
                        const int j = 8 * (__ffs(rest) - 1);
                        float hi[8], lo[8];
                        tmem_ld8(hi, tmem_o + j);
                        tmem_ld8(lo, tmem_o + Sh::kLo + j);
                        tmem_wait_ld8(hi), tmem_wait_ld8(lo);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            hi[k] *= f_o[j + k], lo[k] *= f_o[j + k];
                        tmem_st8(tmem_o + j, hi);
                        tmem_st8(tmem_o + Sh::kLo + j, lo);
                    }
                    tmem_wait_st();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.s_read[stream]);
            if (!there)
                wait(&s.o_done[stream], (step - 1) & 1);
            tc_fence_after();
            // every span O moves out of the tensor core, to be added up to nearest
            if (span) {
#pragma unroll 1
                for (int j = 0; j < kOwn; j += 8) {
                    float hi[8], lo[8];
                    tmem_ld8(hi, tmem_o + j);
                    tmem_ld8(lo, tmem_o + Sh::kLo + j);
                    tmem_wait_ld8(hi), tmem_wait_ld8(lo);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float v = hi[k] + lo[k];
                        if (summed)
                            v = fmaf(sums[(j + k) * kHeadDim], g_sums[j + k], v);
                        sums[(j + k) * kHeadDim] = v;
                    }
                }
                summed = true;
                stream_sync(stream);
                if (key_row < kOwn)
                    g_sums[key_row] = 1.f;
                stream_sync(stream);
            }
            // ---- weights: their sum, and with the V scale as a pair into shared memory
            unsigned char *p_row = s.p16[stream] + (key_row >> 3) * (kOwn == 64 ? 2048 : 1024) + (key_row & 7) * 128;
            // lo's place: the other half of the key's row, or its second panel
            const int lo_by = kOwn == 64 ? 1024 : 0, lo_part = kOwn == 64 ? 0 : Sh::kLo / 8;
#pragma unroll
            for (int j = 0; j < kOwn; j += 8) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const f32x2 w(ex2(x[j + k]), ex2(x[j + k + 1]));
                    add2(f32x2(l[j + k], l[j + k + 1]), w).get(l[j + k], l[j + k + 1]);
                    split_f16(mul2(w, f32x2(vf, vf)), hi[k / 2], lo[k / 2]);
                }
                *reinterpret_cast<uint4 *>(p_row + (((j >> 3) ^ (key_row & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(p_row + lo_by + ((((j >> 3) + lo_part) ^ (key_row & 7)) << 4)) =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            // a V scale that is no number goes as it is to those who see it
            if (!number()) {
#pragma unroll 1
                for (int j = 0; j < kOwn; ++j)
                    if (seen(j) & 1u)
                        *reinterpret_cast<uint16_t *>(p_row + (((j >> 3) ^ (key_row & 7)) << 4) + 2 * (j & 7)) =
                            vs != vs ? 0x7FFFu : vs > 0.f ? 0x7C00u : 0xFC00u;
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.p_ready[stream]);
        }
        unit0 += tiles;

        // ---- the end of the segment: both streams' states joined, O written
#pragma unroll
        for (int j0 = 0; j0 < kOwn; j0 += 32) {
            constexpr int kAtOnce = kOwn < 32 ? kOwn : 32;
            const float sum = sum_lanes<kAtOnce>(l + j0);
            if (lane % (32 / kAtOnce) == 0)
                warp_part[warp][j0 + lane / (32 / kAtOnce)] = sum;
        }
        if (first < tiles)
            wait(&s.o_done[stream], (step - 1) & 1);
        tc_fence_after();
        if (summed) {
#pragma unroll 1
            for (int j = 0; j < kOwn; j += 8) {
                float hi[8];
                tmem_ld8(hi, tmem_o + j);
                tmem_wait_ld8(hi);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    hi[k] = fmaf(sums[(j + k) * kHeadDim], g_sums[j + k], hi[k]);
                tmem_st8(tmem_o + j, hi);
            }
            tmem_wait_st();
        }
        tc_fence_before();
        stream_sync(stream);
        if (key_row < kOwn) {
            s.l_end[stream][key_row] = (warp_part[0][key_row] + warp_part[1][key_row]) +
                                       (warp_part[2][key_row] + warp_part[3][key_row]);
            s.m_end[stream][key_row] = -neg_m[key_row];
            if (key_row == 0)
                s.inv_f[stream] = f == 0.f ? 0.f : 1.f / f;
        }
        both_streams_sync();
        tc_fence_after();
        const bool whole = seg.seg_tile0 == 0 && seg.seg_tile1 == seg.tiles;
        const int token0 = rg * p.tile_tokens;
        const int live_rows = min(p.tile_tokens, seg.n - token0) * p.g; // may be negative
        const int cta = blockIdx.x / ((p.row_groups + Sh::kSets - 1) / Sh::kSets);
        const size_t rec = static_cast<size_t>(2 * (cta * p.row_groups + rg) + (seg.seg_tile0 > 0 ? 0 : 1)) * p.rec_rows;
        if (key_row < kOwn) {
            // of a pair each stream has rows of its own, and no other has a share in them
            const float m0 = s.m_end[set][key_row], m1 = s.m_end[1][key_row];
            const float l0 = s.l_end[set][key_row], l1 = Sh::kPair ? 0.f : s.l_end[1][key_row];
            const float top = fmaxf(l0 == 0.f ? -INFINITY : m0, l1 == 0.f ? -INFINITY : m1);
            float w0 = l0 == 0.f ? 0.f : ex2(m0 - top), w1 = l1 == 0.f ? 0.f : ex2(m1 - top);
            const float sum = (l0 == 0.f ? 0.f : l0 * w0) + (l1 == 0.f ? 0.f : l1 * w1);
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            s.weight[stream][0][key_row] = w0 * inv * s.inv_f[set];
            s.weight[stream][1][key_row] = w1 * inv * s.inv_f[1];
            if (!whole && stream == set && key_row < live_rows) {
                p.rec_m[rec + key_row] = top;
                p.rec_l[rec + key_row] = sum;
            }
        }
        stream_sync(stream);
        // eight rows at a time, the streams in turn; a thread has a dim
#pragma unroll 1
        for (int j = Sh::kPair ? 0 : 8 * stream; j < min(kOwn, live_rows); j += 8 * kTurns) {
            const uint32_t o = s.tmem_base + lanes + set * kStreamColumns + kColO + j;
            float h0[8], g0[8], h1[8], g1[8];
            tmem_ld8(h0, o), tmem_ld8(g0, o + Sh::kLo);
            if constexpr (!Sh::kPair) {
                tmem_ld8(h1, o + kStreamColumns), tmem_ld8(g1, o + kStreamColumns + Sh::kLo);
                tmem_wait_ld8(h1), tmem_wait_ld8(g1);
            }
            tmem_wait_ld8(h0), tmem_wait_ld8(g0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int row = j + k;
                if (row >= live_rows)
                    break;
                const float w0 = s.weight[stream][0][row], w1 = s.weight[stream][1][row];
                // a stream without a visible key may hold anything
                float v = w0 == 0.f ? 0.f : (h0[k] + g0[k]) * w0;
                if constexpr (!Sh::kPair)
                    v = w1 == 0.f ? v : fmaf(h1[k] + g1[k], w1, v);
                if (!whole) {
                    p.rec_acc[(rec + row) * kHeadDim + key_row] = v;
                } else {
                    const size_t at = ((static_cast<size_t>(seg.b) * p.M + token0 + row / p.g) * p.Hq + seg.h * p.g +
                                       row % p.g) * kHeadDim + key_row;
                    if (p.out_f32)
                        p.out_f32[at] = v;
                    if (p.out_bf16)
                        p.out_bf16[at] = f32_to_bf16_bits(v);
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&s.rows_empty[buf]);
        // neither stream's O or state may be overwritten before both have it
        tc_fence_before();
        both_streams_sync();
        tc_fence_after();
    }
    return ok;
}

template <int kScore, int kRows>
__global__ void __launch_bounds__(Shape<kRows>::kThreads, 1)
    tree_int8_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                     const __grid_constant__ TreeInt8Params p)
{
    using Sh = Shape<kRows>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    TreeInt8Smem<kRows> &s = *reinterpret_cast<TreeInt8Smem<kRows> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // one CTA for a row group or a pair of them (the second of the last pair may not exist)
    const int groups = (p.row_groups + Sh::kSets - 1) / Sh::kSets;
    const int rg = blockIdx.x % groups * Sh::kSets, cta = blockIdx.x / groups;
    if (tid == 0) {
        prefetch_tensormap(&mk), prefetch_tensormap(&mv);
        for (int i = 0; i < Sh::kRing + Sh::kRingV; ++i)
            mbar_init(&s.code_full[i], 1), mbar_init(&s.code_empty[i], 4);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&s.rows_full[w], 1), mbar_init(&s.rows_empty[w], 8);
            mbar_init(&s.k_ready[w], 4), mbar_init(&s.v_ready[w], 4); // a warp each
            mbar_init(&s.k_free[w], 2), mbar_init(&s.v_free[w], 2);
            mbar_init(&s.s_read[w], 4), mbar_init(&s.p_ready[w], 4);
            mbar_init(&s.s_full[w], 1), mbar_init(&s.o_done[w], 1), mbar_init(&s.drain[w], 1);
        }
        for (int i = 0; i < Sh::kQueries; ++i)
            mbar_init(&s.q_full[i], 1), mbar_init(&s.q_empty[i], 2);
        fence_mbar_init();
    }
    if (warp == Sh::kCodeWarp)
        tmem_alloc_all(&s.tmem_base);
    // columns of P that no row fills stay zero
    for (int i = tid; i < static_cast<int>(sizeof(s.p16) / 16); i += Sh::kThreads)
        reinterpret_cast<uint4 *>(&s.p16[0][0])[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();

    // Everything read from here on may come from the kernel before this one, and
    // the next kernel may start once that one is done.
    grid_dependency_wait();
    allow_dependent_launch();
    plan_run<Sh::kThreads>(p, s, cta);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    bool ok = true;
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kLeast));
        if (s.units > 0) {
            if (warp < 12)
                ok = widen<kRows, true, !Sh::kApart>(p, s);
            else if (Sh::kApart && warp < 16)
                ok = widen<kRows, false, true>(p, s);
            else if (warp == Sh::kCodeWarp)
                ok = fetch_codes(p, s, &mk, &mv);
            else if (warp == Sh::kQueryWarp)
                ok = fetch_rows<kScore>(p, s, rg);
            else
                ok = multiply(p, s, warp - Sh::kMmaWarp);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::kMost));
        if (s.units > 0)
            ok = soften<kScore>(p, s, Sh::kPair ? rg + (warp >> 2) : rg, warp >> 2);
    }
    if (!ok && lane == 0)
        atomicOr(&g_flags_tree_int8, PGQA_DEVERR_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Sh::kCodeWarp)
        tmem_free_all(s.tmem_base);
}

// How a call's rows and CTAs are laid out; from sizes alone, so that the
// workspace query and the launch agree.
struct Layout {
    int rows, tile_tokens, row_groups, cta_groups, rec_rows, ctas;
    size_t base_bytes, stat_bytes, acc_bytes, sum_bytes;
};

size_t align256(size_t x) { return (x + 255) & ~size_t{255}; }

Layout layout(int B, int M, int Hq, int Hkv, int page_size, int max_pages, int sm_count)
{
    Layout y{};
    const int g = Hq / Hkv;
    const int most = kMaxRows / g; // tokens of a row group
    y.row_groups = (M + most - 1) / most;
    y.tile_tokens = (M + y.row_groups - 1) / y.row_groups;
    y.row_groups = (M + y.tile_tokens - 1) / y.tile_tokens;
    y.rec_rows = y.tile_tokens * g;
    y.rows = y.rec_rows <= 8 ? 8 : y.rec_rows <= 16 ? 16 : y.rec_rows <= 32 ? 32 : 64;
    const long long tiles = (static_cast<long long>(max_pages) * page_size + kTileKeys - 1) / kTileKeys;
    const long long units = tiles * B * Hkv;
    if (y.row_groups > 1)
        y.rows = 128;
    y.cta_groups = y.rows == 128 ? (y.row_groups + 1) / 2 : 1;
    const int ctas = sm_count / y.cta_groups;
    y.ctas = static_cast<int>(units < ctas ? units : ctas);
    if (y.ctas < 1)
        y.ctas = 1;
    const size_t records = static_cast<size_t>(2) * y.ctas * y.row_groups;
    y.base_bytes = align256((static_cast<size_t>(B) + 1) * sizeof(int32_t));
    y.stat_bytes = align256(records * y.rec_rows * sizeof(float));
    y.acc_bytes = align256(records * y.rec_rows * kHeadDim * sizeof(float));
    // a stream passes a span only where a (sequence, head) has that many tiles
    y.sum_bytes = tiles > kSpan ? records * (y.rows < kMaxRows ? y.rows : kMaxRows) * kHeadDim * sizeof(float) : 0;
    return y;
}

CUresult encode_codes(EncodeTiledFn fn, CUtensorMap *map, const void *base, long long rows, int page_size)
{
    const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {kHeadDim};
    const cuuint32_t box[2] = {kHeadDim, static_cast<cuuint32_t>(page_size < kTileKeys ? page_size : kTileKeys)};
    const cuuint32_t elem[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

constexpr int kMaxDevices = 64;

template <int kScore, int kRows>
cudaError_t launch_rows(const CUtensorMap &mk, const CUtensorMap &mv, const TreeInt8Params &p, cudaStream_t stream)
{
    static std::atomic<bool> configured[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const auto kernel = tree_int8_kernel<kScore, kRows>;
    if (dev >= kMaxDevices || !configured[dev].load(std::memory_order_acquire)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kInt8Smem<kRows>);
        if (err != cudaSuccess)
            return err;
        if (dev < kMaxDevices)
            configured[dev].store(true, std::memory_order_release);
    }
    const int groups = (p.row_groups + Shape<kRows>::kSets - 1) / Shape<kRows>::kSets; // that have CTAs of their own
    return launch_pdl(kernel, dim3(static_cast<unsigned>(p.ctas * groups)), dim3(Shape<kRows>::kThreads), kInt8Smem<kRows>,
                      stream, mk, mv, p);
}

template <int kScore>
cudaError_t launch_score(int rows, const CUtensorMap &mk, const CUtensorMap &mv, const TreeInt8Params &p, cudaStream_t stream)
{
    switch (rows) {
    case 8: return launch_rows<kScore, 8>(mk, mv, p, stream);
    case 16: return launch_rows<kScore, 16>(mk, mv, p, stream);
    case 32: return launch_rows<kScore, 32>(mk, mv, p, stream);
    case 64: return launch_rows<kScore, 64>(mk, mv, p, stream);
    default: return launch_rows<kScore, 128>(mk, mv, p, stream);
    }
}

} // namespace

size_t tree_attn_int8_workspace_bytes(int B, int M, int Hq, int Hkv, int page_size, int max_pages, int sm_count)
{
    if (B == 0)
        return 0;
    const Layout y = layout(B, M, Hq, Hkv, page_size, max_pages, sm_count);
    return y.base_bytes + 2 * y.stat_bytes + y.acc_bytes + y.sum_bytes;
}

cudaError_t launch_tree_attn_int8(const TreeAttnInt8Args &a, cudaStream_t stream)
{
    const EncodeTiledFn fn = tensor_map_encoder();
    if (!fn)
        return cudaErrorNotSupported;
    const Layout y = layout(a.B, a.M, a.Hq, a.Hkv, a.page_size, a.max_pages, a.sm_count);
    TreeInt8Params p{};
    p.q = a.q;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.block_table = a.block_table;
    p.context_lens = a.context_lens;
    p.tree_mask = a.tree_mask;
    p.positions = a.positions;
    p.draft_lens = a.draft_lens;
    p.slopes = a.slopes;
    p.B = a.B;
    p.M = a.M;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.log2_page = __builtin_ctz(static_cast<unsigned>(a.page_size));
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.g = a.Hq / a.Hkv;
    p.tile_tokens = y.tile_tokens;
    p.row_groups = y.row_groups;
    p.rec_rows = y.rec_rows;
    p.ctas = y.ctas;
    p.c = std::fmin(std::fmax(a.scale * kLog2e, -FLT_MAX), FLT_MAX);
    if (a.softcap > 0.f) {
        const float cap = std::fmin(a.softcap, 1e30f); // no cap to any score, and its products stay finite
        p.cap_u = std::fmin(std::fmax(a.scale / cap, -FLT_MAX), FLT_MAX);
        p.cap_out = cap * kLog2e;
        for (int k = 0; k < kTanhTerms; ++k)
            p.tanh_c[k] = static_cast<float>(kTanh[k] * cap * 1.4426950408889634);
    } else {
        p.cap_u = p.c;
    }
    p.out_f32 = a.out_f32;
    p.out_bf16 = a.out_bf16;
    unsigned char *ws = static_cast<unsigned char *>(a.ws);
    p.unit_base = reinterpret_cast<int32_t *>(ws);
    p.rec_m = reinterpret_cast<float *>(ws + y.base_bytes);
    p.rec_l = reinterpret_cast<float *>(ws + y.base_bytes + y.stat_bytes);
    p.rec_acc = reinterpret_cast<float *>(ws + y.base_bytes + 2 * y.stat_bytes);
    if (a.out_f32 && y.sum_bytes)
        p.sums = reinterpret_cast<float *>(ws + y.base_bytes + 2 * y.stat_bytes + y.acc_bytes);
    CUtensorMap mk, mv;
    const long long rows = static_cast<long long>(a.num_pages) * a.Hkv * a.page_size;
    if (encode_codes(fn, &mk, a.k_cache8, rows, a.page_size) != CUDA_SUCCESS ||
        encode_codes(fn, &mv, a.v_cache8, rows, a.page_size) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cudaError_t err;
    switch ((a.softcap > 0.f ? 1 : 0) | (a.slopes ? 2 : 0)) {
    case 0: err = launch_score<0>(y.rows, mk, mv, p, stream); break;
    case 1: err = launch_score<1>(y.rows, mk, mv, p, stream); break;
    case 2: err = launch_score<2>(y.rows, mk, mv, p, stream); break;
    default: err = launch_score<3>(y.rows, mk, mv, p, stream); break;
    }
    if (err != cudaSuccess)
        return err;
    return launch_tree_merge(p, y.ctas, stream);
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
