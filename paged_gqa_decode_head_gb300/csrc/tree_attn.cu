// tree_attn.cu -- decode_attn_paged_tree: attention of a tree of drafted
// tokens over the paged cache, with an optional tanh cap and distance bias.
//
// Mathematics. For the R = M * g query rows (drafted token, head) that share a
// KV head: x = scale Q K^T, capped and biased; softmax over the keys that the
// row sees (the prefix, and the drafted tokens of its mask); O = P V. Computed
// over tiles of 128 keys with a running reference m and sum l per row (the online
// normaliser of Milakov and Gimelshein, 2018, in base 2): p = 2^(y - m), l += p, O
// += p V. m need not be the maximum: only when a row's scores rise more than 8 above
// it does it move up, and l and O are scaled (2^8 is far inside fp32's range, so
// most tiles need no rescale).
//
// Bound. The cache is read once: 512 bytes per (key, KV head) against 4 * 128 * R
// flops. Up to R of about 200 the memory bounds it, above that the tensor cores.
// mma.sync cannot follow the memory from R = 32 on; tcgen05 with M = 128 rows can,
// even with rows to spare.
//
// Work split. The tiles of all sequences and KV heads are numbered in one row
// (sequence, head, tile) and each CTA takes an equal run of them, whatever the
// lengths: no partition size, no waves, ragged batches balance by themselves.
// A run that covers a (sequence, head) from its first to its last tile writes
// the output; the pieces of the others go to the workspace (at most two per
// CTA) and tree_merge_kernel joins them, in order, in the same stream.
//
// CTA: one per SM, 12 warps around a ring of five 32 KB shared-memory slots
// (K and V tiles in consumption order), Q, and all of tensor memory (S/P of
// two streams, O of two streams, 128 columns each):
//   warp 8   requests Q, K and V tiles by TMA, one lane per page of a tile;
//   warps 9 and 10  issue the tcgen05 products of one stream each: S = Q K^T
//            (both operands from shared memory), O += P V (P from tensor memory);
//   warps 0-3 and 4-7  one softmax warpgroup per stream: a thread owns a row,
//            reads its 128 scores from tensor memory and writes P over them.
// Two streams keep the tensor core and the softmax busy at once. With up to
// 128 rows the streams take alternate key tiles of the same rows and are joined
// at the end of a run; with more, they are two row tiles over the same keys.
//
// A stream's step: S from the tensor core, 128 scores of a row in a thread's
// registers (2000 clocks for a full tile, some 1100 instructions a warp), P in
// two halves, the first handed over while the second is formed, then O += P V
// and the next S in one go. The streams' products alternate (a stream's next
// scores before the other's products with V). The tensor core's queue is a few
// products deep, so every gap in issuing shows: operands are waited for ahead,
// and each stream has an issuing warp of its own.
//
// Rounding: P enters its product as a bf16 pair hi + lo (17 significant bits, so
// that fp32 outputs keep their meaning: 1.3e-6 from the formula, 2-norm), which
// is half as much tensor work again; S, O, m and l are fp32.
//
// Measured (GB300; bf16 outputs; HBM at the measured copy bandwidth of 6.78 TB/s):
//   B = 64, ragged to 32768, 16 drafted, g = 2 (3.9 GB): 614 us, 6.4 TB/s of K and V (95 %);
//   B = 1, T = 131072, 16 drafted, g = 4, capped: 113 to 120 us, 4.5 to 4.7 TB/s (the
//     cap's polynomial, and the run's start and end);
//   B = 8, T = 16384, 64 drafted, g = 8: 279 us, 986 TFLOP/s and half as much again
//     for lo, under the power limit (4000 clocks for two steps, whose 48 products
//     take 64 each);
//   B = 1, T = 8192, g = 2: 16 drafted 20.8 us, 64 drafted 24.8 us (the lengths, the
//     table and the first tile are three trips to memory before the first product;
//     joining the pieces is a second kernel);
//   B = 33, ragged to 4001, one token, g = 3, capped and biased: 119 to 129 us, 2.1 to
//     2.3 TB/s (one warp of each stream holds all rows, both on the same SM partition).
// Chains of M * g <= 8 rows without cap and bias are faster in decode_attn_paged_multi
// (T = 8192, g = 2, 1 and 4 tokens: 8.7 and 10.0 us, here 19.6 and 20.3; B = 64, ragged to
// 32768, 4 tokens: 634 and 721 us).
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

__device__ unsigned g_flags_tree;

constexpr int kTileRows = 128;
constexpr int kTileBytes = kTileKeys * kRowBytes; // 32 KB of K or V
constexpr int kSlots = 5;
constexpr int kValidRing = 8;      // units whose page masks are kept (the ring holds at most 4 ahead)
constexpr int kSoftmaxThreads = 256;
constexpr int kTreeThreads = 384; // three warpgroups (the last warp idles)
constexpr int kProducerWarp = 8, kMmaWarp = 9; // and kMmaWarp + 1
constexpr float kRescaleLog2 = 8.f; // rise of a row's scores that moves its reference
constexpr int kSpan = 16; // a stream's tiles between two moves of O out of the tensor core (fp32 outputs)

// TMEM columns of stream s's S (fp32, 128 columns, P over it) and O, + 128 s.
constexpr uint32_t kColS = 0, kColO = 256;

struct TreeParams {
    // for tree_merge_kernel: row tiles of a record, rows of a row tile
    static constexpr int kTilesPerRecord = 2, kRowsPerTile = kTileRows;
    static __device__ void raise(unsigned flag) { atomicOr(&g_flags_tree, flag); }
    const uint16_t *v;
    const int32_t *block_table, *context_lens;
    const uint64_t *tree_mask;
    const int32_t *positions, *draft_lens;
    const float *slopes;
    int B, M, Hq, Hkv, log2_page, max_pages, num_pages;
    int g;             // query heads per KV head
    int tile_tokens;   // drafted tokens per row tile (g * tile_tokens <= 128 rows)
    int row_tiles;     // ceil(M / tile_tokens)
    int row_groups;    // CTAs that share a run of tiles: one per pair of row tiles
    int rec_rows;      // rows of a partial record
    int ctas;          // grid size / row_groups
    float c;           // plain scores: y = |scale| log2 e * x (the sign is in the MMA descriptor)
    float cap_u, cap_out;  // capped: y = cap_out tanh(cap_u x)
    float tanh_c[7];       // cap_out times the polynomial's coefficients
    uint32_t negate_q;     // scale < 0
    float *out_f32;
    uint16_t *out_bf16;
    int32_t *unit_base;     // [B + 1] first tile number of each sequence, total
    float *rec_m, *rec_l;   // [2 * grid][rec_rows]
    float *rec_acc;         // [2 * grid][rec_rows][128]
    float *sums;            // [2 * grid][128][sum_rows]: O of earlier spans; null: bf16 outputs only
    int sum_rows;           // rows of a row tile, to whole warps
};

struct __align__(1024) TreeSmem {
    unsigned char slots[kSlots][kTileBytes];
    unsigned char q[2][kTileRows * kRowBytes];
    // barriers
    // a slot's loads complete on the barrier of the stream that reads them (the
    // first one's where both do), so that each stream sees every phase it waits for
    uint64_t full[2][kSlots], empty[kSlots];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_half[2], p_ready[2];
    uint64_t round_done[2]; // a stream's products of a step, and its next scores, are issued
    uint64_t seg_done, ml_ready, epi_done, drain[2];
    // drafted tokens of a stream's tiles of a segment whose V row is not finite
    // (with two row tiles a stream may be two segments ahead of the other's readers)
    uint64_t bad_rows[4][2];
    uint32_t valid[kValidRing]; // pages inside the pool, a bit per 16 keys of a tile
    uint32_t tmem_base;
    int start_b, start_h, start_tile, start_T, start_n, units; // this CTA's run
    int scan[kTreeThreads / 32];
    float zero;
    float2 ml[2][kTileRows]; // (m, l) of both streams
};
constexpr int kTreeSmem = sizeof(TreeSmem);
static_assert(kTreeSmem <= 232448, "one CTA's shared memory");

// The steps of one stream in a CTA's run. A step is a (tile, stream); with one
// row tile the streams take alternate tiles of the whole run, with two (pair)
// each takes every tile.
struct Steps {
    Segments seg;
    int stream, index; // segments begun before this one
    int begin, end;    // the segment's steps, of either stream
    int n;             // the current step
    bool pair, any;
    __device__ Steps(const TreeParams &p, const TreeSmem &s, int stream, bool pair)
        : seg(s), stream(stream), index(-1), begin(0), end(0), n(0), pair(pair), any(true)
    {
        advance(p);
    }
    __device__ __forceinline__ void advance(const TreeParams &p)
    {
        n += 2;
        if (n >= end)
            enter(p);
    }
    __device__ __forceinline__ void enter(const TreeParams &p)
    {
        while (any && n >= end) {
            any = seg.next(p);
            if (!any)
                break;
            ++index;
            begin = end;
            end = begin + (seg.seg_tile1 - seg.seg_tile0) * (pair ? 2 : 1);
            n = begin + ((begin ^ stream) & 1);
        }
    }
    __device__ int tile() const { return seg.seg_tile0 + ((n - begin) >> (pair ? 1 : 0)); }
    __device__ bool first() const { return n < begin + 2; }
    __device__ bool last() const { return n + 2 >= end; }
    // the segment has a single step: its stream signals for the other one too
    __device__ bool alone() const { return end - begin == 1; }
};

// ---------------------------------------------------------------- producer
__device__ bool produce(const TreeParams &p, TreeSmem &s, const CUtensorMap *mq, const CUtensorMap *mk,
                        const CUtensorMap *mv, int rg, bool pair)
{
    const int lane = threadIdx.x & 31;
    const int P = 1 << p.log2_page;
    const int box_keys = min(P, kTileKeys);
    const int boxes = kTileKeys / box_keys; // pages of a tile
    const int outside = static_cast<int>((static_cast<long long>(p.num_pages) * p.Hkv << p.log2_page) >> 3);
    // one row group reads K and V once; of several, running side by side, the
    // first leaves them in L2 for the others
    const uint64_t policy = p.row_groups == 1 ? l2_evict_first_policy() : l2_evict_normal_policy();
    int put = 0;
    uint32_t issued = 0, phases = 0; // per barrier (stream, slot): used, parity of its last load
    bool ok = true;
    const auto load_tile = [&](const CUtensorMap *map, int group, int reader) {
        const int slot = put % kSlots;
        ok = ok && warp_wait(&s.empty[slot], ((put / kSlots) & 1) ^ 1);
        if (!ok)
            return;
        uint64_t *full = &s.full[reader][slot];
        if (lane == 0)
            mbar_arrive_expect_tx(full, kTileBytes);
        __syncwarp();
        if (lane < boxes)
            tma_load_4d(s.slots[slot] + lane * box_keys * kRowBytes, map, 0, 0, 0, group, full, policy);
        const uint32_t bit = 1u << (reader * kSlots + slot);
        phases = issued & bit ? phases ^ bit : phases;
        issued |= bit;
        ++put;
    };
    const int ahead = pair ? 1 : 2; // tiles of K requested before the V of the first of them
    int group1 = 0, group2 = 0;     // this lane's page of the last tile and of the one before
    Segments seg(s);
    int unit = 0;
    for (int index = 0; ok && seg.next(p); ++index) {
        const int32_t *table = p.block_table + static_cast<size_t>(seg.b) * p.max_pages;
        const auto entry = [&](int tile) {
            const int key = tile * kTileKeys + lane * box_keys;
            return lane < boxes && key < seg.T ? table[key >> p.log2_page] : 0;
        };
        int phys_next = entry(seg.seg_tile0);
        for (int tile = seg.seg_tile0; ok && tile < seg.seg_tile1; ++tile, ++unit) {
            const int phys = phys_next;
            if (tile + 1 < seg.seg_tile1)
                phys_next = entry(tile + 1);
            const int key = tile * kTileKeys + lane * box_keys;
            const bool needed = lane < boxes && key < seg.T;
            const bool in_pool = phys >= 0 && phys < p.num_pages;
            const int group = needed && in_pool
                                  ? static_cast<int>((((static_cast<long long>(phys) * p.Hkv + seg.h) << p.log2_page) +
                                                      (key & (P - 1))) >>
                                                     3)
                                  : outside; // a box outside the tensor arrives as zeros
            if (needed && !in_pool)
                atomicOr(&g_flags_tree, PGQA_DEVERR_BAD_PAGE);
            uint32_t valid = __ballot_sync(0xFFFFFFFFu, !needed || in_pool);
            if (unit >= ahead)
                load_tile(mv, pair ? group1 : group2, pair ? 0 : unit & 1);
            if (tile == seg.seg_tile0 && ok) {
                // Q: one buffer per segment in turn, or both for two row tiles
                const int buf = pair ? 0 : index & 1;
                ok = warp_wait(&s.q_empty[buf], ((pair ? index : index >> 1) & 1) ^ 1);
                if (ok && lane == 0) {
                    const int bytes = p.tile_tokens * p.g * 128; // one 64-column half of a row tile
                    mbar_arrive_expect_tx(&s.q_full[buf], (pair ? 4 : 2) * bytes);
                    for (int i = 0; i < (pair ? 2 : 1); ++i)
                        for (int half = 0; half < 2; ++half)
                            tma_load_3d_default(s.q[buf + i] + half * (kTileRows * 128), mq, 64 * half, seg.h * p.g,
                                                seg.b * p.M + (2 * rg + i) * p.tile_tokens, &s.q_full[buf]);
                }
            }
            if (lane == 0) {
                uint32_t by16 = 0; // a bit per 16 keys
                for (int i = 0; i < 8; ++i)
                    by16 |= ((valid >> (i * 16 / box_keys)) & 1u) << i;
                s.valid[unit % kValidRing] = by16;
            }
            load_tile(mk, group, pair ? 0 : unit & 1);
            group2 = group1;
            group1 = group;
        }
    }
    if (ok && !pair && unit > 1)
        load_tile(mv, group2, unit & 1);
    if (ok && unit > 0)
        load_tile(mv, group1, pair ? 0 : (unit - 1) & 1);
    // nothing may still be on its way into shared memory when the CTA ends
    for (int i = 0; i < 2 * kSlots; ++i)
        if (issued >> i & 1u)
            ok = warp_wait(&s.full[i / kSlots][i % kSlots], phases >> i & 1u) && ok;
    return ok;
}

// ---------------------------------------------------------------- matrix products
// Before a V tile that holds the end of the sequence or drafted tokens enters
// a product: rows past T become zeros (their weights are zeros, and 0 * NaN is
// not), and elements of drafted tokens that are not finite become zeros and are
// noted, so that they reach only the rows that see them (at the end).
__device__ uint64_t settle_v_tile(unsigned char *v, int key0, int T, int n, int box_keys)
{
    const int lane = threadIdx.x & 31;
    const int sub = lane >> 4, part = lane & 15; // two rows at a time, 16 bytes per lane
    const auto at = [&](int row) { // the row's eighth-of-a-half `part` (order within the row does not matter)
        return v + (row >> 3) * 2048 + (part >> 3) * 1024 + (row & 7) * 128 + (part & 7) * 16;
    };
    uint64_t bad = 0;
    const int end = T - key0;                                     // rows that exist
    const int loaded = min(kTileKeys, (end + box_keys - 1) / box_keys * box_keys);
    const int first = max(0, end - n);
    for (int row = first + sub; row < min(end, kTileKeys); row += 2) {
        uint4 *x = reinterpret_cast<uint4 *>(at(row));
        uint32_t w[4] = {x->x, x->y, x->z, x->w};
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7F80u) == 0x7F80u)
                w[i] &= 0xFFFF0000u, any = true;
            if ((w[i] & 0x7F800000u) == 0x7F800000u)
                w[i] &= 0x0000FFFFu, any = true;
        }
        if (any) {
            *x = make_uint4(w[0], w[1], w[2], w[3]);
            bad |= 1ull << (row - (end - n));
        }
    }
    for (int row = end + sub; row < loaded; row += 2)
        *reinterpret_cast<uint4 *>(at(row)) = make_uint4(0, 0, 0, 0);
    const uint32_t lo = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(bad));
    const uint32_t hi = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(bad >> 32));
    fence_proxy_async_smem();
    __syncwarp();
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// One warp per stream, so that one's waits lie under the other's products.
__device__ bool multiply(const TreeParams &p, TreeSmem &s, bool pair, int stream)
{
    const int N = s.units; // tiles
    const bool leader = elect_one(); // issues every product and commit
    const uint32_t tmem_s = warp_uniform(s.tmem_base + kColS + stream * 128);
    const uint32_t idesc_s = tc_idesc_bf16(kTileKeys, p.negate_q != 0, false);
    const uint32_t idesc_o = tc_idesc_bf16(kHeadDim, false, true);
    const int box_keys = min(1 << p.log2_page, kTileKeys);
    uint64_t bad = 0;
    uint64_t *full = s.full[pair ? 0 : stream];
    uint32_t phases = 0; // of `full`, a bit per slot
    bool ok = true;
    // Order of the tiles in the ring. Two row tiles (pair): K0 V0 K1 V1 ...; one
    // row tile, whose scores run two tiles ahead of its products with V: K0 K1
    // V0 K2 V1 K3 ... K(N-1) V(N-2) V(N-1).
    int k_slot = pair ? 0 : stream, v_slot = pair ? 1 : 2 + 2 * stream;
    const auto move_on = [&](int &slot, int tiles) {
        slot += tiles;
        slot -= slot >= kSlots ? kSlots : 0;
    };
    const auto landed = [&](int slot) {
        const bool yes = warp_wait(&full[slot], phases >> slot & 1u);
        phases ^= 1u << slot;
        return yes;
    };

    Steps su(p, s, stream, pair), pu(p, s, stream, pair); // of the next score product and of the next product with V
    // Every operand of a round is waited for before its first product where
    // possible, so that the products follow each other without a gap.
    bool k_there = false;
    const auto wait_for_scores = [&] {
        // K first: once it is there, the buffer's earlier Q was there too (a
        // stream may have had no step in that segment), and the parity of
        // q_full means this segment's Q
        ok = ok && landed(k_slot);
        if (su.first())
            ok = ok && warp_wait(&s.q_full[pair ? 0 : su.index & 1], (pair ? su.index : su.index >> 1) & 1);
        k_there = true;
    };
    // the first round issues only the first scores
    for (bool started = false; ok && (pu.any || !started); started = true) {
        if (started) { // O += P V; P lies in S's place, for each 16 keys 8 columns hi and 8 lo
            const int n = pu.n;
            int slot = v_slot;
            if (!pair && n == N - 1) // the last tile has no K between V and the V before
                move_on(slot, kSlots - 1);
            move_on(v_slot, pair ? 2 : 4);
            unsigned char *v = s.slots[slot];
            ok = landed(slot);
            if (!ok)
                break;
            if (pu.first())
                bad = 0;
            const int key0 = pu.tile() * kTileKeys;
            if (key0 + kTileKeys > pu.seg.T - pu.seg.n) // of two streams on one tile both do this: the same zeros
                bad |= settle_v_tile(v, key0, pu.seg.T, pu.seg.n, box_keys);
            if (su.any && !su.first())
                wait_for_scores();
            // The streams' products alternate: a stream's next scores go before
            // the other's products with V, so that its softmax can start.
            if (n > 0)
                ok = ok && warp_wait(&s.round_done[stream ^ 1], ((n - 1) >> 1) & 1);
            const uint32_t va = warp_uniform(tc_desc_low(smem_addr(v), 1024));
            // a segment's first product, and a span's, overwrites O
            const uint32_t keep = warp_uniform(!pu.first() && !(p.sums && ((n - pu.begin) >> 1) % kSpan == 0));
#pragma unroll
            for (int half = 0; half < 2; ++half) { // 64 keys each
                ok = ok && warp_wait(half == 0 ? &s.p_half[stream] : &s.p_ready[stream], (n >> 1) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) // 16 keys: hi, then lo
                        tc_mma_ts(tmem_s + (kColO - kColS), tmem_s + half * 64 + k * 8,
                                  va + (half * 4 + (k >> 1)) * (4096 / 16), tc_desc_high(2048), idesc_o,
                                  half > 0 || k > 0 ? 1u : keep);
                }
            }
            if (!ok)
                break;
            if (leader) {
                tc_commit(&s.empty[slot]);
                if (pu.last()) {
                    s.bad_rows[pu.index & 3][stream] = bad;
                    tc_commit(&s.seg_done);
                    if (pu.alone()) {
                        s.bad_rows[pu.index & 3][stream ^ 1] = 0;
                        tc_commit(&s.seg_done);
                        mbar_arrive(&s.seg_done);
                    }
                    mbar_arrive(&s.seg_done); // orders bad_rows before its readers
                }
            }
        }
        if (su.any) { // S = Q K^T over the place of the P that was just used
            if (!k_there)
                wait_for_scores();
            k_there = false;
            if (!ok)
                break;
            tc_fence_after();
            const int slot = k_slot;
            const int buf = pair ? 0 : su.index & 1;
            const uint32_t qa = warp_uniform(tc_desc_low(smem_addr(s.q[pair ? stream : buf]), 16));
            const uint32_t ka = warp_uniform(tc_desc_low(smem_addr(s.slots[slot]), 16));
            if (leader) {
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k) {
                    const int half = k >> 2, off = (k & 3) * 2; // 64 columns each; 32 bytes a step
                    tc_mma_ss(tmem_s, qa + half * (kTileRows * 128 / 16) + off, tc_desc_high(1024),
                              ka + half * (1024 / 16) + off, tc_desc_high(2048), idesc_s, k > 0);
                }
                tc_commit(&s.s_full[stream]);
                mbar_arrive(&s.s_full[stream]); // orders the page mask's write before its readers
                if (started)
                    mbar_arrive(&s.round_done[stream]);
                tc_commit(&s.empty[slot]);
                if (su.last()) {
                    tc_commit(&s.q_empty[buf]);
                    if (su.alone())
                        tc_commit(&s.q_empty[buf]);
                }
            }
            __syncwarp();
            move_on(k_slot, pair ? 2 : (su.n == 0 ? 3 : 4));
            su.advance(p);
        } else if (started && leader) {
            mbar_arrive(&s.round_done[stream]);
        }
        __syncwarp();
        if (started)
            pu.advance(p);
    }
    // no product may still be running when the CTA ends
    if (leader)
        tc_commit(&s.drain[stream]);
    return warp_wait(&s.drain[stream], 0) && ok;
}

// ---------------------------------------------------------------- softmax
// Bits of the 32 keys of which the first `below` lie in the prefix (any
// integer; drafted token j is key below + j) that a row sees: the prefix, the
// drafted tokens of its mask, without pages outside the pool (two bits of
// `valid`, 16 keys each).
__device__ __forceinline__ uint32_t visible_word(int below, uint64_t mask, uint32_t valid)
{
    uint32_t bits = below >= 32 ? 0xFFFFFFFFu : (below > 0 ? (1u << below) - 1u : 0u);
    if (below < 32)
        bits |= static_cast<uint32_t>(below >= 0 ? mask << below : (below > -64 ? mask >> -below : 0ull));
    return bits & (((valid & 1u) ? 0xFFFFu : 0u) | ((valid & 2u) ? 0xFFFF0000u : 0u));
}

// N scores of a row, capped (kScore bit 0) or scaled, in base 2, with the bias
// (bit 1) of keys whose positions are their slots; far0: the first one's
// distance. Returns the largest u^2: above 1 the capped ones are not valid.
template <int kScore, int N>
__device__ __forceinline__ float prepare_scores(const TreeParams &p, float *x, float slope, float far0)
{
    float over = 0.f;
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        f32x2 y(x[j], x[j + 1]);
        if constexpr ((kScore & 1) != 0) {
            const f32x2 u = mul2(y, f32x2(p.cap_u, p.cap_u)), t = mul2(u, u);
            float t0, t1;
            t.get(t0, t1);
            over = max3(over, t0, t1);
            y = f32x2(p.tanh_c[kTanhTerms - 1], p.tanh_c[kTanhTerms - 1]);
#pragma unroll
            for (int k = kTanhTerms - 2; k >= 0; --k)
                y = fma2(y, t, f32x2(p.tanh_c[k], p.tanh_c[k]));
            y = mul2(u, y);
        } else {
            y = mul2(y, f32x2(p.c, p.c));
        }
        if constexpr ((kScore & 2) != 0)
            y = fma2(f32x2(slope, slope), add2(f32x2(far0, far0), f32x2(j, j + 1)), y);
        y.get(x[j], x[j + 1]);
    }
    return over;
}

// 16 scores of any size from key `key` on, any of them drafted tokens, whose
// positions are their own (pos_lo and pos_hi: this lane's, lane and lane + 32).
template <int kScore>
__device__ __forceinline__ void prepare_any_scores(const TreeParams &p, float *x, float slope, int key, int prefix, int anchor,
                                                   int pos_lo, int pos_hi)
{
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float y;
        if constexpr ((kScore & 1) != 0) {
            const float u = x[j] * p.cap_u, size = fabsf(u);
            y = p.tanh_c[kTanhTerms - 1];
#pragma unroll
            for (int k = kTanhTerms - 2; k >= 0; --k)
                y = fmaf(y, u * u, p.tanh_c[k]);
            y *= u;
            const float rest = rcp(1.f + ex2(size * (2.f * kLog2e)));
            if (size > 1.f)
                y = copysignf(fmaf(-2.f * p.cap_out, rest, p.cap_out), u);
        } else {
            y = x[j] * p.c;
        }
        if constexpr ((kScore & 2) != 0) {
            const int d = key + j - prefix;
            const int drafted = __shfl_sync(0xFFFFFFFFu, d < 32 ? pos_lo : pos_hi, d & 31);
            y = fmaf(slope, distance(d < 0 ? key + j : drafted, anchor), y);
        }
        x[j] = y;
    }
}

// Lane q of each group of four gets the others' fourth q: o[4 i + j] of lane q
// becomes o[4 q + j] of lane i.
__device__ __forceinline__ void transpose4(float *o)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1) {
        const bool odd = lane & bit;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!(k & bit)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? o[4 * k + j] : o[4 * (k | bit) + j], bit);
                    if (odd)
                        o[4 * k + j] = got;
                    else
                        o[4 * (k | bit) + j] = got;
                }
            }
    }
}

// This thread's row of O (TMEM) and of earlier spans: v = O + f * sums. `out`
// writes v to `sums` (which counts from `earlier` on), else to O. sums[column * stride].
__device__ __forceinline__ void add_up(float *sums, int stride, uint32_t o, bool earlier, float f, bool out)
{
#pragma unroll 1
    for (int col = 0; col < kHeadDim; col += 16) {
        float acc[16], was[16];
        tmem_ld16(acc, o + col);
        if (earlier) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                was[j] = sums[static_cast<size_t>(col + j) * stride];
        }
        tmem_wait_ld16(acc);
        if (earlier) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                acc[j] = fmaf(was[j], f, acc[j]);
        }
        if (out) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                sums[static_cast<size_t>(col + j) * stride] = acc[j];
        } else {
            tmem_st16(o + col, acc);
        }
    }
}

template <int kScore>
__device__ bool soften(const TreeParams &p, TreeSmem &s, int rg, bool pair, int cta)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stream = warp >> 2;
    const int row = (warp & 3) * 32 + lane; // of the row tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tmem_s = s.tmem_base + lanes + kColS + stream * 128;
    const int row_tile = 2 * rg + (pair ? stream : 0);
    const int token = row_tile * p.tile_tokens + row / p.g;
    const bool real = row < p.tile_tokens * p.g && token < p.M;
    const bool warp_works = __any_sync(0xFFFFFFFFu, real);
    const float c = kScore ? 1.f : p.c;

    // What a row brings into a segment; the next segment's is fetched while this
    // one's last products run.
    struct Row {
        uint64_t mask;
        float slope;
        int pos_lo, pos_hi; // this lane's drafted tokens' positions (lane, lane + 32)
        bool live;
    };
    const auto fetch_row = [&](const Segments &of) {
        Row r{0, 0.f, 0, 0, real && token < of.n};
        if (r.live) {
            r.mask = p.tree_mask[static_cast<size_t>(of.b) * p.M + token];
            if constexpr ((kScore & 2) != 0)
                r.slope = p.slopes[of.h * p.g + row % p.g] * kLog2e;
        }
        if constexpr ((kScore & 2) != 0) {
            const int32_t *at = p.positions + static_cast<size_t>(of.b) * p.M;
            r.pos_lo = lane < of.n ? at[lane] : 0;
            r.pos_hi = lane + 32 < of.n ? at[lane + 32] : 0;
        }
        return r;
    };
    float *sums = p.sums ? p.sums + static_cast<size_t>(2 * cta + stream) * kHeadDim * p.sum_rows + row : nullptr;
    Segments seg(s);
    bool more = seg.next(p);
    Row next_row = fetch_row(seg);
    int step = 0; // the run's next step, of either stream
    bool ok = true;
    for (int index = 0; ok && more; ++index) {
        const int prefix = seg.T - seg.n;
        const bool live = next_row.live;
        const uint64_t mask = seg.n < 64 ? next_row.mask & ((1ull << seg.n) - 1ull) : next_row.mask;
        const float slope = next_row.slope;
        const int pos_lo = next_row.pos_lo, pos_hi = next_row.pos_hi;
        // A row's own position is a constant of its scores, slope * pos_i, and cancels in
        // the softmax. The bias is taken relative to `anchor` instead, at or within 64
        // positions of the visible key that it favours most, so that the scores that count
        // keep their bits however far pos_i lies from them. It depends on the row alone,
        // so the pieces of a (sequence, head) agree. Drafted tokens around the prefix's end
        // and slopes of at most 2 in base 2 (a bias of at most 256 there: half a unit in the
        // last place is 2^-17, as much as a weight's pair loses) leave the prefix's first key
        // or its end; otherwise the drafted tokens are looked through.
        int anchor = 0;
        if constexpr ((kScore & 2) != 0) {
            const bool falls = slope < 0.f; // along the keys
            const auto near = [&](int j, int pos) {
                return j >= seg.n || static_cast<uint32_t>(pos) - static_cast<uint32_t>(prefix) + 64u < 128u;
            };
            anchor = falls ? 0 : prefix;
            if (!__all_sync(0xFFFFFFFFu, near(lane, pos_lo) && near(lane + 32, pos_hi) && fabsf(slope) <= 2.f)) {
                if (prefix == 0)
                    anchor = falls ? INT_MAX : INT_MIN;
#pragma unroll 1
                for (int j = 0; j < seg.n; ++j) {
                    const int pos = __shfl_sync(0xFFFFFFFFu, j < 32 ? pos_lo : pos_hi, j & 31);
                    if (mask >> j & 1u)
                        anchor = falls ? min(anchor, pos) : max(anchor, pos);
                }
            }
        }
        const int seg_steps = (seg.seg_tile1 - seg.seg_tile0) * (pair ? 2 : 1);
        float m = -INFINITY; // the reference, in units of 1 / c
        float l = 0.f;
        bool fresh = true;  // nothing of this segment yet
        bool summed = false; // `sums` holds earlier spans, relative to m_sums
        float m_sums = 0.f;
        for (int n = step + ((step ^ stream) & 1); ok && n < step + seg_steps; n += 2) {
            const int tile = seg.seg_tile0 + ((n - step) >> (pair ? 1 : 0));
            const int unit = pair ? n >> 1 : n;
            ok = warp_wait(&s.s_full[stream], (n >> 1) & 1);
            if (!ok)
                break;
            tc_fence_after();
            if (warp_works) {
                const int key0 = tile * kTileKeys;
                const uint32_t valid = s.valid[unit % kValidRing];
                const bool tail = key0 + kTileKeys > prefix;
                const bool fix = tail || valid != 0xFFu;
                // Capped and biased scores, 16 keys at a time. Biased ones are formed
                // in place, in a loop small enough for the instruction cache (118
                // us for token decoding of 33 ragged sequences, 129 us unrolled in
                // registers); capped ones in registers (t = 131072 113 us, in place
                // 116 us). What the common form does not cover (drafted tokens'
                // own positions, scores past their cap) is left as it is and done
                // after it.
                uint32_t left = 0; // a bit per 16 keys
                if constexpr ((kScore & 2) != 0) {
                    float y[2][16];
                    tmem_ld16(y[0], tmem_s);
#pragma unroll 1
                    for (int i = 0; i < 8; i += 2) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            tmem_wait_ld16(y[k]);
                            tmem_ld16(y[k ^ 1], tmem_s + 16 * ((i + k + 1) & 7));
                            const int key = key0 + 16 * (i + k);
                            const float over = prepare_scores<kScore, 16>(p, y[k], slope, distance(key, anchor));
                            const bool rest = __any_sync(0xFFFFFFFFu, live && over > 1.f) || (key + 16 > prefix && key < seg.T);
                            if (rest)
                                left |= 1u << (i + k);
                            else
                                tmem_st16(tmem_s + 16 * (i + k), y[k]);
                        }
                    }
                    tmem_wait_ld16(y[0]); // the last prefetch, of no use
                }
                float x[kTileKeys];
                if constexpr (kScore == 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        tmem_ld16(x + 16 * i, tmem_s + 16 * i);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        tmem_wait_ld16(x + 16 * i);
                    const float over = prepare_scores<kScore, kTileKeys>(p, x, 0.f, 0.f);
                    left = __any_sync(0xFFFFFFFFu, live && over > 1.f) ? 0xFFu : 0u;
                }
                if constexpr (kScore != 0) {
                    if (left) {
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            if (!(left >> i & 1u))
                                continue;
                            float y[16];
                            tmem_ld16(y, tmem_s + 16 * i);
                            tmem_wait_ld16(y);
                            prepare_any_scores<kScore>(p, y, slope, key0 + 16 * i, prefix, anchor, pos_lo, pos_hi);
                            tmem_st16(tmem_s + 16 * i, y);
                        }
                    }
                    tmem_wait_st();
                }
                if (kScore != 1 || left) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        tmem_ld16(x + 16 * i, tmem_s + 16 * i);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        tmem_wait_ld16(x + 16 * i);
                }
                if (fix) { // hidden keys
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t bits = visible_word(prefix - key0 - 32 * w, mask, valid >> (2 * w));
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            x[32 * w + j] = (bits >> j) & 1u ? x[32 * w + j] : -INFINITY;
                    }
                }
                float tops[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int j = 4; j < kTileKeys; j += 2)
                    tops[j >> 1 & 3] = max3(tops[j >> 1 & 3], x[j], x[j + 1]);
                const float high = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                // The tensor core rounds its accumulators towards zero at each product:
                // over thousands of keys O loses some 2^-25 of itself a time. For fp32
                // outputs O moves out every kSpan tiles and is added up in fp32, to
                // nearest (4 x 131072 keys: 2.3e-5 -> 4.7e-6 of the result; bf16 outputs round
                // far above that).
                const bool span = p.sums && !fresh && ((n - step) >> 1) % kSpan == 0;
                if (span) {
                    const float f = summed && m_sums > -INFINITY ? ex2((m_sums - m) * c) : 0.f;
                    add_up(sums, p.sum_rows, s.tmem_base + lanes + kColO + stream * 128, summed, f, true);
                    summed = true;
                    m_sums = m;
                }
                // move the reference where the row has none yet, or its scores left its range
                const bool move =
                    fresh || (live && (m == -INFINITY ? high > -INFINITY : (high - m) * c > kRescaleLog2));
                if (__any_sync(0xFFFFFFFFu, move)) {
                    const float before = m;
                    if (move)
                        m = high;
                    const float f = !move ? 1.f : (before == -INFINITY ? 0.f : ex2((before - m) * c));
                    l *= f;
                    if (!fresh && !span) {
                        const uint32_t o = s.tmem_base + lanes + kColO + stream * 128;
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            float acc[16];
                            tmem_ld16(acc, o + 16 * i);
                            tmem_wait_ld16(acc);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                acc[j] *= f;
                            tmem_st16(o + 16 * i, acc);
                        }
                    }
                }
                // p = 2^(x c - m c). For scores so large that the rounding of m c
                // matters the difference is taken before the product.
                const float ref = m == -INFINITY ? 0.f : m * c;
                const bool large = kScore == 0 && fabsf(ref) > 65536.f;
                const float shift = large ? m : 0.f, neg_ref = large ? 0.f : -ref;
                const bool any_large = __any_sync(0xFFFFFFFFu, large);
                if (any_large) {
#pragma unroll
                    for (int j = 0; j < kTileKeys; ++j)
                        x[j] -= shift;
                }
                f32x2 sum(0.f, 0.f);
                float offset = neg_ref;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float w[16]; // 8 columns hi, 8 columns lo
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a, b;
                        fma2(f32x2(x[16 * i + 2 * j], x[16 * i + 2 * j + 1]), f32x2(c, c), f32x2(offset, offset)).get(a, b);
                        a = ex2(a), b = ex2(b);
                        const f32x2 ab(a, b);
                        sum = add2(sum, ab);
                        // hi: nearest bf16; lo: the exact rest, rounded
                        const uint32_t hi = pack_bf16x2(a, b);
                        w[j] = __uint_as_float(hi);
                        float ra, rb;
                        fma2(f32x2(bf16_lo(hi), bf16_hi(hi)), f32x2(-1.f, -1.f), ab).get(ra, rb);
                        w[8 + j] = __uint_as_float(pack_bf16x2(ra, rb));
                    }
                    tmem_st16(tmem_s + 16 * i, w);
                    if (i == 3) { // half of P: its product can start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&s.p_half[stream]);
                        // a zero read after the arrival: the second half's work
                        // depends on it and so stays behind it
                        offset += lds_f32(smem_addr(&s.zero));
                    }
                }
                float even, odd;
                sum.get(even, odd);
                l += even + odd;
                tmem_wait_st();
            } else if (lane == 0) {
                mbar_arrive(&s.p_half[stream]);
            }
            fresh = false;
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.p_ready[stream]);
        }
        step += seg_steps;
        if (!ok)
            break;

        Segments following = seg;
        more = following.next(p);
        if (more)
            next_row = fetch_row(following);

        // ---- the end of the segment: O of the last product, joined and written
        float w_own = 1.f, w_other = 0.f, top = m == -INFINITY ? -INFINITY : m * c;
        if (p.sums) {
            ok = warp_wait(&s.seg_done, index & 1);
            if (!ok)
                break;
            tc_fence_after();
            if (summed) { // (the same for the whole warpgroup)
                const float f = m_sums > -INFINITY ? ex2((m_sums - m) * c) : 0.f;
                add_up(sums, p.sum_rows, s.tmem_base + lanes + kColO + stream * 128, true, f, false);
                tmem_wait_st();
            }
            tc_fence_before();
        }
        if (!pair) {
            // both streams hold part of every row: exchange (m, l)
            s.ml[stream][row] = make_float2(top, l);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.ml_ready);
            ok = warp_wait(&s.ml_ready, index & 1);
            if (!ok)
                break;
            const float2 other = s.ml[stream ^ 1][row];
            const float own_top = top;
            top = fmaxf(own_top, other.x);
            w_own = l == 0.f ? 0.f : ex2(own_top - top);
            w_other = other.y == 0.f ? 0.f : ex2(other.x - top);
            l = (l == 0.f ? 0.f : l * w_own) + (other.y == 0.f ? 0.f : other.y * w_other);
        } else if (l == 0.f) {
            w_own = 0.f;
        }
        if (!p.sums)
            ok = warp_wait(&s.seg_done, index & 1);
        if (!ok)
            break;
        tc_fence_after();
        const uint64_t bad = (s.bad_rows[index & 3][0] | s.bad_rows[index & 3][1]) & mask;
        const bool whole = seg.seg_tile0 == 0 && seg.seg_tile1 == seg.tiles;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const uint32_t out_row = (static_cast<uint32_t>(seg.b) * p.M + token) * p.Hq + seg.h * p.g + row % p.g;
        const uint32_t live_rows = __ballot_sync(0xFFFFFFFFu, live);
        const size_t rec = static_cast<size_t>(2 * cta + (seg.seg_tile0 > 0 ? 0 : 1)) * p.rec_rows +
                           (pair ? stream * kTileRows : 0) + (warp & 3) * 32; // this warp's first row
        // 16 columns at a time: all 128 of the stream's row tile, or 64 of the joined streams
        const int col0 = pair ? 0 : 64 * stream, columns = pair ? 128 : 64;
        const uint32_t tmem_o = s.tmem_base + lanes + kColO;
        if (warp_works) {
#pragma unroll 1
            for (int col = col0; col < col0 + columns; col += 16) {
                float o[16];
                tmem_ld16(o, tmem_o + stream * 128 + col);
                if (!pair) {
                    float o2[16];
                    tmem_ld16(o2, tmem_o + (stream ^ 1) * 128 + col);
                    tmem_wait_ld16(o), tmem_wait_ld16(o2);
#pragma unroll
                    for (int j = 0; j < 16; ++j) { // a stream without a visible key may hold anything
                        const float a = w_own == 0.f ? 0.f : o[j] * w_own;
                        o[j] = w_other == 0.f ? a : fmaf(o2[j], w_other, a);
                    }
                } else {
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = w_own == 0.f ? 0.f : o[j];
                }
                if (live) {
                    // V elements left out of the products because they are not finite
                    for (uint64_t rest = bad; rest; rest &= rest - 1) {
                        const int slot = prefix + __ffsll(static_cast<long long>(rest)) - 1;
                        const int tile = slot / kTileKeys;
                        const int phys = p.block_table[static_cast<size_t>(seg.b) * p.max_pages + (slot >> p.log2_page)];
                        if (tile < seg.seg_tile0 || tile >= seg.seg_tile1 || phys < 0 || phys >= p.num_pages)
                            continue;
                        const uint16_t *v = p.v + ((((static_cast<size_t>(phys) * p.Hkv + seg.h) << p.log2_page) +
                                                    (slot & ((1 << p.log2_page) - 1))) *
                                                       kHeadDim +
                                                   col);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if ((v[j] & 0x7F80u) == 0x7F80u)
                                o[j] += __uint_as_float(static_cast<uint32_t>(v[j]) << 16);
                    }
                }
                if (whole) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] *= inv;
                }
                // 4 x 4 transpose in groups of four lanes: lane q gets columns
                // 4q .. 4q+3 of the group's rows, and a store covers 64 bytes
                // of each of 8 rows instead of 16 bytes of each of 32
                transpose4(o);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = (lane & ~3) + i;
                    const uint32_t row_i = __shfl_sync(0xFFFFFFFFu, out_row, from);
                    if (live_rows >> from & 1u) {
                        const int c = col + 4 * (lane & 3);
                        const float4 v = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        if (!whole)
                            *reinterpret_cast<float4 *>(p.rec_acc + (rec + from) * kHeadDim + c) = v;
                        if (whole && p.out_f32)
                            *reinterpret_cast<float4 *>(p.out_f32 + static_cast<size_t>(row_i) * kHeadDim + c) = v;
                        if (whole && p.out_bf16)
                            *reinterpret_cast<uint2 *>(p.out_bf16 + static_cast<size_t>(row_i) * kHeadDim + c) =
                                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                    }
                }
                __syncwarp();
            }
            if (live && !whole && (pair || stream == 0)) {
                p.rec_m[rec + lane] = top;
                p.rec_l[rec + lane] = l;
            }
        }
        if (!pair) { // neither stream's O may be overwritten before both warpgroups have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s.epi_done);
            ok = warp_wait(&s.epi_done, index & 1);
        }
        seg = following;
    }
    return ok;
}

template <int kScore>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ TreeParams p)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    TreeSmem &s = *reinterpret_cast<TreeSmem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rg = blockIdx.x % p.row_groups, cta = blockIdx.x / p.row_groups;
    const bool pair = 2 * rg + 1 < p.row_tiles;
    if (tid == 0) {
        prefetch_tensormap(&mq), prefetch_tensormap(&mk), prefetch_tensormap(&mv);
        for (int i = 0; i < kSlots; ++i)
            mbar_init(&s.full[0][i], 1), mbar_init(&s.full[1][i], 1),
                mbar_init(&s.empty[i], pair ? 2 : 1); // the streams that read a slot
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1), mbar_init(&s.q_empty[i], 2);
            mbar_init(&s.drain[i], 1);
            mbar_init(&s.s_full[i], 2);  // the products' completion, and the issuing thread
            mbar_init(&s.round_done[i], 1);
            mbar_init(&s.p_half[i], 4); // one arrival per warp of the stream
            mbar_init(&s.p_ready[i], 4);
        }
        mbar_init(&s.seg_done, 4); // per stream: the products' completion, and the issuing thread
        mbar_init(&s.ml_ready, kSoftmaxThreads / 32);
        mbar_init(&s.epi_done, kSoftmaxThreads / 32);
        fence_mbar_init();
    }
    if (warp == kMmaWarp)
        tmem_alloc_all(&s.tmem_base);

    // Everything read from here on may come from the kernel before this one, and
    // the next kernel may start once that one is done (it may read inputs before
    // it waits).
    grid_dependency_wait();
    allow_dependent_launch();
    plan_run<kTreeThreads>(p, s, cta);
    if (tid == 0)
        s.zero = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    // Registers move from the third warpgroup to the softmax, whose threads
    // hold 128 scores: 256 * 216 + 128 * 72 = 384 * 168 as launched.
    bool ok = true;
    if (warp >= kProducerWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kProducerWarp && s.units > 0)
            ok = produce(p, s, &mq, &mk, &mv, rg, pair);
        else if (warp <= kMmaWarp + 1 && s.units > 0)
            ok = multiply(p, s, pair, warp - kMmaWarp);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        if (s.units > 0)
            ok = soften<kScore>(p, s, rg, pair, blockIdx.x);
    }
    if (!ok && lane == 0)
        atomicOr(&g_flags_tree, PGQA_DEVERR_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        tmem_free_all(s.tmem_base);
}

// How a call's rows and CTAs are laid out; from sizes alone, so that the
// workspace query and the launch agree.
struct Layout {
    int tile_tokens, row_tiles, row_groups, rec_rows, ctas;
    size_t base_bytes, stat_bytes, acc_bytes, sum_bytes;
    int sum_rows;
};

size_t align256(size_t x) { return (x + 255) & ~size_t{255}; }

Layout layout(int B, int M, int Hq, int Hkv, int page_size, int max_pages, int sm_count)
{
    Layout y{};
    const int g = Hq / Hkv;
    y.tile_tokens = M < kTileRows / g ? M : kTileRows / g;
    y.row_tiles = (M + y.tile_tokens - 1) / y.tile_tokens;
    y.row_groups = (y.row_tiles + 1) / 2;
    y.rec_rows = y.row_tiles > 1 ? 2 * kTileRows : y.tile_tokens * g;
    const long long tiles = (static_cast<long long>(max_pages) * page_size + kTileKeys - 1) / kTileKeys;
    const long long units = tiles * B * Hkv;
    const int ctas = sm_count / y.row_groups;
    y.ctas = static_cast<int>(units < ctas ? units : ctas);
    if (y.ctas < 1)
        y.ctas = 1;
    const size_t records = static_cast<size_t>(2) * y.ctas * y.row_groups;
    y.base_bytes = align256((static_cast<size_t>(B) + 1) * sizeof(int32_t));
    y.stat_bytes = align256(records * y.rec_rows * sizeof(float));
    y.acc_bytes = records * y.rec_rows * kHeadDim * sizeof(float);
    // a stream passes a span only where a (sequence, head) has that many tiles
    y.sum_rows = (y.tile_tokens * g + 31) / 32 * 32;
    y.sum_bytes = tiles > kSpan ? records * kHeadDim * y.sum_rows * sizeof(float) : 0;
    return y;
}

CUresult encode_cache(EncodeTiledFn fn, CUtensorMap *map, const void *base, long long rows, int page_size)
{
    // [row group of 8][half][row][64 columns]: a box is a page's (or half a
    // page's) rows as 1 KB swizzle atoms, two per 8 rows
    const int box_groups = (page_size < kTileKeys ? page_size : kTileKeys) / 8;
    const cuuint64_t dims[4] = {64u, 8u, 2u, static_cast<cuuint64_t>(rows / 8)};
    const cuuint64_t strides[3] = {kRowBytes, 128u, 8u * kRowBytes};
    const cuuint32_t box[4] = {64u, 8u, 2u, static_cast<cuuint32_t>(box_groups)};
    const cuuint32_t elem[4] = {1u, 1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult encode_query(EncodeTiledFn fn, CUtensorMap *map, const void *base, int tokens, int Hq, int g, int tile_tokens)
{
    const cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {kRowBytes, static_cast<cuuint64_t>(Hq) * kRowBytes};
    const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(g), static_cast<cuuint32_t>(tile_tokens)};
    const cuuint32_t elem[3] = {1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

constexpr int kMaxDevices = 64;

template <int kScore>
cudaError_t launch_score(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const TreeParams &p,
                         cudaStream_t stream)
{
    static std::atomic<bool> configured[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev >= kMaxDevices || !configured[dev].load(std::memory_order_acquire)) {
        err = cudaFuncSetAttribute(tree_attn_kernel<kScore>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTreeSmem);
        if (err != cudaSuccess)
            return err;
        if (dev < kMaxDevices)
            configured[dev].store(true, std::memory_order_release);
    }
    return launch_pdl(tree_attn_kernel<kScore>, dim3(static_cast<unsigned>(p.ctas * p.row_groups)), dim3(kTreeThreads),
                      kTreeSmem, stream, mq, mk, mv, p);
}

} // namespace

size_t tree_attn_workspace_bytes(int B, int M, int Hq, int Hkv, int page_size, int max_pages, int sm_count)
{
    if (B == 0)
        return 0;
    const Layout y = layout(B, M, Hq, Hkv, page_size, max_pages, sm_count);
    return y.base_bytes + 2 * y.stat_bytes + y.acc_bytes + y.sum_bytes;
}

cudaError_t launch_tree_attn(const TreeAttnArgs &a, cudaStream_t stream)
{
    const EncodeTiledFn fn = tensor_map_encoder();
    if (!fn)
        return cudaErrorNotSupported;
    const Layout y = layout(a.B, a.M, a.Hq, a.Hkv, a.page_size, a.max_pages, a.sm_count);
    TreeParams p{};
    p.v = a.v_cache;
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
    p.row_tiles = y.row_tiles;
    p.row_groups = y.row_groups;
    p.rec_rows = y.rec_rows;
    p.ctas = y.ctas;
    p.negate_q = a.scale < 0.f;
    // A scale of 0 gives every key the same weight; the smallest positive
    // factor does the same and keeps -inf * c, the score of a hidden key, -inf.
    p.c = std::fmin(std::fmax(std::fabs(a.scale) * kLog2e, FLT_MIN), FLT_MAX);
    if (a.softcap > 0.f) {
        const float cap = std::fmin(a.softcap, 1e30f); // no cap to any score, and its products stay finite
        p.cap_u = std::fmin(std::fabs(a.scale) / cap, FLT_MAX);
        p.cap_out = cap * kLog2e;
        for (int k = 0; k < kTanhTerms; ++k)
            p.tanh_c[k] = static_cast<float>(kTanh[k] * cap * 1.4426950408889634);
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
    p.sum_rows = y.sum_rows;
    CUtensorMap mq, mk, mv;
    const long long rows = static_cast<long long>(a.num_pages) * a.Hkv * a.page_size;
    if (encode_query(fn, &mq, a.q, a.B * a.M, a.Hq, p.g, y.tile_tokens) != CUDA_SUCCESS ||
        encode_cache(fn, &mk, a.k_cache, rows, a.page_size) != CUDA_SUCCESS ||
        encode_cache(fn, &mv, a.v_cache, rows, a.page_size) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cudaError_t err;
    switch ((a.softcap > 0.f ? 1 : 0) | (a.slopes ? 2 : 0)) {
    case 0: err = launch_score<0>(mq, mk, mv, p, stream); break;
    case 1: err = launch_score<1>(mq, mk, mv, p, stream); break;
    case 2: err = launch_score<2>(mq, mk, mv, p, stream); break;
    default: err = launch_score<3>(mq, mk, mv, p, stream); break;
    }
    if (err != cudaSuccess)
        return err;
    return launch_tree_merge(p, y.ctas, stream);
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
