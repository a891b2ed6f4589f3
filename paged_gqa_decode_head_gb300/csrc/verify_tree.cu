// verify_tree.cu -- verify_drafted_tree: which drafted tokens the target model
// accepts, and the token behind the accepted path, from given random numbers.
//
// Mathematics. At the path's last node: p = softmax(target / T), q = softmax(draft
// / T), E the rejected children's tokens. The children are tested in order; child
// t is accepted if u < p'(t) / q'(t), where q' is q without E, renormalised, and p'
// the renormalised residual that each rejection leaves, p' <- max(p' - q', 0). With
// unnormalised sums the residuals telescope, max(max(x - a, 0) - b, 0) = max(x - a
// - b, 0): after any rejections the residual is max(p - C q, 0) outside E, and a
// rejection adds S / Q to C, where S is the residual's sum and Q that of q outside
// E. So a node's state is one number and a short list. Without draft logits q is a
// point mass on t: accepted if u S < p(t), and E leaves p. The last token is the
// winner of an exponential race, argmax residual_i / e_i with given e_i ~ Exp(1),
// which draws from the residual in one pass and, unlike an inverse distribution
// function, does not hang on the last bits of a sum over the vocabulary.
//
// Bound. The path's rows are read once from memory (V logits each, two models'
// with draft logits) and the noise once; what a call costs is the chain of its nodes:
// a pass over a row, a reduction over the cluster, a handful of scalar tests. With point
// masses a rejection needs no pass: the residual's sum loses p(t), unless so little is
// left that the difference would lose its precision. Measured (us, a path of 4 nodes
// behind 151936 bf16 logits / 64 sequences with draft logits / 24 of 32003 fp32
// logits): 32.4 / 132 / 38.4 with the statistics joined pair by pair, a division per
// element of the race and the children searched one by one; 23.4 / 110 / 30.4 with sums
// rescaled once a level, divisions only for scores that may win and children by ballot.
//
// Split: a cluster of blocks per sequence; every thread of it holds the same
// scalars and takes the same turns. A pass's loads are on their way several pieces at a
// time, from 16-byte boundaries of the row whatever its alignment.
//
// Rounding: logits are widened to fp32; exponentials, sums and tests in fp32, sums
// over a row as a tree of threads' partial sums.
#include "common.cuh"
#include "launch.h"

#include <atomic>
#include <cfloat>
#include <climits>

namespace pgqa {
namespace {

__device__ unsigned g_flags_verify;

constexpr int kVerifyThreads = 512;
constexpr int kMaxCluster = 16;
constexpr int kMaxDrafted = 64;
constexpr int kPiece = 8; // logits a thread takes at a time
// Less than this of q left is nothing: S / Q is at most its reciprocal then, 64 of them and
// their products with q are finite.
constexpr float kLeastRest = 0x1p-119f;
// Higher temperatures count as this one: a difference of logits past fp32's range stays no
// weight, and is not infinity times zero.
constexpr float kMostTemperature = 0x1p100f;
constexpr int kMaxDevices = 64;

struct VerifyParams {
    const void *target, *draft;
    long long target_stride, draft_stride;
    const int32_t *tokens, *parents, *draft_lens;
    const float *temperatures, *accept, *noise;
    int M, A, V;
    int32_t *path, *path_lens, *new_tokens;
    float *logprobs;
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const float *local, uint32_t rank, float v)
{
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// A logit as the tests see it: NaN counts as -inf, +inf as the largest number.
__device__ __forceinline__ float usable(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

template <typename T> __device__ __forceinline__ float logit_at(const T *row, int i)
{
    if constexpr (sizeof(T) == 2)
        return usable(__uint_as_float(static_cast<uint32_t>(row[i]) << 16));
    else
        return usable(row[i]);
}

// Eight elements of a row as they lie in memory.
template <typename T> struct Raw;
template <> struct Raw<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t *at) { a = *reinterpret_cast<const uint4 *>(at); }
    __device__ __forceinline__ void get(float *x) const { unpack8(a, x); }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *at)
    {
        a = reinterpret_cast<const float4 *>(at)[0], b = reinterpret_cast<const float4 *>(at)[1];
    }
    __device__ __forceinline__ void get(float *x) const
    {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

// A piece of a row of V, elements e .. e + 7, and kCount of them `stride` apart; -inf outside
// the row. Rows lie anywhere on their element's alignment. All of a batch's loads are on
// their way before the first is used: a pass is as long as its round trips to memory.
template <typename T, int kCount> struct Batch {
    Raw<T> raw[kCount];
    const T *row;
    int e, stride, V;
    bool aligned;
    __device__ __forceinline__ bool inside(int i) const
    {
        return aligned && e + i * stride >= 0 && e + i * stride + kPiece <= V;
    }
    __device__ __forceinline__ Batch(const T *row_, int e_, int stride_, int V_)
        : row(row_), e(e_), stride(stride_), V(V_), aligned((reinterpret_cast<uintptr_t>(row_ + e_) & 15u) == 0)
    {
#pragma unroll
        for (int i = 0; i < kCount; ++i)
            if (inside(i))
                raw[i].load(row + e + i * stride);
    }
    // Whether piece i has elements; they are in x then, as they are in memory.
    __device__ __forceinline__ bool get(int i, float *x) const
    {
        const int at = e + i * stride;
        if (inside(i)) {
            raw[i].get(x);
            return true;
        }
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            x[j] = -INFINITY;
        if (at >= V)
            return false;
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (at + j >= 0 && at + j < V)
                x[j] = logit_at(row, at + j);
        return true;
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// 2^((x - m) k), 0 for a logit of -inf.
__device__ __forceinline__ float weight(float x, float m, float k) { return x == -INFINITY ? 0.f : ex2((x - m) * k); }

__device__ __forceinline__ void clean(float *x)
{
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
        x[j] = usable(x[j]);
}

// Element l of a piece, if it has one, takes no part.
__device__ __forceinline__ void leave_out(int l, float *x)
{
    if (static_cast<unsigned>(l) < kPiece) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            x[j] = j == l ? -INFINITY : x[j];
    }
}

// Maximum, its first place, and the sum of weights relative to it.
struct RowStats {
    float m, s;
    int at;
};
struct VerifySmem {
    float parts[2][kMaxCluster][6]; // a block's result of one reduction, from every block, twice in turn
    float warp_parts[kVerifyThreads / 32][6];
    int tokens[kMaxDrafted], parents[kMaxDrafted];
    float accept[kMaxDrafted], child_p[kMaxDrafted], child_q[kMaxDrafted];
    int tried[kMaxDrafted];
};

// Sets of N values joined over lanes that differ in the bits below `width` (32 lanes hold
// width different sets), in a fixed order; every lane gets the result.
struct AddAcross {
    template <int N> __device__ __forceinline__ void operator()(float (&v)[N], int width) const
    {
        for (int off = width / 2; off > 0; off >>= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], off);
        }
    }
};
// A score and its place: the highest, of equal ones the first.
struct BestAcross {
    __device__ __forceinline__ void operator()(float (&v)[2], int) const
    {
        const float top = warp_max(v[0]);
        const int at = __reduce_min_sync(0xFFFFFFFFu, v[0] == top ? __float_as_int(v[1]) : INT_MAX);
        v[0] = top, v[1] = __int_as_float(at);
    }
};
// Statistics of one row (m, s, at) or of two (and m, s): every lane's sum is rescaled once.
struct StatsAcross {
    float k;
    template <int N> __device__ __forceinline__ void operator()(float (&v)[N], int width) const
    {
        const float top = warp_max(v[0]);
        const int at = __reduce_min_sync(0xFFFFFFFFu, v[0] == top ? __float_as_int(v[2]) : INT_MAX);
        float s[N == 5 ? 2 : 1];
        s[0] = v[1] * weight(v[0], top, k);
        v[0] = top, v[2] = __int_as_float(at);
        if constexpr (N == 5) {
            const float top_q = warp_max(v[3]);
            s[1] = v[4] * weight(v[3], top_q, k);
            v[3] = top_q;
        }
        AddAcross()(s, width);
        v[1] = s[0];
        if constexpr (N == 5)
            v[4] = s[1];
    }
};

// The cluster's reduction: every thread gives N values, every thread of every block gets the
// result.
template <int N, typename Across>
__device__ __forceinline__ void reduce(VerifySmem &s, int &turn, float (&v)[N], const Across &across)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    across(v, 32);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            s.warp_parts[warp][i] = v[i];
    }
    __syncthreads();
    constexpr int kWarps = kVerifyThreads / 32;
    static_assert((kWarps & (kWarps - 1)) == 0, "a lane per warp");
    const int blocks = cluster_size(), rank = cluster_rank(); // a power of two
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = s.warp_parts[lane & (kWarps - 1)][i];
        across(v, kWarps);
        if (lane < blocks) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                store_remote(&s.parts[turn][rank][i], lane, v[i]);
        }
    }
    cluster_sync();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = s.parts[turn][lane & (blocks - 1)][i];
    across(v, blocks);
    turn ^= 1;
}

// kDraft: with draft logits.
template <typename T, bool kDraft>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const __grid_constant__ VerifyParams p)
{
    __shared__ VerifySmem s;
    grid_dependency_wait();
    allow_dependent_launch();
    const int tid = threadIdx.x, blocks = cluster_size(), rank = cluster_rank();
    const int b = blockIdx.x / blocks;
    const int first = (rank * kVerifyThreads + tid) * kPiece, stride = blocks * kVerifyThreads * kPiece;
    constexpr int kBatch = (sizeof(T) == 2 ? 4 : 2) / (kDraft ? 2 : 1); // pieces on their way per row
    const int n = p.draft_lens ? p.draft_lens[b] : p.M;
    const float temperature = p.temperatures[b];
    const size_t out0 = static_cast<size_t>(b) * p.A;
    const bool writes = rank == 0 && tid == 0;
    // what no step below writes
    if (rank == 0)
        for (int i = tid; i < p.A; i += kVerifyThreads) {
            p.path[out0 + i] = -1;
            p.new_tokens[out0 + i] = -1;
            if (p.logprobs)
                p.logprobs[out0 + i] = 0.f;
        }
    if (n <= 0 || n > p.M || !(temperature >= 0.f)) {
        if (writes) {
            p.path_lens[b] = 0;
            if (n != 0)
                atomicOr(&g_flags_verify, PGQA_DEVERR_BAD_CONTEXT);
        }
        return; // the whole cluster
    }
    if (tid < n) {
        const size_t i = static_cast<size_t>(b) * p.M + tid;
        const int token = p.tokens[i];
        s.tokens[tid] = token >= 0 && token < p.V ? token : -1;
        if (s.tokens[tid] < 0 && tid > 0 && rank == 0)
            atomicOr(&g_flags_verify, PGQA_DEVERR_BAD_PATH);
        s.parents[tid] = tid > 0 ? p.parents[i] : -1;
        s.accept[tid] = p.accept[i];
    }
    cluster_sync(); // every block has started before one writes to another
    const bool greedy = temperature == 0.f;
    const float k = fminf(kLog2e / (greedy ? 1.f : fminf(temperature, kMostTemperature)), FLT_MAX);
    const float *noise = p.noise + static_cast<size_t>(b) * p.V;
    int turn = 0;
    int cur = 0, count = 0;
    for (;;) {
        const T *row = static_cast<const T *>(p.target) + (static_cast<long long>(b) * p.M + cur) * p.target_stride;
        const T *drow = kDraft ? static_cast<const T *>(p.draft) + (static_cast<long long>(b) * p.M + cur) * p.draft_stride
                               : nullptr;
        if (writes)
            p.path[out0 + count] = cur;
        ++count;
        // the children's logits, wanted after the row's statistics
        if (tid > cur && tid < n && s.parents[tid] == cur && s.tokens[tid] >= 0) {
            s.child_p[tid] = logit_at(row, s.tokens[tid]);
            if constexpr (kDraft)
                s.child_q[tid] = logit_at(drow, s.tokens[tid]);
        }
        // ---- statistics of the node's rows
        RowStats st{-INFINITY, 0.f, INT_MAX}, sq{-INFINITY, 0.f, INT_MAX};
        const auto take = [&](float *x, int e, RowStats &a) {
            float top = x[0];
#pragma unroll
            for (int j = 1; j < kPiece; ++j)
                top = fmaxf(top, x[j]); // NaN is passed over
            if (!(top <= FLT_MAX)) {
                clean(x);
                top = x[0];
#pragma unroll
                for (int j = 1; j < kPiece; ++j)
                    top = fmaxf(top, x[j]);
            }
            if (top > a.m) {
                a.s *= weight(a.m, top, k);
                a.m = top;
#pragma unroll
                for (int j = kPiece - 1; j >= 0; --j)
                    a.at = x[j] == top ? e + j : a.at;
            }
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                sum += ex2((x[j] - a.m) * k);
            if (sum != sum) { // a NaN, or nothing but -inf so far
                clean(x);
                sum = 0.f;
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    sum += weight(x[j], a.m, k);
            }
            a.s += sum;
        };
        // pieces begin on the row's 16-byte boundaries, up to seven elements before it
        const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        const int begin = first - lead;
        for (int e = begin; e < p.V; e += kBatch * stride) {
            const Batch<T, kBatch> bx(row, e, stride, p.V);
            if constexpr (kDraft) {
                const Batch<T, kBatch> by(drow, e, stride, p.V);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    float x[kPiece];
                    if (by.get(i, x))
                        take(x, e + i * stride, sq);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float x[kPiece];
                if (bx.get(i, x))
                    take(x, e + i * stride, st);
            }
        }
        if constexpr (kDraft) {
            float v[5] = {st.m, st.s, __int_as_float(st.at), sq.m, sq.s};
            reduce(s, turn, v, StatsAcross{k});
            st = {v[0], v[1], __float_as_int(v[2])};
            sq = {v[3], v[4], 0};
        } else {
            float v[3] = {st.m, st.s, __int_as_float(st.at)};
            reduce(s, turn, v, StatsAcross{k});
            st = {v[0], v[1], __float_as_int(v[2])};
        }
        const float inv = st.s > 0.f ? 1.f / st.s : 0.f, inv_q = kDraft && sq.s > 0.f ? 1.f / sq.s : 0.f;
        // ---- the children
        int accepted = -1, token = -1, tried = 0;
        float taken = 0.f;            // C
        float mass = 1.f, rest = !kDraft || sq.s > 0.f ? 1.f : 0.f; // S and Q
        if (st.m > -INFINITY && count < p.A) {
            // the node's children, a bit each (every warp for itself)
            const auto children = [&](int i) { return i > cur && i < n && s.parents[i] == cur && s.tokens[i] >= 0; };
            const int lane = tid & 31;
            uint64_t left_to_try = __ballot_sync(0xFFFFFFFFu, children(lane)) |
                                   static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, children(lane + 32))) << 32;
            const auto next_child = [&] {
                const int i = left_to_try ? __ffsll(static_cast<long long>(left_to_try)) - 1 : n;
                left_to_try &= left_to_try - 1;
                return i;
            };
            for (int i = next_child(); i < n;) {
                const int t = s.tokens[i];
                if (greedy) {
                    if (t == st.at) {
                        accepted = i;
                        break;
                    }
                    i = next_child();
                    continue;
                }
                bool again = false;
                for (int j = 0; j < tried; ++j)
                    again = again || s.tried[j] == t;
                const float pt = again ? 0.f : weight(s.child_p[i], st.m, k) * inv;
                const float qt = kDraft && !again ? weight(s.child_q[i], sq.m, k) * inv_q : 0.f;
                const float left = kDraft ? fmaxf(fmaf(-taken, qt, pt), 0.f) : pt;
                const bool given = !kDraft || !(rest >= kLeastRest); // a point mass
                if (s.accept[i] * mass * (given ? 1.f : qt) < left * (given ? 1.f : rest)) {
                    accepted = i;
                    break;
                }
                if (!given)
                    taken += mass / rest;
                if (tid == 0)
                    s.tried[tried] = t;
                ++tried;
                __syncthreads();
                i = next_child();
                if (!kDraft && mass - pt >= 0.25f) {
                    // what is left of p without another pass, as long as the difference keeps
                    // the sum's precision but for two bits
                    mass -= pt;
                } else if (i < n) { // the sums that the next child's test needs
                    float v[2] = {0.f, 0.f};
                    for (int e0 = begin; e0 < p.V; e0 += kBatch * stride) {
                        const Batch<T, kBatch> bx(row, e0, stride, p.V), by(kDraft ? drow : row, e0, stride, kDraft ? p.V : 0);
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const int e = e0 + i * stride;
                            float x[kPiece], y[kPiece];
                            if (!bx.get(i, x))
                                break;
                            clean(x);
                            if constexpr (kDraft) {
                                by.get(i, y);
                                clean(y);
                            }
                            for (int j = 0; j < tried; ++j) {
                                leave_out(s.tried[j] - e, x);
                                if constexpr (kDraft)
                                    leave_out(s.tried[j] - e, y);
                            }
#pragma unroll
                            for (int l = 0; l < kPiece; ++l) {
                                const float pl = weight(x[l], st.m, k) * inv;
                                if constexpr (kDraft) {
                                    const float ql = weight(y[l], sq.m, k) * inv_q;
                                    v[0] += fmaxf(fmaf(-taken, ql, pl), 0.f);
                                    v[1] += ql;
                                } else {
                                    v[0] += pl;
                                }
                            }
                        }
                    }
                    reduce(s, turn, v, AddAcross());
                    mass = v[0];
                    if constexpr (kDraft)
                        rest = v[1];
                }
            }
        }
        float logit = 0.f;
        if (accepted >= 0) {
            token = s.tokens[accepted];
            logit = s.child_p[accepted];
        } else if (st.m > -INFINITY) {
            // ---- the token behind the path
            if (greedy) {
                token = st.at;
            } else {
                for (int whole = 0; whole < 2; ++whole) { // of p itself if rounding left nothing of the residual
                    float v[2] = {0.f, __int_as_float(INT_MAX)};
                    constexpr int kRace = kDraft ? 1 : 2;
                    for (int e0 = begin; e0 < p.V; e0 += kRace * stride) {
                        const Batch<T, kRace> bx(row, e0, stride, p.V), by(kDraft ? drow : row, e0, stride, kDraft ? p.V : 0);
                        const Batch<float, kRace> bw(noise, e0, stride, p.V);
#pragma unroll
                        for (int i = 0; i < kRace; ++i) {
                            const int e = e0 + i * stride;
                            float x[kPiece], y[kPiece], w[kPiece];
                            if (!bx.get(i, x))
                                break;
                            clean(x);
                            if constexpr (kDraft) {
                                by.get(i, y);
                                clean(y);
                            }
                            bw.get(i, w);
                            if (!whole)
                                for (int j = 0; j < tried; ++j)
                                    leave_out(s.tried[j] - e, x);
                            // p alone says for most that they cannot win
#pragma unroll
                            for (int l = 0; l < kPiece; ++l) {
                                float left = weight(x[l], st.m, k) * inv;
                                if (left > v[0] * w[l]) {
                                    if (kDraft && !whole)
                                        left = fmaf(-taken, weight(y[l], sq.m, k) * inv_q, left);
                                    const float score = left > 0.f ? left / w[l] : 0.f;
                                    if (score > v[0])
                                        v[0] = score, v[1] = __int_as_float(e + l);
                                }
                            }
                        }
                    }
                    reduce(s, turn, v, BestAcross());
                    if (v[0] > 0.f) {
                        token = __float_as_int(v[1]);
                        break;
                    }
                }
            }
            if (token >= 0)
                logit = logit_at(row, token);
        }
        if (writes) {
            p.new_tokens[out0 + count - 1] = token;
            if (p.logprobs && token >= 0)
                p.logprobs[out0 + count - 1] = ((logit - st.m) * k - log2f(st.s)) * kLn2;
        }
        if (accepted < 0)
            break;
        cur = accepted;
        __syncthreads(); // s.child_* and s.tried are written anew
    }
    if (writes)
        p.path_lens[b] = count;
    cluster_sync(); // no block ends while another may still write to it
}

template <typename T, bool kDraft>
cudaError_t launch(const VerifyParams &p, int B, int blocks, cudaStream_t stream)
{
    const auto kernel = verify_kernel<T, kDraft>;
    static std::atomic<bool> configured[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev >= kMaxDevices || !configured[dev].load(std::memory_order_acquire)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess)
            return err;
        if (dev < kMaxDevices)
            configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

} // namespace

cudaError_t launch_verify_tree(const VerifyTreeArgs &a, cudaStream_t stream)
{
    VerifyParams p{a.target, a.draft, a.target_stride, a.draft_stride, a.tokens, a.parents, a.draft_lens, a.temperatures,
                   a.accept, a.noise, a.M, a.A, a.V, a.path, a.path_lens, a.new_tokens, a.logprobs};
    // As many blocks a sequence as all run at once, two an SM, and no more than have a piece
    // for each thread; a power of two. 151936 bf16 logits, 4, 8 and 16 blocks: one sequence
    // 44.2, 30.2, 23.4 us; 64 with draft logits 110.5, 103.5, 151.0 us; 24 of 32003 fp32 logits
    // 32.8, 30.4, 34.6 us. (64 sequences get 4: with 8 half of them start when short paths of
    // the others have ended, which this rule cannot foresee.)
    int blocks = kMaxCluster;
    while (blocks > 1 && (a.B > 2 * a.sm_count / blocks || a.V <= blocks / 2 * kVerifyThreads * kPiece))
        blocks /= 2;
    if (a.f32)
        return a.draft ? launch<float, true>(p, a.B, blocks, stream) : launch<float, false>(p, a.B, blocks, stream);
    return a.draft ? launch<uint16_t, true>(p, a.B, blocks, stream) : launch<uint16_t, false>(p, a.B, blocks, stream);
}

cudaError_t read_flags_verify_tree(unsigned *flags, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_flags_verify, sizeof(unsigned));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_flags_verify, &zero, sizeof(unsigned));
    }
    return err;
}

} // namespace pgqa
