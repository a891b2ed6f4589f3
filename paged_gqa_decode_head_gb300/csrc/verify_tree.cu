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
// a pass over a row, a reduction over the cluster, a handful of scalar tests.
//
// Split: a cluster of blocks per sequence; every thread of it holds the same
// scalars and takes the same turns.
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

// Elements e .. e + 7 of a row of V; -inf past its end. Rows lie anywhere on
// their element's alignment.
template <typename T> __device__ __forceinline__ void load_piece(const T *row, int e, int V, float *x)
{
    const T *at = row + e;
    if (e + kPiece <= V && (reinterpret_cast<uintptr_t>(at) & 15u) == 0) {
        if constexpr (sizeof(T) == 2) {
            unpack8(*reinterpret_cast<const uint4 *>(at), x);
        } else {
            const float4 a = reinterpret_cast<const float4 *>(at)[0], b = reinterpret_cast<const float4 *>(at)[1];
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        }
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            x[j] = usable(x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            x[j] = e + j < V ? logit_at(row, e + j) : -INFINITY;
    }
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^((x - m) k), 0 for a logit of -inf.
__device__ __forceinline__ float weight(float x, float m, float k) { return x == -INFINITY ? 0.f : ex2((x - m) * k); }

// Maximum, its first place, and the sum of weights relative to it.
struct RowStats {
    float m, s;
    int at;
};
__device__ __forceinline__ RowStats join(const RowStats &a, const RowStats &b, float k)
{
    const bool take_b = b.m > a.m || (b.m == a.m && b.at < a.at);
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY)
        return {m, 0.f, a.at < b.at ? a.at : b.at};
    return {m, a.s * weight(a.m, m, k) + b.s * weight(b.m, m, k), take_b ? b.at : a.at};
}

struct VerifySmem {
    float parts[2][kMaxCluster][6]; // a block's result of one reduction, from every block, twice in turn
    float warp_parts[kVerifyThreads / 32][6];
    int tokens[kMaxDrafted], parents[kMaxDrafted];
    float accept[kMaxDrafted], child_p[kMaxDrafted], child_q[kMaxDrafted];
    int tried[kMaxDrafted];
};

// The cluster's reduction: every thread gives N values, `fold` joins two sets (in
// a fixed order), every thread of every block gets the result.
template <int N, typename Fold>
__device__ __forceinline__ void reduce(VerifySmem &s, int &turn, float (&v)[N], Fold fold)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = __shfl_xor_sync(0xFFFFFFFFu, v[i], off);
        // the lower lane's first, so that both lanes form the same sum
        if (lane & off) {
            float t[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                t[i] = v[i], v[i] = o[i], o[i] = t[i];
        }
        fold(v, o);
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            s.warp_parts[warp][i] = v[i];
    }
    __syncthreads();
    const int blocks = cluster_size(), rank = cluster_rank();
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = s.warp_parts[0][i];
        for (int w = 1; w < kVerifyThreads / 32; ++w) {
            float o[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = s.warp_parts[w][i];
            fold(v, o);
        }
        if (lane < blocks) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                store_remote(&s.parts[turn][rank][i], lane, v[i]);
        }
    }
    cluster_sync();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = s.parts[turn][0][i];
    for (int r = 1; r < blocks; ++r) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = s.parts[turn][r][i];
        fold(v, o);
    }
    turn ^= 1;
}

// kDraft: with draft logits.
template <typename T, bool kDraft>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyParams p)
{
    __shared__ VerifySmem s;
    grid_dependency_wait();
    allow_dependent_launch();
    const int tid = threadIdx.x, blocks = cluster_size(), rank = cluster_rank();
    const int b = blockIdx.x / blocks;
    const int first = (rank * kVerifyThreads + tid) * kPiece, stride = blocks * kVerifyThreads * kPiece;
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
    const float k = fminf(kLog2e / (greedy ? 1.f : temperature), FLT_MAX);
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
        const auto scan = [&](const T *r, RowStats &a) {
            for (int e = first; e < p.V; e += stride) {
                float x[kPiece];
                load_piece(r, e, p.V, x);
                float top = x[0];
#pragma unroll
                for (int j = 1; j < kPiece; ++j)
                    top = fmaxf(top, x[j]);
                if (top > a.m) {
                    a.s *= weight(a.m, top, k);
                    a.m = top;
#pragma unroll
                    for (int j = kPiece - 1; j >= 0; --j)
                        a.at = x[j] == top ? e + j : a.at;
                }
                if (top > -INFINITY) {
#pragma unroll
                    for (int j = 0; j < kPiece; ++j)
                        a.s += weight(x[j], a.m, k);
                }
            }
        };
        scan(row, st);
        if constexpr (kDraft)
            scan(drow, sq);
        if constexpr (kDraft) {
            float v[5] = {st.m, st.s, __int_as_float(st.at), sq.m, sq.s};
            reduce(s, turn, v, [&](float (&a)[5], const float (&o)[5]) {
                const RowStats x = join({a[0], a[1], __float_as_int(a[2])}, {o[0], o[1], __float_as_int(o[2])}, k);
                const RowStats y = join({a[3], a[4], 0}, {o[3], o[4], 0}, k);
                a[0] = x.m, a[1] = x.s, a[2] = __int_as_float(x.at), a[3] = y.m, a[4] = y.s;
            });
            st = {v[0], v[1], __float_as_int(v[2])};
            sq = {v[3], v[4], 0};
        } else {
            float v[3] = {st.m, st.s, __int_as_float(st.at)};
            reduce(s, turn, v, [&](float (&a)[3], const float (&o)[3]) {
                const RowStats x = join({a[0], a[1], __float_as_int(a[2])}, {o[0], o[1], __float_as_int(o[2])}, k);
                a[0] = x.m, a[1] = x.s, a[2] = __int_as_float(x.at);
            });
            st = {v[0], v[1], __float_as_int(v[2])};
        }
        const float inv = st.s > 0.f ? 1.f / st.s : 0.f, inv_q = kDraft && sq.s > 0.f ? 1.f / sq.s : 0.f;
        // ---- the children
        int accepted = -1, token = -1, tried = 0;
        float taken = 0.f;            // C
        float mass = 1.f, rest = !kDraft || sq.s > 0.f ? 1.f : 0.f; // S and Q
        if (st.m > -INFINITY && count < p.A) {
            const auto next_child = [&](int i) {
                while (i < n && (s.parents[i] != cur || s.tokens[i] < 0))
                    ++i;
                return i;
            };
            for (int i = next_child(cur + 1); i < n;) {
                const int t = s.tokens[i];
                if (greedy) {
                    if (t == st.at) {
                        accepted = i;
                        break;
                    }
                    i = next_child(i + 1);
                    continue;
                }
                bool again = false;
                for (int j = 0; j < tried; ++j)
                    again = again || s.tried[j] == t;
                const float pt = again ? 0.f : weight(s.child_p[i], st.m, k) * inv;
                const float qt = kDraft && !again ? weight(s.child_q[i], sq.m, k) * inv_q : 0.f;
                const float left = kDraft ? fmaxf(fmaf(-taken, qt, pt), 0.f) : pt;
                const bool given = !kDraft || !(rest > 0.f); // a point mass
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
                i = next_child(i + 1);
                if (i < n) { // the sums that the next child's test needs
                    float v[2] = {0.f, 0.f};
                    for (int e = first; e < p.V; e += stride) {
                        float x[kPiece], y[kPiece];
                        load_piece(row, e, p.V, x);
                        if constexpr (kDraft)
                            load_piece(drow, e, p.V, y);
                        for (int j = 0; j < tried; ++j)
                            if (s.tried[j] / kPiece == e / kPiece) {
#pragma unroll
                                for (int l = 0; l < kPiece; ++l)
                                    if (s.tried[j] % kPiece == l)
                                        x[l] = y[l] = -INFINITY;
                            }
#pragma unroll
                        for (int j = 0; j < kPiece; ++j) {
                            const float pj = weight(x[j], st.m, k) * inv;
                            if constexpr (kDraft) {
                                const float qj = weight(y[j], sq.m, k) * inv_q;
                                v[0] += fmaxf(fmaf(-taken, qj, pj), 0.f);
                                v[1] += qj;
                            } else {
                                v[0] += pj;
                            }
                        }
                    }
                    reduce(s, turn, v, [](float (&a)[2], const float (&o)[2]) { a[0] += o[0], a[1] += o[1]; });
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
                    for (int e = first; e < p.V; e += stride) {
                        float x[kPiece], y[kPiece], w[kPiece];
                        load_piece(row, e, p.V, x);
                        if constexpr (kDraft)
                            load_piece(drow, e, p.V, y);
                        load_piece(noise, e, p.V, w);
                        if (!whole)
                            for (int j = 0; j < tried; ++j)
                                if (s.tried[j] / kPiece == e / kPiece) {
#pragma unroll
                                    for (int l = 0; l < kPiece; ++l)
                                        if (s.tried[j] % kPiece == l)
                                            x[l] = -INFINITY;
                                }
#pragma unroll
                        for (int j = 0; j < kPiece; ++j) {
                            float left = weight(x[j], st.m, k) * inv;
                            if (kDraft && !whole)
                                left = fmaf(-taken, weight(y[j], sq.m, k) * inv_q, left);
                            const float score = left > 0.f ? left / w[j] : 0.f;
                            if (score > v[0])
                                v[0] = score, v[1] = __int_as_float(e + j);
                        }
                    }
                    reduce(s, turn, v, [](float (&a)[2], const float (&o)[2]) {
                        if (o[0] > a[0] || (o[0] == a[0] && __float_as_int(o[1]) < __float_as_int(a[1])))
                            a[0] = o[0], a[1] = o[1];
                    });
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

size_t verify_tree_workspace_bytes(int, int, int, int) { return 0; }

cudaError_t launch_verify_tree(const VerifyTreeArgs &a, cudaStream_t stream)
{
    VerifyParams p{a.target, a.draft, a.target_stride, a.draft_stride, a.tokens, a.parents, a.draft_lens, a.temperatures,
                   a.accept, a.noise, a.M, a.A, a.V, a.path, a.path_lens, a.new_tokens, a.logprobs};
    const int blocks = 8;
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
