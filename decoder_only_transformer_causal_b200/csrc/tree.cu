// Drafted trees (gpt.h, "drafted trees"): the embedding of the nodes and the acceptance of the path that
// the model confirms.  Their attention is in tree_attention.cu.
#include "internal.h"
#include "tree.cuh"

namespace gpt {

namespace {

GPT_DEVINL float to_f(bf16 v) { return __bfloat162float(v); }
GPT_DEVINL float to_f(float v) { return v; }

// x[b, i, :] = wte[tok] + wpe[lengths[b] + depth(i)], zeros where there is no node.  One node per CTA.
template <typename E>
__global__ void tree_embed_kernel(const E* __restrict__ wte, const E* __restrict__ wpe, const int64_t* __restrict__ tok,
                                  const int* __restrict__ parents, const int* __restrict__ lengths,
                                  float* __restrict__ x, int N, int C, int V, int block_size, int32_t* status) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ int par[kMaxNodes];
    const int b = blockIdx.y, i = blockIdx.x;
    for (int j = threadIdx.x; j < N; j += blockDim.x) par[j] = __ldcg(parents + static_cast<long long>(b) * N + j);
    __syncthreads();
    const unsigned long long see = ancestors(par, i);
    float* row = x + (static_cast<long long>(b) * N + i) * C;
    if (see == 0) {
        for (int c = threadIdx.x; c < C; c += blockDim.x) row[c] = 0.f;
        return;
    }
    long long t = __ldcg(tok + static_cast<long long>(b) * N + i);
    if (t < 0 || t >= V) {
        set_status(status, GPT_ERR_INDEX);
        t = 0;
    }
    int p = clamp_length(__ldcg(lengths + b), block_size, status) + __popcll(see) - 1;
    if (p >= block_size) {
        set_status(status, GPT_ERR_BAD_SHAPE);
        p = block_size - 1;
    }
    for (int c = threadIdx.x; c < C; c += blockDim.x)
        row[c] = to_f(wte[t * C + c]) + to_f(wpe[static_cast<long long>(p) * C + c]);
}

// ---------------------------------------------------------------- acceptance
// A cluster of kAcceptCtas CTAs per sequence.  The first warp of every CTA finds the path (a lane per
// pair of nodes: with M the set of nodes that match their parent's choice, node i is accepted iff
// A(i) is inside M; the path is A of the accepted node with the most ancestors, and its nodes in
// index order run from the root down); then the cluster's warps copy the path's k and v rows of
// every layer, a row at a time with 8 loads of 16 bytes per lane in flight.  All CTAs have read the length before the cluster barrier, so
// lengths_out may be lengths itself.
constexpr int kAcceptCtas = 8;
constexpr int kAcceptThreads = 256;
constexpr int kAcceptLoads = 8;

__global__ void __launch_bounds__(kAcceptThreads)
    tree_accept_kernel(const int* __restrict__ parents, const int64_t* __restrict__ tok,
                       const int64_t* __restrict__ chosen, const int* lengths, int N, int n_layer,
                       const uint8_t* __restrict__ tree_qkv, uint8_t* __restrict__ cache, long long c_bytes, int B,
                       int block_size, int* __restrict__ path, int* __restrict__ n_accepted,
                       int64_t* __restrict__ next_token, int* lengths_out, int32_t* status) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ int par[kMaxNodes], way[kMaxNodes];
    __shared__ int64_t want[kMaxNodes];
    __shared__ int s_n, s_len;
    const int rank = static_cast<int>(cluster_ctarank());
    const int b = blockIdx.x / kAcceptCtas;
    const long long row0 = static_cast<long long>(b) * N;
    const int tid = threadIdx.x;
    if (tid < 32) {
        const int i0 = tid, i1 = tid + 32;
        int64_t t0 = 0, t1 = 0;
        if (i0 < N) par[i0] = __ldcg(parents + row0 + i0), want[i0] = __ldcg(chosen + row0 + i0), t0 = __ldcg(tok + row0 + i0);
        if (i1 < N) par[i1] = __ldcg(parents + row0 + i1), want[i1] = __ldcg(chosen + row0 + i1), t1 = __ldcg(tok + row0 + i1);
        const int raw = __ldcg(lengths + b);
        __syncwarp();
        const unsigned long long a0 = i0 < N ? ancestors(par, i0) : 0, a1 = i1 < N ? ancestors(par, i1) : 0;
        if (rank == 0 && ((i0 < N && a0 == 0 && par[i0] != -2) || (i1 < N && a1 == 0 && par[i1] != -2)))
            set_status(status, GPT_ERR_INDEX);
        const bool m0 = a0 && (par[i0] == -1 || t0 == want[par[i0]]);
        const bool m1 = a1 && (par[i1] == -1 || t1 == want[par[i1]]);
        const unsigned long long M = static_cast<unsigned long long>(__ballot_sync(0xffffffffu, m1)) << 32 |
                                     __ballot_sync(0xffffffffu, m0);
        const unsigned r0 = a0 && (a0 & ~M) == 0 ? __popcll(a0) * 64 + 63 - i0 : 0;
        const unsigned r1 = a1 && (a1 & ~M) == 0 ? __popcll(a1) * 64 + 63 - i1 : 0;
        const unsigned best = __reduce_max_sync(0xffffffffu, r0 > r1 ? r0 : r1);
        const int leaf = 63 - static_cast<int>(best & 63);
        const unsigned long long lo = __shfl_sync(0xffffffffu, a0, leaf & 31), hi = __shfl_sync(0xffffffffu, a1, leaf & 31);
        const unsigned long long A = best ? (leaf < 32 ? lo : hi) : 0;
        const int len = clamp_length(raw, block_size, rank == 0 && tid == 0 ? status : nullptr);
        const int n = min(__popcll(A), block_size - len);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = k ? i1 : i0;
            const int at = __popcll(A & ((1ull << i) - 1));
            if (((A >> i) & 1) && at < n) way[at] = i;
        }
        if (tid == 0) s_n = n, s_len = len;
        __syncwarp();
        if (rank == 0) {
            if (i0 < N) path[row0 + i0] = i0 < n ? way[i0] : -1;
            if (i1 < N) path[row0 + i1] = i1 < n ? way[i1] : -1;
            if (tid == 0) {
                n_accepted[b] = n;
                next_token[b] = n ? want[way[n - 1]] : -1;
            }
        }
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int n = s_n, len = s_len;
    const int units = static_cast<int>(2 * c_bytes / 16);   // of a row's k and v
    const int warps = kAcceptCtas * kAcceptThreads / 32, lane = tid & 31;
    for (int row = rank * (kAcceptThreads / 32) + (tid >> 5); row < n_layer * n; row += warps) {
        const int l = row / n, j = row - l * n;
        const uint4* src = reinterpret_cast<const uint4*>(
            tree_qkv + ((static_cast<long long>(l) * B + b) * N + way[j]) * 3 * c_bytes + c_bytes);
        uint4* dst = reinterpret_cast<uint4*>(cache + ((static_cast<long long>(l) * B + b) * block_size + len + j) * 2 * c_bytes);
        for (int u0 = lane; u0 < units; u0 += 32 * kAcceptLoads) {
            uint4 w[kAcceptLoads];
#pragma unroll
            for (int x = 0; x < kAcceptLoads; ++x)
                if (u0 + 32 * x < units) w[x] = __ldcg(src + u0 + 32 * x);
#pragma unroll
            for (int x = 0; x < kAcceptLoads; ++x)
                if (u0 + 32 * x < units) dst[u0 + 32 * x] = w[x];
        }
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) lengths_out[b] = len + n;
}

}  // namespace

int launch_tree_embed(const void* wte, const void* wpe, const int64_t* tok, const int* parents, const int* lengths,
                      float* x, int B, int N, int C, int V, int block_size, int dtype, int32_t* status,
                      cudaStream_t s) {
    const dim3 grid(N, B), block(128);
    if (dtype == GPT_DTYPE_BF16)
        return launch_overlapped(tree_embed_kernel<bf16>, grid, block, 0, s, static_cast<const bf16*>(wte),
                                 static_cast<const bf16*>(wpe), tok, parents, lengths, x, N, C, V, block_size, status);
    return launch_overlapped(tree_embed_kernel<float>, grid, block, 0, s, static_cast<const float*>(wte),
                             static_cast<const float*>(wpe), tok, parents, lengths, x, N, C, V, block_size, status);
}

int launch_tree_accept(const int* parents, const int64_t* tok, const int64_t* chosen, const int* lengths, int B, int N,
                       int n_layer, const void* tree_qkv, void* cache, long long c_bytes, int block_size, int* path,
                       int* n_accepted, int64_t* next_token, int* lengths_out, int32_t* status, cudaStream_t s) {
    return launch_overlapped_cluster(tree_accept_kernel, kAcceptCtas, dim3(B * kAcceptCtas), dim3(kAcceptThreads), 0, s,
                                     parents, tok, chosen, lengths, N, n_layer, static_cast<const uint8_t*>(tree_qkv),
                                     static_cast<uint8_t*>(cache), c_bytes, B, block_size, path, n_accepted, next_token,
                                     lengths_out, status);
}

}  // namespace gpt
