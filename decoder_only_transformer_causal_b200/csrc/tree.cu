// Drafted trees (gpt.h, "drafted trees"): attention of up to 64 candidate tokens per sequence over a
// key/value cache and their ancestors, the embedding of the nodes, and the acceptance of the path
// that the model confirms.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gpt {

namespace {

constexpr int kMaxNodes = GPT_TREE_MAX_NODES;

GPT_DEVINL float to_f(bf16 v) { return __bfloat162float(v); }
GPT_DEVINL float to_f(float v) { return v; }
template <typename E> GPT_DEVINL E from_f(float v);
template <> GPT_DEVINL bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }
template <> GPT_DEVINL float from_f<float>(float v) { return v; }
GPT_DEVINL float ld_act(const bf16* p) {
    return __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(p))));
}
GPT_DEVINL float ld_act(const float* p) { return __ldcg(p); }

// The set A(i) (node i and its ancestors) as a bit mask, 0 for no node.  par: the sequence's parents
// in shared memory.  A parent lies below its child, so the walk ends after at most i steps.
GPT_DEVINL unsigned long long ancestors(const int* par, int i) {
    unsigned long long m = 0;
    for (int j = i;;) {
        m |= 1ull << j;
        const int p = par[j];
        if (p == -1) return m;
        if (p < 0 || p >= j) return 0;
        j = p;
    }
}

GPT_DEVINL int clamp_length(int len, int block_size, int32_t* status) {
    if (len >= 0 && len <= block_size) return len;
    set_status(status, GPT_ERR_BAD_SHAPE);
    return len < 0 ? 0 : block_size;
}

// One node and head per CTA: scores of 128 keys at a time (a key per thread), an online softmax, and
// p.v with a dimension per thread.
template <typename E>
__global__ void __launch_bounds__(128)
    tree_attention_kernel(const E* __restrict__ qkv, const E* __restrict__ kv, const int* __restrict__ lengths,
                          const int* __restrict__ parents, E* __restrict__ y, int N, int nh, int hs, int block_size,
                          float scale_log2, int32_t* status) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float qs[128], ps[128], red[4];
    __shared__ int par[kMaxNodes];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i = blockIdx.y, b = blockIdx.x / nh, h = blockIdx.x % nh;
    const long long C = static_cast<long long>(nh) * hs;
    const E* node = qkv + static_cast<long long>(b) * N * 3 * C + h * hs;
    const E* cache = kv + static_cast<long long>(b) * block_size * 2 * C + h * hs;
    if (tid < N) par[tid] = __ldcg(parents + static_cast<long long>(b) * N + tid);
    if (tid < hs) qs[tid] = ld_act(node + i * 3 * C + tid);
    __syncthreads();
    const unsigned long long see = ancestors(par, i);
    E* out = y + (static_cast<long long>(b) * N + i) * C + h * hs;
    if (see == 0) {
        if (tid == 0 && par[i] != -2) set_status(status, GPT_ERR_INDEX);
        if (tid < hs) out[tid] = from_f<E>(0.f);
        return;
    }
    const int len = clamp_length(__ldcg(lengths + b), block_size, status);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int t0 = 0; t0 < len + N; t0 += 128) {
        const int t = t0 + tid;
        const bool live = t < len || (t < len + N && ((see >> (t - len)) & 1));
        float s = -INFINITY;
        if (live) {
            const E* k = t < len ? cache + t * 2 * C : node + (t - len) * 3 * C + C;
            float acc = 0.f;
            for (int d = 0; d < hs; ++d) acc = fmaf(qs[d], ld_act(k + d), acc);
            s = acc * scale_log2;
        }
        float mx = s;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        __syncthreads();
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float p = live ? exp2f(s - mn) : 0.f;
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
        m = mn;
        ps[tid] = p;
        float sum = p;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        __syncthreads();
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        l = l * f + ((red[0] + red[1]) + (red[2] + red[3]));
        o *= f;
        if (tid < hs)
            for (int j = 0; j < 128; ++j) {
                const int tj = t0 + j;
                if (!(tj < len || (tj < len + N && ((see >> (tj - len)) & 1)))) continue;
                const E* v = tj < len ? cache + tj * 2 * C + C : node + (tj - len) * 3 * C + 2 * C;
                o = fmaf(ps[j], ld_act(v + tid), o);
            }
    }
    if (tid < hs) out[tid] = from_f<E>(o / l);
}

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
// index order run from the root down); then the cluster's threads copy the path's k and v rows of
// every layer, 16 bytes each.  All CTAs have read the length before the cluster barrier, so
// lengths_out may be lengths itself.
constexpr int kAcceptCtas = 8;
constexpr int kAcceptThreads = 256;

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
    const int per_row = static_cast<int>(2 * c_bytes / 16);
    const int total = n_layer * n * per_row;
    for (int u = rank * kAcceptThreads + tid; u < total; u += kAcceptCtas * kAcceptThreads) {
        const int row = u / per_row, off = (u % per_row) * 16;
        const int l = row / n, j = row % n;
        const uint8_t* src = tree_qkv + ((static_cast<long long>(l) * B + b) * N + way[j]) * 3 * c_bytes + c_bytes + off;
        uint8_t* dst = cache + ((static_cast<long long>(l) * B + b) * block_size + len + j) * 2 * c_bytes + off;
        *reinterpret_cast<uint4*>(dst) = __ldcg(reinterpret_cast<const uint4*>(src));
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) lengths_out[b] = len + n;
}

}  // namespace

int launch_tree_attention(int dtype, const void* qkv, const void* kv, const int* lengths, const int* parents, void* y,
                          int B, int N, int nh, int hs, int block_size, int32_t* status, cudaStream_t s) {
    const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hs));
    const dim3 grid(B * nh, N), block(128);
    if (dtype == GPT_DTYPE_BF16)
        return launch_overlapped(tree_attention_kernel<bf16>, grid, block, 0, s, static_cast<const bf16*>(qkv),
                                 static_cast<const bf16*>(kv), lengths, parents, static_cast<bf16*>(y), N, nh, hs,
                                 block_size, scale_log2, status);
    return launch_overlapped(tree_attention_kernel<float>, grid, block, 0, s, static_cast<const float*>(qkv),
                             static_cast<const float*>(kv), lengths, parents, static_cast<float*>(y), N, nh, hs,
                             block_size, scale_log2, status);
}

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
