// Log probabilities of given tokens, entropy and top alternatives of rows of logits, and the gradient
// (gpt.h, gpt_token_logprobs).
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gpt {

namespace {

constexpr int kThreads = 256;

GPT_DEVINL float ld_act(const bf16* p) {
    return __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(p))));
}
GPT_DEVINL float ld_act(const float* p) { return __ldcg(p); }
GPT_DEVINL void st(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
GPT_DEVINL void st(float* p, float v) { *p = v; }

// Order-preserving key: larger value, larger key; -0 as +0, NaN above every number.
GPT_DEVINL uint32_t order_key(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename T, typename F>
GPT_DEVINL T block_reduce(T v, T* red, F op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kThreads / 32; ++w) v = op(v, red[w]);
    return v;
}

template <typename E>
__global__ void __launch_bounds__(kThreads)
    logprobs_kernel(const E* __restrict__ logits, long long ld, const int64_t* __restrict__ tokens, int V, float inv_t,
                    float* __restrict__ logp, float* __restrict__ entropy, float* __restrict__ lse_out, int k,
                    int64_t* __restrict__ top_ids, float* __restrict__ top_logp, int32_t* status) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float red[kThreads / 32];
    __shared__ unsigned long long red64[kThreads / 32];
    const long long r = blockIdx.x;
    const E* z = logits + r * ld;
    const int tid = threadIdx.x;
    float m = -INFINITY;
    for (int i = tid; i < V; i += kThreads) m = fmaxf(m, ld_act(z + i));
    m = block_reduce(m, red, [](float a, float b) { return fmaxf(a, b); });
    const float m0 = m == -INFINITY ? 0.f : m;
    float s = 0.f, t = 0.f;
    for (int i = tid; i < V; i += kThreads) {
        const float e = (ld_act(z + i) - m0) * inv_t;
        const float p = expf(e);
        s += p;
        t += p > 0.f ? p * e : (p == p ? 0.f : p);
    }
    auto add = [](float a, float b) { return a + b; };
    s = block_reduce(s, red, add);
    t = block_reduce(t, red, add);
    const float ls = logf(s);
    const bool none = m == -INFINITY && s == s;
    const float nan = __int_as_float(0x7fc00000);
    if (tid == 0) {
        if (lse_out) lse_out[r] = none ? -INFINITY : m0 * inv_t + ls;
        if (entropy) entropy[r] = none ? nan : ls - t / s;
        if (logp) {
            const long long tok = __ldcg(tokens + r);
            float v = 0.f;
            if (tok >= 0 && tok < V) v = none ? nan : (ld_act(z + tok) - m0) * inv_t - ls;
            else if (tok != -1) set_status(status, GPT_ERR_INDEX);
            logp[r] = v;
        }
    }
    unsigned long long last = ~0ull;
    for (int j = 0; j < k; ++j) {
        unsigned long long best = 0;
        for (int i = tid; i < V; i += kThreads) {
            const unsigned long long key = static_cast<unsigned long long>(order_key(ld_act(z + i))) << 32 | (0xfffffffeu - i);
            if (key < last && key > best) best = key;
        }
        best = block_reduce(best, red64, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; });
        last = best;
        if (tid == 0) {
            const int id = static_cast<int>(0xfffffffeu - static_cast<uint32_t>(best));
            top_ids[r * k + j] = id;
            top_logp[r * k + j] = none ? nan : (ld_act(z + id) - m0) * inv_t - ls;
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads)
    logprobs_backward_kernel(const E* logits, long long ld, const int64_t* __restrict__ tokens, int V, float inv_t,
                             const float* __restrict__ lse, const float* __restrict__ entropy,
                             const float* __restrict__ dlogp, const float* __restrict__ dentropy, E* dlogits,
                             long long ldd, int32_t* status) {
    griddep_launch_dependents();
    griddep_wait();
    const long long r = blockIdx.x;
    const E* z = logits + r * ld;
    E* d = dlogits + r * ldd;
    long long tok = -1;
    float g = 0.f, h = 0.f, H = 0.f;
    if (dlogp) {
        tok = __ldcg(tokens + r);
        if (tok >= 0 && tok < V) {
            g = __ldcg(dlogp + r);
        } else {
            if (tok != -1 && threadIdx.x == 0) set_status(status, GPT_ERR_INDEX);
            tok = -1;
        }
    }
    if (dentropy) h = __ldcg(dentropy + r), H = __ldcg(entropy + r);
    const float L = __ldcg(lse + r);
    const bool zero = (g == 0.f && h == 0.f) || L == -INFINITY;
    const float bad = L - L;   // NaN for a row with no distribution, 0 otherwise
    for (int i = threadIdx.x; i < V; i += kThreads) {
        float v = 0.f;
        if (!zero) {
            const float lp = fmaxf(ld_act(z + i) * inv_t - L, -1e30f);
            const float p = expf(lp);
            v = -p * (g + h * (lp + H));
            if (i == tok) v += g;
            v = v * inv_t + bad;
        }
        st(d + i, v);
    }
}

}  // namespace

int launch_logprobs(const void* logits, long long ld, const int64_t* tokens, int rows, int V, int dtype,
                    float temperature, float* logp, float* entropy, float* lse, int k, int64_t* top_ids,
                    float* top_logp, int32_t* status, cudaStream_t s) {
    const float inv_t = 1.f / temperature;
    if (dtype == GPT_DTYPE_BF16)
        return launch_overlapped(logprobs_kernel<bf16>, dim3(rows), dim3(kThreads), 0, s,
                                 static_cast<const bf16*>(logits), ld, tokens, V, inv_t, logp, entropy, lse, k, top_ids,
                                 top_logp, status);
    return launch_overlapped(logprobs_kernel<float>, dim3(rows), dim3(kThreads), 0, s,
                             static_cast<const float*>(logits), ld, tokens, V, inv_t, logp, entropy, lse, k, top_ids,
                             top_logp, status);
}

int launch_logprobs_backward(const void* logits, long long ld, const int64_t* tokens, int rows, int V, int dtype,
                             float temperature, const float* lse, const float* entropy, const float* dlogp,
                             const float* dentropy, void* dlogits, long long ldd, int32_t* status, cudaStream_t s) {
    const float inv_t = 1.f / temperature;
    if (dtype == GPT_DTYPE_BF16)
        return launch_overlapped(logprobs_backward_kernel<bf16>, dim3(rows), dim3(kThreads), 0, s,
                                 static_cast<const bf16*>(logits), ld, tokens, V, inv_t, lse, entropy, dlogp, dentropy,
                                 static_cast<bf16*>(dlogits), ldd, status);
    return launch_overlapped(logprobs_backward_kernel<float>, dim3(rows), dim3(kThreads), 0, s,
                             static_cast<const float*>(logits), ld, tokens, V, inv_t, lse, entropy, dlogp, dentropy,
                             static_cast<float*>(dlogits), ldd, status);
}

}  // namespace gpt
