// Log probabilities of given tokens, entropy and top alternatives of rows of logits, and the gradient
// (gpt.h, gpt_token_logprobs).
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace gpt {

namespace {

constexpr int kThreads = 256;
constexpr int kUnrollLog2 = 2;
constexpr int kUnroll = 1 << kUnrollLog2;   // 16-byte loads in flight per thread
constexpr int kMaxCluster = 4;
// Places for the values at or above a part's top-k bound, and for the steps that reach it.
constexpr uint32_t places(int threads) { return threads < 64 ? 256 : 512; }   // (candidates fit where the slots were)
constexpr int kSlots = 32;          // places per thread for the maxima of its steps (of kUnroll loads)

template <typename E> constexpr int kVec = 16 / sizeof(E);

GPT_DEVINL float ld_act(const bf16* p) {
    return __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(p))));
}
GPT_DEVINL float ld_act(const float* p) { return __ldcg(p); }
GPT_DEVINL void st(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
GPT_DEVINL void st(float* p, float v) { *p = v; }

// Maximum that keeps NaN.
GPT_DEVINL float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
GPT_DEVINL uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Order-preserving key: larger value, larger key; -0 as +0, NaN above every number; key_value undoes it.
GPT_DEVINL uint32_t order_key(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
GPT_DEVINL float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k); }

// The key's upper half, and a value cut to its upper half (the key of the one is that half of the other's).
GPT_DEVINL uint32_t key16(float f) { return order_key(f) >> 16; }
GPT_DEVINL float slot_value(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }

// A value and its column in one number that orders as the top list does: by value, equal values by
// index.  0 stands for no entry (the lowest key is that of -inf, above 0).
GPT_DEVINL unsigned long long entry(float z, uint32_t col) {
    return static_cast<unsigned long long>(order_key(z)) << 32 | (0xffffffffu - col);
}
GPT_DEVINL uint32_t entry_col(unsigned long long e) { return 0xffffffffu - static_cast<uint32_t>(e); }

template <int NT, typename T, typename F>
GPT_DEVINL T block_reduce(T v, T* red, F op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) v = op(v, red[w]);
    return v;
}

// The part of a row that one thread of the row's CTAs reads: the 16-byte units first, first + stride, ...
// and at most one of the elements before the first and behind the last whole unit.
template <typename E>
struct Slice {
    const E* z;
    uint32_t head, units, ends;   // elements before the first unit, units, elements outside units
    uint32_t stride;

    GPT_DEVINL Slice(const E* row, uint32_t V, uint32_t stride_) : z(row), stride(stride_) {
        const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15) / sizeof(E);
        head = mis ? kVec<E> - mis : 0;
        if (head > V) head = V;
        units = (V - head) / kVec<E>;
        ends = V - units * kVec<E>;
    }
    GPT_DEVINL uint32_t end_col(uint32_t i) const { return i < head ? i : i + units * kVec<E>; }
    GPT_DEVINL uint32_t unit_col(uint32_t u) const { return head + u * kVec<E>; }
    // f(value, column) over the elements of thread `first`.
    template <typename F>
    GPT_DEVINL void each(uint32_t first, F f) const {
        uint32_t u = first;
        for (; u + 3 * stride < units; u += 4 * stride) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldcg(reinterpret_cast<const uint4*>(z + unit_col(u + i * stride)));
#pragma unroll
            for (int i = 0; i < 4; ++i) values(w[i], unit_col(u + i * stride), f);
        }
        for (; u < units; u += stride) unit(u, f);
        if (first < ends) f(ld_act(z + end_col(first)), end_col(first));
    }
    template <typename F>
    GPT_DEVINL void unit(uint32_t u, F f) const {
        values(__ldcg(reinterpret_cast<const uint4*>(z + unit_col(u))), unit_col(u), f);
    }
    template <typename F>
    GPT_DEVINL static void values(const uint4& w, uint32_t col, F f) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sizeof(E) == 4) {
                f(__uint_as_float(x[i]), col + i);
            } else {
                f(__uint_as_float(x[i] << 16), col + 2 * i);
                f(__uint_as_float(x[i] & 0xffff0000u), col + 2 * i + 1);
            }
        }
    }
};

// Sums relative to a reference value: with e = z c - ref, c = log2(e) / T and ref = rn(c max z) (taken as
// it is, so that its rounding cancels), the sums of 2^e and of 2^e e.  A thread's running form:
struct Running {
    float m, ref;
    uint64_t s, t;   // two partial sums each
    GPT_DEVINL void raise(float to, float c) {
        m = max_nan(m, to);
        const float next = m * c, d = ref - next, f = exp2_approx(d);
        const uint64_t ff = f2_pack(f, f);
        t = f2_mul(f2_fma(s, f2_pack(d, d), t), ff);
        s = f2_mul(s, ff);
        ref = next;
    }
    GPT_DEVINL void add2(float a, float b, uint64_t cc, uint64_t neg_ref) {
        const uint64_t e = f2_fma(f2_pack(a, b), cc, neg_ref);
        float e0, e1;
        f2_unpack(e, e0, e1);
        const uint64_t p = f2_pack(exp2_approx(e0), exp2_approx(e1));
        s = f2_add(s, p);
        t = f2_fma(p, e, t);
    }
};

GPT_DEVINL float take(Running& a, const uint4 (&w)[kUnroll], float floor_z, uint32_t floor2, float c, const bf16*) {
    uint32_t x[4 * kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) x[4 * i] = w[i].x, x[4 * i + 1] = w[i].y, x[4 * i + 2] = w[i].z, x[4 * i + 3] = w[i].w;
    uint32_t mx = floor2;
#pragma unroll
    for (int i = 0; i < 4 * kUnroll; ++i) {
        x[i] = max2_nan(x[i], floor2);
        mx = max2_nan(mx, x[i]);
    }
    const float top = max_nan(__uint_as_float(mx << 16), __uint_as_float(mx & 0xffff0000u));
    a.raise(top, c);
    const uint64_t cc = f2_pack(c, c), ref = f2_pack(-a.ref, -a.ref);
#pragma unroll
    for (int i = 0; i < 4 * kUnroll; ++i)
        a.add2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u), cc, ref);
    return top;
}
GPT_DEVINL float take(Running& a, const uint4 (&w)[kUnroll], float floor_z, uint32_t floor2, float c, const float*) {
    float x[4 * kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        x[4 * i] = __uint_as_float(w[i].x), x[4 * i + 1] = __uint_as_float(w[i].y);
        x[4 * i + 2] = __uint_as_float(w[i].z), x[4 * i + 3] = __uint_as_float(w[i].w);
    }
    float mx = floor_z;
#pragma unroll
    for (int i = 0; i < 4 * kUnroll; ++i) {
        x[i] = max_nan(x[i], floor_z);
        mx = max_nan(mx, x[i]);
    }
    a.raise(mx, c);
    const uint64_t cc = f2_pack(c, c), ref = f2_pack(-a.ref, -a.ref);
#pragma unroll
    for (int i = 0; i < 4 * kUnroll; i += 2) a.add2(x[i], x[i + 1], cc, ref);
    return mx;
}

struct Part {   // one CTA's share of a row: reference, sums, and whether any value is above -inf
    double ref;
    float s, t;
    int any;
};

struct ScoreArgs {
    long long ld;
    const int64_t* tokens;
    uint32_t V;
    int cluster, threads;
    float c, floor_z;        // log2(e) / T; the value that stands for everything at or below it
    uint32_t floor2;         // floor_z as a pair of bf16
    float *logp, *entropy, *lse;
    int k;
    int slot_shift;      // 2^slot_shift steps of a thread share a slot
    int64_t* top_ids;
    float* top_logp;
    int32_t* status;
};

// A row is read once from HBM by a cluster of 1, 2 or 4 CTAs, 16 bytes per load.  Many rows: 32, 64 or 128
// threads each (the launch has the rule), the SM's registers full of rows: with 256 threads the ends of the rows
// (reductions, the list) left the memory idle (228 us against 206 without a list); two steps in flight per thread
// cost a quarter of the threads and were slower (313 against 265 us with 20 entries), as was asking L2 for the
// next row (325 against 228).
//
// Sums.  Each thread keeps a running maximum, raised once per 64 bytes, and the sums relative to it; the
// threads' and then the CTAs' sums are joined in a fixed order.  Values are first raised to floor_z, so
// that -inf needs no test in the loop (2^e is 0 and e finite); where that could show (a maximum that is
// not finite or not far above floor_z: NaN, +-inf, rows of the type's lowest value, extreme temperatures)
// the CTA repeats its part from L2 with a maximum first and 64-bit arguments.
//
// Top list.  The k-th largest of the CTA's thread maxima is a bound that at least k of its values
// reach, and hardly more do: only the steps whose maximum reaches it (about k of them) are read
// again, from L2.  More such values than places (long ties, masked rows with fewer than k tokens left): passes
// over the row that halve the range of values in question, until few are left or all are equal, of which the
// first count.  12288 rows x 50257 bf16, in a burst / back to back (power cap): without a list 192 / 207 us (6.4 TB/s),
// one entry 205 / 221, 20 entries 229 / 240, 32 entries 248 / 250.  The values' ranks among the candidates, and across
// CTAs by binary search in the others' lists, are their places in the list.
template <typename E, int NT>
__global__ void __launch_bounds__(NT, NT > 128 ? 4 : NT == 32 ? 32 : (sizeof(E) == 2 ? 9 : 8) * 128 / NT)
logprobs_kernel(const E* __restrict__ logits, const ScoreArgs a) {
    constexpr uint32_t kPlaces = places(NT);
    griddep_launch_dependents();
    __shared__ float red[NT / 32], red_s[NT / 32], red_t[NT / 32];
    __shared__ uint4 crowd[NT / 32];
    // the candidates lie where the slots were: shared memory is taken from the L1 that the loads in flight need
    // (9000 rows x 9001 bf16, 20 entries: 57.0 us with 10.9 KB per row of 64 threads, 52.5 with 6.8)
    __shared__ __align__(16) uint16_t slots[kSlots][NT];
    static_assert(sizeof(slots) >= kPlaces * sizeof(unsigned long long));
    unsigned long long* cand = reinterpret_cast<unsigned long long*>(slots);
    __shared__ unsigned long long lists[NT < 256 ? 1 : kMaxCluster][GPT_TOP_MAX];
    __shared__ Part parts[kMaxCluster];
    __shared__ uint16_t keys[NT];
    __shared__ uint32_t hits[kPlaces];
    __shared__ uint32_t s_bound, s_hits, s_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = NT < 256 ? 1 : a.cluster;   // (known to the compiler for CTAs that are alone)
    const int rank = ncta > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    if (ncta > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const long long r = blockIdx.x / ncta;
    const Slice<E> row(logits + r * a.ld, a.V, ncta * NT);
    const uint32_t first = rank * NT + tid;
    griddep_wait();
    // what is needed at the end travels with the row: the token's logit, the element outside the units
    long long tok = -1;
    if (a.logp && first == 0) tok = __ldcg(a.tokens + r);
    const float z_end = first < row.ends ? ld_act(row.z + row.end_col(first)) : 0.f;
    float z_tok = 0.f;
    if (tok >= 0 && tok < a.V) z_tok = ld_act(row.z + tok);
    Running run = {a.floor_z, a.floor_z * a.c, 0, 0};
    if (a.k > 0 && a.slot_shift)
        for (int j = 0; j < kSlots; ++j) slots[j][tid] = static_cast<uint16_t>(a.floor2);
    const uint32_t mine = first < row.units ? (row.units - first - 1) / row.stride + 1 : 0;   // this thread's units
    uint32_t step = 0;
    auto finish_step = [&](const uint4(&w)[kUnroll]) {
        const float top = take(run, w, a.floor_z, a.floor2, a.c, row.z);
        if (a.k > 0) {
            uint16_t& slot = slots[step >> a.slot_shift][tid];
            if (a.slot_shift == 0 || key16(top) > key16(slot_value(slot))) slot = static_cast<uint16_t>(__float_as_uint(top) >> 16);
        }
        ++step;
    };
    const uint4* units = reinterpret_cast<const uint4*>(row.z + row.head) + first;
    for (uint32_t n = mine / kUnroll; n > 0; --n, units += kUnroll * row.stride) {
        uint4 w[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) w[i] = __ldcg(units + i * row.stride);
        finish_step(w);
    }
    if (mine % kUnroll) {
        const uint32_t f = sizeof(E) == 4 ? __float_as_uint(a.floor_z) : a.floor2;
        uint4 w[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) w[i] = i < mine % kUnroll ? __ldcg(units + i * row.stride) : make_uint4(f, f, f, f);
        finish_step(w);
    }
    if (first < row.ends) {
        const float z = max_nan(z_end, a.floor_z);
        run.raise(z, a.c);
        const float e = fmaf(z, a.c, -run.ref), p = exp2_approx(e);
        run.s = f2_add(run.s, f2_pack(p, 0.f));
        run.t = f2_fma(f2_pack(p, 0.f), f2_pack(e, 0.f), run.t);
    }

    const uint32_t my_key = key16(run.m);
    keys[tid] = static_cast<uint16_t>(my_key);
    float m = run.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[warp] = m;
    if (tid == 0) s_count = 0, s_hits = 0;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) m = max_nan(m, red[w]);
    double ref = m * a.c;
    float s, t;
    {
        const float d = run.ref - m * a.c, f = exp2_approx(d);
        float s0, s1, t0, t1;
        f2_unpack(run.s, s0, s1);
        f2_unpack(run.t, t0, t1);
        s0 += s1;
        s = s0 * f;
        t = (t0 + t1 + s0 * d) * f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            t += __shfl_xor_sync(0xffffffffu, t, o);
        }
        if (lane == 0) red_s[warp] = s, red_t[warp] = t;
    }
    if (a.k > 0 && warp == 0) {
        // the upper 16 bits of the k-th largest key, two bits at a time (three counts of at most 256 in one
        // sum): mostly it lies within 255 of the largest, else anywhere; 0 (every value) when fewer than k
        // threads hold a value above floor_z
        uint32_t mine[NT / 32];
#pragma unroll
        for (int j = 0; j < NT / 32; ++j) mine[j] = keys[j * 32 + lane];
        const uint32_t k = a.k, top = key16(m);
        uint32_t near = top > 255 ? top - 255 : 0;
        int reach = 0;
#pragma unroll
        for (int j = 0; j < NT / 32; ++j) reach += mine[j] >= near;
        int bit = 6;
        if (static_cast<uint32_t>(__reduce_add_sync(0xffffffffu, reach)) < k) near = 0, bit = 14;
        uint32_t bound = near;
        for (; bit >= 0; bit -= 2) {
            const uint32_t b1 = bound + (1u << bit), b2 = bound + (2u << bit), b3 = bound + (3u << bit);
            uint32_t above = 0;
#pragma unroll
            for (int j = 0; j < NT / 32; ++j)
                above += (mine[j] >= b1 ? 1u : 0u) + (mine[j] >= b2 ? 1u << 10 : 0u) + (mine[j] >= b3 ? 1u << 20 : 0u);
            above = __reduce_add_sync(0xffffffffu, above);
            bound = above >> 20 >= k ? b3 : (above >> 10 & 1023u) >= k ? b2 : (above & 1023u) >= k ? b1 : bound;
        }
        if (lane == 0) s_bound = bound <= key16(a.floor_z) ? 0 : bound;
    }
    __syncthreads();
    s = red_s[0], t = red_t[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) s += red_s[w], t += red_t[w];
    int any = 1;
    // floor_z and what it stands for are at least 2^200 times less likely than the maximum, and nothing
    // overflows; else once more
    if (!(fabsf(m) < 1e30f && fabsf(m) * a.c < 1e30f && (m - a.floor_z) * a.c > 200.f)) {
        float mt = -INFINITY;
        row.each(first, [&](float z, uint32_t) { mt = fmaxf(mt, z); });
        m = block_reduce<NT>(mt, red, [](float x, float y) { return fmaxf(x, y); });
        any = m > -INFINITY;
        ref = any ? static_cast<double>(m) * a.c : 0.;   // (may pass the range of 32 bits)
        float st = 0.f, tt = 0.f;
        row.each(first, [&](float z, uint32_t) {
            const float e = static_cast<float>(static_cast<double>(z) * a.c - ref), p = exp2f(e);
            st += p;
            tt += p == 0.f ? 0.f : p * e;
        });
        auto add = [](float x, float y) { return x + y; };
        s = block_reduce<NT>(st, red, add);
        t = block_reduce<NT>(tt, red, add);
    }

    unsigned long long* list = lists[rank];
    if (a.k > 0) {
        const uint32_t bound16 = s_bound;
        const float bound = bound16 == 0 ? -INFINITY : bound16 == 0xffffu ? INFINITY : key_value(bound16 << 16);
        uint32_t end = 0;   // this thread's element outside the units reaches the bound
        {   // this thread's steps that do (at most 32 slots)
            uint32_t in = 0;
            if (my_key >= bound16) {
                const uint32_t n = (step + (1u << a.slot_shift) - 1) >> a.slot_shift;
#pragma unroll 8
                for (uint32_t j = 0; j < n; ++j) in |= static_cast<uint32_t>(!(slot_value(slots[j][tid]) < bound)) << j;
                end = first < row.ends && !(z_end < bound);
            }
            uint32_t at = in ? atomicAdd(&s_hits, static_cast<uint32_t>(__popc(in))) : 0;
            for (; in; in &= in - 1, ++at)
                if (at < kPlaces) hits[at] = static_cast<uint32_t>(__ffs(in) - 1) << 16 | tid;
        }
        __syncthreads();   // (the slots are done with)
        if (end) {
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < kPlaces) cand[at] = entry(z_end, row.end_col(first));
        }
        const uint32_t n_hits = s_hits, each_log2 = kUnrollLog2 + a.slot_shift;
        if (n_hits <= kPlaces)
            for (uint32_t i0 = warp * 32; i0 < n_hits << each_log2; i0 += 4 * NT) {   // four units per lane at a time
                uint4 w[4];
                uint32_t cols[4], in[4], n = 0;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t i = i0 + x * NT + lane;
                    cols[x] = 0xffffffffu;
                    if (i < n_hits << each_log2) {
                        const uint32_t hit = hits[i >> each_log2];
                        const uint32_t u = rank * NT + (hit & 0xffffu) + (((hit >> 16) << each_log2) + (i & ((1u << each_log2) - 1))) * row.stride;
                        if (u < row.units) {
                            cols[x] = row.unit_col(u);
                            w[x] = __ldcg(reinterpret_cast<const uint4*>(row.z + cols[x]));
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    in[x] = 0;
                    if (cols[x] != 0xffffffffu) {
                        uint32_t e = 0;
                        row.values(w[x], 0, [&](float z, uint32_t) { in[x] |= static_cast<uint32_t>(!(z < bound)) << e++; });
                    }
                    n += __popc(in[x]);
                }
                if (n == 0) continue;
                uint32_t at = atomicAdd(&s_count, n);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    for (; in[x]; in[x] &= in[x] - 1, ++at) {
                        const uint32_t e = __ffs(in[x]) - 1, pos = sizeof(E) == 4 ? e : e >> 1;
                        const uint32_t bits = pos == 0 ? w[x].x : pos == 1 ? w[x].y : pos == 2 ? w[x].z : w[x].w;
                        const float z = __uint_as_float(sizeof(E) == 4 ? bits : (e & 1) ? bits & 0xffff0000u : bits << 16);
                        if (at < kPlaces) cand[at] = entry(z, cols[x] + e);
                    }
            }
        __syncthreads();
        uint32_t count = s_count;
        if (count > kPlaces || n_hits > kPlaces) {
            // The crowd is cut down by passes that halve the keys in question, [lo, hi]: at least k values reach lo
            // and n_above < k lie above hi.  Each pass also narrows the range to keys that occur, so that one
            // value many times over (a masked row's -inf, a uniform row) is known after the first.  1000 rows x 50257
            // bf16, 20 entries: 18 tokens left 125 us, a uniform row 75 (64 passes, one per bit of value and
            // index, took 2130), against 29 for a row that needs none of this.
            uint32_t lo = bound16 << 16, hi = 0xffffffffu, n_above = 0;
            uint32_t mid = bound16 == 0 ? 0x00800000u : lo + 0x10000u;   // (first: the bound's own keys, or -inf, against those above)
            if (bound16 == 0xffffu) lo = hi;
            bool few = false;
            while (lo < hi) {
                uint32_t reach = 0, lowest = 0, below = 0, floor = 0;   // (the minima as maxima of ~key)
                row.each(first, [&](float z, uint32_t) {
                    const uint32_t key = order_key(z);
                    if (key >= mid) {
                        ++reach;
                        lowest = max(lowest, ~key);
                    } else if (key >= lo) {
                        below = max(below, key);
                        floor = max(floor, ~key);
                    }
                });
                reach = __reduce_add_sync(0xffffffffu, reach);
                lowest = __reduce_max_sync(0xffffffffu, lowest);
                below = __reduce_max_sync(0xffffffffu, below);
                floor = __reduce_max_sync(0xffffffffu, floor);
                __syncthreads();
                if (lane == 0) crowd[warp] = make_uint4(reach, lowest, below, floor);
                __syncthreads();
                uint4 c = crowd[0];
#pragma unroll
                for (int w = 1; w < NT / 32; ++w) {
                    const uint4 o = crowd[w];
                    c = make_uint4(c.x + o.x, max(c.y, o.y), max(c.z, o.z), max(c.w, o.w));
                }
                if (c.x >= static_cast<uint32_t>(a.k)) {
                    lo = ~c.y;
                    few = c.x <= kPlaces;
                    if (few) break;
                } else {
                    n_above = c.x, hi = c.z, lo = ~c.w;
                }
                mid = lo + (hi - lo) / 2 + 1;
            }
            // the values above, in any order; of those equal to lo the first in the order of the columns
            __syncthreads();
            if (tid == 0) s_count = 0;
            __syncthreads();
            if (few || n_above)
                row.each(first, [&](float z, uint32_t col) {
                    const uint32_t key = order_key(z);
                    if (few ? key >= lo : key > lo) cand[atomicAdd(&s_count, 1u)] = entry(z, col);
                });
            if (!few && first < row.ends && order_key(z_end) == lo) cand[atomicAdd(&s_count, 1u)] = entry(z_end, row.end_col(first));
            __syncthreads();
            count = s_count;
            const uint32_t need = few ? 0 : a.k - n_above;
            uint32_t got = 0;
            for (uint32_t u0 = rank * NT; u0 < row.units && got < need; u0 += row.stride) {
                uint4 w = {};
                uint32_t in = 0;
                if (u0 + tid < row.units) {
                    w = __ldcg(reinterpret_cast<const uint4*>(row.z + row.unit_col(u0 + tid)));
                    row.values(w, 0, [&](float z, uint32_t e) { in |= static_cast<uint32_t>(order_key(z) == lo) << e; });
                }
                uint32_t at = __popc(in);   // up to and with this lane's
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t before = __shfl_up_sync(0xffffffffu, at, o);
                    if (lane >= o) at += before;
                }
                __syncthreads();
                if (lane == 31) crowd[warp].x = at;
                __syncthreads();
                at += got - __popc(in);
#pragma unroll
                for (int x = 0; x < NT / 32; ++x) {
                    if (x < warp) at += crowd[x].x;
                    got += crowd[x].x;
                }
                for (; in && at < need; in &= in - 1, ++at)
                    cand[count + at] = static_cast<unsigned long long>(lo) << 32 | (0xffffffffu - (row.unit_col(u0 + tid) + __ffs(in) - 1));
            }
            count += min(got, need);
        }
        // places by counting
        const uint32_t padded = (count + 7) & ~7u;   // (at most kPlaces)
        if (tid < static_cast<int>(padded - count)) cand[count + tid] = 0;
        __syncthreads();
        for (uint32_t i = tid; i < count; i += NT) {
            const unsigned long long e = cand[i];
            int place = 0;
            for (uint32_t j = 0; j < padded; j += 8) {
                ulonglong2 c[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) c[x] = *reinterpret_cast<const ulonglong2*>(&cand[j + 2 * x]);
#pragma unroll
                for (int x = 0; x < 4; ++x) place += (c[x].x > e) + (c[x].y > e);
            }
            if (place < a.k) list[place] = e;
        }
        for (int i = tid; i < a.k; i += NT)
            if (i >= static_cast<int>(count)) list[i] = 0;   // a part shorter than k
        __syncthreads();
    }
    if (ncta > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA has started
        if (rank != 0) {
            if (tid < a.k) st_cluster_u64(map_to_rank(&list[tid], 0), list[tid]);
            if (tid == 0) {
                st_cluster_u64(map_to_rank(&parts[rank].ref, 0), __double_as_longlong(ref));
                st_cluster_u32(map_to_rank(&parts[rank].s, 0), __float_as_uint(s));
                st_cluster_u32(map_to_rank(&parts[rank].t, 0), __float_as_uint(t));
                st_cluster_u32(map_to_rank(&parts[rank].any, 0), any);
            }
        }
        __syncwarp();
        cluster_sync();
        if (rank != 0) return;
        // the parts joined in the order of their ranks, relative to the largest reference; a part with
        // nothing above -inf has sums of 0 (or NaN)
        double top = any ? ref : -INFINITY;
        for (int q = 1; q < ncta; ++q)
            if (parts[q].any) top = any ? fmax(top, parts[q].ref) : parts[q].ref, any = 1;
        float ss = 0.f, tt = 0.f;
        for (int q = 0; q < ncta; ++q) {
            const float sq = q ? parts[q].s : s, tq = q ? parts[q].t : t;
            const double rq = q ? parts[q].ref : ref;
            if (sq == 0.f) continue;
            const float d = rq == top ? 0.f : static_cast<float>(rq - top), f = exp2f(d);
            ss += sq * f;
            if (f != 0.f) tt += (tq + sq * d) * f;
        }
        s = ss, t = tt, ref = any ? top : 0.;
    }

    // ---- the first CTA: the row's outputs
    const bool none = !any && s == s;
    const double ln2 = 0.6931471805599453, log2_s = log2f(s);
    const float nan = __int_as_float(0x7fc00000);
    auto logprob = [&](float z) {
        return none ? nan : static_cast<float>((static_cast<double>(z) * a.c - ref - log2_s) * ln2);
    };
    if (tid == 0) {
        if (a.lse) a.lse[r] = none ? -INFINITY : static_cast<float>((ref + log2_s) * ln2);
        if (a.entropy) a.entropy[r] = none ? nan : static_cast<float>(ln2 * (log2_s - t / s));
        if (a.logp) {
            float v = 0.f;
            if (tok >= 0 && tok < a.V) v = logprob(z_tok);
            else if (tok != -1) set_status(a.status, GPT_ERR_INDEX);
            a.logp[r] = v;
        }
    }
    for (int i = tid; i < ncta * a.k; i += NT) {
        const int q = i / a.k, j = i % a.k;
        const unsigned long long e = lists[q][j];
        if (e == 0) continue;
        int place = j;
        for (int o = 0; o < ncta; ++o) {
            if (o == q) continue;
            int lo = 0, hi = a.k;   // entries of list o above e
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (lists[o][mid] > e) lo = mid + 1;
                else hi = mid;
            }
            place += lo;
        }
        if (place < a.k) {
            const uint32_t key = static_cast<uint32_t>(e >> 32);
            a.top_ids[r * a.k + place] = entry_col(e);
            a.top_logp[r * a.k + place] = logprob(key == 0xffffffffu ? nan : key_value(key));
        }
    }
}

struct GradArgs {
    long long ld, ldd;
    const int64_t* tokens;
    uint32_t V;
    float inv_t;
    const float *lse, *entropy, *dlogp, *dentropy;
    int32_t* status;
};

// What a row's elements share: with l = z / T - lse, the gradient is -2^(l log2 e) (h l + gh) and g more
// at the token's column (factors divided by T).
struct RowGrad {
    float inv_t, L, g, h, gh;
    GPT_DEVINL uint64_t two(float a, float b) const {
        const uint64_t l = f2_fma(f2_pack(a, b), f2_pack(inv_t, inv_t), f2_pack(-L, -L));
        float l0, l1, v0, v1;
        f2_unpack(f2_mul(l, f2_pack(1.4426950408889634f, 1.4426950408889634f)), l0, l1);
        const float p0 = exp2_approx(l0), p1 = exp2_approx(l1);
        const uint64_t w = f2_fma(f2_pack(h, h), l, f2_pack(gh, gh));
        f2_unpack(f2_mul(f2_pack(-p0, -p1), w), v0, v1);
        // where p is 0 so is the gradient, whatever the factors' size makes of l = -inf or far below 0
        return f2_pack(p0 == 0.f ? 0.f : v0, p1 == 0.f ? 0.f : v1);
    }
    GPT_DEVINL float one(float z, bool hit) const {
        float v, unused;
        f2_unpack(two(z, z), v, unused);
        return hit ? v + g : v;
    }
};

GPT_DEVINL uint4 grad_unit(const RowGrad& q, const uint4& w, uint32_t hit, const bf16*) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(q.two(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)), a, b);
        if (hit < 8) {   // the token's column is one of these eight
            if (hit == 2 * i) a += q.g;
            if (hit == 2 * i + 1) b += q.g;
        }
        y[i] = pack_bf16x2(a, b);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
}
GPT_DEVINL uint4 grad_unit(const RowGrad& q, const uint4& w, uint32_t hit, const float*) {
    float y[4];
    f2_unpack(q.two(__uint_as_float(w.x), __uint_as_float(w.y)), y[0], y[1]);
    f2_unpack(q.two(__uint_as_float(w.z), __uint_as_float(w.w)), y[2], y[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (hit == i) y[i] += q.g;
    return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
}

// One read and one write of the row: gridDim.x CTAs share row blockIdx.y + k gridDim.y's 16-byte units.
template <typename E>
__global__ void __launch_bounds__(kThreads)
    logprobs_backward_kernel(const E* logits, E* dlogits, long long rows, const GradArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t first = blockIdx.x * blockDim.x + threadIdx.x;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
        const Slice<E> z(logits + r * a.ld, a.V, gridDim.x * blockDim.x);
        E* d = dlogits + r * a.ldd;
        long long tok = -1;
        float g = 0.f, h = 0.f, H = 0.f;
        if (a.dlogp) {
            tok = __ldcg(a.tokens + r);
            if (tok >= 0 && tok < a.V) {
                g = __ldcg(a.dlogp + r);
            } else {
                if (tok != -1 && first == 0) set_status(a.status, GPT_ERR_INDEX);
                tok = -1;
            }
        }
        if (a.dentropy) h = __ldcg(a.dentropy + r), H = __ldcg(a.entropy + r);
        const float L = __ldcg(a.lse + r);
        const Slice<E> out(d, a.V, z.stride);
        // rows without a gradient, and those without a distribution (L - L is NaN)
        const bool zero = (g == 0.f && h == 0.f) || L == -INFINITY;
        if (zero || L - L != 0.f) {
            const float v = zero ? 0.f : __int_as_float(0x7fffffff);
            const uint32_t v2 = zero ? 0u : 0x7fff7fffu;
            for (uint32_t u = first; u < out.units; u += out.stride)
                *reinterpret_cast<uint4*>(d + out.unit_col(u)) = sizeof(E) == 2 ? make_uint4(v2, v2, v2, v2)
                    : make_uint4(__float_as_uint(v), __float_as_uint(v), __float_as_uint(v), __float_as_uint(v));
            if (first < out.ends) st(d + out.end_col(first), v);
            continue;
        }
        const RowGrad q = {a.inv_t, L, g * a.inv_t, h * a.inv_t, (g + h * H) * a.inv_t};
        if (z.head == out.head) {
            for (uint32_t u0 = first; u0 < z.units; u0 += z.stride * kUnroll) {
                uint4 w[kUnroll];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    const uint32_t u = u0 + i * z.stride;
                    if (u < z.units) w[i] = __ldcg(reinterpret_cast<const uint4*>(z.z + z.unit_col(u)));
                }
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    const uint32_t u = u0 + i * z.stride;
                    if (u < z.units)
                        *reinterpret_cast<uint4*>(d + z.unit_col(u)) =
                            grad_unit(q, w[i], static_cast<uint32_t>(tok) - z.unit_col(u), z.z);
                }
            }
            if (first < z.ends) {
                const uint32_t col = z.end_col(first);
                st(d + col, q.one(ld_act(z.z + col), col == tok));
            }
        } else {   // rows that start at different places of a 16-byte unit: by element, eight loads in flight
            // (6035 rows x 27626 bf16: 147 us, 375 with one load in flight)
            constexpr int kEach = 8;
            uint32_t col = first;
            for (; a.V > (kEach - 1) * z.stride && col < a.V - (kEach - 1) * z.stride; col += kEach * z.stride) {
                float v[kEach];
#pragma unroll
                for (int i = 0; i < kEach; ++i) v[i] = ld_act(z.z + col + i * z.stride);
#pragma unroll
                for (int i = 0; i < kEach; i += 2) {
                    float x, y;
                    f2_unpack(q.two(v[i], v[i + 1]), x, y);
                    const uint32_t c0 = col + i * z.stride, c1 = c0 + z.stride;
                    st(d + c0, c0 == tok ? x + q.g : x);
                    st(d + c1, c1 == tok ? y + q.g : y);
                }
            }
            for (; col < a.V; col += z.stride) st(d + col, q.one(ld_act(z.z + col), col == tok));
        }
    }
}

template <typename E>
int launch_score(const E* logits, const ScoreArgs& a, int rows, cudaStream_t s) {
    if (a.cluster > 1)
        return launch_overlapped_cluster(logprobs_kernel<E, 256>, a.cluster, dim3(rows * a.cluster), dim3(256), 0, s, logits, a);
    if (a.threads == 256) return launch_overlapped(logprobs_kernel<E, 256>, dim3(rows), dim3(256), 0, s, logits, a);
    if (a.threads == 32) return launch_overlapped(logprobs_kernel<E, 32>, dim3(rows), dim3(32), 0, s, logits, a);
    if (a.threads == 64) return launch_overlapped(logprobs_kernel<E, 64>, dim3(rows), dim3(64), 0, s, logits, a);
    return launch_overlapped(logprobs_kernel<E, 128>, dim3(rows), dim3(128), 0, s, logits, a);
}

}  // namespace

int launch_logprobs(const void* logits, long long ld, const int64_t* tokens, int rows, int V, int dtype,
                    float temperature, float* logp, float* entropy, float* lse, int k, int64_t* top_ids,
                    float* top_logp, int32_t* status, cudaStream_t s) {
    ScoreArgs a = {};
    a.ld = ld;
    a.tokens = tokens;
    a.V = V;
    const double c = 1.4426950408889634 / temperature;
    a.c = static_cast<float>(c);
    const float low = static_cast<float>(-1e30 / (c > 1. ? c : 1.));
    uint32_t bits;
    memcpy(&bits, &low, 4);
    bits &= 0xffff0000u;   // a bf16 value
    memcpy(&a.floor_z, &bits, 4);
    a.floor2 = bits | bits >> 16;
    a.logp = logp;
    a.entropy = entropy;
    a.lse = lse;
    a.k = k;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.status = status;
    // Rows are split only while that leaves SMs without a CTA, and not below 2048 columns: joining the parts'
    // lists costs more than it saves (64 rows x 50304 bf16, 64 alternatives: 2 CTAs a row 10.8,
    // 4: 12.3, 8: 22.5 us; 8 rows fp32: 2: 11.8, 4: 11.3, 8: 15.4 us).
    int cluster = kMaxCluster;
    while (cluster > 1 && (static_cast<long long>(rows) * cluster > 148 || V < cluster * 2048)) cluster /= 2;
    a.cluster = cluster;
    // Threads per row, from the 16-byte units of a row (measured at every power of two; us with 0 / 1 / 20
    // alternatives).  More than a wave of 128-thread CTAs: a row's end (reductions, the list) costs a CTA about
    // the same however many threads it has, so that short rows want few.  9000 rows x 2057 bf16: 32 threads
    // 12.4 / 17.6 / 23.2, 64: 13.4 / 27.3 / 32.1, 128: 19.1 / 36.0 / 40.7; 9000 x 5000 bf16: 25.5 / 31.7 / 37.8,
    // 23.2 / 36.6 / 41.7, 30.2 / 48.1 / 52.5; 9000 x 9001 fp32: 66.3 / 72.9 / 92.7, 56.7 / 68.7 / 73.9, 60.0 / 80.9 /
    // 84.9.  The list's bound needs more threads than entries: 64 threads with 64 entries pass over a crowd (8805 x
    // 2057 bf16: 40 entries 41 against 48 us with 128 threads, 48: 49 and 51, 56: 65 and 56, 64: 179 and 59).
    // Long rows want enough CTAs for several waves as well (us with 0 / 1 / 20 / 32 alternatives, 64 threads | 128),
    // from 3 rows per 2 units on: 12288 x 50257 bf16 192 / 205 / 229 / 248 | 194 / 231 / 236 / 242, 9000 x 32000 99 /
    // 116 / 118 / 126 | 95 / 124 / 123 / 120, 6000 x 20000 47 / 56 / 61 / 64 | 45 / 62 / 62 / 65, 9000 x 12000 fp32 69 / 87 / 89 /
    // 93 | 74 / 98 / 99 / 102, 13000 x 32003 255 / 277 / 293 / 305 | 252 / 284 / 295 / 303; below: 3000 x 32000 bf16 43 / 49 / 52 / 53 | 39 /
    // 46 / 48 / 50, 2500 x 20000 24 / 28 / 29 / 30 | 23 / 28 / 30 / 31, 3000 x 12000 fp32 30 / 36 / 38 / 40 | 29 / 36 / 38 / 40; 8000 x
    // 50257 bf16 (2.5 rows per 2 units) and 4000 x 32003 fp32 (1) lie within 6% of one another, either way.
    // At most four rows per SM: twice the loads in flight once a row or all of them are long (592 x 50257 bf16:
    // 256 threads 15.0 / 18.0 / 18.5, 128: 17.6 / 20.3 / 20.8; 300 rows: 11.4 / 14.2 / 14.7, 9.8 / 12.4 / 12.9).
    const long long row_units = (static_cast<long long>(V) * (dtype == GPT_DTYPE_BF16 ? 2 : 4) + 15) / 16;
    a.threads = 128;
    if (cluster > 1 || (rows <= 148 && row_units >= 2048) || (rows <= 148 * 4 && rows * row_units >= 1 << 21)) a.threads = 256;
    else if (rows > 148 * 9 && k <= 20 && row_units <= (k ? 640 : 512)) a.threads = 32;
    else if (rows > 148 * 9 && k <= 40 && (row_units <= 1280 || (k <= 32 && 2ll * rows >= 3 * row_units))) a.threads = 64;
    const long long step = static_cast<long long>(a.threads) * cluster * kUnroll * (dtype == GPT_DTYPE_BF16 ? 8 : 4);
    while ((V + step - 1) / step > static_cast<long long>(kSlots) << a.slot_shift) ++a.slot_shift;
    return dtype == GPT_DTYPE_BF16 ? launch_score(static_cast<const bf16*>(logits), a, rows, s)
                                   : launch_score(static_cast<const float*>(logits), a, rows, s);
}

int launch_logprobs_backward(const void* logits, long long ld, const int64_t* tokens, int rows, int V, int dtype,
                             float temperature, const float* lse, const float* entropy, const float* dlogp,
                             const float* dentropy, void* dlogits, long long ldd, int32_t* status, cudaStream_t s) {
    const GradArgs a = {ld, ldd, tokens, static_cast<uint32_t>(V), 1.f / temperature, lse, entropy, dlogp, dentropy, status};
    // a CTA takes at least 4 units per thread; rows are split only while there are fewer than 8 CTAs per SM
    // Threads per CTA, from the 16-byte units of a row (us with 64 / 128 / 256).  Logits and gradient aligned alike: 9000
    // rows x 2057 bf16 15.6 / 16.9 / 25.8, x 5000 32.2 / 34.6 / 41.3, x 9001 55.5 / 55.6 / 62.0, x 18001 106.8 / 104.0 /
    // 103.6, x 27001 161 / 155 / 151; differently: 19.7 / 21.6 / 27.8, 51.0 / 53.4 / 63.7, 84 / 86 / 88, 151 / 155 / 163,
    // 227 / 226 / 218.  fp32 9000 x 5000 60.3 / 60.6 / 67.9 and 77.9 / 78.0 / 84.9, 4000 x 32003 180 / 170 / 163 and 207 / 207 / 197
    const long long row_units = (static_cast<long long>(V) * (dtype == GPT_DTYPE_BF16 ? 2 : 4) + 15) / 16;
    const int threads = row_units <= 640 ? 64 : row_units <= 2304 ? 128 : kThreads;
    const int per = threads * kUnroll * (dtype == GPT_DTYPE_BF16 ? kVec<bf16> : kVec<float>);
    int split = 1;
    while (static_cast<long long>(rows) * split < 148 * 8 && split * per < V) ++split;
    const dim3 grid(split, rows < 65535 ? rows : 65535), block(threads);
    if (dtype == GPT_DTYPE_BF16)
        return launch_overlapped(logprobs_backward_kernel<bf16>, grid, block, 0, s, static_cast<const bf16*>(logits),
                                 static_cast<bf16*>(dlogits), static_cast<long long>(rows), a);
    return launch_overlapped(logprobs_backward_kernel<float>, grid, block, 0, s, static_cast<const float*>(logits),
                             static_cast<float*>(dlogits), static_cast<long long>(rows), a);
}

}  // namespace gpt
