// Attention of the nodes of drafted trees over a key/value cache and their ancestors
// (gpt.h, gpt_tree_attention):
//   y_i = sum_j softmax_j(q_i . k_j / sqrt(hs)) v_j,  j over the cached positions and A(i).
//
// Per sequence and head the cached k and v are read once for all nodes, so the work is bound by HBM: 256
// bytes (bf16) per key and head, against 4 x 64 x N operations.  A cluster of 1 to 8 CTAs takes a sequence
// and head: its tiles of keys, the last of them the nodes' own, go round to the CTAs, each keeps an online
// softmax (running maximum, sum and weighted values, all fp32), and the parts are joined over distributed
// shared memory in a fixed order, so the call needs no workspace and its results are reproducible.
#include <math.h>

#include "internal.h"
#include "tree.cuh"

namespace gpt {

namespace {

struct TreeArgs {
    const int* lengths;
    const int* parents;
    int B, N, nh, hs, block_size, cluster;
    int longest_first;   // CTAs take the sequences in the order of their lengths
    float scale_log2;   // log2(e) / sqrt(hs)
    int32_t* status;
};

GPT_DEVINL float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}
GPT_DEVINL float2 ld_cluster_f2(uint32_t cluster_addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr) : "memory");
    return v;
}

// named_barrier that returns whether any of its threads passed true.
GPT_DEVINL bool named_barrier_or(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %3, 0;\n\t"
        "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

// One lane of a converged warp.
GPT_DEVINL bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

GPT_DEVINL float4 sum(const float4& a, const float4& b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// Parts of a softmax over disjoint keys: weighted values o (eight of a row), {maximum (log2 units), sum}.
// A part without keys has a sum of 0 and its o is not looked at.
struct Joined {
    float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    GPT_DEVINL void see(const float2& ml) {
        if (ml.y != 0.f) M = fmaxf(M, ml.x);
    }
    GPT_DEVINL void add(const float2& ml, const float4& v, const float4& w) {
        const float f = ml.x == M ? 1.f : exp2_approx(ml.x - M);
        L = fmaf(f, ml.y, L);
        o[0] = fmaf(f, v.x, o[0]), o[1] = fmaf(f, v.y, o[1]), o[2] = fmaf(f, v.z, o[2]), o[3] = fmaf(f, v.w, o[3]);
        o[4] = fmaf(f, w.x, o[4]), o[5] = fmaf(f, w.y, o[5]), o[6] = fmaf(f, w.z, o[6]), o[7] = fmaf(f, w.w, o[7]);
    }
    GPT_DEVINL void finish() {
        const float inv = 1.f / L;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= inv;
    }
    // ... and adds the values that are not finite of the rows in `from` (at v, stride elements apart)
    template <typename E>
    GPT_DEVINL void finish(unsigned long long from, const E* v, long long stride) {
        finish();
        for (; from; from &= from - 1) {
            float f[8];
            ld8(v + (__ffsll(from) - 1) * stride, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!isfinite(f[e])) o[e] += f[e];
        }
    }
};

// The parts that the cluster's CTAs left at the same place of their shared memory (o [N][ld], ml [N]),
// joined in the order of their ranks and written; each CTA takes a share of the rows' pieces of eight.
// per: pieces of a row; finish(i, d, joined): the rows that are nodes.
template <typename E, typename F>
GPT_DEVINL void join_cluster(const float* o, int ld, const float2* ml, const unsigned long long* see, const TreeArgs& a,
                             int per, int rank, E* y, long long row_stride, F finish) {
    for (int it = rank * blockDim.x + threadIdx.x; it < a.N * per; it += a.cluster * blockDim.x) {
        const int i = it / per, d = (it - i * per) * 8;
        Joined j;
        if (see[i]) {
            float2 part[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < a.cluster) part[q] = ld_cluster_f2(map_to_rank(&ml[i], q));
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < a.cluster) j.see(part[q]);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < a.cluster && part[q].y != 0.f) {
                    const uint32_t at = map_to_rank(&o[i * ld + d], q);
                    j.add(part[q], ld_cluster_f4(at), ld_cluster_f4(at + 16));
                }
            finish(i, d, j);
        }
        st8(y + i * row_stride + d, j.o);
    }
}

// Loads the sequence's parents and finds every node's A(i) (0: no node); all threads, ends with a barrier.
GPT_DEVINL void load_tree(const TreeArgs& a, int b, bool report, int* par, unsigned long long* see) {
    const int tid = threadIdx.x;
    if (tid < a.N) par[tid] = __ldcg(a.parents + static_cast<long long>(b) * a.N + tid);
    __syncthreads();
    if (tid < kMaxNodes) {
        see[tid] = tid < a.N ? ancestors(par, tid) : 0;
        if (report && tid < a.N && see[tid] == 0 && par[tid] != -2) set_status(a.status, GPT_ERR_INDEX);
    }
    __syncthreads();
}

// ---------------------------------------------------------------- bf16, head size 64
// Tiles of 128 keys by TMA (a two-deep ring), both products on the tensor cores (tcgen05):
//   S [128 x 128] = Q' K^T, Q' the R = 32 or 64 node rows repeated 128 / R times, so that the 128 TMEM
//     lanes are 128 / R groups of all nodes; group g uses the columns [g R, (g + 1) R) of its rows only:
//     every thread has R scores, a row of its own, and no reduction between threads;
//   O [128 x 64] += P V, one chain of products for the shares of all groups, joined at the end.
// The repeated rows cost tensor time (2 cycles per key of the 11 that its bytes take at this GPU's copy
// rate) and save the transposes and shuffles that splitting the keys over lanes would take.
//
// A bf16 operand holds 8 bits of a weight that was computed in 32, so a weight p enters the product as
// hi + lo: hi its upper 16 bits, lo the rest rounded to bf16, off by at most 2^-15 p.  hi and lo have a lane each and
// their rows of O are added at the end, so that the tensor cores do no more than for hi alone:
//   N <= 16 (TWICE): a group has 16 nodes' rows twice; both lanes compute p, one hands on hi and one lo;
//   else groups 2 k and 2 k + 1 keep a running maximum together, and a lane has hi of its own columns and lo of the
//     other group's, which come through shared memory.
// P is 0 in the columns that are not a lane's (written once).  Against p rounded to bf16 (2-norm error 1.7e-3 to
// 2.3e-3; now 1.5e-3 to 1.7e-3, the rounding of y alone), us in a burst / back to back: 8 sequences x 16 nodes x 12
// heads 13.0 / 13.0 -> 13.5 / 13.5, 48 x 23 x 25 up to 8185 keys 244 / 278 -> 253 / 292, 32 x 64 x 16 up to 4096 keys
// 56 / 64 -> 63 / 73.5.  Two products per tile instead, lo's behind hi's: 281 / 333 and 66 / 78.
//
// The nodes' own keys lie in the last R rows of the last tile, behind the cache's rest if that leaves room.
//
// Warp 0 issues the loads, warp 1 the products, warps 2-5 the softmax; two CTAs share an SM.  With more
// pairs of sequence and head than run at a time the CTAs are persistent, so that a pair's first loads and
// products run under the join of the one before, and take the pairs longest first, every other round in
// reverse (sequences of up to THREADS; beyond that in the order given).
//
// The product multiplies masked values by 0, so values that must not be seen are made harmless in shared
// memory: V rows between the cache's end and the nodes, and of absent nodes, are cleared; values of nodes
// that are not finite are replaced by 0 and added at the end to the rows that see them.
namespace tc {
constexpr int HS = 64;
constexpr int KEYS = 128;
constexpr int BOX = 32;                       // rows per load of the cache's rest
constexpr int node_box(bool twice) { return twice ? 16 : 32; }   // ... and of the nodes' q, k, v
constexpr int ROW_BYTES = HS * 2;
constexpr int THREADS = 192;
constexpr int TILE = KEYS * HS * 2;           // 16 KB
constexpr int HALF = HS / 2, HALF_LD = HALF + 4;   // the groups' parts are joined half a row at a time
constexpr int LD = HS + 4;                    // floats per row of the CTA's part
constexpr int STAGES = 2;
constexpr uint32_t TMEM_COLS = 256, COL_S = 0, COL_P = 128, COL_O = 192;
constexpr float kRescaleThreshold = 8.f;      // as in the causal kernel: P stays below 2^8

struct Tail {
    uint64_t q_full, q_empty, k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES], s_free, p_full, drain;
    unsigned long long see[kMaxNodes], bad;   // bad: node rows of V with values that are not finite
    float2 ml[KEYS], joined_ml[kMaxNodes];
    float mx[KEYS];
    int par[kMaxNodes];
    int lengths[THREADS];                     // with longest_first: in the order of the pairs,
    short order[THREADS];                     // and the sequences they belong to
    uint32_t tmem;
    int abort;
};
constexpr int SMEM = (1 + 2 * STAGES) * TILE + KEYS * HALF_LD * 4 + static_cast<int>(sizeof(Tail)) + 1024;

// One sequence and head, as one CTA of its cluster sees it.
struct Work {
    int b, h, len, n_cache, rest, n_tiles, n_steps;   // rest: keys of the cache in the last tile
    GPT_DEVINL bool last(int j) const { return j == n_steps - 1 && has_nodes; }
    bool has_nodes;
};

template <int R>
GPT_DEVINL Work work_of(int pair, const TreeArgs& a, const Tail& T, int rank, int32_t* status) {
    Work w;
    w.b = pair / a.nh;
    w.h = pair - w.b * a.nh;
    int len;
    if (a.longest_first) {
        len = T.lengths[w.b];
        w.b = T.order[w.b];
    } else {
        len = __ldcg(a.lengths + w.b);
    }
    w.len = clamp_length(len, a.block_size, w.h == 0 ? status : nullptr);
    w.n_cache = w.len / KEYS;               // tiles of the cache alone
    w.rest = w.len - w.n_cache * KEYS;
    if (w.rest > KEYS - R) ++w.n_cache, w.rest = 0;
    w.n_tiles = w.n_cache + 1;
    w.n_steps = rank < w.n_tiles ? (w.n_tiles - 1 - rank) / a.cluster + 1 : 0;
    w.has_nodes = w.n_cache % a.cluster == rank;
    return w;
}

template <int R, bool TWICE>
__global__ void __launch_bounds__(THREADS, 2)
    tree_attention_tc(const __grid_constant__ CUtensorMap tmNode, const __grid_constant__ CUtensorMap tmCache,
                      const __grid_constant__ CUtensorMap tmRest, const bf16* __restrict__ qkv, bf16* __restrict__ y,
                      const TreeArgs a) {
    constexpr int ROWS = TWICE ? R / 2 : R, NODE_BOX = node_box(TWICE);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sK = smem + TILE;
    uint8_t* sV = sK + STAGES * TILE;
    float* sPart = reinterpret_cast<float*>(sV + STAGES * TILE);
    float* joined = reinterpret_cast<float*>(sK) + KEYS * LD;   // in a cluster, which has one pair
    Tail& T = *reinterpret_cast<Tail*>(sPart + KEYS * HALF_LD);
    volatile int* abort_flag = &T.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    // pairs: this CTA's (its cluster's) first, then one per round of the grid, every other round in reverse
    const int n_pairs = a.B * a.nh, pair_stride = static_cast<int>(gridDim.x) / a.cluster;
    const int pair0 = static_cast<int>(blockIdx.x) / a.cluster;
    auto pair_at = [&](int round) {
        return round * pair_stride + ((round & 1) ? pair_stride - 1 - pair0 : pair0);
    };

    if (threadIdx.x == 0) {
        uint64_t* bars = &T.q_full;
        constexpr int n_bars = 2 + 4 * STAGES + 3;
        for (int i = 0; i < n_bars; ++i) mbar_init(&bars[i], (&bars[i] == &T.s_free || &bars[i] == &T.p_full) ? 128u : 1u);
        T.abort = 0;
        T.bad = 0;
        fence_barrier_init();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tma_prefetch_desc(&tmNode);
        tma_prefetch_desc(&tmCache);
        tma_prefetch_desc(&tmRest);
    }
    if (warp == 1) {
        tmem_alloc(&T.tmem, TMEM_COLS);
        tmem_relinquish();
        griddep_launch_dependents();   // not before: a dependent could hold the columns that this warp waits for
    }
    griddep_wait();
    if (a.longest_first) {   // the sequences in the order of their lengths, equal ones by index
        const int t = threadIdx.x;
        const int mine = t < a.B ? __ldcg(a.lengths + t) : 0;
        int* all = reinterpret_cast<int*>(sPart);
        if (t < a.B) all[t] = mine;
        __syncthreads();
        if (t < a.B) {
            int place = 0;
            for (int j = 0; j < a.B; ++j) place += all[j] > mine || (all[j] == mine && j < t);
            T.lengths[place] = mine;
            T.order[place] = static_cast<short>(t);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = T.tmem;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int n = 0, n_q = 0;   // tiles and query loads issued
            bool ok = true;
            int issued_v = 0;
            for (int round = 0; ok && pair_at(round) < n_pairs; ++round) {
                const Work w = work_of<R>(pair_at(round), a, T, rank, nullptr);
                for (int j = 0; ok && j < w.n_steps; ++j, ++n) {
                    const int st = n % STAGES;
                    const uint32_t ph = (n / STAGES) & 1;
                    const int t = rank + j * a.cluster;
                    auto tile = [&](int v) {
                        uint64_t* full = v ? &T.v_full[st] : &T.k_full[st];
                        uint8_t* dst = (v ? sV : sK) + st * TILE;
                        if (!w.last(j)) {
                            mbar_arrive_expect_tx(full, TILE);
                            tma_load_4d(dst, &tmCache, full, 0, v * a.nh + w.h, t * KEYS, w.b);
                            return;
                        }
                        const int boxes = (w.rest + BOX - 1) / BOX;
                        mbar_arrive_expect_tx(full, (boxes * BOX + R) * ROW_BYTES);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_4d(dst + i * BOX * ROW_BYTES, &tmRest, full, 0, v * a.nh + w.h, t * KEYS + i * BOX, w.b);
                        for (int i = 0; i < R; i += NODE_BOX)
                            tma_load_4d(dst + (KEYS - R + i) * ROW_BYTES, &tmNode, full, 0, (1 + v) * a.nh + w.h, i, w.b);
                    };
                    if (!(ok = mbar_wait(&T.k_empty[st], ph ^ 1u, abort_flag))) break;
                    tile(0);
                    if (j == 0) {
                        if (n_q > 0 && !mbar_wait(&T.q_empty, (n_q - 1) & 1, abort_flag)) {
                            ok = false;
                            ++n;
                            break;
                        }
                        mbar_arrive_expect_tx(&T.q_full, TILE);
                        for (int i = 0; i < KEYS; i += NODE_BOX)
                            tma_load_4d(sQ + i * ROW_BYTES, &tmNode, &T.q_full, 0, w.h, i % ROWS, w.b);
                        ++n_q;
                    }
                    if (!mbar_wait(&T.v_empty[st], ph ^ 1u, abort_flag)) {
                        ok = false;
                        ++n;
                        break;
                    }
                    tile(1);
                    ++issued_v;
                }
            }
            // No bulk copy may still target shared memory when the CTA exits (n: K tiles issued).
            if (n_q > 0) mbar_drain(&T.q_full, (n_q - 1) & 1);
            for (int i = 1; i <= STAGES; ++i) {
                if (n >= i) mbar_drain(&T.k_full[(n - i) % STAGES], ((n - i) / STAGES) & 1);
                if (issued_v >= i) mbar_drain(&T.v_full[(issued_v - i) % STAGES], ((issued_v - i) / STAGES) & 1);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // The whole warp follows the steps (uniform addresses and descriptors), one lane issues.
        constexpr uint32_t idesc_s = make_idesc_bf16(128, KEYS, false), idesc_o = make_idesc_bf16(128, HS, true);
        const uint32_t tS = tmem + COL_S, tP = tmem + COL_P, tO = tmem + COL_O;
        const uint32_t q_addr = smem_addr(sQ), k_addr = smem_addr(sK), v_addr = smem_addr(sV);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag); };
        auto all = [](bool v) { return __all_sync(0xffffffffu, v) != 0; };
        // Testing aid (gpt_set_wait_limit_ns): nothing arrives on `drain` before the commit below.
        if (g_force_timeout) all(wait(&T.drain, 0));
        bool ok = !g_force_timeout;
        int n = 0, n_q = 0;
        bool first = true;   // step n - 1 was its pair's first
        auto values = [&]() {   // O (+)= P_{n-1} V_{n-1}, once the softmax has written P_{n-1}
            const int st = (n - 1) % STAGES;
            if (!all(wait(&T.p_full, (n - 1) & 1) && wait(&T.v_full[st], ((n - 1) / STAGES) & 1))) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < KEYS / 16; ++kk)
                    umma_ts(tO, tP + kk * 8, make_sdesc_sw128(v_addr + st * TILE + kk * 2048), idesc_o, !first || kk > 0);
                umma_commit(&T.v_empty[st]);
            }
            __syncwarp();
            return true;
        };
        for (int round = 0; ok && pair_at(round) < n_pairs; ++round) {
            const Work w = work_of<R>(pair_at(round), a, T, rank, nullptr);
            for (int j = 0; j < w.n_steps; ++j, ++n) {
                // between pairs the values first: the softmax waits for them, not for the next scores
                if (j == 0 && n > 0 && !(ok = values())) break;
                const int st = n % STAGES;
                // S_n, once the softmax has taken S_{n-1} out of TMEM
                ok = all((j > 0 || wait(&T.q_full, n_q & 1)) && wait(&T.k_full[st], (n / STAGES) & 1) &&
                         (n == 0 || wait(&T.s_free, (n - 1) & 1)));
                if (!ok) break;
                n_q += j == 0;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HS / 16; ++kk)
                        umma_ss(tS, make_sdesc_sw128(q_addr + kk * 32), make_sdesc_sw128(k_addr + st * TILE + kk * 32), idesc_s, kk > 0);
                    umma_commit(&T.k_empty[st]);
                    if (j == w.n_steps - 1) umma_commit(&T.q_empty);
                }
                __syncwarp();
                if (j > 0 && !(ok = values())) break;
                first = j == 0;
            }
        }
        if (ok && n > 0) values();
        if (elect_one()) {
            umma_commit(&T.drain);
            mbar_drain(&T.drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and join
        const int t = threadIdx.x - 64;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane, group = r / R, node = r % R, col0 = group * R;   // node: of key row r
        // the pair of groups that share their weights, and the warps that hold it
        const int pair_bar = 2 + (R == 64 ? quarter & 1 : quarter >> 1);
        uint4* swap = reinterpret_cast<uint4*>(sPart);
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + COL_S + lane_off + col0, tP = tmem + COL_P + lane_off, tO = tmem + COL_O + lane_off;
        const bool node_group = group == KEYS / R - 1;
        const long long C = static_cast<long long>(a.nh) * HS;
        {
            uint32_t zero[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) zero[i] = 0;
            tmem_st32(tP, zero);
            tmem_st32(tP + 32, zero);
        }
        int32_t* status = rank == 0 && t == 0 ? a.status : nullptr;
        int n = 0;
        bool ok = true, more = pair_at(0) < n_pairs;
        Work next = {};
        int next_parent = 0;
        auto look_ahead = [&](int round) {   // the pair of that round, its parents on their way
            more = pair_at(round) < n_pairs;
            if (!more) return;
            next = work_of<R>(pair_at(round), a, T, rank, status);
            if (t < a.N) next_parent = __ldcg(a.parents + static_cast<long long>(next.b) * a.N + t);
        };
        look_ahead(0);
        for (int round = 0; ok && more; ++round) {
            const Work w = next;
            if (t < a.N) T.par[t] = next_parent;
            if (t == 0) T.bad = 0;
            named_barrier(1, 128);
            if (t < kMaxNodes) {
                T.see[t] = t < a.N ? ancestors(T.par, t) : 0;
                if (w.h == 0 && rank == 0 && t < a.N && T.see[t] == 0 && T.par[t] != -2) set_status(a.status, GPT_ERR_INDEX);
            }
            named_barrier(1, 128);
            const unsigned long long see = T.see[r % ROWS], see_key = T.see[node];
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < w.n_steps; ++j, ++n) {
                const bool last = w.last(j);
                const int st = n % STAGES;
                const int keys = last ? w.rest : min(KEYS, w.len - (rank + j * a.cluster) * KEYS);   // of the cache
                if (keys < KEYS) {
                    // V rows that must not matter
                    const bool got = mbar_wait(&T.v_full[st], (n / STAGES) & 1, abort_flag);
                    uint4* row = reinterpret_cast<uint4*>(sV + st * TILE + r * (HS * 2));
                    const bool is_node = last && node_group;
                    if (got && (is_node ? see_key == 0 : r >= keys)) {
#pragma unroll
                        for (int i = 0; i < HS / 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
                    } else if (got && is_node) {
                        bool any = false;
#pragma unroll
                        for (int i = 0; i < HS / 8; ++i) {
                            uint32_t v[4] = {row[i].x, row[i].y, row[i].z, row[i].w};
                            bool here = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u, here = true;
                                if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu, here = true;
                            }
                            if (here) row[i] = make_uint4(v[0], v[1], v[2], v[3]);
                            any |= here;
                        }
                        if (any) atomicOr(&T.bad, 1ull << node);
                    }
                    fence_proxy_async_shared();
                }
                // K_n read: S_n is there
                const bool got = __all_sync(0xffffffffu, mbar_wait(&T.k_empty[st], (n / STAGES) & 1, abort_flag));
                if (TWICE && !got) {
                    ok = false;
                    break;
                }
                float s[R];
                if (got) {   // (tcgen05.ld / st are warp-collective)
                    tc_fence_after();
                    uint32_t u[R];
                    if constexpr (R == 32) tmem_ld32(tS, u);
                    else tmem_ld64(tS, u);
#pragma unroll
                    for (int c = 0; c < R; ++c) s[c] = __uint_as_float(u[c]);
                    tc_fence_before();
                    mbar_arrive(&T.s_free);
                }
                if (last && node_group) {
#pragma unroll
                    for (int c = 0; c < R; ++c)
                        if (!((see >> c) & 1)) s[c] = -INFINITY;
                } else if (keys - col0 < R) {
#pragma unroll
                    for (int c = 0; c < R; ++c)
                        if (c >= keys - col0) s[c] = -INFINITY;
                }
                float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < R; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
                float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
                if constexpr (!TWICE) {   // ... of both groups; a time-out of one warp ends the steps of its partner as well
                    T.mx[r] = mx;
                    if (named_barrier_or(pair_bar, 64, !got)) {
                        ok = false;
                        break;
                    }
                    mx = fmaxf(mx, T.mx[r ^ R]);
                }
                float alpha = 1.f;
                if (mx > m_used + kRescaleThreshold || (m_used == -INFINITY && mx > -INFINITY)) {
                    alpha = m_used == -INFINITY ? 0.f : exp2_approx(m_used - mx);
                    m_used = mx;
                }
                const float off = m_used == -INFINITY ? 0.f : -m_used;   // nothing visible yet: 2^-inf
                const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), off2 = f2_pack(off, off);
                uint64_t acc[2] = {0, 0};
                uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
                for (int c = 0; c < R; c += 2) {
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), sc2, off2), x0, x1);
                    const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
                    acc[(c >> 1) & 1] = f2_add(acc[(c >> 1) & 1], f2_pack(p0, p1));
                    // (hi is cut, not rounded: lo need not wait for a conversion; 69 us with it, 65.5 without)
                    const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                    hi[c / 2] = __byte_perm(b0, b1, 0x7632);
                    float r0, r1;
                    f2_unpack(f2_sub(f2_pack(p0, p1), f2_pack(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u))), r0, r1);
                    lo[c / 2] = pack_bf16x2(r0, r1);
                }
                float a0, a1;
                f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
                l = l * alpha + (a0 + a1);
                // P_n may overwrite P_{n-1} and O may be rescaled only after O += P_{n-1} V_{n-1} (for a
                // pair's first step the join before it has waited for that).
                auto p_free = [&]() {
                    if (j == 0) return true;
                    const bool done = __all_sync(0xffffffffu, mbar_wait(&T.v_empty[(n - 1) % STAGES], ((n - 1) / STAGES) & 1, abort_flag));
                    tc_fence_after();
                    return done;
                };
                if constexpr (TWICE) {
#pragma unroll
                    for (int c = 0; c < R / 2; ++c)
                        if (r & ROWS) hi[c] = lo[c];
                    ok = p_free();
                    if (ok) tmem_st_nowait(tP + group * (R / 2), hi);
                } else {
#pragma unroll
                    for (int c = 0; c < R / 2; c += 4) swap[c * (KEYS / 4) + r] = make_uint4(lo[c], lo[c + 1], lo[c + 2], lo[c + 3]);
                    ok = p_free();
                    if (ok) tmem_st_nowait(tP + group * (R / 2), hi);
                    ok = !named_barrier_or(pair_bar, 64, !ok);
                    if (ok) {
#pragma unroll
                        for (int c = 0; c < R / 2; c += 4) {
                            const uint4 v = swap[c * (KEYS / 4) + (r ^ R)];
                            lo[c] = v.x, lo[c + 1] = v.y, lo[c + 2] = v.z, lo[c + 3] = v.w;
                        }
                        tmem_st_nowait(tP + (group ^ 1) * (R / 2), lo);
                    }
                }
                tmem_wait_st();
                if (!ok) break;
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                    for (int c = 0; c < HS; c += 32) {
                        uint32_t u[32];
                        tmem_ld32(tO + c, u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
                        tmem_st32(tO + c, u);
                    }
                }
                tc_fence_before();
                mbar_arrive(&T.p_full);
            }
            look_ahead(round + 1);
            bool have = false;
            if (ok && w.n_steps > 0) {
                const bool done = mbar_wait(&T.v_empty[(n - 1) % STAGES], ((n - 1) / STAGES) & 1, abort_flag);
                __syncwarp();
                ok = have = __all_sync(0xffffffffu, done);
                tc_fence_after();
            }
            T.ml[r] = make_float2(m_used, have ? l : 0.f);

            // The groups' parts joined: half rows at a time beside the ring while it fills for the next pair,
            // whole rows in the ring's place after the last; alone, the CTA writes the rows.
            bf16* out = y + static_cast<long long>(w.b) * a.N * C + w.h * HS;
            const bf16* values = qkv + static_cast<long long>(w.b) * a.N * 3 * C + 2 * C + w.h * HS;
            auto join = [&](const float* part, int ld, int d0, int pieces_log2) {
                named_barrier(1, 128);
                const unsigned long long bad = T.bad;
                for (int it = t; it < a.N << pieces_log2; it += 128) {
                    const int i = it >> pieces_log2, dp = (it & ((1 << pieces_log2) - 1)) * 8, d = d0 + dp;
                    // rows (2 ROWS) g + i and ROWS further: the same weights' hi and lo, or two groups' shares of them
                    constexpr int PARTS = KEYS / (2 * ROWS);
                    float2 ml[PARTS];
                    Joined x;
#pragma unroll
                    for (int g = 0; g < PARTS; ++g) {
                        ml[g] = T.ml[2 * ROWS * g + i];
                        if constexpr (!TWICE) ml[g].y += T.ml[2 * ROWS * g + ROWS + i].y;
                        x.see(ml[g]);
                    }
#pragma unroll
                    for (int g = 0; g < PARTS; ++g)
                        if (ml[g].y != 0.f) {
                            const float4* o = reinterpret_cast<const float4*>(part + (2 * ROWS * g + i) * ld + dp);
                            const float4* lo = reinterpret_cast<const float4*>(part + (2 * ROWS * g + ROWS + i) * ld + dp);
                            x.add(ml[g], sum(o[0], lo[0]), sum(o[1], lo[1]));
                        }
                    if (a.cluster > 1) {
                        st8(joined + i * LD + d, x.o);
                        if (d == 0) T.joined_ml[i] = make_float2(x.M, x.L);
                    } else {
                        if (T.see[i]) {
                            x.finish(bad & T.see[i], values + d, 3 * C);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x.o[e] = 0.f;
                        }
                        st8(out + i * C + d, x.o);
                    }
                }
            };
            auto leave = [&](float* row, int d0) {   // 32 dimensions of this thread's row
                uint32_t u[32];
                tmem_ld32(tO + d0, u);
#pragma unroll
                for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4*>(row + e) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
            };
            if (more) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (have) leave(sPart + r * HALF_LD, half * HALF);
                    join(sPart, HALF_LD, half * HALF, 2);
                    // (a time-out seen by one warp ends the rounds of all)
                    ok = !named_barrier_or(1, 128, !ok);
                }
            } else {
                float* whole = reinterpret_cast<float*>(sK);
                if (have) leave(whole + r * LD, 0), leave(whole + r * LD + HALF, HALF);
                join(whole, LD, 0, 3);
            }
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag) set_status(a.status, GPT_ERR_TIMEOUT);
    if (a.cluster == 1) return;
    // A cluster has one pair: its CTAs' parts joined.
    __syncwarp();
    cluster_sync();
    const Work w = work_of<R>(pair0, a, T, rank, nullptr);
    const int holder = w.n_cache % a.cluster;   // of the nodes' tile
    const unsigned long long bad =
        static_cast<unsigned long long>(ld_cluster_u32(map_to_rank(reinterpret_cast<uint32_t*>(&T.bad) + 1, holder))) << 32 |
        ld_cluster_u32(map_to_rank(&T.bad, holder));
    const long long C = static_cast<long long>(a.nh) * HS;
    const bf16* values = qkv + static_cast<long long>(w.b) * a.N * 3 * C + 2 * C + w.h * HS;
    join_cluster(joined, LD, T.joined_ml, T.see, a, HS / 8, rank,
                 y + static_cast<long long>(w.b) * a.N * C + w.h * HS, C,
                 [&](int i, int d, Joined& x) { x.finish(bad & T.see[i], values + d, 3 * C); });
    __syncwarp();
    cluster_sync();   // no CTA leaves while another reads its part
}
}  // namespace tc

// ---------------------------------------------------------------- fp32, head size 8 to 128
// The same split with fp32 operands: every product of two fp32 numbers is taken as three TF32 products
// (x = hi + lo, TF32 each; hi hi + hi lo + lo hi, fp32 accumulation), off by at most 5 x 2^-22 of it (the
// product of the two lo, 2^-10 and 2^-11 of their numbers, and the roundings of each lo).  The refinement is that of
// S. Markidis et al., "NVIDIA Tensor Core Programmability, Performance & Precision" (IPDPSW 2018); that the products'
// accumulator is cut and needs short chains, of H. Ootomo and R. Yokota, "Recovering single precision accuracy from
// Tensor Cores while surpassing the FP32 theoretical peak performance" (IJHPCA 2022).
//
// Tiles of 64 keys come by TMA (panels of 32 dimensions, 128-byte swizzle), two in flight.  A warp has 16 of a
// tile's keys and 16 MT nodes (NG groups of four warps take the nodes of up to 64): each K and V element is
// read from shared memory once per group, the weights go from the scores' registers to the second product as
// they are (the key order of its operands is chosen to match), and a warp keeps a softmax of its own, joined
// at the end.
//
// Against CUDA-core tiles of 2 x 4 scores per thread, which shared-memory reads bind: 19 / 26 us (8 sequences
// x 9 nodes x 12 heads of 64, up to 1013 keys), 68 / 84 us (32 x 30 x 12 of 64, 700 keys), 352 / 545 us
// (20 x 50 x 16 of 128, 2000 keys).  The TF32 products bind it from about 32 nodes on (mma.sync: a 16 x 8 x 8
// product took about 16 cycles per scheduler), their latency below.  With two node tiles per warp registers spill
// (bytes stored, as ptxas counts them, for P, MT, NG): 2, 2, 1: 160; 4, 2, 1 and 4, 2, 2: 16; 1, 2, 1: 12.
namespace f32 {
constexpr int KEYS = 64;
constexpr int STAGES = 2;
// With one group a warp of its own issues the loads (a thousand cycles per tile); with two that ninth warp would
// cost every thread a third of its registers, and thread 0 does it.
constexpr int block_threads(int ng) { return ng == 1 ? 160 : 256; }
constexpr int PANEL = KEYS * 128;   // bytes of 32 dimensions of a tile's rows

template <int P, int MT, int NG>
constexpr int smem_bytes() {
    return 2 * STAGES * P * PANEL + P * 4 * MT * NG * 2 * 32 * 16 + 1024;
}

GPT_DEVINL uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
GPT_DEVINL void split(float x, uint32_t& hi, uint32_t& lo) {
    hi = tf32(x);
    lo = tf32(x - __uint_as_float(hi));
}
// K and V: hi cut, not rounded, so that the type's largest values stay finite (a masked one is multiplied by 0).
GPT_DEVINL void split_cut(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = tf32(x - __uint_as_float(hi));
}
// Queries: hi rounded, but cut where the type's largest values would round to infinity (there lo is 2^-11 of x as well).
GPT_DEVINL void split_finite(float x, uint32_t& hi, uint32_t& lo) {
    hi = tf32(x);
    if ((hi & 0x7f800000u) == 0x7f800000u) hi = __float_as_uint(x) & 0xffffe000u;
    lo = tf32(x - __uint_as_float(hi));
}
GPT_DEVINL void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 16-byte piece `chunk` of a panel's row.
GPT_DEVINL float4 piece(const uint8_t* panel, int row, int chunk) {
    return *reinterpret_cast<const float4*>(panel + row * 128 + ((chunk ^ (row & 7)) << 4));
}

template <int P, int MT, int NG>
__global__ void __launch_bounds__(block_threads(NG), NG > 1 || P > 2 ? 1 : MT > 1 ? 2 : 3)
    tree_attention_f32(const __grid_constant__ CUtensorMap tmNode, const __grid_constant__ CUtensorMap tmCache,
                       const float* __restrict__ qkv, float* __restrict__ y, const TreeArgs a) {
    constexpr int THREADS = 128 * NG, ROWS = 16 * MT * NG, LD = 32 * P + 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint4* sQ = reinterpret_cast<uint4*>(ring + 2 * STAGES * P * PANEL);   // [step][node tile][hi, lo][lane]
    __shared__ unsigned long long see[kMaxNodes], s_bad;
    __shared__ uint64_t full[STAGES], empty[STAGES], never;   // nothing arrives on never
    __shared__ int par[kMaxNodes];
    __shared__ float2 ml[2][ROWS], joined_ml[ROWS];
    __shared__ int s_abort;
    volatile int* abort_flag = &s_abort;
    const int hs = a.hs, N = a.N;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int key_warp = (tid >> 5) & 3, group = tid >> 7;
    const int rank = static_cast<int>(cluster_ctarank());
    const int pair = static_cast<int>(blockIdx.x) / a.cluster;
    const int b = pair / a.nh, h = pair - b * a.nh;
    const long long C = static_cast<long long>(a.nh) * hs;
    const float* node = qkv + static_cast<long long>(b) * N * 3 * C + h * hs;
    if (tid == 0) {
        for (int st = 0; st < STAGES; ++st) mbar_init(&full[st], 1), mbar_init(&empty[st], 4 * NG);
        mbar_init(&never, 1);
        s_abort = 0;
        s_bad = 0;
        fence_barrier_init();
        fence_proxy_async_shared();
        tma_prefetch_desc(&tmNode);
        tma_prefetch_desc(&tmCache);
    }
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();
    const int len = clamp_length(__ldcg(a.lengths + b), a.block_size, h == 0 && rank == 0 && tid == 0 ? a.status : nullptr);
    const int n_cache = (len + KEYS - 1) / KEYS;   // tile n_cache is the nodes'
    const int n_panels = (hs + 31) / 32;
    int issued = 0;   // tiles whose copies the loading thread has issued: one after another, round the stages
    auto load_tile = [&](int t, int stage) {   // one thread
        if (t > n_cache) return;
        ++issued;
        mbar_arrive_expect_tx(&full[stage], 2 * n_panels * PANEL);
        for (int v = 0; v < 2; ++v)
            for (int p = 0; p < n_panels; ++p) {
                uint8_t* dst = ring + (2 * stage + v) * P * PANEL + p * PANEL;
                if (t < n_cache) tma_load_4d(dst, &tmCache, &full[stage], 32 * p, v * a.nh + h, t * KEYS, b);
                else tma_load_4d(dst, &tmNode, &full[stage], 32 * p, (1 + v) * a.nh + h, 0, b);
            }
    };
    constexpr int LOADER = NG == 1 ? THREADS : 0;   // the loading thread
    if (tid == LOADER)
        for (int st = 0; st < STAGES; ++st) load_tile(rank + st * a.cluster, st);

    // The queries as operand fragments.  Step 2c + e of a chunk of 16 dimensions takes dimensions
    // 16 c + 4 t + 2 e (k = t) and the next one (k = t + 4), so that a thread's K values are 16 bytes.
    const int n_steps = 2 * ((hs + 15) / 16);
#pragma unroll 4
    for (int it = tid; it < n_steps * MT * NG * 32; it += block_threads(NG)) {
        const int l = it & 31, tile = (it >> 5) % (MT * NG), s = (it >> 5) / (MT * NG);
        const int row = tile * 16 + (l >> 2), dim = (s >> 1) * 16 + (l & 3) * 4 + (s & 1) * 2;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = row + e * 8;
            const float2 q = i < N && dim < hs ? __ldcg(reinterpret_cast<const float2*>(node + i * 3 * C + dim)) : make_float2(0.f, 0.f);
            split_finite(q.x, hi[e], lo[e]), split_finite(q.y, hi[e + 2], lo[e + 2]);
        }
        sQ[((s * MT * NG + tile) * 2) * 32 + l] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        sQ[((s * MT * NG + tile) * 2 + 1) * 32 + l] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    load_tree(a, b, h == 0 && rank == 0, par, see);

    float o[MT][P][4][4];
    float m[MT][2], l[MT][2];   // of rows g and g + 8 of a node tile
    unsigned long long sees[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            m[mt][r] = -INFINITY, l[mt][r] = 0.f;
            sees[mt][r] = see[((group * MT + mt) * 16 + g + 8 * r) & (kMaxNodes - 1)];
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][p][q][e] = 0.f;
    }
    const int key0 = key_warp * 16;
    // After a wait that gave up, a warp still goes through the remaining tiles (the others may wait for it at a
    // barrier), on whatever the stages hold, but arrives on nothing, so that the loading thread issues no more.
    bool ok = true;
    // Testing aid (gpt_set_wait_limit_ns): with the first loads under way, no tile is waited for.
    if (g_force_timeout && tid < THREADS) ok = mbar_wait(&never, 0, abort_flag);
    int n = 0;   // tiles gone through
    if (tid >= THREADS) {
        if (lane == 0) {
            for (int t = rank; t <= n_cache; t += a.cluster, ++n) {
                if (t + STAGES * a.cluster > n_cache) continue;
                if (!(ok = mbar_wait(&empty[n % STAGES], (n / STAGES) & 1, abort_flag))) break;
                load_tile(t + STAGES * a.cluster, n % STAGES);
            }
        }
    } else for (int t = rank; t <= n_cache; t += a.cluster, ++n) {
        const int stage = n % STAGES;
        uint8_t* sK = ring + 2 * stage * P * PANEL;
        uint8_t* sV = sK + P * PANEL;
        const bool nodes = t == n_cache;
        const int keys = nodes ? N : min(KEYS, len - t * KEYS);
        ok = mbar_wait(&full[stage], (n / STAGES) & 1, abort_flag) && ok;
        if (nodes || keys < KEYS) {
            // V rows that must not matter are cleared; values of nodes that are not finite wait for the end
            for (int it = tid; it < n_panels * KEYS * 8; it += THREADS) {
                const int row = (it >> 3) & (KEYS - 1);
                uint4* at = reinterpret_cast<uint4*>(sV + it * 16);
                if (row >= keys || (nodes && see[row] == 0)) {
                    *at = make_uint4(0, 0, 0, 0);
                } else if (nodes) {
                    uint32_t w[4] = {at->x, at->y, at->z, at->w};
                    bool any = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] = 0, any = true;
                    if (any) {
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                        atomicOr(&s_bad, 1ull << row);
                    }
                }
            }
            named_barrier(1, THREADS);
        }
        if (key0 < keys) {   // (warp-uniform)
            // A product's accumulator is cut, not rounded, at every step: short chains of them (16 dimensions; a
            // tile's keys) are summed by ordinary adds.
            float s[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
#pragma unroll 2
            for (int c = 0; c < n_steps / 2; ++c) {
                uint32_t bh[2][4], bl[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 k = piece(sK + (c >> 1) * PANEL, key0 + 8 * j + g, (c & 1) * 4 + t4);
                    split_cut(k.x, bh[j][0], bl[j][0]), split_cut(k.y, bh[j][1], bl[j][1]);
                    split_cut(k.z, bh[j][2], bl[j][2]), split_cut(k.w, bh[j][3], bl[j][3]);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint4* f = sQ + ((2 * c * MT * NG + group * MT + mt) * 2) * 32 + lane;
                    const uint4* f1 = f + MT * NG * 2 * 32;
                    const uint4 w[4] = {f[0], f[32], f1[0], f1[32]};
                    const uint32_t ah[2][4] = {{w[0].x, w[0].y, w[0].z, w[0].w}, {w[2].x, w[2].y, w[2].z, w[2].w}};
                    const uint32_t al[2][4] = {{w[1].x, w[1].y, w[1].z, w[1].w}, {w[3].x, w[3].y, w[3].z, w[3].w}};
                    float big[2][4] = {}, small[2][4] = {};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) mma(small[j], al[e], bh[j][2 * e], bh[j][2 * e + 1]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) mma(big[j], ah[e], bh[j][2 * e], bh[j][2 * e + 1]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) mma(small[j], ah[e], bl[j][2 * e], bl[j][2 * e + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][j][e] += big[j][e] + small[j][e];
                }
            }
            float x[MT][2][4], mx[MT][2], alpha[MT][2];   // [row g, g + 8][key 2 t, 2 t + 1, the same + 8]
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t live = nodes ? static_cast<uint32_t>(sees[mt][r] >> key0) : keys - key0 >= 16 ? 0xffffu : (1u << (keys - key0)) - 1;
                    mx[mt][r] = m[mt][r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = e >> 1, c = 2 * r + (e & 1);
                        x[mt][r][e] = (live >> (8 * j + 2 * t4 + (e & 1))) & 1 ? s[mt][j][c] * a.scale_log2 : -INFINITY;
                        mx[mt][r] = fmaxf(mx[mt][r], x[mt][r][e]);
                    }
                }
#pragma unroll
            for (int d = 1; d <= 2; ++d)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) mx[mt][r] = fmaxf(mx[mt][r], __shfl_xor_sync(0xffffffffu, mx[mt][r], d));
            uint32_t ph[MT][2][4], pl[MT][2][4];   // the weights as operands: {row g, g + 8} x {key 2 t, 2 t + 1}
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float off = mx[mt][r] == -INFINITY ? 0.f : mx[mt][r];
                    alpha[mt][r] = m[mt][r] == mx[mt][r] ? 1.f : exp2_approx(m[mt][r] - off);
                    m[mt][r] = mx[mt][r];
                    l[mt][r] *= alpha[mt][r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = exp2_approx(x[mt][r][e] - off);
                        l[mt][r] += p;
                        split(p, ph[mt][e >> 1][r + 2 * (e & 1)], pl[mt][e >> 1][r + 2 * (e & 1)]);
                    }
                }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (p >= n_panels) break;
                float tile[MT][4][4] = {};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = key0 + 8 * j + 2 * t4;
                    const float4 v0 = piece(sV + p * PANEL, row, g), v1 = piece(sV + p * PANEL, row + 1, g);
                    const float x0[4] = {v0.x, v0.y, v0.z, v0.w}, x1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {   // dimensions 4 n + q of the panel
                        uint32_t b0h, b0l, b1h, b1l;
                        split_cut(x0[q], b0h, b0l), split_cut(x1[q], b1h, b1l);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma(tile[mt][q], pl[mt][j], b0h, b1h);
                            mma(tile[mt][q], ph[mt][j], b0l, b1l);
                            mma(tile[mt][q], ph[mt][j], b0h, b1h);
                        }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][p][q][e] = fmaf(o[mt][p][q][e], alpha[mt][e >> 1], tile[mt][q][e]);
            }
        }
        fence_proxy_async_shared();   // what was read and cleared here before what the next copies write
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&empty[stage]);
        if (NG > 1 && tid == LOADER && t + STAGES * a.cluster <= n_cache) {
            ok = ok && mbar_wait(&empty[stage], (n / STAGES) & 1, abort_flag);
            if (ok) load_tile(t + STAGES * a.cluster, stage);
        }
        __syncwarp();
    }
    // No bulk copy may still target shared memory when it is used again below, or when the CTA exits.
    if (tid == LOADER)
        for (int i = 1; i <= STAGES && i <= issued; ++i) mbar_drain(&full[(issued - i) % STAGES], ((issued - i) / STAGES) & 1);
    __syncthreads();
    if (tid == 0 && *abort_flag) set_status(a.status, GPT_ERR_TIMEOUT);

    // In the ring's place: the first and third key warp leave their parts, the second and fourth join theirs to
    // them, then the two, then the CTAs'.
    float* sO = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[mt][r] += __shfl_xor_sync(0xffffffffu, l[mt][r], 1);
            l[mt][r] += __shfl_xor_sync(0xffffffffu, l[mt][r], 2);
        }
    const int half = key_warp >> 1;
    for (int w = 0; w < 2; ++w) {
        if ((key_warp & 1) == w && tid < THREADS) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = (group * MT + mt) * 16 + g + 8 * r;
                    const float2 old = w ? ml[half][i] : make_float2(-INFINITY, 0.f);
                    const bool have_old = old.y != 0.f, have = l[mt][r] != 0.f;
                    const float M = have_old ? have ? fmaxf(old.x, m[mt][r]) : old.x : m[mt][r];
                    const float f_old = !have_old ? 0.f : old.x == M ? 1.f : exp2_approx(old.x - M);
                    const float f = !have ? 0.f : m[mt][r] == M ? 1.f : exp2_approx(m[mt][r] - M);
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {   // four dimensions
                            float4* at = reinterpret_cast<float4*>(sO + (half * ROWS + i) * LD + p * 32 + 8 * t4 + 4 * e);
                            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (have_old) v = *at;
                            if (have_old) v.x *= f_old, v.y *= f_old, v.z *= f_old, v.w *= f_old;
                            if (have) {
                                v.x = fmaf(f, o[mt][p][0][2 * r + e], v.x), v.y = fmaf(f, o[mt][p][1][2 * r + e], v.y);
                                v.z = fmaf(f, o[mt][p][2][2 * r + e], v.z), v.w = fmaf(f, o[mt][p][3][2 * r + e], v.w);
                            }
                            *at = v;
                        }
                    __syncwarp();
                    if (t4 == 0) ml[half][i] = make_float2(M, (have_old ? old.y * f_old : 0.f) + (have ? l[mt][r] * f : 0.f));
                }
        }
        __syncthreads();
    }
    const bool alone = a.cluster == 1;
    float* out = y + static_cast<long long>(b) * N * C + h * hs;
    unsigned long long bad = s_bad;
    for (int it = tid; it < N * 4 * P; it += block_threads(NG)) {
        const int i = it / (4 * P), d = it % (4 * P) * 8;
        if (d >= hs) continue;
        Joined x;
        const float2 m0 = ml[0][i], m1 = ml[1][i];
        x.see(m0), x.see(m1);
        float* o0 = sO + i * LD + d;
        const float* o1 = o0 + ROWS * LD;
        if (m0.y != 0.f) x.add(m0, reinterpret_cast<const float4*>(o0)[0], reinterpret_cast<const float4*>(o0)[1]);
        if (m1.y != 0.f) x.add(m1, reinterpret_cast<const float4*>(o1)[0], reinterpret_cast<const float4*>(o1)[1]);
        if (alone) {
            if (see[i]) {
                x.finish(bad & see[i], node + 2 * C + d, 3 * C);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x.o[e] = 0.f;
            }
            st8(out + i * C + d, x.o);
        } else {
            st8(o0, x.o);
            if (d == 0) joined_ml[i] = make_float2(x.M, x.L);
        }
    }
    if (alone) return;
    __syncwarp();
    cluster_sync();
    const int holder = n_cache % a.cluster;   // of the nodes' tile
    bad = static_cast<unsigned long long>(ld_cluster_u32(map_to_rank(reinterpret_cast<uint32_t*>(&s_bad) + 1, holder))) << 32 |
          ld_cluster_u32(map_to_rank(&s_bad, holder));
    join_cluster(sO, LD, joined_ml, see, a, hs / 8, rank, out, C,
                 [&](int i, int d, Joined& x) { x.finish(bad & see[i], node + 2 * C + d, 3 * C); });
    __syncwarp();
    cluster_sync();
}

template <int P, int MT, int NG>
int launch(const CUtensorMap& node_map, const CUtensorMap& cache_map, const void* qkv, void* y, const TreeArgs& a,
           unsigned ctas, cudaStream_t s) {
    static size_t opted[kMaxDevices] = {};
    const int rc = opt_in_smem(reinterpret_cast<const void*>(tree_attention_f32<P, MT, NG>), smem_bytes<P, MT, NG>(), opted);
    if (rc) return rc;
    return launch_overlapped_cluster(tree_attention_f32<P, MT, NG>, a.cluster, dim3(ctas), dim3(block_threads(NG)),
                                     smem_bytes<P, MT, NG>(), s, node_map, cache_map, static_cast<const float*>(qkv),
                                     static_cast<float*>(y), a);
}
template <int P>
int launch(const CUtensorMap& node_map, const CUtensorMap& cache_map, const void* qkv, void* y, const TreeArgs& a,
           unsigned ctas, cudaStream_t s) {
    if (a.N <= 16) return launch<P, 1, 1>(node_map, cache_map, qkv, y, a, ctas, s);
    if (a.N <= 32) return launch<P, 2, 1>(node_map, cache_map, qkv, y, a, ctas, s);
    return launch<P, 2, 2>(node_map, cache_map, qkv, y, a, ctas, s);
}
}  // namespace f32

}  // namespace

int launch_tree_attention(int dtype, const void* qkv, const void* kv, const int* lengths, const int* parents, void* y,
                          int B, int N, int nh, int hs, int block_size, int32_t* status, cudaStream_t s) {
    TreeArgs a = {};
    a.lengths = lengths;
    a.parents = parents;
    a.B = B;
    a.N = N;
    a.nh = nh;
    a.hs = hs;
    a.block_size = block_size;
    a.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(hs)));
    a.status = status;
    const bool is_f32 = dtype == GPT_DTYPE_F32;
    const long long pairs = static_cast<long long>(B) * nh;
    const int tiles = (block_size - 1) / (is_f32 ? f32::KEYS : tc::KEYS) + 2;
    a.cluster = 1;
    // As many CTAs as run at a time; twice as many where a CTA keeps at least 24 tiles (fp32, whose tiles take
    // longer: 8), so that long sequences do not outlast the rest.  bf16, 12 x 20 nodes x 16 heads up to 8192
    // keys: 52 us with 2 CTAs a pair, 72 with 1; 18 x 20 x 16 up to 4096 keys: 43 and 43; 8 x 20 x 25 up to 1024:
    // 21 and 15.  fp32, 3 x 50 x 16 up to 2000 keys: 71, 52 and 86 us with 2, 4 and 8.
    const long long slots = 148 * (!is_f32 ? 2 : hs > 64 || N > 32 ? 1 : N > 16 ? 2 : 3);
    const int keep = is_f32 ? 8 : 24;
    while (a.cluster < 8 && a.cluster < tiles &&
           (pairs * a.cluster * 2 <= slots || (pairs * a.cluster <= slots && tiles >= keep * 2 * a.cluster)))
        a.cluster *= 2;
    // more CTAs than run at a time: those with the most work start first
    a.longest_first = !is_f32 && B > 1 && B <= tc::THREADS && pairs * a.cluster > slots;
    // bf16 without clusters: persistent CTAs
    const dim3 grid(static_cast<unsigned>((is_f32 || a.cluster > 1 || pairs < slots ? pairs : slots) * a.cluster));
    // {hs, heads of q, k, v (nodes) or k, v (cache), rows, sequences}
    const uint64_t heads = nh, row = heads * hs * (is_f32 ? 4 : 2), hs_bytes = row / heads;
    const uint64_t node_dims[4] = {static_cast<uint64_t>(hs), 3 * heads, static_cast<uint64_t>(N), static_cast<uint64_t>(B)};
    const uint64_t node_strides[3] = {hs_bytes, 3 * row, 3 * row * N};
    const uint64_t cache_dims[4] = {static_cast<uint64_t>(hs), 2 * heads, static_cast<uint64_t>(block_size), static_cast<uint64_t>(B)};
    const uint64_t cache_strides[3] = {hs_bytes, 2 * row, 2 * row * block_size};
    CUtensorMap node_map, cache_map, rest_map;
    int rc;
    if (is_f32) {
        const uint32_t box[4] = {32, 1, f32::KEYS, 1};
        rc = make_tmap_f32_4d(&node_map, qkv, node_dims, node_strides, box);
        if (!rc) rc = make_tmap_f32_4d(&cache_map, kv, cache_dims, cache_strides, box);
        if (rc) return rc;
        return hs <= 32   ? f32::launch<1>(node_map, cache_map, qkv, y, a, grid.x, s)
               : hs <= 64 ? f32::launch<2>(node_map, cache_map, qkv, y, a, grid.x, s)
                          : f32::launch<4>(node_map, cache_map, qkv, y, a, grid.x, s);
    }
    const bool twice = N <= 16;
    const uint32_t node_box[4] = {64, 1, static_cast<uint32_t>(tc::node_box(twice)), 1}, cache_box[4] = {64, 1, tc::KEYS, 1}, rest_box[4] = {64, 1, tc::BOX, 1};
    rc = make_tmap_bf16_4d(&node_map, qkv, node_dims, node_strides, node_box);
    if (!rc) rc = make_tmap_bf16_4d(&cache_map, kv, cache_dims, cache_strides, cache_box);
    if (!rc) rc = make_tmap_bf16_4d(&rest_map, kv, cache_dims, cache_strides, rest_box);
    if (rc) return rc;
    static size_t opted[3][kMaxDevices] = {};
    auto kern = twice ? tc::tree_attention_tc<32, true> : N <= 32 ? tc::tree_attention_tc<32, false> : tc::tree_attention_tc<64, false>;
    rc = opt_in_smem(reinterpret_cast<const void*>(kern), tc::SMEM, opted[twice ? 0 : N <= 32 ? 1 : 2]);
    if (rc) return rc;
    return launch_overlapped_cluster(kern, a.cluster, grid, dim3(tc::THREADS), tc::SMEM, s, node_map, cache_map, rest_map,
                                     static_cast<const bf16*>(qkv), static_cast<bf16*>(y), a);
}

// Pipeline-wait limit of this file's kernels on the current device (0: the default).
GPT_DEFINE_WAIT_LIMIT_SETTER(set_wait_limit_tree)

}  // namespace gpt
