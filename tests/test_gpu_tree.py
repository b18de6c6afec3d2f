"""Drafted trees on the GPU: the attention, the whole-model step, the acceptance, and decoding that uses
all three, against 64-bit definitions.

Tolerance of the attention, with u = 2^-24, a = sum_j p_j |v_j| of the exact probabilities, n keys and
D = max_j sum_d |q_d k_jd| / sqrt(hs): a score is off by at most (hs + 4) u D, its exponential's argument
by 2 u more of the scores' spread (at most 2 D), the exponential by 4 u, and the sums of p and of p v by
n u each, so y is off by 2 a ((hs + 8) u D + (n + 8) u).  bf16 rounds each p as an operand (a 2^-8 more;
the sum of p may be taken before or after that rounding) and y itself (2^-8 |y|).  fp32 takes each product
as three TF32 products, 20 u of it more, in both places.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import seeded
from gpu_helpers import BF16_ATOL, F32_ATOL, f64, max_abs, model_inputs, needs_gpu
from operator_refs import accept_ref, see_sets, tree_attention_ref

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def random_parents(B, N, seed, absent=True, chain=2):
    rng = np.random.default_rng(seed)
    par = np.full((B, N), -2, np.int32)
    for b in range(B):
        n = max(1, N - (b % 4 if absent else 0))
        for i in range(n):
            par[b, i] = i - 1 if i < chain else rng.integers(-1, i)
        par[b, 0] = -1
    return par


def attn_tol(qkv, kv, lens, nh, y, a, dtype):
    B, N, _, C = qkv.shape
    hs = C // nh
    tol = np.zeros_like(y)
    for b in range(B):
        n = int(lens[b])
        k = np.nan_to_num(np.abs(np.concatenate([kv[b, :n, 0], qkv[b, :, 1]])), posinf=0.0)
        D = np.einsum("ihd,jhd->ihj", np.abs(qkv[b, :, 0]).reshape(N, nh, hs), k.reshape(-1, nh, hs)).max(2) / np.sqrt(hs)
        tf32 = 20 if dtype == "f32" else 0
        rel = 2 * ((hs + 8 + tf32) * U * D + (n + N + 8 + tf32) * U)
        tol[b] = (a[b].reshape(N, nh, hs) * rel[:, :, None]).reshape(N, C)
    if dtype == "bf16":
        tol += 2.0 ** -8 * a * 1.01 + 2.0 ** -8 * (np.abs(y) + tol)
    else:
        tol += U * np.abs(y)
    return tol + 1e-30


def run_attention(B, N, nh, hs, cap, lens, par, dtype, seed=0, qscale=1.0, poison=True):
    from decoder_only_transformer_causal_b200 import native
    g = torch.Generator().manual_seed(seed)
    C = nh * hs
    qkv = torch.randn((B, N, 3, C), generator=g)
    qkv[:, :, 0] *= qscale
    qkv = qkv.to(DT[dtype])
    kv = torch.randn((B, cap, 2, C), generator=g).to(DT[dtype])
    if poison:                                   # what nobody sees may hold anything
        for b in range(B):
            kv[b, lens[b]:] = float("nan")
            for i, s in enumerate(see_sets(par)[b]):
                if not s:
                    qkv[b, i] = float("nan")
    d = [t.cuda() for t in (qkv, kv, torch.tensor(lens, dtype=torch.int32), torch.tensor(par))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = native.tree_attention(*d, nh, status=status)
    y2 = native.tree_attention(*d, nh)
    assert torch.equal(y, y2)
    q64, kv64 = f64(qkv), f64(kv)
    ref, a = tree_attention_ref(q64, kv64, lens, par, nh)
    tol = attn_tol(np.nan_to_num(q64), kv64, lens, nh, ref, a, dtype)
    err = np.abs(f64(y) - ref)
    assert np.isfinite(f64(y)).all()
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()), np.unravel_index((err - tol).argmax(), err.shape))
    return y, int(status.item()), d


CASES = [
    # B, N, nh, cap, lens
    (1, 1, 1, 1, [0]), (1, 1, 1, 1, [1]), (1, 1, 12, 1024, [700]), (2, 1, 4, 70, [63, 64]), (3, 1, 2, 300, [0, 65, 300]),
    (4, 7, 3, 200, [0, 1, 127, 200]), (4, 8, 4, 129, [128, 129, 64, 63]), (2, 16, 12, 1024, [1000, 3]),
    (5, 17, 2, 257, [256, 255, 257, 0, 31]), (4, 23, 5, 515, [515, 514, 192, 191]), (3, 32, 4, 100, [99, 32, 0]),
    (4, 33, 2, 300, [0, 128, 300, 5]), (4, 48, 3, 400, [400, 129, 65, 1]), (4, 64, 2, 700, [700, 640, 64, 0]),
    (1, 64, 1, 5000, [4999]), (1, 5, 1, 9000, [8191]), (70, 3, 16, 130, [(13 * i) % 131 for i in range(70)]),
    (12, 64, 16, 70, [6 * i for i in range(12)]),
    (40, 50, 12, 300, [(77 * i) % 301 for i in range(40)]),      # more pairs than run at a time, 64-row groups
    (200, 2, 2, 40, [(7 * i) % 41 for i in range(200)]),         # ... and too many sequences to order
]


@pytest.mark.parametrize("dtype,hs", [("bf16", 64), ("f32", 64), ("f32", 8), ("f32", 40), ("f32", 128)])
@pytest.mark.parametrize("B,N,nh,cap,lens", CASES)
def test_tree_attention(B, N, nh, cap, lens, dtype, hs):
    if hs in (8, 40, 128) and cap > 1024:
        nh = 1
    _, status, _ = run_attention(B, N, nh, hs, cap, lens, random_parents(B, N, seed=N), dtype, seed=cap)
    assert status == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qscale", [0.0, 30.0, 300.0])
def test_tree_attention_score_ranges(qscale, dtype):
    """From uniform weights to a single key taking nearly all of the weight."""
    run_attention(3, 21, 2, 64, 400, [399, 64, 0], random_parents(3, 21, 5), dtype, qscale=qscale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 6, 16, 40, 64])
def test_tree_attention_shapes_of_trees(N, dtype):
    """A chain, a star (every node a root, every node a child of the first), and broken parents."""
    from decoder_only_transformer_causal_b200 import native
    par = np.full((5, N), -2, np.int32)
    par[0] = np.arange(N) - 1
    par[1] = -1
    par[2, 0], par[2, 1:] = -1, 0
    par[4] = np.arange(N)                        # each its own parent: none is a node
    _, status, _ = run_attention(5, N, 2, 64, 200, [130, 7, 200, 150, 60], par, dtype)
    assert status == native.GPT_ERR_INDEX
    par[4] = -2
    assert run_attention(5, N, 2, 64, 200, [130, 7, 200, 150, 60], par, dtype)[1] == 0
    for bad in (N, N + 5, -3, 1 << 30, -(1 << 31)):
        par[4, 0] = bad
        assert run_attention(5, N, 2, 64, 200, [130, 7, 200, 150, 60], par, dtype)[1] == native.GPT_ERR_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_bad_lengths(dtype):
    from decoder_only_transformer_causal_b200 import native
    B, N, nh, cap = 3, 4, 2, 50
    par = random_parents(B, N, 1)
    y, _, (qkv, kv, _, p) = run_attention(B, N, nh, 64, cap, [0, 50, 20], par, dtype, poison=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([-5, 51, 20], dtype=torch.int32, device="cuda")
    assert torch.equal(native.tree_attention(qkv, kv, bad, p, nh, status=status), y)
    assert int(status.item()) == native.GPT_ERR_BAD_SHAPE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [9, 64])
def test_tree_attention_branches_do_not_mix(N, dtype):
    """Bits of a row depend on the row's own path only: NaN in every other node changes nothing."""
    from decoder_only_transformer_causal_b200 import native
    y, _, (qkv, kv, lens, par) = run_attention(2, N, 2, 64, 300, [300, 77], random_parents(2, N, 2, absent=False), dtype)
    for i in (0, N // 2, N - 1):
        q2 = torch.full_like(qkv, float("nan"))
        for b in range(2):
            keep = sorted(see_sets(par.cpu().numpy())[b][i])
            q2[b, keep] = qkv[b, keep]
        y2 = native.tree_attention(q2, kv, lens, par, 2)
        assert torch.equal(y2[:, i], y[:, i])


def test_tree_attention_values_that_are_not_numbers():
    """A visible key or value that is NaN or infinite reaches the rows that see it, and no others."""
    from decoder_only_transformer_causal_b200 import native
    for dtype in ("bf16", "f32"):
        y, _, (qkv, kv, lens, par) = run_attention(2, 5, 2, 64, 300, [300, 77], random_parents(2, 5, 2, absent=False), dtype)
        kv[1, 70, 1, 64 + 3] = float("nan")      # sequence 1, head 1, dimension 3
        y2 = native.tree_attention(qkv, kv, lens, par, 2)
        assert torch.isnan(y2[1, :, 64 + 3]).all()
        y2[1, :, 64 + 3] = y[1, :, 64 + 3]
        assert torch.equal(y2, y)


@pytest.mark.parametrize("dtype,hs", [("bf16", 64), ("f32", 64), ("f32", 8), ("f32", 128)])
@pytest.mark.parametrize("N", [5, 20, 50])
def test_tree_attention_largest_queries(N, dtype, hs):
    """Queries of the type's largest values against keys that are 0 or tiny there: scores are ordinary numbers."""
    from decoder_only_transformer_causal_b200 import native
    B, nh, cap, lens, par = 3, 2, 300, [300, 77, 0], random_parents(3, N, 3)
    g = torch.Generator().manual_seed(N)
    qkv, kv = torch.randn((B, N, 3, nh * hs), generator=g), torch.randn((B, cap, 2, nh * hs), generator=g)
    sign = torch.randint(0, 2, (B, N, nh), generator=g) * 2.0 - 1
    qkv, kv = qkv.to(DT[dtype]), kv.to(DT[dtype])
    qkv[:, :, 0, 1::hs] = (sign * torch.finfo(DT[dtype]).max).to(DT[dtype])
    qkv[:, :, 1, 1::hs] = (torch.randint(-1, 2, (B, N, nh), generator=g) * 2.0 ** -123).to(DT[dtype])
    kv[:, :, 0, 1::hs] = (torch.randint(-1, 2, (B, cap, nh), generator=g) * 2.0 ** -123).to(DT[dtype])
    y = f64(native.tree_attention(qkv.cuda(), kv.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(par).cuda(), nh))
    q64, kv64 = f64(qkv), f64(kv)
    ref, a = tree_attention_ref(q64, kv64, lens, par, nh)
    tol = attn_tol(q64, kv64, lens, nh, ref, a, dtype)
    assert (np.abs(y - ref) <= tol).all(), float(np.abs(y - ref).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 40])
def test_tree_attention_offsets_past_32_bits(N, dtype):
    from decoder_only_transformer_causal_b200 import native
    cap = (1 << 25) + 3 if dtype == "bf16" else (1 << 24) + 3
    kv = torch.empty((2, cap, 2, 64), dtype=DT[dtype], device="cuda")     # 8.6 GB a sequence
    small = torch.randn((2, 150, 2, 64), generator=torch.Generator().manual_seed(4)).to(DT[dtype])
    kv[:, :150] = small.cuda()
    qkv = torch.randn((2, N, 3, 64), generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    par, lens = random_parents(2, N, 7), [100, 149]
    y = native.tree_attention(qkv.cuda(), kv, torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(par).cuda(), 1)
    ref, a = tree_attention_ref(f64(qkv), f64(small), lens, par, 1)
    assert (np.abs(f64(y) - ref) <= attn_tol(f64(qkv), f64(small), lens, 1, ref, a, dtype)).all()


@pytest.mark.parametrize("N", [3, 50])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_streams_and_graph_replay(N, dtype):
    """A recorded call follows lengths, parents and values that change between replays."""
    from decoder_only_transformer_causal_b200 import native
    y, _, (qkv, kv, lens, par) = run_attention(3, N, 2, 64, 300, [300, 77, 1], random_parents(3, N, 3), dtype, poison=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert torch.equal(native.tree_attention(qkv, kv, lens, par, 2), y)
    s.synchronize()
    l2, p2 = torch.zeros_like(lens), torch.full_like(par, -2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = native.tree_attention(qkv, kv, l2, p2, 2)
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 0).all()
    l2.copy_(lens), p2.copy_(par)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_calls_at_once(dtype):
    """Calls in flight together on two streams share nothing."""
    from decoder_only_transformer_causal_b200 import native
    args, want = [], []
    for N, nh in ((5, 12), (40, 12)):
        y, _, d = run_attention(30, N, nh, 64, 400, [(37 * i) % 401 for i in range(30)], random_parents(30, N, N), dtype, seed=N)
        args.append(d + [nh])
        want.append(y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(native.tree_attention(*args[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


@pytest.mark.parametrize("B,N,nh,cap,lens", [
    (1, 1, 12, 1024, [700]), (3, 1, 2, 300, [0, 65, 300]), (2, 16, 12, 1024, [1000, 3]), (5, 17, 2, 257, [256, 255, 257, 0, 31]),
    (4, 23, 5, 515, [515, 514, 192, 191]), (3, 32, 4, 130, [130, 32, 0]), (4, 33, 2, 300, [0, 128, 300, 5]),
    (4, 64, 2, 700, [700, 640, 64, 0]), (1, 64, 1, 5000, [4999]), (70, 3, 16, 130, [(13 * i) % 131 for i in range(70)]),
    (40, 20, 16, 300, [(77 * i) % 301 for i in range(40)]), (40, 50, 12, 300, [(77 * i) % 301 for i in range(40)])])
@pytest.mark.parametrize("qscale", [0.3, 3.0])
def test_tree_attention_keeps_the_weights_bits(B, N, nh, cap, lens, qscale):
    """bf16: a weight is off by 2^-15 of itself (its upper 16 bits and the rest, off by half a step, 2^-8, of at most
    2^-7 of it), where one bf16 number would be off by 2^-8; everything else as in the tolerance above."""
    from decoder_only_transformer_causal_b200 import native
    g = torch.Generator().manual_seed(cap + N)
    qkv = torch.randn((B, N, 3, nh * 64), generator=g)
    qkv[:, :, 0] *= qscale
    qkv = qkv.to(torch.bfloat16)
    kv = torch.randn((B, cap, 2, nh * 64), generator=g).to(torch.bfloat16)
    par = random_parents(B, N, seed=N)
    y = f64(native.tree_attention(qkv.cuda(), kv.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(par).cuda(), nh))
    q64, kv64 = f64(qkv), f64(kv)
    ref, a = tree_attention_ref(q64, kv64, lens, par, nh)
    tol = attn_tol(q64, kv64, lens, nh, np.zeros_like(ref), a, "f32") + 2.0 ** -15 * a     # of the sums
    tol += 2.0 ** -8 * (np.abs(ref) + tol)                                                 # of the result's rounding
    err = np.abs(y - ref)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()), np.unravel_index((err - tol).argmax(), err.shape))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [9, 20, 64])
@pytest.mark.parametrize("B,nh,cap", [(2, 2, 400), (30, 12, 300)])
def test_tree_attention_nodes_with_values_that_are_not_numbers(B, nh, cap, N, dtype):
    """A node's key or value that is NaN or infinite reaches the rows that see the node, in the value's dimensions
    (a key: in all of its head), and leaves every other bit as it is: with clusters (few pairs) and without, for
    nodes below and above the 32nd."""
    from decoder_only_transformer_causal_b200 import native
    par = random_parents(B, N, 3)
    lens = [(77 * i + 300) % (cap + 1) for i in range(B)]
    y, _, (qkv, kv, l, p) = run_attention(B, N, nh, 64, cap, lens, par, dtype, seed=N, poison=False)
    sees = see_sets(par)
    inf, nan = float("inf"), float("nan")

    def compare(bad, want):
        y2 = native.tree_attention(bad, kv, l, p, nh)
        both = torch.isnan(want) & torch.isnan(y2)
        assert torch.equal(torch.where(both, 0, y2), torch.where(both, 0, want))

    for first in (1, N // 2, N - 4):             # values: one node, then another with the opposite infinity
        bad, want = qkv.clone(), y.clone()
        for b in range(B):
            for node, vals in ((first, (inf, -inf, nan)), (0, (0, inf, -inf))):
                for i in range(N):
                    if node in sees[b][i]:
                        for d, v in zip((3, 40, 63), vals):
                            want[b, i, 64 * (nh - 1) + d] += v if v else 0
                for d, v in zip((3, 40, 63), vals):
                    if v:
                        bad[b, node, 2, 64 * (nh - 1) + d] = v
        compare(bad, want)
        bad, want = qkv.clone(), y.clone()       # keys: NaN, and an infinity that every query meets with its sign
        bad[:, :, 0, 5] = bad[:, :, 0, 5].abs() + 0.5
        y3 = native.tree_attention(bad, kv, l, p, nh)
        for key in (nan, inf):
            bad[:, first, 1, 5] = key
            want = y3.clone()
            for b in range(B):
                for i in range(N):
                    if first in sees[b][i]:
                        want[b, i, :64] = nan
            compare(bad, want)


# ------------------------------------------------------------------ the model over a tree
def tree_model(name, layers, B, T0, **over):
    from decoder_only_transformer_causal_b200 import GPT, GPTConfig, native
    over = dict(over, **({"n_layer": layers} if layers else {}))
    cfg, W, W64, _, _ = model_inputs(name, stress=True, **over)
    m = GPT(GPTConfig.from_dict(cfg), W)
    prompt, _ = seeded.make_tokens(B, T0, min(cfg["vocab_size"], 50257), seed=9101)
    kv = native.alloc_kv_cache(m.cfg, B)
    ws = native.alloc_workspace(native.decode_workspace_bytes(m.cfg, B, T0))
    native.prefill(m.cfg, m.weights, prompt.cuda(), kv, ws, sync_check=True)
    return m, cfg, W64, prompt, kv


STEP_CASES = [
    ("tiny", None, 3, 40, 9, [40, 13, 1]),
    ("tiny", None, 2, 60, 4, [60, 0]),             # the last positions of the window; an empty cache
    ("gpt2", 2, 2, 130, 13, [130, 64]),
    ("gpt2", 2, 1, 20, 1, [20]),
    ("gpt2", 2, 2, 40, 64, [40, 7]),
]


@pytest.mark.parametrize("name,layers,B,T0,N,lens", STEP_CASES)
def test_tree_step_matches_forward(name, layers, B, T0, N, lens):
    from decoder_only_transformer_causal_b200 import native
    m, cfg, W64, prompt, kv = tree_model(name, layers, B, T0)
    V = min(cfg["vocab_size"], 50257)
    tok, _ = seeded.make_tokens(B, N, V, seed=9102)
    par = random_parents(B, N, 11)
    before = kv.clone()
    tq = native.alloc_tree_qkv(m.cfg, B, N)
    logits = native.tree_step(m.cfg, m.weights, tok.cuda(), torch.tensor(par).cuda(),
                              torch.tensor(lens, dtype=torch.int32).cuda(), kv, tq, m.workspace(B, N), sync_check=True)
    assert torch.equal(kv, before)
    got = f64(logits)
    tol = F32_ATOL if cfg["dtype"] == "f32" else BF16_ATOL
    sees = see_sets(par)
    pick = range(N) if N <= 16 else sorted({0, 1, N // 3, N // 2, N - 5, N - 4})
    for b in range(B):
        for i in pick:
            nodes = sorted(sees[b][i])
            if not nodes or lens[b] + len(nodes) > cfg["block_size"]:
                continue
            seq = np.concatenate([prompt[b, :lens[b]].numpy(), tok[b, nodes].numpy()])[None]
            ref = oracle.forward(W64, cfg, seq, None)["logits"][0, -1]
            assert max_abs(got[b, i], ref) <= tol, (b, i)


def test_tree_step_reports_what_is_wrong():
    from decoder_only_transformer_causal_b200 import native
    m, cfg, _, _, kv = tree_model("tiny", None, 1, 60)
    tq = native.alloc_tree_qkv(m.cfg, 1, 6)

    def step(tok, par, length):
        return native.tree_step(m.cfg, m.weights, torch.tensor([tok]).cuda(), torch.tensor([par], dtype=torch.int32).cuda(),
                                torch.tensor([length], dtype=torch.int32).cuda(), kv, tq, m.workspace(1, 6), sync_check=True)
    chain = [-1, 0, 1, 2, 3, 4]
    step([1, 2, 3, 4, 5, 6], chain, 58)
    step([1, 2, 3, 4, 5, 10 ** 9], chain[:5] + [-2], 58)          # an absent node's token does not matter
    for tok, par, length, code in (([1, 2, 3, 4, 5, 65], chain, 58, native.GPT_ERR_INDEX),
                                   ([1, 2, 3, 4, 5, -1], chain, 58, native.GPT_ERR_INDEX),
                                   ([1] * 6, chain[:5] + [5], 58, native.GPT_ERR_INDEX),
                                   ([1] * 6, chain, 59, native.GPT_ERR_BAD_SHAPE),
                                   ([1] * 6, chain, 65, native.GPT_ERR_BAD_SHAPE)):
        with pytest.raises(native.GPTError) as e:
            step(tok, par, length)
        assert e.value.status == code, (tok, par, length)


# ------------------------------------------------------------------ acceptance
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,L,cap,seed", [(1, 1, 1, 8, 0), (7, 5, 3, 40, 1), (9, 31, 2, 33, 2), (12, 64, 2, 70, 3), (66, 33, 1, 64, 4)])
def test_tree_accept(B, N, L, cap, seed, dtype):
    from decoder_only_transformer_causal_b200 import GPTConfig, native
    cfg = GPTConfig(n_layer=L, n_head=2, n_embd=128, block_size=cap, vocab_size=64, dtype=dtype)
    rng = np.random.default_rng(seed)
    par = random_parents(B, N, seed, chain=1)
    par[B // 2] = -2                                     # a sequence with no node
    tok = rng.integers(0, 3, (B, N)) + (1 << 40)         # few tokens: many paths agree; beyond 32 bits
    cho = rng.integers(0, 3, (B, N)) + (1 << 40)
    lens = rng.integers(0, cap + 1, B).astype(np.int32)
    lens[0] = cap if B > 1 else 3
    g = torch.Generator().manual_seed(seed)
    tq = torch.randn((L, B, N, 3, 128), generator=g).to(DT[dtype]).cuda()
    kv = torch.randn((L, B, cap, 2, 128), generator=g).to(DT[dtype]).cuda()
    want = kv.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = [torch.tensor(v).cuda() for v in (par, tok, cho, lens)]
    r = native.tree_accept(cfg, *dev, tq, kv, status=status)
    paths, counts, nxt = accept_ref(par, tok, cho, lens, cap)
    assert int(status.item()) == 0
    assert r.n_accepted.tolist() == counts and r.next_token.tolist() == nxt
    assert r.lengths.tolist() == [int(n) + c for n, c in zip(lens, counts)]
    assert r.path.tolist() == [p + [-1] * (N - len(p)) for p in paths]
    for b, p in enumerate(paths):
        for j, node in enumerate(p):
            want[:, b, lens[b] + j] = tq[:, b, node, 1:]
    assert torch.equal(kv, want)
    # the new lengths in the place of the old ones
    kv2 = want.clone()
    out = native.TreeAccept(torch.empty_like(r.path), torch.empty_like(r.n_accepted), torch.empty_like(r.next_token), dev[3])
    native.tree_accept(cfg, *dev, tq, kv2, out=out)
    assert torch.equal(out.lengths, r.lengths) and torch.equal(out.path, r.path) and torch.equal(kv2, want)


def test_tree_accept_reports_bad_parents_and_lengths():
    from decoder_only_transformer_causal_b200 import GPTConfig, native
    cfg = GPTConfig(n_layer=1, n_head=1, n_embd=64, block_size=8, vocab_size=64, dtype="bf16")
    tq, kv = torch.zeros((1, 1, 3, 3, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((1, 1, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    tok = torch.tensor([[1, 2, 3]], device="cuda")
    for par, length, code, n in (([-1, 1, 0], 2, native.GPT_ERR_INDEX, 2), ([5, 0, -9], 2, native.GPT_ERR_INDEX, 0),
                                 ([-1, 0, -2], 9, native.GPT_ERR_BAD_SHAPE, 0), ([-1, 0, -2], -1, native.GPT_ERR_BAD_SHAPE, 2)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cho = torch.tensor([[2 if par[1] == 0 else 3, 7, 7]], device="cuda")
        r = native.tree_accept(cfg, torch.tensor([par], dtype=torch.int32, device="cuda"), tok, cho,
                               torch.tensor([length], dtype=torch.int32, device="cuda"), tq, kv, status=status)
        assert int(status.item()) == code and r.n_accepted.item() == n, par
        assert r.lengths.item() == min(max(length, 0), 8) + n


# ------------------------------------------------------------------ all of them together
@pytest.mark.parametrize("name,layers,new", [("tiny", None, 30), ("gpt2", 2, 14)])
def test_drafted_greedy_decoding_gives_the_greedy_tokens(name, layers, new):
    """Draft a tree, score it in one step, choose with the top alternative, keep the confirmed path: the
    tokens are those of a greedy generation as long as its choices are not within rounding of a tie."""
    from decoder_only_transformer_causal_b200 import native
    B, T0, N = 3, 12, 7
    m, cfg, W64, prompt, kv = tree_model(name, layers, B, T0)
    greedy = m.generate(prompt.cuda(), new, top_k=1, uniforms=torch.zeros((new, B), device="cuda")).cpu()
    tol = F32_ATOL if cfg["dtype"] == "f32" else BF16_ATOL
    # the cache is refilled: the loop below keeps prompt[:-1] and starts from the last token
    lens = torch.full((B,), T0 - 1, dtype=torch.int32, device="cuda")
    root = prompt[:, -1].clone()
    par = torch.tensor([[-1, 0, 0, 1, 2, 4, 5]] * B, dtype=torch.int32)
    tq, ws = native.alloc_tree_qkv(m.cfg, B, N), m.workspace(B, N)
    got = [[] for _ in range(B)]
    rng = np.random.default_rng(0)
    steps = 0
    while min(len(g) for g in got) < new and int(lens.max()) + N <= cfg["block_size"]:
        tok = torch.tensor(rng.integers(0, min(cfg["vocab_size"], 50257), (B, N)))
        for b in range(B):                       # a draft that is often right: the path 0-2-4-5-6
            at = T0 + len(got[b])
            for j, node in enumerate((2, 4, 5, 6)):
                if at + j < T0 + new and rng.random() < 0.8:
                    tok[b, node] = greedy[b, at + j]
        tok[:, 0] = root
        logits = native.tree_step(m.cfg, m.weights, tok.cuda(), par.cuda(), lens, kv, tq, ws, sync_check=True)
        flat = native.token_logprobs(logits.view(B * N, -1), None, k=2)
        chosen = flat.top_ids[:, 0].reshape(B, N).contiguous()
        acc = native.tree_accept(m.cfg, par.cuda(), tok.cuda(), chosen, lens, tq, kv)
        for b in range(B):
            n = int(acc.n_accepted[b])
            path = acc.path[b, :n].tolist()
            assert path[0] == 0
            got[b] += [int(chosen[b, i]) for i in path]
        lens, root = acc.lengths, acc.next_token.cpu()
        steps += 1
    assert steps < max(len(g) for g in got)      # some drafted tokens were kept
    for b in range(B):
        for s, g in enumerate(got[b][:new]):
            if g != int(greedy[b, T0 + s]):      # allowed only where the two best logits nearly tie
                z = oracle.forward(W64, cfg, greedy[b:b + 1, :T0 + s].numpy(), None)["logits"][0, -1]
                assert z.max() - z[g] <= 2 * tol, (b, s)
                break


def test_other_streams_and_graph_of_a_whole_step():
    """tree_step, the choice and the acceptance recorded once and replayed as the cache grows."""
    from decoder_only_transformer_causal_b200 import native
    B, T0, N = 2, 10, 5
    m, cfg, _, prompt, kv = tree_model("tiny", None, B, T0)
    kv0 = kv.clone()
    par = torch.tensor([[-1, 0, 1, 0, 3]] * B, dtype=torch.int32, device="cuda")
    toks = [torch.randint(0, 65, (B, N), generator=torch.Generator().manual_seed(i)).cuda() for i in range(3)]
    tq, ws = native.alloc_tree_qkv(m.cfg, B, N), m.workspace(B, N)
    tok, lens = torch.zeros((B, N), dtype=torch.int64, device="cuda"), torch.full((B,), T0, dtype=torch.int32, device="cuda")
    out = native.TreeAccept(torch.empty((B, N), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"),
                            torch.empty(B, dtype=torch.int64, device="cuda"), lens)

    def step():
        logits = native.tree_step(m.cfg, m.weights, tok, par, lens, kv, tq, ws)
        ids = native.token_logprobs(logits.view(B * N, -1), None, k=1).top_ids
        native.tree_accept(m.cfg, par, tok, ids.view(B, N), lens, tq, kv, out=out)

    def run(go):
        kv.copy_(kv0)
        lens.fill_(T0)
        seen = []
        for t in toks:
            tok.copy_(t)
            go()
            seen.append([x.clone() for x in out] + [kv.clone()])
        return seen
    eager = run(step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = run(step)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    replayed = run(graph.replay)
    torch.cuda.synchronize()
    for a, b, c in zip(eager, side, replayed):
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and all(torch.equal(x, y) for x, y in zip(a, c))


def test_model_calls():
    """GPT.verify is tree_step, the likeliest token and tree_accept; GPT.score is the log probabilities of
    the forward's logits."""
    from decoder_only_transformer_causal_b200 import native
    B, T0, N = 2, 10, 5
    m, cfg, W64, prompt, kv = tree_model("tiny", None, B, T0)
    par = torch.tensor([[-1, 0, 1, 0, 3]] * B, dtype=torch.int32, device="cuda")
    tok = torch.randint(0, 65, (B, N), generator=torch.Generator().manual_seed(1)).cuda()
    lens = torch.full((B,), T0, dtype=torch.int32, device="cuda")
    kv2, tq = kv.clone(), native.alloc_tree_qkv(m.cfg, B, N)
    logits = native.tree_step(m.cfg, m.weights, tok, par, lens, kv2, tq, m.workspace(B, N))
    want = native.tree_accept(m.cfg, par, tok, logits.argmax(-1), lens, tq, kv2)
    acc, chosen = m.verify(tok, par, lens, kv)
    assert torch.equal(chosen, logits.argmax(-1))
    assert all(torch.equal(a, b) for a, b in zip(acc, want)) and torch.equal(kv, kv2)

    idx, tgt = seeded.make_tokens(3, 20, 65, seed=77, ignore_frac=0.2)
    r = m.score(idx.cuda(), tgt.cuda(), k=4)
    z = oracle.forward(W64, cfg, idx.numpy(), None if tgt is None else tgt.numpy())["logits"]
    lp = z - np.log(np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)) - z.max(-1, keepdims=True)
    ref = np.where(tgt.numpy() >= 0, np.take_along_axis(lp, np.maximum(tgt.numpy(), 0)[..., None], -1)[..., 0], 0)
    # a log probability moves by at most twice what the logits do
    assert max_abs(f64(r.logp), ref) <= 2 * F32_ATOL and r.top_ids.shape == (3, 20, 4)
    assert max_abs(f64(r.entropy), -(np.exp(lp) * lp).sum(-1)) <= 2 * F32_ATOL * (1 + np.abs(lp).max())


def test_verify_keeps_no_buffers():
    """Batches and draft widths that vary leave nothing behind but the model's workspace."""
    B, T0 = 4, 10
    m, cfg, _, _, kv = tree_model("tiny", None, B, T0)

    def verify(B, N):
        par = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(B, 1)
        m.verify(torch.ones((B, N), dtype=torch.int64, device="cuda"), par, torch.full((B,), T0, dtype=torch.int32, device="cuda"), kv)
        torch.cuda.synchronize()
    verify(B, 12)
    held = torch.cuda.memory_allocated()
    for b in range(1, B + 1):
        for n in range(1, 13):
            verify(b, n)
    assert torch.cuda.memory_allocated() == held


def test_verify_and_score_report_what_is_wrong():
    from decoder_only_transformer_causal_b200 import native
    m, cfg, _, _, kv = tree_model("tiny", None, 1, 20)
    chain = [-1, 0, 1, 2]

    def verify(tok, par, length, **kw):
        return m.verify(torch.tensor([tok]).cuda(), torch.tensor([par], dtype=torch.int32).cuda(),
                        torch.tensor([length], dtype=torch.int32).cuda(), kv, **kw)
    verify([1, 2, 3, 4], chain, 20, sync_check=True)
    for tok, par, length, code in (([1, 65, 3, 4], chain, 20, native.GPT_ERR_INDEX), ([1, 2, -1, 4], chain, 20, native.GPT_ERR_INDEX),
                                   ([1, 2, 3, 4], [-1, 0, 2, 1], 20, native.GPT_ERR_INDEX), ([1, 2, 3, 4], chain, -1, native.GPT_ERR_BAD_SHAPE),
                                   ([1, 2, 3, 4], chain, 65, native.GPT_ERR_BAD_SHAPE)):
        with pytest.raises(native.GPTError) as e:
            verify(tok, par, length, sync_check=True)
        assert e.value.status == code, (tok, par, length)
        verify(tok, par, length)
        assert native.check_status(m.workspace(1, 4)) == code
    verify([1, 2, 3, 4], chain, 20, sync_check=True)              # an error is not kept for the next call

    idx, tgt = torch.randint(0, 65, (2, 9)), torch.randint(0, 65, (2, 9))
    tgt[0, 3] = -1
    m.score(idx.cuda(), tgt.cuda(), k=2, sync_check=True)
    for i, t in ((idx, 65), (idx, -1), (tgt, 65), (tgt, -2)):
        keep = i[1, 4].item()
        i[1, 4] = t
        with pytest.raises(native.GPTError) as e:
            m.score(idx.cuda(), tgt.cuda(), k=2, sync_check=True)
        assert e.value.status == native.GPT_ERR_INDEX, t
        m.score(idx.cuda(), tgt.cuda())
        assert native.check_status(m.workspace(2, 9)) == native.GPT_ERR_INDEX
        i[1, 4] = keep
    m.score(idx.cuda(), tgt.cuda(), sync_check=True)


def test_verify_and_score_of_a_padded_vocabulary():
    """Columns behind the last token are neither chosen nor counted."""
    from decoder_only_transformer_causal_b200 import native
    B, T0, N = 2, 10, 5
    m, cfg, _, prompt, kv = tree_model("tiny", None, B, T0)
    par = torch.tensor([[-1, 0, 1, 0, 3]] * B, dtype=torch.int32, device="cuda")
    tok = torch.randint(0, 65, (B, N), generator=torch.Generator().manual_seed(1)).cuda()
    lens = torch.full((B,), T0, dtype=torch.int32, device="cuda")
    kv2, tq = kv.clone(), native.alloc_tree_qkv(m.cfg, B, N)
    logits = native.tree_step(m.cfg, m.weights, tok, par, lens, kv2, tq, m.workspace(B, N))
    real = int(logits.argmax(-1).max())                           # the last of the likeliest is padding
    assert real > 1
    acc, chosen = m.verify(tok, par, lens, kv, vocab=real, sync_check=True)
    assert torch.equal(chosen, logits[..., :real].argmax(-1))
    want = native.tree_accept(m.cfg, par, tok, chosen, lens, tq, kv2)
    assert all(torch.equal(a, b) for a, b in zip(acc, want)) and torch.equal(kv, kv2)

    idx, tgt = (t % real for t in seeded.make_tokens(3, 20, 65, seed=77))
    r = m.score(idx.cuda(), tgt.cuda(), k=4, vocab=real, sync_check=True)
    z = f64(m(idx.cuda(), tgt.cuda())[0])[..., :real]
    lp = z - np.log(np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)) - z.max(-1, keepdims=True)
    # logits of the same kernels: what is left are fp32 roundings of values below 32 (2^-24 * 32, four of them)
    assert max_abs(f64(r.logp), np.take_along_axis(lp, tgt.numpy()[..., None], -1)[..., 0]) <= 2.0 ** -17
    assert max_abs(f64(r.entropy), -(np.exp(lp) * lp).sum(-1)) <= 2.0 ** -17 and int(r.top_ids.max()) < real
    with pytest.raises(native.GPTError):                          # a target in the padding
        m.score(idx.cuda(), torch.full_like(tgt, real).cuda(), vocab=real, sync_check=True)
    for bad in (0, -1, 66):
        with pytest.raises(ValueError):
            m.score(idx.cuda(), tgt.cuda(), vocab=bad)
        with pytest.raises(ValueError):
            m.verify(tok, par, lens, kv, vocab=bad)


def test_captured_calls_outlive_a_larger_workspace():
    """A recorded GPT.verify and forward stay right, and write into nobody else's memory, after a larger call has
    replaced the model's workspace."""
    from decoder_only_transformer_causal_b200 import native
    B, T0, N = 2, 10, 5
    m, cfg, _, prompt, kv = tree_model("tiny", None, B, T0)
    kv0 = kv.clone()
    par = torch.tensor([[-1, 0, 1, 0, 3]] * B, dtype=torch.int32, device="cuda")
    tok = torch.randint(0, 65, (B, N), generator=torch.Generator().manual_seed(1)).cuda()
    lens = torch.full((B,), T0, dtype=torch.int32, device="cuda")
    want, chosen = m.verify(tok, par, lens, kv)
    want, after = [t.clone() for t in (*want, chosen)], kv.clone()
    logits, _ = m(tok, tok)
    logits = logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        acc, got = m.verify(tok, par, lens, kv)
        z, _ = m(tok, tok)
    size = m.workspace(B, N).numel()
    idx = torch.zeros((64, 64), dtype=torch.int64, device="cuda")
    m(idx, idx)                                       # a larger workspace
    assert m.workspace(B, N).numel() > size
    canaries = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(2):
        kv.copy_(kv0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*acc, got), want)) and torch.equal(kv, after) and torch.equal(z, logits)
        assert all((c == 7).all() for c in canaries)
