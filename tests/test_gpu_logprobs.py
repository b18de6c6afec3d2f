"""Token log probabilities, entropy, top alternatives and their gradient against the 64-bit definitions.

Tolerances.  u = 2^-24 is half a step of fp32.  A kernel that takes p_v ~ exp(e_v), e_v = z_v - max z, in
fp32 has a relative error of at most (3 |e_v| + 4) u in each term (the scaled logit, the subtraction, the
exponential's argument, and its own 2 ulp) and depth u from summing (depth: the adds that one partial sum
goes through).  With A = sum p |e|, M2 = sum p e^2 (of the exact p):
  sum of p:     r = (3 A + 4 + depth) u, relative
  lse:          r + u (3 |max| + 2 |lse| + 2 ln V)
  log p of v:   r + u (4 |e_v| + 2 ln V + |log p|)
  entropy:      r (1 + A) + u (3 M2 + (8 + depth) A + 2 ln V + H)
"""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import f64, needs_gpu
from operator_refs import logprob_grad_ref, logprob_ref

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def close(got, ref, tol, what):
    """|got - ref| <= tol where ref is finite, the same infinities and NaN elsewhere."""
    got = np.asarray(got, np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)]), what
    with np.errstate(invalid="ignore"):
        # a row without a finite maximum has no bound (NaN): what is finite there, the 0 of an ignored row, is exact
        tol = np.where(np.isnan(tol), 0, tol)
        d = np.where(fin, np.abs(got - ref) - np.where(fin, tol, 0), 0)
    assert d.max(initial=0) <= 0, (what, float(d.max()), np.unravel_index(d.argmax(), d.shape))


def bounds(z, lse, T, threads=64):
    V = z.shape[1]
    with np.errstate(invalid="ignore", over="ignore"):
        s = z / T
        m = s.max(1)
        e = s - m[:, None]
        p = np.exp(e) / np.exp(e).sum(1, keepdims=True)
        ae = np.where(p > 0, np.abs(e), 0)
        A, M2 = (p * ae).sum(1), (p * ae * ae).sum(1)
        depth = V / (2 * threads) + 16   # two partial sums per thread of a row
        r = (3 * A + 4 + depth) * U
    return m, e, A, M2, depth, r


def check(z, tokens, k=0, T=1.0, dev_logits=None, threads=64):
    """z: CPU tensor [rows, V] in the stored dtype; dev_logits: the same values as the kernel gets them."""
    from decoder_only_transformer_causal_b200 import native
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = z.cuda() if dev_logits is None else dev_logits
    res = native.token_logprobs(x, tokens.cuda(), k=k, temperature=T, status=status)
    again = native.token_logprobs(x, tokens.cuda(), k=k, temperature=T, status=status)
    for a, b in zip(res, again):
        assert (a is None) == (b is None)
        if a is not None:                          # bit-reproducible, NaN included
            assert torch.equal(a.view(torch.int32) if a.dtype == torch.float32 else a,
                               b.view(torch.int32) if b.dtype == torch.float32 else b)
    assert int(status.item()) == 0
    z64 = f64(z)
    logp, ent, lse, ids, tlp = logprob_ref(z64, tokens.numpy(), k, T)
    m, e, A, M2, depth, r = bounds(z64, lse, T, threads)
    V = z64.shape[1]
    with np.errstate(invalid="ignore"):
        lv = 2 * math.log(V) * U
        # a row with NaN or +inf has no defined lse
        ok = ~(np.isnan(z64).any(1) | np.isposinf(z64).any(1))
        close(f64(res.lse)[ok], lse[ok], (r + U * (3 * np.abs(m) + 2 * np.abs(lse)) + lv)[ok], "lse")
        et = np.abs(e[np.arange(len(m)), np.clip(tokens.numpy(), 0, V - 1)])
        close(f64(res.logp), logp, r + U * (4 * et + np.abs(logp)) + lv, "logp")
        close(f64(res.entropy), ent, r * (1 + A) + U * (3 * M2 + (8 + depth) * A + ent) + lv, "entropy")
        if k:
            assert np.array_equal(res.top_ids.cpu().numpy(), ids)
            ek = np.abs(np.take_along_axis(e, ids, 1))
            close(f64(res.top_logp), tlp, r[:, None] + U * (4 * ek + np.abs(tlp)) + lv, "top_logp")
        else:
            assert res.top_ids is None and res.top_logp is None


def make(rows, V, dtype, seed=0, std=3.0, banned=0):
    g = torch.Generator().manual_seed(seed + 7 * V + rows)
    z = (std * torch.randn((rows, V), generator=g)).to(DT[dtype])
    ids = torch.randperm(V, generator=g)
    z[:, ids[:banned]] = -math.inf
    tok = ids[torch.randint(banned, V, (rows,), generator=g)]
    tok[1::5] = -1
    return z, tok


SIZES = [
    # rows, V, k
    (1, 1, 1), (1, 1, 0), (3, 2, 2), (5, 7, 7), (4, 63, 63), (4, 64, 64), (7, 65, 5), (2, 255, 64), (9, 257, 0), (6, 1000, 3),
    (2, 4097, 64), (1, 8191, 20), (3, 32003, 33), (8, 50304, 5), (2, 50257, 20), (1, 131072, 1), (1, 262147, 64),
    (700, 515, 8), (1500, 97, 0), (300, 32003, 20),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,k", SIZES)
def test_sizes(rows, V, k, dtype):
    z, tok = make(rows, V, dtype)
    check(z, tok, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.3, 0.8, 1.7, 1e-3, 1e4])
def test_temperatures_and_banned_tokens(T, dtype):
    z, tok = make(5, 3001, dtype, banned=700)
    check(z, tok, 10, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [4, 900])
@pytest.mark.parametrize("off,pad", [(1, 0), (3, 1), (0, 5), (7, 9), (2, 47), (5, 3)])
def test_alignments(rows, off, pad, dtype):
    """Rows that start anywhere, and lie apart; what lies around them is NaN."""
    V = 1237
    z, tok = make(rows, V, dtype)
    buf = torch.full((off + rows * (V + pad) + 8,), math.nan, dtype=DT[dtype], device="cuda")
    x = buf[off:off + rows * (V + pad)].view(rows, V + pad)[:, :V]
    x.copy_(z)
    check(z, tok, 9, 1.0, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [11, 2050, 50257])
def test_special_rows(V, dtype):
    low = torch.finfo(DT[dtype]).min
    z = torch.zeros((16, V))
    g = torch.Generator().manual_seed(3)
    z[0] = -math.inf                                          # nothing left
    z[1] = low                                                # the type's lowest everywhere: uniform
    z[2] = -math.inf; z[2, V // 2] = 4.0                      # one token left
    z[3] = -math.inf; z[3, -1] = low                          # ... at the lowest value
    z[4] = torch.randn(V, generator=g); z[4, V // 3] = math.nan
    z[5] = torch.randn(V, generator=g); z[5, 1] = math.inf
    z[6] = -math.inf; z[6, 2] = math.nan
    z[7] = 2.5                                                # all equal
    z[8] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)   # equal zeros of both signs
    z[9] = torch.arange(V) / 4096.0                           # rising
    z[10] = -torch.arange(V) / 4096.0                         # falling
    z[11] = torch.randint(0, 3, (V,), generator=g).float()    # a third of the row ties for the first place
    z[12] = low; z[12, 3] = 0.0
    z[13] = torch.randn(V, generator=g) * 1e4
    z[14] = torch.randn(V, generator=g) * 1e-30
    z[15] = math.nan
    tok = torch.randint(0, V, (16,), generator=g)
    tok[2], tok[3], tok[12] = V // 2, V - 1, 3
    check(z.to(DT[dtype]), tok, min(V, 64))
    check(z.to(DT[dtype]), tok, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,k", [
    (1333, 1, 1), (1400, 31, 20), (1400, 127, 20), (1400, 300, 1), (1400, 1283, 20), (1400, 2557, 7), (1400, 4097, 0),
    (1400, 5113, 1), (1333, 65, 40), (1400, 511, 40), (1400, 513, 21), (1500, 1030, 40), (1400, 5117, 20), (1400, 2051, 64),
    (2800, 4100, 33), (1400, 10237, 3), (1332, 900, 20), (149, 16001, 2), (80, 16390, 9), (592, 28400, 5)])
def test_rows_of_a_warp_or_two(rows, V, k, dtype):
    """Sizes on both sides of where the number of threads per row changes; at least 32 of them."""
    z, tok = make(rows, V, dtype)
    check(z, tok, k, threads=32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,ks", [(11, (1, 11)), (1237, (1, 20, 40)), (2563, (1, 20))])
def test_special_values_in_many_rows(V, ks, dtype):
    """Rows that keep, tie or lose everything, at more rows than run at once, each with another start."""
    low = torch.finfo(DT[dtype]).min
    z, tok = make(1408, V, dtype, banned=3)
    z[0::11] = -math.inf
    z[1::11] = low
    z[2::11] = 2.5
    z[3::11, V // 3] = math.nan
    z[4::11, V // 2] = math.inf
    z[5::11] = torch.randint(0, 3, z[5::11].shape, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    z[6::11] = -math.inf; z[6::11, 2] = low
    z[7::11] = (torch.arange(V) / 4096.0).to(DT[dtype])
    tok[tok >= 0] %= V
    buf = torch.full((1408 * (V + 1) + 9,), math.nan, dtype=DT[dtype], device="cuda")
    x = buf[1:1 + 1408 * (V + 1)].view(1408, V + 1)[:, :V]
    x.copy_(z)
    for k in ks:
        check(z, tok, k, 1.0, x, threads=32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,k", [(6, 50257, 64), (6, 4099, 20), (160, 20011, 40), (700, 1501, 64), (1400, 1501, 20), (1400, 1501, 40), (2, 131, 64)])
def test_fewer_values_than_entries(rows, V, k, dtype):
    """Rows whose mask leaves fewer tokens than entries are asked for, rows of one or two values, and rows whose
    upper half lies within a 256th of one value; equal values are listed by index."""
    z, tok = make(rows, V, dtype)
    g = torch.Generator().manual_seed(V)
    order = torch.rand((rows, V), generator=g).argsort(1).argsort(1)
    left = torch.tensor([0, 1, k - 1, k, k // 2, V])[torch.arange(rows) % 6]
    z[order >= left[:, None]] = -math.inf
    z[3::6] = (torch.arange(V) >= V - 5).to(DT[dtype])            # few ones, behind
    z[4::6] = (torch.arange(V) % 97 == 96).to(DT[dtype]) * -2.0   # ones apart: ties in the order of the columns
    z[5::6, V // 2:] = (100.0 + torch.rand((z[5::6].shape[0], V - V // 2), generator=g) * 0.3).to(DT[dtype])
    low = torch.finfo(DT[dtype]).min
    z[0::12, ::2] = low                                           # nothing but the lowest value and -inf
    check(z, torch.where(tok >= 0, order.argmin(1), tok), k, threads=32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_crowded_top(dtype):
    """Many more values at or above the k-th largest of any partition than a short list holds."""
    V = 50257
    z = torch.full((3, V), -1.0)
    z[0, 7::8] = 5.0
    z[1, :20000] = torch.linspace(1, 2, 20000)
    z[2, V - 9000:] = 3.0
    check(z.to(DT[dtype]), torch.tensor([7, 5, -1]), 64)


def test_bad_tokens_and_optional_outputs():
    from decoder_only_transformer_causal_b200 import native
    z, tok = make(4, 100, "f32")
    tok[:] = torch.tensor([5, 100, -2, 7])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    res = native.token_logprobs(z.cuda(), tok.cuda(), status=status)
    assert int(status.item()) == native.GPT_ERR_INDEX
    assert res.logp[1].item() == 0 and res.logp[2].item() == 0 and res.logp[0].item() != 0
    none = native.token_logprobs(z.cuda(), None, k=2)
    assert none.logp is None and torch.equal(none.lse, res.lse) and torch.equal(none.entropy, res.entropy)
    only = native.token_logprobs(z.cuda(), tok.cuda(), out=native.TokenLogprobs(res.logp.clone(), None, None, None, None))
    assert torch.equal(only.logp, res.logp)
    assert native.token_logprobs(z.cuda()[:0], tok.cuda()[:0]).lse.shape == (0,)
    with pytest.raises(native.GPTError) as e:
        native.token_logprobs(z.cuda(), tok.cuda(), k=101)
    assert e.value.status == native.GPT_ERR_BAD_SHAPE
    with pytest.raises(ValueError):
        native.token_logprobs(z.cuda(), tok)                   # tokens on the CPU
    with pytest.raises(ValueError):
        native.token_logprobs(z.cuda(), tok.cuda().int())


def test_rows_behind_the_last_are_left_alone():
    from decoder_only_transformer_causal_b200 import native
    z, tok = make(5, 333, "bf16")
    bufs = [torch.full((7,), 42.0, device="cuda") for _ in range(3)]
    ids, tlp = torch.full((7, 4), -9, device="cuda"), torch.full((7, 4), 42.0, device="cuda")
    native.token_logprobs(z.cuda(), tok.cuda(), k=4, out=native.TokenLogprobs(*[b[:5] for b in bufs], ids[:5], tlp[:5]))
    assert all((b[5:] == 42).all() for b in bufs) and (ids[5:] == -9).all() and (tlp[5:] == 42).all()
    d = torch.full((7, 340), 42.0, dtype=torch.bfloat16, device="cuda")
    native.token_logprobs_backward(z.cuda(), tok.cuda(), bufs[2][:5], bufs[1][:5], dlogp=torch.ones(5, device="cuda"),
                                   dlogits=d[:5, :333])
    assert (d[5:] == 42).all() and (d[:, 333:] == 42).all() and (d[:5, :333] != 42).all()


def test_streams_and_graph_replay():
    from decoder_only_transformer_causal_b200 import native
    z, tok = make(40, 5003, "bf16")
    x, t = z.cuda(), tok.cuda()
    want = native.token_logprobs(x, t, k=3)
    g, h = torch.randn(40, device="cuda"), torch.randn(40, device="cuda")
    dwant = native.token_logprobs_backward(x, t, want.lse, want.entropy, g, h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = native.token_logprobs(x, t, k=3)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    xin = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        out = native.token_logprobs(xin, t, k=3)
        dout = native.token_logprobs_backward(xin, t, out.lse, out.entropy, g, h)
    for _ in range(2):
        xin.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)) and torch.equal(dout, dwant)
        xin.zero_()


def test_calls_at_once():
    """Calls in flight together on two streams share nothing."""
    from decoder_only_transformer_causal_b200 import native
    xs = [make(rows, V, dt) for rows, V, dt in ((700, 9001, "bf16"), (9, 50257, "f32"))]
    xs = [(z.cuda(), t.cuda()) for z, t in xs]
    want = [native.token_logprobs(z, t, k=7) for z, t in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(native.token_logprobs(*xs[i], k=7))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for r in got[i] for a, b in zip(r, want[i]))


# ------------------------------------------------------------------ gradient
def check_grad(z, tok, g, h, T, x=None, out=None):
    from decoder_only_transformer_causal_b200 import native
    z64 = f64(z)
    _, ent, lse, _, _ = logprob_ref(z64, tok.numpy(), 0, T)
    lse32, ent32 = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in (lse, ent))
    x = z.cuda() if x is None else x
    d = native.token_logprobs_backward(x, tok.cuda(), lse32, ent32, None if g is None else g.cuda(),
                                       None if h is None else h.cuda(), T, dlogits=out)
    rows = len(tok)
    g64 = np.zeros(rows) if g is None else f64(g)
    h64 = np.zeros(rows) if h is None else f64(h)
    ref = logprob_grad_ref(z64, tok.numpy(), g64, h64, T)
    with np.errstate(invalid="ignore", over="ignore"):
        lp = z64 / T - lse[:, None]
        p = np.exp(lp)
        alp = np.where(p > 0, np.abs(lp), 0)
        H = np.abs(ent)[:, None]
        ga, ha = np.abs(g64)[:, None], np.abs(h64)[:, None]
        # error of log p: the scaled logit, lse's storage, the difference, and 2 roundings of constants
        dl = U * (3 * np.where(p > 0, np.abs(z64 / T), 0) + 3 * np.abs(lse)[:, None] + 3 * alp + 4)
        tol = p * (ga + ha * (alp + H)) * (dl + 6 * U) + p * ha * (dl + U * (alp + 2 * H))
        tok64 = tok.numpy()
        r = np.nonzero(tok64 >= 0)[0]
        tol[r, tok64[r]] += 3 * U * np.abs(g64[r])
        tol = tol / T + 4 * U * np.abs(ref) + torch.finfo(z.dtype).eps / 2 * np.abs(ref) * (1 + 1e-3)
        tol += 2.0 ** -126 * (1 + 1 / T) * (1 + ga + ha)         # p below the normal range counts as 0
        # the storage rounding applies to the computed value, off by tol itself
        tol *= 1 + torch.finfo(z.dtype).eps
    close(f64(d), ref, np.where(np.isfinite(tol), tol, 0), "dlogits")
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (5, 7), (4, 65), (9, 257), (6, 1000), (2, 4097), (3, 32003), (2, 50304),
                                    (1, 131075), (700, 515), (1500, 33)])
def test_gradient_sizes(rows, V, dtype):
    z, tok = make(rows, V, dtype, seed=5, banned=V // 9)
    g = torch.Generator().manual_seed(V)
    check_grad(z, tok, torch.randn(rows, generator=g), torch.randn(rows, generator=g), 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(1300, 2057), (1200, 5121), (1190, 2563), (40, 9217), (5, 18440), (65600, 3)])
def test_gradient_thread_counts(rows, V, dtype):
    z, tok = make(rows, V, dtype, seed=5, banned=V // 9)
    g = torch.Generator().manual_seed(V)
    check_grad(z, tok, torch.randn(rows, generator=g), torch.randn(rows, generator=g), 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.3, 1.7, 1e3])
def test_gradient_terms(T, dtype):
    z, tok = make(6, 777, dtype, seed=6)
    g, h = torch.randn(6), torch.randn(6)
    check_grad(z, tok, g, None, T)
    check_grad(z, tok, None, h, T)
    g[2], h[3] = 0, 0
    check_grad(z, tok, g, h, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,pad,doff,dpad", [(0, 0, 1, 0), (1, 0, 0, 3), (3, 5, 3, 5), (2, 1, 2, 4), (7, 47, 1, 0), (4, 8, 0, 16)])
def test_gradient_alignments(off, pad, doff, dpad, dtype):
    rows, V = 6, 1237
    z, tok = make(rows, V, dtype, seed=7)

    def place(o, p, fill):
        buf = torch.full((o + rows * (V + p) + 8,), fill, dtype=DT[dtype], device="cuda")
        return buf, buf[o:o + rows * (V + p)].view(rows, V + p)[:, :V]
    _, x = place(off, pad, math.nan)
    x.copy_(z)
    buf, d = place(doff, dpad, 42.0)
    g, h = torch.randn(rows), torch.randn(rows)
    check_grad(z, tok, g, h, 0.9, x, d)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[doff:doff + rows * (V + dpad)].view(rows, V + dpad)[:, :V] = False
    assert (buf[mask] == 42).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_in_place(dtype):
    z, tok = make(5, 1003, dtype, seed=8)
    g, h = torch.randn(5), torch.randn(5)
    away = check_grad(z, tok, g, h, 1.0)
    x = z.cuda()
    assert torch.equal(check_grad(z, tok, g, h, 1.0, x, x), away)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_special_rows(dtype):
    V = 1001
    z, tok = make(7, V, dtype, seed=9)
    z[0] = -math.inf
    z[1, 5] = math.nan
    z[2] = math.nan                      # factors 0: written as zeros all the same
    z[3] = torch.finfo(DT[dtype]).min
    z[4] = -math.inf
    z[4, 9] = 1.0
    tok[:] = torch.tensor([3, 4, 5, 6, 9, -1, 8])
    g, h = torch.tensor([1.0, 1, 0, 1, 1, 1, 1]), torch.tensor([1.0, 1, 0, 1, 1, 0, 1])
    d = check_grad(z, tok, g, h, 1.0)
    assert (d[0] == 0).all() and (d[2] == 0).all() and (d[5] == 0).all() and torch.isnan(d[1]).all()


def test_gradient_bad_token():
    from decoder_only_transformer_causal_b200 import native
    z, tok = make(3, 50, "f32")
    tok[:] = torch.tensor([4, 50, 7])
    r = native.token_logprobs(z.cuda(), None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = native.token_logprobs_backward(z.cuda(), tok.cuda(), r.lse, None, torch.ones(3, device="cuda"), status=status)
    assert int(status.item()) == native.GPT_ERR_INDEX
    assert (d[1] == 0).all() and (d[0] != 0).any()


def test_forward_backward_against_differences():
    """The pair as a training step uses it: the gradient's directional derivative against differences
    of the 64-bit objective at the kernel's own outputs."""
    from decoder_only_transformer_causal_b200 import native
    z, tok = make(6, 301, "f32", seed=11)
    g, h, T, eps = torch.randn(6), torch.randn(6), 0.8, 1e-5
    r = native.token_logprobs(z.cuda(), tok.cuda(), temperature=T)
    d = f64(native.token_logprobs_backward(z.cuda(), tok.cuda(), r.lse, r.entropy, g.cuda(), h.cuda(), T))
    rng = np.random.default_rng(0)
    for _ in range(4):
        w = rng.standard_normal(z.shape)

        def f(s):
            lp, ent, *_ = logprob_ref(f64(z) + s * w, tok.numpy(), 0, T)
            return float((f64(g) * lp + f64(h) * ent).sum())
        num = (f(eps) - f(-eps)) / (2 * eps)
        # differences: eps^2 times a third derivative of order 100; rounding 1e-15 * 100 / eps.
        # gradient: entries off by about 1e-6 of themselves (tolerances above), 1800 of them
        assert abs(num - float((d * w).sum())) <= 1e-6 + 4e-6 * np.abs(d * w).sum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,T", [(1.0, 1.0), (4e8, 1.0), (1.0, 2e-9), (2.0 ** 20, 1e-3), (-3e9, 0.5), (1e30, 1.0), (1e20, 1e-12)])
@pytest.mark.parametrize("V,doff", [(1003, 0), (1003, 1), (50304, 0)])
def test_gradient_of_forbidden_tokens_is_zero_at_any_factor(V, doff, h, T, dtype):
    """Logits of -inf, and those so far below the maximum that their probability is 0, get 0 however large the
    entropy's factor over the temperature is."""
    g = torch.Generator().manual_seed(V)
    z = torch.randint(0, 2, (4, V), generator=g).to(DT[dtype]) * (-1.0 if T < 1e-2 else 0.25)
    z[:, ::3] = -math.inf
    z[1, 1::3] = -200.0
    z[2, 1:] = -math.inf; z[2, 0] = 0.0                          # one token left: its gradient is 0 as well
    z[3, 1:] = torch.finfo(DT[dtype]).min; z[3, 0] = 0.0
    tok = torch.tensor([1, 2, 0, -1])
    buf = torch.full((doff + 4 * V,), 42.0, dtype=DT[dtype], device="cuda")
    d = check_grad(z, tok, torch.ones(4), torch.full((4,), h), T, out=buf[doff:].view(4, V))
    assert (d[:2, ::3] == 0).all() and (d[1, 1::3] == 0).all() and (d[2:] == 0).all()
