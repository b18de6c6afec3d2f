"""Drafted trees and token log probabilities without a GPU: the host-side refusals of their entry
points, and the 64-bit definitions that the GPU tests compare with, held against differences and
closed forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

import seeded
from decoder_only_transformer_causal_b200 import native
from decoder_only_transformer_causal_b200.native import GPTConfig
from operator_refs import accept_ref, logprob_grad_ref, logprob_ref, see_sets, tree_attention_ref

L = native.LIB
FAKE = 1 << 20          # aligned, never dereferenced: the calls below are refused first
BF16, F32 = native.GPT_DTYPE_BF16, native.GPT_DTYPE_F32
NULL, SHAPE, ALIGN, UNSUP, SMALL = (native.GPT_ERR_NULL, native.GPT_ERR_BAD_SHAPE, native.GPT_ERR_BAD_ALIGN,
                                    native.GPT_ERR_UNSUPPORTED, native.GPT_ERR_WS_TOO_SMALL)


def tree(qkv=FAKE, kv=FAKE, lengths=FAKE, parents=FAKE, y=FAKE, B=2, N=8, nh=12, hs=64, cap=1024, dtype=BF16):
    return L.gpt_tree_attention(qkv, kv, lengths, parents, y, B, N, nh, hs, cap, dtype, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(qkv=None), NULL), (dict(kv=None), NULL), (dict(lengths=None), NULL), (dict(parents=None), NULL),
    (dict(y=None), NULL), (dict(B=0), SHAPE), (dict(N=0), SHAPE), (dict(nh=0), SHAPE), (dict(hs=0), SHAPE),
    (dict(cap=0), SHAPE), (dict(dtype=7), SHAPE), (dict(N=65), UNSUP), (dict(hs=32), UNSUP), (dict(hs=128), UNSUP),
    (dict(hs=36, dtype=F32), UNSUP), (dict(hs=136, dtype=F32), UNSUP), (dict(B=65536), UNSUP),
    (dict(B=65535, nh=1 << 20), UNSUP), (dict(nh=1 << 24), UNSUP), (dict(cap=0x7fffffff), UNSUP), (dict(qkv=FAKE + 8), ALIGN), (dict(kv=FAKE + 2), ALIGN),
    (dict(y=FAKE + 4), ALIGN), (dict(lengths=FAKE + 2), ALIGN), (dict(parents=FAKE + 1), ALIGN),
])
def test_tree_attention_refusals(kw, code):
    assert tree(**kw) == code


def _cfg(name="gpt2", **kw):
    return GPTConfig.from_dict(dict(seeded.WORKLOADS[name].model_dict(), **kw))


def step(cfg, w=FAKE, tok=FAKE, par=FAKE, lens=FAKE, B=2, N=8, kv=FAKE, tq=FAKE, lg=FAKE, ws=FAKE, nws=1 << 40):
    return L.gpt_tree_step(ctypes.byref(cfg.c()), w, tok, par, lens, B, N, kv, tq, lg, ws, nws, None, 0)


def test_tree_step_refusals():
    c = _cfg()
    for name in ("w", "tok", "par", "lens", "kv", "tq", "lg", "ws"):
        assert step(c, **{name: None}) == NULL, name
    assert step(c, N=65) == UNSUP
    assert step(c, N=0) == SHAPE and step(c, B=0) == SHAPE
    assert step(_cfg(block_size=4), N=8) == SHAPE                 # more nodes than positions
    assert step(c, nws=1024) == SMALL
    assert step(c, kv=FAKE + 8) == ALIGN and step(c, tq=FAKE + 8) == ALIGN and step(c, lg=FAKE + 8) == ALIGN
    assert step(c, w=FAKE + 16) == ALIGN
    assert step(_cfg(vocab_size=50257)) == UNSUP                   # bf16 rows of 16-byte units
    assert step(_cfg(n_head=24)) == UNSUP


def accept(cfg, N=8, B=2, **kw):
    names = ("par", "tok", "cho", "lens", "tq", "kv", "path", "n", "nxt", "lo")
    a = {n: FAKE for n in names}
    a.update(kw)
    return L.gpt_tree_accept(ctypes.byref(cfg.c()), a["par"], a["tok"], a["cho"], a["lens"], B, N, a["tq"], a["kv"],
                             a["path"], a["n"], a["nxt"], a["lo"], None, None)


def test_tree_accept_refusals():
    c = _cfg()
    for name in ("par", "tok", "cho", "lens", "tq", "kv", "path", "n", "nxt", "lo"):
        assert accept(c, **{name: None}) == NULL, name
    assert accept(c, N=65) == UNSUP and accept(c, N=0) == SHAPE and accept(c, B=0) == SHAPE
    assert accept(c, tq=FAKE + 8) == ALIGN and accept(c, kv=FAKE + 8) == ALIGN
    assert accept(_cfg(n_head=24)) == UNSUP
    assert L.gpt_tree_accept(None, *([FAKE] * 4), 1, 1, *([FAKE] * 6), None, None) == NULL


def test_index_arrays_must_be_aligned():
    c = _cfg()
    for name in ("tok", "par", "lens"):
        assert step(c, **{name: FAKE + 2}) == ALIGN, name
    for name in ("par", "tok", "cho", "lens", "path", "n", "nxt", "lo"):
        assert accept(c, **{name: FAKE + 2}) == ALIGN, name
    assert accept(c, tok=FAKE + 4) == ALIGN and accept(c, nxt=FAKE + 4) == ALIGN
    assert score(tok=FAKE + 4) == ALIGN and score(logp=FAKE + 2) == ALIGN
    assert score(k=1, ids=FAKE + 4, lp=FAKE) == ALIGN and score(k=1, ids=FAKE, lp=FAKE + 1) == ALIGN
    for name in ("lse", "ent", "g", "h"):
        assert grad(**{name: FAKE + 2}) == ALIGN, name


def test_tree_qkv_bytes():
    c = _cfg()
    assert L.gpt_tree_qkv_bytes(ctypes.byref(c.c()), 3, 5) == 12 * 3 * 5 * 3 * 768 * 2
    assert L.gpt_tree_qkv_bytes(ctypes.byref(c.c()), 3, 65) == 0
    assert L.gpt_tree_qkv_bytes(ctypes.byref(c.c()), 0, 5) == 0
    assert L.gpt_tree_qkv_bytes(ctypes.byref(_cfg(n_head=24).c()), 1, 1) == 0


def score(z=FAKE, ld=100, tok=FAKE, rows=4, V=100, dtype=BF16, T=1.0, logp=FAKE, k=0, ids=None, lp=None):
    return L.gpt_token_logprobs(z, ld, tok, rows, V, dtype, T, logp, FAKE, FAKE, k, ids, lp, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(z=None), NULL), (dict(tok=None), NULL), (dict(k=3), NULL), (dict(k=3, ids=FAKE), NULL), (dict(rows=-1), SHAPE),
    (dict(V=0), SHAPE), (dict(ld=99), SHAPE), (dict(dtype=3), SHAPE), (dict(T=0.0), SHAPE), (dict(T=-1.0), SHAPE),
    (dict(T=math.inf), SHAPE), (dict(T=math.nan), SHAPE), (dict(T=1e-39), SHAPE), (dict(k=-1), SHAPE),
    (dict(k=101, ids=FAKE, lp=FAKE), SHAPE), (dict(k=65, ids=FAKE, lp=FAKE), UNSUP), (dict(z=FAKE + 1), ALIGN),
    (dict(z=FAKE + 2, dtype=F32), ALIGN), (dict(rows=0), native.GPT_OK),
])
def test_token_logprobs_refusals(kw, code):
    assert score(**kw) == code


def grad(z=FAKE, ld=100, tok=FAKE, rows=4, V=100, dtype=BF16, T=1.0, lse=FAKE, ent=FAKE, g=FAKE, h=FAKE, d=2 * FAKE, ldd=100):
    return L.gpt_token_logprobs_backward(z, ld, tok, rows, V, dtype, T, lse, ent, g, h, d, ldd, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(z=None), NULL), (dict(lse=None), NULL), (dict(d=None), NULL), (dict(tok=None), NULL), (dict(ent=None), NULL),
    (dict(ldd=99), SHAPE), (dict(ld=99), SHAPE), (dict(d=FAKE, ldd=104), SHAPE), (dict(T=0.0), SHAPE), (dict(V=0), SHAPE),
    (dict(d=2 * FAKE + 1), ALIGN), (dict(d=2 * FAKE + 2, dtype=F32), ALIGN), (dict(rows=0), native.GPT_OK),
])
def test_token_logprobs_backward_refusals(kw, code):
    assert grad(**kw) == code


def test_python_argument_checks():
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    kv = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)
    par, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        native.tree_attention(q, kv, lens, par, 1)               # not on a GPU
    with pytest.raises(ValueError):
        native.tree_attention(q[0], kv, lens, par, 1)
    with pytest.raises(ValueError):
        native.tree_attention(q, kv, lens, par, 5)               # C % n_head
    z = torch.zeros((3, 10))
    with pytest.raises(ValueError):
        native.token_logprobs(z)                                 # not on a GPU
    with pytest.raises(ValueError):
        native.token_logprobs(z.t())                             # columns contiguous, not rows
    with pytest.raises(ValueError):
        native.token_logprobs(z[:1].expand(3, 10))               # rows overlap
    with pytest.raises(ValueError):
        native.token_logprobs(z.double())


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 1), (2 ** 31, 2), (1, 2 ** 32 + 100), (3, 2 ** 31)])
def test_sizes_past_the_calls_integers_are_refused(shape):
    z = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="at most"):
        native.token_logprobs(z)
    with pytest.raises(ValueError, match="at most"):
        native.token_logprobs_backward(z, None, torch.empty(shape[0], device="meta"))


def test_score_checks_its_tensors_before_the_forward():
    """The forward reads B T 64-bit integers from idx and from targets: others are refused before it is launched."""
    from decoder_only_transformer_causal_b200 import GPT
    m = GPT.__new__(GPT)
    m.cfg, m.weights = _cfg(), torch.empty(1)

    def launched(*a):
        raise AssertionError("the forward was reached")
    m.workspace = launched
    idx = torch.zeros((2, 9), dtype=torch.int64)
    with pytest.raises(AssertionError, match="reached"):
        m.score(idx, idx)
    for a, b in ((idx, idx[:, :8].contiguous()), (idx, idx.int()), (idx.int(), idx), (idx, idx.view(-1)), (idx, idx[:1]),
                 (idx, torch.zeros((9, 2), dtype=torch.int64).t()), (idx, idx.to("meta"))):
        with pytest.raises(ValueError):
            m.score(a, b)


# ------------------------------------------------------------------ the definitions themselves
def test_see_sets():
    par = np.array([[-1, 0, 0, 1, 3, -2, 5, 9, -1, 8]])
    see = see_sets(par)[0]
    assert [sorted(s) for s in see] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [], [], [], [8], [8, 9]]


def test_tree_attention_ref_is_causal_attention_on_a_chain():
    """A chain over a cache is the tail of causal attention over the whole sequence."""
    rng = np.random.default_rng(0)
    T, len0, nh, hs = 11, 6, 2, 8
    x = rng.standard_normal((1, T, 3, nh * hs))
    kv = np.zeros((1, 16, 2, nh * hs))
    kv[0, :len0] = x[0, :len0, 1:]
    kv[0, len0:] = np.nan
    n = T - len0
    got, _ = tree_attention_ref(x[:, len0:], kv, np.array([len0]), np.arange(-1, n - 1)[None], nh)
    q, k, v = (torch.tensor(x[0, :, j]).view(T, nh, hs).transpose(0, 1) for j in range(3))
    want = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True).transpose(0, 1).reshape(T, -1)
    assert np.abs(got[0] - want.numpy()[len0:]).max() < 1e-12


def test_logprob_ref_closed_forms():
    z = np.array([[0.0, 0.0, 0.0, 0.0], [5.0, -np.inf, 5.0, -np.inf], [-np.inf] * 4])
    lp, ent, lse, ids, tlp = logprob_ref(z, np.array([2, 0, 1]), 3, 1.0)
    assert np.allclose(lp[:2], [-math.log(4), -math.log(2)]) and np.isnan(lp[2])
    assert np.allclose(ent[:2], [math.log(4), math.log(2)]) and np.isnan(ent[2])
    assert ids.tolist() == [[0, 1, 2], [0, 2, 1], [0, 1, 2]]
    assert lse[2] == -np.inf and tlp[1, 2] == -np.inf


def test_logprob_grad_ref_against_differences():
    rng = np.random.default_rng(1)
    z = rng.standard_normal((5, 7)) * 2
    t = np.array([0, 3, -1, 6, 2])
    g, h, T, eps = rng.standard_normal(5), rng.standard_normal(5), 0.7, 1e-6
    d = logprob_grad_ref(z, t, g, h, T)

    def f(zz):
        lp, ent, *_ = logprob_ref(zz, t, 0, T)
        return float((g * lp + h * ent).sum())
    num = np.zeros_like(z)
    for i in np.ndindex(*z.shape):
        a, b = z.copy(), z.copy()
        a[i] += eps
        b[i] -= eps
        num[i] = (f(a) - f(b)) / (2 * eps)
    assert np.abs(num - d).max() < 1e-8


def test_accept_ref():
    par = np.array([[-1, 0, 0, 1, 2, 4]])
    tok = np.array([[9, 5, 5, 1, 2, 3]])
    cho = np.array([[5, 1, 2, 8, 3, 7]])
    path, n, nxt = accept_ref(par, tok, cho, np.array([10]), 100)
    assert path[0] == [0, 2, 4, 5] and n == [4] and nxt == [7]     # the longer of two equal first tokens
    path, n, nxt = accept_ref(par, tok, cho, np.array([97]), 100)
    assert path[0] == [0, 2, 4] and nxt == [3]                     # cut at the end of the cache
    path, n, nxt = accept_ref(par, tok, cho, np.array([100]), 100)
    assert path[0] == [] and nxt == [-1]
