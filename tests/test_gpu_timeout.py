"""The time-out path of the tensor-core kernels and of the single-launch decode step, made to run on
purpose without faulting the GPU.

Every pipeline wait in the tensor-core kernels is bounded: when a wait gives up, the kernel records
GPT_ERR_TIMEOUT in its status word, lets the copies and products it already issued finish, frees
its tensor memory and returns.  gpt_set_wait_limit_ns lowers the limit to 1 ms and makes the
kernel's issuing thread first wait for an event that never happens (a barrier nothing arrives
on), so that wait gives up and the whole kernel takes its time-out path; the test then checks the
status, restores the defaults and checks that the next call on the same context computes the
right result."""
import pytest
import torch

from gpu_helpers import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture
def short_waits():
    from decoder_only_transformer_causal_b200 import native
    torch.cuda.synchronize()
    native.set_wait_limit_ns(1_000_000, force_timeout=True)
    try:
        yield native
    finally:
        torch.cuda.synchronize()
        native.set_wait_limit_ns(0)


def _attention_inputs():
    g = torch.Generator(device="cuda").manual_seed(71)
    return [torch.randn((2, 4, 512, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]


def test_attention_wait_limit_gives_timeout_then_recovers(short_waits):
    native = short_waits
    q, k, v = _attention_inputs()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.attention(q, k, v, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_ERR_TIMEOUT
    native.set_wait_limit_ns(0)
    st.zero_()
    y = native.attention(q, k, v, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_OK
    ref = torch.nn.functional.scaled_dot_product_attention(q.float(), k.float(), v.float(), is_causal=True)
    assert float((y.float() - ref).abs().max()) <= 2e-2


@pytest.mark.parametrize("M", [128, 512])
def test_gemm_wait_limit_gives_timeout_then_recovers(short_waits, M):
    """M = 128: one CTA per 128-row tile; M = 512: CTA pairs (2-SM products), whose leader waits
    for the peer's copies, counted on the leader's barriers, before the pair exits."""
    native = short_waits
    g = torch.Generator(device="cuda").manual_seed(72)
    x = torch.randn((M, 768), generator=g, device="cuda").to(torch.bfloat16)
    W = (0.02 * torch.randn((2304, 768), generator=g, device="cuda")).to(torch.bfloat16)
    b = (0.02 * torch.randn(2304, generator=g, device="cuda")).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros((M, 2304), dtype=torch.bfloat16, device="cuda")
    native.linear(x, W, b, out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_ERR_TIMEOUT
    native.set_wait_limit_ns(0)
    st.zero_()
    native.linear(x, W, b, out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_OK
    ref = x.float() @ W.float().T + b.float()
    assert float((out.float() - ref).abs().max()) <= 2e-2


def test_decode_step_wait_limit_gives_timeout_then_recovers():
    """The single-launch decode step waits at its first grid barrier for an arrival that never
    comes: every CTA gives up after 1 ms, lets its weight copies land and returns, the position stays
    where it was, and the next step (limits restored) gives the logits of an undisturbed step."""
    import seeded
    from decoder_only_transformer_causal_b200 import GPT, GPTConfig, native
    from gpu_helpers import model_inputs
    cfg_d, W, _, _, _ = model_inputs("gpt2", stress=True, n_layer=2)
    m = GPT(GPTConfig.from_dict(cfg_d), W)
    B, T0 = 1, 40
    prompt, _ = seeded.make_tokens(B, T0, 50257, seed=9021)
    tok = torch.tensor([123], dtype=torch.int64, device="cuda")
    runs = []
    for forced in (False, True):
        kv = native.alloc_kv_cache(m.cfg, B)
        ws = native.alloc_workspace(native.decode_workspace_bytes(m.cfg, B, T0))
        native.prefill(m.cfg, m.weights, prompt.cuda(), kv, ws, sync_check=True)
        if forced:
            torch.cuda.synchronize()
            native.set_wait_limit_ns(1_000_000, force_timeout=True)
            try:
                native.decode_step(m.cfg, m.weights, tok, kv, ws)
                assert native.check_status(ws) == native.GPT_ERR_TIMEOUT
            finally:
                torch.cuda.synchronize()
                native.set_wait_limit_ns(0)
        logits = native.decode_step(m.cfg, m.weights, tok, kv, ws, sync_check=True).clone()
        assert native.check_status(ws) == native.GPT_OK
        runs.append(logits)
    assert torch.equal(runs[0], runs[1])


def test_tree_attention_of_many_rounds_ends_after_a_timeout(short_waits):
    """More sequences and heads than run at a time: a CTA's warps leave their rounds together."""
    native = short_waits
    qkv = torch.ones((64, 5, 3, 1024), dtype=torch.bfloat16, device="cuda")
    kv = torch.ones((64, 300, 2, 1024), dtype=torch.bfloat16, device="cuda")
    lens = torch.arange(64, dtype=torch.int32, device="cuda") * 4
    par = torch.arange(-1, 4, dtype=torch.int32, device="cuda").repeat(64, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.tree_attention(qkv, kv, lens, par, 16, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_ERR_TIMEOUT
    native.set_wait_limit_ns(0)
    st.zero_()
    y = native.tree_attention(qkv, kv, lens, par, 16, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_OK and (y == 1).all()


@pytest.mark.parametrize("N", [20, 64])
def test_tree_attention_wait_limit_gives_timeout_then_recovers(short_waits, N):
    """Clusters of CTAs: every CTA gives up, and none leaves before the others have read its part."""
    native = short_waits
    g = torch.Generator(device="cuda").manual_seed(73)
    qkv = torch.randn((2, N, 3, 128), generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn((2, 700, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([700, 300], dtype=torch.int32, device="cuda")
    par = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(2, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.tree_attention(qkv, kv, lens, par, 2, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_ERR_TIMEOUT
    native.set_wait_limit_ns(0)
    st.zero_()
    y = native.tree_attention(qkv, kv, lens, par, 2, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_OK
    for b in range(2):                                   # a chain: the tail of causal attention
        n = int(lens[b])
        x = torch.cat([kv[b, :n], qkv[b, :, 1:]]).float().view(n + N, 2, 2, 64)
        q = qkv[b, :, 0].float().view(N, 2, 64).transpose(0, 1)
        mask = torch.ones((N, n + N), dtype=torch.bool, device="cuda").tril(n)
        ref = torch.nn.functional.scaled_dot_product_attention(q, x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1), attn_mask=mask)
        assert float((y[b].float() - ref.transpose(0, 1).reshape(N, 128)).abs().max()) <= 2e-2


# B, N, heads, head size, cache, lengths: one to three loads per CTA or many, with and without a cluster, both ways
# of loading (a warp of its own up to 32 nodes, a thread of the products beyond), whole and cut tiles
F32_TREES = [(2, 20, 2, 64, 1000, [1000, 130]), (2, 64, 2, 64, 1000, [1000, 130]), (60, 5, 16, 64, 700, [700 - 11 * i for i in range(60)]),
             (60, 40, 8, 32, 700, [700 - 11 * i for i in range(60)]), (40, 17, 12, 128, 300, [7 * i for i in range(40)]), (1, 3, 1, 8, 64, [0])]


@pytest.mark.parametrize("B,N,nh,hs,cap,lens", F32_TREES)
def test_fp32_tree_attention_wait_limit_gives_timeout_then_recovers(short_waits, B, N, nh, hs, cap, lens):
    """The warps of the products give up with the first copies under way: all leave together, the copies that were
    issued land, and the next call is undisturbed."""
    native = short_waits
    g = torch.Generator(device="cuda").manual_seed(74)
    qkv = torch.randn((B, N, 3, nh * hs), generator=g, device="cuda")
    kv = torch.randn((B, cap, 2, nh * hs), generator=g, device="cuda")
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    par = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.tree_attention(qkv, kv, lens, par, nh, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_ERR_TIMEOUT
    native.set_wait_limit_ns(0)
    st.zero_()
    y = native.tree_attention(qkv, kv, lens, par, nh, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_OK
    for b in (0, B // 2, B - 1):                         # a chain: the tail of causal attention
        n = int(lens[b])
        x = torch.cat([kv[b, :n], qkv[b, :, 1:]]).double().view(n + N, 2, nh, hs)
        q = qkv[b, :, 0].double().view(N, nh, hs).transpose(0, 1)
        mask = torch.ones((N, n + N), dtype=torch.bool, device="cuda").tril(n)
        s = (q @ x[:, 0].permute(1, 2, 0) * hs ** -0.5).masked_fill(~mask, -float("inf"))
        ref = (torch.softmax(s, -1) @ x[:, 1].transpose(0, 1)).transpose(0, 1).reshape(N, nh * hs)
        # 2 a ((hs + 28) u D + (n + N + 28) u) of test_gpu_tree's tolerance with hs 128, D 10, n 1100, a 1
        assert float((y[b] - ref).abs().max()) <= 4e-4


@pytest.mark.parametrize("N", [16, 17, 32, 33, 64])
def test_tree_attention_of_paired_warps_ends_after_a_timeout(short_waits, N):
    """Warps that exchange their weights' parts at a barrier of two leave the steps, and the rounds, together."""
    native = short_waits
    B, nh = 40, 16
    g = torch.Generator(device="cuda").manual_seed(75)
    qkv = torch.randn((B, N, 3, nh * 64), generator=g, device="cuda").to(torch.bfloat16)
    qkv[:, :, 2] = 0.75
    kv = torch.randn((B, 400, 2, nh * 64), generator=g, device="cuda").to(torch.bfloat16)
    kv[:, :, 1] = 0.75
    lens = (torch.arange(B, dtype=torch.int32, device="cuda") * 10)
    par = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.tree_attention(qkv, kv, lens, par, nh, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == native.GPT_ERR_TIMEOUT
    native.set_wait_limit_ns(0)
    st.zero_()
    y = native.tree_attention(qkv, kv, lens, par, nh, status=st)
    torch.cuda.synchronize()
    # values all alike: their mean is the value, whatever the weights (sums off by 2^-15, which rounding to bf16 hides)
    assert int(st.item()) == native.GPT_OK and (y == 0.75).all()
