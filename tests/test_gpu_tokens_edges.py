"""The many-token operators on the int8 matrix where they can go wrong: followed by the single-token calls in one
stream, signs of zero, tokens that are not finite, row scales of very different sizes, optional outputs, and the size of
their rounding errors."""
import numpy as np
import pytest
import torch

import test_gpu_tokens as base
from bit_quantized_mamba_b200 import inputs

pytestmark = pytest.mark.gpu

F8 = torch.float64


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_mamba_b200 import build, dfssm
    build.build()
    dfssm.lib()
    return torch.device("cuda:0")


def gen(seed, dev):
    return torch.Generator(dev).manual_seed(seed)


def matrix(g, V, d, dev):
    """Codes and row scales, complete before any call is enqueued."""
    W = torch.randint(-127, 128, (V, d), generator=g, device=dev, dtype=torch.int8)
    s = torch.rand(V, generator=g, device=dev) * 9e-4 + 1e-4
    torch.cuda.synchronize()
    return W, s


# ------------------------------------------------------------------------------------ one stream


@pytest.mark.parametrize("B", [1, 4, 16])
def test_single_token_calls_read_what_the_embedding_just_wrote(dev, B):
    """embed_tokens lets the next kernel of the stream start before its rows are written.  The head, the greedy head
    and the streaming linear on those rows, in a captured chain over one buffer, give the bits of calls made one
    at a time."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(40 + B, dev)
    V, d, n = 1187, 2048, 6
    W, sr = matrix(g, V, d, dev)
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    L = dfssm.Linear.from_host(inputs.linear(np.random.default_rng(B), 4096, d), dev)
    tok = torch.randint(0, V, (n, B), generator=g, device=dev, dtype=torch.int32)
    h = torch.zeros(B, d, device=dev)
    size = dfssm.workspace_size
    ws = [dfssm.workspace(size(op, *dims), dev) for op, dims in (
        (dfssm.OP_EMBED_TOKENS, (0, 0, 0)), (dfssm.OP_HEAD_GREEDY, (1, d, V)), (dfssm.OP_LM_HEAD, (1, d, V)),
        (dfssm.OP_LINEAR_DECODE, (B, d, 4096)))]
    torch.cuda.synchronize()

    def chain(pause):
        outs = []
        for k in range(n):
            for call in (lambda: list(dfssm.head_greedy(W, sr, h[0], nw, ws=ws[1])),
                         lambda: [dfssm.lm_head(W, sr, h[0], ws=ws[2])],
                         lambda: [dfssm.linear_decode(L, h, ws=ws[3])]):
                dfssm.embed_tokens(W, sr, tok[k], h=h, ws=ws[0])
                pause()
                outs += call()
                pause()
                dfssm.embed_tokens(W, sr, tok[(k + 1) % n], h=h, ws=ws[0])  # other rows, which none of them may see
                pause()
        return outs

    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------------------------ signs of zero


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("M", [1, 3, 16, 100, 300])
def test_linear_int8_signs_of_zero(dev, M):
    """A zero accumulator times a negative row scale is -0 in the definition, in the single-token head and here,
    whatever the neighbouring outputs are."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(60 + M, dev)
    V, d = 700, 512
    W, sr = matrix(g, V, d, dev)
    W[::5] = 0
    sr = sr * (torch.randint(0, 2, (V,), generator=g, device=dev) * 2 - 1)
    sr[7::50] *= 2.0 ** -45  # beyond what the fp32 pairs take
    x = torch.randn(M, d, generator=g, device=dev)
    x[::3] = 0.0
    torch.cuda.synchronize()
    acc = torch.zeros(M, V, dtype=torch.int32, device=dev)
    scale = torch.zeros(M, device=dev)
    y = dfssm.linear_int8(W, sr, x, debug=dict(acc=acc, xscale=scale))
    want = (acc.double() * scale.double()[:, None] * sr.double()).float()
    assert bool((bits(want) == -2 ** 31).any())
    assert torch.equal(bits(y), bits(want))
    yb = dfssm.linear_int8(W, sr, x, out_dtype=torch.bfloat16)
    assert torch.equal(bits(yb), bits(want.bfloat16()))
    for t in range(0, M, 37):
        assert torch.equal(bits(dfssm.lm_head(W, sr, x[t].contiguous())), bits(y[t]))


# ------------------------------------------------------------------------------------ odd tokens


@pytest.mark.parametrize("M", [1, 3, 40, 100, 300])
def test_head_loss_of_one_row_and_tokens_that_are_not_finite(dev, M):
    """A vocabulary of one row has loss and gradients zero, but a token that is not finite has NaN in its own."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(80 + M, dev)
    W, sr = matrix(g, 1, 64, dev)
    x = torch.randn(M, 64, generator=g, device=dev)
    x[0, 5] = float("nan")
    if M > 2:
        x[2, 6] = float("inf")
    labels = torch.zeros(M, dtype=torch.int32, device=dev)
    if M > 2:
        labels[1] = -1
        x[1, 0] = float("nan")  # ignored
    bad = torch.zeros(M, dtype=torch.bool, device=dev)
    bad[0::2][:2] = True
    loss, stats = dfssm.head_loss(W, sr, x, labels)
    assert torch.equal(loss.isnan(), bad) and not loss[~bad].any()
    dx, ds, _ = dfssm.head_loss_backward(W, sr, x, labels, stats, torch.ones(M, device=dev))
    assert bool(dx[bad].isnan().all()) and not dx[~bad].any() and bool(ds.isnan().all())
