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


@pytest.mark.parametrize("M", [3, 40, 100, 200, 300])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_loss_of_odd_tokens_in_every_kernel(dev, M, norm, dtype):
    """Ignored labels, labels past the vocabulary, rows of zeros and rows that are not finite, at the sizes of every
    variant of the products and with the norm's backward."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(100 + M, dev)
    V, d = 700, 144
    W, sr = matrix(g, V, d, dev)
    nw = torch.rand(d, generator=g, device=dev) + 0.5 if norm else None
    x = torch.randn(M, d, generator=g, device=dev).to(dtype)
    ones = torch.ones(M, device=dev)
    # all ignored, some of them not finite
    none = torch.full((M,), -2 ** 31, dtype=torch.int32, device=dev)
    none[1::2] = -1
    xi = x.clone()
    xi[0] = float("nan")
    loss, stats = dfssm.head_loss(W, sr, xi, none, norm_w=nw)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, xi, none, stats, ones, norm_w=nw)
    assert not loss.any() and not dx.any() and not ds.any() and (dn is None or not dn.any())
    # finite losses and gradients beside a bad label, an ignored row that is not finite, and zeros
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    labels[0], labels[1] = V, -1
    x[1, 7] = float("nan")
    x[2] = 0.0
    ws = dfssm.workspace(dfssm.workspace_size(dfssm.OP_HEAD_LOSS, M, d, V), dev)
    loss, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw, ws=ws)
    assert dfssm.device_status(ws) == -1 and dfssm.device_status(ws) == 0
    assert float(loss[0]) == 0 and float(loss[1]) == 0 and bool(loss.isfinite().all())
    # flat logits: the sum of V - 1 ones is exact, its logarithm and the loss are rounded
    assert abs(float(loss[2]) - np.log(V)) <= 2.0 ** -22 * np.log(V)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, ones, norm_w=nw)
    assert not dx[:2].any()
    for t in (dx, ds, dn):
        assert t is None or bool(t.isfinite().all())
    # a row that is not finite and has a label: NaN in its own loss and dx, and in the sums over tokens
    for value in (float("inf"), float("nan")):
        x[2, 100] = value
        loss, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw)
        assert bool(loss[2].isnan()) and int(loss.isnan().sum()) == 1
        dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, ones, norm_w=nw)
        assert bool(dx[2].isnan().all()) and int(dx.isnan().sum()) == d
        assert bool(ds.isnan().all()) and (dn is None or bool(dn.isnan().all()))


@pytest.mark.parametrize("M", [1, 4, 20, 130, 300])
@pytest.mark.parametrize("norm", [False, True])
def test_linear_int8_of_odd_tokens_in_every_kernel(dev, M, norm):
    """Rows of zeros, tiny rows and rows that are not finite among ordinary ones, at the sizes of every variant."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(120 + M, dev)
    V, d = 500, 272
    W, sr = matrix(g, V, d, dev)
    nw = torch.rand(d, generator=g, device=dev) + 0.5 if norm else None
    for first in range(3):  # every kind of row is the first token once
        x = torch.randn(M, d, generator=g, device=dev)
        kinds = [(first + k) % 4 for k in range(M)]
        x[[k == 0 for k in kinds]] = 0.0
        x[[k == 1 for k in kinds]] *= 1e-38
        bad = torch.tensor([k == 2 for k in kinds], device=dev)
        x[bad, 17] = float("nan") if first else float("-inf")
        acc = torch.zeros(M, V, dtype=torch.int32, device=dev)
        scale = torch.zeros(M, device=dev)
        y = dfssm.linear_int8(W, sr, x, norm_w=nw, debug=dict(acc=acc, xscale=scale))
        want = (acc.double() * scale.double()[:, None] * sr.double()).float()
        assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], want[~bad]) and bool(y[~bad].isfinite().all())
        _, q, s, _ = base.quantized(x, nw)
        assert torch.equal(scale[~bad], s[~bad, 0])
        assert torch.equal(acc[~bad].double(), (q @ W.double().t())[~bad])


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("norm", [False, True])
def test_head_gradient_of_weights_of_zero(dev, M, norm):
    """A token whose dloss is 0 has no gradient, but 0 times NaN is NaN: one that is not finite has to be left out by its
    label."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(130 + M, dev)
    V, d = 900, 272
    W, sr = matrix(g, V, d, dev)
    nw = torch.rand(d, generator=g, device=dev) + 0.5 if norm else None
    x = torch.randn(M, d, generator=g, device=dev)
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    dloss = torch.rand(M, generator=g, device=dev)
    dloss[1] = 0
    _, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=nw)
    assert not dx[1].any() and bool(dx[0].any())
    # the same as without its label (from the same statistics: the order of a token's sums in the forward pass may
    # depend on where the labels around it are)
    without = labels.clone()
    without[1] = -1
    for a, b in zip(dfssm.head_loss_backward(W, sr, x, without, stats, dloss, norm_w=nw), (dx, ds, dn)):
        assert a is None or torch.equal(a, b)
    _, stats = dfssm.head_loss(W, sr, x, without, norm_w=nw)
    finite = dfssm.head_loss_backward(W, sr, x, without, stats, dloss, norm_w=nw)
    x[1, 3] = float("inf")
    _, stats = dfssm.head_loss(W, sr, x, without, norm_w=nw)
    for a, b in zip(dfssm.head_loss_backward(W, sr, x, without, stats, dloss, norm_w=nw), finite):
        assert a is None or torch.equal(a, b)
    _, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=nw)
    assert bool(dx[1].isnan().all()) and int(dx.isnan().sum()) == d
    assert bool(ds.isnan().all()) and (dn is None or bool(dn.isnan().all()))


# ------------------------------------------------------------------------------------ optional outputs


@pytest.mark.parametrize("n,V,d", [(1, 40, 16), (700, 90, 272), (3000, 5000, 4096), (17000, 300, 64)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_gradient_of_one_kind(dev, n, V, d, accumulate):
    """The table's or the row scales' gradient alone has the bits that it has beside the other, written or added."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(n + d, dev)
    W, _ = matrix(g, V, d, dev)
    tok = (torch.rand(n, generator=g, device=dev) ** 3 * V).int().clamp(max=V - 1)
    dh = torch.randn(n, d, generator=g, device=dev)

    def start():
        return (torch.full((V, d), 0.5, device=dev), torch.full((V,), 0.25, device=dev)) if accumulate else (None, None)

    both = dfssm.embed_tokens_backward(W, tok, dh, *start(), accumulate=accumulate)
    dE, none = dfssm.embed_tokens_backward(W, tok, dh, start()[0], accumulate=accumulate, scales=False)
    assert none is None and torch.equal(dE, both[0])
    none, ds = dfssm.embed_tokens_backward(W, tok, dh, None, start()[1], accumulate=accumulate, table=False)
    assert none is None and torch.equal(ds, both[1])


def test_embed_gradient_of_nothing_is_refused(dev):
    from bit_quantized_mamba_b200 import dfssm
    W, _ = matrix(gen(1, dev), 10, 32, dev)
    tok, dh = torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(2, 32, device=dev)
    with pytest.raises(ValueError):
        dfssm.embed_tokens_backward(W, tok, dh, table=False, scales=False)
    with pytest.raises(ValueError):
        dfssm.embed_tokens_backward(W, tok, dh, accumulate=True)


@pytest.mark.parametrize("M", [5, 200])
def test_head_gradient_without_the_norms(dev, M):
    """dnorm_w may be left out although there is a norm (through the C ABI): dx and ds_row keep their bits, what lies
    where it would be stays."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(M, dev)
    V, d = 800, 144
    W, sr = matrix(g, V, d, dev)
    x = torch.randn(M, d, generator=g, device=dev)
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    y = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    dl = torch.rand(M, generator=g, device=dev)
    _, stats = dfssm.head_loss(W, sr, x, y, norm_w=nw)
    dx, ds, _ = dfssm.head_loss_backward(W, sr, x, y, stats, dl, norm_w=nw)
    size = dfssm.workspace_size(dfssm.OP_HEAD_LOSS_BACKWARD, M, d, V)
    ws, dx2, ds2 = dfssm.workspace(size, dev), torch.zeros_like(dx), torch.zeros_like(ds)
    torch.cuda.synchronize()
    p = [t.data_ptr() for t in (W, sr, x, nw, y, stats, dl, dx2, ds2, ws)]
    for scale_grad in (p[8], None):
        assert dfssm.lib().dfssm_head_loss_backward(p[0], p[1], V, d, p[2], 0, d, M, p[3], p[4], p[5], p[6], p[7], d,
                                                    scale_grad, None, p[9], size, None) == 0
        torch.cuda.synchronize()
        assert torch.equal(dx2, dx) and torch.equal(ds2, ds)
        dx2.zero_()
        torch.cuda.synchronize()


# ------------------------------------------------------------------------------------ size of the errors


def scale_top(sr):
    """The row scale that the fixed point of du counts in, and whether rows are beyond it: the largest, or, where an
    eighth of 128 parts of the rows have nothing above an eighth of that, the largest part's maximum within 8 times the
    least but an eighth of the parts' (include/dfssm.h; parts are runs of 32 rows in turn, of one up to 4096 rows)."""
    s, V = sr.abs(), len(sr)
    run = 1 if V <= 4096 else 32
    part = torch.arange(V, device=s.device) // run % 128
    m = torch.zeros(128, device=s.device).scatter_reduce_(0, part, s, "amax")[:min(128, -(-V // run))].sort().values
    least = m[len(m) * 16 // 128]
    top = m[m <= 8 * least].max()
    return (float(top), True) if least < m[-1] / 8 and top < m[-1] else (float(m[-1]), False)


def error_sizes(ref, W, sr, labels):
    """Variances to expect of the errors of du [M][d] and ds_row [V].

    A coefficient c = |G s_row| of a token (G the derivative by the logit) has a relative error of about
    U (|l| + |m| + 4): the roundings of its logit and of the largest, the exponential, a few products.  In du it is
    rounded to steps of its fixed point with a dither, which has the variance f (1 - f) <= min(c / step, 1/4) steps
    squared.  Steps are 2^-24 (2^-23 with negative scales) of tau.  With p the token's largest |G| but the label's, S the
    others' sum in units of it and `top` as above, tau is top p 2^-k, k <= 4 the largest with S 2^k <= 32; where rows are
    beyond the top, C and A the largest and the sum of the token's c in those, it is the power of two above
    max(top p min(1, S / 16), min(C, A / 16)), and 2^-8 more; more than 1024 such rows count as if C were the largest
    scale times p, and A that times S.  The rows' errors are independent, so their squares add
    up, weighted with the squares of W."""
    u = base.U
    at = torch.where(ref["kept"], labels, torch.zeros_like(labels)).long()[:, None]
    s = sr.double().abs()
    L = ref["acc_s"] * sr.double()
    m = L.scatter(1, at, -float("inf")).amax(1, keepdim=True)
    r = u * (L.abs() + m.abs() + 4)
    c = ref["G"].abs() * s
    rest = c.scatter(1, at, 0.0)
    others = ref["G"].abs().scatter(1, at, 0.0)
    p = others.amax(1)
    S = others.sum(1) / p
    top, beyond = scale_top(sr)
    if beyond:
        out = rest[:, sr.abs() > top]
        C, A = (out.amax(1), out.sum(1)) if out.shape[1] <= 1024 else (s.max() * p, s.max() * p * S)
        tau = 2.02 * torch.maximum(top * p * (S / 16).clamp(max=1), torch.minimum(C, A / 16))
    else:
        tau = top * p * 2.0 ** -torch.floor(torch.log2(32 / (S * 1.0001))).clamp(0, 4)
    step = (2.0 ** -23 if bool((sr < 0).any()) else 2.0 ** -24) * tau[:, None]
    var = (r * c).square() + torch.minimum(rest * step, step.square() / 4)
    e_du = var @ W.double().square() + (u * ref["du"]).square()
    # products of three fp32 numbers, sums of 32 tokens in fp32
    e_ds = ((r + 6 * u) * ref["G"] * ref["acc_s"]).square().sum(0)
    return e_du, e_ds


def rms(x, dim=()):
    return x.double().square().mean(dim).sqrt()


ERROR_SHAPES = [(40, 20000, 512, 0.0), (40, 20000, 512, 0.5), (300, 20000, 512, 0.0), (300, 20000, 512, 0.5),
                (3, 5000, 1024, 0.2), (100, 3001, 256, 1.0), (600, 50288, 1040, 0.1)]
# row scales, and of how many rows (one by one, or side by side) they are larger, how much, and whether those rows have
# codes
ERROR_SCALES = [("even", 0, 1, False), ("even", 1, 10, False), ("even", 1, 1e2, False), ("even", 1, 1e4, False),
                ("even", 1, 1e4, True), ("even", 2, 1e5, True), ("even", 200, 1e3, True), ("signed", 0, 1, False),
                ("signed", 1, 1e3, True), ("decades", 0, 1, False), ("decades", 3, 1e3, True), ("even", -100, 1e3, False),
                ("even", -2000, 1e3, False)]


@pytest.mark.parametrize("kind,count,factor,codes", ERROR_SCALES)
@pytest.mark.parametrize("M,V,d,peak", ERROR_SHAPES)
def test_head_gradient_errors_in_the_mean(dev, M, V, d, peak, kind, count, factor, codes):
    """Errors of dx, the row scales' and the norm weight's gradient against their expected root mean square, token by
    token (three times) and altogether (twice), for flat and peaked distributions, and for row scales of very different
    sizes: a row whose scale is large must not cost the tokens that give it no weight their precision."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(140 + M, dev)
    W, sr = matrix(g, V, d, dev)
    if kind == "decades":
        sr = 10.0 ** (torch.rand(V, generator=g, device=dev) * -4 - 3)
    elif kind == "signed":
        sr = sr * (torch.randint(0, 2, (V,), generator=g, device=dev) * 2 - 1)
    if count:
        large = torch.randperm(V, generator=g, device=dev)[:count] if count > 0 else torch.arange(V + count - 7, V - 7)
        sr[large] = factor * sr.abs().max()
        if not codes:
            W[large] = 0
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    other = torch.randint(0, V, (M,), generator=g, device=dev)
    x = torch.randn(M, d, generator=g, device=dev) + peak * W[other].float() / 73
    dloss = torch.rand(M, generator=g, device=dev) + 0.5
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    torch.cuda.synchronize()
    for w in (None, nw):
        ref = base.head_reference(W, sr, x, w, labels, dloss)
        e_du, e_ds = error_sizes(ref, W, sr, labels)
        _, stats = dfssm.head_loss(W, sr, x, labels, norm_w=w)
        dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=w)
        got, want = rms(ds.double() - ref["ds"]), e_ds.mean().sqrt()
        print(f"ds {got / rms(ref['ds']):.2e} of {want / rms(ref['ds']):.2e}", end="; ")
        assert got <= 2 * want
        if w is None:
            got, want = rms(dx.double() - ref["dx"]), e_du.mean().sqrt()
            print(f"dx {got / rms(ref['dx']):.2e} of {want / rms(ref['dx']):.2e}", end="; ")
            assert got <= 2 * want
            got, want, size = rms(dx.double() - ref["dx"], 1), e_du.mean(1).sqrt(), rms(ref["dx"], 1)
            print(f"tokens {(got / size).median():.2e}, {(got / size).max():.2e} at most {(got / want).max():.2f} of expected")
            assert bool((got <= 3 * want).all())
        else:
            # a few fp32 roundings of each term, and of the sums
            n = x.double() * ref["inv"]
            got = rms(dn.double() - ref["dn"])
            want = ((e_du + (4 * base.U * ref["du"]).square()) * n.square()).sum(0).mean().sqrt()
            print(f"dnorm {got / rms(ref['dn']):.2e} of {want / rms(ref['dn']):.2e}")
            assert got <= 2 * want


@pytest.mark.parametrize("M,V,d,count", [(3, 40, 64, 2), (20, 9000, 272, 1), (20, 9000, 272, 300), (300, 9000, 144, 30),
                                         (300, 20000, 144, 1500), (700, 6000, 1040, 7)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_gradient_with_outlying_rows(dev, M, V, d, count, dtype):
    """Some rows' scales a thousand times the others', their labels among the tokens', ignored labels, strides: within the
    bounds, bit for bit again, and in a captured step."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(170 + M + count, dev)
    W, sr = matrix(g, V, d, dev)
    large = torch.randperm(V, generator=g, device=dev)[:count]
    sr[large] *= 1000
    x = base.rows(g, M, d, dev, dtype, pad=8)
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    labels[::4] = large[torch.arange(len(labels[::4]), device=dev) % count].int()
    labels[1::5] = -1
    dloss = torch.randn(M, generator=g, device=dev)
    base.check_head(dfssm, W, sr, x, nw, labels, dloss)
    size = dfssm.workspace_size
    ws = [dfssm.workspace(size(op, M, d, V), dev) for op in (dfssm.OP_HEAD_LOSS, dfssm.OP_HEAD_LOSS_BACKWARD)]

    def step():
        loss, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw, ws=ws[0])
        return [loss, *dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=nw, ws=ws[1])]

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M", [1, 3, 16, 40, 128, 500])
def test_loss_of_confident_tokens_in_the_mean(dev, M):
    """Tokens whose label's logit is tens above flat others: the relative error of a loss near exp(-z) is the error of z.
    The label's logit, the largest number there, must not cost it fp32's rounding (U |l| / sqrt 3 in the mean, 2e-6 to
    4e-6 here).  What remains: the others' logits (two roundings of at most max|l| = 6 each, independent over thousands of
    rows), their exponentials (2^-22 each, likewise), the sums of up to 20000 positive terms by threads that each add
    some tens or hundreds (a few U), and five roundings after z: 12 U in the mean."""
    from bit_quantized_mamba_b200 import dfssm
    d, V = 1024, 20000
    got = []
    for k in range(-(-60 // M)):
        g = gen(500 + M + k, dev)
        W, sr = matrix(g, V, d, dev)
        labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
        x = torch.randn(M, d, generator=g, device=dev)
        x += (torch.rand(M, 1, generator=g, device=dev) * 1.5 + 0.8) * W[labels.long()].float() / 73
        torch.cuda.synchronize()
        ref = base.head_reference(W, sr, x, None, labels)
        loss, _ = dfssm.head_loss(W, sr, x, labels)
        L = ref["loss"]
        some = (L > 1e-30) & (L < 1e-6)
        got.append(((loss.double() - L) / L)[some])
    got = torch.cat(got)
    print(f"{len(got)} tokens, {rms(got):.2e}")
    assert len(got) >= 8 and float(rms(got)) <= 12 * base.U
