"""The many-token operators on the int8 matrix (int8 linear, embedding and its gradient, vocabulary cross
entropy and its gradient) against plain 64-bit evaluations of their definitions.

Bars: codes, accumulators, linear outputs and embeddings equal (the definitions fix every rounding);
losses and gradients within bounds derived from the roundings the kernels make (u = 2^-24, half an fp32
step), written beside each check.
"""
import numpy as np
import pytest
import torch

import oracle
from bit_quantized_mamba_b200 import inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
F8 = torch.float64


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_mamba_b200 import build, dfssm
    build.build()
    dfssm.lib()
    return torch.device("cuda:0")


def matrix(g, V, d, dev, signed=False):
    W = torch.randint(-127, 128, (V, d), generator=g, device=dev, dtype=torch.int8)
    s = torch.rand(V, generator=g, device=dev) * 9e-4 + 1e-4
    if signed:
        s = s * (torch.randint(0, 2, (V,), generator=g, device=dev) * 2 - 1)
    return W, s


def gen(seed, dev):
    return torch.Generator(dev).manual_seed(seed)


def rows(g, M, d, dev, dtype, pad=0):
    """M rows of d values inside rows of d + pad."""
    x = torch.randn(M, d + pad, generator=g, device=dev).to(dtype)
    return x[:, :d] if pad else x


def quantized(x, norm_w):
    """The definition: u (fp32), codes (fp64), scale (fp32), 1/rms (fp64)."""
    xf = x.float()
    inv = None
    u = xf
    if norm_w is not None:
        inv = 1.0 / torch.sqrt(xf.double().square().mean(1, keepdim=True) + EPS)
        u = xf * inv.float() * norm_w
    s = (u.abs().amax(1, keepdim=True).double() / 127).float()
    q = torch.where(s > 0, torch.round(u / s), torch.zeros_like(u)).clamp(-127, 127)
    return u, q.double(), s, inv


def status_ok(dfssm, ws):
    assert dfssm.device_status(ws) == 0


# ------------------------------------------------------------------------------------ int8 linear

SHAPES = [(1, 1, 16), (1, 33, 48), (3, 31, 128), (16, 257, 144), (17, 1187, 2048), (64, 500, 272), (255, 129, 160),
          (256, 400, 1024), (257, 300, 640), (300, 1187, 4112), (513, 128, 16), (2, 100, 8192), (129, 4097, 64)]


@pytest.mark.parametrize("M,V,d", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_int8_equals_definition(dev, M, V, d, dtype):
    from bit_quantized_mamba_b200 import dfssm
    g = gen(M * 1000 + V + d, dev)
    W, sr = matrix(g, V, d, dev, signed=True)
    x = rows(g, M, d, dev, dtype, pad=8 if M % 2 else 0)
    nw = torch.rand(d, generator=g, device=dev) + 0.5 if M % 3 else None
    ws = dfssm.workspace(dfssm.workspace_size(dfssm.OP_LINEAR_INT8, M, d, V), dev)
    taps = dict(acc=torch.zeros(M, V, dtype=torch.int32, device=dev), xq=torch.zeros(M, d, dtype=torch.int8, device=dev),
                xscale=torch.zeros(M, device=dev))
    _, q, s, _ = quantized(x, nw)
    acc = q @ W.double().t()
    want = (acc * s.double() * sr.double()).float()
    wide = torch.full((M, V + 3), 7.0, device=dev)
    y = dfssm.linear_int8(W, sr, x, y=wide[:, :V], norm_w=nw, ws=ws, debug=taps)
    status_ok(dfssm, ws)
    assert torch.equal(taps["xq"].double(), q)
    assert torch.equal(taps["xscale"], s[:, 0])
    assert torch.equal(taps["acc"].double(), acc)
    assert torch.equal(y, want)
    assert bool((wide[:, V:] == 7.0).all())  # what lies between rows is left as it was
    yb = dfssm.linear_int8(W, sr, x, norm_w=nw, out_dtype=torch.bfloat16)
    assert torch.equal(yb, want.bfloat16())


def test_linear_int8_is_the_heads_product(dev):
    """Row for row the single-token head's logits, on the GPU and in the oracle."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(5, dev)
    V, d, M = 5003, 2048, 5
    W, sr = matrix(g, V, d, dev)
    x = rows(g, M, d, dev, torch.float32)
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    y = dfssm.linear_int8(W, sr, x)
    yn = dfssm.linear_int8(W, sr, x, norm_w=nw)
    for t in range(M):
        assert torch.equal(y[t], dfssm.lm_head(W, sr, x[t].contiguous()))
        assert torch.equal(yn[t], dfssm.head_greedy(W, sr, x[t].contiguous(), nw)[1])
    ref, _ = oracle.final_head(W.cpu().numpy(), sr.cpu().numpy(), x[0].cpu().numpy(), nw.cpu().numpy())
    assert np.array_equal(yn[0].cpu().numpy(), ref)


def test_linear_int8_extremes(dev):
    """Largest accumulators (d = 8192, every product 127 * -128), zero rows, tiny rows, rows that are not
    finite (NaN in their own outputs only)."""
    from bit_quantized_mamba_b200 import dfssm
    V, d = 40, 8192
    W = torch.full((V, d), -128, dtype=torch.int8, device=dev)
    W[1::2] = 127
    sr = torch.linspace(1e-4, 1e-3, V, device=dev)
    x = torch.ones(6, d, device=dev)
    x[1] = 0.0
    x[2] = 1e-38
    x[3, 17] = float("nan")
    x[4, 8191] = float("inf")
    acc = torch.zeros(6, V, dtype=torch.int32, device=dev)
    y = dfssm.linear_int8(W, sr, x, debug=dict(acc=acc))
    _, q, s, _ = quantized(x[:3], None)
    want = (q @ W.double().t() * s.double() * sr.double()).float()
    assert torch.equal(y[:3], want)
    assert int(acc[0, 0]) == -128 * 127 * d
    assert bool(y[3:5].isnan().all())
    assert torch.equal(y[5], y[0])


# ------------------------------------------------------------------------------------ embedding


@pytest.mark.parametrize("n,V,d", [(1, 1, 16), (5, 7, 48), (333, 1187, 2048), (2500, 64, 1040), (3, 20, 8192)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_embed_tokens_equals_definition(dev, n, V, d, dtype):
    from bit_quantized_mamba_b200 import dfssm
    g = gen(n + V + d, dev)
    W, sr = matrix(g, V, d, dev)
    tok = torch.randint(0, V, (n,), generator=g, device=dev, dtype=torch.int32)
    ws = dfssm.workspace(dfssm.workspace_size(dfssm.OP_EMBED_TOKENS, 0, 0, 0), dev)
    wide = torch.full((n + 1, d + 8), 7.0, device=dev, dtype=dtype)
    h = dfssm.embed_tokens(W, sr, tok, h=wide[:n, :d], ws=ws)
    status_ok(dfssm, ws)
    want = (W[tok.long()].double() * sr[tok.long(), None].double()).float().to(dtype)
    assert torch.equal(h, want)
    assert bool((wide[n] == 7.0).all()) and bool((wide[:, d:] == 7.0).all())
    one = dfssm.embed(W, sr, tok[:1])
    assert torch.equal(one, (W[tok[0].long()].float() * sr[tok[0].long()]))


def test_embed_tokens_reports_a_bad_token(dev):
    from bit_quantized_mamba_b200 import dfssm
    g = gen(2, dev)
    W, sr = matrix(g, 50, 64, dev)
    ws = dfssm.workspace(256, dev)
    tok = torch.tensor([3, 50, -1, 49], dtype=torch.int32, device=dev)
    h = dfssm.embed_tokens(W, sr, tok, ws=ws)
    assert dfssm.device_status(ws) == -1
    assert not h[1].any() and not h[2].any() and h[0].any() and h[3].any()
    bw = dfssm.workspace(dfssm.workspace_size(dfssm.OP_EMBED_BACKWARD, 4, 64, 50), dev)
    dh = torch.ones(4, 64, device=dev)
    dE, ds = dfssm.embed_tokens_backward(W, tok, dh, ws=bw)
    assert dfssm.device_status(bw) == -1
    assert float(dE.sum()) == 128.0 and bool((dE[[3, 49]] == 1).all())
    status_ok(dfssm, bw)


def embed_grad_reference(W, tok, dh):
    i = tok.long()
    dE = torch.zeros(W.shape, dtype=F8, device=W.device).index_add_(0, i, dh.double())
    mag = torch.zeros(W.shape, dtype=F8, device=W.device).index_add_(0, i, dh.double().abs())
    n = torch.bincount(i, minlength=W.shape[0]).double()
    return dE, mag, n


@pytest.mark.parametrize("n,V,d,kind", [
    (1, 1, 16, "uniform"), (7, 5, 48, "uniform"), (500, 1187, 2048, "uniform"), (500, 40, 1040, "skew"),
    (4097, 70000, 64, "uniform"), (1000, 300, 4096, "skew"), (130, 20, 8192, "skew"), (3000, 9, 128, "same"),
    (16384, 5000, 128, "skew"), (16385, 5000, 128, "skew"), (40000, 70001, 32, "skew"), (20000, 3, 64, "same")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_embed_gradient(dev, n, V, d, kind, dtype):
    from bit_quantized_mamba_b200 import dfssm
    g = gen(n + V + d, dev)
    W, _ = matrix(g, V, d, dev)
    if kind == "uniform":
        tok = torch.randint(0, V, (n,), generator=g, device=dev, dtype=torch.int32)
    elif kind == "skew":
        tok = (torch.rand(n, generator=g, device=dev) ** 4 * V).int().clamp(max=V - 1)
    else:
        tok = torch.full((n,), V - 1, dtype=torch.int32, device=dev)
    dh = rows(g, n, d, dev, dtype, pad=16 if n % 2 else 0)
    ws = dfssm.workspace(dfssm.workspace_size(dfssm.OP_EMBED_BACKWARD, n, d, V), dev)
    dE, ds = dfssm.embed_tokens_backward(W, tok, dh, ws=ws)
    status_ok(dfssm, ws)
    ref, mag, cnt = embed_grad_reference(W, tok, dh)
    # n - 1 fp32 additions per sum, each off by at most U of a partial sum that mag bounds
    assert bool(((dE.double() - ref).abs() <= U * 1.01 * (cnt - 1).clamp(min=0)[:, None] * mag).all())
    # the products with W add d more roundings of terms that 128 mag bounds
    bound = U * 1.01 * ((cnt + d)[:, None] * W.double().abs() * mag).sum(1)
    assert bool(((ds.double() - (ref * W.double()).sum(1)).abs() <= bound).all())
    # the same again on the same workspace: bit for bit
    dE2, ds2 = dfssm.embed_tokens_backward(W, tok, dh, ws=ws)
    assert torch.equal(dE, dE2) and torch.equal(ds, ds2)
    # added to what is there: one more rounding; untouched rows keep their bits (a NaN among them)
    base = torch.randn(V, d, generator=g, device=dev)
    free = torch.nonzero(cnt == 0)
    if len(free):
        base[free[0, 0]] = float("nan")
    into, into_s = base.clone(), torch.ones(V, device=dev)
    dfssm.embed_tokens_backward(W, tok, dh, dE=into, ds_row=into_s, accumulate=True, ws=ws)
    hit = cnt > 0
    assert torch.equal(into[~hit].view(torch.int32), base[~hit].view(torch.int32))
    assert torch.equal(into[hit], (base[hit] + dE[hit]))
    assert torch.equal(into_s, torch.where(hit, 1 + ds, torch.ones_like(ds)))


def test_embed_gradient_without_tokens(dev):
    from bit_quantized_mamba_b200 import dfssm
    W = torch.ones(10, 32, dtype=torch.int8, device=dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    dE, ds = dfssm.embed_tokens_backward(W, none, torch.zeros(0, 32, device=dev))
    assert not dE.any() and not ds.any()
    one = torch.ones(10, 32, device=dev)
    dfssm.embed_tokens_backward(W, none, torch.zeros(0, 32, device=dev), dE=one, accumulate=True)
    assert bool((one == 1).all())


# ------------------------------------------------------------------------------------ loss


def head_reference(W, sr, x, nw, labels, dloss=None):
    """Losses and gradients in fp64, and what the bounds need."""
    u, q, s, inv = quantized(x, nw)
    z = q * s.double()
    acc_s = z @ W.double().t()
    L = acc_s * sr.double()
    y = labels.long()
    kept = (y >= 0) & (y < W.shape[0])
    lse = torch.logsumexp(L, 1)
    at = torch.where(kept, y, torch.zeros_like(y))
    ly = L.gather(1, at[:, None])[:, 0]
    L2 = L.clone().scatter_(1, at[:, None], -float("inf"))
    rest = torch.logsumexp(L2, 1)  # -inf when the vocabulary is one row
    loss = torch.where(kept, torch.nn.functional.softplus(rest - ly, threshold=700.0), torch.zeros_like(lse))
    loss = torch.where(torch.isinf(rest), torch.zeros_like(loss), loss)
    out = dict(loss=loss, top=L.abs().amax(1), kept=kept)
    if dloss is None:
        return out
    G = torch.softmax(L, 1)
    G.scatter_(1, at[:, None], (-1 / (1 + torch.exp(ly - rest)))[:, None])
    G = G * (dloss.double() * kept)[:, None]
    du = G @ (W.double() * sr.double()[:, None])
    out.update(du=du, ds=(G * acc_s).sum(0), G=G, acc_s=acc_s, inv=inv, u=u,
               pmax=torch.exp(L2.amax(1) - lse) * kept)
    if nw is None:
        out["dx"] = du
        return out
    h = x.double()
    n = h * inv
    v = du * nw.double()
    out["dx"] = inv * (v - n * (v * n).mean(1, keepdim=True))
    out["dn"] = (du * n).sum(0)
    return out


def loss_bound(ref):
    """Logits: three roundings each (scale, product, difference), so 3 U |l| for the largest, and as much for the
    label's; exp2 is within 2^-22 and a thread's running sum of up to 128 terms per tile, some tens of tiles,
    rounds by at most U each (512 in all); one rounding of the loss."""
    return U * (6 * ref["top"] + 512 + ref["loss"]) + 2.0 ** -22


def grad_bounds(ref, W, sr, nw, dloss, x):
    """p is off by rel = 6 U max|l| + 2^-22 + 520 U of itself; a coefficient is off by half a step more (at most
    2^-24 of its largest value, pmax max|s_row|); du is rounded to fp32.  The linear steps after that carry the
    bound with them, with a few more roundings of what they add.  exp(l - m) below the normal range (2^-126) counts
    as zero: in ds that is at most 2^-126 pmax |g acc s| a token (logits hundreds apart; du's step is larger)."""
    rel = U * (6 * ref["top"] + 520) + 2.0 ** -22
    g = dloss.double().abs() * ref["kept"]
    A = W.double().abs()
    mag = ref["G"].abs() @ (A * sr.double().abs()[:, None])
    step = 2.0 ** -24 * 1.001 * ref["pmax"] * g * float(sr.abs().max())
    e_du = rel[:, None] * mag + step[:, None] * A.sum(0)[None, :] + U * ref["du"].abs()
    e_ds = (rel[:, None] * ref["G"].abs() * ref["acc_s"].abs()).sum(0) * 1.01 + 40 * U * (ref["G"] * ref["acc_s"]).abs().sum(0)
    e_ds = e_ds + 2.0 ** -126 * ((ref["pmax"] * g)[:, None] * ref["acc_s"].abs()).sum(0)
    if nw is None:
        return e_du, e_ds, None
    n = (x.double() * ref["inv"]).abs()
    v, e_v = (ref["du"] * nw.double()).abs(), (e_du * nw.double())
    mean_v, mean_e = (v * n).mean(1, keepdim=True), (e_v * n).mean(1, keepdim=True)
    e_dx = ref["inv"] * (e_v + n * mean_e + 8 * U * (v + n * mean_v))
    parts = ref["du"].shape[0]
    e_dn = (e_du * n).sum(0) + U * (6 + parts) * (ref["du"].abs() * n).sum(0)
    return e_dx, e_ds, e_dn


def check_head(dfssm, W, sr, x, nw, labels, dloss):
    M, d = x.shape
    V = W.shape[0]
    dev = x.device
    ws = dfssm.workspace(dfssm.workspace_size(dfssm.OP_HEAD_LOSS, M, d, V), dev)
    bw = dfssm.workspace(dfssm.workspace_size(dfssm.OP_HEAD_LOSS_BACKWARD, M, d, V), dev)
    ref = head_reference(W, sr, x, nw, labels, dloss)
    loss, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw, ws=ws)
    status_ok(dfssm, ws)
    assert bool(((loss.double() - ref["loss"]).abs() <= loss_bound(ref)).all())
    assert not loss[~ref["kept"]].any()
    wide = torch.full((M + 1, d + 8), 7.0, device=dev, dtype=x.dtype)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=nw, dx=wide[:M, :d], ws=bw)
    status_ok(dfssm, bw)
    e_dx, e_ds, e_dn = grad_bounds(ref, W, sr, nw, dloss, x)
    if x.dtype == torch.bfloat16:
        e_dx = e_dx + (ref["dx"].abs() + e_dx) * 2.0 ** -8 + 2.0 ** -134  # one rounding to bf16
    assert bool(((dx.double() - ref["dx"]).abs() <= e_dx + 1e-45).all())
    assert bool(((ds.double() - ref["ds"]).abs() <= e_ds + 1e-45).all())
    assert bool((wide[M] == 7.0).all()) and bool((wide[:, d:] == 7.0).all())
    assert not dx[~ref["kept"]].any()
    if nw is not None:
        assert bool(((dn.double() - ref["dn"]).abs() <= e_dn + 1e-45).all())
    else:
        assert dn is None
    # again, on the same workspaces and without the scales' gradient: bit for bit
    loss2, stats2 = dfssm.head_loss(W, sr, x, labels, norm_w=nw, ws=ws)
    dx2, none, dn2 = dfssm.head_loss_backward(W, sr, x, labels, stats2, dloss, norm_w=nw, scales=False, ws=bw)
    assert none is None
    assert torch.equal(loss, loss2) and torch.equal(stats, stats2) and torch.equal(dx, dx2)
    assert nw is None or torch.equal(dn, dn2)
    dx3, ds3, _ = dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=nw, ws=bw)
    assert torch.equal(ds, ds3) and torch.equal(dx, dx3)
    return ref, loss, dx


HEAD_SHAPES = [(1, 1, 16), (1, 2, 16), (2, 31, 48), (3, 33, 128), (16, 257, 144), (17, 1187, 2048), (127, 300, 272),
               (128, 129, 160), (129, 256, 64), (255, 1000, 96), (256, 2500, 128), (257, 300, 640), (300, 4999, 1040),
               (513, 511, 16), (5, 700, 8192), (40, 9000, 4112), (1100, 6000, 144)]


@pytest.mark.parametrize("M,V,d", HEAD_SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_loss_and_gradients(dev, M, V, d, dtype):
    from bit_quantized_mamba_b200 import dfssm
    g = gen(M + V + d, dev)
    W, sr = matrix(g, V, d, dev, signed=V % 2 == 0)
    x = rows(g, M, d, dev, dtype, pad=8 if V % 3 else 0)
    nw = torch.rand(d, generator=g, device=dev) + 0.5 if M % 2 else None
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    labels[torch.rand(M, generator=g, device=dev) < 0.2] = -100
    dloss = torch.randn(M, generator=g, device=dev)
    check_head(dfssm, W, sr, x, nw, labels, dloss)


@pytest.mark.parametrize("M,V,d,signed", [(300, 70000, 48, False), (20, 140000, 32, True), (4096, 9000, 64, False),
                                          (64, 66000, 16, False), (65, 1000, 4096, True)])
def test_head_gradient_in_pieces_of_the_vocabulary(dev, M, V, d, signed):
    """Vocabularies of several pieces, and past one set of int32 accumulators; token counts at the kernels' limits."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(M + V, dev)
    W, sr = matrix(g, V, d, dev, signed=signed)
    x = rows(g, M, d, dev, torch.float32)
    labels = torch.randint(-V // 9, V, (M,), generator=g, device=dev, dtype=torch.int32)
    check_head(dfssm, W, sr, x, torch.rand(d, generator=g, device=dev) + 0.5, labels, torch.rand(M, generator=g, device=dev))


@pytest.mark.parametrize("M,V,d", [(2100, 3001, 2048), (1300, 2500, 1536), (1300, 1000, 1024), (2304, 700, 640),
                                   (128, 1500, 8192), (600, 26000, 1040), (2048, 50288, 2048)])
def test_head_gradient_in_rounds_of_whole_units(dev, M, V, d):
    """Sizes whose second product has whole units for every SM: with a full last round, one split along K, none, and
    in two pieces of the vocabulary."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(M + V + d, dev)
    W, sr = matrix(g, V, d, dev)
    x = rows(g, M, d, dev, torch.float32)
    labels = torch.randint(-V // 9, V, (M,), generator=g, device=dev, dtype=torch.int32)
    check_head(dfssm, W, sr, x, torch.rand(d, generator=g, device=dev) + 0.5, labels, torch.rand(M, generator=g, device=dev))


def test_head_gradient_of_constant_rows_stays_in_range(dev):
    """Every code at its limit and uniform coefficients: the largest digit sums there can be."""
    from bit_quantized_mamba_b200 import dfssm
    V, d, M = 65536, 16, 3
    for code in (-128, 127):
        W = torch.full((V, d), code, dtype=torch.int8, device=dev)
        sr = torch.full((V,), 1e-3, device=dev)
        x = torch.randn(M, d, generator=gen(3, dev), device=dev)
        labels = torch.tensor([0, V - 1, 77], dtype=torch.int32, device=dev)
        check_head(dfssm, W, sr, x, None, labels, torch.ones(M, device=dev))


@pytest.mark.parametrize("strength", [0.3, 1.0, 4.0])
def test_head_loss_of_confident_tokens(dev, strength):
    """Tokens that point at their label, up to losses far below the fp32 step of the logits: loss and gradient
    keep their relative precision (the bounds scale with 1 - p)."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(9, dev)
    V, d, M = 3000, 512, 70
    W, sr = matrix(g, V, d, dev)
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    x = torch.randn(M, d, generator=g, device=dev) + strength * W[labels.long()].float() / 70
    dloss = torch.rand(M, generator=g, device=dev)
    ref, loss, dx = check_head(dfssm, W, sr, x, None, labels, dloss)
    rel = U * (12 * ref["top"] + 600) + 2.0 ** -21
    assert bool(((loss.double() - ref["loss"]).abs() <= rel * ref["loss"] + 1e-45).all())


def test_head_loss_masks_and_odd_tokens(dev):
    """All labels ignored; a label outside the vocabulary; zero tokens' rows; rows that are not finite."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(11, dev)
    V, d, M = 700, 128, 40
    W, sr = matrix(g, V, d, dev)
    x = rows(g, M, d, dev, torch.float32)
    ones = torch.ones(M, device=dev)
    none = torch.full((M,), -1, dtype=torch.int32, device=dev)
    loss, stats = dfssm.head_loss(W, sr, x, none)
    dx, ds, _ = dfssm.head_loss_backward(W, sr, x, none, stats, ones)
    assert not loss.any() and not dx.any() and not ds.any()
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    labels[3], labels[5] = V, -1
    x[5, 7] = float("nan")  # ignored: stays without effect
    x[6] = 0.0              # uniform logits
    ws = dfssm.workspace(dfssm.workspace_size(dfssm.OP_HEAD_LOSS, M, d, V), dev)
    loss, stats = dfssm.head_loss(W, sr, x, labels, ws=ws)
    assert dfssm.device_status(ws) == -1
    status_ok(dfssm, ws)
    assert float(loss[3]) == 0 and float(loss[5]) == 0 and bool(loss.isfinite().all())
    assert abs(float(loss[6]) - np.log(V)) <= U * (np.log(V) + 512) + 2.0 ** -22
    dx, ds, _ = dfssm.head_loss_backward(W, sr, x, labels, stats, ones)
    assert not dx[3].any() and not dx[5].any()
    assert bool(dx.isfinite().all()) and bool(ds.isfinite().all())
    x[8, 100] = float("inf")
    loss, stats = dfssm.head_loss(W, sr, x, labels)
    assert bool(loss[8].isnan()) and int(loss.isnan().sum()) == 1
    dx, ds, _ = dfssm.head_loss_backward(W, sr, x, labels, stats, ones)
    assert bool(dx[8].isnan().all()) and int(dx.isnan().sum()) == d
    # no tokens at all
    empty = torch.zeros(0, d, device=dev)
    noi = torch.zeros(0, dtype=torch.int32, device=dev)
    nw = torch.ones(d, device=dev)
    loss, stats = dfssm.head_loss(W, sr, empty, noi, norm_w=nw)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, empty, noi, stats, torch.zeros(0, device=dev), norm_w=nw,
                                          ds_row=torch.ones(V, device=dev), dnorm_w=torch.ones(d, device=dev))
    assert loss.numel() == 0 and dx.numel() == 0 and not ds.any() and not dn.any()
    assert dfssm.linear_int8(W, sr, empty).shape == (0, V)


def test_head_loss_row_scales_of_zero_and_large_logits(dev):
    """Scales of zero (no row left but flat logits), and logits in the hundreds."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(12, dev)
    V, d, M = 900, 256, 33
    W, sr = matrix(g, V, d, dev)
    x = rows(g, M, d, dev, torch.float32)
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    dloss = torch.rand(M, generator=g, device=dev)
    check_head(dfssm, W, torch.zeros_like(sr), x, None, labels, dloss)
    half = sr.clone()
    half[::2] = 0
    check_head(dfssm, W, half, x, None, labels, dloss)
    check_head(dfssm, W, sr * 300, x, None, labels, dloss)


def test_head_gradients_against_differences(dev):
    """Central differences of the fp64 loss at the dequantised activations, along random directions: of x through
    the norm, of the row scales and of the norm weight."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(13, dev)
    V, d, M = 400, 64, 9
    W, sr = matrix(g, V, d, dev)
    sr = sr * 5
    x = rows(g, M, d, dev, torch.float32)
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    labels = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    labels[4] = -1
    dloss = torch.rand(M, generator=g, device=dev)
    _, stats = dfssm.head_loss(W, sr, x, labels, norm_w=nw)
    dx, ds, dn = dfssm.head_loss_backward(W, sr, x, labels, stats, dloss, norm_w=nw)
    u, q, s, _ = quantized(x, nw)
    zhat = q * s.double()

    def norm(h, w):
        return h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w

    def total(h, scales, w):
        z = zhat + norm(h, w) - norm(x.double(), nw.double())  # straight through the int8 rounding
        L = z @ W.double().t() * scales
        kept = labels >= 0
        at = labels.long().clamp(min=0)
        return ((torch.logsumexp(L, 1) - L.gather(1, at[:, None])[:, 0]) * dloss.double() * kept).sum()

    X, S, N = x.double(), sr.double(), nw.double()
    for k in range(4):
        for name, grad, args in (("x", dx, 0), ("s", ds, 1), ("n", dn, 2)):
            base = [X, S, N]
            v = torch.randn(base[args].shape, generator=g, device=dev, dtype=F8) * base[args].abs().mean()
            e = 1e-5
            up, dn_ = list(base), list(base)
            up[args] = base[args] + e * v
            dn_[args] = base[args] - e * v
            diff = float((total(*up) - total(*dn_)) / (2 * e))
            got = float((grad.double() * v).sum())
            # e^2 third-order terms and the fp32 gradient's own error
            assert abs(got - diff) <= 2e-5 * float((grad.double().abs() * v.abs()).sum()), (name, k)


# ------------------------------------------------------------------------------------ used together


def training_step(dfssm, W, sr, nw, tok, labels, dloss, ws):
    h = dfssm.embed_tokens(W, sr, tok, ws=ws[0])
    loss, stats = dfssm.head_loss(W, sr, h, labels, norm_w=nw, ws=ws[1])
    dh, ds, dn = dfssm.head_loss_backward(W, sr, h, labels, stats, dloss, norm_w=nw, ws=ws[2])
    dE, ds2 = dfssm.embed_tokens_backward(W, tok, dh, ws=ws[3])
    return loss, dE, ds + ds2, dn


def workspaces(dfssm, M, d, V, dev):
    return [dfssm.workspace(dfssm.workspace_size(op, M, d, V), dev)
            for op in (dfssm.OP_EMBED_TOKENS, dfssm.OP_HEAD_LOSS, dfssm.OP_HEAD_LOSS_BACKWARD, dfssm.OP_EMBED_BACKWARD)]


def test_training_step_in_a_graph_and_on_another_stream(dev):
    """Embedding -> loss -> gradients: eager, captured and replayed on new tokens, and two steps at once on two
    streams with workspaces of their own, all bit-identical."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(21, dev)
    V, d, M = 3001, 256, 300
    W, sr = matrix(g, V, d, dev)
    nw = torch.rand(d, generator=g, device=dev) + 0.5
    batches = [(torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32),
                torch.randint(-1, V, (M,), generator=g, device=dev, dtype=torch.int32)) for _ in range(3)]
    dloss = torch.full((M,), 1 / M, device=dev)
    ws = workspaces(dfssm, M, d, V, dev)
    eager = [[t.clone() for t in training_step(dfssm, W, sr, nw, t, y, dloss, ws)] for t, y in batches]
    tok, lab = batches[0][0].clone(), batches[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = training_step(dfssm, W, sr, nw, tok, lab, dloss, ws)
    for k in (1, 2, 0):
        tok.copy_(batches[k][0])
        lab.copy_(batches[k][1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager[k]):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [ws, workspaces(dfssm, M, d, V, dev)]
    torch.cuda.synchronize()
    got = []
    for k, s in enumerate(streams):
        with torch.cuda.stream(s):
            got.append(training_step(dfssm, W, sr, nw, *batches[k], dloss, wss[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(got[k], eager[k]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_parameters_updated_in_the_stream(dev, M):
    """Row scales and norm weights that the stream itself updates between steps (a captured loop without a pause
    between its kernels) give the bits of steps taken one at a time."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(23, dev)
    V, d, n = 1501, 512, 4
    W, sr0 = matrix(g, V, d, dev)
    nw0 = torch.rand(d, generator=g, device=dev) + 0.5
    tok = torch.randint(0, V, (n, M), generator=g, device=dev, dtype=torch.int32)
    lab = torch.randint(-1, V, (n, M), generator=g, device=dev, dtype=torch.int32)
    dloss = torch.full((M,), 1 / M, device=dev)
    ws = workspaces(dfssm, M, d, V, dev)
    sr, nw, t, y = sr0.clone(), nw0.clone(), tok[0].clone(), lab[0].clone()

    def steps(pause):
        sr.copy_(sr0), nw.copy_(nw0)
        outs = []
        for k in range(n):
            t.copy_(tok[k]), y.copy_(lab[k])
            pause()
            out = training_step(dfssm, W, sr, nw, t, y, dloss, ws)
            pause()
            outs.append(out)
            sr.mul_(1.25), nw.mul_(0.75)
        return outs

    want = [[a.clone() for a in out] for out in steps(torch.cuda.synchronize)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(lambda: None)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_offsets_past_32_bits(dev):
    """Outputs, gradients and accumulators of more than 2^31 elements, and rows 2^31 - 1 apart: the last tokens get
    the bits that they get in a small call."""
    from bit_quantized_mamba_b200 import dfssm
    g = gen(24, dev)
    W, sr = matrix(g, 50000, 16, dev)
    x = rows(g, 45000, 16, dev, torch.bfloat16)
    y = dfssm.linear_int8(W, sr, x, out_dtype=torch.bfloat16)
    assert y.numel() > 2 ** 31
    assert torch.equal(y[-300:], dfssm.linear_int8(W, sr, x[-300:], out_dtype=torch.bfloat16))
    del y
    far = torch.empty(3 * (2 ** 31 - 1), device=dev, dtype=torch.bfloat16).as_strided((3, 50000), (2 ** 31 - 1, 1))
    dfssm.linear_int8(W, sr, x[:3], y=far)
    assert torch.equal(far, dfssm.linear_int8(W, sr, x[:3], out_dtype=torch.bfloat16))
    del far
    M, V, d = 100000, 300, 8192  # three digits of 819 M accumulators
    W, sr = matrix(g, V, d, dev)
    x = rows(g, M, d, dev, torch.bfloat16)
    lab = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
    dl = torch.rand(M, generator=g, device=dev)
    loss, stats = dfssm.head_loss(W, sr, x, lab)
    dx, _, _ = dfssm.head_loss_backward(W, sr, x, lab, stats, dl, scales=False)
    few = slice(M - 300, M)
    loss1, _ = dfssm.head_loss(W, sr, x[few], lab[few])
    # (the forward's sums are grouped by its tiles: equal up to their roundings, so the same statistics go in)
    assert torch.allclose(loss[few], loss1, rtol=0, atol=40 * U * float(loss1.abs().max() + 10))
    dx1, _, _ = dfssm.head_loss_backward(W, sr, x[few], lab[few], stats[:, few].contiguous(), dl[few], scales=False)
    assert torch.equal(dx[few], dx1)
    del x, dx, dx1
    V = 300000  # 2.5 G elements of the dense gradient
    W = torch.ones(V, d, device=dev, dtype=torch.int8)
    tok = torch.tensor([V - 1, 5, V - 1, 262144], device=dev, dtype=torch.int32)
    dh = rows(g, 4, d, dev, torch.float32)
    dE, ds = dfssm.embed_tokens_backward(W, tok, dh)
    assert torch.equal(dE[V - 1], dh[0] + dh[2]) and torch.equal(dE[5], dh[1]) and torch.equal(dE[262144], dh[3])
    assert int(torch.count_nonzero(dE[300:262144:997])) == 0 and int(torch.count_nonzero(ds)) == 3


def test_outputs_allocated_for_an_explicit_stream(dev):
    from bit_quantized_mamba_b200 import dfssm
    g = gen(22, dev)
    W, sr = matrix(g, 5000, 512, dev)
    x = rows(g, 40, 512, dev, torch.float32)
    want = dfssm.linear_int8(W, sr, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = dfssm.linear_int8(W, sr, x, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    y = dfssm.linear_int8(W, sr, x, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, want)


def test_scoring_a_prompt_matches_generation_logits(dev):
    """A prompt embedded, taken through the layer stack and scored: the losses are those of the logits that the
    one-token head gives for the same hidden states."""
    from bit_quantized_mamba_b200 import dfssm
    dims = dict(d_model=128, nheads=8, headdim=32, d_state=16, ngroups=1)
    m = inputs.generation_model(seed=8, n_layers=2, vocab=1187, **dims)
    conv, ssm = inputs.zero_states(1, 2, 8, 32, 16, 1)
    layers = [dfssm.Layer.from_host(l, dev) for l in m["layers"]]
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    stack = dfssm.LayerStack(layers, dims, [to(c) for c in conv], [to(s) for s in ssm])
    W, sr, nw = to(m["emb_w"]), to(m["emb_s"]), to(m["final_norm_w"])
    g = np.random.default_rng(3)
    text = to(g.integers(0, 1187, size=21).astype(np.int32))
    h = dfssm.embed_tokens(W, sr, text[:-1].contiguous())
    dfssm.layer_prefill(stack, h)
    loss, _ = dfssm.head_loss(W, sr, h, text[1:].contiguous(), norm_w=nw)
    logits = dfssm.linear_int8(W, sr, h, norm_w=nw)
    for t in (0, 7, 19):
        _, one = dfssm.head_greedy(W, sr, h[t].contiguous(), nw)
        assert torch.equal(one, logits[t])
    want = torch.logsumexp(logits.double(), 1) - logits.double().gather(1, text[1:].long()[:, None])[:, 0]
    assert bool(((loss.double() - want).abs() <= U * (8 * logits.abs().max().double() + 512) + 2.0 ** -22 + U * want).all())
