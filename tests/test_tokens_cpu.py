"""Host-side checks of the many-token operators on the int8 matrix (no GPU): sizes, pointers, alignment and types
are refused before anything is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from bit_quantized_mamba_b200 import build, dfssm
    build.build()
    return dfssm.lib()


BIG = 1 << 40


def test_workspace_sizes():
    from bit_quantized_mamba_b200 import dfssm as D
    for op in (D.OP_LINEAR_INT8, D.OP_EMBED_BACKWARD, D.OP_HEAD_LOSS, D.OP_HEAD_LOSS_BACKWARD):
        assert D.workspace_size(op, 0, 64, 10) == 256
        assert D.workspace_size(op, -1, 64, 10) == 0
        assert D.workspace_size(op, 4, 60, 10) == 0      # d % 16
        assert D.workspace_size(op, 4, 8208, 10) == 0    # d > 8192
        assert D.workspace_size(op, 4, 64, 0) == 0       # no rows
        assert D.workspace_size(op, 4, 64, (1 << 30) + 1) == 0
        a, b = D.workspace_size(op, 100, 2048, 50288), D.workspace_size(op, 3000, 2048, 50288)
        assert 256 < a < b
    assert D.workspace_size(D.OP_EMBED_TOKENS, 0, 0, 0) == 256
    # the logits of a long batch (2048 x 50288 fp32) are never kept
    assert D.workspace_size(D.OP_HEAD_LOSS, 2048, 2048, 50288) < 16 << 20
    assert D.workspace_size(D.OP_HEAD_LOSS_BACKWARD, 2048, 2048, 50288) < 2048 * 50288 * 4 // 2
    # vocabularies past the range of one set of int32 accumulators get more of them
    one, many = D.workspace_size(D.OP_HEAD_LOSS_BACKWARD, 64, 64, 100000), D.workspace_size(D.OP_HEAD_LOSS_BACKWARD, 64, 64, 10 ** 6)
    assert many - one >= 6 * 3 * 64 * 64 * 4


def matrix_refusals(call):
    """call(W, V, d) with everything else valid."""
    assert call(None, 10, 32) == -1
    assert call(16, 0, 32) == -1
    assert call(16, 10, 24) == -1
    assert call(16, 10, 0) == -1
    assert call(16, 10, 8208) == -3
    assert call(16, (1 << 30) + 1, 32) == -3
    assert call(8, 10, 32) == -2


def test_linear_int8_refusals(L):
    def f(W=16, s=16, V=10, d=32, x=16, xt=0, ldx=32, M=4, nw=None, y=16, yt=0, ldy=10, ws=256, n=BIG):
        return L.dfssm_linear_int8(W, s, V, d, x, xt, ldx, M, nw, y, yt, ldy, ws, n, None, None)
    matrix_refusals(lambda W, V, d: f(W=W, V=V, d=d, ldx=max(d, 32), ldy=max(V, 10)))
    assert f(s=None) == -1
    assert f(x=None) == -1
    assert f(y=None) == -1
    assert f(M=-1) == -1
    assert f(xt=2) == -1
    assert f(yt=-1) == -1
    assert f(ldx=31) == -1
    assert f(ldy=9) == -1
    assert f(ldy=1 << 31) == -3
    assert f(x=24) == -2
    assert f(ldx=34) == -2            # fp32 rows not 16-byte aligned
    assert f(xt=1, ldx=36) == -2      # bf16 rows
    assert f(nw=8) == -2
    assert f(y=18) == -2
    assert f(yt=1, y=17) == -2
    assert f(ws=None) == -7
    assert f(ws=128) == -7
    assert f(n=256) == -7
    assert f(M=0, x=None, y=None, ws=None) == 0


def test_embed_tokens_refusals(L):
    def f(W=16, s=16, V=10, d=32, tok=16, n=4, h=16, ht=0, ldh=32, ws=256, nb=256):
        return L.dfssm_embed_tokens(W, s, V, d, tok, n, h, ht, ldh, ws, nb, None)
    matrix_refusals(lambda W, V, d: f(W=W, V=V, d=d, ldh=max(d, 32)))
    for kw, want in ((dict(s=None), -1), (dict(tok=None), -1), (dict(n=-1), -1), (dict(h=None), -1), (dict(ht=5), -1),
                     (dict(ldh=16), -1), (dict(h=8), -2), (dict(ldh=33), -2), (dict(tok=2), -2), (dict(ws=None), -7),
                     (dict(ws=64), -7), (dict(nb=128), -7), (dict(n=0, tok=None, h=None, ws=None), 0)):
        assert f(**kw) == want, kw


def test_embed_backward_refusals(L):
    def f(W=16, V=10, d=32, tok=16, n=4, dh=16, t=0, ld=32, dE=16, ds=16, acc=0, ws=256, nb=BIG):
        return L.dfssm_embed_tokens_backward(W, V, d, tok, n, dh, t, ld, dE, ds, acc, ws, nb, None)
    matrix_refusals(lambda W, V, d: f(W=W, V=V, d=d, ld=max(d, 32)))
    for kw, want in ((dict(tok=None), -1), (dict(n=-1), -1), (dict(dh=None), -1), (dict(t=3), -1), (dict(ld=31), -1),
                     (dict(dE=None, ds=None), -1), (dict(dE=8), -2), (dict(ds=2), -2), (dict(dh=4), -2),
                     (dict(ld=33), -2), (dict(tok=1), -2), (dict(ws=None), -7), (dict(ws=8), -7), (dict(nb=300), -7),
                     (dict(n=0, acc=1, tok=None, dh=None, ws=None), 0)):
        assert f(**kw) == want, kw


def test_head_loss_refusals(L):
    def f(W=16, s=16, V=10, d=32, x=16, t=0, ldx=32, M=4, nw=None, y=16, loss=16, st=16, ws=256, nb=BIG):
        return L.dfssm_head_loss(W, s, V, d, x, t, ldx, M, nw, y, loss, st, ws, nb, None)
    matrix_refusals(lambda W, V, d: f(W=W, V=V, d=d, ldx=max(d, 32)))
    for kw, want in ((dict(s=None), -1), (dict(x=None), -1), (dict(M=-1), -1), (dict(y=None), -1), (dict(loss=None), -1),
                     (dict(st=None), -1), (dict(t=2), -1), (dict(ldx=0), -1), (dict(x=4), -2), (dict(nw=4), -2),
                     (dict(y=2), -2), (dict(loss=1), -2), (dict(ws=None), -7), (dict(nb=1000), -7),
                     (dict(M=0, x=None, y=None, loss=None, st=None, ws=None), 0)):
        assert f(**kw) == want, kw


def test_head_loss_backward_refusals(L):
    def f(W=16, s=16, V=10, d=32, x=16, t=0, ldx=32, M=4, nw=16, y=16, st=16, g=16, dx=16, lddx=32, ds=16, dn=16,
          ws=256, nb=BIG):
        return L.dfssm_head_loss_backward(W, s, V, d, x, t, ldx, M, nw, y, st, g, dx, lddx, ds, dn, ws, nb, None)
    matrix_refusals(lambda W, V, d: f(W=W, V=V, d=d, ldx=max(d, 32), lddx=max(d, 32)))
    assert f(V=(1 << 24) + 1) == -3
    for kw, want in ((dict(s=None), -1), (dict(x=None), -1), (dict(M=-1), -1), (dict(y=None), -1), (dict(st=None), -1),
                     (dict(g=None), -1), (dict(dx=None), -1), (dict(nw=None), -1), (dict(t=9), -1), (dict(lddx=16), -1),
                     (dict(lddx=33), -2), (dict(dx=8), -2), (dict(ds=1), -2), (dict(dn=2), -2), (dict(g=3), -2),
                     (dict(ws=None), -7), (dict(nb=1000), -7),
                     (dict(M=0, x=None, y=None, st=None, g=None, dx=None, ds=None, dn=None, ws=None), 0)):
        assert f(**kw) == want, kw


def test_too_many_tokens(L):
    """More than 2^30 tokens are refused before anything is looked at, and have no workspace."""
    M = (1 << 30) + 1
    assert L.dfssm_linear_int8(16, 16, 10, 32, 16, 0, 32, M, None, 16, 0, 10, 256, BIG, None, None) == -3
    assert L.dfssm_embed_tokens(16, 16, 10, 32, 16, M, 16, 0, 32, 256, BIG, None) == -3
    assert L.dfssm_embed_tokens_backward(16, 10, 32, 16, M, 16, 0, 32, 16, 16, 0, 256, BIG, None) == -3
    assert L.dfssm_head_loss(16, 16, 10, 32, 16, 0, 32, M, None, 16, 16, 16, 256, BIG, None) == -3
    assert L.dfssm_head_loss_backward(16, 16, 10, 32, 16, 0, 32, M, None, 16, 16, 16, 16, 32, 16, None, 256, BIG,
                                      None) == -3
    for op in (10, 12, 13, 14):
        assert L.dfssm_workspace_size(op, M, 32, 10) == 0 and L.dfssm_workspace_size(op, M - 1, 32, 10) > 0


def test_binding_checks_shapes_and_types():
    from bit_quantized_mamba_b200 import dfssm as D
    with pytest.raises(ValueError):
        D._matrix(torch.zeros(4, 32))
    with pytest.raises(ValueError):
        D._matrix(torch.zeros(4, 64, dtype=torch.int8)[:, ::2])
    x = torch.zeros(4, 32)
    assert D._rows(x, 4, 32, "x")[1:] == (0, 32)
    assert D._rows(torch.zeros(4, 40, dtype=torch.bfloat16)[:, :32], 4, 32, "x")[1:] == (1, 40)
    assert D._rows(torch.zeros(1, 32).expand(1, 32), 1, 32, "x")[2] == 32
    for bad in (x.double(), x.t(), x[:2], torch.zeros(4, 64)[:, ::2]):
        with pytest.raises(ValueError):
            D._rows(bad, 4, 32, "x")
    assert D._vector(None, 3, torch.float32, "v") is None
    for bad in (torch.zeros(4), torch.zeros(3, dtype=torch.int32), torch.zeros(6)[::2]):
        with pytest.raises(ValueError):
            D._vector(bad, 3, torch.float32, "v")


def test_binding_refuses_another_device(monkeypatch):
    """Tensors have to live on the current device: the library launches there."""
    from bit_quantized_mamba_b200 import dfssm as D
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)

    class Fake:
        def __init__(self, i):
            self.device, self.is_cuda = torch.device("cuda", i), True

        def get_device(self):
            return self.device.index


    assert D._on(7, Fake(1), None) == 7
    with pytest.raises(ValueError):
        D._on(7, Fake(1), Fake(0))
    with pytest.raises(ValueError):
        D._on(7, torch.zeros(3))
