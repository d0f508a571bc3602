"""The 8-bit calls refuse buffers that their kernels would read or write past the end of, or in host memory: outputs,
scales, workspaces, and layers on another device.  Nothing is launched in any of these calls."""
import numpy as np
import pytest

from bit_diffusion_model_amd import svdq

pytestmark = pytest.mark.gpu
M, K, N, LD = 40, 200, 48, 256


def _torch():
    import torch

    return torch


def make():
    torch = _torch()
    lin = svdq.Int8Linear(np.zeros((N, LD), np.int8), np.ones(N, np.float32), K, inv_s=np.ones(K, np.float32))
    return lin, svdq.GroupNorm(8, K, np.ones(K, np.float32)), torch.ones((M, K), device="cuda:0")


def code_buffers():
    """Pairs that are no place for the codes and scales of M rows of K values, each by one property."""
    torch = _torch()
    q = lambda *s, dtype=torch.int8, device="cuda:0": torch.empty(s, dtype=dtype, device=device)  # noqa: E731
    s = lambda n=M, dtype=torch.float32, device="cuda:0": torch.empty(n, dtype=dtype, device=device)  # noqa: E731
    return {"rows too few": (q(M - 1, LD), s()), "rows as long as X's": (q(M, K), s()), "scales too few": (q(M, LD), s(M - 1)),
            "codes' type": (q(M, LD, dtype=torch.uint8), s()), "scales' type": (q(M, LD), s(dtype=torch.float64)),
            "strided codes": (q(M, 2 * LD)[:, :LD], s()), "strided scales": (q(M, LD), s(2 * M)[::2]),
            "flat codes": (q(M * LD), s()), "codes on the host": (q(M, LD, device="cpu"), s()),
            "scales on the host": (q(M, LD), s(device="cpu"))}


@pytest.mark.parametrize("what", ["rows too few", "rows as long as X's", "scales too few", "codes' type", "scales' type",
                                  "strided codes", "strided scales", "flat codes", "codes on the host", "scales on the host"])
def test_code_outputs(what):
    lin, gn, X = make()
    bad = code_buffers()[what]
    for call in (lambda: svdq.quantize_act_int8(X, out=bad), lambda: lin.quantize(X, out=bad),
                 lambda: gn.quantize(X[None], out=bad), lambda: gn.quantize(X[None], lin.inv_s, out=bad)):
        with pytest.raises(svdq.SvdqError, match="out"):
            call()
    ok = code_buffers()["rows too few"]
    q, s = svdq.quantize_act_int8(X[:M - 1], out=(ok[0], ok[1][:M - 1]))  # the buffers of the right size
    assert q is ok[0] and (q[:, :K] == 127).all()


def test_scales_outputs_and_workspaces_off_the_device():
    torch = _torch()
    lin, gn, X = make()
    q, s = lin.quantize(X)
    with pytest.raises(svdq.SvdqError, match="sX"):
        lin.gemm(q, s.cpu())
    for bad in (q.cpu(), q[0], q.view(-1)):
        with pytest.raises(svdq.SvdqError):
            lin.gemm(bad, s)
    host = torch.empty((M, N))
    for call in (lambda: lin.gemm(q, s, out=host), lambda: lin.forward(X, out=host),
                 lambda: gn.forward_linear(X[None], lin, svdq.F32, out=host),
                 lambda: gn.forward(X[None], svdq.F32, out=torch.empty((1, M, K)))):
        with pytest.raises(svdq.SvdqError, match="out"):
            call()
    n = 1 << 24
    strided = torch.empty(2 * n, dtype=torch.uint8, device="cuda:0")[::2]
    Xl = torch.ones((1, 20000, K), device="cuda:0")  # large enough that the norm has a workspace
    for ws in (torch.empty(n, dtype=torch.uint8), strided):
        for call in (lambda: lin.gemm(q, s, workspace=ws), lambda: lin.forward(X, workspace=ws),
                     lambda: gn.forward(Xl, workspace=ws), lambda: gn.quantize(Xl, workspace=ws),
                     lambda: gn.forward_linear(Xl, lin, workspace=ws)):
            with pytest.raises(svdq.SvdqError, match="workspace"):
                call()
    for inv in (lin.inv_s.cpu(), lin.inv_s[:-1]):
        for call in (lambda: svdq.quantize_act_int8(X, inv), lambda: gn.quantize(X[None], inv)):
            with pytest.raises(svdq.SvdqError, match="inv_s"):
                call()
    # a workspace of another type counts by its bytes
    need = lin.workspace(M, svdq.F32).numel()
    assert torch.equal(lin.forward(X, workspace=torch.empty((need + 3) // 4, device="cuda:0")), lin.forward(X))


def test_layer_and_norm_on_another_device(monkeypatch):
    """A layer or norm whose tensors are on another device than the input (played by the number that it keeps)."""
    lin, gn, X = make()
    q, s = lin.quantize(X)
    monkeypatch.setattr(lin, "_dev", 1)
    for call in (lambda: lin.forward(X), lambda: lin.gemm(q, s), lambda: gn.forward_linear(X[None], lin)):
        with pytest.raises(svdq.SvdqError, match="cuda:1"):
            call()
    monkeypatch.setattr(lin, "_dev", 0)
    monkeypatch.setattr(gn, "_dev", 1)
    for call in (lambda: gn.forward(X[None]), lambda: gn.quantize(X[None]), lambda: gn.forward_linear(X[None], lin)):
        with pytest.raises(svdq.SvdqError, match="cuda:1"):
            call()


def test_one_channel_out_of_any_stride():
    """With one channel the column stride of `out` addresses nothing, as with one value a row in X."""
    torch = _torch()
    lin = svdq.Int8Linear(np.ones((1, 128), np.int8), np.ones(1, np.float32), 5)
    for m in (1, 3, 90):
        X = torch.arange(5.0 * m, device="cuda:0").view(m, 5)
        out = torch.as_strided(torch.full((3 * m + 7,), 8.0, device="cuda:0"), (m, 1), (3, 7))
        assert torch.equal(lin.forward(X, out=out), lin.forward(X))
        assert torch.equal(lin.gemm(*lin.quantize(X), out=out), lin.forward(X))
