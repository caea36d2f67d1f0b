"""Gradients of the norms around a block for rows far from magnitude one, and for rows of zeros under a
small eps, against the definition in 64 bits, with the bounds of test_gpu_block_norm.py (relative to
the sum of a result's terms, so they hold at any magnitude whose squares fp32 can add up)."""
import pytest
import test_gpu_block_norm as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _powers(T, low, high):
    """A row's factor: powers of ten from low to high."""
    import torch
    return (10.0 ** torch.linspace(low, high, T, dtype=torch.float64)).float().cuda()[:, None]


def _scaled(s, name, by):
    s[name] = (s[name].float() * by).to(s[name].dtype)


@pytest.mark.parametrize("dtype,residual", B.TYPES)
@pytest.mark.parametrize("D", [64, 1000, 4096, 8192])
def test_large_rows(kda, monkeypatch, dtype, residual, D):
    """Block outputs and residuals up to 1e16."""
    monkeypatch.setattr(B, "EPS", 1e-6)
    s = B._inputs(21, 33, D, dtype, residual)
    _scaled(s, "y", _powers(33, -3, 16))
    _scaled(s, "r", _powers(33, 0, 16).flip(0))
    B._check(kda, s)


@pytest.mark.parametrize("dtype,residual", B.TYPES)
@pytest.mark.parametrize("D", [72, 4104])
def test_small_and_large_rows_without_eps(kda, monkeypatch, dtype, residual, D):
    """Without a post-norm the residual has the rows' magnitude, here 1e-16 to 1e16."""
    monkeypatch.setattr(B, "EPS", 0.0)
    s = B._inputs(22, 33, D, dtype, residual, post=False)
    by = _powers(33, -16, 16)
    _scaled(s, "y", by)
    _scaled(s, "r", by)
    B._check(kda, s)


@pytest.mark.parametrize("dtype,residual", B.TYPES)
def test_small_residual_without_eps(kda, monkeypatch, dtype, residual):
    """Both norms over small rows: a residual of 1e-13, and what a scale of 1e-13 adds to it."""
    monkeypatch.setattr(B, "EPS", 0.0)
    s = B._inputs(23, 33, 520, dtype, residual)
    _scaled(s, "y", _powers(33, -13, 3))
    _scaled(s, "r", 1e-13)
    _scaled(s, "scale", 1e-13)
    B._check(kda, s)


@pytest.mark.parametrize("dtype,residual", B.TYPES)
@pytest.mark.parametrize("eps", [1e-12, 1e-30])
def test_zero_rows_with_a_small_eps(kda, monkeypatch, dtype, residual, eps):
    """Rows of zeros have gradients of size 1 / sqrt(eps)."""
    import torch
    monkeypatch.setattr(B, "EPS", eps)
    s = B._inputs(24, 12, 264, dtype, residual)
    s["y"][1], s["y"][3], s["r"][3] = 0.0, 0.0, 0.0
    s["y"][4] = (s["y"][4].float() * 1e-15).to(s["y"].dtype)
    B._check(kda, s)
    r, _ = kda.block_norm(s["y"], s["r"], **B._kw(s))
    assert not bool(r[3].any())
    for n, t in kda.block_norm_bwd(s["y"], r, s["dx"], s["dr"], **B._kw(s)).items():
        assert bool(torch.isfinite(t).all()), n
