"""Layer norm over token rows (forward, backward) and the backward of the
norm over channels, against the fp64 oracle."""
import numpy as np
import pytest

from gpu_helpers import torch_cuda
from oracle import delta

pytestmark = pytest.mark.gpu

# A stored value is off by half a step of its type (eps / 2 relative), plus
# the float arithmetic: sums of up to 8192 terms in registers, warps and
# blocks are trees of at most ~32 serial additions of 2^-24 each, and the
# normalised value passes ~10 operations: 64 * 2^-24 = 4e-6 of the scale of the
# terms (|x - mu| rstd |gamma| and the like, taken as the largest output).
FLOAT = 64 * 2.0 ** -24


def _make(shape, dtype, seed=0, offset=0.3):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    D = shape[-1]
    return ((r(*shape) * 1.7 + offset).to(dtype), r(*shape).to(dtype), 1 + 0.2 * r(D), 0.1 * r(D))


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, ref, dtype, name, terms=None):
    torch = torch_cuda()
    step = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    scale = np.abs(ref).max() if terms is None else terms
    err = np.abs(_f64(got) - ref)
    assert (err <= 1.01 * step * np.abs(ref) + FLOAT * scale).all(), f"{name}: {err.max()} of {scale}"


SHAPES = [(1, 1), (3, 1), (5, 8), (7, 33), (64, 64), (2, 3, 250), (997, 250), (33, 1000), (300, 1024), (9, 2049),
          (5, 4096), (3, 4100), (4, 8192), (2, 8191), (4097, 40)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_rows(shape, dtype):
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    dt = getattr(torch, dtype)
    x, dz, gamma, beta = _make(shape, dt)
    z, mean, rstd = s4.layernorm(x, gamma, beta, 1e-5)
    dx, dg, db = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    zr, mr, rr, dxr, dgr, dbr = delta.layer_norm_backward(_f64(dz), _f64(x), _f64(gamma), 1e-5)
    assert z.dtype == dx.dtype == dt and mean.dtype == dg.dtype == torch.float32
    _close(mean, mr, torch.float32, "mean", np.abs(_f64(x)).max())
    assert (np.abs(_f64(rstd) / rr - 1) < FLOAT * (1 + np.abs(_f64(x)).max() * rr)).all()
    big = max(1.0, (rr * np.abs(_f64(x)).max()).max())   # x - mu loses |x| 2^-24 before it is scaled
    _close(z, zr + _f64(beta), dt, "z", big * np.abs(_f64(gamma)).max())
    h = np.abs(_f64(dz) * _f64(gamma)).max()
    _close(dx, dxr, dt, "dx", rr.max() * h * big)
    n = np.prod(shape[:-1])
    _close(dg, dgr, torch.float32, "dgamma", np.sqrt(n) * 4 * np.abs(_f64(dz)).max())
    _close(db, dbr, torch.float32, "dbeta", np.sqrt(n) * 4 * np.abs(_f64(dz)).max())


# rows that are multiples of 8 bytes and not of 16 take accesses of 8
@pytest.mark.parametrize("dtype,D", [(t, D) for t in ("bfloat16", "float16") for D in (4, 36, 132, 500, 1020, 2052, 8188)]
                         + [("float32", D) for D in (2, 66, 502, 1022, 2050, 8190)])
@pytest.mark.parametrize("rows", [1, 41, 700])
def test_rows_of_eight_bytes(rows, dtype, D):
    test_rows((rows, D), dtype)


def test_rows_unaligned_in_place_and_repeatable():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    x, dz, gamma, beta = _make((130, 256), torch.bfloat16)
    z, mean, rstd = s4.layernorm(x, gamma, beta)
    # rows that start two bytes past a 16-byte boundary take the element path
    buf = torch.empty(130 * 256 + 1, device="cuda", dtype=torch.bfloat16)
    xu = buf[1:].view(130, 256)
    xu.copy_(x)
    zu, mu, ru = s4.layernorm(xu, gamma, beta)
    # other order of the same sums: float rounding, which moves a 16-bit result by one step at most
    assert (zu.float() - z.float()).abs().max() <= 2 ** -7 * z.float().abs().max()
    assert (mu - mean).abs().max() <= FLOAT * x.float().abs().max()
    one = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    two = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    d2 = dz.clone()
    dx, dg, db = s4.layernorm_backward(d2, x, gamma, mean, rstd, dx=d2)
    assert dx.data_ptr() == d2.data_ptr() and torch.equal(dx, one[0]) and torch.equal(dg, one[1])
    x2 = x.clone()
    s4.layernorm(x2, gamma, beta, out=x2)
    assert torch.equal(x2, z)


def test_rows_none_and_constant_and_not_finite():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    x, dz, gamma, beta = _make((0, 64), torch.float32)
    z, mean, rstd = s4.layernorm(x, gamma, beta)
    dx, dg, db = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    assert z.shape == dx.shape == (0, 64) and not dg.any() and not db.any()
    x, dz, gamma, beta = _make((6, 64), torch.float32)
    x[2] = 3.0                    # no variance: xhat = 0, z = beta
    x[4, 5] = float("nan")
    z, mean, rstd = s4.layernorm(x, gamma, beta)
    assert torch.allclose(z[2], beta, atol=1e-6) and torch.isnan(z[4]).all()
    assert torch.isfinite(z[[0, 1, 2, 3, 5]]).all()      # a row's NaN stays in the row
    dx, dg, db = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    assert torch.isnan(dx[4]).all() and torch.isfinite(dx[[0, 1, 2, 3, 5]]).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("Bt,H,L", [(1, 1, 16), (2, 3, 32), (3, 64, 16), (2, 65, 128), (3, 100, 64), (2, 256, 512),
                                    (1, 257, 64), (2, 1000, 256), (1, 8192, 16), (8, 40, 8192)])
def test_channels(Bt, H, L):
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    x, dz, gamma, beta = _make((Bt, L, H), torch.float32, seed=2, offset=5.0)
    x, dz = x.transpose(1, 2).contiguous(), dz.transpose(1, 2).contiguous()
    dx, dg, db = s4.layernorm_channels_backward(dz, x, gamma, 1e-5)
    zr, mr, rr, dxr, dgr, dbr = delta.layer_norm_backward(_f64(dz).transpose(0, 2, 1), _f64(x).transpose(0, 2, 1),
                                                          _f64(gamma), 1e-5)
    big = max(1.0, (rr * np.abs(_f64(x)).max()).max())
    h = np.abs(_f64(dz)).max() * np.abs(_f64(gamma)).max()
    _close(dx, dxr.transpose(0, 2, 1), torch.float32, "dx", rr.max() * h * big)
    n = Bt * L
    _close(dg, dgr, torch.float32, "dgamma", np.sqrt(n) * 4 * np.abs(_f64(dz)).max() * big)
    _close(db, dbr, torch.float32, "dbeta", np.sqrt(n) * 4 * np.abs(_f64(dz)).max())
    again = s4.layernorm_channels_backward(dz, x, gamma, 1e-5)
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, db), again))


def test_channels_of_every_width_in_a_new_process():
    """From 5633 channels on the weight gradients and the kernel's static
    shared memory together pass the 48 KB that a launch has unasked; in a
    process of its own, where no wider call has raised the limit before."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]; import test_gpu_norm as t\n"
            "for H in (5632, 5633, 5640, 6144, 6145): t.test_channels(1, H, 16)" % (os.path.dirname(here), here))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_channels_backward_fits_its_forward():
    """The directional difference of s4.layernorm_channels itself."""
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    x, dz, gamma, beta = _make((2, 32, 64), torch.float32, seed=3)
    x, dz = x.transpose(1, 2).contiguous(), dz.transpose(1, 2).contiguous()
    d = torch.randn(x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    dx, _, _ = s4.layernorm_channels_backward(dz, x, gamma, 1e-5)
    f = lambda h: (s4.layernorm_channels(x + h * d, gamma, beta, 1e-5).double() * dz.double()).sum().item()  # noqa: E731
    h = 2.0 ** -6   # difference error ~h^2 times third derivatives (~2e-4), float error 1e-7 * 64 / h = 4e-4
    diff = (f(h) - f(-h)) / (2 * h)
    scale = (dx.double().abs() * d.double().abs()).sum().item()
    assert abs(diff - (dx.double() * d.double()).sum().item()) < 2e-3 * scale


def test_other_stream_and_graph():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    x, dz, gamma, beta = _make((300, 512), torch.bfloat16)
    z, mean, rstd = s4.layernorm(x, gamma, beta)
    want = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = s4.layernorm_backward(dz, x, gamma, mean, rstd)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = torch.empty(s4.layernorm_backward_workspace_size(512), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s4.layernorm_backward(dz, x, gamma, mean, rstd, dx=outs[0], dgamma=outs[1], dbeta=outs[2], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
