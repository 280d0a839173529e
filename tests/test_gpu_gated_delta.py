"""The chunked gated delta rule (forward, backward) against the fp64 oracle."""
import numpy as np
import pytest

from gpu_helpers import torch_cuda
from oracle import delta
from test_gpu_gated_delta_scan import f64, make

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")

# Every product is a float sum of 24-bit operands: its error is a few 2^-24 of
# the sum of its terms' sizes. A chunk passes five products one after the
# other (T's two, K S, T R, K^T E) of up to 128 terms of 3 parts each, the
# tensor cores add groups of 16 terms with a truncated carry (one step of the
# largest, 2^-23, a group: 24 groups), and T is solved in float over 64 rows.
# Errors of the state are damped like the state. Relative 2-norm over a
# tensor: 5 products * 24 groups * 2^-23 = 1.5e-5 if every group erred fully
# and the same way; the signs differ, so that a root of the count remains:
# 5 * sqrt(24) * 2^-23 = 3e-6, and half as much again for T.
REL = 4.5e-6


def check(got, ref, dtype, what, passes=1, rounded=1):
    torch = torch_cuda()
    step = rounded * torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    real = ~np.isnan(ref)
    g, r = f64(got)[real], ref[real]
    assert np.isfinite(g).all(), f"{what}: not finite"
    if not r.size:
        return
    norm = np.linalg.norm(r)
    err = np.linalg.norm(g - r)
    # the norm of the roundings to 16 bits is at most a half step of each value
    assert err <= (passes * REL + step) * norm + 1e-30, f"{what}: {err} of {norm}"
    if norm == 0.0:      # then the values are zeros, as the line above says
        return
    rms = norm / np.sqrt(r.size)
    big = (np.abs(g - r) / np.maximum(np.abs(r), rms)).max()
    assert big <= 1.01 * step + 16 * passes * REL, f"{what}: one value {big}"


def forward(d, **more):
    import structured_state_space_dplr_b200 as s4
    torch = torch_cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = s4.gated_delta_forward(*(d[n] for n in NAMES), flags=flags, **more)
    assert flags.item() == 0
    return r


SHAPES = [(1, 64, 1, 1, 64, 64), (1, 1, 1, 1, 8, 8), (2, 65, 1, 2, 64, 64), (1, 130, 2, 2, 128, 128),
          (2, 63, 2, 6, 96, 80), (3, 200, 1, 3, 72, 128), (1, 321, 2, 4, 128, 40), (5, 7, 4, 4, 16, 120),
          (2, 128, 3, 3, 40, 8)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_forward(shape, dtype):
    torch = torch_cuda()
    d = make(*shape, dtype=dtype)
    Dk = shape[4]
    args = [f64(d[n]) for n in NAMES]
    ref, last = delta.gated_delta(*args, Dk ** -0.5)
    o, got, _ = forward(d)
    check(o, ref, d["v"].dtype, "o")
    check(got, last, torch.float32, "state")
    ref, last = delta.gated_delta(*args, 0.7, f64(d["state"]))
    for keep in (False, True):
        o, got, _ = forward(d, scale=0.7, initial_state=d["state"], keep=keep)
        check(o, ref, d["v"].dtype, "o from a state")
        check(got, last, torch.float32, "state from a state")


def backward(d, do, work, **more):
    import structured_state_space_dplr_b200 as s4
    torch = torch_cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = s4.gated_delta_backward(*(d[n] for n in NAMES), do, work, flags=flags, **more)
    assert flags.item() == 0
    return r


def gen(seed):
    torch = torch_cuda()
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_backward(shape, dtype):
    torch = torch_cuda()
    d = make(*shape, dtype=dtype)
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(d["v"].dtype)
    ds = torch.randn(d["state"].shape, device="cuda", generator=gen(2))
    args = [f64(d[n]) for n in NAMES]
    _, _, ref = delta.gated_delta(*args, 0.7, f64(d["state"]), do=f64(do), dstate=f64(ds))
    _, _, work = forward(d, scale=0.7, initial_state=d["state"], keep=True)
    got = backward(d, do, work, scale=0.7, dfinal_state=ds)
    # a gradient passes the forward chain, the backward chain and three more products: twice the forward's error
    for m in (*NAMES, "initial_state"):
        check(got[m], ref[m], got[m].dtype, "d" + m, 2)
    again = backward(d, do, work, scale=0.7, dfinal_state=ds)
    assert all(torch.equal(got[m], again[m]) for m in got)     # the workspace is not used up, the bits are the same
    _, _, ref = delta.gated_delta(*args, shape[4] ** -0.5, do=f64(do))
    _, _, work = forward(d, keep=True)
    got = backward(d, do, work)
    for m in NAMES:
        check(got[m], ref[m], got[m].dtype, "d" + m + " from zero", 2)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_many_blocks_at_once(dtype):
    """Thousands of chunks, several blocks an SM: against the recurrent form
    (whose own error is the float of its ~2000 damped steps), and the same bits
    from run to run."""
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(3, 2000, 8, 16, 128, 128, dtype, seed=5)
    state = d["state"].clone()
    want = s4.gated_delta_scan(*(d[n] for n in NAMES), state)
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(3)).to(d["v"].dtype)
    first = None
    for _ in range(4):
        o, last, work = forward(d, initial_state=d["state"], keep=True)
        # both are rounded to the stored type
        check(o, f64(want), d["v"].dtype, "o", 2, 2)
        check(last, f64(state), torch.float32, "state", 2)
        got = (o, last, *backward(d, do, work).values())
        assert all(torch.isfinite(t).all() for t in got)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
