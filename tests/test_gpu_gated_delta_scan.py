"""The gated delta rule token by token (decode) against the fp64 oracle."""
import numpy as np
import pytest

from gpu_helpers import torch_cuda
from oracle import delta

pytestmark = pytest.mark.gpu


def make(Bt, T, Hk, Hv, Dk, Dv, dtype="float32", seed=0):
    torch = torch_cuda()
    dt = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    return {"q": unit(r(Bt, T, Hk, Dk)).to(dt), "k": unit(r(Bt, T, Hk, Dk)).to(dt), "v": r(Bt, T, Hv, Dv).to(dt),
            "g": -torch.rand(Bt, T, Hv, device="cuda", generator=gen), "beta": torch.sigmoid(r(Bt, T, Hv)),
            "state": 0.5 * r(Bt, Hv, Dk, Dv)}


def f64(t):
    return t.double().cpu().numpy()


def oracle(d, scale, **more):
    names = ("q", "k", "v", "g", "beta")
    return delta.gated_delta(*(f64(d[n]) for n in names), scale, f64(d["state"]), **more)


# Per token a sum over Dk <= 128 products (16 serial additions a thread, then
# trees), a handful of roundings on u and the state, damped from token to token
# (unit keys, beta < 1): 64 * 2^-24 relative to the values' norm, times the
# tokens for the undamped worst case of the few tokens here. The stored o is
# off by half a step of its type besides.
def check(got, ref, T, dtype, what):
    torch = torch_cuda()
    step = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    err = np.abs(f64(got) - ref)
    bound = 1.01 * step * np.abs(ref) + 64 * 2.0 ** -24 * max(T, 1) * max(1.0, np.abs(ref).max())
    assert (err <= bound).all(), f"{what}: {err.max()}"


SHAPES = [(1, 1, 1, 1, 8, 8), (1, 1, 4, 4, 64, 64), (2, 1, 2, 6, 96, 80), (3, 5, 1, 3, 128, 128), (1, 7, 8, 16, 128, 40),
          (40, 2, 2, 8, 72, 128), (80, 1, 2, 4, 128, 128), (5, 33, 1, 2, 16, 120), (2, 1, 100, 100, 24, 56)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_scan(shape, dtype):
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    Bt, T, Hk, Hv, Dk, Dv = shape
    d = make(*shape, dtype=dtype)
    ref, last = oracle(d, Dk ** -0.5)
    state = d["state"].clone()
    o = s4.gated_delta_scan(d["q"], d["k"], d["v"], d["g"], d["beta"], state)
    assert o.dtype == d["v"].dtype and o.shape == d["v"].shape
    check(o, ref, T, d["v"].dtype, "o")
    check(state, last, T, torch.float32, "state")
    if T == 1:
        s2 = d["state"].clone()
        o1 = s4.gated_delta_step(*(d[n].squeeze(1) for n in ("q", "k", "v", "g", "beta")), s2)
        assert torch.equal(o1, o[:, 0]) and torch.equal(s2, state)


def test_steps_are_the_scan():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(2, 9, 2, 4, 64, 96, "bfloat16")
    a, b = d["state"].clone(), d["state"].clone()
    whole = s4.gated_delta_scan(d["q"], d["k"], d["v"], d["g"], d["beta"], a, scale=0.3)
    for t in range(9):
        one = s4.gated_delta_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), b, scale=0.3)
        assert torch.equal(one, whole[:, t])
    assert torch.equal(a, b)


def test_slices_of_one_projection():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    Bt, T, Hk, Hv, Dk, Dv = 3, 4, 2, 4, 64, 32
    d = make(Bt, T, Hk, Hv, Dk, Dv, "bfloat16")
    wide = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], -1)
    q, k, v = wide.split([Hk * Dk, Hk * Dk, Hv * Dv], -1)
    q, k, v = q.unflatten(-1, (Hk, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (Hv, Dv))
    a, b = d["state"].clone(), d["state"].clone()
    assert torch.equal(s4.gated_delta_scan(q, k, v, d["g"], d["beta"], a),
                       s4.gated_delta_scan(d["q"], d["k"], d["v"], d["g"], d["beta"], b))
    assert torch.equal(a, b)


def test_no_tokens_reset_and_strength_zero():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(2, 3, 1, 2, 32, 32)
    state = d["state"].clone()
    none = {n: d[n][:, :0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    o = s4.gated_delta_scan(*(none[n] for n in ("q", "k", "v", "g", "beta")), state)
    assert o.shape == (2, 0, 2, 32) and torch.equal(state, d["state"])
    d["g"][:, 1] = -float("inf")      # the state is cleared before the second token
    ref, last = oracle(d, 1.0)
    o = s4.gated_delta_scan(d["q"], d["k"], d["v"], d["g"], d["beta"], state, scale=1.0)
    check(o, ref, 3, torch.float32, "o")
    d["beta"].zero_()
    d["g"].zero_()
    state = d["state"].clone()
    s4.gated_delta_scan(d["q"], d["k"], d["v"], d["g"], d["beta"], state)
    assert torch.equal(state, d["state"])
