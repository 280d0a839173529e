"""The gated delta rule where every matrix product has one term: sequences of
one token, q and k with one channel, the gradients from behind with one value
channel. Errors then follow operation by operation, and a bound of a few steps
of float shows a left-out order of the parts' products (2^-16) at once."""
import numpy as np
import pytest

from gpu_helpers import torch_cuda
from oracle import delta
from test_gpu_gated_delta import NAMES, backward, forward, gen
from test_gpu_gated_delta_scan import f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


class V:
    """A value in 64 bits and a bound of the kernels' error in it."""

    def __init__(self, x, err=0.0):
        self.x = np.asarray(x, np.float64)
        self.err = np.zeros_like(self.x) + err

    def times(self, s):            # by a power of two or a sign: exact
        return V(self.x * s, self.err * abs(s))

    def at(self, i):
        return V(self.x[i], self.err[i])


def product(a, b):
    """On the tensor cores. Parts are |p1| <= 2^-8 |x|, |p2| <= 2^-16 |x| (half a
    step of bf16 each time) and exact together; the orders left out, p1 q2, p2 q1
    and p2 q2, are 2^-23 (1 + 2^-9) of the product. The accumulator truncates, by
    less than 2^-23 of what it holds: once of the whole product (the largest
    parts' comes last), five times of at most 3 2^-8 of it."""
    x = a.x * b.x
    return V(x, abs(a.x) * b.err + abs(b.x) * a.err + a.err * b.err + (2 + 0.08) * U * abs(x))


def by_one(a):
    """A product with T = 1: its only part is exact, the accumulator truncates three times."""
    return V(a.x, a.err + 1.02 * U * abs(a.x))


def together(a, b):
    """Two products in one accumulator: their largest parts come last, and
    truncate what is there, at most the sum of both."""
    return V(a.x + b.x, a.err + b.err + 2.1 * U * (abs(a.x) + abs(b.x)))


def rounded(x, err):               # a float operation: half a step
    return V(x, err + 0.5 * U * (abs(x) + err))


def mul(a, b):
    return rounded(a.x * b.x, abs(a.x) * b.err + abs(b.x) * a.err + a.err * b.err)


def add(a, b):
    return rounded(a.x + b.x, a.err + b.err)


def close(got, want, what):
    err = np.abs(f64(got) - want.x)
    # what float does to values below 2^-126 is no matter here
    assert (err <= want.err * (1 + 1e-6)).all(), f"{what}: {(err / np.maximum(want.err, 1e-300)).max()} of the bound"


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (72, 40), (8, 120)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_products_of_one_term(dtype, Dk, Dv):
    torch = torch_cuda()
    dt, B, H = getattr(torch, dtype), 48, 3
    r = lambda seed, *s: torch.randn(*s, device="cuda", generator=gen(seed))  # noqa: E731
    pick = lambda seed, n: torch.randint(n, (B, H), device="cuda", generator=gen(seed))  # noqa: E731
    kd, v0 = pick(1, Dk), pick(2, Dv)
    hot = lambda t, i, n: torch.zeros(*t.shape, n, device="cuda", dtype=t.dtype).scatter_(-1, i[..., None], t[..., None])  # noqa: E731
    q1, k1, do1 = (r(s, B, H).to(dt) for s in (3, 4, 5))
    d = {"q": hot(q1, kd, Dk)[:, None], "k": hot(k1, kd, Dk)[:, None], "v": r(6, B, 1, H, Dv).to(dt),
         "g": torch.zeros(B, 1, H, device="cuda"), "beta": torch.rand(B, 1, H, device="cuda", generator=gen(7)),
         "state": r(8, B, H, Dk, Dv)}
    do = hot(do1, v0, Dv)[:, None]
    ds = hot(r(9, B, H, Dk), v0[..., None].expand(B, H, Dk), Dv)
    scale = 0.5
    o, last, work = forward(d, scale=scale, initial_state=d["state"], keep=True)
    got = backward(d, do, work, scale=scale, dfinal_state=ds)

    b, h = np.meshgrid(np.arange(B), np.arange(H), indexing="ij")
    at, va = kd.cpu().numpy(), v0.cpu().numpy()
    S0, dS1 = f64(d["state"]), f64(ds)
    col = lambda x: V(x[..., None])                                # noqa: E731  a number for every head, against rows
    q, k, g_o, beta = (V(f64(x)) for x in (q1, k1, do1, d["beta"][:, 0]))
    row, v = V(S0[b, h, at]), V(f64(d["v"][:, 0]))                 # [B, H, Dv]: the state's row of the channel
    A = product(col(k.x), row)
    R = add(v, A.times(-1))
    E = by_one(R)
    written = add(row, product(col(k.x), mul(col(beta.x), E)))
    qk = product(q, k)
    PT = by_one(mul(qk.times(scale), beta))
    out = add(product(col(q.x), row).times(scale), product(V(PT.x[..., None], PT.err[..., None]), R))

    want, end, grads = delta.gated_delta(*(f64(d[n]) for n in NAMES), scale, S0, do=f64(do), dstate=dS1)
    np.testing.assert_allclose(out.x, want[:, 0], atol=1e-13)
    np.testing.assert_allclose(written.x, end[b, h, at], atol=1e-13)
    exact = S0.copy()
    exact[b, h, at] = f64(last)[b, h, at]
    assert (f64(last) == exact).all()                              # the other rows are as they were
    close(last[torch.arange(B)[:, None], torch.arange(H), kd], written, "state")
    if dtype == "float32":
        close(o[:, 0], out, "o")

    E0 = E.at((b, h, va))
    back = V(dS1[b, h, at, va])                                    # the state gradient's one value that k meets
    dR = together(by_one(mul(beta, product(k, back))), product(g_o, PT))
    first = add(back, together(product(g_o.times(scale), q), product(dR.times(-1), k)))
    np.testing.assert_allclose(first.x, grads["initial_state"][b, h, at, va], atol=1e-13)
    exact = dS1.copy()
    gi = f64(got["initial_state"])
    exact[b, h, at, va] = gi[b, h, at, va]
    assert (gi == exact).all()
    close(got["initial_state"][torch.arange(B)[:, None], torch.arange(H), kd, v0], first, "dstate")

    F = product(g_o, E0)
    c1 = mul(F.times(scale), qk)
    M = mul(F.times(scale), beta)
    column, behind = V(S0[b, h, :, va]), V(dS1[b, h, :, va])       # [B, H, Dk]
    e0, dr = V(E0.x[..., None], E0.err[..., None]), V(dR.x[..., None], dR.err[..., None])
    H_ = product(behind, e0)
    take = lambda x: x.at((b, h, at))                              # noqa: E731
    dbeta = add(c1, mul(k, take(H_)))
    np.testing.assert_allclose(dbeta.x, grads["beta"][:, 0], atol=1e-13)
    close(got["beta"][:, 0], dbeta, "dbeta")
    from_o, from_r = product(col(g_o.x), column).times(scale), product(dr, column).times(-1)
    both = (S0 * dS1).sum((-1, -2))                                # up to 64 in a row in a thread, 13 more between them
    dots = V(both, 80 * 0.5 * U * np.abs(S0 * dS1).sum((-1, -2)))
    dg = add(add(mul(q, take(from_o)), mul(k, take(from_r))), dots)
    np.testing.assert_allclose(dg.x, grads["g"][:, 0], atol=1e-13)
    # sums with zeros are exact; q.(S0 dO) and k.(S0 dR) meet in one more addition
    close(got["g"][:, 0], V(dg.x, dg.err + U * (abs(dg.x) + dg.err)), "dg")
    if dtype != "float32":
        return
    dq, dk = from_o, add(from_r, mul(col(beta.x), H_))
    for name, x, w in (("q", dq, product(M, k)), ("k", dk, product(M, q))):
        more = add(take(x), w)
        x.x[b, h, at], x.err[b, h, at] = more.x, more.err
        np.testing.assert_allclose(x.x, grads[name][:, 0], atol=1e-13)
        close(got[name][:, 0], x, "d" + name)
    dv = np.zeros((B, H, Dv))
    err = dv.copy()
    dv[b, h, va], err[b, h, va] = dR.x, dR.err
    close(got["v"][:, 0], V(dv, err), "dv")
