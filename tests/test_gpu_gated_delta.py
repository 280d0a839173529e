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


def packed(d, cu):
    """The oracle's arguments for sequences packed in d, with a state for each."""
    torch = torch_cuda()
    n, (Hv, Dk, Dv) = len(cu) - 1, d["state"].shape[1:]
    d["state"] = 0.5 * torch.randn(n, Hv, Dk, Dv, device="cuda", generator=gen(7))
    d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    return [f64(d[n]) for n in NAMES]


# offsets with sequences of no and of one token, ends inside and at the end of
# a chunk, tokens before the first and behind the last sequence; few heads, so
# that the longest one runs in segments
CUS = [[0, 300], [0, 0, 1, 64, 129, 300], [5, 5, 6, 70, 198, 199], [0, 1200], [3, 3, 900, 1111, 1111], [0, 0, 0]]


@pytest.mark.parametrize("cu", CUS)
@pytest.mark.parametrize("dtype,shape", [("bfloat16", (2, 4, 64, 48)), ("float32", (1, 3, 72, 128))])
def test_packed(cu, dtype, shape):
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    T = max(cu[-1] + 9, 20)
    d = make(1, T, *shape, dtype=dtype)
    args = packed(d, cu)
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    inside[cu[0]:cu[-1]] = True
    for n in NAMES:        # what lies outside the sequences is not looked at
        d[n][:, ~inside] = float("nan")
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(d["v"].dtype)
    do[:, ~inside] = float("inf")
    ds = torch.randn(d["state"].shape, device="cuda", generator=gen(2))
    ref, last, gr = delta.gated_delta(*args, 0.5, f64(d["state"]), cu=cu, do=f64(do), dstate=f64(ds))
    o = torch.full_like(d["v"], 7.0)
    final = d["state"].clone()
    _, final, work = forward(d, scale=0.5, initial_state=final, final_state=final, cu_seqlens=d["cu"], keep=True, out=o)
    check(o, ref, o.dtype, "o")
    check(final, last, torch.float32, "state")
    assert (o[:, ~inside] == 7.0).all()
    got = backward(d, do, work, scale=0.5, dfinal_state=ds, cu_seqlens=d["cu"])
    for m in (*NAMES, "initial_state"):
        check(got[m], gr[m], got[m].dtype, "d" + m, 2)
        if m != "initial_state":
            assert not got[m][:, ~inside].any()
    for i in range(len(cu) - 1):     # an empty sequence hands its state (and the state's gradient) through
        if cu[i] == cu[i + 1]:
            assert torch.equal(final[i], d["state"][i]) and torch.equal(got["initial_state"][i], ds[i])


# most tokens in one of several sequences, which then run in segments of their own number
@pytest.mark.parametrize("cu", [[0, 2500, 2500, 2501, 2740], [0, 200, 500, 2730, 2731], [7, 900, 1700, 2600, 2731]])
@pytest.mark.parametrize("dtype,shape", [("float16", (1, 3, 96, 80)), ("float32", (2, 2, 64, 128))])
def test_packed_of_unequal_lengths(cu, dtype, shape):
    test_packed(cu, dtype, shape)


@pytest.mark.parametrize("shape", [(1, 1500, 1, 2, 64, 64), (1, 3000, 2, 2, 128, 96), (2, 2000, 1, 1, 40, 128)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_few_long_sequences_run_in_segments(shape, dtype):
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(*shape, dtype=dtype)
    d["g"] *= 0.02                  # slow decay: states reach over many segments
    ref, last = delta.gated_delta(*(f64(d[n]) for n in NAMES), shape[4] ** -0.5, f64(d["state"]))
    state = d["state"].clone()
    o, got, _ = forward(d, initial_state=state, final_state=state)
    check(o, ref, d["v"].dtype, "o", 2)       # the segments' states pass one more chain and the joins
    check(got, last, torch.float32, "state", 2)
    assert torch.equal(got, state)


def test_decode_continues_prefill():
    """norm -> projections -> prefill in chunks -> decode steps, against one pass over all tokens."""
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    T, more, D, Hk, Hv, Dk, Dv = 150, 5, 96, 2, 4, 64, 32
    x = torch.randn(2, T + more, D, device="cuda", generator=gen(0)) * 2 + 1
    gamma, beta = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    z, _, _ = s4.layernorm(x, gamma, beta)
    w = torch.randn(D, (2 * Hk * Dk + Hv * Dv), device="cuda", generator=gen(1)) / D ** 0.5
    mixed = (z @ w).to(torch.bfloat16)
    q, k, v = mixed.split([Hk * Dk, Hk * Dk, Hv * Dv], -1)
    q, k, v = q.unflatten(-1, (Hk, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (Hv, Dv))
    k = torch.nn.functional.normalize(k.float(), dim=-1).to(torch.bfloat16)
    g = -torch.rand(2, T + more, Hv, device="cuda", generator=gen(2))
    b = torch.rand(2, T + more, Hv, device="cuda", generator=gen(3))
    whole, last, _ = s4.gated_delta_forward(q, k, v, g, b)
    cut = lambda s: [t[:, s] for t in (q, k, v)] + [t[:, s].contiguous() for t in (g, b)]  # noqa: E731
    pre = cut(slice(0, T))
    with pytest.raises(ValueError):           # a cut in time of a batch is not evenly spaced
        s4.gated_delta_forward(*pre)
    o, state, _ = s4.gated_delta_forward(*(t.contiguous() for t in pre))
    outs = [o]
    for t in range(T, T + more):
        one = [x[:, t] for x in (q, k, v)] + [x[:, t].contiguous() for x in (g, b)]
        outs.append(s4.gated_delta_step(*one, state).unsqueeze(1))
    check(torch.cat(outs, 1), f64(whole), torch.bfloat16, "o", 2, 2)
    check(state, f64(last), torch.float32, "state", 2)


def test_resets_and_values_that_are_not_finite():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(1, 200, 1, 2, 64, 64)
    d["g"][0, 70] = -float("inf")
    d["g"][0, 130, 0] = -1e30
    d["g"][0, 20, 1] = -300.0                 # no later difference of sums may lose what follows
    with np.errstate(all="ignore"):
        ref, last, gr = delta.gated_delta(*(f64(d[n]) for n in NAMES), 1.0, f64(d["state"]),
                                          do=np.ones(d["v"].shape), dstate=np.ones(d["state"].shape))
    o, got, work = forward(d, scale=1.0, initial_state=d["state"], keep=True)
    check(o, ref, torch.float32, "o")
    check(got, last, torch.float32, "state")
    grads = backward(d, torch.ones_like(d["v"]), work, scale=1.0, dfinal_state=torch.ones_like(d["state"]))
    for m in (*NAMES, "initial_state"):
        check(grads[m], gr[m], torch.float32, "d" + m, 2)
    # a NaN in one head's v stays in that head, and before it nothing changes
    d["v"][0, 100, 1, 3] = float("nan")
    o2, got2, _ = forward(d, scale=1.0, initial_state=d["state"])
    assert torch.equal(o2[:, :, 0], o[:, :, 0]) and torch.equal(got2[:, 0], got[:, 0])
    assert torch.equal(o2[:, :64, 1], o[:, :64, 1]) and torch.isnan(o2[0, 101:, 1, 3]).all()


@pytest.mark.parametrize("scale", [1e-18, 1e18])
def test_any_scale_of_the_values(scale):
    """Parts have float's exponents: results scale with v and the states (by a power of two exactly)."""
    torch = torch_cuda()
    scale = 2.0 ** round(np.log2(scale))
    d = make(1, 130, 1, 1, 64, 64)
    one, last, _ = forward(d, initial_state=d["state"])
    d["v"] *= scale
    two, last2, _ = forward(d, initial_state=d["state"] * scale)
    assert torch.equal(two, one * scale) and torch.equal(last2, last * scale)


def test_strided_tokens_and_streams_and_graph():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    B, T, Hk, Hv, Dk, Dv = 2, 140, 2, 4, 64, 64
    d = make(B, T, Hk, Hv, Dk, Dv, "bfloat16")
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(torch.bfloat16)
    want = forward(d, initial_state=d["state"], keep=True)
    grads = backward(d, do, want[2])
    wide = torch.cat([d[n].flatten(2) for n in ("q", "k", "v")], -1)
    e = dict(d)
    for n, t, h, w in zip(("q", "k", "v"), wide.split([Hk * Dk, Hk * Dk, Hv * Dv], -1), (Hk, Hk, Hv), (Dk, Dk, Dv)):
        e[n] = t.unflatten(-1, (h, w))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = forward(e, initial_state=d["state"], keep=True)
        g2 = backward(e, do, got[2])
    stream.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(g2[m], grads[m]) for m in grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, last, work = s4.gated_delta_forward(*(d[n] for n in NAMES), initial_state=d["state"], keep=True)
        g3 = s4.gated_delta_backward(*(d[n] for n in NAMES), do, work)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(last, want[1]) and all(torch.equal(g3[m], grads[m]) for m in grads)


def test_segments_in_a_graph_and_two_calls_at_once():
    """A captured call in segments answers for the inputs and offsets of its
    replay, not of its capture; a workspace is used again; calls on two
    streams with workspaces of their own do not touch each other."""
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(1, 2740, 1, 3, 64, 64, "bfloat16")
    other = make(1, 2740, 1, 3, 64, 64, "bfloat16", seed=9)
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(torch.bfloat16)
    cu = torch.tensor([0, 2500, 2501, 2740], dtype=torch.int32, device="cuda")
    cu2 = torch.tensor([3, 200, 400, 2739], dtype=torch.int32, device="cuda")
    run = lambda x, c, w=None: (  # noqa: E731
        lambda f: (f[0], f[1], *s4.gated_delta_backward(*(x[n] for n in NAMES), do, f[2], cu_seqlens=c).values()))(
            s4.gated_delta_forward(*(x[n] for n in NAMES), cu_seqlens=c, keep=True, workspace=w,
                                   out=torch.zeros_like(x["v"])))
    first, second = run(d, cu), run(other, cu2)
    work = torch.empty(s4.gated_delta_workspace_size(torch.bfloat16, 3, 2740, 1, 3, 64, 64, True), dtype=torch.uint8,
                       device="cuda").fill_(255)
    x, c = {n: d[n].clone() for n in NAMES}, cu.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x, c, work)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, first))
    for n in NAMES:
        x[n].copy_(other[n])
    c.copy_(cu2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, second))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = [[], []]
    for i, (y, k) in enumerate(((d, cu), (other, cu2))):
        streams[i].wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for i, (y, k) in enumerate(((d, cu), (other, cu2))):
            with torch.cuda.stream(streams[i]):
                results[i].append(run(y, k))
    torch.cuda.synchronize()
    for got, want in zip(results, (first, second)):
        assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))


def test_refusals():
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    d = make(2, 70, 2, 4, 64, 64, "bfloat16")
    args = lambda **c: [c.get(n, d[n]) for n in NAMES]  # noqa: E731
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    for bad, kind in [(dict(q=d["q"].float()), TypeError), (dict(g=d["g"].double()), TypeError),
                      (dict(k=d["k"][:, :5]), ValueError), (dict(v=d["v"].cpu()), TypeError),
                      (dict(beta=d["beta"][:, :, :2]), ValueError), (dict(q=d["q"][..., :32]), ValueError),
                      (dict(q=d["q"].transpose(1, 2)), ValueError)]:
        with pytest.raises(kind):
            s4.gated_delta_forward(*args(**bad))
    with pytest.raises(ValueError):
        s4.gated_delta_forward(*args(), cu_seqlens=cu)                       # a batch of two cannot be packed
    with pytest.raises(s4.S4Error):
        s4.gated_delta_forward(*args(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(s4.S4Error):
        s4.gated_delta_forward(*args(), scale=float("nan"))
    o, last, work = s4.gated_delta_forward(*args())
    with pytest.raises(s4.S4Error):                                          # a workspace without what backward reads
        s4.gated_delta_backward(*args(), torch.empty_like(d["v"]), work)
    with pytest.raises(TypeError):
        s4.gated_delta_backward(*args(), torch.empty_like(d["v"]), None)
    e = make(1, 8, 1, 1, 20, 64)
    with pytest.raises(s4.S4Error):
        s4.gated_delta_forward(*(e[n] for n in NAMES))                       # Dk not a multiple of 8
    with pytest.raises(s4.S4Error):
        s4.gated_delta_scan(*(e[n] for n in NAMES), e["state"])


@pytest.mark.parametrize("shape", [(1, 1500, 1, 2, 64, 64), (2, 2000, 1, 1, 40, 128)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_few_long_sequences_backward(shape, dtype):
    torch = torch_cuda()
    d = make(*shape, dtype=dtype)
    d["g"] *= 0.02
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(d["v"].dtype)
    ds = torch.randn(d["state"].shape, device="cuda", generator=gen(2))
    _, _, ref = delta.gated_delta(*(f64(d[n]) for n in NAMES), 0.3, f64(d["state"]), do=f64(do), dstate=f64(ds))
    _, _, work = forward(d, scale=0.3, initial_state=d["state"], keep=True)
    for _ in range(2):
        got = backward(d, do, work, scale=0.3, dfinal_state=ds)
        for m in (*NAMES, "initial_state"):      # one more chain and the joins, both ways
            check(got[m], ref[m], got[m].dtype, "d" + m, 4)


@pytest.mark.parametrize("packed", [False, True])
def test_one_workspace_for_all_lengths(packed):
    """A workspace made for the longest call serves shorter ones, in segments
    or not, whatever it holds."""
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    most, Hk, Hv, Dk, Dv = 3300, 1, 2, 64, 48
    work = torch.empty(s4.gated_delta_workspace_size(torch.bfloat16, 2, most, Hk, Hv, Dk, Dv, True), dtype=torch.uint8,
                       device="cuda")
    for tokens in (2, 130, 1024, 1026, 1980, 2048, 2050, 3200, 3264, 3300):
        d = make(1, tokens, Hk, Hv, Dk, Dv, "bfloat16") if packed else make(2, tokens // 2, Hk, Hv, Dk, Dv, "bfloat16")
        cu = torch.tensor([0, tokens // 5, tokens], dtype=torch.int32, device="cuda") if packed else None
        do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(torch.bfloat16)
        results = []
        for w in (None, work.fill_(255)):
            o, last, kept = forward(d, cu_seqlens=cu, keep=True, workspace=w)
            results.append((o, last, *backward(d, do, kept, cu_seqlens=cu).values()))
        assert all(torch.equal(a, b) for a, b in zip(*results)), tokens


def used(d, n):
    """A workspace of d's sizes for n sequences that holds what no call left: NaN in every type."""
    torch = torch_cuda()
    import structured_state_space_dplr_b200 as s4
    (B, T, Hk, Dk), (Hv, Dv) = d["q"].shape, d["v"].shape[2:]
    return torch.empty(s4.gated_delta_workspace_size(d["v"].dtype, n, B * T, Hk, Hv, Dk, Dv, True), dtype=torch.uint8,
                       device="cuda").fill_(255)


# In segments from no state: the first segment's M is not computed and the join
# leaves its product out; backward, no gradient comes from behind the last one.
@pytest.mark.parametrize("shape", [(1, 1500, 1, 2, 64, 64), (1, 2200, 2, 2, 128, 96), (2, 2000, 1, 1, 40, 128)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("state,dstate", [(False, False), (True, False), (False, True)])
def test_segments_without_states(shape, dtype, state, dstate):
    torch = torch_cuda()
    d = make(*shape, dtype=dtype)
    d["g"] *= 0.02
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(d["v"].dtype)
    ds = torch.randn(d["state"].shape, device="cuda", generator=gen(2)) if dstate else None
    start = d["state"] if state else None
    ref, last, gr = delta.gated_delta(*(f64(d[n]) for n in NAMES), 0.3, f64(start) if state else None, do=f64(do),
                                      dstate=f64(ds) if dstate else None)
    for keep in (False, True):
        o, got, work = forward(d, scale=0.3, initial_state=start, keep=keep, workspace=used(d, shape[0]))
        check(o, ref, d["v"].dtype, "o", 2)
        check(got, last, torch.float32, "state", 2)
    got = backward(d, do, work, scale=0.3, dfinal_state=ds)
    for m in (*NAMES, "initial_state"):
        check(got[m], gr[m], got[m].dtype, "d" + m, 4)


@pytest.mark.parametrize("cu", [[0, 2500, 2500, 2501, 2740], [7, 900, 1700, 2600, 2731]])
@pytest.mark.parametrize("dtype,shape", [("float16", (1, 3, 96, 80)), ("float32", (2, 2, 64, 128))])
def test_packed_segments_without_states(cu, dtype, shape):
    torch = torch_cuda()
    T = cu[-1] + 9
    d = make(1, T, *shape, dtype=dtype)
    args = packed(d, cu)
    do = torch.randn(d["v"].shape, device="cuda", generator=gen(1)).to(d["v"].dtype)
    ref, last, gr = delta.gated_delta(*args, 0.5, None, cu=cu, do=f64(do))
    o, final, work = forward(d, scale=0.5, cu_seqlens=d["cu"], keep=True, workspace=used(d, len(cu) - 1))
    check(o, ref, o.dtype, "o")
    check(final, last, torch.float32, "state")
    got = backward(d, do, work, scale=0.5, cu_seqlens=d["cu"])
    for m in (*NAMES, "initial_state"):
        check(got[m], gr[m], got[m].dtype, "d" + m, 2)
        if m != "initial_state":
            assert not got[m][:, :cu[0]].any() and not got[m][:, cu[-1]:].any()


def test_calls_from_two_threads_in_a_new_process():
    """Value heads of different sizes, and rows of different lengths, share
    kernels whose shared memory is asked for by whoever comes first."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import sys, threading
sys.path[:0] = [%r, %r]
import torch
import structured_state_space_dplr_b200 as s4
from test_gpu_gated_delta import NAMES, gen
from test_gpu_gated_delta_scan import make
cases = [make(1, 70, 1, 2, 128, Dv, "bfloat16") for Dv in (128, 64, 128, 8)]
x = [torch.randn(40, D, device="cuda", generator=gen(1)).bfloat16() for D in (8192, 520, 4096, 2048)]
torch.cuda.synchronize()
start, results = threading.Barrier(4), [[] for _ in cases]
def run(i):
    start.wait()
    for _ in range(20):
        d = cases[i]
        o, last, work = s4.gated_delta_forward(*(d[n] for n in NAMES), keep=True)
        grads = s4.gated_delta_backward(*(d[n] for n in NAMES), d["v"], work)
        w = torch.ones(x[i].shape[1], device="cuda")
        z, mean, rstd = s4.layernorm(x[i], w, w)
        results[i].append((o, last, *grads.values(), z, *s4.layernorm_backward(z, x[i], w, mean, rstd)))
    torch.cuda.synchronize()
threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
for r in results:
    assert len(r) == 20, len(r)
    assert all(torch.equal(a, b) for one in r for a, b in zip(one, r[0]))
    assert all(torch.isfinite(a).all() for a in r[0])
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
