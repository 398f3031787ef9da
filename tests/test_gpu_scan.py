"""GPU parity of scan_prefill and scan_decode with their 64-bit restatement, whose running
error bound (tests/plain_ops.py) is the tolerance."""

import pytest
import torch

import plain_ops as po
from linear_attention_recurrent_selective_b200 import ssu
from parity import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")


def make(seed, batch, T, ch, G, N, xdt=F32, ddt=None, bdt=None, sdt=F32, z=True, D=True,
         bias=True, slots=None, wide=0, slot_pad=0, positive=False):
    """CPU inputs; with ``wide`` every tensor is a slice of rows that much wider."""
    g = po.generator(seed)
    ddt, bdt, P = ddt or xdt, bdt or xdt, batch + 2

    def rows(*inner, dtype):
        n = 1
        for v in inner:
            n *= v
        t = po.rand(g, batch, T, n + wide).to(dtype)
        return t, (wide // 2, n, inner)
    c = dict(batch=batch, T=T, ch=ch, G=G, N=N, P=P, sdt=sdt, xdt=xdt, slot_pad=slot_pad)
    c["x"] = rows(ch, dtype=xdt)
    c["dt"] = rows(ch, dtype=ddt)
    if positive:
        c["dt"] = (c["dt"][0].abs(), c["dt"][1])
    c["B"], c["C"] = rows(G, N, dtype=bdt), rows(G, N, dtype=bdt)
    c["z"] = rows(ch, dtype=xdt) if z else None
    c["A"] = -torch.exp(po.rand(g, ch, N))
    c["D"] = po.rand(g, ch) if D else None
    c["bias"] = po.rand(g, ch) - 2 if bias else None
    c["pool"] = po.rand(g, P * (ch * N + slot_pad)).to(sdt)
    c["slots"] = (torch.randperm(P, generator=g)[:batch].int() if slots is None
                  else torch.tensor(slots, dtype=torch.int32))
    return c


def cut(t, cuda=False):
    if t is None:
        return None
    full, (at, n, inner) = t
    full = full.cuda() if cuda else full
    return full[..., at:at + n].unflatten(-1, inner) if len(inner) > 1 else full[..., at:at + n]


def run(c, lengths=None, update=True, out=True, active=None, softplus=True, stream=None):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    pool, err = c["pool"].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((c["batch"], c["T"], c["ch"]), NAN, dtype=c["xdt"], device="cuda")
    ssu.scan_prefill(cut(c["x"], 1), cut(c["dt"], 1), d(c["A"]), cut(c["B"], 1), cut(c["C"], 1),
                     pool, o if out else None, D=d(c["D"]), z=cut(c["z"], 1),
                     dt_bias=d(c["bias"]), dt_softplus=softplus, state_indices=d(c["slots"]),
                     context_lengths=d(lengths), update_state=update, active_batch=active,
                     err_flags=err, slot_stride=c["ch"] * c["N"] + c["slot_pad"], P=c["P"],
                     stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), pool.cpu(), int(err.item())


def run_decode(c, t=0, pool=None, active=None, softplus=True):
    d = lambda v: None if v is None else v.cuda()  # noqa: E731
    one = lambda v: None if v is None else cut(v, 1)[:, t]  # noqa: E731
    pool = c["pool"].cuda() if pool is None else pool
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((c["batch"], c["ch"]), NAN, dtype=c["xdt"], device="cuda")
    ssu.scan_decode(one(c["x"]), one(c["dt"]), d(c["A"]), one(c["B"]), one(c["C"]), pool, o,
                    D=d(c["D"]), z=one(c["z"]), dt_bias=d(c["bias"]), dt_softplus=softplus,
                    state_indices=d(c["slots"]), active_batch=active, err_flags=err,
                    slot_stride=c["ch"] * c["N"] + c["slot_pad"], P=c["P"])
    torch.cuda.synchronize()
    return o.cpu(), pool.cpu(), int(err.item())


def plain(c, **kw):
    pool = c["pool"].view(c["P"], -1)[:, :c["ch"] * c["N"]].reshape(c["P"], c["ch"], c["N"])
    return po.scan(cut(c["x"]), cut(c["dt"]), c["A"], cut(c["B"]), cut(c["C"]), pool, c["slots"],
                   D=c["D"], z=cut(c["z"]), dt_bias=c["bias"], **kw)


def near(got, want, lim, dtype, what):
    lim = lim + (want.abs() + lim) * po.half_step(dtype) + po.tiny(dtype)
    bad = ~((got.double() - want).abs() <= lim) & ~torch.isnan(want)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           ((got.double() - want).abs() / lim)[bad].max().item())


def compare(c, o, pool, err, want, state, lim, slim, flags, out=True):
    assert err == flags
    if out:
        assert torch.equal(torch.isnan(o), torch.isnan(want))
        near(o, want, lim, c["xdt"], "out")
    else:
        assert torch.isnan(o).all()
    flat = pool.view(c["P"], -1)
    got = flat[:, :c["ch"] * c["N"]].reshape(c["P"], c["ch"], c["N"])
    near(got, state, slim, c["sdt"], "state")
    before = c["pool"].view(c["P"], -1)
    touched = (slim.flatten(1) > 0).any(1)
    assert same_bits(flat[~touched], before[~touched])           # other slots: not a bit
    assert same_bits(flat[:, c["ch"] * c["N"]:], before[:, c["ch"] * c["N"]:])


def check(c, lengths=None, update=True, out=True, active=None, softplus=True):
    o, pool, err = run(c, lengths, update, out, active, softplus)
    want = plain(c, lengths=lengths, update=update, active=active, softplus=softplus)
    compare(c, o, pool, err, *want, out=out)
    return o, pool


DTYPES = [(F32, F32, F32, F32), (BF16, BF16, BF16, F32), (F16, F32, F16, F16),
          (BF16, F32, F32, BF16)]


@pytest.mark.parametrize("xdt,ddt,bdt,sdt", DTYPES)
@pytest.mark.parametrize("N", [8, 16, 32, 64, 128, 256])
def test_prompts(N, xdt, ddt, bdt, sdt):
    c = make(N, 5, 37, 72, 1, N, xdt, ddt, bdt, sdt)
    check(c, torch.tensor([37, 0, 1, 8, 33], dtype=torch.int32))


@pytest.mark.parametrize("ch,G", [(1, 1), (7, 1), (7, 7), (63, 3), (65, 1), (130, 2), (200, 25)])
@pytest.mark.parametrize("N", [8, 16, 128])
def test_odd_channels_and_groups(ch, G, N):
    check(make(ch, 2, 19, ch, G, N, BF16, F32, BF16))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 64, 257])
@pytest.mark.parametrize("N", [16, 256])
def test_token_counts(T, N):
    check(make(T, 2, T, 40, 1, N, BF16))


@pytest.mark.parametrize("wide", [16, 6, 3])
@pytest.mark.parametrize("xdt", [F32, BF16])
def test_slices_of_wider_rows(wide, xdt):
    c = make(wide, 3, 21, 48, 2, 16, xdt, wide=wide, slot_pad=8)
    check(c)
    o, pool, err = run_decode(c)
    w = plain_decode(c)
    compare(c, o, pool, err, *w)


@pytest.mark.parametrize("N", [8, 16, 128, 256])
@pytest.mark.parametrize("T", [300, 1100])
def test_long_rows_of_few_channels(T, N):
    """Rows split over several CTAs: ragged, empty and shorter than one part."""
    c = make(T, 10, T, 20, 1, N, BF16 if N == 16 else F32, slots=[2, 5, -1, 3, 9, 0, 1, 40, 7, 4])
    lengths = torch.tensor([T, 0, 5, 1, 15, 17, 100, 3, T - 1, T // 2 + 3], dtype=torch.int32)
    o, pool = check(c, lengths)
    check(c, lengths, update=False)
    check(c, lengths, out=False)
    again, same, _ = run(c, lengths)
    assert same_bits(again, o) and same_bits(same, pool)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("ch,G,xdt", [(1, 1, F32), (70, 2, BF16), (33, 3, F16)])
def test_one_long_row(N, ch, G, xdt):
    """One row cut into as many segments as there are."""
    c = make(N + ch, 1, 4500, ch, G, N, xdt, F32 if N == 8 else None)
    c["A"] = c["A"] * 0.05
    check(c)
    check(c, torch.tensor([4097], dtype=torch.int32), out=False)


def test_options_padding_and_flags():
    c = make(2, 6, 9, 24, 1, 32, F32, slots=[3, -1, 99, 0, 5, 1], z=False, D=False, bias=False,
             positive=True)
    lengths = torch.tensor([9, 4, 5, 12, -2, 3], dtype=torch.int32)
    o, _ = check(c, lengths, softplus=False)
    assert (o[1] == 0).all()
    check(c, lengths, active=2)
    check(c, lengths, update=False)
    check(c, lengths, out=False)


def test_steps_of_every_size():
    """softplus over its whole range (a step of e^-90 to one of 80) and infinite inputs."""
    c = make(3, 1, 24, 16, 1, 16, F32, bias=False, z=False)
    v = torch.linspace(-90, 80, 24 * 16).view(1, 24, 16)
    c["dt"] = (v, c["dt"][1])
    c["A"] = -torch.rand(16, 16) - 0.01
    check(c)
    v[0, 3, 2], v[0, 3, 3] = -float("inf"), NAN
    o, pool, _ = run(c)
    want, state, _, _, _ = plain(c)
    got = pool.view(c["P"], 16, 16).double()
    s = int(c["slots"][0])
    assert torch.isfinite(got[s, 2]).all() and torch.isnan(got[s, 3]).all()
    assert torch.allclose(got[s, 2], state[s, 2], rtol=1e-4, atol=1e-6)
    assert torch.isnan(o[0, 3:, 3]).all() and torch.isfinite(o[0, :, 2]).all()


def plain_decode(c, **kw):
    one = {k: (c[k][0][:, :1], c[k][1]) for k in ("x", "dt", "B", "C")}
    one["z"] = None if c["z"] is None else (c["z"][0][:, :1], c["z"][1])
    out, state, lim, slim, flags = plain({**c, **one, "T": 1}, **kw)
    return out[:, 0], state, lim[:, 0], slim, flags


@pytest.mark.parametrize("xdt,ddt,bdt,sdt", DTYPES)
@pytest.mark.parametrize("N", [8, 16, 32, 64, 128, 256])
def test_decode(N, xdt, ddt, bdt, sdt):
    c = make(N, 7, 1, 53, 1, N, xdt, ddt, bdt, sdt, slot_pad=16)
    compare(c, *run_decode(c), *plain_decode(c))


@pytest.mark.parametrize("batch,ch,G", [(1, 1, 1), (2, 64, 4), (5, 300, 3), (9, 33, 33)])
def test_decode_shapes(batch, ch, G):
    c = make(batch, batch, 1, ch, G, 16, BF16)
    compare(c, *run_decode(c), *plain_decode(c))


def test_decode_padding_flags_and_options():
    c = make(4, 6, 1, 40, 1, 64, F32, slots=[3, -1, 99, 0, -5, 1], z=False, D=False, bias=False,
             positive=True)
    o, pool, err = run_decode(c, softplus=False, active=5)
    compare(c, o, pool, err, *plain_decode(c, softplus=False, active=5))
    assert (o[1] == 0).all() and torch.isnan(o[2]).all() and torch.isnan(o[5]).all()


def test_prompt_is_its_tokens_one_by_one():
    """Both forms within their bounds of one truth: the difference is within both."""
    c = make(8, 4, 12, 100, 2, 16, F32)
    o, pool, _ = run(c)
    want, state, lim, slim, _ = plain(c)
    step = c["pool"].cuda()
    for t in range(12):
        ot, _, _ = run_decode(c, t, step)
        near(ot, want[:, t], lim[:, t], F32, t)
    near(step.cpu().view(c["P"], 100, 16), state, slim, F32, "state")


def test_verify_then_commit():
    """update_state off leaves the pool, out = None with the accepted lengths commits what a
    prompt of that length would."""
    c = make(9, 3, 6, 64, 1, 16, BF16)
    acc = torch.tensor([0, 6, 4], dtype=torch.int32)
    o, pool, _ = run(c, update=False)
    assert same_bits(pool, c["pool"])
    full, want, _ = run(c, acc)
    _, got, _ = run(c, acc, out=False)
    assert same_bits(got, want)
    assert same_bits(o[1], full[1])


def test_long_memory():
    """4099 tokens with decays near one: errors add up as the bound says, no faster."""
    c = make(10, 1, 4099, 8, 1, 16, F32, z=False)
    c["A"] = c["A"] * 1e-3
    check(c)


def test_in_cuda_graph_and_on_another_stream():
    c = make(11, 3, 50, 96, 1, 16, BF16)
    lengths = torch.tensor([50, 0, 17], dtype=torch.int32)
    o, pool, _ = run(c, lengths)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, pool2, _ = run(c, lengths, stream=s)
    assert same_bits(o2, o) and same_bits(pool2, pool)
    t = {k: cut(c[k], 1) for k in ("x", "dt", "B", "C", "z")}
    A, D, bias, sl, ln = (c[k].cuda() if k != "L" else lengths.cuda()
                          for k in ("A", "D", "bias", "slots", "L"))
    p = c["pool"].cuda()
    out = torch.full((3, 50, 96), NAN, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ssu.scan_prefill(t["x"], t["dt"], A, t["B"], t["C"], p, out, D=D, z=t["z"], dt_bias=bias,
                         state_indices=sl, context_lengths=ln, P=c["P"])
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(out, o) and same_bits(p, pool)


def test_refusals():
    c = make(1, 2, 4, 32, 1, 16, BF16)
    good = [cut(c["x"], 1), cut(c["dt"], 1), c["A"].cuda(), cut(c["B"], 1), cut(c["C"], 1),
            c["pool"].cuda(), torch.empty(2, 4, 32, dtype=BF16, device="cuda")]

    def bad(i, t, exc=ValueError, **kw):
        args = list(good)
        args[i] = t
        with pytest.raises(exc):
            ssu.scan_prefill(*args, P=c["P"], **kw)
    bad(0, good[0].cpu())
    bad(0, good[0].transpose(1, 2).contiguous().transpose(1, 2))
    bad(1, good[1][:, :3])
    bad(2, good[2].double())
    bad(2, good[2][:, :8])
    bad(4, good[4].float())
    bad(5, good[5][:-1])
    bad(6, good[6].float())
    bad(6, None, ssu.SSUError, update_state=False)
    with pytest.raises(ValueError):
        ssu.scan_prefill(*good, P=c["P"], context_lengths=torch.zeros(3, dtype=torch.int32,
                                                                       device="cuda"))


@pytest.mark.parametrize("N", [8, 16, 128])
def test_steps_of_zero_keep_every_bit(N):
    c = make(12, 2, 70, 24, 1, N, F32, z=False, bias=False)
    c["dt"][0].zero_()
    _, pool, _ = run(c, softplus=False)
    assert same_bits(pool, c["pool"])
    step = c["pool"].cuda()
    for _ in range(3):
        run_decode(c, 0, step, softplus=False)
    assert same_bits(step, c["pool"])


def test_errors_do_not_gather():
    """500 slow steps: the states' error stays that of a few roundings (a decay that is half a
    step low every time would be off by 500 * 2^-25 = 1.5e-5)."""
    c = make(13, 2, 500, 32, 1, 16, F32, z=False, bias=False)
    c["dt"] = (torch.full_like(c["dt"][0], 0.05) * (1 + 0.1 * c["x"][0].cos()), c["dt"][1])
    c["A"] = -0.02 * torch.rand(32, 16, generator=po.generator(3))
    _, pool, _ = run(c, softplus=False)
    _, state, _, _, _ = plain(c, softplus=False)
    live = c["slots"].long()
    got = pool.view(c["P"], 32, 16).double()[live]
    # 500 independent roundings of a half step each, four deep, add up to about
    # sqrt(500) * 4 * 2^-25 = 2.7e-6 of the state's size
    assert ((got - state[live]).norm() / state[live].norm()).item() < 2.7e-6


@pytest.mark.parametrize("T", [9, 1100])
def test_nan_behind_the_rows_is_never_read(T):
    c = make(14, 4, T, 24, 1, 16, F32, slots=[3, 1, -1, 0])
    lengths = torch.tensor([0, T - 1, 3, 5], dtype=torch.int32)
    o, pool = check(c, lengths)
    for b, n in enumerate(lengths.tolist()):
        for k in ("x", "dt", "B", "C", "z"):
            c[k][0][b, 0 if b == 2 else n:] = NAN
    o2, pool2 = check(c, lengths)
    assert same_bits(o, o2) and same_bits(pool, pool2)
    o, pool, err = run_decode(c)            # rows 0 and 2: NaN inputs, row 2 is padding
    assert (o[2] == 0).all() and err == 0
    assert torch.isfinite(pool.view(c["P"], -1)[1]).all()


def test_pool_past_32_bits():
    """A slot whose states lie beyond 2^31 elements of the pool."""
    c = make(15, 2, 5, 5120, 1, 16, BF16, sdt=BF16, z=False)
    P, per = 27000, 5120 * 16
    assert (P - 1) * per > 2 ** 31
    small = c["pool"].view(c["P"], per)
    pool = torch.zeros(P, 5120, 16, dtype=BF16, device="cuda")
    slots = [int(s) for s in c["slots"]]
    far = [P - 1, 7]
    for f, s in zip(far, slots):
        pool[f] = small[s].view(5120, 16).cuda()
    want, state, lim, slim, _ = plain(c)
    out = torch.empty(2, 5, 5120, dtype=BF16, device="cuda")
    idx = torch.tensor(far, dtype=torch.int32, device="cuda")
    ssu.scan_prefill(cut(c["x"], 1), cut(c["dt"], 1), c["A"].cuda(), cut(c["B"], 1),
                     cut(c["C"], 1), pool, out, D=c["D"].cuda(), dt_bias=c["bias"].cuda(),
                     state_indices=idx)
    torch.cuda.synchronize()
    near(out.cpu(), want, lim, BF16, "out")
    near(pool[far].cpu(), state[slots], slim[slots], BF16, "state")
    one = torch.empty(2, 5120, dtype=BF16, device="cuda")
    before = pool[far].clone()
    ssu.scan_decode(cut(c["x"], 1)[:, 0].contiguous(), cut(c["dt"], 1)[:, 0].contiguous(),
                    c["A"].cuda(), cut(c["B"], 1)[:, 0].contiguous(),
                    cut(c["C"], 1)[:, 0].contiguous(), pool, one, state_indices=idx)
    assert not torch.equal(pool[far], before)
    assert int((pool != 0).flatten(1).any(1).sum()) == 2


def test_long_row_in_a_graph_beside_another_stream():
    """Segments over a cluster, captured by a first call and replayed, while the same call
    runs on another stream with buffers of its own."""
    c = make(16, 1, 3000, 40, 1, 16, BF16)
    want, pool, _ = run(c)
    t = {k: cut(c[k], 1) for k in ("x", "dt", "B", "C", "z")}
    A, D, bias, sl = (c[k].cuda() for k in ("A", "D", "bias", "slots"))
    pools = [c["pool"].cuda() for _ in range(2)]
    outs = [torch.zeros(1, 3000, 40, dtype=BF16, device="cuda") for _ in range(2)]
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()

    def go(i, stream=None):
        ssu.scan_prefill(t["x"], t["dt"], A, t["B"], t["C"], pools[i], outs[i], D=D, z=t["z"],
                         dt_bias=bias, state_indices=sl, P=c["P"], stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go(0)
    graph.replay()
    go(1, s2)
    torch.cuda.synchronize()
    for i in range(2):
        assert same_bits(outs[i], want) and same_bits(pools[i], pool)


@pytest.mark.parametrize("T,ch,N", [(1, 72, 8), (37, 72, 16), (45, 40, 128), (300, 16, 16),
                                    (1100, 16, 64)])
def test_rates_of_minus_infinity(T, ch, N):
    """A state that forgets at once holds the last token's input, as with any rate whose decay
    is 0 in fp32, whatever the tokens that a tile holds behind the row."""
    c = make(T + N, 2, T, ch, 1, N, BF16)
    hit = torch.rand(ch, N, generator=po.generator(9)) < 0.3
    c["A"] = torch.where(hit, torch.tensor(-1e30), c["A"])
    lengths = torch.tensor([T, max(T - 2, 1)], dtype=torch.int32)
    want = run(c, lengths), run_decode(c)
    c["A"] = torch.where(hit, torch.tensor(float("-inf")), c["A"])
    for got, ref in zip((run(c, lengths), run_decode(c)), want):
        assert torch.isfinite(ref[1]).all() and got[2] == ref[2]
        assert same_bits(got[0], ref[0]) and same_bits(got[1], ref[1])


def test_negative_sizes_are_refused():
    c = make(1, 2, 4, 32, 1, 16, BF16)
    args = [cut(c["x"], 1), cut(c["dt"], 1), c["A"].cuda(), cut(c["B"], 1), cut(c["C"], 1),
            c["pool"].cuda(), torch.empty(2, 4, 32, dtype=BF16, device="cuda")]
    for kw in (dict(P=-1), dict(P=c["P"], slot_stride=-1)):
        with pytest.raises(ValueError):
            ssu.scan_prefill(*args, **kw)
