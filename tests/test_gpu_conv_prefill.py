"""GPU parity of ssu_conv_prefill (prompts and draft trees) and ssu_conv_replay with their
64-bit restatements, and with the fused single-token ssu_conv_decode."""

import pytest
import torch

import plain_ops as po
from linear_attention_recurrent_selective_b200 import ssu
from parity import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")


def make(seed, batch, T, xd, bc, width, dtype, layout="channel", slots=None, extra=0, shift=0,
         pad=0, bias=True):
    """CPU inputs; xbc a slice of rows that are ``extra`` elements wider, ``shift`` in."""
    g = po.generator(seed)
    ch, taps, P = xd + 2 * bc, width - 1, batch + 3
    rows = po.rand(g, batch, T, ch + extra).to(dtype)
    strides = {"channel": (ch * taps + pad, taps, 1), "tap": (ch * taps + pad, 1, ch),
               "spread": (2 * ch * taps + pad, 2 * taps, 2)}[layout]
    order = torch.randperm(P, generator=g)[:batch].to(torch.int32)
    return dict(rows=rows, shift=shift, ch=ch, xd=xd, bc=bc, width=width, P=P, strides=strides,
                weight=po.rand(g, ch, width).to(dtype), T=T, batch=batch, dtype=dtype,
                bias=po.rand(g, ch).to(dtype) if bias else None,
                pool=po.rand(g, max(P * strides[0], 1)).to(dtype),
                slots=order if slots is None else torch.tensor(slots, dtype=torch.int32))


def xbc_of(c, rows):
    return rows[..., c["shift"]:c["shift"] + c["ch"]]


def run(c, lengths=None, parents=None, silu=True, update=True, active=None, stream=None):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    pool, err = c["pool"].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full((c["batch"], c["T"], n), NAN, dtype=c["dtype"], device="cuda")
            for n in (c["xd"], c["bc"], c["bc"]) if n]
    x, B, C = outs + [None] * (3 - len(outs))
    ssu.ssu_conv_prefill(xbc_of(c, c["rows"].cuda()), d(c["weight"]), pool, x, B, C,
                         width=c["width"], conv_strides=c["strides"], conv_bias=d(c["bias"]),
                         conv_silu=silu, state_indices=d(c["slots"]), context_lengths=d(lengths),
                         parent_ids=d(parents), update_state=update, active_batch=active,
                         err_flags=err, P=c["P"], stream=stream)
    torch.cuda.synchronize()
    return torch.cat([o.cpu() for o in outs], 2), pool.cpu(), int(err.item())


def check(c, lengths=None, parents=None, silu=True, update=True, active=None):
    y, pool, err = run(c, lengths, parents, silu, update, active)
    want, after, lim, flags = po.conv(
        xbc_of(c, c["rows"]), c["weight"], c["bias"], c["pool"], c["strides"], c["width"],
        c["slots"], c["P"], lengths, parents, silu, update, active)
    assert err == flags
    assert same_bits(pool, after)                       # taps are copies
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    # the output is rounded once, on top of the fp32 arithmetic's bound
    lim = lim + (want.abs() + lim) * po.half_step(c["dtype"]) + po.tiny(c["dtype"])
    bad = ((y.double() - want).abs() > lim) & ~torch.isnan(want)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    return y, pool


LEN = [0, 1, 2, 3, 5, 32, 33, 70]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 7, 8, 16])
@pytest.mark.parametrize("layout", ["channel", "tap", "spread"])
def test_prompts_of_every_length(dtype, width, layout):
    c = make(width, 8, 70, 24, 8, width, dtype, layout, pad=8)
    check(c, torch.tensor(LEN, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("xd,bc,extra,shift", [(13, 3, 0, 0), (16, 8, 3, 0), (16, 8, 16, 8),
                                               (16, 8, 16, 5), (1, 0, 0, 0), (40, 0, 8, 8),
                                               (8, 1, 0, 0)])
def test_odd_channels_and_slices(dtype, xd, bc, extra, shift):
    c = make(xd, 3, 9, xd, bc, 4, dtype, extra=extra, shift=shift)
    check(c, torch.tensor([9, 2, 7], dtype=torch.int32))


@pytest.mark.parametrize("T", [1, 2, 31, 32, 34, 64, 97])
def test_token_counts(T):
    check(make(T, 2, T, 64, 16, 4, BF16))


def test_options_padding_and_flags():
    c = make(1, 6, 5, 16, 8, 4, F32, slots=[3, -1, 99, 0, 5, 1], bias=False)
    lengths = torch.tensor([5, 4, 5, 9, -2, 3], dtype=torch.int32)
    y, _ = check(c, lengths, silu=False)
    assert (y[1] == 0).all()
    y, _ = check(c, lengths, active=2, update=False)
    assert torch.isnan(y[2:]).all()


def trees(seed, batch, T):
    g = po.generator(seed)
    par = torch.full((batch, T), -1, dtype=torch.int32)
    for b in range(batch):
        for i in range(1, T):
            if torch.rand(1, generator=g) < 0.9:
                par[b, i] = int(torch.randint(0, i, (1,), generator=g))
    return par


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("width,xd", [(1, 16), (2, 16), (3, 13), (4, 16), (4, 13), (6, 16)])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_trees(dtype, width, xd, T):
    c = make(width + T, 3, T, xd, 8, width, dtype, "tap")
    check(c, parents=trees(T, 3, T), update=False)


def test_shuffled_and_malformed_trees():
    c = make(2, 3, 6, 16, 8, 4, F32)
    par = torch.tensor([[3, 0, 0, -1, 3, 1],          # parents after their children
                        [-1, 0, 7, 2, -5, 4],         # out of range on both sides
                        [0, 2, 1, -1, 3, 5]], dtype=torch.int32)   # cycles of one and two
    check(c, parents=par, update=False)
    check(c, torch.tensor([6, 2, 4], dtype=torch.int32), parents=par, update=False)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("width", [2, 3, 4, 5, 16])
@pytest.mark.parametrize("layout,xd", [("channel", 24), ("tap", 24), ("channel", 13), ("spread", 8)])
@pytest.mark.parametrize("tree", [False, True])
def test_commit(dtype, width, layout, xd, tree):
    c = make(width, 8, 20, xd, 0, width, dtype, layout, slots=[4, 2, -1, 0, 50, 9, 7, 1], pad=8)
    acc = torch.tensor([0, 1, 3, 2, 2, 20, 25, -1], dtype=torch.int32)
    nodes = None
    if tree:
        g = po.generator(8)
        nodes = torch.stack([torch.randperm(20, generator=g)[:18] for _ in range(8)]).int()
        nodes[3, 1] = 20                              # an id past the tokens: row untouched
        nodes[0, 0] = -7                              # not among the accepted: ignored
    pool, err = c["pool"].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ssu.ssu_conv_replay(c["rows"].cuda(), pool, acc.cuda(), width=width,
                        conv_strides=c["strides"], state_indices=c["slots"].cuda(),
                        accepted_node_ids=None if nodes is None else nodes.cuda(),
                        err_flags=err, P=c["P"])
    want, flags = po.conv_replay(c["rows"], c["pool"], c["strides"], width, c["slots"], c["P"],
                                 acc, nodes)
    torch.cuda.synchronize()
    assert int(err.item()) == flags and same_bits(pool, want)


def test_prompt_equals_single_tokens_of_the_fused_decode():
    """The windows that ssu_conv_decode leaves after T tokens, and (T = 1) the same x, B and
    C: a state of zero with dt = 1 and A = 0 takes B x in, so its outputs follow them."""
    H, G, Dm, N, T = 2, 1, 16, 32, 6
    ch = H * Dm + 2 * G * N
    c = make(9, 3, T, H * Dm, G * N, 4, BF16)
    _, pool = check(c)
    step = c["pool"].cuda()
    dev = dict(device="cuda")
    state = torch.zeros(c["P"], H, Dm, N, **dev)
    out = torch.empty(3, H, Dm, dtype=BF16, **dev)
    for t in range(T):
        ssu.ssu_conv_decode(c["rows"][:, t].contiguous().cuda(), c["weight"].cuda(), step,
                            torch.zeros(H, **dev), torch.ones(3, H, **dev), state, out, width=4,
                            conv_strides=c["strides"], nheads=H, ngroups=G, dim=Dm,
                            conv_bias=c["bias"].cuda(), state_indices=c["slots"].cuda(),
                            P=c["P"])
    assert ch == c["ch"] and same_bits(step, pool)


def test_whole_headline_prompt():
    """80 heads of 64 and a group of 128 states, 16 ragged rows of 512 tokens, against the
    same sums in 64 bits by torch on the device."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    b, T, xd, bc, W = 16, 512, 5120, 128, 4
    ch = xd + 2 * bc
    rows = torch.randn(b, T, ch + 80, generator=g, device="cuda").to(BF16)
    xbc = rows[..., 16:16 + ch]
    w = torch.randn(ch, W, generator=g, device="cuda").to(BF16)
    pool = torch.randn(20, ch, W - 1, generator=g, device="cuda").to(BF16)
    L = torch.randint(0, T + 1, (b,), generator=g, device="cuda").int()
    slots = torch.randperm(20, generator=g, device="cuda")[:b].int()
    full = torch.cat([pool[slots.long()].transpose(1, 2), xbc], 1).double()
    v = sum(full[:, k:k + T] * w[:, k].double() for k in range(W))
    mag = sum((full[:, k:k + T] * w[:, k].double()).abs() for k in range(W))
    outs = [torch.full((b, T, n), NAN, dtype=BF16, device="cuda") for n in (xd, bc, bc)]
    ssu.ssu_conv_prefill(xbc, w, pool, *outs, width=W, conv_strides=(ch * 3, 3, 1),
                         state_indices=slots, context_lengths=L)
    want = v * torch.sigmoid(v)
    got = torch.cat(outs, 2)
    live = (torch.arange(T, device="cuda") < L[:, None])[..., None]
    assert torch.isnan(got.masked_select(~live)).all()
    lim = 1.1 * 5 * po.U * mag + want.abs() * ((8 + 2 * v.abs()) * po.U + 2.0 ** -8 * 1.01)
    assert (((got.double() - want).abs() <= lim + 1e-38) | ~live).all()
    after = torch.stack([full[i, int(n):int(n) + 3].T for i, n in enumerate(L.tolist())])
    assert torch.equal(pool[slots.long()].double(), after)


def test_in_cuda_graph_and_on_another_stream():
    c = make(5, 3, 40, 64, 16, 4, BF16)
    lengths = torch.tensor([40, 0, 17], dtype=torch.int32)
    y, pool, _ = run(c, lengths)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, pool2, _ = run(c, lengths, stream=s)
    assert same_bits(y2, y) and same_bits(pool2, pool)
    rows, w, bias = c["rows"].cuda(), c["weight"].cuda(), c["bias"].cuda()
    p, sl, ln = c["pool"].cuda(), c["slots"].cuda(), lengths.cuda()
    outs = [torch.full((3, 40, n), NAN, dtype=BF16, device="cuda") for n in (64, 16, 16)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ssu.ssu_conv_prefill(rows, w, p, *outs, width=4, conv_strides=c["strides"],
                             conv_bias=bias, state_indices=sl, context_lengths=ln, P=c["P"])
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(torch.cat(outs, 2), y) and same_bits(p, pool)
    # other lengths in the same graph, from the original windows
    ln.copy_(torch.tensor([3, 40, 0]))
    p.copy_(c["pool"])
    for o in outs:
        o.fill_(NAN)
    graph.replay()
    torch.cuda.synchronize()
    y3, pool3, _ = run(c, torch.tensor([3, 40, 0], dtype=torch.int32))
    assert same_bits(torch.cat(outs, 2), y3) and same_bits(p, pool3)


def test_refusals():
    c = make(1, 2, 5, 16, 8, 4, BF16)
    rows, w, pool = c["rows"].cuda(), c["weight"].cuda(), c["pool"].cuda()
    new = lambda n, dt=BF16: torch.empty(2, 5, n, dtype=dt, device="cuda")  # noqa: E731
    x, B, C = new(16), new(8), new(8)
    kw = dict(width=4, conv_strides=c["strides"], P=c["P"])
    with pytest.raises(ValueError):
        ssu.ssu_conv_prefill(c["rows"], w, pool, x, B, C, **kw)       # a CPU tensor
    with pytest.raises(ValueError):
        ssu.ssu_conv_prefill(rows, w, pool, new(15), B, C, **kw)
    with pytest.raises(ValueError):
        ssu.ssu_conv_prefill(rows, w, pool, new(16, F16), B, C, **kw)
    with pytest.raises(ValueError):
        ssu.ssu_conv_prefill(rows.transpose(0, 1), w, pool, x, B, C, **kw)
    with pytest.raises(ValueError):
        ssu.ssu_conv_prefill(rows, w, pool, x, B, C, **{**kw, "P": c["P"] + 1})
    with pytest.raises(ValueError):
        ssu.ssu_conv_prefill(rows, w, pool.float(), x, B, C, **kw)
    par = torch.full((2, 5), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(ssu.SSUError):
        ssu.ssu_conv_prefill(rows, w, pool, x, B, C, parent_ids=par, **kw)
    with pytest.raises(ssu.SSUError):                                 # taps that overlap
        ssu.ssu_conv_prefill(rows, w, pool, x, B, C, **{**kw, "conv_strides": (96, 2, 1)})
    with pytest.raises(ValueError):
        ssu.ssu_conv_replay(rows, pool, torch.zeros(3, dtype=torch.int32, device="cuda"), **kw)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("width", [2, 3, 4, 5])
@pytest.mark.parametrize("layout", ["channel", "tap", "spread"])
def test_single_tokens(dtype, width, layout):
    """One token a row, an odd number of rows, with padding, an index past the pool and lengths
    of zero and beyond one."""
    c = make(width, 9, 1, 64, 16, width, dtype, layout, pad=8,
             slots=[3, -1, 99, 0, 5, 1, 11, 7, 2])
    lengths = torch.tensor([1, 1, 1, 0, 3, -2, 1, 1, 1], dtype=torch.int32)
    check(c, lengths)
    check(c, active=6)
    check(c, update=False, silu=False)


@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("width", [2, 4, 8, 16])
def test_weights_bias_and_outputs_off_16_bytes(T, width):
    """Contiguous tensors that start two bytes behind an aligned address."""
    c = make(T + width, 3, T, 16, 8, width, BF16)

    def off(t):
        wide = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        wide[1:] = t.reshape(-1).cuda()
        return wide[1:].view(t.shape)
    want, after, lim, _ = po.conv(c["rows"], c["weight"], c["bias"], c["pool"], c["strides"],
                                  width, c["slots"], c["P"])
    lim = lim + (want.abs() + lim) * po.half_step(BF16) + po.tiny(BF16)
    for moved in ("rows", "weight", "bias", "pool", "outs"):
        t = {k: off(c[k]) if k == moved else c[k].cuda() for k in ("rows", "weight", "bias", "pool")}
        outs = [torch.zeros(3, T, n, dtype=BF16) for n in (16, 8, 8)]
        outs = [off(o) if moved == "outs" else o.cuda() for o in outs]
        ssu.ssu_conv_prefill(t["rows"], t["weight"], t["pool"], *outs, width=width,
                             conv_strides=c["strides"], conv_bias=t["bias"],
                             state_indices=c["slots"].cuda(), P=c["P"])
        torch.cuda.synchronize()
        got = torch.cat([o.cpu() for o in outs], 2).double()
        assert ((got - want).abs() <= lim).all(), moved
        assert same_bits(t["pool"], after), moved


def test_nan_behind_the_rows_is_never_read():
    c = make(3, 4, 70, 16, 8, 4, F32)
    lengths = torch.tensor([0, 1, 33, 69], dtype=torch.int32)
    y, pool = check(c, lengths)
    for b, n in enumerate(lengths.tolist()):
        c["rows"][b, n:] = NAN
    y2, pool2 = check(c, lengths)
    assert same_bits(y, y2) and same_bits(pool, pool2)


def test_pool_past_32_bits():
    """A slot whose taps lie beyond 2^31 elements of the pool."""
    ch, W, P = 5376, 4, 140000
    pool = torch.zeros(P, ch, W - 1, dtype=BF16, device="cuda")
    assert (P - 1) * ch * (W - 1) > 2 ** 31
    g = po.generator(2)
    xbc, w = po.rand(g, 2, 3, ch).to(BF16).cuda(), po.rand(g, ch, W).to(BF16).cuda()
    taps = po.rand(g, ch, W - 1).to(BF16)
    pool[P - 1] = taps.cuda()
    x = torch.empty(2, 3, ch, dtype=BF16, device="cuda")
    slots = torch.tensor([P - 1, 5], dtype=torch.int32, device="cuda")
    kw = dict(width=W, conv_strides=(ch * (W - 1), W - 1, 1), state_indices=slots)
    ssu.ssu_conv_prefill(xbc, w, pool, x, **kw)
    torch.cuda.synchronize()
    first = (torch.cat([taps.cuda(), xbc[0, :1].T], 1).double() * w.double()).sum(1)
    want = first * torch.sigmoid(first)
    assert torch.allclose(x[0, 0].double(), want, rtol=2.0 ** -8, atol=1e-5)
    assert torch.equal(pool[P - 1], xbc[0].T) and torch.equal(pool[5], xbc[1].T)
    ssu.ssu_conv_replay(xbc, pool, torch.tensor([1, 0], dtype=torch.int32, device="cuda"), **kw)
    assert torch.equal(pool[P - 1], torch.cat([xbc[0, 1:], xbc[0, :1]]).T)
    assert int((pool != 0).flatten(1).any(1).sum()) == 2
