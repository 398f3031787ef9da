"""GPU parity of spec_verify with its 64-bit restatement (whole numbers: equal), and a run of
the speculative operators together, as a serving loop calls them."""

import pytest
import torch

import plain_ops as po
from linear_attention_recurrent_selective_b200 import ssu
from parity import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


def probs(g, *shape, spread=3.0):
    return torch.softmax(spread * po.rand(g, *shape), -1)


def chain(seed, b, T, V, dtype=F32, draft=True):
    g = po.generator(seed)
    p = probs(g, b, T, V)
    q = torch.softmax(torch.log(p[:, :-1] + 1e-9) + po.rand(g, b, T - 1, V), -1)
    tok = torch.randint(0, V, (b, T), generator=g)
    if T > 1:
        tok[:, 1:] = torch.multinomial(q.flatten(0, 1), 1, generator=g).view(b, T - 1)
    return dict(tokens=tok.int(), p=p.to(dtype), q=q.to(dtype) if draft else None,
                u=torch.rand(b, T, generator=g), us=torch.rand(b, generator=g), parents=None)


def tree(seed, b, T, V, dtype=F32, roots=False):
    g = po.generator(seed)
    p = probs(g, b, T, V)
    par = torch.full((b, T), -1, dtype=I32)
    for i in range(1, T):
        par[:, i] = (torch.rand(b, generator=g) * i).int().clamp_max(i - 1)
        if roots:
            par[torch.rand(b, generator=g) < 0.2, i] = -1
    tok = torch.randint(0, V, (b, T), generator=g)
    rows = p.gather(1, par.long().clamp_min(0)[..., None].expand(-1, -1, V))
    tok[:, 1:] = torch.multinomial(rows.flatten(0, 1), 1, generator=g).view(b, T)[:, 1:]
    return dict(tokens=tok.int(), p=p.to(dtype), q=None, parents=par,
                u=torch.rand(b, T, generator=g), us=torch.rand(b, generator=g))


def run(c, most=None, lengths=None, slots=None, active=None, stride=0, stream=None, shift=0):
    def dev(t, rows=False):
        if t is None or not rows or not stride:
            return None if t is None else t.cuda()
        wide = torch.full((*t.shape[:2], t.shape[2] + stride), float("nan"), dtype=t.dtype)
        wide[..., shift:shift + t.shape[2]] = t
        return wide.cuda()[..., shift:shift + t.shape[2]]
    b, T, V = c["p"].shape
    acc = torch.full((b,), -9, dtype=I32, device="cuda")
    nxt, err = acc.clone(), torch.zeros(1, dtype=I32, device="cuda")
    nodes = None
    if c["parents"] is not None and most:
        nodes = torch.full((b, most), -9, dtype=I32, device="cuda")
    ssu.spec_verify(dev(c["tokens"]), dev(c["p"], 1), dev(c["u"]), dev(c["us"]), acc, nxt,
                    draft_probs=dev(c["q"], 1), parent_ids=dev(c["parents"]),
                    accepted_node_ids=nodes, context_lengths=dev(lengths),
                    state_indices=dev(slots), active_batch=active, err_flags=err, stream=stream)
    torch.cuda.synchronize()
    return (acc.cpu().tolist(), nxt.cpu().tolist(),
            None if nodes is None else nodes.cpu().tolist(), int(err.item()))


def check(c, most=None, lengths=None, slots=None, active=None, stride=0, shift=0):
    acc, nxt, nodes, err = run(c, most, lengths, slots, active, stride, shift=shift)
    wa, wn, wp, flags = po.verify(c["tokens"], c["p"], c["u"], c["us"], q=c["q"],
                                  parents=c["parents"], most=most, lengths=lengths, slots=slots,
                                  active=active)
    keep = lambda v, w: [-9 if x is None else x for x in w]  # noqa: E731
    assert err == flags
    assert acc == keep(acc, wa) and nxt == keep(nxt, wn)
    if nodes is not None:
        assert nodes == [[-9] * most if x is None else x for x in wp]
    return acc, nxt


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 100, 1000, 1024, 4097, 20000])
def test_chains(dtype, draft, V):
    check(chain(V, 9, 5, V, dtype, draft))


@pytest.mark.parametrize("T", [1, 2, 17, 600])
def test_chain_lengths(T):
    c = chain(T, 6, T, 50)
    check(c)
    check(c, lengths=torch.tensor([T, 0, 1, T + 3, -1, max(T - 1, 0)], dtype=I32),
          slots=torch.tensor([0, 4, 2, 1, 3, -1], dtype=I32))


@pytest.mark.parametrize("stride,shift", [(8, 0), (8, 8), (3, 0), (5, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_apart(stride, shift, dtype):
    check(chain(5, 4, 4, 1000, dtype), stride=stride, shift=shift)
    check(tree(5, 4, 9, 1000, dtype), most=9, stride=stride, shift=shift)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,V", [(1, 7), (2, 33), (17, 40), (64, 300), (128, 8), (128, 5000)])
def test_trees(dtype, T, V):
    c = tree(T + V, 6, T, V, dtype, roots=True)
    check(c, most=T)
    check(c)
    check(c, most=2)
    check(c, most=1)
    check(c, most=T + 3, lengths=torch.tensor([T, 1, 0, T - 1, T + 1, -4], dtype=I32),
          slots=torch.tensor([0, -1, 2, 1, 3, 9], dtype=I32), active=5)


def test_shuffled_and_malformed_trees():
    c = tree(3, 5, 6, 20)
    c["parents"] = torch.tensor([[3, 0, 0, -1, 3, 1], [1, 0, 3, 2, 5, 4], [-1, 0, 9, -2, 0, 1],
                                 [0, -1, 1, 1, 1, 1], [5, 5, 5, 5, 5, -1]], dtype=I32)
    c["tokens"][2, 4] = 20                      # outside the vocabulary
    c["tokens"][4] = 7                          # five children with one token
    for seed in range(6):
        c["u"] = torch.rand(5, 6, generator=po.generator(seed)) * 0.4
        check(c, most=6)


def test_masses_that_are_none():
    """Zeros, negatives, NaN and infinities carry no mass; rows without any give -1."""
    c = chain(1, 8, 3, 64)
    p, q = c["p"], c["q"]
    inf, nan = float("inf"), float("nan")
    p[0] = 0.0
    p[1, :, ::2] = nan
    p[2, :, 1::3] = -1.0
    p[3, :, 5:] = inf
    p[4] = q[4, :1].expand(3, 64)               # p = q: a rejection leaves no residual
    q[4] = p[4, :2] * (1 + 2.0 ** -20)          # q above p everywhere
    c["u"][4] = 1.0
    p[5] = 0.0
    p[5, :, 17] = 1.0                           # one token holds everything
    q[6] = nan
    p[7, :, :] = 2.0 ** -149                    # subnormals
    acc, nxt = check(c)
    assert nxt[0] == -1 and nxt[5] in (17,) and 0 <= nxt[4] < 64
    c["q"] = None
    check(c)


def test_uniforms_at_the_ends():
    c = chain(2, 6, 4, 500)
    for u, us in ((0.0, 0.0), (1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24), (1.0, 1.0), (2.0, 5.0),
                  (float("nan"), float("nan")), (-1.0, -1.0)):
        c["u"].fill_(u)
        c["us"].fill_(us)
        check(c)


def test_tokens_outside_the_vocabulary():
    c = chain(3, 3, 4, 30)
    c["tokens"][0, 2], c["tokens"][1, 1], c["tokens"][2, 0] = 30, -1, -5
    c["u"].fill_(0.0)
    check(c)
    c["q"] = None
    check(c)


def test_draws_over_a_large_vocabulary_follow_the_sum():
    """2^17 tokens, 64 rows: every drawn token is where the 64-bit running sum says."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    b, V = 64, 131072
    p = torch.softmax(2 * torch.randn(b, 1, V, generator=g, device="cuda"), -1)
    us = torch.rand(b, generator=g, device="cuda")
    acc = torch.zeros(b, dtype=I32, device="cuda")
    nxt = acc.clone()
    ssu.spec_verify(acc.view(b, 1).clone(), p, us.view(b, 1), us, acc, nxt)
    run_sum = p[:, 0].double().cumsum(1)
    want = (run_sum <= us.double()[:, None] * run_sum[:, -1:]).sum(1)
    assert (acc == 1).all() and torch.equal(nxt.long(), want)


def test_same_call_twice_in_a_graph_and_on_a_stream():
    c = tree(8, 4, 30, 3000)
    want = run(c, most=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert run(c, most=8, stream=s) == want
    t = {k: v.cuda() for k, v in c.items() if v is not None}
    acc, nxt = torch.zeros(4, dtype=I32, device="cuda"), torch.zeros(4, dtype=I32, device="cuda")
    nodes = torch.zeros(4, 8, dtype=I32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ssu.spec_verify(t["tokens"], t["p"], t["u"], t["us"], acc, nxt, parent_ids=t["parents"],
                        accepted_node_ids=nodes)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert (acc.tolist(), nxt.tolist(), nodes.tolist()) == want[:3]
    t["u"].copy_(torch.rand(4, 30, generator=po.generator(77)))
    c["u"] = t["u"].cpu()
    graph.replay()
    torch.cuda.synchronize()
    assert (acc.tolist(), nxt.tolist(), nodes.tolist()) == run(c, most=8)[:3]


def test_refusals():
    c = chain(1, 2, 3, 40)
    t = {k: v.cuda() for k, v in c.items() if v is not None}
    acc, nxt = torch.zeros(2, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
    ok = dict(tokens=t["tokens"], target_probs=t["p"], uniforms=t["u"], uniform_sample=t["us"],
              accepted_lengths=acc, next_tokens=nxt, draft_probs=t["q"])
    par = torch.full((2, 3), -1, dtype=I32, device="cuda")
    for kw in (dict(tokens=t["tokens"].long()), dict(target_probs=t["p"].double()),
               dict(uniforms=t["u"][:, :2]), dict(uniform_sample=t["us"][:1]),
               dict(draft_probs=t["q"][:, :1]), dict(draft_probs=t["q"].half()),
               dict(accepted_lengths=acc[:1]), dict(next_tokens=nxt.cpu()),
               dict(target_probs=t["p"].transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            ssu.spec_verify(**{**ok, **kw})
    for kw in (dict(parent_ids=par), dict(accepted_node_ids=par)):
        with pytest.raises(ssu.SSUError):
            ssu.spec_verify(**{**ok, **kw})


def test_no_tokens_are_refused():
    none = dict(dtype=F32, device="cuda")
    acc, nxt = torch.zeros(2, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
    with pytest.raises(ValueError):
        ssu.spec_verify(torch.empty(2, 0, dtype=I32, device="cuda"), torch.empty(2, 0, 40, **none),
                        torch.empty(2, 0, **none), torch.empty(2, **none), acc, nxt)


# ---------------------------------------------------------------- the operators together

def layer(seed, b, P, H, G, Dm, N, W):
    g = po.generator(seed)
    ch = H * Dm + 2 * G * N
    c = dict(ch=ch, w=po.rand(g, ch, W), bias=po.rand(g, ch), A=-torch.rand(H, generator=g),
             D=po.rand(g, H), conv=po.rand(g, P * ch * (W - 1)), pool=po.rand(g, P, H, Dm, N),
             slots=torch.randperm(P, generator=g)[:b].int())
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}, g


@pytest.mark.parametrize("form", ["chain", "tree"])
def test_speculative_step_equals_single_tokens(form):
    """conv -> state update -> verification -> commit of window and state, against the
    accepted tokens decoded one by one with ssu_conv_decode from the same start."""
    b, P, H, G, Dm, N, W, T, V = 3, 5, 4, 1, 16, 32, 4, 7, 50
    c, g = layer(21, b, P, H, G, Dm, N, W)
    strides = (c["ch"] * (W - 1), W - 1, 1)
    xbc, dt = po.rand(g, b, T, c["ch"]).cuda(), torch.rand(b, T, H, generator=g).cuda()
    draft = (tree if form == "tree" else chain)(31, b, T, V)
    draft["u"] *= 0.5                                     # accept some
    par = None if form == "chain" else draft["parents"].cuda()
    f = dict(dtype=F32, device="cuda")
    x, B, C = (torch.empty(b, T, n, **f) for n in (H * Dm, G * N, G * N))
    conv, pool = c["conv"].clone(), c["pool"].clone()
    ssu.ssu_conv_prefill(xbc, c["w"], conv, x, B, C, width=W, conv_strides=strides, P=P,
                         conv_bias=c["bias"], state_indices=c["slots"], parent_ids=par,
                         update_state=False)
    assert same_bits(conv, c["conv"])
    stash = (torch.empty(b, T, H, **f), torch.empty(b, T, H, Dm, **f),
             torch.empty(b, T, G, N, **f), torch.empty(b, T, H, **f))
    out = torch.empty(b, T, H, Dm, **f)
    args = (x.view(b, T, H, Dm), c["A"], B.view(b, T, G, N), C.view(b, T, G, N), dt, pool, out)
    if form == "chain":
        ssu.ssu_prefill(*args, D=c["D"], state_indices=c["slots"], stash=stash)
    else:
        depth = torch.zeros_like(par)
        for i in range(1, T):
            up = par[:, i].long()
            depth[:, i] = torch.where(up >= 0, depth.gather(1, up.clamp_min(0)[:, None])[:, 0] + 1,
                                      0)
        ssu.ssu_ddtree(*args, par, depth, stash, D=c["D"], state_indices=c["slots"])
    acc, nxt = torch.empty(b, dtype=I32, device="cuda"), torch.empty(b, dtype=I32, device="cuda")
    nodes = torch.empty(b, T, dtype=I32, device="cuda") if form == "tree" else None
    t = {k: None if v is None else v.cuda() for k, v in draft.items()}
    ssu.spec_verify(t["tokens"], t["p"], t["u"], t["us"], acc, nxt, draft_probs=t["q"],
                    parent_ids=par, accepted_node_ids=nodes, state_indices=c["slots"])
    ssu.ssu_replay(pool, stash, acc, state_indices=c["slots"], accepted_node_ids=nodes)
    ssu.ssu_conv_replay(xbc, conv, acc, width=W, conv_strides=strides, P=P,
                        state_indices=c["slots"], accepted_node_ids=nodes)
    n = acc.tolist()
    assert max(n) > 1 and min(n) >= 1
    for i in range(b):
        one_pool, one_conv = c["pool"].clone(), c["conv"].clone()
        ids = range(n[i]) if form == "chain" else nodes[i, :n[i]].tolist()
        for j in ids:
            o = torch.empty(1, H, Dm, **f)
            ssu.ssu_conv_decode(xbc[i:i + 1, j].contiguous(), c["w"], one_conv, c["A"],
                                dt[i:i + 1, j].contiguous(), one_pool, o, width=W,
                                conv_strides=strides, nheads=H, ngroups=G, dim=Dm,
                                conv_bias=c["bias"], D=c["D"],
                                state_indices=c["slots"][i:i + 1].contiguous(), P=P)
            assert torch.allclose(o[0], out[i, j], rtol=1e-4, atol=1e-4)
        s = int(c["slots"][i])
        per = strides[0]
        assert same_bits(conv[s * per:(s + 1) * per], one_conv[s * per:(s + 1) * per])
        assert torch.allclose(pool[s], one_pool[s], rtol=1e-5, atol=1e-5)


def test_rows_past_32_bits():
    """Distributions that lie beyond 2^31 elements: a chain's and a tree's last rows."""
    b, T, V = 140, 128, 131072
    assert b * T * V > 2 ** 31
    p = torch.zeros(b, T, V, dtype=F16, device="cuda")
    i = torch.arange(b, device="cuda")
    hot = (i * 911 + 17) % V
    for t in (0, T - 1):
        p[i, t, hot] = 0.75
        p[i, t, (hot + 5) % V] = 0.25
    p[:, 1:T - 1, 3] = 1.0
    tokens = torch.full((b, T), 3, dtype=I32, device="cuda")
    tokens[:, 1] = hot.int()
    u = torch.full((b, T), 0.5, device="cuda")
    us = torch.full((b,), 0.9, device="cuda")
    acc, nxt = torch.zeros(b, dtype=I32, device="cuda"), torch.zeros(b, dtype=I32, device="cuda")
    ssu.spec_verify(tokens, p, u, us, acc, nxt)
    # position 0 takes its token (0.5 < 0.75), positions 1.. token 3 (0.5 < 1): all accepted,
    # and 0.9 of the last row's mass lies on its second token
    low = torch.minimum(hot, (hot + 5) % V)
    want = torch.where(low == hot, (hot + 5) % V, hot)
    assert (acc == T).all() and torch.equal(nxt.long(), want)
    parents = torch.arange(-1, T - 1, dtype=I32, device="cuda").expand(b, T).contiguous()
    nodes = torch.zeros(b, T, dtype=I32, device="cuda")
    ssu.spec_verify(tokens, p, u, us, acc, nxt, parent_ids=parents, accepted_node_ids=nodes)
    assert (acc == T).all() and torch.equal(nxt.long(), want)
    assert torch.equal(nodes, torch.arange(T, dtype=I32, device="cuda").expand(b, T))
