"""Measured cases of the operators around the state update: the short causal convolution
over prompts and draft trees with the commit of its windows, the selective scan with a
decay for every channel and state, and the verification of drafted tokens.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits,
64 where 32 would lose what matters) or, with ``own`` set, by the package's entry points.

The operators, for a batch row b whose slot is s:

  conv          v[t,c] = sum_k w[c,k] in[t - (W-1) + k, c] + bias[c], out = v * sigmoid(v);
                in[t < 0] is the slot's window of W-1 raw inputs (oldest first), which
                becomes the last W-1 inputs of window ++ tokens. Over a draft tree in[t-1],
                in[t-2], ... are node t's ancestors and then the window, which is only read.
  conv_replay   the window becomes the last W-1 of window ++ accepted tokens (or nodes).
  scan_prefill  dt = softplus(dt + bias); h[d,n] = exp(dt A[d,n]) h[d,n] + dt x[d] B[n];
                out[d] = (sum_n h[d,n] C[n] + D[d] x[d]) * silu(z[d]), token after token.
  scan_decode   the same for one token of every row.
  verify        chain: drafted token x at position t is accepted while u q(x) < p(x); then
                one token of max(p - q, 0) (of p when all were accepted) by inverse CDF.
                tree: at a node the first child (in node order) whose running sum of p
                exceeds u is accepted; where none is, one token of p without the children's.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- cases

def _conv(name, **kw):
    c = dict(op="conv", batch=1, tokens=1, x_dim=5120, bc_dim=128, width=4, dtype="bf16",
             layout="channel", tree=False, ragged=False, slots=8)
    c.update(kw)
    return dict(c, name=name) if name else c


def _commit(name, **kw):
    c = dict(op="conv_replay", batch=64, tokens=5, conv_dim=5376, width=4, dtype="bf16",
             layout="channel", tree=False, slots=128)
    c.update(kw)
    return dict(c, name=name) if name else c


def _scan(name, op, **kw):
    c = dict(op=op, batch=1, tokens=1, channels=5120, groups=1, dstate=16, dtype="bf16",
             state="f32", gate=True, ragged=False, slots=8)
    c.update(kw)
    return dict(c, name=name) if name else c


def _verify(name, **kw):
    c = dict(op="verify", batch=1, tokens=5, vocab=32768, dtype="f32", draft=True, tree=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a batch of ragged prompts through one layer's convolution (80 heads of 64, one
        # group of 128 states), the channels a slice of the projected rows
        _conv("conv_prompt_b16_t512", batch=16, tokens=512, ragged=True, slots=32),
        # one token of each of 256 sequences: the windows are most of the traffic
        _conv("conv_token_b256", batch=256, tokens=1, slots=512),
        # draft trees of 128 nodes, each node convolved over its own ancestors
        _conv("conv_tree_b16_n128", batch=16, tokens=128, tree=True, dtype="f16",
              layout="tap", slots=32),
        # the accepted part of a five-token draft enters the windows: a launch-bound call
        _commit("conv_commit_b64_t5"),
        # accepted tree paths, windows of an odd number of channels
        _commit("conv_commit_tree_odd", batch=33, tokens=63, conv_dim=1337, width=3,
                dtype="f32", layout="tap", tree=True, slots=40),
        # ragged prompts through one layer's scan
        _scan("scan_prompt_b16_t512", "scan_prefill", batch=16, tokens=512, ragged=True,
              slots=32),
        # one long prompt, few channels, odd length: little to spread over the card
        _scan("scan_prompt_b1_t4099", "scan_prefill", batch=1, tokens=4099, channels=1000,
              dtype="f16", gate=False, slots=2),
        # one token of each of 256 sequences: the state is read and written once
        _scan("scan_token_b256", "scan_decode", batch=256, slots=512),
        # one token of a few sequences with a half-precision state: latency
        _scan("scan_token_b3_odd", "scan_decode", batch=3, channels=1111, groups=1, dstate=64,
              dtype="f32", state="f16", slots=5),
        # four drafted tokens a row against a large vocabulary, with the draft's distribution
        _verify("verify_chain_b64", batch=64, tokens=5, vocab=131072),
        # one sequence, tokens drafted without a distribution, odd vocabulary: latency
        _verify("verify_chain_b1_odd", batch=1, tokens=9, vocab=65537, dtype="bf16",
                draft=False),
        # a draft tree of 128 nodes a row
        _verify("verify_tree_b16_n128", batch=16, tokens=128, tree=True, draft=False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    op = rng.choice(["conv", "conv", "conv_replay", "scan_prefill", "scan_prefill",
                     "scan_decode", "verify", "verify"])
    if op == "conv":
        tree = rng.random() < 0.3
        batch = _log(rng, 1, 64 if tree else 256)
        tokens = rng.randint(1, 128) if tree else _log(rng, 1, max(1, 8192 // batch))
        x_dim = _log(rng, 16, 5120)
        bc = _log(rng, 8, 1024) if rng.random() < 0.7 else 0
        if rng.random() < 0.7:
            x_dim, bc = max(8, x_dim // 8 * 8), bc // 8 * 8
        return _conv(None, batch=batch, tokens=tokens, x_dim=x_dim, bc_dim=bc,
                     width=rng.choice([2, 3, 4, 4, 4, 7]), dtype=dtype, tree=tree,
                     layout=rng.choice(["channel", "tap"]), ragged=rng.random() < 0.6,
                     slots=batch + rng.randint(0, 9))
    if op == "conv_replay":
        batch = _log(rng, 1, 256)
        return _commit(None, batch=batch, tokens=rng.randint(1, 64), conv_dim=_log(rng, 16, 5376),
                       width=rng.choice([2, 3, 4, 4, 7]), dtype=dtype, tree=rng.random() < 0.5,
                       layout=rng.choice(["channel", "tap"]), slots=batch + rng.randint(0, 9))
    if op == "scan_prefill":
        batch, n = _log(rng, 1, 32), rng.choice([8, 16, 16, 16, 32, 64, 128])
        channels = _log(rng, 16, 5120) * rng.choice([1, 1, 1, 2])
        if rng.random() < 0.7:
            channels = max(16, channels // 16 * 16)
        most = max(2, min(4099, (1 << 28) // (batch * channels * n)))
        groups = 2 if channels % 2 == 0 and rng.random() < 0.3 else 1
        return _scan(None, op, batch=batch, tokens=_log(rng, 1, most), channels=channels,
                     groups=groups, dstate=n, dtype=dtype, state=rng.choice(["f32", "f32", dtype]),
                     gate=rng.random() < 0.7, ragged=rng.random() < 0.5,
                     slots=batch + rng.randint(0, 5))
    if op == "scan_decode":
        batch, n = _log(rng, 1, 256), rng.choice([8, 16, 16, 16, 32, 64, 128, 256])
        channels = max(16, min(_log(rng, 16, 10240), (1 << 25) // (batch * n)))
        groups = 2 if channels % 2 == 0 and rng.random() < 0.3 else 1
        return _scan(None, op, batch=batch, channels=channels, groups=groups, dstate=n,
                     dtype=dtype, state=rng.choice(["f32", "f32", dtype]),
                     gate=rng.random() < 0.7, slots=batch + rng.randint(0, 9))
    tree = rng.random() < 0.4
    batch = _log(rng, 1, 64)
    vocab = _log(rng, 32, 262144)
    tokens = rng.randint(2, 128) if tree else rng.randint(1, 17)
    tokens = max(2, min(tokens, (1 << 26) // (batch * vocab)))
    return _verify(None, batch=batch, tokens=tokens, vocab=vocab,
                   dtype=rng.choice(["f32", "f32", dtype]), tree=tree,
                   draft=not tree and rng.random() < 0.6)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _slots(g, case):
    return torch.randperm(case["slots"], generator=g, device="cuda")[:case["batch"]].to(torch.int32)


def _lengths(g, case):
    """Ragged prompt lengths (an empty row now and then), or None: every token."""
    if not case.get("ragged"):
        return None
    return torch.randint(0, case["tokens"] + 1, (case["batch"],), generator=g,
                         device="cuda").to(torch.int32)


def _trees(g, batch, nodes):
    """Parent ids of random recursive trees: node i hangs on one of 0..i-1."""
    u = torch.rand(batch, nodes, generator=g, device="cuda")
    at = torch.arange(nodes, device="cuda")
    parents = (u * at).long().clamp_max((at - 1).clamp_min(0))
    parents[:, 0] = -1
    return parents.to(torch.int32)


def _windows(g, case, channels):
    """The window pool of either layout and its (slot, channel, tap) strides."""
    taps, dt = case["width"] - 1, DTYPES[case["dtype"]]
    if case["layout"] == "channel":
        return _randn(g, case["slots"], channels, taps).to(dt), (channels * taps, taps, 1)
    return _randn(g, case["slots"], taps, channels).to(dt), (channels * taps, 1, channels)


def prepare(case, seed):
    g, b, T = _gen(seed), case["batch"], case["tokens"]
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "conv":
        xd, bc, W = case["x_dim"], case["bc_dim"], case["width"]
        ch = xd + 2 * bc
        # rows of an in-projection: gate | convolved channels | steps
        rows = _randn(g, b, T, xd + ch + 16).to(dt)
        st["xbc"] = rows[..., xd:xd + ch]
        st["weight"] = (_randn(g, ch, W) * 0.5).to(dt)
        st["bias"] = (_randn(g, ch) * 0.1).to(dt)
        st["pool"], st["strides"] = _windows(g, case, ch)
        st["slots"], st["lengths"] = _slots(g, case), _lengths(g, case)
        st["parents"] = _trees(g, b, T) if case["tree"] else None
        zeros = [torch.zeros(b, T, n, dtype=dt, device="cuda") for n in (xd, bc, bc) if n]
        st["out"] = zeros + [None] * (3 - len(zeros))
    elif case["op"] == "conv_replay":
        st["xbc"] = _randn(g, b, T, case["conv_dim"]).to(dt)
        st["pool"], st["strides"] = _windows(g, case, case["conv_dim"])
        st["slots"] = _slots(g, case)
        u = torch.rand(b, generator=g, device="cuda")
        st["accepted"] = (u * (T + 1)).to(torch.int32).clamp_max(T)
        st["nodes"] = None
        if case["tree"]:      # ascending node ids, as on a path away from the root
            pick = torch.rand(b, T, generator=g, device="cuda").argsort(1)
            order = torch.where(torch.arange(T, device="cuda") < st["accepted"][:, None], pick, T)
            nodes = order.sort(1).values
            st["nodes"] = torch.where(nodes < T, nodes, -1).to(torch.int32)
    elif case["op"] in ("scan_prefill", "scan_decode"):
        D, G, N = case["channels"], case["groups"], case["dstate"]
        tok = (b, T) if case["op"] == "scan_prefill" else (b,)
        st["x"] = _randn(g, *tok, D).to(dt)
        # the gate is half of an in-projection's row, B and C the end of another's
        st["z"] = _randn(g, *tok, 2 * D).to(dt)[..., D:] if case["gate"] else None
        rank = max(8, D // 128 * 8)
        low = _randn(g, *tok, rank + 2 * G * N).to(dt)
        st["B"] = low[..., rank:rank + G * N].unflatten(-1, (G, N))
        st["C"] = low[..., rank + G * N:].unflatten(-1, (G, N))
        st["dt"] = (0.5 * _randn(g, *tok, D)).to(dt)
        step = torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3)
        st["dt_bias"] = torch.log(torch.expm1(step.exp()))
        n = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        st["A"] = -n * torch.exp(0.1 * _randn(g, D, N))
        st["D"] = _randn(g, D)
        st["pool"] = _randn(g, case["slots"], D, N).to(DTYPES[case["state"]])
        st["slots"], st["lengths"] = _slots(g, case), _lengths(g, case)
        st["out"] = torch.zeros(*tok, D, dtype=dt, device="cuda")
    else:
        V = case["vocab"]
        logits = 3.0 * _randn(g, b, T, V)
        p = torch.softmax(logits, -1)
        tokens = torch.randint(0, V, (b, T), generator=g, device="cuda")
        st["q"] = st["parents"] = st["nodes"] = None
        if case["tree"]:
            st["parents"] = _trees(g, b, T)
            src = st["parents"].long().clamp_min(0)
            rows = p.gather(1, src[..., None].expand(-1, -1, V))
            drawn = torch.multinomial(rows.flatten(0, 1), 1, generator=g).view(b, T)
            tokens[:, 1:] = drawn[:, 1:]
            st["nodes"] = torch.zeros(b, min(T, 16), dtype=torch.int32, device="cuda")
        elif T > 1:
            q = torch.softmax(logits[:, :-1] + 1.5 * _randn(g, b, T - 1, V), -1)
            tokens[:, 1:] = torch.multinomial(q.flatten(0, 1), 1, generator=g).view(b, T - 1)
            if case["draft"]:
                st["q"] = q.to(dt)
        st["p"], st["tokens"] = p.to(dt), tokens.to(torch.int32)
        st["u"] = torch.rand(b, T, generator=g, device="cuda")
        st["u_sample"] = torch.rand(b, generator=g, device="cuda")
        st["accepted"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        st["next"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

def _old_windows(st, taps):
    """[batch, taps, channels] of the rows' windows, oldest first."""
    rows = st["pool"][st["slots"].long()]
    return rows.transpose(1, 2) if st["case"]["layout"] == "channel" else rows


def _put_windows(st, win):
    st["pool"][st["slots"].long()] = (win.transpose(1, 2) if st["case"]["layout"] == "channel"
                                      else win)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_conv(st):
    c, W, T = st["case"], st["case"]["width"], st["case"]["tokens"]
    old = _old_windows(st, W - 1)
    full = torch.cat([old, st["xbc"]], 1)                      # [b, W-1+T, ch]
    w = st["weight"].float()
    here = torch.arange(T, device="cuda")
    if c["tree"]:
        at = here.expand(c["batch"], T)
        taps = []
        for k in range(W):              # the node, its parent, ... then the window backwards
            taps.append(full.gather(1, (at + W - 1)[..., None].expand(-1, -1, full.shape[2])))
            up = st["parents"].long().gather(1, at.clamp_min(0))
            at = torch.where(at >= 0, up, at - 1)
        v = sum(taps[k].float() * w[:, W - 1 - k] for k in range(W))
    else:
        v = sum(full[:, k:k + T].float() * w[:, k] for k in range(W))
    y = _silu(v + st["bias"].float())
    if st["lengths"] is not None:
        y = torch.where((here < st["lengths"][:, None])[..., None], y, 0.0)
    y = y.to(st["xbc"].dtype)
    xd, bc = c["x_dim"], c["bc_dim"]
    out = [y[..., :xd]] + ([y[..., xd:xd + bc], y[..., xd + bc:]] if bc else [])
    out = [o.contiguous() for o in out]
    if c["tree"]:
        return out
    L = st["lengths"].long() if st["lengths"] is not None else torch.full_like(here[:1], T)
    at = L[:, None] + torch.arange(W - 1, device="cuda")
    at = at.expand(c["batch"], W - 1)
    _put_windows(st, full.gather(1, at[..., None].expand(-1, -1, full.shape[2])))
    return out + [st["pool"]]


def _plain_conv_replay(st):
    W = st["case"]["width"]
    xbc = st["xbc"]
    if st["nodes"] is not None:
        xbc = xbc.gather(1, st["nodes"].long().clamp_min(0)[..., None].expand(-1, -1, xbc.shape[2]))
    full = torch.cat([_old_windows(st, W - 1), xbc], 1)
    at = st["accepted"].long()[:, None] + torch.arange(W - 1, device="cuda")
    _put_windows(st, full.gather(1, at[..., None].expand(-1, -1, full.shape[2])))
    return [st["pool"]]


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp_max(20))))


def _plain_scan(st):
    c = st["case"]
    one = c["op"] == "scan_decode"
    lift = (lambda t: t.unsqueeze(1)) if one else (lambda t: t)
    x, B, C = lift(st["x"]).float(), lift(st["B"]).float(), lift(st["C"]).float()
    T, G = x.shape[1], c["groups"]
    dt = _softplus(lift(st["dt"]).float() + st["dt_bias"])
    if st["lengths"] is not None:       # a step of zero leaves the state as it is
        live = (torch.arange(T, device="cuda") < st["lengths"][:, None])[..., None]
        dt = torch.where(live, dt, 0.0)
    slots = st["slots"].long()
    s = st["pool"][slots].float()
    per = c["channels"] // G
    # [b, T, D, N] at once, so that a token costs one small operation
    decay = torch.exp(dt[..., None] * st["A"])
    states = ((dt * x).unflatten(-1, (G, per))[..., None] * B[..., None, :]).flatten(2, 3)
    for t in range(T):
        s = torch.addcmul(states[:, t], decay[:, t], s, out=states[:, t])
    del decay
    y = (states.unflatten(2, (G, per)) * C[..., None, :]).sum(-1).flatten(2, 3)
    y = y + st["D"] * x
    if st["z"] is not None:
        y = y * _silu(lift(st["z"]).float())
    if st["lengths"] is not None:
        y = torch.where(live, y, 0.0)
    st["pool"][slots] = s.to(st["pool"].dtype)
    y = y.to(st["x"].dtype)
    return [y.squeeze(1) if one else y, st["pool"]]


def _pick(mass, fallback, u):
    """The first token at which the running sum of the masses exceeds u times their total
    (the last with any mass where none does), in 64 bits."""
    mass = torch.where(mass.sum(-1, keepdim=True) > 0, mass, fallback)
    run = mass.cumsum(-1)
    over = (run > u.double()[:, None] * run[:, -1:]) & (mass > 0)
    at = torch.arange(mass.shape[-1], device="cuda")
    first = torch.where(over, at, mass.shape[-1]).amin(-1)
    last = torch.where(mass > 0, at, -1).amax(-1)
    return torch.where(first < mass.shape[-1], first, last).to(torch.int32)


def _plain_chain(st):
    p, q, tok, u = st["p"], st["q"], st["tokens"].long(), st["u"].double()
    b, T, V = p.shape
    rows = torch.arange(b, device="cuda")
    px = p[:, :-1].gather(2, tok[:, 1:, None])[..., 0].double()
    qx = q.gather(2, tok[:, 1:, None])[..., 0].double() if q is not None else 1.0
    ok = u[:, :-1] * qx < px
    n = 1 + ok.long().cumprod(1).sum(1)
    at = n - 1
    left = p[rows, at].double()
    rejected = (n < T)[:, None]
    if T == 1:
        mass = left
    elif q is not None:
        mass = torch.where(rejected, (left - q[rows, at.clamp_max(T - 2)].double()).clamp_min(0),
                           left)
    else:
        drafted = tok[rows, n.clamp_max(T - 1)][:, None]
        mass = torch.where(rejected, left.scatter(1, drafted, 0.0), left)
    return [n.to(torch.int32), _pick(mass, left, st["u_sample"])]


def _plain_tree(st):
    p, tok, par, u = st["p"], st["tokens"].long(), st["parents"].long(), st["u"].double()
    b, T, V = p.shape
    rows, at = torch.arange(b, device="cuda"), torch.arange(T, device="cuda")
    most = st["nodes"].shape[1]
    up = par.clamp_min(0)
    mass = p[rows[:, None], up, tok].double()
    same = (par[:, :, None] == par[:, None, :]) & (par >= 0)[:, :, None]
    before = same & (at[None, :] < at[:, None])                # [node, earlier sibling]
    again = (before & (tok[:, :, None] == tok[:, None, :])).any(2)
    mass = torch.where(again | (par < 0), 0.0, mass)
    run = ((before | (same & torch.eye(T, dtype=torch.bool, device="cuda"))).double()
           * mass[:, None, :]).sum(2)
    over = (u.gather(1, up) < run) & (mass > 0)
    taken = torch.where(over, at, T)
    first = torch.full((b, T), T, device="cuda").scatter_reduce(1, up, taken, "amin")
    # a node is on the path when every edge above it was taken: pointer doubling
    on = (first.gather(1, up) == at) & (par >= 0)
    on[:, 0] = True
    depth, jump = (par >= 0).long(), up
    for _ in range(max(1, (T - 1).bit_length())):
        on = on & on.gather(1, jump)
        depth = depth + depth.gather(1, jump)
        jump = jump.gather(1, jump)
    on = on & (depth < most)
    n = on.sum(1)
    nodes = torch.full((b, most + 1), -1, device="cuda")
    nodes = nodes.scatter(1, torch.where(on, depth, most), at.expand(b, T))[:, :most]
    nodes = torch.where(torch.arange(most, device="cuda") < n[:, None], nodes, -1)
    end = nodes.gather(1, (n - 1)[:, None])
    left = p[rows, end[:, 0]].double()
    drop = torch.where((par == end) & (n < most)[:, None], tok, V)
    rest = torch.cat([left, left[:, :1]], 1).scatter(1, drop, 0.0)[:, :V]
    return [n.to(torch.int32), _pick(rest, left, st["u_sample"]), nodes.to(torch.int32)]


def _plain_verify(st):
    return _plain_tree(st) if st["case"]["tree"] else _plain_chain(st)


# ---------------------------------------------------------------- the package's calls

def _own(st):
    from linear_attention_recurrent_selective_b200 import ssu
    c = st["case"]
    if c["op"] == "conv":
        x, B, C = st["out"]
        ssu.ssu_conv_prefill(st["xbc"], st["weight"], st["pool"], x, B, C, width=c["width"],
                             conv_strides=st["strides"], conv_bias=st["bias"],
                             state_indices=st["slots"], context_lengths=st["lengths"],
                             parent_ids=st["parents"], update_state=not c["tree"])
        out = [o for o in (x, B, C) if o is not None]
        return out if c["tree"] else out + [st["pool"]]
    if c["op"] == "conv_replay":
        ssu.ssu_conv_replay(st["xbc"], st["pool"], st["accepted"], width=c["width"],
                            conv_strides=st["strides"], state_indices=st["slots"],
                            accepted_node_ids=st["nodes"])
        return [st["pool"]]
    if c["op"] == "scan_prefill":
        ssu.scan_prefill(st["x"], st["dt"], st["A"], st["B"], st["C"], st["pool"], st["out"],
                         D=st["D"], z=st["z"], dt_bias=st["dt_bias"],
                         state_indices=st["slots"], context_lengths=st["lengths"])
        return [st["out"], st["pool"]]
    if c["op"] == "scan_decode":
        ssu.scan_decode(st["x"], st["dt"], st["A"], st["B"], st["C"], st["pool"], st["out"],
                        D=st["D"], z=st["z"], dt_bias=st["dt_bias"], state_indices=st["slots"])
        return [st["out"], st["pool"]]
    ssu.spec_verify(st["tokens"], st["p"], st["u"], st["u_sample"], st["accepted"], st["next"],
                    draft_probs=st["q"], parent_ids=st["parents"],
                    accepted_node_ids=st["nodes"])
    return [st["accepted"], st["next"]] + ([st["nodes"]] if c["tree"] else [])


PLAIN = {"conv": _plain_conv, "conv_replay": _plain_conv_replay, "scan_prefill": _plain_scan,
         "scan_decode": _plain_scan, "verify": _plain_verify}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    """Bytes and operations of one pass. Ragged rows are half as long on average; a window
    is read and written once; a verification reads the distributions at the drafted tokens
    and one whole row of p (and of q where a token was rejected, about nine rows in ten)."""
    b, T, e = case["batch"], case["tokens"], SIZE[case["dtype"]]
    n = b * T / 2 if case.get("ragged") else b * T
    if case["op"] == "conv":
        ch, W = case["x_dim"] + 2 * case["bc_dim"], case["width"]
        window = b * ch * (W - 1) * e * (1 if case["tree"] else 2)
        return {"bytes": 2 * n * ch * e + window + ch * (W + 1) * e, "flops": n * ch * (2 * W + 4)}
    if case["op"] == "conv_replay":
        # every row keeps or replaces its W-1 taps: read once, written once
        moved = b * case["conv_dim"] * (case["width"] - 1) * e
        return {"bytes": 2 * moved, "flops": 0}
    if case["op"] in ("scan_prefill", "scan_decode"):
        D, N = case["channels"], case["dstate"]
        token = (3 + (1 if case["gate"] else 0)) * D * e + 2 * case["groups"] * N * e
        state = 2 * b * D * N * SIZE[case["state"]]
        return {"bytes": n * token + state + D * N * 4 + 8 * D, "flops": 7 * n * D * N}
    V = case["vocab"]
    rows = 1.9 if case["draft"] and T > 1 else 1.0
    return {"bytes": b * (rows * V * e + T * (8 + 32)), "flops": 2 * b * V}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_conv(st):
    c, W, T, b = st["case"], st["case"]["width"], st["case"]["tokens"], st["case"]["batch"]
    raw, w = st["xbc"].double(), st["weight"].double()
    win = st["pool"].double()[st["slots"].long()]
    if c["layout"] == "tap":
        win = win.transpose(1, 2)                              # [b, ch, W-1]
    v = st["bias"].double() + raw * w[:, W - 1]
    if c["tree"]:
        for i in range(b):
            par = st["parents"][i].tolist()
            for k in range(1, W):
                src, tap = [], []
                for t in range(T):
                    a, up = t, 0
                    while a >= 0 and up < k:
                        a, up = par[a], up + 1
                    src.append(a)
                    tap.append(W - 1 - (k - up) - 1 if a < 0 else 0)
                s, q = (torch.tensor(z, device="cuda") for z in (src, tap))
                past = torch.where((s >= 0)[:, None], raw[i, s.clamp_min(0)], win[i].T[q])
                v[i] += past * w[:, W - 1 - k]
    else:
        for k in range(1, W):
            m = min(k, T)
            v[:, k:] += raw[:, :T - m] * w[:, W - 1 - k] if T > k else 0.0
            v[:, :m] += win.transpose(1, 2)[:, W - 1 - k:W - 1 - k + m] * w[:, W - 1 - k]
    y = v * torch.sigmoid(v)
    L = [T] * b if st["lengths"] is None else st["lengths"].tolist()
    for i in range(b):
        y[i, L[i]:] = 0
    xd, bc = c["x_dim"], c["bc_dim"]
    out = [y[..., :xd]] + ([y[..., xd:xd + bc], y[..., xd + bc:]] if bc else [])
    return out if c["tree"] else out + [_exact_windows(st, [list(range(n)) for n in L])]


def _exact_windows(st, entered):
    """The pool after row b's tokens entered[b] have passed through its window."""
    c, pool = st["case"], st["pool"].double().clone()
    if c["layout"] == "tap":
        pool = pool.transpose(1, 2).contiguous()
    for i, slot in enumerate(st["slots"].tolist()):
        for t in entered[i][-(c["width"] - 1):]:
            pool[slot] = torch.cat([pool[slot][:, 1:], st["xbc"][i, t].double()[:, None]], 1)
    return pool.transpose(1, 2).contiguous() if c["layout"] == "tap" else pool


def _exact_conv_replay(st):
    acc = st["accepted"].tolist()
    ids = st["nodes"].tolist() if st["nodes"] is not None else [list(range(n)) for n in acc]
    return [_exact_windows(st, [ids[i][:n] for i, n in enumerate(acc)])]


def _exact_scan(st):
    c = st["case"]
    one = c["op"] == "scan_decode"
    D, G = c["channels"], c["groups"]
    group = torch.arange(D, device="cuda") // (D // G)
    A, pool = st["A"].double(), st["pool"].double()
    slots = st["slots"].long()
    h = pool[slots]
    T = 1 if one else c["tokens"]
    out = torch.zeros(c["batch"], T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        at = (lambda v: v.double()) if one else (lambda v: v[:, t].double())
        x = at(st["x"])
        v = at(st["dt"]) + st["dt_bias"].double()
        dt = torch.logaddexp(v, torch.zeros_like(v))
        new = h * torch.exp(dt[..., None] * A) + (dt * x)[..., None] * at(st["B"])[:, group]
        y = torch.einsum("bdn,bdn->bd", new, at(st["C"])[:, group]) + st["D"].double() * x
        if st["z"] is not None:
            z = at(st["z"])
            y = y * z * torch.sigmoid(z)
        if st["lengths"] is not None:
            live = (t < st["lengths"])[:, None]
            y, new = torch.where(live, y, 0.0), torch.where(live[..., None], new, h)
        out[:, t], h = y, new
    pool[slots] = h
    return [out[:, 0] if one else out, pool]


def _exact_pick(mass, fallback, u):
    if not float(mass.sum()) > 0:
        mass = fallback
    run = mass.cumsum(0)
    at = int(torch.searchsorted(run, u * float(run[-1]), right=True))
    return at if at < len(run) else int(mass.nonzero()[-1])


def _exact_verify(st):
    c = st["case"]
    b, T, V = c["batch"], c["tokens"], c["vocab"]
    p = st["p"].cpu().double() if b * T * V < 1 << 22 else st["p"]
    tok, u, us = st["tokens"].tolist(), st["u"].double().tolist(), st["u_sample"].double().tolist()
    accepted, chosen, paths = [], [], []
    for i in range(b):
        if c["tree"]:
            par, path, most = st["parents"][i].tolist(), [0], st["nodes"].shape[1]
            while True:
                row = p[i, path[-1]].double()
                kids = [j for j in range(T) if par[j] == path[-1]]
                if len(path) == most:
                    kids = []
                run, seen, to = 0.0, set(), None
                for j in kids:
                    m = 0.0 if tok[i][j] in seen else float(row[tok[i][j]])
                    seen.add(tok[i][j])
                    run += m
                    if m > 0 and u[i][path[-1]] < run:
                        to = j
                        break
                if to is None:
                    break
                path.append(to)
            left = row.clone()
            left[[tok[i][j] for j in kids]] = 0
            accepted.append(len(path))
            paths.append(path + [-1] * (most - len(path)))
        else:
            t = 0
            while t + 1 < T:
                x = tok[i][t + 1]
                qx = 1.0 if st["q"] is None else float(st["q"][i, t, x])
                if not u[i][t] * qx < float(p[i, t, x]):
                    break
                t += 1
            row = p[i, t].double()
            left = row.clone()
            if t + 1 < T and st["q"] is not None:
                left = (left - st["q"][i, t].to(left.device).double()).clamp_min(0)
            elif t + 1 < T:
                left[tok[i][t + 1]] = 0
            accepted.append(t + 1)
        chosen.append(_exact_pick(left, row, us[i]))
    out = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (accepted, chosen)]
    if c["tree"]:
        out.append(torch.tensor(paths, dtype=torch.int32, device="cuda"))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "conv":
        return _exact_conv(st)
    if case["op"] == "conv_replay":
        return _exact_conv_replay(st)
    if case["op"] in ("scan_prefill", "scan_decode"):
        return _exact_scan(st)
    return _exact_verify(st)
