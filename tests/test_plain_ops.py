"""CPU checks of the 64-bit restatements the operator tests compare with: identities
between them, the conv oracle, and the distribution that a verified token follows."""

import itertools

import pytest
import torch

import plain_ops as po
from linear_attention_recurrent_selective_b200.workloads import make_case


def test_conv_of_a_prompt_is_the_oracles_window_update(orc):
    """T single tokens through the oracle's fused conv + decode leave the window that the
    prompt form leaves."""
    case = make_case(seed=3, batch=3, P=5, H=2, G=1, Dm=8, N=16, conv=4)
    ch = case.xbc.shape[1]
    xbc = torch.randn(3, 6, ch, generator=po.generator(1))
    _, pool, _, _ = po.conv(xbc, case.conv_w, case.conv_b, case.conv_state, case.conv_strides, 4,
                            case.state_indices, case.P)
    step = case.conv_state
    for t in range(6):
        case.xbc, case.conv_state = xbc[:, t].contiguous(), step
        _, _, step, _ = orc.conv_decode_case(case)
    assert torch.equal(pool, step)


@pytest.mark.parametrize("width", [1, 2, 4, 7])
def test_conv_over_a_chain_tree_is_the_prompt_form(width):
    g = po.generator(width)
    xbc, w = po.rand(g, 2, 9, 5), po.rand(g, 5, width)
    pool = po.rand(g, 3 * 5 * max(width - 1, 1))
    strides = (5 * (width - 1), width - 1, 1)
    chain = torch.arange(-1, 8).expand(2, 9)
    y, after, _, f = po.conv(xbc, w, None, pool, strides, width, None, 3, update=False)
    yt, _, _, ft = po.conv(xbc, w, None, pool, strides, width, None, 3, parents=chain)
    assert f == ft == 0 and torch.allclose(y, yt, rtol=1e-14, atol=0) and torch.equal(after, pool)


@pytest.mark.parametrize("width", [2, 4, 7])
def test_commit_of_k_tokens_is_a_prompt_of_k(width):
    g = po.generator(width)
    xbc, pool = po.rand(g, 4, 6, 3), po.rand(g, 4 * 3 * (width - 1))
    strides = (3 * (width - 1), 1, 3)
    acc = torch.tensor([0, 1, 4, 6], dtype=torch.int32)
    _, want, _, _ = po.conv(xbc, torch.ones(3, width), None, pool, strides, width, None, 4, acc)
    got, _ = po.conv_replay(xbc, pool, strides, width, None, 4, acc)
    same, _ = po.conv_replay(xbc, pool, strides, width, None, 4, acc,
                             torch.arange(6).expand(4, 6))
    assert torch.equal(got, want) and torch.equal(same, want)


def test_scan_of_a_prompt_is_its_tokens_one_by_one():
    g = po.generator(5)
    x, dt, z = po.rand(g, 2, 4, 6), po.rand(g, 2, 4, 6), po.rand(g, 2, 4, 6)
    A = -torch.rand(6, 8, generator=g)
    B, C, pool = po.rand(g, 2, 4, 3, 8), po.rand(g, 2, 4, 3, 8), po.rand(g, 2, 6, 8)
    out, state, _, _, _ = po.scan(x, dt, A, B, C, pool, None, z=z)
    step = pool.double()
    for t in range(4):
        s = slice(t, t + 1)
        o, step, _, _, _ = po.scan(x[:, s], dt[:, s], A, B[:, s], C[:, s], step, None, z=z[:, s])
        assert torch.allclose(o[:, 0], out[:, t], rtol=1e-13, atol=1e-13)
    assert torch.allclose(step, state, rtol=1e-13, atol=1e-13)


def test_scan_closed_forms():
    """dt = 0 keeps the state; B = 0 is pure decay exp(A sum dt)."""
    g = po.generator(6)
    x, A = po.rand(g, 1, 5, 4), -torch.rand(4, 8, generator=g)
    B, C, pool = po.rand(g, 1, 5, 1, 8), po.rand(g, 1, 5, 1, 8), po.rand(g, 1, 4, 8)
    zero = torch.zeros(1, 5, 4)
    _, state, _, _, _ = po.scan(x, zero, A, B, C, pool, None, softplus=False)
    assert torch.equal(state, pool.double())
    dt = torch.rand(1, 5, 4, generator=g)
    _, state, _, _, _ = po.scan(x, dt, A, 0 * B, C, pool, None, softplus=False)
    want = pool.double() * torch.exp(A.double() * dt.double().sum(1)[0][:, None])
    assert torch.allclose(state, want, rtol=1e-12)


def _grid(n):
    return [(i + 0.5) / n for i in range(n)]


def test_chain_verification_follows_the_target():
    """Over a fine grid of uniforms and every drafted token weighted by q, the token at the
    first position is distributed as p."""
    p = torch.tensor([[[0.5, 0.2, 0.3, 0.0], [0.1, 0.2, 0.3, 0.4]]])
    q = torch.tensor([[[0.25, 0.5, 0.125, 0.125]]])
    n, got = 60, [0.0] * 4
    for x, u, us in itertools.product(range(4), _grid(n), _grid(n)):
        acc, nxt, _, _ = po.verify(torch.tensor([[0, x]]), p, torch.tensor([[u, 0.0]]),
                                   torch.tensor([us]), q=q)
        got[x if acc[0] == 2 else nxt[0]] += float(q[0, 0, x]) / (n * n)
    assert all(abs(a - float(b)) < 2 / n for a, b in zip(got, p[0, 0]))


def test_tree_verification_follows_the_target():
    """A root with three children (two of one token): the next token is distributed as p."""
    p = torch.tensor([[0.5, 0.2, 0.2, 0.1]]).expand(1, 4, 4)
    n, got = 200, [0.0] * 4
    tok, par = torch.tensor([[0, 2, 1, 2]]), torch.tensor([[-1, 0, 0, 0]])
    for u, us in itertools.product(_grid(n), _grid(n)):
        acc, nxt, nodes, _ = po.verify(tok, p, torch.full((1, 4), u), torch.tensor([us]),
                                       parents=par, most=2)
        got[int(tok[0, nodes[0][1]]) if acc[0] == 2 else nxt[0]] += 1 / (n * n)
    assert all(abs(a - float(b)) < 3 / n for a, b in zip(got, p[0, 0]))
