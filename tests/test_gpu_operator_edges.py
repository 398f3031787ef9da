"""GPU tests of the calls at the edges of the convolution, scan and verification operators."""

import ctypes

import pytest
import torch

import plain_ops as po
import test_gpu_scan as ts
from linear_attention_recurrent_selective_b200 import ssu
from parity import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
DEV = dict(device="cuda")


# ---------------------------------------------------------------- empty lists of nodes

def test_a_commit_of_an_empty_list_of_nodes_takes_nothing():
    """accepted_node_ids of no columns bounds every length to zero."""
    xbc, pool = torch.randn(2, 5, 8, **DEV), torch.randn(2, 8, 3, **DEV)
    before, err = pool.clone(), torch.zeros(1, dtype=I32, **DEV)
    acc, none = torch.tensor([2, 0], dtype=I32, **DEV), torch.empty(2, 0, dtype=I32, **DEV)
    ssu.ssu_conv_replay(xbc, pool, acc, width=4, conv_strides=(24, 3, 1), accepted_node_ids=none,
                        err_flags=err)
    assert same_bits(pool, before) and int(err.item()) == ssu.FLAG_ACCEPTED_RANGE


def test_a_verification_into_an_empty_list_of_nodes_is_refused():
    p = torch.softmax(torch.randn(2, 3, 40, **DEV), -1)
    tok, par = torch.zeros(2, 3, dtype=I32, **DEV), torch.full((2, 3), -1, dtype=I32, **DEV)
    acc, nxt = torch.zeros(2, dtype=I32, **DEV), torch.zeros(2, dtype=I32, **DEV)
    with pytest.raises(ssu.SSUError):
        ssu.spec_verify(tok, p, torch.rand(2, 3, **DEV), torch.rand(2, **DEV), acc, nxt,
                        parent_ids=par, accepted_node_ids=torch.empty(2, 0, dtype=I32, **DEV))


def test_a_replay_of_an_empty_list_of_nodes_takes_nothing():
    b, T, H, G, Dm, N = 2, 3, 2, 1, 8, 16
    pool = torch.randn(b, H, Dm, N, **DEV)
    stash = (torch.rand(b, T, H, **DEV), torch.randn(b, T, H, Dm, **DEV),
             torch.randn(b, T, G, N, **DEV), torch.rand(b, T, H, **DEV))
    acc, none = torch.tensor([2, 0], dtype=I32, **DEV), torch.empty(b, 0, dtype=I32, **DEV)
    for layers in (False, True):
        got, err = pool.clone(), torch.zeros(1, dtype=I32, **DEV)
        if layers:
            table = ssu.replay_layer_table([(got, stash)])
            ssu.ssu_replay_layers(table, 1, got, stash, acc, accepted_node_ids=none, err_flags=err)
        else:
            ssu.ssu_replay(got, stash, acc, accepted_node_ids=none, err_flags=err)
        assert same_bits(got, pool) and int(err.item()) == ssu.FLAG_ACCEPTED_RANGE


# ---------------------------------------------------------------- inputs that overflow

@pytest.mark.parametrize("T,ch,N,batch", [(9, 40, 16, 2), (300, 16, 16, 2), (1100, 16, 64, 1),
                                          (9, 285, 64, 40)])
def test_an_infinite_input_without_a_skip_connection(T, ch, N, batch):
    """Without D the output is the sum of states alone: all of one sign, it is infinite."""
    c = ts.make(T, batch, T, ch, 1, N, F32, z=False, D=False, bias=False, positive=True)
    for k in ("B", "C", "x"):
        c[k] = (c[k][0].abs() + 0.1, c[k][1])
    c["dt"] = (c["dt"][0] + 0.01, c["dt"][1])
    c["A"], c["pool"] = c["A"] * 1e-3, c["pool"].abs()
    at = T // 2
    c["x"][0][:, at, ::3] = float("inf")
    o, pool, _ = ts.run(c, softplus=False)
    want = torch.zeros(T, ch, dtype=torch.bool)
    want[at:, ::3] = True
    assert torch.equal(o == float("inf"), want.expand(batch, T, ch))
    assert not torch.isnan(o).any() and not torch.isnan(pool).any()
    c["x"] = (c["x"][0][:, at:], c["x"][1])
    o, _, _ = ts.run_decode(c, softplus=False)
    assert torch.equal(o == float("inf"), want[at].expand(batch, ch)) and not torch.isnan(o).any()


# ---------------------------------------------------------------- gates far below zero

def silu_bound(v, dtype):
    """v sigmoid(v) in 64 bits and how far the kernels may be off: a few fp32 steps and those of
    the exponential's rounded argument, and the output's rounding. The arithmetic of 16-bit
    outputs has no 1 / (1 + e^-v) below 2^-126, where v is beyond -88 and the result 2^-119."""
    v = v.double()
    want = v * torch.sigmoid(v)
    lim = want.abs() * (8 + 2 * v.abs()) * po.U
    lim = lim + (want.abs() + lim) * po.half_step(dtype) + po.tiny(dtype)
    return want, lim + (0.0 if dtype == F32 else 2.0 ** -119)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T", [1, 5, 32])
def test_silu_over_its_whole_range(dtype, T):
    """From gates of -110, whose outputs are below the smallest normal number, to 110, and of
    every size around zero."""
    ch = 64
    v = torch.cat([torch.linspace(-110, 110, T * ch // 2),
                   torch.logspace(-36, 2, T * ch - T * ch // 2) * -1.0]).view(1, T, ch).to(dtype)
    w = torch.tensor([0.0, 1.0]).expand(ch, 2).to(dtype).contiguous()
    x = torch.empty(1, T, ch, dtype=dtype, **DEV)
    ssu.ssu_conv_prefill(v.cuda(), w.cuda(), torch.zeros(1, ch, 1, dtype=dtype, **DEV), x, width=2,
                         conv_strides=(ch, 1, 1))
    want, lim = silu_bound(v, dtype)
    bad = (x.cpu().double() - want).abs() > lim
    assert not bad.any(), (v[bad][:4].tolist(), x.cpu()[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_gates_over_their_whole_range(dtype):
    """A state and inputs of zero but for x, and D = 1: the output is x silu(z)."""
    T, ch, N = 8, 64, 16
    z = torch.linspace(-110, 110, T * ch).view(1, T, ch).to(dtype).cuda()
    one, none = torch.ones_like(z), torch.zeros(1, T, 1, N, dtype=dtype, **DEV)
    A, D = -torch.ones(ch, N, **DEV), torch.ones(ch, **DEV)
    want, lim = silu_bound(z.cpu(), dtype)
    out = torch.empty_like(z)
    ssu.scan_prefill(one, one, A, none, none, torch.zeros(1, ch, N, **DEV), out, D=D, z=z)
    assert ((out.cpu().double() - want).abs() <= lim).all()
    for t in range(T):
        y = torch.empty(1, ch, dtype=dtype, **DEV)
        ssu.scan_decode(one[:, t], one[:, t], A, none[:, t], none[:, t],
                        torch.zeros(1, ch, N, **DEV), y, D=D, z=z[:, t])
        assert ((y.cpu().double() - want[:, t]).abs() <= lim[:, t]).all()


# ---------------------------------------------------------------- the binding

def test_launches_run_without_the_interpreter_lock():
    """A launch into a full queue waits for the device: the marshalled entry points are called
    as ctypes calls them, with the lock released (in place of the entry point here: the
    interpreter's own question whether this thread holds it)."""
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    assert ctypes.pythonapi.PyGILState_Check() == 1
    native = ssu._load_marshal()
    x, B = torch.zeros(2, 3, 8, **DEV), torch.zeros(2, 3, 1, 8, **DEV)
    pool, w = torch.zeros(2, 8, 8, **DEV), torch.zeros(8, 2, **DEV)
    A, i = torch.zeros(8, 8, **DEV), torch.zeros(2, dtype=I32, **DEV)
    p, tok = torch.zeros(2, 3, 9, **DEV), torch.zeros(2, 3, dtype=I32, **DEV)
    no = None
    calls = {
        "ssu_conv_prefill": (x, w, torch.zeros(2, 8, 1, **DEV), x, no, no, no, no, no, no, no,
                             2, 8, 1, 1, True, True, no, no),
        "ssu_conv_replay": (x, torch.zeros(2, 8, 1, **DEV), i, no, no, no, 2, 8, 1, 1, no, no),
        "scan_prefill": (x, x, A, B, B, pool, x, no, no, no, no, no, True, no, no, no, no, True),
        "scan_decode": (x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], pool, x[:, 0].clone(), no,
                        no, no, no, no, True, no, no, no),
        "spec_verify": (tok, p, torch.zeros(2, 3, **DEV), torch.zeros(2, **DEV), i, i, no, no, no,
                        no, no, no, no),
    }
    for name, args in calls.items():
        assert getattr(native, name)(held, None, *args) == 0, name


# ---------------------------------------------------------------- forms of large calls

@pytest.mark.parametrize("ch,G", [(285, 3), (288, 3), (301, 1)])
@pytest.mark.parametrize("N,xdt", [(64, BF16), (128, F32), (256, F16)])
def test_many_rows_of_many_states(N, ch, G, xdt):
    """64 states and more with rows enough for two channels a lane: odd channels, groups and
    more ragged rows than are ordered by length, padding and empty rows among them."""
    b, T = 40, 19
    order = torch.randperm(b + 2, generator=po.generator(N))[:b].tolist()
    order[5], order[17] = -1, b + 2
    c = ts.make(N + ch, b, T, ch, G, N, xdt, slots=order)
    lengths = torch.randint(0, T + 1, (b,), generator=po.generator(ch)).to(I32)
    lengths[:3] = torch.tensor([0, T, 1])
    ts.check(c, lengths)
    ts.check(c, lengths, out=False)


def test_more_ragged_rows_than_are_ordered():
    c = ts.make(33, 40, 35, 24, 1, 16, BF16)
    ts.check(c, torch.randint(0, 36, (40,), generator=po.generator(2)).to(I32))


@pytest.mark.parametrize("N", [128, 256])
@pytest.mark.parametrize("ch,G", [(1, 1), (34, 2)])
def test_one_long_row_of_many_states(N, ch, G):
    """One row over as many CTAs as a cluster holds."""
    c = ts.make(N + ch, 1, 3000, ch, G, N, BF16)
    c["A"] = c["A"] * 0.05
    ts.check(c)
    ts.check(c, torch.tensor([2049], dtype=I32), out=False)


# ---------------------------------------------------------------- slots past 32 bits

def test_single_tokens_of_slots_past_32_bits():
    """Outputs and states of one token whose slot lies beyond 2^31 elements of the pool."""
    ch, N, P = 5120, 16, 27000
    assert (P - 1) * ch * N > 2 ** 31
    c = ts.make(15, 2, 1, ch, 1, N, BF16, sdt=BF16)
    small = c["pool"].view(c["P"], ch, N)
    slots, far = [int(s) for s in c["slots"]], [P - 1, 7]
    pool = torch.zeros(P, ch, N, dtype=BF16, **DEV)
    for f, s in zip(far, slots):
        pool[f] = small[s].cuda()
    want, state, lim, slim, _ = ts.plain_decode(c)
    one = lambda k: ts.cut(c[k], 1)[:, 0].contiguous()  # noqa: E731
    out = torch.empty(2, ch, dtype=BF16, **DEV)
    ssu.scan_decode(one("x"), one("dt"), c["A"].cuda(), one("B"), one("C"), pool, out,
                    D=c["D"].cuda(), z=one("z"), dt_bias=c["bias"].cuda(),
                    state_indices=torch.tensor(far, dtype=I32, **DEV))
    ts.near(out.cpu(), want, lim, BF16, "out")
    ts.near(pool[far].cpu(), state[slots], slim[slots], BF16, "state")
    assert int((pool != 0).flatten(1).any(1).sum()) == 2
