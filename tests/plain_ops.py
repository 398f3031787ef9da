"""Plain 64-bit restatements of the conv-prefill, window commit, per-channel scan and draft
verification operators (include/ssu.h gives the formulas), written as loops over rows and
tokens on the CPU, with the error bounds that fp32 arithmetic may reach beside them.

A rounding to a type is off by at most ``finfo(type).eps / 2`` of the value."""

import math

import torch

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24                      # fp32: half a step, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the smallest step of the type (subnormals)."""
    return torch.finfo(dtype).tiny * half_step(dtype)


def rand(gen, *shape):
    return torch.randn(*shape, generator=gen)


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def lengths_of(b, T, lengths):
    if lengths is None:
        return [T] * b
    return [max(0, min(T, int(v))) for v in lengths]


# ------------------------------------------------------------------ convolution

def taps_view(pool, P, ch, width, strides):
    """[P, ch, width-1] view of a flat conv pool."""
    return pool.as_strided((P, ch, width - 1), strides)


def conv_inputs(xbc, window, b, t, parents, L, width):
    """[width, ch] float64 inputs of token t of row b, oldest first, or None (malformed)."""
    rows, at = [], t
    for k in range(width):
        if at >= 0:
            rows.append(xbc[b, at].double())
        else:
            rows.append(window[:, width - 1 + at].double())
        if k + 1 < width:
            if at >= 0 and parents is not None:
                up = int(parents[b, at])
                if up < -1 or up >= L:
                    return None
                at = up
            else:
                at -= 1
    return torch.stack(rows[::-1])


def conv(xbc, weight, bias, pool, strides, width, slots, P, lengths=None, parents=None,
         silu=True, update=True, active=None):
    """Returns (y [b, T, ch] with NaN where nothing is written, the pool after, the error
    bound of y before its rounding, flags)."""
    batch, T, ch = xbc.shape
    active = batch if active is None else active
    y = torch.full((batch, T, ch), math.nan, dtype=torch.float64)
    lim = torch.zeros_like(y)
    pool = pool.clone()
    flags = 0
    w = weight.double().T                                          # [width, ch]
    for b in range(active):
        slot = b if slots is None else int(slots[b])
        if slot >= P:
            flags |= 1
            continue
        if slot < 0:
            y[b] = 0
            continue
        if lengths is not None and not 0 <= int(lengths[b]) <= T:
            flags |= 8 if int(lengths[b]) < 0 else 4
        L = lengths_of(batch, T, lengths)[b]
        window = taps_view(pool, P, ch, width, strides)[slot].clone() if width > 1 else None
        for t in range(L):
            ins = conv_inputs(xbc, window, b, t, parents, L, width)
            if ins is None:
                flags |= 64
                y[b, t] = 0
                continue
            v = (w * ins).sum(0)
            mag = (w * ins).abs().sum(0)
            if bias is not None:
                v, mag = v + bias.double(), mag + bias.double().abs()
            # width products and sums in fp32; v * sigmoid(v) has a slope below 1.1
            e = (width + 1) * U * mag
            if silu:
                o = v * torch.sigmoid(v)
                # approximate exponential (its argument rounded: |v| steps) and division
                e = 1.1 * e + o.abs() * (8 + 2 * v.abs()) * U
            else:
                o = v
            y[b, t], lim[b, t] = o, e
        if update and parents is None and width > 1:
            hist = [window[:, k] for k in range(width - 1)] + [xbc[b, t] for t in range(L)]
            new = torch.stack(hist[len(hist) - (width - 1):], 1)
            taps_view(pool, P, ch, width, strides)[slot] = new
    return y, pool, lim, flags


def conv_replay(xbc, pool, strides, width, slots, P, accepted, nodes=None, active=None):
    batch, T, ch = xbc.shape
    active = batch if active is None else active
    pool = pool.clone()
    most = T if nodes is None else nodes.shape[1]
    flags = 0
    for b in range(active):
        slot = b if slots is None else int(slots[b])
        if slot >= P:
            flags |= 1
            continue
        if slot < 0:
            continue
        k = int(accepted[b])
        if not 0 <= k <= most:
            flags |= 8 if k < 0 else 2
        k = max(0, min(most, k))
        ids = list(range(k)) if nodes is None else [int(v) for v in nodes[b, :k]]
        if any(not 0 <= i < T for i in ids):
            flags |= 64
            continue
        if width > 1 and k > 0:
            win = taps_view(pool, P, ch, width, strides)[slot]
            hist = [win[:, j].clone() for j in range(width - 1)] + [xbc[b, i] for i in ids]
            win.copy_(torch.stack(hist[len(hist) - (width - 1):], 1))
    return pool, flags


# ------------------------------------------------------------------ scan

def scan(x, dt, A, B, C, pool, slots, *, D=None, z=None, dt_bias=None, softplus=True,
         lengths=None, update=True, active=None):
    """x [b, T, ch]; pool [P, ch, N]. Returns (out with NaN where nothing is written, state
    of every slot after (float64), the bounds of both before their last rounding, flags)."""
    batch, T, ch = x.shape
    P, _, N = pool.shape
    G = B.shape[2]
    active = batch if active is None else active
    group = torch.arange(ch) // (ch // G)
    out = torch.full((batch, T, ch), math.nan, dtype=torch.float64)
    lim = torch.zeros_like(out)
    state, slim = pool.double().clone(), torch.zeros(P, ch, N, dtype=torch.float64)
    A64, flags = A.double(), 0
    for b in range(active):
        slot = b if slots is None else int(slots[b])
        if slot >= P:
            flags |= 1
            continue
        if slot < 0:
            out[b] = 0
            continue
        if lengths is not None and not 0 <= int(lengths[b]) <= T:
            flags |= 8 if int(lengths[b]) < 0 else 4
        h, e = pool[slot].double(), torch.zeros(ch, N, dtype=torch.float64)
        L = lengths_of(batch, T, lengths)[b]
        for t in range(L):
            xv, v = x[b, t].double(), dt[b, t].double()
            if dt_bias is not None:
                v = v + dt_bias.double()
            s = torch.where(v > 30, v, torch.log1p(torch.exp(v.clamp_max(30)))) if softplus else v
            # the sum's rounding moves softplus by at most |v| U of itself; the series,
            # exponential and division of the kernel add a few steps
            es = (v.abs() + (16 if softplus else 1)) * U
            sA = s[:, None] * A64
            a = torch.exp(sA)
            # the exponent: A * log2(e), its product with s, and s itself; then exp2 (2 ulp)
            ea = sA.abs() * (3 * U + es[:, None]) + 4 * U
            inp = (s * xv)[:, None] * B[b, t].double()[group]
            e = a * e + (a * h).abs() * ea + inp.abs() * (es[:, None] + 3 * U)
            h = a * h + inp
            e = e + h.abs() * U + inp.abs() * U
            Cv = C[b, t].double()[group]
            y = (h * Cv).sum(1)
            ey = (e * Cv.abs()).sum(1) + (N.bit_length() + 4) * U * (h * Cv).abs().sum(1)
            if D is not None:
                y = y + D.double() * xv
                ey = ey + 2 * U * (D.double() * xv).abs() + U * y.abs()
            if z is not None:
                zv = z[b, t].double()
                g = zv * torch.sigmoid(zv)
                ey = ey * g.abs() + (y * g).abs() * (9 + 2 * zv.abs()) * U
                y = y * g
            out[b, t], lim[b, t] = y, ey
        if update and L > 0:
            state[slot], slim[slot] = h, e
    return out, state, lim, slim, flags


# ------------------------------------------------------------------ verification

def mass(v):
    v = float(v)
    return v if 0 < v < math.inf else 0.0


def pick(masses, fallback, us):
    """Index drawn by inverse CDF, or -1 when neither row holds any mass."""
    for row in (masses, fallback):
        total = 0.0
        for m in row:
            total += m
        if total > 0:
            run, last = 0.0, -1
            for i, m in enumerate(row):
                run += m
                if m > 0:
                    last = i
                    if run > us * total:
                        return i
            return last
    return -1


def verify(tokens, p, u, us, *, q=None, parents=None, most=None, lengths=None, slots=None,
           active=None):
    """Returns (accepted, next, nodes [b, most] or None, flags); rows beyond ``active`` None."""
    batch, T, V = p.shape
    active = batch if active is None else active
    cap = T if most is None else most
    acc, nxt, nodes, flags = [None] * batch, [None] * batch, [None] * batch, 0
    for b in range(active):
        pad = slots is not None and int(slots[b]) < 0
        if not pad and lengths is not None and not 0 <= int(lengths[b]) <= T:
            flags |= 8 if int(lengths[b]) < 0 else 4
        L = lengths_of(batch, T, lengths)[b]
        tok = [int(v) for v in tokens[b]]
        path, drop, row, sub = [], set(), None, None
        if pad or L == 0:
            pass
        elif parents is None:
            t = 0
            # every drafted token of the row is looked at, accepted or not
            flags |= 256 if any(not 0 <= x < V for x in tok[1:L]) else 0
            while t + 1 < L:
                x = tok[t + 1]
                if not 0 <= x < V:
                    break
                qx = 1.0 if q is None else mass(q[b, t, x])
                if not float(u[b, t]) * qx < mass(p[b, t, x]):
                    break
                t += 1
            path = list(range(t + 1))
            row = t
            if t + 1 < L:
                if q is None:
                    drop = {tok[t + 1]}
                else:
                    sub = q[b, t]
        else:
            par = [int(v) for v in parents[b, :L]]
            if any(v < -1 or v >= L for v in par):
                flags |= 64
            if any(0 <= par[j] < L and not 0 <= tok[j] < V for j in range(L)):
                flags |= 256
            roots = [j for j in range(L) if par[j] == -1]
            if not roots:
                flags |= 64
            else:
                path = [roots[0]]
                while len(path) < cap:
                    at, run, seen, to = path[-1], 0.0, set(), None
                    for j in range(L):
                        if par[j] != at:
                            continue
                        x = tok[j]
                        m = mass(p[b, at, x]) if 0 <= x < V and x not in seen else 0.0
                        seen.add(x)
                        run += m
                        if m > 0 and float(u[b, at]) < run:
                            to = j
                            break
                    if to is None:
                        break
                    path.append(to)
                row = path[-1]
                if len(path) < cap:
                    drop = {tok[j] for j in range(L) if par[j] == row}
        acc[b] = len(path)
        nodes[b] = path + [-1] * (cap - len(path))
        if not path:
            nxt[b] = -1
            continue
        full = [mass(v) for v in p[b, row]]
        left = [0.0 if i in drop else m for i, m in enumerate(full)]
        if sub is not None:
            left = [max(m - mass(s), 0.0) for m, s in zip(left, sub)]
        nxt[b] = pick(left, full, float(us[b]))
        if nxt[b] < 0:
            flags |= 512
    return acc, nxt, nodes if parents is not None else None, flags
