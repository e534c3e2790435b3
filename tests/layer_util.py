"""Helpers for the layer operators' tests: tensors inside guarded buffers, and
the operators in plain 64-bit arithmetic on the CPU."""
import math

import torch

GUARD = 64


class Guarded:
    """A (rows, cols) tensor inside a larger buffer: `pad` elements between its
    rows and a margin at both ends hold `fill`, which has to survive."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0, fill=math.nan, data=None):
        ld = cols + pad
        n = max(0, (rows - 1) * ld + cols) if rows else 0
        self.buf = torch.full((n + 2 * GUARD + shift,), fill, dtype=dtype, device="cuda")
        self.t = self.buf[GUARD + shift:].as_strided((rows, cols), (ld, 1))
        if data is not None:
            self.t.copy_(data)
        self.before = self.buf.clone()
        self.inside = torch.zeros_like(self.buf, dtype=torch.bool)
        self.inside[GUARD + shift:].as_strided((rows, cols), (ld, 1)).fill_(True)

    def check(self, name="", rows=None):
        """Nothing outside the tensor (or its first `rows` rows) was written."""
        inside = self.inside
        if rows is not None:
            inside = torch.zeros_like(inside)
            start = self.t.storage_offset()
            inside[start:].as_strided((rows, self.t.shape[1]), self.t.stride()).fill_(True)
        bits = {4: torch.int32, 2: torch.int16}[self.buf.element_size()]
        now, was = self.buf.view(bits), self.before.view(bits)
        assert torch.equal(now[~inside], was[~inside]), "%s: written outside" % name


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    z = z.clone().requires_grad_(True)
    act64(z, act).sum().backward()
    return z.grad


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def weight(gen, lead, k, n, order, dtype, integer=False, pad=0, scale=1.0):
    """A (..., k, n) weight in the order asked for, rows padded with NaN."""
    rows, cols = (k, n) if order == "kn" else (n, k)
    data = ints(gen, *lead, rows, cols) if integer else \
        torch.randn(*lead, rows, cols, generator=gen) * scale
    buf = torch.full((*lead, rows, cols + pad), math.nan, dtype=dtype, device="cuda")
    w = buf[..., :cols]
    w.copy_(data.to(dtype))
    return w if order == "kn" else w.transpose(-1, -2)


def ints(gen, *shape, hi=3):
    return torch.randint(-hi, hi + 1, shape, generator=gen).float()


def plan64(experts, E):
    """offsets, tokens, slots of choices (m, top), in plain Python."""
    m, top = experts.shape
    rows, slots = [], [[-1] * top for _ in range(m)]
    offsets = [0]
    for e in range(E):
        for t in range(m):
            for j in range(top):
                if int(experts[t, j]) == e:
                    slots[t][j] = len(rows)
                    rows.append(t)
        offsets.append(len(rows))
    return offsets, rows, slots


def route64(logits, lowest, top, bias=None, score="softmax", groups=1, top_groups=1, renorm=True,
            scale=1.0):
    """Routing of one call in plain Python floats (64 bits): experts, weights."""
    m, E = logits.shape
    size = E // groups
    out_e, out_w = [], []
    for t in range(m):
        l = [float(x) for x in logits[t]]
        live = [x > lowest for x in l]
        if score == "softmax":
            top_l = max([x for x, a in zip(l, live) if a], default=0.0)
            ex = [(1.0 if x == top_l else math.exp(x - top_l)) if a else 0.0
                  for x, a in zip(l, live)]
            tot = sum(ex)
            s = [x / tot if tot > 0 else 0.0 for x in ex]
        else:
            s = [(1 / (1 + math.exp(-x)) if x > -700 else 0.0) if a else 0.0
                 for x, a in zip(l, live)]
        key = list(l) if groups == 1 and bias is None else list(s)
        if bias is not None:
            key = [x + float(b) for x, b in zip(key, bias)]
        live = [a and x > -math.inf for a, x in zip(live, key)]
        if top_groups < groups:
            sums = []
            for g in range(groups):
                ks = sorted([key[e] for e in range(g * size, (g + 1) * size) if live[e]],
                            reverse=True)
                sums.append(sum(ks[:2]) if ks else -math.inf)
            best = sorted([g for g in range(groups) if sums[g] > -math.inf],
                          key=lambda g: (-sums[g], g))[:top_groups]
            live = [a and e // size in best for e, a in enumerate(live)]
        order = sorted([e for e in range(E) if live[e]], key=lambda e: (-key[e], e))[:top]
        w = [s[e] for e in order]
        if renorm:
            tot = sum(w)
            w = [x / tot if tot > 0 else 0.0 for x in w]
        out_e.append(order + [-1] * (top - len(order)))
        out_w.append([x * scale for x in w] + [0.0] * (top - len(order)))
    return torch.tensor(out_e, dtype=torch.int32).reshape(m, top), \
        torch.tensor(out_w, dtype=torch.float64).reshape(m, top)
