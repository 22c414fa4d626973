"""Plain 64-bit implementations of the attention step's operators, for the tests (torch on any
device, or Python integers)."""
import math

import torch


def plan(lens, num_new, held, table, free, count, page, tokens):
    """Lists of ints in, the state afterwards out: a sequence at a time, as the definition reads."""
    width, table = len(table[0]) if table else 0, [list(r) for r in table]
    left = min(max(count, 0), len(free))
    cu, kv, now, full = [0], [], [], False
    positions, slots = [0] * tokens, [-1] * tokens
    end = 0  # new tokens so far, whether they have rows or not
    for s, (a, n) in enumerate(zip(lens, num_new)):
        a, n = max(a, 0), max(n, 0)
        mine = -(-a // page) if held is None else max(held[s], 0)
        mine = min(mine, width)
        need = -(-(a + n) // page) if n else 0
        ok = n == 0 or (need <= width and end + n <= tokens and a + n < 2 ** 31)
        more = max(0, need - mine) if ok else 0
        if more:
            full = full or more > left
            ok = not full
            if ok:
                for j in range(mine, need):
                    left -= 1
                    table[s][j] = free[left]
        for j in range(n):
            if end + j < tokens:
                positions[end + j] = min(a + j, 2 ** 31 - 1)
                if ok:
                    slots[end + j] = table[s][(a + j) // page] * page + (a + j) % page
        end += n
        cu.append(min(end, tokens))
        kv.append(a + n if ok else a)
        now.append(max(mine, need) if ok else mine)
    return table, cu, kv, positions, slots, now, left


def rotate(x, positions, inv_freq, axis):
    """x [tokens, heads, dim] -> float64; positions [axes, tokens]; inv_freq, axis: a pair's each."""
    half = len(inv_freq)
    angle = torch.stack([positions[a].double() * f for f, a in zip(inv_freq, axis)], 1)[:, None]
    a, b = x[..., :half].double(), x[..., half:2 * half].double()
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos(),
                      x[..., 2 * half:].double()], -1)


def attend(q, k, v, first, scale=None):
    """q [n, heads, d] at positions first, first + 1, ... over k, v [m, kv_heads, d].

    Returns the result in binary64 and the error that the kernels' roundings may add up to.
    With w the weights and A = sum_j w_j |v_j|:
    * the result's rounding to BF16: 2^-8 |out|;
    * each weight's rounding to BF16 before it multiplies v: 2^-8 A;
    * a score's error: d products summed in FP32, (d + 8) 2^-24 scale sum |q k|, and 2^-24 of
      the exponent's magnitude: as much relative error of a weight, and of their sum: twice it;
    * the sums over m keys in FP32: 2 m 2^-24 A for the weighted values, as much for the weights;
    * 2^-20 for the exponential, the quotient and the joining of parts."""
    n, heads, d = q.shape
    m, group = k.shape[0], heads // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((n, heads, d), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    seen = torch.arange(m, device=q.device)[None] <= first + torch.arange(n, device=q.device)[:, None]
    rows = seen.any(1)
    if m == 0 or not bool(rows.any()):
        return out, tol
    seen = seen[rows]
    for h in range(heads):
        qh, kh, vh = q[rows, h].double(), k[:, h // group].double(), v[:, h // group].double()
        s = (qh @ kh.t()) * scale
        size = (qh.abs() @ kh.abs().t()) * abs(scale)
        s = s.masked_fill(~seen, -math.inf)
        w = torch.softmax(s, 1)
        o, a = w @ vh, w @ vh.abs()
        size = size.masked_fill(~seen, 0.0).amax(1, keepdim=True)
        rel = 2 ** -8 + 2 * (d + 10) * 2 ** -24 * size + 4 * m * 2 ** -24 + 2 ** -20
        out[rows, h] = o
        tol[rows, h] = 2 ** -8 * o.abs() + rel * a * (1 + 2 ** -7)
    return out, tol


def gather(cache, table_row, m):
    """The first m cached rows of a sequence, [m, kv_heads, d]."""
    page = cache.shape[1]
    if m == 0:
        return cache.new_zeros((0, *cache.shape[2:]))
    pages = table_row[: -(-m // page)].long()
    return cache[pages].flatten(0, 1)[:m]


def norm_bound(q, k, v, first, scale=None):
    """The result in binary64 and the root mean square error, summed over all its elements, that the kernels'
    two BF16 roundings may come to.

    The result's rounding is off by at most 2^-8 |out| an element; each weight's by at most 2^-8 of it, with
    signs that v's do not follow, so that the squares add: 2^-16 (|out|^2 + sum_j w_j^2 |v_j|^2).  (Evenly spread
    errors have a third of that mean square; FP32's are a thousandth.)  A tile of keys lost or counted twice is
    off by its share of sum_j w_j v_j, of which this sees one in ten thousand."""
    n, heads, d = q.shape
    m, group = k.shape[0], heads // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, square = torch.zeros((n, heads, d), dtype=torch.float64, device=q.device), 0.0
    hidden = torch.arange(m, device=q.device)[None] > first + torch.arange(n, device=q.device)[:, None]
    for h in range(heads):
        kh, vh = k[:, h // group].double(), v[:, h // group].double()
        w = torch.softmax(((q[:, h].double() @ kh.t()) * scale).masked_fill(hidden, -math.inf), 1)
        out[:, h] = w @ vh
        square += float((w.square() @ vh.square()).sum() + out[:, h].square().sum())
    return out, 2.0 ** -8 * math.sqrt(square)
