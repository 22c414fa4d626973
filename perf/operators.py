"""The operators of the verify step, as they are measured: cases, inputs, plain forms, definitions in 64 bits.

* ``quantize``: BF16 weight -> E4M3 codes with one FP32 scale per 128 x 128 block (load time);
* ``norm``:     residual addition + RMSNorm -> E4M3 activations with one FP32 scale per row and 128 columns;
* ``gemm``:     the product of the two, FP32 accumulation, BF16 or FP32 result;
* ``verify``:   speculative verification of drafted tokens from given uniform numbers.

A case is a dict of plain values whose ``op`` is one of these.  ``run`` computes a case either with elementary
torch operations or, where ``own`` is true, with the framework's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def listed():
    return [
        # load time: the combiner projection, and the full-vocabulary LM head (the largest weight)
        {"name": "quantize fc", "op": "quantize", "n": 5120, "k": 10240},
        {"name": "quantize head", "op": "quantize", "n": 151936, "k": 5120},
        # one decoded token (latency); the input of a down projection, ragged batch, no norm; a long prefill
        {"name": "norm one token", "op": "norm", "m": 1, "k": 5120, "residual": True, "gamma": True},
        {"name": "norm down input", "op": "norm", "m": 333, "k": 17408, "residual": False, "gamma": False},
        {"name": "norm prefill", "op": "norm", "m": 8192, "k": 5120, "residual": True, "gamma": True},
        # one token through the combiner; the LM head over two sequences' positions to verify;
        # an odd batch through an up projection; the prefill product
        {"name": "gemm one token", "op": "gemm", "m": 1, "n": 5120, "k": 10240, "f32": False},
        {"name": "gemm head", "op": "gemm", "m": 10, "n": 151936, "k": 5120, "f32": True},
        {"name": "gemm odd batch", "op": "gemm", "m": 77, "n": 17408, "k": 5120, "f32": False},
        {"name": "gemm prefill", "op": "gemm", "m": 2048, "n": 17408, "k": 5120, "f32": False},
        # one sequence with greedy drafts over the reduced vocabulary (latency); a ragged batch whose drafts come
        # from the reduced-vocabulary head; a full server batch with sampled drafts
        {"name": "verify one", "op": "verify", "batch": 1, "g": 3, "vocab": 32768, "draft_vocab": 0, "bf16": False,
         "ragged": False, "cut": False},
        {"name": "verify reduced", "op": "verify", "batch": 24, "g": 5, "vocab": 151936, "draft_vocab": 32768,
         "bf16": True, "ragged": True, "cut": False},
        {"name": "verify batch", "op": "verify", "batch": 256, "g": 4, "vocab": 151936, "draft_vocab": 151936,
         "bf16": False, "ragged": True, "cut": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "norm", "gemm", "gemm", "gemm", "verify", "verify"])
    while True:
        k = max(16, _log(rng, 64, 17408) // 16 * 16)
        if op == "quantize":
            c = {"op": op, "n": _log(rng, 64, 151936), "k": k}
            if c["n"] * k <= 151936 * 5120:
                return c
        elif op == "norm":
            gamma = rng.random() < 0.7
            c = {"op": op, "m": _log(rng, 1, 8192), "k": k, "residual": rng.random() < 0.7, "gamma": gamma}
            if c["m"] * k <= 8192 * 5120:
                return c
        elif op == "gemm":
            c = {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, 151936), "k": k, "f32": rng.random() < 0.4}
            if c["m"] * c["n"] * k <= 2048 * 17408 * 5120 and c["n"] * k <= 151936 * 5120 and \
                    c["m"] * c["n"] <= 2048 * 17408:
                return c
        else:
            vocab = _log(rng, 500, 151936)
            kind = rng.random()
            c = {"op": op, "batch": _log(rng, 1, 256), "g": rng.randint(0, 8), "vocab": vocab,
                 "draft_vocab": 0 if kind < 0.3 else vocab if kind < 0.7 else max(1, vocab * 2 // 9),
                 "bf16": rng.random() < 0.4, "ragged": rng.random() < 0.6, "cut": rng.random() < 0.5}
            if c["batch"] * (c["g"] + 1) * vocab <= 256 * 5 * 151936:
                return c


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _weight(g, n, k):
    """Rows of N(0, 0.02), some of them eight times larger, as trained projections have them."""
    w = _randn(g, n, k).mul_(0.02)
    w[torch.rand(n, generator=g, device="cuda") < 0.01] *= 8.0
    return w.to(torch.bfloat16)


def _probs(logits, cut):
    """Probabilities of a row; with ``cut`` what a nucleus filter leaves: small ones exactly zero."""
    p = torch.softmax(logits, -1)
    if cut:
        p = torch.where(p < p.amax(-1, keepdim=True) * 1e-3, torch.zeros_like(p), p)
        p = p / p.sum(-1, keepdim=True)
    return p


def prepare(case, seed):
    c, g, dev = case, _gen(seed), "cuda"
    s = {"case": dict(c)}
    if c["op"] == "quantize":
        s["w"] = _weight(g, c["n"], c["k"])
    elif c["op"] == "norm":
        m, k = c["m"], c["k"]
        s["x"] = _randn(g, m, k).to(torch.bfloat16)
        # the residual stream has a few channels far larger than the others
        big = torch.where(torch.rand(k, generator=g, device=dev) < 0.005, 20.0, 1.5)
        s["residual"] = (_randn(g, m, k) * big).to(torch.bfloat16) if c["residual"] else None
        s["gamma"] = (1.0 + 0.05 * _randn(g, k)).to(torch.bfloat16) if c["gamma"] else None
        s["eps"] = 1e-6
    elif c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        codes, s["w_scales"] = _quantize_plain(_weight(g, n, k))
        s["w_codes"] = codes.view(torch.uint8)
        codes, scales = _groups_plain(_randn(g, m, k))
        s["a_codes"] = codes.view(torch.uint8)
        padded = torch.zeros((_blocks(k), (m + 3) // 4 * 4), device=dev)  # K-block major, rows of whole 16 bytes
        padded[:, :m] = scales
        s["a_scales"] = padded[:, :m]
    else:
        b, n, v, dv = c["batch"], c["g"], c["vocab"], c["draft_vocab"]
        kind = torch.bfloat16 if c["bf16"] else torch.float32
        s["target"] = torch.empty((b, n + 1, v), dtype=kind, device=dev)
        s["draft"] = torch.empty((b, n, dv), dtype=kind, device=dev) if dv else None
        s["tokens"] = torch.zeros((b, n), dtype=torch.int32, device=dev)
        spread = 4.0 * torch.rand((b, n + 1, 1), generator=g, device=dev) + 1.0  # flat rows and peaked ones
        for i in range(n + 1):  # a position at a time, to bound the memory
            logits = _randn(g, b, v) * spread[:, i]
            s["target"][:, i] = _probs(logits, c["cut"]).to(kind)
            if i < n and dv:  # the draft head is near the target, over its own vocabulary
                q = _probs(logits[:, :dv] + 0.3 * _randn(g, b, dv), c["cut"])
                s["draft"][:, i] = q.to(kind)
                gumbel = -torch.log(-torch.log(torch.rand((b, dv), generator=g, device=dev).clamp_(1e-30, 1 - 1e-7)))
                s["tokens"][:, i] = (torch.log(q) + gumbel).argmax(-1).to(torch.int32)
            elif i < n:
                s["tokens"][:, i] = (logits + 0.3 * _randn(g, b, v)).argmax(-1).to(torch.int32)
        s["accept_u"] = torch.rand((b, n), generator=g, device=dev)
        s["sample_u"] = torch.rand((b,), generator=g, device=dev)
        s["num_draft"] = None
        if c["ragged"]:
            s["num_draft"] = torch.randint(0, n + 1, (b,), generator=g, device=dev, dtype=torch.int32)
    return s


# ------------------------------------------------------------- plain forms

def _codes_plain(y, scale):
    q = torch.where(scale > 0, y / scale, torch.zeros_like(y))
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(F8)


def _scale_plain(amax):
    return amax / torch.full_like(amax, E4M3_MAX)  # one correctly rounded division


def _quantize_plain(w):
    """E4M3 codes [n, k] and FP32 scales [ceil(n/128), ceil(k/128)]."""
    n, k = w.shape
    bn, bk = _blocks(n), _blocks(k)
    f = torch.nn.functional.pad(w.float(), (0, bk * BLOCK - k, 0, bn * BLOCK - n)).view(bn, BLOCK, bk, BLOCK)
    scale = _scale_plain(f.abs().amax((1, 3), keepdim=True))
    codes = _codes_plain(f, scale).view(torch.uint8).view(bn * BLOCK, bk * BLOCK)[:n, :k].contiguous()
    return codes.view(F8), scale.view(bn, bk)


def _groups_plain(y):
    """E4M3 codes [m, k] and FP32 scales [ceil(k/128), m] of FP32 rows."""
    m, k = y.shape
    bk = _blocks(k)
    f = torch.nn.functional.pad(y, (0, bk * BLOCK - k)).view(m, bk, BLOCK)
    scale = _scale_plain(f.abs().amax(2, keepdim=True))
    codes = _codes_plain(f, scale).view(torch.uint8).view(m, bk * BLOCK)[:, :k].contiguous()
    return codes.view(F8), scale.view(m, bk).t().contiguous()


def _norm_plain(x, residual, gamma, eps):
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    y = h.float()
    if gamma is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * gamma.float()
    codes, scales = _groups_plain(y)
    return (codes, scales) if residual is None else (codes, scales, h)


def _gemm_plain(a_codes, a_scales, w_codes, w_scales, f32):
    k, n = a_codes.shape[1], w_codes.shape[0]
    a = a_codes.view(F8).float() * a_scales.t().repeat_interleave(BLOCK, 1)[:, :k]
    w = w_codes.view(F8).float()
    w *= w_scales.repeat_interleave(BLOCK, 1)[:, :k].repeat_interleave(BLOCK, 0)[:n]
    c = a @ w.t()
    return c if f32 else c.to(torch.bfloat16)


def _verify_plain(target, draft, tokens, accept_u, sample_u, num_draft):
    b, n1, v = target.shape
    n, rows, dev = n1 - 1, torch.arange(b, device=target.device), target.device
    num = torch.full((b,), n, device=dev) if num_draft is None else num_draft.long()
    at = torch.arange(n, device=dev)
    tok = tokens.long()
    p = target[rows[:, None], at, tok].double()
    q = torch.ones_like(p) if draft is None else draft[rows[:, None], at, tok].double()
    ok = (accept_u.double() * q < p) & (at < num[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    row = target[rows, accepted].double()
    w = row
    if n:
        refused = accepted < num
        i = accepted.clamp(max=n - 1)
        less = torch.zeros_like(row)
        if draft is None:
            less[rows, tok[rows, i]] = 1.0
        else:
            less[:, : draft.shape[2]] = draft[rows, i].double()
        w = torch.where(refused[:, None], (row - less).clamp(min=0.0), row)
        w = torch.where(w.sum(1, keepdim=True) > 0, w, row)
    c = w.cumsum(1)
    last = v - 1 - (w > 0).flip(1).long().argmax(1)
    j = torch.searchsorted(c, c[:, -1:] * sample_u.double()[:, None], right=True)[:, 0]
    token = torch.minimum(j, last)
    out = torch.full((b, n1), -1, dtype=torch.int32, device=dev)
    out[:, :n] = torch.where(at < accepted[:, None], tokens, out[:, :n])
    out[rows, accepted] = token.int()
    return out, accepted.int()


# --------------------------------------------------------------------- run

def _run_own(s):
    import nvfp4_speculative_draft_gb300 as nd
    c = s["case"]
    if c["op"] == "quantize":
        w = nd.fp8b_quantize(s["w"])
        return w.codes.view(F8), w.scales
    if c["op"] == "norm":
        a, h = nd.fp8b_rmsnorm(s["x"], s["gamma"], s["eps"], residual=s["residual"])
        out = a.codes.view(F8), a.scales
        return out if h is None else (*out, h)
    if c["op"] == "gemm":
        a = nd.Fp8BlockActs(s["a_codes"], s["a_scales"], c["m"], c["k"])
        w = nd.Fp8BlockWeight(s["w_codes"], s["w_scales"], c["n"], c["k"])
        return nd.fp8b_gemm(a, w, out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    return nd.spec_verify(s["target"], s["tokens"], s["accept_u"], s["sample_u"], draft_probs=s["draft"],
                          num_draft=s["num_draft"])


def run(state):
    if own:
        return _run_own(state)
    s, c = state, state["case"]
    if c["op"] == "quantize":
        return _quantize_plain(s["w"])
    if c["op"] == "norm":
        return _norm_plain(s["x"], s["residual"], s["gamma"], s["eps"])
    if c["op"] == "gemm":
        return _gemm_plain(s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"], c["f32"])
    return _verify_plain(s["target"], s["draft"], s["tokens"], s["accept_u"], s["sample_u"], s["num_draft"])


def work(case):
    c = case
    if c["op"] == "quantize":
        n, k = c["n"], c["k"]
        return {"bytes": 3 * n * k + 4 * _blocks(n) * _blocks(k), "flops": 3 * n * k}
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        each = 2 + 1 + (4 if c["residual"] else 0)
        return {"bytes": m * k * each + 4 * m * _blocks(k) + (2 * k if c["gamma"] else 0), "flops": 8 * m * k}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        scales = 4 * (_blocks(k) * m + _blocks(n) * _blocks(k))
        return {"bytes": n * k + m * k + scales + m * n * (4 if c["f32"] else 2), "flops": 2 * m * n * k}
    b, each = c["batch"], 2 if c["bf16"] else 4
    rows = c["vocab"] + (c["draft_vocab"] if c["g"] else 0)  # one row of the target's, one of the draft's
    return {"bytes": b * (rows * each + c["g"] * (8 + 2 * each) + 4 * (c["g"] + 4)), "flops": 3 * b * rows}


# ---------------------------------------------------- definitions in 64 bits

def _round_e4m3(v):
    """Nearest E4M3 value, ties to even, of float64 values of magnitude up to 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_blocks(y, rows):
    """E4M3 values of y and the scales of its blocks of ``rows`` x 128, a strip of rows at a time."""
    n, k = y.shape
    scales = torch.zeros((-(-n // rows), _blocks(k)), dtype=torch.float64, device=y.device)
    values = torch.zeros((n, k), dtype=torch.float32, device=y.device)
    strip = rows * max(1, (1 << 26) // (rows * k))
    for r in range(0, n, strip):
        part = y[r:r + strip].double()
        for b in range(_blocks(k)):
            cols = part[:, b * BLOCK:(b + 1) * BLOCK]
            most = cols.abs().amax(1)
            blocks = -(-most.shape[0] // rows)
            most = torch.nn.functional.pad(most, (0, blocks * rows - most.shape[0])).view(blocks, rows).amax(1)
            scale = most / torch.full_like(most, E4M3_MAX)
            scales[r // rows:r // rows + blocks, b] = scale
            each = scale.float().double().repeat_interleave(rows)[: cols.shape[0], None]  # the scale as it is held
            values[r:r + strip, b * BLOCK:(b + 1) * BLOCK] = torch.where(
                each > 0, _round_e4m3(cols / each.clamp(min=1e-300)), 0.0).float()
    return values, scales


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        return _exact_blocks(s["w"], BLOCK)
    if c["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(torch.bfloat16).double()
        y = h
        if s["gamma"] is not None:
            r = 1.0 / torch.sqrt((h * h).sum(1) / c["k"] + s["eps"])
            y = h * r[:, None] * s["gamma"].double()[None, :]
        values, scales = _exact_blocks(y, 1)
        out = (values, scales.t())
        return out if s["residual"] is None else (*out, h)
    if c["op"] == "gemm":
        total = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device="cuda")
        for b in range(_blocks(c["k"])):  # block by block: the codes' sums are exact, then the two scales
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            sums = s["a_codes"][:, cols].view(F8).double() @ s["w_codes"][:, cols].view(F8).double().t()
            column = s["w_scales"][:, b].double().repeat_interleave(BLOCK)[: c["n"]]
            total += sums * s["a_scales"][b].double()[:, None] * column[None, :]
        return total
    tokens, given = s["tokens"].cpu().numpy(), s["accept_u"].cpu().numpy().astype(np.float64)
    r = s["sample_u"].cpu().numpy().astype(np.float64)
    out = np.full((c["batch"], c["g"] + 1), -1, np.int32)
    accepted = np.zeros(c["batch"], np.int32)
    for i in range(c["batch"]):
        num = c["g"] if s["num_draft"] is None else int(s["num_draft"][i])
        a = 0
        while a < num:
            d = int(tokens[i, a])
            q = 1.0 if s["draft"] is None else float(s["draft"][i, a, d])
            if not given[i, a] * q < float(s["target"][i, a, d]):
                break
            out[i, a] = d
            a += 1
        accepted[i] = a
        p = s["target"][i, a].double().cpu().numpy()
        w = p.copy()
        if a < num and s["draft"] is None:
            w[tokens[i, a]] = max(0.0, p[tokens[i, a]] - 1.0)
        elif a < num:
            q = s["draft"][i, a].double().cpu().numpy()
            w[: q.size] = np.maximum(p[: q.size] - q, 0.0)
        if not w.sum() > 0:
            w = p
        sums = np.cumsum(w)
        out[i, a] = min(int(np.searchsorted(sums, r[i] * sums[-1], side="right")), int(np.flatnonzero(w > 0)[-1]))
    return torch.from_numpy(out), torch.from_numpy(accepted)
