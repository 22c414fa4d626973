"""The operators of the attention step, as they are measured: cases, inputs, plain forms, definitions in 64 bits.

* ``plan``:   block tables, slot maps and positions of a batch's new tokens, built from request lengths;
* ``rope``:   rotary positions (one axis, or time / height / width) of q and k, k and v into the paged cache;
* ``prompt``: causal attention over whole prompts, packed, grouped heads;
* ``paged``:  attention of each sequence's new tokens (one to many) over the paged cache.

A case is a dict of plain values whose ``op`` is one of these; ``mix`` seeds the lengths of its sequences, which belong
to the case and not to the inputs.  ``run`` computes a case either with elementary torch operations or, where ``own``
is true, with the framework's calls.
"""
import math
import random

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's bookkeeping: 24 sequences, a few drafted tokens each (latency); a full server's step with
        # chunks of prompts among the decoding sequences
        {"name": "plan draft step", "op": "plan", "batch": 24, "new": 5, "kv": 9000, "page": 16, "mix": 1},
        {"name": "plan server", "op": "plan", "batch": 1000, "new": 400, "kv": 16000, "page": 16, "mix": 2},
        # one decoded token of a head with rotary positions on a quarter of it (latency); a verify batch; a long
        # prompt of images and text with three position axes
        {"name": "rope one token", "op": "rope", "tokens": 1, "heads": 32, "kv_heads": 4, "dim": 256, "rot": 64,
         "axes": 1, "page": 16, "far": 100000},
        {"name": "rope verify", "op": "rope", "tokens": 315, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "axes": 1, "page": 16, "far": 16000},
        {"name": "rope images", "op": "rope", "tokens": 16384, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128,
         "axes": 3, "page": 32, "far": 30000},
        # one short prompt (latency); a packed batch of ragged prompts; one long prompt; heads of 256
        {"name": "prompt short", "op": "prompt", "batch": 1, "len": 77, "heads": 32, "kv_heads": 8, "dim": 128,
         "mix": 3},
        {"name": "prompt packed", "op": "prompt", "batch": 11, "len": 1900, "heads": 28, "kv_heads": 4, "dim": 128,
         "mix": 4},
        {"name": "prompt long", "op": "prompt", "batch": 1, "len": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "mix": 5},
        {"name": "prompt wide heads", "op": "prompt", "batch": 2, "len": 4001, "heads": 32, "kv_heads": 4, "dim": 256,
         "mix": 6},
        # one sequence, one token (latency); a verify batch of drafted positions over ragged caches; chunks of two
        # prompts over what is cached of them
        {"name": "paged one token", "op": "paged", "batch": 1, "new": 1, "kv": 4000, "heads": 32, "kv_heads": 4,
         "dim": 256, "page": 16, "ragged": False, "mix": 7},
        {"name": "paged verify", "op": "paged", "batch": 64, "new": 5, "kv": 16000, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "ragged": True, "mix": 8},
        {"name": "paged chunk", "op": "paged", "batch": 2, "new": 1500, "kv": 12000, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "ragged": True, "mix": 20},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _layout(rng):
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (32, 4), (40, 8), (16, 16), (14, 2), (24, 8), (12, 1)])
    return heads, kv_heads, rng.choice([64, 128, 128, 128, 256])


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "prompt", "prompt", "prompt", "paged", "paged", "paged"])
    mix = rng.randrange(1, 1 << 30)
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    while True:
        heads, kv_heads, dim = _layout(rng)
        if op == "plan":
            return {"op": op, "batch": _log(rng, 1, 1000), "new": _log(rng, 1, 400), "kv": _log(rng, 10, 16000),
                    "page": page, "mix": mix}
        if op == "rope":
            c = {"op": op, "tokens": _log(rng, 1, 16384), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                 "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "axes": rng.choice([1, 1, 3]), "page": page,
                 "far": _log(rng, 100, 1000000)}
            if c["tokens"] * (heads + kv_heads) * dim <= 16384 * 48 * 128:
                return c
        elif op == "prompt":
            c = {"op": op, "batch": _log(rng, 1, 64), "len": _log(rng, 1, 16384), "heads": heads,
                 "kv_heads": kv_heads, "dim": dim, "mix": mix}
            n = _lengths(c)
            if sum(x * x for x in n) * heads * dim <= 16384 * 16384 * 32 * 128 / 2 and sum(n) <= 32768:
                return c
        else:
            c = {"op": op, "batch": _log(rng, 1, 128), "new": rng.choice([1, 1, 2, 5, 9, _log(rng, 10, 2000)]),
                 "kv": _log(rng, 10, 65536), "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
                 "ragged": rng.random() < 0.7, "mix": mix}
            new, kv = _chunks(c)
            pairs = sum(a * b for a, b in zip(new, kv))
            if pairs * heads * dim <= 16384 * 16384 * 32 * 128 / 4 and sum(kv) * kv_heads * dim <= 600000 * 8 * 128:
                return c


def _lengths(c):
    """Lengths of a packed batch of prompts: one is ``len``, the others spread below it."""
    r = random.Random(c["mix"])
    n = [c["len"]] + [_log(r, max(1, c["len"] // 30), c["len"]) for _ in range(c["batch"] - 1)]
    r.shuffle(n)
    return n


def _chunks(c):
    """New tokens and cache lengths (the new tokens included) of each sequence."""
    r = random.Random(c["mix"])
    new = [c["new"]] * c["batch"]
    kv = [max(c["kv"], c["new"])] * c["batch"]
    if c["ragged"]:
        new = [r.randint(1, c["new"]) for _ in new]
        kv = [max(a, _log(r, max(1, c["kv"] // 40), c["kv"])) for a in new]
    return new, kv


def _requests(c):
    """Cached lengths, new tokens and held pages of a batch's requests: one in eight brings a chunk of its prompt, some
    are absent, some hold pages of drafts that were refused."""
    r = random.Random(c["mix"])
    lens, new, held = [], [], []
    for _ in range(c["batch"]):
        lens.append(_log(r, max(1, c["kv"] // 50), c["kv"]))
        kind = r.random()
        new.append(r.randint(1, c["new"]) if kind < 0.125 else -1 if kind < 0.2 else r.randint(1, min(c["new"], 5)))
        held.append(-(-lens[-1] // c["page"]) + (1 if r.random() < 0.1 else 0))
    return lens, new, held


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _prefix(n):
    return [0] + [int(x) for x in np.cumsum(n)]


def _keys(g, *shape):
    """Keys have a few channels with a large offset, as trained models' keys do; their scores differ by a constant."""
    offset = torch.where(torch.rand(shape[-2:], generator=g, device=DEV) < 0.03, 4.0, 0.0)
    return (_randn(g, *shape) + offset).to(BF16)


def _queries(g, *shape):
    """Flat heads and peaked ones."""
    sharp = 0.5 + 2.0 * torch.rand((shape[-2], 1), generator=g, device=DEV)
    return (_randn(g, *shape) * sharp).to(BF16)


THETA = 1000000.0


def _sections(rot, axes):
    """Pairs of each position axis: time, height, width."""
    half = rot // 2
    return [half] if axes == 1 else [half - 2 * (half * 3 // 8), half * 3 // 8, half * 3 // 8]


def _positions(g, tokens, axes, far):
    """Text counts on; of an image (every other stretch of 256 tokens) time stands still and height and width run."""
    start = int(torch.randint(0, far, (1,), generator=g, device=DEV).item())
    t = torch.arange(tokens, device=DEV, dtype=torch.int32)
    if axes == 1:
        return start + t
    image = (t // 256) % 2 == 1
    base = t - t % 256
    return torch.stack([torch.where(image, start + base, start + t),
                        torch.where(image, start + base + (t % 256) // 16, start + t),
                        torch.where(image, start + base + t % 16, start + t)]).contiguous()


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if c["op"] == "plan":
        lens, new, held = _requests(c)
        s["lens"], s["new"], s["held"] = _ints(lens), _ints(new), _ints(held)
        page, width = c["page"], -(-(c["kv"] + c["new"]) // c["page"]) + 2
        pages = sum(held) + sum(max(n, 0) // page + 1 for n in new) + 8
        order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
        s["table"] = torch.full((c["batch"], width), -1, dtype=torch.int32, device=DEV)
        mine = torch.arange(width, device=DEV)[None, :] < s["held"][:, None]
        s["table"][mine] = order[: sum(held)]
        s["free"] = order[sum(held):].clone()
        s["count"] = _ints([s["free"].numel()])
        s["tokens"] = (sum(max(n, 0) for n in new) + 7) // 8 * 8  # a padded batch
    elif c["op"] == "rope":
        t, hq, hk, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        s["qkv"] = _randn(g, t, (hq + 2 * hk) * d).to(BF16)  # one projection's rows
        s["positions"] = _positions(g, t, c["axes"], c["far"])
        pages = -(-t // c["page"]) + 5
        s["k_cache"] = torch.zeros((pages, c["page"], hk, d), dtype=BF16, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        order = torch.randperm(pages, generator=g, device=DEV)
        i = torch.arange(t, device=DEV) + 3
        s["slots"] = (order[i // c["page"]] * c["page"] + i % c["page"]).to(torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = torch.tensor([THETA ** (-2.0 * j / c["rot"]) for j in range(half)], dtype=torch.float64,
                                     device=DEV)
        s["axis"] = torch.tensor([a for a, n in enumerate(_sections(c["rot"], c["axes"])) for _ in range(n)],
                                 device=DEV)
        if own:
            import nvfp4_speculative_draft_gb300 as nd
            s["rotary"] = nd.rotary_table(c["rot"], theta=THETA, sections=_sections(c["rot"], c["axes"]), device=DEV)
    elif c["op"] == "prompt":
        t, hq, hk, d = sum(_lengths(c)), c["heads"], c["kv_heads"], c["dim"]
        s["q"], s["k"], s["v"] = _queries(g, t, hq, d), _keys(g, t, hk, d), _randn(g, t, hk, d).to(BF16)
        s["cu"] = _ints(_prefix(_lengths(c)))
    else:
        new, kv = _chunks(c)
        hk, d, page = c["kv_heads"], c["dim"], c["page"]
        need = [-(-n // page) for n in kv]
        pages = sum(need) + 3
        s["q"] = _queries(g, sum(new), c["heads"], d)
        s["k_cache"], s["v_cache"] = _keys(g, pages, page, hk, d), _randn(g, pages, page, hk, d).to(BF16)
        order = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
        s["table"] = torch.full((c["batch"], max(need) + 1), -1, dtype=torch.int32, device=DEV)
        mine = torch.arange(max(need) + 1, device=DEV)[None, :] < _ints(need)[:, None]
        s["table"][mine] = order[: sum(need)]
        s["kv_lens"], s["cu"] = _ints(kv), _ints(_prefix(new))
    return s


# ------------------------------------------------------------- plain forms

def _plan_plain(lens, new, held, table, free, count, page, tokens):
    dev = lens.device
    n, have, width = new.clamp(min=0).long(), lens.clamp(min=0).long(), table.shape[1]
    held = held.long()
    end = n.cumsum(0)
    need = torch.where(n > 0, (have + n + page - 1) // page, held)
    fits = (need <= width) & (end <= tokens)
    extra = torch.where(fits, (need - held).clamp(min=0), torch.zeros_like(need))
    upto = extra.cumsum(0)
    ok = fits & ((extra == 0) | (upto <= count.long()))
    taken = torch.where(ok, upto, torch.zeros_like(upto)).amax() if n.numel() else 0
    j = torch.arange(width, device=dev)[None, :]
    fresh = ok[:, None] & (j >= held[:, None]) & (j < need[:, None])
    at = count.long() - 1 - ((upto - extra)[:, None] + j - held[:, None])
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), end.clamp(max=tokens)])
    i = torch.arange(tokens, device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    real = seq < n.numel()
    seq = seq.clamp(max=n.numel() - 1)
    pos = have[seq] + i - cu[seq]
    slot = table[seq, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    slots = torch.where(real & ok[seq], slot, torch.full_like(slot, -1))
    positions = torch.where(real, pos, torch.zeros_like(pos))
    kv = torch.where(ok, have + n, have)
    now = torch.where(ok, torch.maximum(held, need), held)
    return tuple(x.to(torch.int32) for x in (table, cu, kv, positions, slots, now, count.long() - taken))


def _rope_plain(s):
    c = s["case"]
    t, hq, hk, d, half = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    q, k, v = s["qkv"].view(t, hq + 2 * hk, d).split([hq, hk, hk], 1)
    pos = s["positions"].view(c["axes"], t)[s["axis"]]                      # [pairs, tokens]
    angle = pos.t().double() * s["inv_freq"]                                # 64 bits: positions reach far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        x = x.float()
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., 2 * half:]], -1).to(BF16)

    slots = s["slots"].long()
    s["k_cache"].view(-1, hk, d)[slots] = turn(k)
    s["v_cache"].view(-1, hk, d)[slots] = v
    return turn(q), s["k_cache"], s["v_cache"]


def _attend_plain(q, k, v, first, scale):
    """q [n, heads, d] at positions first, first + 1, ... over k, v [m, kv_heads, d]; FP32 in and out."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    out = torch.empty_like(q)
    kt = k.permute(1, 2, 0)                                                 # [kv_heads, d, m]
    vt = v.permute(1, 0, 2)
    step = max(1, (1 << 29) // (heads * k.shape[0]))                        # bounds the scores' memory
    for r in range(0, n, step):
        rows = min(step, n - r)
        seen = min(k.shape[0], first + r + rows)
        part = q[r:r + rows].view(rows, k.shape[1], group, d).permute(1, 2, 0, 3).reshape(k.shape[1], group * rows, d)
        scores = ((part * scale) @ kt[..., :seen]).view(k.shape[1], group, rows, seen)
        hidden = torch.arange(seen, device=q.device)[None, :] > first + r + torch.arange(rows, device=q.device)[:, None]
        scores.masked_fill_(hidden, float("-inf"))
        scores -= scores.amax(-1, keepdim=True)
        scores.exp_()
        scores /= scores.sum(-1, keepdim=True)
        o = scores.view(k.shape[1], group * rows, seen) @ vt[:, :seen]
        out[r:r + rows] = o.view(k.shape[1], group, rows, d).permute(2, 0, 1, 3).reshape(rows, heads, d)
    return out


def _prompt_plain(q, k, v, lengths):
    out, at = torch.empty_like(q), 0
    for n in lengths:
        part = slice(at, at + n)
        out[part] = _attend_plain(q[part].float(), k[part].float(), v[part].float(), 0, q.shape[-1] ** -0.5).to(BF16)
        at += n
    return out


def _paged_plain(q, k_cache, v_cache, table, new, kv):
    out, at, page = torch.empty_like(q), 0, k_cache.shape[1]
    for i, (n, m) in enumerate(zip(new, kv)):
        pages = table[i, : -(-m // page)].long()
        k = k_cache[pages].flatten(0, 1)[:m].float()
        v = v_cache[pages].flatten(0, 1)[:m].float()
        out[at:at + n] = _attend_plain(q[at:at + n].float(), k, v, m - n, q.shape[-1] ** -0.5).to(BF16)
        at += n
    return out


# --------------------------------------------------------------------- run

def _run_own(s):
    import nvfp4_speculative_draft_gb300 as nd
    c = s["case"]
    if c["op"] == "plan":
        p = nd.kv_plan(s["lens"], s["new"], s["table"], s["free"], s["count"], page_size=c["page"],
                       tokens=s["tokens"], held=s["held"])
        return s["table"], p.cu_new, p.kv_lens, p.positions, p.slots, p.held, p.free_count
    if c["op"] == "rope":
        t, hq, hk, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        q, k, v = s["qkv"].view(t, hq + 2 * hk, d).split([hq, hk, hk], 1)
        q, _ = nd.rope_kv_write(q, k, v, s["positions"], s["rotary"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                                slots=s["slots"])
        return q, s["k_cache"], s["v_cache"]
    if c["op"] == "prompt":
        return nd.prompt_attention(s["q"], s["k"], s["v"], s["cu"])
    return nd.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu"])


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s)
    if c["op"] == "plan":
        return _plan_plain(s["lens"], s["new"], s["held"], s["table"], s["free"], s["count"], c["page"], s["tokens"])
    if c["op"] == "rope":
        return _rope_plain(s)
    if c["op"] == "prompt":
        return _prompt_plain(s["q"], s["k"], s["v"], _lengths(c))
    return _paged_plain(s["q"], s["k_cache"], s["v_cache"], s["table"], *_chunks(c))


def work(case):
    c = case
    if c["op"] == "plan":
        lens, new, held = _requests(c)
        fresh = sum(max(0, -(-(a + n) // c["page"]) - h) for a, n, h in zip(lens, new, held) if n > 0)
        tokens = sum(max(n, 0) for n in new)
        # lengths, new tokens, held pages in; prefix, lengths, held pages out; positions and slots; a page in and out
        return {"bytes": 24 * c["batch"] + 8 * tokens + 8 * fresh, "flops": 10 * (c["batch"] + tokens)}
    if c["op"] == "rope":
        each = c["heads"] + 2 * c["kv_heads"]
        rotated = (c["heads"] + c["kv_heads"]) * c["rot"]
        return {"bytes": c["tokens"] * (4 * each * c["dim"] + 4 * c["axes"] + 4), "flops": 3 * c["tokens"] * rotated}
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "prompt":
        n = _lengths(c)
        return {"bytes": sum(n) * d * (4 * hq + 4 * hk), "flops": 4 * d * hq * sum(x * (x + 1) // 2 for x in n)}
    new, kv = _chunks(c)
    seen = sum(a * b - a * (a - 1) // 2 for a, b in zip(new, kv))
    return {"bytes": sum(new) * d * 4 * hq + sum(kv) * d * 4 * hk, "flops": 4 * d * hq * seen}


# ---------------------------------------------------- definitions in 64 bits

def _exact_plan(c, s):
    lens, new, held = (s[x].tolist() for x in ("lens", "new", "held"))
    table, free, left = s["table"].cpu().numpy().copy(), s["free"].tolist(), int(s["count"][0])
    page, tokens, width = c["page"], s["tokens"], table.shape[1]
    cu, kv, now = [0], [], []
    positions, slots = np.zeros(tokens, np.int32), np.full(tokens, -1, np.int32)
    full = False
    for i in range(len(lens)):
        n, have, mine = max(new[i], 0), max(lens[i], 0), held[i]
        need = -(-(have + n) // page) if n else mine
        ok = need <= width and cu[-1] + n <= tokens
        more = max(0, need - mine)
        if ok and more:
            full = full or more > left
            ok = not full
            if ok:
                for j in range(mine, need):
                    left -= 1
                    table[i, j] = free[left]
        for j in range(n):
            if cu[-1] + j < tokens:
                positions[cu[-1] + j] = have + j
                if ok:
                    slots[cu[-1] + j] = table[i, (have + j) // page] * page + (have + j) % page
        cu.append(min(tokens, cu[-1] + n))
        kv.append(have + n if ok else have)
        now.append(max(mine, need) if ok else mine)
    whole = (table, cu, kv, positions, slots, now, [left])
    return tuple(torch.tensor(np.asarray(x), dtype=torch.int32) for x in whole)


def _exact_rope(c, s):
    t, hq, hk, d, half = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    x = s["qkv"].view(t, hq + 2 * hk, d)
    pairs = [a for a, n in enumerate(_sections(c["rot"], c["axes"])) for _ in range(n)]
    rows = s["positions"].view(c["axes"], t).double()
    out = x[:, : hq + hk].double()
    for j in range(half):
        angle = rows[pairs[j]] * THETA ** (-2.0 * j / c["rot"])
        cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        a, b = x[:, : hq + hk, j].double(), x[:, : hq + hk, half + j].double()
        out[..., j] = a * cos - b * sin
        out[..., half + j] = b * cos + a * sin
    pages = s["k_cache"].shape
    k, v = (torch.zeros((pages[0] * pages[1], hk, d), dtype=torch.float64, device=DEV) for _ in range(2))
    k.index_copy_(0, s["slots"].long(), out[:, hq:])
    v.index_copy_(0, s["slots"].long(), x[:, hq + hk:].double())
    return out[:, :hq], k.view(pages), v.view(pages)


def _exact_attend(q, k, v, first, out):
    """One head at a time, a strip of queries at a time, over the keys that some query of it sees."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    strip = max(1, min(1024, (1 << 27) // k.shape[0]))
    for h in range(heads):
        keys, values = k[:, h // group].double(), v[:, h // group].double()
        for r in range(0, n, strip):
            part = q[r:r + strip, h].double()
            last = first + r + part.shape[0]
            score = torch.mm(part, keys[:last].t()).div_(math.sqrt(d))
            position = torch.arange(first + r, last, device=q.device)
            score[torch.arange(last, device=q.device)[None] > position[:, None]] = -math.inf
            weight = torch.softmax(score, 1)
            out[r:r + strip, h] = torch.mm(weight, values[:last])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return _exact_plan(c, s)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    out, at = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), 0
    if c["op"] == "prompt":
        for n in _lengths(c):
            part = slice(at, at + n)
            _exact_attend(s["q"][part], s["k"][part], s["v"][part], 0, out[part])
            at += n
        return out
    page = c["page"]
    for i, (n, m) in enumerate(zip(*_chunks(c))):
        slots = torch.arange(m, device=DEV)
        slots = s["table"][i].long()[slots // page] * page + slots % page
        k, v = (s[x].reshape(-1, c["kv_heads"], c["dim"])[slots] for x in ("k_cache", "v_cache"))
        _exact_attend(s["q"][at:at + n], k, v, m - n, out[at:at + n])
        at += n
    return out
