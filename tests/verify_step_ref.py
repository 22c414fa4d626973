"""Plain 64-bit implementations of the verify step's operators, for the tests.

Elementary torch and numpy operations on the CPU or the GPU; nothing here comes
from the library."""
import numpy as np
import torch

BLOCK = 128
F8 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // BLOCK)


def e4m3(v):
    """Nearest E4M3 value of float64 values, ties to even, saturating at 448 (by
    the format: 3 mantissa bits, exponents from 2^-6, subnormal step 2^-9)."""
    a = v.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def quantize(w):
    """BF16 [n, k] -> (values of the codes float64 [n, k], scales float32), by the binary32 steps
    s = amax / 448, code = e4m3(fl32(w / s))."""
    n, k = w.shape
    values = torch.zeros((n, k), dtype=torch.float64, device=w.device)
    scales = torch.zeros((blocks(n), blocks(k)), dtype=torch.float32, device=w.device)
    f = w.float()
    for i in range(blocks(n)):
        for j in range(blocks(k)):
            part = f[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            amax = part.abs().amax().reshape(1)
            s = (amax / torch.full_like(amax, 448.0))
            scales[i, j] = s[0]
            if s[0] > 0:
                values[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = e4m3((part / s).double())
    return values, scales


def decode(codes):
    return codes.view(F8).double()


def norm(x, residual, gamma, eps):
    """(y float64, h bfloat16)."""
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    y = h.double()
    if gamma is not None:
        ms = (y * y).mean(1, keepdim=True) + eps
        y = torch.where(ms > 0, y / torch.sqrt(ms.clamp(min=1e-300)), torch.zeros_like(y)) * gamma.double()
    return y, h


def group_amax(y):
    m, k = y.shape
    y = torch.nn.functional.pad(y, (0, blocks(k) * BLOCK - k)).view(m, blocks(k), BLOCK)
    return y.abs().amax(2)


def gemm(a_codes, a_scales, w_codes, w_scales):
    """(C float64, sum of the terms' magnitudes)."""
    k, n = a_codes.shape[1], w_codes.shape[0]
    a = decode(a_codes) * a_scales.double().t().repeat_interleave(BLOCK, 1)[:, :k]
    w = decode(w_codes) * w_scales.double().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return a @ w.t(), a.abs() @ w.abs().t()


def verify(target, draft, tokens, accept_u, sample_u, num_draft=None):
    """numpy arrays of one dtype; float64 throughout, one token after another."""
    b, g1, v = target.shape
    out = np.full((b, g1), -1, np.int32)
    acc = np.zeros(b, np.int32)
    for s in range(b):
        num = g1 - 1 if num_draft is None else min(int(num_draft[s]), g1 - 1)
        a = 0
        while a < num:
            d = int(tokens[s, a])
            if not 0 <= d < v:
                break
            q = 1.0
            if draft is not None:
                q = float(draft[s, a, d]) if d < draft.shape[2] else 0.0
            if not float(accept_u[s, a]) * q < float(target[s, a, d]):
                break
            out[s, a] = d
            a += 1
        acc[s] = a
        p = target[s, a].astype(np.float64)
        w = p.copy()
        if a < num:
            if draft is not None:
                w[:draft.shape[2]] -= draft[s, a].astype(np.float64)
            elif 0 <= int(tokens[s, a]) < v:
                w[int(tokens[s, a])] -= 1.0
        w = np.where(np.isfinite(w) & (w > 0), w, 0.0)
        if not w.sum() > 0:
            w = np.where(np.isfinite(p) & (p > 0), p, 0.0)
        if not w.sum() > 0:
            out[s, a] = 0
            continue
        c = np.cumsum(w)
        over = np.flatnonzero((c > float(sample_u[s]) * c[-1]) & (w > 0))
        out[s, a] = over[0] if over.size else np.flatnonzero(w > 0)[-1]
    return out, acc
