"""The verify step's operators on the GPU against plain 64-bit implementations.

Tolerances (unit roundings: binary32 2^-24, BF16 2^-8 relative):
* quantiser: codes and scales are binary32 steps, compared exactly.
* norm: a row's sum of squares is at most 32 additions in a thread, 5 in a warp and
  32 over warps deep, and each square rounds once: 70 x 2^-24 relative; its root
  halves that; the mean's division, eps, root, reciprocal, two products and the
  scale's division add 7 more: 42 x 2^-24 = 2.6e-6 for y and the scales.  A code may
  be that of any value twice that near to y / s (the quotient rounds too).
* gemm: each K block's products are exact in binary32 and its sum is taken by the
  tensor core; allowing it 128 additions, and one product and one addition for each
  of the K blocks: (128 + 2 blocks) x 2^-24 of the sum of magnitudes; BF16 results one
  rounding more.
* verify: tokens and counts exactly.
"""
import numpy as np
import pytest
import torch

import verify_step_ref as ref

pytestmark = pytest.mark.gpu

NORM_TOL = 42 * 2.0 ** -24


def nd():
    import nvfp4_speculative_draft_gb300 as m
    return m


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def randn(dev, seed, *shape):
    return torch.randn(shape, generator=gen(dev, seed), device=dev)


def u8(codes):
    return codes.view(torch.uint8)


# ------------------------------------------------------------------ quantiser

def check_quantize(w, q):
    values, scales = ref.quantize(w)
    assert torch.equal(q.scales, scales)
    assert torch.equal(ref.decode(q.codes), values)


@pytest.mark.parametrize("n,k", [(1, 16), (1, 128), (127, 112), (128, 128), (129, 144), (300, 272), (5, 1040),
                                 (257, 2048), (640, 80)])
def test_quantize_exact(dev, n, k):
    w = (randn(dev, n * 7 + k, n, k) * 0.02).to(torch.bfloat16)
    check_quantize(w, nd().fp8b_quantize(w))


def test_quantize_special_blocks(dev):
    w = (randn(dev, 3, 384, 384) * 0.02).to(torch.bfloat16)
    w[:128, :128] = 0.0                       # scale 0: codes +0
    w[0, 0] = -0.0
    w[:128, 128:256] = 1e-38                  # scales near binary32's smallest
    w[128:256, :128] = 3e38                   # ... and largest
    w[130, 5] = -1.0
    w[128:256, 128:256] *= torch.exp2(torch.randint(-30, 30, (128, 128), device=dev)).to(torch.bfloat16)
    w[256:, :128] = -448.0
    w[256:, 128:256] = torch.arange(128, device=dev).to(torch.bfloat16)[None] * 3.5  # quotients on code borders
    w[256, 128] = 448.0
    q = nd().fp8b_quantize(w)
    check_quantize(w, q)
    assert q.codes.dtype == torch.float8_e4m3fn
    assert (u8(q.codes)[:128, :128] == 0).all() and (q.scales[0, 0] == 0).item()


def test_quantize_padded_rows_and_guards(dev):
    m = nd()
    wide = (randn(dev, 5, 150, 400) * 0.02).to(torch.bfloat16)
    w = wide[:, 8:8 + 304]
    n, k = w.shape
    buf = torch.full((n * k + 64,), 0xA5, dtype=torch.uint8, device=dev)
    sc = torch.full((2 * 3 + 8,), 7.0, device=dev)
    out = m.Fp8BlockWeight(buf[32:32 + n * k].view(n, k), sc[4:10].view(2, 3), n, k)
    m.fp8b_quantize(w, out=out)
    check_quantize(w.contiguous(), out)
    assert (buf[:32] == 0xA5).all() and (buf[32 + n * k:] == 0xA5).all()
    assert (sc[:4] == 7).all() and (sc[10:] == 7).all()


def test_quantize_reports_nonfinite(dev):
    m = nd()
    w = torch.ones((256, 256), dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    good = m.fp8b_quantize(w, dev_status=status)
    assert status.item() == 0
    w[200, 10] = float("nan")
    bad = m.fp8b_quantize(w, dev_status=status)
    assert status.item() == 7
    assert torch.equal(u8(bad.codes)[:128], u8(good.codes)[:128]) and torch.equal(u8(bad.codes)[128:, 128:], u8(good.codes)[128:, 128:])


# ----------------------------------------------------------------------- norm

def check_norm(acts, h, x, residual, gamma, eps):
    y, h_ref = ref.norm(x, residual, gamma, eps)
    if residual is not None:
        assert torch.equal(h, h_ref)
    tol = NORM_TOL if gamma is not None else 2.0 ** -24
    s_ref = ref.group_amax(y) / 448.0
    s = acts.scales.t().double()
    assert ((s - s_ref).abs() <= s_ref * tol + 2.0 ** -149).all()
    rows = s.repeat_interleave(ref.BLOCK, 1)[:, :x.shape[1]]
    got = ref.decode(acts.codes)
    q = torch.where(rows > 0, y / rows.clamp(min=1e-300), torch.zeros_like(y))
    a, b = ref.e4m3(q * (1 - 2 * tol)), ref.e4m3(q * (1 + 2 * tol))
    assert ((got >= torch.minimum(a, b)) & (got <= torch.maximum(a, b))).all()


@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (3, 144), (7, 496), (1, 4096), (5, 5120), (130, 1024), (33, 8192),
                                 (2, 8208), (3, 17408), (2, 32768), (700, 112)])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("with_gamma", [False, True])
def test_norm(dev, m, k, with_res, with_gamma):
    x = randn(dev, m + k, m, k).to(torch.bfloat16)
    r = (randn(dev, m + k + 1, m, k) * 3).to(torch.bfloat16) if with_res else None
    g = (1 + 0.05 * randn(dev, k, k)).to(torch.bfloat16) if with_gamma else None
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    acts, h = nd().fp8b_rmsnorm(x, g, 1e-6, residual=r, dev_status=status)
    assert (h is None) == (r is None) and status.item() == 0
    check_norm(acts, h, x, r, g, 1e-6)


def test_norm_zero_rows_and_eps(dev):
    x = randn(dev, 1, 6, 256).to(torch.bfloat16)
    x[1] = 0.0
    x[2, 128:] = 0.0
    x[3] *= 1e-3
    g = torch.ones(256, dtype=torch.bfloat16, device=dev)
    for eps in (0.0, 1e-6, 1.0):
        acts, _ = nd().fp8b_rmsnorm(x, g, eps)
        check_norm(acts, None, x, None, g, eps)
        assert (u8(acts.codes)[1] == 0).all() and (acts.scales[:, 1] == 0).all()
        assert (u8(acts.codes)[2, 128:] == 0).all() and acts.scales[1, 2].item() == 0


@pytest.mark.parametrize("alias", ["residual", "x"])
@pytest.mark.parametrize("k", [256, 5120, 17408])
def test_norm_in_place(dev, alias, k):
    m = nd()
    x = randn(dev, 2, 9, k).to(torch.bfloat16)
    r = randn(dev, 3, 9, k).to(torch.bfloat16)
    g = torch.ones(k, dtype=torch.bfloat16, device=dev)
    want, h = m.fp8b_rmsnorm(x, g, residual=r)
    x2, r2 = x.clone(), r.clone()
    target = r2 if alias == "residual" else x2
    got, h2 = m.fp8b_rmsnorm(x2, g, residual=r2, residual_out=target)
    assert h2 is target and torch.equal(target, h)
    assert torch.equal(u8(got.codes), u8(want.codes)) and torch.equal(got.scales, want.scales)


def test_norm_strides_and_guards(dev):
    m = nd()
    rows, k = 37, 400
    x = randn(dev, 4, rows, 520).to(torch.bfloat16)[:, 8:8 + k]
    r = randn(dev, 5, rows, 408).to(torch.bfloat16)[:, :k]
    ro = torch.full((rows, 424), 5.0, dtype=torch.bfloat16, device=dev)
    codes = torch.full((rows + 2, 432), 0xA5, dtype=torch.uint8, device=dev)
    scales = torch.full((6, 48), -7.0, device=dev)
    out = m.Fp8BlockActs(codes[1:-1, :k], scales[1:5, :rows], rows, k)
    g = randn(dev, 6, k).to(torch.bfloat16)
    m.fp8b_rmsnorm(x, g, 1e-5, residual=r, residual_out=ro[:, 8:8 + k], out=out)
    check_norm(out, ro[:, 8:8 + k], x, r, g, 1e-5)
    assert (ro[:, :8] == 5).all() and (ro[:, 8 + k:] == 5).all()
    assert (codes[0] == 0xA5).all() and (codes[-1] == 0xA5).all() and (codes[:, k:] == 0xA5).all()
    assert (scales[0] == -7).all() and (scales[5] == -7).all() and (scales[:, rows:] == -7).all()


def test_norm_reports_nonfinite(dev):
    m = nd()
    g = torch.ones(512, dtype=torch.bfloat16, device=dev)
    good = randn(dev, 7, 4, 512).to(torch.bfloat16)
    for value in (float("nan"), float("inf"), 3e38):
        for gamma in (g, None):
            x = good.clone()
            x[2, 300] = value
            status = torch.zeros(1, dtype=torch.int32, device=dev)
            acts, _ = m.fp8b_rmsnorm(x, gamma, dev_status=status)
            want, _ = m.fp8b_rmsnorm(good, gamma)
            assert status.item() == (7 if gamma is not None or value != 3e38 else 0)
            assert torch.equal(u8(acts.codes)[[0, 1, 3]], u8(want.codes)[[0, 1, 3]])


# ----------------------------------------------------------------------- gemm

def make_gemm(dev, m, n, k, seed=0):
    """Random codes of every finite value and scales over a wide range."""
    g = gen(dev, seed + m * 31 + n * 7 + k)
    mod = nd()

    def codes(r):
        c = torch.randint(0, 256, (r, k), generator=g, device=dev, dtype=torch.int32)
        c = torch.where((c & 0x7F) == 0x7F, c - 1, c)  # NaN codes
        return c.to(torch.uint8)

    ws = torch.exp2(torch.rand((ref.blocks(n), ref.blocks(k)), generator=g, device=dev) * 8 - 12)
    sc = torch.exp2(torch.rand((ref.blocks(k), m), generator=g, device=dev) * 8 - 10)
    return (mod.Fp8BlockActs(codes(m), sc, m, k), mod.Fp8BlockWeight(codes(n), ws, n, k))


def gemm_tol(c, s, k, bf16):
    tol = (128 + 2 * ref.blocks(k)) * 2.0 ** -24 * s
    return tol + (c.abs() + tol) * 2.0 ** -8 if bf16 else tol


def check_gemm(got, a, w):
    c, s = ref.gemm(a.codes, a.scales, w.codes, w.scales)
    assert ((got.double() - c).abs() <= gemm_tol(c, s, a.k, got.dtype == torch.bfloat16)).all()


GEMM_SIZES = [(1, 1, 16), (1, 128, 128), (1, 200, 5120), (2, 1000, 1024), (7, 129, 272), (16, 640, 2048), (17, 640, 2048),
              (31, 100, 144), (33, 257, 1040), (64, 5120, 512), (65, 128, 3200), (77, 1111, 400), (128, 300, 1024),
              (129, 640, 656), (255, 385, 528), (256, 256, 256), (300, 2000, 1152), (513, 129, 5120), (1000, 1500, 640)]


@pytest.mark.parametrize("m,n,k", GEMM_SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm(dev, m, n, k, dtype):
    a, w = make_gemm(dev, m, n, k)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = nd().fp8b_gemm(a, w, out_dtype=dtype, dev_status=status)
    assert got.dtype == dtype and status.item() == 0
    check_gemm(got, a, w)


# (the last five: 256-column tiles, several a CTA, one row of tiles and more, the last rows and columns ragged)
@pytest.mark.parametrize("m,n,k", [(1, 5120, 10240), (24, 20000, 5120), (2048, 2176, 5120), (1, 151936, 512), (128, 40000, 272),
                                   (300, 20001, 256), (385, 40000, 144), (1000, 9000, 400), (600, 20000, 1152)])
def test_gemm_large(dev, m, n, k):
    a, w = make_gemm(dev, m, n, k)
    check_gemm(nd().fp8b_gemm(a, w, out_dtype=torch.float32), a, w)


@pytest.mark.parametrize("m,n,k", [(3, 5120, 1024), (20, 333, 512), (100, 500, 384), (300, 700, 384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm_strides_and_guards(dev, m, n, k, dtype):
    mod = nd()
    a, w = make_gemm(dev, m, n, k)
    codes = torch.full((m, k + 48), 0x7F, dtype=torch.uint8, device=dev)  # NaN codes in the padding
    codes[:, 16:16 + k] = a.codes
    scales = torch.full((ref.blocks(k), m + 5), float("nan"), device=dev)
    scales[:, 1:1 + m] = a.scales
    padded = mod.Fp8BlockActs(codes[:, 16:16 + k], scales[:, 1:1 + m], m, k)
    buf = torch.full((m + 2, n + 9), -3.0, dtype=dtype, device=dev)
    out = buf[1:-1, 3:3 + n]
    mod.fp8b_gemm(padded, w, out=out)
    assert torch.equal(out, mod.fp8b_gemm(a, w, out_dtype=dtype))
    check_gemm(out, a, w)
    assert (buf[0] == -3).all() and (buf[-1] == -3).all() and (buf[:, :3] == -3).all() and (buf[:, 3 + n:] == -3).all()


def test_gemm_rows_do_not_mix(dev):
    """A row of NaN codes stays in its row; rows are the same whatever batch they come in, where the same tile serves them."""
    mod = nd()
    a, w = make_gemm(dev, 12, 700, 640)
    want = mod.fp8b_gemm(a, w, out_dtype=torch.float32)
    a.codes[5, 100] = 0x7F
    got = mod.fp8b_gemm(a, w, out_dtype=torch.float32)
    assert torch.isnan(got[5]).all()
    keep = [i for i in range(12) if i != 5]
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("m", [1, 9, 40, 100, 600])
def test_gemm_repeats_bitwise(dev, m):
    a, w = make_gemm(dev, m, 5120, 5120)
    first = nd().fp8b_gemm(a, w)
    for _ in range(5):
        assert torch.equal(nd().fp8b_gemm(a, w), first)


# --------------------------------------------------------------------- verify

def make_verify(dev, b, g, v, dv, dtype, seed, cut=False):
    gg = gen(dev, seed)
    t = torch.softmax(torch.randn((b, g + 1, v), generator=gg, device=dev) * 3, -1)
    q = None
    if cut:
        t = torch.where(t < t.amax(-1, keepdim=True) * 1e-2, torch.zeros_like(t), t)
    if dv:
        q = torch.softmax(torch.log(t[:, :g, :dv].clamp(min=1e-9)) + 0.3 * torch.randn((b, g, dv), generator=gg, device=dev), -1)
        tok = torch.multinomial(q.reshape(-1, dv), 1, generator=gg).view(b, g).int() if g else \
            torch.zeros((b, 0), dtype=torch.int32, device=dev)
        q = q.to(dtype)
    else:
        tok = t[:, :g].argmax(-1).int()
    t = t.to(dtype)
    return t, q, tok, torch.rand((b, g), generator=gg, device=dev), torch.rand(b, generator=gg, device=dev)


def host(x):
    return None if x is None else (x.float() if x.dtype == torch.bfloat16 else x).cpu().numpy()


def check_verify(t, q, tok, u, r, num=None, **kw):
    out, acc = nd().spec_verify(t, tok, u, r, draft_probs=q, num_draft=num, **kw)
    w_out, w_acc = ref.verify(host(t), host(q), host(tok), host(u), host(r), host(num))
    assert np.array_equal(acc.cpu().numpy(), w_acc)
    assert np.array_equal(out.cpu().numpy(), w_out)
    return out, acc


@pytest.mark.parametrize("b,g,v", [(1, 0, 1), (1, 1, 1), (2, 3, 2), (3, 1, 5), (4, 2, 31), (5, 4, 129), (1, 3, 4096), (7, 5, 4097),
                                   (64, 3, 1001), (2, 7, 32768), (3, 2, 50257), (2, 3, 151936), (400, 1, 300), (1, 40, 64)])
@pytest.mark.parametrize("kind", ["greedy", "sampled", "reduced"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify(dev, b, g, v, kind, dtype):
    dv = {"greedy": 0, "sampled": v, "reduced": max(1, v * 2 // 9)}[kind]
    t, q, tok, u, r = make_verify(dev, b, g, v, dv, dtype, b + g + v, cut=v % 2 == 1)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    check_verify(t, q, tok, u, r, dev_status=status)
    assert status.item() == 0


def test_verify_ragged_and_absent(dev):
    b, g, v = 9, 4, 777
    t, q, tok, u, r = make_verify(dev, b, g, v, v, torch.float32, 1)
    num = torch.tensor([0, 1, 2, 3, 4, 0, 4, 2, 1], dtype=torch.int32, device=dev)
    check_verify(t, q, tok, u, r, num)
    want, wacc = nd().spec_verify(t, tok, u, r, draft_probs=q, num_draft=num)
    num2 = num.clone()
    num2[[2, 8]] = -1
    out = torch.full((b, g + 3), 99, dtype=torch.int32, device=dev)
    acc = torch.full((b,), 99, dtype=torch.int32, device=dev)
    nd().spec_verify(t, tok, u, r, draft_probs=q, num_draft=num2, out_tokens=out, out_accepted=acc)
    assert (out[[2, 8]] == 99).all() and (acc[[2, 8]] == 99).all() and (out[:, g + 1:] == 99).all()
    keep = [0, 1, 3, 4, 5, 6, 7]
    assert torch.equal(out[keep, :g + 1], want[keep]) and torch.equal(acc[keep], wacc[keep])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    num3 = num.clone()
    num3[0] = g + 5  # counts as g
    got, _ = nd().spec_verify(t, tok, u, r, draft_probs=q, num_draft=num3, dev_status=status)
    num3[0] = g
    assert status.item() == 9 and torch.equal(got, nd().spec_verify(t, tok, u, r, draft_probs=q, num_draft=num3)[0])


def test_verify_tokens_outside_the_vocabulary(dev):
    t, q, tok, u, r = make_verify(dev, 4, 3, 100, 100, torch.float32, 2)
    u *= 0.0
    tok[0, 0], tok[1, 1], tok[2, 2] = 100, -1, 2 ** 31 - 1
    for draft in (q, None):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        _, acc = check_verify(t, draft, tok, u, r, dev_status=status)
        assert status.item() == 9 and acc.tolist()[:3] == [0, 1, 2]


def test_verify_masks_and_empty_rows(dev):
    v = 3000
    t = torch.zeros((6, 2, v), device=dev)
    q = torch.zeros((6, 1, v), device=dev)
    tok = torch.full((6, 1), 7, dtype=torch.int32, device=dev)
    u = torch.full((6, 1), 0.5, device=dev)
    r = torch.tensor([0.0, 0.3, 0.999999, 0.5, 1.0, float("nan")], device=dev)
    t[1, 0, 1234] = 1.0          # one token left
    t[2, 0] = q[2, 0] = 1.0 / v  # p = q: nothing left of the difference, p is sampled
    u[2, 0] = 1.0
    t[3, 0, :5] = torch.tensor([0.2, float("inf"), 0.2, float("nan"), -0.5], device=dev)  # what is not a weight counts as 0
    t[4:, 0, 10:13] = 0.25       # r = 1 and NaN: the last with a weight
    q[1, 0, 7] = q[3, 0, 7] = q[4:, 0, 7] = 1.0
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out, acc = nd().spec_verify(t, tok, u, r, draft_probs=q, dev_status=status)
    assert acc.tolist() == [0] * 6 and status.item() == 7
    assert out[:, 0].tolist() == [0, 1234, int(0.999999 * v), 2, 12, 12]
    check_verify(t, q, tok, u, r)


def test_verify_borders_are_exact(dev):
    """u q = p exactly is a refusal, one unit below an acceptance; a cumulative sum that equals r W belongs to the next token."""
    v = 1024
    p = torch.full((1, 2, v), 1.0 / v, device=dev)
    q = torch.full((1, 1, v), 2.0 / v, device=dev)
    tok = torch.tensor([[5]], dtype=torch.int32, device=dev)
    for u, want in ((0.5, 0), (float(np.nextafter(np.float32(0.5), np.float32(0))), 1)):
        _, acc = nd().spec_verify(p, tok, torch.tensor([[u]], device=dev), torch.tensor([0.0], device=dev), draft_probs=q)
        assert acc.item() == want
    no = torch.zeros((1, 0), dtype=torch.int32, device=dev)
    u = torch.zeros((1, 0), device=dev)
    for j in (0, 1, 511, 512, 1023):
        for r, want in ((j / v, j), (float(np.nextafter(np.float32((j + 1) / v), np.float32(0))), j)):
            out, _ = nd().spec_verify(p[:, :1], no, u, torch.tensor([r], device=dev))
            assert out.item() == want


def test_verify_fine_borders(dev):
    """Flat rows of 150 000 tokens: neighbouring borders are 7e-6 apart, and r falls on both sides of each within 1e-12."""
    v = 150001
    w = (1.0 + 0.5 * torch.rand((1, 1, v), generator=gen(dev, 3), device=dev)).expand(64, 1, v).contiguous()
    c = np.cumsum(w[0, 0].cpu().numpy().astype(np.float64))
    r = np.random.RandomState(0).rand(64).astype(np.float32)
    no = torch.zeros((64, 0), dtype=torch.int32, device=dev)
    out, _ = nd().spec_verify(w, no, torch.zeros((64, 0), device=dev), torch.from_numpy(r).to(dev))
    want = np.searchsorted(c, r.astype(np.float64) * c[-1], side="right")
    assert np.array_equal(out[:, 0].cpu().numpy(), want)


@pytest.mark.parametrize("v,dv,dtype", [(6000001, 0, torch.float32), (6000001, 6000001, torch.float32), (9000003, 2000001, torch.bfloat16)])
def test_verify_very_wide_rows(dev, v, dv, dtype):
    """Rows so wide that the search narrows in several steps."""
    t, q, tok, u, r = make_wide(dev, v, dv)
    t, q = t.to(dtype), None if q is None else q.to(dtype)
    check_verify(t, q, tok, u, r)
    check_verify(t, q, tok, u * 0 + 0.999, r)  # refused: the difference is sampled


def make_wide(dev, v, dv):
    g = gen(dev, v)
    t = torch.softmax(torch.randn((2, 2, v), generator=g, device=dev) * 2, -1)
    q = torch.softmax(torch.randn((2, 1, dv), generator=g, device=dev) * 2, -1) if dv else None
    tok = torch.randint(0, v, (2, 1), generator=g, device=dev).int()
    return t, q, tok, torch.rand((2, 1), generator=g, device=dev), torch.rand(2, generator=g, device=dev)


def test_verify_most_drafts(dev):
    t, q, tok, u, r = make_verify(dev, 3, 1024, 9, 9, torch.float32, 7)
    out, acc = check_verify(t, q, tok, u * 1e-3, r)
    check_verify(t, q, tok, u * 0, r, torch.tensor([1024, 1000, 31], dtype=torch.int32, device=dev))
    assert acc.max().item() > 32


@pytest.mark.parametrize("off_p,off_q", [(0, 1), (1, 1), (3, 2), (1, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_strides(dev, off_p, off_q, dtype):
    b, g, v = 5, 3, 2000
    t, q, tok, u, r = make_verify(dev, b, g, v, v, dtype, 5)
    tp = torch.full((b, g + 2, v + 13), float("nan"), dtype=dtype, device=dev)
    qp = torch.full((b, g + 1, v + 6), float("nan"), dtype=dtype, device=dev)
    tp[:, :g + 1, off_p:off_p + v] = t
    qp[:, :g, off_q:off_q + v] = q
    tk = torch.zeros((b, g + 4), dtype=torch.int32, device=dev)
    uu = torch.zeros((b, g + 2), device=dev)
    tk[:, :g], uu[:, :g] = tok, u
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = nd().spec_verify(tp[:, :g + 1, off_p:off_p + v], tk[:, :g], uu[:, :g], r, draft_probs=qp[:, :g, off_q:off_q + v],
                           dev_status=status)
    want = check_verify(t, q, tok, u, r)
    assert status.item() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_verify_distribution(dev):
    """Over many sequences the first token follows the target whatever the draft: a chi-square statistic of 15 degrees of
    freedom stays below 50 (probability 1e-5); the numbers are given, so the outcome is fixed."""
    n, v = 20000, 16
    p = torch.softmax(torch.randn(v, generator=gen(dev, 8), device=dev), 0)
    q = torch.softmax(torch.randn(v, generator=gen(dev, 9), device=dev), 0)
    t = p.expand(n, 2, v).contiguous()
    tok = torch.multinomial(q.expand(n, v), 1, generator=gen(dev, 10)).int()
    u = torch.rand((n, 1), generator=gen(dev, 11), device=dev)
    r = torch.rand(n, generator=gen(dev, 12), device=dev)
    out, _ = nd().spec_verify(t, tok, u, r, draft_probs=q.expand(n, 1, v).contiguous())
    seen = torch.bincount(out[:, 0].long(), minlength=v).double()
    assert ((seen - n * p.double()) ** 2 / (n * p.double())).sum().item() < 50


# ------------------------------------------------------------------- together

def chain(m, x, res, gamma, w, drafted, u, r, num, batch, g):
    acts, h = m.fp8b_rmsnorm(x, gamma, 1e-6, residual=res)
    logits = m.fp8b_gemm(acts, w, out_dtype=torch.float32)
    p = torch.softmax(logits.view(batch, g + 1, -1), -1)
    tokens, accepted = m.spec_verify(p, drafted, u, r, num_draft=num)
    return acts, h, logits, p, tokens, accepted


def chain_inputs(dev, batch=3, g=4, k=1024, v=5003, seed=0):
    m = nd()
    rows = batch * (g + 1)
    x = randn(dev, seed, rows, k).to(torch.bfloat16)
    res = randn(dev, seed + 1, rows, k).to(torch.bfloat16)
    gamma = (1 + 0.05 * randn(dev, seed + 2, k)).to(torch.bfloat16)
    w = m.fp8b_quantize((randn(dev, seed + 3, v, k) * 0.1).to(torch.bfloat16))
    drafted = torch.randint(0, v, (batch, g), generator=gen(dev, seed + 4), device=dev).int()
    u = torch.rand((batch, g), generator=gen(dev, seed + 5), device=dev) * 0.3
    r = torch.rand(batch, generator=gen(dev, seed + 6), device=dev)
    num = torch.tensor([g, g - 1, 0][:batch], dtype=torch.int32, device=dev)
    return x, res, gamma, w, drafted, u, r, num, batch, g


def test_verify_step_together(dev):
    """Greedy drafts from the target's own logits are accepted until one is spoiled."""
    m = nd()
    x, res, gamma, w, drafted, u, r, num, batch, g = chain_inputs(dev)
    _, _, logits, _, _, _ = chain(m, x, res, gamma, w, drafted, u, r, num, batch, g)
    drafted = logits.view(batch, g + 1, -1)[:, :g].argmax(-1).int()
    drafted[0, 2] = (drafted[0, 2] + 1) % w.n
    acts, h, logits, p, tokens, accepted = chain(m, x, res, gamma, w, drafted, u * 0, r, num, batch, g)
    check_norm(acts, h, x, res, gamma, 1e-6)
    check_gemm(logits, acts, w)
    want, wacc = ref.verify(host(p), None, host(drafted), host(u * 0), host(r), host(num))
    assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(accepted.cpu().numpy(), wacc)
    check_verify(p, None, drafted, u, r, num)


def test_verify_step_captured_and_replayed(dev):
    """Two captured graphs of the chain, replayed in turn on new inputs, and eager calls on another stream meanwhile."""
    m = nd()
    sets = [chain_inputs(dev, seed=s) for s in (0, 50)]
    fresh = [chain_inputs(dev, seed=s) for s in (100, 150)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for s in sets:
        chain(m, *s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(chain(m, *s))
        graphs.append(gr)
    eager = [chain(m, *f) for f in fresh]
    torch.cuda.synchronize()
    for s, f in zip(sets, fresh):
        for a, b in zip((s[0], s[1], s[2], s[4], s[5], s[6]), (f[0], f[1], f[2], f[4], f[5], f[6])):
            a.copy_(b)
        s[3].codes.copy_(f[3].codes)
        s[3].scales.copy_(f[3].scales)
    torch.cuda.synchronize()
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        with torch.cuda.stream(side):
            again = chain(m, *fresh[0])
    torch.cuda.synchronize()
    for got, want in [(outs[0], eager[0]), (outs[1], eager[1]), (again, eager[0])]:
        assert torch.equal(u8(got[0].codes), u8(want[0].codes))
        for i in (1, 2, 4, 5):
            assert torch.equal(got[i], want[i])


def test_nvfp4_draft_then_verify(dev):
    """The framework's own draft head proposes, the verify step judges: the drafts' hidden rows go through the NVFP4 head
    with argmax, the same rows through the block-scaled head."""
    m = nd()
    k, v, g = 1024, 4096, 3
    w = (randn(dev, 1, v, k) * 0.1).to(torch.bfloat16)
    x = randn(dev, 2, g + 1, k).to(torch.bfloat16)
    gamma = torch.ones(k, dtype=torch.bfloat16, device=dev)
    head, _ = m.nvfp4_quantize(w)
    _, drafted = m.w4a16_gemv_argmax([(x[:g], gamma, 1e-6)], head, logits=False)
    acts, _ = m.fp8b_rmsnorm(x, gamma, 1e-6)
    p = torch.softmax(m.fp8b_gemm(acts, m.fp8b_quantize(w), out_dtype=torch.float32), -1).view(1, g + 1, v)
    check_verify(p, None, drafted.view(1, g), torch.full((1, g), 1e-4, device=dev), torch.tensor([0.5], device=dev))


def test_on_another_stream(dev):
    m = nd()
    x, res, gamma, w, drafted, u, r, num, batch, g = chain_inputs(dev)
    want = chain(m, x, res, gamma, w, drafted, u, r, num, batch, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    acts, h = m.fp8b_rmsnorm(x, gamma, 1e-6, residual=res, stream=s)
    logits = m.fp8b_gemm(acts, w, out_dtype=torch.float32, stream=s)
    tokens, accepted = m.spec_verify(want[3], drafted, u, r, num_draft=num, stream=s)
    s.synchronize()
    assert torch.equal(logits, want[2]) and torch.equal(tokens, want[4]) and torch.equal(accepted, want[5])


def test_refusals_leave_outputs_alone(dev):
    """Tensors of the wrong shape, type, stride or device are refused before anything is launched."""
    m = nd()
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.ones((4, 256), dtype=bf, device=dev)
    g = torch.ones(256, dtype=bf, device=dev)
    bad_norm = [dict(x=x.float()), dict(x=x.t()), dict(x=x[0]), dict(gamma=g[:128]), dict(gamma=g.float()), dict(gamma=torch.ones(512, dtype=bf, device=dev)[::2]),
                dict(residual=x[:3]), dict(residual=x.cpu()), dict(residual=x, residual_out=x[:, :128]), dict(dev_status=torch.zeros(1, device=dev)),
                dict(gamma=torch.ones(256, dtype=bf))]
    for kw in bad_norm:
        args = dict(x=x, gamma=g)
        args.update(kw)
        with pytest.raises(ValueError):
            m.fp8b_rmsnorm(args.pop("x"), args.pop("gamma"), 1e-6, **args)
    acts, _ = m.fp8b_rmsnorm(x, g)
    w = m.fp8b_quantize(torch.ones((64, 256), dtype=bf, device=dev))
    out = torch.full((4, 64), 7.0, device=dev)
    for a in (m.Fp8BlockActs(acts.codes, acts.scales, 3, 256), m.Fp8BlockActs(acts.codes, acts.scales[:1], 4, 256),
              m.Fp8BlockActs(acts.codes[:, :128], acts.scales[:1], 4, 128), m.Fp8BlockActs(acts.codes.float(), acts.scales, 4, 256),
              m.Fp8BlockActs(acts.codes.cpu(), acts.scales.cpu(), 4, 256)):
        with pytest.raises(ValueError):
            m.fp8b_gemm(a, w, out=out)
    for bad in (m.Fp8BlockWeight(w.codes, w.scales[:, :1], 64, 256), m.Fp8BlockWeight(w.codes.t(), w.scales, 256, 64),
                m.Fp8BlockWeight(w.codes, w.scales.double(), 64, 256)):
        with pytest.raises(ValueError):
            m.fp8b_gemm(acts, bad, out=out)
    for o in (out[:3], out.half(), torch.full((4, 128), 7.0, device=dev)[:, ::2]):
        with pytest.raises(ValueError):
            m.fp8b_gemm(acts, w, out=o)
    with pytest.raises(ValueError):
        m.fp8b_gemm(acts, w, out_dtype=torch.float16)
    with pytest.raises(m.Nvfp4Error):  # k not a multiple of 16: the library's own check
        m.fp8b_quantize(torch.ones((4, 24), dtype=bf, device=dev))
    with pytest.raises(m.Nvfp4Error):
        m.fp8b_rmsnorm(torch.ones((0, 256), dtype=bf, device=dev), g)
    assert (out == 7).all()
    t = torch.full((2, 3, 10), 0.1, device=dev)
    q = t[:, :2].contiguous()
    tok, u, r = torch.zeros((2, 2), dtype=i32, device=dev), torch.zeros((2, 2), device=dev), torch.zeros(2, device=dev)
    res = torch.full((2, 3), 9, dtype=i32, device=dev)
    good = dict(target=t, tok=tok, u=u, r=r, draft_probs=q, out_tokens=res)
    bad = [dict(target=t.double()), dict(target=t.transpose(1, 2)), dict(target=t[0]), dict(tok=tok.long()), dict(tok=tok[:, :1]), dict(u=u[:1]),
           dict(r=r[:1]), dict(r=r.double()), dict(draft_probs=q.bfloat16()), dict(draft_probs=q[:, :1]), dict(draft_probs=torch.zeros((2, 2, 11), device=dev)),
           dict(num_draft=torch.zeros(3, dtype=i32, device=dev)), dict(out_tokens=res[:, :2]), dict(out_accepted=torch.zeros(1, dtype=i32, device=dev)),
           dict(tok=tok.cpu())]
    for kw in bad:
        a = dict(good)
        a.update(kw)
        with pytest.raises(ValueError):
            m.spec_verify(a.pop("target"), a.pop("tok"), a.pop("u"), a.pop("r"), **a)
    torch.cuda.synchronize()
    assert (res == 9).all()


# ------------------------------------------------- offsets beyond 32 bits

def test_offsets_pass_32_bits(dev):
    """Tensors of more than 2^31 elements; the parts that lie beyond are checked."""
    m = nd()
    # quantiser: 2.2e9 elements, the last two blocks of rows
    n, k = 131328, 16640
    w = torch.empty((n, k), dtype=torch.bfloat16, device=dev)
    for r in range(0, n, 16416):
        w[r:r + 16416] = (randn(dev, r, 16416, k) * 0.02).to(torch.bfloat16)
    q = m.fp8b_quantize(w)
    values, scales = ref.quantize(w[-256:, :1024].contiguous())
    assert torch.equal(q.scales[-2:, :8], scales) and torch.equal(ref.decode(q.codes[-256:, :1024]), values)
    # norm: the same matrix as rows of activations
    acts, h = m.fp8b_rmsnorm(w, torch.ones(k, dtype=torch.bfloat16, device=dev), 1e-6, residual=w)
    tail = m.Fp8BlockActs(acts.codes[-3:], acts.scales[:, -3:], 3, k)
    check_norm(tail, h[-3:], w[-3:], w[-3:], torch.ones(k, dtype=torch.bfloat16, device=dev), 1e-6)
    del w, q, acts, h, tail
    # product: 2.3e9 outputs
    a, wt = make_gemm(dev, 15000, 151936, 32)
    c = m.fp8b_gemm(a, wt)
    last = m.Fp8BlockActs(a.codes[-70:], a.scales[:, -70:], 70, 32)
    check_gemm(c[-70:], last, wt)
    check_gemm(c[:70], m.Fp8BlockActs(a.codes[:70], a.scales[:, :70], 70, 32), wt)
    del a, wt, c, last
    # verification: 2.4e9 probabilities; sequences of one repeated set of rows
    b, g, v = 4000, 3, 150001
    t1, q1, tok1, u1, r1 = make_verify(dev, 4, g, v, v, torch.bfloat16, 3)
    t = t1.repeat(b // 4, 1, 1)
    out, acc = m.spec_verify(t, tok1.repeat(b // 4, 1), u1.repeat(b // 4, 1), r1.repeat(b // 4),
                             draft_probs=q1.repeat(b // 4, 1, 1))
    want, wacc = check_verify(t1, q1, tok1, u1, r1)
    assert torch.equal(out, want.repeat(b // 4, 1)) and torch.equal(acc, wacc.repeat(b // 4))
