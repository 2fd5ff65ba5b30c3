"""The CTA-pair kernel of the block-scaled product: layouts, in-place residuals, shared operands, NaN blocks, far
offsets, exact sums, and the chain, at shapes that the few-row kernel does not take (each test asserts that).

Tolerances as in test_gpu_linear8.py.  `u` is fp32's 2^-24.
"""
import numpy as np
import pytest
import torch

import linear8_ref as R
from linear8_route import few_rows
from test_gpu_linear8 import HALF, U, bytes_of, codes_of, ffn, ffn_tensors, gen, h64, operand, rm, up16  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def for_pairs(rm, G, M, N, K, out, act=None):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert not few_rows(rm, G, M, N, K, out, act, sms)


def bmm64(a, w):
    """a [G, M, K] times w [G, N, K] transposed, in 64 bits."""
    return torch.bmm(torch.from_numpy(np.ascontiguousarray(a)), torch.from_numpy(np.ascontiguousarray(w)).mT).numpy()


def result(out, G, M, N):
    """Output (and scale) arrays with sentinels behind the rows: (view, buffer, scale view, scale buffer)."""
    o = torch.full((G, M, N + 32), 3, dtype=torch.float32).to(TYPES[out]).cuda()
    s = torch.full((G, M, (N + 127) // 128 + 1), 9, dtype=torch.uint8, device="cuda") if out == "e4m3" else None
    return o[..., :N], o, None if s is None else s[..., :-1], s


# columns that end in every 16 of a tile's second 128, and in its first
@pytest.mark.parametrize("N", [912, 928, 944, 960, 976, 992, 1008, 1024, 1040, 1136])
@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("br", [1, 128])
def test_exact(rm, N, out, br):
    """Small whole numbers and scales 1/2, 1, 2: every sum is exact in fp32, so each result is the exact one rounded
    once.  With a residual of whole numbers too (not for 8 bits)."""
    g = gen(N + br)
    G, M, K = 2, 1285, 400
    for_pairs(rm, G, M, N, K, out)
    av, wv = torch.randint(-3, 4, (G, M, K), generator=g).float(), torch.randint(-3, 4, (G, N, K), generator=g).float()
    nb = (K + 127) // 128
    As = torch.randint(126, 129, (G, M, nb), generator=g, dtype=torch.uint8)
    Ws = torch.randint(126, 129, (G, -(-N // br), nb), generator=g, dtype=torch.uint8)
    a, w = R.values(h64(av), As.numpy().astype(np.int64), 1), R.values(h64(wv), Ws.numpy().astype(np.int64), br)
    v = bmm64(a, w)
    A, W = (t.to(torch.float8_e4m3fn).cuda() for t in (av, wv))
    r = torch.randint(-64, 65, (G, M, N), generator=g).float()
    for resid in (False, True) if out != "e4m3" else (False,):
        o, buf, s, sbuf = result(out, G, M, N)
        rm.rm_matmul_fp8_block(A, As.cuda(), W, Ws.cuda(), o, s, resid=r.to(TYPES[out]).cuda() if resid else None,
                               w_block_rows=br)
        torch.cuda.synchronize()
        want = v + h64(r) if resid else v
        if out == "e4m3":
            codes, sb = R.quantize(want, 1)
            assert np.array_equal(bytes_of(s), sb) and np.array_equal(codes_of(o), codes)
            assert bool((sbuf[..., -1] == 9).all())
        else:
            assert torch.equal(o.cpu(), torch.from_numpy(want).to(TYPES[out]))
        assert bool((buf[..., N:].float() == 3).all())


@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
def test_layouts(rm, out):
    """Tokens inside the rows ([B, T, ..] in memory) for every operand, bias and residual, results added in place;
    operands that the groups share: the same bits as from contiguous copies, which are near 64 bits."""
    g = gen(3)
    T, B, N, K = 4, 701, 912, 272
    for_pairs(rm, T, B, N, K, out)
    A, As, a = operand(g, B, T, K, 1)
    W, Ws, w = operand(g, N, T, K, 1, 0.1)                       # [N, T, K]: rows of W inside the groups too
    At, Ast, Wt, Wst = (t.transpose(0, 1) for t in (A, As, W, Ws))
    bias, r = 0.1 * torch.randn(T, N, generator=g).cuda(), torch.randn(B, T, N, generator=g).to(
        torch.bfloat16 if out == "bf16" else torch.float32).cuda()

    def call(A, As, W, Ws, layout, inplace=True):
        rows = layout == "rows"
        shape = (T, B, N) if rows else (B, T, N)
        o = torch.zeros(shape, device="cuda").to(TYPES[out])
        s = torch.zeros(shape[:2] + ((N + 127) // 128,), dtype=torch.uint8, device="cuda") if out == "e4m3" else None
        turn = (lambda t: t) if rows else (lambda t: None if t is None else t.transpose(0, 1))
        resid = None
        if out != "e4m3":
            resid = r.transpose(0, 1)
            if inplace:
                turn(o).copy_(resid)
                resid = turn(o)
        rm.rm_matmul_fp8_block(A, As, W, Ws, turn(o), turn(s), bias, None, resid, 1)
        torch.cuda.synchronize()
        o, s = turn(o), turn(s)
        return o.contiguous().view(torch.uint8), None if s is None else s.contiguous()

    def same(x, y):
        return torch.equal(x[0], y[0]) and (x[1] is None or torch.equal(x[1], y[1]))

    def near(got, a, w):
        v = bmm64(a, w) + h64(bias)[:, None]
        slack = (2 * K / 32 + 64) * U * bmm64(np.abs(a), np.abs(w)) + U * np.abs(v)
        if out == "e4m3":
            R.assert_quantized(codes_of(got[0]), bytes_of(got[1]), v, slack)
            return
        v = v + h64(r.transpose(0, 1))
        assert np.all(np.abs(h64(got[0].view(TYPES[out])) - v) <= slack + U * np.abs(v) + HALF[TYPES[out]] * np.abs(v) * 1.001)

    av, wv = a.swapaxes(0, 1), w.swapaxes(0, 1)
    packed = [t.contiguous() for t in (At, Ast, Wt, Wst)]        # (rows of 272 bytes: 16-byte starts)
    first = call(*packed, "rows", inplace=False)
    near(first, av, wv)
    assert same(call(At, Ast, Wt, Wst, "tokens"), first)
    assert same(call(At, Ast, Wt, Wst, "rows"), first)
    assert same(call(*packed, "tokens", inplace=False), first)
    shared_a = [t[:1].expand(T, *t.shape[1:]) for t in packed[:2]]
    near(call(*shared_a, Wt, Wst, "tokens"), np.broadcast_to(av[:1], av.shape), wv)
    shared_w = [t[:1].expand(T, *t.shape[1:]) for t in packed[2:]]
    near(call(At, Ast, *shared_w, "rows"), av, np.broadcast_to(wv[:1], wv.shape))


def test_residual_shared_by_the_groups(rm):
    g = gen(4)
    G, M, N, K = 3, 900, 1200, 130
    for out in ("bf16", "f32"):
        for_pairs(rm, G, M, N, K, out)
        A, As, a = operand(g, G, M, K, 1)
        W, Ws, w = operand(g, G, N, K, 128, 0.1)
        r = torch.randn(1, M, N, generator=g).to(TYPES[out]).cuda()
        o, p = (torch.empty(G, M, N, dtype=TYPES[out], device="cuda") for _ in range(2))
        rm.rm_matmul_fp8_block(A, As, W, Ws, o, resid=r.expand(G, M, N))
        rm.rm_matmul_fp8_block(A, As, W, Ws, p, resid=r.repeat(G, 1, 1))
        torch.cuda.synchronize()
        assert torch.equal(o, p)


def test_not_finite(rm):
    """A block that held an infinity makes exactly its row's (its weight column's) results NaN."""
    M, N, K = 2500, 1040, 384
    g = gen(M)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    x[1, 200] = x[2400, 383] = float("inf")
    w[140, 7] = w[1030, 300] = float("nan")
    q = [torch.empty(t.shape, dtype=torch.uint8, device="cuda") for t in (x, w)]
    s = [torch.empty(t.shape[0], 3, dtype=torch.uint8, device="cuda") for t in (x, w)]
    rm.rm_quantize_fp8_block(x.cuda(), q[0], s[0])
    rm.rm_quantize_fp8_block(w.cuda(), q[1], s[1])
    want = torch.zeros(M, N, dtype=torch.bool)
    want[[1, 2400]] = True
    want[:, [140, 1030]] = True
    nb = (N + 127) // 128
    blocks = torch.nn.functional.pad(want, (0, nb * 128 - N)).view(M, nb, 128).any(-1)
    for act in (None, "relu", "tanh", "erf"):
        for out in ("bf16", "f32", "e4m3"):
            for_pairs(rm, 1, M, N, K, out, act)
            o = torch.empty(M, N, dtype=TYPES[out], device="cuda")
            os_ = torch.empty(M, nb, dtype=torch.uint8, device="cuda") if out == "e4m3" else None
            rm.rm_matmul_fp8_block(q[0], s[0], q[1], s[1], o, os_, act=act, w_block_rows=1)
            torch.cuda.synchronize()
            if out == "e4m3":
                assert torch.equal(os_.cpu() == 255, blocks)
                spread = blocks.repeat_interleave(128, 1)[:, :N]
                assert torch.equal(o.cpu().float().isnan(), spread)
            else:
                assert torch.equal(o.cpu().isnan(), want)


@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
def test_offsets_beyond_32_bits(rm, out):
    """Two groups 2^31 + 2^20 elements apart, operands, scales, residual and results: the bits of near ones."""
    far = (1 << 31) + (1 << 20)
    g = gen(11)
    M, N, K = 1300, 1168, 256
    for_pairs(rm, 2, M, N, K, out)
    A, As, _ = operand(g, 2, M, K, 1)
    W, Ws, _ = operand(g, 2, N, K, 128, 0.1)

    def apart(t):
        shape = (2,) + tuple(t.shape[1:])
        b = torch.empty(far + t[0].numel(), dtype=t.dtype, device="cuda")
        v = b.as_strided(shape, (far, shape[2], 1))
        v.copy_(t)
        return v
    near = torch.zeros(2, M, N, dtype=TYPES[out], device="cuda")
    ns = torch.zeros(2, M, (N + 127) // 128, dtype=torch.uint8, device="cuda") if out == "e4m3" else None
    r = torch.randn(2, M, N, generator=g).to(TYPES[out]).cuda() if out != "e4m3" else None
    rm.rm_matmul_fp8_block(A, As, W, Ws, near, ns, resid=r)
    o = apart(torch.zeros_like(near)) if r is None else apart(r)          # (the residual in place)
    os_ = None if ns is None else apart(torch.zeros_like(ns))
    rm.rm_matmul_fp8_block(apart(A), apart(As), apart(W), apart(Ws), o, os_, resid=None if r is None else o)
    torch.cuda.synchronize()
    assert torch.equal(o.contiguous().view(torch.uint8), near.view(torch.uint8)) and bool((near.float() != 0).any())
    assert ns is None or torch.equal(os_.contiguous(), ns)


def test_ffn_chain_captured(rm):
    """Norm, two products (both on the CTA pairs) captured on a side stream and replayed on new inputs, another chain
    running on a second stream meanwhile: bit for bit what direct calls give."""
    T, B, D, Hd = 8, 300, 1040, 1168
    for_pairs(rm, T, B, Hd, D, "e4m3", "tanh")
    for_pairs(rm, T, B, D, Hd, "bf16")
    t, u = ffn_tensors(rm, T, B, D, Hd, 1), ffn_tensors(rm, T, B, D, Hd, 2)
    ffn(rm, t)
    ffn(rm, u)
    torch.cuda.synchronize()
    want_u = u["y"].clone()
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ffn(rm, t, side)
    for k in range(2):
        t["x"].copy_(torch.randn(t["x"].shape, generator=gen(k)).bfloat16())
        ffn(rm, t)
        torch.cuda.synchronize()
        want = t["y"].clone()
        t["y"].zero_()
        u["y"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        ffn(rm, u, other)
        torch.cuda.synchronize()
        assert torch.equal(t["y"], want) and torch.equal(u["y"], want_u)


def test_ffn_chain(rm):
    """The chain against 64 bits with exact operands; the bound is derived in test_gpu_linear8.py's chain test."""
    T, B, D, Hd = 8, 260, 1040, 1168
    for_pairs(rm, T, B, Hd, D, "e4m3", "tanh")
    for_pairs(rm, T, B, D, Hd, "bf16")
    t = ffn_tensors(rm, T, B, D, Hd, 7)
    ffn(rm, t)
    torch.cuda.synchronize()
    s = h64((t["x"].float() + t["r"].float()).bfloat16())
    y = R.rmsnorm(s, h64(t["gamma"]), 1e-5)[0].reshape(B, T, D)
    h = R.activation(bmm64(y.swapaxes(0, 1), h64(t["W1f"])) + h64(t["b1"])[:, None], "tanh")
    v = (bmm64(h, h64(t["W2f"])) + h64(t["b2"])[:, None]).swapaxes(0, 1)
    got = h64(t["y"]).reshape(B, T, D) - s.reshape(B, T, D)
    rel = np.linalg.norm(got - v) / np.linalg.norm(v)
    assert 5e-3 < rel < 0.108, rel


def test_linear_backward(rm):
    """A linear layer's three products, the input and weight gradients on the transposed operands."""
    g = gen(5)
    B, N, K = 1210, 2320, 2320
    for M_, N_, K_ in ((B, N, K), (B, K, N), (N, K, B)):
        for_pairs(rm, 1, M_, N_, K_, "f32")
    x, w, dy = torch.randn(B, K, generator=g), 0.1 * torch.randn(N, K, generator=g), 0.01 * torch.randn(B, N, generator=g)
    z = dict(dtype=torch.uint8, device="cuda")

    def q(t, br):
        r, c = t.shape
        o = dict(q=torch.empty(r, c, **z), s=torch.empty(-(-r // br), -(-c // 128), **z),
                 qt=torch.zeros(c, up16(r), **z)[:, :r], st=torch.empty(-(-c // br), -(-r // 128), **z))
        rm.rm_quantize_fp8_block(t.bfloat16().cuda(), o["q"], o["s"], o["qt"], o["st"], br)
        return o
    X, W, DY = q(x, 1), q(w, 128), q(dy, 1)
    y, dx, dw = (torch.empty(s, device="cuda") for s in ((B, N), (B, K), (N, K)))
    rm.rm_matmul_fp8_block(X["q"], X["s"], W["q"], W["s"], y)
    rm.rm_matmul_fp8_block(DY["q"], DY["s"], W["qt"], W["st"], dx)
    rm.rm_matmul_fp8_block(DY["qt"], DY["st"], X["qt"], X["st"], dw, w_block_rows=1)
    torch.cuda.synchronize()
    val = lambda o, k, br: R.values(codes_of(o["q" + k]), bytes_of(o["s" + k]), br)               # noqa: E731
    for got, a, b in ((y, val(X, "", 1), val(W, "", 128)), (dx, val(DY, "", 1), val(W, "", 128).T),
                      (dw, val(DY, "t", 1), val(X, "t", 1))):
        tol = (2 * a.shape[1] / 32 + 64) * U * (np.abs(a) @ np.abs(b).T)
        assert np.all(np.abs(h64(got) - a @ b.T) <= tol)
