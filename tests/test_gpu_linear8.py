"""Block-scaled 8-bit linear layer against its 64-bit definitions (tests/linear8_ref.py).

Tolerances.  fp32 arithmetic with u = 2^-24 per rounding:
* rstd: a sum of squares is at most 32 + 5 + 16 additions deep (a thread's elements, the warp's butterflies, the
  row's warps), all terms positive, so it is within 53 u (and D's division and eps 2 u); the square root halves
  that, square root and reciprocal add 2 u: below 30 u.  y adds two products: below 32 u, plus half a step of its type.
* dx: a (1 u), the dot product (53 u of its absolute terms) and five more operations: below 64 u of the sum of the
  absolute terms, plus half a step.
* dgamma: one addition a row, the partials' tree behind it: (rows + 64) u of the sum of absolute values.
* product: K/32 accumulations of 32 products each; the tensor core may truncate, 2 u a step, and aligns the 32
  products of a step to the largest, 2 u each at most: (2 K/32 + 64) u of sum |a w|, plus bias, residual and
  activation (GELU with tanh.approx: 2^-10.9 of the value's half, see activation_slack).
* e4m3: half a step, 2^-4 of the value, 2^-10 of the block's scale at the least (assert_quantized).
"""
import numpy as np
import pytest
import torch

import linear8_ref as R

pytestmark = pytest.mark.gpu
U = R.F32_HALF
HALF = {torch.bfloat16: R.BF16_HALF, torch.float32: U}


@pytest.fixture(scope="module")
def rm():
    from token_mixing_feature_b200 import rankmixer
    return rankmixer


def gen(seed):
    return torch.Generator().manual_seed(seed)


def h64(t):
    return t.detach().cpu().double().numpy()


def codes_of(t):
    return R.decode_e4m3(t.detach().cpu().contiguous().view(torch.uint8).numpy())


def bytes_of(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy().astype(np.int64)


def rows_of(t, extra):
    """The same matrix on the GPU as rows of a wider buffer filled with sentinels: (view, buffer)."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), 7, dtype=torch.float32).to(t.dtype).cuda()
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]], wide


def up16(n):
    return (n + 15) // 16 * 16


# ---------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 16), (1, 1536), (3, 128), (5, 144), (257, 64), (130, 1040), (64, 2048), (33, 4112), (9, 7184), (5, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", NORM_SHAPES)
def test_norm(rm, rows, D, dtype):
    g = gen(rows + D)
    x = (torch.randn(rows, D, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    r = torch.randn(rows, D, generator=g).to(dtype)
    gamma = 1 + 0.2 * torch.randn(D, generator=g)
    x[rows // 2] = 0                       # a row whose sum with r is r
    r[rows // 2] = 0                       # ... and here zero altogether
    (xd, _), (rd, _) = rows_of(x, 48), rows_of(r, 16)
    sm, smw = rows_of(torch.zeros_like(x), 32)
    y, yw = rows_of(torch.zeros_like(x), 16)
    q = torch.full((rows, D + 16), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, (D + 127) // 128 + 3), 9, dtype=torch.uint8, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    rm.rm_rmsnorm_forward(xd, rd, gamma.cuda(), sm, y, q[:, :D], s[:, :-3], rstd, 1e-6)
    torch.cuda.synchronize()
    st = (x.float() + r.float()).to(dtype)
    assert torch.equal(sm.cpu(), st)
    ref, rr = R.rmsnorm(h64(st), h64(gamma), 1e-6)
    assert np.all(np.abs(h64(rstd) - rr) <= 30 * U * rr)
    assert np.all(np.abs(h64(y) - ref) <= (32 * U + HALF[dtype]) * np.abs(ref))
    R.assert_quantized(codes_of(q[:, :D]), bytes_of(s[:, :-3]), ref, 32 * U * np.abs(ref), "norm")
    # nothing beside the rows is touched
    assert bool((smw[:, D:] == 7).all() and (yw[:, D:] == 7).all() and (q[:, D:] == 9).all() and (s[:, -3:] == 9).all())
    # the outputs one at a time, without residual and gamma, sums in place
    xi, _ = rows_of(x, 0)
    rm.rm_rmsnorm_forward(xi, rd, None, Sum=xi)
    q2, s2 = torch.empty(rows, D, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(s[:, :-3])
    rm.rm_rmsnorm_forward(xi, Yq=q2, Ys=s2, eps=1e-6)
    torch.cuda.synchronize()
    assert torch.equal(xi.cpu(), st)
    ref1, _ = R.rmsnorm(h64(st), np.ones(D), 1e-6)
    R.assert_quantized(codes_of(q2), bytes_of(s2), ref1, 32 * U * np.abs(ref1), "norm without gamma")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(9001, 80), (5001, 256), (3001, 1536), (1201, 3600), (700, 7184), (310, 16384)])
def test_norm_many_rows(rm, rows, D, dtype):
    """Every group walks over several rows (the ring's places are used again), gamma kept in shared memory."""
    test_norm(rm, rows, D, dtype)


def test_norm_not_finite(rm):
    x = torch.ones(4, 272)
    x[1, 130], x[2, 3] = float("nan"), float("inf")
    q, s = torch.zeros(4, 272, dtype=torch.uint8, device="cuda"), torch.zeros(4, 3, dtype=torch.uint8, device="cuda")
    rm.rm_rmsnorm_forward(x.cuda(), Yq=q, Ys=s)
    torch.cuda.synchronize()
    assert s[1].tolist() == [255] * 3 and bool((q[1] == 127).all())     # the row's mean is NaN
    assert s[0].tolist() == s[3].tolist() and 255 not in s[0].tolist()
    # an infinite element: rstd = 0, the element itself 0 * inf = NaN, the other blocks zero
    assert s[2].tolist() == [255, 127, 127] and bool((q[2, 128:] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 16), (2, 1536), (300, 64), (3001, 256), (2500, 1040), (37, 5120), (700, 3600), (6, 16384)])
@pytest.mark.parametrize("dsum", [False, True])
def test_norm_grad(rm, rows, D, dtype, dsum):
    g = gen(rows * 3 + D)
    s = torch.randn(rows, D, generator=g).to(dtype)
    dy = torch.randn(rows, D, generator=g).to(dtype)
    ds = torch.randn(rows, D, generator=g).to(dtype) if dsum else None
    gamma = 1 + 0.2 * torch.randn(D, generator=g)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    (sd, _), (dyd, _) = rows_of(s, 16), rows_of(dy, 0)
    dx, dxw = rows_of(torch.zeros_like(s), 16)
    dg = torch.full((D,), 5.0, device="cuda")
    ws = torch.empty(rm.rm_rmsnorm_backward_workspace_bytes(rows, D) // 4, device="cuda")
    rm.rm_rmsnorm_backward(dyd, sd, gamma.cuda(), rstd.cuda(), ds.cuda() if dsum else None, dx, dg, ws)
    torch.cuda.synchronize()
    S, DY, G, RS = h64(s), h64(dy), h64(gamma), h64(rstd)
    rx, rg = R.rmsnorm_grad(DY, S, G, RS, h64(ds) if dsum else 0.0)
    r = RS[:, None]
    terms = r * (np.abs(DY * G) + np.abs(S) * r ** 2 * np.abs(DY * G * S).mean(1, keepdims=True)) + (np.abs(h64(ds)) if dsum else 0)
    assert np.all(np.abs(h64(dx) - rx) <= 64 * U * terms + HALF[dtype] * np.abs(rx) * 1.001)
    assert np.all(np.abs(h64(dg) - rg) <= (rows + 64) * U * np.abs(DY * S * r).sum(0))
    assert bool((dxw[:, D:] == 7).all())
    # in place of dY, without dgamma: the same bits; and again with dgamma: the same bits
    rm.rm_rmsnorm_backward(dyd, sd, gamma.cuda(), rstd.cuda(), ds.cuda() if dsum else None, dyd)
    dyd2, dg2 = rows_of(dy, 0)[0], torch.empty_like(dg)
    rm.rm_rmsnorm_backward(dyd2, sd, gamma.cuda(), rstd.cuda(), ds.cuda() if dsum else None, dyd2, dg2, ws)
    torch.cuda.synchronize()
    assert torch.equal(dyd.cpu(), dx.cpu()) and torch.equal(dyd2.cpu(), dx.cpu()) and torch.equal(dg, dg2)


def test_norm_grad_differences(rm):
    """dX and dgamma against central differences of the 64-bit forward: h = 1e-5, error O(h^2) + 1e-16/h."""
    g = gen(2)
    x, dy, gamma = torch.randn(3, 48, generator=g), torch.randn(3, 48, generator=g), 1 + 0.1 * torch.randn(48, generator=g)
    X, DY, G = h64(x), h64(dy), h64(gamma)
    rstd = torch.from_numpy(R.rmsnorm(X, G, 1e-6)[1]).float()
    dx, dg = torch.empty(3, 48, device="cuda"), torch.empty(48, device="cuda")
    ws = torch.empty(rm.rm_rmsnorm_backward_workspace_bytes(3, 48), dtype=torch.uint8, device="cuda")
    rm.rm_rmsnorm_backward(dy.cuda(), x.cuda(), gamma.cuda(), rstd.cuda(), None, dx, dg, ws)

    def loss(xx, gg):
        return (R.rmsnorm(xx, gg, 1e-6)[0] * DY).sum()

    def diff(f, at):
        out = np.zeros_like(at)
        for i in np.ndindex(at.shape):
            d = np.zeros_like(at)
            d[i] = 1e-5
            out[i] = (f(at + d) - f(at - d)) / 2e-5
        return out
    np.testing.assert_allclose(h64(dx), diff(lambda v: loss(v, G), X), atol=2e-5)
    np.testing.assert_allclose(h64(dg), diff(lambda v: loss(X, v), G), atol=2e-5)


def test_norm_grad_no_rows(rm):
    e, dg = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    rm.rm_rmsnorm_backward(e, e, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), None, e, dg)
    torch.cuda.synchronize()
    assert bool((dg == 0).all())


# ----------------------------------------------------------------- quantiser
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("G,rows,cols", [(1, 1, 16), (1, 128, 128), (3, 127, 144), (2, 130, 400), (1, 1000, 256), (5, 17, 1040)])
def test_quantize(rm, G, rows, cols, block_rows, dtype):
    g = gen(G + rows + cols)
    x = (torch.randn(G, rows, cols, generator=g) * torch.exp2(torch.randint(-20, 20, (G, rows, 1), generator=g))).to(dtype)
    x[0, 0] = 0
    x[-1, -1, :9] = torch.tensor([448.0, -448.0, 1e-30, -1e-38, 3e38, 2.0 ** -133, 0.0, 1.75, 1.0]).to(dtype)
    if rows > 100:
        x[0, 40, 5], x[0, 70, 12] = float("nan"), float("-inf")
    X = h64(x)
    (codes, sb), (codes_t, sb_t) = R.quantize(X, block_rows), R.quantize(X.swapaxes(1, 2), block_rows)
    src = x.cuda().transpose(0, 1).contiguous().transpose(0, 1)      # [rows, G, cols] in memory
    q = torch.full((G, rows, up16(cols) + 16), 9, dtype=torch.uint8, device="cuda")
    qt = torch.full((G, cols, up16(rows) + 16), 9, dtype=torch.uint8, device="cuda")
    s = torch.full(sb.shape, 9, dtype=torch.uint8, device="cuda")
    st = torch.full(sb_t.shape[:2] + (sb_t.shape[2] + 1,), 9, dtype=torch.uint8, device="cuda")
    rm.rm_quantize_fp8_block(src, q[..., :cols], s, qt[..., :rows], st[..., :-1], block_rows)
    torch.cuda.synchronize()
    assert np.array_equal(bytes_of(s), sb) and np.array_equal(bytes_of(st[..., :-1]), sb_t)
    assert np.array_equal(codes_of(q[..., :cols]), codes, equal_nan=True)
    assert np.array_equal(codes_of(qt[..., :rows]), codes_t, equal_nan=True)
    assert bool((q[..., cols:] == 9).all() and (qt[..., rows:] == 9).all() and (st[..., -1] == 9).all())
    # each orientation alone gives the same
    q1, qt1 = torch.empty_like(q[..., :cols].contiguous()), torch.full_like(qt, 9)
    s1, st1 = torch.empty_like(s), torch.empty_like(st[..., :-1].contiguous())
    rm.rm_quantize_fp8_block(src, q1, s1, block_rows=block_rows)
    rm.rm_quantize_fp8_block(src, dst_t=qt1[..., :rows], scale_t=st1, block_rows=block_rows)
    torch.cuda.synchronize()
    assert torch.equal(q1, q[..., :cols]) and torch.equal(s1, s) and torch.equal(qt1, qt) and torch.equal(st1, st[..., :-1])


# ------------------------------------------------------------------- product
def operand(g, G, rows, K, block_rows, std=1.0):
    """Quantised [G, rows, K] with padded rows: (codes on the GPU, scales on the GPU, values in 64 bits)."""
    codes, sb = R.quantize(h64((torch.randn(G, rows, K, generator=g) * std).float()), block_rows)
    buf = torch.full((G, rows, up16(K) + 16), 0x7f, dtype=torch.uint8)       # NaN behind the rows
    buf[..., :K] = torch.from_numpy(codes).to(torch.float8_e4m3fn).view(torch.uint8)
    return buf.cuda()[..., :K], torch.from_numpy(sb.astype(np.uint8)).cuda(), R.values(codes, sb, block_rows)


def activation_slack(v, act, precise):
    """Error of the activation's own arithmetic: tanh.approx is good to 2^-10.9 of tanh (|tanh| <= 1), scaled by
    v / 2; expf, erfc and the polynomial around them to a few u of |v|."""
    if act == "tanh" and not precise:
        return 0.5 * np.abs(v) * 2.0 ** -10.9 + 8 * U * np.abs(v)
    return 0 if act in (None, "relu") else 32 * U * np.abs(v)


def check_product(rm, seed, G, M, N, K, br=128, out=torch.bfloat16, act=None, bias=False, resid=False, call=None):
    g = gen(seed)
    A, As, a = operand(g, G, M, K, 1)
    W, Ws, w = operand(g, G, N, K, br, (2.0 / (N + K)) ** 0.5)
    b = 0.1 * torch.randn(G, N, generator=g) if bias else None
    e4 = out is torch.float8_e4m3fn
    r = torch.randn(G, M, N, generator=g).to(out) if resid else None
    pad = 32
    O = torch.full((G, M, N + pad), 3, dtype=torch.float32).to(out).cuda()
    os_ = torch.full((G, M, (N + 127) // 128 + 1), 9, dtype=torch.uint8, device="cuda") if e4 else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rm.rm_matmul_fp8_block(A, As, W, Ws, O[..., :N], os_[..., :-1] if e4 else None, b.cuda() if bias else None, act,
                           r.cuda() if resid else None, br, status)
    torch.cuda.synchronize()
    assert int(status) == rm.RM_OK
    v = np.einsum("gmk,gnk->gmn", a, w, optimize=True)
    slack = (2 * K / 32 + 64) * U * np.einsum("gmk,gnk->gmn", np.abs(a), np.abs(w), optimize=True)
    if bias:
        v = v + h64(b)[:, None]
        slack = slack + U * np.abs(v)
    ref = R.activation(v, act)
    slack = slack * (1.13 if act in ("tanh", "erf") else 1) + activation_slack(v, act, out is torch.float32)  # |GELU'| < 1.13
    if resid:
        ref = ref + h64(r)
        slack = slack + U * np.abs(ref)
    if e4:
        R.assert_quantized(codes_of(O[..., :N]), bytes_of(os_[..., :-1]), ref, slack, "product")
        assert bool((os_[..., -1] == 9).all())
    else:
        err = np.abs(h64(O[..., :N]) - ref)
        assert np.all(err <= slack * (1 + 2 ** -7) + HALF[out] * np.abs(ref) * 1.001), f"worst {np.max(err - slack)}"
    assert bool((O[..., N:].float() == 3).all())
    return O


PRODUCTS = [
    # G, M, N, K, w_block_rows: one token, ragged edges, several tiles, K behind one chunk of 512
    (1, 1, 16, 16, 128), (1, 1, 1536, 1536, 128), (1, 2, 128, 128, 128), (2, 3, 48, 100, 1), (1, 17, 272, 1, 1),
    (3, 16, 128, 640, 128), (2, 33, 400, 1040, 128), (1, 64, 256, 2064, 1), (2, 65, 144, 513, 128), (4, 100, 512, 256, 128),
    (1, 128, 128, 512, 1), (2, 129, 272, 768, 128), (1, 255, 1024, 384, 128), (1, 257, 528, 1536, 1), (3, 513, 640, 272, 128),
    (1, 700, 2064, 320, 1), (1, 1030, 784, 4112, 128),
]


@pytest.mark.parametrize("G,M,N,K,br", PRODUCTS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
def test_product(rm, G, M, N, K, br, out):
    check_product(rm, G + M + N + K, G, M, N, K, br, out)


@pytest.mark.parametrize("act", ["tanh", "erf", "relu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("G,M,N,K", [(2, 5, 176, 400), (2, 300, 400, 272)])
def test_product_epilogue(rm, G, M, N, K, out, act):
    check_product(rm, M, G, M, N, K, 128, out, act, bias=True, resid=out is not torch.float8_e4m3fn)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", [(3, 700, 592, 144), (9, 300, 784, 128), (2, 1000, 1040, 640), (20, 257, 336, 256)])
def test_product_residual(rm, G, M, N, K, out):
    """Large enough for the pair kernel, columns ending in every part of a tile."""
    check_product(rm, N, G, M, N, K, 128, out, None, False, True)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("G,M,N,K,br,act", [(9, 300, 784, 700, 128, None), (9, 300, 784, 400, 128, "tanh"),
                                            (3, 1000, 784, 640, 1, "erf"), (3, 1000, 784, 16, 1, "relu")])
def test_product_many_tiles(rm, G, M, N, K, br, out, act):
    """More 64 x 128 tiles than fit on the GPU at once: the pair kernel for every type and activation."""
    check_product(rm, K, G, M, N, K, br, out, act, bias=act is not None, resid=act == "erf" and out is not torch.float8_e4m3fn)


@pytest.mark.parametrize("G,M,N,K", [(300, 40, 256, 144), (150, 300, 272, 128), (90, 260, 528, 16)])
def test_product_short_last_rows(rm, G, M, N, K):
    """8-bit results, several tiles a CTA pair, the last 32-row part of a group with at most 16 rows: one store a tile."""
    check_product(rm, M, G, M, N, K, 128, torch.float8_e4m3fn)


@pytest.mark.parametrize("M", [1, 8, 40, 130, 600])
@pytest.mark.parametrize("br", [1, 128])
def test_product_exact(rm, M, br):
    """Small whole numbers and scales 1/2, 1, 2: every partial sum is exact in fp32, so are the results."""
    g = gen(M)
    G, N, K = 2, 304, 1168
    av, wv = torch.randint(-3, 4, (G, M, K), generator=g).float(), torch.randint(-3, 4, (G, N, K), generator=g).float()
    nb = (K + 127) // 128
    As = torch.randint(126, 129, (G, M, nb), generator=g, dtype=torch.uint8)
    Ws = torch.randint(126, 129, (G, -(-N // br), nb), generator=g, dtype=torch.uint8)
    out = torch.empty(G, M, N, device="cuda")
    rm.rm_matmul_fp8_block(av.to(torch.float8_e4m3fn).cuda(), As.cuda(), wv.to(torch.float8_e4m3fn).cuda(), Ws.cuda(), out,
                           w_block_rows=br)
    a, w = R.values(h64(av), As.numpy().astype(np.int64), 1), R.values(h64(wv), Ws.numpy().astype(np.int64), br)
    assert np.array_equal(h64(out), np.einsum("gmk,gnk->gmn", a, w, optimize=True))


def test_product_layouts(rm):
    """Tokens inside the rows ([B, T, D] in memory), inputs shared by the groups, results added in place."""
    g = gen(8)
    T, B, N, K = 3, 70, 160, 272
    A, As, a = operand(g, B, T, K, 1)                # [B, T, K]
    W, Ws, w = operand(g, T, N, K, 128, 0.1)
    out = torch.full((B, T, N), 2.0, device="cuda")
    first = torch.empty(B, T, N, device="cuda")
    rm.rm_matmul_fp8_block(A.transpose(0, 1), As.transpose(0, 1), W, Ws, first.transpose(0, 1))
    rm.rm_matmul_fp8_block(A.transpose(0, 1), As.transpose(0, 1), W, Ws, out.transpose(0, 1), resid=out.transpose(0, 1))
    shared = torch.empty(T, B, N, device="cuda")
    rm.rm_matmul_fp8_block(A.transpose(0, 1)[:1].expand(T, B, K), As.transpose(0, 1)[:1].expand(T, B, As.shape[-1]), W, Ws, shared)
    one = torch.empty(T, B, N, device="cuda")
    rm.rm_matmul_fp8_block(A.transpose(0, 1), As.transpose(0, 1), W[:1].expand(T, N, K), Ws[:1].expand(T, *Ws.shape[1:]), one)
    torch.cuda.synchronize()
    slack = (2 * K / 32 + 64) * U * np.einsum("btk,tnk->btn", np.abs(a), np.abs(w))
    assert np.all(np.abs(h64(first) - np.einsum("btk,tnk->btn", a, w)) <= slack)
    assert torch.equal(out, first + 2.0)
    assert np.all(np.abs(h64(shared) - np.einsum("bk,tnk->tbn", a[:, 0], w)) <=
                  (2 * K / 32 + 64) * U * np.einsum("bk,tnk->tbn", np.abs(a[:, 0]), np.abs(w)))
    assert np.all(np.abs(h64(one) - np.einsum("btk,nk->tbn", a, w[0])) <=
                  (2 * K / 32 + 64) * U * np.einsum("btk,nk->tbn", np.abs(a), np.abs(w[0])))


@pytest.mark.parametrize("M", [3, 200])
def test_product_not_finite(rm, M):
    """A block that held an infinity makes exactly its row's (its weight column's) results NaN."""
    g = gen(M)
    x, w = torch.randn(M, 384, generator=g), torch.randn(256, 384, generator=g)
    x[1, 200] = float("inf")
    w[140, 7] = float("nan")
    q = [torch.empty(t.shape, dtype=torch.uint8, device="cuda") for t in (x, w)]
    s = [torch.empty(t.shape[0], 3, dtype=torch.uint8, device="cuda") for t in (x, w)]
    rm.rm_quantize_fp8_block(x.cuda(), q[0], s[0])
    rm.rm_quantize_fp8_block(w.cuda(), q[1], s[1])
    out = torch.empty(M, 256, device="cuda")
    o8, os8 = torch.empty(M, 256, dtype=torch.uint8, device="cuda"), torch.empty(M, 2, dtype=torch.uint8, device="cuda")
    for act in (None, "relu"):
        rm.rm_matmul_fp8_block(q[0], s[0], q[1], s[1], out, act=act, w_block_rows=1)
        rm.rm_matmul_fp8_block(q[0], s[0], q[1], s[1], o8, os8, act=act, w_block_rows=1)
        torch.cuda.synchronize()
        want = torch.zeros(M, 256, dtype=torch.bool)
        want[1], want[:, 140] = True, True
        assert torch.equal(out.cpu().isnan(), want)
        blocks = torch.tensor([[False, True]]).repeat(M, 1)
        blocks[1] = True
        assert torch.equal(os8.cpu() == 255, blocks)
        assert torch.equal(o8.cpu() == 127, blocks.repeat_interleave(128, 1))


def test_offsets_beyond_32_bits(rm):
    """Groups 2^31 + 2^20 elements apart: the norm, the quantiser both ways and the product (few rows and many)."""
    far = (1 << 31) + (1 << 20)
    g = gen(11)
    for B in (3, 400):
        x = torch.randn(2, B, 256, generator=g).bfloat16()
        buf = torch.empty(far + B * 256, dtype=torch.bfloat16, device="cuda")
        v = buf.as_strided((2, B, 256), (far, 256, 1))
        v.copy_(x)
        n = buf.as_strided((2, 256), (far, 1))                 # two rows far apart
        y = torch.empty(2, 256, dtype=torch.bfloat16, device="cuda")
        rm.rm_rmsnorm_forward(n, Y=y, eps=1e-6)
        ref, _ = R.rmsnorm(h64(x[:, 0]), np.ones(256), 1e-6)
        assert np.all(np.abs(h64(y) - ref) <= (32 * U + R.BF16_HALF) * np.abs(ref))
        b8 = torch.empty(far + B * 256, dtype=torch.uint8, device="cuda")
        q, s = b8.as_strided((2, B, 256), (far, 256, 1)), torch.empty(2, B, 2, dtype=torch.uint8, device="cuda")
        bt = torch.empty(far + 256 * up16(B), dtype=torch.uint8, device="cuda")
        qt = bt.as_strided((2, 256, B), (far, up16(B), 1))
        st = torch.empty(2, 256, (B + 127) // 128, dtype=torch.uint8, device="cuda")
        rm.rm_quantize_fp8_block(v, q, s, qt, st)
        torch.cuda.synchronize()
        for got, gots, want in ((q, s, h64(x)), (qt, st, h64(x).swapaxes(1, 2))):
            codes, sb = R.quantize(want, 1)
            assert np.array_equal(codes_of(got), codes) and np.array_equal(bytes_of(gots), sb)
        w, ws, wv = operand(g, 2, 128, 256, 128)
        ob = torch.empty(far + B * 128, dtype=torch.bfloat16, device="cuda")
        out = ob.as_strided((2, B, 128), (far, 128, 1))
        rm.rm_matmul_fp8_block(q, s, w, ws, out)
        near = torch.empty(2, B, 128, dtype=torch.bfloat16, device="cuda")
        rm.rm_matmul_fp8_block(q.contiguous(), s, w, ws, near)
        torch.cuda.synchronize()
        a = R.values(codes_of(q), bytes_of(s), 1)
        assert torch.equal(out, near)
        tol = (2 * 256 / 32 + 64) * U * np.einsum("gmk,gnk->gmn", np.abs(a), np.abs(wv))
        ref = np.einsum("gmk,gnk->gmn", a, wv)
        assert np.all(np.abs(h64(out) - ref) <= tol * 1.01 + R.BF16_HALF * np.abs(ref) * 1.001)
        del buf, b8, bt, ob


def test_empty(rm):
    z = dict(dtype=torch.uint8, device="cuda")
    rm.rm_matmul_fp8_block(torch.empty(0, 64, **z), torch.empty(0, 1, **z), torch.empty(32, 64, **z),
                           torch.empty(1, 1, **z), torch.empty(0, 32, device="cuda"))
    rm.rm_quantize_fp8_block(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, **z), torch.empty(0, 1, **z))
    rm.rm_rmsnorm_forward(torch.empty(0, 64, device="cuda"), Y=torch.empty(0, 64, device="cuda"))
    torch.cuda.synchronize()


# ------------------------------------------------------- together, as one layer
def ffn(rm, t, stream=None):
    """Residual norm -> first projection, GELU -> second projection + residual, 8-bit between them."""
    rm.rm_rmsnorm_forward(t["x"], t["r"], t["gamma"], t["s"], None, t["q"], t["qs"], t["rstd"], 1e-5, stream)
    T, B, D = t["T"], t["B"], t["D"]
    per_token = lambda a: a.view(B, T, -1).transpose(0, 1)                                        # noqa: E731
    rm.rm_matmul_fp8_block(per_token(t["q"]), per_token(t["qs"]), t["W1"], t["W1s"], t["h"], t["hs"], t["b1"], "tanh",
                           stream=stream)
    rm.rm_matmul_fp8_block(t["h"], t["hs"], t["W2"], t["W2s"], per_token(t["y"]), None, t["b2"], None, per_token(t["s"]),
                           stream=stream)


def ffn_tensors(rm, T, B, D, Hd, seed, std=1.0):
    g = gen(seed)
    t = {"T": T, "B": B, "D": D}
    z = dict(dtype=torch.uint8, device="cuda")
    t["x"], t["r"] = ((std * torch.randn(B * T, D, generator=g)).bfloat16().cuda() for _ in range(2))
    t["gamma"] = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    for k, n, kk in (("W1", Hd, D), ("W2", D, Hd)):
        w = ((2 / (D + Hd)) ** 0.5 * torch.randn(T, n, kk, generator=g)).bfloat16()
        t[k + "f"] = w
        t[k], t[k + "s"] = torch.empty(T, n, kk, **z), torch.empty(T, -(-n // 128), -(-kk // 128), **z)
        rm.rm_quantize_fp8_block(w.cuda(), t[k], t[k + "s"], block_rows=128)
    t["b1"], t["b2"] = (0.1 * torch.randn(T, n, generator=g).cuda() for n in (Hd, D))
    t["s"], t["y"] = (torch.empty(B * T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    t["q"], t["qs"], t["rstd"] = torch.empty(B * T, D, **z), torch.empty(B * T, -(-D // 128), **z), torch.empty(B * T, device="cuda")
    t["h"], t["hs"] = torch.empty(T, B, Hd, **z), torch.empty(T, B, -(-Hd // 128), **z)
    return t


@pytest.mark.parametrize("T,B,D,Hd", [(4, 1, 256, 512), (4, 6, 256, 1040), (3, 150, 272, 640), (8, 256, 256, 1024)])
def test_ffn_chain(rm, T, B, D, Hd):
    """The chain against 64 bits with exact operands.  Each projection multiplies two operands rounded to e4m3
    (about 2.4 % RMS each over a binade, 3.4 % together); the second adds H's rounding and the first's error: about
    5.4 % of V, which the bf16 residual stream of equal size dilutes.  Bound: twice that."""
    t = ffn_tensors(rm, T, B, D, Hd, B + D)
    ffn(rm, t)
    torch.cuda.synchronize()
    s = h64((t["x"].float() + t["r"].float()).bfloat16())
    y, _ = R.rmsnorm(s, h64(t["gamma"]), 1e-5)
    y = y.reshape(B, T, D)
    h = R.activation(np.einsum("btd,thd->bth", y, h64(t["W1f"])) + h64(t["b1"]), "tanh")
    v = np.einsum("bth,tdh->btd", h, h64(t["W2f"])) + h64(t["b2"])
    got = h64(t["y"]).reshape(B, T, D) - s.reshape(B, T, D)
    rel = np.linalg.norm(got - v) / np.linalg.norm(v)
    assert 5e-3 < rel < 0.108, rel


def test_ffn_chain_captured(rm):
    """The chain captured on a side stream, replayed twice on new inputs: bit for bit what direct calls give, also
    while other calls run on a second stream."""
    t = ffn_tensors(rm, 4, 33, 256, 640, 1)
    u = ffn_tensors(rm, 4, 130, 256, 640, 2)
    ffn(rm, t)
    ffn(rm, u)
    torch.cuda.synchronize()
    want_u = u["y"].clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ffn(rm, t, side)
    other = torch.cuda.Stream()
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


def test_linear_backward(rm):
    """A linear layer's three products on the quantiser's operands: each equals the product of the quantised values
    in 64 bits, and the weight squares of the input gradient are the forward's own."""
    g = gen(5)
    B, N, K = 203, 272, 400
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
    assert np.array_equal(val(W, "t", 128), val(W, "", 128).T)
    for got, a, b in ((y, val(X, "", 1), val(W, "", 128)), (dx, val(DY, "", 1), val(W, "", 128).T),
                      (dw, val(DY, "t", 1), val(X, "t", 1))):
        tol = (2 * a.shape[1] / 32 + 64) * U * (np.abs(a) @ np.abs(b).T)
        assert np.all(np.abs(h64(got) - a @ b.T) <= tol)
    # against the unquantised layer: two e4m3 operands, 3.4 % RMS expected, twice that allowed
    for got, want in ((y, x @ w.T), (dx, dy @ w), (dw, dy.T @ x)):
        assert np.linalg.norm(h64(got) - h64(want)) < 0.068 * np.linalg.norm(h64(want))


# ------------------------------------------------------------------- refusals
def test_wrapper_refusals(rm):
    z = dict(dtype=torch.uint8, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    q, s = torch.zeros(4, 64, **z), torch.zeros(4, 1, **z)
    w, ws = torch.zeros(32, 64, **z), torch.zeros(1, 1, **z)
    o = torch.zeros(4, 32, device="cuda")
    bad = [
        lambda: rm.rm_rmsnorm_forward(x.cpu(), Y=x), lambda: rm.rm_rmsnorm_forward(x, Y=x.cpu()),
        lambda: rm.rm_rmsnorm_forward(x.half(), Y=x), lambda: rm.rm_rmsnorm_forward(x, x.bfloat16(), Y=x),
        lambda: rm.rm_rmsnorm_forward(x, Y=x[:3]), lambda: rm.rm_rmsnorm_forward(x.t(), Y=x.t()),
        lambda: rm.rm_rmsnorm_forward(x, gamma=torch.ones(63, device="cuda"), Y=x), lambda: rm.rm_rmsnorm_forward(x),
        lambda: rm.rm_rmsnorm_forward(x, Yq=q), lambda: rm.rm_rmsnorm_forward(x, Yq=x, Ys=s),
        lambda: rm.rm_rmsnorm_forward(x[0], Y=x[0]), lambda: rm.rm_rmsnorm_forward(x[:, 1:17], Y=x[:, :16]),
        lambda: rm.rm_rmsnorm_backward(x, x, None, torch.ones(4, device="cuda"), None, x, torch.ones(64, device="cuda")),
        lambda: rm.rm_quantize_fp8_block(x), lambda: rm.rm_quantize_fp8_block(x, q),
        lambda: rm.rm_quantize_fp8_block(x, q, s, block_rows=2), lambda: rm.rm_quantize_fp8_block(x, q, s, block_rows=128),
        lambda: rm.rm_quantize_fp8_block(x, dst_t=torch.zeros(64, 4, **z), scale_t=torch.zeros(64, 1, **z)),
        lambda: rm.rm_matmul_fp8_block(q, s, w, ws, o.half()), lambda: rm.rm_matmul_fp8_block(q, s, w, ws, o[:3]),
        lambda: rm.rm_matmul_fp8_block(q, s, w, ws, o, act="swish"), lambda: rm.rm_matmul_fp8_block(q, s, w, ws, o, w_block_rows=1),
        lambda: rm.rm_matmul_fp8_block(q, s, w, ws, torch.zeros(4, 32, **z)),
        lambda: rm.rm_matmul_fp8_block(q, s, w, ws, o, resid=o.bfloat16()), lambda: rm.rm_matmul_fp8_block(q, s, w[:, :63], ws, o),
        lambda: rm.rm_matmul_fp8_block(q[:, 8:], s, w[:, 8:], ws, o), lambda: rm.rm_matmul_fp8_block(q.cpu(), s, w, ws, o),
        lambda: rm.rm_matmul_fp8_block(q, s, w, ws, o, bias=torch.zeros(31, device="cuda")),
        lambda: rm.rm_matmul_fp8_block(q[None], s[None], w, ws, o[None]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(rm.RankMixerError) as e:
            call()
        assert e.value.status in (rm.RM_ERR_INVALID_ARG, rm.RM_ERR_UNSUPPORTED), i
    torch.cuda.synchronize()
