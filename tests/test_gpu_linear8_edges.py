"""The block-scaled 8-bit linear layer where it can go wrong: small values of GELU, gradients in place, rings of a
single row, waits that run out.

u = 2^-24 is half a step of fp32 relative to the value.
"""
import numpy as np
import pytest
import torch

import linear8_ref as R
from linear8_route import few_rows
from test_gpu_linear8 import HALF, U, bytes_of, codes_of, gen, h64, rm, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ activations
def gelu64(v, act):
    """v sigmoid(2 sqrt(2/pi) (v + 0.044715 v^3)), v Phi(v): forms without cancellation."""
    from scipy.special import expit, ndtr
    if act == "tanh":
        return v * expit(2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3))
    return v * ndtr(v)


def gelu_slack(v, act):
    """Errors relative to the result.  tanh: the sigmoid's argument 2 w (w the tanh form's) takes six roundings at most
    (v^2, three of the cubic coefficient, the sum's fma, the last product), so e^-2w is off by 6 u * 2|w| and its exp2
    by 4 u (2^-22); 1 + e rounds once, the reciprocal is good to 2 u, the product rounds once: (12 |w| + 8) u.
    erf: half of erfc(x) as t Q(t) exp(-x^2) is within 32 u of its value (a fit of 2 u at most, t and its effect 8 u,
    Horner's nine steps 10 u, the exponent's two parts and exp2 8 u, three products); where v > 0 less.
    Results below 2^-118 may be flushed to zero."""
    if act == "erf":
        return 32 * U * np.abs(gelu64(v, act)) + 2.0 ** -118
    w = np.abs(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3))
    return (12 * w + 8) * U * np.abs(gelu64(v, act)) + 2.0 ** -118


def activated(rm, v, out, act, pairs):
    """act(v) through the product: operands of zeros, v the bias.  pairs: by the CTA pairs, else by few rows."""
    M, N = (2600, v.numel()) if pairs else (5, v.numel())
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert few_rows(rm, 1, M, N, 16, out, act, sms) != pairs
    z = dict(dtype=torch.uint8, device="cuda")
    A, W = torch.zeros(M, 16, **z), torch.zeros(N, 16, **z)
    As, Ws = torch.full((M, 1), 127, **z), torch.full(((N + 127) // 128, 1), 127, **z)
    o = torch.full((M, N), 3, dtype=torch.float32).to(TYPES[out]).cuda()
    s = torch.empty(M, (N + 127) // 128, **z) if out == "e4m3" else None
    rm.rm_matmul_fp8_block(A, As, W, Ws, o, s, bias=v.cuda(), act=act)
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.uint8), o[:1].expand(M, N).contiguous().view(torch.uint8))     # every row the same
    return o[:1], None if s is None else s[:1]


SPANS = {"near zero": (-0.02, 0.02), "bulk": (-3.0, 3.0), "left": (-6.0, -2.0), "far left": (-13.5, -6.0), "wide": (-40.0, 40.0)}


@pytest.mark.parametrize("act", ["tanh", "erf"])
@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("span", SPANS)
@pytest.mark.parametrize("pairs", [False, True])
def test_gelu_is_relatively_exact(rm, act, out, span, pairs):
    """GELU keeps its relative precision where it is small (v = -3: -0.004, v = -5: -1.4e-6 by the erf form)."""
    v = torch.linspace(*SPANS[span], 1024)
    ref, slack = gelu64(h64(v), act)[None], gelu_slack(h64(v), act)[None]
    got, s = activated(rm, v, out, act, pairs)
    if out == "e4m3":
        R.assert_quantized(codes_of(got), bytes_of(s), ref, slack, act)
    else:
        err = np.abs(h64(got) - ref)
        assert np.all(err <= slack + HALF[TYPES[out]] * np.abs(ref) * 1.001), f"{np.max(err / np.maximum(np.abs(ref), 1e-37))}"


@pytest.mark.parametrize("act", ["tanh", "erf", "relu"])
@pytest.mark.parametrize("pairs", [False, True])
def test_activations_of_extremes(rm, act, pairs):
    """Infinities, NaN and values whose squares leave fp32: the definition's limits."""
    v = torch.zeros(1024)
    v[:8] = torch.tensor([float("inf"), 3e38, 1e20, -1e20, -3e38, float("nan"), 0.0, -0.0])
    for out in ("bf16", "f32"):
        got = activated(rm, v, out, act, pairs)[0][0].float().cpu()
        assert got[0] == float("inf") and bool((got[1:3] == v[1:3].to(TYPES[out]).float()).all())
        assert bool((got[3:5] == 0).all()) and bool(got[5].isnan()) and bool((got[6:] == 0).all())


# ------------------------------------------------------------- waits that run out
def bits(t):
    return t.contiguous().view(torch.uint8)


def run_out(rm, G, M, N, K, out, resid=False, act=None, pairs=False):
    """Products with wait budgets from 1 ns on: whatever ran out, each element of the results is the right one or what
    it was, and the status tells if any is missing.  The calls return and later calls are right."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert few_rows(rm, G, M, N, K, out, act, sms) != pairs
    g = torch.Generator("cuda").manual_seed(K)
    nb = (K + 127) // 128
    A, W = (torch.randn(G, n, K, generator=g, device="cuda").to(torch.float8_e4m3fn) for n in (M, N))
    As, Ws = (torch.full((G, n, nb), 120, dtype=torch.uint8, device="cuda") for n in (M, -(-N // 128)))
    r = torch.randn(G, M, N, generator=g, device="cuda").to(TYPES[out]) if resid else None
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")

    def call(budget):
        o = torch.full((G, M, N), 77, dtype=torch.float32, device="cuda").to(TYPES[out])
        s = torch.full((G, M, (N + 127) // 128), 77, dtype=torch.uint8, device="cuda") if out == "e4m3" else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        flush.fill_(1)      # the operands come from HBM
        rm.rm_matmul_fp8_block(A, As, W, Ws, o, s, None, act, r, 128, status, budget)
        torch.cuda.synchronize()
        return o, s, int(status)

    want, want_s, status = call(0)
    assert status == rm.RM_OK
    untouched = torch.full((1,), 77, dtype=torch.float32, device="cuda").to(TYPES[out])
    missing = []
    for budget in (1, 1, 500, 2000, 8000):
        o, s, status = call(budget)
        assert status in (rm.RM_OK, rm.RM_ERR_DEVICE_TIMEOUT)
        right = bits(o).view(-1, o.element_size()) == bits(want).view(-1, o.element_size())
        left = bits(o).view(-1, o.element_size()) == bits(untouched).view(1, -1)
        assert bool((right.all(1) | left.all(1)).all()), budget
        if s is not None:
            assert bool(((s == want_s) | (s == 77)).all()), budget
        missing.append(int((~right.all(1)).sum()))
        if status == rm.RM_OK:
            assert missing[-1] == 0 and (s is None or torch.equal(s, want_s))
        if budget == 1:
            assert status == rm.RM_ERR_DEVICE_TIMEOUT
    again, again_s, status = call(0)
    assert status == rm.RM_OK and torch.equal(bits(again), bits(want))
    assert again_s is None or torch.equal(again_s, want_s)
    print(missing, "of", want.numel())


@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("G,M,N,K", [(1, 64, 1024, 16384), (1, 20, 2048, 4096), (1, 5, 9472, 8192), (32, 4, 2048, 1536)])
def test_few_row_waits_run_out(rm, G, M, N, K, out):
    """K split over clusters of 8, 8 and 4 CTAs and not at all: a tile of which one slice gave up is not stored."""
    run_out(rm, G, M, N, K, out, resid=out == "f32")


@pytest.mark.parametrize("out,resid", [("bf16", False), ("f32", False), ("e4m3", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("G,M,N,K", [(2, 1300, 1168, 1536), (1, 2560, 2576, 4096), (5, 800, 1008, 272), (1, 2600, 1040, 16)])
def test_pair_waits_run_out(rm, G, M, N, K, out, resid):
    """The two CTAs of a pair give up apart, their producers up to a ring's length from each other."""
    run_out(rm, G, M, N, K, out, resid, None if resid else "relu", pairs=True)


# ------------------------------------------------------------- norm: rings, aliases
def check_norm(rm, rows, D, dtype, resid):
    """Forward over rows that leave the ring room for one or two of them; bounds of test_gpu_linear8.py."""
    g = gen(rows + D)
    x = (torch.randn(rows, D, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    r = torch.randn(rows, D, generator=g).to(dtype) if resid else None
    gamma = 1 + 0.2 * torch.randn(D, generator=g)
    y, s = torch.empty(rows, D, dtype=dtype, device="cuda"), torch.empty(rows, D, dtype=dtype, device="cuda") if resid else None
    q = torch.empty(rows, D, dtype=torch.uint8, device="cuda")
    qs, rstd = torch.empty(rows, (D + 127) // 128, dtype=torch.uint8, device="cuda"), torch.empty(rows, device="cuda")
    rm.rm_rmsnorm_forward(x.cuda(), r.cuda() if resid else None, gamma.cuda(), s, y, q, qs, rstd, 1e-6)
    torch.cuda.synchronize()
    st = (x.float() + r.float()).to(dtype) if resid else x
    if resid:
        assert torch.equal(s.cpu(), st)
    ref, rr = R.rmsnorm(h64(st), h64(gamma), 1e-6)
    assert np.all(np.abs(h64(rstd) - rr) <= 30 * U * rr)
    assert np.all(np.abs(h64(y) - ref) <= (32 * U + HALF[dtype]) * np.abs(ref))
    R.assert_quantized(codes_of(q), bytes_of(qs), ref, 32 * U * np.abs(ref), "norm")


@pytest.mark.parametrize("D", [8192, 11344, 11360, 11376, 12288, 14208, 14224, 16384])
@pytest.mark.parametrize("resid", [False, True])
def test_norm_wide_rows(rm, D, resid):
    """Several rows a CTA around the widths where gamma and the ring's second row no longer fit together."""
    check_norm(rm, 400, D, torch.float32, resid)


def check_grad(rm, rows, D, dtype, dsum, gamma=True, alias=None):
    """dX and dgamma against 64 bits (bounds of test_gpu_linear8.py); alias: dX written over dY or dSum."""
    g = gen(rows + D)
    s, dy = (torch.randn(rows, D, generator=g).to(dtype) for _ in range(2))
    ds = torch.randn(rows, D, generator=g).to(dtype) if dsum else None
    gam = 1 + 0.2 * torch.randn(D, generator=g) if gamma else None
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    dyd, dsd = dy.cuda(), ds.cuda() if dsum else None
    dx = {None: torch.empty(rows, D, dtype=dtype, device="cuda"), "dy": dyd, "dsum": dsd}[alias]
    dg = torch.full((D,), 5.0, device="cuda")
    ws = torch.empty(rm.rm_rmsnorm_backward_workspace_bytes(rows, D) // 4, device="cuda")
    rm.rm_rmsnorm_backward(dyd, s.cuda(), gam.cuda() if gamma else None, rstd.cuda(), dsd, dx, dg, ws)
    torch.cuda.synchronize()
    S, DY, RS = h64(s), h64(dy), h64(rstd)
    G, DS = h64(gam) if gamma else np.ones(D), h64(ds) if dsum else 0.0
    rx, rg = R.rmsnorm_grad(DY, S, G, RS, DS)
    r = RS[:, None]
    terms = r * (np.abs(DY * G) + np.abs(S) * r ** 2 * np.abs(DY * G * S).mean(1, keepdims=True)) + np.abs(DS)
    assert np.all(np.abs(h64(dx) - rx) <= 64 * U * terms + HALF[dtype] * np.abs(rx) * 1.001)
    assert np.all(np.abs(h64(dg) - rg) <= (rows + 64) * U * np.abs(DY * S * r).sum(0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("D", [8192, 9472, 12288, 14224, 16384])
def test_norm_grad_one_row_rings(rm, D, dsum, dtype):
    """Several wide rows a CTA: fp32 with dSum from 8192 on has a single row at a time in the ring."""
    check_grad(rm, 400, D, dtype, dsum)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 16), (333, 272), (3001, 256), (400, 16384)])
@pytest.mark.parametrize("alias,gamma", [("dy", True), ("dsum", True), ("dsum", False), (None, False)])
def test_norm_grad_in_place(rm, rows, D, dtype, alias, gamma):
    """dX in the place of dY or dSum, gamma left out."""
    check_grad(rm, rows, D, dtype, True, gamma, alias)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 16), (333, 272), (3001, 256), (700, 4112), (400, 16384)])
def test_norm_in_place(rm, rows, D, dtype):
    """Y in the place of X, Sum in that of R: the bits of separate outputs."""
    g = gen(rows + D)
    x, r = (torch.randn(rows, D, generator=g).to(dtype).cuda() for _ in range(2))
    gamma = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    y, s, xi, ri = torch.empty_like(x), torch.empty_like(x), x.clone(), r.clone()
    rm.rm_rmsnorm_forward(x, r, gamma, s, y)
    rm.rm_rmsnorm_forward(xi, ri, gamma, ri, xi)
    torch.cuda.synchronize()
    assert torch.equal(xi, y) and torch.equal(ri, s)
    rm.rm_rmsnorm_forward(x, gamma=gamma, Y=y)
    rm.rm_rmsnorm_forward(x, gamma=gamma, Y=x)
    torch.cuda.synchronize()
    assert torch.equal(x, y)


# ------------------------------------------------------------------- refusals
def test_wrapper_refuses_budgets_and_status(rm):
    z = dict(dtype=torch.uint8, device="cuda")
    args = (torch.zeros(4, 64, **z), torch.zeros(4, 1, **z), torch.zeros(32, 64, **z), torch.zeros(1, 1, **z),
            torch.zeros(4, 32, device="cuda"))
    word = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(wait_budget_ns=-1), dict(wait_budget_ns=1 << 64), dict(device_status=word),
               dict(device_status=word[:0]), dict(device_status=word[:1].long()), dict(device_status=word[:1].cpu())):
        with pytest.raises(rm.RankMixerError) as e:
            rm.rm_matmul_fp8_block(*args, **kw)
        assert e.value.status == rm.RM_ERR_INVALID_ARG, kw
    rm.rm_matmul_fp8_block(*args, device_status=word[:1])
    rm.rm_matmul_fp8_block(*args, device_status=word[0])
    torch.cuda.synchronize()
    assert word.tolist() == [0, 0]
