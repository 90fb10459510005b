"""The 8-bit layer on the GPU against its 64-bit reference (tests/_fp8_ref.py).

Tolerances, from the arithmetic of each call (u = 2^-24, half an fp32 step):
- quantise and pack without GELU: none.  Scaling by a power of two is exact.
- GELU: |error| <= 2^-18 |GELU(x)| for inputs in [-13, 13].  Horner's rule for
  g = log2 Phi(-z) at z = 5.5, where it is worst, has partial values 25.7, 4.5,
  0.61, 0.027, ... after 0, 1, 2, 3, ... more multiplications by z: half an ulp
  of each, times z^k, is 9.5e-7 + 1.3e-6 + 9e-7 + 4e-7 = 3.6e-6 in g, 2.5e-6
  in ln Phi; with the fit's 1.3e-7, 2.4e-7 of the exponential and u of the
  product 2.9e-6 < 2^-18 = 3.8e-6.  (In a block whose largest result is 0.1 or more, values of x < -5.5 are
  -1.05e-7 or nearer to 0 on both sides, below half the smallest code.)
- norm: the sum of squares is a chain of at most 32 fused steps, then two
  five-step trees, so 42 u relative, of which the root takes half; division,
  addition, root, two products: 5 u more.  26 u < 2^-19.
- linear: an fp32 accumulation of ceil(K / 32) MMA results, each step off by
  at most one step of the running sum (2^-23 of the sum of absolute terms E),
  the bias one more, then half a bf16 step.
- linear + GELU: the same accumulation error times max |GELU'| < 1.13, then
  the GELU's own."""

import numpy as np
import pytest

from tests import _fp8_ref as ref

pytestmark = pytest.mark.gpu

GELU_REL = 2.0 ** -18
NORM_REL = 2.0 ** -19


def _m():
    import torch
    import bit_w4a4_quantized_smooth_b200 as svdq
    return torch, svdq


def _np(t):
    import torch
    if t.element_size() == 1:
        return t.view(torch.uint8).cpu().numpy()
    return t.double().cpu().numpy()


def _dev(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _ok():
    torch, svdq = _m()
    torch.cuda.synchronize()
    assert svdq.sync_status() == (0, 0)


def _act(rng, M, K):
    """bf16 activations with large channels, zeros of both signs, an all-zero
    block and a block of tiny values."""
    torch, _ = _m()
    x = rng.normal(size=(M, K))
    x[:, rng.random(K) < 0.02] *= 60.0
    x[0, : min(K, 128)] = 0.0
    x[M // 2, 0] = -0.0
    x[M - 1, -min(K, 100):] *= 1e-38
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


# --------------------------------------------------------------- quantise --
SHAPES = [(1, 16), (1, 128), (3, 112), (5, 144), (33, 512), (127, 528), (128, 640), (129, 1040), (300, 2064),
          (2, 12288), (9477, 528), (1301, 4112)]


@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_bit_exact(M, K):
    torch, svdq = _m()
    X = _act(np.random.default_rng(M * 7 + K), M, K)
    codes, scales = svdq.quantize_fp8(X)
    _ok()
    c, s = ref.encode(_np(X))
    assert np.array_equal(_np(codes), c)
    assert np.array_equal(_np(scales), ref.tiles(s))


def test_quantize_strided_rows_into_given_outputs():
    """A column range of a wider tensor; outputs of uint8 type, dirty before."""
    torch, svdq = _m()
    W = _act(np.random.default_rng(5), 70, 1024)
    X = W[:, 384:384 + 272]
    codes = torch.full((70, 272), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((512,), 0xAA, dtype=torch.uint8, device="cuda")
    svdq.quantize_fp8(X, codes, scales)
    _ok()
    c, s = ref.encode(_np(X))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), ref.tiles(s))


def test_quantize_special_values():
    """Every exponent of bf16, E4M3 ties, the scale's borders, NaN and infinity."""
    torch, svdq = _m()
    bits = np.arange(0, 0x7F80, 1, dtype=np.int32)            # every finite positive bf16
    X = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16).cuda().view(-1, 128)
    X = torch.cat([X, -X, X.flip(0) * 1.0])
    codes, scales = svdq.quantize_fp8(X)
    _ok()
    c, s = ref.encode(_np(X))
    assert np.array_equal(_np(codes), c) and np.array_equal(_np(scales), ref.tiles(s))
    Y = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    Y[0, 5], Y[1, 7], Y[1, 200] = float("nan"), float("inf"), float("-inf")
    codes, scales = svdq.quantize_fp8(Y)
    _ok()
    v = codes.float().cpu()
    s, _ = ref.untile(_np(scales), 2, 256)
    assert torch.isnan(v[0, 5]) and torch.isnan(v).sum() == 1 and (v[0, 6:] == v[0, 6]).all()
    assert s[0, 0] == s[0, 1] and s[1, 0] == s[1, 1] == 247 and v[1, 7] == 448 and v[1, 200] == -448


@pytest.mark.parametrize("M,K", [(1, 128), (9, 400), (130, 2048)])
def test_quantize_gelu(M, K):
    torch, svdq = _m()
    rng = np.random.default_rng(K)
    X = _dev(rng.normal(size=(M, K)) * 2.5, torch.bfloat16)
    X[0, :100] = torch.linspace(-13, 13, 100)
    codes, scales = svdq.quantize_fp8(X, gelu=True)
    _ok()
    g = ref.gelu(_np(X))
    ref.assert_encodes(_np(codes), _np(scales), g, np.abs(g) * GELU_REL)


def test_gelu_over_its_range():
    """Blocks of one sign and size each, so that small results are not hidden by large ones."""
    torch, svdq = _m()
    x = np.concatenate([np.linspace(a, b, 128) for a, b in
                        ((-13, -12), (-9, -8), (-6, -5.2), (-5.6, -5.4), (-4, -3), (-1, -0.5), (-1e-3, 1e-3),
                         (-1e-30, 1e-30), (0.5, 1), (5.4, 5.6), (8, 9), (100, 1000))])
    X = _dev(x.reshape(1, -1), torch.bfloat16)
    codes, scales = svdq.quantize_fp8(X, gelu=True)
    _ok()
    g = ref.gelu(_np(X))
    ref.assert_encodes(_np(codes), _np(scales), g, np.abs(g) * GELU_REL)


@pytest.mark.parametrize("path", ["large", "small"])
def test_fused_gelu_of_deep_negative_rows(path):
    """Rows whose results are all tiny, all in the far tail, or mixed: the
    product passes x through (w the identity), so the GELU's tail is reached."""
    torch, svdq = _m()
    K = 256
    rng = np.random.default_rng(5)
    x = np.stack([np.linspace(-13, -6, K), np.linspace(-9, 0.1, K), np.linspace(-30, 3, K), np.linspace(-5.6, -5.4, K),
                  rng.normal(size=K) * 3 - 6, np.linspace(-12, 0.19, K), np.linspace(-12, 0.21, K), np.zeros(K)])
    (xc, xs), (wc, ws) = ref.encode(np.repeat(x, 40, axis=0)), ref.encode(np.eye(K))
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    t = lambda a, d: torch.from_numpy(a).cuda().view(d)
    svdq.set_linear_fp8_path(path)
    try:
        codes, scales = svdq.linear_fp8_gelu(t(xc, f8), t(ref.tiles(xs), e8), t(wc, f8), t(ref.tiles(ws), e8))
    finally:
        svdq.set_linear_fp8_path("auto")
    _ok()
    g = ref.gelu(ref.decode(xc, xs))                       # the product itself is exact
    ref.assert_encodes(_np(codes), _np(scales), g, np.abs(g) * GELU_REL)


def test_gelu_of_nan_and_infinity():
    torch, svdq = _m()
    Y = torch.ones((3, 256), dtype=torch.bfloat16, device="cuda")
    Y[0, 5], Y[1, 7], Y[2, 200] = float("nan"), float("inf"), float("-inf")
    Y[2, 201:] = -9.0
    codes, scales = svdq.quantize_fp8(Y, gelu=True)
    _ok()
    v = codes.float().cpu()
    s, _ = ref.untile(_np(scales), 3, 256)
    assert torch.isnan(v[0, 5]) and torch.isnan(v).sum() == 1 and (v[0, 6:] == v[0, 6]).all()
    assert s[1, 0] == 247 and v[1, 7] == 448 and (v[1, :7] == 0).all()
    assert v[2, 200] == 0 and s[2, 1] == s[2, 0]


# ------------------------------------------------------------------- pack --
@pytest.mark.parametrize("K,N", [(16, 8), (64, 16), (128, 128), (144, 136), (520 - 8, 264), (1040, 1000), (2064, 72)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pack_weight_bit_exact(K, N, dt):
    torch, svdq = _m()
    rng = np.random.default_rng(K + N)
    w = rng.normal(size=(K, N)) * 10.0 ** rng.uniform(-6, 3, (1, N))
    w[:, 0] = 0.0
    W = _dev(w, torch.bfloat16 if dt == "bf16" else torch.float32)
    codes, scales = svdq.pack_weight_fp8(W)
    _ok()
    c, s = ref.encode(np.ascontiguousarray(_np(W).T))
    assert np.array_equal(_np(codes), c) and np.array_equal(_np(scales), ref.tiles(s))


# ------------------------------------------------------------------- norm --
@pytest.mark.parametrize("M,K", [(1, 16), (1, 3072), (2, 128), (5, 144), (129, 528), (64, 4112), (3, 8208), (2, 16384),
                                 (1, 32768), (1300, 528), (1203, 3072), (400, 8208), (2, 20016)])
@pytest.mark.parametrize("res", ["none", "bf16", "f32"])
@pytest.mark.parametrize("gamma", [True, False])
def test_rmsnorm(M, K, res, gamma):
    torch, svdq = _m()
    rng = np.random.default_rng(M + K)
    X = _act(rng, M, K)
    R = None if res == "none" else _dev(rng.normal(size=(M, K)) * 3, torch.float32 if res == "f32" else torch.bfloat16)
    G = _dev(1 + 0.2 * rng.normal(size=K), torch.bfloat16) if gamma else None
    eps = 1e-5
    codes, scales, out, Y = svdq.rmsnorm(X, G, R, eps=eps, bf16_out=True)
    _ok()
    if R is None:
        assert out is None
        h = _np(X)
    else:
        assert torch.equal(out, (X.float() + R.float()).to(R.dtype))
        h = _np(out)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    if gamma:
        y = y * _np(G)
    err = np.abs(y) * NORM_REL
    ref.assert_encodes(_np(codes), _np(scales), y, err)
    got = _np(Y)
    ok = np.abs(y) > 1e-30
    assert (got[ok] >= ref.bf16_round(y - err)[ok]).all() and (got[ok] <= ref.bf16_round(y + err)[ok]).all()
    assert np.abs(got[~ok]).max(initial=0.0) <= 1.01e-30


def test_rmsnorm_in_place_strided_and_partial_outputs():
    """The residual stream updated in place, X a column range, one output only."""
    torch, svdq = _m()
    rng = np.random.default_rng(11)
    W = _act(rng, 40, 2048)
    X = W[:, 512:512 + 1040]
    R = _dev(rng.normal(size=(40, 1040)), torch.bfloat16)
    G = _dev(1 + 0.1 * rng.normal(size=1040), torch.bfloat16)
    a = svdq.rmsnorm(X, G, R, bf16_out=True)
    Xc = X.contiguous()
    b = svdq.rmsnorm(Xc, G, R, fp8_out=False, Y=Xc)            # Y over X
    assert b[0] is None and b[1] is None and torch.equal(b[3], a[3]) and torch.equal(b[2], a[2])
    R2 = R.clone()
    c = svdq.rmsnorm(X, G, R2, residual_out=R2)                # in place
    _ok()
    assert c[2] is R2 and torch.equal(R2, a[2]) and c[3] is None
    assert torch.equal(c[0].view(torch.uint8), a[0].view(torch.uint8))
    assert torch.equal(c[1].view(torch.uint8), a[1].view(torch.uint8))


def test_rmsnorm_rows_of_zeros_and_of_huge_values():
    """A zero row divides by sqrt(eps) alone (eps 0: 0 / 0 is NaN); a row whose
    squares leave the fp32 range gives zeros, a NaN stays in its row."""
    torch, svdq = _m()
    X = torch.ones((4, 256), dtype=torch.bfloat16, device="cuda")
    X[0] = 0.0
    X[1] = 3e38
    X[2, 3] = float("nan")
    codes, scales, _, Y = svdq.rmsnorm(X, bf16_out=True)
    _ok()
    v = codes.float()
    assert (v[0] == 0).all() and (Y[0] == 0).all()
    assert (v[1] == 0).all()
    assert torch.isnan(v[2]).all() and not torch.isnan(v[3]).any() and (Y[3] == 1).all()


# ----------------------------------------------------------------- linear --
LINEAR = [(1, 16, 8), (1, 128, 16), (2, 144, 136), (3, 528, 248), (8, 1024, 256), (9, 640, 264), (16, 2064, 520),
          (31, 512, 72), (64, 3200, 384), (127, 1168, 512), (128, 512, 128), (129, 1040, 264), (255, 400, 304),
          (256, 1024, 512), (257, 912, 776), (300, 112, 1032), (600, 1552, 1288), (5, 12288, 320), (130, 12288, 256)]


def _layer(rng, M, K, N, bias, fine=False):
    """Operands of one product as tensors and as fp64 values: x with large
    channels, a zero row, w with a zero row; blocks of very different scales."""
    torch, svdq = _m()
    x = rng.normal(size=(M, K))
    x[:, rng.random(K) < 0.02] *= 40.0
    x[M // 2] = 0.0
    w = rng.normal(size=(N, K)) / np.sqrt(K) * 2.0 ** rng.integers(-3, 4, (N, 1))
    w[N // 3] = 0.0
    (xc, xs), (wc, ws) = ref.encode(x), ref.encode(w)
    b = rng.normal(size=N) * 0.3
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    t = lambda a, d: torch.from_numpy(a).cuda().view(d)
    ten = (t(xc, f8), t(ref.tiles(xs), e8), t(wc, f8), t(ref.tiles(ws), e8), _dev(b, torch.bfloat16) if bias else None)
    xv, wv = ref.decode(xc, xs), ref.decode(wc, ws)
    y = xv @ wv.T
    E = np.abs(xv) @ np.abs(wv).T
    if bias:
        y = y + _np(ten[4])
        E = E + np.abs(_np(ten[4]))
    return ten, y, (-(-K // 32) + 1) * 2.0 ** -23 * E


@pytest.fixture(params=["auto", "large", "small"])
def path(request):
    """Each test of the product runs by shape, and on both kernels by force."""
    _, svdq = _m()
    svdq.set_linear_fp8_path(request.param)
    yield request.param
    svdq.set_linear_fp8_path("auto")


def _check_y(Y, y, acc):
    got = _np(Y)
    big = np.maximum(np.abs(got), np.abs(y)).astype(np.float32)
    half = np.spacing(big).astype(np.float64) * 65536.0 / 2.0
    bad = np.abs(got - y) > half + acc + 1e-38
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], got[bad][0], y[bad][0])


@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("bias", [True, False])
def test_linear(M, K, N, bias, path):
    torch, svdq = _m()
    ten, y, acc = _layer(np.random.default_rng(M + K + N), M, K, N, bias)
    guard = torch.full(((M + 2), N), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = svdq.linear_fp8(*ten, Y=guard[1:M + 1])
    _ok()
    _check_y(Y, y, acc)
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()


@pytest.mark.parametrize("M,K,N", [(M, K, (N + 15) // 16 * 16) for M, K, N in LINEAR])
@pytest.mark.parametrize("bias", [True, False])
def test_linear_gelu(M, K, N, bias, path):
    torch, svdq = _m()
    ten, y, acc = _layer(np.random.default_rng(M + K + N), M, K, N, bias)
    codes = torch.full((M + 2, N), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((svdq.fp8_sizes(M, N)[1] + 64,), 0x55, dtype=torch.uint8, device="cuda")
    svdq.linear_fp8_gelu(*ten, y_codes=codes[1:M + 1], y_scales=scales[:-64])
    _ok()
    g = ref.gelu(y)
    ref.assert_encodes(codes[1:M + 1].cpu().numpy(), scales[:-64].cpu().numpy(), g, 1.13 * acc + np.abs(g) * GELU_REL)
    assert (codes[0] == 0x55).all() and (codes[M + 1] == 0x55).all() and (scales[-64:] == 0x55).all()


@pytest.mark.parametrize("K", [272, 1552])
def test_linear_many_tiles(K):
    """More than two output tiles for each CTA pair: both accumulators reused."""
    torch, svdq = _m()
    M, N = 6000, 2064
    ten, y, acc = _layer(np.random.default_rng(K), M, K, N, True)
    _check_y(svdq.linear_fp8(*ten), y, acc)
    codes, scales = svdq.linear_fp8_gelu(*ten)
    _ok()
    rows = np.concatenate([np.arange(0, M, 9), np.arange(M - 40, M)])
    s, rest = ref.untile(_np(scales), M, N)
    assert not _np(scales)[rest].any()
    g = ref.gelu(y[rows])
    ref.assert_encodes(_np(codes)[rows], ref.tiles(s[rows]), g, 1.13 * acc[rows] + np.abs(g) * GELU_REL)


def test_linear_nan_stays_in_its_row(path):
    torch, svdq = _m()
    for M in (4, 17, 200):
        ten, y, acc = _layer(np.random.default_rng(M), M, 640, 264, False)
        xc = ten[0].view(torch.uint8).clone()
        xc[3, 500] = 0x7F
        Y = svdq.linear_fp8(xc, *ten[1:])
        _ok()
        assert torch.isnan(Y[3]).sum() >= 263                  # the zero row of w: NaN * 0 is NaN too
        assert not torch.isnan(Y[:3]).any() and not torch.isnan(Y[4:]).any()


def test_linear_same_bits_again(path):
    torch, svdq = _m()
    for M, K, N in ((5, 4096, 520), (70, 4096, 384), (300, 2064, 776)):
        ten, _, _ = _layer(np.random.default_rng(M), M, K, N, True)
        a = svdq.linear_fp8(*ten)
        for _ in range(3):
            assert torch.equal(a, svdq.linear_fp8(*ten))
    _ok()


# ----------------------------------------------------- as they are used --
def _mlp(svdq, L, X, R):
    """norm -> up + GELU -> down, the residual stream updated in place."""
    xc, xs, R, _ = svdq.rmsnorm(X, L["gamma"], R, residual_out=R)
    hc, hs = svdq.linear_fp8_gelu(xc, xs, L["uc"], L["us"], L["ub"])
    return svdq.linear_fp8(hc, hs, L["dc"], L["ds"], L["db"])


def _mlp_weights(svdq, torch, rng, D, H):
    bf = torch.bfloat16
    uc, us = svdq.pack_weight_fp8(_dev(rng.normal(size=(D, H)) / np.sqrt(D), bf))
    dc, ds = svdq.pack_weight_fp8(_dev(rng.normal(size=(H, D)) / np.sqrt(H), torch.float32))
    return dict(gamma=_dev(1 + 0.1 * rng.normal(size=D), bf), uc=uc, us=us, ub=_dev(rng.normal(size=H) * 0.1, bf),
                dc=dc, ds=ds, db=_dev(rng.normal(size=D) * 0.1, bf))


@pytest.mark.parametrize("M", [1, 7, 48, 200])
def test_mlp_chain(M):
    """Two blocks in a row against the same chain in 64 bits, each step on what
    the step before really gave; then against the unfused calls, bit for bit."""
    torch, svdq = _m()
    rng = np.random.default_rng(M)
    D, H = 512, 1424
    L = _mlp_weights(svdq, torch, rng, D, H)
    X = _dev(rng.normal(size=(M, D)), torch.bfloat16)
    R = _dev(rng.normal(size=(M, D)), torch.float32)
    R1 = R.clone()
    Y = _mlp(svdq, L, X, R1)
    Y2 = _mlp(svdq, L, Y, R1)
    _ok()
    Rr = R.clone()
    for x, want in ((X, Y), (Y, Y2)):
        xc, xs, Rr, Yb = svdq.rmsnorm(x, L["gamma"], Rr, bf16_out=True)
        hc, hs = svdq.linear_fp8_gelu(xc, xs, L["uc"], L["us"], L["ub"])
        got = svdq.linear_fp8(hc, hs, L["dc"], L["ds"], L["db"])
        assert torch.equal(got, want)
        s, _ = ref.untile(_np(hs), M, H)
        ws, _ = ref.untile(_np(L["ds"]), D, H)
        hv, wv = ref.decode(_np(hc), s), ref.decode(_np(L["dc"]), ws)
        acc = (-(-H // 32) + 1) * 2.0 ** -23 * (np.abs(hv) @ np.abs(wv).T + np.abs(_np(L["db"])))
        _check_y(got, hv @ wv.T + _np(L["db"]), acc)
    assert torch.equal(R1, Rr)
    _ok()


def test_mlp_chain_on_streams_and_in_graphs():
    """The chain on a side stream, two chains at once, and captured twice with
    replays interleaved: the same bits as on the default stream."""
    torch, svdq = _m()
    rng = np.random.default_rng(3)
    D, H = 512, 1040
    L = _mlp_weights(svdq, torch, rng, D, H)
    Xs = [_dev(rng.normal(size=(m, D)), torch.bfloat16) for m in (4, 150)]
    Rs = [_dev(rng.normal(size=(m, D)), torch.bfloat16) for m in (4, 150)]
    want = [_mlp(svdq, L, x, r.clone()) for x, r in zip(Xs, Rs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(3):
        got = []
        for st, x, r in zip(streams, Xs, Rs):
            with torch.cuda.stream(st):
                got.append(_mlp(svdq, L, x, r.clone()))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs, res = [], [], []
    for x, r in zip(Xs, Rs):
        rr = r.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = _mlp(svdq, L, x, rr)
        graphs.append(g)
        outs.append(y)
        res.append(rr)
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                res[i].copy_(Rs[i])
                outs[i].fill_(float("nan"))
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    _ok()
    # the stream argument, with the current stream another one
    st = torch.cuda.Stream()
    r = Rs[0].clone()
    st.wait_stream(torch.cuda.current_stream())
    xc, xs, _, _ = svdq.rmsnorm(Xs[0], L["gamma"], r, residual_out=r, stream=st)
    hc, hs = svdq.linear_fp8_gelu(xc, xs, L["uc"], L["us"], L["ub"], stream=st)
    y = svdq.linear_fp8(hc, hs, L["dc"], L["ds"], L["db"], stream=st)
    st.synchronize()
    assert torch.equal(y, want[0])


def test_norm_feeds_the_4_bit_layer():
    """The norm's bf16 output through the 4-bit layer's own calls, beside the FP8
    output of the same read: the two layers in one block."""
    torch, svdq = _m()
    rng = np.random.default_rng(9)
    M, K, N = 40, 512, 256
    X = _dev(rng.normal(size=(M, K)), torch.bfloat16)
    R = _dev(rng.normal(size=(M, K)), torch.bfloat16)
    w = rng.normal(size=(K, N)) / np.sqrt(K)
    rc, rs = svdq.pack_residual(_dev(w, torch.float32))
    wc, ws = svdq.pack_weight_fp8(_dev(w, torch.float32))
    inv = torch.ones(K, device="cuda")
    xc, xs, h, Yn = svdq.rmsnorm(X, None, R, bf16_out=True)
    qc, qs, _ = svdq.quantize_act(Yn, inv, None)
    y4 = svdq.linear(qc, qs, None, rc, rs, None, None, M, K, N)
    y8 = svdq.linear_fp8(xc, xs, wc, ws)
    _ok()
    hv = _np(h)
    y = hv / np.sqrt((hv * hv).mean(axis=1, keepdims=True) + 1e-6) @ w
    rel = lambda t: np.linalg.norm(_np(t) - y) / np.linalg.norm(y)
    # one rounding of x and one of w to 4 bits (steps of 1/2 to 2 of 6, rms about
    # 0.1 each) or to E4M3 (rms 2^-4 / sqrt 3 = 0.036 each, at the most)
    assert rel(y8) < 0.052 and rel(y8) < rel(y4) < 0.3
    # the FP8 output equals the quantiser's of the unrounded y: within the norm's error of Yn's
    c2, s2 = svdq.quantize_fp8(Yn)
    assert (codes_differ := (c2.view(torch.uint8) != xc.view(torch.uint8)).float().mean().item()) < 0.1, codes_differ


def test_calls_leave_launch_overlap_off_unchanged():
    torch, svdq = _m()
    rng = np.random.default_rng(13)
    L = _mlp_weights(svdq, torch, rng, 512, 1040)
    X, R = (_dev(rng.normal(size=(33, 512)), torch.bfloat16) for _ in range(2))
    a = _mlp(svdq, L, X, R.clone())
    try:
        svdq.set_launch_overlap(False)
        b = _mlp(svdq, L, X, R.clone())
    finally:
        svdq.set_launch_overlap(True)
    _ok()
    assert torch.equal(a, b)


def test_binding_refusals_on_the_device():
    torch, svdq = _m()
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")
    xc, xs = svdq.quantize_fp8(z(4, 256))
    wc, ws = svdq.pack_weight_fp8(z(256, 32))
    for call in (lambda: svdq.linear_fp8(xc, xs, wc[:, :128], ws), lambda: svdq.linear_fp8(xc, xs[:-1], wc, ws),
                 lambda: svdq.linear_fp8(xc, xs, wc, ws, z(31)), lambda: svdq.linear_fp8(xc, xs, wc, ws, Y=z(4, 31)),
                 lambda: svdq.linear_fp8(xc, xs, wc, ws.cpu()), lambda: svdq.linear_fp8(xc.float(), xs, wc, ws),
                 lambda: svdq.linear_fp8_gelu(xc, xs, wc, ws, y_codes=z(4, 32)),
                 lambda: svdq.quantize_fp8(z(256, 4).t()), lambda: svdq.quantize_fp8(z(4, 256), x_scales=xs[:-1]),
                 lambda: svdq.rmsnorm(z(4, 256), z(255)), lambda: svdq.rmsnorm(z(4, 256), z(256), z(3, 256)),
                 lambda: svdq.rmsnorm(z(4, 256), z(256), z(4, 256), residual_out=z(4, 256, d=torch.float32)),
                 lambda: svdq.rmsnorm(z(4, 256), residual_out=z(4, 256)),
                 lambda: svdq.rmsnorm(z(4, 256), z(256), z(4, 512)[:, ::2]),
                 lambda: svdq.pack_weight_fp8(z(256, 64)[:, :32])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: svdq.quantize_fp8(z(4, 40)), lambda: svdq.quantize_fp8(z(0, 64)),
                 lambda: svdq.rmsnorm(z(4, 256), fp8_out=False), lambda: svdq.pack_weight_fp8(z(64, 12)),
                 lambda: svdq.linear_fp8_gelu(xc, xs, wc[:24], svdq.pack_weight_fp8(z(256, 24))[1])):
        with pytest.raises(svdq.SvdqError):
            call()
    _ok()


# -------------------------------------------------- what is easily missed --
def test_first_call_of_a_process_inside_a_capture():
    """No call needs a warm-up: attributes, maps and plans are set up on the host."""
    import subprocess
    import sys
    code = """
import torch
import bit_w4a4_quantized_smooth_b200 as svdq
X = torch.randn(4, 512, device="cuda").bfloat16()
W = torch.randn(512, 256, device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    wc, ws = svdq.pack_weight_fp8(W)
    xc, xs, _, _ = svdq.rmsnorm(X)
    hc, hs = svdq.linear_fp8_gelu(xc, xs, wc, ws)
    qc, qs = svdq.quantize_fp8(X)
    y = svdq.linear_fp8(qc, qs, wc, ws)
g.replay()
torch.cuda.synchronize()
assert svdq.sync_status()[0] == 0
assert torch.equal(y, svdq.linear_fp8(*svdq.quantize_fp8(X), *svdq.pack_weight_fp8(W)))
a = svdq.linear_fp8_gelu(*svdq.rmsnorm(X)[:2], *svdq.pack_weight_fp8(W))
assert torch.equal(hc.view(torch.uint8), a[0].view(torch.uint8))
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_offsets_beyond_32_bits():
    """Rows of X, of the weights and of their codes that start past 2^32 bytes."""
    torch, svdq = _m()
    rng = np.random.default_rng(2)
    ld, M, K = 600_000, 4100, 528                              # 4.9 GB of bf16
    big = torch.zeros((M, ld), dtype=torch.bfloat16, device="cuda")
    X = big[:, ld - K:]
    rows = [0, 1, 1789, 1790, 3579, 3580, M - 1]
    v = torch.from_numpy(rng.normal(size=(len(rows), K))).to(torch.bfloat16).cuda()
    X[rows] = v
    codes, scales = svdq.quantize_fp8(X)
    c, s = ref.encode(_np(v))
    assert np.array_equal(_np(codes[rows]), c)
    assert np.array_equal(ref.untile(_np(scales), M, K)[0][rows], s)
    want = svdq.rmsnorm(v, bf16_out=True)[3]
    assert torch.equal(svdq.rmsnorm(X, bf16_out=True)[3][rows], want)
    del big, X
    K, N = 4112, 1_048_560                                     # 4.3 GB of codes, 8.6 GB of bf16 weights
    W = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    cols = torch.tensor([0, 7, 522_301, 1_044_480, 1_044_481, N - 1])
    w = torch.from_numpy(rng.normal(size=(K, len(cols)))).to(torch.bfloat16).cuda()
    W[:, cols.cuda()] = w
    wc, ws = svdq.pack_weight_fp8(W)
    _ok()
    del W
    c, s = ref.encode(np.ascontiguousarray(_np(w).T))
    assert np.array_equal(_np(wc.view(torch.uint8)[cols.cuda()]), c)
    x = torch.from_numpy(rng.normal(size=(3, K))).to(torch.bfloat16).cuda()
    xc, xs = svdq.quantize_fp8(x)
    xv = ref.decode(_np(xc), ref.untile(_np(xs), 3, K)[0])
    wv = ref.decode(c, s)
    y, E = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for path in ("large", "small"):
        svdq.set_linear_fp8_path(path)
        try:
            Y = svdq.linear_fp8(xc, xs, wc, ws)
            gc, gs = svdq.linear_fp8_gelu(xc, xs, wc, ws)
        finally:
            svdq.set_linear_fp8_path("auto")
        _ok()
        _check_y(Y[:, cols.cuda()], y, (-(-K // 32) + 1) * 2.0 ** -23 * E)
        others = torch.ones(N, dtype=torch.bool, device="cuda")
        others[cols.cuda()] = False
        assert (Y[:, others] == 0).all()
        g = ref.gelu(y)
        top = _np(gc[:, cols.cuda()])
        sb = ref.untile(_np(gs), 3, N)[0][:, (cols // 128).numpy()]
        got = ref.E4M3[top] * np.exp2(sb.astype(np.float64) - 127)
        assert (np.abs(got - g) <= np.abs(g) * 0.0626 + 2.0 ** -10 * np.exp2(sb.astype(np.float64) - 127)).all()


def test_unaligned_rows_take_the_16_byte_path():
    """Row strides and starts that are multiples of 16 bytes but not of 32."""
    torch, svdq = _m()
    rng = np.random.default_rng(8)
    W = _dev(rng.normal(size=(70, 1048)), torch.bfloat16)
    R = _dev(rng.normal(size=(70 * 528 + 8,)), torch.float32)
    for start in (0, 8, 24):
        X = W[:, start:start + 528]
        c, s = ref.encode(_np(X))
        codes, scales = svdq.quantize_fp8(X)
        assert np.array_equal(_np(codes), c) and np.array_equal(_np(scales), ref.tiles(s))
        for res in (None, R[4:4 + 70 * 528].view(70, 528), R[:70 * 528].view(70, 528)):
            a = svdq.rmsnorm(X, None, res, bf16_out=True)
            b = svdq.rmsnorm(X.contiguous(), None, None if res is None else res.clone(), bf16_out=True)
            assert all(torch.equal(p, q) for p, q in zip(a[2:], b[2:]) if p is not None)
            assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
    _ok()


def test_zero_rows_with_eps_zero_are_nan():
    torch, svdq = _m()
    X = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    X[1] = 2.0
    codes, scales, _, Y = svdq.rmsnorm(X, eps=0.0, bf16_out=True)
    _ok()
    assert torch.isnan(Y[0]).all() and torch.isnan(codes.float()[0]).all() and (Y[1] == 1).all()


def test_two_threads_call_at_once():
    """Plans, maps and attributes are shared by the process's threads."""
    import threading
    torch, svdq = _m()
    rng = np.random.default_rng(21)
    L = _mlp_weights(svdq, torch, rng, 512, 1040)
    Xs = [_dev(rng.normal(size=(m, 512)), torch.bfloat16) for m in (3, 17, 90, 200)]
    want = [_mlp(svdq, L, x, torch.zeros_like(x)) for x in Xs]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(20):
                    j = (i + k) % len(Xs)
                    if not torch.equal(_mlp(svdq, L, Xs[j], torch.zeros_like(Xs[j])), want[j]):
                        bad.append((k, i))
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    ts = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad, bad[:3]
    _ok()


def test_few_rows_products_of_several_sizes_share_the_gpu():
    """Clusters with 64, 128 and 256 columns of tensor memory a CTA, and the
    4-bit few-rows kernel, on four streams at once: no CTA may wait for its
    cluster while it holds columns that another one's cluster needs."""
    torch, svdq = _m()
    rng = np.random.default_rng(22)
    K, N = 2048, 1536
    wc, ws = svdq.pack_weight_fp8(_dev(rng.normal(size=(K, N)), torch.bfloat16))
    X8 = [svdq.quantize_fp8(_dev(rng.normal(size=(m, K)), torch.bfloat16)) for m in (1, 40, 128)]
    rc, rs = svdq.pack_residual(_dev(rng.normal(size=(K, N)), torch.float32))
    X4 = _dev(rng.normal(size=(64, K)), torch.bfloat16)
    x4, x4s, _ = svdq.quantize_act(X4, torch.ones(K, device="cuda"), None)
    svdq.set_linear_fp8_path("small")
    svdq.set_linear_path("small")
    try:
        calls = [lambda x=x: svdq.linear_fp8(*x, wc, ws) for x in X8] + [
            lambda: svdq.linear(x4, x4s, None, rc, rs, None, None, 64, K, N)]
        want = [c() for c in calls]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in calls]
        for _ in range(10):
            got = [[] for _ in calls]
            for _ in range(10):
                for i, st in enumerate(streams):
                    with torch.cuda.stream(st):
                        got[i].append(calls[i]())
            torch.cuda.synchronize()
            assert all(torch.equal(y, w) for g, w in zip(got, want) for y in g)
    finally:
        svdq.set_linear_fp8_path("auto")
        svdq.set_linear_path("auto")
    _ok()


def test_flags_without_a_truth_value_are_refused():
    torch, svdq = _m()
    X = torch.ones((4, 256), dtype=torch.bfloat16, device="cuda")
    two = torch.ones(2)
    for call in (lambda: svdq.rmsnorm(X, bf16_out=two), lambda: svdq.rmsnorm(X, fp8_out=two),
                 lambda: svdq.quantize_fp8(X, gelu=two)):
        with pytest.raises(RuntimeError):
            call()
    _ok()


@pytest.mark.parametrize("M,K,N", [(3700, 12288, 528), (1300, 32768, 1536), (300, 262144, 272)])
def test_linear_visits_tiles_in_groups(M, K, N):
    """x too large for L2: the tiles are visited in groups of rows of tiles
    (2, 4 and 1 here), the last group smaller or equal."""
    torch, svdq = _m()
    gen = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = svdq.quantize_fp8((rand(M, K) * torch.exp(rand(M, 1))).bfloat16())
    w = svdq.pack_weight_fp8((rand(K, N) / K ** 0.5).bfloat16())
    b = rand(N).bfloat16()
    svdq.set_linear_fp8_path("large")
    try:
        Y = svdq.linear_fp8(*x, *w, b)
        codes, scales = svdq.linear_fp8_gelu(*x, *w, b)
    finally:
        svdq.set_linear_fp8_path("auto")
    _ok()
    rows = np.unique(np.concatenate([np.arange(0, M, 41), np.arange(255, M, 256), np.arange(0, M, 256), [M - 1]]))
    xv = torch.from_numpy(ref.decode(_np(x[0])[rows], ref.untile(_np(x[1]), M, K)[0][rows])).cuda()
    wv = torch.from_numpy(ref.decode(_np(w[0]), ref.untile(_np(w[1]), N, K)[0])).cuda()
    y = (xv @ wv.T + b.double()).cpu().numpy()
    acc = (-(-K // 32) + 1) * 2.0 ** -23 * (xv.abs() @ wv.abs().T + b.double().abs()).cpu().numpy()
    _check_y(Y[torch.from_numpy(rows).cuda()], y, acc)
    g = ref.gelu(y)
    s, rest = ref.untile(_np(scales), M, N)
    assert not _np(scales)[rest].any()
    ref.assert_encodes(_np(codes)[rows], ref.tiles(s[rows]), g, 1.13 * acc + np.abs(g) * GELU_REL)


@pytest.mark.parametrize("M", [1, 77, 700])
def test_outputs_made_by_a_call_are_apart(M):
    """Small outputs share an allocation: 256-byte aligned parts that do not
    overlap.  A large residual or bf16 output holds no other one's memory."""
    torch, svdq = _m()
    K = 1040
    X, R = (torch.randn((M, K), device="cuda").bfloat16() for _ in range(2))
    outs = svdq.rmsnorm(X, None, R.float(), bf16_out=True)
    want = svdq.rmsnorm(X, None, R.float(), residual_out=torch.empty((M, K), device="cuda"), Y=torch.empty_like(X),
                        x_codes=torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda"),
                        x_scales=torch.zeros(svdq.fp8_sizes(M, K)[1], dtype=torch.uint8, device="cuda"))
    _ok()
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs)
    assert all(a % 256 == 0 for a, _ in spans)
    assert all(e <= b for (_, e), (b, _) in zip(spans, spans[1:]))
    for t, w in zip(outs, want):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
        assert t.is_contiguous() and t.untyped_storage().nbytes() >= t.numel() * t.element_size()
    if M == 700:
        for t in outs[2:]:
            assert t.untyped_storage().nbytes() < t.numel() * t.element_size() + 256


@pytest.mark.parametrize("M,K,N", [(96, 3072, 9208), (77, 2064, 5000), (70, 2576, 6152), (129, 1552, 5128),
                                   (256, 3072, 3080), (127, 1040, 9600), (200, 4112, 2568)])
def test_linear_few_rows_with_many_tokens(M, K, N):
    """Two to four CTAs share a tile of more than 64 tokens (several tokens'
    partials are added at a time), and their neighbours."""
    torch, svdq = _m()
    gen = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = svdq.quantize_fp8((rand(M, K) * torch.exp(rand(M, 1))).bfloat16())
    svdq.set_linear_fp8_path("small")
    try:
        for n in (N, N // 16 * 16):
            w = svdq.pack_weight_fp8((rand(K, n) / K ** 0.5).bfloat16())
            b = rand(n).bfloat16()
            gelu = n != N or N % 16 == 0
            out = svdq.linear_fp8_gelu(*x, *w, b) if gelu else svdq.linear_fp8(*x, *w, b)
            _ok()
            xv = torch.from_numpy(ref.decode(_np(x[0]), ref.untile(_np(x[1]), M, K)[0])).cuda()
            wv = torch.from_numpy(ref.decode(_np(w[0]), ref.untile(_np(w[1]), n, K)[0])).cuda()
            y = (xv @ wv.T + b.double()).cpu().numpy()
            acc = (-(-K // 32) + 1) * 2.0 ** -23 * (xv.abs() @ wv.abs().T + b.double().abs()).cpu().numpy()
            if gelu:
                g = ref.gelu(y)
                ref.assert_encodes(_np(out[0]), _np(out[1]), g, 1.13 * acc + np.abs(g) * GELU_REL)
            else:
                _check_y(out, y, acc)
    finally:
        svdq.set_linear_fp8_path("auto")


@pytest.mark.parametrize("N", [8, 72, 136, 192, 256 + 72])
@pytest.mark.parametrize("K", [16, 640])
def test_linear_tiles_that_end_inside_n(N, K):
    """Tiles of which only the first 64 to 192 columns are stored, several for
    each CTA pair, so both accumulators meet them: a group of columns without a
    store must not let the next one overwrite what a store still reads."""
    torch, svdq = _m()
    M = 60000 + 40                                             # 235 rows of tiles for 74 pairs; the last warp rows clipped
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = svdq.quantize_fp8((rand(M, K) * torch.exp(rand(M, 1))).bfloat16())
    w = svdq.pack_weight_fp8((rand(K, N) / K ** 0.5).bfloat16())
    b = rand(N).bfloat16()
    svdq.set_linear_fp8_path("large")
    try:
        Y = svdq.linear_fp8(*x, *w, b)
        for _ in range(20):
            assert torch.equal(Y, svdq.linear_fp8(*x, *w, b))
    finally:
        svdq.set_linear_fp8_path("auto")
    _ok()
    xv = torch.from_numpy(ref.decode(_np(x[0]), ref.untile(_np(x[1]), M, K)[0])).cuda()
    wv = torch.from_numpy(ref.decode(_np(w[0]), ref.untile(_np(w[1]), N, K)[0])).cuda()
    y = (xv @ wv.T + b.double()).cpu().numpy()
    acc = (-(-K // 32) + 1) * 2.0 ** -23 * (xv.abs() @ wv.abs().T + b.double().abs()).cpu().numpy()
    _check_y(Y, y, acc)


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-39, 1e-30])
def test_rmsnorm_of_rows_near_the_bottom_of_fp32(eps):
    """Rows whose mean square is a subnormal fp32 number, with an eps of that
    size or none.  There every square, the mean, eps and their sum are off by
    half a subnormal step, 2^-150, each: 4 of them, and the root takes half."""
    torch, svdq = _m()
    rng = np.random.default_rng(17)
    h = rng.normal(size=(6, 400)) * np.array([3e-21, 1e-20, 3e-20, 6e-20, 1e-19, 1e-18])[:, None]
    X = _dev(h, torch.bfloat16)
    R = torch.zeros((6, 400), dtype=torch.float32, device="cuda")
    G = _dev(1 + 0.1 * rng.normal(size=400), torch.bfloat16)
    for res in (None, R):
        codes, scales, _, Y = svdq.rmsnorm(X, G, res, eps=eps, bf16_out=True)
        _ok()
        x = _np(X)
        s = (x * x).mean(axis=1, keepdims=True) + eps
        y = x / np.sqrt(s) * _np(G)
        err = np.abs(y) * (NORM_REL + 2.0 ** -149 / s)
        ref.assert_encodes(_np(codes), _np(scales), y, err)
        got, ok = _np(Y), np.abs(y) > 1e-30
        assert (got[ok] >= ref.bf16_round(y - err)[ok]).all() and (got[ok] <= ref.bf16_round(y + err)[ok]).all()
        assert np.abs(got[~ok]).max(initial=0.0) <= 1.01e-30


def test_calls_do_not_report_an_error_of_somebody_else():
    """A refused runtime call of the program's own, not yet looked at, is not
    taken for the launch's; and it is left for its owner."""
    import ctypes
    torch, svdq = _m()
    X = _dev(np.random.default_rng(1).normal(size=(4, 256)), torch.bfloat16)
    W = _dev(np.random.default_rng(2).normal(size=(256, 64)), torch.bfloat16)
    want = svdq.linear_fp8(*svdq.rmsnorm(X)[:2], *svdq.pack_weight_fp8(W))
    _ok()
    rt = ctypes.CDLL("libcudart.so.12")
    W32 = W.float()
    for call in (lambda: svdq.rmsnorm(X), lambda: svdq.quantize_fp8(X), lambda: svdq.pack_weight_fp8(W),
                 lambda: svdq.pack_residual(W32)):
        first = call()
        assert rt.cudaSetDevice(-1) != 0                        # refused on the host: invalid device
        got = call()
        assert rt.cudaGetLastError() != 0 and rt.cudaGetLastError() == 0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, first) if a is not None)
    assert torch.equal(want, svdq.linear_fp8(*svdq.rmsnorm(X)[:2], *svdq.pack_weight_fp8(W)))
    _ok()


def test_a_failed_call_leaves_no_error_behind():
    """A capture is ended by a synchronisation, so the calls into its stream are
    refused by the runtime: each says so itself, and no later check of the
    program (torch shares the runtime's last error) finds it again."""
    import ctypes
    torch, svdq = _m()
    X = _dev(np.random.default_rng(1).normal(size=(4, 512)), torch.bfloat16)
    wc, ws = svdq.pack_weight_fp8(_dev(np.random.default_rng(2).normal(size=(512, 64)), torch.bfloat16))
    xc, xs = svdq.quantize_fp8(X)
    Y = svdq.linear_fp8(xc, xs, wc, ws)
    inv = torch.ones(512, device="cuda")
    R = torch.ones((64, 16), device="cuda")
    q4 = svdq.quantize_act(X, inv, None)
    r4 = svdq.pack_residual(R)
    c8, s8, y8 = xc.clone(), xs.clone(), Y.clone()
    _ok()
    rt = ctypes.CDLL("libcudart.so.12")
    st = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(handle, 1) == 0             # this thread only
    try:
        assert svdq.sync_status(st)[0] == 4                      # not allowed in a capture, and ends it
        assert rt.cudaGetLastError() == 0
        for call in (lambda: svdq.quantize_fp8(X, c8, s8, stream=st),
                     lambda: svdq.rmsnorm(X, x_codes=c8, x_scales=s8, stream=st),
                     lambda: svdq.linear_fp8(xc, xs, wc, ws, Y=y8, stream=st),
                     lambda: svdq.pack_residual(R, *r4, stream=st)):
            with pytest.raises(svdq.SvdqError) as e:
                call()
            assert e.value.status == 4
            assert rt.cudaGetLastError() == 0
    finally:
        assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
    got = svdq.linear_fp8(*svdq.quantize_fp8(X, stream=st), wc, ws, stream=st)
    st.synchronize()
    assert torch.equal(got, Y)
    again = svdq.quantize_act(X, inv, None)
    assert torch.equal(again[0], q4[0]) and torch.equal(again[1], q4[1])
    _ok()


@pytest.fixture(params=range(1, 9))
def splits(request):
    _, svdq = _m()
    svdq.set_linear_fp8_path("small")
    svdq.set_linear_fp8_splits(request.param)
    yield request.param
    svdq.set_linear_fp8_splits(0)
    svdq.set_linear_fp8_path("auto")


@pytest.mark.parametrize("M", [1, 21, 64, 77, 128, 200])
def test_linear_few_rows_with_every_split(M, splits):
    """One to eight CTAs share a tile (56 stages along K: each number divides
    them so that none is left without any), up to and above the 64 tokens from
    which several tokens' partials are added at a time; K, N and the last tile
    of tokens end inside a tile."""
    torch, svdq = _m()
    K = 7056                                                   # 55 stages and a short one
    gen = torch.Generator(device="cuda").manual_seed(8 * M + splits)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = svdq.quantize_fp8((rand(M, K) * torch.exp(rand(M, 1))).bfloat16())
    for N in (280, 272):
        w = svdq.pack_weight_fp8((rand(K, N) / K ** 0.5).bfloat16())
        b = rand(N).bfloat16()
        Y = svdq.linear_fp8(*x, *w, b)
        _ok()
        xv = torch.from_numpy(ref.decode(_np(x[0]), ref.untile(_np(x[1]), M, K)[0])).cuda()
        wv = torch.from_numpy(ref.decode(_np(w[0]), ref.untile(_np(w[1]), N, K)[0])).cuda()
        y = (xv @ wv.T + b.double()).cpu().numpy()
        acc = (-(-K // 32) + splits) * 2.0 ** -23 * (xv.abs() @ wv.abs().T + b.double().abs()).cpu().numpy()
        _check_y(Y, y, acc)
        if N % 16 == 0:
            codes, scales = svdq.linear_fp8_gelu(*x, *w, b)
            _ok()
            g = ref.gelu(y)
            ref.assert_encodes(_np(codes), _np(scales), g, 1.13 * acc + np.abs(g) * GELU_REL)


def test_linear_few_rows_with_more_splits_than_stages(splits):
    """The next smaller number that leaves no CTA without a part of K: 5 stages
    are shared by 5, 3 (2 + 2 + 1), 2 or 1, and 1 stage by nobody."""
    torch, svdq = _m()
    for K in (592, 16):
        ten, y, acc = _layer(np.random.default_rng(K + splits), 9, K, 136, True)
        _check_y(svdq.linear_fp8(*ten), y, acc + 7 * acc / (-(-K // 32) + 1))
    _ok()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pack_weight_special_values(dt):
    """A NaN is the code NaN and leaves its block's scale alone; an infinity is
    +-448 with the largest scale; both stay in their channel and block."""
    torch, svdq = _m()
    K, N = 272, 24
    W = _dev(np.random.default_rng(6).normal(size=(K, N)), torch.bfloat16 if dt == "bf16" else torch.float32)
    plain, plain_s = svdq.pack_weight_fp8(W)
    V = W.clone()
    V[3, 1] = V[130, 5] = float("nan")
    V[128:256, 2] = float("nan")                               # a whole block
    V[7, 9], V[271, 10] = float("inf"), float("-inf")
    codes, scales = svdq.pack_weight_fp8(V)
    _ok()
    c, p = _np(codes), _np(plain)
    s, rest = ref.untile(_np(scales), N, K)
    sp, _ = ref.untile(_np(plain_s), N, K)
    assert not _np(scales)[rest].any()
    nan = np.zeros((N, K), dtype=bool)
    nan[1, 3] = nan[5, 130] = True
    nan[2, 128:256] = True
    assert np.array_equal(np.isnan(ref.E4M3[c]), nan)
    assert s[9, 0] == s[10, 2] == 247 and s[2, 1] == 0
    assert ref.E4M3[c[9, 7]] == 448 and ref.E4M3[c[10, 271]] == -448
    assert not ref.E4M3[c[9, :7]].any() and not ref.E4M3[c[10, 256:271]].any()
    same = np.ones((N, 3), dtype=bool)                         # blocks whose scale is an amax of what is left
    same[9, 0] = same[10, 2] = same[2, 1] = False
    v = _np(V).T.copy()
    v[np.isnan(v)] = 0.0
    v[9, :128] = v[10, 256:] = 0.0
    want, ws = ref.encode(v)
    assert np.array_equal(s[same], ws[same])
    keep = np.repeat(same, 128, axis=1)[:, :K] & ~nan
    assert np.array_equal(c[keep], want[keep])
    others = [0, 3, 4, 6, 7, 8] + list(range(11, N))
    assert np.array_equal(c[others], p[others]) and np.array_equal(s[others], sp[others])


@pytest.mark.parametrize("res", ["none", "bf16", "f32"])
def test_rmsnorm_of_infinities(res):
    """An infinite h: inf / inf is NaN in its element, and the rest of its row is
    divided by infinity.  An infinite or overflowing gamma: NaN in its column.
    The other rows are what they are without."""
    torch, svdq = _m()
    K = 400
    X = _dev(np.random.default_rng(7).normal(size=(5, K)), torch.bfloat16)
    R = None if res == "none" else torch.ones((5, K), dtype=torch.float32 if res == "f32" else torch.bfloat16, device="cuda")
    plain = svdq.rmsnorm(X, None, R, bf16_out=True)
    V = X.clone()
    V[1, 5], V[3, 300] = float("inf"), float("-inf")
    codes, scales, h, Y = svdq.rmsnorm(V, None, R, bf16_out=True)
    _ok()
    v, y = ref.E4M3[_np(codes)], _np(Y)
    s, rest = ref.untile(_np(scales), 5, K)
    assert not _np(scales)[rest].any() and not s[1].any() and not s[3].any()
    for row, col in ((1, 5), (3, 300)):
        assert np.isnan(v[row, col]) and np.isnan(y[row, col])
        assert not np.delete(v[row], col).any() and not np.delete(y[row], col).any()
    ok = [0, 2, 4]
    assert np.array_equal(_np(codes)[ok], _np(plain[0])[ok]) and torch.equal(Y[ok], plain[3][ok])
    if h is not None:
        assert h[1, 5] == float("inf") and h[3, 300] == float("-inf")
    G = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    G[17] = float("inf")
    Y = svdq.rmsnorm(X, G, R, fp8_out=False, bf16_out=True)[3]
    _ok()
    assert torch.isnan(Y[:, 17]).all() and torch.isnan(Y).sum() == 5
    Y[:, 17] = plain[3][:, 17]
    assert torch.equal(Y, plain[3])


def test_linear_of_nan_and_large_scales(path):
    """The scale byte 255 is NaN: of x it takes its token, of w its channel.
    Products beyond bf16 and fp32 are infinite, and 448 2^120 as FP8."""
    torch, svdq = _m()
    rng = np.random.default_rng(8)
    for M in (5, 150):
        K, N = 640, 272
        (xc, xs, wc, ws, b), y, acc = _layer(rng, M, K, N, True)
        at = lambda row, blk: (blk // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + blk % 4  # of the first band
        xs, ws = xs.view(torch.uint8).clone(), ws.view(torch.uint8).clone()
        xs[at(3, 2)] = 255
        ws[at(40, 4)] = 255
        Y = svdq.linear_fp8(xc, xs, wc, ws, b)
        codes, scales = svdq.linear_fp8_gelu(xc, xs, wc, ws, b)
        _ok()
        nan = np.zeros((M, N), dtype=bool)
        nan[3], nan[:, 40] = True, True
        assert np.array_equal(np.isnan(_np(Y)), nan)
        assert np.array_equal(np.isnan(ref.E4M3[_np(codes)]), nan)
        _check_y(torch.where(torch.from_numpy(nan).cuda(), 0.0, Y), np.where(nan, 0.0, y), acc)
        keep = np.array([r for r in range(M) if r != 3])
        s, _ = ref.untile(_np(scales), M, N)
        g = np.where(nan, 0.0, ref.gelu(y))[keep]              # a NaN does not change its block's scale
        c = np.where(nan, 0, _np(codes)).astype(np.uint8)[keep]
        ref.assert_encodes(c, ref.tiles(s[keep]), g, 1.13 * acc[keep] + np.abs(g) * GELU_REL)
    x = torch.full((2, 256), 3e38, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((256, 256), dtype=torch.float32, device="cuda")
    w[0, 0], w[0, 1], w[0, 2] = 2.0, -2.0, 1.0
    q, p = svdq.quantize_fp8(x), svdq.pack_weight_fp8(w)
    Y = svdq.linear_fp8(*q, *p)
    codes, scales = svdq.linear_fp8_gelu(*q, *p)
    _ok()
    assert (Y[:, 0] == float("inf")).all() and (Y[:, 1] == float("-inf")).all() and torch.isfinite(Y[:, 2]).all()
    assert not Y[:, 3:].any()
    v, s = ref.E4M3[_np(codes)], ref.untile(_np(scales), 2, 256)[0]
    assert (s[:, 0] == 247).all() and (v[:, 0] == 448).all() and not v[:, 1].any() and not v[:, 3:].any()


def test_given_outputs_are_seen_by_autograd_as_written():
    """A tensor saved for a backward pass and then given as an output: the pass
    is refused, as after any in-place operation.  Inference tensors may be given."""
    torch, svdq = _m()
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")
    X = torch.ones((4, 256), dtype=torch.bfloat16, device="cuda")
    wc, ws = svdq.pack_weight_fp8(z(256, 32))
    xc, xs = svdq.quantize_fp8(X)
    R, Y, Y2 = z(4, 256), z(4, 256), z(4, 32)
    for out, call in ((R, lambda: svdq.rmsnorm(X, None, R, residual_out=R)), (Y, lambda: svdq.rmsnorm(X, Y=Y)),
                      (Y2, lambda: svdq.linear_fp8(xc, xs, wc, ws, Y=Y2))):
        a = torch.ones_like(out, requires_grad=True)
        loss = (a * out).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    c, s = z(4, 256, d=torch.uint8), z(512, d=torch.uint8)
    hc, hs = z(4, 32, d=torch.uint8), z(512, d=torch.uint8)
    pc, ps = z(32, 256, d=torch.uint8), z(512, d=torch.uint8)
    for outs, call in (((c, s), lambda: svdq.quantize_fp8(X, c, s)), ((c, s), lambda: svdq.rmsnorm(X, x_codes=c, x_scales=s)),
                       ((pc, ps), lambda: svdq.pack_weight_fp8(z(256, 32), pc, ps)),
                       ((hc, hs), lambda: svdq.linear_fp8_gelu(xc, xs, wc, ws, None, hc, hs))):
        before = [t._version for t in outs]
        call()
        assert [t._version for t in outs] == [v + 1 for v in before]
    with torch.inference_mode():
        I = z(4, 32)
    assert svdq.linear_fp8(xc, xs, wc, ws, Y=I) is I
    with torch.inference_mode():
        assert svdq.linear_fp8(xc, xs, wc, ws, Y=I) is I and svdq.rmsnorm(X, Y=Y)[3] is Y
    _ok()


@pytest.mark.parametrize("M,K", [(9481, 528), (1583, 6160), (9470, 528)])
def test_quantize_gelu_many_rows(M, K):
    """Enough rows that a warp takes four (not so in the last): rows and columns end inside its share."""
    torch, svdq = _m()
    gen = torch.Generator(device="cuda").manual_seed(M)
    X = (torch.randn((M, K), generator=gen, device="cuda") * 2.0).bfloat16()
    X[:, 128:256] -= 8.0                                       # blocks without a value above 0.3
    codes, scales = svdq.quantize_fp8(X, gelu=True)
    _ok()
    g = ref.gelu(_np(X))
    ref.assert_encodes(_np(codes), _np(scales), g, np.abs(g) * GELU_REL)


@pytest.mark.parametrize("M,K,N", [(1 << 22, 16, 16), (3, 16, 1 << 22), (3, 1 << 20, 16), (1, 16, 8)])
def test_the_largest_and_the_smallest_sizes(M, K, N):
    """Every size at its limit once, the others small; both kernels, both outputs."""
    torch, svdq = _m()
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    X = rand(M, K).bfloat16()
    W = rand(K, N) / K ** 0.5
    rows = np.unique(np.concatenate([np.arange(min(M, 300)), np.arange(max(0, M - 300), M), np.arange(0, M, 65521)]))
    cols = np.unique(np.concatenate([np.arange(min(N, 300)), np.arange(max(0, N - 300), N), np.arange(0, N, 65521)]))
    rt, ct = torch.from_numpy(rows).cuda(), torch.from_numpy(cols).cuda()
    (xc, xs), (wc, ws) = svdq.quantize_fp8(X), svdq.pack_weight_fp8(W)
    _ok()
    c, s = ref.encode(_np(X[rt]))
    assert np.array_equal(_np(xc.view(torch.uint8)[rt]), c)
    assert np.array_equal(ref.untile(_np(xs), M, K)[0][rows], s)
    wr, wsr = ref.encode(np.ascontiguousarray(_np(W[:, ct]).T))
    assert np.array_equal(_np(wc.view(torch.uint8)[ct]), wr)
    assert np.array_equal(ref.untile(_np(ws), N, K)[0][cols], wsr)
    xv, wv = ref.decode(c, s), ref.decode(wr, wsr)
    y, acc = xv @ wv.T, (-(-K // 32) + 8) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T)
    for path in ("large", "small"):
        svdq.set_linear_fp8_path(path)
        try:
            Y = svdq.linear_fp8(xc, xs, wc, ws)
            _ok()
            _check_y(Y[rt][:, ct], y, acc)
            del Y
            if N % 16 == 0 and N <= 1 << 20:
                codes, scales = svdq.linear_fp8_gelu(xc, xs, wc, ws)
                _ok()
                sc = ref.untile(_np(scales), M, N)[0][rows]
                g = ref.gelu(y)
                ref.assert_encodes(_np(codes.view(torch.uint8)[rt]), ref.tiles(sc), g, 1.13 * acc + np.abs(g) * GELU_REL)
        finally:
            svdq.set_linear_fp8_path("auto")
    if K <= 32768:
        Yn = svdq.rmsnorm(X, fp8_out=False, bf16_out=True, eps=1e-5)[3]
        h = _np(X[rt])
        n = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + 1e-5)
        got, err = _np(Yn[rt]), np.abs(n) * NORM_REL
        assert (got >= ref.bf16_round(n - err)).all() and (got <= ref.bf16_round(n + err)).all()
    _ok()


def test_the_default_stream_and_foreign_streams_as_arguments():
    """The stream argument may be the default stream while another is current, or
    a stream that torch did not make."""
    import ctypes
    torch, svdq = _m()
    rng = np.random.default_rng(31)
    L = _mlp_weights(svdq, torch, rng, 512, 1040)
    X, R = (_dev(rng.normal(size=(20, 512)), torch.bfloat16) for _ in range(2))
    want = _mlp(svdq, L, X, R.clone())
    torch.cuda.synchronize()
    rt, h = ctypes.CDLL("libcudart.so.12"), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0
    try:
        for st in (torch.cuda.default_stream(), torch.cuda.ExternalStream(h.value)):
            r = R.clone()
            torch.cuda.synchronize()
            with torch.cuda.stream(torch.cuda.Stream()):
                xc, xs, _, _ = svdq.rmsnorm(X, L["gamma"], r, residual_out=r, stream=st)
                hc, hs = svdq.linear_fp8_gelu(xc, xs, L["uc"], L["us"], L["ub"], stream=st)
                y = svdq.linear_fp8(hc, hs, L["dc"], L["ds"], L["db"], stream=st)
            st.synchronize()
            assert torch.equal(y, want)
            del xc, xs, hc, hs, y
        torch.cuda.synchronize()
        torch.cuda.empty_cache()                               # the foreign stream's blocks
    finally:
        assert rt.cudaStreamDestroy(h) == 0
    _ok()
