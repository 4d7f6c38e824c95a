"""The mixture-of-experts layer on the GPU, stage by stage against its 64-bit form: logits
within the bound of a binary32 sum, the choice of experts exact for the kernel's own logits,
then probabilities, h and Y each from the stage before it, so that no bound has to cover a
rounding that went the other way earlier."""
import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import fp8_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _layer(d, f, E, k, gated, renorm, rt, seed, kind=0, router=None):
    rng = np.random.default_rng(seed)
    r = (rng.standard_normal((E, d)) * 2 / np.sqrt(d)).astype(np.float32) if router is None else router
    if rt == BF16:
        r = R.bf16(r)
    mats = {}
    for name, shape in (("gate", (E, f, d)), ("up", (E, f, d)), ("down", (E, d, f))):
        if name == "gate" and not gated:
            continue
        w = (rng.standard_normal(shape) * 0.05).astype(np.float32)
        packed = B.w4a4_fp8_pack_weights(torch.from_numpy(w).cuda(), kind)
        v = packed.views()
        c, s = v["codes"].cpu().numpy(), v["scales"].cpu().numpy()
        mats[name] = (packed, [R.dequant_blocks(c[e], s[e]) for e in range(E)])
    layer = B.moe_layer(torch.from_numpy(r).to(rt).cuda(), mats["gate"][0] if gated else None, mats["up"][0], mats["down"][0], k, renorm)
    return layer, r, mats


def _act(g, u):
    if g is not None:
        with np.errstate(over="ignore"):
            return g / (1 + np.exp(-g)) * u
    return 0.5 * u * (1 + np.tanh(np.sqrt(2 / np.pi) * (u + 0.044715 * u ** 3)))


def _check(x, xt, layer, r, mats, yt):
    T, d = x.shape
    E, k, f, renorm, gated = layer.n_experts, layer.top_k, layer.f, layer.desc.renormalize, "gate" in mats
    print(f"moe T={T} d={d} f={f} E={E} k={k} gated={gated} renorm={renorm} x={xt} y={yt}", flush=True)
    ws = torch.full((B.w4a4_moe_workspace_size(T, layer) + 512,), 255, dtype=torch.uint8, device="cuda")
    xbuf = torch.full((T * d + 512,), float("nan"), dtype=xt, device="cuda")
    X = xbuf[256:256 + T * d].view(T, d)
    X.copy_(torch.from_numpy(x))
    ybuf = torch.full((T * d + 512,), 7.0, dtype=yt, device="cuda")
    Y = ybuf[256:256 + T * d].view(T, d)
    B.w4a4_moe_forward(X, layer, Y, ws[:-512])
    torch.cuda.synchronize()
    assert bool((ws[-512:] == 255).all()) and bool((ybuf[:256] == 7).all()) and bool((ybuf[256 + T * d:] == 7).all())
    v = {n: t.float().cpu().numpy() if n != "ids" else t.cpu().numpy() for n, t in B.workspace_moe_views(ws, T, layer).items()}

    x64, r64 = x.astype(np.float64), r.astype(np.float64)
    with np.errstate(all="ignore"):
        l64, mag = x64 @ r64.T, np.abs(x64) @ np.abs(r64).T
    R.close(v["logits"], l64, (d + 8) * 2.0 ** -24 * mag, "logits")
    ids = R.topk(v["logits"], k)
    assert np.array_equal(v["ids"], ids), "chosen experts differ"
    with np.errstate(all="ignore"):
        l = v["logits"].astype(np.float64)
        ex = np.exp(l - np.where(np.isnan(l).any(1), np.nan, l.max(1))[:, None])
        p = np.take_along_axis(ex, ids, 1)
        if not renorm:
            p = p / ex.sum(1, keepdims=True)
        ptol = (E + 64) * 2.0 ** -23
        R.close(v["p"], p, ptol * np.abs(p), "p")
        if renorm:
            p = p / p.sum(1, keepdims=True)

    xb = R.bf16(x).astype(np.float64) if xt == F32 else x64
    if xt == F32:
        xb = np.where(np.isnan(x64), np.nan, xb)
    y, ytol = np.zeros((T, d)), np.zeros((T, d))
    nkb = -(-d // 128)
    for e in range(E):
        tt, rk = np.nonzero(ids == e)
        if not len(tt):
            continue
        u, du = R.product(xb[tt], mats["up"][1][e])
        g = dg = None
        with np.errstate(all="ignore"):
            if gated:
                g, dg = R.product(xb[tt], mats["gate"][1][e])
                sg = np.abs(g / (1 + np.exp(-g)))
                dh = 1.1 * dg * (np.abs(u) + du) + sg * du
            else:
                dh = 1.13 * du
            h = _act(g, u)
            # exp, the division or the reciprocal, and the products: a few binary32 units; the
            # GELU's far tail ends in binary32's subnormals
            dh = dh + 2.0 ** -19 * np.abs(h) + 2.0 ** -120
            R.close(v["h"][tt, rk], h, dh + R.BF16_U * (np.abs(h) + dh), f"h of expert {e}")
            hk = v["h"][tt, rk].astype(np.float64)
            part, dp = R.product(hk, mats["down"][1][e])
            mag = np.abs(hk) @ np.abs(mats["down"][1][e]).T
            pe = p[tt, rk][:, None]
            np.add.at(y, tt, pe * part)
            np.add.at(ytol, tt, pe * (dp + (2 * ptol + (k + 24) * 2.0 ** -23) * mag))
    if yt == BF16:
        ytol = ytol + R.BF16_U * (np.abs(y) + ytol)
    R.close(Y.double().cpu().numpy(), y, ytol, "Y")
    return Y, v


def _tokens(T, d, dtype, seed):
    x = (np.random.default_rng(seed).standard_normal((T, d)) * 0.7).astype(np.float32)
    return R.bf16(x) if dtype == BF16 else x


@pytest.mark.parametrize("T,d,f,E,k", [(1, 1, 1, 1, 1), (1, 128, 16, 4, 2), (1, 500, 130, 40, 8), (2, 260, 33, 7, 7), (3, 129, 257, 20, 4),
                                       (5, 384, 128, 64, 6), (16, 200, 100, 6, 3), (17, 136, 300, 4, 4), (40, 333, 48, 12, 2), (64, 256, 160, 3, 2),
                                       (65, 128, 40, 2, 1), (128, 130, 72, 5, 3), (4, 64, 24, 300, 9), (1, 96, 16, 1024, 32)])
def test_shapes(T, d, f, E, k):
    for gated, renorm, xt, rt, yt in [(True, True, BF16, BF16, BF16), (False, False, F32, F32, F32)]:
        layer, r, mats = _layer(d, f, E, k, gated, renorm, rt, T + d)
        _check(_tokens(T, d, xt, 3), xt, layer, r, mats, yt)


@pytest.mark.parametrize("gated,renorm,xt,rt,yt,kind", [(True, False, BF16, F32, F32, 0), (True, True, F32, BF16, BF16, 1),
                                                        (False, True, BF16, BF16, F32, 1), (False, False, F32, F32, BF16, 0)])
def test_variants(gated, renorm, xt, rt, yt, kind):
    layer, r, mats = _layer(272, 144, 10, 3, gated, renorm, rt, 50, kind)
    _check(_tokens(21, 272, xt, 51), xt, layer, r, mats, yt)


@pytest.mark.parametrize("T", [1, 2, 70])
def test_ties_go_to_the_lowest_index(T):
    """Zero tokens tie every logit at 0; equal router rows tie in pairs."""
    rng = np.random.default_rng(60)
    router = np.repeat((rng.standard_normal((8, 64)) / 4).astype(np.float32), 2, axis=0)
    layer, r, mats = _layer(64, 32, 16, 3, True, True, BF16, 61, router=router)
    x = _tokens(T, 64, BF16, 62)
    x[0] = 0
    if T > 1:
        x[1] = -0.0
    _, v = _check(x, BF16, layer, r, mats, F32)
    assert v["ids"][0].tolist() == [0, 1, 2]


@pytest.mark.parametrize("T", [20, 64, 128])
def test_every_token_on_one_expert(T):
    """One expert takes all tokens (several token tiles), the others one token or none."""
    rng = np.random.default_rng(70)
    router = (rng.standard_normal((9, 160)) * 0.01).astype(np.float32)
    router[5, 0] = 30
    x = _tokens(T, 160, BF16, 71)
    x[:, 0] = 1
    layer, r, mats = _layer(160, 80, 9, 2, True, True, BF16, 72, router=router)
    _, v = _check(x, BF16, layer, r, mats, BF16)
    assert (v["ids"][:, 0] == 5).all()


@pytest.mark.parametrize("T", [2, 30])
def test_nan_and_infinite_tokens(T):
    """A token with a NaN takes the lowest experts, gives a NaN row and touches no other; an
    infinite value goes through the formula."""
    layer, r, mats = _layer(192, 64, 12, 3, True, True, BF16, 80)
    x = _tokens(T, 192, BF16, 81)
    clean, _ = _check(x, BF16, layer, r, mats, F32)
    x[1, 17] = np.nan
    Y, v = _check(x, BF16, layer, r, mats, F32)
    assert v["ids"][1].tolist() == [0, 1, 2] and bool(torch.isnan(Y[1]).all())
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(Y[keep], clean[keep])


@pytest.mark.parametrize("T,E,k", [(1, 32, 4), (6, 16, 3), (33, 8, 2)])
def test_streams_repeats_and_graphs(T, E, k):
    layer, r, mats = _layer(300, 140, E, k, True, True, BF16, 90)
    X = torch.from_numpy(_tokens(T, 300, BF16, 91)).to(BF16).cuda()
    ws, Y = B.alloc_workspace_moe(T, layer), torch.empty(T, 300, device="cuda")
    print(f"moe repeats T={T} E={E} k={k}", flush=True)
    B.w4a4_moe_forward(X, layer, Y, ws)
    torch.cuda.synchronize()
    ref = Y.clone()
    s = torch.cuda.Stream()
    Y.fill_(float("nan"))
    torch.cuda.synchronize()
    B.w4a4_moe_forward(X, layer, Y, ws, s)
    s.synchronize()
    assert torch.equal(Y, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.w4a4_moe_forward(X, layer, Y, ws)
    for i in range(4):
        Y.fill_(float("nan"))
        ws.fill_(255 if i % 2 else 0)
        (X.float() @ torch.ones(300, 8, device="cuda")).sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref)


def test_binding_refusals():
    up = B.w4a4_fp8_pack_weights(torch.randn(4, 24, 40, device="cuda"))
    down = B.w4a4_fp8_pack_weights(torch.randn(4, 40, 24, device="cuda"))
    router = torch.randn(4, 40, device="cuda")
    layer = B.moe_layer(router, None, up, down, 2)
    X, Y, ws = torch.zeros(3, 40, device="cuda"), torch.zeros(3, 40, device="cuda"), B.alloc_workspace_moe(3, layer)
    for args, exc in [((X.half(), layer, Y, ws), TypeError), ((X, layer, Y[:, :39], ws), ValueError), ((X[:2], layer, Y, ws), ValueError),
                      ((X, layer, Y, ws[:256]), B.W4A4Error), ((X, layer, Y, ws[8:]), B.W4A4Error)]:
        with pytest.raises(exc):
            B.w4a4_moe_forward(*args)
    big = torch.zeros(B.MOE_MAX_T + 1, 40, device="cuda")
    with pytest.raises(B.W4A4Error):
        B.w4a4_moe_forward(big, layer, torch.zeros_like(big), ws)
    for bad in (dict(top_k=0), dict(top_k=5)):
        with pytest.raises(B.W4A4Error):
            B.moe_layer(router, None, up, down, **bad)
    with pytest.raises(B.W4A4Error):
        B.moe_layer(router, None, up, up, 2)
    with pytest.raises(ValueError):
        B.moe_layer(router[:3], None, up, down, 2)


@pytest.mark.parametrize("T,d,f,E,k,gated", [(1, 260, 1600, 8, 8, True), (12, 260, 1600, 8, 3, True), (7, 131, 1000, 10, 4, False),
                                             (40, 260, 1600, 6, 3, True), (40, 4100, 1700, 2, 2, False), (100, 200, 900, 5, 3, True),
                                             (2, 8300, 100, 2, 1, False), (64, 300, 400, 40, 6, True)])
def test_divided_down_tiles(T, d, f, E, k, gated):
    """Sizes at which several workgroups share a tile of outputs, or one takes several, and the
    passes over codes of 4, 8 and 16 tokens and of two row tiles; twice, for the same bits."""
    layer, r, mats = _layer(d, f, E, k, gated, True, BF16, T + d)
    x = _tokens(T, d, BF16, 5)
    Y, _ = _check(x, BF16, layer, r, mats, F32)
    ws, again = B.alloc_workspace_moe(T, layer), torch.empty_like(Y)
    X = torch.from_numpy(x).to(BF16).cuda()
    for _ in range(3):
        again.fill_(float("nan"))
        B.w4a4_moe_forward(X, layer, again, ws)
        assert torch.equal(again, Y)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.w4a4_moe_forward(X, layer, again, ws)
    for _ in range(3):
        again.fill_(float("nan"))
        (X.float() @ torch.ones(d, 8, device="cuda")).sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, Y)


@pytest.mark.parametrize("T,d,f,E,k", [(1, 260, 1600, 8, 8), (12, 260, 1600, 8, 3), (40, 4100, 1700, 2, 2), (64, 300, 400, 40, 6)])
def test_workspace_used_again_with_other_tokens(T, d, f, E, k):
    """Parts of an earlier call never reach a later one's sums."""
    layer, _, _ = _layer(d, f, E, k, True, True, BF16, 90)
    ws, Y = B.alloc_workspace_moe(T, layer), torch.empty(T, d, device="cuda")
    xs = [torch.from_numpy(_tokens(T, d, BF16, 91 + i)).to(BF16).cuda() for i in range(3)]
    want = []
    for x in xs:
        B.w4a4_moe_forward(x, layer, Y, B.alloc_workspace_moe(T, layer))
        want.append(Y.clone())
    for i in (0, 1, 2, 1, 0, 2, 0, 2, 1):
        B.w4a4_moe_forward(xs[i], layer, Y, ws)
        assert torch.equal(Y, want[i])


# Many tokens in passes of four tokens (T k <= E) and eight (T k <= 3 E), found by slots (T k < E <= 256)
# or by counting; down steps for 17 to 64 and 65 to 128 tokens, whole tiles and divided ones; the
# most experts, pairs and segments that a call may have.
NARROW = [(40, 130, 72, 64, 1), (40, 260, 1600, 64, 4), (64, 130, 72, 300, 4), (24, 264, 500, 64, 6), (100, 200, 100, 128, 1),
          (100, 260, 1600, 128, 3), (65, 128, 900, 256, 8), (128, 40, 24, 1024, 8), (128, 40, 24, 1024, 24), (128, 40, 24, 1024, 32),
          (20, 136, 64, 256, 12)]


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("T,d,f,E,k", NARROW)
def test_narrow_passes_of_many_tokens(T, d, f, E, k, skew):
    """skew: one expert takes every token, in as many passes as they need."""
    gated, renorm = T % 8 != 0, E % 3 != 0
    router = (np.random.default_rng(T + k).standard_normal((E, d)) * 2 / np.sqrt(d)).astype(np.float32)
    x = _tokens(T, d, BF16, 100)
    if skew:
        router[:, 0], x[:, 0] = 0, 1
        router[E // 2, 0] = 30
    layer, r, mats = _layer(d, f, E, k, gated, renorm, BF16, 101, router=router)
    Y, v = _check(x, BF16, layer, r, mats, F32)
    assert not skew or (v["ids"][:, 0] == E // 2).all()
    X, ws, again = torch.from_numpy(x).to(BF16).cuda(), B.alloc_workspace_moe(T, layer), torch.empty_like(Y)
    for _ in range(3):
        again.fill_(float("nan"))
        B.w4a4_moe_forward(X, layer, again, ws)
        assert torch.equal(again, Y)
    x[T // 3, 2] = np.nan
    Y, v = _check(x, BF16, layer, r, mats, BF16)
    assert v["ids"][T // 3].tolist() == list(range(k)) and bool(torch.isnan(Y[T // 3]).all()) and not bool(torch.isnan(Y[T // 3 + 1]).any())


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,E,k", [(2, 12, 3), (30, 12, 3), (40, 64, 1)])
def test_infinite_tokens(T, E, k, gated):
    """Infinities of both signs go through the formula (infinite and NaN h, a NaN row) and touch no
    other token; logits that are all -Inf tie."""
    router = (np.random.default_rng(110).standard_normal((E, 192)) / 7).astype(np.float32)
    router[:, 20] = np.abs(router[:, 20]) + np.float32(0.01)
    layer, r, mats = _layer(192, 64, E, k, gated, True, BF16, 111, router=router)
    x = _tokens(T, 192, BF16, 112)
    x[0, 17], x[1, 20] = np.inf, -np.inf
    Y, v = _check(x, BF16, layer, r, mats, F32)
    assert v["ids"][1].tolist() == list(range(k)) and bool(torch.isnan(Y[:2]).all()) and not bool(torch.isnan(Y[2:]).any())


@pytest.mark.parametrize("xt,rt", [(F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("T,d", [(1, 256), (1, 131), (6, 131)])
def test_tokens_and_router_of_different_types(T, d, xt, rt):
    layer, r, mats = _layer(d, 48, 20, 4, True, False, rt, 120)
    _check(_tokens(T, d, xt, 121), xt, layer, r, mats, BF16)
