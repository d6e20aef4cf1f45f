"""MXFP4 quantisation, dispatch and expert products on the GPU against 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

import sparse_mixture_experts_49_amd as moe
from tests import _mx_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32, U16 = 2.0 ** -24, 2.0 ** -8      # half a step, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _hard_rows(rows, cols, dtype, seed):
    """Values over many magnitudes, with ties, zeros, subnormals and non-finite blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, cols // 32, generator=g)).repeat_interleave(32, 1)
    flat = x.view(-1, 32)
    flat[0] = 0.0
    if len(flat) > 8:
        flat[1] = torch.tensor([0.25, -0.25, 0.75, -0.75, 1.25, 1.75, 2.5, -2.5, 3.5, 5.0, -5.0, 6.0, 7.0, 4.0] + [0.0] * 17 + [-0.0])
        flat[2] = 2.0 ** -127 * torch.arange(32)                  # subnormals
        flat[3] = 2.0 ** -133 * torch.arange(32)
        flat[4] = 3.0e38
        flat[5, 7] = float("nan")
        flat[6, 31] = -float("inf")
        flat[7] = 2.0 ** -126
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,stride", [(1, 32, 32), (1, 4096, 4096), (3, 96, 104), (37, 160, 160), (129, 1408, 2048)])
def test_quantize_and_dequantize_exactly(rows, cols, stride, dtype):
    x = _hard_rows(rows, cols, dtype, rows + cols)
    big = torch.full((rows + 1, stride), float("nan"), dtype=dtype, device=DEV)
    big[:rows, :cols] = x.to(DEV)
    view = big[:rows, :cols]
    codes, scales = moe.alloc_mx(rows + 1, cols, DEV)
    codes.fill_(0xA5), scales.fill_(0xA5)
    moe.moe_mx_quantize(view, codes[:rows], scales[:rows])
    rc, rs = R.quantize(x)
    assert torch.equal(scales[:rows].cpu(), rs)
    assert torch.equal(codes[:rows].cpu(), rc)
    assert torch.all(codes[rows] == 0xA5) and torch.all(scales[rows] == 0xA5)
    for out_dtype in (torch.bfloat16, torch.float32):
        out = torch.full((rows + 1, stride), 7.0, dtype=out_dtype, device=DEV)
        moe.moe_mx_dequantize(codes[:rows], scales[:rows], out[:rows, :cols])
        want = R.values(rc, rs).to(out_dtype)
        assert torch.equal(out[:rows, :cols].cpu().isnan(), want.isnan())
        assert torch.equal(out[:rows, :cols].cpu().nan_to_num(0.0), want.nan_to_num(0.0))
        assert torch.all(out[rows] == 7.0) and torch.all(out[:rows, cols:] == 7.0)


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :16 * 16].contiguous()
    scales = torch.arange(256, dtype=torch.uint8).view(-1, 1).repeat(1, 16).contiguous()
    out = torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_dequantize(codes.to(DEV), scales.to(DEV), out)
    want = R.values(codes, scales).to(torch.bfloat16)
    got = out.cpu()
    assert torch.equal(got[255].isnan(), torch.ones(512, dtype=torch.bool))
    assert torch.equal(got[:255], want[:255])


def test_quantize_no_rows_and_refusals():
    codes, scales = moe.alloc_mx(0, 64, DEV)
    moe.moe_mx_quantize(torch.empty(0, 64, device=DEV), codes, scales)
    with pytest.raises(moe.MoeError, match="needs"):
        moe.moe_mx_quantize(torch.zeros(2, 64, device=DEV), *moe.alloc_mx(1, 64, DEV))
    with pytest.raises(moe.MoeError, match="contiguous rows"):
        moe.moe_mx_quantize(torch.zeros(64, 64, device=DEV).t()[:, ::2], *moe.alloc_mx(64, 64, DEV))
    with pytest.raises(moe.MoeError, match="bf16 or fp32"):
        moe.moe_mx_quantize(torch.zeros(2, 64, device=DEV).half(), *moe.alloc_mx(2, 64, DEV))


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (32, 2, 8), (128, 8, 255), (129, 8, 256), (700, 6, 64), (3000, 8, 160)])
def test_dispatch(T, k, E):
    g = torch.Generator().manual_seed(T + E)
    idx = (torch.rand(T, E, generator=g) + torch.rand(E, generator=g)).topk(k, 1).indices.to(torch.int32)
    if T > 20:
        idx[3, 0], idx[5, :], idx[9, -1] = -1, -1, E
    desc = moe.MxDesc(T, 128, 128, E, k)
    r = moe.Routing(topk_idx=idx.to(DEV), counts=torch.empty(E, dtype=torch.int32, device=DEV),
                    offsets=torch.empty(E + 1, dtype=torch.int32, device=DEV),
                    dest=torch.empty(T, k, dtype=torch.int32, device=DEV),
                    src=torch.full((T * k,), -9, dtype=torch.int32, device=DEV))
    ws = moe.alloc_mx_workspace(desc, DEV)
    ws.fill_(0xFF)
    moe.moe_mx_dispatch(desc, r, workspace=ws)
    counts, offsets, dest, src = R.dispatch(idx, E)
    assert r.counts.tolist() == counts and r.offsets.tolist() == offsets.tolist()
    assert torch.equal(r.dest.cpu().long(), torch.from_numpy(dest))
    assert r.src.tolist() == src + [-9] * (T * k - len(src))


def _layer(T, k, E, d, F, bias, seed, idx=None):
    """Random MXFP4 experts and a dispatch of T tokens (some slots dropped)."""
    g = torch.Generator().manual_seed(seed)

    def mx(n, kk):
        return R.quantize((torch.randn(E * n, kk, generator=g) * kk ** -0.5).bfloat16())

    w1, w2 = mx(F, d), mx(d, F)
    b = [(0.1 * torch.randn(E, n, generator=g)).bfloat16() for n in (F, d)] if bias else [None, None]
    if idx is None:
        idx = (torch.rand(T, E, generator=g) + 0.5 * torch.rand(E, generator=g)).topk(k, 1).indices
        if T > 2:
            idx[T // 2, 0] = -1
    counts, offsets, dest, src = R.dispatch(idx, E)
    return dict(w1=w1, w2=w2, b1=b[0], b2=b[1], idx=idx, offsets=torch.tensor(offsets, dtype=torch.int32),
                src=torch.tensor(src + [0] * (T * k - len(src)), dtype=torch.int32), rows=len(src),
                x=torch.randn(T, d, generator=g).bfloat16(), gen=g)


def _weights(L):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return moe.MxWeights(to(L["w1"][0]), to(L["w1"][1]), to(L["b1"]), to(L["w2"][0]), to(L["w2"][1]), to(L["b2"]))


def _poisoned(desc, route=None):
    ws = moe.alloc_mx_workspace(desc, DEV, route)
    ws.fill_(0xFF)
    return ws


# T, k, E, d, F, expert bias
SHAPES = [
    (1, 1, 1, 128, 128, True), (1, 2, 8, 4096, 1024, True), (3, 3, 4, 256, 384, False),
    (16, 2, 8, 640, 1152, True), (17, 2, 3, 1024, 256, False), (32, 2, 8, 2176, 640, True),
    (40, 6, 64, 512, 1408, True), (70, 1, 2, 384, 512, True), (130, 2, 4, 512, 640, False),
    (257, 8, 160, 256, 256, True), (300, 1, 1, 1280, 384, True), (700, 4, 8, 896, 640, True),
    (1100, 2, 4, 384, 1408, False), (520, 2, 2, 128, 2304, True),
]


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d_k%d_E%d_d%d_F%d_b%d" % s)
def test_products(shape, act):
    T, k, E, d, F, bias = shape
    L = _layer(T, k, E, d, F, bias, T + E + d)
    desc = moe.MxDesc(T, d, F, E, k, act=act, has_expert_bias=bias)
    w, rows, off = _weights(L), L["rows"], L["offsets"]
    h_in = torch.nn.functional.gelu(torch.randn(T * k, F, generator=L["gen"])).bfloat16()

    def seen(a):                       # the values the product multiplies
        return R.values(*R.quantize(a)) if act == "mxfp4" else a.double()

    # Any order of K fp32 additions of exact products: K roundings of partial sums, each at
    # most the sum of |terms|; GELU has slope under 1.13 and its own error of 1.3e-5 |z|
    # Phi(-|z|) (its polynomial's), at least in part under 2e-7 |z|, the rest, under 6.3e-6 |z|,
    # within the room of the additions (128 * 1.13 U32 size > 8.6e-6 |z|, which a sum of exact
    # 8-bit products uses no quarter of); then bf16 or fp32 rounding.
    W1, W2 = R.values(*L["w1"]).view(E, F, d), R.values(*L["w2"]).view(E, d, F)
    perm = L["x"][L["src"][:rows].long() // k]
    z, size = R.product(seen(perm), off, W1, L["b1"])
    want = R.gelu(z)
    room = 1.13 * (d + 1) * U32 * size + 2e-7 * z.abs()
    room = room + U16 * (want.abs() + room)
    for src in (L["src"], None):
        x = L["x"] if src is not None else torch.cat([perm, perm.new_zeros(T * k - rows, d)])
        h = torch.full((T * k + 3, F), -77.0, device=DEV).bfloat16()
        moe.moe_mx_ffn_up(desc, x.to(DEV), off.to(DEV), w, h, src=None if src is None else src.to(DEV),
                          workspace=_poisoned(desc))
        got = h[:rows].cpu().double()
        assert torch.all((got - want).abs() <= room), float(((got - want).abs() / room).max())
        assert torch.all(h[rows:] == -77.0)           # rows behind the last segment
    z, size = R.product(seen(h_in[:rows]), off, W2, L["b2"])
    o = torch.full((T * k + 3, d), -77.0, device=DEV)
    moe.moe_mx_ffn_down(desc, h_in.to(DEV), off.to(DEV), w, o, workspace=_poisoned(desc))
    room = (F + 2) * U32 * size
    got = o[:rows].cpu().double()
    assert torch.all((got - z).abs() <= room), float(((got - z).abs() / room).max())
    assert torch.all(o[rows:] == -77.0)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,k,E", [(20, 2, 8), (300, 2, 4)])
def test_nan_scales_stay_in_their_column(T, k, E, act):
    d, F = 256, 256
    L = _layer(T, k, E, d, F, False, 9)
    e, n = 1, 37
    s1 = L["w1"][1].view(E, F, d // 32)
    s1[e, n, 3] = 255
    desc = moe.MxDesc(T, d, F, E, k, act=act, has_expert_bias=False)
    h = torch.zeros(T * k, F, dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_ffn_up(desc, L["x"].to(DEV), L["offsets"].to(DEV), _weights(L), h, src=L["src"].to(DEV))
    want = torch.zeros(T * k, F, dtype=torch.bool)
    want[int(L["offsets"][e]):int(L["offsets"][e + 1]), n] = True
    assert torch.equal(h.cpu().isnan(), want)
    # A NaN token poisons its own rows only.
    s1[e, n, 3] = 100
    x = L["x"].clone()
    x[2, 5] = float("nan")
    moe.moe_mx_ffn_up(desc, x.to(DEV), L["offsets"].to(DEV), _weights(L), h, src=L["src"].to(DEV))
    rows = torch.zeros(T * k, dtype=torch.bool)
    rows[:L["rows"]] = (L["src"][:L["rows"]] // k) == 2
    assert torch.equal(h.cpu().isnan().all(1), rows) and torch.equal(h.cpu().isnan().any(1), rows)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [40, 600])
def test_everything_on_one_expert_and_nothing(T, act):
    E, k, d, F = 8, 1, 256, 384
    desc = moe.MxDesc(T, d, F, E, k, act=act)
    for idx in (torch.full((T, 1), 5), torch.full((T, 1), -1)):
        L = _layer(T, k, E, d, F, True, 4, idx)
        h = torch.full((T, F), -77.0, device=DEV).bfloat16()
        moe.moe_mx_ffn_up(desc, L["x"].to(DEV), L["offsets"].to(DEV), _weights(L), h, src=L["src"].to(DEV))
        if L["rows"] == 0:
            assert torch.all(h == -77.0)
            continue
        a = R.values(*R.quantize(L["x"])) if act == "mxfp4" else L["x"].double()
        z, size = R.product(a, L["offsets"], R.values(*L["w1"]).view(E, F, d), L["b1"])
        room = 1.13 * (d + 1) * U32 * size + 2e-7 * z.abs()
        assert torch.all((h.cpu().double() - R.gelu(z)).abs() <= room + U16 * (R.gelu(z).abs() + room))


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,k,E,G", [(1, 2, 8, 1), (33, 6, 64, 8), (900, 4, 16, 4), (200, 8, 256, 8)])
def test_forward_is_the_chain_of_calls(T, k, E, G, act):
    """moe_mx_forward bit for bit as its parts, with moe_permute and moe_combine of the
    existing layer where they reach (64 experts); captured, replayed, on another stream."""
    d, F = 384, 256
    L = _layer(T, k, E, d, F, True, T)
    g = torch.Generator().manual_seed(T)
    wr = (torch.randn(E, d, generator=g) * d ** -0.5).bfloat16().to(DEV)
    route = moe.ScoreDesc(T, d, E, k, score="sigmoid", n_groups=G, top_groups=max(1, G // 2), scale=2.5)
    desc = moe.MxDesc(T, d, F, E, k, act=act)
    w, x = _weights(L), L["x"].to(DEV)
    y = torch.empty(T, d, device=DEV)
    r = moe.ScoreRouting.allocate(route, DEV, train=True)
    ws = _poisoned(desc, route)
    moe.moe_mx_forward(route, desc, x, wr, w, y, routing=r, workspace=ws)

    r2 = moe.ScoreRouting.allocate(route, DEV)
    moe.moe_score_route(route, x, wr, r2)
    lay = moe.Routing(topk_idx=r2.topk_idx, counts=torch.empty(E, dtype=torch.int32, device=DEV),
                      offsets=torch.empty(E + 1, dtype=torch.int32, device=DEV), dest=torch.empty(T, k, dtype=torch.int32, device=DEV),
                      src=torch.empty(T * k, dtype=torch.int32, device=DEV))
    old = moe.Desc(T, d, F, min(E, 64), k)
    if E <= 64:
        x_perm = torch.empty(T * k, d, dtype=torch.bfloat16, device=DEV)
        moe.moe_permute(old, x, lay, x_perm)
    else:
        moe.moe_mx_dispatch(desc, lay)
    h = torch.empty(T * k, F, dtype=torch.bfloat16, device=DEV)
    o = torch.empty(T * k, d, device=DEV)
    moe.moe_mx_ffn_up(desc, x, lay.offsets, w, h, src=lay.src)
    if E <= 64:
        h2 = torch.empty_like(h)
        moe.moe_mx_ffn_up(desc, x_perm, lay.offsets, w, h2)
        assert torch.equal(h, h2)
    moe.moe_mx_ffn_down(desc, h, lay.offsets, w, o)
    y2 = torch.empty_like(y)
    moe.moe_combine(old, o, lay.dest, r2.topk_w, y2)
    assert torch.equal(r.topk_idx, r2.topk_idx) and torch.equal(r.topk_w, r2.topk_w)
    assert torch.equal(y, y2)
    assert torch.equal(r.load, lay.counts)

    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_mx_forward(route, desc, x, wr, w, y, routing=r, workspace=ws)
    for _ in range(3):
        y.zero_()
        r.topk_idx.fill_(-3)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(r.topk_idx, r2.topk_idx)
    y.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_mx_forward(route, desc, x, wr, w, y, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


def test_quantized_layer_is_near_the_layer_it_was_made_from():
    """MxWeights.quantize of a bf16 layer: each weight is off by at most half a step of its
    block (a quarter of the block's largest value at most), so against the same layer in
    MXFP4 values the product is exact, and against bf16 it is a bounded step away."""
    T, E, d, F = 24, 4, 256, 384
    g = torch.Generator().manual_seed(1)
    w1 = (torch.randn(E, F, d, generator=g) * d ** -0.5).bfloat16()
    w2 = (torch.randn(E, d, F, generator=g) * F ** -0.5).bfloat16()
    mx = moe.MxWeights.quantize(w1.to(DEV), w2.to(DEV))
    for w, c, s in ((w1, mx.w1, mx.s1), (w2, mx.w2, mx.s2)):
        assert c.shape == (*w.shape[:2], w.shape[2] // 2) and s.shape == (*w.shape[:2], w.shape[2] // 32)
        v = R.values(c.cpu(), s.cpu())
        top = w.double().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True)
        step = torch.exp2(torch.floor(torch.log2(top)))          # the block's largest grid step is half of this
        assert torch.all((v - w.double()).unflatten(-1, (-1, 32)).abs() <= step / 2)


def test_two_streams_with_their_own_workspaces():
    T, k, E, d, F = 64, 2, 8, 512, 512
    desc = moe.MxDesc(T, d, F, E, k)
    L = _layer(T, k, E, d, F, True, 6)
    w, x, off, src = _weights(L), L["x"].to(DEV), L["offsets"].to(DEV), L["src"].to(DEV)
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            ws = _poisoned(desc)
            h = torch.zeros(T * k, F, dtype=torch.bfloat16, device=DEV)
            for _ in range(5):
                moe.moe_mx_ffn_up(desc, x, off, w, h, src=src, workspace=ws)
            outs.append((h, ws))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0])
    assert not math.isnan(float(outs[0][0][:L["rows"]].float().sum()))


# More tiles than CUs, so that blocks go on to further tiles: 128 and 256 rows high, k an odd
# multiple of 128; 15 rows per expert, streamed 32 rows at a time over a long k.
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("shape", [(640, 6, 64, 640, 1408, True), (600, 8, 8, 512, 2816, False),
                                   (60, 2, 8, 4096, 256, True), (150, 2, 8, 512, 640, True)],
                         ids=lambda s: "T%d_k%d_E%d_d%d_F%d_b%d" % s)
def test_products_over_many_tiles(shape, act):
    test_products(shape, act)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_tiled_products_of_uneven_experts(act):
    """K = 512 and 75 rows per expert on average: one expert has them all, or none has any, or
    all but two slots go to one expert."""
    T, E, k, d, F = 600, 8, 1, 512, 384
    desc = moe.MxDesc(T, d, F, E, k, act=act)
    mostly = torch.full((T, 1), 6)
    mostly[0], mostly[599] = 0, 7
    for idx in (torch.full((T, 1), 5), mostly, torch.full((T, 1), -1)):
        L = _layer(T, k, E, d, F, True, 4, idx)
        n = L["rows"]
        h = torch.full((T, F), -77.0, device=DEV).bfloat16()
        moe.moe_mx_ffn_up(desc, L["x"].to(DEV), L["offsets"].to(DEV), _weights(L), h, src=L["src"].to(DEV),
                          workspace=_poisoned(desc))
        assert torch.all(h[n:] == -77.0)
        if n == 0:
            continue
        x = L["x"][L["src"][:n].long() // k]
        a = R.values(*R.quantize(x)) if act == "mxfp4" else x.double()
        z, size = R.product(a, L["offsets"], R.values(*L["w1"]).view(E, F, d), L["b1"])
        room = 1.13 * (d + 1) * U32 * size + 1.3e-5 * R.gelu(-z.abs()).abs()
        assert torch.all((h[:n].cpu().double() - R.gelu(z)).abs() <= room + U16 * (R.gelu(z).abs() + room))


@pytest.mark.parametrize("d", [128, 512], ids=["streamed", "tiled"])
def test_gelu_of_every_bf16_value(d):
    """One weight of 1 per column, so that z is x itself: every finite value, against 64 bits.
    z is exact, so the error is the polynomial's (1.3e-5 of |z| Phi(-|z|) up to |z| = 7, that
    whole term, under 1e-11, beyond) and two fp32 roundings, then the rounding to bf16."""
    F, T = d, 65536 // d
    codes = torch.zeros(1, F, d // 2, dtype=torch.uint8)
    n = torch.arange(F)
    codes[0, n, n // 2] = torch.where(n % 2 == 0, 0x02, 0x20).to(torch.uint8)      # e2m1 1.0
    scales = torch.full((1, F, d // 32), 127, dtype=torch.uint8)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(T, d).clone()
    x[~x.isfinite()] = 0.0
    desc = moe.MxDesc(T, d, F, 1, 1, has_expert_bias=False)
    h = torch.empty(T, F, dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_ffn_up(desc, x.to(DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV),
                      moe.MxWeights(w1=codes.to(DEV), s1=scales.to(DEV)), h)
    z = x.double()
    tail = z.abs() * 0.5 * torch.special.erfc(z.abs() * 0.5 ** 0.5)      # Phi by 1 + erf ends at -8.3
    want = torch.where(z > 0, z - tail, -tail)
    room = torch.where(z.abs() <= 7, 1.3e-5 * tail, tail.clamp(min=1e-30)) + 2 * U32 * want.abs()
    got = h.cpu().double()
    assert torch.all((got - want).abs() <= room + U16 * (want.abs() + room) + 2.0 ** -133)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_forward_on_the_tiled_path(act):
    """A layer whose products are tiled, bit for bit as its parts; captured, and replayed with
    eager calls of the same layer between."""
    T, k, E, d, F = 450, 4, 16, 512, 640
    L = _layer(T, k, E, d, F, True, 12)
    g = torch.Generator().manual_seed(3)
    wr = (torch.randn(E, d, generator=g) * d ** -0.5).bfloat16().to(DEV)
    route, desc = moe.ScoreDesc(T, d, E, k), moe.MxDesc(T, d, F, E, k, act=act)
    w, x = _weights(L), L["x"].to(DEV)
    y, ws, eager_ws = torch.empty(T, d, device=DEV), _poisoned(desc, route), _poisoned(desc, route)
    r = moe.ScoreRouting.allocate(route, DEV)
    moe.moe_score_route(route, x, wr, r)
    lay = moe.Routing(topk_idx=r.topk_idx, counts=torch.empty(E, dtype=torch.int32, device=DEV),
                      offsets=torch.empty(E + 1, dtype=torch.int32, device=DEV), dest=torch.empty(T, k, dtype=torch.int32, device=DEV),
                      src=torch.empty(T * k, dtype=torch.int32, device=DEV))
    moe.moe_mx_dispatch(desc, lay)
    h, o = torch.empty(T * k, F, dtype=torch.bfloat16, device=DEV), torch.empty(T * k, d, device=DEV)
    moe.moe_mx_ffn_up(desc, x, lay.offsets, w, h, src=lay.src)
    moe.moe_mx_ffn_down(desc, h, lay.offsets, w, o)
    want = torch.empty_like(y)
    moe.moe_combine(moe.Desc(T, d, F, E, k), o, lay.dest, r.topk_w, want)
    moe.moe_mx_forward(route, desc, x, wr, w, y, workspace=ws)
    assert torch.equal(y, want)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_mx_forward(route, desc, x, wr, w, y, workspace=ws)
    for _ in range(3):
        y.zero_()
        ws.fill_(0xFF)
        eager = torch.empty_like(y)
        moe.moe_mx_forward(route, desc, x, wr, w, eager, workspace=eager_ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(eager, want)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,d,F", [(3, 4096, 256), (40, 128, 256), (300, 512, 256)], ids=["split", "streamed", "tiled"])
def test_gelu_of_overflow_and_infinite_bias(T, d, F, act):
    """z = +inf is +inf, z = -inf and z = NaN are NaN (-inf * 0 in z Phi(z)): from a bias, and
    from a product past fp32's range; the largest finite z stays itself."""
    desc = moe.MxDesc(T, d, F, 1, 1, act=act)
    codes = torch.zeros(1, F, d // 2, dtype=torch.uint8)
    scales = torch.full((1, F, d // 32), 127, dtype=torch.uint8)
    codes[0, :, 0], scales[0, :, 0] = 0x02, 127 + 100        # column n: 2^100 times the token's first value
    x = torch.zeros(T, d).bfloat16()
    x[:, 0] = 2.0 ** -100
    x[T // 2:, 0] = 2.0 ** 100                               # 2^200 in all columns
    x[T // 2::2, 0] = -2.0 ** 100
    bias = torch.zeros(1, F).bfloat16()
    inf = float("inf")
    bias[0, :5] = torch.tensor([inf, -inf, float("nan"), 3e38, -3e38]).bfloat16()
    h = torch.full((T, F), -77.0, device=DEV).bfloat16()
    moe.moe_mx_ffn_up(desc, x.to(DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV),
                      moe.MxWeights(w1=codes.to(DEV), s1=scales.to(DEV), b1=bias.to(DEV)), h, workspace=_poisoned(desc))
    z = x[:, :1].double() * 2.0 ** 100
    z = torch.where(z.abs() > 3.4e38, z * inf, z) + bias.double()
    want = torch.where(z == inf, inf, torch.where((z == -inf) | z.isnan(), float("nan"), R.gelu(z)))
    want = torch.where(z == bias[0, 3].double(), z, torch.where(z == bias[0, 4].double(), 0.0, want))
    got = h.cpu().double()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got == inf, want == inf)
    fine = want.isfinite()
    assert torch.all((got - want)[fine].abs() <= 2 * U16 * want[fine].abs())


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,k,E,d,F", [(300, 2, 4, 512, 512), (450, 4, 16, 640, 384), (600, 8, 8, 1024, 1408)])
def test_nan_scales_and_tokens_in_tiled_products(T, k, E, d, F, act):
    """Experts that average 56 rows or more over k >= 512: a block of weights whose scale is NaN
    makes its column of its expert NaN and nothing else, a NaN token its own rows, an infinite
    activation no row but its own."""
    L = _layer(T, k, E, d, F, False, 9)
    e, n = 1, F - 100
    s1 = L["w1"][1].view(E, F, d // 32)
    old = int(s1[e, n, d // 32 - 1])
    s1[e, n, d // 32 - 1] = 255
    desc = moe.MxDesc(T, d, F, E, k, act=act, has_expert_bias=False)
    off, src, rows = L["offsets"].to(DEV), L["src"].to(DEV), L["rows"]
    h = torch.zeros(T * k, F, dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_ffn_up(desc, L["x"].to(DEV), off, _weights(L), h, src=src, workspace=_poisoned(desc))
    want = torch.zeros(T * k, F, dtype=torch.bool)
    want[int(L["offsets"][e]):int(L["offsets"][e + 1]), n] = True
    assert torch.equal(h.cpu().isnan(), want) and not h.isinf().any()
    s1[e, n, d // 32 - 1] = old
    for bad in (float("nan"), float("inf")):
        x = L["x"].clone()
        x[2, d - 3], x[T - 1, 0] = bad, bad
        moe.moe_mx_ffn_up(desc, x.to(DEV), off, _weights(L), h, src=src, workspace=_poisoned(desc))
        mine = torch.zeros(T * k, dtype=torch.bool)
        token = L["src"][:rows] // k
        mine[:rows] = (token == 2) | (token == T - 1)
        got = h.cpu()
        assert got[~mine].isfinite().all()
        if act == "mxfp4" or bad != bad:                       # the block's scale is NaN
            assert got[mine].isnan().all()
        else:
            assert not got[mine].isfinite().any()
    # The second product, h with a NaN and its weights with a NaN scale.
    s2 = L["w2"][1].view(E, d, F // 32)
    s2[E - 1, 5, 0] = 255
    a = torch.nn.functional.gelu(torch.randn(T * k, F, generator=L["gen"])).bfloat16()
    a[7, F - 1] = float("nan")
    o = torch.zeros(T * k, d, device=DEV)
    moe.moe_mx_ffn_down(desc, a.to(DEV), off, _weights(L), o, workspace=_poisoned(desc))
    want = torch.zeros(T * k, d, dtype=torch.bool)
    want[int(L["offsets"][E - 1]):int(L["offsets"][E]), 5] = True
    want[7] = True
    assert torch.equal(o.cpu().isnan(), want)


@pytest.mark.parametrize("T,k,E", [(1, 8, 256), (200, 8, 256), (33, 3, 65), (70, 2, 160)])
def test_combine_of_up_to_256_experts(T, k, E):
    """The layer step by step with public calls only: moe_combine takes the layer's own number
    of experts, bit for bit what moe_mx_forward gives."""
    d, F = 384, 256
    L = _layer(T, k, E, d, F, True, T + 1)
    g = torch.Generator().manual_seed(T)
    wr = (torch.randn(E, d, generator=g) * d ** -0.5).bfloat16().to(DEV)
    route, desc = moe.ScoreDesc(T, d, E, k, score="sigmoid", scale=2.5), moe.MxDesc(T, d, F, E, k)
    w, x, y = _weights(L), L["x"].to(DEV), torch.empty(T, d, device=DEV)
    moe.moe_mx_forward(route, desc, x, wr, w, y)
    r = moe.ScoreRouting.allocate(route, DEV)
    moe.moe_score_route(route, x, wr, r)
    i32 = dict(dtype=torch.int32, device=DEV)
    lay = moe.Routing(topk_idx=r.topk_idx, counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                      dest=torch.empty(T, k, **i32), src=torch.empty(T * k, **i32))
    moe.moe_mx_dispatch(desc, lay)
    h, o = torch.empty(T * k, F, dtype=torch.bfloat16, device=DEV), torch.empty(T * k, d, device=DEV)
    moe.moe_mx_ffn_up(desc, x, lay.offsets, w, h, src=lay.src)
    moe.moe_mx_ffn_down(desc, h, lay.offsets, w, o)
    y2 = torch.empty_like(y)
    moe.moe_combine(moe.Desc(T, d, F, E, k), o, lay.dest, r.topk_w, y2)
    assert torch.equal(y, y2)
    want = torch.zeros(T, d, dtype=torch.float64)
    for s in range(k):
        want += r.topk_w[:, s, None].double().cpu() * o.cpu().double()[lay.dest[:, s].long().cpu()]
    size = sum(r.topk_w[:, s, None].abs().double().cpu() * o.cpu().double()[lay.dest[:, s].long().cpu()].abs() for s in range(k))
    assert torch.all((y2.cpu().double() - want).abs() <= k * U32 * size)
