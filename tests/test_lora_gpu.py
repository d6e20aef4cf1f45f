"""The projection with low-rank adapters on the GPU against 64 bits."""
from __future__ import annotations

import pytest
import torch

import sparse_mixture_experts_49_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24            # half a step of fp32, relative
U16 = 2.0 ** -8             # of bf16


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def _ids(T, N, kind, g):
    if kind == "one":
        return torch.full((T,), N - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "random":                             # ids past both ends among them
        ids = torch.randint(-1, N + 1, (T,), generator=g).to(torch.int32)
        ids[::7] = -(1 << 31)
        ids[3::11] = (1 << 31) - 1
        return ids
    cuts = torch.rand(T, generator=g) < 1 / 40       # runs of about 40
    return (torch.randint(0, N + 1, (T,), generator=g)[cuts.cumsum(0)] - 1).to(torch.int32)


def _small_integers(T, d, n, r, N, bias, g):
    """Values whose every product and sum is exact in fp32, whatever the order."""
    x = torch.randint(-2, 3, (T, d), generator=g).bfloat16()
    w = (torch.randint(-2, 3, (n, d), generator=g) / 4).bfloat16()
    a = (torch.randint(0, 8, (N, r, d), generator=g) < 1).bfloat16()
    b = (torch.randint(-2, 3, (N, n, r), generator=g) / 8).bfloat16()
    scale = 2.0 ** torch.randint(-1, 2, (N,), generator=g)
    return x, w, a, b, scale, (torch.randint(-9, 10, (n,), generator=g) / 4).bfloat16() if bias else None


def _reference(x, w, a, b, scale, bias, ids):
    """(y, sum of the absolute products) in 64 bits."""
    x, w = x.double(), w.double()
    y, size = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        y, size = y + bias.double(), size + bias.double().abs()
    for i in range(a.shape[0]):
        rows = (ids == i).nonzero()[:, 0]
        if len(rows):
            s = float(scale[i]) if scale is not None else 1.0
            y[rows] += s * (x[rows] @ a[i].double().T @ b[i].double().T)
            size[rows] += abs(s) * (x[rows].abs() @ a[i].double().abs().T @ b[i].double().abs().T)
    return y, size


def _run(desc, x, ids, w, a, b, scale, bias, guard=64):
    T, n = desc.tokens, desc.d_out
    dt = torch.bfloat16 if desc.out_dtype == "bf16" else torch.float32
    y = torch.full((T * n + guard,), 7.0, dtype=dt, device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    ws = moe.alloc_lora_workspace(desc, DEV).fill_(0xFF)          # NaN in every type
    moe.moe_lora_linear(desc, x.to(DEV), ids.to(DEV), moe.LoraWeights(dev(w), dev(a), dev(b), dev(scale), dev(bias)), y,
                        workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(y[T * n:] == 7)
    return y[:T * n].view(T, n).cpu()


# T, d, n, rank, N, ids, bias, scale
SHAPES = [
    (1, 128, 128, 8, 1, "one", False, True), (1, 4096, 4096, 16, 8, "one", False, True),
    (1, 640, 256, 24, 3, "one", True, True), (1, 1152, 384, 32, 2, "one", True, False),
    (1, 8192, 2176, 16, 2, "one", False, True), (1, 5120, 384, 8, 2, "none", True, True),
    (1, 1024, 128, 128, 2, "one", False, True), (1, 2048, 256, 128, 2, "one", True, True),
    (2, 256, 384, 16, 3, "random", True, False), (16, 640, 128, 24, 40, "random", False, True),
    (17, 128, 256, 128, 5, "random", True, True), (32, 384, 8192, 16, 32, "random", True, True),
    (33, 512, 512, 40, 2, "runs", False, False), (64, 2048, 256, 72, 70, "random", True, True),
    (65, 256, 1024, 16, 300, "random", False, True), (200, 384, 384, 64, 4, "runs", True, True),
    (512, 128, 640, 8, 9, "random", False, True), (513, 128, 256, 16, 3, "runs", True, True),
    (513, 256, 256, 16, 3, "runs", True, True), (600, 320 * 2, 384, 8, 40, "random", False, True),
    (777, 384, 128, 48, 2, "one", True, False), (1100, 512, 1152, 128, 6, "runs", False, True),
    (1024, 256, 256, 16, 5, "none", True, True), (8200, 256, 2176, 24, 30, "runs", True, True),
    (12300, 384, 1280, 16, 200, "random", False, True), (16400, 256, 1024, 72, 3, "runs", True, True),
    (2000, 256, 1536, 40, 60, "random", True, True), (1500, 384, 2176, 128, 5, "random", False, True),
    (1400, 256, 2176, 16, 300, "random", True, False),
]
IDS = ["T%d_%dx%d_r%d_N%d_%s" % s[:6] for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_exact_values(shape):
    """Integers: the fp32 result is exact, the bf16 one rounded once."""
    T, d, n, r, N, kind, bias, scaled = shape
    g = torch.Generator().manual_seed(T + d + r)
    x, w, a, b, scale, bi = _small_integers(T, d, n, r, N, bias, g)
    scale = scale if scaled else None
    ids = _ids(T, N, kind, g)
    ref, size = _reference(x, w, a, b, scale, bi, ids)
    # multiples of 1/32 under 2^19 in absolute sum are exact; A x is an integer under 2^16, times
    # a power of two, so two bf16 terms hold it
    assert float(size.max()) < 2 ** 19 and d * 2 < 2 ** 16
    for out in ("f32", "bf16"):
        desc = moe.LoraDesc(T, d, n, r, N, out_dtype=out, has_bias=bias)
        got = _run(desc, x, ids, w, a, b, scale, bi)
        assert torch.equal(got, ref.float() if out == "f32" else ref.float().bfloat16()), out


def _gaussians(T, d, n, r, N, bias, g):
    x, w = torch.randn(T, d, generator=g).bfloat16(), (torch.randn(n, d, generator=g) * d ** -0.5).bfloat16()
    a = (torch.randn(N, r, d, generator=g) * d ** -0.5).bfloat16()
    b = (torch.randn(N, n, r, generator=g) * r ** -0.5).bfloat16()
    return x, w, a, b, 0.5 + torch.rand(N, generator=g), torch.randn(n, generator=g).bfloat16() if bias else None


@pytest.mark.parametrize("shape", [SHAPES[i] for i in (1, 3, 10, 13, 14, 18, 21, 23, 27)],
                         ids=[IDS[i] for i in (1, 3, 10, 13, 14, 18, 21, 23, 27)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_gaussian_values(shape, out, act):
    T, d, n, r, N, kind, bias, _ = shape
    g = torch.Generator().manual_seed(T + d)
    x, w, a, b, scale, bi = _gaussians(T, d, n, r, N, bias, g)
    ids = _ids(T, N, kind, g)
    ref, size = _reference(x, w, a, b, scale, bi, ids)
    got = _run(moe.LoraDesc(T, d, n, r, N, act=act, out_dtype=out, has_bias=bias), x, ids, w, a, b, scale, bi).double()
    # d products in one sum, the adapter's r after d: never more than d + r + 8 roundings of partial
    # sums under `size`; bf16 results have u in two terms, 2^-17 of it.
    tol = (d + r + 8) * U32 * size + (2.0 ** -17 * size if out == "bf16" else 0.0)
    if act == "gelu":
        ref = torch.special.ndtr(ref) * ref
        # the slope is at most 1.13; GELU itself good to 1e-7 |z| (fp32) or, under bf16's rounding, 2e-5 |z| Phi(-|z|)
        tol = 1.13 * tol + (2e-7 if out == "f32" else 1.3e-5) * size
    half = U16 if out == "bf16" else U32
    assert torch.all((got - ref).abs() <= tol + half * (ref.abs() + tol))


@pytest.mark.parametrize("T,kind", [(5, "random"), (40, "random"), (600, "random"), (600, "runs")])
def test_what_others_hold_stays_out(T, kind):
    """Infinities and NaN in one adapter and in one token reach nobody else, bit for bit."""
    d, n, r, N = 256, 256, 16, 4
    g = torch.Generator().manual_seed(T)
    x, w, a, b, scale, _ = _gaussians(T, d, n, r, N, False, g)
    ids = _ids(T, N, kind, g)
    ids[0], ids[1], ids[2] = 2, 1, -1
    for out in ("f32", "bf16"):
        desc = moe.LoraDesc(T, d, n, r, N, out_dtype=out)
        want = _run(desc, x, ids, w, a, b, scale, None)
        a2, b2, x2, s2 = a.clone(), b.clone(), x.clone(), scale.clone()
        a2[2, 0, 5] = float("nan")
        b2[2, 7] = float("inf")
        s2[3] = float("inf")
        x2[1, 9] = float("inf")
        got = _run(desc, x2, ids, w, a2, b2, s2, None)
        clean = (ids != 2) & (ids != 3)
        clean[1] = False
        assert torch.equal(got[clean], want[clean])
        assert torch.all(torch.isnan(got[0])) and not torch.any(torch.isfinite(got[1]))


def test_a_large_first_product():
    """A x past bf16's range is infinite in the terms, and the result infinite or NaN, not a
    finite number; just under it stays finite."""
    T, d, n, r = 600, 256, 128, 8
    x = torch.zeros(T, d).bfloat16()
    x[:, 0] = 2.0 ** 100
    a = torch.zeros(1, r, d).bfloat16()
    a[0, 0, 0] = 2.0 ** 27
    w, b = torch.zeros(n, d).bfloat16(), torch.full((1, n, r), 2.0 ** -100).bfloat16()
    ids = torch.zeros(T, dtype=torch.int32)
    desc = moe.LoraDesc(T, d, n, r, 1, out_dtype="f32")
    assert torch.all(_run(desc, x, ids, w, a, b, None, None) == 2.0 ** 27)
    got = _run(desc, x, ids, w, a, b, torch.tensor([4.0]), None)
    assert not torch.any(torch.isfinite(got))


@pytest.mark.parametrize("T", [1, 20, 100, 600])
def test_gelu_of_large_values(T):
    """GELU of what is past any doubt: +inf stays, large values stay, -large is 0."""
    d, n = 256, 128
    x, w = torch.zeros(T, d).bfloat16(), torch.zeros(n, d).bfloat16()
    x[:, 0], w[:, 0] = 1.0, torch.tensor([float("inf"), 3e38, 1e5, 20.0, -20.0, -1e5, 0.0, 1.0] * 16).bfloat16()
    a, b = torch.zeros(1, 8, d).bfloat16(), torch.zeros(1, n, 8).bfloat16()
    ids = torch.full((T,), -1, dtype=torch.int32)
    ref = w[:, 0].double()
    ref = torch.where(ref > 1e4, ref, torch.special.ndtr(ref) * ref)
    for out, half in (("f32", U32), ("bf16", U16)):
        got = _run(moe.LoraDesc(T, d, n, 8, 1, act="gelu", out_dtype=out), x, ids, w, a, b, None, None).double()
        assert torch.all((got == ref) | ((got - ref).abs() <= half * ref.abs() + 2e-7 * 20))


@pytest.mark.parametrize("T", [3, 100, 700])
def test_shared_expert_is_its_two_products(T):
    d, F, g = 256, 640, torch.Generator().manual_seed(T)
    up, down = moe.LoraDesc(T, d, F, 16, 3, act="gelu", has_bias=True), moe.LoraDesc(T, F, d, 8, 2, out_dtype="f32")
    x, w, a, b, s, bi = _gaussians(T, d, F, 16, 3, True, g)
    _, w2, a2, b2, s2, _ = _gaussians(1, F, d, 8, 2, False, g)
    ids = _ids(T, 3, "runs", g).to(DEV)
    wu = moe.LoraWeights(w.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV), bi.to(DEV))
    wd = moe.LoraWeights(w2.to(DEV), a2.to(DEV), b2.to(DEV), s2.to(DEV))
    x = x.to(DEV)
    h, o, q = torch.empty(T, F, dtype=torch.bfloat16, device=DEV), torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    moe.moe_lora_linear(up, x, ids, wu, h)
    moe.moe_lora_linear(down, h, ids, wd, o)
    moe.moe_lora_shared_ffn(up, down, x, ids, wu, wd, q, workspace=moe.alloc_lora_shared_workspace(up, down, DEV).fill_(0xFF))
    assert torch.equal(o, q)


@pytest.mark.parametrize("T", [4, 90, 700])
def test_capture_streams_and_repetition(T):
    d, n, r, N = 256, 384, 16, 5
    g = torch.Generator().manual_seed(T)
    x, w, a, b, s, _ = _gaussians(T, d, n, r, N, False, g)
    weights = moe.LoraWeights(w.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV))
    x, ids = x.to(DEV), _ids(T, N, "random", g).to(DEV)
    desc = moe.LoraDesc(T, d, n, r, N)
    y, ws = torch.empty(T, n, dtype=torch.bfloat16, device=DEV), moe.alloc_lora_workspace(desc, DEV)
    moe.moe_lora_linear(desc, x, ids, weights, y, workspace=ws)
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.zero_()
        moe.moe_lora_linear(desc, x, ids, weights, y)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_lora_linear(desc, x, ids, weights, y, workspace=ws)
    for k in range(3):
        ids.copy_(_ids(T, N, "random", torch.Generator().manual_seed(k)))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        moe.moe_lora_linear(desc, x, ids, weights, y, workspace=ws)
        assert torch.equal(y, got)


# Under the tiled kernels: 128 x 128 tiles, and 256 x 256.
TILED = [(1400, 256, 2176), (8200, 256, 2176)]


@pytest.mark.parametrize("T,d,n", [(1, 256, 384), (20, 256, 384), (100, 256, 384), (600, 256, 384)] + TILED)
@pytest.mark.parametrize("kind", ["one", "runs", "random"])
def test_infinite_and_nan_factors_of_its_own(T, d, n, kind):
    """What a token's own adapter holds of infinities and NaN comes out as in 64 bits, sign and
    all, whatever tokens are beside it; other tokens keep their bits.  Exact values, as above."""
    r, N = 24, 4
    g = torch.Generator().manual_seed(T + d)
    x, w, a, b, scale, _ = _small_integers(T, d, n, r, N, False, g)
    ids = _ids(T, N, kind, g)
    inf, nan = float("inf"), float("nan")
    for i, c, q, v in ((0, 3, 2, inf), (1, 9, 5, -inf), (3, 70, 7, nan), (3, 100, 9, inf), (2, 33, 15, -inf), (1, 131, 12, nan),
                       (3, 200, 19, inf), (0, 255, 23, -inf), (2, 300, 16, nan), (3, 301, 0, -inf), (3, 301, 11, inf)):
        b[i, c, q] = v
    a[3, 6, 17], b[3, 310, 6], b[3, 311, 6] = inf, inf, -inf       # an infinite u, which meets them too
    ref, _ = _reference(x, w, a, b, scale, None, ids)
    for out in ("f32", "bf16"):
        got = _run(moe.LoraDesc(T, d, n, r, N, out_dtype=out), x, ids, w, a, b, scale, None)
        want = ref.float() if out == "f32" else ref.float().bfloat16()
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert torch.all(same), (out, (~same).nonzero()[:8].tolist())


# The cases above whose rows and columns are few run in parts of k; the same under the tiles.

@pytest.mark.parametrize("T,d,n", TILED)
@pytest.mark.parametrize("kind", ["random", "runs"])
def test_what_others_hold_stays_out_of_tiles(T, d, n, kind):
    r, N = 16, 4
    g = torch.Generator().manual_seed(T)
    x, w, a, b, scale, _ = _gaussians(T, d, n, r, N, False, g)
    ids = _ids(T, N, kind, g)
    ids[0], ids[1], ids[2] = 2, 1, -1
    for out in ("f32", "bf16"):
        desc = moe.LoraDesc(T, d, n, r, N, out_dtype=out)
        want = _run(desc, x, ids, w, a, b, scale, None)
        a2, b2, x2, s2 = a.clone(), b.clone(), x.clone(), scale.clone()
        a2[2, 0, 5] = float("nan")
        b2[2, 7, 3], b2[2, 9, 12] = float("inf"), float("nan")
        s2[3] = float("inf")
        x2[1, 9] = float("inf")
        got = _run(desc, x2, ids, w, a2, b2, s2, None)
        clean = (ids != 2) & (ids != 3)
        clean[1] = False
        assert torch.equal(got[clean], want[clean])
        assert torch.all(torch.isnan(got[0])) and not torch.any(torch.isfinite(got[1]))
        assert not torch.any(torch.isfinite(got[ids == 3]))


@pytest.mark.parametrize("T,d,n", TILED)
def test_a_large_first_product_in_tiles(T, d, n):
    r = 8
    x, a = torch.zeros(T, d).bfloat16(), torch.zeros(1, r, d).bfloat16()
    x[:, 0], a[0, 0, 0] = 2.0 ** 100, 2.0 ** 27
    w, b = torch.zeros(n, d).bfloat16(), torch.full((1, n, r), 2.0 ** -100).bfloat16()
    ids = torch.zeros(T, dtype=torch.int32)
    desc = moe.LoraDesc(T, d, n, r, 1, out_dtype="f32")
    assert torch.all(_run(desc, x, ids, w, a, b, None, None) == 2.0 ** 27)
    assert torch.all(_run(desc, x, ids, w, a, b, torch.tensor([4.0]), None) == float("inf"))


@pytest.mark.parametrize("T,n", [(1400, 2176), (8200, 2176)])
def test_a_first_product_of_24_bits_in_tiles(T, n):
    """A x of up to 24 bits, exact in fp32 in whatever order, and every bit of it in an fp32 result."""
    d, r, N = 1024, 24, 3
    g = torch.Generator().manual_seed(T)
    x = torch.randint(120, 128, (T, d), generator=g).bfloat16()
    a = torch.randint(100, 128, (N, r, d), generator=g).bfloat16()
    b = torch.zeros(N, n, r).bfloat16()
    b[:, torch.arange(n), torch.arange(n) % r] = 1.0
    ids = torch.randint(0, N, (T,), generator=g).to(torch.int32)
    u = torch.stack([x.double() @ a[i].double().T for i in range(N)])[ids.long(), torch.arange(T)]
    assert 2 ** 23 < u.min() and u.max() < 2 ** 24 and (u % 2 == 1).any()
    got = _run(moe.LoraDesc(T, d, n, r, N, out_dtype="f32"), x, ids, torch.zeros(n, d).bfloat16(), a, b, None, None)
    assert torch.equal(got.double(), u[:, torch.arange(n) % r])


@pytest.mark.parametrize("T,d,n", TILED)
def test_gelu_of_large_values_in_tiles(T, d, n):
    x, w = torch.zeros(T, d).bfloat16(), torch.zeros(n, d).bfloat16()
    x[:, 0], w[:, 0] = 1.0, torch.tensor([float("inf"), 3e38, 1e5, 20.0, -20.0, -1e5, 0.0, 1.0] * (n // 8)).bfloat16()
    a, b = torch.zeros(1, 8, d).bfloat16(), torch.zeros(1, n, 8).bfloat16()
    ids = torch.full((T,), -1, dtype=torch.int32)
    ref = w[:, 0].double()
    ref = torch.where(ref > 1e4, ref, torch.special.ndtr(ref) * ref)
    for out, half in (("f32", U32), ("bf16", U16)):
        got = _run(moe.LoraDesc(T, d, n, 8, 1, act="gelu", out_dtype=out), x, ids, w, a, b, None, None).double()
        assert torch.all((got == ref) | ((got - ref).abs() <= half * ref.abs() + 2e-7 * 20))


@pytest.mark.parametrize("T", [1400, 8200])
def test_shared_expert_in_tiles_is_its_two_products(T):
    d, F, g = 2176, 2304, torch.Generator().manual_seed(T)
    up, down = moe.LoraDesc(T, d, F, 16, 3, act="gelu", has_bias=True), moe.LoraDesc(T, F, d, 8, 2, out_dtype="f32")
    x, w, a, b, s, bi = _gaussians(T, d, F, 16, 3, True, g)
    _, w2, a2, b2, s2, _ = _gaussians(1, F, d, 8, 2, False, g)
    ids = _ids(T, 3, "runs", g).to(DEV)
    wu = moe.LoraWeights(w.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV), bi.to(DEV))
    wd = moe.LoraWeights(w2.to(DEV), a2.to(DEV), b2.to(DEV), s2.to(DEV))
    x = x.to(DEV)
    h, o, q = torch.empty(T, F, dtype=torch.bfloat16, device=DEV), torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    moe.moe_lora_linear(up, x, ids, wu, h)
    moe.moe_lora_linear(down, h, ids, wd, o)
    moe.moe_lora_shared_ffn(up, down, x, ids, wu, wd, q, workspace=moe.alloc_lora_shared_workspace(up, down, DEV).fill_(0xFF))
    assert torch.equal(o, q)


@pytest.mark.parametrize("T,d,n", TILED)
def test_capture_streams_and_repetition_in_tiles(T, d, n):
    r, N = 16, 5
    g = torch.Generator().manual_seed(T)
    x, w, a, b, s, _ = _gaussians(T, d, n, r, N, False, g)
    weights = moe.LoraWeights(w.to(DEV), a.to(DEV), b.to(DEV), s.to(DEV))
    x, ids = x.to(DEV), _ids(T, N, "random", g).to(DEV)
    desc = moe.LoraDesc(T, d, n, r, N)
    y, ws = torch.empty(T, n, dtype=torch.bfloat16, device=DEV), moe.alloc_lora_workspace(desc, DEV)
    moe.moe_lora_linear(desc, x, ids, weights, y, workspace=ws)
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.zero_()
        moe.moe_lora_linear(desc, x, ids, weights, y)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_lora_linear(desc, x, ids, weights, y, workspace=ws)
    for k in range(3):
        ids.copy_(_ids(T, N, "random", torch.Generator().manual_seed(k)))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        moe.moe_lora_linear(desc, x, ids, weights, y, workspace=ws)
        assert torch.equal(y, got)


def test_the_most_tokens_with_the_most_columns_of_a():
    """As many tokens as int32 allows, of 128 adapters of rank 128: 17.8 million blocks, offsets past 32 bits.  Exact
    values; the first rows, the last and some between are compared."""
    T, d, n, r, N = (1 << 24) - 1, 128, 128, 128, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("40 GB needed")
    g = torch.Generator().manual_seed(1)
    few, w, a, b, scale, _ = _small_integers(4096, d, n, r, N, False, g)
    x = few.to(DEV).repeat(4096, 1)[:T]
    ids = (torch.arange(T, device=DEV, dtype=torch.int32) // 517) % (N + 1) - 1
    y = torch.full((T, n), 7.0, dtype=torch.bfloat16, device=DEV)
    desc = moe.LoraDesc(T, d, n, r, N)
    moe.moe_lora_linear(desc, x, ids, moe.LoraWeights(w.to(DEV), a.to(DEV), b.to(DEV), scale.to(DEV)), y)
    at = torch.cat([torch.arange(3000), torch.randint(0, T, (20000,), generator=g), torch.arange(T - 3000, T)])
    ref, _ = _reference(few[at % 4096], w, a, b, scale, None, ids[at.to(DEV)].cpu())
    assert torch.equal(y[at.to(DEV)].cpu(), ref.float().bfloat16())
