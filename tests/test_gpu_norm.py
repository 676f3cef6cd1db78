"""The norm before a GEMM (scaled_gemm_norm_quantize) against 64-bit arithmetic and the CPU oracle's quantiser.

The header states each fp32 step: the kept sum, the nearest fp32 number to the inverse root, two products.
So y is formed here by the same steps from a 64-bit root, and codes and scales have to match
bit for bit; a row may have the root's neighbour instead (about one in 2^16 does)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

MODES = ["bf16", "ptpc", "blockscale", "mxfp8"]


@pytest.fixture(scope="module")
def norm():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")
    import gpu_util

    gpu_util.lib_ready()
    from fp8_scaled_gemm_sm_gb300 import norm_quantize

    return norm_quantize


def _make(R, C, seed, dtype):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-12, 12, (R, 1), generator=g).float())
    r = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-3, 6, (1, C), generator=g).float())
    w = 1 + 0.5 * torch.randn(C, generator=g)
    if R > 4:
        x[1], r[1] = 0.0, 0.0               # y is zero
        x[2] *= 1e-12                       # eps decides
        r[2] = 0.0
        x[3, 3 % C] = 2.0 ** 60             # one value outweighs the rest
        x[4] *= 2.0 ** 80                   # squares past fp32's largest
    return x.to(dtype), r.to(dtype), w.to(dtype)


def _expect(mode, kept, w, eps, root):
    y = (kept * root[:, None]).astype(np.float32) * w[None, :]
    assert y.dtype == np.float32
    if mode == "bf16":
        return torch.from_numpy(y).bfloat16().view(torch.int16).numpy(), None
    return oracle.quantize(mode, y)


def _check(mode, x, r, w, eps, got):
    codes, scale, kept = (None if t is None else t.cpu() for t in got)
    total = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(kept.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                       total.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32))
    t = total.float().numpy()
    root = (1.0 / np.sqrt((t.astype(np.float64) ** 2).mean(1) + eps)).astype(np.float32)
    have = codes.view(torch.int16).numpy() if mode == "bf16" else codes.numpy()
    per_row = (lambda s: s) if mode in ("ptpc", "bf16") else (lambda s: s.T)

    def wrong(root):
        q, s = _expect(mode, t, w.float().numpy(), eps, root)
        bad = (have != q).any(1)
        if s is not None:
            differ = per_row(scale.numpy()).reshape(len(t), -1) != per_row(s).reshape(len(t), -1)
            bad |= differ.any(1)
        return bad

    bad = wrong(root)
    near = [wrong(np.nextafter(root, np.float32(to))) for to in (np.inf, 0)]
    assert not (bad & near[0] & near[1]).any(), np.flatnonzero(bad & near[0] & near[1])[:5]
    assert bad.sum() <= 2, bad.sum()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(1, 128), (7, 1792), (301, 2048), (40, 7168), (9, 8320), (5, 16512), (3, 32768), (1400, 256)])
def test_steps(norm, mode, dtype, R, C):
    x, r, w = _make(R, C, R + C, dtype)
    got = norm(mode, x.cuda(), w.cuda(), 1e-6, residual=r.cuda())
    _check(mode, x, r, w, 1e-6, got)


@pytest.mark.parametrize("mode,C", [("bf16", 8), ("bf16", 200), ("ptpc", 16), ("ptpc", 2064), ("mxfp8", 32), ("mxfp8", 2080), ("bf16", 2056)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_odd_widths_without_residual(norm, mode, C, dtype):
    x, _, w = _make(6, C, C, dtype)
    dx = x.cuda()
    codes, scale, kept = norm(mode, dx, w.cuda(), 0.5)
    assert kept.data_ptr() == dx.data_ptr()
    _check(mode, x, None, w, 0.5, (codes, scale, kept))


def test_in_place(norm):
    x, r, w = _make(33, 2048, 3, torch.bfloat16)
    want = norm("ptpc", x.cuda(), w.cuda(), residual=r.cuda())
    for target in (0, 1):
        dev = [x.cuda(), r.cuda()]
        got = norm("ptpc", dev[0], w.cuda(), residual=dev[1], residual_out=dev[target])
        assert got[2].data_ptr() == dev[target].data_ptr()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("R,C", [(700, 7168), (1250, 2048), (611, 2304), (613, 4992), (610, 8192), (612, 16384)])
def test_many_rows(norm, mode, R, C):
    """More rows than the CTAs have in their first turns, in place; every thread's vectors there, or some past the row."""
    x, r, w = _make(R, C, R + C, torch.bfloat16)
    x[R - 1] *= 2.0 ** 80  # the last row of a CTA
    dx = x.cuda()
    got = norm(mode, dx, w.cuda(), 1e-6, residual=r.cuda(), residual_out=dx)
    assert got[2].data_ptr() == dx.data_ptr()
    _check(mode, x, r, w, 1e-6, got)


def test_many_rows_without_residual(norm):
    x, _, w = _make(700, 4096, 9, torch.bfloat16)
    _check("ptpc", x, None, w, 1e-6, norm("ptpc", x.cuda(), w.cuda(), 1e-6))


def test_many_rows_of_bf16_over_the_residual(norm):
    from fp8_scaled_gemm_sm_gb300 import binding

    x, r, w = (t.cuda() for t in _make(900, 4096, 10, torch.bfloat16))
    want, _, kept = norm("bf16", x, w, residual=r)
    binding.scaled_gemm_norm_quantize("bf16", "bf16", x.data_ptr(), r.data_ptr(), x.data_ptr(), w.data_ptr(), 1e-6, 900, 4096, r.data_ptr(), 0,
                                      torch.cuda.current_stream().cuda_stream)
    assert torch.equal(r, want) and torch.equal(x, kept)


def test_bf16_over_its_input(norm):
    from fp8_scaled_gemm_sm_gb300 import binding

    x, r, w = (t.cuda() for t in _make(20, 1024, 4, torch.bfloat16))
    want = norm("bf16", x, w, residual=r)[0]
    kept = torch.empty_like(x)
    binding.scaled_gemm_norm_quantize("bf16", "bf16", x.data_ptr(), r.data_ptr(), kept.data_ptr(), w.data_ptr(), 1e-6, 20, 1024, x.data_ptr(), 0,
                                      torch.cuda.current_stream().cuda_stream)
    assert torch.equal(x, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_eps_beside_large_rows(norm, dtype):
    """Row sums past 2^90, where squares are formed of scaled elements, and an eps of 2^-20 and 2^-25 of their means."""
    g = torch.Generator("cpu").manual_seed(8)
    x = ((1 + torch.rand(6, 32768, generator=g)) * torch.tensor([2.0 ** 40, 2.0 ** 42, 2.0 ** 38, 2.0 ** 37.5, 2.0 ** 30, 2.0 ** 60])[:, None]).to(dtype)
    w = torch.ones(32768, dtype=dtype)
    for eps in (2.0 ** 60, 3e17):
        _check("ptpc", x, None, w, eps, norm("ptpc", x.cuda(), w.cuda(), eps))


def test_the_quantiser_gives_the_same_codes(norm):
    """What the norm quantises is what binding.quantize makes of the same y in fp32."""
    from fp8_scaled_gemm_sm_gb300 import binding

    x, r, w = (t.cuda() for t in _make(50, 1024, 5, torch.float32))
    kept = norm("bf16", x, w, residual=r)[2]
    root = (1.0 / (kept.double().square().mean(1, keepdim=True) + 1e-6).sqrt()).float()
    for mode in MODES[1:]:
        q, s = binding.quantize(mode, kept * root * w)
        codes, scale, _ = norm(mode, x, w, residual=r)
        assert (codes != q).any(1).sum() <= 1 and torch.equal(scale.view(torch.uint8), s.view(torch.uint8))


def test_graph_and_stream(norm):
    x, r, w = (t.cuda() for t in _make(17, 7168, 6, torch.bfloat16))
    want = norm("mxfp8", x, w, residual=r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = norm("mxfp8", x, w, residual=r)
    for t in got:
        t.zero_()
    graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm("mxfp8", x, w, residual=r, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_many_rows_captured_in_place(norm):
    """The graph adds the residual again with each replay, and rows that are not finite stay alone."""
    x, r, w = (t.cuda() for t in _make(1000, 4096, 11, torch.bfloat16))
    x[7, 5], x[650, 9] = float("inf"), float("nan")
    add, kept = r.clone(), x.clone()
    norm("mxfp8", kept.clone(), w, residual=add)  # loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scale, _ = norm("mxfp8", kept, w, residual=add, residual_out=kept)
    want = x
    for _ in range(3):
        graph.replay()
        wc, ws, want = norm("mxfp8", want, w, residual=add)
        assert torch.equal(codes, wc) and torch.equal(scale, ws) and torch.equal(kept.view(torch.int16), want.view(torch.int16))
    rest = [i for i in range(1000) if i not in (7, 650)]
    clean, _, _ = norm("mxfp8", torch.where(torch.isfinite(x), x, 0), w, residual=add)
    first, _, _ = norm("mxfp8", x, w, residual=add)
    assert torch.equal(first[rest], clean[rest])


def test_tensor_refusals(norm):
    from fp8_scaled_gemm_sm_gb300 import ScaledGemmError

    x, r, w = (t.cuda() for t in _make(4, 256, 7, torch.bfloat16))
    for bad in (dict(x=x.cpu()), dict(x=x.half()), dict(x=x[:, ::2]), dict(x=x[0]), dict(weight=w[:-8]), dict(weight=w.float()),
                dict(residual=r[:2]), dict(residual=r.float()), dict(residual=None, residual_out=r), dict(residual_out=r[:2]), dict(mode="fp4")):
        a = dict(dict(mode="ptpc", x=x, weight=w, residual=r), **bad)
        with pytest.raises((ValueError, TypeError)):
            norm(**a)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ScaledGemmError):
            norm("ptpc", x, w, eps)
    with pytest.raises(ScaledGemmError):
        norm("blockscale", x[:, :144].contiguous(), w[:144].contiguous())
    assert norm("ptpc", x[:0], w)[0].shape == (0, 256)


def _pieces(norm, mode, x, r, w, each):
    """The same rows in calls of `each` and the rest: a row or less for every CTA."""
    codes, scale = [], []
    for i in range(0, x.shape[0], each):
        c, s, _ = norm(mode, x[i:i + each], w, 1e-6, residual=None if r is None else r[i:i + each])
        codes.append(c), scale.append(s)
    return torch.cat(codes), None if scale[0] is None else torch.cat(scale, 0 if mode == "ptpc" else 1)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("R,C,dtype,residual", [
    (9000, 256, torch.bfloat16, True),     # a warp a row
    (9000, 384, torch.float32, False),     # two, with the next row on its way
    (8000, 896, torch.bfloat16, True),     # two, some lanes past the row
    (3000, 2048, torch.float32, True),
    (2600, 8192, torch.float32, True),     # a vector a thread, 1024 threads
    (2700, 4096, torch.bfloat16, False),
    (2500, 7680, torch.bfloat16, True),    # wide rows whose threads have no whole vectors
    (2500, 12288, torch.float32, True),
    (2600, 16384, torch.bfloat16, False),
    (2490, 10752, torch.bfloat16, True),
    (2500, 20480, torch.bfloat16, True),   # eight vectors a thread
    (2450, 20608, torch.float32, False),
])
def test_rows_in_their_ctas_later_turns(norm, mode, R, C, dtype, residual):
    """The loop over rows without shared memory, in place: as in calls whose CTAs have a row each, bit for bit."""
    g = torch.Generator("cuda").manual_seed(R + C)
    x = torch.randn(R, C, generator=g, device="cuda") * torch.exp2(torch.randint(-12, 12, (R, 1), generator=g, device="cuda").float())
    r = torch.randn(R, C, generator=g, device="cuda") if residual else None
    for i in (1215, 1216, 1217, 2432, 2433, 3647, 3648, R - 1):  # the last row of a turn, the first ones of the next
        if i < R:
            x[i] *= 2.0 ** 80
    x[1300, 5], x[2440, C - 1] = float("inf"), float("nan")
    w = 1 + 0.5 * torch.randn(C, generator=g, device="cuda")
    x, w = x.to(dtype), w.to(dtype)
    r = None if r is None else r.to(dtype)
    want = _pieces(norm, mode, x, r, w, 1000)
    total = x if r is None else (x.float() + r.float()).to(dtype)
    kept = x.clone() if residual else None
    codes, scale, got = norm(mode, x if kept is None else kept, w, 1e-6, residual=r, residual_out=kept)
    rows = torch.tensor([i for i in range(R) if i not in (1300, 2440)], device="cuda")
    assert torch.equal(codes[rows].view(torch.uint8), want[0][rows].view(torch.uint8))
    if scale is not None:
        dim = 0 if mode == "ptpc" else 1
        assert torch.equal(scale.index_select(dim, rows).view(torch.uint8), want[1].index_select(dim, rows).view(torch.uint8))
    assert torch.equal(got[rows], total[rows])


@pytest.mark.parametrize("mode", ["blockscale", "mxfp8"])
@pytest.mark.parametrize("R,C,dtype,residual", [(8000, 256, torch.bfloat16, True), (3000, 2048, torch.float32, True), (2600, 1152, torch.bfloat16, False)])
def test_later_turns_against_the_oracle(norm, mode, R, C, dtype, residual):
    x, r, w = _make(R, C, R + C, dtype)
    x[R - 1] *= 2.0 ** 80
    dx = x.cuda()
    got = norm(mode, dx, w.cuda(), 1e-6, residual=r.cuda() if residual else None, residual_out=dx if residual else None)
    _check(mode, x, r if residual else None, w, 1e-6, got)


@pytest.mark.parametrize("R,C,residual", [(140000, 16384, True), (66000, 32768, False)])
def test_offsets_past_31_bits(norm, R, C, residual):
    """More than 2^31 elements: the last rows as in a call of their own."""
    g = torch.Generator("cuda").manual_seed(R)
    some = torch.randn(1000, C, generator=g, device="cuda").bfloat16()
    x = some.repeat(R // 1000, 1)
    x[-700:] = torch.randn(700, C, generator=g, device="cuda").bfloat16()
    w = (1 + 0.3 * torch.randn(C, generator=g, device="cuda")).bfloat16()
    r = x.flip(0) if residual else None
    part = x[-700:].clone()
    want = norm("mxfp8", part, w, residual=r[-700:].clone() if residual else None)
    codes, scale, kept = norm("mxfp8", x, w, residual=r, residual_out=x if residual else None)
    assert torch.equal(codes[-700:], want[0]) and torch.equal(scale[:, -700:], want[1]) and torch.equal(kept[-700:], want[2])
