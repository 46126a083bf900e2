"""GPU tests of the batched low-rank adapters against 64-bit references with element-wise bounds (tests/serving_reference.py):
sizes on both sides of every border (few rows and tiles, ragged tiles, ranks that are no multiple of 16, more adapters than
one pass or tile holds), rows without an adapter, and what a caller may do with them."""
import pytest
import torch

import nvfp4_block_scaled_16_b200 as nv
from tests import serving_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_block_scaled_16_b200 import build
    build.build()
    nv.load_library()
    yield


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert nv.nvfp4_device_status(clear=True) == 0, "a device-side wait timed out"


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def adapters_of(g, m, A, how):
    if how == "mixed":
        return torch.randint(-1, A, (m,), generator=g, device="cuda", dtype=torch.int32)
    if how == "sorted":
        return torch.randint(-1, A, (m,), generator=g, device="cuda", dtype=torch.int32).sort().values
    if how == "none":
        return torch.full((m,), -1, dtype=torch.int32, device="cuda")
    return torch.full((m,), A - 1, dtype=torch.int32, device="cuda")


DOWN = [(1, 64, 8, 1, "one"), (3, 320, 24, 4, "mixed"), (64, 128, 256, 3, "mixed"), (65, 192, 8, 70, "mixed"), (128, 1024, 64, 9, "mixed"),
        (129, 64, 8, 2, "mixed"), (130, 128, 40, 3, "none"), (200, 192, 256, 5, "mixed"), (257, 1024, 16, 40, "mixed"),
        (384, 320, 72, 200, "mixed"), (512, 64, 64, 30, "mixed"), (513, 64, 64, 30, "mixed"), (600, 192, 64, 300, "mixed"), (700, 576, 128, 6, "sorted"), (1000, 64, 200, 3, "sorted"), (513, 448, 104, 1, "one"),
        (400, 64, 200, 3, "none"), (400, 128, 104, 130, "none"), (400, 128, 256, 130, "mixed")]


@pytest.mark.parametrize("m,k,r,A,how", DOWN)
def test_lora_down_batched(m, k, r, A, how):
    g = gen(m + k + r)
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = (torch.randn((A, r, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
    adapter = adapters_of(g, m, A, how)
    big = torch.full((m + 2, r), 9.0, dtype=torch.bfloat16, device="cuda")
    d = nv.nvfp4_lora_down_batched(x, w, adapter, d_out=big[1:m + 1])
    assert (big[0] == 9).all() and (big[m + 1] == 9).all()
    R.assert_within(d, *R.lora_down(x, w, adapter))
    assert (d[adapter < 0] == 0).all()
    again = nv.nvfp4_lora_down_batched(x, w, adapter)
    assert torch.equal(again.view(torch.int16), d.view(torch.int16))


@pytest.mark.parametrize("r", [64, 104])
def test_lora_down_mixed_tiles_between_others(r):
    # tiles of one adapter, of 100 in turns, of none, of three, of 30, and a last one that ends inside
    g = gen(r)
    m, k, A = 5 * 128 + 72, 448, 100
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = (torch.randn((A, r, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
    i = torch.arange(m, device="cuda")
    kinds = torch.stack((torch.full_like(i, 7), i * 37 % A, torch.full_like(i, -1), i % 3, i % 31 - 1, i * 13 % (A + 2)))
    adapter = kinds[(i // 128).clamp(max=5), i].int()
    want = R.lora_down(x, w, adapter)
    big = torch.full((m + 2, r), 9.0, dtype=torch.bfloat16, device="cuda")
    d = nv.nvfp4_lora_down_batched(x, w, adapter, d_out=big[1:m + 1])
    assert (big[0] == 9).all() and (big[m + 1] == 9).all()
    R.assert_within(d, *want)
    nv.nvfp4_set_pdl(False)
    try:
        off = nv.nvfp4_lora_down_batched(x, w, adapter)
    finally:
        nv.nvfp4_set_pdl(True)
    assert torch.equal(off.view(torch.int16), d.view(torch.int16))
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out = nv.nvfp4_lora_down_batched(x, w, adapter)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            nv.nvfp4_lora_down_batched(x, w, adapter, d_out=out)
            nv.nvfp4_lora_down_batched(x, w, adapter, d_out=out)
    adapter.copy_(adapter.flip(0))
    out.fill_(9.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    R.assert_within(out, *R.lora_down(x, w, adapter))


def test_lora_down_rows_and_tiles_agree():
    # the first 128 rows of a longer call (tiles) and a call of their own (rows): the same products, fp32 sums in another order
    g = gen(3)
    x = torch.randn((1100, 512), generator=g, device="cuda").bfloat16()
    w = (torch.randn((7, 32, 512), generator=g, device="cuda") / 20).bfloat16()
    adapter = adapters_of(g, 1100, 7, "mixed")
    ref, err = R.lora_down(x, w, adapter)
    R.assert_within(nv.nvfp4_lora_down_batched(x, w, adapter), ref, err)
    R.assert_within(nv.nvfp4_lora_down_batched(x[:128], w, adapter[:128].contiguous()), ref[:128], err[:128])


@pytest.mark.parametrize("m", [40, 2100])
def test_lora_down_ids_out_of_range_and_non_finite_rows(m):
    g = gen(5)
    x = torch.randn((m, 192), generator=g, device="cuda").bfloat16()
    w = (torch.randn((4, 16, 192), generator=g, device="cuda") / 14).bfloat16()
    adapter = adapters_of(g, m, 4, "mixed")
    adapter[:4] = torch.tensor([4, 2 ** 31 - 1, -2 ** 31, -1], dtype=torch.int32, device="cuda")
    x[:4] = float("nan")                       # rows without an adapter are not read into anything
    x[7, 3] = float("inf")
    adapter[7] = 2
    d = nv.nvfp4_lora_down_batched(x, w, adapter)
    assert (d[:4] == 0).all() and not d[7].isfinite().any()
    ok = torch.ones(m, dtype=torch.bool, device="cuda")
    ok[7] = False
    ok[:4] = False
    ref, err = R.lora_down(x, w, torch.where((adapter < 0) | (adapter >= 4), -1, adapter))
    R.assert_within(d[ok], ref[ok], err[ok])


GEMM = [(1, 8, 64, 8, 1, "one", False), (1, 5120, 256, 16, 4, "one", True), (3, 440, 320, 48, 39, "mixed", False),
        (16, 256, 128, 16, 20, "mixed", True), (17, 264, 192, 64, 3, "mixed", False), (128, 392, 320, 16, 50, "mixed", True), (129, 392, 320, 16, 50, "mixed", True),
        (8, 136, 64, 256, 3, "mixed", True), (9, 136, 64, 256, 3, "mixed", False), (64, 1000, 320, 8, 64, "mixed", True),
        (65, 384, 448, 24, 5, "mixed", True), (128, 128, 64, 256, 3, "mixed", False), (129, 520, 576, 32, 30, "mixed", True),
        (256, 256, 256, 72, 300, "mixed", False), (257, 136, 128, 16, 7, "none", True), (300, 776, 832, 40, 6, "sorted", True),
        (700, 2048, 192, 128, 4, "sorted", False), (1024, 264, 1024, 16, 500, "mixed", True)]


def operands(g, m, n, k, r, A):
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = (torch.randn((n, k), generator=g, device="cuda") * 0.05).bfloat16()
    amax_b, _, _, b, b_sf = nv.nvfp4_global_scale_quantize(w)
    _, _, alpha, a, a_sf = nv.nvfp4_global_scale_quantize(x, other_amax=amax_b)
    d = torch.randn((m, r), generator=g, device="cuda").bfloat16()
    l1 = (torch.randn((A, n, r), generator=g, device="cuda") * (0.5 / r ** 0.5)).bfloat16()
    bias = (torch.randn(n, generator=g, device="cuda") * 0.1).bfloat16()
    return a, b, a_sf, b_sf, alpha, d, l1, bias


@pytest.mark.parametrize("m,n,k,r,A,how,with_bias", GEMM)
def test_gemm_lora_batched(m, n, k, r, A, how, with_bias):
    g = gen(m + n + k)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, n, k, r, A)
    adapter = adapters_of(g, m, A, how)
    bias = bias if with_bias else None
    big = torch.full((m * n + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias, out=big[32:32 + m * n].view(m, n))
    assert (big[:32] == 9).all() and (big[32 + m * n:] == 9).all()
    R.assert_within(out, *R.gemm_lora(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias))
    need = nv.nvfp4_gemm_lora_batched_workspace(m, n, k, r, A)
    dirty = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    again = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias, workspace=dirty)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("m", [5, 70, 300])
def test_gemm_lora_without_adapters_is_the_plain_gemm(m):
    g = gen(11)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, 264, 320, 16, 3)
    d.fill_(float("nan"))                      # not read where a row has no adapter
    adapter = adapters_of(g, m, 3, "none")
    adapter[1] = 3
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    R.assert_within(out, *R.gemm_lora(a, b, a_sf, b_sf, alpha, d, l1, torch.full_like(adapter, -1), bias))
    plain = nv.nvfp4_gemm(a, b, a_sf, b_sf, alpha, bias=bias)
    R.assert_within(plain, *R.gemm_lora(a, b, a_sf, b_sf, alpha, d, l1, torch.full_like(adapter, -1), bias))


@pytest.mark.parametrize("m", [6, 300])
def test_gemm_lora_non_finite_row_leaves_the_others(m):
    g = gen(12)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, 264, 320, 16, 3)
    adapter = adapters_of(g, m, 3, "one")
    clean = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter)
    d[3, 5] = float("nan")
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter)
    rest = torch.arange(m, device="cuda") != 3
    assert out[3].isnan().all()
    assert torch.equal(out[rest].view(torch.int16), clean[rest].view(torch.int16))


@pytest.mark.parametrize("m", [7, 300])
def test_lora_captured_and_replayed_on_another_stream(m):
    g = gen(13)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, 264, 320, 16, 5)
    x = torch.randn((m, 320), generator=g, device="cuda").bfloat16()
    w = (torch.randn((5, 16, 320), generator=g, device="cuda") / 18).bfloat16()
    adapter = adapters_of(g, m, 5, "mixed")

    def step():
        dd = nv.nvfp4_lora_down_batched(x, w, adapter)
        return dd, nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, dd, l1, adapter, bias=bias)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    adapter.copy_(adapters_of(g, m, 5, "sorted"))
    x.copy_(torch.randn((m, 320), generator=g, device="cuda"))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        graph.replay()
        graph.replay()
    st.synchronize()
    R.assert_within(got[0], *R.lora_down(x, w, adapter))
    R.assert_within(got[1], *R.gemm_lora(a, b, a_sf, b_sf, alpha, got[0], l1, adapter, bias))


def test_lora_pdl_on_and_off_give_identical_bytes():
    g = gen(14)
    before = nv.nvfp4_get_pdl()
    try:
        for m in (9, 300):
            a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, 264, 320, 16, 5)
            adapter = adapters_of(g, m, 5, "mixed")
            got = []
            for pdl in (True, False):
                nv.nvfp4_set_pdl(pdl)
                got.append(nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias))
            assert torch.equal(got[0].view(torch.int16), got[1].view(torch.int16))
    finally:
        nv.nvfp4_set_pdl(before)


def test_lora_refusals():
    g = gen(15)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, 4, 264, 320, 16, 5)
    adapter = adapters_of(g, 4, 5, "mixed")
    x = torch.zeros((4, 320), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((5, 16, 320), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="adapter"):
        nv.nvfp4_lora_down_batched(x, w, adapter.long())
    with pytest.raises(ValueError, match="adapter"):
        nv.nvfp4_lora_down_batched(x, w, adapter[:3])
    with pytest.raises(ValueError, match="w"):
        nv.nvfp4_lora_down_batched(x, w.float(), adapter)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_lora_down_batched(x, w[:, :12].contiguous(), adapter)
    with pytest.raises(ValueError, match="l1"):
        nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1[:, :8].contiguous(), adapter)
    with pytest.raises(ValueError, match="bias"):
        nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias.float())
    with pytest.raises(ValueError, match="must be on"):
        nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter.cpu())
    many = operands(g, 400, 264, 320, 16, 5)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_gemm_lora_batched(*many[:7], adapters_of(g, 400, 5, "mixed"),
                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert nv.nvfp4_lora_down_batched(x[:0], w, adapter[:0]).shape == (0, 16)


def test_lora_adapters_beyond_four_gigabytes():
    A, n, r, k = 300, 65536, 128, 64                     # l1: 5 GB
    l1 = torch.zeros((A, n, r), dtype=torch.bfloat16, device="cuda")
    g = gen(21)
    for a in (0, A - 1):
        l1[a] = (torch.randn((n, r), generator=g, device="cuda") * 0.05).bfloat16()
    for m in (3, 300):
        a, b, a_sf, b_sf, alpha, d, _, bias = operands(g, m, n, k, r, 1)
        adapter = torch.where(torch.arange(m, device="cuda") % 2 == 0, A - 1, 0).int()
        out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
        at = torch.where(adapter == 0, 0, 1).int()
        R.assert_within(out, *R.gemm_lora(a, b, a_sf, b_sf, alpha, d, torch.stack((l1[0], l1[A - 1])), at, bias))
