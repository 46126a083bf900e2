"""GPU tests of what the serving-step operators must not depend on or disturb: scale bytes of rows beyond a matrix, memory that
another stream still uses; and of scale factors at the ends of their range."""
import pytest
import torch

import nvfp4_block_scaled_16_b200 as nv
from tests import serving_reference as R
from tests.test_lora_batched_gpu import adapters_of, gen, operands
from tests.test_moe_gpu import call, case

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


def bits(t):
    return t.view(torch.int16)


def padding(rows, k):
    """Which bytes of a scale tensor (128x4 layout) of a [rows, k] matrix belong to rows beyond it."""
    at = torch.arange(nv.nvfp4_scale_bytes(rows, k), device="cuda")
    chunk, byte = at // 512, at % 512
    row = chunk // (-(-k // 64)) * 128 + byte // 16 + byte % 16 // 4 * 32
    return row >= rows


# ---- expert layer: scale bytes of the rows beyond n (gate, up) and k (down) -----------------------------------------

@pytest.mark.parametrize("byte", [0x7F, 0xFF, 0x7E])     # NaN, NaN, the largest finite scale
@pytest.mark.parametrize("t,E,topk,n,k", [(1, 3, 2, 192, 320), (5, 3, 2, 192, 320), (20, 3, 2, 192, 320), (1, 2, 1, 64, 64),
                                          (7, 2, 2, 704, 128), (40, 5, 3, 64, 192), (33, 4, 2, 320, 256)])
def test_moe_ignores_scales_of_padding_rows(t, E, topk, n, k, byte):
    x, ids, weights, w = case(t, E, topk, n, k)
    want = call(x, ids, weights, w)
    R.assert_within(want, *R.moe(x, ids, weights, w, E))
    other = {}
    for name, (rows, cols) in (("gate", (n, k)), ("up", (n, k)), ("down", (k, n))):
        q, sf, amax = w[name]
        sf = sf.clone()
        sf[:, padding(rows, cols)] = byte
        other[name] = (q, sf, amax)
    assert torch.equal(bits(call(x, ids, weights, other)), bits(want))


def test_moe_of_weights_quantized_with_a_mask():
    # the masked quantizer leaves the scales of padding rows as they were
    t, E, topk, n, k = 6, 3, 2, 192, 320
    x, ids, weights, w = case(t, E, topk, n, k)
    want = call(x, ids, weights, w)
    g = torch.Generator(device="cuda")
    g.manual_seed(101)                                    # the matrices of case()
    other = {}
    for name, (rows, cols) in (("gate", (n, k)), ("up", (n, k)), ("down", (k, n))):
        m = (torch.randn((E, rows, cols), generator=g, device="cuda") * 0.05 *
             (0.5 + torch.rand((E, 1, 1), generator=g, device="cuda"))).bfloat16()
        full = torch.full((E,), rows, dtype=torch.int32, device="cuda")
        amax, gsf = nv.nvfp4_global_scale_batched(m, mask=full)
        sf = torch.full((E, nv.nvfp4_scale_bytes(rows, cols)), 0xFF, dtype=torch.uint8, device="cuda")
        q, sf = nv.nvfp4_quantize_masked_batched(m, gsf, mask=full, sf_out=sf)
        assert torch.equal(q, w[name][0])
        other[name] = (q, sf, amax)
    assert torch.equal(bits(call(x, ids, weights, other)), bits(want))


# ---- a stream of its own ------------------------------------------------------------------------------------------------

def test_memory_in_use_on_the_current_stream_is_left_alone():
    # temporaries of the sizes that the call needs are freed here while this stream's kernels have yet to read them
    t, E, topk, n, k = 24, 6, 2, 320, 448
    x, ids, weights, w = case(t, E, topk, n, k)
    want = call(x, ids, weights, w)
    need = nv.nvfp4_moe_few_tokens_workspace(t, topk, E, n, k)
    st = torch.cuda.Stream()
    for _ in range(3):
        temps = [torch.full((need,), 5, dtype=torch.uint8, device="cuda"), torch.full_like(x, 5)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        copies = [torch.empty_like(v) for v in temps]
        for c, v in zip(copies, temps):
            c.copy_(v)
        del temps, v
        got = call(x, ids, weights, w, stream=st)
        st.synchronize()
        assert torch.equal(bits(got), bits(want))
        torch.cuda.synchronize()
        assert all((c == 5).all() for c in copies)


# ---- batched adapters: alpha 0, and d / alpha beyond what bf16 and the accumulator hold ------------------------------------

# both sides of the border between the two forms (m * r 2048), ragged tiles, a rank that is no multiple of 16, more adapters
# than rows
SIZES = [(6, 264, 320, 16, 3), (128, 136, 64, 16, 5), (129, 264, 320, 16, 5), (64, 520, 192, 40, 80), (300, 776, 320, 256, 4),
         (513, 136, 576, 24, 300)]


def low_rank_in_fp32(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias):
    """out and its bound where d * l1 is summed in fp32 and nothing but the output is rounded to fewer bits."""
    av, bv, al = R.values(a, a_sf), R.values(b, b_sf), alpha.double()
    out, mag = av @ bv.t() * al, (av.abs() @ bv.abs().t()) * al.abs()
    for i in range(l1.shape[0]):
        at = (adapter == i).nonzero()[:, 0]
        out[at] += d[at].double() @ l1[i].double().t()
        mag[at] += d[at].double().abs() @ l1[i].double().abs().t()
    if bias is not None:
        out, mag = out + bias.double(), mag + bias.double().abs()
    err = R.FP32_SUM * mag
    return out, err + R.BF16_HALF_STEP * (out.abs() + err)


@pytest.mark.parametrize("m,n,k,r,A", SIZES)
@pytest.mark.parametrize("alpha", [0.0, -0.0, 2.0 ** -140, -2.0 ** -100])
def test_gemm_lora_with_alpha_zero_or_tiny(m, n, k, r, A, alpha):
    g = gen(m + n + r)
    a, b, a_sf, b_sf, al, d, l1, bias = operands(g, m, n, k, r, A)
    al.fill_(alpha)
    for how in ("mixed", "none"):
        adapter = adapters_of(g, m, A, how)
        for bi in (bias, None):
            big = torch.full((m * n + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
            out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, al, d, l1, adapter, bias=bi, out=big[32:32 + m * n].view(m, n))
            assert (big[:32] == 9).all() and (big[32 + m * n:] == 9).all()
            R.assert_within(out, *low_rank_in_fp32(a, b, a_sf, b_sf, al, d, l1, adapter, bi), how)
        out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, al, torch.zeros_like(d), l1, adapter, bias=bias)
        if abs(alpha) < 2.0 ** -130:
            assert torch.equal(out, bias.expand(m, n))


@pytest.mark.parametrize("m,n,k,r,A", SIZES)
@pytest.mark.parametrize("alpha", [2.0 ** 33, 2.0 ** 126, -2.0 ** 127])
def test_gemm_lora_with_a_large_alpha(m, n, k, r, A, alpha):
    # d / alpha would leave bf16's normal range; the FP4 product is zero, so that the low-rank term is all there is
    g = gen(m + n + r + 4)
    a, b, a_sf, b_sf, al, d, l1, bias = operands(g, m, n, k, r, A)
    a.zero_()
    al.fill_(alpha)
    d[::3] *= 2.0 ** -70
    adapter = adapters_of(g, m, A, "mixed")
    for bi in (bias, None):
        out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, al, d, l1, adapter, bias=bi)
        R.assert_within(out, *low_rank_in_fp32(a, b, a_sf, b_sf, al, d, l1, adapter, bi))


def test_gemm_lora_of_an_all_zero_activation():
    # as a warm-up or a graph's capture on a zeroed batch runs it
    m, n, k, r, A = 300, 264, 320, 16, 3
    g = gen(31)
    _, b, _, b_sf, _, _, l1, bias = operands(g, m, n, k, r, A)
    w = (torch.randn((n, k), generator=g, device="cuda") * 0.05).bfloat16()
    amax_b, _, _, b, b_sf = nv.nvfp4_global_scale_quantize(w)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    _, _, alpha, a, a_sf = nv.nvfp4_global_scale_quantize(x, other_amax=amax_b)
    adapter = adapters_of(g, m, A, "mixed")
    d = nv.nvfp4_lora_down_batched(x, torch.randn((A, r, k), generator=g, device="cuda").bfloat16(), adapter)
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    assert torch.equal(out, bias.expand(m, n))


@pytest.mark.parametrize("m,n,k,r,A", SIZES)
def test_gemm_lora_rows_of_large_d_beside_others(m, n, k, r, A):
    g = gen(m + n + r + 1)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, n, k, r, A)
    adapter = adapters_of(g, m, A, "mixed")
    clean = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    big = torch.rand(m, generator=g, device="cuda") < 0.2
    big[m - 1] = True
    big[0] = False
    d[big] *= 2.0 ** 80
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    assert torch.equal(bits(out[~big]), bits(clean[~big]))
    ref, err = low_rank_in_fp32(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias)
    R.assert_within(out[big], ref[big], err[big])
    need = nv.nvfp4_gemm_lora_batched_workspace(m, n, k, r, A)
    dirty = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    again = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias, workspace=dirty)
    assert torch.equal(bits(again), bits(out))


# ---- batched adapters: an adapter's weights reach its own rows only ------------------------------------------------------

@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38, 2.0 ** 51])
@pytest.mark.parametrize("m,n,k,r,A", SIZES)
def test_gemm_lora_adapter_of_any_values_leaves_the_others(m, n, k, r, A, value):
    g = gen(m + n + r + 2)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, n, k, r, A)
    for how in ("mixed", "sorted"):
        adapter = adapters_of(g, m, A, how)
        l1 = l1.clone().nan_to_num(0.25, 0.25, 0.25).clamp(-4, 4)
        clean = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
        bad = sorted({int(adapter.max()), A - 1, int(adapter[m // 2])} - {-1})
        if len(bad) == A:
            bad = bad[:1]
        for i, e in enumerate(bad):                       # a value in the first row of l1, in the last, in the middle
            l1[e, (0, n - 1, n // 2)[i], (r - 1, 0, r // 2)[i]] = value
        out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
        own = torch.isin(adapter, torch.tensor(bad, device="cuda", dtype=torch.int32))
        assert own.any()
        assert torch.equal(bits(out[~own]), bits(clean[~own]))
        # its own rows: what the formula gives, column by column
        ref, err = low_rank_in_fp32(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias)
        ref, err, got = ref[own], err[own], out[own].double()
        edge = ref.abs() + err >= torch.finfo(torch.bfloat16).max          # may round to an infinity, or be one
        R.assert_within(torch.where(edge | ref.isnan(), 0.0, got), torch.where(edge | ref.isnan(), 0.0, ref), err.nan_to_num(1.0), how)
        assert (got.isnan() | got.isinf())[ref.isnan() | ref.isinf()].all()
        assert torch.equal(got.isnan() & ~edge, ref.isnan() & ~edge)
        assert (ref.isnan() | edge).any(0).sum() <= len(bad)


@pytest.mark.parametrize("A,m", [(40, 700), (3000, 1300), (65536, 2100)])
def test_gemm_lora_many_bad_adapters_among_good_ones(A, m):
    n, k, r = 64, 128, 32
    g = gen(A)
    a, b, a_sf, b_sf, alpha, d, _, bias = operands(g, m, n, k, r, 1)
    l1 = torch.zeros((A, n, r), dtype=torch.bfloat16, device="cuda")
    adapter = torch.randint(-1, A, (m,), generator=g, device="cuda", dtype=torch.int32)
    used = adapter.unique()
    used = used[used >= 0].long()
    l1[used] = (torch.randn((used.numel(), n, r), generator=g, device="cuda") * 0.1).bfloat16()
    clean = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    bad = used[torch.rand(used.numel(), generator=g, device="cuda") < 0.4]
    l1[bad, torch.randint(0, n, (bad.numel(),), generator=g, device="cuda")] = float("nan")
    need = nv.nvfp4_gemm_lora_batched_workspace(m, n, k, r, A)
    for byte in (0, 0xFF):
        ws = torch.full((need,), byte, dtype=torch.uint8, device="cuda")
        out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias, workspace=ws)
        own = torch.isin(adapter.long(), bad)
        assert own.any() and torch.equal(bits(out[~own]), bits(clean[~own]))
        assert (out[own].isnan().sum(1) == 1).all()


def assert_within_bf16(got, ref, err):
    """R.assert_within, where a result beyond bf16's range (values from 2^128 - 2^119 on round to an infinity) has to be the
    infinity of its sign.  No result may lie so near to that border that its bound allows both."""
    beyond = ref.abs() - err >= 2.0 ** 128
    assert (beyond | (ref.abs() + err < 2.0 ** 127)).all()
    assert torch.equal(got[beyond].double(), torch.sign(ref[beyond]) * float("inf"))
    R.assert_within(got[~beyond], ref[~beyond], err[~beyond])


@pytest.mark.parametrize("m,n,k", [(2011, 2568, 320), (2048, 4864, 4096)])
def test_gemm_lora_direct_rows_in_every_accumulator(m, n, k):
    # more output tiles than CTA pairs, so that both accumulators of a pair are used; short and long K loops
    r, A = 24, 9
    g = gen(m + k)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, n, k, r, A)
    adapter = adapters_of(g, m, A, "sorted")
    adapter[::7] = 4
    clean = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    R.assert_within(clean, *R.gemm_lora(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias))
    big = (torch.rand(m, generator=g, device="cuda") < 0.02) & (adapter >= 0)
    d[big] *= 2.0 ** 80
    l1[4, ::5, 3] = 2.0 ** 60
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    direct = big | (adapter == 4)
    assert torch.equal(bits(out[~direct]), bits(clean[~direct]))
    ref, err = low_rank_in_fp32(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias)
    assert_within_bf16(out[direct], ref[direct], err[direct])
    alpha.zero_()
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    assert_within_bf16(out, *low_rank_in_fp32(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias))


def test_gemm_lora_bad_adapter_comes_and_goes_in_a_replayed_graph():
    m, n, k, r, A = 300, 264, 320, 16, 5
    g = gen(77)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, n, k, r, A)
    adapter = adapters_of(g, m, A, "mixed")
    good, al = l1.clone(), alpha.clone()
    want = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    for bad in (2, None, 0, None):
        l1.copy_(good)
        if bad is not None:
            l1[bad, 11] = float("nan")
        for zero in (False, True):
            alpha.copy_(al * (not zero))
            graph.replay()
            torch.cuda.synchronize()
            got, own = out.clone(), adapter == (-2 if bad is None else bad)
            assert got[own][:, 11].isnan().all() and int(got.isnan().sum()) == int(own.sum())
            if zero:
                keep = ~got.isnan()
                ref, err = low_rank_in_fp32(a, b, a_sf, b_sf, alpha, d, good, adapter, bias)
                R.assert_within(got[keep], ref[keep], err[keep])
            else:
                assert torch.equal(bits(got[~own]), bits(want[~own]))


@pytest.mark.parametrize("m,k,r,A", [(40, 192, 16, 4), (700, 192, 64, 5), (1100, 128, 64, 60)])     # rows, tiles, mixed tiles
def test_lora_down_adapter_of_any_values_leaves_the_others(m, k, r, A):
    g = gen(m + r)
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = (torch.randn((A, r, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
    adapter = adapters_of(g, m, A, "mixed")
    clean = nv.nvfp4_lora_down_batched(x, w, adapter)
    w[1, 3, 5], w[2, r - 1, k - 1] = float("nan"), float("inf")
    out = nv.nvfp4_lora_down_batched(x, w, adapter)
    touched = torch.zeros_like(out, dtype=torch.bool)
    touched[adapter == 1, 3] = True
    touched[adapter == 2, r - 1] = True
    assert touched.any() and not out[touched].isfinite().any()
    assert torch.equal(bits(out)[~touched], bits(clean)[~touched])


# ---- projection with adapters: scale bytes of the rows beyond m and n ---------------------------------------------------------

@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("m,n,k,r,A", SIZES + [(1, 8, 64, 8, 1), (17, 392, 192, 8, 3), (700, 1000, 256, 16, 5)])
def test_gemm_lora_ignores_scales_of_padding_rows(m, n, k, r, A, byte):
    g = gen(m + n + r + 3)
    a, b, a_sf, b_sf, alpha, d, l1, bias = operands(g, m, n, k, r, A)
    adapter = adapters_of(g, m, A, "mixed")
    a_sf[padding(m, k)] = 0
    b_sf[padding(n, k)] = 0
    want = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)
    plain = nv.nvfp4_gemm(a, b, a_sf, b_sf, alpha, bias=bias)
    a_sf[padding(m, k)] = byte
    b_sf[padding(n, k)] = byte
    assert torch.equal(bits(nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias=bias)), bits(want))
    assert torch.equal(bits(nv.nvfp4_gemm(a, b, a_sf, b_sf, alpha, bias=bias)), bits(plain))


# ---- router: logits that begin off a 16-byte boundary -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,E", [(1, 128), (9, 256), (5, 64), (3, 512), (2, 1024), (4, 8)])
def test_route_from_any_address(t, E, dtype):
    x = (torch.randn((t, E), generator=gen(E), device="cuda") * 3).to(dtype)
    ids, w = nv.nvfp4_moe_route(x, 4)
    assert (ids.cpu().numpy() == R.route(x, 4, 1)[0]).all()
    for off in (1, 2, 3, 5):
        room = torch.full((t * E + 16,), float("inf"), dtype=dtype, device="cuda")
        room[off:off + t * E] = x.view(-1)
        moved = room[off:off + t * E].view(t, E)
        assert moved.data_ptr() % 16 != 0
        other = nv.nvfp4_moe_route(moved, 4)
        assert torch.equal(other[0], ids) and torch.equal(other[1], w)
