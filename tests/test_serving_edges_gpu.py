"""GPU tests of what the serving-step operators must not depend on or disturb: scale bytes of rows beyond a matrix, memory that
another stream still uses."""
import pytest
import torch

import nvfp4_block_scaled_16_b200 as nv
from tests import serving_reference as R
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
