"""GPU tests of the router and the few-token expert layer against 64-bit references (tests/serving_reference.py), with
element-wise bounds derived there, and of what a caller may do with them: dirty workspaces, other streams, graphs, repeated
and out-of-range expert ids, padded tokens, non-finite tokens, extreme magnitudes."""
import numpy as np
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


# ---- router ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("t,E,topk", [(1, 1, 1), (1, 2, 2), (3, 31, 5), (9, 32, 32), (8, 33, 7), (257, 100, 8), (5, 256, 16),
                                      (17, 513, 3), (2, 1024, 32)])
@pytest.mark.parametrize("weighting", [0, 1, 2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(t, E, topk, weighting, dtype):
    g = gen(t * 1000 + E)
    x = (torch.randn((t, E), generator=g, device="cuda") * 3).to(dtype)
    x[torch.rand((t, E), generator=g, device="cuda") < 0.2] = float("-inf")
    x[torch.rand((t, E), generator=g, device="cuda") < 0.05] = float("nan")
    x[torch.rand((t, E), generator=g, device="cuda") < 0.2] = 0.5            # ties
    x[0] = float("-inf")                                                     # nothing left
    ids, w = nv.nvfp4_moe_route(x, topk, weighting)
    rids, rw = R.route(x, topk, weighting)
    assert (ids.cpu().numpy() == rids).all()
    # expf and a sum of up to 1024 positive fp32 terms: at most (1024 / 32 + 5 + 8) roundings of 2^-24, the
    # exponent's argument is rounded to 2^-24 of up to 40
    assert np.abs(w.cpu().numpy() - rw).max() <= 2.0 ** -17
    assert (w.cpu().numpy()[rids < 0] == 0).all()


def test_route_signed_zeros_infinity_and_extremes():
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0], [float("inf"), 1.0, float("inf"), 2.0], [-big, big, -big, 0.0],
                      [float("nan"), float("-inf"), -big, float("nan")]], device="cuda")
    for weighting in (0, 1, 2):
        ids, w = nv.nvfp4_moe_route(x, 3, weighting)
        rids, rw = R.route(x, 3, weighting)
        assert (ids.cpu().numpy() == rids).all()
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -20, atol=1e-30)


def test_route_leaves_what_is_around_its_outputs():
    x = torch.randn((5, 40), generator=gen(3), device="cuda")
    ids = torch.full((7, 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((7, 3), 5.0, device="cuda")
    nv.nvfp4_moe_route(x, 3, ids_out=ids[1:6], weights_out=w[1:6])
    assert (ids[[0, 6]] == 77).all() and (w[[0, 6]] == 5.0).all()
    assert (ids[1:6].cpu().numpy() == R.route(x, 3, 1)[0]).all()


def test_route_of_no_tokens():
    ids, w = nv.nvfp4_moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


# ---- few-token expert layer -------------------------------------------------------------------------------

def expert_weights(E, n, k, seed, std=0.05):
    """gate, up, down as a user prepares them: (codes, scales, amax) of bf16 matrices."""
    g = gen(seed)
    out = {}
    for name, shape in (("gate", (E, n, k)), ("up", (E, n, k)), ("down", (E, k, n))):
        w = (torch.randn(shape, generator=g, device="cuda") * std * (0.5 + torch.rand((E, 1, 1), generator=g, device="cuda"))).bfloat16()
        amax, gsf = nv.nvfp4_global_scale_batched(w)
        q, sf = nv.nvfp4_quantize_masked_batched(w, gsf)
        out[name] = (q, sf, amax)
    return out


def call(x, ids, weights, w, **kw):
    return nv.nvfp4_moe_few_tokens(x, ids, weights, *(w[m][0] for m in ("gate", "up", "down")),
                                   *(w[m][1] for m in ("gate", "up", "down")), *(w[m][2] for m in ("gate", "up", "down")), **kw)


def case(t, E, topk, n, k, seed=1, ids=None):
    g = gen(seed)
    x = torch.randn((t, k), generator=g, device="cuda")
    x = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, x * 40, x).bfloat16()
    if ids is None:
        ids = torch.randint(0, E, (t, topk), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand((t, topk), generator=g, device="cuda") - 0.2
    return x, ids, weights, expert_weights(E, n, k, seed + 100)


def check(x, ids, weights, w, E, what=""):
    out = call(x, ids, weights, w)
    ref, err = R.moe(x, ids, weights, w, E)
    R.assert_within(out, ref, err, what)
    # three independent contributions (rounding of the output, slices of x, slices of h), each with a root mean
    # square of at most 2^-8 / sqrt(3) of the values': together 2^-8
    n = ref.norm()
    assert float((out.double() - ref).norm()) <= 2.0 ** -8 * float(n) or n == 0
    return out


@pytest.mark.parametrize("t,E,topk,n,k", [
    (1, 1, 1, 64, 64), (1, 4, 2, 128, 64), (1, 8, 8, 256, 256), (2, 3, 1, 192, 320), (3, 5, 3, 320, 192), (4, 1, 1, 64, 576),
    (5, 2, 1, 448, 64), (7, 16, 4, 704, 832), (16, 1, 1, 128, 128), (17, 1, 1, 192, 448), (33, 128, 4, 640, 320),
    (48, 2, 2, 1088, 192), (64, 2, 2, 64, 64), (64, 40, 8, 192, 256), (64, 3, 16, 128, 192), (9, 1024, 16, 64, 64),
    # 32 slots are grouped by one warp, more by the whole CTA; the most slots and experts
    (4, 9, 8, 128, 192), (32, 1, 1, 128, 128), (32, 2, 1, 192, 64), (11, 40, 3, 128, 192), (64, 1024, 16, 64, 128)])
def test_moe(t, E, topk, n, k):
    x, ids, weights, w = case(t, E, topk, n, k)
    check(x, ids, weights, w, E)


def test_moe_segment_borders():
    # experts with 1, 4, 5, 8, 9, 16, 17 and 4 slots: every segment width and a second segment
    counts = [1, 4, 5, 8, 9, 16, 17, 4]
    ids = torch.tensor([e for e, c in enumerate(counts) for _ in range(c)], dtype=torch.int32, device="cuda")
    ids = ids[torch.randperm(64, generator=gen(9), device="cuda")].view(64, 1).contiguous()
    x, ids, weights, w = case(64, 8, 1, 192, 320, ids=ids)
    check(x, ids, weights, w, 8)


def test_moe_skips_ids_out_of_range_and_pads_with_zeros():
    t, E, topk, n, k = 9, 4, 3, 128, 192
    x, ids, weights, w = case(t, E, topk, n, k)
    ids[0] = -1
    ids[1] = torch.tensor([4, 100, -7], device="cuda")
    ids[2, 1] = 2 ** 31 - 1
    ids[3, 0] = -2 ** 31
    x[0] = float("nan")                                   # a padded token's row may hold anything
    weights[1] = float("inf")                             # and a skipped slot's weight
    out = torch.full((t + 2, k), 7.0, dtype=torch.bfloat16, device="cuda")
    call(x, ids, weights, w, out=out[1:t + 1])
    assert (out[0] == 7).all() and (out[t + 1] == 7).all()
    assert (out[1:3] == 0).all()
    ok = torch.where((ids < 0) | (ids >= E), torch.full_like(ids, -1), ids)
    ref, err = R.moe(x, ok, weights, w, E)
    R.assert_within(out[3:t + 1], ref[2:], err[2:])


@pytest.mark.parametrize("t", [5, 20])
def test_moe_without_any_valid_slot(t):
    x, ids, weights, w = case(t, 4, 2, 128, 192)
    out = torch.full_like(x, 3.0)
    call(x, torch.full_like(ids, -1), weights, w, out=out)
    assert (out == 0).all()


def test_moe_same_expert_twice_counts_twice():
    x, ids, weights, w = case(6, 4, 4, 128, 192)
    ids[:, 1] = ids[:, 0]
    ids[2] = 3
    check(x, ids, weights, w, 4)


def test_moe_non_finite_token_leaves_the_others():
    t, E = 8, 3
    x, ids, weights, w = case(t, E, 2, 128, 320)
    clean = call(x, ids, weights, w)
    y = x.clone()
    y[2, 5] = float("nan")
    y[5, 300] = float("inf")
    out = call(y, ids, weights, w)
    bad = torch.tensor([i in (2, 5) for i in range(t)], device="cuda")
    assert out[bad].isnan().all()
    assert torch.equal(out[~bad].view(torch.int16), clean[~bad].view(torch.int16))


@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e-12, 1e12, 1e30])
def test_moe_extreme_magnitudes(scale):
    x, ids, weights, w = case(4, 3, 2, 128, 192)
    if scale > 1:                                          # keep h = silu(g) * u within fp32
        w = {m: (q, sf, amax * (1.0 / scale if m != "down" else 1.0)) for m, (q, sf, amax) in w.items()}
    x = (x.float() * scale).bfloat16()
    out = call(x, ids, weights, w)
    ref, err = R.moe(x, ids, weights, w, 3)
    # values of x below 2^-120 are held to 2^-117 (far below the smallest tested), products below fp32's range vanish
    R.assert_within(out, ref, err + 1e-37)


def test_moe_outlier_does_not_drown_its_row():
    # one value 2^17 times the others: the other 256-value chunks keep their precision, its own is held to the documented share
    x, ids, weights, w = case(3, 2, 2, 128, 768)
    x[1, 300] = 131072.0
    check(x, ids, weights, w, 2)


def test_moe_extreme_weight_scales():
    # block scales over ue4m3's whole range (448 to subnormal), zero blocks, all codes
    E, n, k = 2, 128, 192
    g = gen(77)
    w = {}
    for name, (r, c) in (("gate", (n, k)), ("up", (n, k)), ("down", (k, n))):
        q = torch.randint(0, 256, (E, r, c // 2), generator=g, device="cuda", dtype=torch.uint8)
        sf = torch.randint(0, 127, (E, nv.nvfp4_scale_bytes(r, c)), generator=g, device="cuda", dtype=torch.uint8)
        w[name] = (q, sf, torch.tensor([0.01, 3.0], device="cuda"))
    x, ids, weights, _ = case(5, E, 2, n, k)
    check(x, ids, weights, w, E)


def test_moe_any_workspace_contents_and_repeated_calls():
    x, ids, weights, w = case(11, 6, 3, 320, 448)
    need = nv.nvfp4_moe_few_tokens_workspace(11, 3, 6, 320, 448)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    first = call(x, ids, weights, w, workspace=ws)
    for _ in range(3):
        assert torch.equal(call(x, ids, weights, w, workspace=ws).view(torch.int16), first.view(torch.int16))
    assert torch.equal(call(x, ids, weights, w).view(torch.int16), first.view(torch.int16))


def test_moe_tokens_do_not_depend_on_their_batch():
    # a token alone and within a batch: segments and splits differ, fp32 sums may be ordered differently
    x, ids, weights, w = case(24, 4, 2, 320, 448)
    whole = call(x, ids, weights, w)
    ref, err = R.moe(x, ids, weights, w, 4)
    for i in (0, 11, 23):
        R.assert_within(call(x[i:i + 1], ids[i:i + 1], weights[i:i + 1], w), ref[i:i + 1], err[i:i + 1])
    R.assert_within(whole, ref, err)


def test_moe_two_streams_at_once():
    sets = [case(12, 5, 2, 704, 832, seed=s) for s in (5, 6)]
    want = [call(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for j, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[j].append(call(*s))
    torch.cuda.synchronize()
    for j in range(2):
        for o in got[j]:
            assert torch.equal(o.view(torch.int16), want[j].view(torch.int16))


def test_moe_captured_and_replayed_with_new_inputs():
    x, ids, weights, w = case(10, 6, 2, 192, 320)
    other = case(10, 6, 2, 192, 320, seed=40)
    call(x, ids, weights, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(x, ids, weights, w)
    x.copy_(other[0])
    ids.copy_(other[1])
    ids[3] = -1
    weights.copy_(other[2])
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    assert torch.equal(replayed.view(torch.int16), call(x, ids, weights, w).view(torch.int16))
    ref, err = R.moe(x, ids, weights, w, 6)
    R.assert_within(replayed, ref, err)


def test_moe_pdl_on_and_off_give_identical_bytes():
    x, ids, weights, w = case(20, 8, 2, 320, 448)
    before = nv.nvfp4_get_pdl()
    try:
        got = []
        for pdl in (True, False):
            nv.nvfp4_set_pdl(pdl)
            got.append(call(x, ids, weights, w))
    finally:
        nv.nvfp4_set_pdl(before)
    assert torch.equal(got[0].view(torch.int16), got[1].view(torch.int16))


def test_moe_refusals():
    x, ids, weights, w = case(4, 3, 2, 128, 192)
    with pytest.raises(ValueError, match="contiguous"):
        call(x.t().contiguous().t(), ids, weights, w)
    with pytest.raises(ValueError, match="ids"):
        call(x, ids.long(), weights, w)
    with pytest.raises(ValueError, match="weights"):
        call(x, ids, weights.double(), w)
    with pytest.raises(ValueError, match="x"):
        call(x.float(), ids, weights, w)
    with pytest.raises(ValueError, match="must be on"):
        call(x, ids.cpu(), weights, w)
    with pytest.raises(ValueError, match="w_down"):
        call(x, ids, weights, {**w, "down": w["gate"]})
    with pytest.raises(nv.NVFP4Error):
        call(x, ids, weights, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(torch.zeros((65, 192), dtype=torch.bfloat16, device="cuda"), ids, weights, w)
    assert call(x[:0], ids[:0], weights[:0], w).shape == (0, 192)


def test_decode_step_of_one_layer():
    """Router, experts and an adapted projection in a row, as a server runs them: route -> experts -> quantize -> projection
    with adapters, each checked on what the one before produced."""
    t, E, topk, n, k, nout, r, A = 13, 6, 2, 192, 320, 264, 16, 5
    g = gen(123)
    x, _, _, w = case(t, E, topk, n, k, seed=8)
    router = (torch.randn((E, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
    ids, weights = nv.nvfp4_moe_route((x @ router.t()).float(), topk)
    y = call(x, ids, weights, w)
    ref, err = R.moe(x, ids, weights, w, E)
    R.assert_within(y, ref, err, "experts")
    proj = (torch.randn((nout, k), generator=g, device="cuda") * 0.05).bfloat16()
    amax_b, _, _, b, b_sf = nv.nvfp4_global_scale_quantize(proj)
    _, _, alpha, a, a_sf = nv.nvfp4_global_scale_quantize(y, other_amax=amax_b)
    down = (torch.randn((A, r, k), generator=g, device="cuda") / k ** 0.5).bfloat16()
    up = (torch.randn((A, nout, r), generator=g, device="cuda") * 0.1).bfloat16()
    adapter = torch.randint(-1, A, (t,), generator=g, device="cuda", dtype=torch.int32)
    d = nv.nvfp4_lora_down_batched(y, down, adapter)
    R.assert_within(d, *R.lora_down(y, down, adapter), "down")
    out = nv.nvfp4_gemm_lora_batched(a, b, a_sf, b_sf, alpha, d, up, adapter)
    R.assert_within(out, *R.gemm_lora(a, b, a_sf, b_sf, alpha, d, up, adapter, None), "projection")


def test_moe_on_a_stream_of_its_own():
    # stream= differs from the current stream: the workspace that the call allocates must outlive the call
    x, ids, weights, w = case(24, 6, 2, 320, 448)
    want = call(x, ids, weights, w)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append(call(x, ids, weights, w, stream=st))
        torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")       # would land in a workspace freed too early
    st.synchronize()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_moe_weights_beyond_four_gigabytes():
    # the last of 600 experts of 2048 x 8192 lies beyond 2^32 bytes of each weight tensor
    E, n, k = 600, 2048, 8192
    w = {}
    for name, (r, c) in (("gate", (n, k)), ("up", (n, k)), ("down", (k, n))):
        q = torch.zeros((E, r, c // 2), dtype=torch.uint8, device="cuda")
        sf = torch.zeros((E, nv.nvfp4_scale_bytes(r, c)), dtype=torch.uint8, device="cuda")
        g = gen(len(name))
        for e in (0, E - 1):
            q[e] = torch.randint(0, 256, (r, c // 2), generator=g, device="cuda", dtype=torch.uint8)
            sf[e] = torch.randint(40, 56, (sf.shape[1],), generator=g, device="cuda", dtype=torch.uint8)
        w[name] = (q, sf, torch.full((E,), 4.0, device="cuda"))
        assert q.numel() > 2 ** 32
    g = gen(5)
    x = torch.randn((3, k), generator=g, device="cuda").bfloat16() * 0.1
    ids = torch.tensor([[E - 1], [0], [E - 1]], dtype=torch.int32, device="cuda")
    weights = torch.rand((3, 1), generator=g, device="cuda")
    out = call(x, ids, weights, w)
    ref, err = R.moe(x, ids, weights, w, E)
    R.assert_within(out, ref, err)


def test_moe_and_route_on_two_devices():
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two visible GPUs")
    x, ids, weights, w = case(9, 4, 2, 128, 192)
    want = call(x, ids, weights, w)
    moved = {m: tuple(t.to("cuda:1") for t in v) for m, v in w.items()}
    got = call(x.to("cuda:1"), ids.to("cuda:1"), weights.to("cuda:1"), moved)       # the current device stays cuda:0
    assert got.device.index == 1 and torch.equal(got.cpu().view(torch.int16), want.cpu().view(torch.int16))
    logits = torch.randn((7, 33), device="cuda:1")
    assert (nv.nvfp4_moe_route(logits, 4)[0].cpu().numpy() == R.route(logits, 4, 1)[0]).all()


@pytest.mark.parametrize("n,k,E,topk", [(64, 64, 3, 2), (192, 5120, 2, 1), (1408, 2048, 40, 8), (8192, 192, 4, 2), (256, 1088, 16, 16)])
def test_moe_one_token(n, k, E, topk):
    x, ids, weights, w = case(1, E, topk, n, k)
    check(x, ids, weights, w, E)
    ids[0, -1] = ids[0, 0]                                   # an expert twice
    out = check(x, ids, weights, w, E)
    want = call(torch.cat([x] * 3), ids.repeat(3, 1), weights.repeat(3, 1), w)          # the form with a slice kernel
    assert float((out.double() - want[1:2].double()).norm()) <= 2.0 ** -7 * float(out.double().norm())
    x[0, k // 2] = float("nan")
    assert call(x, ids, weights, w).isnan().all()
    x[0, k // 2] = 0.5
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(x, ids, weights, w)
        st.synchronize()
        with torch.cuda.graph(g, stream=st):
            a = call(x, ids, weights, w)
            b = call(a, ids, weights, w)                     # the next call reads the last one's result
    x.copy_(x.flip(1))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    first = call(x, ids, weights, w)
    assert torch.equal(a.view(torch.int16), first.view(torch.int16))
    assert torch.equal(b.view(torch.int16), call(first, ids, weights, w).view(torch.int16))


def test_moe_one_token_without_an_expert():
    x, ids, weights, w = case(1, 4, 2, 128, 192)
    ids.fill_(-1)
    assert (call(x, ids, weights, w) == 0).all()
    ids[0, 1] = 3
    check(x, ids, weights, w, 4)
