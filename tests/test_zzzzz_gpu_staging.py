"""GPU tests of gnf4_moe_experts and gnf4_gemv where a CTA stages several sets of
activation rows one after the other: state of one staging must not reach the next.
Bounds as in test_zzzz_gpu_serving.py."""
import math

import pytest
import torch

import grouped_nf4_w4a16_b200 as gnf4
from test_w4_stream_staging import ALTERNATING, LAYERS_IN_CHUNKS, PRODUCTS_IN_CHUNKS, alternating
from test_zzzz_gpu_serving import (FMT, close, experts_case, experts_ref, gemv_case, gemv_ref, gen, packed,
                                   run_experts)

pytestmark = pytest.mark.gpu


def layer(seed, T, H, F, E, fmt, scale="f32"):
    g = gen(seed)
    group = 32 if fmt == "mxfp4" else 64
    hidden = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w1, s1 = packed(g, (E, 2 * F), H, fmt, group, "e8m0" if fmt == "mxfp4" else scale)
    w2, s2 = packed(g, (E, H), F, fmt, group, "e8m0" if fmt == "mxfp4" else scale)
    return hidden, (w1, s1, w2, s2)


@pytest.mark.parametrize("case", ALTERNATING)
def test_no_token_scales_another_one(case):
    """A token 2^40 larger, or infinite, leaves every other token's result as it was, bit for bit."""
    T, H, F, E, k, fmt, _ = case
    ids, tokens = alternating(*case, sms=torch.cuda.get_device_properties(0).multi_processor_count)
    hidden, weights = layer(3, T, H, F, E, fmt)
    ids = torch.from_numpy(ids).cuda()
    share = torch.rand((T, k), generator=gen(4), device="cuda")
    clean = gnf4.gnf4_moe_experts(hidden, ids, share, *weights, fmt=FMT[fmt])
    assert torch.isfinite(clean.float()).all()
    for t in tokens[:24]:
        for factor in (2.0 ** 40, math.inf):
            large = hidden.clone()
            large[t] *= factor
            out = gnf4.gnf4_moe_experts(large, ids, share, *weights, fmt=FMT[fmt])
            others = torch.arange(T, device="cuda") != t
            assert torch.equal(out[others], clean[others]), (t, factor)


@pytest.mark.parametrize("layer,up,down,shared", LAYERS_IN_CHUNKS)
def test_layers_in_chunks_against_fp64(layer, up, down, shared):
    T, H, F, E, k, fmt, scale, inter = layer
    case = experts_case(T + H + F, T, H, F, E, k, fmt, scale)
    close(run_experts(case, fmt, inter), *experts_ref(*case, fmt, inter))


@pytest.mark.parametrize("product,chunks,shared", PRODUCTS_IN_CHUNKS)
def test_vector_products_in_chunks_against_fp64(product, chunks, shared):
    M, N, K, fmt, group, scale, zeros = product
    x, w, s, z, b = gemv_case(M + N + K, M, N, K, fmt, group, scale, zeros, True)
    close(gnf4.gnf4_gemv(x, w, s, fmt=FMT[fmt], zeros=z, bias=b), *gemv_ref(x, w, s, z, b, fmt, group))


def test_zero_points_up_to_255():
    x, w, s, z, _ = gemv_case(3, 9, 100, 512, "int4", 64, "f32", True)
    z = torch.randint(0, 256, z.shape, generator=gen(8), device="cuda", dtype=torch.uint8)
    close(gnf4.gnf4_gemv(x, w, s, fmt=FMT["int4"], zeros=z), *gemv_ref(x, w, s, z, None, "int4", 64))


@pytest.mark.parametrize("layer,up,down,shared", LAYERS_IN_CHUNKS)
def test_a_special_token_reaches_no_other_in_chunks(layer, up, down, shared):
    """Each token in turn with a NaN, an infinity or everything 2^40 larger: the others keep their bits."""
    T, H, F, E, k, fmt, scale, inter = layer
    case = list(experts_case(T + H + F, T, H, F, E, k, fmt, scale))
    hidden, clean = case[0], run_experts(case, fmt, inter)
    for t in range(T):
        for what in range(3):
            case[0] = hidden.clone()
            if what == 0:
                case[0][t, 7 * t % H] = math.nan
            elif what == 1:
                case[0][t, 11 * t % H] = math.inf
            else:
                case[0][t] *= 2.0 ** 40
            out = run_experts(case, fmt, inter)
            others = torch.arange(T, device="cuda") != t
            assert torch.equal(out[others], clean[others]), (t, what)
            assert what != 0 or torch.isnan(out[t].float()).all()


def test_gemv_small_scales():
    """Scales enter times 2^-14: exactly from 2^-112 on, below as multiples of 2^-135 (half a step
    is 2^-136). Sums are fp32 of rows with a largest magnitude below 2: each of the K / 64 additions
    is off by up to 2^-150 there, times the row's largest magnitude in the result."""
    x, w, _, _, _ = gemv_case(12, 4, 60, 512, "nf4", 64, "f32")
    x = (x.float() * 2.0 ** 90).to(torch.bfloat16)
    top = x.double().abs().amax(1, keepdim=True)
    step = torch.exp2(-torch.arange(100, 127, device="cuda").double())       # 2^-100 to 2^-126
    s = (torch.rand((60, 8), generator=gen(6), device="cuda").double() + 1) * step[torch.arange(60, device="cuda") % 27, None]
    s = s.float()
    ref, err = gemv_ref(x, w, s, None, None, "nf4", 64)
    total = x.double().abs() @ torch.ones((512, 60), dtype=torch.float64, device="cuda")
    below = (s < 2.0 ** -112).any(1)
    err = err + torch.where(below, 2.0 ** -136 * total, torch.zeros_like(total)) + 8 * 2.0 ** -150 * top
    assert below.any() and not below.all()
    close(gnf4.gnf4_gemv(x, w, s), ref, err)


@pytest.mark.parametrize("T,k", [(1, 4), (3, 5), (8, 4), (2, 16)])
def test_few_slots_with_an_expert_named_often(T, k):
    """Up to 32 slots, more of one expert than a batch has rows: the general tables."""
    case = list(experts_case(T + k, T, 192, 128, 6, k, "nf4", "f32", distinct=False))
    case[1][:] = 4
    case[1][0, 0] = -1
    close(run_experts(case, "nf4", False), *experts_ref(*case, "nf4", False))
    case[1][T - 1, k - 1] = 1
    close(run_experts(case, "nf4", False), *experts_ref(*case, "nf4", False))
