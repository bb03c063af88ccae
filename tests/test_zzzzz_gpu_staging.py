"""GPU tests of gnf4_moe_experts and gnf4_gemv where a CTA stages several sets of
activation rows one after the other: state of one staging must not reach the next.
Bounds as in test_zzzz_gpu_serving.py."""
import math

import pytest
import torch

import grouped_nf4_w4a16_b200 as gnf4
from test_w4_stream_staging import ALTERNATING, alternating
from test_zzzz_gpu_serving import FMT, gen, packed

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
