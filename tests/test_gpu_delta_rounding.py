"""o of the gated delta rule where it is read from the state alone, on the GPU: rounded to BF16 once."""

import pytest
import torch

from test_gpu_delta import D, SCALE, library, make, reference, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefill", [False, True])
def test_the_states_part_of_o_is_rounded_once(prefill):
    """With step sizes of zero o_t = s S q_t. S is taken in two BF16 parts: what they leave is at most half a step of a half step
    of a value, 2^-16 of it, and 256 products of FP32 sums add up to 256 2^-24 of the terms' absolute sum; then o's own half step."""
    from linear_attention_gated_gb300 import kda_gated_delta_prefill
    x = make((64, 1, 150), 2, 4, seed=60, gate=False)
    x["beta"].zero_()
    ref = reference(x, grads=False)["o"][0]
    if prefill:
        d = {n: t.cuda() for n, t in x.items()}
        got = kda_gated_delta_prefill(d["q"], d["k"], d["v"], None, d["beta"], d["h0"].clone(), d["cu"], cu_seqlens_cpu=x["cu"])
    else:
        got = run(x, grads=False)[0]["o"]
    got = got[0].double().cpu()
    q = x["q"][0].double().repeat_interleave(2, 1).abs()
    for n, (a, b) in enumerate(((0, 64), (64, 65), (65, 215))):
        terms = SCALE * (x["h0"][n].double().abs() @ q[a:b, :, :, None])[..., 0]
        off = (2.0 ** -16 + 256 * 2.0 ** -24) * terms
        bad = (got[a:b] - ref[a:b]).abs() > off + 2.0 ** -8 * (ref[a:b].abs() + off)
        assert not bad.any(), (n, int(bad.sum()))
