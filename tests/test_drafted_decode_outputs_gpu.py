"""What a step of the drafted example hands on: the residual stream and the output projection, against 64 bits."""
import numpy as np
import pytest

import step_ref as ref
from test_drafted_decode_gpu import weights

pytestmark = pytest.mark.gpu


def test_what_every_step_hands_on(ctx):
    import drafted_decode as dd

    layer, records = dd.run(ctx)
    ctx.check_status()
    w = weights(layer.w_out, layer.s_out)
    for rec in records:
        h = ref.f64(rec["x"]) + ref.f64(rec["r"])
        assert (np.abs(ref.f64(rec["h"]) - h) <= (ref.HALF_ULP["bf16"] * 1.01 + 2.0**-23) * np.abs(h)).all()
        heads = ref.f64(rec["heads"])
        heads = heads.reshape(len(heads), -1)
        y, mag = heads @ w, np.abs(heads) @ np.abs(w)
        # K + 64 roundings of the sums, bf16 rows off by 2^-39 of their largest, one rounding to bf16
        bound = ((heads.shape[1] + 64) * 2.0**-23 * mag + ref.HALF_ULP["bf16"] * 1.01 * np.abs(y)
                 + 2.0**-39 * np.abs(heads).max(1, keepdims=True) * np.abs(w).sum(0))
        assert y.any() and (np.abs(ref.f64(rec["out"]) - y) <= bound).all()


def test_steps_ask_for_the_tokens_they_have(ctx):
    """Masks of one word for trees of 7 tokens, and the same answer as with the layer's limit."""
    import torch

    import drafted_decode as dd

    layer, records = dd.run(ctx, steps=1)
    rec = records[-1]
    assert rec["mask"].shape[1] == 1
    for t, was in ((layer.k, "pool_k"), (layer.v, "pool_v"), (layer.pages, "pages"), (layer.lens, "lens")):
        t.copy_(rec[was])
    _, _, wide = layer.step(rec["x"], rec["r"], rec["m"], parents=rec["parents"])
    assert wide["mask"].shape[1] == -(-layer.most // 32) and torch.equal(wide["mask"][:, :1], rec["mask"])
    want, _, _, x = ref.tree_attention(ref.f64(rec["q"]), ref.f64(rec["pool_k"]), ref.f64(rec["pool_v"]),
                                       rec["pages"].cpu().numpy(), rec["lens"].tolist(), layer.P, layer.d**-0.5,
                                       rec["m"]["cu"].tolist(), layer.most, rec["mask"].cpu().numpy())
    ob, _ = ref.tree_attention_bounds((want, np.zeros(want.shape[:2]), None, x), "bf16", layer.d)
    for heads in (rec["heads"], wide["heads"]):
        assert (np.abs(ref.f64(heads) - want) <= ob).all()
