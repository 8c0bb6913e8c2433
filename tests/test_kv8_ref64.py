"""The 64-bit form on whole requests (kv8_ref64.py) against the one a row at a time (kv8_ref.py)."""
import numpy as np
import pytest

import kv8_ref as ref
import kv8_ref64 as r64


@pytest.mark.parametrize("lens,new,Hq,Hkv,d,page,dtype,causal,window", [
    ([40, 0, 3, 70], [2, 1, 5, 1], 4, 2, 64, 16, "bf16", True, 0),
    ([40, 0, 3, 70], [2, 1, 5, 1], 4, 4, 128, 32, "f16", True, 7),
    ([33, 90], [33, 2], 6, 2, 64, 64, "bf16", False, 0),
])
def test_both_forms_agree(lens, new, Hq, Hkv, d, page, dtype, causal, window):
    c = r64.make(1, lens, new, Hq, Hkv, d, page, dtype, spread=2.0, device="cpu")
    if lens[0] == 40:
        c["table"][0, 1] = -5          # a page that the cache does not have
    o, lse, bo, bl = r64.attend(c, causal=causal, window=window)
    k8, ks, v8, vs = c["cache"]
    import torch
    bits = [x.view(torch.uint8).numpy() for x in (k8, v8)]
    wo, wl, wbo, wbl = ref.attend(c["q"].double().numpy(), bits[0], ks.double().numpy(), bits[1],
                                  vs.double().numpy(), c["table"].numpy(), c["lens"].numpy(), c["cu"].numpy(),
                                  d ** -0.5, causal, window, r64.P_ROUND[dtype], r64.OUT_ROUND[dtype])
    assert np.allclose(o.numpy(), wo, rtol=1e-12, atol=1e-12)
    fine = np.isfinite(wl)
    assert np.array_equal(np.isfinite(lse.numpy()), fine)
    assert np.allclose(lse.numpy()[fine], wl[fine], rtol=1e-12, atol=1e-12)
    # the bounds here count the pieces of q too
    assert (bo.numpy() >= wbo * (1 - 1e-9)).all() and (bl.numpy() >= wbl * (1 - 1e-9)).all()
    r64.close(c, o, lse, (o, lse, bo, bl))
    with pytest.raises(AssertionError):
        bad = o.clone()
        bad[0, 0, 0] = float("nan")
        r64.close(c, bad, lse, (o, lse, bo, bl))
