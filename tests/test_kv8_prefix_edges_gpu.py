"""Attention over shared prefixes in the 8-bit cache at its edges, on the GPU."""
import pytest

import kv8_ref64 as ref
import test_kv8_prefix_gpu as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("bf16", 128, 8, 2), ("f16", 64, 8, 1)])
def test_many_small_groups(fa, dtype, d, Hq, Hkv):
    """Groups of one to three requests, most of a single new token, some without prefix or own tokens."""
    groups = [((37 * g) % 700 if g % 7 else 0, [(1 + (11 * g + i) % 150, 1 + (g + i) % 19 // 18) for i in range(1 + g % 3)])
              for g in range(40)]
    groups[5] = (groups[5][0], [(0, 0), (3, 1)])
    c = base.make(1, groups, Hq, Hkv, d, 16, dtype)
    ref.close(c, *base.run(fa, c), base.attend(c))


@pytest.mark.parametrize("groups,Hq,Hkv,d,page,dtype", [
    ([(900, [(60, 1), (300, 1)]), (2000, [(5, 1)])], 8, 2, 128, 64, "bf16"),       # few rows
    ([(5000, [(100, 1)] * 20), (70, [(9, 1)] * 3)], 16, 4, 64, 16, "f16"),         # rows in blocks of 128, own keys' few
    ([(3000, [(200, 130), (150, 150)]), (0, [(40, 2)])], 8, 8, 128, 32, "bf16"),   # many rows
])
def test_the_same_bits_whatever_the_workspace_held(fa, groups, Hq, Hkv, d, page, dtype):
    import torch
    c = base.make(2, groups, Hq, Hkv, d, page, dtype)
    size = fa.fa_fwd_kv8_prefix_workspace_size(len(c["new"]), Hq, Hkv, max(c["new"]), d, len(c["q"]))
    first = None
    for i, byte in enumerate((0, 255, 127, 63, 1, 200)):
        ws = torch.full((size + 256,), byte, dtype=torch.uint8, device="cuda")
        if i % 2:
            torch.randn(2048, 2048, device="cuda") @ torch.randn(2048, 2048, device="cuda")
        o, lse = base.run(fa, c, workspace=ws[:size], out=torch.full_like(c["q"], torch.nan))
        assert (ws[size:] == byte).all()
        if first is None:
            first = o, lse
            ref.close(c, o, lse, base.attend(c))
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_launch_events_stay_armed(fa):
    """The call takes none: the next one that does finds them."""
    import torch
    c = base.make(3, [(100, [(20, 1)])], 4, 2, 64, 16, "bf16")
    events = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in events:
        e.record()
    torch.cuda.synchronize()
    own = lambda: fa.attention_forward_kv8(c["q"], fa.Kv8Cache(c["cache"]), c["table"], c["lens"], cu_seqlens=c["cu"],
                                           max_seqlen=1)
    fa.fa_set_launch_events(events[:1])     # too few for fa_fwd_kv8's two kernels
    base.run(fa, c)
    with pytest.raises(fa.FAError):
        own()
    fa.fa_set_launch_events(events)
    base.run(fa, c)
    own()
    torch.cuda.synchronize()
    assert events[0].elapsed_time(events[2]) > 0
    own()
