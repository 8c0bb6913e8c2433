"""The 8-bit cache's entry points on the host (no GPU needed): refusals, sizes, and the plain
forms that the GPU tests compare with."""
import numpy as np
import pytest

import kv8_ref as ref


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_tcgen05_gb300 import build as b
    b.build()
    import exact_io_aware_tcgen05_gb300 as fa
    fa.load()
    return fa


def _plan(fa, **over):
    a = dict(lens=16, grow=32, B=2, table=48, width=4, ring=64, num_pages=8, page=64, state=80,
             lens_out=96, cu_out=112, slots=128, T=5, state_out=144)
    a.update(over)
    return fa.fa_kv8_plan(*a.values(), None, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(lens=None), 1), (dict(grow=None), 1), (dict(table=None), 1), (dict(ring=None), 1),
    (dict(state=None), 1), (dict(lens_out=None), 1), (dict(cu_out=None), 1), (dict(slots=None), 1),
    (dict(state_out=None), 1), (dict(slots=130), 1), (dict(lens_out=16), 1), (dict(state_out=80), 1),
    (dict(T=-1), 1), (dict(B=0), 1), (dict(width=0), 1), (dict(num_pages=0), 1), (dict(page=24), 2),
    (dict(page=256), 2), (dict(page=8), 2), (dict(B=8193), 2), (dict(num_pages=1 << 26), 2),
    (dict(width=1 << 26), 2),
])
def test_plan_refuses(lib, over, status):
    assert _plan(lib, **over) == status and lib.fa_last_error()


def _append(fa, **over):
    a = dict(dtype=0, k=16, v=32, stride=256, k8=48, k_scale=64, v8=80, v_scale=96, num_pages=8,
             page=64, Hkv=2, d=128, slots=112, T=5)
    a.update(over)
    return fa.fa_kv8_append(*a.values(), None, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(k8=None), 1), (dict(v8=None), 1),
    (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(slots=None), 1), (dict(k=24), 1),
    (dict(v8=24), 1), (dict(k_scale=66), 1), (dict(slots=66), 1), (dict(stride=255), 1),
    (dict(stride=248), 1), (dict(stride=260), 1), (dict(Hkv=0), 1), (dict(d=96), 2), (dict(T=-1), 1),
    (dict(page=48), 2), (dict(num_pages=0), 1),
])
def test_append_refuses(lib, over, status):
    assert _append(lib, **over) == status and lib.fa_last_error()


def test_empty_calls_do_nothing(lib):
    assert _append(lib, T=0, k=None, v=None, slots=None) == 0
    assert _fwd(lib, cu_seqlens=16, total_tokens=0) == 0


def _fwd(fa, **over):
    a = dict(dtype=0, q=16, q_stride=512, k8=16, k_scale=16, v8=16, v_scale=16, num_pages=8, page=64,
             table=16, width=4, lens=16, o=16, lse=16, B=2, Hq=4, Hkv=2, N=3, d=128, causal=1,
             window=0, cu_seqlens=None, total_tokens=0, scale=0.1, workspace=256,
             workspace_bytes=1 << 30)
    a.update(over)
    return fa.fa_fwd_kv8(*a.values(), None, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=5), 2), (dict(q=None), 1), (dict(k8=None), 1), (dict(v8=None), 1),
    (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(o=None), 1), (dict(lse=None), 1), (dict(q=24), 1), (dict(o=24), 1), (dict(table=18), 1),
    (dict(q_stride=504), 1), (dict(q_stride=516), 1), (dict(d=96), 2), (dict(Hkv=3), 1), (dict(N=0), 1),
    (dict(B=0), 1), (dict(B=8193), 2), (dict(width=0), 1), (dict(page=20), 2), (dict(num_pages=0), 1),
    (dict(window=-1), 1), (dict(window=4, causal=0), 1), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
    (dict(cu_seqlens=16, total_tokens=-1), 1), (dict(workspace=None), 3), (dict(workspace_bytes=0), 3),
    (dict(workspace=16), 3),
])
def test_attention_refuses(lib, over, status):
    assert _fwd(lib, **over) == status and lib.fa_last_error()


@pytest.mark.parametrize("over", [
    # num_pages * Hkv, new tokens * group, table rows of nearly 2^31 tokens, key tiles of all requests
    dict(num_pages=1 << 23, page=16, Hkv=256, Hq=256, q_stride=256 * 128),
    dict(cu_seqlens=16, total_tokens=1 << 26, Hq=64, Hkv=2, q_stride=64 * 128, N=1),
    dict(width=(1 << 24) - 1, page=128),
    dict(B=8192, Hkv=64, Hq=64, q_stride=64 * 128, width=1 << 12, page=128),
])
def test_attention_refuses_what_32_bits_do_not_count(lib, over):
    assert _fwd(lib, **over) == 2 and lib.fa_last_error()
    smaller = {k: v for k, v in over.items() if k not in ("num_pages", "total_tokens", "width")}
    if "total_tokens" in over:
        smaller["total_tokens"] = 7
    # the same call is sound with a smaller count: only the workspace is missing
    assert _fwd(lib, workspace=None, **smaller) == 3


def test_cache_of_other_shapes_is_refused(lib):
    for kw in (dict(d=128, page=24), dict(d=96, page=64), dict(d=64, page=256), dict(d=64, page=8)):
        with pytest.raises(ValueError):
            lib.kv8_cache(4, 2, device="cpu", **kw)
    k8, k_scale, v8, v_scale = lib.kv8_cache(4, 2, 64, page=32, device="cpu")
    assert k8.shape == v8.shape == (4, 2, 32, 64) and k_scale.shape == v_scale.shape == (4, 2, 2)


def test_workspace_size(lib):
    f = lib.fa_fwd_kv8_workspace_size
    assert f(1, 4, 2, 1, 128, 0) > 0 and f(1, 4, 2, 1, 128, 0) % 256 == 0
    assert f(1, 4, 3, 1, 128, 0) == 0 and f(1, 4, 2, 1, 96, 0) == 0 and f(0, 4, 2, 1, 64, 0) == 0


# ------------------------------------------------------------------- the plain forms

def test_codes_round_to_the_nearest_value():
    import torch
    x = np.concatenate([np.random.default_rng(0).normal(0, 60, 4000), ref.VALUES[:127],
                        (ref.VALUES[1:127] + ref.VALUES[:126]) / 2, [448.0, -448.0, 2.0 ** -11, 0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_codes(x.astype(np.float64)), want)
    assert np.array_equal(ref.VALUES[want], torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_plan_of_a_few_requests():
    table = np.full((4, 3), -7, np.int32)
    table[0, :2] = (5, 3)
    table[1, :1] = 4
    ring = np.array([0, 1, 2, 6, 7, -1, -1, -1], np.int32)
    lens, cu, slots, state = ref.plan(np.array([20, 3, 0, 16]), np.array([2, -1, 33, 1]), table, ring,
                                      np.array([6, 4, 0]), 16, 40)
    # the free pages are ring[6], ring[7], ring[0], ring[1]; request 2 takes the first three
    assert lens.tolist() == [22, 0, 33, 17] and cu.tolist() == [0, 2, 2, 35, 36]
    assert slots[:2].tolist() == [3 * 16 + 4, 3 * 16 + 5] and (slots[36:] == -1).all()
    assert ring[2] == 4 and state.tolist() == [2, 1, 0]
    assert table[2].tolist() == [-1, -1, 0] and table[3, 1] == 1


@pytest.mark.parametrize("shape", ["type", "codes", "scales", "table", "lens", "q", "cu", "stride"])
def test_python_refuses(lib, shape):
    """The Python entry points check types and shapes before the devices (here: all on the CPU)."""
    import torch
    fa = lib
    cache = fa.kv8_cache(4, 2, 64, page=16, device="cpu")
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    kw = {}
    if shape == "type":
        q = q.float()
    elif shape == "codes":
        cache = fa.Kv8Cache((cache.k8.view(torch.uint8),) + cache[1:])
    elif shape == "scales":
        cache = fa.Kv8Cache((cache.k8, cache.k_scale[:, :, :0], cache.v8, cache.v_scale))
    elif shape == "table":
        table = table[:1]
    elif shape == "lens":
        lens = lens.long()
    elif shape == "q":
        q = q[0]
    elif shape == "cu":
        kw = dict(cu_seqlens=torch.zeros(3, dtype=torch.int32), max_seqlen=None)
        q = q[:, 0]
    elif shape == "stride":
        q = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)[..., ::2]
    with pytest.raises((TypeError, ValueError)):
        fa.attention_forward_kv8(q, cache, table, lens, **kw)
    # everything in order but the device
    with pytest.raises(ValueError, match="device"):
        fa.attention_forward_kv8(torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16),
                                 fa.kv8_cache(4, 2, 64, page=16, device="cpu"),
                                 torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32))
