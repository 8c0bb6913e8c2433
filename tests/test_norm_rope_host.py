"""Norms and rotation, and attention over shared prefixes, on the host (no GPU needed): refusals,
plans, sizes."""
import math
import random
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_tcgen05_gb300 import build as b
    b.build()
    import exact_io_aware_tcgen05_gb300 as fa
    fa.load()
    return fa


ROPE = dict(positions=16, axes=None, num_axes=1, turns=16, rot=64, interleaved=0)
NORM = dict(T=5, Hq=4, Hkv=2, d=128, norm=1, q_weight=16, k_weight=16, weights_f32=0, eps=1e-6)


def _fwd(fa, **over):
    a = dict(dtype=0, q=16, q_stride=1024, k=16, k_stride=1024, q_out=16, q_out_stride=512, k_out=16, k_out_stride=256,
             **NORM, **ROPE)
    a.update(over)
    return fa.fa_norm_rope(*a.values(), None, check=False)


def _bwd(fa, **over):
    a = dict(dtype=0, q=16, q_stride=1024, k=16, k_stride=1024, dq_out=16, dq_out_stride=512, dk_out=16,
             dk_out_stride=256, dq=16, dq_stride=512, dk=16, dk_stride=256, **NORM, dq_weight=16, dk_weight=16, **ROPE,
             workspace=256, workspace_bytes=1 << 30)
    a.update(over)
    return fa.fa_norm_rope_bwd(*a.values(), None, check=False)


def _append(fa, **over):
    a = dict(dtype=0, q=16, q_stride=1024, k=16, k_stride=1024, v=16, v_stride=1024, q_out=16, q_out_stride=512, k8=16,
             k_scale=16, v8=16, v_scale=16, num_pages=8, page=64, Hq=4, Hkv=2, d=128, slots=16, T=5, norm=1, q_weight=16,
             k_weight=16, weights_f32=0, eps=1e-6, **ROPE)
    a.update(over)
    return fa.fa_kv8_append_norm_rope(*a.values(), None, check=False)


COMMON = [
    (dict(dtype=2), 2), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(d=96), 2), (dict(d=256), 2),
    (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1), (dict(turns=None), 1), (dict(positions=None), 1),
    (dict(num_axes=0), 1), (dict(num_axes=5, axes=16), 1), (dict(num_axes=2), 1), (dict(num_axes=2, axes=18), 1),
    (dict(positions=18), 1), (dict(turns=20), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(eps=math.inf), 1), (dict(norm=0), 1), (dict(norm=0, q_weight=None), 1), (dict(q_weight=24), 1),
    (dict(k_weight=8), 1), (dict(q=24), 1), (dict(k=24), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(q_stride=504), 1), (dict(k_stride=252), 1), (dict(k_stride=248), 1),
]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(q_out=None), 1), (dict(k_out=None), 1), (dict(q_out=24), 1), (dict(k_out_stride=260), 1),
])
def test_forward_refuses(lib, over, status):
    assert _fwd(lib, **over) == status and lib.fa_last_error()


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(dq_out=None), 1), (dict(dk_out=24), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dq_stride=500), 1),
    (dict(dq_weight=18), 1), (dict(norm=0, q_weight=None, k_weight=None), 1), (dict(workspace=None), 3),
    (dict(workspace=128), 3), (dict(workspace_bytes=1), 3),
])
def test_backward_refuses(lib, over, status):
    assert _bwd(lib, **over) == status and lib.fa_last_error()


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(v=None), 1), (dict(v=24), 1), (dict(v_stride=248), 1), (dict(q_out=None), 1), (dict(q_out_stride=504), 1),
    (dict(k8=None), 1), (dict(v8=24), 1), (dict(k_scale=18), 1), (dict(slots=None), 1), (dict(slots=18), 1),
    (dict(page=48), 2), (dict(num_pages=0), 1), (dict(num_pages=1 << 26), 2),
])
def test_append_refuses(lib, over, status):
    assert _append(lib, **over) == status and lib.fa_last_error()


def test_calls_without_tokens(lib):
    none = dict(T=0, q=None, k=None, positions=None)
    assert _fwd(lib, **none, q_out=None, k_out=None) == 0
    assert _append(lib, **none, v=None, q_out=None, slots=None) == 0
    assert _bwd(lib, **none, dq_out=None, dk_out=None, dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None,
                workspace_bytes=0) == 0


def test_workspace_of_the_weights_gradients(lib):
    assert lib.fa_norm_rope_bwd_workspace_size(0, 4, 2, 128) == 0
    assert lib.fa_norm_rope_bwd_workspace_size(5, 4, 2, 96) == 0
    for d in (64, 128):
        sizes = [lib.fa_norm_rope_bwd_workspace_size(T, 32, 8, d) for T in (1, 10, 1000, 100000, 2 ** 31 - 1)]
        assert all(0 < s <= 4 * 2 * 152 * d for s in sizes)
    # every side has a CTA, whatever the heads
    for Hq, Hkv in ((1, 1000), (1000, 1), (7, 3)):
        assert lib.fa_norm_rope_bwd_workspace_size(10 ** 6, Hq, Hkv, 64) >= 2 * 64 * 4


def _prefix(fa, **over):
    a = dict(dtype=0, q=16, q_stride=512, k8=16, k_scale=16, v8=16, v_scale=16, num_pages=8, page=64, prefix_table=16,
             prefix_width=4, prefix_lens=16, prefix_cu=16, groups=2, table=16, width=4, lens=16, o=16, lse=16, B=2, Hq=4,
             Hkv=2, N=3, d=128, cu_seqlens=None, total_tokens=0, scale=0.1, workspace=256, workspace_bytes=1 << 40)
    a.update(over)
    return fa.fa_fwd_kv8_prefix(*a.values(), None, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), 2), (dict(q=None), 1), (dict(q=24), 1), (dict(q_stride=508), 1), (dict(k8=None), 1),
    (dict(v8=24), 1), (dict(k_scale=18), 1), (dict(num_pages=0), 1), (dict(page=24), 2), (dict(prefix_table=None), 1),
    (dict(prefix_table=18), 1), (dict(prefix_lens=None), 1), (dict(prefix_lens=18), 1), (dict(prefix_cu=None), 1),
    (dict(prefix_cu=18), 1), (dict(groups=0), 1), (dict(groups=8193), 2), (dict(prefix_width=0), 1),
    (dict(prefix_width=1 << 26), 2), (dict(table=None), 1), (dict(width=0), 1), (dict(lens=None), 1), (dict(o=None), 1),
    (dict(lse=None), 1), (dict(o=24), 1), (dict(B=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(N=0), 1),
    (dict(d=96), 2), (dict(scale=0.0), 1), (dict(scale=math.nan), 1), (dict(cu_seqlens=18, total_tokens=6), 1),
    (dict(cu_seqlens=16, total_tokens=-1), 1), (dict(workspace=None), 3), (dict(workspace=128), 3),
    (dict(workspace_bytes=1000), 3),
])
def test_prefix_refuses(lib, over, status):
    assert _prefix(lib, **over) == status and lib.fa_last_error()


def test_prefix_without_tokens(lib):
    assert _prefix(lib, cu_seqlens=16, total_tokens=0, q=None, o=None, lse=None, workspace=None, workspace_bytes=0) == 0


def test_prefix_workspace(lib):
    assert lib.fa_fwd_kv8_prefix_workspace_size(0, 4, 2, 1, 128, 0) == 0
    for B, N, T in ((3, 1, 0), (3, 5, 0), (3, 70, 100)):
        rows = (T or B * N) * 32
        assert lib.fa_fwd_kv8_prefix_workspace_size(B, 32, 8, N, 128, T) >= 2 * rows * 129 * 4


# ------------------------------------------------------------------------------------ plans

def test_turns_are_the_nearest(lib):
    """round(2^64 f / (2 pi)) mod 2^64, by pi to 70 digits from Machin's formula."""
    def arctan(x):   # of 1 / x
        total, term, n = Fraction(0), Fraction(1, x), 0
        while abs(term) > Fraction(1, 10 ** 75):
            total += (-1) ** n * term / (2 * n + 1)
            term /= x * x
            n += 1
        return total
    pi = 4 * (4 * arctan(5) - arctan(239))
    rng = random.Random(1)
    f = [10000.0 ** (-i / 32) for i in range(24)] + [0.0, -0.5, 1e-30, 1e6, 7.0] + [rng.gauss(0, 3) for _ in range(35)]
    turns = lib.rope_plan(f, device="cpu").turns.tolist()
    for x, t in zip(f, turns):
        exact = Fraction(x) * 2 ** 64 / (2 * pi)
        assert abs((t - exact + 2 ** 63) % 2 ** 64 - 2 ** 63) <= Fraction(1, 2) + Fraction(1, 10 ** 40), x


def test_plans(lib):
    import torch
    p = lib.rope_plan([1.0] * 8, device="cpu")
    assert p.axes is None and p.num_axes == 1 and p.interleaved is False and p.turns.shape == (8,)
    p = lib.rope_plan(torch.ones(16, dtype=torch.float64), axes=torch.tensor([0, 2] * 8), interleaved=True, device="cpu")
    assert p.num_axes == 3 and p.axes.tolist() == [0, 2] * 8 and p.axes.dtype == torch.int32 and p.interleaved
    assert lib.rope_plan([1.0] * 8, axes=[0] * 8, device="cpu").axes is None
    with pytest.raises(AttributeError):
        p.other


@pytest.mark.parametrize("f,axes", [
    ([], None), ([1.0] * 7, None), ([1.0] * 72, None), ([math.nan] * 8, None), ([math.inf] + [1.0] * 7, None),
    ([1.0] * 8, [0] * 7), ([1.0] * 8, [4] * 8), ([1.0] * 8, [-1] * 8),
])
def test_plans_that_are_refused(lib, f, axes):
    with pytest.raises(ValueError):
        lib.rope_plan(f, axes=axes, device="cpu")


def test_tensors_on_the_cpu_are_refused(lib):
    import torch
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lib.norm_rope_forward(q, k)
    with pytest.raises(ValueError, match="CUDA"):
        lib.norm_rope_backward(q, k, q, k)
    cache = lib.kv8_cache(4, 2, 64, page=16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lib.kv8_append_norm_rope(cache, q, k, k, torch.zeros(3, dtype=torch.int32))
    one = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lib.attention_forward_kv8_prefix(q, cache, one[None], one, one, one[None], one, cu_seqlens=one, max_seqlen=3)
    with pytest.raises(TypeError):
        lib.norm_rope_forward(q, k.to(torch.float16))
    with pytest.raises(TypeError):
        lib.norm_rope_forward(q.float(), k.float())


# ------------------------------------------------------------- the reference of the GPU tests

@pytest.mark.parametrize("interleaved,norm,rot", [(False, True, 64), (True, True, 32), (False, True, 0), (True, False, 64)])
def test_the_references_gradients(interleaved, norm, rot):
    """Against autograd and against differences, in 64 bits."""
    import torch
    import norm_rope_ref as ref
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(3, 2, 64, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=torch.float64) if norm else None
    dy = torch.randn(3, 2, 64, generator=g, dtype=torch.float64)
    angle = ref.angles(torch.tensor([0, 7, 1000], dtype=torch.int32), ref.frequencies(rot)) if rot else None

    def loss(x, w):
        return (ref.forward(x, w, angle, interleaved, norm, 1e-6)[0] * dy).sum()

    dx, _, dw, _ = ref.backward(x, dy, w, angle, interleaved, norm, 1e-6)
    leaves = [x.clone().requires_grad_()] + ([w.clone().requires_grad_()] if norm else [])
    loss(leaves[0], leaves[1] if norm else None).backward()
    assert (leaves[0].grad - dx).abs().max() < 1e-12
    if norm:
        assert (leaves[1].grad - dw).abs().max() < 1e-12
    h = 1e-6
    for i in range(0, x.numel(), 37):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view(x.shape)
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx.reshape(-1)[i]) < 1e-7
    if norm:
        for i in range(0, 64, 11):
            e = torch.zeros_like(w)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_the_references_far_angles():
    import torch
    import norm_rope_ref as ref
    freq = ref.frequencies(32)
    pos = [0, 1, -5, 4097, 10 ** 6]
    a = ref.exact_angles(pos, freq)
    b = ref.angles(torch.tensor(pos, dtype=torch.int32), freq)
    assert (torch.cos(a) - torch.cos(b)).abs().max() < 1e-9 and (torch.sin(a) - torch.sin(b)).abs().max() < 1e-9
