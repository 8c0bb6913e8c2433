"""The 8-bit cache's entry points on the host, at the edges (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_tcgen05_gb300 import build as b
    b.build()
    import exact_io_aware_tcgen05_gb300 as fa
    fa.load()
    return fa


def _q(*shape):
    import torch
    return torch.zeros(*shape, dtype=torch.bfloat16)


# q of 4 heads, d 64, whose tokens lie in the same place, or overlap
OVERLAPPING = {
    "requests": lambda: _q(1, 1, 4, 64).expand(6, 1, 4, 64),
    "tokens": lambda: _q(2, 1, 4, 64).expand(2, 5, 4, 64),
    "both": lambda: _q(1, 1, 4, 64).expand(6, 5, 4, 64),
    "requests of several tokens": lambda: _q(1, 5, 4, 64).expand(6, 5, 4, 64),
    "one request": lambda: _q(1, 1, 4, 64).expand(1, 5, 4, 64),
    "packed": lambda: _q(1, 4, 64).expand(5, 4, 64),
    "shifted": lambda: _q(4096).as_strided((5, 4, 64), (64, 64, 1)),
    "shifted requests": lambda: _q(4096).as_strided((6, 1, 4, 64), (128, 256, 64, 1)),
    "no heads' distance": lambda: _q(5, 1, 64).expand(5, 4, 64),
}


@pytest.mark.parametrize("kind", list(OVERLAPPING))
def test_expanded_queries_are_refused(lib, kind):
    import torch
    q = OVERLAPPING[kind]()
    B = 1 if q.dim() == 3 else q.shape[0]
    kw = dict(cu_seqlens=torch.tensor([0, 5], dtype=torch.int32), max_seqlen=5) if q.dim() == 3 else {}
    cache = lib.kv8_cache(4, 2, 64, page=16, device="cpu")
    with pytest.raises(ValueError, match="evenly"):
        lib.attention_forward_kv8(q, cache, torch.zeros(B, 3, dtype=torch.int32),
                                  torch.ones(B, dtype=torch.int32), **kw)


@pytest.mark.parametrize("side", ["k", "v", "both"])
def test_expanded_keys_and_values_are_refused(lib, side, monkeypatch):
    import torch
    monkeypatch.setattr(lib, "_kv8_shape", lambda cache, device: tuple(cache.k8.shape))   # (tensors on the CPU)
    cache = lib.kv8_cache(4, 4, 64, page=16, device="cpu")
    x = dict(k=_q(5, 4, 64), v=_q(5, 4, 64))
    for name in x if side == "both" else side:
        x[name] = _q(1, 4, 64).expand(5, 4, 64)
    with pytest.raises(ValueError, match="evenly|same distance"):
        lib.kv8_append(cache, x["k"], x["v"], torch.zeros(5, dtype=torch.int32))


@pytest.mark.parametrize("make,stride", [
    (lambda: _q(5, 4, 64), 256),
    (lambda: _q(5, 9, 64)[:, 2:6], 576),                    # slices of a wider tensor
    (lambda: _q(10, 9, 64)[::2, 2:6], 1152),
    (lambda: _q(3, 5, 9, 64)[:, :, 2:6], 576),
    (lambda: _q(6, 5, 4, 64)[:, :1], 1280),                 # one token of each request
    (lambda: _q(6, 5, 4, 64)[2:3, ::2], 512),               # one request
    (lambda: _q(1, 4, 64), 256),                            # single tokens, wherever they lie
    (lambda: _q(1, 1, 4, 64), 256),
    (lambda: _q(8, 4, 64)[3:4].expand(1, 4, 64), 256),
    (lambda: _q(0, 4, 64), 256),                            # no token
    (lambda: _q(3, 0, 4, 64), 256),
    (lambda: _q(0).as_strided((0, 4, 64), (0, 0, 0)), 256),
])
def test_distance_of_tokens(lib, make, stride):
    assert lib._rows("q", make(), 4, 64) == stride


def test_distance_of_tokens_of_one_head(lib):
    assert lib._rows("q", _q(5, 3, 64)[:, 1:2], 1, 64) == 192
    with pytest.raises(ValueError):
        lib._rows("q", _q(5, 3, 64)[:, 1:2], 4, 64)
    with pytest.raises(ValueError):
        lib._rows("q", _q(3, 5, 4, 64)[:, ::2], 4, 64)       # requests and tokens at odds


def test_wait_for_a_parts_last_product():
    """The narrow kernel's wait at a part's end, for every state that its products can be in then.

    The scores of tile t are issued before the product of tile t - 1, so when a part's last tile t
    has had its scores, products up to t - 2 are known to be complete and t - 1 and t may be running.
    A wait for a phase passes where the barrier's last completed phase has its parity."""
    import os
    import re
    import exact_io_aware_tcgen05_gb300 as fa
    with open(os.path.join(os.path.dirname(fa.__file__), "csrc", "fa_kv8_fwd.cu")) as f:
        m = re.search(r"uint64_t [^;]*pv_done(?:\[(\d+)\])?;", f.read())
    bars = int(m.group(1) or 1)                             # product t completes phase t // bars of one of them
    for t in range(9):
        for complete in range(max(t - 1, 0), t + 2):       # products that are complete when the wait begins
            phases = len(range(t % bars, complete, bars))   # completed ones of the barrier waited for
            passes = (phases - 1) % 2 == t // bars % 2
            assert passes == (complete > t), (bars, t, complete)


def test_a_step_without_tokens(lib):
    """Empty tensors have no address: no token, none needed (nor a workspace)."""
    def fwd(**over):
        a = dict(dtype=0, q=None, q_stride=512, k8=16, k_scale=16, v8=16, v_scale=16, num_pages=8, page=64,
                 table=16, width=4, lens=16, o=None, lse=None, B=2, Hq=4, Hkv=2, N=3, d=128, causal=1, window=0,
                 cu_seqlens=16, total_tokens=0, scale=0.1, workspace=None, workspace_bytes=0)
        a.update(over)
        return lib.fa_fwd_kv8(*a.values(), None, check=False)
    assert fwd() == 0
    for name in ("k8", "k_scale", "v8", "v_scale", "table", "lens"):
        assert fwd(**{name: None}) == 1
    assert fwd(total_tokens=1) == 1 and fwd(page=24) == 2 and fwd(q_stride=516) == 1


def test_kernels_that_begin_early_read_nothing_as_constant():
    """These kernels are launched while the ones before them, which write what they read, may still
    run.  The read-only path (__ldg, and what the compiler makes of const __restrict__) is for data
    that nothing writes while a kernel lives."""
    import os
    import re
    import exact_io_aware_tcgen05_gb300 as fa
    csrc = os.path.join(os.path.dirname(fa.__file__), "csrc")
    for name in ("fa_kv8_work.cuh", "fa_kv8_cache.cu", "fa_kv8_fwd.cu", "fa_kv8_rows.cu"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//.*", "", f.read())
        assert not re.search(r"__ldg|__restrict__|\.nc\b|ld\.global\.nc|\bseq_bounds\s*\(", code), name


@pytest.mark.parametrize("over", [dict(tokens=2 ** 32 + 3), dict(tokens=2 ** 31), dict(page=2 ** 32 + 16),
                                  dict(tokens=-2 ** 32)])
def test_plan_refuses_numbers_beyond_32_bits(lib, over):
    import torch
    i32 = dict(dtype=torch.int32)
    args = dict(page=16, tokens=3) | over
    with pytest.raises(ValueError, match="32 bits"):
        lib.kv8_plan(torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32), torch.zeros(8, **i32),
                     torch.zeros(3, **i32), **args)


@pytest.mark.parametrize("over", [dict(window=2 ** 32 + 1), dict(window=2 ** 31), dict(window=-2 ** 32),
                                  dict(max_seqlen=2 ** 32 + 1), dict(max_seqlen=2 ** 31)])
def test_attention_refuses_numbers_beyond_32_bits(lib, over, monkeypatch):
    """(A window of 2^32 + 1 would be one of 1.)"""
    import torch
    kw = dict(cu_seqlens=torch.tensor([0, 2, 5], dtype=torch.int32), max_seqlen=3) | over
    args = _q(5, 4, 64), lib.kv8_cache(4, 2, 64, page=16, device="cpu")
    tables = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with monkeypatch.context() as m:
        m.setattr(lib, "_int32", lambda *a: None)                                # (tensors on the CPU)
        m.setattr(lib, "_kv8_shape", lambda cache, device: tuple(cache.k8.shape))
        with pytest.raises(ValueError, match="32 bits"):
            lib.attention_forward_kv8(*args, *tables, **kw)
