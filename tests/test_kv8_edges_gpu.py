"""The 8-bit paged cache on the GPU where a call can go wrong: rows that see nothing between long
requests, and others that come up in a server's batches."""
import pytest

import kv8_ref64 as r64

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- items without keys

# Long requests with requests that see nothing between them, one and several in a row, so many
# that every CTA has items of both kinds: (tokens, new tokens) of one stretch, repeated.
SEATS = {
    "one": [(4096, 1), (0, 1), (3000, 1)],
    "six": [(2048, 1)] + [(0, 1)] * 6 + [(129, 1)],
    "ends": [(0, 1)] * 5 + [(5000, 1)] + [(0, 1)] * 2,
    "short": [(1, 1), (0, 1), (128, 1), (0, 1), (0, 1)],
}


@pytest.mark.parametrize("Hkv", [1, 8])
@pytest.mark.parametrize("group", [1, 8, 16, 24])
@pytest.mark.parametrize("kind", list(SEATS))
def test_idle_seats_between_long_requests(fa, kind, group, Hkv):
    """Single tokens (up to 8 and up to 16 rows, and items of 128)."""
    times = 40 if Hkv == 1 else 10
    stretch = SEATS[kind] * times
    lens, new = [x[0] for x in stretch], [x[1] for x in stretch]
    c = r64.make(3, lens, new, group * Hkv, Hkv, 64 if group == 8 else 128, 64, "f16" if group == 1 else "bf16")
    r64.close(c, *r64.run(fa, c), r64.attend(c))


@pytest.mark.parametrize("Hkv", [1, 8])
@pytest.mark.parametrize("group,new", [(2, 4), (4, 4), (8, 20), (1, 300)])
def test_refused_prompts_between_long_requests(fa, group, new, Hkv):
    """Requests with more new tokens than keys: their first blocks of rows see nothing."""
    stretch = [(2500, new), (0, new), (3, new), (new // 2, new), (700, new), (0, new), (0, new), (0, new),
               (0, new), (0, new), (1500, 1)] * (8 if Hkv == 1 else 3)
    c = r64.make(4, [x[0] for x in stretch], [x[1] for x in stretch], group * Hkv, Hkv, 128, 32, "bf16")
    r64.close(c, *r64.run(fa, c), r64.attend(c))
    r64.close(c, *r64.run(fa, c, window=100), r64.attend(c, window=100))


def test_nothing_but_idle_seats(fa):
    for n, group in ((1, 8), (2, 8), (40, 8)):
        c = r64.make(5, [0] * 50, [n] * 50, group * 2, 2, 128, 64, "bf16")
        o, lse = r64.run(fa, c)
        assert (o == 0).all() and (lse == -float("inf")).all()


def test_a_refused_prompt_in_a_step(fa):
    """A prompt that kv8_plan refuses keeps its place in cu_seqlens; the others' rows are right."""
    import torch
    H, Hq, d, page, pages = 2, 8, 128, 64, 160
    cache = fa.kv8_cache(pages, H, d, page=page)
    grow = [3000, 500, 2500, 1, 400]
    T = sum(grow)
    table = torch.zeros(5, 60, dtype=torch.int32, device="cuda")
    ring = torch.arange(pages, dtype=torch.int32, device="cuda")
    state = torch.tensor([0, 100, 0], dtype=torch.int32, device="cuda")   # 100 free pages: 47 + 8 + 40 + 1
    lens = torch.zeros(5, dtype=torch.int32, device="cuda")
    x = torch.randn(T, Hq + 2 * H, d, device="cuda").bfloat16()
    ln, cu, slots, st = fa.kv8_plan(lens, torch.tensor(grow, dtype=torch.int32, device="cuda"), table, ring, state,
                                    page=page, tokens=T)
    assert ln.tolist() == [3000, 500, 2500, 1, 0] and st.tolist()[2] == 1
    fa.kv8_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], slots)
    c = dict(q=x[:, :Hq].contiguous(), cache=tuple(cache), table=table, lens=ln, cu=cu, new=grow, dtype="bf16")
    r64.close(c, *r64.run(fa, c), r64.attend(c))


# ------------------------------------------------------------------------- windows

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 50, 2 ** 30, 140, 1])
@pytest.mark.parametrize("group,new", [(1, 9), (2, 8), (4, 200)])
def test_any_window_with_more_tokens_than_keys(fa, group, new, window):
    """Positions below 0 and windows as long as an int, in items of up to 8, 16 and 128 rows."""
    c = r64.make(6, [5, 300, 0, new // 2], [new, 1, new, new], group * 2, 2, 128, 16, "bf16")
    r64.close(c, *r64.run(fa, c, window=window), r64.attend(c, window=window))


# ------------------------------------------------------- queries that are not finite

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,group,new", [(128, 1, 6), (64, 2, 7), (128, 4, 6), (64, 1, 150)])
def test_queries_that_are_not_finite_and_rows_that_see_nothing(fa, d, group, new, dtype):
    """An infinity or NaN in a query makes its row NaN where the row sees a key, and no other row; a
    row that sees none has O = 0 and LSE = -inf, whatever its query holds."""
    import torch
    # positions from -3 on; pages that the cache does not have in the second and third
    c = r64.make(7, [new - 3, 200, 64 + new], [new, new, new], group * 2, 2, d, 16, dtype)
    c["table"][1, :] = -1
    c["table"][2, 4:] = 2 ** 30
    clean = r64.run(fa, c)
    want = r64.attend(c)
    r64.close(c, *clean, want)
    bad = torch.zeros(c["q"].shape[:2], dtype=torch.bool, device="cuda")
    for b in range(3):
        for i, (h, x) in zip((0, 2, 3, new - 1), ((0, "nan"), (1, "inf"), (group * 2 - 1, "-inf"), (0, "inf"))):
            c["q"][b * new + i, h, 5 * i % d] = float(x)
            bad[b * new + i, h] = True
    o, lse = r64.run(fa, c)
    sees = (want[1] > -float("inf")).T                     # [T, Hq]
    assert bool((sees & bad).any()) and bool((~sees & bad).any())
    assert torch.isnan(o[sees & bad]).all() and torch.isnan(lse.T[sees & bad]).all()
    assert (o[~sees] == 0).all() and (lse.T[~sees] == -float("inf")).all()
    fine = ~(sees & bad)
    assert torch.equal(o[fine], clean[0][fine]) and torch.equal(lse.T[fine], clean[1].T[fine])


def test_a_step_without_tokens(fa):
    """Plan, append and attend of a packed batch that holds no token."""
    import torch
    cache = fa.kv8_cache(8, 2, 128, page=16)
    was = [t.view(torch.uint8).clone() for t in cache]
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table = torch.tensor([20, 0, 7], **i32), torch.tensor([[1, 2], [0, 0], [3, 0]], **i32)
    ln, cu, slots, st = fa.kv8_plan(lens, torch.zeros(3, **i32), table, torch.arange(8, **i32),
                                    torch.tensor([4, 4, 0], **i32), page=16, tokens=0)
    assert ln.tolist() == [20, 0, 7] and cu.tolist() == [0] * 4 and slots.numel() == 0 and st.tolist() == [4, 4, 0]
    x = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    fa.kv8_append(cache, x[:, 4:6], x[:, 6:], slots)
    for n in (1, 2 ** 30):
        o, lse = fa.attention_forward_kv8(x[:, :4], cache, table, ln, cu_seqlens=cu, max_seqlen=n)
        assert o.shape == (0, 4, 128) and lse.shape == (4, 0)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(was, cache))
    fa.fa_device_status()
