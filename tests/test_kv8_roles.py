"""Who waits for whom in the attention kernels over the 8-bit cache, on a model (kv8_roles.py) under
random schedules: nothing goes wrong, and each thing that the kernels do for it is needed."""
import pytest

import kv8_roles as roles


@pytest.mark.parametrize("kind", ["narrow", "rows"])
@pytest.mark.parametrize("empty", [False, True])
@pytest.mark.parametrize("abort", [False, True])
def test_every_schedule_ends_well(kind, empty, abort):
    assert roles.outcomes(kind, 400, empty=empty, abort=abort) == {"fine": 400}


# what is left out, and what then goes wrong in some schedules
NEEDED = [
    ("narrow", "empty parts", "stuck", dict(empty=True)),
    ("rows", "empty parts", "stuck", dict(empty=True, slots=(4,))),
    ("narrow", "two products", "a wait passed for an older phase", {}),
    ("rows", "first keys", "a wait passed for an older phase", dict(slots=(4,))),
    ("rows", "issuer's waits", "twice at a barrier", dict(abort=True)),
    ("rows", "parts' ends", "twice at a barrier", dict(abort=True)),
    ("narrow", "queries' part", "stuck", dict(abort=True)),
    ("narrow", "abort seen", "a copy into a place with a copy in flight", dict(abort=True)),
    ("rows", "abort seen", "a copy into a place with a copy in flight", dict(abort=True)),
]


@pytest.mark.parametrize("kind,what,wrong,kw", NEEDED, ids=[f"{n[0]}-{n[1]}" for n in NEEDED])
def test_what_goes_wrong_without(kind, what, wrong, kw):
    assert roles.outcomes(kind, 150, what, **kw).get(wrong, 0) > 0
