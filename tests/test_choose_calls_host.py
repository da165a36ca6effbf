"""expert_choose takes whole numbers where it counts, and refuses what is none (CPU only)."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests.test_model_operators_host import calls, lib  # noqa: F401  (fixtures)


def test_numbers_that_are_not_whole(calls):  # noqa: F811
    lib, S, torch = calls  # noqa: F811
    x = S.Tensor((20, 8))
    for call in (lambda n: sg.expert_choose(x, n), lambda n: sg.expert_choose(x, 2, groups=n), lambda n: sg.expert_choose(x, 2, groups=4, kept_groups=n),
                 lambda n: sg.expert_choose(x, 2, groups=4, kept_groups=2, group_top=n)):
        for n in (2.0, 2.9, "2", None):
            with pytest.raises(TypeError):
                call(n)


def test_whole_numbers_of_other_types(calls):  # noqa: F811
    import numpy as np
    lib, S, torch = calls  # noqa: F811
    x, seen = S.Tensor((20, 8)), []
    lib.does["expert_choose"] = lambda *a: seen.append(a[:4] + a[8:11]) or 0
    for n in (2, np.int32(2), np.int64(2), torch.tensor(2)):
        sg.expert_choose(x, n, groups=n, kept_groups=n, group_top=n)
    assert seen == [(1, 20, 8, 2, 2, 2, 2)] * 4
