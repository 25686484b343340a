"""dq_kv_plan refuses outputs that are its inputs (CPU; nothing is launched)."""
import pytest

from test_kv_ref import A, ARG, PLAN, so  # noqa: F401  (the fixture)


@pytest.mark.parametrize("change", [dict(kv=A), dict(new=2 * A), dict(ctx=2 * A), dict(left=A)])
def test_plan_refuses_outputs_that_are_inputs(so, change):  # noqa: F811
    assert so.lib.dq_kv_plan(*{**PLAN, **change}.values(), None) == ARG
