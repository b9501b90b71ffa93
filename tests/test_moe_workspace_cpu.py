"""The workspace of the choice and of the experts' layer: one that serves a batch serves
every smaller one."""
import pytest

from test_moe_cpu import lib, router, weights  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("experts,hidden", [(1, 32), (8, 512), (17, 4096), (64, 2080), (300, 8192), (1024, 4096)])
def test_workspaces_grow_with_tokens(lib, experts, hidden):  # noqa: F811
    f = lib.qbn_moe_workspace
    r, w = router(n=experts, top=1, hidden=hidden), weights(n=experts, hidden=hidden)
    for a, b in ((r, None), (None, w), (r, w)):
        got = [f(a, b, t, 1) for t in list(range(0, 600)) + [4095, 4096, 4097, 8193, 1 << 20]]
        assert got[0] == 0 and all(x <= y for x, y in zip(got, got[1:]))
