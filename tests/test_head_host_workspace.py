"""A workspace of the largest call serves every smaller one: sizes grow with each argument."""

import random

from tests.test_head_host import lib  # noqa: F401 (a fixture)


def test_process_workspace_grows_with_requests_and_history(lib):  # noqa: F811
    size = lib.lp_head_process_workspace_size
    rng = random.Random(3)
    for _ in range(20000):
        B, n = int(2 ** rng.uniform(0, 16)), int(2 ** rng.uniform(0, 31))
        b, m = rng.randint(1, B), rng.randint(0, n)
        assert size(b, m) <= size(B, n), (b, m, B, n)
    assert size(256, 1_000_000) >= size(4, 100_000)
    assert size(1, 0) == 256 and size(300, 4095) == 256


def test_project_workspace_grows_with_rows_and_rank(lib):  # noqa: F811
    size = lib.lp_head_workspace_size
    rng = random.Random(4)
    for _ in range(20000):
        T, r = int(2 ** rng.uniform(0, 20)), rng.randint(0, 64)
        assert size(rng.randint(1, T), rng.randint(0, r)) <= size(T, r)


def test_one_workspace_for_all(lib):  # noqa: F811
    import ragged_log_probs_gb300 as lp
    most = lp.head_workspace_size(256, 16, 256, 1_000_000)
    for T, rank, requests, history in ((4, 16, 4, 100_000), (256, 16, 256, 0), (1, 1, 1, 1_000_000), (200, 16, 100, 999_999)):
        assert lp.head_workspace_size(T, rank, requests, history) <= most
