"""The bounded waits of attention over shared prefixes, made to run out by the test hook (a limit of 50 us and a signal that
is withheld: that data has landed in the kernel of many rows, that a piece is posted in that of few).  The call
returns and reports it, and the next call is right: every block has let go of its shared and tensor memory and no
copy of its own is left in flight."""
import pytest
import torch

from test_gpu_shared import call, check, jf, make, new_err  # noqa: F401  (jf: a fixture)

pytestmark = pytest.mark.gpu

# few rows a group in teams of one, two and four warps, one and two row tiles, both kernels; long items and short ones
CASES = [([3, 2], 1, 128, [90, 40], [70, 33, 40, 90, 50]), ([6], 1, 64, [70], [40, 3, 9, 0, 1, 5]),
         ([16, 9], 1, 128, [9, 30], [b for b in range(25)]), ([2, 2], 20, 128, [60, 40], [200, 33, 140, 60]),
         ([2, 1, 2], 40, 64, [7, 0, 50], [9, 0, 500, 64, 128]), ([20], 2, 128, [60], [30 + 7 * b for b in range(20)])]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_waits_run_out_then_recover(jf, case):  # noqa: F811
    groups, N, D, pages, own = CASES[case]
    w = make(groups, N, 8, 2, D, pages, own, seed=500 + case)
    torch.cuda.synchronize()
    for _ in range(2):
        jf.jf_debug_set_wait_limit_ns(50_000, withhold_arrivals=True)
        try:
            err = new_err()
            call(jf, w, "padded", err)
            torch.cuda.synchronize()
        finally:
            jf.jf_debug_set_wait_limit_ns(0, withhold_arrivals=False)
        assert err.item() & jf.DEVERR_TIMEOUT, f"device error bits {err.item():#x}"
        err = new_err()
        out, lse = call(jf, w, "padded", err)
        assert err.item() == 0
        check(w, "padded", out, lse)
