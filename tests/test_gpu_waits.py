"""The bounded waits of the pipelined kernels run out: every form of the polling loop gives up
after its limit, and a wait leaves when another one has raised the CTA's flag."""
import ctypes
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cycles", [1, 1000, 2_000_000, 50_000_000])
def test_all_waits_give_up(cycles):
    """The status is set only when all three have.  The third has a limit of its own of two to
    four seconds: it must leave on the flag, long before that."""
    import eagle_tree_speculative_gb300 as E
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert E.lib().eagle_wait_selftest(st.data_ptr(), cycles, stream) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert int(st.item()) == E.EAGLE_DEV_TIMEOUT
