"""The several-token operators where their inputs, gates and waits leave the ordinary range, against plain
implementations in 64 bits (helpers and tolerances: tests/test_gpu_operators.py)."""
import pytest
import torch

from tests.test_gpu_operators import K, check_gdn, make_gdn, run_gdn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_a_wait_that_runs_out_is_reported_and_changes_no_state(K, dt):  # noqa: F811
    """Failure detection without a GPU fault: a run of tokens is never handed to the warps that hold the
    state, whose waits give up after 2 s.  The status says so, the state in place is what it was, and the
    next call is right."""
    T = 100
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=12)
    S1, out = S.clone(), torch.empty_like(v)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kva_test_gdn_forward_wait_timeout(q, k, v, gb, S1, S1, out, err)
    torch.cuda.synchronize()
    assert int(err.item()) == K.KVA_DEV_WAIT_TIMEOUT
    assert torch.equal(S1, S)
    err.zero_()
    out, S1 = run_gdn(K, q, k, v, gb, S, err=err)
    assert int(err.item()) == 0
    check_gdn(out, S1, q, k, v, gb, S, [T])
