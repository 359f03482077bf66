"""The several-token operators where their inputs, gates and waits leave the ordinary range, against plain
implementations in 64 bits (helpers and tolerances: tests/test_gpu_operators.py)."""
import numpy as np
import pytest
import torch

from tests.parity import f64
from tests.test_gpu_operators import K, check_gdn, gdn_plain, make_gdn, run_gdn  # noqa: F401

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


def stored(o, dt):
    """A 64-bit array rounded once to dt (fp32 between the two could move a tie only)."""
    return f64(torch.from_numpy(o).to(dt))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(9, 128), (16, 64), (100, 128), (256, 128)])
@pytest.mark.parametrize("g", [0.0, -0.005])
def test_gdn_readout_of_a_carried_state_is_rounded_once(K, dt, T, d, g):  # noqa: F811
    """A state that nothing is written to (beta 0): o = e^gam S0 q.  The path to the output is off by at
    most e = (4 + runs) 2^-20 A, A = sum |S0| |q|: two fp16 terms of S0 (2^-21) and, where they count, of q
    (2^-22), a sum of 2 x 128 products in fp32 (2^-20 covers it), and a factor e^gam of a few 2^-23, which a
    decayed state meets once a run.  Rounded once, an output is then at most 2 e further from the exact value
    than the exact value's own rounding is: half a step and e where it falls on the other side."""
    q, k, v, gb, S = make_gdn(2, T, 2, 6, d, dt, seed=13)
    gb[:, 0], gb[:, 1] = g, 0.0
    out, S1 = run_gdn(K, q, k, v, gb, S)
    o, Sw, bo, _, _ = gdn_plain(f64(q), f64(k), f64(v), f64(gb), f64(S), [T, T], 1.0, run=T)
    runs = (T + 15) // 16
    over = np.abs(f64(out) - o) - np.abs(stored(o, dt) - o)
    assert (over <= 2 * (4 + runs) * 2.0 ** -20 * bo).all(), f"{(over / bo).max():.2e} of sum |S0||q|"
    assert (np.abs(f64(S1) - Sw) <= runs * 2.0 ** -21 * np.abs(Sw)).all()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("g", [0.0, 0.01, 2.0])
def test_gdn_readouts_of_a_long_run_have_the_error_of_their_storage(K, dt, g):  # noqa: F811
    """Long memories (g from 0 to -g): the readouts' 2-norm error is that of rounding the exact ones, within
    5 %: what the path adds in quadrature may be 0.32 of it, 6.6e-5 of the result in fp16, which is the 2^-14
    that two fp32 paths stay far below."""
    T = 400
    q, k, v, gb, S = make_gdn(1, T, 2, 6, 128, dt, seed=14, g_scale=g)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    o, Sw, _, _, _ = gdn_plain(f64(q), f64(k), f64(v), f64(gb), f64(S), [T], 1.0)
    assert np.linalg.norm(f64(out) - o) <= 1.05 * np.linalg.norm(stored(o, dt) - o)
    assert np.linalg.norm(f64(S1) - Sw) <= 2.0 ** -18 * np.linalg.norm(Sw)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [-12, 14])
def test_gdn_queries_of_any_size(K, dt, power):  # noqa: F811
    """Queries of another size at every token (to 2^-12 or 2^14 of norm 1): each readout is one rounding (in
    fp16 below 2^-14 of steps of 2^-24) and what the path adds, at most 2^-14 of its row's size: the 2 x 4 x
    2^-20 sum |S| |q| of above, with sum |S| |q| at most 11.4 |S row| |q|, whose size over the rows is the
    readouts' own."""
    T, scale = 40, 2.0 ** -14 if power > 0 else 2.0 ** 8
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=15, g_scale=0.1)
    e = 5 * torch.arange(T, device="cuda") % (abs(power) + 1)
    q = (q * torch.exp2(e if power > 0 else -e).view(1, T, 1, 1)).to(dt)
    out, S1 = run_gdn(K, q, k, v, gb, S, scale=scale)
    o, _, _, _, _ = gdn_plain(f64(q), f64(k), f64(v), f64(gb), f64(S), [T], scale)
    err, row = np.abs(f64(out) - o), np.sqrt((o * o).mean(-1, keepdims=True))
    half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    assert (err <= half * np.abs(o) + 2.0 ** -14 * row + 2.0 ** -25).all(), f"{(err / row).max():.2e}"
