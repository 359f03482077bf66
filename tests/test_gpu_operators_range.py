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


@pytest.mark.parametrize("dt", [torch.bfloat16])
@pytest.mark.parametrize("T", [16, 17, 90])
@pytest.mark.parametrize("size,value,g", [(0.3, 0, -0.7), (0.3, 0, -1.0), (1.0, 0, -3.0), (1e4, 1, -0.7), (1e4, 1, -2.0),
                                          (1e4, 0, -1.0), (2.0 ** 60, 1, -1.0), (2.0 ** 60, 0, -0.7), (2.0 ** 60, 1, -3.0)])
def test_gdn_states_that_decay_below_what_the_first_tokens_met(K, dt, T, size, value, g):  # noqa: F811
    """Strong decay of a state that is far above the values (0: padding that writes nothing): finite, and
    within the bounds of what the run began with."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=16, sigma=size)
    v = v * value
    gb[:, 0] = g
    out, S1 = run_gdn(K, q, k, v, gb, S)
    check_gdn(out, S1, q, k, v, gb, S, [T])


def check_decaying(out, S1, q, k, v, gb, S0, scale=1.0):
    """As check_gdn, but what a token adds to the state's error is in proportion to the state that it meets and its
    update's parts, and decays with the state: B_t = c_t B_(t-1) + e^g |S| + (|beta| |v| + |u|) |k| with c_t the factor by
    which the recurrence enlarges a difference, e^g max(1, |1 - beta |k|^2|); the state is off by at most
    8 (2^-21 + 2^-20) 4 B in the Frobenius norm, a readout by half a step (fp16: of 2^-24 at least) and |q| times
    that.  One sequence."""
    eps = 8 * (2.0 ** -21 + 2.0 ** -20) * 4
    u = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[q.dtype]
    q, k, v, gb, S = f64(q)[0], f64(k)[0], f64(v)[0], f64(gb)[0], f64(S0)[0].copy()
    T, nk, d = q.shape
    nv = v.shape[1]
    kh = np.arange(nv) // (nv // nk)
    got, B, o = f64(out)[0], np.zeros(nv), np.zeros((nv, d))
    for t in range(T):
        dec, beta, kt, qt = np.exp(gb[0, :, t]), gb[1, :, t], k[t, kh], q[t, kh]
        S = dec[:, None, None] * S
        ut = beta[:, None] * (v[t] - np.einsum("hij,hj->hi", S, kt))
        k2 = (kt * kt).sum(1)
        B = dec * np.maximum(1, np.abs(1 - beta * k2)) * B + np.sqrt((S * S).sum((1, 2)))
        B += (np.abs(beta) * np.sqrt((v[t] ** 2).sum(1)) + np.sqrt((ut ** 2).sum(1))) * np.sqrt(k2)
        S = S + ut[:, :, None] * kt[:, None, :]
        o = scale * np.einsum("hij,hj->hi", S, qt)
        lim = u * np.abs(o) + 2.0 ** -25 + (scale * (1 + u) * eps * B * np.sqrt((qt * qt).sum(1)))[:, None]
        err = np.abs(got[t] - o)
        assert (err <= lim).all(), f"token {t}: {np.nanmax(err / lim):.2f} of the bound"
    es = np.sqrt(((f64(S1)[0] - S) ** 2).sum((1, 2)))
    # (a state that decays out of fp32's normal range, 2^-126 for each of 128 x 128 entries, has fewer bits or none)
    lim = eps * B + 128 * 2.0 ** -126
    assert (es <= lim).all(), f"state: {np.max(es / lim):.2e} of the bound"


@pytest.mark.parametrize("T", [16, 17, 90])
@pytest.mark.parametrize("dt,size,value", [(torch.float16, 1.0, 0), (torch.float16, 1.0, 1), (torch.bfloat16, 1.0, 0),
                                           (torch.bfloat16, 1.0, 1), (torch.bfloat16, 1e4, 0), (torch.bfloat16, 1e4, 1),
                                           (torch.bfloat16, 2.0 ** 60, 1)])
@pytest.mark.parametrize("g", [-0.3, -0.7, -1.0, -3.0])
def test_gdn_the_states_own_size_sets_its_precision(K, T, dt, size, value, g):  # noqa: F811
    """A state that decays from far above the values to their size, or to nothing where they are 0."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=17, sigma=size)
    v = v * value
    gb[:, 0] = g
    out, S1 = run_gdn(K, q, k, v, gb, S)
    check_decaying(out, S1, q, k, v, gb, S)


@pytest.mark.parametrize("T", [7, 40, 90])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("what", ["growth", "beta", "keys", "late decay"])
def test_gdn_gates_and_keys_beyond_their_range(K, T, dt, what):  # noqa: F811
    """g above 0, beta up to 2 and below 0, keys of norm 2, a decay to nothing behind tokens without any: some
    tokens of them, in some heads."""
    q, k, v, gb, S = make_gdn(1, T, 2, 6, 128, dt, seed=18, g_scale=0.2)
    k = k.clone()
    if what == "growth":
        gb[:, 0, ::2, T // 3:T // 3 + 6] = 0.7
    elif what == "beta":
        gb[:, 1, 1] *= 2
        gb[:, 1, 4, ::5] *= -1
    elif what == "keys":
        k[:, T // 2:T // 2 + 3] *= 2
    else:
        v[:, T // 4:T // 4 + 24] = 0
        gb[:, 0, ::2, T // 4:] = 0
        gb[:, 0, ::2, T // 4 + 2] = -float("inf")
    out, S1 = run_gdn(K, q, k, v, gb, S)
    check_decaying(out, S1, q, k, v, gb, S)


@pytest.mark.parametrize("T", [16, 17, 40])
@pytest.mark.parametrize("dt,size", [(torch.bfloat16, 1.0), (torch.bfloat16, 2.0 ** 60), (torch.bfloat16, 2.0 ** 90),
                                     (torch.float16, 1.0), (torch.float16, 2.0 ** 12)])
def test_gdn_a_state_that_is_wiped_out(K, T, dt, size):  # noqa: F811
    """A decay to nothing at the first token and values of 0, then (from token 16 on) values far below the state
    that was; and values that drop from far above to far below 1 with nothing written."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=19, sigma=size)
    v = v / size
    v[:, :16] = 0
    gb[:, 0, :, 0] = -float("inf")
    out, S1 = run_gdn(K, q, k, v, gb, S)
    assert torch.isfinite(S1).all() and (out[:, :16] == 0).all()
    check_decaying(out, S1, q, k, v, gb, S)
    v = torch.cat((v[:, 16:] * 0 + size, v[:, 16:] * 0 + 1 / size), 1)[:, :T]
    T = v.shape[1]
    if T > 8:
        q, k, gb = q[:, :T], k[:, :T], gb[..., :T].contiguous()
        gb[:, 1], S[:] = 0, 0
        out, S1 = run_gdn(K, q, k, v, gb, S)
        assert (S1 == 0).all() and (out == 0).all()


@pytest.mark.parametrize("T", [8, 16, 80])
@pytest.mark.parametrize("dt,state,value", [
    (torch.float16, 1e-2, 1e-2), (torch.float16, 1e-3, 1e-3), (torch.float16, 1e-4, 1e-4), (torch.float16, 0, 1e-5),
    (torch.float16, 1e-30, 1e-6), (torch.float16, 1e6, 1e4), (torch.float16, 1e30, 0), (torch.bfloat16, 0, 1e-30),
    (torch.bfloat16, 1e-30, 1e-30), (torch.bfloat16, 1e30, 1e30), (torch.bfloat16, 1e34, 0)])
def test_gdn_values_and_states_of_any_size(K, T, dt, state, value):  # noqa: F811
    """fp32's precision relative to what the state and the values are, as token by token."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=20, sigma=state, g_scale=0.2)
    v = (v.float() * value).to(dt)
    scale = 1 / max(state, value, 1.0)
    out, S1 = run_gdn(K, q, k, v, gb, S, scale=scale)
    check_decaying(out, S1, q, k, v, gb, S, scale)


@pytest.mark.parametrize("T", [8, 80])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_a_row_of_the_state_depends_on_its_own_column_of_v_only(K, T, dt):  # noqa: F811
    """An outlier column, and a NaN and an infinity in two others: everything else keeps every bit, those
    columns' tokens before them too."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=21, g_scale=0.2)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    v2, t = v.clone(), 5
    v2[:, :, 1, 5] *= 2.0 ** 12
    out2, S2 = run_gdn(K, q, k, v2, gb, S)
    same = torch.ones(4, 128, dtype=torch.bool, device="cuda")
    same[1, 5] = False
    assert torch.equal(out2[0][:, same], out[0][:, same]) and torch.equal(S2[0][same], S1[0][same])
    v2 = v.clone()
    v2[0, t, 0, 17], v2[0, t, 3, 127] = float("nan"), float("inf")
    out2, S2 = run_gdn(K, q, k, v2, gb, S)
    lost = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    lost[0, 17] = lost[3, 127] = True
    assert not torch.isfinite(out2[0, t:][:, lost]).any() and not torch.isfinite(S2[0][lost]).any()
    v3 = v2.clone()
    v3[0, t, 0, 17], v3[0, t, 3, 127] = 0, 0
    o, _, _, _, _ = gdn_plain(f64(q), f64(k), f64(v3), f64(gb), f64(S), [T], 1.0)
    half = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    got, o = f64(out2[0, :t][:, lost]), o[0, :t][:, lost.cpu().numpy()]
    assert (np.abs(got - o) <= (half + 2.0 ** -12) * np.abs(o).max() + 2.0 ** -20).all()
    rest = ~lost
    check = torch.where(rest, out2[0], out2.new_zeros(())), torch.where(rest[..., None], S2[0], S2.new_zeros(()))
    v3[0, :, 0, 17], v3[0, :, 3, 127] = 0, 0
    S3 = S.clone()
    S3[0][lost] = 0
    check_decaying(check[0][None], check[1][None], q, k, v3, gb, S3)


@pytest.mark.parametrize("T", [8, 16, 90])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("state", [0, 1e-4, 1.0])
@pytest.mark.parametrize("beta", [1e-2, 1e-4, 1e-6, 1e-12])
def test_gdn_heads_that_write_little(K, T, dt, state, beta):  # noqa: F811
    """beta far below 1, alone or beside a head that writes in full: fp32's precision of what is written."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=22, sigma=state, g_scale=0.2)
    gb[:, 1, :3] *= beta
    scale = 1.0 if state else 2.0 ** -10 / beta  # readouts in the output's range
    out, S1 = run_gdn(K, q, k, v, gb, S, scale=scale)
    for i in range(2 if state else 1):  # (with that scale the head that writes in full leaves the range)
        h, kh = slice(2 * i, 2 * i + 2), slice(i, i + 1)
        check_decaying(out[:, :, h], S1[:, h], q[:, :, kh], k[:, :, kh], v[:, :, h], gb[:, :, h], S[:, h], scale)


@pytest.mark.parametrize("T", [8, 16, 90])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [-6, -14, -60])
def test_gdn_keys_of_any_size(K, T, dt, power):  # noqa: F811
    """Keys far below norm 1 (fp16: with the bits that fp16 leaves them), alone and among keys of norm 1."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=23, sigma=0.0, g_scale=0.2)
    k = k.clone()
    k[:, :, 0] *= 2.0 ** power
    k[:, ::3, 1] *= 2.0 ** power
    scale = 2.0 ** (-power - 6) if dt == torch.bfloat16 else 1.0
    for i in range(2):
        h, kh = slice(2 * i, 2 * i + 2), slice(i, i + 1)
        qi, ki, vi, gi, Si = q[:, :, kh], k[:, :, kh], v[:, :, h], gb[:, :, h].contiguous(), S[:, h].contiguous()
        out, S1 = run_gdn(K, qi, ki, vi, gi, Si, scale=scale if i == 0 else 1.0)
        check_decaying(out, S1, qi, ki, vi, gi, Si, scale if i == 0 else 1.0)


@pytest.mark.parametrize("T", [8, 16, 80])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gdn_what_is_not_finite_reaches_no_token_before_it(K, T, dt, bad):  # noqa: F811
    """In q: its token's readouts only; in k, g or beta: from its token on, in the heads that read it."""
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=24, g_scale=0.2)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    t = T // 2 + 2
    others = torch.arange(T, device="cuda") != t
    q2 = q.clone()
    q2[0, t, 0, 9] = bad
    out2, S2 = run_gdn(K, q2, k, v, gb, S)
    assert torch.equal(S2, S1) and torch.equal(out2[:, others], out[:, others])
    assert torch.equal(out2[0, t, 2:], out[0, t, 2:]) and not torch.isfinite(out2[0, t, :2]).any()
    k2, g2, b2 = k.clone(), gb.clone(), gb.clone()
    k2[0, t, 0, 9], g2[0, 0, :2, t], b2[0, 1, :2, t] = bad, bad, bad
    for ki, gi in ((k2, gb), (k, g2), (k, b2)):
        out2, S2 = run_gdn(K, q, ki, v, gi, S)
        assert torch.equal(S2[:, 2:], S1[:, 2:]) and torch.equal(out2[:, :, 2:], out[:, :, 2:])
        assert not torch.isfinite(S2[:, :2]).all() and not torch.isfinite(out2[0, t, :2]).all()
        check_decaying(out2[:, :t, :2], run_gdn(K, q[:, :t], k[:, :t], v[:, :t], gb[..., :t].contiguous(), S)[1][:, :2],
                       q[:, :t, :1], k[:, :t, :1], v[:, :t, :2], gb[:, :, :2, :t], S[:, :2])


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens", [[1, 100], [0, 8, 9, 1, 40, 8], [3, 17] * 9])
def test_gdn_a_sequence_goes_by_its_own_length(K, dt, lens):  # noqa: F811
    """Single and drafted tokens next to prompts in one call: each short sequence has every bit of a call of its
    own, in place too, and nothing behind it is read or written."""
    n, T = len(lens), max(lens)
    q, k, v, gb, S = make_gdn(n, T, 2, 4, 128, dt, seed=25)
    out, S1 = run_gdn(K, q, k, v, gb, S, lens=lens)
    check_gdn(out, S1, q, k, v, gb, S, lens)
    S2, out2 = S.clone(), torch.full_like(out, float("nan"))
    K.kva_op_gdn_forward(q, k, v, gb, S2, S2, out2, lens=lens)
    assert torch.equal(S2, S1)
    for i, m in enumerate(lens):
        assert torch.equal(out2[i, :m], out[i, :m]) and torch.isnan(out[i, m:]).all() and torch.isnan(out2[i, m:]).all()
        if m <= 8:
            a = [x[i:i + 1, :m] for x in (q, k, v)]
            o, s = run_gdn(K, *a, gb[i:i + 1, :, :, :m].contiguous(), S[i:i + 1])
            assert torch.equal(o[0], out[i, :m]) and torch.equal(s[0], S1[i])


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,nv,n", [(128, 50, 7), (128, 24, 4), (64, 100, 3)])
def test_gdn_a_sequence_has_the_same_bits_in_any_batch(K, dt, d, nv, n):  # noqa: F811
    """Alone, beside others of its length, and beside others of other lengths, whatever layout of the work that
    takes."""
    T = 50
    q, k, v, gb, S = make_gdn(n, T, 2, nv, d, dt, seed=26, g_scale=0.3)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    lens = [T, 3, 30, 0, 20, 8, 9][:n]
    out2, S2 = run_gdn(K, q, k, v, gb, S, lens=lens)
    assert torch.equal(out2[0], out[0]) and torch.equal(S2[0], S1[0])
    for i in (0, n - 1):
        one = [x[i:i + 1] for x in (q, k, v, gb, S)]
        o, s = run_gdn(K, *one)
        assert torch.equal(o[0], out[i]) and torch.equal(s[0], S1[i])


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_mixed_calls_one_after_another_captured_and_replayed(K, dt):  # noqa: F811
    """Prompts and single tokens (two launches a call), the state of one call going into the next, in place, with
    runs that go token by token among them: a replayed graph and eager calls on another stream end alike."""
    n, T, lens = 4, 60, [[1, 60, 8, 33], [40, 1, 0, 9], [3, 2, 60, 1]]
    q, k, v, gb, S = make_gdn(n, T, 2, 6, 128, dt, seed=27)
    gb[1, 0, 2, 20] = 0.5
    out = torch.full((3, *v.shape), float("nan"), dtype=dt, device="cuda")

    def calls(state, o, **kw):
        for i, m in enumerate(lens):
            K.kva_op_gdn_forward(q, k, v, gb, state, state, o[i], lens=m, **kw)

    S1, side = S.clone(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(S1, out, stream=side)
    side.synchronize()
    S2, out2 = S.clone(), torch.full_like(out, float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(S2, out2)
    for _ in range(3):
        S2.copy_(S)
        out2.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(S2, S1) and torch.equal(out2.nan_to_num(7.0), out.nan_to_num(7.0))
    want = S
    for i, m in enumerate(lens):
        o, after = run_gdn(K, q, k, v, gb, want, lens=m)
        assert torch.equal(o.nan_to_num(7.0), out[i].nan_to_num(7.0))
        want = after
    assert torch.equal(want, S1)


# ------------------------------------------------------------------ residual add + RMSNorm, q8_0 codes
def q8_of(K, g):  # noqa: F811
    """Codes and scales of rows whose normalised values are +g and -g: a row of ones has the norm 1, which
    leaves every bit of g."""
    n = g.numel()
    h = torch.ones(2, n, device="cuda")
    h[1] = -1
    x, ho = torch.zeros_like(h), torch.empty_like(h)
    codes, sc = torch.empty(2, n, dtype=torch.int8, device="cuda"), torch.empty(n // 32, 2, dtype=torch.float16, device="cuda")
    K.kva_op_add_rmsnorm(x, h, g, ho, codes, scales=sc, eps=0.0)
    return f64(codes), f64(sc)


def test_add_rmsnorm_q8_codes_are_the_nearest(K):  # noqa: F811
    """y / d with d = max|y| / 127, to the nearest, halves away from zero.  The kernel's reciprocal is off by at
    most 1.5 last places and its product by half of one, 127 x 2^-22 of a code together: nearer to a half
    than that, and only there, either neighbour stands.  Exact halves (max|y| a power of two times 127) go away from
    zero."""
    rng = np.random.default_rng(5)
    blocks = 512
    big = (rng.uniform(1, 2, blocks) * 2.0 ** rng.integers(-20, 12, blocks)).astype(np.float32)
    big[:32] = 127 * 2.0 ** rng.integers(-20, 12, 32)
    half = (rng.integers(-127, 127, (blocks, 32)) + 0.5) * big[:, None].astype(np.float64) / 127
    y = half.astype(np.float32)
    for step in range(1, 5):  # the floats on both sides of a half
        y[:, step] = np.nextafter(y[:, step], np.float32(np.inf))
        y[:, 4 + step] = np.nextafter(y[:, 4 + step], np.float32(-np.inf))
    y[:, 9:20] = (rng.uniform(-1, 1, (blocks, 11)) * big[:, None]).astype(np.float32)
    y[32:, 20:31] *= (1 + rng.uniform(-1e-4, 1e-4, (blocks - 32, 11))).astype(np.float32)
    y[:, 31] = big * np.where(rng.random(blocks) < 0.5, 1, -1)
    y = np.clip(y, -big[:, None], big[:, None])
    codes, sc = q8_of(K, torch.from_numpy(y.reshape(-1)).cuda())
    for r, sign in ((0, 1), (1, -1)):
        q = sign * y.astype(np.float64) * 127 / big[:, None].astype(np.float64)
        want = np.sign(q) * np.floor(np.abs(q) + 0.5)
        got = codes[r].reshape(blocks, 32)
        near = np.abs(np.abs(q) % 1 - 0.5) <= 127 * 2.0 ** -22
        assert (np.abs(got - q) <= 0.5 + 127 * 2.0 ** -22).all()
        assert np.array_equal(got[~near], want[~near]) and near.sum() < near.size / 2
        exact = np.abs(q) % 1 == 0.5
        assert np.array_equal(got[exact], want[exact]) and exact.sum() > 300
        d = (big.astype(np.float64) / 127)
        assert (np.abs(sc[:, r] - d) <= d * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all()


def test_add_rmsnorm_q8_codes_of_the_largest_and_smallest_blocks(K):  # noqa: F811
    """Up to fp32's largest value: the codes stand, the scale is infinite where fp16 ends.  Blocks below fp16's
    scales have the scale 0."""
    tops = [2.0 ** 20, 2.0 ** 100, 2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 126, 2.0 ** 127, 3.4e38, 2.0 ** -40, 2.0 ** -118]
    y = torch.linspace(-1, 1, 32, dtype=torch.float64)[None] * torch.tensor(tops, dtype=torch.float64)[:, None]
    codes, sc = q8_of(K, y.float().reshape(-1).cuda())
    q = y.float().double() * 127 / y.float().double().abs().amax(1, keepdim=True)
    assert np.array_equal(codes[0].reshape(-1, 32), f64(torch.round(q))) and np.array_equal(codes[1], -codes[0])
    assert np.isfinite(sc[0]).all() and (sc[1:7] == np.inf).all()
    assert (sc[7:] == 0).all()


def test_add_rmsnorm_as_many_rows_as_an_int32_counts(K):  # noqa: F811
    """2^31 - 1 rows of 4 (17 GB a tensor)."""
    rows = 2 ** 31 - 1
    x = torch.zeros(rows, 4, dtype=torch.float16, device="cuda")
    h = torch.ones_like(x)
    h[-3:] *= torch.tensor([[2.0], [-1.0], [0.0]], device="cuda", dtype=torch.float16)
    g = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    out = torch.empty_like(x)
    K.kva_op_add_rmsnorm(x, h, g, h, out, eps=0.0)
    want = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda", dtype=torch.float16)
    for part in out[:-3].split(2 ** 28):
        assert (part == want).all()
    assert torch.equal(out[-3], want) and torch.equal(out[-2], -want) and torch.isnan(out[-1]).all()
