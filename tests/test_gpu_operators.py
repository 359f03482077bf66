"""The several-token operators on the GPU against plain implementations in 64 bits.

Tolerances.  u = eps / 2 of the 16-bit type (fp16 2^-11, bf16 2^-8) is the largest relative
rounding of one stored value.  Two fp16 terms hold a value to u2 = 2^-21 (cut to 11 bits, the remainder
below 2^-10 rounded).

gdn_forward.  A readout is a sum over the state at the start of a run of at most 16 tokens and over
that run's updates; both operands may be rounded to 16 bits once (the state and the updates u_s, and
the coefficients e^(gam_t - gam_s) k_s.q_t), the result once more:
    |err o| <= scale (u A1 + 2 u A2) + u |o|,  A1 = e^gam sum |S0| |q|,  A2 = sum_s |u_s| |coefficient|,
with (1 + 16 u + 2^-18) on the sums for second-order terms and fp32 noise.  The state may not see a
16-bit rounding: five operands of two 16-bit terms (u2 each) and fp32 sums (2^-20 covers 128 terms)
move the state of one run by at most 8 (u2 + 2^-20) 4 (|S0| + |V| + |U|) in the Frobenius norm
(16 unit keys have a 2-norm of at most 4; 8 counts the roundings and what they meet on the way), and
later runs do not enlarge it.  It is summed over the runs.

bf16 runs hold their fp16 terms in units of 2^-7 to 2^-8 of M, the largest of |v| of the run and the norms
of the state's rows before it: a term drops at most d = 2^-25 2^-7 M.  On the way to a readout that is 11.3 d
through S k (128 columns, a key of norm 1), 12.3 d in w, 16 times that in u (16 coefficients of at most 1), d
more for u itself, and 16 of those meet in a readout: below 3300 d < 2^-20 M.  Only values far below their
run's largest can tell.
"""
import math

import numpy as np
import pytest
import torch

from tests.parity import f64

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TWO_TERMS = 2.0 ** -21
NAN = float("nan")


@pytest.fixture(scope="module")
def K():
    import hybrid_deltanet_attention_kva_b200 as K
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return K


# ------------------------------------------------------------------ gated delta rule
def gdn_plain(q, k, v, gb, S0, lens, scale, run=16):
    """o, S and the error bounds above; float64 numpy, token by token."""
    n, T, nk, d = q.shape
    nv = v.shape[2]
    kh = np.arange(nv) // (nv // nk)
    S, o, bo = S0.copy(), np.zeros((n, T, nv, d)), np.zeros((n, T, nv, d))
    bs = np.zeros((n, nv))
    bm = np.zeros((n, T, nv, 1))
    for i in range(n):
        for t in range(lens[i]):
            if t % run == 0:
                St, a1 = S[i].copy(), np.ones(nv)
                hist = []
                vn = np.sqrt((v[i, t:min(t + run, lens[i])] ** 2).sum((0, 2)))
                base = np.sqrt((St ** 2).sum((1, 2))) + vn
                bm[i, t:t + run, :, 0] = np.maximum(np.abs(v[i, t:min(t + run, lens[i])]).max((0, 2)),
                                                    np.sqrt((St ** 2).sum(2)).max(1))
            with np.errstate(invalid="ignore"):
                dec = np.exp(gb[i, 0, :, t])
            kt, qt = k[i, t, kh], q[i, t, kh]
            u = gb[i, 1, :, t][:, None] * (v[i, t] - dec[:, None] * np.einsum("hij,hj->hi", S[i], kt))
            S[i] = dec[:, None, None] * S[i] + u[:, :, None] * kt[:, None, :]
            o[i, t] = scale * np.einsum("hij,hj->hi", S[i], qt)
            a1 = a1 * dec
            hist = [(c * dec, uu, kk) for c, uu, kk in hist] + [(np.ones(nv), u, kt)]
            A1 = a1[:, None] * np.einsum("hij,hj->hi", np.abs(St), np.abs(qt))
            A2 = sum((c * np.abs((kk * qt).sum(1)))[:, None] * np.abs(uu) for c, uu, kk in hist)
            bo[i, t] = A1 + 2 * A2
            if (t + 1) % run == 0 or t + 1 == lens[i]:
                bs[i] += base + np.sqrt(sum((uu ** 2).sum(1) for _, uu, _ in hist))
    return o, S, bo, bs, bm


def check_gdn(out, S, q, k, v, gb, S0, lens, scale=1.0):
    u = HALF_STEP[q.dtype]
    o, Sw, bo, bs, bm = gdn_plain(f64(q), f64(k), f64(v), f64(gb), f64(S0), lens, scale)
    units = q.dtype == torch.bfloat16 and max(lens) > 8
    out, S = f64(out), f64(S)
    for i, m in enumerate(lens):
        lim = abs(scale) * bo[i, :m] * u * (1 + 16 * u + 2.0 ** -18 / u) + u * np.abs(o[i, :m]) + 2.0 ** -24
        if units:
            lim = lim + abs(scale) * 2.0 ** -20 * bm[i, :m]
        err = np.abs(out[i, :m] - o[i, :m])
        assert np.isfinite(out[i, :m]).all(), "non-finite output"
        assert (err <= lim).all(), f"sequence {i}: {np.max(err / lim):.2f} of the bound"
    es = np.sqrt(((S - Sw) ** 2).sum((2, 3)))
    lim = 8 * (TWO_TERMS + 2.0 ** -20) * 4 * bs + 2.0 ** -24 * (1 + np.sqrt((Sw ** 2).sum((2, 3))))
    assert np.isfinite(S).all(), "non-finite state"
    assert (es <= lim).all(), f"state: {np.max(es / lim):.2f} of the bound"


def make_gdn(n, T, nk, nv, d, dt, seed=0, g_scale=1.0, sigma=0.3):
    g = torch.Generator().manual_seed(1000 * n + 7 * T + nv + d + seed)
    x = torch.randn(n, T, 2 * nk + nv, d, generator=g)
    x[:, :, :2 * nk] /= x[:, :, :2 * nk].norm(dim=-1, keepdim=True).clamp_min(1e-6)
    x = x.to(dt).cuda()
    gate = -g_scale * torch.rand(n, nv, T, generator=g)
    gb = torch.stack((gate, torch.rand(n, nv, T, generator=g)), 1).cuda()
    S = (sigma * torch.randn(n, nv, d, d, generator=g)).cuda()
    return x[:, :, :nk], x[:, :, nk:2 * nk], x[:, :, 2 * nk:], gb, S


def run_gdn(K, q, k, v, gb, S, lens=None, scale=1.0, **kw):
    out = torch.full(v.shape, NAN, dtype=q.dtype, device="cuda")
    S1 = torch.full_like(S, NAN)
    K.kva_op_gdn_forward(q, k, v, gb, S, S1, out, lens=lens, scale=scale, **kw)
    torch.cuda.synchronize()
    return out, S1


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 150])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_lengths(K, T, d, dt):
    q, k, v, gb, S = make_gdn(2, T, 2, 6, d, dt)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    check_gdn(out, S1, q, k, v, gb, S, [T, T])


@pytest.mark.parametrize("n,nk,nv,d", [(1, 1, 1, 64), (1, 1, 1, 128), (3, 1, 5, 64), (2, 16, 48, 128), (40, 2, 2, 128)])
def test_gdn_heads(K, n, nk, nv, d):
    for T in (4, 37):
        q, k, v, gb, S = make_gdn(n, T, nk, nv, d, torch.float16, seed=1)
        out, S1 = run_gdn(K, q, k, v, gb, S, scale=0.25)
        check_gdn(out, S1, q, k, v, gb, S, [T] * n, 0.25)


@pytest.mark.parametrize("T", [6, 70])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_ragged_lengths_leave_the_rest_alone(K, T, dt):
    """Sequences of 0, 1, some and all tokens: nothing behind a sequence is read (it holds NaN) or written."""
    lens = [0, 1, T, T - 1, T // 2, 17 if T > 17 else 3]
    n = len(lens)
    q, k, v, gb, S = make_gdn(n, T, 2, 4, 128, dt, seed=2)
    for i, m in enumerate(lens):
        for t in (q, k, v):
            t[i, m:] = NAN
        gb[i, :, :, m:] = NAN
    out, S1 = run_gdn(K, q, k, v, gb, S, lens=lens)
    for i, m in enumerate(lens):
        assert torch.isnan(out[i, m:]).all()
    assert torch.equal(S1[0], S[0])
    check_gdn(out, S1, q, k, v, gb, S, lens)


def test_gdn_no_tokens_and_in_place(K):
    q, k, v, gb, S = make_gdn(2, 0, 2, 4, 64, torch.float16)
    _, S1 = run_gdn(K, q, k, v, gb, S)
    assert torch.equal(S1, S)
    for T in (3, 50):
        q, k, v, gb, S = make_gdn(2, T, 2, 4, 64, torch.float16)
        out, S1 = run_gdn(K, q, k, v, gb, S)
        S2, out2 = S.clone(), torch.empty_like(out)
        K.kva_op_gdn_forward(q, k, v, gb, S2, S2, out2)
        assert torch.equal(S2, S1) and torch.equal(out2, out)


@pytest.mark.parametrize("T", [7, 90])
def test_gdn_gates_at_their_ends(K, T):
    """No decay, decay to nothing (g of -1e4, -infinity), decays that accumulate to thousands, beta 0 and
    1, and the same key again and again: no overflow, no NaN, the same bounds."""
    q, k, v, gb, S = make_gdn(1, T, 1, 8, 128, torch.float16, seed=3)
    k[:, 1:] = k[:, :1]
    gb[:, 0, 0] = 0.0
    gb[:, 0, 1, ::3] = -1e4
    gb[:, 0, 2, ::2] = -math.inf
    gb[:, 0, 3] = -90.0
    gb[:, 0, 4, ::2] = -40.0
    gb[:, 0, 5] *= 1e-6
    gb[:, 1, 0] = 1.0
    gb[:, 1, 1, 1::2] = 0.0
    gb[:, 1, 6] = 0.0
    gb[:, 1, 7] = 1.0
    gb[:, 0, 7] = 0.0
    out, S1 = run_gdn(K, q, k, v, gb, S)
    check_gdn(out, S1, q, k, v, gb, S, [T])


def test_gdn_strides_and_far_offsets(K):
    """Views into wider rows, tokens-first outputs, and offsets that pass 32 bits."""
    n, T, nk, nv, d = 2, 20, 2, 4, 64
    q, k, v, gb, S = make_gdn(n, T, nk, nv, d, torch.bfloat16, seed=4)
    want, Sw = run_gdn(K, q.contiguous(), k.contiguous(), v.contiguous(), gb, S)
    out = torch.full((T, n, nv, d), NAN, dtype=v.dtype, device="cuda")
    S1 = torch.empty_like(S)
    K.kva_op_gdn_forward(q, k, v, gb, S, S1, out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want) and torch.equal(S1, Sw)
    far = 2 ** 31 + 64
    big = torch.empty(far + T * nv * d, dtype=v.dtype, device="cuda")
    vv, oo = torch.as_strided(big, v.shape, (far, nv * d, d, 1)), torch.empty_like(want)
    vv.copy_(v)
    K.kva_op_gdn_forward(q, k, vv, gb, S, S1, oo)
    assert torch.equal(oo, want) and torch.equal(S1, Sw)
    o2 = torch.as_strided(big, v.shape, (far, nv * d, d, 1))
    K.kva_op_gdn_forward(q, k, v.contiguous(), gb, S, S1, o2)
    assert torch.equal(o2, want) and torch.equal(S1, Sw)


@pytest.mark.parametrize("T", [4, 200])
def test_gdn_split_runs_agree(K, T):
    """One call over T tokens and two calls over its halves: the state carries over."""
    q, k, v, gb, S = make_gdn(1, T, 2, 6, 128, torch.float16, seed=5, g_scale=0.05)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    m = T // 2 + 1
    _, Sa = run_gdn(K, q[:, :m], k[:, :m], v[:, :m], gb[..., :m].contiguous(), S)
    ob, Sb = run_gdn(K, q[:, m:], k[:, m:], v[:, m:], gb[..., m:].contiguous(), Sa)
    check_gdn(ob, Sb, q[:, m:], k[:, m:], v[:, m:], gb[..., m:], Sa, [T - m])
    assert (Sb - S1).norm() <= 2.0 ** -14 * S1.norm()  # far above two fp32 paths, far below 16 bits' 2^-11


@pytest.mark.parametrize("T", [5, 80])
@pytest.mark.parametrize("power", [-70, -20, 12, 60])
def test_gdn_bf16_follows_the_values_scale(K, T, power):
    """v and the state times a power of two: everything scales exactly, however far from 1 it is."""
    q, k, v, gb, S = make_gdn(2, T, 2, 4, 128, torch.bfloat16, seed=7, g_scale=0.2)
    out, S1 = run_gdn(K, q, k, v, gb, S)
    f = 2.0 ** power
    out2, S2 = run_gdn(K, q, k, v * f, gb, S * f)
    assert torch.equal(out2, out * f) and torch.equal(S2, S1 * f)


@pytest.mark.parametrize("T", [5, 80])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_scales_that_change_and_lost_columns(K, T, dt):
    """Tokens of very different sizes and states far from them stay within the bounds of their own size;
    a NaN or infinity in v spoils its own column only."""
    big = 64.0 if dt == torch.float16 else 2.0 ** 30
    q, k, v, gb, S = make_gdn(1, T, 2, 4, 128, dt, seed=8)
    v = v.clone()
    v[:, T // 2:] *= big
    S[:, 1] *= big
    S[:, 2] = 0
    out, S1 = run_gdn(K, q, k, v, gb, S)
    check_gdn(out, S1, q, k, v, gb, S, [T])
    v2 = v.clone()
    v2[0, T // 3, 0, 5], v2[0, T // 4, 3, 127] = math.inf, NAN
    out2, S2 = run_gdn(K, q, k, v2, gb, S)
    spoiled = torch.zeros(4, 128, dtype=torch.bool)
    spoiled[0, 5] = spoiled[3, 127] = True
    assert not torch.isfinite(out2[0, -1].cpu()[spoiled]).any() and torch.isfinite(out2[0].cpu()[:, ~spoiled]).all()
    assert torch.isfinite(S2[0].cpu()[~spoiled]).all()
    v3 = v2.clone()
    v3[0, T // 3, 0, 5], v3[0, T // 4, 3, 127] = 0, 0
    out3, S3 = run_gdn(K, q, k, v3, gb, S)
    check_gdn(out3, S3, q, k, v3, gb, S, [T])
    lim = 2.0 ** -18 * S3[0].norm(dim=(1, 2)).max().item()  # another scale, other last bits
    assert ((S2 - S3)[0].cpu()[~spoiled].abs() <= lim).all()


@pytest.mark.parametrize("T", [5, 40])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_a_sequence_without_tokens_keeps_any_state(K, T, dt):
    """Next to sequences with tokens, bit for bit: values 10^68 apart, subnormals and infinities."""
    q, k, v, gb, S = make_gdn(2, T, 2, 4, 128, dt, seed=9)
    S[0] = torch.exp2(252 * torch.rand(S[0].shape, generator=torch.Generator().manual_seed(3)) - 126).cuda()
    S[0, :, ::7] = 2.0 ** -140
    S[0, 1, 3, 5], S[0, 2, 3, 5], S[0, 3, ::2] = math.inf, -3e38, 0.0
    out, S1 = run_gdn(K, q, k, v, gb, S, lens=[0, T])
    assert torch.equal(S1[0], S[0])
    check_gdn(out[1:], S1[1:], q[1:], k[1:], v[1:], gb[1:], S[1:], [T])


@pytest.mark.parametrize("n,nv", [(1, 70), (1, 100), (3, 50), (5, 47)])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_gdn_more_heads_than_the_gpu_takes_at_once(K, n, nv, dt):
    """Up to and past the counts of heads at which the work is laid out in another way, with ragged
    lengths, in place."""
    T = 36
    lens = [T - 3 * i for i in range(n)]
    q, k, v, gb, S = make_gdn(n, T, 1, nv, 128, dt, seed=10)
    out, S1 = run_gdn(K, q, k, v, gb, S, lens=lens)
    check_gdn(out, S1, q, k, v, gb, S, lens)
    S2, out2 = S.clone(), torch.full_like(out, NAN)
    K.kva_op_gdn_forward(q, k, v, gb, S2, S2, out2, lens=lens)
    assert torch.equal(S2, S1) and torch.equal(out2.nan_to_num(), out.nan_to_num())


def test_gdn_as_many_sequences_as_a_call_takes(K):
    n = K.kva.GDN_MAX_SEQ
    lens = [(7 * i) % 20 for i in range(n)]
    q, k, v, gb, S = make_gdn(n, 19, 1, 2, 64, torch.bfloat16, seed=11)
    out, S1 = run_gdn(K, q, k, v, gb, S, lens=lens)
    check_gdn(out, S1, q, k, v, gb, S, lens)
    for i, m in enumerate(lens):
        assert torch.isnan(out[i, m:]).all()


def test_gdn_scan_and_forward_reach_one_state(K):
    """The state of kva_op_gdn_scan (16-bit operands, its own 1e-2) and of this operator."""
    T, nk, nv, d = 130, 2, 6, 128
    q, k, v, gb, S = make_gdn(1, T, nk, nv, d, torch.float16, seed=6)
    _, S1 = run_gdn(K, q, k, v, gb, S)
    S2 = S.clone()
    K.kva_op_gdn_scan(k.reshape(1, T, nk * d).contiguous(), v.reshape(1, T, nv * d).contiguous(), gb, S2, 1, 1, nk, nv, d)
    rel = ((S2 - S1).flatten(2).norm(dim=2) / S1.flatten(2).norm(dim=2)).max()
    assert rel <= 1e-2


# ------------------------------------------------------------------ residual add + RMSNorm
def norm_plain(x, h, g, eps=1e-6):
    hs = (h.float() + x.float()).to(h.dtype)
    f = f64(hs)
    return hs, f / np.sqrt((f * f).mean(-1, keepdims=True) + eps) * f64(g)


# fp32 statistics: a thread adds up to 64 squares, then 8 warps' trees: 80 roundings of 2^-24, rsqrt 2 ulp
FP32_ROW = 2.0 ** -17


@pytest.mark.parametrize("rows,n", [(1, 4), (1, 5120), (3, 36), (37, 1028), (130, 5120), (5, 16384), (2, 12288)])
@pytest.mark.parametrize("xd", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("od", [torch.float16, torch.bfloat16])
def test_add_rmsnorm(K, rows, n, xd, hd, od):
    gen = torch.Generator().manual_seed(rows + n)
    x, h = torch.randn(rows, n, generator=gen).to(xd).cuda(), (3 * torch.randn(rows, n, generator=gen)).to(hd).cuda()
    g = (torch.rand(n, generator=gen) + 0.5).cuda()
    hs, y = norm_plain(x, h, g)
    ho, out = torch.empty_like(h), torch.empty(rows, n, dtype=od, device="cuda")
    K.kva_op_add_rmsnorm(x, h, g, ho, out)
    assert torch.equal(ho, hs)
    lim = np.abs(y) * (HALF_STEP[od] + FP32_ROW) + 2.0 ** -25  # fp16 below 2^-14 has steps of 2^-24
    assert (np.abs(f64(out) - y) <= lim).all()
    out2 = torch.empty_like(out)
    K.kva_op_add_rmsnorm(x, h, g, h, out2)  # in place
    assert torch.equal(h, hs) and torch.equal(out2, out)


@pytest.mark.parametrize("rows,n", [(1, 32), (1, 5120), (7, 96), (129, 2560), (33, 16384), (64, 1056)])
@pytest.mark.parametrize("xd,hd", [(torch.float32, torch.float32), (torch.float16, torch.bfloat16),
                                   (torch.bfloat16, torch.float32)])
def test_add_rmsnorm_q8(K, rows, n, xd, hd):
    """A code reads back within half a step of fp32 (0.5 d), plus what rounding d to fp16 moves 127
    steps by (127 * 2^-11 d < 0.0625 d; 2^-25 * 127 where d is below fp16's normal range)."""
    gen = torch.Generator().manual_seed(rows + n)
    x, h = torch.randn(rows, n, generator=gen).to(xd).cuda(), (3 * torch.randn(rows, n, generator=gen)).to(hd).cuda()
    x[0, :32] = 0
    h[0, :32] = 0  # a block of zeros
    g = (torch.rand(n, generator=gen) + 0.5).cuda()
    hs, y = norm_plain(x, h, g)
    ho = torch.empty_like(h)
    codes = torch.full((rows, n + 32), 99, dtype=torch.int8, device="cuda")[:, :n]  # rows with padding
    if (n + 32) % 16:
        codes = torch.empty(rows, n, dtype=torch.int8, device="cuda")
    sc = torch.empty(n // 32, rows, dtype=torch.float16, device="cuda")
    K.kva_op_add_rmsnorm(x, h, g, ho, codes, scales=sc)
    assert torch.equal(ho, hs)
    d = np.abs(y.reshape(rows, -1, 32)).max(-1)[..., None] / 127
    c = f64(codes).reshape(rows, -1, 32)
    back = c * f64(sc).T[..., None]
    lim = (0.5625 + 127 * FP32_ROW) * d + 127 * 2.0 ** -25
    assert (np.abs(back - y.reshape(rows, -1, 32)) <= lim).all()
    full = np.abs(c).max(-1)
    assert np.array_equal(full, np.where(d[..., 0] > 0, 127, 0))


def test_add_rmsnorm_strides_and_specials(K):
    rows, n = 6, 64
    gen = torch.Generator().manual_seed(1)
    X, H = torch.randn(rows, 100, generator=gen).cuda(), torch.randn(rows, 80, generator=gen).half().cuda()
    g = torch.rand(n, generator=gen).cuda()
    O = torch.full((rows, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    HO = torch.full((rows, 80), 7.0, dtype=torch.float16, device="cuda")
    X[1, 3], H[2, 5], X[3, 7] = NAN, math.inf, -math.inf
    X[4, :n], H[4, :n] = 0, 0
    hs, y = norm_plain(X[:, :n].contiguous(), H[:, :n].contiguous(), g)
    K.kva_op_add_rmsnorm(X[:, :n], H[:, :n], g, HO[:, :n], O[:, :n])
    got = f64(O[:, :n])
    assert np.array_equal(f64(HO[:, :n]), f64(hs), equal_nan=True)
    for r in (0, 4, 5):
        assert (np.abs(got[r] - y[r]) <= np.abs(y[r]) * (2.0 ** -8 + FP32_ROW)).all()
    assert np.isnan(got[1]).all()
    for r, c in ((2, 5), (3, 7)):  # inf / inf is NaN, the others inf's share: 0
        assert np.isnan(got[r, c]) and (np.delete(got[r], c) == 0).all()
    assert (O[:, n:] == 7).all() and (HO[:, n:] == 7).all()
    codes = torch.zeros(rows, n, dtype=torch.int8, device="cuda")
    sc = torch.zeros(n // 32, rows, dtype=torch.float16, device="cuda")
    K.kva_op_add_rmsnorm(X[:, :n], H[:, :n], g, HO[:, :n], codes, scales=sc)
    assert torch.isnan(sc[:, 1]).all() and (codes[1] == 0).all()
    assert torch.isnan(sc[0, 2]) and sc[1, 2] == 0 and (codes[2] == 0).all()
    assert (sc[:, 4] == 0).all() and (codes[4] == 0).all()


# ------------------------------------------------------------------ token log probabilities
def logp_plain(x, n_top):
    """lse, entropy, order of the alternatives: float64."""
    x = x.double().cpu()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    lse = (m + torch.log(s))[:, 0]
    p = e / s
    H = -torch.where(p > 0, p * (x - lse[:, None]), torch.zeros(())).sum(1)
    srt = torch.sort(x, dim=1, descending=True, stable=True)
    return x, lse.numpy(), H.numpy(), srt.indices[:, :n_top].numpy(), (srt.values[:, :n_top] - lse[:, None]).numpy()


def run_logp(K, x, tok, n_top):
    rows = x.shape[0]
    o = {k: torch.full((rows,), 5.0, device="cuda") for k in ("logprob", "lse", "entropy")}
    ids = torch.full((rows, n_top), -7, dtype=torch.int32, device="cuda")
    tl = torch.full((rows, n_top), 5.0, device="cuda")
    more = dict(top_id=ids, top_logprob=tl) if n_top else {}
    K.kva_op_token_logprobs(x, tok, o["logprob"], lse=o["lse"], entropy=o["entropy"], **more)
    return o["logprob"], o["lse"], o["entropy"], ids, tl


def check_logp(K, x, n_top, seed=0):
    """fp32: a thread's chain of at most V / 256 + 64 additions, each 2^-24, exponentials of 2 ulp of an
    argument of 2^-24 |x - m|: relative error of the sums `r`; results add half a step of their size."""
    rows, V = x.shape
    tok = torch.randint(0, V, (rows,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
    lp, lse, H, ids, tl = run_logp(K, x, tok, n_top)
    xd, wl, wH, wi, wt = logp_plain(x, n_top)
    r = (V / 256 + 64 + 40) * 2.0 ** -24
    big = np.abs(xd.numpy()[np.isfinite(xd.numpy())]).max() + np.abs(wl)
    lim = r + 2.0 ** -23 * big
    assert (np.abs(f64(lse) - wl) <= lim).all()
    assert (np.abs(f64(H) - wH) <= 4 * r * (1 + np.abs(wH) + np.log(V)) + 2.0 ** -23 * big).all()
    want = xd[torch.arange(rows), tok.long().cpu()].numpy() - wl
    got = f64(lp)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    assert (np.abs(got - want)[fin] <= lim[fin] + 2.0 ** -23 * np.abs(want[fin])).all()
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert (np.abs(f64(tl) - wt) <= lim[:, None] + 2.0 ** -23 * np.abs(wt)).all()


@pytest.mark.parametrize("rows,V", [(1, 1), (1, 7), (3, 33), (2, 1000), (5, 4099), (37, 50257), (400, 513), (1, 131072),
                                    (2, 262147)])
@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n_top", [0, 1, 8, 32])
def test_token_logprobs(K, rows, V, dt, n_top):
    gen = torch.Generator(device="cuda").manual_seed(rows + V)
    x = (3 * torch.randn(rows, V, generator=gen, device="cuda")).to(dt)
    check_logp(K, x, min(n_top, V))


@pytest.mark.parametrize("rows,V,dt", [(1000, 9001, torch.bfloat16), (1000, 16390, torch.float32),
                                       (1900, 6000, torch.float32), (1900, 8195, torch.float16)])
def test_token_logprobs_many_rows(K, rows, V, dt):
    gen = torch.Generator(device="cuda").manual_seed(V)
    check_logp(K, (3 * torch.randn(rows, V, generator=gen, device="cuda")).to(dt), 8)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
def test_token_logprobs_any_alignment(K, dt):
    """Rows that begin at every offset inside a 16-byte piece."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    buf = (3 * torch.randn(9 * 2051 + 64, generator=gen, device="cuda")).to(dt)
    for off in range(0, 9):
        for V in (1, 5, 515, 2048):
            check_logp(K, torch.as_strided(buf, (9, V), (2051, 1), off), min(6, V))


def test_token_logprobs_ties_and_orders(K):
    """Equal logits everywhere, sorted both ways, a peak, two-valued rows: ids in token order."""
    V = 5000
    up = torch.arange(V).float() / 100
    rows = [torch.zeros(V), up, up.flip(0), (torch.arange(V) % 2).float(), (torch.arange(V) % 997 == 3).float() * 50,
            torch.where(torch.arange(V) >= V - 40, 1.0, 0.0), torch.full((V,), -3e38), torch.full((V,), 3e38),
            torch.linspace(-3e4, 3e4, V)]
    for dt in (torch.float32, torch.bfloat16):
        check_logp(K, torch.stack(rows).to(dt).cuda(), 32)


def test_token_logprobs_masks_and_specials(K):
    V, inf = 700, math.inf
    gen = torch.Generator().manual_seed(4)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        x = torch.randn(8, V, generator=gen).to(dt)
        x[0] = -inf                       # nothing left
        x[1] = -inf
        x[1, 650] = 2.0                   # one token left
        x[2, 3] = NAN
        x[3, 699] = inf
        x[4] = torch.finfo(dt).min        # the type's lowest value is a logit like any other
        x[5, :690] = -inf
        tok = torch.tensor([5, 650, 5, 5, 5, 5, -1, V], dtype=torch.int32).cuda()
        lp, lse, H, ids, tl = (t.cpu() for t in run_logp(K, x.cuda(), tok, 12))
        assert lse[0] == -inf and lp[0] == -inf and H[0] == 0 and (ids[0] == -1).all() and (tl[0] == -inf).all()
        assert lse[1] == 2.0 and lp[1] == 0 and H[1] == 0
        assert ids[1].tolist() == [650] + [-1] * 11 and tl[1, 0] == 0 and (tl[1, 1:] == -inf).all()
        for r in (2, 3):
            assert torch.isnan(torch.stack((lp[r], lse[r], H[r]))).all()
            assert (ids[r] == -1).all() and torch.isnan(tl[r]).all()
        assert ids[4].tolist() == list(range(12)) and abs(H[4] - math.log(V)) < 1e-4 and abs(lp[4] + math.log(V)) < 1e-4
        assert lp[5] == -inf and (ids[5, :10] >= 690).all() and (ids[5, 10:] == -1).all()
        assert lp[6] == 0 and torch.isfinite(lse[6]) and torch.isnan(lp[7]) and torch.isfinite(lse[7])
        out = run_logp(K, x.cuda()[2:3], torch.tensor([-1], dtype=torch.int32).cuda(), 1)
        assert torch.isnan(out[0]).all()  # a row without a distribution, token or not


def test_token_logprobs_parts_and_far_offsets(K):
    V = 1000
    far = 2 ** 31 + 8
    buf = torch.empty(far + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, V), (far, 1))
    x.copy_(torch.randn(2, V, generator=torch.Generator().manual_seed(9)))
    check_logp(K, x, 8)
    lse, H = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    K.kva_op_token_logprobs(x, lse=lse)
    K.kva_op_token_logprobs(x, entropy=H)
    _, a, b, _, _ = run_logp(K, x, torch.zeros(2, dtype=torch.int32, device="cuda"), 0)
    assert torch.equal(lse, a) and torch.equal(H, b)


# ------------------------------------------------------------------ together
def layer(K, W, x, h, S, q8, out, stream=None):
    """One DeltaNet mixer on exact inputs, the step to the next layer, the head and its scores."""
    n, T, nk, nv, d = W["dims"]
    s = dict(stream=stream)
    q, k, v = x[:, :, :nk], x[:, :, nk:2 * nk], x[:, :, 2 * nk:]
    K.kva_op_gdn_forward(q, k, v, W["gb"], S, out["S"], out["o"], scale=d ** -0.5, **s)
    K.kva_op_gemm(out["o"].view(n * T, nv * d), [W["o"]], out["y"], N=W["o"].shape[0], **s)
    if q8:  # the codes are the rows of a q8_0 matrix: logits^T = W_head y^T
        K.kva_op_add_rmsnorm(out["y"], h, W["g"], out["h"], out["codes"], scales=out["sc"], **s)
        K.kva_op_gemm_q8_0(W["head"], [out["codes"]], [out["sc"]], out["logits_t"], N=n * T, **s)
        return out["logits_t"].t()
    K.kva_op_add_rmsnorm(out["y"], h, W["g"], out["h"], out["u"], **s)
    K.kva_op_gemm(out["u"], [W["head"]], out["logits"], N=W["head"].shape[0], epilogue=K.EPI_STORE_F32, **s)
    return out["logits"]


def make_layer(K, n, T, seed=0):
    nk, nv, d, H, V = 2, 4, 64, 256, 1024
    gen = torch.Generator().manual_seed(seed)
    q, k, v, gb, S = make_gdn(n, T, nk, nv, d, torch.float16, seed=seed)
    x = torch.cat((q, k, v), 2)
    W = {"dims": (n, T, nk, nv, d), "gb": gb, "o": (torch.randn(H, nv * d, generator=gen) * 0.3).half().cuda(),
         "g": (torch.rand(H, generator=gen) + 0.5).cuda(), "head": (torch.randn(V, H, generator=gen) * 0.2).half().cuda()}
    h = torch.randn(n * T, H, generator=gen).cuda()
    e = lambda *s, t=torch.float16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    out = {"S": torch.empty_like(S), "o": e(n, T, nv, d), "y": e(n * T, H), "h": torch.empty_like(h), "u": e(n * T, H),
           "codes": e(n * T, H, t=torch.int8), "sc": e(H // 32, n * T), "logits": e(n * T, V, t=torch.float32),
           "logits_t": e(V, n * T)}
    return W, x, h, S, out


def layer_plain(W, x, h, S, tok):
    n, T, nk, nv, d = W["dims"]
    xd = f64(x)
    o, S1, _, _, _ = gdn_plain(xd[:, :, :nk], xd[:, :, nk:2 * nk], xd[:, :, 2 * nk:], f64(W["gb"]), f64(S), [T] * n, d ** -0.5)
    f = f64(h) + o.reshape(n * T, -1) @ f64(W["o"]).T
    u = f / np.sqrt((f * f).mean(1, keepdims=True) + 1e-6) * f64(W["g"])
    z = u @ f64(W["head"]).T
    m = z.max(1, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    return S1, f, u, z, z[np.arange(n * T), tok.cpu().numpy()] - lse


@pytest.mark.parametrize("n,T", [(1, 1), (3, 8), (2, 40)])
@pytest.mark.parametrize("q8", [False, True])
def test_a_layer_and_its_scores(K, n, T, q8):
    """The three operators around the framework's GEMMs, on a stream of their own and in a replayed graph.
    The logits' error: each of |W_head| |u| meets u's relative error, which is fp16's 2^-11 (a step of
    the q8_0 block with q8) plus the mixer path's (16-bit o and y: 2^-9 of their size over the row's RMS);
    8-fold standard deviation of a sum of independent roundings (2048 logits a row at most)."""
    W, x, h, S, out = make_layer(K, n, T)
    rows = n * T
    if q8 and rows % 8:
        pytest.skip("q8_0 matrices have rows in multiples of 8")
    tok = torch.randint(0, 1024, (rows,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    lp = torch.empty(rows, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    logits = layer(K, W, x, h, S, q8, out, stream=side)
    side.synchronize()
    scores = torch.empty(rows, 1024, dtype=logits.dtype, device="cuda")

    def rest(stream=None):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            scores.copy_(logits)
        K.kva_op_token_logprobs(scores, tok, lp, stream=stream)

    rest()
    torch.cuda.synchronize()
    S1, f, u, z, want = layer_plain(W, x, h, S, tok)
    assert np.linalg.norm(f64(out["S"]) - S1) <= 2.0 ** -14 * np.linalg.norm(S1)
    Wd = np.sqrt((f64(W["head"]) ** 2).sum(1)).max()
    rms = np.sqrt((u * u).mean())
    step = np.abs(u).max() / 127 / math.sqrt(12) if q8 else 0.0
    sd = Wd * math.sqrt((2.0 ** -9 * rms * 2) ** 2 + step ** 2) + (2.0 ** -11 * np.abs(z).max() if q8 else 0)
    assert (np.abs(f64(scores) - z) <= 8 * sd).all()
    assert (np.abs(f64(lp) - want) <= 16 * sd).all()
    # captured and replayed on other inputs
    first = (lp.clone(), out["S"].clone(), out["h"].clone())
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        layer(K, W, x, h, S, q8, out)
        rest()
    x0, h0 = x.clone(), h.clone()
    x.mul_(0.5)
    h.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    other = lp.clone()
    x.copy_(x0)
    h.copy_(h0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lp, first[0]) and torch.equal(out["S"], first[1]) and torch.equal(out["h"], first[2])
    assert not torch.equal(other, lp)


def test_calls_on_two_streams_do_not_meet(K):
    """The operators keep nothing between calls: the same work on two streams at once, and again."""
    sets = [make_layer(K, 2, 64, seed=i) for i in range(2)]
    want = []
    for W, x, h, S, out in sets:
        layer(K, W, x, h, S, False, out)
        torch.cuda.synchronize()
        want.append((out["logits"].clone(), out["S"].clone()))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (W, x, h, S, out), st in zip(sets, streams):
            layer(K, W, x, h, S, False, out, stream=st)
    torch.cuda.synchronize()
    for (W, x, h, S, out), (lg, S1) in zip(sets, want):
        assert torch.equal(out["logits"], lg) and torch.equal(out["S"], S1)
