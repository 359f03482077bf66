"""Refusals of the several-token operators (gdn_forward, add_rmsnorm, token_logprobs): every bad
argument is answered on the host before anything is enqueued (CPU only, no device memory)."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import hybrid_deltanet_attention_kva_b200 as K
from hybrid_deltanet_attention_kva_b200 import kva as kmod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = K.KVA_ERR_INVALID_ARG, K.KVA_ERR_UNSUPPORTED
TOO_LARGE, ALIGNMENT = K.KVA_ERR_TOO_LARGE, K.KVA_ERR_ALIGNMENT


def _gdn(**kw):
    a = K.KvaGdnForwardArgs(dtype=K.KVA_BF16, n_seq=2, T=7, n_k=2, n_v=4, d=64, q=16, k=16, v=16, gb=16,
                            state_in=16, state_out=16, out=16, q_ld=128, q_seq=896, k_ld=128, k_seq=896,
                            v_ld=256, v_seq=1792, out_ld=256, out_seq=1792, scale=1.0)
    for n, x in kw.items():
        setattr(a, n, x)
    return K.lib().kva_op_gdn_forward(C.byref(a), None, None)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=K.KVA_F32), INVALID), (dict(dtype=7), INVALID), (dict(n_seq=-1), INVALID), (dict(T=-1), INVALID),
    (dict(n_k=0), INVALID), (dict(n_v=3), INVALID), (dict(d=96), UNSUPPORTED), (dict(n_seq=257), TOO_LARGE),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(gb=None), INVALID),
    (dict(out=None), INVALID), (dict(state_in=None), INVALID), (dict(state_out=None), INVALID),
    (dict(T=0, state_out=None), INVALID), (dict(q_ld=120), INVALID), (dict(v_ld=248), INVALID),
    (dict(out_ld=0), INVALID), (dict(k_seq=-8), INVALID),
    (dict(out_seq=0), INVALID),                       # the sequences' outputs share rows
    (dict(out_seq=256, out_ld=256), INVALID),
    (dict(q_ld=132), ALIGNMENT), (dict(k_seq=900), ALIGNMENT), (dict(q=8), ALIGNMENT), (dict(out=24), ALIGNMENT),
    (dict(state_in=20), ALIGNMENT), (dict(gb=18), ALIGNMENT),
    (dict(lens=(C.c_int32 * 2)(7, 8)), INVALID), (dict(lens=(C.c_int32 * 2)(-1, 7)), INVALID),
])
def test_gdn_forward_refuses(change, want):
    assert _gdn(**change) == want


def test_gdn_forward_nothing_to_do():
    assert K.lib().kva_op_gdn_forward(None, None, None) == INVALID
    assert _gdn(n_seq=0) == K.KVA_OK


def test_gdn_wait_timeout_test_refuses():
    """The test of the failure path takes one sequence of more than two runs, and a status to report to."""
    def call(err=16, **kw):
        a = K.KvaGdnForwardArgs(dtype=K.KVA_BF16, n_seq=1, T=33, n_k=2, n_v=4, d=64, q=16, k=16, v=16, gb=16,
                                state_in=16, state_out=16, out=16, q_ld=128, k_ld=128, v_ld=256, out_ld=256, scale=1.0)
        for n, x in kw.items():
            setattr(a, n, x)
        return K.lib().kva_test_gdn_forward_wait_timeout(C.byref(a), err, None)
    for bad in (dict(err=None), dict(T=32), dict(n_seq=2), dict(n_seq=0), dict(lens=(C.c_int32 * 1)(33)), dict(q=None)):
        assert call(**bad) == INVALID
    assert K.lib().kva_test_gdn_forward_wait_timeout(None, 16, None) == INVALID


def _norm(**kw):
    a = dict(x=16, x_dtype=K.KVA_F16, ldx=64, h=32, h_out=48, h_dtype=K.KVA_F32, ldh=64, g=64, out=80,
             out_dtype=K.KVA_BF16, ldo=64, scales=None, rows=3, n=64, eps=1e-6)
    a.update(kw)
    return K.lib().kva_op_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), INVALID), (dict(n=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x_dtype=K.KVA_Q8_0), INVALID), (dict(h_dtype=9), INVALID), (dict(out_dtype=K.KVA_F32), INVALID),
    (dict(n=16388, ldx=16388, ldh=16388, ldo=16388), UNSUPPORTED), (dict(x=None), INVALID), (dict(h=None), INVALID),
    (dict(h_out=None), INVALID), (dict(g=None), INVALID), (dict(out=None), INVALID), (dict(ldx=60), INVALID),
    (dict(ldh=0), INVALID), (dict(ldo=60), INVALID), (dict(n=62), ALIGNMENT), (dict(ldx=66), ALIGNMENT),
    (dict(h=36), ALIGNMENT), (dict(g=68), ALIGNMENT), (dict(scales=2), INVALID),
    (dict(out_dtype=K.KVA_Q8_0), INVALID), (dict(out_dtype=K.KVA_Q8_0, scales=3), ALIGNMENT),
    (dict(out_dtype=K.KVA_Q8_0, scales=2, ldo=68), ALIGNMENT),
    (dict(out_dtype=K.KVA_Q8_0, scales=2, n=48), UNSUPPORTED),
])
def test_add_rmsnorm_refuses(change, want):
    assert _norm(**change) == want
    assert _norm(rows=0) == K.KVA_OK


def _logp(**kw):
    a = dict(logits=16, dtype=K.KVA_BF16, ld=100, rows=2, V=100, tokens=16, logprob=16, lse=16, entropy=16, n_top=3,
             top_id=16, top_logprob=16)
    a.update(kw)
    return K.lib().kva_op_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), INVALID), (dict(V=0), INVALID), (dict(V=2 ** 30 + 1, ld=2 ** 31), TOO_LARGE), (dict(n_top=-1), INVALID), (dict(n_top=33), TOO_LARGE),
    (dict(dtype=K.KVA_Q8_0), INVALID), (dict(logits=None), INVALID), (dict(ld=99), INVALID),
    (dict(tokens=None), INVALID), (dict(logprob=None), INVALID), (dict(top_id=None), INVALID),
    (dict(top_logprob=None), INVALID), (dict(logits=17), ALIGNMENT), (dict(dtype=K.KVA_F32, logits=18), ALIGNMENT),
    (dict(lse=18), ALIGNMENT), (dict(top_id=17), ALIGNMENT),
    (dict(tokens=None, logprob=None, lse=None, entropy=None, n_top=0), INVALID),
])
def test_token_logprobs_refuses(change, want):
    assert _logp(**change) == want
    assert _logp(rows=0) == K.KVA_OK


def test_binding_refuses_cpu_tensors_and_wrong_shapes(monkeypatch):
    q, v = torch.zeros(1, 3, 2, 64, dtype=torch.float16), torch.zeros(1, 3, 4, 64, dtype=torch.float16)
    gb, S = torch.zeros(1, 2, 4, 3), torch.zeros(1, 4, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        K.kva_op_gdn_forward(q, q, v, gb, S, S, v)
    with pytest.raises(ValueError, match="CUDA"):
        K.kva_op_add_rmsnorm(S[0, 0], S[0, 0], gb, S[0, 0], q[0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        K.kva_op_token_logprobs(S[0, 0])
    # the binding's own shape checks, without a device: nothing may reach the library
    monkeypatch.setattr(kmod, "_one_device", lambda *a: (0, 0))
    for bad in (dict(lens=[4]), dict(lens=[-1]), dict(lens=[1, 1]), dict(lens=[2 ** 32]), dict(gb=gb[:, :1]),
                dict(state_in=S.half()), dict(state_out=S.transpose(2, 3)), dict(v=v.bfloat16()),
                dict(k=q[..., ::2]), dict(k=q.transpose(1, 2)), dict(out=v[:, :2])):
        a = dict(q=q, k=q, v=v, gb=gb, state_in=S, state_out=S.clone(), out=v.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            K.kva_op_gdn_forward(**a)
    x, y = torch.zeros(3, 64), torch.zeros(3, 64, dtype=torch.float16)
    c, sc, g = torch.zeros(3, 64, dtype=torch.int8), torch.zeros(2, 3, dtype=torch.float16), torch.zeros(64)
    for bad in (dict(scales=sc), dict(out=c), dict(out=c, scales=sc.t()), dict(g=g[:32]), dict(h_out=y),
                dict(x=x.t().contiguous().t()), dict(out=y[:2]), dict(g=g.half()),
                dict(h_out=torch.zeros(3, 128)[:, :64])):
        a = dict(x=x, h=x, g=g, h_out=x, out=y)
        a.update(bad)
        with pytest.raises(ValueError):
            K.kva_op_add_rmsnorm(**a)
    t, f = torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    for bad in (dict(tokens=t.long(), logprob=f), dict(tokens=t), dict(lse=f[:2]), dict(entropy=f.double()),
                dict(top_id=t.view(3, 1)), dict(top_id=t.view(3, 1), top_logprob=torch.zeros(3, 2))):
        with pytest.raises(ValueError):
            K.kva_op_token_logprobs(x, **bad)


def test_binding_refuses_sizes_above_int32(monkeypatch):
    """The C entries take int32 sizes: 2^32 + 3 rows may not pass as 3.  (Tensors without memory; nothing
    may reach the library.)"""
    monkeypatch.setattr(kmod, "_one_device", lambda *a: (0, 0))

    def reached(*a):
        raise AssertionError("reached the library")
    monkeypatch.setattr(kmod, "_call_on", reached)
    big, e = 2 ** 32 + 3, torch.empty
    f16, f32 = dict(dtype=torch.float16, device="meta"), dict(dtype=torch.float32, device="meta")
    for rows, n in ((big, 4), (1, big)):
        with pytest.raises(ValueError, match="above"):
            K.kva_op_add_rmsnorm(e(rows, n, **f16), e(rows, n, **f32), e(n, **f32), e(rows, n, **f32), e(rows, n, **f16))
        with pytest.raises(ValueError, match="above"):
            K.kva_op_token_logprobs(e(rows, n, **f16), lse=e(rows, **f32))
    for T, nk, nv in ((big, 1, 1), (1, big, big), (1, 1, big)):
        q, v, S = e(1, T, nk, 64, **f16), e(1, T, nv, 64, **f16), e(1, nv, 64, 64, **f32)
        with pytest.raises(ValueError, match="above"):
            K.kva_op_gdn_forward(q, q, v, e(1, 2, nv, T, **f32), S, S, v)
    with pytest.raises(ValueError, match="sequences|above"):
        q = e(big, 1, 1, 64, **f16)
        K.kva_op_gdn_forward(q, q, q, e(big, 2, 1, 1, **f32), e(big, 1, 64, 64, **f32), e(big, 1, 64, 64, **f32), q)


def test_argument_struct_and_limits_match_the_c_compiler(tmp_path):
    fields = [n for n, _ in K.KvaGdnForwardArgs._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "kva_ops.h"', "int main(void){",
           'printf("size %zu\\n", sizeof(kva_gdn_forward_args));',
           'printf("seq %d\\n", KVA_GDN_MAX_SEQ);', 'printf("top %d\\n", KVA_LOGPROB_MAX_TOP);']
    src += [f'printf("{f} %zu\\n", offsetof(kva_gdn_forward_args, {f}));' for f in fields] + ["return 0;}"]
    (tmp_path / "a.c").write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")],
                   check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    assert int(got.pop("size")) == C.sizeof(K.KvaGdnForwardArgs)
    assert int(got.pop("seq")) == K.GDN_MAX_SEQ and int(got.pop("top")) == K.LOGPROB_MAX_TOP
    assert {n: int(o) for n, o in got.items()} == {f: getattr(K.KvaGdnForwardArgs, f).offset for f in fields}
