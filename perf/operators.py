"""Three operators that run a hybrid gated-DeltaNet / attention stack exactly over several tokens,
measured against their plain forms: the gated delta rule with its readout for every token, the
residual addition with RMSNorm (16-bit or q8_0 output), and the log probabilities of given tokens.

`own = False`: elementary torch operations in 32 bits.  `own = True`: the entry points of
hybrid_deltanet_attention_kva_b200.  `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _gdn(name, n_seq, T, dtype, n_k=16, n_v=48, d=128, ragged=False):
    return {"name": name, "op": "gdn", "n_seq": n_seq, "T": T, "n_k": n_k, "n_v": n_v, "d": d,
            "dtype": dtype, "ragged": ragged}


def _norm(name, rows, n, x, h, out):
    return {"name": name, "op": "norm", "rows": rows, "n": n, "x": x, "h": h, "out": out}


def _logp(name, rows, V, dtype, n_top, pad=0):
    return {"name": name, "op": "logp", "rows": rows, "V": V, "dtype": dtype, "n_top": n_top, "pad": pad}


def listed():
    return [
        # one decoded token of one sequence through one DeltaNet layer: latency
        _gdn("gdn_token", 1, 1, "f16"),
        # one decoded token each of a served batch
        _gdn("gdn_batch_token", 64, 1, "bf16"),
        # drafted tokens of several sequences, checked in one pass; sequences end at different tokens
        _gdn("gdn_drafted", 16, 5, "bf16", ragged=True),
        # an exact ubatch of one prompt
        _gdn("gdn_ubatch", 1, 1024, "f16"),
        # exact ubatches of several prompts (the batch of the state-update workload)
        _gdn("gdn_batch_ubatch", 8, 1024, "bf16"),
        # the small geometry of the tests: 64-dim heads, odd length, padded batch
        _gdn("gdn_small_ragged", 5, 333, "f16", 2, 4, 64, True),
        # between two layers: the decoded token's residual
        _norm("norm_token", 1, 5120, "f16", "f32", "f16"),
        # between two layers: a ubatch's residual, normalised into q8_0 rows
        _norm("norm_ubatch_q8", 1024, 5120, "f32", "f32", "q8_0"),
        # a batch of ubatches with a 16-bit residual stream
        _norm("norm_batch", 8192, 5120, "bf16", "bf16", "bf16"),
        # the next token's probabilities for one sequence: latency
        _logp("logp_token", 1, 131072, "bf16", 8),
        # scoring a ubatch's own tokens (perplexity, greedy agreement)
        _logp("logp_ubatch", 1024, 131072, "bf16", 8),
        # an odd vocabulary in fp32, rows with padding behind them
        _logp("logp_odd_f32", 37, 50257, "f32", 20, 15),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdn", "gdn", "norm", "logp"])
    if op == "gdn":
        n_k, n_v, d = rng.choice([(16, 48, 128), (16, 48, 128), (4, 4, 128), (3, 6, 128), (2, 4, 64), (1, 5, 64)])
        T = _spread(rng, 1, 1500)
        n_seq = _spread(rng, 1, max(1, min(64, 8192 // T)))
        return {"op": "gdn", "n_seq": n_seq, "T": T, "n_k": n_k, "n_v": n_v, "d": d,
                "dtype": rng.choice(["f16", "bf16"]), "ragged": rng.random() < 0.4}
    if op == "norm":
        out = rng.choice(["f16", "bf16", "q8_0", "q8_0"])
        n = _spread(rng, 64, 16384) // 32 * 32 if out == "q8_0" else _spread(rng, 64, 16384) // 4 * 4
        return {"op": "norm", "rows": _spread(rng, 1, max(1, min(8192, (8192 * 5120) // n))), "n": n,
                "x": rng.choice(["f16", "bf16", "f32"]), "h": rng.choice(["f16", "bf16", "f32"]), "out": out}
    V = _spread(rng, 200, 262144)
    return {"op": "logp", "rows": _spread(rng, 1, max(1, min(4096, (1024 * 65536) // V))), "V": V,
            "dtype": rng.choice(["f16", "bf16", "f32"]), "n_top": rng.choice([0, 1, 5, 8, 20, 32]),
            "pad": rng.choice([0, 0, 1, 24])}


def _lens(case, seed):
    if not case["ragged"]:
        return [case["T"]] * case["n_seq"]
    g = torch.Generator().manual_seed(seed * 31 + 7)
    lens = torch.randint(0, case["T"] + 1, (case["n_seq"],), generator=g).tolist()
    lens[0] = case["T"]
    return lens


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed * 65537 + 11)

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev)

    s = {"case": dict(case)}
    if case["op"] == "gdn":
        n, T, nk, nv, d = (case[k] for k in ("n_seq", "T", "n_k", "n_v", "d"))
        dt = _DT[case["dtype"]]
        C = 2 * nk * d + nv * d
        x = torch.nn.functional.silu(randn(n, T, C))  # after the conv, [q | k | v] of a token
        qk = x[..., :2 * nk * d].view(n, T, 2 * nk, d)
        qk /= torch.sqrt((qk * qk).sum(-1, keepdim=True) + 1e-6)
        x = x.to(dt)
        s["q"] = x[..., :nk * d].view(n, T, nk, d)
        s["k"] = x[..., nk * d:2 * nk * d].view(n, T, nk, d)
        s["v"] = x[..., 2 * nk * d:].view(n, T, nv, d)
        s["lens"] = _lens(case, seed)
        A = torch.exp(torch.rand(nv, generator=g, device=dev) * 2.7)
        gate = -A[:, None] * torch.nn.functional.softplus(randn(n, nv, T) + 0.5 * randn(nv)[:, None])
        s["gb"] = torch.stack((gate, torch.sigmoid(randn(n, nv, T))), 1).contiguous()
        s["state"] = 0.1 * randn(n, nv, d, d)
        s["state_out"] = torch.empty_like(s["state"])
        s["out"] = torch.zeros(n, T, nv, d, dtype=dt, device=dev)
    elif case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        h = randn(rows, n)
        h[:, torch.randint(0, n, (8,), generator=g, device=dev)] *= 20.0  # outlier channels of a residual
        s["h"] = h.to(_DT[case["h"]])
        s["x"] = (0.3 * randn(rows, n)).to(_DT[case["x"]])
        s["gain"] = torch.rand(n, generator=g, device=dev) + 0.5
        s["h_out"] = torch.empty_like(s["h"])
        if case["out"] == "q8_0":
            s["codes"] = torch.empty(rows, n, dtype=torch.int8, device=dev)
            s["scales"] = torch.empty(n // 32, rows, dtype=torch.float16, device=dev)
        else:
            s["out"] = torch.empty(rows, n, dtype=_DT[case["out"]], device=dev)
    else:
        rows, V, n_top = case["rows"], case["V"], case["n_top"]
        buf = 2.5 * randn(rows, V + case["pad"])
        s["logits"] = buf.to(_DT[case["dtype"]])[:, :V]
        s["logits"][:, V // 3] = -math.inf  # a token that the program rules out
        s["tokens"] = torch.randint(0, V, (rows,), generator=g, device=dev, dtype=torch.int32)
        for k in ("logprob", "lse", "entropy"):
            s[k] = torch.empty(rows, device=dev)
        s["top_id"] = torch.empty(rows, n_top, dtype=torch.int32, device=dev)
        s["top_logprob"] = torch.empty(rows, n_top, device=dev)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_gdn(s):
    """S_t = e^g_t S_{t-1} + beta_t (v_t - e^g_t S_{t-1} k_t) k_t^T, o_t = S_t q_t, token by token."""
    c = s["case"]
    n, T, nk, nv, d = (c[k] for k in ("n_seq", "T", "n_k", "n_v", "d"))
    q, k, v = (s[i].float() for i in "qkv")
    dev = v.device
    kh = torch.arange(nv, device=dev) // (nv // nk)
    live = torch.arange(T, device=dev)[None, :] < torch.tensor(s["lens"], device=dev)[:, None]
    dec = torch.where(live[:, None, :], torch.exp(s["gb"][:, 0]), 1.0)
    beta = torch.where(live[:, None, :], s["gb"][:, 1], 0.0)
    S = s["state"].clone()
    o = torch.zeros(n, T, nv, d, device=dev)
    for t in range(T):
        kt = k[:, t, kh][:, :, None, :]
        S *= dec[:, :, t, None, None]
        u = beta[:, :, t, None] * (v[:, t] - (S * kt).sum(-1))
        S += u[..., None] * kt
        o[:, t] = (S * q[:, t, kh][:, :, None, :]).sum(-1)
    o = torch.where(live[:, :, None, None], o, 0.0)
    return {"out": o.to(s["out"].dtype), "state": S}


def _plain_norm(s):
    """h + x rounded to the stream's type, then RMSNorm of the stored row times the gain."""
    h = (s["h"].float() + s["x"].float()).to(s["h"].dtype)
    f = h.float()
    y = f / torch.sqrt((f * f).sum(-1, keepdim=True) / f.shape[-1] + 1e-6) * s["gain"]
    if "out" in s:
        return {"h": h, "out": y.to(s["out"].dtype)}
    b = y.view(y.shape[0], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    r = b / torch.where(d > 0, d, 1.0)
    codes = torch.sign(r) * torch.floor(r.abs() + 0.5)
    return {"h": h, "out": (codes * d.half().float()).half()}


def _plain_logp(s):
    """Log softmax at the given tokens, the entropy, and the largest entries in order."""
    x, n_top = s["logits"].float(), s["case"]["n_top"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    lp = x - lse
    ent = -torch.where(e > 0, e / z * lp, 0.0).sum(-1)
    top = torch.sort(x, dim=-1, descending=True, stable=True)
    return {"logprob": lp.gather(1, s["tokens"].long()[:, None])[:, 0], "lse": lse[:, 0], "entropy": ent,
            "top_id": top.indices[:, :n_top].int(), "top_logprob": top.values[:, :n_top] - lse}


def run(s):
    c = s["case"]
    if not own:
        return {"gdn": _plain_gdn, "norm": _plain_norm, "logp": _plain_logp}[c["op"]](s)
    import hybrid_deltanet_attention_kva_b200 as K
    if c["op"] == "gdn":
        K.kva_op_gdn_forward(s["q"], s["k"], s["v"], s["gb"], s["state"], s["state_out"], s["out"],
                             lens=s["lens"] if c["ragged"] else None)
        return {"out": s["out"], "state": s["state_out"]}
    if c["op"] == "norm":
        if "out" in s:
            K.kva_op_add_rmsnorm(s["x"], s["h"], s["gain"], s["h_out"], s["out"])
            return {"h": s["h_out"], "out": s["out"]}
        K.kva_op_add_rmsnorm(s["x"], s["h"], s["gain"], s["h_out"], s["codes"], scales=s["scales"])
        rows, n = s["codes"].shape
        return {"h": s["h_out"],  # the values that the codes stand for
                "out": s["codes"].view(rows, n // 32, 32) * s["scales"].t().unsqueeze(-1)}
    top = {"top_id": s["top_id"], "top_logprob": s["top_logprob"]} if c["n_top"] else {}
    K.kva_op_token_logprobs(s["logits"], s["tokens"], s["logprob"], lse=s["lse"], entropy=s["entropy"], **top)
    return {k: s[k] for k in ("logprob", "lse", "entropy", "top_id", "top_logprob")}


def work(case):
    if case["op"] == "gdn":
        n, T, nk, nv, d = (case[k] for k in ("n_seq", "T", "n_k", "n_v", "d"))
        if case["ragged"]:
            T = (T + (n - 1) * T / 2) / n  # the first sequence is whole, the others end anywhere
        tokens = n * T
        return {"bytes": tokens * (2 * nk * d * 2 + 2 * nv * d * 2 + 8 * nv) + 2 * n * nv * d * d * 4,
                # decay, S k, the rank-1 update and S q of every token and value head
                "flops": tokens * nv * 7 * d * d}
    if case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        size = {"f16": 2, "bf16": 2, "f32": 4, "q8_0": 1 + 2 / 32}
        return {"bytes": rows * n * (size[case["x"]] + 2 * size[case["h"]] + size[case["out"]]) + 4 * n,
                "flops": rows * n * (8 if case["out"] == "q8_0" else 5)}
    rows, V = case["rows"], case["V"]
    size = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
    return {"bytes": rows * (V * size + 16 + 8 * case["n_top"]), "flops": rows * V * 6}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gdn":
        n, T, nk, nv, d = (case[k] for k in ("n_seq", "T", "n_k", "n_v", "d"))
        q, k = (s[i].double().repeat_interleave(nv // nk, dim=2) for i in "qk")
        v = x = s["v"].double()
        g, b = s["gb"][:, 0].double(), s["gb"][:, 1].double()
        S = s["state"].double()
        out = torch.zeros(n, T, nv, d, dtype=torch.float64, device=x.device)
        for t in range(max(s["lens"])):
            on = torch.tensor([i for i, m in enumerate(s["lens"]) if t < m], device=x.device)
            kt, bt = k[on, t], b[on, :, t][..., None, None]
            # S e^g (I - beta k k^T) + beta v k^T, as matrix products
            M = S[on] * torch.exp(g[on, :, t])[..., None, None]
            Sk = torch.matmul(M, kt[..., None])
            new = M - bt * torch.matmul(Sk, kt[..., None, :]) + bt * torch.matmul(v[on, t][..., None], kt[..., None, :])
            S[on] = new
            out[on, t] = torch.matmul(new, q[on, t][..., None])[..., 0]
        return {"out": out, "state": S}
    if case["op"] == "norm":
        h = (s["h"].double() + s["x"].double()).to(s["h"].dtype)
        f = h.double()
        y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * s["gain"].double()
        if case["out"] != "q8_0":
            return {"h": h.double(), "out": y}
        b = y.reshape(y.shape[0], -1, 32)
        d = b.abs().amax(-1, keepdim=True) / 127.0
        return {"h": h.double(), "out": torch.trunc(b / d.clamp_min(1e-300) + 0.5 * torch.sign(b)) * d.half().double()}
    x, n_top = s["logits"].double(), case["n_top"]
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    ent = lse - torch.nan_to_num(p * x, nan=0.0, neginf=0.0).sum(-1)
    rows = torch.arange(x.shape[0], device=x.device)
    col = torch.arange(x.shape[1], device=x.device)
    lp, ids, vals = x[rows, s["tokens"].long()] - lse, [], []
    for _ in range(n_top):
        best = x.amax(-1)
        first = torch.where(x == best[:, None], col, x.shape[1]).amin(-1)
        ids.append(first)
        vals.append(best - lse)
        x[rows, first] = -math.inf
    none = x.new_zeros(x.shape[0], 0)
    return {"logprob": lp, "lse": lse, "entropy": ent,
            "top_id": torch.stack(ids, 1).int() if ids else none.int(),
            "top_logprob": torch.stack(vals, 1) if vals else none}
