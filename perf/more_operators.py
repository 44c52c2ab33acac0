"""Linear attention with one decay for each head, and the rotary positions of its queries and keys: inputs, plain forms
and 64-bit results.

Per (sequence, head), with an fp32 state S [d, d] and a log-decay g (of each token, or one for the whole head),

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = S_t^T q_t.

  prompt  the chunked form over packed documents (cu_seqlens), with incoming and outgoing states
  token   the recurrent form: one token for each listed slot of a state pool, in place
  rope    positions rotated into q and k before either: pairs side by side or half a head apart, the whole head or its
          first part, plain or scaled for long contexts

q and k may have fewer heads than v (each shared by a run of v's heads).  `fused` adds what stands on either side of the
recurrence in a layer: L2-normalised q and k, and the gated normalisation of the output.
"""
import math
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64


def listed():
    return [
        # a short question to one model layer: the latency of a small prompt
        _prompt("prompt_t77_h16", N=1, T=77, H=16, fused=True),
        # the benchmark's prompt, with everything that stands around the recurrence
        _prompt("prompt_t4096_h16", N=1, T=4096, H=16, fused=True),
        # an ordinary packed batch that continues earlier documents
        _prompt("prompt_packed8_t33000_h32", N=8, T=33000, H=32, S0=True),
        # one long document, each head with a decay of its own that is the same for all tokens: the largest
        _prompt("prompt_t65536_h16", N=1, T=65536, H=16, decay="head"),
        # single precision, a smaller head, q and k shared by all heads, ragged documents
        _prompt("prompt_fp32_d64_t1501_h5", N=6, T=1501, H=5, Hqk=1, d=64, dtype="fp32", S0=True),
        # one request's next token
        _token("token_n1_h16", N=1, H=16, fused=True),
        # the decode benchmark's batch
        _token("token_n256_h32", N=256, H=32, fused=True),
        # single precision, a smaller head, shared q and k, a constant decay, an odd batch
        _token("token_fp32_d64_n17_h6", N=17, H=6, Hqk=2, d=64, dtype="fp32", decay="head"),
        # the next token of 64 requests, each at its own position
        _rope("rope_t64_h32", T=64, Hq=32, Hk=32, d=128, rot=128, far=30000),
        # the benchmark's prompt
        _rope("rope_t4096_h16", T=4096, Hq=16, Hk=16, d=128, rot=128, packed=True),
        # a long document behind an earlier part of it, half of each head rotated in pairs, scaled for a long context
        _rope("rope_t65536_h16", T=65536, Hq=16, Hk=16, d=128, rot=64, interleaved=True, packed=True, far=1000000, scaled=True),
        # single precision, a width and a part that fill no vector, one shared key head, an odd number of tokens
        _rope("rope_fp32_d80_t1001_h6", T=1001, Hq=6, Hk=1, d=80, rot=20, dtype="fp32", far=5000),
    ]


def _prompt(name, N, T, H, Hqk=None, d=128, dtype="bf16", decay="token", fused=False, S0=False):
    return {"name": name, "op": "prompt", "N": N, "T": T, "H": H, "Hqk": Hqk or H, "d": d, "dtype": dtype, "decay": decay, "fused": fused, "S0": S0}


def _token(name, N, H, Hqk=None, d=128, dtype="bf16", decay="token", fused=False):
    return {"name": name, "op": "token", "N": N, "H": H, "Hqk": Hqk or H, "d": d, "dtype": dtype, "decay": decay, "fused": fused}


def _rope(name, T, Hq, Hk, d, rot, dtype="bf16", interleaved=False, packed=False, far=0, scaled=False):
    return {"name": name, "op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "dtype": dtype, "interleaved": interleaved,
            "packed": packed, "far": far, "scaled": scaled}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    """(heads of v, heads of q and k): mostly the same, else a divisor."""
    H = rng.randint(1, most)
    return H, H if rng.random() < 0.7 else rng.choice([h for h in range(1, H + 1) if H % h == 0])


def draw(rng):
    op = rng.choice(["prompt", "prompt", "token", "rope"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "rope":
        d = rng.choice([128, 128, 64, 16, 80, 96, 256])
        Hq, Hk = _heads(rng, 32)
        T = min(_log_int(rng, 1, 65536), 65536 * 32 * 128 // ((Hq + Hk) * d))
        return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]), "dtype": dtype,
                "interleaved": rng.random() < 0.5, "packed": rng.random() < 0.5, "far": rng.choice([0, 5000, 1000000]), "scaled": rng.random() < 0.5}
    d = rng.choice([128, 128, 128, 64, 16])
    H, Hqk = _heads(rng, 32)
    case = {"op": op, "H": H, "Hqk": Hqk, "d": d, "dtype": dtype, "decay": rng.choice(["token", "token", "head"]), "fused": rng.random() < 0.5}
    if op == "token":
        return {**case, "N": _log_int(rng, 1, 256)}
    T = _log_int(rng, 1, 65536)
    T = max(1, min(T, (65536 * 16 if dtype == "bf16" else 65536) // H))
    return {**case, "T": T, "N": _log_int(rng, 1, min(T, 64)), "S0": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"prompt": _prepare_prompt, "token": _prepare_token, "rope": _prepare_rope}[case["op"]](case, seed)


def _cuts(N, T, seed):
    """Ends of N documents of T tokens in all, at random places: a document may be empty."""
    r = random.Random(seed * 7919 + 17)
    return [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]


def _recurrence(case, rows, g):
    """q, k, v, the decay and what the fused steps need, for `rows` tokens."""
    H, Hqk, d, dt = case["H"], case["Hqk"], case["d"], _dtype(case)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    q, k = randn(rows, Hqk, d), randn(rows, Hqk, d)
    if not case["fused"]:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    if case["decay"] == "head":  # 1 - 2^-5 for the first head to 1 - 2^-12 for the last
        power = -5.0 - 7.0 * torch.arange(H, device="cuda", dtype=torch.float64) / max(1, H - 1)
        decay = torch.log1p(-torch.exp2(power)).float()
    else:  # from tokens that forget nearly everything to tokens that keep nearly all
        decay = -torch.exp(1.2 * randn(rows, H) - 2.5)
    s = {"op": case["op"], "fused": case["fused"], "q": q.to(dt), "k": k.to(dt), "v": randn(rows, H, d).to(dt), "g": decay,
         "o": torch.empty((rows, H, d), dtype=dt, device="cuda")}
    if case["fused"]:
        s.update(z=randn(rows, H, d).to(dt), weight=1.0 + 0.1 * randn(d))
    return s


def _prepare_prompt(case, seed):
    g = _gen(seed)
    N, T, H, d = case["N"], case["T"], case["H"], case["d"]
    cuts = _cuts(N, T, seed)
    s = _recurrence(case, T, g)
    # the plain form's view of the same documents: their chunks, and which of them follow one another
    doc, start = [], []
    for n in range(N):
        begins = range(cuts[n], cuts[n + 1], CHUNK)
        doc += [n] * len(begins)
        start += list(begins)
    doc = torch.tensor(doc, device="cuda")
    cu = torch.tensor(cuts, device="cuda")
    rows = torch.tensor(start, device="cuda")[:, None] + torch.arange(CHUNK, device="cuda")
    there = rows < cu[doc + 1][:, None]
    s.update(cu=cu.to(torch.int32), rows=rows.clamp_max(T - 1), there=there, flat=there.flatten().nonzero()[:, 0], doc=doc,
             S0=0.1 * torch.randn((N, H, d, d), generator=g, device="cuda") if case["S0"] else None,
             S=torch.empty((N, H, d, d), device="cuda"))
    return s


def _prepare_token(case, seed):
    g = _gen(seed)
    N, H, d = case["N"], case["H"], case["d"]
    total = N + N // 4 + 1  # a pool a quarter larger than the batch, its slots in no order
    s = _recurrence(case, N, g)
    s.update(slots=_i32(random.Random(seed * 31 + 5).sample(range(total), N)), S=torch.randn((total, H, d, d), generator=g, device="cuda"))
    return s


def _frequencies(rot, scaled):
    """(radians a position of each pair, factor of the rotated values).  Scaled: pairs that turn less than once in the
    original 4096 positions are slowed down 16 times, those that turn over 32 times kept, those between blended, and the
    values grow by 0.1 ln 16 + 1."""
    pair = torch.arange(rot // 2, dtype=torch.float64)
    plain = 10000.0 ** (-2.0 * pair / rot)
    if not scaled:
        return plain, 1.0
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(0.0, math.floor(at(32.0))), min(rot - 1.0, math.ceil(at(1.0)))
    slow = ((pair - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return plain * (1 - slow) + plain / 16 * slow, 0.1 * math.log(16.0) + 1.0


def _prepare_rope(case, seed):
    g, r = _gen(seed), random.Random(seed * 17 + 3)
    T, d, dt = case["T"], case["d"], _dtype(case)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if case["packed"]:  # a document's tokens one after another, behind `far` earlier ones at most
        positions = torch.arange(T, device="cuda") + r.randint(case["far"] // 2, case["far"])
    else:  # every row a request of its own
        positions = torch.randint(0, max(1, case["far"]), (T,), generator=g, device="cuda")
    freq, scale = _frequencies(case["rot"], case["scaled"])
    q, k = randn(T, case["Hq"], d).to(dt), randn(T, case["Hk"], d).to(dt)
    return {"op": "rope", "q": q, "k": k, "positions": positions.to(torch.int32), "freq": freq.cuda(), "scale": scale, "interleaved": case["interleaved"],
            "q_out": torch.empty_like(q), "k_out": torch.empty_like(k)}


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"prompt": _plain_prompt, "token": _plain_token, "rope": _plain_rope}[s["op"]](s)


def _own(s):
    from gated_delta_rule_27_gb300 import libkda
    if s["op"] == "rope":
        if "steps" not in s:  # the table that a model keeps
            s["steps"] = libkda.rope_steps(s["freq"])
        libkda.kda_rope(s["q"], s["k"], s["positions"], s["steps"], s["q_out"], s["k_out"], interleaved=s["interleaved"], scale=s["scale"])
        return {"q": s["q_out"], "k": s["k_out"]}
    fusion = dict(qk_l2norm=True, qk_eps=EPS, out_gate=s["z"], out_weight=s["weight"], out_eps=EPS) if s["fused"] else {}
    if s["op"] == "token":
        libkda.kda_linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], s["o"], seq_idx=s["slots"], **fusion)
        return {"o": s["o"], "S": s["S"]}
    if "workspace" not in s:  # kept from call to call, as for the other prefill
        s["workspace"] = libkda.new_linear_workspace(s["q"], s["v"], s["cu"])
    libkda.kda_linear_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"], s["o"], S0=s["S0"], S_final=s["S"], workspace=s["workspace"], **fusion)
    return {"o": s["o"], "S": s["S"]}


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _qkv(s):
    """q, k, v in single precision, q and k as the recurrence takes them, one for each head of v."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["fused"]:
        q, k = _unit(q), _unit(k)
    shared = v.shape[1] // q.shape[1]
    if shared > 1:
        q, k = q.repeat_interleave(shared, 1), k.repeat_interleave(shared, 1)
    return q, k, v


def _finish(s, o):
    if s["fused"]:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"] * torch.sigmoid(s["z"].float())
    return o.to(s["o"].dtype)


def _plain_prompt(s):
    T, H, d = s["v"].shape
    there, doc, cu = s["there"], s["doc"], s["cu"].long()
    zero = torch.zeros((), device="cuda")
    q, k, v = (torch.where(there[..., None, None], x[s["rows"]], zero).transpose(1, 2) for x in _qkv(s))  # [C, H, 64, d]
    g = s["g"].expand(T, H)[s["rows"]].double()
    b = torch.where(there[..., None], g, zero.double()).cumsum(1).transpose(1, 2)  # [C, H, 64], sums of many logarithms in 64 bits
    causal = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device="cuda").tril()
    within = torch.where(causal, b[..., :, None] - b[..., None, :], -math.inf).float().exp()
    local = torch.matmul((k * (b[..., -1:] - b).float().exp()[..., None]).transpose(-1, -2), v)  # what a chunk adds by its end
    total = b[..., -1].cumsum(0)  # [C, H]
    # a chunk's state: what the chunks before it in its document have added, decayed since, and the incoming state
    C = len(doc)
    before = (doc[:, None] == doc) & torch.ones((C, C), dtype=torch.bool, device="cuda").tril(-1)
    reach = torch.where(before, (total - b[..., -1]).t()[:, :, None] - total.t()[:, None, :], -math.inf).float().exp()  # [H, C, C]
    S = torch.matmul(reach, local.transpose(0, 1).flatten(2)).view(H, C, d, d).transpose(0, 1)
    S0 = s["S0"] if s["S0"] is not None else torch.zeros_like(s["S"])
    first = (doc[:, None] == doc).int().argmax(1)
    S = S + (total - b[..., -1] - (total - b[..., -1])[first]).float().exp()[..., None, None] * S0[doc]
    o = b.float().exp()[..., None] * torch.matmul(q, S) + torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * within, v)
    end = S0.clone()
    last = torch.ones(C, dtype=torch.bool, device="cuda")
    last[:-1] = doc[1:] != doc[:-1]
    end[doc[last]] = b[last][..., -1].float().exp()[..., None, None] * S[last] + local[last]
    o = o.transpose(1, 2).flatten(0, 1)[s["flat"]]
    return {"o": _finish(s, o), "S": end}


def _plain_token(s):
    q, k, v = _qkv(s)
    slots = s["slots"].long()
    S = s["g"].exp().expand(v.shape[:2])[..., None, None] * s["S"][slots] + k[..., None] * v[..., None, :]
    s["S"][slots] = S
    return {"o": _finish(s, torch.matmul(q[..., None, :], S)[..., 0, :]), "S": s["S"]}


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = (s["scale"] * angle.cos()).float()[:, None], (s["scale"] * angle.sin()).float()[:, None]
    return {"q": _rotated(s["q"], cos, sin, s["interleaved"]), "k": _rotated(s["k"], cos, sin, s["interleaved"])}


def _rotated(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a.float(), b.float()
    a, b = (a * cos - b * sin).to(x.dtype), (b * cos + a * sin).to(x.dtype)
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    el = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":  # q and k once each way, the positions
        n = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": n * case["d"] * 2 * el + case["T"] * 4, "flops": n * case["rot"] * 3}
    H, Hqk, d = case["H"], case["Hqk"], case["d"]
    rows = case["T"] if case["op"] == "prompt" else case["N"]
    bytes_ = rows * d * el * (2 * Hqk + H * (3 if case["fused"] else 2)) + 4 * H * (rows if case["decay"] == "token" else 1)
    states = case["N"] * (2 if case["op"] == "token" or case["S0"] else 1)  # read and written, or only written
    return {"bytes": bytes_ + states * H * d * d * 4, "flops": rows * H * d * d * 4}


# ---------------------------------------------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "token": _exact_token, "rope": _exact_rope}[case["op"]](case, s)


def _exact_rows(case, s, name, at):
    x = s[name][at].double()
    if name in ("q", "k"):
        if case["fused"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)
        of = torch.arange(case["H"], device="cuda") // (case["H"] // case["Hqk"])
        x = x[:, of]
    return x


def _exact_finish(case, s, o):
    if case["fused"]:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"].double() / (1 + torch.exp(-s["z"].double()))
    return o


def _exact_prompt(case, s):
    """Token by token, all documents that are long enough at once."""
    H, d = case["H"], case["d"]
    cu = s["cu"].tolist()
    order = sorted(range(case["N"]), key=lambda n: cu[n] - cu[n + 1])
    S = torch.zeros((case["N"], H, d, d), dtype=torch.float64, device="cuda") if s["S0"] is None else s["S0"].double()
    S = S[order]
    lengths, begin = [cu[n + 1] - cu[n] for n in order], torch.tensor([cu[n] for n in order], device="cuda")
    o = torch.zeros((case["T"], H, d), dtype=torch.float64, device="cuda")
    live = case["N"]
    some = max(1, 2 ** 24 // (case["N"] * H * d))  # as many steps' rows as are taken to 64 bits at once
    for t0 in range(0, lengths[0], some):
        at = (begin + torch.arange(t0, min(lengths[0], t0 + some), device="cuda")[:, None]).clamp_max(case["T"] - 1)
        q, k, v = (_exact_rows(case, s, x, at.flatten()).view(*at.shape, H, d) for x in ("q", "k", "v"))
        decay = torch.exp(s["g"].double())
        decay = decay.expand(*at.shape, H) if decay.dim() == 1 else decay[at]
        for i in range(len(at)):
            while lengths[live - 1] <= t0 + i:
                live -= 1
            S[:live] = decay[i, :live, :, None, None] * S[:live] + k[i, :live, :, :, None] * v[i, :live, :, None, :]
            o[at[i, :live]] = torch.matmul(q[i, :live, :, None, :], S[:live])[..., 0, :]
    end = torch.empty_like(S)
    end[order] = S
    return {"o": _exact_finish(case, s, o), "S": end}


def _exact_token(case, s):
    rows = torch.arange(case["N"], device="cuda")
    q, k, v = (_exact_rows(case, s, x, rows) for x in ("q", "k", "v"))
    S, o = s["S"].double(), torch.zeros_like(v)
    for i, slot in enumerate(s["slots"].tolist()):
        g = s["g"][i] if s["g"].dim() == 2 else s["g"]
        S[slot] = torch.exp(g.double())[:, None, None] * S[slot] + k[i, :, :, None] * v[i, :, None, :]
        o[i] = (S[slot] * q[i, :, :, None]).sum(-2)
    return {"o": _exact_finish(case, s, o), "S": S}


def _exact_rope(case, s):
    """Each pair as a complex number, turned by its angle less the whole turns."""
    rot, turns = case["rot"], s["positions"].double()[:, None] * (s["freq"] / (2 * math.pi))
    turn = torch.polar(torch.full_like(turns, s["scale"]), 2 * math.pi * (turns - torch.floor(turns)))[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        x[..., :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
        out[name] = x
    return out
