"""Workloads of the prompt path: causal attention over packed prompts and decayed linear attention.

Two operators stand beside the video layer's two branches for the tokens that come as text, one after
another: causal softmax attention with grouped heads over packed sequences (with its gradients, and with
single new tokens against a cache of keys and values), and linear attention whose state decays by a factor
of each head (whole prompts, single tokens, and its gradients). Each case below is one pass of one of them.

``run`` computes a case in its plain form, torch operations in 32 bits, or, where ``own`` is true, by the
calls of ``frame_level_delta_b200.vda``. ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
# lens: the sequences' lengths, in packed order. For "attention_tokens" they are the lengths of the caches
# that N single new tokens attend to, each in a row of `room` slots.
def listed():
    return [
        # one text prompt as the clips of this repository carry it (512 tokens, 24 heads): latency counts
        {"name": "attention_text", "op": "attention", "Hq": 24, "Hkv": 24, "d": 128, "lens": "512"},
        # a batch of prompts of users, packed, three query heads to a key head
        {"name": "attention_packed", "op": "attention", "Hq": 24, "Hkv": 8, "d": 128,
         "lens": "1,37,128,129,255,511,512,640,777,901,1024,1111,1280,1333,1499,64"},
        # one long document
        {"name": "attention_long", "op": "attention", "Hq": 32, "Hkv": 8, "d": 128, "lens": "8191"},
        # serving: one new token for each of 48 requests against caches of very different lengths
        {"name": "attention_tokens", "op": "attention_tokens", "Hq": 32, "Hkv": 8, "d": 128, "room": 8192,
         "lens": ",".join(str(1 + (i * 2741) % 8192) for i in range(48))},
        # a small training step of 64-channel heads on ragged sequences
        {"name": "attention_train_small", "op": "attention_train", "Hq": 8, "Hkv": 8, "d": 64,
         "lens": "300,64,1,212,447"},
        # a training step on longer sequences with grouped heads
        {"name": "attention_train", "op": "attention_train", "Hq": 24, "Hkv": 8, "d": 128, "lens": "4096,2500,3999"},
        # the same text prompt through the linear operator
        {"name": "decay_text", "op": "decay", "H": 24, "d": 128, "lens": "512"},
        # packed prompts, ragged, 64-channel heads
        {"name": "decay_packed", "op": "decay", "H": 24, "d": 64,
         "lens": "1,37,128,129,255,511,512,640,777,901,1024,1111,1280,1333,1499,64"},
        # one long document
        {"name": "decay_long", "op": "decay", "H": 24, "d": 128, "lens": "11300"},
        # serving: one new token of one request, then of 160 requests
        {"name": "decay_step_one", "op": "decay_step", "H": 24, "d": 128, "N": 1},
        {"name": "decay_step_batch", "op": "decay_step", "H": 24, "d": 128, "N": 160},
        # a training step
        {"name": "decay_train", "op": "decay_train", "H": 24, "d": 128, "lens": "2048,1500,3333,700"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_tokens", "attention_train", "decay", "decay",
                     "decay_step", "decay_train"])
    d = rng.choice([64, 128, 128])
    if op == "decay_step":
        return {"op": op, "H": rng.randint(1, 32), "d": d, "N": _log_int(rng, 1, 160)}
    if op == "attention_tokens":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
        N, room = _log_int(rng, 1, 48), _log_int(rng, 64, 8192)
        return {"op": op, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "room": room,
                "lens": ",".join(str(rng.randint(1, room)) for _ in range(N))}
    train = op.endswith("train")
    N = _log_int(rng, 1, 24)
    top = _log_int(rng, 16, (3000 if train else 6000) // (1 if N < 4 else 3))
    lens = ",".join(str(rng.randint(1, top)) for _ in range(N))
    if op.startswith("decay"):
        return {"op": op, "H": rng.randint(1, 24), "d": d, "lens": lens}
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3])
    return {"op": op, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "lens": lens}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------ what a program has in hand
def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    def bf(x):
        return x.to(torch.bfloat16)

    op, d = case["op"], case["d"]
    s = {"op": op}
    if op == "decay_step":
        N, H = case["N"], case["H"]
        s.update(Q=bf(unit(randn(N, H, d))), K=bf(unit(randn(N, H, d))), V=bf(randn(N, H, d)), S=randn(N, H, d, d))
        s["log_decay"] = _slopes(H)
        return s
    lens = _lens(case)
    T, N = sum(lens), len(lens)
    if op.startswith("decay"):
        H = case["H"]
        s.update(Q=bf(unit(randn(T, H, d))), K=bf(unit(randn(T, H, d))), V=bf(randn(T, H, d)), cu=_cu(lens),
                 longest=max(lens), log_decay=_slopes(H), S0=randn(N, H, d, d))
        if op == "decay_train":
            s.update(dO=bf(randn(T, H, d)), dS=randn(N, H, d, d))
        return s
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "attention_tokens":
        room = case["room"]
        s.update(Q=bf(1.5 * randn(N, Hq, d)), K=bf(randn(N * room, Hkv, d)), V=bf(randn(N * room, Hkv, d)),
                 cu=_cu([1] * N), cu_k=_cu([room] * N), k_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 room=room)
        return s
    s.update(Q=bf(1.5 * randn(T, Hq, d)), K=bf(randn(T, Hkv, d)), V=bf(randn(T, Hkv, d)), cu=_cu(lens),
             longest=max(lens))
    if op == "attention_train":
        s["dO"] = bf(randn(T, Hq, d))
    return s


def _slopes(H):
    """log decay of each head, -2^(-8 (h + 1) / H): from heads that forget in two tokens to ones that keep 256."""
    return -torch.exp2(-8.0 * (torch.arange(H, device=DEV, dtype=torch.float32) + 1) / H)


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        from frame_level_delta_b200 import vda
        op = s["op"]
        if op == "attention":
            return vda.causal_attention(s["Q"], s["K"], s["V"], s["cu"])
        if op == "attention_tokens":
            return vda.causal_attention(s["Q"], s["K"], s["V"], s["cu"], cu_k=s["cu_k"], k_len=s["k_len"])
        if op == "attention_train":
            O, lse = vda.causal_attention(s["Q"], s["K"], s["V"], s["cu"], return_lse=True)
            g = vda.causal_attention_backward(s["Q"], s["K"], s["V"], O, s["dO"], lse, s["cu"])
            return {"O": O, "dQ": g["dQ"], "dK": g["dK"], "dV": g["dV"]}
        if op == "decay":
            O, S = vda.decay_attention(s["Q"], s["K"], s["V"], s["log_decay"], s["cu"], S0=s["S0"])
            return {"O": O, "S": S}
        if op == "decay_step":
            O = vda.decay_attention_step(s["Q"], s["K"], s["V"], s["log_decay"], s["S"])
            return {"O": O, "S": s["S"]}
        O, S = vda.decay_attention(s["Q"], s["K"], s["V"], s["log_decay"], s["cu"], S0=s["S0"])
        g = vda.decay_attention_backward(s["Q"], s["K"], s["V"], s["dO"], s["log_decay"], s["cu"], S0=s["S0"],
                                         dS=s["dS"])
        return {"O": O, "S": S, "dQ": g["dQ"], "dK": g["dK"], "dV": g["dV"], "dS0": g["dS0"]}
    return {"attention": _plain_attention, "attention_tokens": _plain_tokens, "attention_train": _plain_attention,
            "decay": _plain_decay, "decay_step": _plain_step, "decay_train": _plain_decay}[s["op"]](s)


class _Pad:
    """Packed rows to [N, heads, longest, d] in 32 bits and back."""

    def __init__(self, cu, longest, T):
        pos = torch.arange(longest, device=cu.device)
        cu = cu.long()
        self.n = cu[1:] - cu[:-1]
        self.take = (cu[:-1, None] + pos).clamp(max=T - 1)
        self.live = pos < self.n[:, None]
        tok = torch.arange(T, device=cu.device)
        self.seq = torch.searchsorted(cu, tok, right=True) - 1
        self.pos = tok - cu[self.seq]

    def pad(self, x):
        return (x[self.take].float() * self.live[..., None, None]).transpose(1, 2)

    def packed(self, x):
        return x[self.seq, :, self.pos]


def _plain_attention(s):
    Q, K, V = s["Q"], s["K"], s["V"]
    (T, Hq, d), Hkv = Q.shape, K.shape[1]
    G, L = Hq // Hkv, s["longest"]
    p = _Pad(s["cu"], L, T)
    q = p.pad(Q).unflatten(1, (Hkv, G))                # [N, Hkv, G, L, d]
    k, v = p.pad(K).unsqueeze(2), p.pad(V).unsqueeze(2)  # [N, Hkv, 1, L, d]
    scale = d ** -0.5
    seen = torch.ones(L, L, dtype=torch.bool, device=Q.device).tril()
    x = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    P = x.div_(x.sum(-1, keepdim=True))
    o = P @ v
    O = p.packed(o.flatten(1, 2)).to(Q.dtype)
    if s["op"] == "attention":
        return O
    do = p.pad(s["dO"]).unflatten(1, (Hkv, G))
    dV = (P.transpose(-1, -2) @ do).sum(2)
    x = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(P).mul_(scale)
    dQ = x @ k
    dK = (x.transpose(-1, -2) @ q).sum(2)
    return {"O": O, "dQ": p.packed(dQ.flatten(1, 2)).to(Q.dtype), "dK": p.packed(dK).to(Q.dtype),
            "dV": p.packed(dV).to(Q.dtype)}


def _plain_tokens(s):
    Q, K, V, room = s["Q"], s["K"], s["V"], s["room"]
    (N, Hq, d), Hkv = Q.shape, K.shape[1]
    q = Q.float().view(N, Hkv, Hq // Hkv, d)
    k, v = (x.float().view(N, room, Hkv, d).transpose(1, 2) for x in (K, V))
    seen = torch.arange(room, device=Q.device) < s["k_len"][:, None, None, None]
    x = (q @ k.transpose(-1, -2) * d ** -0.5).masked_fill(~seen, -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    return ((x / x.sum(-1, keepdim=True)) @ v).view(N, Hq, d).to(Q.dtype)


def _plain_decay(s):
    Q, K, V, S0 = s["Q"], s["K"], s["V"], s["S0"]
    (T, H, d), L = Q.shape, s["longest"]
    p = _Pad(s["cu"], L, T)
    q, k, v = p.pad(Q), p.pad(K), p.pad(V)  # [N, H, L, d]
    # powers of the decay, exponents in 64 bits (positions are far apart)
    pos = torch.arange(L, device=Q.device)
    g = s["log_decay"].double()[:, None]
    power = torch.exp(g * torch.arange(L + 1, device=Q.device)).float()  # [H, L + 1]
    far = pos[:, None] - pos
    W = power[:, far.clamp(min=0)].mul_((far >= 0).float())              # [H, L, L]
    x = (q @ k.transpose(-1, -2)).mul_(W)
    into = power[:, 1:, None]                                            # a^(i + 1)
    o = x @ v + into * (q @ S0.transpose(-1, -2))
    left = (p.n[:, None, None] - 1 - pos).clamp(min=0)                   # steps from token j to its sequence's end
    out = power.expand(p.n.numel(), H, L + 1).gather(2, left.expand(-1, H, L))[..., None]
    whole = power.expand(p.n.numel(), H, L + 1).gather(2, p.n[:, None, None].expand(-1, H, 1))[..., None]
    S = whole * S0 + (v * out).transpose(-1, -2) @ k
    r = {"O": p.packed(o).to(Q.dtype), "S": S}
    if s["op"] == "decay":
        return r
    do, dS = p.pad(s["dO"]), s["dS"]
    dV = x.transpose(-1, -2) @ do + out * (k @ dS.transpose(-1, -2))
    x = (do @ v.transpose(-1, -2)).mul_(W)
    dQ = x @ k + into * (do @ S0)
    dK = x.transpose(-1, -2) @ q + out * (v @ dS)
    dS0 = whole * dS + (do * into).transpose(-1, -2) @ q
    return {**r, "dQ": p.packed(dQ).to(Q.dtype), "dK": p.packed(dK).to(Q.dtype), "dV": p.packed(dV).to(Q.dtype),
            "dS0": dS0}


def _plain_step(s):
    q, k, v = s["Q"].float(), s["K"].float(), s["V"].float()
    S = s["S"]
    S.mul_(torch.exp(s["log_decay"])[:, None, None]).add_(v[..., :, None] * k[..., None, :])
    return {"O": (S * q[..., None, :]).sum(-1).to(s["Q"].dtype), "S": S}


# ------------------------------------------------------------------ the least a pass has to do
def work(case):
    op, d = case["op"], case["d"]
    if op == "decay_step":
        rows = case["N"] * case["H"]
        return {"bytes": rows * (2 * d * d * 4 + 4 * d * 2), "flops": rows * 5 * d * d}
    lens = _lens(case)
    T, N = sum(lens), len(lens)
    if op.startswith("decay"):
        H = case["H"]
        tok, st = T * H * d * 2, N * H * d * d * 4
        if op == "decay":  # Q, K, V, O; S0, S
            return {"bytes": 4 * tok + 2 * st, "flops": T * H * 5 * d * d}
        # and backward: dO in, dQ, dK, dV out; dS in, dS0 out
        return {"bytes": 8 * tok + 4 * st, "flops": T * H * 16 * d * d}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "attention_tokens":
        return {"bytes": 2 * N * Hq * d * 2 + 2 * T * Hkv * d * 2, "flops": 4 * T * Hq * d}
    pairs = sum(n * (n + 1) // 2 for n in lens) * Hq
    tok = T * d * 2
    if op == "attention":
        return {"bytes": tok * (2 * Hq + 2 * Hkv), "flops": 4 * pairs * d}
    return {"bytes": tok * (4 * Hq + 4 * Hkv), "flops": 14 * pairs * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "decay_step":
        a = s["log_decay"].double().exp()
        S = torch.einsum("h,nhvk->nhvk", a, s["S"].double()) + torch.einsum("nhv,nhk->nhvk", s["V"].double(),
                                                                           s["K"].double())
        return {"O": torch.einsum("nhvk,nhk->nhv", S, s["Q"].double()), "S": S}
    lens = _lens(case)
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    if op.startswith("decay"):
        return _exact_decay(s, case, ends)
    Hq, Hkv = case["Hq"], case["Hkv"]
    G = Hq // Hkv
    if op == "attention_tokens":
        O = torch.empty(len(lens), Hq, d, dtype=torch.float64, device=DEV)
        for i, n in enumerate(lens):
            lo = i * case["room"]
            k, v = s["K"][lo:lo + n].double(), s["V"][lo:lo + n].double()
            for h in range(Hq):
                w = torch.softmax(k[:, h // G] @ s["Q"][i, h].double() / math.sqrt(d), 0)
                O[i, h] = w @ v[:, h // G]
        return O
    train = op == "attention_train"
    O = torch.empty(ends[-1], Hq, d, dtype=torch.float64, device=DEV)
    dQ, dK, dV = torch.zeros_like(O), *(torch.zeros(ends[-1], Hkv, d, dtype=torch.float64, device=DEV)
                                        for _ in range(2))
    for lo, hi in zip(ends, ends[1:]):
        mask = torch.full((hi - lo, hi - lo), -math.inf, dtype=torch.float64, device=DEV).triu(1)
        for h in range(Hq):
            leaf = [s[x][lo:hi, i].double().requires_grad_(train)
                    for x, i in (("Q", h), ("K", h // G), ("V", h // G))]
            o = torch.softmax(leaf[0] @ leaf[1].T / math.sqrt(d) + mask, -1) @ leaf[2]
            O[lo:hi, h] = o.detach()
            if train:
                a, b, c = torch.autograd.grad(o, leaf, s["dO"][lo:hi, h].double())
                dQ[lo:hi, h] = a
                dK[lo:hi, h // G] += b
                dV[lo:hi, h // G] += c
    return {"O": O, "dQ": dQ, "dK": dK, "dV": dV} if train else O


def _exact_decay(s, case, ends):
    """The recurrence S = a S + v k^T, o = S q in blocks of tokens, its gradients by autograd over it."""
    H, d, N, train = case["H"], case["d"], len(ends) - 1, case["op"] == "decay_train"
    T = ends[-1]
    r = {"O": torch.empty(T, H, d, dtype=torch.float64, device=DEV),
         "S": torch.empty(N, H, d, d, dtype=torch.float64, device=DEV)}
    if train:
        r.update({x: torch.empty_like(r["O"]) for x in ("dQ", "dK", "dV")}, dS0=torch.empty_like(r["S"]))
    a = s["log_decay"].double().exp()
    C = 64
    up = torch.arange(C, device=DEV, dtype=torch.float64)
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        leaf = [s[x][lo:hi].double().transpose(0, 1).contiguous().requires_grad_(train) for x in "QKV"]
        leaf.append(s["S0"][i].double().requires_grad_(train))
        q, k, v, S = leaf
        got = []
        for t in range(0, hi - lo, C):
            n = min(C, hi - lo - t)
            x, y, z = q[:, t:t + n], k[:, t:t + n], v[:, t:t + n]
            e = up[:n]
            past = a[:, None, None] ** (e[:, None] - e).clamp(min=0) * torch.ones(n, n, device=DEV).tril()
            got.append(torch.einsum("hij,hjv->hiv", past * torch.einsum("hic,hjc->hij", x, y), z)
                       + torch.einsum("hi,hvc,hic->hiv", a[:, None] ** (e + 1), S, x))
            S = a[:, None, None] ** n * S + torch.einsum("hj,hjv,hjc->hvc", a[:, None] ** (n - 1 - e), z, y)
        o = torch.cat(got, 1)
        r["O"][lo:hi], r["S"][i] = o.detach().transpose(0, 1), S.detach()
        if train:
            up_o = s["dO"][lo:hi].double().transpose(0, 1)
            *tok, dS0 = torch.autograd.grad([o, S], leaf, [up_o, s["dS"][i].double()])
            for x, y in zip(("dQ", "dK", "dV"), tok):
                r[x][lo:hi] = y.transpose(0, 1)
            r["dS0"][i] = dS0
    return r
