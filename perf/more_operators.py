"""The measured cases of more operators for hybrid models:

  delta   gated_delta_rule: a batch of prompts, packed end to end, through the gated delta rule (the prefill of such
          layers); the state slots advance in place
  dstep   gated_delta_rule_step: one decode token per request on the same state slots
  shared  shared_prefix_attention: one new token per request over a paged cache, all requests behind one common prefix
  norm    add_rms_norm: root-mean-square norm with the residual's addition, optionally to 8 bits with scales

`run` makes the library's calls where `own` is true and computes the same from elementary torch operations where it is
false; `exact` computes it in 64 bits from the definitions."""
import math

import torch

own = False

BF16, F16, F32, F64, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f16": F16, "f32": F32}
TINY = 2.0 ** -126  # the least scale of 8-bit values
FAINT = 1e-6  # beside the squares of queries and keys that are normed


# ------------------------------------------------------------------ cases --
def listed():
    small = dict(H=16, P=64, N=128, G=16, unit=False)  # the headline shape's heads, keys of length 1 from the caller
    large = dict(H=32, P=128, N=128, G=16, unit=True)  # two value heads share a key head, normed in the operator
    return [
        # a chat turn appended to a request: one short prompt, latency
        dict(name="delta_turn", op="delta", B=1, L=37, ragged=False, **small),
        # continuous batching: 16 prompts of very different lengths in one packed call
        dict(name="delta_ragged", op="delta", B=16, L=2048, ragged=True, **large),
        # one long document
        dict(name="delta_long", op="delta", B=1, L=16384, ragged=False, **large),
        # one request decoding: latency
        dict(name="dstep_one", op="dstep", B=1, **small),
        # a decode batch of an odd size
        dict(name="dstep_batch", op="dstep", B=253, **large),
        # a few requests behind a short system prompt: latency
        dict(name="shared_few", op="shared", B=3, Lp=500, L=40, ragged=True, Hq=16, Hk=2, D=128, page=16, dtype="bf16"),
        # a decode batch behind a long system prompt
        dict(name="shared_batch", op="shared", B=64, Lp=8192, L=1024, ragged=True, Hq=32, Hk=8, D=128, page=64, dtype="bf16"),
        # many answers about one document
        dict(name="shared_many", op="shared", B=256, Lp=30011, L=300, ragged=True, Hq=64, Hk=8, D=128, page=16, dtype="f16"),
        # one request's next token between two layers: latency
        dict(name="norm_one", op="norm", T=1, D=4096, res="bf16", group=None, dtype="bf16"),
        # a decode batch, 8 bits with one scale a token
        dict(name="norm_batch", op="norm", T=509, D=8192, res="bf16", group=0, dtype="bf16"),
        # a long prompt, the residual stream in fp32, 8 bits with a scale for each 128 values
        dict(name="norm_prompt", op="norm", T=16384, D=5120, res="f32", group=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("delta", "dstep", "shared", "norm"))
        if op in ("delta", "dstep"):
            H = rng.choice((2, 5, 8, 12, 16, 32))
            G = rng.choice([g for g in (1, 2, 4, 5, H) if H % g == 0])
            c = dict(op=op, H=H, P=16 * rng.randint(1, 16), N=rng.choice((16, 32, 64, 128, 256)), G=G, unit=rng.random() < 0.5)
            if op == "delta":
                c.update(B=_log(rng, 1, 32), L=_log(rng, 1, 16384), ragged=rng.random() < 0.7)
                if c["B"] * c["L"] * H > 16384 * 32:
                    continue
            else:
                c.update(B=_log(rng, 1, 512))
        elif op == "shared":
            Hk = rng.choice((1, 2, 4, 8))
            c = dict(op=op, B=_log(rng, 1, 256), Lp=_log(rng, 1, 100000), L=_log(rng, 1, 4096), ragged=rng.random() < 0.7,
                     Hq=Hk * rng.randint(1, 16), Hk=Hk, D=rng.choice((64, 128, 256)), page=rng.choice((1, 8, 16, 20, 64, 128)),
                     dtype=rng.choice(("bf16", "f16")))
            if c["B"] * c["L"] * Hk * c["D"] > 64 * 8192 * 8 * 128:
                continue
        else:
            group = rng.choice((None, 0, 32, 64, 128, 256))
            D = group * rng.randint(1, 16384 // group) if group else _log(rng, 16, 16384)
            c = dict(op=op, T=_log(rng, 1, 16384), D=D, res=rng.choice((None, "same", "f32")), group=group, dtype=rng.choice(("bf16", "f16")))
            c["res"] = c["dtype"] if c["res"] == "same" else c["res"]
        if _cost(c) <= most:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _lengths(c):
    """The requests' lengths: all L, or spread evenly from 1 to L in a scattered order (known without a device)."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    B, L = c["B"], c["L"]
    return [1 + (i * 7919 % B) * (L - 1) // max(1, B - 1) for i in range(B)]


def work(c):
    if c["op"] in ("delta", "dstep"):
        T = sum(_lengths(c)) if c["op"] == "delta" else c["B"]
        H, P, N, G = c["H"], c["P"], c["N"], c["G"]
        per_token = 2 * (2 * G * N + 2 * H * P) + 8 * H  # q, k, v, out; log_decay, beta
        return {"bytes": T * per_token + 8 * c["B"] * H * P * N, "flops": 6 * T * H * P * N}
    if c["op"] == "shared":
        own_tokens = sum(_lengths(c))
        return {"bytes": 4 * (c["Lp"] + own_tokens) * c["Hk"] * c["D"] + 4 * c["B"] * c["Hq"] * c["D"],
                "flops": 4 * (c["B"] * c["Lp"] + own_tokens) * c["Hq"] * c["D"]}
    T, D = c["T"], c["D"]
    size = 2 + {None: 0, "f32": 8}.get(c["res"], 4) + (2 if c["group"] is None else 1)
    scales = 0 if c["group"] is None else 4 * (D // c["group"] if c["group"] else 1)
    return {"bytes": T * (D * size + scales) + 2 * D, "flops": 6 * T * D}


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=F32):
        return torch.randn(*shape, generator=gen, device=dev).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    def scattered(n, many):
        return torch.randperm(n, generator=gen, device=dev)[:many].to(torch.int32)

    s = {"case": dict(c)}
    if c["op"] in ("delta", "dstep"):
        B, H, P, N, G = c["B"], c["H"], c["P"], c["N"], c["G"]
        lens = _lengths(c) if c["op"] == "delta" else [1] * B
        T = sum(lens)
        # v, q, k in one packed projection, as a layer has them; keys that the operator does not norm are about of length 1
        packed = normal(T, H * P + 2 * G * N)
        if not c["unit"]:
            packed[:, H * P:] *= N ** -0.5
        packed = packed.to(BF16)
        s["v"] = packed[:, :H * P].view(T, H, P)
        s["q"] = packed[:, H * P:H * P + G * N].view(T, G, N)
        s["k"] = packed[:, H * P + G * N:].view(T, G, N)
        # gates as such layers have them: gains in 0 .. 1, step sizes and rates as the Mamba2 decode step's
        s["beta"] = torch.sigmoid(normal(T, H))
        bias = torch.log(torch.expm1(uniform(1e-3, 0.1, H)))
        s["log_decay"] = -torch.exp(uniform(0.0, math.log(16.0), H)) * torch.log1p(torch.exp(normal(T, H) + bias))
        s["scale"] = N ** -0.5 if c["unit"] else 1.0
        pool = B + 3
        s["state"] = normal(pool, H, P, N)
        s["idx"] = scattered(pool, B)
        if c["op"] == "delta":
            s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
            s["longest"] = max(lens)
        s["out"] = torch.empty(T, H, P, dtype=BF16, device=dev)
        return s
    if c["op"] == "shared":
        B, Hq, Hk, D, page, lens, dtype = c["B"], c["Hq"], c["Hk"], c["D"], c["page"], _lengths(c), TYPES[c["dtype"]]
        first, width = -(-c["Lp"] // page), -(-c["L"] // page)
        pages = first + sum(-(-n // page) for n in lens) + 1
        s["q"] = normal(B, Hq, D, dtype=dtype)
        s["k_cache"] = torch.empty(pages, page, Hk, D, dtype=dtype, device=dev).normal_(generator=gen)
        s["v_cache"] = torch.empty(pages, page, Hk, D, dtype=dtype, device=dev).normal_(generator=gen)
        # scattered pages, none of them twice; entries behind a request's last page stay 0
        ids = scattered(pages, pages - 1)
        s["prefix"], ids = ids[:first].contiguous(), ids[first:]
        used = torch.tensor([-(-n // page) for n in lens], device=dev)
        taken = torch.arange(width, device=dev)[None] < used[:, None]
        s["table"] = torch.zeros(B, width, dtype=torch.int32, device=dev)
        s["table"][taken] = ids
        s["prefix_len"] = torch.tensor([c["Lp"]], dtype=torch.int32, device=dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["scale"] = D ** -0.5
        return s
    T, D, dtype = c["T"], c["D"], TYPES[c["dtype"]]
    s["x"] = normal(T, D, dtype=dtype)
    s["weight"] = (1 + 0.1 * normal(D)).to(dtype)
    # a residual stream is larger than one layer's part of it, and some of its channels are much larger
    s["residual"] = None if c["res"] is None else (4 * normal(T, D) * torch.exp(normal(D))).to(TYPES[c["res"]])
    s["eps"] = 1e-6
    return s


# -------------------------------------------------------------- the calls --
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"delta": _delta, "dstep": _dstep, "shared": _shared, "norm": _norm}[op](s)
    import selective_state_update_amd as ssu

    if op == "delta":
        out = ssu.gated_delta_rule(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["cu"], s["idx"],
                                   scale=s["scale"], normalize=s["case"]["unit"], out=s["out"])
        return out, s["state"]
    if op == "dstep":
        out = ssu.gated_delta_rule_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["idx"],
                                        scale=s["scale"], normalize=s["case"]["unit"], out=s["out"])
        return out, s["state"]
    if op == "shared":
        return ssu.shared_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix"], s["prefix_len"], s["table"],
                                           s["lens"], scale=s["scale"], return_lse=True)
    group = s["case"]["group"]
    if group is None:
        return ssu.add_rms_norm(s["x"], s["residual"], s["weight"], eps=s["eps"]), s["residual"]
    out, scales = ssu.add_rms_norm(s["x"], s["residual"], s["weight"], eps=s["eps"], quantize=True, group=group)
    return out, scales, s["residual"]


# ------------------------------------------------------- the plain forms --
def _unit(x, on):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + FAINT) if on else x


def _delta(s, C=64):
    """Chunks of C tokens: what the tokens of a chunk take from each other as one triangular inverse (rows one after the
    other, all chunks at once), then the chunks in order."""
    c, cu = s["case"], s["cu"].long()
    B, H, P, N, G = c["B"], c["H"], c["P"], c["N"], c["G"]
    hg, nc = H // G, -(-s["longest"] // C)
    at = torch.arange(nc * C, device=cu.device)
    valid = at[None] < (cu[1:] - cu[:-1])[:, None]  # [B, L]
    token = torch.where(valid, cu[:-1, None] + at[None], 0)

    def heads(x):  # [B, L, H] -> [B, G, hg, nc, C]
        return x.view(B, nc, C, G, hg).permute(0, 3, 4, 1, 2)

    def chunks(x):  # [B, L, heads, n] -> [B, heads, nc, C, n]
        return x.float().view(B, nc, C, x.shape[2], -1).permute(0, 3, 1, 2, 4)

    gain = heads(s["beta"][token] * valid[..., None])[..., None]
    to = heads(s["log_decay"][token].double() * valid[..., None]).cumsum(-1)
    q, k = (_unit(chunks(s[n][token]), c["unit"])[:, :, None] for n in ("q", "k"))  # [B, G, 1, nc, C, N]
    k = k * heads(valid[..., None].float().expand(B, nc * C, H))[:, :, :1, ..., None]  # nothing behind a prompt's end
    v = chunks(s["v"][token]).view(B, G, hg, nc, C, P)
    inside = torch.ones(C, C, dtype=torch.bool, device=cu.device).tril()
    between = torch.where(inside, to[..., :, None] - to[..., None, :], -math.inf).exp().float()
    pairs = (k @ k.transpose(-1, -2)) * between * gain
    inverse = torch.eye(C, device=cu.device).expand(pairs.shape).contiguous()
    for i in range(1, C):
        inverse[..., i, :i] = -(pairs[..., i:i + 1, :i] @ inverse[..., :i, :i])[..., 0, :]
    grow, late = to.exp().float()[..., None], (to[..., -1:] - to).exp().float()[..., None]
    values, keys = inverse @ (v * gain), inverse @ (k * grow * gain)
    weight = (q @ k.transpose(-1, -2)) * between
    asked, kept, whole = q * grow, (k * late).transpose(-1, -2), grow[..., -1:, :]
    state = s["state"][s["idx"].long()].view(B, G, hg, P, N).transpose(-1, -2)
    out = torch.empty(B, G, hg, nc, C, P, device=cu.device)
    for n in range(nc):
        u = values[..., n, :, :] - keys[..., n, :, :] @ state
        out[..., n, :, :] = asked[..., n, :, :] @ state + weight[..., n, :, :] @ u
        state = whole[..., n, :, :] * state + kept[..., n, :, :] @ u
    out = (out * s["scale"]).view(B, H, nc * C, P).transpose(1, 2)
    row = torch.arange(s["out"].shape[0], device=cu.device)
    request = torch.searchsorted(cu, row, right=True) - 1  # each packed token's request
    s["out"].copy_(out[request, row - cu[request]])
    s["state"][s["idx"].long()] = state.transpose(-1, -2).reshape(B, H, P, N)
    return s["out"], s["state"]


def _dstep(s):
    c, idx = s["case"], s["idx"].long()
    hg = c["H"] // c["G"]
    q, k = (_unit(s[n].float(), c["unit"]).repeat_interleave(hg, 1)[:, :, None] for n in ("q", "k"))
    state = s["state"][idx] * s["log_decay"].exp()[..., None, None]
    u = (s["v"].float() - (state * k).sum(-1)) * s["beta"][..., None]
    state = state + u[..., None] * k
    s["state"][idx] = state
    s["out"].copy_((state * q).sum(-1) * s["scale"])
    return s["out"], s["state"]


def _shared(s):
    c = s["case"]
    B, Hq, Hk, D, Lp = c["B"], c["Hq"], c["Hk"], c["D"], c["Lp"]
    rows = Hq // Hk
    kp, vp = (s[n][s["prefix"].long()].flatten(0, 1)[:Lp].float().transpose(0, 1) for n in ("k_cache", "v_cache"))  # [Hk, Lp, D]
    q = s["q"].float().view(B, Hk, rows, D)
    first = (q.transpose(0, 1).reshape(Hk, B * rows, D) @ kp.transpose(1, 2)) * s["scale"]  # [Hk, B * rows, Lp]
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).float().permute(0, 2, 3, 1)  # [B, Hk, D, L]
    v = s["v_cache"][table].flatten(1, 2).float().transpose(1, 2)  # [B, Hk, L, D]
    score = (q @ k) * s["scale"]
    seen = torch.arange(score.shape[-1], device=table.device) < s["lens"][:, None, None, None]
    score = torch.where(seen, score, -math.inf)
    top = torch.maximum(score.amax(-1), first.amax(-1).view(Hk, B, rows).transpose(0, 1))  # [B, Hk, rows]
    score = (score - top[..., None]).exp()
    first = first.sub_(top.transpose(0, 1).reshape(Hk, B * rows, 1)).exp_()
    total = score.sum(-1) + first.sum(-1).view(Hk, B, rows).transpose(0, 1)
    out = (score @ v + (first @ vp).view(Hk, B, rows, D).transpose(0, 1)) / total[..., None]
    return out.view(B, Hq, D).to(s["q"].dtype), (top + total.log()).view(B, Hq)


def _norm(s):
    c, y = s["case"], s["x"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
        s["residual"].copy_(y)
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if c["group"] is None:
        return y.to(s["x"].dtype), s["residual"]
    y = y.unflatten(-1, (-1, c["group"] or c["D"]))
    scales = (y.abs().amax(-1) / 448.0).clamp(min=TINY)
    return (y / scales[..., None]).clamp(-448.0, 448.0).to(E4M3).flatten(1), scales, s["residual"]


# ---------------------------------------------- the definitions in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    c, dev = s["case"], torch.device("cuda")

    def tokens(cu, longest):
        """The recurrence, token after token, every request at once."""
        hg, idx = c["H"] // c["G"], s["idx"].long()
        n, last = cu[1:] - cu[:-1], s["q"].shape[0] - 1
        state = s["state"][idx].double()
        out = torch.zeros(s["out"].shape, dtype=F64, device=dev)
        for t in range(longest):
            live = t < n
            row = (cu[:-1] + t).clamp(max=last)
            q, k = (s[x][row].double() for x in ("q", "k"))
            if c["unit"]:
                q, k = (x / (x.pow(2).sum(-1, keepdim=True) + FAINT).sqrt() for x in (q, k))
            q, k = (x.repeat_interleave(hg, 1) for x in (q, k))
            new = state * s["log_decay"][row].double().exp()[..., None, None]
            u = s["beta"][row].double()[..., None] * (s["v"][row].double() - torch.matmul(new, k[..., None])[..., 0])
            new.addcmul_(u[..., None], k[:, :, None, :])
            y = torch.matmul(new, q[..., None])[..., 0] * s["scale"]
            state = torch.where(live[:, None, None, None], new, state)
            # a request that has ended adds nothing to the row it points at
            out.index_add_(0, row, y * live[:, None, None])
        whole = s["state"].double()
        whole[idx] = state
        return out, whole

    def attention():
        """One request after the other, over the prefix and its own tokens in one row."""
        out = torch.empty(c["B"], c["Hq"], c["D"], dtype=F64, device=dev)
        lse = torch.empty(c["B"], c["Hq"], dtype=F64, device=dev)
        j = torch.arange(max(c["Lp"], c["L"]), device=dev)
        page, off = j // c["page"], j % c["page"]
        at = s["prefix"].long()[page[:c["Lp"]]], off[:c["Lp"]]
        head_k, head_v = s["k_cache"][at].double(), s["v_cache"][at].double()
        for b, n in enumerate(_lengths(c)):
            at = s["table"][b].long()[page[:n]], off[:n]
            k = torch.cat((head_k, s["k_cache"][at].double()))  # [Lp + n, Hk, D]
            v = torch.cat((head_v, s["v_cache"][at].double()))
            q = s["q"][b].double().view(c["Hk"], -1, c["D"])
            score = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]
            lse[b] = torch.logsumexp(score, -1).flatten()
            out[b] = torch.matmul(torch.softmax(score, -1), v.transpose(0, 1)).view(c["Hq"], c["D"])
        return out, lse

    def norm():
        """8-bit values: what they are rounded from."""
        y = s["x"].double()
        total = None
        if s["residual"] is not None:
            total = y = y + s["residual"].double()
        y = y / (y.pow(2).sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * s["weight"].double()
        if c["group"] is None:
            return y, total
        y = y.reshape(c["T"], -1, c["group"] or c["D"])
        scales = torch.clamp(y.abs().max(-1).values / 448, min=TINY)
        return (y / scales[..., None]).reshape(c["T"], c["D"]), scales, total

    if c["op"] == "delta":
        return tokens(s["cu"].long(), s["longest"])
    if c["op"] == "dstep":
        return tokens(torch.arange(c["B"] + 1, device=dev), 1)
    return attention() if c["op"] == "shared" else norm()
