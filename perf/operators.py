"""The measured cases of the library's sequence operators for hybrid models:

  prompt  linear_attention: a batch of prompts, packed end to end, through linear attention with a decay per head
          (the prefill of Mamba2 and linear-attention layers); the state slots advance in place
  step    linear_attention_step: one decode token per request on the same state slots
  rope    qk_norm_rope: norms of queries and keys per head with the position rotation, optionally into a paged cache
  attend  paged_attention: one new token per request over a paged key-value cache

`run` makes the library's calls where `own` is true and computes the same from elementary torch operations where it is
false; `exact` computes it in 64 bits from the definitions."""
import math

import torch

own = False

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f16": F16}


# ------------------------------------------------------------------ cases --
def listed():
    mamba = dict(H=16, P=64, N=128, G=1, mamba=True)  # one rank's heads of a Mamba2 layer: the library's headline shape
    mha = dict(H=32, P=128, N=128, G=32, mamba=False)  # a linear-attention layer: every head its own q and k, fixed decays
    return [
        # a chat turn appended to a request: one short prompt, latency
        dict(name="prompt_short", op="prompt", B=1, L=37, ragged=False, **mamba),
        # continuous batching: 16 prompts of very different lengths in one packed call
        dict(name="prompt_ragged", op="prompt", B=16, L=2048, ragged=True, **mamba),
        # one long document, every head with its own queries and keys
        dict(name="prompt_long", op="prompt", B=1, L=16384, ragged=False, **mha),
        # one request decoding: latency
        dict(name="step_one", op="step", B=1, **mamba),
        # the headline decode batch
        dict(name="step_batch", op="step", B=512, **mamba),
        # linear-attention decode, an odd batch
        dict(name="step_heads", op="step", B=45, **mha),
        # one request's next token, its key and value into the cache: latency
        dict(name="rope_one", op="rope", T=1, Hq=16, Hk=2, D=128, rot=128, inter=False, page=16, dtype="bf16"),
        # a decode batch's next tokens into the cache
        dict(name="rope_batch", op="rope", T=509, Hq=32, Hk=8, D=128, rot=128, inter=False, page=64, dtype="bf16"),
        # a long prompt, interleaved pairs, half of each head rotated, no cache
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hk=8, D=128, rot=64, inter=True, page=0, dtype="f16"),
        # one request, a short context: latency
        dict(name="attend_one", op="attend", B=1, L=777, ragged=False, Hq=16, Hk=2, D=128, page=16, dtype="bf16"),
        # a decode batch over contexts of very different lengths
        dict(name="attend_batch", op="attend", B=64, L=8192, ragged=True, Hq=32, Hk=8, D=128, page=64, dtype="bf16"),
        # three requests with long contexts: the cache's length is what there is to split
        dict(name="attend_long", op="attend", B=3, L=100003, ragged=False, Hq=64, Hk=4, D=128, page=16, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("prompt", "step", "rope", "attend"))
        if op in ("prompt", "step"):
            H = rng.choice((2, 5, 8, 12, 16, 32))
            G = rng.choice([g for g in (1, 2, 4, 5, H) if H % g == 0])
            c = dict(op=op, H=H, P=16 * rng.randint(1, 16), N=rng.choice((16, 32, 64, 128, 256)), G=G, mamba=rng.random() < 0.5)
            if op == "prompt":
                c.update(B=_log(rng, 1, 32), L=_log(rng, 1, 16384), ragged=rng.random() < 0.7)
                if c["B"] * c["L"] * H > 16384 * 32:
                    continue
            else:
                c.update(B=_log(rng, 1, 512))
        elif op == "rope":
            Hk = rng.choice((1, 2, 4, 8))
            D = rng.choice((64, 80, 96, 128, 192, 256))
            rot = rng.choice((D, D // 2, 2 * rng.randint(1, D // 2)))
            c = dict(op=op, T=_log(rng, 1, 16384), Hq=Hk * rng.randint(1, 8), Hk=Hk, D=D, rot=rot, inter=rng.random() < 0.5,
                     page=rng.choice((0, 1, 16, 48, 64)), dtype=rng.choice(("bf16", "f16")))
        else:
            Hk = rng.choice((1, 2, 4, 8))
            c = dict(op=op, B=_log(rng, 1, 256), L=_log(rng, 1, 100000), ragged=rng.random() < 0.7, Hq=Hk * rng.randint(1, 16), Hk=Hk,
                     D=rng.choice((64, 128, 256)), page=rng.choice((1, 8, 16, 20, 64, 128)), dtype=rng.choice(("bf16", "f16")))
            if c["B"] * c["L"] * Hk * c["D"] > 64 * 8192 * 8 * 128:
                continue
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
    if c["op"] in ("prompt", "step"):
        T = sum(_lengths(c)) if c["op"] == "prompt" else c["B"]
        H, P, N, G = c["H"], c["P"], c["N"], c["G"]
        per_token = 2 * (2 * G * N + 2 * H * P) + (8 * H if c["mamba"] else 0)  # q, k, v, out; log_decay, beta
        return {"bytes": T * per_token + 8 * c["B"] * H * P * N, "flops": 4 * T * H * P * N}
    if c["op"] == "rope":
        T, D = c["T"], c["D"]
        rows = c["Hq"] + c["Hk"] + (c["Hk"] if c["page"] else 0)
        return {"bytes": T * (4 * rows * D + 4 * c["rot"]), "flops": T * (c["Hq"] + c["Hk"]) * D * 7}
    tokens = sum(_lengths(c))
    return {"bytes": 4 * tokens * c["Hk"] * c["D"] + 4 * c["B"] * c["Hq"] * c["D"], "flops": 4 * tokens * c["Hq"] * c["D"]}


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
    if c["op"] in ("prompt", "step"):
        B, H, P, N, G = c["B"], c["H"], c["P"], c["N"], c["G"]
        lens = _lengths(c) if c["op"] == "prompt" else [1] * B
        T = sum(lens)
        # v, q, k in one packed projection, as a layer has them
        packed = normal(T, H * P + 2 * G * N, dtype=BF16)
        s["v"] = packed[:, :H * P].view(T, H, P)
        s["q"] = packed[:, H * P:H * P + G * N].view(T, G, N)
        s["k"] = packed[:, H * P + G * N:].view(T, G, N)
        if c["mamba"]:  # step sizes and rates as the decode step's: delta = softplus(dt + bias), decay exp(A delta)
            bias = torch.log(torch.expm1(uniform(1e-3, 0.1, H)))
            s["beta"] = torch.log1p(torch.exp(normal(T, H) + bias))
            s["log_decay"] = -torch.exp(uniform(0.0, math.log(16.0), H)) * s["beta"]
            s["scale"] = 1.0
        else:  # a fixed rate for each head, 1/2 to 1/256 a token
            s["beta"] = None
            s["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev) / H).float()
            s["scale"] = N ** -0.5
        pool = B + 3
        s["state"] = normal(pool, H, P, N)
        s["idx"] = scattered(pool, B)
        if c["op"] == "prompt":
            s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
            s["longest"] = max(lens)
        s["out"] = torch.empty(T, H, P, dtype=BF16, device=dev)
        return s
    Hq, Hk, D, dtype = c["Hq"], c["Hk"], c["D"], TYPES[c["dtype"]]
    if c["op"] == "rope":
        T, rot = c["T"], c["rot"]
        packed = normal(T, (Hq + 2 * Hk) * D, dtype=dtype)
        s["q"] = packed[:, :Hq * D].view(T, Hq, D)
        s["k"] = packed[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["v"] = packed[:, (Hq + Hk) * D:].view(T, Hk, D)
        far = 40960
        angle = torch.arange(far, device=dev, dtype=F64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=F64) / rot)
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        if c["page"]:  # decode: every token is at a place of its own
            s["positions"] = torch.randint(0, far, (T,), generator=gen, device=dev)
            pages = -(-2 * T // c["page"]) + 1
            s["k_cache"] = normal(pages, c["page"], Hk, D, dtype=dtype)
            s["v_cache"] = normal(pages, c["page"], Hk, D, dtype=dtype)
            s["slots"] = torch.randperm(pages * c["page"], generator=gen, device=dev)[:T]
        else:  # a prompt: consecutive positions
            s["positions"] = torch.arange(T, device=dev) + seed % 1000
        s["wq"], s["wk"] = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        s["wq"], s["wk"] = s["wq"].to(dtype), s["wk"].to(dtype)
        s["eps"] = 1e-6
        return s
    B, page, lens = c["B"], c["page"], _lengths(c)
    width = -(-c["L"] // page)
    pages = sum(-(-n // page) for n in lens) + 1
    s["q"] = normal(B, Hq, D, dtype=dtype)
    s["k_cache"] = torch.empty(pages, page, Hk, D, dtype=dtype, device=dev).normal_(generator=gen)
    s["v_cache"] = torch.empty(pages, page, Hk, D, dtype=dtype, device=dev).normal_(generator=gen)
    # scattered pages, none of them twice; entries behind a request's last page stay 0
    used = torch.tensor([-(-n // page) for n in lens], device=dev)
    taken = torch.arange(width, device=dev)[None] < used[:, None]
    s["table"] = torch.zeros(B, width, dtype=torch.int32, device=dev)
    s["table"][taken] = scattered(pages, pages - 1)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["longest"] = max(lens)
    s["scale"] = D ** -0.5
    return s


# -------------------------------------------------------------- the calls --
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"prompt": _prompt, "step": _step, "rope": _rope, "attend": _attend}[op](s)
    import selective_state_update_amd as ssu

    if op == "prompt":
        out = ssu.linear_attention(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["idx"],
                                   beta=s["beta"], scale=s["scale"], out=s["out"])
        return out, s["state"]
    if op == "step":
        out = ssu.linear_attention_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["idx"],
                                        beta=s["beta"], scale=s["scale"], out=s["out"])
        return out, s["state"]
    if op == "rope":
        if s["case"]["page"]:
            q, _ = ssu.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["wq"], s["wk"], eps=s["eps"],
                                    interleaved=s["case"]["inter"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                                    slots=s["slots"])
            return q, s["k_cache"], s["v_cache"]
        return ssu.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["wq"], s["wk"], eps=s["eps"],
                                interleaved=s["case"]["inter"])
    return ssu.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale=s["scale"], return_lse=True)


# ------------------------------------------------------- the plain forms --
def _prompt(s, C=64):
    """Chunks of C tokens: products inside a chunk, and the chunks' states joined by one product over the chunks."""
    c, cu = s["case"], s["cu"].long()
    B, H, P, N, G = c["B"], c["H"], c["P"], c["N"], c["G"]
    hg, nc = H // G, -(-s["longest"] // C)
    at = torch.arange(nc * C, device=cu.device)
    valid = at[None] < (cu[1:] - cu[:-1])[:, None]  # [B, L]
    token = torch.where(valid, cu[:-1, None] + at[None], 0)
    decay = s["log_decay"].expand(s["v"].shape[0], H)[token].double() * valid[..., None]
    gain = valid[..., None].float() * (torch.ones_like(decay) if s["beta"] is None else s["beta"][token]).float()

    def chunks(x):  # [B, L, heads, n] -> [B, heads, nc, C, n]
        return x.float().view(B, nc, C, x.shape[2], -1).permute(0, 3, 1, 2, 4)

    q, k = chunks(s["q"][token])[:, :, None], chunks(s["k"][token])[:, :, None]  # [B, G, 1, nc, C, N]
    v = chunks(s["v"][token]).view(B, G, hg, nc, C, P)
    gain = gain.view(B, nc, C, G, hg).permute(0, 3, 4, 1, 2)  # [B, G, hg, nc, C]
    to = decay.view(B, nc, C, G, hg).permute(0, 3, 4, 1, 2).cumsum(-1)
    total = to[..., -1].cumsum(-1)  # up to each chunk's end
    inside = torch.ones(C, C, dtype=torch.bool, device=cu.device).tril()
    weight = torch.where(inside, to[..., :, None] - to[..., None, :], -math.inf).exp().float() * gain[..., None, :]
    out = ((q @ k.transpose(-1, -2)) * weight) @ v
    late = (to[..., -1:] - to).exp().float() * gain
    own_state = (v * late[..., None]).transpose(-1, -2) @ k  # [B, G, hg, nc, P, N]
    # states before each chunk and behind the last: row r takes chunk j < r with the decay between them
    start = torch.cat((torch.zeros_like(total[..., :1]), total), -1)
    before = torch.ones(nc + 1, nc, dtype=torch.bool, device=cu.device).tril(-1)
    join = torch.where(before, start[..., :, None] - total[..., None, :], -math.inf).exp().float()
    states = (join @ own_state.reshape(B, G, hg, nc, P * N)).view(B, G, hg, nc + 1, P, N)
    first = s["state"][s["idx"].long()].view(B, G, hg, 1, P, N)
    states = states + start.exp().float()[..., None, None] * first
    out = out + to.exp().float()[..., None] * (q @ states[..., :-1, :, :].transpose(-1, -2))
    out = (out * s["scale"]).view(B, H, nc * C, P).transpose(1, 2)
    row = torch.arange(s["out"].shape[0], device=cu.device)
    request = torch.searchsorted(cu, row, right=True) - 1  # each packed token's request
    s["out"].copy_(out[request, row - cu[request]])
    s["state"][s["idx"].long()] = states[..., -1, :, :].reshape(B, H, P, N)
    return s["out"], s["state"]


def _step(s):
    c, idx = s["case"], s["idx"].long()
    hg = c["H"] // c["G"]
    q, k = (s[n].float().repeat_interleave(hg, 1) for n in ("q", "k"))
    v = s["v"].float()
    if s["beta"] is not None:
        v = v * s["beta"][..., None]
    decay = s["log_decay"].exp().expand(c["B"], c["H"])
    state = s["state"][idx] * decay[..., None, None] + v[..., None] * k[:, :, None, :]
    s["state"][idx] = state
    s["out"].copy_((state @ q[..., None])[..., 0] * s["scale"])
    return s["out"], s["state"]


def _turned(x, cos, sin, rot, inter):
    """The rotation of the first `rot` values of each head."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _rope(s):
    c = s["case"]
    cos, sin = s["cos_sin"][s["positions"]].chunk(2, -1)

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        return _turned(y, cos, sin, c["rot"], c["inter"]).to(x.dtype)

    q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
    if not c["page"]:
        return q, k
    s["k_cache"].view(-1, c["Hk"], c["D"])[s["slots"]] = k
    s["v_cache"].view(-1, c["Hk"], c["D"])[s["slots"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _attend(s):
    c = s["case"]
    B, Hq, Hk, D = c["B"], c["Hq"], c["Hk"], c["D"]
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).float().permute(0, 2, 3, 1)  # [B, Hk, D, L]
    v = s["v_cache"][table].flatten(1, 2).float().transpose(1, 2)  # [B, Hk, L, D]
    score = (s["q"].float().view(B, Hk, Hq // Hk, D) @ k) * s["scale"]
    seen = torch.arange(score.shape[-1], device=table.device) < s["lens"][:, None, None, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    score = (score - top).exp()
    total = score.sum(-1, keepdim=True)
    out = (score @ v) / total
    return out.view(B, Hq, D).to(s["q"].dtype), (top + total.log()).view(B, Hq)


# ---------------------------------------------- the definitions in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    c, dev = s["case"], s["q"].device

    def tokens(cu, longest):
        """The recurrence, token after token, every request at once."""
        hg, idx = c["H"] // c["G"], s["idx"].long()
        n, last = cu[1:] - cu[:-1], s["q"].shape[0] - 1
        state = s["state"][idx].double()
        out = torch.zeros(s["out"].shape, dtype=F64, device=dev)
        for t in range(longest):
            live = t < n
            row = (cu[:-1] + t).clamp(max=last)
            q, k = (s[x][row].double().repeat_interleave(hg, 1) for x in ("q", "k"))
            v = s["v"][row].double()
            if s["beta"] is not None:
                v = v * s["beta"][row].double()[..., None]
            a = (s["log_decay"] if s["log_decay"].dim() == 1 else s["log_decay"][row]).double().exp().expand(c["B"], c["H"])
            new = (v[..., None] * k[:, :, None, :]).addcmul_(state, a[..., None, None])
            state = torch.where(live[:, None, None, None], new, state)
            y = (new * q[:, :, None, :]).sum(-1) * s["scale"]
            # a request that has ended adds nothing to the row it points at
            out.index_add_(0, row, y * live[:, None, None])
        whole = s["state"].double()
        whole[idx] = state
        return out, whole

    def rotation():
        """Pairs as complex numbers, turned by one product."""
        half = c["rot"] // 2
        row = s["cos_sin"][s["positions"]].double()
        turn = torch.complex(row[:, :half], row[:, half:])[:, None]

        def one(x, w):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * w.double()
            part = y[..., :c["rot"]]
            part = part.unflatten(-1, (half, 2)) if c["inter"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
            part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            y[..., :c["rot"]] = (part if c["inter"] else part.transpose(-1, -2)).flatten(-2)
            return y

        q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
        if not c["page"]:
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        page, off = s["slots"] // c["page"], s["slots"] % c["page"]
        kc[page, off] = k
        vc[page, off] = s["v"].double()
        return q, kc, vc

    def attention():
        """One request after the other, over its own tokens alone."""
        out = torch.empty(c["B"], c["Hq"], c["D"], dtype=F64, device=dev)
        lse = torch.empty(c["B"], c["Hq"], dtype=F64, device=dev)
        for b, n in enumerate(_lengths(c)):
            j = torch.arange(n, device=dev)
            page, off = s["table"][b].long()[j // c["page"]], j % c["page"]
            k, v = s["k_cache"][page, off].double(), s["v_cache"][page, off].double()  # [n, Hk, D]
            q = s["q"][b].double().view(c["Hk"], -1, c["D"])
            score = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]
            lse[b] = torch.logsumexp(score, -1).flatten()
            out[b] = torch.matmul(torch.softmax(score, -1), v.transpose(0, 1)).view(c["Hq"], c["D"])
        return out, lse

    if c["op"] == "prompt":
        return tokens(s["cu"].long(), s["longest"])
    if c["op"] == "step":
        return tokens(torch.arange(c["B"] + 1, device=dev), 1)
    return rotation() if c["op"] == "rope" else attention()
