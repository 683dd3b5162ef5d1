"""Linear attention over long prompts whose state lasts, for tests of what one segment hands to the next.

All of q, k, v, beta and the states are positive, so that nothing cancels: every value is as large as the sum of the
magnitudes it is made of, and an error in a decay shows in full. The reference is the recurrence in 64 bits; the bound
follows the kernels' scheme, in units of eps = 2^-24, for chunks of 32 tokens with S before and S' behind a chunk and L
its summed log decay (its magnitude):

  the state's factor exp(L)    |L| for the argument's rounding, 2 for the power, 1 for the product
  beta v exp(...) in 3 pieces  |L| for the argument, 2 for the power, 2 for the products, 1 for the pieces
  k times the pieces, summed   3 products of 32 tokens and the sum so far: 99 additions, each off by 2 at most
                               (truncated) of a sum that S' bounds
  the join of segments         |L| for the argument, 2 for the power, 2 for the product and the sum

together at most 2 |L| + 210 of S' for a chunk, which later decays carry along with it (E' = exp(L) E + eps (2 |L| + 210) S').

An output adds, of its own size, the state's and the scores' pairs of 16 bits (2^-16 each), sums over N and over a
chunk (2 eps an addition, N + 99 of them), factors (2 |L| + 10) and its rounding to bf16 (2^-8)."""
import torch

EPS = 2.0 ** -24
CHUNK = 32
F64 = torch.float64


def inputs(lens, H, P, N, G, rate, seed, device, fixed=False):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(lens), len(lens)

    def positive(*shape, dtype=torch.bfloat16):  # 0.5 to 1.5
        return (0.5 + torch.rand(*shape, generator=g)).to(dtype).to(device)

    decay = -rate * (torch.rand(H, generator=g) if fixed else torch.rand(T, H, generator=g))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    return dict(state=positive(B + 1, H, P, N, dtype=torch.float32) * (1.0 / max(rate, 1e-3)), q=positive(T, G, N), k=positive(T, G, N),
                v=positive(T, H, P), log_decay=decay.to(device), cu_seqlens=cu.to(device),
                state_batch_indices=torch.randperm(B + 1, generator=g)[:B].to(torch.int32).to(device),
                beta=positive(T, H, dtype=torch.float32), scale=0.25)


def exact(a, seg_len=0, bend=None):
    """(out, state, out's bound, state's bound). With `bend`, what a kernel would give whose factor exp(L) for a segment
    of seg_len tokens were bend(exp(L))."""
    state, out = a["state"].double().clone(), torch.zeros(a["v"].shape, dtype=F64, device=a["v"].device)
    otol, tol = torch.zeros_like(out), torch.zeros_like(state)
    T, H, P = a["v"].shape
    G, N = a["q"].shape[1:]
    group = torch.arange(H, device=out.device) // (H // G)
    decay = a["log_decay"].double().expand(T, H)
    cu = a["cu_seqlens"].tolist()
    for b, slot in enumerate(a["state_batch_indices"].tolist()):
        S, E = state[slot], torch.zeros_like(state[slot])
        first, moved = S, torch.zeros(H, dtype=F64, device=out.device)
        for t in range(cu[b], cu[b + 1]):
            at = t - cu[b]
            if at % CHUNK == 0:
                L = decay[t:min(t + CHUNK, cu[b + 1])].sum(0)
                whole = L.exp()[:, None, None]
            if bend and at % seg_len == 0:
                first, moved = S, torch.zeros_like(moved)
            new = (a["beta"][t].double()[:, None] * a["v"][t].double())[:, :, None] * a["k"][t].double()[group][:, None, :]
            S = S * decay[t].exp()[:, None, None] + new
            moved = moved + decay[t]
            if bend and at % seg_len == seg_len - 1 and t + 1 < cu[b + 1]:
                S = S + first * (bend(moved.exp()) - moved.exp())[:, None, None]
            last = at % CHUNK == CHUNK - 1 or t + 1 == cu[b + 1]
            # (inside a chunk the errors of the state before it, undecayed, bound what it hands on)
            q = a["q"][t].double()[group][:, None, :]
            y = a["scale"] * (S * q).sum(-1)
            out[t] = y
            size = (2 * L.abs() + 210)[:, None]
            otol[t] = y * (2.0 ** -8 + 2.0 ** -15 + EPS * (2 * N + 200 + size)) + a["scale"] * (E * q).sum(-1)
            if last:
                E = whole * E + EPS * size[..., None] * S
        state[slot], tol[slot] = S, E
    return out, state, otol, tol
