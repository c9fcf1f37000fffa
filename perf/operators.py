"""Workloads of the operators that serve and train low-rank adapters over packed projections.

Every case is one call (or the two of a forward pass) as a serving or training program makes it
next to the packed W4/W8 x A8 linear layers:

  adapters   y + scale_l (x A_l^T) B_l^T, the adapter l chosen per token, beside a shared projection
  adapters_backward  gradients of A, B and x of the same, x taken from its 8-bit checkpoint (the codes the
             projection was given) or from bf16
  gated      silu(gate) * up quantized per token to INT8 for the down projection, with or without the
             8-bit checkpoints of gate and up
  gated_backward     gradients of gate and up from those checkpoints
  packed_backward    dx = dy W of a packed projection (the gradient that goes on to the layer before)

Where `own` is false, run() computes the operators from elementary torch operations.
"""
import math

import torch

own = False

GROUP = 128  # features per scale of a gated checkpoint


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request answering: the next token of one chat, its adapter beside the attention output projection
        dict(name="adapters 1 token", op="adapters", M=1, N=4096, K=4096, L=8, rmin=16, rmax=16, layout="tokens",
             none=0.0, dtype="bf16", save=False),
        # a decode batch of 64 requests over 40 adapters of unequal rank, some requests without one; fp32 outputs
        dict(name="adapters 64 tokens", op="adapters", M=64, N=9728, K=2560, L=40, rmin=5, rmax=64, layout="tokens",
             none=0.1, dtype="f32", save=False),
        # prefill of ragged requests, 4001 tokens in all, beside a gate projection
        dict(name="adapters prefill", op="adapters", M=4001, N=14336, K=4096, L=6, rmin=8, rmax=64, layout="segments",
             none=0.1, dtype="bf16", save=False),
        # a short training sequence: one adapter, k/v-sized projection, gradients into an fp32 input gradient
        dict(name="adapters backward short", op="adapters_backward", M=77, N=1024, K=2560, L=1, rmin=8, rmax=8,
             layout="segments", none=0.0, dtype="f32", codes=True),
        # a training batch of four tasks over the down projection, activations kept in 8 bits
        dict(name="adapters backward batch", op="adapters_backward", M=8192, N=4096, K=14336, L=4, rmin=16, rmax=32,
             layout="segments", none=0.0, dtype="bf16", codes=True),
        # decode of 16 requests: the down projection's input, nothing kept
        dict(name="gated 16 tokens", op="gated", M=16, F=9728, keep=False),
        # a training batch's forward: codes for the down projection, gate and up kept in 8 bits
        dict(name="gated batch", op="gated", M=4096, F=14336, keep=True),
        # backward of a short sequence
        dict(name="gated backward short", op="gated_backward", M=77, F=9728),
        # backward of the training batch
        dict(name="gated backward batch", op="gated_backward", M=4096, F=14336),
        # a short sequence through a k/v-sized projection of 64-row tiles
        dict(name="packed backward short", op="packed_backward", M=77, N=1088, K=2560, bN=64, frac8=0.5),
        # a training sequence through the up projection
        dict(name="packed backward sequence", op="packed_backward", M=2048, N=9728, K=2560, bN=128, frac8=0.25),
        # a training batch through the down projection
        dict(name="packed backward batch", op="packed_backward", M=8192, N=4096, K=14336, bN=128, frac8=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the same ranges."""
    op = rng.choice(["adapters", "adapters_backward", "gated", "gated_backward", "packed_backward"])
    if op in ("gated", "gated_backward"):
        F = 16 * _log(rng, 8, 1088)
        M = min(_log(rng, 1, 8192), max(1, 4096 * 14336 // F))
        return dict(op=op, M=M, F=F, keep=rng.random() < 0.5) if op == "gated" else dict(op=op, M=M, F=F)
    if op == "packed_backward":
        bN = rng.choice([64, 128])
        N, K = bN * _log(rng, 1, 14336 // bN), 128 * _log(rng, 1, 112)
        M = min(_log(rng, 1, 8192), max(1, 8192 * 4096 * 14336 // (N * K)))
        return dict(op=op, M=M, N=N, K=K, bN=bN, frac8=rng.choice([0.0, 0.25, 0.5, 1.0]))
    N, K = 64 * _log(rng, 1, 224), 128 * _log(rng, 1, 112)
    M = min(_log(rng, 1, 8192), max(1, 4001 * 14336 // max(N, K)))
    tokens = M <= 64 and rng.random() < 0.7
    rmin = rng.randint(1, 24)
    case = dict(op=op, M=M, N=N, K=K, L=rng.randint(1, 48 if tokens else 8), rmin=rmin, rmax=rng.randint(rmin, 64),
                layout="tokens" if tokens else "segments", none=rng.choice([0.0, 0.2]),
                dtype=rng.choice(["bf16", "f32"]))
    if op == "adapters":
        case["save"] = rng.random() < 0.5
    else:
        case["codes"] = rng.random() < 0.7
    return case


def _ranks(c):
    """Ranks of the case's adapters: spread over rmin .. rmax, odd ones among them."""
    return [c["rmin"] + (11 * i + 5) % (c["rmax"] - c["rmin"] + 1) for i in range(c["L"])]


def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _normal(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _activations(g, M, K):
    """N(0, 1) with one input channel in a hundred 20 times as large."""
    x = _normal(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 20
    return x.to(torch.bfloat16)


def _absmax_codes(x, width):
    """INT8 codes of groups of `width` features and their scales: round(x / s), s = max|x| / 127."""
    M, F = x.shape
    pad = (-F) % width
    v = torch.nn.functional.pad(x.double(), (0, pad)).view(M, -1, width)
    s = (v.abs().amax(2, keepdim=True) / 127).clamp_min(1e-12)
    q = torch.round(v / s).clamp(-127, 127).to(torch.int8).view(M, F + pad)[:, :F].contiguous()
    return q, s.float().squeeze(2)


def _adapter_inputs(c, g):
    M, N, K, L = c["M"], c["N"], c["K"], c["L"]
    ranks = _ranks(c)
    R = sum(ranks)
    if c["layout"] == "tokens":
        ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
        ids[torch.rand(M, generator=g, device="cuda") < c["none"]] = -1
    else:  # contiguous requests of unequal length, one adapter each
        n = min(M, L)
        cuts = torch.sort(torch.randint(0, M, (n - 1,), generator=g, device="cuda")).values
        request = torch.bucketize(torch.arange(M, device="cuda"), cuts, right=True)
        of = torch.randperm(L, generator=g, device="cuda")[:n].to(torch.int32)
        if L > 1:
            of[torch.rand(n, generator=g, device="cuda") < c["none"]] = -1
        ids = of[request].contiguous()
    scales = [32.0 / (r + 8) for r in ranks]
    off = torch.tensor([sum(ranks[:i]) for i in range(L + 1)], device="cuda")
    s = dict(case=c, ids=ids, ranks=ranks, scales=scales, off=off, scale=torch.tensor(scales, device="cuda"),
             owner=torch.repeat_interleave(torch.arange(L, device="cuda"), torch.tensor(ranks, device="cuda")),
             rank=torch.tensor(ranks, device="cuda"), width=max(ranks),
             a=_normal(g, R, K, scale=K ** -0.5).to(torch.bfloat16), bt=_normal(g, R, N, scale=0.02).to(torch.bfloat16))
    if own:
        from w8_a8_quantized_b200 import aq
        s["adapters"] = aq.Adapters(s["a"], s["bt"], ranks, scales)
    return s


def prepare(case, seed):
    g = _generator(seed)
    c, op = case, case["op"]
    if op == "adapters":
        s = _adapter_inputs(c, g)
        s["x"] = _activations(g, c["M"], c["K"])
        s["y"] = _normal(g, c["M"], c["N"]).to(_dtype(c))
        return s
    if op == "adapters_backward":
        s = _adapter_inputs(c, g)
        x = _activations(g, c["M"], c["K"])
        s["dy"] = _normal(g, c["M"], c["N"], scale=1e-3).to(torch.bfloat16)
        s["dx"] = _normal(g, c["M"], c["K"], scale=1e-3).to(_dtype(c))  # the projection's own input gradient
        if c["codes"]:
            q, sx = _absmax_codes(x, c["K"])
            s["x"], s["sx"] = q, sx.reshape(-1).contiguous()
            x = q.float() * s["sx"][:, None]
        else:
            s["x"], s["sx"] = x, None
        s["s"] = _narrow(s, _masked(s, x.float() @ s["a"].float().t() * s["scale"][s["owner"]]))
        return s
    if op == "gated":
        return dict(case=c, gate=_activations(g, c["M"], c["F"]), up=_activations(g, c["M"], c["F"]))
    if op == "gated_backward":
        s = dict(case=c, dh=_normal(g, c["M"], c["F"], scale=1e-3).to(torch.bfloat16))
        s["gq"], s["gs"] = _absmax_codes(_activations(g, c["M"], c["F"]), GROUP)
        s["uq"], s["us"] = _absmax_codes(_activations(g, c["M"], c["F"]), GROUP)
        return s
    M, N, K, bN = c["M"], c["N"], c["K"], c["bN"]
    R, C = N // bN, K // 128
    pmap = torch.ones(R * C, dtype=torch.uint8, device="cuda")  # 1 marks an INT4 tile
    pmap[torch.randperm(R * C, generator=g, device="cuda")[: round(c["frac8"] * R * C)]] = 0
    pmap = pmap.view(R, C)
    raw = torch.randint(-128, 128, (N, K), dtype=torch.int16, generator=g, device="cuda")
    int4 = pmap.bool().repeat_interleave(bN, 0).repeat_interleave(128, 1)
    s = dict(case=c, codes=torch.where(int4, (raw & 15) - 8, raw).to(torch.int8), pmap=pmap,
             scales=(torch.rand((N, C), generator=g, device="cuda") * 9e-3 + 1e-3).to(torch.float16),
             dy=_normal(g, M, N, scale=1e-3).to(torch.bfloat16))
    if own:
        from w8_a8_quantized_b200 import aq
        s["packed"] = aq.aq_pack(s["codes"], s["scales"], pmap, bN, 128)
    return s


# ------------------------------------------------------------------ the plain forms
def _masked(s, v):
    """v [M][R] with zeros where row r is not of the token's adapter."""
    return torch.where(s["owner"][None, :] == s["ids"][:, None], v, torch.zeros((), device=v.device))


def _narrow(s, v):
    """[M][R] -> [M][widest rank]: the columns of each token's own adapter, zeros behind its rank."""
    ids = s["ids"].long()
    col = torch.arange(s["width"], device=v.device)[None, :]
    at = (s["off"][ids.clamp_min(0)][:, None] + col).clamp_max(v.shape[1] - 1)
    has = (ids[:, None] >= 0) & (col < s["rank"][ids.clamp_min(0)][:, None])
    return torch.where(has, v.gather(1, at), torch.zeros((), device=v.device))


def _widen(s, v):
    """The inverse of _narrow."""
    ids = s["ids"].long().clamp_min(0)
    at = torch.arange(s["owner"].numel(), device=v.device)[None, :] - s["off"][ids][:, None]
    return _masked(s, v.gather(1, at.clamp(0, v.shape[1] - 1)))


def _silu_parts(g):
    sig = 1 / (1 + torch.exp(-g))
    return sig, g * sig


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        from w8_a8_quantized_b200 import aq
        if op == "adapters":
            if c["save"]:
                kept = torch.empty((c["M"], s["width"]), dtype=torch.float32, device=s["x"].device)
                return aq.aq_lora_apply(s["adapters"], s["x"], s["ids"], s["y"], s=kept), kept
            return aq.aq_lora_apply(s["adapters"], s["x"], s["ids"], s["y"])
        if op == "adapters_backward":
            return aq.aq_lora_backward(s["adapters"], s["dy"], s["ids"], s["s"], s["x"], sx=s["sx"], add=s["dx"])
        if op == "gated":
            return aq.aq_silu_mul_quant(s["gate"], s["up"], keep=c["keep"])
        if op == "gated_backward":
            return aq.aq_silu_mul_backward(s["dh"], s["gq"], s["gs"], s["uq"], s["us"])
        return aq.aq_linear_backward(s["packed"], s["dy"])
    if op == "adapters":
        low = _masked(s, s["x"].float() @ s["a"].float().t() * s["scale"][s["owner"]])
        out = (s["y"].float() + low @ s["bt"].float()).to(s["y"].dtype)
        return (out, _narrow(s, low)) if c["save"] else out
    if op == "adapters_backward":
        dy, a = s["dy"].float(), s["a"].float()
        x = s["x"].float() * s["sx"][:, None] if c["codes"] else s["x"].float()
        dlow = _masked(s, dy @ s["bt"].float().t() * s["scale"][s["owner"]])
        return dlow.t() @ x, _widen(s, s["s"]).t() @ dy, (s["dx"].float() + dlow @ a).to(s["dx"].dtype)
    if op == "gated":
        # in 64 bits: the codes are whole numbers, and a quotient next to a half rounds either way in 32
        h = _silu_parts(s["gate"].double())[1] * s["up"].double()
        hq, sh = _absmax_codes(h, c["F"])
        if not c["keep"]:
            return hq, sh.reshape(-1)
        return (hq, sh.reshape(-1)) + _absmax_codes(s["gate"], GROUP) + _absmax_codes(s["up"], GROUP)
    if op == "gated_backward":
        F, dh = c["F"], s["dh"].float()
        g = s["gq"].float() * s["gs"].repeat_interleave(GROUP, 1)[:, :F]
        u = s["uq"].float() * s["us"].repeat_interleave(GROUP, 1)[:, :F]
        sig, silu = _silu_parts(g)
        return (dh * u * sig * (1 + g * (1 - sig))).to(torch.bfloat16), (dh * silu).to(torch.bfloat16)
    w = (s["codes"].float().view(c["N"], -1, 128) * s["scales"].float()[:, :, None]).view(c["N"], c["K"])
    return (s["dy"].float() @ w).to(torch.bfloat16)


# ------------------------------------------------------------------ work
def work(case):
    c, op = case, case["op"]
    if op in ("adapters", "adapters_backward"):
        ranks = _ranks(c)
        used = sum(ranks) * min(1.0, c["M"] / c["L"])  # rows of the adapters that some token has
        mean = sum(ranks) / len(ranks)
        M, N, K = c["M"], c["N"], c["K"]
        b = 4 if c["dtype"] == "f32" else 2
        if op == "adapters":
            save = 4 * M * max(ranks) if c["save"] else 0
            return {"bytes": 2 * M * K + 2 * b * M * N + 2 * used * (K + N) + 4 * M + save,
                    "flops": 2 * M * mean * (K + N)}
        x = M * K + 4 * M if c["codes"] else 2 * M * K
        return {"bytes": 2 * M * N + x + 2 * b * M * K + 2 * used * (K + N) + 4 * sum(ranks) * (K + N)
                + 4 * M * max(ranks) + 4 * M, "flops": 4 * M * mean * (K + N)}
    if op in ("gated", "gated_backward"):
        M, F = c["M"], c["F"]
        G = -(-F // GROUP)
        if op == "gated":
            return {"bytes": 5 * M * F + 4 * M + (2 * M * F + 8 * M * G if c["keep"] else 0), "flops": 8 * M * F}
        return {"bytes": 8 * M * F + 8 * M * G, "flops": 12 * M * F}
    M, N, K, bN = c["M"], c["N"], c["K"], c["bN"]
    T = (N // bN) * (K // 128)
    t8 = round(c["frac8"] * T)
    return {"bytes": 2 * M * N + 2 * M * K + bN * 128 * (t8 + (T - t8) / 2) + 2 * N * (K // 128) + 4 * T,
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits, adapter by adapter, group by group."""
    s, c, op = prepare(case, seed), case, case["op"]
    d = torch.float64
    if op in ("adapters", "adapters_backward"):
        M, N, K = c["M"], c["N"], c["K"]
        R = sum(s["ranks"])
        kept = torch.zeros(M, s["width"], dtype=d, device="cuda")
        if op == "adapters":
            out = s["y"].to(d)
        else:
            dx = s["dx"].to(d)
            da = torch.zeros(R, K, dtype=d, device="cuda")
            dbt = torch.zeros(R, N, dtype=d, device="cuda")
        row = 0
        for l, r in enumerate(s["ranks"]):
            at = torch.nonzero(s["ids"] == l).reshape(-1)
            A, Bt = s["a"][row:row + r].to(d), s["bt"][row:row + r].to(d)
            alpha = float(torch.tensor(s["scales"][l], dtype=torch.float32))
            if op == "adapters":
                low = torch.einsum("mk,rk->mr", s["x"][at].to(d), A).mul(alpha)
                kept[at, :r] = low
                out[at] += low @ Bt
            else:
                x = s["x"][at].to(d)
                if c["codes"]:
                    x = x * s["sx"][at].to(d)[:, None]
                dy = s["dy"][at].to(d)
                dlow = torch.einsum("mn,rn->mr", dy, Bt).mul(alpha)
                da[row:row + r] = torch.einsum("mr,mk->rk", dlow, x)
                dbt[row:row + r] = torch.einsum("mr,mn->rn", s["s"][at, :r].to(d), dy)
                dx[at] += dlow @ A
            row += r
        if op == "adapters":
            return (out, kept) if c["save"] else out
        return da, dbt, dx
    if op == "gated":
        g, u = s["gate"].to(d), s["up"].to(d)
        sh = (g * torch.sigmoid(g) * u).abs().max(1).values / 127
        if not c["keep"]:
            return None, sh
        groups = lambda v: torch.stack([p.abs().max(1).values for p in v.split(GROUP, 1)], 1) / 127  # noqa: E731
        return None, sh, None, groups(g), None, groups(u)
    if op == "gated_backward":
        cols = torch.arange(c["F"], device="cuda") // GROUP
        g, u = s["gq"].to(d) * s["gs"].to(d)[:, cols], s["uq"].to(d) * s["us"].to(d)[:, cols]
        dh, p = s["dh"].to(d), torch.sigmoid(g)
        return dh * u * (p + g * p * (1 - p)), dh * g * p
    out = torch.zeros(c["M"], c["K"], dtype=d, device="cuda")
    for j in range(c["K"] // 128):  # one column of tiles at a time
        w = s["codes"][:, 128 * j:128 * (j + 1)].to(d) * s["scales"][:, j:j + 1].to(d)
        out[:, 128 * j:128 * (j + 1)] = s["dy"].to(d) @ w
    return out
