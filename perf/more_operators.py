"""The steps of a decoder layer between its projections and the KV cache: what is measured of them.

adapt   qadapt: low-rank adapters, one for each request of a batch, added to a shared projection's output
norm    qnorm_rope: RMS norm of every query and key head and the position rotation, in one pass
prompt  qprompt_attend: causal attention of whole prompts, packed sequences, bf16 keys and values

Sizes are those of the 70B decoder layer (hidden 8192, MLP 28672, 64 query heads and 8 KV heads of 128), of the 512 x
512 layer and of smaller heads of 64.
"""
import math

import numpy as np
import torch

own = False

# Activations: a few channels carry larger values, as keys and hidden states have them.
_LOUD_CHANNELS, _LOUD = 4, 4.0
# Elements of a temporary of the plain attention.
_CHUNK = 1 << 28


# ------------------------------------------------------------------- cases
def _name(c, name):
    if name:
        c["name"] = name
    return c


def _adapt(K, N, rank, adapters, batch, rows=(1, 1), bare=0, ragged=False, bf16=False, name=None):
    """batch requests with rows[0] .. rows[1] rows each, every one with one of the adapters, `bare` of them without.
    ragged: the adapters' own ranks differ, up to rank.  bf16: the projection's output and the result are bf16."""
    return _name({"op": "adapt", "K": K, "N": N, "rank": rank, "adapters": adapters, "batch": batch, "row_min": rows[0],
                  "row_max": rows[1], "bare": bare, "ragged": ragged, "bf16": bf16}, name)


def _norm(head_dim, kv_heads, group, batch, lens, new, rot=None, pairs=False, f32=False, weights=True, prefix=0,
          name=None):
    """lens, new: (least, most) tokens a sequence holds, and of these the ones that are new in this pass.  rot: values of
    a head that are rotated, as pairs (2i, 2i + 1) or as halves.  f32: the projection's output is fp32.  prefix: tokens
    of a shared prefix before each sequence."""
    return _name({"op": "norm", "head_dim": head_dim, "kv_heads": kv_heads, "q_heads": kv_heads * group, "batch": batch,
                  "len_min": lens[0], "len_max": lens[1], "new_min": new[0], "new_max": new[1],
                  "rot": head_dim if rot is None else rot, "pairs": pairs, "f32": f32, "weights": weights,
                  "prefix": prefix}, name)


def _prompt(head_dim, kv_heads, group, batch, lens, name=None):
    """lens: (least, most) tokens of a prompt."""
    return _name({"op": "prompt", "head_dim": head_dim, "kv_heads": kv_heads, "q_heads": kv_heads * group,
                  "batch": batch, "len_min": lens[0], "len_max": lens[1]}, name)


def listed():
    return [
        # one user's adapter beside the k or v projection: latency
        _adapt(8192, 1024, 16, 4, 1, name="adapt_1_k_r16"),
        # a decode batch at the q projection, a dozen adapters of different ranks among its requests, some without
        _adapt(8192, 8192, 64, 12, 64, bare=5, ragged=True, name="adapt_64_q_r64"),
        # a decode batch at the gate projection, an adapter for each request
        _adapt(8192, 28672, 16, 16, 16, bf16=True, name="adapt_16_gate_r16"),
        # prompts of several requests at the down projection
        _adapt(28672, 8192, 32, 6, 5, rows=(77, 1500), bare=1, name="adapt_prompts_5x1500_down_r32"),
        # one decode step of a small batch
        _norm(128, 8, 8, 16, (1, 48), (1, 1), name="norm_step_16"),
        # one decode step of a large batch far into its contexts, small heads of which half is rotated, in pairs
        _norm(64, 4, 4, 200, (1000, 131072), (1, 1), rot=32, pairs=True, f32=True, prefix=701, name="norm_step_200_d64"),
        # chunks of two prompts behind what the cache holds of them
        _norm(128, 8, 8, 2, (4500, 6001), (700, 1024), name="norm_chunk_2x6001x1024"),
        # prompts of four requests, from the fp32 output of the projection
        _norm(128, 8, 8, 4, (517, 4096), (517, 4096), f32=True, name="norm_prompts_4x4096_f32"),
        # one short prompt: latency
        _prompt(128, 8, 8, 1, (77, 77), name="prompt_1x77"),
        # many short chats at once, small heads
        _prompt(64, 4, 4, 32, (1, 333), name="prompt_32x333_d64"),
        # ordinary prompts of ragged lengths
        _prompt(128, 8, 8, 3, (999, 2500), name="prompt_3x2500"),
        # one long document
        _prompt(128, 8, 8, 1, (16000, 16000), name="prompt_1x16000"),
    ]


def _between(rng, a, b):
    """A whole number of [a, b], spread over its logarithm."""
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["adapt", "norm", "prompt"])
    if op == "adapt":
        K, N, rank = 8 * _between(rng, 8, 3584), _between(rng, 16, 28672), 8 * _between(rng, 1, 16)
        flags = {"ragged": rng.random() < 0.3, "bf16": rng.random() < 0.5}
        adapters = _between(rng, 1, 16)
        if rng.random() < 0.5:
            batch = _between(rng, 1, 256)
            return _adapt(K, N, rank, adapters, batch, bare=rng.choice([0, 0, batch // 4]), **flags)
        batch = _between(rng, 1, 12)
        most = _between(rng, 2, max(2, 4000 // batch))
        return _adapt(K, N, rank, adapters, batch, (_between(rng, 1, most), most), bare=rng.choice([0, 0, batch // 4]),
                      **flags)
    head_dim, kv_heads, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if op == "norm":
        flags = {"rot": rng.choice([16, 32, 64, head_dim, head_dim]), "pairs": rng.random() < 0.3, "f32": rng.random() < 0.5,
                 "weights": rng.random() < 0.8, "prefix": rng.choice([0, 0, _between(rng, 1, 8192)])}
        if rng.random() < 0.5:
            most = _between(rng, 1, 131072)
            return _norm(head_dim, kv_heads, group, _between(rng, 1, 256), (_between(rng, 1, most), most), (1, 1), **flags)
        batch = _between(rng, 1, 16)
        most = _between(rng, 2, max(2, 9000 // batch))
        least = _between(rng, 1, most)
        return _norm(head_dim, kv_heads, group, batch, (least, most), (_between(rng, 1, least), most), **flags)
    batch = _between(rng, 1, 32)
    most = _between(rng, 1, min(12000, 20000 // batch))
    return _prompt(head_dim, kv_heads, group, batch, (_between(rng, 1, most), most))


def _spread(least, most, batch):
    """Lengths of the sequences, evenly between least and most."""
    return [most] if batch == 1 else [least + (most - least) * b // (batch - 1) for b in range(batch)]


def _rows_of(c):
    """Rows of each request or sequence in this pass."""
    if c["op"] == "adapt":
        return _spread(c["row_min"], c["row_max"], c["batch"])
    if c["op"] == "prompt":
        return _spread(c["len_min"], c["len_max"], c["batch"])
    return _spread(c["new_min"], c["new_max"], c["batch"])


# ------------------------------------------------------------------ inputs
def _loud(shape, gen, dev):
    x = torch.randn(shape, generator=gen, device=dev)
    x[..., :_LOUD_CHANNELS] *= _LOUD
    return x


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    rows = _rows_of(c)
    T = sum(rows)
    st = {"case": c, "T": T, "rows": rows, "single": max(rows) == 1,
          "starts": torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=dev)}
    if c["op"] == "adapt":
        n, K, N, r = c["adapters"], c["K"], c["N"], c["rank"]
        ids = host.integers(0, n, c["batch"])
        ids[host.permutation(c["batch"])[:c["bare"]]] = -1
        ranks = host.integers(1, r + 1, n) if c["ragged"] else np.full(n, r)
        st["host_ids"], st["host_ranks"] = ids.tolist(), ranks.tolist()
        st["ids"] = torch.tensor(ids, dtype=torch.int32, device=dev)
        st["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=dev)
        st["x"] = _loud((T, K), gen, dev).bfloat16()
        st["A"] = (torch.randn((n, r, K), generator=gen, device=dev) * K ** -0.5).bfloat16()
        st["B"] = (torch.randn((n, N, r), generator=gen, device=dev) * 0.1).bfloat16()
        st["scales"] = 32.0 / st["ranks"].float() * (0.5 + torch.rand(n, generator=gen, device=dev))
        y = torch.randn((T, N), generator=gen, device=dev) * 2.0
        st["y"] = y.bfloat16() if c["bf16"] else y
        return st
    D, H, Hq = c["head_dim"], c["kv_heads"], c["q_heads"]
    if c["op"] == "norm":
        lens = _spread(c["len_min"], c["len_max"], c["batch"])
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        # the output of one fused projection: rows of q, k and v lie side by side
        qkv = _loud((T, Hq + 2 * H, D), gen, dev)
        qkv = qkv if c["f32"] else qkv.bfloat16()
        st["Q"], st["K"] = qkv[:, :Hq], qkv[:, Hq:Hq + H]
        base = 5e5 if D == 128 else 1e4
        st["freqs"] = base ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        if c["weights"]:
            st["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device=dev)).bfloat16()
            st["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device=dev)).bfloat16()
        return st
    st["Q"] = torch.randn((T, Hq, D), generator=gen, device=dev).bfloat16()
    st["K"] = _loud((T, H, D), gen, dev).bfloat16()
    # values come as they left the fused projection
    st["V"] = _loud((T, Hq + 2 * H, D), gen, dev).bfloat16()[:, Hq + H:]
    st["scale"] = 1.0 / math.sqrt(D)
    return st


# ---------------------------------------------------------------- plain form
def _plain_adapt(st):
    c, ids, r = st["case"], st["ids"], st["case"]["rank"]
    held = torch.arange(r, device=ids.device)[None] < st["ranks"][:, None]                 # [adapters][r]
    if st["single"]:                     # a row for each request: its adapter's matrices gathered
        a = ids.clamp(min=0).long()
        h = (st["A"][a].float() * st["x"].float()[:, None]).sum(-1)
        h = torch.where(held[a], h, torch.zeros_like(h)) * st["scales"][a][:, None]
        d = (st["B"][a].float() * h[:, None]).sum(-1)
        return (st["y"].float() + torch.where(ids[:, None] >= 0, d, torch.zeros_like(d))).to(st["y"].dtype)
    out, t = st["y"].float().clone(), 0
    for n, a in zip(st["rows"], st["host_ids"]):
        if a >= 0:
            k = st["host_ranks"][a]
            h = torch.matmul(st["x"][t:t + n].float(), st["A"][a, :k].float().t()) * st["scales"][a]
            out[t:t + n] += torch.matmul(h, st["B"][a, :, :k].float().t())
        t += n
    return out.to(st["y"].dtype)


def _plain_norm(st):
    c, starts = st["case"], st["starts"]
    t = torch.arange(st["T"], device=starts.device)
    b = torch.searchsorted(starts, t.int(), right=True) - 1
    pos = st["lens"][b].long() - (starts[b + 1].long() - t) + c["prefix"]
    turn = pos.double()[:, None] * st["freqs"]
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
    outs = []
    for x, w in ((st["Q"], st.get("q_weight")), (st["K"], st.get("k_weight"))):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        r = x[..., :c["rot"]]
        if c["pairs"]:
            a, z = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - z * sin, z * cos + a * sin), -1).flatten(-2)
        else:
            a, z = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
            r = torch.cat((a * cos - z * sin, z * cos + a * sin), -1)
        outs.append(torch.cat((r, x[..., c["rot"]:]), -1).bfloat16())
    return tuple(outs)


def _plain_prompt(st):
    c, H, D = st["case"], st["case"]["kv_heads"], st["case"]["head_dim"]
    G = c["q_heads"] // H
    out = torch.empty_like(st["Q"])
    t = 0
    for n in st["rows"]:
        q = st["Q"][t:t + n].float().view(n, H, G, D).permute(1, 2, 0, 3)                   # [H][G][n][D]
        k = st["K"][t:t + n].float().transpose(0, 1)[:, None]                               # [H][1][n][D]
        v = st["V"][t:t + n].float().transpose(0, 1)[:, None]
        at = torch.arange(n, device=out.device)
        heads = max(1, min(H, _CHUNK // (G * n * n)))
        step = max(1, min(n, _CHUNK // (heads * G * n)))
        for h in range(0, H, heads):
            for i in range(0, n, step):
                s = torch.matmul(q[h:h + heads, :, i:i + step] * st["scale"], k[h:h + heads].transpose(2, 3))
                s = s.masked_fill(at[None] > at[i:i + step, None], -math.inf)
                p = torch.exp(s - s.amax(-1, keepdim=True))
                o = torch.matmul(p, v[h:h + heads]) / p.sum(-1, keepdim=True)               # [h][G][step][D]
                m = o.shape[2]
                out[t + i:t + i + m, h * G:(h + o.shape[0]) * G] = o.permute(2, 0, 1, 3).reshape(m, -1, D).bfloat16()
        t += n
    return out


def run(state):
    st, c = state, state["case"]
    if own:
        import compressed_gemv_amd as cg
        starts = None if st["single"] and c["op"] != "prompt" else st["starts"]
        if c["op"] == "adapt":
            held = st.get("held")
            if held is None:             # the adapters' handle, made once as a program keeps it
                held = st["held"] = cg.make_qadapters(st["A"], st["B"], st["scales"], st["ranks"] if c["ragged"] else None)
            return cg.qadapt(held, st["x"], st["y"], st["ids"], starts)
        if c["op"] == "norm":
            return cg.qnorm_rope(st["Q"], st["K"], st["lens"], starts, freqs=st["freqs"], q_weight=st.get("q_weight"),
                                 k_weight=st.get("k_weight"), eps=1e-6, pairs=c["pairs"], offset=c["prefix"])
        return cg.qprompt_attend(st["Q"], st["K"], st["V"], starts, scale=st["scale"])
    return {"adapt": _plain_adapt, "norm": _plain_norm, "prompt": _plain_prompt}[c["op"]](st)


# -------------------------------------------------------------------- exact
def _exact_adapt(c, st):
    out, t = st["y"].double(), 0
    for n, a in zip(st["rows"], st["host_ids"]):
        if a >= 0:
            k = st["host_ranks"][a]
            delta = st["B"][a].double()[:, :k] @ (st["A"][a].double()[:k] @ st["x"][t:t + n].double().T)
            out[t:t + n] = out[t:t + n] + delta.T * st["scales"][a].double()
        t += n
    return out


def _exact_norm(c, st):
    """Pairs as complex numbers, sequence by sequence."""
    lens = _spread(c["len_min"], c["len_max"], c["batch"])
    half, outs = c["rot"] // 2, []
    for x, w in ((st["Q"], st.get("q_weight")), (st["K"], st.get("k_weight"))):
        x = x.double().clone()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / c["head_dim"] + 1e-6).sqrt() * w.double()
        first = torch.arange(half, device=x.device) * (2 if c["pairs"] else 1)
        other = first + (1 if c["pairs"] else half)
        t = 0
        for n, m in zip(lens, st["rows"]):
            pos = torch.arange(n - m, n, device=x.device, dtype=torch.float64) + c["prefix"]
            z = torch.complex(x[t:t + m][..., first], x[t:t + m][..., other])
            z = z * torch.polar(torch.ones_like(pos)[:, None], torch.outer(pos, st["freqs"]))[:, None]
            x[t:t + m, :, first] = z.real
            x[t:t + m, :, other] = z.imag
            t += m
        outs.append(x)
    return tuple(outs)


def _exact_prompt(c, st):
    D, G = c["head_dim"], c["q_heads"] // c["kv_heads"]
    out = torch.empty(st["Q"].shape, dtype=torch.float64, device=st["Q"].device)
    t = 0
    for n in st["rows"]:
        step = max(1, min(n, (1 << 26) // n))
        for h in range(c["q_heads"]):
            kt, v = st["K"][t:t + n, h // G].double().T.contiguous(), st["V"][t:t + n, h // G].double()
            for i in range(0, n, step):
                m = min(step, n - i)
                s = st["Q"][t + i:t + i + m, h].double() @ kt[:, :i + m] * st["scale"]
                later = torch.ones((m, i + m), dtype=torch.bool, device=s.device).triu(i + 1)
                w = torch.softmax(s.masked_fill(later, -math.inf), 1)
                out[t + i:t + i + m, h] = w @ v[:i + m]
        t += n
    return out


def exact(case, seed):
    """From the definitions in fp64."""
    return {"adapt": _exact_adapt, "norm": _exact_norm, "prompt": _exact_prompt}[case["op"]](case, prepare(case, seed))


# --------------------------------------------------------------------- work
def work(case):
    c, rows = case, _rows_of(case)
    T = sum(rows)
    if c["op"] == "adapt":
        # adapters that a request may name, each matrix once; every row's x, y and result
        used, r = min(c["adapters"], max(1, c["batch"] - c["bare"])), c["rank"] * (0.5 if c["ragged"] else 1)
        served = T * (c["batch"] - c["bare"]) // max(1, c["batch"])
        es = 2 if c["bf16"] else 4
        return {"bytes": int(used * r * 2 * (c["K"] + c["N"]) + served * 2 * c["K"] + T * 2 * es * c["N"]),
                "flops": int(2 * served * r * (c["K"] + c["N"]))}
    D, H, Hq = c["head_dim"], c["kv_heads"], c["q_heads"]
    if c["op"] == "norm":
        n = T * (Hq + H) * D
        return {"bytes": n * ((4 if c["f32"] else 2) + 2), "flops": n * 8}
    return {"bytes": T * (2 * Hq + 2 * H) * D * 2, "flops": sum(4 * D * Hq * (n * (n + 1) // 2) for n in rows)}
