"""The quantised, paged KV cache: what is measured of its operators.

write   qcache_write of new tokens, then qcache_read of the sequences whole
read    qcache_read of ragged sequences
attend  qcache_attend: one token each, a few drafted tokens, or a chunk of a prompt
shared  qcache_attend_shared: one long prefix for the whole batch, own tokens behind it

Head counts are those of the 70B decoder layer (64 query heads, 8 KV heads of
128) and smaller ones of 64.  A cache row is one token of one KV head: b-bit
codes with an fp16 scale and an fp16 offset, row = s * q + o.
"""
import math

import numpy as np
import torch

own = False

# Rows of K and V: a few channels carry larger values, as keys have them.
_LOUD_CHANNELS, _LOUD = 4, 4.0


# ------------------------------------------------------------------- cases
def _case(op, bits, head_dim, kv_heads, group, page, batch, lens, new, prefix=0, idle=0, name=None):
    """lens, new: (least, most) tokens a sequence holds, and of these the ones that are new in this pass; sequence
    b of the batch lies evenly between.  idle: sequences of length zero at the end (a padded batch)."""
    c = {"op": op, "bits": bits, "head_dim": head_dim, "kv_heads": kv_heads, "q_heads": kv_heads * group, "page": page,
         "batch": batch, "len_min": lens[0], "len_max": lens[1], "new_min": new[0], "new_max": new[1],
         "prefix": prefix, "idle": idle}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the cache update of one decode step: one token for each of 16 short chats
        _case("write", 8, 128, 8, 8, 16, 16, (1, 48), (1, 1), name="write_step_16x1_b8"),
        # four prompts of different lengths enter the cache at once
        _case("write", 4, 128, 8, 8, 64, 4, (517, 4096), (517, 4096), name="write_prompts_4x4096_b4"),
        # a small cache handed to a kernel that wants bf16
        _case("read", 4, 64, 8, 4, 16, 7, (1, 333), (1, 333), name="read_7x333_d64_b4"),
        # sixteen conversations moved out of the cache
        _case("read", 8, 128, 8, 8, 32, 16, (300, 4000), (300, 4000), name="read_16x4000_b8"),
        # one user, one token: latency
        _case("attend", 8, 128, 8, 8, 16, 1, (517, 517), (1, 1), name="step_1x517_b8"),
        # an ordinary serving batch, padded by two idle rows
        _case("attend", 8, 128, 8, 8, 32, 32, (1000, 8000), (1, 1), idle=2, name="step_32x8000_b8"),
        # few users with very long contexts
        _case("attend", 4, 128, 8, 8, 256, 4, (100000, 131072), (1, 1), name="step_4x131072_b4"),
        # five drafted tokens verified for each of eight sequences
        _case("attend", 4, 64, 8, 4, 32, 8, (200, 3001), (5, 5), name="verify_8x3001x5_d64_b4"),
        # chunks of two prompts behind what the cache holds of them
        _case("attend", 8, 128, 8, 8, 64, 2, (4500, 6001), (700, 1024), name="chunk_2x6001x1024_b8"),
        # whole prompts of ragged lengths
        _case("attend", 4, 128, 8, 8, 16, 3, (999, 2500), (999, 2500), name="prompt_3x2500_b4"),
        # a small batch behind a system prompt
        _case("shared", 4, 64, 8, 4, 16, 6, (1, 40), (1, 1), prefix=701, name="shared_6x40_p701_d64_b4"),
        # a large batch behind a long document
        _case("shared", 8, 128, 8, 8, 64, 64, (1, 500), (1, 1), prefix=8229, name="shared_64x500_p8229_b8"),
    ]


def _between(rng, a, b):
    """A whole number of [a, b], spread over its logarithm."""
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "shared"])
    bits, head_dim, kv_heads = rng.choice([4, 8]), rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    group, page = rng.choice([1, 2, 4, 5, 8]), rng.choice([16, 32, 64, 128, 256])
    batch, idle = _between(rng, 1, 64), rng.choice([0, 0, 1])
    # tokens in all, bounded so that no case costs more than the largest listed one
    if op in ("write", "read"):
        most = _between(rng, 2, max(2, 8192 // batch))
        least = _between(rng, 1, most)
        new = (1, 1) if op == "write" and rng.random() < 0.5 else (least, most)
        return _case(op, bits, head_dim, kv_heads, group, page, batch, (least, most), new, idle=idle)
    if op == "shared":
        most = _between(rng, 2, 500)
        return _case(op, bits, head_dim, kv_heads, group, page, batch, (_between(rng, 1, most), most), (1, 1),
                     prefix=_between(rng, 65, 8192), idle=idle)
    kind = rng.choice(["step", "verify", "chunk"])
    if kind == "step":
        most = _between(rng, 2, max(2, min(65536, 200000 // batch)))
        return _case(op, bits, head_dim, kv_heads, group, page, batch, (_between(rng, 1, most), most), (1, 1), idle=idle)
    if kind == "verify":
        most = _between(rng, 16, max(16, min(16384, 100000 // batch)))
        new = rng.randint(2, 9)
        return _case(op, bits, head_dim, kv_heads, group, page, batch, (_between(rng, new, most), most), (new, new), idle=idle)
    batch = rng.randint(1, 4)
    new = _between(rng, 17, 1024)
    least = new + _between(rng, 1, 2048) - 1
    return _case(op, bits, head_dim, kv_heads, group, page, batch, (least, least + rng.randint(0, 1500)),
                 (max(1, new // 2), new), idle=idle)


def _spread(least, most, batch, idle):
    """Lengths of the sequences, evenly between least and most; the idle ones hold nothing."""
    n = [least + (most - least) * b // max(1, batch - 1) for b in range(batch)]
    if batch == 1:
        n = [most]
    return n + [0] * idle


def _lengths(c):
    lens = _spread(c["len_min"], c["len_max"], c["batch"], c["idle"])
    new = _spread(c["new_min"], c["new_max"], c["batch"], c["idle"])
    if c["new_max"] == 1:
        new = [1] * len(lens)            # one row for every sequence, the idle ones too
    return lens, new


# ------------------------------------------------------------------ inputs
def _f16_step(h, up):
    """The next fp16 value above (up) or below each of h."""
    b = h.view(torch.int16).to(torch.int32) & 0xFFFF
    mag, neg = b & 0x7FFF, b >= 0x8000
    away = ~neg if up else neg                                # the step leads away from zero
    nb = torch.where(mag == 0, torch.full_like(b, 1 if up else 0x8001),
                     torch.where(away, b + 1, b - 1))
    return nb.to(torch.int16).view(torch.float16)


def _quantise(x, bits):
    """x[..., D] -> (codes int64, s, o fp16): rows by round-to-nearest in fp64, offset rounded down, scale up."""
    x, top = x.double(), (1 << bits) - 1
    mn, mx = x.amin(-1), x.amax(-1)
    o = mn.half()
    o = torch.where(o.double() > mn, _f16_step(o, False), o)
    o = torch.where(o == 0, torch.zeros_like(o), o)
    v = (mx - o.double()) / top
    s = v.half()
    s = torch.where(s.double() < v, _f16_step(s, True), s)
    sd = s.double().unsqueeze(-1)
    q = torch.round((x - o.double().unsqueeze(-1)) / torch.where(sd == 0, torch.ones_like(sd), sd))
    return torch.where(sd == 0, torch.zeros_like(q), q).clamp(0, top).long(), s, o


def _pack(q, s, o, bits):
    """Codes as bytes (4 bits: the even code in the low half) and meta words (s low, o high)."""
    if bits == 4:
        q = q[..., 0::2] | (q[..., 1::2] << 4)
    meta = (s.view(torch.int16).int() & 0xFFFF) | (o.view(torch.int16).int() << 16)
    return q.to(torch.uint8), meta


def _rows(shape, gen, dev):
    x = torch.randn(shape, generator=gen, device=dev)
    x[..., :_LOUD_CHANNELS] *= _LOUD
    return x.bfloat16()


def _filled(n_pages, c, gen, dev):
    """A K or V cache of n_pages pages whose every row holds a token (a page of a freed sequence keeps its rows)."""
    H, P, D, bits = c["kv_heads"], c["page"], c["head_dim"], c["bits"]
    codes = torch.empty((n_pages, H, P, D * bits // 8), dtype=torch.uint8, device=dev)
    meta = torch.empty((n_pages, H, P), dtype=torch.int32, device=dev)
    step = max(1, (1 << 25) // (H * P * D))
    for a in range(0, n_pages, step):
        n = min(step, n_pages - a)
        codes[a:a + n], meta[a:a + n] = _pack(*_quantise(_rows((n, H, P, D), gen, dev), bits), bits)
    return codes, meta


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    lens, new = _lengths(c)
    P, D, H, Hq = c["page"], c["head_dim"], c["kv_heads"], c["q_heads"]
    width = max(1, max((n + P - 1) // P for n in lens))
    own_pages, pre_pages = [(n + P - 1) // P for n in lens], (c["prefix"] + P - 1) // P
    n_pages = sum(own_pages) + pre_pages + 1
    order = host.permutation(n_pages)
    pages = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(own_pages):
        pages[b, :n] = order[at:at + n]
        at += n
    T = sum(new)
    st = {"case": c, "T": T, "single": c["new_max"] == 1,
          "pages": torch.from_numpy(pages).to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
          "starts": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev),
          "whole": torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev),
          "tokens": sum(lens), "new_max": max(new), "scale": 1.0 / math.sqrt(D)}
    st["k_codes"], st["k_meta"] = _filled(n_pages, c, gen, dev)
    st["v_codes"], st["v_meta"] = _filled(n_pages, c, gen, dev)
    if c["prefix"]:
        st["prefix_pages"] = torch.from_numpy(order[at:at + pre_pages].astype(np.int32)).to(dev)
    if c["op"] == "write":
        # slices of one fused projection's output: rows of q, k and v lie side by side
        qkv = _rows((T, Hq + 2 * H, D), gen, dev)
        st["K"], st["V"] = qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    elif c["op"] in ("attend", "shared"):
        st["Q"] = torch.randn((T, Hq, D), generator=gen, device=dev).bfloat16()
    return st


# ---------------------------------------------------------------- plain form
def _values(codes, meta, bits):
    """Rows as fp32 values s * q + o."""
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    h = meta.view(torch.int16).view(torch.float16).view(meta.shape + (2,)).float()
    return codes.float() * h[..., :1] + h[..., 1:]


def _where(st, starts):
    """(sequence, position) of every row of a ragged batch, rows behind the last one left out."""
    n = int(st["T"] if starts is st["starts"] else st["tokens"])
    t = torch.arange(n, device=starts.device, dtype=torch.int32)
    b = torch.searchsorted(starts, t, right=True) - 1
    return b, st["lens"][b] - (starts[b + 1] - t)


def _plain_write(st):
    c, (b, pos) = st["case"], _where(st, st["starts"])
    ok = pos >= 0
    b, pos = b[ok], pos[ok].long()
    page, slot = st["pages"][b, pos // c["page"]].long(), pos % c["page"]
    for x, n in ((st["K"], "k"), (st["V"], "v")):
        codes, meta = _pack(*_quantise(x[ok], c["bits"]), c["bits"])
        st[n + "_codes"][page, :, slot] = codes
        st[n + "_meta"][page, :, slot] = meta


def _plain_read(st):
    c, (b, pos) = st["case"], _where(st, st["whole"])
    pos = pos.long()
    page, slot = st["pages"][b, pos // c["page"]].long(), pos % c["page"]
    return tuple(_values(st[n + "_codes"][page, :, slot], st[n + "_meta"][page, :, slot], c["bits"]).bfloat16()
                 for n in "kv")


def _gathered(st, pages, n):
    """[B][heads][positions][D] of the pages named, fp32."""
    c, p = st["case"], pages.clamp(min=0).long()
    x = _values(st[n + "_codes"][p], st[n + "_meta"][p], c["bits"])          # [B][pages][H][page][D]
    return x.transpose(1, 2).reshape(p.shape[0], c["kv_heads"], -1, c["head_dim"])


def _plain_attend(st):
    c, starts, lens = st["case"], st["starts"], st["lens"]
    H, G, D, B, M = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"], len(st["pages"]), st["new_max"]
    b, pos = _where(st, starts)
    i = torch.arange(st["T"], device=starts.device) - starts[b]
    q = torch.zeros((B, M, H, G, D), device=starts.device)
    q[b, i] = st["Q"].float().view(-1, H, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    k, v = _gathered(st, st["pages"], "k"), _gathered(st, st["pages"], "v")
    last = torch.full((B, M), -1, device=starts.device, dtype=torch.int32)
    last[b, i] = pos
    sees = torch.arange(k.shape[2], device=starts.device)[None, None] <= last[..., None]     # [B][M][positions]
    sees = sees.repeat_interleave(G, 1)[:, None]
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    s = s.masked_fill(~sees, -math.inf)
    m = s.amax(-1, keepdim=True)
    if c["op"] == "shared":
        kp, vp = _gathered(st, st["prefix_pages"][None], "k"), _gathered(st, st["prefix_pages"][None], "v")
        n = c["prefix"]
        qa = q.transpose(0, 1).reshape(H, -1, D)
        sp = (torch.matmul(qa, kp[0, :, :n].transpose(1, 2)) * st["scale"]).view(H, B, M * G, n).transpose(0, 1)
        m = torch.maximum(m, sp.amax(-1, keepdim=True))
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total, o = p.sum(-1, keepdim=True), torch.matmul(p, v)
    if c["op"] == "shared":
        p = torch.exp(sp - m)
        total = total + p.sum(-1, keepdim=True)
        o = o + torch.matmul(p.transpose(0, 1).reshape(H, B * M * G, n), vp[0, :, :n]).view(H, B, M * G, D).transpose(0, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.view(B, H, M, G, D).permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D)
    return o[b, i].bfloat16()


def run(state):
    op, c = state["case"]["op"], state["case"]
    if own:
        import compressed_gemv_amd as cg
        cache = state.get("cache")
        if cache is None:                # the handle, made once as a program keeps it
            cache = state["cache"] = cg.make_qcache(len(state["k_codes"]), c["page"], c["kv_heads"], c["head_dim"],
                                                    c["bits"], state["k_codes"], state["k_meta"], state["v_codes"],
                                                    state["v_meta"])
        starts = None if state["single"] else state["starts"]
        if op == "write":
            cg.qcache_write(cache, state["K"], state["V"], state["pages"], state["lens"], starts)
        if op in ("write", "read"):
            return cg.qcache_read(cache, state["pages"], state["lens"], state["whole"], rows=state["tokens"])
        if op == "attend":
            return cg.qcache_attend(cache, state["Q"], state["pages"], state["lens"], starts, scale=state["scale"])
        return cg.qcache_attend_shared(cache, state["Q"], state["prefix_pages"], c["prefix"], state["pages"],
                                       state["lens"], starts, scale=state["scale"])
    if op == "write":
        _plain_write(state)
    if op in ("write", "read"):
        return _plain_read(state)
    return _plain_attend(state)


# -------------------------------------------------------------------- exact
def _np_row_values(x, bits):
    """fp64 rows [n][D] as the cache gives them back, by the definition: numpy's fp16 neighbours."""
    top = float((1 << bits) - 1)
    with np.errstate(divide="ignore", invalid="ignore"):
        lo = x.min(1)
        o = lo.astype(np.float16)
        o = np.where(o.astype(np.float64) > lo, np.nextafter(o, np.float16(-np.inf)), o).astype(np.float64)
        need = (x.max(1) - o) / top
        s = need.astype(np.float16)
        s = np.where(s.astype(np.float64) < need, np.nextafter(s, np.float16(np.inf)), s).astype(np.float64)
        q = np.where(s[:, None] > 0, np.clip(np.rint((x - o[:, None]) / s[:, None]), 0, top), 0)
    return q * s[:, None] + o[:, None]


def exact(case, seed):
    """From the definitions in fp64, sequence by sequence."""
    c, st = case, prepare(case, seed)
    lens, new = _lengths(c)
    P, D, H, bits = c["page"], c["head_dim"], c["kv_heads"], c["bits"]
    G = c["q_heads"] // H

    def stored(pages, n, which):
        """[H][n][D] fp64 of the first n positions behind these pages."""
        codes, meta = (st[which + "_" + x][pages[:(n + P - 1) // P].long()] for x in ("codes", "meta"))
        if bits == 4:
            codes = torch.stack([codes % 16, codes // 16], dim=-1).reshape(codes.shape[:3] + (D,))
        s = (meta & 0xFFFF).to(torch.int16).view(torch.float16).double().unsqueeze(-1)
        o = (meta >> 16).to(torch.int16).view(torch.float16).double().unsqueeze(-1)
        return (codes.double() * s + o).permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n]

    if c["op"] in ("write", "read"):
        outs = []
        for which, fresh in (("k", st.get("K")), ("v", st.get("V"))):
            rows, t = [], 0
            for b, n in enumerate(lens):
                x = stored(st["pages"][b], n, which).transpose(0, 1).clone()
                if fresh is not None and n:
                    f = fresh[t:t + new[b]].double().cpu().numpy()[max(0, new[b] - n):]
                    f = _np_row_values(f.reshape(-1, D), bits).reshape(f.shape)
                    x[n - len(f):] = torch.from_numpy(f).to(x.device)
                rows.append(x)
                t += new[b]
            outs.append(torch.cat(rows))
        return tuple(outs)
    out = torch.zeros((st["T"], c["q_heads"], D), dtype=torch.float64, device=st["Q"].device)
    pre = c["prefix"]
    kp, vp = (stored(st["prefix_pages"], pre, w) for w in "kv") if pre else (None, None)
    t = 0
    for b, n in enumerate(lens):
        m = new[b]
        k, v = stored(st["pages"][b], n, "k"), stored(st["pages"][b], n, "v")
        place = torch.arange(n, device=out.device)[None] <= (n - m + torch.arange(m, device=out.device))[:, None]
        for h in range(H):
            kk, vv = (torch.cat([a[h], z[h]]) if pre else z[h] for a, z in ((kp, k), (vp, v))) if pre else (k[h], v[h])
            keep = torch.cat([torch.ones((m, pre), dtype=torch.bool, device=out.device), place], 1)
            for g in range(G):
                z = st["Q"][t:t + m, h * G + g].double() @ kk.T * st["scale"]
                z = torch.where(keep, z, torch.full_like(z, -math.inf))
                top = z.max(1, keepdim=True).values if z.shape[1] else z.new_zeros((m, 1))
                w = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
                den = w.sum(1, keepdim=True)
                out[t:t + m, h * G + g] = torch.where(den > 0, w @ vv / den.clamp(min=1e-300), torch.zeros_like(out[t:t + m, 0]))
        t += m
    return out


# --------------------------------------------------------------------- work
def work(case):
    c = case
    lens, new = _lengths(c)
    row = c["head_dim"] * c["bits"] // 8 + 4                     # one cached row: codes and constants
    held, heads = sum(lens), c["kv_heads"]
    if c["op"] in ("write", "read"):
        plain = 2 * 2 * heads * c["head_dim"]                    # K and V of a token in bf16
        n = held * (2 * heads * row + plain)
        fresh = sum(min(a, b) for a, b in zip(lens, new)) if c["op"] == "write" else 0
        return {"bytes": n + fresh * (2 * heads * row + plain), "flops": 2 * held * 2 * heads * c["head_dim"]}
    seen = sum(max(0, n - m + i + 1) for n, m in zip(lens, new) for i in range(m)) + c["prefix"] * sum(new)
    io = 2 * 2 * sum(new) * c["q_heads"] * c["head_dim"]
    return {"bytes": (held + c["prefix"]) * 2 * heads * row + io, "flops": 4 * seen * c["q_heads"] * c["head_dim"]}
