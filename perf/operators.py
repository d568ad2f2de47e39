"""Cases of the latent-cache operators: rotary positions, writing and reading
the paged cache, attention in the expanded form over per-head keys and values,
and attention in the absorbed form of few query tokens over a whole cache.

run(state) computes an operator in its plain form (elementary torch
operations in 32 bits, angles in 64), or, where `own` is true, by the calls
that a user makes of the package.  exact(case, seed) is the definition in 64
bits.
"""
import math
import random

import torch

own = False

NOPE, ROPE, V_DIM = 128, 64, 128      # expanded form: head widths
LATENT, LATENT_V = 576, 512           # absorbed form: cache row width, value columns
E4M3_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's queries far into a long context (8 sequences, 2 tokens each): latency
        dict(name="rope decode", op="rope", B=8, q_len=2, kv_len=130001, H=128, D=576, offset=512, dim=64,
             half=False, yarn=True, out="bf16", shape=1),
        # a prompt's queries turned into the native FP8 path's operand
        dict(name="rope prefill e4m3", op="rope", B=1, q_len=4096, kv_len=4096, H=128, D=576, offset=512, dim=64,
             half=True, yarn=False, out="e4m3", shape=2),
        # a decode step's latents: 16 rows normalised, rotated, scaled and written; latency
        dict(name="append decode row", op="append", B=8, q_len=2, kv_len=8192, D=576, norm=512, offset=512, dim=64,
             half=False, yarn=True, cache="row", rows=False, shape=3),
        # a long chunk's latents into a cache with block scales, kept in bf16 too for the expansion
        dict(name="append chunk block", op="append", B=8, q_len=2048, kv_len=8192, D=576, norm=512, offset=512,
             dim=64, half=False, yarn=True, cache="block", rows=True, shape=4),
        # indexer keys of a ragged batch
        dict(name="append indexer keys", op="append", B=4, q_len=2500, kv_len=4099, D=128, norm=0, offset=64, dim=64,
             half=True, yarn=False, cache="row", rows=False, shape=5),
        # one short sequence's rows back in bf16
        dict(name="gather short", op="gather", B=1, kv_len=257, D=576, cache="unit", page=64, shape=6),
        # the context of a chunk: 8 sequences of up to 8192 tokens
        dict(name="gather context", op="gather", B=8, kv_len=8192, D=576, cache="row", page=64, shape=7),
        # a few short prompts of odd lengths together
        dict(name="expanded short", op="expanded", B=5, q_len=131, kv_len=131, H=16, sink=False, shape=8),
        # one long prompt, all heads
        dict(name="expanded prompt", op="expanded", B=1, q_len=4096, kv_len=4096, H=128, sink=False, shape=9),
        # a chunk of each of four sequences over what they hold already
        dict(name="expanded chunk", op="expanded", B=4, q_len=1025, kv_len=6100, H=32, sink=True, shape=10),
        # decode with two tokens a sequence, all heads, ragged lengths
        dict(name="decode two tokens", op="decode", B=8, q_len=2, kv_len=8192, H=128, q="bf16", cache="row", page=64,
             shape=11),
        # decode of a few very long sequences with one rank's share of the heads
        dict(name="decode long", op="decode", B=4, q_len=1, kv_len=120000, H=16, q="bf16", cache="unit", page=64,
             shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "gather", "expanded", "decode"])
    shape = rng.randrange(1 << 20)
    B = _log(rng, 1, 32)
    if op == "rope":
        D, offset, dim = rng.choice([(576, 512, 64), (192, 128, 64), (128, 0, 64), (128, 64, 64), (64, 0, 64)])
        H = rng.choice([1, 8, 16, 64, 128])
        q_len = min(_log(rng, 1, 4096), max(1, 4096 * 128 * 576 // (H * D * B)))
        return dict(op=op, B=B, q_len=q_len, kv_len=q_len + _log(rng, 1, 150000), H=H, D=D, offset=offset, dim=dim,
                    half=rng.random() < 0.5, yarn=rng.random() < 0.5, out=rng.choice(["bf16", "e4m3", "f32"]),
                    shape=shape)
    if op == "append":
        latent = rng.random() < 0.7
        q_len = min(_log(rng, 1, 4096), 16384 // B)
        return dict(op=op, B=B, q_len=q_len, kv_len=q_len + _log(rng, 1, 4096), D=576 if latent else 128,
                    norm=512 if latent else 0, offset=512 if latent else rng.choice([0, 64]), dim=64,
                    half=rng.random() < 0.5, yarn=rng.random() < 0.5, cache=rng.choice(["unit", "row", "block", "bf16"]),
                    rows=rng.random() < 0.5, shape=shape)
    if op == "gather":
        return dict(op=op, B=B, kv_len=min(_log(rng, 1, 16384), 65536 // B), D=rng.choice([576, 128]),
                    cache=rng.choice(["unit", "row", "block", "bf16"]), page=rng.choice([8, 16, 64, 256]), shape=shape)
    if op == "expanded":
        H = rng.choice([1, 3, 8, 16, 32, 128])
        most = 4096 * 4096 * 128 / 2  # (token, key, head) triples of the largest listed case
        kv_len = max(1, min(_log(rng, 1, 8192), int(math.sqrt(most / (H * B)))))
        q_len = kv_len if rng.random() < 0.5 else _log(rng, 1, kv_len)
        return dict(op=op, B=B, q_len=q_len, kv_len=kv_len, H=H, sink=rng.random() < 0.3, shape=shape)
    cache = rng.choice(["unit", "row", "block", "bf16"])
    kv_len = min(_log(rng, 1, 100000), 480000 // B)
    return dict(op=op, B=B, q_len=min(rng.choice([1, 1, 2, 3, 4]), kv_len), kv_len=kv_len,
                H=rng.choice([16, 32, 48, 64, 128]),
                q="e4m3" if cache == "block" else "bf16" if cache == "bf16" else rng.choice(["bf16", "e4m3"]),
                cache=cache, page=rng.choice([16, 64, 256]), shape=shape)


def _lens(case):
    """Query and key lengths of the case's sequences: the first has the
    largest, the others spread below it (decode and append steps keep their
    q_len)."""
    rng = random.Random(case["shape"])
    kv = [case["kv_len"]] + [rng.randint(max(1, case["kv_len"] // 2), case["kv_len"]) for _ in range(case["B"] - 1)]
    if "q_len" not in case:
        return None, kv
    if case["q_len"] <= 4:
        q = [min(case["q_len"], k) for k in kv]
    else:
        q = [case["q_len"]] + [rng.randint(max(1, case["q_len"] // 2), case["q_len"]) for _ in range(case["B"] - 1)]
        q = [min(a, b) for a, b in zip(q, kv)]
    if case["op"] == "expanded" and case["q_len"] == case["kv_len"]:
        q = list(kv)
    return q, kv


def _nscale(cache, D):
    return {"unit": 0, "bf16": 0, "row": 1, "block": (D + 31) // 32}[cache]


def work(case):
    q, kv = _lens(case)
    op = case["op"]
    if op == "rope":
        n = sum(q) * case["H"]
        return {"bytes": n * case["D"] * (2 + {"bf16": 2, "e4m3": 1, "f32": 4}[case["out"]]), "flops": 3 * n * case["dim"]}
    if op in ("append", "gather"):
        rows, D = sum(q if op == "append" else kv), case["D"]
        cached = (2 if case["cache"] == "bf16" else 1) * D + 4 * _nscale(case["cache"], D)
        plain = 2 * D * (1 + int(case["rows"])) if op == "append" else 2 * D
        return {"bytes": rows * (cached + plain), "flops": rows * (4 * D if op == "append" else D)}
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))  # keys 0..pos of each token
    H = case["H"]
    if op == "expanded":
        rows = 2 * (sum(q) * H * (NOPE + ROPE + V_DIM) + sum(kv) * (H * (NOPE + V_DIM) + ROPE))
        return {"bytes": rows, "flops": 2 * H * (NOPE + ROPE + V_DIM) * pairs}
    cached = LATENT * (2 if case["cache"] == "bf16" else 1) + 4 * _nscale(case["cache"], LATENT)
    head = LATENT * (2 if case["q"] == "bf16" else 1) + 2 * LATENT_V
    return {"bytes": sum(kv) * cached + sum(q) * H * head, "flops": 2 * H * (LATENT + LATENT_V) * pairs}


# ------------------------------------------------------------------ inputs
def _cumulative(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _frequencies(dim, yarn):
    """Radians a position of each rotated pair, and the factor on the rotated
    values: base 10000, for long contexts stretched by 40 over 4096 positions
    (fast pairs keep their frequency, slow ones are divided, a linear ramp
    between 32 and 1 turns over the original length)."""
    base, factor, length = 10000.0, 40.0, 4096
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if not yarn:
        return f, 1.0
    at = [dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
    ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(dim // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def _paged(case, kv, page, gen):
    """Page table of randomly placed pages (-1 past a sequence's own), with a
    few pages of the pool that belong to no sequence."""
    pages = [-(-n // page) for n in kv]
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    width = max(pages)
    table = torch.full((len(kv), width), -1, dtype=torch.int32, device=DEV)
    own_pages = torch.arange(width, device=DEV)[None, :] < torch.tensor(pages, device=DEV)[:, None]
    table[own_pages] = perm[: sum(pages)]
    return table, total * page


def _cache_rows(x, cache):
    """A pool's bytes and scales for the float rows x [rows, D]."""
    if cache == "bf16":
        return x.to(torch.bfloat16), None
    if cache == "unit":
        return x.to(torch.float8_e4m3fn).view(torch.uint8), None
    rows, D = x.shape
    blocks = x.view(rows, -1, D if cache == "row" else 32)
    scale = blocks.abs().amax(2) / E4M3_MAX
    return (blocks / scale[:, :, None]).view(rows, D).to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous()


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    q, kv = _lens(case)
    op, s = case["op"], dict(case)
    s["kv_host"], s["q_host"] = kv, q
    s["kv"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cu_kv"] = _cumulative(kv)
    if q is not None:
        s["cu_q"], s["T"] = _cumulative(q), sum(q)
        s["positions"] = torch.cat([torch.arange(k - n, k, device=DEV) for n, k in zip(q, kv)])
    if op in ("rope", "append"):
        f, s["amplitude"] = _frequencies(case["dim"], case["yarn"])
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if op == "rope":
        s["x"] = _normal(gen, s["T"], case["H"], case["D"])
        s["table"] = torch.zeros((len(kv), 1), dtype=torch.int32, device=DEV)
        s["out_dtype"] = {"bf16": torch.bfloat16, "e4m3": torch.uint8, "f32": torch.float32}[case["out"]]
    elif op == "append":
        D = case["D"]
        s["x"] = _normal(gen, s["T"], D)
        s["weight"] = (1 + 0.1 * torch.randn(case["norm"], generator=gen, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        s["table"], n = _paged(case, kv, 64, gen)
        s["pool"] = torch.zeros((n, D), dtype=torch.bfloat16 if case["cache"] == "bf16" else torch.uint8, device=DEV)
        ns = _nscale(case["cache"], D)
        s["scales"] = torch.ones((n, ns), dtype=torch.float32, device=DEV) if ns else None
    elif op == "gather":
        s["table"], n = _paged(case, kv, case["page"], gen)
        s["pool"], s["scales"] = _cache_rows(_normal(gen, n, case["D"], dtype=torch.float32), case["cache"])
    elif op == "expanded":
        H, S = case["H"], sum(kv)
        s["q"] = _normal(gen, s["T"], H, NOPE + ROPE)
        s["kv_up"] = _normal(gen, S, H, NOPE + V_DIM)  # the up-projection's output: keys and values side by side
        s["k_rope"] = _normal(gen, S, ROPE)
        s["sinks"] = torch.randn(H, generator=gen, device=DEV) if case["sink"] else None
        s["scale"] = (NOPE + ROPE) ** -0.5
    else:
        s["table"], n = _paged(case, kv, case["page"], gen)
        s["pool"], s["scales"] = _cache_rows(_normal(gen, n, LATENT, dtype=torch.float32), case["cache"])
        x = _normal(gen, s["T"], case["H"], LATENT)
        s["q"] = x if case["q"] == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)
        s["scale"] = LATENT ** -0.5
    return s


# ------------------------------------------------------------------ plain forms
def _as_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _rotated(x, positions, inv_freq, amplitude, half):
    """x [T, ..., dim] in 32 bits, angles in 64."""
    angle = positions.double()[:, None] * inv_freq
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (-1,)
    cos, sin = (angle.cos() * amplitude).float().view(shape), (angle.sin() * amplitude).float().view(shape)
    a, b = x.chunk(2, -1) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.cat((u, v), -1) if half else torch.stack((u, v), -1).flatten(-2)


def _key_rows(s, page):
    """Physical row of every key, sequence after sequence."""
    seq = torch.repeat_interleave(torch.arange(len(s["kv_host"]), device=DEV), s["kv"].long(), output_size=sum(s["kv_host"]))
    key = torch.arange(seq.numel(), device=DEV) - s["cu_kv"].long()[seq]
    return s["table"].long()[seq, key // page] * page + key % page


def _values(s, rows):
    """What the pool's rows stand for, in 32 bits."""
    if s["cache"] == "bf16":
        return s["pool"][rows].float()
    x = s["pool"][rows].view(torch.float8_e4m3fn).float()
    if s["scales"] is None:
        return x
    sc = s["scales"][rows]
    return (x.view(x.shape[0], sc.shape[1], -1) * sc[:, :, None]).view_as(x)


def _plain_rope(s):
    x, a, b = s["x"].float(), s["offset"], s["offset"] + s["dim"]
    y = torch.cat((x[..., :a], _rotated(x[..., a:b], s["positions"], s["inv_freq"], s["amplitude"], s["half"]), x[..., b:]), -1)
    return _as_e4m3(y) if s["out"] == "e4m3" else y.to(s["out_dtype"])


def _plain_append(s):
    x, a, b, n = s["x"].float(), s["offset"], s["offset"] + s["dim"], s["norm"]
    if n:
        c = x[:, :n]
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
        x = torch.cat((c, x[:, n:]), 1)
    x = torch.cat((x[:, :a], _rotated(x[:, a:b], s["positions"], s["inv_freq"], s["amplitude"], s["half"]), x[:, b:]), 1)
    T, D = x.shape
    seq = torch.repeat_interleave(torch.arange(s["B"], device=DEV), (s["cu_q"][1:] - s["cu_q"][:-1]).long(), output_size=T)
    rows = s["table"].long()[seq, s["positions"] // 64] * 64 + s["positions"] % 64
    pool, scales = s["pool"], s["scales"]
    if s["cache"] == "bf16":
        pool[rows] = x.to(torch.bfloat16)
    else:
        y = x
        if scales is not None:
            blocks = x.view(T, scales.shape[1], -1)
            amax = blocks.abs().amax(2)
            scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), 1.0)
            scales[rows] = scale
            y = (blocks / scale[:, :, None]).view(T, D)
        pool[rows] = _as_e4m3(y).view(torch.uint8)
    return x.to(torch.bfloat16) if s["rows"] else None


def _plain_expanded(s):
    H = s["H"]
    out = torch.empty((s["T"], H, V_DIM), dtype=torch.bfloat16, device=DEV)
    q0 = k0 = 0
    for n, m in zip(s["q_host"], s["kv_host"]):
        hidden = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
        step = max(1, min(H, (1 << 29) // (n * m)))  # heads at a time: 2 GB of logits at most
        for h in range(0, H, step):
            q = s["q"][q0:q0 + n, h:h + step].float().transpose(0, 1)
            kv = s["kv_up"][k0:k0 + m, h:h + step].float().transpose(0, 1)
            z = q[..., :NOPE] @ kv[..., :NOPE].transpose(1, 2) + q[..., NOPE:] @ s["k_rope"][k0:k0 + m].float().t()
            z = (z * s["scale"]).masked_fill(hidden, -math.inf)
            top = z.amax(2, keepdim=True)
            if s["sinks"] is not None:
                top = torch.maximum(top, s["sinks"][h:h + step, None, None])
            p = torch.exp(z - top)
            total = p.sum(2, keepdim=True)
            if s["sinks"] is not None:
                total = total + torch.exp(s["sinks"][h:h + step, None, None] - top)
            out[q0:q0 + n, h:h + step] = (p @ kv[..., NOPE:] / total).transpose(0, 1).to(torch.bfloat16)
        q0, k0 = q0 + n, k0 + m
    return out


def _plain_decode(s):
    H = s["H"]
    q_all = s["q"].float() if s["q"].dtype == torch.bfloat16 else s["q"].view(torch.float8_e4m3fn).float()
    rows = _key_rows(s, s["page"])
    out = torch.empty((s["T"], H, LATENT_V), dtype=torch.bfloat16, device=DEV)
    q0 = k0 = 0
    for n, m in zip(s["q_host"], s["kv_host"]):
        c = _values(s, rows[k0:k0 + m])
        hidden = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
        z = (q_all[q0:q0 + n].reshape(n * H, LATENT) @ c.t() * s["scale"]).view(n, H, m).masked_fill(hidden[:, None], -math.inf)
        p = torch.exp(z - z.amax(2, keepdim=True))
        o = p.view(n * H, m) @ c[:, :LATENT_V] / p.sum(2).view(n * H, 1)
        out[q0:q0 + n] = o.view(n, H, LATENT_V).to(torch.bfloat16)
        q0, k0 = q0 + n, k0 + m
    return out


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import serving_fp8_indexer_gb300 as smla

    op = s["op"]
    sbs = {"unit": 0, "bf16": 0, "row": s.get("D", LATENT), "block": 32}.get(s.get("cache"), 0)
    if op in ("rope", "append"):
        rope = smla.Rope(s["inv_freq"], s["offset"], smla.ROPE_HALF if s["half"] else smla.ROPE_INTERLEAVED, s["amplitude"])
    if op == "rope":
        seqs = smla.Seqs(s["cu_q"], s["kv"], s["table"], 64, s["T"])
        out = torch.empty(s["x"].shape, dtype=s["out_dtype"], device=DEV)
        smla.rope(s["x"], seqs, rope, out)
        return out.view(torch.float8_e4m3fn) if s["out"] == "e4m3" else out
    if op == "append":
        seqs = smla.Seqs(s["cu_q"], s["kv"], s["table"], 64, s["T"])
        rows = torch.empty(s["x"].shape, dtype=torch.bfloat16, device=DEV) if s["rows"] else None
        smla.cache_append(s["x"], seqs, s["pool"], s["scales"], sbs, rope, norm_weight=s["weight"], norm_eps=1e-6, rows_out=rows)
        return rows
    if op == "gather":
        seqs = smla.Seqs(s["cu_kv"], s["kv"], s["table"], s["page"], sum(s["kv_host"]))
        rows = torch.empty((seqs.T, s["D"]), dtype=torch.bfloat16, device=DEV)
        return smla.cache_gather(s["pool"], s["scales"], sbs, seqs, rows)
    if op == "expanded":
        if "workspace" not in s:  # a serving loop keeps it
            n = smla.expanded_prefill_workspace_size(s["T"], sum(s["kv_host"]), len(s["kv_host"]), s["H"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        out = torch.empty((s["T"], s["H"], V_DIM), dtype=torch.bfloat16, device=DEV)
        return smla.expanded_prefill(s["q"], s["kv_up"][..., :NOPE], s["k_rope"], s["kv_up"][..., NOPE:], s["cu_q"],
                                     s["cu_kv"], s["scale"], out, s["workspace"], attn_sink=s["sinks"])
    seqs = smla.Seqs(s["cu_q"], s["kv"], s["table"], s["page"], s["T"])
    most = max(s["kv_host"])
    if "workspace" not in s:  # a serving loop keeps it
        n = smla.dense_decode_workspace_size(s["T"], s["H"], most)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    out = torch.empty((s["T"], s["H"], LATENT_V), dtype=torch.bfloat16, device=DEV)
    return smla.dense_decode(s["q"], s["pool"], s["scales"], sbs, seqs, most, s["scale"], out, s["workspace"])


def run(state):
    op = state["op"]
    if own:
        got = _own(state)
    elif op == "rope":
        got = _plain_rope(state)
    elif op == "append":
        got = _plain_append(state)
    elif op == "gather":
        got = _values(state, _key_rows(state, state["page"])).to(torch.bfloat16)
    elif op == "expanded":
        got = _plain_expanded(state)
    else:
        got = _plain_decode(state)
    if op != "append":
        return {"out": got}
    pool = state["pool"] if state["cache"] == "bf16" else state["pool"].view(torch.float8_e4m3fn)
    res = {"pool": pool}
    if state["scales"] is not None:
        res["scales"] = state["scales"]
    if got is not None:
        res["rows"] = got
    return res


# ------------------------------------------------------------------ the definitions, in 64 bits
def _e4m3_table():
    """The value of each e4m3 byte, from the format."""
    v = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if byte & 127 == 127 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if byte & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _turned(x, s):
    """The rotated columns of x [T, ..., D] (in 64 bits) as complex numbers
    times amplitude * exp(i angle)."""
    a, d = s["offset"], s["dim"]
    part = x[..., a:a + d]
    pairs = part.unflatten(-1, (2, d // 2)).transpose(-1, -2) if s["half"] else part.unflatten(-1, (d // 2, 2))
    z = torch.view_as_complex(pairs.contiguous())
    angle = torch.outer(s["positions"].double(), s["inv_freq"])
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)
    z = torch.view_as_real(z * turn.view((z.shape[0],) + (1,) * (z.dim() - 2) + (d // 2,)))
    y = x.clone()
    y[..., a:a + d] = (z.transpose(-1, -2) if s["half"] else z).flatten(-2)
    return y


def _decoded(s, rows):
    if s["cache"] == "bf16":
        return s["pool"][rows].double()
    x = _e4m3_table()[s["pool"][rows].long()]
    if s["scales"] is not None:
        x = x * s["scales"][rows].double().repeat_interleave(x.shape[1] // s["scales"].shape[1], 1)
    return x


def _physical(s, b, keys, page):
    return s["table"][b].long().index_select(0, torch.div(keys, page, rounding_mode="floor")) * page + keys.remainder(page)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        y = torch.cat([_turned(part, {**s, "positions": at}) for part, at in
                       zip(s["x"].split(512), s["positions"].split(512)) for part in (part.double(),)])
        return {"out": y.clamp(-E4M3_MAX, E4M3_MAX) if case["out"] == "e4m3" else y}
    if op == "append":
        x = s["x"].double()
        n = case["norm"]
        if n:
            power = torch.linalg.vector_norm(x[:, :n], dim=1, keepdim=True).square() / n
            x[:, :n] = x[:, :n] / torch.sqrt(power + 1e-6) * s["weight"].double()
        x = _turned(x, s)
        at = [_physical(s, b, s["positions"][a:e], 64) for b, (a, e) in enumerate(zip(s["cu_q"].tolist(), s["cu_q"].tolist()[1:]))]
        at = torch.cat(at)
        pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device=DEV)
        res = {"pool": pool}
        if s["scales"] is None:
            pool[at] = x
        else:
            width = case["D"] // s["scales"].shape[1]
            scale = s["scales"].double()
            most = x.abs().unfold(1, width, width).max(2).values
            scale[at] = torch.where(most > 0, most / E4M3_MAX, torch.ones_like(most))
            pool[at] = x / scale[at].repeat_interleave(width, 1)
            res["scales"] = scale
        if case["rows"]:
            res["rows"] = x
        return res
    if op == "gather":
        return {"out": torch.cat([_decoded(s, _physical(s, b, torch.arange(m, device=DEV), case["page"]))
                                  for b, m in enumerate(s["kv_host"])])}
    heads, outs, q0, k0 = case["H"], [], 0, 0
    for b, (n, m) in enumerate(zip(s["q_host"], s["kv_host"])):
        seen = torch.ones((n, m), dtype=torch.bool, device=DEV).tril(m - n)
        of_heads = []
        if op == "decode":
            c = _decoded(s, _physical(s, b, torch.arange(m, device=DEV), case["page"]))
            q_all = s["q"][q0:q0 + n].double() if case["q"] == "bf16" else _e4m3_table()[s["q"][q0:q0 + n].long()]
        for h in range(heads):
            if op == "decode":
                q, k, v = q_all[:, h], c, c[:, :LATENT_V]
            else:
                q = s["q"][q0:q0 + n, h].double()
                k = torch.cat((s["kv_up"][k0:k0 + m, h, :NOPE], s["k_rope"][k0:k0 + m]), 1).double()
                v = s["kv_up"][k0:k0 + m, h, NOPE:].double()
            z = torch.where(seen, torch.einsum("td,kd->tk", q, k) * s["scale"], -math.inf)
            if s.get("sinks") is not None:
                z = torch.cat((z, s["sinks"][h].double().expand(n, 1)), 1)
            of_heads.append(torch.softmax(z, 1)[:, :m] @ v)
        outs.append(torch.stack(of_heads, 1))
        q0, k0 = q0 + n, k0 + m
    return {"out": torch.cat(outs)}
