"""Cases of the projections around the attention calls and of the latent cache
held in 4 bits: activations quantised by blocks of 128 columns, the 8-bit matrix
product with a scale for each such block, writing and reading the 4-bit cache,
and attention of few query tokens over it.

run(state) computes an operator in its plain form (elementary torch
operations in 32 bits, angles in 64), or, where `own` is true, by the calls
that a user makes of the package.  exact(case, seed) is the definition in 64
bits.
"""
import math
import random

import torch

own = False

BLOCK = 128                       # columns of a scale of the 8-bit operands
LATENT, LATENT_V, ROTARY = 576, 512, 64
ROW = 320                         # bytes of a 4-bit cache row
CODES, SHIFTS, SIGMA = 288, 18, 308  # bytes of codes and shifts, offset of the row's scale
TOP = 384.0                       # 6 * 2^6, a row's largest value in units of its scale
E4M3_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's compressed queries, normalised on the way to their up-projection: latency
        dict(name="quantize decode norm", op="quantize", M=16, K=2048, norm=True),
        # a prompt's attention outputs, all heads, on the way to the output projection
        dict(name="quantize prompt", op="quantize", M=4096, K=16384, norm=False),
        # a decode step's output projection: the weights are what is read
        dict(name="matmul decode out", op="matmul", G=1, M=16, N=4096, K=16384, out="bf16"),
        # a decode step's queries taken into the latent space, one small product for each of 128 heads
        dict(name="matmul absorb heads", op="matmul", G=128, M=16, N=512, K=128, out="bf16"),
        # a ragged chunk's keys and values up-projected from the latents
        dict(name="matmul chunk kv up", op="matmul", G=1, M=4101, N=32768, K=512, out="bf16"),
        # a prompt's output projection
        dict(name="matmul prompt out", op="matmul", G=1, M=4096, N=4096, K=16384, out="bf16"),
        # a decode step's latents written and taken back (8 sequences, 2 tokens each): latency
        dict(name="append decode", op="append", B=8, q_len=2, kv_len=8192, norm=True, yarn=True, half=False, page=64,
             shape=1),
        # a ragged chunk's latents written, and taken back as the rows that attention reads
        dict(name="append chunk", op="append", B=8, q_len=2048, kv_len=8192, norm=True, yarn=True, half=False, page=64,
             shape=2),
        # one short sequence's rows back in 8 bits
        dict(name="gather short e4m3", op="gather", B=1, kv_len=257, rows="e4m3", page=64, shape=3),
        # the context of a chunk in bf16, for its up-projection
        dict(name="gather context", op="gather", B=8, kv_len=8192, rows="bf16", page=64, shape=4),
        # decode with two tokens a sequence, all heads, ragged lengths
        dict(name="decode two tokens", op="decode", B=8, q_len=2, kv_len=8192, H=128, q="bf16", sink=True, page=64,
             shape=5),
        # decode of a few very long sequences with one rank's share of the heads
        dict(name="decode long", op="decode", B=4, q_len=1, kv_len=120000, H=16, q="bf16", sink=False, page=64, shape=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "append", "gather", "decode", "decode"])
    if op == "quantize":
        K = 16 * _log(rng, 1, 1024)
        return dict(op=op, M=min(_log(rng, 1, 65536), max(1, 4096 * 16384 // K)), K=K, norm=rng.random() < 0.5)
    if op == "matmul":
        G = rng.choice([1, 1, 1, 8, 16, 128])
        M = _log(rng, 1, 8192 if G == 1 else 512)
        N = 8 * _log(rng, 1, 4096 if G == 1 else 128)
        K = 16 * _log(rng, 1, 1024 if G == 1 else 64)
        M = max(1, min(M, (1 << 27) // (G * N), 4096 * 4096 * 16384 // (G * N * K)))
        return dict(op=op, G=G, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]))
    shape = rng.randrange(1 << 20)
    B = _log(rng, 1, 32)
    page = rng.choice([8, 16, 64, 256])
    if op == "append":
        q_len = min(_log(rng, 1, 4096), 16384 // B)
        return dict(op=op, B=B, q_len=q_len, kv_len=q_len + _log(rng, 1, 4096), norm=rng.random() < 0.7,
                    yarn=rng.random() < 0.5, half=rng.random() < 0.5, page=page, shape=shape)
    if op == "gather":
        return dict(op=op, B=B, kv_len=min(_log(rng, 1, 16384), 65536 // B), rows=rng.choice(["bf16", "e4m3"]), page=page,
                    shape=shape)
    kv_len = min(_log(rng, 1, 100000), 480000 // B)
    return dict(op=op, B=B, q_len=min(rng.choice([1, 1, 2, 3, 4]), kv_len), kv_len=kv_len,
                H=rng.choice([16, 32, 48, 64, 128]), q=rng.choice(["bf16", "e4m3"]), sink=rng.random() < 0.3, page=page,
                shape=shape)


def _lens(case):
    """Query and key lengths of the case's sequences: the first has the
    largest, the others spread below it (decode steps keep their q_len)."""
    rng = random.Random(case["shape"])
    kv = [case["kv_len"]] + [rng.randint(max(1, case["kv_len"] // 2), case["kv_len"]) for _ in range(case["B"] - 1)]
    if "q_len" not in case:
        return None, kv
    if case["q_len"] <= 4:
        return [min(case["q_len"], k) for k in kv], kv
    q = [case["q_len"]] + [rng.randint(max(1, case["q_len"] // 2), case["q_len"]) for _ in range(case["B"] - 1)]
    return [min(a, b) for a, b in zip(q, kv)], kv


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * (3 * K + 4 * _blocks(K)) + (2 * K if case["norm"] else 0), "flops": 3 * M * K}
    if op == "matmul":
        G, M, N, K = (case[k] for k in "GMNK")
        scales = 4 * _blocks(K) * (M + _blocks(N))
        return {"bytes": G * (M * K + N * K + scales + M * N * (2 if case["out"] == "bf16" else 4)), "flops": 2 * G * M * N * K}
    q, kv = _lens(case)
    held = CODES + SHIFTS + 4
    if op == "append":  # the row in, the cache's bytes, and the row in 8 bits with its scale
        return {"bytes": sum(q) * (2 * LATENT + held + LATENT + 4), "flops": 6 * sum(q) * LATENT}
    if op == "gather":
        return {"bytes": sum(kv) * (held + (2 * LATENT if case["rows"] == "bf16" else LATENT + 4)), "flops": sum(kv) * LATENT}
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))  # keys 0..pos of each token
    H = case["H"]
    return {"bytes": sum(kv) * held + sum(q) * H * (LATENT * (2 if case["q"] == "bf16" else 1) + 2 * LATENT_V),
            "flops": 2 * H * (LATENT + LATENT_V) * pairs}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _cumulative(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _frequencies(yarn):
    """Radians a position of each rotated pair, and the factor on the rotated
    values: base 10000, for long contexts stretched by 40 over 4096 positions
    (fast pairs keep their frequency, slow ones are divided, a linear ramp
    between 32 and 1 turns over the original length)."""
    base, factor, length, dim = 10000.0, 40.0, 4096, ROTARY
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if not yarn:
        return f, 1.0
    at = [dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
    ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(dim // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def _paged(kv, page, gen):
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


def _channels(gen, K):
    """Factors of an activation's columns: most near 1, a few several times that."""
    return torch.exp(0.5 * _normal(gen, K))


def _as_bytes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _weights(gen, G, N, K):
    """Weights in 8 bits with a scale for each 128 x 128 block."""
    nb, kb = _blocks(N), _blocks(K)
    w = torch.zeros((G, nb * BLOCK, kb * BLOCK), device=DEV)
    w[:, :N, :K] = _normal(gen, G, N, K) * K ** -0.5
    tiles = w.view(G, nb, BLOCK, kb, BLOCK)
    scale = tiles.abs().amax((2, 4)) / E4M3_MAX
    w = (tiles / scale[:, :, None, :, None]).view(G, nb * BLOCK, kb * BLOCK)[:, :N, :K]
    return _as_bytes(w).view(torch.uint8).contiguous(), scale.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op == "quantize":
        M, K = case["M"], case["K"]
        s["x"] = (_normal(gen, M, K) * _channels(gen, K)).to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * _normal(gen, K)).to(torch.bfloat16) if case["norm"] else None
        return s
    if op == "matmul":
        G, M, N, K = (case[k] for k in "GMNK")
        x = _normal(gen, M, G, K) * _channels(gen, K)
        a, scales = _plain_quantize({"x": x.view(M * G, K), "weight": None})
        s["a"], s["a_scales"] = a.view(torch.uint8).view(M, G, K), scales.view(M, G, -1)  # token by token, its heads side by side
        s["b"], s["b_scales"] = _weights(gen, G, N, K)
        return s
    q, kv = _lens(case)
    s["kv_host"], s["q_host"] = kv, q
    s["kv"], s["cu_kv"] = torch.tensor(kv, dtype=torch.int32, device=DEV), _cumulative(kv)
    if q is not None:
        s["cu_q"], s["T"] = _cumulative(q), sum(q)
        s["positions"] = torch.cat([torch.arange(k - n, k, device=DEV) for n, k in zip(q, kv)])
    s["table"], n = _paged(kv, case["page"], gen)
    if op == "append":
        f, s["amplitude"] = _frequencies(case["yarn"])
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        s["x"] = _normal(gen, s["T"], LATENT).to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * _normal(gen, LATENT_V)).to(torch.bfloat16) if case["norm"] else None
        s["pool"] = torch.zeros((n, ROW), dtype=torch.uint8, device=DEV)
        return s
    s["pool"] = torch.cat([_packed(_normal(gen, part, LATENT) * _channels(gen, LATENT))
                           for part in [min(1 << 15, n - at) for at in range(0, n, 1 << 15)]])
    if op == "decode":
        x = _normal(gen, s["T"], case["H"], LATENT)
        s["q"] = x.to(torch.bfloat16) if case["q"] == "bf16" else _as_bytes(x).view(torch.uint8)
        s["sinks"] = _normal(gen, case["H"]) if case["sink"] else None
        s["scale"] = LATENT ** -0.5
    return s


# ------------------------------------------------------------------ plain forms
def _plain_quantize(s):
    x = s["x"].float()
    if s["weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    M, K = x.shape
    kb = _blocks(K)
    blocks = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    amax = blocks.abs().amax(2)
    scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), 1.0)
    return _as_bytes(blocks / scale[:, :, None]).view(M, kb * BLOCK)[:, :K].contiguous(), scale


def _plain_matmul(s):
    G, N, K = s["G"], s["N"], s["K"]
    a = s["a"].view(torch.float8_e4m3fn).float() * s["a_scales"].repeat_interleave(BLOCK, 2)[:, :, :K]
    scale = s["b_scales"].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    b = s["b"].view(torch.float8_e4m3fn).float() * scale
    out = (a[:, 0] @ b[0].t())[:, None] if G == 1 else torch.bmm(a.transpose(0, 1), b.transpose(1, 2)).transpose(0, 1)
    return out.to(torch.bfloat16 if s["out"] == "bf16" else torch.float32).contiguous()


def _power(n):
    """2^n of whole numbers n, in 32 bits."""
    return (n.int() + 127 << 23).view(torch.float32)


def _packed(x):
    """Cache rows of the float rows x [n, 576]."""
    n = x.shape[0]
    blocks = x.view(n, LATENT // 16, 16)
    top = blocks.abs().amax(2)
    most = top.amax(1)
    sigma = torch.where(most > 0, (most / TOP).clamp_min(2.0 ** -126), 1.0)
    shift = (top[:, :, None] * _power(torch.arange(1, 15, device=DEV)) <= most[:, None, None]).sum(2)
    y = blocks / sigma[:, None, None] * _power(shift - 6)[:, :, None]
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).view(n, LATENT)
    code = code | (y < 0).view(n, LATENT).byte() << 3
    shift = shift.byte()
    rows = torch.zeros((n, ROW), dtype=torch.uint8, device=DEV)
    rows[:, :CODES] = code[:, 0::2] | code[:, 1::2] << 4
    rows[:, CODES:CODES + SHIFTS] = shift[:, 0::2] | shift[:, 1::2] << 4
    rows[:, SIGMA:SIGMA + 4] = sigma.view(n, 1).view(torch.uint8)
    return rows


def _unpacked(rows):
    """Values of cache rows in units of their scale (each an e4m3 number), and the scales."""
    n = rows.shape[0]
    code = torch.stack((rows[:, :CODES] & 15, rows[:, :CODES] >> 4), 2).view(n, LATENT // 16, 16)
    shift = rows[:, CODES:CODES + SHIFTS]
    shift = torch.stack((shift & 15, shift >> 4), 2).view(n, LATENT // 16, 1)
    m, e = (code & 1).float(), code >> 1 & 3
    value = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _power(e.int() - 1))
    value = torch.where(code > 7, -value, value) * _power(6 - shift.int())
    return value.view(n, LATENT), rows[:, SIGMA:SIGMA + 4].contiguous().view(torch.float32)


def _rotated(x, positions, inv_freq, amplitude, half):
    """x [T, 64] in 32 bits, angles in 64."""
    angle = positions.double()[:, None] * inv_freq
    cos, sin = (angle.cos() * amplitude).float(), (angle.sin() * amplitude).float()
    a, b = x.chunk(2, -1) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.cat((u, v), -1) if half else torch.stack((u, v), -1).flatten(-2)


def _key_rows(s):
    """Physical row of every key, sequence after sequence."""
    seq = torch.repeat_interleave(torch.arange(len(s["kv_host"]), device=DEV), s["kv"].long(), output_size=sum(s["kv_host"]))
    key = torch.arange(seq.numel(), device=DEV) - s["cu_kv"].long()[seq]
    return s["table"].long()[seq, key // s["page"]] * s["page"] + key % s["page"]


def _plain_append(s):
    x = s["x"].float()
    c = x[:, :LATENT_V]
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    x = torch.cat((c, _rotated(x[:, LATENT_V:], s["positions"], s["inv_freq"], s["amplitude"], s["half"])), 1)
    seq = torch.repeat_interleave(torch.arange(s["B"], device=DEV), (s["cu_q"][1:] - s["cu_q"][:-1]).long(), output_size=s["T"])
    rows = s["table"].long()[seq, s["positions"] // s["page"]] * s["page"] + s["positions"] % s["page"]
    s["pool"][rows] = _packed(x)
    value, scale = _unpacked(s["pool"][rows])
    return value.to(torch.float8_e4m3fn), scale


def _plain_gather(s):
    value, scale = _unpacked(s["pool"][_key_rows(s)])
    return ((value * scale).to(torch.bfloat16), None) if s["rows"] == "bf16" else (value.to(torch.float8_e4m3fn), scale)


def _plain_decode(s):
    H = s["H"]
    q_all = s["q"].float() if s["q"].dtype == torch.bfloat16 else s["q"].view(torch.float8_e4m3fn).float()
    rows = _key_rows(s)
    out = torch.empty((s["T"], H, LATENT_V), dtype=torch.bfloat16, device=DEV)
    q0 = k0 = 0
    for n, m in zip(s["q_host"], s["kv_host"]):
        value, scale = _unpacked(s["pool"][rows[k0:k0 + m]])
        c = value * scale
        hidden = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
        z = (q_all[q0:q0 + n].reshape(n * H, LATENT) @ c.t() * s["scale"]).view(n, H, m).masked_fill(hidden[:, None], -math.inf)
        top = z.amax(2, keepdim=True)
        if s["sinks"] is not None:
            top = torch.maximum(top, s["sinks"][:, None])
        p = torch.exp(z - top)
        total = p.sum(2, keepdim=True)
        if s["sinks"] is not None:
            total = total + torch.exp(s["sinks"][:, None] - top)
        out[q0:q0 + n] = ((p.view(n * H, m) @ c[:, :LATENT_V]).view(n, H, LATENT_V) / total).to(torch.bfloat16)
        q0, k0 = q0 + n, k0 + m
    return out


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import serving_fp8_indexer_gb300 as smla

    op = s["op"]
    if op == "quantize":
        M, K = s["x"].shape
        out = torch.empty((M, K), dtype=torch.uint8, device=DEV)
        scales = torch.empty((M, _blocks(K)), dtype=torch.float32, device=DEV)
        smla.quantize_blocks(s["x"], out, scales, norm_weight=s["weight"], norm_eps=1e-6)
        return {"bytes": out.view(torch.float8_e4m3fn), "scales": scales}
    if op == "matmul":
        out = torch.empty((s["M"], s["G"], s["N"]), dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32, device=DEV)
        smla.block_matmul(s["a"].transpose(0, 1), s["a_scales"].transpose(0, 1), s["b"], s["b_scales"], out.transpose(0, 1))
        return {"out": out}
    if op == "append":
        seqs = smla.Seqs(s["cu_q"], s["kv"], s["table"], s["page"], s["T"])
        rope = smla.Rope(s["inv_freq"], LATENT_V, smla.ROPE_HALF if s["half"] else smla.ROPE_INTERLEAVED, s["amplitude"])
        smla.cache_append_fp4(s["x"], seqs, s["pool"], rope, norm_weight=s["weight"], norm_eps=1e-6)
        rows = torch.empty((s["T"], LATENT), dtype=torch.uint8, device=DEV)
        scales = torch.empty((s["T"], 1), dtype=torch.float32, device=DEV)
        smla.cache_gather_fp4(s["pool"], seqs, rows, scales)
        return {"rows": rows.view(torch.float8_e4m3fn), "scales": scales}
    if op == "gather":
        seqs = smla.Seqs(s["cu_kv"], s["kv"], s["table"], s["page"], sum(s["kv_host"]))
        if s["rows"] == "bf16":
            return {"rows": smla.cache_gather_fp4(s["pool"], seqs, torch.empty((seqs.T, LATENT), dtype=torch.bfloat16, device=DEV))}
        rows = torch.empty((seqs.T, LATENT), dtype=torch.uint8, device=DEV)
        scales = torch.empty((seqs.T, 1), dtype=torch.float32, device=DEV)
        smla.cache_gather_fp4(s["pool"], seqs, rows, scales)
        return {"rows": rows.view(torch.float8_e4m3fn), "scales": scales}
    seqs = smla.Seqs(s["cu_q"], s["kv"], s["table"], s["page"], s["T"])
    most = max(s["kv_host"])
    if "workspace" not in s:  # a serving loop keeps it
        n = smla.dense_decode_workspace_size(s["T"], s["H"], most)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    out = torch.empty((s["T"], s["H"], LATENT_V), dtype=torch.bfloat16, device=DEV)
    return {"out": smla.dense_decode_fp4(s["q"], s["pool"], seqs, most, s["scale"], out, s["workspace"], attn_sink=s["sinks"])}


def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "quantize":
        out, scales = _plain_quantize(state)
        return {"bytes": out, "scales": scales}
    if op == "matmul":
        return {"out": _plain_matmul(state)}
    if op == "decode":
        return {"out": _plain_decode(state)}
    rows, scales = _plain_append(state) if op == "append" else _plain_gather(state)
    return {"rows": rows} if scales is None else {"rows": rows, "scales": scales}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _e4m3_table():
    """The value of each e4m3 byte, from the format."""
    v = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if byte & 127 == 127 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if byte & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _e2m1_table():
    """The value of each e2m1 code, from the format."""
    v = []
    for code in range(16):
        e, m = code >> 1 & 3, code & 1
        x = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        v.append(-x if code & 8 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _decoded(rows):
    """(values in units of the row's scale, scales) of cache rows."""
    byte = rows[:, :CODES + SHIFTS].long()
    nibble = torch.empty((rows.shape[0], 2 * (CODES + SHIFTS)), dtype=torch.int64, device=DEV)
    nibble[:, 0::2], nibble[:, 1::2] = byte.remainder(16), byte.div(16, rounding_mode="floor")
    unit = torch.pow(2.0, (6 - nibble[:, LATENT:]).double())
    value = _e2m1_table()[nibble[:, :LATENT]].unflatten(1, (-1, 16)) * unit[:, :, None]
    return value.flatten(1), rows[:, SIGMA:SIGMA + 4].contiguous().view(torch.float32).double()


def _physical(s, b, keys):
    page = s["page"]
    return s["table"][b].long().index_select(0, torch.div(keys, page, rounding_mode="floor")) * page + keys.remainder(page)


def _normed(x, weight):
    power = torch.linalg.vector_norm(x, dim=1, keepdim=True).square() / x.shape[1]
    return x / torch.sqrt(power + 1e-6) * weight.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        if case["norm"]:
            x = _normed(x, s["weight"])
        scales = []
        for part in x.split(BLOCK, 1):
            most = part.abs().max(1, keepdim=True).values
            scales.append(torch.where(most > 0, most / E4M3_MAX, torch.ones_like(most)))
            part /= scales[-1]
        return {"bytes": x, "scales": torch.cat(scales, 1)}
    if op == "matmul":
        G, M, N, K = (case[k] for k in "GMNK")
        if 2.0 * G * M * N * K > 2e12:
            return None
        table = _e4m3_table()
        out = torch.zeros((M, G, N), dtype=torch.float64, device=DEV)
        for g in range(G):
            for k in range(_blocks(K)):
                at = slice(k * BLOCK, min(K, (k + 1) * BLOCK))
                a = table[s["a"][:, g, at].int()] * s["a_scales"][:, g, k, None].double()
                column = torch.cat([v.expand(n) for v, n in zip(s["b_scales"][g, :, k].double(), [len(r) for r in s["b"][g].split(BLOCK)])])
                out[:, g] += torch.einsum("mk,nk->mn", a, table[s["b"][g][:, at].int()]) * column
        return {"out": out}
    if op == "append":
        x = s["x"].double()
        if case["norm"]:
            x[:, :LATENT_V] = _normed(x[:, :LATENT_V], s["weight"])
        part = x[:, LATENT_V:]
        pairs = part.unflatten(-1, (2, ROTARY // 2)).transpose(-1, -2) if case["half"] else part.unflatten(-1, (ROTARY // 2, 2))
        angle = torch.outer(s["positions"].double(), s["inv_freq"])
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, s["amplitude"]), angle))
        x[:, LATENT_V:] = (z.transpose(-1, -2) if case["half"] else z).flatten(-2)
        most = torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True)
        top = x.abs().unfold(1, 16, 16).max(2).values
        unit = torch.pow(2.0, 6 - torch.log2(most / top).floor().clamp(0, 14)).repeat_interleave(16, 1)
        value = x / (most / TOP) / unit  # in units of the block's code, to the nearest one
        codes = _e2m1_table()[:8]
        near = codes[torch.bucketize(value.abs(), (codes[1:] + codes[:-1]) / 2)]
        return {"rows": torch.copysign(near, value) * unit, "scales": most / TOP}
    if op == "gather":
        rows = torch.cat([_physical(s, b, torch.arange(m, device=DEV)) for b, m in enumerate(s["kv_host"])])
        value, scale = _decoded(s["pool"][rows])
        return {"rows": value * scale} if case["rows"] == "bf16" else {"rows": value, "scales": scale}
    outs, q0 = [], 0
    for b, (n, m) in enumerate(zip(s["q_host"], s["kv_host"])):
        seen = torch.ones((n, m), dtype=torch.bool, device=DEV).tril(m - n)
        value, scale = _decoded(s["pool"][_physical(s, b, torch.arange(m, device=DEV))])
        c = value * scale
        q_all = s["q"][q0:q0 + n].double() if case["q"] == "bf16" else _e4m3_table()[s["q"][q0:q0 + n].long()]
        of_heads = []
        for h in range(case["H"]):
            z = torch.where(seen, torch.einsum("td,kd->tk", q_all[:, h], c) * s["scale"], -math.inf)
            if s["sinks"] is not None:
                z = torch.cat((z, s["sinks"][h].double().expand(n, 1)), 1)
            of_heads.append(torch.softmax(z, 1)[:, :m] @ c[:, :LATENT_V])
        outs.append(torch.stack(of_heads, 1))
        q0 += n
    return {"out": torch.cat(outs)}
