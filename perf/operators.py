"""The 4-bit key/value cache's operators and the norm-and-rotation before them, as measured.

Four entry points that a block of the diffusion transformer calls one after the other:
  rope    fastar_qk_norm_rope: RMS norm of every head of q and k, rotary positions of
          three axes (frame, row, column) in the same pass;
  append  fastar_kv4_append, then fastar_kv4_read of the appended rows: rows of K and V
          held in 4 bits, and the values that they stand for;
  read    fastar_kv4_read: a long range of the cache back as 16- or 32-bit rows;
  attn    fastar_kv4_attn: softmax attention over the 4-bit cache.

`run` computes them in plain torch operations (own = False) or with the library's kernels
(own = True); `exact` gives the same outputs from the definitions in 64 bits.

The 4-bit form: 16 consecutive channels share a scale s (float8 e4m3, one byte), a value is
a 4-bit float e2m1 (sign, 0 0.5 1 1.5 2 3 4 6) times s; two channels to a byte, the even one
in the low nibble.  codes uint8 [H, cap, d / 2], scales uint8 [H, cap, d / 16].
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # rope: one new token of a small model, the latency of the call
        dict(name="rope_token", kind="rope", dtype="bf16", n=1, Hq=12, Hk=12, d=128, axes="44,42,42", pos="grid",
             first=37, grid_h=30, grid_w=52),
        # a chunk of three latent frames out of a fused projection, 12 heads
        dict(name="rope_chunk", kind="rope", dtype="bf16", n=4680, Hq=12, Hk=12, d=128, axes="44,42,42", pos="grid",
             first=21, grid_h=30, grid_w=52),
        # fp32 rows of an odd count, fewer key heads, far positions given one by one, 8 channels unrotated
        dict(name="rope_far_f32", kind="rope", dtype="f32", n=1001, Hq=10, Hk=5, d=64, axes="24,16,16", pos="list",
             first=900000, grid_h=0, grid_w=0),
        # append: a chunk's keys and values of 12 heads go behind a long history
        dict(name="append_chunk", kind="append", dtype="bf16", n=4680, H=12, d=128, cap=18720, at=14040),
        # one fp32 token behind heads of different lengths
        dict(name="append_token_f32", kind="append", dtype="f32", n=1, H=8, d=64, cap=4096, at=4001),
        # read: the whole history handed over to a bf16 path
        dict(name="read_history", kind="read", dtype="bf16", n=14033, H=12, d=128, cap=14048, at=9),
        # attention of one token over a short history: the latency of the call
        dict(name="attn_token_short", kind="attn", dtype="bf16", nq=1, Hq=12, Hkv=12, d=128, cap=1024, len=333,
             ragged=False, block=0),
        # one token, 32 heads over 8 shared ones, a long history: the bandwidth of the cache
        dict(name="attn_token_long", kind="attn", dtype="bf16", nq=1, Hq=32, Hkv=8, d=128, cap=131072, len=131071,
             ragged=False, block=0),
        # a few fp32 tokens over heads of different lengths (one of them empty), 64 channels
        dict(name="attn_ragged_f32", kind="attn", dtype="f32", nq=5, Hq=16, Hkv=4, d=64, cap=8192, len=7777,
             ragged=True, block=0),
        # an odd number of tokens, each seeing only what came before it, 64 channels
        dict(name="attn_causal_odd", kind="attn", dtype="bf16", nq=331, Hq=16, Hkv=8, d=64, cap=4096, len=3001,
             ragged=True, block=1),
        # the first chunk of a rollout, each latent frame seeing itself and the frames before it
        dict(name="attn_frames", kind="attn", dtype="bf16", nq=4680, Hq=12, Hkv=12, d=128, cap=18720, len=4680,
             ragged=False, block=1560),
        # a chunk over the whole history of 60 latent frames
        dict(name="attn_chunk_long", kind="attn", dtype="bf16", nq=4680, Hq=12, Hkv=12, d=128, cap=93600, len=93600,
             ragged=False, block=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pad16(n):
    return (n + 15) // 16 * 16


def draw(rng):
    kind = rng.choice(["rope", "append", "read", "attn", "attn", "attn", "attn"])
    if kind == "rope":
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 4, 5, 8, 12, 24])
        part = 2 * rng.randint(0, d // 6)
        part2 = 2 * rng.randint(0, d // 6)
        axes = (2 * rng.randint(0, (d - part - part2) // 2), part, part2)
        return dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), n=_log(rng, 1, 9000), Hq=Hk * rng.choice([1, 2]),
                    Hk=Hk, d=d, axes="%d,%d,%d" % axes, pos=rng.choice(["grid", "list"]), first=_log(rng, 1, 1000000),
                    grid_h=rng.randint(1, 45), grid_w=rng.randint(1, 80))
    if kind in ("append", "read"):
        n, at = _log(rng, 1, 15000), _log(rng, 1, 30000)
        return dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), n=n, H=rng.choice([1, 3, 8, 12, 24]),
                    d=rng.choice([64, 128]), cap=_pad16(n + at + rng.randint(0, 500)), at=at)
    f32 = rng.random() < 0.15
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 8, 12])
    G = rng.choice([1, 1, 2, 4])
    if f32:
        nq, length = _log(rng, 1, 16), _log(rng, 1, 8192)
    elif rng.random() < 0.5:
        nq, length = _log(rng, 1, 64), _log(rng, 1, 131072)
    else:
        nq, length = _log(rng, 64, 9000), _log(rng, 64, 93600)
        most = 4680 * 93600 * 12 // (Hkv * G)          # no more pairs than the largest listed case
        length = max(1, min(length, most // nq))
    return dict(kind=kind, dtype="f32" if f32 else "bf16", nq=nq, Hq=Hkv * G, Hkv=Hkv, d=d,
                cap=_pad16(length + rng.randint(0, 300)), len=length, ragged=rng.random() < 0.4,
                block=rng.choice([0, 0, 1, max(1, nq // 3)]))


# ---- the inputs --------------------------------------------------------------------------------

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000 + salt)


def _rows(H, n, d, seed, salt, std=1.0):
    """fp32 rows [H, n, d] as the projections give them: normal, with a few strong channels."""
    g = _gen(seed, salt)
    x = torch.randn(H, n, d, generator=g, device="cuda")
    ch = 1.0 + 2.0 * (torch.rand(H, 1, d, generator=g, device="cuda") > 0.97)
    return x.mul_(ch).mul_(std)


def _lens(case, seed):
    if not case["ragged"]:
        return [case["len"]] * case["Hkv"]
    r = torch.rand(case["Hkv"], generator=torch.Generator().manual_seed(seed)).tolist()
    lens = [int(round(case["len"] * x)) for x in r]
    lens[0] = case["len"]
    if len(lens) > 1:
        lens[1] = 0                     # a head that has seen nothing yet
    return lens


def _starts(case, seed):
    """First row of each head: the heads' lengths differ by a few tokens."""
    r = torch.rand(case["H"], generator=torch.Generator().manual_seed(seed)).tolist()
    return [case["at"] - int(min(case["at"], 40) * x) for x in r]


def _axes(case):
    return tuple(int(a) for a in case["axes"].split(","))


def prepare(case, seed):
    dt = _DT[case["dtype"]]
    s = {"case": dict(case)}
    if case["kind"] == "rope":
        n, Hq, Hk, d = case["n"], case["Hq"], case["Hk"], case["d"]
        qkv = _rows(1, n, (Hq + 2 * Hk) * d, seed, 1, 2.0).view(n, (Hq + 2 * Hk), d).to(dt)   # a fused projection
        s["q"], s["k"] = qkv[:, :Hq].transpose(0, 1), qkv[:, Hq:Hq + Hk].transpose(0, 1)
        s["wq"] = 1 + 0.1 * torch.randn(d, generator=_gen(seed, 2), device="cuda")
        s["wk"] = 1 + 0.1 * torch.randn(d, generator=_gen(seed, 3), device="cuda")
        s["q_out"] = torch.empty(Hq, n, d, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(Hk, n, d, dtype=dt, device="cuda")
        s["first"] = case["first"] + seed % 5
        if case["pos"] == "list":
            s["pos"] = torch.randint(0, s["first"] + 1, (n, 3), generator=_gen(seed, 4), device="cuda",
                                     dtype=torch.int32)
        return s
    if case["kind"] in ("append", "read"):
        H, n, d, cap = case["H"], case["n"], case["d"], case["cap"]
        x = _rows(2, n, H * d, seed, 1).view(2, n, H, d).to(dt)       # token-major, as the projection leaves them
        s["k"], s["v"] = x[0].transpose(0, 1), x[1].transpose(0, 1)
        for t in "kv":
            s[t + "c"] = torch.zeros(H, cap, d // 2, dtype=torch.uint8, device="cuda")
            s[t + "s"] = torch.zeros(H, cap, d // 16, dtype=torch.uint8, device="cuda")
            s[t + "_out"] = torch.empty(H, n, d, dtype=dt, device="cuda")
        if case["kind"] == "read":
            for t in "kv":
                c, sc = _quantise(s[t])
                s[t + "c"][:, case["at"]:case["at"] + n] = c
                s[t + "s"][:, case["at"]:case["at"] + n] = sc
            return s
        s["starts"] = _starts(case, seed)
        s["at"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
        s["len_out"] = torch.zeros(H, dtype=torch.int32, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["first"] = case["at"] - min(case["at"], 40)
        s["span"] = n + min(case["at"], 40)
        for t in "kv":
            s[t + "_out"] = torch.empty(H, s["span"], d, dtype=dt, device="cuda")
        return s
    Hq, Hkv, d, nq, cap = case["Hq"], case["Hkv"], case["d"], case["nq"], case["cap"]
    s["q"] = _rows(1, nq, Hq * d, seed, 1, 1.5).view(nq, Hq, d).to(dt).transpose(0, 1)        # token-major
    s["lens_host"] = _lens(case, seed)
    s["lens"] = torch.tensor(s["lens_host"], dtype=torch.int32, device="cuda")
    for i, t in enumerate("kv"):
        s[t + "c"] = torch.empty(Hkv, cap, d // 2, dtype=torch.uint8, device="cuda")
        s[t + "s"] = torch.empty(Hkv, cap, d // 16, dtype=torch.uint8, device="cuda")
        for h in range(Hkv):
            c, sc = _quantise(_rows(1, cap, d, seed, 100 + 2 * h + i).to(dt))
            s[t + "c"][h], s[t + "s"][h] = c[0], sc[0]
    s["out"] = torch.empty(nq, Hq, d, dtype=dt, device="cuda").transpose(0, 1)
    s["lse"] = torch.empty(Hq, nq, dtype=torch.float32, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        from kv_cache_tempcache_gb300 import _lib as L
        nb = L.workspace_bytes(L.OP_KV4_ATTN, Hq, nq, cap, d, Hkv)
        s["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None
    return s


# ---- plain forms -----------------------------------------------------------------------------------

def _quantise(x):
    """codes, scales of rows x [H, n, d]; 64 bits, because a scale or a code that lies on a
    border between two has to fall to the right side."""
    H, n, d = x.shape
    y = x.double().reshape(H, n, d // 16, 16)
    a = y.abs().amax(-1) / 6
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6.0, max=8.0)
    step = torch.exp2(e - 3)
    sc = (torch.round(a / step) * step).clamp(max=448.0).float().to(torch.float8_e4m3fn)      # exact cast
    sd = sc.double()[..., None]
    m = torch.where(sd > 0, y.abs() / sd, torch.zeros_like(y))
    code = torch.where(m < 2, torch.round(m * 2), torch.where(m < 4, torch.round(m) + 2, torch.round(m / 2) + 4))
    code = code.clamp(max=7).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.reshape(H, n, d // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), sc.view(torch.uint8)


def _values(codes, scales, dtype=torch.float32):
    """The values that rows of the cache stand for, [..., d]."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype,
                        device=codes.device)
    idx = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    v = grid[idx]
    sc = scales.view(torch.float8_e4m3fn).to(dtype)
    return v * sc.repeat_interleave(16, -1)


def _positions(s):
    c = s["case"]
    if c["pos"] == "list":
        return s["pos"].double()
    i = torch.arange(c["n"], device="cuda")
    gh, gw = c["grid_h"], c["grid_w"]
    return torch.stack((s["first"] + i // (gh * gw), (i // gw) % gh, i % gw), -1).double()


def _rope_plain(s, x, w):
    c, pos = s["case"], _positions(s)
    x = x.float()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    at = 0
    parts = []
    for a, width in enumerate(_axes(c)):
        f = 10000.0 ** (-torch.arange(0, width, 2, device="cuda", dtype=torch.float64) / max(width, 1))
        ang = pos[:, a:a + 1] * f                    # far positions: 64 bits
        cs, sn = torch.cos(ang).float(), torch.sin(ang).float()
        e, o = x[..., at:at + width:2], x[..., at + 1:at + width:2]
        parts.append(torch.stack((e * cs - o * sn, e * sn + o * cs), -1).flatten(-2))
        at += width
    parts.append(x[..., at:])
    return torch.cat(parts, -1).to(_DT[c["dtype"]])


def _limits(case, length):
    """How many keys each of the nq tokens of a head with `length` cached rows sees."""
    nq, block = case["nq"], case["block"]
    if not block:
        return None
    t = torch.arange(nq, device="cuda")
    end = torch.clamp((t // block + 1) * block, max=nq)
    return torch.clamp(length - nq + end, min=0, max=length)


def _attn_plain(s):
    c = s["case"]
    G, nq, d = c["Hq"] // c["Hkv"], c["nq"], c["d"]
    out, lse = torch.zeros(c["Hq"], nq, d, device="cuda"), torch.full((c["Hq"], nq), -math.inf, device="cuda")
    for h, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        k = _values(s["kc"][h, :n], s["ks"][h, :n])
        v = _values(s["vc"][h, :n], s["vs"][h, :n])
        lim = _limits(c, n)
        for g in range(h * G, (h + 1) * G):
            x = s["q"][g].float() @ k.t()
            x *= 1.0 / math.sqrt(d)
            if lim is not None:
                x.masked_fill_(torch.arange(n, device="cuda")[None] >= lim[:, None], -math.inf)
            m = x.amax(-1, keepdim=True).clamp(min=-3e38)
            x = x.sub_(m).exp_()
            l = x.sum(-1, keepdim=True)
            out[g] = (x @ v) / l.clamp(min=1e-30)
            lse[g] = (m + torch.log(l))[:, 0]
    return out.to(_DT[c["dtype"]]), lse


def _plain(s):
    c = s["case"]
    if c["kind"] == "rope":
        return _rope_plain(s, s["q"], s["wq"]), _rope_plain(s, s["k"], s["wk"])
    if c["kind"] == "read":
        r = slice(c["at"], c["at"] + c["n"])
        return tuple(_values(s[t + "c"][:, r], s[t + "s"][:, r]).to(_DT[c["dtype"]]) for t in "kv")
    if c["kind"] == "append":
        outs = []
        for t in "kv":
            codes, scales = _quantise(s[t])
            for h, a in enumerate(s["starts"]):
                s[t + "c"][h, a:a + c["n"]] = codes[h]
                s[t + "s"][h, a:a + c["n"]] = scales[h]
            r = slice(s["first"], s["first"] + s["span"])
            outs.append(_values(s[t + "c"][:, r], s[t + "s"][:, r]).to(_DT[c["dtype"]]))
        return outs[0], outs[1], s["at"] + c["n"]
    return _attn_plain(s)


# ---- one pass -----------------------------------------------------------------------------------------

def run(s):
    if not own:
        return _plain(s)
    from kv_cache_tempcache_gb300 import _lib as L
    c = s["case"]
    if c["kind"] == "rope":
        if c["pos"] == "list":
            L.fastar_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], wq=s["wq"], wk=s["wk"], eps=1e-6,
                                  axes=_axes(c), pos=s["pos"])
        else:
            L.fastar_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], wq=s["wq"], wk=s["wk"], eps=1e-6,
                                  axes=_axes(c), t0=s["first"], grid=(c["grid_h"], c["grid_w"]))
        return s["q_out"], s["k_out"]
    if c["kind"] == "append":
        L.fastar_kv4_append(s["k"], s["v"], s["kc"], s["ks"], s["vc"], s["vs"], s["at"], s["len_out"], s["status"])
        L.fastar_kv4_read(s["kc"], s["ks"], s["first"], s["k_out"])
        L.fastar_kv4_read(s["vc"], s["vs"], s["first"], s["v_out"])
        return s["k_out"], s["v_out"], s["len_out"]
    if c["kind"] == "read":
        L.fastar_kv4_read(s["kc"], s["ks"], c["at"], s["k_out"])
        L.fastar_kv4_read(s["vc"], s["vs"], c["at"], s["v_out"])
        return s["k_out"], s["v_out"]
    L.fastar_kv4_attn(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["lens"], 1.0 / math.sqrt(c["d"]), s["out"],
                      s["lse"], block=c["block"], dev_status=s["status"], workspace=s["ws"])
    return s["out"], s["lse"]


# ---- what a pass cannot do without -------------------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "rope":
        el = case["n"] * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": 2 * el * es + 8 * case["d"] + (12 * case["n"] if case["pos"] == "list" else 0),
                "flops": 10 * el}
    if case["kind"] in ("append", "read"):
        el = 2 * case["n"] * case["H"] * case["d"]
        packed = el // 2 + el // 16
        if case["kind"] == "read":
            return {"bytes": packed + el * es, "flops": el}
        return {"bytes": 2 * (el * es + packed), "flops": 4 * el}
    d, nq, G = case["d"], case["nq"], case["Hq"] // case["Hkv"]
    lens = [case["len"]] * case["Hkv"]
    if case["ragged"]:                                    # half full on average, one head full, one empty
        lens = [case["len"]] + [0] * (case["Hkv"] > 1) + [case["len"] // 2] * max(0, case["Hkv"] - 2)
    pairs, rows = 0, 0
    for n in lens:
        rows += n
        if case["block"]:
            b = case["block"]
            for t0 in range(0, nq, b):
                pairs += (min(nq, t0 + b) - t0) * max(0, n - nq + min(nq, t0 + b))
        else:
            pairs += nq * n
    return {"bytes": 2 * rows * (d // 2 + d // 16) + 2 * case["Hq"] * nq * d * es + 4 * case["Hq"] * nq,
            "flops": 4 * d * G * pairs}


# ---- the definitions in 64 bits -------------------------------------------------------------------------

_MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_values(x):
    """The values that the 4-bit form of rows x [H, n, d] stands for, by search: the nearest of
    the representable scales, the nearest of the representable values, the even one of two."""
    H, n, d = x.shape
    y = x.double().reshape(H, n, d // 16, 16)
    e4m3 = torch.tensor([(m / 8) * 2.0 ** -6 for m in range(8)]
                        + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=x.device)
    s = e4m3[_nearest(y.abs().amax(-1), 6 * e4m3)][..., None]
    mag = torch.tensor(_MAG, dtype=torch.float64, device=x.device)
    code = torch.zeros_like(y, dtype=torch.long)
    for i in range(7):                                    # past the middle of i and i + 1 (at it: to the even one)
        mid = (mag[i] + mag[i + 1]) / 2 * s
        code += ((y.abs() > mid) | ((y.abs() == mid) & (i % 2 == 1) & (s > 0))).long()
    return (torch.sign(y) * mag[code] * s).reshape(H, n, d)


def _nearest(a, grid):
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_unpack(codes, scales):
    """Rows of the cache from the bits: sign, two bits of exponent, one of mantissa; the scale
    sign-less with four and three."""
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    for i in (0, 1):
        b = (codes.int() >> (4 * i)) & 15
        e, m = (b >> 1) & 3, (b & 1).double()
        mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
        out[..., i::2] = torch.where(b >= 8, -mag, mag)
    b = scales.int()
    e, m = b >> 3, (b & 7).double()
    sc = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    return (out.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        outs = []
        pos = _positions(s)
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            x = x.double()
            y = x * w.double() * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6)
            z = y.clone()
            at = 0
            for a, width in enumerate(_axes(case)):
                for j in range(width // 2):
                    ang = pos[:, a] * math.exp(-2 * j / width * math.log(10000.0))
                    c0, c1 = at + 2 * j, at + 2 * j + 1
                    z[..., c0] = y[..., c0] * torch.cos(ang) - y[..., c1] * torch.sin(ang)
                    z[..., c1] = y[..., c0] * torch.sin(ang) + y[..., c1] * torch.cos(ang)
                at += width
            outs.append(z)
        return tuple(outs)
    if case["kind"] == "read":
        r = slice(case["at"], case["at"] + case["n"])
        return tuple(_exact_unpack(s[t + "c"][:, r], s[t + "s"][:, r]) for t in "kv")
    if case["kind"] == "append":
        outs = []
        for t in "kv":
            full = torch.zeros(case["H"], s["span"], case["d"], dtype=torch.float64, device="cuda")
            vals = _exact_values(s[t])
            for h, a in enumerate(s["starts"]):
                full[h, a - s["first"]:a - s["first"] + case["n"]] = vals[h]
            outs.append(full)
        return outs[0], outs[1], torch.tensor(s["starts"], device="cuda", dtype=torch.int32) + case["n"]
    if 4 * case["d"] * case["Hq"] * case["nq"] * case["len"] > 4e12:
        return None
    Hq, nq, d = case["Hq"], case["nq"], case["d"]
    G = Hq // case["Hkv"]
    out = torch.zeros(Hq, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    b = case["block"]
    for h, n in enumerate(s["lens_host"]):
        k, v = _exact_unpack(s["kc"][h, :n], s["ks"][h, :n]), _exact_unpack(s["vc"][h, :n], s["vs"][h, :n])
        for t0 in range(0, nq, 512):
            t = torch.arange(t0, min(nq, t0 + 512), device="cuda")
            see = torch.full_like(t, n) if not b else (n - nq + torch.clamp(t - t % b + b, max=nq)).clamp(min=0)
            for g in range(h * G, (h + 1) * G):
                logit = s["q"][g, t].double() @ k.t() / math.sqrt(d)
                logit[torch.arange(n, device="cuda").expand(len(t), n) >= see[:, None]] = -math.inf
                lse[g, t] = torch.logsumexp(logit, -1)
                out[g, t] = torch.softmax(logit, -1).nan_to_num(0.0) @ v      # a token that sees nothing: 0
    return out, lse
