"""The operators around the integer decode, as a serving loop calls them.

  norm    qk_norm_rope: the norm of each query and key head and the position rotation, in one pass
  cache   cache_write, then cache_read of the rows just written: new K / V rows quantised with the caches' fixed
          scales into int8 or int4 caches (with the keys' norm and rotation in the same pass where the case says
          so), and the values those codes stand for
  shared  decode_shared: one query per (sequence, head) against a prefix that all sequences share followed by a
          cache of each sequence's own

Each has a plain form here (elementary torch operations) and the framework's call (``own``).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence through a 12-head layer (GPT-2 small heads): launch latency
        norm_case("norm_token_h12_d64", 1, 12, 12, 1, 64, 64, "fp16", False, 700),
        # a ragged batch with grouped heads, half of each head rotated, interleaved pairs
        norm_case("norm_b5_l197_gqa_partial", 5, 12, 4, 197, 128, 64, "bf16", True, 9000),
        # the prefill of a LLaMA-7B layer, far positions
        norm_case("norm_llama7b_l8192", 1, 32, 32, 8192, 128, 128, "bf16", False, 57000),
        # one decode step of 64 sequences with grouped heads: norm, rotation and quantising in one pass
        cache_case("cache_step_b64_gqa_norm", 64, 32, 8, 1, 4096, 128, "bf16", 8, False, True),
        # a ragged batch of prompts into an int4 cache with zero-points
        cache_case("cache_int4_zp_b6_l333", 6, 12, 12, 333, 1024, 64, "fp16", 4, True, False),
        # prompts of a LLaMA-7B layer into an int8 cache
        cache_case("cache_llama7b_b4_l4096", 4, 32, 32, 4096, 4096, 128, "bf16", 8, False, False),
        # a few sequences behind a short system prompt (GPT-2 small heads)
        shared_case("shared_b4_h12_l500", 4, 12, 12, 500, 64, 64, False),
        # grouped heads, a batch of 64 behind a long document
        shared_case("shared_b64_gqa_l8192", 64, 32, 8, 8192, 1024, 128, False),
        # LLaMA-7B heads (one K / V head per query head), u8 codes with zero-points, odd lengths
        shared_case("shared_llama7b_zp_l4001", 64, 32, 32, 4001, 777, 128, True),
        # few sequences behind a very long prefix
        shared_case("shared_b9_gqa_l50000", 9, 32, 8, 50000, 333, 128, False),
    ]


def norm_case(name, B, H, Hkv, L, d, rot, dtype, interleaved, first):
    return {"name": name, "op": "norm", "B": B, "H": H, "Hkv": Hkv, "L": L, "d": d, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "first": first}


def cache_case(name, B, H, Hkv, L, Lmax, d, dtype, bits, zp, norm):
    return {"name": name, "op": "cache", "B": B, "H": H, "Hkv": Hkv, "L": L, "Lmax": Lmax, "d": d, "dtype": dtype,
            "bits": bits, "zp": zp, "norm": norm}


def shared_case(name, B, H, Hkv, Lp, Lmax, d, zp):
    return {"name": name, "op": "shared", "B": B, "H": H, "Hkv": Hkv, "Lp": Lp, "Lmax": Lmax, "d": d, "zp": zp}


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def batch(most, room):
        most = max(1, min(most, room))
        return size(max(1, most // 16), most)

    op = rng.choice(["norm", "cache", "shared", "shared"])
    d = rng.choice([64, 128])
    Hkv = size(2, 32)
    G = rng.choice([1, 1, 2, 3, 4, 8]) if Hkv <= 12 else 1
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm":
        L = rng.choice([1, size(8, 8192), size(8, 8192)])
        B = batch(64, 260000 // (L * Hkv * (G + 1)))
        rot = rng.choice([d, d, d // 2, 16])
        c = norm_case("", B, Hkv * G, Hkv, L, d, rot, dtype, rng.choice([False, True]), rng.randrange(0, 50000))
    elif op == "cache":
        L = rng.choice([1, size(8, 4096), size(8, 4096)])
        B = batch(64, 260000 // (L * Hkv))
        c = cache_case("", B, Hkv * G, Hkv, L, L + rng.randrange(0, 300), d, dtype, rng.choice([8, 4]),
                       rng.choice([False, True]), rng.choice([False, True]))
    else:
        Lp = size(30, 60000)
        B = batch(64, 16000000 // (Hkv * G * Lp))
        Lmax = size(8, max(8, min(1024, 40000000 // (B * Hkv * 64))))
        c = shared_case("", B, Hkv * G, Hkv, Lp, Lmax, d, rng.choice([False, True]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def projection(g, B, L, heads, d, dtype):
    """A packed q / k / v projection's output [B, L, heads * d] with some outlier channels, as per-head views [B, h, L, d]."""
    x = torch.randn((B, L, sum(heads) * d), generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((sum(heads) * d,), generator=g, device="cuda"))
    x = x.to(dtype).view(B, L, sum(heads), d)
    return [t.transpose(1, 2) for t in x.split(list(heads), dim=2)]


def rotation_table(positions, rot):
    """[positions, rot / 2, 2]: cos and sin of position * 10000^(-2 i / rot), the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).to(torch.float32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    s = {"case": case}
    if case["op"] == "shared":
        return prepare_shared(case, g, s)
    dtype = DTYPES[case["dtype"]]
    L = case["L"]
    s["q"], s["k"], s["v"] = projection(g, B, L, (H, Hkv, Hkv), d, dtype)
    if case["op"] == "norm":
        rot, reach = case["rot"], case["first"] + 1000 + L
        start = case["first"] + torch.randint(0, 1000, (B,), generator=g, device="cuda")
    else:
        rot, reach = d, case["Lmax"]
        start = torch.randint(0, case["Lmax"] - L + 1, (B,), generator=g, device="cuda")
    s["start"] = start.to(torch.int32)
    if case["op"] == "norm" or case["norm"]:
        s["table"] = rotation_table(reach, rot)
        s["positions"] = (start[:, None] + torch.arange(L, device="cuda")).to(torch.int32).contiguous()
        s["w_q"], s["w_k"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda") for _ in range(2))
    if case["op"] == "cache":
        # the fixed scales of the caches: most values inside the range, the largest saturate
        bits, zp = case["bits"], case["zp"]
        head = torch.rand((2, Hkv), generator=g, device="cuda", dtype=torch.float32).cpu()
        width = 5.0 + 3.0 * head
        steps = float(2 ** bits - 1) if zp else float(2 ** (bits - 1) - 1)
        s["s_k"], s["s_v"] = ((w * (2.0 if zp else 1.0) / steps).numpy() for w in width)
        s["z_k"] = s["z_v"] = None
        if zp:
            z = 2 ** (bits - 1) + torch.randint(-2, 3, (2, Hkv), generator=g, device="cuda").cpu()
            s["z_k"], s["z_v"] = (t.to(torch.int32).numpy() for t in z)
        shape = (B, Hkv, case["Lmax"], d * bits // 8)
        code = torch.uint8 if zp or bits == 4 else torch.int8
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=code, device="cuda") for _ in range(2))
    return s


def prepare_shared(case, g, s):
    """Codes of N(0, 1) draws; logits of spread 3, so that a few keys of a long row carry its weight."""
    B, H, Hkv, Lp, Lmax, d, zp = (case[n] for n in ("B", "H", "Hkv", "Lp", "Lmax", "d", "zp"))

    def codes(shape, z):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(28.0).round_()
        if z is None:
            return x.clamp_(-127, 127).to(torch.int8)
        return x.add_(torch.as_tensor(z, device="cuda", dtype=torch.float32).view(-1, 1, 1)).clamp_(0, 255).to(torch.uint8)

    z = torch.randint(110, 146, (2, Hkv), generator=g, device="cuda").cpu().to(torch.int32).numpy()
    s["z_k"], s["z_v"] = z if zp else (None, None)
    s["q"] = codes((B, H, 1, d), None)
    s["k_prefix"], s["v_prefix"] = (codes((Hkv, Lp, d), t) for t in (s["z_k"], s["z_v"]))
    s["k_cache"], s["v_cache"] = (codes((B, Hkv, Lmax, d), t) for t in (s["z_k"], s["z_v"]))
    s["lengths"] = torch.randint(0, Lmax + 1, (B,), generator=g, device="cuda").to(torch.int32)
    wobble = torch.rand((4, H), generator=g, device="cuda", dtype=torch.float32).cpu().numpy() * 0.2 + 0.9
    s["s_q"] = wobble[0] * (math.sqrt(3.0) / 28.0)
    s["s_k"] = wobble[1, :Hkv] * (math.sqrt(3.0) / 28.0)
    s["s_v"] = wobble[2, :Hkv] / 28.0
    s["s_o"] = wobble[3] * (3.0 / 127.0)
    s["clip_c"] = 10.0
    return s


# --------------------------------------------------------------- one pass
def run(s):
    return {"norm": run_norm, "cache": run_cache, "shared": run_shared}[s["case"]["op"]](s)


def run_norm(s):
    if own:
        import integer_only_quantized_b200 as ia
        rn = ia.RopeNorm(s["table"], s["positions"], w_q=s["w_q"], w_k=s["w_k"], eps=1e-6,
                         interleaved=s["case"]["interleaved"])
        return ia.qk_norm_rope(s["q"], s["k"], rn)
    case = s["case"]
    return tuple(plain_norm(x, w, s["table"], s["positions"], case["interleaved"]).to(x.dtype)
                 for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])))


def plain_norm(x, w, table, positions, interleaved):
    x = x.to(torch.float32)
    y = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)) * w
    rot = 2 * table.shape[1]
    cs = table[positions.long()][:, None]  # [B, 1, L, rot / 2, 2]
    c, n = cs[..., 0], cs[..., 1]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat([a * c - b * n, a * n + b * c], -1)
    return torch.cat([r, y[..., rot:]], -1)


def run_cache(s):
    case = s["case"]
    bits, L = case["bits"], case["L"]
    dtype = DTYPES[case["dtype"]]
    if own:
        import integer_only_quantized_b200 as ia
        sc = ia.Scales(1.0, s["s_k"], s["s_v"], 1.0, per_head=True, z_k=s["z_k"], z_v=s["z_v"])
        rn = ia.RopeNorm(s["table"], s["positions"], w_k=s["w_k"], eps=1e-6) if case["norm"] else None
        ia.cache_write(s["k"], s["v"], sc, s["k_cache"], s["v_cache"], s["start"], bits=bits, norm=rn)
        return ia.cache_read(s["k_cache"], s["v_cache"], sc, s["start"], L, bits=bits, dtype=dtype)
    k = plain_norm(s["k"], s["w_k"], s["table"], s["positions"], False) if case["norm"] else s["k"].to(torch.float32)
    return (plain_cache(k, s["s_k"], s["z_k"], s["k_cache"], s["start"], bits).to(dtype),
            plain_cache(s["v"].to(torch.float32), s["s_v"], s["z_v"], s["v_cache"], s["start"], bits).to(dtype))


def plain_cache(x, scale, zero, cache, start, bits):
    """Codes of x [B, H, L, d] into the cache rows start[b] + t, and the values of those rows read back."""
    B, H, L, d = x.shape
    sc = torch.as_tensor(scale, device=x.device).view(1, H, 1, 1)
    c = torch.round(x * (1.0 / sc))
    if zero is None:
        z = 0.0
        top = 2 ** (bits - 1) - 1
        c = c.clamp(-top, top)
    else:
        z = torch.as_tensor(zero, device=x.device, dtype=torch.float32).view(1, H, 1, 1)
        c = (c + z).clamp(0, 2 ** bits - 1)
    c = c.to(torch.int16)
    if bits == 4:
        c = (c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)
    b = torch.arange(B, device=x.device)[:, None, None]
    h = torch.arange(H, device=x.device)[None, :, None]
    rows = (start.long()[:, None] + torch.arange(L, device=x.device))[:, None, :]
    cache[b, h, rows] = c.to(cache.dtype)
    c = cache[b, h, rows]
    if bits == 4:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).to(torch.float32)
        c = c if zero is not None else torch.where(c >= 8, c - 16, c)
    return (c.to(torch.float32) - z) * sc


def run_shared(s):
    case = s["case"]
    if own:
        import integer_only_quantized_b200 as ia
        sc = ia.Scales(s["s_q"], s["s_k"], s["s_v"], s["s_o"], per_head=True, z_k=s["z_k"], z_v=s["z_v"])
        return ia.decode_shared(s["q"], s["k_prefix"], s["v_prefix"], s["k_cache"], s["v_cache"], s["lengths"], sc,
                                s["clip_c"], dtype=torch.bfloat16)
    B, H, Hkv, Lp, Lmax, d = (case[n] for n in ("B", "H", "Hkv", "Lp", "Lmax", "d"))
    G = H // Hkv
    dev = s["q"].device
    par = torch.tensor([head_parameters(s, h, G, d) for h in range(H)], device=dev).view(1, Hkv, G, 5)
    lut = torch.round(32768.0 * torch.exp(torch.arange(32, device=dev, dtype=torch.float64) * (-s["clip_c"] / 31)))
    lut = (lut * (torch.arange(32, device=dev) < 31)).long()
    q = s["q"].view(B, Hkv, G, d).to(torch.float32)

    def codes(x, z):
        x = x.to(torch.float32)
        return x if z is None else x - torch.as_tensor(z, device=dev, dtype=torch.float32).view(Hkv, 1, 1)

    # whole numbers below 2^24 throughout both products, so that 32-bit floats hold them exactly
    sp = torch.einsum("bhgd,hkd->bhgk", q, codes(s["k_prefix"], s["z_k"]))
    ss = torch.einsum("bhgd,bhkd->bhgk", q, codes(s["k_cache"], s["z_k"]))
    seen = torch.arange(Lmax, device=dev) < s["lengths"].view(B, 1, 1, 1)
    score = torch.cat([sp, ss.masked_fill(~seen, -math.inf)], -1)
    gap = score.amax(-1, keepdim=True) - score
    M, sh, D, Mo, so = (par[..., i:i + 1] for i in range(5))
    gap = torch.minimum(gap, D.to(torch.float32)).long()
    idx = (gap * M + (1 << (sh - 1))) >> sh
    E = lut[idx]  # the last entry, where a masked key's gap ends, is 0
    Z = E.sum(-1, keepdim=True)
    R = ((255 << 32) + Z // 2) // Z
    P = ((E * R + (1 << 31)) >> 32).to(torch.float32)
    acc = (torch.einsum("bhgk,hkd->bhgd", P[..., :Lp], codes(s["v_prefix"], s["z_v"]))
           + torch.einsum("bhgk,bhkd->bhgd", P[..., Lp:], codes(s["v_cache"], s["z_v"]))).long()
    out = ((acc * Mo + (1 << (so - 1))) >> so).clamp(-127, 127).reshape(B, H, 1, d)
    return (out.to(torch.float32) * torch.as_tensor(s["s_o"], device=dev).view(1, H, 1, 1)).to(torch.bfloat16)


def head_parameters(s, h, G, d):
    """M, s, D, Mo, so of one head, by the library's definition in 64-bit floats."""
    hk = h // G
    r = float(s["s_q"][h]) * float(s["s_k"][hk]) / math.sqrt(d) * 31.0 / s["clip_c"]
    sh = 26
    while sh > 1 and math.floor(r * 2 ** sh + 0.5) > 1 << 24:
        sh -= 1
    M = math.floor(r * 2 ** sh + 0.5)
    f, e = math.frexp(float(s["s_v"][hk]) / (255.0 * float(s["s_o"][h])))
    Mo = math.floor(f * 2 ** 31 + 0.5)
    if Mo == 1 << 31:
        Mo, e = 1 << 30, e + 1
    return M, sh, -(-(61 << (sh - 1)) // M), Mo, 31 - e


# ------------------------------------------------------------------- work
def work(case):
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    if case["op"] == "norm":
        n = B * case["L"] * (H + Hkv) * d
        return {"bytes": 4 * n + B * case["L"] * (4 + 4 * case["rot"]), "flops": 8 * n}
    if case["op"] == "cache":
        n = 2 * B * case["L"] * Hkv * d
        # values in, codes out, codes in, values out
        return {"bytes": 4 * n + 2 * n * case["bits"] // 8, "flops": 6 * n}
    own_rows = B * Hkv * case["Lmax"] / 2.0  # lengths are uniform over 0 .. Lmax
    keys = Hkv * case["Lp"] + own_rows
    return {"bytes": 2 * d * keys + 3 * B * H * d,
            "flops": 4.0 * d * H * B * (case["Lp"] + case["Lmax"] / 2.0)}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return tuple(exact_norm(x, w, s, case["interleaved"]) for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])))
    if case["op"] == "cache":
        k = exact_norm(s["k"], s["w_k"], s, False) if case["norm"] else s["k"].double()
        return exact_values(k, s["s_k"], s["z_k"], case["bits"]), exact_values(s["v"].double(), s["s_v"], s["z_v"],
                                                                                case["bits"])
    return exact_shared(case, s)


def exact_norm(x, w, s, interleaved):
    """The rotation as a product of complex numbers, the norm by the vector's length."""
    x = x.double()
    d = x.shape[-1]
    y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + 1e-6) * w.double()
    half = s["table"].shape[1]
    turn = torch.view_as_complex(s["table"].double())[s["positions"].long()].unsqueeze(1)
    head = y[..., :2 * half]
    pairs = head.unflatten(-1, (half, 2)) if interleaved else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[..., :2 * half] = (z if interleaved else z.transpose(-1, -2)).flatten(-2)
    return y


def exact_values(x, scale, zero, bits):
    """The nearest of the values that the codes stand for (the reciprocal and the product as 32-bit floats, by definition)."""
    sc = torch.as_tensor(scale, device=x.device)[:, None, None]
    n = (x.float() * sc.reciprocal()).double().round()
    lo, hi = (-(2 ** (bits - 1) - 1), 2 ** (bits - 1) - 1)
    if zero is not None:
        z = torch.as_tensor(zero, device=x.device).double()[:, None, None]
        lo, hi = -z, 2 ** bits - 1 - z
    return torch.minimum(torch.maximum(n, n.new_tensor(lo) if zero is None else lo),
                         n.new_tensor(hi) if zero is None else hi) * sc.double()


def exact_shared(case, s):
    """Sequence by sequence, over the keys the sequence sees, in 64-bit whole numbers."""
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    G = H // Hkv
    dev = s["q"].device
    heads = [head_parameters(s, h, G, d) for h in range(H)]
    M, sh, D, Mo, so = (torch.tensor(t, device=dev).view(Hkv, G, 1) for t in zip(*heads))
    table = [math.floor(32768 * math.exp(-i * s["clip_c"] / 31) + 0.5) for i in range(31)] + [0]
    table = torch.tensor(table, device=dev)

    def real(x, z):
        x = x.double()
        return x if z is None else x - torch.as_tensor(z, device=dev).double()[:, None, None]

    kp, vp = real(s["k_prefix"], s["z_k"]), real(s["v_prefix"], s["z_v"])
    out = []
    for b, n in enumerate(s["lengths"].tolist()):
        keys = torch.cat([kp, real(s["k_cache"][b, :, :n], s["z_k"])], 1)
        vals = torch.cat([vp, real(s["v_cache"][b, :, :n], s["z_v"])], 1)
        S = (s["q"][b].view(Hkv, G, d).double() @ keys.transpose(1, 2)).round().long()
        g = S.max(-1, keepdim=True).values - S
        idx = torch.where(g >= D, 31, torch.div(g * M * 2 + 2 ** sh, 2 * 2 ** sh, rounding_mode="floor"))
        E = table[idx.clamp(max=31)]
        Z = E.sum(-1, keepdim=True)
        R = torch.div(255 * 2 ** 32 + torch.div(Z, 2, rounding_mode="floor"), Z, rounding_mode="floor")
        P = torch.div(E * R + 2 ** 31, 2 ** 32, rounding_mode="floor")
        acc = (P.double() @ vals).round().long()
        out.append(torch.div(acc * Mo + 2 ** (so - 1), 2 ** so, rounding_mode="floor").clamp(-127, 127))
    y = torch.stack(out).view(len(out), H, 1, d).double()
    return y * torch.as_tensor(s["s_o"], device=dev).double()[:, None, None]
