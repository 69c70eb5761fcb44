"""Cases for the operators between two LUT linears of a decoder layer.

    residual_norm   post norm of a block's output, gate and residual scale,
                    residual add, norm before the next block, and optionally
                    the rotated int8 / int4 codes that the next LUT product reads
    lora_add        low-rank adapters of many requests beside a shared projection
    rope_qkv        per-head q/k norm, rotary positions and cache rows of the
                    fused QKV projection

``run`` computes them in elementary torch operations, or (``own``) through this
package.  ``exact`` is the definition in fp64 on the host.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases


def _norm(T, H, norm="rms", resid=16, block=True, post=False, gate="none", bits=0, had=0,
          resid_scale=1.0, block_scale=1.0):
    return dict(op="residual_norm", T=T, H=H, norm=norm, resid=resid, block=block, post=post,
                gate=gate, bits=bits, had=had, resid_scale=resid_scale, block_scale=block_scale)


def _lora(M, K, N, n, r, mixed_ranks=False, runs=False, none=0.0):
    return dict(op="lora_add", M=M, K=K, N=N, n=n, r=r, mixed_ranks=mixed_ranks, runs=runs,
                none=none)


def _rope(M, nq, nkv, D, rot, interleaved=False, qk_norm=False, cache=0, far=4096,
          attn_scale=1.0):
    return dict(op="rope_qkv", M=M, nq=nq, nkv=nkv, D=D, rot=rot, interleaved=interleaved,
                qk_norm=qk_norm, cache=cache, far=far, attn_scale=attn_scale)


def listed():
    return [
        # one token entering the dense Qwen3-4B-shaped FFN: pure latency
        dict(_norm(1, 2560, bits=8, had=512), name="norm_decode_1"),
        # a decode batch entering the 30B-A3B-shaped MoE, int4 codes, sandwich norms and a
        # gate per token
        dict(_norm(64, 2048, post=True, gate="token", bits=4, had=2048, block_scale=0.5),
             name="norm_decode_64"),
        # the prefill MoE layer's input: 4096 tokens, one rotation block a row
        dict(_norm(4096, 2048, bits=8, had=2048), name="norm_prefill_4096"),
        # odd token count, LayerNorm with bias on both sides, fp32 residual stream, a gate for
        # every element, no codes (the next consumer is a bf16/fp16 product)
        dict(_norm(1021, 4096, norm="layer", resid=32, post=True, gate="element",
                   resid_scale=0.75, block_scale=1.5), name="norm_layer_1021"),
        # one request with its adapter beside the Qwen3-4B-shaped QKV projection
        dict(_lora(1, 2560, 6144, 1, 16), name="lora_decode_1"),
        # a decode batch of 64 requests over 32 adapters of ranks 64, 32 and 16
        dict(_lora(64, 4096, 4096, 32, 64, mixed_ranks=True), name="lora_decode_64"),
        # chunked prefill and decode mixed, odd row count, an eighth of the rows without adapter
        dict(_lora(517, 9728, 2560, 16, 32, runs=True, none=0.125), name="lora_mixed_517"),
        # prefill of a few long requests beside a gate||up projection
        dict(_lora(4096, 2048, 2816, 8, 64, runs=True), name="lora_prefill_4096"),
        # one token of a Qwen3-4B-shaped attention, q and k norms
        dict(_rope(1, 32, 8, 128, 128, qk_norm=True), name="rope_decode_1"),
        # a decode batch of the 30B-A3B shape writing its keys and values into a cache
        dict(_rope(64, 32, 4, 128, 128, qk_norm=True, cache=2048, far=32768),
             name="rope_decode_64"),
        # prefill of the Mixtral shape into a cache
        dict(_rope(4096, 32, 8, 128, 128, cache=8192, far=32768), name="rope_prefill_4096"),
        # odd row count, part of an odd head, neighbouring pairs, positions of a scaled long context
        dict(_rope(1021, 24, 4, 96, 64, interleaved=True, far=1 << 20, attn_scale=1.2),
             name="rope_long_1021"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("residual_norm", "lora_add", "rope_qkv"))
    if op == "residual_norm":
        bits = rng.choice((0, 4, 8))
        had = rng.choice((16, 64, 128, 256, 512, 1024, 2048, 4096)) if bits else 0
        step = max(had, 64)
        H = step * max(1, _log(rng, 256, 8192) // step)
        T = _log(rng, 1, max(2, min(4096, (1 << 23) // H)))
        block = rng.random() < 0.85
        layer = rng.random() < 0.4
        return _norm(T, H, norm="layer" if layer else "rms", resid=rng.choice((16, 32)),
                     block=block, post=block and rng.random() < 0.5,
                     gate=rng.choice(("none", "channel", "token", "element")) if block else "none",
                     bits=bits, had=had,
                     resid_scale=rng.choice((1.0, 0.75)) if block else 1.0,
                     block_scale=rng.choice((1.0, 0.5, 0.125)) if block else 1.0)
    if op == "lora_add":
        K = 8 * _log(rng, 32, 1216)
        N = 8 * _log(rng, 16, 768)
        M = _log(rng, 1, max(2, min(4096, (1 << 26) // (2 * K + 8 * N))))
        return _lora(M, K, N, rng.randint(1, 32), rng.choice((8, 16, 32, 64, 128)),
                     mixed_ranks=rng.random() < 0.5, runs=rng.random() < 0.5,
                     none=rng.choice((0.0, 0.0, 0.125, 0.5)))
    D = rng.choice((64, 80, 96, 128, 192, 256))
    nkv = rng.choice((1, 2, 4, 8))
    nq = nkv * rng.choice((1, 2, 4, 7, 8))
    M = _log(rng, 1, max(2, min(4096, (1 << 24) // ((nq + 2 * nkv) * D))))
    return _rope(M, nq, nkv, D, rng.choice((D, D, 8 * rng.randint(1, D // 8))),
                 interleaved=rng.random() < 0.5, qk_norm=rng.random() < 0.5,
                 cache=rng.choice((0, 2 * M)), far=rng.choice((4096, 32768, 1 << 20)),
                 attn_scale=rng.choice((1.0, 1.1)))


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _sylvester(b):
    """H_b of the rotation, fp64 (+-1), H[i][j] = (-1)^popcount(i & j), b <= 2^16."""
    i = torch.arange(b, dtype=torch.int32, device=DEV)
    v = i[:, None] & i
    v = v ^ (v >> 8)
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    v = v ^ (v >> 1)
    return 1.0 - 2.0 * (v & 1).double()


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]

    def rnd(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    # a residual stream with a few massive channels, as the activations of the framework have
    r = rnd(T, H) * 2
    ch = torch.randperm(H, device=DEV, generator=g)[:4]
    r[:, ch] *= 50
    rd = torch.float16 if c["resid"] == 16 else torch.float32
    st = dict(resid=r.to(rd), resid_out=torch.empty((T, H), dtype=rd, device=DEV),
              x=torch.empty((T, H), dtype=torch.float16, device=DEV),
              pre_weight=(1 + 0.2 * rnd(H)).half())
    layer = c["norm"] == "layer"
    if layer:
        st["pre_bias"] = (0.1 * rnd(H)).half()
    if c["block"]:
        st["y"] = rnd(T, H)
        if c["post"]:
            st["post_weight"] = (1 + 0.2 * rnd(H)).half()
            if layer:
                st["post_bias"] = (0.1 * rnd(H)).half()
        shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[c["gate"]]
        if shape:
            st["gate"] = torch.sigmoid(rnd(*shape)).half()
    if c["bits"]:
        st["q"] = torch.empty((T, H * c["bits"] // 8), device=DEV,
                              dtype=torch.uint8 if c["bits"] == 4 else torch.int8)
        st["s"] = torch.empty((T,), dtype=torch.float32, device=DEV)
        st["hadamard"] = _sylvester(c["had"])
        # byte -> its two int4 codes, low nibble first
        v = torch.arange(256, device=DEV)
        st["nibbles"] = torch.stack((((v & 15) ^ 8) - 8, ((v >> 4) ^ 8) - 8), 1).to(torch.int8)
    return st


def _prepare_lora(c, g):
    M, K, N, n, r = c["M"], c["K"], c["N"], c["n"], c["r"]

    def rnd(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    live = M - int(M * c["none"])
    used = min(n, live)
    # every used adapter has a row; the rest fall on them at random
    ids = torch.cat((torch.arange(used, device=DEV),
                     torch.randint(0, max(used, 1), (live - used,), device=DEV, generator=g),
                     torch.full((M - live,), -1, device=DEV, dtype=torch.int64)))
    if c["runs"]:      # requests of many tokens: their rows stand together
        ids = ids.sort()[0]
    else:              # one row a request
        ids = ids[torch.randperm(M, device=DEV, generator=g)]
    ranks = torch.tensor([max(1, r >> (i % 3)) if c["mixed_ranks"] else r for i in range(n)],
                         dtype=torch.int32, device=DEV)
    x = rnd(M, K)
    ch = torch.randperm(K, device=DEV, generator=g)[:4]
    x[:, ch] *= 10
    return dict(x=x.half(), ids=ids.to(torch.int32), ranks=ranks,
                a=(rnd(n, r, K) / math.sqrt(K)).half(), b=(rnd(n, N, r) / math.sqrt(r)).half(),
                scale=0.5 + torch.rand((n,), device=DEV, generator=g), y=rnd(M, N),
                out=torch.empty((M, N), device=DEV))


def _prepare_rope(c, g):
    M, nq, nkv, D, rot = c["M"], c["nq"], c["nkv"], c["D"], c["rot"]

    def rnd(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    rows = c["cache"] or M
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    st = dict(qkv=rnd(M, (nq + 2 * nkv) * D),
              positions=torch.randint(0, c["far"], (M,), device=DEV, generator=g,
                                      dtype=torch.int32),
              inv_freq=(1e6 ** (-2 * i / rot)).float(),
              q=torch.empty((M, nq, D), dtype=torch.float16, device=DEV),
              k=rnd(rows, nkv, D).half(), v=rnd(rows, nkv, D).half())
    if c["cache"]:
        st["slots"] = torch.randperm(rows, device=DEV, generator=g)[:M]
    if c["qk_norm"]:
        st["q_weight"] = (1 + 0.2 * rnd(D)).half()
        st["k_weight"] = (1 + 0.2 * rnd(D)).half()
    return st


def prepare(case, seed):
    make = {"residual_norm": _prepare_norm, "lora_add": _prepare_lora, "rope_qkv": _prepare_rope}
    return dict(case=case, **make[case["op"]](case, _gen(seed)))


# ---------------------------------------------------------------------------
# one pass


def _half(v):
    """fp64 -> fp16, rounded once: to fp32 with the lost bits kept in the last
    one (round to odd), then to fp16."""
    f = v.float()
    back = f.double()
    bits = f.view(torch.int32) - (back.abs() > v.abs()).int()
    bits = torch.where(back != v, bits | 1, bits)
    return bits.view(torch.float32).half()


def _normed(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * weight.double()
    return v if bias is None else v + bias.double()


def _unpacked(q, nibbles):
    return nibbles.index_select(0, q.view(-1).int()).view(q.shape[0], -1)


def _run_norm(st):
    c = st["case"]
    if own:
        import lut_clustered_weight_b200 as cq
        got = cq.cq_residual_norm(
            st["resid"], st.get("y"), norm=c["norm"], eps=1e-6, pre_weight=st["pre_weight"],
            pre_bias=st.get("pre_bias"), post_norm=c["post"], post_weight=st.get("post_weight"),
            post_bias=st.get("post_bias"), gate=st.get("gate"), resid_scale=c["resid_scale"],
            block_scale=c["block_scale"], had_block=c["had"], act_bits=c["bits"],
            resid_out=st["resid_out"] if c["block"] else None, x_out=st["x"],
            q_out=st.get("q"), s_out=st.get("s"))
        if c["bits"] == 4:
            return got[0], got[1], _unpacked(got[2], st["nibbles"]), got[3]
        return got
    # codes are whole numbers decided on x, and x on r': all of it in 64 bits, as a
    # value next to a rounding border must fall on the same side
    r = st["resid"]
    if c["block"]:
        v = st["y"].double()
        if c["post"]:
            v = _normed(v, c["norm"], st["post_weight"], st.get("post_bias"))
        if "gate" in st:
            v = v * st["gate"].double()
        v = r.double() * c["resid_scale"] + v * c["block_scale"]
        r = _half(v) if c["resid"] == 16 else v.float()
    x = _half(_normed(r.double(), c["norm"], st["pre_weight"], st.get("pre_bias")))
    if not c["bits"]:
        return r, x
    T, H, b, qmax = c["T"], c["H"], c["had"], (1 << (c["bits"] - 1)) - 1
    rot = (x.double().view(-1, b) @ st["hadamard"]).view(T, H)
    top = rot.abs().amax(1, keepdim=True)
    q = torch.round(qmax * rot / top.clamp_min(1e-300)).to(torch.int8)
    return r, x, q, (top.view(-1) / math.sqrt(b) / qmax).float()


def _run_lora(st):
    x, ids, a, b = st["x"], st["ids"], st["a"], st["b"]
    if own:
        import lut_clustered_weight_b200 as cq
        return cq.cq_lora_add(x, ids, a, b, st["y"], scale=st["scale"], ranks=st["ranks"],
                              out=st["out"])
    n, r, K = a.shape
    N = b.shape[1]
    # all adapters at once: t of the other adapters and of the unused ranks is zeroed
    t = (x.float() @ a.float().view(n * r, K).T).view(-1, n, r)
    one = ids[:, None] == torch.arange(n, device=ids.device)
    rank = torch.arange(r, device=ids.device) < st["ranks"][:, None]
    t = torch.where(one[:, :, None] & rank, t * st["scale"][:, None], 0.0)
    return st["y"] + t.view(-1, n * r) @ b.float().transpose(0, 1).reshape(N, n * r).T


def _head_norm(t, weight):
    return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * weight.float()


def _turned(t, cos, sin, rot, interleaved):
    head, rest = t[..., :rot], t[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((head, rest), -1)


def _run_rope(st):
    c = st["case"]
    M, nq, nkv, D, rot = c["M"], c["nq"], c["nkv"], c["D"], c["rot"]
    if own:
        import lut_clustered_weight_b200 as cq
        return cq.cq_rope_qkv(
            st["qkv"], st["positions"], st["inv_freq"], nq, nkv, head_dim=D,
            interleaved=c["interleaved"], attn_scale=c["attn_scale"],
            q_weight=st.get("q_weight"), k_weight=st.get("k_weight"), eps=1e-6, q_out=st["q"],
            k_out=st["k"], v_out=st["v"], slots=st.get("slots"))
    # the angle of a far position needs 64 bits
    angle = st["positions"].double()[:, None, None] * st["inv_freq"].double()
    cos = (torch.cos(angle) * c["attn_scale"]).float()
    sin = (torch.sin(angle) * c["attn_scale"]).float()
    q, k, v = st["qkv"].view(M, nq + 2 * nkv, D).split((nq, nkv, nkv), 1)
    if c["qk_norm"]:
        q, k = _head_norm(q, st["q_weight"]), _head_norm(k, st["k_weight"])
    st["q"].copy_(_turned(q, cos, sin, rot, c["interleaved"]))
    k = _turned(k, cos, sin, rot, c["interleaved"]).half()
    if "slots" in st:
        st["k"][st["slots"]] = k
        st["v"][st["slots"]] = v.half()
    else:
        st["k"].copy_(k)
        st["v"].copy_(v)
    return st["q"], st["k"], st["v"]


def run(state):
    op = state["case"]["op"]
    if op == "residual_norm":
        return _run_norm(state)
    return _run_lora(state) if op == "lora_add" else _run_rope(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "residual_norm":
        T, H, rb = c["T"], c["H"], c["resid"] // 8
        per = rb + 2 + c["bits"] / 8
        flops = 6
        if c["block"]:
            per += 4 + rb + (2 if c["gate"] == "element" else 0)
            flops += 4 + (5 if c["post"] else 0)
        if c["bits"]:
            flops += int(math.log2(c["had"])) + 3
        vectors = 1 + (c["norm"] == "layer")
        vectors = vectors * (2 if c["post"] else 1) + (c["gate"] == "channel")
        small = 2 * H * vectors + T * (4 if c["bits"] else 0) + T * (2 if c["gate"] == "token" else 0)
        return {"bytes": T * H * per + small, "flops": T * H * flops}
    if c["op"] == "lora_add":
        M, K, N, n, r = c["M"], c["K"], c["N"], c["n"], c["r"]
        live = M - int(M * c["none"])
        ranks = [max(1, r >> (i % 3)) if c["mixed_ranks"] else r for i in range(min(n, live))]
        mean = sum(ranks) / max(1, len(ranks))
        return {"bytes": 2 * live * K + 8 * M * N + 2 * sum(ranks) * (K + N) + 4 * M,
                "flops": 2 * live * mean * (K + N)}
    M, heads, D = c["M"], c["nq"] + 2 * c["nkv"], c["D"]
    return {"bytes": 6 * M * heads * D + M * (12 if c["cache"] else 4), "flops": 8 * M * heads * D}


# ---------------------------------------------------------------------------
# the definitions in fp64 on the host


def _f64(t):
    return t.cpu().numpy().astype(np.float64)


def _exact_norm(c, st):
    def norm(v, weight, bias):
        if c["norm"] == "layer":
            v = v - v.mean(axis=1)[:, None]
        v = v / np.sqrt(np.mean(np.square(v), axis=1) + 1e-6)[:, None] * _f64(weight)
        return v if bias is None else v + _f64(bias)

    full = _f64(st["resid"])
    r = full
    if c["block"]:
        y = _f64(st["y"])
        if c["post"]:
            y = norm(y, st["post_weight"], st.get("post_bias"))
        g = _f64(st["gate"]) if "gate" in st else 1.0
        full = c["resid_scale"] * full + c["block_scale"] * (g * y)
        r = full.astype(np.float16 if c["resid"] == 16 else np.float32).astype(np.float64)
    x = norm(r, st["pre_weight"], st.get("pre_bias"))
    if not c["bits"]:
        return full, x
    T, H, b, qmax = c["T"], c["H"], c["had"], 2 ** (c["bits"] - 1) - 1
    z = x.astype(np.float16).astype(np.float64).reshape(-1, b)
    h = 1
    while h < b:       # butterflies over pairs h apart
        z = z.reshape(-1, b // (2 * h), 2, h)
        z = np.stack((z[:, :, 0] + z[:, :, 1], z[:, :, 0] - z[:, :, 1]), axis=2).reshape(-1, b)
        h *= 2
    z = z.reshape(T, H)
    top = np.abs(z).max(axis=1)
    q = np.rint(qmax * z / np.where(top > 0, top, 1)[:, None])
    return full, x, q.astype(np.int8), top / np.sqrt(b) / qmax


def _exact_lora(c, st):
    x, y, a, b = (_f64(st[k]) for k in ("x", "y", "a", "b"))
    ids, ranks, scale = st["ids"].cpu().numpy(), st["ranks"].cpu().numpy(), _f64(st["scale"])
    for i in range(c["n"]):
        rows, k = np.flatnonzero(ids == i), ranks[i]
        if rows.size:
            y[rows] += scale[i] * ((x[rows] @ a[i, :k].T) @ b[i, :, :k].T)
    return y


def _exact_rope(c, st):
    M, nq, nkv, D, rot = c["M"], c["nq"], c["nkv"], c["D"], c["rot"]
    z = _f64(st["qkv"]).reshape(M, nq + 2 * nkv, D)
    z = z.copy()
    if c["qk_norm"]:
        for lo, hi, w in ((0, nq, "q_weight"), (nq, nq + nkv, "k_weight")):
            t = z[:, lo:hi]
            z[:, lo:hi] = t * _f64(st[w]) / np.sqrt((t ** 2).sum(axis=-1) / D + 1e-6)[..., None]
    turn = np.exp(1j * np.outer(_f64(st["positions"]), _f64(st["inv_freq"])))[:, None]
    turn = turn * c["attn_scale"]
    i = np.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
    t = z[:, : nq + nkv]
    w = (t[..., first] + 1j * t[..., second]) * turn
    t[..., first], t[..., second] = w.real, w.imag
    k, v = _f64(st["k"]), _f64(st["v"])
    at = st["slots"].cpu().numpy() if "slots" in st else np.arange(M)
    k[at], v[at] = z[:, nq: nq + nkv], z[:, nq + nkv:]
    return z[:, :nq], k, v


def exact(case, seed):
    st = prepare(case, seed)
    solve = {"residual_norm": _exact_norm, "lora_add": _exact_lora, "rope_qkv": _exact_rope}
    return solve[case["op"]](case, st)
