"""Operators between two LUT linears on the GPU: cq_residual_norm, cq_lora_add
and cq_rope_qkv against their fp64 definitions, alone and as a chain."""
import numpy as np
import pytest
import torch

import layer_ops_ref as ref
import oracle
import synth

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def cq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import lut_clustered_weight_b200 as m
    return m


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _bits(t):
    a = t.cpu().numpy()
    return a.view({2: np.uint16, 4: np.uint32, 1: np.uint8}[a.dtype.itemsize])


# ---------------------------------------------------------------- residual norm


def _norm_inputs(T, H, kind, rbits, block, post, gate, seed, weights=True):
    g = np.random.default_rng(seed)

    def rnd(*s):
        return g.standard_normal(s)

    r = rnd(T, H) * 2
    r[:, g.choice(H, min(4, H), replace=False)] *= 50
    if T >= 4:
        r[1] = 0                                  # a zero row
        r[2] *= 1e-4                              # small values: fp16 subnormals
        r[3] = 3.0                                # a constant row (zero variance)
    d = dict(resid=r.astype(np.float16 if rbits == 16 else np.float32))
    layer = kind == "layer"

    def wb():
        return ((1 + 0.2 * rnd(H)).astype(np.float16) if weights else None,
                (0.1 * rnd(H)).astype(np.float16) if layer and weights else None)

    d["pre"] = wb()
    d["y"] = d["post"] = d["gate"] = None
    if block:
        y = rnd(T, H)
        if T >= 4:
            y[1] = 0
            y[3] = -1.0
        d["y"] = y.astype(np.float32)
        d["post"] = wb() if post else None
        shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[gate]
        if shape:
            d["gate"] = rnd(*shape).astype(np.float16)
    return d


def _norm_run(cq, d, kind, rs, bs, had, bits, **kw):
    o = {k: None if d[k] is None else _dev(d[k]) for k in ("resid", "y", "gate")}
    dv = lambda a: None if a is None else _dev(a)  # noqa: E731
    post = d["post"] or (None, None)
    return cq.cq_residual_norm(o["resid"], o["y"], norm=kind, eps=1e-6, pre_weight=dv(d["pre"][0]),
                               pre_bias=dv(d["pre"][1]), post_norm=d["post"] is not None,
                               post_weight=dv(post[0]), post_bias=dv(post[1]), gate=o["gate"],
                               resid_scale=rs, block_scale=bs, had_block=had, act_bits=bits, **kw)


def _norm_ref(d, kind, rs, bs):
    f = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
    pair = lambda p: None if p is None else (f(p[0]), f(p[1]))  # noqa: E731
    return ref.residual_norm(d["resid"], f(d["y"]), kind, 1e-6, pair(d["pre"]), pair(d["post"]),
                             f(d["gate"]), rs, bs)


NORM_CASES = [
    # (T, H, kind, resid bits, block, post, gate, rs, bs, had, bits)
    (1, 2560, "rms", 16, True, False, "none", 1.0, 1.0, 512, 8),
    (64, 2048, "rms", 16, True, True, "token", 1.0, 0.5, 2048, 4),
    (5, 8, "rms", 16, True, False, "none", 1.0, 1.0, 8, 4),
    (7, 24, "layer", 32, True, True, "element", 0.75, 1.5, 1, 8),
    (4, 200, "layer", 16, True, True, "channel", -0.5, 2.0, 0, 0),
    (33, 264, "rms", 32, True, True, "channel", 1.0, 0.3, 8, 4),
    (1, 16384, "layer", 32, True, True, "element", 1.0, 1.0, 8192, 8),
    (3, 16384, "rms", 16, True, False, "channel", 1.0, 1.0, 16, 4),
    (2, 14336, "rms", 16, True, True, "none", 1.0, 1.0, 2048, 8),
    (6, 9728, "rms", 32, False, False, "none", 1.0, 1.0, 256, 4),
    (9, 4096, "layer", 16, False, False, "none", 1.0, 1.0, 4096, 8),
    (17, 5120, "rms", 16, True, False, "token", 1.0, 0.0, 1024, 4),
    (4, 8192, "rms", 16, True, False, "none", 1.0, 1.0, 8192, 4),
    # many rows
    (301, 1408, "rms", 16, True, True, "element", 1.0, 1.0, 128, 4),
    (700, 2048, "rms", 16, True, False, "none", 1.0, 1.0, 2048, 8),
    (611, 64, "layer", 16, True, True, "token", 1.0, 1.0, 64, 8),
    (1021, 96, "rms", 32, True, False, "element", 1.0, 1.0, 32, 4),
    (600, 4096, "layer", 32, True, True, "element", 0.75, 1.5, 0, 0),
    (593, 40, "rms", 16, False, False, "none", 1.0, 1.0, 8, 4),
    (400, 8192, "rms", 32, True, True, "channel", 1.0, 1.0, 4096, 8),
    (320, 2304, "layer", 16, True, False, "none", 1.0, 1.0, 256, 8),
    (310, 16384, "rms", 16, True, False, "none", 1.0, 1.0, 16, 4),
    (310, 512, "layer", 16, True, False, "element", 1.0, 1.0, 0, 0),
    (304, 2048, "rms", 32, True, False, "none", 0.5, 1.0, 0, 0),
    (305, 2048, "rms", 16, True, False, "channel", 1.0, 1.0, 0, 0),
    (170, 5120, "rms", 32, True, False, "token", 1.0, 1.0, 1024, 8),
    (160, 5120, "rms", 16, True, True, "none", 1.0, 1.0, 512, 4),
    (159, 7168, "layer", 32, True, True, "element", 1.0, 1.0, 1024, 4),
    (150, 8192, "layer", 16, True, False, "none", 1.0, 1.0, 0, 0),
    # the last thread of a row has 8 channels less
    (3, 8200, "rms", 16, True, True, "element", 1.0, 1.0, 8, 4),
    (300, 8216, "layer", 32, True, False, "none", 1.0, 1.0, 4, 8),
    (298, 4104, "rms", 32, True, True, "channel", 1.0, 1.0, 2, 8),
    # a mean far from the spread
    (310, 1000, "layer", 32, True, True, "none", 1.0, 1e4, 0, 0),
]


@pytest.mark.parametrize("T,H,kind,rb,block,post,gate,rs,bs,had,bits", NORM_CASES)
def test_residual_norm_is_the_rounded_definition(cq, T, H, kind, rb, block, post, gate, rs, bs,
                                                 had, bits):
    """r' and x bit for bit.  Kernel and reference both work in fp64: they differ
    by about 1e-15 of a value (1e-12 at the worst order of 16384 additions), so
    the chance that a rounding border (2^-11 apart in fp16, 2^-24 in fp32) lies
    between them is below 1e-7 per value, and the inputs are fixed.  A value that
    the formula puts on a border (a constant row, whose LayerNorm is the bias) has
    to be formed without any difference."""
    d = _norm_inputs(T, H, kind, rb, block, post, gate, seed=T + H)
    got = _norm_run(cq, d, kind, rs, bs, had, bits)
    torch.cuda.synchronize()
    r, x = _norm_ref(d, kind, rs, bs)
    assert np.array_equal(got[0].cpu().numpy(), r)
    assert np.array_equal(got[1].cpu().numpy(), x)
    if bits:
        qr, sr = oracle.rotate_quantize(x, had, bits)
        assert np.array_equal(oracle.unpack_codes(got[2].cpu().numpy(), H, bits), qr)
        assert np.array_equal(_bits(got[3]), sr.view(np.uint32))


@pytest.mark.parametrize("T,H", [(3, 512), (400, 1024)])
def test_residual_norm_codes_are_cq_rotate_quantize_of_x(cq, T, H):
    d = _norm_inputs(T, H, "rms", 16, True, True, "token", seed=5)
    for had in (1, 2, 4, 8, 16, 32, 64, 128, 256, 512, 1024):
        if had > H:
            continue
        for bits in (4, 8):
            _, x, q, s = _norm_run(cq, d, "rms", 1.0, 1.0, had, bits)
            q2, s2 = cq.cq_rotate_quantize(x, had, bits)
            assert torch.equal(q, q2) and torch.equal(s, s2)


def test_residual_norm_rounding_ties(cq):
    """Sums that land exactly on fp16 ties go to the even neighbour, and a value
    just beside a tie (one fp32 step of y) goes its own way: a detour through
    fp32 would lose it."""
    H = 64
    r = np.full((2, H), 1.0, np.float16)
    y = np.full((2, H), 2.0 ** -11, np.float32)              # half a step of 1.0
    y[0, 1::2] = np.nextafter(np.float32(2.0 ** -11), np.float32(1))
    y[1] = 3 * np.float32(2.0 ** -11)                        # tie between steps 1 and 2
    y[1, 1::2] = np.nextafter(y[1, 0], np.float32(0))
    got, _ = cq.cq_residual_norm(_dev(r), _dev(y))
    want = (r.astype(np.float64) + y.astype(np.float64)).astype(np.float16)
    assert want[0, 0] == 1.0 and want[0, 1] > 1.0 and want[1, 0] > want[1, 1]
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T", [2, 500])
def test_residual_norm_in_place_and_without_weights(cq, T):
    d = _norm_inputs(T, 768, "rms", 16, True, False, "none", seed=9, weights=False)
    r, x = _norm_ref(d, "rms", 1.0, 1.0)
    resid = _dev(d["resid"])
    a, b = cq.cq_residual_norm(resid, _dev(d["y"]), resid_out=resid)
    assert a is resid and np.array_equal(resid.cpu().numpy(), r)
    assert np.array_equal(b.cpu().numpy(), x)


def test_residual_norm_writes_only_its_rows(cq):
    T, H = 5, 136
    d = _norm_inputs(T, H, "rms", 16, True, False, "none", seed=3)
    big = torch.full((T + 3, H), 7.0, dtype=torch.float16, device=DEV)
    ro = torch.full((T + 3, H), 7.0, dtype=torch.float16, device=DEV)
    q = torch.full((T + 3, H // 2), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((T + 3,), 7.0, device=DEV)
    _norm_run(cq, d, "rms", 1.0, 1.0, 8, 4, resid_out=ro[:T], x_out=big[:T], q_out=q[:T], s_out=s[:T])
    torch.cuda.synchronize()
    assert (big[T:] == 7).all() and (ro[T:] == 7).all() and (q[T:] == 77).all() and (s[T:] == 7).all()
    assert not (big[:T] == 7).all()


def test_residual_norm_empty(cq):
    z = torch.empty((0, 64), dtype=torch.float16, device=DEV)
    r, x = cq.cq_residual_norm(z, torch.empty((0, 64), device=DEV))
    assert r.shape == x.shape == (0, 64)


@pytest.mark.parametrize("T,H,had,bits", [(6, 512, 64, 8), (6, 2048, 2048, 4), (400, 2048, 16, 8),
                                          (150, 8216, 8, 4), (400, 2048, 0, 0)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["channel", "token", "element"])
def test_residual_norm_passes_on_what_is_not_finite(cq, T, H, had, bits, kind, gate):
    """A NaN or an infinity in an operand gives in r' and x what the formula gives.
    A row whose x holds one has the scale NaN and codes 0; the other rows do not
    change.  (A finite x beyond fp16 is an infinity like another.)"""
    clean = _norm_inputs(T, H, kind, 16, True, True, gate, seed=11)
    # resid and y at (row 1, ..): their row alone; a weight or bias: every row
    spots = [("resid", 1), ("y", 1), ("gate", 1), ("pre", 0), ("post", 0)]
    if kind == "layer":
        spots += [("pre", 1), ("post", 1)]
    for n, (name, i) in enumerate(spots):
        for bad in (np.nan, np.inf, -np.inf):
            d = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in clean.items()}
            c = (8 * n + 5) % H
            if name in ("pre", "post"):
                d[name] = tuple(None if w is None else w.copy() for w in d[name])
                d[name][i][c] = bad
            elif d[name].ndim == 1:
                d[name][c] = bad
            else:
                d[name][1, min(c, d[name].shape[1] - 1)] = bad
            got = _norm_run(cq, d, kind, 1.0, 1.0, had, bits)
            with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                r, x = _norm_ref(d, kind, 1.0, 1.0)
            np.testing.assert_array_equal(got[0].cpu().numpy(), r)
            np.testing.assert_array_equal(got[1].cpu().numpy(), x)
            if bits:
                ok = np.isfinite(x).all(axis=1)
                q, s = oracle.unpack_codes(got[2].cpu().numpy(), H, bits), got[3].cpu().numpy()
                assert not ok.all() and np.isnan(s[~ok]).all() and not q[~ok].any()
                if ok.any():
                    qr, sr = oracle.rotate_quantize(np.ascontiguousarray(x[ok]), had, bits)
                    assert np.array_equal(q[ok], qr) and np.array_equal(s[ok], sr)


def test_residual_norm_scale_of_a_row_beyond_fp16(cq):
    """x overflows fp16 in one channel of a row of finite operands."""
    T, H = 3, 64
    d = _norm_inputs(T, H, "rms", 16, False, False, "none", seed=2)
    w = d["pre"][0]
    w[:] = 1
    w[9] = 6e4
    d["resid"][:] = 1
    d["resid"][0, 9] = 0
    d["resid"][1, 9] = 4                                      # 4 / sqrt(79 / 64) * 6e4 > 65504
    d["resid"][2, 9] = 1 / 64
    _, x, q, s = _norm_run(cq, d, "rms", 1.0, 1.0, 16, 8)
    x, q, s = x.cpu().numpy(), q.cpu().numpy(), s.cpu().numpy()
    assert np.isinf(x[1, 9]) and np.isfinite(x[[0, 2]]).all()
    assert np.isnan(s[1]) and not q[1].any()
    qr, sr = oracle.rotate_quantize(np.ascontiguousarray(x[[0, 2]]), 16, 8)
    assert np.array_equal(q[[0, 2]], qr) and np.array_equal(s[[0, 2]], sr)


@pytest.mark.parametrize("eps", [1e-12, 1e-5, 0.25, 30.0])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_residual_norm_eps_is_the_one_given(cq, kind, eps):
    """In both norms, in rows of mean squares from 0 to 1e6; codes too."""
    T, H = 8, 256
    d = _norm_inputs(T, H, kind, 32, True, True, "none", seed=4)
    d["y"] *= np.logspace(-4, 2, T, dtype=np.float32)[:, None]
    d["resid"] *= np.logspace(2, -4, T, dtype=np.float32)[:, None]
    pw, pb = d["pre"]
    qw, qb = d["post"]
    dv = lambda a: None if a is None else _dev(a)  # noqa: E731
    got = cq.cq_residual_norm(_dev(d["resid"]), _dev(d["y"]), norm=kind, eps=eps, pre_weight=dv(pw),
                              pre_bias=dv(pb), post_norm=True, post_weight=dv(qw), post_bias=dv(qb),
                              had_block=64, act_bits=8)
    f = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
    r, x = ref.residual_norm(d["resid"], f(d["y"]), kind, eps, (f(pw), f(pb)), (f(qw), f(qb)), None,
                             1.0, 1.0)
    assert np.array_equal(got[0].cpu().numpy(), r) and np.array_equal(got[1].cpu().numpy(), x)
    qr, sr = oracle.rotate_quantize(x, 64, 8)
    assert np.array_equal(got[2].cpu().numpy(), qr) and np.array_equal(got[3].cpu().numpy(), sr)


# ---------------------------------------------------------------- low-rank adapters


def _lora_inputs(M, K, N, n, r, ids, seed, mixed=False):
    g = np.random.default_rng(seed)
    ids = np.asarray(ids, np.int32)
    ranks = np.array([max(0, r - 5 * i) if mixed else r for i in range(n)], np.int32)
    if mixed and n > 2:
        ranks[1], ranks[2] = r + 100, -3           # clamped to r and to 0
    a = (g.standard_normal((n, r, K)) / np.sqrt(K)).astype(np.float16)
    b = g.standard_normal((n, N, r)).astype(np.float16)
    if mixed:                                      # what unused ranks hold does not matter
        for i in range(n):
            k = int(np.clip(ranks[i], 0, r))
            a[i, k:] = np.nan
            b[i, :, k:] = np.nan
    x = g.standard_normal((M, K))
    x[:, g.choice(K, 4, replace=False)] *= 30
    return dict(x=x.astype(np.float16), ids=ids, a=a, b=b, ranks=ranks,
                scale=(0.5 + g.random(n)).astype(np.float32),
                y=g.standard_normal((M, N)).astype(np.float32))


def _lora_run(cq, d, **kw):
    t = {k: _dev(v) for k, v in d.items()}
    return cq.cq_lora_add(t["x"], t["ids"], t["a"], t["b"], t["y"], scale=t["scale"],
                          ranks=t["ranks"], **kw)


def _lora_check(got, d):
    f = {k: v.astype(np.float64) for k, v in d.items() if k not in ("ids", "ranks")}
    want, tol = ref.lora_add(f["x"], d["ids"], f["a"], f["b"], f["scale"], d["ranks"], f["y"])
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= tol), f"worst err/tol {(err / np.maximum(tol, 1e-300)).max()}"


def _runs(M, n, g):
    return np.sort(g.integers(0, n, M))


LORA_CASES = [
    # (M, K, N, n, r, kind of ids, mixed ranks)
    (1, 2560, 6144, 1, 16, "all", False),
    (1, 8, 8, 1, 8, "all", False),
    (2, 72, 40, 3, 8, "rows", False),
    (3, 1000, 1000, 4, 24, "rows", True),
    (16, 2048, 512, 16, 64, "each", True),
    (17, 512, 264, 2, 128, "rows", True),
    (33, 4096, 136, 5, 40, "rows", True),
    (64, 1024, 1024, 32, 64, "rows", False),
    (64, 1024, 1024, 1, 32, "all", False),
    (130, 9728, 64, 7, 16, "none", True),
    (257, 264, 2056, 9, 104, "runs", True),
    (513, 2048, 320, 16, 32, "runs", False),
    (700, 328, 200, 300, 16, "rows", False),       # more adapters than a tile has rows
    (1100, 640, 512, 8, 64, "runs", False),
    (1500, 136, 72, 4096, 8, "rows", False),       # the largest bank
    (2100, 256, 264, 3, 128, "rows", True),
    (256, 64, 40, 300, 16, "rows", False),         # one row a thread of the tile search
    (255, 40, 24, 2, 24, "none", False),
    (2048, 96, 72, 2, 16, "none", True),
    (2048, 4096, 24, 2, 16, "runs", False),        # every stage of the ring in use, per rank size
    (2050, 4096, 24, 2, 32, "runs", False),
    (2048, 4096, 136, 2, 64, "runs", True),
    (2049, 4096, 40, 2, 128, "runs", True),
    (300, 8192, 24, 2, 8, "runs", False),
    (300, 8192, 24, 2, 32, "runs", False),
    (300, 8192, 24, 2, 64, "runs", False),
    (300, 8192, 2056, 2, 128, "runs", False),
    (5, 8192, 4104, 2, 16, "rows", False),
    (5, 8192, 4104, 2, 128, "rows", False),
    # up to 256 rows in either form, by the work
    (41, 4096, 4104, 60, 64, "each", True),
    (100, 1024, 1032, 200, 16, "rows", False),
    (161, 2048, 1032, 40, 32, "runs", True),
    (161, 136, 136, 40, 32, "runs", True),
    (256, 2560, 264, 3, 128, "rows", True),
    (200, 1024, 1024, 7, 64, "none", False),
    (9000, 16, 24, 5, 8, "rows", False),           # more rows than the sorting CTA holds
    (17000, 8, 8, 1100, 8, "rows", True),
]


@pytest.mark.parametrize("M,K,N,n,r,kind,mixed", LORA_CASES)
def test_lora_add_against_definition(cq, M, K, N, n, r, kind, mixed):
    g = np.random.default_rng(M + K)
    ids = {"all": np.zeros(M), "rows": g.integers(0, n, M), "each": np.arange(M) % n,
           "runs": _runs(M, n, g), "none": np.where(g.random(M) < 0.5, -1, g.integers(0, n, M))}[kind]
    if kind in ("rows", "runs") and M > 8:
        ids[5], ids[7], ids[M - 1] = -1, n, 2 ** 31 - 1      # no adapter
    d = _lora_inputs(M, K, N, n, r, ids, seed=M + N, mixed=mixed)
    out = torch.full((M, N), float("nan"), device=DEV)
    got = _lora_run(cq, d, out=out)
    assert got is out
    torch.cuda.synchronize()
    _lora_check(got, d)
    # in place gives the same bits
    assert torch.equal(_lora_run(cq, d), out)


def test_lora_add_without_scale_and_ranks_is_ones_and_full(cq):
    d = _lora_inputs(9, 256, 64, 3, 16, np.arange(9) % 3, seed=1)
    d["scale"][:] = 1
    t = {k: _dev(v) for k, v in d.items()}
    got = cq.cq_lora_add(t["x"], t["ids"], t["a"], t["b"], t["y"], out=torch.empty_like(t["y"]))
    _lora_check(got, d)


@pytest.mark.parametrize("M", [5, 600])
def test_lora_add_on_column_slices(cq, M):
    """q, k and v of a fused projection get adapters of their own, in place; what
    lies beside a slice stays as it was."""
    K, widths = 512, (256, 64, 64)
    g = np.random.default_rng(4)
    wide = g.standard_normal((M, sum(widths) + 8)).astype(np.float32)
    buf = _dev(wide)
    want, at = wide.copy(), 0
    for i, N in enumerate(widths):
        d = _lora_inputs(M, K, N, 4, 16, g.integers(-1, 4, M), seed=i)
        d["y"] = np.ascontiguousarray(wide[:, at:at + N])
        t = {k: _dev(v) for k, v in d.items()}
        sl = buf[:, at:at + N]
        assert cq.cq_lora_add(t["x"], t["ids"], t["a"], t["b"], sl, scale=t["scale"]) is sl
        torch.cuda.synchronize()
        _lora_check(sl, d)
        want[:, at:at + N] = sl.cpu().numpy()
        at += N
    assert np.array_equal(buf.cpu().numpy(), want)


@pytest.mark.parametrize("M", [1, 7, 130, 600, 2100])
def test_lora_add_from_one_row_stride_to_another(cq, M):
    """y a slice of rows of one width, out of another; rows with an adapter, with one of
    rank 0, and without."""
    K, N = 256, 72
    g = np.random.default_rng(M)
    d = _lora_inputs(M, K, N, 4, 16, g.integers(-1, 4, M), seed=M)
    d["ranks"][2] = 0
    t = {k: _dev(v) for k, v in d.items()}
    want = _lora_run(cq, d)
    y = torch.full((M, N + 40), 3.0, device=DEV)
    y[:, 16:16 + N] = t["y"]
    y0 = y.clone()
    out = torch.full((M, N + 12), 5.0, device=DEV)
    got = cq.cq_lora_add(t["x"], t["ids"], t["a"], t["b"], y[:, 16:16 + N], scale=t["scale"],
                         ranks=t["ranks"], out=out[:, 4:4 + N])
    assert torch.equal(got, want) and torch.equal(y, y0)
    assert (out[:, :4] == 5).all() and (out[:, 4 + N:] == 5).all()
    _lora_check(got, d)


def test_lora_add_in_a_workspace_of_the_caller(cq):
    """Calls of different sizes in turn in one buffer, each given exactly the bytes that
    its size function states: the results of the calls that allocate, and nothing
    written beside those bytes."""
    shapes = [(41, 64, 40, 9, 16), (300, 256, 136, 300, 8), (2100, 128, 72, 3, 128),
              (9000, 16, 24, 5, 8), (256, 2560, 264, 60, 64), (41, 64, 40, 4096, 8)]
    need = [cq.cq_lora_add_workspace_size(M, n, r) for M, _, _, n, r in shapes]
    assert min(need) > 0
    buf = torch.full((max(need) + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    for (M, K, N, n, r), size in list(zip(shapes, need)) * 2:
        g = np.random.default_rng(M)
        d = _lora_inputs(M, K, N, n, r, g.integers(-1, n, M), seed=M)
        want = _lora_run(cq, d)
        buf.fill_(0xA5)
        assert torch.equal(_lora_run(cq, d, workspace=buf[256:256 + size]), want)
        assert (buf[:256] == 0xA5).all() and (buf[256 + size:] == 0xA5).all()
        with pytest.raises(cq.CQError) as e:
            _lora_run(cq, d, workspace=buf[256:256 + size - 1])
        assert e.value.status == cq.CQ_ERR_WORKSPACE


@pytest.mark.parametrize("M", [40, 900])
def test_lora_add_rows_do_not_depend_on_their_neighbours(cq, M):
    """A row gives the same bits whatever adapters the other rows have, and a
    permutation of the rows permutes the results."""
    g = np.random.default_rng(6)
    d = _lora_inputs(M, 768, 256, 6, 32, g.integers(-1, 6, M), seed=6)
    base = _lora_run(cq, d).cpu().numpy()
    p = g.permutation(M)
    e = dict(d, x=d["x"][p], ids=d["ids"][p], y=d["y"][p])
    assert np.array_equal(_lora_run(cq, e).cpu().numpy(), base[p])
    assert np.array_equal(base[d["ids"] < 0], d["y"][d["ids"] < 0])   # untouched rows: y's bits


def test_lora_add_large_and_tiny_values(cq):
    """t far beyond fp16's range and far below its smallest step."""
    for size in (3e4, 1e-6):
        d = _lora_inputs(20, 1024, 64, 2, 16, np.arange(20) % 2, seed=8)
        d["x"] = np.clip(d["x"].astype(np.float32) * size, -6e4, 6e4).astype(np.float16)
        if size > 1:
            d["a"] = (d["a"].astype(np.float32) * 100).astype(np.float16)
        _lora_check(_lora_run(cq, d), d)


@pytest.mark.parametrize("r", [8, 32, 64, 128])
@pytest.mark.parametrize("M", [40, 600, 2100])
def test_lora_add_infinite_and_nan_rows(cq, M, r):
    """An infinite x gives what the sums give, at rank 1 an infinity; a NaN stays in
    its row; adapters' unused parts hold NaN."""
    d = _lora_inputs(M, 256, 64, 3, r, np.arange(M) % 3 - 1, seed=M + r)
    d["ranks"] = np.array([1, r - 3, r], np.int32)
    d["a"][0, 1:], d["b"][0, :, 1:] = np.nan, np.nan
    d["a"][1, r - 3:], d["b"][1, :, r - 3:] = np.nan, np.nan
    bad = [1, 2, 4, M - 2, M - 1]
    for i, v in zip(bad, (np.inf, np.nan, -np.inf, np.inf, -np.inf)):
        d["x"][i, 17 + i % 7] = v
    got = _lora_run(cq, d)
    ok = np.setdiff1d(np.arange(M), bad)
    _lora_check(got[torch.from_numpy(ok).to(DEV)], dict(d, x=d["x"][ok], ids=d["ids"][ok], y=d["y"][ok]))
    for m in bad:
        i = d["ids"][m]
        want = d["y"][m].astype(np.float64)
        if i >= 0:
            k = d["ranks"][i]
            with np.errstate(invalid="ignore"):
                t = d["a"][i, :k].astype(np.float64) @ d["x"][m].astype(np.float64)
                want = want + float(d["scale"][i]) * (d["b"][i, :, :k].astype(np.float64) @ t)
            if k == 1 and not np.isnan(d["x"][m]).any():
                assert np.isinf(want).all()
        np.testing.assert_array_equal(got[m].cpu().numpy(), want.astype(np.float32))


def test_lora_add_refusals(cq):
    d = {k: _dev(v) for k, v in _lora_inputs(4, 64, 32, 2, 8, [0, 1, 0, 1], seed=0).items()}
    ok = lambda **kw: cq.cq_lora_add(*[kw.get(k, d[k]) for k in ("x", "ids", "a", "b", "y")])  # noqa: E731
    for kw in (dict(ids=d["ids"].long()), dict(x=d["x"].float()), dict(x=d["x"].t().contiguous().t()),
               dict(y=d["y"].half()), dict(b=d["b"][:, :, :4]), dict(a=d["a"][:1]),
               dict(y=d["y"].t().contiguous().t()), dict(ids=d["ids"].cpu())):
        with pytest.raises(cq.CQError):
            ok(**kw)
    ok()


# ---------------------------------------------------------------- rotary positions


ROPE_CASES = [
    # (M, nq, nkv, D, rot, interleaved, norms, far, attn_scale, cache)
    (1, 32, 8, 128, 128, False, "qk", 4096, 1.0, None),
    (1, 1, 1, 8, 8, False, "", 10, 1.0, None),
    (3, 2, 1, 8, 8, True, "q", 10, 1.0, None),
    (5, 3, 1, 40, 16, False, "qk", 1000, 1.0, "rows"),
    (7, 7, 1, 80, 80, True, "k", 1 << 20, 1.3, "rows"),
    (33, 24, 4, 96, 64, True, "", 1 << 20, 1.2, "heads"),
    (64, 32, 4, 128, 128, False, "qk", 32768, 1.0, "rows"),
    (9, 4, 2, 256, 256, False, "qk", 1 << 30, 1.0, None),
    (9, 4, 2, 256, 72, True, "", 1 << 30, 1.0, "heads"),
    (11, 5, 5, 192, 0, False, "qk", 8, 1.0, "rows"),
    (2, 300, 10, 16, 8, False, "", 8, 0.5, None),
    (1021, 8, 2, 64, 32, False, "qk", 1 << 20, 1.0, "rows"),
    # heads whose units are not a power of two, in several rounds of one CTA
    (600, 30, 5, 80, 40, False, "", 32768, 1.0, "rows"),
    (601, 9, 3, 248, 248, True, "", 32768, 1.0, "heads"),
    (613, 6, 2, 24, 24, False, "", 32768, 0.7, None),
    (640, 16, 4, 64, 64, False, "", 32768, 1.0, "rows"),      # fewer threads than 256
    (602, 25, 2, 120, 64, False, "k", 32768, 1.0, "rows"),
]


@pytest.mark.parametrize("M,nq,nkv,D,rot,inter,norms,far,scale,cache", ROPE_CASES)
def test_rope_qkv_against_definition(cq, M, nq, nkv, D, rot, inter, norms, far, scale, cache):
    g = np.random.default_rng(M + D + rot)
    qkv = (3 * g.standard_normal((M, (nq + 2 * nkv) * D))).astype(np.float32)
    pos = g.integers(0, far, M).astype(np.int32)
    if M > 2:
        pos[1], pos[2], qkv[0, :D] = -5, 0, 0        # before the start, the start, a zero head
    freq = cq.rope_inv_freq(rot, 1e4, "parts", factor=4.0, context=4096) if rot else None
    qw = (1 + 0.3 * g.standard_normal(D)).astype(np.float16) if "q" in norms else None
    kw = (1 + 0.3 * g.standard_normal(D)).astype(np.float16) if "k" in norms else None
    dv = lambda a: None if a is None else _dev(a)  # noqa: E731
    args = dict(head_dim=D, interleaved=inter, attn_scale=scale, q_weight=dv(qw), k_weight=dv(kw),
                eps=1e-6)
    rows = None
    if cache:
        R = 2 * M + 3
        shape = (R, nkv, D) if cache == "rows" else (nkv, R, D)
        kc = torch.full(shape, 9.0, dtype=torch.float16, device=DEV)
        vc = torch.full(shape, 9.0, dtype=torch.float16, device=DEV)
        if cache == "heads":                          # a cache with the heads outermost
            kc, vc = kc.transpose(0, 1), vc.transpose(0, 1)
        rows = g.permutation(R)[:M].astype(np.int64)
        if M > 4:
            rows[0], rows[3] = -1, R                  # no place in the cache
        args.update(k_out=kc, v_out=vc, slots=_dev(rows))
    q, k, v = cq.cq_rope_qkv(_dev(qkv), _dev(pos), dv(freq), nq, nkv, **args)
    torch.cuda.synchronize()
    f = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
    want, tol = ref.rope_qkv(f(qkv), f(pos), f(freq), nq, nkv, D, inter, scale, f(qw), f(kw), 1e-6)
    got = [t.cpu().numpy().astype(np.float64) for t in (q, k, v)]
    if cache:
        live = (rows >= 0) & (rows < R)
        for i in (1, 2):
            rest = np.ones(R, bool)
            rest[rows[live]] = False
            assert np.all(got[i][rest] == 9.0)        # other rows as they were
        got = [got[0]] + [t[rows[live]] for t in got[1:]]
        want = [want[0]] + [t[live] for t in want[1:]]
        tol = [tol[0]] + [t[live] for t in tol[1:]]
    for a, b, t in zip(got, want, tol):
        assert a.shape == b.shape
        assert np.all(np.abs(a - b) <= t), float((np.abs(a - b) / t).max())


@pytest.mark.parametrize("eps", [1e-12, 1e-2, 5.0])
def test_rope_qkv_eps_is_the_one_given(cq, eps):
    """As above: eps is fp32, an input of the same formula."""
    M, nq, nkv, D = 6, 3, 2, 48
    g = np.random.default_rng(1)
    qkv = (g.standard_normal((M, (nq + 2 * nkv) * D)) *
           np.logspace(-3, 1, M)[:, None]).astype(np.float32)
    w = [(1 + 0.3 * g.standard_normal(D)).astype(np.float16) for _ in range(2)]
    pos = np.arange(M, dtype=np.int32)
    freq = cq.rope_inv_freq(D)
    got = cq.cq_rope_qkv(_dev(qkv), _dev(pos), _dev(freq), nq, nkv, head_dim=D, q_weight=_dev(w[0]),
                         k_weight=_dev(w[1]), eps=eps)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    want, tol = ref.rope_qkv(f(qkv), f(pos), f(freq), nq, nkv, D, False, 1.0, f(w[0]), f(w[1]),
                             float(np.float32(eps)))
    for a, b, t in zip(got, want, tol):
        assert np.all(np.abs(ref.f64(a) - b) <= t)


def test_rope_qkv_keeps_the_dot_product_of_equal_distances(cq):
    """Rotation by position: q.k depends on the distance alone (fp16 outputs: each
    entry is off by 2^-11 of itself, so the dot by 2^-10 sum|q k| and a little)."""
    M, D = 6, 64
    g = np.random.default_rng(0)
    one = g.standard_normal(3 * D).astype(np.float32)
    qkv = _dev(np.tile(one, (M, 1)))
    pos = np.array([0, 17, 1000, 1017, 500000, 500017], np.int32)
    q, k, _ = cq.cq_rope_qkv(qkv, _dev(pos), _dev(cq.rope_inv_freq(D)), 1, 1, head_dim=D)
    q, k = ref.f64(q)[:, 0], ref.f64(k)[:, 0]
    d = [float(q[i + 1] @ k[i]) for i in (0, 2, 4)]
    size = max(float(np.abs(q[i + 1]) @ np.abs(k[i])) for i in (0, 2, 4))
    assert max(d) - min(d) <= 2 * (2.0 ** -10 + 1e-5) * size


def test_rope_qkv_into_a_cache_of_sequences(cq):
    """A cache [sequence, head, token, channel]: token stride D, head stride
    tokens * D, and sequence m's token p at row m * heads * tokens + p of a strided
    view (the decoder-layer leg of bench.py writes its cache so)."""
    M, nq, nkv, D, ctx = 5, 4, 2, 32, 7
    g = np.random.default_rng(3)
    qkv = _dev(g.standard_normal((M, (nq + 2 * nkv) * D)).astype(np.float32))
    pos = g.integers(0, ctx, M).astype(np.int32)
    freq = _dev(cq.rope_inv_freq(D))
    q0, k0, v0 = cq.cq_rope_qkv(qkv, _dev(pos), freq, nq, nkv, head_dim=D)
    kc = torch.full((M, nkv, ctx, D), 5.0, dtype=torch.float16, device=DEV)
    vc = torch.full_like(kc, 6.0)

    def rows(c):
        return c.as_strided((M * nkv * ctx - (nkv - 1) * ctx, nkv, D), (D, ctx * D, 1))

    slots = torch.arange(M, device=DEV) * (nkv * ctx) + _dev(pos.astype(np.int64))
    q1, _, _ = cq.cq_rope_qkv(qkv, _dev(pos), freq, nq, nkv, head_dim=D, k_out=rows(kc),
                              v_out=rows(vc), slots=slots)
    want_k, want_v = torch.full_like(kc, 5.0), torch.full_like(kc, 6.0)
    for m in range(M):
        want_k[m, :, pos[m]], want_v[m, :, pos[m]] = k0[m], v0[m]
    assert torch.equal(q0, q1) and torch.equal(kc, want_k) and torch.equal(vc, want_v)


@pytest.mark.parametrize("M,nkv,ts,hs", [
    (3, 2, 2, 1),      # rows of a token
    (3, 2, 1, 3),      # heads outermost
    (3, 2, 5, 2),      # gaps between heads and rows
    (3, 2, 2, 3),      # neither inside the other, and nothing shared
    (1, 3, 0, 1),      # one row: its stride does not matter
    (4, 1, 1, 0),      # one head: the same
])
def test_rope_qkv_writes_any_rows_that_share_nothing(cq, M, nkv, ts, hs):
    """k and v rows without slots, strides in heads of 16 channels."""
    nq, D = 2, 16
    g = np.random.default_rng(M + 10 * nkv)
    qkv = _dev(g.standard_normal((M, (nq + 2 * nkv) * D)).astype(np.float32))
    pos = _dev(np.arange(M, dtype=np.int32))
    freq = _dev(cq.rope_inv_freq(D))
    _, k0, v0 = cq.cq_rope_qkv(qkv, pos, freq, nq, nkv, head_dim=D)
    n = ((M - 1) * ts + (nkv - 1) * hs + 1) * D
    bufs = [torch.full((n + 8,), 9.0, dtype=torch.float16, device=DEV) for _ in range(2)]
    want = [b.clone() for b in bufs]
    kv = [b[:n].as_strided((M, nkv, D), (ts * D, hs * D, 1)) for b in bufs]
    cq.cq_rope_qkv(qkv, pos, freq, nq, nkv, head_dim=D, k_out=kv[0], v_out=kv[1])
    for w, b, ref0 in zip(want, bufs, (k0, v0)):
        w[:n].as_strided((M, nkv, D), (ts * D, hs * D, 1)).copy_(ref0)
        assert torch.equal(w, b)
    if M > 1 and nkv > 1:
        with pytest.raises(cq.CQError):
            same = [b[:n].as_strided((M, nkv, D), (D, D, 1)) for b in bufs]
            cq.cq_rope_qkv(qkv, pos, freq, nq, nkv, head_dim=D, k_out=same[0], v_out=same[1])


def test_rope_qkv_refusals(cq):
    qkv = torch.zeros((2, 64), device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    k = torch.zeros((4, 1, 16), dtype=torch.float16, device=DEV)
    for kw in (dict(positions=pos.long()), dict(qkv=qkv.half()), dict(n_q=3), dict(k_out=k),
               dict(slots=pos.long()), dict(slots=pos, k_out=k, v_out=k.clone()),
               dict(k_out=k[:1], v_out=k[:1].clone()),
               dict(k_out=k, v_out=torch.zeros((1, 4, 16), dtype=torch.float16, device=DEV).transpose(0, 1))):
        a = dict(qkv=qkv, positions=pos, inv_freq=None, n_q=2, n_kv=1, head_dim=16)
        a.update(kw)
        with pytest.raises(cq.CQError):
            cq.cq_rope_qkv(**a)
    q, ko, vo = cq.cq_rope_qkv(qkv, pos, None, 2, 1, head_dim=16)
    assert q.shape == (2, 2, 16) and ko.shape == vo.shape == (2, 1, 16)


# ---------------------------------------------------------------- used together


class _Layer:
    """The path around one QKV projection of a decoder layer: residual norm with
    codes, the LUT product, the adapters, rotary positions and cache rows."""

    def __init__(self, cq, M, seed):
        H, nq, nkv, D, n = 512, 4, 2, 64, 3
        self.cq, self.H, self.nq, self.nkv, self.D = cq, H, nq, nkv, D
        N = (nq + 2 * nkv) * D
        g = np.random.default_rng(seed)
        self.d = _norm_inputs(M, H, "rms", 16, True, False, "none", seed=seed)
        self.lora = _lora_inputs(M, H, N, n, 16, g.integers(-1, n, M), seed=seed)
        self.w, self.cb = synth.lut_weights(N, H, seed=seed, name="layer_ops.w")
        self.pos = g.integers(0, 5000, M).astype(np.int32)
        self.freq = cq.rope_inv_freq(D)
        self.slots = g.permutation(2 * M)[:M].astype(np.int64)
        self.t = {k: _dev(v) for k, v in self.lora.items() if k != "x"}
        for k in ("resid", "y"):
            self.t["n" + k] = _dev(self.d[k])
        self.t.update(pre=_dev(self.d["pre"][0]), w=_dev(self.w), cb=_dev(self.cb),
                      pos=_dev(self.pos), freq=_dev(self.freq), slots=_dev(self.slots))
        self.k = torch.zeros((2 * M, nkv, D), dtype=torch.float16, device=DEV)
        self.v = torch.zeros_like(self.k)

    def run(self, stream=None):
        cq, t = self.cq, self.t
        r, x, q, s = cq.cq_residual_norm(t["nresid"], t["ny"], pre_weight=t["pre"], had_block=512,
                                         act_bits=4, stream=stream)
        base = cq.cq_lut_gemm(q, s, self.H, 4, t["w"], t["cb"], stream=stream)
        full = cq.cq_lora_add(x, t["ids"], t["a"], t["b"], base, scale=t["scale"],
                              ranks=t["ranks"], out=torch.empty_like(base), stream=stream)
        qo, _, _ = cq.cq_rope_qkv(full, t["pos"], t["freq"], self.nq, self.nkv, head_dim=self.D,
                                  k_out=self.k, v_out=self.v, slots=t["slots"], stream=stream)
        return r, x, q, s, base, full, qo, self.k, self.v


@pytest.mark.parametrize("M", [1, 16, 300])
def test_chain_around_a_projection(cq, M):
    L = _Layer(cq, M, seed=M)
    r, x, q, s, base, full, qo, kc, vc = L.run()
    torch.cuda.synchronize()
    rr, xr = _norm_ref(L.d, "rms", 1.0, 1.0)
    assert np.array_equal(r.cpu().numpy(), rr) and np.array_equal(x.cpu().numpy(), xr)
    qr, sr = oracle.rotate_quantize(xr, 512, 4)
    assert np.array_equal(oracle.unpack_codes(q.cpu().numpy(), L.H, 4), qr)
    yr, mag, _ = oracle.lut_gemm(qr, sr, L.w, L.cb)
    assert np.all(np.abs(base.cpu().numpy() - yr) <= oracle.lut_tolerance(mag))
    d = dict(L.lora, x=xr, y=base.cpu().numpy())
    _lora_check(full, d)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    want, tol = ref.rope_qkv(ref.f64(full), f(L.pos), f(L.freq), L.nq, L.nkv, L.D, False, 1.0,
                             None, None, 1e-6)
    for got, w, t in zip((ref.f64(qo), ref.f64(kc)[L.slots], ref.f64(vc)[L.slots]), want, tol):
        assert np.all(np.abs(got - w) <= t)


@pytest.mark.parametrize("M", [2, 700])
def test_chain_captured_replayed_and_on_two_streams(cq, M):
    """A captured chain replays the eager bits, on new inputs too; two chains with
    their own buffers on two streams do not disturb each other."""
    A, B = _Layer(cq, M, seed=1), _Layer(cq, M, seed=2)
    want = [[t.clone() for t in L.run()] for L in (A, B)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = A.run()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want[0]):
        assert torch.equal(a, b)
    # the replay reads what its inputs hold now
    A.t["ny"].mul_(-2)
    A.t["ids"].copy_(A.t["ids"].flip(0))
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    for a, b in zip(A.run(), got):
        assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    A2, B2 = _Layer(cq, M, seed=1), _Layer(cq, M, seed=2)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            o1 = A2.run()
        with torch.cuda.stream(s2):
            o2 = B2.run()
    torch.cuda.synchronize()
    for o, w in ((o1, want[0]), (o2, want[1])):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


def test_calls_are_counted_and_timed_by_kind(cq):
    L = _Layer(cq, 4, seed=3)
    L.run()
    torch.cuda.synchronize()
    before = cq.cq_launch_count()
    cq.cq_timing_enable(True, every_kernel=True)
    L.run()
    cq.cq_timing_enable(False)
    kinds = [k for k, _ in cq.cq_timing_read_launches()]
    assert cq.cq_launch_count() - before >= 4
    for k in ("residual_norm", "lora_add", "rope_qkv"):
        assert k in kinds


@pytest.mark.parametrize("M", [3, 700])
def test_calls_on_a_given_stream(cq, M):
    """stream= takes a torch stream or its address; what the call allocates belongs
    to that stream, so its memory is not handed to another one's work too early."""
    A = _Layer(cq, M, seed=4)
    want = [t.clone() for t in A.run()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (s, s.cuda_stream):
        for _ in range(3):
            got = A.run(stream=st)
            junk = torch.full((M * 2048,), float("nan"), device=DEV)   # current stream's memory
            del junk
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    with pytest.raises(AttributeError):
        cq.cq_residual_norm(A.t["nresid"], stream="no stream")


def test_refusals_name_the_call_and_the_operand(cq):
    h = torch.zeros((2, 64), dtype=torch.float16, device=DEV)
    y = torch.zeros((2, 64), device=DEV)
    w = torch.zeros(64, dtype=torch.float16, device=DEV)
    for kw, word in ((dict(y=y.half()), "y"), (dict(y=y[:1]), "y"), (dict(pre_weight=w.float()), "pre_weight"),
                     (dict(y=y, gate=w[:32]), "gate"), (dict(x_out=h.t()), "x_out"),
                     (dict(q_out=h), "act_bits"), (dict(act_bits=3), "act_bits"),
                     (dict(resid_out=h), "resid_out"), (dict(norm="batch"), "norm"),
                     (dict(y=y, post_weight=w), ""), (dict(pre_bias=w), ""),
                     (dict(act_bits=4, had_block=3), ""), (dict(eps=0.0), ""),
                     (dict(y=y, x_out=h), ""), (dict(pre_weight=w.cpu()), "pre_weight"),
                     (dict(pre_weight=3), "pre_weight")):
        with pytest.raises(cq.CQError) as e:
            cq.cq_residual_norm(h, **kw)
        assert e.value.status in (cq.CQ_ERR_INVALID_ARGUMENT, cq.CQ_ERR_UNSUPPORTED)
        assert "cq_residual_norm" in str(e.value) and word in str(e.value)
    with pytest.raises(cq.CQError):
        cq.cq_residual_norm(h[:, :32])                       # rows of a wider tensor
    with pytest.raises(cq.CQError):
        cq.cq_residual_norm(torch.zeros((2, 12), dtype=torch.float16, device=DEV))
    with pytest.raises(TypeError):
        cq.cq_residual_norm(h, eps="small")
    r, x = cq.cq_residual_norm(h)
    assert r is h and (x == 0).all()


@pytest.mark.parametrize("M", [1, 5])
def test_decoder_layer_step_of_the_benchmark_is_the_same_layer(cq, M):
    """The step with these operators gives the hidden state and the cache rows of the
    step with torch norms and rotary positions.  They differ by what rounding moves
    between two int4 codes.  With s the spread of a row, its codes are s / 2 apart:
    a difference of e s in the row moves a share of 2 e of the codes by one, which
    is a difference of sqrt(2 e) / 2.  The new k and v rows: x differs by an fp16 step
    in at most 1 % of the channels (e <= 1e-4): 0.7 %, and 2^-11 of rounding; bound 2 %.
    The state: that 1 % in the attention's output becomes 7 % of o, which is 0.06 of the
    state: 0.5 %; 5 % in the gate and up products, 6 % in h, 17 % in the FFN's output,
    which is 1.2 of a state of 1.6: 13 %; bound 30 %.  Without the FFN's output it
    would be off by 75 %."""
    import bench
    g = torch.Generator(device=DEV).manual_seed(5)
    ctx = 200
    steps, layers = bench.decoder_layer_steps(cq, M, ctx, 1, torch.device(DEV), g)
    L = layers[0]
    old = L["kc"].clone(), L["vc"].clone()
    state, rows = {}, {}
    for nm in ("lut", "lut_ops"):
        L["kc"].copy_(old[0])
        L["vc"].copy_(old[1])
        state[nm] = steps[nm]().double()
        rows[nm] = [c[:, :, ctx].double() for c in (L["kc"], L["vc"])]
        assert torch.equal(L["kc"][:, :, :ctx], old[0][:, :, :ctx])
        assert torch.equal(L["vc"][:, :, :ctx], old[1][:, :, :ctx])

    def off(a, b):
        return float((a - b).norm() / b.norm())

    assert state["lut"].shape == state["lut_ops"].shape == (M, 2560)
    assert off(state["lut_ops"], state["lut"]) <= 0.3
    for a, b, c in zip(rows["lut_ops"], rows["lut"], old):
        assert off(a, b) <= 0.02 and off(c[:, :, ctx].double(), b) > 0.5
