"""Operators between two LUT linears, host side: the rotary frequency tables,
and every argument check of the three C entry points (nothing is launched)."""
import ctypes
import importlib.util
import math
import os
import shutil
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import lut_clustered_weight_b200 as cq

FAKE = 1 << 20  # a 16-byte aligned address that is never dereferenced
BAD, UNS, WSP, OK = (cq.CQ_ERR_INVALID_ARGUMENT, cq.CQ_ERR_UNSUPPORTED, cq.CQ_ERR_WORKSPACE,
                     cq.CQ_OK)


# ---------------------------------------------------------------- rotary tables


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 1e6), (96, 500.0)])
def test_plain_table(rot, base):
    t = cq.rope_inv_freq(rot, base)
    assert t.dtype == np.float32 and t.shape == (rot // 2,)
    for i in range(rot // 2):
        want = math.exp(-2 * i / rot * math.log(base))
        assert abs(float(t[i]) - want) <= want * (2.0 ** -24 + 1e-14)


def test_linear_and_base_scaling():
    plain = cq.rope_inv_freq(128, 1e4).astype(np.float64)
    lin = cq.rope_inv_freq(128, 1e4, "linear", factor=8.0)
    assert np.allclose(lin, plain / 8, rtol=2.0 ** -23, atol=0)
    b = cq.rope_inv_freq(128, 1e4, "base", factor=8.0)
    assert b[0] == 1.0                                            # fastest pair kept
    assert abs(b[-1] / (plain[-1] / 8) - 1) < 2.0 ** -22          # slowest divided by the factor
    assert np.all(np.diff(b) < 0)


def test_parts_scaling_keeps_fast_and_divides_slow_pairs():
    s, ctx = 4.0, 4096
    plain = cq.rope_inv_freq(128, 1e4).astype(np.float64)
    t = cq.rope_inv_freq(128, 1e4, "parts", factor=s, context=ctx).astype(np.float64)
    turns = ctx * plain / (2 * math.pi)
    fast, slow = turns >= 32 * (1 + 1e-6), turns <= 1 - 1e-6
    mid = (turns > 1 + 1e-6) & (turns < 32 * (1 - 1e-6))
    assert fast.any() and slow.any() and mid.any()
    assert np.allclose(t[fast], plain[fast], rtol=2.0 ** -22, atol=0)
    assert np.allclose(t[slow], plain[slow] / s, rtol=2.0 ** -22, atol=0)
    assert np.all((t[mid] < plain[mid]) & (t[mid] > plain[mid] / s))
    g = (turns[mid] - 1) / 31
    assert np.allclose(t[mid], plain[mid] * (g + (1 - g) / s), rtol=1e-6, atol=0)


@pytest.mark.parametrize("rot,base,s,ctx", [(128, 1e6, 4.0, 32768), (128, 1e4, 16.0, 4096),
                                            (64, 5e5, 8.0, 8192), (96, 1e4, 2.0, 100)])
def test_parts_scaling_by_index(rot, base, s, ctx):
    """Kept up to the last pair that makes 32 turns or more over the context, divided
    from the first that makes 1 or less, and between these two a line over the index."""
    t = cq.rope_inv_freq(rot, base, "parts", factor=s, context=ctx, ramp="index").astype(np.float64)
    plain = [math.exp(-2 * i / rot * math.log(base)) for i in range(rot)]
    turns = [ctx * f / (2 * math.pi) for f in plain]
    lo = max([i for i in range(rot) if turns[i] >= 32], default=0)
    hi = min([i for i in range(rot) if turns[i] <= 1], default=rot - 1)
    assert hi > lo
    for i in range(rot // 2):
        w = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert abs(t[i] / (plain[i] * (1 - w + w / s)) - 1) <= 2.0 ** -23
    other = cq.rope_inv_freq(rot, base, "parts", factor=s, context=ctx).astype(np.float64)
    assert np.abs(other / t - 1).max() > 0.1          # the two ramps are different tables
    assert np.array_equal(other, cq.rope_inv_freq(rot, base, "parts", s, ctx, ramp="turns"))


def test_ramp_refusals():
    parts = dict(rot_dim=8, scaling="parts", factor=2.0, context=4096)
    for kw in (dict(ramp="other"), dict(ramp="index", base=1.0), dict(ramp="index", slow_turns=0.0)):
        with pytest.raises(ValueError):
            cq.rope_inv_freq(**parts, **kw)


def test_table_refusals_and_attention_scale():
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, base=0.0),
               dict(rot_dim=8, factor=0.0), dict(rot_dim=8, scaling="other"),
               dict(rot_dim=8, scaling="parts", factor=2.0),
               dict(rot_dim=8, scaling="parts", factor=2.0, context=4096, slow_turns=4, fast_turns=4),
               dict(rot_dim=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            cq.rope_inv_freq(**kw)
    assert cq.rope_attn_scale(1.0) == 1.0 and cq.rope_attn_scale(0.5) == 1.0
    assert abs(cq.rope_attn_scale(16.0) - (0.1 * math.log(16) + 1)) < 1e-15


# ---------------------------------------------------------------- cq_residual_norm


def _norm_call(T=2, y=FAKE, gate=None, qw=None, qb=None, r=2 * FAKE, ro=3 * FAKE, pw=None, pb=None,
               x=4 * FAKE, q=5 * FAKE, s=6 * FAKE, desc=True, **kw):
    d = dict(H=64, norm=0, post_norm=0, gate_mode=0, resid_bits=16, had_block=16, act_bits=4,
             eps=1e-6, resid_scale=1.0, block_scale=1.0)
    d.update(kw)
    nd = cq.NormDesc(*[d[n] for n, _ in cq.NormDesc._fields_])
    return cq.lib.cq_residual_norm(ctypes.byref(nd) if desc else None, T, y, gate, qw, qb, r, ro,
                                   pw, pb, x, q, s, None)


def test_residual_norm_argument_checks():
    f = _norm_call
    nan, inf = float("nan"), float("inf")
    for kw in (dict(desc=False), dict(T=-1), dict(H=0), dict(norm=2), dict(norm=-1),
               dict(post_norm=2), dict(gate_mode=4, gate=FAKE), dict(gate_mode=-1),
               dict(resid_bits=8), dict(act_bits=5), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan),
               dict(eps=inf), dict(resid_scale=nan), dict(block_scale=inf), dict(had_block=12),
               dict(had_block=0), dict(had_block=128), dict(had_block=-16),
               dict(act_bits=0, q=None, s=None),                 # a block without codes
               dict(act_bits=0, had_block=0),                    # code outputs without codes
               dict(q=None), dict(s=None), dict(r=None), dict(x=None), dict(ro=None),
               dict(gate=FAKE), dict(gate_mode=1),               # gate iff its mode
               dict(qw=FAKE), dict(qb=FAKE),                     # post_* without post_norm
               dict(pb=FAKE), dict(post_norm=1, qb=FAKE),        # biases are LayerNorm's
               dict(y=None, post_norm=1), dict(y=None, gate_mode=1, gate=FAKE),
               dict(y=None, resid_scale=0.5), dict(y=None, block_scale=0.5),
               dict(x=2 * FAKE), dict(x=3 * FAKE), dict(x=FAKE), dict(ro=FAKE),   # overlaps
               dict(r=2 * FAKE + 8), dict(y=FAKE + 4), dict(x=4 * FAKE + 2), dict(q=5 * FAKE + 1),
               dict(s=6 * FAKE + 4), dict(pw=FAKE + 2), dict(gate_mode=2, gate=FAKE + 2)):
        assert f(**kw) == BAD, kw
    for kw in (dict(H=12, had_block=4), dict(H=32768), dict(T=1 << 31),
               dict(H=16384, had_block=16384)):
        assert f(**kw) == UNS, kw
    assert f(T=0) == OK
    assert f(T=0, y=None, ro=None) == OK
    assert f(T=0, norm=1, post_norm=1, qw=FAKE, qb=FAKE, pw=FAKE, pb=FAKE, gate_mode=3) == OK


# ---------------------------------------------------------------- cq_lora_add


def _lora_call(x=FAKE, ids=FAKE, M=3, K=64, a=FAKE, b=FAKE, sc=None, rk=None, n=2, r=16, y=FAKE,
               ldy=128, out=FAKE, ldo=128, N=128, ws=FAKE, wsb=1 << 40):
    return cq.lib.cq_lora_add(x, ids, M, K, a, b, sc, rk, n, r, y, ldy, out, ldo, N, ws, wsb, None)


def test_lora_add_argument_checks():
    f = _lora_call
    for kw in (dict(M=-1), dict(K=0), dict(N=0), dict(n=0), dict(r=0), dict(ldy=120), dict(ldo=64),
               dict(a=None), dict(b=None), dict(x=None), dict(ids=None), dict(y=None),
               dict(out=None), dict(ldo=256), dict(x=FAKE + 2), dict(a=FAKE + 8), dict(b=FAKE + 8),
               dict(sc=FAKE + 4), dict(rk=FAKE + 4), dict(y=FAKE + 4), dict(out=FAKE + 8),
               dict(ids=FAKE + 4), dict(ws=FAKE + 8)):
        assert f(**kw) == BAD, kw
    for kw in (dict(K=60), dict(N=124), dict(r=12), dict(r=136), dict(ldy=130, ldo=130),
               dict(n=4097), dict(M=(1 << 24) + 1), dict(K=(1 << 20) + 8),
               dict(N=(1 << 20) + 8, ldy=1 << 21, ldo=1 << 21)):
        assert f(**kw) == UNS, kw
    assert f(M=0) == OK
    assert f(M=0, x=None, ids=None, y=None, out=None, ws=None, wsb=0) == OK


def test_lora_add_workspace():
    for M in (1, 64, 4096, 1 << 20):
        for n in (1, 64, 4096):
            need = cq.cq_lora_add_workspace_size(M, n, 16)
            assert need <= cq.cq_lora_add_workspace_size(M, n, 128)
            if need:
                assert _lora_call(M=M, n=n, ws=None, wsb=0) == WSP
                assert _lora_call(M=M, n=n, wsb=need - 1) == WSP
    assert cq.cq_lora_add_workspace_size(0, 4, 16) == 0
    assert cq.cq_lora_add_workspace_size(-1, 4, 16) == 0


def test_lora_add_workspace_is_asked_for_above_40_rows():
    for M in (41, 64, 4096, 1 << 20):
        for n in (1, 4096):
            need = cq.cq_lora_add_workspace_size(M, n, 16)
            # the sorted rows' t in two fp16 parts, their factors, their list
            assert need >= M * (2 * 16 * 2 + 4 + 4)
            assert need < cq.cq_lora_add_workspace_size(2 * M, n, 16)
            assert need < cq.cq_lora_add_workspace_size(M, n, 128)
    for M in (1, 40):
        assert cq.cq_lora_add_workspace_size(M, 8, 16) == 0


# ---------------------------------------------------------------- cq_rope_qkv


def _rope_call(M=2, qkv=FAKE, pos=FAKE, freq=FAKE, qw=None, kw_=None, q=2 * FAKE, k=3 * FAKE,
               v=4 * FAKE, slots=None, desc=True, **kw):
    d = dict(n_q=4, n_kv=2, head_dim=64, rot_dim=64, kv_token_stride=128, kv_head_stride=64,
             n_slots=16, interleaved=0, attn_scale=1.0, eps=1e-6)
    d.update(kw)
    rd = cq.RopeDesc(*[d[n] for n, _ in cq.RopeDesc._fields_])
    return cq.lib.cq_rope_qkv(ctypes.byref(rd) if desc else None, M, qkv, pos, freq, qw, kw_, q, k,
                              v, slots, None)


def test_rope_qkv_argument_checks():
    f = _rope_call
    nan = float("nan")
    for kw in (dict(desc=False), dict(M=-1), dict(n_q=0), dict(n_kv=0), dict(head_dim=0),
               dict(rot_dim=-8), dict(rot_dim=72), dict(interleaved=2), dict(attn_scale=nan),
               dict(eps=0.0), dict(eps=nan), dict(kv_token_stride=-8), dict(kv_head_stride=-8),
               dict(slots=FAKE, n_slots=-1), dict(freq=None), dict(rot_dim=0), dict(qkv=None),
               dict(pos=None), dict(q=None), dict(k=None), dict(v=None), dict(v=3 * FAKE),
               dict(q=3 * FAKE), dict(qkv=FAKE + 4), dict(q=FAKE + 8), dict(k=3 * FAKE + 2),
               dict(slots=FAKE + 8), dict(qw=FAKE + 2), dict(kw_=FAKE + 2)):
        assert f(**kw) == BAD, kw
    for kw in (dict(head_dim=60, rot_dim=56), dict(head_dim=264), dict(rot_dim=60),
               dict(n_q=1023, n_kv=1), dict(n_kv=1025), dict(kv_token_stride=132),
               dict(kv_head_stride=68), dict(M=1 << 31)):
        assert f(**kw) == UNS, kw
    assert f(M=0) == OK
    assert f(M=0, rot_dim=0, freq=None, slots=FAKE) == OK


def test_rope_qkv_refuses_cache_rows_on_top_of_one_another():
    for kw in (dict(kv_head_stride=0), dict(kv_head_stride=56), dict(kv_token_stride=0),
               dict(kv_token_stride=56), dict(kv_token_stride=0, slots=FAKE)):
        assert _rope_call(**kw) == BAD, kw


def test_rope_qkv_refuses_heads_of_one_row_on_heads_of_another():
    """Without slots the rows written are known: strides that put head h of row m and
    another head of another row at common addresses are refused, each larger than a
    head though they be."""
    D = 16
    for M in (2, 3, 5):
        for nkv in (2, 3, 4):
            for ts in range(D, 8 * D, 8):
                for hs in range(D, 8 * D, 8):
                    at = sorted(m * ts + h * hs for m in range(M) for h in range(nkv))
                    if any(b - a < D for a, b in zip(at, at[1:])):
                        kw = dict(M=M, n_kv=nkv, head_dim=D, rot_dim=D, kv_token_stride=ts,
                                  kv_head_stride=hs)
                        assert _rope_call(**kw) == BAD, kw
    assert _rope_call(kv_token_stride=64) == BAD
    big = 1 << 62                              # no product of a stride and a count wraps
    assert _rope_call(M=1 << 20, n_kv=500, kv_token_stride=big, kv_head_stride=big) == BAD


# ---------------------------------------------------------------- the binding's checks


def test_binding_refuses_host_tensors_and_wrong_operands():
    h = torch.zeros((2, 64), dtype=torch.float16)
    with pytest.raises(cq.CQError) as e:
        cq.cq_residual_norm(h)
    assert e.value.status == BAD
    with pytest.raises(cq.CQError):
        cq.cq_lora_add(h, torch.zeros(2, dtype=torch.int32), h[None], h[None], h.float())
    with pytest.raises(cq.CQError):
        cq.cq_rope_qkv(h.float(), torch.zeros(2, dtype=torch.int32), None, 2, 1, head_dim=16)


PKG = Path(cq.__file__).resolve().parent


def _python_in(folder, code):
    env = dict(os.environ, PYTHONPATH=str(folder))
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env,
                          cwd=folder, timeout=300)


@pytest.mark.parametrize("module", ["absent", "not a library"])
def test_package_without_the_binding_module_has_everything_else(tmp_path, module):
    """Only the three calls that it marshals fail, and say how to build it."""
    to = tmp_path / PKG.name
    to.mkdir()
    for f in PKG.glob("*.py"):
        shutil.copy(f, to)
    (to / "libcq_b200.so").symlink_to(PKG / "libcq_b200.so")
    if module != "absent":
        (to / "_cq_bind.so").write_bytes(b"no library")
    r = _python_in(tmp_path, f"""
import {PKG.name} as cq, torch
assert cq.__file__.startswith({str(tmp_path)!r})
assert cq.status_string(0) and cq.rope_inv_freq(8).shape == (4,)
h = torch.zeros((2, 64), dtype=torch.float16)
n = 0
for call in (lambda: cq.cq_residual_norm(h), lambda: cq.cq_lora_add(h, h, h, h, h),
             lambda: cq.cq_rope_qkv(h, h, None, 2, 1, head_dim=16)):
    try:
        call()
    except ImportError as e:
        assert "_cq_bind" in str(e) and "build.py" in str(e), e
        n += 1
assert n == 3
""")
    assert r.returncode == 0, r.stderr


def test_binding_module_of_another_torch_is_not_used():
    from types import SimpleNamespace
    assert cq._usable_bind(SimpleNamespace(torch_version=torch.__version__)) is None
    for m in (SimpleNamespace(), SimpleNamespace(torch_version="1.0")):
        assert "torch" in cq._usable_bind(m)
    assert cq._bind.torch_version == torch.__version__


def test_binding_module_is_built_again_for_another_torch_and_left_out_without_a_compiler(
        tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_cq_build_test", PKG / "build.py")
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert b.torch_version() == torch.__version__
    ran = []
    monkeypatch.setattr(b, "_run", lambda cmd, *a, **k: (ran.append(cmd), Path(
        cmd[cmd.index("-o") + 1]).write_bytes(b"")))
    monkeypatch.setattr(b, "BIND", tmp_path / "_cq_bind.so")
    monkeypatch.setattr(b, "BIND_STAMP", tmp_path / "stamp")
    b.build_bind()
    assert len(ran) == 1 and b.BIND.exists()
    b.build_bind()
    assert len(ran) == 1                                   # nothing changed
    monkeypatch.setattr(b, "torch_version", lambda: "9.9")
    b.build_bind()
    assert len(ran) == 2
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    monkeypatch.setattr(b, "torch_version", lambda: "9.8")
    with pytest.warns(UserWarning, match="g[+][+]"):
        b.build_bind()
    assert len(ran) == 2
