"""CPU checks of the operators that serve from the paged cache: struct layouts as
a C99 compiler sees them, the frequencies' fixed-point form, and every refusal
that happens before a CUDA call."""
import ctypes
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest
import torch

from block_diffusion_lm_gb300 import csbp
from oracle import generate_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000          # aligned, never dereferenced on these paths
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_lm_gb300 import build
    build.build()


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"csbp_rotary": csbp.RotaryStruct, "csbp_append_queries": csbp.AppendQueries,
               "csbp_paged_problem": csbp.PagedProblem, "csbp_paged_inputs": csbp.PagedInputs}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "csbp_generate.h"',
             'int main(void) {']
    for name, s in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = str(tmp_path / "layout")
    r = subprocess.run([cc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = dict(ln.split() for ln in subprocess.run([exe], capture_output=True,
                                                   text=True).stdout.splitlines())
    for name, s in structs.items():
        assert int(out[name]) == ctypes.sizeof(s), name
        for f, _ in s._fields_:
            assert int(out[f"{name}.{f}"]) == getattr(s, f).offset, (name, f)


# ----------------------------------------------------------------- rotary form
def turns_of(freq):
    n = len(freq)
    out = (ctypes.c_uint64 * n)()
    st = csbp.lib().csbp_rotary_turns((ctypes.c_double * n)(*freq), n, out)
    return st, list(out)


def test_rotary_turns_are_the_nearest_fixed_point_numbers():
    """Within half a unit of 2^-64 turns (and the oracle's pi to 60 digits)."""
    rng = random.Random(5)
    freq = [rng.choice((-1, 1)) * 10 ** rng.uniform(-12, 6) for _ in range(500)]
    freq += [0.0, -0.0, 1.0, 2.0 ** 20, -2.0 ** 20, 5e-324, 2.0 ** -70]
    freq += [1e6 ** (-i / 64) for i in range(64)]
    st, got = turns_of(freq)
    assert st == OK
    two_pi = Fraction(O._TWO_PI, 10 ** 60)
    for f, t in zip(freq, got):
        d = (Fraction(f) / two_pi * 2 ** 64 - t) % 2 ** 64
        assert min(d, 2 ** 64 - d) <= Fraction(1, 2) + Fraction(1, 1000), f


def test_bad_frequencies_are_refused():
    for bad in (float("nan"), float("inf"), 2.0 ** 20 + 1, -1e7):
        assert turns_of([1.0, bad])[0] == INVALID
    assert csbp.lib().csbp_rotary_turns(None, 1, (ctypes.c_uint64 * 1)()) == INVALID
    assert csbp.lib().csbp_rotary_turns(None, 0, None) == OK
    with pytest.raises(csbp.CsbpError):
        csbp.Rotary([1.0] * 7 + [1e9], device="cpu")
    for n in (0, 4, 9):
        with pytest.raises(ValueError, match="multiple of 8"):
            csbp.Rotary([1.0] * n, device="cpu")


# ----------------------------------------------------------------------- C ABI
def cache(**kw):
    c = csbp.KvCache(10, 16, 4, 64, PTR, PTR, PTR, PTR)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rows(tok=(0, 0), bat=(0, 0), **kw):
    r = csbp.CacheRows(2, 8, 5, PTR, PTR, PTR, tok, bat)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def rotary(**kw):
    r = csbp.RotaryStruct(64, 0, PTR)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def queries(tok=(0, 0), bat=(0, 0), **kw):
    q = csbp.AppendQueries(8, 0, PTR, PTR, tok, bat)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def append(c=None, r=None, ro=None, q=None, k=PTR, v=PTR):
    c, r, ro = c or cache(), r or rows(), ro or rotary()
    return csbp.lib().csbp_cache_append(ctypes.byref(c), ctypes.byref(r), ctypes.byref(ro), k, v,
                                        None if q is None else ctypes.byref(q), None)


def test_bad_appends_are_refused():
    for kw in (dict(pages=0), dict(page_size=0), dict(d=48), dict(k=None), dict(v=PTR + 8)):
        assert append(c=cache(**kw)) == INVALID
    for kw in (dict(batch=-1), dict(table=None), dict(start=PTR + 2), dict(tok=(128, 0)),
               dict(bat=(2052, 0))):
        assert append(r=rows(**kw)) == INVALID
    for kw in (dict(dim=0), dict(dim=8), dict(dim=24), dict(dim=80), dict(dim=-16),
               dict(interleaved=2), dict(turns=None), dict(turns=PTR + 4)):
        assert append(ro=rotary(**kw)) == INVALID
    for kw in (dict(Hq=-1), dict(clear=2), dict(clear=-1), dict(q=None), dict(out=None),
               dict(q=PTR + 8), dict(out=PTR + 4),
               dict(tok=(504, 0)), dict(tok=(0, 516)), dict(bat=(4088, 0)), dict(bat=(0, 4100)),
               dict(tok=(-512, 0)), dict(bat=(0, 1 << 60)), dict(tok=(1 << 60, 0))):
        assert append(q=queries(**kw)) == INVALID
    assert append(k=None) == INVALID
    assert append(v=PTR + 2) == INVALID
    assert append(c=cache(d=1024), ro=rotary(dim=64)) == UNSUPPORTED
    assert append(q=queries(Hq=65537)) == UNSUPPORTED
    assert append(r=rows(batch=0)) == OK
    assert append(r=rows(rows=0), k=None, v=None) == OK
    L = csbp.lib()
    c, r, ro = (ctypes.byref(x) for x in (cache(), rows(), rotary()))
    assert L.csbp_cache_append(None, r, ro, PTR, PTR, None, None) == INVALID
    assert L.csbp_cache_append(c, None, ro, PTR, PTR, None, None) == INVALID
    assert L.csbp_cache_append(c, r, None, PTR, PTR, None, None) == INVALID


def problem(**kw):
    p = csbp.PagedProblem(2, 3, 5, 8, 1, 0, 0, 0.125)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def inputs(**kw):
    i = csbp.PagedInputs(PTR, 0, 0, PTR, PTR)
    for k, v in kw.items():
        setattr(i, k, v)
    return i


def attn(p=None, c=None, i=None, o=PTR, lse=PTR, ws=PTR, n=1 << 40):
    p, c, i = p or problem(), c or cache(), i or inputs()
    return csbp.lib().csbp_attn_paged(ctypes.byref(p), ctypes.byref(c), ctypes.byref(i), o, lse,
                                      ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), INVALID), (dict(queries=0), INVALID), (dict(table_pages=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Hq=6), INVALID), (dict(causal=2), INVALID),
    (dict(causal=-1), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(table_pages=1 << 27), UNSUPPORTED),
    (dict(batch=1 << 28, queries=1 << 20), UNSUPPORTED)])
def test_bad_paged_problems_are_refused(kw, want):
    p = problem(**kw)
    assert csbp.paged_workspace_bytes(p, cache()) == 0
    assert attn(p=p) == want


def test_bad_paged_calls_are_refused():
    for kw, want in ((dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(d=48), INVALID),
                     (dict(Hkv=3), INVALID), (dict(page_size=0), INVALID)):
        assert attn(c=cache(**kw)) == want
        assert csbp.paged_workspace_bytes(problem(), cache(**kw)) == 0
    for kw in (dict(pages=1 << 27), dict(pages=1 << 26, page_size=16, Hkv=4)):
        assert attn(c=cache(**kw)) == UNSUPPORTED
    assert attn(c=cache(pages=(1 << 26) - 1, page_size=16, Hkv=4), n=256) == WORKSPACE
    for kw in (dict(pages=0), dict(pages=1 << 31), dict(k=None), dict(v_scale=None),
               dict(v=PTR + 8)):
        assert attn(c=cache(**kw)) == INVALID
    for kw in (dict(q=None), dict(table=None), dict(length=None), dict(q=PTR + 8),
               dict(table=PTR + 2), dict(length=PTR + 1), dict(stride_tok=504),
               dict(stride_tok=516), dict(stride_tok=-512), dict(stride_batch=1528),
               dict(stride_batch=1540), dict(stride_tok=1 << 60), dict(stride_batch=1 << 60)):
        assert attn(i=inputs(**kw)) == INVALID
    for kw in (dict(o=None), dict(lse=None), dict(ws=None), dict(o=PTR + 8), dict(lse=PTR + 2),
               dict(ws=PTR + 8)):
        assert attn(**kw) == INVALID
    assert attn(n=255) == WORKSPACE
    # sizes alone are enough to ask for the workspace
    n = csbp.paged_workspace_bytes(problem(), csbp.KvCache(0, 16, 4, 64))
    assert n >= 256 and attn(n=n - 1) == WORKSPACE
    L = csbp.lib()
    p, c, i = (ctypes.byref(x) for x in (problem(), cache(), inputs()))
    assert L.csbp_attn_paged(None, c, i, PTR, PTR, PTR, 1 << 40, None) == INVALID
    assert L.csbp_attn_paged(p, None, i, PTR, PTR, PTR, 1 << 40, None) == INVALID
    assert L.csbp_attn_paged(p, c, None, PTR, PTR, PTR, 1 << 40, None) == INVALID
    assert L.csbp_paged_workspace_bytes(None, c) == 0 == L.csbp_paged_workspace_bytes(p, None)


# --------------------------------------------------------------------- binding
def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_append_binding_checks():
    c = csbp.QuantCache(6, 16, 2, 64, device="cpu")
    ro = csbp.Rotary([1.0] * 32, device="cpu")
    k = z(3, 5, 2, 64)
    args = dict(k=k, v=k.clone(), table=i32(3, 2), start=i32(3), rotary=ro)
    q = z(3, 5, 4, 64)
    for kw, msg in [
            (dict(k=k.float()), "k must be torch.bfloat16"),
            (dict(v=z(3, 5, 2, 32)), "v must have shape"),
            (dict(count=i32(2)), "count must have shape"),
            (dict(rotary=None), "must be a Rotary"),
            (dict(rotary=csbp.Rotary([1.0] * 40, device="cpu")), "80 features"),
            (dict(q=q.float()), "q must be torch.bfloat16"),
            (dict(q=z(3, 4, 4, 64)), "q must have shape"),
            (dict(q=z(3, 5, 256)), "q must be a"),
            (dict(q=z(5, 3, 4, 64).transpose(0, 1)), "must not interleave"),
            (dict(q=q[:1].expand(3, 5, 4, 64)), "must not interleave"),
            (dict(q=q, out=z(3, 5, 2, 64)), "out must have shape"),
            (dict(q=q, out=q[:, :1].expand(3, 5, 4, 64)), "token stride"),
            (dict(out=q), "out without q"),
            ({}, "must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            c.append(**{**args, **kw})
    e = z(0, 5, 2, 64)
    got = c.append(e, e, i32(0, 2), i32(0), rotary=ro, q=z(0, 5, 4, 64))
    assert got.shape == (0, 5, 4, 64)
    assert c.append(e, e, i32(0, 2), i32(0), rotary=ro) is None


def test_paged_binding_checks():
    c = csbp.QuantCache(6, 16, 2, 64, device="cpu")
    a = csbp.PagedAttention(2, 3, 4, 16, 8, 2, 64, device="cpu")
    args = dict(q=z(2, 3, 8, 64), cache=c, table=i32(2, 4), length=i32(2))
    for kw, msg in [
            (dict(q=None), "q is required"),
            (dict(q=z(2, 3, 8, 64).float()), "q must be torch.bfloat16"),
            (dict(q=z(2, 3, 4, 64)), "q must have shape"),
            (dict(q=z(2, 8, 3, 64).transpose(1, 2)), "contiguous heads"),
            (dict(q=z(1, 3, 8, 64).expand(2, 3, 8, 64)), "must not interleave"),
            (dict(cache=c.k), "must be a QuantCache"),
            (dict(cache=csbp.QuantCache(6, 8, 2, 64, device="cpu")), "the cache has"),
            (dict(cache=csbp.QuantCache(6, 16, 2, 32, device="cpu")), "the cache has"),
            (dict(table=i32(2, 3)), "table must have shape"),
            (dict(length=i32(2).long()), "length must be torch.int32"),
            ({}, "must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            a.forward(**{**args, **kw})
    o, lse = a.alloc_outputs()
    with pytest.raises(ValueError, match="o must be contiguous"):
        a.forward(**args, out=(z(2, 8, 3, 64).transpose(1, 2), lse))
    with pytest.raises(ValueError, match="lse must have shape"):
        a.forward(**args, out=(o, lse.transpose(1, 2)))
    for kw in (dict(Hq=7), dict(d=96), dict(window=-1), dict(scale=-1.0)):
        with pytest.raises(csbp.CsbpError):
            csbp.PagedAttention(**{**dict(batch=2, queries=3, table_pages=4, page_size=16, Hq=8,
                                          Hkv=2, d=64, device="cpu"), **kw})
