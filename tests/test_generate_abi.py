"""CPU checks of the generation operators' C ABI and binding: struct layouts
as a C99 compiler sees them, and every refusal that happens before a CUDA
call (none of these paths needs a GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from block_diffusion_lm_gb300 import csbp

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
    structs = {"csbp_kv_cache": csbp.KvCache, "csbp_cache_rows": csbp.CacheRows,
               "csbp_prefix_problem": csbp.PrefixProblem,
               "csbp_prefix_inputs": csbp.PrefixInputs,
               "csbp_verify_problem": csbp.VerifyProblem}
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


def test_header_compiles_as_cpp(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "use.cpp"
    src.write_text('#include "csbp_generate.h"\n'
                   'static_assert(sizeof(csbp_prefix_problem) > 0, "");\n'
                   'int main() { return csbp_prefix_workspace_bytes == nullptr; }\n')
    r = subprocess.run([cxx, "-std=c++11", "-pedantic", "-Wall", "-Wextra", "-Werror", "-c", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "use.o"),
                        "-Wno-address", "-Wno-nonnull-compare"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# ------------------------------------------------------------------- C ABI
def cache(**kw):
    c = csbp.KvCache(10, 16, 4, 64, PTR, PTR, PTR, PTR)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def cache_rows(tok=(0, 0), bat=(0, 0), **kw):
    r = csbp.CacheRows(2, 8, 5, PTR, PTR, PTR, tok, bat)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def both(c, r, k=PTR, v=PTR):
    L = csbp.lib()
    st = [f(ctypes.byref(c), ctypes.byref(r), k, v, None)
          for f in (L.csbp_cache_write, L.csbp_cache_read)]
    assert st[0] == st[1]
    return st[0]


@pytest.mark.parametrize("kw", [
    dict(pages=0), dict(pages=1 << 31), dict(page_size=0), dict(page_size=65537), dict(Hkv=0),
    dict(d=48), dict(d=0), dict(d=2048), dict(k=None), dict(v_scale=None), dict(v=PTR + 8)])
def test_bad_caches_are_refused(kw):
    assert both(cache(**kw), cache_rows()) == INVALID


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(rows=-1), dict(table_pages=-1), dict(table=None), dict(start=None),
    dict(start=PTR + 2), dict(count=PTR + 1), dict(tok=(128, 0)), dict(tok=(0, 260)),
    dict(tok=(-256, 0)), dict(bat=(0, 2040)), dict(bat=(2052, 0)), dict(tok=(1 << 60, 0)),
    dict(bat=(0, 1 << 60))])
def test_bad_cache_rows_are_refused(kw):
    assert both(cache(), cache_rows(**kw)) == INVALID


def test_cache_pointers_sizes_and_empty_calls():
    assert both(cache(), cache_rows(), k=None) == INVALID
    assert both(cache(), cache_rows(), v=PTR + 4) == INVALID
    assert both(cache(Hkv=65536, d=1024), cache_rows(batch=1 << 30)) == UNSUPPORTED
    assert both(cache(), cache_rows(batch=0)) == OK
    assert both(cache(), cache_rows(rows=0), k=None, v=None) == OK
    L = csbp.lib()
    assert L.csbp_cache_write(None, None, PTR, PTR, None) == INVALID


def prefix(**kw):
    p = csbp.PrefixProblem(2, 4, 100, 50, 8, 2, 64, 0, 0.125)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def prefix_inputs(tok=(0,) * 5, bat=(0,) * 5, **kw):
    i = csbp.PrefixInputs(PTR, PTR, PTR, PTR, PTR, PTR, tok, bat)
    for k, v in kw.items():
        setattr(i, k, v)
    return i


def attn(p, i, o=PTR, lse=PTR, ws=PTR, n=1 << 40):
    return csbp.lib().csbp_attn_prefix(ctypes.byref(p), ctypes.byref(i), o, lse, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), INVALID), (dict(queries=0), INVALID), (dict(prefix_len=-1), INVALID),
    (dict(own_max=-1), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID),
    (dict(causal=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(batch=1 << 30, queries=1 << 30), UNSUPPORTED),
    (dict(prefix_len=(1 << 31) - 1, Hkv=8), UNSUPPORTED)])
def test_bad_prefix_problems_are_refused(kw, want):
    p = prefix(**kw)
    assert csbp.prefix_workspace_bytes(p) == 0
    assert attn(p, prefix_inputs()) == want


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k_prefix=None), dict(v_own=None), dict(own_len=None),
    dict(own_len=PTR + 2), dict(q=PTR + 8), dict(v_prefix=PTR + 2),
    dict(tok=(500, 0, 0, 0, 0)), dict(tok=(0, 64, 0, 0, 0)), dict(tok=(0, 0, 0, 132, 0)),
    dict(bat=(1024, 0, 0, 0, 0)), dict(bat=(0, 0, 0, 0, 6404)), dict(tok=(0, -128, 0, 0, 0))])
def test_bad_prefix_inputs_are_refused(kw):
    assert attn(prefix(), prefix_inputs(**kw)) == INVALID


def test_prefix_outputs_and_workspace_are_checked():
    for kw in (dict(o=None), dict(lse=None), dict(ws=None), dict(o=PTR + 8), dict(lse=PTR + 4)):
        assert attn(prefix(), prefix_inputs(), **kw) == INVALID
    assert attn(prefix(), prefix_inputs(), n=255) == WORKSPACE
    assert csbp.prefix_workspace_bytes(prefix()) >= 256


def test_prefix_sizes_past_the_counters_are_unsupported():
    """q in 16-byte units within 32 bits, rows within 2^30, keys within 2^31."""
    big = prefix_inputs()
    big.stride_batch[0] = 1 << 33
    assert attn(prefix(batch=3), big) == UNSUPPORTED
    assert attn(prefix(batch=1 << 20, queries=1 << 10), prefix_inputs()) == UNSUPPORTED
    for kw in (dict(prefix_len=(1 << 31) - 1), dict(own_max=(1 << 31) - 100, batch=1)):
        p = prefix(Hq=1, Hkv=1, **kw)
        assert csbp.prefix_workspace_bytes(p) == 0
        assert attn(p, prefix_inputs()) == UNSUPPORTED
    assert csbp.prefix_workspace_bytes(prefix(Hq=1, Hkv=1, prefix_len=(1 << 31) - 200)) > 256


def verify(pr, p=PTR, q=PTR, token=PTR, u=PTR, r=PTR, length=None, acc=PTR, out=PTR):
    return csbp.lib().csbp_draft_verify(ctypes.byref(pr), p, q, token, u, r, length, acc, out,
                                        None)


def test_bad_verifications_are_refused():
    V = csbp.VerifyProblem
    assert verify(V(0, 4, 100)) == OK
    for bad in (V(-1, 4, 100), V(2, -1, 100), V(2, 4097, 100), V(2, 4, 0), V(2, 4, 100, 99),
                V(2, 4, 100, 0, 499), V(2, 4, 100, 0, 0, 64), V(2, 4, 100, 0, 0, 0, 399),
                V(2, 4, 100, -100), V(2, 4, 100, 1 << 60), V(2, 4, 100, 0, 1 << 60)):
        assert verify(bad) == INVALID
    good = V(2, 4, 100)
    for kw in (dict(p=None), dict(q=None), dict(token=None), dict(u=None), dict(r=None),
               dict(acc=None), dict(out=None), dict(p=PTR + 2), dict(u=PTR + 1),
               dict(length=PTR + 2), dict(out=PTR + 3)):
        assert verify(good, **kw) == INVALID
    assert csbp.lib().csbp_draft_verify(None, *([PTR] * 8), None) == INVALID


# ----------------------------------------------------------------- binding
def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_cache_binding_checks():
    c = csbp.QuantCache(6, 16, 2, 64, device="cpu")
    k = z(3, 5, 2, 64)
    args = dict(k=k, v=k.clone(), table=i32(3, 2), start=i32(3))
    for kw, msg in [
            (dict(k=k.float()), "k must be torch.bfloat16"),
            (dict(v=z(3, 5, 2, 32)), "v must have shape"),
            (dict(v=k.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous heads"),
            (dict(k=z(5, 3, 2, 64).transpose(0, 1)), "must not interleave"),
            (dict(k=k[:, :1].expand(3, 5, 2, 64)), "token stride"),
            (dict(k=k[:1].expand(3, 5, 2, 64)), "must not interleave"),
            (dict(table=i32(3)), "table must be"),
            (dict(table=i32(2, 2)), "table must have shape"),
            (dict(start=z(3, dtype=torch.int64)), "start must be torch.int32"),
            (dict(count=i32(2)), "count must have shape"),
            ({}, "k must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            c.write(**{**args, **kw})
    with pytest.raises(ValueError, match="needs `rows` or `out`"):
        c.read(i32(3, 2), i32(3))
    with pytest.raises(ValueError, match="CUDA tensor"):
        c.read(i32(3, 2), i32(3), rows=4)
    with pytest.raises(ValueError, match="k_scale must have shape"):
        csbp.QuantCache(6, 16, 2, 64, storage=(c.k, c.v, c.k, c.v_scale))
    with pytest.raises(ValueError, match="on one device"):
        csbp.QuantCache(6, 16, 2, 64, storage=(c.k, c.v.to("meta"), c.k_scale, c.v_scale))
    with pytest.raises(ValueError, match="multiple of 32"):
        csbp.QuantCache(6, 16, 2, 48, device="cpu")
    assert c.write(z(0, 5, 2, 64), z(0, 5, 2, 64), i32(0, 2), i32(0)) is None


def test_attention_binding_checks():
    a = csbp.PrefixAttention(2, 3, 10, 7, 4, 2, 64, device="cpu")
    args = dict(q=z(2, 3, 4, 64), k_prefix=z(10, 2, 64), v_prefix=z(10, 2, 64),
                k_own=z(2, 7, 2, 64), v_own=z(2, 7, 2, 64), own_len=i32(2))
    for kw, msg in [
            (dict(q=None), "q is required"),
            (dict(q=z(2, 3, 4, 64).float()), "q must be torch.bfloat16"),
            (dict(k_prefix=z(9, 2, 64)), "k_prefix must have shape"),
            (dict(v_prefix=z(2, 10, 64).transpose(0, 1)), "contiguous heads"),
            (dict(own_len=i32(2).long()), "own_len must be torch.int32"),
            (dict(k_own=z(1, 7, 2, 64).expand(2, 7, 2, 64)), "must not interleave"),
            ({}, "q must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            a.forward(**{**args, **kw})
    o, lse = a.alloc_outputs()
    with pytest.raises(ValueError, match="o must be contiguous"):
        a.forward(**args, out=(z(2, 4, 3, 64).transpose(1, 2), lse))
    with pytest.raises(ValueError, match="lse must have shape"):
        a.forward(**args, out=(o, lse.transpose(1, 2)))
    with pytest.raises(csbp.CsbpError):
        csbp.PrefixAttention(2, 3, 10, 7, 4, 3, 64, device="cpu")


def test_verify_binding_checks():
    f = torch.float32
    args = dict(p=z(2, 4, 9, dtype=f), q=z(2, 3, 9, dtype=f), token=i32(2, 3),
                u=z(2, 3, dtype=f), r=z(2, dtype=f))
    for kw, msg in [
            (dict(p=z(2, 9, dtype=f)), "p must be a"),
            (dict(p=z(2, 0, 9, dtype=f)), "p must be a"),
            (dict(p=args["p"].double()), "p must be torch.float32"),
            (dict(q=z(2, 4, 9, dtype=f)), "q must have shape"),
            (dict(q=z(2, 9, 3, dtype=f).transpose(1, 2)), "contiguous rows"),
            (dict(p=z(4, 2, 9, dtype=f).transpose(0, 1)), "must not interleave"),
            (dict(q=z(2, 1, 9, dtype=f).expand(2, 3, 9)), "must not overlap"),
            (dict(token=args["token"].long()), "token must be torch.int32"),
            (dict(length=i32(3)), "length must have shape"),
            (dict(out=(i32(2), i32(2, 3))), "tokens must have shape"),
            ({}, "must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            csbp.draft_verify(**{**args, **kw})
    acc, tok = csbp.draft_verify(z(0, 4, 9, dtype=f), z(0, 3, 9, dtype=f), i32(0, 3),
                                 z(0, 3, dtype=f), z(0, dtype=f))
    assert acc.shape == (0,) and tok.shape == (0, 4)
