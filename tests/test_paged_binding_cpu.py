"""More of what the paged cache's calls refuse on the host, each refusal told by its own message or
status; on the CPU, where nothing is launched."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest
import torch

from test_paged_cpu import POOL, TABLE, lib


@pytest.mark.parametrize("want,pos", [
    (1, 1024), (1, 1024 - 12), (1, 1024 + 12),          # delta: 4 rows, from 1024 on
    (1, 2048), (1, 2048 + 12), (1, 4096), (1, 4096 + 396),      # seq_lens; ref, of 100 pages
])
def test_resize_pos_of_its_own(want, pos):
    """pos is written while delta, seq_lens and ref are still read: it cannot be one of them."""
    G = lib()
    a = dict(delta=1024, lens=2048, S=4, **TABLE, ref=4096, **POOL, H=8, d=128, pos=pos, status=None,
             ws=8192, wsb=16, stream=None)
    assert G._lib.gret_paged_resize(*a.values()) == want


KP = torch.zeros((4, 16, 2, 64))
Q, LENS = torch.zeros((3, 6, 64)), torch.zeros(3, dtype=torch.int32)
PT, REF = torch.zeros((3, 5), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
KV = Q[:, :2]


def decode(q=Q, lens=LENS, table=PT, kp=KP, vp=KP, **kw):
    return lib().gret_paged_attention_decode(q, lens, table, kp, vp, **kw)


def append(k=KV, v=KV, pos=LENS, table=PT, kp=KP, vp=KP, **kw):
    return lib().gret_paged_append(k, v, pos, table, kp, vp, **kw)


def resize(delta=LENS, lens=LENS, table=PT, ref=REF, kp=KP, vp=KP, **kw):
    return lib().gret_paged_resize(delta, lens, table, ref, kp, vp, **kw)


def fork(src=LENS, dst=LENS, lens=LENS, table=PT, ref=REF, page=16):
    return lib().gret_paged_fork(src, dst, lens, table, ref, page)


def compact(lens=LENS, table=PT, ref=REF, kp=KP, vp=KP, **kw):
    return lib().gret_paged_compact(lens, table, ref, kp, vp, **kw)


OTHER_STRIDES = KP.transpose(1, 2).contiguous().transpose(1, 2)
LAST_APART = torch.zeros((4, 16, 2, 128))[..., ::2]
Q_RULE = r"q must be contiguous \[B, Hq, d\] with the pool's d and dtype"
TABLE_RULE = r"page_table must be int32 \[3, max_pages\] with contiguous rows"
KV_RULE = r"k and v must be \[T, Hkv, d\] with the pool's heads and dtype"


@pytest.mark.parametrize("error,message,call", [
    # the checks come before the one that every tensor is on a GPU: what passes them all gets there
    (ValueError, "must be on a GPU", lambda: decode()),
    (ValueError, "must be on a GPU", lambda: append()),
    (ValueError, "must be on a GPU", lambda: resize()),
    (ValueError, "must be on a GPU", lambda: fork()),
    (ValueError, "must be on a GPU", lambda: compact()),
    (ValueError, "must be on a GPU", lambda: decode(table=PT[:, :1])),
    (ValueError, "must be on a GPU", lambda: decode(table=torch.zeros((3, 9), dtype=torch.int32)[:, 2:7])),
    (ValueError, Q_RULE, lambda: decode(q=Q.bfloat16())),
    (ValueError, Q_RULE, lambda: decode(q=Q[..., :32].contiguous())),
    (ValueError, Q_RULE, lambda: decode(q=Q[0])),
    (ValueError, Q_RULE, lambda: decode(q=Q.transpose(0, 1))),
    (ValueError, TABLE_RULE, lambda: decode(table=PT[:2])),
    (ValueError, TABLE_RULE, lambda: decode(table=PT.long())),
    (ValueError, TABLE_RULE, lambda: decode(table=PT[0])),
    (ValueError, TABLE_RULE, lambda: decode(table=torch.zeros((5, 3), dtype=torch.int32).t())),
    (ValueError, TABLE_RULE, lambda: append(table=PT.long())),
    (ValueError, TABLE_RULE, lambda: resize(table=PT[:2])),
    (ValueError, TABLE_RULE, lambda: fork(table=PT.float())),
    (ValueError, TABLE_RULE, lambda: compact(table=torch.zeros((4, 5), dtype=torch.int32))),
] + [
    (error, message, lambda f=f, kp=kp, vp=vp: f(kp=kp, vp=vp))
    for f in (decode, append, resize, compact)
    for error, message, kp, vp in [
        (ValueError, "must be 4-D and alike", KP, KP[:2]),
        (ValueError, "must be 4-D and alike", KP[0], KP[0]),
        (ValueError, "must be 4-D and alike", KP, KP.bfloat16()),
        (ValueError, "must share strides", KP, OTHER_STRIDES),
        (ValueError, "the last one 1", LAST_APART, LAST_APART),
        (TypeError, "must be bfloat16 or float32, got Half", KP.half(), KP.half()),
    ]
] + [
    (ValueError, KV_RULE, lambda: append(k=Q, v=Q)),                       # heads
    (ValueError, KV_RULE, lambda: append(k=KV[..., :32], v=KV[..., :32])),
    (ValueError, KV_RULE, lambda: append(v=KV[:2])),
    (ValueError, KV_RULE, lambda: append(k=KV.bfloat16(), v=KV.bfloat16())),
    (ValueError, KV_RULE, lambda: append(v=KV.bfloat16())),
    (ValueError, KV_RULE, lambda: append(k=KV[0], v=KV[0])),
    (ValueError, "last dimension must be contiguous",
     lambda: append(k=torch.zeros((3, 2, 128))[..., ::2])),
    (ValueError, "last dimension must be contiguous",
     lambda: append(v=torch.zeros((3, 2, 128))[..., ::2])),
    (ValueError, "window is out of range", lambda: decode(window=2 ** 31)),
    (ValueError, "page_size is out of range", lambda: fork(page=-2 ** 31 - 1)),
    (TypeError, "q must be a tensor", lambda: decode(q=[1.0])),
    (TypeError, "status must be a tensor", lambda: decode(status=0)),
    (TypeError, "lse must be a tensor", lambda: decode(lse=False)),
    (TypeError, "cu_seqlens must be a tensor", lambda: append(cu_seqlens=[0, 3])),
    (TypeError, "pos must be a tensor", lambda: resize(pos=3)),
    (TypeError, "n_live must be a tensor", lambda: compact(n_live=3)),
])
def test_binding_tells_what_is_wrong(error, message, call):
    with pytest.raises(error, match=message):
        call()


def copied_package(tmp_path, *names):
    import gated_retention_linear_b200 as G
    src = os.path.dirname(G.__file__)
    dst = tmp_path / os.path.basename(src)
    dst.mkdir()
    for name in names:
        shutil.copy(os.path.join(src, name), dst / name)
    return dst


@pytest.mark.parametrize("what", ["missing", "not loadable"])
def test_import_without_the_binding(tmp_path, what):
    """_paged.so serves the paged cache's calls alone: without it, or with one that does not fit the
    installed torch, the library imports, everything else works, and those calls say what is wrong."""
    dst = copied_package(tmp_path, "__init__.py", "libgret.so")
    if what != "missing":
        (dst / "_paged.so").write_bytes(b"not a library")
    code = """
import torch
import gated_retention_linear_b200 as G
assert G.__file__.startswith(%r)
assert G.gret_prefill_workspace_size(torch.bfloat16, 100, 1, 2, 128, 128) >= 0
assert G.gret_paged_attention_workspace_size(torch.bfloat16, 24, 8, 128) > 0
x = torch.zeros(3, dtype=torch.int32)
pool = torch.zeros((4, 16, 2, 64))
for call in (lambda: G.gret_paged_attention_decode(pool[0, :3], x, x[None], pool, pool),
             lambda: G.gret_paged_append(pool[0], pool[0], x, x[None], pool, pool),
             lambda: G.gret_paged_resize(x, x, x[None], x, pool, pool),
             lambda: G.gret_paged_fork(x, x, x, x[None], x, 16),
             lambda: G.gret_paged_compact(x, x[None], x, pool, pool)):
    try:
        call()
    except ImportError as e:
        assert "_paged.so" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("no ImportError")
""" % str(tmp_path)
    subprocess.run([sys.executable, "-c", code], cwd=tmp_path, check=True,
                   env={**os.environ, "PYTHONPATH": str(tmp_path)})


def test_binding_is_rebuilt_for_another_torch_or_python(tmp_path, monkeypatch):
    """_paged.so uses torch's C++ interface and Python's: build() makes it anew when either is not the
    one it was made for, when it or what it is made of has changed, and not otherwise."""
    import gated_retention_linear_b200 as G
    spec = importlib.util.spec_from_file_location(
        "build_under_test", os.path.join(os.path.dirname(G.__file__), "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    so = tmp_path / "_paged.so"
    monkeypatch.setattr(b, "BINDING", str(so))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()

    monkeypatch.setattr(b.subprocess, "run", run)

    def builds(force=False):
        n = len(runs)
        b._build_binding(force)
        assert so.exists()
        return len(runs) - n

    assert builds() == 1 and builds() == 0
    with monkeypatch.context() as m:
        m.setattr(b.importlib.metadata, "version", lambda name: "2.12.0")
        assert builds() == 1 and builds() == 0
    assert builds() == 1 and builds() == 0
    config = b.sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(b.sysconfig, "get_config_var",
                  lambda name: "cpython-313" if name == "SOABI" else config(name))
        assert builds() == 1 and builds() == 0
    assert builds() == 1 and builds() == 0
    os.utime(so, (0, 0))                               # older than its source
    assert builds() == 1 and builds() == 0
    so.unlink()
    assert builds() == 1 and builds(force=True) == 1 and builds() == 0
