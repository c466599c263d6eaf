"""What the attention, embedding and gradient calls refuse, on the host, before any
device work (CPU)."""

import ctypes
import os
import shutil
import subprocess

import pytest

import context_packed_sequence_amd as thd
from conftest import ROOT

# addresses far apart; nothing is read through them
Q, K, V, OUT, LSE, DOUT, DQ, DK, DV, STATUS, WS, CU, CUR, IDS, MASK, T = (i << 36 for i in range(1, 17))


@pytest.fixture(scope="module")
def lib():
    return thd.binding.library()


# ---- attention --------------------------------------------------------------------

SHAPE = dict(dtype=thd.THD_BF16, heads=4, kv_heads=2, dim=64, causal=1, window=0, cp_size=1, rank=0, n_slots=3,
             total_tokens=64, scale=0.125, cap=0.0, cu_seqlens_padded=CU, cu_seqlens=CUR)
BAD_SHAPES = [dict(dtype=thd.THD_FP32), dict(dtype=-1), dict(heads=3), dict(heads=0), dict(kv_heads=0), dict(dim=0),
              dict(dim=12), dict(dim=136), dict(causal=2), dict(window=-1), dict(cp_size=0), dict(rank=1),
              dict(rank=-1), dict(cp_size=thd.THD_MAX_CP + 1), dict(n_slots=-1), dict(total_tokens=-1),
              dict(total_tokens=2 ** 31), dict(total_tokens=65, cp_size=2), dict(scale=0.0), dict(scale=-1.0),
              dict(scale=1e-39), dict(total_tokens=2 ** 31 - 1, heads=16, kv_heads=16, dim=8),
              dict(scale=float("inf")), dict(scale=float("nan")), dict(cap=-1.0), dict(cap=float("inf")),
              dict(cap=float("nan")), dict(cap=1e-60), dict(scale=1e-30, cap=1e30), dict(scale=1e30, cap=1e-30)]


def _shape(**kw):
    return thd.thd_attention_shape(**{**SHAPE, **kw})


def _tensor(at, heads, dim=64, **kw):
    return thd.thd_heads(**{**dict(data=at, row_stride=heads * dim, head_stride=dim), **kw})


def _attention(lib, shape=None, ws_bytes=1 << 20, backward=False, null=(), **tensors):
    t = dict(q=_tensor(Q, 4), k=_tensor(K, 2), v=_tensor(V, 2), out=_tensor(OUT, 4), dout=_tensor(DOUT, 4),
             dq=_tensor(DQ, 4), dk=_tensor(DK, 2), dv=_tensor(DV, 2))
    t.update({n: x for n, x in tensors.items() if n in t})
    rest = {**dict(lse=LSE, status=STATUS, ws=WS), **{n: x for n, x in tensors.items() if n not in t}}
    ref = {n: None if n in null else ctypes.byref(x) for n, x in t.items()}
    shape = ctypes.byref(shape or _shape())
    if backward:
        return lib.thd_attention_backward(shape, ref["q"], ref["k"], ref["v"], ref["out"], rest["lse"], ref["dout"],
                                          ref["dq"], ref["dk"], ref["dv"], rest["status"], rest["ws"], ws_bytes, None)
    return lib.thd_attention(shape, ref["q"], ref["k"], ref["v"], ref["out"], rest["lse"], rest["status"], rest["ws"],
                             ws_bytes, None)


@pytest.mark.parametrize("bad", BAD_SHAPES)
def test_attention_shapes(lib, bad):
    for backward in (0, 1):
        assert lib.thd_attention_workspace_bytes(ctypes.byref(_shape(**bad)), backward) == -1
        assert _attention(lib, _shape(**bad), backward=bool(backward)) == thd.THD_ERR_ARG


def test_attention_arguments(lib):
    assert lib.thd_attention_workspace_bytes(None, 0) == -1
    assert lib.thd_attention_workspace_bytes(ctypes.byref(_shape()), 2) == -1
    need = [lib.thd_attention_workspace_bytes(ctypes.byref(_shape()), b) for b in (0, 1)]
    assert 0 < need[0] < need[1]
    for backward in (False, True):
        call = lambda **kw: _attention(lib, backward=backward, **kw)  # noqa: E731
        for n in ("q", "k", "v", "out", *(("dout", "dq", "dk", "dv") if backward else ())):
            heads = 2 if n in ("k", "v", "dk", "dv") else 4
            assert call(null=(n,)) == thd.THD_ERR_ARG
            for bad in (dict(at=None), dict(at=Q + 8), dict(row_stride=60), dict(row_stride=heads * 64 + 4),
                        dict(head_stride=68), dict(row_stride=-64), dict(head_stride=-64), dict(row_stride=2 ** 23)):
                at = bad.pop("at", Q)
                assert call(**{n: _tensor(at, heads, **bad)}) == thd.THD_ERR_ARG, (n, bad)
        assert call(lse=None) == thd.THD_ERR_ARG
        assert call(ws=None) == thd.THD_ERR_ARG
        assert call(ws=WS + 8) == thd.THD_ERR_ARG
        assert call(ws_bytes=need[backward] - 1) == thd.THD_ERR_ARG
        assert call(shape=_shape(cu_seqlens_padded=None)) == thd.THD_ERR_ARG
        # outputs whose own rows or heads overlap
        for n, heads in (("out", 4),) if not backward else (("dq", 4), ("dk", 2), ("dv", 2)):
            assert call(**{n: _tensor(OUT + (1 << 30), heads, row_stride=64)}) == thd.THD_ERR_ARG
            assert call(**{n: _tensor(OUT + (1 << 30), heads, head_stride=0)}) == thd.THD_ERR_ARG


def test_attention_overlaps(lib):
    alias = thd.THD_ERR_ALIAS
    assert _attention(lib, out=_tensor(Q, 4)) == alias
    assert _attention(lib, out=_tensor(K + 64, 4)) == alias
    assert _attention(lib, lse=V) == alias
    assert _attention(lib, status=OUT) == alias
    assert _attention(lib, ws=CU) == alias
    assert _attention(lib, backward=True, dq=_tensor(DOUT, 4)) == alias
    assert _attention(lib, backward=True, dk=_tensor(DV, 2)) == alias
    assert _attention(lib, backward=True, dk=_tensor(LSE, 2)) == alias
    # views of one buffer: rows of 8 heads, queries' 4, keys' 2, values' 2 -- unless they share elements
    def view(first, heads):
        return thd.thd_heads(data=DQ + 128 * first, row_stride=512, head_stride=64)
    assert _attention(lib, backward=True, dq=view(0, 4), dk=view(3, 2), dv=view(6, 2)) == alias
    assert _attention(lib, backward=True, dq=view(0, 4), dk=view(4, 2), dv=view(7, 2)) == alias   # wraps into the next row
    # the views themselves pass the check: a bad workspace is what is found then
    good = dict(dq=view(0, 4), dk=view(4, 2), dv=view(6, 2))
    assert _attention(lib, backward=True, status=DQ, **good) == alias
    assert _attention(lib, backward=True, ws_bytes=0, **good) == thd.THD_ERR_ARG


def test_attention_wrapper_checks():
    import torch
    x = torch.zeros((8, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for bad, match in ((dict(q=x.float()), "bfloat16 or float16"), (dict(k=x.half()), "k must be torch.bfloat16"),
                       (dict(q=x[0]), "rows, heads, dim"), (dict(v=x[:4]), "v must be"),
                       (dict(q=x[:, :1], k=x, v=x), "multiple of the key heads"), (dict(q=x[:4]), "rows, got 4"),
                       (dict(cp_size=2, rank=2), "is none"), (dict(window=-1), "window"),
                       (dict(q=x[:, :, :4], k=x[:, :, :4], v=x[:, :, :4]), "multiple of 8"),
                       (dict(k=x[:, :, ::2]), "elements"), (dict(cu=cu[:0]), "boundary"),
                       (dict(cu=cu.long()), "int32"), (dict(cu_seqlens=cu[:1]), "2 elements"), (dict(), "GPU")):
        a = {**dict(q=x, k=x, v=x, cu=cu), **bad}
        with pytest.raises(ValueError, match=match):
            thd.packed_attention(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("cu"), **a)
    with pytest.raises(ValueError, match="contiguous"):
        thd.packed_attention(x.transpose(1, 2).contiguous().transpose(1, 2), x, x, cu)
    with pytest.raises(ValueError, match="16 bytes"):
        thd.packed_attention(torch.zeros((8, 2, 68), dtype=torch.bfloat16)[:, :, :64], x, x, cu)


# ---- embedding ----------------------------------------------------------------------

@pytest.fixture
def lookup(lib):
    good = dict(ids=IDS, mask=MASK, rows=40, table=T, dtype=0, vocab=100, width=64, tstride=64, scale=1.0, out=OUT,
                ostride=64, status=STATUS, stream=None)

    def call(**kw):
        assert set(kw) <= set(good)
        return lib.thd_embedding(*{**good, **kw}.values())
    return call


@pytest.fixture
def backward(lib):
    good = dict(drows=DOUT, dtype=0, ids=IDS, mask=MASK, rows=40, vocab=100, width=64, rstride=64, scale=1.0,
                accumulate=0, dtable=T, out_dtype=0, tstride=64, status=STATUS, ws=WS,
                ws_bytes=lib.thd_embedding_workspace_bytes(40, 100, 64), stream=None)

    def call(**kw):
        assert set(kw) <= set(good)
        return lib.thd_embedding_backward(*{**good, **kw}.values())
    return call


BAD_TABLES = [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(rows=2 ** 31), dict(vocab=0),
              dict(vocab=thd.THD_MAX_VOCAB + 1), dict(width=0), dict(width=thd.THD_MAX_WIDTH + 1), dict(tstride=63),
              dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=1e39), dict(ids=None),
              dict(rows=2 ** 31 - 1, width=thd.THD_MAX_WIDTH, tstride=thd.THD_MAX_WIDTH)]


@pytest.mark.parametrize("bad", BAD_TABLES)
def test_embedding_sizes(lookup, backward, bad):
    assert lookup(**bad) == thd.THD_ERR_ARG
    assert backward(**bad) == thd.THD_ERR_ARG


def test_embedding_arguments(lib, lookup, backward):
    for bad in (dict(table=None), dict(table=T + 1), dict(out=None), dict(out=OUT + 1), dict(ostride=63)):
        assert lookup(**bad) == thd.THD_ERR_ARG, bad
    for bad in (dict(drows=None), dict(drows=DOUT + 1), dict(rstride=63), dict(dtable=None), dict(dtable=T + 1),
                dict(out_dtype=1), dict(out_dtype=3), dict(accumulate=2), dict(ws=None), dict(ws=WS + 8),
                dict(ws_bytes=0), dict(dtype=2, out_dtype=0)):
        assert backward(**bad) == thd.THD_ERR_ARG, bad
    for bad in (dict(out=T), dict(out=IDS + 64), dict(status=OUT), dict(status=T)):
        assert lookup(**bad) == thd.THD_ERR_ALIAS, bad
    for bad in (dict(dtable=DOUT), dict(dtable=IDS), dict(status=T), dict(ws=T), dict(ws=MASK - 16)):
        assert backward(**bad) == thd.THD_ERR_ALIAS, bad
    assert lib.thd_embedding_workspace_bytes(-1, 100, 64) == -1
    assert lib.thd_embedding_workspace_bytes(40, 100, 0) == -1


# ---- gradients -----------------------------------------------------------------------

def _clip(lib, grads, outs=None, elements=None, dtypes=None, out_dtypes=None, max_norm=1.0, scale=1.0, norm_in=None,
          norm=LSE, ws=WS, ws_bytes=1 << 20, status=STATUS, n=None):
    count = len(grads)
    at = (ctypes.c_void_p * max(count, 1))(*grads)
    to = (ctypes.c_void_p * max(count, 1))(*(grads if outs is None else outs))
    size = (ctypes.c_int64 * max(count, 1))(*(elements or [100] * count))
    kind = (ctypes.c_int32 * max(count, 1))(*(dtypes or [0] * count))
    out_kind = (ctypes.c_int32 * max(count, 1))(*(out_dtypes or dtypes or [0] * count))
    a = [ctypes.cast(x, ctypes.c_void_p) for x in (at, to, size, kind, out_kind)]
    return lib.thd_clip_gradients(*a, count if n is None else n, max_norm, scale, norm_in, norm, status, ws, ws_bytes,
                                  None)


def test_clipping_arguments(lib):
    bad = thd.THD_ERR_ARG
    assert _clip(lib, [T], n=-1) == bad
    assert _clip(lib, [T], n=thd.THD_MAX_TENSORS + 1) == bad
    assert _clip(lib, [T], elements=[-1]) == bad
    assert _clip(lib, [T], elements=[2 ** 60]) == bad
    assert _clip(lib, [T], dtypes=[3]) == bad
    assert _clip(lib, [None]) == bad
    assert _clip(lib, [T + 1]) == bad
    assert _clip(lib, [T], outs=[None]) == bad
    assert _clip(lib, [T], outs=[OUT + 1]) == bad
    assert _clip(lib, [T], outs=[OUT], dtypes=[2], out_dtypes=[0]) == bad
    assert _clip(lib, [T], outs=[OUT], out_dtypes=[1]) == bad
    for value in (0.0, -1.0, float("nan")):
        assert _clip(lib, [T], max_norm=value) == bad
    for value in (float("inf"), float("nan"), 1e39):
        assert _clip(lib, [T], scale=value) == bad
    assert _clip(lib, [T], ws=None) == bad
    assert _clip(lib, [T], ws=WS + 4) == bad
    assert _clip(lib, [T], ws_bytes=8) == bad
    assert lib.thd_gradients_workspace_bytes(-1) == -1
    assert lib.thd_gradients_workspace_bytes(thd.THD_MAX_TENSORS + 1) == -1
    assert lib.thd_gradient_norm(None, None, None, 1, 1.0, LSE, STATUS, WS, 1 << 20, None) == bad
    assert lib.thd_gradient_norm(None, None, None, 0, 1.0, None, STATUS, WS, 1 << 20, None) == bad


def test_clipping_overlaps(lib):
    alias = thd.THD_ERR_ALIAS
    assert _clip(lib, [T, T + 100]) == alias                        # in place, the tensors share elements
    assert _clip(lib, [T, T]) == alias                              # the same one twice
    assert _clip(lib, [T, Q], outs=[OUT, OUT + 100]) == alias       # outputs share elements
    assert _clip(lib, [T, Q], outs=[Q, T]) == alias                 # another's gradient
    assert _clip(lib, [T], outs=[T + 2]) == alias                   # its own, shifted
    assert _clip(lib, [T], outs=[T], out_dtypes=[2]) == alias       # its own, wider
    assert _clip(lib, [T], outs=[OUT], norm=T + 4) == alias
    assert _clip(lib, [T], outs=[OUT], ws=T - 8) == alias
    assert _clip(lib, [T], outs=[OUT], norm_in=LSE) == alias
    assert _clip(lib, [T], outs=[OUT], status=OUT + 8) == alias
    assert _clip(lib, [T, Q], outs=[OUT, K], norm=LSE, status=LSE) == alias


def test_params_wrapper_checks():
    import torch
    table, ids = torch.zeros((10, 8)), torch.zeros(4, dtype=torch.int64)
    for bad, match in ((dict(ids=ids.int()), "int64"), (dict(table=table.int()), "table must be"),
                       (dict(table=table[0]), "table must be"), (dict(table=table.t()), "contiguous"),
                       (dict(table=table.expand(2, 10, 8)), "table must be"),
                       (dict(mask=torch.zeros(3, dtype=torch.uint8)), "4 elements"), (dict(), "GPU")):
        a = {**dict(ids=ids, table=table), **bad}
        with pytest.raises(ValueError, match=match):
            thd.embedding(a.pop("ids"), a.pop("table"), **a)
    rows = torch.zeros((4, 8))
    for bad, match in ((dict(ids=ids[:3]), "4 elements"), (dict(drows=rows.double()), "drows must be"), (dict(), "GPU")):
        a = {**dict(drows=rows, ids=ids), **bad}
        with pytest.raises(ValueError, match=match):
            thd.embedding_backward(a.pop("drows"), a.pop("ids"), 10, **a)
    with pytest.raises(ValueError, match="GPU"):
        thd.clip_gradients([rows], 1.0)


@pytest.mark.parametrize("header", ["thd_attention.h", "thd_params.h"])
def test_headers_are_plain_c(tmp_path, header):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "x.c"
    src.write_text(f'#include "{header}"\nint main(void) {{ return THD_OK; }}\n')
    res = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", f"-I{os.path.join(ROOT, 'include')}",
                          str(src), "-c", "-o", str(tmp_path / "x.o")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in thd.thd_attention_shape._fields_]
    src = tmp_path / "x.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "thd_attention.h"\nint main(void) {\n'
                   + "".join(f'  printf("%d ", (int)offsetof(thd_attention_shape, {f}));\n' for f in fields)
                   + '  printf("%d %d", (int)sizeof(thd_attention_shape), (int)sizeof(thd_heads));\n  return 0;\n}\n')
    exe = str(tmp_path / "x")
    subprocess.run([cc, f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = [getattr(thd.thd_attention_shape, f).offset for f in fields]
    assert got == want + [ctypes.sizeof(thd.thd_attention_shape), ctypes.sizeof(thd.thd_heads)]
