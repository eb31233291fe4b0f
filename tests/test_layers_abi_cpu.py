"""The C ABI of opt8_layers.h without a GPU: symbols, struct layouts, constants, refusals of the
library and of the binding, the table of a list.  No call reaches a device."""

import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

from precision_optimizer_step_amd import opt8, opt8_layers as ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "opt8_layers.h")
A = 0x7F0000000000
STEP = 1 << 38
REACHED = (opt8.OPT8_OK, opt8.OPT8_E_HIP)     # every check passed (with no device the launch fails)
NULL, SIZE, MODE, ALIGN, ALIAS, HPARAM = (opt8.OPT8_E_NULL, opt8.OPT8_E_SIZE, opt8.OPT8_E_MODE, opt8.OPT8_E_ALIGN,
                                          opt8.OPT8_E_ALIAS, opt8.OPT8_E_HPARAM)
BF, F32 = ops.OPT8_TYPE_BF16, ops.OPT8_TYPE_FP32


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(opt8.LIB_PATH):
        pytest.fail("libopt8.so is not built (run __graft_entry__.build())")
    if torch.cuda.is_available():
        pytest.skip("the addresses here are made up: checked where no GPU could follow them")
    return opt8.lib()


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(opt8_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(list(ops._CALLS) + ["opt8_embedding_workspace", "opt8_rms_norm_workspace", "opt8_grad_table",
                                               "opt8_grad_table_bytes"])
    out = subprocess.run(["nm", "-D", "--defined-only", opt8.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\bT (opt8_\w+)", out))


def test_structs_and_constants_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = sorted({*ops._CALLS.values(), ops.opt8_grad}, key=lambda s: s.__name__)
    text = open(HEADER).read()
    consts = sorted(set(re.findall(r"\b(OPT8_ID_[A-Z0-9]+)\s*=", text)) | set(re.findall(r"#define (OPT8_GRAD_\w+)", text)))
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    for s in structs:
        lines.append(f'printf("{s.__name__} - %zu\\n", sizeof({s.__name__}));')
        lines += [f'printf("{s.__name__} {f} %zu\\n", offsetof({s.__name__}, {f}));' for f, _ in s._fields_]
    lines += [f'printf("const {c} %ld\\n", (long){c});' for c in consts]
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    by_name = {s.__name__: s for s in structs}
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert len(out.splitlines()) > 60
    for line in out.splitlines():
        kind, name, value = line.split()
        if kind == "const":
            assert getattr(ops, name) == int(value), name
        elif name == "-":
            assert ctypes.sizeof(by_name[kind]) == int(value)
        else:
            assert getattr(by_name[kind], name).offset == int(value), line


def call(name, defaults, over):
    return getattr(ops, name)(ops._CALLS[name](**{**defaults, **over}), stream=0, check=False)


def spots(*names):
    return {n: A + i * STEP for i, n in enumerate(names)}


def embed(**over):
    return call("opt8_embedding_forward", dict(spots("ids", "table", "place_ids", "place_table", "y"), tokens=100, vocab=500,
                                               places=64, d=33, ldtable=33, ldplace=40, ldy=48, scale=1.0, type=BF, id_type=1), over)


def embed_grad(**over):
    return call("opt8_embedding_backward", dict(spots("ids", "dy", "dtable", "workspace"), workspace_bytes=1 << 24, tokens=100, vocab=500,
                                                d=33, lddy=33, lddtable=40, scale=1.0, type=BF, dtable_type=F32), over)


def norm(**over):
    return call("opt8_rms_norm_forward", dict(spots("x", "residual", "weight", "sum", "y", "q", "scale", "rstd"), rows=100, d=200,
                                              ldx=200, ldresidual=201, ldsum=202, ldy=203, ldq=208, eps=1e-6, type=BF,
                                              weight_type=F32, q_type=ops.OPT8_TYPE_E4M3), over)


def norm_grad(**over):
    return call("opt8_rms_norm_backward", dict(spots("dy", "x", "weight", "rstd", "dsum", "dx", "dweight", "workspace"),
                                               workspace_bytes=1 << 24, rows=100, d=200, lddy=200, ldx=201, lddsum=202, lddx=203,
                                               type=BF, weight_type=BF, dweight_type=F32), over)


def grads(name="opt8_grad_norm", **over):
    return call(name, dict(spots("table", "squares", "norm", "workspace"), table_bytes=240, workspace_bytes=16384, max_norm=1.0), over)


def clip(**over):
    return grads("opt8_grad_clip", **over)


def expect(rc, status, fragment):
    assert rc == status, (rc, opt8.opt8_last_error())
    assert fragment in opt8.opt8_last_error(), opt8.opt8_last_error()


def test_valid_arguments_pass_every_check(L):
    assert all(f() in REACHED for f in (embed, embed_grad, norm, norm_grad, grads, clip)), opt8.opt8_last_error()


@pytest.mark.parametrize("name", list(ops._CALLS))
def test_null_struct(L, name):
    ops._functions()
    assert getattr(L, name)(None, None) == NULL


@pytest.mark.parametrize("over,status,fragment", [
    (dict(ids=None), NULL, "ids"), (dict(table=None), NULL, "table"), (dict(y=None), NULL, "y is NULL"),
    (dict(place_ids=None), NULL, "go together"), (dict(place_table=None), NULL, "go together"),
    (dict(tokens=-1), SIZE, "tokens"), (dict(tokens=(1 << 22) + 1), SIZE, "tokens"), (dict(vocab=-1), SIZE, "vocab"),
    (dict(d=(1 << 20) + 1), SIZE, "d must"), (dict(places=-1), SIZE, "places"), (dict(ldtable=32), SIZE, "table: ld"),
    (dict(ldy=32), SIZE, "y: ld"), (dict(ldplace=32), SIZE, "place_table: ld"), (dict(ldy=(1 << 38) + 1), SIZE, "too large"),
    (dict(tokens=1 << 22, d=4097, ldy=5000, ldtable=5000, ldplace=5000), SIZE, "2^34"),
    (dict(type=ops.OPT8_TYPE_E4M3), MODE, "embedding"), (dict(id_type=2), MODE, "id type"),
    (dict(scale=float("nan")), HPARAM, "scale"), (dict(scale=float("inf")), HPARAM, "scale"),
    (dict(ids=A + 4), ALIGN, "ids"), (dict(y=A + 4 * STEP + 1), ALIGN, "y"),
    (dict(y=A + STEP + 64), ALIAS, "y overlaps table"), (dict(y=A + 64), ALIAS, "y overlaps ids")])
def test_embedding_refusals(L, over, status, fragment):
    expect(embed(**over), status, fragment)


@pytest.mark.parametrize("over,status,fragment", [
    (dict(ids=None), NULL, "ids"), (dict(dy=None), NULL, "dy"), (dict(dtable=None), NULL, "dtable"),
    (dict(workspace=None), NULL, "workspace"), (dict(workspace_bytes=100), SIZE, "workspace"), (dict(lddy=32), SIZE, "dy: ld"),
    (dict(lddtable=32), SIZE, "dtable: ld"), (dict(vocab=(1 << 22) + 1), SIZE, "vocab"),
    (dict(type=ops.OPT8_TYPE_E5M2), MODE, "dy"), (dict(dtable_type=ops.OPT8_TYPE_FP16), MODE, "dtable"), (dict(id_type=-1), MODE, "id type"),
    (dict(scale=float("-inf")), HPARAM, "scale"), (dict(workspace=A + 3 * STEP + 8), ALIGN, "workspace"),
    (dict(dtable=A + 2 * STEP + 2), ALIGN, "dtable"), (dict(dtable=A + STEP), ALIAS, "dtable overlaps dy"),
    (dict(workspace=A + 16), ALIAS, "overlaps")])
def test_embedding_gradient_refusals(L, over, status, fragment):
    expect(embed_grad(**over), status, fragment)


@pytest.mark.parametrize("over,status,fragment", [
    (dict(x=None), NULL, "x or weight"), (dict(weight=None), NULL, "x or weight"), (dict(scale=None), NULL, "q and scale"),
    (dict(q=None), NULL, "q and scale"), (dict(residual=None), NULL, "sum goes"), (dict(sum=None, y=None, q=None, scale=None, rstd=None), NULL, "no output"),
    (dict(d=0), SIZE, "d must"), (dict(rows=-1), SIZE, "rows"), (dict(ldsum=199), SIZE, "sum: ld"), (dict(ldq=192), SIZE, "q: ld"),
    (dict(ldq=216), ALIGN, "q"), (dict(q=A + 5 * STEP + 8), ALIGN, "q"), (dict(weight=A + 2 * STEP + 2), ALIGN, "weight"),
    (dict(type=ops.OPT8_TYPE_E4M3), MODE, "x:"), (dict(weight_type=ops.OPT8_TYPE_FP16), MODE, "weight"), (dict(q_type=BF), MODE, "codes"),
    (dict(eps=-1e-9), HPARAM, "eps"), (dict(eps=float("nan")), HPARAM, "eps"), (dict(eps=float("inf")), HPARAM, "eps"),
    (dict(y=A), ALIAS, "y overlaps x"), (dict(sum=A, ldsum=201), ALIAS, "sum overlaps x"), (dict(sum=A + STEP + 2, ldsum=201), ALIAS, "sum overlaps residual"),
    (dict(sum=A, ldsum=200, y=A + 64), ALIAS, "overlaps"), (dict(rstd=A + 6 * STEP), ALIAS, "overlaps")])
def test_norm_refusals(L, over, status, fragment):
    expect(norm(**over), status, fragment)


@pytest.mark.parametrize("over,status,fragment", [
    (dict(dy=None), NULL, "dy"), (dict(x=None), NULL, "x"), (dict(rstd=None), NULL, "rstd"), (dict(weight=None), NULL, "weight"),
    (dict(dx=None, dweight=None), NULL, "both NULL"), (dict(workspace=None), NULL, "workspace"), (dict(workspace_bytes=64), SIZE, "workspace"),
    (dict(lddsum=199), SIZE, "dsum: ld"), (dict(d=(1 << 20) + 1), SIZE, "d must"), (dict(dweight_type=ops.OPT8_TYPE_FP16), MODE, "dweight"),
    (dict(weight_type=ops.OPT8_TYPE_E4M3), MODE, "weight"), (dict(rstd=A + 3 * STEP + 2), ALIGN, "rstd"),
    (dict(dx=A + STEP), ALIAS, "dx overlaps x"), (dict(dx=A, lddx=201), ALIAS, "dx overlaps dy"), (dict(dweight=A + 2 * STEP), ALIAS, "dweight overlaps weight"),
    (dict(workspace=A + 5 * STEP), ALIAS, "overlaps")])
def test_norm_gradient_refusals(L, over, status, fragment):
    expect(norm_grad(**over), status, fragment)


@pytest.mark.parametrize("over,status,fragment", [
    (dict(table=None), NULL, "table"), (dict(squares=None), NULL, "squares"), (dict(table_bytes=0), SIZE, "24 bytes"),
    (dict(table_bytes=25), SIZE, "24 bytes"), (dict(table_bytes=((1 << 26) + 2) * 24), SIZE, "24 bytes"), (dict(table=A + 4), ALIGN, "table"),
    (dict(squares=A + STEP + 4), ALIGN, "squares"), (dict(norm=A + STEP), ALIAS, "overlaps"), (dict(norm=A + 8), ALIAS, "overlaps")])
@pytest.mark.parametrize("name", ["opt8_grad_norm", "opt8_grad_clip"])
def test_gradient_list_refusals(L, name, over, status, fragment):
    expect(grads(name, **over), status, fragment)


def test_refusals_of_one_of_the_list_s_calls(L):
    expect(grads(workspace=None), NULL, "workspace")
    expect(grads(workspace_bytes=16383), SIZE, "workspace")
    expect(grads(squares=A + 3 * STEP), ALIAS, "overlaps")
    for bad in (-1.0, float("nan"), float("inf")):
        expect(clip(max_norm=bad), HPARAM, "max_norm")
        assert grads(max_norm=bad) in REACHED
    assert clip(workspace=None, workspace_bytes=0) in REACHED and clip(norm=None) in REACHED and grads(table_bytes=24) in REACHED


def test_calls_that_take_an_operand_s_place(L):
    """The residual's sum on either operand, dx on dy or on the residual's gradient."""
    assert norm(sum=A, ldsum=200) in REACHED and norm(sum=A + STEP, ldsum=201) in REACHED
    assert norm_grad(dx=A, lddx=200) in REACHED and norm_grad(dx=A + 4 * STEP, lddx=202) in REACHED


def test_empty_calls_are_no_ops(L):
    none = dict(ids=None, table=None, y=None, place_ids=None, place_table=None)
    assert embed(tokens=0, **none) == opt8.OPT8_OK and embed(d=0, **none) == opt8.OPT8_OK
    assert embed(vocab=0, table=None) in REACHED and embed(places=0, place_table=None) in REACHED
    assert embed(place_ids=None, place_table=None, places=-7) in REACHED       # read with place_ids only
    assert embed_grad(vocab=0, dtable=None, workspace=None) == opt8.OPT8_OK
    assert embed_grad(tokens=0, accumulate=1, ids=None, dy=None, dtable=None, workspace=None) == opt8.OPT8_OK
    assert embed_grad(tokens=0, ids=None, dy=None) in REACHED
    assert norm(rows=0, x=None, weight=None, y=None) == opt8.OPT8_OK
    assert norm_grad(rows=0, dweight=None) == opt8.OPT8_OK
    assert norm_grad(rows=0, dy=None, x=None, rstd=None, weight=None, dx=None, workspace=None, workspace_bytes=0) in REACHED


def test_one_sided_gradients_need_only_their_inputs(L):
    assert norm_grad(dweight=None, workspace=None, workspace_bytes=0) in REACHED
    assert norm_grad(dx=None, weight=None, dsum=None) in REACHED


def test_workspaces_are_pure_functions_of_the_sizes(L):
    assert ops.opt8_embedding_workspace(-1, 5, 5) == 0 and ops.opt8_embedding_workspace(5, 5, (1 << 20) + 1) == 0
    assert ops.opt8_rms_norm_workspace(0, 64) == 0 and ops.opt8_rms_norm_workspace(5, 0) == 0
    for tokens, vocab, d in [(0, 1, 1), (1, 1, 1), (1000, 50257, 1600), (16384, 50257, 4096), (1 << 22, 1 << 22, 16), (77, 262145, 128)]:
        need = ops.opt8_embedding_workspace(tokens, vocab, d)
        assert need % 16 == 0 and need >= 8 * tokens + 4 * vocab + tokens * d // 4 and need <= 32 * tokens + 16 * vocab + tokens * d + 64 * d + (1 << 20)
    for rows, d in [(1, 1), (1, 1 << 20), (1 << 22, 64), (16384, 4096), (9, 16385)]:
        assert 4 * d <= ops.opt8_rms_norm_workspace(rows, d) <= 4096 * d + 16


def listed(entries):
    return struct.pack("=" + "QQqii" * len(entries), *[v for e in entries for v in e])


def table_of(L, entries):
    ops._functions()
    raw = listed(entries)
    size = L.opt8_grad_table_bytes(raw, len(entries))
    if size < 0:
        return size, None
    out = (ctypes.c_char * size)()
    return L.opt8_grad_table(raw, len(entries), out, size), bytes(out)


def test_the_table_of_a_list(L):
    """Pieces of 8192 values, those with a place of their own first; every value in one piece."""
    other = A + STEP
    rc, table = table_of(L, [(A, 0, 20000, BF, BF), (A + (1 << 20), other, 8193, F32, BF), (0, 0, 0, BF, 0), (A + (1 << 21), A + (1 << 21), 5, F32, F32)])
    assert rc == opt8.OPT8_OK
    pieces, own, reserved = struct.unpack_from("=qqq", table, 0)
    assert (pieces, own, reserved) == (6, 2, 0) and len(table) == 24 * 7
    got = [struct.unpack_from("=QQihh", table, 24 * (i + 1)) for i in range(pieces)]
    assert got == [(A + (1 << 20), other, 8192, F32, BF), (A + (1 << 20) + 4 * 8192, other + 2 * 8192, 1, F32, BF),
                   (A, A, 8192, BF, BF), (A + 2 * 8192, A + 2 * 8192, 8192, BF, BF), (A + 4 * 8192, A + 4 * 8192, 3616, BF, BF),
                   (A + (1 << 21), A + (1 << 21), 5, F32, F32)]


@pytest.mark.parametrize("entries,status,fragment", [
    ([(0, 0, 5, BF, BF)], NULL, "gradient 0 is NULL"), ([(A, 0, -1, BF, BF)], SIZE, "numel"), ([(A, 0, (1 << 37) + 1, BF, BF)], SIZE, "numel"),
    ([(A, 0, 5, 3, 3)], MODE, "gradient 0"), ([(A, A + 4096, 5, BF, 4)], MODE, "gradient 0"), ([(A, A, 5, BF, F32)], MODE, "another type"),
    ([(A + 1, 0, 5, BF, BF)], ALIGN, "gradient 0"), ([(A, A + 4098, 5, BF, F32)], ALIGN, "gradient 0"),
    ([(A, 0, 5, BF, BF), (A + 8, 0, 5, BF, BF)], ALIAS, "0 and 1"), ([(A, 0, 5, BF, BF), (A, 0, 5, BF, BF)], ALIAS, "0 and 1"),
    ([(A, A + 4, 5, F32, F32)], ALIAS, "overlap"), ([(A + 64, 0, 5, BF, BF), (A, A + 4096, 40, BF, BF)], ALIAS, "overlap"),
    ([(A + (i << 39), 0, 1 << 37, BF, BF) for i in range(5)], SIZE, "2^26")])
def test_refusals_of_a_list(L, entries, status, fragment):
    rc, _ = table_of(L, entries)
    expect(rc, status, fragment)


def test_list_sizes(L):
    ops._functions()
    assert L.opt8_grad_table_bytes(None, 0) == 24 and L.opt8_grad_table_bytes(None, 1) == NULL
    assert L.opt8_grad_table_bytes(None, -1) == SIZE and L.opt8_grad_table_bytes(None, (1 << 22) + 1) == SIZE
    one = listed([(A, 0, 5, BF, BF)])
    assert L.opt8_grad_table(one, 1, (ctypes.c_char * 48)(), 47) == SIZE and L.opt8_grad_table(one, 1, None, 48) == NULL


# ----------------------------------------------------------------------------- binding
def h(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_binding_checks_the_embedding():
    ids, table, y = torch.zeros(10, dtype=torch.int64), h(50, 33), h(10, 33)
    make = ops.make_embedding
    with pytest.raises(ValueError, match="run on a GPU"):
        make(ids, table, y)
    for args, kw, match in [((ids.short(), table, y), {}, "ids: dtype"), ((ids.view(2, 5), table, y), {}, "ids: shape"), ((ids.repeat(2)[::2], table, y), {}, "contiguous"),
                            ((ids, table.double(), y), {}, "table: dtype"), ((ids, table[0], y), {}, "expected a matrix"), ((ids, table, h(9, 33)), {}, "y: shape"),
                            ((ids, table, y.float()), {}, "y: dtype"), ((ids, table, h(33, 10).t()), {}, "adjacent"), ((ids, table, y), dict(place_ids=ids), "go together"),
                            ((ids, table, y), dict(place_ids=ids.int(), place_table=table), "place_ids: dtype"),
                            ((ids, table, y), dict(place_ids=ids, place_table=table.half()), "place_table: dtype")]:
        with pytest.raises(ValueError, match=match):
            make(*args, **kw)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    make = ops.make_embedding_grad
    with pytest.raises(ValueError, match="run on a GPU"):
        make(ids, y, table, ws)
    for args, match in [((ids, y, table.half(), ws), "dtable: dtype"), ((ids, h(10, 32), table, ws), "dy: shape"), ((ids, y.double(), table, ws), "dy: dtype"),
                        ((ids, y, table, ws.float()), "workspace"), ((ids, y, table[0], ws), "expected a matrix")]:
        with pytest.raises(ValueError, match=match):
            make(*args)


def test_binding_checks_the_norm():
    x, w = h(10, 200), h(200)
    q, s = torch.zeros(10, 208, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :200], torch.zeros(2, 10)
    make = ops.make_rms_norm
    with pytest.raises(ValueError, match="run on a GPU"):
        make(x, w, y=x, q=q, scale=s, rstd=torch.zeros(10), residual=x, sum=x)
    for kw, match in [(dict(weight=h(199)), "weight: shape"), (dict(weight=w.half()), "weight: dtype"), (dict(y=x.float()), "y: dtype"), (dict(q=q), "go together"),
                      (dict(sum=x), "goes with a residual"), (dict(residual=h(9, 200)), "residual: shape"), (dict(q=q, scale=torch.zeros(10, 2)), "scale: shape"),
                      (dict(q=q.float(), scale=s), "q: dtype"), (dict(rstd=torch.zeros(9)), "rstd: shape"), (dict(x=x[0]), "expected a matrix")]:
        with pytest.raises(ValueError, match=match):
            make(**{**dict(x=x, weight=w), **kw})
    r, ws = torch.zeros(10), torch.zeros(1 << 16, dtype=torch.uint8)
    good = dict(dy=x, x=x, weight=w, rstd=r, dx=x, dweight=w, workspace=ws)
    with pytest.raises(ValueError, match="run on a GPU"):
        ops.make_rms_norm_grad(**good)
    for kw, match in [(dict(dy=h(10, 199)), "dy: shape"), (dict(dx=None, dweight=None), "both None"), (dict(workspace=None), "needed for dweight"),
                      (dict(rstd=r.double()), "rstd: dtype"), (dict(dweight=w.half()), "dweight: dtype"), (dict(dsum=x.half()), "dsum: dtype"),
                      (dict(weight=w.double()), "weight: dtype"), (dict(workspace=ws[::2]), "workspace")]:
        with pytest.raises(ValueError, match=match):
            ops.make_rms_norm_grad(**{**good, **kw})


def test_binding_checks_the_list():
    g = [h(10), h(20)]
    with pytest.raises(ValueError, match="run on a GPU"):
        ops.opt8_grad_table(g)
    for args, match in [((g, [None]), "outs: 1 of them"), (([h(10), h(20).double()],), "gradient 1: dtype"), (([h(20)[::2]],), "contiguous"),
                        ((g, [None, h(21)]), "out 1: holds 21"), ((g, [h(10).int(), None]), "out 0: dtype")]:
        with pytest.raises(ValueError, match=match):
            ops.opt8_grad_table(*args)
    table, sq = torch.zeros(48, dtype=torch.uint8), torch.zeros(1, dtype=torch.float64)
    with pytest.raises(ValueError, match="run on a GPU"):
        ops.make_grads(table, sq)
    for args, match in [((table.float(), sq), "table"), ((table, sq.float()), "squares: dtype"), ((table, torch.zeros(2, dtype=torch.float64)), "squares: shape"),
                        ((table, sq, sq), "norm: dtype"), ((table, sq, None, table.float()), "workspace")]:
        with pytest.raises(ValueError, match=match):
            ops.make_grads(*args)


class Stream:
    def __init__(self, index, handle=64):
        self.device = torch.device("cuda", index)
        self.cuda_stream = handle


@pytest.mark.parametrize("name", list(ops._CALLS))
def test_a_call_on_another_device_is_refused(name, monkeypatch):
    queued = []
    monkeypatch.setattr(ops, "_fns", {name: lambda desc, stream: queued.append(stream) or 0})
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    desc = ops._on(1, ops._CALLS[name]())
    fn = getattr(ops, name)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for stream in (None, Stream(1), 64):
        with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
            fn(desc, stream=stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="stream.*cuda:0"):
        fn(desc, stream=Stream(0))
    assert queued == []
    assert fn(desc) == 0 and fn(desc, stream=Stream(1)) == 0 and fn(desc, stream=7) == 0
    assert queued == [101, 64, 7]
