"""The operators' C ABI without a GPU: symbols, struct layouts, constants, refusals of the
library and of the binding.  No call reaches a device."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from precision_optimizer_step_amd import opt8, opt8_products as ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "opt8_products.h")
A = 0x7F0000000000
STEP = 1 << 36
REACHED = (opt8.OPT8_OK, opt8.OPT8_E_HIP)     # every check passed (with no device the launch fails)


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
    assert names == ["opt8_fp8_matmul", "opt8_fp8_quantize", "opt8_gated_ffn_backward", "opt8_gated_ffn_forward",
                     "opt8_gated_ffn_workspace"]
    out = subprocess.run(["nm", "-D", "--defined-only", opt8.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (opt8_\w+)", out))
    assert set(names) <= exported


def test_structs_and_constants_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = [ops.opt8_fp8_quant, ops.opt8_fp8_product, ops.opt8_gated_ffn, ops.opt8_gated_ffn_grad]
    text = open(HEADER).read()
    consts = sorted(set(re.findall(r"\b(OPT8_[A-Z0-9_]+)\s*=", text)) | {"OPT8_FP8_BLOCK"})
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    for s in structs:
        lines.append(f'printf("{s.__name__} - %zu\\n", sizeof({s.__name__}));')
        lines += [f'printf("{s.__name__} {f} %zu\\n", offsetof({s.__name__}, {f}));' for f, _ in s._fields_]
    lines += [f'printf("const {c} %ld\\n", (long){c});' for c in consts]
    lines.append("return 0;}")
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    by_name = {s.__name__: s for s in structs}
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        kind, name, value = line.split()
        if kind == "const":
            assert getattr(ops, name) == int(value), name
        elif name == "-":
            assert ctypes.sizeof(by_name[kind]) == int(value)
        else:
            assert getattr(by_name[kind], name).offset == int(value), line


def quant(**over):
    d = dict(x=A, q=A + STEP, scale=A + 2 * STEP, qt=A + 3 * STEP, scale_t=A + 4 * STEP, rows=100, cols=200, ldx=200,
             ldq=208, ldt=112, x_type=ops.OPT8_TYPE_BF16, q_type=ops.OPT8_TYPE_E4M3, block=ops.OPT8_FP8_BLOCK_ROW)
    d.update(over)
    return ops.opt8_fp8_quantize(ops.opt8_fp8_quant(**d), stream=0, check=False)


def product(**over):
    d = dict(a=A, scale_a=A + STEP, b=A + 2 * STEP, scale_b=A + 3 * STEP, c=A + 4 * STEP, m=100, n=200, k=300, lda=304,
             ldb=304, ldc=200, a_type=ops.OPT8_TYPE_E4M3, b_type=ops.OPT8_TYPE_E4M3, c_type=ops.OPT8_TYPE_BF16,
             block_b=ops.OPT8_FP8_BLOCK_TILE)
    d.update(over)
    return ops.opt8_fp8_matmul(ops.opt8_fp8_product(**d), stream=0, check=False)


def ffn(**over):
    d = dict(x=A, w_gate=A + STEP, w_up=A + 2 * STEP, h=A + 3 * STEP, gate=A + 4 * STEP, up=A + 5 * STEP, rows=100, d=64,
             f=96, ldx=64, ldw=64, ldh=96, ldg=96, type=ops.OPT8_TYPE_BF16, act=ops.OPT8_ACT_SILU)
    d.update(over)
    return ops.opt8_gated_ffn_forward(ops.opt8_gated_ffn(**d), stream=0, check=False)


def grad(**over):
    names = ["dh", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up", "workspace"]
    d = {n: A + i * STEP for i, n in enumerate(names)}
    d.update(workspace_bytes=1 << 30, rows=100, d=64, f=96, ldx=64, ldw=64, lddh=96, ldg=96, lddx=64, lddw=64,
             type=ops.OPT8_TYPE_BF16, act=ops.OPT8_ACT_SILU)
    d.update(over)
    return ops.opt8_gated_ffn_backward(ops.opt8_gated_ffn_grad(**d), stream=0, check=False)


def expect(rc, status, fragment):
    assert rc == status, (rc, opt8.opt8_last_error())
    assert fragment in opt8.opt8_last_error(), opt8.opt8_last_error()


def test_valid_arguments_pass_every_check(L):
    assert quant() in REACHED and product() in REACHED and ffn() in REACHED and grad() in REACHED


NULL, SIZE, MODE, ALIGN, ALIAS = (opt8.OPT8_E_NULL, opt8.OPT8_E_SIZE, opt8.OPT8_E_MODE, opt8.OPT8_E_ALIGN,
                                  opt8.OPT8_E_ALIAS)


@pytest.mark.parametrize("name", ["opt8_fp8_quantize", "opt8_fp8_matmul", "opt8_gated_ffn_forward",
                                  "opt8_gated_ffn_backward"])
def test_null_struct(L, name):
    ops._functions()
    assert getattr(L, name)(None, None) == NULL


@pytest.mark.parametrize("over,status,fragment", [
    (dict(x=None), NULL, "x is NULL"), (dict(q=None), NULL, "q and scale"), (dict(scale_t=None), NULL, "qt and scale_t"),
    (dict(q=None, scale=None, qt=None, scale_t=None), NULL, "both NULL"),
    (dict(rows=-1), SIZE, "rows"), (dict(cols=(1 << 22) + 1), SIZE, "cols"), (dict(ldx=199), SIZE, "x: ld"),
    (dict(ldq=192), SIZE, "q: ld"), (dict(rows=1 << 22, cols=1 << 22, ldx=1 << 22, ldq=1 << 22, ldt=1 << 22), SIZE, "2^37"),
    (dict(x_type=ops.OPT8_TYPE_E4M3), MODE, "x is"), (dict(q_type=ops.OPT8_TYPE_BF16), MODE, "codes"),
    (dict(block=2), MODE, "block"), (dict(x=A + 1), ALIGN, "x"), (dict(q=A + STEP + 8), ALIGN, "q"),
    (dict(ldt=104), ALIGN, "qt"), (dict(scale=A + 2 * STEP + 2), ALIGN, "scale"),
    (dict(q=A + 16), ALIAS, "q overlaps x"), (dict(qt=A + STEP + 16), ALIAS, "overlaps"),
    (dict(scale_t=A + 2 * STEP + 4), ALIAS, "overlaps")])
def test_quantize_refusals(L, over, status, fragment):
    expect(quant(**over), status, fragment)


def test_empty_calls_are_no_ops(L):
    assert quant(rows=0, x=None) == opt8.OPT8_OK and quant(cols=0, x=None) == opt8.OPT8_OK
    assert product(m=0, c=None) == opt8.OPT8_OK and product(n=0, c=None) == opt8.OPT8_OK
    assert ffn(rows=0, x=None, h=None) == opt8.OPT8_OK
    assert product(k=0, a=None, b=None, scale_a=None, scale_b=None) in REACHED
    assert grad(rows=0, dh=None, x=None, gate=None, up=None, workspace=None, workspace_bytes=0) in REACHED


@pytest.mark.parametrize("over,status,fragment", [
    (dict(a=None), NULL, "NULL"), (dict(scale_b=None), NULL, "NULL"), (dict(c=None), NULL, "c is NULL"),
    (dict(m=-1), SIZE, "m must"), (dict(k=(1 << 22) + 1), SIZE, "k must"), (dict(lda=288), SIZE, "a: ld"),
    (dict(ldc=199), SIZE, "c: ld"), (dict(ldb=1 << 24), SIZE, "b: ld"), (dict(lda=300), ALIGN, "a"),
    (dict(b=A + 2 * STEP + 4), ALIGN, "b"), (dict(c=A + 4 * STEP + 1), ALIGN, "c"),
    (dict(a_type=ops.OPT8_TYPE_BF16), MODE, "a is"), (dict(b_type=ops.OPT8_TYPE_E5M2), MODE, "b is"),
    (dict(c_type=ops.OPT8_TYPE_E4M3), MODE, "c is"), (dict(c_type=ops.OPT8_TYPE_FP32), MODE, "c is"), (dict(block_b=-1), MODE, "block"),
    (dict(c=A + 128), ALIAS, "c overlaps a"), (dict(c=A + 3 * STEP), ALIAS, "scale_b")])
def test_product_refusals(L, over, status, fragment):
    expect(product(**over), status, fragment)


@pytest.mark.parametrize("over,status,fragment", [
    (dict(h=None), NULL, "h is NULL"), (dict(up=None), NULL, "go together"), (dict(d=0), SIZE, "d must"),
    (dict(f=(1 << 20) + 1), SIZE, "f must"), (dict(rows=-5), SIZE, "rows"), (dict(ldw=56), SIZE, "w_gate: ld"),
    (dict(ldx=68), ALIGN, "x"), (dict(w_up=A + 2 * STEP + 2), ALIGN, "w_up"), (dict(h=A + 3 * STEP + 1), ALIGN, "h"),
    (dict(type=ops.OPT8_TYPE_FP32), MODE, "bf16 or fp16"), (dict(act=3), MODE, "act"),
    (dict(h=A + STEP), ALIAS, "h overlaps w_gate"), (dict(gate=A + 3 * STEP + 32), ALIAS, "overlaps")])
def test_gated_forward_refusals(L, over, status, fragment):
    expect(ffn(**over), status, fragment)


@pytest.mark.parametrize("over,status,fragment", [
    (dict(dh=None), NULL, "NULL"), (dict(x=None), NULL, "NULL"), (dict(w_up=None), NULL, "NULL"),
    (dict(workspace=None), NULL, "NULL"), (dict(dw_up=None), NULL, "go together"),
    (dict(dx=None, dw_gate=None, dw_up=None), NULL, "both dw"), (dict(workspace_bytes=100), SIZE, "workspace"),
    (dict(lddh=88), SIZE, "dh: ld"), (dict(ldg=100), ALIGN, "gate"), (dict(workspace=A + 9 * STEP + 8), ALIGN, "workspace"),
    (dict(type=ops.OPT8_TYPE_E4M3), MODE, "bf16 or fp16"), (dict(act=-1), MODE, "act"),
    (dict(dx=A + STEP), ALIAS, "dx overlaps x"), (dict(dw_up=A + 7 * STEP), ALIAS, "overlaps"),
    (dict(workspace=A + 16), ALIAS, "overlaps")])
def test_gated_backward_refusals(L, over, status, fragment):
    expect(grad(**over), status, fragment)


def test_halves_of_one_matrix_do_not_overlap(L):
    """gate and up as the column halves of one [rows, 2f] matrix, and the cases next to it."""
    g = A + 4 * STEP
    assert ffn(gate=g, up=g + 2 * 96, ldg=192) in REACHED
    assert ffn(gate=g + 2 * 96, up=g, ldg=192) in REACHED
    expect(ffn(gate=g, up=g + 2 * 96 - 2, ldg=192), ALIAS, "overlaps")
    expect(ffn(gate=g, up=g + 2 * 97, ldg=192), ALIAS, "overlaps")
    expect(ffn(gate=g, up=g + 2 * 96, ldg=191), ALIAS, "overlaps")
    expect(ffn(gate=g, h=g + 2 * 96, ldg=192, ldh=384), ALIAS, "overlaps")
    assert ffn(rows=1, gate=g, up=g + 2 * 96, ldg=96) in REACHED
    assert quant(rows=100, q=A + STEP, ldq=416, qt=A + 3 * STEP, x=A + STEP + 208, x_type=ops.OPT8_TYPE_BF16, cols=100,
                 ldx=208) in REACHED      # x beside q in rows of 416 bytes


def test_one_sided_backward_needs_only_its_inputs(L):
    assert grad(dx=None, w_gate=None, w_up=None) in REACHED
    assert grad(dw_gate=None, dw_up=None, x=None) in REACHED


def test_workspace_is_a_pure_function_of_the_sizes(L):
    assert ops.opt8_gated_ffn_workspace(0, 64, 64) >= 0
    assert ops.opt8_gated_ffn_workspace(-1, 64, 64) == 0 and ops.opt8_gated_ffn_workspace(1, 64, 1 << 40) == 0
    assert ops.opt8_gated_ffn_workspace(100, 64, 100) >= 100 * 2 * 128 * 2
    assert ops.opt8_gated_ffn_workspace(100, 64, 100) == ops.opt8_gated_ffn_workspace(100, 64, 100)


def test_a_refusal_clears_with_the_next_call(L):
    expect(ffn(act=9), MODE, "act")
    assert quant(rows=0) == opt8.OPT8_OK and opt8.opt8_last_error() == ""


# ----------------------------------------------------------------------------- binding
E4 = torch.float8_e4m3fn


def codes(r, c, kind=E4, ld=None):
    return torch.zeros(r, ld or -(-c // 16) * 16, dtype=torch.uint8).view(kind)[:, :c]


def test_binding_checks_the_quantiser():
    x = torch.zeros(10, 200, dtype=torch.bfloat16)
    q, s = codes(10, 200), torch.zeros(2, 10)
    make = ops.make_fp8_quant
    with pytest.raises(ValueError, match="runs? on a GPU"):
        make(x, q, s)
    for args, match in [((x.double(), q, s), "x: dtype"), ((x[0], q, s), "expected a matrix"), ((x, q.float(), s), "q: dtype"),
                        ((x, codes(10, 199), s), "q: shape"), ((x, q, torch.zeros(10, 2)), "scale: shape"),
                        ((x, q, s.double()), "scale: dtype"), ((x, q, None), "go together"), ((x,), "both None"),
                        ((x, q, torch.zeros(2, 20)[:, ::2]), "contiguous"), ((x.t()[:10].t()[:, ::2], codes(10, 5), s), "adjacent|scale"),
                        ((x, q, s, codes(200, 10, torch.float8_e5m2), torch.zeros(1, 200)), "different types")]:
        with pytest.raises(ValueError, match=match):
            make(*args)
    with pytest.raises(ValueError, match="unknown block"):
        make(x, q, s, block=5)
    short = torch.zeros(9 * 208 + 200, dtype=torch.uint8).view(E4).as_strided((10, 200), (208, 1))
    with pytest.raises(ValueError, match="storage ends"):
        make(x, short, s)


def test_binding_checks_the_product():
    a, b = codes(10, 200), codes(300, 200)
    sa, sb, c = torch.zeros(2, 10), torch.zeros(2, 3), torch.zeros(10, 300, dtype=torch.bfloat16)
    make = ops.make_fp8_product
    with pytest.raises(ValueError, match="run on a GPU"):
        make(a, sa, b, sb, c)
    for args, match in [((a, sa, codes(300, 208), sb, c), "b: shape"), ((a, sa, codes(300, 200, torch.float8_e5m2), sb, c), "b: dtype"),
                        ((a, sa, b, torch.zeros(2, 300), c), "scale_b: shape"), ((a, sa, b, sb, c.t()), "c: shape"),
                        ((a, sa, b, sb, c.float()), "c: dtype"), ((a, sb, b, sb, c), "scale_a: shape")]:
        with pytest.raises(ValueError, match=match):
            make(*args)


def test_binding_checks_the_gated_block():
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)   # noqa: E731
    x, w, o = h(10, 64), h(96, 64), h(10, 96)
    with pytest.raises(ValueError, match="run on a GPU"):
        ops.make_gated_ffn(x, w, w, o)
    for args, match in [((x.float(), w, w, o), "x: dtype"), ((x, w.half(), w, o), "w_gate: dtype"),
                        ((x, w, h(95, 64), o), "w_up: shape"), ((x, w, w, h(10, 64)), "h: shape"),
                        ((x, w, w, o, o), "go together"), ((x, w, h(96, 128)[:, :64], o), "row distances")]:
        with pytest.raises(ValueError, match=match):
            ops.make_gated_ffn(*args)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    make = ops.make_gated_ffn_grad
    with pytest.raises(ValueError, match="run on a GPU"):
        make(o, x, w, w, o, o, x, w, w, ws)
    for args, match in [((h(10, 95), x, w, w, o, o, x, w, w, ws), "dh: shape"), ((o, x, w, w, o, h(10, 64), x, w, w, ws), "up: shape"),
                        ((o, x, w, w, o, o, w, w, w, ws), "dx: shape"), ((o, x, w, w, o, o, x, w, None, ws), "go together"),
                        ((o, x, w, w, o, o, None, None, None, ws), "are None"), ((o, x, w, w, o, o, x, w, w, ws.float()), "workspace")]:
        with pytest.raises(ValueError, match=match):
            make(*args)


def test_a_single_row_may_have_any_distance():
    """torch gives a one-row view any stride; the binding passes one that keeps 16-byte rows."""
    one = torch.zeros(1, 208, dtype=torch.uint8).view(E4)[:, :200]
    assert ops._matrix("a", one, (E4,), 1, 200, owned=True) == 208
    with pytest.raises(ValueError, match="storage ends"):
        ops._matrix("a", torch.zeros(1, 200, dtype=torch.uint8).view(E4), (E4,), 1, 200, owned=True)
