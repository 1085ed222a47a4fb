"""The training operators on the CPU: the library loads, exports what
include/gq_train.h declares and refuses bad arguments before touching the
device; the plain implementations that the GPU tests compare with are pinned
here (the generator against the oracle, gradients against differences)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import allreduce_compatible_gradient_amd as gq
import oracle
import train_plain as plain
from allreduce_compatible_gradient_amd import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000     # a 16-byte aligned address, never dereferenced: rejected first
ODD = 0x10001
NUL = None


def copy8(codes=A, exps=A, rounding=0, seed=0):
    return train._CAct8(codes, exps, rounding, seed)


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "gq_train.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(gqt_[a-z_0-9]+)\s*\(", src)))
    assert len(names) >= 12
    for name in names:
        assert hasattr(train.lib(), name), name
        assert name in train.SIGNATURES, name
    assert sorted(train.SIGNATURES) == names


def test_header_serves_a_plain_c_caller(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    src = tmp_path / "caller.c"
    src.write_text(r"""
#include <stdio.h>
#include "gq_train.h"
int main(void)
{
    gqt_act8 a = {0, 0, GQT_ROUND_NEAREST, 0};
    if (gqt_act8_code_pitch(33) != 64 || gqt_act8_groups(33) != 2) return 1;
    if (gqt_act8_save(NULL, GQ_IN_F32, 4, 100, 100, &a, NULL) != GQ_ERR_NULL) return 2;
    if (gqt_last_error()[0] == '\0') return 3;
    if (gqt_act8_save(NULL, GQ_IN_F32, 0, 100, 100, &a, NULL) != GQ_OK) return 4;
    puts("ok");
    return 0;
}
""")
    lib_dir = os.path.join(ROOT, "allreduce_compatible_gradient_amd")
    exe = tmp_path / "caller"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I", os.path.join(ROOT, "include"), str(src), "-L", lib_dir, "-lgq_train",
                    f"-Wl,-rpath,{lib_dir}", "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)


def test_sizes():
    for d, g in ((1, 1), (32, 1), (33, 2), (4096, 128)):
        assert train.gqt_act8_groups(d) == g and train.gqt_act8_code_pitch(d) == 32 * g
    for d in (0, -1, 1 << 27, 1 << 31):
        assert train.gqt_act8_groups(d) == train.gqt_act8_code_pitch(d) == -1
    L = train.lib()
    ws = L.gqt_layer_norm_backward_workspace_bytes
    assert ws(0, 64) == 0 and ws(-1, 64) == -1 and ws(4, 0) == -1 and ws(1 << 32, 4) == -1
    assert ws(1, 64) == 8 * 64
    wg = L.gqt_weight_grad_workspace_bytes
    assert wg(0, 8, 8, 0) == 0 and wg(-1, 8, 8, 0) == -1 and wg(8, 0, 8, 0) == -1
    assert wg(8, 8, 8, 7) == -1 and wg(8, 1 << 20, 1 << 20, 0) == -1
    assert wg(1 << 20, 64, 64, 0) % (4 * (64 * 64 + 64)) == 0


# (arguments, expected status); every call is refused before any HIP call
@pytest.mark.parametrize("args,expect", [
    ((NUL, 0, 4, 100, 100, copy8(), NUL), 1),
    ((A, 0, 4, 100, 100, None, NUL), 1),
    ((A, 0, 4, 100, 100, copy8(codes=None), NUL), 1),
    ((A, 0, 4, 100, 100, copy8(exps=None), NUL), 1),
    ((A, 2, 4, 100, 100, copy8(), NUL), 2),
    ((A, 0, -1, 100, 100, copy8(), NUL), 2),
    ((A, 0, 4, 0, 100, copy8(), NUL), 2),
    ((A, 0, 4, 100, 99, copy8(), NUL), 2),          # rows overlap
    ((A, 0, 4, 100, -100, copy8(), NUL), 2),
    ((A, 0, 4, 100, 100, copy8(rounding=2), NUL), 2),
    ((A, 0, 1 << 32, 1, 1, copy8(), NUL), 2),
    ((A, 0, 1 << 20, 1 << 14, 1 << 14, copy8(), NUL), 3),  # 2^29 groups
    ((A, 0, 4, 100, 100, copy8(codes=A + 8), NUL), 6),
    ((ODD, 1, 4, 100, 100, copy8(), NUL), 6),
    ((A + 2, 0, 4, 100, 100, copy8(), NUL), 6),
])
def test_save_refuses(args, expect):
    assert train.lib().gqt_act8_save(*args) == expect
    assert train.lib().gqt_last_error().decode() != ""


@pytest.mark.parametrize("args,expect", [
    ((None, 4, 100, 0, A, NUL), 1),
    ((copy8(), 4, 100, 0, NUL, NUL), 1),
    ((copy8(codes=None), 4, 100, 0, A, NUL), 1),
    ((copy8(), 4, 100, 3, A, NUL), 2),
    ((copy8(), 4, 0, 0, A, NUL), 2),
    ((copy8(), 4, 100, 0, A + 2, NUL), 6),
])
def test_restore_refuses(args, expect):
    assert train.lib().gqt_act8_restore(*args) == expect


def _norm_args(x=A, dtype=0, rows=4, d=100, ldx=100, w=A, b=A, wdtype=0, eps=1e-5, y=A, mean=A,
               rstd=A, sx=None, sy=None):
    return x, dtype, rows, d, ldx, w, b, wdtype, eps, y, mean, rstd, sx, sy, NUL


@pytest.mark.parametrize("kw,expect", [
    ({"x": NUL}, 1), ({"y": NUL}, 1), ({"sx": copy8(codes=None)}, 1),
    ({"dtype": 9}, 2), ({"wdtype": 9}, 2), ({"d": 0}, 2), ({"rows": -1}, 2), ({"ldx": 99}, 2),
    ({"eps": -1e-5}, 2), ({"eps": math.nan}, 2), ({"eps": math.inf}, 2),
    ({"sy": copy8(rounding=5)}, 2), ({"rows": 1 << 30, "d": 64, "ldx": 64}, 3),
    ({"w": ODD}, 6), ({"b": A + 2}, 6), ({"mean": A + 2}, 6), ({"rstd": A + 2}, 6),
    ({"sx": copy8(codes=A + 4)}, 6), ({"y": A + 1}, 6),
])
def test_layer_norm_refuses(kw, expect):
    assert train.lib().gqt_layer_norm(*_norm_args(**kw)) == expect


def _back_args(dy=A, dtype=0, rows=4, d=100, lddy=100, x=A, ldx=100, x8=None, mean=A, rstd=A, w=A,
               wdtype=0, dx=A, dw=A, db=A, ws=A, nws=1 << 30):
    return dy, dtype, rows, d, lddy, x, ldx, x8, mean, rstd, w, wdtype, dx, dw, db, ws, nws, NUL


@pytest.mark.parametrize("kw,expect", [
    ({"dy": NUL}, 1), ({"x": NUL}, 1), ({"mean": NUL}, 1), ({"rstd": NUL}, 1), ({"dx": NUL}, 1),
    ({"ws": NUL}, 1), ({"x": NUL, "x8": copy8(exps=None)}, 1),
    ({"dtype": 2}, 2), ({"wdtype": 2}, 2), ({"lddy": 50}, 2), ({"ldx": 50}, 2), ({"d": 0}, 2),
    ({"nws": 8 * 100 - 1}, 5), ({"ws": A + 4}, 6), ({"dw": A + 2}, 6), ({"db": A + 2}, 6),
    ({"dx": A + 2}, 6), ({"x": NUL, "x8": copy8(codes=A + 1)}, 6),
])
def test_layer_norm_backward_refuses(kw, expect):
    assert train.lib().gqt_layer_norm_backward(*_back_args(**kw)) == expect


def test_gelu_refuses():
    L = train.lib()
    assert L.gqt_gelu(NUL, 0, 4, 100, 100, 0, A, None, None, NUL) == 1
    assert L.gqt_gelu(A, 0, 4, 100, 100, 0, NUL, None, None, NUL) == 1
    assert L.gqt_gelu(A, 0, 4, 100, 100, 2, A, None, None, NUL) == 2
    assert L.gqt_gelu(A, 0, 4, 100, 98, 0, A, None, None, NUL) == 2
    assert L.gqt_gelu(A, 0, 4, 100, 100, 0, A, copy8(rounding=-1), None, NUL) == 2
    assert L.gqt_gelu(A + 2, 0, 4, 100, 100, 0, A, None, None, NUL) == 6
    b = L.gqt_gelu_backward
    assert b(A, 0, 4, 100, 100, NUL, 0, None, 0, A, NUL) == 1
    assert b(NUL, 0, 4, 100, 100, A, 100, None, 0, A, NUL) == 1
    assert b(A, 0, 4, 100, 100, A, 100, None, 7, A, NUL) == 2
    assert b(A, 0, 4, 100, 100, A, 10, None, 0, A, NUL) == 2
    assert b(A, 0, 4, 100, 100, NUL, 0, copy8(codes=A + 2), 0, A, NUL) == 6
    assert b(A, 0, 4, 100, 100, A, 100, None, 0, A + 1, NUL) == 6


def _grad_args(dy=A, dtype=1, m=4096, n=100, lddy=100, x8=copy8(), k=60, dw=A, db=A, wdtype=0, ws=A,
               nws=1 << 40):
    return dy, dtype, m, n, lddy, x8, k, dw, db, wdtype, ws, nws, NUL


@pytest.mark.parametrize("kw,expect", [
    ({"dy": NUL}, 1), ({"dw": NUL}, 1), ({"x8": None}, 1), ({"x8": copy8(codes=None)}, 1),
    ({"ws": NUL}, 1), ({"dtype": 5}, 2), ({"wdtype": 5}, 2), ({"m": -1}, 2), ({"n": 0}, 2),
    ({"k": 0}, 2), ({"lddy": 99}, 2), ({"n": 1 << 20, "lddy": 1 << 20, "k": 1 << 20}, 2),
    ({"m": 1 << 28, "k": 64}, 3), ({"nws": 16}, 5), ({"dy": ODD}, 6), ({"dw": A + 2}, 6),
    ({"db": A + 2}, 6), ({"ws": A + 8}, 6), ({"x8": copy8(codes=A + 8)}, 6),
])
def test_weight_grad_refuses(kw, expect):
    assert train.lib().gqt_weight_grad(*_grad_args(**kw)) == expect


def test_nothing_to_do_enqueues_nothing():
    """No rows: accepted on a machine without a GPU, so no HIP call was made."""
    L = train.lib()
    empty = copy8(codes=None, exps=None)
    assert L.gqt_act8_save(NUL, 0, 0, 100, 100, empty, NUL) == 0
    assert L.gqt_act8_restore(empty, 0, 100, 0, NUL, NUL) == 0
    assert L.gqt_gelu(NUL, 0, 0, 100, 100, 0, NUL, empty, None, NUL) == 0
    assert L.gqt_gelu_backward(NUL, 0, 0, 100, 100, NUL, 0, empty, 0, NUL, NUL) == 0
    assert L.gqt_layer_norm(*_norm_args(x=NUL, rows=0, y=NUL, mean=NUL, rstd=NUL)) == 0
    assert L.gqt_layer_norm_backward(*_back_args(dy=NUL, x=NUL, x8=empty, rows=0, mean=NUL,
                                                 rstd=NUL, dx=NUL, dw=NUL, db=NUL, ws=NUL,
                                                 nws=0)) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    a = train.Act8.empty(2, 8, "cpu")
    v = torch.zeros(2)
    for call in (lambda: train.gqt_act8_save(x), lambda: train.gqt_act8_restore(a),
                 lambda: train.gqt_layer_norm(x), lambda: train.gqt_gelu(x),
                 lambda: train.gqt_layer_norm_backward(x, x, v, v),
                 lambda: train.gqt_gelu_backward(x, x), lambda: train.gqt_weight_grad(x, a)):
        with pytest.raises(ValueError):
            call()
    assert a.codes.shape == (2, 32) and a.exps.shape == (2, 1) and a.shape == (2, 8)


# ---------------------------------------------------------------------------
# the plain implementations

def test_uniforms_are_the_compressors():
    seed = 0x123456789ABCDEF
    u = plain.uniforms(3, 19, seed)
    for r in range(3):
        for j in range(19):
            assert u[r, j] == oracle.uniform32(seed, r, j)


def test_saved_values():
    x = np.array([[1.0, -0.5, 127.0, 0.0], [127.5, 0.25, -1e-3, 3.0]])
    codes, exps = plain.save(x)
    assert exps.tolist() == [[127], [128]]
    assert codes[0, :4].tolist() == [1, 0, 127, 0] and not codes[:, 4:].any()  # -0.5 to even
    assert codes[1, :4].tolist() == [64, 0, 0, 2]
    f32 = np.float32
    top = np.full((1, 40), np.finfo(f32).max)
    codes, exps = plain.save(top)
    assert exps.tolist() == [[249, 249]] and (codes[0, :40] == 63).all()
    codes, exps = plain.save(np.array([[np.inf, 1.0]]))
    assert exps.tolist() == [[255]] and np.isnan(plain.restore(codes, exps, 2)).all()
    codes, exps = plain.save(np.zeros((1, 3)))
    assert exps.tolist() == [[1]] and not codes.any()


def test_random_rounding_is_unbiased():
    """The mean over 4096 draws of one value lies within 5 deviations."""
    rng = np.random.default_rng(1)
    v = rng.uniform(-1, 1, 64)
    x = np.tile(v, (4096 // 2, 1))
    r = plain.restore(*plain.save(x, seed=77), 64)
    step = np.exp2(plain.save(x[:1])[1].astype(float) - 127).repeat(32)
    p = np.abs(v / step) % 1
    dev = step * np.sqrt(p * (1 - p) / x.shape[0])
    assert (np.abs(r.mean(axis=0) - v) <= 5 * dev + 1e-9).all()
    assert (np.abs(r - x) < step).all()


@pytest.mark.parametrize("form", ["none", "tanh"])
def test_gelu_slope_against_differences(form):
    h = np.linspace(-8, 8, 401)
    e = 1e-5
    diff = (plain.gelu(h + e, form) - plain.gelu(h - e, form)) / (2 * e)
    # truncation e^2/6 |y'''| < 1e-10, cancellation 2^-53 8 / e < 1e-10
    assert np.abs(diff - plain.gelu_slope(h, form)).max() < 2e-10 * 5


def test_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((5, 37)), rng.standard_normal((5, 37))
    w, b = rng.standard_normal(37), rng.standard_normal(37)
    mean, rstd = plain.norm_stats(x, 1e-5)
    dx, dw, db = plain.layer_norm_backward(dy, x, mean, rstd, w)
    e = 1e-6
    for grad, var in ((dx, x), (dw, w), (db, b)):
        v = rng.standard_normal(var.shape)
        args = [x, w, b]
        at = [i for i, a in enumerate(args) if a is var][0]

        def loss(t):
            a = list(args)
            a[at] = var + t * v
            return (dy * plain.layer_norm(*a, 1e-5)).sum()
        assert abs((loss(e) - loss(-e)) / (2 * e) - (grad * v).sum()) < 1e-6


def test_library_status_names_are_shared():
    assert gq.STATUS[5] == "GQ_ERR_WORKSPACE"
    assert isinstance(ctypes.c_char_p(train.lib().gqt_last_error()).value, bytes)
