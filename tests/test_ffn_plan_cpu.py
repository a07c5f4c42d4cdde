"""Which kernels the GPU tests of the feed-forward block reach, checked on the
CPU: csrc/ffn_plan.hpp, the rules that pick them, is compiled here
(tests/kernel_model/ffn_plan.cpp), and every kernel, tile and form of joining
that some size takes has to be taken by a size that a parity test runs."""
import ctypes
import itertools
import math
import os
import random
import subprocess

import pytest

import test_gpu_ffn
import test_gpu_ffn_few
import test_gpu_ffn_tiles

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kernel_model", "ffn_plan.cpp")
HIDDEN = ("128 x 64", "128 x 128", "hidden8")
ROWS = ("128 x 64", "128 x 128", "128 x 192")
DW = ("128 x 128", "256 x 256")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("plan") / "libplan.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", SRC, "-o", lib])
    L = ctypes.CDLL(lib)
    L.model_plan.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]
    L.model_plan.restype = None
    f, b = (ctypes.c_int32 * 5)(), (ctypes.c_int32 * 7)()

    def kernels(T, F, numbers=False):
        """What a forward and a backward of T positions and F hidden units launch."""
        L.model_plan(T, F, f, b)
        if numbers:
            return list(f), list(b)
        few, wide, hidden, rows, parts = f
        if few:
            out = {("few", 1 if T <= 16 else 2 if T <= 32 else 4, "two bf16" if wide else "one bf16")}
        else:
            out = {("H", HIDDEN[hidden]), ("Y", ROWS[rows], "parts" if parts > 1 else "whole")}
        wide, merged, hidden, rows, parts, dw, dw_parts = b
        out.add(("hidden gradients", HIDDEN[hidden], "two bf16" if wide else "one bf16"))
        how = "parts" if parts > 1 else "whole"
        if merged:
            out.add(("dX with the weights' gradients", ROWS[rows], how, "two bf16" if wide else "one bf16"))
        else:
            out |= {("dX", ROWS[rows], how), ("weights' gradients", DW[dw], "parts" if dw_parts > 1 else "whole")}
        return out

    return kernels


def test_workspace_holds_what_its_calls_take(plan):
    # bytes of a config's workspace, and of what a call of up to its positions keeps there
    from sparse_hashed_gram_amd import ffn
    up = lambda n: -(-n // 256) * 256   # noqa: E731
    for F in (8, 128, 1000, 2048, 8192, 8200, 65536):
        Fp = -(-F // 64) * 64
        for T in (1, 2, 40, 64, 65, 128, 300, 512, 513, 4096, 49152):
            cfg = ffn.config(F, T)
            rows = min(16 * 768 * 4 * T, 2 * 256 * 128 * 128 * 4)
            parts = min(8, -(-T // 64))
            few = min(T, 64, 8192 // F) * (16 * 768 * 4 + 6 * Fp)
            part = max(rows, parts * 3 * Fp * 768 * 4 if parts > 1 else 0, few)
            assert ffn.workspace_bytes(cfg, False) == up(2 * T * Fp) + up(rows)
            assert ffn.workspace_bytes(cfg) == up(6 * T * Fp) + up(1536 * T) + up(part)
    assert ffn.workspace_bytes(ffn.config(8192, 1)) < 200_000   # one position needs no parts of the weights' gradients
    r = random.Random(4)
    spread = lambda hi: int(math.exp(r.uniform(0, math.log(hi + 1))))   # noqa: E731
    for _ in range(4000):
        T, F = spread(60000), 8 * spread(8192)
        Fp = -(-F // 64) * 64
        for most in (T, T + 1 + spread(4000)):
            cfg = ffn.config(F, most)
            fwd = ffn.workspace_bytes(cfg, False) - 2 * most * Fp
            bwd = ffn.workspace_bytes(cfg) - 6 * most * Fp - 1536 * most
            (few, wide, _, _, parts), (_, merged, _, _, rows, _, dw) = plan(T, F, numbers=True)
            assert fwd >= (2 * T * Fp if wide else 0 if few or parts == 1 else parts * T * 768 * 4)
            assert bwd >= (16 * T * 768 * 4 + 6 * T * Fp if wide else rows * T * 768 * 4 if rows > 1 else 0)
            assert rows <= 16
            assert dw == 1 or (not merged and bwd >= dw * 3 * Fp * 768 * 4)


def _sizes(module):
    """(T, F) of every case that the module's parametrised tests run."""
    for name, f in vars(module).items():
        marks = [m for m in getattr(f, "pytestmark", []) if m.name == "parametrize"] if name.startswith("test_") else []
        if not marks:
            continue
        for values in itertools.product(*(m.args[1] for m in marks)):
            case = {}
            for m, v in zip(marks, values):
                names = [n.strip() for n in m.args[0].split(",")]
                case.update(zip(names, v if len(names) > 1 else [v]))
            if "T" in case and "F" in case:
                yield case["T"], case["F"]


def test_every_kernel_is_reached(plan):
    r = random.Random(3)
    spread = lambda hi: int(math.exp(r.uniform(0, math.log(hi + 1))))   # noqa: E731
    taken = set()
    for _ in range(40000):
        taken |= plan(spread(60000), 8 * spread(8192))
    # sizes of a narrow range that the draws above may pass over
    for T in range(1, 1500, 7):
        for F in range(2800, 3060, 20):
            taken |= plan(T, F // 8 * 8)
    tested = set()
    for case in itertools.chain(_sizes(test_gpu_ffn), _sizes(test_gpu_ffn_few), _sizes(test_gpu_ffn_tiles)):
        tested |= plan(*case)
    assert len(taken) > 25
    assert not taken - tested, f"no parity test reaches {sorted(taken - tested)}"


def test_real_values_reach_the_kernels_of_many_positions(plan):
    many = {("H", "hidden8"), ("Y", "128 x 192", "whole"), ("hidden gradients", "hidden8", "one bf16"),
            ("dX", "128 x 192", "whole"), ("weights' gradients", "256 x 256", "parts")}
    for kind in ("silu", "gelu"):
        tested = set().union(*(plan(c[0], c[1]) for c in test_gpu_ffn_tiles.REAL if c[3] == kind))
        assert not many - tested, kind


def test_accumulation_reaches_both_ends(plan):
    tested = set().union(*(plan(c[0], c[1]) for c in test_gpu_ffn_tiles.ACCUM))
    for tile in DW:
        assert ("weights' gradients", tile, "parts") in tested
    assert any(k[0] == "dX with the weights' gradients" for k in tested)
    assert ("weights' gradients", "256 x 256", "whole") in tested


def test_calls_of_few_values_take_the_kernels_they_are_launched_on(plan):
    # ffn.hip launches one form of each for them, whatever the plan's tile
    for T in range(1, 65):
        for F in range(8, 8192 // T + 1, 8):
            for k in plan(T, F):
                if k[-1] == "two bf16":
                    assert k[0] in ("few", "hidden gradients") or k[:2] == ("dX with the weights' gradients", "128 x 64"), k
                    assert k[0] != "hidden gradients" or k[1] == "128 x 64"
