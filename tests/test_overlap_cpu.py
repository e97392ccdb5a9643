"""Results that share memory with what a call reads, or with another result, at another
address than its start, are refused before any device work (no GPU here: the pointers are
never followed); columns of one wider matrix are not taken for that."""
import ctypes
import os
import shutil
import subprocess

import pytest

from packed_quantized_lm_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_overlap_against_every_byte(tmp_path):
    """overlap() of two buffers of rows against their sets of bytes, for all small layouts."""
    if not shutil.which("g++"):
        pytest.skip("g++ missing")
    (tmp_path / "all.cpp").write_text("""
#include "overlap.hpp"
#include <cstdio>
#include <vector>
using namespace archead;
int main()
{
    static char room[64];
    long wrong = 0, seen[2] = {};
    auto bytes = [&](const Span &s) {
        uint64_t set = 0;
        for (int64_t r = 0; r < s.rows; ++r)
            for (int64_t c = 0; c < s.width; ++c)
                set |= uint64_t(1) << (((const char *)s.at - room) + r * s.stride + c);
        return set;
    };
    std::vector<Span> all;
    for (int at = 0; at < 9; ++at)
        for (int rows = 0; rows < 5; ++rows)
            for (int stride = 1; stride < 8; ++stride)
                for (int width = 0; width <= stride; ++width)
                    all.push_back({room + 10 + at, rows, width, stride});
    for (const Span &a : all)
        for (const Span &b : all) {
            const bool want = (bytes(a) & bytes(b)) != 0;
            ++seen[want];
            wrong += overlap(a, b) != want;
        }
    const Span far{(void *)(uintptr_t(1) << 40), int64_t(1) << 31, 4, int64_t(1) << 42};
    wrong += overlap({room, 3, 4, 8}, {nullptr, 3, 4, 8}) || !overlap(far, far);
    printf("%ld %ld %ld\\n", wrong, seen[0], seen[1]);
    return wrong != 0;
}
""")
    exe = str(tmp_path / "all")
    p = subprocess.run(["g++", "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "packed_quantized_lm_amd", "csrc"),
                        str(tmp_path / "all.cpp"), "-o", exe], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([exe], capture_output=True, text=True)
    assert p.returncode == 0, p.stdout
    _, apart, shared = map(int, p.stdout.split())
    assert apart > 10000 and shared > 10000


A = [1 << (40 + i) for i in range(14)]  # far from each other


def _ptr(v):
    return ctypes.c_void_p(v)


def _refused(status, lib):
    assert status == binding.EINVAL
    assert "overlap" in lib.archead_last_error().decode()


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


M, D = 3, 32  # bf16 rows of 64 bytes


def _norm(lib, **over):
    b = dict(x=A[0], ldx=D, res=A[1], ldr=D, h=A[2], ldh=D, w=A[3], y=A[4], ldy=D, q=A[5], ldq=D, s=A[6])
    b.update(over)
    p = {k: _ptr(v) if not k.startswith("ld") else v for k, v in b.items()}
    return lib.archead_rms_norm(M, D, p["x"], 1, p["ldx"], p["res"], 1, p["ldr"], p["h"], p["ldh"], p["w"], 1, 1e-6, 0.0,
                                p["y"], 1, p["ldy"], p["q"], p["ldq"], p["s"], M, None)


@pytest.mark.parametrize("over", [
    dict(h=A[1] + 2), dict(h=A[1] + 64), dict(h=A[1] - 64), dict(h=A[0] + 130), dict(y=A[0] + 190), dict(y=A[0] - 190),
    dict(y=A[1] + 64), dict(y=A[2] + 4), dict(q=A[0] + 16), dict(q=A[1] + 64), dict(q=A[2] + 96), dict(q=A[4] + 32),
    dict(s=A[0] + 188), dict(s=A[5] + 92), dict(h=A[3] + 60), dict(y=A[3] - 128), dict(s=A[3] + 8), dict(q=A[3]),
    dict(h=A[1] + 32, ldr=64, ldh=64), dict(y=A[1] + 2, ldy=40), dict(h=A[1] - 130, ldh=64)])
def test_norm(lib, over):
    _refused(_norm(lib, **over), lib)


def _back(lib, n=1 << 20, **over):
    b = dict(u=A[0], h=A[1], w=A[2], res=A[3], dh=A[4], dw=A[5], ws=A[6])
    b.update(over)
    u, h, w, res, dh, dw, ws = (_ptr(v) for v in b.values())
    return lib.archead_rms_norm_backward(M, D, u, 1, D, h, 1, D, w, 1, 1e-6, 0.0, res, D, dh, D, dw, ws, n, None)


@pytest.mark.parametrize("over", [
    dict(dh=A[0] + 64), dict(dh=A[1] - 2), dict(dh=A[3] + 64), dict(dh=A[2] + 62), dict(dw=A[0] + 188), dict(dw=A[1]),
    dict(dw=A[2] + 4), dict(dw=A[3] + 4), dict(dw=A[4] + 64), dict(ws=A[0] + 16), dict(ws=A[3] - 16), dict(ws=A[4] + 176),
    dict(ws=A[5] + 112)])
def test_norm_backward(lib, over):
    _refused(_back(lib, **over), lib)


@pytest.mark.parametrize("over", [dict(out=A[0] + 64), dict(out=A[0] - 2), dict(out=A[1] + 8), dict(out=A[2] - 64),
                                  dict(out=A[0] + 32, ldo=24, ldt=40)])
def test_lookup(lib, over):
    b = dict(table=A[0], tok=A[1], scales=A[2], out=A[3], ldt=D, ldo=D)
    b.update(over)
    for tt, ot in ((1, 1), (2, 1)):
        if tt == 1 and b["out"] == A[2] - 64 or tt == 2 and b["ldt"] % 16:
            continue  # scales are of 8-bit tables, whose strides are multiples of 16
        d = 16 if b["ldo"] == 24 else D
        st = lib.archead_embed(M, 200, d, _ptr(b["table"]), tt, b["ldt"], _ptr(b["scales"]), 1, _ptr(b["tok"]), -1, 1.0,
                               _ptr(b["out"]), ot, b["ldo"], None)
        _refused(st, lib)


@pytest.mark.parametrize("over", [dict(grad=A[0] + 64), dict(grad=A[0] - 64), dict(grad=A[1] + 8), dict(ws=A[0] + 176),
                                  dict(ws=A[1]), dict(ws=A[2] + 16)])
@pytest.mark.parametrize("add", [0, 1])
def test_gradient(lib, over, add):
    b = dict(dout=A[0], tok=A[1], grad=A[2], ws=A[3])
    b.update(over)
    st = lib.archead_embed_backward(M, 200, D, _ptr(b["dout"]), 1, D, _ptr(b["tok"]), -1, 1.0, add, _ptr(b["grad"]), 1, D,
                                    _ptr(b["ws"]), 1 << 20, None)
    _refused(st, lib)


V = 100
RULES = dict(y=A[0], hist=A[1], lens=A[2], prompts=A[3], rep=A[4], freq=A[5], pres=A[6], ids=A[7], vals=A[8], mask=A[9],
             rows=A[10])


def _rules(b):
    p = {k: _ptr(b[k]) for k in RULES}
    return [M, V, p["y"], 0, V, p["hist"], 8, 8, p["lens"], p["prompts"], p["rep"], p["freq"], p["pres"], p["ids"], p["vals"],
            4, 4, p["mask"], 2, 4, p["rows"]]


IN = [(k, v + 4) for k, v in RULES.items()]  # the second element of each


@pytest.mark.parametrize("what,at", IN + [("before", A[0] - 4), ("between", A[0] + 400)])
def test_adjusted_logits(lib, what, at):
    _refused(lib.archead_adjust_logits(*_rules(RULES), _ptr(at), V, None, 0, None), lib)


@pytest.mark.parametrize("what,at", IN + [("taus", A[12] + 4), ("u", A[13] + 4)])
@pytest.mark.parametrize("result", ["values", "indices", "samples", "ws"])
def test_draw(lib, what, at, result):
    if result == "ws":  # aligned to 16 bytes, in front of it
        at = at - 4 - 16
    b = dict(values=A[11], indices=A[11] + 4096, samples=A[11] + 8192, ws=A[11] + 16384, taus=A[12], u=A[13])
    b[result] = at
    st = lib.archead_sample_logits(*_rules(RULES), 4, 1.0, _ptr(b["taus"]), _ptr(b["u"]), _ptr(b["values"]),
                                   _ptr(b["indices"]), _ptr(b["samples"]), _ptr(b["ws"]), 1 << 20, None)
    _refused(st, lib)


def test_results_of_a_draw_in_each_other(lib):
    for b in (dict(indices=A[11] + 44), dict(samples=A[11] + 4), dict(ws=A[11] + 32)):
        c = dict(dict(values=A[11], indices=A[11] + 4096, samples=A[11] + 8192, ws=A[11] + 16384), **b)
        st = lib.archead_sample_logits(*_rules(RULES), 4, 1.0, _ptr(A[12]), _ptr(A[13]), _ptr(c["values"]), _ptr(c["indices"]),
                                       _ptr(c["samples"]), _ptr(c["ws"]), 1 << 20, None)
        _refused(st, lib)
