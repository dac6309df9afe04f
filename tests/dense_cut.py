"""The dense layer's own choice of kernels, compiled for the host from the header that makes it.

describe(...) names every kernel that a training step (forward and all gradients) of given sizes runs:
  small forward <type> fi=.. [split]      small gradients <type> fi=..
  <staged|direct> <type> <tile> <layouts> [split] [one buffer]     pad, slope
"""
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "qml_gradients_amd", "csrc")
TILES = ((64, 64), (128, 128), (256, 256), (64, 32), (32, 64))

SOURCE = r"""
#include "hqml_dense_cut.hpp"
using namespace hqml::gemm;
extern "C" void forward(int M, int K, int N, int elem, int xs, int ws, int words, int pad, int *o)
{
    const ForwardChoice f = choose_forward(M, K, N, elem, xs, ws, words, pad);
    const int v[] = {f.small, f.few.fi, f.few.waves, f.few.parts, f.tiles.shape, f.tiles.parts, f.direct, f.copy_x, f.copy_w};
    for (int k = 0; k < 9; ++k) o[k] = v[k];
}
extern "C" void backward(int M, int K, int N, int elem, int act, int dx, int dw, int dys, int xs, int ws, int words, int room,
                         int pad, int *o)
{
    const BackwardChoice b = choose_backward(M, K, N, elem, act, dx, dw, dys, xs, ws, words, room, pad);
    const int v[] = {b.small, b.few.fi, b.few.waves, b.dx.shape, b.dx.parts, b.dw.shape, b.dw.parts, b.direct, b.copy_x,
                     b.copy_w, b.form};
    for (int k = 0; k < 11; ++k) o[k] = v[k];
}
"""


def compile_choice(folder):
    """The choice as a library, built in `folder`."""
    src, lib = os.path.join(folder, "choice.cpp"), os.path.join(folder, "choice.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", lib, src])
    return ctypes.CDLL(lib)


def up(a, b):
    return -(-a // b)


def parts_of(K, parts):
    """Parts that are not empty: each takes a multiple of 32 of k."""
    return up(K, up(up(K, parts), 32) * 32)


def choose_forward(lib, M, K, N, dtype, x_straight, w_straight, words, pad):
    o = (ctypes.c_int * 9)()
    lib.forward(M, K, N, 2 if dtype == "bf16" else 4, x_straight, w_straight, words, pad, o)
    return dict(zip(("small", "fi", "waves", "few_parts", "shape", "parts", "direct", "copy_x", "copy_w"), o))


def choose_backward(lib, M, K, N, dtype, act, dx, dw, dy_straight, x_straight, w_straight, words, room, pad):
    o = (ctypes.c_int * 11)()
    lib.backward(M, K, N, 2 if dtype == "bf16" else 4, act, dx, dw, dy_straight, x_straight, w_straight, words, room, pad, o)
    return dict(zip(("small", "fi", "waves", "dx_shape", "dx_parts", "dw_shape", "dw_parts", "direct", "copy_x", "copy_w",
                     "form"), o))


def tile_name(dtype, direct, shape, layouts, I, J, K, parts):
    parts = parts_of(K, parts)
    rows, cols = TILES[shape]
    name = f"{'direct' if direct else 'staged'} {dtype} {rows}x{cols} {layouts}"
    if parts > 1:
        name += " split"
    if dtype == "fp32" and shape == 1 and up(I, rows) * up(J, cols) * parts > 256:
        name += " one buffer"
    return name


def describe(lib, M, K, N, dtype, offset=0, gap=0, act=True):
    """Arrays begin `offset` elements after a 16-byte boundary, with rows `gap` elements apart."""
    elem = 2 if dtype == "bf16" else 4

    def straight(length, across):
        return offset * elem % 16 == 0 and (length + gap) * elem % 16 == 0 and (across or length % 8 == 0)

    def word(length):
        return offset * elem % 4 == 0 and (length + gap) % 2 == 0

    pad = dtype == "bf16" and K % 8 != 0
    room = act or (dtype == "bf16" and N % 8 != 0)
    out = set()
    f = choose_forward(lib, M, K, N, dtype, straight(K, False), straight(K, False), word(K), pad)
    if f["small"]:
        out.add(f"small forward {dtype} fi={f['fi']}" + (" split" if parts_of(K, f["few_parts"]) > 1 else ""))
    else:
        out.add(tile_name(dtype, f["direct"], f["shape"], "rows rows", M, N, K, f["parts"]))
        if f["copy_x"] or f["copy_w"]:
            out.add("pad")
    b = choose_backward(lib, M, K, N, dtype, act, True, True, straight(N, False), straight(K, True), straight(K, True),
                        word(K) and word(N), room, pad)
    if b["small"]:
        out.add(f"small gradients {dtype} fi={b['fi']}")
    else:
        out.add(tile_name(dtype, b["direct"], b["dx_shape"], "rows cols", M, K, N, b["dx_parts"]))
        out.add(tile_name(dtype, b["direct"], b["dw_shape"], "cols cols", N, K, M, b["dw_parts"]))
        out.add("slope")
        if b["copy_x"] or b["copy_w"]:
            out.add("pad")
    return out
