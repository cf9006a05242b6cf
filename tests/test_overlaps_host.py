"""CPU checks of the overlaps that the adapter, checkpoint and input-gradient calls refuse: what
shares an element is refused before anything is enqueued, in every position."""

import ctypes
import os

import pytest

from post_weight_quantization_23_b200 import _lib

INVALID = 1
BASE = 1 << 32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from post_weight_quantization_23_b200 import build
        build.build()
    return _lib.load()


def _bytes(at, ld, cols, es, rows):
    return {at + r * ld * es + c for r in range(rows) for c in range(cols * es)}


def p(v):
    return ctypes.c_void_p(v)  # never dereferenced: only calls that are refused are made


def _shared(lib, at, ld, cols, es, pos, ldo, ocols, oes, rows, call):
    """call(lib, pos, ldo) must refuse where the two matrices share a byte; their number."""
    if not _bytes(at, ld, cols, es, rows) & _bytes(pos, ldo, ocols, oes, rows):
        return 0
    assert call(lib, pos, ldo) == INVALID, (pos - at, ldo)
    return 1


@pytest.mark.parametrize("ld", [64, 72, 200])
@pytest.mark.parametrize("rows", [1, 2, 4])
def test_dgrad_over_its_gradient(lib, ld, rows):
    # dY (rows, 64) with row pitch ld; dX (rows, 32) of the same pitch anywhere near it
    def call(lib, pos, ldo):
        return lib.gptq_gemm_dgrad(p(BASE), 1, rows, 64, ld, p(1 << 40), p(1 << 41), p(1 << 42), None,
                                   32, 4, 32, 1, p(pos), ldo, None)

    n = sum(_shared(lib, BASE, ld, 64, 2, BASE + 2 * o, ldo, 32, 2, rows, call)
            for ldo in {ld, 32, 100, 2 * ld} for o in range(-ld * rows - 40, ld * rows + 40))
    assert n > 100


@pytest.mark.parametrize("ld", [64, 96])
@pytest.mark.parametrize("rows", [1, 3])
def test_checkpoint_over_its_activations(lib, ld, rows):
    # codes of one byte with twice the leading dimension have the pitch of 16-bit values
    def call(lib, pos, ldo):
        return lib.gptq_act_checkpoint(p(BASE), 1, rows, 64, ld, p(pos), ldo, p(1 << 41), None)

    n = sum(_shared(lib, BASE, ld, 64, 2, BASE + o, ldo, 64, 1, rows, call)
            for ldo in {2 * ld, ld} for o in range(-2 * ld * rows - 70, 2 * ld * rows + 70))
    assert n > 100


@pytest.mark.parametrize("rows", [1, 2, 4])
def test_adapters_over_x_and_y(lib, rows):
    x, y, ld = BASE, 1 << 33, 80

    def call(lib, pos, ldo):
        return lib.gptq_lora_add(p(y), ld, p(x), 1, rows, 64, ld, p(1 << 40), p(1 << 41), p(1 << 42), 2, 16,
                                 p(1 << 43), p(1 << 44), 2, 32, p(pos), ldo, None, None)

    n = sum(_shared(lib, at, ld, cols, 2, at + 2 * o, ldo, 32, 2, rows, call)
            for at, cols in ((x, 64), (y, 32)) for ldo in (ld, 32) for o in range(-ld * rows, ld * rows + 40)
            if not (at == y and o == 0 and ldo == ld))
    assert n > 100
