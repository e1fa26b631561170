"""Layer norm refuses outputs that share memory with its inputs, or with each other, other than
whole and in place: no GPU, nothing launched."""

import itertools

import pytest
import torch

from chunk_schedule_execution_amd import capi

X, R, OUT, TOTAL = (1 << 30 << i for i in range(4))
SIZE = 2  # bf16


def call(rows=8, width=40, x=X, residual=R, out=OUT, total=TOTAL, **ld):
    d = capi.ccl_norm_desc(dtype=capi.CCL_BF16, eps=1e-5, rows=rows, width=width, **ld)
    capi.ccl_layer_norm(d, x, residual, 0, 0, out, total, 0, 0)


def refused(text, **kw):
    with pytest.raises(capi.CCLError) as e:
        call(**kw)
    assert e.value.status == capi.CCL_ERR_INVALID_ARGUMENT and text in capi.ccl_last_error_detail()


def unrefused(**kw):
    """Comes as far as the launch, which finds no GPU here."""
    with pytest.raises(capi.CCLError) as e:
        call(**kw)
    assert e.value.status == capi.CCL_ERR_HIP, capi.ccl_last_error_detail()


def test_out_and_total_in_one_place():
    refused("out and total", out=OUT, total=OUT)
    refused("out and total", out=X, total=X)
    refused("out and total", out=R, total=R, x=R)
    refused("out and total", out=OUT, total=OUT + SIZE)
    refused("out and total", out=OUT, total=OUT + 7 * 40 * SIZE)
    refused("out and total", rows=1, out=OUT, total=OUT + 39 * SIZE)


@pytest.mark.parametrize("name,place", [("out", "x"), ("out", "residual"), ("total", "x"), ("total", "residual")])
def test_other_rows_of_an_input(name, place):
    base = X if place == "x" else R
    refused(f"{name}: memory of {place}", **{name: base + 40 * SIZE})
    refused(f"{name}: memory of {place}", **{name: base - 40 * SIZE})
    refused(f"{name}: memory of {place}", **{name: base + SIZE, f"ld_{name}": 41, f"ld_{place}": 41})
    # in place, but the rows further apart than the input's
    refused(f"{name}: memory of {place}", **{name: base, f"ld_{name}": 48})
    refused(f"{name}: memory of {place}", **{name: base + 32 * SIZE, f"ld_{name}": 48, f"ld_{place}": 48})


def bytes_of(base, ld, rows, width):
    return {base + (r * ld + c) for r in range(rows) for c in range(width)}


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would run on made-up addresses")
def test_every_arrangement_of_two_small_matrices():
    """Against the sets of their elements: what is refused is exactly what shares one and is not
    the same rows in place."""
    seen = set()
    for rows, width in ((1, 3), (2, 3), (4, 2), (3, 1)):
        for ld, ld_out in itertools.product(range(width, width + 5), repeat=2):
            for shift in range(-20, 21):
                inside = bytes_of(100, ld, rows, width)
                outside = bytes_of(100 + shift, ld_out, rows, width)
                same = shift == 0 and (ld == ld_out or rows == 1)
                kw = dict(rows=rows, width=width, out=X + shift * SIZE, total=0, ld_x=ld, ld_out=ld_out)
                if inside & outside and not same:
                    refused("out: memory of x", **kw)
                    seen.add("refused")
                else:
                    unrefused(**kw)
                    seen.add("same" if same else "apart")
    assert seen == {"refused", "same", "apart"}
