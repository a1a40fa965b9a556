"""What the binding and the Python classes around the experts check and hand on (no
GPU)."""

import pytest

torch = pytest.importorskip("torch")

import expanded_dispatch_layout_amd as M  # noqa: E402

CPU = -1                                             # what get_device() says of it


@pytest.mark.parametrize("pitch", [264, 265, 271, 1 << 31])
def test_a_single_row_has_no_distance_to_the_next(pitch):
    held = torch.empty(272, dtype=torch.bfloat16)
    for rows in (0, 1):
        view = held.as_strided((rows, 264), (pitch, 1))
        got = M._need_rows("f", "x", view, (torch.bfloat16,), (rows, 264), CPU)
        assert got == 264


def test_rows_apart_keep_their_distance():
    held = torch.empty((5, 272), dtype=torch.bfloat16)
    assert M._need_rows("f", "x", held[:, :264], (torch.bfloat16,), (5, 264), CPU) == 272
    for bad in (held[:, ::2][:, :100], held.t(), held[:1].expand(5, 272)):
        with pytest.raises(ValueError):
            M._need_rows("f", "x", bad, (torch.bfloat16,), bad.shape, CPU)
