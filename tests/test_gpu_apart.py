"""Outputs that lie between the elements of another argument are taken, outputs that share one are refused."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_row_between_the_rows_of_an_output(cuda_lib, dt):
    buf = torch.randn(6, 64, device="cuda").to(dt)
    x, w, b = torch.randn(6, 24, device="cuda").to(dt), buf[2, 24:48].clone(), buf[5, 40:64].clone()
    want = api.lce_layer_norm_forward(x, w, b)
    kept = buf.clone()
    kept[:, :24] = want
    got = api.lce_layer_norm_forward(x, buf[2, 24:48], buf[5, 40:64], out=buf[:, :24])
    assert torch.equal(got, want) and torch.equal(buf, kept)
    # the other way round: one row written between the rows that are read
    one = api.lce_layer_norm_forward(buf[1:2, :24], out=buf[3:4, 24:48])
    assert torch.equal(one, api.lce_layer_norm_forward(kept[1:2, :24]))
    # a table of one row between the rows of the result
    table = buf[4:5, 24:48]
    y, _ = api.lce_embedding_forward(torch.zeros(6, dtype=torch.int64, device="cuda"), table, out=buf[:, :24])
    assert torch.equal(y, table.expand(6, 24))


def test_shared_elements_are_refused(cuda_lib):
    buf = torch.randn(6, 64, device="cuda")
    x = torch.randn(6, 24, device="cuda")
    for w in (buf[2, 23:47], buf[2, 41:].as_strided((24,), (1,), 2 * 64 + 41), buf[0, :24], buf[5, :24], buf[2, 10:34]):
        with pytest.raises(ValueError, match="shares memory"):
            api.lce_layer_norm_forward(x, w, out=buf[:, :24])
    with pytest.raises(ValueError, match="shares memory"):          # wider than the gap
        api.lce_layer_norm_forward(x[:, :8], out=buf.view(-1)[:48].view(6, 8), weight=buf[0, 40:48])
    with pytest.raises(ValueError, match="shares memory"):
        api.lce_layer_norm_forward(buf[:, :24], out=buf.as_strided((6, 24), (64, 1), 12))
    with pytest.raises(ValueError, match="shares memory"):          # a row over the step of the others
        api.lce_layer_norm_forward(torch.randn(1, 64, device="cuda"), out=buf.view(-1)[30:94].view(1, 64),
                                   weight=buf.view(-1)[64:128])
