"""The append tests' helpers against the packing of the other paged tests, without a GPU."""
import numpy as np
import pytest
import torch

from oracle import oracle
from tests import append_testlib as A
from tests import paged_testlib as P


def test_check_q4_takes_the_definition_and_nothing_else():
    rows = A.Rows("q4", [5, 0, 40], [3, 9, 70], 32, pad_rows=2)
    kv = A.draw(1, 2, rows.M, 2, 256).double().numpy()
    kv[0, 8, 1, 70] = np.nan
    kv[1, 9] = 0.0
    rec = torch.full(rows.shape, 0xFF, dtype=torch.uint8)
    for m in rows.stored():
        r = rows.off[m] % 16
        line = rec[rows.page_id[m], :, rows.off[m] // 16].numpy()
        for x, at, sz in ((kv[0, m], 0, 4096), (kv[1, m], 2048, 4352)):
            c, s, z, _ = oracle.kv4(x)
            c = np.where(np.isnan(z)[..., None], 0, c)
            line[:, at + 128 * r:at + 128 * r + 128] = P.row_bytes(c)
            line[:, sz + 16 * r:sz + 16 * r + 16] = P.bf16_bytes(np.stack([s, z], -1)).reshape(2, 16)
    assert len(rows.stored()) == 43 and rows.pos[0] == -2
    A.check_q4(rows, rec, *kv)
    for spot in ((rows.page_id[20], 1, rows.off[20] // 16, 128 * (rows.off[20] % 16) + 5), (rows.page_id[2], 0, 1, 700)):
        wrong = rec.clone()
        wrong[spot] ^= 1
        with pytest.raises(AssertionError):
            A.check_q4(rows, wrong, *kv)
