"""Workspaces of the attention calls: attn_prefill's holds sums of real query rows, however the rows
are packed, and is bounded (CPU)."""
import pytest

import fp8_e4m3_quantization_amd as fq

MOST_PARTS, MOST_BYTES = 64, 256 << 20


@pytest.mark.parametrize("seqs,tq,tk,hq,d", [
    (39, 39, 39 * 8192, 40, 128), (39, 39, 39 * 8192, 40, 256),  # one-token chunks behind histories
    (15, 15, 15 * 131072, 40, 256), (6, 24042, 2582747, 8, 256), (1, 9590, 2610032, 16, 256),
    (1, 3210, 912658, 40, 256), (2, 1526, 3044908, 40, 256), (1, 512, 8704, 40, 128),
    (1, 23, 2794, 10, 128), (1, 1, 1 << 30, 64, 256), (200, 200, 1 << 22, 8, 64)])
def test_prefill_workspace_is_what_its_rows_need(seqs, tq, tk, hq, d):
    need = fq.attn_prefill_workspace_size(seqs, tq, tk, hq, hq, d)
    row = 4 * d + 16  # its sums, and their reference and totals
    assert need % (tq * hq * row) == 0 and need // (tq * hq * row) <= MOST_PARTS
    assert need <= MOST_BYTES
