"""Attention over the cache in the form that each call takes: rows of a tile and
workgroups, as the size of the workspace shows them, and whether it is cut."""
import ctypes

import numpy as np
import pytest
import torch

import attention_refs as refs
from gpu_helpers import note, to_dev
from q4_q8_integer_amd import binding as b
from test_kv_attend_gpu import FMT, Case

pytestmark = pytest.mark.gpu


def workspace(c, most, window=0, out_half=None, width=None):
    n = ctypes.c_int64()
    out_half = c.half if out_half is None else out_half
    rc = b.load_library().kv_attend_workspace(
        b.CacheArgs(0, len(c.data), c.heads, c.dim, c.page, FMT[c.bits]),
        b.PlanArgs(0, 0, 1, len(c.lengths), width or c.table.shape[1], 0),
        b.QueryArgs(n=c.n, most=most, heads=c.heads * c.group, q_half=c.half, out_half=out_half, window=window, scale=1.0), n)
    assert rc == 0
    return n.value


def form(c, most, **kw):
    """(rows of a tile, runs) of the call, as it would be over a table that has to be cut."""
    size = workspace(c, most, width=8192 // c.page, **kw)
    found = [(rows, size // per) for rows in (16, 32, 64, 128) for per in (2 * rows * (4 * c.dim + 8) + 32,)
             if size % per == 0 and size // per in (256, 512, 768)]
    assert len(found) == 1, (size, found)
    return found[0]


def check_some(c, out, lse, s, rows, window=0):
    """Rows (of the sequence) of all heads against 64 bits."""
    a, new, length = int(c.offsets[s]), c.new[s], int(c.lengths[s])
    for i in rows:
        q = c.q[a + i:a + i + 1].reshape(1, -1, c.dim)
        ref, l, tol = refs.attend(q, c.k[s], c.v[s], np.ones(length, bool), length - new + i, c.group, c.dim ** -0.5, window,
                                  not c.half)
        refs.check(out[a + i:a + i + 1], ref.reshape(1, -1), tol.reshape(1, -1), c.half, "sequence %d row %d" % (s, i))
        assert (np.abs(lse[a + i] - l[0]) <= 2e-4 + 4e-7 * np.abs(l[0])).all()


@pytest.mark.parametrize("half,bits,window", [(True, 8, 0), (False, 4, 0), (True, 4, 700)])
def test_prompt_uncut_past_short_contexts(half, bits, window):
    """One sequence's tiles that fill the chip go uncut on a table of any length."""
    c = Case(101, 32, 1, 32, 64, bits, [2150], [2050], half)
    assert c.table.shape[1] * c.page > 1280 and workspace(c, 2050, window) == 0
    note("uncut prompt half=%d bits=%d window=%d" % (half, bits, window))
    out, lse = c.run(window, most=2050)
    torch.cuda.synchronize()
    out, lse = out.cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    check_some(c, out, lse, 0, [0, 1, 15, 16, 31, 127, 128, 129, 1023, 1919, 1920, 2047, 2048, 2049], window)


FORMS = [
    # dim, bits, group, most, sequences, rows of a tile, waves' form
    (64, 8, 4, 4, 2, 16), (128, 8, 4, 4, 2, 16), (160, 4, 16, 1, 2, 16),        # up to 16 rows
    (64, 8, 17, 1, 3, 64), (128, 4, 9, 2, 70, 64), (192, 8, 17, 1, 3, 32),      # from 17, few tiles
    (64, 8, 20, 3, 260, 64), (96, 8, 10, 5, 260, 64), (128, 4, 20, 1, 260, 64), (160, 8, 20, 3, 140, 32),   # many
    (64, 8, 20, 5, 135, 64), (32, 4, 42, 3, 135, 64),                            # in two tiles and more
    (160, 8, 8, 8, 3, 32), (256, 4, 32, 2, 3, 32), (160, 8, 13, 5, 3, 128), (256, 4, 13, 5, 3, 128),   # 64 and 65 rows
    (64, 8, 127, 1, 3, 64), (64, 8, 32, 4, 3, 128), (128, 8, 17, 1, 3, 128), (96, 4, 17, 1, 3, 128),   # the tall ones
]


@pytest.mark.parametrize("dim,bits,group,most,seqs,rows", FORMS)
@pytest.mark.parametrize("half", [False, True])
def test_forms(dim, bits, group, most, seqs, rows, half):
    """Each border of the choice on both sides, over short contexts and, cut,
    over a longer table."""
    rng = np.random.default_rng([102, dim, group])
    lengths = [int(x) for x in rng.integers(0, 40, seqs)]
    lengths[0], lengths[1], lengths[-1] = 200, 33, 90
    new = [min(most, max(l, 1)) for l in lengths]
    c = Case(102, 1, group, dim, 16, bits, lengths, new, half)
    assert max(new) == most and form(c, most)[0] == rows
    c.both(most=most)


@pytest.mark.parametrize("dim,bits,half,group,new,seqs,rows", [
    (64, 8, True, 4, 4, 2, 16), (128, 4, False, 4, 4, 2, 16), (160, 8, False, 4, 4, 2, 16), (256, 8, True, 2, 8, 2, 16),
    (64, 8, True, 4, 20, 2, 64), (128, 4, False, 4, 20, 140, 64), (160, 8, False, 4, 12, 2, 32),     # wide
    (64, 8, False, 4, 20, 150, 64), (32, 4, True, 8, 8, 270, 64), (192, 8, True, 4, 12, 140, 32),    # of 4 waves
    (128, 8, False, 4, 6, 2, 128), (64, 4, True, 4, 40, 2, 128)])
def test_hidden_tokens_leave_rows_of_each_form(dim, bits, half, group, new, seqs, rows):
    """The last token of a call is no number, or has values 2^17 times the others':
    rows that do not see it keep their bits."""
    lengths = [180] + [3] * (seqs - 2) + [64]
    c = Case(103, 1, group, dim, 16, bits, lengths, [new] + [1] * (seqs - 1), half)
    assert form(c, new)[0] == rows
    wide = c.table
    for more in (0, 1280 // 16):                            # and cut
        c.table = np.concatenate((wide, np.full((seqs, more), -1, np.int32)), 1)
        want, lse = c.run(most=new)
        torch.cuda.synchronize()
        c.check(want, lse)
        parts, sb = refs.record_parts(dim, 16, bits), dim // 16
        rec = c.data[c.table[0, 179 // 16], 0]
        at = rec[parts[3] + 179 % 16 * sb:][:sb]
        was = at.copy()
        for what in (np.nan, np.inf, 6e4):
            at[:] = np.full(sb // 2, what, np.float16).view(np.uint8)
            out, l2 = c.run(most=new)
            torch.cuda.synchronize()
            for got, w in ((out, want), (l2, lse)):
                assert torch.equal(got[:new - 1], w[:new - 1]) and torch.equal(got[new:], w[new:])
            # the row that sees it: its references go by its values, its weights do not
            assert (l2[new - 1] - lse[new - 1]).abs().max() <= 4e-7 * lse[new - 1].abs().max() + 2e-4
            assert what == 6e4 or not torch.isfinite(out[new - 1]).any()
        at[:] = was


def test_tiles_of_several_sequences_are_cut():
    """A chunk, a long history and a short one in one call: as many tiles as fill the
    chip, but their lengths may differ, so that they are cut."""
    c = Case(104, 8, 2, 32, 64, 8, [2048, 9000, 5], [2048, 2, 1], True)
    assert workspace(c, 2048) > 0
    out, lse = c.run(most=2048)
    torch.cuda.synchronize()
    out, lse = out.cpu().numpy(), lse.cpu().numpy()
    check_some(c, out, lse, 0, [0, 63, 64, 1000, 2047])
    check_some(c, out, lse, 1, [0, 1])
    check_some(c, out, lse, 2, [0])
