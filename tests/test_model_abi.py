"""Refusals of the embedding, norm and cross-entropy entry points: every argument check runs on the host
before anything is enqueued (no GPU needed; the addresses are never read)."""
import ctypes

import pytest

import selective_state_space_17_amd as M

BASE = 0x7F0000000000
MB = 1 << 20
AT = [BASE + i * 100 * MB for i in range(16)]
INV, UNS, MIS, WS = M.MSSM_ERR_INVALID_ARG, M.MSSM_ERR_UNSUPPORTED, M.MSSM_ERR_MISALIGNED, M.MSSM_ERR_WORKSPACE


def desc(cls, **kw):
    base = {
        M.EmbeddingDesc: dict(tokens=8, vocab=32, dim=16, scale=1.0, io_dtype=M.MSSM_BF16, id_bytes=8, flags=0),
        M.NormDesc: dict(rows=8, dim=16, eps=1e-5, kind=M.MSSM_LAYER_NORM, io_dtype=M.MSSM_BF16,
                         res_dtype=M.MSSM_F32, flags=0),
        M.CrossEntropyDesc: dict(tokens=8, vocab=32, dim=64, ignore_id=-100, io_dtype=M.MSSM_BF16, id_bytes=8, flags=0),
    }[cls]
    base.update(kw)
    return cls(**base)


def ref(d):
    return None if d is None else ctypes.byref(d)


def embed_fwd(d, ids=AT[0], weight=AT[1], out=AT[2]):
    return M.lib.mssm_embedding_fwd(ref(d), ids, weight, out, None)


def embed_bwd(d, ids=AT[0], dout=AT[1], dweight=AT[2], gd=M.MSSM_BF16, acc=0, ws=AT[3], nb=MB):
    return M.lib.mssm_embedding_bwd(ref(d), ids, dout, dweight, gd, acc, ws, nb, None)


def norm_fwd(d, x=AT[0], residual=AT[1], weight=AT[2], bias=AT[3], out=AT[4], residual_out=AT[5], mean=AT[6], rstd=AT[7]):
    return M.lib.mssm_norm_fwd(ref(d), x, residual, weight, bias, out, residual_out, mean, rstd, None)


def norm_bwd(d, h=AT[0], weight=AT[1], mean=AT[2], rstd=AT[3], dout=AT[4], dres=AT[5], dx=AT[6], dres_in=AT[7],
             dweight=AT[8], dbias=AT[9], ws=AT[10], nb=MB):
    return M.lib.mssm_norm_bwd(ref(d), h, weight, mean, rstd, dout, dres, dx, dres_in, dweight, dbias, ws, nb, None)


def xent_fwd(d, x=AT[0], weight=AT[1], targets=AT[2], loss=AT[3], lse=AT[4], ws=AT[5], nb=90 * MB):
    return M.lib.mssm_linear_cross_entropy_fwd(ref(d), x, weight, targets, loss, lse, ws, nb, None)


def xent_bwd(d, x=AT[0], weight=AT[1], targets=AT[2], lse=AT[3], dloss=AT[4], dlse=AT[5], dx=AT[6], dweight=AT[7],
             gd=M.MSSM_BF16, acc=0, ws=AT[8], nb=90 * MB):
    return M.lib.mssm_linear_cross_entropy_bwd(ref(d), x, weight, targets, lse, dloss, dlse, dx, dweight, gd, acc, ws,
                                               nb, None)


E, N, X = M.EmbeddingDesc, M.NormDesc, M.CrossEntropyDesc


@pytest.mark.parametrize("call,cls", [(embed_fwd, E), (embed_bwd, E), (norm_fwd, N), (norm_bwd, N), (xent_fwd, X),
                                      (xent_bwd, X)])
def test_descriptors(call, cls):
    size = "rows" if cls is N else "tokens"
    assert call(None) == INV
    for kw, want in (({size: -1}, INV), ({"dim": 0}, INV), ({"dim": -3}, INV), ({"flags": 1}, INV),
                     ({"io_dtype": 7}, UNS), ({size: 1 << 27}, UNS), ({"dim": 1 << 21}, UNS),
                     ({size: 1 << 60, "dim": 1 << 20}, INV)):
        assert call(desc(cls, **kw)) == want, kw
    if cls is not N:
        for kw, want in (({"vocab": 0}, INV), ({"vocab": (1 << 30) + 1, "dim": 64}, UNS), ({"id_bytes": 2}, UNS),
                         ({"vocab": 1 << 62}, INV)):
            assert call(desc(cls, **kw)) == want, kw


def test_embedding_arguments():
    d = desc(E)
    for scale in (float("nan"), float("inf")):
        assert embed_fwd(desc(E, scale=scale)) == INV
    most = (1 << 26) - 4
    assert embed_fwd(desc(E, tokens=most + 1, dim=1)) == UNS and embed_fwd(desc(E, tokens=most, dim=1), ids=None) == INV
    assert embed_fwd(d, ids=None) == INV and embed_fwd(d, weight=None) == INV and embed_fwd(d, out=None) == INV
    assert embed_fwd(d, ids=AT[0] + 4) == MIS and embed_fwd(d, weight=AT[1] + 1) == MIS and embed_fwd(d, out=AT[2] + 1) == MIS
    assert embed_fwd(d, out=AT[1]) == INV and embed_fwd(d, out=AT[0] - 100) == INV
    assert embed_fwd(desc(E, tokens=0), ids=None, out=None) == M.MSSM_OK
    assert embed_bwd(d, ids=None) == INV and embed_bwd(d, dout=None) == INV and embed_bwd(d, dweight=None) == INV
    assert embed_bwd(d, gd=5) == UNS and embed_bwd(desc(E, io_dtype=M.MSSM_F32), gd=M.MSSM_BF16) == UNS
    assert embed_bwd(d, dweight=AT[2] + 1) == MIS and embed_bwd(d, ws=AT[3] + 8) == MIS
    need = M.embedding_bwd_workspace_size(8, 32, 16)
    assert need > 0 and embed_bwd(d, nb=need - 1) == WS and embed_bwd(d, ws=None) == WS
    assert embed_bwd(d, dweight=AT[1]) == INV and embed_bwd(d, ws=AT[2]) == INV and embed_bwd(d, ws=AT[1]) == INV
    assert M.embedding_bwd_workspace_size(8, 0, 16) == 0 and M.embedding_bwd_workspace_size(0, 8, 16) == 0


def test_norm_arguments():
    d = desc(N)
    for kw in ({"eps": 0.0}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"kind": 2}):
        assert norm_fwd(desc(N, **kw)) == INV, kw
    assert norm_fwd(desc(N, io_dtype=M.MSSM_F32, res_dtype=M.MSSM_BF16)) == UNS
    assert norm_fwd(desc(N, res_dtype=3)) == UNS
    assert norm_fwd(desc(N, rows=1 << 22, dim=257)) == UNS
    most = (1 << 26) - 4
    assert norm_fwd(desc(N, rows=most + 1, dim=1)) == UNS and norm_fwd(desc(N, rows=most, dim=1), x=None) == INV
    rms = desc(N, kind=M.MSSM_RMS_NORM)
    assert norm_fwd(rms, mean=None) == INV, "the RMS norm has no bias"
    assert norm_fwd(rms, bias=None) == INV, "nor a mean"
    assert norm_bwd(rms, mean=None) == INV and norm_bwd(rms, dbias=None) == INV
    assert norm_fwd(d, residual_out=None) == INV, "a residual that is added is kept"
    for k in ("x", "weight", "out"):
        assert norm_fwd(d, **{k: None}) == INV, k
    for k in ("h", "weight", "mean", "rstd", "dout", "dweight"):
        assert norm_bwd(d, **{k: None}) == INV, k
    assert norm_bwd(d, dx=None, dres_in=None) == INV
    assert norm_fwd(d, x=AT[0] + 1) == MIS and norm_fwd(d, residual=AT[1] + 2) == MIS and norm_fwd(d, weight=AT[2] + 2) == MIS
    assert norm_bwd(d, h=AT[0] + 2) == MIS and norm_bwd(d, dres_in=AT[7] + 2) == MIS
    assert norm_fwd(d, out=AT[0]) == INV and norm_fwd(d, residual_out=AT[1]) == INV and norm_fwd(d, residual_out=AT[4]) == INV
    assert norm_bwd(d, dx=AT[4]) == INV and norm_bwd(d, dres_in=AT[5]) == INV and norm_bwd(d, dweight=AT[9]) == INV
    need = M.norm_bwd_workspace_size(8, 16)
    assert norm_bwd(d, nb=need - 1) == WS and norm_bwd(d, ws=None) == WS and norm_bwd(d, ws=AT[10] + 4) == MIS
    assert norm_fwd(desc(N, rows=0), x=None, out=None, weight=None) == M.MSSM_OK


def test_cross_entropy_arguments():
    d = desc(X)
    for k in ("x", "weight", "targets", "loss", "lse"):
        assert xent_fwd(d, **{k: None}) == INV, k
    for k in ("x", "weight", "targets", "lse", "dloss"):
        assert xent_bwd(d, **{k: None}) == INV, k
    assert xent_bwd(d, dx=None, dweight=None) == INV
    assert xent_bwd(d, gd=9) == UNS and xent_bwd(desc(X, io_dtype=M.MSSM_F32), gd=M.MSSM_BF16) == UNS
    assert xent_fwd(d, weight=AT[1] + 8) == MIS, "a weight read in place is read 16 bytes at a time"
    assert xent_fwd(d, x=AT[0] + 1) == MIS and xent_fwd(d, targets=AT[2] + 4) == MIS and xent_fwd(d, loss=AT[3] + 2) == MIS
    assert xent_bwd(d, dx=AT[6] + 1) == MIS and xent_bwd(d, dweight=AT[7] + 1) == MIS and xent_bwd(d, dlse=AT[5] + 1) == MIS
    assert xent_fwd(d, loss=AT[4]) == INV and xent_fwd(d, lse=AT[2]) == INV
    assert xent_bwd(d, dx=AT[0]) == INV and xent_bwd(d, dweight=AT[1]) == INV and xent_bwd(d, dx=AT[7]) == INV
    need = M.linear_cross_entropy_fwd_workspace_size(8, 32, 64)
    assert need > 0 and xent_fwd(d, nb=need - 1) == WS and xent_fwd(d, ws=None) == WS and xent_fwd(d, ws=AT[5] + 16) == MIS
    need = M.linear_cross_entropy_bwd_workspace_size(8, 32, 64)
    assert need > 0 and xent_bwd(d, nb=need - 1) == WS and xent_bwd(d, ws=AT[7]) == INV
    assert xent_fwd(desc(X, tokens=0), x=None, targets=None, loss=None, lse=None) == M.MSSM_OK
    assert M.linear_cross_entropy_bwd_workspace_size(8, 0, 64) == 0


def test_workspaces_stay_bounded():
    """The loss needs no [tokens, vocab] of anything: its workspace grows with the tokens, not with the vocabulary."""
    for io in (M.MSSM_BF16, M.MSSM_F32):
        t, d = 32768, 2048
        x = t * d * (2 if io == M.MSSM_BF16 else 6)
        fwd = M.linear_cross_entropy_fwd_workspace_size(t, 1 << 20, d, io)
        bwd = M.linear_cross_entropy_bwd_workspace_size(t, 1 << 20, d, io)
        assert fwd < x + (1100 << 20) and bwd < x + t * d * 4 + (1100 << 20), (fwd, bwd)
        # (the whole logits would be 128 GiB)
    # many tokens and a wide table keep at least 256 vocabulary rows a piece
    assert M.linear_cross_entropy_bwd_workspace_size((1 << 26) - 1, 1 << 30, 64) > 0
