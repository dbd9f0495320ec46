"""Limits of the entry points of include/fp8lin_train.h that test_train_abi.py
does not reach, without a GPU."""
from test_train_abi import A, HEADS, MASK, L, caller, refused, seqs


def test_scale_in_units_of_log2():
    """The kernels multiply logits by scale log2(e), which has to be finite too:
    2^127 log2(e) is, 2^128 / log2(e) and more is not."""
    rows = dict(q=A, qs=256, k=A, ks=128, v=A, vs=128)
    fwd = caller(L.fp8_attention_fwd, **rows, seqs=seqs(), **HEADS, **MASK, out=A, lse=A, stream=None)
    need = L.fp8_attention_bwd_workspace_bytes(seqs(), 4, 2, 64)
    bwd = caller(L.fp8_attention_bwd, dout=A, gs=256, **rows, out=A, lse=A, seqs=seqs(), **HEADS, **MASK, dq=A, dqs=256,
                 dk=A, dks=128, dv=A, dvs=128, ws=A, nbytes=need, stream=None)
    for call in (fwd, bwd):
        refused(call, "SIZE", dict(scale=2.4e38), dict(scale=-3.4e38), dict(scale=float("-inf")))
        for scale in (2.0 ** 127, -2.0 ** 127, 0.0, 1e-45):      # taken: what is refused here comes behind the scale
            refused(call, "NULL", dict(scale=scale, q=None))
