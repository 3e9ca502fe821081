"""What the cross entropy's C calls take and refuse before any device work (no GPU)."""
import vocab_selected_token_tile_gb300 as rlk


def contract(**kw):
    base = dict(T=8, V=1000, H=64)
    base.update(kw)
    return rlk.LinearCeContract(**base)


def test_no_rows_need_no_output(built):
    # a frozen head's step of an empty batch: its dhidden has no element and so no address
    assert rlk.rlk_linear_ce_bwd(contract(T=0), *[None] * 10) == rlk.RLK_OK
    assert rlk.rlk_linear_ce_bwd(contract(T=1), *[None] * 10) == rlk.RLK_ERR_INVALID_ARG
